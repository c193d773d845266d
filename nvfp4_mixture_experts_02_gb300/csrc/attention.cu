// Attention of one new token per sequence over a paged key-value cache.
//
//   s_j = scale * k_scale * (q . k_j)    for j in [max(0, len - window), len)
//   out = sum_j exp(s_j - m) v_scale v_j / sum_j exp(s_j - m),  m = max_j s_j
//   lse = m + ln(sum_j exp(s_j - m));   an empty sequence: out = 0, lse = -inf
//
// Every key and value is read once, by one block, for up to 16 query heads that share it, and once more
// for every 16 beyond: the call is bound by the cache's bytes (4 G operations per key element of 1 or 2
// bytes).
//
// k_attend: the work is the list of (sequence, key heads, unit of keys), in that order; every block
// takes an equal run of it, whatever the lengths, found from the lengths on the device (no host
// synchronisation). A run covers pieces of one or more (sequence, key heads) segments. Inside a piece
// each warp has a key head, or shares it with others and takes 16 or 32 keys in turn, with its own ring of
// asynchronous 16-byte copies (rows of the pages to swizzled shared memory), its own running maximum and
// sum and its own 16 x D sums in registers; a head's warps are joined at the piece's end. A piece that
// is its whole segment is finished there; the others leave (maximum, sum, sums) in the workspace for
// k_join, which adds a segment's pieces in order. Masked and missing keys are not read: their rows are
// zeros in shared memory, so that whatever the pages hold there (NaN, stale values) cannot reach a sum.
//
// Products, m16n8k16 with float32 sums, the query heads as the eight columns (two groups of columns for
// nine to sixteen heads): s^T = k q^T and o^T = v^T p^T, so that all 16 rows are keys, then dims, and
// the operands read from shared memory serve every head. The weights p leave s^T's register layout for
// the other operand's by movmatrix. bf16 caches: bf16 operands; p, in (0, 1], is split into two bf16
// (16 significant bits, so that p is not rounded to 8). E4M3 caches: keys and values become f16
// exactly, q is f16 after a scaling of its row by a power of two (exact but for elements under 2^-29
// of the row's largest), p, in (0, 2^15], is split into two f16 (22 bits down to 2^-18 of the largest key's
// weight, see kLift). One f16 for p moves outputs over their bf16 rounding: 48 ragged sequences are 8.1e-4 off the
// rounded exact result with one, 0.8e-4 with two (bf16 caches 0.6e-4), at 0 to 1 % of the time, 4 to 5 % with heads
// of 64 (200 ragged sequences up to 700, 26.3 and 27.5 us) or 16 heads a key head (16 x 8192, 40.9 and 43.2 us).
// Statistics and sums are float32.
//
// Measured (of the copy rate of 6786 GB/s): three sequences up to 131072, bf16, 962 MB: 155 us (91 %).
// 48 ragged ones up to 8192, E4M3, 423 MB: 85 us (73 %), of which some 10 us are launches, fill and
// join, and the runs' pieces differ in cost. One sequence of 777: 7.8 us, two launches and the chain
// length, page, keys, scores, sums, join.
#include <cmath>
#include <cuda_runtime.h>

#include "ftmoe_internal.h"
#include "ftmoe_mma.cuh"
#include "ftmoe_tc.cuh"

namespace ftmoe {

namespace {

template <int D, bool F8, int NG>
struct AttnShape {
  static constexpr int kRow = D * (F8 ? 1 : 2);       // bytes of a key or value
  static constexpr int kCpr = kRow / 16;              // 16-byte pieces of it
  static constexpr int kKeys = kRow <= 128 ? 32 : 16; // keys of a warp's step
  static constexpr int kStageBytes = 2 * kKeys * kRow;   // those keys and values
  // blocks an SM: the others stream while one joins a piece's warps. Three of two stages each, not two of
  // three, where the registers allow it: 256 sequences up to 1024 with 8-bit keys of 128: 68 us for 79.
  // (Past some 2600 sequences their running sums in shared memory leave room for two.)
  static constexpr int kBlocks = kRow >= 512 ? 1 : kRow == 128 && NG == 1 ? kAttendBlocks : 2;
  static constexpr int kWarps = kRow >= 128 ? 4 : 8;
  static constexpr int kStages = 192 * 1024 / (kBlocks * kWarps * kStageBytes);
  static constexpr int kUnit = kKeys * kWarps;        // keys of a unit
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  static constexpr int kSumsLd = D + 4;               // floats between heads of a warp's sums, in its ring
  static_assert(8 * NG * kSumsLd * 4 <= kStages * kStageBytes && kBlocks * kWarps <= attend_warps(D));
};

// From this many units in a run, the warps of a block take several key heads at once instead of stripes of
// one head's keys: rows of the same slot are then read together (256 sequences up to 1024, bf16, 8 heads of
// 128: 97 us for 118; 8 of 32768, E4M3, 8 heads of 64: 54 for 80), and no join in the block holds the
// copies up. Shorter runs would leave k_join as many times more pieces: 48 sequences of 256 take 12.8 us, and
// 17.0 when runs of two units are long; 8 up to 2048 take 14.0 us, and 15.5 when only runs of eight are.
constexpr int kLongRun = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// log2 of the largest weight. f16 holds 11 bits of weights down to 2^-14 and nothing under 2^-25: with
// weights of up to 2^15 the two parts of a key's weight hold 22 bits of it, or all but 2^-40 of the largest
// key's weight. The sums carry the same factor, which their quotient does not see.
constexpr float kLift = 15.f;
template <bool F8>
__device__ __forceinline__ float lse_of(float m, float l) {   // ln of l 2^m
  return F8 ? (m + kLift + log2f(l * (1.f / 32768.f))) * kLn2 : (m + log2f(l)) * kLn2;
}

// Offset of 16-byte piece c of row r in a tile of rows of kCpr pieces: pieces are exchanged within
// groups of eight (four) so that eight rows' same piece lie in different banks.
template <int CPR>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  if constexpr (CPR >= 8) return (uint32_t)(r * CPR + (c ^ (r & 7))) * 16;
  else return (uint32_t)(r * CPR + (c ^ ((r >> 1) & 3))) * 16;
}

__device__ __forceinline__ uint32_t transpose8(uint32_t v) {   // an 8 x 8 matrix of 16-bit elements
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}

// Four E4M3 bytes -> f16x2 of the lower two and of the upper two, exact.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t v, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi) : "r"(v));
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Four values of an output row, divided by the weights' sum (no weight at all: zeros).
__device__ __forceinline__ void store_row(const AttendArgs& a, int64_t at, float4 v, float sum) {
  uint2 y = make_uint2(0, 0);
  if (!(sum == 0.f)) {
    const float s = a.kv.v_scale;
    y = make_uint2(pack_bf16(v.x / sum * s, v.y / sum * s), pack_bf16(v.z / sum * s, v.w / sum * s));
  }
  *reinterpret_cast<uint2*>(a.out + at) = y;
}

// A sequence's length, cut to what its row of the block table can hold.
__device__ __forceinline__ int length_of(const AttendArgs& a, int b) { return min(a.seq_lens[b], a.max_len); }

// First key and number of units of a sequence.
__device__ __forceinline__ void span(int len, int window, int unit, int& first, int& units) {
  first = window > 0 && len > window ? len - window : 0;
  units = len > 0 ? (len + unit - 1) / unit - first / unit : 0;
}

template <int D, bool F8, int NG>
__global__ void __launch_bounds__(AttnShape<D, F8, NG>::kWarps * 32, AttnShape<D, F8, NG>::kBlocks)
    k_attend(const AttendArgs a) {
  using S = AttnShape<D, F8, NG>;
  constexpr int W = S::kWarps, ST = S::kStages, CPR = S::kCpr, KS = D / 16, MT = D / 16;
  constexpr int KT = S::kKeys, NH = KT / 16;   // keys of a step, in 16-row tiles
  constexpr int LD = S::kSumsLd;
  constexpr int kUnitLog2 = S::kUnit == 64 ? 6 : S::kUnit == 128 ? 7 : 8;
  static_assert(S::kUnit == 1 << kUnitLog2);
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ float wm[W][16], wl[W][16], share[W][16];
  __shared__ int scan[W];
  int* cum = reinterpret_cast<int*>(smem + S::kRing);   // [B + 1] units before each sequence (B > 32)
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = lane & 3, r = lane >> 2;
  const int HS = a.kv.Hkv * a.gt;   // segments of a sequence

  // units before each sequence: in every warp's lanes, or in shared memory past 32 sequences
  int inc = 0;       // B <= 32: units up to and with sequence `lane`
  int all;
  if (a.B <= 32) {
    int first, n = 0;
    if (lane < a.B) {
      const int len = length_of(a, lane);
      span(len, a.window, S::kUnit, first, n);
      if (blockIdx.x == 0 && warp == 0 && a.seq_lens[lane] > len) atomicOr(a.err, kErrBadPage);
    }
    inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    all = __shfl_sync(0xffffffffu, inc, 31);
  } else {
    const int per = (a.B + W * 32 - 1) / (W * 32);
    const int b0 = threadIdx.x * per;
    int mine = 0;
    for (int b = b0; b < min(b0 + per, a.B); ++b) {
      int first, n;
      const int len = length_of(a, b);
      span(len, a.window, S::kUnit, first, n);
      mine += n;
      if (blockIdx.x == 0 && a.seq_lens[b] > len) atomicOr(a.err, kErrBadPage);
    }
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) scan[warp] = upto;
    __syncthreads();
    int at = upto - mine;
    for (int w = 0; w < warp; ++w) at += scan[w];
    for (int b = b0; b < min(b0 + per, a.B); ++b) {
      int first, n;
      span(length_of(a, b), a.window, S::kUnit, first, n);
      cum[b] = at;
      at += n;
    }
    if (b0 < a.B && b0 + per >= a.B) cum[a.B] = at;
    __syncthreads();
    all = cum[a.B];
  }
  const int64_t total = (int64_t)all * HS;
  const int64_t quota = (total + gridDim.x - 1) / gridDim.x;
  int64_t u = quota * blockIdx.x;
  const int64_t u_end = min(u + quota, total);
  const uint32_t ring = smem_addr(smem) + (uint32_t)(warp * ST * S::kStageBytes);
  // HW heads a block, W / HW stripes of keys each
  const int hl = quota >= kLongRun ? a.heads_log2 : 0, HW = 1 << hl, stripes = W >> hl;
  const int hw = warp & (HW - 1), stripe = warp >> hl;
  const int unit = S::kUnit >> hl;
  auto sync = [&]() {   // the warps that share a head
    if (stripes == 1) __syncwarp();
    else __syncthreads();
  };
  if (u >= u_end && threadIdx.x == 0) a.shared_segs[blockIdx.x] = make_int4(-1, 0, 0, 0);

  while (u < u_end) {
    // the piece that begins at u: sequence b, with `before` units ahead of it
    int b, before;
    if (a.B <= 32) {
      b = __ffs(__ballot_sync(0xffffffffu, (int64_t)inc * HS > u)) - 1;
      before = __shfl_sync(0xffffffffu, inc, b > 0 ? b - 1 : 0);
      if (b == 0) before = 0;
    } else {
      int lo = 0, hi = a.B;   // cum[lo] * HS <= u < cum[hi] * HS
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((int64_t)cum[mid] * HS <= u) lo = mid;
        else hi = mid;
      }
      b = lo;
      before = cum[b];
    }
    const int len = length_of(a, b);
    int first, units;
    span(len, a.window, S::kUnit, first, units);
    const int64_t local = u - (int64_t)before * HS;
    const int cost = units << hl;   // of HW heads
    const int hg = (int)(local / cost);
    const int u0 = (int)(local - (int64_t)hg * cost);
    const int n_units = (int)min((int64_t)(cost - u0), u_end - u);
    const int hs = hg * HW + hw;
    const int kvh = hs / a.gt, g0 = (hs - kvh * a.gt) * 16;
    const int G = min(a.group - g0, 16);
    if (u == quota * blockIdx.x && threadIdx.x == 0) {
      // for k_join: the segment that this run goes on with, if it does not begin here
      const int64_t s0 = u - u0, s1 = s0 + cost;
      a.shared_segs[blockIdx.x] =
          make_int4(u0 > 0 ? b : -1, hg * 16 + hl, (int)(s0 / quota) * 2 + (s0 % quota != 0),
                    (int)((s1 - 1) / quota));
    }
    // this warp's keys of the piece: key0 + i * unit .. + KT - 1 in step i, up to key1
    const int piece0 = first / S::kUnit * S::kUnit + u0 * unit;
    const int key1 = min(len, piece0 + n_units * unit), key0 = piece0 + stripe * KT;
    const int n_sub = key1 > key0 ? (key1 - key0 + unit - 1) >> (kUnitLog2 - hl) : 0;
    const int32_t* table = a.block_table + (int64_t)b * a.table_width;
    int page = -1, slot = 0;
    auto look_up = [&](int i) {   // lane l < KT: the page and slot of key l of step i
      const int j = key0 + i * unit + lane % KT;
      page = -1;
      if (i < n_sub && j >= first && j < key1) {
        const int col = (int)((__umulhi((uint32_t)a.div_mul, (uint32_t)j) + (uint32_t)j) >> a.div_shift);
        slot = j - col * a.kv.page_size;
        page = table[col];   // col < table_width: the length is cut to the table
      }
    };
    auto fetch = [&](int i) {     // the copies of step i, whose pages look_up has found
      if (i < n_sub) {
        int64_t ko = -1, vo = -1;
        if (page >= 0 && page < a.kv.num_pages) {
          ko = ((int64_t)page * a.kv.k_page_stride + (int64_t)slot * a.kv.k_slot_stride +
                (int64_t)kvh * a.kv.k_head_stride) * (F8 ? 1 : 2);
          if (!a.same_strides)
            vo = ((int64_t)page * a.kv.v_page_stride + (int64_t)slot * a.kv.v_slot_stride +
                  (int64_t)kvh * a.kv.v_head_stride) * (F8 ? 1 : 2);
        } else if (lane < KT) {
          const int j = key0 + i * unit + lane;
          if (j >= first && j < key1) atomicOr(a.err, kErrBadPage);   // no such page: read as zeros
        }
        const uint32_t st = ring + (uint32_t)((i % ST) * S::kStageBytes);
        constexpr int RPI = 32 / CPR;   // rows of one warp-wide copy
#pragma unroll
        for (int p = 0; p < KT / RPI; ++p) {
          const int row = p * RPI + lane / CPR, ch = lane % CPR;
          const int64_t k_at = __shfl_sync(0xffffffffu, ko, row);
          const int64_t v_at = a.same_strides ? k_at : __shfl_sync(0xffffffffu, vo, row);
          const bool on = k_at >= 0;
          cp_async16(st + swz<CPR>(row, ch),
                     static_cast<const char*>(a.kv.k) + (on ? k_at + ch * 16 : 0), on);
          cp_async16(st + KT * S::kRow + swz<CPR>(row, ch),
                     static_cast<const char*>(a.kv.v) + (on ? v_at + ch * 16 : 0), on);
        }
      }
      cp_async_commit();
    };
    look_up(0);
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) {
      fetch(i);
      look_up(i + 1);
    }

    // ---- q as the column operand: column l / 4 of group g is head 8 g + l / 4
    uint32_t q[NG][KS][2];
    float sl[NG][2];   // log2 units per unit of the raw product, heads 8 g + 2 c, + 1
    {
      const uint16_t* qb = a.q + (int64_t)b * a.q_stride + (int64_t)(kvh * a.group + g0) * D;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const bool on = 8 * g + r < G;
        const uint16_t* qh = qb + (8 * g + r) * D;
        sl[g][0] = sl[g][1] = a.scale * a.kv.k_scale * kLog2e;
        if constexpr (!F8) {
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            q[g][ks][0] = on ? *reinterpret_cast<const uint32_t*>(qh + 16 * ks + 2 * c) : 0u;
            q[g][ks][1] = on ? *reinterpret_cast<const uint32_t*>(qh + 16 * ks + 2 * c + 8) : 0u;
          }
        } else {
          float top = 0.f;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {   // E4M3 keys come four elements to a lane
            uint2 v = make_uint2(0, 0);
            if (on) v = *reinterpret_cast<const uint2*>(qh + 16 * ks + 4 * c);
            q[g][ks][0] = v.x;
            q[g][ks][1] = v.y;
            top = fmaxf(top, finite_top(v.x, v.y));
          }
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          float up, down;
          f16_scale(top, up, down);
#pragma unroll
          for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              q[g][ks][e] = pack_f16(bf16_lo(q[g][ks][e]) * up, bf16_hi(q[g][ks][e]) * up);
          sl[g][0] *= __shfl_sync(0xffffffffu, down, 8 * c);       // head 2 c: lanes 8 c ..
          sl[g][1] *= __shfl_sync(0xffffffffu, down, 8 * c + 4);
        }
      }
    }

    float o[NG][MT][4], m[NG][2], l[NG][2];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
#pragma unroll
      for (int t = 0; t < MT; ++t) o[g][t][0] = o[g][t][1] = o[g][t][2] = o[g][t][3] = 0.f;
      m[g][0] = m[g][1] = -INFINITY;
      l[g][0] = l[g][1] = 0.f;
    }
    const int krow = ((lane >> 3) & 1) * 8 + (lane & 7), half = lane >> 4;

    for (int i = 0; i < n_sub; ++i) {
      cp_async_wait<ST - 2>();
      __syncwarp();
      // the next copies go into the stage that the previous step has left
      fetch(i + ST - 1);
      look_up(i + ST);
      const uint32_t st = ring + (uint32_t)((i % ST) * S::kStageBytes);
      // s^T = k q^T: 16 keys a tile
      float s[NG][NH][4];
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int h = 0; h < NH; ++h) s[g][h][0] = s[g][h][1] = s[g][h][2] = s[g][h][3] = 0.f;
      if constexpr (!F8) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            uint32_t k[4];   // keys 0-7 and 8-15 of dims 0-7, then of dims 8-15
            ldmatrix4(k, st + swz<CPR>(16 * h + krow, 2 * ks + half));
#pragma unroll
            for (int g = 0; g < NG; ++g)
              mma_bf16(s[g][h], k[0], k[1], k[2], k[3], q[g][ks][0], q[g][ks][1]);
          }
      } else {
#pragma unroll
        for (int ks = 0; ks < KS; ks += 2)
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            uint32_t k[4];   // keys 0-7 and 8-15 of 16 dims, then of the next 16
            ldmatrix4(k, st + swz<CPR>(16 * h + krow, ks + half));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint32_t a0, a1, a2, a3;
              e4m3x4_to_f16(k[2 * e], a0, a2);
              e4m3x4_to_f16(k[2 * e + 1], a1, a3);
#pragma unroll
              for (int g = 0; g < NG; ++g)
                mma_f16(s[g][h], a0, a1, a2, a3, q[g][ks + e][0], q[g][ks + e][1]);
            }
          }
      }
      // scores in log2 units: key j0 + 16 h + r (elements 0, 1) and + 8; keys outside [first, key1)
      // do not count
      const int j0 = key0 + i * unit;
      bool up = false;
      float top[NG][2];
#pragma unroll
      for (int g = 0; g < NG; ++g) {
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[g][h][e] *= sl[g][e & 1];
        if (j0 < first || j0 + KT > key1) {
#pragma unroll
          for (int h = 0; h < NH; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = j0 + 16 * h + r + (e >> 1) * 8;
              if (j < first || j >= key1) s[g][h][e] = -INFINITY;
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float t = fmaxf(s[g][0][e], s[g][0][2 + e]);
#pragma unroll
          for (int h = 1; h < NH; ++h) t = fmaxf(t, fmaxf(s[g][h][e], s[g][h][2 + e]));
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, x));
          if constexpr (F8) t = __fsub_ru(t, kLift);   // upwards: no weight above 2^15 at any size of t
          top[g][e] = t;
          up |= t > m[g][e];
        }
      }
      if (__any_sync(0xffffffffu, up)) {   // a new maximum: what is summed shrinks
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          float f[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float n = fmaxf(m[g][e], top[g][e]);
            f[e] = m[g][e] == -INFINITY ? 0.f : exp2_fast(m[g][e] - n);
            m[g][e] = n;
            l[g][e] *= f[e];
          }
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            o[g][t][0] *= f[0]; o[g][t][1] *= f[1];
            o[g][t][2] *= f[0]; o[g][t][3] *= f[1];
          }
        }
      }
      uint32_t p[NG][NH][2], rest[NG][NH][2];   // p^T: columns heads, rows keys 0-7 and 8-15 of a tile
#pragma unroll
      for (int g = 0; g < NG; ++g) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float base = m[g][e] == -INFINITY ? 0.f : m[g][e];   // no key yet: every p is 0
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            s[g][h][e] = exp2_fast(s[g][h][e] - base);
            s[g][h][2 + e] = exp2_fast(s[g][h][2 + e] - base);
            l[g][e] += s[g][h][e] + s[g][h][2 + e];
          }
        }
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float p0 = s[g][h][2 * x], p1 = s[g][h][2 * x + 1];
            if constexpr (F8) {
              const uint32_t v = pack_f16(p0, p1);
              p[g][h][x] = transpose8(v);
              rest[g][h][x] = transpose8(pack_f16(p0 - f16_lo(v), p1 - f16_hi(v)));
            } else {
              const uint32_t v = pack_bf16(p0, p1);
              p[g][h][x] = transpose8(v);
              rest[g][h][x] = transpose8(pack_bf16(p0 - bf16_lo(v), p1 - bf16_hi(v)));
            }
          }
      }
      // o^T += v^T p^T: 16 dims at a time
      const uint32_t vs = st + KT * S::kRow;
      if constexpr (!F8) {
        const int vrow = half * 8 + (lane & 7), vch = (lane >> 3) & 1;
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            uint32_t v[4];   // dims 0-7 and 8-15 of keys 0-7, then of keys 8-15
            ldmatrix4_trans(v, vs + swz<CPR>(16 * h + vrow, 2 * t + vch));
#pragma unroll
            for (int g = 0; g < NG; ++g) {
              mma_bf16(o[g][t], v[0], v[1], v[2], v[3], p[g][h][0], p[g][h][1]);
              mma_bf16(o[g][t], v[0], v[1], v[2], v[3], rest[g][h][0], rest[g][h][1]);
            }
          }
      } else {
#pragma unroll
        for (int t = 0; t < MT; t += 2)
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            uint32_t v[4];   // keys 0-7 and 8-15 of 16 dims, then of the next 16
            ldmatrix4_trans(v, vs + swz<CPR>(16 * h + krow, t + half));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              // (key, dim d), (key, d + 1), (key + 1, d), (key + 1, d + 1): rows 0-7 take the even dims
              uint32_t a0, a1, a2, a3;
              e4m3x4_to_f16(__byte_perm(v[2 * e], 0, 0x3120), a0, a1);
              e4m3x4_to_f16(__byte_perm(v[2 * e + 1], 0, 0x3120), a2, a3);
#pragma unroll
              for (int g = 0; g < NG; ++g) {
                mma_f16(o[g][t + e], a0, a1, a2, a3, p[g][h][0], p[g][h][1]);
                mma_f16(o[g][t + e], a0, a1, a2, a3, rest[g][h][0], rest[g][h][1]);
              }
            }
          }
      }
      __syncwarp();   // every lane has read the stage before it is filled again
    }
    cp_async_wait<0>();

    // ---- join the warps of a head: sums [head][LD] in each one's ring
    sync();
    float* sums = reinterpret_cast<float*>(smem + (size_t)warp * ST * S::kStageBytes);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[g][e] += __shfl_xor_sync(0xffffffffu, l[g][e], x);
        const int h = 8 * g + 2 * c + e;
        if (r == 0) {
          wm[warp][h] = m[g][e];
          wl[warp][h] = l[g][e];
        }
        if (h < G) {
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            const int d0 = F8 ? 16 * t + 2 * r : 16 * t + r, d1 = F8 ? d0 + 1 : d0 + 8;
            sums[h * LD + d0] = o[g][t][e];
            sums[h * LD + d1] = o[g][t][2 + e];
          }
        }
      }
    }
    sync();
    // each warp's share in its heads' sums, and the joined maximum and sum
    float2 ms = make_float2(-INFINITY, 0.f);
    if (lane < G) {
#pragma unroll
      for (int s = 0; s < W; ++s)
        if (s < stripes) ms.x = fmaxf(ms.x, wm[hw + (s << hl)][lane]);
      const float base = ms.x == -INFINITY ? 0.f : ms.x;
#pragma unroll
      for (int s = 0; s < W; ++s)
        if (s < stripes)
          ms.y = fmaf(exp2_fast(wm[hw + (s << hl)][lane] - base), wl[hw + (s << hl)][lane], ms.y);
      share[warp][lane] = exp2_fast(wm[warp][lane] - base);
    }
    sync();
    const bool whole = n_units == cost;
    const int64_t part = ((2 * (int64_t)blockIdx.x + (u == quota * blockIdx.x ? 0 : 1)) * W + hw) * 16;
    const int64_t row = (int64_t)b * a.Hq + kvh * a.group + g0;
    if (lane < G && stripe == 0) {
      if (!whole) *reinterpret_cast<float2*>(a.part_ml + (part + lane) * 2) = ms;
      else if (a.lse) a.lse[row + lane] = lse_of<F8>(ms.x, ms.y);
    }
    for (int x = stripe * 32; x < G * (D / 4); x += stripes * 32) {   // four dims of a head a lane
      const int g = (x + lane) / (D / 4), d = (x + lane) % (D / 4) * 4;
      const float sum = __shfl_sync(0xffffffffu, ms.y, g);
      if (g >= G) continue;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int s = 0; s < W; ++s) {
        if (s >= stripes) break;
        const int w = hw + (s << hl);
        const float f = share[w][g];
        const float4 y = *reinterpret_cast<const float4*>(
            reinterpret_cast<const float*>(smem + (size_t)w * ST * S::kStageBytes) + g * LD + d);
        v.x = fmaf(f, y.x, v.x); v.y = fmaf(f, y.y, v.y);
        v.z = fmaf(f, y.z, v.z); v.w = fmaf(f, y.w, v.w);
      }
      if (whole) store_row(a, (row + g) * D + d, v, sum);
      else *reinterpret_cast<float4*>(a.part_o + (part + g) * D + d) = v;
    }
    sync();   // before the ring is filled again
    u += n_units;
  }
}

// Segments that several runs share, and empty sequences. Block i belongs to run i: with the blocks of the
// other runs that go on with the same segment it shares that segment's query heads. A head is a job of one
// to kTeam warps, more where the pieces are many and the jobs few: each adds a share of the pieces in
// order, the first of them adds the shares in order. The blocks also zero the heads of empty sequences. W:
// warps of k_attend's blocks.
constexpr int kJoinWarps = 16, kTeam = 8;   // warps of a block, of a job at most
constexpr int kFlight = 4;                  // pieces of a warp in flight
template <int D, int W>
__global__ void __launch_bounds__(kJoinWarps * 32) k_join(const AttendArgs a) {
  constexpr int E = D / 32;
  __shared__ float sums[kJoinWarps][D], wm[kJoinWarps], wl[kJoinWarps];
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // sequence or -1; its part, * 16 + log2 of the key heads in it; first run (* 2, + 1 where the segment
  // begins inside that run); last run
  const int4 seg = a.shared_segs[blockIdx.x];
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    if (length_of(a, b) > 0) continue;
    for (int x = threadIdx.x; x < a.Hq * D / 8; x += kJoinWarps * 32)
      reinterpret_cast<uint4*>(a.out + (int64_t)b * a.Hq * D)[x] = make_uint4(0, 0, 0, 0);
    if (a.lse)
      for (int x = threadIdx.x; x < a.Hq; x += kJoinWarps * 32)
        a.lse[(int64_t)b * a.Hq + x] = -INFINITY;
  }
  if (seg.x < 0) return;
  const int heads = min(a.group, 16), hl = seg.y & 15, jobs = heads << hl;
  const int run0 = seg.z >> 1, blocks = seg.w - run0, me = (int)blockIdx.x - run0 - 1;
  const int mine = (jobs - me + blocks - 1) / blocks;   // jobs me, me + blocks, ..
  int tl = 0;   // log2 of the warps of a job
  while (2 << tl <= kTeam && kFlight << tl <= blocks && mine << (tl + 1) <= kJoinWarps) ++tl;
  const int team = warp >> tl, part = warp & ((1 << tl) - 1), teams = kJoinWarps >> tl;
  for (int i0 = 0; i0 < mine; i0 += teams) {
    const int job = me + (i0 + team) * blocks;
    const int hw = job / heads, g = job - hw * heads;
    const int hs = ((seg.y >> 4) << hl) + hw, kvh = a.gt == 1 ? hs : hs / a.gt, g0 = (hs - kvh * a.gt) * 16;
    const bool on = job < jobs && g0 + g < a.group;
    float m = -INFINITY, l = 0.f, v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = 0.f;
    if (on) {
      for (int p0 = run0 + part; p0 <= seg.w; p0 += kFlight << tl) {
        float2 ml[kFlight];
        float y[kFlight][E];
#pragma unroll
        for (int j = 0; j < kFlight; ++j) {
          const int p = p0 + (j << tl);
          // a run's first piece, but for a segment that begins inside its first run
          const int64_t at = ((2 * (int64_t)p + (p == run0 ? seg.z & 1 : 0)) * W + hw) * 16 + g;
          ml[j] = make_float2(-INFINITY, 0.f);
          if (p <= seg.w) ml[j] = *reinterpret_cast<const float2*>(a.part_ml + at * 2);
#pragma unroll
          for (int e = 0; e < E; ++e) y[j][e] = p <= seg.w ? a.part_o[at * D + lane + 32 * e] : 0.f;
        }
        float top = m;
#pragma unroll
        for (int j = 0; j < kFlight; ++j) top = fmaxf(top, ml[j].x);
        const float base = top == -INFINITY ? 0.f : top, f = exp2_fast(m - base);
        m = top;
        l *= f;
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] *= f;
#pragma unroll
        for (int j = 0; j < kFlight; ++j) {
          const float fj = exp2_fast(ml[j].x - base);
          l = fmaf(fj, ml[j].y, l);
#pragma unroll
          for (int e = 0; e < E; ++e) v[e] = fmaf(fj, y[j][e], v[e]);
        }
      }
    }
    if (tl > 0) {   // uniform over the block, as are i0 and mine
#pragma unroll
      for (int e = 0; e < E; ++e) sums[warp][lane + 32 * e] = v[e];
      if (lane == 0) {
        wm[warp] = m;
        wl[warp] = l;
      }
      __syncthreads();
      if (part == 0) {
        float top = m;
#pragma unroll
        for (int w = 1; w < kTeam; ++w)
          if (w < 1 << tl) top = fmaxf(top, wm[warp + w]);
        const float base = top == -INFINITY ? 0.f : top, f0 = exp2_fast(m - base);
        m = top;
        l *= f0;
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] *= f0;
#pragma unroll
        for (int w = 1; w < kTeam; ++w) {
          if (w >= 1 << tl) break;
          const float f = exp2_fast(wm[warp + w] - base);
          l = fmaf(f, wl[warp + w], l);
#pragma unroll
          for (int e = 0; e < E; ++e) v[e] = fmaf(f, sums[warp + w][lane + 32 * e], v[e]);
        }
      }
      __syncthreads();
    }
    if (on && part == 0) {
      const int64_t row = (int64_t)seg.x * a.Hq + kvh * a.group + g0 + g;
#pragma unroll
      for (int e = 0; e < E; ++e)
        a.out[row * D + lane + 32 * e] =
            (uint16_t)(pack_bf16(l == 0.f ? 0.f : v[e] / l * a.kv.v_scale, 0.f) & 0xFFFFu);
      if (lane == 0 && a.lse)
        a.lse[row] = a.kv.dtype == FT_KV_E4M3 ? lse_of<true>(m, l) : lse_of<false>(m, l);
    }
  }
}

template <int D, bool F8, int NG>
cudaError_t launch_d(AttendArgs a, int num_sms, cudaStream_t stream) {
  using S = AttnShape<D, F8, NG>;
  a.heads_log2 = 0;
  while (2 << a.heads_log2 <= S::kWarps && a.kv.Hkv * a.gt % (2 << a.heads_log2) == 0) ++a.heads_log2;
  const size_t smem = S::kRing + (a.B > 32 ? (size_t)(a.B + 1) * 4 : 0);
  cudaError_t e;
  static SmemGrant grant;   // for the most sequences that a call may have
  if ((e = grant_smem(grant, k_attend<D, F8, NG>, S::kRing + 4 * (kMaxSeqs + 1))) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const int grid = S::kBlocks * num_sms;
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(S::kWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, k_attend<D, F8, NG>, a)) != cudaSuccess) return e;
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, k_join<D, S::kWarps>, a);
}

template <int D>
cudaError_t launch_g(const AttendArgs& a, int num_sms, cudaStream_t stream) {
  const bool f8 = a.kv.dtype == FT_KV_E4M3;
  if (a.group <= 8)
    return f8 ? launch_d<D, true, 1>(a, num_sms, stream) : launch_d<D, false, 1>(a, num_sms, stream);
  return f8 ? launch_d<D, true, 2>(a, num_sms, stream) : launch_d<D, false, 2>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_attend(const AttendArgs& args, int num_sms, cudaStream_t stream) {
  AttendArgs a = args;
  a.group = a.Hq / a.kv.Hkv;
  a.gt = (a.group + 15) / 16;
  a.same_strides = a.kv.k_page_stride == a.kv.v_page_stride && a.kv.k_slot_stride == a.kv.v_slot_stride &&
                   a.kv.k_head_stride == a.kv.v_head_stride;
  page_division(a.kv.page_size, a.div_mul, a.div_shift);
  const int64_t slots = (int64_t)a.table_width * a.kv.page_size;
  a.max_len = (int)(slots < (1 << 30) ? slots : 1 << 30);
  switch (a.kv.D) {
    case 64: return launch_g<64>(a, num_sms, stream);
    case 128: return launch_g<128>(a, num_sms, stream);
    case 256: return launch_g<256>(a, num_sms, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ftmoe
