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
// NVFP4 caches (ftmoe_attend4.cuh): f16 products and weights in two f16 as for E4M3. Statistics and sums are float32.
//
// Measured (of the copy rate of 6786 GB/s): three sequences up to 131072, bf16, 962 MB: 147 us (96 %).
// 48 ragged ones up to 8192, E4M3, 423 MB: 80 us (78 %), of which some 10 us are launches, fill and
// join, and the runs' pieces differ in cost. One sequence of 777: 7.6 us, two launches and the chain
// length, page, keys, scores, sums, join.
// NVFP4: the three 63.4 us (270 MB, 63 %), the 48 60.8 us (239 MB, 58 %), 64 of 6500 104 us with pages head by head or slot
// by slot (481 MB, 68 %). The SM's twelve warps take a step of 55 KB in 1.46 us, of which the copy rate would take 1.24,
// the instructions (some 620 a warp) 0.95 and the tensor pipe (48 products of 8 cycles) 0.59. Outside the steps of the 48:
// 5 us until data flow, 3 for the pieces' results, 5 (in the mean) until the last run ends, 5 of join.
// With heads of 64 (200 sequences, a window of 1023: 28.5 us for 7.4) rows of 32 bytes copy at 77 % and as many bytes take
// a third more instructions; 18 of the 28.5 us are the runs, 8.7 of them steps; the last one ends 4.4 us later, the join
// takes 4.6. Heads of 256 with 16 heads a key head (49.3 us for 14.6): 27 us are steps, 1.52 each for 37 KB, where the copy
// rate would take 0.83, the tensor pipe 0.79 (96 products) and the instructions 0.70; two warps a scheduler do not hide
// one's latencies behind the other. The rest: 6 us until data flow, 5 for the results, 5 until the last run ends, 5 of join.
#include <cmath>
#include <cuda_runtime.h>

#include "ftmoe_attend4.cuh"
#include "ftmoe_internal.h"
#include "ftmoe_mma.cuh"
#include "ftmoe_tc.cuh"

namespace ftmoe {

namespace {

// DT: the cache's type (FT_KV_BF16, FT_KV_E4M3, kKvNvfp4).
template <int D, int DT, int NG>
struct AttnShape {
  static constexpr int kRow = DT == kKvNvfp4 ? D / 2 : DT == FT_KV_E4M3 ? D : 2 * D;   // bytes of a key or value
  static constexpr int kCpr = kRow / 16;              // 16-byte pieces of it
  static constexpr int kScaleRow = DT == kKvNvfp4 ? D / 16 : 0;   // bytes of its block scales
  static constexpr int kKeys = DT == kKvNvfp4 ? 4096 / D : kRow <= 128 ? 32 : 16;   // keys of a warp's step
  static constexpr int kStageBytes = 2 * kKeys * (kRow + kScaleRow);   // those keys and values
  // blocks an SM: the others stream while one joins a piece's warps. Three of two stages each, not two of
  // three, where the registers allow it: 256 sequences up to 1024 with 8-bit keys of 128: 68 us for 79.
  // (Past some 2600 sequences their running sums in shared memory leave room for two.)
  static constexpr int kBlocks =
      kRow >= 512 || DT == kKvNvfp4 ? 1 : kRow == 128 && NG == 1 ? kAttendBlocks : 2;
  // NVFP4: one block an SM, whose groups of warps each do what a block does otherwise. With heads of 64 three groups of
  // four warps at 64 keys a step, not two of eight at 32: 200 sequences with a window of 1023 27.2 us for 29.2 (with
  // weights in one f16).
  static constexpr int kGroups = DT != kKvNvfp4 ? 1 : D == 64 || (D == 128 && NG == 1) ? kAttendBlocks : 2;
  static constexpr int kWarps = DT == kKvNvfp4 || kRow >= 128 ? 4 : 8;   // of a group
  static constexpr int kQShared = DT != kKvNvfp4 || NG == 1 ? 0 : D == 256 ? 2 : D == 64 ? 1 : 0;   // groups of q in shared memory
  static constexpr int kQBytes = kQShared * (D / 16) * 256;
  static constexpr int kStages =
      ((DT == kKvNvfp4 ? 208 : 192) * 1024 / (kBlocks * kGroups * kWarps) - kQBytes) / kStageBytes;
  static constexpr int kWarpBytes = kStages * kStageBytes + kQBytes;
  static constexpr int kUnit = kKeys * kWarps;        // keys of a unit
  // Units that a segment is charged for (see kChargeFrom).
  static constexpr int kCharge = DT != kKvNvfp4 ? 0 : D == 256 ? 4 : 1;
  static constexpr int kRing = kWarps * kWarpBytes;
  // floats between heads of a warp's sums, in its ring. NVFP4: lane r has elements D/8 r + 2 t, + 1 of a head, which
  // lie at 20 t + 2 r, so that neither the lanes that write them nor those that read four of them share banks.
  static constexpr int kSumsLd = (DT == kKvNvfp4 ? 20 * (D / 16) : D) + 4;
  static_assert(8 * NG * kSumsLd * 4 <= kWarpBytes && kBlocks * kGroups * kWarps <= attend_warps(D));
};

// From this many units in a run, the warps of a block take several key heads at once instead of stripes of
// one head's keys: rows of the same slot are then read together (256 sequences up to 1024, bf16, 8 heads of
// 128: 97 us for 118; 8 of 32768, E4M3, 8 heads of 64: 54 for 80), and no join in the block holds the
// copies up. Shorter runs would leave k_join as many times more pieces: 48 sequences of 256 take 12.8 us, and
// 17.0 when runs of two units are long; 8 up to 2048 take 14.0 us, and 15.5 when only runs of eight are.
constexpr int kLongRun = 4;
// NVFP4, runs of at least this many units: a segment begins with kCharge units without keys, for the copies that
// begin anew and the results that are joined. It helps ragged lengths and costs 2 to 5 % of even ones whose runs cut every
// segment: with 0, 1, 2 and 4 of them 48 ragged sequences up to 8192 take 61.6, 60.8, 62.2 and 63.6 us, 100 up to 4000
// 55.6, 52.5, 55.3 and 58.0, 19 of 22272 100.3, 102.5, 102.2 and 103.3, 64 of 1000 31.8, 33.4, 32.3 and 32.4; with heads of
// 256 (units half as long) 13 up to 24001 53.8, 51.0, 50.7 and 49.3, 16 of 8192 48.2, 45.6, 45.0 and 44.8.
// From runs of 12, 8, 6 and 4 units on: 100 ragged sequences up to 2000 29.7, 29.8, 26.7 and 26.7 us, 200 up to 700 with
// heads of 64 30.5, 30.5, 27.9 and 27.9, 200 with a window of 1023 28.5, 28.4, 28.5 and 30.1, 64 of 1000 31.8 and 33.4
// from eight units or fewer on.
constexpr int kChargeFrom = 6;
// NVFP4: no segment is cut, and none is left to the join, where the longest is no more than this many units longer than
// a run; a run then takes the segments that begin in it. 32 sequences with a window of 512 18.0 -> 14.0 us, 60 ragged
// ones up to 300 15.9 -> 14.2; with eight units 128 of 512 would take 34.4 us for 30.3, one of 777 11.3 for 7.0.
constexpr int kUncut = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// log2 of the largest weight. f16 holds 11 bits of weights down to 2^-14 and nothing under 2^-25: with
// weights of up to 2^15 the two parts of a key's weight hold 22 bits of it, or all but 2^-40 of the largest
// key's weight. The sums carry the same factor, which their quotient does not see.
constexpr float kLift = 15.f;
template <bool F16>
__device__ __forceinline__ float lse_of(float m, float l) {   // ln of l 2^m
  return F16 ? (m + kLift + log2f(l * (1.f / 32768.f))) * kLn2 : (m + log2f(l)) * kLn2;
}

// Offset of 16-byte piece c of row r in a tile of rows of kCpr pieces: pieces are exchanged within
// groups of eight (four) so that eight rows' same piece lie in different banks.
template <int CPR>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  if constexpr (CPR >= 8) return (uint32_t)(r * CPR + (c ^ (r & 7))) * 16;
  else return (uint32_t)(r * CPR + (c ^ ((r >> 1) & 3))) * 16;
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

// A sequence's length, cut to what its row of the block table can hold (and the call can count).
__device__ __forceinline__ int length_of(const AttendArgs& a, int b) { return min(a.seq_lens[b], a.max_len); }

// First key, number of units of a sequence and the first unit's first key: a multiple of the unit, or (NVFP4, whose
// copies find each key's page) the first key itself, which saves a window up to a unit of steps.
template <int DT>
__device__ __forceinline__ void span(int len, int window, int unit, int& first, int& units, int& base) {
  first = window > 0 && len > window ? len - window : 0;
  base = DT == kKvNvfp4 ? first : first / unit * unit;
  units = len > 0 ? (len - base + unit - 1) / unit : 0;
}

template <int D, int DT, int NG>
__global__ void __launch_bounds__(AttnShape<D, DT, NG>::kGroups * AttnShape<D, DT, NG>::kWarps * 32,
                                  AttnShape<D, DT, NG>::kBlocks)
    k_attend(const AttendArgs a) {
  using S = AttnShape<D, DT, NG>;
  constexpr bool F4 = DT == kKvNvfp4, F16 = DT != FT_KV_BF16;   // f16 products
  constexpr int W = S::kWarps, ST = S::kStages, CPR = S::kCpr, KS = D / 16, MT = D / 16;
  constexpr int KT = S::kKeys, NH = KT / 16;   // keys of a step, in 16-row tiles
  constexpr int LD = S::kSumsLd;
  constexpr int kUnitLog2 = S::kUnit == 64 ? 6 : S::kUnit == 128 ? 7 : 8;
  static_assert(S::kUnit == 1 << kUnitLog2);
  extern __shared__ __align__(1024) unsigned char smem[];
  constexpr int GR = S::kGroups;
  __shared__ float all_wm[GR * W][16], all_wl[GR * W][16], all_share[GR * W][16];
  __shared__ int scan[GR * W], scan_some[F4 ? GR * W : 1], scan_most[F4 ? GR * W : 1];
  int* cum = reinterpret_cast<int*>(smem + GR * S::kRing);   // [B + 1] units before each sequence (B > 32)
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int group = GR > 1 ? (int)threadIdx.x / (W * 32) : 0;
  const int warp = (int)(threadIdx.x >> 5) - group * W, tid = threadIdx.x - group * W * 32;   // in the group
  const int block = (int)(blockIdx.x + group * gridDim.x), blocks = (int)gridDim.x * GR;   // groups stand for blocks
  float (*const wm)[16] = all_wm + group * W;
  float (*const wl)[16] = all_wl + group * W;
  float (*const share)[16] = all_share + group * W;
  unsigned char* const rings = smem + group * S::kRing;
  const int c = lane & 3, r = lane >> 2;
  const int HS = a.kv.Hkv * a.gt;   // segments of a sequence

  // units before each sequence: in every warp's lanes, or in shared memory past 32 sequences
  // NVFP4: a segment's first units may stand for the cost of a piece's copies beginning and its results being
  // joined, `charge` of them
  auto charge_of = [&](int units) { return (int64_t)units * HS >= (int64_t)kChargeFrom * blocks ? S::kCharge : 0; };
  int charge = 0;
  int longest = 0;   // units of a sequence at most
  int inc = 0;       // B <= 32: units up to and with sequence `lane`
  int all;
  if (a.B <= 32) {
    int first, base, n = 0;
    if (lane < a.B) {
      const int len = length_of(a, lane);
      span<DT>(len, a.window, S::kUnit, first, n, base);
      if (block == 0 && warp == 0 && a.seq_lens[lane] > len) atomicOr(a.err, kErrBadPage);
    }
    inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    all = __shfl_sync(0xffffffffu, inc, 31);
    if constexpr (F4) {
      const uint32_t some = __ballot_sync(0xffffffffu, n > 0);
      longest = __reduce_max_sync(0xffffffffu, n);
      charge = charge_of(all);
      inc += charge * __popc(some & (0xffffffffu >> (31 - lane)));
      all += charge * __popc(some);
    }
  } else {
    const int per = (a.B + GR * W * 32 - 1) / (GR * W * 32);
    const int b0 = threadIdx.x * per;
    int mine = 0, some = 0, most = 0;   // units, sequences with any, units of one
    for (int b = b0; b < min(b0 + per, a.B); ++b) {
      int first, base, n;
      const int len = length_of(a, b);
      span<DT>(len, a.window, S::kUnit, first, n, base);
      mine += n;
      some += n > 0;
      most = max(most, n);
      if (blockIdx.x == 0 && a.seq_lens[b] > len) atomicOr(a.err, kErrBadPage);
    }
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) scan[threadIdx.x >> 5] = upto;
    int some_upto = some;
    if constexpr (F4) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, some_upto, o);
        if (lane >= o) some_upto += v;
      }
      most = __reduce_max_sync(0xffffffffu, most);
      if (lane == 31) {
        scan_some[threadIdx.x >> 5] = some_upto;
        scan_most[threadIdx.x >> 5] = most;
      }
    }
    __syncthreads();
    int at = upto - mine;
    if constexpr (F4) {
      int units = 0, before = some_upto - some;
#pragma unroll
      for (int w = 0; w < GR * W; ++w) {
        const bool ahead = w < (int)(threadIdx.x >> 5);
        units += scan[w];
        at += ahead ? scan[w] : 0;
        before += ahead ? scan_some[w] : 0;
        longest = max(longest, scan_most[w]);
      }
      charge = charge_of(units);
      at += charge * before;
    } else {
      for (int w = 0; w < (int)(threadIdx.x >> 5); ++w) at += scan[w];
    }
    for (int b = b0; b < min(b0 + per, a.B); ++b) {
      int first, base, n;
      span<DT>(length_of(a, b), a.window, S::kUnit, first, n, base);
      cum[b] = at;
      at += n + (n > 0 ? charge : 0);
    }
    if (b0 < a.B && b0 + per >= a.B) cum[a.B] = at;
    __syncthreads();
    all = cum[a.B];
  }
  const int64_t total = (int64_t)all * HS;
  const int64_t quota = (total + blocks - 1) / blocks;
  int64_t u = quota * block;
  const int64_t u_end = min(u + quota, total);
  const uint32_t ring = smem_addr(rings) + (uint32_t)(warp * S::kWarpBytes);
  // HW heads a block, W / HW stripes of keys each
  const int hl = quota >= kLongRun ? a.heads_log2 : 0, HW = 1 << hl, stripes = W >> hl;
  const int hw = warp & (HW - 1), stripe = warp >> hl;
  const int unit = S::kUnit >> hl;
  auto sync = [&]() {   // the warps that share a head
    if (stripes == 1) __syncwarp();
    else if constexpr (GR == 1) __syncthreads();
    else asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(W * 32) : "memory");
  };
  const bool uncut = F4 && (int64_t)((longest + charge) << hl) <= quota + kUncut;
  const int64_t cap = uncut ? max(total, u_end + 1) : u_end;   // where its last piece ends at the latest
  if ((uncut || u >= u_end) && tid == 0) a.shared_segs[block] = make_int4(-1, 0, 0, 0);

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
    int first, units, base;
    span<DT>(len, a.window, S::kUnit, first, units, base);
    const int64_t local = u - (int64_t)before * HS;
    const int cost = (units + charge) << hl;   // of HW heads
    const int hg = (int)(local / cost);
    const int u0 = (int)(local - (int64_t)hg * cost);
    if (u0 > 0 && cap > u_end) {   // the run's that the segment begins in
      u += cost - u0;
      continue;
    }
    const int n_units = (int)min((int64_t)(cost - u0), cap - u);
    const int hs = hg * HW + hw;
    const int kvh = hs / a.gt, g0 = (hs - kvh * a.gt) * 16;
    const int G = min(a.group - g0, 16);
    if (!uncut && u == quota * block && tid == 0) {
      // for k_join: the segment that this run goes on with, if it does not begin here
      const int64_t s0 = u - u0, s1 = s0 + cost;
      a.shared_segs[block] =
          make_int4(u0 > 0 ? b : -1, hg * 16 + hl, (int)(s0 / quota) * 2 + (s0 % quota != 0),
                    (int)((s1 - 1) / quota));
    }
    // this warp's keys of the piece: key0 + i * unit .. + KT - 1 in step i, up to key1
    const int at0 = max(u0 - (charge << hl), 0), at1 = max(u0 + n_units - (charge << hl), 0);
    const int piece0 = base + at0 * unit;
    const int key1 = min(len, base + at1 * unit), key0 = piece0 + stripe * KT;
    const int n_sub = key1 > key0 ? (key1 - key0 + unit - 1) >> (kUnitLog2 - hl) : 0;
    float o[NG][MT][4], m[NG][2], l[NG][2];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
#pragma unroll
      for (int t = 0; t < MT; ++t) o[g][t][0] = o[g][t][1] = o[g][t][2] = o[g][t][3] = 0.f;
      m[g][0] = m[g][1] = -INFINITY;
      l[g][0] = l[g][1] = 0.f;
    }
    if constexpr (F4) {
      attend_piece4<D, NG, S>(a, reinterpret_cast<char*>(rings) + warp * S::kWarpBytes, b, kvh, g0, G, first, key0, key1,
                              unit, n_sub, o, m, l);
    } else {
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
                  (int64_t)kvh * a.kv.k_head_stride) * (F16 ? 1 : 2);
            if (!a.same_strides)
              vo = ((int64_t)page * a.kv.v_page_stride + (int64_t)slot * a.kv.v_slot_stride +
                    (int64_t)kvh * a.kv.v_head_stride) * (F16 ? 1 : 2);
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
            // the place written out twice: kept in a register, it costs three more spilled ones with heads of 256
            cp_async16(st + swz<CPR>(row, ch), static_cast<const char*>(a.kv.k) + (on ? k_at + ch * 16 : 0), on);
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
          if constexpr (!F16) {
            sl[g][0] = sl[g][1] = a.scale * a.kv.k_scale * kLog2e;
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
            const float unit_s = copysignf(product3(fabsf(a.scale), a.kv.k_scale, down), a.scale) * kLog2e;
            sl[g][0] = __shfl_sync(0xffffffffu, unit_s, 8 * c);       // head 2 c: lanes 8 c ..
            sl[g][1] = __shfl_sync(0xffffffffu, unit_s, 8 * c + 4);
          }
        }
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
        if constexpr (!F16) {
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
            if constexpr (F16) t = __fsub_ru(t, kLift);   // upwards: no weight above 2^15 at any size of t
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
              if constexpr (F16) {
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
        if constexpr (!F16) {
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
    }

    // ---- join the warps of a head: sums [head][LD] in each one's ring
    sync();
    float* sums = reinterpret_cast<float*>(rings + (size_t)warp * S::kWarpBytes);
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
            if constexpr (F4) {
              *reinterpret_cast<float2*>(sums + h * LD + 20 * t + 2 * r) = make_float2(o[g][t][e], o[g][t][2 + e]);
              continue;
            }
            const int d0 = F16 ? 16 * t + 2 * r : 16 * t + r;
            const int d1 = F16 ? d0 + 1 : d0 + 8;
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
    const int64_t part = ((2 * (int64_t)block + (u == quota * block ? 0 : 1)) * W + hw) * 16;
    const int64_t row = (int64_t)b * a.Hq + kvh * a.group + g0;
    if (lane < G && stripe == 0) {
      if (!whole) *reinterpret_cast<float2*>(a.part_ml + (part + lane) * 2) = ms;
      else if (a.lse) a.lse[row + lane] = lse_of<F16>(ms.x, ms.y);
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
        const float* from = reinterpret_cast<const float*>(rings + (size_t)w * S::kWarpBytes) + g * LD;
        float4 y;
        if constexpr (F4) {
          const float* at = from + 10 * (d % (D / 8)) + 2 * (d / (D / 8));
          const float2 y0 = *reinterpret_cast<const float2*>(at), y1 = *reinterpret_cast<const float2*>(at + 20);
          y = make_float4(y0.x, y0.y, y1.x, y1.y);
        } else {
          y = *reinterpret_cast<const float4*>(from + d);
        }
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
constexpr int kTeam = 8;                    // warps of a job at most
// Adds N pieces to a running maximum, sum and row.
template <int N, int E>
__device__ __forceinline__ void add_pieces(const float2* ml, const float (*y)[E], float& m, float& l, float (&v)[E]) {
  float top = m;
#pragma unroll
  for (int j = 0; j < N; ++j) top = fmaxf(top, ml[j].x);
  const float base = top == -INFINITY ? 0.f : top, f = exp2_fast(m - base);
  m = top;
  l *= f;
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] *= f;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float fj = exp2_fast(ml[j].x - base);
    l = fmaf(fj, ml[j].y, l);
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = fmaf(fj, y[j][e], v[e]);
  }
}

// kFlight: pieces of a warp in flight; kJoinBlocks: blocks that an SM holds
template <int D, int W, int kJoinWarps, int kJoinBlocks, int kFlight>
__global__ void __launch_bounds__(kJoinWarps * 32, kJoinBlocks) k_join(const AttendArgs a) {
  constexpr int E = D / 32;
  static_assert(kJoinWarps % kTeam == 0);   // whole teams
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
  // a job's output row, its head among the segment's key heads, or -1 where the group of heads is not full
  auto row_of = [&](int job) -> int64_t {
    const int hw = job / heads, g = job - hw * heads;
    const int hs = ((seg.y >> 4) << hl) + hw, kvh = a.gt == 1 ? hs : hs / a.gt, g0 = (hs - kvh * a.gt) * 16;
    if (job >= jobs || g0 + g >= a.group) return -1;
    return (int64_t)seg.x * a.Hq + kvh * a.group + g0 + g;
  };
  auto piece_of = [&](int job, int p) -> int64_t {   // where piece p of a job lies
    const int hw = job / heads, g = job - hw * heads;
    // a run's first piece, but for a segment that begins inside its first run
    return ((2 * (int64_t)p + (p == run0 ? seg.z & 1 : 0)) * W + hw) * 16 + g;
  };
  auto finish = [&](int64_t row, float m, float l, const float (&v)[E]) {
    uint32_t y[E / 2];
#pragma unroll
    for (int e = 0; e < E; e += 2)
      y[e / 2] = l == 0.f ? 0u : pack_bf16(v[e] / l * a.kv.v_scale, v[e + 1] / l * a.kv.v_scale);
    uint16_t* to = a.out + row * D + lane * E;
    if constexpr (E == 2) *reinterpret_cast<uint32_t*>(to) = y[0];
    else if constexpr (E == 4) *reinterpret_cast<uint2*>(to) = make_uint2(y[0], y[1]);
    else *reinterpret_cast<uint4*>(to) = make_uint4(y[0], y[1], y[2], y[3]);
    if (lane == 0 && a.lse)
      a.lse[row] = a.kv.dtype != FT_KV_BF16 ? lse_of<true>(m, l) : lse_of<false>(m, l);
  };
  auto load = [&](int64_t at, bool on, float2& ml, float (&y)[E]) {
    ml = make_float2(-INFINITY, 0.f);
#pragma unroll
    for (int e = 0; e < E; ++e) y[e] = 0.f;
    if (!on) return;
    ml = *reinterpret_cast<const float2*>(a.part_ml + at * 2);
    const float* p = a.part_o + at * D + lane * E;
    if constexpr (E == 2) {
      const float2 x = *reinterpret_cast<const float2*>(p);
      y[0] = x.x; y[1] = x.y;
    } else {
#pragma unroll
      for (int e = 0; e < E; e += 4) {
        const float4 x = *reinterpret_cast<const float4*>(p + e);
        y[e] = x.x; y[e + 1] = x.y; y[e + 2] = x.z; y[e + 3] = x.w;
      }
    }
  };
  float2 ml[kFlight];
  float y[kFlight][E];
  if (seg.w - run0 < 2) {   // two pieces: as many jobs of a warp at once as are in flight
    constexpr int JF = kFlight / 2;
    for (int i0 = warp; i0 < mine; i0 += JF * kJoinWarps) {
#pragma unroll
      for (int j = 0; j < kFlight; ++j) {
        const int job = me + (i0 + (j >> 1) * kJoinWarps) * blocks;
        load(piece_of(job, run0 + (j & 1)), row_of(job) >= 0, ml[j], y[j]);
      }
#pragma unroll
      for (int j = 0; j < JF; ++j) {
        const int64_t row = row_of(me + (i0 + j * kJoinWarps) * blocks);
        if (row < 0) continue;
        float m = -INFINITY, l = 0.f, v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = 0.f;
        add_pieces<2, E>(ml + 2 * j, y + 2 * j, m, l, v);
        finish(row, m, l, v);
      }
    }
    return;
  }
  for (int i0 = 0; i0 < mine; i0 += teams) {
    const int job = me + (i0 + team) * blocks;
    const int64_t row = row_of(job);
    float m = -INFINITY, l = 0.f, v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = 0.f;
    if (row >= 0) {
      for (int p0 = run0 + part; p0 <= seg.w; p0 += kFlight << tl) {
#pragma unroll
        for (int j = 0; j < kFlight; ++j) {
          const int p = p0 + (j << tl);
          load(piece_of(job, p), p <= seg.w, ml[j], y[j]);
        }
        add_pieces<kFlight, E>(ml, y, m, l, v);
      }
    }
    if (tl > 0) {   // uniform over the block, as are i0 and mine
#pragma unroll
      for (int e = 0; e < E; ++e) sums[warp][lane * E + e] = v[e];
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
          for (int e = 0; e < E; ++e) v[e] = fmaf(f, sums[warp + w][lane * E + e], v[e]);
        }
      }
      __syncthreads();
    }
    if (row >= 0 && part == 0) finish(row, m, l, v);
  }
}

template <int D, int DT, int NG>
cudaError_t launch_d(AttendArgs a, int num_sms, cudaStream_t stream) {
  using S = AttnShape<D, DT, NG>;
  a.heads_log2 = 0;
  while (2 << a.heads_log2 <= S::kWarps && a.kv.Hkv * a.gt % (2 << a.heads_log2) == 0) ++a.heads_log2;
  const size_t smem = S::kGroups * S::kRing + (a.B > 32 ? (size_t)(a.B + 1) * 4 : 0);
  cudaError_t e;
  static SmemGrant grant;   // for the most sequences that a call may have
  if ((e = grant_smem(grant, k_attend<D, DT, NG>, S::kGroups * S::kRing + 4 * (kMaxSeqs + 1))) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(S::kBlocks * num_sms));
  cfg.blockDim = dim3(S::kGroups * S::kWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, k_attend<D, DT, NG>, a)) != cudaSuccess) return e;
  // Warps of a block of k_join. NVFP4: eight, so that all blocks run at once (48 ragged sequences, weights still in one
  // f16, 58.2 us, 60.5 with sixteen of as many registers, 57.2 for 56.3 with sixteen of 40; one of 777 keys 6.7, 6.8 and 7.8).
  // Heads of 256 where an SM has two runs (E4M3): eight as well, because two blocks of sixteen leave 64 registers, too
  // few for four rows of 256 in flight: two sequences of 62648 51.7 -> 50.0 us, 13 up to 24001 60.8 -> 59.9, one of 777 9.4 -> 8.8.
  constexpr int kRuns = S::kBlocks * S::kGroups;   // an SM
  constexpr int kJoinWarps = DT == kKvNvfp4 || (D == 256 && kRuns > 1) ? 8 : 16;
  // Blocks of k_join that an SM holds: as many as there are runs, but not more than two of sixteen warps, which leaves
  // each thread 64 registers. One would take 36.1 us for 34.4 (64 sequences of 1000, E4M3), 51.2 for 49.9 (bf16).
  constexpr int kJoinBlocks = DT == kKvNvfp4 ? 3 : kRuns < 2 ? kRuns : 2;
  cfg.gridDim = dim3((unsigned)(kRuns * num_sms));   // a block for every run
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, k_join<D, S::kWarps, kJoinWarps, kJoinBlocks, DT == kKvNvfp4 && D <= 128 ? 8 : 4>, a);
}

template <int D, int DT>
cudaError_t launch_g(const AttendArgs& a, int num_sms, cudaStream_t stream) {
  return a.group <= 8 ? launch_d<D, DT, 1>(a, num_sms, stream) : launch_d<D, DT, 2>(a, num_sms, stream);
}

template <int DT>
cudaError_t launch_t(const AttendArgs& a, int num_sms, cudaStream_t stream) {
  switch (a.kv.D) {
    case 64: return launch_g<64, DT>(a, num_sms, stream);
    case 128: return launch_g<128, DT>(a, num_sms, stream);
    case 256: return launch_g<256, DT>(a, num_sms, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_attend(const AttendArgs& args, int num_sms, cudaStream_t stream) {
  AttendArgs a = args;
  a.group = a.Hq / a.kv.Hkv;
  a.gt = (a.group + 15) / 16;
  a.same_strides = a.kv.k_page_stride == a.kv.v_page_stride && a.kv.k_slot_stride == a.kv.v_slot_stride &&
                   a.kv.k_head_stride == a.kv.v_head_stride && a.sc.k_page == a.sc.v_page &&
                   a.sc.k_slot == a.sc.v_slot && a.sc.k_head == a.sc.v_head;
  page_division(a.kv.page_size, a.div_mul, a.div_shift);
  const int64_t slots = (int64_t)a.table_width * a.kv.page_size;
  a.max_len = (int)(slots < (1 << 30) ? slots : 1 << 30);
  // The kernels number the units of all sequences (64 keys at least, up to six more of a sequence for its ends and its
  // charge) in 32 bits: 4096 sequences may have 2^25 - 512 keys each inside the window, 128 of them 2^30 - 512.
  const int64_t most = ((1ll << 31) / a.B - 8) * 64;
  if (a.max_len > most && (a.window == 0 || a.window > most)) a.max_len = (int)most;
  switch (a.kv.dtype) {
    case FT_KV_BF16: return launch_t<FT_KV_BF16>(a, num_sms, stream);
    case FT_KV_E4M3: return launch_t<FT_KV_E4M3>(a, num_sms, stream);
  }
  return launch_t<kKvNvfp4>(a, num_sms, stream);
}

}  // namespace ftmoe
