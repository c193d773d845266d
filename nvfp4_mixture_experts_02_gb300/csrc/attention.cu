// Attention of one new token per sequence over a paged key-value cache.
//
//   s_j = scale * k_scale * (q . k_j)    for j in [max(0, len - window), len)
//   out = sum_j exp(s_j - m) v_scale v_j / sum_j exp(s_j - m),  m = max_j s_j
//   lse = m + ln(sum_j exp(s_j - m));   an empty sequence: out = 0, lse = -inf
//
// Every key and value is read once, by one block, for all the query heads that share it: the call
// is bound by the cache's bytes (4 G operations per key element of 1 or 2 bytes).
//
// k_attend: the work is the list of (sequence, key head, unit of keys), in that order; every block
// takes an equal run of it, whatever the lengths, found from the lengths on the device (no host
// synchronisation). A run covers pieces of one or more (sequence, head) segments. Inside a piece
// the warps take 16 keys in turn, each with its own ring of asynchronous 16-byte copies (rows of
// the pages to swizzled shared memory), its own running maximum and sum and its own 16 x D sums in
// registers; they are joined at the piece's end. A piece that is its whole segment is finished
// there; the others leave (maximum, sum, sums) in the workspace for k_join, which adds a segment's
// pieces in order. Masked and missing keys are not read: their rows are zeros in shared memory, so
// that whatever the pages hold there (NaN, stale values) cannot reach a sum.
//
// Products: q k^T and p v as m16n8k16 with the 16 rows as query heads, float32 sums. bf16 caches:
// bf16 operands; p, in (0, 1], is split into two bf16 (16 significant bits, so that p is not rounded
// to 8); up to eight heads the second part rides in the idle rows 8 to 15. E4M3 caches: keys and values
// become f16 exactly, q is f16 after a scaling of its row by a power of two (exact but for elements
// under 2^-29 of the row's largest), p rounds to f16 (11 bits). Statistics and sums are float32.
#include <cmath>
#include <cuda_runtime.h>

#include "ftmoe_internal.h"
#include "ftmoe_mma.cuh"
#include "ftmoe_tc.cuh"

namespace ftmoe {

namespace {

template <int D, bool F8>
struct AttnShape {
  static constexpr int kRow = D * (F8 ? 1 : 2);       // bytes of a key or value
  static constexpr int kCpr = kRow / 16;              // 16-byte pieces of it
  static constexpr int kWarps = !F8 && D == 256 ? 4 : 8;
  static constexpr int kStageBytes = 2 * 16 * kRow;   // 16 keys and 16 values
  static constexpr int kFit = 192 * 1024 / (kWarps * kStageBytes);
  static constexpr int kStages = kFit < 8 ? kFit : 8;
  static constexpr int kUnit = 16 * kWarps;           // keys of a unit
  static constexpr int kRing = kWarps * kStages * kStageBytes;
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Offset of 16-byte piece c of row r in a tile of rows of kCpr pieces: pieces are exchanged within
// groups of eight (four) so that eight rows' same piece lie in different banks.
template <int CPR>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  if constexpr (CPR >= 8) return (uint32_t)(r * CPR + (c ^ (r & 7))) * 16;
  else return (uint32_t)(r * CPR + (c ^ ((r >> 1) & 3))) * 16;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// First key and number of units of a sequence.
__device__ __forceinline__ void span(int len, int window, int unit, int& first, int& units) {
  first = window > 0 && len > window ? len - window : 0;
  units = len > 0 ? (len + unit - 1) / unit - first / unit : 0;
}

template <int D, bool F8, int GM>
__global__ void __launch_bounds__(AttnShape<D, F8>::kWarps * 32, 1) k_attend(const AttendArgs a) {
  using S = AttnShape<D, F8>;
  constexpr int W = S::kWarps, ST = S::kStages, CPR = S::kCpr, NT = D / 8, KS = D / 16;
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ float wm[W][16], wl[W][16];
  __shared__ int scan[W];
  int* cum = reinterpret_cast<int*>(smem + S::kRing);   // [B + 1] units before each sequence
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = lane & 3, r = lane >> 2;
  const int HS = a.kv.Hkv * a.gt;   // segments of a sequence

  // units before each sequence
  {
    const int per = (a.B + W * 32 - 1) / (W * 32);
    const int b0 = threadIdx.x * per;
    int mine = 0;
    for (int b = b0; b < min(b0 + per, a.B); ++b) {
      int first, n;
      span(a.seq_lens[b], a.window, S::kUnit, first, n);
      mine += n;
    }
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    int at = inc - mine;
    for (int w = 0; w < warp; ++w) at += scan[w];
    for (int b = b0; b < min(b0 + per, a.B); ++b) {
      int first, n;
      span(a.seq_lens[b], a.window, S::kUnit, first, n);
      cum[b] = at;
      at += n;
    }
    if (b0 < a.B && b0 + per >= a.B) cum[a.B] = at;
    __syncthreads();
  }
  const int64_t total = (int64_t)cum[a.B] * HS;
  const int64_t quota = (total + gridDim.x - 1) / gridDim.x;
  if (blockIdx.x == 0) {   // the plan, for k_join
    for (int b = threadIdx.x; b <= a.B; b += W * 32) a.plan[b] = cum[b];
  }
  int64_t u = quota * blockIdx.x;
  const int64_t u_end = min(u + quota, total);
  const uint32_t ring = smem_addr(smem) + (uint32_t)(warp * ST * S::kStageBytes);

  while (u < u_end) {
    // the piece that begins at u
    int lo = 0, hi = a.B;   // cum[lo] * HS <= u < cum[hi] * HS
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((int64_t)cum[mid] * HS <= u) lo = mid;
      else hi = mid;
    }
    const int b = lo;
    const int len = a.seq_lens[b];
    int first, units;
    span(len, a.window, S::kUnit, first, units);
    const int64_t local = u - (int64_t)cum[b] * HS;
    const int hs = (int)(local / units);
    const int u0 = (int)(local - (int64_t)hs * units);
    const int n_units = (int)min((int64_t)(units - u0), u_end - u);
    const int kvh = hs / a.gt, g0 = (hs - kvh * a.gt) * 16;
    const int G = min(a.group - g0, 16);
    const int key0 = (first / S::kUnit + u0) * S::kUnit;
    const int key1 = min(len, key0 + n_units * S::kUnit);   // keys of the piece: [key0, key1)

    // ---- the ring: sub-tile i of this warp = keys key0 + (i * W + warp) * 16 ..
    const int subs = (key1 - key0 - warp * 16 + W * 16 - 1) / (W * 16);   // may be <= 0
    const int n_sub = key1 - key0 > warp * 16 ? subs : 0;
    const int32_t* table = a.block_table + (int64_t)b * a.table_width;
    int page = -1, slot = 0;
    auto look_up = [&](int i) {   // lane l < 16: the page and slot of key l of sub-tile i
      const int j = key0 + (i * W + warp) * 16 + (lane & 15);
      page = -1;
      if (i < n_sub && j >= first && j < key1) {
        const int col = (int)((__umulhi((uint32_t)a.div_mul, (uint32_t)j) + (uint32_t)j) >> a.div_shift);
        slot = j - col * a.kv.page_size;
        page = col < a.table_width ? table[col] : a.kv.num_pages;
      }
    };
    auto fetch = [&](int i) {     // the copies of sub-tile i, whose pages look_up has found
      int64_t ko = -1, vo = -1;
      if (page >= 0 && page < a.kv.num_pages) {
        ko = ((int64_t)page * a.kv.k_page_stride + (int64_t)slot * a.kv.k_slot_stride +
              (int64_t)kvh * a.kv.k_head_stride) * (F8 ? 1 : 2);
        vo = ((int64_t)page * a.kv.v_page_stride + (int64_t)slot * a.kv.v_slot_stride +
              (int64_t)kvh * a.kv.v_head_stride) * (F8 ? 1 : 2);
      } else if (i < n_sub && lane < 16) {
        const int j = key0 + (i * W + warp) * 16 + lane;
        if (j >= first && j < key1) atomicOr(a.err, kErrBadPage);   // no such page: read as zeros
      }
      if (i < n_sub) {
        const uint32_t st = ring + (uint32_t)((i % ST) * S::kStageBytes);
        constexpr int RPI = 32 / CPR;   // rows of one warp-wide copy
#pragma unroll
        for (int p = 0; p < 16 / RPI; ++p) {
          const int row = p * RPI + lane / CPR, ch = lane % CPR;
          const int64_t k_at = __shfl_sync(0xffffffffu, ko, row);
          const int64_t v_at = __shfl_sync(0xffffffffu, vo, row);
          cp_async16(st + swz<CPR>(row, ch),
                     static_cast<const char*>(a.kv.k) + (k_at < 0 ? 0 : k_at) + ch * 16, k_at >= 0);
          cp_async16(st + 16 * S::kRow + swz<CPR>(row, ch),
                     static_cast<const char*>(a.kv.v) + (v_at < 0 ? 0 : v_at) + ch * 16, v_at >= 0);
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

    // ---- q: the A operand, 16 heads x D
    uint32_t q[KS][4];
    float sl0, sl1;   // log2 units per unit of the raw product, rows r and r + 8
    {
      const uint16_t* qb = a.q + (int64_t)b * a.q_stride + (int64_t)(kvh * a.group + g0) * D;
      const bool on0 = r < G, on1 = GM == 16 && r + 8 < G;
      sl0 = sl1 = a.scale * a.kv.k_scale * kLog2e;
      if constexpr (!F8) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const int d = 16 * ks + 2 * c;
          q[ks][0] = on0 ? *reinterpret_cast<const uint32_t*>(qb + r * D + d) : 0u;
          q[ks][2] = on0 ? *reinterpret_cast<const uint32_t*>(qb + r * D + d + 8) : 0u;
          q[ks][1] = on1 ? *reinterpret_cast<const uint32_t*>(qb + (r + 8) * D + d) : 0u;
          q[ks][3] = on1 ? *reinterpret_cast<const uint32_t*>(qb + (r + 8) * D + d + 8) : 0u;
        }
      } else {
        float top0 = 0.f, top1 = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const int d = 16 * ks + 4 * c;   // E4M3 keys come four elements to a lane
          uint2 v0 = make_uint2(0, 0), v1 = make_uint2(0, 0);
          if (on0) v0 = *reinterpret_cast<const uint2*>(qb + r * D + d);
          if (on1) v1 = *reinterpret_cast<const uint2*>(qb + (r + 8) * D + d);
          q[ks][0] = v0.x; q[ks][2] = v0.y; q[ks][1] = v1.x; q[ks][3] = v1.y;
          top0 = fmaxf(top0, finite_top(v0.x, v0.y));
          top1 = fmaxf(top1, finite_top(v1.x, v1.y));
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, o));
          top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, o));
        }
        float up0, up1, down0, down1;
        f16_scale(top0, up0, down0);
        f16_scale(top1, up1, down1);
        sl0 *= down0;
        sl1 *= down1;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          q[ks][0] = pack_f16(bf16_lo(q[ks][0]) * up0, bf16_hi(q[ks][0]) * up0);
          q[ks][2] = pack_f16(bf16_lo(q[ks][2]) * up0, bf16_hi(q[ks][2]) * up0);
          q[ks][1] = pack_f16(bf16_lo(q[ks][1]) * up1, bf16_hi(q[ks][1]) * up1);
          q[ks][3] = pack_f16(bf16_lo(q[ks][3]) * up1, bf16_hi(q[ks][3]) * up1);
        }
      }
    }

    float o[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

    for (int i = 0; i < n_sub; ++i) {
      cp_async_wait<ST - 2>();
      __syncwarp();
      const uint32_t st = ring + (uint32_t)((i % ST) * S::kStageBytes);
      // s = q k^T, two tiles of eight keys
      float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
      {
        const int key = (lane >> 4) * 8 + (lane & 7), half = (lane >> 3) & 1;
        if constexpr (!F8) {
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            uint32_t k[4];
            ldmatrix4(k, st + swz<CPR>(key, 2 * ks + half));
            mma_bf16(s0, q[ks][0], q[ks][1], q[ks][2], q[ks][3], k[0], k[1]);
            mma_bf16(s1, q[ks][0], q[ks][1], q[ks][2], q[ks][3], k[2], k[3]);
          }
        } else {
#pragma unroll
          for (int ks = 0; ks < KS; ks += 2) {
            uint32_t k[4];
            ldmatrix4(k, st + swz<CPR>(key, ks + half));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              mma_f16(s0, q[ks + e][0], q[ks + e][1], q[ks + e][2], q[ks + e][3],
                      e4m3x2_to_f16x2(k[e]), e4m3x2_to_f16x2(k[e] >> 16));
              mma_f16(s1, q[ks + e][0], q[ks + e][1], q[ks + e][2], q[ks + e][3],
                      e4m3x2_to_f16x2(k[2 + e]), e4m3x2_to_f16x2(k[2 + e] >> 16));
            }
          }
        }
      }
      // the next copies go into the stage that the previous sub-tile has left
      fetch(i + ST - 1);
      look_up(i + ST);
      // scores in log2 units; keys outside [first, key1) do not count
      const int j0 = key0 + (i * W + warp) * 16;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        s0[e] *= sl0; s1[e] *= sl0;
        s0[2 + e] *= sl1; s1[2 + e] *= sl1;
      }
      if (j0 < first || j0 + 16 > key1) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = j0 + 2 * c + (e & 1);
          if (j < first || j >= key1) s0[e] = -INFINITY;
          if (j + 8 < first || j + 8 >= key1) s1[e] = -INFINITY;
        }
      }
      float t0 = fmaxf(fmaxf(s0[0], s0[1]), fmaxf(s1[0], s1[1]));
      float t1 = fmaxf(fmaxf(s0[2], s0[3]), fmaxf(s1[2], s1[3]));
#pragma unroll
      for (int x = 1; x < 4; x <<= 1) {
        t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, x));
        if (GM == 16) t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, x));
      }
      const bool up = t0 > m0 || (GM == 16 && t1 > m1);
      if (__any_sync(0xffffffffu, up)) {   // a new maximum: what is summed shrinks
        const float n0 = fmaxf(m0, t0), n1 = GM == 16 ? fmaxf(m1, t1) : n0;
        const float f0 = m0 == -INFINITY ? 0.f : exp2_fast(m0 - n0);
        const float f1 = GM == 16 ? (m1 == -INFINITY ? 0.f : exp2_fast(m1 - n1)) : f0;
        m0 = n0;
        m1 = n1;
        l0 *= f0;
        l1 *= f1;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          o[n][0] *= f0; o[n][1] *= f0;
          o[n][2] *= f1; o[n][3] *= f1;
        }
      }
      const float b0 = m0 == -INFINITY ? 0.f : m0;   // no key yet: every p is 0
      const float b1 = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        s0[e] = exp2_fast(s0[e] - b0);
        s1[e] = exp2_fast(s1[e] - b0);
        l0 += s0[e] + s1[e];
        if (GM == 16) {
          s0[2 + e] = exp2_fast(s0[2 + e] - b1);
          s1[2 + e] = exp2_fast(s1[2 + e] - b1);
          l1 += s0[2 + e] + s1[2 + e];
        }
      }
      // o += p v
      const int key = ((lane >> 3) & 1) * 8 + (lane & 7), half = lane >> 4;
      const uint32_t vs = st + 16 * S::kRow;
      if constexpr (!F8) {
        uint32_t p[4], pl[4];
        p[0] = pack_bf16(s0[0], s0[1]);
        p[2] = pack_bf16(s1[0], s1[1]);
        const uint32_t rest0 = pack_bf16(s0[0] - bf16_lo(p[0]), s0[1] - bf16_hi(p[0]));
        const uint32_t rest2 = pack_bf16(s1[0] - bf16_lo(p[2]), s1[1] - bf16_hi(p[2]));
        if (GM == 16) {
          p[1] = pack_bf16(s0[2], s0[3]);
          p[3] = pack_bf16(s1[2], s1[3]);
          pl[0] = rest0;
          pl[2] = rest2;
          pl[1] = pack_bf16(s0[2] - bf16_lo(p[1]), s0[3] - bf16_hi(p[1]));
          pl[3] = pack_bf16(s1[2] - bf16_lo(p[3]), s1[3] - bf16_hi(p[3]));
        } else {   // rows 8 to 15 carry what rows 0 to 7 lose by rounding
          p[1] = rest0;
          p[3] = rest2;
        }
#pragma unroll
        for (int n = 0; n < NT; n += 2) {
          uint32_t v[4];
          ldmatrix4_trans(v, vs + swz<CPR>(key, n + half));
          mma_bf16(o[n], p[0], p[1], p[2], p[3], v[0], v[1]);
          mma_bf16(o[n + 1], p[0], p[1], p[2], p[3], v[2], v[3]);
          if (GM == 16) {
            mma_bf16(o[n], pl[0], pl[1], pl[2], pl[3], v[0], v[1]);
            mma_bf16(o[n + 1], pl[0], pl[1], pl[2], pl[3], v[2], v[3]);
          }
        }
      } else {
        uint32_t p[4];
        p[0] = pack_f16(s0[0], s0[1]);
        p[2] = pack_f16(s1[0], s1[1]);
        p[1] = GM == 16 ? pack_f16(s0[2], s0[3]) : 0u;
        p[3] = GM == 16 ? pack_f16(s1[2], s1[3]) : 0u;
#pragma unroll
        for (int n = 0; n < NT; n += 4) {   // two 16-byte pieces: dims 8 n .. 8 n + 31
          uint32_t v[4];
          ldmatrix4_trans(v, vs + swz<CPR>(key, n / 2 + half));
          // a register holds (key, dim d), (key, d + 1), (key + 1, d), (key + 1, d + 1)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t x = __byte_perm(v[2 * h], 0, 0x3120);
            const uint32_t y = __byte_perm(v[2 * h + 1], 0, 0x3120);
            mma_f16(o[n + 2 * h], p[0], p[1], p[2], p[3], e4m3x2_to_f16x2(x),
                    e4m3x2_to_f16x2(y));            // even dims
            mma_f16(o[n + 2 * h + 1], p[0], p[1], p[2], p[3], e4m3x2_to_f16x2(x >> 16),
                    e4m3x2_to_f16x2(y >> 16));      // odd dims
          }
        }
      }
      __syncwarp();   // every lane has read the stage before it is filled again
    }
    cp_async_wait<0>();
#pragma unroll
    for (int x = 1; x < 4; x <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, x);
      l1 += __shfl_xor_sync(0xffffffffu, l1, x);
    }

    // ---- join the warps: sums [warp][head][D] in the ring's memory
    __syncthreads();
    float* sums = reinterpret_cast<float*>(smem) + (size_t)warp * 16 * D;
    if (c == 0) {
      wm[warp][r] = m0;
      wl[warp][r] = l0;
      if (GM == 16) {
        wm[warp][r + 8] = m1;
        wl[warp][r + 8] = l1;
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (GM == 8) {
        o[n][0] += o[n][2];
        o[n][1] += o[n][3];
      }
      // dims of this lane's two columns
      const int d0 = F8 ? 16 * (n / 2) + 4 * c + (n & 1) : 8 * n + 2 * c;
      const int d1 = F8 ? d0 + 2 : d0 + 1;
      if (r < G) {
        sums[r * D + d0] = o[n][0];
        sums[r * D + d1] = o[n][1];
      }
      if (GM == 16 && r + 8 < G) {
        sums[(r + 8) * D + d0] = o[n][2];
        sums[(r + 8) * D + d1] = o[n][3];
      }
    }
    __syncthreads();
    const bool whole = n_units == units;
    const int64_t part = 2 * (int64_t)blockIdx.x + (u == quota * blockIdx.x ? 0 : 1);
    for (int x = threadIdx.x; x < G * D; x += W * 32) {
      const int g = x / D, d = x - g * D;
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < W; ++w) m = fmaxf(m, wm[w][g]);
      const float base = m == -INFINITY ? 0.f : m;
      float l = 0.f, v = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float f = exp2_fast(wm[w][g] - base);
        l = fmaf(f, wl[w][g], l);
        v = fmaf(f, reinterpret_cast<const float*>(smem)[(size_t)w * 16 * D + x], v);
      }
      const int64_t row = (int64_t)b * a.Hq + kvh * a.group + g0 + g;
      if (whole) {
        const float y = l == 0.f ? 0.f : v / l * a.kv.v_scale;   // no weight at all: zeros
        a.out[row * D + d] = (uint16_t)(pack_bf16(y, 0.f) & 0xFFFFu);
        if (d == 0 && a.lse) a.lse[row] = (m + log2f(l)) * kLn2;
      } else {
        a.part_o[(part * 16 + g) * D + d] = v;
        if (d == 0) {
          a.part_ml[(part * 16 + g) * 2] = m;
          a.part_ml[(part * 16 + g) * 2 + 1] = l;
        }
      }
    }
    __syncthreads();   // before the ring is filled again
    u += n_units;
  }
}

// One warp per (sequence, query head) that k_attend has not finished: its pieces in order, or
// zeros for an empty sequence.
constexpr int kJoinWarps = 4;
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) k_join(const AttendArgs a, int grid) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
  if (row >= (int64_t)a.B * a.Hq) return;
  const int b = (int)(row / a.Hq), head = (int)(row - (int64_t)b * a.Hq);
  constexpr int E = D / 32;
  const int units = a.plan[b + 1] - a.plan[b];
  if (units == 0) {
#pragma unroll
    for (int e = 0; e < E; ++e) a.out[row * D + lane + 32 * e] = 0;
    if (lane == 0 && a.lse) a.lse[row] = -INFINITY;
    return;
  }
  const int HS = a.kv.Hkv * a.gt;
  const int64_t total = (int64_t)a.plan[a.B] * HS;
  const int64_t quota = (total + grid - 1) / grid;
  const int kvh = head / a.group, in = head - kvh * a.group;
  const int hs = kvh * a.gt + in / 16, g = in % 16;
  const int64_t s0 = (int64_t)a.plan[b] * HS + (int64_t)hs * units, s1 = s0 + units;
  const int64_t first = s0 / quota, last = (s1 - 1) / quota;   // blocks with a piece of it
  if (first == last) return;   // one piece: k_attend has finished it
  float m = -INFINITY;
  for (int64_t p = first + lane; p <= last; p += 32) {
    const int64_t part = 2 * p + (p * quota >= s0 ? 0 : 1);
    m = fmaxf(m, a.part_ml[(part * 16 + g) * 2]);
  }
  m = warp_max(m);
  const float base = m == -INFINITY ? 0.f : m;
  float l = 0.f, v[E];
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = 0.f;
#pragma unroll 4
  for (int64_t p = first; p <= last; ++p) {
    const int64_t part = 2 * p + (p * quota >= s0 ? 0 : 1);
    const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + (part * 16 + g) * 2);
    const float f = exp2_fast(ml.x - base);
    l = fmaf(f, ml.y, l);
#pragma unroll
    for (int e = 0; e < E; ++e)
      v[e] = fmaf(f, a.part_o[(part * 16 + g) * D + lane + 32 * e], v[e]);
  }
#pragma unroll
  for (int e = 0; e < E; ++e)
    a.out[row * D + lane + 32 * e] =
        (uint16_t)(pack_bf16(l == 0.f ? 0.f : v[e] / l * a.kv.v_scale, 0.f) & 0xFFFFu);
  if (lane == 0 && a.lse) a.lse[row] = (m + log2f(l)) * kLn2;
}

template <int D, bool F8, int GM>
cudaError_t launch_d(const AttendArgs& a, int num_sms, cudaStream_t stream) {
  using S = AttnShape<D, F8>;
  const size_t smem = S::kRing + (size_t)(a.B + 1) * 4;
  cudaError_t e;
  // set on every call: the attribute is per device and the call is host-side only
  if ((e = cudaFuncSetAttribute(k_attend<D, F8, GM>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)smem)) != cudaSuccess)
    return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)num_sms);
  cfg.blockDim = dim3(S::kWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, k_attend<D, F8, GM>, a)) != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)(((int64_t)a.B * a.Hq + kJoinWarps - 1) / kJoinWarps));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, k_join<D>, a, num_sms);
}

template <int D>
cudaError_t launch_g(const AttendArgs& a, int num_sms, cudaStream_t stream) {
  const bool f8 = a.kv.dtype == FT_KV_E4M3;
  if (a.group <= 8)
    return f8 ? launch_d<D, true, 8>(a, num_sms, stream) : launch_d<D, false, 8>(a, num_sms, stream);
  return f8 ? launch_d<D, true, 16>(a, num_sms, stream) : launch_d<D, false, 16>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_attend(const AttendArgs& args, int num_sms, cudaStream_t stream) {
  AttendArgs a = args;
  a.group = a.Hq / a.kv.Hkv;
  a.gt = (a.group + 15) / 16;
  // j / page_size for 0 <= j < 2^31 as (umulhi(mul, j) + j) >> shift
  int shift = 0;
  while ((1ll << shift) < a.kv.page_size) ++shift;
  a.div_shift = shift;
  a.div_mul = (int)(uint32_t)(((1ull << 32) * ((1ull << shift) - a.kv.page_size)) / a.kv.page_size + 1);
  switch (a.kv.D) {
    case 64: return launch_g<64>(a, num_sms, stream);
    case 128: return launch_g<128>(a, num_sms, stream);
    case 256: return launch_g<256>(a, num_sms, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ftmoe
