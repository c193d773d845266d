// y_t = W x_t for 1 to 64 tokens with a dense NVFP4 matrix W [N][K] (E2M1 codes, an E4M3 scale per
// 16 elements of a row, one float32 scale): the projections of a decode step.
//
// The matrix is read once: 9/16 byte per weight, and up to 64 products with each. A warp takes 16
// rows and, at a time, 128 elements of K: lane l the 32 elements 32 (l % 4) .. of rows l / 4 and
// l / 4 + 8 (one 16-byte load and two scale bytes each). e2m1 * e4m3 is exact in f16 (at most six
// significant bits, 2^-10 .. 2688), so a weight is one conversion and one multiply away from the A
// operand of m16n8k16; the order of K inside a product is free, as long as x follows it. x becomes
// f16 after a scaling per token by a power of two (exact but for elements under 2^-29 of the
// largest), the sums are float32, and the matrix's scale multiplies them at the end.
//
// k_linear_few (up to 8 tokens): the block's eight warps each hold an eighth of K and go down the
// block's row tiles, some pieces of 128 elements ahead in registers across tile ends, so the stream of
// weights does not stop; x is laid out once per block. A cluster of S blocks splits K when there are
// fewer row tiles than SMs or x does not fit one block. Partial sums are added in a fixed order (warps
// in shared memory, blocks through the cluster's).
//
// k_linear_mid (from 9 tokens, few rows): the same in one launch with tiles of 128 rows by 16 or 32
// tokens and K over a cluster, each of whose blocks lays its own slice of x out.
//
// k_linear_more (9 to 64 tokens, many rows): a launch of its own lays x out (k_linear_x). The work is
// the list of (256-row tile, 256 elements of K); each block takes an equal run of it. Every warp has 32
// rows of the tile, so that a piece of x read from shared memory meets 32 rows; the blocks' x comes by
// bulk copies into a ring. A tile that two runs share leaves float32 sums for k_linear_join, which adds
// them in order.
//
// What bounds it: a weight costs half a conversion, half a multiply and 1/256 of a product per eight
// tokens on the warp schedulers. At 100003 x 4096 (34 us of memory time): 1 token 41 us, 83 % of the
// measured copy rate; 5 tokens 43; 16 tokens 57; 32 and 64 tokens 87 and 138 us, where the m16n8k16 rate
// (1024 products per clock and SM: 44 and 88 us) is the larger bound. The same tiles through tcgen05 with
// the converted weights in tensor memory took 103 us at 16 tokens and 118 at 64, where it was the faster; it
// is not in this file. Its rate per 128 x 16 block does not depend on the tokens, but the hand-over through
// tensor memory and barriers costs 1.2 us per 128 x 256 weights. Small matrices are bound by latency: 1 x 4096 x 4096 takes 4.6 us for 1.4 us of
// memory time, a chain of launch, x's layout, load, conversion, sum and store; two pieces ahead beat four
// there (5.2 or 5.9 us before x's layout was one token's own code).
#include <cmath>
#include <cuda_runtime.h>

#include "ftmoe_internal.h"
#include "ftmoe_mma.cuh"
#include "ftmoe_tc.cuh"

namespace ftmoe {

namespace {

constexpr int kLinWarps = 8;
constexpr int kLinUnit = 256;              // elements of K in a unit of work
constexpr size_t kLinXMax = 200 * 1024;    // x of one block in shared memory

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
__device__ __forceinline__ float ld_cluster(uint32_t addr, uint32_t rank) {
  float v;
  asm volatile("{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\t"
               "ld.shared::cluster.f32 %0, [a];\n\t}"
               : "=f"(v)
               : "r"(addr), "r"(rank)
               : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr, uint32_t rank) {
  float4 v;
  asm volatile("{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\t"
               "ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [a];\n\t}"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr), "r"(rank)
               : "memory");
  return v;
}
__device__ __forceinline__ uint4 ld_once(const uint8_t* p) {   // weights: read once
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// 128 elements of 16 MT rows: this lane's 32 of rows l / 4, l / 4 + 8, ...
template <int MT>
struct Piece {
  uint4 w[2 * MT];
  uint32_t s[2 * MT];
};

// This lane's place in 16 MT rows of the matrix (rows past the last read the last one again).
template <int MT>
struct Rows {
  const uint8_t *codes, *scales;    // row0 + l / 4, element k0
  uint32_t to_row[2 * MT];          // from there to rows l / 4 + 8 i, in codes; an eighth in scales
  __device__ __forceinline__ void set(const LinearArgs& a, int row0, int r, int k0) {
    const int row = min(row0 + r, a.N - 1);
    codes = a.codes + (size_t)row * (a.K >> 1) + (k0 >> 1);
    scales = a.scales + (size_t)row * (a.K >> 4) + (k0 >> 4);
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i)
      to_row[i] = (uint32_t)(min(row0 + r + 8 * i, a.N - 1) - row) * (uint32_t)(a.K >> 1);
  }
  // piece p's lines towards L2: no data is taken, so this may run ahead of the launches before
  __device__ __forceinline__ void prefetch(int p) const {
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(codes + to_row[i] + p * 64));
    asm volatile("prefetch.global.L2 [%0];" ::"l"(scales + p * 8));
  }
  // piece p from k0 on; off: scales of zero, so that nothing counts
  __device__ __forceinline__ void load(Piece<MT>& w, int p, bool on) const {
    if (on) {
#pragma unroll
      for (int i = 0; i < 2 * MT; ++i) w.w[i] = ld_once(codes + to_row[i] + p * 64);
#pragma unroll
      for (int i = 0; i < 2 * MT; ++i)
        w.s[i] = *reinterpret_cast<const uint16_t*>(scales + (to_row[i] >> 3) + p * 8);
    } else {
#pragma unroll
      for (int i = 0; i < 2 * MT; ++i) w.s[i] = 0;
    }
  }
};

// Eight codes (a word) times a splat scale: four f16x2.
__device__ __forceinline__ void dequant8(uint32_t w, uint32_t s, uint32_t (&h)[4]) {
  e2m1x8_to_f16x2x4(w, h[0], h[1], h[2], h[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = hmul2(h[i], s);
}
__device__ __forceinline__ uint32_t word(const uint4& v, int j) {
  return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
}

// acc += the piece's products with x, NT groups of eight tokens; xp: this lane's first unit of x, the
// next eight elements' units xj further, the next eight tokens' 32
template <int MT, int NT>
__device__ __forceinline__ void products(float (&acc)[MT][NT][4], const Piece<MT>& w, const uint4* xp,
                                         int xj) {
  uint32_t lo[2 * MT], hi[2 * MT];   // scales of elements 0-15 and 16-31, splat
#pragma unroll
  for (int i = 0; i < 2 * MT; ++i) {
    const uint32_t s = e4m3x2_to_f16x2(w.s[i]);
    lo[i] = splat_lo(s);
    hi[i] = splat_hi(s);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t h[2 * MT][4];
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) dequant8(word(w.w[i], j), j < 2 ? lo[i] : hi[i], h[i]);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint4 b = xp[j * xj + n * 32];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        mma_f16(acc[m][n], h[2 * m][0], h[2 * m + 1][0], h[2 * m][1], h[2 * m + 1][1], b.x, b.y);
        mma_f16(acc[m][n], h[2 * m][2], h[2 * m + 1][2], h[2 * m][3], h[2 * m + 1][3], b.z, b.w);
      }
    }
  }
}

// Eight bf16 times a power of two `up` (splat, exact in bf16) as f16.
__device__ __forceinline__ uint4 to_f16(uint4 v, uint32_t up) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(w[j]) : "r"(up));
    w[j] = pack_f16(bf16_lo(w[j]), bf16_hi(w[j]));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// Running largest magnitudes of bf16 pairs (NaN does not count).
__device__ __forceinline__ void pair_top(uint32_t& top, uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    asm("max.bf16x2 %0, %0, %1;" : "+r"(top) : "r"(w[j] & 0x7FFF7FFFu));
}
__device__ __forceinline__ float top_of(uint32_t pair) { return fmaxf(bf16_lo(pair), bf16_hi(pair)); }
__device__ __forceinline__ float finite_top8(uint4 v) {
  return fmaxf(finite_top(v.x, v.y), finite_top(v.z, v.w));
}
__device__ __forceinline__ uint32_t splat_bf16(float v) {   // of a power of two
  return __byte_perm(__float_as_uint(v), 0, 0x3232);
}

// 16-byte unit of elements k .. k + 7 of token n in the B operand's order, `tok` tokens wide: unit
// ((piece * 4 + j) * tok + n) * 4 + q holds elements 32 q + 8 j .. of the 128-element piece.
__device__ __forceinline__ int x_unit(int k, int n, int tok) {
  const int k8 = (k >> 3) & 15;
  return (((k >> 7) * 4 + (k8 & 3)) * tok + n) * 4 + (k8 >> 2);
}

// x of tokens n0 .. n0 + TN - 1 (of T), elements [ka, kb), to f16 at dst (units of the block's slice, which
// begins at element k0), with a power of two per token in down[]. One warp; up to 512 elements stay in
// registers between the search for the largest and the conversion, TN tokens' loads at a time.
template <int TN>
__device__ __forceinline__ void stage_x(const LinearArgs& a, int t0, int n0, int T, int ka, int kb, int k0,
                                        int tok, uint4* dst, float* down) {
  const int lane = threadIdx.x & 31;
  const uint16_t* x = a.x + (size_t)(t0 + n0) * a.x_stride;
  const int cnt = min(T - n0, TN);
  uint4 v[TN][2];
  uint32_t top[TN] = {};
  auto get = [&](int j, int k) {
    return j < cnt && k < kb && k < a.K
               ? *reinterpret_cast<const uint4*>(x + (size_t)j * a.x_stride + k)
               : make_uint4(0, 0, 0, 0);
  };
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) v[j][i] = get(j, ka + lane * 8 + i * 256);
#pragma unroll
  for (int j = 0; j < TN; ++j)
#pragma unroll
    for (int i = 0; i < 2; ++i) pair_top(top[j], v[j][i]);
  for (int k = ka + lane * 8 + 512; k < kb; k += 256)
#pragma unroll
    for (int j = 0; j < TN; ++j) pair_top(top[j], get(j, k));
  uint32_t up[TN];
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    float most = warp_max(top_of(top[j]));
    if (most == INFINITY) {   // an infinity among them: the largest finite one (uniform, rare)
      most = 0.f;
      for (int k = ka + lane * 8; k < kb; k += 256) most = fmaxf(most, finite_top8(get(j, k)));
      most = warp_max(most);
    }
    float f, dn;
    f16_scale(most, f, dn);
    up[j] = splat_bf16(f);
    if (lane == 0 && j < cnt) down[n0 + j] = dn;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int k = ka + lane * 8 + i * 256;
      if (j < cnt && k < kb) dst[x_unit(k - k0, n0 + j, tok)] = to_f16(v[j][i], up[j]);
    }
  for (int k = ka + lane * 8 + 512; k < kb; k += 256)
#pragma unroll
    for (int j = 0; j < TN; ++j)
      if (j < cnt) dst[x_unit(k - k0, n0 + j, tok)] = to_f16(get(j, k), up[j]);
}

__device__ __forceinline__ void store_out(const LinearArgs& a, int t, int row, float v) {
  const size_t at = (size_t)t * a.N + row;
  if (a.out_f32) static_cast<float*>(a.out)[at] = v;
  else static_cast<uint16_t*>(a.out)[at] = (uint16_t)(pack_bf16(v, 0.f) & 0xFFFFu);
}

// Up to 8 tokens: tiles of 16 MT rows, AHEAD pieces in flight per warp.
template <int MT, int AHEAD>
__global__ void __launch_bounds__(kLinWarps * 32, 2) k_linear_few(const LinearArgs a) {
  constexpr int W = kLinWarps, ROWS = 16 * MT;
  extern __shared__ __align__(128) unsigned char few_smem[];   // x [piece][j][token][q]
  __shared__ float down[W][8];
  __shared__ float sums[2][W][8][ROWS + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = lane & 3, r = lane >> 2;
  const int rank = a.split > 1 ? (int)cluster_rank() : 0;
  const int T = a.T;
  const int tiles = (a.N + ROWS - 1) / ROWS, step = gridDim.x / a.split;
  const int tile0 = blockIdx.x / a.split;
  // pieces of K: the block's [b0, b1), this warp's [p0, p0 + np), those past p1 are zeros
  const int pieces = (a.K + 127) >> 7;
  const int bp = (pieces + a.split - 1) / a.split;
  const int b0 = min(rank * bp, pieces), b1 = min(b0 + bp, pieces);
  const int np = (bp + W - 1) / W;
  const int p0 = min(b0 + warp * np, b1), p1 = min(p0 + np, b1);
  const int k0 = p0 * 128 + q * 32;
  const int mine = min(p1 - p0, (a.K - k0 + 127) >> 7);   // pieces in which this lane has elements
  griddep_launch_dependents();

  // the cursor of the loads, AHEAD pieces before that of the products
  Piece<MT> buf[AHEAD];
  Rows<MT> rows;
  int lt = tile0, lp = 0, limit = mine;
  rows.set(a, lt * ROWS, r, k0);
#pragma unroll
  for (int i = 0; i < AHEAD; ++i)
    if (i < mine && i < np) rows.prefetch(i);
  griddep_wait();
  const float g = *a.gscale;
  auto advance = [&](Piece<MT>& w) {
    rows.load(w, lp, lp < limit);
    if (++lp == np) {
      lp = 0;
      lt += step;
      if (lt < tiles) rows.set(a, lt * ROWS, r, k0);
      else limit = 0;
    }
  };
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) advance(buf[i]);

  // this warp's slice of x
  uint4* xs = reinterpret_cast<uint4*>(few_smem);
  if (T == 1) {
    stage_x<1>(a, 0, 0, T, p0 * 128, p1 * 128, b0 * 128, T, xs, down[warp]);
  } else {
    for (int n = 0; n < T; n += 2)
      stage_x<2>(a, 0, n, T, p0 * 128, p1 * 128, b0 * 128, T, xs, down[warp]);
  }
  __syncwarp();
  const float d0 = 2 * q < T ? down[warp][2 * q] : 0.f;
  const float d1 = 2 * q + 1 < T ? down[warp][2 * q + 1] : 0.f;
  // columns past T repeat the last token's (nobody reads them)
  const uint4* const xw = xs + (size_t)(p0 - b0) * (T * 16) + min(r, T - 1) * 4 + q;

  float acc[MT][1][4];
#pragma unroll
  for (int m = 0; m < MT; ++m) acc[m][0][0] = acc[m][0][1] = acc[m][0][2] = acc[m][0][3] = 0.f;
  int p = 0, flip = 0;
  for (int tile = tile0; tile < tiles;) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (tile >= tiles) break;   // uniform over the block
      if (p0 + p < p1) products<MT, 1>(acc, buf[i], xw + p * (T * 16), T * 4);
      advance(buf[i]);
      if (++p < np) continue;
      // the tile's end: lane has rows r + 8 i of tokens 2 q, 2 q + 1
      float (*part)[8][ROWS + 1] = sums[flip];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        part[warp][2 * q][16 * m + r] = acc[m][0][0] * d0;
        part[warp][2 * q + 1][16 * m + r] = acc[m][0][1] * d1;
        part[warp][2 * q][16 * m + r + 8] = acc[m][0][2] * d0;
        part[warp][2 * q + 1][16 * m + r + 8] = acc[m][0][3] * d1;
        acc[m][0][0] = acc[m][0][1] = acc[m][0][2] = acc[m][0][3] = 0.f;
      }
      p = 0;
      __syncthreads();   // one per tile: the other copy of sums is free again after the next one
      const int x = threadIdx.x, t = x / ROWS, row = tile * ROWS + x % ROWS;
      float v = 0.f;
      if (t < T) {
#pragma unroll
        for (int s = 0; s < W; ++s) v += part[s][t][x % ROWS];
      }
      if (a.split > 1) {
        __syncthreads();
        if (t < T) part[0][t][x % ROWS] = v;
        cluster_sync();
        // the tile's outputs go round the cluster's blocks
        if (t < T && x % a.split == rank) {
          v = 0.f;
          for (int s = 0; s < a.split; ++s) v += ld_cluster(smem_addr(&part[0][t][x % ROWS]), s);
          if (row < a.N) store_out(a, t, row, v * g);
        }
        cluster_sync();   // no block goes on (or leaves) while its sums are read
      } else if (t < T && row < a.N) {
        store_out(a, t, row, v * g);
      }
      flip ^= 1;
      tile += step;
    }
  }
}

// ---------------------------------------------------------------- 9 to 64 tokens, few rows
// One launch: tiles of 128 rows (four groups of 32 rows x two slices of K in a block), K over a cluster
// of S blocks, each of which lays its own slice of x out. Up to 8 NT tokens per grid row.
constexpr int kMidRows = 128;
template <int NT>
__global__ void __launch_bounds__(kLinWarps * 32, NT <= 4 ? 2 : 1) k_linear_mid(const LinearArgs a) {
  constexpr int WK = 2, TOK = NT * 8, ROWS = kMidRows, AHEAD = 2;
  extern __shared__ __align__(128) unsigned char mid_smem[];   // x, then sums [token][row]
  __shared__ float down[WK][TOK];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wm = warp >> 1, wk = warp & 1;
  const int q = lane & 3, r = lane >> 2;
  const int rank = a.split > 1 ? (int)cluster_rank() : 0;
  const int t0 = blockIdx.y * TOK, T = min(a.T - t0, TOK);
  const int tile = blockIdx.x / a.split;
  const int pieces = (a.K + 127) >> 7;
  const int bp = (pieces + a.split - 1) / a.split;
  const int b0 = min(rank * bp, pieces), b1 = min(b0 + bp, pieces);
  const int np = (bp + WK - 1) / WK;
  const int p0 = min(b0 + wk * np, b1), p1 = min(p0 + np, b1);
  const int k0 = p0 * 128 + q * 32;
  const int mine = min(p1 - p0, (a.K - k0 + 127) >> 7);
  griddep_launch_dependents();
  Rows<2> rows;
  rows.set(a, tile * ROWS + wm * 32, r, k0);
#pragma unroll
  for (int i = 0; i < AHEAD; ++i)
    if (i < mine) rows.prefetch(i);
  griddep_wait();
  Piece<2> buf[AHEAD];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) rows.load(buf[i], i, i < mine);
  const float g = *a.gscale;
  uint4* xs = reinterpret_cast<uint4*>(mid_smem);
  // (four tokens, slice) pairs go round the warps
  for (int job = warp; job < (T + 3) / 4 * WK; job += kLinWarps) {
    const int s = job & 1, n = (job >> 1) * 4;
    const int c0 = min(b0 + s * np, b1), c1 = min(c0 + np, b1);
    stage_x<4>(a, t0, n, T, c0 * 128, c1 * 128, b0 * 128, TOK, xs, down[s]);
  }
  __syncthreads();
  float acc[2][NT][4];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n][0] = acc[m][n][1] = acc[m][n][2] = acc[m][n][3] = 0.f;
  const uint4* xw = xs + (size_t)(p0 - b0) * (TOK * 16) + lane;
  for (int p = 0; p < p1 - p0; p += AHEAD) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (p + i >= p1 - p0) break;   // uniform over the warp
      products<2, NT>(acc, buf[i], xw + (p + i) * (TOK * 16), TOK * 4);
      rows.load(buf[i], p + i + AHEAD, p + i + AHEAD < mine);
    }
  }
  // the block's sums [token][row]: the second slice adds to the first
  constexpr int LD = ROWS + 4;
  float* sums = reinterpret_cast<float*>(mid_smem);
  __syncthreads();
#pragma unroll
  for (int s = 0; s < WK; ++s) {
    if (wk == s) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int t = n * 8 + 2 * q + e;
          const float d = t < T ? down[wk][t] : 0.f;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            float* at = sums + t * LD + wm * 32 + 8 * x + r;
            const float v = acc[x >> 1][n][(x & 1) * 2 + e] * d;
            *at = s == 0 ? v : *at + v;
          }
        }
    }
    __syncthreads();
  }
  // the cluster's sums, four rows at a time: the tokens' rows go round the blocks
  if (a.split > 1) cluster_sync();
  const int items = T * (ROWS / 4);
  for (int x = rank * kLinWarps * 32 + threadIdx.x; x < items; x += a.split * kLinWarps * 32) {
    const int t = x / (ROWS / 4), in = x % (ROWS / 4) * 4, row = tile * ROWS + in;
    const uint32_t at = smem_addr(sums + t * LD + in);
    float4 v[8];
#pragma unroll
    for (int s = 0; s < 8; ++s)   // all in flight, added in order
      v[s] = s < a.split ? ld_cluster4(at, s) : make_float4(0.f, 0.f, 0.f, 0.f);
    float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      y[0] += v[s].x; y[1] += v[s].y; y[2] += v[s].z; y[3] += v[s].w;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (row + j < a.N) store_out(a, t0 + t, row + j, y[j] * g);
  }
  if (a.split > 1) cluster_sync();   // no block leaves while its sums are read
}

// ---------------------------------------------------------------- 9 to 64 tokens, many rows
constexpr int kMoreRows = 32 * kLinWarps;   // rows of a tile
constexpr int kMoreStages = 4;              // units of x in shared memory

// x in f16 with a power of two per token, in the B operand's order (x_unit) `width` tokens wide. A
// block per token; the tokens past T stay unwritten (they only reach sums that nobody reads), elements
// past K are zeros.
constexpr int kPrepThreads = 256;
constexpr int kPrepKeep = 4;   // 8-element pieces a thread keeps between the two passes
__global__ void __launch_bounds__(kPrepThreads) k_linear_x(const LinearArgs a, int width) {
  __shared__ float red[kPrepThreads / 32];
  griddep_launch_dependents();
  griddep_wait();
  const int t = blockIdx.x, lane = threadIdx.x & 31;
  const uint16_t* x = a.x + (size_t)t * a.x_stride;
  const int Kp = (a.K + kLinUnit - 1) / kLinUnit * kLinUnit;
  auto get = [&](int k) {
    return k < a.K ? *reinterpret_cast<const uint4*>(x + k) : make_uint4(0, 0, 0, 0);
  };
  uint4 v[kPrepKeep];
#pragma unroll
  for (int i = 0; i < kPrepKeep; ++i) v[i] = get((i * kPrepThreads + (int)threadIdx.x) * 8);
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < kPrepKeep; ++i) top = fmaxf(top, finite_top8(v[i]));
  for (int k = (kPrepKeep * kPrepThreads + (int)threadIdx.x) * 8; k < a.K; k += kPrepThreads * 8)
    top = fmaxf(top, finite_top8(get(k)));
  top = warp_max(top);
  if (lane == 0) red[threadIdx.x >> 5] = top;
  __syncthreads();
  top = warp_max(lane < kPrepThreads / 32 ? red[lane] : 0.f);
  float factor, down;
  f16_scale(top, factor, down);
  const uint32_t up = splat_bf16(factor);
  if (threadIdx.x == 0) a.xdown[t] = down;
  uint4* xh = reinterpret_cast<uint4*>(a.xh);
#pragma unroll
  for (int i = 0; i < kPrepKeep; ++i) {
    const int k = (i * kPrepThreads + (int)threadIdx.x) * 8;
    if (k < Kp) xh[x_unit(k, t, width)] = to_f16(v[i], up);
  }
  for (int k = (kPrepKeep * kPrepThreads + (int)threadIdx.x) * 8; k < Kp; k += kPrepThreads * 8)
    xh[x_unit(k, t, width)] = to_f16(get(k), up);
}

template <int NT>
__global__ void __launch_bounds__(kLinWarps * 32, NT <= 4 ? 2 : 1)
    k_linear_more(const LinearArgs a, int uk, int quota) {
  constexpr int TOK = NT * 8, ST = kMoreStages, AHEAD = 2, PU = kLinUnit / 128;
  constexpr uint32_t kX = TOK * kLinUnit * 2;   // bytes of a unit of x
  extern __shared__ __align__(128) unsigned char more_smem[];   // x [stage][unit]
  __shared__ __align__(8) uint64_t full[ST], empty[ST];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = lane & 3, r = lane >> 2;
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kLinWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  griddep_launch_dependents();
  griddep_wait();
  const int total = ((a.N + kMoreRows - 1) / kMoreRows) * uk;
  const int u0 = min((int)blockIdx.x * quota, total), u1 = min(u0 + quota, total);
  const float g = *a.gscale;

  auto send = [&](int i) {   // x of unit u0 + i (one thread)
    const int st = i % ST;
    asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}" ::
                     "r"(smem_addr(&full[st])), "r"(kX) : "memory");
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes "
                 "[%0], [%1], %2, [%3];" ::"r"(smem_addr(more_smem) + st * kX),
                 "l"(reinterpret_cast<const char*>(a.xh) + (size_t)((u0 + i) % uk) * kX), "r"(kX),
                 "r"(smem_addr(&full[st])) : "memory");
  };
  int sent = 0;   // units of x (one thread)
  if (threadIdx.x == 0)
    for (; sent < ST && u0 + sent < u1; ++sent) send(sent);

  // the cursor of the loads: units from u0 on, PU pieces each
  Piece<2> buf[AHEAD];
  Rows<2> rows;
  int lu = u0, lp = 0, limit = 0;
  auto enter = [&]() {   // the rows and this lane's pieces of unit lu
    limit = 0;
    if (lu < u1) {
      const int tile = lu / uk, k0 = (lu - tile * uk) * kLinUnit + q * 32;
      rows.set(a, tile * kMoreRows + warp * 32, r, k0);
      limit = min(PU, (a.K - k0 + 127) >> 7);
    }
  };
  auto advance = [&](Piece<2>& w) {
    rows.load(w, lp, lp < limit);
    if (++lp == PU) {
      lp = 0;
      ++lu;
      enter();
    }
  };
  enter();
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) advance(buf[i]);

  float acc[2][NT][4];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n][0] = acc[m][n][1] = acc[m][n][2] = acc[m][n][3] = 0.f;
  for (int u = u0; u < u1; ++u) {
    const int i = u - u0, st = i % ST;
    if (!mbar_wait(&full[st], (uint32_t)(i / ST) & 1u, a.err, kErrTimeout, a.wait_rounds)) {
      // flagged, the results are undefined; the block leaves once its copies have landed
      if (threadIdx.x == 0)
        for (int j = sent > ST ? sent - ST : 0; j < sent; ++j)
          mbar_wait(&full[j % ST], (uint32_t)(j / ST) & 1u, nullptr, 0);
      break;
    }
    __syncwarp();
    const uint4* xu = reinterpret_cast<const uint4*>(more_smem + st * kX) + lane;
#pragma unroll
    for (int p = 0; p < PU; ++p) {
      products<2, NT>(acc, buf[p % AHEAD], xu + p * (TOK * 16), TOK * 4);
      advance(buf[p % AHEAD]);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[st]);
    // the stage before this one again, once every warp has read it
    if (threadIdx.x == 0 && i > 0 && sent == i - 1 + ST && u0 + sent < u1 &&
        mbar_wait(&empty[(i - 1) % ST], (uint32_t)((i - 1) / ST) & 1u, a.err, kErrTimeout, a.wait_rounds))
      send(sent++);
    const int tile = u / uk;
    if (u + 1 < u1 && (u + 1) % uk != 0) continue;
    // the end of the tile or of the run: lane has rows r + 8 i of tokens 8 n + 2 q, + 1
    const bool whole = (u + 1) % uk == 0 && u - uk + 1 >= u0;
    float* part = a.part + (size_t)(2 * blockIdx.x + (tile * uk <= u0 ? 0 : 1)) * TOK * kMoreRows;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int t = n * 8 + 2 * q + e;
        if (t < a.T) {
          const float d = whole ? a.xdown[t] * g : 1.f;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int in = warp * 32 + 8 * x + r, row = tile * kMoreRows + in;
            const float v = acc[x >> 1][n][(x & 1) * 2 + e] * d;
            if (!whole) part[(size_t)t * kMoreRows + in] = v;
            else if (row < a.N) store_out(a, t, row, v);
          }
        }
      }
#pragma unroll
      for (int m = 0; m < 2; ++m) acc[m][n][0] = acc[m][n][1] = acc[m][n][2] = acc[m][n][3] = 0.f;
    }
  }
}

// Tiles that several runs share: their sums in order, four rows of a token per thread. Grid (tile, 4
// tokens).
__global__ void __launch_bounds__(kMoreRows) k_linear_join(const LinearArgs a, int width, int uk,
                                                           int quota) {
  griddep_launch_dependents();
  griddep_wait();
  const int tile = blockIdx.x, t = blockIdx.y * 4 + (threadIdx.x >> 6), in = (threadIdx.x & 63) * 4;
  const int s0 = tile * uk, s1 = s0 + uk;
  const int first = s0 / quota, last = (s1 - 1) / quota;
  const int row = tile * kMoreRows + in;
  if (first == last || t >= a.T || row >= a.N) return;
  const float d = a.xdown[t] * *a.gscale;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int b = first; b <= last; ++b) {
    const float4 u = *reinterpret_cast<const float4*>(
        a.part + ((size_t)(2 * b + (b * quota >= s0 ? 0 : 1)) * width + t) * kMoreRows + in);
    v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
  }
  const float y[4] = {v.x * d, v.y * d, v.z * d, v.w * d};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (row + j < a.N) store_out(a, t, row + j, y[j]);
}

template <typename K, typename... Args>
cudaError_t start(K kernel, dim3 grid, int threads, size_t smem, int cluster, cudaStream_t stream,
                  Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int MT, int AHEAD>
cudaError_t launch_few(LinearArgs a, int num_sms, cudaStream_t stream) {
  const int tiles = (a.N + 16 * MT - 1) / (16 * MT), pieces = (a.K + 127) / 128;
  auto x_bytes = [&](int split) { return (size_t)((pieces + split - 1) / split) * 256 * a.T; };
  // K is split over a cluster while x does not fit, or while there are fewer blocks than SMs and
  // every warp keeps a piece
  int split = 1;
  while (split < 8 && (x_bytes(split) > kLinXMax ||
                       (tiles * split < num_sms && pieces >= 2 * split * kLinWarps)))
    split *= 2;
  a.split = split;
  // resident blocks: two an SM, one when x takes more than half of the shared memory
  const int most = (x_bytes(split) > kLinXMax / 2 ? 1 : 2) * num_sms / split;
  const int blocks = tiles < most ? tiles : most;
  static SmemGrant grant;
  const cudaError_t e = grant_smem(grant, k_linear_few<MT, AHEAD>, (int)kLinXMax);
  if (e != cudaSuccess) return e;
  return start(k_linear_few<MT, AHEAD>, dim3((unsigned)(blocks * split)), kLinWarps * 32, x_bytes(split),
               split, stream, a);
}

template <int NT>
cudaError_t launch_mid(LinearArgs a, int num_sms, cudaStream_t stream) {
  constexpr int TOK = NT * 8;
  const int tiles = (a.N + kMidRows - 1) / kMidRows, pieces = (a.K + 127) / 128;
  const int groups = (a.T + TOK - 1) / TOK;
  auto x_bytes = [&](int split) { return (size_t)((pieces + split - 1) / split) * 256 * TOK; };
  // K over a cluster while twice the blocks are at most two an SM and every warp keeps a piece, and
  // while x does not fit. This counts blocks, not rounds: 256 blocks (32 tokens of 4096 x 4096) leave 104 SMs
  // with two of them and 48 with one, and clusters of eight take two rounds from 34 row tiles on (11 x 4718 x
  // 4096 12.5 us, 9.3 with clusters of four).
  int split = 1;
  while (split < 8 && (x_bytes(split) > kLinXMax / 2 ||
                       (tiles * groups * split <= num_sms && pieces >= 4 * split)))
    split *= 2;
  a.split = split;
  const size_t sums = (size_t)TOK * (kMidRows + 4) * 4;
  const size_t smem = x_bytes(split) > sums ? x_bytes(split) : sums;
  static SmemGrant grant;
  const cudaError_t e = grant_smem(grant, k_linear_mid<NT>, (int)kLinXMax);
  if (e != cudaSuccess) return e;
  return start(k_linear_mid<NT>, dim3((unsigned)(tiles * split), (unsigned)groups),
               kLinWarps * 32, smem, split, stream, a);
}

template <int NT>
cudaError_t launch_more(LinearArgs a, int num_sms, cudaStream_t stream) {
  a.wait_rounds = wait_limit(kWaitRounds);
  constexpr int TOK = NT * 8;
  const int uk = (a.K + kLinUnit - 1) / kLinUnit;
  const int tiles = (a.N + kMoreRows - 1) / kMoreRows, total = tiles * uk;
  const int most = (NT <= 4 ? 2 : 1) * num_sms;   // resident blocks
  const int quota = (total + most - 1) / most;
  const int blocks = (total + quota - 1) / quota;
  static SmemGrant grant;
  constexpr size_t smem = (size_t)kMoreStages * TOK * kLinUnit * 2;
  cudaError_t e = grant_smem(grant, k_linear_more<NT>, (int)smem);
  if (e != cudaSuccess) return e;
  e = start(k_linear_x, dim3((unsigned)a.T), kPrepThreads, 0, 1, stream, a, TOK);
  if (e != cudaSuccess) return e;
  e = start(k_linear_more<NT>, dim3((unsigned)blocks), kLinWarps * 32,
            smem, 1, stream, a, uk, quota);
  if (e != cudaSuccess || quota % uk == 0) return e;   // every run ends with a tile
  return start(k_linear_join, dim3((unsigned)tiles, (unsigned)((a.T + 3) / 4)), kMoreRows, 0, 1, stream,
               a, TOK, uk, quota);
}

}  // namespace

cudaError_t launch_linear(const LinearArgs& a, int num_sms, cudaStream_t stream) {
  // Up to 8 tokens: 32-row tiles once 16-row ones take more than one round of the resident blocks (us, one
  // token, K = 4096, 16- or 32-row tiles: 4.6 or 5.6 at 4096 rows, 6.2 or 6.3 at 5120, 6.8 or 6.4 at 6144,
  // 46 or 41 at 100003). 32 tokens, one launch or three: 12.3 or 14.5 at 4096 rows, 37 or 29 at 20000.
  const bool wide = a.N >= 64 * num_sms;
  if (a.T <= kLinearFew)
    return a.N > 32 * num_sms ? launch_few<2, 2>(a, num_sms, stream) : launch_few<1, 2>(a, num_sms, stream);
  const int nt = (a.T + 7) / 8;
  // Groups of 16 tokens on blocks of their own read the matrix again, from L2, but where SMs are idle
  // otherwise that pays (us, one group or groups of 16): 32 tokens 8.7 or 6.4 at 2048 x 2048, 11.6 or 10.9 at
  // 4096 x 4096, 30 or 33 at 8000 x 8192; 64 tokens, three launches or groups of 16: 10.8 or 7.6 at
  // 2048 x 2048, 15.6 or 10.7 at 2048 x 4096.
  const int tiles = (a.N + kMidRows - 1) / kMidRows;
  if (!wide && (nt <= 2 || tiles * ((nt + 1) / 2) * 2 <= num_sms || (nt <= 4 && a.K > 16384)))
    return launch_mid<2>(a, num_sms, stream);
  if (!wide && nt <= 4) return launch_mid<4>(a, num_sms, stream);
  if (nt <= 2) return launch_more<2>(a, num_sms, stream);
  if (nt <= 4) return launch_more<4>(a, num_sms, stream);
  if (nt <= 6) return launch_more<6>(a, num_sms, stream);
  return launch_more<8>(a, num_sms, stream);
}

}  // namespace ftmoe
