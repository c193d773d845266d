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
// The block's warps are WM groups of 16 rows times 8 / WM slices of K; a cluster of S blocks splits
// K further when there are fewer row groups than SMs or x does not fit. Partial sums are added in a
// fixed order (warps in shared memory, blocks through the cluster's shared memory).
#include <cmath>
#include <cuda_runtime.h>

#include "ftmoe_internal.h"
#include "ftmoe_mma.cuh"
#include "ftmoe_tc.cuh"

namespace ftmoe {

namespace {

constexpr int kLinWarps = 8;
constexpr int kLinAhead = 4;               // 128-element pieces whose loads are in flight per warp
constexpr size_t kLinXMax = 96 * 1024;     // x of one block in shared memory

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
__device__ __forceinline__ uint4 ld_once(const uint8_t* p) {   // weights: read once
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

struct Piece {   // 128 elements of 16 rows: this lane's 32 of two rows
  uint4 w0, w1;
  uint32_t s0, s1;
};

template <int NT, int WM>
__global__ void __launch_bounds__(kLinWarps * 32) k_linear(const LinearArgs a) {
  constexpr int WK = kLinWarps / WM;   // slices of K in the block
  constexpr int TOK = NT * 8;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float down[WK][TOK];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wm = warp / WK, wk = warp % WK;
  const int q = lane & 3, r = lane >> 2;
  const uint32_t rank = a.split > 1 ? cluster_rank() : 0;
  const int t0 = blockIdx.y * TOK;
  const int T = min(a.T - t0, TOK);
  const int row0 = (blockIdx.x / a.split) * (16 * WM) + wm * 16;

  // this warp's pieces of K: [p0, p1) of ceil(K / 128), the block's and the warp's share
  const int pieces = (a.K + 127) >> 7;
  const int bp = (pieces + a.split - 1) / a.split;
  const int bp0 = min((int)rank * bp, pieces), bp1 = min(bp0 + bp, pieces);
  const int wp = (bp + WK - 1) / WK;
  const int p0 = min(bp0 + wk * wp, bp1), p1 = min(p0 + wp, bp1);

  const int ra = min(row0 + r, a.N - 1), rb = min(row0 + r + 8, a.N - 1);
  const uint8_t* wa = a.codes + (size_t)ra * (a.K >> 1);
  const uint8_t* wb = a.codes + (size_t)rb * (a.K >> 1);
  const uint8_t* sa = a.scales + (size_t)ra * (a.K >> 4);
  const uint8_t* sb = a.scales + (size_t)rb * (a.K >> 4);
  auto load = [&](int p, Piece& w) {
    const int k = p * 128 + q * 32;
    if (p < p1 && k < a.K) {
      w.w0 = ld_once(wa + (k >> 1));
      w.w1 = ld_once(wb + (k >> 1));
      w.s0 = *reinterpret_cast<const uint16_t*>(sa + (k >> 4));
      w.s1 = *reinterpret_cast<const uint16_t*>(sb + (k >> 4));
    } else {
      w.w0 = w.w1 = make_uint4(0, 0, 0, 0);
      w.s0 = w.s1 = 0;
    }
  };
  Piece buf[kLinAhead];
#pragma unroll
  for (int i = 0; i < kLinAhead; ++i) load(p0 + i, buf[i]);

  // x of the block's K to shared memory as f16, in the B operand's order: 16-byte unit
  // ((piece * 4 + j) * TOK + token) * 4 + q = elements 32 q + 8 j .. + 7 of the piece
  uint4* xs = reinterpret_cast<uint4*>(smem);
  for (int job = warp; job < T * WK; job += kLinWarps) {   // (token, slice)
    // with one row group a warp stages its own slice only
    const int n = WM == 1 ? job / WK : job % T, s = WM == 1 ? warp : job / T;
    const int c0 = min(bp0 + s * wp, bp1), c1 = min(c0 + wp, bp1);
    const uint16_t* x = a.x + (size_t)(t0 + n) * a.x_stride;
    float top = 0.f;
    for (int k = c0 * 128 + lane * 8; k < c1 * 128; k += 256) {
      if (k < a.K) {
        const uint4 v = *reinterpret_cast<const uint4*>(x + k);
        top = fmaxf(top, fmaxf(finite_top(v.x, v.y), finite_top(v.z, v.w)));
      }
    }
    top = warp_max(top);
    float up, dn;
    f16_scale(top, up, dn);
    if (lane == 0) down[s][n] = dn;
    for (int k = c0 * 128 + lane * 8; k < c1 * 128; k += 256) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (k < a.K) v = *reinterpret_cast<const uint4*>(x + k);
      const uint4 h = make_uint4(pack_f16(bf16_lo(v.x) * up, bf16_hi(v.x) * up),
                                 pack_f16(bf16_lo(v.y) * up, bf16_hi(v.y) * up),
                                 pack_f16(bf16_lo(v.z) * up, bf16_hi(v.z) * up),
                                 pack_f16(bf16_lo(v.w) * up, bf16_hi(v.w) * up));
      const int k8 = (k >> 3) & 15;
      xs[(((k >> 7) - bp0) * 4 + (k8 & 3)) * (TOK * 4) + n * 4 + (k8 >> 2)] = h;
    }
  }
  if constexpr (WM == 1) __syncwarp();
  else __syncthreads();

  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
  for (int p = p0; p < p1; p += kLinAhead) {
#pragma unroll
    for (int i = 0; i < kLinAhead; ++i) {
      if (p + i >= p1) break;   // uniform over the warp
      const Piece w = buf[i];
      load(p + i + kLinAhead, buf[i]);
      uint32_t ca[16], cb[16];
      dequant32(w.w0, w.s0, ca);
      dequant32(w.w1, w.s1, cb);
      const uint4* xp = xs + (size_t)(p + i - bp0) * (TOK * 16);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          uint4 b = make_uint4(0, 0, 0, 0);
          if (n * 8 + r < T) b = xp[j * (TOK * 4) + n * 32 + lane];
          mma_f16(acc[n], ca[4 * j], cb[4 * j], ca[4 * j + 1], cb[4 * j + 1], b.x, b.y);
          mma_f16(acc[n], ca[4 * j + 2], cb[4 * j + 2], ca[4 * j + 3], cb[4 * j + 3], b.z, b.w);
        }
    }
  }
  // lane: rows r, r + 8, tokens 8 n + 2 q, + 1
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const float d0 = n * 8 + 2 * q < T ? down[wk][n * 8 + 2 * q] : 0.f;
    const float d1 = n * 8 + 2 * q + 1 < T ? down[wk][n * 8 + 2 * q + 1] : 0.f;
    acc[n][0] *= d0; acc[n][1] *= d1;
    acc[n][2] *= d0; acc[n][3] *= d1;
  }

  // add the slices: sums [slice][token][row] over x's memory
  constexpr int ROWS = 16 * WM;
  __syncthreads();
  float* sums = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int t = n * 8 + 2 * q, row = wm * 16 + r;
    float* at = sums + (size_t)(wk * TOK + t) * ROWS + row;
    at[0] = acc[n][0];
    at[ROWS] = acc[n][1];
    at[8] = acc[n][2];
    at[ROWS + 8] = acc[n][3];
  }
  __syncthreads();
  const float g = *a.gscale;
  if (a.split > 1) {
    // the block's own sum over its slices, then the cluster's, each block an equal part
    for (int x = threadIdx.x; x < T * ROWS; x += kLinWarps * 32) {
      float v = sums[x];
#pragma unroll
      for (int s = 1; s < WK; ++s) v += sums[s * TOK * ROWS + x];
      sums[x] = v;
    }
    cluster_sync();
    const int share = (T * ROWS + a.split - 1) / a.split;
    const int x0 = (int)rank * share, x1 = min(x0 + share, T * ROWS);
    for (int x = x0 + threadIdx.x; x < x1; x += kLinWarps * 32) {
      float v = 0.f;
      for (int s = 0; s < a.split; ++s) v += ld_cluster(smem_addr(sums + x), s);
      const int t = x / ROWS, row = (blockIdx.x / a.split) * ROWS + x % ROWS;
      if (row < a.N) {
        const size_t at = (size_t)(t0 + t) * a.N + row;
        if (a.out_f32) static_cast<float*>(a.out)[at] = v * g;
        else static_cast<uint16_t*>(a.out)[at] = (uint16_t)(pack_bf16(v * g, 0.f) & 0xFFFFu);
      }
    }
    cluster_sync();   // no block leaves while its sums are read
  } else {
    for (int x = threadIdx.x; x < T * ROWS; x += kLinWarps * 32) {
      float v = sums[x];
#pragma unroll
      for (int s = 1; s < WK; ++s) v += sums[s * TOK * ROWS + x];
      const int t = x / ROWS, row = blockIdx.x * ROWS + x % ROWS;
      if (row < a.N) {
        const size_t at = (size_t)(t0 + t) * a.N + row;
        if (a.out_f32) static_cast<float*>(a.out)[at] = v * g;
        else static_cast<uint16_t*>(a.out)[at] = (uint16_t)(pack_bf16(v * g, 0.f) & 0xFFFFu);
      }
    }
  }
}

template <int NT, int WM>
cudaError_t launch(LinearArgs a, int num_sms, cudaStream_t stream) {
  constexpr int ROWS = 16 * WM, TOK = NT * 8, WK = kLinWarps / WM;
  const int groups = (a.N + ROWS - 1) / ROWS, pieces = (a.K + 127) / 128;
  auto x_bytes = [&](int split) { return (size_t)((pieces + split - 1) / split) * 128 * TOK * 2; };
  // K is split over a cluster while x does not fit, or while there are fewer blocks than SMs and
  // every warp keeps at least two pieces
  int split = 1;
  while (split < 8 && (x_bytes(split) > kLinXMax ||
                       (groups * split < num_sms && pieces >= 2 * split * WK * 2)))
    split *= 2;
  a.split = split;
  const size_t sums = (size_t)WK * TOK * ROWS * 4;
  const size_t smem = x_bytes(split) > sums ? x_bytes(split) : sums;
  cudaError_t e;
  if ((e = cudaFuncSetAttribute(k_linear<NT, WM>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)smem)) != cudaSuccess)
    return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(groups * split), (unsigned)((a.T + TOK - 1) / TOK));
  cfg.blockDim = dim3(kLinWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)split;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k_linear<NT, WM>, a);
}

}  // namespace

cudaError_t launch_linear(const LinearArgs& a, int num_sms, cudaStream_t stream) {
  // K <= 32768 in eight blocks: 4096 elements of x for each of 8, 16 or (K <= 16384) 32 tokens is
  // at most 128 KB; more tokens than that are a second dimension of the grid
  if (a.T <= 8) return launch<1, 1>(a, num_sms, stream);
  if (a.T <= 16 || a.K > 16384) return launch<2, 4>(a, num_sms, stream);
  return launch<4, 4>(a, num_sms, stream);
}

}  // namespace ftmoe
