// The norm after a block, its gated residual sum and the norm before the next block, in one pass,
// and the gradient.
//
//   z  = y * s1 * w_post,  s1 = 1 / sqrt(mean(y^2) + eps)      (w_post absent: z = y)
//   r' = r + scale * gate * z                                  (r absent: 0; gate absent: 1)
//   x' = r' * s2 * w_pre,  s2 = 1 / sqrt(mean(r'^2) + eps)     (w_pre absent: no x')
//
// Gradient, with dr and dx those of r' and x' and means over the row:
//   d = dx w_pre            dr' = dr + s2 (d - r' s2^2 mean(d r'))     dresidual = dr'
//   dw_pre = sum_t dx r' s2 dz  = scale gate dr'                       dgate = scale z dr'
//   h = dz w_post           dy  = s1 (h - y s1^2 mean(h y))            dw_post = sum_t dz y s1
//
// A row stays in the registers of one block (or of one warp, for short rows): each input is read
// once and each output written once. Sums run in float32 in a fixed order; x' is taken from r'
// before r' is rounded to its stored type.
#include <cuda_runtime.h>

#include "ftmoe_internal.h"
#include "ftmoe_mma.cuh"

namespace ftmoe {

namespace {

constexpr int kWarpRowMax = 512;    // elements of a row that one warp holds
constexpr int kRowWarps = 8;        // rows (warps) per block in that form

// Sum over the row's threads: the warp, or the whole block through red[] (one array per call
// site, so that one barrier per sum is enough).
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = warp_sum(v);
  if constexpr (WARP) return v;
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum(lane < warps ? red[lane] : 0.f);
}

__device__ __forceinline__ void cached8(const uint16_t* p, float (&f)[8]) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = bf16_lo(w[j]);
    f[2 * j + 1] = bf16_hi(w[j]);
  }
}

__device__ __forceinline__ float one_bf16(const uint16_t* p) {
  return __uint_as_float((uint32_t)*p << 16);
}

template <int NV, typename RT, bool WARP>
__global__ void __launch_bounds__(WARP ? kRowWarps * 32 : 1024) k_norm(const NormArgs a) {
  __shared__ float red[2][32];
  griddep_launch_dependents();
  griddep_wait();
  const int tid = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int nth = WARP ? 32 : blockDim.x;
  const int t = WARP ? blockIdx.x * kRowWarps + (threadIdx.x >> 5) : blockIdx.x;
  if (t >= a.T) return;   // a whole warp or block
  const size_t row = (size_t)t * a.H;
  const int chunks = a.H >> 3;
  const float inv_h = 1.0f / (float)a.H;

  float y[NV][8], r[NV][8];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = tid + i * nth;
    if (c < chunks) {
      load8(a.y + row + 8 * c, y[i]);
      if (a.r) load8(static_cast<const RT*>(a.r) + row + 8 * c, r[i]);
    }
    if (c >= chunks || !a.r) {
#pragma unroll
      for (int j = 0; j < 8; ++j) r[i][j] = 0.f;
    }
    if (c >= chunks) {
#pragma unroll
      for (int j = 0; j < 8; ++j) y[i][j] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(y[i][j], y[i][j], ss);
  }
  float s1 = 1.f;
  if (a.w_post) s1 = rsqrtf(row_sum<WARP>(ss, red[0]) * inv_h + a.eps);
  const float tg = a.scale * (a.gate_kind == FT_GATE_TOKEN ? one_bf16(a.gate + t) : 1.f);
  ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = tid + i * nth;
    if (c >= chunks) continue;
    float w[8], g[8];
    if (a.w_post) {
      cached8(a.w_post + 8 * c, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[i][j] *= s1 * w[j];
    }
    if (a.gate_kind == FT_GATE_CHANNEL || a.gate_kind == FT_GATE_ELEMENT) {
      if (a.gate_kind == FT_GATE_CHANNEL) cached8(a.gate + 8 * c, g);
      else load8(a.gate + row + 8 * c, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[i][j] *= g[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      r[i][j] = fmaf(tg, y[i][j], r[i][j]);
      ss = fmaf(r[i][j], r[i][j], ss);
    }
    if (a.r_out) store8(static_cast<RT*>(a.r_out) + row + 8 * c, r[i]);
  }
  if (!a.w_pre) return;
  const float s2 = rsqrtf(row_sum<WARP>(ss, red[1]) * inv_h + a.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = tid + i * nth;
    if (c >= chunks) continue;
    float w[8];
    cached8(a.w_pre + 8 * c, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) r[i][j] *= s2 * w[j];
    store8(a.x_out + row + 8 * c, r[i]);
  }
}

template <int NV, typename RT, bool WARP>
__global__ void __launch_bounds__(WARP ? kRowWarps * 32 : 1024) k_norm_bwd(const NormArgs a) {
  __shared__ float red[4][32];
  griddep_launch_dependents();
  griddep_wait();
  const int tid = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int nth = WARP ? 32 : blockDim.x;
  const int group = WARP ? blockIdx.x * kRowWarps + (threadIdx.x >> 5) : blockIdx.x;
  const int groups = WARP ? gridDim.x * kRowWarps : gridDim.x;
  const int chunks = a.H >> 3;
  const float inv_h = 1.0f / (float)a.H;
  const bool channel = a.gate_kind == FT_GATE_CHANNEL;

  float acc_post[NV][8], acc_pre[NV][8], acc_gate[NV][8];   // this group's column sums
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc_post[i][j] = acc_pre[i][j] = acc_gate[i][j] = 0.f;

  for (int t = group; t < a.T; t += groups) {
    const size_t row = (size_t)t * a.H;
    float y[NV][8], r[NV][8], dr[NV][8], dx[NV][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tid + i * nth;
#pragma unroll
      for (int j = 0; j < 8; ++j) y[i][j] = r[i][j] = dr[i][j] = dx[i][j] = 0.f;
      if (c < chunks) {
        load8(a.y + row + 8 * c, y[i]);
        if (a.r) load8(static_cast<const RT*>(a.r) + row + 8 * c, r[i]);
        if (a.dr) load8(static_cast<const RT*>(a.dr) + row + 8 * c, dr[i]);
        if (a.w_pre) load8(a.dx + row + 8 * c, dx[i]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(y[i][j], y[i][j], ss);
    }
    float s1 = 1.f;
    if (a.w_post) s1 = rsqrtf(row_sum<WARP>(ss, red[0]) * inv_h + a.eps);
    const float tg = a.scale * (a.gate_kind == FT_GATE_TOKEN ? one_bf16(a.gate + t) : 1.f);
    // r <- r'
    float rr = 0.f, dot = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tid + i * nth;
      if (c >= chunks) continue;
      float w[8], g[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = g[j] = 1.f;
      if (a.w_post) cached8(a.w_post + 8 * c, w);
      if (channel) cached8(a.gate + 8 * c, g);
      else if (a.gate_kind == FT_GATE_ELEMENT) cached8(a.gate + row + 8 * c, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) r[i][j] = fmaf(tg * g[j], y[i][j] * (s1 * w[j]), r[i][j]);
      if (a.w_pre) {
        cached8(a.w_pre + 8 * c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          rr = fmaf(r[i][j], r[i][j], rr);
          dot = fmaf(dx[i][j] * w[j], r[i][j], dot);
        }
      }
    }
    float s2 = 0.f, cr = 0.f;
    if (a.w_pre) {
      rr = row_sum<WARP>(rr, red[1]);
      dot = row_sum<WARP>(dot, red[2]);
      s2 = rsqrtf(rr * inv_h + a.eps);
      cr = s2 * s2 * (dot * inv_h);
    }
    float hy = 0.f, dgt = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tid + i * nth;
      if (c >= chunks) continue;
      float w[8], g[8], dg[8];
      if (a.w_pre) {
        cached8(a.w_pre + 8 * c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          acc_pre[i][j] = fmaf(dx[i][j], r[i][j] * s2, acc_pre[i][j]);
          dr[i][j] = fmaf(s2, dx[i][j] * w[j] - r[i][j] * cr, dr[i][j]);
        }
      }
      store8(static_cast<RT*>(a.dres) + row + 8 * c, dr[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = g[j] = 1.f;
      if (a.w_post) cached8(a.w_post + 8 * c, w);
      if (channel) cached8(a.gate + 8 * c, g);
      else if (a.gate_kind == FT_GATE_ELEMENT) cached8(a.gate + row + 8 * c, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float yn = y[i][j] * s1;
        dg[j] = a.scale * (yn * w[j]) * dr[i][j];
        const float dz = tg * g[j] * dr[i][j];
        if (channel) acc_gate[i][j] += dg[j];
        dgt += dg[j];
        if (a.w_post) {
          acc_post[i][j] = fmaf(dz, yn, acc_post[i][j]);
          hy = fmaf(dz * w[j], y[i][j], hy);
        }
        dx[i][j] = dz * w[j];   // h, or dy itself
      }
      if (a.gate_kind == FT_GATE_ELEMENT)
        store8(static_cast<uint16_t*>(a.dgate) + row + 8 * c, dg);
    }
    float cy = 0.f;
    if (a.w_post) cy = s1 * s1 * (row_sum<WARP>(hy, red[3]) * inv_h);
    if (a.gate_kind == FT_GATE_TOKEN) {
      __syncwarp();
      if constexpr (!WARP) __syncthreads();   // red[0] is free: every thread has passed red[3]
      dgt = row_sum<WARP>(dgt, red[0]);
      if (tid == 0) static_cast<float*>(a.dgate)[t] = dgt;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tid + i * nth;
      if (c >= chunks) continue;
      if (a.w_post) {
#pragma unroll
        for (int j = 0; j < 8; ++j) dx[i][j] = s1 * (dx[i][j] - y[i][j] * cy);
      }
      store8(a.dy + row + 8 * c, dx[i]);
    }
    if constexpr (!WARP) __syncthreads();   // before the next row writes red[]
  }

  // the group's column sums: [block][quantity][H]
  float* part = a.part + (size_t)blockIdx.x * a.nq * a.H;
  if constexpr (!WARP) {
    int q = 0;
#pragma unroll
    for (int which = 0; which < 3; ++which) {
      if (which == 0 ? !a.w_post : which == 1 ? !a.w_pre : !channel) continue;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = tid + i * nth;
        if (c < chunks)
          store8(part + (size_t)q * a.H + 8 * c,
                 which == 0 ? acc_post[i] : which == 1 ? acc_pre[i] : acc_gate[i]);
      }
      ++q;
    }
  } else {
    __shared__ float cols[kRowWarps][kWarpRowMax];
    int q = 0;
#pragma unroll
    for (int which = 0; which < 3; ++which) {
      if (which == 0 ? !a.w_post : which == 1 ? !a.w_pre : !channel) continue;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = tid + i * nth;
        if (c < chunks)
          store8(&cols[threadIdx.x >> 5][8 * c],
                 which == 0 ? acc_post[i] : which == 1 ? acc_pre[i] : acc_gate[i]);
      }
      __syncthreads();
      for (int h = threadIdx.x; h < a.H; h += kRowWarps * 32) {
        float v = 0.f;
        for (int w = 0; w < kRowWarps; ++w) v += cols[w][h];
        part[(size_t)q * a.H + h] = v;
      }
      ++q;
    }
  }
}

// The blocks' column sums in a fixed order: a block sums 128 columns (four per lane), its warps
// take the partial rows in turn.
constexpr int kColWarps = 16;
__global__ void __launch_bounds__(kColWarps * 32) k_norm_cols(const NormArgs a, int parts) {
  __shared__ float4 sum[kColWarps][32];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = (blockIdx.x * 32 + lane) * 4;   // over nq * H columns, H a multiple of 8
  const int width = a.nq * a.H;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (col < width) {
#pragma unroll 4
    for (int p = warp; p < parts; p += kColWarps) {
      const float4 u = *reinterpret_cast<const float4*>(a.part + (size_t)p * width + col);
      v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
    }
  }
  sum[warp][lane] = v;
  __syncthreads();
  if (warp != 0 || col >= width) return;
  for (int w = 1; w < kColWarps; ++w) {
    const float4 u = sum[w][lane];
    v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
  }
  int q = col / a.H;
  const int h = col - q * a.H;
  float* const to[3] = {a.dw_post, a.dw_pre,
                        a.gate_kind == FT_GATE_CHANNEL ? static_cast<float*>(a.dgate) : nullptr};
  const bool on[3] = {a.w_post != nullptr, a.w_pre != nullptr, a.gate_kind == FT_GATE_CHANNEL};
  for (int which = 0; which < 3; ++which) {
    if (!on[which]) continue;
    if (q-- == 0) *reinterpret_cast<float4*>(to[which] + h) = v;
  }
}

template <typename K>
cudaError_t launch(K kernel, int grid, int threads, cudaStream_t stream, const NormArgs& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

// Threads of a block that holds rows of `chunks` 8-element pieces, nv per thread.
int row_threads(int chunks, int nv) { return ((chunks + nv - 1) / nv + 31) / 32 * 32; }

}  // namespace

int norm_bwd_groups(int T, int H, int num_sms) {
  const int rows = H <= kWarpRowMax ? (T + kRowWarps - 1) / kRowWarps : T;
  const int most = 2 * num_sms;
  return rows < most ? rows : most;
}

cudaError_t launch_norm(const NormArgs& a, cudaStream_t stream) {
  const int chunks = a.H / 8;
  if (a.H <= kWarpRowMax) {
    const int grid = (a.T + kRowWarps - 1) / kRowWarps;
    return a.res_f32 ? launch(k_norm<2, float, true>, grid, kRowWarps * 32, stream, a)
                     : launch(k_norm<2, uint16_t, true>, grid, kRowWarps * 32, stream, a);
  }
  const int th = row_threads(chunks, 2);
  return a.res_f32 ? launch(k_norm<2, float, false>, a.T, th, stream, a)
                   : launch(k_norm<2, uint16_t, false>, a.T, th, stream, a);
}

cudaError_t launch_norm_bwd(const NormArgs& a, int num_sms, cudaStream_t stream) {
  const int chunks = a.H / 8;
  const int grid = norm_bwd_groups(a.T, a.H, num_sms);
  cudaError_t e;
  if (a.H <= kWarpRowMax) {
    e = a.res_f32 ? launch(k_norm_bwd<2, float, true>, grid, kRowWarps * 32, stream, a)
                  : launch(k_norm_bwd<2, uint16_t, true>, grid, kRowWarps * 32, stream, a);
  } else {
    const int th = row_threads(chunks, 2);
    e = a.res_f32 ? launch(k_norm_bwd<2, float, false>, grid, th, stream, a)
                  : launch(k_norm_bwd<2, uint16_t, false>, grid, th, stream, a);
  }
  if (e != cudaSuccess || a.nq == 0) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.nq * a.H + 127) / 128));
  cfg.blockDim = dim3(kColWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_norm_cols, a, grid);
}

}  // namespace ftmoe
