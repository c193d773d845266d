// The new tokens' keys and values into the paged cache, with the rotary embedding of q and k.
//
//   rotary   for i < R/2: (u_i, u_{i+R/2}) -> (u_i c_i - u_{i+R/2} s_i, u_{i+R/2} c_i + u_i s_i)
//            with c, s = rope[position][i], rope[position][R/2 + i]; elements past R unchanged
//   cache    page = block_table[seq][position / page_size], slot = position % page_size;
//            bf16, or E4M3 of the value times 1 / scale, saturated at +-448
//
// One thread takes two 8-element pieces of one head: a pair of pieces R/2 apart, which rotate into
// each other, or two neighbours past R. Products and sums are rounded one by one (no fused
// multiply-add), so that a value on the edge between two E4M3 codes falls as plain float32
// arithmetic lets it fall.
#include <cuda_runtime.h>

#include "ftmoe_internal.h"
#include "ftmoe_mma.cuh"

namespace ftmoe {

namespace {

constexpr int kAppendThreads = 256;

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

__device__ __forceinline__ void store_cache(void* base, int64_t at, bool f8, float inv,
                                            const float (&f)[8]) {
  if (f8) {
    float g[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = __fmul_rn(f[j], inv);
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(base) + at) =
        make_uint2(e4m3x4(g[0], g[1], g[2], g[3]), e4m3x4(g[4], g[5], g[6], g[7]));
  } else {
    store8(static_cast<uint16_t*>(base) + at, f);
  }
}

__global__ void __launch_bounds__(kAppendThreads) k_kv_append(const AppendArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int per_head = a.kv.D / 16;
  const int heads = a.Hq + 2 * a.kv.Hkv;
  const int64_t id = (int64_t)blockIdx.x * kAppendThreads + threadIdx.x;
  const int64_t per_token = (int64_t)heads * per_head;
  if (id >= per_token * a.T) return;
  const int t = (int)(id / per_token);
  const int rest = (int)(id - t * per_token);
  const int head = rest / per_head, item = rest - head * per_head;
  const int kind = head < a.Hq ? 0 : head < a.Hq + a.kv.Hkv ? 1 : 2;   // q, k, v
  const int h = kind == 0 ? head : kind == 1 ? head - a.Hq : head - a.Hq - a.kv.Hkv;
  const int pairs = kind == 2 ? 0 : a.rope_dim / 16;
  const bool turn = item < pairs;
  const int c0 = turn ? 8 * item : kind == 2 ? 16 * item : a.rope_dim + 16 * (item - pairs);
  const int c1 = turn ? c0 + a.rope_dim / 2 : c0 + 8;

  const int pos = a.positions[t];
  bool ok = pos >= 0;   // a negative position: a padding token, neither stored nor an error
  if (ok && a.rope_dim > 0 && pos >= a.rope_rows) {
    ok = false;
    if (a.err) atomicOr(a.err, kErrBadPage);
  }
  int64_t page = 0;
  if (ok && kind != 0) {
    const int seq = a.seq_ids ? a.seq_ids[t] : t;
    const int col = pos / a.kv.page_size;
    ok = seq >= 0 && seq < a.B && col < a.table_width;
    if (ok) {
      page = a.block_table[(int64_t)seq * a.table_width + col];
      ok = page >= 0 && page < a.kv.num_pages;
    }
    if (!ok && a.err) atomicOr(a.err, kErrBadPage);
  }
  uint16_t* qo = kind == 0 ? a.q_out + ((int64_t)t * a.Hq + h) * a.kv.D : nullptr;
  if (!ok) {
    if (kind == 0) {   // the query of a token without a position: zeros
      *reinterpret_cast<uint4*>(qo + c0) = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(qo + c1) = make_uint4(0, 0, 0, 0);
    }
    return;
  }
  const uint16_t* src = (kind == 0 ? a.q + t * a.q_stride : kind == 1 ? a.k + t * a.k_stride
                                                                      : a.v + t * a.v_stride) +
                        (int64_t)h * a.kv.D;
  float u[8], w[8];
  load8(src + c0, u);
  load8(src + c1, w);
  if (turn) {
    const float* rp = a.rope + (int64_t)pos * a.rope_dim + c0;
    const int half = a.rope_dim / 2;
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
      const float4 c = *reinterpret_cast<const float4*>(rp + j);
      const float4 s = *reinterpret_cast<const float4*>(rp + half + j);
      const float cc[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = u[j + i], y = w[j + i];
        u[j + i] = __fsub_rn(__fmul_rn(x, cc[i]), __fmul_rn(y, sn[i]));
        w[j + i] = __fadd_rn(__fmul_rn(y, cc[i]), __fmul_rn(x, sn[i]));
      }
    }
  }
  if (kind == 0) {
    store8(qo + c0, u);
    store8(qo + c1, w);
    return;
  }
  const int slot = pos % a.kv.page_size;
  if (kind == 1) {
    const int64_t at = page * a.kv.k_page_stride + slot * a.kv.k_slot_stride + h * a.kv.k_head_stride;
    store_cache(a.kv.k, at + c0, a.kv.dtype == FT_KV_E4M3, a.inv_k, u);
    store_cache(a.kv.k, at + c1, a.kv.dtype == FT_KV_E4M3, a.inv_k, w);
  } else {
    const int64_t at = page * a.kv.v_page_stride + slot * a.kv.v_slot_stride + h * a.kv.v_head_stride;
    store_cache(a.kv.v, at + c0, a.kv.dtype == FT_KV_E4M3, a.inv_v, u);
    store_cache(a.kv.v, at + c1, a.kv.dtype == FT_KV_E4M3, a.inv_v, w);
  }
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t stream) {
  const int64_t items = (int64_t)a.T * (a.Hq + 2 * a.kv.Hkv) * (a.kv.D / 16);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((items + kAppendThreads - 1) / kAppendThreads));
  cfg.blockDim = dim3(kAppendThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_kv_append, a);
}

}  // namespace ftmoe
