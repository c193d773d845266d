// The new tokens' keys and values into the paged cache, with the rotary embedding of q and k.
//
//   rotary   for i < R/2: (u_i, u_{i+R/2}) -> (u_i c_i - u_{i+R/2} s_i, u_{i+R/2} c_i + u_i s_i)
//            with c, s = rope[position][i], rope[position][R/2 + i]; elements past R unchanged
//   cache    page = block_table[seq][position / page_size], slot = position % page_size;
//            bf16, or E4M3 of the value times 1 / scale, saturated at +-448
//
// One block takes a token, one thread two 8-element pieces of one head at a time: a pair of pieces R/2
// apart, which rotate into each other, or two neighbours past R; the values of four such items are on
// their way before the token's page is known. Products and sums are rounded one by one (no fused
// multiply-add), so that a value on the edge between two E4M3 codes falls as plain float32 arithmetic
// lets it fall. Bound by memory: every value is read once and written once.
#include <cuda_runtime.h>

#include "ftmoe_internal.h"
#include "ftmoe_mma.cuh"

namespace ftmoe {

namespace {

constexpr int kAppendThreads = 128;
constexpr int kAppendItems = 4;   // items of a thread whose loads are in flight together

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

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = bf16_lo(w[j]);
    f[2 * j + 1] = bf16_hi(w[j]);
  }
}

struct Item {   // a head of q, k or v (kind 0, 1, 2) and its two pieces
  int kind, head, c0, c1;
  bool turn;
  __device__ __forceinline__ Item(const AppendArgs& a, int id) {
    const int per_head = a.kv.D / 16;
    const int row = id / per_head, item = id - row * per_head;
    kind = row < a.Hq ? 0 : row < a.Hq + a.kv.Hkv ? 1 : 2;
    head = kind == 0 ? row : kind == 1 ? row - a.Hq : row - a.Hq - a.kv.Hkv;
    const int pairs = kind == 2 ? 0 : a.rope_dim / 16;
    turn = item < pairs;
    c0 = turn ? 8 * item : kind == 2 ? 16 * item : a.rope_dim + 16 * (item - pairs);
    c1 = turn ? c0 + a.rope_dim / 2 : c0 + 8;
  }
};

__global__ void __launch_bounds__(kAppendThreads) k_kv_append(const AppendArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t t = blockIdx.x;
  const int items = (a.Hq + 2 * a.kv.Hkv) * (a.kv.D / 16);
  const int pos = a.positions[t];
  const int seq = a.seq_ids ? a.seq_ids[t] : (int)t;
  bool placed = pos >= 0;   // a negative position: a padding token, neither stored nor an error
  bool found = false;
  int64_t page = 0;
  int slot = 0;
  for (int id0 = threadIdx.x; id0 < items; id0 += kAppendThreads * kAppendItems) {
    uint4 x[kAppendItems], y[kAppendItems];
#pragma unroll
    for (int i = 0; i < kAppendItems; ++i) {
      const int id = id0 + i * kAppendThreads;
      if (id >= items) continue;
      const Item it(a, id);
      const uint16_t* src = (it.kind == 0 ? a.q + t * a.q_stride
                             : it.kind == 1 ? a.k + t * a.k_stride : a.v + t * a.v_stride) +
                            (int64_t)it.head * a.kv.D;
      x[i] = ld16(src + it.c0);
      y[i] = ld16(src + it.c1);
    }
    if (id0 == threadIdx.x) {   // the token's place, while the first values travel
      if (placed && a.rope_dim > 0 && pos >= a.rope_rows) {
        placed = false;
        if (a.err && threadIdx.x == 0) atomicOr(a.err, kErrBadPage);
      }
      if (placed) {
        const int col = pos / a.kv.page_size;
        slot = pos - col * a.kv.page_size;
        found = seq >= 0 && seq < a.B && col < a.table_width;
        if (found) {
          page = a.block_table[(int64_t)seq * a.table_width + col];
          found = page >= 0 && page < a.kv.num_pages;
        }
        if (!found && a.err && threadIdx.x == 0) atomicOr(a.err, kErrBadPage);
      }
    }
#pragma unroll
    for (int i = 0; i < kAppendItems; ++i) {
      const int id = id0 + i * kAppendThreads;
      if (id >= items) continue;
      const Item it(a, id);
      float u[8], w[8];
      unpack8(x[i], u);
      unpack8(y[i], w);
      if (it.turn && placed) {
        const float* rp = a.rope + (int64_t)pos * a.rope_dim + it.c0;
        const int half = a.rope_dim / 2;
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
          const float4 c = *reinterpret_cast<const float4*>(rp + j);
          const float4 s = *reinterpret_cast<const float4*>(rp + half + j);
          const float cc[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float p = u[j + e], r = w[j + e];
            u[j + e] = __fsub_rn(__fmul_rn(p, cc[e]), __fmul_rn(r, sn[e]));
            w[j + e] = __fadd_rn(__fmul_rn(r, cc[e]), __fmul_rn(p, sn[e]));
          }
        }
      }
      if (it.kind == 0) {
        uint16_t* to = a.q_out + (t * a.Hq + it.head) * a.kv.D;
        if (!placed) {   // the query of a token without a position: zeros
#pragma unroll
          for (int j = 0; j < 8; ++j) u[j] = w[j] = 0.f;
        }
        store8(to + it.c0, u);
        store8(to + it.c1, w);
      } else if (found) {
        const bool key = it.kind == 1;
        const int64_t at =
            key ? page * a.kv.k_page_stride + slot * a.kv.k_slot_stride + it.head * a.kv.k_head_stride
                : page * a.kv.v_page_stride + slot * a.kv.v_slot_stride + it.head * a.kv.v_head_stride;
        void* to = key ? a.kv.k : a.kv.v;
        const float inv = key ? a.inv_k : a.inv_v;
        store_cache(to, at + it.c0, a.kv.dtype == FT_KV_E4M3, inv, u);
        store_cache(to, at + it.c1, a.kv.dtype == FT_KV_E4M3, inv, w);
      }
    }
  }
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.T);
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
