// The new tokens' keys and values into the paged cache, with the rotary embedding of q and k.
//
//   rotary   for i < R/2: (u_i, u_{i+R/2}) -> (u_i c_i - u_{i+R/2} s_i, u_{i+R/2} c_i + u_i s_i)
//            with c, s = rope[position][i], rope[position][R/2 + i]; elements past R unchanged
//   cache    page = block_table[seq][position / page_size], slot = position % page_size;
//            bf16 or E4M3 of the value times 1 / scale (E4M3: saturated at +-448)
//
// A thread takes two 8-element pieces of one head: a pair of pieces R/2 apart, which rotate into each
// other, or two neighbours past R. A block takes one token, or a few of few heads; the values are on
// their way before the token's page is known. Products and sums are rounded one by one (no fused
// multiply-add), so that a value on the edge between two E4M3 codes falls as plain float32 arithmetic
// lets it fall.
// Bound by memory: every value is read once and written once. 16000 tokens of 48 heads of 128 without
// rotation 70 us (82 % of the measured copy rate); 4093 tokens, rotated, into E4M3 22 us (62 %), where the
// conversions and the tables' reads (as many bytes as the values, from L1) come on top; three blocks an
// SM of 512 threads at 40 registers beat two at 64 (25 us), also with two tokens a thread in flight, and
// persistent blocks with the next token's values ahead (26 us) or tokens in a ring of bulk copies (28 us).
#include <cuda_runtime.h>

#include "ftmoe_internal.h"
#include "ftmoe_mma.cuh"

namespace ftmoe {

namespace {

constexpr int kAppendThreads = 256;   // of a block, or as many as one token needs up to 512

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

template <bool F8>
__device__ __forceinline__ void store_cache(void* base, int64_t at, float inv, const float (&f)[8]) {
  float g[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) g[j] = __fmul_rn(f[j], inv);
  if constexpr (F8) {
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(base) + at) =
        make_uint2(e4m3x4(g[0], g[1], g[2], g[3]), e4m3x4(g[4], g[5], g[6], g[7]));
  } else {
    store8(static_cast<uint16_t*>(base) + at, g);
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

template <int D, bool F8>
__global__ void __launch_bounds__(512, 3) k_kv_append(const AppendArgs a, int items, int tokens) {
  constexpr int PER_HEAD = D / 16;
  griddep_launch_dependents();
  griddep_wait();
  const int local = tokens > 1 ? (int)threadIdx.x / items : 0;
  const int t = blockIdx.x * tokens + local;
  if (local >= tokens || t >= a.T) return;
  for (int id = threadIdx.x - local * items; id < items; id += blockDim.x) {
    const int row = id / PER_HEAD, item = id % PER_HEAD;
    const int kind = row < a.Hq ? 0 : row < a.Hq + a.kv.Hkv ? 1 : 2;   // q, k, v
    const int head = kind == 0 ? row : kind == 1 ? row - a.Hq : row - a.Hq - a.kv.Hkv;
    const int pairs = kind == 2 ? 0 : a.rope_dim / 16;
    const bool turn = item < pairs;
    const int c0 = turn ? 8 * item : kind == 2 ? 16 * item : a.rope_dim + 16 * (item - pairs);
    const int c1 = turn ? c0 + a.rope_dim / 2 : c0 + 8;
    const uint16_t* src = (kind == 0 ? a.q + t * a.q_stride : kind == 1 ? a.k + t * a.k_stride
                                                                        : a.v + t * a.v_stride) + head * D;
    const uint4 x = ld16(src + c0), y = ld16(src + c1);
    // the token's place, while its values travel. A negative position: a padding token, neither
    // stored nor an error
    const int pos = a.positions[t];
    bool placed = pos >= 0;
    if (placed && a.rope_dim > 0 && pos >= a.rope_rows) {
      placed = false;
      if (a.err) atomicOr(a.err, kErrBadPage);
    }
    int64_t at = -1;
    if (placed && kind != 0) {
      const int seq = a.seq_ids ? a.seq_ids[t] : t;
      const int col = (int)((__umulhi((uint32_t)a.div_mul, (uint32_t)pos) + (uint32_t)pos) >> a.div_shift);
      const int slot = pos - col * a.kv.page_size;
      if (seq >= 0 && seq < a.B && col < a.table_width) {
        const int64_t page = a.block_table[(int64_t)seq * a.table_width + col];
        if (page >= 0 && page < a.kv.num_pages)
          at = kind == 1
                   ? page * a.kv.k_page_stride + slot * a.kv.k_slot_stride + head * a.kv.k_head_stride
                   : page * a.kv.v_page_stride + slot * a.kv.v_slot_stride + head * a.kv.v_head_stride;
      }
      if (at < 0 && a.err) atomicOr(a.err, kErrBadPage);
    }
    float u[8], w[8];
    unpack8(x, u);
    unpack8(y, w);
    if (turn && placed) {
      const float* rp = a.rope + (int64_t)pos * a.rope_dim + c0;
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
    if (kind == 0) {
      uint16_t* to = a.q_out + ((int64_t)t * a.Hq + head) * D;
      if (!placed) {   // the query of a token without a position: zeros
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = w[j] = 0.f;
      }
      store8(to + c0, u);
      store8(to + c1, w);
    } else if (at >= 0) {
      void* to = kind == 1 ? a.kv.k : a.kv.v;
      const float inv = kind == 1 ? a.inv_k : a.inv_v;
      store_cache<F8>(to, at + c0, inv, u);
      store_cache<F8>(to, at + c1, inv, w);
    }
  }
}

template <int D>
cudaError_t launch_d(const AppendArgs& a, cudaStream_t stream) {
  const int items = (a.Hq + 2 * a.kv.Hkv) * (D / 16);
  const int tokens = items < kAppendThreads ? kAppendThreads / items : 1;
  const int need = (items * tokens + 31) / 32 * 32;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.T + tokens - 1) / tokens));
  cfg.blockDim = dim3((unsigned)(need < 512 ? need : 512));
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return a.kv.dtype == FT_KV_E4M3 ? cudaLaunchKernelEx(&cfg, k_kv_append<D, true>, a, items, tokens)
                                  : cudaLaunchKernelEx(&cfg, k_kv_append<D, false>, a, items, tokens);
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& args, cudaStream_t stream) {
  AppendArgs a = args;
  page_division(a.kv.page_size, a.div_mul, a.div_shift);
  switch (a.kv.D) {
    case 64: return launch_d<64>(a, stream);
    case 128: return launch_d<128>(a, stream);
    case 256: return launch_d<256>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ftmoe
