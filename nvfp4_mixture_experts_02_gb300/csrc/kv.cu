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

// Eight values as E2M1 codes, the first in the lowest four bits.
__device__ __forceinline__ uint32_t e2m1x8(const float (&f)[8]) {
  uint32_t d;
  asm("{\n\t.reg .b8 a, b, c, e;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 e, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, e};\n\t}"
      : "=r"(d)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return d;
}

__device__ __forceinline__ float max_nan(float a, float b) {   // NaN if either is
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float top8(const float (&f)[8]) {
  float m = fabsf(f[0]);
#pragma unroll
  for (int j = 1; j < 8; ++j) m = max_nan(m, fabsf(f[j]));
  return m;
}

// The E4M3 scale of a block of largest magnitude `top`, and what its elements are multiplied by.
__device__ __forceinline__ uint8_t block_scale(float top, float inv6, float g, float& mul) {
  const uint32_t s = e4m3x4(__fmul_rn(top, inv6), 0.f, 0.f, 0.f);
  const float d = __fmul_rn(f16_lo(e4m3x2_to_f16x2(s)), g);
  mul = d > 0.f ? __frcp_rn(d) : 0.f;
  return (uint8_t)s;
}
__device__ __forceinline__ uint32_t codes8(float (&f)[8], float mul) {
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = __fmul_rn(f[j], mul);
  return e2m1x8(f);
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

// Column of the block table, and slot in its page, of a place.
struct Place {
  int col, slot;
};
template <typename A>
__device__ __forceinline__ Place place_of(const A& a, int pos) {
  const int col = (int)((__umulhi((uint32_t)a.div_mul, (uint32_t)pos) + (uint32_t)pos) >> a.div_shift);
  return {col, pos - col * a.kv.page_size};
}
// The page of a column for token t, or -1.
template <typename A>
__device__ __forceinline__ int64_t page_of(const A& a, int t, int col) {
  const int seq = a.seq_ids ? a.seq_ids[t] : t;
  if (seq < 0 || seq >= a.B || col >= a.table_width) return -1;
  const int64_t page = a.block_table[(int64_t)seq * a.table_width + col];
  return page >= 0 && page < a.kv.num_pages ? page : -1;
}

// cos and sin of four pairs from pair c0 on, whose axes `which` names, two bits each.
__device__ __forceinline__ void axis_rows(const AppendArgs& a, const int (&pos)[4], int c0, uint32_t which,
                                          float (&c)[4], float (&s)[4]) {
  const int half = a.rope_dim / 2;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    bool any = false;
#pragma unroll
    for (int e = 0; e < 4; ++e) any |= ((which >> (2 * e)) & 3) == x;
    if (!any) continue;
    const float* rp = a.rope + (int64_t)pos[x] * a.rope_dim + c0;
    const float4 vc = *reinterpret_cast<const float4*>(rp);
    const float4 vs = *reinterpret_cast<const float4*>(rp + half);
    const float cc[4] = {vc.x, vc.y, vc.z, vc.w}, ss[4] = {vs.x, vs.y, vs.z, vs.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (((which >> (2 * e)) & 3) == x) {
        c[e] = cc[e];
        s[e] = ss[e];
      }
  }
}

template <int D, int DT, bool AXES>
__global__ void __launch_bounds__(512, DT == kKvNvfp4 || AXES ? 2 : 3)
    k_kv_append(const AppendArgs a, int items, int tokens) {
  constexpr int PER_HEAD = D / 16;
  constexpr bool F8 = DT == FT_KV_E4M3, F4 = DT == kKvNvfp4;
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
    int on_axis[4] = {pos, pos, pos, pos};
    if constexpr (AXES) {
      bool in = true;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < a.axes) {
          on_axis[i] = a.axis_pos[i * a.axis_stride + t];
          in &= on_axis[i] >= 0 && on_axis[i] < a.rope_rows;
        }
      if (placed && !in) {
        placed = false;
        if (a.err) atomicOr(a.err, kErrBadPage);
      }
    } else if (placed && a.rope_dim > 0 && pos >= a.rope_rows) {
      placed = false;
      if (a.err) atomicOr(a.err, kErrBadPage);
    }
    int64_t page = -1;
    int slot = 0;
    if (placed && kind != 0) {
      const Place p = place_of(a, pos);
      slot = p.slot;
      page = page_of(a, t, p.col);
      if (page < 0 && a.err) atomicOr(a.err, kErrBadPage);
    }
    float u[8], w[8];
    unpack8(x, u);
    unpack8(y, w);
    if (turn && placed) {
      const int half = a.rope_dim / 2;
      uint32_t which = 0;   // the axes of the eight pairs, two bits each
      bool one = true;      // they turn alike
      if constexpr (AXES) {
        which = a.axis_of[item >> 1] >> (16 * (item & 1)) & 0xFFFFu;
        one = which == (which & 3) * 0x5555u;
      }
      const float* rp = a.rope + (int64_t)(AXES ? on_axis[which & 3] : pos) * a.rope_dim + c0;
#pragma unroll
      for (int j = 0; j < 8; j += 4) {
        float cc[4], sn[4];
        if (!AXES || one) {
          const float4 c = *reinterpret_cast<const float4*>(rp + j);
          const float4 s = *reinterpret_cast<const float4*>(rp + half + j);
          cc[0] = c.x; cc[1] = c.y; cc[2] = c.z; cc[3] = c.w;
          sn[0] = s.x; sn[1] = s.y; sn[2] = s.z; sn[3] = s.w;
        } else {
          axis_rows(a, on_axis, c0 + j, which >> (2 * j), cc, sn);
        }
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
    } else if (page >= 0) {
      const int64_t at =
          kind == 1 ? page * a.kv.k_page_stride + slot * a.kv.k_slot_stride + head * a.kv.k_head_stride
                    : page * a.kv.v_page_stride + slot * a.kv.v_slot_stride + head * a.kv.v_head_stride;
      void* to = kind == 1 ? a.kv.k : a.kv.v;
      const float inv = kind == 1 ? a.inv_k : a.inv_v;
      if constexpr (F4) {
        // The two pieces of a block of 16 are this thread's own, or, where they turn, this thread's and
        // its neighbour's (item ^ 1: rope_dim is a multiple of 32, so they turn both, and items a head
        // are even, so they are lanes 2 i and 2 i + 1).
        const float g = kind == 1 ? a.kv.k_scale : a.kv.v_scale;
        uint8_t* scales =
            kind == 1 ? a.sc.k + page * a.sc.k_page + slot * a.sc.k_slot + head * a.sc.k_head
                      : a.sc.v + page * a.sc.v_page + slot * a.sc.v_slot + head * a.sc.v_head;
        float tu = top8(u), tw = top8(w), mu, mw;
        if (turn) {
          const uint32_t both = 3u << (threadIdx.x & 30);
          tu = max_nan(tu, __shfl_xor_sync(both, tu, 1));
          tw = max_nan(tw, __shfl_xor_sync(both, tw, 1));
          const uint8_t su = block_scale(tu, inv, g, mu), sw = block_scale(tw, inv, g, mw);
          if (!(item & 1)) {
            scales[c0 / 16] = su;
            scales[c1 / 16] = sw;
          }
        } else {
          scales[c0 / 16] = block_scale(max_nan(tu, tw), inv, g, mu);
          mw = mu;
        }
        uint8_t* codes = static_cast<uint8_t*>(to) + at;
        *reinterpret_cast<uint32_t*>(codes + c0 / 2) = codes8(u, mu);
        *reinterpret_cast<uint32_t*>(codes + c1 / 2) = codes8(w, mw);
      } else {
        store_cache<F8>(to, at + c0, inv, u);
        store_cache<F8>(to, at + c1, inv, w);
      }
    }
  }
}

// 16 elements (32 bytes) of a result, in one store.
__device__ __forceinline__ void store16(uint16_t* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// Cached tokens as dense bf16. A thread takes 16 elements of a key and of the value beside it.
template <int DT>
__device__ __forceinline__ void read16(const void* base, int64_t at, const uint8_t* scales, float mul,
                                       uint32_t (&o)[8]) {
  if constexpr (DT == FT_KV_BF16) {
    const uint16_t* p = static_cast<const uint16_t*>(base) + at;
    float f[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      load8(p + 8 * h, f);
#pragma unroll
      for (int j = 0; j < 4; ++j) o[4 * h + j] = pack_bf16(f[2 * j] * mul, f[2 * j + 1] * mul);
    }
  } else if constexpr (DT == FT_KV_E4M3) {
    const uint4 v = ld16(static_cast<const uint8_t*>(base) + at);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t h = e4m3x2_to_f16x2(w[j / 2] >> (16 * (j & 1)));
      o[j] = pack_bf16(f16_lo(h) * mul, f16_hi(h) * mul);
    }
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(base) + at);
    const uint32_t s = splat_lo(e4m3x2_to_f16x2(*scales));
    const uint32_t w[2] = {v.x, v.y};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t x[4];
      e2m1x8_to_f16x2x4(w[h], x[0], x[1], x[2], x[3]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t y = hmul2(x[j], s);   // exact: six significant bits
        o[4 * h + j] = pack_bf16(f16_lo(y) * mul, f16_hi(y) * mul);
      }
    }
  }
}

template <int D, int DT>
__global__ void __launch_bounds__(256) k_kv_gather(const GatherArgs a) {
  constexpr int PER_HEAD = D / 16;
  griddep_launch_dependents();
  griddep_wait();
  const int items = a.kv.Hkv * PER_HEAD;
  const int64_t all = (int64_t)a.T * items;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < all; i += (int64_t)gridDim.x * blockDim.x) {
    const int t = (int)(i / items), id = (int)(i - (int64_t)t * items);
    const int head = id / PER_HEAD, block = id % PER_HEAD;
    uint32_t k[8] = {}, v[8] = {};
    const int pos = a.positions[t];
    if (pos >= 0) {   // else padding: zeros
      const Place p = place_of(a, pos);
      const int64_t page = page_of(a, t, p.col);
      if (page >= 0) {
        const int64_t ka = page * a.kv.k_page_stride + p.slot * a.kv.k_slot_stride + head * a.kv.k_head_stride;
        const int64_t va = page * a.kv.v_page_stride + p.slot * a.kv.v_slot_stride + head * a.kv.v_head_stride;
        const uint8_t *ks = nullptr, *vs = nullptr;
        if constexpr (DT == kKvNvfp4) {
          ks = a.sc.k + page * a.sc.k_page + p.slot * a.sc.k_slot + head * a.sc.k_head + block;
          vs = a.sc.v + page * a.sc.v_page + p.slot * a.sc.v_slot + head * a.sc.v_head + block;
        }
        constexpr int STEP = DT == kKvNvfp4 ? 8 : 16;   // of a block, in the unit of the strides
        read16<DT>(a.kv.k, ka + block * STEP, ks, a.kv.k_scale, k);
        read16<DT>(a.kv.v, va + block * STEP, vs, a.kv.v_scale, v);
      } else if (a.err) {
        atomicOr(a.err, kErrBadPage);
      }
    }
    store16(a.k_out + i * 16, k);
    store16(a.v_out + i * 16, v);
  }
}

template <int D, int DT>
cudaError_t launch_axes(const cudaLaunchConfig_t& cfg, const AppendArgs& a, int items, int tokens) {
  return a.axis_pos ? cudaLaunchKernelEx(&cfg, k_kv_append<D, DT, true>, a, items, tokens)
                    : cudaLaunchKernelEx(&cfg, k_kv_append<D, DT, false>, a, items, tokens);
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
  switch (a.kv.dtype) {
    case FT_KV_BF16: return launch_axes<D, FT_KV_BF16>(cfg, a, items, tokens);
    case FT_KV_E4M3: return launch_axes<D, FT_KV_E4M3>(cfg, a, items, tokens);
  }
  return launch_axes<D, kKvNvfp4>(cfg, a, items, tokens);
}

template <int D>
cudaError_t launch_gather_d(const GatherArgs& a, cudaStream_t stream) {
  const int64_t blocks = ((int64_t)a.T * a.kv.Hkv * (D / 16) + 255) / 256;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(blocks < (1 << 30) ? blocks : 1 << 30));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  switch (a.kv.dtype) {
    case FT_KV_BF16: return cudaLaunchKernelEx(&cfg, k_kv_gather<D, FT_KV_BF16>, a);
    case FT_KV_E4M3: return cudaLaunchKernelEx(&cfg, k_kv_gather<D, FT_KV_E4M3>, a);
  }
  return cudaLaunchKernelEx(&cfg, k_kv_gather<D, kKvNvfp4>, a);
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

cudaError_t launch_kv_gather(const GatherArgs& args, cudaStream_t stream) {
  GatherArgs a = args;
  page_division(a.kv.page_size, a.div_mul, a.div_shift);
  switch (a.kv.D) {
    case 64: return launch_gather_d<64>(a, stream);
    case 128: return launch_gather_d<128>(a, stream);
    case 256: return launch_gather_d<256>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ftmoe
