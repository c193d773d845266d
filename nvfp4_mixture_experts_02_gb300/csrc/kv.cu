// The new tokens' keys and values into the paged cache, with the rotary embedding of q and k.
//
//   rotary   for i < R/2: (u_i, u_{i+R/2}) -> (u_i c_i - u_{i+R/2} s_i, u_{i+R/2} c_i + u_i s_i)
//            with c, s = rope[position][i], rope[position][R/2 + i]; elements past R unchanged
//   cache    page = block_table[seq][position / page_size], slot = position % page_size;
//            bf16 or E4M3 of the value times 1 / scale (E4M3: saturated at +-448)
//
//   NVFP4    block of 16: s = e4m3(max|x| / (6 g)), code = e2m1(x / (s g)); see the header
//   axes     pair i turns by the position on its own axis
//
// A thread takes two 8-element pieces of one head: a pair of pieces R/2 apart, which rotate into each
// other, or two neighbours past R. Products and sums are rounded one by one (no fused multiply-add), so
// that a value on the edge between two codes falls as plain float32 arithmetic lets it fall.
//
// k_kv_append: a block takes one token, or a few of few heads; the values are on their way before the token's page
// is known. Three dependent loads (position, row of the table of angles or page, then the stores), no barrier: for
// few tokens (four 2.2 us) and without rotation (16000 tokens of 48 heads of 128 71 us, 82 % of the measured copy
// rate). Bound by load latency at the 48 warps an SM that 40 registers allow: 4093 rotated tokens into E4M3 23.3 us.
// k_kv_append_many: the blocks that the device holds at once share the tokens. A block looks up the places of all of
// its tokens and lays their cosines and sines out in shared memory, where all heads of a token read them and each
// pair's axis has been chosen; then a thread keeps its piece of a head and goes through the tokens with the next one's
// values on their way. 4093 tokens into NVFP4 19.7 us, into E4M3 18.8, into bf16 19.9, 9001 with three axes 38.1, 37.6
// and 40.2 (66 to 83 % of the copy rate): the loads' latency at the 36 warps that 56 registers allow, whose instructions, some
// 200 a thread and token, fill 63 % of the issue slots.
// k_kv_gather: a thread takes 16 elements of a key and of its value. Bound by memory: 115 thousand tokens of 8 heads
// of 128 from NVFP4 123 us (90 %), from E4M3 134 (96 %), from bf16 173 (99 %), most of it for the results.
#include <algorithm>
#include <cuda_runtime.h>

#include "ftmoe_internal.h"
#include "ftmoe_mma.cuh"

namespace ftmoe {

namespace {

constexpr int kAppendThreads = 256;   // of a block, or as many as one token needs up to 512
// k_kv_append_many: threads of a block at most, blocks that an SM holds (384 x 56 registers; 4093 tokens of 32 + 16 heads
// of 128 into NVFP4 19.7 us, 20.6 with two blocks of 72, 25.7 with four of 40; two tokens ahead 21.3 for 20.7).
constexpr int kManyThreads = 384, kManyBlocks = 3;
// From this many tokens a block (of those that the device holds at once) on, rotated ones of more than a few heads go
// through it: 1200 of those tokens (three a block) 8.7 us for 9.6, 4093 19.7 for 26.1 (into E4M3 18.8 for 23.3, into bf16 19.9
// for 24.2), 800 (two) 7.0 for 6.8. Not tokens that share a block: 40000 of 2 + 2 heads of 64 would take 16.0 for 14.7. Not
// without rotation: into bf16 k_kv_append is the faster there up to 16000 tokens or so (8000 36.8 us for 41.4, 16000 70.4 for
// 74.5, but 40000 172 for 161); into E4M3 and NVFP4 it is not (8000 34.3 for 31.9 and 40.3 for 32.4). Several axes always
// take it: 37 tokens 2.7 us, 3.2 with the choice of rows in each thread, 9001 38 us for 110.
constexpr int kManyTokens = 3;
constexpr int kAppendTokens = 32, kAppendBytes = 40 * 1024;   // most tokens of a group, most shared memory

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

// Two pieces of eight of a head as codes and scales. The halves of a block of 16 are this thread's own, or, where
// they turn, this thread's and its neighbour's (item ^ 1: rope_dim is a multiple of 32, so they turn both, and items
// a head are even, so they are lanes 2 i and 2 i + 1).
__device__ __forceinline__ void store_codes(uint8_t* codes, uint8_t* scales, bool turn, int item, int c0, int c1,
                                            float (&u)[8], float (&w)[8], float inv6, float g) {
  float tu = top8(u), tw = top8(w), mu, mw;
  if (turn) {
    const uint32_t both = 3u << (threadIdx.x & 30);
    tu = max_nan(tu, __shfl_xor_sync(both, tu, 1));
    tw = max_nan(tw, __shfl_xor_sync(both, tw, 1));
    const uint8_t su = block_scale(tu, inv6, g, mu), sw = block_scale(tw, inv6, g, mw);
    if (!(item & 1)) {
      scales[c0 / 16] = su;
      scales[c1 / 16] = sw;
    }
  } else {
    scales[c0 / 16] = block_scale(max_nan(tu, tw), inv6, g, mu);
    mw = mu;
  }
  *reinterpret_cast<uint32_t*>(codes + c0 / 2) = codes8(u, mu);
  *reinterpret_cast<uint32_t*>(codes + c1 / 2) = codes8(w, mw);
}

template <int D, int DT>
__global__ void __launch_bounds__(512, DT == kKvNvfp4 ? 2 : 3) k_kv_append(const AppendArgs a, int items, int tokens) {
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
    if (placed && a.rope_dim > 0 && pos >= a.rope_rows) {
      placed = false;
      if (a.err) atomicOr(a.err, kErrBadPage);
    }
    int64_t at = -1;
    [[maybe_unused]] int64_t scales_at = 0;
    if (placed && kind != 0) {
      const Place p = place_of(a, pos);
      const int slot = p.slot;
      const int64_t page = page_of(a, t, p.col);
      if (page >= 0) {
        at = kind == 1 ? page * a.kv.k_page_stride + slot * a.kv.k_slot_stride + head * a.kv.k_head_stride
                       : page * a.kv.v_page_stride + slot * a.kv.v_slot_stride + head * a.kv.v_head_stride;
        if constexpr (F4)
          scales_at = kind == 1 ? page * a.sc.k_page + slot * a.sc.k_slot + head * a.sc.k_head
                                : page * a.sc.v_page + slot * a.sc.v_slot + head * a.sc.v_head;
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
      if constexpr (F4) {
        store_codes(static_cast<uint8_t*>(to) + at, (kind == 1 ? a.sc.k : a.sc.v) + scales_at, turn, item, c0, c1, u, w,
                    inv, kind == 1 ? a.kv.k_scale : a.kv.v_scale);
      } else {
        store_cache<F8>(to, at + c0, inv, u);
        store_cache<F8>(to, at + c1, inv, w);
      }
    }
  }
}

// Where a token goes: offsets of its row without the head, in the unit of the strides.
struct TokenPlace {
  int64_t k_at, v_at, ks_at, vs_at;
  int placed, stored;   // it has a position (else its query is zero); it has a page
};

// Two pieces of a head: u and w of a turning pair, or neighbours.
struct Pieces {
  uint4 x, y;
};

template <int D, int DT, bool AXES>
__global__ void __launch_bounds__(kManyThreads, kManyBlocks)
    k_kv_append_many(const AppendArgs a, int items, int groups, int per) {
  constexpr int PER_HEAD = D / 16;
  constexpr bool F8 = DT == FT_KV_E4M3, F4 = DT == kKvNvfp4;
  extern __shared__ __align__(16) unsigned char smem[];
  const int R = a.rope_dim, half = R / 2;
  float* const factors = reinterpret_cast<float*>(smem);                                   // [token][R]
  TokenPlace* const places = reinterpret_cast<TokenPlace*>(factors + groups * per * R);    // [token]
  griddep_launch_dependents();
  griddep_wait();
  const int group = groups > 1 ? (int)threadIdx.x / items : 0;
  const int t0 = blockIdx.x * groups * per, n = min(groups * per, a.T - t0);   // the block's tokens
  bool first = true;
  for (int id = threadIdx.x - group * items;; id += blockDim.x) {
    const bool mine = group < groups && id < items;
    if (!first && !mine) break;
    const int row = id / PER_HEAD, item = id % PER_HEAD;
    const int kind = row < a.Hq ? 0 : row < a.Hq + a.kv.Hkv ? 1 : 2;   // q, k, v
    const int head = kind == 0 ? row : kind == 1 ? row - a.Hq : row - a.Hq - a.kv.Hkv;
    const int pairs = kind == 2 ? 0 : R / 16;
    const bool turn = item < pairs;
    const int c0 = turn ? 8 * item : kind == 2 ? 16 * item : R + 16 * (item - pairs);
    const int c1 = turn ? c0 + half : c0 + 8;
    const uint16_t* src = (kind == 0 ? a.q : kind == 1 ? a.k : a.v) + head * D;
    const int64_t stride = kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride;
    auto load = [&](int j) {
      const uint16_t* p = src + (t0 + j) * stride;
      return Pieces{ld16(p + c0), ld16(p + c1)};
    };
    Pieces next = {};
    if (mine && group < n) next = load(group);
    if (first) {   // places and factors of the block's tokens, while the first values travel
      first = false;
      for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int t = t0 + i, pos = a.positions[t];
        TokenPlace p = {0, 0, 0, 0, pos >= 0, 0};   // a negative position: a padding token, not an error
        if (pos >= 0) {
          bool in = true;
          if constexpr (AXES) {
            for (int x = 0; x < a.axes; ++x) {
              const int at = a.axis_pos[x * a.axis_stride + t];
              in &= at >= 0 && at < a.rope_rows;
            }
          } else {
            in = R == 0 || pos < a.rope_rows;
          }
          const Place where = place_of(a, pos);
          const int64_t page = in ? page_of(a, t, where.col) : -1;
          p.placed = in;
          if (page >= 0) {
            p.stored = 1;
            p.k_at = page * a.kv.k_page_stride + where.slot * a.kv.k_slot_stride;
            p.v_at = page * a.kv.v_page_stride + where.slot * a.kv.v_slot_stride;
            if constexpr (F4) {
              p.ks_at = page * a.sc.k_page + where.slot * a.sc.k_slot;
              p.vs_at = page * a.sc.v_page + where.slot * a.sc.v_slot;
            }
          } else if (a.err) {
            atomicOr(a.err, kErrBadPage);
          }
        }
        places[i] = p;
      }
      // Factor f of pair 8 i + 4 j + e lies at 4 (R/16 j + i) + e of its half: the threads of a head read
      // neighbouring 16 bytes.
      for (int i = threadIdx.x; i < n * half; i += blockDim.x) {
        const int j = i / half, pair = i - j * half, t = t0 + j;
        int at;
        if constexpr (AXES) at = a.axis_pos[(a.axis_of[pair >> 4] >> (2 * (pair & 15)) & 3) * a.axis_stride + t];
        else at = a.positions[t];
        float c = 1.f, s = 0.f;
        if (at >= 0 && at < a.rope_rows) {
          c = a.rope[(int64_t)at * R + pair];
          s = a.rope[(int64_t)at * R + half + pair];
        }
        float* to = factors + j * R + 4 * ((R / 16) * (pair >> 2 & 1) + (pair >> 3)) + (pair & 3);
        to[0] = c;
        to[half] = s;
      }
      __syncthreads();
    }
    if (!mine) break;
    for (int j = group; j < n; j += groups) {
      const Pieces now = next;
      if (j + groups < n) next = load(j + groups);
      const TokenPlace& place = places[j];
      float u[8], w[8];
      unpack8(now.x, u);
      unpack8(now.y, w);
      if (turn) {   // without a place nothing comes of it
        const float4* f = reinterpret_cast<const float4*>(factors + j * R) + item;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float4 c = f[x * (R / 16)], s = f[R / 8 + x * (R / 16)];
          const float cc[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float p = u[4 * x + e], r = w[4 * x + e];
            u[4 * x + e] = __fsub_rn(__fmul_rn(p, cc[e]), __fmul_rn(r, sn[e]));
            w[4 * x + e] = __fadd_rn(__fmul_rn(r, cc[e]), __fmul_rn(p, sn[e]));
          }
        }
      }
      if (kind == 0) {
        uint16_t* to = a.q_out + ((int64_t)(t0 + j) * a.Hq + head) * D;
        if (!place.placed) {   // the query of a token without a position: zeros
#pragma unroll
          for (int e = 0; e < 8; ++e) u[e] = w[e] = 0.f;
        }
        store8(to + c0, u);
        store8(to + c1, w);
      } else if (place.stored) {
        const int64_t at = kind == 1 ? place.k_at + head * a.kv.k_head_stride : place.v_at + head * a.kv.v_head_stride;
        void* to = kind == 1 ? a.kv.k : a.kv.v;
        const float inv = kind == 1 ? a.inv_k : a.inv_v;
        if constexpr (F4) {
          store_codes(static_cast<uint8_t*>(to) + at,
                      kind == 1 ? a.sc.k + place.ks_at + head * a.sc.k_head : a.sc.v + place.vs_at + head * a.sc.v_head,
                      turn, item, c0, c1, u, w, inv, kind == 1 ? a.kv.k_scale : a.kv.v_scale);
        } else {
          store_cache<F8>(to, at + c0, inv, u);
          store_cache<F8>(to, at + c1, inv, w);
        }
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
cudaError_t launch_t(cudaLaunchConfig_t cfg, const AppendArgs& a, int num_sms) {
  const int items = (a.Hq + 2 * a.kv.Hkv) * (D / 16);   // of a token
  const int groups = items < kAppendThreads ? kAppendThreads / items : 1;
  const int turns = (items + kManyThreads - 1) / kManyThreads;
  const int threads = ((turns > 1 ? (items + turns - 1) / turns : items * groups) + 31) / 32 * 32;
  const int resident = num_sms * (kManyBlocks * kManyThreads / threads);   // blocks of k_kv_append_many at once
  int per = (int)(((int64_t)a.T + (int64_t)resident * groups - 1) / ((int64_t)resident * groups));
  if (!a.axis_pos && (groups > 1 || per < kManyTokens || a.rope_dim == 0)) {
    const int need = (items * groups + 31) / 32 * 32;
    cfg.gridDim = dim3((unsigned)((a.T + groups - 1) / groups));
    cfg.blockDim = dim3((unsigned)(need < 512 ? need : 512));
    return cudaLaunchKernelEx(&cfg, k_kv_append<D, DT>, a, items, groups);
  }
  const int bytes = groups * (a.rope_dim * (int)sizeof(float) + (int)sizeof(TokenPlace));   // for one token each
  // Tokens that do not fit the blocks at once go in rounds. A last one of less than half of the blocks takes as long as
  // any other: all blocks then take fewer tokens instead (16000 tokens of 32 + 16 heads of 128 into bf16, half of each
  // head rotated, 85.4 -> 68.4 us). Fuller ones are left: 40000 with a quarter rotated 158 us, 174 in equal rounds.
  const int most = std::min(kAppendBytes / bytes, kAppendTokens), rounds = (per + most - 1) / most;
  per = per > most && 2 * (per % most) < most ? (per + rounds - 1) / rounds : std::min(per, most);
  cfg.gridDim = dim3((unsigned)((a.T + groups * per - 1) / (groups * per)));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)(per * bytes);
  return a.axis_pos ? cudaLaunchKernelEx(&cfg, k_kv_append_many<D, DT, true>, a, items, groups, per)
                    : cudaLaunchKernelEx(&cfg, k_kv_append_many<D, DT, false>, a, items, groups, per);
}

template <int D>
cudaError_t launch_d(const AppendArgs& a, int num_sms, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  switch (a.kv.dtype) {
    case FT_KV_BF16: return launch_t<D, FT_KV_BF16>(cfg, a, num_sms);
    case FT_KV_E4M3: return launch_t<D, FT_KV_E4M3>(cfg, a, num_sms);
  }
  return launch_t<D, kKvNvfp4>(cfg, a, num_sms);
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
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorNoDevice;
  page_division(a.kv.page_size, a.div_mul, a.div_shift);
  switch (a.kv.D) {
    case 64: return launch_d<64>(a, sms, stream);
    case 128: return launch_d<128>(a, sms, stream);
    case 256: return launch_d<256>(a, sms, stream);
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
