// One warp's keys of a piece of paged attention (attention.cu) over an NVFP4 cache.
//
// Row operands from registers. Lane (r, c) = (lane / 4, lane % 4) of a 16-key tile takes D/4 consecutive elements of
// keys r and r + 8 as the row operand of k q^T, and D/8 consecutive elements, from r D/8 on, of keys 2c, 2c + 1,
// 2c + 8 and 2c + 9 as that of v^T p^T: whole words of codes under one scale or two. Products do not care which
// element is which column (q is laid out to match), nor which key is which row.
//
// A code becomes f16 by one conversion for two and one multiplication by its scale (e2m1 * e4m3 has six significant
// bits), so a step of 32 keys of 128 elements issues some 620 instructions (256 of them these), which the 12 warps of an
// SM overlap with the copies: products of the next step and values of this one are independent and stand side by side.
// A weight is two f16, as for E4M3 caches. One alone, 11 bits, puts one output in some thirty on the neighbouring bf16
// (8e-4 off the rounded exact result for 1e-4) and takes 56.9 us for 60.7 (48 ragged sequences), 56.6 for 63.1 (three
// long ones), 27.1 for 28.4 (heads of 64, a window of 1023): half of the value products. The second product of a pair
// right behind the first: 60.7 us, 62.1 behind all four first ones of a word.
// Measured and not kept, with weights still in one f16: 16 warps of 128 registers (spills and two stages: 123 us for 103 at 64 x 6500, with three
// stages 109), four stages for three (no change), groups held to the slowest one's pace (2 to 5 % slower), copies of
// whole tiles by the tensor memory accelerator (rows of 64 bytes at 6.5 TB/s for 6.7, of 32 at 4.6 for 5.2 in a copy
// of the same pattern), hints that fetch 128 or 256 bytes into L2 (no change).
#pragma once

#include <cmath>

#include "ftmoe_internal.h"
#include "ftmoe_mma.cuh"
#include "ftmoe_tc.cuh"

namespace ftmoe {

// Which key of a tile is its row i (0 <= i < 8; 8 + i follows), and where the 16-byte pieces of a row lie: so that
// the rows of k that eight lanes read at once, and the pieces of v, find 32 banks.
template <int D>
__device__ __forceinline__ int key_of_row(int i) {
  return D == 64 ? i ^ (i >> 2) : D == 128 ? i ^ ((i >> 1) & 1) : i;
}
template <int D>
__device__ __forceinline__ int piece4(int row, int ch) {   // offset of 16-byte piece ch of a row
  return row * (D / 2) + (D == 64 ? ch : D == 128 ? ch ^ (2 * ((row >> 2) & 1)) : ch ^ (row & 7)) * 16;
}

// N bytes (4, 8 or 16) from global to shared memory; zeros (and no access) when !valid.
template <int N>
__device__ __forceinline__ void cp_async_scales(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(valid ? N : 0)
               : "memory");
}

// 16 bytes from global to shared memory, past L1.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Pairs of floats.
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
  return d;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(v));
  return d;
}
__device__ __forceinline__ uint64_t pair_mul(uint64_t x, uint64_t y) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
  return d;
}
__device__ __forceinline__ uint64_t pair_add(uint64_t x, uint64_t y) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
  return d;
}

__device__ __forceinline__ uint32_t transpose8(uint32_t v) {   // an 8 x 8 matrix of 16-bit elements
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Four E4M3 bytes -> f16x2 of the lower two and of the upper two, exact.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t v, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi) : "r"(v));
}

// x times the lower (upper) half of s.
__device__ __forceinline__ uint32_t hmul2_lo(uint32_t x, uint32_t s) {
  const __half2 y = __hmul2(*reinterpret_cast<__half2*>(&x), __low2half2(*reinterpret_cast<__half2*>(&s)));
  return *reinterpret_cast<const uint32_t*>(&y);
}
__device__ __forceinline__ uint32_t hmul2_hi(uint32_t x, uint32_t s) {
  const __half2 y = __hmul2(*reinterpret_cast<__half2*>(&x), __high2half2(*reinterpret_cast<__half2*>(&s)));
  return *reinterpret_cast<const uint32_t*>(&y);
}

// W words from shared memory.
template <int W>
__device__ __forceinline__ void words(uint32_t (&v)[W], const char* p) {
  if constexpr (W == 1) {
    v[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (W == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    v[0] = x.x; v[1] = x.y;
  } else {
    const uint4 x = *reinterpret_cast<const uint4*>(p);
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
  }
}

// The scales of lane c's elements of a key, two in a word (with heads of 64: one).
template <int D>
__device__ __forceinline__ void key_scales(uint32_t (&s)[D == 256 ? 2 : 1], const char* row, int c) {
  if constexpr (D == 64) s[0] = e4m3x2_to_f16x2(*reinterpret_cast<const uint8_t*>(row + c));
  else if constexpr (D == 128) s[0] = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(row + 2 * c));
  else e4m3x4_to_f16(*reinterpret_cast<const uint32_t*>(row + 4 * c), s[0], s[1]);
}
// The scales of lane r's elements of two values, the first one's in the lower half of a word.
template <int D>
__device__ __forceinline__ void value_scales(uint32_t (&s)[D == 256 ? 2 : 1], const char* row0, const char* row1, int r) {
  if constexpr (D == 256) {
    const uint32_t x = *reinterpret_cast<const uint16_t*>(row0 + 2 * r);
    const uint32_t y = *reinterpret_cast<const uint16_t*>(row1 + 2 * r);
    s[0] = e4m3x2_to_f16x2(__byte_perm(x, y, 0x0040));
    s[1] = e4m3x2_to_f16x2(__byte_perm(x, y, 0x0051));
  } else {
    const int at = D == 64 ? r >> 1 : r;
    const uint32_t x = *reinterpret_cast<const uint8_t*>(row0 + at), y = *reinterpret_cast<const uint8_t*>(row1 + at);
    s[0] = e4m3x2_to_f16x2(x | y << 8);
  }
}

// A weight is at most 2^kTop4, and the largest of a head's is set to 2^kSet4 where the running maximum is set anew,
// which is when one would pass 2^kTop4: few steps after the first do, and the others need no maximum over the
// lanes. Two f16 hold 22 bits of weights down to 2^-3 and all but 2^-25 of smaller ones: 2^-35 of the largest.
constexpr float kTop4 = 15.f, kSet4 = 10.f;

// Steps of S::kKeys keys, key0 + i * unit on, up to key1 (and from `first` on). Leaves the warp's o^T, running
// maximum (log2, less kSet4 or so) and sums of weights of heads 2c and 2c + 1 over this lane's rows.
template <int D, int NG, class S>
__device__ __forceinline__ void attend_piece4(const AttendArgs& a, char* ring, int b, int kvh, int g0, int G, int first,
                                              int key0, int key1, int unit, int n_sub, float (&o)[NG][D / 16][4],
                                              float (&m)[NG][2], float (&l)[NG][2]) {
  constexpr int KT = S::kKeys, NH = KT / 16, ST = S::kStages, KS = D / 16, ROW = D / 2, SROW = D / 16;
  constexpr int V = KT * ROW, KSC = 2 * V, VSC = KSC + KT * SROW;   // values, scales of a stage
  const int lane = threadIdx.x & 31, c = lane & 3, r = lane >> 2;
  const int32_t* table = a.block_table + (int64_t)b * a.table_width;

  // ---- copies: lane l looks after keys l and, with 64 a step, l + 32 of it
  // offsets of rows in 16-byte pieces, of scales in rows of them: 32 bits (checked on the host)
  constexpr int KL = KT > 32 ? KT / 32 : 1, KR = KT / KL;   // keys of a lane, keys between them
  int page[KL], slot[KL];
  bool live[KL];
  auto look_up = [&](int i) {
#pragma unroll
    for (int z = 0; z < KL; ++z) {
      const int j = key0 + i * unit + 32 * z + lane;
      live[z] = i < n_sub && lane < KR && j >= first && j < key1;
      page[z] = -1;
      slot[z] = 0;
      if (live[z]) {
        const int col = (int)((__umulhi((uint32_t)a.div_mul, (uint32_t)j) + (uint32_t)j) >> a.div_shift);
        slot[z] = j - col * a.kv.page_size;
        page[z] = table[col];   // col < table_width: the length is cut to the table
      }
    }
  };
  constexpr int CPR = ROW / 16, RPI = 32 / CPR;   // 16-byte pieces of a row, rows of one warp-wide copy
  const int ch = lane % CPR;
  const char* const kb = static_cast<const char*>(a.kv.k) + kvh * a.kv.k_head_stride + ch * 16;
  const char* const vb = static_cast<const char*>(a.kv.v) + kvh * a.kv.v_head_stride + ch * 16;
  const uint8_t *const ksb = a.sc.k + kvh * a.sc.k_head, *const vsb = a.sc.v + kvh * a.sc.v_head;
  const uint32_t to0 = smem_addr(ring);
  auto fetch = [&](int i, uint32_t stage) {   // the copies of step i, whose pages look_up has found
    if (i < n_sub) {
#pragma unroll
      for (int z = 0; z < KL; ++z) {
        const bool in = (uint32_t)page[z] < (uint32_t)a.kv.num_pages;
        if (live[z] && !in) atomicOr(a.err, kErrBadPage);   // no such page: read as zeros
        // A key that is not there has codes and scales of zero.
        const uint32_t p = in ? (uint32_t)page[z] : 0u, s = in ? (uint32_t)slot[z] : 0u;
        const uint32_t st = to0 + stage + 32 * z * ROW, sc = to0 + stage + (32 * z + lane) * SROW;
        const uint32_t ko = p * (uint32_t)(a.kv.k_page_stride >> 4) + s * (uint32_t)(a.kv.k_slot_stride >> 4);
        const uint32_t kso = p * (uint32_t)(a.sc.k_page / SROW) + s * (uint32_t)(a.sc.k_slot / SROW);
        uint32_t vo = ko, vso = kso;
        if (!a.same_strides) {
          vo = p * (uint32_t)(a.kv.v_page_stride >> 4) + s * (uint32_t)(a.kv.v_slot_stride >> 4);
          vso = p * (uint32_t)(a.sc.v_page / SROW) + s * (uint32_t)(a.sc.v_slot / SROW);
        }
        if (KR == 32 || lane < KR) {
          cp_async_scales<SROW>(sc + KSC, ksb + (uint64_t)kso * SROW, in);
          cp_async_scales<SROW>(sc + VSC, vsb + (uint64_t)vso * SROW, in);
        }
        const uint32_t rows = __ballot_sync(0xffffffffu, in);
        if (rows == 0xffffffffu >> (32 - KR) && a.same_strides) {   // as a rule
#pragma unroll
          for (int x = 0; x < KR / RPI; ++x) {
            const uint32_t at = __shfl_sync(0xffffffffu, ko, x * RPI + lane / CPR);
            const uint32_t to = st + piece4<D>(x * RPI + lane / CPR, ch);
            copy16(to, kb + (uint64_t)at * 16);
            copy16(to + V, vb + (uint64_t)at * 16);
          }
        } else {
#pragma unroll
          for (int x = 0; x < KR / RPI; ++x) {
            const int row = x * RPI + lane / CPR;
            const bool on = rows >> row & 1;
            const uint32_t to = st + piece4<D>(row, ch);
            cp_async16(to, kb + (uint64_t)__shfl_sync(0xffffffffu, ko, row) * 16, on);
            cp_async16(to + V, vb + (uint64_t)__shfl_sync(0xffffffffu, vo, row) * 16, on);
          }
        }
      }
    }
    cp_async_commit();
  };
  look_up(0);
#pragma unroll
  for (int i = 0; i < ST - 1; ++i) {
    fetch(i, i * S::kStageBytes);
    look_up(i + 1);
  }

  // ---- q as the column operand, f16 after a power of two: column l / 4 of group g is head 8 g + l / 4. The
  // sign of the scale goes into q, so that a larger product is a larger score.
  uint32_t q[NG][KS][2];
  // Of two groups, one (two with heads of 256) stays in shared memory, where each lane keeps its own words: its
  // registers would cost warps.
  constexpr int QS = S::kQShared;
  uint2* const qs = reinterpret_cast<uint2*>(ring + ST * S::kStageBytes) + lane;
  uint64_t sl[NG];   // log2 units per unit of the raw product, heads 8 g + 2 c, + 1
  {
    const uint16_t* qb = a.q + (int64_t)b * a.q_stride + (int64_t)(kvh * a.group + g0) * D;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const bool on = 8 * g + r < G;
      const uint16_t* qh = qb + (8 * g + r) * D + D / 4 * c;
      float top = 0.f, up, down;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint2 v = make_uint2(0, 0);
        if (on) v = *reinterpret_cast<const uint2*>(qh + 4 * ks);
        q[g][ks][0] = v.x;
        q[g][ks][1] = v.y;
        top = fmaxf(top, finite_top(v.x, v.y));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      f16_scale(top, up, down);
      if (a.scale < 0.f) up = -up;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int e = 0; e < 2; ++e) q[g][ks][e] = pack_f16(bf16_lo(q[g][ks][e]) * up, bf16_hi(q[g][ks][e]) * up);
      const float unit_s = product3(fabsf(a.scale), a.kv.k_scale, down) * 1.4426950408889634f;
      sl[g] = pair(__shfl_sync(0xffffffffu, unit_s, 8 * c),   // head 2 c: lanes 8 c ..
                   __shfl_sync(0xffffffffu, unit_s, 8 * c + 4));
    }
#pragma unroll
    for (int g = 0; g < QS; ++g)
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) qs[32 * (g * KS + ks)] = make_uint2(q[NG - 1 - g][ks][0], q[NG - 1 - g][ks][1]);
  }

  uint64_t less[NG], sum[NG];   // - the running maximum (0 without one), sums of weights
  float bar[NG][2];             // scores past it set the maximum anew
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    less[g] = sum[g] = 0;
    bar[g][0] = bar[g][1] = -INFINITY;
  }
  float s[NG][NH][4];
  uint32_t p[NG][NH][2], rest[NG][NH][2];   // p^T: columns heads, rows keys 0-7 and 8-15 of a tile

  // s^T = k q^T of a stage
  const int krow = key_of_row<D>(r);
  auto products = [&](const char* st) {
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      constexpr int NW = D / 32;   // words of a lane's elements of a key
      uint32_t k0[NW], k1[NW], s0[D == 256 ? 2 : 1], s1[D == 256 ? 2 : 1];
      const int row = 16 * h + krow;
      if constexpr (D == 64) {
        words(k0, st + piece4<D>(row, c >> 1) + (c & 1) * 8);
        words(k1, st + piece4<D>(row + 8, c >> 1) + (c & 1) * 8);
      } else {
#pragma unroll
        for (int x = 0; x < NW / 4; ++x) {
          uint32_t t0[4], t1[4];
          words(t0, st + piece4<D>(row, NW / 4 * c + x));
          words(t1, st + piece4<D>(row + 8, NW / 4 * c + x));
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            k0[4 * x + y] = t0[y];
            k1[4 * x + y] = t1[y];
          }
        }
      }
      key_scales<D>(s0, st + KSC + row * SROW, c);
      key_scales<D>(s1, st + KSC + (row + 8) * SROW, c);
#pragma unroll
      for (int g = 0; g < NG; ++g) s[g][h][0] = s[g][h][1] = s[g][h][2] = s[g][h][3] = 0.f;
#pragma unroll
      for (int j = 0; j < NW; ++j) {
        uint32_t x[4], y[4];
        e2m1x8_to_f16x2x4(k0[j], x[0], x[1], x[2], x[3]);
        e2m1x8_to_f16x2x4(k1[j], y[0], y[1], y[2], y[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {   // exact: six significant bits
          x[e] = j / 2 % 2 ? hmul2_hi(x[e], s0[j / 4]) : hmul2_lo(x[e], s0[j / 4]);
          y[e] = j / 2 % 2 ? hmul2_hi(y[e], s1[j / 4]) : hmul2_lo(y[e], s1[j / 4]);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            uint2 w = make_uint2(q[g][2 * j + e][0], q[g][2 * j + e][1]);
            if (NG - 1 - g < QS) w = qs[32 * ((NG - 1 - g) * KS + 2 * j + e)];
            mma_f16(s[g][h], x[2 * e], y[2 * e], x[2 * e + 1], y[2 * e + 1], w.x, w.y);
          }
        }
      }
    }
  };

  // weights of the scores of step i: key j0 + 16 h + row r (elements 0, 1) and + 8
  auto weigh = [&](int i) {
    const int j0 = key0 + i * unit;
    uint64_t x[NG][NH][2];
    bool past = false;
    float top[NG][2];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        x[g][h][0] = pair_mul(pair(s[g][h][0], s[g][h][1]), sl[g]);
        x[g][h][1] = pair_mul(pair(s[g][h][2], s[g][h][3]), sl[g]);
      }
    }
    if (j0 < first || j0 + KT > key1) {   // keys outside do not count
#pragma unroll
      for (int h = 0; h < NH; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = j0 + 16 * h + krow + 8 * e;
          if (j < first || j >= key1) {
#pragma unroll
            for (int g = 0; g < NG; ++g) x[g][h][e] = pair(-INFINITY, -INFINITY);
          }
        }
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      top[g][0] = top[g][1] = -INFINITY;
#pragma unroll
      for (int h = 0; h < NH; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 v = unpair(x[g][h][e]);
          top[g][0] = fmaxf(top[g][0], v.x);
          top[g][1] = fmaxf(top[g][1], v.y);
        }
      past |= top[g][0] > bar[g][0] || top[g][1] > bar[g][1];
    }
    if (__any_sync(0xffffffffu, past)) {   // a new maximum: what is summed shrinks
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float f[2], n[2];
        const float2 was = unpair(less[g]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float t = top[g][e];
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, d));
          const bool none = bar[g][e] == -INFINITY;
          const float old = e ? -was.y : -was.x;
          t = __fsub_ru(t, kSet4);   // upwards: no weight above 2^kSet4 at any size of t
          n[e] = none ? t : fmaxf(old, t);
          f[e] = none ? 0.f : exp2_fast(old - n[e]);
          bar[g][e] = __fadd_rd(n[e], kTop4);   // downwards: no weight above 2^kTop4 either
          if (n[e] == -INFINITY) n[e] = 0.f;   // no key yet: every weight is 0
        }
        less[g] = pair(-n[0], -n[1]);
        sum[g] = pair_mul(sum[g], pair(f[0], f[1]));
#pragma unroll
        for (int t = 0; t < D / 16; ++t) {
          o[g][t][0] *= f[0]; o[g][t][1] *= f[1];
          o[g][t][2] *= f[0]; o[g][t][3] *= f[1];
        }
      }
    }
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int h = 0; h < NH; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 v = unpair(pair_add(x[g][h][e], less[g]));
          const float w0 = exp2_fast(v.x), w1 = exp2_fast(v.y);
          sum[g] = pair_add(sum[g], pair(w0, w1));
          const uint32_t v16 = pack_f16(w0, w1);
          p[g][h][e] = transpose8(v16);
          rest[g][h][e] = transpose8(pack_f16(w0 - f16_lo(v16), w1 - f16_hi(v16)));
        }
  };

  // o^T += v^T p^T of a stage
  const int vrow0 = key_of_row<D>(2 * c), vrow1 = key_of_row<D>(2 * c + 1);
  auto add_values = [&](const char* st) {
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      constexpr int NW = D / 64;   // words of a lane's elements of a value
      constexpr int NS = D == 256 ? 2 : 1;
      uint32_t v[4][NW], s01[NS], s89[NS];   // keys 2 c, 2 c + 1, 2 c + 8, 2 c + 9
      const int rows[4] = {16 * h + vrow0, 16 * h + vrow1, 16 * h + vrow0 + 8, 16 * h + vrow1 + 8};
#pragma unroll
      for (int x = 0; x < 4; ++x) words(v[x], st + V + piece4<D>(rows[x], D * r / 256) + (D * r / 16 & 15));
      const char* sc = st + VSC;
      value_scales<D>(s01, sc + rows[0] * SROW, sc + rows[1] * SROW, r);
      value_scales<D>(s89, sc + rows[2] * SROW, sc + rows[3] * SROW, r);
#pragma unroll
      for (int j = 0; j < NW; ++j) {
        // elements 2 i (a0, a2) and 2 i + 1 (a1, a3) of two keys in byte i of a word
        uint32_t a0[4], a1[4], a2[4], a3[4];
        const uint32_t lo = 0x0F0F0F0Fu;
        e2m1x8_to_f16x2x4((v[0][j] & lo) | (v[1][j] << 4 & ~lo), a0[0], a0[1], a0[2], a0[3]);
        e2m1x8_to_f16x2x4((v[0][j] >> 4 & lo) | (v[1][j] & ~lo), a1[0], a1[1], a1[2], a1[3]);
        e2m1x8_to_f16x2x4((v[2][j] & lo) | (v[3][j] << 4 & ~lo), a2[0], a2[1], a2[2], a2[3]);
        e2m1x8_to_f16x2x4((v[2][j] >> 4 & lo) | (v[3][j] & ~lo), a3[0], a3[1], a3[2], a3[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t b0 = hmul2(a0[e], s01[j / 2]), b1 = hmul2(a1[e], s01[j / 2]);
          const uint32_t b2 = hmul2(a2[e], s89[j / 2]), b3 = hmul2(a3[e], s89[j / 2]);
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            mma_f16(o[g][4 * j + e], b0, b1, b2, b3, p[g][h][0], p[g][h][1]);
            mma_f16(o[g][4 * j + e], b0, b1, b2, b3, rest[g][h][0], rest[g][h][1]);
          }
        }
      }
    }
  };

  // the products of step i + 1 beside the values of step i
  if (n_sub > 0) {
    cp_async_wait<ST - 2>();
    __syncwarp();
    products(ring);
    weigh(0);
    uint32_t at = 0, to = (ST - 1) * S::kStageBytes;   // stage of step i; of step i + ST - 1
    constexpr uint32_t END = ST * S::kStageBytes;
    for (int i = 0; i + 1 < n_sub; ++i) {
      // these copies go into the stage whose values the last turn added
      __syncwarp();
      fetch(i + ST - 1, to);
      look_up(i + ST);
      to = to + S::kStageBytes == END ? 0 : to + S::kStageBytes;
      const uint32_t next = at + S::kStageBytes == END ? 0 : at + S::kStageBytes;
      cp_async_wait<ST - 2>();
      __syncwarp();
      products(ring + next);
      add_values(ring + at);
      weigh(i + 1);
      at = next;
    }
    add_values(ring + at);
  }
  cp_async_wait<0>();
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const float2 n = unpair(less[g]), w = unpair(sum[g]);
    m[g][0] = bar[g][0] == -INFINITY ? -INFINITY : -n.x;
    m[g][1] = bar[g][1] == -INFINITY ? -INFINITY : -n.y;
    l[g][0] = w.x;
    l[g][1] = w.y;
  }
}

}  // namespace ftmoe
