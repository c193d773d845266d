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
// Every input is read once and every output written once; the work is bound by memory, with float32
// sums in a fixed order, and x' taken from r' before r' is rounded to its stored type. k_norm: a row per
// block, per warp (up to 512 elements) or per 8 or 16 lanes (up to 64 or 128, the heads of q and k) in
// registers. k_norm_rows (wide rows, many of them) and k_norm_bwd: persistent blocks whose row groups get
// their rows by bulk copies into rings, so that the next rows travel while one is worked on;
// k_norm_bwd_narrow: rows of up to 256 elements by 8 to 32 lanes each. The gradient's column sums stay in
// registers over all of a block's rows; k_norm_cols adds the blocks' sums.
//
// Measured (of the copy rate of 6786 GB/s): forward 8191 x 4096 with a float32 stream 72 us (82 %), 8192 x
// 8192 93 us (85 %), 131072 x 128 22 us (89 %; a warp per row 50); gradient 8192 x 8192 170 us (70 %), where
// about half of a row's 3 us is arithmetic (9 unpackings and 9 packed operations an element) and two
// barriers; 131072 x 128 43 us (70 %; rows of a warp through rings 121), 262144 x 64 42 us (234), 65536 x 256
// 43 us (64); 2048 x 16384 168 us (35 %: 32 columns a thread spill). One token: 2.9 us, a launch and three
// dependent latencies.
#include <cuda_runtime.h>

#include "ftmoe_internal.h"
#include "ftmoe_mma.cuh"
#include "ftmoe_tc.cuh"

namespace ftmoe {

namespace {

constexpr int kWarpRowMax = 512;    // elements of a row that one warp holds
constexpr int kNarrowRowMax = 256;  // ... with one 8-element piece a lane, or several rows a warp
constexpr int kRowThreads = 256;    // of a block in those forms

// 1 / sqrt(sum / n + eps) and scale * gate times it, as a float and what it lacks: where r and the
// block's output nearly cancel, r' keeps the error of this factor many times over. inv_n + inv_n_lo is
// 1 / n.
struct Factor {
  float hi, lo, root;
};
__device__ __forceinline__ Factor row_factor(float sum, float inv_n, float inv_n_lo, float eps,
                                             float scale, float gate, bool norm) {
  const float tg = scale * gate, tg_lo = fmaf(scale, gate, -tg);
  if (!norm) return {tg, tg_lo, 1.f};
  const float mean = sum * inv_n, mean_lo = fmaf(sum, inv_n_lo, fmaf(sum, inv_n, -mean));
  const float v = mean + eps, from = v - mean;
  const float v_lo = (mean - (v - from)) + (eps - from) + mean_lo;
  const float s = rsqrtf(v), t = v * s;
  float left = fmaf(-t, s, 1.f);   // 1 - (v + v_lo) s^2
  left = fmaf(-fmaf(v, s, -t), s, left);
  left = fmaf(-v_lo * s, s, left);
  const float s_lo = s > 0.f ? 0.5f * s * left : 0.f, hi = tg * s;   // 0: the sum has overflowed
  return {hi, fmaf(tg, s, -hi) + fmaf(tg, s_lo, tg_lo * s), s + s_lo};
}

// Sum over groups of GS lanes.
template <int GS>
__device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
  for (int o = GS / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the row's threads: GS lanes of a warp, or (GS = 0) the whole block through red[] (one array per
// call site, so that one barrier per sum is enough).
template <int GS>
__device__ __forceinline__ float row_sum(float v, float* red) {
  if constexpr (GS > 0) return lane_sum<GS>(v);
  v = warp_sum(v);
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

// A row per GS lanes, or (GS = 0) per block.
template <int NV, typename RT, int GS>
__global__ void __launch_bounds__(GS > 0 ? kRowThreads : 1024) k_norm(const NormArgs a) {
  __shared__ float red[2][32];
  griddep_launch_dependents();
  griddep_wait();
  constexpr int G = GS > 0 ? GS : 32;
  const int tid = GS > 0 ? threadIdx.x % G : threadIdx.x;
  const int nth = GS > 0 ? GS : blockDim.x;
  const int64_t t = GS > 0 ? (int64_t)blockIdx.x * (kRowThreads / G) + threadIdx.x / G : blockIdx.x;
  if (GS > 0 && GS < 32 ? t - (int)(threadIdx.x % 32) / G >= a.T : t >= a.T) return;   // a whole warp or block
  const int chunks = t < a.T ? a.H >> 3 : 0;   // none in a warp's rows past the last
  const size_t row = (size_t)t * a.H;
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
  if (a.w_post) s1 = rsqrtf(row_sum<GS>(ss, red[0]) * inv_h + a.eps);
  const float ts = a.scale * (a.gate_kind == FT_GATE_TOKEN && chunks > 0 ? one_bf16(a.gate + t) : 1.f) * s1;
  ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = tid + i * nth;
    if (c >= chunks) continue;
    float w[8], g[8];
    if (a.w_post) {   // y times the weight and the gate, all bf16, is exact in float32
      cached8(a.w_post + 8 * c, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[i][j] *= w[j];
    }
    if (a.gate_kind == FT_GATE_CHANNEL || a.gate_kind == FT_GATE_ELEMENT) {
      if (a.gate_kind == FT_GATE_CHANNEL) cached8(a.gate + 8 * c, g);
      else load8(a.gate + row + 8 * c, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[i][j] *= g[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      r[i][j] = fmaf(ts, y[i][j], r[i][j]);
      ss = fmaf(r[i][j], r[i][j], ss);
    }
    if (a.r_out) store8(static_cast<RT*>(a.r_out) + row + 8 * c, r[i]);
  }
  if (!a.w_pre) return;
  const float s2 = rsqrtf(row_sum<GS>(ss, red[1]) * inv_h + a.eps);
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

// The gradient. A block of 512 threads is RG row groups of GT threads, 8 NV columns per thread; a group's
// rows come whole by bulk copies into its ring of stages, so that the next rows travel while one is worked
// on. A row's values are read from shared memory where they are used; r', h and the column sums stay in
// registers. Two barriers a row: the sum that y needs is taken for the next row together with the last
// sums of this one.
constexpr int kRingThreads = 512;
constexpr size_t kRingBytes = 224 * 1024;   // one stage of the widest rows: 16384, float32, every input

struct RowRing {   // a stage: y | r | dr | dx | gate rows (dr, dx: the gradient's), those that there are
  int stage = 0, off_r = 0, off_dr = 0, off_dx = 0, off_gate = 0, stages = 0;
  uint32_t rounds = wait_limit(kWaitRounds);   // of a wait for a row
  RowRing(const NormArgs& a, int groups, size_t bytes) {
    const int res = a.H * (a.res_f32 ? 4 : 2);
    off_r = 2 * a.H;
    off_dr = off_r + (a.r ? res : 0);
    off_dx = off_dr + (a.dr ? res : 0);
    off_gate = off_dx + (a.dx ? 2 * a.H : 0);
    stage = off_gate + (a.gate_kind == FT_GATE_ELEMENT ? 2 * a.H : 0);
    stages = (int)(bytes / ((size_t)groups * stage));
    if (stages > 8) stages = 8;
  }
};

// One thread: the copies of row t into a stage. The stage's parts say what is copied, so that its barrier
// expects what comes.
__device__ __forceinline__ void send_row(const NormArgs& a, const RowRing& ring, uint64_t* bar, unsigned char* st,
                                         int t) {
  asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}" ::
                   "r"(smem_addr(bar)), "r"(ring.stage) : "memory");
  auto copy = [&](int off, int end, const void* src) {
    if (off == end) return;
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes "
                 "[%0], [%1], %2, [%3];" ::"r"(smem_addr(st + off)),
                 "l"(static_cast<const char*>(src) + (size_t)t * (end - off)), "r"(end - off),
                 "r"(smem_addr(bar)) : "memory");
  };
  copy(0, ring.off_r, a.y);
  copy(ring.off_r, ring.off_dr, a.r);
  copy(ring.off_dr, ring.off_dx, a.dr);
  copy(ring.off_dx, ring.off_gate, a.dx);
  copy(ring.off_gate, ring.stage, a.gate);
}

// What a row group keeps in shared memory beside its ring.
template <typename V, int W>
struct RowGroup {
  V red[2][W];        // the warps' sums, two arrays in turn
  uint64_t full[8];   // a stage's row has arrived
  int lost, sent;     // a wait has run out; rows sent
};

// A row's wait. One that runs out (only a copy that never lands would let it) sets lost: the group sends no
// more, its later waits are one poll each, and before its block leaves, one thread waits for what the group's
// last copies still bring, so that no copy comes to shared memory that is someone else's. The rare part is a
// function of its own: inside the loops it costs registers that they spill (8192 x 2048 gradient, float32
// stream, 56.4 us for 52.0).
__device__ __noinline__ bool row_late(uint64_t* bar, uint32_t parity, uint32_t rounds, volatile int* lost, int* err) {
  for (uint32_t it = 0; it < rounds && !*lost; ++it)
    if (mbar_poll(bar, parity)) return true;
  *lost = 1;
  if (err) atomicOr(err, kErrTimeout);
  return false;
}
template <typename G>
__device__ __forceinline__ bool row_arrived(G& grp, int i, int stages, uint32_t rounds, int* err) {
  uint64_t* bar = &grp.full[i % stages];
  const uint32_t parity = (uint32_t)(i / stages) & 1u;
  return (rounds > 0 && mbar_poll(bar, parity)) || row_late(bar, parity, rounds, &grp.lost, err);
}
template <typename G>
__device__ __forceinline__ void drain_rows(G& grp, int stages) {
  for (int i = grp.sent > stages ? grp.sent - stages : 0; i < grp.sent; ++i)
    mbar_wait(&grp.full[i % stages], (uint32_t)(i / stages) & 1u, nullptr, 0);
}

// Two float32 in one 64-bit register pair: half the arithmetic instructions (packed operations round
// each half as the scalar ones do).
using f2 = unsigned long long;
__device__ __forceinline__ f2 make2(float lo, float hi) {
  f2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ f2 both(float v) { return make2(v, v); }
__device__ __forceinline__ float2 split2(f2 v) {
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(v));
  return d;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float sum_of(f2 v) {
  const float2 x = split2(v);
  return x.x + x.y;
}
__device__ __forceinline__ void open8(const uint4& v, f2 (&f)[4]) {
  f[0] = make2(bf16_lo(v.x), bf16_hi(v.x));
  f[1] = make2(bf16_lo(v.y), bf16_hi(v.y));
  f[2] = make2(bf16_lo(v.z), bf16_hi(v.z));
  f[3] = make2(bf16_lo(v.w), bf16_hi(v.w));
}
// Eight values of column piece c from a row in shared memory.
__device__ __forceinline__ void get8(const unsigned char* row, int c, const uint16_t*, f2 (&f)[4]) {
  open8(reinterpret_cast<const uint4*>(row)[c], f);
}
__device__ __forceinline__ void get8(const unsigned char* row, int c, const float*, f2 (&f)[4]) {
  const ulonglong2* p = reinterpret_cast<const ulonglong2*>(row) + 2 * c;
  const ulonglong2 u = p[0], v = p[1];
  f[0] = u.x; f[1] = u.y; f[2] = v.x; f[3] = v.y;
}
__device__ __forceinline__ void put8(uint16_t* p, const f2 (&f)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 v = split2(f[j]);
    w[j] = pack_bf16(v.x, v.y);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void put8(float* p, const f2 (&f)[4]) {
  reinterpret_cast<ulonglong2*>(p)[0] = make_ulonglong2(f[0], f[1]);
  reinterpret_cast<ulonglong2*>(p)[1] = make_ulonglong2(f[2], f[3]);
}

// Many rows: the row groups and rings of the gradient. One barrier a row: the sum over r' for x' and the
// one over the next row's y are taken together, and the row's stage is free once it is passed.
template <int GT, int NV, typename RT>
__global__ void __launch_bounds__(kRingThreads, NV == 2 ? 2 : 1)
    k_norm_rows(const NormArgs a, const RowRing ring) {
  constexpr int RG = kRingThreads / GT, W = GT / 32;
  extern __shared__ __align__(128) unsigned char ring_smem[];
  __shared__ __align__(16) RowGroup<float2, W> groups[RG];
  RowGroup<float2, W>& grp = groups[threadIdx.x / GT];
  const int g = threadIdx.x / GT, tid = threadIdx.x % GT, warp = tid >> 5, lane = tid & 31;
  const int chunks = a.H >> 3, ST = ring.stages;
  const float inv_h = 1.0f / (float)a.H;
  const bool channel = a.gate_kind == FT_GATE_CHANNEL, element = a.gate_kind == FT_GATE_ELEMENT;
  const bool post = a.w_post != nullptr, pre = a.w_pre != nullptr;
  const RT* const kind = nullptr;
  if (tid < ST) mbar_init(&grp.full[tid], 1);
  if (tid == 0) {
    grp.lost = grp.sent = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  griddep_launch_dependents();
  griddep_wait();
  unsigned char* const mine = ring_smem + (size_t)g * ST * ring.stage;
  const int t0 = blockIdx.x + g * gridDim.x, dt = RG * gridDim.x;   // rows of this group: t0, t0 + dt, ...
  const int n_rows = t0 < a.T ? (a.T - t0 + dt - 1) / dt : 0;
  auto send = [&](int i) {   // one thread: the copies of row i into stage i % ST
    send_row(a, ring, &grp.full[i % ST], mine + (size_t)(i % ST) * ring.stage, t0 + i * dt);
  };
  auto sum2 = [&](int which, float x, float y) -> float2 {   // two sums over the group's threads
    x = warp_sum(x);
    y = warp_sum(y);
    if (lane == 0) grp.red[which][warp] = make_float2(x, y);
    asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "n"(GT) : "memory");
    float2 v = grp.red[which][lane % W];
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) {
      v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
      v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    return v;
  };
  // this thread's columns of w_post and w_pre
  const uint4 one = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
  uint4 wpost[NV], wpre[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = tid + v * GT;
    wpost[v] = post && c < chunks ? *reinterpret_cast<const uint4*>(a.w_post + 8 * c) : one;
    wpre[v] = pre && c < chunks ? *reinterpret_cast<const uint4*>(a.w_pre + 8 * c) : one;
  }
  auto square_sum = [&](const unsigned char* st) -> float {   // of this thread's part of y
    f2 ss = 0ull;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = tid + v * GT;
      if (c >= chunks) continue;
      f2 y[4];
      get8(st, c, a.y, y);
#pragma unroll
      for (int j = 0; j < 4; ++j) ss = fma2(y[j], y[j], ss);
    }
    return sum_of(ss);
  };
  auto y_sum = [&](int i) -> float {   // waits for row i; NaN if it does not come
    if (!row_arrived(grp, i, ST, ring.rounds, nullptr)) return __int_as_float(0x7FC00000);
    return post ? square_sum(mine + (size_t)(i % ST) * ring.stage) : 0.f;
  };

  if (n_rows == 0) return;   // a whole group: its barriers are its own
  if (tid == 0) {
    grp.sent = min(ST, n_rows);
    for (int i = 0; i < ST && i < n_rows; ++i) send(i);
  }
  float ss = sum2(1, y_sum(0), 0.f).x;
  for (int i = 0; i < n_rows; ++i) {
    const int t = t0 + i * dt;
    const size_t row = (size_t)t * a.H;
    const unsigned char* st = mine + (size_t)(i % ST) * ring.stage;
    const float s1 = post ? rsqrtf(ss * inv_h + a.eps) : 1.f + ss;
    const f2 ts = both(a.scale * (a.gate_kind == FT_GATE_TOKEN ? one_bf16(a.gate + t) : 1.f) * s1);
    f2 r[NV][4], rr = 0ull;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = tid + v * GT;
#pragma unroll
      for (int j = 0; j < 4; ++j) r[v][j] = 0ull;
      if (c >= chunks) continue;
      f2 y[4], w[4];
      get8(st, c, a.y, y);
      if (a.r) get8(st + ring.off_r, c, kind, r[v]);
      open8(wpost[v], w);   // y times the weight and the gate, all bf16, is exact in float32
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = mul2(y[j], w[j]);
      if (element || channel) {
        if (element) get8(st + ring.off_gate, c, a.gate, w);
        else open8(*reinterpret_cast<const uint4*>(a.gate + 8 * c), w);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = mul2(y[j], w[j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        r[v][j] = fma2(y[j], ts, r[v][j]);
        rr = fma2(r[v][j], r[v][j], rr);
      }
      if (a.r_out) put8(static_cast<RT*>(a.r_out) + row + 8 * c, r[v]);
    }
    const float next = i + 1 < n_rows ? y_sum(i + 1) : 0.f;
    const float2 sums = sum2(i & 1, sum_of(rr), next);
    ss = sums.y;
    if (tid == 0 && i + ST < n_rows && !grp.lost) {   // every thread has read the row
      send(i + ST);
      grp.sent = i + ST + 1;
    }
    if (!pre) continue;
    const f2 s2 = both(rsqrtf(sums.x * inv_h + a.eps));
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = tid + v * GT;
      if (c >= chunks) continue;
      f2 w[4];
      open8(wpre[v], w);
#pragma unroll
      for (int j = 0; j < 4; ++j) r[v][j] = mul2(r[v][j], mul2(w[j], s2));
      put8(a.x_out + row + 8 * c, r[v]);
    }
  }
  if (tid == 0 && grp.lost) drain_rows(grp, ST);
}

// With u = w_post * (channel gate), tg = scale * (token gate) and e the elementwise gate:
//   r' = r + (tg s1) y u e     h = tg dr' u e     dy = s1 (h - y s1^2 mean(h y))
//   A = sum_t tg s1 y dr' e    dw_post = A * (channel gate), dgate = A * w_post (channel: tg = scale)
//   dgate = scale s1 sum_h y u dr' (token),  scale s1 y u dr' (element)
// so one column sum serves both the weight and the channel's gate.
template <int GT, int NV, typename RT>
__global__ void __launch_bounds__(kRingThreads, 1) k_norm_bwd(const NormArgs a, const RowRing ring) {
  constexpr int RG = kRingThreads / GT, W = GT / 32;
  extern __shared__ __align__(128) unsigned char bwd_smem[];
  __shared__ __align__(16) RowGroup<float4, W> groups[RG];
  RowGroup<float4, W>& grp = groups[threadIdx.x / GT];
  const int g = threadIdx.x / GT, tid = threadIdx.x % GT, warp = tid >> 5, lane = tid & 31;
  const int chunks = a.H >> 3, ST = ring.stages;
  const bool ahead = ST >= 3;   // stages enough to look at the next row's y within this one
  const float inv_h = 1.0f / (float)a.H, inv_h_lo = fmaf(-inv_h, (float)a.H, 1.f) * inv_h;
  const bool channel = a.gate_kind == FT_GATE_CHANNEL, element = a.gate_kind == FT_GATE_ELEMENT;
  const bool post = a.w_post != nullptr, pre = a.w_pre != nullptr;
  const RT* const kind = nullptr;
  if (tid < ST) mbar_init(&grp.full[tid], 1);
  if (tid == 0) {
    grp.lost = grp.sent = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  griddep_launch_dependents();
  griddep_wait();
  unsigned char* const mine = bwd_smem + (size_t)g * ST * ring.stage;
  // rows of this group: t0, t0 + dt, ...
  const int t0 = blockIdx.x + g * gridDim.x, dt = RG * gridDim.x;
  const int n_rows = t0 < a.T ? (a.T - t0 + dt - 1) / dt : 0;
  auto send = [&](int i) {   // one thread: the copies of row i into stage i % ST
    send_row(a, ring, &grp.full[i % ST], mine + (size_t)(i % ST) * ring.stage, t0 + i * dt);
  };
  auto barrier = [&]() {
    if constexpr (GT == 32) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "n"(GT) : "memory");
  };
  // two sums over the group's threads (two arrays in turn: one barrier each)
  auto sum2 = [&](int which, float x, float y) -> float2 {
    x = warp_sum(x);
    y = warp_sum(y);
    if (lane == 0) grp.red[which][warp] = make_float4(x, y, 0.f, 0.f);
    barrier();
    float4 v = grp.red[which][lane % W];
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) {
      v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
      v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    return make_float2(v.x, v.y);
  };
  // this thread's columns: u in float32, w_pre packed
  f2 u[NV][4], acc_post[NV][4], acc_pre[NV][4];
  uint4 wpre[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = tid + v * GT;
    const uint4 one = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
    f2 gt[4];
    open8(post && c < chunks ? *reinterpret_cast<const uint4*>(a.w_post + 8 * c) : one, u[v]);
    open8(channel && c < chunks ? *reinterpret_cast<const uint4*>(a.gate + 8 * c) : one, gt);
    wpre[v] = pre && c < chunks ? *reinterpret_cast<const uint4*>(a.w_pre + 8 * c) : one;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u[v][j] = mul2(u[v][j], gt[j]);
      acc_post[v][j] = acc_pre[v][j] = 0ull;
    }
  }
  auto square_sum = [&](const unsigned char* st) -> float {   // of this thread's part of y
    f2 ss = 0ull;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = tid + v * GT;
      if (c >= chunks) continue;
      f2 y[4];
      get8(st, c, a.y, y);
#pragma unroll
      for (int j = 0; j < 4; ++j) ss = fma2(y[j], y[j], ss);
    }
    return sum_of(ss);
  };
  auto arrived = [&](int i) {
    row_arrived(grp, i, ST, ring.rounds, a.err);   // one that does not come is flagged
  };

  if (tid == 0) {
    grp.sent = min(ST, n_rows);
    for (int i = 0; i < ST && i < n_rows; ++i) send(i);
  }
  float ss = 0.f;   // of the coming row's y, already summed
  if (n_rows > 0 && ahead) {
    arrived(0);
    ss = sum2(0, square_sum(mine), 0.f).x;
    barrier();   // red[] is written again within the first row
  }
  for (int i = 0; i < n_rows; ++i) {
    const int t = t0 + i * dt;
    const size_t row = (size_t)t * a.H;
    const unsigned char* st = mine + (size_t)(i % ST) * ring.stage;
    // once every thread is past the row before this one its stage takes a new row
    auto refill = [&]() {
      if (ST > 1 && tid == 0 && i > 0 && i - 1 + ST < n_rows && !grp.lost) {
        send(i - 1 + ST);
        grp.sent = i + ST;
      }
    };
    if (!ahead) {
      arrived(i);
      ss = sum2(0, square_sum(st), 0.f).x;
      refill();
      barrier();
    }
    const float tgate = a.gate_kind == FT_GATE_TOKEN ? one_bf16(a.gate + t) : 1.f, tg = a.scale * tgate;
    const Factor factor = row_factor(ss, inv_h, inv_h_lo, a.eps, a.scale, tgate, post);
    const float s1 = factor.root;
    const f2 ts = both(factor.hi), ts_lo = both(factor.lo);
    // r' and the sums that x' needs
    f2 r[NV][4], rr = 0ull, dot = 0ull;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = tid + v * GT;
#pragma unroll
      for (int j = 0; j < 4; ++j) r[v][j] = 0ull;
      if (c >= chunks) continue;
      f2 y[4], w[4], d[4];
      get8(st, c, a.y, y);
      if (a.r) get8(st + ring.off_r, c, kind, r[v]);
      if (element) {
        get8(st + ring.off_gate, c, a.gate, w);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = mul2(y[j], w[j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {   // y u is exact
        const f2 yu = mul2(y[j], u[v][j]);
        r[v][j] = fma2(yu, ts_lo, fma2(yu, ts, r[v][j]));
      }
      if (pre) {
        get8(st + ring.off_dx, c, a.dx, d);
        open8(wpre[v], w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          rr = fma2(r[v][j], r[v][j], rr);
          dot = fma2(mul2(d[j], w[j]), r[v][j], dot);
        }
      }
    }
    f2 s2 = 0ull, cr = 0ull;
    if (pre) {
      const float2 v = sum2(1, sum_of(rr), sum_of(dot));
      const float s = rsqrtf(v.x * inv_h + a.eps);
      s2 = both(s);
      cr = both(-(s * (s * s * (v.y * inv_h))));
      if (ahead) refill();
    }
    f2 h[NV][4], hy = 0ull;   // h without tg
    const f2 gs = both(a.scale * s1);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = tid + v * GT;
#pragma unroll
      for (int j = 0; j < 4; ++j) h[v][j] = 0ull;
      if (c >= chunks) continue;
      f2 dr[4] = {0ull, 0ull, 0ull, 0ull}, d[4], w[4], y[4];
      if (a.dr) get8(st + ring.off_dr, c, kind, dr);
      if (pre) {
        get8(st + ring.off_dx, c, a.dx, d);
        open8(wpre[v], w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f2 ds = mul2(d[j], s2);
          acc_pre[v][j] = fma2(ds, r[v][j], acc_pre[v][j]);
          dr[j] = fma2(ds, w[j], fma2(r[v][j], cr, dr[j]));
        }
      }
      put8(static_cast<RT*>(a.dres) + row + 8 * c, dr);
      get8(st, c, a.y, y);
      if (element) {
        f2 dg[4];
        get8(st + ring.off_gate, c, a.gate, w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          dg[j] = mul2(mul2(mul2(y[j], dr[j]), u[v][j]), gs);
          dr[j] = mul2(dr[j], w[j]);
        }
        put8(static_cast<uint16_t*>(a.dgate) + row + 8 * c, dg);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f2 yd = mul2(y[j], dr[j]);
        acc_post[v][j] = fma2(yd, ts, acc_post[v][j]);
        hy = fma2(yd, u[v][j], hy);
        h[v][j] = mul2(dr[j], u[v][j]);
      }
    }
    float next = 0.f;
    if (ahead && i + 1 < n_rows) {
      arrived(i + 1);
      if (post) next = square_sum(mine + (size_t)((i + 1) % ST) * ring.stage);
    }
    const float2 sums = sum2(0, sum_of(hy), next);
    ss = sums.y;
    if (ahead && !pre) refill();
    if (a.gate_kind == FT_GATE_TOKEN && tid == 0)
      static_cast<float*>(a.dgate)[t] = a.scale * s1 * sums.x;
    // one factor s1 at a time: s1^3 leaves float32's range for rows of 1e13, or of 1e-13, already
    const f2 k1 = both(post ? tg * s1 : tg), k2 = both(post ? -(s1 * (s1 * (sums.x * inv_h))) : 0.f);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = tid + v * GT;
      if (c >= chunks) continue;
      if (post) {
        f2 y[4];
        get8(st, c, a.y, y);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[v][j] = mul2(fma2(y[j], k2, h[v][j]), k1);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) h[v][j] = mul2(h[v][j], k1);
      }
      put8(a.dy + row + 8 * c, h[v]);
    }
    if (ST == 1) {
      barrier();
      if (tid == 0 && i + 1 < n_rows && !grp.lost) {
        send(i + 1);
        grp.sent = i + 2;
      }
    } else if (!pre || !ahead) {
      barrier();   // red[0] is written again before another barrier of the next row
    }
  }

  if (tid == 0 && grp.lost) drain_rows(grp, ST);
  // the block's column sums, its groups added in order: [block][quantity][H]
  float* part = a.part + (size_t)blockIdx.x * a.nq * a.H;
  float* cols = reinterpret_cast<float*>(bwd_smem);   // [group][H], over the rings
  int q = 0;
#pragma unroll
  for (int which = 0; which < 3; ++which) {
    if (which == 0 ? !post : which == 1 ? !pre : !channel) continue;
    __syncthreads();
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = tid + v * GT;
      if (c >= chunks) continue;
      f2 sum[4], w[4];
      const uint4 one = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
      open8(which == 0 ? (channel ? *reinterpret_cast<const uint4*>(a.gate + 8 * c) : one)
            : which == 2 && post ? *reinterpret_cast<const uint4*>(a.w_post + 8 * c) : one, w);
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[j] = which == 1 ? acc_pre[v][j] : mul2(acc_post[v][j], w[j]);
      put8((RG > 1 ? cols + (size_t)g * a.H : part + (size_t)q * a.H) + 8 * c, sum);
    }
    if constexpr (RG > 1) {
      __syncthreads();
      for (int x = threadIdx.x; x < a.H; x += kRingThreads) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < RG; ++w) v += cols[(size_t)w * a.H + x];
        part[(size_t)q * a.H + x] = v;
      }
    }
    ++q;
  }
}

// Narrow rows (heads): a row per GS lanes, one 8-element piece a lane, the next row's inputs in registers
// while one is worked on; the sums are shuffles.
constexpr int kNarrowThreads = 512;
template <typename RT>
struct RowPiece {   // eight elements as they are stored
  static constexpr int Q = sizeof(RT) / 2;
  uint4 q[Q];
  __device__ __forceinline__ void load(const void* base, size_t at, bool on) {
#pragma unroll
    for (int i = 0; i < Q; ++i)
      q[i] = on && base ? ld16(static_cast<const char*>(base) + at * sizeof(RT) + 16 * i) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void open(f2 (&f)[4]) const {
    if constexpr (Q == 1) {
      open8(q[0], f);
    } else {
#pragma unroll
      for (int i = 0; i < Q; ++i) {
        f[2 * i] = make2(__uint_as_float(q[i].x), __uint_as_float(q[i].y));
        f[2 * i + 1] = make2(__uint_as_float(q[i].z), __uint_as_float(q[i].w));
      }
    }
  }
};
template <int GS, typename RT>
__global__ void __launch_bounds__(kNarrowThreads, 1) k_norm_bwd_narrow(const NormArgs a) {
  constexpr int RG = kNarrowThreads / GS;
  __shared__ __align__(16) float cols[RG * GS * 8];   // [group][H]
  griddep_launch_dependents();
  griddep_wait();
  const int g = threadIdx.x / GS, c = threadIdx.x % GS, chunks = a.H >> 3;
  const float inv_h = 1.0f / (float)a.H, inv_h_lo = fmaf(-inv_h, (float)a.H, 1.f) * inv_h;
  const bool channel = a.gate_kind == FT_GATE_CHANNEL, element = a.gate_kind == FT_GATE_ELEMENT;
  const bool post = a.w_post != nullptr, pre = a.w_pre != nullptr;
  const uint4 one = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
  const bool col = c < chunks;
  f2 u[4], wpre[4], acc_post[4], acc_pre[4], chan[4];
  open8(post && col ? *reinterpret_cast<const uint4*>(a.w_post + 8 * c) : one, u);
  open8(channel && col ? *reinterpret_cast<const uint4*>(a.gate + 8 * c) : one, chan);
  open8(pre && col ? *reinterpret_cast<const uint4*>(a.w_pre + 8 * c) : one, wpre);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    u[j] = mul2(u[j], chan[j]);
    acc_post[j] = acc_pre[j] = 0ull;
  }
  struct Row {
    RowPiece<uint16_t> y, dx, gate;
    RowPiece<RT> r, dr;
    float tgate;
  };
  auto load = [&](Row& w, int64_t t) {
    const bool on = col && t < a.T;
    const size_t at = (size_t)t * a.H + 8 * c;
    w.y.load(a.y, at, on);
    w.r.load(a.r, at, on);
    w.dr.load(a.dr, at, on);
    w.dx.load(pre ? a.dx : nullptr, at, on);
    w.gate.load(element ? a.gate : nullptr, at, on);
    w.tgate = a.gate_kind == FT_GATE_TOKEN && t < a.T ? one_bf16(a.gate + t) : 1.f;
  };
  const int step = (int)gridDim.x * RG;
  Row now;
  load(now, (int)blockIdx.x * RG + g);
  for (int64_t t0 = (int)blockIdx.x * RG; t0 < a.T; t0 += step) {   // uniform over the block
    const int64_t t = t0 + g;
    const bool on = col && t < a.T;
    const size_t at = (size_t)t * a.H + 8 * c;
    const Row w = now;
    load(now, t + step);
    f2 y[4], r[4], d[4], gate[4], ss = 0ull;
    w.y.open(y);
    w.r.open(r);
    if (post) {
#pragma unroll
      for (int j = 0; j < 4; ++j) ss = fma2(y[j], y[j], ss);
    }
    const Factor factor = row_factor(post ? lane_sum<GS>(sum_of(ss)) : 0.f, inv_h, inv_h_lo, a.eps, a.scale,
                                     w.tgate, post);
    const float s1 = factor.root, tg = a.scale * w.tgate;
    const f2 ts = both(factor.hi), ts_lo = both(factor.lo);
    w.gate.open(gate);
    w.dx.open(d);
    f2 rr = 0ull, dot = 0ull;
#pragma unroll
    for (int j = 0; j < 4; ++j) {   // y u is exact
      const f2 yu = mul2(element ? mul2(y[j], gate[j]) : y[j], u[j]);
      r[j] = fma2(yu, ts_lo, fma2(yu, ts, r[j]));
      rr = fma2(r[j], r[j], rr);
      dot = fma2(mul2(d[j], wpre[j]), r[j], dot);
    }
    f2 s2 = 0ull, cr = 0ull;
    if (pre) {
      const float sum = lane_sum<GS>(sum_of(rr)), with = lane_sum<GS>(sum_of(dot));
      const float s = rsqrtf(sum * inv_h + a.eps);
      s2 = both(s);
      cr = both(-(s * (s * s * (with * inv_h))));
    }
    f2 dr[4], h[4], hy = 0ull;
    w.dr.open(dr);
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = 0ull;
    if (on) {
      if (pre) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f2 ds = mul2(d[j], s2);
          acc_pre[j] = fma2(ds, r[j], acc_pre[j]);
          dr[j] = fma2(ds, wpre[j], fma2(r[j], cr, dr[j]));
        }
      }
      put8(static_cast<RT*>(a.dres) + at, dr);
      if (element) {
        const f2 gs = both(a.scale * s1);
        f2 dg[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          dg[j] = mul2(mul2(mul2(y[j], dr[j]), u[j]), gs);
          dr[j] = mul2(dr[j], gate[j]);
        }
        put8(static_cast<uint16_t*>(a.dgate) + at, dg);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f2 yd = mul2(y[j], dr[j]);
        acc_post[j] = fma2(yd, ts, acc_post[j]);
        hy = fma2(yd, u[j], hy);
        h[j] = mul2(dr[j], u[j]);
      }
    }
    const float sum = lane_sum<GS>(sum_of(hy));
    if (!on) continue;
    if (a.gate_kind == FT_GATE_TOKEN && c == 0) static_cast<float*>(a.dgate)[t] = a.scale * s1 * sum;
    const f2 k1 = both(post ? tg * s1 : tg), k2 = both(post ? -(s1 * (s1 * (sum * inv_h))) : 0.f);
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = mul2(post ? fma2(y[j], k2, h[j]) : h[j], k1);
    put8(a.dy + at, h);
  }
  // the block's column sums, its groups added in order: [block][quantity][H]
  float* part = a.part + (size_t)blockIdx.x * a.nq * a.H;
  int q = 0;
#pragma unroll
  for (int which = 0; which < 3; ++which) {
    if (which == 0 ? !post : which == 1 ? !pre : !channel) continue;
    __syncthreads();
    if (col) {
      f2 sum[4], w[4];
      open8(which == 0 && channel ? *reinterpret_cast<const uint4*>(a.gate + 8 * c)
            : which == 2 && post  ? *reinterpret_cast<const uint4*>(a.w_post + 8 * c) : one, w);
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[j] = which == 1 ? acc_pre[j] : mul2(acc_post[j], w[j]);
      put8(cols + (size_t)g * a.H + 8 * c, sum);
    }
    __syncthreads();
    for (int x = threadIdx.x; x < a.H; x += kNarrowThreads) {
      float v = 0.f;
#pragma unroll 8
      for (int w = 0; w < RG; ++w) v += cols[(size_t)w * a.H + x];
      part[(size_t)q * a.H + x] = v;
    }
    ++q;
  }
}

// The blocks' column sums in a fixed order: a block sums 64 columns (two per lane), its warps take the
// partial rows in turn, ten of them in flight (gradient of 509 x 4096 15.8 us; with 128 columns and five in
// flight 16.4).
constexpr int kColWarps = 16, kCols = 64;
__global__ void __launch_bounds__(kColWarps * 32) k_norm_cols(const NormArgs a, int parts) {
  __shared__ float2 sum[kColWarps][32];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = blockIdx.x * kCols + lane * 2;   // over nq * H columns, H a multiple of 8
  const int width = a.nq * a.H;
  float2 v = make_float2(0.f, 0.f);
  if (col < width) {
    constexpr int FLIGHT = 10;
    for (int p0 = warp; p0 < parts; p0 += FLIGHT * kColWarps) {
      float2 u[FLIGHT];
#pragma unroll
      for (int j = 0; j < FLIGHT; ++j) {
        const int p = p0 + j * kColWarps;
        u[j] = p < parts ? *reinterpret_cast<const float2*>(a.part + (size_t)p * width + col)
                         : make_float2(0.f, 0.f);
      }
#pragma unroll
      for (int j = 0; j < FLIGHT; ++j) {
        v.x += u[j].x;
        v.y += u[j].y;
      }
    }
  }
  sum[warp][lane] = v;
  __syncthreads();
  if (warp != 0 || col >= width) return;
#pragma unroll
  for (int w = 1; w < kColWarps; ++w) {
    const float2 u = sum[w][lane];
    v.x += u.x;
    v.y += u.y;
  }
  int q = col / a.H;
  const int h = col - q * a.H;
  float* const to[3] = {a.dw_post, a.dw_pre,
                        a.gate_kind == FT_GATE_CHANNEL ? static_cast<float*>(a.dgate) : nullptr};
  const bool on[3] = {a.w_post != nullptr, a.w_pre != nullptr, a.gate_kind == FT_GATE_CHANNEL};
  for (int which = 0; which < 3; ++which) {
    if (!on[which]) continue;
    if (q-- == 0) *reinterpret_cast<float2*>(to[which] + h) = v;
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

// Many rows by rings, two blocks an SM (one for the widest rows). ok: false when a ring of two stages
// does not fit.
template <int GT, int NV, typename RT>
cudaError_t launch_rows_t(const NormArgs& a, int num_sms, cudaStream_t stream, bool& ok) {
  constexpr int blocks = NV == 2 ? 2 : 1;
  const RowRing ring(a, kRingThreads / GT, kRingBytes / blocks);
  ok = ring.stages >= 2;
  if (!ok) return cudaSuccess;
  const size_t smem = (size_t)kRingThreads / GT * ring.stages * ring.stage;
  cudaError_t e;
  static SmemGrant grant;
  if ((e = grant_smem(grant, k_norm_rows<GT, NV, RT>, (int)kRingBytes)) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(blocks * num_sms));
  cfg.blockDim = dim3(kRingThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_norm_rows<GT, NV, RT>, a, ring);
}
template <int GT, int NV>
cudaError_t launch_rows(const NormArgs& a, int num_sms, cudaStream_t stream, bool& ok) {
  return a.res_f32 ? launch_rows_t<GT, NV, float>(a, num_sms, stream, ok)
                   : launch_rows_t<GT, NV, uint16_t>(a, num_sms, stream, ok);
}

template <int GT, int NV, typename RT>
cudaError_t launch_bwd_t(const NormArgs& a, int grid, cudaStream_t stream) {
  const RowRing ring(a, kRingThreads / GT, kRingBytes);
  const size_t sums = (size_t)kRingThreads / GT * a.H * 4;
  size_t smem = (size_t)kRingThreads / GT * ring.stages * ring.stage;
  if (GT < kRingThreads && smem < sums) smem = sums;
  cudaError_t e;
  static SmemGrant grant;
  if ((e = grant_smem(grant, k_norm_bwd<GT, NV, RT>, (int)kRingBytes)) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kRingThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_norm_bwd<GT, NV, RT>, a, ring);
}

template <int GT, int NV>
cudaError_t launch_bwd(const NormArgs& a, int grid, cudaStream_t stream) {
  return a.res_f32 ? launch_bwd_t<GT, NV, float>(a, grid, stream)
                   : launch_bwd_t<GT, NV, uint16_t>(a, grid, stream);
}

}  // namespace

int norm_bwd_groups(int T, int num_sms) { return T < num_sms ? T : num_sms; }

cudaError_t launch_norm(const NormArgs& a, int num_sms, cudaStream_t stream) {
  const int chunks = a.H / 8;
  // Rings for wide rows, from four rows a group on (us, one row a block or rings: 8192 x 8192 119 or 93,
  // 2048 x 16384 67 or 48; 8192 x 2048 27 either way, and narrower rows alike)
  if (chunks > 256 && (int64_t)a.T >= (int64_t)(chunks <= 512 ? 16 : chunks <= 1024 ? 8 : 4) * num_sms) {
    bool ok = false;
    const cudaError_t e = chunks <= 512    ? launch_rows<256, 2>(a, num_sms, stream, ok)
                          : chunks <= 1024 ? launch_rows<512, 2>(a, num_sms, stream, ok)
                                           : launch_rows<512, 4>(a, num_sms, stream, ok);
    if (ok || e != cudaSuccess) return e;
  }
  if (a.H <= kWarpRowMax) {
    const int gs = chunks <= 8 ? 8 : chunks <= 16 ? 16 : 32, rows = kRowThreads / gs;
    const int grid = (a.T - 1) / rows + 1;
    auto go = [&](auto kernel_f32, auto kernel_bf16) {
      return a.res_f32 ? launch(kernel_f32, grid, kRowThreads, stream, a)
                       : launch(kernel_bf16, grid, kRowThreads, stream, a);
    };
    if (a.H > kNarrowRowMax) return go(k_norm<2, float, 32>, k_norm<2, uint16_t, 32>);
    if (gs == 32) return go(k_norm<1, float, 32>, k_norm<1, uint16_t, 32>);
    if (gs == 16) return go(k_norm<1, float, 16>, k_norm<1, uint16_t, 16>);
    return go(k_norm<1, float, 8>, k_norm<1, uint16_t, 8>);
  }
  const int th = row_threads(chunks, 2);
  return a.res_f32 ? launch(k_norm<2, float, 0>, a.T, th, stream, a)
                   : launch(k_norm<2, uint16_t, 0>, a.T, th, stream, a);
}

cudaError_t launch_norm_bwd(const NormArgs& a, int num_sms, cudaStream_t stream) {
  const int chunks = a.H / 8;
  const int grid = norm_bwd_groups(a.T, num_sms);
  cudaError_t e;
  if (chunks <= 8) {
    e = a.res_f32 ? launch(k_norm_bwd_narrow<8, float>, grid, kNarrowThreads, stream, a)
                  : launch(k_norm_bwd_narrow<8, uint16_t>, grid, kNarrowThreads, stream, a);
  } else if (chunks <= 16) {
    e = a.res_f32 ? launch(k_norm_bwd_narrow<16, float>, grid, kNarrowThreads, stream, a)
                  : launch(k_norm_bwd_narrow<16, uint16_t>, grid, kNarrowThreads, stream, a);
  } else if (chunks <= 32) {
    e = a.res_f32 ? launch(k_norm_bwd_narrow<32, float>, grid, kNarrowThreads, stream, a)
                  : launch(k_norm_bwd_narrow<32, uint16_t>, grid, kNarrowThreads, stream, a);
  } else if (chunks <= 64) {
    e = launch_bwd<32, 2>(a, grid, stream);
  } else if (chunks <= 128) {
    e = launch_bwd<64, 2>(a, grid, stream);
  } else if (chunks <= 256) {
    e = launch_bwd<128, 2>(a, grid, stream);
  } else if (chunks <= 512) {
    e = launch_bwd<256, 2>(a, grid, stream);
  } else if (chunks <= 1024) {
    e = launch_bwd<512, 2>(a, grid, stream);
  } else {
    e = launch_bwd<512, 4>(a, grid, stream);
  }
  if (e != cudaSuccess || a.nq == 0) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.nq * a.H + kCols - 1) / kCols));
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
