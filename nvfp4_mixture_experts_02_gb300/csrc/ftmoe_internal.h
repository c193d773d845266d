// Internal declarations shared by the library's translation units (not part of the ABI).
#pragma once

#include <atomic>
#include <cuda_runtime.h>
#include <cstdint>

#include "../../include/ft_moe.h"
#include "ftmoe_layout.h"

namespace ftmoe {

// FT_ERR_CUDA for a failed runtime call, with the error kept for ft_moe_last_cuda_error
// (FT_OK for cudaSuccess). Every runtime call whose failure an entry point returns goes
// through it.
ft_status cuda_status(cudaError_t e);

// The bound of a decode kernel's waits on other CTAs: `dflt` unless the test hook
// ft_moe_debug_set_wait_limit set one.
unsigned wait_limit(unsigned dflt);

// Host checks of a layer call's arguments (experts, shared expert, T, k, limit, pointers
// and their alignment; ws must be non-null and 256-byte aligned when T > 0). Enqueues
// nothing; FT_OK or the first failure.
ft_status check_layer_args(const uint16_t* x, int32_t T, const int32_t* topk_idx,
                           const float* topk_w, int32_t k, const ft_nvfp4_experts* ex,
                           const ft_nvfp4_shared_expert* sh, float limit, const uint16_t* out,
                           const void* ws);

cudaError_t launch_route(const float* logits, int T, int E, int k, int* idx, float* w,
                         cudaStream_t stream);

// Router logits W_router x_t [T][E] and, when gate is not null, the gate dots x_t . gv [T]
// (router.cu).
cudaError_t launch_router(const uint16_t* x, int T, int H, const uint16_t* w_router, int E,
                          const uint16_t* gate, float* logits, float* gate_dot,
                          cudaStream_t stream);

struct ExpertPtrs {
  int E, H, I;
  const uint8_t *w13, *s13;
  const float* g13;
  const uint8_t *w2, *s2;
  const float* g2;
  // shared expert (all null when absent)
  const uint8_t *sh_w13, *sh_s13, *sh_w2, *sh_s2;
  const float *sh_g13, *sh_g2;
  const uint16_t* sh_gate;
};

// logits != null (T = 1 only): the kernel routes the token itself (topk_idx / topk_w are
// then ignored) and CTA 0 writes the slots to topk_idx_out / topk_w_out when not null.
cudaError_t launch_decode(const uint16_t* x, int T, const int* topk_idx, const float* topk_w,
                          int k, const ExpertPtrs& ex, float limit, uint16_t* out, void* ws,
                          int num_sms, cudaStream_t stream, const float* logits = nullptr,
                          int* topk_idx_out = nullptr, float* topk_w_out = nullptr);

// The one-token kernel (decode1.cu) for a workspace laid out by DecodeLayout with t1 set.
cudaError_t launch_decode1(const uint16_t* x, const int* topk_idx, const float* topk_w, int k,
                           const ExpertPtrs& ex, float limit, float hscale, uint16_t* out,
                           void* ws, const DecodeLayout& WL, int grid, unsigned spin_limit,
                           cudaStream_t stream, const float* logits, int* topk_idx_out,
                           float* topk_w_out);

// Workspace regions of the prefill path (byte offsets, 256-byte aligned).
struct PrefillLayout {
  int max_pairs = 0, max_groups = 0;
  size_t err = 0, hdr = 0, act_expert = 0, act_pair0 = 0, group_act = 0, group_p0 = 0,
         group_n = 0, pair_tok = 0, pair_w = 0, pair_slot = 0, xf = 0, xscale = 0, h = 0,
         part = 0, e_pair0 = 0, e_ratio = 0, e_fill = 0, total = 0;
  PrefillLayout(int T, int k, int E, int H, int I, bool shared);
};

cudaError_t launch_prefill(const uint16_t* x, int T, const int* topk_idx, const float* topk_w,
                           int k, const ExpertPtrs& ex, float limit, uint16_t* out, void* ws,
                           int num_sms, cudaStream_t stream);

// Block-FP8 routed experts (fp8block.cu): E4M3 codes [rows][K] and float32 scales per
// 128 x 128 tile [ceil(rows/128)][ceil(K/128)], per expert; the shared expert likewise.
struct F8Ptrs {
  int E, H, I;
  const uint8_t *w13, *w2;
  const float *s13, *s2;
  const uint8_t *sh_w13, *sh_w2;   // null without a shared expert
  const float *sh_s13, *sh_s2;
  const uint16_t* sh_gate;
};

// Workspace regions of the block-FP8 decode (byte offsets, 256-byte aligned).
struct F8Layout {
  int P = 0;   // (token, slot) pairs, then one pair per token for the shared expert
  size_t err = 0, xf = 0, xscale = 0, gdot = 0, h = 0, part = 0, total = 0;
  F8Layout(int T, int k, int H, int I, bool shared);
};

cudaError_t launch_f8_decode(const uint16_t* x, int T, const int* topk_idx, const float* topk_w,
                             int k, const F8Ptrs& ex, float limit, uint16_t* out, void* ws,
                             int num_sms, cudaStream_t stream);

// Dense NVFP4 matrix times 1 to 64 tokens (linear.cu).
struct LinearArgs {
  const uint16_t* x;       // [T][x_stride] bf16
  int64_t x_stride;
  int T, N, K;
  const uint8_t *codes, *scales;
  const float* gscale;
  void* out;               // [T][N] bf16 or float
  int out_f32;
  int* err;                // workspace: error word, x's powers of two [T], x as f16, partial tiles
  float* xdown;
  uint16_t* xh;
  float* part;
  int split;               // blocks of a cluster that share K (set by the launch)
  unsigned wait_rounds;    // of a wait for x (set by the launch)
};
// Workspace regions (byte offsets, 256-byte aligned): none for the calls that lay x out themselves.
constexpr int kLinearFew = 8;   // tokens up to which they do
struct LinearLayout {
  size_t xdown = 0, xh = 0, part = 0, total = 0;
  LinearLayout(int T, int K, int num_sms) {
    if (T <= kLinearFew) return;
    const size_t width = (T + 15) / 16 * 16;
    xdown = 1024;
    xh = xdown + 256;   // 64 floats
    part = xh + width * (align_up(K, 256) * 2);
    total = part + (size_t)num_sms * 4 * width * 256 * 4;   // two blocks an SM, two pieces each
  }
};
cudaError_t launch_linear(const LinearArgs& a, int num_sms, cudaStream_t stream);

// j / d for 0 <= j < 2^31 as (umulhi(mul, j) + j) >> shift.
inline void page_division(int d, int& mul, int& shift) {
  shift = 0;
  while ((1ll << shift) < d) ++shift;
  mul = (int)(uint32_t)(((1ull << 32) * ((1ull << shift) - (uint64_t)d)) / (uint64_t)d + 1);
}

// An NVFP4 cache inside the library: ft_paged_kv with strides and offsets of the codes in bytes, gscale for
// scale and this dtype, and its block scales.
constexpr int kKvNvfp4 = 2;
struct KvScales {
  uint8_t *k, *v;
  int64_t k_page, k_slot, k_head, v_page, v_slot, v_head;   // strides in bytes
};

// Rotary embedding and cache append (kv.cu). err: error word or null.
struct AppendArgs {
  const uint16_t *k, *v, *q;
  int64_t k_stride, v_stride, q_stride;   // elements between tokens
  uint16_t* q_out;
  int T, Hq;
  ft_paged_kv kv;
  float inv_k, inv_v;
  const int *block_table, *seq_ids, *positions;
  int B, table_width;
  const float* rope;
  int rope_rows, rope_dim;
  int* err;
  int div_mul, div_shift;   // division by the page size (set by the launch)
  KvScales sc;              // NVFP4: inv_k, inv_v are 1 / (6 gscale)
  const int* axis_pos;      // several rotary axes: positions [axes], axis_stride apart, or null
  int64_t axis_stride;
  int axes;
  uint32_t axis_of[8];      // the axis of each pair, two bits each
};
cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t stream);

// Cached tokens as dense bf16 (kv.cu).
struct GatherArgs {
  ft_paged_kv kv;
  KvScales sc;
  const int *block_table, *seq_ids, *positions;
  int B, table_width, T;
  uint16_t *k_out, *v_out;
  int* err;
  int div_mul, div_shift;   // division by the page size (set by the launch)
};
cudaError_t launch_kv_gather(const GatherArgs& a, cudaStream_t stream);

// Paged attention of one new token per sequence (attention.cu).
struct AttendArgs {
  const uint16_t* q;
  int64_t q_stride;
  int B, Hq;
  ft_paged_kv kv;
  const int *block_table, *seq_lens;
  int table_width;
  float scale;
  int window;
  uint16_t* out;
  float* lse;
  int* err;                // workspace: error word, shared segments [run], pieces' (max, sum) and sums
  int4* shared_segs;
  float *part_ml, *part_o;
  int group, gt;           // query heads per key head, 16-head parts of them (set by the launch)
  int same_strides;        // keys and values lie alike (set by the launch)
  int div_mul, div_shift;  // division by the page size (set by the launch)
  int max_len;             // slots of a row of the block table, or what the call can count (set by the launch)
  int heads_log2;          // log2 of the key heads that a block may take at once (set by the launch)
  KvScales sc;             // NVFP4
};
// Workspace regions (byte offsets, 256-byte aligned), for kAttendBlocks blocks and attend_warps warps an SM
// at most, two pieces each, 16 query heads a piece.
constexpr int kAttendBlocks = 3;
constexpr int attend_warps(int D) { return D == 64 ? 16 : D == 128 ? 12 : 8; }
struct AttendLayout {
  size_t segs = 0, ml = 0, o = 0, total = 0;
  AttendLayout(int D, int num_sms) {
    segs = 1024;
    const size_t rows = (size_t)num_sms * attend_warps(D) * 2 * 16;
    ml = align_up(segs + (size_t)num_sms * kAttendBlocks * 16, 256);
    o = align_up(ml + rows * 2 * 4, 256);
    total = align_up(o + rows * D * 4, 256);
  }
};
cudaError_t launch_attend(const AttendArgs& a, int num_sms, cudaStream_t stream);

// Norms around a gated residual sum, and the gradient (norm.cu).
struct NormArgs {
  const uint16_t* y;
  const void* r;           // bf16 or float (res_f32), or null
  const uint16_t *w_post, *w_pre, *gate;
  int T, H, gate_kind, res_f32;
  float scale, eps;
  void* r_out;             // forward
  uint16_t* x_out;
  const void* dr;          // backward
  const uint16_t* dx;
  uint16_t* dy;
  void* dres;
  float *dw_post, *dw_pre;
  void* dgate;             // float [H] / [T], bf16 [T][H]
  int* err;                // workspace: error word, column sums [block][nq][H]
  float* part;
  int nq;
};
// Blocks (rows of the workspace's partial sums) of the backward pass.
int norm_bwd_groups(int T, int num_sms);
cudaError_t launch_norm(const NormArgs& a, int num_sms, cudaStream_t stream);
cudaError_t launch_norm_bwd(const NormArgs& a, int num_sms, cudaStream_t stream);

// SM count of the current device (0: no device).
int device_sms();

// Lets a kernel take up to `bytes` of dynamic shared memory, once per device (`done`: one flag per device
// and kernel; setting it twice is harmless).
struct SmemGrant {
  std::atomic<bool> done[64];
};
template <typename K>
cudaError_t grant_smem(SmemGrant& grant, K kernel, int bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (grant.done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) grant.done[dev].store(true, std::memory_order_relaxed);
  return e;
}

}  // namespace ftmoe
