// C ABI of the decode block's operators: argument checks and dispatch. Every check runs on the
// host before anything is enqueued.
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/ft_moe.h"
#include "ftmoe_internal.h"
#include "ftmoe_layout.h"

using namespace ftmoe;

namespace {

constexpr int kMaxLinearK = 32768;
constexpr int kMaxLinearN = 1 << 30;
constexpr int kMaxHeads = 1024;
constexpr int kMaxAppend = 1 << 20;
constexpr int kMaxGather = 1 << 26;
constexpr int kMaxNormH = 16384;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

ft_status check_cache(const ft_paged_kv* c) {
  if (!c || c->num_pages < 1 || c->page_size < 1 || c->Hkv < 1 || !c->k || !c->v)
    return FT_ERR_INVALID_ARG;
  if (c->dtype != FT_KV_BF16 && c->dtype != FT_KV_E4M3) return FT_ERR_INVALID_ARG;
  if (!(c->k_scale > 0.f) || !(c->v_scale > 0.f) || !std::isfinite(c->k_scale) ||
      !std::isfinite(c->v_scale) || !std::isfinite(1.f / c->k_scale) ||
      !std::isfinite(1.f / c->v_scale))
    return FT_ERR_INVALID_ARG;
  if ((c->D != 64 && c->D != 128 && c->D != 256) || c->Hkv > kMaxHeads)
    return FT_ERR_UNSUPPORTED_SHAPE;
  const int64_t unit = c->dtype == FT_KV_E4M3 ? 16 : 8;   // elements of 16 bytes
  const int64_t strides[6] = {c->k_page_stride, c->k_slot_stride, c->k_head_stride,
                              c->v_page_stride, c->v_slot_stride, c->v_head_stride};
  for (int64_t s : strides) {
    if (s < 0) return FT_ERR_INVALID_ARG;
    if (s % unit != 0) return FT_ERR_MISALIGNED;
  }
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return FT_ERR_MISALIGNED;
  return FT_OK;
}

// An NVFP4 cache as the library's launches take it. Checks everything but what the call's own sizes decide.
ft_status nvfp4_cache(const ft_nvfp4_kv* c, ft_paged_kv& kv, KvScales& sc) {
  if (!c || c->num_pages < 1 || c->page_size < 1 || c->Hkv < 1 || !c->k || !c->v || !c->k_scales || !c->v_scales)
    return FT_ERR_INVALID_ARG;
  for (float g : {c->k_gscale, c->v_gscale})   // 1 / (6 g) and every 1 / (e4m3 * g) stay normal floats
    if (!(g >= 0x1p-100f) || !(g <= 0x1p100f)) return FT_ERR_INVALID_ARG;
  if ((c->D != 64 && c->D != 128 && c->D != 256) || c->Hkv > kMaxHeads) return FT_ERR_UNSUPPORTED_SHAPE;
  const int64_t codes[6] = {c->k_page_stride, c->k_slot_stride, c->k_head_stride,
                            c->v_page_stride, c->v_slot_stride, c->v_head_stride};
  const int64_t scales[6] = {c->ks_page_stride, c->ks_slot_stride, c->ks_head_stride,
                             c->vs_page_stride, c->vs_slot_stride, c->vs_head_stride};
  const int row = c->D / 16;   // bytes of a head's scales
  for (int i = 0; i < 6; ++i) {
    if (codes[i] < 0 || scales[i] < 0) return FT_ERR_INVALID_ARG;
    if (codes[i] % 16 != 0 || scales[i] % row != 0) return FT_ERR_MISALIGNED;
  }
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scales, row) || !aligned(c->v_scales, row))
    return FT_ERR_MISALIGNED;
  kv = {c->k, c->v, c->num_pages, c->page_size, c->Hkv, c->D, codes[0], codes[1], codes[2],
        codes[3], codes[4], codes[5], kKvNvfp4, c->k_gscale, c->v_gscale};
  sc = {c->k_scales, c->v_scales, scales[0], scales[1], scales[2], scales[3], scales[4], scales[5]};
  return FT_OK;
}

// ft_kv_append for a checked cache (a.kv, and a.sc of an NVFP4 one).
ft_status append(AppendArgs& a, const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride,
                 const uint16_t* q, int64_t q_stride, uint16_t* q_out, int32_t T, int32_t Hq,
                 const int32_t* block_table, int32_t B, int32_t table_width, const int32_t* seq_ids,
                 const int32_t* positions, const float* rope, int32_t rope_rows, int32_t rope_dim,
                 const ft_rope_axes* axes, void* workspace, void* stream) {
  if (T < 0 || Hq < 0 || B < 0 || table_width < 0 || rope_dim < 0 || rope_rows < 0)
    return FT_ERR_INVALID_ARG;
  const bool f4 = a.kv.dtype == kKvNvfp4;
  if (T > kMaxAppend || Hq > kMaxHeads || rope_dim % (f4 ? 32 : 16) != 0 || rope_dim > a.kv.D)
    return FT_ERR_UNSUPPORTED_SHAPE;
  if (axes && rope_dim > 0) {
    if (axes->axes < 1 || axes->axes > 4 || axes->stride < 0) return FT_ERR_INVALID_ARG;
    for (int i = 0; i < rope_dim / 2; ++i) {
      if (axes->axis[i] >= axes->axes) return FT_ERR_INVALID_ARG;
      a.axis_of[i / 16] |= (uint32_t)axes->axis[i] << 2 * (i % 16);
    }
  }
  if (T == 0) return FT_OK;
  if (!k || !v || (B > 0 && table_width > 0 && !block_table) || !positions || (Hq > 0 && (!q || !q_out)) ||
      (rope_dim > 0 && (!rope || (axes && !axes->positions))) || (!seq_ids && T > B))
    return FT_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || (Hq > 0 && (!aligned(q, 16) || !aligned(q_out, 16))) ||
      k_stride % 8 != 0 || v_stride % 8 != 0 || (Hq > 0 && q_stride % 8 != 0) ||
      !aligned(block_table, 4) || !aligned(seq_ids, 4) || !aligned(positions, 4) ||
      (rope_dim > 0 && (!aligned(rope, 16) || (axes && !aligned(axes->positions, 4)))) ||
      !aligned(workspace, 256))
    return FT_ERR_MISALIGNED;
  a.k = k; a.v = v; a.q = q;
  a.k_stride = k_stride; a.v_stride = v_stride; a.q_stride = q_stride;
  a.q_out = q_out; a.T = T; a.Hq = Hq;
  a.inv_k = 1.0f / (f4 ? 6.0f * a.kv.k_scale : a.kv.k_scale);
  a.inv_v = 1.0f / (f4 ? 6.0f * a.kv.v_scale : a.kv.v_scale);
  a.block_table = block_table; a.seq_ids = seq_ids; a.positions = positions;
  a.B = B; a.table_width = table_width;
  a.rope = rope; a.rope_rows = rope_rows; a.rope_dim = rope_dim;
  if (axes && rope_dim > 0) {
    a.axis_pos = axes->positions; a.axis_stride = axes->stride; a.axes = axes->axes;
  }
  a.err = static_cast<int*>(workspace);
  return cuda_status(launch_kv_append(a, static_cast<cudaStream_t>(stream)));
}

// ft_kv_gather for a checked cache.
ft_status gather(GatherArgs& a, const int32_t* block_table, int32_t B, int32_t table_width,
                 const int32_t* seq_ids, const int32_t* positions, int32_t T, uint16_t* k_out,
                 uint16_t* v_out, void* workspace, void* stream) {
  if (T < 0 || B < 0 || table_width < 0) return FT_ERR_INVALID_ARG;
  if (T > kMaxGather) return FT_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return FT_OK;
  if ((B > 0 && table_width > 0 && !block_table) || !positions || !k_out || !v_out || (!seq_ids && T > B))
    return FT_ERR_INVALID_ARG;
  if (!aligned(block_table, 4) || !aligned(seq_ids, 4) || !aligned(positions, 4) || !aligned(k_out, 32) ||
      !aligned(v_out, 32) || !aligned(workspace, 256))
    return FT_ERR_MISALIGNED;
  a.block_table = block_table; a.B = B; a.table_width = table_width;
  a.seq_ids = seq_ids; a.positions = positions; a.T = T;
  a.k_out = k_out; a.v_out = v_out;
  a.err = static_cast<int*>(workspace);
  return cuda_status(launch_kv_gather(a, static_cast<cudaStream_t>(stream)));
}

// ft_paged_decode_attention for a checked cache.
ft_status attend(AttendArgs& a, const uint16_t* q, int64_t q_stride, int32_t B, int32_t Hq,
                 const int32_t* block_table, int32_t table_width, const int32_t* seq_lens, float scale,
                 int32_t window, uint16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                 void* stream) {
  if (B < 0 || Hq < 1 || Hq % a.kv.Hkv != 0 || table_width < 0 || window < 0 || !std::isfinite(scale))
    return FT_ERR_INVALID_ARG;
  if (B > kMaxSeqs || Hq > kMaxHeads) return FT_ERR_UNSUPPORTED_SHAPE;
  if (B == 0) return FT_OK;
  if (!q || (table_width > 0 && !block_table) || !seq_lens || !out || !workspace) return FT_ERR_INVALID_ARG;
  if (!aligned(q, 16) || q_stride % 8 != 0 || !aligned(out, 16) || !aligned(lse, 4) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(workspace, 256))
    return FT_ERR_MISALIGNED;
  if (workspace_bytes < AttendLayout(a.kv.D, 1).total) return FT_ERR_WORKSPACE_TOO_SMALL;
  const int sms = device_sms();
  if (sms <= 0) return FT_ERR_CUDA;
  const AttendLayout L(a.kv.D, sms);
  if (workspace_bytes < L.total) return FT_ERR_WORKSPACE_TOO_SMALL;
  char* ws = static_cast<char*>(workspace);
  a.q = q; a.q_stride = q_stride; a.B = B; a.Hq = Hq;
  a.block_table = block_table; a.seq_lens = seq_lens; a.table_width = table_width;
  a.scale = scale; a.window = window; a.out = out; a.lse = lse;
  a.err = reinterpret_cast<int*>(ws);
  a.shared_segs = reinterpret_cast<int4*>(ws + L.segs);
  a.part_ml = reinterpret_cast<float*>(ws + L.ml);
  a.part_o = reinterpret_cast<float*>(ws + L.o);
  return cuda_status(launch_attend(a, sms, static_cast<cudaStream_t>(stream)));
}

size_t norm_bwd_workspace(int T, int H, int sms) {
  return 1024 + align_up((size_t)norm_bwd_groups(T, sms) * 3 * H * sizeof(float), 256);
}

ft_status check_norm(const uint16_t* y, const void* residual, const uint16_t* w_post,
                     const uint16_t* w_pre, const uint16_t* gate, int32_t gate_kind, int32_t T,
                     int32_t H, float scale, float eps) {
  if (T < 0 || H < 1 || gate_kind < FT_GATE_NONE || gate_kind > FT_GATE_ELEMENT ||
      !std::isfinite(scale) || !(eps >= 0.f) || !std::isfinite(eps))
    return FT_ERR_INVALID_ARG;
  if (H % 8 != 0 || H > kMaxNormH) return FT_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return FT_OK;
  if (!y || (gate_kind != FT_GATE_NONE && !gate)) return FT_ERR_INVALID_ARG;
  if (!aligned(y, 16) || !aligned(residual, 16) || !aligned(w_post, 16) || !aligned(w_pre, 16) ||
      (gate_kind != FT_GATE_NONE && !aligned(gate, gate_kind == FT_GATE_TOKEN ? 2 : 16)))
    return FT_ERR_MISALIGNED;
  return FT_OK;
}

}  // namespace

extern "C" {

size_t ft_nvfp4_linear_workspace_bytes(int32_t T, int32_t K) {
  if (T < 1 || T > kMaxDecodeT || K < 32 || K % 32 != 0 || K > kMaxLinearK) return 0;
  if (T <= kLinearFew) return 0;
  const int sms = device_sms();
  return sms > 0 ? LinearLayout(T, K, sms).total : 0;
}

ft_status ft_nvfp4_linear(const uint16_t* x, int32_t T, int64_t x_stride,
                          const ft_nvfp4_matrix* w, void* out, int32_t out_f32, void* workspace,
                          size_t workspace_bytes, void* stream) {
  if (!w || T < 0 || w->N < 1 || w->K < 1) return FT_ERR_INVALID_ARG;
  if (T > kMaxDecodeT || w->K % 32 != 0 || w->K > kMaxLinearK || w->N > kMaxLinearN)
    return FT_ERR_UNSUPPORTED_SHAPE;
  if (!w->codes || !w->scales || !w->gscale) return FT_ERR_INVALID_ARG;
  if (!aligned(w->codes, 16) || !aligned(w->scales, 2) || !aligned(w->gscale, 4))
    return FT_ERR_MISALIGNED;
  if (T == 0) return FT_OK;
  if (!x || !out || (T > 1 && x_stride < w->K)) return FT_ERR_INVALID_ARG;
  if (!aligned(x, 16) || x_stride % 8 != 0 || !aligned(out, out_f32 ? 4 : 2))
    return FT_ERR_MISALIGNED;
  if (T > kLinearFew) {
    if (!workspace) return FT_ERR_INVALID_ARG;
    if (!aligned(workspace, 256)) return FT_ERR_MISALIGNED;
    if (workspace_bytes < LinearLayout(T, w->K, 1).total) return FT_ERR_WORKSPACE_TOO_SMALL;
  }
  const int sms = device_sms();
  if (sms <= 0) return FT_ERR_CUDA;
  const LinearLayout L(T, w->K, sms);
  if (workspace_bytes < L.total) return FT_ERR_WORKSPACE_TOO_SMALL;
  LinearArgs a = {};
  if (L.total > 0) {
    char* ws = static_cast<char*>(workspace);
    a.err = reinterpret_cast<int*>(ws);
    a.xdown = reinterpret_cast<float*>(ws + L.xdown);
    a.xh = reinterpret_cast<uint16_t*>(ws + L.xh);
    a.part = reinterpret_cast<float*>(ws + L.part);
  }
  a.x = x; a.x_stride = x_stride; a.T = T; a.N = w->N; a.K = w->K;
  a.codes = w->codes; a.scales = w->scales; a.gscale = w->gscale;
  a.out = out; a.out_f32 = out_f32 ? 1 : 0;
  return cuda_status(launch_linear(a, sms, static_cast<cudaStream_t>(stream)));
}

ft_status ft_kv_append_axes(const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride,
                            const uint16_t* q, int64_t q_stride, uint16_t* q_out, int32_t T,
                            int32_t Hq, const ft_paged_kv* cache, const int32_t* block_table,
                            int32_t B, int32_t table_width, const int32_t* seq_ids,
                            const int32_t* positions, const float* rope, int32_t rope_rows,
                            int32_t rope_dim, const ft_rope_axes* axes, void* workspace, void* stream) {
  AppendArgs a = {};
  const ft_status st = check_cache(cache);
  if (st != FT_OK) return st;
  a.kv = *cache;
  return append(a, k, k_stride, v, v_stride, q, q_stride, q_out, T, Hq, block_table, B, table_width, seq_ids,
                positions, rope, rope_rows, rope_dim, axes, workspace, stream);
}

ft_status ft_kv_append(const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride,
                       const uint16_t* q, int64_t q_stride, uint16_t* q_out, int32_t T,
                       int32_t Hq, const ft_paged_kv* cache, const int32_t* block_table,
                       int32_t B, int32_t table_width, const int32_t* seq_ids,
                       const int32_t* positions, const float* rope, int32_t rope_rows,
                       int32_t rope_dim, void* workspace, void* stream) {
  return ft_kv_append_axes(k, k_stride, v, v_stride, q, q_stride, q_out, T, Hq, cache, block_table, B,
                           table_width, seq_ids, positions, rope, rope_rows, rope_dim, nullptr, workspace,
                           stream);
}

ft_status ft_nvfp4_kv_append(const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride,
                             const uint16_t* q, int64_t q_stride, uint16_t* q_out, int32_t T,
                             int32_t Hq, const ft_nvfp4_kv* cache, const int32_t* block_table,
                             int32_t B, int32_t table_width, const int32_t* seq_ids,
                             const int32_t* positions, const float* rope, int32_t rope_rows,
                             int32_t rope_dim, const ft_rope_axes* axes, void* workspace, void* stream) {
  AppendArgs a = {};
  const ft_status st = nvfp4_cache(cache, a.kv, a.sc);
  if (st != FT_OK) return st;
  return append(a, k, k_stride, v, v_stride, q, q_stride, q_out, T, Hq, block_table, B, table_width, seq_ids,
                positions, rope, rope_rows, rope_dim, axes, workspace, stream);
}

ft_status ft_kv_gather(const ft_paged_kv* cache, const int32_t* block_table, int32_t B,
                       int32_t table_width, const int32_t* seq_ids, const int32_t* positions, int32_t T,
                       uint16_t* k_out, uint16_t* v_out, void* workspace, void* stream) {
  GatherArgs a = {};
  const ft_status st = check_cache(cache);
  if (st != FT_OK) return st;
  a.kv = *cache;
  return gather(a, block_table, B, table_width, seq_ids, positions, T, k_out, v_out, workspace, stream);
}

ft_status ft_nvfp4_kv_gather(const ft_nvfp4_kv* cache, const int32_t* block_table, int32_t B,
                             int32_t table_width, const int32_t* seq_ids, const int32_t* positions,
                             int32_t T, uint16_t* k_out, uint16_t* v_out, void* workspace, void* stream) {
  GatherArgs a = {};
  const ft_status st = nvfp4_cache(cache, a.kv, a.sc);
  if (st != FT_OK) return st;
  return gather(a, block_table, B, table_width, seq_ids, positions, T, k_out, v_out, workspace, stream);
}

size_t ft_paged_attention_workspace_bytes(int32_t B, int32_t D) {
  if (B < 1 || B > kMaxSeqs || (D != 64 && D != 128 && D != 256)) return 0;
  const int sms = device_sms();
  return sms > 0 ? AttendLayout(D, sms).total : 0;
}

ft_status ft_paged_decode_attention(const uint16_t* q, int64_t q_stride, int32_t B, int32_t Hq,
                                    const ft_paged_kv* cache, const int32_t* block_table,
                                    int32_t table_width, const int32_t* seq_lens, float scale,
                                    int32_t window, uint16_t* out, float* lse, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  AttendArgs a = {};
  const ft_status st = check_cache(cache);
  if (st != FT_OK) return st;
  a.kv = *cache;
  return attend(a, q, q_stride, B, Hq, block_table, table_width, seq_lens, scale, window, out, lse, workspace,
                workspace_bytes, stream);
}

ft_status ft_nvfp4_paged_decode_attention(const uint16_t* q, int64_t q_stride, int32_t B, int32_t Hq,
                                          const ft_nvfp4_kv* cache, const int32_t* block_table,
                                          int32_t table_width, const int32_t* seq_lens, float scale,
                                          int32_t window, uint16_t* out, float* lse, void* workspace,
                                          size_t workspace_bytes, void* stream) {
  AttendArgs a = {};
  const ft_status st = nvfp4_cache(cache, a.kv, a.sc);
  if (st != FT_OK) return st;
  // the kernel's offsets of rows are 32 bits of 16-byte pieces of codes, and of rows of scales
  const auto spans = [&](int64_t page_stride, int64_t slot_stride, int64_t head_stride, int64_t unit) {
    const auto far = [&](int64_t n, int64_t stride) { return (double)(n - 1) * (double)(stride / unit); };
    return far(cache->num_pages, page_stride) + far(cache->page_size, slot_stride) + far(cache->Hkv, head_stride) <
           4294967296.0;
  };
  if (!spans(cache->k_page_stride, cache->k_slot_stride, cache->k_head_stride, 16) ||
      !spans(cache->v_page_stride, cache->v_slot_stride, cache->v_head_stride, 16) ||
      !spans(cache->ks_page_stride, cache->ks_slot_stride, cache->ks_head_stride, cache->D / 16) ||
      !spans(cache->vs_page_stride, cache->vs_slot_stride, cache->vs_head_stride, cache->D / 16))
    return FT_ERR_UNSUPPORTED_SHAPE;
  return attend(a, q, q_stride, B, Hq, block_table, table_width, seq_lens, scale, window, out, lse, workspace,
                workspace_bytes, stream);
}

ft_status ft_residual_norm(const uint16_t* y, const void* residual, const uint16_t* w_post,
                           const uint16_t* w_pre, const uint16_t* gate, int32_t gate_kind,
                           int32_t T, int32_t H, int32_t res_f32, float scale, float eps,
                           void* r_out, uint16_t* x_out, void* stream) {
  ft_status st = check_norm(y, residual, w_post, w_pre, gate, gate_kind, T, H, scale, eps);
  if (st != FT_OK || T == 0) return st;
  if ((w_pre && !x_out) || (!w_pre && !r_out)) return FT_ERR_INVALID_ARG;
  if (!aligned(r_out, 16) || (w_pre && !aligned(x_out, 16))) return FT_ERR_MISALIGNED;
  NormArgs a = {};
  a.y = y; a.r = residual; a.w_post = w_post; a.w_pre = w_pre; a.gate = gate;
  a.gate_kind = gate_kind; a.T = T; a.H = H; a.res_f32 = res_f32 ? 1 : 0;
  a.scale = scale; a.eps = eps; a.r_out = r_out; a.x_out = x_out;
  const int sms = device_sms();
  if (sms <= 0) return FT_ERR_CUDA;
  return cuda_status(launch_norm(a, sms, static_cast<cudaStream_t>(stream)));
}

size_t ft_residual_norm_backward_workspace_bytes(int32_t T, int32_t H) {
  if (T < 0 || H < 8 || H % 8 != 0 || H > kMaxNormH) return 0;
  const int sms = device_sms();
  if (sms <= 0) return 0;
  return norm_bwd_workspace(T, H, sms);
}

ft_status ft_residual_norm_backward(const uint16_t* y, const void* residual,
                                    const uint16_t* w_post, const uint16_t* w_pre,
                                    const uint16_t* gate, int32_t gate_kind, const void* d_r,
                                    const uint16_t* d_x, int32_t T, int32_t H, int32_t res_f32,
                                    float scale, float eps, uint16_t* dy, void* dresidual,
                                    float* dw_post, float* dw_pre, void* dgate, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  ft_status st = check_norm(y, residual, w_post, w_pre, gate, gate_kind, T, H, scale, eps);
  if (st != FT_OK) return st;
  if ((w_post && !dw_post) || (w_pre && !dw_pre) ||
      (gate_kind == FT_GATE_CHANNEL && !dgate))
    return FT_ERR_INVALID_ARG;
  if ((w_post && !aligned(dw_post, 16)) || (w_pre && !aligned(dw_pre, 16)) ||
      (gate_kind != FT_GATE_NONE && !aligned(dgate, gate_kind == FT_GATE_TOKEN ? 4 : 16)))
    return FT_ERR_MISALIGNED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) {   // sums over no rows
    const size_t n = (size_t)H * sizeof(float);
    if (w_post && (st = cuda_status(cudaMemsetAsync(dw_post, 0, n, s))) != FT_OK) return st;
    if (w_pre && (st = cuda_status(cudaMemsetAsync(dw_pre, 0, n, s))) != FT_OK) return st;
    if (gate_kind == FT_GATE_CHANNEL) return cuda_status(cudaMemsetAsync(dgate, 0, n, s));
    return FT_OK;
  }
  if (!dy || !dresidual || (w_pre && !d_x) || (gate_kind != FT_GATE_NONE && !dgate) || !workspace)
    return FT_ERR_INVALID_ARG;
  if (!aligned(workspace, 256) || !aligned(dy, 16) || !aligned(dresidual, 16) || !aligned(d_r, 16) ||
      (w_pre && !aligned(d_x, 16)))
    return FT_ERR_MISALIGNED;
  if (workspace_bytes < norm_bwd_workspace(T, H, 1)) return FT_ERR_WORKSPACE_TOO_SMALL;
  NormArgs a = {};
  a.nq = (w_post ? 1 : 0) + (w_pre ? 1 : 0) + (gate_kind == FT_GATE_CHANNEL ? 1 : 0);
  const int sms = device_sms();
  if (sms <= 0) return FT_ERR_CUDA;
  if (workspace_bytes < norm_bwd_workspace(T, H, sms)) return FT_ERR_WORKSPACE_TOO_SMALL;
  a.err = static_cast<int*>(workspace);
  a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + 1024);
  a.y = y; a.r = residual; a.w_post = w_post; a.w_pre = w_pre; a.gate = gate;
  a.gate_kind = gate_kind; a.T = T; a.H = H; a.res_f32 = res_f32 ? 1 : 0;
  a.scale = scale; a.eps = eps; a.dr = d_r; a.dx = w_pre ? d_x : nullptr; a.dy = dy; a.dres = dresidual;
  a.dw_post = dw_post; a.dw_pre = dw_pre; a.dgate = dgate;
  return cuda_status(launch_norm_bwd(a, sms, s));
}

}  // extern "C"
