// api_serving.hip -- the C ABI of include/moe_serving.h: host-side validation,
// workspace carving and kernel launches.  Every argument is checked before
// anything is enqueued; no call allocates, frees or synchronises.
#include "../../include/moe_serving.h"
#include "checks.hpp"

using namespace tre;

namespace {

static_assert(kFewTokens == MOE_FEW_MAX_TOKENS && kFewPairs == MOE_FEW_MAX_PAIRS, "limits of the few-token layer");

// Whether every address is a multiple of 16 (rows are read and written in
// 16-byte vectors; a NULL that reaches here is a missing workspace).
template <typename... P>
bool aligned16(const P*... p) {
  return ((((uintptr_t)p & 15) == 0) && ...);
}

// A row tile of 288 rows of 8-bit codes is addressed with 31 bits.
constexpr int32_t kMaxWidth = 1 << 22;

// E experts of widths d and I, whose gate/up weights are of `size` bytes an
// element: one expert's stay below 2 GiB, the reach of one buffer descriptor
// (2 for the calls that take weights in moe.h's layouts, which are refused
// where moe.h's calls refuse them, float32 or not; 1 for 8-bit codes).
moe_status check_layer(int32_t E, int32_t d, int32_t I, int32_t size) {
  TRY(check_experts(E));
  TRY(check_width(d));
  TRY(check_width(I));
  if (d >= kMaxWidth || I >= kMaxWidth) return MOE_ERR_UNSUPPORTED;
  if ((int64_t)E * d * 2 * I >= 8 * kMaxElems) return MOE_ERR_UNSUPPORTED;
  if ((int64_t)d * I * 2 * size >= kMaxElems) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Byte layout of the few-token workspace.
struct FewLayout {
  size_t h, part, counters, total;
};

FewLayout few_layout(int64_t T, int64_t d, int64_t k, int64_t I, size_t act, int split) {
  FewLayout L;
  size_t o = 0;
  L.h = o;        o += align256((size_t)(T * k * I) * act);
  L.part = o;     o += align256((size_t)split * (size_t)(T * k * d) * 4);
  L.counters = o; o += align256((size_t)few_counters((int)d) * 4);
  L.total = o;
  return L;
}

bool few_sizes_ok(int32_t T, int32_t d, int32_t E, int32_t k, int32_t I) {
  return T >= 0 && T <= kFewTokens && d >= 1 && E >= 1 && k >= 1 && I >= 1 && (int64_t)T * k <= kFewPairs;
}

moe_status check_few(const void* x, const float* logits, int32_t T, int32_t d, int32_t E, int32_t k, int32_t I,
                     int32_t size, const int32_t* topk_idx, const float* topk_w, const void* out) {
  if (T < 0 || k < 1) return MOE_ERR_ARG;
  TRY(check_layer(E, d, I, size));
  if (logits && k > E) return MOE_ERR_ARG;
  if (T > kFewTokens || (int64_t)T * k > kFewPairs) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || !topk_idx || !topk_w || !out) return MOE_ERR_ARG;
  return MOE_OK;
}

// Row scales of `cols` columns.
size_t scale_bytes(int64_t rows, int64_t cols) { return (size_t)(rows * ceil_div(cols, 128)) * 4; }

// Bytes between rows of 8-bit codes in a workspace: whole cache lines, where
// that keeps the array's offsets below 2^31 (the caller's own arrays are
// dense; 2880 columns are 22.5 lines, and every other row's loads then take
// two halves for each line: the 128-expert layer's products are 4% slower).
int row_bytes8(int64_t rows, int64_t cols) {
  const int64_t padded = round_up(cols, 128);
  return (int)(rows * padded < kMaxElems ? padded : cols);
}

// Byte layout of moe_grouped_ffn_fp8's workspace: h in codes and scales.
struct Ffn8Layout {
  size_t h_q, h_s, total;
};

Ffn8Layout ffn8_layout(int64_t rows, int64_t I) {
  Ffn8Layout L;
  size_t o = 0;
  L.h_q = o; o += align256((size_t)(rows * row_bytes8(rows, I)));
  L.h_s = o; o += align256(scale_bytes(rows, I));
  L.total = o;
  return L;
}

// Byte layout of moe_forward_fp8's workspace.
struct Forward8Layout {
  size_t x_q, x_s, pair_row, row_token, offsets, perm_ws, ffn, y, total;
};

Forward8Layout forward8_layout(int64_t T, int64_t d, int64_t E, int64_t k, int64_t I) {
  const int64_t P = T * k;
  Forward8Layout L;
  size_t o = 0;
  L.x_q = o;       o += align256((size_t)(T * row_bytes8(T, d)));
  L.x_s = o;       o += align256(scale_bytes(T, d));
  L.pair_row = o;  o += align256((size_t)P * 4);
  L.row_token = o; o += align256((size_t)P * 4);
  L.offsets = o;   o += align256((size_t)(E + 1) * 4);
  L.perm_ws = o;   o += permute_index_workspace(P, (int)E);
  L.ffn = o;       o += ffn8_layout(P, I).total;
  L.y = o;         o += align256((size_t)(P * d) * 2);
  L.total = o;
  return L;
}

moe_status check_rows8(int32_t max_rows, int32_t E, int32_t d, int32_t I) {
  if (max_rows < 0) return MOE_ERR_ARG;
  TRY(check_layer(E, d, I, 1));
  if ((int64_t)max_rows * (d > I ? d : I) >= kMaxElems) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

FewScratch carve_few(const FewLayout& L, void* workspace) {
  char* ws = (char*)workspace;
  return {ws + L.h, (float*)(ws + L.part), (int32_t*)(ws + L.counters)};
}

}  // namespace

extern "C" {

moe_status moe_quantize_rows(const void* x, moe_dtype dt, int32_t rows, int32_t cols, void* q, float* scale,
                             void* stream) {
  if (!dtype_ok(dt) || rows < 0) return MOE_ERR_ARG;
  TRY(check_width(cols));
  if ((int64_t)rows * cols >= kMaxElems) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!x || !q || !scale || !aligned16(x, q)) return MOE_ERR_ARG;
  hipStream_t s = (hipStream_t)stream;
  if (dt == MOE_BF16)
    return from_hip(launch_quantize_rows_bf16((const bf16_t*)x, rows, cols, (uint8_t*)q, cols, scale, s));
  return from_hip(launch_quantize_rows_f32((const float*)x, rows, cols, (uint8_t*)q, cols, scale, s));
}

moe_status moe_quantize_weights(const void* w_gate_up, const void* w_down, moe_dtype dt, int32_t E, int32_t d,
                                int32_t I, void* w_gate_up_q, float* w_gate_up_s, void* w_down_q, float* w_down_s,
                                void* stream) {
  if (!dtype_ok(dt)) return MOE_ERR_ARG;
  TRY(check_layer(E, d, I, 2));
  if (!w_gate_up || !w_down || !w_gate_up_q || !w_gate_up_s || !w_down_q || !w_down_s) return MOE_ERR_ARG;
  if (!aligned16(w_gate_up, w_down, w_gate_up_q, w_down_q)) return MOE_ERR_ARG;
  hipStream_t s = (hipStream_t)stream;
  if (dt == MOE_BF16)
    return from_hip(launch_quantize_weights_bf16((const bf16_t*)w_gate_up, (const bf16_t*)w_down, E, d, I,
                                                 (uint8_t*)w_gate_up_q, w_gate_up_s, (uint8_t*)w_down_q, w_down_s,
                                                 s));
  return from_hip(launch_quantize_weights_f32((const float*)w_gate_up, (const float*)w_down, E, d, I,
                                              (uint8_t*)w_gate_up_q, w_gate_up_s, (uint8_t*)w_down_q, w_down_s, s));
}

moe_status moe_gate_up_swiglu_fp8(const void* x_q, const float* x_s, const int32_t* expert_offsets, int32_t max_rows,
                                  int32_t E, int32_t d, int32_t I, const void* w_gate_up_q, const float* w_gate_up_s,
                                  const int32_t* row_token, int32_t x_rows, void* h_q, float* h_s, void* stream) {
  TRY(check_rows8(max_rows, E, d, I));
  if (row_token) {
    if (x_rows < 0) return MOE_ERR_ARG;
    if ((int64_t)x_rows * d >= kMaxElems) return MOE_ERR_UNSUPPORTED;
  }
  if (max_rows == 0) return MOE_OK;
  if (!expert_offsets || !w_gate_up_q || !w_gate_up_s || !h_q || !h_s) return MOE_ERR_ARG;
  if (!x_q || !x_s) return MOE_ERR_ARG;
  if (!aligned16(x_q, w_gate_up_q, h_q)) return MOE_ERR_ARG;
  return from_hip(launch_gate_up_fp8((const uint8_t*)x_q, d, x_s, expert_offsets, max_rows, E, d, I,
                                     (const uint8_t*)w_gate_up_q, w_gate_up_s, row_token, x_rows, (uint8_t*)h_q, I,
                                     h_s, (hipStream_t)stream));
}

moe_status moe_down_proj_fp8(const void* h_q, const float* h_s, const int32_t* expert_offsets, int32_t max_rows,
                             int32_t E, int32_t d, int32_t I, const void* w_down_q, const float* w_down_s,
                             void* y_perm, void* stream) {
  TRY(check_rows8(max_rows, E, d, I));
  if (max_rows == 0) return MOE_OK;
  if (!h_q || !h_s || !expert_offsets || !w_down_q || !w_down_s || !y_perm) return MOE_ERR_ARG;
  if (!aligned16(h_q, w_down_q, y_perm)) return MOE_ERR_ARG;
  return from_hip(launch_down_fp8((const uint8_t*)h_q, I, h_s, expert_offsets, max_rows, E, d, I,
                                  (const uint8_t*)w_down_q, w_down_s, (bf16_t*)y_perm, (hipStream_t)stream));
}

size_t moe_grouped_ffn_fp8_workspace_size(int32_t max_rows, int32_t I) {
  if (max_rows < 0 || I < 1) return 0;
  return ffn8_layout(max_rows, I).total;
}

moe_status moe_grouped_ffn_fp8(const void* x_q, const float* x_s, const int32_t* expert_offsets, int32_t max_rows,
                               int32_t E, int32_t d, int32_t I, const void* w_gate_up_q, const float* w_gate_up_s,
                               const void* w_down_q, const float* w_down_s, void* y_perm, void* workspace,
                               size_t workspace_bytes, void* stream) {
  TRY(check_rows8(max_rows, E, d, I));
  if (max_rows == 0) return MOE_OK;
  if (!w_gate_up_q || !w_gate_up_s || !w_down_q || !w_down_s || !y_perm || !x_q || !x_s || !expert_offsets)
    return MOE_ERR_ARG;
  if (!aligned16(x_q, w_gate_up_q, w_down_q, y_perm, workspace)) return MOE_ERR_ARG;
  const Ffn8Layout L = ffn8_layout(max_rows, I);
  if (!workspace || workspace_bytes < L.total) return MOE_ERR_WORKSPACE;
  char* ws = (char*)workspace;
  const int ldh = row_bytes8(max_rows, I);
  hipStream_t s = (hipStream_t)stream;
  TRY(from_hip(launch_gate_up_fp8((const uint8_t*)x_q, d, x_s, expert_offsets, max_rows, E, d, I,
                                  (const uint8_t*)w_gate_up_q, w_gate_up_s, nullptr, 0, (uint8_t*)(ws + L.h_q), ldh,
                                  (float*)(ws + L.h_s), s)));
  return from_hip(launch_down_fp8((const uint8_t*)(ws + L.h_q), ldh, (const float*)(ws + L.h_s), expert_offsets,
                                  max_rows, E, d, I, (const uint8_t*)w_down_q, w_down_s, (bf16_t*)y_perm, s));
}

size_t moe_forward_fp8_workspace_size(int32_t T, int32_t d, int32_t E, int32_t k, int32_t I) {
  if (T < 0 || d < 1 || E < 1 || k < 1 || I < 1) return 0;
  return forward8_layout(T, d, E, k, I).total;
}

moe_status moe_forward_fp8(const void* x, const float* logits, int32_t T, int32_t d, int32_t E, int32_t k, int32_t I,
                           const void* w_gate_up_q, const float* w_gate_up_s, const void* w_down_q,
                           const float* w_down_s, int32_t* topk_idx, float* topk_w, int32_t* expert_offsets,
                           int32_t* row_token, int32_t* pair_row, void* out, void* workspace, size_t workspace_bytes,
                           void* stream) {
  if (T < 0 || k < 1) return MOE_ERR_ARG;
  TRY(check_layer(E, d, I, 1));
  if (logits && k > E) return MOE_ERR_ARG;
  const int64_t P = (int64_t)T * k;
  if (P * (d > I ? d : I) >= kMaxElems || (int64_t)T * E >= kMaxElems) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || !w_gate_up_q || !w_gate_up_s || !w_down_q || !w_down_s || !topk_idx || !topk_w || !out) return MOE_ERR_ARG;
  if (!aligned16(x, w_gate_up_q, w_down_q, out, workspace)) return MOE_ERR_ARG;
  const Forward8Layout L = forward8_layout(T, d, E, k, I);
  if (!workspace || workspace_bytes < L.total) return MOE_ERR_WORKSPACE;
  char* ws = (char*)workspace;
  uint8_t* x_q = (uint8_t*)(ws + L.x_q);
  float* x_s = (float*)(ws + L.x_s);
  int32_t* p_row = pair_row ? pair_row : (int32_t*)(ws + L.pair_row);
  int32_t* r_tok = row_token ? row_token : (int32_t*)(ws + L.row_token);
  int32_t* offs = expert_offsets ? expert_offsets : (int32_t*)(ws + L.offsets);
  bf16_t* y = (bf16_t*)(ws + L.y);   // rounded once before the combine, as moe_forward's: half the bytes of float32
  const Ffn8Layout F = ffn8_layout(P, I);
  uint8_t* h_q = (uint8_t*)(ws + L.ffn + F.h_q);
  float* h_s = (float*)(ws + L.ffn + F.h_s);
  hipStream_t s = (hipStream_t)stream;
  if (logits) TRY(from_hip(launch_route_topk(logits, T, E, k, topk_idx, topk_w, s)));
  TRY(from_hip(launch_permute_index(topk_idx, P, k, E, r_tok, p_row, offs, ws + L.perm_ws, s)));
  const int ldx = row_bytes8(T, d), ldh = row_bytes8(P, I);
  TRY(from_hip(launch_quantize_rows_bf16((const bf16_t*)x, T, d, x_q, ldx, x_s, s)));
  TRY(from_hip(launch_gate_up_fp8(x_q, ldx, x_s, offs, P, E, d, I, (const uint8_t*)w_gate_up_q, w_gate_up_s, r_tok, T,
                                  h_q, ldh, h_s, s)));
  TRY(from_hip(launch_down_fp8(h_q, ldh, h_s, offs, P, E, d, I, (const uint8_t*)w_down_q, w_down_s, y, s)));
  return from_hip(launch_combine_bf16(y, P, p_row, topk_w, T, k, d, (bf16_t*)out, s));
}

size_t moe_forward_few_workspace_size(int32_t T, int32_t d, int32_t E, int32_t k, int32_t I, moe_dtype dt) {
  if (!few_sizes_ok(T, d, E, k, I) || !dtype_ok(dt)) return 0;
  const int split = dt == MOE_BF16 ? few_split_bf16(T * k, E, d, I) : few_split_f32(T * k, E, d, I);
  return few_layout(T, d, k, I, elem_size(dt), split).total;
}

moe_status moe_forward_few(const void* x, const float* logits, int32_t T, int32_t d, int32_t E, int32_t k, int32_t I,
                           const void* w_gate_up, const void* w_down, moe_dtype dt, int32_t* topk_idx, float* topk_w,
                           void* out, void* workspace, size_t workspace_bytes, void* stream) {
  if (!dtype_ok(dt)) return MOE_ERR_ARG;
  TRY(check_few(x, logits, T, d, E, k, I, 2, topk_idx, topk_w, out));
  if (T == 0) return MOE_OK;
  if (!w_gate_up || !w_down || !aligned16(x, w_gate_up, w_down, out, workspace)) return MOE_ERR_ARG;
  const int split = dt == MOE_BF16 ? few_split_bf16(T * k, E, d, I) : few_split_f32(T * k, E, d, I);
  const FewLayout L = few_layout(T, d, k, I, elem_size(dt), split);
  if (!workspace || workspace_bytes < L.total) return MOE_ERR_WORKSPACE;
  const FewScratch ws = carve_few(L, workspace);
  hipStream_t s = (hipStream_t)stream;
  if (dt == MOE_BF16)
    return from_hip(launch_few_bf16((const bf16_t*)x, logits, T, d, E, k, I, (const bf16_t*)w_gate_up,
                                    (const bf16_t*)w_down, topk_idx, topk_w, (bf16_t*)out, ws, s));
  return from_hip(launch_few_f32((const float*)x, logits, T, d, E, k, I, (const float*)w_gate_up,
                                 (const float*)w_down, topk_idx, topk_w, (float*)out, ws, s));
}

size_t moe_forward_few_fp8_workspace_size(int32_t T, int32_t d, int32_t E, int32_t k, int32_t I) {
  if (!few_sizes_ok(T, d, E, k, I)) return 0;
  return few_layout(T, d, k, I, 2, few_split_fp8(T * k, E, d, I)).total;
}

moe_status moe_forward_few_fp8(const void* x, const float* logits, int32_t T, int32_t d, int32_t E, int32_t k,
                               int32_t I, const void* w_gate_up_q, const float* w_gate_up_s, const void* w_down_q,
                               const float* w_down_s, int32_t* topk_idx, float* topk_w, void* out, void* workspace,
                               size_t workspace_bytes, void* stream) {
  TRY(check_few(x, logits, T, d, E, k, I, 1, topk_idx, topk_w, out));
  if (T == 0) return MOE_OK;
  if (!w_gate_up_q || !w_gate_up_s || !w_down_q || !w_down_s) return MOE_ERR_ARG;
  if (!aligned16(x, w_gate_up_q, w_down_q, out, workspace)) return MOE_ERR_ARG;
  const FewLayout L = few_layout(T, d, k, I, 2, few_split_fp8(T * k, E, d, I));
  if (!workspace || workspace_bytes < L.total) return MOE_ERR_WORKSPACE;
  return from_hip(launch_few_fp8((const bf16_t*)x, logits, T, d, E, k, I, (const uint8_t*)w_gate_up_q, w_gate_up_s,
                                 (const uint8_t*)w_down_q, w_down_s, topk_idx, topk_w, (bf16_t*)out,
                                 carve_few(L, workspace), (hipStream_t)stream));
}

}  // extern "C"
