// api_training.hip -- the C ABI of include/moe_training.h: host-side
// validation, workspace carving and kernel launches.  Every argument is checked
// before anything is enqueued; no call allocates, frees or synchronises.
#include "../../include/moe_training.h"
#include "checks.hpp"

using namespace tre;

namespace {

// Whether every address is a multiple of 16 (a NULL that reaches here is a
// missing workspace).
template <typename... P>
bool aligned16(const P*... p) {
  return ((((uintptr_t)p & 15) == 0) && ...);
}

// A tile's 256 rows of [dg | du] are addressed with 31 bits.
constexpr int32_t kMaxWidth = 1 << 21;

moe_status check_sizes(moe_dtype dt, int32_t E, int32_t d, int32_t I) {
  if (!dtype_ok(dt)) return MOE_ERR_ARG;
  TRY(check_experts(E));
  TRY(check_width(d));
  TRY(check_width(I));
  if (d >= kMaxWidth || I >= kMaxWidth) return MOE_ERR_UNSUPPORTED;
  if ((int64_t)E * d * 2 * I >= 8 * kMaxElems) return MOE_ERR_UNSUPPORTED;
  if ((int64_t)d * I * 4 >= kMaxElems) return MOE_ERR_UNSUPPORTED;   // one expert's weights < 2 GiB
  return MOE_OK;
}

moe_status check_rows(moe_dtype dt, int64_t rows, int32_t E, int32_t d, int32_t I) {
  if (rows < 0) return MOE_ERR_ARG;
  TRY(check_sizes(dt, E, d, I));
  if (rows * (d > 2 * (int64_t)I ? d : 2 * (int64_t)I) >= kMaxElems) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status check_layer(moe_dtype dt, int32_t T, int32_t d, int32_t E, int32_t k, int32_t I) {
  if (T < 0 || k < 1) return MOE_ERR_ARG;
  TRY(check_rows(dt, (int64_t)T * k, E, d, I));
  if ((int64_t)T * E >= kMaxElems) return MOE_ERR_UNSUPPORTED;
  if ((int64_t)T * d >= kMaxElems / 2) return MOE_ERR_UNSUPPORTED;   // token rows are addressed with 32-bit byte offsets
  return MOE_OK;
}

bool sizes_positive(int64_t rows, int32_t d, int32_t E, int32_t I, moe_dtype dt) {
  return rows >= 0 && d >= 1 && E >= 1 && I >= 1 && dtype_ok(dt);
}

// What the two products of a forward use beside their operands: h, float32's
// pre-activations before they are rounded (bf16: those of a few rows, or, where
// gate/up's k-stages are cut into gu_split > 1 ranges, theirs), and (bf16) the down
// projection's float32 rows in ranges (y_split of them; 0: it writes bf16 rows at once), its
// split tail and the products' tile counters.
struct FfnLayout {
  size_t h, gu, extra, y, split, sched, total;
  int gu_split, y_split;
  bool few;
};

// Of few tiles, whether gate/up is the bf16 product with its k-stages in ranges: a
// tile in float32 walks all of d by itself (the forward of 16 rows, 1 expert, 2560 x
// 64: 60 us, in ranges 21; 4 rows, 3 experts, 1536 x 128: 40 and 19).
bool few_wide(int64_t d, moe_dtype dt) { return dt == MOE_BF16 && d > 768; }

FfnLayout ffn_layout(int64_t rows, int64_t d, int64_t E, int64_t I, moe_dtype dt, bool rows32) {
  FfnLayout L{};
  size_t o = 0;
  L.few = small_products(rows, (int)E, (int)d, (int)I, dt == MOE_BF16);
  if (L.few) {   // h, g | u of a wide product, and (a layer's) y
    L.h = o; o += align256((size_t)(rows * I) * 4);
    L.gu_split = few_wide(d, dt) ? rows_split(rows, (int)E, (int)d, (int)(2 * I)) : 0;
    L.gu = o; o += align256((size_t)(L.gu_split * rows * 2 * I) * 4);
    L.y = o; o += rows32 ? align256((size_t)(rows * d) * 4) : 0;
    L.y_split = 1;
    L.total = o;
    return L;
  }
  L.gu_split = dt == MOE_BF16 ? rows_split(rows, (int)E, (int)d, (int)(2 * I)) : 1;
  L.y_split = dt == MOE_BF16 ? rows_split(rows, (int)E, (int)I, (int)d) : 0;
  if (!rows32 && L.y_split == 1) L.y_split = 0;
  L.h = o;     o += align256((size_t)(rows * I) * elem_size(dt));
  L.gu = o;    o += dt == MOE_F32 || L.gu_split > 1 ? align256((size_t)(L.gu_split * rows * 2 * I) * 4) : 0;
  L.extra = o; o += dt == MOE_BF16 ? align256((size_t)keep_extra_floats(rows, (int)E, (int)d, (int)I) * 4) : 0;
  L.y = o;     o += align256((size_t)(L.y_split * rows * d) * 4);
  L.split = o; o += dt == MOE_BF16 ? align256(split_workspace(rows, (int)E, (int)d, (int)I)) : 0;
  L.sched = o; o += dt == MOE_BF16 ? align256(kSchedWords * 4) : 0;
  L.total = o;
  return L;
}

struct LayerLayout {
  size_t perm_ws, x_perm, y, ffn, total;
};

LayerLayout layer_layout(int64_t T, int64_t d, int64_t E, int64_t k, int64_t I, moe_dtype dt) {
  const int64_t P = T * k;
  LayerLayout L;
  size_t o = 0;
  L.perm_ws = o; o += permute_index_workspace(P, (int)E);
  const FfnLayout F = ffn_layout(P, d, E, I, dt, true);
  const size_t f32 = dt == MOE_F32 && !F.few ? align256((size_t)(P * d) * 4) : 0;
  L.x_perm = o;  o += f32;   // (the others gather rows in place, and have y among the products')
  L.y = o;       o += f32;
  L.ffn = o;     o += F.total;
  L.total = o;
  return L;
}

// The gradients of grouped rows: h and dgu (times the rows' weights), g | u
// where they are computed again (float32, or bf16's 16-bit codes and their
// scales), float32's dh.
// (dx: bf16 rows' dx as float32 ranges, dx_split of them; 0: the product writes
// bf16 rows at once; gu32, dh: ranges of bf16's other two products of rows, where
// they are cut)
struct GradLayout {
  size_t h, dgu, gu, gu_s, extra, gu32, dh, dx, dw, total;
  int gu_split, dh_split, dx_split, dw_split;   // ranges of the row gradients' k and of the weight gradients' rows
  bool few;                                     // the kernels of few tiles
};

GradLayout grad_layout(int64_t rows, int64_t E, int64_t d, int64_t I, moe_dtype dt, bool layer) {
  const size_t s = elem_size(dt);
  const bool again = !layer;
  GradLayout L{};
  L.few = small_products(rows, (int)E, (int)d, (int)I, dt == MOE_BF16);
  if (L.few) {
    size_t o = 0;
    L.h = o;   o += align256((size_t)(rows * I) * 4);
    L.dgu = o; o += align256((size_t)(rows * 2 * I) * 4);
    L.gu_split = again && few_wide(d, dt) ? rows_split(rows, (int)E, (int)d, (int)(2 * I)) : 0;
    L.gu32 = o; o += align256((size_t)(L.gu_split * rows * 2 * I) * 4);
    L.gu = o;   o += L.gu_split ? align256((size_t)(rows * 2 * I) * 2) : 0;
    L.gu_s = o; o += L.gu_split ? align256((size_t)(rows * 2 * (I / kKeepBlock)) * 4) : 0;
    L.dx = o;  o += layer ? align256((size_t)(rows * d) * 4) : 0;
    L.dx_split = 1;
    L.total = o;
    return L;
  }
  L.gu_split = dt == MOE_BF16 && again ? rows_split(rows, (int)E, (int)d, (int)(2 * I)) : 1;
  L.dh_split = dt == MOE_BF16 ? rows_split(rows, (int)E, (int)d, (int)I) : 1;
  L.dx_split = dt == MOE_BF16 ? rows_split(rows, (int)E, (int)(2 * I), (int)d) : layer ? 1 : 0;
  if (!layer && L.dx_split == 1) L.dx_split = 0;
  size_t o = 0;
  L.h = o;   o += align256((size_t)(rows * I) * s);
  L.dgu = o; o += align256((size_t)(rows * 2 * I) * s);
  L.gu = o;  o += again ? align256((size_t)(rows * 2 * I) * s) : 0;
  L.gu_s = o; o += again && dt == MOE_BF16 ? align256((size_t)(rows * 2 * (I / kKeepBlock)) * 4) : 0;
  L.extra = o;
  o += again && dt == MOE_BF16 ? align256((size_t)keep_extra_floats(rows, (int)E, (int)d, (int)I) * 4) : 0;
  L.gu32 = o;
  o += L.gu_split > 1 ? align256((size_t)(L.gu_split * rows * 2 * I) * 4) : 0;
  L.dh = o;  o += dt == MOE_F32 || L.dh_split > 1 ? align256((size_t)(L.dh_split * rows * I) * 4) : 0;
  L.dx = o;  o += align256((size_t)(L.dx_split * rows * d) * 4);
  L.dw_split = dt == MOE_BF16 ? ffn_wgrad_split(rows, (int)E, (int)d, (int)I) : 1;
  L.dw = o;  o += L.dw_split > 1 ? align256((size_t)(L.dw_split * E * 3 * d * I) * 4) : 0;
  L.total = o;
  return L;
}

// The layer's backward around them: the rows' weights, the dot products' parts,
// and the grouped rows of x and dout.
struct BackwardLayout {
  size_t x_perm, dout_perm, row_w, dot, grad, total;
};

int64_t dot_columns(int64_t rows, int64_t E, int64_t d, int64_t I, moe_dtype dt) {
  if (small_products(rows, (int)E, (int)d, (int)I, dt == MOE_BF16)) return I / 32;
  return dt == MOE_F32 || rows_split(rows, (int)E, (int)d, (int)I) > 1 ? 1 : dot_parts((int)I);
}

BackwardLayout backward_layout(int64_t T, int64_t d, int64_t E, int64_t k, int64_t I, moe_dtype dt) {
  const int64_t P = T * k;
  const size_t copy = align256((size_t)(P * d) * elem_size(dt));
  BackwardLayout L;
  size_t o = 0;
  L.x_perm = o;    o += copy;
  L.dout_perm = o; o += copy;
  L.row_w = o;     o += align256((size_t)P * 4);
  L.dot = o;       o += align256((size_t)(P * dot_columns(P, E, d, I, dt)) * 4);
  L.grad = o;      o += grad_layout(P, E, d, I, dt, true).total;
  L.total = o;
  return L;
}

moe_status zero_weight_gradients(int32_t E, int32_t d, int32_t I, moe_dtype dt, void* dw_gate_up, void* dw_down,
                                 hipStream_t s) {
  if (!dw_gate_up || !dw_down || !aligned16(dw_gate_up, dw_down)) return MOE_ERR_ARG;
  const int64_t halves = dt == MOE_F32 ? 2 : 1;   // a float32 element is cleared as two bf16 ones
  TRY(from_hip(launch_zero_bf16((bf16_t*)dw_gate_up, (int64_t)E * d * 2 * I * halves, s)));
  return from_hip(launch_zero_bf16((bf16_t*)dw_down, (int64_t)E * I * d * halves, s));
}

// The checkpoint (of 8 or 16 bits) of rows x, and of 8 bits h: in one kernel, or,
// where the product's k-stages are cut into ranges, in gu and from there.
moe_status gate_up_keep(const bf16_t* x, int64_t x_rows, const int32_t* row_token, const int32_t* offs, int64_t rows,
                        int32_t E, int32_t d, int32_t I, const bf16_t* wgu, bf16_t* h, const Kept& kept, int bits,
                        int gu_split, float* gu, hipStream_t s, int32_t* sched) {
  if (gu_split > 1) {
    TRY(from_hip(launch_gate_up_rows32(x, offs, rows, E, d, I, wgu, gu, gu_split, s, row_token, x_rows)));
    return from_hip(launch_keep_rows(gu, gu_split, offs, E, rows, I, kept, bits, h, nullptr, s));
  }
  if (bits == 16) return from_hip(launch_gate_up_keep16_bf16(x, offs, rows, E, d, I, wgu, kept, s, sched));
  return from_hip(launch_gate_up_keep8_bf16(x, offs, rows, E, d, I, wgu, h, kept, s, row_token, x_rows, sched));
}

// The forward of few tiles (gu_split: ranges of gate/up's bf16 product; 0: in float32).
template <typename T, typename O>
moe_status few_rows(const T* x, int64_t x_rows, const int32_t* row_token, const int32_t* offs, int64_t rows, int32_t E,
                    int32_t d, int32_t I, const T* wgu, const T* wd, float* h, const Kept& kept, int gu_split,
                    float* gu, O* y, hipStream_t s) {
  if constexpr (sizeof(T) == 2) {
    if (gu_split) {
      TRY(from_hip(launch_gate_up_rows32(x, offs, rows, E, d, I, wgu, gu, gu_split, s, row_token, x_rows)));
      TRY(from_hip(launch_keep_rows(gu, gu_split, offs, E, rows, I, kept, 8, nullptr, h, s)));
      return from_hip(launch_small_down(h, offs, rows, E, d, I, wd, y, s));
    }
  }
  TRY(from_hip(launch_small_gate_up(x, x_rows, row_token, offs, rows, E, d, I, wgu, h, kept, s)));
  return from_hip(launch_small_down(h, offs, rows, E, d, I, wd, y, s));
}

// w [dg | du], w h and the parts of <dh, h> of rows with gradient dy, the same way.
moe_status down_bwd(const bf16_t* dy, const int32_t* offs, int64_t rows, int32_t E, int32_t d, int32_t I,
                    const bf16_t* wd, const Kept& kept, int bits, const float* row_w, bf16_t* dgu, bf16_t* h,
                    float* dot, int dh_split, float* dh, hipStream_t s) {
  if (dh_split > 1) {
    TRY(from_hip(launch_down_dgrad_rows32(dy, offs, rows, E, d, I, wd, dh, dh_split, s)));
    return from_hip(launch_swiglu_bwd_rows(dh, dh_split, kept, bits, row_w, offs, E, rows, I, dgu, h, dot, s));
  }
  return from_hip(launch_down_bwd_bf16(dy, offs, rows, E, d, I, wd, kept, bits, row_w, dgu, h, dot, s));
}

// The gradients of grouped rows x with dy (times row_w), float32: from the
// checkpoint, or, where kept.q is null, from g | u computed again.
moe_status grad_rows_f32(const float* x, const float* dy, const float* row_w, const int32_t* offs, int64_t rows,
                         int32_t E, int32_t d, int32_t I, const float* wgu, const float* wd, const Kept& kept,
                         float* dx, float* dw_gate_up, float* dw_down, float* dot, char* ws, const GradLayout& L,
                         hipStream_t s) {
  const bool again = kept.q == nullptr;
  float *h = (float*)(ws + L.h), *dgu = (float*)(ws + L.dgu), *gu = (float*)(ws + L.gu), *dh = (float*)(ws + L.dh);
  if (L.few)
    return from_hip(launch_small_grads(x, dy, offs, rows, E, d, I, wgu, wd, kept, 8, row_w, dgu, h, dot, dx,
                                       dw_gate_up, dw_down, s));
  if (again) TRY(from_hip(launch_gate_up_save_f32(x, offs, rows, E, d, I, wgu, h, gu, s)));
  TRY(from_hip(launch_down_dgrad_f32(dy, offs, rows, E, d, I, wd, dh, s)));
  TRY(from_hip(launch_swiglu_bwd_f32(dh, again ? gu : nullptr, kept, row_w, offs, E, rows, I, dgu, h, dot, s)));
  TRY(from_hip(launch_wgrad_f32(h, I, I, dy, d, d, offs, rows, E, dw_down, s)));
  TRY(from_hip(launch_gate_up_dgrad_f32(dgu, offs, rows, E, d, I, wgu, dx, s)));
  return from_hip(launch_wgrad_f32(x, d, d, dgu, 2 * I, 2 * I, offs, rows, E, dw_gate_up, s));
}

}  // namespace

extern "C" {

size_t moe_grouped_ffn_train_workspace_size(int32_t max_rows, int32_t E, int32_t d, int32_t I, moe_dtype dt) {
  if (!sizes_positive(max_rows, d, E, I, dt)) return 0;
  return ffn_layout(max_rows, d, E, I, dt, false).total;
}

moe_status moe_grouped_ffn_train(const void* x_perm, const int32_t* expert_offsets, int32_t max_rows, int32_t E,
                                 int32_t d, int32_t I, const void* w_gate_up, const void* w_down, moe_dtype dt,
                                 void* y_perm, void* gu_q, float* gu_s, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  TRY(check_rows(dt, max_rows, E, d, I));
  if (max_rows == 0) return MOE_OK;
  if (!x_perm || !expert_offsets || !w_gate_up || !w_down || !y_perm || !gu_q || !gu_s) return MOE_ERR_ARG;
  if (!aligned16(x_perm, w_gate_up, w_down, y_perm, gu_q, workspace)) return MOE_ERR_ARG;
  const FfnLayout L = ffn_layout(max_rows, d, E, I, dt, false);
  if (!workspace || workspace_bytes < L.total) return MOE_ERR_WORKSPACE;
  char* ws = (char*)workspace;
  const Kept kept{(int8_t*)gu_q, gu_s, (float*)(ws + L.extra)};
  hipStream_t s = (hipStream_t)stream;
  if (L.few) {
    float *h = (float*)(ws + L.h), *gu = (float*)(ws + L.gu);
    if (dt == MOE_F32)
      return few_rows((const float*)x_perm, 0, nullptr, expert_offsets, max_rows, E, d, I, (const float*)w_gate_up,
                      (const float*)w_down, h, kept, 0, gu, (float*)y_perm, s);
    return few_rows((const bf16_t*)x_perm, 0, nullptr, expert_offsets, max_rows, E, d, I, (const bf16_t*)w_gate_up,
                    (const bf16_t*)w_down, h, kept, L.gu_split, gu, (bf16_t*)y_perm, s);
  }
  if (dt == MOE_F32) {
    float *h = (float*)(ws + L.h), *gu = (float*)(ws + L.gu);
    TRY(from_hip(launch_gate_up_save_f32((const float*)x_perm, expert_offsets, max_rows, E, d, I,
                                         (const float*)w_gate_up, h, gu, s)));
    TRY(from_hip(launch_keep8_f32(gu, expert_offsets, E, max_rows, I, kept, s)));
    return from_hip(launch_down_f32(h, expert_offsets, max_rows, E, d, I, (const float*)w_down, (float*)y_perm, s));
  }
  int32_t* sched = claims_tiles(max_rows, E, d, I) ? (int32_t*)(ws + L.sched) : nullptr;
  bf16_t* h = (bf16_t*)(ws + L.h);
  if (sched) TRY(from_hip(launch_sched_reset(sched, s)));
  TRY(gate_up_keep((const bf16_t*)x_perm, 0, nullptr, expert_offsets, max_rows, E, d, I, (const bf16_t*)w_gate_up, h,
                   kept, 8, L.gu_split, (float*)(ws + L.gu), s, sched));
  if (L.y_split) {
    float* y = (float*)(ws + L.y);
    TRY(from_hip(launch_down_rows32(h, expert_offsets, max_rows, E, d, I, (const bf16_t*)w_down, y, L.y_split, s,
                                    nullptr, nullptr)));
    return from_hip(launch_split_sum(y, L.y_split, expert_offsets, E, max_rows, d, (bf16_t*)y_perm, s));
  }
  return from_hip(launch_down_bf16(h, expert_offsets, max_rows, E, d, I, (const bf16_t*)w_down, (bf16_t*)y_perm, s,
                                   (float*)(ws + L.split), sched));
}

size_t moe_grouped_ffn_backward_workspace_size(int32_t max_rows, int32_t E, int32_t d, int32_t I, moe_dtype dt) {
  if (!sizes_positive(max_rows, d, E, I, dt)) return 0;
  return grad_layout(max_rows, E, d, I, dt, false).total;
}

moe_status moe_grouped_ffn_backward(const void* x_perm, const int32_t* expert_offsets, int32_t max_rows, int32_t E,
                                    int32_t d, int32_t I, const void* w_gate_up, const void* w_down, moe_dtype dt,
                                    const void* gu_q, const float* gu_s, const void* dy_perm, void* dx_perm,
                                    void* dw_gate_up, void* dw_down, void* workspace, size_t workspace_bytes,
                                    void* stream) {
  TRY(check_rows(dt, max_rows, E, d, I));
  if ((gu_q == nullptr) != (gu_s == nullptr)) return MOE_ERR_ARG;
  hipStream_t s = (hipStream_t)stream;
  if (max_rows == 0) return zero_weight_gradients(E, d, I, dt, dw_gate_up, dw_down, s);
  if (!x_perm || !expert_offsets || !w_gate_up || !w_down || !dy_perm || !dx_perm || !dw_gate_up || !dw_down)
    return MOE_ERR_ARG;
  if (!aligned16(x_perm, w_gate_up, w_down, dy_perm, dx_perm, dw_gate_up, dw_down, gu_q, workspace)) return MOE_ERR_ARG;
  const GradLayout L = grad_layout(max_rows, E, d, I, dt, false);
  if (!workspace || workspace_bytes < L.total) return MOE_ERR_WORKSPACE;
  char* ws = (char*)workspace;
  const Kept kept{(int8_t*)gu_q, (float*)gu_s, nullptr};
  if (dt == MOE_F32)
    return grad_rows_f32((const float*)x_perm, (const float*)dy_perm, nullptr, expert_offsets, max_rows, E, d, I,
                         (const float*)w_gate_up, (const float*)w_down, kept, (float*)dx_perm, (float*)dw_gate_up,
                         (float*)dw_down, nullptr, ws, L, s);
  const bf16_t *x = (const bf16_t*)x_perm, *dy = (const bf16_t*)dy_perm, *wgu = (const bf16_t*)w_gate_up,
               *wd = (const bf16_t*)w_down;
  const Kept again{(int8_t*)(ws + L.gu), (float*)(ws + L.gu_s), (float*)(ws + L.extra)};
  if (L.few) {
    const bool wide = !gu_q && L.gu_split;
    if (wide) {
      float* gu = (float*)(ws + L.gu32);
      TRY(from_hip(launch_gate_up_rows32(x, expert_offsets, max_rows, E, d, I, wgu, gu, L.gu_split, s, nullptr, 0)));
      TRY(from_hip(launch_keep_rows(gu, L.gu_split, expert_offsets, E, max_rows, I, again, 16, nullptr, nullptr, s)));
    }
    return from_hip(launch_small_grads(x, dy, expert_offsets, max_rows, E, d, I, wgu, wd, wide ? again : kept,
                                       wide ? 16 : 8, nullptr, (float*)(ws + L.dgu), (float*)(ws + L.h), nullptr,
                                       (bf16_t*)dx_perm, (bf16_t*)dw_gate_up, (bf16_t*)dw_down, s));
  }
  bf16_t *h = (bf16_t*)(ws + L.h), *dgu = (bf16_t*)(ws + L.dgu);
  if (!gu_q)
    TRY(gate_up_keep(x, 0, nullptr, expert_offsets, max_rows, E, d, I, wgu, nullptr, again, 16, L.gu_split,
                     (float*)(ws + L.gu32), s, nullptr));
  TRY(down_bwd(dy, expert_offsets, max_rows, E, d, I, wd, gu_q ? kept : again, gu_q ? 8 : 16, nullptr, dgu, h, nullptr,
               L.dh_split, (float*)(ws + L.dh), s));
  if (L.dx_split) {
    float* dx = (float*)(ws + L.dx);
    TRY(from_hip(launch_gate_up_dgrad_rows32(dgu, expert_offsets, max_rows, E, d, I, wgu, dx, L.dx_split, s)));
    TRY(from_hip(launch_split_sum(dx, L.dx_split, expert_offsets, E, max_rows, d, (bf16_t*)dx_perm, s)));
  } else {
    TRY(from_hip(launch_gate_up_dgrad_bf16(dgu, expert_offsets, max_rows, E, d, I, wgu, (bf16_t*)dx_perm, s)));
  }
  return from_hip(launch_ffn_wgrad_bf16(x, dy, h, dgu, expert_offsets, max_rows, E, d, I,
                                        (bf16_t*)dw_gate_up, (bf16_t*)dw_down, L.dw_split, (float*)(ws + L.dw), s));
}

size_t moe_forward_train_q8_workspace_size(int32_t T, int32_t d, int32_t E, int32_t k, int32_t I, moe_dtype dt) {
  if (!sizes_positive(T, d, E, I, dt) || k < 1) return 0;
  return layer_layout(T, d, E, k, I, dt).total;
}

moe_status moe_forward_train_q8(const void* x, const float* logits, int32_t T, int32_t d, int32_t E, int32_t k,
                                int32_t I, const void* w_gate_up, const void* w_down, moe_dtype dt, int32_t* topk_idx,
                                float* topk_w, int32_t* expert_offsets, int32_t* row_token, int32_t* pair_row,
                                void* gu_q, float* gu_s, void* out, void* workspace, size_t workspace_bytes,
                                void* stream) {
  TRY(check_layer(dt, T, d, E, k, I));
  if (logits && k > E) return MOE_ERR_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !w_gate_up || !w_down || !topk_idx || !topk_w || !expert_offsets || !row_token || !pair_row || !gu_q ||
      !gu_s || !out)
    return MOE_ERR_ARG;
  if (!aligned16(x, w_gate_up, w_down, gu_q, out, workspace)) return MOE_ERR_ARG;
  const LayerLayout L = layer_layout(T, d, E, k, I, dt);
  if (!workspace || workspace_bytes < L.total) return MOE_ERR_WORKSPACE;
  const int64_t P = (int64_t)T * k;
  const FfnLayout F = ffn_layout(P, d, E, I, dt, true);
  char *ws = (char*)workspace, *fws = ws + L.ffn;
  const Kept kept{(int8_t*)gu_q, gu_s, (float*)(fws + F.extra)};
  hipStream_t s = (hipStream_t)stream;
  if (logits) TRY(from_hip(launch_route_topk(logits, T, E, k, topk_idx, topk_w, s)));
  if (F.few) {
    float *h = (float*)(fws + F.h), *gu = (float*)(fws + F.gu), *y = (float*)(fws + F.y);
    TRY(from_hip(launch_permute_index(topk_idx, P, k, E, row_token, pair_row, expert_offsets, ws + L.perm_ws, s)));
    if (dt == MOE_F32) {
      TRY(few_rows((const float*)x, T, row_token, expert_offsets, P, E, d, I, (const float*)w_gate_up,
                   (const float*)w_down, h, kept, 0, gu, y, s));
      return from_hip(launch_combine_f32(y, P, pair_row, topk_w, T, k, d, (float*)out, s));
    }
    TRY(few_rows((const bf16_t*)x, T, row_token, expert_offsets, P, E, d, I, (const bf16_t*)w_gate_up,
                 (const bf16_t*)w_down, h, kept, F.gu_split, gu, y, s));
    return from_hip(launch_combine_rows32(y, 1, P, pair_row, topk_w, T, k, d, (bf16_t*)out, s));
  }
  if (dt == MOE_F32) {
    float *xp = (float*)(ws + L.x_perm), *h = (float*)(fws + F.h), *gu = (float*)(fws + F.gu), *y = (float*)(ws + L.y);
    TRY(from_hip(launch_permute_rows(topk_idx, T, k, E, row_token, pair_row, expert_offsets, ws + L.perm_ws, s,
                                     nullptr, x, (int64_t)d * 4, xp)));
    TRY(from_hip(launch_gate_up_save_f32(xp, expert_offsets, P, E, d, I, (const float*)w_gate_up, h, gu, s)));
    TRY(from_hip(launch_keep8_f32(gu, expert_offsets, E, P, I, kept, s)));
    TRY(from_hip(launch_down_f32(h, expert_offsets, P, E, d, I, (const float*)w_down, y, s)));
    return from_hip(launch_combine_f32(y, P, pair_row, topk_w, T, k, d, (float*)out, s));
  }
  // rows gathered in the products' loads; y stays float32 until the output's one rounding
  int32_t* sched = (int32_t*)(fws + F.sched);
  bf16_t* h = (bf16_t*)(fws + F.h);
  float* y = (float*)(fws + F.y);
  TRY(from_hip(launch_permute_index(topk_idx, P, k, E, row_token, pair_row, expert_offsets, ws + L.perm_ws, s, sched)));
  TRY(gate_up_keep((const bf16_t*)x, T, row_token, expert_offsets, P, E, d, I, (const bf16_t*)w_gate_up, h, kept, 8,
                   F.gu_split, (float*)(fws + F.gu), s, sched));
  TRY(from_hip(launch_down_rows32(h, expert_offsets, P, E, d, I, (const bf16_t*)w_down, y, F.y_split, s,
                                  (float*)(fws + F.split), sched)));
  return from_hip(launch_combine_rows32(y, F.y_split, P, pair_row, topk_w, T, k, d, (bf16_t*)out, s));
}

size_t moe_backward_q8_workspace_size(int32_t T, int32_t d, int32_t E, int32_t k, int32_t I, moe_dtype dt) {
  if (!sizes_positive(T, d, E, I, dt) || k < 1) return 0;
  return backward_layout(T, d, E, k, I, dt).total;
}

moe_status moe_backward_q8(const void* x, int32_t T, int32_t d, int32_t E, int32_t k, int32_t I,
                           const void* w_gate_up, const void* w_down, moe_dtype dt, const int32_t* topk_idx,
                           const float* topk_w, const int32_t* expert_offsets, const int32_t* row_token,
                           const int32_t* pair_row, const void* gu_q, const float* gu_s, const void* dout, void* dx,
                           void* dw_gate_up, void* dw_down, float* dtopk_w, float* dlogits, void* workspace,
                           size_t workspace_bytes, void* stream) {
  TRY(check_layer(dt, T, d, E, k, I));
  if (dlogits && k > E) return MOE_ERR_ARG;
  hipStream_t s = (hipStream_t)stream;
  if (T == 0) return zero_weight_gradients(E, d, I, dt, dw_gate_up, dw_down, s);
  if (!x || !w_gate_up || !w_down || !topk_idx || !topk_w || !expert_offsets || !row_token || !pair_row || !gu_q ||
      !gu_s || !dout || !dx || !dw_gate_up || !dw_down || !dtopk_w)
    return MOE_ERR_ARG;
  if (!aligned16(x, w_gate_up, w_down, gu_q, dout, dx, dw_gate_up, dw_down, workspace)) return MOE_ERR_ARG;
  const BackwardLayout L = backward_layout(T, d, E, k, I, dt);
  if (!workspace || workspace_bytes < L.total) return MOE_ERR_WORKSPACE;
  const int64_t P = (int64_t)T * k;
  char* ws = (char*)workspace;
  float *row_w = (float*)(ws + L.row_w), *dot = (float*)(ws + L.dot);
  const Kept kept{(int8_t*)gu_q, (float*)gu_s, nullptr};
  // the combine's backward puts w_p before dout; it is applied to h and [dg | du] instead, so that dout stays exact
  // (a token's rows of dx stay float32 until its sum's one rounding)
  const GradLayout G = grad_layout(P, E, d, I, dt, true);
  char* gws = ws + L.grad;
  float* dxp = (float*)(gws + G.dx);
  void *x_perm = ws + L.x_perm, *dout_perm = ws + L.dout_perm;
  TRY(from_hip(launch_pair_rows(x, dout, T, k, (int64_t)d * elem_size(dt), pair_row, topk_w, P, x_perm, dout_perm,
                                row_w, s)));
  if (dt == MOE_F32) {
    TRY(grad_rows_f32((const float*)x_perm, (const float*)dout_perm, row_w, expert_offsets, P, E, d, I,
                      (const float*)w_gate_up, (const float*)w_down, kept, dxp, (float*)dw_gate_up, (float*)dw_down,
                      dot, gws, G, s));
    return from_hip(launch_combine_grad_f32(dxp, G.dx_split, dot, dot_columns(P, E, d, I, dt), P, pair_row, topk_w,
                                            topk_idx, T, k, d, E, (float*)dx, dtopk_w, dlogits, s));
  }
  const bf16_t *xp = (const bf16_t*)x_perm, *dyp = (const bf16_t*)dout_perm, *wgu = (const bf16_t*)w_gate_up,
               *wd = (const bf16_t*)w_down;
  if (G.few) {
    TRY(from_hip(launch_small_grads(xp, dyp, expert_offsets, P, E, d, I, wgu, wd, kept, 8, row_w,
                                    (float*)(gws + G.dgu), (float*)(gws + G.h), dot, dxp, (bf16_t*)dw_gate_up,
                                    (bf16_t*)dw_down, s)));
  } else {
    bf16_t *h = (bf16_t*)(gws + G.h), *dgu = (bf16_t*)(gws + G.dgu);
    TRY(down_bwd(dyp, expert_offsets, P, E, d, I, wd, kept, 8, row_w, dgu, h, dot, G.dh_split, (float*)(gws + G.dh),
                 s));
    TRY(from_hip(launch_gate_up_dgrad_rows32(dgu, expert_offsets, P, E, d, I, wgu, dxp, G.dx_split, s)));
    TRY(from_hip(launch_ffn_wgrad_bf16(xp, dyp, h, dgu, expert_offsets, P, E, d, I, (bf16_t*)dw_gate_up,
                                       (bf16_t*)dw_down, G.dw_split, (float*)(gws + G.dw), s)));
  }
  return from_hip(launch_combine_grad_bf16(dxp, G.dx_split, dot, dot_columns(P, E, d, I, dt), P, pair_row, topk_w,
                                           topk_idx, T, k, d, E, (bf16_t*)dx, dtopk_w, dlogits, s));
}

moe_status moe_checkpoint_values(const void* gu_q, const float* gu_s, int32_t rows, int32_t I, moe_dtype dt, void* gu,
                                 void* stream) {
  if (!dtype_ok(dt) || rows < 0) return MOE_ERR_ARG;
  TRY(check_width(I));
  if ((int64_t)rows * 2 * I >= kMaxElems) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!gu_q || !gu_s || !gu || !aligned16(gu_q, gu)) return MOE_ERR_ARG;
  const Kept kept{(int8_t*)gu_q, (float*)gu_s, nullptr};
  hipStream_t s = (hipStream_t)stream;
  if (dt == MOE_BF16) return from_hip(launch_keep8_values_bf16(kept, rows, I, (bf16_t*)gu, s));
  return from_hip(launch_keep8_values_f32(kept, rows, I, (float*)gu, s));
}

}  // extern "C"
