// train.hip -- the steps of the training operators beside the products: the
// 8-bit checkpoint of float32 rows and its values, the float32 SwiGLU
// backward, the grouped rows of x and dout, and the routing weights' gradients.
// (In bf16 the checkpoint is written and read, and the SwiGLU backward done, in
// the products' epilogues, grouped_ffn.hip, or, where the products are cut into
// ranges, here on their sums.)
//
// Each passes over its rows once and is bound by memory, or by its launch.
// Measured on the 128-expert layer (8192 tokens, 4 of 128, 2880 x 2880, bf16):
// k_keep8_values 100 us (5.8 TB/s), k_pair_rows 77 us (6.1 TB/s).
#include "keep8.hpp"

namespace tre {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / kWave;

// 16 lanes take a block of 64, four values each.
__global__ __launch_bounds__(kThreads) void k_keep8_f32(const float* __restrict__ gu,
                                                        const int32_t* __restrict__ offsets, int E, int64_t max_rows,
                                                        int nb, Kept kept) {
  const int64_t b = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / 16;   // block of the checkpoint (nb a row)
  const int64_t rows = clampi<int64_t>(offsets[E], 0, max_rows);
  if (b >= rows * nb) return;   // (the same for a block's 16 lanes)
  const int l16 = threadIdx.x % 16;
  const f32x4 v = *(const f32x4*)(gu + b * kKeepBlock + 4 * l16);
  const uint32_t m = max16(max(max(abs_bits(v[0]), abs_bits(v[1])), max(abs_bits(v[2]), abs_bits(v[3]))));
  float s, inv;
  keep_scale(m, s, inv);
  *(uint32_t*)(kept.q + b * kKeepBlock + 4 * l16) = keep_codes4(v[0], v[1], v[2], v[3], inv);
  if (l16 == 0) kept.s[b] = s;
}

// 16 codes a thread.
template <typename Elem>
__global__ __launch_bounds__(kThreads) void k_keep8_values(Kept kept, int64_t n_vec, Elem* __restrict__ gu) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= n_vec) return;
  const u32x4 q = ((const u32x4*)kept.q)[i];
  const float s = kept.s[i / (kKeepBlock / 16)];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float v[8];
    const uint32_t q0 = q[2 * h], q1 = q[2 * h + 1];
    keep_values4(q0, s, v);
    keep_values4(q1, s, v + 4);
    if constexpr (sizeof(Elem) == 4) {
      *(f32x4*)(gu + 16 * i + 8 * h) = f32x4{v[0], v[1], v[2], v[3]};
      *(f32x4*)(gu + 16 * i + 8 * h + 4) = f32x4{v[4], v[5], v[6], v[7]};
    } else {
      *(u32x4*)(gu + 16 * i + 8 * h) = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                             pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
    }
  }
}

// One wave a grouped row, four columns a lane: the SwiGLU backward of
// include/moe_training.h in float32, and the row's <dh, h>.
template <bool K8>
__global__ __launch_bounds__(kThreads) void k_swiglu_bwd_f32(const float* __restrict__ dh, const float* __restrict__ gu,
                                                             Kept kept, const float* __restrict__ row_w,
                                                             const int32_t* __restrict__ offsets, int E,
                                                             int64_t max_rows, int I, float* __restrict__ dgu,
                                                             float* __restrict__ h, float* __restrict__ dot) {
  const int64_t r = (int64_t)blockIdx.x * kWaves + threadIdx.x / kWave;
  if (r >= clampi<int64_t>(offsets[E], 0, max_rows)) return;
  const int lane = threadIdx.x % kWave;
  const float w = row_w ? row_w[r] : 1.f;
  float sum = 0.f;
  for (int c = 4 * lane; c < I; c += 4 * kWave) {
    float g[4], u[4];
    if constexpr (K8) {
      const int nb = I / kKeepBlock;
      keep_values4(*(const uint32_t*)(kept.q + r * 2 * I + c), kept.s[r * 2 * nb + c / kKeepBlock], g);
      keep_values4(*(const uint32_t*)(kept.q + r * 2 * I + I + c), kept.s[r * 2 * nb + nb + c / kKeepBlock], u);
    } else {
      const f32x4 a = *(const f32x4*)(gu + r * 2 * I + c), b = *(const f32x4*)(gu + r * 2 * I + I + c);
#pragma unroll
      for (int i = 0; i < 4; ++i) g[i] = a[i], u[i] = b[i];
    }
    const f32x4 d = *(const f32x4*)(dh + r * I + c);
    f32x4 dg, du, hv;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float sg = 1.f / (1.f + expf(-g[i]));
      const float silu = g[i] * sg, wd = w * d[i];
      sum = fmaf(silu * u[i], d[i], sum);
      dg[i] = wd * u[i] * (sg + silu * (1.f - sg));
      du[i] = wd * silu;
      hv[i] = w * (silu * u[i]);
    }
    *(f32x4*)(dgu + r * 2 * I + c) = dg;
    *(f32x4*)(dgu + r * 2 * I + I + c) = du;
    *(f32x4*)(h + r * I + c) = hv;
  }
  if (!dot) return;
#pragma unroll
  for (int off = kWave / 2; off > 0; off >>= 1) sum += __shfl_xor(sum, off, kWave);
  if (lane == 0) dot[r] = sum;
}

// The sum of n_split ranges' four elements at p, `stride` floats apart.
__device__ __forceinline__ f32x4 add_ranges(const float* __restrict__ p, int n_split, int64_t stride) {
  f32x4 sum = *(const f32x4*)p;
  for (int sp = 1; sp < n_split; ++sp) sum += *(const f32x4*)(p + sp * stride);
  return sum;
}

// 16 lanes take a row's block of 64 gates and ups.
template <int BITS, typename H>
__global__ __launch_bounds__(kThreads) void k_keep_rows(const float* __restrict__ gu, int n_split,
                                                        const int32_t* __restrict__ offsets, int E, int64_t max_rows,
                                                        int I, Kept kept, H* __restrict__ h) {
  const int nb = I / kKeepBlock;
  const int64_t item = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / 16;
  const int64_t row = item / nb;
  if (row >= clampi<int64_t>(offsets[E], 0, max_rows)) return;   // (the same for 16 lanes)
  const int l16 = threadIdx.x % 16, c = (int)(item - row * nb) * kKeepBlock + 4 * l16;
  const float* p = gu + row * 2 * I + c;
  const f32x4 v[2] = {add_ranges(p, n_split, max_rows * 2 * I), add_ranges(p + I, n_split, max_rows * 2 * I)};
  keep_block<BITS>(v, row, c, I, l16, kept, h);
}

// One wave a grouped row, four columns a lane: the bf16 products' SwiGLU backward
// (grouped_ffn.hip, kEpiBwd8) of whole sums.
template <int BITS>
__global__ __launch_bounds__(kThreads) void k_swiglu_bwd_rows(const float* __restrict__ dh, int n_split, Kept kept,
                                                              const float* __restrict__ row_w,
                                                              const int32_t* __restrict__ offsets, int E,
                                                              int64_t max_rows, int I, bf16_t* __restrict__ dgu,
                                                              bf16_t* __restrict__ h, float* __restrict__ dot) {
  const int64_t r = (int64_t)blockIdx.x * kWaves + threadIdx.x / kWave;
  if (r >= clampi<int64_t>(offsets[E], 0, max_rows)) return;
  const int lane = threadIdx.x % kWave, nb = I / kKeepBlock;
  const float w = row_w ? row_w[r] : 1.f;
  float sum = 0.f;
  for (int c = 4 * lane; c < I; c += 4 * kWave) {
    float v[2][4];
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int64_t at = (r * 2 + hf) * I + c;
      const float s = kept.s[(r * 2 + hf) * nb + c / kKeepBlock];
      if constexpr (BITS == 8) {
        keep_values4(*(const uint32_t*)(kept.q + at), s, v[hf]);
      } else {
        const uint2 q = *(const uint2*)(kept.q + 2 * at);
        keep_values2(q.x, s, v[hf]);
        keep_values2(q.y, s, v[hf] + 2);
      }
    }
    const f32x4 d = add_ranges(dh + r * I + c, n_split, max_rows * I);
    float dg[4], du[4], hv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float g = v[0][i], u = v[1][i];
      const float sg = __builtin_amdgcn_rcpf(1.f + __expf(-g)), silu = g * sg, wdh = w * d[i];
      hv[i] = silu * u;
      sum = fmaf(hv[i], d[i], sum);
      dg[i] = wdh * u * (sg + silu * (1.f - sg));
      du[i] = wdh * silu;
      hv[i] *= w;
    }
    *(uint2*)(dgu + r * 2 * I + c) = make_uint2(pack_bf16x2(dg[0], dg[1]), pack_bf16x2(dg[2], dg[3]));
    *(uint2*)(dgu + r * 2 * I + I + c) = make_uint2(pack_bf16x2(du[0], du[1]), pack_bf16x2(du[2], du[3]));
    *(uint2*)(h + r * I + c) = make_uint2(pack_bf16x2(hv[0], hv[1]), pack_bf16x2(hv[2], hv[3]));
  }
  if (!dot) return;
#pragma unroll
  for (int off = kWave / 2; off > 0; off >>= 1) sum += __shfl_xor(sum, off, kWave);
  if (lane == 0) dot[r] = sum;
}

// One wave a token: its rows of x and dout to every grouped row its pairs have,
// and those rows' routing weights.
__global__ __launch_bounds__(kThreads) void k_pair_rows(const u32x4* __restrict__ x, const u32x4* __restrict__ dout,
                                                        int64_t T, int k, int64_t vec_per_row,
                                                        const int32_t* __restrict__ pair_row,
                                                        const float* __restrict__ pair_w, int64_t max_rows,
                                                        u32x4* __restrict__ x_perm, u32x4* __restrict__ dout_perm,
                                                        float* __restrict__ row_w) {
  const int64_t t = (int64_t)blockIdx.x * kWaves + threadIdx.x / kWave;
  if (t >= T) return;
  const int lane = threadIdx.x % kWave;
  constexpr int kVec = 4;
  for (int64_t base = lane; base < vec_per_row; base += kVec * kWave) {
    u32x4 a[kVec], b[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int64_t v = base + i * kWave;
      if (v < vec_per_row) {
        a[i] = x[t * vec_per_row + v];
        b[i] = dout[t * vec_per_row + v];
      }
    }
    for (int j = 0; j < k; ++j) {
      const int64_t r = pair_row[t * k + j];
      MOE_DCHECK(r >= -1 && r < max_rows);
      if (r < 0 || r >= max_rows) continue;
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const int64_t v = base + i * kWave;
        if (v < vec_per_row) {
          x_perm[r * vec_per_row + v] = a[i];
          dout_perm[r * vec_per_row + v] = b[i];
        }
      }
    }
  }
  for (int j = lane; j < k; j += kWave) {
    const int64_t r = pair_row[t * k + j];
    if (r >= 0 && r < max_rows) row_w[r] = pair_w[t * k + j];
  }
}

unsigned blocks_of(int64_t n, int64_t per) { return (unsigned)ceil_div(n, per); }

}  // namespace

hipError_t launch_keep8_f32(const float* gu, const int32_t* expert_offsets, int E, int64_t max_rows, int I,
                            const Kept& kept, hipStream_t s) {
  const int nb = 2 * I / kKeepBlock;
  k_keep8_f32<<<blocks_of(max_rows * nb, kThreads / 16), kThreads, 0, s>>>(gu, expert_offsets, E, max_rows, nb, kept);
  return hipGetLastError();
}

hipError_t launch_keep8_values_f32(const Kept& kept, int64_t rows, int I, float* gu, hipStream_t s) {
  const int64_t n_vec = rows * 2 * I / 16;
  k_keep8_values<float><<<blocks_of(n_vec, kThreads), kThreads, 0, s>>>(kept, n_vec, gu);
  return hipGetLastError();
}

hipError_t launch_keep8_values_bf16(const Kept& kept, int64_t rows, int I, bf16_t* gu, hipStream_t s) {
  const int64_t n_vec = rows * 2 * I / 16;
  k_keep8_values<bf16_t><<<blocks_of(n_vec, kThreads), kThreads, 0, s>>>(kept, n_vec, gu);
  return hipGetLastError();
}

hipError_t launch_swiglu_bwd_f32(const float* dh, const float* gu, const Kept& kept, const float* row_w,
                                 const int32_t* expert_offsets, int E, int64_t max_rows, int I, float* dgu, float* h,
                                 float* dot, hipStream_t s) {
  const unsigned blocks = blocks_of(max_rows, kWaves);
  if (gu)
    k_swiglu_bwd_f32<false><<<blocks, kThreads, 0, s>>>(dh, gu, kept, row_w, expert_offsets, E, max_rows, I, dgu, h,
                                                        dot);
  else
    k_swiglu_bwd_f32<true><<<blocks, kThreads, 0, s>>>(dh, gu, kept, row_w, expert_offsets, E, max_rows, I, dgu, h,
                                                       dot);
  return hipGetLastError();
}

hipError_t launch_keep_rows(const float* gu, int n_split, const int32_t* expert_offsets, int E, int64_t max_rows, int I,
                            const Kept& kept, int bits, bf16_t* h, float* h32, hipStream_t s) {
  const unsigned blocks = blocks_of(max_rows * (I / kKeepBlock), kThreads / 16);
  if (h32) {
    k_keep_rows<8><<<blocks, kThreads, 0, s>>>(gu, n_split, expert_offsets, E, max_rows, I, kept, h32);
    return hipGetLastError();
  }
  const auto kernel = bits == 16 ? k_keep_rows<16, bf16_t> : k_keep_rows<8, bf16_t>;
  kernel<<<blocks, kThreads, 0, s>>>(gu, n_split, expert_offsets, E, max_rows, I, kept, h);
  return hipGetLastError();
}

hipError_t launch_swiglu_bwd_rows(const float* dh, int n_split, const Kept& kept, int bits, const float* row_w,
                                  const int32_t* expert_offsets, int E, int64_t max_rows, int I, bf16_t* dgu,
                                  bf16_t* h, float* dot, hipStream_t s) {
  const auto kernel = bits == 16 ? k_swiglu_bwd_rows<16> : k_swiglu_bwd_rows<8>;
  kernel<<<blocks_of(max_rows, kWaves), kThreads, 0, s>>>(dh, n_split, kept, row_w, expert_offsets, E, max_rows, I, dgu,
                                                          h, dot);
  return hipGetLastError();
}

hipError_t launch_pair_rows(const void* x, const void* dout, int64_t T, int k, int64_t row_bytes,
                            const int32_t* pair_row, const float* pair_w, int64_t max_rows, void* x_perm,
                            void* dout_perm, float* row_w, hipStream_t s) {
  k_pair_rows<<<blocks_of(T, kWaves), kThreads, 0, s>>>((const u32x4*)x, (const u32x4*)dout, T, k, row_bytes / 16,
                                                        pair_row, pair_w, max_rows, (u32x4*)x_perm,
                                                        (u32x4*)dout_perm, row_w);
  return hipGetLastError();
}

}  // namespace tre
