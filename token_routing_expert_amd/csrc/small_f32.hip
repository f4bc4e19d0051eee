// small_f32.hip -- the training operators' float32 products where the tiles of
// k_grouped_gemm_f32 (64 x 128, one a workgroup) are too few for the card.
//
// A workgroup takes 32 rows of one expert and 32 columns (gate/up: 64 gate and
// the 64 up columns beside them) and its four waves share the summed dimension:
// 8 values in turn, so a wave's operands are 16 bytes a lane, straight from
// memory to registers, with no stages to wait for one another.  The order of k
// inside v_mfma_f32_32x32x2_f32 is free as long as both operands use the same:
// lane i + 32 k of matrix instruction m holds element 4 k + m of the 8.  The four
// partial tiles are added in LDS in wave order (equal calls give equal bits), and
// the sums come out as four consecutive columns of one row a thread.
//
// What such a call costs is its launches and one memory round trip each, so the
// steps are few: the SwiGLU backward sits behind dh (with g | u computed again
// beside it where there is no checkpoint), and dx and both weight gradients, which
// do not read one another, are one launch.  Measured: at small_f32 below.
#include "keep8.hpp"

#include <algorithm>

namespace tre {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / kWave;
constexpr int kRows = 32, kCols = 32;

struct Rows {
  int e, r0, n;   // expert, first grouped row, rows (0: no tile)
};

// Row tile u of the list of every expert's 32-row tiles, from the device offsets.
__device__ __forceinline__ Rows row_tile(const int32_t* __restrict__ offsets, int64_t max_rows, int E, int u) {
  __shared__ int s_wave[kWaves];
  __shared__ int s_tile[3];
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  int lo = 0, cnt = 0;
  if (tid < E) {
    MOE_DCHECK(0 <= offsets[tid] && offsets[tid] <= offsets[tid + 1] && offsets[tid + 1] <= max_rows);
    lo = (int)clampi<int64_t>(offsets[tid], 0, max_rows);
    cnt = (int)clampi<int64_t>(offsets[tid + 1], lo, max_rows) - lo;
  }
  const int mt = (cnt + kRows - 1) / kRows;
  int incl = mt;
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    const int y = __shfl_up(incl, off, kWave);
    if (lane >= off) incl += y;
  }
  if (lane == kWave - 1) s_wave[wave] = incl;
  if (tid == 0) s_tile[2] = 0;
  __syncthreads();
  int before = incl - mt;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) before += w < wave ? s_wave[w] : 0;
  if (before <= u && u < before + mt) {
    s_tile[0] = tid;
    s_tile[1] = lo + (u - before) * kRows;
    s_tile[2] = min(kRows, cnt - (u - before) * kRows);
  }
  __syncthreads();
  return {s_tile[0], s_tile[1], s_tile[2]};
}

// acc[b] += this wave's share of A W over K, for column blocks at w[b].  a: the
// lane's row (row lane % 32 of the tile).  BT: W is [N][K] and w[b] the lane's row
// of it; else W is [K][ldw] and w[b] column lane % 32 of the block.
template <bool BT, int NB>
__device__ __forceinline__ void multiply(const float* __restrict__ a, const float* const (&w)[NB], int K, int ldw,
                                         f32x16 (&acc)[NB]) {
  const int wave = threadIdx.x / kWave, kh = (threadIdx.x % kWave) / 32;
  constexpr int U = NB > 2 && !BT ? 2 : 4;   // chunks of 8 whose loads go out together
  for (int k0 = 8 * wave; k0 < K; k0 += 32 * U) {
    f32x4 av[U], wv[U][NB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + 32 * u + 4 * kh;
      if (k0 + 32 * u >= K) continue;   // (wave-uniform)
      av[u] = *(const f32x4*)(a + k);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        if constexpr (BT) {
          wv[u][b] = *(const f32x4*)(w[b] + k);
        } else {
#pragma unroll
          for (int m = 0; m < 4; ++m) wv[u][b][m] = w[b][(int64_t)(k + m) * ldw];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k0 + 32 * u >= K) continue;
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int b = 0; b < NB; ++b)
          acc[b] = __builtin_amdgcn_mfma_f32_32x32x2f32(av[u][m], wv[u][b][m], acc[b], 0, 0, 0);
    }
  }
}

// The waves' partial tiles added: thread t gets row t / 8, columns 4 (t % 8) .. +3
// of every block.
template <int NB>
__device__ __forceinline__ void add_waves(const f32x16 (&acc)[NB], float (&s)[NB][kWaves][kRows * kCols],
                                          f32x4 (&sum)[NB]) {
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int q = 0; q < 16; ++q)
      s[b][wave][(8 * (q / 4) + 4 * (lane / 32) + q % 4) * kCols + lane % 32] = acc[b][q];
  __syncthreads();
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    sum[b] = *(const f32x4*)&s[b][0][4 * tid];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) sum[b] += *(const f32x4*)&s[b][w][4 * tid];
  }
}

__device__ __forceinline__ float max8(float v) {   // over 8 consecutive lanes
#pragma unroll
  for (int off = 1; off < 8; off <<= 1) {
    const float o = __shfl_xor(v, off, kWave);
    v = __builtin_bit_cast(float, max(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, o)));
  }
  return v;
}

// h and the checkpoint of 32 rows and 64 columns of I.  With row_token, row r's x
// is row row_token[r] of x (x_rows of them).
__global__ __launch_bounds__(kThreads) void k_small_gate_up(const float* __restrict__ x, int64_t x_rows,
                                                            const int32_t* __restrict__ row_token,
                                                            const int32_t* __restrict__ offsets, int64_t max_rows,
                                                            int E, int d, int I, const float* __restrict__ wgu,
                                                            float* __restrict__ h, Kept kept) {
  __shared__ float s[4][kWaves][kRows * kCols];
  const Rows t = row_tile(offsets, max_rows, E, (int)blockIdx.x);
  if (t.n == 0) return;   // (the whole workgroup)
  const int lane = threadIdx.x % kWave, n0 = 64 * (int)blockIdx.y;
  int64_t row = t.r0 + min(lane % 32, t.n - 1);
  if (row_token) {
    const int64_t tok = row_token[row];
    MOE_DCHECK(tok >= 0 && tok < x_rows);
    row = clampi<int64_t>(tok, 0, x_rows - 1);
  }
  const float* w0 = wgu + (int64_t)t.e * d * 2 * I + n0 + lane % 32;
  const float* const w[4] = {w0, w0 + 32, w0 + I, w0 + I + 32};
  f32x16 acc[4] = {};
  multiply<false, 4>(x + row * d, w, d, 2 * I, acc);
  f32x4 sum[4];
  add_waves<4>(acc, s, sum);
  const int r = threadIdx.x / 8, c = 4 * (threadIdx.x % 8);
  if (r >= t.n) return;   // (a row's 8 lanes together)
  const int64_t at = t.r0 + r;
#pragma unroll
  for (int hf = 0; hf < 2; ++hf) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max(abs_bits(sum[2 * hf][i]), abs_bits(sum[2 * hf + 1][i])));
    float sc, inv;
    keep_scale(__builtin_bit_cast(uint32_t, max8(__builtin_bit_cast(float, m))), sc, inv);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const f32x4& v = sum[2 * hf + b];
      *(uint32_t*)(kept.q + at * 2 * I + hf * I + n0 + 32 * b + c) = keep_codes4(v[0], v[1], v[2], v[3], inv);
    }
    if (c == 0) kept.s[(at * 2 + hf) * (I / kKeepBlock) + n0 / kKeepBlock] = sc;
  }
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    f32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float g = sum[b][i];
      v[i] = g / (1.f + expf(-g)) * sum[2 + b][i];
    }
    *(f32x4*)(h + at * I + n0 + 32 * b + c) = v;
  }
}

// out = a W: the down projection.
__global__ __launch_bounds__(kThreads) void k_small_product(const float* __restrict__ a,
                                                            const int32_t* __restrict__ offsets, int64_t max_rows,
                                                            int E, int K, int N, const float* __restrict__ w,
                                                            float* __restrict__ out) {
  __shared__ float s[1][kWaves][kRows * kCols];
  const Rows t = row_tile(offsets, max_rows, E, (int)blockIdx.x);
  if (t.n == 0) return;
  const int lane = threadIdx.x % kWave, n0 = kCols * (int)blockIdx.y;
  const float* const ws[1] = {w + (int64_t)t.e * K * N + n0 + lane % 32};
  f32x16 acc[1] = {};
  multiply<false, 1>(a + (int64_t)(t.r0 + min(lane % 32, t.n - 1)) * K, ws, K, N, acc);
  f32x4 sum[1];
  add_waves<1>(acc, s, sum);
  const int r = threadIdx.x / 8, c = 4 * (threadIdx.x % 8);
  if (r < t.n) *(f32x4*)(out + (int64_t)(t.r0 + r) * N + n0 + c) = sum[0];
}

// dgu = w [dg | du] and h = w silu(g) u of 32 rows and 32 columns of I from dh = dy
// Wd^T and the checkpoint, or (AGAIN) g | u = x Wgu computed beside it; dot
// (optional, [max_rows, I / 32]): the row's <dh, silu(g) u> over the columns.
template <bool AGAIN>
__global__ __launch_bounds__(kThreads) void k_small_down_bwd(
    const float* __restrict__ dy, const float* __restrict__ x, const int32_t* __restrict__ offsets, int64_t max_rows,
    int E, int d, int I, const float* __restrict__ wd, const float* __restrict__ wgu, Kept kept,
    const float* __restrict__ row_w, float* __restrict__ dgu, float* __restrict__ h, float* __restrict__ dot) {
  constexpr int NB = AGAIN ? 3 : 1;
  __shared__ float s[NB][kWaves][kRows * kCols];
  const Rows t = row_tile(offsets, max_rows, E, (int)blockIdx.x);
  if (t.n == 0) return;
  const int lane = threadIdx.x % kWave, n0 = kCols * (int)blockIdx.y;
  const int64_t mine = t.r0 + min(lane % 32, t.n - 1);
  f32x16 acc[NB] = {};
  {
    const float* const w[1] = {wd + ((int64_t)t.e * I + n0 + lane % 32) * d};
    f32x16 a[1] = {};
    multiply<true, 1>(dy + mine * d, w, d, 0, a);
    acc[0] = a[0];
  }
  if constexpr (AGAIN) {
    const float* w0 = wgu + (int64_t)t.e * d * 2 * I + n0 + lane % 32;
    const float* const w[2] = {w0, w0 + I};
    f32x16 a[2] = {};
    multiply<false, 2>(x + mine * d, w, d, 2 * I, a);
    acc[1] = a[0];
    acc[2] = a[1];
  }
  f32x4 sum[NB];
  add_waves<NB>(acc, s, sum);
  const int r = threadIdx.x / 8, c = n0 + 4 * (threadIdx.x % 8);
  if (r >= t.n) return;
  const int64_t at = t.r0 + r;
  float g[4], u[4];
  if constexpr (AGAIN) {
#pragma unroll
    for (int i = 0; i < 4; ++i) g[i] = sum[1][i], u[i] = sum[2][i];
  } else {
    const int nb = I / kKeepBlock;
    keep_values4(*(const uint32_t*)(kept.q + at * 2 * I + c), kept.s[at * 2 * nb + c / kKeepBlock], g);
    keep_values4(*(const uint32_t*)(kept.q + at * 2 * I + I + c), kept.s[at * 2 * nb + nb + c / kKeepBlock], u);
  }
  const float w = row_w ? row_w[at] : 1.f;
  f32x4 dg, du, hv;
  float part = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float dh = sum[0][i], sg = 1.f / (1.f + expf(-g[i])), silu = g[i] * sg, wdh = w * dh;
    part = fmaf(silu * u[i], dh, part);
    dg[i] = wdh * u[i] * (sg + silu * (1.f - sg));
    du[i] = wdh * silu;
    hv[i] = w * (silu * u[i]);
  }
  *(f32x4*)(dgu + at * 2 * I + c) = dg;
  *(f32x4*)(dgu + at * 2 * I + I + c) = du;
  *(f32x4*)(h + at * I + c) = hv;
  if (!dot) return;
#pragma unroll
  for (int off = 1; off < 8; off <<= 1) part += __shfl_xor(part, off, kWave);
  if (threadIdx.x % 8 == 0) dot[at * (I / kCols) + n0 / kCols] = part;
}

// One expert's dW = A^T B tile of 32 x 128, each wave 32 columns: matrix
// instruction kk takes rows 2 kk and 2 kk + 1 (lanes 0-31 and 32-63).
__device__ __forceinline__ void weight_tile(const float* __restrict__ a, int lda, int M, const float* __restrict__ b,
                                            int ldb, int N, int64_t lo, int cnt, int m0, int n0,
                                            float* __restrict__ out) {
  const int lane = threadIdx.x % kWave, n = n0 + 32 * (threadIdx.x / kWave) + lane % 32;
  if (n >= N) return;   // (the wave: N is a multiple of 32)
  constexpr int U = 8;
  f32x16 acc = {};
  for (int r0 = 0; r0 < cnt; r0 += 2 * U) {
    float av[U], bv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + 2 * u + lane / 32;
      const int64_t at = lo + min(r, cnt - 1);
      const float p = a[at * lda + m0 + lane % 32], q = b[at * ldb + n];
      av[u] = r < cnt ? p : 0.f;
      bv[u] = r < cnt ? q : 0.f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(av[u], bv[u], acc, 0, 0, 0);
  }
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    const int m = m0 + 8 * (q / 4) + 4 * (lane / 32) + q % 4;
    if (m < M) out[(int64_t)m * N + n] = acc[q];
  }
}

// The three gradients that read dgu and h, by workgroup: first the tiles of dx =
// dgu Wgu^T, then those of dWd = h^T dy and dWgu = x^T dgu, expert by expert.
__global__ __launch_bounds__(kThreads) void k_small_grads(
    const float* __restrict__ x, const float* __restrict__ dy, const float* __restrict__ h,
    const float* __restrict__ dgu, const int32_t* __restrict__ offsets, int64_t max_rows, int E, int d, int I,
    const float* __restrict__ wgu, float* __restrict__ dx, float* __restrict__ dwgu, float* __restrict__ dwd,
    int dx_blocks) {
  __shared__ float s[1][kWaves][kRows * kCols];
  const int lane = threadIdx.x % kWave;
  int b = (int)blockIdx.x;
  if (b < dx_blocks) {
    const int cols = d / kCols;
    const Rows t = row_tile(offsets, max_rows, E, b / cols);
    if (t.n == 0) return;
    const int n0 = kCols * (b % cols), K = 2 * I;
    const float* const w[1] = {wgu + ((int64_t)t.e * d + n0 + lane % 32) * K};
    f32x16 acc[1] = {};
    multiply<true, 1>(dgu + (int64_t)(t.r0 + min(lane % 32, t.n - 1)) * K, w, K, 0, acc);
    f32x4 sum[1];
    add_waves<1>(acc, s, sum);
    const int r = threadIdx.x / 8, c = 4 * (threadIdx.x % 8);
    if (r < t.n) *(f32x4*)(dx + (int64_t)(t.r0 + r) * d + n0 + c) = sum[0];
    return;
  }
  b -= dx_blocks;
  const int down_n = (d + 127) / 128, down = (I / 32) * down_n, up_n = (2 * I + 127) / 128;
  const int per_e = down + (d / 32) * up_n;
  const int e = b / per_e;
  b -= e * per_e;
  const int64_t lo = clampi<int64_t>(offsets[e], 0, max_rows);
  const int cnt = (int)(clampi<int64_t>(offsets[e + 1], lo, max_rows) - lo);
  if (b < down)
    weight_tile(h, I, I, dy, d, d, lo, cnt, 32 * (b / down_n), 128 * (b % down_n), dwd + (int64_t)e * I * d);
  else
    weight_tile(x, d, d, dgu, 2 * I, 2 * I, lo, cnt, 32 * ((b - down) / up_n), 128 * ((b - down) % up_n),
                dwgu + (int64_t)e * d * 2 * I);
}

unsigned row_tiles(int64_t max_rows, int E) { return (unsigned)(max_rows / kRows + std::min<int64_t>(E, max_rows)); }

}  // namespace

// Few tiles of 64 x 128, and few rows an expert (more of them where the tiles are
// fewest): a weight gradient's tile walks all of an expert's rows.  Measured (one step of moe_grouped_ffn_train and
// moe_grouped_ffn_backward, this way and with the 64 x 128 tiles, us): 128 rows, 8
// experts, 128 x 256: 31 and 70; 512, 16, 512 x 512: 83 and 153; 64, 16, 1024 x
// 1024: 201 and 332; 1024, 8, 512 x 1024: 228 and 264; above, 2048, 16, 512 x 512:
// 222 and 204; 2000, 2, 704 x 320: 272 and 221; 1000, 1, 1024 x 1024: 369 and 329.
// Of more than 128 rows an expert: 264, 2, 640 x 704: 81 and 181; 512, 1, 1024 x
// 512: 158 and 218; 1500, 3, 128 x 1024: 144 and 227; 2000, 8, 128 x 128: 61 and 83.
bool small_f32(int64_t max_rows, int E, int d, int I) {
  const int64_t tiles = max_rows / 64 + std::min<int64_t>(E, max_rows);
  const int width = d < I ? d : I;
  const int64_t t = tiles * ceil_div(width, 128);
  return ((max_rows <= 128 * (int64_t)E && t <= 160) || (max_rows <= 512 * (int64_t)E && t <= 64)) &&
         (int64_t)E * d * I <= ((int64_t)1 << 24);
}

hipError_t launch_small_gate_up_f32(const float* x, int64_t x_rows, const int32_t* row_token,
                                    const int32_t* expert_offsets, int64_t max_rows, int E, int d, int I,
                                    const float* w_gate_up, float* h, const Kept& kept, hipStream_t s) {
  k_small_gate_up<<<dim3(row_tiles(max_rows, E), I / 64), kThreads, 0, s>>>(x, x_rows, row_token, expert_offsets,
                                                                            max_rows, E, d, I, w_gate_up, h, kept);
  return hipGetLastError();
}

hipError_t launch_small_down_f32(const float* h, const int32_t* expert_offsets, int64_t max_rows, int E, int d, int I,
                                 const float* w_down, float* y, hipStream_t s) {
  k_small_product<<<dim3(row_tiles(max_rows, E), d / kCols), kThreads, 0, s>>>(h, expert_offsets, max_rows, E, I, d,
                                                                               w_down, y);
  return hipGetLastError();
}

hipError_t launch_small_grads_f32(const float* x, const float* dy, const int32_t* expert_offsets, int64_t max_rows,
                                  int E, int d, int I, const float* w_gate_up, const float* w_down, const Kept& kept,
                                  const float* row_w, float* dgu, float* h, float* dot, float* dx, float* dw_gate_up,
                                  float* dw_down, hipStream_t s) {
  const dim3 grid(row_tiles(max_rows, E), I / kCols);
  if (kept.q)
    k_small_down_bwd<false><<<grid, kThreads, 0, s>>>(dy, x, expert_offsets, max_rows, E, d, I, w_down, w_gate_up,
                                                      kept, row_w, dgu, h, dot);
  else
    k_small_down_bwd<true><<<grid, kThreads, 0, s>>>(dy, x, expert_offsets, max_rows, E, d, I, w_down, w_gate_up,
                                                     kept, row_w, dgu, h, dot);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t dx_blocks = (int64_t)row_tiles(max_rows, E) * (d / kCols);
  const int64_t per_e = (I / 32) * ceil_div(d, 128) + (d / 32) * ceil_div(2 * I, 128);
  k_small_grads<<<(unsigned)(dx_blocks + E * per_e), kThreads, 0, s>>>(x, dy, h, dgu, expert_offsets, max_rows, E, d,
                                                                        I, w_gate_up, dx, dw_gate_up, dw_down,
                                                                        (int)dx_blocks);
  return hipGetLastError();
}

}  // namespace tre
