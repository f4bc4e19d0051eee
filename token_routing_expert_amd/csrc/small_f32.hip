// small_f32.hip -- the training operators' products where the tiles of the other
// kernels are too few for the card: in float32, of float32 or bf16 operands (T),
// with h, dg and du float32 between them in either type.
//
// A workgroup takes 32 rows of one expert and 32 columns (gate/up: 64 gate and
// the 64 up columns beside them) and its eight waves share the summed dimension:
// 8 values in turn, so a wave's operands are 16 bytes a lane, straight from
// memory to registers, with no stages to wait for one another.  The order of k
// inside v_mfma_f32_32x32x2_f32 is free as long as both operands use the same:
// lane i + 32 k of matrix instruction m holds element 4 k + m of the 8.  The
// partial tiles are added in LDS in a fixed order (equal calls give equal bits), and
// the sums come out as four consecutive columns of one row a thread.
//
// What such a call costs is its launches and one memory round trip each, so the
// steps are few: the SwiGLU backward sits behind dh (with g | u computed again
// beside it where there is no checkpoint), and dx and both weight gradients, which
// do not read one another, are one launch.  Measured: at
// small_products below.
#include "keep8.hpp"

#include <algorithm>

namespace tre {
namespace {

constexpr int kThreads = 512, kWaves = kThreads / kWave, kHalf = kWaves / 2;
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

// Four consecutive elements, or one, as float32; and back, rounded once.
__device__ __forceinline__ f32x4 load4(const float* p) { return *(const f32x4*)p; }
__device__ __forceinline__ f32x4 load4(const bf16_t* p) {
  const uint2 v = *(const uint2*)p;
  return f32x4{bf16_to_f32((bf16_t)(v.x & 0xffff)), bf16_to_f32((bf16_t)(v.x >> 16)),
               bf16_to_f32((bf16_t)(v.y & 0xffff)), bf16_to_f32((bf16_t)(v.y >> 16))};
}
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const bf16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ void store4(float* p, const f32x4& v) { *(f32x4*)p = v; }
__device__ __forceinline__ void store4(bf16_t* p, const f32x4& v) {
  *(uint2*)p = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

// acc[b] += this wave's share of A W over K, for column blocks at w[b].  a: the
// lane's row (row lane % 32 of the tile).  BT: W is [N][K] and w[b] the lane's row
// of it; else W is [K][ldw] and w[b] column lane % 32 of the block.
template <bool BT, int NB, typename A, typename W>
__device__ __forceinline__ void multiply(const A* __restrict__ a, const W* const (&w)[NB], int K, int ldw,
                                         f32x16 (&acc)[NB]) {
  const int wave = threadIdx.x / kWave, kh = (threadIdx.x % kWave) / 32;
  constexpr int U = NB > 2 && !BT ? 2 : 4;   // chunks of 8 whose loads go out together
  for (int k0 = 8 * wave; k0 < K; k0 += 8 * kWaves * U) {
    f32x4 av[U], wv[U][NB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + 8 * kWaves * u + 4 * kh;
      if (k0 + 8 * kWaves * u >= K) continue;   // (wave-uniform)
      av[u] = load4(a + k);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        if constexpr (BT) {
          wv[u][b] = load4(w[b] + k);
        } else {
#pragma unroll
          for (int m = 0; m < 4; ++m) wv[u][b][m] = load1(w[b] + (int64_t)(k + m) * ldw);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k0 + 8 * kWaves * u >= K) continue;
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int b = 0; b < NB; ++b)
          acc[b] = __builtin_amdgcn_mfma_f32_32x32x2f32(av[u][m], wv[u][b][m], acc[b], 0, 0, 0);
    }
  }
}

// Where a lane's 16 sums of a 32 x 32 block lie in it.
__device__ __forceinline__ int block_at(int q) {
  const int lane = threadIdx.x % kWave;
  return (8 * (q / 4) + 4 * (lane / 32) + q % 4) * kCols + lane % 32;
}

// The waves' partial tiles added, those of the upper half of the waves first to the
// lower half's: thread t < 256 gets row t / 8, columns 4 (t % 8) .. +3 of every block.
template <int NB>
__device__ __forceinline__ void add_waves(f32x16 (&acc)[NB], float (&s)[NB][kHalf][kRows * kCols],
                                          f32x4 (&sum)[NB]) {
  const int tid = threadIdx.x, wave = tid / kWave;
#pragma unroll
  for (int half = 1; half >= 0; --half) {
    if (wave / kHalf == half) {
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          float& at = s[b][wave % kHalf][block_at(q)];
          at = half ? acc[b][q] : at + acc[b][q];
        }
    }
    __syncthreads();
  }
  if (tid >= kRows * kCols / 4) return;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    sum[b] = *(const f32x4*)&s[b][0][4 * tid];
#pragma unroll
    for (int w = 1; w < kHalf; ++w) sum[b] += *(const f32x4*)&s[b][w][4 * tid];
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
template <typename T>
__global__ __launch_bounds__(kThreads) void k_small_gate_up(const T* __restrict__ x, int64_t x_rows,
                                                            const int32_t* __restrict__ row_token,
                                                            const int32_t* __restrict__ offsets, int64_t max_rows,
                                                            int E, int d, int I, const T* __restrict__ wgu,
                                                            float* __restrict__ h, Kept kept) {
  __shared__ float s[4][kHalf][kRows * kCols];
  const Rows t = row_tile(offsets, max_rows, E, (int)blockIdx.x);
  if (t.n == 0) return;   // (the whole workgroup)
  const int lane = threadIdx.x % kWave, n0 = 64 * (int)blockIdx.y;
  int64_t row = t.r0 + min(lane % 32, t.n - 1);
  if (row_token) {
    const int64_t tok = row_token[row];
    MOE_DCHECK(tok >= 0 && tok < x_rows);
    row = clampi<int64_t>(tok, 0, x_rows - 1);
  }
  const T* w0 = wgu + (int64_t)t.e * d * 2 * I + n0 + lane % 32;
  const T* const w[4] = {w0, w0 + 32, w0 + I, w0 + I + 32};
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

// out = h W: the down projection, in T or (a layer's bf16 rows) float32.
template <typename T, typename O>
__global__ __launch_bounds__(kThreads) void k_small_product(const float* __restrict__ a,
                                                            const int32_t* __restrict__ offsets, int64_t max_rows,
                                                            int E, int K, int N, const T* __restrict__ w,
                                                            O* __restrict__ out) {
  __shared__ float s[1][kHalf][kRows * kCols];
  const Rows t = row_tile(offsets, max_rows, E, (int)blockIdx.x);
  if (t.n == 0) return;
  const int lane = threadIdx.x % kWave, n0 = kCols * (int)blockIdx.y;
  const T* const ws[1] = {w + (int64_t)t.e * K * N + n0 + lane % 32};
  f32x16 acc[1] = {};
  multiply<false, 1>(a + (int64_t)(t.r0 + min(lane % 32, t.n - 1)) * K, ws, K, N, acc);
  f32x4 sum[1];
  add_waves<1>(acc, s, sum);
  const int r = threadIdx.x / 8, c = 4 * (threadIdx.x % 8);
  if (r < t.n) store4(out + (int64_t)(t.r0 + r) * N + n0 + c, sum[0]);
}

// dgu = w [dg | du] and h = w silu(g) u of 32 rows and 32 columns of I from dh = dy
// Wd^T and the checkpoint (FROM: its bits, 8 or 16), or (FROM 0) g | u = x Wgu
// computed beside it; dot
// (optional, [max_rows, I / 32]): the row's <dh, silu(g) u> over the columns.
template <typename T, int FROM>
__global__ __launch_bounds__(kThreads) void k_small_down_bwd(
    const T* __restrict__ dy, const T* __restrict__ x, const int32_t* __restrict__ offsets, int64_t max_rows,
    int E, int d, int I, const T* __restrict__ wd, const T* __restrict__ wgu, Kept kept,
    const float* __restrict__ row_w, float* __restrict__ dgu, float* __restrict__ h, float* __restrict__ dot) {
  constexpr bool AGAIN = FROM == 0;
  constexpr int NB = AGAIN ? 3 : 1;
  __shared__ float s[NB][kHalf][kRows * kCols];
  const Rows t = row_tile(offsets, max_rows, E, (int)blockIdx.x);
  if (t.n == 0) return;
  const int lane = threadIdx.x % kWave, n0 = kCols * (int)blockIdx.y;
  const int64_t mine = t.r0 + min(lane % 32, t.n - 1);
  f32x16 acc[NB] = {};
  {
    const T* const w[1] = {wd + ((int64_t)t.e * I + n0 + lane % 32) * d};
    f32x16 a[1] = {};
    multiply<true, 1>(dy + mine * d, w, d, 0, a);
    acc[0] = a[0];
  }
  if constexpr (AGAIN) {
    const T* w0 = wgu + (int64_t)t.e * d * 2 * I + n0 + lane % 32;
    const T* const w[2] = {w0, w0 + I};
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
    const int64_t q = at * 2 * I + c, b = at * 2 * nb + c / kKeepBlock;
    if constexpr (FROM == 8) {
      keep_values4(*(const uint32_t*)(kept.q + q), kept.s[b], g);
      keep_values4(*(const uint32_t*)(kept.q + q + I), kept.s[b + nb], u);
    } else {
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        keep_values2(*(const uint32_t*)(kept.q + 2 * (q + i)), kept.s[b], g + i);
        keep_values2(*(const uint32_t*)(kept.q + 2 * (q + I + i)), kept.s[b + nb], u + i);
      }
    }
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

// One expert's dW = A^T B tile of 32 x 128: wave w the 32 columns w % 4 of every
// other 16 rows; matrix instruction kk takes rows 2 kk and 2 kk + 1 (lanes 0-31 and
// 32-63).
template <typename A, typename B, typename T>
__device__ __forceinline__ void weight_tile(const A* __restrict__ a, int lda, const B* __restrict__ b, int ldb, int N,
                                            int64_t lo, int cnt, int m0, int n0,
                                            float (&s)[1][kHalf][kRows * kCols], T* __restrict__ out) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, n = n0 + 32 * (wave % kHalf) + lane % 32;
  const bool upper = wave >= kHalf, live = n < N;   // (the wave's: N is a multiple of 32)
  constexpr int U = 8;
  f32x16 acc = {};
  for (int r0 = upper ? 2 * U : 0; live && r0 < cnt; r0 += 4 * U) {
    float av[U], bv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + 2 * u + lane / 32;
      const int64_t at = lo + min(r, cnt - 1);
      const float p = load1(a + at * lda + m0 + lane % 32), q = load1(b + at * ldb + n);
      av[u] = r < cnt ? p : 0.f;
      bv[u] = r < cnt ? q : 0.f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(av[u], bv[u], acc, 0, 0, 0);
  }
  // a thread stores 8 of a row's 128 columns
#pragma unroll
  for (int half = 1; half >= 0; --half) {
    if (upper == (half == 1))
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        float& at = s[0][wave % kHalf][block_at(q)];
        at = half ? acc[q] : at + acc[q];
      }
    __syncthreads();
  }
  const int r = threadIdx.x / 16, c = 8 * (threadIdx.x % 16);
  if (n0 + c >= N) return;
  const float* v = &s[0][c / kCols][r * kCols + c % kCols];
  T* at = out + (int64_t)(m0 + r) * N + n0 + c;
  store4(at, *(const f32x4*)v);
  store4(at + 4, *(const f32x4*)(v + 4));
}

// The three gradients that read dgu and h, by workgroup: first the tiles of dx =
// dgu Wgu^T, then those of dWd = h^T dy and dWgu = x^T dgu, expert by expert.
template <typename T, typename O>
__global__ __launch_bounds__(kThreads) void k_small_grads(
    const T* __restrict__ x, const T* __restrict__ dy, const float* __restrict__ h,
    const float* __restrict__ dgu, const int32_t* __restrict__ offsets, int64_t max_rows, int E, int d, int I,
    const T* __restrict__ wgu, O* __restrict__ dx, T* __restrict__ dwgu, T* __restrict__ dwd, int dx_blocks) {
  __shared__ float s[1][kHalf][kRows * kCols];
  const int lane = threadIdx.x % kWave;
  int b = (int)blockIdx.x;
  if (b < dx_blocks) {
    const int cols = d / kCols;
    const Rows t = row_tile(offsets, max_rows, E, b / cols);
    if (t.n == 0) return;
    const int n0 = kCols * (b % cols), K = 2 * I;
    const T* const w[1] = {wgu + ((int64_t)t.e * d + n0 + lane % 32) * K};
    f32x16 acc[1] = {};
    multiply<true, 1>(dgu + (int64_t)(t.r0 + min(lane % 32, t.n - 1)) * K, w, K, 0, acc);
    f32x4 sum[1];
    add_waves<1>(acc, s, sum);
    const int r = threadIdx.x / 8, c = 4 * (threadIdx.x % 8);
    if (r < t.n) store4(dx + (int64_t)(t.r0 + r) * d + n0 + c, sum[0]);
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
    weight_tile(h, I, dy, d, d, lo, cnt, 32 * (b / down_n), 128 * (b % down_n), s, dwd + (int64_t)e * I * d);
  else
    weight_tile(x, d, dgu, 2 * I, 2 * I, lo, cnt, 32 * ((b - down) / up_n), 128 * ((b - down) % up_n), s,
                dwgu + (int64_t)e * d * 2 * I);
}

unsigned row_tiles(int64_t max_rows, int E) { return (unsigned)(max_rows / kRows + std::min<int64_t>(E, max_rows)); }

}  // namespace

// Few tiles of 64 x 128, and few rows an expert (more of them where the tiles are
// fewest): a weight gradient's tile walks all of an expert's rows.
// Measured (one step of moe_grouped_ffn_train and moe_grouped_ffn_backward, this
// way and the other, us; rows, experts, d x I).
// float32: 128, 8, 128 x 256: 33 and 70; 512, 16, 512 x 512: 87 and 153; 64, 16,
// 1024 x 1024: 200 and 332; 1024, 8, 512 x 1024: 221 and 264; 264, 2, 640 x 704: 78
// and 181; 2000, 8, 128 x 128: 49 and 83; 2000, 4, 256 x 256: 92 and 132; 1000, 1,
// 512 x 512: 148 and 223; above, 2000, 2, 704 x 320: 216 and 222; 2048, 16, 512 x
// 512: 218 and 204; 1000, 1, 1024 x 1024: 350 and 328.
// bf16, whose other kernels multiply 16 times as fast, but in stages of more rows
// and columns: 128, 8, 128 x 256: 33 and 50; 2000, 8, 128 x 128: 49 and 85; 400, 1,
// 512 x 512: 75 and 103; 264, 2, 640 x 704: 74 and 109; 10, 60, 512 x 512: 63 and
// 106; 30, 100, 256 x 384: 52 and 129; above, 512, 16, 512 x 512: 88 and 82; 100,
// 1, 1024 x 1024: 88 and 77; 1500, 3, 128 x 1024: 116 and 99.
// The least bf16 calls come here too where that costs little: rounding h, dg
// and du to bf16 makes the outputs' error 1.4 times their own rounding's where many
// roundings average out, but up to 1.55 times by chance over a few hundred values.
// A workgroup walks the longest sum, d or 2 I terms, by itself (9 ns a term), where
// the other kernels cut it into ranges; they in turn write the zero gradients of
// experts without rows at half the rate.  Rows, experts, d x I, this way and the
// other: 8, 128, 1024 x 1024: 291 and 680; 37, 11, 832 x 64: 41 and 63; 64, 1, 2880
// x 64: 61 and 54; the dearest, 64, 1, 64 x 2880: 98 and 63; 1, 8, 8192 x 8192: 1353
// and 2563; above, 16, 1, 8192 x 128: 114 and 78; 16, 1, 128 x 8192: 209 and 89; 1, 1,
// 512 x 65536: 2300 and 451.
bool small_products(int64_t max_rows, int E, int d, int I, bool bf16) {
  const int64_t tiles = max_rows / 64 + std::min<int64_t>(E, max_rows);
  const int width = std::min(d, I);
  const int64_t t = tiles * ceil_div(width, 128);
  if (bf16)   // (2^32: the weight gradients' tiles have to fit a grid of 2^32 threads)
    return (max_rows * width <= 8192 && (int64_t)E * d * I <= ((int64_t)1 << 32) &&
            std::max<int64_t>(d, 2 * (int64_t)I) <= 6000 + std::max<int64_t>(E - max_rows, 0) * d * I / 3000) ||
           (max_rows <= 400 * (int64_t)E && t <= 64 && std::max(d, I) <= 768);
  return ((max_rows <= 128 * (int64_t)E && t <= 160) || (max_rows <= 1024 * (int64_t)E && t <= 80)) &&
         (int64_t)E * d * I <= ((int64_t)1 << 24);
}

template <typename T>
hipError_t launch_small_gate_up(const T* x, int64_t x_rows, const int32_t* row_token, const int32_t* expert_offsets,
                                int64_t max_rows, int E, int d, int I, const T* w_gate_up, float* h, const Kept& kept,
                                hipStream_t s) {
  k_small_gate_up<T><<<dim3(row_tiles(max_rows, E), I / 64), kThreads, 0, s>>>(x, x_rows, row_token, expert_offsets,
                                                                               max_rows, E, d, I, w_gate_up, h, kept);
  return hipGetLastError();
}

template <typename T, typename O>
hipError_t launch_small_down(const float* h, const int32_t* expert_offsets, int64_t max_rows, int E, int d, int I,
                             const T* w_down, O* y, hipStream_t s) {
  k_small_product<T, O><<<dim3(row_tiles(max_rows, E), d / kCols), kThreads, 0, s>>>(h, expert_offsets, max_rows, E, I,
                                                                                     d, w_down, y);
  return hipGetLastError();
}

template <typename T, typename O>
hipError_t launch_small_grads(const T* x, const T* dy, const int32_t* expert_offsets, int64_t max_rows, int E, int d,
                              int I, const T* w_gate_up, const T* w_down, const Kept& kept, int bits,
                              const float* row_w, float* dgu, float* h, float* dot, O* dx, T* dw_gate_up, T* dw_down,
                              hipStream_t s) {
  const dim3 grid(row_tiles(max_rows, E), I / kCols);
  auto down = kept.q ? k_small_down_bwd<T, 8> : k_small_down_bwd<T, 0>;
  if constexpr (sizeof(T) == 2)
    if (bits == 16) down = k_small_down_bwd<T, 16>;
  down<<<grid, kThreads, 0, s>>>(dy, x, expert_offsets, max_rows, E, d, I, w_down, w_gate_up, kept, row_w, dgu, h, dot);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t dx_blocks = (int64_t)row_tiles(max_rows, E) * (d / kCols);
  const int64_t per_e = (I / 32) * ceil_div(d, 128) + (d / 32) * ceil_div(2 * I, 128);
  k_small_grads<T, O><<<(unsigned)(dx_blocks + E * per_e), kThreads, 0, s>>>(
      x, dy, h, dgu, expert_offsets, max_rows, E, d, I, w_gate_up, dx, dw_gate_up, dw_down, (int)dx_blocks);
  return hipGetLastError();
}

#define SMALL_GATE_UP(T)                                                                                             \
  template hipError_t launch_small_gate_up<T>(const T*, int64_t, const int32_t*, const int32_t*, int64_t, int, int,  \
                                              int, const T*, float*, const Kept&, hipStream_t);
#define SMALL_ROWS(T, O)                                                                                            \
  template hipError_t launch_small_down<T, O>(const float*, const int32_t*, int64_t, int, int, int, const T*, O*,   \
                                              hipStream_t);                                                         \
  template hipError_t launch_small_grads<T, O>(const T*, const T*, const int32_t*, int64_t, int, int, int, const T*, \
                                               const T*, const Kept&, int, const float*, float*, float*, float*, O*, T*, \
                                               T*, hipStream_t);
SMALL_GATE_UP(float)
SMALL_GATE_UP(bf16_t)
SMALL_ROWS(float, float)
SMALL_ROWS(bf16_t, bf16_t)
SMALL_ROWS(bf16_t, float)

}  // namespace tre
