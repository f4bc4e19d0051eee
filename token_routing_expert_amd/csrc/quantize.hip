// quantize.hip -- rows and expert weights to e4m3 codes with a float32 scale
// for each block of 128 (activations: a row's 128 columns; weights: 128 x 128).
// fp8.hpp has the arithmetic of a block.
// One pass: a block's values stay in registers between its maximum and its codes.
// Rows, measured: 8192 of 2880 bf16, 71.5 MB in 12.9 us, 5.5 TB/s (partly from the
// caches); 4093 of 1024 float32 4.7 us; 64 of 5120 bf16 3.3 us, a launch's length.
#include "fp8.hpp"

namespace tre {
namespace {

// max over 16 consecutive lanes: quads by lane permutation, then the other
// quad of the half row and the other half by mirroring
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true);   // lane ^ 1
  v = o > v ? o : v;
  o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true);            // lane ^ 2
  v = o > v ? o : v;
  o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, true);           // mirror in 8 lanes
  v = o > v ? o : v;
  o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, true);           // mirror in 16 lanes
  return o > v ? o : v;
}

// Eight consecutive elements as they are stored, and as floats.  (Loads and
// conversions stay apart: a conversion behind each load waits for it alone.)
// ONCE: non-temporal, for weights; activations were just written and are read
// from the caches (batch of 8192 rows: 12.8 us, non-temporal 13.9).
template <typename Elem>
struct Eight {
  u32x4 v[sizeof(Elem) / 2];
};

template <bool ONCE, typename Elem>
__device__ __forceinline__ Eight<Elem> load8(const Elem* p) {
  Eight<Elem> e;
#pragma unroll
  for (int i = 0; i < (int)sizeof(Elem) / 2; ++i)
    e.v[i] = ONCE ? __builtin_nontemporal_load((const u32x4*)p + i) : ((const u32x4*)p)[i];
  return e;
}

template <typename Elem>
__device__ __forceinline__ Eight<Elem> zero8() {
  Eight<Elem> e;
#pragma unroll
  for (int i = 0; i < (int)sizeof(Elem) / 2; ++i) e.v[i] = u32x4{0, 0, 0, 0};
  return e;
}

__device__ __forceinline__ void to_floats(const Eight<bf16_t>& e, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = e.v[0][i];
    f[2 * i] = __builtin_bit_cast(float, w << 16);
    f[2 * i + 1] = __builtin_bit_cast(float, w & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void to_floats(const Eight<float>& e, float (&f)[8]) {
  const f32x4 a = __builtin_bit_cast(f32x4, e.v[0]), b = __builtin_bit_cast(f32x4, e.v[1]);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = a[i], f[4 + i] = b[i];
}

// Rows: 16 lanes take a block, eight elements each, so a wave reads four
// blocks with 16-byte loads and one 4-step lane reduction finds all four
// maxima; nothing is kept but the eight elements.  kRowUnroll blocks a group
// keep several loads in flight.  Bound by HBM: one read of x, 1 byte written
// an element.
constexpr int kRowThreads = 256, kRowUnroll = 4;

template <typename Elem>
__global__ __launch_bounds__(kRowThreads) void k_quantize_rows(const Elem* __restrict__ x, uint32_t n_blocks, int cols,
                                                               int nb, uint8_t* __restrict__ q, int ldq,
                                                               float* __restrict__ scale) {
  const int l16 = threadIdx.x % 16;
  const uint32_t first = blockIdx.x * (kRowThreads / 16 * kRowUnroll) + threadIdx.x / 16;
  Eight<Elem> raw[kRowUnroll];
  int64_t at[kRowUnroll], to[kRowUnroll];
#pragma unroll
  for (int u = 0; u < kRowUnroll; ++u) {
    const uint32_t b = first + u * (kRowThreads / 16);
    const uint32_t row = b / (uint32_t)nb;
    const int c = (int)(b - row * nb) * kBlock + l16 * 8;
    at[u] = b < n_blocks && c < cols ? (int64_t)row * cols + c : -1;   // the last block may be half a block
    to[u] = (int64_t)row * ldq + c;
    raw[u] = zero8<Elem>();
    if (at[u] >= 0) raw[u] = load8<false>(x + at[u]);
  }
#pragma unroll
  for (int u = 0; u < kRowUnroll; ++u) {
    float v[8];
    to_floats(raw[u], v);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = abs_bits(v[i]) > m ? abs_bits(v[i]) : m;
    m = max16(m);
    float s, inv;
    bool finite;
    power_scale(m, s, inv, finite);
    const uint32_t b = first + u * (kRowThreads / 16);
    if (b < n_blocks && l16 == 0) scale[b] = s;
    if (at[u] >= 0) {
      const uint32_t lo = pack_fp8x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
      const uint32_t hi = pack_fp8x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
      *(uint2*)(q + to[u]) = finite ? make_uint2(lo, hi) : make_uint2(kNan8, kNan8);
    }
  }
}

// Weights: a workgroup takes one 128 x 128 block of a [K, N] matrix and writes
// it as [N, K].  Thread (c, r) = (tid % 16, tid / 16) reads columns 8 c .. +7
// of rows 8 r .. +7, so it holds eight consecutive k of eight n in registers:
// a code word of eight k for each n goes to LDS, and the block leaves as rows
// of 128 bytes.  Blocks 0, 1, 2 of a triple are gate, up and down: all three
// are ceil(I/128) x ceil(d/128) blocks, and one launch does the layer.
// Bound by memory through lines of 128 bytes (a code row of a block).  bf16, 16
// experts, 1024 x 2816: 415 MB in 67 to 71 us, 6 TB/s, past a copy's 4.7 (two
// thirds of it is read, and the codes partly stay in the last-level cache); 128
// experts, 2880 x 2880: 9.6 GB in 2.28 ms, 4.2 TB/s.  float32, 16 experts, 1024 x
// 2816: 692 MB in 133 us, 5.2 TB/s.
constexpr int kTileStride = kBlock + 4;    // bytes: 33 words, so that a wave's writes (8 rows apart) fill all banks

template <typename Elem>
__global__ __launch_bounds__(256) void k_quantize_weights(const Elem* __restrict__ wgu, const Elem* __restrict__ wd,
                                                          int d, int I, int db, int ib, uint8_t* __restrict__ gu_q,
                                                          float* __restrict__ gu_s, uint8_t* __restrict__ dn_q,
                                                          float* __restrict__ dn_s) {
  __shared__ __attribute__((aligned(16))) uint8_t tile[kBlock * kTileStride];
  __shared__ uint32_t s_max[4];
  const int tid = threadIdx.x;
  const int j = blockIdx.x % (db * ib), which = (int)blockIdx.y;
  const int64_t e = blockIdx.x / (db * ib);
  const int bd = j % db, bi = j / db;                       // block of d, block of I
  const bool down = which == 2;
  // source block: rows k0 .. of K, columns n0 .. of ld; destination rows n0d
  const int K = down ? I : d, N = down ? d : I, ld = down ? d : 2 * I;
  const int k0 = (down ? bi : bd) * kBlock, n0 = (down ? bd : bi) * kBlock;
  const Elem* src = (down ? wd + e * I * d : wgu + e * d * 2 * I + (which ? I : 0)) + (int64_t)k0 * ld + n0;
  uint8_t* dst = (down ? dn_q + e * d * I : gu_q + e * 2 * I * d + (which ? (int64_t)I * d : 0)) + (int64_t)n0 * K + k0;
  float* sdst = down ? dn_s + (e * db + bd) * ib + bi : gu_s + ((e * 2 + which) * ib + bi) * db + bd;
  const int nk = K - k0 < kBlock ? K - k0 : kBlock, nn = N - n0 < kBlock ? N - n0 : kBlock;
  const int c = tid % 16 * 8, r = tid / 16 * 8;
  const bool in = c < nn && r < nk;                         // both are multiples of 64: all eight or none
  Eight<Elem> raw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) raw[i] = zero8<Elem>();
  if (in) {
#pragma unroll
    for (int i = 0; i < 8; ++i) raw[i] = load8<true>(src + (int64_t)(r + i) * ld + c);
  }
  float f[8][8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) to_floats(raw[i], f[i]);
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int v = 0; v < 8; ++v) m = abs_bits(f[i][v]) > m ? abs_bits(f[i][v]) : m;
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    const uint32_t o = __shfl_xor(m, off, kWave);
    m = o > m ? o : m;
  }
  if (tid % kWave == 0) s_max[tid / kWave] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 4; ++w) m = s_max[w] > m ? s_max[w] : m;
  float s, inv;
  bool finite;
  power_scale(m, s, inv, finite);
  if (tid == 0) *sdst = s;
  if (in) {
#pragma unroll
    for (int v = 0; v < 8; ++v) {
      const uint32_t lo = pack_fp8x4(f[0][v] * inv, f[1][v] * inv, f[2][v] * inv, f[3][v] * inv);
      const uint32_t hi = pack_fp8x4(f[4][v] * inv, f[5][v] * inv, f[6][v] * inv, f[7][v] * inv);
      uint32_t* to = (uint32_t*)(tile + (c + v) * kTileStride + r);
      to[0] = finite ? lo : kNan8;
      to[1] = finite ? hi : kNan8;
    }
  }
  __syncthreads();
#pragma unroll
  for (int p = 0; p < kBlock * kBlock / 16 / 256; ++p) {
    const int n = p * 32 + tid / 8, k = tid % 8 * 16;
    const uint32_t* from = (const uint32_t*)(tile + n * kTileStride + k);
    if (n < nn && k < nk) *(u32x4*)(dst + (int64_t)n * K + k) = u32x4{from[0], from[1], from[2], from[3]};
  }
}

template <typename Elem>
hipError_t rows(const Elem* x, int64_t n, int cols, uint8_t* q, int ldq, float* scale, hipStream_t s) {
  const int nb = (int)ceil_div(cols, kBlock);
  const int64_t blocks = n * nb;
  k_quantize_rows<Elem><<<(unsigned)ceil_div(blocks, kRowThreads / 16 * kRowUnroll), kRowThreads, 0, s>>>(
      x, (uint32_t)blocks, cols, nb, q, ldq, scale);
  return hipGetLastError();
}

template <typename Elem>
hipError_t weights(const Elem* wgu, const Elem* wd, int E, int d, int I, uint8_t* gu_q, float* gu_s, uint8_t* dn_q,
                   float* dn_s, hipStream_t s) {
  const int db = (int)ceil_div(d, kBlock), ib = (int)ceil_div(I, kBlock);
  k_quantize_weights<Elem><<<dim3((unsigned)((int64_t)E * db * ib), 3), 256, 0, s>>>(wgu, wd, d, I, db, ib, gu_q, gu_s,
                                                                                   dn_q, dn_s);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_rows_bf16(const bf16_t* x, int64_t n, int cols, uint8_t* q, int ldq, float* scale,
                                     hipStream_t s) {
  return rows(x, n, cols, q, ldq, scale, s);
}
hipError_t launch_quantize_rows_f32(const float* x, int64_t n, int cols, uint8_t* q, int ldq, float* scale,
                                    hipStream_t s) {
  return rows(x, n, cols, q, ldq, scale, s);
}
hipError_t launch_quantize_weights_bf16(const bf16_t* wgu, const bf16_t* wd, int E, int d, int I, uint8_t* gu_q,
                                        float* gu_s, uint8_t* dn_q, float* dn_s, hipStream_t s) {
  return weights(wgu, wd, E, d, I, gu_q, gu_s, dn_q, dn_s, s);
}
hipError_t launch_quantize_weights_f32(const float* wgu, const float* wd, int E, int d, int I, uint8_t* gu_q,
                                       float* gu_s, uint8_t* dn_q, float* dn_s, hipStream_t s) {
  return weights(wgu, wd, E, d, I, gu_q, gu_s, dn_q, dn_s, s);
}

}  // namespace tre
