// fp8_ffn.hip -- the grouped products on e4m3 rows and expert weights with a
// float32 scale for each block of 128, on v_mfma_f32_16x16x128_f8f6f4.
//
// For row r of expert e and output column n, blocks b of 128 k:
//   sum_b xs[r, b] ws[e, n / 128, b] * (sum_{k in b} xq[r, k] wq[e, n, k])
// One matrix instruction covers a block of k exactly, so a block's sums leave
// it unscaled (its addend is the constant zero) and are added to the float32
// accumulators with one multiplied-add an element: four vector instructions
// beside each matrix instruction of 32 cycles, in the shadow of the other
// waves' matrix work.
//
// Tile: BM rows x 256 weight rows, one block of 128 bytes of k a stage, both
// operands loaded straight to LDS (16-byte chunk c of row r in slot
// c ^ (r & 7), so that consecutive rows of one chunk fall into different
// banks), two stages: the next one loads while this one multiplies.  Weights
// are the instruction's first operand, so a lane ends up with four consecutive
// columns of one row and needs one row scale a fragment.  The row's scales and
// the tile's weight scales ride along in the stage.
//   - gate/up: 128 columns of h a tile -- one quantisation block.  A wave holds
//     the gate and up sums of the same columns, so SwiGLU stays in registers;
//     the waves exchange the block's largest magnitude through LDS and write
//     codes: h never exists in more than 8 bits.
//   - Row fragments (16 rows) are dealt to the waves round-robin and a wave
//     multiplies only those that hold rows, so a partly filled tile costs what
//     its rows cost (beyond the weights' loads).
// XCDs: consecutive tiles go to one XCD, in groups of up to 8 row tiles for
// each weight slice, so that a slice is fetched once for the group and the
// group's rows stay in that XCD's L2.
#include "fp8.hpp"

namespace tre {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kThreads8 = 512, kBN = 256, kStageK = 128;
constexpr int kXcds = 8;                         // workgroups are dealt round-robin over the XCDs
constexpr int kGroupM = 8;                       // row tiles of a weight slice that run together
constexpr uint32_t kPark = 0x80000000u;          // past every buffer: reads zeros

struct Gemm8Args {
  const uint8_t* a;          // rows [*, K]
  const float* a_s;          // [*, KB]
  const int32_t* row_token;  // gathered rows, or null
  int64_t a_rows;            // rows of a
  const int32_t* offsets;
  int64_t max_rows;
  int E, K, N;               // N: output columns (gate/up: I)
  const uint8_t* w;          // [E, NW, K], NW = 2 N for gate/up
  const float* w_s;
  void* out;                 // gate/up: codes [max_rows, N]; down: bf16 [max_rows, N]
  float* out_s;              // gate/up: [max_rows, NB]
};

// One dword a lane, straight to LDS at lds_base + 4 * lane.
__device__ __forceinline__ void dma4s(__amdgpu_buffer_rsrc_t rsrc, uint32_t lds_base, uint32_t voffset,
                                      uint32_t soffset) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dword %1, %2, %3 offen lds"
               :
               : "s"(lds_base), "v"(voffset), "s"(rsrc), "s"(soffset)
               : "memory");
}

template <int BM>
struct Stage8 {
  uint8_t a[BM * kStageK];
  uint8_t b[kBN * kStageK];
  float as[BM < 64 ? 64 : BM];
  float bs[64];              // [0], [1]: the tile's two weight blocks
};

// 32 bytes of k for one row of an operand: chunks q and q + 4 of the row (the
// same k for both operands, in an order of no consequence to the sum).
__device__ __forceinline__ i32x8 operand8(const uint8_t* tile, int row, int q) {
  const uint8_t* p = tile + row * kStageK + ((q ^ (row & 7)) * 16);
  const u32x4 lo = *(const u32x4*)p, hi = *(const u32x4*)(tile + row * kStageK + (((q + 4) ^ (row & 7)) * 16));
  return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

__device__ __forceinline__ f32x4 mfma8(i32x8 a, i32x8 b) {
  // both operands e4m3 (format 0); zero scale operands select the form without scales
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

template <bool GATE_UP, int BM, int WM>
__global__ __launch_bounds__(kThreads8) void k_gemm8(Gemm8Args g) {
  constexpr int NW = kThreads8 / kWave, WN = NW / WM, MF = BM / 16 / WM, NF = kBN / 16 / WN, BW = kBN / WN;
  constexpr int TN = GATE_UP ? kBN / 2 : kBN;      // output columns of a tile
  constexpr int A_LOADS = BM / 8, B_LOADS = kBN / 8;   // 1 KB loads of a stage
  constexpr int A_PER = (A_LOADS + NW - 1) / NW, B_PER = B_LOADS / NW;
  __shared__ __attribute__((aligned(1024))) Stage8<BM> st[2];
  __shared__ int s_tiles[kMaxExperts];
  __shared__ int s_found[4];
  __shared__ int s_total;
  const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int n_tiles = (g.N + TN - 1) / TN;

  // ---- which tile: experts' row tiles counted from the offsets
  if (tid < kMaxExperts) {
    int n = 0;
    if (tid < g.E) {
      const int64_t r0 = clampi<int64_t>(g.offsets[tid], 0, g.max_rows);
      const int64_t r1 = clampi<int64_t>(g.offsets[tid + 1], r0, g.max_rows);
      n = (int)((r1 - r0 + BM - 1) / BM);
    }
    // inclusive scan over the experts: in the wave, then over the four waves
    int x = n;
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
      const int y = __shfl_up(x, off, kWave);
      if (lane >= off) x += y;
    }
    s_tiles[tid] = x;
  }
  __syncthreads();
  int before = 0;
  if (tid < kMaxExperts) {
    for (int w = 0; w < wave; ++w) before += s_tiles[w * kWave + kWave - 1];
    if (tid == kMaxExperts - 1) s_total = before + s_tiles[tid];
  }
  __syncthreads();
  const int64_t total = (int64_t)s_total * n_tiles, per = (total + kXcds - 1) / kXcds;
  const int64_t mine = blockIdx.x / kXcds, tile = (blockIdx.x % kXcds) * per + mine;
  if (mine >= per || tile >= total) return;
  if (tid < kMaxExperts) {
    const int64_t hi = (int64_t)(before + s_tiles[tid]) * n_tiles;
    const int64_t lo = (int64_t)(before + (lane ? s_tiles[tid - 1] : 0)) * n_tiles;
    if (tile >= lo && tile < hi) {
      const int m_tiles = (int)((hi - lo) / n_tiles), at = (int)(tile - lo);
      const int group = at / (kGroupM * n_tiles), in = at - group * (kGroupM * n_tiles);
      const int wide = m_tiles - group * kGroupM < kGroupM ? m_tiles - group * kGroupM : kGroupM;
      s_found[0] = tid;
      s_found[1] = group * kGroupM + in % wide;
      s_found[2] = in / wide;
    }
  }
  __syncthreads();
  const int e = __builtin_amdgcn_readfirstlane(s_found[0]), mt = __builtin_amdgcn_readfirstlane(s_found[1]),
            n0 = __builtin_amdgcn_readfirstlane(s_found[2]) * TN;
  const int64_t first = clampi<int64_t>(g.offsets[e], 0, g.max_rows);
  const int64_t last = clampi<int64_t>(g.offsets[e + 1], first, g.max_rows);
  const int64_t row0 = first + (int64_t)mt * BM;
  const int rows = (int)(last - row0 < BM ? last - row0 : BM);

  // ---- operands
  const int K = g.K, KB = (K + 127) / 128, steps = KB;
  const bool tail = K % 128 != 0;                    // the last stage has half a block
  const int chunk = (lane & 7) ^ (lane >> 3);        // the 16 bytes of a row this lane loads
  const bool gather = g.row_token != nullptr;
  const uint8_t* a_base = gather ? g.a : g.a + row0 * K;
  const float* as_base = gather ? g.a_s : g.a_s + row0 * KB;
  const int64_t a_span = gather ? g.a_rows : rows;
  const __amdgpu_buffer_rsrc_t a_rsrc =
      __builtin_amdgcn_make_buffer_rsrc(uniform_ptr(a_base), (short)0, (int)(a_span * K), kBufferConfig);
  const __amdgpu_buffer_rsrc_t as_rsrc =
      __builtin_amdgcn_make_buffer_rsrc(uniform_ptr(as_base), (short)0, (int)(a_span * KB * 4), kBufferConfig);
  const int64_t w_rows = GATE_UP ? 2 * (int64_t)g.N : g.N;
  const __amdgpu_buffer_rsrc_t w_rsrc = __builtin_amdgcn_make_buffer_rsrc(
      uniform_ptr(g.w + e * w_rows * K), (short)0, (int)(w_rows * K), kBufferConfig);
  const int NB = (g.N + 127) / 128;
  const int64_t ws_rows = GATE_UP ? 2 * NB : NB;
  const __amdgpu_buffer_rsrc_t ws_rsrc = __builtin_amdgcn_make_buffer_rsrc(
      uniform_ptr(g.w_s + e * ws_rows * KB), (short)0, (int)(ws_rows * KB * 4), kBufferConfig);
  // row of `a` behind the tile's row r, or -1
  auto source_row = [&](int r) -> int64_t {
    if (r >= rows) return -1;
    if (!gather) return r;
    const int64_t t = g.row_token[row0 + r];
    MOE_DCHECK(t >= 0 && t < g.a_rows);
    return t >= 0 && t < g.a_rows ? t : -1;
  };
  uint32_t a_off[A_PER], b_off[B_PER], as_off = kPark, bs_off = kPark;
#pragma unroll
  for (int p = 0; p < A_PER; ++p) {
    const int i = wave + NW * p;
    const int64_t r = i < A_LOADS ? source_row(8 * i + lane / 8) : -1;
    a_off[p] = r < 0 ? kPark : (uint32_t)(r * K + chunk * 16);
  }
#pragma unroll
  for (int p = 0; p < B_PER; ++p) {
    const int r = 8 * (wave + NW * p) + lane / 8;
    int64_t src;
    if constexpr (GATE_UP) {
      const int col = n0 + r / BW * (BW / 2) + r % (BW / 2);
      src = col < g.N ? (int64_t)(r % BW / (BW / 2)) * g.N + col : -1;
    } else {
      src = n0 + r < g.N ? n0 + r : -1;
    }
    b_off[p] = src < 0 ? kPark : (uint32_t)(src * K + chunk * 16);
  }
  constexpr int AS_WAVES = (BM + 63) / 64;
  if (wave < AS_WAVES) {
    const int64_t r = wave * 64 + lane < BM ? source_row(wave * 64 + lane) : -1;
    as_off = r < 0 ? kPark : (uint32_t)(r * KB * 4);
  }
  if (wave == NW - 1 && lane < 2) {
    const int64_t b = GATE_UP ? (int64_t)lane * NB + n0 / 128 : n0 / 128 + lane;
    bs_off = b < ws_rows ? (uint32_t)(b * KB * 4) : kPark;
  }
  auto issue = [&](int step) {
    Stage8<BM>* s = &st[step & 1];
    const bool cut = tail && step == steps - 1 && chunk >= 4;
#pragma unroll
    for (int p = 0; p < B_PER; ++p)
      dma16s(w_rsrc, lds_address(s->b) + (wave + NW * p) * 1024, cut ? kPark : b_off[p], step * kStageK);
#pragma unroll
    for (int p = 0; p < A_PER; ++p)
      if (A_LOADS % NW == 0 || wave + NW * p < A_LOADS)
        dma16s(a_rsrc, lds_address(s->a) + (wave + NW * p) * 1024, cut ? kPark : a_off[p], step * kStageK);
    if (wave < AS_WAVES) dma4s(as_rsrc, lds_address(s->as) + wave * 256, as_off, step * 4);
    if (wave == NW - 1) dma4s(ws_rsrc, lds_address(s->bs), bs_off, step * 4);
  };

  // ---- the products
  const int wm = wave % WM, wn = wave / WM, q = lane / 16, l16 = lane % 16;
  const int frags = (rows + 15) / 16;
  const int live = frags > wm ? (frags - wm + WM - 1) / WM : 0;   // this wave's fragments that hold rows
  f32x4 acc[MF][NF];
#pragma unroll
  for (int m = 0; m < MF; ++m)
#pragma unroll
    for (int f = 0; f < NF; ++f) acc[m][f] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](auto count, const Stage8<BM>& s) {
    constexpr int M = decltype(count)::value;
    i32x8 x[M];
    float sc[M][2];
    const float s0 = GATE_UP ? s.bs[0] : s.bs[wn * BW / 128], s1 = GATE_UP ? s.bs[1] : 0.f;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int r = (m * WM + wm) * 16 + l16;
      x[m] = operand8(s.a, r, q);
      const float as = s.as[r];
      sc[m][0] = as * s0;
      sc[m][1] = GATE_UP ? as * s1 : 0.f;
    }
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const i32x8 w = operand8(s.b, wn * BW + f * 16 + l16, q);
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const f32x4 part = mfma8(w, x[m]);
        const float c = sc[m][GATE_UP && f >= NF / 2 ? 1 : 0];
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[m][f][v] = fmaf(c, part[v], acc[m][f][v]);
      }
    }
  };
  auto loop = [&](auto count) {
    for (int step = 0; step < steps; ++step) {
      // this wave's loads of the stage have landed and its reads of the other
      // buffer have returned (vmcnt and lgkmcnt 0); with the barrier, everyone's
      __builtin_amdgcn_s_waitcnt(7 << 4);
      stage_barrier();
      if (step + 1 < steps) issue(step + 1);
      if constexpr (decltype(count)::value > 0) multiply(count, st[step & 1]);
    }
  };
  issue(0);
  if (live >= MF) loop(Count<MF>{});
  else if (MF > 3 && live == 3) loop(Count<(MF > 3 ? 3 : 0)>{});
  else if (MF > 2 && live == 2) loop(Count<(MF > 2 ? 2 : 0)>{});
  else if (MF > 1 && live == 1) loop(Count<(MF > 1 ? 1 : 0)>{});
  else loop(Count<0>{});

  // ---- results: lane has columns 4 q .. +3 of each fragment, of row l16
  if constexpr (GATE_UP) {
    uint32_t* s_amax = (uint32_t*)st[0].a;   // [WN][BM]
    __syncthreads();                          // the stages' readers are done
    uint32_t top[MF];
#pragma unroll
    for (int m = 0; m < MF; ++m) {
      top[m] = 0;
      if (m < live) {
#pragma unroll
        for (int f = 0; f < NF / 2; ++f)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const float gate = acc[m][f][v], h = gate / (1.f + expf(-gate)) * acc[m][f + NF / 2][v];
            acc[m][f][v] = h;
            top[m] = abs_bits(h) > top[m] ? abs_bits(h) : top[m];
          }
#pragma unroll
        for (int off = 16; off < kWave; off <<= 1) {
          const uint32_t o = __shfl_xor(top[m], off, kWave);
          top[m] = o > top[m] ? o : top[m];
        }
        if (q == 0) s_amax[wn * BM + (m * WM + wm) * 16 + l16] = top[m];
      }
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MF; ++m) {
      const int r = (m * WM + wm) * 16 + l16;
      if (m >= live || r >= rows) continue;
      uint32_t t = 0;
#pragma unroll
      for (int w = 0; w < WN; ++w) t = s_amax[w * BM + r] > t ? s_amax[w * BM + r] : t;
      float scale, inv;
      bool finite;
      power_scale(t, scale, inv, finite);
      if (wn == 0 && q == 0) g.out_s[(row0 + r) * NB + n0 / 128] = scale;
      uint8_t* o = (uint8_t*)g.out + (row0 + r) * g.N;
#pragma unroll
      for (int f = 0; f < NF / 2; ++f) {
        const int col = n0 + wn * (BW / 2) + f * 16 + q * 4;
        const uint32_t c = pack_fp8x4(acc[m][f][0] * inv, acc[m][f][1] * inv, acc[m][f][2] * inv, acc[m][f][3] * inv);
        if (col < g.N) *(uint32_t*)(o + col) = finite ? c : kNan8;
      }
    }
  } else {
#pragma unroll
    for (int m = 0; m < MF; ++m) {
      const int r = (m * WM + wm) * 16 + l16;
      if (m >= live || r >= rows) continue;
      bf16_t* o = (bf16_t*)g.out + (row0 + r) * g.N;
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const int col = n0 + wn * BW + f * 16 + q * 4;
        if (col < g.N)
          *(uint2*)(o + col) = make_uint2(pack_bf16x2(acc[m][f][0], acc[m][f][1]),
                                          pack_bf16x2(acc[m][f][2], acc[m][f][3]));
      }
    }
  }
}

template <bool GATE_UP, int BM, int WM>
hipError_t gemm8(const Gemm8Args& g, hipStream_t s) {
  // every expert may leave one partly filled tile
  const int64_t m_tiles = g.max_rows / BM + (g.max_rows < g.E ? g.max_rows : g.E);
  const int64_t tiles = m_tiles * ceil_div(g.N, GATE_UP ? kBN / 2 : kBN);
  k_gemm8<GATE_UP, BM, WM><<<(unsigned)round_up(tiles, kXcds), kThreads8, 0, s>>>(g);
  return hipGetLastError();
}

// Tile height by the mean number of rows an expert gets: the lowest that holds
// one and a half times as many, so that most experts take one tile and their
// weights are loaded once.
template <bool GATE_UP>
hipError_t gemm8_any(const Gemm8Args& g, hipStream_t s) {
  const int64_t mean = ceil_div(g.max_rows, g.E), want = mean + mean / 2;
  if (want <= 32) return gemm8<GATE_UP, 32, 1>(g, s);
  if (want <= 64) return gemm8<GATE_UP, 64, 1>(g, s);
  if (want <= 128) return gemm8<GATE_UP, 128, 2>(g, s);
  return gemm8<GATE_UP, 256, 4>(g, s);
}

}  // namespace

hipError_t launch_gate_up_fp8(const uint8_t* xq, const float* xs, const int32_t* expert_offsets, int64_t max_rows, int E,
                              int d, int I, const uint8_t* wq, const float* ws, const int32_t* row_token,
                              int64_t x_rows, uint8_t* hq, float* hs, hipStream_t s) {
  return gemm8_any<true>({xq, xs, row_token, x_rows, expert_offsets, max_rows, E, d, I, wq, ws, hq, hs}, s);
}

hipError_t launch_down_fp8(const uint8_t* hq, const float* hs, const int32_t* expert_offsets, int64_t max_rows, int E,
                           int d, int I, const uint8_t* wq, const float* ws, bf16_t* y, hipStream_t s) {
  return gemm8_any<false>({hq, hs, nullptr, max_rows, expert_offsets, max_rows, E, I, d, wq, ws, y, nullptr}, s);
}

}  // namespace tre
