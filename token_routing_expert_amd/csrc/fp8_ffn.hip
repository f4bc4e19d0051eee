// fp8_ffn.hip -- the grouped products on e4m3 rows and expert weights with a
// float32 scale for each block of 128, on v_mfma_f32_16x16x128_f8f6f4.
//
// For row r of expert e and output column n, blocks b of 128 k:
//   sum_b xs[r, b] ws[e, n / 128, b] * (sum_{k in b} xq[r, k] wq[e, n, k])
// One matrix instruction covers a block of k, so a block's sums leave it
// unscaled (its addend is the constant zero) and are added to the float32
// accumulators with one multiplied-add an element: four vector instructions
// beside each matrix instruction of 32 cycles.  Most of them run beside the
// other waves' matrix work, not all (32768 rows, 16 experts, 2880 x 2880: 372
// us, without them 330).
//
// Tile: BM rows x BN weight rows, one block of 128 bytes of k a stage, both
// operands loaded straight to LDS (16-byte chunk c of row r in slot
// c ^ (r & 7), so that consecutive rows of one chunk fall into different
// banks), a ring of NS stages: NS - 1 load while one multiplies.  Weights
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
//   - The 8-bit instruction is not exact: of 8 consecutive products it drops what
//     lies 13 binary places below the largest.  Behind gate/up that moves h over
//     an edge of its e4m3 rounding now and then (17 tokens, 64 x 2560: the layer
//     0.43% off in the 2-norm where the roundings of y and of the output alone
//     make 0.24%).  Gate/up tiles of 32 and 64 rows wait for the weights' stream
//     and multiply in bf16, which holds every code and sums as float32 does, four
//     instructions a block (64 rows, 16 experts, 2880 x 2880: 50.1 us, in 8 bits
//     48.5; 256 rows 52.0 and 49.7; 512 rows, 1024 x 2816, 31.9 and 26.7).  Higher
//     ones are bound by the matrix work itself and stay in 8 bits (8192 tokens, 4
//     of 128 experts, 2880 x 2880: 856 us, in bf16 1423; 1024 rows, 16 experts,
//     1024 x 2816: 30.6 and 40.2; both before weights came two stages ahead),
//     0.22% to 0.45% off over forty shapes.
// Measured in streams of calls, two sets of inputs and weights in turn: down, 64
// rows, 16 experts, 8192 x 5120: 122 us, 5.5 TB/s of weights; 32768 rows, 16
// experts, 2880 x 2880: 349 to 367 us on four cards, 1.5 PFLOP/s; gate/up of 64
// rows, 16 experts, 2880 x 2880: 63 us, 4.2 TB/s of weights; of 32768 rows, 128
// experts, 2880 x 2880: 806 to 822 us, 1.34 PFLOP/s.  A call by itself takes up
// to 10% longer (the 32768-row product 375 to 406 us).  Where two forms are
// compared, here and below, both ran on one card and the same inputs, which
// repeat, so that weights partly come from the last-level cache.  With the loads dropped the 32768-row product took 247 us, with the
// matrix instructions dropped 296, loads alone 283, all 372: the three wait for
// each other at the stages' barriers.
// XCDs: consecutive tiles go to one XCD, in groups of up to 8 row tiles for
// each weight slice, so that a slice is fetched once for the group and the
// group's rows stay in that XCD's L2.
#include "fp8.hpp"

namespace tre {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kThreads8 = 512, kStageK = 128;
constexpr int kCus = 256, kXcds = 8;             // workgroups are dealt round-robin over the XCDs
constexpr int kGroupM = 8;                       // row tiles of a weight slice that run together
constexpr uint32_t kPark = 0x80000000u;          // past every buffer: reads zeros

struct Gemm8Args {
  const uint8_t* a;          // rows [*, K], lda bytes apart
  int64_t lda;
  const float* a_s;          // [*, KB]
  const int32_t* row_token;  // gathered rows, or null
  int64_t a_rows;            // rows of a
  const int32_t* offsets;
  int64_t max_rows;
  int E, K, N;               // N: output columns (gate/up: I)
  const uint8_t* w;          // [E, NW, K], NW = 2 N for gate/up
  const float* w_s;
  void* out;                 // gate/up: codes [max_rows, N], ldo bytes apart; down: bf16 [max_rows, N]
  int64_t ldo;
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

template <int BM, int BN>
struct Stage8 {
  uint8_t a[BM * kStageK];
  uint8_t b[BN * kStageK];
  float as[(BM + 63) / 64 * 64];   // whole loads of 64
  float bs[64];              // [0], [1]: the tile's two weight blocks
};

// 32 bytes of k of an operand row, chunks q and q + 4 (the same k for both
// operands, in an order of no consequence to the sum): `lo` and `hi` are the
// lane's places of the two in the first 16 rows, `at` the rows' distance.
__device__ __forceinline__ i32x8 operand8(const uint8_t* lo, const uint8_t* hi, int at) {
  const u32x4 a = *(const u32x4*)(lo + at), b = *(const u32x4*)(hi + at);
  return i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

// The same 32 bytes as bf16: four operands of a 16x16x32 instruction.
__device__ __forceinline__ void operand16(bf16x8 (&v)[4], const uint8_t* lo, const uint8_t* hi, int at) {
  const u32x4 a = *(const u32x4*)(lo + at), b = *(const u32x4*)(hi + at);
  v[0] = fp8x8_to_bf16(a[0], a[1]);
  v[1] = fp8x8_to_bf16(a[2], a[3]);
  v[2] = fp8x8_to_bf16(b[0], b[1]);
  v[3] = fp8x8_to_bf16(b[2], b[3]);
}

__device__ __forceinline__ f32x4 mfma8(i32x8 a, i32x8 b) {
  // both operands e4m3 (format 0); zero scale operands select the form without scales
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

// The same number, which the compiler takes for a new one: what is derived from
// it inside a loop is computed there, not kept in registers across the loop.
__device__ __forceinline__ int fresh(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// What a tile is: `rows` rows from row0 on, of expert e, times its weights from
// output column n0 on.
struct Tile8 {
  int e, n0, rows;
  int64_t row0;
};

template <bool GATE_UP, int BM, int BN, int WM, int NS>
__global__ __launch_bounds__(kThreads8) void k_gemm8(Gemm8Args g) {
  constexpr int NW = kThreads8 / kWave, WN = NW / WM, MF = BM / 16 / WM, NF = BN / 16 / WN, BW = BN / WN;
  constexpr int TN = GATE_UP ? BN / 2 : BN;      // output columns of a tile
  constexpr bool BF16 = GATE_UP && BM <= 64;     // multiply in bf16 (why: at the top)
  // a stage's 1 KB loads, dealt to the waves: weights first (they come from
  // further away), then rows, then one of scales.  With more than two stages
  // the waits count loads, so every wave issues as many: of zeros into the
  // sink where it has none.
  constexpr int A_LOADS = BM / 8, B_PER = BN / 8 / NW, A_PER = (A_LOADS + NW - 1) / NW, COUNT = B_PER + A_PER + 1;
  constexpr int AS_WAVES = (BM + 63) / 64;
  constexpr bool EVEN = NS > 2, AHEAD = NS == 2 && BM >= 128 && BN == 256;   // AHEAD: weights two stages ahead (below)
  static_assert(BN % (8 * NW) == 0 && AS_WAVES < NW && (NS - 2) * COUNT < 64, "loads, scale loads, the load counter");
  __shared__ __attribute__((aligned(1024))) Stage8<BM, BN> st[NS];
  __shared__ uint8_t s_sink[NS > 2 ? 1024 : 4];
  __shared__ int s_tiles[kMaxExperts];    // row tiles of the experts up to and with this one
  __shared__ int s_wave[4];
  __shared__ int s_found[2][3];           // expert, row tile, column tile
  __shared__ int s_rows[BM];              // rows behind the next tile's rows, or -1
  __shared__ uint32_t s_amax[GATE_UP ? WN * BM : 1];
  const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int n_tiles = (g.N + TN - 1) / TN;
#ifdef MOE_DEVICE_CHECKS
  // (here and not where a row is used: a trap inside the tile loop would make
  // its uniform values differ between lanes)
  if (blockIdx.x == 0 && g.row_token)
    for (int64_t r = tid; r < clampi<int64_t>(g.offsets[g.E], 0, g.max_rows); r += kThreads8)
      MOE_DCHECK(g.row_token[r] >= 0 && g.row_token[r] < g.a_rows);
#endif

  // ---- the experts' row tiles, counted from the offsets
  {
    int n = 0;
    if (tid < g.E) {
      const int64_t r0 = clampi<int64_t>(g.offsets[tid], 0, g.max_rows);
      const int64_t r1 = clampi<int64_t>(g.offsets[tid + 1], r0, g.max_rows);
      n = (int)((r1 - r0 + BM - 1) / BM);
    }
    // inclusive scan: in the wave, then over the four waves of experts
    int x = n;
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
      const int y = __shfl_up(x, off, kWave);
      if (lane >= off) x += y;
    }
    if (wave < 4 && lane == kWave - 1) s_wave[wave] = x;
    __syncthreads();
    if (wave < 4) {
      for (int w = 0; w < wave; ++w) x += s_wave[w];
      s_tiles[tid] = x;
    }
    __syncthreads();
  }
  const int64_t total = (int64_t)__builtin_amdgcn_readfirstlane(s_tiles[kMaxExperts - 1]) * n_tiles;
  // this XCD's share of the tiles, and this workgroup's walk through it
  const int64_t per = (total + kXcds - 1) / kXcds, x0 = (blockIdx.x % kXcds) * per;
  const int64_t x1 = x0 + per < total ? x0 + per : total;
  const int64_t stride = gridDim.x / kXcds;

  const int K = g.K, KB = (K + 127) / 128, steps = KB;
  const int NB = (g.N + 127) / 128;
  const bool tail = K % 128 != 0;                    // the last stage has half a block
  const int chunk = (lane & 7) ^ (lane >> 3);        // the 16 bytes of a row this lane loads
  const bool gather = g.row_token != nullptr;
  const int64_t w_rows = GATE_UP ? 2 * (int64_t)g.N : g.N, ws_rows = GATE_UP ? 2 * NB : NB;

  // Finds a tile's expert and place; `which` alternates.  One thread writes,
  // everyone reads after the next barrier.
  auto find = [&](int64_t tile, int which) {
    const int width = fresh(n_tiles);   // (the divisions' reciprocals stay out of the tile loop's registers)
    if (tid < kMaxExperts) {
      const int64_t hi = (int64_t)s_tiles[tid] * width, lo = tid ? (int64_t)s_tiles[tid - 1] * width : 0;
      if (tile >= lo && tile < hi) {
        const int m_tiles = (int)((hi - lo) / width), at = (int)(tile - lo);
        const int group = at / (kGroupM * width), in = at - group * (kGroupM * width);
        const int wide = m_tiles - group * kGroupM < kGroupM ? m_tiles - group * kGroupM : kGroupM;
        s_found[which][0] = tid;
        s_found[which][1] = group * kGroupM + in % wide;
        s_found[which][2] = in / wide;
      }
    }
  };
  auto found = [&](int which) {
    Tile8 t;
    t.e = __builtin_amdgcn_readfirstlane(s_found[which][0]);
    t.n0 = __builtin_amdgcn_readfirstlane(s_found[which][2]) * TN;
    const int64_t first = clampi<int64_t>(g.offsets[t.e], 0, g.max_rows);
    const int64_t last = clampi<int64_t>(g.offsets[t.e + 1], first, g.max_rows);
    t.row0 = first + (int64_t)__builtin_amdgcn_readfirstlane(s_found[which][1]) * BM;
    t.rows = (int)(last - t.row0 < BM ? last - t.row0 : BM);
    return t;
  };
  auto fetch_rows = [&](const Tile8& t) {   // into s_rows
    if (gather && tid < BM) {
      int64_t src = -1;
      if (tid < t.rows) {
        src = g.row_token[t.row0 + tid];
        src = src >= 0 && src < g.a_rows ? src : -1;
      }
      s_rows[tid] = (int)src;
    }
  };

  // ---- the operands of the tile whose stages are being loaded (a descriptor
  // each: one chosen by wave for the scales made the loop 4% slower)
  __amdgpu_buffer_rsrc_t a_rsrc, as_rsrc, w_rsrc, ws_rsrc;
  uint32_t a_off[A_PER], b_off[B_PER], scale_off = kPark;
  auto aim_weights = [&](const Tile8& t) {
    const int ln = fresh(lane), piece = ((ln & 7) ^ (ln >> 3)) * 16;
    w_rsrc = __builtin_amdgcn_make_buffer_rsrc(uniform_ptr(g.w + t.e * w_rows * K), (short)0, (int)(w_rows * K),
                                               kBufferConfig);
#pragma unroll
    for (int p = 0; p < B_PER; ++p) {
      const int r = 8 * (wave + NW * p) + ln / 8;
      int64_t src = -1;
      if constexpr (GATE_UP) {
        const int col = t.n0 + r / BW * (BW / 2) + r % (BW / 2);
        if (col < g.N) src = (int64_t)(r % BW / (BW / 2)) * g.N + col;
      } else {
        if (t.n0 + r < g.N) src = t.n0 + r;
      }
      b_off[p] = src < 0 ? kPark : (uint32_t)(src * K + piece);
    }
  };
  auto aim_rows = [&](const Tile8& t) {
    const int ln = fresh(lane), piece = ((ln & 7) ^ (ln >> 3)) * 16;
    const int64_t a_span = gather ? g.a_rows : t.rows;
    a_rsrc = __builtin_amdgcn_make_buffer_rsrc(uniform_ptr(gather ? g.a : g.a + t.row0 * g.lda), (short)0,
                                               (int)(a_span * g.lda), kBufferConfig);
    auto source_row = [&](int r) { return r >= t.rows ? -1 : gather ? s_rows[r] : r; };
#pragma unroll
    for (int p = 0; p < A_PER; ++p) {
      const int i = wave + NW * p, r = i < A_LOADS ? source_row(8 * i + ln / 8) : -1;
      a_off[p] = r < 0 ? kPark : (uint32_t)r * (uint32_t)g.lda + piece;
    }
    as_rsrc = __builtin_amdgcn_make_buffer_rsrc(uniform_ptr(gather ? g.a_s : g.a_s + t.row0 * KB), (short)0,
                                                (int)(a_span * KB * 4), kBufferConfig);
    ws_rsrc = __builtin_amdgcn_make_buffer_rsrc(uniform_ptr(g.w_s + t.e * ws_rows * KB), (short)0,
                                                (int)(ws_rows * KB * 4), kBufferConfig);
    if (wave < AS_WAVES) {
      const int r = wave * 64 + ln < BM ? source_row(wave * 64 + ln) : -1;
      scale_off = r < 0 ? kPark : (uint32_t)r * (uint32_t)(KB * 4);
    }
    if (wave == NW - 1 && ln < 2) {
      const int64_t b = GATE_UP ? (int64_t)ln * NB + t.n0 / 128 : t.n0 / 128 + ln;
      scale_off = b < ws_rows ? (uint32_t)(b * KB * 4) : kPark;
    }
  };
  auto aim = [&](const Tile8& t) {
    aim_weights(t);
    aim_rows(t);
  };
  auto issue_weights = [&](int step, int slot) {
    Stage8<BM, BN>* s = &st[slot];
    const bool cut = tail && step == steps - 1 && chunk >= 4;
#pragma unroll
    for (int p = 0; p < B_PER; ++p)
      dma16s(w_rsrc, lds_address(s->b) + (wave + NW * p) * 1024, cut ? kPark : b_off[p], step * kStageK);
  };
  auto issue_rows = [&](int step, int slot) {   // and both operands' scales
    Stage8<BM, BN>* s = &st[slot];
    const bool cut = tail && step == steps - 1 && chunk >= 4;
#pragma unroll
    for (int p = 0; p < A_PER; ++p) {
      const int i = wave + NW * p;
      if (EVEN || A_LOADS % NW == 0 || i < A_LOADS)
        dma16s(a_rsrc, !EVEN || i < A_LOADS ? lds_address(s->a) + i * 1024 : lds_address(s_sink),
               cut ? kPark : a_off[p], step * kStageK);
    }
    if (wave < AS_WAVES) dma4s(as_rsrc, lds_address(s->as) + wave * 256, scale_off, step * 4);
    else if (wave == NW - 1) dma4s(ws_rsrc, lds_address(s->bs), scale_off, step * 4);
    else if (EVEN) dma4s(ws_rsrc, lds_address(s_sink), kPark, step * 4);
  };
  auto issue = [&](int step, int slot) {
    issue_weights(step, slot);
    issue_rows(step, slot);
  };

  // ---- the products
  const int wm = wave % WM, wn = wave / WM, q = lane / 16, l16 = lane % 16;
  const int place = l16 * kStageK + ((q ^ (l16 & 7)) * 16);   // rows are 16 apart: l16 & 7 is row & 7
  f32x4 acc[MF][NF];
  // the weights' fragments stay in registers, the rows' go by
  auto multiply = [&](auto count, const Stage8<BM, BN>& s, auto weights_read) {
    constexpr int M = decltype(count)::value;
    const float s0 = GATE_UP ? s.bs[0] : s.bs[wn * BW / 128], s1 = GATE_UP ? s.bs[1] : 0.f;
    const uint8_t *a_lo = s.a + wm * 16 * kStageK + place, *a_hi = s.a + wm * 16 * kStageK + (place ^ 64);
    const uint8_t *b_lo = s.b + wn * BW * kStageK + place, *b_hi = s.b + wn * BW * kStageK + (place ^ 64);
    const float* as = s.as + wm * 16 + l16;
    if constexpr (BF16) {
      bf16x8 w[NF][4];
#pragma unroll
      for (int f = 0; f < NF; ++f) operand16(w[f], b_lo, b_hi, f * 16 * kStageK);
#pragma unroll
      for (int m = 0; m < M; ++m) {
        __builtin_amdgcn_sched_barrier(0);
        bf16x8 x[4];
        operand16(x, a_lo, a_hi, m * WM * 16 * kStageK);
        const float xs = as[m * WM * 16], c0 = xs * s0, c1 = xs * s1;
        f32x4 part[NF];
#pragma unroll
        for (int f = 0; f < NF; ++f) part[f] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int f = 0; f < NF; ++f)
            part[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[f][i], x[i], part[f], 0, 0, 0);
#pragma unroll
        for (int f = 0; f < NF; ++f) {
          const float c = f >= NF / 2 ? c1 : c0;
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[m][f][v] = fmaf(c, part[f][v], acc[m][f][v]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      return;
    }
    i32x8 w[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) w[f] = operand8(b_lo, b_hi, f * 16 * kStageK);
    // row fragment m multiplies while m + 1 is read; the scheduling barriers
    // keep the compiler from reading all fragments ahead, which no register is
    // left for
    i32x8 x[2];
    float xs[2];
    x[0] = operand8(a_lo, a_hi, 0);
    xs[0] = as[0];
#pragma unroll
    for (int m = 0; m < M; ++m) {
      __builtin_amdgcn_sched_barrier(0);
      f32x4 part[NF];
#pragma unroll
      for (int f = 0; f < NF; ++f) part[f] = mfma8(w[f], x[m & 1]);
      if (m + 1 < M) {
        x[(m + 1) & 1] = operand8(a_lo, a_hi, (m + 1) * WM * 16 * kStageK);
        xs[(m + 1) & 1] = as[(m + 1) * WM * 16];
      }
      const float c0 = xs[m & 1] * s0, c1 = xs[m & 1] * s1;
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const float c = GATE_UP && f >= NF / 2 ? c1 : c0;
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[m][f][v] = fmaf(c, part[f][v], acc[m][f][v]);
      }
      if (m == 0) weights_read();
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  int64_t tile = x0 + blockIdx.x / kXcds;
  if (tile >= x1) return;
  find(tile, 0);
  __syncthreads();
  Tile8 t = found(0);
  fetch_rows(t);
  __syncthreads();
  aim(t);
  int in_flight = 0, to = 0, from = 0, which = 0;   // stages issued and not multiplied; next slots to fill and to read
  auto fill = [&](int step) {
    issue(step, to);
    to = to + 1 == NS ? 0 : to + 1;
    ++in_flight;
  };
  if constexpr (NS == 2) {
    issue(0, 0);
    if constexpr (AHEAD) issue_weights(1, 1);
  } else {
    for (int s = 0; s < NS - 1 && s < steps; ++s) fill(s);
  }
  while (true) {
    const int frags = (t.rows + 15) / 16;
    const int live = frags > wm ? (frags - wm + WM - 1) / WM : 0;   // this wave's fragments that hold rows
    const bool more = tile + stride < x1;
    Tile8 next = t;
#pragma unroll
    for (int m = 0; m < MF; ++m)
#pragma unroll
      for (int f = 0; f < NF; ++f) acc[m][f] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto walk = [&](auto count) {
      int filled = 0;   // stages of the next tile on their way, once it is aimed at
      bool aimed = false;
      auto look = [&]() {   // the next tile's place
        find(tile + stride, which ^ 1);
        lds_barrier();
        next = found(which ^ 1);
        fetch_rows(next);
      };
      if constexpr (NS == 2) {
        // Two slots: one stage loads while the other multiplies.  (The ring
        // below does the same with NS = 2, 2% slower: it has two places to
        // issue from.)  AHEAD: a wave reads its weights at a stage's start and
        // keeps them, so behind the first row fragment, once every wave has,
        // the slot's half that held them takes those of the stage after the
        // next (behind a tile's end the next tile's; the launch sees to it
        // that a tile has three stages or more).  32768 rows, 128 experts, 2880
        // x 2880: gate/up 831 -> 750 us, down 412 -> 394; 16 experts 762 -> 689
        // and 338 -> 336; gate/up in tiles of 128 rows, 1024 rows, 1024 x 2816,
        // 31 -> 27 (there against three whole stages).  Lower tiles gain nothing
        // (64 rows: 50 and 52 us) and narrower ones lose (8192 rows, 2816 x 1024
        // in tiles of 160 x 128: 35 and 37).
        const int n_ahead = AHEAD ? steps - (more ? 1 : 2) : -1;   // stages that issue weights
        for (int step = 0; step < steps; ++step) {
          // this wave's loads of the stage have landed -- with AHEAD all but
          // its youngest, the next stage's weights -- and its reads of the
          // other slot have returned (lgkmcnt 0); with the barrier, everyone's
          if (step <= n_ahead) wait_vmcnt<AHEAD ? B_PER : 0>(); else wait_vmcnt<0>();
          __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4));   // lgkmcnt(0)
          stage_barrier();
          if (step + 1 < steps) {
            if constexpr (!AHEAD) issue_weights(step + 1, from ^ 1);
            issue_rows(step + 1, from ^ 1);
          }
          if (step == 0 && more) look();
          if (AHEAD && step + 2 == steps && more) aim_weights(next);
          if (step + 1 == steps && more) {
            if constexpr (!AHEAD) {
              if (steps == 1) lds_barrier();
              aim_weights(next);
              issue_weights(0, from ^ 1);
            }
            aim_rows(next);
            issue_rows(0, from ^ 1);
          }
          auto weights_read = [&]() {
            if (!AHEAD || step >= n_ahead) return;
            __builtin_amdgcn_sched_barrier(0);
            lds_barrier();   // this wave's reads have returned; with the barrier, everyone's
            issue_weights(step + 2 < steps ? step + 2 : 0, from);
          };
          if constexpr (decltype(count)::value > 0) multiply(count, st[from], weights_read); else weights_read();
          from ^= 1;
        }
        return;
      }
      for (int step = 0; step < steps; ++step) {
        // this wave's loads of the stage have landed (all but the younger
        // stages'; near the end all) and its reads of the last one have
        // returned; with the barrier, everyone's, and that slot is free
        if (NS > 2 && in_flight >= NS - 1) wait_vmcnt<(NS - 2) * COUNT>(); else wait_vmcnt<0>();
        __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4));   // lgkmcnt(0)
        stage_barrier();
        if (step == 0 && more && steps < NS) {
          look();
          lds_barrier();
        }
        // the stage NS - 1 ahead: this tile's, or behind its last one the next tile's
        if (step + NS - 1 < steps) {
          fill(step + NS - 1);
        } else if (more) {
          if (!aimed) aim(next);
          aimed = true;
          while (filled < steps && in_flight < NS) fill(filled++);
        }
        if (step == 0 && more && steps >= NS) look();
        if constexpr (decltype(count)::value > 0) multiply(count, st[from], [] {});
        from = from + 1 == NS ? 0 : from + 1;
        --in_flight;
      }
    };
    // as many fragments as hold rows, in steps of two (one without rows is
    // zeros in the stage)
    if (live > 8) walk(Count<MF>{});
    else if (live > 6) walk(Count<(MF < 8 ? MF : 8)>{});
    else if (live > 4) walk(Count<(MF < 6 ? MF : 6)>{});
    else if (live > 2) walk(Count<(MF < 4 ? MF : 4)>{});
    else if (live > 0) walk(Count<(MF < 2 ? MF : 2)>{});
    else walk(Count<0>{});

    // ---- results: lane has columns 4 eq .. +3 of each fragment, of row er
    const int eq = fresh(lane) / 16, er = fresh(lane) % 16;
    if constexpr (GATE_UP) {
      uint32_t top[MF];
#pragma unroll
      for (int m = 0; m < MF; ++m) {
        top[m] = 0;
        if (m < live) {
#pragma unroll
          for (int f = 0; f < NF / 2; ++f)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              const float h = swiglu(acc[m][f][v], acc[m][f + NF / 2][v]);
              acc[m][f][v] = h;
              top[m] = abs_bits(h) > top[m] ? abs_bits(h) : top[m];
            }
#pragma unroll
          for (int off = 16; off < kWave; off <<= 1) {
            const uint32_t o = __shfl_xor(top[m], off, kWave);
            top[m] = o > top[m] ? o : top[m];
          }
          if (eq == 0) s_amax[wn * BM + (m * WM + wm) * 16 + er] = top[m];
        }
      }
      lds_barrier();   // (not a full one: the next tile's stage is on its way)
      // the codes gather in the slot that was multiplied last, 128 bytes a row
      // (16-byte chunk c in place c ^ (row & 7)), and leave as whole lines
      uint8_t* rows_out = st[from == 0 ? NS - 1 : from - 1].a;
#pragma unroll
      for (int m = 0; m < MF; ++m) {
        const int r = (m * WM + wm) * 16 + er;
        if (m >= live) continue;
        uint32_t a = 0;
#pragma unroll
        for (int w = 0; w < WN; ++w) a = s_amax[w * BM + r] > a ? s_amax[w * BM + r] : a;
        float scale, inv;
        bool finite;
        power_scale(a, scale, inv, finite);
        if (wn == 0 && eq == 0 && r < t.rows) g.out_s[(t.row0 + r) * NB + t.n0 / 128] = scale;
#pragma unroll
        for (int f = 0; f < NF / 2; ++f) {
          const int c = wn * (BW / 32) + f;
          const uint32_t v = pack_fp8x4(acc[m][f][0] * inv, acc[m][f][1] * inv, acc[m][f][2] * inv, acc[m][f][3] * inv);
          *(uint32_t*)(rows_out + r * 128 + ((c ^ (r & 7)) * 16) + eq * 4) = finite ? v : kNan8;
        }
      }
      lds_barrier();
      const int et = fresh(tid);
#pragma unroll
      for (int i = 0; i < BM * 8; i += kThreads8) {
        const int r = (i + et) / 8, c = et % 8;
        if (r < t.rows && t.n0 + c * 16 < g.N)
          *(u32x4*)((uint8_t*)g.out + (t.row0 + r) * g.ldo + t.n0 + c * 16) =
              *(const u32x4*)(rows_out + r * 128 + ((c ^ (r & 7)) * 16));
      }
    } else {
      // rows gather in the slot that was multiplied last, as many at a time as
      // it holds (16-byte chunk c in place c ^ (row & 7)), and leave as whole
      // lines
      constexpr int ROW = BN * 2, PASS_M = (BM + BN) * kStageK / (ROW * WM * 16) < MF ? 4 : MF, PASS = PASS_M * WM * 16;
      static_assert(PASS * ROW <= (BM + BN) * kStageK, "a pass fits a stage");
      uint8_t* rows_out = st[from == 0 ? NS - 1 : from - 1].a;
      const int et = fresh(tid);
#pragma unroll
      for (int m0 = 0; m0 < MF; m0 += PASS_M) {
        if (m0 * WM * 16 >= t.rows) break;
        lds_barrier();   // the stage's, or the last pass's, readers are done
#pragma unroll
        for (int m = m0; m < m0 + PASS_M && m < MF; ++m) {
          const int r = ((m - m0) * WM + wm) * 16 + er;
          if (m >= live) continue;
#pragma unroll
          for (int f = 0; f < NF; ++f) {
            const int c = wn * (BW / 8) + f * 2 + eq / 2;
            *(uint2*)(rows_out + r * ROW + ((c ^ (r & 7)) * 16) + eq % 2 * 8) = make_uint2(
                pack_bf16x2(acc[m][f][0], acc[m][f][1]), pack_bf16x2(acc[m][f][2], acc[m][f][3]));
          }
        }
        lds_barrier();
#pragma unroll
        for (int i = 0; i < PASS * (ROW / 16); i += kThreads8) {
          const int r = (i + et) / (ROW / 16), c = (i + et) % (ROW / 16), at = m0 * WM * 16 + r;
          if (r < PASS && at < t.rows && t.n0 + c * 8 < g.N)
            *(u32x4*)((bf16_t*)g.out + (t.row0 + at) * g.N + t.n0 + c * 8) =
                *(const u32x4*)(rows_out + r * ROW + ((c ^ (r & 7)) * 16));
        }
      }
    }
    if (!more) return;
    if constexpr (AHEAD) {
      lds_barrier();   // the results' readers are done
      issue_weights(1, from ^ 1);
    }
    tile += stride;
    which ^= 1;
    t = next;
  }
}

// Tile height by the mean number of rows an expert gets: the lowest of 32, 64,
// 128 and 288 that holds one and a half times as many, so that most experts
// take one tile and their weights are loaded once (32768 rows, 128 experts, 2880
// x 2880: 288-row tiles 507 us, 256-row ones 561, both before weights came ahead) -- but no higher than gives
// every compute unit a tile (2048 rows, 4 experts, 1024 x 704: gate/up 33 us in
// 48 tiles of 288 rows, 17 in 384 of 32; down 27 and, in 256 of 64, 10.5).
// columns: output columns of a tile of each height; from height number `ahead`
// on, tiles need three stages of k (AHEAD).
int tile_rows(const Gemm8Args& g, const int (&columns)[4], int ahead) {
  const int heights[4] = {32, 64, 128, 288};
  const int64_t mean = ceil_div(g.max_rows, g.E);
  int h = 0;
  while (h < 3 && heights[h] < mean + mean / 2) ++h;
  while (h > 0 && g.E * ceil_div(mean, heights[h]) * ceil_div(g.N, columns[h]) < kCus) --h;
  if (h >= ahead && g.K <= 2 * kStageK) h = ahead - 1;
  return heights[h];
}

template <bool GATE_UP, int BM, int BN, int WM, int NS>
hipError_t gemm8(const Gemm8Args& g, hipStream_t s) {
  // every expert may leave one partly filled tile
  const int64_t m_tiles = g.max_rows / BM + (g.max_rows < g.E ? g.max_rows : g.E);
  const int64_t tiles = m_tiles * ceil_div(g.N, GATE_UP ? BN / 2 : BN);
  // resident workgroups: by LDS (2 KB beside the stages, and what gate/up exchanges), at most 4 by their waves
  constexpr int fit = 160 * 1024 / (int)(NS * sizeof(Stage8<BM, BN>) + 4096 + (GATE_UP ? 8 / WM * BM * 4 : 0) + BM * 4);
  const int64_t most = kCus * (fit > 4 ? 4 : fit);
  k_gemm8<GATE_UP, BM, BN, WM, NS><<<(unsigned)(tiles < most ? round_up(tiles, kXcds) : most), kThreads8, 0, s>>>(g);
  return hipGetLastError();
}

hipError_t gate_up8(const Gemm8Args& g, hipStream_t s) {
  switch (tile_rows(g, {128, 128, 128, 128}, 2)) {
    case 32: return gemm8<true, 32, 256, 1, 2>(g, s);
    case 64: return gemm8<true, 64, 256, 1, 3>(g, s);
    case 128: return gemm8<true, 128, 256, 2, 2>(g, s);
    default: return gemm8<true, 288, 256, 2, 2>(g, s);
  }
}

// The rows that the busiest compute unit walks through in tiles of h rows, with
// every expert one standard deviation over the mean (random routing).
int64_t longest_walk(const Gemm8Args& g, int h, int columns) {
  const int64_t mean = ceil_div(g.max_rows, g.E), rows = mean + (int64_t)__builtin_sqrt((double)mean);
  return h * ceil_div(g.E * ceil_div(rows, h) * ceil_div(g.N, columns), kCus);
}

// Lower tiles are narrower: with few rows the weights' stream is the work, and
// more, smaller workgroups keep more of it in flight (64 rows, 16 experts, 8192 x
// 5120: 32 rows by 64 columns and three stages 121 us, by 256 and two 143; 8192
// rows, 16 experts, 2816 x 1024: 128 x 128 39 us, 128 x 256 41, 288 x 256 62).
hipError_t down8(const Gemm8Args& g, hipStream_t s) {
  switch (tile_rows(g, {64, 128, 128, 256}, 3)) {
    case 32: return gemm8<false, 32, 64, 2, 3>(g, s);
    case 64: return gemm8<false, 64, 128, 1, 2>(g, s);
    case 128:
      // 160 where the rows over a multiple of 128 would leave most units idle in
      // the last round (8192 rows, 16 experts, 2816 x 1024, on one card: 34 us,
      // 128 rows 43.5; 4096 rows 24 and 28; but 6144 rows 31.5 and 29, 10240 48
      // and 44; by the rows' spread over the experts, 8192 take up to 41)
      if (longest_walk(g, 160, 128) < longest_walk(g, 128, 128)) return gemm8<false, 160, 128, 2, 2>(g, s);
      return gemm8<false, 128, 128, 2, 2>(g, s);
    default: return gemm8<false, 288, 256, 2, 2>(g, s);
  }
}

}  // namespace

hipError_t launch_gate_up_fp8(const uint8_t* xq, int ldx, const float* xs, const int32_t* expert_offsets, int64_t max_rows, int E,
                              int d, int I, const uint8_t* wq, const float* ws, const int32_t* row_token,
                              int64_t x_rows, uint8_t* hq, int ldh, float* hs, hipStream_t s) {
  return gate_up8({xq, ldx, xs, row_token, x_rows, expert_offsets, max_rows, E, d, I, wq, ws, hq, ldh, hs}, s);
}

hipError_t launch_down_fp8(const uint8_t* hq, int ldh, const float* hs, const int32_t* expert_offsets, int64_t max_rows, int E,
                           int d, int I, const uint8_t* wq, const float* ws, bf16_t* y, hipStream_t s) {
  return down8({hq, ldh, hs, nullptr, max_rows, expert_offsets, max_rows, E, I, d, wq, ws, y, 0, nullptr}, s);
}

}  // namespace tre
