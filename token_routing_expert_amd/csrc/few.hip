// few.hip -- the whole layer for a few tokens (T <= 64) in two kernels.
//
//   k_few_gate_up  routing and grouping in every workgroup, then
//                  h[p] = silu(x[t] Wg[e]) * (x[t] Wu[e]) for the pairs p of one expert
//   k_few_down     h[p] Wd[e] over a range of I, and, in the last workgroup
//                  that works on a column tile, out[t] = sum_j w[t,j] y[t*k+j]
//
// With few rows the live experts' weights are the work: 3 d I elements an
// expert, read once, against 6 d I flops a row.  At 8 TB/s a CU gets about 13
// bytes a cycle, so the loop is built around bytes in flight: a wave loads
// weights straight to registers (no LDS, no barrier), several k-steps at a
// time, and multiplies them with 16x16 matrix instructions whose 16 rows are
// the expert's tokens -- idle rows cost nothing that the loads do not hide.
// The waves of a workgroup take k-steps in turn and add their sums in LDS in
// wave order; workgroups split I further in the second kernel and the last
// one adds their partial rows in order, so equal calls give equal bits.
//
// Measured (gate/up and down, and the weights' rate over both): one token, 4 of
// 128 experts, 2880 x 2880, bf16 24.8 + 17.4 us, 4.7 TB/s; 64 tokens, 1 of 16,
// 5120 x 8192, bf16 454 + 227 us, 5.9 TB/s; 8 tokens, 4 of 128, 8 bits 96 + 52
// us, 4.8 TB/s; 3 tokens of a 128 x 256 float32 layer 5.7 + 7.0 us, all latency.
// With many live experts the 8-bit weights stream at 4.4 to 4.6 TB/s, the grouped
// products' at 4.8 to 5.0, so from about 32 tokens on those are ahead (64 tokens, 4
// of 128, cold: 603 us, moe_forward_fp8 575; 1 of 16, 5120 x 8192: 456 and 398).
//
// The order of k inside a matrix instruction is free as long as both operands
// use the same: each policy below lets a lane's 16-byte weight loads run along
// the stored row and assigns k accordingly.
#include "fp8.hpp"
#include "route_token.hpp"

namespace tre {
namespace {

// ---- how a wave streams an expert's matrix ----------------------------------
//
// kSteps of kStep values of k; a tile of 16 * NF output columns; lane l is
// column (l % 16) of each of the NF fragments and k-group l / 16.  The result
// of fragment f has, in lane l, rows 4 (l / 16) + v and column l % 16.

// [K, N] row-major weights of the activations' type (bf16, float32).  With V
// = 16 bytes / element, lane l loads V columns of V rows (k = V (l/16) .. +V-1
// of the step): its c-th columns form fragment c.  bf16 pairs two rows into a
// register with one byte permutation each (half an instruction a weight).
template <typename Elem>
struct RowMajor {
  using Act = Elem;
  static constexpr int V = 16 / (int)sizeof(Elem), NF = V, kStep = 4 * V, kBytes = 16 * V;
  static constexpr int kGuWaves = 8, kDnWaves = 8, kMaxTiles = 4;
  static constexpr int kXVec = 1;                     // 16-byte activation loads a row and step
  static constexpr int kCols = 16 * V;                // columns of a tile; gate/up: half gate, half up
  struct Args {
    const Elem* w;
  };
  struct Regs {
    u32x4 r[V];
  };
  const char* base;    // the step-0 rows of this expert
  uint32_t lane_off;   // this lane's bytes into them
  int64_t row_bytes;

  __device__ __forceinline__ static RowMajor gate_up(const Args& a, int e, int d, int I, int n0, int lane) {
    const int cg = lane % 16, col = cg < 8 ? n0 + cg * V : I + n0 + (cg - 8) * V;
    return RowMajor(a.w + (int64_t)e * d * 2 * I, 2 * I, col, lane);
  }
  __device__ __forceinline__ static RowMajor down(const Args& a, int e, int d, int I, int n0, int lane) {
    const int col = n0 + lane % 16 * V;
    return RowMajor(a.w + (int64_t)e * I * d, d, col < d ? col : n0, lane);   // past the matrix: not stored
  }
  __device__ __forceinline__ RowMajor(const Elem* w, int ld, int col, int lane)
      : base((const char*)w), lane_off((uint32_t)(((int64_t)(lane / 16 * V) * ld + col) * sizeof(Elem))),
        row_bytes((int64_t)ld * sizeof(Elem)) {}

  __device__ __forceinline__ static int x_offset(int lane) { return lane / 16 * V; }
  __device__ __forceinline__ static int x_load(int) { return 0; }
  __device__ __forceinline__ static bool x_valid(int, int, int) { return true; }   // K is a multiple of kStep
  __device__ __forceinline__ void load(Regs& g, int step) const {
    const char* p = base + (int64_t)step * kStep * row_bytes;
#pragma unroll
    for (int r = 0; r < V; ++r)
      g.r[r] = __builtin_nontemporal_load((const u32x4*)(p + r * row_bytes + lane_off));
  }
  template <int MT>
  __device__ __forceinline__ static void mma(const Regs& g, const u32x4 (&x)[MT][kXVec], f32x4 (&acc)[MT][NF]) {
    if constexpr (sizeof(Elem) == 2) {
#pragma unroll
      for (int c = 0; c < NF; ++c) {
        u32x4 b;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          b[i] = __builtin_amdgcn_perm(g.r[2 * i + 1][c / 2], g.r[2 * i][c / 2], c % 2 ? 0x07060302u : 0x05040100u);
        const bf16x8 bf = __builtin_bit_cast(bf16x8, b);
#pragma unroll
        for (int m = 0; m < MT; ++m)
          acc[m][c] =
              __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[m][0]), bf, acc[m][c], 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int r = 0; r < V; ++r) {
        const f32x4 b = __builtin_bit_cast(f32x4, g.r[r]);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const f32x4 a = __builtin_bit_cast(f32x4, x[m][0]);
#pragma unroll
          for (int c = 0; c < NF; ++c) acc[m][c] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], b[c], acc[m][c], 0, 0, 0);
        }
      }
    }
  }
  // where a tile's column sits in the reduction rows (fragment * 16 + lane)
  __device__ __forceinline__ static int gate_slot(int c) { return c % V * 16 + c / V; }
  __device__ __forceinline__ static int up_slot(int c) { return c % V * 16 + c / V + 8; }
  __device__ __forceinline__ static int down_slot(int c) { return c % V * 16 + c / V; }
};

// 8-bit [N, K] weights with bf16 activations.  A step is one block of 128
// columns, in two halves of 64: lane l loads 16 bytes (k = 16 (l/16) .. +15 of
// the half) of row l % 16 of each fragment, 64 contiguous bytes a row.  e4m3
// codes are exact in bf16, so the block's sum comes from bf16 matrix
// instructions and the scale is applied to it in float32, once a block.  The
// last block may be half a block: its upper half is not loaded (activations
// neither: what lies behind a row may be a NaN) and multiplies zeros.
struct Blocked8 {
  using Act = bf16_t;
  static constexpr int NF = 2, kStep = 128, kBytes = 32 * NF;
  static constexpr int kGuWaves = 4, kDnWaves = 4, kMaxTiles = 2;
  static constexpr int kXVec = 4;
  static constexpr int kCols = 16 * NF;
  struct Args {
    const uint8_t* w;
    const float* s;
  };
  struct Regs {
    u32x4 r[NF][2];
    float s[NF];
  };
  const uint8_t* base[NF];   // first row of each fragment
  const float* scale[NF];
  uint32_t lane_off;
  int K;

  __device__ __forceinline__ static Blocked8 gate_up(const Args& a, int e, int d, int I, int n0, int lane) {
    Blocked8 m;
    const int ib = (I + 127) / 128, db = (d + 127) / 128;
#pragma unroll
    for (int f = 0; f < NF; ++f) {   // the lower half of the fragments gate, the upper up
      const int half = f / (NF / 2), n = n0 + f % (NF / 2) * 16;
      m.base[f] = a.w + ((int64_t)e * 2 + half) * I * d + (int64_t)n * d;
      m.scale[f] = a.s + (((int64_t)e * 2 + half) * ib + n / 128) * db;
    }
    m.set(d, lane);
    return m;
  }
  __device__ __forceinline__ static Blocked8 down(const Args& a, int e, int d, int I, int n0, int lane) {
    Blocked8 m;
    const int ib = (I + 127) / 128, db = (d + 127) / 128;
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      m.base[f] = a.w + (int64_t)e * d * I + (int64_t)(n0 + 16 * f) * I;
      m.scale[f] = a.s + ((int64_t)e * db + (n0 + 16 * f) / 128) * ib;
    }
    m.set(I, lane);
    return m;
  }
  __device__ __forceinline__ void set(int k, int lane) {
    K = k;
    lane_off = (uint32_t)(lane % 16) * (uint32_t)K + (uint32_t)(lane / 16 * 16);
  }
  // 16-byte activation load c of a step: k = 64 (c / 2) + 16 (l / 16) + 8 (c % 2)
  __device__ __forceinline__ static int x_offset(int lane) { return lane / 16 * 16; }
  __device__ __forceinline__ static int x_load(int c) { return c / 2 * 64 + c % 2 * 8; }
  __device__ __forceinline__ static bool x_valid(int step, int c, int K) { return c < 2 || step * kStep + 64 < K; }
  __device__ __forceinline__ void load(Regs& g, int step) const {
    const bool whole = step * kStep + 64 < K;
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const uint8_t* p = base[f] + (int64_t)step * kStep + lane_off;
      g.s[f] = scale[f][step];
      g.r[f][0] = *(const u32x4*)p;
      g.r[f][1] = u32x4{0, 0, 0, 0};
      if (whole) g.r[f][1] = *(const u32x4*)(p + 64);
    }
  }
  template <int MT>
  __device__ __forceinline__ static void mma(const Regs& g, const u32x4 (&x)[MT][kXVec], f32x4 (&acc)[MT][NF]) {
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      bf16x8 b[4];
#pragma unroll
      for (int h = 0; h < 4; ++h) b[h] = fp8x8_to_bf16(g.r[f][h / 2][h % 2 * 2], g.r[f][h / 2][h % 2 * 2 + 1]);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        f32x4 part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 4; ++h)
          part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[m][h]), b[h], part, 0, 0, 0);
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[m][f][v] = fmaf(g.s[f], part[v], acc[m][f][v]);
      }
    }
  }
  __device__ __forceinline__ static int gate_slot(int c) { return c; }
  __device__ __forceinline__ static int up_slot(int c) { return NF / 2 * 16 + c; }
  __device__ __forceinline__ static int down_slot(int c) { return c; }
};

// ---- the parts the two kernels share ------------------------------------------

__device__ __forceinline__ void few_store(bf16_t* p, float f) { *p = f32_to_bf16(f); }
__device__ __forceinline__ void few_store(float* p, float f) { *p = f; }
__device__ __forceinline__ void few_store4(bf16_t* p, f32x4 f) {
  *(uint2*)p = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
}
__device__ __forceinline__ void few_store4(float* p, f32x4 f) { *(f32x4*)p = f; }

// The grouping, in every workgroup, from the pairs' expert ids in LDS.
struct FewGroup {
  int32_t idx[kFewPairs];      // expert of each pair
  int32_t list[kFewPairs];     // one expert's pairs, ascending
  int32_t count[kMaxExperts];
  int32_t live[kMaxExperts];   // the experts that have pairs, ascending
  int32_t n_live;
};

// Counts and live experts.  An id outside [0, E) belongs to no expert.
template <int NT>
__device__ __forceinline__ void few_group(FewGroup& g, int P, int E) {
  const int tid = threadIdx.x, lane = tid % kWave;
  const uint64_t below = lane == 0 ? 0ull : ~0ull >> (kWave - lane);
  for (int e = tid; e < kMaxExperts; e += NT) g.count[e] = 0;
  __syncthreads();
  for (int p = tid; p < P; p += NT) {
    const int e = g.idx[p];
    MOE_DCHECK(e >= -1 && e < E);
    if (e >= 0 && e < E) atomicAdd(&g.count[e], 1);
  }
  __syncthreads();
  if (tid < kWave) {
    int n = 0;
    for (int b = 0; b < E; b += kWave) {
      const bool has = g.count[b + lane] > 0;   // zero past E (E <= 256 = four waves of counts)
      const uint64_t m = __ballot(has);
      if (has) g.live[n + __popcll(m & below)] = b + lane;
      n += __popcll(m);
    }
    if (lane == 0) g.n_live = n;
  }
  __syncthreads();
}

// The pairs of expert e, into g.list (read by everyone after this).
__device__ __forceinline__ void few_list(FewGroup& g, int P, int e) {
  const int lane = threadIdx.x % kWave;
  const uint64_t below = lane == 0 ? 0ull : ~0ull >> (kWave - lane);
  __syncthreads();   // the last list's readers are done
  if (threadIdx.x < kWave) {
    int n = 0;
    for (int b = 0; b < P; b += kWave) {
      const bool hit = b + lane < P && g.idx[b + lane] == e;
      const uint64_t m = __ballot(hit);
      if (hit) g.list[n + __popcll(m & below)] = b + lane;
      n += __popcll(m);
    }
  }
  __syncthreads();
}

// Every token's selection, into LDS: the lane groups of the routing kernel
// (the same sums in the same order, so the same bits).
template <int G, int S, int NT>
__device__ __forceinline__ void few_route_all(const float* __restrict__ logits, int T, int E, int k, int32_t* idx,
                                              float* w) {
  for (int t0 = 0; t0 < T; t0 += NT / G) {
    const int t = t0 + (int)threadIdx.x / G;
    const bool active = t < T;
    float lg[S];
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int e = s * G + (int)threadIdx.x % G;
      lg[s] = active && e < E ? logits[t * E + e] : 0.f;
      MOE_DCHECK(__builtin_isfinite(lg[s]));
    }
    route_token<G, S>(lg, t, active, E, k, idx, w);
  }
}

template <int NT>
__device__ __forceinline__ void few_route(const float* __restrict__ logits, int T, int E, int k, int32_t* idx,
                                          float* w) {
  if (E <= 16) few_route_all<16, 1, NT>(logits, T, E, k, idx, w);
  else if (E <= 32) few_route_all<32, 1, NT>(logits, T, E, k, idx, w);
  else if (E <= 64) few_route_all<64, 1, NT>(logits, T, E, k, idx, w);
  else if (E <= 128) few_route_all<16, 8, NT>(logits, T, E, k, idx, w);
  else few_route_all<64, 4, NT>(logits, T, E, k, idx, w);
}

// acc[m] = the 16 rows x[m] times steps wave, wave + NW, ... below s1 of the
// matrix, several steps loaded together: with 2-3 waves a SIMD more than 100 KB
// a CU are in flight, several times what the HBM latency asks for.  There is
// no branch on the number of row tiles between the matrix instructions (the
// caller picks C): a result read right behind a branch was not waited for by
// the code the compiler wrote (ROCm 7.2.0), tests/test_mfma_waits.py.
template <class M, int C, int NW>
__device__ __forceinline__ void few_stream(const M& w, const typename M::Act* const (&x)[C], int K, int s0, int s1,
                                           int wave, int lane, f32x4 (&acc)[C][M::NF]) {
  // steps loaded together: 128 bytes of weights a lane, fewer with more row
  // tiles (their sums and activations need the registers)
  constexpr int U0 = 128 / M::kBytes / C, U = U0 > 0 ? U0 : 1;
#pragma unroll
  for (int m = 0; m < C; ++m)
#pragma unroll
    for (int f = 0; f < M::NF; ++f) acc[m][f] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma clang loop unroll(disable)
  for (int st = s0 + wave; st < s1; st += NW * U) {
    typename M::Regs g[U];
    u32x4 xr[U][C][M::kXVec];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = st + u * NW;
      if (s >= s1) break;
      w.load(g[u], s);
#pragma unroll
      for (int m = 0; m < C; ++m)
#pragma unroll
        for (int c = 0; c < M::kXVec; ++c) {
          xr[u][m][c] = u32x4{0, 0, 0, 0};
          if (M::x_valid(s, c, K)) xr[u][m][c] = *(const u32x4*)(x[m] + (int64_t)s * M::kStep + M::x_load(c));
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (st + u * NW >= s1) break;
      M::template mma<C>(g[u], xr[u], acc);
    }
  }
}

// rows(Count<C>, r0) for the n rows of an expert, C row tiles at a time: 1, 2
// or 4, as many as are left and MT allows.  A tile's lanes past the last row
// repeat it, and their sums are not used.
template <int MT, class F>
__device__ __forceinline__ void few_row_tiles(int n, F rows) {
  for (int r0 = 0; r0 < n; r0 += 16 * MT) {
    if (MT >= 4 && n - r0 > 32) rows(Count<(MT >= 4 ? 4 : 1)>{}, r0);
    else if (MT >= 2 && n - r0 > 16) rows(Count<(MT >= 2 ? 2 : 1)>{}, r0);
    else rows(Count<1>{}, r0);
  }
}

// Rows of the reduction buffer are 4 floats apart modulo 16, so that the four
// row groups of a store fall into different banks.
template <class M>
constexpr int kRedStride = M::kCols + 4;

template <class M>
__device__ __forceinline__ void few_spill(float* red, const f32x4 (&acc)[M::NF], int wave, int lane) {
#pragma unroll
  for (int f = 0; f < M::NF; ++f)
#pragma unroll
    for (int v = 0; v < 4; ++v)
      red[(wave * 16 + lane / 16 * 4 + v) * kRedStride<M> + f * 16 + lane % 16] = acc[f][v];
}

template <class M, int NW>
__device__ __forceinline__ float few_sum(const float* red, int row, int slot) {
  float v = red[row * kRedStride<M> + slot];
#pragma unroll
  for (int w = 1; w < NW; ++w) v += red[(w * 16 + row) * kRedStride<M> + slot];
  return v;
}

// ---- gate/up -----------------------------------------------------------------
// Items (live expert, column tile of kCols / 2 columns of h), dealt round-robin
// to the workgroups, so that routing and grouping are done once a workgroup.
// The first one also writes the selection and clears the column tiles'
// counters for k_few_down.
template <class M, int MT>
__global__ __launch_bounds__(M::kGuWaves * kWave) void k_few_gate_up(
    const typename M::Act* __restrict__ x, const float* __restrict__ logits, int32_t* __restrict__ topk_idx,
    float* __restrict__ topk_w, int T, int d, int E, int k, int I, typename M::Args wa,
    typename M::Act* __restrict__ h, int32_t* __restrict__ counters, int n_counters) {
  constexpr int NW = M::kGuWaves, NT = NW * kWave, CT = M::kCols / 2;
  __shared__ FewGroup g;
  __shared__ float red[NW * 16 * kRedStride<M>];
  float* s_w = red;   // routing weights, before the sums need the buffer
  static_assert(kFewPairs <= NW * 16 * kRedStride<M>, "routing weights fit the reduction buffer");
  const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int P = T * k;
  const bool first = blockIdx.x == 0;
  if (logits) {
    few_route<NT>(logits, T, E, k, g.idx, s_w);
    if (first) {
      __syncthreads();
      for (int p = tid; p < P; p += NT) {
        topk_idx[p] = g.idx[p];
        topk_w[p] = s_w[p];
      }
    }
  } else {
    for (int p = tid; p < P; p += NT) g.idx[p] = topk_idx[p];
  }
  if (first)
    for (int c = tid; c < n_counters; c += NT) counters[c] = 0;
  few_group<NT>(g, P, E);

  const int tiles = I / CT, items = __builtin_amdgcn_readfirstlane(g.n_live) * tiles;
  const int steps = (d + M::kStep - 1) / M::kStep;
  int slot = -1, n = 0, e = 0;
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int n0 = item % tiles * CT;
    if (item / tiles != slot) {
      slot = item / tiles;
      e = __builtin_amdgcn_readfirstlane(g.live[slot]);
      n = __builtin_amdgcn_readfirstlane(g.count[e]);
      few_list(g, P, e);
    }
    const M w = M::gate_up(wa, e, d, I, n0, lane);
    few_row_tiles<MT>(n, [&](auto count, int r0) {
      constexpr int C = decltype(count)::value;
      const typename M::Act* xr[C];
#pragma unroll
      for (int m = 0; m < C; ++m) {
        const int r = r0 + m * 16 + lane % 16;
        xr[m] = x + (int64_t)(g.list[r < n ? r : n - 1] / k) * d + M::x_offset(lane);
      }
      f32x4 acc[C][M::NF];
      few_stream<M, C, NW>(w, xr, d, 0, steps, wave, lane, acc);
#pragma unroll
      for (int m = 0; m < C; ++m) {
        __syncthreads();   // the buffer's last readers are done
        few_spill<M>(red, acc[m], wave, lane);
        __syncthreads();
        for (int i = tid; i < 16 * CT; i += NT) {
          const int row = i / CT, c = i % CT, r = r0 + m * 16 + row;
          if (r >= n) break;   // rows ascend with i
          const float gate = few_sum<M, NW>(red, row, M::gate_slot(c)), up = few_sum<M, NW>(red, row, M::up_slot(c));
          // h is an operand of the second kernel's matrix instructions, so it is
          // rounded to their type here, once (float32 layers keep it whole)
          few_store(h + (int64_t)g.list[r] * I + n0 + c, gate / (1.f + expf(-gate)) * up);
        }
      }
    });
  }
}

// ---- down and combine ------------------------------------------------------------
// Items (live expert, share of I, column tile of kCols columns).  Partial rows
// part[share][pair][d] in float32 go through memory, and a counter a column
// tile tells the workgroup that brings the tile's last share, which adds each
// token's pairs in slot order (a pair's shares in order before).  The partial
// rows are written and read by device-scope accesses, which pass the XCDs'
// separate L2s: a workgroup waits until its own are through (vmcnt 0, then the
// barrier) before it counts.  Device-wide fences in their place flush a whole
// L2 a workgroup: 98 us instead of 23 for one token of the 128-expert layer.
template <class M, int MT>
__global__ __launch_bounds__(M::kDnWaves * kWave, 2) void k_few_down(
    const typename M::Act* __restrict__ h, const int32_t* __restrict__ topk_idx, const float* __restrict__ topk_w,
    int T, int d, int E, int k, int I, typename M::Args wa, int n_split, float* __restrict__ part,
    int32_t* __restrict__ counters, typename M::Act* __restrict__ out) {
  constexpr int NW = M::kDnWaves, NT = NW * kWave, CT = M::kCols;
  __shared__ FewGroup g;
  __shared__ float red[NW * 16 * kRedStride<M>];
  __shared__ int s_last;
  const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int P = T * k, tiles = (d + CT - 1) / CT;
  for (int p = tid; p < P; p += NT) g.idx[p] = topk_idx[p];
  few_group<NT>(g, P, E);
  const int n_live = __builtin_amdgcn_readfirstlane(g.n_live), per = n_split * tiles;
  // with no live expert at all, one pass over the columns writes zeros
  const int items = n_live > 0 ? n_live * per : tiles;
  const int steps = (I + M::kStep - 1) / M::kStep;
  int slot = -1, n = 0, e = 0;
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int tile = item % tiles, split = item / tiles % n_split, n0 = tile * CT;
    const int cols = d - n0 < CT ? d - n0 : CT;
    if (n_live > 0) {
      if (item / per != slot) {
        slot = item / per;
        e = __builtin_amdgcn_readfirstlane(g.live[slot]);
        n = __builtin_amdgcn_readfirstlane(g.count[e]);
        few_list(g, P, e);
      }
      const M w = M::down(wa, e, d, I, n0, lane);
      const int s0 = split * steps / n_split, s1 = (split + 1) * steps / n_split;
      few_row_tiles<MT>(n, [&](auto count, int r0) {
        constexpr int C = decltype(count)::value;
        const typename M::Act* hr[C];
#pragma unroll
        for (int m = 0; m < C; ++m) {
          const int r = r0 + m * 16 + lane % 16;
          hr[m] = h + (int64_t)g.list[r < n ? r : n - 1] * I + M::x_offset(lane);
        }
        f32x4 acc[C][M::NF];
        few_stream<M, C, NW>(w, hr, I, s0, s1, wave, lane, acc);
#pragma unroll
        for (int m = 0; m < C; ++m) {
          __syncthreads();
          few_spill<M>(red, acc[m], wave, lane);
          __syncthreads();
          for (int i = tid; i < 16 * CT; i += NT) {
            const int row = i / CT, c = i % CT, r = r0 + m * 16 + row;
            if (r >= n) break;
            if (c < cols)
              __hip_atomic_store(part + ((int64_t)split * P + g.list[r]) * d + n0 + c,
                                 few_sum<M, NW>(red, row, M::down_slot(c)), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          }
        }
      });
      compiler_fence();
      wait_vmcnt<0>();
      __syncthreads();
      if (tid == 0)
        s_last = __hip_atomic_fetch_add(&counters[tile], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                 n_live * n_split - 1;
      __syncthreads();
      if (!s_last) continue;
    }
    for (int i = tid; i < T * (CT / 4); i += NT) {
      const int t = i / (CT / 4), c = i % (CT / 4) * 4;
      if (c >= cols) continue;
      f32x4 sum = {0.f, 0.f, 0.f, 0.f};
      for (int j = 0; j < k; ++j) {
        const int p = t * k + j, pe = g.idx[p];
        if (pe < 0 || pe >= E) continue;
        const float wt = topk_w[p];
        f32x4 y = {0.f, 0.f, 0.f, 0.f};
        for (int s = 0; s < n_split; ++s) {
          const float* yp = part + ((int64_t)s * P + p) * d + n0 + c;
#pragma unroll
          for (int v = 0; v < 4; ++v) y[v] += __hip_atomic_load(yp + v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
#pragma unroll
        for (int v = 0; v < 4; ++v) sum[v] = fmaf(wt, y[v], sum[v]);
      }
      few_store4(out + (int64_t)t * d + n0 + c, sum);
    }
  }
}

// ---- launch ------------------------------------------------------------------------

constexpr int kFewCus = 256, kFewWaves = 16;   // compute units, and waves that one holds at these register counts

// Shares of I in the second kernel: 128 workgroups at least (of 8 waves; every
// further share is a partial row more to write, wait for and read), while a
// wave keeps two steps of its own.
template <class M>
int few_split(int P, int E, int d, int I) {
  if (P == 0) return 1;   // no tokens: a workspace is asked for all the same
  const int64_t tiles = ceil_div(d, M::kCols) * (P < E ? P : E);
  const int steps = (int)ceil_div(I, M::kStep);
  int64_t n = ceil_div(128, tiles);
  const int64_t most = steps / (2 * M::kDnWaves);
  n = n > most ? most : n;
  return (int)(n < 1 ? 1 : n > kFewSplitMax ? kFewSplitMax : n);
}

template <class M, int MT>
hipError_t few_run(const typename M::Act* x, const float* logits, int T, int d, int E, int k, int I,
                   typename M::Args gu, typename M::Args dn, int32_t* topk_idx, float* topk_w,
                   typename M::Act* out, const FewScratch& ws, hipStream_t s) {
  const int P = T * k, slots = P < E ? P : E;
  const int tiles = (int)ceil_div(d, M::kCols), n_split = few_split<M>(P, E, d, I);
  const int64_t gu_items = (int64_t)slots * (I / (M::kCols / 2)), dn_items = (int64_t)slots * n_split * tiles;
  const auto grid = [](int64_t items, int waves) {
    const int64_t most = (int64_t)kFewCus * ((kFewWaves + waves - 1) / waves);
    return dim3((unsigned)(items < most ? items : most));
  };
  k_few_gate_up<M, MT><<<grid(gu_items, M::kGuWaves), M::kGuWaves * kWave, 0, s>>>(
      x, logits, topk_idx, topk_w, T, d, E, k, I, gu, (typename M::Act*)ws.h, ws.counters, tiles);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_few_down<M, MT><<<grid(dn_items, M::kDnWaves), M::kDnWaves * kWave, 0, s>>>(
      (const typename M::Act*)ws.h, topk_idx, topk_w, T, d, E, k, I, dn, n_split, ws.part, ws.counters, out);
  return hipGetLastError();
}

// Row tiles held in registers: as many as the tokens can fill, so that an
// expert's weights are read once (a given pair list may repeat an expert in
// one token; the kernels then take further rounds).  With 8-bit weights two at
// most: a step has four times the k, and four tiles of it do not fit beside
// the weights; an expert with more than 32 rows takes two rounds.
template <class M>
hipError_t few_dispatch(const typename M::Act* x, const float* logits, int T, int d, int E, int k, int I,
                        typename M::Args gu, typename M::Args dn, int32_t* topk_idx, float* topk_w,
                        typename M::Act* out, const FewScratch& ws, hipStream_t s) {
  if (T <= 16) return few_run<M, 1>(x, logits, T, d, E, k, I, gu, dn, topk_idx, topk_w, out, ws, s);
  if (T <= 32 || M::kMaxTiles == 2)
    return few_run<M, 2>(x, logits, T, d, E, k, I, gu, dn, topk_idx, topk_w, out, ws, s);
  return few_run<M, M::kMaxTiles>(x, logits, T, d, E, k, I, gu, dn, topk_idx, topk_w, out, ws, s);
}

}  // namespace

int few_split_bf16(int P, int E, int d, int I) { return few_split<RowMajor<bf16_t>>(P, E, d, I); }
int few_split_f32(int P, int E, int d, int I) { return few_split<RowMajor<float>>(P, E, d, I); }
int few_split_fp8(int P, int E, int d, int I) { return few_split<Blocked8>(P, E, d, I); }
int few_counters(int d) { return (int)ceil_div(d, 32); }   // the narrowest column tile

hipError_t launch_few_bf16(const bf16_t* x, const float* logits, int T, int d, int E, int k, int I, const bf16_t* wgu,
                           const bf16_t* wd, int32_t* topk_idx, float* topk_w, bf16_t* out, const FewScratch& ws,
                           hipStream_t s) {
  return few_dispatch<RowMajor<bf16_t>>(x, logits, T, d, E, k, I, {wgu}, {wd}, topk_idx, topk_w, out, ws, s);
}
hipError_t launch_few_f32(const float* x, const float* logits, int T, int d, int E, int k, int I, const float* wgu,
                          const float* wd, int32_t* topk_idx, float* topk_w, float* out, const FewScratch& ws,
                          hipStream_t s) {
  return few_dispatch<RowMajor<float>>(x, logits, T, d, E, k, I, {wgu}, {wd}, topk_idx, topk_w, out, ws, s);
}
hipError_t launch_few_fp8(const bf16_t* x, const float* logits, int T, int d, int E, int k, int I, const uint8_t* wgu,
                          const float* wgu_s, const uint8_t* wd, const float* wd_s, int32_t* topk_idx, float* topk_w,
                          bf16_t* out, const FewScratch& ws, hipStream_t s) {
  return few_dispatch<Blocked8>(x, logits, T, d, E, k, I, {wgu, wgu_s}, {wd, wd_s}, topk_idx, topk_w, out, ws, s);
}

}  // namespace tre
