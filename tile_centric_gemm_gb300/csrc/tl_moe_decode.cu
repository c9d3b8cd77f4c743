// tl_moe_decode.cu -- a whole mixture-of-experts layer for the tokens of a decode
// step, in two launches.
//
//   ids, gates = top-k and softmax of the logits
//   h_s = silu(x W1_e[:, :I]) * (x W1_e[:, I:])   e = ids[s]      (launch 1)
//   out = sum_s gates[s] (h_s W2_e)                                (launch 2)
//
// For so few tokens the layer is the reading of the chosen experts' weights, so
// both launches are one stream of weights through one CTA per SM.  The work is the
// list of (row tile of one expert, column tile, 128 rows of the contraction), cut
// into equal runs, one to a CTA, whatever the routing was: with one token and two
// experts the contraction is shared by several CTAs, with 64 tokens a CTA has
// several tiles.  A tile whose steps fall to several CTAs leaves partial sums in
// the workspace, and the CTA that arrives last adds them in CTA order.  Each CTA
// finds the routing out for itself from the logits: no launch for it, no wait.
//
// The second launch starts while the first runs (programmatic dependent launch):
// its CTAs take the SMs that become free, work out the routing and fill their
// rings with W2 before they wait for the first launch's results.
//
// Inside a CTA warp (group, sub, kq) takes 64 columns (group 0: gate columns, group 1:
// up columns; in the down launch the tile's two halves) and, where the tile is narrow,
// its share of the rows: every row's strips lie next to one another, so that lines are
// read whole whatever the row length.  Weights are row-major [K, N], the product wants pairs along K: the
// warp copies (cp.async) whole lines of 32 rows and 64 columns into a ring of its own,
// a lane takes eight rows' eight columns from it and interleaves two rows' words with a
// byte permutation; since the order of the contraction is free, those eight rows are
// also the eight consecutive elements of a token that one 16-byte load brings for the
// other operand.  No barrier and no transposition between memory and the tensor cores.
// (Copies of single sectors, each lane fetching what it multiplies, ran at half the
// rate.)
//
// h goes from launch to launch as two bf16 terms (16 bits of mantissa): the down
// product takes one multiplication more for each, which the stream of weights
// hides, and the result keeps the accuracy of fp32 activations.
//
// Bound by memory where every expert is met (27 tokens, top 2 of 32 experts of 4096 x
// 1408: 147-155 us for 914 MB, 88-93 % of a copy's rate).  One token (27 us for 69 MB) waits for
// the launches' latency: routing, opening and join cost about 2 us each in both.  Rows
// that are no whole number of lines (64 tokens over 64 experts of 2048 x 1000: 173-178 us,
// 66 %; 157 us for 1024) are read partly twice, for two strips; the selection of 64
// tokens takes 10 us of it.
#include <algorithm>
#include <cmath>

#include "tl_internal.h"
#include "tl_ptx.cuh"

namespace tl {
namespace {

constexpr int WARPS = 8;
constexpr int THREADS = WARPS * 32;
constexpr int TILE = 16;             // rows of one product
constexpr int MAX_T = 64, MAX_K = 16, MAX_ROWS = MAX_T * MAX_K;
constexpr int MAX_CTAS = 256;
constexpr int MAX_HD = 65536;
// What a tile costs a CTA beside its steps, in steps: the list of work has that many places before a tile's steps, so that
// runs of equal length take equally long (one token: 29.0 us without, 27.0 us with; no difference from 16 tokens on).
constexpr int LEAD = 4;
constexpr int W_BYTES = 32 * 128;    // one warp's weights of one step: 32 rows of 64 columns

struct MoeParams {
  const void* w[TL_MAX_EXPERTS];
  const uint16_t* x;
  const float* logits;
  uint16_t* out;
  int32_t* ids;
  float* gates;
  uint16_t* act;        // [2][P][I]: the two terms of h, expert-sorted rows
  float* y;             // [P][Hd]
  float* partial;       // [CTAs][2][slot_rows][128 * SUB]
  uint32_t* counters;   // [MAX_CTAS] runs of launch 1, [MAX_CTAS] of launch 2, then one for each column tile and token
  int32_t T, H, I, Hd, E, topk, normalize;
  int32_t slot_rows;    // rows that a tile can have
};

template <bool DOWN, int MT>
struct MoeSmem {
  static constexpr int PLANES = DOWN ? 2 : 1;
  static constexpr int STAGE = W_BYTES + PLANES * MT * 1024;
  static constexpr int STAGES = (24 * 1024) / STAGE;
  uint8_t ring[WARPS][STAGES][STAGE];  // a tile's merge takes the stage that each warp used last
  unsigned long long mask[TL_MAX_EXPERTS];  // the tokens that chose the expert
  float gates[MAX_T][MAX_K];
  uint16_t row_of[MAX_T][MAX_K];            // sorted row of (token, slot)
  uint16_t base[TL_MAX_EXPERTS];            // first sorted row of the expert
  uint16_t tile_expert[TL_MAX_EXPERTS + MAX_ROWS / TILE];
  uint16_t tile_first[TL_MAX_EXPERTS + MAX_ROWS / TILE];  // first sorted row of the row tile
  uint8_t tile_rows[TL_MAX_EXPERTS + MAX_ROWS / TILE];
  uint8_t ids[MAX_T][MAX_K];
  uint8_t row_token[MAX_ROWS];
  int16_t ready[2 * TILE];                  // the tile's tokens that are complete, or -1
  int32_t tiles, last;
};

__device__ __forceinline__ void cp_async16z(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Where the 16 bytes `unit` of a step's weight row lie: a product's loads (unit g of rows 8t + const) meet in no bank.
__device__ __forceinline__ uint32_t w_at(int row, int unit) { return uint32_t(row * 128 + ((unit ^ ((row >> 3) << 1)) << 4)); }
// 16-byte unit c of row r of a warp's 16 x 64 sums
__device__ __forceinline__ int merge_at(int r, int c) { return r * 16 + (c ^ (r & 1) ^ ((c >> 3) << 1)); }

// ---------------------------------------------------------------- routing, by every CTA for itself
// Order of the logits as unsigned keys: larger first, zeros of both signs equal, NaN (1) below -infinity, 0 = taken.
__device__ __forceinline__ uint32_t logit_key(float v) {
  const uint32_t u = __float_as_uint(__fadd_rn(v, 0.0f));  // -0 + 0 = 0
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 1u;
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// One warp selects for N tokens at once (their chains of reductions overlap); J: experts of a lane.
template <int J, int N, class Smem>
__device__ __forceinline__ void select(const MoeParams& p, Smem& sm, int t0, int step, bool write) {
  const int lane = int(lane_id());
  float v[N][J], top[N], chosen[N];
  uint32_t key[N][J];
  int chosen_e[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int t = min(t0 + i * step, p.T - 1);
    top[i] = chosen[i] = -INFINITY;
    chosen_e[i] = 0;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int e = j * 32 + lane;
      v[i][j] = -INFINITY;
      key[i][j] = 0;
      if (e < p.E) {
        v[i][j] = p.logits[int64_t(t) * p.E + e];
        key[i][j] = logit_key(v[i][j]);
      }
    }
  }
  for (int s = 0; s < p.topk; ++s) {
    // step by step for all tokens (reductions keep their order: token by token each would wait for the last one's)
    uint32_t best[N], most[N];
    int at[N], e[N];
    float val[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      best[i] = 0;
      at[i] = 0x7FFFFFFF;
      val[i] = 0.0f;
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (key[i][j] > best[i]) {
          best[i] = key[i][j];
          at[i] = j * 32 + lane;
          val[i] = v[i][j];
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) most[i] = __reduce_max_sync(0xffffffffu, best[i]);
#pragma unroll
    for (int i = 0; i < N; ++i) e[i] = __reduce_min_sync(0xffffffffu, best[i] == most[i] ? at[i] : 0x7FFFFFFF);
#pragma unroll
    for (int i = 0; i < N; ++i) val[i] = __shfl_sync(0xffffffffu, val[i], e[i] & 31);
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
      for (int j = 0; j < J; ++j) key[i][j] = j * 32 + lane == e[i] ? 0u : key[i][j];
      chosen[i] = lane == s ? val[i] : chosen[i];
      chosen_e[i] = lane == s ? e[i] : chosen_e[i];
      top[i] = s == 0 ? val[i] : top[i];
    }
  }
  float sums[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    sums[i] = 0.0f;
    if (p.normalize) {
      if (lane < p.topk) sums[i] = expf(chosen[i] - top[i]);
    } else {
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (j * 32 + lane < p.E) sums[i] += expf(v[i][j] - top[i]);
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) sums[i] += __shfl_xor_sync(0xffffffffu, sums[i], d);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int t = t0 + i * step;
    const float sum = sums[i];
    if (lane < p.topk && t < p.T) {
      const float gate = top[i] == -INFINITY && !(sum > 0.0f) ? 0.0f : expf(chosen[i] - top[i]) / sum;
      sm.ids[t][lane] = uint8_t(chosen_e[i]);
      sm.gates[t][lane] = gate;
      atomicOr(&sm.mask[chosen_e[i]], 1ull << t);
      if (write) {
        p.ids[t * p.topk + lane] = chosen_e[i];
        p.gates[t * p.topk + lane] = gate;
      }
    }
  }
}

template <class Smem>
__device__ void route(const MoeParams& p, Smem& sm, int rows_per_tile, bool write) {
  const int warp = int(warp_id()), lane = int(lane_id());
  for (int e = threadIdx.x; e < p.E; e += THREADS) sm.mask[e] = 0;
  __syncthreads();
  if (p.T <= WARPS && p.E <= 64) {  // a token to a warp: the short form, for what little there is to wait for
    if (warp < p.T) select<2, 1>(p, sm, warp, 0, write);
  } else if (p.E <= 64) {
    for (int t = warp; t < p.T; t += 4 * WARPS) select<2, 4>(p, sm, t, WARPS, write);
  } else {
    for (int t = warp; t < p.T; t += 2 * WARPS) select<TL_MAX_EXPERTS / 32, 2>(p, sm, t, WARPS, write);
  }
  __syncthreads();
  if (warp == 0) {
    // rows and row tiles of each expert: running sums over the experts
    int rows_before = 0, tiles_before = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      const int n = e < p.E ? __popcll(sm.mask[e]) : 0;
      const int m = (n + rows_per_tile - 1) / rows_per_tile;
      int rn = n, rm = m;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, rn, d), b = __shfl_up_sync(0xffffffffu, rm, d);
        if (lane >= d) {
          rn += a;
          rm += b;
        }
      }
      const int base = rows_before + rn - n, tile = tiles_before + rm - m;
      if (e < p.E) sm.base[e] = uint16_t(base);
      for (int i = 0; i < m; ++i) {
        sm.tile_expert[tile + i] = uint16_t(e);
        sm.tile_first[tile + i] = uint16_t(base + i * rows_per_tile);
        sm.tile_rows[tile + i] = uint8_t(min(rows_per_tile, n - i * rows_per_tile));
      }
      rows_before += __shfl_sync(0xffffffffu, rn, 31);
      tiles_before += __shfl_sync(0xffffffffu, rm, 31);
    }
    if (lane == 0) sm.tiles = tiles_before;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.T * p.topk; i += THREADS) {
    const int t = i / p.topk, s = i % p.topk, e = sm.ids[t][s];
    const int row = sm.base[e] + __popcll(sm.mask[e] & ((1ull << t) - 1));
    sm.row_of[t][s] = uint16_t(row);
    sm.row_token[row] = uint8_t(t);
  }
  __syncthreads();
}

// ---------------------------------------------------------------- one launch: up (DOWN = false) or down
// SUB: 64-column strips of a group that lie next to one another; 4 / SUB warps share a strip's contraction
template <bool DOWN, int MT, int SUB>
__global__ void __launch_bounds__(THREADS, 1) moe_decode_kernel(const __grid_constant__ MoeParams p) {
  using Smem = MoeSmem<DOWN, MT>;
  constexpr int STAGES = Smem::STAGES, PLANES = Smem::PLANES;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  constexpr int KQ = 4 / SUB, STEP = 32 * KQ;    // rows of the contraction in one step
  constexpr int WIDE = (DOWN ? 128 : 64) * SUB;  // columns of a tile
  const int group = warp >> 2, sub = (warp & 3) / KQ, kq = warp % KQ;
  if (!DOWN) pdl_launch_dependents();
  route(p, sm, MT * TILE, !DOWN && blockIdx.x == 0);

  // the list of steps; this CTA's run.  Up: (row tile, column tile, step), so that neighbouring column tiles are read
  // at about the same time and a line that two of them share (rows that are no multiple of 128 bytes) is read from
  // memory once.  Down: (column tile, row tile, step), so that column tiles are combined as the launch goes on.
  const int K = DOWN ? p.I : p.H;                      // contraction
  const int cols = DOWN ? p.Hd : p.I;                  // columns of one group's matrix
  const int ld = DOWN ? p.Hd : 2 * p.I;                // weights' row length
  const int col_tiles = (cols + WIDE - 1) / WIDE;
  const int ks = (K + STEP - 1) / STEP;
  const int places = ks + LEAD;
  const int64_t units = int64_t(col_tiles) * sm.tiles, total = units * places;
  const int64_t n = min(int64_t(gridDim.x), max(int64_t(1), units * ks / 2));
  const int64_t cta = blockIdx.x;
  const int64_t run0 = cta < n ? cta * total / n : 0, run1 = cta < n ? (cta + 1) * total / n : 0;
  const int o0 = int(run0 % places);
  auto steps = [&](int64_t at) { return at / places * ks + max(0, int(at % places) - LEAD); };  // of the list's first places
  int64_t f_left = steps(run1) - steps(run0);
  if (f_left <= 0) return;

  // ---------------------------------------------------------------- copies of one warp: a cursor over the run
  const uint32_t ring = smem_u32(sm.ring[warp]);
  struct Cursor {
    int unit, k;
  };
  Cursor f{int(run0 / places), max(0, o0 - LEAD)};
  bool f_open = false;
  const uint16_t* f_w = nullptr;
  bool f_col = false;
  const uint16_t* f_a[MT][2];
  bool f_row[MT][2];
  const int64_t plane = int64_t(p.T) * p.topk * p.I;

  auto open = [&]() {
    const int rt = DOWN ? f.unit % sm.tiles : f.unit / col_tiles, ct = DOWN ? f.unit / sm.tiles : f.unit % col_tiles;
    const int col = ct * WIDE + ((DOWN ? group * SUB : 0) + sub) * 64 + (lane & 7) * 8;
    f_col = col < cols;
    f_w = static_cast<const uint16_t*>(p.w[sm.tile_expert[rt]]) + (f_col ? col + (DOWN ? 0 : group * p.I) : 0);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = m * TILE + h * 8 + g;
        f_row[m][h] = r < sm.tile_rows[rt];
        const int row = f_row[m][h] ? sm.tile_first[rt] + r : 0;
        f_a[m][h] = DOWN ? p.act + int64_t(row) * p.I : p.x + int64_t(f_row[m][h] ? sm.row_token[row] : 0) * p.H;
      }
    f_open = true;
  };
  auto copy_w = [&](int stage) {
    // whole 128-byte lines by eight neighbouring lanes, four rows an instruction
    const int k0 = f.k * STEP + kq * 32 + (lane >> 3);
    const uint32_t dst = ring + uint32_t(stage * Smem::STAGE);
    const uint16_t* src = f_w + (f_col && k0 < K ? int64_t(k0) * ld : 0);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool ok = f_col && k0 + j * 4 < K;
      cp_async16z(dst + w_at((lane >> 3) + j * 4, lane & 7), src + (ok ? int64_t(j * 4) * ld : 0), ok);
    }
  };
  auto copy_a = [&](int stage) {
    const int k0 = f.k * STEP + kq * 32 + t * 8;
    const uint32_t dst = ring + uint32_t(stage * Smem::STAGE + W_BYTES) + uint32_t(lane * 16);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool ok = f_row[m][h] && k0 < K;
        const uint16_t* src = f_a[m][h] + (ok ? k0 : 0);
#pragma unroll
        for (int q = 0; q < PLANES; ++q)
          cp_async16z(dst + uint32_t(((m * 2 + h) * PLANES + q) * 512), src + (ok ? q * plane : 0), ok);
      }
  };
  auto advance = [&]() {
    --f_left;
    if (++f.k == ks) {
      f.k = 0;
      ++f.unit;
      f_open = false;
    }
  };
  if (DOWN) {
    // the first stages' weights, then wait for the first launch, then its results
    const Cursor f0 = f;
    const int64_t left0 = f_left;
    for (int i = 0; i < STAGES - 1 && f_left > 0; ++i) {
      if (!f_open) open();
      copy_w(i);
      advance();
    }
    pdl_wait_previous();
    f = f0;
    f_left = left0;
    f_open = false;
    for (int i = 0; i < STAGES - 1; ++i) {
      if (f_left > 0) {
        if (!f_open) open();
        copy_a(i);
        advance();
      }
      cp_commit();  // the weights are all in the first group
    }
  } else {
    for (int i = 0; i < STAGES - 1; ++i) {
      if (f_left > 0) {
        if (!f_open) open();
        copy_w(i);
        copy_a(i);
        advance();
      }
      cp_commit();
    }
  }

  // ---------------------------------------------------------------- products, tile by tile
  int stage = 0;
  int64_t at = run0;
  while (at < run1) {
    const int unit = int(at / places), o = int(at % places), used = int(min(int64_t(places - o), run1 - at));
    const int k_begin = max(0, o - LEAD), k_end = o + used - LEAD;
    if (k_end <= k_begin) break;  // the run ends before a tile's first step
    const int rt = DOWN ? unit % sm.tiles : unit / col_tiles, ct = DOWN ? unit / sm.tiles : unit % col_tiles;
    const int rows = sm.tile_rows[rt], row0 = sm.tile_first[rt];
    float acc[MT][8][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[m][i][j] = 0.0f;

    for (int k = k_begin; k < k_end; ++k) {
      cp_wait<STAGES - 2>();
      __syncwarp();
      const uint32_t src = ring + uint32_t(stage * Smem::STAGE);
      uint32_t a[MT][2][PLANES][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int q = 0; q < PLANES; ++q) {
            const uint4 w = lds128(src + uint32_t(W_BYTES + ((m * 2 + h) * PLANES + q) * 512 + lane * 16));
            a[m][h][q][0] = w.x;
            a[m][h][q][1] = w.y;
            a[m][h][q][2] = w.z;
            a[m][h][q][3] = w.w;
          }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t w[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 v = lds128(src + w_at(t * 8 + u * 4 + j, g));
          w[j][0] = v.x;
          w[j][1] = v.y;
          w[j][2] = v.z;
          w[j][3] = v.w;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t sel = (i & 1) ? 0x7632u : 0x5410u;
          const uint32_t b0 = __byte_perm(w[0][i >> 1], w[1][i >> 1], sel);
          const uint32_t b1 = __byte_perm(w[2][i >> 1], w[3][i >> 1], sel);
#pragma unroll
          for (int m = 0; m < MT; ++m)
            if (m == 0 || rows > m * TILE) {
#pragma unroll
              for (int q = PLANES - 1; q >= 0; --q)
                mma_bf16(acc[m][i], a[m][0][q][2 * u], a[m][1][q][2 * u], a[m][0][q][2 * u + 1], a[m][1][q][2 * u + 1],
                         b0, b1);
            }
        }
      }
      {
        const int next = stage + STAGES - 1 >= STAGES ? stage - 1 : stage + STAGES - 1;
        if (f_left > 0) {
          if (!f_open) open();
          copy_w(next);
          copy_a(next);
          advance();
        }
        cp_commit();
        stage = stage + 1 == STAGES ? 0 : stage + 1;
      }
    }

    // ---------------------------------------------------------------- the warps' sums become one; sixteen threads to a row
    const bool whole = k_begin == 0 && k_end == ks;
    const int64_t t0 = at - o + LEAD;  // the tile's first step in the list
    const int row = tid >> 4, c4 = tid & 15;
    const int64_t slot_size = int64_t(p.slot_rows) * (128 * SUB);
    float* slot = p.partial + (2 * cta + (k_begin == 0 ? 1 : 0)) * slot_size;
    // four columns of each group: [0..3] group 0, [4..7] group 1, at column 4 c4 of strip s
    auto finish = [&](int m, int s, const float(&v)[8]) {
      const int r = m * TILE + row;
      if (r >= rows) return;
      if (!DOWN) {
        const int col = ct * WIDE + s * 64 + 4 * c4;
        if (col >= p.I) return;
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float h[2], rest[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float gate = v[2 * i + j];
            h[j] = gate / (1.0f + expf(-gate)) * v[4 + 2 * i + j];
          }
          hi[i] = pack_bf16x2(h[0], h[1]);
          const float b0 = __uint_as_float(hi[i] << 16), b1 = __uint_as_float(hi[i] & 0xFFFF0000u);
          rest[0] = isfinite(b0) ? h[0] - b0 : 0.0f;  // an infinity has no second term
          rest[1] = isfinite(b1) ? h[1] - b1 : 0.0f;
          lo[i] = pack_bf16x2(rest[0], rest[1]);
        }
        uint16_t* dst = p.act + int64_t(row0 + r) * p.I + col;
        *reinterpret_cast<uint2*>(dst) = make_uint2(hi[0], hi[1]);
        *reinterpret_cast<uint2*>(dst + plane) = make_uint2(lo[0], lo[1]);
      } else {
        const int col = ct * WIDE + s * 64 + 4 * c4;
        float* dst = p.y + int64_t(row0 + r) * p.Hd + col;
        if (col < p.Hd) st_global_cg_v4f(dst, v[0], v[1], v[2], v[3]);
        if (col + SUB * 64 < p.Hd) st_global_cg_v4f(dst + SUB * 64, v[4], v[5], v[6], v[7]);
      }
    };
    const int spare = stage == 0 ? STAGES - 1 : stage - 1;  // the stage that the warp's next copy will fill: all warps' alike
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (m > 0 && rows <= m * TILE) break;
      if (m > 0) __syncthreads();
      float4* buf = reinterpret_cast<float4*>(sm.ring[warp][spare]);
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i4 = 0; i4 < 2; ++i4)
            buf[merge_at(g + 8 * x, 4 * t + 2 * h + i4)] =
                make_float4(acc[m][4 * i4][2 * x + h], acc[m][4 * i4 + 1][2 * x + h], acc[m][4 * i4 + 2][2 * x + h],
                            acc[m][4 * i4 + 3][2 * x + h]);
      __syncthreads();
#pragma unroll
      for (int s = 0; s < SUB; ++s) {
        float v[8];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float4 a = reinterpret_cast<const float4*>(sm.ring[4 * q + s * KQ][spare])[merge_at(row, c4)];
#pragma unroll
          for (int w = 1; w < KQ; ++w) {
            const float4 b = reinterpret_cast<const float4*>(sm.ring[4 * q + s * KQ + w][spare])[merge_at(row, c4)];
            a.x += b.x;
            a.y += b.y;
            a.z += b.z;
            a.w += b.w;
          }
          v[4 * q] = a.x;
          v[4 * q + 1] = a.y;
          v[4 * q + 2] = a.z;
          v[4 * q + 3] = a.w;
        }
        if (whole) {
          finish(m, s, v);
        } else if (m * TILE + row < rows) {
          float* dst = slot + (m * TILE + row) * (128 * SUB) + s * 64 + 4 * c4;
          st_global_cg_v4f(dst, v[0], v[1], v[2], v[3]);
          st_global_cg_v4f(dst + SUB * 64, v[4], v[5], v[6], v[7]);
        }
      }
    }
    bool done = whole;
    if (!whole) {
      const int64_t c0 = ((t0 + 1) * n - 1) / total, c1 = ((t0 + ks) * n - 1) / total;
      uint32_t* counter = p.counters + (DOWN ? MAX_CTAS : 0) + c0;
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        sm.last = atomicAdd(counter, 1u) == uint32_t(c1 - c0);
        if (sm.last) *counter = 0;
      }
      __syncthreads();
      done = sm.last;
      if (done) {
        __threadfence();
        for (int m = 0; m * TILE < rows; ++m) {
          float v[SUB][8] = {};  // the strips' parts of a CTA on their way together
          if (m * TILE + row < rows) {
#pragma unroll 2
            for (int64_t c = c0; c <= c1; ++c) {
              const float* src = p.partial + (2 * c + (c == c0)) * slot_size + (m * TILE + row) * (128 * SUB) + 4 * c4;
#pragma unroll
              for (int s = 0; s < SUB; ++s) {
                const float4 a = ld_global_cg_v4f(src + s * 64), b = ld_global_cg_v4f(src + s * 64 + SUB * 64);
                v[s][0] += a.x;
                v[s][1] += a.y;
                v[s][2] += a.z;
                v[s][3] += a.w;
                v[s][4] += b.x;
                v[s][5] += b.y;
                v[s][6] += b.z;
                v[s][7] += b.w;
              }
            }
          }
#pragma unroll
          for (int s = 0; s < SUB; ++s) finish(m, s, v[s]);
        }
      }
    }
    if (DOWN && done) {
      // combine the column tile for every token whose last slot this tile was
      __threadfence();
      __syncthreads();
      if (tid < rows) {
        const int tok = sm.row_token[row0 + tid];
        uint32_t* counter = p.counters + 2 * MAX_CTAS + ct * MAX_T + tok;
        const bool last = atomicAdd(counter, 1u) == uint32_t(p.topk - 1);
        if (last) *counter = 0;
        sm.ready[tid] = last ? tok : -1;
      }
      __syncthreads();
      __threadfence();
      constexpr int TPT = WIDE / 4;  // threads to a token
      for (int r = tid / TPT; r < rows; r += THREADS / TPT) {
        const int tok = sm.ready[r], col = ct * WIDE + tid % TPT * 4;
        if (tok < 0 || col >= p.Hd) continue;
        float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int s0 = 0; s0 < p.topk; s0 += 8) {
          float4 w[8];
#pragma unroll
          for (int s = 0; s < 8; ++s)  // all on their way at once
            w[s] = ld_global_cg_v4f(p.y + int64_t(sm.row_of[tok][min(s0 + s, p.topk - 1)]) * p.Hd + col);
#pragma unroll
          for (int s = 0; s < 8; ++s) {
            if (s0 + s >= p.topk) break;
            const float gate = sm.gates[tok][s0 + s];
            o[0] = fmaf(gate, w[s].x, o[0]);
            o[1] = fmaf(gate, w[s].y, o[1]);
            o[2] = fmaf(gate, w[s].z, o[2]);
            o[3] = fmaf(gate, w[s].w, o[3]);
          }
        }
        *reinterpret_cast<uint2*>(p.out + int64_t(tok) * p.Hd + col) =
            make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
      }
    }
    at += used;
    __syncthreads();  // the spare stages are free again
  }
  cp_wait<0>();
}

struct MoeLayout {
  size_t partial, act, y, bytes;
};
size_t up256(size_t v) { return (v + 255) / 256 * 256; }
MoeLayout moe_layout(int T, int topk, int I, int Hd) {
  const size_t P = size_t(T) * topk;
  MoeLayout l{};
  // the counters' place does not depend on the sizes: one workspace may serve calls of many
  l.partial = up256((2 * MAX_CTAS + size_t(MAX_HD / 128) * MAX_T) * 4);
  l.act = l.partial + size_t(MAX_CTAS) * 2 * std::min(T, 2 * TILE) * 512 * 4;
  l.y = l.act + up256(P * I * 2 * 2);
  l.bytes = l.y + P * Hd * 4;
  return l;
}
bool moe_sizes_ok(int T, int topk, int E, int H, int I, int Hd) {
  return T >= 0 && T <= MAX_T && E >= 1 && E <= TL_MAX_EXPERTS && topk >= 1 && topk <= MAX_K && topk <= E && H >= 8 &&
         H % 8 == 0 && I >= 8 && I % 8 == 0 && Hd >= 8 && Hd % 8 == 0 && H <= (1 << 20) && I <= (1 << 20) &&
         Hd <= MAX_HD;
}

template <bool DOWN, int MT>
tl_status launch_moe(const MoeParams& p, int sub, int ctas, cudaStream_t st) {
  static_assert(sizeof(MoeSmem<DOWN, MT>) <= 232448, "shared memory above the per-CTA limit");
  const void* kernel = sub == 4   ? reinterpret_cast<const void*>(&moe_decode_kernel<DOWN, MT, 4>)
                       : sub == 2 ? reinterpret_cast<const void*>(&moe_decode_kernel<DOWN, MT, 2>)
                                  : reinterpret_cast<const void*>(&moe_decode_kernel<DOWN, MT, 1>);
  void* args[] = {const_cast<MoeParams*>(&p)};
  return launch(kernel, ctas, THREADS, sizeof(MoeSmem<DOWN, MT>), st, args, DOWN);
}

// Strips of 64 columns next to one another in a tile of `one * sub` columns: the width that reads least.  Columns that a
// last tile lacks cost the time of their strips; where the rows are no multiples of 128 bytes, a tile's two edges cost
// about a line in each row (reads 1.84 times the weights with strips alone, 64 x 2048 x 2000: 161 us, 124 us with four).
// Of equals the widest, which has the fewest tiles to finish.  With fewer tiles than CTAs, strips alone: a tile is then
// shared by fewer CTAs (one token, two experts of 4096 x 1408: 31 us, 38 us with the widest).
int strips(int cols, int one, bool aligned, int row_tiles, int ctas) {
  int best = 1;
  double least = 1e30;
  for (int sub : {1, 2, 4}) {
    const int tiles = cdiv(cols, one * sub);
    const double cost = double(tiles) * sub * (aligned ? 1.0 : 1.0 + 0.84 / sub);
    if (cost <= least && (sub == 1 || tiles * row_tiles >= ctas)) {
      least = cost;
      best = sub;
    }
  }
  return best;
}

}  // namespace
}  // namespace tl

extern "C" size_t tl_moe_decode_workspace_size(int T, int topk, int E, int H, int I, int Hd) {
  return tl::moe_sizes_ok(T, topk, E, H, I, Hd) ? tl::moe_layout(T, topk, I, Hd).bytes : 0;
}

extern "C" tl_status tl_moe_decode(const tl_moe_decode_args* a, void* stream) {
  using namespace tl;
  if (!a) return fail(TL_ERR_INVALID, "tl_moe_decode: NULL args");
  if (a->T < 0 || a->H < 1 || a->I < 1 || a->Hd < 1 || a->E < 1 || a->topk < 1 || a->topk > a->E)
    return fail(TL_ERR_INVALID, "tl_moe_decode: T %d, H %d, I %d, Hd %d, E %d, topk %d", a->T, a->H, a->I, a->Hd, a->E,
                a->topk);
  if (!moe_sizes_ok(a->T, a->topk, a->E, a->H, a->I, a->Hd))
    return fail(TL_ERR_UNSUPPORTED,
                "tl_moe_decode: up to %d tokens, %d experts, top %d; H, I and Hd multiples of 8 (T %d, H %d, I %d, Hd "
                "%d, E %d, topk %d)",
                MAX_T, TL_MAX_EXPERTS, MAX_K, a->T, a->H, a->I, a->Hd, a->E, a->topk);
  if (a->normalize != 0 && a->normalize != 1)
    return fail(TL_ERR_INVALID, "tl_moe_decode: normalize %d", a->normalize);
  if (a->T == 0) return TL_OK;
  if (!a->x || !a->logits || !a->W1 || !a->W2 || !a->out || !a->ids || !a->gates || !a->workspace)
    return fail(TL_ERR_INVALID, "tl_moe_decode: NULL pointer argument");
  for (const void* ptr : {a->x, (const void*)a->out, (const void*)a->workspace})
    if (!aligned16(ptr)) return fail(TL_ERR_INVALID, "tl_moe_decode: pointers must be 16-byte aligned");
  for (const void* ptr : {(const void*)a->logits, (const void*)a->ids, (const void*)a->gates})
    if (reinterpret_cast<uintptr_t>(ptr) & 3u)
      return fail(TL_ERR_INVALID, "tl_moe_decode: logits, ids and gates must be 4-byte aligned");
  const MoeLayout l = moe_layout(a->T, a->topk, a->I, a->Hd);
  if (a->workspace_bytes < l.bytes)
    return fail(TL_ERR_INVALID, "tl_moe_decode: workspace of %zu bytes, need %zu", a->workspace_bytes, l.bytes);
  MoeParams p{};
  for (int e = 0; e < a->E; ++e) {
    if (!a->W1[e] || !a->W2[e] || !aligned16(a->W1[e]) || !aligned16(a->W2[e]))
      return fail(TL_ERR_INVALID, "tl_moe_decode: weights of expert %d", e);
    p.w[e] = a->W1[e];
  }
  DeviceInfo di{};
  if (tl_status s = device_info(&di)) return s;
  uint8_t* ws = static_cast<uint8_t*>(a->workspace);
  p.x = static_cast<const uint16_t*>(a->x);
  p.logits = a->logits;
  p.out = static_cast<uint16_t*>(a->out);
  p.ids = a->ids;
  p.gates = a->gates;
  p.counters = reinterpret_cast<uint32_t*>(ws);
  p.partial = reinterpret_cast<float*>(ws + l.partial);
  p.act = reinterpret_cast<uint16_t*>(ws + l.act);
  p.y = reinterpret_cast<float*>(ws + l.y);
  p.T = a->T;
  p.H = a->H;
  p.I = a->I;
  p.Hd = a->Hd;
  p.E = a->E;
  p.topk = a->topk;
  p.normalize = a->normalize;
  const int ctas = std::min(di.sm_count, MAX_CTAS);
  // Row tiles of 32 where an expert expects more than a tile of 16: its weights are then read once for both
  const bool two = a->T > TILE && a->T * a->topk > 12 * a->E;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  p.slot_rows = std::min(a->T, two ? 2 * TILE : TILE);
  const int row_tiles = std::min(a->E, a->T * a->topk);  // about as many experts are chosen
  const int up = strips(a->I, 64, a->I % 32 == 0, row_tiles, ctas), down = strips(a->Hd, 128, a->Hd % 64 == 0, row_tiles, ctas);
  if (tl_status s = two ? launch_moe<false, 2>(p, up, ctas, st) : launch_moe<false, 1>(p, up, ctas, st)) return s;
  for (int e = 0; e < a->E; ++e) p.w[e] = a->W2[e];
  return two ? launch_moe<true, 2>(p, down, ctas, st) : launch_moe<true, 1>(p, down, ctas, st);
}
