// tl_kv_attn.cu -- attention of a ragged batch's new tokens over the 8-bit paged
// cache: the split kernel for few query rows per kv head (single tokens, drafts).
//
//   s_j = scale <q, k_j>,  O = sum_j exp(s_j - lse) v_j
//
// The cache is read once; everything else is small, so the kernel is a stream of
// pages through the SMs, by one CTA each where there are few tiles.  The work is the list of (sequence, kv head,
// tile of 8 or 16 rows, 32-token chunk), cut into equal runs, one to a CTA: a long context
// is spread over many CTAs and short ones share a CTA, whatever the mix.  Runs are
// found on the device from the lengths, so the host needs no lengths.  A tile
// whose chunks fall to several CTAs leaves partial results (mean value, maximum,
// sum) in the workspace; the CTA that arrives last joins them in CTA order, so
// the result does not depend on timing.
//
// Inside a CTA the warps (of an SM 12 for tiles of 8 rows, 8 for 16, which need the registers)
// take a run's chunks of 32 tokens in turn, each on its own.  Keys and values are the products' first operand (S^T = K Q^T, O^T = V^T P^T):
// 16 tokens or dims by 8 query rows, so a tile of 8 rows wastes little of a product,
// and a tile of 16 takes two.
//  * The contraction index of a product may be permuted at will if both operands
//    are.  So lane (g, t) multiplies, for key g, the dims of two 16-byte units of that
//    key's codes, and for values four tokens' 16 dims: wide loads from the chunk as it
//    lies in the cache, nothing transposed.  Each warp copies (cp.async) whole tokens
//    into a ring of its own, so no barrier stands between copy and use; P^T comes from
//    S^T by 8 x 8 transpositions in registers (movmatrix).
//  * e4m3 to fp16 is exact (one conversion for two codes).  Queries are brought
//    to fp16 by a power of two for each row, off by at most 2^-25 of the row's
//    largest element.  The K scale multiplies the scores in fp32, the V scale of the
//    half chunk relative to a reference multiplies P, both powers of two.
//  * That reference is one for the warp's rows while the V scales that it meets lie within
//    2^3 of the first ones, as they mostly do (64 single tokens over 8192 take 132 us with it
//    and 140 us without, 16 drafts of 4 over 6000 40 and 50 us, in a graph).  Otherwise each row has its own,
//    2^e with e at least what the largest product of weight and scale asks for among the keys
//    that the row sees: P times the scale relative to 2^e is at most 2^7, and a block that the
//    row does not see, or hardly, takes no bits from the others.
//  * P is kept as exp2(s - m + 7) with m raised only when a score passes it by 8:
//    at most 2^15, in fp16 with full precision down to 2^-21 of the largest and a
//    grain of 2^-31 of it, so even a tail of millions of small weights counts.
//    Sums of P are taken in fp32 before P is rounded.
//
// Bound by memory when there are many tokens to read: 64 single tokens over 8192 at most
// (8 kv heads of 128): 136 us for 826 MB, 91 % of a copy's rate; three over 131072 at most,
// 102 us for 615 MB, 90 %.  Copies of 64-byte half lines, which fit the products' lanes
// without a swizzle, ran at 75 %.  A single short context (14 us for 8 MB, 13 us in a
// graph) is a chain of loads that wait for one another (lengths, page, scale and codes,
// merge, the join); 16-row tiles (16 sequences of 4 drafts over 6000 at most: 43 us for
// 141 MB, 49 %) lose to opening and joining tiles, 8000 cycles each, and to eight warps'
// latency: their 255 registers leave no room for more.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "tl_internal.h"
#include "tl_kv.cuh"
#include "tl_kv_prefill.h"

namespace tl {
namespace {

constexpr int MAX_TILE = 16;  // query rows of one tile: 8 or 16
constexpr int CHUNK = 32;     // tokens of one chunk; its halves of 16 lie in one page each
// Query rows per kv head up to which this kernel serves a sequence.  It reads the cache once for each 16 of them (16
// sequences of 6000: 85 us for 32 rows, 152 us for 64); the kernel for many rows takes as long for a few as for 128
// (100 us), but has more to set up (one sequence of 16000: 37 us here for 64 rows, 72 us there).
int few_rows(int B) { return B >= 8 ? 32 : 64; }
// What a tile costs a CTA beside its chunks, in chunks (about 9000 cycles): the list of work has that many places before a
// tile's chunks, so that runs of equal length take equally long (16 sequences of 4 drafts over 6000: 45 -> 41 us; 200
// single tokens over 300 each: 72 -> 57 us).
constexpr int LEAD = 24;
// CTAs of an SM, by the tiles of 8 (16) query rows that a batch has at least.  While one opens or joins a tile, which takes
// latency and no bandwidth, the others read; but a tile cut among more CTAs takes longer to join.  For tiles of 8, with 1, 2
// and 4 of 12, 6 and 3 warps, 8 kv heads: 200 tokens over 300 57, 39, 29 us; 76 over 1500 47, 41, 38 us; 38 over 500 23,
// 12, 15 us; 24 over 2000 25, 21, 25 us; 19 over 500 12, 13, 14 us; one over 4099 15, 18, 29 us; 64 over 8192 132, 133, 134 us.
// For tiles of 16, with 1 and 2 of 8 and 4 warps: 32 sequences of 4 tokens over 3000 37, 35 us; 16 over 750 14, 16 us.
constexpr int MAX_PER_SM = 4;
int per_sm(int64_t tiles, bool small, int sms) { return tiles <= sms ? 1 : small && tiles > 3 * sms ? 4 : 2; }
constexpr float kShift = 7.0f;
constexpr float kSlack = 8.0f;
// A warp's reference for a tile's value blocks is 2^kRoom above the first ones' scale; it serves scales up to it and down
// to 2^kNear below.
constexpr int kRoom = 3, kNear = 6;
constexpr int kOwn = 1000;  // above all scales: once a row has its own reference it keeps it

struct DecodeParams {
  KvCacheDev c;
  KvBatch b;
  const uint16_t* q;
  int64_t q_ts, q_hs;
  uint16_t* out;
  float* lse;
  uint32_t* counters;  // [CTAs], zero between calls; CTAs up to MAX_PER_SM times the SMs
  float* partial;      // [CTAs][2][TILE * D + 2 * TILE]
  int32_t H, group, causal;
  int32_t max_rows;    // sequences of more query rows per kv head are left to the kernel for many
  float scale_log2;
};

template <int D, int NR, int WARPS, int PER_SM>
struct DecodeSmem {
  static constexpr int TILE = 8 * NR;
  static constexpr int STAGES = 24 / WARPS / PER_SM;  // 192 KB of an SM for head_dim 128
  static constexpr int STAGE = CHUNK * D * 2;  // bytes of one chunk, keys and values
  uint8_t ring[WARPS][STAGES][STAGE];          // a tile's merge takes the stage that each warp used last
  float2 ml[TILE][WARPS];                      // maximum and sum of each row and warp
  int32_t e[TILE][WARPS];                      // what the row's sums are in units of: 2^e
  uint2 meta[WARPS][STAGES];  // scale bytes (k, v of the first half, k, v of the second); which halves' pages are good
  int32_t spare[WARPS];
  int64_t warp_sum[WARPS];
  int32_t warp_items[WARPS];
  int64_t begin_off;
  int32_t begin_seq, last;
  int32_t pieces[WARPS];
};

// One run's piece of one tile: chunks cb .. ce-1 of the tile's nch.
struct Segment {
  KvSeq seq;
  int s, nch, tiles, hk, rt, cb, ce;  // kv head and row tile
  int o, used;                        // places of the list: of the piece's first in its tile, and how many it takes
  int64_t left;                       // of the run from there on
};

// a / b, in 32 bits where that is enough (a 64-bit division takes about 500 cycles)
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) ? a / b : int64_t(uint32_t(a) / uint32_t(b));
}
template <int TILE>
__device__ __forceinline__ int seq_tiles(const DecodeParams& p, const KvSeq& q) {
  const uint32_t rows = uint32_t(q.q) * uint32_t(p.group);  // in 31 bits (checked by the host)
  return rows > uint32_t(p.max_rows) ? 0 : int((rows + TILE - 1) / TILE);
}
__device__ __forceinline__ int seq_chunks(const KvSeq& q) { return max(1, (q.len + CHUNK - 1) / CHUNK); }

__device__ __forceinline__ void seg_cut(Segment& g, int o) {
  g.o = o;
  g.used = int(min(int64_t(g.nch + LEAD - o), g.left));
  g.cb = max(0, o - LEAD);
  g.ce = o + g.used - LEAD;  // not above cb: nothing but places that stand for a tile's cost
}
template <int TILE>
__device__ __forceinline__ void seg_open(const DecodeParams& p, Segment& g, int s, int64_t off, int64_t left) {
  g.seq = kv_seq(p.b, p.c.ps, s);
  g.s = s;
  g.nch = seq_chunks(g.seq);
  g.tiles = seq_tiles<TILE>(p, g.seq);
  const int sub = int(quotient(off, g.nch + LEAD));
  g.hk = sub / max(g.tiles, 1);
  g.rt = sub - g.hk * g.tiles;
  g.left = left;
  seg_cut(g, int(off - int64_t(sub) * (g.nch + LEAD)));
}
template <int TILE>
__device__ __forceinline__ bool seg_next(const DecodeParams& p, Segment& g) {
  g.left -= g.used;
  if (g.left <= LEAD) return false;
  if (++g.rt == g.tiles) {
    g.rt = 0;
    ++g.hk;
  }
  if (g.hk < p.c.Hkv) {
    seg_cut(g, 0);
    return true;
  }
  int s = g.s + 1;
  while (s < p.b.B && seq_tiles<TILE>(p, kv_seq(p.b, p.c.ps, s)) == 0) ++s;
  if (s >= p.b.B) return false;
  seg_open<TILE>(p, g, s, 0, g.left);
  return true;
}

// 16 bytes, zeros when not ok
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(const uint8_t* a) { return *reinterpret_cast<const uint4*>(a); }
__device__ __forceinline__ uint2 lds64(const uint8_t* a) { return *reinterpret_cast<const uint2*>(a); }
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
// over the eight lanes that share t
__device__ __forceinline__ float column_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
__device__ __forceinline__ float column_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 4);
  x += __shfl_xor_sync(0xffffffffu, x, 8);
  return x + __shfl_xor_sync(0xffffffffu, x, 16);
}
// Transpose of an 8 x 8 matrix of 16-bit elements, two to a lane
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// Where 16-byte unit `unit` of a chunk's token `row` lies, so that neither the copies (whole tokens by
// neighbouring lanes) nor a product's loads (keys: unit t or 4 + t of tokens g; values: unit g, or half of
// unit g / 2, of tokens 2t) meet in a bank.
template <int D>
__device__ __forceinline__ int k_at(int row, int unit) {
  return D == 128 ? row * 128 + ((unit ^ ((row & 1) << 2)) << 4) : row * 64 + (unit << 4);
}
template <int D>
__device__ __forceinline__ int v_at(int row, int unit) {
  return D == 128 ? row * 128 + ((unit ^ (row & 7)) << 4)
                  : (row >> 1) * 128 + (((((row & 1) << 2) | unit) ^ (((row >> 1) & 3) << 1)) << 4);
}
// Which bytes are e4m3 NaN (0x7f, 0xff): 0x80 there.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// 16-byte unit c of row r in a merge buffer (the exclusive-or spreads a column's lanes over the banks)
template <int D>
__device__ __forceinline__ int merge_at(int r, int c) {
  return r * (D / 4) + (c ^ ((c >> 3) & 3) ^ ((r >> 1) & 3));
}

// A row's own reference (at `at`, 2^e) and maximum (mo, now mn) move on: h0 and h1 are the lane's largest scores of a chunk's
// halves, b0 and b1 their value scales' bytes.  Returns what the row's sum and its O have to be multiplied by.
__device__ __noinline__ float2 own_reference(int32_t* at, float mo, float mn, float h0, float h1, int b0, int b1) {
  const int eo = *at;
  h0 = column_max(h0);
  h1 = column_max(h1);
  int e = mo == -INFINITY ? -127 : max(eo + int(ceilf(fmaxf(mo - mn, -1000.0f))), -127);
  if (b0 != 255 && h0 > -INFINITY) e = max(e, b0 - 127 + int(ceilf(fmaxf(h0 - mn, -1000.0f))));
  if (b1 != 255 && h1 > -INFINITY) e = max(e, b1 - 127 + int(ceilf(fmaxf(h1 - mn, -1000.0f))));
  __syncwarp();
  if (lane_id() < 4) *at = e;
  __syncwarp();
  return make_float2(mo != mn ? ex2_approx(mo - mn) : 1.0f, mo == -INFINITY ? 1.0f : ex2_approx(mo - mn + float(eo - e)));
}

// NR: products of 8 query rows to a tile
// PER_SM: CTAs of an SM
template <int D, int NR, int WARPS, int PER_SM>
__global__ void __launch_bounds__(WARPS * 32, PER_SM) kv_decode_kernel(const __grid_constant__ DecodeParams p) {
  using Smem = DecodeSmem<D, NR, WARPS, PER_SM>;
  constexpr int THREADS = WARPS * 32, STAGES = Smem::STAGES;
  constexpr int TILE = 8 * NR;
  constexpr int KL = D / 64;   // 16-byte key loads of one lane and key
  constexpr int MTS = D / 16;  // m tiles of the output
  constexpr int VB = D / 8;    // value bytes of one lane and token: dims g * VB + (0 .. VB-1)
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const KvBatch& b = p.b;

  // ---------------------------------------------------------------- this CTA's run of chunks
  const int per = (b.B + THREADS - 1) / THREADS;
  const int first = min(b.B, tid * per), end = min(b.B, first + per);
  int64_t mine = 0;
  uint32_t items = 0;
  for (int s = first; s < end; ++s) {
    const KvSeq q = kv_seq(b, p.c.ps, s);
    const int tiles = seq_tiles<TILE>(p, q) * p.c.Hkv;
    items += uint32_t(tiles);
    mine += int64_t(tiles) * (seq_chunks(q) + LEAD);
  }
  int64_t before = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, before, d);
    if (lane >= d) before += x;
  }
  items = __reduce_add_sync(0xffffffffu, items);
  if (lane == 31) {
    sm.warp_sum[warp] = before;
    sm.warp_items[warp] = int(items);
  }
  __syncthreads();
  int64_t total = 0, all_items = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w == warp) before += total;
    total += sm.warp_sum[w];
    all_items += sm.warp_items[w];
  }
  before -= mine;
  const int64_t chunks = total - all_items * LEAD;
  Segment f, c;  // where copies are, and where products are
  // A run's first place in the list and the number of runs; a tile's CTAs where runs end with tiles (below 0: they do not).
  const int64_t cta = blockIdx.x;
  int64_t run0 = 0, n = 0;
  int tile_c0 = -1, tile_c1 = -1;
  if (total == 0) {
    pdl_wait_previous();
    return;
  }
  if (all_items <= int64_t(gridDim.x)) {
    // Few tiles: a CTA that works on two of them pays for two merges one after the other, so each tile is cut for
    // itself, into pieces of at most L chunks, with the least L that the CTAs suffice for.  Each warp tries one L.
    constexpr int TRY = (LEAD + WARPS - 2) / (WARPS - 1);
    const int least = max(WARPS, int(quotient(chunks + gridDim.x - 1, gridDim.x)));
    uint32_t pieces = 0;
    for (int s = lane; s < b.B; s += 32) {
      const KvSeq q = kv_seq(b, p.c.ps, s);
      const int L = least + warp * TRY;
      pieces += uint32_t(seq_tiles<TILE>(p, q) * p.c.Hkv) * uint32_t((seq_chunks(q) + L - 1) / L);
    }
    pieces = __reduce_add_sync(0xffffffffu, pieces);
    if (lane == 0) sm.pieces[warp] = int(pieces);
    __syncthreads();
    int w = 0;
    while (w < WARPS && sm.pieces[w] > int(gridDim.x)) ++w;
    if (w < WARPS) {
      if (cta >= sm.pieces[w]) {
        pdl_wait_previous();
        return;
      }
      const int L = least + w * TRY;
      int at = int(cta);
      for (int s0 = 0;; s0 += 32) {  // the sequence that this CTA's piece is of
        const int s = s0 + lane;
        int cnt = 0;
        if (s < b.B) {
          const KvSeq q = kv_seq(b, p.c.ps, s);
          cnt = seq_tiles<TILE>(p, q) * p.c.Hkv * ((seq_chunks(q) + L - 1) / L);
        }
        int sum = cnt;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, sum, d);
          if (lane >= d) sum += x;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, at < sum);
        if (hit) {
          const int src = __ffs(hit) - 1;
          at -= __shfl_sync(0xffffffffu, sum - cnt, src);
          seg_open<TILE>(p, c, s0 + src, 0, 1);
          break;
        }
        at -= __shfl_sync(0xffffffffu, sum, 31);
      }
      const int parts = (c.nch + L - 1) / L, sub = at / parts, part = at - sub * parts;
      c.hk = sub / c.tiles;
      c.rt = sub - c.hk * c.tiles;
      c.cb = int(quotient(int64_t(c.nch) * part, parts));
      c.ce = int(quotient(int64_t(c.nch) * (part + 1), parts));
      c.left = c.used = c.ce - c.cb;
      tile_c0 = int(cta) - part;
      tile_c1 = tile_c0 + parts - 1;
    }
  }
  if (tile_c0 < 0) {
    // a CTA gets a chunk for each warp at least
    n = min(int64_t(gridDim.x), max(int64_t(1), quotient(chunks, WARPS)));
    run0 = cta < n ? quotient(cta * total, n) : 0;
    const int64_t run1 = cta < n ? quotient((cta + 1) * total, n) : 0;
    if (run0 >= run1) {
      pdl_wait_previous();
      return;
    }
    if (mine > 0 && before <= run0 && run0 < before + mine) {
      int64_t at = before;
      for (int s = first; s < end; ++s) {
        const KvSeq q = kv_seq(b, p.c.ps, s);
        const int64_t size = int64_t(seq_tiles<TILE>(p, q)) * p.c.Hkv * (seq_chunks(q) + LEAD);
        if (run0 < at + size) {
          sm.begin_seq = s;
          sm.begin_off = run0 - at;
          break;
        }
        at += size;
      }
    }
    __syncthreads();
    seg_open<TILE>(p, c, sm.begin_seq, sm.begin_off, run1 - run0);
    if (c.ce <= c.cb) {
      pdl_wait_previous();
      return;
    }
  }
  f = c;

  // ---------------------------------------------------------------- the copies of one warp
  const uint32_t ring = smem_u32(sm.ring[warp]);
  const int page_halves = p.c.ps / 16;
  constexpr int UNITS = D / 16, RPC = 32 / UNITS;  // 16-byte units of a token, tokens of one copy instruction
  const int64_t lane_off = int64_t(lane / UNITS) * p.c.token_stride + lane % UNITS * 16;
  const int64_t rows_off = RPC * p.c.token_stride;
  bool f_ok = true, f_new = true;
  int fc = f.cb + warp, f_at = 0;
  int64_t offs[2] = {-1, -1};  // of the lane's chunk: where its halves begin in the pool, below 0: nowhere
  uint32_t scale_bytes[2][2] = {{0, 0}, {0, 0}};
  auto settle = [&]() {  // on to a segment that has a chunk for this warp
    while (f_ok && fc >= f.ce) {
      f_ok = seg_next<TILE>(p, f);
      fc = f.cb + warp;
      f_new = true;
    }
  };
  settle();
  auto fetch = [&](int stage) {
    if (f_ok) {
      if (f_new || f_at == 32) {  // the next 32 chunks' pages and scales, a chunk to a lane
        f_new = false;
        f_at = 0;
        const int ch = fc + lane * WARPS;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int half = ch * 2 + h;
          offs[h] = -1;
          scale_bytes[h][0] = scale_bytes[h][1] = h ? scale_bytes[0][1] : 0u;  // nothing of another tile's stays
          if (ch < f.ce && half * 16 < f.seq.len) {
            const int no = half / page_halves;
            const int page = __ldg(b.table + int64_t(f.s) * b.max_pages + no);
            if (page < 0 || page >= p.c.num_pages) {
              record_error(b.status, kKvInvalid, uint32_t(f.s), uint32_t(page), uint32_t(no));
            } else {
              offs[h] = int64_t(page) * p.c.page_stride + int64_t(f.hk) * p.c.head_stride +
                        int64_t((half - no * page_halves) * 16) * p.c.token_stride;
              const int64_t i = int64_t(page) * p.c.Hkv + f.hk;
              scale_bytes[h][0] = p.c.ks[i];  // looked at after the copies are on their way
              scale_bytes[h][1] = p.c.vs[i];
            }
          }
        }
        __syncwarp();
      }
      const uint32_t dst = ring + uint32_t(stage * Smem::STAGE);
      uint32_t good = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t off = __shfl_sync(0xffffffffu, offs[h], f_at);
        const bool ok = off >= 0;
        good |= ok ? 1u << h : 0u;
        const uint8_t* ksrc = p.c.k + (ok ? off + lane_off : 0);
        const uint8_t* vsrc = p.c.v + (ok ? off + lane_off : 0);
        const int64_t step = ok ? rows_off : 0;
#pragma unroll
        for (int i = 0; i < 16 / RPC; ++i) {
          const int row = h * 16 + i * RPC + lane / UNITS;
          cp_async16(dst + k_at<D>(row, lane % UNITS), ksrc + i * step, ok);
          cp_async16(dst + CHUNK * D + v_at<D>(row, lane % UNITS), vsrc + i * step, ok);
        }
      }
      const uint32_t sc = __shfl_sync(0xffffffffu, scale_bytes[0][0] | scale_bytes[0][1] << 8 | scale_bytes[1][0] << 16 |
                                                       scale_bytes[1][1] << 24, f_at);
      if (lane == 0) sm.meta[warp][stage] = make_uint2(sc, good);
      ++f_at;
      fc += WARPS;
      settle();
    }
    cp_async_commit();
  };
  uint4 qraw[NR][KL * 2];  // row g of each product's queries, on their way while pages are looked up
  auto load_q = [&](const Segment& c) {
#pragma unroll
    for (int x = 0; x < NR; ++x) {
      const int last = int(int64_t(c.seq.q) * p.group) - 1;
      const int r = min(c.rt * TILE + 8 * x + g, last);
      const int i = r / p.group;
      const uint16_t* src = p.q + int64_t(c.seq.row0 + i) * p.q_ts + int64_t(c.hk * p.group + r - i * p.group) * p.q_hs;
#pragma unroll
      for (int j = 0; j < KL; ++j) {
        qraw[x][2 * j] = *reinterpret_cast<const uint4*>(src + j * 64 + t * 16);
        qraw[x][2 * j + 1] = *reinterpret_cast<const uint4*>(src + j * 64 + t * 16 + 8);
      }
    }
  };
  load_q(c);
  for (int i = 0; i < STAGES - 1; ++i) fetch(i);

  // ---------------------------------------------------------------- segment by segment
  int stage = 0;
  int64_t at = run0;  // the piece's first place in the list
  while (true) {
    const int r0 = c.rt * TILE;
    const int rows = min(TILE, int(int64_t(c.seq.q) * p.group - r0));
    const int start = c.seq.len - c.seq.q;
    auto limit = [&](int row) {  // keys that a row of the tile sees
      return p.causal ? max(0, min(c.seq.len, start + (r0 + min(row, rows - 1)) / p.group + 1)) : c.seq.len;
    };
    // queries: row g of each product; scales and limits of rows 2t and 2t + 1
    uint32_t qb[NR][KL * 4][2];
    float f_row[NR][2];
    int lim[NR][2];
#pragma unroll
    for (int x = 0; x < NR; ++x) {
      const uint4(&w)[KL * 2] = qraw[x];
      float amax = 0.0f;
#pragma unroll
      for (int j = 0; j < KL * 2; ++j) {
        const uint32_t u[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(u[k] << 16)), fabsf(__uint_as_float(u[k] & 0xFFFF0000u))));
      }
      amax = quad_max(amax);
      const int e = max(int(__float_as_uint(amax) >> 23) - 127, -126);
      const float down = pow2f(-e), fr = pow2f(e) * p.scale_log2;
#pragma unroll
      for (int j = 0; j < KL * 2; ++j) {
        const uint32_t u[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
        uint32_t h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          h[k] = pack_f16x2(__uint_as_float(u[k] << 16) * down, __uint_as_float(u[k] & 0xFFFF0000u) * down);
        // dims 4v .. 4v+3 of the lane's 16 are the k slots (2t, 2t+1, 2t+8, 2t+9) of step v
        qb[x][2 * j][0] = h[0];
        qb[x][2 * j][1] = h[1];
        qb[x][2 * j + 1][0] = h[2];
        qb[x][2 * j + 1][1] = h[3];
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        f_row[x][y] = __shfl_sync(0xffffffffu, fr, (2 * t + y) * 4);
        lim[x][y] = limit(8 * x + 2 * t + y);
      }
    }
    const int min_lim = limit(0);

    float o[NR][MTS][4];  // dims g * VB + i and g * VB + VB/2 + i of rows 2t, 2t + 1
#pragma unroll
    for (int x = 0; x < NR; ++x)
#pragma unroll
      for (int i = 0; i < MTS; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[x][i][j] = 0.0f;
    float m[NR][2], l[NR][2];
#pragma unroll
    for (int x = 0; x < NR; ++x) {
      m[x][0] = m[x][1] = -INFINITY;
      l[x][0] = l[x][1] = 0.0f;
    }
    int ve = -128;  // O is in units of 2^ve (-128: nothing yet); kOwn: of a row's own, sm.e

    for (int ch = c.cb + warp; ch < c.ce; ch += WARPS) {
      cp_async_wait<STAGES - 2>();
      __syncwarp();
      fetch(stage == 0 ? STAGES - 1 : stage - 1);  // over the chunk before this one
      const uint2 meta = sm.meta[warp][stage];
      const uint8_t* src = sm.ring[warp][stage];
      const int tok = ch * CHUNK;
      const bool edge = tok + CHUNK > min_lim || meta.y != 3u;
      float s[2][NR][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // two chains of products, one for each half of the dims
        float part[KL][NR][4];
#pragma unroll
        for (int j = 0; j < KL; ++j) {
#pragma unroll
          for (int x = 0; x < NR; ++x)
#pragma unroll
            for (int k = 0; k < 4; ++k) part[j][x][k] = 0.0f;
          const uint4 a = lds128(src + k_at<D>(h * 16 + g, j * 4 + t));
          const uint4 d = lds128(src + k_at<D>(h * 16 + 8 + g, j * 4 + t));
          const uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t a0 = e4m3x2_to_f16x2(u[k]), a2 = e4m3x2_to_f16x2_hi(u[k]);
            const uint32_t a1 = e4m3x2_to_f16x2(v[k]), a3 = e4m3x2_to_f16x2_hi(v[k]);
#pragma unroll
            for (int x = 0; x < NR; ++x) mma_f16(part[j][x], a0, a1, a2, a3, qb[x][j * 4 + k][0], qb[x][j * 4 + k][1]);
          }
        }
        const float kf = pow2f(int((meta.x >> (16 * h)) & 0xFFu) - 127);
#pragma unroll
        for (int x = 0; x < NR; ++x)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            s[h][x][k] = (KL == 2 ? part[0][x][k] + part[KL - 1][x][k] : part[0][x][k]) * (f_row[x][k & 1] * kf);
      }
      if (edge) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int x = 0; x < NR; ++x)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (!(meta.y >> h & 1u) || tok + h * 16 + g + (k >> 1) * 8 >= lim[x][k & 1]) s[h][x][k] = -INFINITY;
      }
      float mx[NR][2];
      bool raise = false;
#pragma unroll
      for (int x = 0; x < NR; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          mx[x][y] = column_max(fmaxf(fmaxf(s[0][x][y], s[0][x][2 + y]), fmaxf(s[1][x][y], s[1][x][2 + y])));
          raise |= mx[x][y] > m[x][y] + kSlack;
        }
      const int vb[2] = {int((meta.x >> 8) & 0xFFu), int(meta.x >> 24)};
      // of both halves (one that does not exist has the other's; 255 is above any reference)
      const int vtop = max(vb[0], vb[1]) - 127, vlow = min(vb[0], vb[1]) - 127;
      bool far = vtop > ve || vlow < ve - kNear;
      if (far && ve == -128) {
        ve = min(vtop + kRoom, 127);
        far = vtop > ve || vlow < ve - kNear;
      }
      if (__builtin_expect(far, 0)) {
        // a reference for each row: see the head of the file
        if (ve != kOwn) {
          if (g == 0) {
#pragma unroll
            for (int x = 0; x < NR; ++x)
#pragma unroll
              for (int y = 0; y < 2; ++y) sm.e[8 * x + 2 * t + y][warp] = ve;
          }
          __syncwarp();
          ve = kOwn;
        }
        const bool has[2] = {(meta.y & 1u) && vb[0] != 255, (meta.y & 2u) && vb[1] != 255};
#pragma unroll
        for (int x = 0; x < NR; ++x)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float mo = m[x][y], mn = fmaxf(mo, mx[x][y]);
            int32_t* at = &sm.e[8 * x + 2 * t + y][warp];
            const float2 r = own_reference(at, mo, mn, fmaxf(s[0][x][y], s[0][x][2 + y]), fmaxf(s[1][x][y], s[1][x][2 + y]),
                                           has[0] ? vb[0] : 255, has[1] ? vb[1] : 255);
            l[x][y] *= r.x;
            const float a = r.y;
            m[x][y] = mn;
#pragma unroll
            for (int i = 0; i < MTS; ++i) {
              o[x][i][y] *= a;
              o[x][i][2 + y] *= a;
            }
          }
      } else if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int x = 0; x < NR; ++x) {
          float a[2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float mn = mx[x][y] > m[x][y] + kSlack ? mx[x][y] : m[x][y];
            a[y] = mn == m[x][y] ? 1.0f : ex2_approx(m[x][y] - mn);
            m[x][y] = mn;
            l[x][y] *= a[y];
          }
#pragma unroll
          for (int i = 0; i < MTS; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) o[x][i][k] *= a[k & 1];
        }
      }
      uint32_t pb[2][NR][2];  // P^T: tokens (2t, 2t+1) and (2t+8, 2t+9) of the half, row g
      if (__builtin_expect(far, 0)) {
        // weight times scale from one exponent: of a small weight and a large scale each alone may leave fp32
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int x = 0; x < NR; ++x) {
            float w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int y = k & 1, d = vb[h] - 127 - sm.e[8 * x + 2 * t + y][warp];
              const float at = s[h][x][k] + (m[x][y] == -INFINITY ? kShift : kShift - m[x][y]);
              s[h][x][k] = ex2_approx(at);
              w[k] = vb[h] != 255 ? ex2_approx(at + float(d)) : s[h][x][k];  // 255: its codes count as NaN
            }
            l[x][0] += s[h][x][0] + s[h][x][2];
            l[x][1] += s[h][x][1] + s[h][x][3];
            pb[h][x][0] = transposed(pack_f16x2(w[0], w[1]));
            pb[h][x][1] = transposed(pack_f16x2(w[2], w[3]));
          }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float vf = pow2f(vb[h] - 127 - ve);
#pragma unroll
          for (int x = 0; x < NR; ++x) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float mm = m[x][k & 1];
              s[h][x][k] = ex2_approx(s[h][x][k] + (mm == -INFINITY ? kShift : kShift - mm));
            }
            l[x][0] += s[h][x][0] + s[h][x][2];
            l[x][1] += s[h][x][1] + s[h][x][3];
            pb[h][x][0] = transposed(pack_f16x2(s[h][x][0] * vf, s[h][x][1] * vf));
            pb[h][x][1] = transposed(pack_f16x2(s[h][x][2] * vf, s[h][x][3] * vf));
          }
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t vw[4][VB / 4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (VB == 16) {
            const uint4 w = lds128(src + CHUNK * D + v_at<D>(h * 16 + 2 * t + (j & 1) + (j >> 1) * 8, g));
            vw[j][0] = w.x;
            vw[j][1] = w.y;
            vw[j][VB / 4 - 2] = w.z;
            vw[j][VB / 4 - 1] = w.w;
          } else {
            const uint2 w = lds64(src + CHUNK * D + v_at<D>(h * 16 + 2 * t + (j & 1) + (j >> 1) * 8, g >> 1) + (g & 1) * 8);
            vw[j][0] = w.x;
            vw[j][1] = w.y;
          }
        }
        if (vb[h] == 255) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < VB / 4; ++k) vw[j][k] = 0x7F7F7F7Fu;
        }
        if (edge) {
          // slots past the sequence's end hold anything: zero.  A NaN value that some rows see and
          // others do not would reach the others as NaN * 0: it is taken out here and counted for
          // the rows that see it by a product of 0/1 matrices.
          uint32_t nans = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bool past = tok + h * 16 + 2 * t + (j & 1) + (j >> 1) * 8 >= c.seq.len;
#pragma unroll
            for (int k = 0; k < VB / 4; ++k) {
              if (past) vw[j][k] = 0;
              nans |= nan_bytes(vw[j][k]);
            }
          }
          if (__any_sync(0xffffffffu, nans != 0)) {
#pragma unroll
            for (int x = 0; x < NR; ++x) {
              const int li = limit(8 * x + g), tk = tok + h * 16 + 2 * t;
              const uint32_t b0 = (tk < li ? 0x3C00u : 0u) | (tk + 1 < li ? 0x3C000000u : 0u);
              const uint32_t b1 = (tk + 8 < li ? 0x3C00u : 0u) | (tk + 9 < li ? 0x3C000000u : 0u);
#pragma unroll
              for (int i = 0; i < MTS; ++i) {
                uint32_t a[2][2];  // [dims i or VB/2 + i][tokens 2t.. or 2t+8..]
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                  for (int y = 0; y < 2; ++y) {
                    const int by = q * (VB / 2) + i;
                    a[q][y] = ((nan_bytes(vw[2 * y][by / 4]) >> (8 * (by % 4))) & 0x80u ? 0x3C00u : 0u) |
                              ((nan_bytes(vw[2 * y + 1][by / 4]) >> (8 * (by % 4))) & 0x80u ? 0x3C000000u : 0u);
                  }
                float cnt[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                mma_f16(cnt, a[0][0], a[1][0], a[0][1], a[1][1], b0, b1);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  if (cnt[k] > 0.0f) o[x][i][k] = __uint_as_float(0x7FFFFFFFu);
              }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int k = 0; k < VB / 4; ++k) vw[j][k] &= ~((nan_bytes(vw[j][k]) >> 7) * 0xFFu);
          }
        }
#pragma unroll
        for (int i = 0; i < MTS; i += 2) {
          const uint32_t sel = (i & 2) ? 0x7362u : 0x5140u;
          const int lo = i / 4, hi = VB / 8 + i / 4;
          const uint32_t a0 = __byte_perm(vw[0][lo], vw[1][lo], sel), a1 = __byte_perm(vw[0][hi], vw[1][hi], sel);
          const uint32_t a2 = __byte_perm(vw[2][lo], vw[3][lo], sel), a3 = __byte_perm(vw[2][hi], vw[3][hi], sel);
          const uint32_t e0 = e4m3x2_to_f16x2(a0), e1 = e4m3x2_to_f16x2(a1), e2 = e4m3x2_to_f16x2(a2),
                         e3 = e4m3x2_to_f16x2(a3);
          const uint32_t h0 = e4m3x2_to_f16x2_hi(a0), h1 = e4m3x2_to_f16x2_hi(a1), h2 = e4m3x2_to_f16x2_hi(a2),
                         h3 = e4m3x2_to_f16x2_hi(a3);
#pragma unroll
          for (int x = 0; x < NR; ++x) {
            mma_f16(o[x][i], e0, e1, e2, e3, pb[h][x][0], pb[h][x][1]);
            mma_f16(o[x][i + 1], h0, h1, h2, h3, pb[h][x][0], pb[h][x][1]);
          }
        }
      }
      stage = stage + 1 == STAGES ? 0 : stage + 1;
    }

    // ---------------------------------------------------------------- the warps' results become one
#pragma unroll
    for (int x = 0; x < NR; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        l[x][y] = column_sum(l[x][y]);
        if (g == 0) {
          const int r = 8 * x + 2 * t + y;
          sm.ml[r][warp] = make_float2(m[x][y], l[x][y]);
          if (m[x][y] == -INFINITY) sm.e[r][warp] = -127;  // it saw nothing
          else if (ve != kOwn) sm.e[r][warp] = ve;
        }
      }
    const int spare = stage == 0 ? STAGES - 1 : stage - 1;  // the stage that this warp's next copy will fill
    {
      float4* buf = reinterpret_cast<float4*>(sm.ring[warp][spare]);
      // a row's dims g * VB .. g * VB + VB - 1 as 16-byte units
#pragma unroll
      for (int x = 0; x < NR; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int u = 0; u < VB / 4; ++u) {
            constexpr int HALF = VB / 8;  // units of dims i, then of dims VB/2 + i
            const int q = u / HALF * 2 + y, i = (u % HALF) * 4;
            buf[merge_at<D>(8 * x + 2 * t + y, g * (VB / 4) + u)] =
                make_float4(o[x][i][q], o[x][i + 1][q], o[x][i + 2][q], o[x][i + 3][q]);
          }
    }
    if (lane == 0) sm.spare[warp] = spare;
    __syncthreads();
    constexpr int EPT = TILE * D <= 4 * THREADS ? 4 : TILE * D <= 8 * THREADS ? 8 : 16;  // elements of one thread, whole 16-byte units
    static_assert(D % EPT == 0 && TILE * D <= EPT * THREADS, "a tile is more than the threads' share");
    const int row = tid / (D / EPT), d0 = tid % (D / EPT) * EPT;
    const bool mine_row = row < rows;
    float M1 = -INFINITY, L = 0.0f;
    float acc[EPT];
    if (mine_row) {
      int em = -127;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) M1 = fmaxf(M1, sm.ml[row][w].x);
      // as for a row's own reference: a warp of large values and no weight must not take the others' bits
#pragma unroll
      for (int w = 0; w < WARPS; ++w) em = max(em, sm.e[row][w] + int(ceilf(fmaxf(sm.ml[row][w].x - M1, -1000.0f))));
#pragma unroll
      for (int i = 0; i < EPT; ++i) acc[i] = 0.0f;
#pragma unroll 4
      for (int w = 0; w < WARPS; ++w) {
        // a warp that saw no key has m = -inf, l = 0 and o = 0 (l is NaN when its scores were)
        const float2 ml = sm.ml[row][w];
        const float a = ml.x == -INFINITY ? (ml.y == 0.0f ? 0.0f : ml.y) : ex2_approx(ml.x - M1);
        L = fmaf(a, ml.x == -INFINITY ? 1.0f : ml.y, L);
        const float av = ml.x == -INFINITY ? a : ex2_approx(ml.x - M1 + float(sm.e[row][w] - em));
        const float4* buf = reinterpret_cast<const float4*>(sm.ring[w][sm.spare[w]]);
#pragma unroll
        for (int u = 0; u < EPT / 4; ++u) {
          const float4 v = buf[merge_at<D>(row, d0 / 4 + u)];
          acc[4 * u] = fmaf(av, v.x, acc[4 * u]);
          acc[4 * u + 1] = fmaf(av, v.y, acc[4 * u + 1]);
          acc[4 * u + 2] = fmaf(av, v.z, acc[4 * u + 2]);
          acc[4 * u + 3] = fmaf(av, v.w, acc[4 * u + 3]);
        }
      }
      const float inv = L == 0.0f ? 0.0f : 1.0f / L, pe = pow2f(em);
#pragma unroll
      for (int i = 0; i < EPT; ++i) acc[i] = acc[i] * inv * pe;
    }

    bool done = true;
    if (c.cb != 0 || c.ce != c.nch) {
      const int64_t t0 = at - c.o + LEAD;  // the tile's first chunk in the list
      const int64_t c0 = tile_c0 >= 0 ? tile_c0 : quotient((t0 + 1) * n - 1, total);
      const int64_t c1 = tile_c0 >= 0 ? tile_c1 : quotient((t0 + c.nch) * n - 1, total);
      constexpr int SLOT = TILE * D + 2 * TILE;
      float* slot = p.partial + (2 * cta + (c.cb == 0 ? 1 : 0)) * SLOT;
      if (mine_row) {
#pragma unroll
        for (int u = 0; u < EPT / 4; ++u)
          st_global_cg_v4f(slot + row * D + d0 + 4 * u, acc[4 * u], acc[4 * u + 1], acc[4 * u + 2], acc[4 * u + 3]);
        if (d0 == 0) {
          __stcg(slot + TILE * D + row, M1);
          __stcg(slot + TILE * D + TILE + row, L);
        }
      }
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const uint32_t old = atomicAdd(p.counters + c0, 1u);
        sm.last = old == uint32_t(c1 - c0);
        if (sm.last) p.counters[c0] = 0;
      }
      __syncthreads();
      done = sm.last;
      if (done && mine_row) {
        __threadfence();
        M1 = -INFINITY;
        L = 0.0f;
#pragma unroll
        for (int i = 0; i < EPT; ++i) acc[i] = 0.0f;
        constexpr int BATCH = EPT < 16 ? 8 : 4;  // slots on their way at once
        for (int64_t x0 = c0; x0 <= c1; x0 += BATCH) {
          float mw[BATCH], lw[BATCH];
          float4 v[BATCH][EPT / 4];
#pragma unroll
          for (int k = 0; k < BATCH; ++k) {
            const int64_t x = min(x0 + k, c1);
            const float* from = p.partial + (2 * x + (x == c0)) * SLOT;
            mw[k] = __ldcg(from + TILE * D + row);
            lw[k] = __ldcg(from + TILE * D + TILE + row);
#pragma unroll
            for (int u = 0; u < EPT / 4; ++u) v[k][u] = ld_global_cg_v4f(from + row * D + d0 + 4 * u);
          }
          float top = M1;
#pragma unroll
          for (int k = 0; k < BATCH; ++k) top = fmaxf(top, mw[k]);
          // factors of a part go in two halves: that of a large mean of little weight may leave fp32 alone
          const float down = M1 == -INFINITY ? 1.0f : ex2_approx(0.5f * (M1 - top));
          M1 = top;
          L *= down * down;
#pragma unroll
          for (int i = 0; i < EPT; ++i) acc[i] = acc[i] * down * down;
#pragma unroll
          for (int k = 0; k < BATCH; ++k) {
            if (x0 + k > c1) break;
            const float half = mw[k] == -INFINITY ? 1.0f : ex2_approx(0.5f * (mw[k] - M1)), wgt = lw[k] * half;
            L = fmaf(wgt, half, L);
#pragma unroll
            for (int u = 0; u < EPT / 4; ++u) {
              acc[4 * u] = fmaf(wgt, half * v[k][u].x, acc[4 * u]);
              acc[4 * u + 1] = fmaf(wgt, half * v[k][u].y, acc[4 * u + 1]);
              acc[4 * u + 2] = fmaf(wgt, half * v[k][u].z, acc[4 * u + 2]);
              acc[4 * u + 3] = fmaf(wgt, half * v[k][u].w, acc[4 * u + 3]);
            }
          }
        }
        const float i2 = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
        for (int i = 0; i < EPT; ++i) acc[i] *= i2;
      }
    }
    if (done && mine_row) {
      const int r = r0 + row, i = r / p.group, tok = c.seq.row0 + i, h = c.hk * p.group + r - i * p.group;
      uint16_t* dst = p.out + (int64_t(tok) * p.H + h) * D + d0;
#pragma unroll
      for (int u = 0; u < EPT / 4; ++u)
        reinterpret_cast<uint2*>(dst)[u] =
            make_uint2(pack_bf16x2(acc[4 * u], acc[4 * u + 1]), pack_bf16x2(acc[4 * u + 2], acc[4 * u + 3]));
      if (d0 == 0 && p.lse)
        p.lse[int64_t(h) * b.n_tokens + tok] = L == 0.0f ? -INFINITY : (M1 - kShift + log2f(L)) * 0.69314718055994531f;
    }
    at += c.used;
    if (!seg_next<TILE>(p, c)) break;
    load_q(c);
    __syncthreads();  // the merge buffers are free again
  }
  cp_async_wait<0>();
  pdl_wait_previous();  // the call ends when the kernel for many rows has ended too
}

template <int D, int NR, int WARPS, int PER_SM>
tl_status launch_decode(void** args, int ctas, cudaStream_t st, bool early) {
  using Smem = DecodeSmem<D, NR, WARPS, PER_SM>;
  static_assert(sizeof(Smem) <= 232448 / PER_SM - (PER_SM - 1) * 1024, "shared memory above the limit");
  return launch(reinterpret_cast<const void*>(&kv_decode_kernel<D, NR, WARPS, PER_SM>), ctas * PER_SM, WARPS * 32, sizeof(Smem), st, args,
                early);
}

// ---------------------------------------------------------------- workspace: counters, then partial tiles
// The counters of both kernels come first, in a place that does not depend on the sizes: one workspace may serve
// calls of many.
size_t counters_bytes(int ctas) { return (size_t(ctas) * (MAX_PER_SM + 2) * 4 + 255) / 256 * 256; }
// (Four CTAs of an SM only with tiles of half MAX_TILE.)
size_t decode_partial_bytes(int ctas, int D) { return size_t(ctas) * (MAX_PER_SM / 2) * 2 * (MAX_TILE * D + 2 * MAX_TILE) * sizeof(float); }

}  // namespace
}  // namespace tl

extern "C" size_t tl_kv_attn_workspace_size(int n_tokens, int B, int H, int H_kv, int head_dim, int sm_count) {
  using namespace tl;
  if (n_tokens < 0 || B < 1 || H < 1 || H_kv < 1 || H % H_kv || (head_dim != 64 && head_dim != 128) || sm_count < 0)
    return 0;
  if (sm_count == 0) {
    DeviceInfo di{};
    if (device_info(&di) != TL_OK) return 0;
    sm_count = di.sm_count;
  }
  size_t bytes = counters_bytes(sm_count) + decode_partial_bytes(sm_count, head_dim);
  if (int64_t(n_tokens) * (H / H_kv) > few_rows(B)) bytes += prefill_partial_bytes(sm_count, head_dim);
  return bytes;
}

extern "C" tl_status tl_kv_attn(const tl_kv_attn_args* a, void* stream) {
  using namespace tl;
  if (!a) return fail(TL_ERR_INVALID, "tl_kv_attn: NULL args");
  if (a->n_tokens < 0 || a->B < 1 || a->B > (1 << 20) || a->max_pages < 1)
    return fail(TL_ERR_INVALID, "tl_kv_attn: n_tokens %d, B %d, max_pages %d", a->n_tokens, a->B, a->max_pages);
  if (tl_status s = check_kv_cache("tl_kv_attn", a->cache)) return s;
  const tl_kv_cache& c = a->cache;
  if (a->H < 1 || a->H > 65536 || a->H % c.H_kv)
    return fail(TL_ERR_INVALID, "tl_kv_attn: H=%d is not a multiple of H_kv=%d", a->H, c.H_kv);
  if (a->causal != 0 && a->causal != 1) return fail(TL_ERR_INVALID, "tl_kv_attn: causal %d", a->causal);
  if (a->max_q_len < 0) return fail(TL_ERR_INVALID, "tl_kv_attn: max_q_len %d", a->max_q_len);
  if (!(a->scale >= 0.0f) || std::isinf(a->scale))
    return fail(TL_ERR_INVALID, "tl_kv_attn: scale must be positive and finite (0 = 1/sqrt(head_dim))");
  if (!a->cu_seqlens || !a->seq_lens || !a->page_table || !a->signals)
    return fail(TL_ERR_INVALID, "tl_kv_attn: NULL pointer argument");
  if (a->n_tokens == 0) return TL_OK;
  if (!a->q || !a->out || !a->workspace) return fail(TL_ERR_INVALID, "tl_kv_attn: NULL pointer argument");
  if (!aligned16(a->q) || !aligned16(a->out) || !aligned16(a->workspace) || (reinterpret_cast<uintptr_t>(a->lse) & 3u))
    return fail(TL_ERR_INVALID, "tl_kv_attn: pointers must be 16-byte aligned (lse 4-byte)");
  for (int64_t s : {a->q_token_stride, a->q_head_stride})
    if (s < 0 || s % 8) return fail(TL_ERR_INVALID, "tl_kv_attn: strides must be multiples of 8 elements");
  if (int64_t(a->n_tokens) * (a->H / c.H_kv) > 0x7FFF0000ll)
    return fail(TL_ERR_UNSUPPORTED, "tl_kv_attn: too many query rows");
  DeviceInfo di{};
  if (tl_status s = device_info(&di)) return s;
  if (a->signals->device != di.device) return fail(TL_ERR_INVALID, "tl_kv_attn: signals belong to another device");
  const size_t need = tl_kv_attn_workspace_size(a->n_tokens, a->B, a->H, c.H_kv, c.head_dim, di.sm_count);
  if (a->workspace_bytes < need)
    return fail(TL_ERR_INVALID, "tl_kv_attn: workspace of %zu bytes, need %zu", a->workspace_bytes, need);

  DecodeParams p{};
  p.c = KvCacheDev{static_cast<uint8_t*>(c.k), static_cast<uint8_t*>(c.v), c.k_scale, c.v_scale, c.page_stride,
                   c.head_stride, c.token_stride, c.num_pages, c.page_size, c.H_kv};
  p.b = KvBatch{a->cu_seqlens, a->seq_lens, a->page_table, a->signals->status, a->B, a->n_tokens, a->max_pages};
  p.q = static_cast<const uint16_t*>(a->q);
  p.q_ts = a->q_token_stride;
  p.q_hs = a->q_head_stride;
  p.out = static_cast<uint16_t*>(a->out);
  p.lse = a->lse;
  p.counters = static_cast<uint32_t*>(a->workspace);
  p.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(a->workspace) + counters_bytes(di.sm_count));
  p.H = a->H;
  p.group = a->H / c.H_kv;
  p.causal = a->causal;
  p.scale_log2 = (a->scale > 0.0f ? a->scale : 1.0f / std::sqrt(float(c.head_dim))) * 1.4426950408889634f;
  // Most new tokens that a sequence can have, as far as the host knows
  const int most = a->max_q_len ? std::min(a->max_q_len, a->n_tokens) : std::max(1, a->n_tokens - a->B + 1);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool many = int64_t(most) * p.group > few_rows(a->B);
  p.max_rows = 0x7FFFFFFF;
  if (many) {
    // A sequence of many rows goes to the tensor-core kernel, one of few to this file's; where there is one
    // sequence only, the first takes it whatever it is.
    PrefillParams f{};
    f.c = p.c;
    f.b = p.b;
    f.q = p.q;
    f.q_ts = p.q_ts;
    f.q_hs = p.q_hs;
    f.out = p.out;
    f.lse = p.lse;
    f.counters = p.counters + MAX_PER_SM * di.sm_count;
    f.partial = p.partial + decode_partial_bytes(di.sm_count, c.head_dim) / sizeof(float);
    f.timeout_ns = 3 * kDefaultTimeoutNs;
    f.H = a->H;
    f.group = p.group;
    f.causal = a->causal;
    f.min_rows = a->B == 1 ? 0 : few_rows(a->B);
    f.scale_log2 = p.scale_log2;
    if (tl_status s = launch_kv_prefill(f, c.head_dim, di.sm_count, st)) return s;
    if (a->B == 1) return TL_OK;
    p.max_rows = few_rows(a->B);
  }
  // Tiles of 8 query rows where a sequence's rows of one kv head fit in one, of 16 otherwise
  const bool small = int64_t(most) * p.group <= 8;
  void* args[] = {&p};
  const int per = per_sm(int64_t(a->B) * c.H_kv, small, di.sm_count);
  auto go = [&](auto dim) {
    constexpr int D = decltype(dim)::value;
    if (!small) return per == 1 ? launch_decode<D, 2, 8, 1>(args, di.sm_count, st, many) : launch_decode<D, 2, 4, 2>(args, di.sm_count, st, many);
    if (per == 1) return launch_decode<D, 1, 12, 1>(args, di.sm_count, st, many);
    return per == 2 ? launch_decode<D, 1, 6, 2>(args, di.sm_count, st, many) : launch_decode<D, 1, 3, 4>(args, di.sm_count, st, many);
  };
  return c.head_dim == 128 ? go(std::integral_constant<int, 128>()) : go(std::integral_constant<int, 64>());
}
