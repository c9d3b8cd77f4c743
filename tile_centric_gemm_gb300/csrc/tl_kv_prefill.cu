// tl_kv_prefill.cu -- attention of many new tokens of a sequence (a prompt's chunk)
// over the 8-bit paged cache, on tcgen05.
//
//   s_j = scale <q, k_j>,  O = sum_j exp(s_j - lse) v_j,  causal within the chunk
//
// Bound by shared memory: a tile of 64 tokens takes 1800 cycles, of which its products
// read operands for 1024 (at 128 bytes a cycle) and the conversion writes for 256; the
// issuing warps stand at the tensor cores' queue for 1250, the softmax is busy for 1400.
// Two chunks of 2048 over 12289 (32 heads, 8 kv heads of 128) take 479 us, 1150 TFLOP/s.
// What moved it: short loops (the instruction cache), no register spills, scores ahead,
// queries and outputs of a unit in whole lines.  Scores of 128 keys at a time would read
// a quarter less, but leave no second buffer in tensor memory.
// A unit is one kv
// head and 256 of a sequence's query rows, rows being (token, head of the group), so
// that all heads of a group share every key/value tile; two 128-row tiles A and B
// take turns, one in the softmax while the tensor cores work for the other.
//   warps 0-5    convert: queries bf16 -> fp16 (each row by a power of two), then
//                each 64-token tile of codes -> fp16, keys and values, 16 tokens an
//                item, into shared memory in the 128-byte-swizzled layout that the
//                products read.  A warp's next item is on its way in registers.
//   warps 6, 7   issue the products, one warp to a query tile X: S_X = Q_X K^T and O_X += P_X V (M = 128), P from
//                tensor memory.  S has two buffers for each query tile and its scores
//                are issued two tiles ahead, PV_X(j) QK_X(j+2), so
//                that a softmax finds its next scores ready: with one buffer of 128
//                keys each round trip from scores to P and back was waited for
//                (590 us for two chunks of 2048 over 12289).
//   warps 8-11   softmax of tile A, warps 12-15 of tile B, a row to a thread.
// Everything is fp16 with powers of two taken out: codes are exact in fp16, also times
// the block scales relative to the largest of the segment's keys (values), as long as
// these lie within 2^15 (2^6) of each other.  Where they do not, codes stay as they are and the
// scales enter in the softmax (far_tile: two chunks of 2048 over 12289 take 905 us with it,
// 469 us without, in a graph).  P runs up to 2^15, with a grain of 2^-24.  A row's reference
// m is its first tile's maximum and is raised, and O rescaled, only when a tile's weights exp2(s - m + 7) add up to more than 2^15, so that
// most tiles are done without looking for their maximum (482 us -> 472 us).  Great scores
// are computed apart (far_tile).
//
// The work is the list of (unit, key/value tile), cut into equal runs, one to a CTA,
// as in the kernel for few rows: short lists fill the SMs by splitting units, long
// ones have no last wave.  Partial results are joined in CTA order by the CTA that
// arrives last.
//
// A NaN value that only some rows of a unit see is taken out of V, and the least such
// token of each dim is kept: rows see prefixes, so a row's result in that dim is NaN
// exactly if the row sees that token.
//
// TMEM (lane = query row of the tile): S_A columns 0-63 and 64-127, S_B 128-191 and
// 192-255 (P in the first half of each), O_A from 256, O_B from 384.
#include <algorithm>
#include <cmath>

#include "tl_common.cuh"
#include "tl_internal.h"
#include "tl_kv.cuh"
#include "tl_kv_prefill.h"

namespace tl {
namespace {

constexpr int THREADS = 512;
constexpr int CONV = 6;           // converting warps
constexpr int WARP_MMA = 6, WARP_SOFTMAX = 8;
constexpr int KV = 64;           // tokens of a tile
constexpr int GROUPS = KV / 16;  // of 16 tokens in a tile
constexpr int ROWS = 128;        // query rows of a tile
constexpr int UNIT = 2 * ROWS;
// Ring stages: keys of tile j + 2 are needed with values of tile j, so that many fewer of them.
constexpr int KST = 4, VST = 6;
// Tiles of a CTA's run, where units are split: shorter ones open and join more than they compute (8 units: 64 tokens over
// 500 25, 22, 22 us with 4, 8, 16; over 4000 89, 60, 54 us, before the join was made shorter; chunks that fill the CTAs anyway do not care).
constexpr int MIN_TILES = 8;
constexpr float kShift = 7.0f, kMost = 32768.0f;
// Relative to a scale up to 2^kNearK larger codes (the least is 2^-9) are exact in fp16 (2^-24).  Values count no more than
// P does: their scales lie so close that the grain of P, times the largest, stays below 2^-25 of a row's largest product.
constexpr int kNearK = 15, kNearV = 6;
constexpr int kFar = 1000;
constexpr float kGreat = 16777216.0f;  // from here on the rounding of a score is as much as the span of a softmax
constexpr uint32_t BOX = ROWS * 64 * 2;    // a query tile's rows of 64 fp16, one swizzle span wide
constexpr uint32_t KV_BOX = KV * 64 * 2;   // a key or value tile's

struct __align__(8) Bars {
  uint64_t q_full, q_empty;
  uint64_t k_full[KST], k_empty[KST], v_full[VST], v_empty[VST];
  uint64_t s_full[2][2], p_full[2][2], o_done[2][2], o_empty[2];  // by query tile, and by the tile number's parity
  uint64_t conv[2], soft[2];                                   // among the converting warps; among a tile's softmax warps
  uint32_t tmem_base, abort;
};

template <int D>
struct Layout {
  static constexpr uint32_t Q_TILE = BOX * (D / 64), TILE = KV_BOX * (D / 64);  // queries; keys or values
  static constexpr uint32_t Q = 0, K = Q + 2 * Q_TILE, V = K + KST * TILE, BARS = V + VST * TILE;
};

struct Side {
  Bars bars;
  int8_t q_exp[2][UNIT];   // rows' exponents, by segment parity
  int16_t kv_exp[4][2];    // exponents of the segment's keys and values; kFar in place of the keys': of each 16 tokens' own
  uint16_t far[8][GROUPS]; // these tokens' scale bytes (keys' and values'), by tile
  union {
    int32_t nan_at[4][128];  // least token whose value is NaN in the dim, among those not all rows see
    struct {                 // before the segments: sums of the work list
      int64_t warp_sum[16];
      uint32_t warp_units[16];
    };
  };
  int8_t warp_range[CONV][4];
  int64_t total, ctas, run0;  // tiles of all runs, runs, this run's first tile
  int32_t begin[4];           // sequence, kv head, row block, tile
  int32_t tiles[4];           // of the segments in work
  int32_t last[2];
};

template <int D>
constexpr uint32_t smem_bytes() {
  return Layout<D>::BARS + uint32_t(sizeof(Side));
}
static_assert(smem_bytes<128>() <= 232448, "shared memory above the per-CTA limit");

constexpr uint32_t idesc_f16_f32(uint32_t M, uint32_t N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// ---------------------------------------------------------------- the list of work
struct Seg {
  KvSeq seq;
  int s, hk, qb, nkv, t0, t1;  // tiles t0 .. t1-1 of the unit's nkv
  int left;                    // tiles of the run from t0 on
};
__device__ __forceinline__ int seq_rows(const PrefillParams& p, const KvSeq& q) {
  const int rows = q.q * p.group;
  return rows > p.min_rows ? rows : 0;
}
__device__ __forceinline__ int row_limit(const PrefillParams& p, const KvSeq& q, int row) {
  return p.causal ? max(0, min(q.len, q.len - q.q + row / p.group + 1)) : q.len;
}
__device__ __forceinline__ int unit_tiles(const PrefillParams& p, const KvSeq& q, int rows, int qb) {
  const int lim = row_limit(p, q, min(rows, (qb + 1) * UNIT) - 1);
  return max(1, (lim + KV - 1) / KV);
}
__device__ __forceinline__ int64_t seq_tiles(const PrefillParams& p, const KvSeq& q) {  // of one kv head
  const int rows = seq_rows(p, q), blocks = (rows + UNIT - 1) / UNIT;
  if (!p.causal) return rows ? int64_t(blocks) * unit_tiles(p, q, rows, 0) : 0;
  int64_t n = 0;
  for (int b = 0; b < blocks; ++b) n += unit_tiles(p, q, rows, b);
  return n;
}
__device__ __forceinline__ bool seg_next(const PrefillParams& p, Seg& g) {
  g.left -= g.t1 - g.t0;
  if (g.left <= 0) return false;
  const int rows = seq_rows(p, g.seq);
  if (++g.qb * UNIT >= rows) {
    g.qb = 0;
    if (++g.hk == p.c.Hkv) {
      g.hk = 0;
      do {
        if (++g.s >= p.b.B) return false;
        g.seq = kv_seq(p.b, p.c.ps, g.s);
      } while (seq_rows(p, g.seq) == 0);
    }
  }
  g.nkv = unit_tiles(p, g.seq, seq_rows(p, g.seq), g.qb);
  g.t0 = 0;
  g.t1 = min(g.nkv, g.left);
  return true;
}

// ---------------------------------------------------------------- products
// The issuing warp runs as one: control flow and operands are the same in all lanes, so that descriptors
// stay in uniform registers, and the lane that issues is chosen by the predicate of the instruction alone.
__device__ __forceinline__ void mma_smem(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void mma_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(leader)
      : "memory");
}
// Some warps wait for one another, like a named barrier but for a bounded time: a warp that has given up does not leave
// the others waiting.
__device__ __forceinline__ bool meet(uint64_t* bar, uint32_t parity, volatile uint32_t* abort, uint32_t* status,
                                     uint64_t timeout_ns, uint32_t tag) {
  __syncwarp();
  if (lane_id() == 0) mbar_arrive(bar);
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, status, timeout_ns, tag)) != 0;
}
// Descriptors count in 16 bytes and lie in one 18-bit address space, so a step is an addition to the first.
template <int D>
__device__ __forceinline__ void issue_qk(uint64_t q0, uint64_t k0, uint32_t d_tmem, uint32_t leader) {
#pragma unroll
  for (int kk = 0; kk < D / UMMA_K; ++kk) {
    const uint64_t at = uint64_t((kk & 3) * 2);
    mma_smem(d_tmem, q0 + at + (kk >> 2) * (BOX >> 4), k0 + at + (kk >> 2) * (KV_BOX >> 4), idesc_f16_f32(ROWS, KV, false),
             kk > 0 ? 1u : 0u, leader);
  }
}
template <int D>
__device__ __forceinline__ void issue_pv(uint32_t p_tmem, uint64_t v0, uint32_t d_tmem, bool accumulate, uint32_t leader) {
#pragma unroll
  for (int kk = 0; kk < KV / UMMA_K; ++kk)
    mma_tmem_a(d_tmem, p_tmem + uint32_t(kk * 8), v0 + uint64_t(kk * (2048 >> 4)), idesc_f16_f32(ROWS, D, true),
               (accumulate || kk > 0) ? 1u : 0u, leader);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Pairs of fp32 in one instruction: (x, y) = (a, b) * f + c, and (x, y) += (a, b).
__device__ __forceinline__ void fma2(float a, float b, float f, float c, float& x, float& y) {
  asm("{\n\t.reg .b64 p, q, r;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %4};\n\tmov.b64 r, {%5, %5};\n\t"
      "fma.rn.f32x2 p, p, q, r;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "=f"(x), "=f"(y)
      : "f"(a), "f"(b), "f"(f), "f"(c));
}
__device__ __forceinline__ void add2(float& x, float& y, float a, float b) {
  asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\t"
      "add.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ void tmem_st_16cols(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// 16 bytes to shared memory, zeros if !in.
__device__ __forceinline__ void cp_async16z(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void ld_shared_v4(uint32_t a, uint32_t& x, uint32_t& y, uint32_t& z, uint32_t& w) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x), "=r"(y), "=r"(z), "=r"(w) : "r"(a) : "memory");
}

// Codes are read once here: no place in L1, which is small beside the tiles
__device__ __forceinline__ uint4 ld_codes(const uint8_t* a) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(a));
  return r;
}

// Factor of a block with this scale byte relative to 2^top, as two halves.
__device__ __forceinline__ uint32_t block_factor(int byte, int top) {
  const float f = byte == 255 ? pow2f(128) : pow2f(max(byte - 127 - top, -127));
  return pack_f16x2(f, f);
}

// Sixteen codes times f into a swizzled tile: eight fp16 each at two places.
__device__ __forceinline__ void put16(uint32_t lo, uint32_t hi, uint4 w, uint32_t f) {
  const uint32_t c[4] = {w.x, w.y, w.z, w.w};
  uint32_t h[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[2 * i] = mul_f16x2(e4m3x2_to_f16x2(c[i]), f);
    h[2 * i + 1] = mul_f16x2(e4m3x2_to_f16x2_hi(c[i]), f);
  }
  st_shared_v4(lo, h[0], h[1], h[2], h[3]);
  st_shared_v4(hi, h[4], h[5], h[6], h[7]);
}

// In 16 tokens of a value tile that not all rows see: NaN out of the tile, and the least token with one kept
// for each dim.  (Slots past the sequence's end are zero, or NaN under a NaN scale: no row's limit is beyond them.)
template <int D>
__device__ __noinline__ void spare_nan(uint32_t tile, int row0, int tok0, int32_t* nan_at) {
  __syncwarp();
  for (int x = int(lane_id()); x < 16 * D / 2; x += 32) {
    const int r = row0 + x / (D / 2), d = x % (D / 2) * 2, c = d >> 3 & 7;
    const uint32_t at = tile + uint32_t((d >> 6) * KV_BOX + r * 128 + ((c ^ (r & 7)) << 4) + (d & 7) * 2);
    uint32_t w;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(at) : "memory");
    const bool lo = (w & 0x7FFFu) > 0x7C00u, hi = (w & 0x7FFF0000u) > 0x7C000000u;
    if (lo) atomicMin(nan_at + d, tok0 + r - row0);
    if (hi) atomicMin(nan_at + d + 1, tok0 + r - row0);
    if (lo | hi) {
      w &= (lo ? 0xFFFF0000u : 0xFFFFFFFFu) & (hi ? 0xFFFFu : 0xFFFFFFFFu);
      asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(w) : "memory");
    }
  }
  __syncwarp();
}

// Scores from the row's limit on become -infinity.
__device__ __forceinline__ void mask(uint32_t (&v)[32], int vis) {
  if (vis < 32) {
#pragma unroll
    for (int k = 0; k < 32; ++k)
      if (k >= vis) v[k] = __float_as_uint(-INFINITY);
  }
}
__device__ __forceinline__ float max32(const uint32_t (&v)[32]) {  // in four chains
  float q[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    q[c] = max3(__uint_as_float(v[8 * c]), __uint_as_float(v[8 * c + 1]), __uint_as_float(v[8 * c + 2]));
    q[c] = max3(q[c], __uint_as_float(v[8 * c + 3]), __uint_as_float(v[8 * c + 4]));
    q[c] = max3(q[c], __uint_as_float(v[8 * c + 5]), __uint_as_float(v[8 * c + 6]));
    q[c] = fmaxf(q[c], __uint_as_float(v[8 * c + 7]));
  }
  return max3(q[0], q[1], fmaxf(q[2], q[3]));
}

// 32 dims of a row of each lane to memory.  Four lanes exchange theirs first, so that a store covers 64 bytes of eight
// rows, not 16 of 32: the rows' lines are what a store costs.
__device__ __forceinline__ void put_rows(const float (&x)[32], uint16_t* row, bool row_ok, int dim) {
  const int lane = int(lane_id());
  uint32_t u[4][4];
#pragma unroll
  for (int k = 0; k < 16; ++k) u[k >> 2][k & 3] = pack_bf16x2(x[2 * k], x[2 * k + 1]);
#pragma unroll
  for (int d = 1; d < 4; d <<= 1) {
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      if (a & d) continue;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, lane & d ? u[a][k] : u[a + d][k], d);
        if (lane & d) u[a][k] = got;
        else u[a + d][k] = got;
      }
    }
  }
  const unsigned long long mine = row_ok ? reinterpret_cast<unsigned long long>(row + dim) : 0ull;
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const unsigned long long at = __shfl_sync(0xffffffffu, mine, (lane & 28) + a);
    if (at) st_global_v4(reinterpret_cast<uint16_t*>(at) + (lane & 3) * 8, u[a][0], u[a][1], u[a][2], u[a][3]);
  }
}

// scale * 2^e, finite and above 0, so that a masked score stays -infinity
__device__ __forceinline__ float score_factor(float scale, int e) {
  return fmaxf(scale * pow2f(max(min(e / 2, 127), -126)) * pow2f(max(min(e - e / 2, 127), -126)), 1e-38f);
}

// A tile's softmax where the scales of the segment's blocks are far apart: S holds products with the codes as they are.
// The scales of 16 tokens' keys enter their scores in fp32; those of their values multiply P relative to 2^e, e a
// row's own: at least what the largest product of weight and scale asks for among the keys that the row sees, so that
// P is at most 2^7 and neither a block that the row does not see nor one of little weight costs the others bits.
// Returns the row's reference, its sum, e, and what O so far has to be multiplied by.
// Without scale bytes (nullptr): f is the factor of all scores, e stays 0.  This is for great scores.  Elsewhere s f - m
// is one fused operation, whose product is not rounded as the maximum m was: of scores above 2^27 the largest would come
// out beyond what P holds, or vanish.
__device__ __noinline__ float4 far_tile(uint32_t s_addr, int vis, const volatile uint16_t* bytes, float scale, int qe, float m,
                                        float l, int e) {
  float most[GROUPS], f[GROUPS];
  int vb[GROUPS];
  float mn = m;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t v[32];
    tmem_ld_32cols(s_addr + uint32_t(h * 32), v);
    tmem_ld_wait();
    mask(v, vis - 32 * h);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint32_t b = bytes ? bytes[2 * h + q] : 127u | 127u << 8;
      const int kb = int(b & 0xFFu);
      f[2 * h + q] = score_factor(scale, qe + (kb == 255 ? 0 : kb - 127));  // 255: the codes are NaN
      vb[2 * h + q] = int(b >> 8);
      float x = -INFINITY;
#pragma unroll
      for (int k = 0; k < 16; ++k) x = fmaxf(x, __uint_as_float(v[16 * q + k]));
      most[2 * h + q] = __fmul_rn(x, f[2 * h + q]);
      mn = fmaxf(mn, most[2 * h + q]);
    }
  }
  int en = m == -INFINITY ? -1000 : e + int(ceilf(fmaxf(m - mn, -1000.0f)));
#pragma unroll
  for (int q = 0; q < GROUPS; ++q)
    if (vb[q] != 255 && most[q] > -INFINITY) en = max(en, vb[q] - 127 + int(ceilf(fmaxf(most[q] - mn, -1000.0f))));
  en = max(en, -127);
  const float alpha = m == -INFINITY ? 1.0f : ex2_approx(m - mn + float(e - en));
  if (m != mn) l *= ex2_approx(m - mn);
  const float add = mn == -INFINITY ? kShift : kShift - mn;
  float sum = 0.0f;
  // P of 32 tokens takes 16 columns: over scores that have been read
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t v[32], w[16];
    tmem_ld_32cols(s_addr + uint32_t(h * 32), v);
    tmem_ld_wait();
    mask(v, vis - 32 * h);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      // weight times scale from one exponent: of a small weight and a large scale each alone may leave fp32
      const float c = vb[2 * h + q] == 255 ? 0.0f : float(vb[2 * h + q] - 127 - en);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float a0 = __fadd_rn(__fmul_rn(__uint_as_float(v[16 * q + 2 * k]), f[2 * h + q]), add);
        const float a1 = __fadd_rn(__fmul_rn(__uint_as_float(v[16 * q + 2 * k + 1]), f[2 * h + q]), add);
        sum += ex2_approx(a0) + ex2_approx(a1);
        w[8 * q + k] = pack_f16x2(ex2_approx(a0 + c), ex2_approx(a1 + c));
      }
    }
    tmem_st_16cols(s_addr + uint32_t(h * 16), w);
  }
  return make_float4(mn, l + sum, float(en), alpha);
}

// A row's parts, those of CTAs c0 .. c1 in this order, become one: its output, and its reference and sum.
template <int D>
__device__ __noinline__ float2 join_parts(const float* rows_at, int c0, int c1, uint16_t* orow, bool row_ok) {
  constexpr int64_t SLOT = 2 * ROWS * (D + 3);
  const int n = c1 - c0;
  const float* first = rows_at + (2 * int64_t(c0) + 1) * SLOT;  // the first CTA's second slot, then the others' first ones
  auto slot = [&](int i) { return first + (i ? (2 * int64_t(i) - 1) * SLOT : 0); };
  float top = -INFINITY, sum = 0.0f;
  for (int i = 0; i <= n; ++i) top = fmaxf(top, __ldcg(slot(i) + D * ROWS));
  // the joined means' unit: by the largest product of weight and unit, as for a row's own reference
  float unit = -127.0f;
  for (int i = 0; i <= n; ++i) {
    const float* at = slot(i) + D * ROWS;
    const float m = __ldcg(at), l = __ldcg(at + ROWS), e = __ldcg(at + 2 * ROWS);
    sum += m == -INFINITY ? l : l * ex2_approx(m - top);
    unit = fmaxf(unit, e + ceilf(fmaxf(m - top, -1000.0f)));
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum, pe = pow2f(int(unit));
#pragma unroll 1
  for (int q = 0; q < D / 32; ++q) {
    float x[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) x[k] = 0.0f;
    const float* from = first;
#pragma unroll 1
    for (int i = 0; i <= n; ++i, from = slot(i)) {
      const float m = __ldcg(from + D * ROWS), l = __ldcg(from + (D + 1) * ROWS), e = __ldcg(from + (D + 2) * ROWS);
      float v[32];
#pragma unroll
      for (int k = 0; k < 32; ++k) v[k] = __ldcg(from + (q * 32 + k) * ROWS);
      const float w = m == -INFINITY ? l : l * ex2_approx(m - top + (e - unit));
#pragma unroll
      for (int k = 0; k < 32; ++k) x[k] = fmaf(w, v[k], x[k]);
    }
#pragma unroll
    for (int k = 0; k < 32; ++k) x[k] = x[k] * inv * pe;
    put_rows(x, orow, row_ok, q * 32);
  }
  return make_float2(top, sum);
}

template <int D>
__global__ void __launch_bounds__(THREADS, 1) kv_prefill_kernel(const __grid_constant__ PrefillParams p) {
  using L = Layout<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t smem = smem_u32(smem_raw);
  Side& sd = *reinterpret_cast<Side*>(smem_raw + L::BARS);
  Bars* bars = &sd.bars;
  // a reduction over the warp: the result is known to be the same in all lanes
  const int tid = threadIdx.x, lane = tid & 31, warp = int(__reduce_max_sync(0xffffffffu, uint32_t(tid) >> 5));
  volatile uint32_t* abort = &bars->abort;
  const KvBatch& b = p.b;
  const uint64_t tmo = p.timeout_ns;
  pdl_launch_dependents();
  if (smem & 1023u) {  // the swizzle counts on it
    if (tid == 0) record_error(b.status, 5u, 0xFFFF0001u, smem, 0u);
    return;
  }

  // ---------------------------------------------------------------- this CTA's run of tiles
  const int per = (b.B + THREADS - 1) / THREADS;
  const int first = min(b.B, tid * per), end = min(b.B, first + per);
  int64_t mine = 0;
  uint32_t units = 0;
  for (int s = first; s < end; ++s) {
    const KvSeq q = kv_seq(b, p.c.ps, s);
    mine += p.c.Hkv * seq_tiles(p, q);
    units += uint32_t(p.c.Hkv) * uint32_t((seq_rows(p, q) + UNIT - 1) / UNIT);
  }
  units = __reduce_add_sync(0xffffffffu, units);
  if (lane == 0) sd.warp_units[warp] = units;
  int64_t before = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, before, d);
    if (lane >= d) before += x;
  }
  if (lane == 31) sd.warp_sum[warp] = before;
  if (tid == 0) {
    mbar_init(&bars->q_full, CONV);
    mbar_init(&bars->q_empty, 2);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bars->s_full[x][0], 1);
      mbar_init(&bars->s_full[x][1], 1);
      mbar_init(&bars->p_full[x][0], 4);
      mbar_init(&bars->p_full[x][1], 4);
      mbar_init(&bars->conv[x], CONV);
      mbar_init(&bars->soft[x], 4);
      mbar_init(&bars->o_done[x][0], 1);
      mbar_init(&bars->o_done[x][1], 1);
      mbar_init(&bars->o_empty[x], 4);
    }
    for (int i = 0; i < KST; ++i) {
      mbar_init(&bars->k_full[i], GROUPS);
      mbar_init(&bars->k_empty[i], 2);
    }
    for (int i = 0; i < VST; ++i) {
      mbar_init(&bars->v_full[i], GROUPS);
      mbar_init(&bars->v_empty[i], 2);
    }
    bars->abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  int64_t total = 0, all_units = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w == warp) before += total;
    total += sd.warp_sum[w];
    all_units += sd.warp_units[w];
  }
  before -= mine;
  // a CTA for each unit as far as they go, and where units are split MIN_TILES to a CTA at least
  const int64_t n = min(int64_t(gridDim.x), max(all_units, total / MIN_TILES));
  const int64_t cta = blockIdx.x;
  const int64_t run0 = cta < n ? cta * total / n : 0, run1 = cta < n ? (cta + 1) * total / n : 0;
  if (run0 >= run1) return;
  if (mine > 0 && before <= run0 && run0 < before + mine) {
    int64_t at = before;
    for (int s = first; s < end; ++s) {
      const KvSeq q = kv_seq(b, p.c.ps, s);
      const int64_t one = seq_tiles(p, q), size = one * p.c.Hkv;
      if (run0 < at + size) {
        int64_t off = run0 - at;
        const int hk = int(off / one);
        off -= hk * one;
        int qb = 0;
        const int rows = seq_rows(p, q);
        for (int t; (t = unit_tiles(p, q, rows, qb)) <= off; ++qb) off -= t;
        sd.begin[0] = s;
        sd.begin[1] = hk;
        sd.begin[2] = qb;
        sd.begin[3] = int(off);
        break;
      }
      at += size;
    }
  }
  if (tid == 0) {
    sd.total = total;
    sd.ctas = n;
    sd.run0 = run0;
  }
  if (warp == WARP_MMA) {
    tmem_alloc(&bars->tmem_base, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = bars->tmem_base;
  Seg g;
  g.s = sd.begin[0];
  g.hk = sd.begin[1];
  g.qb = sd.begin[2];
  g.t0 = sd.begin[3];
  g.left = int(run1 - run0);
  g.seq = kv_seq(b, p.c.ps, g.s);
  g.nkv = unit_tiles(p, g.seq, seq_rows(p, g.seq), g.qb);
  g.t1 = min(g.nkv, g.t0 + g.left);

  if (warp < CONV) {
    // ---------------------------------------------------------------- conversion, item by item
    // Item n of a segment: keys and values of 16 tokens, group n % 4 of its tile n / 4.  Warp w takes items w,
    // w + 6, ...; the next one's codes are on their way in registers.  (The loop is kept short: with the softmax and
    // the issuing loop it has to live in the instruction cache; two or three items ahead measured slower.)
    constexpr int PASS = D / 64;     // 16-code units of one thread and token
    const int r8 = lane >> 2, u4 = lane & 3;
    // where a lane's 16 dims of token r8 go: 16-byte units 2 u4 and 2 u4 + 1 of the row, swizzled by the row
    const uint32_t lane_lo = uint32_t(r8 * 128 + (((2 * u4) ^ r8) << 4)), lane_hi = uint32_t(r8 * 128 + (((2 * u4 + 1) ^ r8) << 4));
    // from a lane's query row to its next
    const int step_tk = CONV * 256 / D / p.group, step_hd = CONV * 256 / D - step_tk * p.group;
    const int64_t q_step = step_tk * p.q_ts + step_hd * p.q_hs, q_wrap = p.q_ts - p.group * p.q_hs;
    int before_seg = 0;              // tiles of earlier segments
    bool ok = true;
    for (int i = 0; ok; ++i) {
      const int rows = seq_rows(p, g.seq);
      const int len = g.seq.len;
      const int min_lim = row_limit(p, g.seq, g.qb * UNIT);
      const int32_t* table = b.table + int64_t(g.s) * b.max_pages;
      // the largest scales of the segment's pages
      const int tok_end = min(len, g.t1 * KV);
      int km = -127, vm = -127, kl = 127, vl = 127;
      for (int pg = g.t0 * KV / p.c.ps + tid; pg * int64_t(p.c.ps) < tok_end; pg += CONV * 32) {
        const int page = __ldg(table + pg);
        if (page < 0 || page >= p.c.num_pages) {
          record_error(b.status, kKvInvalid, uint32_t(g.s), uint32_t(page), uint32_t(pg));
          continue;
        }
        const int kb = p.c.ks[int64_t(page) * p.c.Hkv + g.hk], vb = p.c.vs[int64_t(page) * p.c.Hkv + g.hk];
        if (kb != 255) {
          km = max(km, kb - 127);
          kl = min(kl, kb - 127);
        }
        if (vb != 255) {
          vm = max(vm, vb - 127);
          vl = min(vl, vb - 127);
        }
      }
      km = __reduce_max_sync(0xffffffffu, km);
      vm = __reduce_max_sync(0xffffffffu, vm);
      kl = __reduce_min_sync(0xffffffffu, kl);
      vl = __reduce_min_sync(0xffffffffu, vl);
      if (lane == 0) {
        sd.warp_range[warp][0] = int8_t(km);
        sd.warp_range[warp][1] = int8_t(vm);
        sd.warp_range[warp][2] = int8_t(kl);
        sd.warp_range[warp][3] = int8_t(vl);
      }
      ok = meet(&bars->conv[0], i & 1, abort, b.status, tmo, 14);
      if (!ok) break;
#pragma unroll
      for (int w = 0; w < CONV; ++w) {
        km = max(km, int(sd.warp_range[w][0]));
        vm = max(vm, int(sd.warp_range[w][1]));
        kl = min(kl, int(sd.warp_range[w][2]));
        vl = min(vl, int(sd.warp_range[w][3]));
      }
      if (km - kl > kNearK || vm - vl > kNearV) km = kFar;
      if (tid == 0) {
        sd.tiles[i & 3] = g.left > g.t1 - g.t0 ? g.t1 - g.t0 : g.t0 - g.t1;  // the run's last one: negative
        sd.kv_exp[i & 3][0] = int16_t(km);
        sd.kv_exp[i & 3][1] = int16_t(vm);
      }
      if (tid < D) sd.nan_at[i & 3][tid] = 0x7FFFFFFF;
      ok = meet(&bars->conv[1], i & 1, abort, b.status, tmo, 15);
      if (!ok) break;

      const int items = (g.t1 - g.t0) * GROUPS;
      const int64_t lane_off = int64_t(g.hk) * p.c.head_stride + int64_t(r8) * p.c.token_stride + u4 * 16;
      const int64_t eight = 8 * p.c.token_stride;
      uint4 ck[2 * PASS], cv[2 * PASS];  // tokens r8 and r8 + 8 of the item
      int sk = 0, sv = 0, page = -1;     // its scale bytes; the page of the item to be loaded next
      auto group = [&](int n) { return g.t0 * GROUPS + n; };                               // of 16 tokens, in the sequence
      // gr / (page_size / 16)
      auto page_of = [&](int gr) { return p.page_magic ? int(__umulhi(uint32_t(gr), p.page_magic)) : gr; };
      auto look_up = [&](int n) {
        const int gr = group(n);
        int pg = -1;
        if (n < items && gr * 16 < len) pg = __ldg(table + page_of(gr));
        return pg < p.c.num_pages ? pg : -1;
      };
      auto load = [&](const uint8_t* pool, uint4(&c)[2 * PASS], int n) {
        const int gr = group(n), slot = gr - page_of(gr) * (p.c.ps >> 4);
        const uint8_t* at = pool + int64_t(page) * p.c.page_stride + int64_t(slot) * 2 * eight + lane_off;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const bool in = page >= 0 && gr * 16 + 8 * y + r8 < len;
#pragma unroll
          for (int u = 0; u < PASS; ++u) {
            c[y * PASS + u] = make_uint4(0, 0, 0, 0);
            if (in) c[y * PASS + u] = ld_codes(at + y * eight + u * 64);
          }
        }
      };
      auto load_scales = [&]() {
        const int64_t at = int64_t(max(page, 0)) * p.c.Hkv + g.hk;
        sk = p.c.ks[at];
        sv = p.c.vs[at];
        if (page < 0) sk = sv = 0;
      };
      page = look_up(warp);

      load(p.c.k, ck, warp);
      load(p.c.v, cv, warp);
      load_scales();
      page = look_up(warp + CONV);
      // Queries: a row to D/8 lanes, copied to its place in bf16, all rows at once, and brought to fp16 there by the lanes
      // that copied it.  (Through registers, row after row, this took 25000 cycles a segment.)
      constexpr int LPR = D / 8, RPW = 32 / LPR, STRIDE = CONV * RPW;  // lanes of a row; rows of a warp, of all
      const int c8 = lane % LPR, r0 = warp * RPW + lane / LPR;
      auto place = [&](int r) {
        return smem + L::Q + uint32_t((r >> 7) * L::Q_TILE + (c8 >> 3) * BOX + (r & 127) * 128 + (((c8 & 7) ^ (r & 7)) << 4));
      };
      const int tk0 = (g.qb * UNIT + r0) / p.group;
      int hd = g.qb * UNIT + r0 - tk0 * p.group;
      const uint16_t* from = p.q + int64_t(g.seq.row0 + tk0) * p.q_ts + int64_t(g.hk * p.group + hd) * p.q_hs + c8 * 8;
      ok = mbar_wait(&bars->q_empty, uint32_t(i & 1) ^ 1u, abort, b.status, tmo, 11);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
#pragma unroll 2
      for (int r = r0; r < UNIT; r += STRIDE) {
        const bool in = g.qb * UNIT + r < rows;
        cp_async16z(place(r), in ? from : p.q, in);
        hd += step_hd;
        from += q_step;
        if (hd >= p.group) {
          hd -= p.group;
          from += q_wrap;
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 1
      for (int r1 = r0; r1 < UNIT; r1 += 4 * STRIDE) {  // four rows side by side: each is a chain of shuffles
        uint32_t u[4][4];
        float amax[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          ld_shared_v4(place(min(r1 + a * STRIDE, UNIT - 1)), u[a][0], u[a][1], u[a][2], u[a][3]);
          amax[a] = 0.0f;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            amax[a] = fmaxf(amax[a], fmaxf(fabsf(__uint_as_float(u[a][k] << 16)), fabsf(__uint_as_float(u[a][k] & 0xFFFF0000u))));
        }
#pragma unroll
        for (int d = LPR / 2; d > 0; d >>= 1) {
#pragma unroll
          for (int a = 0; a < 4; ++a) amax[a] = fmaxf(amax[a], __shfl_xor_sync(0xffffffffu, amax[a], d));
        }
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          const int r = r1 + a * STRIDE;
          const int e = min(max(int(__float_as_uint(amax[a]) >> 23) - 127, -126), 127);
          const float down = pow2f(-e);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            u[a][k] = pack_f16x2(__uint_as_float(u[a][k] << 16) * down, __uint_as_float(u[a][k] & 0xFFFF0000u) * down);
          if (r < UNIT) {
            st_shared_v4(place(r), u[a][0], u[a][1], u[a][2], u[a][3]);
            if (c8 == 0) sd.q_exp[i & 1][r] = int8_t(e);
          }
        }
      }
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->q_full);

      for (int n = warp; n < items; n += CONV) {
        const int count = before_seg + n / GROUPS, kst = count % KST, vst = count % VST;
        const uint32_t fk = block_factor(sk, km == kFar ? sk - 127 : km), fv = block_factor(sv, km == kFar ? sv - 127 : vm);
        const uint16_t bytes = uint16_t(sk | sv << 8);
        ok = mbar_wait(bars->k_empty + kst, uint32_t(count / KST & 1) ^ 1u, abort, b.status, tmo, 12) &&
             mbar_wait(bars->v_empty + vst, uint32_t(count / VST & 1) ^ 1u, abort, b.status, tmo, 13);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        const uint32_t ktile = smem + L::K + uint32_t(kst) * L::TILE, vtile = smem + L::V + uint32_t(vst) * L::TILE;
        const int row0 = n % GROUPS * 16;
        const uint32_t klo = ktile + uint32_t(row0 * 128) + lane_lo, khi = ktile + uint32_t(row0 * 128) + lane_hi;
        const uint32_t vlo = vtile + uint32_t(row0 * 128) + lane_lo, vhi = vtile + uint32_t(row0 * 128) + lane_hi;
#pragma unroll
        for (int x = 0; x < 2 * PASS; ++x) put16(klo + x / PASS * 1024 + x % PASS * KV_BOX, khi + x / PASS * 1024 + x % PASS * KV_BOX, ck[x], fk);
        load(p.c.k, ck, n + CONV);
#pragma unroll
        for (int x = 0; x < 2 * PASS; ++x) put16(vlo + x / PASS * 1024 + x % PASS * KV_BOX, vhi + x / PASS * 1024 + x % PASS * KV_BOX, cv[x], fv);
        load(p.c.v, cv, n + CONV);
        load_scales();
        page = look_up(n + 2 * CONV);
        if (group(n) * 16 + 16 > min_lim) spare_nan<D>(vtile, row0, group(n) * 16, sd.nan_at[i & 3]);
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
          // (a softmax has read these when the scores two tiles on are issued, and the ring of keys is four tiles long)
          if (km == kFar) sd.far[count & 7][n % GROUPS] = bytes;
          mbar_arrive(bars->k_full + kst);
          mbar_arrive(bars->v_full + vst);
        }
      }
      before_seg += g.t1 - g.t0;
      if (!ok || !seg_next(p, g)) break;
    }
  } else if (warp < WARP_SOFTMAX) {
    // ---------------------------------------------------------------- the issuing warps, one to a query tile
    {
      const int X = warp - WARP_MMA;
      const uint32_t leader = lane == 0, tmem = __reduce_max_sync(0xffffffffu, tmem_base);
      auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t tag) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, b.status, tmo, tag)) != 0;
      };
      const uint64_t q0 = sdesc_sw128(smem + L::Q + X * L::Q_TILE, 16, 1024), k0 = sdesc_sw128(smem + L::K, 16, 1024);
      const uint64_t v0 = sdesc_sw128(smem + L::V, KV_BOX, 1024);
      constexpr uint64_t TSTEP = L::TILE >> 4;
      const uint32_t s_tmem = tmem + X * 128, o_tmem = tmem + 256 + X * 128;
      int ks = 0, vs = 0;
      uint32_t kph = 0, vph = 0;
      uint32_t scount = 0, pcount = 0;  // tiles whose S, whose O += P V has been issued
      bool ok = true;
      auto scores = [&](bool last) {
        issue_qk<D>(q0, k0 + ks * TSTEP, s_tmem + (scount & 1) * 64, leader);
        commit(&bars->s_full[X][scount & 1], leader);
        commit(&bars->k_empty[ks], leader);
        if (last) commit(&bars->q_empty, leader);
        ++scount;
        if (++ks == KST) {
          ks = 0;
          kph ^= 1u;
        }
      };
      for (int i = 0; ok; ++i) {
        ok = wait(&bars->q_full, uint32_t(i & 1), 21);
        if (!ok) break;
        const int said = int(__reduce_max_sync(0xffffffffu, uint32_t(*reinterpret_cast<volatile int32_t*>(&sd.tiles[i & 3]))));
        const int tiles = said < 0 ? -said : said;
        for (int j = 0; j < min(tiles, 2) && ok; ++j) {  // two tiles' scores ahead
          if (!(ok = wait(&bars->k_full[ks], kph, 22))) break;
          tc_fence_after();
          scores(j + 1 == tiles);
        }
        for (int j = 0; j < tiles && ok; ++j) {
          ok = wait(&bars->v_full[vs], vph, 23) && wait(&bars->p_full[X][pcount & 1], (pcount >> 1) & 1u, 24);
          if (ok && j == 0) ok = wait(&bars->o_empty[X], uint32_t(i & 1) ^ 1u, 25);
          if (!ok) break;
          tc_fence_after();
          issue_pv<D>(s_tmem + (pcount & 1) * 64, v0 + vs * TSTEP, o_tmem, j > 0, leader);
          commit(&bars->o_done[X][pcount & 1], leader);
          commit(&bars->v_empty[vs], leader);
          ++pcount;
          if (++vs == VST) {
            vs = 0;
            vph ^= 1u;
          }
          if (j + 2 < tiles) {
            if (!(ok = wait(&bars->k_full[ks], kph, 26))) break;
            tc_fence_after();
            scores(j + 3 == tiles);  // where P of this tile was: products run in the order they are issued in
          }
        }
        if (!ok || said < 0) break;
      }
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- softmax, a row to a thread
    const int X = (warp - WARP_SOFTMAX) >> 2;
    const int row = (warp & 3) * 32 + lane;  // row of the tile = TMEM lane
    const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;
    const uint32_t s_base = tmem_base + lane_base + uint32_t(X * 128);
    const uint32_t o_addr = tmem_base + lane_base + uint32_t(256 + X * 128);
    uint32_t sc = 0, meets = 0;  // tiles so far; times that the tile's four warps have met
    bool ok = true;
    int done = 0;  // tiles of the run before this segment
    for (int i = 0;; ++i) {
      const int r = g.qb * UNIT + X * ROWS + row;
      const int rows = seq_rows(p, g.seq);
      const int lim = row_limit(p, g.seq, min(r, rows - 1));
      float m = -INFINITY, l = 0.0f, f = 0.0f;
      int e = kFar;  // O is in units of 2^e where scales are far apart
      for (int j = g.t0; j < g.t1; ++j, ++sc) {
        ok = mbar_wait(&bars->s_full[X][sc & 1], (sc >> 1) & 1u, abort, b.status, tmo, 31);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (j == g.t0) {
          const int qe = int(sd.q_exp[i & 1][X * ROWS + row]), ke = sd.kv_exp[i & 3][0];
          if (ke == kFar) e = -127;
          else f = score_factor(p.scale_log2, qe + ke);
        }
        const uint32_t s_addr = s_base + (sc & 1) * 64;
        const int vis = lim - j * KV;
        // P first with the maximum as it is; the sum tells whether that was enough (each weight is at most the sum, and up to
        // 2^15 is fine).  Only if it was not is the tile's maximum taken, for the rows concerned, and P once more: on a
        // segment's first tile, and seldom after it.
        uint32_t va[32], w[32];
        float sum = 0.0f, alpha = 1.0f;
        bool bad = false, again = false, resc = false;
#pragma unroll 1
        while (e == kFar) {
          uint32_t vb[32];
          tmem_ld_32cols(s_addr, va);
          tmem_ld_32cols(s_addr + 32u, vb);
          tmem_ld_wait();
          mask(va, vis);
          mask(vb, vis - 32);
          if (again) {
            const float mnew = __fmul_rn(fmaxf(max32(va), max32(vb)), f);
            resc = bad && mnew > m;
            if (resc) {
              alpha = ex2_approx(m - mnew);
              m = mnew;
              l *= alpha;
            }
          }
          const float add = m == -INFINITY ? kShift : kShift - m;
          float sq[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          // P as fp16 pairs over the first 32 columns of S
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const uint32_t* s = k < 16 ? &va[2 * k] : &vb[2 * k - 32];
            float p0, p1;
            fma2(__uint_as_float(s[0]), __uint_as_float(s[1]), f, add, p0, p1);
            p0 = ex2_approx(p0);
            p1 = ex2_approx(p1);
            add2(sq[2 * (k & 1)], sq[2 * (k & 1) + 1], p0, p1);
            w[k] = pack_f16x2(p0, p1);
          }
          sum = (sq[0] + sq[1]) + (sq[2] + sq[3]);
          if (again) break;
          bad = !(sum <= kMost) || !(fabsf(m) < kGreat);  // (m = -infinity: none yet)
          again = __any_sync(0xffffffffu, bad) != 0;
          if (!again) break;
        }
        const bool far = e != kFar;
        if (far || (again && __any_sync(0xffffffffu, fabsf(m) >= kGreat && m != -INFINITY))) {
          const float4 r = far ? far_tile(s_addr, vis, sd.far[sc & 7], p.scale_log2, sd.q_exp[i & 1][X * ROWS + row], m, l, e)
                               : far_tile(s_addr, vis, nullptr, f, 0, m, l, 0);
          m = r.x;
          l = r.y;
          sum = 0.0f;
          if (far) e = int(r.z);
          alpha *= r.w;
          resc = alpha != 1.0f;
        } else {
          tmem_st_32cols(s_addr, w);
        }
        if (j > g.t0 && __any_sync(0xffffffffu, resc)) {
          // O holds everything up to the tile before this one once that tile's product is done
          ok = mbar_wait(&bars->o_done[X][(sc - 1) & 1], ((sc - 1) >> 1) & 1u, abort, b.status, tmo, 33);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int q = 0; q < D / 32; ++q) {
            tmem_ld_32cols(o_addr + uint32_t(q * 32), va);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 32; ++k) va[k] = __float_as_uint(__uint_as_float(va[k]) * alpha);
            tmem_st_32cols(o_addr + uint32_t(q * 32), va);
          }
        }
        l += sum;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_full[X][sc & 1]);
      }
      if (!ok) break;
      ok = mbar_wait(&bars->o_done[X][(sc - 1) & 1], ((sc - 1) >> 1) & 1u, abort, b.status, tmo, 32);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      const int unit = e == kFar ? sd.kv_exp[i & 3][1] : e;  // O is in units of 2^unit
      int least_nan = sd.nan_at[i & 3][lane];
#pragma unroll
      for (int k = 1; k < D / 32; ++k) least_nan = min(least_nan, sd.nan_at[i & 3][lane + 32 * k]);
      least_nan = __reduce_min_sync(0xffffffffu, least_nan);
      const bool row_ok = r < rows;
      const bool whole = g.t0 == 0 && g.t1 == g.nkv;
      const float pe = whole ? pow2f(unit) : 1.0f;
      const int tk = r / p.group, head = g.hk * p.group + r - tk * p.group;
      uint16_t* orow = p.out + (int64_t(g.seq.row0 + tk) * p.H + head) * D;
      // a segment's partial result: for each tile D means, maximum, sum and the means' unit, row next to row
      constexpr int64_t SLOT = 2 * ROWS * (D + 3);
      float* mine_row = p.partial + (2 * int64_t(blockIdx.x) + (g.t0 == 0 ? 1 : 0)) * SLOT + X * (D + 3) * ROWS + row;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tmem_ld_32cols(o_addr + uint32_t(c * 32), o);
        tmem_ld_wait();
        float x[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) x[k] = __uint_as_float(o[k]) * inv * pe;
        if (least_nan < lim) {
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (sd.nan_at[i & 3][c * 32 + k] < lim) x[k] = __uint_as_float(0x7FFFFFFFu);
        }
        if (whole) {
          put_rows(x, orow, row_ok, c * 32);
        } else if (row_ok) {
#pragma unroll
          for (int k = 0; k < 32; ++k) __stcg(mine_row + (c * 32 + k) * ROWS, x[k]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->o_empty[X]);
      if (whole) {
        if (row_ok && p.lse)
          p.lse[int64_t(head) * b.n_tokens + g.seq.row0 + tk] =
              l == 0.0f ? -INFINITY : (m - kShift + log2f(l)) * 0.69314718055994531f;
      } else {
        if (row_ok) {
          __stcg(mine_row + D * ROWS, m);
          __stcg(mine_row + (D + 1) * ROWS, l);
          __stcg(mine_row + (D + 2) * ROWS, float(unit));
        }
        const int64_t t0 = sd.run0 + done - g.t0;
        const int64_t c0 = ((t0 + 1) * sd.ctas - 1) / sd.total, c1 = ((t0 + g.nkv) * sd.ctas - 1) / sd.total;
        __threadfence();
        ok = meet(&bars->soft[X], meets++ & 1, abort, b.status, tmo, 34);
        if (!ok) break;
        if ((tid & 127) == 0) {
          uint32_t* counter = p.counters + 2 * c0 + X;
          sd.last[X] = atomicAdd(counter, 1u) == uint32_t(c1 - c0);
          if (sd.last[X]) *counter = 0;
        }
        ok = meet(&bars->soft[X], meets++ & 1, abort, b.status, tmo, 35);
        if (!ok) break;
        if (sd.last[X]) {
          __threadfence();
          const float2 all = join_parts<D>(p.partial + X * (D + 3) * ROWS + row, int(c0), int(c1), orow, row_ok);
          if (p.lse && row_ok)
            p.lse[int64_t(head) * b.n_tokens + g.seq.row0 + tk] =
                all.y == 0.0f ? -INFINITY : (all.x - kShift + log2f(all.y)) * 0.69314718055994531f;
        }
      }
      done += g.t1 - g.t0;
      if (!seg_next(p, g)) break;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (bars->abort) {  // products that nobody waits for end before their memory is given back
    const uint64_t t0 = now_ns();
    while (now_ns() - t0 < 50000) {
    }
  }
  if (warp == WARP_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

}  // namespace

size_t prefill_partial_bytes(int ctas, int D) { return size_t(ctas) * 2 * UNIT * (D + 3) * sizeof(float); }

tl_status launch_kv_prefill(PrefillParams& p, int D, int ctas, cudaStream_t st) {
  // floor(g / h) = floor(g m / 2^32), m = floor(2^32 / h) + 1, as long as g < 2^32 / h: g < 2^27, h <= 16
  const uint32_t halves = uint32_t(p.c.ps) / 16;
  p.page_magic = halves == 1 ? 0u : uint32_t((uint64_t(1) << 32) / halves) + 1;
  void* args[] = {&p};
  return D == 128 ? launch(reinterpret_cast<const void*>(&kv_prefill_kernel<128>), ctas, THREADS, smem_bytes<128>(), st,
                           args, false)
                  : launch(reinterpret_cast<const void*>(&kv_prefill_kernel<64>), ctas, THREADS, smem_bytes<64>(), st,
                           args, false);
}

}  // namespace tl
