// tl_kv_append.cu -- rotate new queries and keys, quantise keys and values to 8
// bits and append them to the paged cache, in one launch.
//
// For position p and pair (a, b): (y_a, y_b) = (x_a c - x_b s, x_b c + x_a s).  A
// page's block of one kv head has one power-of-two scale 2^(byte-127), the least
// that holds its largest magnitude within e4m3's 448.
//
// One team of threads owns one (page, kv head, keys or values) that receives
// tokens: it alone reads the block's scale, takes the new rows' maximum, re-codes
// the older rows where the scale grows, and writes.  So there are no atomics and
// no order that could change a result.  Other blocks rotate the queries.
//
// Which page is which: sequence s owns the items f(s) .. f(s+1)-1 of the grid with
// f(s) = cu[s] / page_size + 2 s.  n new tokens touch at most n / page_size + 2
// pages, wherever they begin, and f(s+1) - f(s) is at least that, so a block
// finds its sequence by counting the f(s) <= item: two loads for each sequence,
// all at once, and no prefix sum.  Where the count meets entries out of order,
// sums over the sequences that are right take its place.
//
// A code is ONE rounding of the exact rotated value.  x_a c is exact as p + e with
// e = fma(x_a, c, -p); the two products' sum is exact as a pair by the two-sum
// identity; and the pair is brought to "round to odd" in fp32 (towards zero, last
// bit set when inexact), from which a second rounding to fewer bits gives what a
// single one would.  Thus keys next to a rounding border do not depend on how
// fp32 rounds on the way.
//
// Bound by latency for single tokens (one sequence, 32 + 8 heads: 3.2 us of GPU time
// in a graph, 15.7 us a call with the host's share) and for prompts by the issue of
// the exact rounding together with the pages' chain from maximum to write.  A team
// keeps the first pass of its rows in registers between the two; the rest are read
// and rotated again (from L2: 106 MB come from memory for the 102 MB of the rows), as
// more rows in registers cost more in occupancy than they saved.  8192 tokens of
// 32 + 8 heads of 128 into pages of 64: 52 us, 3.65 TB/s over the bytes read and
// written, issue slots 65 % busy.
//
// tl_kv_append_norm is the same kernel with norms, x w / sqrt(mean x^2 + eps), and positions
// of its own.  The exact normed value costs ten times the instructions (a sum of squares in
// pairs, a Newton step for the root, products in pairs), and a code needs it only next to
// a border, so keys are computed in fp32 with a bound on what they are off by; where both
// ends of the bound have one code that is the code, else (one element of some 20000) the row
// is computed exactly, out of line.  Queries and keys have both elements of a rotated pair in one thread
// (77 -> 64 us for 8192 tokens as above), values stay in registers between maximum and write (61 -> 59), and so 8192
// tokens take 55 us (96 all exact), 3.4 TB/s, the queries 33 of them alone, keys 31 and values 10; 32 trees of
// up to 60 drafts behind 2000: 20 us.  Bound by the issue of instructions and the chains of a
// block of queries (position, tables) and of keys (two passes over the rows, the exact rows); six
// blocks of 128 threads (80 registers) share an SM (5: 56 us, 7: 64).  Rows kept in shared memory, tables fetched ahead,
// blocks of several tokens' queries or between those of the keys were slower.
#include <algorithm>
#include <type_traits>

#include "tl_internal.h"
#include "tl_kv.cuh"

namespace tl {
namespace {

constexpr int APP_THREADS = 128;

struct AppendParams {
  KvCacheDev c;
  KvBatch b;
  const uint16_t* k;
  const uint16_t* v;
  const uint16_t* q;
  int64_t k_ts, k_hs, v_ts, v_hs, q_ts, q_hs;
  uint16_t* q_out;
  const float* cos;
  const float* sin;
  int32_t H, rot, interleaved, max_pos;
  int32_t kv_blocks, groups;  // blocks for keys and values; blocks of one item
  const uint16_t* q_w;        // tl_kv_append_norm: weights of the norms, and where the tables are read
  const uint16_t* k_w;
  const int32_t* positions;
  float eps;
};

__device__ __forceinline__ void unpack8(uint4 w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ void load8(const uint16_t* p, float (&x)[8]) { unpack8(*reinterpret_cast<const uint4*>(p), x); }

// x c + t s as hi + rest, exactly but for what lies below 2^-48 of it; hi is the nearest float.  False: not finite,
// and hi is the plain fp32 value.
__device__ __forceinline__ bool dot2_pair(float x, float c, float t, float s, float& hi, float& rest) {
  const float p = __fmul_rn(x, c), r = __fmul_rn(t, s);
  const float pe = __fmaf_rn(x, c, -p), re = __fmaf_rn(t, s, -r);
  const float sum = __fadd_rn(p, r);
  const float back = __fsub_rn(sum, p);
  const float err = __fadd_rn(__fsub_rn(p, __fsub_rn(sum, back)), __fsub_rn(r, back));
  const float lo = __fadd_rn(err, __fadd_rn(pe, re));
  const bool finite = (__float_as_uint(sum) & 0x7FFFFFFFu) < 0x7F800000u;
  hi = finite ? __fadd_rn(sum, lo) : sum;
  rest = __fsub_rn(lo, __fsub_rn(hi, sum));
  return finite;
}
// hi + rest rounded to odd (see above): one step towards zero where rest points there, and the last bit set
__device__ __forceinline__ float to_odd(float hi, float rest) {
  const uint32_t u = __float_as_uint(hi);
  const uint32_t odd = (u + uint32_t(int32_t(__float_as_uint(rest) ^ u) >> 31)) | 1u;
  return __uint_as_float(rest != 0.0f ? odd : u);
}
__device__ __forceinline__ float dot2_odd(float x, float c, float t, float s) {
  float hi, rest;
  const bool finite = dot2_pair(x, c, t, s, hi, rest);
  return finite ? to_odd(hi, rest) : hi;
}

template <bool EXACT>
__device__ __forceinline__ float dot2(float x, float c, float t, float s) {
  return EXACT ? dot2_odd(x, c, t, s) : fmaf(x, c, t * s);
}

// What a thread needs of the tables for dims 8u .. 8u+7 at one position: eight pairs' (halves) or four pairs'
// (interleaved) cos and sin, and where in a row the other element of each pair is.
struct Turn {
  float c[8], s[8];
  int partner;  // first dim of the partner unit (halves); below 0: not rotated
  bool first;
};
__device__ __forceinline__ void load4(const float* p, float* x) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  x[0] = v.x;
  x[1] = v.y;
  x[2] = v.z;
  x[3] = v.w;
}
__device__ __forceinline__ void turn_at(const AppendParams& p, int u, int pos, Turn& w) {
  w.partner = -1;
  w.first = true;
  if (8 * u >= p.rot) return;
  const int half = p.rot >> 1;
  const float* cr = p.cos + int64_t(pos) * half;
  const float* sr = p.sin + int64_t(pos) * half;
  if (p.interleaved) {
    w.partner = 8 * u;
    load4(cr + 4 * u, w.c);
    load4(sr + 4 * u, w.s);
    return;
  }
  w.first = 8 * u < half;
  const int j = w.first ? 8 * u : 8 * u - half;
  w.partner = w.first ? 8 * u + half : j;
  load4(cr + j, w.c);
  load4(cr + j + 4, w.c + 4);
  load4(sr + j, w.s);
  load4(sr + j + 4, w.s + 4);
}
// x: the unit's dims, t: its partner's (halves)
template <bool EXACT>
__device__ __forceinline__ void turn(const AppendParams& p, const Turn& w, const float (&x)[8], const float (&t)[8], float (&y)[8]) {
  if (w.partner < 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i];
  } else if (p.interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[2 * i] = dot2<EXACT>(x[2 * i], w.c[i], -x[2 * i + 1], w.s[i]);
      y[2 * i + 1] = dot2<EXACT>(x[2 * i + 1], w.c[i], x[2 * i], w.s[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = dot2<EXACT>(x[i], w.c[i], w.first ? -t[i] : t[i], w.s[i]);
  }
}
// Dims 8u .. 8u+7 of one row, rotated by the table row at `pos`.
template <bool EXACT>
__device__ __forceinline__ void rotated8(const AppendParams& p, const uint16_t* row, int u, int pos, float (&y)[8]) {
  Turn w;
  turn_at(p, u, pos, w);
  float x[8], t[8];
  load8(row + 8 * u, x);
  load8(row + max(w.partner, 0), t);
  turn<EXACT>(p, w, x, t, y);
}

// ---------------------------------------------------------------- norms
// A row's factor 1 / sqrt(mean x^2 + eps), as hi + lo, for its elements times `scale` (1, or 2^-80 where the sum of
// squares would leave fp32).  A row with an infinity has 0 (finite elements become 0 and infinities NaN), one with a
// NaN has NaN.
struct Norm {
  float hi, lo, scale;
};
// The sum of squares over the D dims of a row that neighbouring lanes hold, 16 of them each: squares of bf16 are exact in
// fp32, sums are pairs.  Below 2^-63 squares lose bits, which eps (1e-12 at least) makes up for.
template <int D, bool EXACT>
__device__ __forceinline__ void square_sum(const float (&x)[16], float scale, uint32_t mask, float& s, float& e) {
  s = e = 0.0f;
  if (EXACT) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float v = x[i] * scale;
      const float2 t = two_sum(s, __fmul_rn(v, v));
      s = t.x;
      e += t.y;
    }
  } else {
    float q[4];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float v = x[i] * scale;
      q[i / 4] = fmaf(v, v, i % 4 ? q[i / 4] : 0.0f);
    }
    s = q[0] + q[1];
    s += q[2] + q[3];
  }
#pragma unroll
  for (int d = 1; d < D / 16; d <<= 1) {
    const float s2 = __shfl_xor_sync(mask, s, d);
    if (EXACT) {
      const float e2 = __shfl_xor_sync(mask, e, d);
      const float2 t = two_sum(s, s2);
      s = t.x;
      e = (e + e2) + t.y;
    } else {
      s += s2;
    }
  }
}
template <int N>
struct Some {
  float x[N];
};
using Eight = Some<8>;
// The sum of a row's squares times 2^-160.  (What is rare is kept out of line: the blocks' three paths share the
// instruction cache.)
template <int D, bool EXACT>
__device__ __noinline__ float2 small_square_sum(Some<16> x, uint32_t mask) {
  float s, e;
  square_sum<D, EXACT>(x.x, 0x1p-80f, mask, s, e);
  return make_float2(s, e);
}
// The lanes that hold a row.
template <int D>
__device__ __forceinline__ uint32_t row_lanes() {
  constexpr uint32_t LANES = D / 16;
  return ((1u << LANES) - 1u) << (lane_id() & ~(LANES - 1u));
}
// EXACT: to about 2^-45 by a step of Newton's iteration from the reciprocal root, its residual taken exactly:
// r (1 + d / 2 + 3 d^2 / 8), d = 1 - a r^2.
template <int D, bool EXACT>
__device__ __forceinline__ Norm row_norm(const float (&x)[16], float eps) {
  const uint32_t mask = row_lanes<D>();
  Norm n{0.0f, 0.0f, 1.0f};
  float s, e;
  square_sum<D, EXACT>(x, 1.0f, mask, s, e);
  if (!(s < INFINITY)) {  // the same for all lanes of the row
    n.scale = 0x1p-80f;
    Some<16> all;
#pragma unroll
    for (int i = 0; i < 16; ++i) all.x[i] = x[i];
    const float2 small = small_square_sum<D, EXACT>(all, mask);
    s = small.x;
    e = small.y;
    if (!(s < INFINITY)) {
      n.hi = s == INFINITY ? 0.0f : s;
      return n;
    }
    eps = 0.0f;
  }
  if (!EXACT) {
    const float a = fmaf(s, 1.0f / D, eps), r = rsqrtf(a);
    n.hi = fmaf(r * 0.5f, fmaf(a * r, -r, 1.0f), r);
    return n;
  }
  const float2 t = two_sum(s * (1.0f / D), eps);
  const float l = fmaf(e, 1.0f / D, t.y);
  const float a = __fadd_rn(t.x, l), b = __fsub_rn(l, __fsub_rn(a, t.x));  // mean + eps = a + b
  const float r = rsqrtf(a);
  const float p = __fmul_rn(r, r), pe = __fmaf_rn(r, r, -p);
  const float u = __fmul_rn(a, p), ue = __fmaf_rn(a, p, -u);
  const float d = __fsub_rn(__fsub_rn(1.0f, u), __fadd_rn(ue, __fmaf_rn(a, pe, __fmul_rn(b, p))));
  const float step = __fmul_rn(r, __fmul_rn(d, fmaf(0.375f, d, 0.5f)));
  n.hi = __fadd_rn(r, step);
  n.lo = __fsub_rn(step, __fsub_rn(n.hi, r));
  return n;
}
// (x c + t s) times the row's factor, rounded to odd; x and t with their weights, exact in fp32.
__device__ __forceinline__ float normed_dot2(const Norm& n, float x, float c, float t, float s) {
  float hi, rest;
  if (!dot2_pair(x, c, t, s, hi, rest)) return hi * n.hi;
  const float y = __fmul_rn(hi, n.hi);
  const float e = __fmaf_rn(hi, n.lo, __fmaf_rn(rest, n.hi, __fmaf_rn(hi, n.hi, -y)));
  const float z = __fadd_rn(y, e);
  return to_odd(z, __fsub_rn(e, __fsub_rn(z, y)));
}
// Dims 8u .. 8u+7 of a row, normed by n with the weights wx (its partner's: wt) and rotated.
__device__ __forceinline__ void turn_normed(const AppendParams& p, const Turn& w, const Norm& n, const float (&x)[8],
                                            const float (&t)[8], uint4 wx, uint4 wt, float (&y)[8]) {
  float a[8], b[8];
  unpack8(wx, a);
  unpack8(wt, b);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a[i] *= x[i] * n.scale;
    b[i] *= t[i] * n.scale;
  }
  if (w.partner < 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = normed_dot2(n, a[i], 1.0f, 0.0f, 0.0f);
  } else if (p.interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[2 * i] = normed_dot2(n, a[2 * i], w.c[i], -a[2 * i + 1], w.s[i]);
      y[2 * i + 1] = normed_dot2(n, a[2 * i + 1], w.c[i], a[2 * i], w.s[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = normed_dot2(n, a[i], w.c[i], w.first ? -b[i] : b[i], w.s[i]);
  }
}

// What a normed and rotated element is off by in fp32, relative to the sum of its two products' magnitudes, in steps of 2^-24:
// the row's factor by 6 (a mean of squares by 9 roundings, halved by the root, and one and a half of the corrected root),
// the products, their sum, the product with the factor and the bound's end by one each: 10, and 11 leave room for what these
// do to one another.
constexpr float kNormErr = 0x1.6p-21f;
// A thread's 16 dims of a row of keys: two units of 8 whose dims are each other's partners, so that a row and the tables
// are read once, and every product of an element and its weight serves two outputs.
struct Pair {
  int first, second;  // units
  int table;          // first of 8 entries of a table's row; below 0: not rotated
};
__device__ __forceinline__ Pair pair_of(const AppendParams& p, int m) {
  const int turned = p.rot >> 4;
  if (m >= turned) return {2 * m, 2 * m + 1, -1};
  return p.interleaved ? Pair{2 * m, 2 * m + 1, 8 * m} : Pair{m, m + turned, 8 * m};
}
__device__ __forceinline__ void unpack_pair(uint4 a, uint4 b, float (&x)[16]) {
  float u[8], v[8];
  unpack8(a, u);
  unpack8(b, v);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = u[i];
    x[8 + i] = v[i];
  }
}
struct PairRow {
  uint4 a, b;
};
__device__ __forceinline__ PairRow raw_pair(const uint16_t* row, const Pair& m) {
  return {*reinterpret_cast<const uint4*>(row + 8 * m.first), *reinterpret_cast<const uint4*>(row + 8 * m.second)};
}
__device__ __forceinline__ void load_pair(const uint16_t* row, const Pair& m, float (&x)[16]) {
  const PairRow r = raw_pair(row, m);
  unpack_pair(r.a, r.b, x);
}
__device__ __forceinline__ void load_tables(const AppendParams& p, const Pair& m, int pos, float (&c)[8], float (&s)[8]) {
  if (m.table < 0) return;
  const int64_t at = int64_t(pos) * (p.rot >> 1) + m.table;
  load4(p.cos + at, c);
  load4(p.cos + at + 4, c + 4);
  load4(p.sin + at, s);
  load4(p.sin + at + 4, s + 4);
}
// Sixteen elements in fp32 but for the row's factor, and their products' magnitudes added up, in pairs of neighbours:
// use(factor, i, y of 2 i, of 2 i + 1, z of both).
template <int D, class Use>
__device__ __forceinline__ void fast_key16(const AppendParams& p, const PairRow& row, const Pair& m, int pos, Use use) {
  float c[8], s[8], x[16], w[16];
  load_tables(p, m, pos, c, s);
  unpack_pair(row.a, row.b, x);
  const Norm n = row_norm<D, false>(x, p.eps);
  if (n.scale != 1.0f) {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] *= n.scale;
  }
  load_pair(p.k_w, m, w);
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] *= w[i];
  auto turn = [&](int a, int b, int j, float& ya, float& yb, float& za, float& zb) {
    const float ac = x[a] * c[j], bs = x[b] * s[j], bc = x[b] * c[j], as = x[a] * s[j];
    ya = ac - bs;
    za = fabsf(ac) + fabsf(bs);
    yb = bc + as;
    zb = fabsf(bc) + fabsf(as);
  };
  if (m.table < 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) use(n.hi, i, x[2 * i], x[2 * i + 1], fabsf(x[2 * i]), fabsf(x[2 * i + 1]));
  } else if (p.interleaved) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float y0, y1, z0, z1;
      turn(2 * j, 2 * j + 1, j, y0, y1, z0, z1);
      use(n.hi, j, y0, y1, z0, z1);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float a0, a1, b0, b1, za0, za1, zb0, zb1;
      turn(2 * j, 8 + 2 * j, 2 * j, a0, b0, za0, zb0);
      turn(2 * j + 1, 9 + 2 * j, 2 * j + 1, a1, b1, za1, zb1);
      use(n.hi, j, a0, a1, za0, za1);
      use(n.hi, 4 + j, b0, b1, zb0, zb1);
    }
  }
}
// The same exactly, rounded to odd.
template <int D>
__device__ __noinline__ Some<16> exact_key16(const AppendParams& p, const uint16_t* row, Pair m, int pos) {
  float x[16], a[8], b[8];
  load_pair(row, m, x);
  const Norm n = row_norm<D, true>(x, p.eps);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a[i] = x[i];
    b[i] = x[8 + i];
  }
  const uint4 wa = *reinterpret_cast<const uint4*>(p.k_w + 8 * m.first), wb = *reinterpret_cast<const uint4*>(p.k_w + 8 * m.second);
  const bool own = m.table < 0 || p.interleaved;  // no partners among the other unit
  Some<16> out;
  float y[8];
  Turn w;
  turn_at(p, m.first, pos, w);
  turn_normed(p, w, n, a, own ? a : b, wa, own ? wa : wb, y);
#pragma unroll
  for (int i = 0; i < 8; ++i) out.x[i] = y[i];
  turn_at(p, m.second, pos, w);
  turn_normed(p, w, n, b, own ? b : a, wb, own ? wb : wa, y);
#pragma unroll
  for (int i = 0; i < 8; ++i) out.x[8 + i] = y[i];
  return out;
}

// A token's queries by the block: a thread has the same dims of every 16th (32nd) head, the tables and weights once, two
// heads' loads at a time, the first ones before the block knows the token's position (8192 tokens: 64 -> 61 us).
struct Nothing {
  __device__ __forceinline__ Nothing(const AppendParams&, int) {}
};
template <int D>
struct Queries {
  static constexpr int PAIRS = D / 16, STRIDE = APP_THREADS / PAIRS, BATCH = 2;
  Pair m;
  const uint16_t* row;
  int h0;
  uint4 xa[BATCH], xb[BATCH];

  __device__ __forceinline__ Queries(const AppendParams& p, int t) : m(pair_of(p, int(threadIdx.x) % PAIRS)),
        row(p.q + int64_t(t) * p.q_ts), h0(int(threadIdx.x) / PAIRS) {
    load(p);
  }
  __device__ __forceinline__ void load(const AppendParams& p) {
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const uint16_t* head = row + min(h0 + k * STRIDE, p.H - 1) * p.q_hs;
      xa[k] = *reinterpret_cast<const uint4*>(head + 8 * m.first);
      xb[k] = *reinterpret_cast<const uint4*>(head + 8 * m.second);
    }
  }
  __device__ __forceinline__ void store(const AppendParams& p, uint16_t* dst, int pos);
};
template <int D>
__device__ __forceinline__ void Queries<D>::store(const AppendParams& p, uint16_t* dst, int pos) {
  float c[8], s[8];
  load_tables(p, m, pos, c, s);
  const bool norm = p.q_w;
  uint4 wa = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u), wb = wa;  // ones
  if (norm) {
    wa = *reinterpret_cast<const uint4*>(p.q_w + 8 * m.first);
    wb = *reinterpret_cast<const uint4*>(p.q_w + 8 * m.second);
  }
  while (h0 < p.H) {
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int h = h0 + k * STRIDE;
      if (h >= p.H) break;
      float x[16], w[16];
      unpack_pair(xa[k], xb[k], x);
      float f = 1.0f;
      if (norm) {
        const Norm n = row_norm<D, false>(x, p.eps);
        f = n.hi;
        if (n.scale != 1.0f) {
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] *= n.scale;
        }
      }
      unpack_pair(wa, wb, w);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] *= w[i];
      auto turn = [&](int a, int b, int j) {
        const float ya = fmaf(x[a], c[j], -x[b] * s[j]), yb = fmaf(x[b], c[j], x[a] * s[j]);
        x[a] = ya;
        x[b] = yb;
      };
      if (m.table >= 0) {
        if (p.interleaved) {
#pragma unroll
          for (int j = 0; j < 8; ++j) turn(2 * j, 2 * j + 1, j);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) turn(j, 8 + j, j);
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] *= f;
      uint16_t* to = dst + h * D;
      st_global_v4(to + 8 * m.first, pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
      st_global_v4(to + 8 * m.second, pack_bf16x2(x[8], x[9]), pack_bf16x2(x[10], x[11]), pack_bf16x2(x[12], x[13]),
                   pack_bf16x2(x[14], x[15]));
    }
    h0 += STRIDE * BATCH;
    if (h0 < p.H) load(p);
  }
}

// Keys that are not normed, out of line.
__device__ __noinline__ Eight rotated_key8(const AppendParams& p, const uint16_t* row, int u, int pos) {
  Eight y;
  rotated8<true>(p, row, u, pos, y.x);
  return y;
}

// How many of the f(s) given by the functor are at or below x, over the block; and in the upper bits whether any
// sequence's rows are out of order or out of range.
constexpr uint32_t kOutOfOrder = 1u << 24;  // B is at most 2^20
template <class F>
__device__ __forceinline__ uint32_t count_below(const KvBatch& b, int x, uint32_t* smem, F f) {
  uint32_t n = 0;
  bool odd = false;
  for (int s = threadIdx.x; s < b.B; s += APP_THREADS) {
    const int c0 = b.cu[s], c1 = b.cu[s + 1];
    n += f(s, c0) <= x;
    odd |= c0 < 0 || c1 < c0 || c1 > b.n_tokens;
  }
  n = __reduce_add_sync(0xffffffffu, n + (odd ? kOutOfOrder : 0u));
  if (lane_id() == 0) smem[warp_id()] = n;
  __syncthreads();
  return smem[0] + smem[1] + smem[2] + smem[3];
}

// The same search where cu_seqlens is wrong somewhere, so that counting would go astray for sequences that are right.
// A sequence counts if its rows are in order, in range and begin no earlier than those of the ones before it end;
// such sequences share no row, so the grid has an item for each of their pages.  The one with token t (PAGES: with
// item t) or -1, and its first item.  All threads of the block call it.
template <bool PAGES>
__device__ __noinline__ int2 find_among_wrong(const KvBatch& b, int ps, int t) {
  __shared__ int ends[4], sums[4], found[2];
  const int lane = int(lane_id()), warp = int(warp_id());
  if (threadIdx.x == 0) found[0] = -1;
  int end_before = 0, items_before = 0;
  for (int s0 = 0; s0 < b.B; s0 += APP_THREADS) {
    const int s = s0 + int(threadIdx.x);
    int c0 = 0, c1 = 0;
    if (s < b.B) {
      c0 = b.cu[s];
      c1 = b.cu[s + 1];
    }
    const bool ordered = c0 >= 0 && c1 >= c0 && c1 <= b.n_tokens;
    int end = ordered ? c1 : 0;  // the largest end so far
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, end, d);
      if (lane >= d) end = max(end, x);
    }
    if (lane == 31) ends[warp] = end;
    __syncthreads();
    int before = __shfl_up_sync(0xffffffffu, end, 1);
    if (lane == 0) before = 0;
    before = max(before, end_before);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if (w < warp) before = max(before, ends[w]);
      end_before = max(end_before, ends[w]);
    }
    const bool own = ordered && c0 >= before;
    if (s < b.B && !own) record_error(b.status, kKvInvalid, uint32_t(s), uint32_t(c0), uint32_t(c1));
    const int need = own && c1 > c0 ? (c1 - c0) / ps + 2 : 0;
    int sum = need;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += x;
    }
    if (lane == 31) sums[warp] = sum;
    __syncthreads();
    sum += items_before;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if (w < warp) sum += sums[w];
      items_before += sums[w];
    }
    if (PAGES ? t >= sum - need && t < sum : own && t >= c0 && t < c1) {  // one thread at most
      found[0] = s;
      found[1] = sum - need;
    }
    __syncthreads();
    if (found[0] >= 0) break;
  }
  return make_int2(found[0], found[1]);
}

// The least scale byte whose 448 * 2^(byte-127) holds the magnitude with these bits.
__device__ __forceinline__ int scale_need(uint32_t amax_bits) {
  return max(0, int(amax_bits >> 23) - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0));
}

// Where the tables are read for the token at `pos`, new token `t` of the batch.
__device__ __forceinline__ int table_row(const AppendParams& p, int t, int pos, int s) {
  if (!p.positions || p.rot == 0) return pos;
  const int at = p.positions[t];
  if (at >= 0 && at < p.max_pos) return at;
  record_error(p.b.status, kKvInvalid, uint32_t(s), uint32_t(at), uint32_t(p.max_pos));
  return 0;
}

// TEAM threads to one (page, head, keys or values); KEEP passes' rows stay in registers.
template <int D, int TEAM, int KEEP, bool NORM>
__global__ void __launch_bounds__(APP_THREADS, NORM ? 6 : 8) kv_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int UNITS = D / 8;             // threads to a row
  constexpr int STEP = TEAM / UNITS;       // rows of one pass
  __shared__ uint32_t counts[4];
  __shared__ uint32_t team_max[4], team_low[4];
  const int tid = threadIdx.x;
  const KvBatch& b = p.b;
  const int ps = p.c.ps;

  if (int(blockIdx.x) >= p.kv_blocks) {
    // ---------------------------------------------------------------- one token's queries
    const int t = int(blockIdx.x) - p.kv_blocks;
    std::conditional_t<NORM, Queries<D>, Nothing> queries(p, t);
    const uint32_t n = count_below(b, t, counts, [](int, int c0) { return c0; });
    const int s = n < kOutOfOrder ? int(n) - 1 : find_among_wrong<false>(b, ps, t).x;
    if (s < 0) return;
    const KvSeq seq = kv_seq(b, ps, s);
    if (t < seq.row0 || t >= seq.row0 + seq.q) return;
    int pos = seq.len - seq.q + (t - seq.row0);
    if (NORM && pos >= 0) pos = table_row(p, t, pos, s);
    if (p.rot > 0 && (pos < 0 || pos >= p.max_pos)) {
      if (tid == 0) record_error(b.status, kKvInvalid, uint32_t(s), uint32_t(pos), uint32_t(p.max_pos));
      return;
    }
    const uint16_t* row = p.q + int64_t(t) * p.q_ts;
    uint16_t* dst = p.q_out + int64_t(t) * p.H * D;
    if constexpr (NORM) {
      queries.store(p, dst, pos);
      return;
    }
    // a thread has the same dims of every fourth (eighth) head or so: the tables once, four heads' loads at a time
    const int u = tid % UNITS;
    constexpr int STRIDE = APP_THREADS / UNITS, BATCH = 4;
    Turn w;
    turn_at(p, u, pos, w);
    for (int h0 = tid / UNITS; h0 < p.H; h0 += STRIDE * BATCH) {
      uint4 x[BATCH], t4[BATCH];
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        const uint16_t* head = row + min(h0 + k * STRIDE, p.H - 1) * p.q_hs;
        x[k] = *reinterpret_cast<const uint4*>(head + 8 * u);
        t4[k] = *reinterpret_cast<const uint4*>(head + max(w.partner, 0));
      }
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        const int h = h0 + k * STRIDE;
        if (h >= p.H) break;
        float a[8], b8[8], y[8];
        unpack8(x[k], a);
        unpack8(t4[k], b8);
        turn<false>(p, w, a, b8, y);
        st_global_v4(dst + h * D + 8 * u, pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                     pack_bf16x2(y[6], y[7]));
      }
    }
    return;
  }

  // ---------------------------------------------------------------- one page's keys and values
  const int item = int(blockIdx.x) / p.groups;
  const uint32_t n = count_below(b, item, counts, [ps](int s, int c0) { return c0 / ps + 2 * s; });
  int2 at = make_int2(int(n) - 1, -1);
  if (n >= kOutOfOrder) at = find_among_wrong<true>(b, ps, item);
  const int s = at.x;
  const int team = (int(blockIdx.x) % p.groups) * (APP_THREADS / TEAM) + tid / TEAM;
  if (s < 0) return;
  const KvSeq seq = kv_seq(b, ps, s);
  const int start = seq.len - seq.q;
  if (seq.q == 0) return;
  const int begin = max(start, 0);
  const int64_t page_no = begin / ps + (item - (at.y >= 0 ? at.y : seq.row0 / ps + 2 * s));
  const int64_t page_begin = page_no * ps;
  if (page_begin >= seq.len || page_no < begin / ps) return;
  const int lo = max(int(page_begin), begin);                    // new positions in the page
  const int hi = int(min(page_begin + ps, int64_t(seq.len)));
  const int page = b.table[int64_t(s) * b.max_pages + page_no];  // page_no < max_pages: the length was checked
  if (page < 0 || page >= p.c.num_pages || (p.rot > 0 && hi > p.max_pos && !(NORM && p.positions))) {
    if (tid == 0) record_error(b.status, kKvInvalid, uint32_t(s), uint32_t(page), uint32_t(page_no));
    return;
  }
  const bool active = team < 2 * p.c.Hkv;  // the whole team or none of it
  if (TEAM < 32 * 4 && !active) return;
  const int head = team >> 1;
  const bool values = team & 1;
  const int64_t block_at = int64_t(page) * p.c.page_stride + int64_t(head) * p.c.head_stride;
  uint8_t* codes = (values ? p.c.v : p.c.k) + block_at;
  uint8_t* scale_at = (values ? p.c.vs : p.c.ks) + int64_t(page) * p.c.Hkv + head;
  const uint16_t* src = values ? p.v + head * p.v_hs : p.k + head * p.k_hs;
  const int64_t src_ts = values ? p.v_ts : p.k_ts;
  const int slot0 = lo - int(page_begin), rows = hi - lo;
  const int src0 = seq.row0 + (lo - start);
  const int member = tid % TEAM, u = member % UNITS, r0 = member / UNITS;
  const int old = slot0 > 0 ? int(*scale_at) : 0;

  float y[KEEP][8];
  uint32_t amax = 0;
  auto row8 = [&](int r, float(&out)[8]) {
    const uint16_t* row = src + int64_t(src0 + r) * src_ts;
    if (values) {
      load8(row + 8 * u, out);
    } else if (NORM) {
      const Eight y = rotated_key8(p, row, u, table_row(p, src0 + r, lo + r, s));
#pragma unroll
      for (int i = 0; i < 8; ++i) out[i] = y.x[i];
    } else {
      rotated8<true>(p, row, u, lo + r, out);
    }
  };
  auto take_max = [&](const auto& x) {
#pragma unroll
    for (int i = 0; i < int(sizeof(x) / sizeof(float)); ++i) {
      const uint32_t a = __float_as_uint(x[i]) & 0x7FFFFFFFu;
      if (a < 0x7F800000u) amax = max(amax, a);
    }
  };
  auto reduce = [&]() {
    amax = __reduce_max_sync(0xffffffffu, amax);
    if (TEAM > 32) {
      if (lane_id() == 0) team_max[warp_id()] = amax;
      __syncthreads();
      amax = max(max(team_max[0], team_max[1]), max(team_max[2], team_max[3]));
    } else {
      __syncwarp();  // the scale is read by the whole team before one of it writes it
    }
  };
  // The older rows to the new scale, and the scale.
  auto settle = [&](int byte) {
    if (slot0 > 0 && byte > old) {
      const float f = pow2f(max(old - byte, -127));
      for (int i = member; i < slot0 * (D / 16); i += TEAM) {
        uint4* at = reinterpret_cast<uint4*>(codes + int64_t(i / (D / 16)) * p.c.token_stride + (i % (D / 16)) * 16);
        *at = recode16(*at, f);
      }
    }
    if (member == 0) *scale_at = uint8_t(byte);
  };
  if (NORM && values) {
    // ---------------------------------------------------------------- values
    // A thread's first rows stay in registers, all on their way at once.
    constexpr int HOLD = 8;
    const uint16_t* from = src + int64_t(src0 + r0) * src_ts + 8 * u;
    auto load = [&](int k) { return *reinterpret_cast<const uint4*>(from + int64_t(k) * STEP * src_ts); };
    auto here = [&](int k) { return r0 + k * STEP < rows; };
    uint4 v[HOLD];
#pragma unroll
    for (int k = 0; k < HOLD; ++k) v[k] = here(k) ? load(k) : make_uint4(0, 0, 0, 0);
    uint32_t most = 0;  // of the halves, without their signs
    auto look = [&](const uint4& x) {
      most = __vmaxu2(most, __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu), __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu)));
    };
#pragma unroll
    for (int k = 0; k < HOLD; ++k) look(v[k]);
    for (int k = HOLD; here(k); ++k) look(load(k));
    amax = max(most << 16, most & 0xFFFF0000u);
    if (amax >= 0x7F800000u) {  // (infinities and NaN do not count)
      amax = 0;
      for (int k = 0; here(k); ++k) {
        float x[8];
        unpack8(load(k), x);
        take_max(x);
      }
    }
    reduce();
    const int byte = max(old, scale_need(amax));
    const float inv = byte == 255 ? __uint_as_float(0x00200000u) : pow2f(127 - byte);
    settle(byte);
    uint8_t* to = codes + int64_t(slot0 + r0) * p.c.token_stride + 8 * u;
    auto write = [&](int k, const uint4& w) {
      float x[8];
      unpack8(w, x);
      *reinterpret_cast<uint2*>(to + int64_t(k) * STEP * p.c.token_stride) =
          make_uint2(f32x2_to_e4m3x2(x[0] * inv, x[1] * inv) | (f32x2_to_e4m3x2(x[2] * inv, x[3] * inv) << 16),
                     f32x2_to_e4m3x2(x[4] * inv, x[5] * inv) | (f32x2_to_e4m3x2(x[6] * inv, x[7] * inv) << 16));
    };
#pragma unroll
    for (int k = 0; k < HOLD; ++k)
      if (here(k)) write(k, v[k]);
    for (int k = HOLD; here(k); ++k) write(k, load(k));
    return;
  }
  if (NORM && !values && p.k_w) {
    // ---------------------------------------------------------------- normed keys
    // A code is that of the exact value; fp32 tells it wherever what it is off by does not reach across a border between
    // two codes.  The exact value is computed where it does (one element of some 20000), and for the block's
    // maximum where its byte hangs on that, or where it is so large that fp32 might not hold it.
    constexpr int PAIRS = D / 16, ROWS = TEAM / PAIRS;  // threads of a row; rows of a pass
    const Pair m = pair_of(p, member % PAIRS);
    auto row_at = [&](int r) { return src + int64_t(src0 + r) * src_ts; };
    auto pos_of = [&](int r) { return table_row(p, src0 + r, lo + r, s); };
    uint32_t low = 0;
    PairRow next = raw_pair(row_at(min(member / PAIRS, rows - 1)), m);
    for (int r = member / PAIRS; r < rows; r += ROWS) {
      const PairRow row = next;
      next = raw_pair(row_at(r + ROWS < rows ? r + ROWS : member / PAIRS), m);  // (at last the first again)
      float h, most = 0.0f;
      uint32_t sum = 0;  // (as whole numbers NaN and infinity are above all)
      fast_key16<D>(p, row, m, pos_of(r), [&](float f, int, float y0, float y1, float z0, float z1) {
        h = f;
        most = fmaxf(most, fmaxf(fabsf(y0), fabsf(y1)));
        sum = max(sum, max(__float_as_uint(z0), __float_as_uint(z1)));
      });
      const float off = __uint_as_float(sum) * kNormErr;
      amax = max(amax, __float_as_uint((most + off) * h) & 0x7FFFFFFFu);
      low = max(low, __float_as_uint(fmaxf((most - off) * h, 0.0f)));
    }
    low = __reduce_max_sync(0xffffffffu, low);
    if (TEAM > 32 && lane_id() == 0) team_low[warp_id()] = low;
    reduce();
    if (TEAM > 32) low = max(max(team_low[0], team_low[1]), max(team_low[2], team_low[3]));
    if (amax >= 0x7E800000u || scale_need(amax) != scale_need(low)) {
      if (TEAM > 32) __syncthreads();
      amax = 0;
      for (int r = member / PAIRS; r < rows; r += ROWS) {
        const Some<16> x = exact_key16<D>(p, row_at(r), m, pos_of(r));
        take_max(x.x);
      }
      reduce();
    }
    const int byte = max(old, scale_need(amax));
    const float inv = byte == 255 ? __uint_as_float(0x00200000u) : pow2f(127 - byte);
    settle(byte);
    // (Scales so small or large that a row's factor times one might leave fp32: exactly.)
    const bool fast = byte >= 40 && byte <= 180;
    for (int r = member / PAIRS; r < rows; r += ROWS) {
      const PairRow row = next;
      next = raw_pair(row_at(min(r + ROWS, rows - 1)), m);
      uint32_t code[8], differ = fast ? 0u : 1u;
      fast_key16<D>(p, row, m, pos_of(r), [&](float f, int i, float y0, float y1, float z0, float z1) {
        const float h = f * inv, err = h * kNormErr, a = y0 * h, b = y1 * h;
        code[i] = f32x2_to_e4m3x2(fmaf(z0, -err, a), fmaf(z1, -err, b));
        differ |= code[i] ^ f32x2_to_e4m3x2(fmaf(z0, err, a), fmaf(z1, err, b));
      });
      if (__any_sync(row_lanes<D>(), differ != 0)) {
        const Some<16> e = exact_key16<D>(p, row_at(r), m, pos_of(r));
#pragma unroll
        for (int i = 0; i < 8; ++i) code[i] = f32x2_to_e4m3x2(e.x[2 * i] * inv, e.x[2 * i + 1] * inv);
      }
      uint8_t* at = codes + int64_t(slot0 + r) * p.c.token_stride;
      *reinterpret_cast<uint2*>(at + 8 * m.first) = make_uint2(code[0] | code[1] << 16, code[2] | code[3] << 16);
      *reinterpret_cast<uint2*>(at + 8 * m.second) = make_uint2(code[4] | code[5] << 16, code[6] | code[7] << 16);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < KEEP; ++j) {
    const int r = r0 + j * STEP;
    if (r < rows) {
      row8(r, y[j]);
      take_max(y[j]);
    }
  }
  for (int r = r0 + KEEP * STEP; r < rows; r += STEP) {
    float x[8];
    row8(r, x);
    take_max(x);
  }
  reduce();
  const int byte = max(old, scale_need(amax));
  const float inv = byte == 255 ? __uint_as_float(0x00200000u) : pow2f(127 - byte);  // 255: NaN it was and stays
  settle(byte);
  auto write8 = [&](int r, const float(&x)[8]) {
    uint2 w;
    w.x = f32x2_to_e4m3x2(x[0] * inv, x[1] * inv) | (f32x2_to_e4m3x2(x[2] * inv, x[3] * inv) << 16);
    w.y = f32x2_to_e4m3x2(x[4] * inv, x[5] * inv) | (f32x2_to_e4m3x2(x[6] * inv, x[7] * inv) << 16);
    *reinterpret_cast<uint2*>(codes + int64_t(slot0 + r) * p.c.token_stride + 8 * u) = w;
  };
#pragma unroll
  for (int j = 0; j < KEEP; ++j) {
    const int r = r0 + j * STEP;
    if (r < rows) write8(r, y[j]);
  }
  for (int r = r0 + KEEP * STEP; r < rows; r += STEP) {
    float x[8];
    row8(r, x);
    write8(r, x);
  }
}

// Whether any of n rows of `span` bytes, `stride` apart from `rows` on, meets the `bytes` at `block`.
bool rows_meet(const void* rows, int64_t stride, int64_t span, int64_t n, const void* block, int64_t bytes) {
  const int64_t at = int64_t(reinterpret_cast<uintptr_t>(block)) - int64_t(reinterpret_cast<uintptr_t>(rows));
  // row t is [t stride, t stride + span): the first that ends behind the block's begin
  const int64_t t = at < span || stride == 0 ? 0 : (at - span) / stride + 1;
  return t < n && t * stride + span > at && t * stride < at + bytes;
}

}  // namespace

// Checks shared by the cache's calls (tl_kv_attn too).
tl_status check_kv_cache(const char* who, const tl_kv_cache& c) {
  if (!c.k || !c.v || !c.k_scale || !c.v_scale) return fail(TL_ERR_INVALID, "%s: NULL cache pointer", who);
  if (!aligned16(c.k) || !aligned16(c.v)) return fail(TL_ERR_INVALID, "%s: cache codes must be 16-byte aligned", who);
  if (c.num_pages < 1 || c.H_kv < 1) return fail(TL_ERR_INVALID, "%s: empty cache", who);
  if (c.head_dim != 64 && c.head_dim != 128)
    return fail(TL_ERR_UNSUPPORTED, "%s: head_dim %d (64 or 128)", who, c.head_dim);
  if (c.page_size < 16 || c.page_size > 256 || c.page_size % 16)
    return fail(TL_ERR_UNSUPPORTED, "%s: page_size %d (a multiple of 16, 16..256)", who, c.page_size);
  for (int64_t s : {c.page_stride, c.head_stride, c.token_stride})
    if (s < c.head_dim || s % 16 || s > (int64_t(1) << 40))
      return fail(TL_ERR_INVALID, "%s: cache strides must be multiples of 16 bytes, head_dim at least", who);
  if (c.H_kv > 4096) return fail(TL_ERR_UNSUPPORTED, "%s: H_kv %d", who, c.H_kv);
  return TL_OK;
}

}  // namespace tl

namespace tl {
namespace {

// Both calls; n: what tl_kv_append_norm has beside the rest, or NULL.
tl_status append(const char* who, const tl_kv_append_args* a, const tl_kv_append_norm_args* n, void* stream) {
  if (!a) return fail(TL_ERR_INVALID, "%s: NULL args", who);
  if (a->n_tokens < 0 || a->B < 1 || a->B > (1 << 20) || a->max_pages < 1)
    return fail(TL_ERR_INVALID, "%s: n_tokens %d, B %d, max_pages %d", who, a->n_tokens, a->B, a->max_pages);
  if (tl_status s = check_kv_cache(who, a->cache)) return s;
  const int D = a->cache.head_dim;
  if (a->H < 0 || a->H > 65536) return fail(TL_ERR_INVALID, "%s: H %d", who, a->H);
  if (a->rot_dim < 0 || a->rot_dim > D || a->rot_dim % 16)
    return fail(TL_ERR_UNSUPPORTED, "%s: rot_dim %d (a multiple of 16, 0..head_dim)", who, a->rot_dim);
  if (a->interleaved != 0 && a->interleaved != 1)
    return fail(TL_ERR_INVALID, "%s: interleaved %d", who, a->interleaved);
  if (a->max_q_len < 0) return fail(TL_ERR_INVALID, "%s: max_q_len %d", who, a->max_q_len);
  if (!a->cu_seqlens || !a->seq_lens || !a->page_table || !a->signals)
    return fail(TL_ERR_INVALID, "%s: NULL pointer argument", who);
  if (a->n_tokens == 0) return TL_OK;
  if (!a->k || !a->v) return fail(TL_ERR_INVALID, "%s: NULL pointer argument", who);
  if ((a->H > 0) != (a->q != nullptr) || (a->H > 0) != (a->q_out != nullptr))
    return fail(TL_ERR_INVALID, "%s: q and q_out go with H > 0", who);
  if (a->rot_dim > 0 && (!a->cos || !a->sin || a->max_pos < 1))
    return fail(TL_ERR_INVALID, "%s: rot_dim %d needs cos, sin and max_pos", who, a->rot_dim);
  for (const void* ptr : {a->k, a->v, a->q, (const void*)a->q_out, (const void*)a->cos, (const void*)a->sin})
    if (!aligned16(ptr)) return fail(TL_ERR_INVALID, "%s: pointers must be 16-byte aligned", who);
  for (int64_t s : {a->k_token_stride, a->k_head_stride, a->v_token_stride, a->v_head_stride, a->q_token_stride,
                    a->q_head_stride})
    if (s < 0 || s % 8) return fail(TL_ERR_INVALID, "%s: strides must be multiples of 8 elements", who);
  // A row's dims are read by the threads of both of a pair's units, with no order between them and the writes.
  if (a->H > 0 && rows_meet(a->q, a->q_token_stride * 2, (int64_t(a->H - 1) * a->q_head_stride + D) * 2, a->n_tokens,
                            a->q_out, int64_t(a->n_tokens) * a->H * D * 2))
    return fail(TL_ERR_INVALID, "%s: q_out overlaps q", who);
  if (n) {
    if (!aligned16(n->q_weight) || !aligned16(n->k_weight) || (reinterpret_cast<uintptr_t>(n->positions) & 3u))
      return fail(TL_ERR_INVALID, "%s: weights must be 16-byte aligned, positions 4-byte", who);
    if (n->q_weight && a->H == 0) return fail(TL_ERR_INVALID, "%s: q_weight without queries", who);
    if ((n->q_weight || n->k_weight) && !(n->eps >= 1e-12f && n->eps <= 1e12f))
      return fail(TL_ERR_INVALID, "%s: eps must lie within 1e-12 and 1e12", who);
  }
  DeviceInfo di{};
  if (tl_status s = device_info(&di)) return s;
  if (a->signals->device != di.device)
    return fail(TL_ERR_INVALID, "%s: signals belong to another device", who);

  AppendParams p{};
  const tl_kv_cache& c = a->cache;
  p.c = KvCacheDev{static_cast<uint8_t*>(c.k), static_cast<uint8_t*>(c.v), c.k_scale, c.v_scale, c.page_stride,
                   c.head_stride, c.token_stride, c.num_pages, c.page_size, c.H_kv};
  p.b = KvBatch{a->cu_seqlens, a->seq_lens, a->page_table, a->signals->status, a->B, a->n_tokens, a->max_pages};
  p.k = static_cast<const uint16_t*>(a->k);
  p.v = static_cast<const uint16_t*>(a->v);
  p.q = static_cast<const uint16_t*>(a->q);
  p.k_ts = a->k_token_stride;
  p.k_hs = a->k_head_stride;
  p.v_ts = a->v_token_stride;
  p.v_hs = a->v_head_stride;
  p.q_ts = a->q_token_stride;
  p.q_hs = a->q_head_stride;
  p.q_out = static_cast<uint16_t*>(a->q_out);
  p.cos = a->cos;
  p.sin = a->sin;
  p.H = a->H;
  p.rot = a->rot_dim;
  p.interleaved = a->interleaved;
  p.max_pos = a->max_pos;
  if (n) {
    p.q_w = static_cast<const uint16_t*>(n->q_weight);
    p.k_w = static_cast<const uint16_t*>(n->k_weight);
    p.positions = n->positions;
    p.eps = n->eps;
  }
  const int per_seq = a->max_q_len ? std::min(a->max_q_len, a->n_tokens) : cdiv(a->n_tokens, a->B);
  // A whole block to a page's keys or values of one head where a page gets 32 rows, else a warp: 8192 tokens of 8 kv heads
  // of 128 into pages of 16, 32, 64 and 256 take 58, 54, 52 and 82 us with blocks, 54, 54, 75 and 211 us with warps.  With
  // norms 76, 63 and 55 us, and 57, 59 and 66 (16, 32, 64); few sequences gain from blocks earlier there, as a key's row has
  // half the lanes and two passes: one tree of 26 takes 10.5 and 17.6 us, 32 trees of 16 10.4 and 15.1, 96 of 16 19.1 and 17.9.
  const bool wide = std::min(per_seq, c.page_size) >= 32;
  const int64_t items = int64_t(a->n_tokens) / c.page_size + 2 * int64_t(a->B);
  p.groups = wide ? 2 * c.H_kv : cdiv(2 * c.H_kv, APP_THREADS / 32);
  const int64_t blocks = items * p.groups + (a->H > 0 ? a->n_tokens : 0);
  if (blocks > 0x7FFFFFFFll) return fail(TL_ERR_UNSUPPORTED, "%s: too many tokens", who);
  p.kv_blocks = int(items * p.groups);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto go = [&](auto dim, auto norm) {
    constexpr int D = decltype(dim)::value;
    constexpr bool NORM = decltype(norm)::value;
    if (wide) kv_append_kernel<D, 128, 1, NORM><<<unsigned(blocks), APP_THREADS, 0, st>>>(p);
    else kv_append_kernel<D, 32, 2, NORM><<<unsigned(blocks), APP_THREADS, 0, st>>>(p);
  };
  auto pick = [&](auto dim) { n ? go(dim, std::true_type()) : go(dim, std::false_type()); };
  if (c.head_dim == 128) pick(std::integral_constant<int, 128>());
  else pick(std::integral_constant<int, 64>());
  return cuda_ok(cudaGetLastError(), who);
}

}  // namespace
}  // namespace tl

extern "C" tl_status tl_kv_append(const tl_kv_append_args* a, void* stream) {
  return tl::append("tl_kv_append", a, nullptr, stream);
}

extern "C" tl_status tl_kv_append_norm(const tl_kv_append_norm_args* a, void* stream) {
  return tl::append("tl_kv_append_norm", a ? &a->append : nullptr, a, stream);
}
