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
#include <algorithm>

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

// x c + t s rounded to odd (see above); not finite: the plain fp32 value.
__device__ __forceinline__ float dot2_odd(float x, float c, float t, float s) {
  const float p = __fmul_rn(x, c), r = __fmul_rn(t, s);
  const float pe = __fmaf_rn(x, c, -p), re = __fmaf_rn(t, s, -r);
  const float sum = __fadd_rn(p, r);
  const float back = __fsub_rn(sum, p);
  const float err = __fadd_rn(__fsub_rn(p, __fsub_rn(sum, back)), __fsub_rn(r, back));
  const float lo = __fadd_rn(err, __fadd_rn(pe, re));
  const float hi = __fadd_rn(sum, lo);
  const float rest = __fsub_rn(lo, __fsub_rn(hi, sum));
  // what is left below hi decides: one step towards zero where it points there, and the last bit set
  const uint32_t u = __float_as_uint(hi);
  const uint32_t odd = (u + uint32_t(int32_t(__float_as_uint(rest) ^ u) >> 31)) | 1u;
  const bool finite = (__float_as_uint(sum) & 0x7FFFFFFFu) < 0x7F800000u;
  return finite ? __uint_as_float(rest != 0.0f ? odd : u) : sum;
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

// Sixteen codes times f (a power of two <= 1), rounded to nearest even.
__device__ __forceinline__ uint4 recode16(uint4 w, float f) {
  uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = f16x2_to_f32x2(e4m3x2_to_f16x2(u[i])), b = f16x2_to_f32x2(e4m3x2_to_f16x2_hi(u[i]));
    u[i] = f32x2_to_e4m3x2(a.x * f, a.y * f) | (f32x2_to_e4m3x2(b.x * f, b.y * f) << 16);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// TEAM threads to one (page, head, keys or values); KEEP passes' rows stay in registers.
template <int D, int TEAM, int KEEP>
__global__ void __launch_bounds__(APP_THREADS, 8) kv_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int UNITS = D / 8;             // threads to a row
  constexpr int STEP = TEAM / UNITS;       // rows of one pass
  __shared__ uint32_t counts[4];
  __shared__ uint32_t team_max[4];
  const int tid = threadIdx.x;
  const KvBatch& b = p.b;
  const int ps = p.c.ps;

  if (int(blockIdx.x) >= p.kv_blocks) {
    // ---------------------------------------------------------------- one token's queries
    const int t = int(blockIdx.x) - p.kv_blocks;
    const uint32_t n = count_below(b, t, counts, [](int, int c0) { return c0; });
    const int s = n < kOutOfOrder ? int(n) - 1 : find_among_wrong<false>(b, ps, t).x;
    if (s < 0) return;
    const KvSeq seq = kv_seq(b, ps, s);
    if (t < seq.row0 || t >= seq.row0 + seq.q) return;
    const int pos = seq.len - seq.q + (t - seq.row0);
    if (p.rot > 0 && (pos < 0 || pos >= p.max_pos)) {
      if (tid == 0) record_error(b.status, kKvInvalid, uint32_t(s), uint32_t(pos), uint32_t(p.max_pos));
      return;
    }
    const uint16_t* row = p.q + int64_t(t) * p.q_ts;
    uint16_t* dst = p.q_out + int64_t(t) * p.H * D;
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
  if (page < 0 || page >= p.c.num_pages || (p.rot > 0 && hi > p.max_pos)) {
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
    if (values) load8(row + 8 * u, out);
    else rotated8<true>(p, row, u, lo + r, out);
  };
  auto take_max = [&](const float(&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t a = __float_as_uint(x[i]) & 0x7FFFFFFFu;
      if (a < 0x7F800000u) amax = max(amax, a);
    }
  };
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
  amax = __reduce_max_sync(0xffffffffu, amax);
  if (TEAM > 32) {
    if (lane_id() == 0) team_max[warp_id()] = amax;
    __syncthreads();
    amax = max(max(team_max[0], team_max[1]), max(team_max[2], team_max[3]));
  } else {
    __syncwarp();  // the scale is read by the whole team before one of it writes it
  }
  const int byte = max(old, scale_need(amax));
  const float inv = byte == 255 ? __uint_as_float(0x00200000u) : pow2f(127 - byte);  // 255: NaN it was and stays
  if (slot0 > 0 && byte > old) {
    const float f = pow2f(max(old - byte, -127));
    for (int i = member; i < slot0 * (D / 16); i += TEAM) {
      uint4* at = reinterpret_cast<uint4*>(codes + int64_t(i / (D / 16)) * p.c.token_stride + (i % (D / 16)) * 16);
      *at = recode16(*at, f);
    }
  }
  if (member == 0) *scale_at = uint8_t(byte);
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

extern "C" tl_status tl_kv_append(const tl_kv_append_args* a, void* stream) {
  using namespace tl;
  if (!a) return fail(TL_ERR_INVALID, "tl_kv_append: NULL args");
  if (a->n_tokens < 0 || a->B < 1 || a->B > (1 << 20) || a->max_pages < 1)
    return fail(TL_ERR_INVALID, "tl_kv_append: n_tokens %d, B %d, max_pages %d", a->n_tokens, a->B, a->max_pages);
  if (tl_status s = check_kv_cache("tl_kv_append", a->cache)) return s;
  const int D = a->cache.head_dim;
  if (a->H < 0 || a->H > 65536) return fail(TL_ERR_INVALID, "tl_kv_append: H %d", a->H);
  if (a->rot_dim < 0 || a->rot_dim > D || a->rot_dim % 16)
    return fail(TL_ERR_UNSUPPORTED, "tl_kv_append: rot_dim %d (a multiple of 16, 0..head_dim)", a->rot_dim);
  if (a->interleaved != 0 && a->interleaved != 1)
    return fail(TL_ERR_INVALID, "tl_kv_append: interleaved %d", a->interleaved);
  if (a->max_q_len < 0) return fail(TL_ERR_INVALID, "tl_kv_append: max_q_len %d", a->max_q_len);
  if (!a->cu_seqlens || !a->seq_lens || !a->page_table || !a->signals)
    return fail(TL_ERR_INVALID, "tl_kv_append: NULL pointer argument");
  if (a->n_tokens == 0) return TL_OK;
  if (!a->k || !a->v) return fail(TL_ERR_INVALID, "tl_kv_append: NULL pointer argument");
  if ((a->H > 0) != (a->q != nullptr) || (a->H > 0) != (a->q_out != nullptr))
    return fail(TL_ERR_INVALID, "tl_kv_append: q and q_out go with H > 0");
  if (a->rot_dim > 0 && (!a->cos || !a->sin || a->max_pos < 1))
    return fail(TL_ERR_INVALID, "tl_kv_append: rot_dim %d needs cos, sin and max_pos", a->rot_dim);
  for (const void* ptr : {a->k, a->v, a->q, (const void*)a->q_out, (const void*)a->cos, (const void*)a->sin})
    if (!aligned16(ptr)) return fail(TL_ERR_INVALID, "tl_kv_append: pointers must be 16-byte aligned");
  for (int64_t s : {a->k_token_stride, a->k_head_stride, a->v_token_stride, a->v_head_stride, a->q_token_stride,
                    a->q_head_stride})
    if (s < 0 || s % 8) return fail(TL_ERR_INVALID, "tl_kv_append: strides must be multiples of 8 elements");
  // A row's dims are read by the threads of both of a pair's units, with no order between them and the writes.
  if (a->H > 0 && rows_meet(a->q, a->q_token_stride * 2, (int64_t(a->H - 1) * a->q_head_stride + D) * 2, a->n_tokens,
                            a->q_out, int64_t(a->n_tokens) * a->H * D * 2))
    return fail(TL_ERR_INVALID, "tl_kv_append: q_out overlaps q");
  DeviceInfo di{};
  if (tl_status s = device_info(&di)) return s;
  if (a->signals->device != di.device)
    return fail(TL_ERR_INVALID, "tl_kv_append: signals belong to another device");

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
  const int per_seq = a->max_q_len ? std::min(a->max_q_len, a->n_tokens) : cdiv(a->n_tokens, a->B);
  // A whole block to a page's keys or values of one head where a page gets 32 rows, else a warp: 8192 tokens of 8 kv heads
  // of 128 into pages of 16, 32, 64 and 256 take 58, 54, 52 and 82 us with blocks, 54, 54, 75 and 211 us with warps.
  const bool wide = std::min(per_seq, c.page_size) >= 32;
  const int64_t items = int64_t(a->n_tokens) / c.page_size + 2 * int64_t(a->B);
  p.groups = wide ? 2 * c.H_kv : cdiv(2 * c.H_kv, APP_THREADS / 32);
  const int64_t blocks = items * p.groups + (a->H > 0 ? a->n_tokens : 0);
  if (blocks > 0x7FFFFFFFll) return fail(TL_ERR_UNSUPPORTED, "tl_kv_append: too many tokens");
  p.kv_blocks = int(items * p.groups);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (c.head_dim == 128) {
    if (wide) kv_append_kernel<128, 128, 1><<<unsigned(blocks), APP_THREADS, 0, st>>>(p);
    else kv_append_kernel<128, 32, 2><<<unsigned(blocks), APP_THREADS, 0, st>>>(p);
  } else {
    if (wide) kv_append_kernel<64, 128, 1><<<unsigned(blocks), APP_THREADS, 0, st>>>(p);
    else kv_append_kernel<64, 32, 2><<<unsigned(blocks), APP_THREADS, 0, st>>>(p);
  }
  return cuda_ok(cudaGetLastError(), "tl_kv_append launch");
}
