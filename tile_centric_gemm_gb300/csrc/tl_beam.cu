// tl_beam.cu -- beam search's selection: the N best continuations of a user's K beams.
//
//   score(k, v) = scores[k] + logits[k][v] - lse[k],   lse[k] = log sum_v exp(logits[k][v])
//
// equal scores by beam, then by logit (which 64 bits may not tell apart beside a large score), then by token.
//
// The logits are read once.  A row is cut into as many parts as fill the GPU with blocks; a block leaves its part's
// maximum, its sum of exponentials and its N largest values, and the block of a user that ends
// last joins the K rows.  (Within a row scores and logits rise together, so the N best of a
// user are among the rows' N largest, ties included.)
//
// The N largest of a part: any bound that N threads' own maxima reach is at or below the N-th
// largest value, and one that at most 2 N reach leaves few values to look at.  It is found
// by bisection, a vote of the block at each step.  Each thread has kept the maximum of each of its
// 16 values that it took at once; the few whose maximum reaches the bound are read again, and
// what reaches it goes to a list in shared memory, in which each value counts those before it.
// Where the bisection ends at a value that too many share, the values above it go to the list
// and the places left are filled with that value's lowest tokens.
//
// Beams are compared by 64-bit scores: the sums of exponentials are kept in pairs of fp32 and
// 64 bits, so that what decides between two beams is not lost beside scores of -20.
//
// Bound by memory for many beams and by latency for few.
#include <algorithm>
#include <cmath>

#include "tl_internal.h"
#include "tl_ptx.cuh"

namespace tl {
namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32;
constexpr int UNIT = 16;              // values that a thread takes at once
constexpr int STEP = THREADS * UNIT;  // and a block
constexpr int MOST_STEPS = 16;        // of a block, at least one
constexpr int BLOCKS = 608;           // that fill the GPU: four to an SM
constexpr int HITS = 1024;            // units that are looked at again, at most
constexpr float kSlack = 1.0f;        // by how much logits may pass a thread's reference: what came before a new one is e times less
constexpr float kLog2e = 1.4426950408889634f;
constexpr int MAX_BEAMS = 64, MAX_N = 64, MAX_B = 16384;
constexpr int NONE = int(0x80000000);

struct BeamParams {
  const void* logits;
  int64_t stride;  // of rows, in elements
  const float* scores;
  const uint8_t* done;
  int32_t* parents;
  int32_t* tokens;
  float* scores_out;
  uint8_t* done_out;
  float* lse;
  const int32_t* history;
  int32_t* history_out;
  uint32_t* counters;  // [B], zero between calls
  uint8_t* parts;      // [B K splits] parts of part_bytes
  int32_t B, K, N, V, eos, splits, part_bytes;
  int32_t steps, list;  // of a block at most; places of the list in shared memory
  int32_t history_stride, length;
};

// What a block leaves of its part of a row: this, then N values and their tokens, the largest first.
struct PartHead {
  float most;
  float pad;
  double sum;  // of exp(x - most)
};

// Floats as whole numbers in the same order (-0 is brought to 0 before).
__device__ __forceinline__ int ordered(float x) {
  const int b = __float_as_int(x);
  return b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float unordered(int o) { return __int_as_float(o ^ ((o >> 31) & 0x7FFFFFFF)); }
__device__ __forceinline__ int64_t ordered(double x) {
  const int64_t b = __double_as_longlong(x + 0.0);
  return b ^ ((b >> 63) & 0x7FFFFFFFFFFFFFFFll);
}

struct Smem {
  float warp_f[WARPS];
  int warp_lo[WARPS], warp_hi[WARPS];
  float2 warp_sum[WARPS];
  uint64_t warp_best[WARPS];
  int count, hits, last;
  double lse[MAX_BEAMS];    // by the joining block: infinity for a row that offers nothing, -infinity for an ended beam
  double score[MAX_BEAMS];  // its beam's
  int64_t best_key[WARPS];
  uint64_t best_tie[WARPS];
  uint32_t best_token[WARPS];
  int winner[MAX_N];  // its beam, or -1
};

// A bound on the threads' keys (NONE: a thread without) that at least n of them reach; and at most 2 n of them, unless
// exact: then fewer than n lie above it.  NONE + 1 where fewer than n threads have one.
__device__ __forceinline__ int bound(Smem& sm, int key, int n, bool& exact) {
  exact = false;
  int lo = __reduce_min_sync(0xffffffffu, key == NONE ? 0x7FFFFFFF : key), hi = __reduce_max_sync(0xffffffffu, key);
  if (lane_id() == 0) {
    sm.warp_lo[warp_id()] = lo;
    sm.warp_hi[warp_id()] = hi;
  }
  int have = __syncthreads_count(key != NONE);
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    lo = min(lo, sm.warp_lo[w]);
    hi = max(hi, sm.warp_hi[w]);
  }
  if (have < n) return NONE + 1;
  if (have <= 2 * n) return lo;
  while (lo < hi) {
    const uint32_t d = uint32_t(hi) - uint32_t(lo);
    const int mid = lo + int((d >> 1) + (d & 1u));
    have = __syncthreads_count(key >= mid);
    if (have >= n) {
      lo = mid;
      if (have <= 2 * n) return lo;
    } else {
      hi = mid - 1;
    }
  }
  exact = true;
  return lo;
}

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int W = 4;
  static __device__ __forceinline__ float one(const float* p) { return *p; }
  static __device__ __forceinline__ uint4 load(const float* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
  }
  static __device__ __forceinline__ void unpack(uint4 v, float* x) {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ void set(uint4& v, int c, float x) { (&v.x)[c] = __float_as_uint(x); }
};
template <>
struct Vec<uint16_t> {
  static constexpr int W = 8;
  static __device__ __forceinline__ float one(const uint16_t* p) { return __uint_as_float(uint32_t(*p) << 16); }
  static __device__ __forceinline__ uint4 load(const uint16_t* p) { return Vec<float>::load(reinterpret_cast<const float*>(p)); }
  static __device__ __forceinline__ void unpack(uint4 v, float* x) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ void set(uint4& v, int c, float x) {  // x is a bf16's value
    uint32_t& w = (&v.x)[c >> 1];
    const uint32_t h = __float_as_uint(x) >> 16;
    w = c & 1 ? (w & 0xFFFFu) | h << 16 : (w & 0xFFFF0000u) | h;
  }
};

// A row's vectors of 16 bytes: vector v holds the row's elements v W - skew .., aligned wherever the row begins;
// elements that are not the row's are -infinity.
template <typename T>
struct Row {
  static constexpr int W = Vec<T>::W;
  const T* first;
  int skew, V;
  __device__ __forceinline__ Row(const BeamParams& p, int row) {
    first = static_cast<const T*>(p.logits) + int64_t(row) * p.stride;
    skew = int((reinterpret_cast<uintptr_t>(first) & 15u) / sizeof(T));
    V = p.V;
  }
  __device__ __forceinline__ int token(int v, int c) const { return v * W - skew + c; }
  __device__ __forceinline__ uint4 load(int v, bool in) const {
    const int e = v * W - skew;
    if (in && e >= 0 && e + W <= V) return Vec<T>::load(first + e);
    uint4 r;
#pragma unroll
    for (int c = 0; c < W; ++c) Vec<T>::set(r, c, in && e + c >= 0 && e + c < V ? Vec<T>::one(first + e + c) : -INFINITY);
    return r;
  }
};

// Larger values first, then lower tokens, as one number; 0 is below all.
__device__ __forceinline__ uint64_t value_key(float x, int token) {
  return uint64_t(uint32_t(ordered(x + 0.0f)) ^ 0x80000000u) << 32 | uint32_t(~token);
}
__device__ __forceinline__ float2 value_of(uint64_t key) {
  return make_float2(unordered(int(uint32_t(key >> 32) ^ 0x80000000u)), __int_as_float(int(~uint32_t(key))));
}

// The N largest one after the other, by reading the part N times: where more reach the bound than there is room for.
template <typename T>
__device__ __noinline__ void take_one_by_one(const BeamParams& p, Smem& sm, int row, int v0, int v1, float2* out) {
  const Row<T> r(p, row);
  constexpr int W = Row<T>::W;
  uint64_t last = ~0ull;
  for (int i = 0; i < p.N; ++i) {
    uint64_t best = 0;
    if (last) {
      for (int v = v0 + int(threadIdx.x); v < v1; v += THREADS) {
        float x[W];
        Vec<T>::unpack(r.load(v, true), x);
#pragma unroll
        for (int c = 0; c < W; ++c) {
          const uint64_t key = value_key(x[c], r.token(v, c));
          if (x[c] > -INFINITY && key < last && key > best) best = key;
        }
      }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) best = max(best, uint64_t(__shfl_xor_sync(0xffffffffu, best, d)));
    __syncthreads();
    if (lane_id() == 0) sm.warp_best[warp_id()] = best;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WARPS; ++w) best = max(best, sm.warp_best[w]);
    if (threadIdx.x == 0) __stcg(out + i, best ? value_of(best) : make_float2(-INFINITY, 0.0f));
    last = best;
  }
}

// One block's part of a row: its sum and its N largest to `part`.
template <typename T>
__device__ __forceinline__ void take_part(const BeamParams& p, Smem& sm, uint64_t* list, int row, int split, uint8_t* part) {
  constexpr int W = Vec<T>::W, VECS = UNIT / W;
  const int tid = threadIdx.x, lane = int(lane_id()), warp = int(warp_id());
  int* hit = reinterpret_cast<int*>(list + p.list);
  float* unit_most = reinterpret_cast<float*>(hit + HITS);  // [steps][threads]
  const Row<T> r(p, row);
  const int vecs = (p.V + r.skew + W - 1) / W, per = (vecs + p.splits - 1) / p.splits;
  const int v0 = split * per, v1 = min(vecs, v0 + per);
  const int steps = max(1, (v1 - v0 + THREADS * VECS - 1) / (THREADS * VECS));
  auto vec = [&](int unit, int i) { return v0 + ((unit / THREADS) * VECS + i) * THREADS + unit % THREADS; };

  // ---------------------------------------------------------------- maxima, and sums of exponentials
  // A thread's sum is relative to its reference m, which follows its maximum at a distance.
  uint4 next[VECS];
  float most = -INFINITY, m = -INFINITY, hi = 0.0f, lo = 0.0f;
#pragma unroll
  for (int i = 0; i < VECS; ++i) next[i] = r.load(vec(tid, i), vec(tid, i) < v1);
  for (int b = 0; b < steps; ++b) {
    float x[UNIT];
#pragma unroll
    for (int i = 0; i < VECS; ++i) Vec<T>::unpack(next[i], x + i * W);
    if (b + 1 < steps) {
#pragma unroll
      for (int i = 0; i < VECS; ++i) next[i] = r.load(vec((b + 1) * THREADS + tid, i), vec((b + 1) * THREADS + tid, i) < v1);
    }
    float top = x[0];
#pragma unroll
    for (int i = 1; i < UNIT; ++i) top = fmaxf(top, x[i]);
    if (!(top >= -INFINITY)) top = -INFINITY;  // nothing but NaN
    unit_most[b * THREADS + tid] = top;
    most = fmaxf(most, top);
    if (top > m + kSlack) {
      const float f = ex2_approx((m - top) * kLog2e);
      hi *= f;
      lo *= f;
      m = top;
    }
    const float base = m == -INFINITY ? 0.0f : m;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < UNIT; ++i) s[i & 3] += ex2_approx((x[i] - base) * kLog2e);
    const float add = (s[0] + s[1]) + (s[2] + s[3]), sum = __fadd_rn(hi, add), back = __fsub_rn(sum, hi);
    lo += __fadd_rn(__fsub_rn(hi, __fsub_rn(sum, back)), __fsub_rn(add, back));
    hi = sum;
  }
  most += 0.0f;
  bool exact;
  const int cut = bound(sm, most > -INFINITY ? ordered(most) : NONE, p.N, exact);
  int top = NONE;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) top = max(top, sm.warp_hi[w]);
  const float block_most = top == NONE ? -INFINITY : unordered(top);
  const float least = cut == NONE + 1 ? -3.402823466e38f : unordered(cut);
  if (tid == 0) sm.count = sm.hits = 0;
  {
    // the block's sum, relative to its maximum
    const float f = block_most == -INFINITY ? 1.0f : ex2_approx((m - block_most) * kLog2e);
    hi *= f;
    lo *= f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const float h2 = __shfl_xor_sync(0xffffffffu, hi, d), l2 = __shfl_xor_sync(0xffffffffu, lo, d);
      const float sum = __fadd_rn(hi, h2), back = __fsub_rn(sum, hi);
      lo = (lo + l2) + __fadd_rn(__fsub_rn(hi, __fsub_rn(sum, back)), __fsub_rn(h2, back));
      hi = sum;
    }
    if (lane == 0) sm.warp_sum[warp] = make_float2(hi, lo);
  }
  __syncthreads();

  // ---------------------------------------------------------------- what reaches the bound
  if (most > -INFINITY && (exact ? most > least : most >= least)) {
    for (int b = 0; b < steps; ++b) {
      const float u = unit_most[b * THREADS + tid];
      if (exact ? u > least : u >= least) {
        const int at = atomicAdd(&sm.hits, 1);
        if (at < HITS) hit[at] = b * THREADS + tid;
      }
    }
  }
  __syncthreads();
  const int hits = sm.hits;
  float2* out = reinterpret_cast<float2*>(part + sizeof(PartHead));
  bool many = hits > HITS;
  if (!many) {
    for (int h = tid; h < hits * VECS; h += THREADS) {
      const int v = vec(hit[h / VECS], h % VECS);
      float x[W];
      Vec<T>::unpack(r.load(v, v < v1), x);
#pragma unroll
      for (int c = 0; c < W; ++c)
        if (x[c] > -INFINITY && (exact ? x[c] > least : x[c] >= least)) {
          const int at = atomicAdd(&sm.count, 1);
          if (at < p.list) list[at] = value_key(x[c], r.token(v, c));
        }
    }
    __syncthreads();
    many = sm.count > p.list - p.N;
  }
  if (many) {
    take_one_by_one<T>(p, sm, row, v0, v1, out);
  } else {
    if (exact && sm.count < p.N) {
      // that value's lowest tokens
      int at = sm.count;
      __syncthreads();
      for (int b = 0; b < steps && at < p.N; ++b) {
        if (!__syncthreads_or(unit_most[b * THREADS + tid] >= least)) continue;
        for (int i = 0; i < VECS && at < p.N; ++i) {
          const int v = vec(b * THREADS + tid, i);
          float x[W];
          Vec<T>::unpack(r.load(v, v < v1), x);
          int mine = 0;
#pragma unroll
          for (int c = 0; c < W; ++c) mine += x[c] == least;
          int before = mine;
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, before, d);
            if (lane >= d) before += y;
          }
          if (lane == 31) sm.warp_lo[warp] = before;
          __syncthreads();
          int all = 0;
          before += at - mine;
#pragma unroll
          for (int w = 0; w < WARPS; ++w) {
            if (w < warp) before += sm.warp_lo[w];
            all += sm.warp_lo[w];
          }
#pragma unroll
          for (int c = 0; c < W; ++c)
            if (x[c] == least) {
              if (before < p.N) list[before] = value_key(least, r.token(v, c));
              ++before;
            }
          at = min(at + all, p.N);
          __syncthreads();
        }
      }
      if (tid == 0) sm.count = at;
      __syncthreads();
    }
    // ---------------------------------------------------------------- the N largest, in order: eight lanes to a value
    const int n = sm.count;
    for (int e0 = 0; e0 < n; e0 += THREADS / 8) {
      const int e = e0 + tid / 8;
      const uint64_t mine = list[min(e, n - 1)];
      int rank = 0;
      for (int k = tid % 8; k < n; k += 8) rank += list[k] > mine;
      rank += __shfl_xor_sync(0xffffffffu, rank, 1);
      rank += __shfl_xor_sync(0xffffffffu, rank, 2);
      rank += __shfl_xor_sync(0xffffffffu, rank, 4);
      if (e < n && tid % 8 == 0 && rank < p.N) __stcg(out + rank, value_of(mine));
    }
    for (int e = n + tid; e < p.N; e += THREADS) __stcg(out + e, make_float2(-INFINITY, 0.0f));
  }
  bool nan = false;
  if (block_most == INFINITY) {  // the sum came to nothing: is there a NaN too?
    for (int v = v0 + tid; v < v1; v += THREADS) {
      float x[W];
      Vec<T>::unpack(r.load(v, true), x);
#pragma unroll
      for (int c = 0; c < W; ++c) nan |= !(x[c] == x[c]);
    }
    nan = __syncthreads_or(nan);
  }
  if (tid == 0) {
    double sum = 0.0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) sum += double(sm.warp_sum[w].x) + double(sm.warp_sum[w].y);
    if (block_most == INFINITY) sum = nan ? __longlong_as_double(0x7FF8000000000000ll) : 1.0;
    __stcg(reinterpret_cast<float*>(part), block_most);
    __stcg(reinterpret_cast<double*>(part) + 1, sum);
  }
}

// The candidates of a user: slot j is candidate j % N of part j / N, or behind the parts' slots an ended beam's only one.
struct Candidate {
  int64_t key;     // the score's; larger is better
  uint64_t tie;    // beam, then logit; smaller is better
  uint32_t token;  // smaller is better
  bool any;
};
__device__ __forceinline__ bool before(int64_t key, uint64_t tie, uint32_t token, int64_t key2, uint64_t tie2, uint32_t token2) {
  return key > key2 || (key == key2 && (tie < tie2 || (tie == tie2 && token < token2)));
}
__device__ __forceinline__ float2 candidate_value(const BeamParams& p, int user, int j) {
  if (j >= p.K * p.splits * p.N) return make_float2(0.0f, 0.0f);
  const int part = j / p.N;
  return __ldcg(reinterpret_cast<const float2*>(p.parts + (int64_t(user) * p.K * p.splits + part) * p.part_bytes + sizeof(PartHead)) +
                (j - part * p.N));
}
__device__ __forceinline__ Candidate candidate(const BeamParams& p, const Smem& sm, int user, int j, float2 v) {
  const int slots = p.K * p.splits * p.N;
  Candidate c;
  double s = -INFINITY;
  if (j >= slots) {
    const int k = j - slots;
    c.token = uint32_t(p.eos);
    c.tie = uint64_t(k) << 32;
    if (sm.lse[k] == -INFINITY) s = sm.score[k];
  } else {
    const int k = j / (p.N * p.splits);
    c.token = uint32_t(__float_as_int(v.y));
    c.tie = uint64_t(k) << 32 | uint32_t(~(uint32_t(ordered(v.x)) ^ 0x80000000u));
    if (v.x > -INFINITY && fabs(sm.lse[k]) < INFINITY) s = sm.score[k] + (double(v.x) - sm.lse[k]);
  }
  c.any = fabs(s) < INFINITY;  // (not for NaN either)
  c.key = ordered(s);
  return c;
}

// The last block of a user: its beams' sums, and the N best of their candidates.
__device__ __noinline__ void join(const BeamParams& p, Smem& sm, uint64_t* list, int user) {
  const int tid = threadIdx.x, lane = int(lane_id()), warp = int(warp_id());
  // a thread's first candidates are on their way while the sums are taken together
  constexpr int AHEAD = 4;
  const int slots = p.K * p.splits * p.N + (p.done ? p.K : 0);
  float2 ahead[AHEAD];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) ahead[i] = tid + i * THREADS < slots ? candidate_value(p, user, tid + i * THREADS) : make_float2(-INFINITY, 0.0f);
  auto each = [&](auto f) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (tid + i * THREADS < slots) f(candidate(p, sm, user, tid + i * THREADS, ahead[i]));
    for (int j = tid + AHEAD * THREADS; j < slots; j += THREADS) f(candidate(p, sm, user, j, candidate_value(p, user, j)));
  };
  // a row's parts to 2^n lanes, several rows to a warp: 64-bit arithmetic takes as long for one lane as for 32
  int seg = 1;
  while (seg < min(p.splits, 32)) seg *= 2;
  for (int k0 = warp * (32 / seg); k0 < p.K; k0 += WARPS * (32 / seg)) {
    const int k = k0 + lane / seg;
    const bool row = k < p.K, ended = row && p.done && p.done[user * p.K + k];
    const uint8_t* parts = p.parts + int64_t(user * p.K + min(k, p.K - 1)) * p.splits * p.part_bytes;
    float most = -INFINITY;
    double sum = 0.0;
    for (int i0 = 0; i0 < p.splits; i0 += seg) {
      const int i = i0 + lane % seg;
      float m = -INFINITY;
      double s = 0.0;
      if (i < p.splits && row && !ended) {
        m = __ldcg(reinterpret_cast<const float*>(parts + int64_t(i) * p.part_bytes));
        s = __ldcg(reinterpret_cast<const double*>(parts + int64_t(i) * p.part_bytes) + 1);
      }
      float top = fmaxf(most, m);
      for (int d = seg / 2; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      if (m != top && m > -INFINITY) s *= exp(double(m) - double(top));
      if (most != top && most > -INFINITY) sum *= exp(double(most) - double(top));
      most = top;
      for (int d = seg / 2; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      sum += s;
    }
    if (row && lane % seg == 0) {
      const double lse = ended ? 0.0 : double(most) + log(sum);
      // a row of -infinity, or with +infinity or NaN, offers nothing
      sm.lse[k] = ended ? -INFINITY : fabs(lse) < INFINITY ? lse : INFINITY;
      sm.score[k] = double(p.scores[user * p.K + k]);
      if (p.lse) p.lse[user * p.K + k] = float(lse);
    }
  }
  if (tid == 0) sm.count = 0;
  __syncthreads();
  int best = NONE;
  each([&](const Candidate& c) {
    if (c.any) best = max(best, int(c.key >> 32));
  });
  bool exact;
  const int cut = bound(sm, best, p.N, exact);
  int64_t* keys = reinterpret_cast<int64_t*>(list);
  const int places = p.list * 8 / 20;
  uint64_t* ties = reinterpret_cast<uint64_t*>(keys + places);
  uint32_t* tokens = reinterpret_cast<uint32_t*>(ties + places);
  if (best != NONE && best >= cut) {
    each([&](const Candidate& c) {
      if (c.any && int(c.key >> 32) >= cut) {
        const int at = atomicAdd(&sm.count, 1);
        if (at < places) {
          keys[at] = c.key;
          ties[at] = c.tie;
          tokens[at] = c.token;
        }
      }
    });
  }
  for (int i = tid; i < p.N; i += THREADS) sm.winner[i] = -1;
  __syncthreads();
  const int n = sm.count;
  auto win = [&](int rank, int64_t key, int k, int t) {
    const double s = __longlong_as_double(key ^ ((key >> 63) & 0x7FFFFFFFFFFFFFFFll));
    const int64_t o = int64_t(user) * p.N + rank;
    sm.winner[rank] = k;
    p.parents[o] = user * p.K + k;
    p.tokens[o] = t;
    p.scores_out[o] = float(s);
    if (p.done_out) p.done_out[o] = sm.lse[k] == -INFINITY || t == p.eos;
    if (p.history) p.history_out[o * p.history_stride + p.length] = t;
  };
  if (n <= places) {
    for (int e0 = 0; e0 < n; e0 += THREADS / 8) {
      const int e = e0 + tid / 8, at = min(e, n - 1);
      const int64_t key = keys[at];
      const uint64_t tie = ties[at];
      const uint32_t t = tokens[at];
      int rank = 0;
      for (int k = tid % 8; k < n; k += 8) rank += before(keys[k], ties[k], tokens[k], key, tie, t);
      rank += __shfl_xor_sync(0xffffffffu, rank, 1);
      rank += __shfl_xor_sync(0xffffffffu, rank, 2);
      rank += __shfl_xor_sync(0xffffffffu, rank, 4);
      if (e < n && tid % 8 == 0 && rank < p.N) win(rank, key, int(tie >> 32), int(t));
    }
  } else {
    // more scores next to one another than the list holds: the best, one after the other
    int64_t last_key = 0x7FFFFFFFFFFFFFFFll;  // (no score has it)
    uint64_t last_tie = 0;
    uint32_t last_token = 0;
    constexpr uint32_t NO_TOKEN = 0xFFFFFFFFu;
    for (int r = 0; r < p.N; ++r) {
      int64_t key = int64_t(0x8000000000000000ull);
      uint64_t tie = ~0ull;
      uint32_t t = NO_TOKEN;
      each([&](const Candidate& c) {
        if (c.any && before(last_key, last_tie, last_token, c.key, c.tie, c.token) && before(c.key, c.tie, c.token, key, tie, t)) {
          key = c.key;
          tie = c.tie;
          t = c.token;
        }
      });
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) {
        const int64_t key2 = __shfl_xor_sync(0xffffffffu, key, d);
        const uint64_t tie2 = __shfl_xor_sync(0xffffffffu, tie, d);
        const uint32_t t2 = __shfl_xor_sync(0xffffffffu, t, d);
        if (before(key2, tie2, t2, key, tie, t)) {
          key = key2;
          tie = tie2;
          t = t2;
        }
      }
      if (lane == 0) {
        sm.best_key[warp] = key;
        sm.best_tie[warp] = tie;
        sm.best_token[warp] = t;
      }
      __syncthreads();
      for (int w = 0; w < WARPS; ++w)
        if (before(sm.best_key[w], sm.best_tie[w], sm.best_token[w], key, tie, t)) {
          key = sm.best_key[w];
          tie = sm.best_tie[w];
          t = sm.best_token[w];
        }
      __syncthreads();
      if (t == NO_TOKEN) break;
      if (tid == 0) win(r, key, int(tie >> 32), int(t));
      last_key = key;
      last_tie = tie;
      last_token = t;
    }
  }
  __syncthreads();
  for (int i = tid; i < p.N; i += THREADS) {
    if (sm.winner[i] >= 0) continue;
    const int64_t o = int64_t(user) * p.N + i;
    p.parents[o] = p.tokens[o] = -1;
    p.scores_out[o] = -INFINITY;
    if (p.done_out) p.done_out[o] = 1;
  }
  if (!p.history) return;
  for (int i = 0; i < p.N; ++i) {
    if (sm.winner[i] < 0) continue;
    const int32_t* from = p.history + int64_t(user * p.K + sm.winner[i]) * p.history_stride;
    int32_t* to = p.history_out + (int64_t(user) * p.N + i) * p.history_stride;
    for (int t = tid; t < p.length; t += THREADS) to[t] = from[t];
  }
}

template <typename T>
__global__ void __launch_bounds__(THREADS, 4) beam_kernel(const __grid_constant__ BeamParams p) {
  extern __shared__ __align__(16) uint64_t list[];
  __shared__ Smem sm;
  const int row = int(blockIdx.x) / p.splits, split = int(blockIdx.x) - row * p.splits, user = row / p.K;
  if (!(p.done && p.done[row])) take_part<T>(p, sm, list, row, split, p.parts + int64_t(blockIdx.x) * p.part_bytes);
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    sm.last = atomicAdd(p.counters + user, 1u) == uint32_t(p.K * p.splits - 1);
    if (sm.last) p.counters[user] = 0;
  }
  __syncthreads();
  if (!sm.last) return;
  __threadfence();
  join(p, sm, list, user);
}

constexpr size_t kCounters = size_t(MAX_B) * 4;  // in a place that does not depend on the sizes
// Parts of a row: as many as fill the GPU, of 4096 elements at least and 65536 at most.  (7: elements that a row may begin
// behind 16 bytes.)
int least_splits(int V) { return int((int64_t(V) + 7 + MOST_STEPS * STEP - 1) / (MOST_STEPS * STEP)); }
int split_count(int64_t rows, int V) {
  const int most = int((int64_t(V) + 7 + STEP - 1) / STEP);
  return std::max(least_splits(V), std::min(std::min(most, 32), int((BLOCKS + rows - 1) / rows)));
}
int part_bytes(int N) { return int(sizeof(PartHead)) + N * 8; }
int list_places(int N) { return std::max(256, 32 * N); }

bool meet(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + uintptr_t(nb) && y < x + uintptr_t(na);
}

}  // namespace
}  // namespace tl

extern "C" size_t tl_beam_select_workspace_size(int B, int K, int N, int V) {
  using namespace tl;
  if (B < 1 || B > MAX_B || K < 1 || K > MAX_BEAMS || N < 1 || N > MAX_N || V < 1 || int64_t(K) * V > 0x7FFFFFFF) return 0;
  // (rows times their parts never fall as rows grow, with BLOCKS beside them)
  return kCounters + (size_t(B) * K * least_splits(V) + BLOCKS) * part_bytes(N);
}

extern "C" tl_status tl_beam_select(const tl_beam_select_args* a, void* stream) {
  using namespace tl;
  const char* who = "tl_beam_select";
  if (!a) return fail(TL_ERR_INVALID, "%s: NULL args", who);
  if (a->B < 0 || a->K < 1 || a->N < 1 || a->V < 1)
    return fail(TL_ERR_INVALID, "%s: B %d, K %d, N %d, V %d", who, a->B, a->K, a->N, a->V);
  if (a->B > MAX_B || a->K > MAX_BEAMS || a->N > MAX_N || int64_t(a->K) * a->V > 0x7FFFFFFF)
    return fail(TL_ERR_UNSUPPORTED, "%s: B %d (at most 16384), K %d, N %d (64 each), K * V below 2^31", who, a->B, a->K, a->N);
  if (a->dtype != 0 && a->dtype != 1) return fail(TL_ERR_INVALID, "%s: dtype %d", who, a->dtype);
  if (a->row_stride < a->V) return fail(TL_ERR_INVALID, "%s: row_stride below V", who);
  if (a->eos < -1 || a->eos >= a->V || (a->done && a->eos < 0))
    return fail(TL_ERR_INVALID, "%s: eos %d (-1 for none, which ended beams need not be)", who, a->eos);
  if (a->B == 0) return TL_OK;
  if (!a->logits || !a->scores || !a->parents || !a->tokens || !a->scores_out || !a->workspace)
    return fail(TL_ERR_INVALID, "%s: NULL pointer argument", who);
  if ((reinterpret_cast<uintptr_t>(a->logits) & (a->dtype ? 1u : 3u)) || !aligned16(a->workspace))
    return fail(TL_ERR_INVALID, "%s: logits must be aligned to their type, the workspace to 16 bytes", who);
  const size_t need = tl_beam_select_workspace_size(a->B, a->K, a->N, a->V);
  if (a->workspace_bytes < need) return fail(TL_ERR_INVALID, "%s: workspace of %zu bytes, need %zu", who, a->workspace_bytes, need);
  const int64_t in = int64_t(a->B) * a->K, out = int64_t(a->B) * a->N;
  if (meet(a->scores, in * 4, a->scores_out, out * 4) || (a->done && a->done_out && meet(a->done, in, a->done_out, out)))
    return fail(TL_ERR_INVALID, "%s: scores_out or done_out overlaps what it is made from", who);
  if ((a->history != nullptr) != (a->history_out != nullptr))
    return fail(TL_ERR_INVALID, "%s: history and history_out go together", who);
  if (a->history) {
    if (a->length < 0 || a->length >= a->history_stride)
      return fail(TL_ERR_INVALID, "%s: length %d, history rows of %d", who, a->length, a->history_stride);
    if (meet(a->history, in * a->history_stride * 4, a->history_out, out * a->history_stride * 4))
      return fail(TL_ERR_INVALID, "%s: history_out overlaps history", who);
  }
  BeamParams p{};
  p.logits = a->logits;
  p.stride = a->row_stride;
  p.scores = a->scores;
  p.done = a->done;
  p.parents = a->parents;
  p.tokens = a->tokens;
  p.scores_out = a->scores_out;
  p.done_out = a->done_out;
  p.lse = a->lse;
  p.history = a->history;
  p.history_out = a->history_out;
  p.history_stride = a->history_stride;
  p.length = a->length;
  p.counters = static_cast<uint32_t*>(a->workspace);
  p.parts = static_cast<uint8_t*>(a->workspace) + kCounters;
  p.B = a->B;
  p.K = a->K;
  p.N = a->N;
  p.V = a->V;
  p.eos = a->eos;
  p.splits = split_count(in, a->V);
  p.part_bytes = part_bytes(a->N);
  p.list = list_places(a->N);
  p.steps = cdiv(cdiv(a->V + 7 + 7, a->dtype ? 8 : 4), p.splits);            // vectors of a part,
  p.steps = std::max(1, cdiv(p.steps, STEP / (a->dtype ? 8 : 4)));           // and its steps
  const size_t smem = size_t(p.list) * 8 + HITS * 4 + size_t(p.steps) * THREADS * 4;
  const int64_t blocks = in * p.splits;
  if (blocks > 0x7FFFFFFF) return fail(TL_ERR_UNSUPPORTED, "%s: too many rows", who);
  void* args[] = {&p};
  const void* kernel = a->dtype ? reinterpret_cast<const void*>(&beam_kernel<uint16_t>) : reinterpret_cast<const void*>(&beam_kernel<float>);
  return launch(kernel, int(blocks), THREADS, smem, static_cast<cudaStream_t>(stream), args, false);
}
