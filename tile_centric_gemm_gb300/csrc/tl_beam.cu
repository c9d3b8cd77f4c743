// tl_beam.cu -- beam search's selection: the N best continuations of a user's K beams.
//
//   score(k, v) = scores[k] + logits[k][v] - lse[k],   lse[k] = log sum_v exp(logits[k][v])
//
// equal scores by beam, then by logit (which scores may not tell apart beside a large sum), then by token.
//
// The logits are read once, as a stream: a row is cut into as many parts as fill the GPU with
// blocks, a thread takes 16 logits at a time, and what a block leaves is its part's sum of
// exponentials and the maximum of each group of up to 256 logits that 16 neighbouring threads took in a step.  The block of a
// user that ends last joins the K rows: the groups' maxima are scores themselves, so any bound
// that N of them reach is at or below the N-th best score.  A bound that few groups reach is found
// from the threads' best ones (256 bins between the least and the largest, then bisection by the
// block's votes), those groups are read again, and what reaches the bound goes to a list in shared
// memory, in which each candidate counts those before it.  (With the selection in each part
// instead, 512 beams of 50001 took 31 us: a block's list cost it as much time as its logits.)
// Where more reach the bound than the list holds (plateaus), rows are taken apart value by value.
//
// Beams are compared by scores in pairs of fp32 (48 bits), and a row's sum of exponentials is joined in pairs
// too, so that joining and comparing add nothing to what the exponentials themselves are off by (2^-22 each, which is
// what lse is good to where a few logits make up the sum).  (64-bit arithmetic took 5000
// of the joining block's cycles: a warp's instruction holds its unit for 16.)
//
// Bound by memory for many beams and by latency for few.  512 beams of 50001 in fp32, a sixth of them ended, 16
// continuations to each 8: 26.8 us in a graph for 86 MB; the stream alone takes 18.2 (4.7 TB/s, 70 % of a copy's rate),
// with three blocks on some SMs and four on others, the users' joins 8.6 behind it, one block to each.  (Smaller parts, so
// that users end one after the other and joins run beside the stream, took 2.5 us more with 2 of them to a row, 6.6 with 3.)
// 4 beams of 32000 in bf16: 9.5 us, 6.3 of them the join, a chain of some 12,000 cycles: the sums 3,500 to 4,000 (with the
// first loads), the threads' best groups 2,000, the bound 1,300, the list of groups 2,300, reading them again 2,100, the
// ranks 1,900.
#include <algorithm>
#include <cmath>

#include "tl_internal.h"
#include "tl_ptx.cuh"

namespace tl {
namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32;
constexpr int UNIT = 16;              // logits that a thread takes at once
constexpr int STEP = THREADS * UNIT;  // and a block
constexpr int GROUP = 16;             // neighbouring threads whose maximum of a step is kept
constexpr int LINE = THREADS / GROUP; // maxima of a block's step
constexpr int MOST_STEPS = 16;        // of a block, at least one
constexpr int BLOCKS = 304;           // wanted: two to an SM at least, all at once (four fit)
constexpr int HITS = 512;             // groups that are looked at again, at most
constexpr int AHEAD = 8;              // groups of a thread that stay in registers
constexpr float kFar = 32768.0f;      // references of sums are whole powers of two up to 2^kFar
constexpr float kLog2e = 1.4426950216f, kLog2eLow = 1.9259629e-08f;
constexpr int MAX_BEAMS = 64, MAX_N = 64, MAX_B = 16384;
constexpr int64_t MAX_LOGITS = int64_t(1) << 30;  // of a user: places in a row, a step or two behind its end too, stay within 32 bits
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
  float4* heads;       // [B K splits] of a part: reference (-infinity, infinity: of nothing but that) and sum of exp(x - reference)
  float* maxima;       // [B K splits][lines][LINE]
  int32_t B, K, N, V, eos, splits, lines;  // lines: of a part, its steps
  int32_t per;         // elements of a part
  int32_t list;                                         // places of the list in shared memory
  int32_t history_stride, length;
};

// Floats as whole numbers in the same order (-0 is brought to 0 before).
__device__ __forceinline__ int ordered(float x) {
  const int b = __float_as_int(x);
  return b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float unordered(int o) { return __int_as_float(o ^ ((o >> 31) & 0x7FFFFFFF)); }

// ---------------------------------------------------------------- pairs: x + y, y below half a step of x
__device__ __forceinline__ float2 normal(float hi, float lo) {  // |hi| >= |lo|, or nearly
  const float sum = __fadd_rn(hi, lo);
  return make_float2(sum, __fsub_rn(lo, __fsub_rn(sum, hi)));
}
__device__ __forceinline__ float2 operator+(float2 a, float2 b) {
  const float2 s = two_sum(a.x, b.x);
  return normal(s.x, s.y + (a.y + b.y));
}
__device__ __forceinline__ float2 operator*(float2 a, float2 b) {
  const float p = __fmul_rn(a.x, b.x);
  return normal(p, fmaf(a.x, b.y, fmaf(a.y, b.x, __fmaf_rn(a.x, b.x, -p))));
}
// exp(a - b) for a <= b, to about 2^-25: 2^n (1 + u), u the series of exp(f ln 2) - 1 for |f| <= 1/2.
__device__ __noinline__ float2 exp_below(float2 a, float2 b) {
  if (!(a.x - b.x > -80.0f)) return make_float2(0.0f, 0.0f);  // (infinities, too)
  const float2 d = a + make_float2(-b.x, -b.y);
  const float t = __fmul_rn(d.x, kLog2e);
  const float rest = fmaf(d.x, kLog2eLow, fmaf(d.y, kLog2e, __fmaf_rn(d.x, kLog2e, -t)));
  const float n = rintf(t), y = ((t - n) + rest) * 0.69314718056f;
  float u = 1.0f / 362880;
  u = fmaf(u, y, 1.0f / 40320);
  u = fmaf(u, y, 1.0f / 5040);
  u = fmaf(u, y, 1.0f / 720);
  u = fmaf(u, y, 1.0f / 120);
  u = fmaf(u, y, 1.0f / 24);
  u = fmaf(u, y, 1.0f / 6);
  u = fmaf(u, y, 0.5f);
  const float2 r = two_sum(1.0f, fmaf(u * y, y, y));
  const float scale = __int_as_float((int(n) + 127) << 23);  // n >= -116
  return make_float2(r.x * scale, r.y * scale);
}
// log(s) for s > 0, finite: s = 2^e f, sqrt(1/2) <= f <= sqrt(2), and log f = 2 atanh(z), z = (f - 1) / (f + 1), by its series.
__device__ __forceinline__ float2 log_of(float2 s) {
  int e = int(__float_as_uint(s.x) >> 23) - 127;
  float scale = __int_as_float((127 - e) << 23);
  if (s.x * scale > 1.4142135f) {
    ++e;
    scale *= 0.5f;
  }
  const float f = s.x * scale, low = s.y * scale, up = f - 1.0f;
  const float2 den = two_sum(f, 1.0f);
  const float z = __fdividef(up, den.x);  // (what it is off by goes to z1)
  const float z1 = __fdividef(__fmaf_rn(-z, den.x, up) + (low - z * (den.y + low)), den.x);
  const float w = z * z;
  float p = 2.0f / 13;
  p = fmaf(p, w, 2.0f / 11);
  p = fmaf(p, w, 2.0f / 9);
  p = fmaf(p, w, 2.0f / 7);
  p = fmaf(p, w, 2.0f / 5);
  p = fmaf(p, w, 2.0f / 3);
  // ln 2 in two parts, the first of 14 bits: exact times e
  return two_sum(float(e) * 0x1.62ep-1f, 2.0f * z) + make_float2(fmaf(float(e), 3.194618e-05f, fmaf(p * w, z, 2.0f * z1)), 0.0f);
}
// Pairs as whole numbers in the same order.
__device__ __forceinline__ int64_t ordered(float2 x) {
  return int64_t(ordered(x.x + 0.0f)) << 32 | (uint32_t(ordered(x.y + 0.0f)) ^ 0x80000000u);
}

// Two at a time: (x, y) = (a, b) f + c; (x, y) += (a, b).
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
__device__ __forceinline__ float ex2_ftz(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// 2^d for whole d <= 0
__device__ __forceinline__ float pow2_below(float d) { return d < -126.0f ? 0.0f : __int_as_float((int(d) + 127) << 23); }

struct Smem {
  int warp_lo[WARPS], warp_hi[WARPS];
  float2 warp_sum[WARPS];
  float warp_most[WARPS];
  int count, hits, last;
  int bins[THREADS];
  float2 lse[MAX_BEAMS];   // by the joining block: infinity for a row that offers nothing, -infinity for an ended beam
  float score[MAX_BEAMS];  // its beam's
  float bias[MAX_BEAMS];   // score - lse in fp32, -infinity for rows that offer nothing
  float next[MAX_BEAMS];   // row by row: the largest logit not taken yet
  int winner[MAX_N];       // its beam, or -1
};

// A bound on the threads' keys (NONE: a thread without) that at least n of them reach; and at most 2 n of them, unless
// exact: then fewer than n lie above it.  NONE + 1 where fewer than n threads have one.  sm.bins is 0 before.
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
  // 256 bins between the least and the largest; the highest ones that hold n, found by every warp
  const int shift = max(0, 24 - __clz(int(uint32_t(hi) - uint32_t(lo))));
  if (key != NONE) atomicAdd(&sm.bins[(uint32_t(key) - uint32_t(lo)) >> shift], 1);
  __syncthreads();
  int mine[THREADS / 32], sum = 0;
  const int top = THREADS - 1 - int(lane_id()) * (THREADS / 32);  // a lane's bins, from its highest down
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) sum += mine[i] = sm.bins[top - i];
  int before = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, before, d);
    if (int(lane_id()) >= d) before += x;
  }
  const int lane = __ffs(__ballot_sync(0xffffffffu, before >= n)) - 1;
  before -= sum;
  int bin = -1;
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) {
    if (bin < 0) {
      before += mine[i];
      if (before >= n) bin = top - i;
    }
  }
  bin = __shfl_sync(0xffffffffu, bin, lane);
  have = __shfl_sync(0xffffffffu, before, lane);
  lo += int(uint32_t(bin) << shift);
  if (have <= 2 * n) return lo;
  hi = min(hi, lo + int((1u << shift) - 1u));
  while (lo < hi) {
    const int mid = lo + int((uint32_t(hi) - uint32_t(lo) + 1u) >> 1);
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
  static constexpr uint32_t NONE_RAW = 0xFF800000u;  // -infinity
  static __device__ __forceinline__ uint32_t raw(const float* p) {
    uint32_t r;
    asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(r) : "l"(p));
    return r;
  }
  static __device__ __forceinline__ float value(uint32_t r) { return __uint_as_float(r); }
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
  static constexpr uint32_t NONE_RAW = 0xFF80u;
  static __device__ __forceinline__ uint32_t raw(const uint16_t* p) { return __ldg(p); }
  static __device__ __forceinline__ float value(uint32_t r) { return __uint_as_float(r << 16); }
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
    uint4 r;
    if (in && e >= 0 && e + W <= V) {
      r = Vec<T>::load(first + e);
    } else if (in && e < V) {
      r = edge(first, e, V);
    } else {
#pragma unroll
      for (int c = 0; c < W; ++c) Vec<T>::set(r, c, -INFINITY);
    }
    return r;
  }
  // Code that runs once a launch costs more to fetch than to run: what is rare is kept out of line.
  static __device__ __noinline__ uint4 edge(const T* first, int e, int V) {
    uint4 r;
#pragma unroll
    for (int c = 0; c < W; ++c) Vec<T>::set(r, c, e + c >= 0 && e + c < V ? Vec<T>::one(first + e + c) : -INFINITY);
    return r;
  }
};

// Which elements of a row a part has.
__device__ __forceinline__ int2 part_range(const BeamParams& p, int split) {
  return make_int2(min(p.V, split * p.per), min(p.V, (split + 1) * p.per));
}
// The UNIT values of a thread at one step: a warp's are 32 UNIT neighbours from `at` on, a lane's every 32nd.  Which thread has
// which goes by the token alone, not by where the row begins in memory, so that rows of the same logits have the same sum, and
// equal beams stay in order.  (Loads of 16 bytes whose elements go by alignment took 512 beams of 50001 in 25 us and not 27,
// one user's 4 of 128256 in 15.3 and not 9.6; by the token in three narrower pieces the former took 38.)
template <typename T>
__device__ __forceinline__ void load_unit(const T* first, int at, int end, uint32_t (&x)[UNIT]) {
  const T* from = first + at + int(lane_id());
  if (at + 32 * UNIT <= end) {
#pragma unroll
    for (int i = 0; i < UNIT; ++i) x[i] = Vec<T>::raw(from + 32 * i);
  } else {
    const int left = end - at - int(lane_id());
#pragma unroll
    for (int i = 0; i < UNIT; ++i) x[i] = 32 * i < left ? Vec<T>::raw(from + 32 * i) : Vec<T>::NONE_RAW;
  }
}

// The block's sum again, relative to the maximum itself: for logits whose powers of two fp32 does not tell apart, and for
// infinities (1 for each; what is NaN stays).
template <typename T>
__device__ __noinline__ void far_sum(Smem& sm, const T* first, int begin, int end, float most) {
  float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll 4
  for (int t = begin + int(threadIdx.x); t < end; t += THREADS) {
    const float x = Vec<T>::value(Vec<T>::raw(first + t));
    const float e = x == most ? 1.0f : x == x ? ex2_approx((x - most) * kLog2e) : x;
    sum = sum + make_float2(most == -INFINITY && x == x ? 0.0f : e, 0.0f);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
    sum = sum + make_float2(__shfl_xor_sync(0xffffffffu, sum.x, d), __shfl_xor_sync(0xffffffffu, sum.y, d));
  __syncthreads();
  if (lane_id() == 0) sm.warp_sum[warp_id()] = sum;
  __syncthreads();
}

// One block's part of a row: its sum and its groups' maxima.
template <typename T>
__device__ __forceinline__ void take_part(const BeamParams& p, Smem& sm, int row, int split) {
  const int tid = threadIdx.x, lane = int(lane_id()), warp = int(warp_id());
  const T* first = static_cast<const T*>(p.logits) + int64_t(row) * p.stride;
  const int2 range = part_range(p, split);
  const int steps = (range.y - range.x + STEP - 1) / STEP, begin = range.x + warp * (32 * UNIT);
  float* out = p.maxima + int64_t(blockIdx.x) * p.lines * LINE + tid / GROUP;
  auto put = [&](int line, float x) {
#pragma unroll
    for (int d = 1; d < GROUP; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
    if (tid % GROUP == 0) __stcg(out + line * LINE, x);
  };
  // A thread's sum is relative to 2^c, c a whole number that follows the maximum times log2 e: one fused operation brings
  // a logit to its exponent, and what changes reference does so exactly.
  uint32_t next[UNIT];
  float most = -INFINITY, c = -kFar, hi = 0.0f, lo = 0.0f;
  load_unit(first, begin, range.y, next);
  for (int b = 0; b < steps; ++b) {
    float x[UNIT];
#pragma unroll
    for (int i = 0; i < UNIT; ++i) x[i] = Vec<T>::value(next[i]);
    if (b + 1 < steps) load_unit(first, begin + (b + 1) * STEP, range.y, next);
    float top = max3(x[0], x[1], -INFINITY);  // (a NaN is below everything)
#pragma unroll
    for (int i = 2; i < UNIT; i += 2) top = max3(top, x[i], x[i + 1]);
    if (top * kLog2e > c + 1.0f) {
      const float now = fminf(rintf(top * kLog2e), kFar), f = pow2_below(c - now);
      hi *= f;
      lo *= f;
      c = now;
    }
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < UNIT; i += 2) {
      float y0, y1;
      fma2(x[i], x[i + 1], kLog2e, -c, y0, y1);
      add2(s[i & 2], s[(i & 2) + 1], ex2_ftz(y0), ex2_ftz(y1));
    }
    const float2 sum = two_sum(hi, (s[0] + s[1]) + (s[2] + s[3]));
    hi = sum.x;
    lo += sum.y;
    put(b, top);
    most = fmaxf(most, top);
  }
  for (int b = steps; b < p.lines; ++b) put(b, -INFINITY);  // (the last part of a row may have fewer)
  float block_most = most;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) block_most = fmaxf(block_most, __shfl_xor_sync(0xffffffffu, block_most, d));
  // the warp's sum, relative to a power of two that no thread's is above
  float warp_c = fminf(fmaxf(rintf(block_most * kLog2e), -kFar), kFar);
  float2 sum = make_float2(hi, lo);
  {
    const float f = pow2_below(c - warp_c);
    sum = make_float2(sum.x * f, sum.y * f);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
    sum = sum + make_float2(__shfl_xor_sync(0xffffffffu, sum.x, d), __shfl_xor_sync(0xffffffffu, sum.y, d));
  if (lane == 0) {
    sm.warp_sum[warp] = sum;
    sm.warp_most[warp] = block_most;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < WARPS; ++w) block_most = fmaxf(block_most, sm.warp_most[w]);
  const bool far = fabsf(block_most) > kFar / 2;  // (no logit above -infinity, too)
  if (far) far_sum<T>(sm, first, range.x, range.y, block_most);
  if (warp == 0) {
    const float block_c = rintf(block_most * kLog2e);
    sum = sm.warp_sum[lane % WARPS];
    if (!far) {
      warp_c = fminf(fmaxf(rintf(sm.warp_most[lane % WARPS] * kLog2e), -kFar), kFar);
      const float f = pow2_below(warp_c - block_c);
      sum = make_float2(sum.x * f, sum.y * f);
    }
#pragma unroll
    for (int d = WARPS / 2; d > 0; d >>= 1)
      sum = sum + make_float2(__shfl_xor_sync(0xffffffffu, sum.x, d), __shfl_xor_sync(0xffffffffu, sum.y, d));
    if (lane == 0) {
      // 2^block_c in natural units, and log2 e's second part: 2^(x low) is 2^(most low) but for what is far below it
      float2 ref = make_float2(block_c * 0x1.62ep-1f, fmaf(block_c, 3.194618e-05f, block_most * (kLog2eLow * 0.69314718f)));
      ref = two_sum(ref.x, ref.y + __fmaf_rn(block_c, 0x1.62ep-1f, -ref.x));
      if (far) ref = make_float2(block_most, 0.0f);
      __stcg(p.heads + blockIdx.x, make_float4(ref.x, ref.y, sum.x, sum.y));
    }
  }
}

// ---------------------------------------------------------------- a user's beams together
// A candidate's score: 0.0 where the row offers it, infinity or NaN where it does not.
__device__ __forceinline__ float2 score_of(const Smem& sm, int k, float x) {
  const float2 lse = sm.lse[k];
  return make_float2(sm.score[k], 0.0f) + (make_float2(x, 0.0f) + make_float2(-lse.x, -lse.y));
}
__device__ __forceinline__ bool offered(const Smem& sm, int k, float x, float2 score) {
  return x > -INFINITY && fabsf(sm.lse[k].x) < INFINITY && fabsf(score.x) < INFINITY;
}
// Beam, then logit: smaller is better among equal scores.
__device__ __forceinline__ uint64_t tie_of(int k, float x) {
  return uint64_t(uint32_t(k)) << 32 | uint32_t(~(uint32_t(ordered(x + 0.0f)) ^ 0x80000000u));
}
__device__ __forceinline__ bool before(int64_t key, uint64_t tie, uint32_t token, int64_t key2, uint64_t tie2, uint32_t token2) {
  return key > key2 || (key == key2 && (tie < tie2 || (tie == tie2 && token < token2)));
}
__device__ __forceinline__ void win(const BeamParams& p, Smem& sm, int user, int rank, float score, int k, int t) {
  const int64_t o = int64_t(user) * p.N + rank;
  sm.winner[rank] = k;
  p.parents[o] = user * p.K + k;
  p.tokens[o] = t;
  p.scores_out[o] = score;
  if (p.done_out) p.done_out[o] = sm.lse[k].x == -INFINITY || t == p.eos;
  if (p.history) p.history_out[o * p.history_stride + p.length] = t;
}
// The beams' sums.
__device__ __forceinline__ void join_sums(const BeamParams& p, Smem& sm, int user) {
  const int lane = int(lane_id()), warp = int(warp_id());
  // a row's parts to 2^n lanes, several rows to a warp
  int seg = 1;
  while (seg < min(p.splits, 32)) seg *= 2;
  const int rows = 32 / seg;
#pragma unroll 1
  for (int k0 = warp * rows; k0 < p.K; k0 += WARPS * rows) {
    const int k = k0 + lane / seg;
    const bool row = k < p.K;
    const int beam = user * p.K + min(k, p.K - 1);
    const float4* heads = p.heads + int64_t(beam) * p.splits;
    // three loads at once
    float4 head = __ldcg(heads + min(lane % seg, p.splits - 1));
    const float score = p.scores[beam];
    const bool ended = p.done && p.done[beam];
    float2 ref = make_float2(-INFINITY, 0.0f), sum = make_float2(0.0f, 0.0f);
#pragma unroll 1
    for (int i0 = 0; i0 < p.splits; i0 += seg) {
      const int i = i0 + lane % seg;
      if (i0 > 0) head = __ldcg(heads + min(i, p.splits - 1));
      float2 m = make_float2(-INFINITY, 0.0f), s = make_float2(0.0f, 0.0f);
      if (i < p.splits && !ended) {
        m = make_float2(head.x, head.y);
        s = make_float2(head.z, head.w);
      }
      float2 top = m.x > ref.x || (m.x == ref.x && m.y > ref.y) ? m : ref;
#pragma unroll 1
      for (int d = seg / 2; d > 0; d >>= 1) {
        const float2 o = make_float2(__shfl_xor_sync(0xffffffffu, top.x, d), __shfl_xor_sync(0xffffffffu, top.y, d));
        if (o.x > top.x || (o.x == top.x && o.y > top.y)) top = o;
      }
      if (m.x != top.x || m.y != top.y) s = s * exp_below(m, top);
      if (i0 > 0 && (ref.x != top.x || ref.y != top.y)) sum = sum * exp_below(ref, top);
      ref = top;
#pragma unroll 1
      for (int d = seg / 2; d > 0; d >>= 1)
        s = s + make_float2(__shfl_xor_sync(0xffffffffu, s.x, d), __shfl_xor_sync(0xffffffffu, s.y, d));
      sum = sum + s;
    }
    if (row && lane % seg == 0) {
      float2 lse = make_float2(0.0f, 0.0f);
      if (!ended) lse = sum.x > 0.0f && fabsf(ref.x) < INFINITY ? ref + log_of(sum) : make_float2(ref.x + (sum.x - sum.x), 0.0f);
      if (p.lse) p.lse[user * p.K + k] = lse.x;
      // a row of -infinity, or with +infinity or NaN, offers nothing; nor does one whose score less lse leaves fp32
      const float bias = score - lse.x;
      const bool offers = !ended && fabsf(lse.x) < INFINITY && fabsf(bias) < INFINITY;
      sm.lse[k] = ended ? make_float2(-INFINITY, 0.0f) : offers ? lse : make_float2(INFINITY, 0.0f);
      sm.score[k] = score;
      sm.bias[k] = offers ? bias : -INFINITY;
    }
  }
}

// The groups' maxima of a user lie in lines, a part's after another's; a thread has its place of every fourth one.
// (Counted on, not divided: code that runs once costs its fetch.)
struct Lines {
  int line, k, left;  // its row; lines left of the row, this one included
  __device__ __forceinline__ Lines(const BeamParams& p) : line(int(threadIdx.x) / LINE), k(0), left(p.splits * p.lines - line) { settle(p); }
  __device__ __forceinline__ void settle(const BeamParams& p) {
    while (left <= 0) {
      ++k;
      left += p.splits * p.lines;
    }
  }
  __device__ __forceinline__ void next(const BeamParams& p) {
    line += THREADS / LINE;
    left -= THREADS / LINE;
    settle(p);
  }
};

// The largest of the row's logits below `below`, over the block (all threads get it).
template <typename T>
__device__ __noinline__ float largest_below(const BeamParams& p, Smem& sm, int row, float below) {
  const Row<T> r(p, row);
  constexpr int W = Row<T>::W;
  const int vecs = (p.V + r.skew + W - 1) / W;
  float best = -INFINITY;
#pragma unroll 4
  for (int v = int(threadIdx.x); v < vecs; v += THREADS) {
    float x[W];
    Vec<T>::unpack(r.load(v, true), x);
#pragma unroll
    for (int c = 0; c < W; ++c)
      if (x[c] < below) best = fmaxf(best, x[c]);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, d));
  __syncthreads();
  if (lane_id() == 0) sm.warp_most[warp_id()] = best;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < WARPS; ++w) best = fmaxf(best, sm.warp_most[w]);
  return best;
}

// The best one value of a row after the other, all tokens that have it in order: for plateaus.
template <typename T>
__device__ __noinline__ void join_by_value(const BeamParams& p, Smem& sm, int user) {
  constexpr int W = Row<T>::W;
  const int tid = threadIdx.x, lane = int(lane_id()), warp = int(warp_id());
  for (int k = 0; k < p.K; ++k) {
    const bool row = fabsf(sm.lse[k].x) < INFINITY;
    const float x = row ? largest_below<T>(p, sm, user * p.K + k, INFINITY) : -INFINITY;  // (such a row has no infinity)
    if (tid == 0) sm.next[k] = sm.lse[k].x == -INFINITY ? 0.0f : x;  // (an ended beam's one candidate)
  }
  __syncthreads();
  int placed = 0;
  while (placed < p.N) {
    // the best row, by every thread
    int best = -1;
    int64_t key = 0;
    float2 score = make_float2(0.0f, 0.0f);
    for (int k = 0; k < p.K; ++k) {
      const bool ended = sm.lse[k].x == -INFINITY;
      const float x = sm.next[k];
      const float2 s = ended ? make_float2(sm.score[k], 0.0f) : score_of(sm, k, x);
      if (!(x > -INFINITY) || !(ended ? fabsf(s.x) < INFINITY : offered(sm, k, x, s))) continue;
      if (best < 0 || ordered(s) > key) {
        best = k;
        key = ordered(s);
        score = s;
      }
    }
    if (best < 0) break;
    const float x = sm.next[best];
    __syncthreads();
    if (sm.lse[best].x == -INFINITY) {
      if (tid == 0) {
        win(p, sm, user, placed, score.x, best, p.eos);
        sm.next[best] = -INFINITY;
      }
      ++placed;
      __syncthreads();
      continue;
    }
    const Row<T> r(p, user * p.K + best);
    const int vecs = (p.V + r.skew + W - 1) / W;
    for (int v0 = 0; v0 < vecs && placed < p.N; v0 += THREADS) {
      const int v = v0 + tid;
      float y[W];
      Vec<T>::unpack(r.load(v, v < vecs), y);
      int mine = 0;
#pragma unroll
      for (int c = 0; c < W; ++c) mine += y[c] == x;
      if (!__syncthreads_or(mine)) continue;
      int at = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, at, d);
        if (lane >= d) at += z;
      }
      if (lane == 31) sm.warp_lo[warp] = at;
      __syncthreads();
      int all = 0;
      at += placed - mine;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        if (w < warp) at += sm.warp_lo[w];
        all += sm.warp_lo[w];
      }
#pragma unroll
      for (int c = 0; c < W; ++c)
        if (y[c] == x) {
          if (at < p.N) win(p, sm, user, at, score.x, best, r.token(v, c));
          ++at;
        }
      placed = min(placed + all, p.N);
      __syncthreads();
    }
    if (placed < p.N) {
      const float y = largest_below<T>(p, sm, user * p.K + best, x);
      if (tid == 0) sm.next[best] = y;
      __syncthreads();
    }
  }
}

// A group that is looked at again.
struct Hit {
  int row, token, end;  // of the user; the group's first token; its part's end
};

// The last block of a user: its beams' sums, and the N best of their candidates.
template <typename T>
__device__ __noinline__ void join(const BeamParams& p, Smem& sm, int64_t* keys, int user) {
  const int tid = threadIdx.x;
  uint64_t* ties = reinterpret_cast<uint64_t*>(keys + p.list);
  uint32_t* tokens = reinterpret_cast<uint32_t*>(ties + p.list);
  Hit* hit = reinterpret_cast<Hit*>(tokens + p.list);
  const int lines = p.K * p.splits * p.lines;
  const float* maxima = p.maxima + int64_t(user) * lines * LINE + tid % LINE;
  sm.bins[tid] = 0;
  if (tid < p.N) sm.winner[tid] = -1;
  if (tid == 0) sm.count = sm.hits = 0;
  float x[AHEAD];  // on their way while the sums are taken together
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) {
    const int line = tid / LINE + i * (THREADS / LINE);
    x[i] = -INFINITY;
    if (line < lines) x[i] = __ldcg(maxima + line * LINE);
  }
  join_sums(p, sm, user);
  __syncthreads();
  // The threads' best groups (and ended beams), in fp32, and a bound that N of them reach.
  const bool ended = tid < p.K && sm.lse[tid].x == -INFINITY && fabsf(sm.score[tid]) < INFINITY;
  float best = ended ? sm.score[tid] : -INFINITY;
  Lines at(p);
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) {
    x[i] += sm.bias[min(at.k, p.K - 1)];
    best = fmaxf(best, x[i]);
    at.next(p);
  }
  {
    Lines l = at;
#pragma unroll 4
    for (; l.line < lines; l.next(p)) best = fmaxf(best, __ldcg(maxima + int64_t(l.line) * LINE) + sm.bias[l.k]);
  }
  bool exact;
  const int cut = bound(sm, best > -INFINITY ? ordered(best + 0.0f) : NONE, p.N, exact);
  // An fp32 score is off by 2^-24 of itself and of the bias: what lies twice that below the bound may be among the N best.
  float large = fmaxf(fabsf(unordered(cut)), 0.0f);
  for (int k = int(lane_id()); k < p.K; k += 32)
    if (sm.bias[k] > -INFINITY) large = fmaxf(large, fabsf(sm.bias[k]));
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) large = fmaxf(large, __shfl_xor_sync(0xffffffffu, large, d));
  const float above = cut == NONE + 1 ? -3.402823466e38f : fmaxf(unordered(cut) - large * 0x1p-20f, -3.402823466e38f);
  if (best >= above) {
    if (ended && sm.score[tid] >= above) {
      const int at = atomicAdd(&sm.count, 1);  // (64 of them: the list has more places)
      ties[at] = uint64_t(uint32_t(tid)) << 32;
      tokens[at] = uint32_t(p.eos);
    }
    auto take = [&](int line) {
      const int at = atomicAdd(&sm.hits, 1);
      if (at >= HITS) return;
      const int k = line / (p.splits * p.lines), part = line / p.lines;
      const int2 range = part_range(p, part - k * p.splits);
      const int q = tid % LINE;
      hit[at] = Hit{k, range.x + (line - part * p.lines) * STEP + q / (32 / GROUP) * (32 * UNIT) + q % (32 / GROUP) * GROUP, range.y};
    };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (x[i] >= above) take(tid / LINE + i * (THREADS / LINE));
#pragma unroll 4
    for (; at.line < lines; at.next(p))
      if (__ldcg(maxima + int64_t(at.line) * LINE) + sm.bias[at.k] >= above) take(at.line);
  }
  __syncthreads();
  const int hits = sm.hits;
  // ---------------------------------------------------------------- what reaches the bound
  if (hits <= HITS) {
    // a group's elements are GROUP neighbours of every 32 of its warp's; a thread takes EACH of them, 32 APART places apart
    constexpr int EACH = 4, APART = UNIT / EACH, PER_HIT = GROUP * APART, BATCH = 4;
    const int offset = tid / GROUP % APART * 32 + tid % GROUP;
#pragma unroll 1
    for (int h0 = tid / PER_HIT; h0 < hits; h0 += BATCH * (THREADS / PER_HIT)) {
      uint32_t w[BATCH][EACH];
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const Hit at = hit[min(h0 + i * (THREADS / PER_HIT), hits - 1)];
        const T* from = static_cast<const T*>(p.logits) + int64_t(user * p.K + at.row) * p.stride + at.token + offset;
#pragma unroll
        for (int j = 0; j < EACH; ++j)
          w[i][j] = at.token + offset + j * (32 * APART) < at.end ? Vec<T>::raw(from + j * (32 * APART)) : Vec<T>::NONE_RAW;
      }
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const int h = h0 + i * (THREADS / PER_HIT);
        if (h >= hits) break;
        const float bias = sm.bias[hit[h].row];
#pragma unroll
        for (int j = 0; j < EACH; ++j) {
          const float y = Vec<T>::value(w[i][j]);
          if (!(y + bias >= above)) continue;
          const int place = atomicAdd(&sm.count, 1);
          if (place < p.list) {
            ties[place] = tie_of(hit[h].row, y);
            tokens[place] = uint32_t(hit[h].token + offset + j * (32 * APART));
          }
        }
      }
    }
  }
  __syncthreads();
  const int n = sm.count;
  if (hits <= HITS && n <= p.list) {
    for (int e = tid; e < n; e += THREADS) {
      const int k = int(ties[e] >> 32);
      const float y = unordered(int(~uint32_t(ties[e]) ^ 0x80000000u));
      const bool ended = sm.lse[k].x == -INFINITY;
      const float2 s = ended ? make_float2(sm.score[k], 0.0f) : score_of(sm, k, y);
      keys[e] = ended || offered(sm, k, y, s) ? ordered(s) : int64_t(0x8000000000000000ull);
    }
    __syncthreads();
    // eight lanes to a candidate
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
      if (e < n && tid % 8 == 0 && rank < p.N && key != int64_t(0x8000000000000000ull)) win(p, sm, user, rank, unordered(int(key >> 32)), int(tie >> 32), int(t));
    }
  } else {
    join_by_value<T>(p, sm, user);
  }
  __syncthreads();
  if (tid < p.N && sm.winner[tid] < 0) {
    const int64_t o = int64_t(user) * p.N + tid;
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
  extern __shared__ __align__(16) int64_t list[];
  __shared__ Smem sm;
  const int row = int(blockIdx.x) / p.splits, split = int(blockIdx.x) - row * p.splits, user = row / p.K;
  if (!(p.done && p.done[row])) take_part<T>(p, sm, row, split);
  __syncthreads();
  if (threadIdx.x == 0) {
    // what the block has written is released, what the others have is acquired
    uint32_t before;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(p.counters + user) : "memory");
    sm.last = before == uint32_t(p.K * p.splits - 1);
    if (sm.last) p.counters[user] = 0;
  }
  __syncthreads();
  if (sm.last) join<T>(p, sm, list, user);
}

constexpr size_t kCounters = size_t(MAX_B) * 4;  // in a place that does not depend on the sizes
// Parts of a row: as many as fill the GPU, of 4096 elements at least and 65536 at most.
int least_splits(int V) { return cdiv(V, MOST_STEPS * STEP); }
int split_count(int64_t rows, int V) {
  return std::max(least_splits(V), std::min(std::min(cdiv(V, STEP), 32), int((BLOCKS + rows - 1) / rows)));
}
// Elements of a part, a multiple of a warp's 32; and its lines of maxima.
int part_elements(int V, int splits) { return cdiv(cdiv(V, splits), 32) * 32; }
int line_count(int V, int splits) { return cdiv(part_elements(V, splits), STEP); }
int64_t part_bytes(int lines) { return int64_t(sizeof(float4)) + lines * LINE * 4; }

}  // namespace
}  // namespace tl

extern "C" size_t tl_beam_select_workspace_size(int B, int K, int N, int V) {
  using namespace tl;
  if (B < 1 || B > MAX_B || K < 1 || K > MAX_BEAMS || N < 1 || N > MAX_N || V < 1 || int64_t(K) * V > MAX_LOGITS) return 0;
  // parts of all rows are at most this many, of at most this size, which never fall as B or K grow
  return kCounters + (size_t(B) * K * least_splits(V) + BLOCKS) * part_bytes(line_count(V, least_splits(V)));
}

extern "C" tl_status tl_beam_select(const tl_beam_select_args* a, void* stream) {
  using namespace tl;
  const char* who = "tl_beam_select";
  if (!a) return fail(TL_ERR_INVALID, "%s: NULL args", who);
  if (a->B < 0 || a->K < 1 || a->N < 1 || a->V < 1)
    return fail(TL_ERR_INVALID, "%s: B %d, K %d, N %d, V %d", who, a->B, a->K, a->N, a->V);
  if (a->B > MAX_B || a->K > MAX_BEAMS || a->N > MAX_N || int64_t(a->K) * a->V > MAX_LOGITS)
    return fail(TL_ERR_UNSUPPORTED, "%s: B %d (at most 16384), K %d, N %d (64 each), K * V = %lld (2^30)", who, a->B, a->K, a->N,
                static_cast<long long>(a->K) * a->V);
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
  if (ranges_meet(a->scores, in * 4, a->scores_out, out * 4) || (a->done && a->done_out && ranges_meet(a->done, in, a->done_out, out)))
    return fail(TL_ERR_INVALID, "%s: scores_out or done_out overlaps what it is made from", who);
  if ((a->history != nullptr) != (a->history_out != nullptr))
    return fail(TL_ERR_INVALID, "%s: history and history_out go together", who);
  if (a->history) {
    if (a->length < 0 || a->length >= a->history_stride)
      return fail(TL_ERR_INVALID, "%s: length %d, history rows of %d", who, a->length, a->history_stride);
    if (ranges_meet(a->history, in * a->history_stride * 4, a->history_out, out * a->history_stride * 4))
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
  p.B = a->B;
  p.K = a->K;
  p.N = a->N;
  p.V = a->V;
  p.eos = a->eos;
  p.splits = split_count(in, a->V);
  p.lines = line_count(a->V, p.splits);
  p.per = part_elements(a->V, p.splits);
  p.heads = reinterpret_cast<float4*>(static_cast<uint8_t*>(a->workspace) + kCounters);
  p.maxima = reinterpret_cast<float*>(p.heads + in * p.splits);
  p.list = std::max(256, 16 * a->N);
  const size_t smem = size_t(p.list) * 20 + HITS * 12;
  const int64_t blocks = in * p.splits;
  if (blocks > 0x7FFFFFFF) return fail(TL_ERR_UNSUPPORTED, "%s: too many rows", who);
  void* args[] = {&p};
  const void* kernel = a->dtype ? reinterpret_cast<const void*>(&beam_kernel<uint16_t>) : reinterpret_cast<const void*>(&beam_kernel<float>);
  return launch(kernel, int(blocks), THREADS, smem, static_cast<cudaStream_t>(stream), args, false);
}
