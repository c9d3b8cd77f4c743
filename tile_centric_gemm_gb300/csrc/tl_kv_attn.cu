// tl_kv_attn.cu -- attention of a ragged batch's new tokens over the 8-bit paged
// cache: the split kernel for few query rows per kv head (single tokens, drafts).
//
//   s_j = scale <q, k_j>,  O = sum_j exp(s_j - lse) v_j
//
// The cache is read once; everything else is small, so the kernel is a stream of
// pages through one CTA per SM.  The work is the list of (sequence, kv head,
// 16-row tile, 16-token chunk), cut into equal runs, one to a CTA: a long context
// is spread over many CTAs and short ones share a CTA, whatever the mix.  Runs are
// found on the device from the lengths, so the host needs no lengths.  A tile
// whose chunks fall to several CTAs leaves partial results (mean value, maximum,
// sum) in the workspace; the CTA that arrives last joins them in CTA order, so
// the result does not depend on timing.
//
// Inside a CTA the eight warps take a run's chunks in turn, each on its own:
//  * The contraction index of a product may be permuted at will if both operands
//    are.  Lane (g, t) of an m16n8k16 product holds, for key g, the dims that it
//    gets from two 16-byte loads of that key's codes, and for values four tokens'
//    16 dims each; so every lane copies (cp.async) just the bytes that it will
//    multiply, into a ring of its own in shared memory: no transposition, no
//    barrier between copy and use, six chunks (4 KB) in flight per warp.
//  * e4m3 to fp16 is exact (one conversion for two codes).  Queries are brought
//    to fp16 by a power of two for each row, exact but below 2^-25 of the row's
//    largest element.  The K scale multiplies the scores, the V scale of the
//    chunk relative to the largest seen multiplies P, both powers of two.
//  * P is kept as exp2(s - m + 7) with m raised only when a score passes it by 8:
//    at most 2^15, in fp16 with full precision down to 2^-21 of the largest and a
//    grain of 2^-31 of it, so even a tail of millions of small weights counts.
//    Sums of P are taken in fp32 before P is rounded.
#include <algorithm>
#include <cmath>

#include "tl_internal.h"
#include "tl_kv.cuh"

namespace tl {
namespace {

constexpr int WARPS = 8;
constexpr int THREADS = WARPS * 32;
constexpr int STAGES = 6;
constexpr int TILE = 16;   // query rows of one tile
constexpr int CHUNK = 16;  // tokens of one chunk (a page holds whole chunks)
constexpr float kShift = 7.0f;
constexpr float kSlack = 8.0f;

struct DecodeParams {
  KvCacheDev c;
  KvBatch b;
  const uint16_t* q;
  int64_t q_ts, q_hs;
  uint16_t* out;
  float* lse;
  uint32_t* counters;  // [CTAs], zero between calls
  float* partial;      // [CTAs][2][TILE * D + 2 * TILE]
  int32_t H, group, causal;
  float scale_log2;
};

template <int D>
struct DecodeSmem {
  static constexpr int STAGE = CHUNK * D * 2;          // bytes of one chunk, keys and values
  static constexpr int PITCH = D / 4 + 1;              // 16-byte units of one row of the merge buffers
  uint8_t ring[WARPS][STAGES][STAGE];
  float4 merge[WARPS / 2][TILE * PITCH];
  float m[WARPS][TILE], l[WARPS][TILE];
  uint32_t meta[WARPS][STAGES];  // bit 16: the page is good; scale bytes of keys (0-7) and values (8-15)
  int32_t e[WARPS];
  int64_t warp_sum[WARPS];
  int64_t begin_off;
  int32_t begin_seq, last;
};

// One run's piece of one tile: chunks cb .. ce-1 of the tile's nch.
struct Segment {
  KvSeq seq;
  int s, nch, tiles, sub, cb, ce;  // sub = kv head * tiles + row tile
  int64_t left;                    // chunks of the run from cb on
};

__device__ __forceinline__ int seq_tiles(const DecodeParams& p, const KvSeq& q) {
  return int((int64_t(q.q) * p.group + TILE - 1) / TILE);
}
__device__ __forceinline__ int seq_chunks(const KvSeq& q) { return max(1, (q.len + CHUNK - 1) / CHUNK); }

__device__ __forceinline__ void seg_open(const DecodeParams& p, Segment& g, int s, int64_t off, int64_t left) {
  g.seq = kv_seq(p.b, p.c.ps, s);
  g.s = s;
  g.nch = seq_chunks(g.seq);
  g.tiles = seq_tiles(p, g.seq);
  g.sub = int(off / g.nch);
  g.cb = int(off - int64_t(g.sub) * g.nch);
  g.left = left;
  g.ce = int(min(int64_t(g.nch), g.cb + left));
}
__device__ __forceinline__ bool seg_next(const DecodeParams& p, Segment& g) {
  g.left -= g.ce - g.cb;
  if (g.left <= 0) return false;
  if (++g.sub < g.tiles * p.c.Hkv) {
    g.cb = 0;
    g.ce = int(min(int64_t(g.nch), g.left));
    return true;
  }
  int s = g.s + 1;
  while (s < p.b.B && kv_seq(p.b, p.c.ps, s).q == 0) ++s;
  if (s >= p.b.B) return false;
  seg_open(p, g, s, 0, g.left);
  return true;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 r;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a) : "memory");
  return r;
}
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
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}
// Which bytes are e4m3 NaN (0x7f, 0xff): 0x80 there.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// 16-byte unit c of row r in a merge buffer (the exclusive-or spreads a quad's blocks over the banks).
template <int D>
__device__ __forceinline__ int merge_at(int r, int c) {
  return r * DecodeSmem<D>::PITCH + (c ^ (((c >> 3) & 3) << 1));
}

template <int D>
__global__ void __launch_bounds__(THREADS, 1) kv_decode_kernel(const __grid_constant__ DecodeParams p) {
  using Smem = DecodeSmem<D>;
  constexpr int KL = D / 64;   // 16-byte key loads of one lane and key
  constexpr int NT = D / 8;    // n tiles of the output: dim = lane group * NT + n tile
  constexpr int VB = NT;       // value bytes of one lane and token
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const KvBatch& b = p.b;

  // ---------------------------------------------------------------- this CTA's run of chunks
  const int per = (b.B + THREADS - 1) / THREADS;
  const int first = min(b.B, tid * per), end = min(b.B, first + per);
  int64_t mine = 0;
  for (int s = first; s < end; ++s) {
    const KvSeq q = kv_seq(b, p.c.ps, s);
    mine += int64_t(seq_tiles(p, q)) * p.c.Hkv * seq_chunks(q);
  }
  int64_t before = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, before, d);
    if (lane >= d) before += x;
  }
  if (lane == 31) sm.warp_sum[warp] = before;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w == warp) before += total;
    total += sm.warp_sum[w];
  }
  before -= mine;
  // a CTA gets a chunk for each warp at least
  const int64_t n = min(int64_t(gridDim.x), max(int64_t(1), total / WARPS));
  const int64_t cta = blockIdx.x;
  if (cta >= n || total == 0) return;
  const int64_t run0 = cta * total / n, run1 = (cta + 1) * total / n;
  if (run0 >= run1) return;
  if (mine > 0 && before <= run0 && run0 < before + mine) {
    int64_t at = before;
    for (int s = first; s < end; ++s) {
      const KvSeq q = kv_seq(b, p.c.ps, s);
      const int64_t size = int64_t(seq_tiles(p, q)) * p.c.Hkv * seq_chunks(q);
      if (run0 < at + size) {
        sm.begin_seq = s;
        sm.begin_off = run0 - at;
        break;
      }
      at += size;
    }
  }
  __syncthreads();
  Segment f, c;  // where copies are, and where products are
  seg_open(p, c, sm.begin_seq, sm.begin_off, run1 - run0);
  f = c;

  // ---------------------------------------------------------------- the copies of one warp
  const uint32_t ring = smem_u32(sm.ring[warp]);
  const int page_chunks = p.c.ps / CHUNK;
  bool f_ok = true;
  int fc = f.cb + warp, f_base = 0, pages = 0, scales = 0;
  bool f_new = true;
  auto settle = [&]() {  // on to a segment that has a chunk for this warp
    while (f_ok && fc >= f.ce) {
      f_ok = seg_next(p, f);
      fc = f.cb + warp;
      f_new = true;
    }
  };
  settle();
  auto fetch = [&](int stage) {
    if (f_ok) {
      int at = (fc - f_base) / WARPS;
      if (f_new || at == 32) {  // the pages of the next 32 chunks, one to a lane
        f_base = fc;
        f_new = false;
        at = 0;
        const int ch = fc + lane * WARPS;
        pages = -1;
        scales = 0;
        if (ch < f.ce && ch * CHUNK < f.seq.len) {
          pages = __ldg(b.table + int64_t(f.s) * b.max_pages + ch / page_chunks);
          if (pages < 0 || pages >= p.c.num_pages) {
            record_error(b.status, kKvInvalid, uint32_t(f.s), uint32_t(pages), uint32_t(ch / page_chunks));
            pages = -1;
          } else {
            const int64_t i = int64_t(pages) * p.c.Hkv + f.sub / f.tiles;
            scales = 0x10000 | int(p.c.ks[i]) | (int(p.c.vs[i]) << 8);
          }
        }
        __syncwarp();
      }
      const int page = __shfl_sync(0xffffffffu, pages, at);
      if (page >= 0) {
        const int64_t off = int64_t(page) * p.c.page_stride + int64_t(f.sub / f.tiles) * p.c.head_stride +
                            int64_t(fc % page_chunks * CHUNK) * p.c.token_stride;
        const uint32_t dst = ring + uint32_t(stage * Smem::STAGE) + uint32_t(lane * 16);
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int j = 0; j < KL; ++j)
            cp_async16(dst + uint32_t((nt * KL + j) * 512), p.c.k + off + (nt * 8 + g) * p.c.token_stride + j * 64 + t * 16);
        const uint32_t vdst = ring + uint32_t(stage * Smem::STAGE + CHUNK * D) + uint32_t(lane * VB);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint8_t* src = p.c.v + off + (2 * t + (j & 1) + (j >> 1) * 8) * p.c.token_stride + g * VB;
          if (VB == 16) cp_async16(vdst + uint32_t(j * 32 * VB), src);
          else cp_async8(vdst + uint32_t(j * 32 * VB), src);
        }
      }
      const int sc = __shfl_sync(0xffffffffu, scales, at);
      if (lane == 0) sm.meta[warp][stage] = uint32_t(sc);
      fc += WARPS;
      settle();
    }
    cp_async_commit();
  };
  for (int i = 0; i < STAGES - 1; ++i) fetch(i);

  // ---------------------------------------------------------------- segment by segment
  int stage = 0;
  int64_t at = run0;  // position of c.cb in the list
  while (true) {
    const int hk = c.sub / c.tiles, r0 = (c.sub % c.tiles) * TILE;
    const int rows = min(TILE, int(int64_t(c.seq.q) * p.group - r0));
    // this lane's two rows: key limits and queries
    int lim[2];
    float f_row[2];
    uint32_t qa[KL * 4][4];
    const int start = c.seq.len - c.seq.q;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = r0 + min(g + 8 * x, rows - 1);
      const int i = r / p.group;
      lim[x] = p.causal ? max(0, min(c.seq.len, start + i + 1)) : c.seq.len;
      const uint16_t* src = p.q + int64_t(c.seq.row0 + i) * p.q_ts + int64_t(hk * p.group + r % p.group) * p.q_hs;
      uint4 w[KL * 2];
      float amax = 0.0f;
#pragma unroll
      for (int j = 0; j < KL; ++j) {
        w[2 * j] = *reinterpret_cast<const uint4*>(src + j * 64 + t * 16);
        w[2 * j + 1] = *reinterpret_cast<const uint4*>(src + j * 64 + t * 16 + 8);
      }
#pragma unroll
      for (int j = 0; j < KL * 2; ++j) {
        const uint32_t u[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(u[k] << 16)), fabsf(__uint_as_float(u[k] & 0xFFFF0000u))));
      }
      amax = quad_max(amax);
      const int e = max(int(__float_as_uint(amax) >> 23) - 127, -126);
      const float down = pow2f(-e);
      f_row[x] = pow2f(e) * p.scale_log2;
#pragma unroll
      for (int j = 0; j < KL * 2; ++j) {
        const uint32_t u[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
        uint32_t h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          h[k] = pack_f16x2(__uint_as_float(u[k] << 16) * down, __uint_as_float(u[k] & 0xFFFF0000u) * down);
        // dims 4v .. 4v+3 of the lane's 16 are the k slots (2t, 2t+1, 2t+8, 2t+9) of step v
        qa[2 * j][x] = h[0];
        qa[2 * j][2 + x] = h[1];
        qa[2 * j + 1][x] = h[2];
        qa[2 * j + 1][2 + x] = h[3];
      }
    }
    const int min_lim = p.causal ? max(0, min(c.seq.len, start + r0 / p.group + 1)) : c.seq.len;

    float o[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    int ve = -127;

    for (int ch = c.cb + warp; ch < c.ce; ch += WARPS) {
      cp_async_wait<STAGES - 2>();
      __syncwarp();
      const uint32_t meta = sm.meta[warp][stage];
      const uint32_t src = ring + uint32_t(stage * Smem::STAGE);
      if (meta & 0x10000u) {
        const int tok = ch * CHUNK;
        float s[2][4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
          for (int j = 0; j < 4; ++j) s[nt][j] = 0.0f;
#pragma unroll
          for (int j = 0; j < KL; ++j) {
            const uint4 w = lds128(src + uint32_t((nt * KL + j) * 512 + lane * 16));
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int v = 0; v < 4; ++v)
              mma_f16(s[nt], qa[j * 4 + v][0], qa[j * 4 + v][1], qa[j * 4 + v][2], qa[j * 4 + v][3],
                      e4m3x2_to_f16x2(u[v]), e4m3x2_to_f16x2_hi(u[v]));
          }
        }
        const float kf = pow2f(int(meta & 0xFFu) - 127);
        const float fx[2] = {f_row[0] * kf, f_row[1] * kf};
        const bool edge = tok + CHUNK > min_lim;
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s[nt][j] *= fx[j >> 1];
            if (edge && tok + nt * 8 + 2 * t + (j & 1) >= lim[j >> 1]) s[nt][j] = -INFINITY;
            mx[j >> 1] = fmaxf(mx[j >> 1], s[nt][j]);
          }
        mx[0] = quad_max(mx[0]);
        mx[1] = quad_max(mx[1]);
        const int vb = int((meta >> 8) & 0xFFu);
        const bool up = vb != 255 && vb - 127 > ve;
        if (__any_sync(0xffffffffu, mx[0] > m[0] + kSlack || mx[1] > m[1] + kSlack) || up) {
          float a[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float mn = mx[x] > m[x] + kSlack ? mx[x] : m[x];
            a[x] = mn == m[x] ? 1.0f : ex2_approx(m[x] - mn);
            m[x] = mn;
            l[x] *= a[x];
          }
          if (up) {
            const float down = pow2f(max(ve - (vb - 127), -127));
            ve = vb - 127;
            a[0] *= down;
            a[1] *= down;
          }
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            o[i][0] *= a[0];
            o[i][1] *= a[0];
            o[i][2] *= a[1];
            o[i][3] *= a[1];
          }
        }
        const float vf = vb == 255 ? pow2f(128) : pow2f(max(vb - 127 - ve, -127));
        const float nm[2] = {m[0] == -INFINITY ? kShift : kShift - m[0], m[1] == -INFINITY ? kShift : kShift - m[1]};
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[nt][j] = ex2_approx(s[nt][j] + nm[j >> 1]);
        l[0] += (s[0][0] + s[0][1]) + (s[1][0] + s[1][1]);
        l[1] += (s[0][2] + s[0][3]) + (s[1][2] + s[1][3]);
        uint32_t pa[4];
        pa[0] = pack_f16x2(s[0][0] * vf, s[0][1] * vf);
        pa[1] = pack_f16x2(s[0][2] * vf, s[0][3] * vf);
        pa[2] = pack_f16x2(s[1][0] * vf, s[1][1] * vf);
        pa[3] = pack_f16x2(s[1][2] * vf, s[1][3] * vf);

        uint32_t vw[4][VB / 4];
        const uint32_t vsrc = src + uint32_t(CHUNK * D + lane * VB);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (VB == 16) {
            const uint4 w = lds128(vsrc + uint32_t(j * 32 * VB));
            vw[j][0] = w.x;
            vw[j][1] = w.y;
            vw[j][VB / 4 - 2] = w.z;
            vw[j][VB / 4 - 1] = w.w;
          } else {
            const uint2 w = lds64(vsrc + uint32_t(j * 32 * VB));
            vw[j][0] = w.x;
            vw[j][1] = w.y;
          }
        }
        if (edge) {
          // slots past the sequence's end hold anything: zero.  A NaN value that some rows see and
          // others do not would reach the others as 0 * NaN: it is taken out here and counted for
          // the rows that see it by a product of 0/1 matrices.
          uint32_t nans = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bool past = tok + 2 * t + (j & 1) + (j >> 1) * 8 >= c.seq.len;
#pragma unroll
            for (int k = 0; k < VB / 4; ++k) {
              if (past) vw[j][k] = 0;
              nans |= nan_bytes(vw[j][k]);
            }
          }
          if (__any_sync(0xffffffffu, nans != 0)) {
            uint32_t sees[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int tk = tok + 2 * t + (j >> 1) * 8, li = lim[j & 1];
              sees[j] = (tk < li ? 0x3C00u : 0u) | (tk + 1 < li ? 0x3C000000u : 0u);
            }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              uint32_t bit[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) bit[j] = (nan_bytes(vw[j][i / 4]) >> (8 * (i % 4))) & 0x80u ? 0x3C00u : 0u;
              float cnt[4] = {0.0f, 0.0f, 0.0f, 0.0f};
              mma_f16(cnt, sees[0], sees[1], sees[2], sees[3], bit[0] | (bit[1] << 16), bit[2] | (bit[3] << 16));
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (cnt[j] > 0.0f) o[i][j] = __uint_as_float(0x7FFFFFFFu);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int k = 0; k < VB / 4; ++k) vw[j][k] &= ~((nan_bytes(vw[j][k]) >> 7) * 0xFFu);
          }
        }
#pragma unroll
        for (int i = 0; i < NT; i += 2) {
          const uint32_t sel = (i & 2) ? 0x7362u : 0x5140u;
          const uint32_t x = __byte_perm(vw[0][i / 4], vw[1][i / 4], sel), y = __byte_perm(vw[2][i / 4], vw[3][i / 4], sel);
          mma_f16(o[i], pa[0], pa[1], pa[2], pa[3], e4m3x2_to_f16x2(x), e4m3x2_to_f16x2(y));
          mma_f16(o[i + 1], pa[0], pa[1], pa[2], pa[3], e4m3x2_to_f16x2_hi(x), e4m3x2_to_f16x2_hi(y));
        }
      }
      __syncwarp();
      fetch((stage + STAGES - 1) % STAGES);
      stage = stage + 1 == STAGES ? 0 : stage + 1;
    }

    // ---------------------------------------------------------------- the eight warps' results become one
    l[0] = quad_sum(l[0]);
    l[1] = quad_sum(l[1]);
    if (t == 0) {
      sm.m[warp][g] = m[0];
      sm.m[warp][g + 8] = m[1];
      sm.l[warp][g] = l[0];
      sm.l[warp][g + 8] = l[1];
    }
    if (lane == 0) sm.e[warp] = ve;
    __syncthreads();
    int em = -127;
    float M[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      em = max(em, sm.e[w]);
      M[0] = fmaxf(M[0], sm.m[w][g]);
      M[1] = fmaxf(M[1], sm.m[w][g + 8]);
    }
    {
      const float vd = pow2f(max(ve - em, -127));
      const float a0 = m[0] == -INFINITY ? vd * (l[0] == 0.0f ? 1.0f : l[0]) : vd * ex2_approx(m[0] - M[0]);
      const float a1 = m[1] == -INFINITY ? vd * (l[1] == 0.0f ? 1.0f : l[1]) : vd * ex2_approx(m[1] - M[1]);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        o[i][0] *= a0;
        o[i][1] *= a0;
        o[i][2] *= a1;
        o[i][3] *= a1;
      }
    }
    // o[i][0..1]: row g, dims 2t * NT + i and (2t+1) * NT + i; o[i][2..3]: row g + 8
    auto each_unit = [&](auto&& fn) {
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i4 = 0; i4 < NT / 4; ++i4) fn(x, h, i4, merge_at<D>(g + 8 * x, (2 * t + h) * (NT / 4) + i4));
    };
    if (warp >= WARPS / 2) {
      float4* buf = sm.merge[warp - WARPS / 2];
      each_unit([&](int x, int h, int i4, int a) {
        buf[a] = make_float4(o[4 * i4][2 * x + h], o[4 * i4 + 1][2 * x + h], o[4 * i4 + 2][2 * x + h], o[4 * i4 + 3][2 * x + h]);
      });
    }
    __syncthreads();
    if (warp < WARPS / 2) {
      float4* buf = sm.merge[warp];
      each_unit([&](int x, int h, int i4, int a) {
        const float4 w = buf[a];
        buf[a] = make_float4(w.x + o[4 * i4][2 * x + h], w.y + o[4 * i4 + 1][2 * x + h], w.z + o[4 * i4 + 2][2 * x + h],
                             w.w + o[4 * i4 + 3][2 * x + h]);
      });
    }
    __syncthreads();
    // sixteen threads to a row now
    constexpr int EPT = D / 16;
    const int row = tid >> 4, d0 = (tid & 15) * EPT;
    float M1 = -INFINITY, L = 0.0f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) M1 = fmaxf(M1, sm.m[w][row]);
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float mw = sm.m[w][row];
      L += mw == -INFINITY ? sm.l[w][row] : sm.l[w][row] * ex2_approx(mw - M1);
    }
    float acc[EPT];
#pragma unroll
    for (int u = 0; u < EPT / 4; ++u) {
      const int a = merge_at<D>(row, d0 / 4 + u);
      const float4 w0 = sm.merge[0][a], w1 = sm.merge[1][a], w2 = sm.merge[2][a], w3 = sm.merge[3][a];
      acc[4 * u] = (w0.x + w1.x) + (w2.x + w3.x);
      acc[4 * u + 1] = (w0.y + w1.y) + (w2.y + w3.y);
      acc[4 * u + 2] = (w0.z + w1.z) + (w2.z + w3.z);
      acc[4 * u + 3] = (w0.w + w1.w) + (w2.w + w3.w);
    }
    const float inv = L == 0.0f ? 0.0f : 1.0f / L, pe = pow2f(em);
#pragma unroll
    for (int i = 0; i < EPT; ++i) acc[i] = acc[i] * inv * pe;

    bool done = true;
    if (c.cb != 0 || c.ce != c.nch) {
      const int64_t t0 = at - c.cb;  // the tile's first chunk in the list
      const int64_t c0 = ((t0 + 1) * n - 1) / total, c1 = ((t0 + c.nch) * n - 1) / total;
      constexpr int SLOT = TILE * D + 2 * TILE;
      float* mineat = p.partial + (2 * cta + (c.cb == 0 ? 1 : 0)) * SLOT;
      if (row < rows) {
#pragma unroll
        for (int u = 0; u < EPT / 4; ++u)
          st_global_cg_v4f(mineat + row * D + d0 + 4 * u, acc[4 * u], acc[4 * u + 1], acc[4 * u + 2], acc[4 * u + 3]);
        if ((tid & 15) == 0) {
          __stcg(mineat + TILE * D + row, M1);
          __stcg(mineat + TILE * D + TILE + row, L);
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
      if (done && row < rows) {
        __threadfence();
        const float* tile = p.partial;
        M1 = -INFINITY;
        for (int64_t x = c0; x <= c1; ++x) M1 = fmaxf(M1, __ldcg(tile + (2 * x + (x == c0)) * SLOT + TILE * D + row));
        L = 0.0f;
#pragma unroll
        for (int i = 0; i < EPT; ++i) acc[i] = 0.0f;
#pragma unroll 4
        for (int64_t x = c0; x <= c1; ++x) {
          const float* slot = tile + (2 * x + (x == c0)) * SLOT;
          const float mw = __ldcg(slot + TILE * D + row), lw = __ldcg(slot + TILE * D + TILE + row);
          const float wgt = mw == -INFINITY ? lw : lw * ex2_approx(mw - M1);
          L += wgt;
#pragma unroll
          for (int u = 0; u < EPT / 4; ++u) {
            const float4 w = ld_global_cg_v4f(slot + row * D + d0 + 4 * u);
            acc[4 * u] = fmaf(wgt, w.x, acc[4 * u]);
            acc[4 * u + 1] = fmaf(wgt, w.y, acc[4 * u + 1]);
            acc[4 * u + 2] = fmaf(wgt, w.z, acc[4 * u + 2]);
            acc[4 * u + 3] = fmaf(wgt, w.w, acc[4 * u + 3]);
          }
        }
        const float i2 = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
        for (int i = 0; i < EPT; ++i) acc[i] *= i2;
      }
    }
    if (done && row < rows) {
      const int r = r0 + row, tok = c.seq.row0 + r / p.group, h = hk * p.group + r % p.group;
      uint32_t w[EPT / 2];
#pragma unroll
      for (int i = 0; i < EPT / 2; ++i) w[i] = pack_bf16x2(acc[2 * i], acc[2 * i + 1]);
      uint16_t* dst = p.out + (int64_t(tok) * p.H + h) * D + d0;
      if (EPT == 8) st_global_v4(dst, w[0], w[1], w[EPT / 2 - 2], w[EPT / 2 - 1]);
      else *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
      if ((tid & 15) == 0 && p.lse)
        p.lse[int64_t(h) * b.n_tokens + tok] =
            L == 0.0f ? -INFINITY : (M1 - kShift + log2f(L)) * 0.69314718055994531f;
    }
    at += c.ce - c.cb;
    if (!seg_next(p, c)) break;
    __syncthreads();  // the merge buffers are free again
  }
  cp_async_wait<0>();
}

// ---------------------------------------------------------------- workspace: counters, then partial tiles
size_t counters_bytes(int ctas) { return (size_t(ctas) * 4 + 255) / 256 * 256; }
size_t decode_partial_bytes(int ctas, int D) { return size_t(ctas) * 2 * (TILE * D + 2 * TILE) * sizeof(float); }

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
  return counters_bytes(sm_count) + decode_partial_bytes(sm_count, head_dim);
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
  const void* kernel = c.head_dim == 128 ? reinterpret_cast<const void*>(&kv_decode_kernel<128>)
                                         : reinterpret_cast<const void*>(&kv_decode_kernel<64>);
  const size_t smem = c.head_dim == 128 ? sizeof(DecodeSmem<128>) : sizeof(DecodeSmem<64>);
  void* args[] = {&p};
  return launch(kernel, di.sm_count, THREADS, smem, static_cast<cudaStream_t>(stream), args, false);
}
