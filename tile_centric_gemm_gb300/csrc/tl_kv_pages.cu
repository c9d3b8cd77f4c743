// tl_kv_pages.cu -- pages of the 8-bit cache shared, copied, compacted, taken and given back.
//
// Which pages are whose is the caller's page tables and, for each page, the number of
// sequences that hold it (0: free).  tl_kv_fork and tl_kv_resize change these once for
// all layers; tl_kv_copy_pages and tl_kv_compact move codes and scales, of all layers in
// one launch.
//
// fork and resize are two launches, or one where there is little to do.  The first has one block that looks at every
// sequence, counts the pages needed in order (a prefix sum) and takes the lowest free
// ones, again by a prefix sum over the holders' counts; its other blocks bring the counts
// to where the new ones go.  The second writes the tables' rows and adds to the counts,
// with integer atomics, whose order does not matter.  A parent of one child adds nothing:
// its pages change hands.
//
// All four are bound by latency: what they move is little.  GPU time in a graph, heads of 128, 8 kv
// heads: four beams of 1000 tokens forked and three part-filled pages copied in 16 layers
// (5 MB) 8.3 us; 512 beams of 900, 4 layers (54 MB) 18.7 us, the copies 10 of them (5.3 TB/s); 26 drafts compacted
// behind 4099 in 16 layers 6.2 us; 64 trees of up to 60 in 8 layers (13 MB) 10.2 us.  A call from Python takes 5 to 9 us
// of the host, 2 to 3 of them the launch.
#include <algorithm>
#include <functional>

#include "tl_internal.h"
#include "tl_kv.cuh"

namespace tl {
namespace {

constexpr int PLAN_THREADS = 1024;
constexpr int ROW_THREADS = 128;
constexpr int COPY_THREADS = 128;
constexpr int LAYERS = 64;  // of one launch: their addresses are kernel parameters

struct Layer {
  uint8_t* k;
  uint8_t* v;
  uint8_t* ks;
  uint8_t* vs;
};

// ---------------------------------------------------------------- tables
struct TableParams {
  const int32_t* table;
  const int32_t* lens;
  const int32_t* to;       // fork: parents; resize: new lengths
  const int32_t* refs;
  int32_t* table_out;      // resize: the table itself
  int32_t* lens_out;
  int32_t* refs_out;
  int32_t* copies;         // [3][B_out]
  int32_t* n_copies;
  int32_t* first;          // workspace, fork: a parent's first child
  int32_t* count;          // and how many it has
  int32_t* base;           // which of the pages taken is a row's first one, or -1
  int32_t* short_of;       // pages that were missing
  uint32_t* status;
  int32_t B_in, B_out, max_pages, ps, pages;
  int32_t rows;            // to be changed by the planning block itself, or 0
};

// Sum of v over the threads before this one, and over all.
template <class T>
__device__ __forceinline__ T block_scan(T v, T* warp_sums, T& all) {
  T sum = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const T x = __shfl_up_sync(0xffffffffu, sum, d);
    if (int(lane_id()) >= d) sum += x;
  }
  __syncthreads();
  if (lane_id() == 31) warp_sums[warp_id()] = sum;
  __syncthreads();
  T before = warp_sums[lane_id()];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const T x = __shfl_up_sync(0xffffffffu, before, d);
    if (int(lane_id()) >= d) before += x;
  }
  all = __shfl_sync(0xffffffffu, before, 31);
  const T others = __shfl_sync(0xffffffffu, before, (warp_id() + 31) & 31);
  return sum - v + (warp_id() ? others : 0);
}
static_assert(PLAN_THREADS == 32 * 32, "a warp sums the warps");

// Whether sequence s may have the length; which pages it holds is not known if not.
__device__ __forceinline__ bool is_len(const TableParams& p, int len, int s) {
  if (len >= 0 && len <= int64_t(p.max_pages) * p.ps) return true;
  record_error(p.status, kKvInvalid, uint32_t(s), uint32_t(len), uint32_t(p.max_pages));
  return false;
}
__device__ __forceinline__ int pages_of(const TableParams& p, int len) { return (len + p.ps - 1) / p.ps; }
__device__ __forceinline__ bool is_page(const TableParams& p, int page) { return page >= 0 && page < p.pages; }

// FORK: an output row's parent, or -1.
__device__ __forceinline__ int parent_of(const TableParams& p, int o) {
  const int b = p.to[o];
  if (b >= 0 && b < p.B_in) return b;
  if (b != -1) record_error(p.status, kKvInvalid, uint32_t(o), uint32_t(b), uint32_t(p.B_in));
  return -1;
}
// How many pages the row takes; a fork's copy: of which page, and how many slots.
__device__ __forceinline__ int fork_need(const TableParams& p, int o, int& src, int& slots) {
  const int b = parent_of(p, o);
  if (b < 0) return 0;
  const int len = p.lens[b];
  if (!is_len(p, len, b)) return 0;
  slots = len % p.ps;
  if (slots == 0) return 0;
  src = p.table[int64_t(b) * p.max_pages + len / p.ps];
  if (!is_page(p, src)) {
    record_error(p.status, kKvInvalid, uint32_t(b), uint32_t(src), uint32_t(len / p.ps));
    return 0;
  }
  return p.first[b] != o || p.refs[src] != 1;
}
// RESIZE: pages before and after; none of either where a length is wrong.
__device__ __forceinline__ int2 resize_pages(const TableParams& p, int s) {
  const int before = p.lens[s], after = p.to[s];
  if (!is_len(p, before, s) || !is_len(p, after, s)) return make_int2(0, 0);
  return make_int2(pages_of(p, before), pages_of(p, after));
}

// What the plan means for one row, by THREADS threads: of a fork a new row (below B_out) or what an old one held.
template <bool FORK, int THREADS>
__device__ __forceinline__ void change_row(const TableParams& p, int row_no, int tid) {
  if (!FORK) {
    const int2 n = resize_pages(p, row_no);
    const int32_t* row = p.table_out + int64_t(row_no) * p.max_pages;
    const int lo = min(n.x, n.y), hi = max(n.x, n.y), add = n.y > n.x ? 1 : -1;
    for (int i = lo + tid; i < hi; i += THREADS) {
      const int page = row[i];
      if (is_page(p, page)) atomicAdd(p.refs_out + page, add);
      else record_error(p.status, kKvInvalid, uint32_t(row_no), uint32_t(page), uint32_t(i));
    }
  } else if (row_no < p.B_out) {
    const int o = row_no, b = p.to[o];
    if (b < 0 || b >= p.B_in || !is_len(p, p.lens[b], b)) {
      if (tid == 0) p.lens_out[o] = 0;
      return;
    }
    const int len = p.lens[b], n = pages_of(p, len), at = p.base[o];
    const int32_t* from = p.table + int64_t(b) * p.max_pages;
    int32_t* row = p.table_out + int64_t(o) * p.max_pages;
    for (int i = tid; i < n; i += THREADS) row[i] = at >= 0 && i == n - 1 ? p.copies[p.B_out + at] : from[i];
    if (tid == 0) {
      p.lens_out[o] = len;
      if (at >= 0) atomicAdd(p.refs_out + p.copies[p.B_out + at], 1);
    }
  } else {
    const int b = row_no - p.B_out;
    const int len = p.lens[b];
    if (!is_len(p, len, b)) return;
    const int full = len / p.ps, children = p.count[b];
    const int32_t* row = p.table + int64_t(b) * p.max_pages;
    if (children != 1) {
      for (int i = tid; i < full; i += THREADS) {
        const int page = row[i];
        if (is_page(p, page)) atomicAdd(p.refs_out + page, children - 1);
        else record_error(p.status, kKvInvalid, uint32_t(b), uint32_t(page), uint32_t(i));
      }
    }
    if (tid == 0 && len % p.ps && is_page(p, row[full]) && (children == 0 || p.base[p.first[b]] >= 0))
      atomicAdd(p.refs_out + row[full], -1);
  }
}

template <bool FORK>
__global__ void __launch_bounds__(PLAN_THREADS, 1) plan_kernel(const __grid_constant__ TableParams p) {
  __shared__ int warp_sums[32];
  __shared__ int64_t warp_needs[32];
  const int tid = threadIdx.x;
  pdl_launch_dependents();
  if (p.rows && p.refs_out != p.refs) {
    for (int64_t i = tid; i < p.pages; i += PLAN_THREADS) p.refs_out[i] = p.refs[i];
  }
  if (blockIdx.x > 0) {  // the counts, to where the new ones go
    const int64_t step = int64_t(gridDim.x - 1) * PLAN_THREADS;
    for (int64_t i = int64_t(blockIdx.x - 1) * PLAN_THREADS + tid; i < p.pages; i += step) p.refs_out[i] = p.refs[i];
    return;
  }
  if (FORK) {
    for (int b = tid; b < p.B_in; b += PLAN_THREADS) {
      p.first[b] = 0x7FFFFFFF;
      p.count[b] = 0;
    }
    __syncthreads();
    for (int o = tid; o < p.B_out; o += PLAN_THREADS) {
      const int b = parent_of(p, o);
      if (b < 0) continue;
      atomicMin(p.first + b, o);
      atomicAdd(p.count + b, 1);
    }
    __syncthreads();
  }
  int64_t total = 0;
  for (int r0 = 0; r0 < p.B_out; r0 += PLAN_THREADS) {
    const int r = r0 + tid;
    int need = 0, src = 0, slots = 0;
    if (r < p.B_out) {
      if (FORK) {
        need = fork_need(p, r, src, slots);
      } else {
        const int2 n = resize_pages(p, r);
        need = max(0, n.y - n.x);
      }
    }
    int64_t all;
    const int64_t at = total + block_scan<int64_t>(need, warp_needs, all);
    if (r < p.B_out) p.base[r] = FORK && !need ? -1 : int(min(at, int64_t(0x7FFFFFFF)));
    if (FORK && need) {
      p.copies[at] = src;
      p.copies[2 * p.B_out + at] = slots;
    }
    total += all;
  }
  __syncthreads();
  // the lowest free pages, in order: sixteen counts to a thread
  constexpr int PER = 16;
  int found = 0;
  for (int64_t i0 = 0; i0 < p.pages && found < total; i0 += PLAN_THREADS * PER) {
    const int64_t i = i0 + tid * PER;
    uint32_t free = 0;
    if (i + PER <= p.pages) {
#pragma unroll
      for (int k = 0; k < PER / 4; ++k) {
        const int4 v = *reinterpret_cast<const int4*>(p.refs + i + 4 * k);
        free |= uint32_t(v.x == 0) << (4 * k) | uint32_t(v.y == 0) << (4 * k + 1) | uint32_t(v.z == 0) << (4 * k + 2) |
                uint32_t(v.w == 0) << (4 * k + 3);
      }
    } else {
      for (int k = 0; k < PER && i + k < p.pages; ++k) free |= uint32_t(p.refs[i + k] == 0) << k;
    }
    int all;
    int rank = found + block_scan<int>(__popc(free), warp_sums, all);
    while (free && rank < total) {
      const int page = int(i) + __ffs(free) - 1;
      free &= free - 1;
      if (FORK) {
        p.copies[p.B_out + rank] = page;
      } else {
        int lo = 0, hi = p.B_out - 1;  // the last row whose first page is at or below this one
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (p.base[mid] <= rank) lo = mid;
          else hi = mid - 1;
        }
        p.table_out[int64_t(lo) * p.max_pages + pages_of(p, p.lens[lo]) + rank - p.base[lo]] = page;
      }
      ++rank;
    }
    found += all;
  }
  if (tid == 0) {
    const int missing = int(min(max(total - found, int64_t(0)), int64_t(0x7FFFFFFF)));
    *p.short_of = missing;
    if (FORK) *p.n_copies = missing ? 0 : int(total);
    if (missing) record_error(p.status, kKvInvalid, uint32_t(missing), uint32_t(found), uint32_t(total));
  }
  if (p.rows == 0 || found < total) return;
  __syncthreads();
  for (int row = int(warp_id()); row < p.rows; row += PLAN_THREADS / 32) change_row<FORK, 32>(p, row, int(lane_id()));
}

template <bool FORK>
__global__ void __launch_bounds__(ROW_THREADS) rows_kernel(const __grid_constant__ TableParams p) {
  pdl_wait_previous();
  if (*p.short_of == 0) change_row<FORK, ROW_THREADS>(p, int(blockIdx.x), int(threadIdx.x));
}

// ---------------------------------------------------------------- copies of pages
struct CopyParams {
  int64_t page_stride, head_stride, token_stride;
  int32_t pages, ps, Hkv, heads;  // heads: of one block
  const int32_t* src;
  const int32_t* dst;
  const int32_t* slots;
  const int32_t* count;
  uint32_t* status;
  Layer layers[LAYERS];
};

// One page's keys or values of some heads to a block: (copy, layer and keys or values, heads).
template <int D>
__global__ void __launch_bounds__(COPY_THREADS) copy_pages_kernel(const __grid_constant__ CopyParams p) {
  const int n = blockIdx.x, tid = threadIdx.x;
  if (p.count && n >= *p.count) return;
  const int src = p.src[n], dst = p.dst[n], slots = p.slots ? p.slots[n] : p.ps;
  if (src < 0 || src >= p.pages || dst < 0 || dst >= p.pages || slots < 0 || slots > p.ps) {
    if (tid == 0) record_error(p.status, kKvInvalid, uint32_t(n), uint32_t(src), uint32_t(dst));
    return;
  }
  if (src == dst) return;
  const Layer& l = p.layers[blockIdx.y >> 1];
  const bool values = blockIdx.y & 1;
  const int h0 = int(blockIdx.z) * p.heads, heads = min(p.heads, p.Hkv - h0);
  uint8_t* pool = values ? l.v : l.k;
  uint8_t* scales = values ? l.vs : l.ks;
  for (int h = tid; h < heads; h += COPY_THREADS)
    scales[int64_t(dst) * p.Hkv + h0 + h] = scales[int64_t(src) * p.Hkv + h0 + h];
  if (slots == 0) return;
  constexpr int UNITS = D / 16, BATCH = 8, STEP = COPY_THREADS / UNITS;  // rows of a pass
  const uint8_t* from = pool + int64_t(src) * p.page_stride + h0 * p.head_stride + tid % UNITS * 16;
  uint8_t* to = pool + int64_t(dst) * p.page_stride + h0 * p.head_stride + tid % UNITS * 16;
  // a thread's rows, counted on through the heads (by divisions the copies of 512 beams, 54 MB, took 12.4 us and not 10.3)
  int h = 0, row = tid / UNITS;
  auto settle = [&]() {
    while (row >= slots) {
      row -= slots;
      ++h;
    }
  };
  settle();
  while (h < heads) {
    uint4 w[BATCH];
    int64_t at[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      at[k] = -1;
      if (h < heads) {
        at[k] = h * p.head_stride + row * p.token_stride;
        w[k] = __ldg(reinterpret_cast<const uint4*>(from + at[k]));
        row += STEP;
        settle();
      }
    }
#pragma unroll
    for (int k = 0; k < BATCH; ++k)
      if (at[k] >= 0) *reinterpret_cast<uint4*>(to + at[k]) = w[k];
  }
}

// ---------------------------------------------------------------- accepted drafts move together
struct CompactParams {
  int64_t page_stride, head_stride, token_stride;
  int32_t pages, ps, Hkv, max_kept;
  KvBatch b;
  const int32_t* kept;
  const int32_t* n_kept;
  int32_t* lens_out;  // written by the first layers' launch; NULL in the others
  Layer layers[LAYERS];
};

// The factor that brings codes of scale byte `from` to byte `to` >= from.  (255 is NaN and stays: the codes do not matter.)
__device__ __forceinline__ float recode_factor(int from, int to) { return to == 255 ? 1.0f : pow2f(max(from - to, -127)); }

// A warp to a sequence's keys and values of one head and layer (one search for both: 64 trees of up to 60 in 8 layers 12.4 -> 10.5 us).
// Token kept[i] goes to place i; places rise with i and lie at or below the tokens, so in ascending order, each batch
// read before it is written, nothing is lost.
template <int D>
__global__ void __launch_bounds__(COPY_THREADS) compact_kernel(const __grid_constant__ CompactParams p) {
  constexpr int UNITS = D / 16, RPP = 32 / UNITS, BATCH = 2;  // rows of a pass; passes on their way at once
  const int s = blockIdx.x, lane = int(lane_id());
  const int head = int(blockIdx.y) * (COPY_THREADS / 32) + int(warp_id());
  const KvSeq seq = kv_seq(p.b, p.ps, s);
  const int start = seq.len - seq.q, n = p.n_kept[s];
  const int32_t* kept = p.kept + int64_t(s) * p.max_kept;
  bool bad = start < 0 || n < 0 || n > seq.q || n > p.max_kept;
  if (!bad) {
    for (int i = lane; i < n; i += 32) bad |= kept[i] >= seq.q || kept[i] <= (i ? kept[i - 1] : -1);
    bad = __any_sync(0xffffffffu, bad);
  }
  if (head == 0 && blockIdx.z == 0 && lane == 0) {
    if (bad) record_error(p.b.status, kKvInvalid, uint32_t(s), uint32_t(n), uint32_t(seq.q));
    if (p.lens_out) p.lens_out[s] = bad ? seq.len : start + n;
  }
  if (bad || n == 0 || head >= p.Hkv) return;
  const Layer& l = p.layers[blockIdx.z];
  uint8_t* const codes[2] = {l.k + head * p.head_stride, l.v + head * p.head_stride};
  uint8_t* const scales[2] = {l.ks + head, l.vs + head};
  const int32_t* table = p.b.table + int64_t(s) * p.b.max_pages;
  auto page_at = [&](int no) {
    const int page = table[no];
    if (page >= 0 && page < p.pages) return page;
    record_error(p.b.status, kKvInvalid, uint32_t(s), uint32_t(page), uint32_t(no));
    return -1;
  };
  const int unit = lane % UNITS * 16, row = lane / UNITS;
  for (int i0 = 0; i0 < n;) {
    const int no = (start + i0) / p.ps, base = no * p.ps;
    const int i1 = min(n, base + p.ps - start);  // those that go to this page
    const int page = page_at(no);
    if (page < 0) return;
    // a lane's token: where it lies in the pool and its scales
    int64_t of = -1;
    int sc[2], old[2], most[2];
    auto look_up = [&](int i) {
      of = -1;
      sc[0] = sc[1] = 0;
      if (i < i1) {
        const int pos = start + kept[i], from = page_at(pos / p.ps);
        if (from >= 0) {
          of = int64_t(from) * p.page_stride + int64_t(pos % p.ps) * p.token_stride;
          sc[0] = scales[0][int64_t(from) * p.Hkv];
          sc[1] = scales[1][int64_t(from) * p.Hkv];
        }
      }
    };
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      old[x] = scales[x][int64_t(page) * p.Hkv];
      most[x] = start + i0 > base ? old[x] : 0;
    }
    for (int c = i0; c < i1; c += 32) {
      look_up(c + lane);
#pragma unroll
      for (int x = 0; x < 2; ++x) most[x] = max(most[x], int(__reduce_max_sync(0xffffffffu, uint32_t(sc[x]))));
    }
    const int64_t page_at0 = int64_t(page) * p.page_stride;
#pragma unroll 1
    for (int x = 0; x < 2; ++x) {
      const int now = x ? most[1] : most[0], was = x ? old[1] : old[0];
      if (now <= was || now == 255) continue;
      const float f = recode_factor(was, now);
      for (int r = row; r < start + i0 - base; r += RPP) {
        uint4* at = reinterpret_cast<uint4*>((x ? codes[1] : codes[0]) + page_at0 + r * p.token_stride + unit);
        *at = recode16(*at, f);
      }
    }
    const bool again = i1 - i0 > 32;
    for (int c = i0; c < i1; c += 32) {
      if (again) look_up(c + lane);
      // (a page's own scale byte is written once all is read: it is what its tokens are in until then)
      for (int k0 = 0; k0 < min(32, i1 - c); k0 += RPP * BATCH) {
        uint4 w[BATCH][2];
        bool move[BATCH][2];
        int b[BATCH][2];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
          const int i = k0 + k * RPP + row;
          const int64_t from = __shfl_sync(0xffffffffu, of, i & 31);
          const bool here = i < 32 && c + i < i1 && from >= 0, moves = from != page_at0 + (start + c + i - base) * p.token_stride;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            b[k][x] = __shfl_sync(0xffffffffu, sc[x], i & 31);
            move[k][x] = here && (moves || b[k][x] != most[x]);
            if (move[k][x]) w[k][x] = *reinterpret_cast<const uint4*>(codes[x] + from + unit);
          }
        }
#pragma unroll
        for (int k = 0; k < BATCH; ++k)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            if (move[k][x] && b[k][x] != most[x]) w[k][x] = recode16(w[k][x], recode_factor(b[k][x], most[x]));
        __syncwarp();
#pragma unroll
        for (int k = 0; k < BATCH; ++k)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            if (move[k][x])
              *reinterpret_cast<uint4*>(codes[x] + page_at0 + (start + c + k0 + k * RPP + row - base) * p.token_stride + unit) = w[k][x];
        __syncwarp();
      }
    }
    __syncwarp();
    if (lane < 2) (lane ? scales[1] : scales[0])[int64_t(page) * p.Hkv] = uint8_t(lane ? most[1] : most[0]);
    __syncwarp();
    i0 = i1;
  }
}

// ---------------------------------------------------------------- checks
tl_status check_layers(const char* who, const tl_kv_cache* caches, int n) {
  if (!caches || n < 1) return fail(TL_ERR_INVALID, "%s: no caches", who);
  if (n > 4096) return fail(TL_ERR_UNSUPPORTED, "%s: %d layers (at most 4096)", who, n);
  const tl_kv_cache& c = caches[0];
  for (int i = 0; i < n; ++i) {
    if (tl_status s = check_kv_cache(who, caches[i])) return s;
    const tl_kv_cache& d = caches[i];
    if (d.page_stride != c.page_stride || d.head_stride != c.head_stride || d.token_stride != c.token_stride ||
        d.num_pages != c.num_pages || d.page_size != c.page_size || d.H_kv != c.H_kv || d.head_dim != c.head_dim)
      return fail(TL_ERR_INVALID, "%s: layer %d's cache is not laid out as the first one's", who, i);
  }
  return TL_OK;
}

// Whether two of the caches are one: it would be written twice at once.
bool a_cache_twice(const tl_kv_cache* caches, int n) {
  const void* all[4096];
  for (const auto side : {&tl_kv_cache::k, &tl_kv_cache::v}) {
    for (int i = 0; i < n; ++i) all[i] = caches[i].*side;
    std::sort(all, all + n, std::less<const void*>());
    if (std::adjacent_find(all, all + n) != all + n) return true;
  }
  return false;
}

// Runs launch(params, first layer) for each LAYERS of them.
template <class P, class F>
tl_status by_layers(P& p, const tl_kv_cache* caches, int n, F launch) {
  for (int at = 0; at < n; at += LAYERS) {
    const int some = std::min(LAYERS, n - at);
    for (int i = 0; i < some; ++i)
      p.layers[i] = Layer{static_cast<uint8_t*>(caches[at + i].k), static_cast<uint8_t*>(caches[at + i].v),
                          caches[at + i].k_scale, caches[at + i].v_scale};
    if (tl_status s = launch(some)) return s;
  }
  return TL_OK;
}

tl_status check_table(const char* who, int B, int max_pages, int page_size, int num_pages) {
  if (B < 1 || B > (1 << 20) || max_pages < 1 || num_pages < 1)
    return fail(TL_ERR_INVALID, "%s: %d sequences, max_pages %d, num_pages %d", who, B, max_pages, num_pages);
  if (page_size < 16 || page_size > 256 || page_size % 16)
    return fail(TL_ERR_UNSUPPORTED, "%s: page_size %d (a multiple of 16, 16..256)", who, page_size);
  if (int64_t(max_pages) * page_size > 0x7FFFFF00ll) return fail(TL_ERR_UNSUPPORTED, "%s: max_pages %d", who, max_pages);
  return TL_OK;
}

size_t table_workspace(int64_t ints) { return size_t(ints * 4 + 64 + 255) / 256 * 256; }

tl_status plan(const char* who, TableParams& p, int rows, bool fork, cudaStream_t st, int sms) {
  void* args[] = {&p};
  const void* first = fork ? reinterpret_cast<const void*>(&plan_kernel<true>) : reinterpret_cast<const void*>(&plan_kernel<false>);
  // One block does it all where a warp has 8 rows at most, of 512 entries, and the counts fit in 16 a thread: a launch less
  // (four beams 9.9 -> 7.4 us a call, 64 sequences cut 7.9 -> 5.7 us).
  const bool apart = p.refs != p.refs_out;
  if (rows <= 8 * (PLAN_THREADS / 32) && p.max_pages <= 512 && (!apart || p.pages <= 16 * PLAN_THREADS)) {
    p.rows = rows;
    return launch(first, 1, PLAN_THREADS, 0, st, args, false);
  }
  // the counts' copy: four to a thread
  const int blocks = 1 + (apart ? std::min(sms - 1, cdiv(p.pages, 4 * PLAN_THREADS)) : 0);
  if (tl_status s = launch(first, blocks, PLAN_THREADS, 0, st, args, false)) return s;
  const void* second = fork ? reinterpret_cast<const void*>(&rows_kernel<true>) : reinterpret_cast<const void*>(&rows_kernel<false>);
  return launch(second, rows, ROW_THREADS, 0, st, args, true);
}

}  // namespace
}  // namespace tl

extern "C" size_t tl_kv_fork_workspace_size(int B_in, int B_out) {
  if (B_in < 1 || B_out < 1 || B_in > (1 << 20) || B_out > (1 << 20)) return 0;
  return tl::table_workspace(2 * int64_t(B_in) + B_out);
}

extern "C" tl_status tl_kv_fork(const tl_kv_fork_args* a, void* stream) {
  using namespace tl;
  const char* who = "tl_kv_fork";
  if (!a) return fail(TL_ERR_INVALID, "%s: NULL args", who);
  if (tl_status s = check_table(who, a->B_in, a->max_pages, a->page_size, a->num_pages)) return s;
  if (tl_status s = check_table(who, a->B_out, a->max_pages, a->page_size, a->num_pages)) return s;
  if (!a->page_table || !a->seq_lens || !a->refs || !a->parents || !a->page_table_out || !a->seq_lens_out || !a->refs_out ||
      !a->copies || !a->n_copies || !a->workspace || !a->signals)
    return fail(TL_ERR_INVALID, "%s: NULL pointer argument", who);
  if (!aligned16(a->refs) || !aligned16(a->workspace))
    return fail(TL_ERR_INVALID, "%s: refs and workspace must be 16-byte aligned", who);
  if (a->workspace_bytes < tl_kv_fork_workspace_size(a->B_in, a->B_out))
    return fail(TL_ERR_INVALID, "%s: workspace of %zu bytes, need %zu", who, a->workspace_bytes,
                tl_kv_fork_workspace_size(a->B_in, a->B_out));
  const int64_t in = int64_t(a->B_in) * a->max_pages * 4, out = int64_t(a->B_out) * a->max_pages * 4;
  if (ranges_meet(a->page_table, in, a->page_table_out, out) || ranges_meet(a->seq_lens, a->B_in * 4ll, a->seq_lens_out, a->B_out * 4ll))
    return fail(TL_ERR_INVALID, "%s: the new table and lengths overlap the old ones", who);
  if (a->refs != a->refs_out && ranges_meet(a->refs, a->num_pages * 4ll, a->refs_out, a->num_pages * 4ll))
    return fail(TL_ERR_INVALID, "%s: refs_out overlaps refs", who);
  DeviceInfo di{};
  if (tl_status s = device_info(&di)) return s;
  if (a->signals->device != di.device) return fail(TL_ERR_INVALID, "%s: signals belong to another device", who);
  TableParams p{};
  p.table = a->page_table;
  p.lens = a->seq_lens;
  p.to = a->parents;
  p.refs = a->refs;
  p.table_out = a->page_table_out;
  p.lens_out = a->seq_lens_out;
  p.refs_out = a->refs_out;
  p.copies = a->copies;
  p.n_copies = a->n_copies;
  p.short_of = static_cast<int32_t*>(a->workspace);
  p.first = p.short_of + 16;
  p.count = p.first + a->B_in;
  p.base = p.count + a->B_in;
  p.status = a->signals->status;
  p.B_in = a->B_in;
  p.B_out = a->B_out;
  p.max_pages = a->max_pages;
  p.ps = a->page_size;
  p.pages = a->num_pages;
  return plan(who, p, a->B_in + a->B_out, true, static_cast<cudaStream_t>(stream), di.sm_count);
}

extern "C" size_t tl_kv_resize_workspace_size(int B) {
  if (B < 1 || B > (1 << 20)) return 0;
  return tl::table_workspace(B);
}

extern "C" tl_status tl_kv_resize(const tl_kv_resize_args* a, void* stream) {
  using namespace tl;
  const char* who = "tl_kv_resize";
  if (!a) return fail(TL_ERR_INVALID, "%s: NULL args", who);
  if (tl_status s = check_table(who, a->B, a->max_pages, a->page_size, a->num_pages)) return s;
  if (!a->page_table || !a->seq_lens || !a->new_lens || !a->refs || !a->refs_out || !a->workspace || !a->signals)
    return fail(TL_ERR_INVALID, "%s: NULL pointer argument", who);
  if (!aligned16(a->refs) || !aligned16(a->workspace))
    return fail(TL_ERR_INVALID, "%s: refs and workspace must be 16-byte aligned", who);
  if (a->workspace_bytes < tl_kv_resize_workspace_size(a->B))
    return fail(TL_ERR_INVALID, "%s: workspace of %zu bytes, need %zu", who, a->workspace_bytes, tl_kv_resize_workspace_size(a->B));
  if (a->refs != a->refs_out && ranges_meet(a->refs, a->num_pages * 4ll, a->refs_out, a->num_pages * 4ll))
    return fail(TL_ERR_INVALID, "%s: refs_out overlaps refs", who);
  DeviceInfo di{};
  if (tl_status s = device_info(&di)) return s;
  if (a->signals->device != di.device) return fail(TL_ERR_INVALID, "%s: signals belong to another device", who);
  TableParams p{};
  p.table = p.table_out = a->page_table;
  p.lens = a->seq_lens;
  p.to = a->new_lens;
  p.refs = a->refs;
  p.refs_out = a->refs_out;
  p.short_of = static_cast<int32_t*>(a->workspace);
  p.base = p.short_of + 16;
  p.status = a->signals->status;
  p.B_in = p.B_out = a->B;
  p.max_pages = a->max_pages;
  p.ps = a->page_size;
  p.pages = a->num_pages;
  return plan(who, p, a->B, false, static_cast<cudaStream_t>(stream), di.sm_count);
}

extern "C" tl_status tl_kv_copy_pages(const tl_kv_copy_pages_args* a, void* stream) {
  using namespace tl;
  const char* who = "tl_kv_copy_pages";
  if (!a) return fail(TL_ERR_INVALID, "%s: NULL args", who);
  if (tl_status s = check_layers(who, a->caches, a->n_layers)) return s;
  if (a->n < 0) return fail(TL_ERR_INVALID, "%s: %d copies", who, a->n);
  if (!a->signals) return fail(TL_ERR_INVALID, "%s: NULL pointer argument", who);
  if (a->n == 0) return TL_OK;
  if (!a->src || !a->dst) return fail(TL_ERR_INVALID, "%s: NULL pointer argument", who);
  DeviceInfo di{};
  if (tl_status s = device_info(&di)) return s;
  if (a->signals->device != di.device) return fail(TL_ERR_INVALID, "%s: signals belong to another device", who);
  const tl_kv_cache& c = a->caches[0];
  CopyParams p{};
  p.page_stride = c.page_stride;
  p.head_stride = c.head_stride;
  p.token_stride = c.token_stride;
  p.pages = c.num_pages;
  p.ps = c.page_size;
  p.Hkv = c.H_kv;
  p.heads = std::max(1, 16384 / (c.page_size * c.head_dim));  // 16 KB to a block: its threads' loads once over
  p.src = a->src;
  p.dst = a->dst;
  p.slots = a->slots;
  p.count = a->count;
  p.status = a->signals->status;
  return by_layers(p, a->caches, a->n_layers, [&](int layers) {
    const dim3 grid(unsigned(a->n), unsigned(2 * layers), unsigned(cdiv(c.H_kv, p.heads)));
    if (c.head_dim == 128) copy_pages_kernel<128><<<grid, COPY_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(p);
    else copy_pages_kernel<64><<<grid, COPY_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return cuda_ok(cudaGetLastError(), who);
  });
}

extern "C" tl_status tl_kv_compact(const tl_kv_compact_args* a, void* stream) {
  using namespace tl;
  const char* who = "tl_kv_compact";
  if (!a) return fail(TL_ERR_INVALID, "%s: NULL args", who);
  if (tl_status s = check_layers(who, a->caches, a->n_layers)) return s;
  if (a->B < 1 || a->B > (1 << 20) || a->max_pages < 1 || a->max_kept < 1)
    return fail(TL_ERR_INVALID, "%s: B %d, max_pages %d, max_kept %d", who, a->B, a->max_pages, a->max_kept);
  if (!a->kept || !a->n_kept || !a->cu_seqlens || !a->seq_lens || !a->page_table || !a->seq_lens_out || !a->signals)
    return fail(TL_ERR_INVALID, "%s: NULL pointer argument", who);
  if (ranges_meet(a->seq_lens, a->B * 4ll, a->seq_lens_out, a->B * 4ll))
    return fail(TL_ERR_INVALID, "%s: seq_lens_out overlaps seq_lens", who);
  if (a_cache_twice(a->caches, a->n_layers)) return fail(TL_ERR_INVALID, "%s: a cache is given twice", who);
  DeviceInfo di{};
  if (tl_status s = device_info(&di)) return s;
  if (a->signals->device != di.device) return fail(TL_ERR_INVALID, "%s: signals belong to another device", who);
  const tl_kv_cache& c = a->caches[0];
  CompactParams p{};
  p.page_stride = c.page_stride;
  p.head_stride = c.head_stride;
  p.token_stride = c.token_stride;
  p.pages = c.num_pages;
  p.ps = c.page_size;
  p.Hkv = c.H_kv;
  p.max_kept = a->max_kept;
  p.b = KvBatch{a->cu_seqlens, a->seq_lens, a->page_table, a->signals->status, a->B, 0x7FFFFFFF, a->max_pages};
  p.kept = a->kept;
  p.n_kept = a->n_kept;
  p.lens_out = a->seq_lens_out;
  return by_layers(p, a->caches, a->n_layers, [&](int layers) {
    const dim3 grid(unsigned(a->B), unsigned(cdiv(c.H_kv, COPY_THREADS / 32)), unsigned(layers));
    if (c.head_dim == 128) compact_kernel<128><<<grid, COPY_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(p);
    else compact_kernel<64><<<grid, COPY_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(p);
    p.lens_out = nullptr;
    return cuda_ok(cudaGetLastError(), who);
  });
}
