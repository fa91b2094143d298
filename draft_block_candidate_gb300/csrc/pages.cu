// Pages of the 8-bit cache that sequences share: who holds them, what is done when hypotheses fork,
// grow and end, and the moving of their contents.
//
// refs[p] is how many entries of block tables name page p; a page with none is free.  An entry of a
// table is the page that its row holds there, or negative.  All that is decided here is whole numbers
// and follows from the order of rows, columns and pages alone, so the same call leaves the same state
// whatever the order in which its threads run.
#include <cooperative_groups.h>

#include <algorithm>
#include <climits>

#include "kv8.cuh"

namespace lilicorr {

namespace cg = cooperative_groups;

static __device__ uint32_t g_err_pages;

// ------------------------------------------------------------------------------------ fork
// Row (b, j) of the tables becomes row (b, parent[b, j]).  A row that c others (itself among them)
// go on from leaves its pages with c - 1 more holders.  A thread for each column of a batch entry
// reads all its beams' entries before it writes any, so the tables are gathered in place.  Bound by
// latency (parents, entries, atomic adds to refs): 64 x 16 rows of 512 columns 6 us, 4 rows 2.5.  W
// beams' entries are under way together; 4, 8, 16 and 32 of them, so that few beams hold few registers.
constexpr int FK_THREADS = 128, FK_MAX = 32;

template <int W>
__global__ void __launch_bounds__(FK_THREADS) page_fork_kernel(int32_t* __restrict__ refs, int64_t n_pages, int32_t* __restrict__ table,
                                                               int64_t batch_stride, int64_t row_stride, int cols, int tiles,
                                                               const int32_t* __restrict__ parent, int beams) {
  __shared__ int s_par[W], s_times[W];
  __shared__ int32_t s_old[W][FK_THREADS];
  const int tid = threadIdx.x;
  const int64_t b = blockIdx.x / tiles;
  const int col = static_cast<int>(blockIdx.x - b * tiles) * FK_THREADS + tid;
  if (tid < W) s_times[tid] = 0;
  __syncthreads();
  if (tid < beams) {
    int q = __ldg(parent + b * beams + tid);
    if (q < 0 || q >= beams) {  // no such beam: the row stays as it is
      if (col == tid) atomicOr(&g_err_pages, ERR_BEAM_PARENT);
      q = tid;
    }
    s_par[tid] = q;
    atomicAdd(&s_times[q], 1);
  }
  __syncthreads();
  if (col >= cols) return;
  int32_t* at = table + b * batch_stride + col;
  int32_t v[W];
#pragma unroll
  for (int j = 0; j < W; ++j)
    if (j < beams && !(s_times[j] == 1 && s_par[j] == j)) v[j] = at[j * row_stride];
#pragma unroll
  for (int j = 0; j < W; ++j)
    if (j < beams && !(s_times[j] == 1 && s_par[j] == j)) {
      s_old[j][tid] = v[j];
      const int more = s_times[j] - 1;
      if (more != 0 && v[j] >= 0) {
        if (v[j] >= n_pages) atomicOr(&g_err_pages, ERR_KV8_PAGE);
        else atomicAdd(refs + v[j], more);
      }
    }
#pragma unroll
  for (int j = 0; j < W; ++j)
    if (j < beams && s_par[j] != j) at[j * row_stride] = s_old[s_par[j]][tid];
}

// ------------------------------------------------------------------------------------ free
// Pages behind a row's first keep[r] tokens lose a holder, and their entries become -1.  A thread an
// entry; bound by latency: 1,024 rows of 512 columns 5 us, 4 rows 3.
constexpr int FR_THREADS = 256;

__global__ void __launch_bounds__(FR_THREADS) page_free_kernel(int32_t* refs, int64_t n_pages, int32_t* table, int64_t row_stride, int cols,
                                                               int tiles, const int32_t* __restrict__ keep, int page) {
  const int64_t r = blockIdx.x / tiles;
  const int col = static_cast<int>(blockIdx.x - r * tiles) * FR_THREADS + threadIdx.x;
  const int k = __ldg(keep + r);
  if (k < 0) {
    if (col == 0) atomicOr(&g_err_pages, ERR_KV8_LENGTH);
    return;
  }
  if (col >= cols || int64_t(col) * page < k) return;
  int32_t* at = table + r * row_stride + col;
  const int id = *at;
  if (id < 0) return;
  *at = -1;
  if (id >= n_pages) {
    atomicOr(&g_err_pages, ERR_KV8_PAGE);
  } else if (atomicSub(refs + id, 1) <= 0) {  // nobody held it
    atomicAdd(refs + id, 1);
    atomicOr(&g_err_pages, ERR_KV8_PAGE);
  }
}

// ------------------------------------------------------------- what the whole pool decides
// Two kernels number pages in their order: a run of pages (and of rows) for each warp of one cluster of CL_CTAS
// CTAs, counts exchanged through distributed shared memory; or of one CTA alone, where a pool is so small that the
// cluster's barriers cost more than they save.
constexpr int CL_CTAS = 8, CL_WARPS = 16, CL_THREADS = 32 * CL_WARPS;
// One CTA's pages, and columns that rows write, at most.  Measured: compaction of 1,500, 3,000 and 4,096 pages 10.9, 11.6
// and 12.0 us by one, 13.9, 14.5 and 14.6 by eight; a step of 216 rows of two columns 14.7 and 17.1, of 621 20.1 and 17.1.
constexpr int CL_SMALL = 4096, CL_SMALL_COLUMNS = 768;

template <int CTAS>
__device__ __forceinline__ int cluster_rank() {
  return CTAS == 1 ? 0 : static_cast<int>(cg::this_cluster().block_rank());
}
template <int CTAS>
__device__ __forceinline__ void cluster_sync() {
  if (CTAS == 1) __syncthreads();
  else cg::this_cluster().sync();
}
// Sums of `mine` (a warp's, the same in its lanes) over the warps before this one, and over all.  Every thread of
// the cluster calls it; a is shared memory of CL_WARPS values.
struct Counts {
  int64_t x;  // rows may want more pages than there are
  int y;
};
struct Place {
  Counts before, all;
};
__device__ __forceinline__ int64_t warp_sum(int64_t v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(FULL_MASK, v, o);
  return v;
}
template <int CTAS>
__device__ __forceinline__ Place cluster_place(Counts mine, Counts* a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, me = cluster_rank<CTAS>() * CL_WARPS + warp;
  if (lane == 0) a[warp] = mine;
  cluster_sync<CTAS>();
  Counts sum{0, 0}, before = sum;
#pragma unroll
  for (int i = 0; i < (CTAS * CL_WARPS + 31) / 32; ++i) {
    const int w = i * 32 + lane;
    if (w < CTAS * CL_WARPS) {
      const Counts v = CTAS == 1 ? a[w] : *cg::this_cluster().map_shared_rank(a + w % CL_WARPS, w / CL_WARPS);
      sum.x += v.x;
      sum.y += v.y;
      if (w < me) {
        before.x += v.x;
        before.y += v.y;
      }
    }
  }
  return Place{{warp_sum(before.x), __reduce_add_sync(FULL_MASK, before.y)}, {warp_sum(sum.x), __reduce_add_sync(FULL_MASK, sum.y)}};
}

// Calls f(page, holders) for the pages of [lo, hi), 32 lanes side by side, UNROLL reads under way;
// every lane calls it the same number of times (page >= hi: none).
template <int UNROLL, typename F>
__device__ __forceinline__ void each_page(const int32_t* refs, int64_t lo, int64_t hi, F f) {
  const int lane = threadIdx.x & 31;
  for (int64_t p0 = lo; p0 < hi; p0 += 32 * UNROLL) {
    int v[UNROLL];
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
      const int64_t p = p0 + i * 32 + lane;
      v[i] = p < hi ? __ldcg(refs + p) : -1;
    }
#pragma unroll
    for (int i = 0; i < UNROLL; ++i)
      if (p0 + i * 32 < hi) f(p0 + i * 32 + lane, v[i], p0 + i * 32 + lane < hi);
  }
}

// ------------------------------------------------------------------------------------ grow
// Row r writes tokens kv_len[r] .. kv_len[r] + new[r] - 1 next.  Each column that they touch needs a
// page of the row's own: where it holds none, or one that others hold too, it takes a free one.  Free
// pages are taken lowest first, in the order of rows and columns.
//
// Rows are written where they get their pages and nowhere else.  Until the pages are dealt the workspace says
// which columns take one: a bit of a row's word for each where no row writes more than 31, else by how many
// held each page before the call (by those counts alone a step of 1,024 rows took 18.7 us for 18.0).
//
// Bound by its dependent reads and its barriers: 1,024 rows of 16 new tokens on a pool of 52,396 pages 13 us,
// 4 rows on a small one 5.5; every count is read, so that a step of 4 rows on a pool of 300,000 takes 23.5 us in
// all.  Pages and rows are counted behind one barrier (with one for each, a small step's three kernels took 12.4 us
// for 8.3).
struct GrowParams {
  int32_t* refs;
  int64_t n_pages;
  int32_t* table;
  int64_t row_stride, rows;
  int cols, page, max_new;
  const int32_t *kv_len, *fresh;
  int32_t* tail_src;
  uint8_t* granted;
  int32_t *need, *list, *held;  // workspace: [rows] columns that take a page, or how many; [n_pages]; [n_pages]
  int steps;                    // columns that a row writes, at most
  int group_log2;               // lanes of a row
};

template <int CTAS>
__global__ void __launch_bounds__(CL_THREADS) page_grow_kernel(const GrowParams p) {
  constexpr int ALL = CTAS * CL_WARPS;
  __shared__ Counts s_a[CL_WARPS];
  const int lane = threadIdx.x & 31, w = cluster_rank<CTAS>() * CL_WARPS + (threadIdx.x >> 5);
  const int G = 1 << p.group_log2, sub = lane >> p.group_log2, in = lane & (G - 1), per = 32 >> p.group_log2;
  // this warp's pages: how many are free
  const int64_t some = ((p.n_pages + ALL - 1) / ALL + 31) / 32 * 32;
  const int64_t p0 = min(p.n_pages, w * some), p1 = min(p.n_pages, p0 + some);
  int free = 0;
  each_page<8>(p.refs, p0, p1, [&](int64_t, int v, bool in_run) { free += in_run && v == 0; });
  free = __reduce_add_sync(FULL_MASK, free);
  // this warp's rows
  const int64_t each = ((p.rows + ALL - 1) / ALL + per - 1) / per * per;
  const int64_t r0 = min(p.rows, w * each), r1 = min(p.rows, r0 + each);
  // columns [c0, c1) that row r writes; whether the first one holds tokens before
  struct Span {
    int c0, c1;
    bool ok, tail;
  };
  auto span = [&](int64_t r) {
    Span s{0, 0, true, false};
    const int len = __ldg(p.kv_len + r), n = __ldg(p.fresh + r);
    if (len < 0 || n < 0 || n > p.max_new || int64_t(len) + n > int64_t(p.cols) * p.page) {
      s.ok = false;
    } else if (n > 0) {
      s.c0 = len / p.page;
      s.c1 = (len + n + p.page - 1) / p.page;  // (below 2^31: host)
      s.tail = len % p.page != 0;
    }
    return s;
  };
  auto sum_group = [&](int v) {
    for (int o = G / 2; o >= 1; o >>= 1) v += __shfl_xor_sync(FULL_MASK, v, o);
    return v;
  };
  const bool bits = p.steps <= 31;  // (and so a column a lane)
  auto pages_of = [&](int need) { return need < 0 ? 0 : bits ? __popc(need) : need; };
  int64_t mine = 0;
  for (int64_t rb = r0; rb < r1; rb += per) {
    const int64_t r = rb + sub;
    Span s{0, 0, true, false};
    if (r < r1) s = span(r);
    int32_t* row = p.table + r * p.row_stride;
    uint32_t err = s.ok ? 0u : uint32_t(ERR_KV8_LENGTH);
    // a column's page, and how many hold it (a lane's first column, which mostly is its only one, is kept)
    int id0 = 0, held0 = 1;
    if (s.ok)
      for (int c = s.c0 + in; c < s.c1; c += G) {
        const int id = row[c];
        int held = 0;
        if (id >= p.n_pages || (id < 0 && s.tail && c == s.c0) || (id >= 0 && (held = __ldcg(p.refs + id)) < 1)) err = ERR_KV8_PAGE;
        if (c < s.c0 + G) {
          id0 = id;
          held0 = held;
        }
      }
    const bool ok = sum_group(err != 0) == 0;
    if (err) atomicOr(&g_err_pages, err);
    int need = 0;
    if (ok)
      for (int c = s.c0 + in; c < s.c1; c += G) {
        const bool kept = c < s.c0 + G;
        const int id = kept ? id0 : row[c];
        if (id >= 0) {
          const int held = kept ? held0 : __ldcg(p.refs + id);
          if (!bits) p.held[id] = held;  // (the same by whoever comes upon it)
          if (held <= 1) continue;
        }
        need += bits ? 1 << in : 1;
      }
    need = sum_group(need);
    if (r < r1 && in == 0) p.need[r] = ok ? need : -1;
    mine += in == 0 ? pages_of(need) : 0;
  }
  const Place at_w = cluster_place<CTAS>(Counts{warp_sum(mine), free}, s_a);
  const int64_t want = at_w.all.x;
  const int have = at_w.all.y;
  // the free pages that are wanted, in order
  int at = at_w.before.y;
  if (free > 0 && at < want)
    each_page<8>(p.refs, p0, p1, [&](int64_t page, int v, bool in_run) {
      const unsigned b = __ballot_sync(FULL_MASK, in_run && v == 0);
      const int k = at + __popc(b & ((1u << lane) - 1));
      if ((b >> lane & 1) && k < want) p.list[k] = static_cast<int32_t>(page);
      at += __popc(b);
    });
  cluster_sync<CTAS>();  // (the list is there, and nobody reads counts of holders any more)

  int64_t start = at_w.before.x;
  for (int64_t rb = r0; rb < r1; rb += per) {
    const int64_t r = rb + sub;
    const int word = r < r1 ? p.need[r] : 0, need = pages_of(word);
    // where the row's pages begin
    int64_t k = start, all = 0;
    for (int i = 0; i < per; ++i) {
      const int v = __shfl_sync(FULL_MASK, need, i << p.group_log2);
      if (i < sub) k += v;
      all += v;
    }
    start += all;
    const bool ok = word == 0 || (word > 0 && k + need <= have);
    int tail = -1;
    Span s{0, 0, true, false};
    if (r < r1 && need > 0) s = span(r);
    int32_t* row = p.table + r * p.row_stride;
    for (int c0 = 0; c0 < p.steps; c0 += G) {
      const int c = s.c0 + c0 + in;
      const bool here = c < s.c1;
      const int e = here ? row[c] : 0;
      const bool give = here && (bits ? word >> in & 1 : e < 0 || p.held[e] > 1);
      const unsigned b = __ballot_sync(FULL_MASK, give) >> (sub << p.group_log2) & (G == 32 ? FULL_MASK : (1u << G) - 1);
      if (give && ok) {
        const int id = __ldcg(p.list + k + __popc(b & ((1u << in) - 1)));
        row[c] = id;
        p.refs[id] = 1;
        if (e >= 0) {
          atomicSub(p.refs + e, 1);
          if (c == s.c0 && s.tail) tail = e;
        }
      }
      k += __popc(b);
      if (!__any_sync(FULL_MASK, s.c0 + c0 + G < s.c1)) break;
    }
    if (r < r1 && in == 0) {
      p.tail_src[r] = tail;
      p.granted[r] = ok ? 1 : 0;
    }
  }
}

// ---------------------------------------------------------------------------------- moving
// Page src[i] of every cache is copied to page dst[i]; where `count` is given, the first *count of
// them.  A CTA takes a tile of 32 KB of a page, or as many small pages as fill one, at a time, eight
// vectors of a thread under way together.  Bound by HBM: 2,048 pages of 64 KB, keys and values of four
// layers, 341 us, 93 % of the copy rate.  In a compaction src and dst are the kernel's before, which may still
// run when this one starts, so they are read by plain loads behind the wait and not as constants of the kernel's
// life (__ldg); through the L2 cache alone (__ldcg) a tile waits for it first, 507 us.
constexpr int MV_THREADS = 256, MV_VECS = 8, MV_TILE = MV_THREADS * MV_VECS, MV_CACHES = 16, MV_TABLES = 8;

struct MoveCache {
  const uint4 *k, *v;
  uint4 *to_k, *to_v;
  const float *ks, *vs;
  float *to_ks, *to_vs;
};
struct MoveTable {
  const int32_t* from;
  int32_t* to;
  int64_t from_stride, to_stride, rows;
  int cols;
};
struct MoveParams {
  MoveCache c[MV_CACHES];
  int n_caches, heads, vecs;  // vectors of a page
  int tiles, pages;           // of a page, of a tile: one of them is 1
  uint32_t inv;               // 2^32 / vecs, rounded up: e * inv >> 32 is e / vecs for a tile's vectors
  int64_t n_src, n_dst;       // pages of the caches
  const int32_t *src, *dst, *count, *map;
  int64_t n;
  MoveTable t[MV_TABLES];
  int n_tables, table_ctas;
};

__device__ __forceinline__ void move_pages(const MoveParams& p, int cta, int ctas) {
  const int64_t n = p.count ? min(p.n, int64_t(__ldcg(p.count))) : p.n;
  // tiles of one cache's keys, or values
  const int64_t half = p.pages > 1 ? (n + p.pages - 1) / p.pages : n * p.tiles, all = half * p.n_caches * 2;
  int c2 = 0;
  int64_t base = 0;  // of cache and keys or values c2
  for (int64_t tile = cta; tile < all; tile += ctas) {
    while (tile - base >= half) {
      base += half;
      ++c2;
    }
    const int64_t at = tile - base;
    const MoveCache& c = p.c[c2 >> 1];
    const bool is_v = c2 & 1;
    int64_t m0 = at * p.pages;
    uint32_t e0 = 0;
    if (p.tiles > 1) {
      m0 = at < UINT_MAX ? static_cast<uint32_t>(at) / static_cast<uint32_t>(p.tiles) : at / p.tiles;
      e0 = static_cast<uint32_t>(at - m0 * p.tiles) * MV_TILE;
    }
    uint4 w[MV_VECS];
    uint4* to[MV_VECS];
#pragma unroll
    for (int i = 0; i < MV_VECS; ++i) {
      uint32_t e = e0 + i * MV_THREADS + threadIdx.x;
      int64_t m = m0;
      to[i] = nullptr;
      if (p.pages > 1) {
        const uint32_t k = __umulhi(e, p.inv);
        e -= k * p.vecs;
        m += k;
        if (k >= static_cast<uint32_t>(p.pages) || m >= n) continue;
      } else if (e >= static_cast<uint32_t>(p.vecs)) {
        continue;
      }
      const int a = p.src[m], b = p.dst[m];
      if (a >= p.n_src || b >= p.n_dst) {
        if (e == 0) atomicOr(&g_err_pages, ERR_KV8_PAGE);
        continue;
      }
      if (a < 0 || b < 0) continue;
      w[i] = __ldcs((is_v ? c.v : c.k) + int64_t(a) * p.vecs + e);
      to[i] = (is_v ? c.to_v : c.to_k) + int64_t(b) * p.vecs + e;
      if (e < static_cast<uint32_t>(p.heads))  // (a page has more vectors than heads)
        (is_v ? c.to_vs : c.to_ks)[int64_t(b) * p.heads + e] = (is_v ? c.vs : c.ks)[int64_t(a) * p.heads + e];
    }
#pragma unroll
    for (int i = 0; i < MV_VECS; ++i)
      if (to[i]) __stcs(to[i], w[i]);
  }
}

__global__ void __launch_bounds__(MV_THREADS) page_copy_kernel(const __grid_constant__ MoveParams p) { move_pages(p, blockIdx.x, gridDim.x); }

// After page_plan_kernel: entries of the tables take their pages' new places, and the pages move.
__global__ void __launch_bounds__(MV_THREADS) page_compact_kernel(const __grid_constant__ MoveParams p, const int32_t* live) {
  pdl_wait();
  if (static_cast<int>(blockIdx.x) >= p.table_ctas) {
    move_pages(p, blockIdx.x - p.table_ctas, gridDim.x - p.table_ctas);
    return;
  }
  const int n_live = __ldcg(live);
  for (int i = 0; i < p.n_tables; ++i) {
    const MoveTable& t = p.t[i];
    const int64_t all = t.rows * t.cols;
    for (int64_t e = int64_t(blockIdx.x) * MV_THREADS + threadIdx.x; e < all; e += int64_t(p.table_ctas) * MV_THREADS) {
      const int64_t r = e / t.cols, c = e - r * t.cols;
      int id = t.from[r * t.from_stride + c];
      if (id >= n_live) {
        if (id >= p.n_src) atomicOr(&g_err_pages, ERR_KV8_PAGE);
        else if ((id = __ldcg(p.map + id)) < 0) {  // an entry of a page that nobody holds
          atomicOr(&g_err_pages, ERR_KV8_PAGE);
          id = t.from[r * t.from_stride + c];
        }
      }
      t.to[r * t.to_stride + c] = id;
    }
  }
}

// The moves that bring the L live pages to 0 .. L - 1: the i-th live page from L on goes to the i-th
// free page below L.  Bound by its passes over refs and its barriers: 9 us for 4,096 pages, 4.5 for 64.
struct PlanParams {
  const int32_t* refs;
  int32_t* to;  // counts of holders afterwards; refs itself, or apart from it
  int64_t n_pages;
  int32_t *src, *dst, *map, *count;  // workspace; map: of pages >= L, -1 where free
  int32_t* live;
};

template <int CTAS>
__global__ void __launch_bounds__(CL_THREADS) page_plan_kernel(const PlanParams p) {
  constexpr int ALL = CTAS * CL_WARPS;
  __shared__ Counts s_a[CL_WARPS], s_b[CL_WARPS];
  const int lane = threadIdx.x & 31, w = cluster_rank<CTAS>() * CL_WARPS + (threadIdx.x >> 5);
  const int64_t some = ((p.n_pages + ALL - 1) / ALL + 31) / 32 * 32;
  const int64_t p0 = min(p.n_pages, w * some), p1 = min(p.n_pages, p0 + some);
  int mine = 0;
  each_page<8>(p.refs, p0, p1, [&](int64_t, int v, bool in_run) { mine += in_run && v > 0; });
  const Place live = cluster_place<CTAS>(Counts{0, __reduce_add_sync(FULL_MASK, mine)}, s_a);
  const int L = live.all.y;
  // live pages from L on, in this warp's run
  int high = 0;
  each_page<8>(p.refs, max(p0, int64_t(L)), p1, [&](int64_t, int v, bool in_run) { high += in_run && v > 0; });
  const Place far = cluster_place<CTAS>(Counts{0, __reduce_add_sync(FULL_MASK, high)}, s_b);
  int l = live.before.y, f = far.before.y;
  each_page<8>(p.refs, p0, p1, [&](int64_t page, int v, bool in_run) {
    const unsigned b = __ballot_sync(FULL_MASK, in_run && v > 0), low = (1u << lane) - 1;
    const unsigned up = __ballot_sync(FULL_MASK, in_run && v > 0 && page >= L);
    if (in_run && page < L && v <= 0) p.dst[page - (l + __popc(b & low))] = static_cast<int32_t>(page);
    if (up >> lane & 1) p.src[f + __popc(up & low)] = static_cast<int32_t>(page);
    if (in_run && page >= L && v <= 0) p.map[page] = -1;
    l += __popc(b);
    f += __popc(up);
  });
  if (w == 0 && lane == 0) {
    *p.count = far.all.y;
    *p.live = L;
  }
  cluster_sync<CTAS>();
  const int64_t thread = int64_t(cluster_rank<CTAS>()) * CL_THREADS + threadIdx.x;
  for (int64_t i = thread; i < far.all.y; i += CTAS * CL_THREADS) {
    const int a = __ldcg(p.src + i), b = __ldcg(p.dst + i);
    p.map[a] = b;
    p.to[b] = __ldcg(p.refs + a);
  }
  cluster_sync<CTAS>();
  for (int64_t i = thread; i < p.n_pages; i += CTAS * CL_THREADS) {
    if (i >= L) p.to[i] = 0;
    else if (p.to != p.refs) {
      const int v = __ldcg(p.refs + i);
      if (v > 0) p.to[i] = v;
    }
  }
}

cudaError_t pages_read_device_error(uint32_t* code) {
  uint32_t v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_err_pages, sizeof(v));
  if (e != cudaSuccess) return e;
  if (v) e = cudaMemcpyToSymbol(g_err_pages, &zero, sizeof(zero));
  *code |= v;
  return e;
}

namespace {

lilicorr_status fail(lilicorr_status st, const char* msg) {
  set_last_error(msg);
  return st;
}
lilicorr_status done(cudaError_t e) { return e == cudaSuccess ? LILICORR_OK : fail(LILICORR_ERR_CUDA, cudaGetErrorString(e)); }

constexpr int64_t LIM = int64_t(1) << 40;
bool page_ok(int page) { return page == 16 || page == 32 || page == 64 || page == 128; }
size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// One CTA, or one cluster of CL_CTAS.
template <class P>
cudaError_t launch_cluster(void (*one)(P), void (*many)(P), bool small, const P& p, cudaStream_t stream) {
  if (small) {
    one<<<1, CL_THREADS, 0, stream>>>(p);
  } else {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(CL_CTAS);
    cfg.blockDim = dim3(CL_THREADS);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CL_CTAS;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, many, p);
    if (e != cudaSuccess) return e;
  }
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) note_launch();
  return e;
}

// Null where the counts and a table's rows are in order, else what is wrong.
const char* pool_error(const int32_t* refs, int64_t n_pages) {
  if (!refs || !word_aligned({refs})) return "refs is null or misaligned";
  return n_pages < 1 || n_pages > INT_MAX ? "1 <= n_pages < 2^31" : nullptr;
}
const char* table_error(const int32_t* table, int64_t rows, int64_t stride, int32_t cols) {
  if (!table || !word_aligned({table})) return "a table is null or misaligned";
  if (rows < 1 || rows > INT_MAX || cols < 1 || cols > INT_MAX - 1024) return "a table's size is out of range";
  if (stride < cols || stride > LIM) return "a table's row stride is at least its columns";
  return nullptr;
}

}  // namespace
}  // namespace lilicorr

using namespace lilicorr;

extern "C" {

size_t lilicorr_kv8_pages_workspace_bytes(int64_t n_pages, int64_t rows) {
  if (n_pages < 1 || n_pages > INT_MAX || rows < 1 || rows > INT_MAX) return 0;
  return align256(size_t(n_pages) * 4) * 2 + align256(size_t(rows) * 4) + 256;
}

lilicorr_status lilicorr_kv8_fork(int32_t* refs, int64_t n_pages, int32_t* table, int64_t batch_stride, int64_t row_stride,
                                  int32_t cols, const int32_t* parent, int64_t batch, int32_t beams, void* stream) {
  const char* why = pool_error(refs, n_pages);
  if (!why) why = table_error(table, batch, beams > 1 ? row_stride : cols, cols);
  if (!why && (beams < 1 || beams > FK_MAX)) why = "1 <= beams <= 32";
  if (!why && batch > 1 && (batch_stride < (beams - 1) * row_stride + cols || batch_stride > LIM)) why = "batch_stride is at least its rows";
  if (!why && (!parent || !word_aligned({parent}))) why = "parent is null or misaligned";
  if (why) return fail(LILICORR_ERR_INVALID_ARG, why);
  const int tiles = (cols + FK_THREADS - 1) / FK_THREADS;
  if (batch > INT_MAX / tiles) return fail(LILICORR_ERR_INVALID_ARG, "batch * cols is too large for one call");
  const dim3 grid(static_cast<unsigned>(batch * tiles));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto go = [&](auto kernel) { kernel<<<grid, FK_THREADS, 0, st>>>(refs, n_pages, table, batch_stride, row_stride, cols, tiles, parent, beams); };
  if (beams <= 4) go(page_fork_kernel<4>);
  else if (beams <= 8) go(page_fork_kernel<8>);
  else if (beams <= 16) go(page_fork_kernel<16>);
  else go(page_fork_kernel<32>);
  note_launch();
  return done(cudaGetLastError());
}

lilicorr_status lilicorr_kv8_grow(int32_t* refs, int64_t n_pages, int32_t* table, int64_t rows, int64_t row_stride, int32_t cols,
                                  const int32_t* kv_len, const int32_t* new_tokens, int32_t page, int32_t max_new, int32_t* tail_src,
                                  uint8_t* granted, void* workspace, size_t workspace_bytes, void* stream) {
  const char* why = pool_error(refs, n_pages);
  if (!why) why = table_error(table, rows, rows > 1 ? row_stride : cols, cols);
  if (!why && !page_ok(page)) why = "page is 16, 32, 64 or 128";
  if (!why && int64_t(cols) * page > INT_MAX - 256) why = "a table row holds 1 page to 2^31 tokens";
  if (!why && (max_new < 1 || max_new > 1 << 24)) why = "1 <= max_new <= 2^24";
  if (!why && (!kv_len || !new_tokens || !tail_src || !granted)) why = "null pointer";
  if (!why && !word_aligned({kv_len, new_tokens, tail_src})) why = "lengths and tail_src are 4-byte aligned";
  if (why) return fail(LILICORR_ERR_INVALID_ARG, why);
  if (!workspace || workspace_bytes < lilicorr_kv8_pages_workspace_bytes(n_pages, rows) || reinterpret_cast<uintptr_t>(workspace) % 256)
    return fail(LILICORR_ERR_WORKSPACE, "lilicorr_kv8_grow: workspace missing, too small or misaligned");
  GrowParams p{};
  p.refs = refs; p.n_pages = n_pages;
  p.table = table; p.row_stride = row_stride; p.rows = rows;
  p.cols = cols; p.page = page; p.max_new = max_new;
  p.kv_len = kv_len; p.fresh = new_tokens; p.tail_src = tail_src; p.granted = granted;
  p.list = static_cast<int32_t*>(workspace);
  p.held = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + align256(size_t(n_pages) * 4));
  p.need = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + align256(size_t(n_pages) * 4) * 2);
  const int most = p.steps = (max_new + page - 2) / page + 1;
  while (p.group_log2 < 5 && (1 << p.group_log2) < most) ++p.group_log2;
  return done(launch_cluster(page_grow_kernel<1>, page_grow_kernel<CL_CTAS>, n_pages <= CL_SMALL && rows * most <= CL_SMALL_COLUMNS, p,
                             static_cast<cudaStream_t>(stream)));
}

lilicorr_status lilicorr_kv8_free(int32_t* refs, int64_t n_pages, int32_t* table, int64_t rows, int64_t row_stride, int32_t cols,
                                  const int32_t* keep, int32_t page, void* stream) {
  const char* why = pool_error(refs, n_pages);
  if (!why) why = table_error(table, rows, rows > 1 ? row_stride : cols, cols);
  if (!why && !page_ok(page)) why = "page is 16, 32, 64 or 128";
  if (!why && (!keep || !word_aligned({keep}))) why = "keep is null or misaligned";
  const int tiles = (cols - 1) / FR_THREADS + 1;
  if (!why && rows > INT_MAX / tiles) why = "rows * cols is too large for one call";
  if (why) return fail(LILICORR_ERR_INVALID_ARG, why);
  page_free_kernel<<<static_cast<unsigned>(rows * tiles), FR_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(refs, n_pages, table, row_stride, cols,
                                                                                                           tiles, keep, page);
  note_launch();
  return done(cudaGetLastError());
}

}  // extern "C"

namespace lilicorr {
namespace {

// Null where the caches' descriptions are in order and alike, else what is wrong.
const char* caches_error(const lilicorr_kv8_cache* c, int32_t n, const lilicorr_kv8_cache& like, bool same_pages) {
  if (!c) return "null caches";
  for (int i = 0; i < n; ++i) {
    const char* why = kv8_cache_error(c + i);
    if (why) return why;
    if (c[i].kv_heads != like.kv_heads || c[i].page != like.page || c[i].head_dim != like.head_dim) return "caches differ in heads, page or head_dim";
    if (c[i].n_pages != c[0].n_pages || (same_pages && c[i].n_pages != like.n_pages)) return "caches differ in their pages";
  }
  return nullptr;
}
void put_caches(MoveParams& p, const lilicorr_kv8_cache* from, const lilicorr_kv8_cache* to, int n) {
  p.n_caches = n;
  p.heads = from->kv_heads;
  p.vecs = static_cast<int>(int64_t(from->kv_heads) * from->page * from->head_dim / 16);  // 32 at least
  p.tiles = (p.vecs - 1) / MV_TILE + 1;
  p.pages = std::max(1, MV_TILE / p.vecs);
  p.inv = static_cast<uint32_t>(((int64_t(1) << 32) + p.vecs - 1) / p.vecs);
  p.n_src = from->n_pages;
  p.n_dst = to->n_pages;
  for (int i = 0; i < n; ++i)
    p.c[i] = MoveCache{static_cast<const uint4*>(from[i].k_pages), static_cast<const uint4*>(from[i].v_pages), static_cast<uint4*>(to[i].k_pages),
                       static_cast<uint4*>(to[i].v_pages), from[i].k_scale, from[i].v_scale, to[i].k_scale, to[i].v_scale};
}
int64_t tiles_of(const MoveParams& p) { return (p.pages > 1 ? (p.n + p.pages - 1) / p.pages : p.n * p.tiles) * p.n_caches * 2; }

}  // namespace
}  // namespace lilicorr

extern "C" {

lilicorr_status lilicorr_kv8_copy(const lilicorr_kv8_cache* from, const lilicorr_kv8_cache* to, int32_t n_caches, const int32_t* src,
                                  const int32_t* dst, int64_t n, void* stream) {
  if (n_caches < 1 || !from || !to) return fail(LILICORR_ERR_INVALID_ARG, "lilicorr_kv8_copy: no caches");
  const char* why = caches_error(from, n_caches, from[0], true);
  if (!why) why = caches_error(to, n_caches, from[0], false);
  if (!why && (!src || !dst || !word_aligned({src, dst}))) why = "src or dst is null or misaligned";
  if (!why && (n < 1 || n > INT_MAX)) why = "1 <= n < 2^31";
  if (why) return fail(LILICORR_ERR_INVALID_ARG, why);
  for (int i = 0; i < n_caches; i += MV_CACHES) {
    MoveParams p{};
    put_caches(p, from + i, to + i, std::min(n_caches - i, MV_CACHES));
    p.src = src; p.dst = dst; p.n = n;
    const int64_t grid = std::min<int64_t>(tiles_of(p), int64_t(device_sm_count()) * 8);
    page_copy_kernel<<<static_cast<unsigned>(grid), MV_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(p);
    note_launch();
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return done(e);
  }
  return LILICORR_OK;
}

lilicorr_status lilicorr_kv8_compact(const lilicorr_kv8_cache* caches, int32_t n_caches, const int32_t* refs, int32_t* refs_out,
                                     int64_t n_pages, const lilicorr_kv8_table* tables, int32_t n_tables, int32_t* live, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  const char* why = pool_error(refs, n_pages);
  if (!why) why = pool_error(refs_out, n_pages);
  if (!why && refs != refs_out && refs < refs_out + n_pages && refs_out < refs + n_pages) why = "refs_out is refs, or shares nothing with it";
  if (!why && (n_caches < 1 || !caches)) why = "no caches";
  if (!why) why = caches_error(caches, n_caches, caches[0], true);
  if (!why && caches[0].n_pages != n_pages) why = "refs counts the caches' pages";
  if (!why && (n_tables < 0 || (n_tables > 0 && !tables))) why = "null tables";
  for (int i = 0; !why && i < n_tables; ++i) {
    const lilicorr_kv8_table& t = tables[i];
    why = table_error(t.table, t.rows, t.rows > 1 ? t.row_stride : t.cols, t.cols);
    if (!why) why = table_error(t.out, t.rows, t.rows > 1 ? t.out_stride : t.cols, t.cols);
    if (!why && t.table == t.out && t.row_stride != t.out_stride) why = "a table in place keeps its stride";
  }
  if (!why && (!live || !word_aligned({live}))) why = "live is null or misaligned";
  if (why) return fail(LILICORR_ERR_INVALID_ARG, why);
  if (!workspace || workspace_bytes < lilicorr_kv8_pages_workspace_bytes(n_pages, 1) || reinterpret_cast<uintptr_t>(workspace) % 256)
    return fail(LILICORR_ERR_WORKSPACE, "lilicorr_kv8_compact: workspace missing, too small or misaligned");
  char* ws = static_cast<char*>(workspace);
  const size_t part = align256(size_t(n_pages) * 4);
  // sources and destinations are at most half the pages each
  PlanParams pl{};
  pl.refs = refs; pl.to = refs_out; pl.n_pages = n_pages;
  pl.src = reinterpret_cast<int32_t*>(ws);
  pl.dst = pl.src + (n_pages + 1) / 2;
  pl.map = reinterpret_cast<int32_t*>(ws + part);
  pl.count = reinterpret_cast<int32_t*>(ws + 2 * part);
  pl.live = live;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_cluster(page_plan_kernel<1>, page_plan_kernel<CL_CTAS>, n_pages <= CL_SMALL, pl, st);
  for (int i = 0, j = 0; e == cudaSuccess && (i < n_caches || j < n_tables); i += MV_CACHES, j += MV_TABLES) {
    MoveParams p{};
    const int nc = std::max(0, std::min(n_caches - i, MV_CACHES));
    if (nc > 0) put_caches(p, caches + i, caches + i, nc);
    p.n_src = p.n_dst = n_pages;
    p.src = pl.src; p.dst = pl.dst; p.count = pl.count; p.map = pl.map;
    p.n = nc > 0 ? n_pages / 2 : 0;
    int64_t entries = 0;
    for (p.n_tables = 0; p.n_tables < MV_TABLES && j + p.n_tables < n_tables; ++p.n_tables) {
      const lilicorr_kv8_table& t = tables[j + p.n_tables];
      p.t[p.n_tables] = MoveTable{t.table, t.out, t.row_stride, t.out_stride, t.rows, t.cols};
      entries += t.rows * t.cols;
    }
    const int sms = device_sm_count();
    p.table_ctas = static_cast<int>(std::min<int64_t>((entries + 4 * MV_THREADS - 1) / (4 * MV_THREADS), 2 * sms));
    const int64_t grid = p.table_ctas + std::min<int64_t>(tiles_of(p), int64_t(sms) * 8);
    if (grid == 0) continue;
    PdlScope pdl(i == 0);
    e = launch_k(page_compact_kernel, dim3(static_cast<unsigned>(grid)), dim3(MV_THREADS), 0, st, p, static_cast<const int32_t*>(live));
    if (e == cudaSuccess) note_launch();
  }
  return done(e);
}

}  // extern "C"
