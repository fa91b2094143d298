// A paged key / value cache held in 8 bits (e4m3) with one scale for each page (block of
// tokens) and key / value head: its writer, and the attention that reads it.
#include <cuda_fp16.h>

#include <climits>
#include <cmath>

#include <algorithm>

#include "kernels.cuh"

namespace lilicorr {

static __device__ uint32_t g_err_kv8;

// Host parameters of the cache, as the kernels take them.
struct Kv8 {
  uint8_t *k, *v;        // [n_pages, heads, page, D]
  float *ks, *vs;        // [n_pages, heads]
  int64_t n_pages;
  int heads, page;
};

__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t x) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(x));
  return r;
}
// Two floats to e4m3 codes (a in the low byte), to nearest even, magnitudes above 448 to 448.
__device__ __forceinline__ uint16_t f32x2_to_e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

// One sequence's rows, or n = 0 where its row range or length is out of range (recorded).
struct SeqRange {
  int64_t q0;  // first row
  int n, len;  // new rows; cached tokens, the new ones among them
};
__device__ __forceinline__ SeqRange seq_range(const int32_t* __restrict__ q_start,
                                              const int32_t* __restrict__ kv_len, int64_t b,
                                              int64_t total, int max_new, int64_t capacity) {
  SeqRange r;
  const int a = __ldg(q_start + b), e = __ldg(q_start + b + 1);
  r.q0 = a;
  r.n = e - a;
  r.len = __ldg(kv_len + b);
  if (a < 0 || e < a || e > total || r.n > max_new || r.len < 0 || r.len > capacity) {
    atomicOr(&g_err_kv8, ERR_KV8_LENGTH);
    r.n = 0;
    r.len = 0;
  }
  return r;
}

// ---------------------------------------------------------------------------- the writer
// One CTA per (sequence, page that grows, head, K or V).  The page's scale is the smallest
// power of two 2^k >= 2^-60 that holds its new rows' largest finite magnitude within 448,
// or the scale that the page has from its earlier rows where that is larger.  A power of two
// costs e4m3 nothing in relative precision, and lets a page's earlier codes move to a larger
// scale exactly (but for e4m3's subnormals), so appending tokens one by one leaves what
// appending them at once does.  Bound by HBM for prompts (2 bytes in and 1 out per value),
// by latency for single tokens.  The rows are kept in registers between the maximum and the
// conversion, so that they are read once.
constexpr int AP_THREADS = 128;

struct AppendParams {
  Kv8 c;
  const __nv_bfloat16 *k, *v;
  int64_t k_tok, k_head, v_tok, v_head;  // elements
  int64_t total;
  const int32_t *q_start, *kv_len, *table, *tail_src;
  int64_t table_stride;
  int cols;      // pages of a table row
  int max_new, grow;  // pages a sequence can touch in one call
};

// 2^k as above, from the bits of the largest magnitude (finite, >= 0).
__device__ __forceinline__ float page_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  // amax = m 2^e with m in [0.5, 1); 448 = 0.875 * 2^9
  int k = static_cast<int>(u >> 23) - 126 - 9 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  k = max(k, -60);
  return __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
}

template <int VPT>  // 8-element vectors a thread holds of a page
__global__ void __launch_bounds__(AP_THREADS) kv8_append_kernel(const AppendParams p, int D) {
  __shared__ uint32_t s_max[AP_THREADS / 32];
  const int tid = threadIdx.x;
  int64_t u = blockIdx.x;
  const int which = static_cast<int>(u & 1);
  u >>= 1;
  const int h = static_cast<int>(u % p.c.heads);
  u /= p.c.heads;
  const int g = static_cast<int>(u % p.grow);
  const int64_t b = u / p.grow;
  const int page = p.c.page;
  const SeqRange r = seq_range(p.q_start, p.kv_len, b, p.total, p.max_new,
                               int64_t(p.cols) * page);
  const int before = r.len - r.n;
  if (r.n == 0) return;
  if (before < 0) {
    if (tid == 0) atomicOr(&g_err_kv8, ERR_KV8_LENGTH);
    return;
  }
  const int at = before / page + g;  // this page's column of the table
  if (int64_t(at) * page >= r.len) return;
  const int id = __ldg(p.table + b * p.table_stride + at);
  const int pos0 = at * page;
  const bool has_old = pos0 < before;
  int src = id;
  if (has_old && p.tail_src) {
    src = __ldg(p.tail_src + b);
    if (src < 0) src = id;
  }
  if (id < 0 || id >= p.c.n_pages || src >= p.c.n_pages) {
    if (tid == 0) atomicOr(&g_err_kv8, ERR_KV8_PAGE);
    return;
  }
  const __nv_bfloat16* x = which ? p.v : p.k;
  const int64_t tok = which ? p.v_tok : p.k_tok, hd = which ? p.v_head : p.k_head;
  uint8_t* codes = (which ? p.c.v : p.c.k) + (int64_t(id) * p.c.heads + h) * page * D;
  float* scales = which ? p.c.vs : p.c.ks;

  const int vrow = D / 8, nvec = page * vrow;
  uint4 w[VPT];
  uint32_t top = 0;  // bits of the largest finite magnitude (of bf16, so 15 bits)
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int e = tid + i * AP_THREADS;
    const int row = e / vrow, pos = pos0 + row;
    w[i] = make_uint4(0u, 0u, 0u, 0u);
    if (e < nvec && pos >= before && pos < r.len)
      w[i] = __ldcs(reinterpret_cast<const uint4*>(x + (r.q0 + pos - before) * tok + h * hd +
                                                   (e - row * vrow) * 8));
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const uint32_t q[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = q[j] & 0x7fffu, hi = (q[j] >> 16) & 0x7fffu;
      if (lo < 0x7f80u) top = max(top, lo);
      if (hi < 0x7f80u) top = max(top, hi);
    }
  }
  top = __reduce_max_sync(FULL_MASK, top);
  if ((tid & 31) == 0) s_max[tid >> 5] = top;
  const float was = has_old ? __ldcg(scales + int64_t(src) * p.c.heads + h) : 0.f;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < AP_THREADS / 32; ++i) top = max(top, s_max[i]);
  const float now = fmaxf(page_scale(__uint_as_float(top << 16)), was);
  // a scale of the caller's own need not be a power of two; then the quotient is divided out
  const bool pow2 = (__float_as_uint(now) & 0x7fffffu) == 0;
  const float inv = 1.f / now;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int e = tid + i * AP_THREADS;
    const int row = e / vrow, pos = pos0 + row;
    if (e < nvec && pos >= before && pos < r.len) {
      const uint32_t q[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
      uint16_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float lo = __uint_as_float(q[j] << 16), hi = __uint_as_float(q[j] & 0xffff0000u);
        o[j] = pow2 ? f32x2_to_e4m3x2(lo * inv, hi * inv) : f32x2_to_e4m3x2(lo / now, hi / now);
      }
      *reinterpret_cast<uint2*>(codes + int64_t(e) * 8) =
          make_uint2(o[0] | uint32_t(o[1]) << 16, o[2] | uint32_t(o[3]) << 16);
    }
  }
  // Earlier rows: moved to the larger scale, or copied from the page they lie in.
  if (has_old && (src != id || now != was)) {
    const uint8_t* from = (which ? p.c.v : p.c.k) + (int64_t(src) * p.c.heads + h) * page * D;
    const float f = was / now;
    const int nold = (min(before, pos0 + page) - pos0) * vrow;
    for (int e = tid; e < nold; e += AP_THREADS) {
      uint2 c = *reinterpret_cast<const uint2*>(from + int64_t(e) * 8);
      if (now != was) {
        uint32_t q[2] = {c.x, c.y};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t a = e4m3x2_to_f16x2(static_cast<uint16_t>(q[j]));
          const uint32_t d = e4m3x2_to_f16x2(static_cast<uint16_t>(q[j] >> 16));
          const float2 fa = __half22float2(*reinterpret_cast<const __half2*>(&a));
          const float2 fd = __half22float2(*reinterpret_cast<const __half2*>(&d));
          q[j] = f32x2_to_e4m3x2(fa.x * f, fa.y * f) |
                 uint32_t(f32x2_to_e4m3x2(fd.x * f, fd.y * f)) << 16;
        }
        c = make_uint2(q[0], q[1]);
      }
      *reinterpret_cast<uint2*>(codes + int64_t(e) * 8) = c;
    }
  }
  // (the old scale was read before the barrier above)
  if (tid == 0) scales[int64_t(id) * p.c.heads + h] = now;
}

// ------------------------------------------------------------------------- the attention
// For new token i of a sequence's n, and query head j of the group that shares a key / value
// head:  o = softmax_t(scale q . k_t) v_t  over the cached tokens t < len - n + i + 1.
//
// The n * group rows of a (sequence, key / value head) are taken in tiles; a work unit is one
// tile against one chunk of 64 cached tokens, and the units of a call, laid out by (sequence,
// head, tile, chunk), are dealt in equal contiguous runs to a fixed grid of CTAs, so that
// ragged lengths and few rows over a long axis load the SMs alike.  A CTA that holds a part
// of a tile's chunks leaves its maxima, sums and products in the workspace, and a second
// kernel joins the parts in order; a tile that one CTA holds whole is finished there.
//
// Within a chunk each of the four warps takes 16 tokens.  Codes go from global memory to
// registers and become f16 there (exact), in the lane layout of the warp's matrix
// instruction: the summation index of q . k and the output columns of p v may be taken in
// any order, so each lane reads 16 contiguous bytes.  The page's key scale multiplies the
// scores; the value scale's logarithm is added to them, so that p' = scale_v exp(s - m) is
// what the second product takes and the sums take p' / scale_v.  q is bf16 moved to f16 by a
// power of two of its row (exact but for values 2^-29 below the row's largest); p' is rounded
// to f16 (2^-11 of its value, 2^-25 of the row's largest below 2^-14); everything else is f32.
constexpr int AT_WARPS = 4;
constexpr int AT_CHUNK = 16 * AT_WARPS;
constexpr float LOG2E_F = 1.4426950408889634f;
constexpr float LN2_F = 0.6931471805599453f;

struct AttnParams {
  Kv8 c;
  const __nv_bfloat16* q;
  int64_t q_tok, q_head;  // elements
  int64_t total;
  int q_heads, group;
  const int32_t *q_start, *kv_len, *table;
  int64_t batch, table_stride;
  int cols, max_new, page_log2;
  float scale2;  // softmax scale * log2 e
  __nv_bfloat16* out;  // [total, q_heads, D]
  float* lse;          // [total, q_heads] or null
  float* part;         // [2 * grid][rows of a tile * (D + 2)]: products, maxima, sums
};

struct SeqUnits {
  int n, len, tiles, chunks;
  int64_t q0, units;
};
template <int RT>
__device__ __forceinline__ SeqUnits seq_units(const AttnParams& p, int64_t b) {
  const SeqRange r = seq_range(p.q_start, p.kv_len, b, p.total, p.max_new,
                               int64_t(p.cols) << p.page_log2);
  SeqUnits u;
  u.n = r.n;
  u.len = r.len;
  u.q0 = r.q0;
  u.tiles = (r.n * p.group + RT - 1) / RT;
  u.chunks = max(1, (r.len + AT_CHUNK - 1) / AT_CHUNK);
  u.units = int64_t(u.tiles) * p.c.heads * u.chunks;
  return u;
}

// The units of all sequences, and where the run of CTA `run` begins: every warp works it out
// for itself.  The counts of the first 128 sequences stay in registers between the two passes.
struct Run {
  int64_t units, per;  // all units; units of a run
  int64_t u, u_end;    // this run's units
  int64_t b, first;    // the sequence of unit u, and that sequence's first unit
};
template <int RT>
__device__ __forceinline__ Run find_run(const AttnParams& p, int64_t run, int64_t runs) {
  constexpr int KEEP = 4;
  const int lane = threadIdx.x & 31;
  auto count = [&](int64_t b) { return b < p.batch ? seq_units<RT>(p, b).units : int64_t(0); };
  int64_t kept[KEEP], t = 0;
#pragma unroll
  for (int i = 0; i < KEEP; ++i) {
    kept[i] = i * 32 < p.batch ? count(i * 32 + lane) : 0;
    t += kept[i];
  }
  for (int64_t b = KEEP * 32 + lane; b < p.batch; b += 32) t += count(b);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) t += __shfl_xor_sync(FULL_MASK, t, o);
  Run r;
  r.units = t;
  r.per = (t + runs - 1) / runs;
  r.u = run * r.per;
  r.u_end = min(t, r.u + r.per);
  r.b = p.batch;
  r.first = 0;
  if (r.u >= r.u_end) return r;
  int64_t base = 0;
  auto look = [&](int64_t b0, int64_t mine) {  // whether unit u is among these 32 sequences'
    int64_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(FULL_MASK, sum, o);
      if (lane >= o) sum += x;
    }
    const unsigned past = __ballot_sync(FULL_MASK, base + sum > r.u);
    if (past) {
      const int l = __ffs(past) - 1;
      r.b = b0 + l;
      r.first = base + __shfl_sync(FULL_MASK, sum - mine, l);
      return true;
    }
    base += __shfl_sync(FULL_MASK, sum, 31);
    return false;
  };
#pragma unroll
  for (int i = 0; i < KEEP; ++i)
    if (i * 32 < p.batch && look(i * 32, kept[i])) return r;
  for (int64_t b0 = KEEP * 32; b0 < p.batch; b0 += 32)
    if (look(b0, count(b0 + lane))) return r;
  return r;
}

// The pieces of a run: the chunks [c0, c1) of one tile each.
struct Piece {
  SeqUnits sq;
  int64_t b, first;  // the sequence, and its first unit
  int h, tile, c0, c1;
  int end;           // tokens that the tile's last row sees
  bool whole;        // all of the tile's chunks
};
template <int RT>
__device__ __forceinline__ void piece_at(const AttnParams& p, int64_t u, int64_t u_end, Piece& x) {
  while (u >= x.first + x.sq.units) {
    x.first += x.sq.units;
    x.sq = seq_units<RT>(p, ++x.b);
  }
  const uint32_t in = static_cast<uint32_t>(u - x.first);  // a sequence's units fit 32 bits (host)
  const uint32_t item = in / x.sq.chunks;
  x.c0 = static_cast<int>(in - item * x.sq.chunks);
  x.c1 = static_cast<int>(min(int64_t(x.sq.chunks), x.c0 + (u_end - u)));
  x.h = item / x.sq.tiles;
  x.tile = item - x.h * x.sq.tiles;
  const int last = min((x.tile + 1) * RT, x.sq.n * p.group) - 1;
  x.end = min(x.sq.len, x.sq.len - x.sq.n + last / p.group + 1);
  x.whole = x.c0 == 0 && x.c1 == x.sq.chunks;
}

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// d += a b for a 16 x 16 tile a and a 16 x 8 tile b; with NR = 1 the upper 8 rows of a are
// zero, and their part of d is neither read nor kept.
template <int NR>
__device__ __forceinline__ void mma_f16(float (&d)[2 * NR], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  if constexpr (NR == 1) {
    float z0, z1;
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%10,%10};"
        : "+f"(d[0]), "+f"(d[1]), "=f"(z0), "=f"(z1)
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}

__device__ __forceinline__ bool any_nan4(uint32_t w) {
  return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;
}
__device__ __forceinline__ uint32_t no_nan4(uint32_t w) {
  return w & ~__vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu);
}

// Writes a row's outputs: D / 32 columns a lane (x), their sum of weights and maximum.
template <int N>
__device__ __forceinline__ void store_row(const AttnParams& p, int64_t at, int D, int d,
                                          const float (&x)[N], float sum, float m) {
  const float inv = sum == 0.f ? 0.f : 1.f / sum;  // no token seen: 0
  __nv_bfloat16* o = p.out + at * D + d;
  if constexpr (N == 4) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0] * inv, x[1] * inv);
    const __nv_bfloat162 c = __floats2bfloat162_rn(x[2] * inv, x[3] * inv);
    *reinterpret_cast<uint2*>(o) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                              *reinterpret_cast<const uint32_t*>(&c));
  } else if constexpr (N == 2) {
    *reinterpret_cast<__nv_bfloat162*>(o) = __floats2bfloat162_rn(x[0] * inv, x[1] * inv);
  } else {
    *o = __float2bfloat16_rn(x[0] * inv);
  }
  if (p.lse && d == 0) p.lse[at] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * LN2_F;
}

template <int D, int RT>
struct AttnShape {
  static constexpr int STAGES = RT == 8 ? 5 : 4;
  static constexpr int CTAS = 2;                        // per SM
  static constexpr int TILE = AT_CHUNK * D;             // bytes of a chunk's keys, or values
  static constexpr int RING = STAGES * 2 * TILE;
  static constexpr int SMEM = RING + AT_WARPS * RT * (D + 4) * 4;
};

struct ChunkScale {  // of 16 tokens
  float k, log2_v, inv_v;
  int ok;  // the page exists
};

// Four warps work on the chunks that a fifth brings into a ring of shared-memory stages by bulk
// copies.  Rows of a tile in the matrix instruction's accumulator layout: lane (g, t) =
// (lane / 4, lane % 4) holds rows g and g + 8.  D = head dimension, RT = rows (8 or 16: with 8
// the upper half of every product is zero and takes no registers).
template <int D, int RT>
__global__ void __launch_bounds__(32 * AT_WARPS + 32, AttnShape<D, RT>::CTAS)
    kv8_attention_kernel(const AttnParams p) {
  using Shape = AttnShape<D, RT>;
  constexpr int KW = D / 16;  // words of a key row a lane reads = steps of 16 of q . k
  constexpr int VW = D / 32;  // words of a value row a lane reads
  constexpr int NU = D / 8;   // output column groups
  constexpr int NR = RT / 8;  // rows a lane holds
  constexpr int ST = Shape::STAGES;
  extern __shared__ __align__(128) uint8_t at_smem[];
  __shared__ __align__(8) uint64_t full[ST], empty[ST];
  __shared__ ChunkScale s_scale[ST][AT_WARPS];
  __shared__ float s_m[AT_WARPS][RT], s_l[AT_WARPS][RT];
  __shared__ int s_abort;
  float(*s_o)[RT][D + 4] = reinterpret_cast<float(*)[RT][D + 4]>(at_smem + Shape::RING);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], AT_WARPS);
    }
    fence_mbar_init();
    s_abort = 0;
  }
  pdl_wait();
  pdl_trigger();
  const Run run = find_run<RT>(p, blockIdx.x, gridDim.x);
  __syncthreads();
  if (run.u >= run.u_end) return;
  Piece x;
  x.b = run.b;
  x.first = run.first;
  x.sq = seq_units<RT>(p, run.b);
  volatile int* abort_flag = &s_abort;
  // A wait that gives up marks the CTA; from then on nothing waits or computes, but every
  // barrier between the warps is still met, so the kernel ends.
  auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t site) -> bool {
    if (*abort_flag) return false;
    if (mbar_wait_bounded(bar, parity, &g_err_kv8, site)) return true;
    *abort_flag = 1;
    return false;
  };

  if (warp == AT_WARPS) {
    // ================= copies: lane i brings the i-th page part of a chunk =================
    const int part = min(p.c.page, AT_CHUNK);  // tokens
    const int parts = AT_CHUNK / part;
    const int bytes = part * D;
    int it = 0;
    for (int64_t u = run.u; u < run.u_end; u += x.c1 - x.c0) {
      piece_at<RT>(p, u, run.u_end, x);
      const int32_t* tab = p.table + x.b * p.table_stride;
      auto page_of = [&](int c) {
        const int tok = c * AT_CHUNK + lane * part;
        return lane < parts && tok < x.end ? __ldg(tab + (tok >> p.page_log2)) : -2;
      };
      int next = page_of(x.c0);
      for (int c = x.c0; c < x.c1; ++c, ++it) {
        if (c * AT_CHUNK >= x.end) {  // nothing of this chunk is seen: the tile's rows end here
          break;
        }
        const int st = it % ST;
        const int id = next;
        if (c + 1 < x.c1) next = page_of(c + 1);
        if (it >= ST && !wait(&empty[st], ((it / ST) - 1) & 1, ERR_KV8_EMPTY_WAIT)) break;
        const bool ok = id >= 0 && id < p.c.n_pages;
        if (id != -2 && !ok) atomicOr(&g_err_kv8, ERR_KV8_PAGE);
        const unsigned have = __ballot_sync(FULL_MASK, ok);
        if (lane == 0) mbar_expect_tx(&full[st], 2u * bytes * __popc(have));
        __syncwarp();
        if (ok) {
          const int tok = c * AT_CHUNK + lane * part;
          const int64_t ph = int64_t(id) * p.c.heads + x.h;
          const int64_t off = (ph * p.c.page + (tok & (p.c.page - 1))) * D;
          uint8_t* dst = at_smem + st * 2 * Shape::TILE + lane * bytes;
          bulk_g2s(dst, p.c.k + off, bytes, &full[st]);
          bulk_g2s(dst + Shape::TILE, p.c.v + off, bytes, &full[st]);
          const float ks = __ldg(p.c.ks + ph), vs = __ldg(p.c.vs + ph);
          const ChunkScale sc{ks, log2f(vs), 1.f / vs, 1};
          for (int w = 0; w < part / 16; ++w) s_scale[st][lane * (part / 16) + w] = sc;
        } else if (lane < parts) {
          for (int w = 0; w < part / 16; ++w) s_scale[st][lane * (part / 16) + w].ok = 0;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[st]);
      }
    }
    // after a wait gave up: what was issued and not waited for by the others has to land
    if (*abort_flag)
      for (int i = max(0, it - ST); i < it; ++i)
        mbar_wait_bounded(&full[i % ST], (i / ST) & 1, &g_err_kv8, ERR_KV8_DRAIN);
    return;
  }

  const int g = lane >> 2, t = lane & 3;
  bool first_piece = true;
  int it = 0;
  for (int64_t u = run.u; u < run.u_end; u += x.c1 - x.c0, first_piece = false) {
    piece_at<RT>(p, u, run.u_end, x);
    const SeqUnits& sq = x.sq;
    const int row0 = x.tile * RT, rows = sq.n * p.group, end = x.end;

    // q of this lane's rows, as f16 of the row's largest power of two
    uint32_t qf[KW][4];
    float f_row[NR];
    int seen[NR];
#pragma unroll
    for (int k = 0; k < KW; ++k) qf[k][0] = qf[k][1] = qf[k][2] = qf[k][3] = 0u;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int row = row0 + g + 8 * r;
      const bool has = row < rows;
      const int i = has ? row / p.group : 0, j = has ? row - i * p.group : 0;
      seen[r] = has ? min(sq.len - sq.n + i + 1, end) : 0;
      const __nv_bfloat16* qr = p.q + (sq.q0 + i) * p.q_tok + (x.h * p.group + j) * p.q_head;
      uint2 raw[KW];
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < KW; ++k) {
        const int d0 = D >= 64 ? (t + 4 * (k / 4)) * 16 + (k % 4) * 4 : t * 8 + k * 4;
        raw[k] = has ? __ldg(reinterpret_cast<const uint2*>(qr + d0)) : make_uint2(0u, 0u);
        top = max(max(top, raw[k].x & 0x7fffu), (raw[k].x >> 16) & 0x7fffu);
        top = max(max(top, raw[k].y & 0x7fffu), (raw[k].y >> 16) & 0x7fffu);
      }
      top = max(top, __shfl_xor_sync(FULL_MASK, top, 1));
      top = max(top, __shfl_xor_sync(FULL_MASK, top, 2));
      // the largest moves to [2^14, 2^15); an infinite or NaN row stays so whatever the power
      const int e = min(max(static_cast<int>(top >> 7), 1), 254) - 127;
      const int sh = min(14 - e, 120);
      const float up = __uint_as_float(static_cast<uint32_t>(127 + sh) << 23);
      f_row[r] = p.scale2 * __uint_as_float(static_cast<uint32_t>(127 - sh) << 23);
#pragma unroll
      for (int k = 0; k < KW; ++k) {
        const __half2 a = __floats2half2_rn(__uint_as_float(raw[k].x << 16) * up,
                                            __uint_as_float(raw[k].x & 0xffff0000u) * up);
        const __half2 c = __floats2half2_rn(__uint_as_float(raw[k].y << 16) * up,
                                            __uint_as_float(raw[k].y & 0xffff0000u) * up);
        qf[k][r] = *reinterpret_cast<const uint32_t*>(&a);
        qf[k][2 + r] = *reinterpret_cast<const uint32_t*>(&c);
      }
    }

    float m[NR], l[NR], o[NU][2 * NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) { m[r] = -INFINITY; l[r] = 0.f; }
#pragma unroll
    for (int n = 0; n < NU; ++n)
#pragma unroll
      for (int e = 0; e < 2 * NR; ++e) o[n][e] = 0.f;

    for (int c = x.c0; c < x.c1; ++c, ++it) {
      if (c * AT_CHUNK >= end) break;
      const int st = it % ST;
      const bool landed = wait(&full[st], (it / ST) & 1, ERR_KV8_FULL_WAIT);
      const int tok0 = c * AT_CHUNK + warp * 16;
      const ChunkScale sc = s_scale[st][warp];
      if (landed && tok0 < end && sc.ok) {
        const uint8_t* kt = at_smem + st * 2 * Shape::TILE + warp * 16 * D;
        const uint8_t* vt = kt + Shape::TILE;
        float s[2][2 * NR];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t kw[KW];
          const uint8_t* kr = kt + (8 * j + g) * D;
          if constexpr (D == 128) {
            // 128-byte rows share banks: odd rows take the other half first
            const int sw = (g & 1) * 64;
            const uint4 a = *reinterpret_cast<const uint4*>(kr + t * 16 + sw);
            const uint4 b = *reinterpret_cast<const uint4*>(kr + t * 16 + 64 - sw);
            const uint4 lo = sw ? b : a, hi = sw ? a : b;
            kw[0] = lo.x; kw[1] = lo.y; kw[2] = lo.z; kw[3] = lo.w;
            kw[4] = hi.x; kw[5] = hi.y; kw[6] = hi.z; kw[7] = hi.w;
          } else if constexpr (D == 64) {
            const uint4 a = *reinterpret_cast<const uint4*>(kr + t * 16);
            kw[0] = a.x; kw[1] = a.y; kw[2] = a.z; kw[3] = a.w;
          } else {
            const uint2 a = *reinterpret_cast<const uint2*>(kr + t * 8);
            kw[0] = a.x; kw[1] = a.y;
          }
#pragma unroll
          for (int e = 0; e < 2 * NR; ++e) s[j][e] = 0.f;
#pragma unroll
          for (int k = 0; k < KW; ++k)
            mma_f16<NR>(s[j], qf[k], e4m3x2_to_f16x2(static_cast<uint16_t>(kw[k])),
                        e4m3x2_to_f16x2(static_cast<uint16_t>(kw[k] >> 16)));
        }
        uint32_t vw[4][VW];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint8_t* vr = vt + (2 * t + (j & 1) + 8 * (j >> 1)) * D + g * (D / 8);
          if constexpr (D == 128) {
            const uint4 a = *reinterpret_cast<const uint4*>(vr);
            vw[j][0] = a.x; vw[j][1] = a.y; vw[j][2] = a.z; vw[j][3] = a.w;
          } else if constexpr (D == 64) {
            const uint2 a = *reinterpret_cast<const uint2*>(vr);
            vw[j][0] = a.x; vw[j][1] = a.y;
          } else {
            vw[j][0] = *reinterpret_cast<const uint32_t*>(vr);
          }
        }
        uint32_t pf[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const float f = f_row[r] * sc.k;
          float y[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int tk = tok0 + 2 * t + (j & 1) + 8 * (j >> 1);
            y[j] = tk < seen[r] ? fmaf(s[j >> 1][2 * r + (j & 1)], f, sc.log2_v) : -INFINITY;
          }
          float mx = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
          mx = fmaxf(mx, __shfl_xor_sync(FULL_MASK, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(FULL_MASK, mx, 2));
          const float nm = fmaxf(m[r], mx);
          const float base = nm == -INFINITY ? 0.f : nm;
          if (nm != m[r]) {  // uniform over the four lanes of the row
            const float back = ex2f(m[r] - base);
            l[r] *= back;
#pragma unroll
            for (int n = 0; n < NU; ++n) { o[n][2 * r] *= back; o[n][2 * r + 1] *= back; }
            m[r] = nm;
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) y[j] = ex2f(y[j] - base);
          l[r] = fmaf((y[0] + y[1]) + (y[2] + y[3]), sc.inv_v, l[r]);
          const __half2 a = __floats2half2_rn(y[0], y[1]), d = __floats2half2_rn(y[2], y[3]);
          pf[r] = *reinterpret_cast<const uint32_t*>(&a);
          pf[2 + r] = *reinterpret_cast<const uint32_t*>(&d);
        }
        // Tokens that some row of the tile does not see (the causal edge, and what lies behind
        // the last token): 0 * NaN is NaN, so their values take part without NaN, and rows that
        // do see a NaN get it afterwards.
        bool fix = false;
        if (tok0 + 16 > sq.len - sq.n) {
          bool nan = false;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bool in = tok0 + 2 * t + (j & 1) + 8 * (j >> 1) < end;
#pragma unroll
            for (int k = 0; k < VW; ++k) {
              if (!in) vw[j][k] = 0u;
              nan |= any_nan4(vw[j][k]);
              vw[j][k] = no_nan4(vw[j][k]);
            }
          }
          fix = __any_sync(FULL_MASK, nan);
        }
#pragma unroll
        for (int k = 0; k < VW; ++k) {
          const uint32_t a0 = __byte_perm(vw[0][k], vw[1][k], 0x5140), a1 = __byte_perm(vw[0][k], vw[1][k], 0x7362);
          const uint32_t b0 = __byte_perm(vw[2][k], vw[3][k], 0x5140), b1 = __byte_perm(vw[2][k], vw[3][k], 0x7362);
          mma_f16<NR>(o[4 * k], pf, e4m3x2_to_f16x2(static_cast<uint16_t>(a0)), e4m3x2_to_f16x2(static_cast<uint16_t>(b0)));
          mma_f16<NR>(o[4 * k + 1], pf, e4m3x2_to_f16x2(static_cast<uint16_t>(a0 >> 16)), e4m3x2_to_f16x2(static_cast<uint16_t>(b0 >> 16)));
          mma_f16<NR>(o[4 * k + 2], pf, e4m3x2_to_f16x2(static_cast<uint16_t>(a1)), e4m3x2_to_f16x2(static_cast<uint16_t>(b1)));
          mma_f16<NR>(o[4 * k + 3], pf, e4m3x2_to_f16x2(static_cast<uint16_t>(a1 >> 16)), e4m3x2_to_f16x2(static_cast<uint16_t>(b1 >> 16)));
        }
        if (fix) {
          for (int tk = 0; tk < 16 && tok0 + tk < end; ++tk)
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int d = 0; d < NU; ++d)
                if ((vt[tk * D + (2 * t + n) * NU + d] & 0x7f) == 0x7f)
#pragma unroll
                  for (int r = 0; r < NR; ++r)
                    if (tok0 + tk < seen[r]) o[d][2 * r + n] = NAN;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }

    // ---- join the warps: each scales its products to the row's largest maximum; added in order
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      l[r] += __shfl_xor_sync(FULL_MASK, l[r], 1);
      l[r] += __shfl_xor_sync(FULL_MASK, l[r], 2);
      if (t == 0) { s_m[warp][g + 8 * r] = m[r]; s_l[warp][g + 8 * r] = l[r]; }
    }
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float* dst = &s_o[warp][g + 8 * r][(2 * t + e) * NU];
#pragma unroll
        for (int n = 0; n < NU; n += 4)
          *reinterpret_cast<float4*>(dst + n) = make_float4(o[n][2 * r + e], o[n + 1][2 * r + e],
                                                            o[n + 2][2 * r + e], o[n + 3][2 * r + e]);
      }
    named_bar_sync(1, 32 * AT_WARPS);
    constexpr int N = D / 32;  // columns a lane takes of a row
    for (int r = warp; r < RT; r += AT_WARPS) {
      float mx = -INFINITY, sum = 0.f, y[N];
#pragma unroll
      for (int w = 0; w < AT_WARPS; ++w) mx = fmaxf(mx, s_m[w][r]);
      const float base = mx == -INFINITY ? 0.f : mx;
#pragma unroll
      for (int n = 0; n < N; ++n) y[n] = 0.f;
#pragma unroll
      for (int w = 0; w < AT_WARPS; ++w) {
        const float back = ex2f(s_m[w][r] - base);
        sum = fmaf(s_l[w][r], back, sum);
#pragma unroll
        for (int n = 0; n < N; ++n) y[n] = fmaf(s_o[w][r][lane * N + n], back, y[n]);
      }
      if (x.whole) {
        const int row = row0 + r;
        if (row < rows) {
          const int i = row / p.group;
          store_row<N>(p, (sq.q0 + i) * p.q_heads + x.h * p.group + (row - i * p.group), D,
                       lane * N, y, sum, mx);
        }
      } else {
        float* part = p.part + (int64_t(blockIdx.x) * 2 + (first_piece ? 0 : 1)) * RT * (D + 2);
#pragma unroll
        for (int n = 0; n < N; ++n) part[r * D + lane * N + n] = y[n];
        if (lane == 0) {
          part[RT * D + r] = mx;
          part[RT * D + RT + r] = sum;
        }
      }
    }
    named_bar_sync(1, 32 * AT_WARPS);
  }
}

// Joins the parts of the tiles that several CTAs hold.  One CTA per boundary between two runs
// of units; the CTA of the first boundary inside a tile joins that tile, from the run that
// holds its first chunk to the one that holds its last, in that order: a warp for each row,
// the weights of 32 parts at a time worked out side by side, then the parts added up.
template <int D, int RT>
__global__ void __launch_bounds__(32 * RT) kv8_join_kernel(const AttnParams p, int grid) {
  constexpr int N = D / 32;
  const int lane = threadIdx.x & 31, r = threadIdx.x >> 5;
  // Lengths and row ranges were there before the attention began: they are read, and the
  // tile is found, while it still runs.
  const Run run = find_run<RT>(p, int64_t(blockIdx.x) + 1, grid);
  const int64_t edge = run.u;  // first unit of run blockIdx.x + 1
  if (edge >= run.u_end) return;
  const SeqUnits sq = seq_units<RT>(p, run.b);
  const int64_t item = (edge - run.first) / sq.chunks;
  const int64_t i0 = run.first + item * sq.chunks, i1 = i0 + sq.chunks;  // the tile's units
  if (edge == i0) return;                  // the boundary lies between two tiles
  if (edge - run.per > i0) return;         // an earlier boundary lies inside this tile too
  const int64_t r0 = i0 / run.per, r1 = (i1 - 1) / run.per;  // runs that hold parts
  const int h = static_cast<int>(item / sq.tiles), tile = static_cast<int>(item % sq.tiles);
  const int row = tile * RT + r;
  if (row >= sq.n * p.group) return;
  constexpr int64_t STEP = RT * (D + 2);
  // the run that holds the tile's first chunk may hold another tile's part before it
  const float* parts = p.part + r0 * 2 * STEP;
  const int64_t lead = r0 * run.per >= i0 ? 0 : STEP;
  pdl_wait();
  float mx = -INFINITY, sum = 0.f, y[N];
#pragma unroll
  for (int n = 0; n < N; ++n) y[n] = 0.f;
  const int count = static_cast<int>(r1 - r0) + 1;
  for (int k0 = 0; k0 < count; k0 += 32) {
    const int mine = k0 + lane;
    const float* q = parts + mine * 2 * STEP + (mine == 0 ? lead : 0);
    const float m = mine < count ? __ldcg(q + RT * D + r) : -INFINITY;
    const float s = mine < count ? __ldcg(q + RT * D + RT + r) : 0.f;
    float nm = fmaxf(m, mx);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) nm = fmaxf(nm, __shfl_xor_sync(FULL_MASK, nm, o));
    const float base = nm == -INFINITY ? 0.f : nm;
    const float w = ex2f(m - base), back = ex2f(mx - base);
    float add = s * w;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) add += __shfl_xor_sync(FULL_MASK, add, o);
    sum = fmaf(sum, back, add);
#pragma unroll
    for (int n = 0; n < N; ++n) y[n] *= back;
    mx = nm;
    const int here = min(32, count - k0);
#pragma unroll 8
    for (int k = 0; k < here; ++k) {
      const float wk = __shfl_sync(FULL_MASK, w, k);
      const float* src = parts + (k0 + k) * 2 * STEP + (k0 + k == 0 ? lead : 0) + r * D + lane * N;
      if constexpr (N == 4) {
        const float4 z = __ldcg(reinterpret_cast<const float4*>(src));
        y[0] = fmaf(z.x, wk, y[0]); y[1] = fmaf(z.y, wk, y[1]);
        y[2] = fmaf(z.z, wk, y[2]); y[3] = fmaf(z.w, wk, y[3]);
      } else if constexpr (N == 2) {
        const float2 z = __ldcg(reinterpret_cast<const float2*>(src));
        y[0] = fmaf(z.x, wk, y[0]); y[1] = fmaf(z.y, wk, y[1]);
      } else {
        y[0] = fmaf(__ldcg(src), wk, y[0]);
      }
    }
  }
  const int i = row / p.group;
  store_row<N>(p, (sq.q0 + i) * p.q_heads + h * p.group + (row - i * p.group), D, lane * N, y, sum, mx);
}

cudaError_t kv8_read_device_error(uint32_t* code) {
  uint32_t v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_err_kv8, sizeof(v));
  if (e != cudaSuccess) return e;
  if (v) e = cudaMemcpyToSymbol(g_err_kv8, &zero, sizeof(zero));
  *code |= v;
  return e;
}

namespace {

lilicorr_status fail(lilicorr_status st, const char* msg) {
  set_last_error(msg);
  return st;
}

// Null where the cache's description is in order, else what is wrong with it.
const char* cache_error(const lilicorr_kv8_cache* c) {
  if (!c || !c->k_pages || !c->v_pages || !c->k_scale || !c->v_scale) return "null cache pointer";
  if (c->head_dim != 32 && c->head_dim != 64 && c->head_dim != 128) return "head_dim is 32, 64 or 128";
  if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) return "page is 16, 32, 64 or 128";
  if (c->kv_heads < 1 || c->kv_heads > 1024) return "1 <= kv_heads <= 1024";
  if (c->n_pages < 1 || c->n_pages > INT_MAX) return "1 <= n_pages < 2^31";
  if (reinterpret_cast<uintptr_t>(c->k_pages) % 16 || reinterpret_cast<uintptr_t>(c->v_pages) % 16)
    return "pages are 16-byte aligned";
  if (reinterpret_cast<uintptr_t>(c->k_scale) % 4 || reinterpret_cast<uintptr_t>(c->v_scale) % 4)
    return "scales are 4-byte aligned";
  return nullptr;
}
const char* batch_error(const int32_t* q_start, const int32_t* kv_len, int64_t batch,
                        const int32_t* table, int64_t table_stride, int32_t cols, int64_t total,
                        int32_t max_new, int page) {
  if (!q_start || !kv_len || !table) return "null pointer";
  if (batch < 1 || batch > (1 << 20)) return "1 <= batch <= 2^20";
  if (cols < 1 || int64_t(cols) * page > INT_MAX - 256) return "a table row holds 1 page to 2^31 tokens";
  if (table_stride < cols) return "table_stride is at least its columns";
  if (total < 0 || total > INT_MAX) return "rows are out of range";
  if (max_new < 1 || max_new > (1 << 24)) return "1 <= max_new <= 2^24";
  return nullptr;
}
const char* rows_error(const void* x, int64_t tok, int64_t head, int64_t heads, int D) {
  if (!x) return "null pointer";
  if (reinterpret_cast<uintptr_t>(x) % 16) return "rows are 16-byte aligned";
  if (tok % 8 || head % 8) return "row strides are multiples of 8 elements";
  if (tok < 0 || head < 0 || tok > (int64_t(1) << 40) || head > (int64_t(1) << 40)) return "a row stride is out of range";
  (void)heads;
  (void)D;
  return nullptr;
}
Kv8 view(const lilicorr_kv8_cache* c) {
  return Kv8{static_cast<uint8_t*>(c->k_pages), static_cast<uint8_t*>(c->v_pages), c->k_scale,
             c->v_scale, c->n_pages, c->kv_heads, c->page};
}

struct AttnPlan {
  int rt;    // rows of a tile
  int grid;  // CTAs
  size_t ws;
};
AttnPlan attn_plan(int32_t max_new, int group, int D) {
  AttnPlan pl{};
  pl.rt = int64_t(max_new) * group <= 8 ? 8 : 16;
  pl.grid = (pl.rt == 8 ? AttnShape<128, 8>::CTAS : AttnShape<128, 16>::CTAS) * device_sm_count();
  pl.ws = size_t(pl.grid) * 2 * pl.rt * (D + 2) * sizeof(float);
  return pl;
}

template <int D, int RT>
cudaError_t attention_launch(const AttnParams& prm, int grid, cudaStream_t stream) {
  constexpr int smem = AttnShape<D, RT>::SMEM;
  cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void*>(kv8_attention_kernel<D, RT>), smem);
  if (e != cudaSuccess) return e;
  kv8_attention_kernel<D, RT><<<grid, 32 * AT_WARPS + 32, smem, stream>>>(prm);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  PdlScope pdl(true);
  e = launch_k(kv8_join_kernel<D, RT>, dim3(grid), dim3(32 * RT), 0, stream, prm, grid);
  if (e == cudaSuccess) note_launch(2);
  return e;
}

}  // namespace
}  // namespace lilicorr

using namespace lilicorr;

extern "C" {

lilicorr_status lilicorr_kv8_append(const lilicorr_kv8_cache* cache, const void* k,
                                    int64_t k_token_stride, int64_t k_head_stride, const void* v,
                                    int64_t v_token_stride, int64_t v_head_stride, int64_t total,
                                    const int32_t* q_start, const int32_t* kv_len, int64_t batch,
                                    const int32_t* block_table, int64_t table_stride, int32_t cols,
                                    int32_t max_new, const int32_t* tail_src, void* stream) {
  const char* why = cache_error(cache);
  if (!why) why = batch_error(q_start, kv_len, batch, block_table, table_stride, cols, total, max_new, cache->page);
  if (!why) why = rows_error(k, k_token_stride, k_head_stride, cache->kv_heads, cache->head_dim);
  if (!why) why = rows_error(v, v_token_stride, v_head_stride, cache->kv_heads, cache->head_dim);
  if (why) return fail(LILICORR_ERR_INVALID_ARG, why);
  AppendParams prm{};
  prm.c = view(cache);
  prm.k = static_cast<const __nv_bfloat16*>(k);
  prm.v = static_cast<const __nv_bfloat16*>(v);
  prm.k_tok = k_token_stride; prm.k_head = k_head_stride;
  prm.v_tok = v_token_stride; prm.v_head = v_head_stride;
  prm.total = total;
  prm.q_start = q_start; prm.kv_len = kv_len; prm.table = block_table; prm.tail_src = tail_src;
  prm.table_stride = table_stride;
  prm.cols = cols;
  prm.max_new = max_new;
  const int page = cache->page, D = cache->head_dim;
  prm.grow = std::min<int>((max_new + page - 2) / page + 1, cols);
  const int64_t ctas = batch * prm.grow * cache->kv_heads * 2;
  if (ctas > INT_MAX) return fail(LILICORR_ERR_INVALID_ARG, "batch * max_new * kv_heads is too large for one call");
  const int vpt = (page * D / 8 + AP_THREADS - 1) / AP_THREADS;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dim3 grid(static_cast<unsigned>(ctas));
  if (vpt <= 1) kv8_append_kernel<1><<<grid, AP_THREADS, 0, st>>>(prm, D);
  else if (vpt <= 2) kv8_append_kernel<2><<<grid, AP_THREADS, 0, st>>>(prm, D);
  else if (vpt <= 4) kv8_append_kernel<4><<<grid, AP_THREADS, 0, st>>>(prm, D);
  else if (vpt <= 8) kv8_append_kernel<8><<<grid, AP_THREADS, 0, st>>>(prm, D);
  else kv8_append_kernel<16><<<grid, AP_THREADS, 0, st>>>(prm, D);
  note_launch();
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(LILICORR_ERR_CUDA, cudaGetErrorString(e));
  return LILICORR_OK;
}

size_t lilicorr_kv8_attention_workspace_bytes(int32_t max_new, int32_t q_heads, int32_t kv_heads,
                                              int32_t head_dim) {
  if (max_new < 1 || max_new > (1 << 24) || kv_heads < 1 || kv_heads > 1024 || q_heads < kv_heads ||
      q_heads % kv_heads || q_heads / kv_heads > 1024 ||
      (head_dim != 32 && head_dim != 64 && head_dim != 128))
    return 0;
  return attn_plan(max_new, q_heads / kv_heads, head_dim).ws;
}

lilicorr_status lilicorr_kv8_attention(const lilicorr_kv8_cache* cache, const void* q,
                                       int64_t q_token_stride, int64_t q_head_stride,
                                       int64_t total, int32_t q_heads, const int32_t* q_start,
                                       const int32_t* kv_len, int64_t batch,
                                       const int32_t* block_table, int64_t table_stride,
                                       int32_t cols, int32_t max_new, float scale, void* out,
                                       float* lse, void* workspace, size_t workspace_bytes,
                                       void* stream) {
  const char* why = cache_error(cache);
  if (!why) why = batch_error(q_start, kv_len, batch, block_table, table_stride, cols, total, max_new, cache->page);
  if (!why) why = rows_error(q, q_token_stride, q_head_stride, q_heads, cache->head_dim);
  if (!why && (!out || reinterpret_cast<uintptr_t>(out) % 16)) why = "out is null or not 16-byte aligned";
  if (!why && (q_heads < 1 || q_heads % cache->kv_heads || q_heads / cache->kv_heads > 1024))
    why = "q_heads is a multiple of kv_heads, at most 1024 times it";
  // one sequence's work units (tiles x heads x chunks of 64 tokens) are counted in 32 bits
  if (!why && (int64_t(max_new) * (q_heads / cache->kv_heads) / 8 + 1) * cache->kv_heads *
                  ((int64_t(cols) * cache->page + 63) / 64) > UINT_MAX)
    why = "max_new * q_heads * the table's tokens are too large";
  if (!why && !std::isfinite(scale)) why = "scale is not finite";
  if (why) return fail(LILICORR_ERR_INVALID_ARG, why);
  const int D = cache->head_dim, group = q_heads / cache->kv_heads;
  const AttnPlan pl = attn_plan(max_new, group, D);
  if (!workspace || workspace_bytes < pl.ws || reinterpret_cast<uintptr_t>(workspace) % 256)
    return fail(LILICORR_ERR_WORKSPACE, "lilicorr_kv8_attention: workspace missing, too small or misaligned");
  AttnParams prm{};
  prm.c = view(cache);
  prm.q = static_cast<const __nv_bfloat16*>(q);
  prm.q_tok = q_token_stride; prm.q_head = q_head_stride;
  prm.total = total;
  prm.q_heads = q_heads;
  prm.group = group;
  prm.q_start = q_start; prm.kv_len = kv_len; prm.table = block_table;
  prm.batch = batch;
  prm.table_stride = table_stride;
  prm.cols = cols;
  prm.max_new = max_new;
  prm.page_log2 = cache->page == 16 ? 4 : cache->page == 32 ? 5 : cache->page == 64 ? 6 : 7;
  prm.scale2 = scale * LOG2E_F;
  prm.out = static_cast<__nv_bfloat16*>(out);
  prm.lse = lse;
  prm.part = static_cast<float*>(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
#define LC_ATTN(DD) \
  e = pl.rt == 8 ? attention_launch<DD, 8>(prm, pl.grid, st) : attention_launch<DD, 16>(prm, pl.grid, st)
  if (D == 128) LC_ATTN(128);
  else if (D == 64) LC_ATTN(64);
  else LC_ATTN(32);
#undef LC_ATTN
  if (e != cudaSuccess) return fail(LILICORR_ERR_CUDA, cudaGetErrorString(e));
  return LILICORR_OK;
}

}  // extern "C"
