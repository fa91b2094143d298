// What the two kernels of the cache attention share: the deal of the work, the ring of its
// pieces, and the joining of tiles that several CTAs hold.
#pragma once

#include "kv8.cuh"

namespace lilicorr {

static __device__ uint32_t g_err_kv8_attn;  // (each unit has its own)

constexpr int AT_CHUNK = 128;
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

// ------------------------------------------------------------------------ the deal of work

// Each tile counts HEAD_UNITS more than its chunks, at its front, for what it costs beside them
// (its q, its first maxima, its outputs), so that runs of many short tiles take no longer than
// others.  Measured: 3, 4, 5 and 6 chunks' for 128 rows, 64 sequences of 16 new tokens, 93.7, 93.7,
// 93.5 and 94.8 us (weights not yet held up in f16); 0, 1 and 2 for few, 128 sequences of one, 199.5, 197.1 and 198.0.
template <int ROWS>
constexpr int HEAD_UNITS = ROWS == 128 ? 4 : 1;

struct SeqUnits {
  int n, len, tiles, chunks;
  int64_t q0, units;
};
template <int ROWS>
__device__ __forceinline__ SeqUnits seq_units(const AttnParams& p, int64_t b) {
  const SeqRange r = seq_range(p.q_start, p.kv_len, b, p.total, p.max_new,
                               int64_t(p.cols) << p.page_log2, &g_err_kv8_attn);
  SeqUnits u;
  u.n = r.n;
  u.len = r.len;
  u.q0 = r.q0;
  u.tiles = (r.n * p.group + ROWS - 1) / ROWS;
  u.chunks = max(1, (r.len + AT_CHUNK - 1) / AT_CHUNK);
  u.units = int64_t(u.tiles) * p.c.heads * (u.chunks + HEAD_UNITS<ROWS>);
  return u;
}

// The units of all sequences, and where run `run` of `runs` begins, by one warp.
struct Run {
  int64_t per;       // units of a run
  int64_t u, u_end;  // this run's units
  int64_t b, first;  // the sequence of unit u, and that sequence's first unit
};
template <int ROWS>
__device__ __forceinline__ Run find_run(const AttnParams& p, int64_t run, int runs) {
  const int lane = threadIdx.x & 31;
  int64_t t = 0;
#pragma unroll 1
  for (int64_t b = lane; b < p.batch; b += 32) t += seq_units<ROWS>(p, b).units;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) t += __shfl_xor_sync(FULL_MASK, t, o);
  Run r;
  r.per = t < INT_MAX / 2 ? int64_t((static_cast<uint32_t>(t) + runs - 1) / static_cast<uint32_t>(runs))
                          : (t + runs - 1) / runs;
  r.u = run * r.per;
  r.u_end = min(t, r.u + r.per);
  r.b = p.batch;
  r.first = 0;
  if (r.u >= r.u_end) return r;
#pragma unroll 1
  for (int64_t b0 = 0; b0 < p.batch; b0 += 32) {  // the 32 sequences among whose units u is
    const int64_t mine = b0 + lane < p.batch ? seq_units<ROWS>(p, b0 + lane).units : 0;
    int64_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(FULL_MASK, sum, o);
      if (lane >= o) sum += x;
    }
    const unsigned past = __ballot_sync(FULL_MASK, r.first + sum > r.u);
    if (past) {
      const int l = __ffs(past) - 1;
      r.b = b0 + l;
      r.first += __shfl_sync(FULL_MASK, sum - mine, l);
      break;
    }
    r.first += __shfl_sync(FULL_MASK, sum, 31);
  }
  return r;
}

// The pieces of a run, in order: the chunks [c0, c1) of one tile each.
template <int ROWS>
struct Pieces {
  const AttnParams& p;
  const Run run;
  int64_t b, u;       // the next unit, and its sequence
  SeqUnits sq;
  int h, tile, at;    // its head and tile, and its place among the tile's units
  int c0, c1, count;  // the piece; pieces so far
  int ph, ptile;
  int64_t pb;
  SeqUnits psq;
  __device__ __forceinline__ Pieces(const AttnParams& p_, const Run& r) : p(p_), run(r), b(r.b), u(r.u), h(0), tile(0), at(0), count(0) {
    if (u < run.u_end) {
      sq = seq_units<ROWS>(p, b);
      const uint32_t in = static_cast<uint32_t>(u - run.first);  // a sequence's units fit 32 bits (host)
      const uint32_t len = sq.chunks + HEAD_UNITS<ROWS>, item = in / len;
      at = static_cast<int>(in - item * len);
      h = item / sq.tiles;
      tile = item - h * sq.tiles;
    }
  }
  __device__ __forceinline__ bool next() {
    while (u < run.u_end) {
      while (sq.units == 0) sq = seq_units<ROWS>(p, ++b);  // sequences without new tokens
      const int len = sq.chunks + HEAD_UNITS<ROWS>;
      const int to = static_cast<int>(min(int64_t(len), at + (run.u_end - u)));
      c0 = max(0, at - HEAD_UNITS<ROWS>);
      c1 = max(0, to - HEAD_UNITS<ROWS>);
      ph = h;
      ptile = tile;
      pb = b;
      psq = sq;
      u += to - at;
      at = to;
      if (at == len) {
        at = 0;
        if (++tile == sq.tiles) {
          tile = 0;
          if (++h == p.c.heads) {
            h = 0;
            if (u < run.u_end) sq = seq_units<ROWS>(p, ++b);
          }
        }
      }
      if (c1 > c0) {
        ++count;
        return true;
      }
    }
    return false;
  }
  __device__ __forceinline__ int rows() const { return min(ROWS, psq.n * p.group - ptile * ROWS); }
  // tokens that the tile's last row sees
  __device__ __forceinline__ int end() const {
    return max(0, min(psq.len, psq.len - psq.n + (ptile * ROWS + rows() - 1) / p.group + 1));
  }
  __device__ __forceinline__ int whole() const { return c0 == 0 && c1 == psq.chunks ? 1 : 0; }
  __device__ __forceinline__ int slot() const { return 2 * static_cast<int>(blockIdx.x) + (count > 1); }
};

struct PageScale {  // of the tokens of one page
  float k, log2_v, inv_v;
  int ok;  // the page was loaded
};
// The logarithm of the mantissa and the reciprocal are the hardware's approximations: exact for
// powers of two, off by 2^-22 and 2^-23 at most for others (besides f32's rounding of the
// logarithm), a relative error of the weights at the level of f32's own.  (The rounded functions held the loading warp up: 108 -> 106 us for a call
// of blocks, 200 -> 197 for one of single tokens.)
__device__ __forceinline__ float log2_of(float x) {  // positive and finite
  const bool small = x < 1e-20f;
  const uint32_t u = __float_as_uint(small ? x * 18446744073709551616.f : x);
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(__uint_as_float((u & 0x7fffffu) | 0x3f800000u)));
  return y + static_cast<float>(static_cast<int>(u >> 23) - (small ? 127 + 64 : 127));
}
__device__ __forceinline__ PageScale page_scale_of(float ks, float vs, bool ok) {
  PageScale s;
  s.k = ks;
  s.log2_v = log2_of(vs);
  asm("rcp.approx.f32 %0, %1;" : "=f"(s.inv_v) : "f"(vs));
  s.ok = ok ? 1 : 0;
  return s;
}

// Writes a row's outputs, E columns a lane, from its products, sum of weights and maximum.
template <int E>
__device__ __forceinline__ void store_row(const AttnParams& p, int64_t at, int D, int lane,
                                          const float (&y)[E], float sum, float m) {
  const float inv = sum == 0.f ? 0.f : 1.f / sum;  // no token seen: 0
  __nv_bfloat16* o = p.out + at * D + lane * E;
  if constexpr (E == 4) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(y[0] * inv, y[1] * inv);
    const __nv_bfloat162 c = __floats2bfloat162_rn(y[2] * inv, y[3] * inv);
    *reinterpret_cast<uint2*>(o) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                              *reinterpret_cast<const uint32_t*>(&c));
  } else if constexpr (E == 2) {
    *reinterpret_cast<__nv_bfloat162*>(o) = __floats2bfloat162_rn(y[0] * inv, y[1] * inv);
  } else {
    *o = __float2bfloat16_rn(y[0] * inv);
  }
  if (p.lse && lane == 0) p.lse[at] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * LN2_F;
}

// ------------------------------------------------------------------------------- joining

// The tile that boundary `at` between two runs lies inside of, among its chunks: `count` parts
// from the run that holds its first chunk to the one that holds its last, and so count - 1
// boundaries, of which this is number `j`.
template <int D, int ROWS>
struct JoinTile {
  static constexpr int64_t STEP = ROWS * (D + 2);
  SeqUnits sq;
  int h, tile, count, j;  // count 0: none
  const float* parts;
  int64_t lead;           // the run of the first chunk may hold another tile's part before it
  __device__ __forceinline__ JoinTile(const AttnParams& p, int64_t at, int runs) : count(0) {
    const Run run = find_run<ROWS>(p, at + 1, runs);
    const int64_t edge = run.u;  // first unit of the run behind the boundary
    if (edge >= run.u_end) return;
    sq = seq_units<ROWS>(p, run.b);
    const uint32_t in = static_cast<uint32_t>(edge - run.first);
    const uint32_t len = sq.chunks + HEAD_UNITS<ROWS>, item = in / len;
    // the tile's units, and the first of its chunks
    const int64_t i0 = run.first + int64_t(item) * len, i1 = i0 + len, ic = i0 + HEAD_UNITS<ROWS>;
    if (edge <= ic) return;  // the boundary lies before the tile's chunks
    h = item / sq.tiles;
    tile = item - h * sq.tiles;
    const int64_t r0 = ic / run.per;
    count = static_cast<int>((i1 - 1) / run.per - r0) + 1;
    j = static_cast<int>(at - r0);
    parts = p.part + r0 * 2 * STEP;
    lead = r0 * run.per >= i0 ? 0 : STEP;
  }
  __device__ __forceinline__ const float* part(int k) const { return parts + k * 2 * STEP + (k == 0 ? lead : 0); }
};

template <int E>
__device__ __forceinline__ void load_row(const float* src, float (&z)[E]) {
  if constexpr (E == 4) {
    const float4 v = __ldcg(reinterpret_cast<const float4*>(src));
    z[0] = v.x; z[1] = v.y; z[2] = v.z; z[3] = v.w;
  } else if constexpr (E == 2) {
    const float2 v = __ldcg(reinterpret_cast<const float2*>(src));
    z[0] = v.x; z[1] = v.y;
  } else {
    z[0] = __ldcg(src);
  }
}

// Row r's maximum, sum and products (a warp's, E columns a lane) of the parts [k0, k1), in order;
// the reads of A parts are under way together.
template <int D, int ROWS, int A>
__device__ __forceinline__ void join_parts(const JoinTile<D, ROWS>& t, int r, int k0, int k1, float& mx, float& sum,
                                           float (&y)[D / 32]) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  mx = -INFINITY;
  sum = 0.f;
#pragma unroll
  for (int n = 0; n < E; ++n) y[n] = 0.f;
#pragma unroll 1
  for (int k = k0; k < k1; k += A) {
    float m[A], s[A], z[A][E];
#pragma unroll
    for (int i = 0; i < A; ++i) {
      m[i] = -INFINITY;
      s[i] = 0.f;
#pragma unroll
      for (int n = 0; n < E; ++n) z[i][n] = 0.f;
      if (k + i < k1) {
        const float* part = t.part(k + i);
        m[i] = __ldcg(part + ROWS * D + r);
        s[i] = __ldcg(part + ROWS * D + ROWS + r);
        load_row<E>(part + r * D + lane * E, z[i]);
      }
    }
    float nm = mx;
#pragma unroll
    for (int i = 0; i < A; ++i) nm = fmaxf(nm, m[i]);
    const float base = nm == -INFINITY ? 0.f : nm, back = ex2(mx - base);
    sum *= back;
#pragma unroll
    for (int n = 0; n < E; ++n) y[n] *= back;
#pragma unroll
    for (int i = 0; i < A; ++i) {
      const float w = ex2(m[i] - base);  // (0 where there is no part)
      sum = fmaf(s[i], w, sum);
#pragma unroll
      for (int n = 0; n < E; ++n) y[n] = fmaf(z[i][n], w, y[n]);
    }
    mx = nm;
  }
}

// Joins the parts of the tiles that several CTAs hold, always in order: Y CTAs of W warps for each
// boundary between two runs.  The CTAs of all boundaries inside a tile share its rows, and where
// there are more warps than rows, W / rows of them share a row's parts.  What bounds it is the
// latency of the reads, so as many as can be are under way: 8 parts of a row, or (a tile of 128 in
// two parts, the usual case: all warps are resident at once then) two parts of four rows.  Measured,
// the whole call: 64 sequences of 16 new tokens 5.9 us less than with a row a warp (99.9 now); 16 new
// tokens of one sequence over 131,072 with one key / value head 32 us, 185 with the CTAs of one
// boundary at work alone; two sequences' single tokens over as many, 8 heads, 56 and 58.
template <int D, int ROWS, int W, int Y>
__global__ void __launch_bounds__(32 * W) kv8_join_kernel(const AttnParams p, int runs) {
  constexpr int E = D / 32, R = ROWS / (W * Y);  // columns of a lane; rows of a warp, in the usual case
  __shared__ float s_y[W][D], s_m[W], s_l[W];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // Lengths and row ranges were there before the attention began: they are read, and the
  // tile is found, while it still runs.  Every CTA waits for it before it may leave: what comes
  // after this kernel takes its end for the attention's too.
  const JoinTile<D, ROWS> t(p, blockIdx.x, runs);
  pdl_wait();
  if (t.count == 0) return;
  const int rows = min(ROWS, t.sq.n * p.group - t.tile * ROWS);
  const int ctas = (t.count - 1) * Y, mine = (ROWS + ctas - 1) / ctas;  // rows of a CTA
  const int r0 = (t.j * Y + blockIdx.y) * mine, r1 = min(rows, r0 + mine);
  if (r0 >= r1) return;
  float mx, sum, y[E];
  auto store = [&](int r) {
    const int row = t.tile * ROWS + r, i = row / p.group;
    store_row<E>(p, (t.sq.q0 + i) * p.q_heads + t.h * p.group + (row - i * p.group), D, lane, y, sum, mx);
  };
  if (R > 1 && t.count == 2) {
    const int q0 = r0 + warp * R;
    float m[2][R], s[2][R], z[2][R][E];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int q = 0; q < R; ++q) {
        const int r = min(q0 + q, r1 - 1);
        m[k][q] = __ldcg(t.part(k) + ROWS * D + r);
        s[k][q] = __ldcg(t.part(k) + ROWS * D + ROWS + r);
        load_row<E>(t.part(k) + r * D + lane * E, z[k][q]);
      }
#pragma unroll
    for (int q = 0; q < R; ++q) {
      if (q0 + q >= r1) break;
      mx = fmaxf(m[0][q], m[1][q]);
      const float base = mx == -INFINITY ? 0.f : mx, a = ex2(m[0][q] - base), b = ex2(m[1][q] - base);
      sum = fmaf(s[1][q], b, s[0][q] * a);
#pragma unroll
      for (int n = 0; n < E; ++n) y[n] = fmaf(z[1][q][n], b, z[0][q][n] * a);
      store(q0 + q);
    }
    return;
  }
  // warps of a row: no more than have 8 parts each
  const int share = mine < W ? min(W / mine, (t.count + 7) / 8) : 1;
  if (share == 1) {
    for (int r = r0 + warp; r < r1; r += W) {
      join_parts<D, ROWS, 8>(t, r, 0, t.count, mx, sum, y);
      store(r);
    }
    return;
  }
  const int r = r0 + warp / share, part = warp % share, each = (t.count + share - 1) / share;
  if (r < r1) {
    join_parts<D, ROWS, 8>(t, r, part * each, min(t.count, (part + 1) * each), mx, sum, y);
#pragma unroll
    for (int n = 0; n < E; ++n) s_y[warp][lane * E + n] = y[n];
    if (lane == 0) {
      s_m[warp] = mx;
      s_l[warp] = sum;
    }
  }
  __syncthreads();
  if (r >= r1 || part != 0) return;
  for (int k = 1; k < share; ++k) mx = fmaxf(mx, s_m[warp + k]);
  const float base = mx == -INFINITY ? 0.f : mx, own = ex2(s_m[warp] - base);
  sum *= own;
#pragma unroll
  for (int n = 0; n < E; ++n) y[n] *= own;
  for (int k = 1; k < share; ++k) {
    const float w = ex2(s_m[warp + k] - base);
    sum = fmaf(s_l[warp + k], w, sum);
#pragma unroll
    for (int n = 0; n < E; ++n) y[n] = fmaf(s_y[warp + k][lane * E + n], w, y[n]);
  }
  store(r);
}

// A tile of at most 16 rows (kv8_attn_few.cu).
int kv8_few_runs(int rows, int D);
cudaError_t kv8_few_launch(const AttnParams& p, int D, int rows, cudaStream_t stream);
cudaError_t kv8_few_read_device_error(uint32_t* code);

}  // namespace lilicorr
