// Beam search next to the rerank: the choice over beams and vocabulary from one step's
// logits (the logit pass of step a1 followed by a merge over the beams), and the gather
// of per-beam states by the chosen parents.
#include <climits>
#include <cmath>

#include <algorithm>

#include "kernels.cuh"

namespace lilicorr {

static __device__ uint32_t g_err_beam;

// ------------------------------------------------------------------------------ selection
// s(i, v) = score_i + x_iv - log sum_u exp x_iu, the M best of a batch entry's beams by
// (s desc, i * V + v asc).  Within a beam the order is that of its logits, so a beam's part
// of the M best are among its own M best logits, which the logit pass leaves, for every
// segment of a beam's row, in a record beside (m2, S): the segment's sum_u exp x_iu is S 2^m2.
//
// Ranks are decided in double: two beams' candidates may differ by less than the float
// rounding of a score of a few tens (2e-6), and then a float score would rank them by its
// rounding.  The score is rounded to float once, as it is stored.  Double arithmetic is slow
// on this part, so the log-partition is put together from floats, log2 S = e + log2 f with f
// near 1, and only the sums m2 + e + log2 f, the division by the float nearest log2 e that the
// logit pass scales its logits by, and the scores themselves are doubles.  The sums S are floats,
// in an order that the rows' alignment sets: beams whose candidates differ by less than what that
// leaves out may change places, and only rows that begin alike have S alike.
//
// One CTA per batch entry; bound by latency, the logit pass by HBM (with K = 32 by the
// instructions of its top-K: 128 entries of 16 beams, V 151,936 in bf16, take 130 us, 117 of them
// that pass at 4.65 TB/s; one entry of 4 beams, K = 8, takes 9.9 in all).  A few warps for each beam
// join its segments' sorted lists (the records of four segments are read at a time); then a thread for each
// candidate finds its rank, the number of better ones, by binary searches in the beams' lists,
// so that no step waits for the one before as in a merge that takes one candidate at a time
// (one entry of 4 beams, V 151,936: 11.4 us for the call with the lists joined one by one and the
// lists searched in turn, 9.7 with them joined two by two and four searched at a time; the look for
// rows of very large logits adds 0.2).

// Order-preserving key: unsigned comparison of keys = comparison of the doubles.
__device__ __forceinline__ uint64_t double_key(double d) {
  const int64_t b = __double_as_longlong(d + 0.0);
  return b < 0 ? ~static_cast<uint64_t>(b) : static_cast<uint64_t>(b) | (1ull << 63);
}

constexpr int BM_MAX = 32;   // beams, and entries taken
constexpr int BM_WARPS = 32;  // up to as many warps join lists
// Rows whose largest logit t is of this magnitude or more (every token masked with the type's lowest
// value, say): a record's m2 = fl(t log2 e) is off by up to 64 octaves and more there, and its sum
// of no use.  But then floats are 64 or more apart, so that of the sum of exp(x - t) only the
// tokens equal to t are left (e^-64 is below a double's half step): they are counted.
constexpr float BM_FAR = 1073741824.f;

// The logarithm of that number into *rest, by the whole CTA; NaN where a token is NaN.  (Out of line, as
// all that such rows need, so that the others' code stays short.)
template <typename T>
__device__ __noinline__ void count_equal(const T* x, int64_t V, float top, unsigned* count, double* rest) {
  unsigned n = 0;
  bool nan = false;
  for (int64_t t = threadIdx.x; t < V; t += blockDim.x) {
    const float z = static_cast<float>(x[t]);
    n += z == top;
    nan |= isnan(z);
  }
  if (threadIdx.x == 0) *count = 0;
  nan = __syncthreads_or(nan);
  n = __reduce_add_sync(FULL_MASK, n);
  if ((threadIdx.x & 31) == 0) atomicAdd(count, n);
  __syncthreads();
  if (threadIdx.x == 0) *rest = nan ? NAN : log(static_cast<double>(*count));
}

// (m, s) takes (om, os): s 2^m + os 2^om.
__device__ __forceinline__ void join_sum(float& m, float& s, float om, float os) {
  const float M = fmaxf(m, om);
  s = s * ex2(m - M) + os * ex2(om - M);
  m = M;
}

__global__ void __launch_bounds__(32 * BM_MAX)
    beam_merge_kernel(const char* __restrict__ records, const float* __restrict__ scores,
                      const uint8_t* __restrict__ finished, const void* __restrict__ logits,
                      int64_t V, int64_t row_stride, int es, int beams, int P, int K, int M,
                      int pad_id, float* __restrict__ out_score, int32_t* __restrict__ out_token,
                      int32_t* __restrict__ out_parent) {
  // lists as the warps leave them, [beam * warps of a beam][32]
  __shared__ float s_v[BM_MAX][32];
  __shared__ int s_id[BM_MAX][32];
  __shared__ float s_m[BM_MAX], s_s[BM_MAX];
  // candidates, [beam][K]
  __shared__ uint64_t s_key[BM_MAX][BM_MAX];
  __shared__ int s_left[BM_MAX];
  __shared__ double s_rest[BM_MAX];
  __shared__ unsigned s_count;
  __shared__ float o_score[BM_MAX];
  __shared__ int o_token[BM_MAX], o_parent[BM_MAX];
  const int64_t b = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (blockDim.x >> 5) / beams;  // warps of a beam
  const int w = warp / per, part = warp - w * per;
  constexpr double NONE = -INFINITY;
  // scores and marks were there before the logit pass began
  const double score = w < beams ? static_cast<double>(__ldg(scores + b * beams + w)) : NONE;
  const bool live = score > NONE;  // a NaN is dead too
  const bool done = live && finished && finished[b * beams + w];
  pdl_wait();
  pdl_trigger();
  if (tid < M) {
    o_score[tid] = -INFINITY;
    o_token[tid] = pad_id;
    o_parent[tid] = 0;
  }
  if (w < beams && live && !done) {
    const int words = 2 * K + 2;
    const int32_t* rec = reinterpret_cast<const int32_t*>(records) + (b * beams + w) * P * words;
    float v = -INFINITY, m = -1e30f, s = 0.f;
    int id = INT_MAX;
    for (int k0 = part; k0 < P; k0 += 4 * per) {
      float bv[4];
      int bi[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = k0 + i * per;
        const bool has = lane < K && k < P;
        bv[i] = has ? __int_as_float(__ldcg(rec + k * words + 2 + lane)) : -INFINITY;
        bi[i] = has ? __ldcg(rec + k * words + 2 + K + lane) : INT_MAX;
      }
      if (k0 + lane * per < P && lane < 4) {
        const float2 ms = __ldcg(reinterpret_cast<const float2*>(rec + (k0 + lane * per) * words));
        join_sum(m, s, ms.x, ms.y);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (k0 + i * per < P) bitonic_merge(v, id, bv[i], bi[i], lane);
    }
#pragma unroll
    for (int o = 2; o >= 1; o >>= 1)
      join_sum(m, s, __shfl_xor_sync(FULL_MASK, m, o), __shfl_xor_sync(FULL_MASK, s, o));
    s_v[warp][lane] = v;
    s_id[warp][lane] = id;
    if (lane == 0) {
      s_m[warp] = m;
      s_s[warp] = s;
    }
  }
  // the warps' lists of a beam, two by two
  for (int d = 1; d < per; d *= 2) {
    __syncthreads();
    if (w < beams && live && !done && part % (2 * d) == 0 && part + d < per) {
      float v = s_v[warp][lane];
      int id = s_id[warp][lane];
      bitonic_merge(v, id, s_v[warp + d][lane], s_id[warp + d][lane], lane);
      s_v[warp][lane] = v;
      s_id[warp][lane] = id;
      if (lane == 0) join_sum(s_m[warp], s_s[warp], s_m[warp + d], s_s[warp + d]);
    }
  }
  auto is_far = [](float t) { return fabsf(t) >= BM_FAR && fabsf(t) < INFINITY; };
  if (__syncthreads_or(lane == 0 && part == 0 && w < beams && live && !done && is_far(s_v[warp][0]))) {
    for (int j = 0; j < beams; ++j) {
      if (!(scores[b * beams + j] > -INFINITY) || (finished && finished[b * beams + j]) || !is_far(s_v[j * per][0])) continue;
      const int64_t at = (b * beams + j) * row_stride;
      if (es == 2) count_equal(static_cast<const __nv_bfloat16*>(logits) + at, V, s_v[j * per][0], &s_count, &s_rest[j]);
      else count_equal(static_cast<const float*>(logits) + at, V, s_v[j * per][0], &s_count, &s_rest[j]);
    }
    __syncthreads();
  }
  const int i = warp;  // from here a warp for each beam
  int left = 0;
  uint64_t key = 0;
  float value = 0.f;
  int token = 0;
  if (i < beams) {
    const double own = static_cast<double>(__ldg(scores + b * beams + i));
    if (own > NONE) {
      if (finished && finished[b * beams + i]) {
        left = 1;
        token = pad_id;
        key = double_key(own);
        value = static_cast<float>(own);
      } else {
        const float v = s_v[i * per][lane], m = s_m[i * per], s = s_s[i * per];
        const int id = s_id[i * per][lane];
        const float top = s_v[i * per][0];
        const bool far = is_far(top);
        if (far || s > 0.f) {  // a row with no finite logit has no candidate
          double norm = top, rest = 0.;  // the log-partition is their sum
          if (far) {
            rest = s_rest[i];
          } else {
            int e;
            float f = frexpf(s, &e);
            if (f < 0.70710678f) { f *= 2.f; --e; }
            norm = (static_cast<double>(m) + static_cast<double>(e) + static_cast<double>(log2f(f))) *
                   (1.0 / static_cast<double>(1.4426950408889634f));
          }
          const double c = own + (static_cast<double>(v) - norm - rest);
          const bool there = lane < K && c > NONE;
          left = __popc(__ballot_sync(FULL_MASK, there));  // the list is sorted
          key = double_key(c);
          value = static_cast<float>(c);
          token = id;
        }
      }
    }
    s_key[i][lane] = lane < left ? key : 0;
    if (lane == 0) s_left[i] = left;
  }
  __syncthreads();
  if (i < beams && lane < left) {
    int rank = lane;
    // entries of the other beams' lists before this candidate (better, or equal in a lower beam),
    // four lists at a time: the steps of their searches overlap
    for (int j0 = 0; j0 < beams && rank < M; j0 += 4) {
      int lo[4] = {0, 0, 0, 0};
#pragma unroll
      for (int step = 32; step >= 1; step >>= 1)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int j = min(j0 + q, beams - 1), to = lo[q] + step;
          const uint64_t x = s_key[j][min(to, BM_MAX) - 1];
          if (to <= s_left[j] && (x > key || (x == key && j < i))) lo[q] = to;
        }
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (j0 + q < beams && j0 + q != i) rank += lo[q];
    }
    if (rank < M) {
      o_score[rank] = value;
      o_token[rank] = token;
      o_parent[rank] = i;
    }
  }
  __syncthreads();
  if (tid < M) {
    out_score[b * M + tid] = o_score[tid];
    out_token[b * M + tid] = o_token[tid];
    out_parent[b * M + tid] = o_parent[tid];
  }
}

// The records of short rows, where the logit pass, made for long ones, has no floor that keeps a
// row's elements from being folded into its list one by one.  One CTA per row: the row in shared
// memory, its maximum, the sum of its exponentials, and for each warp the K best of its quarter,
// 32 elements sorted and merged at a time where one of them passes the list's last; then the
// four lists are merged.  Bound by latency.
constexpr int BS_MAX_V = 1024, BS_WARPS = 4;

template <typename T>
__global__ void __launch_bounds__(32 * BS_WARPS)
    beam_short_kernel(const T* __restrict__ logits, int V, int64_t row_stride, int K,
                      const float* __restrict__ scores, const uint8_t* __restrict__ finished, char* __restrict__ records) {
  __shared__ float s_x[BS_MAX_V], s_v[BS_WARPS][32], s_top[BS_WARPS], s_sum[BS_WARPS];
  __shared__ int s_id[BS_WARPS][32];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  if (!(scores[row] > -INFINITY) || (finished && finished[row])) return;  // (its record is not read)
  const T* x = logits + row * row_stride;
  float top = -INFINITY;
  for (int i = tid; i < V; i += 32 * BS_WARPS) {
    const float z = static_cast<float>(x[i]);
    s_x[i] = z;
    top = fmaxf(top, z);
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, o));
  if (lane == 0) s_top[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < BS_WARPS; ++w) top = fmaxf(top, s_top[w]);
  // (a row without a finite logit has the sum 0, one with a NaN or +inf a NaN: no candidates)
  const float m2 = top == -INFINITY ? 0.f : top * 1.4426950408889634f;
  float sum = 0.f, v = -INFINITY;
  int id = INT_MAX;
#pragma unroll 1
  for (int i0 = warp * 32; i0 < V; i0 += 32 * BS_WARPS) {
    const int i = i0 + lane;
    float bv = i < V ? s_x[i] : -INFINITY;
    sum += ex2(fmaf(bv, 1.4426950408889634f, -m2));
    // (an equal value further on has a larger id, and is not better)
    if (!__any_sync(FULL_MASK, bv > __shfl_sync(FULL_MASK, v, K - 1))) continue;
    int bi = bv == -INFINITY ? INT_MAX : i;
    warp_sort_pairs(bv, bi, lane);
    bitonic_merge(v, id, bv, bi, lane);
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(FULL_MASK, sum, o);
  s_v[warp][lane] = v;
  s_id[warp][lane] = id;
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  if (warp != 0) return;
#pragma unroll 1
  for (int w = 1; w < BS_WARPS; ++w) {
    bitonic_merge(v, id, s_v[w][lane], s_id[w][lane], lane);
    sum += s_sum[w];
  }
  float* rec = reinterpret_cast<float*>(records + row * (2 * K + 2) * sizeof(float));
  if (lane == 0) {
    rec[0] = m2;
    rec[1] = sum;
  }
  if (lane < K) {
    rec[2 + lane] = v;
    reinterpret_cast<int32_t*>(rec)[2 + K + lane] = id;
  }
}

// ---------------------------------------------------------------------------- reordering
// dst[b, j] = src[b, parent[b, j]] for every state.  A thread owns one column (a vector of
// up to 16 bytes at the same place of every beam's row) of a batch entry: it reads the
// column of every wanted parent, then writes every beam's, so a gather in place needs no
// second buffer and no order between threads; a beam that keeps its own row in place is
// neither read nor written.  Bound by HBM; several parents' reads of one line meet in L1 (caches
// of 8 x 8 beams, 868 MB to move: 129 us, 6.7 TB/s, the copy rate).
constexpr int BR_MAX_STATES = 16;
constexpr int BR_THREADS = 256;

struct ReorderState {
  const char* src;
  char* dst;
  int64_t s_batch, s_beam, s_seg, d_batch, d_beam, d_seg;  // bytes
  int64_t segs;
  uint32_t seg_cols;   // vectors of a segment
  int vec;             // bytes of a vector: 16, 8, 4, 2 or 1
  int64_t cols;        // vectors of a row: segs * seg_cols
  int64_t first_tile;  // of the whole grid; tiles of BR_THREADS columns, batch-major
  int64_t tiles;       // of one batch entry
};
struct ReorderParams {
  ReorderState st[BR_MAX_STATES];
  int n;
  const int32_t* parent;
  int64_t batch;
  int beams;
};

template <typename T, int W>
__device__ __forceinline__ void reorder_column(const ReorderState& s, const int* par, int beams,
                                               int64_t b, int64_t seg, int64_t off) {
  const char* src = s.src + b * s.s_batch + seg * s.s_seg + off;
  char* dst = s.dst + b * s.d_batch + seg * s.d_seg + off;
  const bool inplace = s.src == s.dst;
  T v[W];
#pragma unroll
  for (int j = 0; j < W; ++j) {
    if (j < beams) {
      const int p = par[j];
      if (p >= 0 && !(inplace && p == j)) v[j] = *reinterpret_cast<const T*>(src + p * s.s_beam);
    }
  }
#pragma unroll
  for (int j = 0; j < W; ++j) {
    if (j < beams) {
      const int p = par[j];
      if (p >= 0 && !(inplace && p == j)) *reinterpret_cast<T*>(dst + j * s.d_beam) = v[j];
    }
  }
}

template <int W>
__global__ void __launch_bounds__(BR_THREADS) beam_reorder_kernel(const __grid_constant__ ReorderParams p) {
  __shared__ int s_par[W];
  const int64_t tile = blockIdx.x;
  int k = 0;
  while (k + 1 < p.n && tile >= p.st[k + 1].first_tile) ++k;
  const ReorderState& s = p.st[k];
  const int64_t t = tile - s.first_tile;
  const int64_t b = t / s.tiles;
  const int64_t col = (t % s.tiles) * BR_THREADS + threadIdx.x;
  if (threadIdx.x < p.beams) {
    int q = p.parent[b * p.beams + threadIdx.x];
    if (q < 0 || q >= p.beams) {  // no such beam: its row stays as it is
      atomicOr(&g_err_beam, ERR_BEAM_PARENT);
      q = -1;
    }
    s_par[threadIdx.x] = q;
  }
  __syncthreads();
  if (col >= s.cols) return;
  const int64_t seg = col / s.seg_cols;
  const int64_t off = (col - seg * s.seg_cols) * s.vec;
  switch (s.vec) {
    case 16: reorder_column<uint4, W>(s, s_par, p.beams, b, seg, off); break;
    case 8: reorder_column<uint2, W>(s, s_par, p.beams, b, seg, off); break;
    case 4: reorder_column<uint32_t, W>(s, s_par, p.beams, b, seg, off); break;
    case 2: reorder_column<uint16_t, W>(s, s_par, p.beams, b, seg, off); break;
    default: reorder_column<uint8_t, W>(s, s_par, p.beams, b, seg, off); break;
  }
}

cudaError_t beam_read_device_error(uint32_t* code) {
  uint32_t v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_err_beam, sizeof(v));
  if (e != cudaSuccess) return e;
  if (v) e = cudaMemcpyToSymbol(g_err_beam, &zero, sizeof(zero));
  *code |= v;
  return e;
}

namespace {

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

struct SelectPlan {
  int K, P;      // entries of a record, segments of a row
  size_t total;  // bytes of the records
};

bool select_sizes_ok(int64_t batch, int32_t beams, int64_t V, int32_t M, lilicorr_dtype dt) {
  if (dt != LILICORR_F32 && dt != LILICORR_BF16) return false;
  if (batch < 1 || beams < 1 || beams > BM_MAX || M < 1 || M > BM_MAX) return false;
  const int es = dt == LILICORR_BF16 ? 2 : 4;
  if (V < 1 || V > (int64_t(1) << 31) - 2 || V * es > (int64_t(1) << 31) - 64) return false;
  return batch <= ((int64_t(1) << 31) - 2) / beams;
}

SelectPlan select_plan(int64_t batch, int32_t beams, int64_t V, int32_t M, int es) {
  const int64_t rows = batch * beams;
  SelectPlan pl{};
  pl.K = static_cast<int>(std::min<int64_t>(M, V));
  const int64_t want = rows >= K1_SPLIT_BELOW_ROWS ? 1 : K1_SPLIT_BELOW_ROWS / rows;
  pl.P = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(want, V * es / 4096)));
  pl.total = align256(size_t(rows) * pl.P * k1_shard_record_bytes(pl.K));
  return pl;
}

// Whether a row is one that the logit pass has no floor for: the K-th largest of its thread groups'
// first chunks of 16 bytes, 32 groups of 16 threads or, above K = 16, 64 of 8.  Measured, the whole
// call, 980 rows in bf16: K = 29, V 95, 500 and 1,024: 10, 17 and 25 us here, 59, 62 and 67 with the
// logit pass; K = 4, V 95 and 500: 10 and 17 here, 51 and 24 with it; 40 rows, K = 16, V 1,024: 20
// and 18; 4 rows, K = 8, V 768 and 1,024 (a floor): 14.8 and 17.5 here, 15.3 and 7.4 with it.  From
// V 1,024 on few rows lose (40 rows, K = 29, V 1,800: 31 and 22).
bool short_row(int64_t V, int es, int K) { return V <= BS_MAX_V && V * es < 16 * K * (K <= 16 ? 16 : 8); }

// Whether the byte ranges that (batch, beam, segment) strides reach from one base are
// apart from one another: nested by stride, each stride at least what lies under it.
bool strides_apart(int64_t batch, int64_t sb, int64_t beams, int64_t sw, int64_t segs, int64_t ss,
                   int64_t bytes) {
  std::pair<int64_t, int64_t> d[3] = {{sb, batch}, {sw, beams}, {ss, segs}};
  std::sort(d, d + 3);
  int64_t extent = bytes;
  for (const auto& x : d) {
    if (x.second <= 1) continue;
    if (x.first < extent) return false;
    extent += (x.second - 1) * x.first;
  }
  return true;
}

template <typename T>
cudaError_t short_launch(const void* logits, int64_t rows, int64_t V, int64_t row_stride, int K, const float* scores,
                         const uint8_t* finished, void* records, cudaStream_t stream) {
  beam_short_kernel<T><<<static_cast<unsigned>(rows), 32 * BS_WARPS, 0, stream>>>(
      static_cast<const T*>(logits), static_cast<int>(V), row_stride, K, scores, finished, static_cast<char*>(records));
  note_launch();
  return cudaGetLastError();
}

cudaError_t reorder_launch(const ReorderParams& prm, int64_t tiles, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(tiles));
  if (prm.beams <= 4) beam_reorder_kernel<4><<<grid, BR_THREADS, 0, stream>>>(prm);
  else if (prm.beams <= 8) beam_reorder_kernel<8><<<grid, BR_THREADS, 0, stream>>>(prm);
  else if (prm.beams <= 16) beam_reorder_kernel<16><<<grid, BR_THREADS, 0, stream>>>(prm);
  else beam_reorder_kernel<32><<<grid, BR_THREADS, 0, stream>>>(prm);
  note_launch();
  return cudaGetLastError();
}

lilicorr_status fail(lilicorr_status st, const char* msg) {
  set_last_error(msg);
  return st;
}

}  // namespace
}  // namespace lilicorr

using namespace lilicorr;

extern "C" {

size_t lilicorr_beam_select_workspace_bytes(int64_t batch, int32_t beams, int64_t V, int32_t M,
                                            lilicorr_dtype ldtype) {
  if (!select_sizes_ok(batch, beams, V, M, ldtype)) return 0;
  return select_plan(batch, beams, V, M, ldtype == LILICORR_BF16 ? 2 : 4).total;
}

lilicorr_status lilicorr_beam_select(const void* logits, lilicorr_dtype ldtype, int64_t batch,
                                     int32_t beams, int64_t V, int64_t row_stride, int32_t M,
                                     const float* scores, const uint8_t* finished, int32_t pad_id,
                                     float* out_score, int32_t* out_token, int32_t* out_parent,
                                     void* workspace, size_t workspace_bytes, void* stream_) {
  if (!logits || !scores || !out_score || !out_token || !out_parent)
    return fail(LILICORR_ERR_INVALID_ARG, "lilicorr_beam_select: null pointer");
  if (!select_sizes_ok(batch, beams, V, M, ldtype) || row_stride < V ||
      row_stride > (int64_t(1) << 40))
    return fail(LILICORR_ERR_INVALID_ARG, "lilicorr_beam_select: a size is out of range");
  const int es = ldtype == LILICORR_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(logits) % es)
    return fail(LILICORR_ERR_INVALID_ARG, "lilicorr_beam_select: misaligned logits");
  const SelectPlan pl = select_plan(batch, beams, V, M, es);
  if (!workspace || workspace_bytes < pl.total || reinterpret_cast<uintptr_t>(workspace) % 256)
    return fail(LILICORR_ERR_WORKSPACE, "lilicorr_beam_select: workspace missing, too small or misaligned");
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  const int64_t rows = batch * beams;
  cudaError_t e =
      !short_row(V, es, pl.K) ? k1_launch_beams(logits, es, rows, V, row_stride, pl.K, pl.P, workspace, scores, finished, stream)
      : es == 2 ? short_launch<__nv_bfloat16>(logits, rows, V, row_stride, pl.K, scores, finished, workspace, stream)
                : short_launch<float>(logits, rows, V, row_stride, pl.K, scores, finished, workspace, stream);
  if (e == cudaSuccess) {
    PdlScope pdl(true);
    e = launch_k(beam_merge_kernel, dim3(static_cast<unsigned>(batch)), dim3(32 * beams * std::max(1, std::min(BM_WARPS / beams, (pl.P + 3) / 4))), 0,
                 stream, static_cast<const char*>(workspace), scores, finished, logits, V, row_stride, es, static_cast<int>(beams),
                 pl.P, pl.K, static_cast<int>(M), static_cast<int>(pad_id), out_score, out_token,
                 out_parent);
    if (e == cudaSuccess) note_launch();
  }
  if (e != cudaSuccess) return fail(LILICORR_ERR_CUDA, cudaGetErrorString(e));
  return LILICORR_OK;
}

lilicorr_status lilicorr_beam_reorder(const lilicorr_beam_state* states, int32_t n_states,
                                      const int32_t* parent, int64_t batch, int32_t beams,
                                      void* stream) {
  if (!states || !parent || n_states < 1)
    return fail(LILICORR_ERR_INVALID_ARG, "lilicorr_beam_reorder: null pointer or no states");
  if (batch < 1 || beams < 1 || beams > BM_MAX)
    return fail(LILICORR_ERR_INVALID_ARG, "lilicorr_beam_reorder: 1 <= beams <= 32 and batch >= 1");
  constexpr int64_t LIM = int64_t(1) << 46;
  auto bad = [&](int64_t n) { return n < 0 || n > LIM; };
  // (a product of the two keeps far inside 64 bits)
  auto far = [&](int64_t stride, int64_t count) { return stride > (int64_t(1) << 60) / count; };
  for (int i = 0; i < n_states; ++i) {
    const lilicorr_beam_state& s = states[i];
    if (!s.src || !s.dst || s.segments < 1 || s.seg_bytes < 1 || s.segments > LIM ||
        s.seg_bytes > (int64_t(1) << 32) - 16 || bad(s.src_batch_stride) ||
        bad(s.src_beam_stride) || bad(s.src_seg_stride) || bad(s.dst_batch_stride) ||
        bad(s.dst_beam_stride) || bad(s.dst_seg_stride) || far(s.src_batch_stride, batch) ||
        far(s.dst_batch_stride, batch) || far(s.src_seg_stride, s.segments) ||
        far(s.dst_seg_stride, s.segments) || far(s.seg_bytes, s.segments))
      return fail(LILICORR_ERR_INVALID_ARG, "lilicorr_beam_reorder: a state's pointer, size or stride is out of range");
    if (!strides_apart(batch, s.dst_batch_stride, beams, s.dst_beam_stride, s.segments,
                       s.dst_seg_stride, s.seg_bytes))
      return fail(LILICORR_ERR_INVALID_ARG, "lilicorr_beam_reorder: a state's destination rows overlap");
    if (s.src == s.dst) {
      if (s.src_batch_stride != s.dst_batch_stride || s.src_beam_stride != s.dst_beam_stride ||
          s.src_seg_stride != s.dst_seg_stride)
        return fail(LILICORR_ERR_INVALID_ARG, "lilicorr_beam_reorder: in place, the strides of source and destination are the same");
    } else {
      auto end = [&](const void* p, int64_t sb, int64_t sw, int64_t ss) {
        return reinterpret_cast<uintptr_t>(p) + uintptr_t((batch - 1) * sb + (beams - 1) * sw +
                                                          (s.segments - 1) * ss + s.seg_bytes);
      };
      const uintptr_t a0 = reinterpret_cast<uintptr_t>(s.src), b0 = reinterpret_cast<uintptr_t>(s.dst);
      const uintptr_t a1 = end(s.src, s.src_batch_stride, s.src_beam_stride, s.src_seg_stride);
      const uintptr_t b1 = end(s.dst, s.dst_batch_stride, s.dst_beam_stride, s.dst_seg_stride);
      if (a0 < b1 && b0 < a1)
        return fail(LILICORR_ERR_INVALID_ARG, "lilicorr_beam_reorder: source and destination overlap without being the same");
    }
    // (states run side by side: one that is written must be no other's)
    for (int j = 0; j < n_states; ++j)
      if (j != i && (s.dst == states[j].dst || s.dst == states[j].src))
        return fail(LILICORR_ERR_INVALID_ARG, "lilicorr_beam_reorder: a destination is another state's source or destination");
  }
  ReorderParams prm{};
  int64_t tiles = 0;
  auto flush = [&]() -> cudaError_t {
    if (!prm.n) return cudaSuccess;
    prm.parent = parent;
    prm.batch = batch;
    prm.beams = beams;
    const cudaError_t e = reorder_launch(prm, tiles, static_cast<cudaStream_t>(stream));
    prm = ReorderParams{};
    tiles = 0;
    return e;
  };
  for (int i = 0; i < n_states; ++i) {
    const lilicorr_beam_state& s = states[i];
    // the widest vector that every address and length is a multiple of
    const uint64_t all = reinterpret_cast<uintptr_t>(s.src) | reinterpret_cast<uintptr_t>(s.dst) |
                         uint64_t(s.src_batch_stride) | uint64_t(s.src_beam_stride) |
                         uint64_t(s.src_seg_stride) | uint64_t(s.dst_batch_stride) |
                         uint64_t(s.dst_beam_stride) | uint64_t(s.dst_seg_stride) |
                         uint64_t(s.seg_bytes);
    const int vec = all % 16 == 0 ? 16 : all % 8 == 0 ? 8 : all % 4 == 0 ? 4 : all % 2 == 0 ? 2 : 1;
    ReorderState r{};
    r.src = static_cast<const char*>(s.src);
    r.dst = static_cast<char*>(s.dst);
    r.s_batch = s.src_batch_stride; r.s_beam = s.src_beam_stride; r.s_seg = s.src_seg_stride;
    r.d_batch = s.dst_batch_stride; r.d_beam = s.dst_beam_stride; r.d_seg = s.dst_seg_stride;
    r.segs = s.segments;
    r.vec = vec;
    r.seg_cols = static_cast<uint32_t>(s.seg_bytes / vec);
    r.cols = r.segs * int64_t(r.seg_cols);
    r.tiles = (r.cols + BR_THREADS - 1) / BR_THREADS;
    constexpr int64_t GRID = (int64_t(1) << 31) - 1;
    if (r.tiles > GRID / batch)
      return fail(LILICORR_ERR_INVALID_ARG, "lilicorr_beam_reorder: a state is too large for one call");
    if (prm.n == BR_MAX_STATES || tiles > GRID - batch * r.tiles) {
      const cudaError_t e = flush();
      if (e != cudaSuccess) return fail(LILICORR_ERR_CUDA, cudaGetErrorString(e));
    }
    r.first_tile = tiles;
    prm.st[prm.n++] = r;
    tiles += batch * r.tiles;
  }
  const cudaError_t e = flush();
  if (e != cudaSuccess) return fail(LILICORR_ERR_CUDA, cudaGetErrorString(e));
  return LILICORR_OK;
}

}  // extern "C"
