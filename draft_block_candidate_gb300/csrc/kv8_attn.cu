// Attention of each sequence's new tokens over the 8-bit cache.
//
// For new token i of a sequence's n, and query head j of the group that shares a key / value
// head:  o = softmax_t(scale q . k_t) v_t  over the cached tokens t < len - n + i + 1.
//
// The n * group rows of a (sequence, key / value head) are taken in tiles of N (16, 32, 64 or
// 128) rows; a work unit is one tile against one chunk of 128 cached tokens.  The units of a
// call, laid out by (sequence, head, tile, chunk), are dealt in equal contiguous runs to one
// CTA per SM, so that ragged lengths, and few rows over a long axis, load the SMs alike.  A CTA
// that holds a part of a tile's chunks leaves its maxima, sums and products in the workspace,
// and a second kernel joins the parts in order: no atomics, the same bits every time.
//
// A single token's few rows would leave most of a tensor-core tile empty if the rows were its M,
// so the products are turned round, with the tokens, and the head dimension, as the 128 rows:
//     S'[128 tokens, N] = K Q^T         kind::f8f6f4: K as it lies in the cache, q as the sum of
//                                       two e4m3 values (two products into one accumulator)
//     O'[D, N]         += V^T P'        kind::f16: V widened from e4m3 (exact), P' in f16
// One warp brings chunks (K through a swizzled tensor map, V by plain bulk copies) into a ring
// of stages, one issues the products, four widen V (and split the tile's q), four take the
// softmax: a thread holds one token's N scores.  The two scores' and the two V buffers let
// K Q^T and the widening of chunk c + 1 run under the softmax of chunk c.
//
// The softmax keeps one reference m per row, the maximum of the tile's first chunk, and raises
// it only where a score passes it by more than 2^8: p' is then at most 256, far inside f16, and
// the accumulated O' is scaled in tensor memory only then, by the threads that own its lanes.
// The page's key scale multiplies the scores; the logarithm of its value scale is added to
// them, so that p' = scale_v exp(s - m) is what the second product takes and the sums take
// p' / scale_v.
//
// Roundings below f32: q (bf16) is moved by a power of two of its row to at most 256 and split
// into hi + lo, exactly but for values 2^-9 below the row's largest, which are off by at most
// 2^-17 of it; p' is rounded to f16 (2^-11 of its value, 2^-25 of the row's reference weight
// below 2^-14); out is rounded to bf16.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>

#include "kv8.cuh"

namespace lilicorr {

static __device__ uint32_t g_err_kv8_attn;

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
  float* part;         // [2 * grid][N * (D + 2)]: products, maxima, sums
};

// ------------------------------------------------------------------------ the deal of work

struct SeqUnits {
  int n, len, tiles, chunks;
  int64_t q0, units;
};
template <int N>
__device__ __forceinline__ SeqUnits seq_units(const AttnParams& p, int64_t b) {
  const SeqRange r = seq_range(p.q_start, p.kv_len, b, p.total, p.max_new,
                               int64_t(p.cols) << p.page_log2, &g_err_kv8_attn);
  SeqUnits u;
  u.n = r.n;
  u.len = r.len;
  u.q0 = r.q0;
  u.tiles = (r.n * p.group + N - 1) / N;
  u.chunks = max(1, (r.len + AT_CHUNK - 1) / AT_CHUNK);
  u.units = int64_t(u.tiles) * p.c.heads * u.chunks;
  return u;
}

// The units of all sequences, and where run `run` of `runs` begins, by one warp.
struct Run {
  int64_t per;       // units of a run
  int64_t u, u_end;  // this run's units
  int64_t b, first;  // the sequence of unit u, and that sequence's first unit
};
template <int N>
__device__ __forceinline__ Run find_run(const AttnParams& p, int64_t run, int runs) {
  const int lane = threadIdx.x & 31;
  int64_t t = 0;
#pragma unroll 1
  for (int64_t b = lane; b < p.batch; b += 32) t += seq_units<N>(p, b).units;
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
    const int64_t mine = b0 + lane < p.batch ? seq_units<N>(p, b0 + lane).units : 0;
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

// The pieces of a run: the chunks [c0, c1) of one tile each, of which [c0, cn) are seen by some
// row of it.
struct Piece {
  SeqUnits sq;
  int64_t b, first;  // the sequence, and its first unit
  int h, tile, c0, c1, cn;
  int end;           // tokens that the tile's last row sees
  bool whole;        // all of the tile's chunks
};
template <int N>
__device__ __forceinline__ void piece_at(const AttnParams& p, int64_t u, int64_t u_end, Piece& x) {
  while (u >= x.first + x.sq.units) {
    x.first += x.sq.units;
    x.sq = seq_units<N>(p, ++x.b);
  }
  const uint32_t in = static_cast<uint32_t>(u - x.first);  // a sequence's units fit 32 bits (host)
  const uint32_t item = in / x.sq.chunks;
  x.c0 = static_cast<int>(in - item * x.sq.chunks);
  x.c1 = static_cast<int>(min(int64_t(x.sq.chunks), x.c0 + (u_end - u)));
  x.h = item / x.sq.tiles;
  x.tile = item - x.h * x.sq.tiles;
  const int last = min((x.tile + 1) * N, x.sq.n * p.group) - 1;
  x.end = max(0, min(x.sq.len, x.sq.len - x.sq.n + last / p.group + 1));
  x.cn = max(x.c0, min(x.c1, (x.end + AT_CHUNK - 1) / AT_CHUNK));
  x.whole = x.c0 == 0 && x.c1 == x.sq.chunks;
}

// ------------------------------------------------------------------- tensor-core plumbing

__device__ __forceinline__ void tma_load3(void* dst, const CUtensorMap* tm, int c0, int c1, int c2,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t t, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(t));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld32(uint32_t t, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(t));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
template <int W>
__device__ __forceinline__ void tmem_ld(uint32_t t, float* v) {
  if constexpr (W == 16) tmem_ld16(t, v);
  else tmem_ld32(t, v);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ void tmem_st16(uint32_t t, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]),
      "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
      : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// OR of a flag over the THREADS threads of named barrier `id`.
template <int THREADS>
__device__ __forceinline__ bool bar_or(int id, bool flag) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %2, 0;\n\t"
      "barrier.cta.red.or.pred p, %1, %3, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(flag ? 1u : 0u), "n"(THREADS)
      : "memory");
  return r != 0;
}

// Shared-memory tiles of rows of 32, 64 or 128 bytes (wider ones are several tiles of 128), in
// the hardware's swizzle for that row width: 16-byte piece c of row r lies at piece
// c ^ (bits of r).  Rows in groups of 8.
template <int BYTES>
__device__ __forceinline__ int swz(int r) {
  return BYTES == 128 ? r & 7 : BYTES == 64 ? (r >> 1) & 3 : (r >> 2) & 1;
}
// Its matrix descriptor.  Row groups are 8 * BYTES apart; `next` is the distance to the next
// tile of an operand whose rows are the summed index (0: the same tile again, for rows of the
// product that nothing reads).
template <int BYTES>
__device__ __forceinline__ uint64_t tile_desc(const void* p, uint32_t next) {
  constexpr uint64_t MODE = BYTES == 128 ? 2 : BYTES == 64 ? 4 : 6;
  const uint64_t a = smem_addr(p);
  return ((a >> 4) & 0x3FFFull) | (uint64_t(next >> 4) << 16) | (uint64_t((8 * BYTES) >> 4) << 32) |
         (1ull << 46) | (MODE << 61);
}
// f32 accumulator; a_mn / b_mn: the operand's rows are the summed index.
constexpr uint32_t tc_idesc(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | (uint32_t(N >> 3) << 17) |
         (uint32_t(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {  // 0xff in each byte that is NaN
  return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu);
}

// --------------------------------------------------------------------------- the kernel

template <int D, int N>
struct AttnShape {
  static constexpr int CTAS = N == 16 ? 2 : 1;         // per SM
  static constexpr int KT = AT_CHUNK * D;              // bytes of a chunk's keys, or values
  static constexpr int STAGES = CTAS == 2 ? 2 : D < 128 ? 4 : N == 128 ? 2 : 3;
  static constexpr int VW = 2 * KT;                    // widened values
  static constexpr int VB = CTAS == 2 ? 1 : 2;         // buffers of them
  static constexpr int PB = CTAS == 2 || N == 128 ? 1 : 2;  // buffers of p'
  static constexpr int PT = AT_CHUNK * N * 2;
  static constexpr int QB = N == 32 ? 2 : 1;           // buffers of q hi, lo
  static constexpr int QT = N * D;                     // bytes of one of the two
  static constexpr int OFF_V = STAGES * 2 * KT;
  static constexpr int OFF_P = OFF_V + VB * VW;
  static constexpr int OFF_Q = OFF_P + PB * PT;
  static constexpr int SMEM = 1024 + OFF_Q + QB * 2 * QT;
  static constexpr int TMEM = N == 16 ? 64 : 4 * N;    // two S' and one O' of N columns
  // Softmax warps: a warp can read the 32 lanes (tokens) of tensor memory of its place among
  // four; with 64 rows and more, two warps share the columns (rows) of each 32 tokens.
  static constexpr int GROUPS = N >= 64 ? 2 : 1, SOFT = 4 * GROUPS, COLS = N / GROUPS;
  // then four that widen V, and one each for loads, S' and O'
  static constexpr int LOAD_WARP = SOFT + 4, S_WARP = SOFT + 5, O_WARP = SOFT + 6;
  static constexpr int THREADS = 32 * (SOFT + 7);
};

constexpr int AT_CONV = 4;                  // warps that widen V
constexpr int SC_RING = 8, PIECE_RING = 4;  // deeper than any warp runs ahead of the softmax
constexpr float RAISE = 14.f;               // log2 of how far a score may pass its reference
constexpr float ANEW = 0x1p-100f;

struct PageScale {  // of the tokens of one page
  float k, log2_v, inv_v;
  int ok;  // the page was loaded
};

// The rest of a wait that did not end at once, at most WAIT_LIMIT_CYCLES.  The first one of a CTA
// that gives up makes every later one give up soon.  (Out of line: the roles' loops share the
// SM's instruction cache, and measured half as fast when their code did not fit it.)
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, uint32_t site, volatile int* fail) {
  const long long t0 = clock64();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63) == 0 && (*fail || clock64() - t0 > WAIT_LIMIT_CYCLES)) {
      atomicOr(&g_err_kv8_attn, site);
      *fail = 1;
      return false;
    }
  }
}

template <int D, int N>
__global__ void __launch_bounds__(AttnShape<D, N>::THREADS, AttnShape<D, N>::CTAS)
    kv8_attention_kernel(const __grid_constant__ CUtensorMap tm, const AttnParams p) {
  using S = AttnShape<D, N>;
  constexpr int ST = S::STAGES, VB = S::VB, PB = S::PB, QB = S::QB;
  constexpr int COLS = S::COLS, W = COLS < 32 ? 16 : 32;  // columns of a softmax thread, and of them at a time
  extern __shared__ uint8_t at_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(at_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full[ST], empty[ST], sready[2], sfree[2], vready[VB], pready[PB],
      pvdone[2], qready[QB], qfree[QB], frready[PIECE_RING];
  __shared__ PageScale s_sc[SC_RING][8];
  __shared__ __align__(16) float s_fr[PIECE_RING][N], s_nref[N];
  __shared__ float s_raw[N], s_fac[N], s_red[4][N];
  __shared__ int s_nan[PIECE_RING][2];  // a NaN was taken out of V, for either group
  __shared__ uint32_t s_tmem;
  __shared__ Run s_run;
  __shared__ volatile int s_fail;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < ST; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1 + AT_CONV); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sready[i], 1);
      mbar_init(&sfree[i], S::SOFT);
      mbar_init(&pvdone[i], 1);
    }
    for (int i = 0; i < VB; ++i) mbar_init(&vready[i], AT_CONV);
    for (int i = 0; i < PB; ++i) mbar_init(&pready[i], S::SOFT);
    for (int i = 0; i < QB; ++i) { mbar_init(&qready[i], AT_CONV); mbar_init(&qfree[i], 1); }
    for (int i = 0; i < PIECE_RING; ++i) { mbar_init(&frready[i], AT_CONV); s_nan[i][0] = s_nan[i][1] = 0; }
    fence_mbar_init();
    s_fail = 0;
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&s_tmem)),
                 "r"(S::TMEM)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  pdl_trigger();
  if (warp == 1) {
    const Run r = find_run<N>(p, blockIdx.x, gridDim.x);
    if (lane == 0) s_run = r;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;  // S' of even and odd chunks, O'
  const uint32_t t_o = tmem + 2 * N;
  const Run run = s_run;
  Piece x;
  x.b = run.b;
  x.first = run.first;
  if (run.u < run.u_end) x.sq = seq_units<N>(p, run.b);

  // Every wait is bounded, and the first that gives up makes every later one of the CTA give up
  // at once, so that all warps still run through their loops and meet at their barriers.
  auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t site) -> bool {
    return mbar_try_wait(bar, parity) || wait_slow(bar, parity, site, &s_fail);
  };
  // ... by all lanes of a warp, which go on together.
  auto wait_warp = [&](uint64_t* bar, uint32_t parity, uint32_t site) {
    const bool ok = wait(bar, parity, site);
    __syncwarp();
    return ok;
  };

  if (warp == S::LOAD_WARP) {
    // ================= loads: lane i brings the i-th page (part) of a chunk =================
    const int part = min(p.c.page, AT_CHUNK), parts = AT_CHUNK >> min(p.page_log2, 7);
    const int bytes = part * D;
    int it = 0;
    bool ok_run = true;
    for (int64_t u = run.u; u < run.u_end && ok_run; u += x.c1 - x.c0) {
      piece_at<N>(p, u, run.u_end, x);
      const int32_t* tab = p.table + x.b * p.table_stride;
      auto page_of = [&](int c) {
        const int tok = c * AT_CHUNK + lane * part;
        return lane < parts && tok < x.end ? __ldg(tab + (tok >> p.page_log2)) : -2;
      };
      // page indices are read two chunks ahead, scales one
      auto exists = [&](int i) { return i >= 0 && i < p.c.n_pages; };
      float ks1 = 0.f, vs1 = 1.f;
      auto read_scales = [&](int i) {
        if (!exists(i)) return;
        const int64_t ph = int64_t(i) * p.c.heads + x.h;
        ks1 = __ldg(p.c.ks + ph);
        vs1 = __ldg(p.c.vs + ph);
      };
      int id1 = x.c0 < x.cn ? page_of(x.c0) : -2, id2 = x.c0 + 1 < x.cn ? page_of(x.c0 + 1) : -2;
      read_scales(id1);
      for (int c = x.c0; c < x.cn; ++c, ++it) {
        const int st = it % ST, slot = it % SC_RING;
        const int id = id1;
        const float ks = ks1, vs = vs1;
        id1 = id2;
        read_scales(id1);
        id2 = c + 2 < x.cn ? page_of(c + 2) : -2;
        const bool ok = exists(id);
        if (id != -2 && !ok) atomicOr(&g_err_kv8_attn, ERR_KV8_PAGE);
        const int64_t ph = int64_t(ok ? id : 0) * p.c.heads + x.h;
        const unsigned have = __ballot_sync(FULL_MASK, ok);
        if (it >= ST && !__all_sync(FULL_MASK, wait_warp(&empty[st], ((it / ST) - 1) & 1, ERR_KV8_EMPTY_WAIT))) {
          ok_run = false;
          break;
        }
        // (whoever waits for the stage, or for what is made from it, sees its scales)
        if (lane < 8) s_sc[slot][lane] = PageScale{ks, log2f(vs), 1.f / vs, ok ? 1 : 0};
        __syncwarp();
        uint8_t* dst = sm + st * 2 * S::KT + lane * bytes;
        if (lane == 0) mbar_arrive_expect_tx(&full[st], 2u * bytes * __popc(have));
        __syncwarp();
        if (ok) {
          tma_load3(dst, &tm, 0, 0, static_cast<int>(ph), &full[st]);
          bulk_g2s(dst + S::KT, p.c.v + ph * bytes, bytes, &full[st]);
        }
      }
    }
    if (!ok_run || s_fail)  // what is in flight has to land
      for (int i = max(0, it - ST); i < it; ++i)
        mbar_wait_bounded(&full[i % ST], (i / ST) & 1, &g_err_kv8_attn, ERR_KV8_EMPTY_WAIT);
  } else if (warp == S::S_WARP) {
    // ================= S' = K Q^T, hi and lo =================
    // (a thread takes 80 cycles or so to issue a product, so the two kinds have one each)
    if (lane == 0) {
      constexpr uint32_t ID = tc_idesc(128, N, false, false);
      const uint64_t d_k = tile_desc<D>(sm, 16), d_q = tile_desc<D>(sm + S::OFF_Q, 16);
      int it = 0, pi = 0;
      for (int64_t u = run.u; u < run.u_end; u += x.c1 - x.c0) {
        piece_at<N>(p, u, run.u_end, x);
        if (x.c0 >= x.cn) continue;
        bool ok = wait(&qready[pi % QB], (pi / QB) & 1, ERR_KV8_S_WAIT);
        for (int c = x.c0; c < x.cn; ++c, ++it) {
          const int st = it % ST, b = it & 1;
          ok = wait(&full[st], (it / ST) & 1, ERR_KV8_FULL_WAIT) && ok;
          if (it >= 2) ok = wait(&sfree[b], ((it >> 1) - 1) & 1, ERR_KV8_S_WAIT) && ok;
          if (ok) {
            tc_fence_after();
            const uint64_t k = d_k + (st * 2 * S::KT >> 4);
            const uint64_t q = d_q + ((pi % QB) * 2 * S::QT >> 4);
#pragma unroll
            for (int d = 0; d < D / 32; ++d) mma_f8(tmem + b * N, k + 2 * d, q + 2 * d, ID, d > 0);
#pragma unroll
            for (int d = 0; d < D / 32; ++d) mma_f8(tmem + b * N, k + 2 * d, q + (S::QT >> 4) + 2 * d, ID, true);
          }
          tc_commit(&sready[b]);
          tc_commit(&empty[st]);
          if (c + 1 == x.cn) tc_commit(&qfree[pi % QB]);
        }
        ++pi;
      }
    }
    __syncwarp();
  } else if (warp == S::O_WARP) {
    // ================= O' += V^T P' =================
    if (lane == 0) {
      constexpr uint32_t ID = tc_idesc(128, N, true, true);
      constexpr int VBY = D < 64 ? 64 : 128, PBY = N < 64 ? 2 * N : 128;  // bytes of a tile's row
      const uint64_t d_v = tile_desc<VBY>(sm + S::OFF_V, D == 128 ? AT_CHUNK * 128 : 0);
      const uint64_t d_p = tile_desc<PBY>(sm + S::OFF_P, AT_CHUNK * 128);
      int it = 0;
      for (int64_t u = run.u; u < run.u_end; u += x.c1 - x.c0) {
        piece_at<N>(p, u, run.u_end, x);
        for (int c = x.c0; c < x.cn; ++c, ++it) {
          const int vb = it % VB, pb = it % PB;
          bool ok = wait(&vready[vb], (it / VB) & 1, ERR_KV8_PV_WAIT);
          ok = wait(&pready[pb], (it / PB) & 1, ERR_KV8_PV_WAIT) && ok;
          if (ok) {
            tc_fence_after();
            const uint64_t v = d_v + (vb * S::VW >> 4), pp = d_p + (pb * S::PT >> 4);
            // (16 tokens further: the address field, in units of 16 bytes, moves on)
#pragma unroll
            for (int k = 0; k < AT_CHUNK / 16; ++k)
              mma_f16(t_o, v + k * VBY, pp + k * PBY, ID, k > 0 || c != x.c0);
          }
          tc_commit(&pvdone[it & 1]);
        }
      }
    }
    __syncwarp();
  } else if (warp >= S::SOFT) {
    // ================= widening of V, and the split of q =================
    const int cw = warp - S::SOFT, ct = tid - 32 * S::SOFT;
    int it = 0, pi = 0;
    for (int64_t u = run.u; u < run.u_end; u += x.c1 - x.c0) {
      piece_at<N>(p, u, run.u_end, x);
      if (x.c0 >= x.cn) continue;
      {
        constexpr int TPR = 128 / N, E = D / TPR;  // threads of a row, elements of a thread
        if (pi >= QB) wait_warp(&qfree[pi % QB], ((pi / QB) - 1) & 1, ERR_KV8_S_WAIT);
        const int r = ct / TPR, e0 = (ct % TPR) * E;
        const int row = x.tile * N + r;
        const bool has = row < x.sq.n * p.group;
        const int i = has ? row / p.group : 0, j = has ? row - i * p.group : 0;
        const __nv_bfloat16* qr = p.q + (x.sq.q0 + i) * p.q_tok + (x.h * p.group + j) * p.q_head + e0;
        uint32_t top = 0;
        // E elements in pieces of 4 (at least: D = 32 with 8 threads of a row)
#pragma unroll
        for (int e = 0; e < E; e += 4) {
          const uint2 w = has ? __ldg(reinterpret_cast<const uint2*>(qr + e)) : make_uint2(0u, 0u);
          top = max(max(top, w.x & 0x7fffu), (w.x >> 16) & 0x7fffu);
          top = max(max(top, w.y & 0x7fffu), (w.y >> 16) & 0x7fffu);
        }
#pragma unroll
        for (int o = TPR / 2; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(FULL_MASK, top, o));
        // the largest moves to [128, 256)
        const int ex = min(max(static_cast<int>(top >> 7), 1), 254) - 127;
        const int sh = min(7 - ex, 120);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + sh) << 23);
        if (e0 == 0)
          s_fr[pi % PIECE_RING][r] = has ? p.scale2 * __uint_as_float(static_cast<uint32_t>(127 - sh) << 23) : 0.f;
        uint8_t* qh = sm + S::OFF_Q + (pi % QB) * 2 * S::QT + r * D;
#pragma unroll
        for (int e = 0; e < E; e += 4) {
          const uint2 w = has ? __ldg(reinterpret_cast<const uint2*>(qr + e)) : make_uint2(0u, 0u);
          const float y[4] = {__uint_as_float(w.x << 16) * up, __uint_as_float(w.x & 0xffff0000u) * up,
                              __uint_as_float(w.y << 16) * up, __uint_as_float(w.y & 0xffff0000u) * up};
          uint32_t hi = 0, lo = 0;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint16_t h2 = f32x2_to_e4m3x2(y[2 * k], y[2 * k + 1]);
            const uint32_t b2 = e4m3x2_to_f16x2(h2);
            const float2 f2 = __half22float2(*reinterpret_cast<const __half2*>(&b2));
            hi |= uint32_t(h2) << (16 * k);
            // a row with an infinity keeps it as NaN: 448 would be a value like any other
            const float l0 = y[2 * k] - f2.x, l1 = y[2 * k + 1] - f2.y;
            lo |= uint32_t(f32x2_to_e4m3x2(isinf(l0) ? NAN : l0, isinf(l1) ? NAN : l1)) << (16 * k);
          }
          const int col = e0 + e;
          const int at = (((col >> 4) ^ swz<D>(r)) << 4) | (col & 15);
          *reinterpret_cast<uint32_t*>(qh + at) = hi;
          *reinterpret_cast<uint32_t*>(qh + S::QT + at) = lo;
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&qready[pi % QB]);
          mbar_arrive(&frready[pi % PIECE_RING]);
        }
      }
      const int part_log2 = min(p.page_log2, 7);
      for (int c = x.c0; c < x.cn; ++c, ++it) {
        const int st = it % ST, b = it % VB, slot = it % SC_RING;
        wait_warp(&full[st], (it / ST) & 1, ERR_KV8_FULL_WAIT);
        if (it >= VB) wait_warp(&pvdone[(it - VB) & 1], ((it - VB) >> 1) & 1, ERR_KV8_PV_WAIT);
        const uint8_t* src = sm + st * 2 * S::KT + S::KT;
        uint8_t* dst = sm + S::OFF_V + b * S::VW;
        // Chunks with tokens that some row does not see (the causal edge), with rows behind the
        // last token or with pages that were not loaded: 0 * NaN is NaN, so there V takes part
        // without NaN, and rows that do see a NaN get it at the end.
        bool edge = (c + 1) * AT_CHUNK > x.sq.len - x.sq.n;
        edge |= __any_sync(FULL_MASK, lane < (AT_CHUNK >> part_log2) && !s_sc[slot][lane & 7].ok);
        constexpr int UPR = D / 16;                     // 16-byte pieces of a row
        constexpr int LPR = UPR < 4 ? UPR : 4;          // lanes on a row
        constexpr int TOKS = 32 / LPR;                  // rows of one round
        bool nan = false;
        constexpr int RB = D < 64 ? 64 : 128;
        constexpr int STEP = UPR < 4 ? UPR : 4;  // pieces of a lane in flight
#pragma unroll 1
        for (int k0 = 0; k0 < UPR; k0 += STEP) {
          uint4 w[STEP];
          int tok[STEP];
#pragma unroll
          for (int i = 0; i < STEP; ++i) {
            const int k = k0 + i;
            tok[i] = cw * 32 + (k % (32 / TOKS)) * TOKS + lane / LPR;
            w[i] = *reinterpret_cast<const uint4*>(src + tok[i] * D + (lane % LPR + (k / (32 / TOKS)) * LPR) * 16);
          }
          if (edge) {
#pragma unroll
            for (int i = 0; i < STEP; ++i) {
              if (c * AT_CHUNK + tok[i] >= x.end || !s_sc[slot][tok[i] >> part_log2].ok) w[i] = make_uint4(0u, 0u, 0u, 0u);
              const uint32_t n0 = nan_codes(w[i].x), n1 = nan_codes(w[i].y), n2 = nan_codes(w[i].z), n3 = nan_codes(w[i].w);
              nan |= (n0 | n1 | n2 | n3) != 0;
              w[i].x &= ~n0; w[i].y &= ~n1; w[i].z &= ~n2; w[i].w &= ~n3;
            }
          }
#pragma unroll
          for (int i = 0; i < STEP; ++i) {
            const int piece = lane % LPR + ((k0 + i) / (32 / TOKS)) * LPR;
            const uint32_t in[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
            uint32_t o[8];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              o[2 * n] = e4m3x2_to_f16x2(static_cast<uint16_t>(in[n]));
              o[2 * n + 1] = e4m3x2_to_f16x2(static_cast<uint16_t>(in[n] >> 16));
            }
            uint8_t* row = dst + (piece / 4) * (AT_CHUNK * 128) + tok[i] * RB;
            const int q0 = (piece % 4) * 2, f = swz<RB>(tok[i]);
            *reinterpret_cast<uint4*>(row + ((q0 ^ f) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4*>(row + (((q0 + 1) ^ f) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
          }
        }
        if (nan) s_nan[pi % PIECE_RING][0] = s_nan[pi % PIECE_RING][1] = 1;
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&vready[b]);
          mbar_arrive(&empty[st]);
        }
      }
      ++pi;
    }
  } else {
    // ================= softmax: thread = token of the chunk; then thread = column of D =======
    const int quarter = warp & 3, col0 = (warp >> 2) * COLS;  // its tokens, its columns
    const int in = quarter * 32 + lane;
    const uint32_t t_lane = static_cast<uint32_t>(quarter * 32) << 16;
    const int part_log2 = min(p.page_log2, 7);
    const int gt = tid & 127;  // the thread's place in its group, which has its own rows and barriers
    auto sync_group = [&]() { named_bar_sync(1 + (warp >> 2), 128); };
    int it = 0, pi = 0;
    bool first_piece = true;
    for (int64_t u = run.u; u < run.u_end; u += x.c1 - x.c0, first_piece = false) {
      piece_at<N>(p, u, run.u_end, x);
      const SeqUnits& sq = x.sq;
      const int row0 = x.tile * N, rows = min(N, sq.n * p.group - row0);
      const bool any_chunk = x.c0 < x.cn;
      float2 l2[COLS / 2];  // this thread's part of each row's sum
#pragma unroll
      for (int i = 0; i < COLS / 2; ++i) l2[i] = make_float2(0.f, 0.f);
      if (any_chunk) wait_warp(&frready[pi % PIECE_RING], (pi / PIECE_RING) & 1, ERR_KV8_S_WAIT);
      const float* fr = s_fr[pi % PIECE_RING] + col0;
      const float* nref = s_nref + col0;
      bool force = true;
      for (int c = x.c0; c < x.cn; ++c, ++it) {
        const int b = it & 1, slot = it % SC_RING, pb = it % PB;
        wait_warp(&sready[b], (it >> 1) & 1, ERR_KV8_S_WAIT);
        tc_fence_after();
        const PageScale sc = s_sc[slot][in >> part_log2];
        const float2 ks2 = make_float2(sc.k, sc.k), lv2 = make_float2(sc.log2_v, sc.log2_v);
        const float2 iv2 = make_float2(sc.inv_v, sc.inv_v);
        // rows below `hid` do not see this token
        const int tok = c * AT_CHUNK + in, after = tok - (sq.len - sq.n);
        const int hid = !sc.ok || tok >= sq.len ? N : after <= 0 ? 0 : min(N, max(0, after * p.group - row0));
        const bool masks = __any_sync(FULL_MASK, hid > 0);
        const uint32_t t_s = tmem + b * N + col0 + t_lane;
        constexpr int RB = N < 64 ? 2 * N : 128;
        uint8_t* pt = sm + S::OFF_P + pb * S::PT + in * RB;
        const int f = swz<RB>(in);
        bool free_p = it < PB;
        float top;
        // The weights of this thread's columns to shared memory and to the rows' sums; a second
        // time, after a raise, only to the sums of rows that start anew.
        auto weights = [&](bool again) {
          top = -INFINITY;
#pragma unroll
          for (int w0 = 0; w0 < COLS; w0 += W) {
            float s[W];
            tmem_ld<W>(t_s + w0, s);
#pragma unroll
            for (int i = 0; i < W; i += 4) {
              const float4 g = *reinterpret_cast<const float4*>(fr + w0 + i);
              const float4 n = *reinterpret_cast<const float4*>(nref + w0 + i);
              const float2 a = __ffma2_rn(make_float2(s[i], s[i + 1]), __fmul2_rn(make_float2(g.x, g.y), ks2),
                                          __fadd2_rn(make_float2(n.x, n.y), lv2));
              const float2 d = __ffma2_rn(make_float2(s[i + 2], s[i + 3]), __fmul2_rn(make_float2(g.z, g.w), ks2),
                                          __fadd2_rn(make_float2(n.z, n.w), lv2));
              s[i] = a.x; s[i + 1] = a.y; s[i + 2] = d.x; s[i + 3] = d.y;
            }
            if (masks) {
#pragma unroll
              for (int i = 0; i < W; ++i)
                if (col0 + w0 + i < hid) s[i] = -INFINITY;
            }
            if (!free_p) {
              wait_warp(&pvdone[(it - PB) & 1], ((it - PB) >> 1) & 1, ERR_KV8_PV_WAIT);
              free_p = true;
            }
#pragma unroll
            for (int k = 0; k < W / 8; ++k) {
              uint32_t h[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float2 y = make_float2(s[8 * k + 2 * i], s[8 * k + 2 * i + 1]);
                top = max3(top, y.x, y.y);
                const float2 e = make_float2(ex2(y.x), ex2(y.y));
                float2& l = l2[(w0 + 8 * k) / 2 + i];
                if (!again) {
                  l = __ffma2_rn(e, iv2, l);
                } else {
                  const int r = col0 + w0 + 8 * k + 2 * i;
                  if (s_fac[r] < ANEW) l.x = fmaf(e.x, sc.inv_v, l.x);
                  if (s_fac[r + 1] < ANEW) l.y = fmaf(e.y, sc.inv_v, l.y);
                }
                const __half2 hh = __floats2half2_rn(e.x, e.y);
                h[i] = *reinterpret_cast<const uint32_t*>(&hh);
              }
              const int piece = (col0 + w0) / 8 + k;
              *reinterpret_cast<uint4*>(pt + (piece / 8) * (AT_CHUNK * 128) + (((piece % 8) ^ f) << 4)) =
                  make_uint4(h[0], h[1], h[2], h[3]);
            }
          }
        };
        // New references: the rows' maxima over this chunk and before.
        auto raise = [&]() {
#pragma unroll 1
          for (int w0 = 0; w0 < COLS; w0 += 16) {
            float y[16];
            tmem_ld16(t_s + w0, y);
            int mine = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float z = fmaf(y[i], fr[w0 + i] * sc.k, sc.log2_v);
              if (col0 + w0 + i < hid) z = -INFINITY;
              const int k = __reduce_max_sync(FULL_MASK, float_key(z));
              if (lane == i) mine = k;
            }
            if (lane < 16) s_red[quarter][col0 + w0 + lane] = key_float(mine);
          }
          sync_group();
          if (gt < COLS) {
            const int r = col0 + gt;
            const float old = c == x.c0 ? -INFINITY : s_raw[r];
            const float m = fmaxf(max3(s_red[0][r], s_red[1][r], s_red[2][r]), fmaxf(s_red[3][r], old));
            s_fac[r] = m == -INFINITY ? 1.f : ex2(old - m);
            s_raw[r] = m;
            s_nref[r] = m == -INFINITY ? 0.f : -m;
          }
          sync_group();
          if (c == x.c0) return;
#pragma unroll
          for (int i = 0; i < COLS; ++i) {
            // a row whose reference moved that far starts anew: what it had is nothing beside
            // what it gets, and its weights of this chunk may have passed the floats
            float& l = i & 1 ? l2[i / 2].y : l2[i / 2].x;
            const float g = s_fac[col0 + i];
            l = g < ANEW ? 0.f : l * g;
          }
          wait_warp(&pvdone[(it - 1) & 1], ((it - 1) >> 1) & 1, ERR_KV8_PV_WAIT);
          tc_fence_after();
#pragma unroll 1
          for (int w0 = 0; w0 < COLS; w0 += 16) {
            float o[16];
            tmem_ld16(t_o + t_lane + col0 + w0, o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= s_fac[col0 + w0 + i];
            tmem_st16(t_o + t_lane + col0 + w0, o);
          }
        };
        if (force) raise();
        weights(false);
        fence_async_smem();
        // Mostly no score is far above its reference and no page is missing.
        force = false;
        const bool lacks = c + 1 < x.cn && __any_sync(FULL_MASK, lane < (AT_CHUNK >> part_log2) && !s_sc[slot][lane & 7].ok);
        if (bar_or<128>(3 + (warp >> 2), top > RAISE || lacks)) {
          const bool up = bar_or<128>(3 + (warp >> 2), top > RAISE);
          force = bar_or<128>(3 + (warp >> 2), lacks);  // rows' maxima may not be known yet
          if (up) {
            raise();
            weights(true);
            fence_async_smem();
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sfree[b]);
          mbar_arrive(&pready[pb]);
        }
      }

      // ---- the piece's sums, and its outputs or part
#pragma unroll
      for (int w0 = 0; w0 < COLS; w0 += W) {
        float l[W];
#pragma unroll
        for (int i = 0; i < W; i += 2) { l[i] = l2[(w0 + i) / 2].x; l[i + 1] = l2[(w0 + i) / 2].y; }
        // halves of the columns go to the other half of the lanes, until lane i holds column i
#pragma unroll
        for (int o = W / 2; o >= 1; o >>= 1) {
          const bool up = lane & o;
#pragma unroll
          for (int i = 0; i < o; ++i) {
            const float keep = up ? l[i + o] : l[i], give = up ? l[i] : l[i + o];
            l[i] = keep + __shfl_xor_sync(FULL_MASK, give, o);
          }
        }
        if (W == 16) l[0] += __shfl_xor_sync(FULL_MASK, l[0], 16);
        if (lane < W) s_red[quarter][col0 + w0 + lane] = l[0];
      }
      sync_group();
      const int d = in;  // this thread's column of the head dimension
      const bool mine = d < D;
      float* part = p.part + (int64_t(blockIdx.x) * 2 + (first_piece ? 0 : 1)) * N * (D + 2);
      if (gt < COLS) {
        const int r = col0 + gt;
        const float m = any_chunk ? s_raw[r] : -INFINITY;
        const float sum = any_chunk ? (s_red[0][r] + s_red[1][r]) + (s_red[2][r] + s_red[3][r]) : 0.f;
        if (x.whole) {
          s_fac[r] = sum == 0.f ? 0.f : 1.f / sum;  // no token seen: 0
          if (p.lse && r < rows) {
            const int i = (row0 + r) / p.group;
            p.lse[(sq.q0 + i) * p.q_heads + x.h * p.group + (row0 + r - i * p.group)] =
                sum == 0.f ? -INFINITY : (m + log2f(sum)) * LN2_F;
          }
        } else {
          part[N * D + r] = m;
          part[N * D + N + r] = sum;
        }
      }
      int nan_row = N;  // rows from here on see a NaN in this column
      if (any_chunk) {
        wait_warp(&pvdone[(it - 1) & 1], ((it - 1) >> 1) & 1, ERR_KV8_PV_WAIT);
        tc_fence_after();
        if (s_nan[pi % PIECE_RING][warp >> 2] && mine) {
          const int edge = sq.len - sq.n;
          const int from = max(x.c0, max(edge, 0) / AT_CHUNK) * AT_CHUNK, to = min(x.end, x.cn * AT_CHUNK);
          for (int t = from; t < to; ++t) {
            const int id = __ldg(p.table + x.b * p.table_stride + (t >> p.page_log2));
            if (id < 0 || id >= p.c.n_pages) continue;
            const int64_t at = ((int64_t(id) * p.c.heads + x.h) * p.c.page + (t & (p.c.page - 1))) * D + d;
            if ((p.c.v[at] & 0x7f) == 0x7f) {
              nan_row = max(0, (t - edge) * p.group - row0);
              break;  // later tokens are seen by fewer rows
            }
          }
        }
      }
      sync_group();
      if (any_chunk && gt == 0) s_nan[pi % PIECE_RING][warp >> 2] = 0;
      int i = (row0 + col0) / p.group, j = row0 + col0 - i * p.group;  // new token and head of a row
#pragma unroll 1
      for (int r0 = col0; r0 < min(rows, col0 + COLS); r0 += 16) {
        float o[16];
        if (any_chunk) {
          tmem_ld16(t_o + t_lane + r0, o);
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int r = r0 + k;
          if (r < rows && mine) {
            const float y = r >= nan_row ? NAN : o[k];
            if (x.whole)
              p.out[((sq.q0 + i) * p.q_heads + x.h * p.group + j) * D + d] = __float2bfloat16_rn(y * s_fac[r]);
            else
              part[r * D + d] = y;
          }
          if (++j == p.group) { j = 0; ++i; }
        }
      }
      tc_fence_before();
      sync_group();  // s_red and s_fac are read
      if (any_chunk) ++pi;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::TMEM)
                 : "memory");
  }
}

// Joins the parts of the tiles that several CTAs hold.  One CTA per boundary between two runs
// of units and 16 rows; the CTAs of the first boundary inside a tile join that tile, from the run
// that holds its first chunk to the one that holds its last, in that order: a warp for each
// row, the weights of 32 parts at a time worked out side by side, then the parts added up.
constexpr int JOIN_ROWS = 16;

template <int D, int N>
__global__ void __launch_bounds__(32 * JOIN_ROWS) kv8_join_kernel(const AttnParams p, int runs) {
  constexpr int E = D / 32;  // columns of a lane
  const int lane = threadIdx.x & 31, r = blockIdx.y * JOIN_ROWS + (threadIdx.x >> 5);
  // Lengths and row ranges were there before the attention began: they are read, and the
  // tile is found, while it still runs.
  const Run run = find_run<N>(p, int64_t(blockIdx.x) + 1, runs);
  const int64_t edge = run.u;  // first unit of run blockIdx.x + 1
  if (edge >= run.u_end) return;
  const SeqUnits sq = seq_units<N>(p, run.b);
  const uint32_t in = static_cast<uint32_t>(edge - run.first);
  const uint32_t item = in / sq.chunks;
  const int64_t i0 = run.first + int64_t(item) * sq.chunks, i1 = i0 + sq.chunks;  // the tile's units
  if (edge == i0) return;                  // the boundary lies between two tiles
  if (edge - run.per > i0) return;         // an earlier boundary lies inside this tile too
  const int64_t r0 = blockIdx.x, r1 = (i1 - 1) / run.per;  // runs that hold parts
  const int h = item / sq.tiles, tile = item - h * sq.tiles;
  const int row = tile * N + r;
  if (row >= sq.n * p.group) return;
  constexpr int64_t STEP = N * (D + 2);
  // the run that holds the tile's first chunk may hold another tile's part before it
  const float* parts = p.part + r0 * 2 * STEP;
  const int64_t lead = r0 * run.per >= i0 ? 0 : STEP;
  pdl_wait();
  float mx = -INFINITY, sum = 0.f, y[E];
#pragma unroll
  for (int n = 0; n < E; ++n) y[n] = 0.f;
  const int count = static_cast<int>(r1 - r0) + 1;
  for (int k0 = 0; k0 < count; k0 += 32) {
    const int mine = k0 + lane;
    const float* q = parts + mine * 2 * STEP + (mine == 0 ? lead : 0);
    const float m = mine < count ? __ldcg(q + N * D + r) : -INFINITY;
    const float s = mine < count ? __ldcg(q + N * D + N + r) : 0.f;
    float nm = fmaxf(m, mx);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) nm = fmaxf(nm, __shfl_xor_sync(FULL_MASK, nm, o));
    const float base = nm == -INFINITY ? 0.f : nm;
    const float w = ex2(m - base), back = ex2(mx - base);
    float add = s * w;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) add += __shfl_xor_sync(FULL_MASK, add, o);
    sum = fmaf(sum, back, add);
#pragma unroll
    for (int n = 0; n < E; ++n) y[n] *= back;
    mx = nm;
    const int here = min(32, count - k0);
#pragma unroll 8
    for (int k = 0; k < here; ++k) {
      const float wk = __shfl_sync(FULL_MASK, w, k);
      const float* src = parts + (k0 + k) * 2 * STEP + (k0 + k == 0 ? lead : 0) + r * D + lane * E;
      if constexpr (E == 4) {
        const float4 z = __ldcg(reinterpret_cast<const float4*>(src));
        y[0] = fmaf(z.x, wk, y[0]); y[1] = fmaf(z.y, wk, y[1]);
        y[2] = fmaf(z.z, wk, y[2]); y[3] = fmaf(z.w, wk, y[3]);
      } else if constexpr (E == 2) {
        const float2 z = __ldcg(reinterpret_cast<const float2*>(src));
        y[0] = fmaf(z.x, wk, y[0]); y[1] = fmaf(z.y, wk, y[1]);
      } else {
        y[0] = fmaf(__ldcg(src), wk, y[0]);
      }
    }
  }
  const int i = row / p.group;
  const int64_t at = (sq.q0 + i) * p.q_heads + h * p.group + (row - i * p.group);
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
  if (p.lse && lane == 0) p.lse[at] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * LN2_F;
}

// -------------------------------------------------------------------------------- host

namespace {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  // looked up once per process (a thread-safe static initialisation)
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = []() {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
  }();
  return fn;
}

int tile_rows(int max_new, int group) {
  const int64_t rows = int64_t(max_new) * group;
  return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
}

int attn_grid(int n) {
  return device_sm_count() * (n == 16 ? AttnShape<128, 16>::CTAS : 1);
}

template <int D, int N>
cudaError_t launch(const CUtensorMap& tm, const AttnParams& prm, int grid, cudaStream_t stream) {
  constexpr int smem = AttnShape<D, N>::SMEM;
  cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void*>(kv8_attention_kernel<D, N>), smem);
  if (e != cudaSuccess) return e;
  kv8_attention_kernel<D, N><<<grid, AttnShape<D, N>::THREADS, smem, stream>>>(tm, prm);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  PdlScope pdl(true);
  e = launch_k(kv8_join_kernel<D, N>, dim3(grid, N / JOIN_ROWS), dim3(32 * JOIN_ROWS), 0, stream, prm, grid);
  if (e == cudaSuccess) note_launch(2);
  return e;
}

}  // namespace

size_t kv8_attention_workspace(int max_new, int group, int D) {
  const int n = tile_rows(max_new, group);
  return size_t(attn_grid(n)) * 2 * n * (D + 2) * sizeof(float);
}

cudaError_t kv8_attention_launch(const Kv8Attention& a, cudaStream_t stream) {
  auto fn = encode_fn();
  const int64_t tiles = a.c.n_pages * a.c.heads;
  if (!fn || tiles > INT_MAX) return cudaErrorInvalidValue;
  const int D = a.D, page = a.c.page;
  CUtensorMap tm;
  const cuuint64_t dims[3] = {cuuint64_t(D), cuuint64_t(page), cuuint64_t(tiles)};
  const cuuint64_t strides[2] = {cuuint64_t(D), cuuint64_t(D) * page};
  const cuuint32_t box[3] = {cuuint32_t(D), cuuint32_t(page), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  if (fn(&tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, a.c.k, dims, strides, box, estr,
         CU_TENSOR_MAP_INTERLEAVE_NONE,
         D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B,
         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  AttnParams prm{};
  prm.c = a.c;
  prm.q = a.q;
  prm.q_tok = a.q_tok; prm.q_head = a.q_head;
  prm.total = a.total;
  prm.q_heads = a.q_heads; prm.group = a.group;
  prm.q_start = a.q_start; prm.kv_len = a.kv_len; prm.table = a.table;
  prm.batch = a.batch; prm.table_stride = a.table_stride;
  prm.cols = a.cols; prm.max_new = a.max_new;
  prm.page_log2 = page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7;
  prm.scale2 = a.scale * LOG2E_F;
  prm.out = a.out;
  prm.lse = a.lse;
  prm.part = static_cast<float*>(a.workspace);
  const int n = tile_rows(a.max_new, a.group), grid = attn_grid(n);
#define LC_N(DD)                                                            \
  (n == 16 ? launch<DD, 16>(tm, prm, grid, stream)                          \
           : n == 32 ? launch<DD, 32>(tm, prm, grid, stream)                \
                     : n == 64 ? launch<DD, 64>(tm, prm, grid, stream)      \
                               : launch<DD, 128>(tm, prm, grid, stream))
  return D == 128 ? LC_N(128) : D == 64 ? LC_N(64) : LC_N(32);
#undef LC_N
}

cudaError_t kv8_attention_read_device_error(uint32_t* code) {
  uint32_t v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_err_kv8_attn, sizeof(v));
  if (e != cudaSuccess) return e;
  if (v) e = cudaMemcpyToSymbol(g_err_kv8_attn, &zero, sizeof(zero));
  *code |= v;
  return e;
}

}  // namespace lilicorr
