// Attention of each request's rows over states of another length (an encoder's, a target's): every row
// sees all of them, and the rows of a request (its beams, the tokens of a drafted block) share them.
//
//   o_i = sum_t softmax_t(scale q_i . k_t) v_t  over the request's states t < kv_len.
//
// The n * group rows of a (request, key / value head) are taken in tiles of 256; a work unit is one tile
// against one chunk of 128 states.  Units are dealt in equal runs to one CTA per SM, and tiles that
// several CTAs hold are joined in order (kv8_attn.cuh).
//
// A tile has two halves of 128 rows, each with scores S, weights P (over S) and outputs O in tensor
// memory and a group of four softmax warps, a thread a row.  Where the tile has more than 128 rows both
// halves take every chunk, so that a chunk's keys and values are read from shared memory for 256 rows;
// where it has fewer, both halves stand for the same rows and take the chunks in turn, and the outputs
// are joined as they are written.  While one group forms its weights the tensor cores work for the other:
// in tiles of 256 rows the groups' warps take turns from a row's maximum to its last weight, and a chunk's
// weights are handed over by 64 columns, so that the second product begins halfway.
// Warps: two groups of four for the softmax, which also write the outputs (through 2 KB of shared memory
// each, so that four lanes write 64 bytes of a row); one that loads keys and values through tensor maps; one
// for each half that issues its products, S of the next chunk right behind the O that reads the P in its
// place; one that finds the run's pieces and brings their tiles' q.
//
// Roundings below f32: the weights are bf16 (off by 2^-8 of their value at most) for the second product, whose operands
// have one type; the sums take them unrounded.  The tensor cores' f32 sums drop what a product has 2^-25 below the first
// bit of the sum that it is added to: values of one sign over T states that one CTA goes over lose up to T 2^-26 of their
// sum (up to 131,072 states no more than bf16's own rounding of the output; 0.8 %, half of it, was measured over 2^20).
// A row's maximum moves only where a score passes it by more than 2^8, and only then is O scaled.  What lies behind a
// request's last state is never summed: its scores are -inf, its values zeros.
#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>

#include "kv8_attn.cuh"
#include "tc.cuh"

namespace lilicorr {

struct CrossParams {
  const __nv_bfloat16* q;
  int64_t q_tok, q_head;  // elements
  int64_t total, total_kv;
  int q_heads, group, heads, D;
  const int32_t *q_start, *kv_start, *kv_len;
  int64_t batch;
  int max_new;
  float scale2;  // |softmax scale| * log2 e
  uint32_t flip;  // sign bits of the scale, which q takes
  int q_map;      // whether q comes through a tensor map
  __nv_bfloat16* out;  // [total, q_heads, D]
  float* lse;          // [total, q_heads] or null
  float* part;         // [2 * grid][256 * (padded D + 2)]: products, maxima, sums
  int half;            // rows of a tile's half
  uint64_t tile_inv;   // 2^40 / (2 half), rounded up: exact quotients of less than 2^32 by 2^8 and less
  __device__ __forceinline__ int kv_heads() const { return heads; }
};

// Rows of a tile and its halves that are used: all, or whole tokens' where a group does not divide 128 (as one kernel the
// usual case was 1 to 3 % slower).
struct CrossFull : CrossParams {
  __device__ __forceinline__ int half_rows() const { return 128; }
  template <int ROWS>
  __device__ __forceinline__ int tile_rows() const { return ROWS; }
  template <int ROWS>
  __device__ __forceinline__ int tiles(int rows) const { return (rows + ROWS - 1) / ROWS; }
};
struct CrossPart : CrossParams {
  __device__ __forceinline__ int half_rows() const { return half; }
  template <int ROWS>
  __device__ __forceinline__ int tile_rows() const { return 2 * half; }
  template <int ROWS>
  __device__ __forceinline__ int tiles(int rows) const { return static_cast<int>((uint64_t(rows + 2 * half - 1) * tile_inv) >> 40); }
};

__device__ __forceinline__ SeqRange attn_range(const CrossParams& p, int64_t b) {
  SeqRange r = seq_range(p.q_start, p.kv_len, b, p.total, p.max_new, p.total_kv, &g_err_kv8_attn);
  const int at = __ldg(p.kv_start + b);
  if (r.n > 0 && (at < 0 || int64_t(at) + r.len > p.total_kv)) {
    atomicOr(&g_err_kv8_attn, ERR_KV8_LENGTH);
    r.n = 0;
    r.len = 0;
  }
  return r;
}

template <int E>
__device__ __forceinline__ void store_row(const CrossParams& p, int64_t at, int, int lane, const float (&y)[E], float sum, float m) {
  const float inv = sum == 0.f ? 0.f : 1.f / sum;  // no state seen: 0
  if (lane * E < p.D) {                            // (a multiple of 8)
    __nv_bfloat162* o = reinterpret_cast<__nv_bfloat162*>(p.out + at * p.D + lane * E);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) o[i] = __floats2bfloat162_rn(y[2 * i] * inv, y[2 * i + 1] * inv);
  }
  if (p.lse && lane == 0) p.lse[at] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * LN2_F;
}

constexpr int CR_ROWS = 256, CR_HALF = 128;

template <int DP>  // head dimension, filled up with zeros
struct CrossShape {
  static constexpr int SUB = AT_CHUNK * 128;        // bytes of 128 rows of 64 values
  static constexpr int T = SUB * (DP / 64);         // bytes of 128 rows
  static constexpr int KS = DP == 64 ? 4 : 2;       // chunks of keys, and of values, in flight or in use
  static constexpr int VS = DP == 64 ? 4 : 2;
  static constexpr int QS = 2;                      // halves of q
  static constexpr int OFF_V = KS * T;
  static constexpr int OFF_Q = OFF_V + VS * T;
  static constexpr int OFF_ST = OFF_Q + QS * T;     // 32 outputs of 32 rows for each softmax warp
  static constexpr int SMEM = 1024 + OFF_ST + 8 * 2048;
};
// Warps: 0 to 3 and 4 to 7 the halves' softmax; then keys and values, each half's products, pieces and q.
constexpr int CR_LOAD = 8, CR_MMA = 9, CR_Q = 11, CR_WARPS = 12, CR_READERS = CR_WARPS - 1, CR_PIECES = 6, CR_AHEAD = 2;
constexpr int CR_S = 0, CR_O = 256;       // columns of S (and P) and O of the first half; the second's are 128 and DP further
constexpr float CR_RAISE = 8.f;           // log2 of how far a score may pass its reference

// A piece of the CTA's run: the chunks [c0, cn) of a tile.
struct CrossPiece {
  int64_t q0;         // the request's first row of q
  int kv0, len;       // its states
  int h, row0, rows;  // key / value head; the tile's first row and its rows
  int c0, cn;
  int whole;          // 1: all of the tile's chunks; 0: a part; -1: there is no further piece
  int slot;           // of the workspace, for a part
};

// -inf to the scores from column lim on.
__device__ __noinline__ void mask_columns(uint32_t t, int lim) {
#pragma unroll 1
  for (int w0 = lim & ~15; w0 < AT_CHUNK; w0 += 16) {
    float s[16];
    tmem_ld16(t + w0, s);
#pragma unroll
    for (int n = 0; n < 16; ++n)
      if (w0 + n >= lim) s[n] = -INFINITY;
    tmem_st16(t + w0, s);
  }
}
// A row's outputs by f (inlined, 8 at a time: the scores stay in registers meanwhile).
template <int DP>
__device__ __forceinline__ void scale_outputs(uint32_t t, float f) {
#pragma unroll 1
  for (int w0 = 0; w0 < DP; w0 += 8) {
    float o[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
                 : "=f"(o[0]), "=f"(o[1]), "=f"(o[2]), "=f"(o[3]), "=f"(o[4]), "=f"(o[5]), "=f"(o[6]), "=f"(o[7])
                 : "r"(t + w0)
                 : "memory");
    uint32_t h[8];
#pragma unroll
    for (int n = 0; n < 8; ++n) h[n] = __float_as_uint(o[n] * f);
    tmem_st8(t + w0, h);
  }
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// 16 bytes to shared memory behind the thread's back (zeros where !there); cp_wait: all of the thread's have landed.
__device__ __forceinline__ void cp16(void* to, const void* from, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(to)), "l"(from), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

template <int DP, class P>
__global__ void __launch_bounds__(32 * CR_WARPS, 1)
    cross_attention_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                           const __grid_constant__ P p) {
  using S = CrossShape<DP>;
  constexpr int KS = S::KS, VS = S::VS, T = S::T, SUB = S::SUB;
  extern __shared__ uint8_t cr_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(cr_raw) + 1023) & ~uintptr_t(1023));
  // sready, pready: of each half, a phase for each of its chunks; pvdone, left: for each piece that it has
  // chunks of; met: for each piece that the second half hands over, by turns.
  __shared__ __align__(8) uint64_t kfull[KS], kempty[KS], vfull[VS], vempty[VS], sready[2], pready[2][2], pvdone[2], qready[2], qfree[2],
      left[2], pc_full[CR_PIECES], pc_empty[CR_PIECES], met[2][4], turn[2][4];
  __shared__ CrossPiece s_piece[CR_PIECES];
  __shared__ float2 s_ml[2][CR_HALF];  // a row's maximum and sum, handed over
  __shared__ uint32_t s_tmem;
  __shared__ volatile uint32_t s_fail;

  const int tid = threadIdx.x, warp = __shfl_sync(FULL_MASK, tid >> 5, 0), lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < KS; ++i) { mbar_init(&kfull[i], 1); mbar_init(&kempty[i], 2); }
    for (int i = 0; i < VS; ++i) { mbar_init(&vfull[i], 1); mbar_init(&vempty[i], 2); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sready[i], 1); mbar_init(&pready[0][i], 4); mbar_init(&pready[1][i], 4); mbar_init(&pvdone[i], 1);
      mbar_init(&qready[i], 1); mbar_init(&qfree[i], 2); mbar_init(&left[i], 4);
      for (int j = 0; j < 4; ++j) { mbar_init(&met[i][j], 1); mbar_init(&turn[i][j], 1); }
    }
    for (int i = 0; i < CR_PIECES; ++i) { mbar_init(&pc_full[i], 1); mbar_init(&pc_empty[i], CR_READERS); }
    fence_mbar_init();
    s_fail = 0;
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s_tmem)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(FULL_MASK, s_tmem, 0);
  pdl_wait();
  pdl_trigger();

  auto wait_warp = [&](uint64_t* bar, uint32_t parity, uint32_t site, uint32_t times = 1) {
    return mbar_wait_warp(bar, parity, site, s_fail, times);
  };
  // The next piece with chunks (or, `all`, any), read by a warp.
  auto next_piece = [&](int& pi, CrossPiece& x, bool all) -> bool {
#pragma unroll 1
    for (;;) {
      const int e = pi % CR_PIECES;
      if (!wait_warp(&pc_full[e], (pi / CR_PIECES) & 1, ERR_KV8_FULL_WAIT)) return false;
      x = s_piece[e];
      if (x.whole < 0) return false;
      __syncwarp();
      if (lane == 0) mbar_arrive(&pc_empty[e]);
      ++pi;
      if (all || x.c0 < x.cn) return true;
    }
  };

  if (warp == CR_LOAD) {
    // ====== keys and values ======
    int it = 0, kit = 0, vit = 0, pi = 0;  // (kit, vit: chunks whose keys, values are on their way)
    CrossPiece x;
    bool ok = true;
    while (ok && next_piece(pi, x, false)) {
#pragma unroll 1
      for (int c = x.c0; c < x.cn; ++c, ++it) {
        auto load = [&](const CUtensorMap* tm, uint8_t* to, uint64_t* full) {
          if (lane == 0) {
            mbar_arrive_expect_tx(full, T);
#pragma unroll
            for (int i = 0; i < DP / 64; ++i) tma_load3(to + i * SUB, tm, 64 * i, x.h, x.kv0 + c * AT_CHUNK, full);
          }
          __syncwarp();
        };
        const int sk = it % KS, sv = it % VS;
        ok = it < KS || wait_warp(&kempty[sk], ((it / KS) - 1) & 1, ERR_KV8_EMPTY_WAIT);
        if (!ok) break;
        load(&tk, sm + sk * T, &kfull[sk]);
        ++kit;
        ok = it < VS || wait_warp(&vempty[sv], ((it / VS) - 1) & 1, ERR_KV8_EMPTY_WAIT);
        if (!ok) break;
        load(&tv, sm + S::OFF_V + sv * T, &vfull[sv]);
        ++vit;
      }
    }
    // what is in flight has to land (it has, unless a wait gave up)
    for (int i = max(0, kit - KS); i < kit; ++i) mbar_wait_bounded(&kfull[i % KS], (i / KS) & 1, &g_err_kv8_attn, ERR_KV8_EMPTY_WAIT);
    for (int i = max(0, vit - VS); i < vit; ++i) mbar_wait_bounded(&vfull[i % VS], (i / VS) & 1, &g_err_kv8_attn, ERR_KV8_EMPTY_WAIT);
  } else if (warp >= CR_MMA && warp < CR_Q) {
    // ====== half g's products: S of its next chunk takes the place of P of the one before, and so is issued
    // behind the product that reads it (the tensor cores do what one thread issues in order) ======
    constexpr uint32_t ID_S = tc_idesc(128, AT_CHUNK, false, false, true), ID_O = tc_idesc(128, DP, false, true, true);
    const int g = warp - CR_MMA;
    const uint64_t d_k = tile_desc<128>(sm, 16), d_q = tile_desc<128>(sm + S::OFF_Q, 16), d_v = tile_desc<128>(sm + S::OFF_V, SUB);
    const uint32_t t_s = tmem + CR_S + g * 128, t_o = tmem + CR_O + g * DP;
    int pi = 0, it = 0, n = 0, t = 0, qs = 0, i0 = 0;  // chunks; the half's chunks and pieces; halves of q; chunks taken in turn
    CrossPiece x;
    while (next_piece(pi, x, false)) {
      const bool two = x.rows > p.half_rows();
      const int step = two ? 1 : 2, d0 = two ? 0 : (g - i0) & 1, chunks = x.cn - x.c0;
      const int slot = (qs + (two ? g : 0)) & 1;
      const uint64_t q = d_q + (slot * T >> 4);
      // (a half without a chunk waits too: what it leaves below is then of this use of the slot)
      bool ok = wait_warp(&qready[slot], ((qs + (two ? g : 0)) >> 1) & 1, ERR_KV8_S_WAIT);
      auto keys = [&](int d) {  // waits for chunk d's keys
        const int i = it + d;
        ok = wait_warp(&kfull[i % KS], (i / KS) & 1, ERR_KV8_FULL_WAIT) && ok;
        if (!two && ((d ^ d0) & 1) && lane == 0) mbar_arrive(&kempty[i % KS]);  // the other half's
      };
      auto scores = [&](int d) {
        const int i = (it + d) % KS;
        if (ok) {
          tc_fence_after();
          const uint64_t k = d_k + (i * T >> 4);
#pragma unroll
          for (int e = 0; e < DP / 64; ++e) mma_f16_x4(t_s, q + e * (SUB >> 4), k + e * (SUB >> 4), ID_S, e > 0);
        }
        tc_commit2(&sready[g], &kempty[i]);
        if (d + step >= chunks) tc_commit(&qfree[slot]);  // q has been read (the slot waits for both halves)
      };
      for (int d = 0; d <= d0 && d < chunks; ++d) keys(d);
      if (d0 < chunks) scores(d0);
      else if (lane == 0) mbar_arrive(&qfree[slot]);
      // What a chunk's products need besides its weights, and the keys of the half's next one, is waited for first.
#pragma unroll 1
      for (int d = 0; d < chunks; ++d) {
        const int i = it + d, sv = i % VS;
        ok = wait_warp(&vfull[sv], (i / VS) & 1, ERR_KV8_PV_WAIT) && ok;
        if (!two && ((d ^ d0) & 1)) {
          if (lane == 0) mbar_arrive(&vempty[sv]);
          continue;
        }
        const int rem = min(AT_CHUNK, x.len - (x.c0 + d) * AT_CHUNK), steps = (rem + 15) / 16;
        if (rem & 15) {  // rows behind the last state: weights of 0, which no NaN may meet
          uint8_t* v = sm + S::OFF_V + sv * T + rem * 128;
          const int all = (steps * 16 - rem) * 8;
          for (int e = lane; e < all; e += 32)
#pragma unroll
            for (int j = 0; j < DP / 64; ++j) *reinterpret_cast<uint4*>(v + j * SUB + e * 16) = make_uint4(0u, 0u, 0u, 0u);
          fence_async_smem();
          __syncwarp();
        }
        // (not so where the halves take turns: the keys are two chunks away, on their way from memory)
        if (two && d + 1 < chunks) keys(d + 1);
        if (d == d0 && t++ > 0) ok = wait_warp(&left[g], t & 1, ERR_KV8_PV_WAIT) && ok;  // the piece before has left O
        // A wait tells only a phase's parity: a half waits for the other one's q too, so that it misses none of a slot's.
        if (two && d == 0) {
          ok = wait_warp(&qready[1 - slot], ((qs + 1 - g) >> 1) & 1, ERR_KV8_S_WAIT) && ok;
          if (lane == 0) mbar_arrive(&qfree[1 - slot]);
        }
        // 64 states at a time (16 further: 8 columns of P, 16 rows of V)
        const uint64_t v = d_v + (sv * T >> 4);
        ok = wait_warp(&pready[0][g], n & 1, ERR_KV8_PV_WAIT) && ok;
        tc_fence_after();
        if (ok && steps >= 4) {
          mma_f16_ts4(t_o, t_s, v, ID_O, d > d0);
        } else if (ok) {
#pragma unroll 1
          for (int e = 0; e < steps; ++e) mma_f16_ts(t_o, t_s + 8 * e, v + e * 128, ID_O, e > 0 || d > d0);
        }
        ok = wait_warp(&pready[1][g], n & 1, ERR_KV8_PV_WAIT) && ok;
        tc_fence_after();
        if (ok && steps == 8) {
          mma_f16_ts4(t_o, t_s + 32, v + 512, ID_O, true);
        } else if (ok) {
#pragma unroll 1
          for (int e = 4; e < steps; ++e) mma_f16_ts(t_o, t_s + 8 * e, v + e * 128, ID_O, true);
        }
        if (!two) {
          tc_commit(&vempty[sv]);
          for (int e = d + 1; e <= d + step && e < chunks; ++e) keys(e);
        }
        if (d + step < chunks) scores(d + step);
        else tc_commit(&pvdone[g]);
        if (two) tc_commit(&vempty[sv]);
        ++n;
      }
      it += chunks;
      i0 += two ? 0 : chunks;
      qs += two ? 2 : 1;
    }
  } else if (warp == CR_Q) {
    // ====== the run's pieces, and q of their tiles, ahead ======
    constexpr int LPR = DP / 8, RPW = 32 / LPR;  // lanes of a row (8 values each), rows at a time
    const int piece = lane % LPR;
    const Run run = find_run<CR_ROWS>(p, blockIdx.x, gridDim.x);
    Pieces<CR_ROWS, P> w(p, run);
    const uint32_t times = wait_times(run.per);  // (a place in the ring, or of q, may be held for all of a piece)
    int qs = 0, pi = 0;
    auto leave = [&]() -> bool {
      const int e = pi % CR_PIECES;
      bool ok = pi < CR_PIECES || wait_warp(&pc_empty[e], ((pi / CR_PIECES) - 1) & 1, ERR_KV8_EMPTY_WAIT, times);
      ok = ok && w.next();
      CrossPiece x{};
      x.whole = -1;
      if (ok)
        x = CrossPiece{w.psq.q0, __ldg(p.kv_start + w.pb), w.psq.len, w.ph, w.row0(), w.rows(), w.c0,
                       max(w.c0, min(w.c1, (w.psq.len + AT_CHUNK - 1) / AT_CHUNK)), w.whole(), w.slot()};
      if (lane == 0) {
        s_piece[e] = x;
        mbar_arrive(&pc_full[e]);
      }
      __syncwarp();
      ++pi;
      return ok;
    };
    // Finding a piece takes as long as a short one's products, so pieces are left ahead, but not so
    // that the first ones' q waits for it.
    bool more = leave();
#pragma unroll 1
    for (int j = 0;; ++j) {
      const CrossPiece x = s_piece[j % CR_PIECES];  // (written over by piece j + CR_PIECES)
      if (x.whole < 0) break;
#pragma unroll 1
      for (int half = 0; x.c0 < x.cn && half * p.half_rows() < x.rows; ++half, ++qs) {
        const int s = qs & 1, row0 = x.row0 + half * p.half_rows(), rows = min(p.half_rows(), x.rows - half * p.half_rows());
        if (qs > 1) wait_warp(&qfree[s], ((qs >> 1) - 1) & 1, ERR_KV8_S_WAIT, times);
        uint8_t* to = sm + S::OFF_Q + s * T;
        if (p.q_map) {  // whole tokens of a group's heads; rows behind the last are other requests', or zeros
          if (lane == 0) {
            mbar_arrive_expect_tx(&qready[s], p.half_rows() * (DP / 64) * 128);
#pragma unroll
            for (int i = 0; i < DP / 64; ++i)
              tma_load3(to + i * SUB, &tq, 64 * i, x.h * p.group, static_cast<int>(x.q0) + row0 / p.group, &qready[s]);
          }
          __syncwarp();
          continue;
        }
        const __nv_bfloat16* q = p.q + x.q0 * p.q_tok + int64_t(x.h) * p.group * p.q_head + piece * 8;
        int i = (row0 + lane / LPR) / p.group, j = row0 + lane / LPR - i * p.group;
#pragma unroll 2
        for (int r = lane / LPR; r < CR_HALF; r += RPW) {
          const bool there = r < rows && piece * 8 < p.D;
          cp16(to + (piece / 8) * SUB + r * 128 + (((piece & 7) ^ (r & 7)) << 4), there ? q + i * p.q_tok + j * p.q_head : p.q, there);
          for (j += RPW; j >= p.group; j -= p.group) ++i;
        }
        cp_wait();
        if (p.flip) {  // a negative scale
#pragma unroll 1
          for (int r = lane / LPR; r < CR_HALF; r += RPW) {
            uint4* at = reinterpret_cast<uint4*>(to + (piece / 8) * SUB + r * 128 + (((piece & 7) ^ (r & 7)) << 4));
            uint4 w = *at;
            w.x ^= p.flip; w.y ^= p.flip; w.z ^= p.flip; w.w ^= p.flip;
            *at = w;
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&qready[s]);
      }
      while (more && pi < min(2 * j + 2, j + 1 + CR_AHEAD)) more = leave();
    }
    for (int i = max(0, qs - S::QS); i < qs; ++i) mbar_wait_bounded(&qready[i & 1], (i >> 1) & 1, &g_err_kv8_attn, ERR_KV8_S_WAIT);
  } else {
    // ====== softmax: half g, rows 32 k + lane of it; then the tile's outputs ======
    const int g = warp >> 2, k = warp & 3, r = 32 * k + lane;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(32 * k) << 16);
    const uint32_t t_s = t_lane + CR_S + g * 128, t_o = t_lane + CR_O + g * DP;
    const float a = p.scale2;
    uint8_t* stage = sm + S::OFF_ST + warp * 2048;
    // This half's chunks; before x: each half's pieces, those that one half handed over to the other, chunks of tiles
    // that both took, and chunks taken in turn.
    int n = 0, pi = 0, t[2] = {0, 0}, u = 0, v = 0, i0 = 0;
    CrossPiece x;
    while (next_piece(pi, x, true)) {
      const bool two = x.rows > p.half_rows();
      const int step = two ? 1 : 2, chunks = x.cn - x.c0;
      const int f = two ? g : i0 & 1, d0 = two || g == f ? 0 : 1;  // f: the half that takes the first chunk
      const int base = two ? g * p.half_rows() : 0, end = min(x.rows, base + p.half_rows());  // the half's rows of the tile
      const bool any = base + 32 * k < end;                                     // of the warp's rows
      // (a row that is not there has weights of 0)
      float m = base + r < end ? -INFINITY : INFINITY, l = 0.f;
#pragma unroll 1
      for (int d = d0; d < chunks; d += step, ++n) {
        const int lim = x.len - (x.c0 + d) * AT_CHUNK;
        wait_warp(&sready[g], n & 1, ERR_KV8_S_WAIT);
        tc_fence_after();
        if (!any) {  // rows that are not there: weights of any value (and turns that are handed on)
          if (lane == 0) {
            mbar_arrive(&pready[0][g]);
            mbar_arrive(&pready[1][g]);
          }
          if (two) {
            if (g == 1 || v > 0) wait_warp(&turn[1 - g][k], (v - (g == 0)) & 1, ERR_KV8_S_WAIT);
            if (lane == 0) mbar_arrive(&turn[g][k]);
            ++v;
          }
          continue;
        }
        if (lim < AT_CHUNK) mask_columns(t_s, lim);
        float z[4][32];
#pragma unroll
        for (int w = 0; w < 4; ++w) tmem_ld32_begin(t_s + 32 * w, z[w]);
#pragma unroll
        for (int w = 0; w < 4; ++w) tmem_ld32_end(z[w]);
        // Where both halves take every chunk they take turns, so that one's products run beside the other's weights.
        if (two && (g == 1 || v > 0)) wait_warp(&turn[1 - g][k], (v - (g == 0)) & 1, ERR_KV8_S_WAIT);
        // 1. the row's largest score
        float big[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          big[w] = fmaxf(z[w][0], z[w][1]);
#pragma unroll
          for (int e = 2; e < 32; e += 2) big[w] = max3(big[w], z[w][e], z[w][e + 1]);
        }
        const float top = max3(fmaxf(big[0], big[1]), big[2], big[3]) * a;  // (a is positive)
        const bool anew = top - m > CR_RAISE || m == -INFINITY;
        if (__any_sync(FULL_MASK, anew)) {
          const float to = fmaxf(top, m), f = to == -INFINITY || l == 0.f ? 1.f : ex2(m - to);
          m = to;
          l *= f;
          if (d > d0) scale_outputs<DP>(t_o, f);  // (the products of the chunks before were done ahead of S)
        }
        const float nref = m == -INFINITY ? 0.f : -m;
        const float2 a2 = make_float2(a, a), b2 = make_float2(nref, nref);
        // 2. the weights, in the scores' place (16 columns of pairs for 32)
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};  // (of the chunk: small weights beside a heavy l)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          // (64 wide, where the products are half as long, the other half may begin earlier)
          if (DP == 64 && w == 2 && two && lane == 0) mbar_arrive(&turn[g][k]);
          uint32_t h[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 y = __ffma2_rn(make_float2(z[w][2 * e], z[w][2 * e + 1]), a2, b2);
            const float2 v = make_float2(ex2(y.x), ex2(y.y));
            sum[e & 1] = __fadd2_rn(sum[e & 1], v);
            const __nv_bfloat162 c = __floats2bfloat162_rn(v.x, v.y);
            h[e] = *reinterpret_cast<const uint32_t*>(&c);
          }
          tmem_st8(t_s + 16 * w, h);
          tmem_st8(t_s + 16 * w + 8, h + 8);
          if (w & 1) {
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&pready[w >> 1][g]);
          }
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        if (DP != 64 && two && lane == 0) mbar_arrive(&turn[g][k]);
        v += two;
      }

      // The outputs.  Where both halves stand for the same rows, the one that had the first chunk writes them.
      const bool both = !two && chunks > 1;
      const int o = 1 - g;
      if (g != f && both) {
        s_ml[u & 1][r] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&met[u & 1][k]);
      } else if (d0 < chunks || chunks == 0) {
        const int row = base + r;
        const bool there = row < end && (chunks > 0 || two || g == f);
        // where the row goes; and 16 bytes of 32 columns of four rows that the lane stores for the warp
        const int i = there ? (x.row0 + row) / p.group : 0, j = there ? x.row0 + row - i * p.group : 0;
        const int64_t at = there ? (x.q0 + i) * p.q_heads + int64_t(x.h) * p.group + j : -1;
        const int piece = lane & 3;
        __nv_bfloat16* to[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t y = __shfl_sync(FULL_MASK, at, 8 * e + (lane >> 2));
          to[e] = y < 0 ? nullptr : p.out + y * p.D + 8 * piece;
        }
        float f0 = 1.f, f1 = 0.f;
        if (l == 0.f) m = -INFINITY;  // (a NaN stays)
        if (both) {
          wait_warp(&met[u & 1][k], (u >> 1) & 1, ERR_KV8_PV_WAIT);
          const float2 ml = s_ml[u & 1][r];
          const float top = fmaxf(m, ml.y == 0.f ? -INFINITY : ml.x);
          f0 = l == 0.f ? 0.f : ex2(m - top);
          f1 = ml.y == 0.f ? 0.f : ex2(ml.x - top);
          l = l * f0 + ml.y * f1;
          m = top;
          wait_warp(&pvdone[o], t[o] & 1, ERR_KV8_PV_WAIT);
        }
        if (chunks > 0) {
          wait_warp(&pvdone[g], t[g] & 1, ERR_KV8_PV_WAIT);
          tc_fence_after();
        }
        if (x.whole) {
          const float inv = l == 0.f ? 0.f : __frcp_rn(l);
          f0 *= inv;
          f1 *= inv;
        }
        float* part = p.part + int64_t(x.slot) * CR_ROWS * (DP + 2);
        if (!any && chunks > 0 && lane == 0) {
          mbar_arrive(&left[g]);
          if (both) mbar_arrive(&left[o]);
        }
#pragma unroll 1
        for (int w0 = any ? 0 : DP; w0 < DP; w0 += 32) {
          float y[32];
          if (chunks > 0) {
            tmem_ld32_begin(t_o + w0, y);
            tmem_ld32_end(y);
          }
          if (chunks > 0) {
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 yy = __fmul2_rn(make_float2(y[e], y[e + 1]), make_float2(f0, f0));
              y[e] = yy.x;
              y[e + 1] = yy.y;
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = 0.f;
          }
          if (both) {
            float z[32];
            tmem_ld32_begin(t_lane + CR_O + o * DP + w0, z);
            tmem_ld32_end(z);
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = fmaf(z[e], f1, y[e]);
          }
          if (w0 + 32 == DP && chunks > 0) {  // O has been read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&left[g]);
              if (both) mbar_arrive(&left[o]);
            }
          }
          if (x.whole) {
            // through shared memory, so that four lanes write 64 bytes of a row
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t h[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 v = __floats2bfloat162_rn(y[8 * q + 2 * e], y[8 * q + 2 * e + 1]);
                h[e] = *reinterpret_cast<const uint32_t*>(&v);
              }
              *reinterpret_cast<uint4*>(stage + lane * 64 + ((q ^ (lane >> 1 & 3)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
            }
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int rr = 8 * e + (lane >> 2);
              const uint4 v = *reinterpret_cast<const uint4*>(stage + rr * 64 + ((piece ^ (rr >> 1 & 3)) << 4));
              if (to[e] && w0 + 8 * piece < p.D) *reinterpret_cast<uint4*>(to[e] + w0) = v;
            }
            __syncwarp();
          } else if (there) {
            float4* dst = reinterpret_cast<float4*>(part + row * DP + w0);
#pragma unroll
            for (int e = 0; e < 8; ++e) dst[e] = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
          }
        }
        if (there && !x.whole) {
          part[CR_ROWS * DP + row] = m;
          part[CR_ROWS * DP + CR_ROWS + row] = l;
        } else if (there && p.lse) {
          p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2_F;
        }
      }
      t[f] += chunks > 0;
      t[1 - f] += chunks > (two ? 0 : 1);
      u += both;
      i0 += two ? 0 : chunks;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && s_fail) atomicOr(&g_err_kv8_attn, s_fail);
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

cudaError_t cross_read_device_error(uint32_t* code) {
  uint32_t v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_err_kv8_attn, sizeof(v));
  if (e != cudaSuccess) return e;
  if (v) e = cudaMemcpyToSymbol(g_err_kv8_attn, &zero, sizeof(zero));
  *code |= v;
  return e;
}

namespace {

lilicorr_status fail(lilicorr_status st, const char* msg) {
  set_last_error(msg);
  return st;
}

size_t workspace_of(int D) { return size_t(device_sm_count()) * 2 * CR_ROWS * ((D <= 64 ? 64 : 128) + 2) * sizeof(float); }
bool dim_ok(int32_t D) { return D >= 8 && D <= 128 && D % 8 == 0; }

// Null where rows of tokens and heads are in order, else what is wrong with them.
const char* rows_error(const void* x, int64_t tok, int64_t head) {
  if (!x) return "null pointer";
  if (reinterpret_cast<uintptr_t>(x) % 16) return "rows are 16-byte aligned";
  if (tok % 8 || head % 8) return "row strides are multiples of 8 elements";
  if (tok < 0 || head < 0 || tok > (int64_t(1) << 38) || head > (int64_t(1) << 38)) return "a row stride is out of range";
  return nullptr;
}

// Boxes of 128 rows, `group` heads of 128 / group tokens, 64 values wide; what lies behind the head dimension
// reads as zeros.
cudaError_t rows_map(CUtensorMap* tm, const void* x, int D, int heads, int64_t total, int64_t tok, int64_t head, int group) {
  auto fn = encode_fn();
  if (!fn) return cudaErrorInvalidValue;
  const cuuint64_t dims[3] = {cuuint64_t(D), cuuint64_t(heads), cuuint64_t(total)};
  // (a dimension of one has no stride of its own)
  const cuuint64_t strides[2] = {cuuint64_t(heads > 1 ? head : D) * 2, cuuint64_t(total > 1 ? tok : D) * 2};
  const cuuint32_t box[3] = {64, cuuint32_t(group), cuuint32_t(AT_CHUNK / group)}, estr[3] = {1, 1, 1};
  return fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(x), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, D <= 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

template <int DP, class P>
cudaError_t launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const CrossParams& params, cudaStream_t stream) {
  P p;
  static_cast<CrossParams&>(p) = params;
  constexpr int smem = CrossShape<DP>::SMEM;
  const int grid = device_sm_count();
  cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void*>(cross_attention_kernel<DP, P>), smem);
  if (e != cudaSuccess) return e;
  cross_attention_kernel<DP, P><<<grid, 32 * CR_WARPS, smem, stream>>>(tq, tk, tv, p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  PdlScope pdl(true);
  // (a warp takes four rows of a tile in two parts)
  const int most = static_cast<int>(std::min<int64_t>(2 * p.half, int64_t(p.max_new) * p.group));
  e = launch_k(kv8_join_kernel<DP, CR_ROWS, 4, 16, P>, dim3(grid, (most + 15) / 16), dim3(128), 0, stream, p, grid, (most + 15) / 16 * 16);
  if (e == cudaSuccess) note_launch(2);
  return e;
}

}  // namespace
}  // namespace lilicorr

using namespace lilicorr;

extern "C" {

size_t lilicorr_cross_attention_workspace_bytes(int32_t head_dim) { return dim_ok(head_dim) ? workspace_of(head_dim) : 0; }

lilicorr_status lilicorr_cross_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride, int64_t total, int32_t q_heads,
                                         const void* k, int64_t k_token_stride, int64_t k_head_stride, const void* v, int64_t v_token_stride,
                                         int64_t v_head_stride, int64_t total_kv, int32_t kv_heads, int32_t head_dim, const int32_t* q_start,
                                         const int32_t* kv_start, const int32_t* kv_len, int64_t batch, int32_t max_new, float scale, void* out,
                                         float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  const char* why = rows_error(q, q_token_stride, q_head_stride);
  if (!why) why = rows_error(k, k_token_stride, k_head_stride);
  if (!why) why = rows_error(v, v_token_stride, v_head_stride);
  if (!why && !dim_ok(head_dim)) why = "head_dim is a multiple of 8, at most 128";
  if (!why && (!q_start || !kv_start || !kv_len)) why = "null pointer";
  if (!why && !word_aligned({q_start, kv_start, kv_len, lse})) why = "row ranges, lengths and lse are 4-byte aligned";
  if (!why && (batch < 1 || batch > (1 << 20))) why = "1 <= batch <= 2^20";
  if (!why && (total < 1 || total > INT_MAX || total_kv < 1 || total_kv > INT_MAX - 256)) why = "rows are out of range";
  if (!why && (max_new < 1 || max_new > (1 << 24))) why = "1 <= max_new <= 2^24";
  if (!why && (kv_heads < 1 || kv_heads > 1024 || q_heads < 1 || q_heads % kv_heads || q_heads / kv_heads > 1024))
    why = "1 <= kv_heads <= 1024, q_heads is a multiple of it, at most 1024 times";
  if (!why && ((kv_heads > 1 && (k_head_stride < head_dim || v_head_stride < head_dim)) ||
               (total_kv > 1 && (k_token_stride < head_dim || v_token_stride < head_dim))))
    why = "rows of keys and values do not overlap";
  if (!why && (!out || reinterpret_cast<uintptr_t>(out) % 16)) why = "out is null or not 16-byte aligned";
  // Halves of whole tokens, which a tensor map brings, but where that would leave a quarter of the rows empty.
  const int group = why ? 1 : q_heads / kv_heads, whole = AT_CHUNK / group * group, half = whole >= 96 ? whole : CR_HALF;
  // a request's rows, and its work units, are counted in 32 bits
  if (!why && int64_t(max_new) * group > INT_MAX - 256) why = "max_new * q_heads / kv_heads is too large";
  if (!why && (int64_t(max_new) * group / (2 * half) + 1) * kv_heads * ((total_kv + 127) / 128 + 8) > UINT_MAX)
    why = "max_new * q_heads * the states are too large";
  if (!why && !std::isfinite(scale * LOG2E_F)) why = "scale, or scale * log2 e, is not finite";
  if (why) return fail(LILICORR_ERR_INVALID_ARG, why);
  if (!workspace || workspace_bytes < workspace_of(head_dim) || reinterpret_cast<uintptr_t>(workspace) % 256)
    return fail(LILICORR_ERR_WORKSPACE, "lilicorr_cross_attention: workspace missing, too small or misaligned");
  // what is written lies apart from what is read
  using wide = unsigned __int128;
  auto extent = [&](int64_t n, int64_t tok, int64_t heads, int64_t head) { return (wide(n - 1) * tok + wide(heads - 1) * head + head_dim) * 2; };
  auto meet = [](const void* a, wide n, const void* b, wide m) {
    const wide x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + m && y < x + n;
  };
  const wide o_bytes = wide(total) * q_heads * head_dim * 2, l_bytes = wide(total) * q_heads * 4;
  const void* in[6] = {q, k, v, q_start, kv_start, kv_len};
  const wide in_bytes[6] = {extent(total, q_token_stride, q_heads, q_head_stride), extent(total_kv, k_token_stride, kv_heads, k_head_stride),
                            extent(total_kv, v_token_stride, kv_heads, v_head_stride), wide(batch + 1) * 4, wide(batch) * 4, wide(batch) * 4};
  bool overlap = lse && meet(out, o_bytes, lse, l_bytes);
  for (int i = 0; i < 6; ++i) overlap = overlap || meet(in[i], in_bytes[i], out, o_bytes) || (lse && meet(in[i], in_bytes[i], lse, l_bytes));
  if (overlap) return fail(LILICORR_ERR_INVALID_ARG, "lilicorr_cross_attention: out and lse overlap one another, or what is read");
  CrossParams p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_tok = q_token_stride; p.q_head = q_head_stride;
  p.total = total; p.total_kv = total_kv;
  p.q_heads = q_heads; p.group = group; p.heads = kv_heads; p.D = head_dim;
  p.half = half; p.tile_inv = ((uint64_t(1) << 40) + 2 * half - 1) / (2 * half);
  p.q_start = q_start; p.kv_start = kv_start; p.kv_len = kv_len;
  p.batch = batch; p.max_new = max_new;
  p.scale2 = std::max(std::fabs(scale) * LOG2E_F, FLT_MIN);  // (never 0, so that a score of infinity stays one)
  p.flip = std::signbit(scale) ? 0x80008000u : 0u;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.part = static_cast<float*>(workspace);
  CUtensorMap tq{}, tk, tv;
  cudaError_t e = rows_map(&tk, k, head_dim, kv_heads, total_kv, k_token_stride, k_head_stride, 1);
  if (e == cudaSuccess) e = rows_map(&tv, v, head_dim, kv_heads, total_kv, v_token_stride, v_head_stride, 1);
  if (e != cudaSuccess) return fail(LILICORR_ERR_INVALID_ARG, "lilicorr_cross_attention: no tensor map for these strides");
  // q through a map too where halves are whole tokens (else, or with a negative scale, or rows that overlap, by copies
  // of 16 bytes: 9 requests of 602 rows over 1,303 states, three rows to a head, 155 us that way)
  p.q_map = half % group == 0 && !p.flip && (q_heads == 1 || q_head_stride >= head_dim) && (total == 1 || q_token_stride >= head_dim) &&
            rows_map(&tq, q, head_dim, q_heads, total, q_token_stride, q_head_stride, p.group) == cudaSuccess;
  auto go = [&](auto f) { return f(tq, tk, tv, p, static_cast<cudaStream_t>(stream)); };
  if (head_dim <= 64) e = half == CR_HALF ? go(launch<64, CrossFull>) : go(launch<64, CrossPart>);
  else e = half == CR_HALF ? go(launch<128, CrossFull>) : go(launch<128, CrossPart>);
  if (e != cudaSuccess) return fail(LILICORR_ERR_CUDA, cudaGetErrorString(e));
  return LILICORR_OK;
}

}  // extern "C"
