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
// are joined as they are written.  While one group forms its weights the tensor cores work for the other.
// Warps: two groups of four for the softmax; four that bring q of the next tile and write the outputs of
// the one before; one that loads keys and values through tensor maps; one that issues S = Q K^T and one
// that issues O += P V.
//
// Roundings below f32: the weights are bf16 (off by 2^-8 of their value at most) for the second product, whose operands
// have one type; the sums take them unrounded.  A row's maximum moves only where a score passes it by
// more than 2^8, and only then is O scaled.  What lies behind a request's last state is never summed: its
// scores are -inf, its values zeros.
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
  __nv_bfloat16* out;  // [total, q_heads, D]
  float* lse;          // [total, q_heads] or null
  float* part;         // [2 * grid][256 * (padded D + 2)]: products, maxima, sums
  __device__ __forceinline__ int kv_heads() const { return heads; }
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
  static constexpr int SMEM = 1024 + OFF_Q + QS * T;
};
constexpr int CR_WARPS = 15, CR_CONSUMERS = 14, CR_PIECES = 4;
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
template <int DP>
__device__ __noinline__ void scale_outputs(uint32_t t, float f) {
#pragma unroll 1
  for (int w0 = 0; w0 < DP; w0 += 16) {
    float o[16];
    tmem_ld16(t + w0, o);
#pragma unroll
    for (int n = 0; n < 16; ++n) o[n] *= f;
    tmem_st16(t + w0, o);
  }
}

template <int DP>
__global__ void __launch_bounds__(32 * CR_WARPS, 1)
    cross_attention_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const __grid_constant__ CrossParams p) {
  using S = CrossShape<DP>;
  constexpr int KS = S::KS, VS = S::VS, T = S::T, SUB = S::SUB;
  extern __shared__ uint8_t cr_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(cr_raw) + 1023) & ~uintptr_t(1023));
  // sready, pready, pvdone: of each half, a phase for each of its chunks.  S of a chunk is made once the
  // half's products before it are done, so who has a chunk's scores knows that.
  __shared__ __align__(8) uint64_t kfull[KS], kempty[KS], vfull[VS], vempty[VS], sready[2], pready[2], pvdone[2], qready[2], qfree[2],
      left[2], pc_full[CR_PIECES], pc_empty[CR_PIECES], met[2][2][4];
  __shared__ CrossPiece s_piece[CR_PIECES];
  __shared__ float2 s_ml[2][2][CR_HALF];  // a row's maximum and sum at the end of a piece: by the half's pieces, in turn
  __shared__ uint32_t s_tmem;
  __shared__ volatile uint32_t s_fail;

  const int tid = threadIdx.x, warp = __shfl_sync(FULL_MASK, tid >> 5, 0), lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < KS; ++i) { mbar_init(&kfull[i], 1); mbar_init(&kempty[i], 1); }
    for (int i = 0; i < VS; ++i) { mbar_init(&vfull[i], 1); mbar_init(&vempty[i], 1); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sready[i], 1); mbar_init(&pready[i], 4); mbar_init(&pvdone[i], 1);
      mbar_init(&qready[i], 4); mbar_init(&qfree[i], 1); mbar_init(&left[i], 4);
      for (int j = 0; j < 4; ++j) { mbar_init(&met[0][i][j], 1); mbar_init(&met[1][i][j], 1); }
    }
    for (int i = 0; i < CR_PIECES; ++i) { mbar_init(&pc_full[i], 1); mbar_init(&pc_empty[i], CR_CONSUMERS); }
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

  // A wait by a whole warp.  The first one that gives up makes every later one give up soon, and the
  // roles' loops end.
  auto wait_warp = [&](uint64_t* bar, uint32_t parity, uint32_t site) -> bool {
#pragma unroll 1
    for (uint32_t i = 0; !__all_sync(FULL_MASK, try_wait_us(bar, parity)); ++i)
      if (__any_sync(FULL_MASK, i == WAIT_TRIES || s_fail != 0)) {
        if (s_fail == 0) s_fail = site;
        return false;
      }
    return true;
  };
  // The next piece, read by a warp.
  auto next_piece = [&](int pi, CrossPiece& x) -> bool {
    const int e = pi % CR_PIECES;
    if (!wait_warp(&pc_full[e], (pi / CR_PIECES) & 1, ERR_KV8_FULL_WAIT)) return false;
    x = s_piece[e];
    if (x.whole < 0) return false;
    __syncwarp();
    if (lane == 0) mbar_arrive(&pc_empty[e]);
    return true;
  };

  if (warp == 12) {
    // ====== the run's pieces, and their keys and values ======
    const Run run = find_run<CR_ROWS>(p, blockIdx.x, gridDim.x);
    Pieces<CR_ROWS, CrossParams> w(p, run);
    int it = 0, kit = 0, vit = 0, pi = 0;  // (kit, vit: chunks whose keys, values are on their way)
    // Pieces are left one ahead of the one that is loaded, so that its q can be made ready.
    auto leave = [&](CrossPiece& x) -> bool {
      const int e = pi % CR_PIECES;
      bool ok = pi < CR_PIECES || wait_warp(&pc_empty[e], ((pi / CR_PIECES) - 1) & 1, ERR_KV8_EMPTY_WAIT);
      ok = ok && w.next();
      if (ok)
        x = CrossPiece{w.psq.q0, __ldg(p.kv_start + w.pb), w.psq.len, w.ph, w.ptile * CR_ROWS, w.rows(), w.c0,
                       max(w.c0, min(w.c1, (w.psq.len + AT_CHUNK - 1) / AT_CHUNK)), w.whole(), w.slot()};
      else
        x.whole = -1;
      if (lane == 0) {
        s_piece[e] = x;
        mbar_arrive(&pc_full[e]);
      }
      ++pi;
      return ok;
    };
    CrossPiece now{}, next{};
    bool ok_run = leave(now);
    while (ok_run) {
      const bool more = leave(next);
#pragma unroll 1
      for (int c = now.c0; c < now.cn; ++c, ++it) {
        auto load = [&](const CUtensorMap* tm, uint8_t* to, uint64_t* full) {
          if (lane == 0) {
            mbar_arrive_expect_tx(full, T);
#pragma unroll
            for (int i = 0; i < DP / 64; ++i) tma_load3(to + i * SUB, tm, 64 * i, now.h, now.kv0 + c * AT_CHUNK, full);
          }
          __syncwarp();
        };
        const int sk = it % KS, sv = it % VS;
        ok_run = it < KS || wait_warp(&kempty[sk], ((it / KS) - 1) & 1, ERR_KV8_EMPTY_WAIT);
        if (!ok_run) break;
        load(&tk, sm + sk * T, &kfull[sk]);
        ++kit;
        ok_run = it < VS || wait_warp(&vempty[sv], ((it / VS) - 1) & 1, ERR_KV8_EMPTY_WAIT);
        if (!ok_run) break;
        load(&tv, sm + S::OFF_V + sv * T, &vfull[sv]);
        ++vit;
      }
      now = next;
      ok_run = ok_run && more;
    }
    if (s_fail) {  // what is in flight has to land
      for (int i = max(0, kit - KS); i < kit; ++i)
        mbar_wait_bounded(&kfull[i % KS], (i / KS) & 1, &g_err_kv8_attn, ERR_KV8_EMPTY_WAIT);
      for (int i = max(0, vit - VS); i < vit; ++i)
        mbar_wait_bounded(&vfull[i % VS], (i / VS) & 1, &g_err_kv8_attn, ERR_KV8_EMPTY_WAIT);
    }
  } else if (warp == 13) {
    // ================= S = Q K^T =================
    constexpr uint32_t ID = tc_idesc(128, AT_CHUNK, false, false, true);
    const uint64_t d_k = tile_desc<128>(sm, 16), d_q = tile_desc<128>(sm + S::OFF_Q, 16);
    int it = 0, qs = 0, n0 = 0, n1 = 0;  // chunks; halves of q; chunks of each half
    CrossPiece x;
    for (int pi = 0; next_piece(pi, x); ++pi) {
      if (x.c0 >= x.cn) continue;
      const bool two = x.rows > CR_HALF;
      bool ok = wait_warp(&qready[qs & 1], (qs >> 1) & 1, ERR_KV8_S_WAIT);
      if (two) ok = wait_warp(&qready[(qs + 1) & 1], ((qs + 1) >> 1) & 1, ERR_KV8_S_WAIT) && ok;
#pragma unroll 1
      for (int c = x.c0; c < x.cn; ++c, ++it) {
        const int st = it % KS;
        ok = wait_warp(&kfull[st], (it / KS) & 1, ERR_KV8_FULL_WAIT) && ok;
        const uint64_t k = d_k + (st * T >> 4);
        auto half = [&](int g, int& n) {
          if (n > 0) ok = wait_warp(&pvdone[g], (n - 1) & 1, ERR_KV8_S_WAIT) && ok;
          if (ok) {
            tc_fence_after();
            const uint64_t q = d_q + (((qs + (two ? g : 0)) & 1) * T >> 4);
#pragma unroll
            for (int d = 0; d < DP / 16; ++d) {
              const int at = (d / 4) * (SUB >> 4) + (d % 4) * 2;
              mma_f16(tmem + CR_S + g * 128, q + at, k + at, ID, d > 0);
            }
          }
          tc_commit(&sready[g]);
          ++n;
        };
        if (two || ((c - x.c0) & 1) == 0) half(0, n0);
        if (two || ((c - x.c0) & 1) == 1) half(1, n1);
        tc_commit(&kempty[st]);
      }
      tc_commit(&qfree[qs & 1]);
      ++qs;
      if (two) {
        tc_commit(&qfree[qs & 1]);
        ++qs;
      }
    }
  } else if (warp == 14) {
    // ================= O += P V =================
    constexpr uint32_t ID = tc_idesc(128, DP, false, true, true);
    const uint64_t d_v = tile_desc<128>(sm + S::OFF_V, SUB);
    int it = 0, n0 = 0, n1 = 0, t0 = 0, t1 = 0;  // chunks; chunks of each half, pieces of each half
    CrossPiece x;
    for (int pi = 0; next_piece(pi, x); ++pi) {
      const bool two = x.rows > CR_HALF;
#pragma unroll 1
      for (int c = x.c0; c < x.cn; ++c, ++it) {
        const int st = it % VS, rem = min(AT_CHUNK, x.len - c * AT_CHUNK), steps = (rem + 15) / 16;
        bool ok = wait_warp(&vfull[st], (it / VS) & 1, ERR_KV8_PV_WAIT);
        if (rem & 15) {  // rows behind the last state: weights of 0, which no NaN may meet
          uint8_t* v = sm + S::OFF_V + st * T + rem * 128;
          const int n = (steps * 16 - rem) * 8;
          for (int i = lane; i < n; i += 32)
#pragma unroll
            for (int j = 0; j < DP / 64; ++j) *reinterpret_cast<uint4*>(v + j * SUB + i * 16) = make_uint4(0u, 0u, 0u, 0u);
          fence_async_smem();
          __syncwarp();
        }
        const uint64_t v = d_v + (st * T >> 4);
        auto half = [&](int g, int& n, int& t, bool first) {
          if (first && t++ > 0) ok = wait_warp(&left[g], t & 1, ERR_KV8_PV_WAIT) && ok;  // the piece before has left O
          ok = wait_warp(&pready[g], n & 1, ERR_KV8_PV_WAIT) && ok;
          if (ok) {
            tc_fence_after();
            // (16 states further: 8 columns of P; 16 rows of V)
#pragma unroll 4
            for (int i = 0; i < steps; ++i)
              mma_f16_ts(tmem + CR_O + g * DP, tmem + CR_S + g * 128 + 8 * i, v + i * 128, ID, i > 0 || !first);
          }
          tc_commit(&pvdone[g]);
          ++n;
        };
        const int d = c - x.c0;
        if (two || (d & 1) == 0) half(0, n0, t0, d == 0);
        if (two || (d & 1) == 1) half(1, n1, t1, d == (two ? 0 : 1));
        tc_commit(&vempty[st]);
      }
    }
  } else if (warp >= 8) {
    // ====== q of a tile, ahead; then the outputs of the tile before ======
    const int k = warp & 3;
    constexpr int LPR = DP / 8, RPW = 32 / LPR;  // lanes of a row (8 values each), rows of a warp at a time
    const int piece = lane % LPR;
    const uint32_t t_lane = static_cast<uint32_t>(32 * k) << 16;
    int qs = 0, n[2] = {0, 0}, t[2] = {0, 0};  // halves of q; up to piece y: chunks and pieces of each half
    auto bring = [&](const CrossPiece& x, int row0, int rows) {  // rows [row0, row0 + rows) of the request
      const int s = qs & 1;
      if (qs > 1) wait_warp(&qfree[s], ((qs >> 1) - 1) & 1, ERR_KV8_S_WAIT);
      uint8_t* to = sm + S::OFF_Q + s * T + (piece / 8) * SUB;
      const __nv_bfloat16* q = p.q + x.q0 * p.q_tok + int64_t(x.h) * p.group * p.q_head + piece * 8;
      constexpr int A = 8;  // reads under way
#pragma unroll 1
      for (int r0 = k * RPW + lane / LPR; r0 < CR_HALF; r0 += 4 * RPW * A) {
        uint4 w[A];
#pragma unroll
        for (int a = 0; a < A; ++a) {
          const int r = r0 + a * 4 * RPW;
          w[a] = make_uint4(0u, 0u, 0u, 0u);
          if (r < rows && piece * 8 < p.D) {
            const int i = (row0 + r) / p.group, j = row0 + r - i * p.group;
            w[a] = __ldg(reinterpret_cast<const uint4*>(q + i * p.q_tok + j * p.q_head));
            w[a].x ^= p.flip; w[a].y ^= p.flip; w[a].z ^= p.flip; w[a].w ^= p.flip;
          }
        }
#pragma unroll
        for (int a = 0; a < A; ++a) {
          const int r = r0 + a * 4 * RPW;
          if (r < CR_HALF) *reinterpret_cast<uint4*>(to + r * 128 + (((piece & 7) ^ (r & 7)) << 4)) = w[a];
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&qready[s]);
      ++qs;
    };
    // Row `row` of piece y's tile from o = f0 O0 + f1 O1, 16 columns at a time; `mine`: whether it is there.
    auto write = [&](const CrossPiece& y, int row, bool mine, bool use0, float f0, bool use1, float f1, float m, float l) {
      const int i = mine ? (y.row0 + row) / p.group : 0, j = mine ? y.row0 + row - i * p.group : 0;
      const int64_t at = (y.q0 + i) * p.q_heads + int64_t(y.h) * p.group + j;
      float* part = p.part + int64_t(y.slot) * CR_ROWS * (DP + 2);
#pragma unroll 1
      for (int w0 = 0; w0 < DP; w0 += 16) {
        float o[16], z[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = 0.f;
        if (use0) {
          tmem_ld16(tmem + t_lane + CR_O + w0, o);
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] *= f0;
        }
        if (use1) {
          tmem_ld16(tmem + t_lane + CR_O + DP + w0, z);
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = use0 ? fmaf(z[e], f1, o[e]) : z[e] * f1;
        }
        if (w0 + 16 == DP) {  // O has been read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (use0) mbar_arrive(&left[0]);
            if (use1) mbar_arrive(&left[1]);
          }
        }
        if (mine && y.whole) {
          uint32_t h[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(o[2 * e], o[2 * e + 1]);
            h[e] = *reinterpret_cast<const uint32_t*>(&v);
          }
          uint4* dst = reinterpret_cast<uint4*>(p.out + at * p.D + w0);
          if (w0 < p.D) dst[0] = make_uint4(h[0], h[1], h[2], h[3]);
          if (w0 + 8 < p.D) dst[1] = make_uint4(h[4], h[5], h[6], h[7]);
        } else if (mine) {
          float4* dst = reinterpret_cast<float4*>(part + row * DP + w0);
#pragma unroll
          for (int e = 0; e < 4; ++e) dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      }
      if (mine && !y.whole) {
        part[CR_ROWS * DP + row] = m;
        part[CR_ROWS * DP + CR_ROWS + row] = l;
      } else if (mine && p.lse) {
        p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2_F;
      }
    };
    CrossPiece x, y{};
    y.whole = -1;
    for (int pi = 0;; ++pi) {
      const bool more = next_piece(pi, x);
      if (more && x.c0 < x.cn) {
        bring(x, x.row0, min(x.rows, CR_HALF));
        if (x.rows > CR_HALF) bring(x, x.row0 + CR_HALF, x.rows - CR_HALF);
      }
      if (y.whole >= 0) {
        const bool two = y.rows > CR_HALF;
        const int r = 32 * k + lane;
        // a half's maximum and sum, once its products are done
        auto half = [&](int g) {
          const int e = (t[g] - 1) & 1;
          wait_warp(&met[e][g][k], ((t[g] - 1) >> 1) & 1, ERR_KV8_PV_WAIT);
          const float2 ml = s_ml[e][g][r];
          wait_warp(&pvdone[g], (n[g] - 1) & 1, ERR_KV8_PV_WAIT);
          tc_fence_after();
          return ml;
        };
        const int chunks = y.cn - y.c0;
        if (two && chunks > 0) {
          for (int g = 0; g < 2; ++g) {
            const float2 ml = half(g);
            const float f = !y.whole ? 1.f : ml.y == 0.f ? 0.f : 1.f / ml.y;
            write(y, g * CR_HALF + r, g * CR_HALF + r < y.rows, g == 0, f, g == 1, f, ml.y == 0.f ? -INFINITY : ml.x, ml.y);
          }
        } else if (chunks > 0) {
          const float2 a = half(0), b = chunks > 1 ? half(1) : make_float2(-INFINITY, 0.f);
          const float top = fmaxf(a.y == 0.f ? -INFINITY : a.x, b.y == 0.f ? -INFINITY : b.x);
          float f0 = a.y == 0.f ? 0.f : ex2(a.x - top), f1 = b.y == 0.f ? 0.f : ex2(b.x - top);
          const float l = a.y * f0 + b.y * f1;
          if (y.whole) {
            const float inv = l == 0.f ? 0.f : 1.f / l;
            f0 *= inv;
            f1 *= inv;
          }
          write(y, r, r < y.rows, true, f0, chunks > 1, f1, top, l);
        } else {  // no states
          write(y, r, r < y.rows, false, 0.f, false, 0.f, -INFINITY, 0.f);
          write(y, CR_HALF + r, CR_HALF + r < y.rows, false, 0.f, false, 0.f, -INFINITY, 0.f);
        }
      }
      if (!more) break;
      y = x;
      const int chunks = x.cn - x.c0, two = x.rows > CR_HALF;
      n[0] += two ? chunks : (chunks + 1) / 2;
      n[1] += two ? chunks : chunks / 2;
      t[0] += chunks > 0;
      t[1] += chunks > (two ? 0 : 1);
    }
  } else {
    // ================= softmax: half g, rows 32 k + lane of it =================
    const int g = warp >> 2, k = warp & 3, r = 32 * k + lane;
    const uint32_t t_s = tmem + (static_cast<uint32_t>(32 * k) << 16) + CR_S + g * 128;
    const uint32_t t_o = tmem + (static_cast<uint32_t>(32 * k) << 16) + CR_O + g * DP;
    const float a = p.scale2;
    int n = 0, t = 0;  // chunks and pieces of this half
    CrossPiece x;
    for (int pi = 0; next_piece(pi, x); ++pi) {
      const bool two = x.rows > CR_HALF;
      const int step = two ? 1 : 2, chunks = x.cn - x.c0;
      float m = -INFINITY, l = 0.f;
      int d = two ? 0 : g;
      if (d >= chunks) continue;
#pragma unroll 1
      for (; d < chunks; d += step, ++n) {
        const int lim = x.len - (x.c0 + d) * AT_CHUNK;
        wait_warp(&sready[g], n & 1, ERR_KV8_S_WAIT);
        tc_fence_after();
        if (lim < AT_CHUNK) mask_columns(t_s, lim);
        // 1. the row's largest score
        float top = -INFINITY;
        {
          float s[2][16];  // (a block is read while the one before is worked on)
          tmem_ld16_begin(t_s, s[0]);
          auto look = [&](int w0, float* now, float* next) {
            tmem_ld_end(now);
            if (w0 + 16 < AT_CHUNK) tmem_ld16_begin(t_s + w0 + 16, next);
            float big = fmaxf(now[0], now[1]);
#pragma unroll
            for (int e = 2; e < 16; e += 2) big = max3(big, now[e], now[e + 1]);
            top = fmaxf(top, big);
          };
#pragma unroll 1
          for (int w0 = 0; w0 < AT_CHUNK; w0 += 32) {
            look(w0, s[0], s[1]);
            look(w0 + 16, s[1], s[0]);
          }
        }
        top *= a;  // (positive)
        const bool anew = top - m > CR_RAISE || m == -INFINITY;
        if (__any_sync(FULL_MASK, anew)) {
          const float to = fmaxf(top, m), f = to == -INFINITY || l == 0.f ? 1.f : ex2(m - to);
          m = to;
          l *= f;
          if (d >= step) scale_outputs<DP>(t_o, f);  // (the products of the chunks before are done)
        }
        const float nref = m == -INFINITY ? 0.f : -m;
        const float2 a2 = make_float2(a, a), b2 = make_float2(nref, nref);
        // 2. the weights, over the scores that have been read (16 columns of pairs for 32 of S)
        float z[32];
        float2 sum[2] = {make_float2(l, 0.f), make_float2(0.f, 0.f)};
        tmem_ld32_begin(t_s, z);
#pragma unroll 1
        for (int w0 = 0; w0 < AT_CHUNK; w0 += 32) {
          uint32_t h[16];
          tmem_ld32_end(z);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 y = __ffma2_rn(make_float2(z[2 * e], z[2 * e + 1]), a2, b2);
            const float2 w = make_float2(ex2(y.x), ex2(y.y));
            sum[e & 1] = __fadd2_rn(sum[e & 1], w);
            const __nv_bfloat162 v = __floats2bfloat162_rn(w.x, w.y);
            h[e] = *reinterpret_cast<const uint32_t*>(&v);
          }
          if (w0 + 32 < AT_CHUNK) tmem_ld32_begin(t_s + w0 + 32, z);
          tmem_st8(t_s + w0 / 2, h);
          tmem_st8(t_s + w0 / 2 + 8, h + 8);
        }
        l = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pready[g]);
      }
      s_ml[t & 1][g][r] = make_float2(m, l);
      __syncwarp();
      if (lane == 0) mbar_arrive(&met[t & 1][g][k]);
      ++t;
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

// Boxes of 128 states of one head, 64 values wide; what lies behind the head dimension reads as zeros.
cudaError_t state_map(CUtensorMap* tm, const void* x, int D, int heads, int64_t total, int64_t tok, int64_t head) {
  auto fn = encode_fn();
  if (!fn) return cudaErrorInvalidValue;
  const cuuint64_t dims[3] = {cuuint64_t(D), cuuint64_t(heads), cuuint64_t(total)};
  // (a dimension of one has no stride of its own)
  const cuuint64_t strides[2] = {cuuint64_t(heads > 1 ? head : D) * 2, cuuint64_t(total > 1 ? tok : D) * 2};
  const cuuint32_t box[3] = {64, 1, AT_CHUNK}, estr[3] = {1, 1, 1};
  return fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(x), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

template <int DP>
cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, const CrossParams& p, cudaStream_t stream) {
  constexpr int smem = CrossShape<DP>::SMEM;
  const int grid = device_sm_count();
  cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void*>(cross_attention_kernel<DP>), smem);
  if (e != cudaSuccess) return e;
  cross_attention_kernel<DP><<<grid, 32 * CR_WARPS, smem, stream>>>(tk, tv, p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  PdlScope pdl(true);
  e = launch_k(kv8_join_kernel<DP, CR_ROWS, 4, 16, CrossParams>, dim3(grid, 16), dim3(128), 0, stream, p, grid);
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
  if (!why && (batch < 1 || batch > (1 << 20))) why = "1 <= batch <= 2^20";
  if (!why && (total < 1 || total > INT_MAX || total_kv < 1 || total_kv > INT_MAX - 256)) why = "rows are out of range";
  if (!why && (max_new < 1 || max_new > (1 << 24))) why = "1 <= max_new <= 2^24";
  if (!why && (kv_heads < 1 || kv_heads > 1024 || q_heads < 1 || q_heads % kv_heads || q_heads / kv_heads > 1024))
    why = "1 <= kv_heads <= 1024, q_heads is a multiple of it, at most 1024 times";
  if (!why && ((kv_heads > 1 && (k_head_stride < head_dim || v_head_stride < head_dim)) ||
               (total_kv > 1 && (k_token_stride < head_dim || v_token_stride < head_dim))))
    why = "rows of keys and values do not overlap";
  if (!why && (!out || reinterpret_cast<uintptr_t>(out) % 16)) why = "out is null or not 16-byte aligned";
  // a request's rows, and its work units, are counted in 32 bits
  if (!why && int64_t(max_new) * (q_heads / kv_heads) > INT_MAX - 256) why = "max_new * q_heads / kv_heads is too large";
  if (!why && (int64_t(max_new) * (q_heads / kv_heads) / CR_ROWS + 1) * kv_heads * ((total_kv + 127) / 128 + 8) > UINT_MAX)
    why = "max_new * q_heads * the states are too large";
  if (!why && !std::isfinite(scale)) why = "scale is not finite";
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
  const void* in[3] = {q, k, v};
  const wide in_bytes[3] = {extent(total, q_token_stride, q_heads, q_head_stride), extent(total_kv, k_token_stride, kv_heads, k_head_stride),
                            extent(total_kv, v_token_stride, kv_heads, v_head_stride)};
  bool overlap = lse && meet(out, o_bytes, lse, l_bytes);
  for (int i = 0; i < 3; ++i) overlap = overlap || meet(in[i], in_bytes[i], out, o_bytes) || (lse && meet(in[i], in_bytes[i], lse, l_bytes));
  if (overlap) return fail(LILICORR_ERR_INVALID_ARG, "lilicorr_cross_attention: out and lse overlap one another, or what is read");
  CrossParams p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_tok = q_token_stride; p.q_head = q_head_stride;
  p.total = total; p.total_kv = total_kv;
  p.q_heads = q_heads; p.group = q_heads / kv_heads; p.heads = kv_heads; p.D = head_dim;
  p.q_start = q_start; p.kv_start = kv_start; p.kv_len = kv_len;
  p.batch = batch; p.max_new = max_new;
  p.scale2 = std::max(std::fabs(scale) * LOG2E_F, FLT_MIN);  // (never 0, so that a score of infinity stays one)
  p.flip = std::signbit(scale) ? 0x80008000u : 0u;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.part = static_cast<float*>(workspace);
  CUtensorMap tk, tv;
  cudaError_t e = state_map(&tk, k, head_dim, kv_heads, total_kv, k_token_stride, k_head_stride);
  if (e == cudaSuccess) e = state_map(&tv, v, head_dim, kv_heads, total_kv, v_token_stride, v_head_stride);
  if (e != cudaSuccess) return fail(LILICORR_ERR_INVALID_ARG, "lilicorr_cross_attention: no tensor map for these strides");
  e = head_dim <= 64 ? launch<64>(tk, tv, p, static_cast<cudaStream_t>(stream)) : launch<128>(tk, tv, p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(LILICORR_ERR_CUDA, cudaGetErrorString(e));
  return LILICORR_OK;
}

}  // extern "C"
