// The cache attention for tiles of at most 16 rows (a token or a few of a sequence): the work is
// the reading of the cache, 2 D bytes a token and head against 4 D operations a row, so what
// counts is that the loads never wait.  A tensor-core tile of 128 rows would be one eighth full at
// best and its barriers cost more than the products: measured, 128 sequences of up to 8,192
// tokens, 8 key / value heads of 128, the tcgen05 kernel of kv8_attn.cu takes 267 to 270 us for 4 to
// 16 rows, and this one 197 for 4 (6.1 TB/s of the cache, 92 % of the copy rate) and 268 for 16,
// where the softmax and the widening fill the warps.
//
// Here the products are warp-level f16 products (m16n8k16) with the tokens, and the head
// dimension, as the 16 rows and 8 query rows as the columns, so that none of a tile is empty:
//     s'[16 tokens, 8 rows] = k q^T,   o'[16 of D, 8 rows] += v^T p'
// Codes are widened to f16 in registers (exact) as they come from shared memory.  The summation
// index of k q^T and the rows of v^T may be taken in any order, which lets each lane read 16
// contiguous bytes; the weights get from the layout of s' to that of p' by a transposition of
// 8 x 8 tiles.  q (bf16) is moved to f16 by a power of two of its row (exact but for values
// 2^-29 below the row's largest); weights are 2^14 of their size, rounded to f16 (2^-11 of their
// value, 2^-39 of the largest).  (Products of e4m3 values as they are would need no widening,
// but this part has them only on tcgen05: the warp-level form took 16 cycles for what two f16
// products take, and its own widening.)
//
// A fifth warp deals out the pieces of the CTA's run and keeps a ring of stages of 64 tokens
// filled by bulk copies; the four others work on them in pairs, 32 tokens a warp, with a
// running maximum and sums of their own, and are put together in order at a tile's end.
#include <algorithm>
#include <cmath>

#include "kv8_attn.cuh"

namespace lilicorr {

namespace {

constexpr int FW_WARPS = 4;
constexpr int FW_HALF = 64;             // tokens of a stage
// CTAs per SM: as many as their registers allow, since what a warp waits for is latency.  Measured
// (8 key / value heads): D = 64, 128 sequences of up to 8,192 tokens, 4 rows: 104 us with 4 and 4
// stages, 115 with 3 and 6, 154 with 2; 16 rows, half the sequences, 82 with 3, 94 with 2; D = 32,
// 16 rows, 62 with 4, 71 with 3, 127 with 6.
template <int D, int RT>
constexpr int FW_CTAS = D == 32 ? 4 : D == 64 ? (RT == 8 ? 4 : 3) : 2;
constexpr int FW_SC_RING = 16, FW_PIECES = 4;
constexpr float P_LOG2 = 14.f;          // log2 of the largest weight as it is held

template <int D, int RT>
struct FewShape {
  static constexpr int TILE = FW_HALF * D;              // bytes of a stage's keys, or values
  // An even number, so that a stage is always the same pair's: a barrier's wait tells only the
  // parity of a phase, and a pair that skipped phases could take an older one for its own.
  static constexpr int STAGES = D == 128 || (D == 64 && RT == 8) ? 4 : 6;
  static_assert(STAGES % 2 == 0);
  static constexpr int RING = STAGES * 2 * TILE;
  static constexpr int SMEM = RING + FW_WARPS * RT * (D + 4) * 4;
};

struct FewPiece {
  int64_t q0;
  int n, len, h, row0, rows;
  int h0, hn, end;  // its stages' first and one behind the last; tokens that its last row sees
  int whole, slot;  // as in kv8_attn.cu
};

// The rest of a wait that did not end at once, at most WAIT_LIMIT_CYCLES.  The first one of a CTA
// that gives up makes every later one give up soon, and the roles' loops end.
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

// d += a b for a 16 x 16 tile a and a 16 x 8 tile b.
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                      uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// An 8 x 8 tile of 16-bit values, a row's pair a lane, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t lo_f16(uint32_t w) { return e4m3x2_to_f16x2(static_cast<uint16_t>(w)); }
__device__ __forceinline__ uint32_t hi_f16(uint32_t w) { return e4m3x2_to_f16x2(static_cast<uint16_t>(w >> 16)); }
__device__ __forceinline__ uint32_t any_nan4(uint32_t w) { return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu); }

// In the products' layouts lane (g, t) = (lane / 4, lane % 4) holds the scores of tokens g and
// g + 8 of a block of 16 against rows 2t and 2t + 1 (of 8), and of o' the columns g D / 8 ..
// of the same rows.  D = head dimension, RT = rows (8 or 16).
template <int D, int RT>
__global__ void __launch_bounds__(32 * FW_WARPS + 32, FW_CTAS<D, RT>) kv8_few_kernel(const AttnParams p) {
  using S = FewShape<D, RT>;
  constexpr int KW = D / 16;  // words of a key row a lane reads = steps of 16 of k q^T
  constexpr int VW = D / 32;  // words of a value row a lane reads
  constexpr int NU = D / 16;  // tiles of o'
  constexpr int NT = RT / 8;  // groups of 8 rows
  constexpr int ST = S::STAGES;
  extern __shared__ __align__(128) uint8_t fw_smem[];
  __shared__ __align__(8) uint64_t full[ST], empty[ST], pc_full[FW_PIECES], pc_empty[FW_PIECES], met, left;
  __shared__ FewPiece s_piece[FW_PIECES];
  __shared__ PageScale s_sc[FW_SC_RING][4];  // of 16 tokens each
  __shared__ float s_m[FW_WARPS][RT], s_l[FW_WARPS][RT];
  __shared__ volatile int s_fail;
  float(*s_o)[RT][D + 4] = reinterpret_cast<float(*)[RT][D + 4]>(fw_smem + S::RING);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 2);
    }
    for (int i = 0; i < FW_PIECES; ++i) {
      mbar_init(&pc_full[i], 1);
      mbar_init(&pc_empty[i], FW_WARPS);
    }
    mbar_init(&met, FW_WARPS);
    mbar_init(&left, FW_WARPS);
    fence_mbar_init();
    s_fail = 0;
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t site) -> bool {
    return __all_sync(FULL_MASK, mbar_try_wait(bar, parity) || wait_slow(bar, parity, site, &s_fail));
  };

  if (warp == FW_WARPS) {
    // ====== the run's pieces, and their stages: lane i brings the i-th page (part) of a stage ======
    const Run run = find_run<RT>(p, blockIdx.x, gridDim.x);
    const int part_log2 = min(p.page_log2, 6), part = 1 << part_log2, parts = FW_HALF >> part_log2;
    const int bytes = part * D;
    Pieces<RT> w(p, run);
    int it = 0, pi = 0;
    bool ok_run = true;
    while (ok_run) {
      const int e = pi % FW_PIECES;
      if (pi >= FW_PIECES) ok_run = wait(&pc_empty[e], ((pi / FW_PIECES) - 1) & 1, ERR_KV8_EMPTY_WAIT);
      if (!ok_run || !w.next()) {
        if (lane == 0) {
          s_piece[e].whole = -1;
          mbar_arrive(&pc_full[e]);
        }
        break;
      }
      const int end = w.end(), h = w.ph;
      const int h0 = 2 * w.c0, hn = max(h0, min(2 * w.c1, (end + FW_HALF - 1) / FW_HALF));
      if (lane == 0) {
        s_piece[e] = FewPiece{w.psq.q0, w.psq.n, w.psq.len, h, w.ptile * RT, w.rows(), h0, hn, end, w.whole(), w.slot()};
        mbar_arrive(&pc_full[e]);
      }
      ++pi;
      const int32_t* tab = p.table + w.pb * p.table_stride;
      auto page_of = [&](int c) {
        const int tok = c * FW_HALF + lane * part;
        return lane < parts && c < hn && tok < end ? __ldg(tab + (tok >> p.page_log2)) : -2;
      };
      auto exists = [&](int i) { return i >= 0 && i < p.c.n_pages; };
      // page indices are read two stages ahead, scales one
      float ks1 = 0.f, vs1 = 1.f;
      auto read_scales = [&](int i) {
        if (!exists(i)) return;
        const int64_t ph = int64_t(i) * p.c.heads + h;
        ks1 = __ldg(p.c.ks + ph);
        vs1 = __ldg(p.c.vs + ph);
      };
      int id1 = page_of(h0), id2 = page_of(h0 + 1);
      read_scales(id1);
#pragma unroll 1
      for (int c = h0; c < hn; ++c, ++it) {
        const int st = it % ST, slot = it % FW_SC_RING;
        const int id = id1;
        const float ks = ks1, vs = vs1;
        id1 = id2;
        read_scales(id1);
        id2 = page_of(c + 2);
        const bool ok = exists(id);
        if (id != -2 && !ok) atomicOr(&g_err_kv8_attn, ERR_KV8_PAGE);
        const int64_t ph = int64_t(ok ? id : 0) * p.c.heads + h;
        const unsigned have = __ballot_sync(FULL_MASK, ok);
        if (it >= ST && !wait(&empty[st], ((it / ST) - 1) & 1, ERR_KV8_EMPTY_WAIT)) {
          ok_run = false;
          break;
        }
        if (lane < parts) {
          const PageScale sc = page_scale_of(ks, vs, ok);
          for (int n = 0; n < part / 16; ++n) s_sc[slot][lane * (part / 16) + n] = sc;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&full[st], 2u * bytes * __popc(have));
        __syncwarp();
        if (ok) {
          const int64_t off = ph * p.c.page * D + ((c * FW_HALF + lane * part) & (p.c.page - 1)) * D;
          uint8_t* dst = fw_smem + st * 2 * S::TILE + lane * bytes;
          bulk_g2s(dst, p.c.k + off, bytes, &full[st]);
          bulk_g2s(dst + S::TILE, p.c.v + off, bytes, &full[st]);
        }
      }
    }
    if (!ok_run || s_fail)  // what is in flight has to land
      for (int i = max(0, it - ST); i < it; ++i)
        mbar_wait_bounded(&full[i % ST], (i / ST) & 1, &g_err_kv8_attn, ERR_KV8_EMPTY_WAIT);
    return;
  }

  const int g = lane >> 2, t = lane & 3, pair = warp >> 1;
  int it0 = 0;
  for (int pi = 0;; ++pi) {
    const int e = pi % FW_PIECES;
    if (!wait(&pc_full[e], (pi / FW_PIECES) & 1, ERR_KV8_FULL_WAIT)) break;
    const FewPiece x = s_piece[e];
    if (x.whole < 0) break;
    __syncwarp();
    if (lane == 0) mbar_arrive(&pc_empty[e]);

    // q of row g of each 8, as f16 of the row's largest power of two; rows 2t, 2t + 1 for the softmax
    uint32_t qf[NT][KW][2];
    float f_row[2 * NT];
    int seen[2 * NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int row = x.row0 + 8 * n + g;
      const bool has = 8 * n + g < x.rows;
      const int i = has ? row / p.group : 0, j = has ? row - i * p.group : 0;
      const int sees = has ? min(x.len - x.n + i + 1, x.end) : 0;
      const __nv_bfloat16* qr = p.q + (x.q0 + i) * p.q_tok + (x.h * p.group + j) * p.q_head;
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
      const int sh = min(14 - (min(max(static_cast<int>(top >> 7), 1), 254) - 127), 120);
      const float up = __uint_as_float(static_cast<uint32_t>(127 + sh) << 23);
      const float f = p.scale2 * __uint_as_float(static_cast<uint32_t>(127 - sh) << 23);
#pragma unroll
      for (int k = 0; k < KW; ++k) {
        const __half2 a = __floats2half2_rn(__uint_as_float(raw[k].x << 16) * up,
                                            __uint_as_float(raw[k].x & 0xffff0000u) * up);
        const __half2 c = __floats2half2_rn(__uint_as_float(raw[k].y << 16) * up,
                                            __uint_as_float(raw[k].y & 0xffff0000u) * up);
        qf[n][k][0] = *reinterpret_cast<const uint32_t*>(&a);
        qf[n][k][1] = *reinterpret_cast<const uint32_t*>(&c);
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        f_row[2 * n + r] = __shfl_sync(FULL_MASK, f, 4 * (2 * t + r));
        seen[2 * n + r] = __shfl_sync(FULL_MASK, sees, 4 * (2 * t + r));
      }
    }

    float m[2 * NT], l[2 * NT], o[NT][NU][4];
#pragma unroll
    for (int r = 0; r < 2 * NT; ++r) { m[r] = -INFINITY; l[r] = 0.f; }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < NU; ++c) o[n][c][0] = o[n][c][1] = o[n][c][2] = o[n][c][3] = 0.f;

    const int stages = x.hn - x.h0;
#pragma unroll 1
    for (int d = (it0 ^ pair) & 1; d < stages; d += 2) {
      const int it = it0 + d, st = it % ST, slot = it % FW_SC_RING;
      const bool landed = wait(&full[st], (it / ST) & 1, ERR_KV8_FULL_WAIT);
      const int tok0 = (x.h0 + d) * FW_HALF + (warp & 1) * 32;
      if (landed && tok0 < x.end) {
        const PageScale sc[2] = {s_sc[slot][(warp & 1) * 2], s_sc[slot][(warp & 1) * 2 + 1]};
        const uint8_t* kt = fw_smem + st * 2 * S::TILE + (warp & 1) * 32 * D;
        const uint8_t* vt = kt + S::TILE;
        // ---- s' of two blocks of 16 tokens
        float s[NT][2][4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t kw[2][KW];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint8_t* kr = kt + (16 * k + 8 * j + g) * D;
            if constexpr (D == 128) {
              // 128-byte rows share banks: odd rows take the other half first
              const int sw = (g & 1) * 64;
              const uint4 a = *reinterpret_cast<const uint4*>(kr + t * 16 + sw);
              const uint4 b = *reinterpret_cast<const uint4*>(kr + t * 16 + 64 - sw);
              const uint4 lo = sw ? b : a, hi = sw ? a : b;
              kw[j][0] = lo.x; kw[j][1] = lo.y; kw[j][2] = lo.z; kw[j][3] = lo.w;
              kw[j][4] = hi.x; kw[j][5] = hi.y; kw[j][6] = hi.z; kw[j][7] = hi.w;
            } else if constexpr (D == 64) {
              const uint4 a = *reinterpret_cast<const uint4*>(kr + t * 16);
              kw[j][0] = a.x; kw[j][1] = a.y; kw[j][2] = a.z; kw[j][3] = a.w;
            } else {
              const uint2 a = *reinterpret_cast<const uint2*>(kr + t * 8);
              kw[j][0] = a.x; kw[j][1] = a.y;
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) s[n][k][0] = s[n][k][1] = s[n][k][2] = s[n][k][3] = 0.f;
#pragma unroll
          for (int i = 0; i < KW; ++i) {
            const uint32_t a0 = lo_f16(kw[0][i]), a1 = lo_f16(kw[1][i]), a2 = hi_f16(kw[0][i]), a3 = hi_f16(kw[1][i]);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16(s[n][k], a0, a1, a2, a3, qf[n][i][0], qf[n][i][1]);
          }
        }
        // ---- softmax
        const bool masks = tok0 + 32 > x.len - x.n || !sc[0].ok || !sc[1].ok;
        uint32_t pf[NT][2][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float y[2][4];  // of row 2t + r: tokens g, g + 8 of either block
#pragma unroll
          for (int r = 0; r < 2; ++r) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float f = f_row[2 * n + r] * sc[k].k;
              y[r][2 * k] = fmaf(s[n][k][r], f, sc[k].log2_v);
              y[r][2 * k + 1] = fmaf(s[n][k][2 + r], f, sc[k].log2_v);
            }
            if (masks) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (tok0 + 8 * i + g >= seen[2 * n + r] || !sc[i >> 1].ok) y[r][i] = -INFINITY;
            }
          }
          float mx[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) mx[r] = fmaxf(fmaxf(y[r][0], y[r][1]), fmaxf(y[r][2], y[r][3]));
#pragma unroll
          for (int q = 4; q < 32; q <<= 1) {
            mx[0] = fmaxf(mx[0], __shfl_xor_sync(FULL_MASK, mx[0], q));
            mx[1] = fmaxf(mx[1], __shfl_xor_sync(FULL_MASK, mx[1], q));
          }
          float* mr = m + 2 * n;
          float* lr = l + 2 * n;
          if (mx[0] > mr[0] || mx[1] > mr[1]) {
            const float n0 = fmaxf(mr[0], mx[0]), n1 = fmaxf(mr[1], mx[1]);
            const float f0 = n0 == -INFINITY ? 1.f : ex2(mr[0] - n0), f1 = n1 == -INFINITY ? 1.f : ex2(mr[1] - n1);
            lr[0] *= f0;
            lr[1] *= f1;
#pragma unroll
            for (int c = 0; c < NU; ++c) { o[n][c][0] *= f0; o[n][c][1] *= f1; o[n][c][2] *= f0; o[n][c][3] *= f1; }
            mr[0] = n0;
            mr[1] = n1;
          }
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float base = mr[r] == -INFINITY ? 0.f : P_LOG2 - mr[r];
#pragma unroll
            for (int i = 0; i < 4; ++i) y[r][i] = ex2(y[r][i] + base);
            lr[r] = fmaf(y[r][0] + y[r][1], sc[0].inv_v, lr[r]);
            lr[r] = fmaf(y[r][2] + y[r][3], sc[1].inv_v, lr[r]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(y[0][i], y[1][i]);
            pf[n][i >> 1][i & 1] = transposed(*reinterpret_cast<const uint32_t*>(&h));
          }
        }
        // ---- o' += v^T p', by blocks of 16 tokens
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t vw[4][VW];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint8_t* vr = vt + (16 * k + 2 * t + (j & 1) + 8 * (j >> 1)) * D + g * (D / 8);
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
          // Tokens that some row of the tile does not see (the causal edge, what lies behind the
          // last token, and pages that were not loaded): 0 * NaN is NaN, so their values take part
          // without NaN, and rows that do see a NaN get it afterwards.
          bool fix = false;
          if (masks) {
            uint32_t nan = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const bool in = tok0 + 16 * k + 2 * t + (j & 1) + 8 * (j >> 1) < x.end && sc[k].ok;
#pragma unroll
              for (int i = 0; i < VW; ++i) {
                if (!in) vw[j][i] = 0u;
                const uint32_t bad = any_nan4(vw[j][i]);
                nan |= bad;
                vw[j][i] &= ~bad;
              }
            }
            fix = __any_sync(FULL_MASK, nan != 0);
          }
#pragma unroll
          for (int i = 0; i < VW; ++i) {
            const uint32_t a = __byte_perm(vw[0][i], vw[1][i], 0x5140), b = __byte_perm(vw[2][i], vw[3][i], 0x5140);
            const uint32_t c = __byte_perm(vw[0][i], vw[1][i], 0x7362), e2 = __byte_perm(vw[2][i], vw[3][i], 0x7362);
            const uint32_t a0 = lo_f16(a), a1 = hi_f16(a), a2 = lo_f16(b), a3 = hi_f16(b);
            const uint32_t c0 = lo_f16(c), c1 = hi_f16(c), c2 = lo_f16(e2), c3 = hi_f16(e2);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma16(o[n][2 * i], a0, a1, a2, a3, pf[n][k][0], pf[n][k][1]);
              mma16(o[n][2 * i + 1], c0, c1, c2, c3, pf[n][k][0], pf[n][k][1]);
            }
          }
          if (fix) {
#pragma unroll 1
            for (int tk = 0; tk < 16 && tok0 + 16 * k + tk < x.end; ++tk)
#pragma unroll
              for (int c = 0; c < NU; ++c)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                  if ((vt[(16 * k + tk) * D + g * (D / 8) + 2 * c + i] & 0x7f) == 0x7f)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                      for (int r = 0; r < 2; ++r)
                        if (tok0 + 16 * k + tk < seen[2 * n + r]) o[n][c][2 * i + r] = NAN;
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }

    // ---- the warps together: each scales its products to the row's largest maximum; in order
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float sum = l[2 * n + r];
#pragma unroll
        for (int q = 4; q < 32; q <<= 1) sum += __shfl_xor_sync(FULL_MASK, sum, q);
        const int row = 8 * n + 2 * t + r;
        if (g == 0) { s_m[warp][row] = m[2 * n + r]; s_l[warp][row] = sum; }
        float* dst = &s_o[warp][row][g * (D / 8)];
#pragma unroll
        for (int c = 0; c < NU; c += 2)
          *reinterpret_cast<float4*>(dst + 2 * c) = make_float4(o[n][c][r], o[n][c][2 + r], o[n][c + 1][r], o[n][c + 1][2 + r]);
      }
    __syncwarp();
    if (lane == 0) mbar_arrive(&met);
    wait(&met, pi & 1, ERR_KV8_PV_WAIT);
    constexpr int N = D / 32;  // columns a lane takes of a row
#pragma unroll 1
    for (int r = warp; r < x.rows; r += FW_WARPS) {
      float mx = -INFINITY, sum = 0.f, y[N];
#pragma unroll
      for (int w = 0; w < FW_WARPS; ++w) mx = fmaxf(mx, s_m[w][r]);
      const float base = mx == -INFINITY ? 0.f : mx;
#pragma unroll
      for (int n = 0; n < N; ++n) y[n] = 0.f;
#pragma unroll
      for (int w = 0; w < FW_WARPS; ++w) {
        const float back = ex2(s_m[w][r] - base);
        sum = fmaf(s_l[w][r], back, sum);
#pragma unroll
        for (int n = 0; n < N; ++n) y[n] = fmaf(s_o[w][r][lane * N + n], back, y[n]);
      }
      mx -= P_LOG2;  // the weights were 2^14 of their size
      if (x.whole) {
        const int row = x.row0 + r, i = row / p.group;
        store_row<N>(p, (x.q0 + i) * p.q_heads + x.h * p.group + (row - i * p.group), D, lane, y, sum, mx);
      } else {
        float* part = p.part + int64_t(x.slot) * RT * (D + 2);
#pragma unroll
        for (int n = 0; n < N; ++n) part[r * D + lane * N + n] = y[n];
        if (lane == 0) {
          part[RT * D + r] = mx;
          part[RT * D + RT + r] = sum;
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&left);
    wait(&left, pi & 1, ERR_KV8_PV_WAIT);
    it0 += stages;
  }
}

template <int D, int RT>
cudaError_t launch(const AttnParams& prm, int runs, cudaStream_t stream) {
  constexpr int smem = FewShape<D, RT>::SMEM;
  cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void*>(kv8_few_kernel<D, RT>), smem);
  if (e != cudaSuccess) return e;
  kv8_few_kernel<D, RT><<<runs, 32 * FW_WARPS + 32, smem, stream>>>(prm);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  PdlScope pdl(true);
  e = launch_k(kv8_join_kernel<D, RT, RT, 1>, dim3(runs), dim3(32 * RT), 0, stream, prm, runs, RT);
  if (e == cudaSuccess) note_launch(2);
  return e;
}

}  // namespace

#define LC_FEW(f) \
  (D == 128 ? (rows == 8 ? f(128, 8) : f(128, 16)) : D == 64 ? (rows == 8 ? f(64, 8) : f(64, 16)) : rows == 8 ? f(32, 8) : f(32, 16))
int kv8_few_runs(int rows, int D) {
#define LC_CTAS(DD, RT) FW_CTAS<DD, RT>
  return LC_FEW(LC_CTAS) * device_sm_count();
#undef LC_CTAS
}

cudaError_t kv8_few_launch(const AttnParams& p, int D, int rows, cudaStream_t stream) {
  const int runs = kv8_few_runs(rows, D);
#define LC_LAUNCH(DD, RT) launch<DD, RT>(p, runs, stream)
  return LC_FEW(LC_LAUNCH);
#undef LC_LAUNCH
}
#undef LC_FEW

cudaError_t kv8_few_read_device_error(uint32_t* code) {
  uint32_t v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_err_kv8_attn, sizeof(v));
  if (e != cudaSuccess) return e;
  if (v) e = cudaMemcpyToSymbol(g_err_kv8_attn, &zero, sizeof(zero));
  *code |= v;
  return e;
}

}  // namespace lilicorr
