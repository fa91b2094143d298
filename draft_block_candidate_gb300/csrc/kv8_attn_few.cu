// The cache attention for tiles of at most 16 rows (a token or a few of a sequence): the work is
// the reading of the cache, 2 D bytes a token and head against 4 D operations a row, so what
// counts is that the loads never wait.  A tensor-core tile of 128 rows would be one eighth full at
// best and its barriers cost more than the products: measured, the tcgen05 kernel of
// kv8_attn.cu took 400 us where this one takes 200 (128 sequences of up to 8,192 tokens, 32
// query heads on 8, head dim 128).
//
// Here the products are warp-level e4m3 products (m16n8k32, 4.2 cycles each on an SM quarter,
// four times the f16 rate per value), which take the cache's codes as they lie in shared memory:
//     s = (q_hi + q_lo) . k      q split into two e4m3 values, as in kv8_attn.cu
//     o += (p1 + p2 + p3) v      p in units of 2^-14 of the row's largest, as three e5m2 values
//                                (3 significant bits each: off by at most 2^-9 of its value,
//                                2^-31 of the largest)
// so that no code is widened; V's bytes are put into the order of the instruction, four tokens
// of one column to a register, by byte permutations.  The summation index of q . k and the output
// columns of p v may be taken in any order, which lets each lane read 16 contiguous bytes.
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
constexpr int FW_CTAS = 2;              // per SM
constexpr int FW_SC_RING = 16, FW_PIECES = 4;
constexpr float P_LOG2 = 14.f;          // log2 of the largest weight's value

template <int D, int RT>
struct FewShape {
  static constexpr int TILE = FW_HALF * D;              // bytes of a stage's keys, or values
  static constexpr int STAGES = D == 128 ? (RT == 8 ? 5 : 4) : 6;
  static constexpr int RING = STAGES * 2 * TILE;
  static constexpr int SMEM = RING + FW_WARPS * RT * (D + 4) * 4;
};

struct FewPiece {
  int64_t q0;
  int n, len, h, row0, rows;
  int h0, hn, end;  // its stages' first and one behind the last; tokens that its last row sees
  int whole, slot;  // as in kv8_attn.cu; chunks
};

// d += a b for a 16 x 32 tile a and a 32 x 8 tile b of 8-bit values; with NR = 1 the upper 8 rows
// of a are zero, and their part of d is neither read nor kept.
template <int NR>
__device__ __forceinline__ void mma_k(float (&d)[2 * NR], const uint32_t (&a)[2 * NR], uint32_t b0, uint32_t b1) {
  if constexpr (NR == 1) {
    float z0, z1;
    asm(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%6,%5,%6}, {%7,%8}, "
        "{%0,%1,%9,%9};"
        : "+f"(d[0]), "+f"(d[1]), "=f"(z0), "=f"(z1)
        : "r"(a[0]), "r"(a[1]), "r"(0u), "r"(b0), "r"(b1), "f"(0.f));
  } else {
    asm(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[2]), "r"(a[1]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}
template <int NR>
__device__ __forceinline__ void mma_v(float (&d)[2 * NR], const uint32_t (&a)[2 * NR], uint32_t b0, uint32_t b1) {
  if constexpr (NR == 1) {
    float z0, z1;
    asm(
        "mma.sync.aligned.m16n8k32.row.col.f32.e5m2.e4m3.f32 {%0,%1,%2,%3}, {%4,%6,%5,%6}, {%7,%8}, "
        "{%0,%1,%9,%9};"
        : "+f"(d[0]), "+f"(d[1]), "=f"(z0), "=f"(z1)
        : "r"(a[0]), "r"(a[1]), "r"(0u), "r"(b0), "r"(b1), "f"(0.f));
  } else {
    asm(
        "mma.sync.aligned.m16n8k32.row.col.f32.e5m2.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[2]), "r"(a[1]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}
__device__ __forceinline__ uint16_t f16x2_to_e5m2x2(uint32_t x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t e5m2x2_to_f16x2(uint16_t x) {
  uint32_t r;
  asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(r) : "h"(x));
  return r;
}
__device__ __forceinline__ uint32_t any_nan4(uint32_t w) { return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu); }

// Rows of a tile in the matrix instruction's accumulator layout: lane (g, t) = (lane / 4, lane % 4)
// holds rows g and g + 8.  D = head dimension, RT = rows (8 or 16: with 8 the upper half of
// every product is zero and takes no registers).
template <int D, int RT>
__global__ void __launch_bounds__(32 * FW_WARPS + 32, FW_CTAS) kv8_few_kernel(const AttnParams p) {
  using S = FewShape<D, RT>;
  constexpr int KW = D / 16;  // words of a key row a lane reads
  constexpr int KS = D / 32;  // steps of 32 of q . k
  constexpr int VW = D / 32;  // words of a value row a lane reads
  constexpr int NU = D / 8;   // output column groups
  constexpr int NR = RT / 8;  // rows a lane holds
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
    int64_t b = run.b, u = run.u;
    SeqUnits sq{};
    int tile = 0, h = 0, c0 = 0;
    if (u < run.u_end) {
      sq = seq_units<RT>(p, b);
      const uint32_t in = static_cast<uint32_t>(u - run.first);  // a sequence's units fit 32 bits (host)
      const uint32_t item = in / sq.chunks;
      c0 = static_cast<int>(in - item * sq.chunks);
      h = item / sq.tiles;
      tile = item - h * sq.tiles;
    }
    int it = 0, pi = 0;
    bool ok_run = true;
    while (ok_run) {
      const int e = pi % FW_PIECES;
      if (pi >= FW_PIECES) ok_run = wait(&pc_empty[e], ((pi / FW_PIECES) - 1) & 1, ERR_KV8_EMPTY_WAIT);
      if (!ok_run || u >= run.u_end) {
        if (lane == 0) {
          s_piece[e].whole = -1;
          mbar_arrive(&pc_full[e]);
        }
        break;
      }
      while (sq.units == 0) sq = seq_units<RT>(p, ++b);  // sequences without new tokens
      const int c1 = static_cast<int>(min(int64_t(sq.chunks), c0 + (run.u_end - u)));
      const int rows = min(RT, sq.n * p.group - tile * RT);
      const int end = max(0, min(sq.len, sq.len - sq.n + (tile * RT + rows - 1) / p.group + 1));
      const int h0 = 2 * c0, hn = max(h0, min(2 * c1, (end + FW_HALF - 1) / FW_HALF));
      if (lane == 0) {
        s_piece[e] = FewPiece{sq.q0, sq.n, sq.len, h, tile * RT, rows, h0, hn, end,
                              c0 == 0 && c1 == sq.chunks ? 1 : 0, 2 * static_cast<int>(blockIdx.x) + (pi > 0)};
        mbar_arrive(&pc_full[e]);
      }
      ++pi;
      const int32_t* tab = p.table + b * p.table_stride;
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
          const PageScale sc{ks, log2f(vs), 1.f / vs, ok ? 1 : 0};
          for (int w = 0; w < part / 16; ++w) s_sc[slot][lane * (part / 16) + w] = sc;
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
      // on to the next tile
      u += c1 - c0;
      c0 = c1;
      if (c0 == sq.chunks) {
        c0 = 0;
        if (++tile == sq.tiles) {
          tile = 0;
          if (++h == p.c.heads) {
            h = 0;
            if (u < run.u_end) sq = seq_units<RT>(p, ++b);
          }
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

    // q of this lane's rows, hi and lo, with the row's largest in [128, 256)
    uint32_t qh[KS][2 * NR], ql[KS][2 * NR];
    float f_row[NR];
    int seen[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int row = x.row0 + g + 8 * r;
      const bool has = g + 8 * r < x.rows;
      const int i = has ? row / p.group : 0, j = has ? row - i * p.group : 0;
      seen[r] = has ? min(x.len - x.n + i + 1, x.end) : 0;
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
      const int sh = min(7 - (min(max(static_cast<int>(top >> 7), 1), 254) - 127), 120);
      const float up = __uint_as_float(static_cast<uint32_t>(127 + sh) << 23);
      f_row[r] = p.scale2 * __uint_as_float(static_cast<uint32_t>(127 - sh) << 23);
#pragma unroll
      for (int k = 0; k < KW; ++k) {
        const float y[4] = {__uint_as_float(raw[k].x << 16) * up, __uint_as_float(raw[k].x & 0xffff0000u) * up,
                            __uint_as_float(raw[k].y << 16) * up, __uint_as_float(raw[k].y & 0xffff0000u) * up};
        uint32_t hi = 0, lo = 0;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const uint16_t h2 = f32x2_to_e4m3x2(y[2 * n], y[2 * n + 1]);
          const uint32_t b2 = e4m3x2_to_f16x2(h2);
          const float2 f2 = __half22float2(*reinterpret_cast<const __half2*>(&b2));
          hi |= uint32_t(h2) << (16 * n);
          // a row with an infinity keeps it as NaN: 448 would be a value like any other
          const float l0 = y[2 * n] - f2.x, l1 = y[2 * n + 1] - f2.y;
          lo |= uint32_t(f32x2_to_e4m3x2(isinf(l0) ? NAN : l0, isinf(l1) ? NAN : l1)) << (16 * n);
        }
        qh[k / 2][2 * r + (k & 1)] = hi;
        ql[k / 2][2 * r + (k & 1)] = lo;
      }
    }

    float m[NR], l[NR], o[NU][2 * NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) { m[r] = -INFINITY; l[r] = 0.f; }
#pragma unroll
    for (int n = 0; n < NU; ++n)
#pragma unroll
      for (int k = 0; k < 2 * NR; ++k) o[n][k] = 0.f;

    const int stages = x.hn - x.h0;
#pragma unroll 1
    for (int d = (it0 ^ pair) & 1; d < stages; d += 2) {
      const int it = it0 + d, st = it % ST, slot = it % FW_SC_RING;
      const bool landed = wait(&full[st], (it / ST) & 1, ERR_KV8_FULL_WAIT);
      const int tok0 = (x.h0 + d) * FW_HALF + (warp & 1) * 32;
      const PageScale sc[2] = {s_sc[slot][(warp & 1) * 2], s_sc[slot][(warp & 1) * 2 + 1]};
      if (landed && tok0 < x.end) {
        const uint8_t* kt = fw_smem + st * 2 * S::TILE + (warp & 1) * 32 * D;
        const uint8_t* vt = kt + S::TILE;
        // ---- s of 32 tokens, in four groups of 8
        float s[4][2 * NR];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
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
          for (int k = 0; k < 2 * NR; ++k) s[j][k] = 0.f;
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            mma_k<NR>(s[j], qh[k], kw[2 * k], kw[2 * k + 1]);
            mma_k<NR>(s[j], ql[k], kw[2 * k], kw[2 * k + 1]);
          }
        }
        // ---- softmax, and the weights as three e5m2 values
        uint32_t p1[2 * NR], p2[2 * NR], p3[2 * NR];
        const bool masks = tok0 + 32 > x.len - x.n || !sc[0].ok || !sc[1].ok;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          float y[8];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float f = f_row[r] * sc[k].k;
#pragma unroll
            for (int i = 0; i < 4; ++i) y[4 * k + i] = fmaf(s[2 * k + (i >> 1)][2 * r + (i & 1)], f, sc[k].log2_v);
          }
          if (masks) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (tok0 + 8 * (i >> 1) + 2 * t + (i & 1) >= seen[r] || !sc[i >> 2].ok) y[i] = -INFINITY;
          }
          float mx = fmaxf(fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])), fmaxf(fmaxf(y[4], y[5]), fmaxf(y[6], y[7])));
          mx = fmaxf(mx, __shfl_xor_sync(FULL_MASK, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(FULL_MASK, mx, 2));
          const float nm = fmaxf(m[r], mx);
          if (nm != m[r]) {  // uniform over the four lanes of the row
            const float back = ex2(m[r] - nm);
            l[r] *= back;
#pragma unroll
            for (int n = 0; n < NU; ++n) { o[n][2 * r] *= back; o[n][2 * r + 1] *= back; }
            m[r] = nm;
          }
          const float base = nm == -INFINITY ? 0.f : P_LOG2 - nm;
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = ex2(y[i] + base);
          l[r] = fmaf((y[0] + y[1]) + (y[2] + y[3]), sc[0].inv_v, l[r]);
          l[r] = fmaf((y[4] + y[5]) + (y[6] + y[7]), sc[1].inv_v, l[r]);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t w[3] = {0u, 0u, 0u};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              __half2 rest = __floats2half2_rn(y[4 * k + 2 * i], y[4 * k + 2 * i + 1]);
#pragma unroll
              for (int n = 0; n < 3; ++n) {
                const uint16_t c2 = f16x2_to_e5m2x2(*reinterpret_cast<const uint32_t*>(&rest));
                w[n] |= uint32_t(c2) << (16 * i);
                if (n < 2) {
                  const uint32_t b2 = e5m2x2_to_f16x2(c2);
                  rest = __hsub2(rest, *reinterpret_cast<const __half2*>(&b2));
                }
              }
            }
            p1[2 * r + k] = w[0];
            p2[2 * r + k] = w[1];
            p3[2 * r + k] = w[2];
          }
        }
        // ---- o += p v, V in two halves of 16 tokens (the first and the second register of b)
        uint32_t vw[8][VW];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
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
        // Tokens that some row of the tile does not see (the causal edge, what lies behind the last
        // token, and pages that were not loaded): 0 * NaN is NaN, so their values take part
        // without NaN, and rows that do see a NaN get it afterwards.
        bool fix = false;
        if (masks) {
          uint32_t nan = 0;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const bool in = tok0 + 2 * t + (j & 1) + 8 * (j >> 1) < x.end && sc[j >> 2].ok;
#pragma unroll
            for (int k = 0; k < VW; ++k) {
              if (!in) vw[j][k] = 0u;
              const uint32_t bad = any_nan4(vw[j][k]);
              nan |= bad;
              vw[j][k] &= ~bad;
            }
          }
          fix = __any_sync(FULL_MASK, nan != 0);
        }
#pragma unroll
        for (int k = 0; k < VW; ++k) {
          uint32_t b[2][4];  // of columns 4k .. 4k + 3 of this lane's, four tokens a register
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint32_t a0 = __byte_perm(vw[4 * q][k], vw[4 * q + 1][k], 0x5140);
            const uint32_t a1 = __byte_perm(vw[4 * q + 2][k], vw[4 * q + 3][k], 0x5140);
            const uint32_t c0 = __byte_perm(vw[4 * q][k], vw[4 * q + 1][k], 0x7362);
            const uint32_t c1 = __byte_perm(vw[4 * q + 2][k], vw[4 * q + 3][k], 0x7362);
            b[q][0] = __byte_perm(a0, a1, 0x5410);
            b[q][1] = __byte_perm(a0, a1, 0x7632);
            b[q][2] = __byte_perm(c0, c1, 0x5410);
            b[q][3] = __byte_perm(c0, c1, 0x7632);
          }
#pragma unroll
          for (int n = 0; n < 4; ++n) mma_v<NR>(o[4 * k + n], p1, b[0][n], b[1][n]);
#pragma unroll
          for (int n = 0; n < 4; ++n) mma_v<NR>(o[4 * k + n], p2, b[0][n], b[1][n]);
#pragma unroll
          for (int n = 0; n < 4; ++n) mma_v<NR>(o[4 * k + n], p3, b[0][n], b[1][n]);
        }
        if (fix) {
#pragma unroll 1
          for (int tk = 0; tk < 32 && tok0 + tk < x.end; ++tk) {
            if (!sc[tk >> 4].ok) continue;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int c = 0; c < NU; ++c)
                if ((vt[tk * D + (2 * t + n) * NU + c] & 0x7f) == 0x7f)
#pragma unroll
                  for (int r = 0; r < NR; ++r)
                    if (tok0 + tk < seen[r]) o[c][2 * r + n] = NAN;
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }

    // ---- the warps together: each scales its products to the row's largest maximum; in order
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      l[r] += __shfl_xor_sync(FULL_MASK, l[r], 1);
      l[r] += __shfl_xor_sync(FULL_MASK, l[r], 2);
      if (t == 0) { s_m[warp][g + 8 * r] = m[r]; s_l[warp][g + 8 * r] = l[r]; }
    }
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float* dst = &s_o[warp][g + 8 * r][(2 * t + k) * NU];
#pragma unroll
        for (int n = 0; n < NU; n += 4)
          *reinterpret_cast<float4*>(dst + n) = make_float4(o[n][2 * r + k], o[n + 1][2 * r + k],
                                                            o[n + 2][2 * r + k], o[n + 3][2 * r + k]);
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
  e = launch_k(kv8_join_kernel<D, RT>, dim3(runs, RT / JOIN_ROWS<RT>), dim3(32 * JOIN_ROWS<RT>), 0, stream, prm, runs);
  if (e == cudaSuccess) note_launch(2);
  return e;
}

}  // namespace

int kv8_few_runs(int) { return FW_CTAS * device_sm_count(); }

cudaError_t kv8_few_launch(const AttnParams& p, int D, int rows, cudaStream_t stream) {
  const int runs = kv8_few_runs(rows);
#define LC_RT(DD) (rows == 8 ? launch<DD, 8>(p, runs, stream) : launch<DD, 16>(p, runs, stream))
  return D == 128 ? LC_RT(128) : D == 64 ? LC_RT(64) : LC_RT(32);
#undef LC_RT
}

cudaError_t kv8_few_read_device_error(uint32_t* code) {
  uint32_t v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_err_kv8_attn, sizeof(v));
  if (e != cudaSuccess) return e;
  if (v) e = cudaMemcpyToSymbol(g_err_kv8_attn, &zero, sizeof(zero));
  *code |= v;
  return e;
}

}  // namespace lilicorr
