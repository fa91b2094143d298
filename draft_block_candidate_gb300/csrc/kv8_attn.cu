// Attention of each sequence's new tokens over the 8-bit cache, for more than 16 query rows to a
// (sequence, key / value head); fewer go to kv8_attn_few.cu.
//
// For new token i of a sequence's n, and query head j of the group that shares a key / value
// head:  o = softmax_t(scale q . k_t) v_t  over the cached tokens t < len - n + i + 1.
//
// The n * group rows of a (sequence, key / value head) are taken in tiles of 128; a work unit is
// one tile against one chunk of 128 cached tokens.  The units of a call, laid out by (sequence,
// head, tile, chunk), are dealt in equal contiguous runs to one CTA per SM, so that ragged
// lengths, and few rows over a long axis, load the SMs alike.  A CTA that holds a part of a
// tile's chunks leaves its maxima, sums and products in the workspace, and a second kernel joins
// the parts in order: no atomics, the same bits every time.
//
// Per chunk, on the tensor cores, rows = the tile's query rows:
//     S[rows, 128 tokens] = Q K^T    kind::f8f6f4: K as it lies in the cache, q as the sum of
//                                    two e4m3 values (two products into one accumulator)
//     O[rows, D]         += P V      kind::f16: P from tensor memory, V widened from e4m3 (exact)
// Warps: one deals out the pieces of the CTA's run and brings their chunks (K through a swizzled
// tensor map, V by plain bulk copies) into a ring for each; one issues the S products and one the
// O products; four split the next tile's q and write the outputs of the one before; four widen V;
// and two groups of four take the softmax, a thread a row.  The groups take turns at the chunks:
// one looks for a chunk's maxima while the other forms the weights of the chunk before, and three
// buffers of S (which P then takes) let the products run ahead.  Maxima and O are the groups' in
// common, sums their own: a group decides on a chunk's maxima after the other has on the chunk
// before.
//
// A row's maximum m moves only where a score passes it by more than 2^6, and only then is O scaled
// in tensor memory, by the warp that owns its lanes.  Weights are 2^9 of their size beside m's: at
// most 2^15, inside f16, and in its normal range down to 2^-23 of the weight of m, so that what many
// tokens beside a heavy one hold together is not lost: 131,072 of them lose 2^-17 of that weight
// at most.  (64 sequences of 16 new tokens, a call: 101.4 us; m moving at 2^4 and weights at 2^11,
// 105.9; 2^8 and 2^7, 100.2; 2^14 and their own size, where the same tokens lose up to 2^-8, 98.1.)
// The page's key scale multiplies the scores; the logarithm of its value scale is added to them, so
// that p' = scale_v exp(s - m) is what the second product takes, and the sums take p' / scale_v.
//
// Roundings below f32: q (bf16) is moved by a power of two of its row to at most 256 and split
// into hi + lo, exactly but for values 2^-9 below the row's largest, which are off by at most
// 2^-17 of it; p' is rounded to f16 (2^-11 of its value, 2^-34 of the weight of m below 2^-23);
// out is rounded to bf16.
//
// Bound: neither memory nor the tensor cores (64 sequences of 16 new tokens over up to 4,096
// cached ones, 64 query and 8 key / value heads of 128: 99.9 us, 94 of them this kernel's; the
// cache's bytes take 50.6 us at 6.7 TB/s, the products 40.5) but the instructions of the softmax
// and the widening, some 5,300 of a warp to a chunk, which four schedulers issue at half their
// rate (2.2 of 4), the first tile's q (12,000 cycles before the first product), and what a tile's change
// leaves idle.  The 19 warps run seven loops at once and share an instruction cache, where a miss
// takes some 300 cycles: the loops are kept small, and what runs once a tile or less is rolled or
// out of line.  That, the split of q by warps of its own, K and V in rings of their own, one O for
// both groups and a third buffer of S took the call from 152 to 114 us, the outputs in those warps
// from 106 to 102.  Weights are formed 32 columns of S at a time (head dimension 32: 348 us with
// 16, 335 with 32; 128: no difference), maxima 16; more columns unrolled, a block kept in registers
// for both passes, or a third softmax group (head dimension 32: 356 us) measured slower.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cfloat>
#include <cmath>

#include "kv8_attn.cuh"

namespace lilicorr {

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
// (products and commits are called by a whole warp and issued by one elected lane: with the
// warp together the compiler keeps their operands in uniform registers, where an issue by a
// single lane took 80 cycles each)
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
      : "memory");
}
// A from tensor memory (packed f16 pairs, one row a lane), B from shared memory.
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
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
// The same in two steps: what is read may be used after tmem_ld_end of it, which ends all reads
// of the warp.
__device__ __forceinline__ void tmem_ld16_begin(uint32_t t, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
        "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
        "=f"(v[14]), "=f"(v[15])
      : "r"(t));
}
__device__ __forceinline__ void tmem_ld_end(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]),
                 "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]),
                 "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_ld32_begin(uint32_t t, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
        "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
        "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]),
        "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]),
        "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(t));
}
__device__ __forceinline__ void tmem_ld32_end(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]),
                 "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]),
                 "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]),
                 "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]),
                 "+f"(v[26]), "+f"(v[27]), "+f"(v[28])
               :
               : "memory");
  asm volatile("" : "+f"(v[29]), "+f"(v[30]), "+f"(v[31]));
}
// Whether a phase has ended; waits for it up to a microsecond or so.  A wait takes at most
// WAIT_TRIES of them, about a second.
constexpr uint32_t WAIT_TRIES = 1u << 20;
__device__ __forceinline__ bool try_wait_us(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity), "r"(1000u)
      : "memory");
  return ok != 0;
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
__device__ __forceinline__ void tmem_st8(uint32_t t, const uint32_t* v) {  // (not waited for)
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(t), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// Shared-memory tiles of rows of 32, 64 or 128 bytes (wider ones are several tiles of 128), in
// the hardware's swizzle for that row width: 16-byte piece c of row r lies at piece
// c ^ (bits of r).  Rows in groups of 8.
template <int BYTES>
__device__ __forceinline__ int swz(int r) {
  return BYTES == 128 ? r & 7 : BYTES == 64 ? (r >> 1) & 3 : (r >> 2) & 1;
}
// Its matrix descriptor.  Row groups are 8 * BYTES apart; `next` is the distance to the next
// tile of an operand whose rows are the summed index.
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

__device__ __forceinline__ uint16_t f16x2_to_e4m3x2(uint32_t x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {  // 0xff in each byte that is NaN
  return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu);
}

// --------------------------------------------------------------------------- the kernel

template <int D, int ROWS>
struct AttnShape {
  static constexpr int KT = AT_CHUNK * D;               // bytes of a chunk's keys, or values
  // chunks of keys, and of values, in flight or in use (D = 128: 3 and 2 took 106 us for 101)
  static constexpr int KS = D < 128 ? 4 : 2;
  static constexpr int VS = D < 128 ? 4 : 3;
  static constexpr int VW = 2 * KT;                     // widened values; two buffers
  static constexpr int QB = 2;                          // buffers of q (one: 152 -> 198 us)
  static constexpr int QT = ROWS * D;                   // bytes of q hi, or lo
  static constexpr int OFF_VR = KS * KT;                // values as they come
  static constexpr int OFF_V = OFF_VR + VS * KT;
  static constexpr int OFF_Q = OFF_V + 2 * VW;
  static constexpr int SMEM = 1024 + OFF_Q + QB * 2 * QT;
  static constexpr int QUARTERS = ROWS / 32;            // softmax warps of a group
  static constexpr int WARPS = 2 * QUARTERS + 11;
  static constexpr int CONSUMERS = WARPS - 1;           // warps that read the pieces
};
constexpr int TMEM_COLS = 512, TMEM_S = 128, TMEM_O = 384;  // S and P of chunk i at 128 (i % 3), O at 384

enum Role : int { SOFT0, SOFT1, CONV, SPLIT, LOAD, S_MMA, O_MMA };
// Role of a warp and its number within it.  (Softmax warps sit where their quarter of the lanes
// is: warp % 4.)
__device__ __forceinline__ Role role_of(int warp, int& k) {
  k = warp & 3;
  return static_cast<Role>(warp < 16 ? warp >> 2 : LOAD + warp - 16);
}

// Deeper than any warp runs ahead of the softmax, and the softmax ahead of the outputs.  With tiles
// of one chunk, q is split for a tile while the softmax may be four behind it.  A softmax group
// that has a chunk of tile t knows that the outputs up to t - 4 have been read (the chunk's scores
// took a buffer whose products came after them), and leaves its sums for the next tile too, where
// it has none.
constexpr int SC_RING = 8, PIECE_RING = 4, FR_RING = 6, OUT_RING = 5;
constexpr float RAISE = 6.f;                // log2 of how far a score may pass its reference
constexpr float HELD = 9.f;                 // log2 of the weight of the reference as it is held

// A piece of the CTA's run: the chunks [c0, cn) of a tile that some row of it sees.
struct Piece {
  int64_t q0;         // the sequence's first row of q
  int64_t table;      // its row of the block table, as an offset
  int n, len;         // its new tokens and its cached ones
  int h, row0, rows;  // key / value head; the tile's first row and its rows
  int c0, cn, end;    // tokens that the tile's last row sees
  int whole;          // 1: all of the tile's chunks; 0: a part; -1: there is no further piece
  int slot;           // of the workspace, for a part
};

// A row's D sums by f; -inf to the scores of tokens that it does not see (lim on), or whose page
// was not loaded.  Out of line, so that the loops do not share the instruction cache with them.
template <int D>
__device__ __noinline__ void scale_columns(uint32_t t, float f) {
#pragma unroll 1
  for (int w0 = 0; w0 < D; w0 += 16) {
    float o[16];
    tmem_ld16(t + w0, o);
#pragma unroll
    for (int n = 0; n < 16; ++n) o[n] *= f;
    tmem_st16(t + w0, o);
  }
}
__device__ __forceinline__ float score_factor(float fr, const PageScale& sc) {
  const float a = fr * sc.k;
  return a == 0.f ? FLT_MIN : a;  // (never 0, so that a score of infinity stays one)
}
__device__ __noinline__ void mask_scores(uint32_t t, int lim, const PageScale* scales, int page_log2) {
#pragma unroll 1
  for (int w0 = 0; w0 < AT_CHUNK; w0 += 16) {
    const PageScale sc = scales[w0 >> page_log2];
    const int see = sc.ok ? lim - w0 : 0;
    if (__all_sync(FULL_MASK, see >= 16)) continue;
    float s[16];
    tmem_ld16(t + w0, s);
#pragma unroll
    for (int n = 0; n < 16; ++n)
      if (n >= see) s[n] = -INFINITY;
    tmem_st16(t + w0, s);
  }
}

// NaN into the columns of a row's outputs, or of its part, where a token of [t0, t1) has one.
__device__ __noinline__ void put_nans(const Kv8 c, const int32_t* table, int page_log2, int D, int h, int t0, int t1,
                                      __nv_bfloat16* out, float* part) {
#pragma unroll 1
  for (int t = t0; t < t1; ++t) {
    const int id = __ldg(table + (t >> page_log2));
    if (id < 0 || id >= c.n_pages) continue;
    const uint8_t* v = c.v + ((int64_t(id) * c.heads + h) * c.page + (t & (c.page - 1))) * D;
#pragma unroll 1
    for (int w = 0; w < D; ++w)
      if ((v[w] & 0x7f) == 0x7f) {
        if (out) out[w] = __float2bfloat16_rn(NAN);
        else part[w] = NAN;
      }
  }
}

template <int D, int ROWS>
__global__ void __launch_bounds__(32 * AttnShape<D, ROWS>::WARPS, 1)
    kv8_attention_kernel(const __grid_constant__ CUtensorMap tm, const AttnParams p) {
  using S = AttnShape<D, ROWS>;
  constexpr int KS = S::KS, VS = S::VS, QB = S::QB, NQ = S::QUARTERS;
  extern __shared__ uint8_t at_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(at_raw) + 1023) & ~uintptr_t(1023));
  // (A wait tells only a phase's parity, so whoever waits for a phase has to have met the one
  // before: sready of chunk i is at i % 6, a group's own.)
  __shared__ __align__(8) uint64_t kfull[KS], kempty[KS], vfull[VS], vempty[VS], sready[6], vready[2], pready[3], pvdone[3],
      qready[QB], qfree[QB], pc_full[PIECE_RING], pc_empty[PIECE_RING], decided[NQ], met[OUT_RING][NQ], left;
  __shared__ Piece s_piece[PIECE_RING];
  __shared__ PageScale s_sc[SC_RING][8];
  __shared__ float s_fr[FR_RING][ROWS], s_m[OUT_RING][ROWS];
  __shared__ float2 s_ml[OUT_RING][2][ROWS];
  __shared__ int s_nan[PIECE_RING];  // 1 + the piece in whose V a NaN was taken out
  __shared__ uint32_t s_tmem;
  __shared__ volatile uint32_t s_fail;

  const int tid = threadIdx.x, warp = __shfl_sync(FULL_MASK, tid >> 5, 0), lane = tid & 31;
  int k;
  const Role role = role_of(warp, k);
  if (tid == 0) {
    for (int i = 0; i < KS; ++i) { mbar_init(&kfull[i], 1); mbar_init(&kempty[i], 1); }
    for (int i = 0; i < VS; ++i) { mbar_init(&vfull[i], 1); mbar_init(&vempty[i], 4); }
    for (int i = 0; i < 6; ++i) mbar_init(&sready[i], 1);
    for (int i = 0; i < 3; ++i) { mbar_init(&pready[i], NQ); mbar_init(&pvdone[i], 1); }
    for (int i = 0; i < 2; ++i) mbar_init(&vready[i], 4);
    for (int i = 0; i < QB; ++i) { mbar_init(&qready[i], 4); mbar_init(&qfree[i], 1); }
    for (int i = 0; i < PIECE_RING; ++i) {
      mbar_init(&pc_full[i], 1);
      mbar_init(&pc_empty[i], S::CONSUMERS);
      s_nan[i] = 0;
    }
    for (int i = 0; i < NQ; ++i) {
      mbar_init(&decided[i], 1);
      for (int j = 0; j < OUT_RING; ++j) mbar_init(&met[j][i], 2);
    }
    mbar_init(&left, 4);
    fence_mbar_init();
    s_fail = 0;
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&s_tmem)),
                 "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(FULL_MASK, s_tmem, 0);
  pdl_wait();
  pdl_trigger();

  // A wait by a whole warp.  The first one that gives up makes every later one give up soon, and
  // the roles' loops end.
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
  auto next_piece = [&](int pi, Piece& x) -> bool {
    const int e = pi % PIECE_RING;
    if (!wait_warp(&pc_full[e], (pi / PIECE_RING) & 1, ERR_KV8_FULL_WAIT)) return false;
    x = s_piece[e];
    return x.whole >= 0;
  };
  auto next_chunks = [&](int pi) -> int {  // how many it has; -1: there is none
    const int e = pi % PIECE_RING;
    if (!wait_warp(&pc_full[e], (pi / PIECE_RING) & 1, ERR_KV8_FULL_WAIT)) return -1;
    const int n = __shfl_sync(FULL_MASK, s_piece[e].whole < 0 ? -1 : max(s_piece[e].cn - s_piece[e].c0, 0), 0);
    if (lane == 0 && n >= 0) mbar_arrive(&pc_empty[e]);
    return n;
  };
  auto piece_read = [&](int pi) { mbar_arrive(&pc_empty[pi % PIECE_RING]); };

  if (role == LOAD) {
    // ====== the run's pieces, and their chunks: lane i brings the i-th page of a chunk ======
    const Run run = find_run<ROWS>(p, blockIdx.x, gridDim.x);
    const int part = p.c.page, parts = AT_CHUNK >> p.page_log2, bytes = part * D;
    Pieces<ROWS> w(p, run);
    int it = 0, kit = 0, vit = 0, pi = 0;  // (kit, vit: chunks whose keys, values are on their way)
    // Pieces are left one ahead of the one that is loaded, so that its q can be made ready.
    auto leave = [&](Piece& x) -> bool {
      const int e = pi % PIECE_RING;
      bool ok = pi < PIECE_RING || wait_warp(&pc_empty[e], ((pi / PIECE_RING) - 1) & 1, ERR_KV8_EMPTY_WAIT);
      ok = ok && w.next();
      if (ok) {
        const int end = w.end(), cn = max(w.c0, min(w.c1, (end + AT_CHUNK - 1) / AT_CHUNK));
        x = Piece{w.psq.q0, w.pb * p.table_stride, w.psq.n, w.psq.len, w.ph, w.ptile * ROWS, w.rows(),
                  w.c0, cn, end, w.whole(), w.slot()};
      } else {
        x.whole = -1;
      }
      if (lane == 0) {
        s_piece[e] = x;
        mbar_arrive(&pc_full[e]);
      }
      ++pi;
      return ok;
    };
    Piece now{}, next{};
    bool ok_run = leave(now);
    while (ok_run) {
      const bool more = leave(next);
      const int c0 = now.c0, cn = now.cn, end = now.end, h = now.h;
      const int32_t* tab = p.table + now.table;
      auto page_of = [&](int c) {
        const int tok = c * AT_CHUNK + lane * part;
        return lane < parts && c < cn && tok < end ? __ldg(tab + (tok >> p.page_log2)) : -2;
      };
      auto exists = [&](int i) { return i >= 0 && i < p.c.n_pages; };
      // page indices are read two chunks ahead, scales one
      float ks1 = 0.f, vs1 = 1.f;
      auto read_scales = [&](int i) {
        if (!exists(i)) return;
        const int64_t ph = int64_t(i) * p.c.heads + h;
        ks1 = __ldg(p.c.ks + ph);
        vs1 = __ldg(p.c.vs + ph);
      };
      int id1 = page_of(c0), id2 = page_of(c0 + 1);
      read_scales(id1);
#pragma unroll 1
      for (int c = c0; c < cn; ++c, ++it) {
        const int st = it % KS, slot = it % SC_RING;
        const int id = id1;
        const float ks = ks1, vs = vs1;
        id1 = id2;
        read_scales(id1);
        id2 = page_of(c + 2);
        const bool ok = exists(id);
        if (id != -2 && !ok) atomicOr(&g_err_kv8_attn, ERR_KV8_PAGE);
        const int64_t ph = int64_t(ok ? id : 0) * p.c.heads + h;
        const unsigned have = __ballot_sync(FULL_MASK, ok);
        ok_run = it < KS || wait_warp(&kempty[st], ((it / KS) - 1) & 1, ERR_KV8_EMPTY_WAIT);
        if (!ok_run) break;
        // (whoever waits for the stage, or for what is made from it, sees its scales)
        if (lane < 8) s_sc[slot][lane] = page_scale_of(ks, vs, ok);
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&kfull[st], bytes * __popc(have));
        __syncwarp();
        if (ok) tma_load3(sm + st * S::KT + lane * bytes, &tm, 0, 0, static_cast<int>(ph), &kfull[st]);
        ++kit;
        const int sv = it % VS;
        ok_run = it < VS || wait_warp(&vempty[sv], ((it / VS) - 1) & 1, ERR_KV8_EMPTY_WAIT);
        if (!ok_run) break;
        if (lane == 0) mbar_arrive_expect_tx(&vfull[sv], bytes * __popc(have));
        __syncwarp();
        if (ok) bulk_g2s(sm + S::OFF_VR + sv * S::KT + lane * bytes, p.c.v + ph * bytes, bytes, &vfull[sv]);
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
  } else if (role == S_MMA) {
    // ================= S = Q K^T, hi and lo =================
    constexpr uint32_t ID = tc_idesc(128, AT_CHUNK, false, false);
    const uint64_t d_k = tile_desc<D>(sm, 16), d_q = tile_desc<D>(sm + S::OFF_Q, 16);
    int it = 0, qi = 0;
    int chunks;
    for (int pi = 0; (chunks = next_chunks(pi)) >= 0; ++pi) {
      if (chunks <= 0) continue;
      bool ok = wait_warp(&qready[qi % QB], (qi / QB) & 1, ERR_KV8_S_WAIT);
      const uint64_t q = d_q + ((qi % QB) * 2 * S::QT >> 4);
#pragma unroll 1
      for (int c = 0; c < chunks; ++c, ++it) {
        const int st = it % KS, b = it % 3;
        ok = wait_warp(&kfull[st], (it / KS) & 1, ERR_KV8_FULL_WAIT) && ok;
        if (it >= 3) ok = wait_warp(&pvdone[b], ((it / 3) - 1) & 1, ERR_KV8_S_WAIT) && ok;
        if (ok) {
          tc_fence_after();
          const uint64_t kk = d_k + (st * S::KT >> 4);
#pragma unroll 1
          for (int lo = 0; lo < 2; ++lo)
#pragma unroll
            for (int d = 0; d < D / 32; ++d)
              mma_f8(tmem + b * TMEM_S, q + lo * (S::QT >> 4) + 2 * d, kk + 2 * d, ID, lo + d > 0);
        }
        tc_commit(&sready[it % 6]);
        tc_commit(&kempty[st]);
      }
      tc_commit(&qfree[qi % QB]);
      ++qi;
    }
  } else if (role == O_MMA) {
    // ================= O += P V =================
    constexpr uint32_t ID = tc_idesc(128, D, false, true);
    constexpr int VBY = D < 64 ? 64 : 128;  // bytes of a row of a tile of V
    const uint64_t d_v = tile_desc<VBY>(sm + S::OFF_V, AT_CHUNK * 128);
    int it = 0, qi = 0;
    int chunks;
    for (int pi = 0; (chunks = next_chunks(pi)) >= 0; ++pi) {
      if (chunks > 0 && qi++ > 0) wait_warp(&left, qi & 1, ERR_KV8_PV_WAIT);  // the tile before has left O
#pragma unroll 1
      for (int c = 0; c < chunks; ++c, ++it) {
        const int b = it % 3;
        bool ok = wait_warp(&vready[it & 1], (it >> 1) & 1, ERR_KV8_PV_WAIT);
        ok = wait_warp(&pready[b], (it / 3) & 1, ERR_KV8_PV_WAIT) && ok;
        if (ok) {
          tc_fence_after();
          const uint64_t v = d_v + ((it & 1) * S::VW >> 4);
          // (16 tokens further: 8 columns of P; the address field of V, in units of 16 bytes)
#pragma unroll 4
          for (int i = 0; i < AT_CHUNK / 16; ++i)
            mma_f16_ts(tmem + TMEM_O, tmem + b * TMEM_S + 8 * i, v + i * VBY, ID, i > 0 || c > 0);
        }
        tc_commit(&pvdone[b]);
      }
    }
  } else if (role == CONV) {
    // ================= widening of V =================
    int it = 0, qi = 0;  // qi: pieces with chunks
    Piece x;
    for (int pi = 0; next_piece(pi, x); ++pi) {
      if (lane == 0) piece_read(pi);
#pragma unroll 1
      for (int c = x.c0; c < x.cn; ++c, ++it) {
        const int st = it % VS, b = it & 1, slot = it % SC_RING;
        wait_warp(&vfull[st], (it / VS) & 1, ERR_KV8_FULL_WAIT);
        if (it >= 2) wait_warp(&pvdone[(it - 2) % 3], ((it - 2) / 3) & 1, ERR_KV8_PV_WAIT);
        uint8_t* src = sm + S::OFF_VR + st * S::KT;
        uint8_t* dst = sm + S::OFF_V + b * S::VW;
        // Chunks with tokens that some row does not see (the causal edge), with rows behind the
        // last token or with pages that were not loaded: 0 * NaN is NaN, so there V takes part
        // without NaN, and rows that do see a NaN get it at the end.
        const bool edge = (c + 1) * AT_CHUNK > x.len - x.n ||
                          __any_sync(FULL_MASK, lane < (AT_CHUNK >> p.page_log2) && !s_sc[slot][lane & 7].ok);
        constexpr int UPR = D / 16;                     // 16-byte pieces of a row
        constexpr int LPR = UPR < 4 ? UPR : 4;          // lanes on a row
        constexpr int TOKS = 32 / LPR;                  // rows of one round
        constexpr int RB = D < 64 ? 64 : 128;
        constexpr int STEP = UPR < 2 ? UPR : 2;         // pieces of a lane in flight
        // (odd rows of 128 bytes begin with their second half: no bank is met twice)
        const int odd = UPR > LPR ? (lane / LPR) & 1 : 0;
        auto piece_at = [&](int i) { return lane % LPR + ((i / (32 / TOKS)) ^ odd) * LPR; };
        auto tok_at = [&](int i) { return k * 32 + (i % (32 / TOKS)) * TOKS + lane / LPR; };
        if (edge) {  // (in the stage itself, by the lane that widens it)
          bool nan = false;
#pragma unroll 1
          for (int i = 0; i < UPR; ++i) {
            const int tok = tok_at(i);
            uint4* at = reinterpret_cast<uint4*>(src + tok * D + piece_at(i) * 16);
            uint4 w = *at;
            if (c * AT_CHUNK + tok >= x.end || !s_sc[slot][tok >> p.page_log2].ok) w = make_uint4(0u, 0u, 0u, 0u);
            const uint32_t n0 = nan_codes(w.x), n1 = nan_codes(w.y), n2 = nan_codes(w.z), n3 = nan_codes(w.w);
            nan |= (n0 | n1 | n2 | n3) != 0;
            *at = make_uint4(w.x & ~n0, w.y & ~n1, w.z & ~n2, w.w & ~n3);
          }
          if (nan) s_nan[qi % PIECE_RING] = qi + 1;
        }
#pragma unroll 1
        for (int k0 = 0; k0 < UPR; k0 += STEP) {
          uint4 w[STEP];
          int tok[STEP];
#pragma unroll
          for (int i = 0; i < STEP; ++i) {
            tok[i] = tok_at(k0 + i);
            w[i] = *reinterpret_cast<const uint4*>(src + tok[i] * D + piece_at(k0 + i) * 16);
          }
#pragma unroll
          for (int i = 0; i < STEP; ++i) {
            const int piece = piece_at(k0 + i);
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
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&vready[b]);
          mbar_arrive(&vempty[st]);
        }
      }
      qi += x.c0 < x.cn;
    }
  } else if (role == SPLIT) {
    // ====== q as the sum of two e4m3 values, a tile ahead; then the outputs of the tile before ======
    // lanes of a row (16 values each), rows of a warp at a time, and of all four
    constexpr int LPR = D / 16, RPW = 32 / LPR, STEP = 4 * RPW;
    const int piece = lane % LPR, r0 = k * RPW + lane / LPR;
    const uint32_t sign = __float_as_uint(p.scale2) & 0x80000000u;  // q takes the scale's
    const int step_i = STEP / p.group, step_j = STEP - step_i * p.group;
    // outputs: row 32 k + lane
    const int r = 32 * k + lane;
    const uint32_t t_o = tmem + (static_cast<uint32_t>(32 * k) << 16) + TMEM_O;
    int it = 0, qi = 0;  // chunks and pieces with chunks, up to x
    Piece x, y{};
    y.cn = -1;
    for (int pi = 0;; ++pi) {
      const bool more = next_piece(pi, x);
      if (more && lane == 0) piece_read(pi);
      if (more && x.c0 < x.cn) {
        const int b = qi % QB;
        if (qi >= QB) wait_warp(&qfree[b], ((qi / QB) - 1) & 1, ERR_KV8_S_WAIT);
        const __nv_bfloat16* q = p.q + x.q0 * p.q_tok + x.h * p.group * p.q_head + piece * 16;
        uint8_t* hi_at = sm + S::OFF_Q + b * 2 * S::QT;
        uint4 w[2][2];
        int i = (x.row0 + r0) / p.group, j = x.row0 + r0 - i * p.group;  // of the row that is read next
        auto load = [&](int r, uint4* w) {
          w[0] = w[1] = make_uint4(0u, 0u, 0u, 0u);
          if (r < x.rows) {
            const uint4* at = reinterpret_cast<const uint4*>(q + i * p.q_tok + j * p.q_head);
            w[0] = __ldg(at);
            w[1] = __ldg(at + 1);
          }
          i += step_i;
          j += step_j;
          if (j >= p.group) {
            j -= p.group;
            ++i;
          }
        };
        load(r0, w[0]);
        load(r0 + STEP, w[1]);
#pragma unroll 1
        for (int r = r0; __any_sync(FULL_MASK, r < x.rows); r += STEP) {
          const uint32_t in[8] = {w[0][0].x, w[0][0].y, w[0][0].z, w[0][0].w, w[0][1].x, w[0][1].y, w[0][1].z, w[0][1].w};
          w[0][0] = w[1][0];
          w[0][1] = w[1][1];
          load(r + 2 * STEP, w[1]);
          uint32_t top = 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) top = __vmaxu2(top, in[e] & 0x7fff7fffu);
#pragma unroll
          for (int o = LPR / 2; o >= 1; o >>= 1) top = __vmaxu2(top, __shfl_xor_sync(FULL_MASK, top, o));
          top = max(top & 0xffffu, top >> 16);
          // the largest moves to [128, 256); a row with an infinity or a NaN is all NaN
          const int sh = min(7 - (min(max(static_cast<int>(top >> 7), 1), 254) - 127), 120);
          const float up = __uint_as_float(static_cast<uint32_t>(127 + sh) << 23 | sign);
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const __half2 y = __floats2half2_rn(__uint_as_float(in[e] << 16) * up,
                                                __uint_as_float(in[e] & 0xffff0000u) * up);
            const uint32_t h2 = f16x2_to_e4m3x2(*reinterpret_cast<const uint32_t*>(&y));
            const uint32_t b2 = e4m3x2_to_f16x2(static_cast<uint16_t>(h2));
            const __half2 rest = __hsub2(y, *reinterpret_cast<const __half2*>(&b2));
            const uint32_t l2 = f16x2_to_e4m3x2(*reinterpret_cast<const uint32_t*>(&rest));
            hi[e >> 1] = e & 1 ? hi[e >> 1] | h2 << 16 : h2;
            lo[e >> 1] = e & 1 ? lo[e >> 1] | l2 << 16 : l2;
          }
          if (r < x.rows) {
            if (piece == 0)
              s_fr[qi % FR_RING][r] = top >= 0x7f80u ? NAN : fabsf(p.scale2) * __uint_as_float(static_cast<uint32_t>(127 - sh) << 23);
            const int at = r * D + ((piece ^ swz<D>(r)) << 4);
            *reinterpret_cast<uint4*>(hi_at + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(hi_at + S::QT + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&qready[b]);
      }
      if (y.cn >= 0) {  // y: the piece before, the (qi - 1)th with chunks if it has any
        const bool has = r < y.rows, some = y.c0 < y.cn;
        const int i = has ? (y.row0 + r) / p.group : 0, j = has ? y.row0 + r - i * p.group : 0;
        float top = -INFINITY, total = 0.f;
        if (some) {
          const int e = (qi - 1) % OUT_RING;
          wait_warp(&met[e][k], ((qi - 1) / OUT_RING) & 1, ERR_KV8_PV_WAIT);
          top = s_m[e][r];
          // the groups' sums; one of 0 is of no chunk, or of none that the row sees
          const float2 s0 = s_ml[e][0][r], s1 = s_ml[e][1][r];
          total = (s0.y == 0.f ? 0.f : s0.y * ex2(s0.x - top)) + (s1.y == 0.f ? 0.f : s1.y * ex2(s1.x - top));
          wait_warp(&pvdone[(it - 1) % 3], ((it - 1) / 3) & 1, ERR_KV8_PV_WAIT);
          tc_fence_after();
        }
        if (total == 0.f) top = -INFINITY;  // (a NaN stays)
        const int64_t at = (y.q0 + i) * p.q_heads + y.h * p.group + j;
        float* part = p.part + int64_t(y.slot) * ROWS * (D + 2);
        const float f = !y.whole ? 1.f : total == 0.f ? 0.f : 1.f / total;  // no token seen: 0
#pragma unroll 1
        for (int w0 = 0; w0 < D; w0 += 16) {
          float o[16];
          if (some) {
            tmem_ld16(t_o + w0, o);
#pragma unroll
            for (int n = 0; n < 16; ++n) o[n] *= f;
          } else {
#pragma unroll
            for (int n = 0; n < 16; ++n) o[n] = 0.f;
          }
          if (w0 + 16 == D && some) {  // O has been read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&left);
          }
          if (has && y.whole) {
            uint32_t h[8];
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              const __nv_bfloat162 v = __floats2bfloat162_rn(o[2 * n], o[2 * n + 1]);
              h[n] = *reinterpret_cast<const uint32_t*>(&v);
            }
            uint4* dst = reinterpret_cast<uint4*>(p.out + at * D + w0);
            dst[0] = make_uint4(h[0], h[1], h[2], h[3]);
            dst[1] = make_uint4(h[4], h[5], h[6], h[7]);
          } else if (has) {
            float4* dst = reinterpret_cast<float4*>(part + r * D + w0);
#pragma unroll
            for (int n = 0; n < 4; ++n) dst[n] = make_float4(o[4 * n], o[4 * n + 1], o[4 * n + 2], o[4 * n + 3]);
          }
        }
        top -= HELD;  // what the products and sums stand for
        if (has && !y.whole) {
          part[ROWS * D + r] = top;
          part[ROWS * D + ROWS + r] = total;
        } else if (has && p.lse) {
          p.lse[at] = total == 0.f ? -INFINITY : (top + log2f(total)) * LN2_F;
        }
        if (has && some && s_nan[(qi - 1) % PIECE_RING] == qi) {
          // NaN codes of V that this row sees, among the tokens where they were taken out
          const int from = max(y.c0, max(y.len - y.n, 0) / AT_CHUNK) * AT_CHUNK;
          put_nans(p.c, p.table + y.table, p.page_log2, D, y.h, from, min(y.len - y.n + i + 1, y.cn * AT_CHUNK),
                   y.whole ? p.out + at * D : nullptr, part + r * D);
        }
      }
      if (!more) break;
      y = x;
      y.cn = max(y.cn, 0);
      if (x.c0 < x.cn) {
        it += x.cn - x.c0;
        ++qi;
      }
    }
  } else {
    // ================= softmax: group g, rows 32 k + lane =================
    const int g = role == SOFT0 ? 0 : 1, r = 32 * k + lane;
    const uint32_t t_lane = static_cast<uint32_t>(32 * k) << 16;
    int it0 = 0, qi = 0;  // the piece's first chunk; pieces with chunks
    Piece x;
    for (int pi = 0; next_piece(pi, x); ++pi) {
      if (lane == 0) piece_read(pi);
      const int chunks = x.cn - x.c0;
      const bool has = r < x.rows;
      const int seen = x.len - x.n + (has ? (x.row0 + r) / p.group : 0) + 1;
      // The maximum that O stands for (s_m, the groups' in common), the one that l stands for, and
      // the sum of this group's weights.  A row that sees nothing needs no maximum.
      float* const common = &s_m[qi % OUT_RING][r];
      float m = has && seen > 0 ? -INFINITY : 0.f, l = 0.f;
#pragma unroll 1
      for (int d = (it0 ^ g) & 1; d < chunks; d += 2) {
        const int it = it0 + d, slot = it % SC_RING;
        const uint32_t t_s = tmem + t_lane + (it % 3) * TMEM_S;
        const int lim = has ? seen - (x.c0 + d) * AT_CHUNK : AT_CHUNK;  // tokens of the chunk that the row sees
        wait_warp(&sready[it % 6], (it / 6) & 1, ERR_KV8_S_WAIT);
        tc_fence_after();
        const float fr = has && seen > 0 ? s_fr[qi % FR_RING][r] : 1.f;
        // Tokens that a row does not see, or whose page was not loaded, get a score of -inf, in S.
        const bool masks = __any_sync(FULL_MASK, lim < AT_CHUNK || (lane < (AT_CHUNK >> p.page_log2) && !s_sc[slot][lane & 7].ok));
        if (masks) mask_scores(t_s, lim, s_sc[slot], p.page_log2);
        // 16 scores, in units of log2, above a reference
        auto score16 = [&](float* s, const PageScale& sc, float nref) {
          const float a = score_factor(fr, sc), b = sc.log2_v + nref;
          const float2 a2 = make_float2(a, a), b2 = make_float2(b, b);
#pragma unroll
          for (int n = 0; n < 16; n += 2) {
            const float2 y = __ffma2_rn(make_float2(s[n], s[n + 1]), a2, b2);
            s[n] = y.x;
            s[n + 1] = y.y;
          }
        };
        // 1. The row's largest score of the chunk.
        float top = -INFINITY;
        float s[2][16];  // (a block is read while the one before is worked on)
        tmem_ld16_begin(t_s, s[0]);
        auto look = [&](int w0, float* now, float* next) {
          tmem_ld_end(now);
          if (w0 + 16 < AT_CHUNK) tmem_ld16_begin(t_s + w0 + 16, next);
          // (a page's factor is positive, so that its largest product is its largest score)
          float big = fmaxf(now[0], now[1]);
#pragma unroll
          for (int n = 2; n < 16; n += 2) big = max3(big, now[n], now[n + 1]);
          const PageScale sc = s_sc[slot][w0 >> p.page_log2];
          top = fmaxf(top, fmaf(big, score_factor(fr, sc), sc.log2_v));
        };
#pragma unroll 1
        for (int w0 = 0; w0 < AT_CHUNK; w0 += 32) {
          look(w0, s[0], s[1]);
          look(w0 + 16, s[1], s[0]);
        }
        // Whether it asks for a new maximum, once the other group has said so of the chunk before.
        if (it > 0) wait_warp(&decided[k], (it - 1) & 1, ERR_KV8_PV_WAIT);
        if (d > 0) {
          const float was = m;
          m = *common;
          if (was != m) l *= was == -INFINITY ? 0.f : ex2(was - m);
        }
        // (rows that are not there have m = 0)
        const bool anew = (has && top - m > RAISE) || (m == -INFINITY && lim > 0);
        if (__any_sync(FULL_MASK, anew)) {
          const float to = fmaxf(top, m), f = to == -INFINITY ? 1.f : ex2(m - to);
          m = to;
          l *= f;
          if (d > 0) {  // O holds the chunks before, once their products are done
            wait_warp(&pvdone[(it - 1) % 3], ((it - 1) / 3) & 1, ERR_KV8_PV_WAIT);
            tc_fence_after();
            scale_columns<D>(tmem + t_lane + TMEM_O, f);
          }
          *common = m;
        } else if (d == 0) {
          *common = m;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&decided[k]);
        const float nref = m == -INFINITY ? 0.f : HELD - m;
        // 2. The weights, over the scores that have been read (16 columns of pairs for 32 of S).
        float z[32];
        tmem_ld32_begin(t_s, z);
#pragma unroll 1
        for (int w0 = 0; w0 < AT_CHUNK; w0 += 32) {
          uint32_t h[2][8];
          float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          const PageScale sc0 = s_sc[slot][w0 >> p.page_log2], sc1 = s_sc[slot][(w0 + 16) >> p.page_log2];
          tmem_ld32_end(z);
          score16(z, sc0, nref);
          score16(z + 16, sc1, nref);
#pragma unroll
          for (int n = 0; n < 16; n += 2)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const float2 e = make_float2(ex2(z[16 * q + n]), ex2(z[16 * q + n + 1]));
              part[q] = __fadd2_rn(part[q], e);
              const __half2 hh = __floats2half2_rn(e.x, e.y);
              h[q][n / 2] = *reinterpret_cast<const uint32_t*>(&hh);
            }
          if (w0 + 32 < AT_CHUNK) tmem_ld32_begin(t_s + w0 + 32, z);
          l = fmaf(part[0].x + part[0].y, sc0.inv_v, l);
          l = fmaf(part[1].x + part[1].y, sc1.inv_v, l);
          tmem_st8(t_s + w0 / 2, h[0]);
          tmem_st8(t_s + w0 / 2 + 8, h[1]);
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pready[it % 3]);
      }

      if (chunks > 0) {
        s_ml[qi % OUT_RING][g][r] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&met[qi % OUT_RING][k]);
        it0 += chunks;
        ++qi;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && s_fail) atomicOr(&g_err_kv8_attn, s_fail);
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS)
                 : "memory");
  }
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

// Rows of a tile, for all sequences of the call.  Up to 16 go to the kernel of kv8_attn_few.cu (8
// where that is all).  Measured, 128 sequences of up to 8,192 tokens, 8 key / value heads of 128: 4
// rows 197 us there and 267 here, 16 rows 268 and 270; 24 rows, two of its tiles, 513 there and
// 272 here.
int tile_rows(int max_new, int group) {
  const int64_t rows = int64_t(max_new) * group;
  return rows <= 8 ? 8 : rows <= 16 ? 16 : 128;
}
int runs_of(int rows, int D) { return rows <= 16 ? kv8_few_runs(rows, D) : device_sm_count(); }

template <int D, int ROWS>
cudaError_t launch(const CUtensorMap& tm, const AttnParams& prm, int grid, cudaStream_t stream) {
  constexpr int smem = AttnShape<D, ROWS>::SMEM;
  cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void*>(kv8_attention_kernel<D, ROWS>), smem);
  if (e != cudaSuccess) return e;
  kv8_attention_kernel<D, ROWS><<<grid, 32 * AttnShape<D, ROWS>::WARPS, smem, stream>>>(tm, prm);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  PdlScope pdl(true);
  e = launch_k(kv8_join_kernel<D, ROWS, 4, 8>, dim3(grid, 8), dim3(128), 0, stream, prm, grid);
  if (e == cudaSuccess) note_launch(2);
  return e;
}

}  // namespace

size_t kv8_attention_workspace(int max_new, int group, int D) {
  const int rows = tile_rows(max_new, group);
  return size_t(runs_of(rows, D)) * 2 * rows * (D + 2) * sizeof(float);
}

cudaError_t kv8_attention_launch(const Kv8Attention& a, cudaStream_t stream) {
  const int D = a.D, page = a.c.page, rows = tile_rows(a.max_new, a.group);
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
  if (rows <= 16) return kv8_few_launch(prm, D, rows, stream);
  auto fn = encode_fn();
  const int64_t tiles = a.c.n_pages * a.c.heads;
  if (!fn || tiles > INT_MAX) return cudaErrorInvalidValue;
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
  const int grid = runs_of(rows, D);
  return D == 128 ? launch<128, 128>(tm, prm, grid, stream)
         : D == 64 ? launch<64, 128>(tm, prm, grid, stream)
                   : launch<32, 128>(tm, prm, grid, stream);
}

cudaError_t kv8_attention_read_device_error(uint32_t* code) {
  uint32_t v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_err_kv8_attn, sizeof(v));
  if (e != cudaSuccess) return e;
  if (v) e = cudaMemcpyToSymbol(g_err_kv8_attn, &zero, sizeof(zero));
  *code |= v;
  return e == cudaSuccess ? kv8_few_read_device_error(code) : e;
}

}  // namespace lilicorr
