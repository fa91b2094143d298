// Penalties for repeated tokens, biases and grammar masks on logits, before they are ranked.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "kernels.cuh"

namespace lilicorr {

static __device__ uint32_t g_err_adjust;

// For token v of a row, with c and g the number of times that v is among the row's seen tokens and
// among those of them that count:
//   x1 = c > 0 ? (x > 0 ? x / rho : x rho) : x,  x2 = x1 - freq g - [g > 0] pres,  x3 = x2 + bias_v,
//   y = allowed(v) ? x3 : -inf.
// Only the tokens of the history and of the bias list need arithmetic.  They are few, and penalties
// and biases may all but cancel, so sums are kept as pairs of floats, hi + lo, off by 2^-46 of their
// terms' magnitudes for each term, and rounded once; where that does not do (values near the ends of
// the type, or not finite, counts of 2^24 and more) in 64 bits, which are slow on this part.
//
// One CTA for each piece of a row.  A mask alone: it reads the piece (a warp's vectors after one coalesced load of their
// mask; in place, what a mask leaves or takes whole is not read) and writes it.  Else it sends for the piece's vectors to
// the L2 cache, works out meanwhile which of the history's tokens lie in the piece and how often they count, copies the
// piece with its mask, and writes the touched tokens over, while their logits are still near.  It goes over the history
// twice: first each token sets its bit of a bit map of the piece, whose running sums then give every token that is there
// a place in a list; then each token counts at its place.  Neither pass waits for what its atomic operations find, and
// all sums are of integers.
//
// Bound by its steps' latency and its instructions: 256 rows of 151,936 in bf16 with histories of up to 4,096, 64 biases
// and 16 grammars 33.7 us in a graph (23.6 at the copy rate), so that as many CTAs as can be share an SM: four of 512
// threads, at 32 registers, of which it spills eight or so (1,280 CTAs are two waves of 608, and 64 more).  Measured when
// each change was made: four CTAs 35.0, three 35.9, two that hold the piece in registers meanwhile 41.5; pieces of 32 KB,
// which go over a history twice as often, 40.5 with 256 threads.  The piece is the same for small calls, where fewer CTAs
// than SMs are at work (16 rows of 32,003 in f32 7.0 us), and for penalties in place, where each of a row's pieces still
// goes over its history (the large case without masks and biases 23 us).  A mask alone, 512 rows in place, 31 us (25 at
// the copy rate for the sectors that a mask takes in part); 256 threads, 37 with 512.
// A history's tokens are at most as many as it is long, so lists grow with it, and fewer CTAs share an SM: lists end at
// 8,192 tokens, and a piece with more different ones takes them a list at a time (256 rows with histories of 32,768, 161 us
// with whole lists, 88; 84 with lists of 4,096, but those make 64 x 4 rows of 32,003 tokens 73 for 50).  That loop stands apart,
// for such histories alone: in every call's kernel it took 16 short rows from 8.4 to 10.3 us.
// Tried and dropped: a word for each of a piece's tokens to count in, cleared and searched, 57 us (209 with 64-bit
// arithmetic and loops with few lanes at work); two kernels, the second a CTA a row for the touched tokens alone, 41 with
// a table of the ids by their hash and 43 with a bit map of the row, when one took 45: the tokens' logits are read and
// written one by one once the row has left the L2 cache.
constexpr int AJ_VECS = 8;                                // vectors of 16 bytes of a lane
constexpr int AJ_MASK = 256, AJ_TOUCH = 512;              // threads of a CTA of either kernel
constexpr int aj_bytes(int threads) { return threads * AJ_VECS * 16; }  // of a piece
constexpr int AJ_MAX_BIAS = 1024;
constexpr int AJ_LIST = 8192;                             // touched tokens of a piece at a time, at most

struct AdjustParams {
  const void* x;
  void* out;  // x itself, or apart from it
  int64_t x_stride, out_stride;
  int V, per;  // rows that share a history
  const int32_t* hist;
  int64_t hist_stride;
  int cap;
  const int32_t *seen, *from;
  const float *rep, *pres, *freq;
  const int32_t* bias_id;
  const float* bias;
  int n_bias;
  const uint32_t* mask;
  int64_t mask_stride;
  int n_masks;
  const int32_t* mask_index;
  int rows;
  int list;    // touched tokens of a piece at a time, at most
};

template <typename T>
__device__ __forceinline__ T minus_inf();
template <>
__device__ __forceinline__ float minus_inf<float>() { return -INFINITY; }
template <>
__device__ __forceinline__ __nv_bfloat16 minus_inf<__nv_bfloat16>() { return __ushort_as_bfloat16(0xff80); }

// ------------------------------------------------------------------------- touched tokens

// (hi, lo) + (c, d), hi again the float nearest the sum of the two.
__device__ __forceinline__ void add_pair(float& hi, float& lo, float c, float d) {
  const float s = hi + c, b = s - hi, e = (hi - (s - b)) + (c - b);
  lo += e + d;
  hi = s + lo;
  lo = (s - hi) + lo;
}
__device__ __forceinline__ void store_value(float* p, float hi, float) { *p = hi; }
__device__ __forceinline__ void store_value(__nv_bfloat16* p, float hi, float lo) {
  // what is left of the sum decides a tie: an odd last bit stands for it
  if (lo != 0.f) hi = __int_as_float((__float_as_int(hi) - ((lo < 0.f) != (hi < 0.f) ? 1 : 0)) | 1);
  *p = __float2bfloat16_rn(hi);
}
__device__ __forceinline__ void store_double(float* p, double y) { *p = static_cast<float>(y); }
__device__ __forceinline__ void store_double(__nv_bfloat16* p, double y) { *p = __double2bfloat16(y); }

// A touched token's value from its logit, whether it was seen, how often it counts, and the biases of entries
// [e0, e1) of the list whose id is its own, as that of e0 is.
struct Penalties {
  float rho, inv, inv_lo, freq, pres;  // inv + inv_lo = 1 / rho, but for 2^-46 (NaN for a large rho)
  int rep;
  const int* ids;
  const float* bias;
};
// The first entry from i on whose id this is (n: none), four at a time.
__device__ __forceinline__ int next_entry(const int* ids, int i, int n, int id) {
#pragma unroll 1
  for (; i < n; i = (i | 3) + 1) {
    const int4 v = *reinterpret_cast<const int4*>(ids + (i & ~3));
    const uint32_t hit = ((v.x == id) | (v.y == id) << 1 | (v.z == id) << 2 | (v.w == id) << 3) & ~0u << (i & 3);
    if (hit) return min(n, (i & ~3) + __ffs(hit) - 1);
  }
  return n;
}
template <typename T>
__device__ __noinline__ void touch_double(T* o, float x, bool seen, uint32_t g, int id, int e0, int e1, const Penalties* p) {
  double y = x;
  if (seen && p->rep) y = y > 0 ? y / p->rho : y * p->rho;
  if (g) y -= static_cast<double>(p->freq) * g + p->pres;
  for (int i = e0; i < e1; i = next_entry(p->ids, i + 1, e1, id)) y += __ldg(p->bias + i);
  store_double(o, y);
}
__device__ __forceinline__ void add_penalties(float& hi, float& lo, float x, bool seen, uint32_t g, const Penalties* p) {
  hi = x;
  lo = 0.f;
  if (seen && p->rep) {
    const float f = x > 0.f ? p->inv : p->rho, d = x > 0.f ? p->inv_lo : 0.f;
    const float y = x * f;
    lo = fmaf(x, f, -y) + x * d;
    hi = y + lo;
    lo = (y - hi) + lo;
  }
  if (g) {
    const float n = static_cast<float>(g), t = p->freq * n;
    add_pair(hi, lo, -t, -fmaf(p->freq, n, -t));
    add_pair(hi, lo, -p->pres, 0.f);
  }
}
// Whether the pair does (else the value is formed again in 64 bits).
__device__ __forceinline__ bool pair_does(float hi, float lo, uint32_t g) {
  const float size = fabsf(hi);
  return size > 7.9e-31f && size < 1.3e36f && fabsf(lo) <= size && g < (1u << 24);
}
template <typename T>
__device__ __forceinline__ void touch(T* o, float x, bool seen, uint32_t g, int id, int e0, int e1, const Penalties* p) {
  float hi, lo;
  add_penalties(hi, lo, x, seen, g, p);
#pragma unroll 1
  for (int i = e0; i < e1; i = next_entry(p->ids, i + 1, e1, id)) add_pair(hi, lo, __ldg(p->bias + i), 0.f);
  if (pair_does(hi, lo, g)) store_value(o, hi, lo);
  else touch_double(o, x, seen, g, id, e0, e1, p);
}
// The same by a warp, for a token whose entry i may not be the only one (nothing where it is not the first).  (Each lane
// by itself: 752 rows of 2,563 with 253 biases, some ten of them twice, 56 us for 33; a call out of line, which needs a
// stack, 16 short rows 10.4 for 8.9.)
template <typename T>
__device__ __forceinline__ void touch_many(T* o, float x, bool seen, uint32_t g, int i, int n, const Penalties* p) {
  const int lane = threadIdx.x & 31, id = p->ids[i];
  float hi, lo;
  add_penalties(hi, lo, x, seen, g, p);
#pragma unroll 1
  for (int c = 0; c < n; c += 32) {
    uint32_t hit = __ballot_sync(FULL_MASK, c + lane < n && p->ids[min(c + lane, n - 1)] == id);
#pragma unroll 1
    for (; hit; hit &= hit - 1) {
      const int j = c + __ffs(hit) - 1;
      if (j < i) return;
      add_pair(hi, lo, __ldg(p->bias + j), 0.f);
    }
  }
  if (lane != 0) return;
  if (pair_does(hi, lo, g)) store_value(o, hi, lo);
  else touch_double(o, x, seen, g, id, i, n, p);
}

// ------------------------------------------------------------------------------ the mask

// Whether token t may be taken.
__device__ __forceinline__ bool allowed(const uint32_t* m, int t) { return __ldg(m + (t >> 5)) >> (t & 31) & 1; }
// A warp's 1,024 tokens from t on: lane i gets the bits of t + 32 i .. t + 32 i + 31 (0 behind the mask's words).
__device__ __forceinline__ uint32_t mask_block(const uint32_t* m, int words, int t, int lane) {
  const int w = (t >> 5) + lane;
  const uint32_t lo = w < words ? __ldg(m + w) : 0u, last = lane == 31 && w + 1 < words && (t & 31) ? __ldg(m + w + 1) : 0u;
  const uint32_t next = __shfl_down_sync(FULL_MASK, lo, 1);
  return __funnelshift_r(lo, lane == 31 ? last : next, t & 31);
}

// A vector of 16 bytes whose elements are -inf where their bit is 0.
template <typename T>
__device__ __forceinline__ uint4 masked(uint4 v, uint32_t bits) {
  if constexpr (sizeof(T) == 4) {
    const uint32_t ninf = 0xff800000u;
    return make_uint4(bits & 1 ? v.x : ninf, bits & 2 ? v.y : ninf, bits & 4 ? v.z : ninf, bits & 8 ? v.w : ninf);
  } else {
    // four bits to the tops of four bytes, each of which is then spread over a half
    const uint32_t lo = (bits & 15) * 0x10204080u, hi = (bits >> 4 & 15) * 0x10204080u;
    auto put = [](uint32_t& x, uint32_t tops, auto which) {
      uint32_t keep;
      asm("prmt.b32 %0, %1, 0, %2;" : "=r"(keep) : "r"(tops), "n"(decltype(which)::value));
      x = (x & keep) | (0xff80ff80u & ~keep);
    };
    put(v.x, lo, std::integral_constant<int, 0x9988>());
    put(v.y, lo, std::integral_constant<int, 0xbbaa>());
    put(v.z, hi, std::integral_constant<int, 0x9988>());
    put(v.w, hi, std::integral_constant<int, 0xbbaa>());
    return v;
  }
}

// Tokens [t0, t0 + n) of a row: a piece, a warp's 32 * AJ_VECS vectors of it, 32 apart for a lane.
template <typename T, bool INPLACE, int THREADS>
struct Piece {
  static constexpr int E = 16 / sizeof(T);
  static constexpr uint32_t FULL = (1u << E) - 1;
  uint32_t bits[AJ_VECS / 4];  // of a vector's elements, 8 bits for each vector
  int head, left;              // elements before the first whole vector; the lane's vectors reach this far

  __device__ __forceinline__ static int first() { return (threadIdx.x >> 5) * 32 * AJ_VECS + (threadIdx.x & 31); }
  __device__ __forceinline__ uint32_t of(int i) const { return bits[i / 4] >> (8 * (i % 4)) & FULL; }
  // Whether x and o lie alike to the 16-byte grid.
  __device__ __forceinline__ static bool alike(const T* x, const T* o) {
    return INPLACE || (reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(o)) % 16 == 0;
  }
  __device__ __forceinline__ void look(const T* x, const T* o, const uint32_t* m, int words, int t0, int n) {
    const int lane = threadIdx.x & 31;
    head = min(n, static_cast<int>((16 - reinterpret_cast<uintptr_t>(o) % 16) % 16 / sizeof(T)));
    left = (n - head) / E - first();
    if ((INPLACE && !m) || !alike(x, o)) left = -lane;  // (nothing to write, or one by one; no warp has vectors then)
#pragma unroll
    for (int i = 0; i < AJ_VECS / 4; ++i) bits[i] = ~0u;
    if (m && left + lane > 0) {
#pragma unroll
      for (int k = 0; k < AJ_VECS / 4; ++k) {
        bits[k] = 0;
        constexpr int PER = 4 * E;  // vectors, by a block of 1,024 tokens (f32: half of it)
        const uint32_t block = mask_block(m, words, t0 + head + (first() - lane) * E + k * 32 * PER, lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) bits[k] |= (__shfl_sync(FULL_MASK, block, i * E + lane * E / 32) >> (lane * E & 31) & FULL) << (8 * i);
      }
    }
  }
  // Whether vector i is read.
  __device__ __forceinline__ bool wanted(int i) const { return 32 * i < left && of(i) != 0 && !(INPLACE && of(i) == FULL); }
  __device__ __forceinline__ void prefetch(const T* x) const {
#pragma unroll
    for (int i = 0; i < AJ_VECS; ++i)
      if (wanted(i)) asm volatile("prefetch.global.L2 [%0];" ::"l"(x + head + (first() + 32 * i) * E));
  }
  // Vectors FROM .. FROM + N - 1, written with their mask.
  template <int FROM, int N>
  __device__ __forceinline__ void move(const T* x, T* o, const uint32_t* m) const {
    uint4 w[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      w[i] = make_uint4(0u, 0u, 0u, 0u);
      if (wanted(FROM + i)) w[i] = *reinterpret_cast<const uint4*>(x + head + (first() + 32 * (FROM + i)) * E);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t b = of(FROM + i);
      if (32 * (FROM + i) < left && !(INPLACE && b == FULL))
        *reinterpret_cast<uint4*>(o + head + (first() + 32 * (FROM + i)) * E) = m ? masked<T>(w[i], b) : w[i];
    }
  }
  // What no vector holds.
  __device__ __forceinline__ void ends(const T* x, T* o, const uint32_t* m, int t0, int n) const {
    if (INPLACE && !m) return;
    if (!alike(x, o)) {
      for (int t = threadIdx.x; t < n; t += THREADS) o[t] = !m || allowed(m, t0 + t) ? x[t] : minus_inf<T>();
      return;
    }
    const int tail = head + (n - head) / E * E, all = head + n - tail;
    if (static_cast<int>(threadIdx.x) < all) {
      const int t = threadIdx.x < head ? threadIdx.x : tail + threadIdx.x - head;
      if (m && !allowed(m, t0 + t)) o[t] = minus_inf<T>();
      else if (!INPLACE) o[t] = x[t];
    }
  }
};

// A row's mask, if any.  False where the row is to be left out.
__device__ __forceinline__ bool row_mask(const AdjustParams& p, int64_t r, const uint32_t*& m) {
  m = nullptr;
  if (!p.mask) return true;
  const int i = p.mask_index ? __ldg(p.mask_index + r) : static_cast<int>(r);
  if (i >= p.n_masks) return false;
  if (i >= 0) m = p.mask + i * p.mask_stride;
  return true;
}
// The tokens that a row sees.  False where the row is to be left out.
__device__ __forceinline__ bool row_seen(const AdjustParams& p, int64_t r, int& seen) {
  seen = p.hist ? __ldg(p.seen + r) : 0;
  return seen >= 0 && seen <= p.cap;
}

// ------------------------------------------------------------------------------- kernels

template <typename T, bool INPLACE>
__global__ void __launch_bounds__(AJ_MASK, 5) adjust_mask_kernel(const AdjustParams p) {
  constexpr int TOKENS = aj_bytes(AJ_MASK) / sizeof(T);
  const int64_t r = blockIdx.z * gridDim.y + blockIdx.y;  // (fits 32 bits: host)
  const int t0 = static_cast<int>(blockIdx.x) * TOKENS, n = min(TOKENS, p.V - t0);
  const uint32_t* m = nullptr;
  const bool has = r < p.rows && row_mask(p, r, m);
  if (r < p.rows && !has && threadIdx.x == 0) atomicOr(&g_err_adjust, ERR_MASK_INDEX);
  if (!has) return;  // the row is left out
  const T* x = static_cast<const T*>(p.x) + r * p.x_stride + t0;
  T* o = static_cast<T*>(p.out) + r * p.out_stride + t0;
  Piece<T, INPLACE, AJ_MASK> piece;
  piece.look(x, o, m, (p.V + 31) >> 5, t0, n);
  piece.template move<0, AJ_VECS>(x, o, m);
  piece.ends(x, o, m, t0, n);
}

// Calls f(ids, position) for the first `seen` tokens of a history, by fours: from the first 16-byte boundary on, `ahead`
// being the thread's first ones, then for the ends (whose other ids are -1).
template <typename F>
__device__ __forceinline__ void each_token(const int32_t* hist, int lead, int seen, int4 ahead, F f) {
  const int tid = threadIdx.x, fours = max(0, seen - lead) / 4, tail = lead + 4 * fours;
#pragma unroll 1
  for (int i = tid; i < fours; i += AJ_TOUCH) {
    const int4 q = ahead;
    if (i + AJ_TOUCH < fours) ahead = __ldg(reinterpret_cast<const int4*>(hist + lead) + i + AJ_TOUCH);
    f(q, lead + 4 * i);
  }
  const int at = tid < 4 ? tid : tail + tid - 4;  // (lead is at most 3, and so is what is left)
  if (tid < 8 && at < (tid < 4 ? min(lead, seen) : seen)) f(make_int4(__ldg(hist + at), -1, -1, -1), at);
}
// Atomic operations on shared memory where t < n, without a branch.
__device__ __forceinline__ void or_below(uint32_t t, uint32_t n, uint32_t at, uint32_t v) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.lt.u32 p, %0, %1;\n\t@p red.shared.or.b32 [%2], %3;\n\t}" ::"r"(t), "r"(n), "r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ void add_below(uint32_t t, uint32_t n, uint32_t at, uint32_t v) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.lt.u32 p, %0, %1;\n\t@p red.shared.add.u32 [%2], %3;\n\t}" ::"r"(t), "r"(n), "r"(at), "r"(v) : "memory");
}

// A piece's touched tokens from the list'th on (of a history with that many different ones in the piece), a list at a
// time: what the kernel does with the first ones, out of its way.
template <typename T>
struct Rest {
  const T* x;
  T* o;
  const uint32_t *m, *map, *biased;
  const uint16_t* place;
  const int* id;
  uint32_t* count;
  uint16_t* token;
  const int32_t* hist;
  const Penalties* pen;
  int t0, n, words, lead, seen, from, list, all, n_bias;
  bool counts;
};
template <typename T>
__device__ __noinline__ void touch_rest(const Rest<T>& r) {
  const int tid = threadIdx.x;
  auto place = [&](uint32_t t) { return static_cast<uint32_t>(r.place[t >> 5] + __popc(r.map[t >> 5] & ((1u << (t & 31)) - 1))); };
#pragma unroll 1
  for (uint32_t w0 = r.list; w0 < static_cast<uint32_t>(r.all); w0 += r.list) {
    __syncthreads();
#pragma unroll 1
    for (int w = tid; w < r.words; w += AJ_TOUCH) {
      uint32_t k = r.place[w] - w0;
      for (uint32_t b = r.map[w]; b; b &= b - 1, ++k)
        if (k < static_cast<uint32_t>(r.list)) {
          r.token[k] = static_cast<uint16_t>(32 * w + __ffs(b) - 1);
          r.count[k] = 0;
        }
    }
    __syncthreads();
    if (r.counts) {
      const int4 ahead = r.lead + 4 * tid + 4 <= r.seen ? __ldg(reinterpret_cast<const int4*>(r.hist + r.lead) + tid) : make_int4(-1, -1, -1, -1);
      each_token(r.hist, r.lead, r.seen, ahead, [&](int4 q, int i) {
        const int id[4] = {q.x, q.y, q.z, q.w};
#pragma unroll 1
        for (int j = 0; j < 4; ++j) {
          const uint32_t t = static_cast<uint32_t>(id[j]) - r.t0, k = t < static_cast<uint32_t>(r.n) && i + j >= r.from ? place(t) - w0 : UINT_MAX;
          add_below(k, r.list, smem_addr(r.count) + 4 * k, 1u);
        }
      });
      __syncthreads();
    }
    for (int i = tid; i < min(r.list, r.all - static_cast<int>(w0)); i += AJ_TOUCH) {
      const int t = r.token[i];
      if (!(r.biased[t >> 5] >> (t & 31) & 1) && (!r.m || allowed(r.m, r.t0 + t)))
        touch(r.o + t, static_cast<float>(r.x[t]), true, r.count[i], 0, 0, 0, r.pen);
    }
    for (int i = tid; i < r.n_bias; i += AJ_TOUCH) {
      const int id = r.id[i];
      const uint32_t t = static_cast<uint32_t>(id) - r.t0;
      if (t >= static_cast<uint32_t>(r.n) || (r.m && !allowed(r.m, id)) || !(r.map[t >> 5] >> (t & 31) & 1)) continue;
      const uint32_t k = place(t) - w0;
      if (next_entry(r.id, 0, i, id) < i || k >= static_cast<uint32_t>(r.list)) continue;
      touch(r.o + t, static_cast<float>(r.x[t]), true, r.count[k], id, i, r.n_bias, r.pen);
    }
  }
}

// LONG: histories that may bring more tokens into a piece than a list of AJ_LIST holds.
template <typename T, bool INPLACE, bool LONG>
__global__ void __launch_bounds__(AJ_TOUCH, 4) adjust_touch_kernel(const AdjustParams p) {
  constexpr int TOKENS = aj_bytes(AJ_TOUCH) / sizeof(T), WORDS = TOKENS / 32;
  constexpr int EACH = WORDS > AJ_TOUCH ? WORDS / AJ_TOUCH : 1;  // words of the bit map for each thread
  extern __shared__ __align__(16) uint32_t s_count[];                       // [list] how often a token of the list counts
  uint16_t* const s_token = reinterpret_cast<uint16_t*>(s_count + p.list);  // [list] its place in the piece
  __shared__ __align__(16) uint32_t s_map[WORDS];                           // a bit a token
  __shared__ uint16_t s_place[WORDS];                                       // tokens of the list before a word's
  __shared__ __align__(16) int s_id[AJ_MAX_BIAS];
  __shared__ uint32_t s_biased[WORDS];                                      // a bit a token of the bias list
  __shared__ int s_sum[AJ_TOUCH / 32];
  __shared__ uint32_t s_twice[32];  // bit t % 1024: tokens of the piece that have several biases, and others
  __shared__ Penalties s_pen;
  const int tid = threadIdx.x, lane = tid & 31;
  const uint32_t row = blockIdx.z * gridDim.y + blockIdx.y;  // (row and group fit 32 bits: host)
  if (row >= static_cast<uint32_t>(p.rows)) return;
  const int64_t r = row, h = p.per == 1 ? row : row / static_cast<uint32_t>(p.per);
  const int t0 = static_cast<int>(blockIdx.x) * TOKENS, n = min(TOKENS, p.V - t0);
  // the first tokens of the history are read before it is known how many are seen
  const int32_t* hist = p.hist + h * p.hist_stride;
  const int lead = static_cast<int>((16 - reinterpret_cast<uintptr_t>(hist) % 16) % 16 / 4);
  int4 ahead = make_int4(-1, -1, -1, -1);
  if (p.hist && lead + 4 * tid + 4 <= p.cap) ahead = __ldg(reinterpret_cast<const int4*>(hist + lead) + tid);
  const uint32_t* m;
  int seen;
  const bool has = row_mask(p, r, m), counts = row_seen(p, r, seen);
  if (tid == 0 && !has) atomicOr(&g_err_adjust, ERR_MASK_INDEX);
  if (tid == 0 && !counts) atomicOr(&g_err_adjust, ERR_KV8_LENGTH);
  if (!has || !counts) return;  // the row is left out
  const T* x = static_cast<const T*>(p.x) + r * p.x_stride + t0;
  T* o = static_cast<T*>(p.out) + r * p.out_stride + t0;
  Piece<T, INPLACE, AJ_TOUCH> piece;
  piece.look(x, o, m, (p.V + 31) >> 5, t0, n);
  piece.prefetch(x);
  const int from = p.from ? __ldg(p.from + h) : 0;
  for (int i = tid; i < WORDS; i += AJ_TOUCH) s_map[i] = s_biased[i] = 0;
  if (tid < 32) s_twice[tid] = 0;
  for (int i = tid; i < p.n_bias; i += AJ_TOUCH) s_id[i] = __ldg(p.bias_id + h * p.n_bias + i);
  if (tid == AJ_TOUCH - 1) {
    Penalties q{p.rep ? __ldg(p.rep + h) : 1.f, 0.f, 0.f, p.freq ? __ldg(p.freq + h) : 0.f, p.pres ? __ldg(p.pres + h) : 0.f,
                p.rep != nullptr, s_id, p.bias + h * p.n_bias};
    // (what is left of a reciprocal near the least normal number has too few bits: in 64 bits then)
    q.inv = fabsf(q.rho) < 1.2e30f ? 1.f / q.rho : NAN;
    q.inv_lo = fmaf(-q.inv, q.rho, 1.f) * q.inv;
    s_pen = q;
  }
  __syncthreads();
  // 1. which tokens there are
  each_token(hist, lead, seen, ahead, [&](int4 q, int) {
    const int id[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t t = static_cast<uint32_t>(id[k]) - t0;
      or_below(t, n, smem_addr(s_map) + (t >> 5) * 4, __funnelshift_l(0u, 1u, t));
    }
  });
  for (int i = tid; i < p.n_bias; i += AJ_TOUCH) {
    const uint32_t t = static_cast<uint32_t>(s_id[i]) - t0;
    if (t < static_cast<uint32_t>(n) && (atomicOr(s_biased + (t >> 5), 1u << (t & 31)) >> (t & 31) & 1))
      atomicOr(s_twice + ((t >> 5) & 31), 1u << (t & 31));
  }
  __syncthreads();
  // their places in the list, a word of the map for each thread
  uint32_t word[EACH];
  int mine = 0;
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    word[i] = tid * EACH < WORDS ? s_map[tid * EACH + i] : 0;
    mine += __popc(word[i]);
  }
  int at = mine;
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) {
    const int y = __shfl_up_sync(FULL_MASK, at, k);
    if (lane >= k) at += y;
  }
  if (lane == 31) s_sum[tid >> 5] = at;
  __syncthreads();
  int all = lane < AJ_TOUCH / 32 ? s_sum[lane] : 0;
  at += __reduce_add_sync(FULL_MASK, lane < tid >> 5 ? all : 0) - mine;
  all = __reduce_add_sync(FULL_MASK, all);
  if (tid * EACH < WORDS)
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      s_place[tid * EACH + i] = static_cast<uint16_t>(at);
      for (uint32_t b = word[i]; b; b &= b - 1, ++at) {
        if (LONG && at >= p.list) continue;  // (of touch_rest)
        s_token[at] = static_cast<uint16_t>(32 * (tid * EACH + i) + __ffs(b) - 1);
        s_count[at] = 0;
      }
    }
  __syncthreads();
  auto place = [&](uint32_t t) { return s_place[t >> 5] + __popc(s_map[t >> 5] & ((1u << (t & 31)) - 1)); };
  // 2. how often they count, where a penalty asks for it
  if (p.freq || p.pres) each_token(hist, lead, seen, ahead, [&](int4 q, int i) {
    const int id[4] = {q.x, q.y, q.z, q.w};
    uint32_t at[4] = {UINT_MAX, UINT_MAX, UINT_MAX, UINT_MAX};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t t = i + k >= from ? static_cast<uint32_t>(id[k]) - t0 : UINT_MAX;
      if (t < static_cast<uint32_t>(n)) at[k] = place(t);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) add_below(at[k], LONG ? p.list : UINT_MAX, smem_addr(s_count) + 4 * at[k], 1u);
  });
  piece.template move<0, AJ_VECS / 2>(x, o, m);
  piece.template move<AJ_VECS / 2, AJ_VECS / 2>(x, o, m);
  piece.ends(x, o, m, t0, n);
  __syncthreads();
  for (int i = tid; i < (LONG ? min(all, p.list) : all); i += AJ_TOUCH) {
    const int t = s_token[i];
    if (!(s_biased[t >> 5] >> (t & 31) & 1) && (!m || allowed(m, t0 + t))) touch(o + t, static_cast<float>(x[t]), true, s_count[i], 0, 0, 0, &s_pen);
  }
  // tokens of the bias list, by the first entry that names them (from the last warps on, whose lists are the shortest)
#pragma unroll 1
  for (int i0 = 0; i0 < p.n_bias; i0 += AJ_TOUCH) {
    const int i = i0 + AJ_TOUCH - 1 - tid, id = i < p.n_bias ? s_id[i] : -1;
    const uint32_t t = static_cast<uint32_t>(id) - t0;
    bool mine = t < static_cast<uint32_t>(n) && (!m || allowed(m, id)), there = false, twice = false;
    float v = 0.f;
    uint32_t g = 0;
    if (mine) {
      there = s_map[t >> 5] >> (t & 31) & 1;
      twice = s_twice[(t >> 5) & 31] >> (t & 31) & 1;
      const int k = there ? place(t) : 0;
      if (there) g = s_count[LONG ? min(k, p.list - 1) : k];
      if (LONG && k >= p.list) mine = false;  // (of touch_rest)
      else v = static_cast<float>(x[t]);
    }
    if (mine && !twice) touch(o + t, v, there, g, id, i, i + 1, &s_pen);
#pragma unroll 1
    for (uint32_t many = __ballot_sync(FULL_MASK, mine && twice); many; many &= many - 1) {
      const int l = __ffs(many) - 1;
      touch_many(o + __shfl_sync(FULL_MASK, t, l), __shfl_sync(FULL_MASK, v, l), __shfl_sync(FULL_MASK, there, l), __shfl_sync(FULL_MASK, g, l),
                 __shfl_sync(FULL_MASK, i, l), p.n_bias, &s_pen);
    }
  }
  if (LONG && all > p.list)
    touch_rest<T>(Rest<T>{x, o, m, s_map, s_biased, s_place, s_id, s_count, s_token, hist, &s_pen, t0, n, WORDS, lead, seen, from, p.list, all, p.n_bias,
                          p.freq || p.pres});
}

cudaError_t adjust_read_device_error(uint32_t* code) {
  uint32_t v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_err_adjust, sizeof(v));
  if (e != cudaSuccess) return e;
  if (v) e = cudaMemcpyToSymbol(g_err_adjust, &zero, sizeof(zero));
  *code |= v;
  return e;
}

namespace {

lilicorr_status fail(lilicorr_status st, const char* msg) {
  set_last_error(msg);
  return st;
}

// Whether [b, b + n) shares a byte with one of the rows of `bytes` from o on, `stride` apart.
using wide = unsigned __int128;
bool rows_meet(const void* o, int64_t rows, wide stride, wide bytes, const void* b, wide n) {
  const wide x = reinterpret_cast<uintptr_t>(o), y = reinterpret_cast<uintptr_t>(b);
  if (!b || y + n <= x || y >= x + (rows - 1) * stride + bytes) return false;
  const wide r = y <= x ? 0 : (y - x) / stride;  // the last row that begins no later than b, or the first
  return y < x + r * stride + bytes || y + n > x + (r + 1) * stride;
}

template <typename T>
cudaError_t adjust_launch(const AdjustParams& p, int64_t pieces, bool touch, cudaStream_t stream) {
  const bool inplace = p.x == p.out;
  const int smem = touch ? p.list * 6 : 0;
  constexpr int Y = 32768;  // (rows that pass the grid's second dimension go on in its third)
  const dim3 grid(static_cast<unsigned>(pieces), std::min(p.rows, Y), (p.rows - 1) / Y + 1);
  auto go = [&](auto kern) -> cudaError_t {
    cudaError_t e = smem > 32 * 1024 ? allow_dynamic_smem(reinterpret_cast<const void*>(kern), smem) : cudaSuccess;
    if (e != cudaSuccess) return e;
    kern<<<grid, touch ? AJ_TOUCH : AJ_MASK, smem, stream>>>(p);
    e = cudaGetLastError();
    if (e == cudaSuccess) note_launch();
    return e;
  };
  if (touch && p.cap > AJ_LIST) return inplace ? go(adjust_touch_kernel<T, true, true>) : go(adjust_touch_kernel<T, false, true>);
  if (touch) return inplace ? go(adjust_touch_kernel<T, true, false>) : go(adjust_touch_kernel<T, false, false>);
  return inplace ? go(adjust_mask_kernel<T, true>) : go(adjust_mask_kernel<T, false>);
}

}  // namespace
}  // namespace lilicorr

using namespace lilicorr;

extern "C" lilicorr_status lilicorr_adjust_logits(const lilicorr_adjust* a, void* stream) {
  auto bad = [](const char* why) { return fail(LILICORR_ERR_INVALID_ARG, why); };
  if (!a || !a->logits || !a->out) return bad("lilicorr_adjust_logits: null pointer");
  if (a->ldtype != LILICORR_F32 && a->ldtype != LILICORR_BF16) return bad("lilicorr_adjust_logits: logits are f32 or bf16");
  const int es = a->ldtype == LILICORR_BF16 ? 2 : 4;
  constexpr int64_t LIM = int64_t(1) << 40;
  if (a->rows < 1 || a->rows > INT_MAX || a->V < 1 || a->V > INT_MAX - (1 << 20) || a->row_stride < a->V || a->row_stride > LIM ||
      a->out_stride < a->V || a->out_stride > LIM)
    return bad("lilicorr_adjust_logits: rows, V or a row stride is out of range");
  const uintptr_t x = reinterpret_cast<uintptr_t>(a->logits), o = reinterpret_cast<uintptr_t>(a->out);
  if (x % es || o % es) return bad("lilicorr_adjust_logits: logits are element aligned");
  if (!word_aligned({a->history, a->seen, a->counted_from, a->repetition, a->presence, a->frequency, a->bias_id, a->bias, a->mask, a->mask_index}))
    return bad("lilicorr_adjust_logits: what is read besides the logits is 4-byte aligned");
  if (a->logits == a->out ? a->row_stride != a->out_stride
                          : x < o + (wide(a->rows - 1) * a->out_stride + a->V) * es &&
                                o < x + (wide(a->rows - 1) * a->row_stride + a->V) * es)
    return bad("lilicorr_adjust_logits: out is the logits themselves, or shares nothing with them");
  if (a->groups < 1 || a->rows % a->groups) return bad("lilicorr_adjust_logits: groups divides rows");
  if (a->history && (!a->seen || a->cap < 1 || a->cap >= 1 << 29 || a->history_stride < a->cap || a->history_stride > LIM))
    return bad("lilicorr_adjust_logits: history needs seen, a capacity below 2^29 and a stride of at least it");
  if (!a->history && (a->repetition || a->presence || a->frequency || a->counted_from))
    return bad("lilicorr_adjust_logits: penalties need a history");
  if (a->n_bias < 0 || a->n_bias > AJ_MAX_BIAS || (a->n_bias > 0 && (!a->bias_id || !a->bias)))
    return bad("lilicorr_adjust_logits: at most 1024 biases, with ids and values");
  if (a->mask && (a->n_masks < 1 || a->n_masks > INT_MAX || a->mask_stride < (a->V + 31) / 32 || a->mask_stride > LIM ||
                  (!a->mask_index && a->n_masks < a->rows)))
    return bad("lilicorr_adjust_logits: masks have (V + 31) / 32 words, one for each row or an index");
  if (!a->mask && a->mask_index) return bad("lilicorr_adjust_logits: an index needs masks");
  // CTAs read what they need of these while others write
  auto met = [&](const void* b, int64_t rows, int64_t row, int64_t stride) {
    return rows_meet(a->out, a->rows, wide(a->out_stride) * es, wide(a->V) * es, b, (wide(rows - 1) * stride + row) * 4);
  };
  if (met(a->history, a->groups, a->cap, a->history_stride) || met(a->seen, a->rows, 1, 1) || met(a->counted_from, a->groups, 1, 1) ||
      met(a->repetition, a->groups, 1, 1) || met(a->presence, a->groups, 1, 1) || met(a->frequency, a->groups, 1, 1) ||
      (a->n_bias > 0 && (met(a->bias_id, a->groups, a->n_bias, a->n_bias) || met(a->bias, a->groups, a->n_bias, a->n_bias))) ||
      met(a->mask, a->n_masks, (a->V + 31) / 32, a->mask_stride) || met(a->mask_index, a->rows, 1, 1))
    return bad("lilicorr_adjust_logits: out shares memory with what is read besides the logits");
  AdjustParams p{};
  p.x = a->logits; p.out = a->out;
  p.x_stride = a->row_stride; p.out_stride = a->out_stride;
  p.V = static_cast<int>(a->V);
  p.per = static_cast<int>(a->rows / a->groups);
  p.hist = a->history; p.hist_stride = a->history_stride; p.cap = a->cap;
  p.seen = a->seen; p.from = a->counted_from;
  p.rep = a->repetition; p.pres = a->presence; p.freq = a->frequency;
  p.bias_id = a->bias_id; p.bias = a->bias; p.n_bias = a->n_bias;
  p.mask = reinterpret_cast<const uint32_t*>(a->mask); p.mask_stride = a->mask_stride;
  p.n_masks = static_cast<int>(a->n_masks); p.mask_index = a->mask_index;
  const bool touch = a->history || a->n_bias > 0;
  if (!touch && !a->mask && a->logits == a->out) return LILICORR_OK;
  const int64_t tokens = aj_bytes(touch ? AJ_TOUCH : AJ_MASK) / es;
  const int64_t pieces = (a->V + tokens - 1) / tokens;
  p.rows = static_cast<int>(a->rows);
  if (a->rows > INT_MAX - 65536 || a->rows * pieces > INT_MAX) return bad("lilicorr_adjust_logits: rows * V is too large for one call");
  // a piece's list holds every token that the history may bring into it, or as many of them as leave room for other CTAs
  p.list = static_cast<int>(std::max<int64_t>(4, (std::min<int64_t>({a->history ? a->cap : 0, tokens, a->V, AJ_LIST}) + 3) / 4 * 4));
  const cudaError_t e = es == 2 ? adjust_launch<__nv_bfloat16>(p, pieces, touch, static_cast<cudaStream_t>(stream))
                                : adjust_launch<float>(p, pieces, touch, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(LILICORR_ERR_CUDA, cudaGetErrorString(e));
  return LILICORR_OK;
}
