// Penalties for repeated tokens, biases and grammar masks on logits, before they are ranked.
#include <climits>

#include "kernels.cuh"

namespace lilicorr {

static __device__ uint32_t g_err_adjust;

// For token v of a row, with c and g the number of times that v is among the row's seen tokens and
// among those of them that count:
//   x1 = c > 0 ? (x > 0 ? x / rho : x rho) : x,  x2 = x1 - freq g - [g > 0] pres,  x3 = x2 + bias_v,
//   y = allowed(v) ? x3 : -inf.
// Only the tokens of the history and of the bias list need arithmetic.  They are few, and penalties
// and biases may all but cancel, so sums are kept as pairs of floats, hi + lo, off by 2^-47 of their
// terms' magnitudes for each term, and rounded once; where that does not do (values near the ends of
// the type, or not finite, counts of 2^24 and more) in 64 bits, which are slow on this part (with them
// throughout, and a quotient for each warp, the large case below took 121 us).
//
// One CTA for each piece of 16 KB of a row.  It counts the history's tokens that lie in its piece in shared
// memory, a word a token (integer sums: any order gives the same), while the piece's logits are on their
// way; writes the logits with the mask; and then writes the touched tokens over, each lane those among its
// own words, one at a time, so that the warp's 64-bit arithmetic is full.  Where there is only a mask a CTA
// has no words and takes AJ_SPAN pieces.  In place, what a mask leaves or takes whole is not read.
constexpr int AJ_THREADS = 256;
constexpr int AJ_VECS = 4;                                // vectors of 16 bytes of a lane
constexpr int AJ_PIECE = AJ_THREADS * AJ_VECS * 16;       // bytes
#ifndef AJ_CTAS
#define AJ_CTAS 6
#endif
#ifndef AJ_SPAN_
#define AJ_SPAN_ 4
#endif
constexpr int AJ_SPAN = AJ_SPAN_;
constexpr int AJ_MAX_BIAS = 1024;
// a token's word: how often it counts, whether it has a bias, whether it was seen without counting
constexpr uint32_t AJ_BIAS = 1u << 30, AJ_SEEN = 1u << 31, AJ_COUNT = AJ_BIAS - 1;

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
  int pieces;
};

template <typename T>
__device__ __forceinline__ T minus_inf();
template <>
__device__ __forceinline__ float minus_inf<float>() { return -INFINITY; }
template <>
__device__ __forceinline__ __nv_bfloat16 minus_inf<__nv_bfloat16>() { return __ushort_as_bfloat16(0xff80); }
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

// A touched token's value; id: its place in the piece.
struct Penalties {
  float rho, inv, inv_lo, freq, pres;  // inv + inv_lo = 1 / rho, but for 2^-46
  bool rep;
  const int* ids;  // padded to a multiple of 4 with ids of no token
  const float* bias;
  int n_bias;
};
template <typename T>
__device__ __noinline__ void touch_double(T* o, float x, uint32_t word, int id, const Penalties& p);

template <typename T>
__device__ __forceinline__ void touch(T* o, float x, uint32_t word, int id, const Penalties& p) {
  float hi = x, lo = 0.f;
  const uint32_t g = word & AJ_COUNT;
  if ((word & ~AJ_BIAS) != 0 && p.rep) {
    const float f = x > 0.f ? p.inv : p.rho, d = x > 0.f ? p.inv_lo : 0.f;
    const float y = x * f;
    lo = fmaf(x, f, -y) + x * d;
    hi = y + lo;
    lo = (y - hi) + lo;
  }
  if (g) {
    const float n = static_cast<float>(g), t = p.freq * n;
    add_pair(hi, lo, -t, -fmaf(p.freq, n, -t));
    add_pair(hi, lo, -p.pres, 0.f);
  }
  if (word & AJ_BIAS)
#pragma unroll 1
    for (int i = 0; i < p.n_bias; i += 4) {
      const int4 q = *reinterpret_cast<const int4*>(p.ids + i);
      if (q.x != id && q.y != id && q.z != id && q.w != id) continue;
      if (q.x == id) add_pair(hi, lo, __ldg(p.bias + i), 0.f);
      if (q.y == id) add_pair(hi, lo, __ldg(p.bias + i + 1), 0.f);
      if (q.z == id) add_pair(hi, lo, __ldg(p.bias + i + 2), 0.f);
      if (q.w == id) add_pair(hi, lo, __ldg(p.bias + i + 3), 0.f);
    }
  const float size = fabsf(hi);
  if (size > 7.9e-31f && size < 1.3e36f && fabsf(lo) <= size && g < (1u << 24)) store_value(o, hi, lo);
  else touch_double(o, x, word, id, p);
}
template <typename T>
__device__ __noinline__ void touch_double(T* o, float x, uint32_t word, int id, const Penalties& p) {
  double y = x;
  const uint32_t g = word & AJ_COUNT;
  if ((word & ~AJ_BIAS) != 0 && p.rep) y = y > 0 ? y / p.rho : y * p.rho;
  if (g) y -= static_cast<double>(p.freq) * g + p.pres;
  if (word & AJ_BIAS)
    for (int i = 0; i < p.n_bias; ++i)
      if (p.ids[i] == id) y += __ldg(p.bias + i);
  store_double(o, y);
}

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
    uint32_t* q = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // two bits to the tops of two bytes, each of which is then spread over a half
      uint32_t keep;
      asm("prmt.b32 %0, %1, 0, 0x9988;" : "=r"(keep) : "r"((bits >> (2 * i) & 3) * 0x4080u));
      q[i] = (q[i] & keep) | (0xff80ff80u & ~keep);
    }
    return v;
  }
}

// Writes tokens [t0, t0 + n) of a row with their mask: a piece of 16 KB, a warp's 32 * AJ_VECS vectors of it.
template <typename T, bool INPLACE>
struct Piece {
  static constexpr int E = 16 / sizeof(T);
  uint4 w[AJ_VECS];
  uint32_t bits[AJ_VECS];  // of a vector's elements
  const T* x;
  T* o;
  const uint32_t* m;
  int t0, n, head, vecs;  // elements before the first whole vector; vectors
  bool same;              // whether input and output lie alike to the 16-byte grid

  __device__ __forceinline__ Piece(const T* x_, T* o_, const uint32_t* m_, int words, int t0_, int n_) : x(x_), o(o_), m(m_), t0(t0_), n(n_) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uintptr_t ax = reinterpret_cast<uintptr_t>(x), ao = reinterpret_cast<uintptr_t>(o);
    same = INPLACE || ax % 16 == ao % 16;
    head = min(n, static_cast<int>((16 - ao % 16) % 16 / sizeof(T)));
    vecs = (n - head) / E;
    if (!same || (INPLACE && !m)) return;
    const int first = warp * 32 * AJ_VECS;
    uint32_t block = ~0u;
    if (m && first < vecs) block = mask_block(m, words, t0 + head + first * E, lane);
#pragma unroll
    for (int i = 0; i < AJ_VECS; ++i) {
      const int v = first + i * 32 + lane;
      bits[i] = __shfl_sync(FULL_MASK, block, (i * 32 + lane) * E / 32) >> (lane * E & 31) & ((1u << E) - 1);
      w[i] = make_uint4(0u, 0u, 0u, 0u);
      if (v < vecs && bits[i] != 0 && !(INPLACE && bits[i] == (1u << E) - 1)) w[i] = *reinterpret_cast<const uint4*>(x + head + v * E);
    }
  }
  __device__ __forceinline__ void write() const {
    if (INPLACE && !m) return;
    if (!same) {  // rows that lie differently to the 16-byte grid
      for (int t = threadIdx.x; t < n; t += AJ_THREADS) o[t] = !m || allowed(m, t0 + t) ? x[t] : minus_inf<T>();
      return;
    }
    const int lane = threadIdx.x & 31, first = (threadIdx.x >> 5) * 32 * AJ_VECS;
#pragma unroll
    for (int i = 0; i < AJ_VECS; ++i) {
      const int v = first + i * 32 + lane;
      if (v < vecs && !(INPLACE && bits[i] == (1u << E) - 1)) *reinterpret_cast<uint4*>(o + head + v * E) = m ? masked<T>(w[i], bits[i]) : w[i];
    }
    const int tail = head + vecs * E, ends = head + n - tail;
    if (static_cast<int>(threadIdx.x) < ends) {
      const int t = threadIdx.x < head ? threadIdx.x : tail + threadIdx.x - head;
      if (m && !allowed(m, t0 + t)) o[t] = minus_inf<T>();
      else if (!INPLACE) o[t] = x[t];
    }
  }
};

template <typename T, bool INPLACE, bool TOUCH>
__global__ void __launch_bounds__(AJ_THREADS, AJ_CTAS) adjust_kernel(const AdjustParams p) {
  constexpr int TOKENS = AJ_PIECE / sizeof(T), SPAN = TOUCH ? 1 : AJ_SPAN;
  __shared__ __align__(16) uint32_t s_word[TOUCH ? TOKENS : 4];
  __shared__ uint32_t s_touched[TOUCH ? TOKENS / 32 : 1];  // a bit a token
  __shared__ __align__(16) int s_id[TOUCH ? AJ_MAX_BIAS : 4];
  const int tid = threadIdx.x;
  const int64_t r = blockIdx.x / p.pieces;
  const int first = static_cast<int>(blockIdx.x - r * p.pieces) * TOKENS * SPAN;
  const int64_t h = r / p.per;
  const int words = (p.V + 31) >> 5;
  int seen = 0, from = 0, mi = -1;
  bool ok = true;
  if (TOUCH && p.hist) {
    seen = __ldg(p.seen + r);
    from = p.from ? __ldg(p.from + h) : 0;
    if (seen < 0 || seen > p.cap) {
      if (tid == 0) atomicOr(&g_err_adjust, ERR_KV8_LENGTH);
      ok = false;
    }
  }
  if (p.mask) {
    mi = p.mask_index ? __ldg(p.mask_index + r) : static_cast<int>(r);
    if (mi >= p.n_masks) {
      if (tid == 0) atomicOr(&g_err_adjust, ERR_MASK_INDEX);
      ok = false;
    }
  }
  if (!ok) return;  // the row is left out
  const uint32_t* m = mi >= 0 ? p.mask + mi * p.mask_stride : nullptr;
  const T* x = static_cast<const T*>(p.x) + r * p.x_stride;
  T* o = static_cast<T*>(p.out) + r * p.out_stride;
  if constexpr (!TOUCH) {
#pragma unroll 1
    for (int t0 = first; t0 < min(p.V, first + TOKENS * SPAN); t0 += TOKENS)
      Piece<T, INPLACE>(x + t0, o + t0, m, words, t0, min(TOKENS, p.V - t0)).write();
  } else {
    const int t0 = first, n = min(TOKENS, p.V - t0);
    const Piece<T, INPLACE> piece(x + t0, o + t0, m, words, t0, n);
    for (int i = tid * 4; i < n; i += AJ_THREADS * 4) *reinterpret_cast<uint4*>(s_word + i) = make_uint4(0u, 0u, 0u, 0u);
    for (int i = tid; i < TOKENS / 32; i += AJ_THREADS) s_touched[i] = 0;
    // (an id that is no token's is none of the piece's)
    for (int i = tid; i < (p.n_bias + 3) / 4 * 4; i += AJ_THREADS) {
      const int id = i < p.n_bias ? __ldg(p.bias_id + h * p.n_bias + i) : -1;
      s_id[i] = id < t0 || id - t0 >= n ? -1 : id - t0;
    }
    __syncthreads();
    auto count = [&](int id, int i) {
      const uint32_t at = static_cast<uint32_t>(id - t0);
      if (at < static_cast<uint32_t>(n)) {
        if (i >= from) atomicAdd(s_word + at, 1u);
        else atomicOr(s_word + at, AJ_SEEN);
        atomicOr(s_touched + (at >> 5), 1u << (at & 31));
      }
    };
    const int32_t* hist = p.hist + h * p.hist_stride;
    // (by fours from the first 16-byte boundary on)
    const int lead = min(seen, static_cast<int>((16 - reinterpret_cast<uintptr_t>(hist) % 16) % 16 / 4)), fours = (seen - lead) / 4;
    if (tid < lead) count(__ldg(hist + tid), tid);
    if (tid < seen - lead - 4 * fours) count(__ldg(hist + lead + 4 * fours + tid), lead + 4 * fours + tid);
#pragma unroll 4
    for (int f = tid; f < fours; f += AJ_THREADS) {
      const int i = lead + 4 * f;
      const int4 q = __ldg(reinterpret_cast<const int4*>(hist + i));
      count(q.x, i);
      count(q.y, i + 1);
      count(q.z, i + 2);
      count(q.w, i + 3);
    }
    for (int i = tid; i < p.n_bias; i += AJ_THREADS)
      if (s_id[i] >= 0) {
        atomicOr(s_word + s_id[i], AJ_BIAS);
        atomicOr(s_touched + (s_id[i] >> 5), 1u << (s_id[i] & 31));
      }
    piece.write();
    __syncthreads();
    // the touched ones among the lane's 32 tokens that may be taken
    uint32_t todo = 0;
    if (tid < TOKENS / 32) {
      todo = s_touched[tid];
      if (m && todo) todo &= __ldg(m + (t0 >> 5) + tid);
    }
    if (!__any_sync(FULL_MASK, todo != 0)) return;
    Penalties pen{p.rep ? __ldg(p.rep + h) : 1.f, 0.f, 0.f, p.freq ? __ldg(p.freq + h) : 0.f, p.pres ? __ldg(p.pres + h) : 0.f,
                  p.rep != nullptr, s_id, p.bias + h * p.n_bias, p.n_bias};
    pen.inv = 1.f / pen.rho;
    pen.inv_lo = fmaf(-pen.inv, pen.rho, 1.f) * pen.inv;
    for (; todo; todo &= todo - 1) {
      const int t = 32 * tid + __ffs(todo) - 1;
      touch(o + t0 + t, static_cast<float>(x[t0 + t]), s_word[t], t, pen);
    }
  }
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

template <typename T>
cudaError_t adjust_launch(const AdjustParams& p, int64_t rows, bool touch, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(rows * p.pieces));
  auto go = [&](auto kernel) { kernel<<<grid, AJ_THREADS, 0, stream>>>(p); };
  const bool inplace = p.x == p.out;
  if (touch) inplace ? go(adjust_kernel<T, true, true>) : go(adjust_kernel<T, false, true>);
  else inplace ? go(adjust_kernel<T, true, false>) : go(adjust_kernel<T, false, false>);
  note_launch();
  return cudaGetLastError();
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
  if (a->logits == a->out ? a->row_stride != a->out_stride
                          : x < o + uintptr_t((a->rows - 1) * a->out_stride + a->V) * es &&
                                o < x + uintptr_t((a->rows - 1) * a->row_stride + a->V) * es)
    return bad("lilicorr_adjust_logits: out is the logits themselves, or shares nothing with them");
  if (a->groups < 1 || a->rows % a->groups) return bad("lilicorr_adjust_logits: groups divides rows");
  if (a->history && (!a->seen || a->cap < 1 || a->cap >= 1 << 30 || a->history_stride < a->cap || a->history_stride > LIM))
    return bad("lilicorr_adjust_logits: history needs seen, a capacity below 2^30 and a stride of at least it");
  if (!a->history && (a->repetition || a->presence || a->frequency || a->counted_from))
    return bad("lilicorr_adjust_logits: penalties need a history");
  if (a->n_bias < 0 || a->n_bias > AJ_MAX_BIAS || (a->n_bias > 0 && (!a->bias_id || !a->bias)))
    return bad("lilicorr_adjust_logits: at most 1024 biases, with ids and values");
  if (a->mask && (a->n_masks < 1 || a->n_masks > INT_MAX || a->mask_stride < (a->V + 31) / 32 || a->mask_stride > LIM ||
                  (!a->mask_index && a->n_masks < a->rows)))
    return bad("lilicorr_adjust_logits: masks have (V + 31) / 32 words, one for each row or an index");
  if (!a->mask && a->mask_index) return bad("lilicorr_adjust_logits: an index needs masks");
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
  const int64_t tokens = int64_t(AJ_PIECE / es) * (touch ? 1 : AJ_SPAN);
  p.pieces = static_cast<int>((a->V + tokens - 1) / tokens);
  if (a->rows * p.pieces > INT_MAX) return bad("lilicorr_adjust_logits: rows * V is too large for one call");
  const cudaError_t e = es == 2 ? adjust_launch<__nv_bfloat16>(p, a->rows, touch, static_cast<cudaStream_t>(stream))
                                : adjust_launch<float>(p, a->rows, touch, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(LILICORR_ERR_CUDA, cudaGetErrorString(e));
  return LILICORR_OK;
}
