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
// and biases may all but cancel, so it is done in 64 bits and rounded once.
//
// One CTA for each piece of AJ_TOKENS tokens of a row.  It counts the history's tokens that lie in its
// piece in shared memory, a word a token (integer sums: any order gives the same), while the piece's
// logits are on their way; writes the logits with the mask; and then writes the touched tokens over.
constexpr int AJ_THREADS = 256;
constexpr int AJ_TOKENS = 8192;
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
__device__ __forceinline__ void store_double(float* p, double y) { *p = static_cast<float>(y); }
__device__ __forceinline__ void store_double(__nv_bfloat16* p, double y) { *p = __double2bfloat16(y); }

// Bits of the 32 tokens from t on (t >= 0), of a mask row of `words` words.
__device__ __forceinline__ uint32_t mask_bits(const uint32_t* m, int words, int t) {
  const int w = t >> 5;
  const uint32_t lo = __ldg(m + w), hi = w + 1 < words ? __ldg(m + w + 1) : 0u;
  return __funnelshift_r(lo, hi, t & 31);
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
      const uint32_t b = bits >> (2 * i);
      const uint32_t keep = (b & 1 ? 0xffffu : 0u) | (b & 2 ? 0xffff0000u : 0u);
      q[i] = (q[i] & keep) | (0xff80ff80u & ~keep);
    }
    return v;
  }
}

template <typename T, bool INPLACE>
__global__ void __launch_bounds__(AJ_THREADS) adjust_kernel(const AdjustParams p) {
  constexpr int E = 16 / sizeof(T), VECS = 4;
  __shared__ __align__(16) uint32_t s_word[AJ_TOKENS];
  __shared__ int s_id[AJ_MAX_BIAS];
  const int tid = threadIdx.x;
  const int64_t r = blockIdx.x / p.pieces;
  const int t0 = static_cast<int>(blockIdx.x - r * p.pieces) * AJ_TOKENS, n = min(AJ_TOKENS, p.V - t0);
  const int64_t h = r / p.per;
  const int words = (p.V + 31) >> 5;
  int seen = 0, from = 0, mi = -1;
  bool ok = true;
  if (p.hist) {
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
  const T* x = static_cast<const T*>(p.x) + r * p.x_stride + t0;
  T* o = static_cast<T*>(p.out) + r * p.out_stride + t0;

  // counts
  const bool touched = seen > 0 || p.n_bias > 0;
  if (touched) {
    for (int i = tid * 4; i < n; i += AJ_THREADS * 4) *reinterpret_cast<uint4*>(s_word + i) = make_uint4(0u, 0u, 0u, 0u);
    for (int i = tid; i < p.n_bias; i += AJ_THREADS) s_id[i] = __ldg(p.bias_id + h * p.n_bias + i);
    __syncthreads();
    const int32_t* hist = p.hist + h * p.hist_stride;
    for (int i = tid; i < seen; i += AJ_THREADS) {
      const int at = __ldg(hist + i) - t0;
      if (static_cast<uint32_t>(at) < static_cast<uint32_t>(n)) {
        if (i >= from) atomicAdd(s_word + at, 1u);
        else atomicOr(s_word + at, AJ_SEEN);
      }
    }
    for (int i = tid; i < p.n_bias; i += AJ_THREADS) {
      const int at = s_id[i] - t0;
      if (static_cast<uint32_t>(at) < static_cast<uint32_t>(n)) atomicOr(s_word + at, AJ_BIAS);
    }
  }

  // the row with its mask
  if (!INPLACE || m) {
    const uintptr_t ax = reinterpret_cast<uintptr_t>(x), ao = reinterpret_cast<uintptr_t>(o);
    if (ax % 16 == ao % 16) {
      const int head = min(n, static_cast<int>((16 - ao % 16) % 16 / sizeof(T))), vecs = (n - head) / E;
      for (int v0 = 0; v0 < vecs; v0 += AJ_THREADS * VECS) {
        uint4 w[VECS];
        uint32_t bits[VECS];
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
          const int v = v0 + i * AJ_THREADS + tid;
          bits[i] = ~0u;
          w[i] = make_uint4(0u, 0u, 0u, 0u);
          if (v >= vecs) continue;
          if (m) bits[i] = mask_bits(m, words, t0 + head + v * E) & ((1u << E) - 1);
          const bool need = INPLACE ? bits[i] != 0 && bits[i] != (1u << E) - 1 : bits[i] != 0;
          if (need) w[i] = *reinterpret_cast<const uint4*>(x + head + v * E);
        }
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
          const int v = v0 + i * AJ_THREADS + tid;
          if (v >= vecs || (INPLACE && bits[i] == (1u << E) - 1)) continue;
          *reinterpret_cast<uint4*>(o + head + v * E) = masked<T>(w[i], bits[i]);
        }
      }
      // the ends
      const int tail = head + vecs * E, ends = head + n - tail;
      if (tid < ends) {
        const int t = tid < head ? tid : tail + tid - head;
        const bool on = !m || (mask_bits(m, words, t0 + t) & 1);
        if (!on) o[t] = minus_inf<T>();
        else if (!INPLACE) o[t] = x[t];
      }
    } else {  // rows that lie differently to the 16-byte grid
      for (int t = tid; t < n; t += AJ_THREADS)
        o[t] = !m || (mask_bits(m, words, t0 + t) & 1) ? x[t] : minus_inf<T>();
    }
  }
  if (!touched) return;
  __syncthreads();
  const double rho = p.rep ? __ldg(p.rep + h) : 1.0, pres = p.pres ? __ldg(p.pres + h) : 0.0,
               freq = p.freq ? __ldg(p.freq + h) : 0.0;
  for (int t = tid; t < n; t += AJ_THREADS) {
    const uint32_t w = s_word[t];
    if (w == 0 || (m && !(mask_bits(m, words, t0 + t) & 1))) continue;
    double y = static_cast<float>(x[t]);
    if ((w & ~AJ_BIAS) != 0 && p.rep) y = y > 0 ? y / rho : y * rho;
    const uint32_t g = w & AJ_COUNT;
    if (g) y -= freq * g + pres;
    if (w & AJ_BIAS)
      for (int i = 0; i < p.n_bias; ++i)
        if (s_id[i] == t0 + t) y += __ldg(p.bias + h * p.n_bias + i);
    store_double(o + t, y);
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
cudaError_t adjust_launch(const AdjustParams& p, int64_t rows, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(rows * p.pieces));
  if (p.x == p.out) adjust_kernel<T, true><<<grid, AJ_THREADS, 0, stream>>>(p);
  else adjust_kernel<T, false><<<grid, AJ_THREADS, 0, stream>>>(p);
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
  if (a->rows < 1 || a->rows > INT_MAX || a->V < 1 || a->V > INT_MAX - 65536 || a->row_stride < a->V || a->row_stride > LIM ||
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
  p.pieces = static_cast<int>((a->V + AJ_TOKENS - 1) / AJ_TOKENS);
  if (a->rows * p.pieces > INT_MAX) return bad("lilicorr_adjust_logits: rows * V is too large for one call");
  const cudaError_t e = es == 2 ? adjust_launch<__nv_bfloat16>(p, a->rows, static_cast<cudaStream_t>(stream))
                                : adjust_launch<float>(p, a->rows, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(LILICORR_ERR_CUDA, cudaGetErrorString(e));
  return LILICORR_OK;
}
