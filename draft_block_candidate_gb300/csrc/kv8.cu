// A paged key / value cache held in 8 bits (e4m3) with one scale for each page (block of
// tokens) and key / value head: its writer, and the attention that reads it.
#include <algorithm>
#include <cmath>

#include "kv8.cuh"

namespace lilicorr {

static __device__ uint32_t g_err_kv8;

// ---------------------------------------------------------------------------- the writer
// One CTA per (sequence, page that grows, head, K or V).  The page's scale is the smallest
// power of two 2^k >= 2^-60 that holds its new rows' largest finite magnitude within 448,
// or the scale that the page has from its earlier rows where that is larger.  A power of two
// costs e4m3 nothing in relative precision, and lets a page's earlier codes move to a larger
// scale exactly (but for e4m3's subnormals), so appending tokens one by one leaves what
// appending them at once does.  Bound by HBM for prompts (2 bytes in and 1 out per value),
// by latency for single tokens.  The rows are kept in registers between the maximum and the
// conversion, so that they are read once, and are loaded before the table's entry is known.
// Prompts of up to 4,096 tokens, 16 sequences, 8 heads of 128: 34 us, 5.6 TB/s, 82 to 84 % of the
// copy rate (51 us with divisions for the rows' places, f32 maxima and a test of the scale at each
// value).  64 sequences' single tokens: 4.1 us, of which a
// launch and two dependent reads are all but a little.
constexpr int AP_THREADS = 128;

struct AppendParams {
  Kv8 c;
  const __nv_bfloat16 *k, *v;
  int64_t k_tok, k_head, v_tok, v_head;  // elements
  int64_t total;
  const int32_t *q_start, *kv_len, *table, *tail_src;
  int64_t table_stride;
  int cols;      // pages of a table row
  int max_new, grow;  // pages a sequence can touch in one call
  int page_log2, row_log2;  // of a page's tokens, and of a row's vectors of 8 values
};

// 2^k as above, from the bits of the largest magnitude (finite, >= 0).
__device__ __forceinline__ float page_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  // amax = m 2^e with m in [0.5, 1); 448 = 0.875 * 2^9
  int k = static_cast<int>(u >> 23) - 126 - 9 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  k = max(k, -60);
  return __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
}

template <int VPT>  // 8-element vectors a thread holds of a page
__global__ void __launch_bounds__(AP_THREADS) kv8_append_kernel(const AppendParams p) {
  __shared__ uint32_t s_max[AP_THREADS / 32];
  const int tid = threadIdx.x;
  int64_t u = blockIdx.x;
  const int which = static_cast<int>(u & 1);
  u >>= 1;
  const int h = static_cast<int>(u % p.c.heads);
  u /= p.c.heads;
  const int g = static_cast<int>(u % p.grow);
  const int64_t b = u / p.grow;
  const int page = p.c.page, D = 8 << p.row_log2;
  const SeqRange r = seq_range(p.q_start, p.kv_len, b, p.total, p.max_new,
                               int64_t(p.cols) << p.page_log2, &g_err_kv8);
  const int before = r.len - r.n;
  if (r.n == 0) return;
  if (before < 0) {
    if (tid == 0) atomicOr(&g_err_kv8, ERR_KV8_LENGTH);
    return;
  }
  const int at = (before >> p.page_log2) + g;  // this page's column of the table
  if (int64_t(at) << p.page_log2 >= r.len) return;
  const int pos0 = at << p.page_log2;
  const int id = __ldg(p.table + b * p.table_stride + at);
  const bool has_old = pos0 < before;
  int src = has_old && p.tail_src ? __ldg(p.tail_src + b) : -1;

  // the new rows, which wait for no table entry
  const __nv_bfloat16* x = (which ? p.v : p.k) + h * (which ? p.v_head : p.k_head);
  const int64_t tok = which ? p.v_tok : p.k_tok;
  const int vrow = 1 << p.row_log2;
  const int lo_row = max(before - pos0, 0), hi_row = min(r.len - pos0, page);  // of the page
  const int64_t row0 = r.q0 + pos0 - before;
  uint4 w[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int e = tid + i * AP_THREADS, row = e >> p.row_log2;
    w[i] = make_uint4(0u, 0u, 0u, 0u);
    if (row >= lo_row && row < hi_row)
      w[i] = __ldcs(reinterpret_cast<const uint4*>(x + (row0 + row) * tok + (e & (vrow - 1)) * 8));
  }
  if (src < 0) src = id;
  if (id < 0 || id >= p.c.n_pages || src >= p.c.n_pages) {
    if (tid == 0) atomicOr(&g_err_kv8, ERR_KV8_PAGE);
    return;
  }
  uint8_t* codes = (which ? p.c.v : p.c.k) + (int64_t(id) * p.c.heads + h) * page * D;
  float* scales = which ? p.c.vs : p.c.ks;
  const float was = has_old ? __ldcg(scales + int64_t(src) * p.c.heads + h) : 0.f;

  // The largest magnitude, in bf16 (NaN is passed over); infinities are looked for where it is one.
  __nv_bfloat162 top2 = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const uint32_t q[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) top2 = __hmax2(top2, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&q[j])));
  }
  float amax = fmaxf(__low2float(top2), __high2float(top2));
  if (isinf(amax)) {
    uint32_t top = 0;  // bits of the largest finite magnitude
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const uint32_t q[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo = q[j] & 0x7fffu, hi = (q[j] >> 16) & 0x7fffu;
        if (lo < 0x7f80u) top = max(top, lo);
        if (hi < 0x7f80u) top = max(top, hi);
      }
    }
    amax = __uint_as_float(top << 16);
  }
  // (magnitudes compare as their bits do)
  uint32_t top = __reduce_max_sync(FULL_MASK, __float_as_uint(amax));
  if ((tid & 31) == 0) s_max[tid >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < AP_THREADS / 32; ++i) top = max(top, s_max[i]);
  const float now = fmaxf(page_scale(__uint_as_float(top)), was);
  const float inv = 1.f / now;
  // a scale of the caller's own need not be a power of two; then the quotient is divided out
  const bool pow2 = (__float_as_uint(now) & 0x7fffffu) == 0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int e = tid + i * AP_THREADS, row = e >> p.row_log2;
    if (row >= lo_row && row < hi_row) {
      const uint32_t q[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
      uint16_t o[4];
      if (pow2) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          o[j] = f32x2_to_e4m3x2(__uint_as_float(q[j] << 16) * inv, __uint_as_float(q[j] & 0xffff0000u) * inv);
      } else {
#pragma unroll 1
        for (int j = 0; j < 4; ++j) {
          const uint32_t z = j == 0 ? q[0] : j == 1 ? q[1] : j == 2 ? q[2] : q[3];
          const uint16_t c = f32x2_to_e4m3x2(__uint_as_float(z << 16) / now, __uint_as_float(z & 0xffff0000u) / now);
          if (j == 0) o[0] = c; else if (j == 1) o[1] = c; else if (j == 2) o[2] = c; else o[3] = c;
        }
      }
      *reinterpret_cast<uint2*>(codes + int64_t(e) * 8) =
          make_uint2(o[0] | uint32_t(o[1]) << 16, o[2] | uint32_t(o[3]) << 16);
    }
  }
  // Earlier rows: moved to the larger scale, or copied from the page they lie in.
  if (has_old && (src != id || now != was)) {
    const uint8_t* from = (which ? p.c.v : p.c.k) + (int64_t(src) * p.c.heads + h) * page * D;
    const float f = was / now;
    const int nold = min(before - pos0, page) << p.row_log2;
    for (int e = tid; e < nold; e += AP_THREADS) {
      uint2 c = *reinterpret_cast<const uint2*>(from + int64_t(e) * 8);
      if (now != was) {
        uint32_t q[2] = {c.x, c.y};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t a = e4m3x2_to_f16x2(static_cast<uint16_t>(q[j]));
          const uint32_t d = e4m3x2_to_f16x2(static_cast<uint16_t>(q[j] >> 16));
          const float2 fa = __half22float2(*reinterpret_cast<const __half2*>(&a));
          const float2 fd = __half22float2(*reinterpret_cast<const __half2*>(&d));
          q[j] = f32x2_to_e4m3x2(fa.x * f, fa.y * f) |
                 uint32_t(f32x2_to_e4m3x2(fd.x * f, fd.y * f)) << 16;
        }
        c = make_uint2(q[0], q[1]);
      }
      *reinterpret_cast<uint2*>(codes + int64_t(e) * 8) = c;
    }
  }
  // (the old scale was read before the barrier above)
  if (tid == 0) scales[int64_t(id) * p.c.heads + h] = now;
}

cudaError_t kv8_read_device_error(uint32_t* code) {
  uint32_t v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_err_kv8, sizeof(v));
  if (e != cudaSuccess) return e;
  if (v) e = cudaMemcpyToSymbol(g_err_kv8, &zero, sizeof(zero));
  *code |= v;
  return e == cudaSuccess ? kv8_attention_read_device_error(code) : e;
}

namespace {

lilicorr_status fail(lilicorr_status st, const char* msg) {
  set_last_error(msg);
  return st;
}

// Null where the cache's description is in order, else what is wrong with it.
const char* cache_error(const lilicorr_kv8_cache* c) {
  if (!c || !c->k_pages || !c->v_pages || !c->k_scale || !c->v_scale) return "null cache pointer";
  if (c->head_dim != 32 && c->head_dim != 64 && c->head_dim != 128) return "head_dim is 32, 64 or 128";
  if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) return "page is 16, 32, 64 or 128";
  if (c->kv_heads < 1 || c->kv_heads > 1024) return "1 <= kv_heads <= 1024";
  if (c->n_pages < 1 || c->n_pages > INT_MAX) return "1 <= n_pages < 2^31";
  if (reinterpret_cast<uintptr_t>(c->k_pages) % 16 || reinterpret_cast<uintptr_t>(c->v_pages) % 16)
    return "pages are 16-byte aligned";
  if (reinterpret_cast<uintptr_t>(c->k_scale) % 4 || reinterpret_cast<uintptr_t>(c->v_scale) % 4)
    return "scales are 4-byte aligned";
  return nullptr;
}
const char* batch_error(const int32_t* q_start, const int32_t* kv_len, int64_t batch,
                        const int32_t* table, int64_t table_stride, int32_t cols, int64_t total,
                        int32_t max_new, int page) {
  if (!q_start || !kv_len || !table) return "null pointer";
  if (batch < 1 || batch > (1 << 20)) return "1 <= batch <= 2^20";
  if (cols < 1 || int64_t(cols) * page > INT_MAX - 256) return "a table row holds 1 page to 2^31 tokens";
  if (table_stride < cols) return "table_stride is at least its columns";
  if (total < 0 || total > INT_MAX) return "rows are out of range";
  if (max_new < 1 || max_new > (1 << 24)) return "1 <= max_new <= 2^24";
  return nullptr;
}
const char* rows_error(const void* x, int64_t tok, int64_t head) {
  if (!x) return "null pointer";
  if (reinterpret_cast<uintptr_t>(x) % 16) return "rows are 16-byte aligned";
  if (tok % 8 || head % 8) return "row strides are multiples of 8 elements";
  if (tok < 0 || head < 0 || tok > (int64_t(1) << 40) || head > (int64_t(1) << 40)) return "a row stride is out of range";
  return nullptr;
}
// Whether [a, a + n) and [b, b + m) share a byte.
bool overlap(const void* a, unsigned __int128 n, const void* b, unsigned __int128 m) {
  const unsigned __int128 x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + m && y < x + n;
}
Kv8 view(const lilicorr_kv8_cache* c) {
  return Kv8{static_cast<uint8_t*>(c->k_pages), static_cast<uint8_t*>(c->v_pages), c->k_scale,
             c->v_scale, c->n_pages, c->kv_heads, c->page};
}

}  // namespace
}  // namespace lilicorr

using namespace lilicorr;

extern "C" {

lilicorr_status lilicorr_kv8_append(const lilicorr_kv8_cache* cache, const void* k,
                                    int64_t k_token_stride, int64_t k_head_stride, const void* v,
                                    int64_t v_token_stride, int64_t v_head_stride, int64_t total,
                                    const int32_t* q_start, const int32_t* kv_len, int64_t batch,
                                    const int32_t* block_table, int64_t table_stride, int32_t cols,
                                    int32_t max_new, const int32_t* tail_src, void* stream) {
  const char* why = cache_error(cache);
  if (!why) why = batch_error(q_start, kv_len, batch, block_table, table_stride, cols, total, max_new, cache->page);
  if (!why) why = rows_error(k, k_token_stride, k_head_stride);
  if (!why) why = rows_error(v, v_token_stride, v_head_stride);
  if (why) return fail(LILICORR_ERR_INVALID_ARG, why);
  AppendParams prm{};
  prm.c = view(cache);
  prm.k = static_cast<const __nv_bfloat16*>(k);
  prm.v = static_cast<const __nv_bfloat16*>(v);
  prm.k_tok = k_token_stride; prm.k_head = k_head_stride;
  prm.v_tok = v_token_stride; prm.v_head = v_head_stride;
  prm.total = total;
  prm.q_start = q_start; prm.kv_len = kv_len; prm.table = block_table; prm.tail_src = tail_src;
  prm.table_stride = table_stride;
  prm.cols = cols;
  prm.max_new = max_new;
  const int page = cache->page, D = cache->head_dim;
  while ((1 << prm.page_log2) < page) ++prm.page_log2;
  while ((8 << prm.row_log2) < D) ++prm.row_log2;
  prm.grow = std::min<int>((max_new + page - 2) / page + 1, cols);
  const int64_t ctas = batch * prm.grow * cache->kv_heads * 2;
  if (ctas > INT_MAX) return fail(LILICORR_ERR_INVALID_ARG, "batch * max_new * kv_heads is too large for one call");
  const int vpt = (page * D / 8 + AP_THREADS - 1) / AP_THREADS;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dim3 grid(static_cast<unsigned>(ctas));
  if (vpt <= 1) kv8_append_kernel<1><<<grid, AP_THREADS, 0, st>>>(prm);
  else if (vpt <= 2) kv8_append_kernel<2><<<grid, AP_THREADS, 0, st>>>(prm);
  else if (vpt <= 4) kv8_append_kernel<4><<<grid, AP_THREADS, 0, st>>>(prm);
  else if (vpt <= 8) kv8_append_kernel<8><<<grid, AP_THREADS, 0, st>>>(prm);
  else kv8_append_kernel<16><<<grid, AP_THREADS, 0, st>>>(prm);
  note_launch();
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(LILICORR_ERR_CUDA, cudaGetErrorString(e));
  return LILICORR_OK;
}

size_t lilicorr_kv8_attention_workspace_bytes(int32_t max_new, int32_t q_heads, int32_t kv_heads,
                                              int32_t head_dim) {
  if (max_new < 1 || max_new > (1 << 24) || kv_heads < 1 || kv_heads > 1024 || q_heads < kv_heads ||
      q_heads % kv_heads || q_heads / kv_heads > 1024 ||
      int64_t(max_new) * (q_heads / kv_heads) > INT_MAX - 256 ||
      (head_dim != 32 && head_dim != 64 && head_dim != 128))
    return 0;
  return kv8_attention_workspace(max_new, q_heads / kv_heads, head_dim);
}

lilicorr_status lilicorr_kv8_attention(const lilicorr_kv8_cache* cache, const void* q,
                                       int64_t q_token_stride, int64_t q_head_stride,
                                       int64_t total, int32_t q_heads, const int32_t* q_start,
                                       const int32_t* kv_len, int64_t batch,
                                       const int32_t* block_table, int64_t table_stride,
                                       int32_t cols, int32_t max_new, float scale, void* out,
                                       float* lse, void* workspace, size_t workspace_bytes,
                                       void* stream) {
  const char* why = cache_error(cache);
  if (!why) why = batch_error(q_start, kv_len, batch, block_table, table_stride, cols, total, max_new, cache->page);
  if (!why) why = rows_error(q, q_token_stride, q_head_stride);
  if (!why && (!out || reinterpret_cast<uintptr_t>(out) % 16)) why = "out is null or not 16-byte aligned";
  if (!why && (q_heads < 1 || q_heads % cache->kv_heads || q_heads / cache->kv_heads > 1024))
    why = "q_heads is a multiple of kv_heads, at most 1024 times it";
  // a sequence's rows, and its work units (tiles x heads x chunks of tokens, and some for
  // each tile), are counted in 32 bits
  if (!why && int64_t(max_new) * (q_heads / cache->kv_heads) > INT_MAX - 256)
    why = "max_new * q_heads / kv_heads is too large";
  if (!why && (int64_t(max_new) * (q_heads / cache->kv_heads) / 8 + 1) * cache->kv_heads *
                  ((int64_t(cols) * cache->page + 127) / 128 + 4) > UINT_MAX)
    why = "max_new * q_heads * the table's tokens are too large";
  if (!why && !std::isfinite(scale)) why = "scale is not finite";
  if (why) return fail(LILICORR_ERR_INVALID_ARG, why);
  const int D = cache->head_dim, group = q_heads / cache->kv_heads;
  if (!workspace || workspace_bytes < kv8_attention_workspace(max_new, group, D) ||
      reinterpret_cast<uintptr_t>(workspace) % 256)
    return fail(LILICORR_ERR_WORKSPACE, "lilicorr_kv8_attention: workspace missing, too small or misaligned");
  if (total > 0) {
    // CTAs read q while others write what they are done with
    using wide = unsigned __int128;
    const wide rows = wide(total) * q_heads, o_bytes = rows * D * 2, l_bytes = lse ? rows * 4 : 0;
    const wide q_bytes = (wide(total - 1) * q_token_stride + wide(q_heads - 1) * q_head_stride + D) * 2;
    if (overlap(q, q_bytes, out, o_bytes) || (lse && (overlap(q, q_bytes, lse, l_bytes) || overlap(out, o_bytes, lse, l_bytes))))
      return fail(LILICORR_ERR_INVALID_ARG, "lilicorr_kv8_attention: q, out and lse overlap");
  }
  Kv8Attention a{};
  a.c = view(cache);
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.q_tok = q_token_stride; a.q_head = q_head_stride;
  a.total = total;
  a.q_heads = q_heads; a.group = group; a.D = D;
  a.q_start = q_start; a.kv_len = kv_len; a.table = block_table;
  a.batch = batch; a.table_stride = table_stride;
  a.cols = cols; a.max_new = max_new;
  a.scale = scale;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.workspace = workspace;
  const cudaError_t e = kv8_attention_launch(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(LILICORR_ERR_CUDA, cudaGetErrorString(e));
  return LILICORR_OK;
}

}  // extern "C"
