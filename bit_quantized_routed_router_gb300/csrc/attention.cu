// Attention of new tokens over paged keys and values: the entry point, and
// the kernel for every geometry.
#include "attention.h"

#include "common.cuh"
#include "errors.h"
#include "internal.h"
#include "kv8.cuh"
#include "serving.cuh"

namespace dsm {
namespace {

constexpr int GA_WARPS = 4;

template <bool BF16>
__device__ __forceinline__ float to_f32(uint16_t x) {
  return BF16 ? bf16_to_f32(x) : fp16_to_f32(x);
}
template <bool BF16>
__device__ __forceinline__ uint16_t from_f32(float x) {
  return BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x)) : __half_as_ushort(__float2half_rn(x));
}

// One block a query row (token, head), any strides and sizes: its warps take
// blocks of 32 keys in turn, a lane scores one key, and the lanes then share
// the head's elements of the second product.  Each warp keeps a running
// maximum and sum; the four are joined in order at the end.  Bound by the
// loads of keys, whose elements are read one at a time: the form for what the
// tensor-core kernels' copies do not take, not for speed (one token for each of
// 64 requests of 217 to 8138 keys, 8 key heads of 128: 4.8 ms, 30 times the
// decode kernel's).  Probabilities stay in 32 bits here.  E8: a cache in 8
// bits, whose elements are multiplied with their block's scale: keys' behind
// the product, values' with the probability.
template <bool BF16, bool E8>
__global__ void __launch_bounds__(GA_WARPS * 32) attention_generic_kernel(const AttnArgs a) {
  __shared__ float qs[128], acc_s[GA_WARPS][128], m_s[GA_WARPS], l_s[GA_WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  bool bad = false;
  for (int64_t row = blockIdx.x; row < (int64_t)a.T * a.H; row += gridDim.x) {
    const int t = (int)(row / a.H), h = (int)(row % a.H);
    // the last request that begins at or before t
    int r = 0, hi_r = a.R;
    while (hi_r - r > 1) {
      const int mid = (r + hi_r) >> 1;
      if (a.cu[mid] <= t) r = mid; else hi_r = mid;
    }
    const Span sp = request_span(a.cu, a.seq, r, a.T, a.max_new, a.max_seq, bad);
    if (t < sp.t0 || t >= sp.t0 + sp.n) continue;
    const int pos = sp.pos0 + t - sp.t0;
    const int hi = pos + 1, lo = a.window && hi > a.window ? hi - a.window : 0;  // keys [lo, hi)
    __syncthreads();
    for (int d = threadIdx.x; d < a.D; d += GA_WARPS * 32)
      qs[d] = to_f32<BF16>(a.q[t * a.qs + (int64_t)h * a.D + d]) * a.scale_log2;
    __syncthreads();
    float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    const int64_t head = (int64_t)(h / a.g) * a.hs;
    const uint8_t *k8 = reinterpret_cast<const uint8_t *>(a.k), *v8 = reinterpret_cast<const uint8_t *>(a.v);
    for (int j0 = (lo & ~31) + 32 * warp; j0 < hi; j0 += 32 * GA_WARPS) {
      const int j = j0 + lane;
      const bool sees = j >= lo && j < hi;
      int64_t at = -1;  // the key's row in the cache; -1: a page of zeros
      float s = -INFINITY, vs = 1.f;
      if (sees) {
        const int col = j / a.page;
        const int page = a.table[r * a.table_stride + col];
        if (page >= 0 && page < a.n_pages) at = page * a.ps + (int64_t)(j - col * a.page) * a.rs + head;
        else bad = true;
        s = 0.f;
        if (at >= 0 && !E8)
          for (int d = 0; d < a.D; ++d) s = fmaf(qs[d], to_f32<BF16>(a.k[at + d]), s);
        if (at >= 0 && E8) {
          for (int d = 0; d < a.D; ++d) s = fmaf(qs[d], f8x2_to(k8[at + d]).x, s);
          const int64_t scale = page * a.sps + (int64_t)((j - col * a.page) / a.block) * a.sbs + (int64_t)(h / a.g) * a.shs;
          s *= kv8_scale(a.ks[scale]);
          vs = kv8_scale(a.vs[scale]);
        }
      }
      float mx = s;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float mn = fmaxf(m, mx), ref = mn == -INFINITY ? 0.f : mn;
      const float p = sees ? exp2f(s - ref) : 0.f, keep = exp2f(m - ref);
      l = l * keep + warp_sum(p);
      m = mn;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] *= keep;
      const unsigned live = __ballot_sync(0xffffffffu, at >= 0);  // seen, and not a page of zeros
      for (int jj = 0; jj < 32; ++jj) {
        const float pj = __shfl_sync(0xffffffffu, E8 ? p * vs : p, jj);
        const int64_t aj = __shfl_sync(0xffffffffu, at, jj);
        if (!(live >> jj & 1u)) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (lane + 32 * i < a.D) acc[i] = fmaf(pj, E8 ? f8x2_to(v8[aj + lane + 32 * i]).x : to_f32<BF16>(a.v[aj + lane + 32 * i]), acc[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) acc_s[warp][lane + 32 * i] = acc[i];
    if (lane == 0) m_s[warp] = m, l_s[warp] = l;
    __syncthreads();
    float mm = m_s[0], ll = 0.f, w[GA_WARPS];
#pragma unroll
    for (int i = 1; i < GA_WARPS; ++i) mm = fmaxf(mm, m_s[i]);
    const float ref = mm == -INFINITY ? 0.f : mm;
#pragma unroll
    for (int i = 0; i < GA_WARPS; ++i) w[i] = exp2f(m_s[i] - ref), ll += w[i] * l_s[i];
    const int d = threadIdx.x;
    if (d < a.D) {
      float o = 0.f;
#pragma unroll
      for (int i = 0; i < GA_WARPS; ++i) o += w[i] * acc_s[i][d];
      a.out[t * a.os + (int64_t)h * a.D + d] = from_f32<BF16>(ll == 0.f ? 0.f : o / ll);
    }
    if (a.lse && threadIdx.x == 0) a.lse[row] = (ref + log2f(ll)) * 0.69314718055994531f;
  }
  if (bad) flag(a.status, ST_PAGING);
}

// What the tensor-core kernels' copies need: 16-byte aligned bases, strides
// and heads, and pages of whole 8-row groups (the swizzle's period).
bool copies_fit(const ds_moe_attn_shape &s, const ds_moe_kv_cache &c, const void *q, int64_t q_stride, int64_t T) {
  constexpr int64_t FAR = (int64_t)1 << 39;  // strides of a tensor map are below 2^40 bytes
  auto fits = [](int64_t n, int64_t stride) { return n <= 1 || (stride > 0 && stride % 8 == 0 && stride < FAR); };
  return s.head_dim % 8 == 0 && s.page_size % 8 == 0 && s.n_head / s.n_head_kv <= 128 && c.n_pages > 0 &&
         aligned(c.k, 16) && aligned(c.v, 16) && aligned(q, 16) && fits(s.page_size, c.row_stride) &&
         fits(s.n_head_kv, c.head_stride) && fits(c.n_pages, c.page_stride) && fits(T, q_stride) && encode_fn() && device_sms();
}

int path_of(const ds_moe_attn_shape &s, const ds_moe_kv_cache &c, const void *q, int64_t q_stride, int64_t T, int32_t max_new) {
  if (!copies_fit(s, c, q, q_stride, T)) return DS_ATTN_GENERIC;
  return (int64_t)max_new * (s.n_head / s.n_head_kv) <= AD_MAX_ROWS ? DS_ATTN_DECODE : DS_ATTN_CHUNK;
}

template <bool E8>
cudaError_t launch_generic(const AttnArgs &a, bool bf16, cudaStream_t s) {
  const int64_t rows = (int64_t)a.T * a.H;
  const unsigned blocks = (unsigned)std::min<int64_t>(rows, 1 << 20);
  if (bf16)
    attention_generic_kernel<true, E8><<<blocks, GA_WARPS * 32, 0, s>>>(a);
  else
    attention_generic_kernel<false, E8><<<blocks, GA_WARPS * 32, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

int attention_blocks() { return std::max(device_sms(), NUM_SMS); }

cudaError_t launch_attention_generic(const AttnArgs &a, bool bf16, cudaStream_t s) { return launch_generic<false>(a, bf16, s); }
cudaError_t launch_attention8_generic(const AttnArgs &a, bool bf16, cudaStream_t s) { return launch_generic<true>(a, bf16, s); }

int attention_args(const ds_moe_attn_shape &shape, size_t need, const int32_t *block_table, int32_t table_width,
                   int64_t table_stride, const void *q, int64_t q_stride, int64_t T, const int32_t *cu_new,
                   const int32_t *seq_lens, int32_t n_requests, int32_t max_new, void *out, int64_t out_stride, float *lse,
                   void *workspace, size_t workspace_bytes, AttnArgs *args, bool *nothing, char *err, size_t errlen) {
  if (table_width < 0) return fail(err, errlen, DS_ERR_INVALID_ARG, "table_width is negative");
  *nothing = T == 0 || n_requests == 0 || max_new == 0;
  if (*nothing) return DS_OK;
  if (n_requests > 1 && table_stride < table_width)
    return fail(err, errlen, DS_ERR_INVALID_ARG, "table_stride is smaller than table_width");
  if ((table_width && !block_table) || !q || !cu_new || !seq_lens || !out || !workspace)
    return fail(err, errlen, DS_ERR_INVALID_ARG, "block_table, q, cu_new, seq_lens, out and workspace are required");
  if (!aligned(q, 2) || !aligned(out, 2) || !aligned(lse, 4) || !aligned(block_table, 4) || !aligned(cu_new, 4) ||
      !aligned(seq_lens, 4))
    return fail(err, errlen, DS_ERR_INVALID_ARG, "arrays must be aligned to their elements");
  const int64_t row = (int64_t)shape.n_head * shape.head_dim;
  if (T > 1 && (q_stride < 0 || out_stride < row))
    return fail(err, errlen, DS_ERR_INVALID_ARG, "q_stride is negative, or out_stride smaller than a token's row");
  if (!aligned(workspace, 256)) return fail(err, errlen, DS_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if (workspace_bytes < need)
    return fail(err, errlen, DS_ERR_INVALID_ARG, "workspace too small: %zu < %zu bytes", workspace_bytes, need);
  AttnArgs &a = *args;
  a.table = block_table; a.width = table_width; a.table_stride = table_stride;
  a.q = (const uint16_t *)q; a.qs = q_stride;
  a.cu = cu_new; a.seq = seq_lens; a.T = (int)T; a.R = n_requests; a.max_new = max_new;
  a.out = (uint16_t *)out; a.os = out_stride; a.lse = lse;
  a.H = shape.n_head; a.G = shape.n_head_kv; a.g = a.H / a.G; a.D = shape.head_dim;
  a.page = shape.page_size;
  a.window = std::min(shape.window, 1 << 30);  // positions stay below 2^30, and sums of two in an int
  const float scale = shape.scale != 0.f ? shape.scale : (float)(1.0 / sqrt((double)a.D));
  a.scale_log2 = (float)((double)scale * 1.4426950408889634);
  a.max_seq = std::min<int64_t>((int64_t)table_width * a.page, 1 << 30);
  if (!(a.status = status_word())) return fail(err, errlen, DS_ERR_CUDA, "no CUDA device");
  return DS_OK;
}

}  // namespace dsm

using namespace dsm;

extern "C" {

int ds_moe_attention_path(const ds_moe_attn_shape *shape, const ds_moe_kv_cache *cache, const void *q,
                          int64_t q_stride, int32_t max_new) {
  if (check_attn_shape(shape, nullptr, 0) || check_kv_cache(shape, cache, false, nullptr, 0) || max_new < 0 || q_stride < 0)
    return DS_ERR_INVALID_ARG;
  return path_of(*shape, *cache, q, q_stride, 2, max_new);
}

int ds_moe_attention_workspace_bytes(const ds_moe_attn_shape *shape, int32_t n_requests, int64_t T, int32_t max_new,
                                     size_t *bytes, char *err, size_t errlen) {
  const int rc = check_attn_shape(shape, err, errlen);
  if (rc) return rc;
  if (!bytes) return fail(err, errlen, DS_ERR_INVALID_ARG, "bytes is NULL");
  if (n_requests < 0 || max_new < 0 || T < 0 || T > (1 << 24))
    return fail(err, errlen, DS_ERR_INVALID_ARG, "n_requests, T or max_new out of range");
  const int64_t rows = (int64_t)max_new * (shape->n_head / shape->n_head_kv);
  const size_t need = rows <= AD_MAX_ROWS ? attention_decode_workspace(rows, attention_blocks()) : attention_chunk_workspace(attention_blocks());
  *bytes = (need + 255) / 256 * 256;
  return DS_OK;
}

int ds_moe_paged_attention(const ds_moe_attn_shape *shape, const ds_moe_kv_cache *cache, const int32_t *block_table,
                           int32_t table_width, int64_t table_stride, const void *q, int64_t q_stride, int64_t T,
                           const int32_t *cu_new, const int32_t *seq_lens, int32_t n_requests, int32_t max_new,
                           void *out, int64_t out_stride, float *lse, void *workspace, size_t workspace_bytes,
                           void *stream, char *err, size_t errlen) {
  int rc = check_attn_shape(shape, err, errlen);
  if (rc) return rc;
  if ((rc = check_kv_cache(shape, cache, false, err, errlen))) return rc;
  size_t need = 0;
  if ((rc = ds_moe_attention_workspace_bytes(shape, n_requests, T, max_new, &need, err, errlen))) return rc;
  AttnArgs a{};
  bool nothing;
  if ((rc = attention_args(*shape, need, block_table, table_width, table_stride, q, q_stride, T, cu_new, seq_lens, n_requests,
                           max_new, out, out_stride, lse, workspace, workspace_bytes, &a, &nothing, err, errlen)) || nothing)
    return rc;
  a.k = (const uint16_t *)cache->k; a.v = (const uint16_t *)cache->v;
  a.n_pages = cache->n_pages; a.ps = cache->page_stride; a.rs = cache->row_stride; a.hs = cache->head_stride;
  const bool bf16 = shape->dtype == DS_BF16;
  const cudaStream_t st = (cudaStream_t)stream;
  const int path = table_width ? path_of(*shape, *cache, q, q_stride, T, max_new) : DS_ATTN_GENERIC;
  const cudaError_t e = path == DS_ATTN_DECODE  ? launch_attention_decode(a, bf16, workspace, st)
                        : path == DS_ATTN_CHUNK ? launch_attention_chunk(a, bf16, workspace, st)
                                                : launch_attention_generic(a, bf16, st);
  return e == cudaSuccess ? DS_OK : cuda_fail(err, errlen, e, "attention");
}

}  // extern "C"
