// Pages for a step's new tokens (ds_moe_page_map) and the copy of their keys
// and values to those pages (ds_moe_kv_append).
#include "common.cuh"
#include "errors.h"
#include "internal.h"
#include "serving.cuh"

namespace dsm {
namespace {

constexpr int PM_THREADS = 512;
constexpr int PM_MAX_REQUESTS = 16384;  // three ints a request in shared memory
constexpr int32_t MAX_LEN = 1 << 30;  // lengths are below it, so that two add up to an int

// Exclusive scan of v over the block (PM_THREADS threads); total to all.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *part, int64_t &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) part[warp] = incl;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < PM_THREADS / 32; ++w) {
    const int64_t p = part[w];
    if (w < warp) before += p;
    all += p;
  }
  __syncthreads();
  total = all;
  return before + incl - v;
}

// Last i in [0, n) with a[i] <= v (a ascending, a[0] <= v).
__device__ __forceinline__ int last_at_most(const int *a, int n, int v) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= v) lo = mid; else hi = mid;
  }
  return lo;
}

// n / d for n < 2^31 and d <= 2^16 as a product and a shift: with 2^(s-1) < d
// <= 2^s and m = ceil(2^(31+s) / d), floor(n m / 2^(31+s)) is the quotient
// (Granlund and Montgomery, "Division by invariant integers", theorem 4.2).
struct Divisor {
  uint64_t m;
  int shift;
  explicit Divisor(uint32_t d) : shift(31) {
    while (((uint64_t)1 << (shift - 31)) < d) ++shift;
    m = (((uint64_t)1 << shift) + d - 1) / d;
  }
  __device__ __forceinline__ int of(int n) const { return (int)(((uint64_t)(uint32_t)n * m) >> shift); }
};

struct PageMapArgs {
  const int32_t *context, *fresh;
  int R, page, n_free, width, cap;
  const int32_t *free_pages;
  int32_t *table;
  int64_t table_stride;
  int64_t *slots;
  int32_t *positions, *cu, *seq, *taken;
  unsigned *status;
  Divisor by_page;
};

// Two exclusive scans over the requests (new tokens, then pages taken), which
// every block makes for itself in shared memory, a thread PER requests, and
// then independent writes: blocks share out the tokens and the new table
// entries.  The page of a token that lies in a new page comes from the free
// list, not from the table, so no block waits for another's entries.  Bound
// by latency: the lengths' loads, the scans' barriers, a search per token (7
// requests, 20 tokens, 3.7 us; 2048 requests, 156,000 tokens 8 us, of which the
// 2 MB that it writes would be 0.3).  PER follows the number of requests, so
// that a thread's lengths are in registers and no more of them than there are
// (with 32 a thread throughout 8.8 and 15 us).
template <int PER>
__global__ void __launch_bounds__(PM_THREADS) page_map_kernel(const PageMapArgs a) {
  extern __shared__ int sm[];
  int *cu = sm;              // [R + 1] first token of each request
  int *base = cu + a.R + 1;  // [R + 1] first free-list index of each request
  int *ctx = base + a.R + 1; // [R] cached tokens
  __shared__ int64_t part[PM_THREADS / 32];
  const int tid = threadIdx.x, r0 = tid * PER;
  bool bad = false;
  auto valid = [&](int v) {
    if (v >= 0 && v < MAX_LEN) return v;
    bad = true;
    return 0;
  };
  int c[PER], n[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const bool some = r0 + i < a.R;
    c[i] = some ? a.context[r0 + i] : 0;
    n[i] = some ? a.fresh[r0 + i] : 0;
  }
  int64_t mine = 0, total;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    c[i] = valid(c[i]);
    n[i] = valid(n[i]);
    mine += n[i];
  }
  int64_t run = block_scan(mine, part, total);
  if (total > a.cap) bad = true;
  mine = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int at = (int)min(run, (int64_t)a.cap);
    run += n[i];
    n[i] = (int)min(run, (int64_t)a.cap) - at;  // what there is room for
    if (r0 + i < a.R) {
      cu[r0 + i] = at;
      ctx[r0 + i] = c[i];
    }
  }
  if (tid == 0) cu[a.R] = (int)min(total, (int64_t)a.cap);
  // pages: held ones, and needed ones as far as the table goes
  int take[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int held = min(a.by_page.of(c[i] + a.page - 1), a.width), need = a.by_page.of(c[i] + n[i] + a.page - 1);
    if (need > a.width) bad = true;
    take[i] = min(need, a.width) - held;
    mine += take[i];
  }
  int64_t pages;
  run = block_scan(mine, part, pages);
  if (pages > a.n_free) bad = true;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (r0 + i < a.R) base[r0 + i] = (int)run;
    run += take[i];
  }
  if (tid == 0) base[a.R] = (int)pages;
  __syncthreads();
  const int step = gridDim.x * PM_THREADS, first = blockIdx.x * PM_THREADS + tid;
  for (int r = first; r < a.R; r += step) {
    a.cu[r] = cu[r];
    a.seq[r] = ctx[r] + (cu[r + 1] - cu[r]);
  }
  if (first == 0) {
    a.cu[a.R] = cu[a.R];
    a.taken[0] = (int)min(pages, (int64_t)a.n_free);
  }
  auto held_of = [&](int r) { return min(a.by_page.of(ctx[r] + a.page - 1), a.width); };
  for (int t = first; t < a.cap; t += step) {
    if (t >= cu[a.R]) {
      a.slots[t] = -1;
      a.positions[t] = -1;
      continue;
    }
    const int r = last_at_most(cu, a.R, t);
    const int pos = ctx[r] + t - cu[r];
    const int col = a.by_page.of(pos), held = held_of(r);
    int page = -1;
    if (col < a.width) {
      if (col < held) {
        page = a.table[r * a.table_stride + col];
      } else {
        const int p = base[r] + col - held;
        page = p < a.n_free ? a.free_pages[p] : -1;
      }
    }
    if (page < 0) bad = true;
    a.slots[t] = page < 0 ? -1 : (int64_t)page * a.page + (pos - col * a.page);
    a.positions[t] = pos;
  }
  for (int p = first; p < base[a.R]; p += step) {
    const int r = last_at_most(base, a.R, p);
    a.table[r * a.table_stride + held_of(r) + p - base[r]] = p < a.n_free ? a.free_pages[p] : -1;
  }
  if (bad) flag(a.status, ST_PAGING);
}

template <int PER>
cudaError_t launch_page_map(const PageMapArgs &a, int sms, cudaStream_t s) {
  static OncePerDevice once;
  const cudaError_t e = once_per_device(once, []() {
    return cudaFuncSetAttribute(page_map_kernel<PER>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)sizeof(int) * (3 * PER * PM_THREADS + 2));
  });
  if (e != cudaSuccess) return e;
  const int blocks = std::max(1, std::min(sms, (std::max(a.cap, a.R) + PM_THREADS - 1) / PM_THREADS));
  page_map_kernel<PER><<<blocks, PM_THREADS, sizeof(int) * (3 * a.R + 2), s>>>(a);
  return cudaGetLastError();
}

struct AppendArgs {
  uint16_t *k, *v;
  const uint16_t *kn, *vn;
  const int64_t *slots;
  int64_t T, n_slots, ps, rs, hs, token_stride, head_stride;
  int page, units, per_head;  // units of VEC elements: of a token's row, of a head
  unsigned *status;
};

// A warp a token, so that its slot is taken apart once; a lane takes units of
// it (16 bytes where everything is aligned, one element elsewhere), four of
// the keys and four of the values under way at once.  Bound by HBM: 15,156
// tokens of 8 heads x 128 (62 MB each way) in 19 to 22 us, 5.5 TB/s and more.
template <int VEC>
__global__ void __launch_bounds__(256) kv_append_kernel(const AppendArgs a) {
  typedef typename std::conditional<VEC == 8, uint4, uint16_t>::type U;
  const int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (t >= a.T) return;
  const int64_t slot = a.slots[t];
  if (slot < 0) return;
  if (slot >= a.n_slots) {
    if (lane == 0) flag(a.status, ST_PAGING);
    return;
  }
  const int64_t page = slot >> 32 ? slot / a.page : (uint32_t)slot / (uint32_t)a.page;
  const int64_t dst = page * a.ps + (slot - page * a.page) * a.rs, src = t * a.token_stride;
  for (int u0 = lane; u0 < a.units; u0 += 128) {
    U kr[4], vr[4];
    int64_t to[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int u = u0 + 32 * i;
      if (u >= a.units) continue;
      const int h = (unsigned)u / (unsigned)a.per_head, d = (u - h * a.per_head) * VEC;
      to[i] = dst + h * a.hs + d;
      const int64_t from = src + h * a.head_stride + d;
      kr[i] = *reinterpret_cast<const U *>(a.kn + from);
      vr[i] = *reinterpret_cast<const U *>(a.vn + from);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (u0 + 32 * i >= a.units) continue;
      *reinterpret_cast<U *>(a.k + to[i]) = kr[i];
      *reinterpret_cast<U *>(a.v + to[i]) = vr[i];
    }
  }
}

}  // namespace
}  // namespace dsm

using namespace dsm;

extern "C" {

int ds_moe_page_map(const int32_t *context_lens, const int32_t *new_lens, int32_t n_requests, int32_t page_size,
                    const int32_t *free_pages, int32_t n_free, int32_t *block_table, int32_t table_width,
                    int64_t table_stride, int64_t *slots, int32_t *positions, int32_t max_tokens, int32_t *cu_new,
                    int32_t *seq_lens, int32_t *n_taken, void *stream, char *err, size_t errlen) {
  if (n_requests < 0 || n_requests > PM_MAX_REQUESTS)
    return fail(err, errlen, DS_ERR_INVALID_ARG, "n_requests=%d: need 0..%d", n_requests, PM_MAX_REQUESTS);
  if (page_size < 1 || page_size > 65536)
    return fail(err, errlen, DS_ERR_INVALID_ARG, "page_size=%d: need 1..65536", page_size);
  if (n_free < 0 || table_width < 0 || max_tokens < 0)
    return fail(err, errlen, DS_ERR_INVALID_ARG, "negative n_free, table_width or max_tokens");
  if (max_tokens > (1 << 24)) return fail(err, errlen, DS_ERR_INVALID_ARG, "max_tokens=%d out of range", max_tokens);
  if (n_requests > 1 && table_stride < table_width)
    return fail(err, errlen, DS_ERR_INVALID_ARG, "table_stride is smaller than table_width");
  if (!cu_new || !n_taken || (n_requests && (!context_lens || !new_lens || !seq_lens)))
    return fail(err, errlen, DS_ERR_INVALID_ARG, "lengths, cu_new, seq_lens and n_taken are required");
  if ((n_free && !free_pages) || (n_requests && table_width && !block_table) || (max_tokens && (!slots || !positions)))
    return fail(err, errlen, DS_ERR_INVALID_ARG, "free_pages, block_table, slots and positions are required");
  if (!aligned(context_lens, 4) || !aligned(new_lens, 4) || !aligned(free_pages, 4) || !aligned(block_table, 4) ||
      !aligned(slots, 8) || !aligned(positions, 4) || !aligned(cu_new, 4) || !aligned(seq_lens, 4) ||
      !aligned(n_taken, 4))
    return fail(err, errlen, DS_ERR_INVALID_ARG, "arrays must be aligned to their elements");
  PageMapArgs a{context_lens, new_lens, n_requests, page_size, n_free, table_width, max_tokens, free_pages, block_table,
                table_stride, slots, positions, cu_new, seq_lens, n_taken, status_word(), Divisor((uint32_t)page_size)};
  const int sms = device_sms();
  if (!a.status || !sms) return fail(err, errlen, DS_ERR_CUDA, "no CUDA device");
  const cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = n_requests <= PM_THREADS       ? launch_page_map<1>(a, sms, s)
                        : n_requests <= 4 * PM_THREADS ? launch_page_map<4>(a, sms, s)
                                                       : launch_page_map<PM_MAX_REQUESTS / PM_THREADS>(a, sms, s);
  return e == cudaSuccess ? DS_OK : cuda_fail(err, errlen, e, "page map");
}

int ds_moe_kv_append(const ds_moe_attn_shape *shape, const ds_moe_kv_cache *cache, const void *k_new,
                     const void *v_new, int64_t token_stride, int64_t head_stride, const int64_t *slots, int64_t T,
                     void *stream, char *err, size_t errlen) {
  int rc = check_attn_shape(shape, err, errlen);
  if (rc) return rc;
  if ((rc = check_kv_cache(shape, cache, err, errlen))) return rc;
  if (T < 0 || T > (1 << 24)) return fail(err, errlen, DS_ERR_INVALID_ARG, "T=%lld out of range", (long long)T);
  if (T == 0) return DS_OK;
  if (!k_new || !v_new || !slots) return fail(err, errlen, DS_ERR_INVALID_ARG, "k_new, v_new and slots are required");
  if (!aligned(k_new, 2) || !aligned(v_new, 2) || !aligned(slots, 8))
    return fail(err, errlen, DS_ERR_INVALID_ARG, "k_new, v_new and slots must be aligned to their elements");
  if (token_stride < 0 || head_stride < 0) return fail(err, errlen, DS_ERR_INVALID_ARG, "negative stride");
  const int D = shape->head_dim, H = shape->n_head_kv;
  const bool wide = D % 8 == 0 && token_stride % 8 == 0 && head_stride % 8 == 0 && cache->page_stride % 8 == 0 &&
                    cache->row_stride % 8 == 0 && cache->head_stride % 8 == 0 && aligned(k_new, 16) &&
                    aligned(v_new, 16) && aligned(cache->k, 16) && aligned(cache->v, 16);
  const int vec = wide ? 8 : 1;
  AppendArgs a{(uint16_t *)cache->k, (uint16_t *)cache->v, (const uint16_t *)k_new, (const uint16_t *)v_new, slots, T,
               cache->n_pages * shape->page_size, cache->page_stride, cache->row_stride, cache->head_stride,
               token_stride, head_stride, shape->page_size, H * (D / vec), D / vec, status_word()};
  if (!a.status) return fail(err, errlen, DS_ERR_CUDA, "no CUDA device");
  const int64_t blocks = (T + 7) / 8;
  if (wide)
    kv_append_kernel<8><<<(unsigned)blocks, 256, 0, (cudaStream_t)stream>>>(a);
  else
    kv_append_kernel<1><<<(unsigned)blocks, 256, 0, (cudaStream_t)stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? DS_OK : cuda_fail(err, errlen, e, "kv append");
}

}  // extern "C"
