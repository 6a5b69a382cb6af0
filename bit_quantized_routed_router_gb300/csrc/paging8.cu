// New keys and values into a cache in 8 bits (ds_moe_kv8_append).
#include "errors.h"
#include "internal.h"
#include "kv8.cuh"
#include "rope.cuh"

namespace dsm {
namespace {

constexpr int A8_WARPS = 8;
constexpr int A8_ROWS = 64;  // tokens whose angles a block holds at a time
constexpr int A8_KEEP = 4;   // units of a lane that are kept

struct Append8Args {
  Rope rope;
  RopeRows q;
  int H, G;  // H = 0: no queries
  const uint16_t *kn, *vn;
  int64_t nt, nh;
  uint8_t *k, *v;
  float *ks, *vs;
  int64_t n_pages, ps, rs, hs, sps, sbs, shs;
  int page, block;
  const int32_t *table;
  int64_t table_stride;
  const int32_t *cu, *seq;
  int T, R, max_new;
  int64_t max_seq;
  int64_t runs;       // blocks in x that take runs: per request `per_request`, or (0) one a token
  int per_request, y_runs, y_queries;
  int64_t groups;     // of tokens whose queries a warp takes
  int per;            // query heads a part
  unsigned *status;
};

// The least power of two, from 2^-60 to 2^60, that brings `most` to 448 =
// 1.75 2^8 or below: its exponent, and one more where the mantissa is beyond 1.75.
__device__ __forceinline__ float scale_for(float most) {
  const int e = (int)((__float_as_uint(most) + 0x1FFFFFu) >> 23) - 127 - 8;
  return __uint_as_float((uint32_t)(min(max(e, -60), 60) + 127) << 23);
}

__device__ __forceinline__ float finite_or_nan(float x) { return fabsf(x) <= 3.402823466e38f ? x : __uint_as_float(0x7FFFFFFFu); }

// A request's rows at the positions that its lengths give them, whether the table
// and T reach so far or not: a token that has no place must not move the others
// onto what is there already.
__device__ __forceinline__ Span append_span(const Append8Args &a, int r, bool &bad) {
  const RawSpan w = request_raw(a.cu, a.seq, r);
  Span s = request_span(w, a.T, a.max_new, a.max_seq, bad);
  s.pos0 = (int)max((int64_t)w.seq - w.c1 + s.t0, -((int64_t)1 << 25));  // (T is 2^24 at most: further back, none is at 0)
  return s;
}

// A unit's elements as e4m3.  (Infinities only where `odd` says that there are
// some: the conversion would make them 448.)
template <int W>
__device__ __forceinline__ void store8(uint8_t *head, const Unit &u, const float (&x)[2 * W], float by, bool odd) {
  float v[2 * W];
#pragma unroll
  for (int i = 0; i < 2 * W; ++i) v[i] = x[i] * by;
  if (odd) {
#pragma unroll
    for (int i = 0; i < 2 * W; ++i) v[i] = finite_or_nan(x[i]) * by;
  }
  if (W == 8) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = f8x2_of(v[4 * i], v[4 * i + 1]) | (uint32_t)f8x2_of(v[4 * i + 2], v[4 * i + 3]) << 16;
    *reinterpret_cast<uint2 *>(head + u.a) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2 *>(head + u.b) = make_uint2(w[2], w[3]);
  } else {
    const uint16_t w = f8x2_of(v[0], v[1]);
    head[u.a] = (uint8_t)w;
    if (u.b >= 0) head[u.b] = (uint8_t)(w >> 8);
  }
}

// A run is the new tokens of one block of a request.  A block of threads takes
// a run under eight of the 2 G rows of heads (keys, then values), a warp each:
// it finds the run's largest element, from it the scale, and then quantises;
// up to A8_KEEP tokens a lane (16 of head_dim 128 a warp) are kept in
// between, longer runs are read twice.  (Four blocks an SM leave 64 registers, of which
// the kernels for 16-byte loads spill 184 to 272 bytes a thread.)  The tokens' angles are computed by the
// whole block into shared memory.  Queries are rotated by further blocks of
// the same launch, as in rotary.cu.  15,156 tokens of 13 prompts, 32 query and
// 8 key heads of 128, blocks of 16 tokens, fp16: 70 us, 72 % of the copy
// bandwidth; the runs alone are 28 to 31 us, under half of it, as each waits in turn for
// lengths, page, elements and old scale, so queries' blocks are mixed with
// them.  64 single tokens: 4.5 us in a graph.
template <int W, bool INTER, bool BF16>
__global__ void __launch_bounds__(A8_WARPS * 32, 4) kv8_append_kernel(const __grid_constant__ Append8Args a) {
  __shared__ __align__(16) float cosine[A8_ROWS][64], sine[A8_ROWS][64];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int units = unit_count<W>(a.rope);
  bool bad = false;
  // the last request that begins at or before token t
  auto request_of = [&](int t) {
    int r = 0, hi = a.R;
    while (hi - r > 1) {
      const int mid = (r + hi) >> 1;
      if (a.cu[mid] <= t) r = mid; else hi = mid;
    }
    return r;
  };
  // blocks for runs and for queries take turns in the grid, so that the one
  // kind's waits and the other's traffic share the SMs
  const unsigned run_blocks = (unsigned)(a.runs * a.y_runs);
  const unsigned run_block = (unsigned)((uint64_t)blockIdx.x * run_blocks / gridDim.x);
  if ((unsigned)((blockIdx.x + 1ull) * run_blocks / gridDim.x) == run_block) {
    // ------------------------------------------------------------ queries --
    const LaneRows lanes(min(units, 32));
    const int64_t w = (int64_t)(blockIdx.x - run_block) * A8_WARPS + warp, group = w / a.y_queries;
    const int part = (int)(w - group * a.y_queries);
    const int64_t t = group * lanes.rows + lanes.row;
    if (group >= a.groups || lanes.row < 0 || t >= a.T) return;
    const Span s = append_span(a, request_of((int)t), bad);
    const int i = (int)t - s.t0;
    if (i < 0 || i >= s.n || s.pos0 + i < 0) return;
    for (int unit = lanes.unit; unit < units; unit += 32)
      rotate_heads<W, INTER, BF16>(
          a.rope, unit_of<W, INTER>(a.rope, unit), s.pos0 + i, part * a.per, min(a.H, (part + 1) * a.per),
          [&](int h) { return a.q.x + t * a.q.xt + h * a.q.xh; }, [&](int h) { return a.q.out + t * a.q.ot + h * a.q.oh; },
          [](int) { return true; });
    return;
  }
  // ------------------------------------------------------------------ runs --
  const int64_t x = run_block / (unsigned)a.y_runs;
  const int row = (int)(run_block - x * a.y_runs) * A8_WARPS + warp;  // of the 2 G rows of heads
  int r, t;    // request, first token of the run
  int64_t at;  // and its position
  Span s;
  if (a.per_request) {
    r = (int)(x / a.per_request);
    const int j = (int)(x - (int64_t)r * a.per_request);
    s = append_span(a, r, bad);
    const int p0 = max(s.pos0, 0);
    at = j ? (int64_t)(p0 / a.block + j) * a.block : p0;
    t = s.t0 + (int)(at - s.pos0);
  } else {
    t = (int)x;
    r = request_of(t);
    s = append_span(a, r, bad);
    at = (int64_t)s.pos0 + t - s.t0;
    if (t < s.t0 || at < 0 || (t > s.t0 && at % a.block)) t = a.T;  // does not begin a run
  }
  if (bad && row == 0 && lane == 0) flag(a.status, ST_PAGING);
  if (t >= s.t0 + s.n || at >= a.max_seq) return;
  const int pos = (int)at;
  const int in_block = pos % a.block, n = min(a.block - in_block, s.t0 + s.n - t);
  const int col = pos / a.page, page = a.table[r * a.table_stride + col];  // (under way while the elements are)
  const bool value = row >= a.G;
  const int h = value ? row - a.G : row;
  const bool some = row < 2 * a.G;
  const uint16_t *src = (value ? a.vn : a.kn) + (int64_t)t * a.nt + (some ? h : 0) * a.nh;
  const int first = pos - col * a.page;  // row of the page
  const bool turn = a.rope.dim && !value;
  // a block's rows are keys and values, so all warps fill the angles or none does
  const bool angles = a.rope.dim && (row - warp) < a.G;
  auto fill = [&](int i0, int rows) {
    const int p = threadIdx.x & 63;
    if (p >= a.rope.dim / 2) return;
    for (int i = threadIdx.x >> 6; i < rows; i += A8_WARPS / 2) {
      const float2 cs = rope_angle(a.rope, p, pos + i0 + i);
      cosine[i][p] = cs.x;
      sine[i][p] = cs.y;
    }
  };
  // a unit's values (token i of the chunk, unit u)
  auto values = [&](const Chunks<W> &c, const Unit &u, int i, float (&v)[2 * W]) {
    c.template get<BF16>(v);
    if (turn && u.pair >= 0) {
      float cc[W], ss[W];
      if (W == 8) {
#pragma unroll
        for (int k = 0; k < W; k += 4) {
          const float4 p = *reinterpret_cast<const float4 *>(&cosine[i][u.pair + k]), q = *reinterpret_cast<const float4 *>(&sine[i][u.pair + k]);
          cc[k] = p.x; cc[k + 1] = p.y; cc[k + 2] = p.z; cc[k + 3] = p.w;
          ss[k] = q.x; ss[k + 1] = q.y; ss[k + 2] = q.z; ss[k + 3] = q.w;
        }
      } else {
        cc[0] = cosine[i][u.pair];
        ss[0] = sine[i][u.pair];
      }
      rotate_unit<W, INTER>(v, cc, ss);
    }
  };
  // the largest magnitude, infinities among it or (odd) not; NaN has no say
  auto most_of = [&](const float (&v)[2 * W], const Unit &u, float most, bool odd) {
#pragma unroll
    for (int k = 0; k < 2 * W; ++k)
      if (W == 8 || k == 0 || u.b >= 0) most = fmaxf(most, fabsf(odd ? finite_or_nan(v[k]) : v[k]));
    return most;
  };
  // A lane has one unit (of 32 at a time) of every `lanes.rows`-th token.
  const LaneRows lanes(min(units, 32));
  const Unit mine = unit_of<W, INTER>(a.rope, lanes.unit);
  const bool once = n <= A8_ROWS && units <= 32 && n <= A8_KEEP * lanes.rows;
  const bool takes = some && lanes.row >= 0;
  Chunks<W> keep[A8_KEEP];  // (as they are in memory: half the registers, and rotated twice)
  float most = 0.f;
  if (once) {
#pragma unroll
    for (int k = 0; k < A8_KEEP; ++k)
      if (takes && lanes.row + k * lanes.rows < n) keep[k].load(src + (lanes.row + k * lanes.rows) * a.nt, mine);
    if (angles) fill(0, n);
  }
  if (page < 0 || page >= a.n_pages) {
    if (row == 0 && lane == 0) flag(a.status, ST_PAGING);
    return;
  }
  uint8_t *dst = (value ? a.v : a.k) + page * a.ps + first * a.rs + h * a.hs;
  float *scale_at = (value ? a.vs : a.ks) + page * a.sps + (int64_t)(first / a.block) * a.sbs + h * a.shs;
  float was = 0.f;
  if (some && in_block) was = kv8_scale(*scale_at);
  float scale = 0.f, by = 0.f;
  bool odd = false;
  // What a run that does not stay in registers goes through three times (the
  // angles chunk by chunk): its largest element, that without infinities, where
  // there are some, and the conversion.
  enum { MOST, FINITE, STORE };
  auto visit = [&](int what) {
    for (int i0 = 0; i0 < n; i0 += A8_ROWS) {
      const int rows = min(A8_ROWS, n - i0);
      if (!once && (what == MOST || n > A8_ROWS)) {
        __syncthreads();
        if (angles) fill(i0, rows);
        __syncthreads();
      }
      if (!takes) continue;
      for (int unit = lanes.unit; unit < units; unit += 32) {
        const Unit u = unit_of<W, INTER>(a.rope, unit);
        for (int i = lanes.row; i < rows; i += A8_KEEP * lanes.rows) {
#pragma unroll
          for (int k = 0; k < A8_KEEP; ++k)
            if (i + k * lanes.rows < rows) keep[k].load(src + (i0 + i + k * lanes.rows) * a.nt, u);
#pragma unroll
          for (int k = 0; k < A8_KEEP; ++k) {
            if (i + k * lanes.rows >= rows) continue;
            float v[2 * W];
            values(keep[k], u, i + k * lanes.rows, v);
            if (what == STORE) store8<W>(dst + (i0 + i + k * lanes.rows) * a.rs, u, v, by, odd);
            else most = most_of(v, u, most, what == FINITE);
          }
        }
      }
    }
  };
  auto over_warp = [&](float m) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
  };
  // the kept units, with their values
  auto kept = [&](auto &&with) {
#pragma unroll
    for (int k = 0; k < A8_KEEP; ++k) {
      const int i = lanes.row + k * lanes.rows;
      if (!takes || i >= n) continue;
      float v[2 * W];
      values(keep[k], mine, i, v);
      with(v, i);
    }
  };
  if (once) {
    __syncthreads();
    if (!some) return;
    kept([&](const float (&v)[2 * W], int) { most = most_of(v, mine, most, false); });
  } else {
    visit(MOST);
  }
  most = over_warp(most);
  odd = most > 3.402823466e38f;  // (of all lanes: an infinity among them, which is rare)
  if (once ? odd : __syncthreads_or(odd)) {
    most = 0.f;
    visit(FINITE);
    most = over_warp(most);
  }
  scale = fmaxf(scale_for(most), was);
  by = 1.f / scale;
  if (some && in_block && scale > was) {  // the block's earlier tokens follow
    const float ratio = was * by;
    uint8_t *begin = dst - in_block * a.rs;
    constexpr int C = W == 8 ? 16 : 1;
    const int words = a.rope.D / C;
    for (int e = lane; e < in_block * words; e += 32) {
      const int i = e / words;
      uint8_t *at = begin + i * a.rs + (e - i * words) * C;
      if (W == 8) {
        uint4 q = *reinterpret_cast<const uint4 *>(at);
        uint32_t *w = reinterpret_cast<uint32_t *>(&q);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 lo = f8x2_to((uint16_t)w[k]), hi = f8x2_to((uint16_t)(w[k] >> 16));
          w[k] = f8x2_of(lo.x * ratio, lo.y * ratio) | (uint32_t)f8x2_of(hi.x * ratio, hi.y * ratio) << 16;
        }
        *reinterpret_cast<uint4 *>(at) = q;
      } else {
        *at = (uint8_t)f8x2_of(f8x2_to(*at).x * ratio, 0.f);
      }
    }
  }
  __syncwarp();  // (every lane has read the old scale)
  if (some && lane == 0) *scale_at = scale;
  if (once && !odd) kept([&](const float (&v)[2 * W], int i) { store8<W>(dst + i * a.rs, mine, v, by, false); });
  else visit(STORE);
}

template <int W>
cudaError_t launch(Append8Args &a, bool inter, bool bf16, cudaStream_t s) {
  a.y_runs = (2 * a.G + A8_WARPS - 1) / A8_WARPS;
  a.groups = 0;
  a.y_queries = 1;
  a.per = 0;
  int64_t query_blocks = 0;
  if (a.H) {
    const int rows = 32 / std::min(unit_count<W>(a.rope), 32);
    a.groups = (a.T + rows - 1) / rows;
    // (three waves of 152 SMs x 4 blocks x 8 warps: runs' blocks fill what the last leaves)
    const int parts = head_parts(a.groups, a.H, 14592);
    a.per = ((a.H + parts - 1) / parts + 1) / 2 * 2;
    a.y_queries = (a.H + a.per - 1) / a.per;
    query_blocks = (a.groups * a.y_queries + A8_WARPS - 1) / A8_WARPS;
  }
  const int64_t blocks = a.runs * a.y_runs + query_blocks;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  const unsigned grid = (unsigned)blocks;
  if (inter && bf16) kv8_append_kernel<W, true, true><<<grid, A8_WARPS * 32, 0, s>>>(a);
  else if (inter) kv8_append_kernel<W, true, false><<<grid, A8_WARPS * 32, 0, s>>>(a);
  else if (bf16) kv8_append_kernel<W, false, true><<<grid, A8_WARPS * 32, 0, s>>>(a);
  else kv8_append_kernel<W, false, false><<<grid, A8_WARPS * 32, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace
}  // namespace dsm

using namespace dsm;

extern "C" int ds_moe_kv8_append(const ds_moe_attn_shape *shape, const ds_moe_kv8_cache *cache, const ds_moe_rope *rope,
                                 const void *k_new, const void *v_new, int64_t token_stride, int64_t head_stride,
                                 const ds_moe_rope_rows *q, const int32_t *block_table, int32_t table_width,
                                 int64_t table_stride, const int32_t *cu_new, const int32_t *seq_lens,
                                 int32_t n_requests, int64_t T, int32_t max_new, void *stream, char *err,
                                 size_t errlen) {
  int rc = check_attn_shape(shape, err, errlen);
  if (rc) return rc;
  if ((rc = check_kv8_cache(shape, cache, true, err, errlen))) return rc;
  const int D = shape->head_dim, G = shape->n_head_kv;
  if (rope && (rc = check_rope(rope, D, err, errlen))) return rc;
  if (q && !rope) return fail(err, errlen, DS_ERR_INVALID_ARG, "q needs rope");
  if (T < 0 || T > (1 << 24)) return fail(err, errlen, DS_ERR_INVALID_ARG, "T=%lld out of range", (long long)T);
  if (n_requests < 0 || max_new < 0 || table_width < 0)
    return fail(err, errlen, DS_ERR_INVALID_ARG, "negative n_requests, max_new or table_width");
  if (T == 0 || n_requests == 0 || max_new == 0) return DS_OK;
  if (n_requests > 1 && table_stride < table_width)
    return fail(err, errlen, DS_ERR_INVALID_ARG, "table_stride is smaller than table_width");
  if (!k_new || !v_new || !cu_new || !seq_lens || (table_width && !block_table))
    return fail(err, errlen, DS_ERR_INVALID_ARG, "k_new, v_new, block_table, cu_new and seq_lens are required");
  if (!aligned(k_new, 2) || !aligned(v_new, 2) || !aligned(block_table, 4) || !aligned(cu_new, 4) || !aligned(seq_lens, 4))
    return fail(err, errlen, DS_ERR_INVALID_ARG, "arrays must be aligned to their elements");
  if (token_stride < 0 || head_stride < 0) return fail(err, errlen, DS_ERR_INVALID_ARG, "negative stride");
  if (q && (rc = check_rope_rows(q, T, shape->n_head, D, err, errlen))) return rc;
  Append8Args a{};
  a.rope = rope_of(rope, D);
  a.q = rows_of(q);
  a.H = q ? shape->n_head : 0;
  a.G = G;
  a.kn = (const uint16_t *)k_new; a.vn = (const uint16_t *)v_new; a.nt = token_stride; a.nh = head_stride;
  a.k = (uint8_t *)cache->k; a.v = (uint8_t *)cache->v; a.ks = cache->k_scale; a.vs = cache->v_scale;
  a.n_pages = cache->n_pages; a.ps = cache->page_stride; a.rs = cache->row_stride; a.hs = cache->head_stride;
  a.sps = cache->scale_page_stride; a.sbs = cache->scale_block_stride; a.shs = cache->scale_head_stride;
  a.page = shape->page_size; a.block = cache->block_rows;
  a.table = block_table; a.table_stride = table_stride;
  a.cu = cu_new; a.seq = seq_lens; a.T = (int)T; a.R = n_requests; a.max_new = max_new;
  a.max_seq = std::min<int64_t>((int64_t)table_width * a.page, 1 << 30);
  // runs: a block of the grid for each that a request can have at most, or for
  // each token that might begin one, whichever is fewer
  const int64_t each = ((int64_t)std::min<int64_t>(max_new, T) + a.block - 2) / a.block + 1;
  a.per_request = n_requests * each <= T ? (int)each : 0;
  a.runs = a.per_request ? n_requests * each : T;
  if (!(a.status = status_word())) return fail(err, errlen, DS_ERR_CUDA, "no CUDA device");
  auto fits = [](int64_t n, int64_t s, int to) { return n <= 1 || s % to == 0; };
  const bool wide = rope_wide(a.rope) && (!q || rows_wide(a.q, T, a.H)) && aligned(k_new, 16) && aligned(v_new, 16) &&
                    aligned(cache->k, 16) && aligned(cache->v, 16) && fits(T, token_stride, 8) && fits(G, head_stride, 8) &&
                    fits(a.n_pages, a.ps, 16) && fits(a.page, a.rs, 16) && fits(G, a.hs, 16);
  const cudaError_t e = wide ? launch<8>(a, rope && rope->interleaved, shape->dtype == DS_BF16, (cudaStream_t)stream)
                             : launch<1>(a, rope && rope->interleaved, shape->dtype == DS_BF16, (cudaStream_t)stream);
  return e == cudaSuccess ? DS_OK : cuda_fail(err, errlen, e, "8-bit append");
}
