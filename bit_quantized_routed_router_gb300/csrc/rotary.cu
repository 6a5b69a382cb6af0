// Rotary positions: ds_moe_rope_init, ds_moe_rotary, and the 16-bit append
// that rotates on the way (ds_moe_kv_append_rotary).
#include <float.h>
#include <math.h>

#include "errors.h"
#include "internal.h"
#include "rope.cuh"

namespace dsm {
namespace {

constexpr int RO_WARPS = 4;

struct RotaryArgs {
  Rope rope;
  RopeRows q;  // heads [0, H) of a token
  int H;
  int G;       // then G keys and G values, to slots (0: there are none)
  const uint16_t *kn, *vn;
  int64_t nt, nh;
  uint16_t *k, *v;
  int64_t n_slots, ps, rs, hs;
  int page;
  const int64_t *slots;
  const int32_t *positions;
  int64_t T;
  int parts, per;  // parts of a token's heads, heads a part
  unsigned *status;
};

// A warp takes a few neighbouring tokens (four of head_dim 128) and part of
// their heads; a lane keeps one unit of one token, so its cosines and sines
// are computed once and stay in registers over the heads.  Bound by HBM for
// many tokens, by latency (position, sine, element) for few.  8192 tokens of 40
// heads of 128, half of each rotated: 32 us, 77 % of the copy bandwidth; 15,156
// tokens with 32 query and 8 key heads of 128 into a cache: 66 us, 83 %; 48
// tokens of 32 heads: 3.2 us in a graph.  Where 16-byte chunks do not serve (W = 1)
// it is bound by its 2-byte loads: the first with 56 elements of each rotated 127 us,
// the prompts with 24 or 56 263 us (into 8 bits 306).
template <int W, bool INTER, bool BF16>
__global__ void __launch_bounds__(RO_WARPS * 32, 8) rotary_kernel(const __grid_constant__ RotaryArgs a) {
  const int64_t w = (int64_t)blockIdx.x * RO_WARPS + (threadIdx.x >> 5);
  const int64_t group = w / a.parts;
  const int part = (int)(w - group * a.parts);
  const int units = unit_count<W>(a.rope), all = a.H + 2 * a.G;
  const int h0 = part * a.per, h1 = min(all, h0 + a.per);
  const LaneRows lanes(min(units, 32));
  const int64_t t = group * lanes.rows + lanes.row;
  if (lanes.row < 0 || t >= a.T) return;
  const int position = a.positions[t];
  if (position < 0) return;
  int64_t place = -1;  // of the token's row in the cache
  if (a.G) {
    const int64_t slot = a.slots[t];
    if (slot >= a.n_slots) {
      flag(a.status, ST_PAGING);
    } else if (slot >= 0) {
      const int64_t page = slot >> 32 ? slot / a.page : (uint32_t)slot / (uint32_t)a.page;
      place = page * a.ps + (slot - page * a.page) * a.rs;
    }
  }
  for (int unit = lanes.unit; unit < units; unit += 32) {
    const Unit u = unit_of<W, INTER>(a.rope, unit);
    rotate_heads<W, INTER, BF16>(
        a.rope, u, position, h0, h1,
        [&](int h) {
          if (h < a.H) return a.q.x + t * a.q.xt + h * a.q.xh;
          h -= a.H;
          return h < a.G ? a.kn + t * a.nt + h * a.nh : a.vn + t * a.nt + (h - a.G) * a.nh;
        },
        [&](int h) -> uint16_t * {
          if (h < a.H) return a.q.out + t * a.q.ot + h * a.q.oh;
          if (place < 0) return nullptr;
          h -= a.H;
          return h < a.G ? a.k + place + h * a.hs : a.v + place + (h - a.G) * a.hs;
        },
        [&](int h) { return h < a.H + a.G; });
  }
}

template <int W>
cudaError_t launch_w(RotaryArgs &a, bool inter, bool bf16, cudaStream_t s) {
  const int rows = 32 / std::min(unit_count<W>(a.rope), 32), all = a.H + 2 * a.G;
  const int64_t groups = (a.T + rows - 1) / rows;
  a.parts = head_parts(groups, all, 4864);  // 152 SMs x 8 blocks x 4 warps, one wave
  a.per = ((all + a.parts - 1) / a.parts + 1) / 2 * 2;
  a.parts = (all + a.per - 1) / a.per;
  const unsigned blocks = (unsigned)((groups * a.parts + RO_WARPS - 1) / RO_WARPS);
  if (inter && bf16) rotary_kernel<W, true, true><<<blocks, RO_WARPS * 32, 0, s>>>(a);
  else if (inter) rotary_kernel<W, true, false><<<blocks, RO_WARPS * 32, 0, s>>>(a);
  else if (bf16) rotary_kernel<W, false, true><<<blocks, RO_WARPS * 32, 0, s>>>(a);
  else rotary_kernel<W, false, false><<<blocks, RO_WARPS * 32, 0, s>>>(a);
  return cudaGetLastError();
}

int launch(RotaryArgs &a, bool wide, bool inter, bool bf16, void *stream, char *err, size_t errlen) {
  if (!(a.status = status_word())) return fail(err, errlen, DS_ERR_CUDA, "no CUDA device");
  const cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = wide ? launch_w<8>(a, inter, bf16, s) : launch_w<1>(a, inter, bf16, s);
  return e == cudaSuccess ? DS_OK : cuda_fail(err, errlen, e, "rotary");
}

}  // namespace
}  // namespace dsm

using namespace dsm;

extern "C" {

int ds_moe_rope_init(ds_moe_rope *rope, int32_t dim, int32_t first, int32_t interleaved, double base, int32_t scaling,
                     double factor, int64_t original, double beta_fast, double beta_slow, double amplitude, char *err,
                     size_t errlen) {
  if (!rope) return fail(err, errlen, DS_ERR_INVALID_ARG, "rope is NULL");
  if (dim < 2 || dim > 128 || dim % 2 || first < 0 || first > 128 - dim)
    return fail(err, errlen, DS_ERR_INVALID_ARG, "dim=%d from element %d: need an even number within 128", dim, first);
  if (interleaved != 0 && interleaved != 1) return fail(err, errlen, DS_ERR_INVALID_ARG, "interleaved must be 0 or 1");
  if (!(base >= 1.0) || !isfinite(base)) return fail(err, errlen, DS_ERR_INVALID_ARG, "base must be finite and >= 1");
  if (scaling < DS_ROPE_NONE || scaling > DS_ROPE_YARN) return fail(err, errlen, DS_ERR_INVALID_ARG, "unknown scaling %d", scaling);
  if (scaling == DS_ROPE_NONE) factor = 1.0;
  if (!(factor >= 1.0) || !isfinite(factor)) return fail(err, errlen, DS_ERR_INVALID_ARG, "factor must be finite and >= 1");
  if (scaling == DS_ROPE_NTK && dim < 4) return fail(err, errlen, DS_ERR_INVALID_ARG, "DS_ROPE_NTK needs dim >= 4");
  if (beta_fast == 0.0 && beta_slow == 0.0) beta_fast = 32.0, beta_slow = 1.0;
  if (scaling == DS_ROPE_YARN &&
      (original < 1 || !(beta_slow > 0.0) || !(beta_fast > beta_slow) || !isfinite(beta_fast) || !(base > 1.0)))
    return fail(err, errlen, DS_ERR_INVALID_ARG, "DS_ROPE_YARN needs original >= 1, beta_fast > beta_slow > 0 and base > 1");
  if (!isfinite(amplitude) || !(amplitude >= 0.0) || amplitude > FLT_MAX)
    return fail(err, errlen, DS_ERR_INVALID_ARG, "amplitude must be finite and >= 0");
  if (amplitude == 0.0) amplitude = scaling == DS_ROPE_YARN ? 0.1 * log(factor) + 1.0 : 1.0;
  const double pi2 = 6.283185307179586476925;
  if (scaling == DS_ROPE_NTK) base *= pow(factor, dim / (dim - 2.0));
  if (!isfinite(base)) return fail(err, errlen, DS_ERR_INVALID_ARG, "base and factor are too large");
  // pairs before `low` turn more than beta_fast times over the trained
  // length, pairs from `high` on fewer than beta_slow times
  double low = 0.0, high = 0.0;
  if (scaling == DS_ROPE_YARN) {
    auto turning = [&](double times) { return dim * log((double)original / (times * pi2)) / (2.0 * log(base)); };
    low = std::max(floor(turning(beta_fast)), 0.0);
    high = std::min(ceil(turning(beta_slow)), dim - 1.0);
  }
  rope->dim = dim;
  rope->first = first;
  rope->interleaved = interleaved;
  rope->amplitude = (float)amplitude;
  for (int i = 0; i < 64; ++i) {
    if (i >= dim / 2) {
      rope->turns[i] = 0;
      continue;
    }
    double f = pow(base, -2.0 * i / dim);
    if (scaling == DS_ROPE_LINEAR) f /= factor;
    if (scaling == DS_ROPE_YARN) {
      const double r = std::min(1.0, std::max(0.0, (i - low) / std::max(high - low, 0.001)));
      f = f * (1.0 - r) + f / factor * r;
    }
    rope->turns[i] = (uint64_t)ldexp(f / pi2, 64);  // (f <= 1)
  }
  return DS_OK;
}

int ds_moe_rotary(const ds_moe_rope *rope, int32_t dtype, int32_t n_head, int32_t head_dim,
                  const ds_moe_rope_rows *rows, const int32_t *positions, int64_t T, void *stream, char *err,
                  size_t errlen) {
  if (head_dim < 1 || head_dim > 128) return fail(err, errlen, DS_ERR_UNSUPPORTED, "head_dim=%d: need 1..128", head_dim);
  if (n_head < 1 || n_head > 1024) return fail(err, errlen, DS_ERR_INVALID_ARG, "n_head=%d: need 1..1024", n_head);
  if (dtype != DS_BF16 && dtype != DS_F16) return fail(err, errlen, DS_ERR_INVALID_ARG, "dtype must be DS_BF16 or DS_F16");
  int rc = check_rope(rope, head_dim, err, errlen);
  if (rc) return rc;
  if (T < 0 || T > (1 << 24)) return fail(err, errlen, DS_ERR_INVALID_ARG, "T=%lld out of range", (long long)T);
  if (T == 0) return DS_OK;
  if (!rows || !positions) return fail(err, errlen, DS_ERR_INVALID_ARG, "rows and positions are required");
  if ((rc = check_rope_rows(rows, T, n_head, head_dim, err, errlen))) return rc;
  if (!aligned(positions, 4)) return fail(err, errlen, DS_ERR_INVALID_ARG, "positions must be aligned to its elements");
  RotaryArgs a{};
  a.rope = rope_of(rope, head_dim);
  a.q = rows_of(rows);
  a.H = n_head;
  a.positions = positions;
  a.T = T;
  return launch(a, rope_wide(a.rope) && rows_wide(a.q, T, n_head), rope->interleaved, dtype == DS_BF16, stream, err, errlen);
}

int ds_moe_kv_append_rotary(const ds_moe_attn_shape *shape, const ds_moe_kv_cache *cache, const ds_moe_rope *rope,
                            const void *k_new, const void *v_new, int64_t token_stride, int64_t head_stride,
                            const ds_moe_rope_rows *q, const int64_t *slots, const int32_t *positions, int64_t T,
                            void *stream, char *err, size_t errlen) {
  int rc = check_attn_shape(shape, err, errlen);
  if (rc) return rc;
  if ((rc = check_kv_cache(shape, cache, true, err, errlen))) return rc;
  const int D = shape->head_dim, G = shape->n_head_kv;
  if ((rc = check_rope(rope, D, err, errlen))) return rc;
  if (T < 0 || T > (1 << 24)) return fail(err, errlen, DS_ERR_INVALID_ARG, "T=%lld out of range", (long long)T);
  if (T == 0) return DS_OK;
  if (!k_new || !v_new || !slots || !positions)
    return fail(err, errlen, DS_ERR_INVALID_ARG, "k_new, v_new, slots and positions are required");
  if (!aligned(k_new, 2) || !aligned(v_new, 2) || !aligned(slots, 8) || !aligned(positions, 4))
    return fail(err, errlen, DS_ERR_INVALID_ARG, "arrays must be aligned to their elements");
  if (token_stride < 0 || head_stride < 0) return fail(err, errlen, DS_ERR_INVALID_ARG, "negative stride");
  if (q && (rc = check_rope_rows(q, T, shape->n_head, D, err, errlen))) return rc;
  RotaryArgs a{};
  a.rope = rope_of(rope, D);
  a.q = rows_of(q);
  a.H = q ? shape->n_head : 0;
  a.G = G;
  a.kn = (const uint16_t *)k_new; a.vn = (const uint16_t *)v_new; a.nt = token_stride; a.nh = head_stride;
  a.k = (uint16_t *)cache->k; a.v = (uint16_t *)cache->v;
  a.n_slots = cache->n_pages * shape->page_size; a.ps = cache->page_stride; a.rs = cache->row_stride; a.hs = cache->head_stride;
  a.page = shape->page_size;
  a.slots = slots; a.positions = positions; a.T = T;
  auto fits = [](int64_t n, int64_t s) { return n <= 1 || s % 8 == 0; };
  const bool wide = rope_wide(a.rope) && (!q || rows_wide(a.q, T, a.H)) && aligned(k_new, 16) && aligned(v_new, 16) &&
                    aligned(cache->k, 16) && aligned(cache->v, 16) && fits(T, token_stride) && fits(G, head_stride) &&
                    fits(cache->n_pages, a.ps) && fits(a.page, a.rs) && fits(G, a.hs);
  return launch(a, wide, rope->interleaved, shape->dtype == DS_BF16, stream, err, errlen);
}

}  // extern "C"
