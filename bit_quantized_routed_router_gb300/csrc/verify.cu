// The check of drafted tokens (ds_moe_verify_drafts): keep drafts while the
// target allows, then draw one token from what is left of its distribution.
//
// With draft distribution q and target p a draft x ~ q is kept with
// probability min(1, p(x) / q(x)), and at the first refusal a token is drawn
// from max(p - q, 0), normalised; the tokens kept are then distributed as p's
// own (speculative sampling, Leviathan et al. 2023, Chen et al. 2023).
#include "common.cuh"
#include "errors.h"
#include "internal.h"
#include "serving.cuh"

namespace dsm {
namespace {

constexpr int VD_THREADS = 1024;
constexpr int VD_CHUNK = 1024;            // vocabulary entries a chunk sum covers
constexpr int VD_MAX_VOCAB = 1 << 22;

struct VerifyArgs {
  const void *p, *q;
  int64_t p_stride, q_stride;
  int T, V, R, max_new;
  const int32_t *tokens, *cu;
  const float *u_accept, *u_sample;
  int32_t *out, *n_accepted;
  unsigned *status;
};

template <bool BF16>
__device__ __forceinline__ float prob(const void *base, int64_t i) {
  return BF16 ? bf16_to_f32(((const uint16_t *)base)[i]) : ((const float *)base)[i];
}

// What sampling takes a probability for: NaN and negative ones for 0, those
// above 1 for 1 (reported).
__device__ __forceinline__ float clean(float p, bool &bad) {
  if (p >= 0.f && p <= 1.f) return p;
  bad = true;
  return p > 1.f ? 1.f : 0.f;
}

// max(p - q, 0) as a whole number of 2^-44 units, hi * 2^22 + lo with
// hi <= 2^22 and |lo| <= 2^21 + 1.  The difference is held as a rounded sum
// and its exact error (Knuth's two-sum); adding 1.5 * 2^23 rounds to whole
// numbers.  Sums of such numbers are exact, so no order of adding changes
// the token that is drawn; fp64 adds would be slower than HBM here.
__device__ __forceinline__ void residual(float p, float q, int &hi, int &lo) {
  const float MAGIC = 12582912.f, UNIT = 4194304.f;  // 1.5 * 2^23, 2^22
  const float s = p - q, b = s - p, e = (p - (s - b)) + (-q - b);
  const float t = fmaf(s, UNIT, MAGIC), h = t - MAGIC;
  const float rem = fmaf(s, UNIT, -h) + e * UNIT;
  const float u = fmaf(rem, UNIT, MAGIC);
  const bool some = s > 0.f;
  hi = some ? __float_as_int(t) - __float_as_int(MAGIC) : 0;
  lo = some ? __float_as_int(u) - __float_as_int(MAGIC) : 0;
}

// Weight of entry x of a row that is sampled from: the target's, less the
// draft's when q is given, or less all of it at the draft `sure`.
template <bool BF16>
__device__ __forceinline__ void weight(const void *p, int64_t prow, const void *q, int64_t qrow, int sure, int x, int &hi,
                                       int &lo, bool &bad) {
  const float pv = clean(prob<BF16>(p, prow + x), bad);
  const float qv = q ? clean(prob<BF16>(q, qrow + x), bad) : (x == sure ? 1.f : 0.f);
  residual(pv, qv, hi, lo);
}

__device__ __forceinline__ int64_t warp_sum64(int64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// One block a request.  Pass 1 sums the row chunk by chunk (a warp a chunk);
// pass 2 finds the chunk that the drawn number falls into and the entry in it.
template <bool BF16>
__global__ void __launch_bounds__(VD_THREADS) verify_kernel(const VerifyArgs a) {
  extern __shared__ int64_t chunk[];
  __shared__ int s_kept, s_sure;
  __shared__ int64_t s_total;
  const int r = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c0 = a.cu[r], c1 = a.cu[r + 1];
  const int t0 = min(max(c0, 0), a.T), n_all = min(max(c1, t0), a.T) - t0, n = min(n_all, a.max_new);
  bool bad = c0 != t0 || c1 != t0 + n;
  int32_t *out = a.out + (int64_t)r * a.max_new;
  if (tid == 0) {
    int kept = 0, sure = -1;
    for (; kept < n - 1; ++kept) {
      const int row = t0 + kept, x = a.tokens[row + 1];
      if (x < 0 || x >= a.V) {
        bad = true;
        break;
      }
      const float pv = prob<BF16>(a.p, (int64_t)row * a.p_stride + x);
      const float qv = a.q ? prob<BF16>(a.q, (int64_t)row * a.q_stride + x) : 1.f;
      // products of two fp32 numbers are exact in fp64
      if (!((double)a.u_accept[row] * (double)qv < (double)pv)) {
        sure = x;
        break;
      }
    }
    s_kept = kept;
    s_sure = sure;
    a.n_accepted[r] = kept;
  }
  __syncthreads();
  const int kept = s_kept;
  const bool refused = kept < n - 1;
  for (int i = tid; i < a.max_new; i += VD_THREADS)
    if (i != kept || n == 0) out[i] = i < kept ? a.tokens[t0 + i + 1] : -1;
  if (n > 0) {
    const int64_t prow = (int64_t)(t0 + kept) * a.p_stride, qrow = (int64_t)(t0 + kept) * a.q_stride;
    const void *q = refused ? a.q : nullptr;
    int sure = refused ? s_sure : -1;
    const int chunks = (a.V + VD_CHUNK - 1) / VD_CHUNK;
    int64_t total = 0;
    for (int turn = 0; turn < 2; ++turn) {
      for (int c = warp; c < chunks; c += VD_THREADS / 32) {
        int hs = 0, ls = 0;
        for (int x = c * VD_CHUNK + lane; x < min(a.V, (c + 1) * VD_CHUNK); x += 32) {
          int hi, lo;
          weight<BF16>(a.p, prow, q, qrow, sure, x, hi, lo, bad);
          hs += hi;
          ls += lo;
        }
        const int64_t sum = warp_sum64(((int64_t)hs << 22) + ls);
        if (lane == 0) chunk[c] = sum;
      }
      __syncthreads();
      if (warp == 0) {
        int64_t v = 0;
        for (int c = lane; c < chunks; c += 32) v += chunk[c];
        v = warp_sum64(v);
        if (lane == 0) s_total = v;
      }
      __syncthreads();
      total = s_total;
      if (total > 0 || (!q && sure < 0)) break;
      q = nullptr;  // nothing left above the draft: the target itself
      sure = -1;
    }
    if (total <= 0) {
      bad = true;
      if (tid == 0) out[kept] = -1;
    } else if (warp == 0) {
      // the entry drawn is the least whose cumulative weight exceeds u * total
      const float u = a.u_sample[r];
      if (!(u >= 0.f && u < 1.f)) bad = true;
      int64_t thr = u >= 1.f ? total - 1 : u >= 0.f ? (int64_t)((double)u * (double)total) : 0;
      thr = min(thr, total - 1);
      // thr is less than the total, so some chunk passes it
      int64_t before = 0;
      int at = 0;
      for (int b = 0; b < chunks; b += 32) {
        int64_t v = b + lane < chunks ? chunk[b + lane] : 0, incl = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t w = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += w;
        }
        const unsigned pass = __ballot_sync(0xffffffffu, before + incl > thr);
        if (pass) {
          const int f = __ffs(pass) - 1;
          at = b + f;
          before += __shfl_sync(0xffffffffu, incl - v, f);
          break;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
      }
      // each lane takes 32 entries in a row of that chunk
      const int x0 = at * VD_CHUNK + lane * 32;
      int64_t v = 0;
      bool none = false;
      for (int x = x0; x < min(a.V, x0 + 32); ++x) {
        int hi, lo;
        weight<BF16>(a.p, prow, q, qrow, sure, x, hi, lo, none);
        v += ((int64_t)hi << 22) + lo;
      }
      int64_t incl = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t w = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += w;
      }
      const unsigned pass = __ballot_sync(0xffffffffu, before + incl > thr);
      if (pass && lane == __ffs(pass) - 1) {
        int64_t run = before + incl - v;
        for (int x = x0; x < min(a.V, x0 + 32); ++x) {
          int hi, lo;
          weight<BF16>(a.p, prow, q, qrow, sure, x, hi, lo, none);
          run += ((int64_t)hi << 22) + lo;
          if (run > thr) {
            out[kept] = x;
            break;
          }
        }
      }
    }
  }
  if (bad) flag(a.status, ST_DRAFT);
}

}  // namespace
}  // namespace dsm

using namespace dsm;

extern "C" {

int ds_moe_verify_drafts(const void *target, int64_t target_stride, const void *draft, int64_t draft_stride,
                         int32_t dtype, int64_t T, int32_t vocab, const int32_t *tokens, const int32_t *cu_new,
                         int32_t n_requests, int32_t max_new, const float *u_accept, const float *u_sample,
                         int32_t *out_tokens, int32_t *n_accepted, void *stream, char *err, size_t errlen) {
  if (dtype != DS_F32 && dtype != DS_BF16)
    return fail(err, errlen, DS_ERR_INVALID_ARG, "dtype must be DS_F32 or DS_BF16");
  if (vocab < 1 || vocab > VD_MAX_VOCAB)
    return fail(err, errlen, DS_ERR_INVALID_ARG, "vocab=%d: need 1..%d", vocab, VD_MAX_VOCAB);
  if (T < 0 || T > (1 << 24)) return fail(err, errlen, DS_ERR_INVALID_ARG, "T=%lld out of range", (long long)T);
  if (n_requests < 0 || max_new < 0)
    return fail(err, errlen, DS_ERR_INVALID_ARG, "negative n_requests or max_new");
  if (n_requests == 0) return DS_OK;
  if (max_new == 0) return fail(err, errlen, DS_ERR_INVALID_ARG, "max_new must be at least 1");
  if (T && (!target || !tokens || !u_accept))
    return fail(err, errlen, DS_ERR_INVALID_ARG, "target, tokens and u_accept are required");
  if (!cu_new || !u_sample || !out_tokens || !n_accepted)
    return fail(err, errlen, DS_ERR_INVALID_ARG, "cu_new, u_sample, out_tokens and n_accepted are required");
  if (T > 1 && (target_stride < vocab || (draft && draft_stride < vocab)))
    return fail(err, errlen, DS_ERR_INVALID_ARG, "a row stride is smaller than vocab");
  const size_t el = dtype == DS_F32 ? 4 : 2;
  if (!aligned(target, el) || !aligned(draft, el) || !aligned(tokens, 4) || !aligned(cu_new, 4) ||
      !aligned(u_accept, 4) || !aligned(u_sample, 4) || !aligned(out_tokens, 4) || !aligned(n_accepted, 4))
    return fail(err, errlen, DS_ERR_INVALID_ARG, "arrays must be aligned to their elements");
  VerifyArgs a{target, draft, target_stride, draft_stride, (int)T, vocab, n_requests, max_new, tokens, cu_new, u_accept,
               u_sample, out_tokens, n_accepted, status_word()};
  if (!a.status) return fail(err, errlen, DS_ERR_CUDA, "no CUDA device");
  const size_t smem = sizeof(int64_t) * ((vocab + VD_CHUNK - 1) / VD_CHUNK);
  if (dtype == DS_F32)
    verify_kernel<false><<<(unsigned)n_requests, VD_THREADS, smem, (cudaStream_t)stream>>>(a);
  else
    verify_kernel<true><<<(unsigned)n_requests, VD_THREADS, smem, (cudaStream_t)stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? DS_OK : cuda_fail(err, errlen, e, "verify drafts");
}

}  // extern "C"
