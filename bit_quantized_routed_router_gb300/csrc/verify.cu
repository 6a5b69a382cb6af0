// The check of drafted tokens (ds_moe_verify_drafts): keep drafts while the
// target allows, then draw one token from what is left of its distribution.
//
// With draft distribution q and target p a draft x ~ q is kept with
// probability min(1, p(x) / q(x)), and at the first refusal a token is drawn
// from max(p - q, 0), normalised; the tokens kept are then distributed as p's
// own (speculative sampling, Leviathan et al. 2023, Chen et al. 2023).
#include <cooperative_groups.h>

#include "common.cuh"
#include "errors.h"
#include "internal.h"
#include "serving.cuh"

namespace dsm {
namespace {

namespace cg = cooperative_groups;

constexpr int VD_THREADS = 256, VD_WARPS = VD_THREADS / 32;
constexpr int VD_CLUSTER = 8;             // blocks a request at most
constexpr int VD_RESIDENT = 4;            // blocks that an SM holds (64 registers a thread)
constexpr int VD_CHUNK = 256;             // vocabulary entries a chunk sum covers
constexpr int VD_MAX_VOCAB = 1 << 22;

struct VerifyArgs {
  const void *p, *q;
  int64_t p_stride, q_stride;
  int T, V, R, max_new;
  const int32_t *tokens, *cu;
  const float *u_accept, *u_sample;
  int32_t *out, *n_accepted;
  float unit;  // 2^22 / 2^k: see weights()
  unsigned *status;
};

template <bool BF16>
__device__ __forceinline__ float prob(const void *base, int64_t i) {
  return BF16 ? bf16_to_f32(__ldg((const uint16_t *)base + i)) : __ldg((const float *)base + i);
}

// What sampling takes a probability for: NaN and negative ones for 0, those
// above 1 for 1 (reported).  Others are what they are: their bits, as unsigned
// words, are those of 1 at most (-0 is handled with the rest, and not
// reported).
constexpr uint32_t ONE_BITS = 0x3F800000u;
__device__ __forceinline__ float clean(float p, bool &bad) {
  if (p >= 0.f && p <= 1.f) return fabsf(p);
  bad = true;
  return p > 1.f ? 1.f : 0.f;
}

// Probabilities of 8 entries x0, x0 + step, ... of a row, all loads under way
// at once; ALL: every entry is in the vocabulary.
template <bool BF16, bool ALL>
__device__ __forceinline__ void load8(const void *base, int64_t row, int x0, int step, int V, float v[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = base && (ALL || x0 + i * step < V) ? prob<BF16>(base, row + x0 + i * step) : 0.f;
}

// Weights of those entries of a row that is sampled from: max(p - q, 0) with
// the target's p and the draft's q (zeros where it is not to count), or none
// at the draft `sure`.
//
// A weight is a whole number of 2^-(44 - k) units, hi * 2^22 + lo, with `unit`
// = 2^(22 - k): k is 0 for vocabularies below 2^19 and goes up to 4 at 2^22,
// so that a vocabulary of ones adds up to less than 2^63.  With q held to at
// most p the difference is s plus an exact error e (Dekker's fast two-sum);
// adding 1.5 * 2^23 rounds to whole numbers, which are the low bits of the
// sum.  Sums of such numbers are exact, so no order of adding changes the
// token that is drawn; fp64 adds would be slower than HBM here.
__device__ __forceinline__ int64_t weights(float pv[8], float qv[8], float unit, int sure, int x0, int step, int64_t each[8], bool &bad) {
  constexpr float MAGIC = 12582912.f, LOW = 4194304.f;  // 1.5 * 2^23, 2^22
  constexpr uint32_t MAGIC_BITS = 0x4B400000u;
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, max(__float_as_uint(pv[i]), __float_as_uint(qv[i])));
  if (top > ONE_BITS) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      pv[i] = clean(pv[i], bad);
      qv[i] = clean(qv[i], bad);
    }
  }
  if (sure >= 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) pv[i] = x0 + i * step == sure ? 0.f : pv[i];
  }
  uint32_t hs = 0, ls = 0;  // (modulo 2^32)
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y = fminf(pv[i], qv[i]), s = pv[i] - y, e = (pv[i] - s) - y;
    const float t = fmaf(s, unit, MAGIC);
    const float rem = fmaf(e, unit, fmaf(s, unit, -(t - MAGIC)));
    const uint32_t hi = __float_as_uint(t) - MAGIC_BITS, lo = __float_as_uint(fmaf(rem, LOW, MAGIC)) - MAGIC_BITS;
    if (each) each[i] = ((int64_t)(int)hi << 22) + (int)lo;
    hs += hi;
    ls += lo;
  }
  return ((int64_t)(int)hs << 22) + (int)ls;
}

__device__ __forceinline__ int64_t warp_sum64(int64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the earlier lanes and this one.
__device__ __forceinline__ int64_t warp_scan64(int64_t v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t w = __shfl_up_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) >= o) v += w;
  }
  return v;
}

// Whole part of u * total, exactly, for 0 <= u < 1: u is m 2^(e - 150), the
// product 87 bits at most.
__device__ __forceinline__ int64_t whole_part(float u, int64_t total) {
  const uint32_t w = __float_as_uint(u) & 0x7FFFFFFFu, e = w >> 23;  // (below 127)
  const uint64_t m = e ? (w & 0x7FFFFFu) | 0x800000u : w;
  const int down = 150 - (int)(e ? e : 1);  // 24 at least
  const uint64_t lo = m * (uint64_t)total, hi = __umul64hi(m, (uint64_t)total);
  return (int64_t)(down < 64 ? hi << (64 - down) | lo >> down : down < 128 ? hi >> (down - 64) : 0);
}

// A cluster of blocks a request, each with a part of the vocabulary: pass 1
// sums the row chunk by chunk (a warp a chunk), the blocks exchange their
// totals through shared memory, and the block that the drawn number falls
// into finds the chunk and the entry in it.  Bound by the dependent loads that
// say which rows are read (lengths, drafts, their probabilities), and then by
// the instructions an entry takes rather than by its bytes: 96 requests of
// 100,003 entries of 32 bits, rows in L2, 15 us with a draft row and 15.5 without
// one, 17 and 16 us with 16-bit entries; 20 us from HBM, 3.4 TB/s; one request of
// 32,768 entries 6.2 us.
template <bool BF16>
__global__ void __launch_bounds__(VD_THREADS, VD_RESIDENT) verify_kernel(const VerifyArgs a) {
  extern __shared__ int64_t chunk[];
  __shared__ int64_t totals[2][VD_CLUSTER], part[VD_WARPS];
  const cg::cluster_group cluster = cg::this_cluster();
  cluster.barrier_arrive();  // this block has begun: its shared memory can be written to
  const int rank = cluster.block_rank(), ranks = cluster.num_blocks();
  const int r = blockIdx.x / ranks, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c0 = a.cu[r], c1 = a.cu[r + 1];
  const int t0 = min(max(c0, 0), a.T), n = min(min(max(c1, t0), a.T) - t0, a.max_new);
  bool bad = c0 != t0 || c1 != t0 + n;
  int32_t *out = a.out + (int64_t)r * a.max_new;
  // every warp counts the drafts that are kept: a lane a draft
  int kept = 0, sure = -1;
  for (; kept < n - 1;) {
    const int row = t0 + kept + lane;
    int x = -1;
    bool keep = false;
    if (kept + lane < n - 1) {
      x = a.tokens[row + 1];
      if (x >= 0 && x < a.V) {
        const float pv = prob<BF16>(a.p, (int64_t)row * a.p_stride + x);
        const float qv = a.q ? prob<BF16>(a.q, (int64_t)row * a.q_stride + x) : 1.f;
        keep = (double)a.u_accept[row] * (double)qv < (double)pv;  // (products of two fp32 numbers are exact in fp64)
      }
    }
    const unsigned refuse = __ballot_sync(0xffffffffu, !keep);
    if (refuse) {
      const int f = __ffs(refuse) - 1;
      kept += f;
      x = __shfl_sync(0xffffffffu, x, f);
      if (kept < n - 1) {
        if (x >= 0 && x < a.V) sure = x;
        else bad = true;
      }
      break;
    }
    kept += 32;
  }
  const bool refused = kept < n - 1;
  if (rank == 0) {
    if (tid == 0) a.n_accepted[r] = max(kept, 0);
    for (int i = tid; i < a.max_new; i += VD_THREADS)
      if (i != kept || n == 0) out[i] = i < kept ? a.tokens[t0 + i + 1] : -1;
  }
  if (n > 0) {
    const int64_t prow = (int64_t)(t0 + kept) * a.p_stride, qrow = (int64_t)(t0 + kept) * a.q_stride;
    const void *q = refused ? a.q : nullptr;
    if (!refused || q) sure = -1;
    const int chunks = (a.V + VD_CHUNK - 1) / VD_CHUNK, per = (chunks + ranks - 1) / ranks;
    const int first = min(chunks, rank * per), mine = min(chunks, first + per) - first;
    int64_t total = 0, before = 0, own = 0;
    for (int turn = 0; turn < 2; ++turn) {
      int64_t sum = 0;
      float pv[8], qv[8], pn[8], qn[8];
      auto load = [&](int c, float p8[8], float q8[8]) {
        const int x0 = (first + c) * VD_CHUNK + lane;
        if ((first + c + 1) * VD_CHUNK <= a.V) {
          load8<BF16, true>(a.p, prow, x0, 32, a.V, p8);
          load8<BF16, true>(q, qrow, x0, 32, a.V, q8);
        } else {
          load8<BF16, false>(a.p, prow, x0, 32, a.V, p8);
          load8<BF16, false>(q, qrow, x0, 32, a.V, q8);
        }
      };
      if (warp < mine) load(warp, pn, qn);
      for (int c = warp; c < mine; c += VD_WARPS) {
#pragma unroll
        for (int i = 0; i < 8; ++i) pv[i] = pn[i], qv[i] = qn[i];
        if (c + VD_WARPS < mine) load(c + VD_WARPS, pn, qn);  // (the next chunk's loads, before this one's arithmetic)
        const int64_t s = warp_sum64(weights(pv, qv, a.unit, sure, (first + c) * VD_CHUNK + lane, 32, nullptr, bad));
        if (lane == 0) chunk[c] = s;
        sum += s;
      }
      if (lane == 0) part[warp] = sum;
      __syncthreads();
      // the others have begun too (that they are scheduled together does not
      // say so; the loads since the arrival hide the wait)
      if (turn == 0) cluster.barrier_wait();
      if (tid < ranks) {  // this block's total to every block
        int64_t s = 0;
#pragma unroll
        for (int w = 0; w < VD_WARPS; ++w) s += part[w];
        *cluster.map_shared_rank(&totals[turn][rank], tid) = s;
      }
      cluster.sync();
      total = before = 0;
#pragma unroll
      for (int i = 0; i < VD_CLUSTER; ++i) {
        if (i >= ranks) break;
        if (i < rank) before += totals[turn][i];
        total += totals[turn][i];
      }
      own = totals[turn][rank];
      if (total > 0 || (!q && sure < 0)) break;
      q = nullptr;  // nothing left above the draft: the target itself
      sure = -1;
    }
    if (total <= 0) {
      bad = true;
      if (rank == 0 && tid == 0) out[kept] = -1;
    } else if (warp == 0) {
      // the entry drawn is the least whose cumulative weight exceeds u * total
      const float u = a.u_sample[r];
      if (!(u >= 0.f && u < 1.f)) bad = true;
      const int64_t thr = u >= 1.f ? total - 1 : u >= 0.f ? whole_part(u, total) : 0;
      if (before <= thr && thr < before + own) {  // it is in this block's entries
        int at = 0;
        for (int b = 0; b < mine; b += 32) {
          const int64_t v = b + lane < mine ? chunk[b + lane] : 0, incl = warp_scan64(v);
          const unsigned pass = __ballot_sync(0xffffffffu, before + incl > thr);
          if (pass) {
            const int f = __ffs(pass) - 1;
            at = b + f;
            before += __shfl_sync(0xffffffffu, incl - v, f);
            break;
          }
          before += __shfl_sync(0xffffffffu, incl, 31);
        }
        // each lane takes 8 entries in a row of that chunk
        const int x0 = (first + at) * VD_CHUNK + lane * 8;
        bool none = false;
        int64_t each[8];
        float pv[8], qv[8];
        load8<BF16, false>(a.p, prow, x0, 1, a.V, pv);
        load8<BF16, false>(q, qrow, x0, 1, a.V, qv);
        const int64_t v = weights(pv, qv, a.unit, sure, x0, 1, each, none), incl = warp_scan64(v);
        const unsigned pass = __ballot_sync(0xffffffffu, before + incl > thr);
        if (pass && lane == __ffs(pass) - 1) {
          int64_t run = before + incl - v;
          int x = x0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (run <= thr) x = x0 + i;
            run += each[i];
          }
          out[kept] = x;
        }
      }
    }
  } else {
    cluster.barrier_wait();
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
  if (n_requests < 0 || n_requests > (1 << 24) || max_new < 0)
    return fail(err, errlen, DS_ERR_INVALID_ARG, "n_requests or max_new out of range");
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
  int k = 0;
  while (vocab >> (19 + k)) ++k;
  VerifyArgs a{target, draft, target_stride, draft_stride, (int)T, vocab, n_requests, max_new, tokens, cu_new, u_accept,
               u_sample, out_tokens, n_accepted, (float)(1 << (22 - k)), status_word()};
  if (!a.status) return fail(err, errlen, DS_ERR_CUDA, "no CUDA device");
  const int chunks = (vocab + VD_CHUNK - 1) / VD_CHUNK, sms = device_sms();
  if (!sms) return fail(err, errlen, DS_ERR_CUDA, "no CUDA device");
  // as many blocks a request as one wave of blocks has room for, and no more
  // than there are chunks for their warps (100,003 entries, rows in L2: 96
  // requests 27 us with 8, in two waves, 15.4 with 6, 16.5 with 4; from HBM 200
  // requests 42 us with 2, 46 with 3, so odd sizes are left out at the low end)
  int ranks = VD_CLUSTER;
  auto fewer = [](int n) { return n > 4 ? n - 1 : n / 2; };
  while (ranks > 1 && ((int64_t)n_requests * ranks > sms * VD_RESIDENT || chunks <= VD_WARPS * fewer(ranks))) ranks = fewer(ranks);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)n_requests * ranks);
  cfg.blockDim = dim3(VD_THREADS);
  cfg.dynamicSmemBytes = sizeof(int64_t) * ((chunks + ranks - 1) / ranks);
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ranks;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  static OncePerDevice once;  // (the largest vocabulary's sums, in one block)
  cudaError_t e = once_per_device(once, []() {
    const int most = (int)sizeof(int64_t) * (VD_MAX_VOCAB / VD_CHUNK);
    const cudaError_t f = cudaFuncSetAttribute(verify_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    return f != cudaSuccess ? f : cudaFuncSetAttribute(verify_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  });
  if (e == cudaSuccess)
    e = dtype == DS_F32 ? cudaLaunchKernelEx(&cfg, verify_kernel<false>, a) : cudaLaunchKernelEx(&cfg, verify_kernel<true>, a);
  return e == cudaSuccess ? DS_OK : cuda_fail(err, errlen, e, "verify drafts");
}

}  // extern "C"
