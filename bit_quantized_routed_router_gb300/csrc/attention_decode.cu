// Attention of few query rows a key head (one new token, or a few drafted
// ones, with the query heads that share the key head): bound by reading the
// cache.
//
// The keys are the rows of the tensor-core tiles and the queries their
// columns: S^T = K Q^T is 128 keys x N, O^T += V^T P^T is head_dim x N, with
// N = 16 or 32, so the work of the softmax and of the matrix products
// goes with the query rows there are, not with a tile of 128 of them.  A
// block is
//
//   two producer warps  copy the tiles' keys (and the query rows), and the
//                   values, out of their pages (TMA, 128-byte swizzle) into a
//                   ring of slots each;
//   MMA thread      S^T of the next four tiles ahead, O^T of a tile when its
//                   probabilities are there;
//   two groups of four warps, which take the tiles in turn, each with its own
//                   scores, running maxima and accumulators: one exponentiates
//                   while the other's products run.  A thread owns one key of
//                   the tile, and one element of the head in the accumulators.
//
// Maxima are raised lazily (AT_SLACK), so that a tile usually costs its group
// one barrier.  The two groups' sums are joined at the end of a segment.
// Probabilities are rounded to the 16-bit type of the values, which the second
// product takes; their sums, the maxima and the accumulators are 32 bits.
//
// Measured: 64 requests of 200 to 8200 keys, 8 key heads of 128 (1.1 GB of
// cache) 174 us, 6.3 TB/s; 3 of 68,000 to 93,000 keys (0.98 GB) 160 us; one of
// 138 keys 11 us, the set-up of a block, its tiles' way from memory, and the
// join.  Heads of 64 in pages of rows are 128-byte pieces, which memory gives at
// 5.2 to 5.5 TB/s; with a head's rows together in the page 5.8 to 6.5 (64 and
// 300 requests, 8 key heads).
#include "attention_tc.cuh"

namespace dsm {
namespace {

constexpr int AD_THREADS = 352;  // two groups of 128, MMA warp, two producer warps
constexpr int AD_MMA = 8, AD_KEYS = 9, AD_VALUES = 10;
// Tiles that an item costs besides its own (200 requests of up to 3000 keys, one
// or two tokens: 226 us with 2, 239 with 4; 29 requests with up to 28 rows: 39
// with 1, 33 with 2, 29 with 4).
constexpr int AD_ITEM = 2;
constexpr int AD_AHEAD = 4;  // tiles whose scores are computed ahead: two buffers of scores a group

template <int N, int DP>
struct AdCfg {
  static constexpr uint32_t TILE = AT_KEYS * DP * 2;
  static constexpr uint32_t Q = N * DP * 2, P = N * AT_KEYS * 2;
  static constexpr int TMEM = 8 * N;  // columns: four tiles' scores, two groups' sums
  static constexpr int ROOM = 227 * 1024 - 1024 - 2 * (Q + P) - 8192;
  static constexpr int SLOTS = ROOM / (2 * (int)TILE) < 6 ? ROOM / (2 * (int)TILE) : 6;  // of keys, and of values
};

template <int N, int SLOTS>
struct AdShared {
  uint64_t full[2][SLOTS], empty[2][SLOTS];  // keys, values
  uint64_t q_full[2], q_empty[2], s_full[AD_AHEAD], p_full[2], o_full[2], drain;
  alignas(16) float ref[2][N];     // running maximum of each query row, by group
  alignas(16) float factor[2][N];  // what a raised maximum multiplies sums with
  alignas(16) float2 weight[N];    // of a segment's row: of its finishing group's sums, and of the other's
  int64_t place[N];                // where the row goes
  float top[2][4][N];   // a tile's largest score, by warp
  float sum[2][4][N];   // sums of probabilities, by warp
  uint32_t odd[2][4];   // keys whose values are not all finite
  int64_t part[AD_THREADS / 32];
  Start start;
  uint32_t tmem;
  int gave_up;
};

template <int N, int DP, bool BF16>
__global__ void __launch_bounds__(AD_THREADS, 1)
    attention_decode_kernel(const AttnArgs a, const Pieces pieces, const __grid_constant__ CUtensorMap tm_q,
                            const __grid_constant__ KvMaps tm_k, const __grid_constant__ KvMaps tm_v, int rows) {
  using C = AdCfg<N, DP>;
  constexpr int SLOTS = C::SLOTS;
  constexpr Plan PLAN = {1 << 20, 1 << 20, AD_ITEM};  // one block of tokens a request
  extern __shared__ uint8_t raw[];
  uint8_t *smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  uint8_t *kring = smem, *vring = kring + SLOTS * C::TILE, *qbuf = vring + SLOTS * C::TILE, *pbuf = qbuf + 2 * C::Q;
  typedef AdShared<N, SLOTS> Sh;
  Sh &S = *reinterpret_cast<Sh *>(pbuf + 2 * C::P);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  asm volatile("griddepcontrol.launch_dependents;");
  const RawSpan raw0 = first_request<AD_THREADS>(a);  // (under way while the block is set up)

  if (tid < 2 * SLOTS) {
    mbar_init(&S.full[tid / SLOTS][tid % SLOTS], 1);
    mbar_init(&S.empty[tid / SLOTS][tid % SLOTS], 1);
    fence_mbar_init();
  } else if (tid >= 32 && tid < 32 + AD_AHEAD) {
    const int i = tid - 32;
    mbar_init(&S.s_full[i], 1);
    if (i < 2) {
      mbar_init(&S.q_full[i], 1);
      mbar_init(&S.q_empty[i], 1);
      mbar_init(&S.p_full[i], 4);
      mbar_init(&S.o_full[i], 1);
    }
    if (i == 0) mbar_init(&S.drain, 1), S.gave_up = 0;
    fence_mbar_init();
  } else if (tid == 64) {
    const CUtensorMap *maps[3] = {&tm_q, &tm_k.one, &tm_v.one};
    for (int i = 0; i < 3; ++i) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(maps[i])) : "memory");
  }
  if (tid == 0) {
    pieces.what[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
    pieces.what[2 * blockIdx.x + 1] = make_int4(0, 0, 0, 0);
  }
  __syncwarp();
  if (warp == AD_MMA) tmem_alloc<C::TMEM>(&S.tmem);
  // query rows that no copy fills stay zero
  for (int i = tid; i < (int)(2 * C::Q / 16); i += AD_THREADS) reinterpret_cast<uint4 *>(qbuf)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async();
  find_start<AD_THREADS>(a, raw0, PLAN, &S.start, S.part);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem;  // scores of tile f at (f mod 4) N, sums of group i at (4 + i) N
  Segments s;
  s.init(a, PLAN, S.start);
  if (warp == AD_KEYS || warp == AD_VALUES) {
    // ------------------------------------------------------------ copies --
    const bool keys = warp == AD_KEYS;
    const KvMaps *maps = keys ? &tm_k : &tm_v;
    bool ok = true, bad = false;
    int segs = 0, f = 0, i = 0;  // segments begun, tile of the stretch, of the segment
    TileRuns now, later;
    int head = s.h;
    if (s.count) now.find(a, s, s.tile, rows);
    for (; s.count; ++f) {
      if (i == 0) {
        head = s.h;
        if (keys) {
          const int b = s.index & 1;
          if (lane == 0 && s.index >= 2 && !at_wait(&S.q_empty[b], ((s.index >> 1) & 1) ^ 1, &S.gave_up, a.status)) ok = false;
          if (!__shfl_sync(0xffffffffu, ok, 0)) break;
          if (lane == 0) {
            const int tokens = N / a.g;
            mbar_arrive_expect_tx(&S.q_full[b], tokens * a.g * DP * 2);
#pragma unroll
            for (int x = 0; x < DP; x += 64)
              tma_load_3d(qbuf + b * C::Q + x / 64 * (N * 128), &tm_q, x, s.h * a.g, s.sp.t0, &S.q_full[b]);
          }
          __syncwarp();
          ++segs;
        }
      }
      if (++i == s.count) {
        s.next(a);
        i = 0;
      }
      if (s.count) later.find(a, s, s.tile + i, rows);
      const int sl = f % SLOTS;
      if (lane == 0 && f >= SLOTS && !at_wait(&S.empty[!keys][sl], ((f / SLOTS) & 1) ^ 1, &S.gave_up, a.status)) ok = false;
      if (!__shfl_sync(0xffffffffu, ok, 0)) break;
      now.copy<DP, true>(a, (keys ? kring : vring) + sl * C::TILE, &maps->one, &maps->two, head, rows, &S.full[!keys][sl], bad);
      now = later;
    }
    if (bad) flag(a.status, ST_PAGING);
    if (lane == 0) {  // every copy of this warp has landed before the block ends
      int off = 0;
      for (int g = max(0, f - SLOTS); g < f; ++g) at_wait(&S.full[!keys][g % SLOTS], (g / SLOTS) & 1, &off, a.status);
      for (int q = max(0, segs - 2); q < segs; ++q) at_wait(&S.q_full[q & 1], (q >> 1) & 1, &off, a.status);
    }
  } else if (warp == AD_MMA) {
    // ----------------------------------------------------------- products --
    // (the whole warp walks; one lane issues)
    const uint32_t by = elect_one(), tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t idesc = f16_idesc(N, BF16);
    const uint64_t k0 = sw128_desc(smem_u32(kring)), q0 = sw128_desc(smem_u32(qbuf)), p0 = sw128_desc(smem_u32(pbuf));
    // head_dim 64: rows 64..127 of the second product repeat other elements and are not used
    const uint64_t v0 = sw128_mn_desc(smem_u32(vring), DP == 128 ? AT_KEYS * 128 : 1024);
    Segments sk = s;
    int ik = 0;  // tile of the segment that scores are at
    bool ok = true;
    auto wait = [&](uint64_t *b, int par) { ok = __all_sync(0xffffffffu, at_wait(b, par & 1, &S.gave_up, a.status)) && ok; };
    int kslot = 0, kpar = 0, vslot = 0, vpar = 0;
    auto scores = [&](int f) {
      const int b = sk.index & 1;
      if (ik == 0) wait(&S.q_full[b], sk.index >> 1);
      wait(&S.full[0][kslot], kpar);
      if (!ok) return;
      tc_fence_after();
      const uint64_t kd = k0 + kslot * (C::TILE / 16), qd = q0 + b * (C::Q / 16);
      const uint32_t d = tm + (f % AD_AHEAD) * N;
#pragma unroll
      for (int x = 0; x < DP / 16; ++x)  // (addresses in a descriptor count 16 bytes)
        mma_f16_by(by, d, kd + (x / 4 * (AT_KEYS * 128) + x % 4 * 32) / 16, qd + (x / 4 * (N * 128) + x % 4 * 32) / 16, idesc, x > 0);
      mma_commit_by(by, &S.s_full[f % AD_AHEAD]);
      mma_commit_by(by, &S.empty[0][kslot]);
      if (++kslot == SLOTS) kslot = 0, kpar ^= 1;
      if (++ik == sk.count) {
        mma_commit_by(by, &S.q_empty[b]);
        sk.next(a);
        ik = 0;
      }
    };
    for (int f = 0; ok && f < AD_AHEAD && sk.count; ++f) scores(f);
    int iv = 0;
    for (int f = 0; ok && s.count; ++f) {
      wait(&S.p_full[f & 1], f >> 1);
      wait(&S.full[1][vslot], vpar);
      if (!ok) break;
      tc_fence_after();
      const uint64_t vd = v0 + vslot * (C::TILE / 16), pd = p0 + (f & 1) * (C::P / 16);
      const uint32_t d = tm + (AD_AHEAD + (f & 1)) * N;
#pragma unroll
      for (int x = 0; x < AT_KEYS / 16; ++x)
        mma_f16_by(by, d, vd + x * 2048 / 16, pd + (x / 4 * (N * 128) + x % 4 * 32) / 16, idesc | IDESC_A_MN, true);
      mma_commit_by(by, &S.o_full[f & 1]);
      mma_commit_by(by, &S.empty[1][vslot]);
      if (++vslot == SLOTS) vslot = 0, vpar ^= 1;
      if (sk.count) scores(f + AD_AHEAD);
      if (++iv == s.count) {
        s.next(a);
        iv = 0;
      }
    }
    mma_commit_by(by, &S.drain);
    int off = 0;
    at_wait(&S.drain, 0, &off, a.status);
    __syncwarp();
  } else {
    // ------------------------------------------------------------- softmax --
    // A wait that runs out ends the waiting, not the walk: every thread still
    // passes every barrier.
    const int grp = warp >> 2, key = tid & 127, wq = warp & 3;
    const uint32_t lanes = (uint32_t)(32 * wq) << 16;
    const uint32_t t_o = tmem + lanes + (AD_AHEAD + grp) * N;
    uint8_t *pm = pbuf + grp * C::P;
    const uint32_t p_off = (uint32_t)((key >> 6) * (N * 128) + (key & 7) * 2);
    const int p_chunk = (key & 63) >> 3;
    const float sc = a.scale_log2;
    int f = 0, mine = 0;  // tile of the stretch, tiles that this group has taken
    for (; s.count; s.next(a)) {
      const int nrows = s.n * a.g, pos0 = s.sp.pos0;
      float l[N];
#pragma unroll
      for (int c = 0; c < N; ++c) l[c] = 0.f;
      __syncwarp();
      {
        const float z[16] = {};
#pragma unroll
        for (int c = 0; c < N; c += 16) tmem_st16(t_o + c, z);
        tmem_st_wait();
      }
      if (key < N) S.ref[grp][key] = AT_NONE;
      warps_bar(1 + grp, 128);
      int done = 0;
      const int f_end = f + s.count;
      for (int i = 0; f < f_end; ++f, ++i) {
        if ((f & 1) != grp) continue;
        const int j = (s.tile + i) * AT_KEYS + key;
        // columns [lo, hi) see this key: those of tokens at j .. j + window - 1
        const int t_lo = max(0, j - pos0), t_hi = a.window ? min(s.n, j - pos0 + a.window) : s.n;
        const int lo = min(t_lo, 1 << 16) * a.g, hi = t_hi > t_lo ? t_hi * a.g : 0;
        const int j0 = (s.tile + i) * AT_KEYS;
        const bool edge = j0 + AT_KEYS - 1 > pos0 || (a.window && j0 < pos0 + s.n - a.window);
        const uint32_t t_s = tmem + lanes + (f % AD_AHEAD) * N;
        at_wait_warp(&S.s_full[f % AD_AHEAD], (f / AD_AHEAD) & 1, &S.gave_up, a.status);
        tc_fence_after();
        // the group's last products: their probabilities' room and the sums are free once they are complete
        bool settled = mine == 0;
        auto settle = [&]() {
          if (!settled) {
            at_wait_warp(&S.o_full[grp], (mine - 1) & 1, &S.gave_up, a.status);
            tc_fence_after();
          }
          settled = true;
        };
        // the scores less the running maxima, in powers of two: masked ones
        // are -infinity whatever the key holds
        float x[N];
        for (bool again = false;; again = true) {
          if (N == 16) tmem_ld16(t_s, x);
          else tmem_ld32(t_s, x);
#pragma unroll
          for (int c = 0; c < N; c += 4) {
            const float4 m = *reinterpret_cast<const float4 *>(&S.ref[grp][c]);
            const float2 u = fma2(make_float2(x[c], x[c + 1]), make_float2(sc, sc), make_float2(-m.x, -m.y));
            const float2 w = fma2(make_float2(x[c + 2], x[c + 3]), make_float2(sc, sc), make_float2(-m.z, -m.w));
            x[c] = u.x; x[c + 1] = u.y; x[c + 2] = w.x; x[c + 3] = w.y;
          }
          if (edge) {
#pragma unroll
            for (int c = 0; c < N; ++c) x[c] = c >= lo && c < hi ? x[c] : -INFINITY;
          }
          float top = -INFINITY;
#pragma unroll
          for (int c = 0; c < N; c += 2) top = fmaxf(top, fmaxf(x[c], x[c + 1]));
          if (again || (done && !bar_or(1 + grp, 128, top > AT_SLACK + AT_LIFT<BF16>))) break;  // (a segment's first tile sets them)
          // raise the maxima to the tile's, and bring the sums down to them
          settle();
          float v[N];
          if (N == 16) tmem_ld16(t_s, v);
          else tmem_ld32(t_s, v);
#pragma unroll
          for (int c = 0; c < N; ++c) v[c] = isnan(v[c]) || (edge && (c < lo || c >= hi)) ? -INFINITY : v[c] * sc;
          const float t = warp_columns<N, true>(v);
          if (lane < N) S.top[grp][wq][lane] = t;
          warps_bar(1 + grp, 128);
          if (key < N) {
            const float was = S.ref[grp][key];
            const float to = fmaxf(fmaxf(fmaxf(S.top[grp][0][key], S.top[grp][1][key]),
                                         fmaxf(S.top[grp][2][key], S.top[grp][3][key])) - AT_LIFT<BF16>, was);
            S.ref[grp][key] = to;
            S.factor[grp][key] = ex2(was - to);
          }
          warps_bar(1 + grp, 128);
          if (done) {
#pragma unroll
            for (int c = 0; c < N; ++c) l[c] *= S.factor[grp][c];
#pragma unroll 1
            for (int c0 = 0; c0 < N; c0 += 16) {
              float o[16];
              tmem_ld16(t_o + c0, o);
#pragma unroll
              for (int c = 0; c < 16; ++c) o[c] *= S.factor[grp][c0 + c];
              tmem_st16(t_o + c0, o);
            }
            tmem_st_wait();
          }
        }
#pragma unroll
        for (int c = 0; c < N; c += 2) {
          const float p0 = ex2(x[c]), p1 = ex2(x[c + 1]);
          const float2 t = add2(make_float2(l[c], l[c + 1]), make_float2(p0, p1));
          l[c] = t.x;
          l[c + 1] = t.y;
          x[c / 2] = __uint_as_float(pack16<BF16>(p0, p1));
        }
        settle();
#pragma unroll
        for (int c = 0; c < N; c += 2) {
          const uint32_t w = __float_as_uint(x[c / 2]);
          uint8_t *at = pm + p_off + c * 128;
          *reinterpret_cast<uint16_t *>(at + ((p_chunk ^ (c & 7)) << 4)) = (uint16_t)w;
          *reinterpret_cast<uint16_t *>(at + 128 + ((p_chunk ^ ((c + 1) & 7)) << 4)) = (uint16_t)(w >> 16);
        }
        if (edge) {
          // values that not every row sees: a probability of zero does not
          // take away an infinity or NaN, so rows that no token sees are
          // cleared, and what is not finite in others is added to the sums of
          // the rows that see it, and cleared
          at_wait_warp(&S.full[1][f % SLOTS], (f / SLOTS) & 1, &S.gave_up, a.status);
          uint8_t *vt = vring + f % SLOTS * C::TILE, *vr = vt + key * 128;
          bool odd = false;
          if (hi <= lo) {
#pragma unroll
            for (int x = 0; x < DP / 8; ++x)
              *reinterpret_cast<uint4 *>(vr + row_word(x, lane)) = make_uint4(0, 0, 0, 0);
          } else if (lo > 0 || hi < nrows) {
            odd = not_finite_row<BF16, DP / 8>(vr, lane);
          }
          if (s.n > 1 && bar_or(1 + grp, 128, odd)) {
            const uint32_t m = __ballot_sync(0xffffffffu, odd);
            if (lane == 0) S.odd[grp][wq] = m;
            warps_bar(1 + grp, 128);
            const int d = key & (DP - 1);
            for (int k = 0; k < AT_KEYS; ++k) {
              if (!(S.odd[grp][k >> 5] >> (k & 31) & 1u)) continue;
              const uint16_t x = *reinterpret_cast<const uint16_t *>(vt + d / 64 * (AT_KEYS * 128) + k * 128 +
                                                                     ((((d & 63) >> 3) ^ (k & 7)) << 4) + (d & 7) * 2);
              const float add = not_finite2<BF16>(x) ? (BF16 ? bf16_to_f32(x) : fp16_to_f32(x)) : 0.f;
              const int jk = j0 + k, k_lo = max(0, jk - pos0), k_hi = a.window ? min(s.n, jk - pos0 + a.window) : s.n;
              for (int c0 = 0; c0 < N; c0 += 16) {
                float o[16];
                tmem_ld16(t_o + c0, o);
#pragma unroll
                for (int c = 0; c < 16; ++c)
                  if (c0 + c >= k_lo * a.g && c0 + c < k_hi * a.g) o[c] += add;
                tmem_st16(t_o + c0, o);
              }
              tmem_st_wait();
            }
            warps_bar(1 + grp, 128);
            if (odd) {
              for (int x = 0; x < DP / 2; ++x) {
                uint32_t *w = reinterpret_cast<uint32_t *>(vr + x / 32 * (AT_KEYS * 128) + x % 32 * 4);
                if (not_finite2<BF16>(*w & 0xFFFFu)) *w &= 0xFFFF0000u;
                if (not_finite2<BF16>(*w & 0xFFFF0000u)) *w &= 0xFFFFu;
              }
            }
          }
        }
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.p_full[grp]);
        __syncwarp();
        ++mine;
        ++done;
      }
      // ---- the segment's end: each group finishes half of the rows ----
      {
        const float t = warp_columns<N, false>(l);
        if (lane < N) S.sum[grp][wq][lane] = t;
      }
      if (done) {
        at_wait_warp(&S.o_full[grp], (mine - 1) & 1, &S.gave_up, a.status);
        tc_fence_after();
      }
      // both groups' products are done before the probabilities' room is
      // taken for the exchange: [rows][DP] sums
      warps_bar(3, 256);
      float *ex = reinterpret_cast<float *>(pbuf);
      constexpr int HALF = N / 2;
      const bool whole = s.has_start() && s.has_end();
      const int64_t piece = 2 * (int64_t)blockIdx.x + (s.index > 0);
      if (key < HALF && grp * HALF + key < nrows) {  // a thread a row: its weights and place
        const int row = grp * HALF + key;
        const float m0 = S.ref[0][row], m1 = S.ref[1][row], m = fmaxf(m0, m1), w0 = ex2(m0 - m), w1 = ex2(m1 - m);
        const float s0 = (S.sum[0][0][row] + S.sum[0][1][row]) + (S.sum[0][2][row] + S.sum[0][3][row]);
        const float s1 = (S.sum[1][0][row] + S.sum[1][1][row]) + (S.sum[1][2][row] + S.sum[1][3][row]);
        const float total = s0 * w0 + s1 * w1, inv = !whole ? 1.f : total == 0.f ? 0.f : 1.f / total;
        S.weight[row] = make_float2((grp ? w1 : w0) * inv, (grp ? w0 : w1) * inv);
        if (whole) {
          const int tok = row / a.g;
          const int64_t t = s.sp.t0 + tok;
          const int h = s.h * a.g + row - tok * a.g;
          S.place[row] = t * a.os + (int64_t)h * a.D;
          if (a.lse) a.lse[t * a.H + h] = total == 0.f ? -INFINITY : (m + log2f(total)) * AT_LN2;
        } else {
          S.place[row] = (piece * N + row) * DP;
          pieces.stats[piece * N + row] = make_float2(m, total);
        }
      }
      __syncwarp();
      float o[HALF];
#pragma unroll
      for (int c = 0; c < HALF; c += 8) tmem_ld8(t_o + (1 - grp) * HALF + c, o + c);
      if (key < DP) {
#pragma unroll
        for (int c = 0; c < HALF; ++c) ex[((1 - grp) * HALF + c) * DP + key] = o[c];
      }
      __syncwarp();
#pragma unroll
      for (int c = 0; c < HALF; c += 8) tmem_ld8(t_o + grp * HALF + c, o + c);
      tc_fence_before();
      warps_bar(3, 256);
      if (key < (whole ? a.D : DP)) {
#pragma unroll
        for (int c = 0; c < HALF; ++c) {
          const int row = grp * HALF + c;
          if (row < nrows) {
            const float2 w = S.weight[row];
            // (a sum of zero keys times a weight of zero: sums are zeros then, not garbage)
            const float v = o[c] * w.x + ex[row * DP + key] * w.y;
            if (whole) a.out[S.place[row] + key] = (uint16_t)pack16<BF16>(v, 0.f);
            else pieces.sums[S.place[row] + key] = v;
          }
        }
      }
      if (!whole && tid == 0)
        pieces.what[piece] = make_int4(s.sp.t0, s.n, s.h, PIECE_USED | (s.has_start() ? PIECE_START : 0) | (s.has_end() ? PIECE_END : 0));
      warps_bar(3, 256);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == AD_MMA) {
    tc_fence_after();
    tmem_free<C::TMEM>(tmem);
  }
}

template <int N, int DP, bool BF16>
cudaError_t launch(const AttnArgs &a, void *ws, cudaStream_t s) {
  using C = AdCfg<N, DP>;
  constexpr size_t smem = 1024 + 2 * C::SLOTS * C::TILE + 2 * (C::Q + C::P) + sizeof(AdShared<N, C::SLOTS>);
  static_assert(smem <= 227 * 1024, "shared memory of a block");
  static OncePerDevice once;
  cudaError_t e = once_per_device(once, []() {
    return cudaFuncSetAttribute(attention_decode_kernel<N, DP, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  });
  if (e != cudaSuccess) return e;
  const int blocks = device_sms(), rows = piece_rows(a.page);
  CUtensorMap tq;
  KvMaps tk, tv;
  if (!make_q_map(&tq, a, N / a.g, BF16) || !make_kv_maps(&tk, a.k, a, rows, BF16) || !make_kv_maps(&tv, a.v, a, rows, BF16))
    return cudaErrorInvalidValue;
  const Pieces p = pieces_of(ws, blocks, N, DP);
  attention_decode_kernel<N, DP, BF16><<<blocks, AD_THREADS, smem, s>>>(a, p, tq, tk, tv, rows);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_join<DP, BF16>(a, p, blocks, N, 1 << 20, s);
}

template <int N>
cudaError_t launch_n(const AttnArgs &a, bool bf16, void *ws, cudaStream_t s) {
  if (a.D <= 64) return bf16 ? launch<N, 64, true>(a, ws, s) : launch<N, 64, false>(a, ws, s);
  return bf16 ? launch<N, 128, true>(a, ws, s) : launch<N, 128, false>(a, ws, s);
}

int columns(int64_t rows) { return rows <= 16 ? 16 : 32; }

}  // namespace

size_t attention_decode_workspace(int64_t rows, int blocks) { return pieces_bytes(blocks, columns(rows), 128); }

cudaError_t launch_attention_decode(const AttnArgs &a, bool bf16, void *ws, cudaStream_t s) {
  const int n = columns((int64_t)a.max_new * a.g);
  return n == 16 ? launch_n<16>(a, bf16, ws, s) : launch_n<32>(a, bf16, ws, s);
}

}  // namespace dsm
