// Attention of many query rows a key head (a prompt's chunk, or chunks and
// single tokens in one batch): bound by the matrix products and the
// exponentials.
//
// A block takes 256 query rows at a time, as two tiles of 128 (whole tokens
// with the g query heads that share a key head: row i of a tile is head
// i mod g of token i / g), over tiles of 128 keys, which both query tiles use
// once they are in shared memory.  Scores S = Q K^T and sums O += P V are in
// tensor memory; the probabilities overwrite the scores there and are the
// second product's first operand, so they never pass through shared memory.
//
//   two groups of four warps   a thread a query row: maximum, exponentials,
//                   sum of its own row, no exchange between threads; while
//                   one group works on its scores, the products of the other
//                   run.  The groups take turns: turn j is group j mod 2's.
//                   Where there are two query tiles, a key tile is two turns,
//                   one a query tile; where there is one (the request's
//                   tokens fit it), a key tile is one turn, and the groups'
//                   sums are joined at the segment's end;
//   MMA thread      per turn: O += P V, then the S that takes P's place (that
//                   of two turns on; for head_dim <= 64, whose sums leave room
//                   for a third tile of scores, of three turns on: a group's
//                   next scores are then there when it has done the last);
//   two producer warps         keys (and the query rows), values;
//   gate warp       in tiles that not every row sees it clears the values that
//                   none sees and looks for infinities and NaN in the others;
//                   and it waits for a turn's values in the MMA thread's
//                   place and tells it what the turn is (a word of flags), as
//                   one more arrival beside the probabilities': the products
//                   stand still while the thread that issues them does
//                   anything else, and a warp that runs alone takes hundreds
//                   of cycles for a little bookkeeping.
//
// Maxima are raised lazily (AT_SLACK), by warp.  Probabilities are rounded to
// the 16-bit type of the values, which the second product takes; their sums,
// the maxima and the accumulators are 32 bits.
//
// Measured: 2048 tokens x 32 heads (8 key heads) of 128 over 30,011 keys 690 us,
// 1.50 PFLOP/s, at the power limit of the board; over 8000 keys 228 us, 58 % of
// the tensor cores' cycles.  head_dim 64 over 8000 keys 185 us (201 with two
// tiles of scores): a turn is 1300 cycles there, of which 512 are products and
// 512 exponentials; what is left is the way of a turn through the warps.  17
// requests of 3 to 666 tokens, a window of 1024, 76 us; 29 requests of 1 to 6
// tokens, 7 query heads a key head, over 34 to 4993 keys 32 us.
#include "attention_tc.cuh"

namespace dsm {
namespace {

constexpr int AC_THREADS = 384;
constexpr int AC_MMA = 8, AC_KEYS = 9, AC_VALUES = 10, AC_GATE = 11;
constexpr int AC_READERS = 10;  // warps that read all segments: softmax, values, gate
constexpr int AC_ROWS = 256;
// Turns that an item costs besides its own: its sums' way out, and the wait
// for its first scores (17 requests of 3 to 666 tokens: 78 us with 3, 76 with
// 4, 75 with 6; 29 requests of 1 to 6: 31, 32, 33).
constexpr int AC_ITEM = 4;
constexpr int AC_HEAD = 3 * 1024;  // bytes of a block's barriers and small arrays

template <int DP>
struct AcCfg {
  static constexpr uint32_t TILE = AT_KEYS * DP * 2;  // keys, values, or a query tile
  static constexpr int KS = DP == 128 ? 2 : 4, VS = DP == 128 ? 3 : 4;
  static constexpr int QS = DP == 128 ? 1 : 2;  // segments' query rows
  static constexpr int NB = DP == 128 ? 2 : 3;  // tiles of scores: what the sums leave of tensor memory
  // Scores that a thread takes at a time.  The wider loop is the faster one in
  // steady state, and its masks are then better out of its way; but a smaller
  // one costs less where the code changes often, at tiles with masks and the
  // ends of segments, which is most of the work of a batch of short chunks
  // (2048 tokens over 30,011 keys, head_dim 128: 677 us with 64, 718 with 32;
  // 17 requests of 3 to 666 tokens, head_dim 64: 94 us with 64, 79 with 32, and 105 and 99 with head_dim 128).
  static constexpr int WIDE = DP == 128 ? 64 : 32;
  static constexpr int SUMS = NB * 128;         // column of the first group's sums
};

// What a turn is, for the MMA thread: its value slot, and of the scores that
// follow (if any) the key slot and query tile, what to wait for, and what to
// let go of behind them.
enum : uint32_t {
  TURN_SCORES = 1u << 0,   // the group has another turn
  TURN_WAIT_K = 1u << 1,   // its keys are new
  TURN_WAIT_Q = 1u << 2,   // its query rows are new
  TURN_K_PAR = 1u << 3,
  TURN_Q_PAR = 1u << 4,
  TURN_Q_TILE = 1u << 5,
  TURN_FREE_K = 1u << 6,
  TURN_FREE_Q = 1u << 7,
  TURN_FREE_V = 1u << 8,
  TURN_SUMS = 1u << 9,     // the group's last of the segment
  TURN_LAST = 1u << 10,    // the stretch's last
  TURN_Q_SLOT = 1u << 11,
  TURN_K_SLOT = 1u << 12,  // times the slot
  TURN_V_SLOT = 1u << 16
};

template <int KS, int VS, int QS>
struct AcShared {
  uint64_t k_full[KS], k_empty[KS], v_full[VS], v_empty[VS];
  uint64_t v_seen[VS];               // looked at
  uint64_t added[2];                 // by group: values that are not finite are in its sums
  uint64_t q_full[QS], q_empty[QS], s_full[4], p_full[4], o_full[4], drain;  // (of turn j at j mod 4)
  uint32_t odd[VS][4];  // keys whose values are not all finite
  float2 stats[2][128]; // maximum and sum of a row, by group
  SegRing segs;
  uint32_t turns[8];    // turn j's word at j mod 8
  int64_t part[AC_THREADS / 32];
  Start start;
  uint32_t tmem;
  int gave_up;
};

// The walk over turns that the scores take, NB turns ahead of the sums.
struct Ahead {
  int k, count, i, f;  // segment, its tiles, tile of it, tile of the stretch
  bool two, half;      // two turns a tile; the first of them is done
  __device__ __forceinline__ void segment(SegRing &ring, int index, int tok, unsigned *status) {
    const Seg &g = ring.get(index, status);
    k = index;
    count = g.count;
    two = g.n > tok;
    i = 0;
  }
  // The scores of the turn: their part of a word.
  template <int KS, int QS>
  __device__ __forceinline__ uint32_t word(int w) const {
    if (!count) return 0;
    const bool last = two ? half : true;  // of the tile
    return TURN_SCORES | (half ? 0u : TURN_WAIT_K | (f / KS & 1 ? TURN_K_PAR : 0u)) |
           (!half && i == 0 ? TURN_WAIT_Q | (k / QS & 1 ? TURN_Q_PAR : 0u) : 0u) | (k % QS ? TURN_Q_SLOT : 0u) | (two && w ? TURN_Q_TILE : 0u) |
           (last ? TURN_FREE_K : 0u) | (last && i + 1 == count ? TURN_FREE_Q : 0u) | (uint32_t)(f % KS) * TURN_K_SLOT;
  }
  // To the next turn.
  __device__ __forceinline__ void step(SegRing &ring, int tok, unsigned *status) {
    if (!count) return;
    half = two && !half;
    if (half) return;
    ++f;
    if (++i == count) segment(ring, k + 1, tok, status);
  }
};

__device__ __forceinline__ void load_scores(uint32_t t, float (&v)[32]) { tmem_ld32(t, v); }
__device__ __forceinline__ void load_scores(uint32_t t, float (&v)[64]) { tmem_ld64(t, v); }

// Replaces a row's scores outside of columns [lo, hi) by -infinity.
__device__ __noinline__ void mask_scores(uint32_t t_s, int lo, int hi) {
#pragma unroll 1
  for (int c0 = 0; c0 < AT_KEYS; c0 += 32) {
    const uint32_t see = bits(lo - c0, hi - c0);
    if (__all_sync(0xffffffffu, see == 0xffffffffu)) continue;
    float x[32];
    tmem_ld32(t_s + c0, x);
#pragma unroll
    for (int c = 0; c < 32; ++c) x[c] = see >> c & 1u ? x[c] : -INFINITY;
    tmem_st32(t_s + c0, x);
  }
  tmem_st_wait();
}

template <int DP>
__device__ __noinline__ void scale_sums(uint32_t t_o, float by) {
#pragma unroll 1
  for (int c = 0; c < DP; c += 16) {
    float o[16];
    tmem_ld16(t_o + c, o);
#pragma unroll
    for (int k = 0; k < 16; ++k) o[k] *= by;
    tmem_st16(t_o + c, o);
  }
  tmem_st_wait();  // (add_odd may load them next)
}

// Adds to a row's sums the values of a tile that are not finite and that the
// row sees: columns [lo, hi).  (Rare: kept out of the loop's code.)
template <int DP, bool BF16>
__device__ __noinline__ void add_odd(const uint8_t *vt, const uint32_t *odd, int lo, int hi, uint32_t t_o) {
  for (int k = 0; k < AT_KEYS; ++k) {
    if (!(odd[k >> 5] >> (k & 31) & 1u)) continue;
    const bool sees = k >= lo && k < hi;
#pragma unroll 1
    for (int c = 0; c < DP; c += 16) {
      float o[16];
      tmem_ld16(t_o + c, o);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int d = c + e;
        const uint16_t v = *reinterpret_cast<const uint16_t *>(vt + d / 64 * (AT_KEYS * 128) + k * 128 +
                                                               ((((d & 63) >> 3) ^ (k & 7)) << 4) + (d & 7) * 2);
        if (sees && not_finite2<BF16>(v)) o[e] += BF16 ? bf16_to_f32(v) : fp16_to_f32(v);
      }
      tmem_st16(t_o + c, o);
    }
    tmem_st_wait();  // the next key's loads are of the same columns
  }
}

// (once a block: kept out of the code that the loops share a cache with)
__device__ __noinline__ void chunk_start(const AttnArgs &a, const RawSpan raw0, const Plan plan, Start *out, int64_t *part) {
  find_start<AC_THREADS>(a, raw0, plan, out, part);
}

template <int DP, bool BF16>
__global__ void __launch_bounds__(AC_THREADS, 1)
    attention_chunk_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ Pieces pieces, const __grid_constant__ CUtensorMap tm_q,
                           const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, int rows,
                           int tok, bool wide_out) {
  using C = AcCfg<DP>;
  constexpr int KS = C::KS, VS = C::VS, QS = C::QS;
  extern __shared__ __align__(1024) uint8_t smem_tiles[];  // (the period of the 128-byte swizzle)
  typedef AcShared<KS, VS, QS> Sh;
  Sh &S = *reinterpret_cast<Sh *>(smem_tiles);
  uint8_t *qbuf = smem_tiles + AC_HEAD, *kring = qbuf + 2 * QS * C::TILE, *vring = kring + KS * C::TILE;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Plan plan = {2 * tok, tok, AC_ITEM};
  asm volatile("griddepcontrol.launch_dependents;");
  const RawSpan raw0 = first_request<AC_THREADS>(a);  // (under way while the block is set up)

  if (tid < KS) {
    mbar_init(&S.k_full[tid], 1);
    mbar_init(&S.k_empty[tid], 1);
    fence_mbar_init();
  } else if (tid >= 32 && tid < 32 + VS) {
    mbar_init(&S.v_full[tid - 32], 1);
    mbar_init(&S.v_empty[tid - 32], 1);
    mbar_init(&S.v_seen[tid - 32], 1);
    fence_mbar_init();
  } else if (tid >= 64 && tid < 66) {
    mbar_init(&S.added[tid - 64], 4);
    for (int i = tid - 64; i < 4; i += 2) {
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.p_full[i], 5);
      mbar_init(&S.o_full[i], 1);
    }
    fence_mbar_init();
  } else if (tid >= 96 && tid < 96 + AT_SEGS) {
    S.segs.init(tid - 96, AC_READERS);
    fence_mbar_init();
  } else if (tid == 128) {
    for (int i = 0; i < QS; ++i) {
      mbar_init(&S.q_full[i], 1);
      mbar_init(&S.q_empty[i], 1);
    }
    mbar_init(&S.drain, 1);
    S.gave_up = 0;
    fence_mbar_init();
  } else if (tid == 160) {
    const CUtensorMap *maps[3] = {&tm_q, &tm_k, &tm_v};
    for (int i = 0; i < 3; ++i) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(maps[i])) : "memory");
  }
  if (tid == 0) {
    pieces.what[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
    pieces.what[2 * blockIdx.x + 1] = make_int4(0, 0, 0, 0);
  }
  __syncwarp();
  if (warp == AC_MMA) tmem_alloc<512>(&S.tmem);
  // query rows that no copy fills stay zero
  for (int i = tid; i < (int)(2 * QS * C::TILE / 16); i += AC_THREADS) reinterpret_cast<uint4 *>(qbuf)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async();
  chunk_start(a, raw0, plan, &S.start, S.part);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem;  // scores of turn j at (j mod NB) 128, sums of group i at SUMS + i DP
  // whether some of n rows' tokens, the first at position p, does not see some key of a tile
  auto edge_of = [&](int p, int n, int j0) { return j0 + AT_KEYS - 1 > p || (a.window && j0 < p + n - a.window); };

  if (warp == AC_KEYS) {
    // -------------------------------- segments, query rows and keys ------
    Segments s;
    s.init(a, plan, S.start);
    bool ok = true, bad = false;
    int segs = 0, asked = 0, f = 0, i = 0;  // segments, those whose query rows are under way, tiles
    TileRuns now, later;
    if (s.count) now.find(a, s, s.tile, rows);
    for (; s.count; ++f) {
      const int head = s.h;
      if (i == 0) {
        S.segs.put(segs, s, ok, &S.gave_up, a.status);
        const int q = segs % QS;
        if (lane == 0 && segs >= QS && !at_wait(&S.q_empty[q], (segs / QS & 1) ^ 1, &S.gave_up, a.status)) ok = false;
        ++segs;
        if (!__shfl_sync(0xffffffffu, ok, 0)) break;
        ++asked;
        if (lane == 0) {
          const int tiles = s.n > tok ? 2 : 1;
          mbar_arrive_expect_tx(&S.q_full[q], tiles * tok * a.g * DP * 2);
          for (int w = 0; w < tiles; ++w)
#pragma unroll
            for (int x = 0; x < DP; x += 64)
              tma_load_3d(qbuf + (2 * q + w) * C::TILE + x / 64 * (128 * 128), &tm_q, x, s.h * a.g, s.sp.t0 + s.first + w * tok, &S.q_full[q]);
        }
        __syncwarp();
      }
      if (++i == s.count) {
        s.next(a);
        i = 0;
      }
      if (s.count) later.find(a, s, s.tile + i, rows);
      const int sl = f % KS;
      if (lane == 0 && f >= KS && !at_wait(&S.k_empty[sl], (f / KS & 1) ^ 1, &S.gave_up, a.status)) ok = false;
      if (!__shfl_sync(0xffffffffu, ok, 0)) break;
      now.copy<DP, false>(a, kring + sl * C::TILE, &tm_k, nullptr, head, rows, &S.k_full[sl], bad);
      now = later;
    }
    S.segs.put(segs, s, false, &S.gave_up, a.status);
    if (bad) flag(a.status, ST_PAGING);
    if (lane == 0) {  // every copy of this warp has landed before the block ends
      int off = 0;
      for (int g = max(0, f - KS); g < f; ++g) at_wait(&S.k_full[g % KS], g / KS & 1, &off, a.status);
      for (int g = max(0, asked - QS); g < asked; ++g) at_wait(&S.q_full[g % QS], g / QS & 1, &off, a.status);
    }
  } else if (warp == AC_VALUES) {
    // ------------------------------------------------------------ values --
    bool ok = true, bad = false;
    int k = 0, f = 0, i = 0;
    TileRuns now, later;
    Seg s = S.segs.get(0, a.status);
    if (s.count) now.find(a, s.r, s.pos0 + s.first, s.n, s.tile, rows);
    for (; s.count; ++f) {
      const int head = s.h;
      if (++i == s.count) {
        S.segs.done(k);
        s = S.segs.get(++k, a.status);
        i = 0;
      }
      if (s.count) later.find(a, s.r, s.pos0 + s.first, s.n, s.tile + i, rows);
      const int sl = f % VS;
      if (lane == 0 && f >= VS && !at_wait(&S.v_empty[sl], (f / VS & 1) ^ 1, &S.gave_up, a.status)) ok = false;
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (ok) now.copy<DP, false>(a, vring + sl * C::TILE, &tm_v, nullptr, head, rows, &S.v_full[sl], bad);
      else break;
      now = later;
    }
    for (; s.count; s = S.segs.get(++k, a.status)) S.segs.done(k);  // (gave up: the others' segments go on to their end)
    if (bad) flag(a.status, ST_PAGING);
    if (lane == 0) {
      int off = 0;
      for (int g = max(0, f - VS); g < f; ++g) at_wait(&S.v_full[g % VS], g / VS & 1, &off, a.status);
    }
  } else if (warp == AC_GATE) {
    // --------------------------------------------------------------- gate --
    int f = 0, turn = 0, adds[2] = {0, 0};
    Ahead z{};
    z.segment(S.segs, 0, tok, a.status);
    for (int j = 0; j < C::NB; ++j) z.step(S.segs, tok, a.status);
    for (int k = 0;; ++k) {
      const Seg s = S.segs.get(k, a.status);
      if (!s.count) break;
      const bool two = s.n > tok;
      const int p = s.pos0 + s.first;
      const int see_lo = a.window ? p + 1 - a.window : 0, see_hi = p + s.n;           // some row sees it
      const int all_lo = a.window ? p + s.n - a.window : 0, all_hi = p + 1;           // every row sees it
      for (int i = 0; i < s.count; ++i, ++f, turn += two ? 2 : 1) {
        const int sl = f % VS, par = (f / VS) & 1, j0 = (s.tile + i) * AT_KEYS;
        at_wait(&S.v_full[sl], par, &S.gave_up, a.status);
        if (edge_of(p, s.n, j0)) {
          uint8_t *vt = vring + sl * C::TILE;
          uint32_t any = 0, m[4];
          for (int k = 0; k < 4; ++k) {
            const int j = j0 + 32 * k + lane;
            uint8_t *vr = vt + (32 * k + lane) * 128;
            bool odd = false;
            if (j >= see_hi || j < see_lo) {
#pragma unroll
              for (int x = 0; x < DP / 8; ++x)
                *reinterpret_cast<uint4 *>(vr + row_word(x, lane)) = make_uint4(0, 0, 0, 0);
            } else if (j >= all_hi || j < all_lo) {
              odd = not_finite_row<BF16, DP / 8>(vr, lane);
            }
            m[k] = __ballot_sync(0xffffffffu, odd);
            any |= m[k];
          }
          if (lane == 0)
            for (int k = 0; k < 4; ++k) S.odd[sl][k] = m[k];
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.v_seen[sl]);
          if (any) {  // once they are added to the rows that see them, they are cleared
            for (int w = 0; w < 2; ++w)
              if (two || w == (turn & 1)) at_wait(&S.added[w], adds[w]++ & 1, &S.gave_up, a.status);
            for (int k = 0; k < 4; ++k) {
              if (!(m[k] >> lane & 1u)) continue;
              uint8_t *vr = vt + (32 * k + lane) * 128;
              for (int x = 0; x < DP / 2; ++x) {
                uint32_t *w = reinterpret_cast<uint32_t *>(vr + x / 32 * (AT_KEYS * 128) + x % 32 * 4);
                if (not_finite2<BF16>(*w & 0xFFFFu)) *w &= 0xFFFF0000u;
                if (not_finite2<BF16>(*w & 0xFFFF0000u)) *w &= 0xFFFFu;
              }
            }
            fence_proxy_async();
            __syncwarp();
          }
        } else if (lane == 0) {
          mbar_arrive(&S.v_seen[sl]);  // (its phases go with the tiles)
        }
        for (int t = 0; t < (two ? 2 : 1); ++t) {
          const int j = turn + t;
          const bool tile_end = !two || t, sums = i + (two ? 1 : 2) >= s.count;
          uint32_t word = z.word<KS, QS>((j + C::NB) & 1) | (uint32_t)sl * TURN_V_SLOT | (tile_end ? TURN_FREE_V : 0u) | (sums ? TURN_SUMS : 0u);
          z.step(S.segs, tok, a.status);
          // (the stretch's last turn has no other behind it: none after the
          // next, and the segment after this one is its end)
          if (tile_end && i + 1 == s.count && !S.segs.get(k + 1, a.status).count) word |= TURN_LAST;
          if (j >= 4) at_wait(&S.p_full[j & 3], ((j >> 2) - 1) & 1, &S.gave_up, a.status);  // the arrival is for this turn
          if (lane == 0) {
            S.turns[j & 7] = word;
            mbar_arrive(&S.p_full[j & 3]);
          }
        }
      }
      S.segs.done(k);
    }
  } else if (warp == AC_MMA) {
    // ----------------------------------------------------------- products --
    // (the whole warp walks; one lane issues)
    const uint32_t by = elect_one();
    const uint32_t id_s = f16_idesc(AT_KEYS, BF16), id_o = f16_idesc(DP, BF16) | IDESC_B_MN;
    const uint64_t q0 = sw128_desc(smem_u32(qbuf)), k0 = sw128_desc(smem_u32(kring));
    const uint64_t v0 = sw128_mn_desc(smem_u32(vring), AT_KEYS * 128);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    bool ok = true;
    auto wait = [&](uint64_t *b, uint32_t par) { ok = __all_sync(0xffffffffu, at_wait(b, par, &S.gave_up, a.status)) && ok; };
    auto scores = [&](int b, int j, uint32_t word) {  // of turn j, to tile b
      const int q = word & TURN_Q_SLOT ? 1 : 0;
      if (word & TURN_WAIT_Q) wait(&S.q_full[q], word & TURN_Q_PAR ? 1 : 0);
      const int slot = word / TURN_K_SLOT & 15;
      if (word & TURN_WAIT_K) wait(&S.k_full[slot], word & TURN_K_PAR ? 1 : 0);
      if (!ok) return;
      tc_fence_after();
      const uint64_t qd = q0 + 2 * q * (C::TILE / 16) + (word & TURN_Q_TILE ? C::TILE / 16 : 0), kd = k0 + slot * (C::TILE / 16);
#pragma unroll
      for (int x = 0; x < DP / 16; ++x) {  // (addresses in a descriptor count 16 bytes)
        const uint32_t at = (x / 4 * (AT_KEYS * 128) + x % 4 * 32) / 16;
        mma_f16_by(by, tm + b * 128, qd + at, kd + at, id_s, x > 0);
      }
      mma_commit_by(by, &S.s_full[j & 3]);
      if (word & TURN_FREE_K) mma_commit_by(by, &S.k_empty[slot]);
      if (word & TURN_FREE_Q) mma_commit_by(by, &S.q_empty[q]);
    };
    // the first turns' scores, which no turn precedes (their
    // segments are not let go of before these scores are used)
    Ahead z{};
    z.segment(S.segs, 0, tok, a.status);
    const bool some = z.count > 0;
    for (int j = 0; ok && j < C::NB && z.count; ++j) {
      scores(j, j, __shfl_sync(0xffffffffu, z.word<KS, QS>(j & 1), 0));
      if (j + 1 < C::NB) z.step(S.segs, tok, a.status);
    }
    for (int j = 0, b = 0; ok && some; ++j, b = b + 1 == C::NB ? 0 : b + 1) {
      const int w = j & 1;
      wait(&S.p_full[j & 3], j >> 2 & 1);
      if (!ok) break;
      const uint32_t word = __shfl_sync(0xffffffffu, S.turns[j & 7], 0);
      tc_fence_after();
      const int slot = word / TURN_V_SLOT & 15;
      const uint64_t vd = v0 + slot * (C::TILE / 16);
#pragma unroll
      for (int x = 0; x < AT_KEYS / 16; ++x)
        mma_f16_ts_by(by, tm + C::SUMS + w * DP, tm + b * 128 + x * 8, vd + x * 2048 / 16, id_o, true);
      if (C::NB > 2) mma_commit_by(by, &S.o_full[j & 3]);
      else if (word & TURN_SUMS) mma_commit_by(by, &S.o_full[w]);
      if (word & TURN_SCORES) scores(b, j + C::NB, word);
      if (word & TURN_FREE_V) mma_commit_by(by, &S.v_empty[slot]);
      if (word & TURN_LAST) break;
    }
    mma_commit_by(by, &S.drain);
    int off = 0;
    at_wait(&S.drain, 0, &off, a.status);
    __syncwarp();
  } else {
    // ------------------------------------------------------------- softmax --
    const int grp = warp >> 2, row = tid & 127;
    constexpr int W = C::WIDE;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t t_o = tmem + lanes + C::SUMS + grp * DP;
    const float sc = a.scale_log2;
    const int my_tok = row / a.g, my_head = row - my_tok * a.g;
    // tile and turn of the stretch; turns of this group (the i-th is turn
    // 2 i + group), and its segments; where the next turn's scores are
    int f = 0, turn = 0, mine = 0, ends = 0, b = grp;
    for (int ks = 0;; ++ks) {
      const Seg &s = S.segs.get(ks, a.status);
      __syncwarp();
      const int count = s.count;
      if (!count) break;
      const bool two = s.n > tok;
      const int skip = two ? grp * tok : 0, n = min(tok, s.n - skip);  // the query tile's tokens
      const int p0 = s.pos0 + s.first, n0 = s.n;                      // the segment's
      const int pos = p0 + skip + my_tok;                             // this row's
      const bool is_row = my_tok < n;
      int j0 = s.tile * AT_KEYS;
      {
        const float z[32] = {};
#pragma unroll
        for (int c = 0; c < DP; c += 32) tmem_st32(t_o + c, z);
        tmem_st_wait();
      }
      float m = AT_NONE, l = 0.f;
      int done = 0;
      for (int i = 0; i < count; ++i, j0 += AT_KEYS, ++f) {
        turn += two ? 2 : 1;
        if (!two && ((turn - 1) & 1) != grp) continue;
        at_wait_warp(&S.s_full[(2 * mine + grp) & 3], mine >> 1 & 1, &S.gave_up, a.status);
        // (the products of the turn before the last, in order, so that the
        // parity tells which)
        if (C::NB > 2 && mine >= 2) at_wait_warp(&S.o_full[(2 * mine + grp) & 3], (mine >> 1) - 1 & 1, &S.gave_up, a.status);
        tc_fence_after();
        // before this thread changes the sums itself, the group's products are complete
        auto settle = [&]() {
          if (C::NB > 2 && done) at_wait_warp(&S.o_full[(2 * mine + grp + 2) & 3], (mine - 1) >> 1 & 1, &S.gave_up, a.status);
          tc_fence_after();
        };
        const uint32_t t_s = tmem + lanes + b * 128;
        // columns [lo, hi) of the tile are seen; the others' scores are
        // replaced in tensor memory too
        const int hi = is_row ? pos + 1 - j0 : 0, lo = a.window ? pos + 1 - a.window - j0 : 0;
        const bool edge = edge_of(p0 + skip, n, j0);
        if (edge && W == 64) mask_scores(t_s, lo, hi);
        float t0 = -INFINITY, t1 = t0, t2 = t0, t3 = t0;
#pragma unroll 1
        for (int c0 = 0; c0 < AT_KEYS; c0 += W) {
          float x[W];
          load_scores(t_s + c0, x);
          if (edge && W == 32) {
            const uint32_t see = bits(lo - c0, hi - c0);
#pragma unroll
            for (int c = 0; c < W; ++c) x[c] = see >> (c & 31) & 1u ? x[c] : -INFINITY;
            tmem_st32(t_s + c0, x);
          }
#pragma unroll
          for (int c = 0; c < W; c += 8) {
            t0 = fmaxf(t0, fmaxf(x[c], x[c + 1]));
            t1 = fmaxf(t1, fmaxf(x[c + 2], x[c + 3]));
            t2 = fmaxf(t2, fmaxf(x[c + 4], x[c + 5]));
            t3 = fmaxf(t3, fmaxf(x[c + 6], x[c + 7]));
          }
        }
        if (edge && W == 32) tmem_st_wait();
        const float top = fmaxf(fmaxf(t0, t1), fmaxf(t2, t3)) * sc;
        if (__any_sync(0xffffffffu, top > m + (AT_SLACK + AT_LIFT<BF16>))) {
          // raise the maximum, and bring the sums down to it
          const float to = fmaxf(m, top - AT_LIFT<BF16>), keep = ex2(m - to);
          l *= keep;
          m = to;
          settle();
          if (done) scale_sums<DP>(t_o, keep);
        }
        const float2 sc2 = make_float2(sc, sc), m2 = make_float2(-m, -m);
        float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
#pragma unroll 1
        for (int c0 = 0; c0 < AT_KEYS; c0 += W) {
          float x[W];
          load_scores(t_s + c0, x);
#pragma unroll
          for (int c = 0; c < W; c += 4) {
            const float2 u = fma2(make_float2(x[c], x[c + 1]), sc2, m2), w = fma2(make_float2(x[c + 2], x[c + 3]), sc2, m2);
            const float2 p = make_float2(ex2(u.x), ex2(u.y)), q = make_float2(ex2(w.x), ex2(w.y));
            sum0 = add2(sum0, p);
            sum1 = add2(sum1, q);
            x[c / 2] = __uint_as_float(pack16<BF16>(p.x, p.y));
            x[c / 2 + 1] = __uint_as_float(pack16<BF16>(q.x, q.y));
          }
          if (W == 64) tmem_st32(t_s + c0 / 2, x);
          else tmem_st16(t_s + c0 / 2, x);
        }
        l += (sum0.x + sum0.y) + (sum1.x + sum1.y);
        if (edge_of(p0, n0, j0)) {
          // values that are not finite, and that not every row sees: a
          // probability of zero does not take them away, so the rows that see
          // them have them added here, and the products get zeros
          const int sl = f % VS;
          at_wait_warp(&S.v_seen[sl], f / VS & 1, &S.gave_up, a.status);
          if (S.odd[sl][0] | S.odd[sl][1] | S.odd[sl][2] | S.odd[sl][3]) {
            settle();
            add_odd<DP, BF16>(vring + sl * C::TILE, S.odd[sl], lo, hi, t_o);
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.added[grp]);
          }
          __syncwarp();
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.p_full[(2 * mine + grp) & 3]);
        __syncwarp();
        b = C::NB == 2 ? b : b ? b - 1 : 2;  // (two turns on, of three)
        ++mine;
        ++done;
      }
      // ---- the segment's end ----
      if (done) {
        if (C::NB > 2) at_wait_warp(&S.o_full[(2 * mine + grp + 2) & 3], (mine - 1) >> 1 & 1, &S.gave_up, a.status);
        else at_wait_warp(&S.o_full[grp], ends++ & 1, &S.gave_up, a.status);
        tc_fence_after();
      }
      const bool whole = (s.flags & (SEG_START | SEG_END)) == (SEG_START | SEG_END);
      const int64_t piece = 2 * (int64_t)blockIdx.x + (s.flags & SEG_LATER ? 1 : 0);
      // one query tile: each group joins both groups' sums (a row's are in
      // the same lanes of tensor memory) for half of the columns
      float scale = 1.f, other = 0.f;
      if (!two) {
        S.stats[grp][row] = make_float2(m, l);
        tc_fence_before();
        warps_bar(1, 256);
        tc_fence_after();
        const float2 o = S.stats[1 - grp][row];
        const float to = fmaxf(m, o.x);
        scale = ex2(m - to);
        other = ex2(o.x - to);
        l = grp ? o.y * other + l * scale : l * scale + o.y * other;
        m = to;
      }
      const float inv = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
      scale *= inv;
      other *= inv;
      const int64_t t = s.t0 + s.first + skip + my_tok;
      const int h = s.h * a.g + my_head;
      const int c0 = two ? 0 : grp * (DP / 2), c1 = two ? DP : c0 + DP / 2;
      uint16_t *out = a.out + t * a.os + (int64_t)h * a.D;
      float *sums = pieces.sums + (piece * AC_ROWS + (two ? grp * 128 : 0) + row) * DP;
      for (int c = c0; c < c1; c += 16) {
        __syncwarp();  // the loads are the whole warp's, the stores those of lanes with a row
        float o[16];
        tmem_ld16(t_o + c, o);
#pragma unroll
        for (int k = 0; k < 16; ++k) o[k] *= scale;
        if (!two) {
          float p[16];
          tmem_ld16(tmem + lanes + C::SUMS + (1 - grp) * DP + c, p);
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = fmaf(p[k], other, o[k]);
        }
        if (is_row && !whole) {
#pragma unroll
          for (int k = 0; k < 16; k += 4) *reinterpret_cast<float4 *>(sums + c + k) = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
        } else if (is_row) {
#pragma unroll
          for (int k = 0; k < 16; k += 8) {
            if (wide_out) {  // (head_dim is a multiple of 8)
              if (c + k < a.D)
                *reinterpret_cast<uint4 *>(out + c + k) =
                    make_uint4(pack16<BF16>(o[k], o[k + 1]), pack16<BF16>(o[k + 2], o[k + 3]),
                               pack16<BF16>(o[k + 4], o[k + 5]), pack16<BF16>(o[k + 6], o[k + 7]));
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (c + k + e < a.D) out[c + k + e] = (uint16_t)pack16<BF16>(o[k + e], 0.f);
            }
          }
        }
      }
      if (is_row && (two || grp == 0)) {
        if (!whole) pieces.stats[piece * AC_ROWS + (two ? grp * 128 : 0) + row] = make_float2(m, l);
        else if (a.lse) a.lse[t * a.H + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * AT_LN2;
      }
      if (!whole && tid == 0)
        pieces.what[piece] = make_int4(s.t0 + s.first, n0, s.h, PIECE_USED | (s.flags & SEG_START ? PIECE_START : 0) | (s.flags & SEG_END ? PIECE_END : 0));
      __syncwarp();
      tc_fence_before();
      S.segs.done(ks);
      if (!two) warps_bar(1, 256);  // both have read both's sums
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == AC_MMA) {
    tc_fence_after();
    tmem_free<512>(tmem);
  }
}

template <int DP, bool BF16>
cudaError_t launch(const AttnArgs &a, void *ws, cudaStream_t s) {
  using C = AcCfg<DP>;
  constexpr size_t smem = AC_HEAD + (2 * C::QS + C::KS + C::VS) * C::TILE;
  static_assert(sizeof(AcShared<C::KS, C::VS, C::QS>) <= AC_HEAD, "head of a block's shared memory");
  static_assert(smem <= 227 * 1024, "shared memory of a block");
  static OncePerDevice once;
  cudaError_t e = once_per_device(once, []() {
    return cudaFuncSetAttribute(attention_chunk_kernel<DP, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  });
  if (e != cudaSuccess) return e;
  const int blocks = device_sms(), rows = piece_rows(a.page), tok = 128 / a.g;
  CUtensorMap tq, tk, tv;
  if (!make_q_map(&tq, a, tok, BF16) || !make_kv_map(&tk, a.k, a, rows, BF16) || !make_kv_map(&tv, a.v, a, rows, BF16))
    return cudaErrorInvalidValue;
  const bool wide_out = ((uintptr_t)a.out % 16) == 0 && a.os % 8 == 0;
  const Pieces p = pieces_of(ws, blocks, AC_ROWS, DP);
  attention_chunk_kernel<DP, BF16><<<blocks, AC_THREADS, smem, s>>>(a, p, tq, tk, tv, rows, tok, wide_out);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_join<DP, BF16>(a, p, blocks, AC_ROWS, tok, s);
}

}  // namespace

size_t attention_chunk_workspace(int blocks) { return pieces_bytes(blocks, AC_ROWS, 128); }

cudaError_t launch_attention_chunk(const AttnArgs &a, bool bf16, void *ws, cudaStream_t s) {
  if (a.D <= 64) return bf16 ? launch<64, true>(a, ws, s) : launch<64, false>(a, ws, s);
  return bf16 ? launch<128, true>(a, ws, s) : launch<128, false>(a, ws, s);
}

}  // namespace dsm
