// Attention of few query rows a key head over a cache in 8 bits: the decode
// kernel of attention_decode.cu, with the cache's e4m3 elements as operands of
// the tensor cores just as they lie in the pages, so that a tile is read from
// memory once, in 8 bits, and no thread converts it.
//
//   S^T = K Q^T   is 128 keys x NQ.  A query row, times the power of two that
//       brings its largest element to 2^7 .. 2^8, is the sum of QP e4m3 numbers
//       (each the nearest to what is left, times 2^5): two hold the 8 bits of
//       a bf16 exactly, three the 11 of an fp16, down to e4m3's last step
//       (2^-22 and 2^-27 of the row's largest).  Each has its columns.
//   O^T += V^T P^T  is head_dim x NP.  The weights are fp16 numbers times their
//       values' scales, kept 2^7 to 2^15 times what they are to the row's
//       largest (AT_LIFT in attention_tc.cuh says why), and cut into e5m2
//       numbers: the upper byte of an fp16 is one, and what is left, less than a
//       quarter of its power of two, goes 8 times larger to the next.  Four hold an
//       fp16 exactly; for a result in bf16 three are enough (9 bits, where rounding
//       to bf16 keeps 8, down to 2^-30 of the row's largest).
//
// A key's scale multiplies its scores, in the row of the tile that its thread
// has; a value's scale is its logarithm added to the score: the running maximum is then
// that of weight times scale, whatever blocks' scales are to one another, and the sum of
// the weights alone takes each with 1 / scale.  There a key may count whose weight times
// scale is far below the maximum: exponentials are kept another 2^22 higher (A8_MORE), so
// that where scales are 2^120 apart weights go down to 2^-35 of the largest, and 2^30 of
// them add up to less than 2^127; sums are brought to another maximum in two steps.
//
// A step is KP tiles of 128 keys, two for up to 8 query rows and one for more:
// what each warp does once a step (waits, barriers, addresses, page ids) costs as
// much as its share of the arithmetic (3 requests of 68 to 93 thousand keys 101 us
// with two, 112 with one).  Warps: two groups of four for the softmax take the
// steps in turn, a thread a key of each tile, its scales loaded a step ahead; one
// issues the products, whichever's operands are there first; one copies keys and
// says which segments there are; one copies values and says where a step's rows
// lie, for the scales; one splits the query rows.  They all share the instruction
// cache, and the kernel's size counts as much as its instructions do: what happens
// once a segment is rolled or out of line, and both copying warps run one code.
//
// Measured (of several cards, the fastest and the slowest): 64
// requests of 217 to 8138 keys, 32 heads over 8 of 128, bf16, 99 to 108 us, 82 to 75 % of
// the copy bandwidth, with 16 rows a key head 118 (fp16 130), with 32 170 (184);
// 3 requests of 68 to 93 thousand keys, 64 heads over 8, pages of 16
// rows, fp16, 92 to 100 us; the same over a 16-bit cache 177 and 165.  29 requests
// of 1 to 4 tokens with 7 query heads a key head of 64, 36 us.  (The room for the sum
// costs nothing up to 8 rows, 1 % with 16 and 32, in fp16 4 %.)  Few-row calls
// wait for memory: 128-byte rows of a head, as the 16-bit kernel's 256-byte ones.
// More rows cost the softmax threads their exponentials and the cut of the weights.
#include "attention_tc.cuh"
#include "kv8.cuh"

namespace dsm {
namespace {

constexpr int A8_THREADS = 384;
constexpr int A8_MMA = 8, A8_KEYS = 9, A8_VALUES = 10, A8_QUERIES = 11;
constexpr float A8_MORE = 22.f, A8_MORE_BY = 0x1p22f, A8_LESS_BY = 0x1p-22f;
constexpr float A8_LIFT = AT_LIFT<false> + A8_MORE;
constexpr int A8_READERS = 10;  // warps that read the segments that the keys' warp publishes
constexpr int A8_QSCALES = 8;  // segments whose query rows' factors are kept

// R query rows at most, heads of up to DP elements.
template <int R, int DP, bool BF16>
struct A8Cfg {
  static constexpr int KP = R <= 8 ? 2 : 1;  // tiles a step
  static constexpr int QP = BF16 ? 2 : 3, PP = BF16 ? 3 : 4;
  static constexpr int NQ = (R * QP + 15) / 16 * 16, NP = (R * PP + 15) / 16 * 16;
  static constexpr uint32_t TILE = AT_KEYS * DP, STEP = KP * TILE, Q = NQ * 128, P = KP * NP * 128;
  // steps whose scores are computed ahead: two buffers a group, as far as tensor memory goes
  static constexpr int AHEAD = 4 * KP * NQ + 2 * NP <= 512 ? 4 : 2;
  static constexpr int COLUMNS = AHEAD * KP * NQ + 2 * NP;
  static constexpr int TMEM = COLUMNS <= 128 ? 128 : COLUMNS <= 256 ? 256 : 512;
  // slots of a step's keys (free once the scores are there), and of its values and scales
  static constexpr int KS = (DP == 128 ? 2 : 3) * (KP == 2 ? 1 : 2);
  static constexpr int ROOM = 227 * 1024 - 1024 - 2 * (Q + P) - KS * (int)STEP - 6144 - 24 * R * 8;
  static constexpr int FIT = ROOM / ((int)STEP + 256);
  static constexpr int VS = FIT < 6 ? FIT : 6;
};

template <int R, int KP, int KS, int VS, int AHEAD>
struct A8Shared {
  int2 run[VS][32];  // a step's runs of rows: page (below zero: none), row
  int head[VS];      // and its key head
  uint64_t k_full[KS], k_empty[KS], v_full[VS], v_empty[VS], placed[VS];
  uint64_t q_full[2], q_empty[2], s_full[AHEAD], p_full[2], o_full[2], drain;
  alignas(16) float query[A8_QSCALES][R];  // what a segment's rows were divided by
  alignas(16) float ref[2][R];
  float2 factor[2][R];  // (one factor, in two parts)
  alignas(16) float2 weight[R];
  int64_t place[R];
  float top[2][4][32];
  float sum[2][4][32];
  uint32_t odd[2][KP][4];
  SegRing segs;
  int64_t part[A8_THREADS / 32];
  Start start;
  uint32_t tmem;
  int gave_up;
};

// A step's runs of rows, as in TileRuns: lane i has the i-th, of KEYS / rows.
struct StepRuns {
  int page, row;
  bool sees;
  __device__ __forceinline__ void find(const AttnArgs &a, int r, int pos0, int n, int tile, int keys, int rows) {
    const int lane = threadIdx.x & 31, j = tile * AT_KEYS + lane * rows, lo = a.window ? pos0 + 1 - a.window : 0;
    sees = lane * rows < keys && j < pos0 + n && j + rows > lo;
    if (sees) {
      const int col = (int)((uint64_t)(uint32_t)j * a.by_page >> a.page_shift);
      row = j - col * a.page;
      page = a.table[r * a.table_stride + col];
      if (page < 0 || page >= a.n_pages) page = -1;
    }
  }
};

// By a whole warp: the copies of a step's `keys` rows of keys or of values into
// a slot, once it is free (`wait`): a run, or two neighbours that lie together
// in a page (KvMaps), each a box.  False where the wait ran out.  (One function
// for both: warps of different roles share an instruction cache.)
template <int DP>
__device__ __noinline__ bool copy_step(const AttnArgs &a, const StepRuns now, uint8_t *slot, const KvMaps *maps, int head, int keys, int rows,
                                       uint64_t *full, uint64_t *empty, int par, bool wait, int *gave_up) {
  const int lane = threadIdx.x & 31;
  bool ok = true;
  if (lane == 0 && wait) ok = at_wait(empty, par, gave_up, a.status);
  if (!__shfl_sync(0xffffffffu, ok, 0)) return false;
  if (lane == 0) mbar_arrive_expect_tx(full, keys * DP);
  __syncwarp();
  const bool there = now.sees && now.page >= 0;
  bool pair = false, paired = false;
  if (rows == AT_PAIR_ROWS && a.page > AT_PAIR_ROWS) {
    const bool next = __shfl_down_sync(0xffffffffu, there, 1);
    pair = there && next && lane < 31 && !(now.row & AT_PAIR_ROWS) && now.row + 2 * AT_PAIR_ROWS <= a.page;
    paired = __shfl_up_sync(0xffffffffu, pair, 1) && lane > 0;
  }
  if (lane * rows < keys && !paired)
    tma_load_4d(slot + lane * rows * DP, pair ? &maps->two : &maps->one, 0, there ? now.row : 0, head, there ? now.page : -1, full);
  __syncwarp();
  return true;
}

template <int W>
__device__ __forceinline__ void tmem_ldw(uint32_t t, float *v) {
  if (W == 8) tmem_ld8(t, v);
  else if (W == 16) tmem_ld16(t, v);
  else tmem_ld32(t, v);
}

// A key's scores of R query rows: the sum of the columns of their QP parts,
// times what each row was divided by.
template <int R, int QP, int NQ>
__device__ __forceinline__ void row_scores(uint32_t t_s, const float *query, float (&x)[R]) {
  constexpr float STEP = 0x1p-5f;
  if (NQ <= 32) {
    float v[NQ];
    tmem_ldw<NQ>(t_s, v);
#pragma unroll
    for (int c = 0; c < R; ++c) {
      float s = v[(QP - 1) * R + c];
#pragma unroll
      for (int p = QP - 2; p >= 0; --p) s = fmaf(s, STEP, v[p * R + c]);
      x[c] = s;
    }
  } else {
#pragma unroll
    for (int c0 = 0; c0 < R; c0 += 16) {
      tmem_ldw<16>(t_s + (QP - 1) * R + c0, x + c0);
#pragma unroll
      for (int p = QP - 2; p >= 0; --p) {
        float v[16];
        tmem_ldw<16>(t_s + p * R + c0, v);
#pragma unroll
        for (int c = 0; c < 16; c += 2) {
          const float2 s = fma2(make_float2(x[c0 + c], x[c0 + c + 1]), make_float2(STEP, STEP), make_float2(v[c], v[c + 1]));
          x[c0 + c] = s.x;
          x[c0 + c + 1] = s.y;
        }
      }
    }
  }
#pragma unroll
  for (int c = 0; c < R; c += 4) {
    const float4 f = *reinterpret_cast<const float4 *>(query + c);
    const float2 u = mul2(make_float2(x[c], x[c + 1]), make_float2(f.x, f.y)), w = mul2(make_float2(x[c + 2], x[c + 3]), make_float2(f.z, f.w));
    x[c] = u.x; x[c + 1] = u.y; x[c + 2] = w.x; x[c + 3] = w.y;
  }
}

// Column sums or maxima over a warp of R values a lane (warp_columns, and for
// 8 columns as well): lane i ends with column i mod R.
template <int R, bool MAX>
__device__ __forceinline__ float warp_rows(float (&v)[R]) {
  if constexpr (R >= 16) {
    return warp_columns<R, MAX>(v);
  } else {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int s = R / 2; s > 0; s >>= 1) {
      const bool up = lane & s;
#pragma unroll
      for (int i = 0; i < s; ++i) {
        const float keep = up ? v[i + s] : v[i], send = up ? v[i] : v[i + s];
        const float got = __shfl_xor_sync(0xffffffffu, send, s);
        v[i] = MAX ? fmaxf(keep, got) : keep + got;
      }
    }
#pragma unroll
    for (int s = R; s < 32; s <<= 1) {
      const float got = __shfl_xor_sync(0xffffffffu, v[0], s);
      v[0] = MAX ? fmaxf(v[0], got) : v[0] + got;
    }
    return v[0];
  }
}

// Where byte d of key k's row is in a tile.
template <int DP>
__device__ __forceinline__ uint32_t tile_byte(int k, int d) {
  return DP == 128 ? k * 128 + (((d >> 4) ^ (k & 7)) << 4) + (d & 15) : k * 64 + (((d >> 4) ^ (k >> 1 & 3)) << 4) + (d & 15);
}

// Whether any of a word's four e4m3 numbers is NaN.
__device__ __forceinline__ uint32_t nan4(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// Approximations of the hardware: log2 to 2^-22, the inverse to one unit in
// the last place.
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float inverse(float x) {
  float y;
  asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// (once a block, and once a segment: kept out of the code that the loops share a
// cache with)
__device__ __noinline__ void decode8_start(const AttnArgs &a, const RawSpan raw0, const Plan plan, Start *out, int64_t *part) {
  find_start<A8_THREADS>(a, raw0, plan, out, part);
}
__device__ __noinline__ const Seg *segment_of(SegRing *ring, int k, unsigned *status) { return &ring->get(k, status); }
__device__ __noinline__ void next_segment(const AttnArgs &a, Segments *s) { s->next(a); }
// NaN among a step's values, added to the sums of the rows that see it (of
// their first parts), R rows: see the caller.
template <int R, int DP>
__device__ __noinline__ void add_nan(const uint8_t *tiles, const uint32_t (*odd)[4], int keys, int j0, int pos0, int n, int g, int window,
                                     int d, uint32_t t_o) {
#pragma unroll 1
  for (int k = 0; k < keys; ++k) {
    if (!(odd[k >> 7][k >> 5 & 3] >> (k & 31) & 1u)) continue;
    const float add = (tiles[(k >> 7) * (AT_KEYS * DP) + tile_byte<DP>(k & 127, d)] & 0x7F) == F8_NAN ? __uint_as_float(0x7FFFFFFFu) : 0.f;
    const int jk = j0 + k, k_lo = max(0, jk - pos0), k_hi = window ? min(n, jk - pos0 + window) : n;
#pragma unroll 1
    for (int c0 = 0; c0 < R; c0 += 8) {
      float o[8];
      tmem_ld8(t_o + c0, o);
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (c0 + c >= k_lo * g && c0 + c < k_hi * g) o[c] += add;
      tmem_st8(t_o + c0, o);
    }
    tmem_st_wait();
  }
}

template <int R, int DP, bool BF16>
__global__ void __launch_bounds__(A8_THREADS, 1)
    attention8_decode_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ Pieces pieces, const __grid_constant__ KvMaps tm_k,
                             const __grid_constant__ KvMaps tm_v, int rows, int item) {
  using C = A8Cfg<R, DP, BF16>;
  constexpr int KP = C::KP, KS = C::KS, VS = C::VS, AHEAD = C::AHEAD, NQ = C::NQ, NP = C::NP, QP = C::QP, PP = C::PP;
  constexpr int KEYS = KP * AT_KEYS;
  const Plan PLAN = {1 << 20, 1 << 20, item};  // one block of tokens a request
  extern __shared__ uint8_t raw[];
  uint8_t *smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  uint8_t *kring = smem, *vring = kring + KS * C::STEP, *qbuf = vring + VS * C::STEP, *pbuf = qbuf + 2 * C::Q;
  typedef A8Shared<R, KP, KS, VS, AHEAD> Sh;
  Sh &S = *reinterpret_cast<Sh *>(pbuf + 2 * C::P);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  asm volatile("griddepcontrol.launch_dependents;");
  const RawSpan raw0 = first_request<A8_THREADS>(a);  // (under way while the block is set up)

  if (tid < KS) {
    mbar_init(&S.k_full[tid], 1);
    mbar_init(&S.k_empty[tid], 1);
    fence_mbar_init();
  } else if (tid >= 32 && tid < 32 + VS) {
    mbar_init(&S.v_full[tid - 32], 1);
    mbar_init(&S.v_empty[tid - 32], 1);
    mbar_init(&S.placed[tid - 32], 1);
    fence_mbar_init();
  } else if (tid >= 64 && tid < 64 + AHEAD) {
    const int i = tid - 64;
    mbar_init(&S.s_full[i], 1);
    if (i < 2) {
      mbar_init(&S.q_full[i], 1);
      mbar_init(&S.q_empty[i], 1);
      mbar_init(&S.p_full[i], 4);
      mbar_init(&S.o_full[i], 1);
    }
    if (i == 0) mbar_init(&S.drain, 1), S.gave_up = 0;
    fence_mbar_init();
  } else if (tid >= 128 && tid < 128 + AT_SEGS) {
    S.segs.init(tid - 128, A8_READERS);
    fence_mbar_init();
  } else if (tid == 96) {
    const CUtensorMap *maps[2] = {&tm_k.one, &tm_v.one};
    for (int i = 0; i < 2; ++i) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(maps[i])) : "memory");
  }
  if (tid == 0) {
    pieces.what[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
    pieces.what[2 * blockIdx.x + 1] = make_int4(0, 0, 0, 0);
  }
  __syncwarp();
  if (warp == A8_MMA) tmem_alloc<C::TMEM>(&S.tmem);
  // columns that no row is written to, and elements behind a head's end, stay zero
  for (int i = tid; i < (int)(2 * (C::Q + C::P) / 16); i += A8_THREADS) reinterpret_cast<uint4 *>(qbuf)[i] = make_uint4(0, 0, 0, 0);
  // (whoever goes on after a wait that ran out finds pages that are none)
  for (int i = tid; i < VS * 32; i += A8_THREADS) S.run[i >> 5][i & 31] = make_int2(-1, 0);
  fence_proxy_async();
  decode8_start(a, raw0, PLAN, &S.start, S.part);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem;  // scores of step f at (f mod AHEAD) KP NQ, sums of group i at AHEAD KP NQ + i NP
  constexpr int SUMS = AHEAD * KP * NQ;
  if (warp == A8_KEYS || warp == A8_VALUES) {
    // ------------------------------------------- segments, keys and values --
    // (the same code for both, so that it is in the instruction cache once)
    const bool keys = warp == A8_KEYS;
    const KvMaps *maps = keys ? &tm_k : &tm_v;
    uint8_t *ring = keys ? kring : vring;
    uint64_t *full = keys ? S.k_full : S.v_full, *empty = keys ? S.k_empty : S.v_empty;
    const int slots = keys ? KS : VS;
    Segments s;
    s.init(a, PLAN, S.start);
    bool bad = false;
    int sl = 0, par = 1;                     // slot, and the phase that frees it
    int f = 0, i = 0, segs = 0;              // step of the stretch; tile of the segment; segments
    StepRuns now, later;
    int count = min(KP, s.count), then = 0;  // tiles of the step, of the next
    if (count) now.find(a, s.r, s.sp.pos0, s.n, s.tile, count * AT_KEYS, rows);
    if (keys) S.segs.put(segs++, s, true, &S.gave_up, a.status);
    while (count) {
      const int head = s.h;
      i += count;
      if (i == s.count) {
        // a segment is published before the last step of the one before it is
        // copied: whoever has that step's scores behind it never waits here
        // for copies that wait for it
        Segments following = s;
        next_segment(a, &following);
        s = following;
        if (keys) S.segs.put(segs++, s, true, &S.gave_up, a.status);
        i = 0;
      }
      then = min(KP, s.count - i);
      if (then > 0) later.find(a, s.r, s.sp.pos0, s.n, s.tile + i, then * AT_KEYS, rows);
      bad = bad || (now.sees && now.page < 0);
      if (!copy_step<DP>(a, now, ring + sl * C::STEP, maps, head, count * AT_KEYS, rows, &full[sl], &empty[sl], par, f >= slots, &S.gave_up))
        break;
      if (!keys) {  // for the scales
        if (lane * rows < KEYS) S.run[sl][lane] = make_int2(now.sees ? now.page : -1, now.row);
        if (lane == 0) S.head[sl] = head;
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.placed[sl]);
        __syncwarp();
      }
      ++f;
      if (++sl == slots) sl = 0, par ^= 1;
      now = later;
      count = then;
    }
    if (keys && s.count) S.segs.put(segs, s, false, &S.gave_up, a.status);  // (gave up)
    if (bad) flag(a.status, ST_PAGING);
    if (lane == 0) {  // every copy of this warp has landed before the block ends
      int off = 0;
      for (int g = max(0, f - slots); g < f; ++g) at_wait(&full[g % slots], (g / slots) & 1, &off, a.status);
    }
  } else if (warp == A8_QUERIES) {
    // ------------------------------------------------------------ queries --
    constexpr int LANES = DP / 8, AT_ONCE = 32 / LANES;  // lanes a row, rows at once
    const int d = lane % LANES * 8;
    bool ok = true;
    int k = 0;
    for (;; S.segs.done(k++)) {
      const Seg s = *segment_of(&S.segs, k, a.status);
      if (!s.count) break;
      if (!ok) continue;  // (gave up: the others' segments go on to their end)
      const int b = k & 1, nrows = s.n * a.g;
      auto row_words = [&](int row) {
        const int tok = row / a.g;
        if (row >= nrows || d >= a.D) return make_uint4(0, 0, 0, 0);
        return *reinterpret_cast<const uint4 *>(a.q + (int64_t)(s.t0 + tok) * a.qs + (int64_t)(s.h * a.g + row - tok * a.g) * a.D + d);
      };
      uint4 words = row_words(lane / LANES);
      if (lane == 0 && k >= 2 && !at_wait(&S.q_empty[b], ((k >> 1) & 1) ^ 1, &S.gave_up, a.status)) ok = false;
      if (!(ok = __shfl_sync(0xffffffffu, ok, 0))) continue;
      uint8_t *buf = qbuf + b * C::Q;
#pragma unroll 1
      for (int row = lane / LANES; row < R; row += AT_ONCE) {
        const uint32_t word[4] = {words.x, words.y, words.z, words.w};
        if (row + AT_ONCE < R) words = row_words(row + AT_ONCE);
        float x[8], most = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint16_t h = (uint16_t)(word[e / 2] >> (e & 1) * 16);
          x[e] = BF16 ? bf16_to_f32(h) : fp16_to_f32(h);
          if (fabsf(x[e]) <= FLT_MAX) most = fmaxf(most, fabsf(x[e]));
          else x[e] = __uint_as_float(0x7FFFFFFFu);
        }
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
        // times 2^(7 - exponent of the largest): its exponent is 7 then
        const int e2 = most > 0.f ? min(7 + 127 - (int)(__float_as_uint(most) >> 23), 120) : 0;
        const float by = __uint_as_float((uint32_t)(127 + e2) << 23);
        if (d == 0) S.query[k % A8_QSCALES][row] = __uint_as_float((uint32_t)(127 - e2) << 23);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= by;
#pragma unroll 1
        for (int p = 0; p < QP; ++p) {
          uint16_t part[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            part[e] = f8x2_of(x[2 * e], x[2 * e + 1]);
            const float2 is = f8x2_to(part[e]);
            x[2 * e] = (x[2 * e] - is.x) * 32.f;
            x[2 * e + 1] = (x[2 * e + 1] - is.y) * 32.f;
          }
          const int at = p * R + row;
          *reinterpret_cast<uint2 *>(buf + at * 128 + (((d >> 4) ^ (at & 7)) << 4) + (d & 8)) =
              make_uint2(part[0] | (uint32_t)part[1] << 16, part[2] | (uint32_t)part[3] << 16);
        }
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.q_full[b]);
      __syncwarp();
    }
  } else if (warp == A8_MMA) {
    // ----------------------------------------------------------- products --
    // (the whole warp walks; one lane issues)
    const uint32_t by = elect_one(), tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t id_s = f8_idesc(NQ), id_o = f8_idesc(NP) | IDESC_A_MN | IDESC_B_E5M2;
    const uint64_t k0 = DP == 128 ? sw128_desc(smem_u32(kring)) : sw64_desc(smem_u32(kring));
    const uint64_t q0 = sw128_desc(smem_u32(qbuf)), p0 = sw128_desc(smem_u32(pbuf));
    // heads of 64: rows 64..127 of the second product are other keys' elements and not used
    const uint64_t v0 = DP == 128 ? sw128_mn_desc(smem_u32(vring), 1024) : sw64_desc(smem_u32(vring), 512);
    // Scores are computed as soon as their keys are there, up to AHEAD steps
    // before the step whose weights are next: neither waits for the other.
    int ks = 0, is = 0, kv = 0, iv = 0;  // segment and tile of it that scores are at, and values
    int ns = segment_of(&S.segs, 0, a.status)->count, nv = ns;
    int fs = 0, fv = 0, kslot = 0, kpar = 0, vslot = 0, vpar = 0, buf = 0;
    bool asked = true;  // the segment's query rows have yet to be waited for
    auto there = [&](uint64_t *b, int par) { return __all_sync(0xffffffffu, mbar_test_wait(b, par & 1)); };
    uint64_t idle = 0;
    while (nv) {
      if (ns && fs < fv + AHEAD && (!asked || there(&S.q_full[ks & 1], ks >> 1)) && there(&S.k_full[kslot], kpar)) {
        asked = false;
        tc_fence_after();
        const uint64_t kd = k0 + kslot * (C::STEP / 16), qd = q0 + (ks & 1) * (C::Q / 16);
#pragma unroll
        for (int t = 0; t < KP; ++t) {
          if (t && is + t >= ns) break;
#pragma unroll
          for (int x = 0; x < DP / 32; ++x)  // (addresses in a descriptor count 16 bytes)
            mma_f8_by(by, tm + (buf * KP + t) * NQ, kd + t * (C::TILE / 16) + x * 2, qd + x * 2, id_s, x > 0);
        }
        mma_commit_by(by, &S.s_full[buf]);
        mma_commit_by(by, &S.k_empty[kslot]);
        if (++buf == AHEAD) buf = 0;
        if (++kslot == KS) kslot = 0, kpar ^= 1;
        ++fs;
        is += KP;
        if (is >= ns) {
          mma_commit_by(by, &S.q_empty[ks & 1]);
          ns = segment_of(&S.segs, ++ks, a.status)->count;
          is = 0;
          asked = true;
        }
        idle = 0;
      } else if (fv < fs && there(&S.p_full[fv & 1], fv >> 1) && there(&S.v_full[vslot], vpar)) {
        tc_fence_after();
        const uint64_t vd = v0 + vslot * (C::STEP / 16), pd = p0 + (fv & 1) * (C::P / 16);
        const uint32_t d = tm + SUMS + (fv & 1) * NP;
#pragma unroll
        for (int t = 0; t < KP; ++t) {
          if (t && iv + t >= nv) break;
#pragma unroll
          for (int x = 0; x < AT_KEYS / 32; ++x)
            mma_f8_by(by, d, vd + t * (C::TILE / 16) + x * (32 * DP / 16), pd + t * (NP * 128 / 16) + x * 2, id_o, true);
        }
        mma_commit_by(by, &S.o_full[fv & 1]);
        mma_commit_by(by, &S.v_empty[vslot]);
        if (++vslot == VS) vslot = 0, vpar ^= 1;
        ++fv;
        iv += KP;
        if (iv >= nv) {
          S.segs.done(kv);
          nv = segment_of(&S.segs, ++kv, a.status)->count;
          iv = 0;
        }
        idle = 0;
      } else {
        // nothing is ready: a short sleep at the weights that come next (or keys), within the limit
        if (fv < fs) mbar_try_wait_sleep(&S.p_full[fv & 1], fv >> 1 & 1, 200u);
        else mbar_try_wait_sleep(&S.k_full[kslot], kpar, 200u);
        __syncwarp();
        const uint64_t now = globaltimer_ns();
        if (!idle) idle = now;
        int late = now - idle > AT_LIMIT_NS;
        if (late) {
          flag(a.status, ST_TIMEOUT);
          *(volatile int *)&S.gave_up = 1;
        }
        late |= *(volatile int *)&S.gave_up;
        if (__any_sync(0xffffffffu, late)) break;
      }
    }
    for (; nv; nv = segment_of(&S.segs, ++kv, a.status)->count) S.segs.done(kv);  // (gave up)
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
    const uint32_t t_o = tmem + lanes + SUMS + grp * NP;
    uint8_t *pm = pbuf + grp * C::P;
    const int p_chunk = key >> 4;
    int st = 0, mine = 0;  // steps before the segment, steps that this group has taken (the i-th is step 2 i + group)
    int sl = grp % VS, par = 0, buf = grp % AHEAD, bpar = 0;  // of the group's next step: value slot and its phase, scores and theirs
    // The scales of this thread's keys, loaded a step of the group ahead where
    // their pages are known by then (the step may not come).
    const int log_rows = 31 - __clz(rows);
    float kscale[KP], vscale[KP];
    bool have = false;
    auto load_scales = [&](int slot) {
      const int head = S.head[slot];
#pragma unroll
      for (int t = 0; t < KP; ++t) {
        const int j = t * AT_KEYS + key;
        const int2 run = S.run[slot][j >> log_rows];
        // (row below 2^16: row / block as a product with 2^32 / block, rounded up)
        const uint32_t row = run.y + (j & (rows - 1));
        const int64_t at = run.x * a.sps + (int64_t)(row * a.by_block >> 32) * a.sbs + head * a.shs;
        kscale[t] = vscale[t] = 0.f;  // (of a page that is none: nothing multiplies them but zeros)
        if (run.x >= 0) kscale[t] = a.ks[at], vscale[t] = a.vs[at];
      }
    };
    for (int ks = 0;; ++ks) {
      const Seg &s = *segment_of(&S.segs, ks, a.status);
      __syncwarp();
      const int count = s.count;
      if (!count) break;
      const int n = s.n, tile = s.tile, nrows = n * a.g, pos0 = s.pos0;
      const float *query = S.query[ks % A8_QSCALES];
      float l[R];
#pragma unroll
      for (int c = 0; c < R; ++c) l[c] = 0.f;
      __syncwarp();
      {
        const float z[16] = {};
#pragma unroll
        for (int c = 0; c < NP; c += 16) tmem_st16(t_o + c, z);
        tmem_st_wait();
      }
      if (key < R) S.ref[grp][key] = AT_NONE;
      warps_bar(1 + grp, 128);
      bool done = false;
      // (tiles of this group's steps of the segment; the group of step 0 is st mod 2)
      for (int i = ((st ^ grp) & 1) * KP; i < count; i += 2 * KP) {
        const int j0 = (tile + i) * AT_KEYS, live = min(KP, count - i);
        // whether some row does not see some key of the step, or a tile of it is none
        const bool edge = j0 + KEYS - 1 > pos0 || (a.window && j0 < pos0 + n - a.window) || live < KP;
        int lo[KP], hi[KP];  // columns [lo, hi) see this thread's keys: those of tokens at j .. j + window - 1
        if (edge) {
#pragma unroll
          for (int t = 0; t < KP; ++t) {
            const int j = j0 + t * AT_KEYS + key, t_lo = max(0, j - pos0), t_hi = a.window ? min(n, j - pos0 + a.window) : n;
            lo[t] = min(t_lo, 1 << 16) * a.g;
            hi[t] = t_hi > t_lo && t < live ? t_hi * a.g : 0;
          }
        }
        const uint32_t t_s = tmem + lanes + buf * (KP * NQ);
        if (!have) {
          at_wait_warp(&S.placed[sl], par, &S.gave_up, a.status);
          load_scales(sl);
        }
        float sc[KP], value[KP], per[KP];
#pragma unroll
        for (int t = 0; t < KP; ++t) {
          const float v = kv8_scale(vscale[t]);
          sc[t] = a.scale_log2 * kv8_scale(kscale[t]);
          value[t] = lg2(v);
          per[t] = inverse(v);
        }
        {
          const int wrap = sl + 2 >= VS;
          have = __all_sync(0xffffffffu, mbar_test_wait(&S.placed[sl + 2 - wrap * VS], par ^ wrap));
          if (have) load_scales(sl + 2 - wrap * VS);
        }
        at_wait_warp(&S.s_full[buf], bpar, &S.gave_up, a.status);
        tc_fence_after();
        // the group's last products: their weights' room and the sums are free once they are complete
        bool settled = mine == 0;
        auto settle = [&]() {
          if (!settled) {
            at_wait_warp(&S.o_full[grp], (mine - 1) & 1, &S.gave_up, a.status);
            tc_fence_after();
          }
          settled = true;
        };
        // scores (and the values' scales) less the running maxima, in powers
        // of two: masked ones are -infinity whatever the key holds
        float x[KP][R];
        auto less_maxima = [&]() {
#pragma unroll
          for (int c = 0; c < R; c += 4) {
            const float4 m = *reinterpret_cast<const float4 *>(&S.ref[grp][c]);
#pragma unroll
            for (int t = 0; t < KP; ++t) {
              const float2 u = add2(make_float2(x[t][c], x[t][c + 1]), make_float2(-m.x, -m.y));
              const float2 w = add2(make_float2(x[t][c + 2], x[t][c + 3]), make_float2(-m.z, -m.w));
              x[t][c] = u.x; x[t][c + 1] = u.y; x[t][c + 2] = w.x; x[t][c + 3] = w.y;
            }
          }
        };
        auto scaled_scores = [&]() {
#pragma unroll
          for (int t = 0; t < KP; ++t) {
            row_scores<R, QP, NQ>(t_s + t * NQ, query, x[t]);
            const float2 v2 = make_float2(value[t], value[t]), s2 = make_float2(sc[t], sc[t]);
#pragma unroll
            for (int c = 0; c < R; c += 2) {
              const float2 u = fma2(make_float2(x[t][c], x[t][c + 1]), s2, v2);
              x[t][c] = u.x; x[t][c + 1] = u.y;
            }
            if (edge) {
#pragma unroll
              for (int c = 0; c < R; ++c) x[t][c] = c >= lo[t] && c < hi[t] ? x[t][c] : -INFINITY;
            }
          }
        };
        bool raise = !done;  // (a segment's first step sets the maxima)
        scaled_scores();
        if (done) {
          less_maxima();
          float top = -INFINITY;
#pragma unroll
          for (int t = 0; t < KP; ++t)
#pragma unroll
            for (int c = 0; c < R; c += 2) top = fmaxf(top, fmaxf(x[t][c], x[t][c + 1]));
          raise = bar_or(1 + grp, 128, top > AT_SLACK + A8_LIFT);
          if (raise) scaled_scores();
        }
        if (raise) {
          // raise the maxima to the step's, and bring the sums down to them
          settle();
          float v[R];
#pragma unroll
          for (int c = 0; c < R; ++c) {
            v[c] = fmaxf(x[0][c], -INFINITY);  // (of a NaN and another: the other)
            if (KP == 2) v[c] = fmaxf(v[c], x[KP - 1][c]);
          }
          const float t = warp_rows<R, true>(v);
          if (lane < R) S.top[grp][wq][lane] = t;
          warps_bar(1 + grp, 128);
          if (key < R) {
            const float was = S.ref[grp][key];
            const float to = fmaxf(fmaxf(fmaxf(S.top[grp][0][key], S.top[grp][1][key]),
                                         fmaxf(S.top[grp][2][key], S.top[grp][3][key])) - A8_LIFT, was);
            S.ref[grp][key] = to;
            S.factor[grp][key] = ex2_parts(was - to);
          }
          warps_bar(1 + grp, 128);
          if (done) {
#pragma unroll
            for (int c = 0; c < R; ++c) l[c] = l[c] * S.factor[grp][c].x * S.factor[grp][c].y;
#pragma unroll 1
            for (int c0 = 0; c0 < NP; c0 += 16) {
              float o[16];
              tmem_ld16(t_o + c0, o);
#pragma unroll
              for (int c = 0; c < 16; ++c) {
                const float2 f = S.factor[grp][(c0 + c) & (R - 1)];
                o[c] *= f.x * f.y;
              }
              tmem_st16(t_o + c0, o);
            }
            tmem_st_wait();
          }
          less_maxima();
        }
#pragma unroll
        for (int t = 0; t < KP; ++t) {
#pragma unroll
          for (int c = 0; c < R; c += 2) {
            const float p0 = ex2(x[t][c]), p1 = ex2(x[t][c + 1]);
            const float2 w = fma2(make_float2(p0, p1), make_float2(per[t], per[t]), make_float2(l[c], l[c + 1]));
            l[c] = w.x;
            l[c + 1] = w.y;
            const float2 q = mul2(make_float2(p0, p1), make_float2(A8_LESS_BY, A8_LESS_BY));
            x[t][c / 2] = __uint_as_float(pack16<false>(q.x, q.y));
          }
        }
        settle();
#pragma unroll
        for (int t = 0; t < KP; ++t) {
#pragma unroll
          for (int c = 0; c < R; c += 2) {
            __half2 rest = *reinterpret_cast<__half2 *>(&x[t][c / 2]);
#pragma unroll
            for (int p = 0; p < PP; ++p) {
              uint32_t w = *reinterpret_cast<uint32_t *>(&rest);
              // (three of them: the last is the nearest, not the one below)
              w = (PP == 3 && p == 2 ? w + 0x00800080u : w) & 0xFF00FF00u;
              const int at = p * R + c;
              uint8_t *to = pm + (t * NP + at) * 128 + (key & 15);
              to[(p_chunk ^ (at & 7)) << 4] = (uint8_t)(w >> 8);
              to[128 + ((p_chunk ^ ((at + 1) & 7)) << 4)] = (uint8_t)(w >> 24);
              if (p + 1 < PP) rest = __hmul2(__hsub2(rest, *reinterpret_cast<__half2 *>(&w)), __float2half2_rn(8.f));
            }
          }
        }
        if (edge) {
          // values that not every row sees: a weight of zero does not take
          // away a NaN, so rows that no token sees are cleared, and what is NaN
          // in others is added to the sums of the rows that see it, and cleared
          at_wait_warp(&S.v_full[sl], par, &S.gave_up, a.status);
          bool odd[KP], any_odd = false;
#pragma unroll
          for (int t = 0; t < KP; ++t) {
            uint8_t *vt = vring + sl * C::STEP + t * C::TILE;
            odd[t] = false;
            if (t < live && hi[t] <= lo[t]) {
#pragma unroll
              for (int x = 0; x < DP / 16; ++x)
                *reinterpret_cast<uint4 *>(vt + key * DP + ((x + lane) & (DP / 16 - 1)) * 16) = make_uint4(0, 0, 0, 0);
            } else if (t < live && (lo[t] > 0 || hi[t] < nrows)) {
              uint32_t any = 0;
#pragma unroll
              for (int x = 0; x < DP / 16; ++x) {
                const uint4 w = *reinterpret_cast<const uint4 *>(vt + key * DP + ((x + lane) & (DP / 16 - 1)) * 16);
                any |= nan4(w.x) | nan4(w.y) | nan4(w.z) | nan4(w.w);
              }
              odd[t] = any != 0;
              any_odd = any_odd || odd[t];
            }
          }
          if (n > 1 && bar_or(1 + grp, 128, any_odd)) {
#pragma unroll
            for (int t = 0; t < KP; ++t) {
              const uint32_t m = __ballot_sync(0xffffffffu, odd[t]);
              if (lane == 0) S.odd[grp][t][wq] = m;
            }
            warps_bar(1 + grp, 128);
            add_nan<R, DP>(vring + sl * C::STEP, S.odd[grp], live * AT_KEYS, j0, pos0, n, a.g, a.window, key & (DP - 1), t_o);
            warps_bar(1 + grp, 128);
#pragma unroll
            for (int t = 0; t < KP; ++t) {
              if (!odd[t]) continue;
#pragma unroll 1
              for (int x = 0; x < DP / 4; ++x) {
                uint32_t *w = reinterpret_cast<uint32_t *>(vring + sl * C::STEP + t * C::TILE + key * DP + x * 4);
                const uint32_t n = nan4(*w);
                if (n) *w &= ~((n >> 7) * 0xFFu);
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
        done = true;
        sl += 2;
        if (sl >= VS) sl -= VS, par ^= 1;
        buf += 2;
        if (buf >= AHEAD) buf -= AHEAD, bpar ^= 1;
      }
      st += (count + KP - 1) / KP;
      // ---- the segment's end: each group finishes half of the rows ----
      {
        const float t = warp_rows<R, false>(l);
        if (lane < R) S.sum[grp][wq][lane] = t;
      }
      if (done) {
        at_wait_warp(&S.o_full[grp], (mine - 1) & 1, &S.gave_up, a.status);
        tc_fence_after();
      }
      // both groups' products are done before the weights' room is taken for
      // the exchange: [rows][DP] sums
      warps_bar(3, 256);
      float *ex = reinterpret_cast<float *>(pbuf);
      constexpr int HALF = R / 2;
      static_assert(R * DP * 4 <= 2 * C::P, "room for the exchange");
      const bool whole = (s.flags & (SEG_START | SEG_END)) == (SEG_START | SEG_END);
      const int64_t piece = 2 * (int64_t)blockIdx.x + (s.flags & SEG_LATER ? 1 : 0);
      if (key < HALF && grp * HALF + key < nrows) {  // a thread a row: its weights and place
        const int row = grp * HALF + key;
        const float m0 = S.ref[0][row], m1 = S.ref[1][row], m = fmaxf(m0, m1), w0 = ex2(m0 - m), w1 = ex2(m1 - m);
        const float s0 = (S.sum[0][0][row] + S.sum[0][1][row]) + (S.sum[0][2][row] + S.sum[0][3][row]);
        const float s1 = (S.sum[1][0][row] + S.sum[1][1][row]) + (S.sum[1][2][row] + S.sum[1][3][row]);
        const float total = times_ex2(s0, m0 - m) + times_ex2(s1, m1 - m);
        const float inv = !whole ? A8_MORE_BY : total == 0.f ? 0.f : A8_MORE_BY / total;
        S.weight[row] = make_float2((grp ? w1 : w0) * inv, (grp ? w0 : w1) * inv);
        if (whole) {
          const int tok = row / a.g;
          const int64_t t = s.t0 + tok;
          const int h = s.h * a.g + row - tok * a.g;
          S.place[row] = t * a.os + (int64_t)h * a.D;
          if (a.lse) a.lse[t * a.H + h] = total == 0.f ? -INFINITY : (m + log2f(total)) * AT_LN2;
        } else {
          S.place[row] = (piece * R + row) * DP;
          pieces.stats[piece * R + row] = make_float2(m, total);
        }
      }
      __syncwarp();
      float o[R];  // the rows' sums: their parts together
      tmem_ldw<R>(t_o + (PP - 1) * R, o);
#pragma unroll
      for (int p = PP - 2; p >= 0; --p) {
        float v[R];
        tmem_ldw<R>(t_o + p * R, v);
#pragma unroll
        for (int c = 0; c < R; ++c) o[c] = fmaf(o[c], 0x1p-3f, v[c]);
      }
      if (key < DP) {
#pragma unroll
        for (int c = 0; c < HALF; ++c) ex[((1 - grp) * HALF + c) * DP + key] = grp ? o[c] : o[HALF + c];
      }
      __syncwarp();
      tc_fence_before();
      warps_bar(3, 256);
      if (key < (whole ? a.D : DP)) {
#pragma unroll
        for (int c = 0; c < HALF; ++c) {
          const int row = grp * HALF + c;
          if (row < nrows) {
            const float2 w = S.weight[row];
            // (a sum of zero keys times a weight of zero: sums are zeros then, not garbage)
            const float v = (grp ? o[HALF + c] : o[c]) * w.x + ex[row * DP + key] * w.y;
            if (whole) a.out[S.place[row] + key] = (uint16_t)pack16<BF16>(v, 0.f);
            else pieces.sums[S.place[row] + key] = v;
          }
        }
      }
      if (!whole && tid == 0)
        pieces.what[piece] = make_int4(s.t0, n, s.h, PIECE_USED | (s.flags & SEG_START ? PIECE_START : 0) | (s.flags & SEG_END ? PIECE_END : 0));
      S.segs.done(ks);
      warps_bar(3, 256);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == A8_MMA) {
    tc_fence_after();
    tmem_free<C::TMEM>(tmem);
  }
}

// Tiles that an item costs besides its own: its first step, and its sums' way
// out.  With more query rows it costs more, which shows where a block has
// several items (64 requests of 200 to 8200 keys, 8 key heads: 16 rows 135 us
// with 4, 122 with 9, 121 with 10; 32 rows 207, 163, 169; 8 rows, before the scales
// were loaded ahead, 126 with 2, 113 with 4 and 7); with few items it is better to
// cut them finely (29 requests of up to 28 rows, 4 key heads: 8 is 5 % slower than 4).
int item_tiles(int rows, int64_t items, int blocks) { return rows > 8 && items > 2 * blocks ? 9 : 4; }

template <int R, int DP, bool BF16>
cudaError_t launch(const AttnArgs &a, void *ws, cudaStream_t s) {
  using C = A8Cfg<R, DP, BF16>;
  constexpr size_t smem = 1024 + (C::KS + C::VS) * C::STEP + 2 * (C::Q + C::P) + sizeof(A8Shared<R, C::KP, C::KS, C::VS, C::AHEAD>);
  static_assert(smem <= 227 * 1024, "shared memory of a block");
  static_assert(C::AHEAD <= C::VS + 1 && C::VS >= 3, "a segment's queries are split before the products in flight wait for them");
  static OncePerDevice once;
  cudaError_t e = once_per_device(once, []() {
    return cudaFuncSetAttribute(attention8_decode_kernel<R, DP, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  });
  if (e != cudaSuccess) return e;
  const int blocks = device_sms(), rows = piece_rows(a.page);
  KvMaps tk, tv;
  if (!make_kv8_maps(&tk, a.k, a, rows, DP) || !make_kv8_maps(&tv, a.v, a, rows, DP)) return cudaErrorInvalidValue;
  const Pieces p = pieces_of(ws, blocks, R, DP);
  attention8_decode_kernel<R, DP, BF16><<<blocks, A8_THREADS, smem, s>>>(a, p, tk, tv, rows, item_tiles(R, (int64_t)a.R * a.G, blocks));
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_join<DP, BF16, true>(a, p, blocks, R, 1 << 20, s);
}

template <int R>
cudaError_t launch_rows(const AttnArgs &a, bool bf16, void *ws, cudaStream_t s) {
  if (a.D <= 64) return bf16 ? launch<R, 64, true>(a, ws, s) : launch<R, 64, false>(a, ws, s);
  return bf16 ? launch<R, 128, true>(a, ws, s) : launch<R, 128, false>(a, ws, s);
}

}  // namespace

cudaError_t launch_attention8_decode(const AttnArgs &a, bool bf16, void *ws, cudaStream_t s) {
  const int64_t rows = (int64_t)a.max_new * a.g;
  return rows <= 8 ? launch_rows<8>(a, bf16, ws, s) : rows <= 16 ? launch_rows<16>(a, bf16, ws, s) : launch_rows<32>(a, bf16, ws, s);
}

}  // namespace dsm
