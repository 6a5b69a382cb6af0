// What the tensor-core attention kernels share: how a launch's work is split,
// the copies of keys and values out of their pages, and the joining of
// pieces.
//
// Work is counted in tiles of 128 keys.  An item is a block of query rows
// (tpb tokens of one request, with the query heads that share a key head)
// and the tiles that any of its tokens sees; items follow one another by
// request, key head and block.  The tiles of all items form one line, on which
// each has the length that it costs (Plan), and which the launch's blocks
// share out evenly whatever the lengths are: a block
// takes a stretch of the line, so it begins inside an item and ends inside
// another.  Each such piece leaves its sums, unnormalised, in the workspace
// (at most two a block), and a second kernel joins them in the order of the
// keys, so results do not depend on timing.
#pragma once
#include <float.h>

#include "attention.h"
#include "common.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "serving.cuh"
#include "tcgen05.cuh"

namespace dsm {
namespace {

constexpr int AT_KEYS = 128;
constexpr uint64_t AT_LIMIT_NS = 2000000000ull;
constexpr float AT_LN2 = 0.69314718055994531f;
// A running maximum is raised only when a score exceeds it by this much (in
// powers of two): probabilities then stay below 2^8, which costs nothing in a
// bf16, and accumulators are rarely rescaled.
constexpr float AT_SLACK = 8.f;
// What is kept as an fp16 row's maximum is this much less than it, so that
// probabilities go from 2^7 (2^15 with the slack) down: fp16's steps end at
// 2^-24, and a long flat tail would lose its weight there.  2^-32 of the
// largest is as much as one can be off by then.
template <bool BF16>
constexpr float AT_LIFT = BF16 ? 0.f : 7.f;
constexpr float AT_NONE = -FLT_MAX;  // maximum of no scores

// Bounded wait; once one has run out, every wait gives up at once.  (What
// follows the first try is one function for the whole kernel: warps of
// different roles share an instruction cache, and inlined at every wait it
// would take most of it.)
__device__ __noinline__ bool at_wait_long(uint64_t *bar, uint32_t par, int *gave_up, unsigned *status) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait_sleep(bar, par, 2000u)) {
    if (*(volatile int *)gave_up) return false;
    if (globaltimer_ns() - t0 > AT_LIMIT_NS) {
      flag(status, ST_TIMEOUT);
      *(volatile int *)gave_up = 1;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool at_wait(uint64_t *bar, uint32_t par, int *gave_up, unsigned *status) {
  return mbar_try_wait(bar, par) || at_wait_long(bar, par, gave_up, status);
}

// The same by a whole warp, which has to be together again for the collective
// instructions that follow (tensor-memory loads and stores, barriers).
__device__ __forceinline__ bool at_wait_warp(uint64_t *bar, uint32_t par, int *gave_up, unsigned *status) {
  const bool ok = at_wait(bar, par, gave_up, status);
  __syncwarp();
  return ok;
}

__device__ __forceinline__ void warps_bar(int id, int count) {
  __syncwarp();
  named_bar(id, count);
}

// Whether any of the `count` threads at named barrier `id` says so.
__device__ __forceinline__ bool bar_or(int id, int count, bool v) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(count), "r"((uint32_t)v)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^d (d <= 0) as a product, of which the second is 1 unless 2^d is below what a float
// holds; and x times 2^d.
__device__ __forceinline__ float2 ex2_parts(float d) { return make_float2(ex2(fmaxf(d, -126.f)), ex2(fminf(d + 126.f, 0.f))); }
__device__ __forceinline__ float times_ex2(float x, float d) {
  const float2 f = ex2_parts(d);
  return x * f.x * f.y;
}

// Column sums (MAX: maxima) over a warp of W = 16 or 32 values a lane: lane i
// ends with column i mod W.  Each step sends away the half of the columns
// that the lane will not own, so it takes W - 1 shuffles (and one more for
// 16 columns) where a butterfly for each column takes 5 W.
template <int W, bool MAX>
__device__ __forceinline__ float warp_columns(float v[W]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int s = W / 2; s > 0; s >>= 1) {
    const bool up = lane & s;
#pragma unroll
    for (int i = 0; i < s; ++i) {
      const float keep = up ? v[i + s] : v[i], send = up ? v[i] : v[i + s];
      const float got = __shfl_xor_sync(0xffffffffu, send, s);
      v[i] = MAX ? fmaxf(keep, got) : keep + got;
    }
  }
  if (W == 16) {
    const float got = __shfl_xor_sync(0xffffffffu, v[0], 16);
    v[0] = MAX ? fmaxf(v[0], got) : v[0] + got;
  }
  return v[0];
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// Two floats as 16-bit ones, a in the low half.
template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  if (BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
  }
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&v);
}

// Whether either 16-bit float of a word is an infinity or NaN.
template <bool BF16>
__device__ __forceinline__ bool not_finite2(uint32_t w) {
  constexpr uint32_t M = BF16 ? 0x7F80u : 0x7C00u;
  return (w & M) == M || (w & (M << 16)) == (M << 16);
}

// Bits [lo, hi) of a word.
__device__ __forceinline__ uint32_t bits(int lo, int hi) {
  const uint32_t below = hi >= 32 ? 0xffffffffu : hi > 0 ? (1u << hi) - 1u : 0u;
  return lo >= 32 ? 0u : lo > 0 ? below & ~((1u << lo) - 1u) : below;
}

// Where the x-th 16-byte word that a lane takes of its key's row is: the lanes
// of a warp, a row each, begin at different words, so that they meet in
// different banks (which word is which does not matter to the callers).
__device__ __forceinline__ uint32_t row_word(int x, int lane) { return x / 8 * (AT_KEYS * 128) + ((x ^ lane) & 7) * 16; }

// Whether any of a key's 16-bit floats is an infinity or NaN: the largest
// magnitude tells.
template <bool BF16, int WORDS>
__device__ __forceinline__ bool not_finite_row(const uint8_t *row, int lane) {
  uint32_t top = 0;
#pragma unroll
  for (int x = 0; x < WORDS; ++x) {
    const uint4 w = *reinterpret_cast<const uint4 *>(row + row_word(x, lane));
    top = __vimax3_u16x2(top, w.x & 0x7fff7fffu, w.y & 0x7fff7fffu);
    top = __vimax3_u16x2(top, w.z & 0x7fff7fffu, w.w & 0x7fff7fffu);
  }
  constexpr uint32_t LEAST = BF16 ? 0x7F80u : 0x7C00u;
  return (top & 0xffffu) >= LEAST || (top >> 16) >= LEAST;
}

// Tiles [begin, end) that tokens first .. first + n - 1 of a request see: one
// at least, so that a block of tokens that sees no key is still written.
__device__ __forceinline__ void tile_range(const Span &s, int first, int n, int window, int &begin, int &end) {
  const int p = s.pos0 + first, lo = window && p + 1 > window ? p + 1 - window : 0;
  begin = lo / AT_KEYS;
  end = max(begin + 1, (p + n + AT_KEYS - 1) / AT_KEYS);
}

// What an item is and what it costs.
struct Plan {
  int tpb;   // tokens
  int wide;  // more tokens than this, and a tile counts twice
  int item;  // units that an item costs besides its tiles
  __device__ __forceinline__ int shift(int n) const { return n > wide; }
  __device__ __forceinline__ int64_t length(int begin, int end, int n) const { return ((int64_t)(end - begin) << shift(n)) + item; }
};

// Length on the line of one key head's items of a request.
__device__ __forceinline__ int64_t request_line(const Span &s, const Plan &p, int window) {
  int64_t sum = 0;
  for (int f = 0; f < s.n; f += p.tpb) {
    const int n = min(p.tpb, s.n - f);
    int b, e;
    tile_range(s, f, n, window, b, e);
    sum += p.length(b, e, n);
  }
  return sum;
}

// Where a block's stretch of the line begins (request and its span, key head,
// block of rows, place in the item), and its length.
struct Start {
  int r, h, b, at;
  int64_t left;
  Span sp;
};

// a / b and the rest; most lines are short, and a 64-bit division takes
// hundreds of cycles.
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b, int64_t &rest) {
  if (((uint64_t)a | (uint64_t)b) >> 32) {
    const int64_t q = a / b;
    rest = a - q * b;
    return q;
  }
  const uint32_t q = (uint32_t)a / (uint32_t)b;
  rest = (uint32_t)a - q * (uint32_t)b;
  return q;
}

// The first request of a thread that find_start() gives `R` requests in turn,
// loaded ahead of it.
template <int THREADS>
__device__ __forceinline__ RawSpan first_request(const AttnArgs &a) {
  const int per = (a.R + THREADS - 1) / THREADS, r0 = threadIdx.x * per;
  return r0 < a.R ? request_raw(a.cu, a.seq, r0) : RawSpan{0, 0, 0};
}

// By all THREADS threads; *out is in shared memory and valid after the
// caller's next barrier.
template <int THREADS>
__device__ __forceinline__ void find_start(const AttnArgs &a, const RawSpan &raw0, const Plan &p, Start *out, int64_t *part) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.R + THREADS - 1) / THREADS, r0 = min(a.R, tid * per), r1 = min(a.R, r0 + per);
  bool bad = false;
  Span sp0 = request_span(raw0, a.T, a.max_new, a.max_seq, bad);
  const int64_t line0 = r0 < r1 ? request_line(sp0, p, a.window) : 0;
  int64_t mine = line0;
  for (int r = r0 + 1; r < r1; ++r)
    mine += request_line(request_span(a.cu, a.seq, r, a.T, a.max_new, a.max_seq, bad), p, a.window);
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) part[warp] = incl;
  __syncthreads();
  int64_t before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += part[w];
    total += part[w];
  }
  total *= a.G;
  before *= a.G;
  // no stretch is shorter than an item's overhead and a unit: with little to
  // do the first blocks have a tile each (or two that count once)
  const int64_t c = blockIdx.x, blocks = gridDim.x, least = p.item + 1;
  int64_t s = min(c * least, total), e = min((c + 1) * least, total);
  if (total >= blocks * least) {
    int64_t rest;
    const int64_t share = divide(total, blocks, rest);  // the first `rest` blocks have one more
    s = c * share + min(c, rest);
    e = s + share + (c < rest);
  }
  if (tid == 0) out->left = e - s;
  if (s >= before && s < before + mine * a.G) {
    int64_t off = s - before;
    Span sp = sp0;
    int64_t line = line0;
    for (int r = r0; r < r1; ++r) {
      if (r > r0) {
        sp = request_span(a.cu, a.seq, r, a.T, a.max_new, a.max_seq, bad);
        line = request_line(sp, p, a.window);
      }
      if (off >= line * a.G) {
        off -= line * a.G;
        continue;
      }
      out->r = r;
      out->sp = sp;
      out->h = (int)divide(off, line, off);
      int b = 0, t0, t1;
      for (;; ++b) {
        const int n = min(p.tpb, sp.n - b * p.tpb);
        tile_range(sp, b * p.tpb, n, a.window, t0, t1);
        const int64_t len = p.length(t0, t1, n);
        if (off < len) break;
        off -= len;
      }
      out->b = b;
      out->at = (int)off;
      break;
    }
  }
  if (bad && blockIdx.x == 0) flag(a.status, ST_PAGING);
}

// The segments of a block's stretch, in order: runs of tiles of one item
// (none of them empty).  An item's places on the line are its overhead and
// then its tiles'; a tile is the block's whose stretch has its first place.
struct Segments {
  Plan p;
  int r, h, b, at, begin, end, tile, count, index;
  int64_t left;
  Span sp;
  // of the segment: its first token in the request, its tokens
  int first, n;

  __device__ __forceinline__ void init(const AttnArgs &a, const Plan &plan, const Start &s) {
    p = plan;
    r = s.r; h = s.h; b = s.b; at = s.at; left = s.left;
    index = 0;
    count = 0;
    if (left > 0) {
      sp = s.sp;
      item(a);
      if (!count) advance(a);
    }
  }
  // The tiles of the current item from place `at` on, as far as the stretch goes.
  __device__ __forceinline__ void item(const AttnArgs &a) {
    first = b * p.tpb;
    n = min(p.tpb, sp.n - first);
    tile_range(sp, first, n, a.window, begin, end);
    auto tiles = [&](int64_t place) {  // that begin before it
      const int sh = p.shift(n);
      return (int)((max(place - p.item, (int64_t)0) + sh) >> sh);
    };
    const int done = tiles(at);
    tile = begin + done;
    count = tiles(min(at + left, p.length(begin, end, n))) - done;
  }
  __device__ __forceinline__ bool has_start() const { return tile == begin; }
  __device__ __forceinline__ bool has_end() const { return tile + count == end; }
  __device__ __forceinline__ void next(const AttnArgs &a) {
    ++index;
    advance(a);
  }
  __device__ __forceinline__ void advance(const AttnArgs &a) {
    do {
      left -= p.length(begin, end, n) - at;
      at = 0;
      count = 0;
      if (left <= 0) return;
      if (++b * (int64_t)p.tpb >= sp.n) {
        b = 0;
        if (++h == a.G) {
          h = 0;
          bool bad = false;
          do {
            if (++r >= a.R) {  // lengths that changed under the kernel
              left = 0;
              return;
            }
            sp = request_span(a.cu, a.seq, r, a.T, a.max_new, a.max_seq, bad);
          } while (sp.n == 0);
        }
      }
      item(a);
    } while (!count);
  }
};

// A segment as one warp of a block publishes it to the others, in shared
// memory; count 0 ends the stretch.  A ring of them: `full` is the
// publisher's, `empty` has an arrival of every reading warp.
constexpr int AT_SEGS = 8;
struct Seg {
  int r, h, b, tile, count, first, n, pos0, t0, flags;
};
constexpr int SEG_START = 1, SEG_END = 2, SEG_LATER = 4;  // has the item's first tile, its last; is not the stretch's first
struct SegRing {
  Seg seg[AT_SEGS];
  uint64_t full[AT_SEGS], empty[AT_SEGS];
  __device__ __forceinline__ void init(int i, int readers) {
    mbar_init(&full[i], 1);
    mbar_init(&empty[i], readers);
  }
  // By one whole warp; the k-th of the stretch.
  __device__ __forceinline__ void put(int k, const Segments &s, bool ok, int *gave_up, unsigned *status) {
    const int i = k % AT_SEGS;
    if ((threadIdx.x & 31) == 0) {
      if (k >= AT_SEGS) at_wait(&empty[i], (k / AT_SEGS & 1) ^ 1, gave_up, status);
      Seg &g = seg[i];
      g.r = s.r; g.h = s.h; g.b = s.b; g.tile = s.tile; g.first = s.first; g.n = s.n;
      g.pos0 = s.sp.pos0; g.t0 = s.sp.t0;
      g.count = ok ? s.count : 0;
      g.flags = (s.has_start() ? SEG_START : 0) | (s.has_end() ? SEG_END : 0) | (s.index ? SEG_LATER : 0);
      mbar_arrive(&full[i]);
    }
    __syncwarp();
  }
  // Readers wait for the publisher alone, whatever else has run out: it ends
  // the stretch by itself then, at the same segment for all of them.
  __device__ __forceinline__ const Seg &get(int k, unsigned *status) {
    int never = 0;
    for (int turns = 0; turns < 8 && !at_wait(&full[k % AT_SEGS], k / AT_SEGS & 1, &never, status); ++turns) never = 0;
    return seg[k % AT_SEGS];
  }
  __device__ __forceinline__ void done(int k) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&empty[k % AT_SEGS]);
  }
};

// Pieces: two a block, described by (first token, tokens, key head, flags),
// with `rows` rows of DP sums, and each row's maximum and sum of
// probabilities.
constexpr int PIECE_USED = 1, PIECE_START = 2, PIECE_END = 4;
struct Pieces {
  int4 *what;     // [2 blocks]
  float *sums;    // [2 blocks][rows][DP]
  float2 *stats;  // [2 blocks][rows]: maximum, sum
};
__host__ __device__ inline size_t pieces_bytes(int blocks, int rows, int dp) {
  const size_t n = 2 * (size_t)blocks;
  return (n * 16 + 255) / 256 * 256 + n * rows * (dp * 4 + 8);
}
inline Pieces pieces_of(void *ws, int blocks, int rows, int dp) {
  const size_t n = 2 * (size_t)blocks;
  Pieces p;
  p.what = (int4 *)ws;
  p.sums = (float *)((char *)ws + (n * 16 + 255) / 256 * 256);
  p.stats = (float2 *)(p.sums + n * rows * dp);
  return p;
}

// The pieces of an item that several blocks share, joined in the order of its
// keys: block x looks at the piece that block x of the attention began and did
// not end (the item's further pieces are the following blocks' first ones).
// Bound by latency: where there are few pieces a warp joins a row; where there
// are many (one request's long sequence under one key head is shared by all
// blocks) the eight warps of a block share a row's pieces, and then their
// results (152 pieces of 100,000 keys: 77 us with a warp a row, 15 us so,
// from a cold cache; with 2 to 4 pieces a row a shared form's warps idle: 17
// requests of 3 to 666 tokens 76 us with a warp a row, 114 shared).
constexpr int JOIN_WARPS = 8, JOIN_FEW = 8, JOIN_BLOCKS = 32;
// APART: maxima are not the weights' own, so that a sum may be large for a
// maximum far below the others (attention8_decode.cu).
template <int DP, bool BF16, bool APART>
__global__ void __launch_bounds__(JOIN_WARPS * 32) attention_join_kernel(const AttnArgs a, const Pieces p, int rows, int tok) {
  __shared__ float2 part_stats[JOIN_WARPS];
  __shared__ float part_sums[JOIN_WARPS][DP];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, block = blockIdx.x, blocks = gridDim.x;
  constexpr int PER = DP / 32;
  auto scaled = [](float x, float d, float f) { return APART ? times_ex2(x, d) : x * f; };  // a sum times f = 2^d
  const int4 w0 = p.what[2 * block], w1 = p.what[2 * block + 1];
  const int own = lane && block + lane < blocks ? p.what[2 * (block + lane)].w : PIECE_END;  // the lane's block's first piece
  auto begun = [](const int4 &w) { return (w.w & (PIECE_USED | PIECE_START | PIECE_END)) == (PIECE_USED | PIECE_START); };
  const bool second = begun(w1);
  if (!second && !begun(w0)) return;
  const int4 w = second ? w1 : w0;
  // how many pieces: up to the block whose first piece ends the item
  unsigned ends = __ballot_sync(0xffffffffu, lane && (own & PIECE_END));
  int n = ends ? __ffs(ends) : 32;
  for (int c = block + 32; !ends; c += 32) {
    const int e = c + lane < blocks ? p.what[2 * (c + lane)].w : PIECE_END;
    ends = __ballot_sync(0xffffffffu, e & PIECE_END);
    n += ends ? __ffs(ends) : 32;
  }
  n = min(n, blocks - block);
  const bool shared = n > JOIN_FEW;
  const int first = shared ? blockIdx.y : blockIdx.y * JOIN_WARPS + warp, step = gridDim.y * (shared ? 1 : JOIN_WARPS);
  // pieces begin, begin + stride, ...
  const int begin = shared ? warp : 0, stride = shared ? JOIN_WARPS : 1;
  for (int row = first; row < rows; row += step) {
    // rows in tiles of 128, each of `tok` tokens' g heads
    const int in_tile = row % 128, token = row / 128 * tok + in_tile / a.g;
    if (in_tile >= tok * (int64_t)a.g || token >= w.y) continue;
    auto piece = [&](int i) { return (int64_t)(2 * (block + i) + (i == 0 && second)) * rows + row; };
    const int mine = (n - begin + stride - 1) / stride;
    float m = AT_NONE, l = 0.f, o[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) o[i] = 0.f;
    for (int i0 = 0; i0 < mine; i0 += 32) {
      float2 st = make_float2(AT_NONE, 0.f);
      if (i0 + lane < mine) st = p.stats[piece(begin + (i0 + lane) * stride)];
      float to = fmaxf(m, st.x);
#pragma unroll
      for (int i = 16; i > 0; i >>= 1) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, i));
      const float keep = ex2(m - to), f = ex2(st.x - to), lf = scaled(st.y, st.x - to, f);
      l = scaled(l, m - to, keep);
      m = to;
#pragma unroll
      for (int i = 0; i < PER; ++i) o[i] *= keep;
      const int k = min(32, mine - i0);
#pragma unroll 8
      for (int i = 0; i < k; ++i) {
        const float fi = __shfl_sync(0xffffffffu, f, i);
        l += __shfl_sync(0xffffffffu, lf, i);
        const float *src = p.sums + piece(begin + (i0 + i) * stride) * DP + PER * lane;
#pragma unroll
        for (int x = 0; x < PER; x += 2) {
          const float2 v = *reinterpret_cast<const float2 *>(src + x);
          o[x] = fmaf(v.x, fi, o[x]);
          o[x + 1] = fmaf(v.y, fi, o[x + 1]);
        }
      }
    }
    if (shared) {
      if (lane == 0) part_stats[warp] = make_float2(m, l);
#pragma unroll
      for (int i = 0; i < PER; ++i) part_sums[warp][PER * lane + i] = o[i];
      __syncthreads();
      if (warp == 0) {
        for (int v = 1; v < JOIN_WARPS; ++v) {
          const float2 st = part_stats[v];
          const float to = fmaxf(m, st.x), keep = ex2(m - to), f = ex2(st.x - to);
          l = scaled(l, m - to, keep) + scaled(st.y, st.x - to, f);
#pragma unroll
          for (int i = 0; i < PER; ++i) o[i] = o[i] * keep + part_sums[v][PER * lane + i] * f;
          m = to;
        }
      }
      __syncthreads();
      if (warp) continue;
    }
    const int64_t t = w.x + token;
    const int h = w.z * a.g + in_tile % a.g;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint16_t *out = a.out + t * a.os + (int64_t)h * a.D + PER * lane;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (PER * lane + i < a.D) out[i] = (uint16_t)pack16<BF16>(o[i] * inv, 0.f);
    if (a.lse && lane == 0) a.lse[t * a.H + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * AT_LN2;
  }
}

// Behind an attention kernel of `blocks` blocks; its set-up overlaps that kernel's end.
template <int DP, bool BF16, bool APART = false>
cudaError_t launch_join(const AttnArgs &a, const Pieces &p, int blocks, int rows, int tok, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(blocks, std::min(rows, JOIN_BLOCKS));
  cfg.blockDim = dim3(JOIN_WARPS * 32);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attention_join_kernel<DP, BF16, APART>, a, p, rows, tok);
}

// The keys or values as a 4-D map {element, row of a page, head, page} with
// boxes of 64 elements x `rows` rows.  A box that begins at page -1 is
// outside the map: the copy fills it with zeros and reads nothing.
inline bool make_kv_map(CUtensorMap *m, const void *base, const AttnArgs &a, int rows, bool bf16) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  auto stride = [](int64_t n, int64_t s) { return n > 1 ? (cuuint64_t)s * 2 : (cuuint64_t)16; };
  const cuuint64_t dims[4] = {(cuuint64_t)a.D, (cuuint64_t)a.page, (cuuint64_t)a.G, (cuuint64_t)a.n_pages};
  const cuuint64_t strides[3] = {stride(a.page, a.rs), stride(a.G, a.hs), stride(a.n_pages, a.ps)};
  const cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1}, estr[4] = {1, 1, 1, 1};
  return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void *>(base), dims,
            strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            // (a head's row: 256-byte fetches of 128-byte rows would bring the next head's along)
            a.D > 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same in 8 bits: boxes of `dp` elements (a head's row, with zeros behind
// its end) in the swizzle of that many bytes.
inline bool make_kv8_map(CUtensorMap *m, const void *base, const AttnArgs &a, int rows, int dp) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  auto stride = [](int64_t n, int64_t s) { return n > 1 ? (cuuint64_t)s : (cuuint64_t)16; };
  const cuuint64_t dims[4] = {(cuuint64_t)a.D, (cuuint64_t)a.page, (cuuint64_t)a.G, (cuuint64_t)a.n_pages};
  const cuuint64_t strides[3] = {stride(a.page, a.rs), stride(a.G, a.hs), stride(a.n_pages, a.ps)};
  const cuuint32_t box[4] = {(cuuint32_t)dp, (cuuint32_t)rows, 1, 1}, estr[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            dp == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The query rows {element, head, token}: a box is 64 elements of the g heads
// of `tokens` tokens, so that row t * g + i of a tile is head i of token t.
inline bool make_q_map(CUtensorMap *m, const AttnArgs &a, int tokens, bool bf16) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)a.D, (cuuint64_t)a.H, (cuuint64_t)a.T};
  const cuuint64_t strides[2] = {(cuuint64_t)a.D * 2, a.T > 1 ? (cuuint64_t)a.qs * 2 : (cuuint64_t)a.D * a.H * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)a.g, (cuuint32_t)tokens}, estr[3] = {1, 1, 1};
  return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<uint16_t *>(a.q),
            dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows that one copy can take: the largest power of two that divides a page,
// so that a copy never runs over a page's end; at most a tile.
inline int piece_rows(int page) {
  int b = 1;
  while (b < AT_KEYS && page % (2 * b) == 0) b *= 2;
  return b;
}

// Maps of keys or values: for boxes of `rows` rows, and of twice as many for
// two runs that lie together in a page.  Only pages of an odd number of 8-row
// runs use the second: an SM's copies run at about 50 cycles a box, which
// boxes of 8 rows do not keep up with memory at and boxes of 16 do (64
// requests of 200 to 8200 keys, 8 key heads of 128: 191 us with pages of 24 in
// single runs, 177 in pairs, 177 with pages of 16).  The chunk kernel takes
// single runs: it reads less, and the code for pairs slows it (17 requests of 3
// to 666 tokens: 82 us without, 93 with).
struct KvMaps {
  CUtensorMap one, two;
};
constexpr int AT_PAIR_ROWS = 8;
inline bool make_kv_maps(KvMaps *m, const void *base, const AttnArgs &a, int rows, bool bf16) {
  if (!make_kv_map(&m->one, base, a, rows, bf16)) return false;
  if (rows == AT_PAIR_ROWS && a.page > rows) return make_kv_map(&m->two, base, a, 2 * rows, bf16);
  m->two = m->one;
  return true;
}
inline bool make_kv8_maps(KvMaps *m, const void *base, const AttnArgs &a, int rows, int dp) {
  if (!make_kv8_map(&m->one, base, a, rows, dp)) return false;
  if (rows == AT_PAIR_ROWS && a.page > rows) return make_kv8_map(&m->two, base, a, 2 * rows, dp);
  m->two = m->one;
  return true;
}

// The copies of one tile's keys (and later its values): lane i < 128 / rows
// has the i-th run of rows, its page and its first row there.  Runs that no
// token of the segment sees, and pages that are none, are filled with zeros.
// find() starts the load of the page ids, copy() uses them: the producers
// look a tile ahead, so that no tile waits for its page ids.
struct TileRuns {
  int page, row;
  bool sees;
  // (r, n tokens from position p on: of the segment)
  __device__ __forceinline__ void find(const AttnArgs &a, int r, int p, int n, int tile, int rows) {
    const int lane = threadIdx.x & 31, j = tile * AT_KEYS + lane * rows;
    const int lo = a.window ? p + 1 - a.window : 0;
    sees = lane * rows < AT_KEYS && j < p + n && j + rows > lo;
    if (sees) {
      const int col = j / a.page;
      row = j - col * a.page;
      page = a.table[r * a.table_stride + col];
    }
  }
  __device__ __forceinline__ void find(const AttnArgs &a, const Segments &s, int tile, int rows) {
    find(a, s.r, s.sp.pos0 + s.first, s.n, tile, rows);
  }
  // (E8: 8-bit elements, a row of DP bytes in one box)
  template <int DP, bool PAIRS, bool E8 = false>
  __device__ __forceinline__ void copy(const AttnArgs &a, uint8_t *slot, const CUtensorMap *one, const CUtensorMap *two, int head, int rows,
                                       uint64_t *full, bool &bad) const {
    const int lane = threadIdx.x & 31;
    if (lane == 0) mbar_arrive_expect_tx(full, AT_KEYS * DP * (E8 ? 1 : 2));
    __syncwarp();
    const bool there = sees && page >= 0 && page < a.n_pages;
    bad = bad || (sees && !there);
    bool pair = false, paired = false;  // takes the next lane's run along; is taken along
    if (PAIRS && rows == AT_PAIR_ROWS && a.page > AT_PAIR_ROWS) {
      const bool next = __shfl_down_sync(0xffffffffu, there, 1);  // (past the tile's last run: not there)
      pair = there && next && !(row & AT_PAIR_ROWS) && row + 2 * AT_PAIR_ROWS <= a.page;
      paired = __shfl_up_sync(0xffffffffu, pair, 1) && lane > 0;
    }
    if (lane * rows < AT_KEYS && !paired) {
      const CUtensorMap *map = pair ? two : one;
#pragma unroll
      for (int x = 0; x < DP; x += E8 ? DP : 64)
        tma_load_4d(slot + x / 64 * (AT_KEYS * 128) + lane * rows * (E8 ? DP : 128), map, x, there ? row : 0, head, there ? page : -1, full);
    }
    __syncwarp();
  }
};

}  // namespace
}  // namespace dsm
