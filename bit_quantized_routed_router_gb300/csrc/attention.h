// Launchers of the attention over pages (internal).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace dsm {

struct AttnArgs {
  const uint16_t *k, *v;
  int64_t n_pages, ps, rs, hs;  // cache strides in elements: page, row, head
  const int32_t *table;
  int width;
  int64_t table_stride;
  const uint16_t *q;
  int64_t qs;
  const int32_t *cu, *seq;
  int T, R, max_new;
  uint16_t *out;
  int64_t os;
  float *lse;
  int H, G, g, D, page, window;  // query heads, key heads, query heads a key head
  float scale_log2;              // scale * log2(e): the softmax works in powers of two
  int64_t max_seq;               // keys that the table has columns for
  unsigned *status;
};

// Query rows a key head up to which the decode kernel serves: its work goes
// with the rows, the chunk kernel's with tiles of 128 of them.  64 requests of
// 200 to 8200 keys, 4 key heads, at 16, 24 and 32 rows: decode 95, 100 and
// 100 us for head_dim 128, chunk 102, 103 and 104; for 64 decode 61, 72 and 72,
// chunk 62, 62 and 63, but with few requests decode is ahead there as well (24
// rows: 4 requests of 1000 to 3000 keys 14 and 16, 3 of 60,000 to 90,000 100
// and 105).  A 64-column form of it was behind at 40 rows (284 us for 128,
// chunk 213, with twice the heads) and is left out.
constexpr int64_t AD_MAX_ROWS = 32;
size_t attention_decode_workspace(int64_t rows, int blocks);
cudaError_t launch_attention_decode(const AttnArgs &a, bool bf16, void *ws, cudaStream_t s);
size_t attention_chunk_workspace(int blocks);
cudaError_t launch_attention_chunk(const AttnArgs &a, bool bf16, void *ws, cudaStream_t s);
cudaError_t launch_attention_generic(const AttnArgs &a, bool bf16, cudaStream_t s);

}  // namespace dsm
