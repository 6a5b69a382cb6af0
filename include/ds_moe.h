/* ds_moe: one routed mixture-of-experts layer with 2-bit (Q2_K) or 4-bit
 * (Q4_K) routed experts, computed on one GB300 (sm_103a) GPU.
 *
 * The layer ("Understanding Dwarf Star", 5.3.2 "The MoE Architecture" and
 * 5.3.7 "The MoE Kernel in Metal"):
 *     logits  = x W_router^T (+ bias)                      router, fp32
 *     ids, w  = top-k of logits, w = softmax over the k     selection
 *     y_e(x)  = W_down,e ( SiLU(W_gate,e x) * (W_up,e x) )  SwiGLU expert
 *     out     = y_shared(x) + sum_j w_j y_{ids_j}(x)        combine, fp32
 * with the routed expert matrices stored as Q2_K super-blocks ("Understanding
 * Dwarf Star", 3.3.3 "Q2_K: 2.625 Bits Per Element"): 84 bytes per 256
 * weights along each matrix's input dimension (or Q4_K, below).  Shapes of the DeepSeek V4
 * Flash layer: n_embd 4096, 256 experts, top-6, one shared expert, expert
 * width 2048 ("Understanding Dwarf Star", 2.4.3 shape table).
 *
 * Conventions (the pages' C engine style: int status, 0 = ok, negative =
 * error, plus a caller-supplied error buffer; caller-owned scratch):
 *   - Every pointer is a DEVICE pointer unless the argument says "host".
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream).  Every call is asynchronous on that stream unless stated.
 *   - The library allocates no device memory for a call: the caller owns
 *     every buffer, including the workspace, and nothing is retained after a
 *     call returns.  (Per device it keeps one status word, and
 *     ds_moe_layer_noalloc's static scratch; ds_moe_cache keeps host state.)
 *   - Argument errors are detected on the host before any launch and return
 *     DS_ERR_INVALID_ARG (or DS_ERR_UNSUPPORTED) with a message in err.
 *     Errors a kernel detects (a non-finite weight given to the quantiser,
 *     a corrupted id, a timed-out wait) are recorded in a per-device sticky
 *     status word, read and cleared by ds_moe_sync_status.
 *   - err may be NULL; otherwise up to errlen bytes (NUL-terminated) are
 *     written on failure.
 *   - Calls are thread-safe as long as concurrent calls use distinct
 *     workspaces and outputs.
 *
 * Q2_K super-block (84 bytes, 256 weights):
 *   bytes [0,16)   sub-block s (16 weights each): scale sc_s in the low
 *                  nibble, min m_s in the high nibble
 *   bytes [16,80)  2-bit codes; weight j at byte 16 + j/4, bits 2*(j%4)
 *   bytes [80,82)  d, fp16 little-endian;  bytes [82,84) dmin, fp16
 *   weight j = d*sc_s*q_j - dmin*m_s  (s = j/16)
 * Q4_K super-block (144 bytes, 256 weights; "Understanding Dwarf Star",
 * 2.3.2 "K-Quant Formats": d at 0, dmin at 2, 12 bytes of 6-bit scales and
 * mins at 4, 128 bytes of 4-bit codes at 16, 8 sub-blocks of 32):
 *   bytes [0,2) d, [2,4) dmin, fp16 little-endian
 *   bytes [4,16)   one 96-bit little-endian integer: field i in bits
 *                  [6i, 6i+6); fields 0..7 = sc_s, 8..15 = m_s
 *   bytes [16,144) 4-bit codes; weight j at byte 16 + j/2, low nibble for
 *                  even j
 *   weight j = d*sc_s*q_j - dmin*m_s  (s = j/32)
 * A row of in_dim weights uses ceil(in_dim/256) blocks (zero-padded).
 * Packed expert e = gate [n_ff rows][n_embd] | up [n_ff][n_embd] |
 * down [n_embd rows][n_ff], each row-major in blocks; experts are contiguous
 * in expert order, each ds_moe_expert_bytes_fmt() long; base 16-byte aligned.
 */
#ifndef DS_MOE_H
#define DS_MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  DS_OK = 0,
  DS_ERR_INVALID_ARG = -1,  /* bad pointer, size, alignment or workspace    */
  DS_ERR_UNSUPPORTED = -2,  /* valid but not implemented (e.g. odd n_embd)  */
  DS_ERR_CUDA = -3,         /* a CUDA runtime call failed                    */
  DS_ERR_TIMEOUT = -4,      /* a device wait hit its iteration limit         */
  DS_ERR_DEVICE_CHECK = -5  /* a kernel found invalid data                   */
} ds_status;

typedef enum {
  DS_F32 = 0,
  DS_BF16 = 1,
  DS_F16 = 2 /* attention and its cache only */
} ds_dtype;

/* Storage format of the routed experts. */
typedef enum { DS_Q2_K = 0, DS_Q4_K = 1 } ds_expert_format;

typedef struct {
  int32_t n_embd;       /* D: model width, multiple of 256, <= 8192          */
  int32_t n_expert;     /* E: routed experts, 1..1024                        */
  int32_t n_ff;         /* F: expert width, multiple of 128, <= 8192         */
  int32_t n_ff_shared;  /* Fs: shared expert width, 0 = none, mult. of 128, <= 8192 */
  int32_t top_k;        /* k: 1..min(E, 16)                                  */
  int32_t x_dtype;      /* ds_dtype of x                                     */
  int32_t router_dtype; /* ds_dtype of router_w                              */
  float routed_scale;   /* multiplies the k routing weights (1.0 default)    */
  float logit_scale;    /* multiplies the selected logits before their softmax
                           (the other reading of [UDS] 5.3.5's 1.5 "before
                           softmax"); 1 = plain softmax, 0 is taken as 1; the
                           selection does not depend on it                  */
  int32_t bias_select_only; /* 0: router_bias is part of the logits (selection
                           and weights); 1: it steers the selection only and
                           the weights use the logits without it            */
  int32_t expert_format; /* ds_expert_format of the routed experts (0 = Q2_K) */
} ds_moe_shape;

typedef struct {
  const void *router_w;       /* [E][D] router_dtype, row-major                 */
  const float *router_bias;   /* [E] fp32 added to the logits, or NULL          */
  const uint16_t *shared_gate; /* [Fs][D] bf16 bits (NULL when Fs == 0)        */
  const uint16_t *shared_up;   /* [Fs][D] bf16 bits                             */
  const uint16_t *shared_down; /* [D][Fs] bf16 bits                             */
  const uint8_t *experts;    /* [E] packed experts in expert_format, 16-byte aligned */
} ds_moe_weights;

/* Optional debug outputs of ds_moe_layer (device pointers; NULL fields and a
 * NULL struct are skipped).  All are written in the same stream order. */
typedef struct {
  float *logits;    /* [T][E] router logits incl. bias (fp32)                 */
  int32_t *ids;     /* [T][k] selected experts, descending logit order        */
  float *w;         /* [T][k] routing weights (after routed_scale)            */
  int32_t *counts;  /* [E] tokens per expert                                  */
  int32_t *offsets; /* [E+1] exclusive scan of counts                         */
  int32_t *perm;    /* [T*k] pair t*k+j at position offsets[e]+rank, stable   */
} ds_moe_debug;

/* Bytes of a Q2_K matrix of `rows` rows of `in_dim` weights:
 * rows * ceil(in_dim/256) * 84 ("Understanding Dwarf Star", 3.3.3).
 * Returns 0 for negative sizes. */
size_t ds_moe_q2k_bytes(int64_t rows, int64_t in_dim);

/* Bytes of a Q4_K matrix: rows * ceil(in_dim/256) * 144 ("Understanding
 * Dwarf Star", 2.3.2).  Returns 0 for negative sizes. */
size_t ds_moe_q4k_bytes(int64_t rows, int64_t in_dim);

/* Bytes of one packed routed expert (gate, up and down; "The sparsity that
 * pays for everything else in DwarfStar", "Where the parameters actually
 * are": gate, up and down per expert), Q2_K. */
size_t ds_moe_expert_bytes(int32_t n_embd, int32_t n_ff);

/* The same in a given ds_expert_format; 0 for an unknown format. */
size_t ds_moe_expert_bytes_fmt(int32_t expert_format, int32_t n_embd, int32_t n_ff);

/* Quantise an fp32 matrix w [rows][in_dim] (row-major, device) to Q2_K
 * blocks in out (ds_moe_q2k_bytes(rows, in_dim) bytes, device, 4-byte
 * aligned).  The encoding picks, per super-block, the smallest fp16 dmin and
 * d and the smallest 4-bit mins and scales whose four evenly spaced levels
 * cover each 16-weight sub-block, then rounds each weight to its nearest
 * level, ties upward ("Understanding Dwarf Star", 2.3.5: Q2_K levels are
 * evenly spaced between the block's min and max; 3.3.3 block layout).  Every
 * decision is exact, so the bytes are a pure function of the inputs.
 * Non-finite inputs or |w| > 65504 set DS_ERR_DEVICE_CHECK in the status
 * word and produce an all-zero block. */
int ds_moe_quantize_q2k(const float *w, int64_t rows, int64_t in_dim, uint8_t *out, void *stream,
                        char *err, size_t errlen);

/* Dequantise Q2_K blocks q [rows][ceil(in_dim/256)*84] to fp32
 * out [rows][in_dim]: out = fp32(d*sc*q - dmin*m), i.e. the exact value
 * rounded once ("Understanding Dwarf Star", 2.8.1: weights are rebuilt from
 * the stored scales and mins).  A test and inspection aid. */
int ds_moe_dequantize_q2k(const uint8_t *q, int64_t rows, int64_t in_dim, float *out, void *stream,
                          char *err, size_t errlen);

/* Quantise to Q4_K blocks (ds_moe_q4k_bytes(rows, in_dim) bytes, device,
 * 4-byte aligned).  The same search as for Q2_K with 4-bit codes and 6-bit
 * scales and mins, per 32-weight sub-block: the smallest fp16 dmin with
 * 63*dmin >= max(-min), the smallest m_s <= 63 covering each sub-block's
 * minimum, the smallest fp16 d with 945*d >= max(hi_s + b_s), the smallest
 * sc_s <= 63 with 15*d*sc_s >= hi_s + b_s, then the nearest of the 16 levels,
 * ties upward ("Understanding Dwarf Star", 2.3.2 layout; 2.3.5 evenly spaced
 * levels).  Exact, like the Q2_K quantiser; the same input checks. */
int ds_moe_quantize_q4k(const float *w, int64_t rows, int64_t in_dim, uint8_t *out, void *stream,
                        char *err, size_t errlen);

/* Dequantise Q4_K blocks to fp32: fp32(d*sc*q - dmin*m), rounded once. */
int ds_moe_dequantize_q4k(const uint8_t *q, int64_t rows, int64_t in_dim, float *out, void *stream,
                          char *err, size_t errlen);

/* Workspace bytes ds_moe_layer needs for T tokens of this shape (host call,
 * synchronous).  The workspace must be 256-byte aligned. */
int ds_moe_workspace_bytes(const ds_moe_shape *shape, int64_t T, size_t *bytes, char *err,
                           size_t errlen);

/* One routed MoE layer on T tokens (the equations at the top of this file).
 *   x    [T][D] x_dtype (device), 16-byte aligned
 *   out  [T][D] fp32 (device), 16-byte aligned; fully overwritten
 *   workspace: ds_moe_workspace_bytes bytes, 256-byte aligned, caller-owned;
 *        its contents need no initialisation and are scratch after return
 *   dbg  optional debug outputs (NULL to skip)
 * Tokens are independent: row t of out depends only on row t of x.
 * A NaN router logit is never selected.  When fewer than top_k of a token's
 * logits are numbers (a NaN in its x, say), its remaining picks take expert
 * 0, its row of out is not meaningful, and ds_moe_sync_status reports
 * DS_ERR_DEVICE_CHECK; nothing of such a call carries over into later calls.
 * T == 0 is a no-op.  The kernels that run depend on T and the shape (see
 * ds_moe_layer_path): one token at the instantiated widths with top_k <= 8
 * streams the whole layer through one cooperative kernel; up to four tokens
 * (and one token otherwise) use a three-kernel decode chain, except where
 * the batched kernels below apply; both compute the routed rows as exact
 * integer dots on 16-bit fixed-point activations.  4..16 tokens with Q2_K
 * experts, bf16 x and router and n_embd, n_ff, n_ff_shared multiples of
 * 1024 run the batched decode kernels (the same integer dots; the shared
 * expert on the tensor cores with exact bf16 products).  Larger batches with bf16 x and router and n_embd, n_ff
 * multiples of 1024 (Q4_K experts: from five tokens) run the expert FFNs as
 * grouped tcgen05 GEMMs with fp16 operands (dequantised weights and
 * activations rounded once to fp16; an |x| or intermediate above 65504 is
 * saturated and reported by ds_moe_sync_status as DS_ERR_DEVICE_CHECK);
 * every other case uses the grouped dequantising GEMV path with fp32
 * arithmetic. */
int ds_moe_layer(const ds_moe_shape *shape, const ds_moe_weights *weights, const void *x, int64_t T,
                 float *out, void *workspace, size_t workspace_bytes, const ds_moe_debug *dbg,
                 void *stream, char *err, size_t errlen);

/* ds_moe_layer with x and out in HOST memory (pinned for best speed): the
 * host-to-device copy of x and the device-to-host copy of out are issued on
 * `stream` around the layer, using the workspace for the device copies
 * (ds_moe_workspace_bytes covers them).  When the one-token kernel serves
 * the call (T == 1 at its widths) and the device can address both buffers
 * (pinned memory), no copy operation is issued: the router grid reads x in
 * host memory and keeps a device copy in the workspace for the streaming
 * kernel, which writes out straight into host memory.  Returns after
 * enqueueing; the caller synchronises the stream before reading out. */
int ds_moe_layer_hostio(const ds_moe_shape *shape, const ds_moe_weights *weights,
                        const void *x_host, int64_t T, float *out_host, void *workspace,
                        size_t workspace_bytes, void *stream, char *err, size_t errlen);

/* A stack of n_layers blocks, each  x <- x + layer_l(bf16(RMSNorm(x)))  with
 * RMSNorm(x) = x / sqrt(mean(x^2) + eps) and unit gain (pages: every layer
 * applies RMSNorm and a residual connection).  x [T][D] fp32 (device) is the
 * residual stream, updated in place.  layers: host array of n_layers weight
 * sets; shape->x_dtype must be DS_BF16.  Workspace as for ds_moe_layer. */
int ds_moe_stack(const ds_moe_shape *shape, const ds_moe_weights *layers, int32_t n_layers,
                 float *x, int64_t T, float eps, void *workspace, size_t workspace_bytes,
                 void *stream, char *err, size_t errlen);

/* ds_moe_stack with a format per layer ("q2-q4" mixed stacks: most layers
 * Q2_K, the last few Q4_K).  formats: host array of n_layers
 * ds_expert_format values that replace shape->expert_format for each layer,
 * or NULL (every layer as the shape says).  The workspace must hold
 * ds_moe_workspace_bytes of the shape with expert_format = DS_Q2_K when any
 * layer is Q2_K, else with DS_Q4_K.  A bad format entry returns
 * DS_ERR_INVALID_ARG before any launch. */
int ds_moe_stack_mixed(const ds_moe_shape *shape, const ds_moe_weights *layers,
                       const int32_t *formats, int32_t n_layers, float *x, int64_t T, float eps,
                       void *workspace, size_t workspace_bytes, void *stream, char *err,
                       size_t errlen);

/* ds_moe_layer for callers that cannot allocate device memory where they
 * call the layer: a plugin or extension inside a host program whose own
 * allocator owns all device memory, or a real-time loop that must not take
 * cudaMalloc's implicit device-wide synchronisation.  It takes no workspace:
 * its scratch is a static 64 MiB device array inside this library, allocated
 * on each GPU when the library is loaded there and held until the process
 * exits.  The pages have no counterpart to this entry point.
 *   x, T, out, stream, err: as for ds_moe_layer (no debug outputs); the
 *   arguments are validated in the same order, so T == 0 with bad weights
 *   is rejected as ds_moe_layer rejects it.
 *   Rejects, with DS_ERR_INVALID_ARG and a message, any T whose
 *   ds_moe_workspace_bytes exceeds 64 MiB (at the 4096/256/6/2048 shape the
 *   limit is reached at about 200 tokens; from 17 tokens the tensor-core
 *   path's scratch includes a 16.8 MB fp16 copy of the shared down matrix).
 *   Allocates nothing: no cudaMalloc, no cudaFree.
 *   The first call on a device looks up the array's device address with
 *   that device current; make that first call before any stream capture.
 *   Every call reuses the same array and leaves its contents behind; the
 *   call clears what must start at zero.  Calls that overlap on the GPU
 *   (other streams or threads) race on the array: serialise them. */
int ds_moe_layer_noalloc(const ds_moe_shape *shape, const ds_moe_weights *weights, const void *x,
                         int64_t T, float *out, void *stream, char *err, size_t errlen);

/* Expert residency beyond device memory ("The sparsity that pays for
 * everything else in DwarfStar", "Page the experts off the SSD" and "The
 * cache is never allowed to become a correctness structure": routed experts
 * are paged in through a cache, and the output does not depend on what the
 * cache holds).  Here every routed expert of a layer has a copy in host
 * memory the device can address (pinned and mapped by cudaHostAlloc,
 * registered by cudaHostRegister, or the memory of a coherent host such as
 * Grace, read over NVLink-C2C), and a caller-owned pool of device slots holds
 * some of them.
 *   slot          [E] int32 (device): the cache slot of expert e, or -1
 *   cache         device: slots of ds_moe_expert_bytes_fmt() bytes each,
 *                 16-byte aligned (may be NULL when no slot is in use)
 *   experts_host  HOST pointer to the layer's E packed experts (the layout of
 *                 ds_moe_weights.experts), 16-byte aligned */
typedef struct {
  const int32_t *slot;
  const uint8_t *cache;
  const uint8_t *experts_host;
} ds_moe_residency;

/* ds_moe_layer with the routed experts read through a residency view: each
 * expert from its cache slot, or from the host copy (ordinary loads) when it
 * has none; weights->experts is ignored and may be NULL.  The same kernels
 * run on the same bytes wherever an expert lives, so the output is
 * bit-identical for every slot table.  Kernels: as ds_moe_layer for up to
 * four tokens at the instantiated widths (the streaming kernel, the
 * three-kernel chain), the grouped dequantising GEMV path otherwise
 * (ds_moe_layer_path_resident).  Errors as ds_moe_layer, and
 * DS_ERR_INVALID_ARG for a missing slot table or a host copy the device
 * cannot address. */
int ds_moe_layer_resident(const ds_moe_shape *shape, const ds_moe_weights *weights,
                          const ds_moe_residency *residency, const void *x, int64_t T, float *out,
                          void *workspace, size_t workspace_bytes, const ds_moe_debug *dbg, void *stream,
                          char *err, size_t errlen);

/* A cache of routed experts for n_layers layers of one shape (opaque host
 * object).  experts_host: host array of n_layers host pointers, each a
 * layer's E packed experts in device-addressable host memory (as for
 * ds_moe_residency).  slots: caller-owned device buffer of n_slots experts
 * (ds_moe_expert_bytes_fmt() bytes each, 16-byte aligned; the byte budget of
 * the cache); tables: caller-owned device buffer of n_layers * E int32 slot
 * tables, set here (synchronously) to "every expert in host memory".  With
 * tables == NULL the object only plans (ds_moe_cache_record; no device
 * memory is touched).  The library allocates no device memory; the object
 * itself is host memory, freed by ds_moe_cache_destroy. */
typedef struct ds_moe_cache ds_moe_cache;
int ds_moe_cache_create(const ds_moe_shape *shape, int32_t n_layers, const void *const *experts_host,
                        void *slots, int64_t n_slots, int32_t *tables, ds_moe_cache **cache, char *err,
                        size_t errlen);
void ds_moe_cache_destroy(ds_moe_cache *cache);

/* One layer through the cache: ds_moe_layer_resident with this layer's slot
 * table, then (after synchronising the stream to read which experts the call
 * used) the experts it missed are copied on `stream` into free slots or the
 * least recently used slots that this call did not use, and the slot tables
 * are updated on `stream` for the calls that follow.  The output does not
 * depend on the cache's contents.  Not for use inside stream capture (it
 * synchronises the stream). */
int ds_moe_cache_layer(ds_moe_cache *cache, int32_t layer, const ds_moe_weights *weights, const void *x, int64_t T,
                       float *out, void *workspace, size_t workspace_bytes, void *stream, char *err,
                       size_t errlen);

/* The cache policy alone, on the host: record that a call of `layer` used
 * the experts with counts[e] > 0 (host array [E]).  Hits refresh their
 * slots; each miss takes a free slot, else the least recently used slot not
 * used by this call (none: the expert stays in host memory).  fills (host,
 * optional, 2 * E int32) receives (slot, expert) pairs of the copies to make,
 * n_fills their number.  ds_moe_cache_layer does this after every call. */
int ds_moe_cache_record(ds_moe_cache *cache, int32_t layer, const int32_t *counts, int32_t *fills,
                        int32_t *n_fills);
/* *slot = the slot of expert `expert` of `layer` (host mirror of the
 * tables), or -1 when it is in host memory.  DS_ERR_INVALID_ARG for a bad
 * cache, layer, expert or NULL slot. */
int ds_moe_cache_slot(const ds_moe_cache *cache, int32_t layer, int32_t expert, int32_t *slot);
/* Counters since creation: experts found in a slot, experts read from host
 * memory, and slots in use. */
int ds_moe_cache_stats(const ds_moe_cache *cache, int64_t *hits, int64_t *misses, int64_t *resident);

/* Which kernels ds_moe_layer runs for T tokens of this shape with this x
 * pointer (host call; nothing is launched).  Returns one of the DS_PATH_*
 * values, or DS_ERR_INVALID_ARG for a shape ds_moe_layer would reject. */
enum {
  DS_PATH_NONE = 0,          /* T == 0 */
  DS_PATH_STREAM = 1,        /* one token: router kernel + one cooperative streaming kernel */
  DS_PATH_DECODE3 = 2,       /* T <= 4 (2..3, or 4 where the batched kernels do not apply): router,
                                gate/up and down kernels chained */
  DS_PATH_GROUPED_GEMV = 3,  /* route kernels + grouped dequantising GEMVs + combine */
  DS_PATH_TENSOR_CORE = 4,   /* route kernels + grouped tcgen05 GEMMs + combine */
  DS_PATH_BATCHED_DECODE = 5 /* 4..16 tokens: router kernel + batched decode kernels (integer
                                routed dots, shared expert on the tensor cores) */
};
int ds_moe_layer_path(const ds_moe_shape *shape, int64_t T, const void *x);
/* The same for ds_moe_layer_resident. */
int ds_moe_layer_path_resident(const ds_moe_shape *shape, int64_t T);

/* Synchronise `stream`, then read and clear this device's sticky status
 * word (one atomic exchange on the device, so bits that kernels on other
 * streams set meanwhile are not lost: they are reported by the next call).
 * Returns DS_OK, DS_ERR_TIMEOUT or DS_ERR_DEVICE_CHECK (with a message
 * naming the check), or DS_ERR_CUDA if the stream itself failed. */
int ds_moe_sync_status(void *stream, char *err, size_t errlen);

/* ------------------------------------------------------------------------
 * One serving step around the layer: pages for the new tokens, their keys
 * and values into the pages, attention over the pages, and the check of
 * drafted tokens.  (The pages describe the engine's key-value cache and its
 * speculative decoding only in outline; these entry points are this
 * library's own.)
 *
 * A request r has context_lens[r] tokens whose keys and values are in pages,
 * and new_lens[r] new ones.  Its key at position j is in page
 * block_table[r][j / page_size], row j % page_size; a slot is
 * page * page_size + row.  The new tokens of all requests follow one another
 * ("ragged"): those of request r are tokens cu_new[r] .. cu_new[r+1]-1, and
 * its sequence, new tokens included, is seq_lens[r] long.
 *
 * Lengths, tables and page ids live on the device, so they are checked there:
 * what is out of range is reported by ds_moe_sync_status
 * (DS_ERR_DEVICE_CHECK), and nothing outside the given buffers is read or
 * written.
 * ---------------------------------------------------------------------- */

/* Pages and places of a step's new tokens, built on the device.
 *   context_lens, new_lens  [n_requests] int32 (n_requests 1..16384; 0: no-op
 *        but for slots, positions, cu_new[0] and n_taken)
 *   free_pages  [n_free] int32, ids of unused pages
 *   block_table [n_requests][table_width] int32, rows table_stride apart: the
 *        first ceil(context/page_size) entries of a row are the request's
 *        pages; the pages that the new tokens begin are written behind them,
 *        taken from free_pages in request order.  Other entries are kept.
 *   slots       [max_tokens] int64 (max_tokens up to 2^24): the slot of each new token, -1 past the
 *        last (a captured step may have room to spare)
 *   positions   [max_tokens] int32: its position in its sequence, -1 past the
 *        last
 *   cu_new      [n_requests+1] int32, seq_lens [n_requests] int32
 *   n_taken     [1] int32: pages taken from free_pages
 * Reported, and still well defined: a length below zero or from 2^30 up
 * counts as zero; new tokens beyond max_tokens are dropped (cu_new and seq_lens say
 * so); a page beyond table_width or beyond n_free is none (table entry -1,
 * where there is one), and the slots of its tokens are -1, as are those in a
 * held page whose entry is negative.  The inputs are not changed (but for
 * the table's new entries), so that the same call again gives the same; no
 * output may share memory with an input.  In a captured graph the addresses,
 * n_requests, n_free, table_width and max_tokens are the capture's; the
 * lengths and the ids are read at each replay.  free_pages is not consumed:
 * before the next step the caller drops its first *n_taken ids, on the device
 * where a graph replays (ids[(i + *n_taken) % n_free], say), and sees to it
 * that no id in use is among those that the step can come to. */
int ds_moe_page_map(const int32_t *context_lens, const int32_t *new_lens, int32_t n_requests, int32_t page_size,
                    const int32_t *free_pages, int32_t n_free, int32_t *block_table, int32_t table_width,
                    int64_t table_stride, int64_t *slots, int32_t *positions, int32_t max_tokens, int32_t *cu_new,
                    int32_t *seq_lens, int32_t *n_taken, void *stream, char *err, size_t errlen);

/* Heads, types and masks of an attention. */
typedef struct {
  int32_t n_head;    /* query heads, a multiple of n_head_kv                  */
  int32_t n_head_kv; /* key and value heads; query head h reads head
                        h / (n_head / n_head_kv)                             */
  int32_t head_dim;  /* 1..128                                               */
  int32_t page_size; /* tokens a page, 1..65536                              */
  int32_t dtype;     /* DS_BF16 or DS_F16: q, the cache, the new keys and
                        values, and out                                      */
  float scale;       /* multiplies q k^T; 0: 1/sqrt(head_dim)                */
  int32_t window;    /* keys that a token sees, itself included; 0: all
                        (sequences are shorter than 2^30)                    */
} ds_moe_attn_shape;

/* Pages of keys and values: element (page, row, head, d) of either is at
 * page * page_stride + row * row_stride + head * head_stride + d, in
 * elements, the last axis dense.  Any order of the axes is fine (pages of
 * rows or of heads; both in one buffer).  The tensor-core attention wants the
 * bases (and q) 16-byte aligned, the strides, head_dim and page_size multiples
 * of 8, and at most 128 query heads a key head; others run on CUDA cores.
 * An append refuses rows that overlap: each stride has to step over all that
 * the smaller ones span. */
typedef struct {
  void *k, *v;
  int64_t n_pages;
  int64_t page_stride, row_stride, head_stride;
} ds_moe_kv_cache;

/* Copies the keys and values of T tokens to their slots: k_new and v_new
 * [T][n_head_kv][head_dim], tokens token_stride and heads head_stride
 * elements apart (so they may be slices of a fused projection).  A slot below
 * zero is none; one beyond the cache is skipped and reported.  Slots have to
 * differ from one another. */
int ds_moe_kv_append(const ds_moe_attn_shape *shape, const ds_moe_kv_cache *cache, const void *k_new,
                     const void *v_new, int64_t token_stride, int64_t head_stride, const int64_t *slots, int64_t T,
                     void *stream, char *err, size_t errlen);

/* Device workspace of ds_moe_paged_attention (host call), for up to
 * n_requests requests, T new tokens and max_new of one request. */
int ds_moe_attention_workspace_bytes(const ds_moe_attn_shape *shape, int32_t n_requests, int64_t T, int32_t max_new,
                                     size_t *bytes, char *err, size_t errlen);

/* Attention of each request's new tokens over its pages (its new keys and
 * values among them: ds_moe_kv_append comes first):
 *     out = sum_j softmax_j(scale q k_j) v_j over the keys j that the token
 *           sees: j <= its position, and with a window j > position - window
 *   q, out      [T][n_head][head_dim], 16-byte aligned or not, tokens
 *               q_stride / out_stride elements apart (heads dense)
 *   lse         [T][n_head] fp32 or NULL: log sum_j exp(scale q k_j)
 *   cu_new, seq_lens, block_table as ds_moe_page_map writes them
 *   max_new     no request has more new tokens than that (more are reported
 *               and dropped: their rows of out are not written)
 * Keys that a token does not see have no influence on it, whatever they or
 * their values hold (infinities and NaN included).  A token that sees no key
 * (its sequence is shorter than its chunk) has out 0 and lse -infinity.
 * Rows of out beyond cu_new[n_requests] are not written.  Sums, maxima and
 * products are held in fp32; on the tensor cores the probabilities are rounded
 * to dtype for the second product (off by at most half a unit in the last place
 * each; in fp16, those below 2^-21 of the row's largest by 2^-32 of it).  A page id
 * outside the cache counts as a page of zeros, and is reported; so is a sequence
 * longer than the table's columns, which counts as ending with them.
 * T == 0 or n_requests == 0 is a no-op.  Workspace: 256-byte aligned, scratch.
 * The result does not depend on the order in which blocks run. */
int ds_moe_paged_attention(const ds_moe_attn_shape *shape, const ds_moe_kv_cache *cache, const int32_t *block_table,
                           int32_t table_width, int64_t table_stride, const void *q, int64_t q_stride, int64_t T,
                           const int32_t *cu_new, const int32_t *seq_lens, int32_t n_requests, int32_t max_new,
                           void *out, int64_t out_stride, float *lse, void *workspace, size_t workspace_bytes,
                           void *stream, char *err, size_t errlen);

/* Checks drafted tokens against the model's probabilities, from given random
 * numbers, so that the tokens kept are distributed as the model's own.
 * Request r was fed tokens[cu_new[r]] (the last one kept) and then its
 * drafts; row cu_new[r] + i of target and draft is the distribution of the
 * token behind its i-th, so draft i (from 1) is checked against row
 * cu_new[r] + i - 1.
 *   target  [T][vocab] (vocab up to 2^22), dtype DS_F32 or DS_BF16, rows
 *           target_stride elements apart: the model's probabilities, each in
 *           [0, 1].  A row need not add up to 1 where it is sampled from (it
 *           is normalised by its sum); drafts are judged by its entries as
 *           they are
 *   draft   the same for the drafter (rows of drafts only are read), or NULL:
 *           the drafter was sure of each draft
 *   u_accept [T] fp32 (entry of draft i: cu_new[r] + i - 1), u_sample
 *           [n_requests] fp32, in [0, 1)
 * Draft x at row i is kept while u_accept * draft(x) < target(x), exactly.
 * At the first that is not, one token is drawn from max(target - draft, 0)
 * (from target where nothing is left); when all were kept, from the
 * target row behind the last.  Drawn is the least token whose cumulative sum
 * exceeds u_sample times the total.  What is summed are entries (or
 * differences) rounded to whole numbers of 2^-44, of 2^-43 for vocabularies
 * from 2^19 up, and so on to 2^-40 for 2^22: the sums are exact, so they do not
 * depend on any order, and less than half a unit counts as nothing.
 *   out_tokens [n_requests][max_new] int32: the drafts kept, the token drawn,
 *           then -1;  n_accepted [n_requests] int32: drafts kept
 * A request without new tokens gives -1s and 0.  Reported: a draft outside
 * the vocabulary (it is not kept), a row that is sampled from and has nothing
 * that counts (token -1), probabilities that are NaN, negative or
 * above 1 in a row that is sampled from (NaN and negative count as 0, others
 * as 1), lengths beyond T or max_new (dropped). */
int ds_moe_verify_drafts(const void *target, int64_t target_stride, const void *draft, int64_t draft_stride,
                         int32_t dtype, int64_t T, int32_t vocab, const int32_t *tokens, const int32_t *cu_new,
                         int32_t n_requests, int32_t max_new, const float *u_accept, const float *u_sample,
                         int32_t *out_tokens, int32_t *n_accepted, void *stream, char *err, size_t errlen);

/* Which kernels ds_moe_paged_attention runs with a table of one column or
 * more (without columns there are no keys, and the call is DS_ATTN_GENERIC's;
 * host call; nothing is launched): one of the DS_ATTN_* values, or a negative
 * ds_status.  q_stride: as for several tokens; the stride of a single one is
 * not used, so n_head * head_dim stands for it. */
enum {
  DS_ATTN_GENERIC = 0, /* any strides, page and head sizes: CUDA cores        */
  DS_ATTN_DECODE = 1,  /* up to 32 query rows (max_new * n_head / n_head_kv)
                          a key head: keys as the rows of tensor-core tiles  */
  DS_ATTN_CHUNK = 2    /* more query rows: queries as the rows               */
};
int ds_moe_attention_path(const ds_moe_attn_shape *shape, const ds_moe_kv_cache *cache, const void *q,
                          int64_t q_stride, int32_t max_new);

/* ------------------------------------------------------------------------
 * Positions.  Queries and keys carry their tokens' positions as rotations:
 * pair i of the rotated elements of a head turns by position * f_i,
 *     (a, b) -> (a cos - b sin, b cos + a sin) * amplitude
 * with f_i = base^(-2i / dim), stretched for contexts longer than the trained
 * one as `scaling` says.
 * ---------------------------------------------------------------------- */

enum {
  DS_ROPE_NONE = 0,
  DS_ROPE_LINEAR = 1, /* f_i / factor (positions brought closer together)    */
  DS_ROPE_NTK = 2,    /* base * factor^(dim / (dim - 2)): the slowest pair turns
                         factor times slower, the fastest as before; dim >= 4 */
  DS_ROPE_YARN = 3    /* by parts (Peng et al., "YaRN", 2023): pairs that turn
                         more than beta_fast times over the `original` trained
                         positions keep f_i, those below beta_slow get
                         f_i / factor, those between a mixture               */
};

/* A rotation (host object, passed by address and copied into the call; a
 * captured graph keeps its copy).  ds_moe_rope_init fills it; frequencies of
 * the caller's own may be put into turns[] instead. */
typedef struct {
  int32_t dim;         /* rotated elements of a head: even, 2..128           */
  int32_t first;       /* the first of them; elements outside are not changed */
  int32_t interleaved; /* 0: pair i is elements i and i + dim/2 (halves);
                          1: elements 2i and 2i + 1                          */
  float amplitude;     /* multiplies the rotated elements                    */
  uint64_t turns[64];  /* f_i / (2 pi) * 2^64: what a position turns pair i by,
                          in fractions of a turn; position * turns[i] wraps to
                          the angle, so far positions lose nothing           */
} ds_moe_rope;

/* (Host call.)  base >= 1, factor >= 1; amplitude 0: 1, or 0.1 ln(factor) + 1
 * with DS_ROPE_YARN.  original (>= 1), beta_fast > beta_slow > 0 (0, 0: 32
 * and 1) are DS_ROPE_YARN's only. */
int ds_moe_rope_init(ds_moe_rope *rope, int32_t dim, int32_t first, int32_t interleaved, double base, int32_t scaling,
                     double factor, int64_t original, double beta_fast, double beta_slow, double amplitude, char *err,
                     size_t errlen);

/* Rows to rotate: head h of token t is head_dim elements from
 * x + t * token_stride + h * head_stride, and goes to out + t *
 * out_token_stride + h * out_head_stride (strides in elements, the last axis
 * dense).  out may be x with the same strides; otherwise the two may not
 * share memory.  Rows of out that overlap are refused (one of its strides has to step
 * over all that the other spans). */
typedef struct {
  const void *x;
  int64_t token_stride, head_stride;
  void *out;
  int64_t out_token_stride, out_head_stride;
} ds_moe_rope_rows;

/* Rotates n_head heads (1..1024) of T tokens, of dtype DS_BF16 or DS_F16, by
 * their positions [T] (int32).  Rows of a negative position are left as they
 * were (ds_moe_page_map writes -1 past the last token).  Products are fp32,
 * rounded once to dtype.  16-byte aligned rows, and head_dim, first and dim
 * multiples of 16, are the fast case. */
int ds_moe_rotary(const ds_moe_rope *rope, int32_t dtype, int32_t n_head, int32_t head_dim,
                  const ds_moe_rope_rows *rows, const int32_t *positions, int64_t T, void *stream, char *err,
                  size_t errlen);

/* ds_moe_kv_append with the keys rotated on the way, and, where q is given,
 * the T tokens' queries (shape->n_head heads) rotated in the same launch.
 * Slots below zero are none (their queries are rotated all the same), rows
 * of a negative position are left out altogether.  slots and positions as
 * ds_moe_page_map writes them. */
int ds_moe_kv_append_rotary(const ds_moe_attn_shape *shape, const ds_moe_kv_cache *cache, const ds_moe_rope *rope,
                            const void *k_new, const void *v_new, int64_t token_stride, int64_t head_stride,
                            const ds_moe_rope_rows *q, const int64_t *slots, const int32_t *positions, int64_t T,
                            void *stream, char *err, size_t errlen);

/* ------------------------------------------------------------------------
 * A cache in 8 bits: pages of e4m3 elements (4 bits of exponent, 3 of
 * mantissa, up to 448, NaN 0x7F and 0xFF, no infinities), and a scale for each
 * block of block_rows rows of a page and each head: an element stands for
 * e4m3 * scale.
 * ---------------------------------------------------------------------- */
typedef struct {
  void *k, *v;           /* elements, placed as in ds_moe_kv_cache            */
  float *k_scale, *v_scale; /* of block b of a page and head h: at page *
                            scale_page_stride + b * scale_block_stride + h *
                            scale_head_stride                                */
  int64_t n_pages;
  int64_t page_stride, row_stride, head_stride;
  int64_t scale_page_stride, scale_block_stride, scale_head_stride;
  int32_t block_rows;    /* 1..page_size, a divisor of it                     */
} ds_moe_kv8_cache;      /* (an append refuses rows that overlap and scales that share
                            a place; attention takes strides of scales that are zero, as of one
                            scale for all heads)                              */

/* Quantises the new tokens' keys and values into their requests' pages:
 * k_new and v_new [T][n_head_kv][head_dim] of shape->dtype, tokens
 * token_stride and heads head_stride elements apart.  Places come from
 * block_table, cu_new and seq_lens as ds_moe_page_map writes them: token i of
 * a request's n is at position seq_len - n + i.  (A token before position 0
 * has no place and is left out, its queries too; so are tokens beyond max_new, which are
 * reported, as are those beyond the table's columns, which have no place.)  With `rope` the keys are rotated first, and q's rows where they
 * are given (q needs rope); q is rotated also where a token has no page.
 * The scale of a block and head is a power of two, the least (from 2^-60 to
 * 2^60) that brings the largest of its new elements to 448 or below.  Where
 * the block holds earlier tokens of the sequence (position not a multiple of
 * block_rows), the scale does not fall, and where it rises the earlier tokens'
 * elements are brought to it (exactly, but for those that leave e4m3's
 * normal range).  Elements are rounded once from fp32, to the nearest; what
 * is not finite becomes NaN and has no say in the scale.  No two requests may
 * have new tokens in the same block, as no two tokens may share a slot.  The
 * same call again gives the same cache. */
int ds_moe_kv8_append(const ds_moe_attn_shape *shape, const ds_moe_kv8_cache *cache, const ds_moe_rope *rope,
                      const void *k_new, const void *v_new, int64_t token_stride, int64_t head_stride,
                      const ds_moe_rope_rows *q, const int32_t *block_table, int32_t table_width, int64_t table_stride,
                      const int32_t *cu_new, const int32_t *seq_lens, int32_t n_requests, int64_t T, int32_t max_new,
                      void *stream, char *err, size_t errlen);

/* ds_moe_paged_attention over a cache in 8 bits: the same arguments and the
 * same rules, with keys and values e4m3 * scale (scales may be any fp32, as
 * another quantiser leaves them; one outside of 2^-60 .. 2^60 counts as the
 * nearest of the two, NaN as the smaller).  q and out are of shape->dtype.
 * What is not finite in q counts as NaN on the tensor cores.
 *   DS_ATTN_DECODE: elements go to the tensor cores as they are, queries as
 *       sums of e4m3 numbers (exact down to 2^-22 of a row's largest element in
 *       bf16, 2^-27 in fp16), weights times their values' scales as sums of
 *       e5m2 numbers (fp16, for bf16 cut to 9 bits: off by 2^-11, 2^-9, or by
 *       2^-30 of the row's largest); the weights' own sum, and lse, in fp32
 *       whatever the values' scales are (where those are 2^120 apart, without
 *       weights below 2^-35 of the largest)
 *   DS_ATTN_CHUNK: e4m3 * scale rounded to dtype (exact in bf16 where the scale is a power
 *       of two; in fp16 values beyond 65504 become 65504), the rest as in
 *       ds_moe_paged_attention
 *   DS_ATTN_GENERIC: fp32 throughout
 * The tensor-core kernels want head_dim and the strides multiples of 16,
 * bases 16-byte aligned, page_size a multiple of 8, q's strides multiples of 8
 * elements. */
int ds_moe_attention8_workspace_bytes(const ds_moe_attn_shape *shape, int32_t n_requests, int64_t T, int32_t max_new,
                                      size_t *bytes, char *err, size_t errlen);
int ds_moe_paged_attention8(const ds_moe_attn_shape *shape, const ds_moe_kv8_cache *cache, const int32_t *block_table,
                            int32_t table_width, int64_t table_stride, const void *q, int64_t q_stride, int64_t T,
                            const int32_t *cu_new, const int32_t *seq_lens, int32_t n_requests, int32_t max_new,
                            void *out, int64_t out_stride, float *lse, void *workspace, size_t workspace_bytes,
                            void *stream, char *err, size_t errlen);
/* As ds_moe_attention_path. */
int ds_moe_attention8_path(const ds_moe_attn_shape *shape, const ds_moe_kv8_cache *cache, const void *q,
                           int64_t q_stride, int32_t max_new);

/* Library version string (static storage). */
const char *ds_moe_version(void);

#ifdef __cplusplus
}
#endif

#endif /* DS_MOE_H */
