/*
 * kvq.h -- layer-wise mixed-precision KV-cache quantization and decode
 * attention over the quantized cache, for NVIDIA GB300 (sm_103a).
 *
 * The method (sources are web pages, cited by title and section):
 *   - every layer stores its cache at a static precision pair KxVy,
 *     x, y in {2, 3, 4, 8}, chosen offline and loaded with no online cost
 *     ("KVTuner: Sensitivity-Aware Layer-Wise Mixed-Precision KV Cache
 *     Quantization ...", sections A1 and A2; "KVmix: Gradient-Based Layer
 *     Importance-Aware Mixed-Precision Quantization for KV Cache", 关键设计 2 and 4);
 *   - keys are quantized asymmetrically per channel over groups of G tokens
 *     (or, per layer, per token), values per token, with scale = (max - min)/(2^b - 1), zero = min and
 *     code = clamp(rint((x - min)/scale), 0, 2^b - 1); codes are packed into
 *     32-bit words, 3-bit words holding ten 3-bit fields and one 2-bit field
 *     (KVTuner section A3 "KV缓存量化基础"; KVmix 关键设计 2; "LLM 量化精读笔记 · 08
 *     KV Cache 量化：KIVI 与误差累积", sections 6.1 and 6.2);
 *   - the most recent tokens stay in an FP16 residual window of R_l tokens;
 *     when the window holds R_l or more tokens the oldest G are quantized as one
 *     key group (KIVI notes section 6.2; KVmix 关键设计 3); with an RPC ratio
 *     (KVmix 关键设计 3, num_RPC = floor(r x current_RPC)) the window bound
 *     shrinks as decoding proceeds (see kvq_layer_cfg.rpc_percent);
 *   - decode attention a = softmax(q K^T / sqrt(d)), o = a V runs over the
 *     quantized tokens (dequantized on the fly) and the FP16 window, after the
 *     new token has been appended (KVTuner section A3 equation).
 *
 * Conventions shared by all entry points:
 *   - The library allocates no device memory.  The caller allocates one device
 *     buffer of kvq_cache_bytes() bytes and hands it to kvq_create(); the
 *     library carves the per-layer caches, their state and its workspace out
 *     of it.  The caller frees it after kvq_destroy().
 *   - Device pointers passed to kvq_append() and kvq_decode_attn() must be
 *     16-byte aligned and stay valid until the work queued on `stream` is done.
 *   - Arguments are checked on the host before anything is launched; a failed
 *     check returns a status and changes nothing.  KVQ_ERR_CUDA reports a
 *     failed launch; the handle's host-side state is then undefined.
 *   - Work is queued on `stream` (a cudaStream_t passed as void*; NULL is the
 *     legacy default stream) and runs asynchronously.  One handle is driven by
 *     one host thread at a time; calls on a handle are ordered by the caller.
 *   - All sequences of a batch share one length.
 *   - No kernel spins without bound and none traps: a device-side wait that
 *     gives up sets an error word that kvq_device_error() reports.
 */
#ifndef KVQ_H
#define KVQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  KVQ_OK = 0,
  KVQ_ERR_ARG = 1,      /* null pointer, bad dimension, layer out of range   */
  KVQ_ERR_BITS = 2,     /* a bit width outside {2, 3, 4, 8}                  */
  KVQ_ERR_ALIGN = 3,    /* a pointer that is not 16-byte aligned             */
  KVQ_ERR_CAPACITY = 4, /* appending past max_tokens, or buffer too small    */
  KVQ_ERR_CUDA = 5,     /* a CUDA runtime call failed                        */
  KVQ_ERR_STATE = 6,    /* call not valid now (e.g. attention on empty layer)*/
  KVQ_ERR_UNSUPPORTED = 7 /* a shape the library has no kernel for        */
} kvq_status;

/* Key quantization mode of a layer (KVTuner sections A3-A4 evaluate both):
 *   KVQ_KEY_PER_CHANNEL: keys per channel over each group of G tokens (KIVI);
 *   KVQ_KEY_PER_TOKEN:   keys per token over their head_dim channels, like
 *                        values ("per-token-asym"); k_bits in {2, 4, 8}. */
#define KVQ_KEY_PER_CHANNEL 0
#define KVQ_KEY_PER_TOKEN 1

/* One layer's static precision pair, key mode and FP16 residual window (tokens).
 * k_bits, v_bits in {2, 3, 4, 8}; residual >= group_size and a multiple of it.
 * key_mode KVQ_KEY_PER_TOKEN with k_bits = 3 is KVQ_ERR_UNSUPPORTED.
 *
 * rpc_percent (0..100; KVQ_ERR_ARG above 100) is KVmix's RPC ratio (关键设计 3:
 * num_RPC = floor(r x current_RPC), 20% on its high-precision layers, 10% on
 * the others, the full-precision count shrinking as decoding proceeds).  0
 * keeps a static window of `residual` tokens.  Otherwise the layer keeps a
 * window bound C, first `residual` (the prompt's share): any append quantizes
 * the oldest group_size window tokens while the window holds C or more, and a
 * single-token append that brings the window to C first sets
 * C = group_size * max(1, floor(rpc_percent * C / (100 * group_size))).
 * Multi-token appends keep C.  The ring keeps `residual` slots. */
typedef struct {
  uint8_t k_bits;
  uint8_t v_bits;
  uint8_t key_mode;     /* KVQ_KEY_PER_CHANNEL or KVQ_KEY_PER_TOKEN */
  uint8_t rpc_percent;  /* 0: static window; else the RPC ratio in percent */
  int32_t residual;
} kvq_layer_cfg;

/* Shape of the cache.
 *   num_q_heads % num_kv_heads == 0 and num_q_heads / num_kv_heads <= 8
 *   head_dim in {64, 128}; group_size in {32, 64, 128}
 *   max_tokens: capacity per sequence (all appended tokens, quantized or not)
 *   layers: num_layers entries, read during kvq_create() only. */
typedef struct {
  int32_t num_layers;
  int32_t batch;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t group_size;
  int32_t max_tokens;
  const kvq_layer_cfg* layers;
} kvq_config;

typedef struct kvq_handle kvq_handle;

/* Device layout of one layer, for tests and for callers that snapshot the
 * cache.  All pointers are device pointers into the buffer given to
 * kvq_create(); counts are the host's view after the calls issued so far.
 *
 * Per (batch b, kv head h) "unit" u = b * num_kv_heads + h:
 *   records + u * unit_record_stride is a sequence of group records, one per
 *   quantized key group (group j covers tokens [j*G, (j+1)*G)), each
 *   record_bytes long:
 *     [K codes: G rows x k_words u32][V codes: G rows x v_words u32]
 *     [K scale: head_dim f16][K zero: head_dim f16]   (per-channel keys), or
 *     [K (scale, zero): G pairs of f16]               (per-token keys)
 *     [V (scale, zero): G pairs of f16]
 *   With 2-, 4- or 8-bit keys each per-channel key row is stored in 8-channel
 *   chunks, chunk j of each channel quarter side by side: position 4j + t
 *   holds the channels of chunk t*head_dim/32 + j (head_dim 64: chunks
 *   0 2 4 6 1 3 5 7); 3-bit keys keep channel order.
 *   A code row is one token's head_dim codes, least significant field first:
 *   for b in {2,4,8} field j of word w is channel w*32/b + j at bits [b*j, b*j+b);
 *   for b = 3 word w holds channels 11w .. 11w+10, fields 0..9 3-bit at bit 3j
 *   and field 10 2-bit at bits 30..31.  Packed word w of token row t (t counted
 *   inside the record) is stored at index w XOR x: key rows of 32 words:
 *   x = 4 on odd t; value rows of 16 words: x = 8 when t & 2; value rows of 32
 *   words: x = 8 * (t & 3); all other rows x = 0.
 *   residual_k + u * residual_stride (and residual_v likewise) is a ring of
 *   `residual` slots of head_dim fp16 holding the window tokens
 *   [quantized_tokens, tokens); token i sits in slot i % residual, and
 *   the 16-byte chunk c of a slot s is stored at chunk position c ^ (s & 7). */
typedef struct {
  int32_t k_bits, v_bits, residual, group_size, head_dim;
  int32_t k_words, v_words;          /* u32 words per code row                */
  int32_t key_mode;                  /* KVQ_KEY_PER_CHANNEL or _PER_TOKEN     */
  int64_t record_bytes;
  int64_t unit_record_stride;        /* bytes between units' record arrays    */
  int64_t residual_stride;           /* bytes between units' rings            */
  int64_t tokens;                    /* tokens appended so far                */
  int64_t quantized_tokens;          /* tokens held as quantized groups       */
  int64_t residual_tokens;           /* tokens held in the FP16 ring          */
  const void* records;
  const void* residual_k;
  const void* residual_v;
  int32_t window_bound;              /* current window bound C (<= residual) */
  int32_t rpc_percent;               /* the layer's RPC ratio (0: static)     */
} kvq_layer_view;

/* Bytes of device memory the caller must provide for `cfg` (0 if cfg is
 * invalid).  Includes every layer's cache sized for max_tokens, per-layer
 * state and the decode workspace. */
size_t kvq_cache_bytes(const kvq_config* cfg);

/* Validate `cfg`, lay the caches out in `dev_buf` (device memory, 256-byte
 * aligned, `bytes` >= kvq_cache_bytes(cfg)), zero it, and select the kernel
 * instantiations for every layer's (k_bits, v_bits, head_dim, heads-per-kv)
 * once, so that later calls dispatch with a table lookup.  Writes a new handle
 * to *out.  Synchronizes the device once (the zeroing). */
kvq_status kvq_create(const kvq_config* cfg, void* dev_buf, size_t bytes, kvq_handle** out);

/* Append n_tokens (>= 0) new tokens to `layer`, oldest first.
 * K, V: device, fp16, [batch][num_kv_heads][n_tokens][head_dim] contiguous,
 * read-only, caller-owned.  New tokens enter the FP16 window; while the
 * window holds the layer's bound (`residual`, or less after an RPC shrink,
 * see kvq_layer_cfg) or more tokens, the oldest group_size tokens are
 * quantized (keys per channel, values per token), packed and stored as the
 * next group record, all in the launched kernels.  Used for prefill
 * (n_tokens = prompt length) and for decode (n_tokens = 1).
 * KVQ_ERR_CAPACITY if tokens + n_tokens > max_tokens. */
kvq_status kvq_append(kvq_handle* h, int layer, const void* K, const void* V, int n_tokens,
                      void* stream);

/* Decode attention of one query token per sequence over everything appended
 * to `layer` so far.
 * q: device fp16 [batch][num_q_heads][head_dim]; query head j reads kv head
 *    j / (num_q_heads / num_kv_heads).
 * out: device fp32 [batch][num_q_heads][head_dim], written entirely.
 * Scores are scaled by 1/sqrt(head_dim).  KVQ_ERR_STATE if the layer is empty.
 * The kernel is launched as a programmatic dependent of the previous kernel on
 * the stream: its CTAs may start while that kernel drains, but each waits for
 * it to complete before its first read, so stream order holds as usual. */
kvq_status kvq_decode_attn(kvq_handle* h, int layer, const void* q, float* out, void* stream);

/* Causal attention of the queries of the n_queries newest tokens over `layer`
 * as it stands: prefill or chunked-prefill attention over the quantized cache
 * (KVTuner, section A2, calibration design: prefill runs over the dequantized
 * cache; the attention is its A3 equation).  Call after appending the chunk.
 * With T tokens appended, query i (0 <= i < n_queries) belongs to the token at
 * position T - n_queries + i and attends the tokens at positions
 * 0 .. T - n_queries + i: quantized groups dequantized (code * s + z), window
 * tokens as stored.  Scores are scaled by 1/sqrt(head_dim).
 * q: device fp16 [batch][num_q_heads][n_queries][head_dim], 16-byte aligned;
 *    query head j reads kv head j / (num_q_heads / num_kv_heads).
 * out: device fp32 [batch][num_q_heads][n_queries][head_dim], written entirely.
 * workspace: caller-owned device scratch of at least
 *    kvq_chunk_workspace_bytes(h) bytes, 16-byte aligned; the layer's tiles are
 *    dequantized into it once, then read by the tensor-core kernel.  Its
 *    contents are overwritten; a call must not share it with another in flight.
 * KVQ_ERR_ARG if n_queries < 1 or > tokens appended; KVQ_ERR_STATE if the layer
 * is empty; KVQ_ERR_CAPACITY if the workspace is too small;
 * KVQ_ERR_UNSUPPORTED if batch * num_kv_heads > 65535.  Runs on the tensor
 * cores (tcgen05). */
kvq_status kvq_chunk_attn(kvq_handle* h, int layer, const void* q, int n_queries, float* out, void* workspace,
                          size_t workspace_bytes, void* stream);

/* Bytes of the workspace kvq_chunk_attn needs for any layer of `h` (its
 * dequantized tiles of every (batch, kv head) at max_tokens).  0 if h is null. */
size_t kvq_chunk_workspace_bytes(const kvq_handle* h);

/* One decode step over every layer: for l = 0 .. num_layers-1,
 * kvq_append(l, K[l], V[l], 1) then kvq_decode_attn(l, q[l], out[l]).
 * K, V, q, out are host arrays of num_layers device pointers, with the shapes
 * above (n_tokens = 1).  The launches of a step do not depend on the cache
 * state, so after the first call with a given set of pointers the step is
 * replayed from a CUDA graph the handle keeps (it is re-captured when the
 * pointers change).  Inside the graph the appends run on a forked stream:
 * decode l waits for append l (and for decode l-1), so later layers' appends
 * overlap earlier layers' decodes.  Decode l is a programmatic dependent of
 * decode l-1: it stages its first items of layer l's cache (which decode l-1
 * does not write) while decode l-1 drains, and reads q[l] and writes out[l]
 * only after it.  KVQ_ERR_CAPACITY if any layer is full. */
kvq_status kvq_decode_step(kvq_handle* h, const void* const* K, const void* const* V,
                           const void* const* q, float* const* out, void* stream);

/* Size of the library's own device scratch for kvq_decode_attn_noalloc():
 * 4 MiB, a file-scope device array that every GPU which loads the library
 * keeps until the process exits. */
#define KVQ_NOALLOC_SCRATCH_BYTES (4u << 20)

/* kvq_decode_attn() for callers that may not allocate device memory at all.
 *
 * The papers have no counterpart to this entry point; it exists for callers
 * such as plugins hosted by another runtime that owns every device
 * allocation, or code on a latency path where cudaMalloc (which synchronises
 * the device) is not allowed.  Such a caller may hold a cache whose buffer it
 * cannot grow, and cannot hand the library extra workspace.
 *
 * Same arguments, result and errors as kvq_decode_attn(), except that the
 * split-merge workspace (per-split partial results and one arrival counter
 * per (batch, kv head) unit) comes from the library's static device array of
 * KVQ_NOALLOC_SCRATCH_BYTES instead of the handle's buffer, and nothing is
 * allocated: no cudaMalloc, no cudaFree, no allocating library call.
 *   - Needs align256(units * 4) + (grid + units) * gqa * (head_dim + 2) * 4
 *     bytes, where units = batch * num_kv_heads and grid is the layer's
 *     launch width (at most 1024 CTAs); a layer needing more returns
 *     KVQ_ERR_CAPACITY and launches nothing.
 *   - The current device must be the one that was current at kvq_create()
 *     (the device holding the handle's buffer); otherwise KVQ_ERR_ARG and
 *     nothing is launched.
 *   - The first call on a device looks up the array's device address with
 *     cudaGetSymbolAddress and keeps it; make that first call before any
 *     stream capture.  KVQ_ERR_CUDA if the lookup fails.
 *   - Each call clears the counters on `stream` (an asynchronous memset of
 *     units * 4 bytes) before it launches the kernel.
 *   - Every call on a device shares the one array: calls that overlap on the
 *     GPU (other streams, or other handles, without ordering between them)
 *     race on it and give wrong results.  Order them on one stream. */
kvq_status kvq_decode_attn_noalloc(kvq_handle* h, int layer, const void* q, float* out, void* stream);

/* Describe `layer` (see kvq_layer_view). */
kvq_status kvq_layer_view_get(const kvq_handle* h, int layer, kvq_layer_view* v);

/* f_m: mean over layers of (k_bits + v_bits) / 2 (KVTuner section A2). */
double kvq_equivalent_bits(const kvq_handle* h);

/* Algorithmic bytes one kvq_decode_attn(layer) call reads for the current
 * state (packed codes, scales/zeros, FP16 window, q) and writes (out). */
int64_t kvq_decode_bytes(const kvq_handle* h, int layer);

/* Reads the device error word (a bounded wait that gave up, or an internal
 * consistency check), clearing it.  Synchronizes `stream`.  0 means none. */
kvq_status kvq_device_error(kvq_handle* h, int32_t* code, void* stream);

/* Failure-detection self-test of the device-side waits.  Launches one warp
 * that waits on an mbarrier nothing ever completes, with a short bound (4096
 * tries), as every wait in the library is bounded.  The wait must give up,
 * record the timeout in the error word and return, with the CUDA context
 * still usable.  KVQ_OK if exactly that happened (the word is read and
 * cleared), KVQ_ERR_STATE if the timeout was not reported.  Synchronizes
 * `stream`; changes nothing else. */
kvq_status kvq_selftest_bounded_wait(kvq_handle* h, void* stream);

/* Snapshots of the streaming state, to rewind a cache to an earlier point
 * (re-running a window of decode steps, or dropping tokens decoded after the
 * snapshot).  A snapshot holds every layer's token counters (appended tokens,
 * quantized tokens, window bound, of every (batch, kv head) unit) and its FP16
 * residual window ring; it does not hold the quantized groups.  That is enough:
 * an append only writes groups at or past the quantized-token count it starts
 * from, and attention reads only groups below the current count, so a group
 * the snapshot does not hold is written again before anything reads it
 * (the cache is the groups quantized so far plus the FP16 window: KIVI notes
 * section 6.2, KVmix 关键设计 3).
 *
 * kvq_state_bytes: bytes of a snapshot of `h` (0 if h is null).
 *
 * kvq_state_save: copies the state into `dst`, a caller-owned device buffer of
 * kvq_state_bytes(h) bytes, 16-byte aligned, on `stream` after the work already
 * queued there (plain device-to-device copies, one per layer plus one for the
 * counters).  KVQ_ERR_ARG if h or dst is null, KVQ_ERR_ALIGN if dst is not
 * 16-byte aligned.
 *
 * kvq_state_restore: makes `src` (a snapshot saved from `h`, or from a handle
 * created with the same configuration) the cache's state.  It first reads the
 * snapshot's counters to the host (synchronizing `stream`) and checks that they
 * describe a state the cache can be in: every unit of a layer agrees, the
 * quantized count is a multiple of G and at most the appended count, which is
 * at most max_tokens, the window holds fewer tokens than its bound, and the
 * bound is a multiple of G between G and R_l (R_l itself on a static window).
 * KVQ_ERR_STATE if not, and nothing changes.  Otherwise the copies back are
 * queued on `stream` and the host mirror is set from the snapshot.  A captured
 * decode step stays valid (its launches read the state from the device). */
size_t kvq_state_bytes(const kvq_handle* h);
kvq_status kvq_state_save(kvq_handle* h, void* dst, void* stream);
kvq_status kvq_state_restore(kvq_handle* h, const void* src, void* stream);

/* Release the handle (host memory and any captured graph).  The device buffer
 * stays the caller's. */
kvq_status kvq_destroy(kvq_handle* h);

const char* kvq_status_string(kvq_status s);

/* ------------------------------------------------------------------ pages
 *
 * A paged cache: the rows of every sequence live in pages of page_size tokens
 * that a table names, so that sequences of any lengths share one pool, join
 * and leave a running batch, and share full pages of a common prefix.  Every
 * layer has its own (k_bits, v_bits): 16 keeps rows in the cache's type;
 * 8, 4 and 2 quantize every row when it is appended, keys and values per token
 * over their head_dim channels (the per-token-asym mode of KVQ_KEY_PER_TOKEN:
 * KVTuner sections A3-A4), with no FP16 window.
 *
 * Shared by the paged entry points:
 *   - Lengths, tables and rows are read on the device: nothing of a call but
 *     pointers, strides and counts is fixed on the host, so a captured call
 *     follows the tensors it was captured with.
 *   - What a call works by is not changed after kvq_paged_create(): calls on
 *     it may come from several threads and streams.  The caller orders calls
 *     that append to a page with those that read or append to the same page.
 *   - The current device must be the one of kvq_paged_create() (KVQ_ERR_ARG).
 *   - The tensors of a batch must not change while a call that reads them runs:
 *     its result has no meaning then (but nothing outside its tensors is
 *     touched, and every wait ends).
 *   - What only the device can see (a page number outside the pool, a length
 *     past the table's width, a position past the rotation's table, fewer
 *     tokens in a sequence than it has new rows) is never followed:
 *     kvq_paged_device_error() reports it, an append or a read leaves the row
 *     out, and what attention returns for that sequence has no meaning. */

#define KVQ_FP16 0
#define KVQ_BF16 1

/* k_bits, v_bits: both 16, or both in {2, 4, 8} (KVQ_ERR_UNSUPPORTED for a
 * 16 beside a smaller width, KVQ_ERR_BITS for any other). */
typedef struct {
  uint8_t k_bits;
  uint8_t v_bits;
} kvq_paged_layer_cfg;

/* num_q_heads % num_kv_heads == 0 and num_q_heads / num_kv_heads <= 8, at most
 * 65536 heads and layers; head_dim in {64, 128}; page_size in {16, 32, 64, 128};
 * dtype: KVQ_FP16 or KVQ_BF16, the type of q, K, V, out and of 16-bit rows. */
typedef struct {
  int32_t num_layers;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t page_size;
  int32_t num_pages;   /* pages of each layer */
  int32_t dtype;
  const kvq_paged_layer_cfg* layers;
} kvq_paged_config;

typedef struct kvq_paged kvq_paged;

/* Device layout of one layer: page p's part of kv head h starts at
 * pages + p * page_stride + h * head_stride and holds page_size / 16 tiles of
 * tile_bytes, 16 consecutive tokens each.  The tile of tokens i = 0 .. 15:
 *   16-bit rows: [K: 16 rows][V: 16 rows] of head_dim values; the 16-byte chunk
 *     c of token i is stored at chunk c ^ (i & 7) of row i.
 *   quantized:   [K codes: 16 rows][V codes: 16 rows][16 x (K scale, K zero,
 *     V scale, V zero) fp16], code rows of head_dim * bits / 8 bytes, least
 *     significant field first.  The key row and the scales of token i sit at
 *     row r(i) = 2 (i & 3) + (i >> 2 & 1) + (i & 8), its value row at row i.
 *     128-byte key rows: on odd r the 64-byte halves are exchanged.  Value
 *     rows keep their 32-byte block b at b ^ (i & 3) (128-byte rows) or at
 *     b ^ (i >> 1 & 1) (64-byte rows). */
typedef struct {
  int32_t k_bits, v_bits, page_size, head_dim;
  int64_t tile_bytes, head_stride, page_stride;
  void* pages;
} kvq_paged_view;

/* The sequences that a call works on.  All pointers are device memory.
 *   page_table: [num_seqs] rows of max_pages page numbers, table_stride
 *     elements apart; entry k of a row holds positions k * page_size .. .
 *     Entries past a sequence's last page, and in attention those of pages
 *     wholly before its window, are not read.  max_pages * page_size is at
 *     most 2^30, and num_seqs * num_kv_heads below 2^31 (KVQ_ERR_ARG).
 *   seq_lens: [num_seqs] tokens of each sequence, the new ones included.
 *   cu_tokens: [num_seqs + 1] ascending, or NULL.  Rows cu_tokens[s] ..
 *     cu_tokens[s + 1] - 1 of a call's row tensors are the newest tokens of
 *     sequence s, oldest first; NULL: row s is the newest token of sequence s
 *     (none where seq_lens[s] is 0).  Rows that belong to no sequence, such as
 *     padding behind the last one, are not written, whatever they hold. */
typedef struct {
  const int32_t* page_table;
  int64_t table_stride;
  const int32_t* seq_lens;
  const int32_t* cu_tokens;
  int32_t num_seqs;
  int32_t max_pages;
} kvq_paged_batch;

/* Rotation of queries and keys by their position.
 *   table: device fp32 [rows][dim]: dim / 2 cosines, then dim / 2 sines, of
 *     each position's angles; 16-byte aligned.
 *   positions: device [n_tokens], each row's position, or NULL: its place in
 *     its sequence.
 *   dim: channels that turn, the first `dim` of a row, a multiple of 16;
 *     interleaved 0 pairs channel i with i + dim / 2, 1 pairs 2i with 2i + 1.
 * (a, b) becomes (a cos - b sin, b cos + a sin) in fp32, rounded once. */
typedef struct {
  const float* table;
  const int32_t* positions;
  int32_t rows;
  int32_t dim;
  int32_t interleaved;
} kvq_rotation;

/* A tensor of rows: row i's head h starts at data + (i * token_stride + h *
 * head_stride) elements; its head_dim values are contiguous. */
typedef struct {
  void* data;
  int64_t token_stride;
  int64_t head_stride;
} kvq_rows;

/* Bytes of the caller's device buffer (0 if cfg is invalid): every layer's
 * pages, layer 0 first, each layer 256-byte aligned, then 256 bytes of the
 * library's own. */
size_t kvq_paged_bytes(const kvq_paged_config* cfg);

/* Validates `cfg` and writes a handle on the pages in `dev_buf` (256-byte
 * aligned, caller-owned) to *out.  What the pages hold stays: a page's slots
 * mean nothing until they are appended to, whatever they hold.  Clears the
 * error word (synchronizes once). */
kvq_status kvq_paged_create(const kvq_paged_config* cfg, void* dev_buf, size_t bytes, kvq_paged** out);

/* Appends the new rows of every sequence of `batch` to `layer`: keys turned by
 * `rotation` (NULL: as they are), rounded to the cache's type or quantized,
 * and written to their slots with the values; queries turned alike into q_out.
 *   K, V: [n_tokens][num_kv_heads] rows.  q, q_out: [n_tokens][num_q_heads]
 *     rows, or both NULL; q_out may be q itself, and overlaps nothing else, nor
 *     its rows one another.
 *   n_tokens: rows of the tensors; without cu_tokens, equal to num_seqs.
 * Rows need only their type's alignment; 16-byte aligned rows are faster.
 * Quantized rows are taken in fp16 (clamped to +-65504): zero = min,
 * scale = fp16((max - min) * r) with r = fp32(1 / (2^b - 1)), code =
 * clamp(rint((x - zero) / scale), 0, 2^b - 1), as kvq_append does per token but
 * for the scale's last bit (it divides by 2^b - 1); a row with a NaN gets
 * NaN scales.  Two rows of one call with the same slot (one page in the tables
 * of two sequences that both append to it) leave one of them or a mixture
 * there. */
kvq_status kvq_paged_append(kvq_paged* h, int layer, const kvq_paged_batch* batch, const kvq_rows* K,
                            const kvq_rows* V, const kvq_rows* q, const kvq_rows* q_out,
                            const kvq_rotation* rotation, int n_tokens, void* stream);

/* Attention of one query token per sequence, the newest one, over its pages:
 * positions max(0, len - window) .. len - 1 (window 0: all of them).
 *   q: [num_seqs][num_q_heads] rows (cu_tokens is not looked at).
 *   out: [num_seqs][num_q_heads][head_dim] contiguous, 16-byte aligned, the
 *     cache's type, overlapping no other argument.
 *   lse: fp32 [num_seqs][num_q_heads] or NULL: the natural logarithm of the sum
 *     of exp(scale * q.k).  A sequence with no token, or with no score above
 *     -infinity, gets 0, and -infinity.  (A NaN in an attended row, a score of
 *     +infinity or an infinite value leaves NaN or infinity where it counts.)
 *   scale: multiplies the scores; 0 means 1 / sqrt(head_dim).
 *   workspace: device scratch of kvq_paged_workspace_bytes(h, num_seqs) bytes,
 *     256-byte aligned, whatever it holds; not shared with a call in flight.
 * KVQ_ERR_ARG for a negative window or a scale that is not finite, or not so
 * times log2(e) (above 2.35e38);
 * KVQ_ERR_CAPACITY for a small workspace; KVQ_ERR_UNSUPPORTED where the tables
 * could hold more than 2^30 tiles of work for every SM. */
kvq_status kvq_paged_decode_attn(kvq_paged* h, int layer, const kvq_paged_batch* batch, const kvq_rows* q, void* out,
                                 float* lse, float scale, int window, void* workspace, size_t workspace_bytes,
                                 void* stream);

/* Bytes of the workspace above (0 if h is null or num_seqs < 1). */
size_t kvq_paged_workspace_bytes(const kvq_paged* h, int num_seqs);

/* Reads the newest rows of every sequence (cu_tokens as for an append) back as
 * the cache holds them: code * scale + zero in fp32, rounded once to the
 * cache's type.  K, V: [n_tokens][num_kv_heads] rows, none of which overlaps
 * another; either may be NULL.
 * Rows with a bad page are left as they were. */
kvq_status kvq_paged_read(kvq_paged* h, int layer, const kvq_paged_batch* batch, const kvq_rows* K, const kvq_rows* V,
                          int n_tokens, void* stream);

kvq_status kvq_paged_view_get(const kvq_paged* h, int layer, kvq_paged_view* v);

/* Takes the error word, synchronizing `stream`; what calls on other streams
 * set meanwhile is in it or stays for the next call.  0, or 1 a device
 * wait gave up, 2 a length or a row count that the batch's tensors cannot
 * mean, 4 a bad page number, 5 a position outside the rotation's table. */
kvq_status kvq_paged_device_error(kvq_paged* h, int32_t* code, void* stream);

kvq_status kvq_paged_destroy(kvq_paged* h);

#ifdef __cplusplus
}
#endif

#endif /* KVQ_H */
