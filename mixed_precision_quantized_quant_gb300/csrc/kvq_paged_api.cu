// Host side of the paged cache's entry points (include/kvq.h): configuration
// checks, the pool's layout in the caller's buffer, argument checks, launches.
// Nothing of a handle changes after its creation.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstring>
#include <mutex>
#include <new>
#include <vector>

#include <nvtx3/nvToolsExt.h>

#include "../../include/kvq.h"
#include "kvq_paged.cuh"

namespace {

struct Trace {
  explicit Trace(const char* name) { nvtxRangePushA(name); }
  ~Trace() { nvtxRangePop(); }
};

constexpr int64_t kAlign = 256;
constexpr int64_t kTail = 256;  // the library's own bytes behind the pages: the error word, and where it is taken to
constexpr int kMaxLayers = 1 << 16, kMaxHeads = 1 << 16;

struct PagedLayer {
  int kb, vb, tile_bytes;
  int64_t head_stride, page_stride, off;
};

bool shape_ok(const kvq_paged_config* c) {
  return c && c->layers && c->num_layers >= 1 && c->num_layers <= kMaxLayers && c->num_q_heads >= 1 &&
         c->num_q_heads <= kMaxHeads &&
         c->num_kv_heads >= 1 && c->num_q_heads % c->num_kv_heads == 0 && (c->head_dim == 64 || c->head_dim == 128) &&
         (c->page_size == 16 || c->page_size == 32 || c->page_size == 64 || c->page_size == 128) &&
         c->num_pages >= 1 && (c->dtype == KVQ_FP16 || c->dtype == KVQ_BF16);
}

bool code_bits(int b) { return b == 2 || b == 4 || b == 8; }

// Layer l's layout, `off` bytes into the buffer.
kvq_status layer_plan(const kvq_paged_config* c, int l, int64_t off, PagedLayer* out, int64_t* end) {
  const int kb = c->layers[l].k_bits, vb = c->layers[l].v_bits;
  if ((kb != 16 && !code_bits(kb)) || (vb != 16 && !code_bits(vb))) return KVQ_ERR_BITS;
  if ((kb == 16) != (vb == 16)) return KVQ_ERR_UNSUPPORTED;
  out->kb = kb;
  out->vb = vb;
  out->tile_bytes = kvq::paged_tile_bytes(c->head_dim, kb, vb);
  out->head_stride = static_cast<int64_t>(c->page_size / kvq::kTile) * out->tile_bytes;
  // a page is at most 2^31 x 2^16 bytes; the pool's size is checked for 62 bits
  out->page_stride = out->head_stride * c->num_kv_heads;
  out->off = off;
  const double total = static_cast<double>(out->page_stride) * c->num_pages + static_cast<double>(off);
  if (total > 4e18) return KVQ_ERR_UNSUPPORTED;
  *end = (off + out->page_stride * c->num_pages + kAlign - 1) / kAlign * kAlign;
  return KVQ_OK;
}

kvq_status paged_size(const kvq_paged_config* c, int64_t* bytes) {
  if (!shape_ok(c)) return KVQ_ERR_ARG;
  if (c->num_q_heads / c->num_kv_heads > 8) return KVQ_ERR_UNSUPPORTED;
  int64_t off = 0;
  for (int l = 0; l < c->num_layers; ++l) {
    PagedLayer lay;
    const kvq_status st = layer_plan(c, l, off, &lay, &off);
    if (st != KVQ_OK) return st;
  }
  *bytes = off + kTail;
  return KVQ_OK;
}

// Takes the error word in one step, so that no call of another stream sets it between its reading and its clearing.
__global__ void take_error_kernel(int32_t* err) { err[1] = atomicExch(err, 0); }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

struct kvq_paged {
  kvq_paged_config cfg;  // its layers pointer is not kept
  std::vector<PagedLayer> layers;
  uint8_t* base = nullptr;
  int32_t* err = nullptr;
  int device = 0, sms = 0;
  std::mutex taking;  // of the error word: err[1] is one call's at a time
  int64_t checked_bytes = INT64_MAX;  // debug builds: where the checks take a layer's pages to end at the latest
};

namespace {

// Errors that every call shares; KVQ_OK with the batch copied where there are none.
kvq_status open_call(const kvq_paged* h, int layer, const kvq_paged_batch* b, kvq::PagedBatch* batch,
                     kvq::PagedPool* pool) {
  if (!h || layer < 0 || layer >= h->cfg.num_layers || !b) return KVQ_ERR_ARG;
  if (b->num_seqs < 1 || b->max_pages < 1 || b->table_stride < b->max_pages || !b->page_table || !b->seq_lens)
    return KVQ_ERR_ARG;
  // positions, rounded up to a chunk, and units are held in 32 bits
  if (static_cast<int64_t>(b->max_pages) * h->cfg.page_size > 1 << 30 ||
      static_cast<int64_t>(b->num_seqs) * h->cfg.num_kv_heads > INT_MAX)
    return KVQ_ERR_ARG;
  int cur = -1;
  if (cudaGetDevice(&cur) != cudaSuccess) return KVQ_ERR_CUDA;
  if (cur != h->device) return KVQ_ERR_ARG;
  batch->table = b->page_table;
  batch->table_stride = b->table_stride;
  batch->lens = b->seq_lens;
  batch->cu = b->cu_tokens;
  batch->seqs = b->num_seqs;
  batch->max_pages = b->max_pages;
  const PagedLayer& l = h->layers[layer];
  pool->pages = h->base + l.off;
  pool->page_stride = l.page_stride;
  pool->head_stride = l.head_stride;
  pool->tile_bytes = l.tile_bytes;
  pool->num_pages = h->cfg.num_pages;
  pool->page_shift = h->cfg.page_size == 16 ? 4 : h->cfg.page_size == 32 ? 5 : h->cfg.page_size == 64 ? 6 : 7;
  pool->kb = l.kb;
  pool->vb = l.vb;
  pool->err = h->err;
  pool->hi = pool->pages + (l.page_stride * h->cfg.num_pages < h->checked_bytes ? l.page_stride * h->cfg.num_pages : h->checked_bytes);
  return KVQ_OK;
}

// `n` rows of `heads` rows of `d` 2-byte values: at least their own alignment;
// *vec cleared unless every row starts on 16 bytes.
kvq_status take_rows(const kvq_rows* r, int n, int heads, int d, kvq::PagedRows* out, int* vec) {
  if (!r || !r->data) return KVQ_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(r->data) & 1u) return KVQ_ERR_ALIGN;
  if (!aligned16(r->data) || r->token_stride % 8 != 0 || r->head_stride % 8 != 0) *vec = 0;
  out->data = static_cast<uint8_t*>(r->data);
  out->token_stride = r->token_stride;
  out->head_stride = r->head_stride;
  const int64_t tokens = (n - 1) * r->token_stride, others = (heads - 1) * r->head_stride;
  out->lo = out->data + 2 * ((tokens < 0 ? tokens : 0) + (others < 0 ? others : 0));
  out->hi = out->data + 2 * ((tokens > 0 ? tokens : 0) + (others > 0 ? others : 0) + d);
  return KVQ_OK;
}

}  // namespace

extern "C" {

size_t kvq_paged_bytes(const kvq_paged_config* cfg) {
  int64_t n = 0;
  return paged_size(cfg, &n) == KVQ_OK ? static_cast<size_t>(n) : 0;
}

kvq_status kvq_paged_create(const kvq_paged_config* cfg, void* dev_buf, size_t bytes, kvq_paged** out) {
  Trace trace("kvq_paged_create");
  if (!out) return KVQ_ERR_ARG;
  *out = nullptr;
  int64_t need = 0;
  const kvq_status st = paged_size(cfg, &need);
  if (st != KVQ_OK) return st;
  if (!dev_buf) return KVQ_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(dev_buf) & (kAlign - 1)) != 0) return KVQ_ERR_ALIGN;
  if (bytes < static_cast<size_t>(need)) return KVQ_ERR_CAPACITY;
  kvq_paged* h = new (std::nothrow) kvq_paged;
  if (!h) return KVQ_ERR_ARG;
  try {
    h->layers.resize(static_cast<size_t>(cfg->num_layers));
  } catch (...) {
    delete h;
    return KVQ_ERR_ARG;
  }
  h->cfg = *cfg;
  h->cfg.layers = nullptr;
  h->base = static_cast<uint8_t*>(dev_buf);
  int64_t off = 0;
  for (int l = 0; l < cfg->num_layers; ++l) {
    layer_plan(cfg, l, off, &h->layers[l], &off);
    if (kvq::paged_attn_prepare(h->layers[l].kb, h->layers[l].vb, cfg->head_dim, cfg->dtype) != cudaSuccess) {
      delete h;
      return KVQ_ERR_CUDA;
    }
  }
  h->err = reinterpret_cast<int32_t*>(h->base + off);
  if (cudaGetDevice(&h->device) != cudaSuccess ||
      cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, h->device) != cudaSuccess ||
      cudaMemset(h->err, 0, kTail) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) {
    delete h;
    return KVQ_ERR_CUDA;
  }
  *out = h;
  return KVQ_OK;
}

kvq_status kvq_paged_append(kvq_paged* h, int layer, const kvq_paged_batch* batch, const kvq_rows* K,
                            const kvq_rows* V, const kvq_rows* q, const kvq_rows* q_out,
                            const kvq_rotation* rotation, int n_tokens, void* stream) {
  Trace trace("kvq_paged_append");
  kvq::PagedAppendParams p = {};
  kvq_status st = open_call(h, layer, batch, &p.batch, &p.pool);
  if (st != KVQ_OK) return st;
  if (n_tokens < 0 || n_tokens > INT_MAX - 31 || (!batch->cu_tokens && n_tokens != batch->num_seqs) || (!q != !q_out)) return KVQ_ERR_ARG;
  if (n_tokens == 0) return KVQ_OK;
  p.vec = 1;
  const int hq = h->cfg.num_q_heads, hkv = h->cfg.num_kv_heads, d = h->cfg.head_dim;
  if ((st = take_rows(K, n_tokens, hkv, d, &p.k, &p.vec)) != KVQ_OK ||
      (st = take_rows(V, n_tokens, hkv, d, &p.v, &p.vec)) != KVQ_OK)
    return st;
  if (q && ((st = take_rows(q, n_tokens, hq, d, &p.q, &p.vec)) != KVQ_OK ||
            (st = take_rows(q_out, n_tokens, hq, d, &p.qo, &p.vec)) != KVQ_OK))
    return st;
  if (rotation) {
    if (!rotation->table || rotation->rows < 1 || rotation->dim < 16 || rotation->dim % 16 != 0 ||
        rotation->dim > h->cfg.head_dim || (rotation->interleaved != 0 && rotation->interleaved != 1))
      return KVQ_ERR_ARG;
    if (!aligned16(rotation->table)) return KVQ_ERR_ALIGN;
    p.rope = rotation->table;
    p.positions = rotation->positions;
    p.rope_rows = rotation->rows;
    p.rope_dim = rotation->dim;
    p.interleaved = rotation->interleaved;
  }
  p.n = n_tokens;
  p.hq = q ? hq : 0;
  p.hkv = hkv;
  return kvq::paged_append_launch(p, d, h->cfg.dtype, h->sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? KVQ_OK
             : KVQ_ERR_CUDA;
}

size_t kvq_paged_workspace_bytes(const kvq_paged* h, int num_seqs) {
  if (!h || num_seqs < 1) return 0;
  return kvq::paged_attn_workspace(h->cfg.head_dim, h->cfg.num_kv_heads,
                                   num_seqs, h->sms);
}

kvq_status kvq_paged_decode_attn(kvq_paged* h, int layer, const kvq_paged_batch* batch, const kvq_rows* q, void* out,
                                 float* lse, float scale, int window, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  Trace trace("kvq_paged_decode_attn");
  kvq::PagedAttnParams p = {};
  kvq_status st = open_call(h, layer, batch, &p.batch, &p.pool);
  if (st != KVQ_OK) return st;
  p.q_vec = 1;
  if ((st = take_rows(q, batch->num_seqs, h->cfg.num_q_heads, h->cfg.head_dim, &p.q, &p.q_vec)) != KVQ_OK) return st;
  if (!out || !workspace || window < 0 || !std::isfinite(scale)) return KVQ_ERR_ARG;
  if (!aligned16(out) || (reinterpret_cast<uintptr_t>(lse) & 3u) ||
      (reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1)))
    return KVQ_ERR_ALIGN;
  if (workspace_bytes < kvq_paged_workspace_bytes(h, batch->num_seqs)) return KVQ_ERR_CAPACITY;
  // a CTA's share of the work is held in 32 bits
  const int64_t units = static_cast<int64_t>(batch->num_seqs) * h->cfg.num_kv_heads;
  const int64_t tiles = static_cast<int64_t>(batch->max_pages) * h->cfg.page_size / kvq::kTile + 16;
  if (tiles > (static_cast<int64_t>(INT_MAX) / 2 * h->sms) / units) return KVQ_ERR_UNSUPPORTED;
  const double sc = scale == 0.0f ? 1.0 / std::sqrt(static_cast<double>(h->cfg.head_dim)) : scale;
  p.out = out;
  p.lse = lse;
  p.alpha = static_cast<float>(sc * 1.4426950408889634);
  if (!std::isfinite(p.alpha)) return KVQ_ERR_ARG;  // scores are taken in base 2
  p.window = window;
  p.hkv = h->cfg.num_kv_heads;
  p.gqa = h->cfg.num_q_heads / h->cfg.num_kv_heads;
  p.ws = static_cast<uint8_t*>(workspace);
  p.ws_hi = p.ws + workspace_bytes;
  return kvq::paged_attn_launch(p, h->cfg.head_dim, h->cfg.dtype, h->sms, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? KVQ_OK
             : KVQ_ERR_CUDA;
}

kvq_status kvq_paged_read(kvq_paged* h, int layer, const kvq_paged_batch* batch, const kvq_rows* K, const kvq_rows* V,
                          int n_tokens, void* stream) {
  Trace trace("kvq_paged_read");
  kvq::PagedReadParams p = {};
  kvq_status st = open_call(h, layer, batch, &p.batch, &p.pool);
  if (st != KVQ_OK) return st;
  if (n_tokens < 0 || n_tokens > INT_MAX - 31 || (!batch->cu_tokens && n_tokens != batch->num_seqs) || (!K && !V)) return KVQ_ERR_ARG;
  if (n_tokens == 0) return KVQ_OK;
  p.vec = 1;
  const int hkv = h->cfg.num_kv_heads, d = h->cfg.head_dim;
  if (K && (st = take_rows(K, n_tokens, hkv, d, &p.k, &p.vec)) != KVQ_OK) return st;
  if (V && (st = take_rows(V, n_tokens, hkv, d, &p.v, &p.vec)) != KVQ_OK) return st;
  p.n = n_tokens;
  p.hkv = hkv;
  return kvq::paged_read_launch(p, d, h->cfg.dtype, h->sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? KVQ_OK
             : KVQ_ERR_CUDA;
}

kvq_status kvq_paged_view_get(const kvq_paged* h, int layer, kvq_paged_view* v) {
  if (!h || !v || layer < 0 || layer >= h->cfg.num_layers) return KVQ_ERR_ARG;
  std::memset(v, 0, sizeof(*v));
  const PagedLayer& l = h->layers[layer];
  v->k_bits = l.kb;
  v->v_bits = l.vb;
  v->page_size = h->cfg.page_size;
  v->head_dim = h->cfg.head_dim;
  v->tile_bytes = l.tile_bytes;
  v->head_stride = l.head_stride;
  v->page_stride = l.page_stride;
  v->pages = h->base + l.off;
  return KVQ_OK;
}

kvq_status kvq_paged_device_error(kvq_paged* h, int32_t* code, void* stream) {
  Trace trace("kvq_paged_device_error");
  if (!h || !code) return KVQ_ERR_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int cur = -1;
  if (cudaGetDevice(&cur) != cudaSuccess) return KVQ_ERR_CUDA;
  if (cur != h->device) return KVQ_ERR_ARG;
  int32_t v = 0;
  try {
    const std::lock_guard<std::mutex> one(h->taking);
    take_error_kernel<<<1, 1, 0, s>>>(h->err);
    if (cudaGetLastError() != cudaSuccess ||
        cudaMemcpyAsync(&v, h->err + 1, 4, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
      return KVQ_ERR_CUDA;
  } catch (...) {
    return KVQ_ERR_CUDA;
  }
  *code = v;
  return KVQ_OK;
}

#ifdef KVQ_DEBUG
// For the tests of the checks: accesses past the first `bytes` of a layer's
// pages count as outside them, so that a check fires on memory that is there.
kvq_status kvq_paged_debug_limit(kvq_paged* h, int64_t bytes);
kvq_status kvq_paged_debug_limit(kvq_paged* h, int64_t bytes) {
  if (!h || bytes < 0) return KVQ_ERR_ARG;
  h->checked_bytes = bytes;
  return KVQ_OK;
}
#endif

kvq_status kvq_paged_destroy(kvq_paged* h) {
  Trace trace("kvq_paged_destroy");
  if (!h) return KVQ_ERR_ARG;
  delete h;
  return KVQ_OK;
}

}  // extern "C"
