// Paged attention of 16-bit layers, the choice by bit width, and the workspace.
#include "kvq_paged_attn.cuh"

namespace kvq {

cudaError_t paged_attn_k16(const PagedAttnParams* p, int D, int dtype, int sms, cudaStream_t s) {
  return paged::attn_quant<16, 16>(p, D, dtype, sms, s);
}

// The units' notes, then two partial results for every CTA of the widest launch.
static int64_t partials_at(int hkv, int seqs) {
  return (static_cast<int64_t>(hkv) * seqs * static_cast<int64_t>(sizeof(paged::Meta)) + 255) / 256 * 256;
}

size_t paged_attn_workspace(int D, int hkv, int seqs, int sms) {
  return static_cast<size_t>(partials_at(hkv, seqs) + 2LL * paged::kMostCtas * sms * paged::partial_floats(D) * 4);
}

static cudaError_t choose(const PagedAttnParams* p, int kb, int vb, int D, int dtype, int sms, cudaStream_t s) {
  if (kb == 16) return paged_attn_k16(p, D, dtype, sms, s);
  if (kb == 8) return paged_attn_k8(p, vb, D, dtype, sms, s);
  if (kb == 4) return paged_attn_k4(p, vb, D, dtype, sms, s);
  return paged_attn_k2(p, vb, D, dtype, sms, s);
}

cudaError_t paged_attn_prepare(int kb, int vb, int D, int dtype) { return choose(nullptr, kb, vb, D, dtype, 0, nullptr); }

cudaError_t paged_attn_launch(PagedAttnParams p, int D, int dtype, int sms, cudaStream_t s) {
  p.ws_partials = partials_at(p.hkv, p.batch.seqs);
  return choose(&p, p.pool.kb, p.pool.vb, D, dtype, sms, s);
}

}  // namespace kvq
