// Paged attention with 4-bit keys.
#include "kvq_paged_attn.cuh"

namespace kvq {

cudaError_t paged_attn_k4(const PagedAttnParams* p, int vb, int D, int dtype, int sms, cudaStream_t s) {
  if (vb == 8) return paged::attn_quant<4, 8>(p, D, dtype, sms, s);
  if (vb == 4) return paged::attn_quant<4, 4>(p, D, dtype, sms, s);
  return paged::attn_quant<4, 2>(p, D, dtype, sms, s);
}

}  // namespace kvq
