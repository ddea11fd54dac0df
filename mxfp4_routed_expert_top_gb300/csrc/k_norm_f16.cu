// k_norm_f16.cu — the norms between blocks (k_norm.cuh) for f16 rows.
#include "k_norm.cuh"

namespace dfm {

cudaError_t block_norm_f16(const BlockNormArgs& p, int wtype, int sms, cudaStream_t s) { return norm_t<__half>(p, wtype, sms, s); }
cudaError_t block_norm_grad_f16(const BlockNormGradArgs& p, int wtype, float* part, int sms, cudaStream_t s) {
  return grad_t<__half>(p, wtype, part, sms, s);
}

}  // namespace dfm
