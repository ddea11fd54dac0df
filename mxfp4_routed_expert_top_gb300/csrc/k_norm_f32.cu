// k_norm_f32.cu — the norms between blocks (k_norm.cuh) for f32 rows, and the
// choice of the type.
#include "k_norm.cuh"

namespace dfm {

cudaError_t block_norm_f32(const BlockNormArgs& p, int, int sms, cudaStream_t s) { return norm_tw<float, float>(p, sms, s); }
cudaError_t block_norm_grad_f32(const BlockNormGradArgs& p, int, float* part, int sms, cudaStream_t s) {
  return grad_tw<float, float>(p, part, sms, s);
}

size_t block_norm_grad_workspace_bytes(int64_t T, int H) { return 8 * (size_t)grad_workers(T, H) * (size_t)H; }

cudaError_t launch_block_norm(const BlockNormArgs& p, int dtype, int wtype, int sms, cudaStream_t s) {
  return (dtype == 0 ? block_norm_bf16 : dtype == 1 ? block_norm_f16 : block_norm_f32)(p, wtype, sms, s);
}
cudaError_t launch_block_norm_grad(const BlockNormGradArgs& p, int dtype, int wtype, void* workspace, int sms, cudaStream_t s) {
  return (dtype == 0 ? block_norm_grad_bf16 : dtype == 1 ? block_norm_grad_f16 : block_norm_grad_f32)(p, wtype, static_cast<float*>(workspace), sms, s);
}

}  // namespace dfm
