// k_balance_f32.cu — the balance loss's kernels (k_balance.cuh) for f32 logits.
#include "k_balance.cuh"

namespace dfm {

cudaError_t balance_rows_f32(const BalanceArgs& p, const Entries& out, int64_t chunk, int64_t blocks, int alone, cudaStream_t s) {
  return rows_t<float>(p, out, chunk, blocks, alone, s);
}
cudaError_t balance_grad_f32(const BalanceGradArgs& p, int sms, cudaStream_t s) {
  return grad_t<float>(p, sms, s);
}

}  // namespace dfm
