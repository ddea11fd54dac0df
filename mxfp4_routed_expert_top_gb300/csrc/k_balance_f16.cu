// k_balance_f16.cu — the balance loss's kernels (k_balance.cuh) for f16 logits.
#include "k_balance.cuh"

namespace dfm {

cudaError_t balance_rows_f16(const BalanceArgs& p, const Entries& out, int64_t chunk, int64_t blocks, int alone, cudaStream_t s) {
  return rows_t<__half>(p, out, chunk, blocks, alone, s);
}
cudaError_t balance_grad_f16(const BalanceGradArgs& p, int sms, cudaStream_t s) {
  return grad_t<__half>(p, sms, s);
}

}  // namespace dfm
