// k_balance_bf16.cu — the balance loss's kernels (k_balance.cuh) for bf16 logits.
#include "k_balance.cuh"

namespace dfm {

cudaError_t balance_rows_bf16(const BalanceArgs& p, const Entries& out, int64_t chunk, int64_t blocks, int alone, cudaStream_t s) {
  return rows_t<__nv_bfloat16>(p, out, chunk, blocks, alone, s);
}
cudaError_t balance_grad_bf16(const BalanceGradArgs& p, int sms, cudaStream_t s) {
  return grad_t<__nv_bfloat16>(p, sms, s);
}

}  // namespace dfm
