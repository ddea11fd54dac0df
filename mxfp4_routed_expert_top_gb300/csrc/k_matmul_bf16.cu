// k_matmul_bf16.cu — the product (k_matmul.cuh) of bf16 matrices.
#include "k_matmul.cuh"

namespace dfm {

const char* gemm_bf16(const GemmArgs& a, int sms, cudaStream_t s) { return gemm<0, 0>(a, sms, s); }

}  // namespace dfm
