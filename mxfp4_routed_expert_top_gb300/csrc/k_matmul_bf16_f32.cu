// k_matmul_bf16_f32.cu — the product (k_matmul.cuh) of bf16 matrices in fp32.
#include "k_matmul.cuh"

namespace dfm {

const char* gemm_bf16_f32(const GemmArgs& a, int sms, cudaStream_t s) { return gemm<0, 2>(a, sms, s); }

}  // namespace dfm
