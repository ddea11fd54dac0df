// k_matmul_f16.cu — the product (k_matmul.cuh) of fp16 matrices.
#include "k_matmul.cuh"

namespace dfm {

const char* gemm_f16(const GemmArgs& a, int sms, cudaStream_t s) { return gemm<1, 1>(a, sms, s); }

}  // namespace dfm
