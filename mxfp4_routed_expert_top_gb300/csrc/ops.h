// ops.h — the expert-path operators that need no handle: argument structs and
// launchers shared by k_permute.cu, k_fp8.cu and ops.cu (not part of the ABI).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace dfm {

constexpr int kOpsMaxExperts = 1024;
constexpr int kOpsMaxTopK = 32;

inline int dtype_bytes(int dtype) {  // DF_MOE_BF16, _F16, _F32, _E4M3
  return dtype == 2 ? 4 : dtype == 3 ? 1 : 2;
}

// n / nb for n < 2^31: with 2^(shift - 1) < nb <= 2^shift and mul =
// ceil(2^(31 + shift) / nb), the error n (mul nb - 2^(31 + shift)) stays below
// 2^(31 + shift).
struct FastDiv {
  uint32_t mul, shift;
  explicit FastDiv(uint32_t nb) : mul(0), shift(0) {
    while ((1ull << shift) < nb) ++shift;
    mul = (uint32_t)(((1ull << (31 + shift)) + nb - 1) / nb);
  }
  __device__ uint32_t operator()(uint32_t n) const {
    return (uint32_t)(((uint64_t)n * mul) >> (31 + shift));
  }
};

// Rows of `bytes` bytes and the distances of consecutive rows, in bytes.
struct PermuteArgs {
  const int32_t* ids;  // [T][k]
  int T, k, E;
  const char* x;
  char* rows;
  int64_t bytes, ldx, ldr;
  const float* xs;  // second payload: n_scales floats a row (or null)
  float* rows_s;
  int n_scales;
  int64_t ldxs, ldrs;  // in floats
  int32_t *offs, *pos, *src;
};
size_t permute_workspace_bytes(int64_t T, int k, int E);
cudaError_t launch_permute(const PermuteArgs& p, void* workspace, int sms, cudaStream_t s);

struct UnpermuteArgs {
  const void* rows;
  const int32_t* pos;    // [T][k]
  const float* weights;  // [T][k] or null: every row counts once
  void* y;
  int T, k, H;
  int64_t n_rows, ldr, ldy;  // in elements
};
cudaError_t launch_unpermute(const UnpermuteArgs& p, int dtype, int sms, cudaStream_t s);

struct UnpermuteGradArgs {
  const void* dy;
  const void* rows;
  const int32_t* pos;
  const float* weights;
  void* drows;
  float* dweights;
  int T, k, H;
  int64_t n_rows, lddy, ldr, lddr;  // in elements
};
cudaError_t launch_unpermute_grad(const UnpermuteGradArgs& p, int dtype, int sms, cudaStream_t s);

struct QuantizeArgs {
  const void* x;
  uint8_t* codes;
  float* scales;
  int64_t M;
  int K;
  int64_t ldx, ldc, lds;  // in elements
};
cudaError_t launch_fp8_quantize(const QuantizeArgs& p, int dtype, int sms, cudaStream_t s);

struct Fp8MatmulArgs {
  const uint8_t* x;
  const float* xs;
  const uint8_t* w;
  const float* ws;
  const int32_t* offs;  // [G + 1] or null (G = 1)
  void* y;
  int G, N, K, transposed;
  int64_t M, ldx, ldxs, ldw, ldy;  // in elements
  uint32_t* status;
  int give_up;  // test hook: 0, or the role (1 to 4) of block 0 that gives up
};
// What it could not do, as text, or null.
const char* launch_fp8_matmul(const Fp8MatmulArgs& p, int dtype, int sms, cudaStream_t s);

}  // namespace dfm
