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

enum Activation { kActNone = 0, kActRelu, kActSilu, kActGelu, kActSwiglu };  // DF_MOE_ACT_*

// 16-bit matrix, `ld` elements a row; mn: stored with the product's k along
// its rows' distance (k rows of R or C values), else R or C rows of k.
struct GemmOperand {
  const void* p;
  int64_t ld;
  bool mn;
};
// y[r][c] = residual[r][c] + act(sum_k row[r][k] col[c][k] + bias[c]); gated:
// col has 2 C rows and act(z)[c] = silu(z[c]) z[C + c].
struct GemmArgs {
  GemmOperand row, col;
  int64_t R, K;
  int C, in, out, act;  // in: 0 bf16, 1 fp16 (operands, bias, pre); out: of y and residual
  const void *bias, *residual;
  void *pre, *y;
  int64_t ldr, ldp, ldy;
  uint32_t* status;
  int give_up;
  // kGemmFirst: kGemmSecond comes next, of the same call, and does not need
  // this one's output: it may run beside it.
  int order;
  int64_t beside;  // tiles of 64 x 128 of the other's output
};
enum { kGemmAlone = 0, kGemmFirst, kGemmSecond };
const char* launch_gemm(const GemmArgs& a, int sms, cudaStream_t s);
// of one pair of types each
const char* gemm_bf16(const GemmArgs& a, int sms, cudaStream_t s);
const char* gemm_bf16_f32(const GemmArgs& a, int sms, cudaStream_t s);
const char* gemm_f16(const GemmArgs& a, int sms, cudaStream_t s);
const char* gemm_f16_f32(const GemmArgs& a, int sms, cudaStream_t s);

struct ActGradArgs {
  const void *dy, *pre;
  void *dz, *dbias;  // dbias or null
  int64_t M, lddy, ldp, lddz;
  int N, in, grad, act;  // grad: type of dbias
  bool follows;          // a product on dz comes next
};
const char* launch_act_grad(const ActGradArgs& a, int sms, cudaStream_t s);

enum GateKind { kGateNone = 0, kGateChannel, kGateToken, kGateFull };  // DF_MOE_GATE_*

constexpr int kNormMaxHidden = 32768;
// Arrays of dtype but: post_w, pre_w and a channel's gate of the weights' type,
// a token's gate and the gradients of weights and of those gates fp32.
struct BlockNormArgs {
  const void *u, *post_w, *gate, *residual, *pre_w;
  void *h, *n;
  int64_t T, ldu, ldg, ldr, ldh, ldn;  // in elements
  int H, post, gate_kind;
  float scale, eps;
};
cudaError_t launch_block_norm(const BlockNormArgs& p, int dtype, int wtype, int sms, cudaStream_t s);

struct BlockNormGradArgs {
  const void *dh, *dn, *u, *h, *post_w, *gate, *pre_w;
  void *du, *dresidual, *dgate;
  float *dpost_w, *dpre_w;
  int64_t T, lddh, lddn, ldu, ldh, ldg, lddu, lddr, lddg;  // in elements
  int H, post, gate_kind;
  float scale, eps;
};
size_t block_norm_grad_workspace_bytes(int64_t T, int H);
// of one type each
cudaError_t block_norm_bf16(const BlockNormArgs& p, int wtype, int sms, cudaStream_t s);
cudaError_t block_norm_f16(const BlockNormArgs& p, int wtype, int sms, cudaStream_t s);
cudaError_t block_norm_f32(const BlockNormArgs& p, int wtype, int sms, cudaStream_t s);
cudaError_t block_norm_grad_bf16(const BlockNormGradArgs& p, int wtype, float* part, int sms, cudaStream_t s);
cudaError_t block_norm_grad_f16(const BlockNormGradArgs& p, int wtype, float* part, int sms, cudaStream_t s);
cudaError_t block_norm_grad_f32(const BlockNormGradArgs& p, int wtype, float* part, int sms, cudaStream_t s);
cudaError_t launch_block_norm_grad(const BlockNormGradArgs& p, int dtype, int wtype, void* workspace, int sms, cudaStream_t s);

struct BalanceArgs {
  const void* logits;
  const int32_t *ids, *offs;  // offs or null (S = 1)
  const uint8_t* mask;        // or null
  float *loss, *probs;        // probs or null
  int32_t *counts, *tokens;
  uint32_t* status;  // or null
  int64_t T, ldl;
  int E, k, S, sigmoid;
  float coef, z_coef;
};
size_t balance_workspace_bytes(int64_t T, int E, int64_t S);
cudaError_t launch_balance_loss(const BalanceArgs& p, int dtype, void* workspace, cudaStream_t s);

struct BalanceGradArgs {
  const float* dloss;
  const void* logits;
  const int32_t *ids, *offs, *counts, *tokens;
  const uint8_t* mask;
  const float *weights, *dweights;  // both or neither
  void* dlogits;
  int64_t T, ldl, lddl;
  int E, k, S, sigmoid;
  float coef, z_coef;
};
cudaError_t launch_balance_loss_grad(const BalanceGradArgs& p, int dtype, int sms, cudaStream_t s);

}  // namespace dfm
