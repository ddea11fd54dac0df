// ops.cu — C entry points of the expert-path operators (no handle): argument
// checks, the device, the launch. They keep nothing between calls but the
// SM count of each device (and what the test hook asks of the next product).
#include <cuda_runtime.h>

#include <atomic>
#include <cstdarg>
#include <cstdio>

#include "df_moe.h"
#include "internal.h"
#include "ops.h"

namespace {

int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int fail(int code, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  dfm::set_thread_error(buf);
  return code;
}

// Makes `device` (or, negative, the current one) current for the call.
class OnDevice {
 public:
  explicit OnDevice(int device) {
    if (cudaGetDevice(&before_) != cudaSuccess) {
      (void)cudaGetLastError();
      rc_ = fail(DF_MOE_ECUDA, "no CUDA device");
      return;
    }
    now_ = device < 0 ? before_ : device;
    if (now_ != before_ && cudaSetDevice(now_) != cudaSuccess) {
      (void)cudaGetLastError();
      rc_ = fail(DF_MOE_EINVAL, "no CUDA device %d", device);
      now_ = before_;
    }
  }
  ~OnDevice() {
    if (now_ != before_) (void)cudaSetDevice(before_);
  }
  int rc() const { return rc_; }
  int sms() const {
    constexpr int kMax = 64;
    static std::atomic<int> known[kMax];
    int n = now_ < kMax ? known[now_].load() : 0;
    if (!n) {
      if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, now_) != cudaSuccess || n < 1)
        n = 1;
      if (now_ < kMax) known[now_].store(n);
    }
    return n;
  }

 private:
  int before_ = 0, now_ = 0, rc_ = DF_MOE_OK;
};

thread_local int give_up_next = 0;

constexpr int64_t kMaxRows = 0x7fffffff;
constexpr int kMaxHidden = 1 << 18;

int launched(const char* what, cudaError_t e) {
  if (e == cudaSuccess) return DF_MOE_OK;
  (void)cudaGetLastError();
  return fail(DF_MOE_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool off(const void* p, int align) { return ((uintptr_t)p & (uintptr_t)(align - 1)) != 0; }

// Shared checks of the routing sizes.
int check_routing(int64_t T, int k, int64_t H) {
  if (T < 0) return fail(DF_MOE_EINVAL, "T = %lld is negative", (long long)T);
  if (k < 1 || k > dfm::kOpsMaxTopK) return fail(DF_MOE_EINVAL, "k must be in [1, 32]");
  if (H < 1 || H > kMaxHidden) return fail(DF_MOE_EINVAL, "H must be in [1, 262144]");
  if (T > kMaxRows / k)
    return fail(DF_MOE_ERANGE, "T * k = %lld assignments: at most 2^31 - 1", (long long)T * k);
  return DF_MOE_OK;
}

// A row distance of 0 stands for rows without gaps.
int check_ld(const char* name, int64_t* ld, int64_t n) {
  if (*ld == 0) *ld = n;
  if (*ld < n) return fail(DF_MOE_EINVAL, "%s is below the row's length", name);
  return DF_MOE_OK;
}

int check_float_dtype(int dtype) {
  if (dtype < DF_MOE_BF16 || dtype > DF_MOE_F32)
    return fail(DF_MOE_EINVAL, "dtype must be DF_MOE_BF16, DF_MOE_F16 or DF_MOE_F32");
  return DF_MOE_OK;
}

int unpermute(int device, const void* rows, int dtype, int64_t n_rows, int64_t ldr,
              const int32_t* pos, const float* weights, int64_t T, int k, int64_t H, void* y,
              int64_t ldy, void* stream) {
  int rc = check_routing(T, k, H);
  if (!rc) rc = check_float_dtype(dtype);
  if (!rc) rc = check_ld("the rows' distance", &ldr, H);
  if (!rc) rc = check_ld("the output's distance", &ldy, H);
  if (rc) return rc;
  if (n_rows < 0) return fail(DF_MOE_EINVAL, "n_rows is negative");
  if (T == 0) return DF_MOE_OK;
  if ((!rows && n_rows > 0) || !pos || !y) return fail(DF_MOE_EINVAL, "rows, pos and the output are required");
  const int size = dfm::dtype_bytes(dtype);
  if (off(rows, size) || off(y, size) || off(pos, 4) || off(weights, 4))
    return fail(DF_MOE_EINVAL, "an array is not aligned to its elements");
  if (T > kMaxRows / ((H + 127) / 128)) return fail(DF_MOE_ERANGE, "T * H is too large");
  OnDevice on(device);
  if (on.rc()) return on.rc();
  const dfm::UnpermuteArgs a{rows, pos, weights, y, (int)T, k, (int)H, n_rows, ldr, ldy};
  return launched("unpermute launch", dfm::launch_unpermute(a, dtype, on.sms(), (cudaStream_t)stream));
}

}  // namespace

extern "C" {

DF_MOE_API size_t df_moe_permute_workspace(int64_t T, int32_t k, int32_t E) {
  if (T < 1 || k < 1 || k > dfm::kOpsMaxTopK || E < 1 || E > dfm::kOpsMaxExperts || T > kMaxRows / k)
    return 0;
  return dfm::permute_workspace_bytes(T, k, E);
}

DF_MOE_API int df_moe_permute(int device, const int32_t* ids, int64_t T, int32_t k, int32_t E,
                              const void* x, int32_t dtype, int64_t H, int64_t ldx,
                              const float* scales, int32_t n_scales, int64_t ld_scales, void* rows,
                              int64_t ldr, float* rows_scales, int64_t ld_rows_scales,
                              int32_t* offs, int32_t* pos, int32_t* src, void* workspace,
                              size_t workspace_bytes, void* stream) {
  int rc = check_routing(T, k, H);
  if (rc) return rc;
  if (E < 1 || E > dfm::kOpsMaxExperts) return fail(DF_MOE_EINVAL, "E must be in [1, 1024]");
  if (dtype < DF_MOE_BF16 || dtype > DF_MOE_E4M3) return fail(DF_MOE_EINVAL, "unknown dtype");
  if (n_scales < 0 || n_scales > kMaxHidden) return fail(DF_MOE_EINVAL, "n_scales must be in [0, 262144]");
  if ((rc = check_ld("ldx", &ldx, H)) || (rc = check_ld("ldr", &ldr, H)) ||
      (rc = check_ld("ld_scales", &ld_scales, n_scales)) ||
      (rc = check_ld("ld_rows_scales", &ld_rows_scales, n_scales)))
    return rc;
  if (!offs) return fail(DF_MOE_EINVAL, "offs is required");
  if (off(offs, 4)) return fail(DF_MOE_EINVAL, "an array is not aligned to its elements");
  if (T == 0) {  // no token: every expert's segment is empty
    OnDevice on(device);
    if (on.rc()) return on.rc();
    return launched("permute", cudaMemsetAsync(offs, 0, sizeof(int32_t) * ((size_t)E + 1), (cudaStream_t)stream));
  }
  if (!ids || !x || !rows || !pos || !src)
    return fail(DF_MOE_EINVAL, "ids, x, rows, offs, pos and src are required");
  if (n_scales && (!scales || !rows_scales))
    return fail(DF_MOE_EINVAL, "n_scales needs scales and rows_scales");
  const int size = dfm::dtype_bytes(dtype);
  if (off(x, size) || off(rows, size) || off(ids, 4) || off(pos, 4) || off(src, 4) ||
      (n_scales && (off(scales, 4) || off(rows_scales, 4))))
    return fail(DF_MOE_EINVAL, "an array is not aligned to its elements");
  const size_t need = dfm::permute_workspace_bytes(T, k, E);
  if (need && (!workspace || workspace_bytes < need || off(workspace, 4)))
    return fail(DF_MOE_EINVAL, "T * k = %lld needs a workspace of %zu bytes (4-byte aligned)",
                (long long)T * k, need);
  OnDevice on(device);
  if (on.rc()) return on.rc();
  dfm::PermuteArgs a{};
  a.ids = ids;
  a.T = (int)T;
  a.k = k;
  a.E = E;
  a.x = static_cast<const char*>(x);
  a.rows = static_cast<char*>(rows);
  a.bytes = H * size;
  a.ldx = ldx * size;
  a.ldr = ldr * size;
  a.xs = scales;
  a.rows_s = rows_scales;
  a.n_scales = n_scales;
  a.ldxs = ld_scales;
  a.ldrs = ld_rows_scales;
  a.offs = offs;
  a.pos = pos;
  a.src = src;
  return launched("permute launch", dfm::launch_permute(a, workspace, on.sms(), (cudaStream_t)stream));
}

DF_MOE_API int df_moe_permute_grad(int device, const void* drows, int32_t dtype, int64_t n_rows,
                                   int64_t ldr, const int32_t* pos, int64_t T, int32_t k,
                                   int64_t H, void* dx, int64_t ldx, void* stream) {
  return unpermute(device, drows, dtype, n_rows, ldr, pos, nullptr, T, k, H, dx, ldx, stream);
}

DF_MOE_API int df_moe_unpermute(int device, const void* rows, int32_t dtype, int64_t n_rows,
                                int64_t ldr, const int32_t* pos, const float* weights, int64_t T,
                                int32_t k, int64_t H, void* y, int64_t ldy, void* stream) {
  if (!weights && T > 0) return fail(DF_MOE_EINVAL, "weights are required");
  return unpermute(device, rows, dtype, n_rows, ldr, pos, weights, T, k, H, y, ldy, stream);
}

DF_MOE_API int df_moe_unpermute_grad(int device, const void* dy, int64_t lddy, const void* rows,
                                     int32_t dtype, int64_t n_rows, int64_t ldr,
                                     const int32_t* pos, const float* weights, int64_t T,
                                     int32_t k, int64_t H, void* drows, int64_t lddr,
                                     float* dweights, void* stream) {
  int rc = check_routing(T, k, H);
  if (!rc) rc = check_float_dtype(dtype);
  if (!rc) rc = check_ld("ldr", &ldr, H);
  if (!rc) rc = check_ld("lddy", &lddy, H);
  if (!rc) rc = check_ld("lddr", &lddr, H);
  if (rc) return rc;
  if (n_rows < 0) return fail(DF_MOE_EINVAL, "n_rows is negative");
  if (T == 0) return DF_MOE_OK;
  if (!dy || !pos || !weights || !dweights || (n_rows > 0 && (!rows || !drows)))
    return fail(DF_MOE_EINVAL, "dy, rows, pos, weights, drows and dweights are required");
  const int size = dfm::dtype_bytes(dtype);
  if (off(dy, size) || off(rows, size) || off(drows, size) || off(pos, 4) || off(weights, 4) || off(dweights, 4))
    return fail(DF_MOE_EINVAL, "an array is not aligned to its elements");
  OnDevice on(device);
  if (on.rc()) return on.rc();
  const dfm::UnpermuteGradArgs a{dy,     rows, pos, weights, drows, dweights, (int)T, k,
                                 (int)H, n_rows, lddy, ldr,  lddr};
  return launched("unpermute gradient launch",
                  dfm::launch_unpermute_grad(a, dtype, on.sms(), (cudaStream_t)stream));
}

DF_MOE_API int df_moe_fp8_quantize(int device, const void* x, int32_t dtype, int64_t M, int64_t K,
                                   int64_t ldx, uint8_t* codes, int64_t ldc, float* scales,
                                   int64_t lds, void* stream) {
  int rc = check_float_dtype(dtype);
  if (rc) return rc;
  if (M < 0) return fail(DF_MOE_EINVAL, "M = %lld is negative", (long long)M);
  if (K < 1 || K > kMaxHidden) return fail(DF_MOE_EINVAL, "K must be in [1, 262144]");
  const int64_t nb = (K + 127) / 128;
  if ((rc = check_ld("ldx", &ldx, K)) || (rc = check_ld("ldc", &ldc, K)) ||
      (rc = check_ld("lds", &lds, nb)))
    return rc;
  if (M == 0) return DF_MOE_OK;
  if (!x || !codes || !scales) return fail(DF_MOE_EINVAL, "x, codes and scales are required");
  if (off(x, dfm::dtype_bytes(dtype)) || off(scales, 4))
    return fail(DF_MOE_EINVAL, "an array is not aligned to its elements");
  if (M > kMaxRows / nb) return fail(DF_MOE_ERANGE, "M * K / 128 must stay below 2^31");
  OnDevice on(device);
  if (on.rc()) return on.rc();
  const dfm::QuantizeArgs a{x, codes, scales, M, (int)K, ldx, ldc, lds};
  return launched("quantize launch",
                  dfm::launch_fp8_quantize(a, dtype, on.sms(), (cudaStream_t)stream));
}

DF_MOE_API int df_moe_test_fp8_give_up(int32_t role) {
  if (role < 0 || role > 4) return fail(DF_MOE_EINVAL, "role must be in [0, 4]");
  give_up_next = role;
  return DF_MOE_OK;
}

DF_MOE_API int df_moe_fp8_matmul(int device, const uint8_t* x, int64_t ldx, const float* xs,
                                 int64_t ldxs, const uint8_t* w, int64_t ldw, const float* ws,
                                 const int32_t* offs, int32_t G, int64_t M, int64_t N, int64_t K,
                                 int32_t transposed, void* y, int32_t dtype, int64_t ldy,
                                 uint32_t* status, void* stream) {
  int rc = check_float_dtype(dtype);
  if (rc) return rc;
  if (M < 0) return fail(DF_MOE_EINVAL, "M = %lld is negative", (long long)M);
  if (M > kMaxRows - 256) return fail(DF_MOE_ERANGE, "M must stay below 2^31 - 256");
  if (N < 1 || N > kMaxHidden) return fail(DF_MOE_EINVAL, "N must be in [1, 262144]");
  if (K < 1 || K > kMaxHidden) return fail(DF_MOE_EINVAL, "K must be in [1, 262144]");
  if (G < 1 || G > dfm::kOpsMaxExperts) return fail(DF_MOE_EINVAL, "G must be in [1, 1024]");
  if (!offs && G != 1) return fail(DF_MOE_EINVAL, "offs is required for more than one group");
  const int64_t cols = transposed ? N : K;
  // rows start on 16-byte boundaries: the tensor copies' rule
  if (ldx == 0 && K % 16 == 0) ldx = K;
  if (ldw == 0 && cols % 16 == 0) ldw = cols;
  if (ldx < K || ldx % 16) return fail(DF_MOE_EINVAL, "ldx must be a multiple of 16, at least K");
  if (ldw < cols || ldw % 16)
    return fail(DF_MOE_EINVAL, "ldw must be a multiple of 16, at least w's columns");
  if ((rc = check_ld("ldxs", &ldxs, (K + 127) / 128)) || (rc = check_ld("ldy", &ldy, N))) return rc;
  if (M == 0) return DF_MOE_OK;
  if (!x || !xs || !w || !ws || !y) return fail(DF_MOE_EINVAL, "x, xs, w, ws and y are required");
  if (off(x, 16) || off(w, 16)) return fail(DF_MOE_EINVAL, "x and w must be 16-byte aligned");
  if (off(xs, 4) || off(ws, 4) || off(offs, 4) || off(status, 4) || off(y, dfm::dtype_bytes(dtype)))
    return fail(DF_MOE_EINVAL, "an array is not aligned to its elements");
  if (ldx >= (1ll << 39) || ldw >= (1ll << 39) || ldw * (transposed ? K : N) >= (1ll << 39))
    return fail(DF_MOE_ERANGE, "a row distance or a group's weights are too large");
  OnDevice on(device);
  if (on.rc()) return on.rc();
  dfm::Fp8MatmulArgs a{};
  a.x = x;
  a.xs = xs;
  a.w = w;
  a.ws = ws;
  a.offs = offs;
  a.y = y;
  a.G = G;
  a.N = (int)N;
  a.K = (int)K;
  a.transposed = transposed ? 1 : 0;
  a.M = M;
  a.ldx = ldx;
  a.ldxs = ldxs;
  a.ldw = ldw;
  a.ldy = ldy;
  a.status = status;
  a.give_up = give_up_next;
  give_up_next = 0;
  const char* err = dfm::launch_fp8_matmul(a, dtype, on.sms(), (cudaStream_t)stream);
  if (err) {
    (void)cudaGetLastError();
    return fail(DF_MOE_ECUDA, "fp8 product: %s", err);
  }
  return DF_MOE_OK;
}

}  // extern "C"
