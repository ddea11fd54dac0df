// ops.cu — C entry points of the expert-path operators (no handle): argument
// checks, the device, the launch. They keep nothing between calls but the
// SM count of each device (and what the test hook asks of the next product).
#include <cuda_runtime.h>

#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <type_traits>
#include <utility>

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

thread_local int give_up_next = 0, gemm_give_up_next = 0;

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

bool is_16_bit(int dtype) { return dtype == DF_MOE_BF16 || dtype == DF_MOE_F16; }

// Rows of a product's operand start on 16-byte boundaries (the tensor copies'
// rule) and are less than 2^40 bytes apart.
int check_operand(const char* name, const void* p, int64_t* ld, int64_t n) {
  if (*ld == 0 && n % 8 == 0) *ld = n;
  if (*ld < n || *ld % 8) return fail(DF_MOE_EINVAL, "ld of %s must be a multiple of 8, at least its row's length", name);
  if (*ld >= (1ll << 39)) return fail(DF_MOE_ERANGE, "ld of %s is too large", name);
  if (off(p, 16)) return fail(DF_MOE_EINVAL, "%s must be 16-byte aligned", name);
  return DF_MOE_OK;
}

int check_matmul(int dtype, int64_t M, int64_t N, int64_t K, int act) {
  if (!is_16_bit(dtype)) return fail(DF_MOE_EINVAL, "dtype must be DF_MOE_BF16 or DF_MOE_F16");
  if (M < 0) return fail(DF_MOE_EINVAL, "M = %lld is negative", (long long)M);
  if (M > kMaxRows - 256) return fail(DF_MOE_ERANGE, "M must stay below 2^31 - 256");
  if (N < 1 || N > kMaxHidden) return fail(DF_MOE_EINVAL, "N must be in [1, 262144]");
  if (K < 1 || K > kMaxHidden) return fail(DF_MOE_EINVAL, "K must be in [1, 262144]");
  if (act < DF_MOE_ACT_NONE || act > DF_MOE_ACT_SWIGLU) return fail(DF_MOE_EINVAL, "unknown activation");
  return DF_MOE_OK;
}

int gemm_done(const char* what, const char* err) {
  if (!err) return DF_MOE_OK;
  (void)cudaGetLastError();
  return fail(DF_MOE_ECUDA, "%s: %s", what, err);
}

// Sizes and types that the norm and its gradient share.
int check_norm(int dtype, int wtype, int64_t T, int64_t H, int gate_kind, float eps) {
  int rc = check_float_dtype(dtype);
  if (rc) return rc;
  if (wtype != DF_MOE_F32 && wtype != dtype) return fail(DF_MOE_EINVAL, "weight_dtype must be dtype or DF_MOE_F32");
  if (T < 0) return fail(DF_MOE_EINVAL, "T = %lld is negative", (long long)T);
  if (T > kMaxRows) return fail(DF_MOE_ERANGE, "T must stay below 2^31");
  if (H < 1 || H > dfm::kNormMaxHidden) return fail(DF_MOE_EINVAL, "H must be in [1, 32768]");
  if (gate_kind < DF_MOE_GATE_NONE || gate_kind > DF_MOE_GATE_FULL) return fail(DF_MOE_EINVAL, "unknown gate_kind");
  if (!(eps >= 1e-30f && eps <= 3e38f)) return fail(DF_MOE_EINVAL, "eps must be in [1e-30, 3e38]");
  return DF_MOE_OK;
}

// An array of rows that may be absent.
int check_rows(const char* name, const void* p, int64_t* ld, int64_t n, int size) {
  if (!p) return DF_MOE_OK;
  if (*ld == 0) *ld = n;
  if (*ld < n) return fail(DF_MOE_EINVAL, "ld of %s is below the row's length", name);
  if (off(p, size)) return fail(DF_MOE_EINVAL, "%s is not aligned to its elements", name);
  return DF_MOE_OK;
}

// A call's arguments as 8-byte values, in order: a float as a double.
template <typename A>
A packed(const int64_t& v) {
  if constexpr (std::is_pointer<A>::value) {
    return reinterpret_cast<A>(static_cast<uintptr_t>(v));
  } else if constexpr (std::is_same<A, float>::value) {
    double d;
    memcpy(&d, &v, sizeof d);
    return (float)d;
  } else {
    return static_cast<A>(v);
  }
}
// Whether an integer is its argument's: a cast cuts none off.
template <typename A>
bool fits(const int64_t& v) {
  if constexpr (std::is_integral<A>::value) return static_cast<int64_t>(static_cast<A>(v)) == v && (std::is_signed<A>::value || v >= 0);
  return true;
}
template <typename... A, size_t... I>
int call_packed(int (*f)(A...), const int64_t* args, std::index_sequence<I...>) {
  int64_t v[sizeof...(A)];
  memcpy(v, args, sizeof v);
  if (!(fits<A>(v[I]) && ...)) return fail(DF_MOE_EINVAL, "an integer does not fit the argument that it stands for");
  return f(packed<A>(v[I])...);
}
template <typename... A>
int call_packed(int (*f)(A...), const int64_t* args) {
  return call_packed(f, args, std::index_sequence_for<A...>());
}

int check_balance(int dtype, int64_t T, int64_t E, int k, const int32_t* offs, int64_t S, int score, float coef, float z_coef) {
  int rc = check_float_dtype(dtype);
  if (rc) return rc;
  if (T < 0) return fail(DF_MOE_EINVAL, "T = %lld is negative", (long long)T);
  if (E < 1 || E > dfm::kOpsMaxExperts) return fail(DF_MOE_EINVAL, "E must be in [1, 1024]");
  if (k < 1 || k > dfm::kOpsMaxTopK) return fail(DF_MOE_EINVAL, "k must be in [1, 32]");
  if (T > kMaxRows / k) return fail(DF_MOE_ERANGE, "T * k must stay below 2^31");
  if (S < 1) return fail(DF_MOE_EINVAL, "S must be at least 1");
  if (S > (1 << 20)) return fail(DF_MOE_ERANGE, "S must be at most 2^20");
  if (!offs && S != 1) return fail(DF_MOE_EINVAL, "offs is required for more than one sequence");
  if (score != DF_MOE_SCORE_SOFTMAX && score != DF_MOE_SCORE_SIGMOID) return fail(DF_MOE_EINVAL, "unknown score");
  if (!(coef - coef == 0.f) || !(z_coef - z_coef == 0.f)) return fail(DF_MOE_EINVAL, "coef and z_coef must be finite");
  return DF_MOE_OK;
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

DF_MOE_API int df_moe_test_matmul_give_up(int32_t role) {
  if (role < 0 || role > 3) return fail(DF_MOE_EINVAL, "role must be in [0, 3]");
  gemm_give_up_next = role;
  return DF_MOE_OK;
}

DF_MOE_API int df_moe_matmul(int device, const void* x, int64_t ldx, const void* w, int64_t ldw,
                             int32_t dtype, int64_t M, int64_t N, int64_t K, const void* bias,
                             int32_t act, const void* residual, int64_t ldr, void* pre, int64_t ldp,
                             void* y, int32_t out_dtype, int64_t ldy, uint32_t* status, void* stream) {
  int rc = check_matmul(dtype, M, N, K, act);
  if (rc) return rc;
  if (out_dtype != dtype && out_dtype != DF_MOE_F32) return fail(DF_MOE_EINVAL, "out_dtype must be dtype or DF_MOE_F32");
  const int64_t wide = act == DF_MOE_ACT_SWIGLU ? 2 * N : N;
  const int so = dfm::dtype_bytes(out_dtype);
  if ((rc = check_operand("x", x, &ldx, K)) || (rc = check_operand("w", w, &ldw, K)) ||
      (rc = check_ld("ldy", &ldy, N)) || (rc = check_rows("residual", residual, &ldr, N, so)) ||
      (rc = check_rows("pre", pre, &ldp, wide, 2)))
    return rc;
  if (M == 0) return DF_MOE_OK;
  if (!x || !w || !y) return fail(DF_MOE_EINVAL, "x, w and y are required");
  if (off(y, so) || off(bias, 2) || off(status, 4)) return fail(DF_MOE_EINVAL, "an array is not aligned to its elements");
  OnDevice on(device);
  if (on.rc()) return on.rc();
  dfm::GemmArgs a{};
  a.row = {x, ldx, false};
  a.col = {w, ldw, false};
  a.R = M;
  a.K = K;
  a.C = (int)N;
  a.in = dtype;
  a.out = out_dtype;
  a.act = act;
  a.bias = bias;
  a.residual = residual;
  a.pre = pre;
  a.y = y;
  a.ldr = ldr;
  a.ldp = ldp;
  a.ldy = ldy;
  a.status = status;
  a.give_up = gemm_give_up_next;
  gemm_give_up_next = 0;
  return gemm_done("product", dfm::launch_gemm(a, on.sms(), (cudaStream_t)stream));
}

DF_MOE_API int df_moe_matmul_grad(int device, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                  const void* w, int64_t ldw, int32_t dtype, int64_t M, int64_t N,
                                  int64_t K, int32_t act, const void* pre, int64_t ldp, void* dz,
                                  int64_t lddz, void* dx, int64_t lddx, void* dw, int64_t lddw,
                                  void* dbias, int32_t grad_dtype, uint32_t* status, void* stream) {
  int rc = check_matmul(dtype, M, N, K, act);
  if (rc) return rc;
  if (grad_dtype != dtype && grad_dtype != DF_MOE_F32) return fail(DF_MOE_EINVAL, "grad_dtype must be dtype or DF_MOE_F32");
  if (!dx && !dw && !dbias && !(dz && act)) return fail(DF_MOE_EINVAL, "none of dx, dw and dbias is wanted");
  const int64_t wide = act == DF_MOE_ACT_SWIGLU ? 2 * N : N;
  const int sg = dfm::dtype_bytes(grad_dtype);
  const bool products = dx || dw;
  if ((rc = check_rows("dx", dx, &lddx, K, 2)) || (rc = check_rows("dw", dw, &lddw, K, sg))) return rc;
  if (off(dbias, sg) || off(status, 4)) return fail(DF_MOE_EINVAL, "an array is not aligned to its elements");
  if (act) {
    if (M > 0 && (!pre || !dz)) return fail(DF_MOE_EINVAL, "an activation needs pre and dz");
    if ((rc = check_rows("pre", pre, &ldp, wide, 2)) || (rc = check_rows("dy", dy, &lddy, N, 2)) ||
        (rc = products ? check_operand("dz", dz, &lddz, wide) : check_rows("dz", dz, &lddz, wide, 2)))
      return rc;
  } else if ((rc = products ? check_operand("dy", dy, &lddy, N) : check_rows("dy", dy, &lddy, N, 2))) {
    return rc;
  }
  if ((dw && (rc = check_operand("x", x, &ldx, K))) || (dx && (rc = check_operand("w", w, &ldw, K)))) return rc;
  if (M > 0 && (!dy || (dw && !x) || (dx && !w))) return fail(DF_MOE_EINVAL, "dy is required, x for dw and w for dx");
  OnDevice on(device);
  cudaStream_t s = (cudaStream_t)stream;
  if (M == 0) {  // sums over no rows
    if (!dw && !dbias) return DF_MOE_OK;
    if (on.rc()) return on.rc();
    cudaError_t e = cudaSuccess;
    if (dw) e = cudaMemset2DAsync(dw, (size_t)(lddw * sg), 0, (size_t)(K * sg), (size_t)wide, s);
    if (dbias && e == cudaSuccess) e = cudaMemsetAsync(dbias, 0, (size_t)(wide * sg), s);
    return launched("product gradient", e);
  }
  if (on.rc()) return on.rc();
  if (act || dbias) {
    dfm::ActGradArgs g{};
    g.dy = dy;
    g.pre = pre;
    g.dz = dz;
    g.dbias = dbias;
    g.M = M;
    g.lddy = lddy;
    g.ldp = ldp;
    g.lddz = lddz;
    g.N = (int)N;
    g.in = dtype;
    g.grad = grad_dtype;
    g.act = act;
    g.follows = products;
    if ((rc = gemm_done("activation gradient", dfm::launch_act_grad(g, on.sms(), s)))) return rc;
  }
  dfm::GemmArgs a{};
  a.in = dtype;
  a.status = status;
  const int64_t columns = (K + 127) / 128;  // of tiles, of both
  const dfm::GemmOperand grad = {act ? dz : dy, act ? lddz : lddy, false};
  if (dx) {
    a.row = grad;
    a.col = {w, ldw, true};
    a.R = M;
    a.K = wide;
    a.C = (int)K;
    a.out = dtype;
    a.y = dx;
    a.ldy = lddx;
    a.order = dw ? dfm::kGemmFirst : dfm::kGemmAlone;
    a.beside = dw ? ((wide + 63) / 64) * columns : 0;
    a.give_up = gemm_give_up_next;
    gemm_give_up_next = 0;
    if ((rc = gemm_done("gradient of x", dfm::launch_gemm(a, on.sms(), s)))) return rc;
  }
  if (dw) {
    a.row = grad;
    a.row.mn = true;
    a.col = {x, ldx, true};
    a.R = wide;
    a.K = M;
    a.C = (int)K;
    a.out = grad_dtype;
    a.y = dw;
    a.ldy = lddw;
    a.order = dx ? dfm::kGemmSecond : dfm::kGemmAlone;
    a.beside = dx ? ((M + 63) / 64) * columns : 0;
    a.give_up = gemm_give_up_next;
    gemm_give_up_next = 0;
    if ((rc = gemm_done("gradient of w", dfm::launch_gemm(a, on.sms(), s)))) return rc;
  }
  return DF_MOE_OK;
}

DF_MOE_API int df_moe_block_norm(int device, const void* u, int64_t ldu, int32_t post,
                                 const void* post_w, int32_t gate_kind, const void* gate, int64_t ldg,
                                 const void* residual, int64_t ldr, float residual_scale,
                                 const void* pre_w, float eps, int64_t T, int64_t H, int32_t dtype,
                                 int32_t weight_dtype, void* h, int64_t ldh, void* n, int64_t ldn,
                                 void* stream) {
  int rc = check_norm(dtype, weight_dtype, T, H, gate_kind, eps);
  if (rc) return rc;
  const int size = dfm::dtype_bytes(dtype), ws = dfm::dtype_bytes(weight_dtype);
  if ((rc = check_rows("u", u, &ldu, H, size)) || (rc = check_rows("residual", residual, &ldr, H, size)) ||
      (rc = check_rows("h", h, &ldh, H, size)) || (rc = check_rows("n", n, &ldn, H, size)))
    return rc;
  if (gate_kind == DF_MOE_GATE_FULL && (rc = check_rows("gate", gate, &ldg, H, size))) return rc;
  if (T == 0) return DF_MOE_OK;
  if (!u && !residual) return fail(DF_MOE_EINVAL, "u or residual is required");
  if (!h && !n) return fail(DF_MOE_EINVAL, "h or n is required");
  if (gate_kind != DF_MOE_GATE_NONE && (!gate || !u)) return fail(DF_MOE_EINVAL, "a gate needs its array and u");
  if ((post || post_w) && !u) return fail(DF_MOE_EINVAL, "the norm after a block needs u");
  if (post_w && !post) return fail(DF_MOE_EINVAL, "post_w without post");
  if (off(post_w, ws) || off(pre_w, ws) || (gate_kind == DF_MOE_GATE_CHANNEL && off(gate, ws)) ||
      (gate_kind == DF_MOE_GATE_TOKEN && off(gate, 4)))
    return fail(DF_MOE_EINVAL, "an array is not aligned to its elements");
  OnDevice on(device);
  if (on.rc()) return on.rc();
  dfm::BlockNormArgs a{};
  a.u = u;
  a.post_w = post_w;
  a.gate = gate;
  a.residual = residual;
  a.pre_w = pre_w;
  a.h = h;
  a.n = n;
  a.T = T;
  a.ldu = ldu;
  a.ldg = ldg;
  a.ldr = ldr;
  a.ldh = ldh;
  a.ldn = ldn;
  a.H = (int)H;
  a.post = post;
  a.gate_kind = gate_kind;
  a.scale = residual_scale;
  a.eps = eps;
  return launched("block norm launch", dfm::launch_block_norm(a, dtype, weight_dtype, on.sms(), (cudaStream_t)stream));
}

DF_MOE_API size_t df_moe_block_norm_grad_workspace(int64_t T, int64_t H) {
  if (T < 1 || T > kMaxRows || H < 1 || H > dfm::kNormMaxHidden) return 0;
  return dfm::block_norm_grad_workspace_bytes(T, (int)H);
}

DF_MOE_API int df_moe_block_norm_grad(int device, const void* dh, int64_t lddh, const void* dn,
                                      int64_t lddn, const void* u, int64_t ldu, const void* h,
                                      int64_t ldh, int32_t post, const void* post_w,
                                      int32_t gate_kind, const void* gate, int64_t ldg,
                                      float residual_scale, const void* pre_w, float eps, int64_t T,
                                      int64_t H, int32_t dtype, int32_t weight_dtype, void* du,
                                      int64_t lddu, void* dresidual, int64_t lddr, float* dpost_w,
                                      void* dgate, int64_t lddg, float* dpre_w, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  int rc = check_norm(dtype, weight_dtype, T, H, gate_kind, eps);
  if (rc) return rc;
  const int size = dfm::dtype_bytes(dtype), ws = dfm::dtype_bytes(weight_dtype);
  if ((rc = check_rows("dh", dh, &lddh, H, size)) || (rc = check_rows("dn", dn, &lddn, H, size)) ||
      (rc = check_rows("u", u, &ldu, H, size)) || (rc = check_rows("h", h, &ldh, H, size)) ||
      (rc = check_rows("du", du, &lddu, H, size)) || (rc = check_rows("dresidual", dresidual, &lddr, H, size)))
    return rc;
  if (gate_kind == DF_MOE_GATE_FULL &&
      ((rc = check_rows("gate", gate, &ldg, H, size)) || (rc = check_rows("dgate", dgate, &lddg, H, size))))
    return rc;
  if (!du && !dresidual && !dpost_w && !dgate && !dpre_w) return fail(DF_MOE_EINVAL, "no gradient is wanted");
  if (dpost_w && !post) return fail(DF_MOE_EINVAL, "dpost_w without post");
  if (dgate && gate_kind == DF_MOE_GATE_NONE) return fail(DF_MOE_EINVAL, "dgate without a gate");
  if (post_w && !post) return fail(DF_MOE_EINVAL, "post_w without post");
  if (off(dpost_w, 4) || off(dpre_w, 4) || (gate_kind != DF_MOE_GATE_FULL && off(dgate, 4)) || off(post_w, ws) ||
      off(pre_w, ws) || (gate_kind == DF_MOE_GATE_CHANNEL && off(gate, ws)) ||
      (gate_kind == DF_MOE_GATE_TOKEN && off(gate, 4)))
    return fail(DF_MOE_EINVAL, "an array is not aligned to its elements");
  const bool channel = dgate && gate_kind == DF_MOE_GATE_CHANNEL;
  if (T > 0) {
    if (!dh && !dn) return fail(DF_MOE_EINVAL, "dh or dn is required");
    if (dn && !h) return fail(DF_MOE_EINVAL, "dn needs h");
    if ((pre_w || dpre_w) && !dn) return fail(DF_MOE_EINVAL, "pre_w and dpre_w need dn");
    if ((post || gate_kind != DF_MOE_GATE_NONE || du) && !u)
      return fail(DF_MOE_EINVAL, "the norm after a block, a gate and du need u");
    if (gate_kind != DF_MOE_GATE_NONE && !gate) return fail(DF_MOE_EINVAL, "a gate needs its array");
    const size_t need = dpost_w || dpre_w || channel ? dfm::block_norm_grad_workspace_bytes(T, (int)H) : 0;
    if (need && (!workspace || workspace_bytes < need || off(workspace, 16)))
      return fail(DF_MOE_EINVAL, "the gradients of weights need a workspace of %zu bytes (16-byte aligned)", need);
  }
  OnDevice on(device);
  cudaStream_t s = (cudaStream_t)stream;
  if (T == 0) {  // sums over no rows
    if (!dpost_w && !dpre_w && !channel) return DF_MOE_OK;
    if (on.rc()) return on.rc();
    cudaError_t e = cudaSuccess;
    if (dpost_w) e = cudaMemsetAsync(dpost_w, 0, (size_t)H * 4, s);
    if (dpre_w && e == cudaSuccess) e = cudaMemsetAsync(dpre_w, 0, (size_t)H * 4, s);
    if (channel && e == cudaSuccess) e = cudaMemsetAsync(dgate, 0, (size_t)H * 4, s);
    return launched("block norm gradient", e);
  }
  if (on.rc()) return on.rc();
  dfm::BlockNormGradArgs a{};
  a.dh = dh;
  a.dn = dn;
  a.u = u;
  a.h = h;
  a.post_w = post_w;
  a.gate = gate;
  a.pre_w = pre_w;
  a.du = du;
  a.dresidual = dresidual;
  a.dgate = dgate;
  a.dpost_w = dpost_w;
  a.dpre_w = dpre_w;
  a.T = T;
  a.lddh = lddh;
  a.lddn = lddn;
  a.ldu = ldu;
  a.ldh = ldh;
  a.ldg = ldg;
  a.lddu = lddu;
  a.lddr = lddr;
  a.lddg = lddg;
  a.H = (int)H;
  a.post = post;
  a.gate_kind = gate_kind;
  a.scale = residual_scale;
  a.eps = eps;
  return launched("block norm gradient launch",
                  dfm::launch_block_norm_grad(a, dtype, weight_dtype, workspace, on.sms(), s));
}

DF_MOE_API size_t df_moe_balance_loss_workspace(int64_t T, int32_t E, int64_t S) {
  if (T < 1 || T > kMaxRows || E < 1 || E > dfm::kOpsMaxExperts || S < 1 || S > (1 << 20)) return 0;
  return dfm::balance_workspace_bytes(T, E, S);
}

DF_MOE_API int df_moe_balance_loss(int device, const void* logits, int32_t dtype, int64_t ldl,
                                   const int32_t* ids, int64_t T, int32_t E, int32_t k,
                                   const int32_t* offs, int64_t S, const uint8_t* mask, int32_t score,
                                   float coef, float z_coef, float* loss, int32_t* counts,
                                   int32_t* tokens, float* probs, void* workspace,
                                   size_t workspace_bytes, uint32_t* status, void* stream) {
  int rc = check_balance(dtype, T, E, k, offs, S, score, coef, z_coef);
  if (rc) return rc;
  if ((rc = check_ld("ldl", &ldl, E))) return rc;
  if (!loss || !counts || !tokens) return fail(DF_MOE_EINVAL, "loss, counts and tokens are required");
  if (off(loss, 4) || off(counts, 4) || off(tokens, 4) || off(probs, 4) || off(ids, 4) || off(offs, 4) ||
      off(status, 4) || off(logits, dfm::dtype_bytes(dtype)))
    return fail(DF_MOE_EINVAL, "an array is not aligned to its elements");
  if (T > 0) {
    if (!logits || !ids) return fail(DF_MOE_EINVAL, "logits and ids are required");
    const size_t need = dfm::balance_workspace_bytes(T, E, S);
    if (!workspace || workspace_bytes < need || off(workspace, 16))
      return fail(DF_MOE_EINVAL, "the call needs a workspace of %zu bytes (16-byte aligned)", need);
  }
  OnDevice on(device);
  if (on.rc()) return on.rc();
  cudaStream_t s = (cudaStream_t)stream;
  if (T == 0) {
    cudaError_t e = cudaMemsetAsync(loss, 0, (size_t)S * 4, s);
    if (e == cudaSuccess) e = cudaMemsetAsync(counts, 0, (size_t)S * E * 4, s);
    if (e == cudaSuccess) e = cudaMemsetAsync(tokens, 0, (size_t)S * 4, s);
    if (e == cudaSuccess && probs) e = cudaMemsetAsync(probs, 0, (size_t)S * E * 4, s);
    return launched("balance loss", e);
  }
  dfm::BalanceArgs a{};
  a.logits = logits;
  a.ids = ids;
  a.offs = offs;
  a.mask = mask;
  a.loss = loss;
  a.probs = probs;
  a.counts = counts;
  a.tokens = tokens;
  a.status = status;
  a.T = T;
  a.ldl = ldl;
  a.E = E;
  a.k = k;
  a.S = (int)S;
  a.sigmoid = score == DF_MOE_SCORE_SIGMOID;
  a.coef = coef;
  a.z_coef = z_coef;
  return launched("balance loss launch", dfm::launch_balance_loss(a, dtype, workspace, s));
}

DF_MOE_API int df_moe_balance_loss_grad(int device, const float* dloss, const void* logits,
                                        int32_t dtype, int64_t ldl, const int32_t* ids, int64_t T,
                                        int32_t E, int32_t k, const int32_t* offs, int64_t S,
                                        const uint8_t* mask, int32_t score, float coef, float z_coef,
                                        const int32_t* counts, const int32_t* tokens,
                                        const float* weights, const float* dweights, void* dlogits,
                                        int64_t lddl, void* stream) {
  int rc = check_balance(dtype, T, E, k, offs, S, score, coef, z_coef);
  if (rc) return rc;
  if ((rc = check_ld("ldl", &ldl, E)) || (rc = check_ld("lddl", &lddl, E))) return rc;
  if (T == 0) return DF_MOE_OK;
  if (!dloss || !logits || !counts || !tokens || !dlogits)
    return fail(DF_MOE_EINVAL, "dloss, logits, counts, tokens and dlogits are required");
  if (!weights != !dweights || (weights && !ids)) return fail(DF_MOE_EINVAL, "weights, dweights and their ids go together");
  const int size = dfm::dtype_bytes(dtype);
  if (off(dloss, 4) || off(logits, size) || off(dlogits, size) || off(ids, 4) || off(offs, 4) || off(counts, 4) ||
      off(tokens, 4) || off(weights, 4) || off(dweights, 4))
    return fail(DF_MOE_EINVAL, "an array is not aligned to its elements");
  OnDevice on(device);
  if (on.rc()) return on.rc();
  dfm::BalanceGradArgs a{};
  a.dloss = dloss;
  a.logits = logits;
  a.ids = ids;
  a.offs = offs;
  a.counts = counts;
  a.tokens = tokens;
  a.mask = mask;
  a.weights = weights;
  a.dweights = dweights;
  a.dlogits = dlogits;
  a.T = T;
  a.ldl = ldl;
  a.lddl = lddl;
  a.E = E;
  a.k = k;
  a.S = (int)S;
  a.sigmoid = score == DF_MOE_SCORE_SIGMOID;
  a.coef = coef;
  a.z_coef = z_coef;
  return launched("balance loss gradient launch", dfm::launch_balance_loss_grad(a, dtype, on.sms(), (cudaStream_t)stream));
}

DF_MOE_API int df_moe_packed(int32_t call, const int64_t* args) {
  switch (call) {
    case DF_MOE_CALL_MATMUL: return call_packed(df_moe_matmul, args);
    case DF_MOE_CALL_MATMUL_GRAD: return call_packed(df_moe_matmul_grad, args);
    case DF_MOE_CALL_BLOCK_NORM: return call_packed(df_moe_block_norm, args);
    case DF_MOE_CALL_BLOCK_NORM_GRAD: return call_packed(df_moe_block_norm_grad, args);
    case DF_MOE_CALL_BALANCE_LOSS: return call_packed(df_moe_balance_loss, args);
    case DF_MOE_CALL_BALANCE_LOSS_GRAD: return call_packed(df_moe_balance_loss_grad, args);
  }
  return fail(DF_MOE_EINVAL, "unknown call %d", call);
}

}  // extern "C"
