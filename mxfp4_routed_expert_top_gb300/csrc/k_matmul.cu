// k_matmul.cu — the gradient of the product's activation and bias, and the choice
// of the product's types; the product is in k_matmul.cuh, a file a pair of types.
#include "k_matmul.cuh"

#include <type_traits>

namespace dfm {
namespace {

// ---- gradient of the activation, and the bias's ---------------------------------
// dz = act'(z) dy (gated: [dy u silu'(g) | dy silu(g)]) and its column sums.
// VEC: a thread has eight columns of a row, a block 64 columns and every
// parts-th 32 rows; else a thread a column, a warp a row, a block 32 columns. A
// few rows' loads go out together (kAgRows). The column sums of the parts meet in the
// cluster's shared memory, in their order.
struct ActGradParams {
  const void *dy, *pre;
  void *dz, *dbias;
  int64_t M, lddy, ldp, lddz;
  int N, grad, parts, follows;
};
constexpr int kAgThreads = 256;

template <typename T>
__device__ __forceinline__ float value(T v);
template <>
__device__ __forceinline__ float value(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float value(__half v) { return __half2float(v); }

// U: rows a thread loads together, as many as the registers of four blocks an SM
// hold: HBM bounds it, and it is the bytes on their way that bring its rate
// (4096 x 2048 swiglu 15.9 us, 5.3 TB/s; twice the rows spill, 26). A kernel an
// activation: with all of them in one it had 128 registers and took 32 us;
// 8192 x 7168 gelu with bias 90 (3.9 TB/s), 226 in one. Without an activation (the
// bias alone, of bf16) 60 bytes of the eight rows spill.
template <bool VEC, int ACT>
constexpr int kAgRows = !VEC || ACT == kActNone ? 8 : ACT == kActSwiglu ? 1 : 2;

template <typename T, bool VEC, int ACT>
__global__ void __launch_bounds__(kAgThreads, 4) act_grad_kernel(const ActGradParams p) {
  constexpr int E = VEC ? 8 : 1;               // columns a thread
  constexpr int LANES = VEC ? 8 : 32;          // threads a row
  constexpr int ROWS = kAgThreads / LANES;     // rows at a time
  constexpr int COLS = E * LANES, U = kAgRows<VEC, ACT>;  // columns a block
  constexpr bool gated = ACT == kActSwiglu, some = ACT != kActNone;
  __shared__ float sums[kAgThreads / 32][2][COLS];
  __shared__ float total[2][COLS];
  const int tid = threadIdx.x, tx = tid % LANES, ty = tid / LANES;
  const int strip = blockIdx.x / p.parts, part = blockIdx.x - strip * p.parts;
  const int c = COLS * strip + E * tx;
  float s0[E], s1[E];
#pragma unroll
  for (int j = 0; j < E; ++j) s0[j] = s1[j] = 0.f;
  pdl_wait();
  // a product of the same call, which waits for the end of this; nothing else may start early
  if (p.follows) pdl_launch_dependents();
  const T* dy = static_cast<const T*>(p.dy) + c;
  const T* pre = static_cast<const T*>(p.pre) + c;
  T* dz = static_cast<T*>(p.dz) + c;
  struct alignas(2 * E) Part { T v[E]; };
  const auto get = [](const T* q) { return *reinterpret_cast<const Part*>(q); };
  if (c < p.N) {
#pragma unroll 1
    for (int64_t r0 = (int64_t)ROWS * part + ty; r0 < p.M; r0 += (int64_t)U * ROWS * p.parts) {
      Part d[U] = {}, z[U] = {}, u[U] = {};
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int64_t r = r0 + (int64_t)i * ROWS * p.parts;
        if (r >= p.M) continue;
        d[i] = get(dy + r * p.lddy);
        if (some) z[i] = get(pre + r * p.ldp);
        if (gated) u[i] = get(pre + r * p.ldp + p.N);
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int64_t r = r0 + (int64_t)i * ROWS * p.parts;
        if (r >= p.M) break;
        float g[E + E % 2], slope[E + E % 2];  // pairs
#pragma unroll
        for (int j = 0; j < E + E % 2; ++j) g[j] = some ? value(z[i].v[j % E]) : 0.f;
        if (some) slope_all(slope, g, ACT);
        Part a, b;
#pragma unroll
        for (int j = 0; j < E; ++j) {
          float x = value(d[i].v[j]);
          if (gated) {
            const float y = x * (g[j] * sigmoid_f(g[j]));
            x *= value(u[i].v[j]);
            s1[j] += y;
            b.v[j] = T(y);
          }
          if (some) x *= slope[j];
          s0[j] += x;
          a.v[j] = T(x);
        }
        if (some) *reinterpret_cast<Part*>(dz + r * p.lddz) = a;
        if (gated) *reinterpret_cast<Part*>(dz + r * p.lddz + p.N) = b;
      }
    }
  }
  if (!p.dbias) return;
#pragma unroll
  for (int j = 0; j < E; ++j) {
#pragma unroll
    for (int o = LANES; o < 32; o <<= 1) {
      s0[j] += __shfl_xor_sync(0xffffffffu, s0[j], o);
      s1[j] += __shfl_xor_sync(0xffffffffu, s1[j], o);
    }
    if ((tid & 31) < LANES) {
      sums[tid >> 5][0][E * tx + j] = s0[j];
      sums[tid >> 5][1][E * tx + j] = s1[j];
    }
  }
  __syncthreads();
  if (tid < 2 * COLS) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kAgThreads / 32; ++w) s += sums[w][tid / COLS][tid % COLS];
    total[tid / COLS][tid % COLS] = s;
  }
  __syncthreads();
  if (p.parts > 1) cluster_barrier();
  const int col = COLS * strip + tid % COLS;
  if (part == 0 && tid < (gated ? 2 * COLS : COLS) && col < p.N) {
    float s = 0.f;
    for (int q = 0; q < p.parts; ++q) {
      float v;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(map_cta(smem_u32(&total[tid / COLS][tid % COLS]), q)) : "memory");
      s += v;
    }
    const int at = tid / COLS * p.N + col;
    if (p.grad == 2) static_cast<float*>(p.dbias)[at] = s;
    else static_cast<T*>(p.dbias)[at] = T(s);
  }
  if (p.parts > 1) {
    __syncwarp();
    cluster_barrier();
  }
}

}  // namespace

const char* launch_gemm(const GemmArgs& a, int sms, cudaStream_t s) {
  if (a.in == 0) return a.out == 2 ? gemm_bf16_f32(a, sms, s) : gemm_bf16(a, sms, s);
  return a.out == 2 ? gemm_f16_f32(a, sms, s) : gemm_f16(a, sms, s);
}

const char* launch_act_grad(const ActGradArgs& a, int sms, cudaStream_t s) {
  ActGradParams p{};
  p.dy = a.dy;
  p.pre = a.pre;
  p.dz = a.dz;
  p.dbias = a.dbias;
  p.M = a.M;
  p.lddy = a.lddy;
  p.ldp = a.ldp;
  p.lddz = a.lddz;
  p.N = a.N;
  p.grad = a.grad;
  p.follows = a.follows;
  const bool some = a.act != kActNone;
  const bool vec = a.N % 8 == 0 && aligned(a.dy, a.lddy, 16, 2) && (!some || (aligned(a.pre, a.ldp, 16, 2) && aligned(a.dz, a.lddz, 16, 2)));
  const int cols = vec ? 64 : 32, rows = 64;  // columns of a block, rows that give it work
  const int64_t strips = (a.N + cols - 1) / cols, most = a.dbias ? 8 : 1 << 20;
  int64_t parts = 1;
  while (2 * parts <= most && rows * parts < a.M && strips * parts < 8 * sms) parts *= 2;
  p.parts = (int)parts;
  const int cluster = a.dbias ? p.parts : 1;
  const auto launch = [&](auto kernel) { return launch_cluster(kernel, strips * parts, kAgThreads, 0, cluster, s, p); };
  const auto by_act = [&](auto t, auto v) {
    using T = decltype(t);
    constexpr bool V = decltype(v)::value;
    switch (a.act) {
      case kActNone: return launch(act_grad_kernel<T, V, kActNone>);
      case kActRelu: return launch(act_grad_kernel<T, V, kActRelu>);
      case kActSilu: return launch(act_grad_kernel<T, V, kActSilu>);
      case kActGelu: return launch(act_grad_kernel<T, V, kActGelu>);
      default: return launch(act_grad_kernel<T, V, kActSwiglu>);
    }
  };
  const auto by_rows = [&](auto t) { return vec ? by_act(t, std::true_type{}) : by_act(t, std::false_type{}); };
  const cudaError_t e = a.in == 0 ? by_rows(__nv_bfloat16{}) : by_rows(__half{});
  return e == cudaSuccess ? nullptr : cudaGetErrorString(e);
}

}  // namespace dfm
