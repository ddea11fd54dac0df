// k_balance.cuh — the router's balance loss with the counts of every expert, and
// the gradient of the logits. For each sequence (rows offs[s] <= t < offs[s + 1]
// whose mask is not zero, n of them)
//
//   p_t = softmax(z_t), or sigmoid(z_t) / sum sigmoid(z_t);  l_t = logsumexp(z_t)
//   count_e = #{(t, j): ids[t][j] = e},  f_e = E count_e / (k n),  P_e = mean p_te
//   loss = coef sum_e f_e P_e + z_coef mean l_t^2
//   dz_te = dloss (coef / n p_te m_te (f_e - sum_j f_j p_tj) + 2 z_coef / n l_t softmax(z_t)_e)
//           + m_te sum_{j: ids[t][j] = e} w_tj (dw_tj - sum_i w_ti dw_ti)
//
// with m = 1 for the softmax and 1 - sigmoid(z) for the sigmoid; the last term
// is the gradient of the routing weights w, the kept scores over their sum.
// sigmoid(z) / sum sigmoid(z) is the softmax of log sigmoid(z), so that scores
// that are all tiny keep their ratios. The logits are read once in either call
// (a row stays in a warp's registers), and HBM bounds the large ones.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cstring>

#include "fastmath.cuh"
#include "internal.h"
#include "ops.h"
#include "pipeline.cuh"

namespace dfm {

// A block has the rows of one chunk and leaves one entry for every sequence it
// meets. Entry chunk + s: along the rows either number only grows and one of
// them does from entry to entry, so no two have the same, and chunks + S are
// enough.
struct Entries {
  float* probs;    // [entries][E]
  int32_t* count;  // [entries][E]
  float2* sums;    // [entries]: rows counted (an int's bits), sum of l^2
};

// How a row lies over a warp: 4, 8 or 16 lanes of eight values (up to 32, 64,
// 128 experts), or all 32 of 8, 16 or 32 values.
inline int balance_shape(int E) { return E <= 32 ? 0 : E <= 64 ? 1 : E <= 128 ? 2 : E <= 256 ? 3 : E <= 512 ? 4 : 5; }
inline int balance_rows_a_warp(int E) { return E <= 32 ? 8 : E <= 64 ? 4 : E <= 128 ? 2 : 1; }

// The rows' kernels of one type each.
cudaError_t balance_rows_bf16(const BalanceArgs& p, const Entries& out, int64_t chunk, int64_t blocks, int alone, cudaStream_t s);
cudaError_t balance_rows_f16(const BalanceArgs& p, const Entries& out, int64_t chunk, int64_t blocks, int alone, cudaStream_t s);
cudaError_t balance_rows_f32(const BalanceArgs& p, const Entries& out, int64_t chunk, int64_t blocks, int alone, cudaStream_t s);
cudaError_t balance_grad_bf16(const BalanceGradArgs& p, int sms, cudaStream_t s);
cudaError_t balance_grad_f16(const BalanceGradArgs& p, int sms, cudaStream_t s);
cudaError_t balance_grad_f32(const BalanceGradArgs& p, int sms, cudaStream_t s);

namespace {

constexpr int kBalThreads = 512, kBalWarps = kBalThreads / 32;
constexpr int kBalBlocks = 152;  // chunks of rows at most, of rows above 512: a block an SM, and few entries to join

template <typename T>
__device__ __forceinline__ float f32_of(T v);
template <>
__device__ __forceinline__ float f32_of(float v) { return v; }
template <>
__device__ __forceinline__ float f32_of(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float f32_of(__half v) { return __half2float(v); }

// A row of E values over L lanes of a warp (which then has 32 / L rows): VEC:
// four side by side, 4 L apart; else one by one, L apart. Element i of lane
// `lane` of the L is column `col(i)`.
template <bool VEC, int NV, int L>
struct Lanes {
  int lane, E;
  __device__ __forceinline__ int col(int i) const { return VEC ? 4 * (lane + L * (i / 4)) + i % 4 : lane + L * i; }
  // Where column c stands among the lanes' float4s [NV][32 lanes], from this
  // row's first lane on.
  static __device__ __forceinline__ int place(int c) {
    const int l = VEC ? c / 4 % L : c % L, i = VEC ? c / (4 * L) * 4 + c % 4 : c / L;
    return 128 * (i / 4) + 4 * l + i % 4;
  }
  template <typename T>
  __device__ __forceinline__ void load(float (&v)[4 * NV], const T* p, float behind) const {
    if (VEC) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = 4 * (lane + L * i);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[4 * i + j] = behind;
        if (c < E) {
          T e[4];
          if (sizeof(T) == 4) {
            const uint4 w = *reinterpret_cast<const uint4*>(p + c);
            memcpy(e, &w, sizeof e);
          } else {
            const uint2 w = *reinterpret_cast<const uint2*>(p + c);
            memcpy(e, &w, sizeof e);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) v[4 * i + j] = f32_of<T>(e[j]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4 * NV; ++i) v[i] = lane + L * i < E ? f32_of<T>(p[lane + L * i]) : behind;
    }
  }
  template <typename T>
  __device__ __forceinline__ void store(T* p, const float (&v)[4 * NV]) const {
    if (VEC) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = 4 * (lane + L * i);
        T e[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) e[j] = T(v[4 * i + j]);
        if (c < E) {
          if (sizeof(T) == 4) {
            uint4 w;
            memcpy(&w, e, sizeof w);
            *reinterpret_cast<uint4*>(p + c) = w;
          } else {
            uint2 w;
            memcpy(&w, e, sizeof w);
            *reinterpret_cast<uint2*>(p + c) = w;
          }
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4 * NV; ++i)
        if (lane + L * i < E) p[lane + L * i] = T(v[i]);
    }
  }
};

__device__ __forceinline__ int warp_sum(int v) { return __reduce_add_sync(0xffffffffu, v); }
// Over L lanes side by side.
template <int L = 32>
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = L / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int L>
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = L / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Sum and maximum of a lane's values, in four chains. (Here and below one
// instruction does a pair of values where it can: issue slots bound the long
// rows as much as their latency.)
template <int N>
__device__ __forceinline__ float lane_max(const float (&v)[N]) {
  float m[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
  for (int i = 4; i < N; ++i) m[i & 3] = fmaxf(m[i & 3], v[i]);
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}
template <int N>
__device__ __forceinline__ float lane_sum(const float (&v)[N]) {
  Pair a = pair(v[0], v[1]), b = pair(v[2], v[3]);
#pragma unroll
  for (int i = 4; i < N; i += 4) a = add2(a, pair(v[i], v[i + 1])), b = add2(b, pair(v[i + 2], v[i + 3]));
  const float2 x = halves(a), y = halves(b);
  return (x.x + x.y) + (y.x + y.y);
}

// v becomes exp(v - l + log(scale)), l = logsumexp(v); `scale` is what the
// values are still to be multiplied by (1 / their sum). The difference from the
// largest comes before the factor log2(e): one product and sum would round most
// log2(e), which is more than 1 off from 1e7 on and leaves fp32 near the end of
// its range. A row of -inf alone (nothing allowed) has neither a softmax nor l:
// zeros, and 0. fmaxf drops a NaN, the sum keeps it.
template <int L, int N>
__device__ __forceinline__ float softmax_row(float (&v)[N], float* scale) {
  const float top = warp_max<L>(lane_max(v)), most = top == -INFINITY ? 0.f : top;
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float2 x = halves(mul2(add2(pair(v[i], v[i + 1]), both(-most)), both(kLog2e)));
    v[i] = exp2_fast(x.x), v[i + 1] = exp2_fast(x.y);
  }
  const float sum = warp_sum<L>(lane_sum(v));
  *scale = sum == 0.f ? 0.f : 1.f / sum;
  return sum == 0.f ? 0.f : most + kLn2 * log2f(sum);
}
// v becomes sigmoid(v) times a factor common to the row, m (if it is given)
// 1 - sigmoid(v); `scale` is 1 over the sum. With M = min(most, 0) and e =
// exp(M - v), sigmoid(v) exp(-M) = 1 / (exp(M) + e): scores that are all tiny
// keep their ratios, and 1 - sigmoid(v) = e / (exp(M) + e). From e = 2^126 on,
// the last that has a quotient, a score is 0 beside the largest, as -inf's is.
template <int L, bool REST, int N>
__device__ __forceinline__ void sigmoid_row(float (&v)[N], float* m, float* scale) {
  const float most = warp_max<L>(lane_max(v));
  const float M = most == -INFINITY ? 0.f : fminf(most, 0.f), low = exp2_fast(M * kLog2e);
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float2 x = halves(mul2(add2(pair(v[i], v[i + 1]), both(-M)), both(-kLog2e)));
    const float e[2] = {fminf(exp2_fast(x.x), 0x1p126f), fminf(exp2_fast(x.y), 0x1p126f)};
    const float2 sum = halves(add2(pair(e[0], e[1]), both(low)));
    const float r[2] = {__fdividef(1.f, sum.x), __fdividef(1.f, sum.y)};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float& z = v[i + j];
      if (REST) m[i + j] = z != z ? z : e[j] * r[j];
      z = (j ? x.y : x.x) >= 126.f ? 0.f : z != z ? z : r[j];  // fminf drops a NaN
    }
  }
  const float sum = warp_sum<L>(lane_sum(v));
  *scale = sum == 0.f ? 0.f : 1.f / sum;
}

struct Span {
  int64_t begin, end;
};
// Rows of sequence s, kept inside [0, T] whatever the caller's array holds.
__device__ __forceinline__ Span sequence(const int32_t* offs, int s, int64_t T) {
  if (!offs) return {0, T};
  return {min(max((int64_t)offs[s], (int64_t)0), T), min(max((int64_t)offs[s + 1], (int64_t)0), T)};
}
// The last sequence that begins at or before `row` (-1: none), looked for by a
// whole warp: 32 places a step, the last 128 in one.
__device__ __forceinline__ int sequence_of(const int32_t* offs, int S, int64_t row) {
  if (!offs) return 0;
  const int lane = threadIdx.x & 31;
  int lo = 0, n = S;  // it is lo - 1, or among the n from lo
  while (n > 128) {
    const int stride = (n + 31) / 32, i = lane * stride;
    const int before = __popc(__ballot_sync(0xffffffffu, i < n && offs[lo + min(i, n - 1)] <= row));
    if (before == 0) return lo - 1;
    const int at = (before - 1) * stride;
    lo += at + 1;
    n = min(stride, n - at) - 1;
  }
  int before = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) before += lane + 32 * i < n && offs[lo + lane + 32 * i] <= row;
  return lo + warp_sum(before) - 1;
}

// A row's scores but for the factor `scale`, in z; returns the squared
// logsumexp of the logits (0 where it has no part in the loss).
template <bool SIGMOID, int L, int N>
__device__ __forceinline__ float scores_row(float (&z)[N], float* scale, bool squares) {
  float l = 0.f;
  if (SIGMOID) {
    if (squares) {
      float w[N];
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = z[i];
      l = softmax_row<L>(w, scale);
    }
    sigmoid_row<L, false>(z, nullptr, scale);
  } else {
    l = softmax_row<L>(z, scale);
  }
  return squares ? l * l : 0.f;
}

// The value at `p` in shared memory of the cluster's block `rank`.
__device__ __forceinline__ uint32_t of_block(const void* p, int rank) {
  uint32_t at, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A call of one cluster: the blocks' sums and counts [E], rows and squares
// (thread 0's) meet in its shared memory, in the blocks' order, each block for a
// share of the experts. `scratch`: a value a warp.
__device__ __forceinline__ void finish_alone(const BalanceArgs& p, float* sums, int* count, int rows, float zz, float* scratch) {
  __shared__ int block_rows;
  __shared__ float block_zz, block_term;
  const int blocks = gridDim.x, rank = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) block_rows = rows, block_zz = zz;
  __syncthreads();
  cluster_barrier();
  rows = 0, zz = 0.f;
  for (int b = 0; b < blocks; ++b) rows += (int)of_block(&block_rows, b), zz += __uint_as_float(of_block(&block_zz, b));
  const float each = rows ? 1.f / (float)rows : 0.f;
  float term = 0.f;
  for (int e = rank * kBalThreads + threadIdx.x; e < p.E; e += blocks * kBalThreads) {
    float v = 0.f;
    int n = 0;
    for (int b = 0; b < blocks; ++b) v += __uint_as_float(of_block(&sums[e], b)), n += (int)of_block(&count[e], b);
    const float mean = rows ? v / (float)rows : 0.f;
    p.counts[e] = n;
    if (p.probs) p.probs[e] = mean;
    term += (float)n * mean;
  }
  term = warp_sum(term);
  if (lane == 0) scratch[warp] = term;
  __syncthreads();
  if (threadIdx.x == 0) {
    term = 0.f;
    for (int w = 0; w < kBalWarps; ++w) term += scratch[w];
    block_term = term;
  }
  __syncthreads();
  cluster_barrier();
  if (rank == 0 && threadIdx.x == 0) {
    term = 0.f;
    for (int b = 0; b < blocks; ++b) term += __uint_as_float(of_block(&block_term, b));
    p.loss[0] = p.coef * (term * ((float)p.E / (float)p.k) * each) + (p.z_coef != 0.f ? p.z_coef * zz * each : 0.f);
    p.tokens[0] = rows;
  }
  __syncwarp();
  cluster_barrier();  // nobody leaves while its values are read
}

// A warp has 32 / L rows side by side, the next ones' logits on their way
// meanwhile (short rows leave most lanes of a whole warp idle: 65536 rows of 128
// 16 us, with one a warp 21). The sums of the probabilities go to shared memory, a
// place a lane and value (in registers they cost the warps that hide the loads).
// With the join 16384 rows of 896 f32 take 20 us (3.0 TB/s: the exponentials and
// the adds of a value bound it as much as its bytes), sigmoid 26. Short rows off
// vector boundaries spill 52 to 76 bytes a thread.
// alone: the blocks are one cluster, which finishes the call.
template <typename T, bool VEC, int NV, int L, bool SIGMOID>
__global__ void __launch_bounds__(kBalThreads) balance_rows_kernel(const BalanceArgs p, const Entries out, int chunk_rows, int alone) {
  extern __shared__ __align__(16) float shared[];  // [warps][NV][32 lanes][4], then counts [E], sums [E]
  __shared__ int warp_rows[kBalWarps];
  __shared__ float warp_zz[kBalWarps];
  constexpr int N = 4 * NV, R = 32 / L;
  int* count = reinterpret_cast<int*>(shared + kBalWarps * 32 * N);
  float* sums = reinterpret_cast<float*>(count + p.E);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = lane / L;
  float4* mine = reinterpret_cast<float4*>(shared + warp * 32 * N) + lane;
  const Lanes<VEC, NV, L> at{lane % L, p.E};
  const int64_t first = (int64_t)blockIdx.x * chunk_rows, last = min(first + chunk_rows, p.T);
  pdl_wait();
  if (!alone) pdl_launch_dependents();  // the join, which waits for the end of this
  for (int s = max(0, sequence_of(p.offs, p.S, first)); s < p.S; ++s) {
    Span span = sequence(p.offs, s, p.T);
    if (span.begin >= last) break;
    span.begin = max(span.begin, first);
    span.end = min(span.end, last);
    if (span.begin >= span.end) continue;
    for (int e = threadIdx.x; e < p.E; e += kBalThreads) count[e] = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) mine[32 * i] = make_float4(0.f, 0.f, 0.f, 0.f);
    __syncthreads();
    int rows = 0;
    float zz = 0.f;
    // a row: its logits, its first ids and whether it counts
    float next[N];
    int id = -1;
    bool counts = false;
    const auto fetch = [&](int64_t t) {
      counts = t < span.end;
      if (!counts) return;
      if (p.mask) counts = p.mask[t] != 0;  // its row is read all the same: one latency, not two
      at.load(next, static_cast<const T*>(p.logits) + t * p.ldl, -INFINITY);
      id = at.lane < p.k ? p.ids[t * p.k + at.lane] : -1;
    };
    fetch(span.begin + warp * R + group);
    for (int64_t t0 = span.begin + warp * R; t0 < span.end; t0 += kBalWarps * R) {
      const bool here = counts;
      const int64_t t = t0 + group;
      float z[N], scale;
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] = R == 1 || here ? next[i] : 0.f;
      if (here) {
        if ((unsigned)id < (unsigned)p.E) atomicAdd(&count[id], 1);
        for (int j = at.lane + L; L < 32 && j < p.k; j += L) {
          const int e = p.ids[t * p.k + j];
          if ((unsigned)e < (unsigned)p.E) atomicAdd(&count[e], 1);
        }
      }
      fetch(t + kBalWarps * R);
      if (R == 1 && !here) continue;
      const float squares = scores_row<SIGMOID, L>(z, &scale, p.z_coef != 0.f);
      if (here) {
        ++rows;
        zz += squares;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const float4 v = mine[32 * i];
          const float2 a = halves(fma2(pair(z[4 * i], z[4 * i + 1]), both(scale), pair(v.x, v.y)));
          const float2 b = halves(fma2(pair(z[4 * i + 2], z[4 * i + 3]), both(scale), pair(v.z, v.w)));
          mine[32 * i] = make_float4(a.x, a.y, b.x, b.y);
        }
      }
    }
    rows = warp_sum(at.lane == 0 ? rows : 0);
    zz = warp_sum(at.lane == 0 ? zz : 0.f);
    if (lane == 0) warp_rows[warp] = rows, warp_zz[warp] = zz;
    __syncthreads();
    if (warp == 0) {  // thread 0 has them
      rows = warp_sum(lane < kBalWarps ? warp_rows[lane] : 0);
      zz = warp_sum(lane < kBalWarps ? warp_zz[lane] : 0.f);
    }
    const int64_t entry = (int64_t)blockIdx.x + s;
    for (int e = threadIdx.x; e < p.E; e += kBalThreads) {
      const float* from = shared + at.place(e);
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kBalWarps; ++w)
#pragma unroll
        for (int g = 0; g < R; ++g) v += from[w * 32 * N + 4 * L * g];
      if (alone) {
        sums[e] = v;
      } else {
        out.probs[entry * p.E + e] = v;
        out.count[entry * p.E + e] = count[e];
      }
    }
    if (alone) finish_alone(p, sums, count, rows, zz, warp_zz);
    else if (threadIdx.x == 0) out.sums[entry] = make_float2(__int_as_float(rows), zz);
    __syncthreads();
  }
}

template <int L, int NV>
__device__ __forceinline__ float dot_row(const float4* f, const float (&v)[4 * NV]) {
  Pair d[2] = {both(0.f), both(0.f)};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const float4 a = f[32 * i];
    d[0] = fma2(pair(a.x, a.y), pair(v[4 * i], v[4 * i + 1]), d[0]);
    d[1] = fma2(pair(a.z, a.w), pair(v[4 * i + 2], v[4 * i + 3]), d[1]);
  }
  const float2 x = halves(d[0]), y = halves(d[1]);
  return warp_sum<L>((x.x + x.y) + (y.x + y.y));
}

constexpr int kBalGradThreads = 256, kBalGradWarps = kBalGradThreads / 32;
// A warp has 32 / L rows side by side, and the ones behind them, so that f is
// worked out once a sequence (it stays in shared memory: in registers it cost a
// third of the warps). The routing weights' terms reach the lanes that hold their
// experts through rows of shared memory that are zero between (comparing every
// expert with every id took more instructions than the rest). 16384 rows of 896
// f32 26 us (4.5 TB/s), sigmoid 43 (a lane's three arrays of 32 values do not fit 128
// registers: 156 bytes spill); 65536 of 128 22 (33 with one row a warp).
template <typename T, bool VEC, int NV, int L, bool SIGMOID>
__global__ void __launch_bounds__(kBalGradThreads, NV < 8 ? 1 : 2) balance_grad_kernel(const BalanceGradArgs p, int64_t warp_rows) {
  extern __shared__ __align__(16) float shared[];  // [warps][NV][32 lanes][4] f, and with weights the same of their terms
  constexpr int N = 4 * NV, R = 32 / L;
  const int lane = threadIdx.x & 31, group = lane / L;
  float* f_rows = shared + (threadIdx.x >> 5) * 32 * N;
  float* kept = f_rows + kBalGradWarps * 32 * N;
  float4 *f4 = reinterpret_cast<float4*>(f_rows) + lane, *mine = reinterpret_cast<float4*>(kept) + lane;
  kept += 4 * L * group;  // of this lane's row
  const Lanes<VEC, NV, L> at{lane % L, p.E};
  const int64_t warp = (int64_t)blockIdx.x * kBalGradWarps + (threadIdx.x >> 5);
  const int64_t first = warp * warp_rows, last = min(first + warp_rows, p.T);
  pdl_wait();
  if (first >= last) return;
  const auto clear = [&] {
#pragma unroll
    for (int i = 0; i < NV; ++i) mine[32 * i] = make_float4(0.f, 0.f, 0.f, 0.f);
    __syncwarp();
  };
  if (p.weights) clear();
  int s = -2;  // not looked for yet
  bool fresh = true;
  Span span{0, 0};
  float aux = 0.f, zc = 0.f;
  for (int64_t t0 = first; t0 < last; t0 += R) {
    // the row first (one that turns out not to count is read all the same), so
    // that its latency is not added to the sequence's
    const int64_t t = t0 + group;
    const bool row = t < last;
    float z[N], w = 0.f, dw = 0.f;
    int id = -1;
    bool counts = row;
    if (row) {
      if (p.mask) counts = p.mask[t] != 0;
      at.load(z, static_cast<const T*>(p.logits) + t * p.ldl, -INFINITY);
      if (p.weights && at.lane < p.k) {
        w = p.weights[t * p.k + at.lane];
        dw = p.dweights[t * p.k + at.lane];
        id = p.ids[t * p.k + at.lane];
      }
    }
    if (s == -2) s = sequence_of(p.offs, p.S, t0);
    if (row) {
      while (s + 1 < p.S && p.offs && p.offs[s + 1] <= t) ++s, fresh = true;
      if (fresh && s >= 0) {
        fresh = false;
        span = sequence(p.offs, s, p.T);
        const float n = (float)p.tokens[s], each = n > 0.f ? 1.f / n : 0.f, g = p.dloss[s];
        aux = g * p.coef * each;
        zc = 2.f * g * p.z_coef * each;
        const float unit = (float)p.E / (float)p.k * each;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          float x[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int c = at.col(4 * i + j);
            x[j] = c < p.E ? (float)p.counts[(int64_t)s * p.E + c] * unit : 0.f;
          }
          f4[32 * i] = make_float4(x[0], x[1], x[2], x[3]);
        }
      }
    }
    const bool inside = row && s >= 0 && t >= span.begin && t < span.end;  // else left as it was
    counts = counts && inside;
    T* out = static_cast<T*>(p.dlogits) + t * p.lddl;
    if (R > 1 || !counts) {
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] = counts ? z[i] : 0.f;
    }
    if (R == 1 && !counts) {  // the whole warp
      if (inside) at.store(out, z);
      continue;
    }
    int place = -1;  // of this lane's routing weight in `kept`, where a row has a lane for each
    if (p.weights) {
      float mean = 0.f;
      for (int j = at.lane, n = 0; n < (L < 32 ? p.k : 1); j += L, n += L) {
        if (n) {
          const bool there = row && j < p.k;
          w = there ? p.weights[t * p.k + j] : 0.f;
          dw = there ? p.dweights[t * p.k + j] : 0.f;
          id = there ? p.ids[t * p.k + j] : -1;
        }
        if (counts && (unsigned)id < (unsigned)p.E) mean = fmaf(w, dw, mean);
      }
      mean = warp_sum<L>(mean);
      for (int j = at.lane, n = 0; n < (L < 32 ? p.k : 1); j += L, n += L) {
        if (L < 32 && p.k > L) {  // read again
          const bool there = row && j < p.k;
          w = there ? p.weights[t * p.k + j] : 0.f;
          dw = there ? p.dweights[t * p.k + j] : 0.f;
          id = there ? p.ids[t * p.k + j] : -1;
        }
        const bool there = counts && (unsigned)id < (unsigned)p.E;
        float x = there ? w * (dw - mean) : 0.f;
        // an expert that the row names again: its terms together, in order, in the first of its lanes
        const uint32_t same = __match_any_sync(0xffffffffu, there ? group << 16 | id : -1 - lane);
        if (__any_sync(0xffffffffu, same & (same - 1))) {
          float all = 0.f;
          for (int l = 0; l < 32; ++l) {
            const float y = __shfl_sync(0xffffffffu, x, l);
            if (same >> l & 1) all += y;
          }
          x = all;
        }
        if (there && lane == __ffs(same) - 1) {
          place = at.place(id);
          kept[place] = L == 32 ? x : kept[place] + x;
        }
        __syncwarp();
      }
    }
    float scale, dot;
    const auto term_of = [&](float (&x)[4], int i) {
      x[0] = x[1] = x[2] = x[3] = 0.f;
      if (p.weights) {
        const float4 k4 = mine[32 * i];
        x[0] = k4.x, x[1] = k4.y, x[2] = k4.z, x[3] = k4.w;
      }
    };
    if constexpr (SIGMOID) {
      float d[N], m[N], soft = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) d[i] = z[i];
      sigmoid_row<L, true>(d, m, &scale);
      dot = dot_row<L, NV>(f4, d) * scale;
      if (p.z_coef != 0.f) {
        const float l = softmax_row<L>(z, &soft);
        soft *= zc * l;
      }
      scale *= aux;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float x[4];
        term_of(x, i);
        const float4 fi = f4[32 * i];
        const float f[4] = {fi.x, fi.y, fi.z, fi.w};
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          const int c = 4 * i + j;
          const Pair t = fma2(mul2(both(scale), pair(d[c], d[c + 1])), add2(pair(f[j], f[j + 1]), both(-dot)), pair(x[j], x[j + 1]));
          Pair r = mul2(pair(m[c], m[c + 1]), t);
          if (p.z_coef != 0.f) r = fma2(both(soft), pair(z[c], z[c + 1]), r);
          const float2 h = halves(r);
          z[c] = h.x, z[c + 1] = h.y;
        }
      }
    } else {
      const float l = softmax_row<L>(z, &scale);
      dot = dot_row<L, NV>(f4, z) * scale;
      const float rest = p.z_coef != 0.f ? scale * (zc * l) : 0.f;
      scale *= aux;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float x[4];
        term_of(x, i);
        const float4 fi = f4[32 * i];
        const float f[4] = {fi.x, fi.y, fi.z, fi.w};
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          const int c = 4 * i + j;
          const Pair t = fma2(both(scale), add2(pair(f[j], f[j + 1]), both(-dot)), both(rest));
          const float2 r = halves(fma2(pair(z[c], z[c + 1]), t, pair(x[j], x[j + 1])));
          z[c] = r.x, z[c + 1] = r.y;
        }
      }
    }
    if (R > 1 && !counts) {
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] = 0.f;
    }
    if (inside) at.store(out, z);
    if (p.weights) {
      __syncwarp();
      if (R > 1) {
        clear();
      } else {
        if (place >= 0) kept[place] = 0.f;
        __syncwarp();
      }
    }
  }
}

bool vec_rows(const void* p, int64_t ld, int E, int size) {
  return E % 4 == 0 && !(((uintptr_t)p | (uint64_t)(ld * size)) & (uint64_t)(4 * size - 1));
}

// A kernel's dynamic shared memory, once a device.
template <typename K>
cudaError_t allow_shared(K kernel, size_t bytes, std::atomic<uint64_t>& done) {
  int device = 0;
  (void)cudaGetDevice(&device);
  if (device < 64 && done.load() >> device & 1) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && device < 64) done.fetch_or(1ull << device);
  return e;
}

template <typename T, bool VEC, bool SIGMOID, int NV, int L>
cudaError_t rows_launch(const BalanceArgs& p, const Entries& out, int64_t chunk, int64_t blocks, int alone, cudaStream_t s) {
  const auto kernel = balance_rows_kernel<T, VEC, NV, L, SIGMOID>;
  const size_t smem = (size_t)(kBalWarps * 128 * NV + 2 * p.E) * sizeof(float);  // 72 KB at most
  if (NV == 8) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_shared(kernel, (kBalWarps * 1024 + 2 * kOpsMaxExperts) * sizeof(float), done);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kBalThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = alone ? (unsigned)blocks : 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = alone ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, out, (int)chunk, alone);
}
template <typename T, bool VEC, bool SIGMOID>
cudaError_t rows_nv(const BalanceArgs& p, const Entries& out, int64_t chunk, int64_t blocks, int alone, cudaStream_t s) {
  switch (balance_shape(p.E)) {
    case 0: return rows_launch<T, VEC, SIGMOID, 2, 4>(p, out, chunk, blocks, alone, s);
    case 1: return rows_launch<T, VEC, SIGMOID, 2, 8>(p, out, chunk, blocks, alone, s);
    case 2: return rows_launch<T, VEC, SIGMOID, 2, 16>(p, out, chunk, blocks, alone, s);
    case 3: return rows_launch<T, VEC, SIGMOID, 2, 32>(p, out, chunk, blocks, alone, s);
    case 4: return rows_launch<T, VEC, SIGMOID, 4, 32>(p, out, chunk, blocks, alone, s);
    default: return rows_launch<T, VEC, SIGMOID, 8, 32>(p, out, chunk, blocks, alone, s);
  }
}
template <typename T>
cudaError_t rows_t(const BalanceArgs& p, const Entries& out, int64_t chunk, int64_t blocks, int alone, cudaStream_t s) {
  if (vec_rows(p.logits, p.ldl, p.E, sizeof(T)))
    return p.sigmoid ? rows_nv<T, true, true>(p, out, chunk, blocks, alone, s) : rows_nv<T, true, false>(p, out, chunk, blocks, alone, s);
  return p.sigmoid ? rows_nv<T, false, true>(p, out, chunk, blocks, alone, s) : rows_nv<T, false, false>(p, out, chunk, blocks, alone, s);
}

template <typename T, bool VEC, bool SIGMOID, int NV, int L>
cudaError_t grad_launch(const BalanceGradArgs& p, int sms, cudaStream_t s) {
  const auto kernel = balance_grad_kernel<T, VEC, NV, L, SIGMOID>;
  constexpr size_t once = (size_t)kBalGradWarps * 128 * NV * sizeof(float);
  const size_t smem = p.weights ? 2 * once : once;  // 64 KB at most
  if (NV == 8) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_shared(kernel, 2 * once, done);
    if (e != cudaSuccess) return e;
  }
  // as many warps as run at once, each with rows side by side
  static std::atomic<int> known{0};  // blocks an SM with the larger shared memory
  int each = known.load();
  if (!each) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&each, kernel, kBalGradThreads, 2 * once) != cudaSuccess || each < 1) {
      (void)cudaGetLastError();
      each = 1;
    }
    known.store(each);
  }
  constexpr int R = 32 / L;
  const int64_t warps = (int64_t)sms * each * kBalGradWarps, rows = ((p.T + warps - 1) / warps + R - 1) / R * R;
  const int64_t blocks = ((p.T + rows - 1) / rows + kBalGradWarps - 1) / kBalGradWarps;
  return launch_after_previous(kernel, dim3((unsigned)blocks), dim3(kBalGradThreads), smem, s, p, rows);
}
template <typename T, bool VEC, bool SIGMOID>
cudaError_t grad_nv(const BalanceGradArgs& p, int sms, cudaStream_t s) {
  switch (balance_shape(p.E)) {
    case 0: return grad_launch<T, VEC, SIGMOID, 2, 4>(p, sms, s);
    case 1: return grad_launch<T, VEC, SIGMOID, 2, 8>(p, sms, s);
    case 2: return grad_launch<T, VEC, SIGMOID, 2, 16>(p, sms, s);
    case 3: return grad_launch<T, VEC, SIGMOID, 2, 32>(p, sms, s);
    case 4: return grad_launch<T, VEC, SIGMOID, 4, 32>(p, sms, s);
    default: return grad_launch<T, VEC, SIGMOID, 8, 32>(p, sms, s);
  }
}
template <typename T>
cudaError_t grad_t(const BalanceGradArgs& p, int sms, cudaStream_t s) {
  if (vec_rows(p.logits, p.ldl, p.E, sizeof(T)) && vec_rows(p.dlogits, p.lddl, p.E, sizeof(T)))
    return p.sigmoid ? grad_nv<T, true, true>(p, sms, s) : grad_nv<T, true, false>(p, sms, s);
  return p.sigmoid ? grad_nv<T, false, true>(p, sms, s) : grad_nv<T, false, false>(p, sms, s);
}

}  // namespace
}  // namespace dfm
