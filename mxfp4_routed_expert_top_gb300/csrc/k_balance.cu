// k_balance.cu — the router's balance loss with the counts of every expert, and
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
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cstring>

#include "fastmath.cuh"
#include "internal.h"
#include "ops.h"
#include "pipeline.cuh"

namespace dfm {
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

// A row of E values over a warp: VEC: four side by side, 128 apart; else one by
// one, 32 apart. Element i of lane l is column `col(i)`.
template <bool VEC, int NV>
struct Lanes {
  int lane, E;
  __device__ __forceinline__ int col(int i) const { return VEC ? 4 * (lane + 32 * (i / 4)) + i % 4 : lane + 32 * i; }
  template <typename T>
  __device__ __forceinline__ void load(float (&v)[4 * NV], const T* p, float behind) const {
    if (VEC) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = 4 * (lane + 32 * i);
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
      for (int i = 0; i < 4 * NV; ++i) v[i] = lane + 32 * i < E ? f32_of<T>(p[lane + 32 * i]) : behind;
    }
  }
  template <typename T>
  __device__ __forceinline__ void store(T* p, const float (&v)[4 * NV]) const {
    if (VEC) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = 4 * (lane + 32 * i);
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
        if (lane + 32 * i < E) p[lane + 32 * i] = T(v[i]);
    }
  }
};

__device__ __forceinline__ int warp_sum(int v) { return __reduce_add_sync(0xffffffffu, v); }
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// v becomes exp(v - l + log(scale)), l = logsumexp(v); `scale` is what the
// values are still to be multiplied by (1 / their sum). exp(v - most) as a
// power of two with one fused product: the rounding of most log2(e) is common to
// the row and leaves with the sum. A row of -inf alone (nothing allowed) has
// neither a softmax nor l: zeros, and 0. fmaxf drops a NaN, the sum keeps it.
template <int N>
__device__ __forceinline__ float softmax_row(float (&v)[N], float* scale) {
  float most = v[0];
#pragma unroll
  for (int i = 1; i < N; ++i) most = fmaxf(most, v[i]);
  most = warp_max(most);
  const float base = most == -INFINITY ? 0.f : most * kLog2e;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = exp2_fast(fmaf(v[i], kLog2e, -base));
    sum += v[i];
  }
  sum = warp_sum(sum);
  *scale = sum == 0.f ? 0.f : 1.f / sum;
  return sum == 0.f ? 0.f : kLn2 * (base + log2f(sum));
}
// v becomes sigmoid(v) times a factor common to the row, m (if it is given)
// 1 - sigmoid(v); `scale` is 1 over the sum. With M = min(most, 0) and e =
// exp(M - v), sigmoid(v) exp(-M) = 1 / (exp(M) + e): scores that are all tiny
// keep their ratios, and 1 - sigmoid(v) = e / (exp(M) + e).
template <int N, bool REST>
__device__ __forceinline__ void sigmoid_row(float (&v)[N], float* m, float* scale) {
  float most = v[0];
#pragma unroll
  for (int i = 1; i < N; ++i) most = fmaxf(most, v[i]);
  most = warp_max(most);
  const float M = most == -INFINITY ? 0.f : fminf(most, 0.f) * kLog2e, low = exp2_fast(M);
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float e = fminf(exp2_fast(fmaf(-v[i], kLog2e, M)), 1e37f), r = __fdividef(1.f, low + e);
    if (REST) m[i] = v[i] != v[i] ? v[i] : e * r;
    v[i] = v[i] == -INFINITY ? 0.f : v[i] != v[i] ? v[i] : r;  // fminf drops a NaN
    sum += v[i];
  }
  sum = warp_sum(sum);
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
// whole warp: 32 places a step.
__device__ __forceinline__ int sequence_of(const int32_t* offs, int S, int64_t row) {
  if (!offs) return 0;
  const int lane = threadIdx.x & 31;
  int lo = 0, n = S;  // it is lo - 1, or among the n from lo
  while (n > 0) {
    const int stride = (n + 31) / 32, i = lane * stride;
    const int before = __popc(__ballot_sync(0xffffffffu, i < n && offs[lo + min(i, n - 1)] <= row));
    if (before == 0) break;
    const int at = (before - 1) * stride;
    lo += at + 1;
    n = min(stride, n - at) - 1;
  }
  return lo - 1;
}

// A block has the rows of one chunk and leaves one entry for every sequence it
// meets. Entry chunk + s: along the rows either number only grows and one of
// them does from entry to entry, so no two have the same, and chunks + S are
// enough.
struct Entries {
  float* probs;    // [entries][E]
  int32_t* count;  // [entries][E]
  float2* sums;    // [entries]: rows counted (an int's bits), sum of l^2
};

// A row's scores but for the factor `scale`, in z; returns the squared
// logsumexp of the logits (0 where it has no part in the loss).
template <bool SIGMOID, int N>
__device__ __forceinline__ float scores_row(float (&z)[N], float* scale, bool squares) {
  float l = 0.f;
  if (SIGMOID) {
    if (squares) {
      float w[N];
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = z[i];
      l = softmax_row(w, scale);
    }
    sigmoid_row<N, false>(z, nullptr, scale);
  } else {
    l = softmax_row(z, scale);
  }
  return squares ? l * l : 0.f;
}

// A warp a row, the next row's logits on their way meanwhile. The sums of the
// probabilities go to a row of shared memory of the warp's own (in registers
// they cost the warps that hide the loads).
template <typename T, bool VEC, int NV, bool SIGMOID>
__global__ void __launch_bounds__(kBalThreads) balance_rows_kernel(const BalanceArgs p, const Entries out, int chunk_rows) {
  extern __shared__ __align__(16) float shared[];  // [warps][128 NV], then counts [E]
  __shared__ int warp_rows[kBalWarps];
  __shared__ float warp_zz[kBalWarps];
  constexpr int N = 4 * NV;
  int* count = reinterpret_cast<int*>(shared + kBalWarps * 32 * N);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float4* mine = reinterpret_cast<float4*>(shared + warp * 32 * N) + lane;  // element i of lane l: [i / 4][l][i % 4]
  const Lanes<VEC, NV> at{lane, p.E};
  const int64_t first = (int64_t)blockIdx.x * chunk_rows, last = min(first + chunk_rows, p.T);
  pdl_wait();
  pdl_launch_dependents();  // the join, which waits for the end of this
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
    // a row: its logits, its ids and whether it counts
    float next[N];
    int id = -1;
    bool counts = false;
    const auto fetch = [&](int64_t t) {
      counts = t < span.end;
      if (!counts) return;
      if (p.mask) counts = p.mask[t] != 0;  // its row is read all the same: one latency, not two
      at.load(next, static_cast<const T*>(p.logits) + t * p.ldl, -INFINITY);
      id = lane < p.k ? p.ids[t * p.k + lane] : -1;
    };
    fetch(span.begin + warp);
    for (int64_t t = span.begin + warp; t < span.end; t += kBalWarps) {
      const bool here = counts;
      float z[N];
      if (here) {
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] = next[i];
        if ((unsigned)id < (unsigned)p.E) atomicAdd(&count[id], 1);
      }
      fetch(t + kBalWarps);
      if (!here) continue;
      ++rows;
      float scale;
      zz += scores_row<SIGMOID>(z, &scale, p.z_coef != 0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float4 v = mine[32 * i];
        v.x = fmaf(z[4 * i], scale, v.x), v.y = fmaf(z[4 * i + 1], scale, v.y);
        v.z = fmaf(z[4 * i + 2], scale, v.z), v.w = fmaf(z[4 * i + 3], scale, v.w);
        mine[32 * i] = v;
      }
    }
    if (lane == 0) warp_rows[warp] = rows, warp_zz[warp] = zz;
    __syncthreads();
    const int64_t entry = (int64_t)blockIdx.x + s;
    for (int e = threadIdx.x; e < p.E; e += kBalThreads) {
      // column e is element i of lane l
      const int l = VEC ? e / 4 % 32 : e % 32, i = VEC ? e / 128 * 4 + e % 4 : e / 32;
      const float* from = shared + 128 * (i / 4) + 4 * l + i % 4;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kBalWarps; ++w) v += from[w * 32 * N];
      out.probs[entry * p.E + e] = v;
      out.count[entry * p.E + e] = count[e];
    }
    if (threadIdx.x == 0) {
      int n = 0;
      float v = 0.f;
      for (int w = 0; w < kBalWarps; ++w) n += warp_rows[w], v += warp_zz[w];
      out.sums[entry] = make_float2(__int_as_float(n), v);
    }
    __syncthreads();
  }
}

// One cluster a sequence, 128 experts a CTA: the entries' sums in their order
// (interleaved over the warps, 32 of them or 8), and the loss.
constexpr int kBalJoin = 1024, kBalJoinFew = 256;
__global__ void __launch_bounds__(kBalJoin) balance_join_kernel(const BalanceArgs p, const Entries in, int chunk_rows, int parts) {
  const int warps = blockDim.x >> 5;
  __shared__ float probs[32][128];
  __shared__ int count[32][128];
  __shared__ int warp_rows[32];
  __shared__ float warp_zz[32];
  __shared__ float terms[4];
  __shared__ float loss;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int s = blockIdx.x / parts, part = blockIdx.x - s * parts;
  pdl_wait();
  const Span span = sequence(p.offs, s, p.T);
  const bool some = span.begin < span.end;
  const int64_t first = some ? span.begin / chunk_rows + s : 0, last = some ? (span.end - 1) / chunk_rows + s : -1;
  if (p.status && p.offs && threadIdx.x == 0 && part == 0 &&
      (p.offs[s + 1] < p.offs[s] || p.offs[s] < 0 || p.offs[s + 1] > p.T))
    atomicOr(p.status, DEV_ERR_RANGE);
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  int n[4] = {0, 0, 0, 0};
  if (p.E % 4 == 0) {
    const int c = 128 * part + 4 * lane;
    if (c < p.E) {
#pragma unroll 4
      for (int64_t i = first + warp; i <= last; i += warps) {
        const float4 a = *reinterpret_cast<const float4*>(in.probs + i * p.E + c);
        const int4 b = *reinterpret_cast<const int4*>(in.count + i * p.E + c);
        v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
        n[0] += b.x, n[1] += b.y, n[2] += b.z, n[3] += b.w;
      }
    }
  } else {
#pragma unroll 2
    for (int64_t i = first + warp; i <= last; i += warps)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = 128 * part + lane + 32 * j;
        if (c < p.E) {
          v[j] += in.probs[i * p.E + c];
          n[j] += in.count[i * p.E + c];
        }
      }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int e = p.E % 4 == 0 ? 4 * lane + j : lane + 32 * j;
    probs[warp][e] = v[j];
    count[warp][e] = n[j];
  }
  // rows counted and l^2: every thread has some entries
  int rows = 0;
  float zz = 0.f;
  for (int64_t i = first + threadIdx.x; i <= last; i += blockDim.x) rows += __float_as_int(in.sums[i].x), zz += in.sums[i].y;
  rows = warp_sum(rows), zz = warp_sum(zz);
  if (lane == 0) warp_rows[warp] = rows, warp_zz[warp] = zz;
  __syncthreads();
  if (threadIdx.x < 128) {
    const int e = threadIdx.x, expert = 128 * part + e;
    rows = warp_sum(lane < warps ? warp_rows[lane] : 0), zz = warp_sum(lane < warps ? warp_zz[lane] : 0.f);
    float all = 0.f;
    int many = 0;
#pragma unroll 8
    for (int w = 0; w < warps; ++w) all += probs[w][e], many += count[w][e];
    const float each = rows > 0 ? 1.f / (float)rows : 0.f, mean = rows > 0 ? all / (float)rows : 0.f;
    float term = 0.f;
    if (expert < p.E) {
      p.counts[(int64_t)s * p.E + expert] = many;
      if (p.probs) p.probs[(int64_t)s * p.E + expert] = mean;
      term = (float)many * ((float)p.E / (float)p.k) * each * mean;
    }
    term = warp_sum(term);
    if (lane == 0) terms[warp] = term;
    named_barrier_sync(1, 128);
    if (threadIdx.x == 0) {
      loss = p.coef * (terms[0] + terms[1] + terms[2] + terms[3]) + (part == 0 ? p.z_coef * zz * each : 0.f);
      if (part == 0) p.tokens[s] = rows;
    }
  }
  __syncthreads();
  if (parts > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  if (part == 0 && threadIdx.x == 0) {
    float all = 0.f;
    for (int q = 0; q < parts; ++q) {
      uint32_t at;
      float x;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(&loss)), "r"(q));
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(at) : "memory");
      all += x;
    }
    p.loss[s] = all;
  }
  if (parts > 1) {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
}

template <int NV>
__device__ __forceinline__ float dot_row(const float4* f, const float (&v)[4 * NV]) {
  float dot = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const float4 a = f[32 * i];
    dot = fmaf(a.x, v[4 * i], fmaf(a.y, v[4 * i + 1], fmaf(a.z, v[4 * i + 2], fmaf(a.w, v[4 * i + 3], dot))));
  }
  return warp_sum(dot);
}

constexpr int kBalGradThreads = 256, kBalGradWarps = kBalGradThreads / 32;
// A warp a row, rows side by side in a chunk of its own, so that f is worked out
// once a sequence (it stays in shared memory: in registers it cost a third of
// the warps). The routing weights' terms reach the lanes
// that hold their experts through a row of shared memory that is zero between
// rows (comparing every expert with every id took more instructions than the
// rest).
template <typename T, bool VEC, int NV, bool SIGMOID>
__global__ void __launch_bounds__(kBalGradThreads, NV < 8 ? 1 : 2) balance_grad_kernel(const BalanceGradArgs p, int64_t warp_rows) {
  extern __shared__ __align__(16) float shared[];  // [warps][128 NV] f, and with weights [warps][128 NV] their terms
  constexpr int N = 4 * NV;
  const int lane = threadIdx.x & 31;
  float* f_row = shared + (threadIdx.x >> 5) * 32 * N;
  float* kept = f_row + kBalGradWarps * 32 * N;
  float4 *f4 = reinterpret_cast<float4*>(f_row) + lane, *mine = reinterpret_cast<float4*>(kept) + lane;  // element i of lane l: [i / 4][l][i % 4]
  const Lanes<VEC, NV> at{lane, p.E};
  const int64_t warp = (int64_t)blockIdx.x * kBalGradWarps + (threadIdx.x >> 5);
  const int64_t first = warp * warp_rows, last = min(first + warp_rows, p.T);
  pdl_wait();
  if (first >= last) return;
  if (p.weights) {
#pragma unroll
    for (int i = 0; i < NV; ++i) mine[32 * i] = make_float4(0.f, 0.f, 0.f, 0.f);
    __syncwarp();
  }
  int s = -2;  // not looked for yet
  Span span{0, 0};
  float aux = 0.f, zc = 0.f;
  for (int64_t t = first; t < last; ++t) {
    // the row first (one that turns out not to count is read all the same), so
    // that its latency is not added to the sequence's
    float z[N], w = 0.f, dw = 0.f;
    int id = -1;
    const bool counts = !p.mask || p.mask[t];
    at.load(z, static_cast<const T*>(p.logits) + t * p.ldl, -INFINITY);
    if (p.weights && lane < p.k) {
      w = p.weights[t * p.k + lane];
      dw = p.dweights[t * p.k + lane];
      id = p.ids[t * p.k + lane];
    }
    bool fresh = s == -2;
    if (fresh) s = sequence_of(p.offs, p.S, t);
    while (s + 1 < p.S && p.offs && p.offs[s + 1] <= t) ++s, fresh = true;
    if (s < 0) continue;
    if (fresh) {
      span = sequence(p.offs, s, p.T);
      const float n = (float)p.tokens[s], each = n > 0.f ? 1.f / n : 0.f, g = p.dloss[s];
      aux = g * p.coef * each;
      zc = 2.f * g * p.z_coef * each;
      const float unit = (float)p.E / (float)p.k * each;
      __syncwarp();
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
    if (t < span.begin || t >= span.end) continue;  // behind every sequence: left as it was
    T* out = static_cast<T*>(p.dlogits) + t * p.lddl;
    if (!counts) {
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] = 0.f;
      at.store(out, z);
      continue;
    }
    int place = -1;  // of this lane's routing weight in `kept`
    if (p.weights) {
      const bool there = (unsigned)id < (unsigned)p.E;
      const float mean = warp_sum(there ? w * dw : 0.f);
      float x = there ? w * (dw - mean) : 0.f;
      // an expert that the row names again: its terms together, in order, in the first of its lanes
      const uint32_t same = __match_any_sync(0xffffffffu, there ? id : -1 - lane);
      if (__any_sync(0xffffffffu, same & (same - 1))) {
        float all = 0.f;
        for (int j = 0; j < p.k; ++j) {
          const float y = __shfl_sync(0xffffffffu, x, j);
          if (same >> j & 1) all += y;
        }
        x = all;
      }
      if (there && lane == __ffs(same) - 1) {
        place = VEC ? id : 128 * (id / 128) + 4 * (id % 32) + id / 32 % 4;
        kept[place] = x;
      }
      __syncwarp();
    }
    float dot = 0.f, scale;
    if constexpr (SIGMOID) {
      float d[N], m[N], soft = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) d[i] = z[i];
      sigmoid_row<N, true>(d, m, &scale);
      dot = dot_row<NV>(f4, d) * scale;
      if (zc != 0.f) {
        const float l = softmax_row(z, &soft);
        soft *= zc * l;
      }
      scale *= aux;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float x[4] = {0.f, 0.f, 0.f, 0.f};
        if (p.weights) {
          const float4 w = mine[32 * i];
          x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w;
        }
        const float4 fi = f4[32 * i];
        const float f[4] = {fi.x, fi.y, fi.z, fi.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = 4 * i + j;
          d[c] = m[c] * fmaf(scale * d[c], f[j] - dot, x[j]);
          if (zc != 0.f) d[c] = fmaf(soft, z[c], d[c]);
        }
      }
      at.store(out, d);
    } else {
      const float l = softmax_row(z, &scale);
      dot = dot_row<NV>(f4, z) * scale;
      const float rest = scale * (zc != 0.f ? zc * l : 0.f);
      scale *= aux;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float x[4] = {0.f, 0.f, 0.f, 0.f};
        if (p.weights) {
          const float4 w = mine[32 * i];
          x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w;
        }
        const float4 fi = f4[32 * i];
        const float f[4] = {fi.x, fi.y, fi.z, fi.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = 4 * i + j;
          z[c] = fmaf(z[c], fmaf(scale, f[j] - dot, rest), x[j]);
        }
      }
      at.store(out, z);
    }
    if (p.weights) {
      __syncwarp();
      if (place >= 0) kept[place] = 0.f;
      __syncwarp();
    }
  }
}

// Rows of a block: short rows have few registers and small entries, so more
// blocks share an SM.
int64_t chunk_rows_of(int64_t T, int E) {
  const int64_t blocks = kBalBlocks * (E <= 128 ? 3 : E <= 512 ? 2 : 1), rows = (T + blocks - 1) / blocks;
  return (rows + kBalWarps - 1) / kBalWarps * kBalWarps;
}
int64_t entries_of(int64_t T, int E, int64_t S) {
  const int64_t rows = chunk_rows_of(T, E);
  return (T + rows - 1) / rows + S;
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

// NV parts of 128 experts: 1, 2, 4 or 8.
template <typename T, bool VEC, bool SIGMOID>
cudaError_t rows_nv(const BalanceArgs& p, const Entries& out, int64_t chunk, int64_t blocks, cudaStream_t s) {
  const int nv = p.E <= 128 ? 1 : p.E <= 256 ? 2 : p.E <= 512 ? 4 : 8;
  const size_t smem = (size_t)(kBalWarps * 128 * nv + p.E) * sizeof(float);  // 68 KB at most
  const dim3 g((unsigned)blocks), b(kBalThreads);
  const int c = (int)chunk;
  if (nv == 8) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_shared(balance_rows_kernel<T, VEC, 8, SIGMOID>, (kBalWarps * 1024 + kOpsMaxExperts) * sizeof(float), done);
    if (e != cudaSuccess) return e;
  }
  if (nv == 1) return launch_after_previous(balance_rows_kernel<T, VEC, 1, SIGMOID>, g, b, smem, s, p, out, c);
  if (nv == 2) return launch_after_previous(balance_rows_kernel<T, VEC, 2, SIGMOID>, g, b, smem, s, p, out, c);
  if (nv == 4) return launch_after_previous(balance_rows_kernel<T, VEC, 4, SIGMOID>, g, b, smem, s, p, out, c);
  return launch_after_previous(balance_rows_kernel<T, VEC, 8, SIGMOID>, g, b, smem, s, p, out, c);
}
template <typename T>
cudaError_t rows_t(const BalanceArgs& p, const Entries& out, int64_t chunk, int64_t blocks, cudaStream_t s) {
  if (vec_rows(p.logits, p.ldl, p.E, sizeof(T)))
    return p.sigmoid ? rows_nv<T, true, true>(p, out, chunk, blocks, s) : rows_nv<T, true, false>(p, out, chunk, blocks, s);
  return p.sigmoid ? rows_nv<T, false, true>(p, out, chunk, blocks, s) : rows_nv<T, false, false>(p, out, chunk, blocks, s);
}
template <typename T, bool VEC, bool SIGMOID>
cudaError_t grad_nv(const BalanceGradArgs& p, int64_t rows, int64_t blocks, cudaStream_t s) {
  const int nv = p.E <= 128 ? 1 : p.E <= 256 ? 2 : p.E <= 512 ? 4 : 8;
  const size_t smem = (p.weights ? 2 : 1) * (size_t)kBalGradWarps * 128 * nv * sizeof(float);  // 64 KB at most
  const dim3 g((unsigned)blocks), b(kBalGradThreads);
  if (nv == 8) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_shared(balance_grad_kernel<T, VEC, 8, SIGMOID>, 2 * kBalGradWarps * 1024 * sizeof(float), done);
    if (e != cudaSuccess) return e;
  }
  if (nv == 1) return launch_after_previous(balance_grad_kernel<T, VEC, 1, SIGMOID>, g, b, smem, s, p, rows);
  if (nv == 2) return launch_after_previous(balance_grad_kernel<T, VEC, 2, SIGMOID>, g, b, smem, s, p, rows);
  if (nv == 4) return launch_after_previous(balance_grad_kernel<T, VEC, 4, SIGMOID>, g, b, smem, s, p, rows);
  return launch_after_previous(balance_grad_kernel<T, VEC, 8, SIGMOID>, g, b, smem, s, p, rows);
}
template <typename T>
cudaError_t grad_t(const BalanceGradArgs& p, int64_t rows, int64_t blocks, cudaStream_t s) {
  if (vec_rows(p.logits, p.ldl, p.E, sizeof(T)) && vec_rows(p.dlogits, p.lddl, p.E, sizeof(T)))
    return p.sigmoid ? grad_nv<T, true, true>(p, rows, blocks, s) : grad_nv<T, true, false>(p, rows, blocks, s);
  return p.sigmoid ? grad_nv<T, false, true>(p, rows, blocks, s) : grad_nv<T, false, false>(p, rows, blocks, s);
}

}  // namespace

size_t balance_workspace_bytes(int64_t T, int E, int64_t S) { return (size_t)entries_of(T, E, S) * (8 * (size_t)E + 8); }

cudaError_t launch_balance_loss(const BalanceArgs& p, int dtype, void* workspace, cudaStream_t s) {
  const int64_t chunk = chunk_rows_of(p.T, p.E), blocks = (p.T + chunk - 1) / chunk, entries = blocks + p.S;
  Entries out;
  out.probs = static_cast<float*>(workspace);
  out.count = reinterpret_cast<int32_t*>(out.probs + entries * p.E);
  out.sums = reinterpret_cast<float2*>(out.count + entries * p.E);
  cudaError_t e = dtype == 0   ? rows_t<__nv_bfloat16>(p, out, chunk, blocks, s)
                  : dtype == 1 ? rows_t<__half>(p, out, chunk, blocks, s)
                               : rows_t<float>(p, out, chunk, blocks, s);
  if (e != cudaSuccess) return e;
  const int parts = (p.E + 127) / 128;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.S * parts));
  cfg.blockDim = dim3(blocks > 64 * (int64_t)p.S ? kBalJoin : kBalJoinFew);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = parts;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, balance_join_kernel, p, out, (int)chunk, parts);
}

cudaError_t launch_balance_loss_grad(const BalanceGradArgs& p, int dtype, int sms, cudaStream_t s) {
  // about as many warps as fit the GPU at once
  const int64_t warps = (int64_t)sms * (p.E <= 128 ? 6 : p.E <= 512 ? 3 : 2) * kBalGradWarps, rows = (p.T + warps - 1) / warps;
  const int64_t blocks = ((p.T + rows - 1) / rows + kBalGradWarps - 1) / kBalGradWarps;
  return dtype == 0   ? grad_t<__nv_bfloat16>(p, rows, blocks, s)
         : dtype == 1 ? grad_t<__half>(p, rows, blocks, s)
                      : grad_t<float>(p, rows, blocks, s);
}

}  // namespace dfm
