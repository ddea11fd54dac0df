// k_permute.cu — tokens sorted by expert and back, with their gradients.
//
// Assignment a = t k + j sends token t to expert ids[a]; it is valid where
// 0 <= ids[a] < E and dropped otherwise. With the stable sort of the valid
// assignments by expert,
//   offs[e] = #{valid a : ids[a] < e},
//   pos[a]  = offs[ids[a]] + #{a' < a : ids[a'] = ids[a]}   (-1 if dropped),
//   src[pos[a]] = a,
// the operators are
//   permute         rows[pos[a]] = x[a / k]
//   its gradient    dx[t] = sum_j drows[pos[t k + j]]
//   unpermute       y[t] = sum_j w[t][j] rows[pos[t k + j]]
//   its gradient    drows[pos[a]] = w[a] dy[t],  dw[a] = <dy[t], rows[pos[a]]>
// (dropped assignments add nothing and have dw = 0). All of them move bytes:
// T + n rows once each (n valid assignments), so HBM bounds them at large T
// and the launch at small T. Every place is counted, never taken by an atomic
// whose order could show, and every sum has a fixed order.
//
// Every kernel here and in k_fp8.cu is launched as a programmatic dependent of
// the one before it: its blocks may start while that one's memory is flushed,
// and wait (griddepcontrol.wait) before they touch global memory. Their loads
// are ordinary ones (not .nc): the lines may have been in L1 since before the
// wait. None of them lets its own dependents start early: a kernel of the
// layer that reads its input without waiting relies on that.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstring>

#include "internal.h"
#include "ops.h"
#include "pipeline.cuh"
#include "rowword.h"

namespace dfm {
namespace {

constexpr int kPermThreads = 512;

// Exclusive prefix sum of one value a thread over the block (a multiple of
// 32 threads, at most 1024); `warp_sums` holds 32 ints. Two barriers.
__device__ __forceinline__ int block_scan(int v, int* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += n;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const int nw = blockDim.x >> 5;
    int s = lane < nw ? warp_sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += n;
    }
    if (lane < nw) warp_sums[lane] = s;
  }
  __syncthreads();
  return (warp ? warp_sums[warp - 1] : 0) + incl - v;
}

// Copies columns [v0, v1) (in V units) of the tokens [t0, t1) to the rows
// their assignments have: each value is read once and written up to k times.
// `pos` points at the first token's k places.
template <typename V>
__device__ __forceinline__ void copy_rows(const PermuteArgs& p, int t0, int t1, const int32_t* pos,
                                          int v0, int v1) {
  const int nv = v1 - v0, items = (t1 - t0) * nv;
  for (int i = threadIdx.x; i < items; i += blockDim.x) {
    const int dt = i / nv, v = v0 + i - dt * nv;
    const V val = reinterpret_cast<const V*>(p.x + (int64_t)(t0 + dt) * p.ldx)[v];
    const int32_t* at = pos + dt * p.k;
    for (int j = 0; j < p.k; ++j) {
      const int32_t q = at[j];
      if (q >= 0) reinterpret_cast<V*>(p.rows + q * p.ldr)[v] = val;
    }
  }
}

// The same for rows that are not aligned to 4 bytes, in words w of [w0, w1):
// word w of a row holds the bytes c .. c + 3 with c = 4 (w - 1) + a, where a
// is what the row lacks to a 4-byte boundary, so that its store is aligned;
// each value comes from three aligned words of x by a funnel shift (words
// without a byte of the row are not read). The first and last words of a row
// are stored byte by byte. ENDS: words of x may reach over the array's ends,
// and are then read byte by byte.
template <bool ENDS>
__device__ __forceinline__ void copy_word_odd(const PermuteArgs& p, int t0, const int32_t* pos, int w0, int nw, int i) {
  const int dt = i / nw, from = 4 * (w0 + i - dt * nw - 1), bytes = (int)p.bytes;
  const char* x = p.x + (int64_t)(t0 + dt) * p.ldx;
  const int m = (int)((uintptr_t)(x + from) & 3);
  uint32_t word[3];
#pragma unroll
  for (int n = 0; n < 3; ++n) {
    const int c = from - m + 4 * n;  // bytes c .. c + 3 of the row
    if (ENDS) {
      const Four<char> four = array_four<char>(ArrayOf<char>{p.x}, x + c - p.x, (int64_t)(p.T - 1) * p.ldx + bytes);
      memcpy(&word[n], &four, 4);
    } else {
      word[n] = c + 3 >= 0 && c < bytes ? *reinterpret_cast<const uint32_t*>(x + c) : 0;
    }
  }
  const int32_t* at = pos + dt * p.k;
  for (int j = 0; j < p.k; ++j) {
    const int32_t q = at[j];
    if (q < 0) continue;
    char* row = p.rows + q * p.ldr;
    const int a = (int)(-(uintptr_t)row & 3), c = from + a, s = m + a;
    const uint32_t v = s < 4 ? __funnelshift_r(word[0], word[1], 8 * s) : __funnelshift_r(word[1], word[2], 8 * (s - 4));
    if (c >= 0 && c + 4 <= bytes) {
      *reinterpret_cast<uint32_t*>(row + c) = v;
    } else {
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (c + b >= 0 && c + b < bytes) row[c + b] = (char)(v >> (8 * b));
    }
  }
}

// Reads reach at most 3 bytes over a row: over the array's start in the first
// two words of token 0, over its end in the last three of the last token (in
// any where rows are nearer than that). The block's last threads take those:
// a test in every word cost 7%, and first threads 1 us a call of short rows.
// 2000 x 8 rows of 3001 bytes (54 MB, 8 us at the copy rate) take 24 us, of 3001
// bf16 39: issue slots (73% busy), mostly the stores of eight rows a word.
__device__ __forceinline__ void copy_rows_odd(const PermuteArgs& p, int t0, int t1, const int32_t* pos, int w0,
                                              int w1) {
  const int nw = w1 - w0, items = (t1 - t0) * nw, last = (int)((p.bytes + 3) / 4) + 1 - 3;
  const int head = p.ldx < 3 ? items : t0 == 0 ? max(0, min(2 - w0, nw)) : 0;
  const int tail = t1 == p.T ? max(0, min(min(w1 - last, nw), items - head)) : 0;
  for (int i = blockDim.x - 1 - threadIdx.x; i < head + tail; i += blockDim.x)
    copy_word_odd<true>(p, t0, pos, w0, nw, i < head ? i : items - tail + i - head);
  for (int i = head + threadIdx.x; i < items - tail; i += blockDim.x) copy_word_odd<false>(p, t0, pos, w0, nw, i);
}

__device__ __forceinline__ void copy_scales(const PermuteArgs& p, int t0, int t1,
                                            const int32_t* pos) {
  const int S = p.n_scales, items = (t1 - t0) * S;
  for (int i = threadIdx.x; i < items; i += blockDim.x) {
    const int dt = i / S, v = i - dt * S;
    const float val = p.xs[(int64_t)(t0 + dt) * p.ldxs + v];
    const int32_t* at = pos + dt * p.k;
    for (int j = 0; j < p.k; ++j) {
      const int32_t q = at[j];
      if (q >= 0) p.rows_s[q * p.ldrs + v] = val;
    }
  }
}

// One launch for up to kSelfCount assignments: every block counts all of them
// itself (before its own and from its own on), so no block waits for another
// and nothing goes through global memory. Block (b, c) then ranks its own
// tokens' assignments and copies column range c of their rows. A block of
// 1024 threads an SM halves what an SM counts against two of 512; clusters
// of eight that shared the counting through distributed shared memory were
// slower (4096 tokens x 16 rows of 256 bf16: 17.5 us, two blocks 21, clusters
// 31). Writes bound the large calls: 4096 x 16 rows of 7168 (999 MB, 940 of
// them written) take 183 us, of which bulk copies through shared memory saved
// nothing.
//
// kSelfCount: where the two ways cross, more or less. This one against counts
// by chunks (four launches), 896 experts, rows of 64 / 256 / 7168 bf16, in a
// graph: 8192 assignments 4.0 / 4.0 / 25 us against 11 / 11 / 33; 32768 6.9 / 8.7 / 93
// against 15 / 16 / 96; 65536 11.8 / 16.9 / 182 against 20 / 26 / 180; 131072 24 / 35 /
// 362 against 31 / 38 / 349. Above it, every block would count and rank ever more
// for the same SMs; the chunks' way has a block's 512 threads for the columns of
// one token, of which short rows use few.
constexpr int kSelfThreads = 1024;
constexpr int kSelfCount = 65536;
constexpr int kSelfChunk = 1024;  // assignments a block may own

template <typename V>
__global__ void __launch_bounds__(kSelfThreads)
permute_kernel(const PermuteArgs p, int tokens_per_block, int vecs, int vecs_per_block) {
  __shared__ int before[kOpsMaxExperts], rest[kOpsMaxExperts];
  __shared__ int own_id[kSelfChunk], own_pos[kSelfChunk];
  __shared__ int warp_sums[32];
  const int tid = threadIdx.x;
  const int t0 = blockIdx.x * tokens_per_block, t1 = min(p.T, t0 + tokens_per_block);
  const int A = p.T * p.k, a0 = t0 * p.k, a1 = t1 * p.k;
  for (int e = tid; e < p.E; e += kSelfThreads) before[e] = rest[e] = 0;
  pdl_wait();
  __syncthreads();
  if (((uintptr_t)p.ids & 15) == 0) {
    const int4* ids4 = reinterpret_cast<const int4*>(p.ids);
#pragma unroll 4
    for (int i = tid; i < A / 4; i += kSelfThreads) {
      const int4 e = ids4[i];
      const int ev[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if ((unsigned)ev[u] < (unsigned)p.E)
          atomicAdd(4 * i + u < a0 ? &before[ev[u]] : &rest[ev[u]], 1);
    }
    for (int a = (A & ~3) + tid; a < A; a += kSelfThreads) {
      const int e = p.ids[a];
      if ((unsigned)e < (unsigned)p.E) atomicAdd(a < a0 ? &before[e] : &rest[e], 1);
    }
  } else {
#pragma unroll 4
    for (int a = tid; a < A; a += kSelfThreads) {
      const int e = p.ids[a];
      if ((unsigned)e < (unsigned)p.E) atomicAdd(a < a0 ? &before[e] : &rest[e], 1);
    }
  }
  for (int i = tid; i < a1 - a0; i += kSelfThreads) {
    const int e = p.ids[a0 + i];
    own_id[i] = (unsigned)e < (unsigned)p.E ? e : -1;
  }
  __syncthreads();
  // before[e] becomes the row of this block's first assignment to expert e
  static_assert(kSelfThreads == kOpsMaxExperts, "one expert a thread");
  const int count = tid < p.E ? before[tid] + rest[tid] : 0;
  const int start = block_scan(count, warp_sums);
  const bool writer = blockIdx.y == 0;
  if (tid < p.E) before[tid] += start;
  if (writer && blockIdx.x == 0) {
    if (tid < p.E) p.offs[tid] = start;
    if (tid == p.E - 1) p.offs[p.E] = start + count;
  }
  __syncthreads();
  for (int i = tid; i < a1 - a0; i += kSelfThreads) {
    const int e = own_id[i];
    int q = -1;
    if (e >= 0) {
      q = before[e];
      for (int u = 0; u < i; ++u) q += own_id[u] == e;
    }
    own_pos[i] = q;
    if (writer) {
      p.pos[a0 + i] = q;
      if (q >= 0) p.src[q] = a0 + i;
    }
  }
  __syncthreads();
  const int v0 = blockIdx.y * vecs_per_block;
  if constexpr (sizeof(V) < 4) copy_rows_odd(p, t0, t1, own_pos, v0, min(vecs, v0 + vecs_per_block));
  else copy_rows<V>(p, t0, t1, own_pos, v0, min(vecs, v0 + vecs_per_block));
  if (p.n_scales && writer) copy_scales(p, t0, t1, own_pos);
}

// ---- more assignments: counted per chunk, summed over the chunks, placed ----
// counts [chunks][E]: how many of chunk c go to expert e.
__global__ void __launch_bounds__(kPermThreads)
permute_count_kernel(const int32_t* ids, int64_t A, int E, int64_t chunk,
                     int32_t* counts) {
  __shared__ int cnt[kOpsMaxExperts];
  for (int e = threadIdx.x; e < E; e += kPermThreads) cnt[e] = 0;
  pdl_wait();
  __syncthreads();
  const int64_t a0 = blockIdx.x * chunk, a1 = a0 + chunk < A ? a0 + chunk : A;
#pragma unroll 4
  for (int64_t a = a0 + threadIdx.x; a < a1; a += kPermThreads) {
    const int e = ids[a];
    if ((unsigned)e < (unsigned)E) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kPermThreads) counts[(int64_t)blockIdx.x * E + e] = cnt[e];
}

// Per expert: counts become exclusive prefix sums over the chunks, and the
// row behind the last chunk the totals. A block holds 32 experts, one a lane,
// and each of its 32 warps a range of chunks.
__global__ void __launch_bounds__(1024)
permute_scan_kernel(int32_t* counts, int E, int chunks) {
  __shared__ int part[32][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int e = blockIdx.x * 32 + lane;
  const int per = (chunks + 31) / 32;
  const int c0 = min(warp * per, chunks), c1 = min(c0 + per, chunks);
  int sum = 0;
  pdl_wait();
  if (e < E) {
#pragma unroll 4
    for (int c = c0; c < c1; ++c) sum += counts[(int64_t)c * E + e];
  }
  part[warp][lane] = sum;
  __syncthreads();
  int run = 0;
  for (int w = 0; w < warp; ++w) run += part[w][lane];
  if (e < E) {
    for (int c = c0; c < c1; ++c) {
      const int64_t i = (int64_t)c * E + e;
      const int n = counts[i];
      counts[i] = run;
      run += n;
    }
    if (warp == 31) counts[(int64_t)chunks * E + e] = run;
  }
}

// Places of one chunk: each warp counts its own part of the chunk, the parts'
// counts become first rows, and the warp walks its part again, 32 assignments
// at a time, ranking equal experts within the 32 by lane.
constexpr int kPlaceWarps = kPermThreads / 32;
__global__ void __launch_bounds__(kPermThreads)
permute_place_kernel(const int32_t* ids, int64_t A, int E, int64_t chunk, int chunks,
                     const int32_t* counts, int32_t* offs,
                     int32_t* pos, int32_t* src) {
  extern __shared__ int part[];  // [kPlaceWarps][E]
  __shared__ int warp_sums[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t a0 = blockIdx.x * chunk, a1 = a0 + chunk < A ? a0 + chunk : A;
  const int64_t per = ((a1 - a0 + kPlaceWarps - 1) / kPlaceWarps + 31) & ~31;
  const int64_t w0 = a0 + warp * per < a1 ? a0 + warp * per : a1;
  const int64_t w1 = w0 + per < a1 ? w0 + per : a1;
  int* const mine = part + warp * E;
  for (int i = tid; i < kPlaceWarps * E; i += kPermThreads) part[i] = 0;
  pdl_wait();
  __syncthreads();
  for (int64_t a = w0; a < w1; a += 32) {
    const int e = a + lane < w1 ? ids[a + lane] : -1;
    const bool valid = (unsigned)e < (unsigned)E;
    const unsigned same = __match_any_sync(0xffffffffu, valid ? e : -1);
    if (valid && lane == __ffs(same) - 1) mine[e] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  const int e0 = 2 * tid, e1 = e0 + 1;
  const int32_t* totals = counts + (int64_t)chunks * E;
  const int c0 = e0 < E ? totals[e0] : 0, c1 = e1 < E ? totals[e1] : 0;
  const int o0 = block_scan(c0 + c1, warp_sums), o1 = o0 + c0;
  if (blockIdx.x == 0) {
    if (e0 < E) offs[e0] = o0;
    if (e1 < E) offs[e1] = o1;
    if (e0 == E - 1) offs[E] = o0 + c0;
    if (e1 == E - 1) offs[E] = o1 + c1;
  }
  const int32_t* first = counts + (int64_t)blockIdx.x * E;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int e = e0 + u;
    if (e < E) {
      int run = (u ? o1 : o0) + first[e];
      for (int w = 0; w < kPlaceWarps; ++w) {
        const int n = part[w * E + e];
        part[w * E + e] = run;
        run += n;
      }
    }
  }
  __syncthreads();
  for (int64_t a = w0; a < w1; a += 32) {
    const int e = a + lane < w1 ? ids[a + lane] : -1;
    const bool valid = (unsigned)e < (unsigned)E;
    const unsigned same = __match_any_sync(0xffffffffu, valid ? e : -1);
    const int q = valid ? mine[e] + __popc(same & ((1u << lane) - 1)) : -1;
    __syncwarp();
    if (valid && lane == __ffs(same) - 1) mine[e] += __popc(same);
    __syncwarp();
    if (a + lane < w1) {
      pos[a + lane] = q;
      if (valid) src[q] = (int32_t)(a + lane);
    }
  }
}

template <typename V>
__global__ void __launch_bounds__(kPermThreads)
permute_copy_kernel(const PermuteArgs p, int vecs) {
  pdl_wait();
  for (int64_t i = blockIdx.x; i < p.T; i += gridDim.x) {
    const int t = (int)i;
    const int32_t* at = p.pos + i * p.k;
    if constexpr (sizeof(V) < 4) copy_rows_odd(p, t, t + 1, at, 0, vecs);
    else copy_rows<V>(p, t, t + 1, at, 0, vecs);
    if (p.n_scales) copy_scales(p, t, t + 1, at);
  }
}

int64_t permute_chunks(int64_t A) {
  const int64_t n = (A + 1023) / 1024;
  return n < 1023 ? n : 1023;
}

template <typename V>
cudaError_t permute_v(const PermuteArgs& p, void* workspace, int sms, cudaStream_t s) {
  const int64_t A = (int64_t)p.T * p.k;
  const int vecs = sizeof(V) < 4 ? (int)((p.bytes + 3) / 4 + 1) : (int)(p.bytes / (int64_t)sizeof(V));
  if (A <= kSelfCount) {
    int tpb = (p.T + sms - 1) / sms;
    if (tpb * p.k > kSelfChunk) tpb = kSelfChunk / p.k;
    const int gx = (p.T + tpb - 1) / tpb;
    // few tokens: their columns are split too, at least 64 values a block
    int gy = sms / gx;
    if (gy > (vecs + 63) / 64) gy = (vecs + 63) / 64;
    if (gy < 1) gy = 1;
    const int vpb = (vecs + gy - 1) / gy;
    return launch_after_previous(permute_kernel<V>, dim3(gx, gy), dim3(kSelfThreads), 0, s, p, tpb, vecs, vpb);
  }
  const int chunks = (int)permute_chunks(A);
  int64_t chunk = (A + chunks - 1) / chunks;
  int32_t* counts = static_cast<int32_t*>(workspace);
  const size_t smem = (size_t)kPlaceWarps * p.E * sizeof(int);
  cudaError_t e = cudaFuncSetAttribute(permute_place_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kPlaceWarps * kOpsMaxExperts * (int)sizeof(int));
  if (e == cudaSuccess)
    e = launch_after_previous(permute_count_kernel, dim3(chunks), dim3(kPermThreads), 0, s, p.ids, A, p.E, chunk,
                              counts);
  if (e == cudaSuccess)
    e = launch_after_previous(permute_scan_kernel, dim3((p.E + 31) / 32), dim3(1024), 0, s, counts, p.E, chunks);
  if (e == cudaSuccess)
    e = launch_after_previous(permute_place_kernel, dim3(chunks), dim3(kPermThreads), smem, s, p.ids, A, p.E, chunk,
                              chunks, counts, p.offs, p.pos, p.src);
  if (e == cudaSuccess)
    e = launch_after_previous(permute_copy_kernel<V>, dim3(4 * sms < p.T ? 4 * sms : p.T), dim3(kPermThreads), 0, s,
                              p, vecs);
  return e;
}

// ---- rows of a type as fp32 vectors -------------------------------------------
template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
};
template <>
struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<__half> {
  static __device__ __forceinline__ float get(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half put(float v) { return __float2half_rn(v); }
};

template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
  T v[N];
};

// A row is read once: its lines are not kept in L1.
template <typename P>
__device__ __forceinline__ P load_once(const void* p) {
  P r;
  if constexpr (sizeof(P) == 16) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    memcpy(&r, &v, 16);
  } else {
    r = *static_cast<const P*>(p);
  }
  return r;
}

// y[t] = sum_j w_j rows[pos_j]: a thread per N columns of a token; the loads
// of four rows are in flight together. Sums in fp32 in the order of j, one
// rounding at the end. HBM bounds it: 4096 tokens x 16 rows of 7168 bf16 (999
// MB) take 153 us with four rows in flight, 184 with eight (fewer threads an
// SM), 165 with two; with the rows in L1 it is 158.
template <typename T, int N, int U, bool WEIGHTED>
__global__ void __launch_bounds__(128)
unpermute_kernel(const UnpermuteArgs p, int nv, uint64_t by_nv) {
  pdl_wait();
  // i / nv: by_nv = ceil(2^64 / nv) (0 for 1) is exact as long as i nv < 2^64
  const uint64_t i = blockIdx.x * (uint64_t)blockDim.x + threadIdx.x;
  const int64_t token = by_nv ? (int64_t)__umul64hi(i, by_nv) : (int64_t)i;
  if (token >= p.T) return;
  const int t = (int)token;
  const int c = (int)(i - (uint64_t)t * nv) * N;
  const T* rows = static_cast<const T*>(p.rows);
  const int32_t* at = p.pos + (int64_t)t * p.k;
  const float* w = p.weights + (int64_t)t * p.k;
  float acc[N];
#pragma unroll
  for (int n = 0; n < N; ++n) acc[n] = 0.f;
  for (int j0 = 0; j0 < p.k; j0 += U) {
    Pack<T, N> r[U];
    float wt[U];
    bool there[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u;
      const int32_t q = j < p.k ? at[j] : -1;
      there[u] = q >= 0 && q < p.n_rows;
      wt[u] = WEIGHTED && there[u] ? w[j] : 1.f;
      if (there[u]) r[u] = load_once<Pack<T, N>>(rows + q * p.ldr + c);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (there[u]) {
#pragma unroll
        for (int n = 0; n < N; ++n)
          acc[n] = WEIGHTED ? fmaf(wt[u], Elem<T>::get(r[u].v[n]), acc[n])
                            : acc[n] + Elem<T>::get(r[u].v[n]);
      }
  }
  Pack<T, N> out;
#pragma unroll
  for (int n = 0; n < N; ++n) out.v[n] = Elem<T>::put(acc[n]);
  *reinterpret_cast<Pack<T, N>*>(static_cast<T*>(p.y) + (int64_t)t * p.ldy + c) = out;
}

// Rows that no 8-byte vector fits: a warp per token and 256 columns, eight a
// lane, value by value; two rows in flight. 2000 x 8 rows of 3001 bf16 (108 MB,
// 16 us at the copy rate) take 26 us, of fp32 (216 MB, 32) 36.
template <typename T, bool WEIGHTED>
__global__ void __launch_bounds__(128)
unpermute_odd_kernel(const UnpermuteArgs p, uint32_t segments, FastDiv by_segments) {
  pdl_wait();
  constexpr int C = 8, U = 2;
  const int lane = threadIdx.x & 31;
  const uint32_t i = blockIdx.x * 4 + (threadIdx.x >> 5);
  const uint32_t t = by_segments(i);
  if (t >= (uint32_t)p.T) return;
  const int c0 = (int)(i - t * segments) * 32 * C + lane;
  const T* rows = static_cast<const T*>(p.rows);
  const int32_t* at = p.pos + (int64_t)t * p.k;
  const float* w = p.weights + (int64_t)t * p.k;
  float acc[C];
#pragma unroll
  for (int n = 0; n < C; ++n) acc[n] = 0.f;
  for (int j0 = 0; j0 < p.k; j0 += U) {
    T r[U][C];
    float wt[U];
    bool there[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int32_t q = j0 + u < p.k ? at[j0 + u] : -1;
      there[u] = q >= 0 && q < p.n_rows;
      wt[u] = WEIGHTED && there[u] ? w[j0 + u] : 1.f;
      const T* row = rows + q * p.ldr + c0;
#pragma unroll
      for (int n = 0; n < C; ++n)
        if (there[u] && c0 + 32 * n < p.H) r[u][n] = row[32 * n];
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (there[u]) {
#pragma unroll
        for (int n = 0; n < C; ++n)
          acc[n] = WEIGHTED ? fmaf(wt[u], Elem<T>::get(r[u][n]), acc[n]) : acc[n] + Elem<T>::get(r[u][n]);
      }
  }
  T* y = static_cast<T*>(p.y) + (int64_t)t * p.ldy + c0;
#pragma unroll
  for (int n = 0; n < C; ++n)
    if (c0 + 32 * n < p.H) y[32 * n] = Elem<T>::put(acc[n]);
}

template <typename T>
cudaError_t unpermute_odd(const UnpermuteArgs& p, cudaStream_t s) {
  const uint32_t segments = (uint32_t)((p.H + 255) / 256);
  const uint64_t warps = (uint64_t)p.T * segments;  // below 2^31
  const dim3 blocks((unsigned)((warps + 3) / 4));
  return p.weights ? launch_after_previous(unpermute_odd_kernel<T, true>, blocks, dim3(128), 0, s, p, segments,
                                           FastDiv(segments))
                   : launch_after_previous(unpermute_odd_kernel<T, false>, blocks, dim3(128), 0, s, p, segments,
                                           FastDiv(segments));
}

template <typename T, int N, int U>
cudaError_t unpermute_u(const UnpermuteArgs& p, unsigned blocks, int nv, cudaStream_t s) {
  const uint64_t by_nv = nv == 1 ? 0 : ~0ull / (uint64_t)nv + 1;
  return p.weights ? launch_after_previous(unpermute_kernel<T, N, U, true>, dim3(blocks), dim3(128), 0, s, p, nv, by_nv)
                   : launch_after_previous(unpermute_kernel<T, N, U, false>, dim3(blocks), dim3(128), 0, s, p, nv, by_nv);
}

template <typename T, int N>
cudaError_t unpermute_n(const UnpermuteArgs& p, int sms, cudaStream_t s) {
  const int nv = p.H / N;
  const int64_t blocks = ((int64_t)p.T * nv + 127) / 128;
  // at most two blocks an SM: sixteen rows in flight, as latency is all there
  // is (one token x 16 rows of 7168: 5.0 us a call against 5.75)
  if (blocks <= 2 * sms && p.k > 4) return unpermute_u<T, N, 16>(p, (unsigned)blocks, nv, s);
  return unpermute_u<T, N, 4>(p, (unsigned)blocks, nv, s);
}

// A block per token and group of J of its assignments: dy is read once a
// group, each row read once and its gradient written beside it; the J dot
// products are summed over the block in a fixed order. Column steps are not
// unrolled: registers cost blocks an SM (1023 x 6 rows of 2049 fp32, 104 MB:
// 21.4 us, 29 unrolled; 2048 x 8 of 7168 bf16, 499 MB: 77). Rows that no vector
// fits go value by value: the same 1023 x 6 rows in bf16 (52 MB, 7.7 us at the
// copy rate) take 16.3.
constexpr int kGradThreads = 128;
template <typename T, int N, int J>
__global__ void __launch_bounds__(kGradThreads)
unpermute_grad_kernel(const UnpermuteGradArgs p, int groups) {
  __shared__ float part[kGradThreads / 32][J];
  pdl_wait();
  const int t = blockIdx.x / groups, j0 = (blockIdx.x - t * groups) * J;
  const T* dy = static_cast<const T*>(p.dy) + (int64_t)t * p.lddy;
  const T* rows = static_cast<const T*>(p.rows);
  T* drows = static_cast<T*>(p.drows);
  int32_t q[J];
  float w[J], dot[J];
#pragma unroll
  for (int u = 0; u < J; ++u) {
    const int j = j0 + u;
    q[u] = j < p.k ? p.pos[(int64_t)t * p.k + j] : -1;
    if (q[u] >= p.n_rows) q[u] = -1;
    w[u] = q[u] >= 0 ? p.weights[(int64_t)t * p.k + j] : 0.f;
    dot[u] = 0.f;
  }
#pragma unroll 1
  for (int c = threadIdx.x * N; c < p.H; c += kGradThreads * N) {
    const Pack<T, N> d = *reinterpret_cast<const Pack<T, N>*>(dy + c);
    Pack<T, N> r[J];
#pragma unroll
    for (int u = 0; u < J; ++u)
      if (q[u] >= 0) r[u] = load_once<Pack<T, N>>(rows + q[u] * p.ldr + c);
#pragma unroll
    for (int u = 0; u < J; ++u)
      if (q[u] >= 0) {
        Pack<T, N> g;
#pragma unroll
        for (int n = 0; n < N; ++n) {
          const float dv = Elem<T>::get(d.v[n]);
          dot[u] = fmaf(dv, Elem<T>::get(r[u].v[n]), dot[u]);
          g.v[n] = Elem<T>::put(w[u] * dv);
        }
        *reinterpret_cast<Pack<T, N>*>(drows + q[u] * p.lddr + c) = g;
      }
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int u = 0; u < J; ++u) {
#pragma unroll
    for (int o = 16; o; o >>= 1) dot[u] += __shfl_xor_sync(0xffffffffu, dot[u], o);
    if (lane == 0) part[warp][u] = dot[u];
  }
  __syncthreads();
  if (threadIdx.x < J && j0 + (int)threadIdx.x < p.k) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kGradThreads / 32; ++i) sum += part[i][threadIdx.x];
    p.dweights[(int64_t)t * p.k + j0 + threadIdx.x] = sum;
  }
}

template <typename T, int N, int J>
cudaError_t unpermute_grad_j(const UnpermuteGradArgs& p, cudaStream_t s) {
  const int groups = (p.k + J - 1) / J;
  return launch_after_previous(unpermute_grad_kernel<T, N, J>, dim3((unsigned)((int64_t)p.T * groups)),
                               dim3(kGradThreads), 0, s, p, groups);
}

template <typename T, int N>
cudaError_t unpermute_grad_n(const UnpermuteGradArgs& p, int sms, cudaStream_t s) {
  // few tokens: one assignment a block, so that more SMs share the rows; else
  // groups of at most four, as even as they come
  const int groups = (p.k + 3) / 4, each = (p.k + groups - 1) / groups;
  if ((int64_t)p.T * p.k <= 4 * sms || each == 1) return unpermute_grad_j<T, N, 1>(p, s);
  return each == 2   ? unpermute_grad_j<T, N, 2>(p, s)
         : each == 3 ? unpermute_grad_j<T, N, 3>(p, s)
                     : unpermute_grad_j<T, N, 4>(p, s);
}

// The widest vector of at most 16 bytes that every address and distance allows.
int vector_bytes(uint64_t bits, int most) {
  int v = most;
  while (v > 1 && (bits & (uint64_t)(v - 1))) v >>= 1;
  return v;
}

template <typename T>
cudaError_t unpermute_t(const UnpermuteArgs& p, int sms, cudaStream_t s) {
  constexpr int B = sizeof(T);
  const uint64_t bits = (uint64_t)p.rows | (uint64_t)p.y | (uint64_t)(p.ldr * B) |
                        (uint64_t)(p.ldy * B) | (uint64_t)((int64_t)p.H * B);
  const int n = vector_bytes(bits, 16) / B;
  if (n >= 16 / B) return unpermute_n<T, 16 / B>(p, sms, s);
  if (n >= 8 / B) return unpermute_n<T, 8 / B>(p, sms, s);
  return unpermute_odd<T>(p, s);
}

template <typename T>
cudaError_t unpermute_grad_t(const UnpermuteGradArgs& p, int sms, cudaStream_t s) {
  constexpr int B = sizeof(T);
  const uint64_t bits = (uint64_t)p.rows | (uint64_t)p.dy | (uint64_t)p.drows |
                        (uint64_t)(p.ldr * B) | (uint64_t)(p.lddr * B) | (uint64_t)(p.lddy * B) |
                        (uint64_t)((int64_t)p.H * B);
  const int n = vector_bytes(bits, 16) / B;
  if (n >= 16 / B) return unpermute_grad_n<T, 16 / B>(p, sms, s);
  if (n >= 8 / B) return unpermute_grad_n<T, 8 / B>(p, sms, s);
  return unpermute_grad_n<T, 1>(p, sms, s);
}

}  // namespace

size_t permute_workspace_bytes(int64_t T, int k, int E) {
  const int64_t A = T * k;
  return A <= kSelfCount ? 0 : (size_t)(permute_chunks(A) + 1) * E * sizeof(int32_t);
}

cudaError_t launch_permute(const PermuteArgs& p, void* workspace, int sms, cudaStream_t s) {
  const uint64_t bits = (uint64_t)p.x | (uint64_t)p.rows | (uint64_t)p.ldx | (uint64_t)p.ldr |
                        (uint64_t)p.bytes;
  switch (vector_bytes(bits, 16)) {
    case 16: return permute_v<uint4>(p, workspace, sms, s);
    case 8: return permute_v<uint2>(p, workspace, sms, s);
    case 4: return permute_v<uint32_t>(p, workspace, sms, s);
    default: return permute_v<uint8_t>(p, workspace, sms, s);  // by words, shifted
  }
}

cudaError_t launch_unpermute(const UnpermuteArgs& p, int dtype, int sms, cudaStream_t s) {
  return dtype == 0   ? unpermute_t<__nv_bfloat16>(p, sms, s)
         : dtype == 1 ? unpermute_t<__half>(p, sms, s)
                      : unpermute_t<float>(p, sms, s);
}

cudaError_t launch_unpermute_grad(const UnpermuteGradArgs& p, int dtype, int sms,
                                  cudaStream_t s) {
  return dtype == 0   ? unpermute_grad_t<__nv_bfloat16>(p, sms, s)
         : dtype == 1 ? unpermute_grad_t<__half>(p, sms, s)
                      : unpermute_grad_t<float>(p, sms, s);
}

}  // namespace dfm
