// k_balance.cu — what joins the entries of the balance loss's rows (k_balance.cuh,
// a file a type), and the choice of the type and the blocks.
#include "k_balance.cuh"

namespace dfm {
namespace {

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
      loss = p.coef * (terms[0] + terms[1] + terms[2] + terms[3]) + (part == 0 && p.z_coef != 0.f ? p.z_coef * zz * each : 0.f);
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

// Rows of a block: short rows have few registers and small entries, so two
// blocks share an SM (30000 of 256 20 us, with one 24; of 896 one block, and
// half the entries to join).
int64_t chunk_rows_of(int64_t T, int E) {
  const int64_t blocks = kBalBlocks * (E <= 256 ? 2 : 1), rows = (T + blocks - 1) / blocks;
  const int64_t once = kBalWarps * balance_rows_a_warp(E);
  return (rows + once - 1) / once * once;
}
int64_t entries_of(int64_t T, int E, int64_t S) {
  const int64_t rows = chunk_rows_of(T, E);
  return (T + rows - 1) / rows + S;
}

}  // namespace

size_t balance_workspace_bytes(int64_t T, int E, int64_t S) { return (size_t)entries_of(T, E, S) * (8 * (size_t)E + 8); }

cudaError_t launch_balance_loss(const BalanceArgs& p, int dtype, void* workspace, cudaStream_t s) {
  // Few rows of one sequence, one a lane group: a cluster that finishes them
  // itself saves the join's launch (us, in one kernel and in two: 1 row of 896 5.0
  // and 6.8, 64 6.3 and 7.7, 128 6.9 and 7.8, 128 of 160 5.7 and 6.2; short rows
  // pass only up to four blocks: 8 of 64 4.3 and 5.1, 256 of 64 5.1 and 5.4, but 512
  // of 64 5.7 and 5.6, 256 of 128 5.7 and 5.4).
  const int64_t once = kBalWarps * balance_rows_a_warp(p.E);
  const int alone = !p.offs && p.T <= (balance_rows_a_warp(p.E) == 1 ? 8 : 4) * once;
  const int64_t chunk = alone ? once : chunk_rows_of(p.T, p.E), blocks = (p.T + chunk - 1) / chunk, entries = blocks + p.S;
  Entries out;
  out.probs = static_cast<float*>(workspace);
  out.count = reinterpret_cast<int32_t*>(out.probs + entries * p.E);
  out.sums = reinterpret_cast<float2*>(out.count + entries * p.E);
  const cudaError_t e = (dtype == 0 ? balance_rows_bf16 : dtype == 1 ? balance_rows_f16 : balance_rows_f32)(p, out, chunk, blocks, alone, s);
  if (e != cudaSuccess || alone) return e;
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
  return (dtype == 0 ? balance_grad_bf16 : dtype == 1 ? balance_grad_f16 : balance_grad_f32)(p, sms, s);
}

}  // namespace dfm
