// k_fp8.cu — rows in 8 bits with one fp32 scale per 128 values, and the
// product of such rows with 8-bit weights scaled per 128 x 128 block, grouped
// by expert.
//
//   quantize  m = max |finite x| of a block of 128 (at least 2^-100),
//             scale = m / 448, code = e4m3(448 x / m); NaN and infinities get
//             the code NaN
//   product   y[r][n] = sum_b xs[r][b] ws[g][n / 128][b] P_b,
//             P_b = sum over the 128 columns of block b of x[r][k] w[g][n][k],
//             g the group that row r lies in
//
// A product of two e4m3 values is exact in fp32, so P_b is what the tensor
// core accumulates (kind::f8f6f4, fp32 accumulators in tensor memory); the
// scales cannot enter it, so every block of K has an accumulator of its own
// that the CUDA cores add, times its two scales, to fp32 sums in registers.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "internal.h"
#include "ops.h"
#include "pipeline.cuh"
#include "umma.cuh"

namespace dfm {
namespace {

// ---- quantize -----------------------------------------------------------------
template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

__device__ __forceinline__ bool finite_f32(float v) {
  return (__float_as_uint(v) & 0x7f800000u) != 0x7f800000u;
}

// Two e4m3 codes, nearest even, saturating; NaN gives 0x7f.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

template <typename T, int N>
struct alignas(sizeof(T) * N <= 16 ? sizeof(T) * N : 16) PackQ {
  T v[N];
};

// Half a warp a block of 128: eight values a lane. The quotient 448 x / m is
// taken as (0.875 x) / (m / 512), so that neither side overflows, by
// Markstein's division (IBM J. R&D 34, 1990): with y the rounded reciprocal of
// d, q0 = n y, q = q0 + (n - q0 d) y is the rounded quotient. Ties of bf16
// and fp16 inputs therefore stay ties, and the codes are those of the exact
// quotient. HBM bounds it: 128 (s + 1) + 4 bytes a block of s-byte values.
constexpr int kQThreads = 256, kQUnroll = 2;
template <typename T, bool VEC>
__global__ void __launch_bounds__(kQThreads) fp8_quantize_kernel(const QuantizeArgs p, int nb, uint32_t total) {
  const int hl = threadIdx.x & 15, half = (threadIdx.x >> 4) & 1;
  const uint32_t warps = gridDim.x * (kQThreads / 32);
  const uint32_t warp = blockIdx.x * (kQThreads / 32) + (threadIdx.x >> 5);
  const T* x = static_cast<const T*>(p.x);
  for (uint64_t w0 = warp; 2 * w0 < total; w0 += (uint64_t)warps * kQUnroll) {
    float v[kQUnroll][8];
    uint32_t row[kQUnroll];
    int col[kQUnroll];
    bool there[kQUnroll];
#pragma unroll
    for (int u = 0; u < kQUnroll; ++u) {
      const uint64_t g = 2 * (w0 + (uint64_t)u * warps) + half;
      there[u] = g < total;
      row[u] = there[u] ? (uint32_t)g / (uint32_t)nb : 0;
      col[u] = there[u] ? ((uint32_t)g - row[u] * nb) * 128 : 0;
      const T* src = x + (int64_t)row[u] * p.ldx + col[u];
      if (VEC) {  // lane hl: columns 8 hl .. 8 hl + 7 (K is a multiple of 8)
        if (there[u] && col[u] + 8 * hl < p.K) {
          const PackQ<T, 16 / sizeof(T)>* q = reinterpret_cast<const PackQ<T, 16 / sizeof(T)>*>(src + 8 * hl);
          constexpr int L = 16 / sizeof(T);
#pragma unroll
          for (int i = 0; i < 8 / L; ++i) {
            const PackQ<T, L> r = q[i];
#pragma unroll
            for (int n = 0; n < L; ++n) v[u][i * L + n] = to_f32<T>(r.v[n]);
          }
        } else {
#pragma unroll
          for (int n = 0; n < 8; ++n) v[u][n] = 0.f;
        }
      } else {  // lane hl: columns hl, hl + 16, ...
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const int c = hl + 16 * n;
          v[u][n] = there[u] && col[u] + c < p.K ? to_f32<T>(src[c]) : 0.f;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kQUnroll; ++u) {
      float m = 0x1p-100f;
#pragma unroll
      for (int n = 0; n < 8; ++n) m = fmaxf(m, finite_f32(v[u][n]) ? fabsf(v[u][n]) : 0.f);
#pragma unroll
      for (int o = 8; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float d = m * 0x1p-9f, y = __frcp_rn(d);
      uint32_t code[4];
#pragma unroll
      for (int n = 0; n < 8; n += 2) {
        float q[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float num = v[u][n + i] * 0.875f, q0 = num * y;
          q[i] = fmaf(fmaf(-q0, d, num), y, q0);
          if (!finite_f32(v[u][n + i])) q[i] = __uint_as_float(0x7fffffffu);
        }
        code[n / 2] = e4m3x2(q[0], q[1]);
      }
      if (!there[u]) continue;
      uint8_t* dst = p.codes + (int64_t)row[u] * p.ldc + col[u];
      if (VEC) {
        if (col[u] + 8 * hl < p.K)
          *reinterpret_cast<uint2*>(dst + 8 * hl) =
              make_uint2(code[0] | code[1] << 16, code[2] | code[3] << 16);
      } else {
#pragma unroll
        for (int n = 0; n < 8; ++n)
          if (col[u] + hl + 16 * n < p.K) dst[hl + 16 * n] = (uint8_t)(code[n / 2] >> (8 * (n & 1)));
      }
      if (hl == 0) p.scales[(int64_t)row[u] * p.lds + col[u] / 128] = __fdiv_rn(m, 448.f);
    }
  }
}

template <typename T>
cudaError_t quantize_t(const QuantizeArgs& p, int sms, cudaStream_t s) {
  const int nb = (p.K + 127) / 128;
  const uint64_t total = (uint64_t)p.M * nb;
  const uint64_t blocks = (total + 2 * (kQThreads / 32) - 1) / (2 * (kQThreads / 32));
  const uint64_t most = (uint64_t)sms * 8 * 4;
  const unsigned grid = (unsigned)(blocks < most ? blocks : most);
  const bool vec = !(((uintptr_t)p.x | (uint64_t)(p.ldx * (int64_t)sizeof(T))) & 15) &&
                   !(((uintptr_t)p.codes | (uint64_t)p.ldc) & 7) && p.K % 8 == 0;
  if (vec)
    fp8_quantize_kernel<T, true><<<grid, kQThreads, 0, s>>>(p, nb, (uint32_t)total);
  else
    fp8_quantize_kernel<T, false><<<grid, kQThreads, 0, s>>>(p, nb, (uint32_t)total);
  return cudaGetLastError();
}

// ---- product --------------------------------------------------------------------
// The weights are the 128-row operand (A), NT rows of x the other (B), as in
// the layer's own batch GEMMs: lane = output column n, tensor memory column =
// row of x. A unit is (a tile of NT rows of one group) x (128 columns n), K in
// blocks of 128, the blocks of the scales.
//
// Roles of a CTA: EW epilogue warps, one TMA warp, one MMA warp. The TMA warp
// fills a ring of stages (A 16 KB, B NT x 128 bytes, both in the 128-byte
// swizzle), the MMA warp issues four K = 32 steps a block into the next of AS
// accumulators, and the epilogue warps add the block, times its scales, to
// their registers. With `split` > 1 a cluster of that many CTAs shares a unit:
// each takes a part of K, and the sums meet in distributed shared memory, in
// the order of the parts.
constexpr int kFM = 128;          // rows of A (columns n of y)
constexpr int kFK = 128;          // K a block
constexpr int kFABytes = kFM * kFK;
constexpr int kFBatch = 8;        // blocks whose scales are fetched together

__host__ __device__ constexpr int fp8_ew(int NT) { return NT > 64 ? 8 : 4; }
__host__ __device__ constexpr int fp8_stages(int NT) {
  return NT == 256 ? 4 : NT == 128 ? 6 : NT == 64 ? 4 : 5;
}
__host__ __device__ constexpr int fp8_accs(int NT) { return NT == 256 ? 2 : 4; }
__host__ __device__ constexpr int fp8_cols(int NT) { return NT * fp8_accs(NT); }
__host__ __device__ constexpr int fp8_ctas_per_sm(int NT) { return NT >= 128 ? 1 : 2; }

struct Fp8Params {
  CUtensorMap w, x;
  const float *xs, *ws;
  const int32_t* offs;
  void* y;
  uint32_t* status;
  int64_t M, ldxs, ldy;
  int G, N, K, KB, NB, split;
};

template <int NT>
struct Fp8Smem {
  float sc[2][kFBatch][NT];  // scales of two batches of blocks
  uint64_t full[fp8_stages(NT)], empty[fp8_stages(NT)];
  uint64_t acc_full[fp8_accs(NT)], acc_empty[fp8_accs(NT)];
  int warp_sums[32];
  uint32_t tmem;
  int err;
};

template <int NT>
size_t fp8_smem_bytes(int G) {
  return (size_t)fp8_stages(NT) * (kFABytes + NT * kFK) + sizeof(Fp8Smem<NT>) +
         2 * (size_t)(G + 1) * sizeof(int);
}

// e4m3 x e4m3, fp32 D; `ta`: A is M-major in shared memory.
__device__ __forceinline__ uint32_t idesc_e4m3(int N, int ta) {
  return (1u << 4) | ((uint32_t)ta << 15) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kFM >> 4) << 24);
}

__device__ __forceinline__ uint32_t uni(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b32 r;\n\telect.sync r|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b32 r;\n\telect.sync r|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];\n\t}" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t (&r)[16], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_ld_wait() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// acc += p * s, two fp32 at a time.
__device__ __forceinline__ void fma2(uint64_t& acc, uint32_t p0, uint32_t p1, uint64_t s) {
  asm("{\n\t.reg .b64 p;\n\tmov.b64 p, {%1, %2};\n\tfma.rn.f32x2 %0, p, %3, %0;\n\t}"
      : "+l"(acc)
      : "r"(p0), "r"(p1), "l"(s));
}

__device__ __forceinline__ void put_y(float* y, float v) { *y = v; }
__device__ __forceinline__ void put_y(__nv_bfloat16* y, float v) { *y = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put_y(__half* y, float v) { *y = __float2half_rn(v); }

// What a unit is: `rows` rows of x from `row0`, all of group g, times columns
// n0 .. n0 + 127.
struct Fp8Unit {
  int g, rows, n0;
  int64_t row0;
};

// tiles[g]: row tiles of the groups before g; offs[g]: first row of group g.
template <int NT>
__device__ __forceinline__ Fp8Unit fp8_unit(int u, int NB, int G, const int* tiles, const int* offs) {
  const int tile = u / NB;
  int lo = 0, hi = G - 1;  // the last g with tiles[g] <= tile
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tiles[mid] <= tile) lo = mid;
    else hi = mid - 1;
  }
  Fp8Unit r;
  r.g = lo;
  const int first = NT * (tile - tiles[lo]);
  r.row0 = (int64_t)offs[lo] + first;
  r.rows = min(NT, offs[lo + 1] - offs[lo] - first);
  r.n0 = (u - tile * NB) * kFM;
  return r;
}

template <int NT, bool TRANS, typename Y>
__global__ void __launch_bounds__((fp8_ew(NT) + 2) * 32, fp8_ctas_per_sm(NT))
fp8_matmul_kernel(const __grid_constant__ Fp8Params p) {
  constexpr int EW = fp8_ew(NT), NS = fp8_stages(NT), AS = fp8_accs(NT);
  constexpr int ET = EW * 32, NTHR = ET + 64;
  constexpr int CW = EW == 8 ? NT / 2 : NT;  // accumulator columns a warp holds
  constexpr int kBBytes = NT * kFK;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sa = smem;
  uint8_t* sb = smem + NS * kFABytes;
  Fp8Smem<NT>* sm = reinterpret_cast<Fp8Smem<NT>*>(sb + NS * kBBytes);
  int* tiles = reinterpret_cast<int*>(sm + 1);
  int* offs = tiles + p.G + 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (warp == EW + 1) {
    constexpr uint32_t cols = fp8_cols(NT);
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&sm->tmem)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&sm->full[i], 1);
      mbar_init(&sm->empty[i], 1);
    }
    for (int i = 0; i < AS; ++i) {
      mbar_init(&sm->acc_full[i], 1);
      mbar_init(&sm->acc_empty[i], EW);
    }
    sm->err = 0;
    fence_barrier_init();
  }
  // the groups' first rows, kept inside [0, M] and in order whatever the
  // caller's array holds, and their tiles
  const int M = (int)p.M;
  for (int g = tid; g <= p.G; g += NTHR)
    offs[g] = p.offs ? min(max(p.offs[g], 0), M) : (g ? M : 0);
  __syncthreads();
  {
    int base = 0;
    for (int g0 = 0; g0 < p.G; g0 += NTHR) {
      const int g = g0 + tid;
      const int n = g < p.G ? (max(0, offs[g + 1] - offs[g]) + NT - 1) / NT : 0;
      // exclusive prefix sum over the block
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (lane == 31) sm->warp_sums[warp] = incl;
      __syncthreads();
      int before = base, all = base;
      for (int w = 0; w < NTHR / 32; ++w) {
        if (w < warp) before += sm->warp_sums[w];
        all += sm->warp_sums[w];
      }
      if (g < p.G) tiles[g] = before + incl - n;
      base = all;
      __syncthreads();
    }
    if (tid == 0) tiles[p.G] = base;
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&sm->tmem);
  const int units = tiles[p.G] * p.NB;
  const int part = blockIdx.x % p.split;
  const int first = blockIdx.x / p.split, step = gridDim.x / p.split;
  const int kb0 = (int)((int64_t)p.KB * part / p.split);
  const int kb1 = (int)((int64_t)p.KB * (part + 1) / p.split);

  if (warp == EW) {
    // ---- copies
    int it = 0;
    bool ok = true;
    for (int u = first; u < units && ok; u += step) {
      const Fp8Unit un = fp8_unit<NT>(u, p.NB, p.G, tiles, offs);
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const int s = it % NS;
        ok = it < NS || mbar_wait(&sm->empty[s], ((it / NS) - 1) & 1);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          sm->err = 1;
          break;
        }
        const uint32_t bar = uni(smem_u32(&sm->full[s]));
        const uint32_t da = uni(smem_u32(sa + s * kFABytes)), db = uni(smem_u32(sb + s * kBBytes));
        if (lane == 0) mbar_arrive_expect_tx(&sm->full[s], kFABytes + kBBytes);
        __syncwarp();
        if (TRANS) tma_load_3d(da, &p.w, un.n0, kb * kFK, un.g, bar);
        else tma_load_3d(da, &p.w, kb * kFK, un.n0, un.g, bar);
        tma_load_2d(db, &p.x, kb * kFK, (int)un.row0, bar);
      }
    }
    if (!ok)  // copies in flight land before the block leaves
      for (int i = max(0, it - NS); i < it; ++i) (void)mbar_wait(&sm->full[i % NS], (i / NS) & 1);
  } else if (warp == EW + 1) {
    // ---- MMAs
    const uint32_t idesc = idesc_e4m3(NT, TRANS ? 1 : 0);
    // K step of 32: 32 bytes along a K-major row; 32 rows of 128 bytes M-major
    constexpr uint32_t ka = TRANS ? 32 * 128 / 16 : 2;
    int it = 0;
    bool ok = true;
    for (int u = first; u < units && ok; u += step) {
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const int s = it % NS, as = it % AS;
        ok = mbar_wait(&sm->full[s], (it / NS) & 1) &&
             (it < AS || mbar_wait(&sm->acc_empty[as], ((it / AS) - 1) & 1));
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          sm->err = 1;
          break;
        }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint64_t ad = umma::smem_desc_sw128(smem_u32(sa + s * kFABytes));
        const uint64_t bd = umma::smem_desc_sw128(smem_u32(sb + s * kBBytes));
        asm volatile(
            "{\n\t"
            ".reg .pred e, p0, pt;\n\t"
            ".reg .b32 r;\n\t"
            ".reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
            "elect.sync r|e, 0xffffffff;\n\t"
            "setp.ne.u32 p0, %3, %3;\n\t"
            "setp.eq.u32 pt, %3, %3;\n\t"
            "add.u64 a1, %1, %6;\n\tadd.u64 a2, a1, %6;\n\tadd.u64 a3, a2, %6;\n\t"
            "add.u64 b1, %2, 2;\n\tadd.u64 b2, %2, 4;\n\tadd.u64 b3, %2, 6;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p0;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, pt;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b2, %3, pt;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b3, %3, pt;\n\t"
            "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n\t"
            "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n\t"
            "}" ::"r"(uni(tmem + (uint32_t)(as * NT))),
            "l"(ad), "l"(bd), "r"(idesc), "r"(uni(smem_u32(&sm->empty[s]))),
            "r"(uni(smem_u32(&sm->acc_full[as]))), "n"(ka)
            : "memory");
      }
    }
    // the MMAs issued must land before the tensor memory is released
    if (it > 0) (void)mbar_wait(&sm->empty[(it - 1) % NS], ((it - 1) / NS) & 1);
  } else {
    // ---- sums: warp w reads tensor memory lanes 32 (w % 4) .. + 31
    const int c0 = (warp >> 2) * CW;
    const uint32_t tbase = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + (uint32_t)c0;
    const int nl = 32 * (warp & 3) + lane;
    constexpr int PER = NT * kFBatch / ET;  // scales a thread fetches of a batch
    // a wait that runs out ends every later wait of its warp, but no warp
    // leaves: all of them meet at the named barriers to the end
    int it = 0;
    bool ok = true;
    for (int u = first; u < units; u += step) {
      const Fp8Unit un = fp8_unit<NT>(u, p.NB, p.G, tiles, offs);
      uint64_t acc[CW / 2];
#pragma unroll
      for (int i = 0; i < CW / 2; ++i) acc[i] = 0;
      const float* ws = p.ws + (int64_t)un.g * p.NB * p.KB;
      const int nb = un.n0 / kFM;
      float fetched[PER];
      // the scales of blocks kb .. kb + 7: value i belongs to block i % 8, row i / 8
      auto fetch = [&](int kb) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int v = tid + i * ET, b = kb + (v & (kFBatch - 1)), r = v / kFBatch;
          fetched[i] = 0.f;
          if (b < kb1 && r < un.rows)
            fetched[i] = p.xs[(un.row0 + r) * p.ldxs + b] *
                         (TRANS ? ws[(int64_t)b * p.NB + nb] : ws[(int64_t)nb * p.KB + b]);
        }
      };
      auto store = [&](int buf) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int v = tid + i * ET;
          sm->sc[buf][v & (kFBatch - 1)][v / kFBatch] = fetched[i];
        }
      };
      fetch(kb0);
      named_barrier_sync(1, ET);  // the last unit's scales have been read
      store(0);
      named_barrier_sync(1, ET);
      int buf = 0;
      for (int kb = kb0; kb < kb1; kb += kFBatch) {
        const bool more = kb + kFBatch < kb1;
        if (more) fetch(kb + kFBatch);
        const int blocks = min(kFBatch, kb1 - kb);
        for (int b = 0; b < blocks; ++b, ++it) {
          const int as = it % AS;
          ok = ok && __all_sync(0xffffffffu, mbar_wait(&sm->acc_full[as], (it / AS) & 1));
          if (!ok) {
            sm->err = 1;
            continue;
          }
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const float* sc = &sm->sc[buf][b][c0];
#pragma unroll
          for (int c = 0; c < CW; c += 16) {
            uint32_t r[16];
            tmem_ld16(r, tbase + (uint32_t)(as * NT + c));
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              const ulonglong2 s = *reinterpret_cast<const ulonglong2*>(sc + c + i);
              fma2(acc[(c + i) / 2], r[i], r[i + 1], s.x);
              fma2(acc[(c + i) / 2 + 1], r[i + 2], r[i + 3], s.y);
            }
          }
          asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm->acc_empty[as]);
        }
        if (more) {
          store(buf ^ 1);
          named_barrier_sync(1, ET);
          buf ^= 1;
        }
      }
      float out[CW];
#pragma unroll
      for (int i = 0; i < CW / 2; ++i) {
        out[2 * i] = __uint_as_float((uint32_t)acc[i]);
        out[2 * i + 1] = __uint_as_float((uint32_t)(acc[i] >> 32));
      }
      // a wait that ran out leaves NaN, never a wrong number
      if (!ok) {
#pragma unroll
        for (int i = 0; i < CW; ++i) out[i] = __uint_as_float(0x7fffffffu);
      }
      if (p.split == 1) {
        const int n = un.n0 + nl;
        if (n < p.N) {
          Y* y = static_cast<Y*>(p.y) + (un.row0 + c0) * p.ldy + n;
#pragma unroll
          for (int c = 0; c < CW; ++c)
            if (c0 + c < un.rows) put_y(y + c * p.ldy, out[c]);
        }
      } else {
        // the stages are idle: this part's sums go there, [row][128]
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        float* red = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int c = 0; c < CW; ++c) red[(c0 + c) * kFM + nl] = out[c];
      }
    }
  }
  if (p.split > 1 && first < units) {
    // one unit a cluster: part q sums the rows r = q, q + split, ... over the
    // parts in their order
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    const Fp8Unit un = fp8_unit<NT>(first, p.NB, p.G, tiles, offs);
    const uint32_t red = smem_u32(smem);
    for (int i = tid; i < kFM * un.rows; i += NTHR) {
      const int r = i / kFM, n = i % kFM;
      if (r % p.split != part || un.n0 + n >= p.N) continue;
      float sum = 0.f;
      for (int q = 0; q < p.split; ++q) {
        uint32_t remote;
        float v;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(red + 4 * (r * kFM + n)), "r"(q));
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote) : "memory");
        sum += v;
      }
      put_y(static_cast<Y*>(p.y) + (un.row0 + r) * p.ldy + un.n0 + n, sum);
    }
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (tid == 0 && *(volatile int*)&sm->err && p.status) atomicOr(p.status, DEV_ERR_TIMEOUT);
  if (warp == EW + 1) {
    constexpr uint32_t cols = fp8_cols(NT);
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols)
                 : "memory");
  }
}

PFN_cuTensorMapEncodeTiled_v12000 fp8_encoder() {
  static std::atomic<void*> encode{nullptr};
  void* fn = encode.load();
  if (!fn) {
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || !fn)
      return nullptr;
    encode.store(fn);
  }
  return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
}

// 8-bit [planes][rows][cols], `ld` bytes a row, boxes of 128 columns x
// box_rows rows in the 128-byte swizzle; what lies outside reads as zero.
bool map_u8(CUtensorMap* out, const void* base, int64_t cols, int64_t rows, int64_t planes,
            int64_t ld, int box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = fp8_encoder();
  if (!encode) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)planes};
  const cuuint64_t strides[2] = {(cuuint64_t)ld, (cuuint64_t)(ld * rows)};
  const cuuint32_t box[3] = {kFK, (cuuint32_t)box_rows, 1};
  const cuuint32_t es[3] = {1, 1, 1};
  return encode(out, CU_TENSOR_MAP_DATA_TYPE_UINT8, planes ? 3 : 2, const_cast<void*>(base), dims,
                strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

template <int NT, bool TRANS, typename Y>
const char* fp8_launch(const Fp8MatmulArgs& a, int sms, cudaStream_t s) {
  static_assert(fp8_ctas_per_sm(NT) * (fp8_stages(NT) * (kFABytes + NT * kFK) + sizeof(Fp8Smem<NT>) +
                                       (kOpsMaxExperts + 1) * 8 + 1024) <= 228 * 1024,
                "shared memory");
  Fp8Params p{};
  p.NB = (a.N + kFM - 1) / kFM;
  p.KB = (a.K + kFK - 1) / kFK;
  const bool maps =
      (a.transposed ? map_u8(&p.w, a.w, a.N, a.K, a.G, a.ldw, kFK) : map_u8(&p.w, a.w, a.K, a.N, a.G, a.ldw, kFM)) &&
      map_u8(&p.x, a.x, a.K, a.M, 0, a.ldx, NT);
  if (!maps) return "tensor map encoding failed";
  p.xs = a.xs;
  p.ws = a.ws;
  p.offs = a.offs;
  p.y = a.y;
  p.status = a.status;
  p.M = a.M;
  p.ldxs = a.ldxs;
  p.ldy = a.ldy;
  p.G = a.G;
  p.N = a.N;
  p.K = a.K;
  // at most this many row tiles: every group's last one may be short
  const int64_t tiles = a.M / NT + (a.M < a.G ? a.M : a.G);
  const int64_t units = tiles * p.NB;
  if (units > 0x3fffffff) return "too many tiles";
  const int slots = sms * fp8_ctas_per_sm(NT);
  p.split = 1;
  while (p.split < 8 && 2 * p.split * units <= slots && 2 * p.split <= p.KB) p.split *= 2;
  const int64_t grid = p.split > 1 ? units * p.split : units < slots ? units : slots;
  const size_t smem = fp8_smem_bytes<NT>(a.G);
  auto kernel = fp8_matmul_kernel<NT, TRANS, Y>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return cudaGetErrorString(cudaGetLastError());
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((fp8_ew(NT) + 2) * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  return e == cudaSuccess ? nullptr : cudaGetErrorString(e);
}

template <int NT>
const char* fp8_nt(const Fp8MatmulArgs& a, int dtype, int sms, cudaStream_t s) {
  if (a.transposed)
    return dtype == 0   ? fp8_launch<NT, true, __nv_bfloat16>(a, sms, s)
           : dtype == 1 ? fp8_launch<NT, true, __half>(a, sms, s)
                        : fp8_launch<NT, true, float>(a, sms, s);
  return dtype == 0   ? fp8_launch<NT, false, __nv_bfloat16>(a, sms, s)
         : dtype == 1 ? fp8_launch<NT, false, __half>(a, sms, s)
                      : fp8_launch<NT, false, float>(a, sms, s);
}

}  // namespace

cudaError_t launch_fp8_quantize(const QuantizeArgs& p, int dtype, int sms, cudaStream_t s) {
  return dtype == 0   ? quantize_t<__nv_bfloat16>(p, sms, s)
         : dtype == 1 ? quantize_t<__half>(p, sms, s)
                      : quantize_t<float>(p, sms, s);
}

const char* launch_fp8_matmul(const Fp8MatmulArgs& a, int dtype, int sms, cudaStream_t s) {
  const int64_t groups = a.M < a.G ? a.M : a.G;
  const int64_t mean = (a.M + groups - 1) / groups;
  if (mean <= 16) return fp8_nt<16>(a, dtype, sms, s);
  if (mean <= 32) return fp8_nt<32>(a, dtype, sms, s);
  if (mean <= 64) return fp8_nt<64>(a, dtype, sms, s);
  if (mean <= 128) return fp8_nt<128>(a, dtype, sms, s);
  return fp8_nt<256>(a, dtype, sms, s);
}

}  // namespace dfm
