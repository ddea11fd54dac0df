// k_matmul.cuh — the product of 16-bit matrices with bias, activation and
// residual in its epilogue, and its gradients.
//
//   z = x w' + b             x [M][K], w [N][K] (gated: [2N][K], gate rows first)
//   y = residual + act(z)    gated: act(z) = silu(z_gate) z_up
//   dz = act'(z) dy,  dx = dz w,  dw = dz' x,  db = the column sums of dz
//
// One product serves all three: out[r][c] = sum_k Q[r][k] P[c][k], where
// either operand lies with its k side by side in memory ("K-major": x, w, dz
// in dx) or with its rows side by side ("MN-major": w in dx, dz and x in dw).
// Both kinds of tile are 64 k deep in the 128-byte swizzle; the tensor core's
// descriptors say which it is, so nothing is transposed in memory. Products
// of 16-bit values are exact in fp32 and the sums are fp32 (tensor memory);
// bias, activation and residual are fp32 too, and each output is rounded once.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cstring>

#include "fastmath.cuh"
#include "internal.h"
#include "ops.h"
#include "pipeline.cuh"
#include "tcgen.cuh"
#include "umma.cuh"

namespace dfm {
namespace {

constexpr int kMK = 64;  // k of a stage: 128 bytes, the swizzle's row

// Stages whose products add up in tensor memory, where an addition drops the
// bits behind the last: a sum of K products comes out 1e-9 K too small (relative;
// measured at random operands, K from 64 to 32768). Behind so many the sum goes
// to registers and is added there, rounded to nearest: for an fp32 output 768 of
// k (7e-7; 4096 x 2048 x 8192 9e-6 without), for a 16-bit one, which is rounded
// by 2e-3 or 2e-4 itself, 8192. Sums of positive terms lose more: fp32 outputs
// 4e-7 at K = 768, 1.3e-6 at 8192. The parts are added one behind the other, 6e-8 of
// the sum each at worst, K / 768 or K / 8192 of them (positive terms: 1.5e-6 in all
// at K = 262144, 1.8e-6 at 4194304).
template <int OUT>
constexpr int kChunk = OUT == 2 ? 12 : 128;

// ---- elements of a type (0 bf16, 1 fp16, 2 fp32) -------------------------------
// The kernels have IN and OUT as constants: branches on the type, and code for
// the others between, slowed the epilogue by a third.
__device__ __forceinline__ float half_bits(uint32_t v, int type) {
  return type == 0 ? __uint_as_float(v << 16) : __half2float(__ushort_as_half((unsigned short)v));
}
__device__ __forceinline__ uint32_t pack_bits(float lo, float hi, int type) {
  return type == 0 ? pack16<__nv_bfloat16>(lo, hi) : pack16<__half>(lo, hi);
}

template <typename Y>
__device__ __forceinline__ Y from_f32(float v);
template <>
__device__ __forceinline__ float from_f32(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32(float v) { return __float2half_rn(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

// Columns i, i + step, ... of a row: n of four. VEC: all four, side by side and
// aligned to them.
template <bool VEC>
__device__ __forceinline__ void load_columns(float (&v)[4], const void* p, int64_t i, int step, int n, int type) {
  if constexpr (VEC) {
    if (type == 2) {
      const float4 w = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
      v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
      v[0] = half_bits(w.x & 0xffffu, type), v[1] = half_bits(w.x >> 16, type);
      v[2] = half_bits(w.y & 0xffffu, type), v[3] = half_bits(w.y >> 16, type);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = j >= n ? 0.f : type == 2 ? static_cast<const float*>(p)[i + j * step]
                                      : half_bits(static_cast<const uint16_t*>(p)[i + j * step], type);
  }
}
template <bool VEC>
__device__ __forceinline__ void store_columns(const float (&v)[4], void* p, int64_t i, int step, int n, int type) {
  if constexpr (VEC) {
    if (type == 2)
      *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(v[0], v[1], v[2], v[3]);
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) =
          make_uint2(pack_bits(v[0], v[1], type), pack_bits(v[2], v[3], type));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j >= n) continue;
      if (type == 2) static_cast<float*>(p)[i + j * step] = v[j];
      else static_cast<uint16_t*>(p)[i + j * step] = (uint16_t)(pack_bits(v[j], 0.f, type) & 0xffffu);
    }
  }
}

// Sixteen columns of a row, 32-byte aligned.
__device__ __forceinline__ void load_sixteen(float (&v)[16], const void* p, int64_t i, int type) {
  if (type == 2) {
    const float* f = static_cast<const float*>(p) + i;
#pragma unroll
    for (int h = 0; h < 16; h += 8)
      asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=f"(v[h]), "=f"(v[h + 1]), "=f"(v[h + 2]), "=f"(v[h + 3]), "=f"(v[h + 4]), "=f"(v[h + 5]),
                     "=f"(v[h + 6]), "=f"(v[h + 7])
                   : "l"(f + h));
  } else {
    uint32_t w[8];
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(static_cast<const uint16_t*>(p) + i));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[2 * j] = half_bits(w[j] & 0xffffu, type);
      v[2 * j + 1] = half_bits(w[j] >> 16, type);
    }
  }
}
__device__ __forceinline__ void store_sixteen(const float (&v)[16], void* p, int64_t i, int type) {
  if (type == 2) {
    float* f = static_cast<float*>(p) + i;
#pragma unroll
    for (int h = 0; h < 16; h += 8)
      asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(f + h), "f"(v[h]), "f"(v[h + 1]),
                   "f"(v[h + 2]), "f"(v[h + 3]), "f"(v[h + 4]), "f"(v[h + 5]), "f"(v[h + 6]), "f"(v[h + 7])
                   : "memory");
  } else {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = pack_bits(v[2 * j], v[2 * j + 1], type);
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(static_cast<uint16_t*>(p) + i), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  }
}

// ---- activations --------------------------------------------------------------
__device__ __forceinline__ float relu_f(float z) { return z < 0.f ? 0.f : z; }  // NaN stays
__device__ __forceinline__ void gelu_two(float& a, float& b) {
  const Pair z = pair(a, b);
  Pair density;
  const float2 f = halves(mul2(z, normal_cdf(z, &density)));
  a = f.x, b = f.y;
}
// z becomes act(z); V even but for one value.
template <int V>
__device__ __forceinline__ void act_all(float (&z)[V], const float (&up)[V], int act) {
  switch (act) {
    case kActNone: break;
    case kActRelu:
#pragma unroll
      for (int j = 0; j < V; ++j) z[j] = relu_f(z[j]);
      break;
    case kActSilu:
#pragma unroll
      for (int j = 0; j < V; ++j) z[j] *= sigmoid_f(z[j]);
      break;
    case kActGelu:
#pragma unroll
      for (int j = 0; j < V; j += 2) gelu_two(z[j], z[j + 1]);
      break;
    default:
#pragma unroll
      for (int j = 0; j < V; ++j) z[j] *= sigmoid_f(z[j]) * up[j];
  }
}
// s becomes act'(z).
template <int V>
__device__ __forceinline__ void slope_all(float (&s)[V], const float (&z)[V], int act) {
  switch (act) {
    case kActRelu:
#pragma unroll
      for (int j = 0; j < V; ++j) s[j] = z[j] > 0.f ? 1.f : z[j] != z[j] ? z[j] : 0.f;
      break;
    case kActGelu:
#pragma unroll
      for (int j = 0; j < V; j += 2) {
        const Pair x = pair(z[j], z[j + 1]);
        Pair density;
        const Pair cdf = normal_cdf(x, &density);
        const float2 f = halves(fma2(mul2(x, both(0.398942280f)), density, cdf));
        s[j] = f.x, s[j + 1] = f.y;
      }
      break;
    default:  // silu, and the gate's of swiglu
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float g = sigmoid_f(z[j]);
        s[j] = g * fmaf(z[j], 1.f - g, 1.f);
      }
  }
}

// ---- product ------------------------------------------------------------------
struct GemmParams {
  CUtensorMap c, r;  // the operands whose rows are the output's columns and rows
  const void *bias, *residual;
  void *pre, *y;
  uint32_t* status;
  int64_t R, ldr, ldp, ldy;
  int C, KB;             // output columns (of y), stages of k
  int in, out;           // types of the operands, bias and pre; of y and residual
  int act, c_mn, r_mn;   // the activation; operands that are MN-major
  int units_r, units, split;
  int vec;               // the arrays are aligned to what a thread writes
  int give_up;           // test hook: the role of block 0 that gives up before its first wait
  int order;             // kGemmFirst, kGemmSecond
};
enum GemmRole { kGemmNone = 0, kGemmCopies, kGemmMmas, kGemmSums };

// Instruction descriptor of kind::f16 (fp32 D, both operands of one type):
// type 0 bf16, 1 fp16; ta, tb: A is M-major, B N-major in shared memory.
__device__ __forceinline__ uint32_t gemm_idesc(int type, int M, int N, int ta, int tb) {
  return (type == 0 ? umma::idesc_bf16_f32(M, N) : umma::idesc_f16_f32(M, N)) | ((uint32_t)ta << 15) | ((uint32_t)tb << 16);
}
// Low word of a tile's descriptor, and how far 16 of k move it. K-major: rows
// of 128 bytes, a step of 32 bytes along them. MN-major: rows of k hold 64
// values of MN (128 bytes), the next 64 lie 64 rows (8192 bytes) further, and
// a step is 16 rows. Either has atoms of 8 rows (1024 bytes), the high word.
constexpr uint32_t kDescHi = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, int mn) {
  return ((saddr >> 4) & 0x3FFFu) | (mn ? (8192u >> 4) << 16 : 1u << 16);
}
__device__ __forceinline__ uint32_t desc_step(int mn) { return mn ? 16 * 128 / 16 : 2; }

// The two products of a gradient run side by side where one leaves SMs free (and
// the second's start under the first's end): the first lets the second start
// when its own blocks have what they need, which is when all that came before
// the two is complete, and the second waits for the first only behind its own
// work, so that what follows finds both complete (256 x 512 x 512 6.7 us, one behind
// the other 11; 1024 x 1024 x 1024 10.3 and 16.3). That the second sees what came
// before is inferred, not promised in so many words (visibility is promised to a grid
// that waits): every block of the first has waited before it lets the second start,
// so what the second reads (dz or dy, and x: nothing of the first's) is complete and
// visible on the device by then, and it reads it by copies that do not pass L1.
__device__ __forceinline__ void product_wait(const GemmParams& p) {
  if (p.order != kGemmSecond) pdl_wait();  // the kernel before this one is complete
}
__device__ __forceinline__ void product_started(const GemmParams& p) {
  if (p.order == kGemmFirst) pdl_launch_dependents();
}
__device__ __forceinline__ void product_end(const GemmParams& p) {
  if (p.order == kGemmSecond) pdl_wait();
}

// The four steps of 16 of a stage; acc: added to what D holds. Issued by the
// lane with `leader`.
__device__ __forceinline__ void gemm_stage(uint32_t d, uint32_t ad, uint32_t as, uint32_t bd, uint32_t bs, uint32_t idesc,
                                           uint32_t acc, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred e, p0, pt;\n\t.reg .b32 l;\n\t.reg .b64 a0, a1, a2, a3, b0, b1, b2, b3;\n\t"
      "setp.ne.u32 e, %7, 0;\n\tsetp.ne.u32 p0, %6, 0;\n\tsetp.eq.u32 pt, %3, %3;\n\t"
      "mov.b64 a0, {%1, %8};\n\tmov.b64 b0, {%2, %8};\n\t"
      "add.u32 l, %1, %4;\n\tmov.b64 a1, {l, %8};\n\t"
      "add.u32 l, l, %4;\n\tmov.b64 a2, {l, %8};\n\t"
      "add.u32 l, l, %4;\n\tmov.b64 a3, {l, %8};\n\t"
      "add.u32 l, %2, %5;\n\tmov.b64 b1, {l, %8};\n\t"
      "add.u32 l, l, %5;\n\tmov.b64 b2, {l, %8};\n\t"
      "add.u32 l, l, %5;\n\tmov.b64 b3, {l, %8};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a0, b0, %3, p0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, pt;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, pt;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, pt;\n\t}" ::"r"(d),
      "r"(ad), "r"(bd), "r"(idesc), "r"(as), "r"(bs), "r"(acc), "r"(leader), "n"(kDescHi)
      : "memory");
}

// An accumulator has been read: into registers, once tcgen05.wait::ld is over, so
// that no memory has to be released with the arrival (a release waits for the
// warp's stores to global memory, 2000 cycles behind an epilogue).
__device__ __forceinline__ void arrive_read(uint32_t bar, uint32_t leader) {
  asm volatile("{\n\t.reg .pred e;\n\tsetp.ne.u32 e, %1, 0;\n\t@e mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n\t}" ::"r"(bar),
               "r"(leader)
               : "memory");
}

// Columns c, c + step, ... (four) of output row `row`: z (and, gated, up)
// come without the bias.
template <bool VEC, int IN, int OUT>
__device__ __forceinline__ void gemm_finish(const GemmParams& p, int64_t row, int c, int step, float (&z)[4], float (&up)[4]) {
  const int n = c >= p.C ? 0 : min(4, (p.C - c + step - 1) / step);
  if (n <= 0) return;
  const bool gated = p.act == kActSwiglu;
  float v[4];
  if (p.bias) {
    load_columns<VEC>(v, p.bias, c, step, n, IN);
#pragma unroll
    for (int j = 0; j < 4; ++j) z[j] += v[j];
    if (gated) {
      load_columns<VEC>(v, p.bias, (int64_t)p.C + c, step, n, IN);
#pragma unroll
      for (int j = 0; j < 4; ++j) up[j] += v[j];
    }
  }
  if (p.pre) {
    store_columns<VEC>(z, p.pre, row * p.ldp + c, step, n, IN);
    if (gated) store_columns<VEC>(up, p.pre, row * p.ldp + p.C + c, step, n, IN);
  }
  act_all(z, up, p.act);
  if (p.residual) {
    load_columns<VEC>(v, p.residual, row * p.ldr + c, step, n, OUT);
#pragma unroll
    for (int j = 0; j < 4; ++j) z[j] += v[j];
  }
  store_columns<VEC>(z, p.y, row * p.ldy + c, step, n, OUT);
}

// A unit: 128 columns of the output (gated: 64, with the gate's and the up
// product's rows of w) as the tensor core's 128 rows, times NT rows of it.
// A cluster of `split` CTAs shares it, each with a part of k; the sums meet in
// distributed shared memory in the order of the parts, where the epilogue
// reads them along the rows. The 128-row operand is the one with the output's
// columns because with few rows it is the weights, which stream: HBM and the start
// bound it (1 x 7168 x 2048 6.9 to 7.2 us, 4.1 to 4.3 TB/s; 24 x 2048 x 7168 swiglu 15,
// 3.9 TB/s).
template <int NT>
struct GemmCfg {
  static constexpr int NS = NT <= 16 ? 6 : NT <= 32 ? 5 : 4;  // stages
  static constexpr int CBytes = 128 * kMK * 2, RBytes = NT * kMK * 2;
  static constexpr uint32_t Cols = 2 * NT;  // two accumulators, for sums of many chunks
  static constexpr int NTHR = 256;
  static_assert(NS * (CBytes + RBytes) >= 128 * NT * 4, "the sums fit the stages");
};
struct GemmSmem {
  uint64_t full[8], empty[8], acc_full[2], acc_empty[2];
  uint32_t tmem;
  int err;
};
template <int NT>
constexpr size_t gemm_smem_bytes() {
  return (size_t)GemmCfg<NT>::NS * (GemmCfg<NT>::CBytes + GemmCfg<NT>::RBytes) + sizeof(GemmSmem);
}

// The sums of SPLIT parts, [row][128] in shared memory of the cluster's CTAs:
// four columns of a row a thread, 32 such items a warp and step, the CTAs in
// turn.
template <int SPLIT, int IN, int OUT>
__device__ __forceinline__ void split_epilogue(const GemmParams& p, const float* red, int part, int64_t r0, int rows, int c0, bool gated) {
  constexpr int WARPS = GemmCfg<16>::NTHR / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quads = gated ? 16 : 32;
  const int step = p.vec ? 1 : quads;
  // the other CTAs' sums, by addresses that the compiler knows nothing of
  // before the barrier (loads of asm that may be reordered among others)
  uint32_t base[SPLIT];
#pragma unroll
  for (int q = 0; q < SPLIT; ++q)
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(base[q]) : "r"(smem_u32(red)), "r"(q) : "memory");
  const auto sums = [&](float (&v)[4], int i) {
    if constexpr (SPLIT == 1) {
      if (p.vec) {
        const float4 f = *reinterpret_cast<const float4*>(red + i);
        v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = red[i + j * step];
      }
    } else {
    float w[SPLIT][4];
#pragma unroll
    for (int q = 0; q < SPLIT; ++q) {
      const uint32_t at = base[q] + 4 * i;
      if (p.vec) {
        asm("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(w[q][0]), "=f"(w[q][1]), "=f"(w[q][2]), "=f"(w[q][3]) : "r"(at));
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) asm("ld.shared::cluster.f32 %0, [%1];" : "=f"(w[q][j]) : "r"(at + 4 * j * step));
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = w[0][j];
#pragma unroll
      for (int q = 1; q < SPLIT; ++q) v[j] += w[q][j];
    }
    }
  };
#pragma unroll 2
  for (int g = part * WARPS + warp; 32 * g < rows * quads; g += SPLIT * WARPS) {
    const int item = 32 * g + lane, q = gated ? item >> 4 : item >> 5, l = item & (quads - 1);
    if (q >= rows) continue;
    const int c = p.vec ? 4 * l : l;
    float z[4], up[4] = {0.f, 0.f, 0.f, 0.f};
    sums(z, q * 128 + c);
    if (gated) sums(up, q * 128 + 64 + c);
    if (p.vec) gemm_finish<true, IN, OUT>(p, r0 + q, c0 + c, 1, z, up);
    else gemm_finish<false, IN, OUT>(p, r0 + q, c0 + c, step, z, up);
  }
}

template <int NT, int IN, int OUT>
__global__ void __launch_bounds__(GemmCfg<NT>::NTHR, 2)
gemm_split_kernel(const __grid_constant__ GemmParams p) {
  using G = GemmCfg<NT>;
  constexpr int NS = G::NS;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sc = smem;
  uint8_t* sr = smem + NS * G::CBytes;
  GemmSmem* sm = reinterpret_cast<GemmSmem*>(sr + NS * G::RBytes);
  const int tid = threadIdx.x, lane = tid & 31, warp = (int)uni(tid >> 5);
  if (tid == 32) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&p.c) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&p.r) : "memory");
  }
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&sm->full[i], 1);
      mbar_init(&sm->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm->acc_full[i], 1);
      mbar_init(&sm->acc_empty[i], 4);
    }
    sm->err = 0;
    fence_barrier_init();
  }
  product_wait(p);  // tensor memory only from here on
  if (warp == 6) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm->tmem)), "r"(G::Cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  product_started(p);
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&sm->tmem);
  const bool gated = p.act == kActSwiglu;
  const int width = gated ? 64 : 128;
  const int part = blockIdx.x % p.split, unit = blockIdx.x / p.split;
  const int tile_c = unit / p.units_r, tile_r = unit - tile_c * p.units_r;
  const int c0 = tile_c * width;
  const int64_t r0 = (int64_t)tile_r * NT;
  const int kb0 = (int)((int64_t)p.KB * part / p.split), kb1 = (int)((int64_t)p.KB * (part + 1) / p.split);
  const int gives_up = blockIdx.x == 0 ? p.give_up : kGemmNone;
  const uint32_t limit = gives_up ? kTestWaitLimit : kWaitLimit;
  float* red = reinterpret_cast<float*>(smem);  // the sums, [NT][128], where the stages were

  if (warp == 4) {
    // ---- copies, issued by one lane
    const uint32_t leader = elect_one(), sc0 = uni(smem_u32(sc)), sr0 = uni(smem_u32(sr));
    const uint32_t full = uni(smem_u32(sm->full)), empty = uni(smem_u32(sm->empty));
    const int cc = (int)uni(c0), rr = (int)uni((uint32_t)r0);
    int s = 0, kb = kb0;
    uint32_t phase = 1;  // the first round finds every stage free
    bool ok = gives_up != kGemmCopies;
    for (; kb < kb1 && ok; ++kb) {
      ok = bar_wait(empty + 8 * s, phase, limit);
      if (!ok) break;
      const uint32_t bar = full + 8 * s, dc = sc0 + s * G::CBytes, dr = sr0 + s * G::RBytes;
      expect_tx(bar, G::CBytes + G::RBytes, leader);
      const int k = kb * kMK;
      if (p.c_mn) {
        tma_load_2d(dc, &p.c, cc, k, bar, leader);
        tma_load_2d(dc + 8192, &p.c, cc + 64, k, bar, leader);
      } else {  // boxes of 64 rows
        tma_load_2d(dc, &p.c, k, cc, bar, leader);
        tma_load_2d(dc + 8192, &p.c, k, gated ? p.C + cc : cc + 64, bar, leader);
      }
      if (p.r_mn) {
#pragma unroll
        for (int i = 0; i < NT; i += 64) tma_load_2d(dr + 128 * i, &p.r, rr + i, k, bar, leader);
      } else {
        tma_load_2d(dr, &p.r, k, rr, bar, leader);
      }
      if (++s == NS) {
        s = 0;
        phase ^= 1;
      }
    }
    if (!ok) sm->err = 1;
    // copies in flight land before the block goes on
    const int issued = kb - kb0;
    for (int i = 0; i < NS && i < issued; ++i) (void)bar_wait(full + 8 * i, ((issued - 1 - i) / NS) & 1, kWaitLimit);
  } else if (warp == 5) {
    // ---- MMAs, issued by one lane
    const uint32_t leader = elect_one(), tm = uni(tmem);
    const uint32_t a0 = uni(desc_lo(smem_u32(sc), p.c_mn)), b0 = uni(desc_lo(smem_u32(sr), p.r_mn));
    const uint32_t as = uni(desc_step(p.c_mn)), bs = uni(desc_step(p.r_mn));
    const uint32_t idesc = uni(gemm_idesc(IN, 128, NT, p.c_mn, p.r_mn));
    const uint32_t full = uni(smem_u32(sm->full)), empty = uni(smem_u32(sm->empty));
    const uint32_t acc_full = uni(smem_u32(sm->acc_full)), acc_empty = uni(smem_u32(sm->acc_empty));
    bool ok = gives_up != kGemmMmas;
    int s = 0, kb = kb0, chunk = 0, in = 0;  // stages in the chunk
    uint32_t phase = 0;
    for (; kb < kb1 && ok; ++kb, ++in) {
      if (in == kChunk<OUT>) {
        mma_commit(acc_full + 8 * (chunk & 1), leader);
        ++chunk, in = 0;
        ok = bar_wait(acc_empty + 8 * (chunk & 1), (chunk >> 1 & 1) ^ 1, limit);  // the first two find theirs free
        if (!ok) break;
      }
      ok = bar_wait(full + 8 * s, phase, limit);
      if (!ok) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      gemm_stage(tm + NT * (chunk & 1), a0 + (uint32_t)(s * (G::CBytes >> 4)), as, b0 + (uint32_t)(s * (G::RBytes >> 4)), bs, idesc,
                 in > 0, leader);
      mma_commit(empty + 8 * s, leader);
      if (++s == NS) {
        s = 0;
        phase ^= 1;
      }
    }
    if (!ok) sm->err = 1;
    // MMAs issued, and their arrivals, land before tensor memory is released
    mma_commit(acc_full + 8 * (chunk & 1), leader);
    const int issued = kb - kb0;
    for (int i = 0; i < NS && i < issued; ++i) (void)bar_wait(empty + 8 * i, ((issued - 1 - i) / NS) & 1, kWaitLimit);
    if (chunk > 0) (void)bar_wait(acc_full + 8 * (chunk - 1 & 1), chunk - 1 >> 1 & 1, kWaitLimit);
    (void)bar_wait(acc_full + 8 * (chunk & 1), chunk >> 1 & 1, kWaitLimit);
  } else if (warp < 4) {
    // ---- sums to shared memory: lane = column
    const int chunks = (kb1 - kb0 + kChunk<OUT> - 1) / kChunk<OUT>;
    const uint32_t acc_full = smem_u32(sm->acc_full), acc_empty = smem_u32(sm->acc_empty);
    bool ok = gives_up != kGemmSums;
    float sum[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) sum[i] = 0.f;
#pragma unroll 1
    for (int chunk = 0; chunk < chunks; ++chunk) {
      ok = ok && bar_wait(acc_full + 8 * (chunk & 1), chunk >> 1 & 1, limit);
      if (!ok) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t ta = tmem + ((uint32_t)(32 * warp) << 16) + NT * (chunk & 1);
      uint32_t v[2][16];
      tmem_ld_rows(v[0], ta);
#pragma unroll
      for (int i = 0; i < NT / 16; ++i) {
        tmem_wait(v[i & 1]);
        if (i + 1 < NT / 16) tmem_ld_rows(v[(i + 1) & 1], ta + 16 * (i + 1));
#pragma unroll
        for (int j = 0; j < 16; ++j) sum[16 * i + j] += __uint_as_float(v[i & 1][j]);
      }
      if (chunk + 1 < chunks) {
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        arrive_read(acc_empty + 8 * (chunk & 1), lane == 0);
      }
    }
    if (!ok) {
      sm->err = 1;
    } else {  // no MMA reads the stages any more
#pragma unroll
      for (int i = 0; i < NT; ++i) red[i * 128 + 32 * warp + lane] = sum[i];
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (*(volatile int*)&sm->err) {  // a wait ran out: NaN
    for (int i = tid; i < 128 * NT; i += G::NTHR) red[i] = __uint_as_float(0x7fffffffu);
    if (tid == 0 && p.status) atomicOr(p.status, DEV_ERR_TIMEOUT);
    __syncthreads();
  }
  if (warp == 6)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(G::Cols) : "memory");
  if (p.split > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  // ---- epilogue
  const int rows = (int)min((int64_t)NT, p.R - r0);
  switch (p.split) {
    case 1: split_epilogue<1, IN, OUT>(p, red, part, r0, rows, c0, gated); break;
    case 2: split_epilogue<2, IN, OUT>(p, red, part, r0, rows, c0, gated); break;
    case 4: split_epilogue<4, IN, OUT>(p, red, part, r0, rows, c0, gated); break;
    default: split_epilogue<8, IN, OUT>(p, red, part, r0, rows, c0, gated);
  }
  if (p.split > 1) {  // nobody leaves while its sums are read
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  product_end(p);
}

// ---- long products: a pair of CTAs on 256 rows x 256 columns -----------------
// Each CTA of the pair (a cluster of two) has 128 of the rows and half of the
// columns' operand; one of them, the leader, issues cta_group::2 MMAs of 256 x
// 256 x 16 over both, so that each operand byte in shared memory feeds twice the
// products of a 128 x 256 tile. Persistent: the pairs take units in turn, and
// two accumulators (all of tensor memory) let the epilogue of one unit run under
// the MMAs of the next. Gated: the first CTA's half of the columns' operand is
// the gate's rows of w, the second's the up product's, so that a unit is 128
// columns and both products of a column sit in the same tensor memory lane.
// BN columns: 256, or 128 where those leave SMs without a unit. The tensor pipe
// bounds it, active 94% of the time in long units (8192 x 7168 x 7168 420 to 440 us,
// 1.9 to 2.0 PFLOP/s as the card's power allows; with bias, gelu and z kept 525);
// with few k the epilogue's stores (4096 x 19456 x 64 46 us, 3.5 TB/s).
template <int BN>
struct PairCfg {
  static constexpr int NS = BN == 256 ? 6 : 8, EW = 8, NTHR = (EW + 4) * 32;
  static constexpr int RBytes = 128 * kMK * 2, CBytes = BN / 2 * kMK * 2;  // the operands' parts of a stage
  static constexpr int Stage = RBytes + CBytes;
};
template <int BN>
struct PairSmem {
  using G = PairCfg<BN>;
  float turn[G::EW][32 * 32];  // what a warp turns
  uint64_t full[G::NS], empty[G::NS], acc_full[2], acc_empty[2];
  uint32_t tmem;
  int err;
};
template <int BN>
constexpr size_t pair_bytes() {
  return (size_t)PairCfg<BN>::NS * PairCfg<BN>::Stage + sizeof(PairSmem<BN>);
}

// What a unit is: units go down eight row tiles before the next column tile, so
// that the pairs at work share their operands in L2.
struct PairUnit {
  int r0, c0;
};
__device__ __forceinline__ PairUnit pair_unit(int u, const GemmParams& p, int width) {
  const int units_c = p.units / p.units_r, band = u / (8 * units_c), in = u - band * 8 * units_c;
  const int tall = min(8, p.units_r - 8 * band), c = in / tall;
  return {256 * (8 * band + in - c * tall), width * c};
}

// A tile of this CTA, signalled at the leader's barrier.
__device__ __forceinline__ void pair_load(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.u32 e, %3, 0;\n\t"
      "@e cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%4, %5}], [%2];\n\t}" ::"r"(dst),
      "l"(map), "r"(bar), "r"(leader), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void pair_stage(uint32_t d, uint32_t ad, uint32_t as, uint32_t bd, uint32_t bs, uint32_t idesc,
                                           uint32_t acc, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred e, p0, pt;\n\t.reg .b32 l;\n\t.reg .b64 a0, a1, a2, a3, b0, b1, b2, b3;\n\t"
      "setp.ne.u32 e, %7, 0;\n\tsetp.ne.u32 p0, %6, 0;\n\tsetp.eq.u32 pt, %3, %3;\n\t"
      "mov.b64 a0, {%1, %8};\n\tmov.b64 b0, {%2, %8};\n\t"
      "add.u32 l, %1, %4;\n\tmov.b64 a1, {l, %8};\n\t"
      "add.u32 l, l, %4;\n\tmov.b64 a2, {l, %8};\n\t"
      "add.u32 l, l, %4;\n\tmov.b64 a3, {l, %8};\n\t"
      "add.u32 l, %2, %5;\n\tmov.b64 b1, {l, %8};\n\t"
      "add.u32 l, l, %5;\n\tmov.b64 b2, {l, %8};\n\t"
      "add.u32 l, l, %5;\n\tmov.b64 b3, {l, %8};\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a0, b0, %3, p0;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a1, b1, %3, pt;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a2, b2, %3, pt;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a3, b3, %3, pt;\n\t}" ::"r"(d),
      "r"(ad), "r"(bd), "r"(idesc), "r"(as), "r"(bs), "r"(acc), "r"(leader), "n"(kDescHi)
      : "memory");
}
// The barrier at this place in both CTAs completes when the MMAs so far have.
__device__ __forceinline__ void pair_commit(uint32_t bar, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b16 m;\n\tsetp.ne.u32 e, %1, 0;\n\tmov.b16 m, 3;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(bar),
      "r"(leader)
      : "memory");
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// 32 rows x 32 columns of a warp, a row a lane, to rows of global memory that
// nothing is known of: turned in shared memory (value (r, c) stands at 32 r + (c ^
// r)), so that a store covers a piece of one row. `rows`, `cols`: those there are.
template <typename Y>
__device__ __forceinline__ void put_rows(float* turn, const float (&v)[32], Y* to, int64_t ld, int rows, int cols) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < 32; ++j) turn[32 * lane + (j ^ lane)] = v[j];
  __syncwarp();
  if (lane < cols) {
    to += lane;
#pragma unroll 8
    for (int r = 0; r < rows; ++r, to += ld) *to = from_f32<Y>(turn[32 * r + (lane ^ r)]);
  }
  __syncwarp();
}
__device__ __forceinline__ void put_rows(float* turn, const float (&v)[32], void* to, int64_t at, int64_t ld, int rows, int cols, int type) {
  if (type == 0) put_rows(turn, v, static_cast<__nv_bfloat16*>(to) + at, ld, rows, cols);
  else if (type == 1) put_rows(turn, v, static_cast<__half*>(to) + at, ld, rows, cols);
  else put_rows(turn, v, static_cast<float*>(to) + at, ld, rows, cols);
}
// The other way: v += the rows' values.
template <typename Y>
__device__ __forceinline__ void add_rows(float* turn, float (&v)[32], const Y* from, int64_t ld, int rows, int cols) {
  const int lane = threadIdx.x & 31;
  if (lane < cols) {
    from += lane;
#pragma unroll 8
    for (int r = 0; r < rows; ++r, from += ld) turn[32 * r + (lane ^ r)] = to_f32(*from);
  }
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] += turn[32 * lane + (j ^ lane)];
  __syncwarp();
}
__device__ __forceinline__ void add_rows(float* turn, float (&v)[32], const void* from, int64_t at, int64_t ld, int rows, int cols, int type) {
  if (type == 0) add_rows(turn, v, static_cast<const __nv_bfloat16*>(from) + at, ld, rows, cols);
  else if (type == 1) add_rows(turn, v, static_cast<const __half*>(from) + at, ld, rows, cols);
  else add_rows(turn, v, static_cast<const float*>(from) + at, ld, rows, cols);
}
// The epilogue of such a piece: z (and, gated, up) come without the bias, of
// which a lane has that of its column.
template <int IN, int OUT>
__device__ __forceinline__ void finish_rows(const GemmParams& p, float* turn, int64_t r0, int rows, int c, float (&z)[32], float (&up)[32],
                                            float bias, float bias_up) {
  const int cols = min(32, p.C - c);
  if (rows <= 0 || cols <= 0) return;  // of the whole warp
  const bool gated = p.act == kActSwiglu;
  if (p.bias) {
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      z[j] += __shfl_sync(0xffffffffu, bias, j);
      if (gated) up[j] += __shfl_sync(0xffffffffu, bias_up, j);
    }
  }
  if (p.pre) {
    put_rows(turn, z, p.pre, r0 * p.ldp + c, p.ldp, rows, cols, IN);
    if (gated) put_rows(turn, up, p.pre, r0 * p.ldp + p.C + c, p.ldp, rows, cols, IN);
  }
  act_all(z, up, p.act);
  if (p.residual) add_rows(turn, z, p.residual, r0 * p.ldr + c, p.ldr, rows, cols, OUT);
  put_rows(turn, z, p.y, r0 * p.ldy + c, p.ldy, rows, cols, OUT);
}

// The epilogue has read its accumulator; the leader's MMAs may have it.
__device__ __forceinline__ void pair_release(uint32_t bar, bool ok) {
  if (!ok || !bar) return;
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncwarp();
  arrive_read(bar, (threadIdx.x & 31) == 0);
}

// What a warp has of a unit: 32 rows from r0 (`rows` of them there), columns c0
// .. + cols of the output, from tensor memory at ta (gated: the up product's
// `up` columns further), with the bias of columns lane, lane + 32, ...
struct WarpTile {
  int64_t r0;
  int rows, c0, cols;
  uint32_t ta, release;
  float bias[4], bias_up[2];
  __device__ __forceinline__ float bias_of(int i) const { return i < 32 ? bias[0] : i < 64 ? bias[1] : i < 96 ? bias[2] : bias[3]; }
  __device__ __forceinline__ float bias_up_of(int i) const { return i < 32 ? bias_up[0] : bias_up[1]; }
};

// Rows that start their groups of sixteen columns on 32-byte boundaries and have
// no part of one: a row a lane, in a loop that stays small (two warps a
// scheduler hide neither its loads from memory nor those of instructions) and
// has nothing of other activations between.
template <int IN, int OUT, int ACT>
__device__ __forceinline__ void finish_straight(const GemmParams& p, const WarpTile& t, int up_at, bool ok) {
  constexpr bool gated = ACT == kActSwiglu;
  const int lane = threadIdx.x & 31;
  const int64_t row = t.r0 + lane;
#pragma unroll 1
  for (int i = 0; i < t.cols; i += 16) {
    uint32_t zr[16], ur[16];
    float z[16], up[gated ? 16 : 1], v[16];
    __syncwarp();  // rows that are not there come back
    if (ok) {
      tmem_ld_rows(zr, t.ta + i);
      if (gated) tmem_ld_rows(ur, t.ta + up_at + i);
    }
    const int c = t.c0 + i;
    const bool there = lane < t.rows && c < p.C;
    if (p.residual && there) load_sixteen(v, p.residual, row * p.ldr + c, OUT);  // on its way meanwhile
    if (ok) {
      if (gated) tmem_wait(ur);
      tmem_wait(zr);
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) zr[j] = ur[j] = 0x7fffffffu;  // NaN
    }
    if (i + 16 == t.cols) pair_release(t.release, ok);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      z[j] = __uint_as_float(zr[j]);
      if (gated) up[j % (gated ? 16 : 1)] = __uint_as_float(ur[j]);
    }
    if (p.bias) {
      const float b = t.bias_of(i), bu = t.bias_up_of(i);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        z[j] += __shfl_sync(0xffffffffu, b, (i & 16) + j);
        if (gated) up[j % (gated ? 16 : 1)] += __shfl_sync(0xffffffffu, bu, (i & 16) + j);
      }
    }
    if (!there) continue;
    if (p.pre) {
      store_sixteen(z, p.pre, row * p.ldp + c, IN);
      if constexpr (gated) store_sixteen(up, p.pre, row * p.ldp + p.C + c, IN);
    }
    if constexpr (gated) act_all(z, up, ACT);
    else act_all(z, z, ACT);
    if (p.residual) {
#pragma unroll
      for (int j = 0; j < 16; ++j) z[j] += v[j];
    }
    store_sixteen(z, p.y, row * p.ldy + c, OUT);
  }
}

// The BN / 2 columns of a warp in an accumulator, sixteen at a time: from ta on,
// or (gated) half of them there and half among the up product's.
template <int BN>
__device__ __forceinline__ uint32_t sixteen_at(uint32_t ta, int i, bool gated) {
  return ta + 16 * i + (gated && i >= BN / 64 ? BN / 2 - BN / 4 : 0);
}
// sum += the accumulator's.
template <int BN>
__device__ __forceinline__ void add_chunk(float (&sum)[BN / 2], uint32_t ta, bool gated) {
  constexpr int G = BN == 128 ? 4 : 2;  // on their way together, as registers allow
#pragma unroll
  for (int i = 0; i < BN / 32; i += G) {
    uint32_t v[G][16];
#pragma unroll
    for (int g = 0; g < G; ++g) tmem_ld_rows(v[g], sixteen_at<BN>(ta, i + g, gated));
#pragma unroll
    for (int g = 0; g < G; ++g) {
      tmem_wait(v[g]);
#pragma unroll
      for (int j = 0; j < 16; ++j) sum[16 * (i + g) + j] += __uint_as_float(v[g][j]);
    }
  }
}
// The sums to the accumulator's place, where the epilogue finds them.
template <int BN>
__device__ __forceinline__ void put_sums(const float (&sum)[BN / 2], uint32_t ta, bool gated) {
#pragma unroll
  for (int i = 0; i < BN / 32; ++i) {
    const float* v = sum + 16 * i;
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(
            sixteen_at<BN>(ta, i, gated)),
        "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]), "f"(v[10]),
        "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
        : "memory");
  }
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// MANY: units of more than one chunk (a kernel of their own: the chunks' sums
// cost the others registers). The vectors' epilogue spills some registers a unit: 52
// to 124 bytes a thread, with MANY 176 to 612.
template <int BN, int IN, int OUT, bool VEC, bool MANY>
__global__ void __launch_bounds__(PairCfg<BN>::NTHR, 1) gemm_pair_kernel(const __grid_constant__ GemmParams p) {
  using G = PairCfg<BN>;
  static_assert(pair_bytes<BN>() <= 227 * 1024, "shared memory");
  constexpr int NS = G::NS, EW = G::EW;
  // the sums' own place in tensor memory, behind the two accumulators, where it is large enough
  constexpr bool SPARE = MANY && BN == 128;
  constexpr uint32_t COLS = SPARE ? 4 * BN : 2 * BN;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sr = smem;                       // rows' operand: the 128-row operand of each CTA
  uint8_t* sc = smem + NS * G::RBytes;      // columns' operand
  PairSmem<BN>* sm = reinterpret_cast<PairSmem<BN>*>(smem + NS * G::Stage);
  const int tid = threadIdx.x, lane = tid & 31, warp = (int)uni(tid >> 5);
  const int rank = blockIdx.x & 1;
  if (tid == 32 * EW) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&p.c) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&p.r) : "memory");
  }
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&sm->full[i], 1);
      mbar_init(&sm->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm->acc_full[i], 1);
      mbar_init(&sm->acc_empty[i], 2 * EW);
    }
    sm->err = 0;
    fence_barrier_init();
  }
  product_wait(p);  // tensor memory only from here on
  if (warp == EW + 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm->tmem)), "r"(COLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  cluster_barrier();  // both CTAs' barriers are there
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  product_started(p);
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&sm->tmem);
  const bool gated = p.act == kActSwiglu;
  const int width = gated ? BN / 2 : BN;
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
  // the test hook: a role of block 0 gives up, the pair's other waits are short
  const int gives_up = blockIdx.x == 0 ? p.give_up : kGemmNone;
  const uint32_t limit = first == 0 && p.give_up ? kTestWaitLimit : kWaitLimit;

  // registers go from the warps that issue to those of the epilogue
  // (128 x 72 + 256 x 216 are the 384 x 168 of the launch)
  if (warp >= EW) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == EW) {
      // ---- copies, issued by one lane
      const uint32_t leader = elect_one(), sr0 = uni(smem_u32(sr)), sc0 = uni(smem_u32(sc));
      const uint32_t empty = uni(smem_u32(sm->empty)), full = uni(smem_u32(sm->full));
      const uint32_t lead_full = uni(map_cta(full, 0));
      int s = 0;
      uint32_t phase = 1;  // the first round finds every stage free
      bool ok = gives_up != kGemmCopies;
      int issued = 0;
      for (int u = first; u < p.units && ok; u += step) {
        const PairUnit un = pair_unit(u, p, width);
        const int rr = (int)uni(un.r0 + 128 * rank), cc = (int)uni(un.c0 + (rank ? (gated ? p.C : BN / 2) : 0));
        for (int kb = 0; kb < p.KB; ++kb) {
          ok = bar_wait(empty + 8 * s, phase, limit);
          if (!ok) break;
          const uint32_t bar = lead_full + 8 * s, dr = sr0 + s * G::RBytes, dc = sc0 + s * G::CBytes;
          if (rank == 0) expect_tx(full + 8 * s, 2 * G::Stage, leader);  // both CTAs' bytes
          const int k = kb * kMK;
          if (p.r_mn) {
            pair_load(dr, &p.r, rr, k, bar, leader);
            pair_load(dr + 8192, &p.r, rr + 64, k, bar, leader);
          } else {
            pair_load(dr, &p.r, k, rr, bar, leader);
          }
          if (p.c_mn) {
            pair_load(dc, &p.c, cc, k, bar, leader);
            if (BN == 256) pair_load(dc + 8192, &p.c, cc + 64, k, bar, leader);
          } else {
            pair_load(dc, &p.c, k, cc, bar, leader);
          }
          ++issued;
          if (++s == NS) {
            s = 0;
            phase ^= 1;
          }
        }
      }
      if (!ok) sm->err = 1;
      // Copies in flight land before the pair leaves: the leader waits for both
      // CTAs' (where its MMAs gave up and wait for none); where the leader's
      // copies gave up, the second CTA's land while its wait runs out.
      if (rank == 0)
        for (int i = 0; i < NS; ++i)
          if (i < issued) (void)bar_wait(full + 8 * i, ((issued - 1 - i) / NS) & 1, limit);
    } else if (warp == EW + 1) {
      if (rank == 0) {
        // ---- MMAs, issued by one lane of the leader
        const uint32_t leader = elect_one(), tm = uni(tmem);
        const uint32_t a0 = uni(desc_lo(smem_u32(sr), p.r_mn)), b0 = uni(desc_lo(smem_u32(sc), p.c_mn));
        const uint32_t as = uni(desc_step(p.r_mn)), bs = uni(desc_step(p.c_mn));
        const uint32_t idesc = uni(gemm_idesc(IN, 256, BN, p.r_mn, p.c_mn));
        const uint32_t full = uni(smem_u32(sm->full)), empty = uni(smem_u32(sm->empty));
        const uint32_t acc_full = uni(smem_u32(sm->acc_full)), acc_empty = uni(smem_u32(sm->acc_empty));
        bool ok = gives_up != kGemmMmas;
        int s = 0;
        uint32_t phase = 0, acc = 0, acc_phase = 1;  // the first round finds both accumulators free
        int stages = 0, chunks = 0;
        for (int u = first; u < p.units && ok; u += step) {
          for (int kb = 0, in = 0; kb < p.KB; ++kb, ++in) {
            if (MANY && in == kChunk<OUT>) {
              pair_commit(acc_full + 8 * acc, leader);
              ++chunks, in = 0;
              acc ^= 1;
              acc_phase ^= acc ^ 1;
            }
            if (in == 0) {
              ok = bar_wait(acc_empty + 8 * acc, acc_phase, limit);
              if (!ok) break;
            }
            ok = bar_wait(full + 8 * s, phase, limit);
            if (!ok) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            pair_stage(tm + BN * acc, a0 + (uint32_t)(s * (G::RBytes >> 4)), as, b0 + (uint32_t)(s * (G::CBytes >> 4)), bs, idesc,
                       in > 0, leader);
            pair_commit(empty + 8 * s, leader);
            ++stages;
            if (++s == NS) {
              s = 0;
              phase ^= 1;
            }
          }
          if (!ok) break;
          pair_commit(acc_full + 8 * acc, leader);
          ++chunks;
          acc ^= 1;
          acc_phase ^= acc ^ 1;
        }
        if (!ok) sm->err = 1;
        // MMAs issued, and their arrivals, land before tensor memory is released
        for (int i = 0; i < NS; ++i)
          if (i < stages) (void)bar_wait(empty + 8 * i, ((stages - 1 - i) / NS) & 1, kWaitLimit);
        for (int i = 0; i < 2; ++i)
          if (i < chunks) (void)bar_wait(acc_full + 8 * i, ((chunks - 1 - i) / 2) & 1, kWaitLimit);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    // ---- epilogue: warp w has tensor memory lanes 32 (w % 4) .. + 31, a row
    // of the output each, and half w / 4 of the columns. A wait that runs out
    // ends every later one of its warp and leaves NaN in what it still writes.
    const int l0 = 32 * (warp & 3), half = warp >> 2, cols = width / 2;
    const uint32_t acc_full = smem_u32(sm->acc_full), acc_empty = uni(map_cta(smem_u32(sm->acc_empty), 0));
    float* turn = sm->turn[warp];
    bool ok = gives_up != kGemmSums;
    uint32_t acc = 0, acc_phase = 0;
    for (int u = first; u < p.units; u += step) {
      const uint32_t ta = tmem + ((uint32_t)l0 << 16) + cols * half;
      int unit = u;
      if constexpr (MANY) {
        float sum[BN / 2];
#pragma unroll
        for (int j = 0; j < BN / 2; ++j) sum[j] = 0.f;
#pragma unroll 1
        for (int kb = kChunk<OUT>;; kb += kChunk<OUT>) {
          ok = ok && bar_wait(acc_full + 8 * acc, acc_phase, limit);
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          add_chunk<BN>(sum, ta + BN * acc, gated);
          if (!SPARE && kb >= p.KB) break;
          pair_release(acc_empty + 8 * acc, ok);
          acc ^= 1;
          acc_phase ^= acc ^ 1;
          if (kb >= p.KB) break;
        }
        if (ok) put_sums<BN>(sum, ta + (SPARE ? 2 * BN : BN * acc), gated);
        asm volatile("" : "+r"(unit));  // what follows is worked out behind the sums, not beside them
      }
      const PairUnit un = pair_unit(unit, p, width);
      WarpTile t;
      t.r0 = (int64_t)un.r0 + 128 * rank + l0;
      t.rows = (int)min((int64_t)32, p.R - t.r0);
      t.c0 = un.c0 + cols * half;
      t.cols = cols;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = lane + 32 * j;
        const bool there = p.bias && c < cols && t.c0 + c < p.C;
        t.bias[j] = there ? half_bits(static_cast<const uint16_t*>(p.bias)[t.c0 + c], IN) : 0.f;
        if (j < 2) t.bias_up[j & 1] = there && gated ? half_bits(static_cast<const uint16_t*>(p.bias)[p.C + t.c0 + c], IN) : 0.f;
      }
      if constexpr (!MANY) {
        ok = ok && bar_wait(acc_full + 8 * acc, acc_phase, limit);
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      }
      t.ta = ta + (SPARE ? 2 * BN : BN * acc);
      t.release = SPARE ? 0 : acc_empty + 8 * acc;
      if constexpr (VEC) {
        switch (p.act) {
          case kActNone: finish_straight<IN, OUT, kActNone>(p, t, BN / 2, ok); break;
          case kActRelu: finish_straight<IN, OUT, kActRelu>(p, t, BN / 2, ok); break;
          case kActSilu: finish_straight<IN, OUT, kActSilu>(p, t, BN / 2, ok); break;
          case kActGelu: finish_straight<IN, OUT, kActGelu>(p, t, BN / 2, ok); break;
          default: finish_straight<IN, OUT, kActSwiglu>(p, t, BN / 2, ok);
        }
      } else {
        // 32 rows and columns at a time, turned
#pragma unroll 1
        for (int i = 0; i < cols; i += 32) {
          uint32_t zr[2][16], ur[2][16];
          float z[32], up[32];
          if (ok) {
            tmem_ld_rows(zr[0], t.ta + i);
            tmem_ld_rows(zr[1], t.ta + i + 16);
            if (gated) {
              tmem_ld_rows(ur[0], t.ta + BN / 2 + i);
              tmem_ld_rows(ur[1], t.ta + BN / 2 + i + 16);
              tmem_wait(ur[0]);
              tmem_wait(ur[1]);
            }
            tmem_wait(zr[0]);
            tmem_wait(zr[1]);
          }
          if (i + 32 == cols) pair_release(t.release, ok);
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            z[j] = ok ? __uint_as_float(zr[j >> 4][j & 15]) : __uint_as_float(0x7fffffffu);
            up[j] = ok && gated ? __uint_as_float(ur[j >> 4][j & 15]) : z[j];
          }
          finish_rows<IN, OUT>(p, turn, t.r0, t.rows, t.c0 + i, z, up, t.bias_of(i), t.bias_up_of(i));
        }
      }
      if (!ok) sm->err = 1;
      if (!SPARE) {
        acc ^= 1;
        acc_phase ^= acc ^ 1;
      }
    }
  }
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  cluster_barrier();  // neither leaves, or frees its tensor memory, before the other is done
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (tid == 0 && *(volatile int*)&sm->err && p.status) atomicOr(p.status, DEV_ERR_TIMEOUT);
  if (warp == EW + 2) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(COLS) : "memory");
  product_end(p);
}

// 16-bit rows, `ld` elements apart: a K-major operand has `rows` rows of k
// (boxes of box_rows x 64), an MN-major one k rows of `rows` (64 x 64).
bool map_16(CUtensorMap* out, const GemmOperand& o, int64_t rows, int64_t k, int box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = map_encoder();
  if (!encode) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)(o.mn ? rows : k), (cuuint64_t)(o.mn ? k : rows)};
  const cuuint64_t strides[1] = {(cuuint64_t)(o.ld * 2)};
  const cuuint32_t box[2] = {64, (cuuint32_t)(o.mn ? 64 : box_rows)};
  const cuuint32_t es[2] = {1, 1};
  return encode(out, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(o.p), dims, strides, box, es,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Once a device: the kernel's dynamic shared memory.
cudaError_t configure(const void* kernel, size_t smem, std::atomic<uint64_t>& configured) {
  int device = 0;
  (void)cudaGetDevice(&device);
  if (device < 64 && configured.load() >> device & 1) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess && device < 64) configured.fetch_or(1ull << device);
  return e;
}

// A launch as a programmatic dependent, in clusters of `cluster` blocks.
template <typename P>
cudaError_t launch_cluster(void (*kernel)(P), int64_t grid, int threads, size_t smem, int cluster, cudaStream_t s, const P& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

bool aligned(const void* p, int64_t ld, int bytes, int size) {
  return !(((uintptr_t)p | (uint64_t)(ld * size)) & (uint64_t)(bytes - 1));
}

// Whether every array of the epilogue is aligned to four of its elements.
int vec4(const GemmArgs& a) {
  const int so = dtype_bytes(a.out);
  return a.C % 4 == 0 && aligned(a.y, a.ldy, 4 * so, so) && aligned(a.residual, a.residual ? a.ldr : 0, 4 * so, so) &&
         aligned(a.pre, a.pre ? a.ldp : 0, 8, 2) && aligned(a.bias, 0, 8, 2);
}

// Whether rows are whole groups of 16 columns that start on 32-byte boundaries.
bool vec16(const GemmArgs& a) {
  const int so = dtype_bytes(a.out);
  return a.C % 16 == 0 && aligned(a.y, a.ldy, 32, so) && aligned(a.residual, a.residual ? a.ldr : 0, 32, so) &&
         aligned(a.pre, a.pre ? a.ldp : 0, 32, 2);
}

GemmParams params_of(const GemmArgs& a) {
  GemmParams p{};
  p.bias = a.bias;
  p.residual = a.residual;
  p.pre = a.pre;
  p.y = a.y;
  p.status = a.status;
  p.R = a.R;
  p.ldr = a.ldr;
  p.ldp = a.ldp;
  p.ldy = a.ldy;
  p.C = a.C;
  p.KB = (int)((a.K + kMK - 1) / kMK);
  p.in = a.in;
  p.out = a.out;
  p.act = a.act;
  p.c_mn = a.col.mn;
  p.r_mn = a.row.mn;
  p.give_up = a.give_up;
  p.order = a.order;
  p.vec = vec4(a);
  return p;
}

// Tiles of 128 columns (gated: 64) x NT rows.
int64_t split_units(const GemmArgs& a, int NT) {
  const int width = a.act == kActSwiglu ? 64 : 128;
  return ((a.C + width - 1) / width) * ((a.R + NT - 1) / NT);
}
// In how many parts of k: as many as leave every one two blocks an SM to run on
// and two stages. A product that runs beside another of few tiles leaves it room
// for those (1001 x 1030 x 777: the two gradients 13 us, without 18, one behind the
// other 20).
int split_of(const GemmArgs& a, int NT, int sms) {
  const int64_t units = split_units(a, NT), KB = (a.K + kMK - 1) / kMK, room = 2 * sms - (a.beside < sms ? a.beside : 0);
  int split = 1;
  while (split < 8 && 2 * split * units <= room && 4 * split <= KB) split *= 2;
  return split;
}

template <int NT, int IN, int OUT>
const char* gemm_split(const GemmArgs& a, int split, cudaStream_t s) {
  using G = GemmCfg<NT>;
  static_assert(2 * (gemm_smem_bytes<NT>() + 1024) <= 228 * 1024, "two blocks an SM");
  GemmParams p = params_of(a);
  const bool gated = a.act == kActSwiglu;
  if (!map_16(&p.c, a.col, gated ? 2 * (int64_t)a.C : a.C, a.K, 64) || !map_16(&p.r, a.row, a.R, a.K, NT))
    return "tensor map encoding failed";
  const int64_t units = split_units(a, NT);
  if (units > 0x3fffffff) return "too many tiles";
  p.units_r = (int)((a.R + NT - 1) / NT);
  p.split = split;
  static std::atomic<uint64_t> configured{0};
  cudaError_t e = configure((const void*)gemm_split_kernel<NT, IN, OUT>, gemm_smem_bytes<NT>(), configured);
  if (e == cudaSuccess) e = launch_cluster(gemm_split_kernel<NT, IN, OUT>, units * p.split, G::NTHR, gemm_smem_bytes<NT>(), p.split, s, p);
  return e == cudaSuccess ? nullptr : cudaGetErrorString(e);
}

// Pairs of CTAs that the device runs at once (its SMs come in groups, some of
// odd size), asked for once.
template <int BN, int IN, int OUT, bool VEC, bool MANY>
int pairs_at_once(int sms) {
  static std::atomic<int> known[64];
  int device = 0;
  (void)cudaGetDevice(&device);
  int n = device < 64 ? known[device].load() : 0;
  if (n > 0) return n;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(sms / 2 * 2));
  cfg.blockDim = dim3(PairCfg<BN>::NTHR);
  cfg.dynamicSmemBytes = pair_bytes<BN>();
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, gemm_pair_kernel<BN, IN, OUT, VEC, MANY>, &cfg) != cudaSuccess || n < 1) {
    (void)cudaGetLastError();
    n = sms / 2 > 0 ? sms / 2 : 1;
  }
  if (device < 64) known[device].store(n);
  return n;
}

template <int BN, int IN, int OUT, bool VEC, bool MANY>
const char* gemm_pair_vec(const GemmArgs& a, int sms, cudaStream_t s) {
  GemmParams p = params_of(a);
  const bool gated = a.act == kActSwiglu;
  if (!map_16(&p.c, a.col, gated ? 2 * (int64_t)a.C : a.C, a.K, BN / 2) || !map_16(&p.r, a.row, a.R, a.K, 128))
    return "tensor map encoding failed";
  const int width = gated ? BN / 2 : BN;
  const int64_t units_c = (a.C + width - 1) / width, units_r = (a.R + 255) / 256;
  if (units_c * units_r > 0x3fffffff) return "too many tiles";
  p.units_r = (int)units_r;
  p.units = (int)(units_c * units_r);
  static std::atomic<uint64_t> configured{0};
  cudaError_t e = configure((const void*)gemm_pair_kernel<BN, IN, OUT, VEC, MANY>, pair_bytes<BN>(), configured);
  if (e != cudaSuccess) return cudaGetErrorString(e);
  const int pairs = pairs_at_once<BN, IN, OUT, VEC, MANY>(sms);
  e = launch_cluster(gemm_pair_kernel<BN, IN, OUT, VEC, MANY>, 2 * (int64_t)(p.units < pairs ? p.units : pairs), PairCfg<BN>::NTHR, pair_bytes<BN>(), 2, s, p);
  return e == cudaSuccess ? nullptr : cudaGetErrorString(e);
}

template <int BN, int IN, int OUT>
const char* gemm_pair(const GemmArgs& a, int sms, cudaStream_t s) {
  if (a.K > kMK * kChunk<OUT>)
    return vec16(a) ? gemm_pair_vec<BN, IN, OUT, true, true>(a, sms, s) : gemm_pair_vec<BN, IN, OUT, false, true>(a, sms, s);
  return vec16(a) ? gemm_pair_vec<BN, IN, OUT, true, false>(a, sms, s) : gemm_pair_vec<BN, IN, OUT, false, false>(a, sms, s);
}

// Which form: up to 64 rows (of a K-major operand) the weights stream past
// tiles of 16 or 32 rows. Above, the one that these times, in us and fitted to
// measurements with 152 SMs, say is the fastest: a start and an end, and so
// much a step of 64 of k, times the rounds that the tiles take. Measured (bf16,
// inputs not in L2; tiles of 64 rows in parts of k | pairs of 128 | of 256
// columns): 1024 x 1024 x 1024 8.9 | 7.8 | 10.6; 256 x 2048 x 7168 15.8 | 22.7 |
// 36; 256 x 7168 x 2048 15.6 | 12.5 | 16.0; 1024 x 2048 x 7168 36.0 | 23.9 |
// 37.0; 512 x 7168 x 7168 66 | 42.8 | 38.6; 4096 x 7168 x 1536 124 | 57.6 | 50.9.
// Tiles of 32 rows for 64: 64 x 2048 x 7168 11.1 (one tile of 64 12.3), 64 x 7168
// x 2048 10.8 (11.3).
template <int IN, int OUT>
const char* gemm(const GemmArgs& a, int sms, cudaStream_t s) {
  // boxes of an MN-major operand are 64 wide
  if (a.R <= 16 && !a.row.mn) return gemm_split<16, IN, OUT>(a, split_of(a, 16, sms), s);
  if (a.R <= 64 && !a.row.mn) return gemm_split<32, IN, OUT>(a, split_of(a, 32, sms), s);
  const double KB = (double)((a.K + kMK - 1) / kMK);
  const auto rounds = [](double units, double slots) { return units <= slots ? 1. : (double)(int64_t)((units + slots - 1) / slots); };
  // a pair's epilogue runs under the next unit's products, where those are long
  // enough; one that turns its rows in shared memory takes the products' bandwidth
  // there, and adds to them (3000 x 3001 x 3000 63 us by 128 columns, 48 by 256)
  const bool whole = vec16(a);
  // fp32 sums of many chunks: by 256 columns they go back to the accumulator they
  // came from, and the epilogue holds up the next products; by 128 a chunk's
  // change costs a little (by 128 | 256: 8192 x 7168 x 7168 493 | 479, 4096 x 7168 x
  // 2048 83 | 99; in one chunk 469 | 440 and 80 | 71, with the sums short of bits)
  const bool many = OUT == 2 && KB > kChunk<OUT>;
  const auto pair_time = [&](int bn, double step, double epilogue) {
    const int width = a.act == kActSwiglu ? bn / 2 : bn;
    const double units = (double)((a.C + width - 1) / width) * (double)((a.R + 255) / 256);
    const double both = KB * step + epilogue, one = KB * step > epilogue ? KB * step : epilogue;
    return 4.6 + (rounds(units, sms / 2) - 1) * (whole && !(many && bn == 256) ? one : both) + both;
  };
  const int split = split_of(a, 64, sms);
  const double blocks = (double)split_units(a, 64) * split;
  double part_log = 0;
  for (int q = split; q > 1; q /= 2) ++part_log;
  const double by_64 = 4.2 + 0.5 * part_log + rounds(blocks, 2 * sms) * (2.6 + (KB + split - 1) / split * (blocks > sms ? 0.27 : 0.2));
  const double by_128 = pair_time(128, many ? 0.163 : 0.155, whole ? 2.2 : 4.5), by_256 = pair_time(256, 0.29, whole ? 3.4 : 5.4);
  if (by_64 <= by_128 && by_64 <= by_256) return gemm_split<64, IN, OUT>(a, split, s);
  return by_128 < by_256 ? gemm_pair<128, IN, OUT>(a, sms, s) : gemm_pair<256, IN, OUT>(a, sms, s);
}

}  // namespace
}  // namespace dfm
