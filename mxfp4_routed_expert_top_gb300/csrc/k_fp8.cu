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
#include <cstring>
#include <type_traits>

#include "internal.h"
#include "ops.h"
#include "pipeline.cuh"
#include "rowword.h"
#include "tcgen.cuh"
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

// Two e4m3 codes, nearest even, saturating; NaN gives 0x7f.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// max(a, |b|), NaN if either is.
__device__ __forceinline__ float max_abs_nan(float a, float b) {
  float r;
  asm("{\n\t.reg .f32 t;\n\tabs.f32 t, %2;\n\tmax.NaN.f32 %0, %1, t;\n\t}" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ bool finite_f32(float v) { return fabsf(v) < INFINITY; }

// The scale and the codes of a block whose values lie N a lane in groups of
// 32 >> SHIFT lanes; lanes without a value hold 0. The quotient 448 x / m is
// taken as (0.875 x) / (m / 512), so that neither side overflows, by
// Markstein's division (IBM J. R&D 34, 1990): with y the rounded reciprocal of
// d, q0 = n y, q = q0 + (n - q0 d) y is the rounded quotient. For bf16 and
// fp16, where 0.875 x is exact, ties therefore stay ties, and the codes are
// those of the exact quotient; for fp32 0.875 x is rounded too, and a quotient
// within 2^-23 of its value from the middle of two codes may get either.
// Blocks with NaN or infinities take a branch of their own.
template <int N, int SHIFT>
__device__ __forceinline__ float quantize_block(float (&v)[N], uint32_t (&code)[N / 2]) {
  float m = 0x1p-100f;
#pragma unroll
  for (int n = 0; n < N; ++n) m = max_abs_nan(m, v[n]);
#pragma unroll
  for (int o = 16 >> SHIFT; o; o >>= 1) m = max_abs_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  const bool odd = !finite_f32(m);
  if (__any_sync(0xffffffffu, odd)) {
    if (odd) {  // the same in all of the block's lanes
      m = 0x1p-100f;
#pragma unroll
      for (int n = 0; n < N; ++n) m = fmaxf(m, finite_f32(v[n]) ? fabsf(v[n]) : 0.f);
    }
#pragma unroll
    for (int o = 16 >> SHIFT; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll
    for (int n = 0; n < N; ++n)
      if (!finite_f32(v[n])) v[n] = __uint_as_float(0x7fffffffu);
  }
  const float d = m * 0x1p-9f, y = __frcp_rn(d);
#pragma unroll
  for (int n = 0; n < N; n += 2) {
    float q[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float num = v[n + i] * 0.875f, q0 = num * y;
      q[i] = fmaf(fmaf(-q0, d, num), y, q0);
    }
    code[n / 2] = e4m3x2(q[0], q[1]);
  }
  return __fdiv_rn(m, 448.f);
}

// Rows of whole 32-byte pieces: eight lanes a block, sixteen values a lane.
// HBM bounds it (128 (s + 1) + 4 bytes a block of s-byte values): 65536 x 1536
// bf16 (305 MB) take 50 us, 54 with two blocks in flight a warp (registers
// cost warps an SM), and took 94 when a value cost 24 instructions (index
// division, tests for finiteness, 16 lanes a block).
constexpr int kQThreads = 256, kQUnroll = 1;
template <typename T>
__global__ void __launch_bounds__(kQThreads)
fp8_quantize_kernel(const QuantizeArgs p, uint32_t nb, uint32_t total, const FastDiv by_nb) {
  constexpr int R = sizeof(T) / 2;  // 32-byte loads a lane
  const int l = threadIdx.x & 7, sub = (threadIdx.x >> 3) & 3;
  const uint32_t warps = gridDim.x * (kQThreads / 32);
  const uint32_t warp = blockIdx.x * (kQThreads / 32) + (threadIdx.x >> 5);
  const T* x = static_cast<const T*>(p.x);
  pdl_wait();
  for (uint64_t w0 = warp; 4 * w0 < total; w0 += (uint64_t)warps * kQUnroll) {
    uint32_t raw[kQUnroll][R][8], row[kQUnroll], blk[kQUnroll];
    bool there[kQUnroll], mine[kQUnroll];
#pragma unroll
    for (int u = 0; u < kQUnroll; ++u) {  // lane l: columns 16 l .. 16 l + 15
      const uint64_t g = 4 * (w0 + (uint64_t)u * warps) + sub;
      there[u] = g < total;
      row[u] = by_nb(there[u] ? (uint32_t)g : 0);
      blk[u] = (there[u] ? (uint32_t)g : 0) - row[u] * nb;
      mine[u] = there[u] && (int)(128 * blk[u]) + 16 * l < p.K;
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int n = 0; n < 8; ++n) raw[u][i][n] = 0;
      if (mine[u]) {
        const char* q = reinterpret_cast<const char*>(x + (int64_t)row[u] * p.ldx + 128 * blk[u] + 16 * l);
#pragma unroll
        for (int i = 0; i < R; ++i)
          asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                       : "=r"(raw[u][i][0]), "=r"(raw[u][i][1]), "=r"(raw[u][i][2]), "=r"(raw[u][i][3]),
                         "=r"(raw[u][i][4]), "=r"(raw[u][i][5]), "=r"(raw[u][i][6]), "=r"(raw[u][i][7])
                       : "l"(q + 32 * i));
      }
    }
#pragma unroll
    for (int u = 0; u < kQUnroll; ++u) {
      T e[16];
      memcpy(e, raw[u], sizeof e);
      float v[16];
#pragma unroll
      for (int n = 0; n < 16; ++n) v[n] = to_f32<T>(e[n]);
      uint32_t code[8];
      const float scale = quantize_block<16, 2>(v, code);
      if (mine[u])
        *reinterpret_cast<uint4*>(p.codes + (int64_t)row[u] * p.ldc + 128 * blk[u] + 16 * l) =
            make_uint4(code[0] | code[1] << 16, code[2] | code[3] << 16, code[4] | code[5] << 16,
                       code[6] | code[7] << 16);
      if (there[u] && l == 0) p.scales[(int64_t)row[u] * p.lds + blk[u]] = scale;
    }
  }
}

// Any other rows: eight lanes a block, in words of four values that are
// aligned in memory (word w holds the block's values 4 w - m .. 4 w - m + 3, m
// what lies between the word boundary and the block), so that a block has 33
// of them and a lane up to five; words without a value of the block are not
// read. Where codes lie like x (the same distance of rows modulo 4) their
// words are aligned too. 14001 x 7167 bf16 (304 MB, 45 us at the copy rate): 89 us, issue slots 70%
// busy; value by value 109.
template <typename T, bool ENDS>
__device__ __forceinline__ void quantize_odd(const QuantizeArgs& p, uint32_t nb, const FastDiv& by_nb, uint32_t g,
                                             bool there) {
  constexpr int R = 5;
  const int l = threadIdx.x & 7;
  const T* x = static_cast<const T*>(p.x);
  const uint32_t row = by_nb(there ? g : 0), blk = (there ? g : 0) - row * nb;
  const int len = there ? min(128, p.K - (int)(128 * blk)) : 0;
  const T* src = x + (int64_t)row * p.ldx + 128 * blk;
  const int first = 4 * l - ((int)((uintptr_t)src / sizeof(T)) & 3);
  Four<T> word[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int e = first + 32 * r;  // the word's first value
    if (e < len && e + 3 >= 0) {
      if (ENDS) word[r] = array_four<T>(ArrayOf<T>{x}, src - x + e, (p.M - 1) * p.ldx + p.K);
      else word[r] = *reinterpret_cast<const Four<T>*>(src + e);
    }
  }
  float v[4 * R];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[4 * r + i] = (unsigned)(first + 32 * r + i) < (unsigned)len ? to_f32<T>(word[r].v[i]) : 0.f;
  uint32_t code[2 * R];
  const float scale = quantize_block<4 * R, 2>(v, code);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int e = first + 32 * r;
    uint8_t* dst = p.codes + (int64_t)row * p.ldc + 128 * blk + e;
    const uint32_t four = code[2 * r] | code[2 * r + 1] << 16;
    if (e >= 0 && e + 3 < len && ((uintptr_t)dst & 3) == 0) {
      *reinterpret_cast<uint32_t*>(dst) = four;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if ((unsigned)(e + i) < (unsigned)len) dst[i] = (uint8_t)(four >> (8 * i));
    }
  }
  if (len > 0 && l == 0) p.scales[(int64_t)row * p.lds + blk] = scale;
}

// Words may reach (at most three values) over an end of x in the first block,
// the last, and the one before it, behind which K may have one value: CTA 0
// takes those, and reads no such word. (A test in every block cost 3%.) Where
// rows are nearer than three values, ALL_ENDS, every block is read like that.
template <typename T, bool ALL_ENDS>
__global__ void __launch_bounds__(kQThreads)
fp8_quantize_odd_kernel(const QuantizeArgs p, uint32_t nb, uint32_t total, const FastDiv by_nb) {
  const int sub = (threadIdx.x >> 3) & 3, ends = ALL_ENDS ? 0 : 1;
  const uint32_t near_end = total < 3 ? 1 : total - 2;
  pdl_wait();
  if (!ALL_ENDS && blockIdx.x == 0) {
    if (threadIdx.x < 32) {
      const uint32_t g = sub ? near_end + sub - 1 : 0;
      quantize_odd<T, true>(p, nb, by_nb, g, g < total);
    }
    return;
  }
  const uint32_t warps = (gridDim.x - ends) * (kQThreads / 32);
  const uint32_t warp = (blockIdx.x - ends) * (kQThreads / 32) + (threadIdx.x >> 5);
  for (uint64_t w0 = warp; 4 * w0 < total; w0 += warps) {
    const uint64_t g = 4 * w0 + sub;
    quantize_odd<T, ALL_ENDS>(p, nb, by_nb, (uint32_t)g, ALL_ENDS ? g < total : g >= 1 && g < near_end);
  }
}

template <typename T>
cudaError_t quantize_t(const QuantizeArgs& p, int sms, cudaStream_t s) {
  const uint32_t nb = (uint32_t)((p.K + 127) / 128);
  const uint64_t total = (uint64_t)p.M * nb;
  const uint64_t blocks = (total + 4 * (kQThreads / 32) - 1) / (4 * (kQThreads / 32));
  const uint64_t most = (uint64_t)sms * 24;
  const unsigned grid = (unsigned)(blocks < most ? blocks : most);
  const bool vec = !(((uintptr_t)p.x | (uint64_t)(p.ldx * (int64_t)sizeof(T))) & 31) &&
                   !(((uintptr_t)p.codes | (uint64_t)p.ldc) & 15) && p.K % 16 == 0;
  const FastDiv by_nb(nb);
  if (vec)
    return launch_after_previous(fp8_quantize_kernel<T>, dim3(grid), dim3(kQThreads), 0, s, p, nb, (uint32_t)total, by_nb);
  return p.ldx < 3 ? launch_after_previous(fp8_quantize_odd_kernel<T, true>, dim3(grid), dim3(kQThreads), 0, s, p, nb,
                                           (uint32_t)total, by_nb)
                   : launch_after_previous(fp8_quantize_odd_kernel<T, false>, dim3(grid + 1), dim3(kQThreads), 0, s, p,
                                           nb, (uint32_t)total, by_nb);
}

// ---- product --------------------------------------------------------------------
// A unit is (a tile of NT rows of x of one group) x (NN columns n), K in
// blocks of 128, the blocks of the scales.
//
// Roles of a CTA: EW epilogue warps and four more: copies, MMAs, and two that
// fetch scales. The copy warp fills a ring of stages (in the 128-byte
// swizzle), the MMA warp issues four K = 32 steps a block into the next of AS
// accumulators, and the epilogue warps add the block, times its scales, to
// their registers.
//
// The scales decide the orientation. With more than 32 rows a group the rows of
// x are the 128-row operand (XA): lane = row of x, and a thread has one
// scale for its whole part of a block. With lane = n every accumulator column
// has its own, and fetching those from shared memory took its bandwidth from
// the MMA's operands. Short tiles (NT = 16, 32) keep the weights as the
// 128-row operand: they stream, and 128 rows of x would be mostly empty.
// Measured with 16 experts of 1536 x 7168 when the forms were chosen: 12 rows
// each 35.4 us (NT = 16) against 37.8 (NT = 128); 24 rows 35.9 (32) and 37.8; 48
// rows 46.8 (32) and 38.7; 80 rows 46.7 and 39.8.
// The host chooses by the mean, rows / min(rows, groups): it does not know the
// groups. Uneven ones are right but pay for it: 4096 rows of 1536 x 7168 take
// 51 us in 8 groups of 8, and 166 in 8 of 256 (mean 16: tiles of 16 rows, each
// of which fetches its expert's weights through L2); 1024 rows in one group 25
// us, in one of 64 groups 48.
//
// What bounds it. Long groups: a block of 128 x 256 x 128 takes 773 cycles, of
// which its MMAs take 512. From clock stamps of one CTA: an epilogue warp takes
// 356 from seeing a block's accumulator to releasing it, and then about 390
// until it looks at the next (the rest of its FMAs, the loop, the barrier),
// which is the period. An accumulator's turn is two periods: 718 from the MMAs'
// issue until the first warp sees it, up to 290 more until the last one does, 356,
// about 135 back to the MMA warp and 95 to issue. Copies are not part of it
// (773 without any). So every instruction between two blocks counts (toggled
// indexes in place of computed ones and no code for failures inside the loop:
// 302 to 285 us on 8192 x 7168 x 7168). Not faster, against
// what the kernel took when each was tried: a pair of CTAs on 256 x 256
// (cta_group::2: 306 for 294), sixteen epilogue warps (325 for 291), packed
// fp32 FMAs (308 for 308), two accumulators of 128 columns in place of one (343
// for 299), two MMA warps (298 for 300), longer tensor memory loads (324 for
// 291), the next block's scale or barrier read early (292 for 285). All of
// these are runs of 3 to 10 ms; longer ones lower the clock: 2048 x 16 rows of
// 32 experts, 1536 x 7168, take 270 to 287 us in a short run (2.6 PFLOP/s) and
// 326 among other work (2.2); 8192 x 7168 x 7168 285 to 325. Short groups stream
// weights at 85% of the copy rate (16 experts of 1536 x 7168, one token: 31 us).
//
// split > 1 (NT <= 32): a cluster of that many CTAs shares a unit, each takes
// a part of K, and the sums meet in distributed shared memory, in the order
// of the parts.
constexpr int kFK = 128;          // K a block, and the columns n of a block of w's scales
constexpr int kFABytes = 128 * kFK;
constexpr int kFBatch = 8;        // blocks whose scales are fetched together

template <int NT>
struct Fp8Cfg {
  static constexpr bool XA = NT >= 128;                  // rows of x are the 128-row operand
  static constexpr int NN = XA ? 256 : 128;              // columns n a unit
  static constexpr int DN = XA ? NN : NT;                // accumulator columns
  static constexpr int EW = XA ? 8 : 4;                  // epilogue warps
  static constexpr int CW = 4 * DN / EW;                 // accumulator columns a warp holds
  static constexpr int NTHR = (EW + 4) * 32;
  static constexpr int BRows = DN;                       // rows of the second operand
  static constexpr int BBytes = BRows * kFK;
  static constexpr int NS = XA ? 4 : 5;                  // stages
  static constexpr int AS = XA ? 2 : 4;                  // accumulators
  static constexpr uint32_t Cols = DN * AS;
  static constexpr int Scales = XA ? 128 : NT;           // a block's scales of x
  static constexpr int CtasPerSm = XA ? 1 : 2;
};

struct Fp8Params {
  CUtensorMap w, x;
  const float *xs, *ws;
  const int32_t* offs;
  void* y;
  uint32_t* status;
  int64_t M, ldxs, ldy;
  int G, N, K, KB, NB, units_n, split, vec;
  int give_up;  // test hook: the role of block 0 (Role) that gives up before its first wait
};

enum Role { kNone = 0, kCopies, kMmas, kScales, kSums };

template <int NT>
struct Fp8Smem {
  using C = Fp8Cfg<NT>;
  uint8_t out[C::EW][C::XA ? 2048 : 512];   // what a warp rearranges of y
  float sc[2][kFBatch][C::Scales + 4];      // scales of two batches of blocks: xs (times ws unless XA or wide)
  float scw[2][kFBatch][2];                 // ws of the unit's blocks of n
  int wide[2][2];                           // a scale warp's rows have a product xs ws out of range
  uint64_t full[C::NS], empty[C::NS];
  uint64_t acc_full[C::AS], acc_empty[C::AS];
  uint64_t sc_full[2], sc_empty[2];
  int warp_sums[32];
  uint32_t tmem;
  int err;
};

template <int NT>
constexpr size_t fp8_smem_bytes(int G) {
  using C = Fp8Cfg<NT>;
  return (size_t)C::NS * (kFABytes + C::BBytes) + sizeof(Fp8Smem<NT>) + 2 * (size_t)(G + 1) * sizeof(int);
}

// e4m3 x e4m3, fp32 D; ta, tb: A is M-major, B N-major in shared memory.
__device__ __forceinline__ uint32_t idesc_e4m3(int M, int N, int ta, int tb) {
  return (1u << 4) | ((uint32_t)ta << 15) | ((uint32_t)tb << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Four MMA steps of 32 along K into one accumulator, issued by the lane with
// `leader`; KA and KB say how far a step moves the operands' descriptors,
// whose low words are given. The whole warp runs this: the operands are then
// the same in every lane as far as the compiler is concerned, and sit in
// uniform registers (issued from a branch of one lane, a block's MMAs and
// waits took 1000 cycles, of which the MMAs need 512).
template <int KA, int KB>
__device__ __forceinline__ void mma_block(uint32_t d, uint32_t ad, uint32_t bd, uint32_t idesc, uint32_t leader) {
  // the high word of umma::smem_desc_sw128: atoms of 1024 bytes, version 1, 128-byte swizzle
  constexpr uint32_t hi = (1024u >> 4) | 1u << 14 | 2u << 29;
  asm volatile(
      "{\n\t.reg .pred e, p0, pt;\n\t.reg .b32 l;\n\t.reg .b64 a0, a1, a2, a3, b0, b1, b2, b3;\n\t"
      "setp.ne.u32 e, %6, 0;\n\tsetp.ne.u32 p0, %3, %3;\n\tsetp.eq.u32 pt, %3, %3;\n\t"
      "mov.b64 a0, {%1, %7};\n\tmov.b64 b0, {%2, %7};\n\t"
      "add.u32 l, %1, %4;\n\tmov.b64 a1, {l, %7};\n\t"
      "add.u32 l, l, %4;\n\tmov.b64 a2, {l, %7};\n\t"
      "add.u32 l, l, %4;\n\tmov.b64 a3, {l, %7};\n\t"
      "add.u32 l, %2, %5;\n\tmov.b64 b1, {l, %7};\n\t"
      "add.u32 l, l, %5;\n\tmov.b64 b2, {l, %7};\n\t"
      "add.u32 l, l, %5;\n\tmov.b64 b3, {l, %7};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a0, b0, %3, p0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, pt;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b2, %3, pt;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b3, %3, pt;\n\t}" ::"r"(d),
      "r"(ad), "r"(bd), "r"(idesc), "n"(KA), "n"(KB), "r"(leader), "n"(hi)
      : "memory");
}
// 16 lanes x 8 N columns of tensor memory: thread l gets, for each group of 8
// columns, columns 2 (l % 4) and the next of lane l / 4 (first two values)
// and of lane l / 4 + 8. The wait names the registers, so that no use of them
// moves above it.
__device__ __forceinline__ void tmem_ld(uint32_t (&r)[16], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_ld(uint32_t (&r)[8], uint32_t addr) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(addr));
}
__device__ __forceinline__ void put_y(float* y, float v) { *y = v; }
__device__ __forceinline__ void put_y(__nv_bfloat16* y, float v) { *y = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put_y(__half* y, float v) { *y = __float2half_rn(v); }

// 32 bytes of a row: 8 fp32 values or 16 of 16 bits (32-byte aligned).
template <typename Y>
__device__ __forceinline__ void store_sector(Y* y, const float* v) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    w[i] = sizeof(Y) == 4 ? __float_as_uint(v[i]) : pack16<Y>(v[2 * i % 16], v[(2 * i + 1) % 16]);
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(y), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// What a unit is: `rows` rows of x from `row0`, all of group g, times columns
// from n0.
struct Fp8Unit {
  int g, rows, n0;
  int64_t row0;
};

// tiles[g]: row tiles of the groups before g; offs[g]: first row of group g.
template <int NT>
__device__ __forceinline__ Fp8Unit fp8_unit(int u, int units_n, int G, const int* tiles, const int* offs) {
  const int tile = u / units_n;
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
  r.n0 = (u - tile * units_n) * Fp8Cfg<NT>::NN;
  return r;
}

// Lane = n: where the scale of row c of a tile stands: a thread's rows of two groups of
// eight (2 q, 2 q + 1 of each) side by side, one 16-byte load.
__device__ __forceinline__ int scale_slot(int c) {
  return (c & ~15) | ((c & 6) << 1) | ((c & 8) >> 2) | (c & 1);
}

// Scales of any size: xs ws may leave fp32's normal range where xs ws P does
// not (rows of zeros have scales of 2^-109). The scale warps look at the
// products of each batch of blocks; one that holds such a product (wide) is
// added with two factors a value, P times the first times the second, at 1.3
// times the usual time (2048 x 16 rows of 32 experts, 1536 x 7168, every
// product wide: 371 us, 272 otherwise); rows whose products are normal get
// the same bits in either.
//
// The two factors: P times the first, times the second, has neither
// overflow nor underflow on the way that the result has not. 1 and xs ws,
// unless that product is not a normal number: then the larger scale first
// where it is too small (the smaller is at least 2^-149, so the larger is below
// 2^23, and |P| below 2^25), the smaller first where it is too large.
__device__ __forceinline__ bool out_of_range(float xs, float ws) {
  const float s = fabsf(xs * ws);
  return !(s >= 0x1p-126f && s < INFINITY) && xs != 0.f && ws != 0.f;
}
// The same for several xs, of which the smallest but zero (its bits less one;
// all ones where there is none) and the largest magnitude are given.
__device__ __forceinline__ bool out_of_range(uint32_t least, float most, float ws) {
  return least != 0xffffffffu && (out_of_range(__uint_as_float(least + 1), ws) || out_of_range(most, ws));
}
__device__ __forceinline__ float2 scale_factors(float xs, float ws) {
  if (!out_of_range(xs, ws)) return make_float2(1.f, xs * ws);
  return (fabsf(xs * ws) < 1.f) == (fabsf(xs) > fabsf(ws)) ? make_float2(xs, ws) : make_float2(ws, xs);
}

template <int NT, bool TRANS, typename Y>
__global__ void __launch_bounds__(Fp8Cfg<NT>::NTHR, Fp8Cfg<NT>::CtasPerSm)
fp8_matmul_kernel(const __grid_constant__ Fp8Params p) {
  using C = Fp8Cfg<NT>;
  constexpr int EW = C::EW, NS = C::NS, AS = C::AS, CW = C::CW;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sa = smem;
  uint8_t* sb = smem + NS * kFABytes;
  Fp8Smem<NT>* sm = reinterpret_cast<Fp8Smem<NT>*>(sb + NS * C::BBytes);
  int* tiles = reinterpret_cast<int*>(sm + 1);
  int* offs = tiles + p.G + 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 32) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&p.w) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&p.x) : "memory");
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
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm->sc_full[i], 2);
      mbar_init(&sm->sc_empty[i], EW);
    }
    sm->err = 0;
    fence_barrier_init();
  }
  pdl_wait();  // the kernel before this one is complete
  // Tensor memory only from here on: a kernel that lets its dependents start
  // and takes its own later would wait for this block, which waits for it.
  if (warp == EW + 2) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm->tmem)), "r"(C::Cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // the groups' first rows, kept inside [0, M] whatever the caller's array
  // holds, and their tiles; groups that are not in order have no units
  bool bad = false;
  const int M = (int)p.M;
  for (int g = tid; g <= p.G; g += C::NTHR)
    offs[g] = p.offs ? min(max(p.offs[g], 0), M) : (g ? M : 0);
  __syncthreads();
  {
    int base = 0;
    for (int g0 = 0; g0 < p.G; g0 += C::NTHR) {
      const int g = g0 + tid;
      const int n = g < p.G ? (max(0, offs[g + 1] - offs[g]) + NT - 1) / NT : 0;
      bad = bad || (g < p.G && offs[g + 1] < offs[g]);
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
      for (int w = 0; w < C::NTHR / 32; ++w) {
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
  bad = __syncthreads_or(bad) != 0;
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&sm->tmem);
  if (bad && blockIdx.x == 0 && tid == 0 && p.status) atomicOr(p.status, DEV_ERR_RANGE);
  const int units = bad ? 0 : tiles[p.G] * p.units_n;
  const int part = blockIdx.x % p.split;
  const int first = blockIdx.x / p.split, step = gridDim.x / p.split;
  const int kb0 = (int)((int64_t)p.KB * part / p.split);
  const int kb1 = (int)((int64_t)p.KB * (part + 1) / p.split);
  // A wait that runs out sets err; every role then stops at its next wait.
  const int gives_up = blockIdx.x == 0 ? p.give_up : kNone;
  const uint32_t limit = gives_up ? kTestWaitLimit : kWaitLimit;

  if (warp >= EW) {
    if (C::XA) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == EW) {
      // ---- copies, issued by one lane
      const uint32_t leader = elect_one(), a0 = uni(smem_u32(sa)), b0 = uni(smem_u32(sb));
      const uint32_t empty = uni(smem_u32(sm->empty)), full = uni(smem_u32(sm->full));
      int s = 0;
      uint32_t phase = 1;  // the first round finds every stage free
      bool ok = gives_up != kCopies;
      for (int u = first; u < units && ok; u += step) {
        const Fp8Unit un = fp8_unit<NT>(u, p.units_n, p.G, tiles, offs);
        const int n0 = (int)uni(un.n0), r0 = (int)uni((uint32_t)un.row0);
        const int g = (int)uni(un.g);
        for (int kb = kb0; kb < kb1; ++kb) {
          ok = bar_wait(empty + 8 * s, phase, limit);
          if (!ok) break;
          const uint32_t bar = full + 8 * s, da = a0 + s * kFABytes, db = b0 + s * C::BBytes;
          expect_tx(bar, kFABytes + C::BBytes, leader);
          // the weights' box is 128 x 128 where it is N-major (TRANS)
          const uint32_t dw = C::XA ? db : da;
          if (TRANS) {
#pragma unroll
            for (int n = 0; n < (C::XA ? C::BRows : 128); n += 128)
              tma_load_3d(dw + n * kFK, &p.w, n0 + n, kb * kFK, g, bar, leader);
          } else {
            tma_load_3d(dw, &p.w, kb * kFK, n0, g, bar, leader);
          }
          tma_load_2d(C::XA ? da : db, &p.x, kb * kFK, r0, bar, leader);
          if (++s == NS) {
            s = 0;
            phase ^= 1;
          }
        }
      }
      if (!ok) sm->err = 1;
      // copies in flight land before the block leaves, also where the MMA warp
      // gave up and waits for none of them: of a stage's last round, or
      // (waiting for nothing) of the round before
      for (int i = 0; i < NS; ++i) (void)bar_wait(full + 8 * i, i < s ? phase ^ 1 : phase, kWaitLimit);
    } else if (warp == EW + 1) {
      // ---- MMAs, issued by one lane
      // transposed weights are M- or N-major: a K step of 32 is 32 rows of
      // 128 bytes, against 32 bytes along a K-major row. An N-major operand
      // is one box of 128 wide: 256 columns n in one CTA are two MMAs.
      constexpr int KA = TRANS && !C::XA ? 32 * 128 / 16 : 2, KB = TRANS && C::XA ? 32 * 128 / 16 : 2;
      constexpr int PARTS = TRANS && C::XA ? C::BRows / 128 : 1;
      const uint32_t idesc = idesc_e4m3(128, C::DN / PARTS, TRANS && !C::XA, TRANS && C::XA);
      const uint32_t leader = elect_one(), tm = uni(tmem);
      const uint32_t a0 = uni((uint32_t)umma::smem_desc_sw128(smem_u32(sa)));
      const uint32_t b0 = uni((uint32_t)umma::smem_desc_sw128(smem_u32(sb)));
      const uint32_t full = uni(smem_u32(sm->full)), empty = uni(smem_u32(sm->empty));
      const uint32_t acc_full = uni(smem_u32(sm->acc_full)), acc_empty = uni(smem_u32(sm->acc_empty));
      bool ok = gives_up != kMmas;
      const int total = ok && first < units ? ((units - first + step - 1) / step) * (kb1 - kb0) : 0;
      int s = 0, as = 0;
      uint32_t phase = 0, acc_phase = 1;  // the first round finds every accumulator free
      int it = 0;
      for (; it < total; ++it) {
        ok = bar_wait(full + 8 * s, phase, limit) && bar_wait(acc_empty + 8 * as, acc_phase, limit);
        if (!ok) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
        for (int h = 0; h < PARTS; ++h)
          mma_block<KA, KB>(tm + (uint32_t)(as * C::DN + h * (C::DN / PARTS)), a0 + (uint32_t)(s * (kFABytes >> 4)),
                                b0 + (uint32_t)((s * C::BBytes + h * (128 * kFK)) >> 4), idesc, leader);
        mma_commit(acc_full + 8 * as, leader);
        mma_commit(empty + 8 * s, leader);
        if (++s == NS) {
          s = 0;
          phase ^= 1;
        }
        if (++as == AS) {
          as = 0;
          acc_phase ^= 1;
        }
      }
      if (!ok) sm->err = 1;
      // the MMAs issued, and their arrivals, must land before the tensor
      // memory is released and the block leaves
      if (it > 0) {
        (void)bar_wait(empty + 8 * (s ? s - 1 : NS - 1), s ? phase : phase ^ 1, kWaitLimit);
        (void)bar_wait(acc_full + 8 * (as ? as - 1 : AS - 1), as ? acc_phase ^ 1 : acc_phase, kWaitLimit);
      }
    } else {
      // ---- scales: xs ws of kFBatch blocks at a time, one value a thread
      // and step: block i % kFBatch, row i / kFBatch
      const int st = tid - (EW + 2) * 32;
      int batch = 0;
      bool ok = gives_up != kScales;
      if (!ok) sm->err = 1;
      for (int u = first; u < units && ok; u += step) {
        const Fp8Unit un = fp8_unit<NT>(u, p.units_n, p.G, tiles, offs);
        const int nb = un.n0 / kFK;
        const float* ws = p.ws + (int64_t)un.g * p.NB * p.KB;
        for (int kb = kb0; kb < kb1; kb += kFBatch, ++batch) {
          const int buf = batch & 1;
          ok = batch < 2 || mbar_wait(&sm->sc_empty[buf], ((batch >> 1) - 1) & 1, limit);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            sm->err = 1;
            break;
          }
          const int b = kb + (st & (kFBatch - 1));
          float wv[2] = {0.f, 0.f};  // XA: of the two blocks of n
#pragma unroll
          for (int h = 0; h < (C::XA ? 2 : 1); ++h)
            if (b < kb1 && nb + h < p.NB)
              wv[h] = TRANS ? ws[(int64_t)b * p.NB + nb + h] : ws[(int64_t)(nb + h) * p.KB + b];
          if (st < kFBatch) {
            sm->scw[buf][st][0] = wv[0];
            sm->scw[buf][st][1] = wv[1];
          }
          const float* xs = p.xs + un.row0 * p.ldxs + b;
          bool wide = false;
          uint32_t least = 0xffffffffu;  // the smallest |xs| but zero, its bits less one, and the largest
          float most = 0.f;
          constexpr int PER = (C::XA ? 128 : NT) * kFBatch / 64, U = PER < 8 ? PER : 8;
          for (int i0 = 0; i0 < PER; i0 += U) {
            float v[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
              const int r = st / kFBatch + 64 / kFBatch * (i0 + i);
              v[i] = b < kb1 && r < un.rows ? xs[r * p.ldxs] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
              least = min(least, __float_as_uint(fabsf(v[i])) - 1);  // zero: the largest
              most = fmaxf(most, fabsf(v[i]));
            }
            static_assert(C::XA || PER == U, "all of a warp's rows are known before the first is stored");
            if (!C::XA) wide = __any_sync(0xffffffffu, out_of_range(least, most, wv[0]));
            float* sc = sm->sc[buf][st & (kFBatch - 1)];
#pragma unroll
            for (int i = 0; i < U; ++i) {
              const int r = st / kFBatch + 64 / kFBatch * (i0 + i);
              sc[C::XA ? r : scale_slot(r)] = C::XA || wide ? v[i] : v[i] * wv[0];
            }
          }
          if (C::XA) wide = __any_sync(0xffffffffu, out_of_range(least, most, wv[0]) || out_of_range(least, most, wv[1]));
          if (lane == 0) sm->wide[buf][st >> 5] = wide;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm->sc_full[buf]);
        }
      }
    }
  } else {
    // ---- sums. A wait that runs out ends every later wait of its warp and
    // leaves NaN in the rows it still writes.
    int it = 0, batch = 0;
    bool ok = gives_up != kSums;
    if constexpr (C::XA) {
      // warp w: tensor memory lanes 32 (w % 4) .. + 31, a row of x each, and
      // columns 128 (w / 4) .. + 127, one block of n
      asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
      static_assert(128 % CW == 0, "a warp's columns lie in one block of w's scales");
      const int c0 = (warp >> 2) * CW, l0 = 32 * (warp & 3);
      const uint32_t tbase = tmem + ((uint32_t)l0 << 16) + (uint32_t)c0;
      static_assert(AS == 2, "the accumulator alternates");
      const uint32_t sc_full = smem_u32(sm->sc_full), sc_empty = smem_u32(sm->sc_empty);
      const uint32_t acc_full = smem_u32(sm->acc_full), acc_empty = smem_u32(sm->acc_empty), leader = lane == 0;
      uint32_t buf = 0, sc_phase = 0, as = 0, acc_phase = 0;
      for (int u = first; u < units; u += step) {
        const Fp8Unit un = fp8_unit<NT>(u, p.units_n, p.G, tiles, offs);
        float acc[CW];
#pragma unroll
        for (int i = 0; i < CW; ++i) acc[i] = 0.f;
        for (int kb = kb0; kb < kb1 && ok; kb += kFBatch) {
          ok = bar_wait(sc_full + 8 * buf, sc_phase, limit);
          if (!ok) break;
          const int blocks = min(kFBatch, kb1 - kb);
          const float* sc = &sm->sc[buf][0][l0 + lane];
          const float* scw = &sm->scw[buf][0][c0 >> 7];
          const auto add_blocks = [&](auto is_wide) {
            constexpr bool WIDE = decltype(is_wide)::value;
#pragma unroll 1
            for (int b = 0; b < blocks; ++b) {
              const float xs = sc[b * (C::Scales + 4)], ws = scw[2 * b];
              const float2 f = WIDE ? scale_factors(xs, ws) : make_float2(1.f, xs * ws);
              ok = bar_wait(acc_full + 8 * as, acc_phase, limit);
              if (!ok) break;
              asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
              const uint32_t ta = tbase + (uint32_t)(as * C::DN);
              constexpr int L = 16;           // columns a load
              constexpr int A = WIDE ? 0 : 1;  // the next load runs while this one is added (WIDE: no registers left)
              uint32_t r[1 + A][L];
              tmem_ld_rows(r[0], ta);
#pragma unroll
              for (int i = 0; i < CW / L; ++i) {
                if (WIDE && i) tmem_ld_rows(r[0], ta + L * i);
                tmem_wait(r[i & A]);
                if (i + 1 < CW / L) {
                  if (!WIDE) tmem_ld_rows(r[(i + 1) & A], ta + L * (i + 1));
                } else {
                  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                  arrive_if(acc_empty + 8 * as, leader);
                }
#pragma unroll
                for (int c = 0; c < L; ++c) {
                  const float v = __uint_as_float(r[i & A][c]);
                  acc[L * i + c] = fmaf(WIDE ? v * f.x : v, f.y, acc[L * i + c]);
                }
              }
              as ^= 1;
              acc_phase ^= as ^ 1;
            }
          };
          const int2 wide = *reinterpret_cast<const int2*>(sm->wide[buf]);
          if (wide.x | wide.y) add_blocks(std::true_type());
          else add_blocks(std::false_type());
          __syncwarp();
          arrive_if(sc_empty + 8 * buf, leader);
          buf ^= 1;
          sc_phase ^= buf ^ 1;
        }
        if (!ok) {
          sm->err = 1;
#pragma unroll
          for (int i = 0; i < CW; ++i) acc[i] = fmaf(acc[i], __uint_as_float(0x7fffffffu), acc[i]);  // NaN (moves: spills)
        }
        const int n0 = un.n0 + c0, row = l0 + lane;
        Y* y = static_cast<Y*>(p.y) + (un.row0 + row) * p.ldy + n0;
        if (p.vec && n0 + CW <= p.N) {
          // a lane's own row, 32 bytes (a sector) a store
          if (row < un.rows) {
#pragma unroll
            for (int i = 0; i < CW; i += 32 / (int)sizeof(Y)) store_sector(y + i, &acc[i]);
          }
        } else {
          // 64 bytes of each row at a time through shared memory, so that a
          // store covers one or two rows (32 rows each, value by value, it
          // took 54 us where this takes 25: 3006 x 2050 x 1111, fp32);
          // piece q of row r stands at q ^ (r / 2) % 4
          uint8_t* stage = sm->out[warp];
          const int rows = un.rows - l0;
          Y* base = static_cast<Y*>(p.y) + (un.row0 + l0) * p.ldy + n0;
          constexpr int CC = 64 / (int)sizeof(Y), RR = 32 / CC > 0 ? 32 / CC : 1;  // columns a piece, rows a store
#pragma unroll
          for (int i = 0; i < CW; i += CC) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = sizeof(Y) == 4 ? __float_as_uint(acc[i + (4 * q + e) % CC])
                                      : pack16<Y>(acc[i + (8 * q + 2 * e) % CC], acc[i + (8 * q + 2 * e + 1) % CC]);
              *reinterpret_cast<uint4*>(stage + 64 * lane + 16 * (q ^ ((lane >> 1) & 3))) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            __syncwarp();
            const int c = lane % CC, at = c * (int)sizeof(Y);
            if (n0 + i + c < p.N) {
#pragma unroll 8
              for (int r = lane / CC; r < min(rows, 32); r += RR)
                base[r * p.ldy + i + c] = *reinterpret_cast<const Y*>(stage + 64 * r + 16 * ((at >> 4) ^ ((r >> 1) & 3)) + (at & 15));
            }
            __syncwarp();
          }
        }
      }
    } else {
      // warp w: lanes (columns n) 32 (w % 4) .. + 31, all columns (rows of x)
      constexpr int LDN = CW >= 32 ? 4 : 2, LC = 8 * LDN, CH = CW / LC;  // CH loads of LC columns a half
      const int l0 = 32 * warp;
      const uint32_t tbase = tmem + ((uint32_t)l0 << 16);
      const int nq = lane >> 2, tq = 2 * (lane & 3);
      uint8_t* stage = sm->out[warp];
      for (int u = first; u < units; u += step) {
        const Fp8Unit un = fp8_unit<NT>(u, p.units_n, p.G, tiles, offs);
        // acc[c / 8][h][j][i]: column 8 (c / 8) + tq + i of lane 16 h + 8 j + nq
        float acc[CW / 8][2][2][2];
#pragma unroll
        for (int i = 0; i < CW / 2; ++i) acc[i >> 2][(i >> 1) & 1][i & 1][0] = acc[i >> 2][(i >> 1) & 1][i & 1][1] = 0.f;
        for (int kb = kb0; kb < kb1; kb += kFBatch, ++batch) {
          const int buf = batch & 1;
          ok = ok && bar_wait(smem_u32(&sm->sc_full[buf]), (batch >> 1) & 1, limit);
          const int blocks = min(kFBatch, kb1 - kb);
          // a thread's rows are all of one scale warp
          const bool raw = sm->wide[buf][tq >> 2], wide = sm->wide[buf][0] | sm->wide[buf][1];
          const auto add_blocks = [&](auto is_wide) {
            constexpr bool WIDE = decltype(is_wide)::value;
            for (int b = 0; b < blocks; ++b, ++it) {
              const int as = it % AS;
              const float* sc = &sm->sc[buf][b][2 * tq];
              const float ws = WIDE ? sm->scw[buf][b][0] : 0.f;
              ok = ok && bar_wait(smem_u32(&sm->acc_full[as]), (it / AS) & 1, limit);
              if (!ok) continue;
              asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
              const uint32_t ta = tbase + (uint32_t)(as * C::DN);
              // load i: columns LC (i / 2) .., lanes 16 (i % 2) ..; the next
              // runs while this one is added
              uint32_t r[2][4 * LDN];
              tmem_ld(r[0], ta);
#pragma unroll
              for (int i = 0; i < 2 * CH; ++i) {
                tmem_wait(r[i & 1]);
                if (i + 1 < 2 * CH) {
                  tmem_ld(r[(i + 1) & 1], ta + ((uint32_t)(16 * ((i + 1) & 1)) << 16) + (uint32_t)(LC * ((i + 1) / 2)));
                } else {
                  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                  if (lane == 0) mbar_arrive(&sm->acc_empty[as]);
                }
#pragma unroll
                for (int g = 0; g < LDN; g += 2) {
                  const int gc = LDN * (i / 2) + g, h = i & 1;
                  const uint32_t* v = &r[i & 1][4 * g];
                  float4 s = *reinterpret_cast<const float4*>(sc + 8 * gc), f;
                  if (WIDE) {
                    const float2 q[4] = {raw ? scale_factors(s.x, ws) : make_float2(1.f, s.x),
                                         raw ? scale_factors(s.y, ws) : make_float2(1.f, s.y),
                                         raw ? scale_factors(s.z, ws) : make_float2(1.f, s.z),
                                         raw ? scale_factors(s.w, ws) : make_float2(1.f, s.w)};
                    f = make_float4(q[0].x, q[1].x, q[2].x, q[3].x);
                    s = make_float4(q[0].y, q[1].y, q[2].y, q[3].y);
                  }
#pragma unroll
                  for (int j = 0; j < 2; ++j) {
                    float* lo = acc[gc][h][j];
                    float* hi = acc[gc + 1][h][j];
                    lo[0] = fmaf(WIDE ? __uint_as_float(v[2 * j]) * f.x : __uint_as_float(v[2 * j]), s.x, lo[0]);
                    lo[1] = fmaf(WIDE ? __uint_as_float(v[2 * j + 1]) * f.y : __uint_as_float(v[2 * j + 1]), s.y, lo[1]);
                    hi[0] = fmaf(WIDE ? __uint_as_float(v[2 * j + 4]) * f.z : __uint_as_float(v[2 * j + 4]), s.z, hi[0]);
                    hi[1] = fmaf(WIDE ? __uint_as_float(v[2 * j + 5]) * f.w : __uint_as_float(v[2 * j + 5]), s.w, hi[1]);
                  }
                }
              }
            }
          };
          if (wide) add_blocks(std::true_type());
          else add_blocks(std::false_type());
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm->sc_empty[buf]);
        }
        if (!ok) {
          sm->err = 1;
#pragma unroll
          for (int i = 0; i < CW / 2; ++i)
            acc[i >> 2][(i >> 1) & 1][i & 1][0] = acc[i >> 2][(i >> 1) & 1][i & 1][1] = __uint_as_float(0x7fffffffu);
        }
        if (p.split > 1) {
          // the stages are idle: this part's sums go there, [row][128]
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          float* red = reinterpret_cast<float*>(smem);
#pragma unroll
          for (int i = 0; i < CW / 8; ++i)
#pragma unroll
            for (int hj = 0; hj < 4; ++hj) {
              const int n = l0 + 8 * hj + nq, c = 8 * i + tq;
              red[c * 128 + n] = acc[i][hj >> 1][hj & 1][0];
              red[(c + 1) * 128 + n] = acc[i][hj >> 1][hj & 1][1];
            }
        } else if (sizeof(Y) == 2 && p.vec && un.n0 + l0 + 32 <= p.N) {
          // eight rows at a time through the warp's staging: four 8 x 8
          // matrices transposed, then 64 bytes a row in 16-byte stores; piece q
          // of row r stands at q ^ (r / 2) % 4
          const int r = lane >> 2, q = lane & 3, mr = lane & 7, mi = lane >> 3;
          const uint32_t put = smem_u32(stage + 64 * mr + 16 * (mi ^ ((mr >> 1) & 3)));
          const uint8_t* get = stage + 64 * r + 16 * (q ^ ((r >> 1) & 3));
          Y* y = static_cast<Y*>(p.y) + (un.row0 + r) * p.ldy + un.n0 + l0 + 8 * q;
#pragma unroll
          for (int i = 0; i < CW / 8; ++i) {
            if (8 * i >= un.rows) break;
            uint32_t v[4];
#pragma unroll
            for (int hj = 0; hj < 4; ++hj)
              v[hj] = pack16<Y>(acc[i][hj >> 1][hj & 1][0], acc[i][hj >> 1][hj & 1][1]);
            asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(put), "r"(v[0]),
                         "r"(v[1]), "r"(v[2]), "r"(v[3])
                         : "memory");
            __syncwarp();
            const uint4 row = *reinterpret_cast<const uint4*>(get);
            if (8 * i + r < un.rows) *reinterpret_cast<uint4*>(y + (int64_t)(8 * i) * p.ldy) = row;
            __syncwarp();
          }
        } else {
          // a warp's store covers 8 columns n of 4 rows
          Y* y = static_cast<Y*>(p.y) + (un.row0 + tq) * p.ldy + un.n0 + l0 + nq;
          const int left = un.rows - tq, nleft = p.N - (un.n0 + l0 + nq);
#pragma unroll
          for (int i = 0; i < CW / 8; ++i)
#pragma unroll
            for (int hj = 0; hj < 4; ++hj) {
              if (8 * hj < nleft) {
                if (8 * i < left) put_y(y + (int64_t)(8 * i) * p.ldy + 8 * hj, acc[i][hj >> 1][hj & 1][0]);
                if (8 * i + 1 < left) put_y(y + (int64_t)(8 * i + 1) * p.ldy + 8 * hj, acc[i][hj >> 1][hj & 1][1]);
              }
            }
        }
      }
    }
  }
  __syncwarp();
  if (!C::XA && p.split > 1 && first < units) {
    // one unit a cluster: part q sums the rows r = q, q + split, ... over the
    // parts in their order. A part whose waits ran out is NaN: its sums were
    // written while copies could still land in the stages, which are drained
    // by now.
    __syncthreads();
    if (*(volatile int*)&sm->err)
      for (int i = tid; i < 128 * NT; i += C::NTHR) reinterpret_cast<float*>(smem)[i] = __uint_as_float(0x7fffffffu);
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    const Fp8Unit un = fp8_unit<NT>(first, p.units_n, p.G, tiles, offs);
    const uint32_t red = smem_u32(smem);
    for (int i = tid; i < 128 * un.rows; i += C::NTHR) {
      const int r = i / 128, n = i % 128;
      if (r % p.split != part || un.n0 + n >= p.N) continue;
      float sum = 0.f;
      for (int q = 0; q < p.split; ++q) {
        float v;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(map_cta(red + 4 * (r * 128 + n), q)) : "memory");
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
  if (warp == EW + 2) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::Cols) : "memory");
  }
}

// 8-bit [planes][rows][cols], `ld` bytes a row, boxes of 128 columns x
// box_rows rows in the 128-byte swizzle; what lies outside reads as zero.
bool map_u8(CUtensorMap* out, const void* base, int64_t cols, int64_t rows, int64_t planes,
            int64_t ld, int box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = map_encoder();
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
  using C = Fp8Cfg<NT>;
  static_assert(C::CtasPerSm * (fp8_smem_bytes<NT>(kOpsMaxExperts) + 1024) <= 228 * 1024, "shared memory");
  static_assert(C::CtasPerSm * C::Cols <= 512, "tensor memory");
  Fp8Params p{};
  p.NB = (a.N + kFK - 1) / kFK;
  p.KB = (a.K + kFK - 1) / kFK;
  p.units_n = (a.N + C::NN - 1) / C::NN;
  const bool maps =
      (a.transposed ? map_u8(&p.w, a.w, a.N, a.K, a.G, a.ldw, kFK) : map_u8(&p.w, a.w, a.K, a.N, a.G, a.ldw, C::XA ? C::BRows : 128)) &&
      map_u8(&p.x, a.x, a.K, a.M, 0, a.ldx, C::XA ? 128 : NT);
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
  p.give_up = a.give_up;
  // XA stores whole sectors, else 16 bytes
  p.vec = !(((uintptr_t)a.y | (uint64_t)(a.ldy * (int64_t)sizeof(Y))) & (C::XA ? 31 : 15));
  // at most this many row tiles: every group's last one may be short
  const int64_t tiles = a.M / NT + (a.M < a.G ? a.M : a.G);
  const int64_t units = tiles * p.units_n;
  if (units > 0x3fffffff) return "too many tiles";
  p.split = 1;
  int64_t grid;
  const int slots = sms * C::CtasPerSm;
  while (!C::XA && p.split < 8 && 2 * p.split * units <= slots && 2 * p.split <= p.KB) p.split *= 2;
  grid = p.split > 1 ? units * p.split : units < slots ? units : slots;
  const size_t smem = fp8_smem_bytes<NT>(a.G);
  auto kernel = fp8_matmul_kernel<NT, TRANS, Y>;
  // once a device: what the largest G needs
  static std::atomic<uint64_t> configured{0};
  int device = 0;
  (void)cudaGetDevice(&device);
  if (device >= 64 || !(configured.load() >> device & 1)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)fp8_smem_bytes<NT>(kOpsMaxExperts)) != cudaSuccess)
      return cudaGetErrorString(cudaGetLastError());
    if (device < 64) configured.fetch_or(1ull << device);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(C::NTHR);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.split > 1 ? 2 : 1;
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
  return fp8_nt<128>(a, dtype, sms, s);
}

}  // namespace dfm
