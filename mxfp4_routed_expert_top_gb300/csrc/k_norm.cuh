// k_norm.cuh — the norms after and before a block, with its gate and the
// residual's scale, and their gradients. With rms(v) = 1 / sqrt(mean(v^2) + eps),
//
//   a = u rms(u) q   (post; else a = u)      u the block's output
//   h = s r + g a                            r the residual stream, g the gate
//   n = h rms(h) v                           the next block's input
//
//   G  = dh + rms(h) (y - H mean(y H)),   H = h rms(h),  y = v dn
//   dr = s G,  dg = G a,  dv = sum over the rows of dn H
//   du = rms(u) (q g G - U mean(q g G U)),   U = u rms(u)   (post; else g G)
//   dq = sum over the rows of g G U
//
// A row stays on chip between its sums and its outputs, so that every array is
// read and written once: HBM bounds the large calls. The sums that a gradient
// row needs are all linear in G's three terms, so one reduction gives them (h^2,
// u^2, y h, and u q g times dh, y and h); its column sums stay in a block's
// registers over its rows and meet in a second kernel, in order. Sums are fp32.
// A row whose squares (with eps) overflow fp32 is summed again at 2^-80, a gradient
// row of which any sum does with h and u at size 1 at most.
//
// Three forms, by the rows. Whole 16-byte pieces: from 513 to 8192 values
// through a ring of bulk copies (block_norm_ring_kernel), shorter, longer and few
// ones straight from memory. Any other rows: value by value, in loops that are
// not unrolled (block_norm_odd_kernel). One file a type includes this one.
// Measured, bf16 with a channel's gate, in us (norms straight | ring, gradients
// straight | ring): 8192 x 7168 149 | 77 (6.1 TB/s), 384 | 142 (5.0 TB/s); 8192 x
// 2048 39 | 27, 103 | 47; 8192 x 640 22 | 15, 44 | 32; 304 x 7168 8.5 | 6.3, 26 | 18.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <type_traits>

#include "fastmath.cuh"
#include "internal.h"
#include "ops.h"
#include "pipeline.cuh"
#include "tcgen.cuh"

namespace dfm {
namespace {

// Of rows whose squares overflow: 32768 squares of 2^128 add up to 2^111, and what
// counts beside a value of 2^56 (the least that overflows) stays normal.
constexpr float kSmall = 0x1p-80f;

template <typename T>
__device__ __forceinline__ float f32_of(T v);
template <>
__device__ __forceinline__ float f32_of(float v) { return v; }
template <>
__device__ __forceinline__ float f32_of(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float f32_of(__half v) { return __half2float(v); }

// ---- eight values as four pairs ------------------------------------------------
// One instruction does a pair (f32x2): the kernels' arithmetic takes half the
// issue slots, which bound the gradient before.
struct Eight {
  Pair v[4];
};

// Eight values, 16-byte aligned, from global or (by its 32-bit address) shared
// memory.
template <typename T>
struct InShared {
  uint32_t at;
};
template <typename T>
__device__ __forceinline__ Eight unpack_eight(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3) {
  const uint32_t w[4] = {w0, w1, w2, w3};
  Eight r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same<T, __half>::value) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      r.v[i] = pair(f.x, f.y);
    } else {
      r.v[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
  }
  return r;
}
template <typename T>
__device__ __forceinline__ Eight load_eight(const T* p, int i) {
  p += i;
  if constexpr (sizeof(T) == 4) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    return {{pair(a.x, a.y), pair(a.z, a.w), pair(b.x, b.y), pair(b.z, b.w)}};
  } else {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    return unpack_eight<T>(w.x, w.y, w.z, w.w);
  }
}
template <typename T>
__device__ __forceinline__ Eight load_eight(InShared<T> p, int i) {
  if constexpr (sizeof(T) == 4) {
    Eight r;
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(r.v[0]), "=l"(r.v[1]) : "r"(p.at + 4 * i));
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(r.v[2]), "=l"(r.v[3]) : "r"(p.at + 4 * i + 16));
    return r;
  } else {
    uint32_t w[4];
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(p.at + 2 * i));
    return unpack_eight<T>(w[0], w[1], w[2], w[3]);
  }
}
template <typename T>
__device__ __forceinline__ void store_eight(T* p, const Eight& e) {
  float2 f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = halves(e.v[i]);
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
  } else {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack16<T>(f[0].x, f[0].y), pack16<T>(f[1].x, f[1].y), pack16<T>(f[2].x, f[2].y), pack16<T>(f[3].x, f[3].y));
  }
}
#define DFM_EIGHT _Pragma("unroll") for (int j = 0; j < 4; ++j)
__device__ __forceinline__ Eight all_of(float x) { return {{pair(x, x), pair(x, x), pair(x, x), pair(x, x)}}; }
__device__ __forceinline__ Eight mul(const Eight& a, const Eight& b) {
  Eight r;
  DFM_EIGHT r.v[j] = mul2(a.v[j], b.v[j]);
  return r;
}
__device__ __forceinline__ Eight mul(const Eight& a, Pair b) {
  Eight r;
  DFM_EIGHT r.v[j] = mul2(a.v[j], b);
  return r;
}

// A row's values as its threads hold them, in parts of eight, tpr such groups
// apart. What lies behind the row is 0.
struct Row {
  int t, tpr, H;
  __device__ __forceinline__ int col(int i) const { return 8 * (t + tpr * i); }
  template <typename P>
  __device__ __forceinline__ Eight load(P p, int i) const {  // a const T* or InShared<T>
    if (col(i) < H) return load_eight(p, col(i));
    return all_of(0.f);
  }
  template <typename T>
  __device__ __forceinline__ void store(T* p, const Eight& e, int i) const {
    if (col(i) < H) store_eight(p + col(i), e);
  }
};

// Sums of N values over a row's threads: a warp, or the whole block of `tpr`.
// Up to eight values share the shuffles: at each of three steps a lane keeps
// half of its values and hands the other half over, so that lane l ends with
// value l / 4 (nine shuffles, not forty). Alternating buffers: one barrier a
// sum. The order of the additions is fixed.
template <int N, int WARPS>
struct RowSum {
  static constexpr int S = WARPS > 16 ? 32 : 16;  // warps of a row at most
  float (*buf)[N][S];                             // [2], shared; zero where the row has no warp
  int which = 0;
  // before the first sum, and a barrier, by the whole block
  __device__ __forceinline__ void init() const {
    for (int i = threadIdx.x; i < 2 * N * S; i += blockDim.x) (&buf[0][0][0])[i] = 0.f;
  }
  __device__ __forceinline__ void operator()(float (&s)[N], int tpr) {
    static_assert(N == 1 || N == 2 || N == 8, "");
    constexpr int G = 32 / N;  // lanes that end with the same value
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int n = N / 2, o = 16; n; n >>= 1, o >>= 1)
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float keep = lane & o ? s[i + n] : s[i], give = lane & o ? s[i] : s[i + n];
        s[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
      }
    float mine = s[0];
#pragma unroll
    for (int o = G / 2; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    // (Two branches for one and two values, one for eight: as the compiler
    // schedules them the norms of 8192 x 7168 take 77 us (6.1 TB/s) and their gradient 142,
    // the other way about 82 and 172.)
    if (N < 8 && tpr > 32 && lane % G == 0) buf[which][lane / G][warp] = mine;
    if (tpr > 32) {
      if (N == 8 && lane % G == 0) buf[which][lane / G][warp] = mine;
      __syncthreads();
      // the G lanes of a value add S / G of its warps each
      mine = 0.f;
      if constexpr (S > G) {
#pragma unroll
        for (int i = 0; i < S / G; i += 4) {
          const float4 f = *reinterpret_cast<const float4*>(&buf[which][lane / G][S / G * (lane % G) + i]);
          mine += (f.x + f.y) + (f.z + f.w);
        }
      } else {
        mine = lane % G < S ? buf[which][lane / G][lane % G] : 0.f;
      }
#pragma unroll
      for (int o = G / 2; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = N == 1 ? mine : __shfl_sync(0xffffffffu, mine, G * i);
    which ^= 1;
  }
};

// 1 / sqrt(mean + eps), of values that were scaled by `small` (and is then of
// those too). rsqrtf is within 2 units of the last place; one Newton step makes
// that one.
__device__ __forceinline__ float rms_of(float sum, float inv, float eps, float small) {
  const float m = fmaf(sum, inv, eps * small * small), r = rsqrtf(m);
  return r == 0.f ? r : fmaf(0.5f * r, fmaf(-m * r, r, 1.f), r);  // 0: an infinite mean
}

// ---- rows, however they are held ----------------------------------------------
// What a kernel knows of a call. kAny asks the arguments; the others stand for
// calls with all of their arrays (u, residual, h and n; u, dh, dn, du and
// dresidual), post norm or not, by what the gate does to a row: nothing (none,
// or a channel's, which is in the weights), a factor, an array.
enum Mode { kAny = -1, kPlain = 0, kToken, kFull, kPost };  // kPost + one of the three: with the post norm
__device__ __forceinline__ constexpr bool mode_is(int mode, int gate) { return mode >= 0 && mode % 3 == gate; }

// What multiplies a thread's columns in every row: the weights behind the
// norms, `q` with a channel's gate. They stay in registers over a block's rows.
template <typename W, int NV>
__device__ __forceinline__ void load_weights(Eight (&q)[NV], Eight (&v)[NV], const Row& at, const void* post_w, const void* channel,
                                             const void* pre_w) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    q[i] = post_w ? at.load(static_cast<const W*>(post_w), i) : all_of(1.f);
    if (channel) q[i] = mul(q[i], at.load(static_cast<const W*>(channel), i));
    v[i] = pre_w ? at.load(static_cast<const W*>(pre_w), i) : all_of(1.f);
  }
}

template <int NV>
__device__ __forceinline__ float square_sum(const Eight (&v)[NV], float factor) {
  Pair s = pair(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (factor != 1.f) {
      const Eight e = mul(v[i], pair(factor, factor));
      DFM_EIGHT s = fma2(e.v[j], e.v[j], s);
    } else {
      DFM_EIGHT s = fma2(v[i].v[j], v[i].v[j], s);
    }
  }
  const float2 f = halves(s);
  return f.x + f.y;
}
// rms of each of R rows.
template <int NV, int R, typename Sum>
__device__ __forceinline__ void rms_rows(float (&rms)[R], const Eight (&v)[R][NV], Sum& sum, int tpr, float inv, float eps) {
  float s[R];
  bool over = false;
#pragma unroll
  for (int r = 0; r < R; ++r) s[r] = square_sum<NV>(v[r], 1.f);
  sum(s, tpr);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    over = over || !(s[r] + eps < INFINITY);
    rms[r] = rms_of(s[r], inv, eps, 1.f);
  }
  if (over) {
    float t[R];
#pragma unroll
    for (int r = 0; r < R; ++r) t[r] = square_sum<NV>(v[r], kSmall);
    sum(t, tpr);
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (!(s[r] + eps < INFINITY)) rms[r] = rms_of(t[r], inv, eps, kSmall) * kSmall;
  }
}

// R rows side by side (their sums share the barriers). in.u(r), in.r(r),
// in.gate(r): where row r's arrays are; there[r]: whether it is one. `poison`
// is 0, or NaN for every output. Every thread of the rows runs this.
template <typename T, int NV, int R, int MODE, typename In, typename Sum>
__device__ __forceinline__ void norm_rows(const BlockNormArgs& p, const Row& at, const In& in, const int64_t (&row)[R],
                                          const bool (&there)[R], Sum& sum, const Eight (&q)[NV], const Eight (&v)[NV], float inv,
                                          float poison) {
  const bool post = MODE < 0 ? p.post != 0 : MODE >= kPost, has_u = MODE >= 0 || p.u, has_r = MODE >= 0 || p.residual;
  const bool token = MODE < 0 ? p.gate_kind == kGateToken : mode_is(MODE, kToken);
  const bool full = MODE < 0 ? p.gate_kind == kGateFull : mode_is(MODE, kFull);
  Eight h[R][NV];
  float rms[R];
  if (has_u) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      rms[r] = 1.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) h[r][i] = at.load(in.u(r), i);
    }
    if (post) rms_rows<NV, R>(rms, h, sum, at.tpr, inv, p.eps);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (token) rms[r] *= there[r] ? static_cast<const float*>(p.gate)[row[r]] : 0.f;
      const Pair factor = pair(rms[r], rms[r]), scale = pair(p.scale, p.scale);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (post || token) h[r][i] = mul(h[r][i], factor);
        h[r][i] = mul(h[r][i], q[i]);
        if (full) h[r][i] = mul(h[r][i], at.load(in.gate(r), i));
        if (has_r) {
          const Eight w = at.load(in.r(r), i);
          DFM_EIGHT h[r][i].v[j] = fma2(scale, w.v[j], h[r][i].v[j]);
        }
      }
    }
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < NV; ++i) h[r][i] = mul(at.load(in.r(r), i), pair(p.scale, p.scale));
  }
  if (poison != 0.f) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < NV; ++i) h[r][i] = all_of(poison);
  }
  if (MODE >= 0 || p.h) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (there[r])
#pragma unroll
        for (int i = 0; i < NV; ++i) at.store(static_cast<T*>(p.h) + row[r] * p.ldh, h[r][i], i);
  }
  if (MODE < 0 && !p.n) return;
  rms_rows<NV, R>(rms, h, sum, at.tpr, inv, p.eps);
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (there[r])
#pragma unroll
      for (int i = 0; i < NV; ++i)
        at.store(static_cast<T*>(p.n) + row[r] * p.ldn, mul(mul(h[r][i], pair(rms[r], rms[r])), v[i]), i);
}

// From a row's sums (s: h^2, u^2, y h, and u q g times dh, y and h; of h and u
// scaled by sh and su): H = h rh, U = u ru, G = dh + rh (y - H along), and
// mean, of q g G U over the row.
struct RowFactors {
  float rh, ru, along, mean, dtoken;
};
__device__ __forceinline__ RowFactors row_factors(const float (&s)[8], float sh, float su, bool dn, bool post, float token, float inv,
                                                  float eps) {
  RowFactors f;
  const float rh = dn ? rms_of(s[0], inv, eps, sh) : 0.f, ru = post ? rms_of(s[1], inv, eps, su) : 1.f / su;
  f.along = rh * s[2] * inv;
  f.rh = rh * sh;
  const float gu = s[3] + f.rh * (s[4] - f.along * rh * s[5]);  // the sum of G q g u su, without a token's gate
  f.dtoken = ru * gu;
  f.mean = token * f.dtoken * inv;
  f.ru = post ? ru * su : 1.f;
  return f;
}

// Whether a row's six sums are all there (what comes of the last four is finite);
// where one left fp32 or has no value, the scales with which h and u are summed
// again: those that make larger rows of size 1, or kSmall where the squares do not
// say. u^2 is summed from the second time on without a norm of u, too.
__device__ __forceinline__ bool summed(const float (&s)[8], const RowFactors& f, float& sh, float& su, float inv, float eps) {
  if (s[0] + s[1] + eps < INFINITY && fabsf(f.along) + fabsf(f.dtoken) < INFINITY) return true;
  constexpr float kNone = 1e-30f;  // beside the squares of what is scaled
  sh = s[0] < INFINITY ? fminf(1.f, sh * rms_of(s[0], inv, kNone, sh)) : kSmall;
  su = s[1] < INFINITY ? fminf(1.f, su * rms_of(s[1], inv, kNone, su)) : kSmall;
  return false;
}

// A row's gradients but the weights', whose terms are added to dq and dv:
//   dq += G U (times the token's or the full gate), dv += dn H.
// A channel's gate does not change from row to row: dpost_w is the gate times
// the sum of G U and the gate's gradient post_w times the same sum. `sums_done`
// runs behind the row's sums (whose barrier comes after the last read of an
// earlier row). ok: false in any thread makes the row NaN.
template <typename T, int NV, int MODE, typename In, typename Sum, typename Done>
__device__ __forceinline__ void grad_row(const BlockNormGradArgs& p, const Row& at, const In& in, int64_t row, Sum& sum,
                                         const Eight (&q)[NV], const Eight (&v)[NV], Eight (&dq)[NV], Eight (&dv)[NV], float inv,
                                         bool ok, Done sums_done) {
  const bool post = MODE < 0 ? p.post != 0 : MODE >= kPost;
  const bool by_token = MODE < 0 ? p.gate_kind == kGateToken : mode_is(MODE, kToken);
  const bool full = MODE < 0 ? p.gate_kind == kGateFull : mode_is(MODE, kFull);
  const bool has_u = MODE >= 0 || p.u, has_dh = MODE >= 0 || p.dh, has_dn = MODE >= 0 || p.dn;
  const float token = by_token ? static_cast<const float*>(p.gate)[row] : 1.f;
  float sh = 1.f, su = 1.f, s[8];
  RowFactors f;
#pragma unroll 1
  for (int again = 0;; ++again) {
    Pair c[6];
#pragma unroll
    for (int i = 0; i < 6; ++i) c[i] = pair(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      Eight h, y;
      if (has_dn) {
        h = at.load(in.h(), i);
        y = mul(at.load(in.dn(), i), v[i]);
        if (again) h = mul(h, pair(sh, sh));
        DFM_EIGHT c[0] = fma2(h.v[j], h.v[j], c[0]);
        DFM_EIGHT c[2] = fma2(h.v[j], y.v[j], c[2]);
      }
      if (!has_u || !(post || by_token)) continue;
      Eight x = at.load(in.u(), i);
      if (again) x = mul(x, pair(su, su));
      if (post || again) DFM_EIGHT c[1] = fma2(x.v[j], x.v[j], c[1]);
      x = mul(x, q[i]);
      if (full) x = mul(x, at.load(in.gate(), i));
      if (has_dh) {
        const Eight w = at.load(in.dh(), i);
        DFM_EIGHT c[3] = fma2(x.v[j], w.v[j], c[3]);
      }
      if (has_dn) {
        DFM_EIGHT c[4] = fma2(x.v[j], y.v[j], c[4]);
        DFM_EIGHT c[5] = fma2(x.v[j], h.v[j], c[5]);
      }
    }
#pragma unroll
    for (int i = 0; i < 6; ++i) {
      const float2 f = halves(c[i]);
      s[i] = f.x + f.y;
    }
    s[6] = ok ? 0.f : 1.f, s[7] = 0.f;
    sum(s, at.tpr);
    f = row_factors(s, sh, su, has_dn, post, token, inv, p.eps);
    if (again == 3 || summed(s, f, sh, su, inv, p.eps)) break;
  }
  const bool bad = s[6] != 0.f;
  float scale = p.scale;
  if (bad) f.rh = f.ru = f.dtoken = scale = __uint_as_float(0x7fffffffu);
  if (by_token && p.dgate && at.t == 0) static_cast<float*>(p.dgate)[row] = f.dtoken;
  sums_done();
  const Pair rh = pair(f.rh, f.rh), ru = pair(f.ru, f.ru), along = pair(-f.along, -f.along), mean = pair(-f.mean, -f.mean);
  const Pair scale2 = pair(scale, scale), token2 = pair(token, token);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    Eight G, y;
    G = has_dh ? at.load(in.dh(), i) : all_of(0.f);
    if (has_dn) {
      const Eight h = mul(at.load(in.h(), i), rh), d = at.load(in.dn(), i);
      DFM_EIGHT {
        dv[i].v[j] = fma2(d.v[j], h.v[j], dv[i].v[j]);
        G.v[j] = fma2(rh, fma2(h.v[j], along, mul2(d.v[j], v[i].v[j])), G.v[j]);
      }
    }
    if (MODE >= 0 || p.dresidual) at.store(static_cast<T*>(p.dresidual) + row * p.lddr, mul(G, scale2), i);
    if (!has_u) continue;
    const Eight x = mul(at.load(in.u(), i), ru);  // U, or u
    if (full) {
      if (p.dgate) at.store(static_cast<T*>(p.dgate) + row * p.lddg, mul(G, mul(x, q[i])), i);  // G a
      G = mul(G, at.load(in.gate(), i));
    }
    if (by_token) G = mul(G, token2);
    DFM_EIGHT {
      dq[i].v[j] = fma2(G.v[j], x.v[j], dq[i].v[j]);
      y.v[j] = mul2(G.v[j], q[i].v[j]);
      if (post) y.v[j] = mul2(ru, fma2(x.v[j], mean, y.v[j]));
    }
    if (bad) y = all_of(scale);
    if (MODE >= 0 || p.du) at.store(static_cast<T*>(p.du) + row * p.lddu, y, i);
  }
}

// The sums of a worker's rows, behind each other: part[array][worker][H].
__device__ __forceinline__ bool wants_dq(const BlockNormGradArgs& p) { return p.dpost_w || (p.dgate && p.gate_kind == kGateChannel); }
// The kernel that joins them, and only that, may start early (it waits for the
// end of this one): what else may follow in the stream need not wait.
__device__ __forceinline__ void let_columns_start(const BlockNormGradArgs& p) {
  if (wants_dq(p) || p.dpre_w) pdl_launch_dependents();
}
template <int NV>
__device__ __forceinline__ void put_columns(const BlockNormGradArgs& p, const Row& at, float* part, int worker, int workers,
                                            const Eight (&dq)[NV], const Eight (&dv)[NV]) {
  float* o = part + (int64_t)worker * p.H;
  if (wants_dq(p)) {
#pragma unroll
    for (int i = 0; i < NV; ++i) at.store(o, dq[i], i);
    o += (int64_t)workers * p.H;
  }
  if (p.dpre_w) {
#pragma unroll
    for (int i = 0; i < NV; ++i) at.store(o, dv[i], i);
  }
}

// ---- rows straight from global memory ------------------------------------------
// Where a row takes a block of 1024 threads (64 registers each at most) these spill: the
// gradient of few or wide rows up to 8192 336 bytes a thread, rows above 8192 728 to
// 1608 and their gradient 1800 to 2790.
template <typename T>
struct GlobalRow {
  const BlockNormArgs& p;
  int64_t row;
  __device__ __forceinline__ const T* u(int) const { return static_cast<const T*>(p.u) + row * p.ldu; }
  __device__ __forceinline__ const T* r(int) const { return static_cast<const T*>(p.residual) + row * p.ldr; }
  __device__ __forceinline__ const T* gate(int) const { return static_cast<const T*>(p.gate) + row * p.ldg; }
};
template <typename T>
struct GlobalGradRow {
  const BlockNormGradArgs& p;
  int64_t row;
  __device__ __forceinline__ const T* dh() const { return static_cast<const T*>(p.dh) + row * p.lddh; }
  __device__ __forceinline__ const T* dn() const { return static_cast<const T*>(p.dn) + row * p.lddn; }
  __device__ __forceinline__ const T* h() const { return static_cast<const T*>(p.h) + row * p.ldh; }
  __device__ __forceinline__ const T* u() const { return static_cast<const T*>(p.u) + row * p.ldu; }
  __device__ __forceinline__ const T* gate() const { return static_cast<const T*>(p.gate) + row * p.ldg; }
};

template <typename T, typename W, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) block_norm_kernel(const BlockNormArgs p, int tpr) {
  __shared__ __align__(16) float buf[2][1][THREADS / 32 > 16 ? 32 : 16];
  const int rows = blockDim.x / tpr, g = threadIdx.x / tpr;
  const int64_t row[1] = {(int64_t)blockIdx.x * rows + g};
  const bool there[1] = {true};
  const Row at{(int)threadIdx.x - g * tpr, tpr, p.H};
  RowSum<1, THREADS / 32> sum{buf};
  sum.init();
  __syncthreads();
  pdl_wait();
  if (row[0] >= p.T) return;  // a whole warp: rows == 1 where a row has more
  Eight q[NV], v[NV];
  load_weights<W, NV>(q, v, at, p.post_w, p.gate_kind == kGateChannel ? p.gate : nullptr, p.pre_w);
  norm_rows<T, NV, 1, kAny>(p, at, GlobalRow<T>{p, row[0]}, row, there, sum, q, v, 1.f / (float)p.H, 0.f);
}

template <typename T, typename W, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) block_norm_grad_kernel(const BlockNormGradArgs p, int tpr, float* part, int workers) {
  __shared__ __align__(16) float buf[2][8][THREADS / 32 > 16 ? 32 : 16];
  const int rows = blockDim.x / tpr, g = threadIdx.x / tpr;
  const int worker = blockIdx.x * rows + g;
  const Row at{(int)threadIdx.x - g * tpr, tpr, p.H};
  RowSum<8, THREADS / 32> sum{buf};
  sum.init();
  __syncthreads();
  const float inv = 1.f / (float)p.H;
  pdl_wait();
  let_columns_start(p);
  if (worker >= workers) return;  // a whole warp: rows == 1 where a row has more
  Eight dq[NV], dv[NV], q[NV], v[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) dq[i] = dv[i] = all_of(0.f);
  load_weights<W, NV>(q, v, at, p.post_w, p.gate_kind == kGateChannel ? p.gate : nullptr, p.pre_w);
  for (int64_t row = worker; row < p.T; row += workers)
    grad_row<T, NV, kAny>(p, at, GlobalGradRow<T>{p, row}, row, sum, q, v, dq, dv, inv, true, [] {});
  put_columns<NV>(p, at, part, worker, workers, dq, dv);
}

// ---- rows through shared memory -------------------------------------------------
// Persistent blocks, R rows at a time; bulk copies bring the arrays of the next
// rows into a ring of stages meanwhile, so that a row's sums and outputs do not
// stop the stream. Lane a of warp 0 copies array a.
constexpr int kArrays = 5;
struct RingArrays {
  const char* base[kArrays];  // null: absent
  int64_t ld[kArrays];        // bytes
  int64_t T;
  int bytes;   // of a row, a multiple of 16
  int arrays;  // those there are
  int stages;
};
template <int R>
struct Ring {
  const RingArrays& r;
  uint32_t start, full;  // shared addresses: the stages, their barriers
  const char* base;      // this lane's array, or null
  int64_t ld;
  uint32_t place;  // of the array in a row's place

  __device__ __forceinline__ Ring(const RingArrays& a, const uint8_t* memory, uint64_t* bars)
      : r(a), start(smem_u32(memory)), full(smem_u32(bars)), base(nullptr), ld(0), place(0) {
    if (threadIdx.x < kArrays) {
      base = r.base[threadIdx.x];
      ld = r.ld[threadIdx.x];
      for (int i = 0; i < (int)threadIdx.x; ++i) place += r.base[i] ? r.bytes : 0;
    }
  }
  __device__ __forceinline__ uint32_t row_at(int s, int i) const { return start + (uint32_t)((s * R + i) * r.arrays) * r.bytes; }
  // Warp 0: the copies of the R rows from `first` (those there are) into stage s.
  __device__ __forceinline__ void fill(int s, int64_t first) const {
    if (threadIdx.x >= kArrays) return;
    const int rows = (int)min((int64_t)R, r.T - first);
    const uint32_t bar = full + 8 * s;
    if (threadIdx.x == 0)
      asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(bar),
                   "r"((uint32_t)(rows * r.arrays * r.bytes))
                   : "memory");
    if (!base) return;
    const uint64_t once = l2_evict_first_policy();
    for (int i = 0; i < rows; ++i)
      asm volatile(
          "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
              row_at(s, i) + place),
          "l"(base + (first + i) * ld), "r"((uint32_t)r.bytes), "r"(bar), "l"(once)
          : "memory");
  }
};
// Where the arrays of the rows of a stage start.
template <typename T, int R>
struct RingRows {
  uint32_t at[R][kArrays];
  template <typename RingT>
  __device__ __forceinline__ void set(const RingT& ring, int i, int s, int from) {
    uint32_t a = ring.row_at(s, from);
#pragma unroll
    for (int n = 0; n < kArrays; ++n) {
      at[i][n] = a;
      a += ring.r.base[n] ? ring.r.bytes : 0;
    }
  }
  __device__ __forceinline__ InShared<T> u(int r) const { return {at[r][0]}; }
  __device__ __forceinline__ InShared<T> r(int r) const { return {at[r][1]}; }
  __device__ __forceinline__ InShared<T> gate(int r) const { return {at[r][2]}; }
};
template <typename T>
struct RingGradRow : RingRows<T, 1> {
  __device__ __forceinline__ InShared<T> dh() const { return {this->at[0][0]}; }
  __device__ __forceinline__ InShared<T> dn() const { return {this->at[0][1]}; }
  __device__ __forceinline__ InShared<T> h() const { return {this->at[0][2]}; }
  __device__ __forceinline__ InShared<T> u() const { return {this->at[0][3]}; }
  __device__ __forceinline__ InShared<T> gate() const { return {this->at[0][4]}; }
};

constexpr int kRingThreads = 512;  // 16 values a thread: rows of up to 8192
constexpr int kRingStages = 6;

// R rows a stage (two of 16 bits: their sums share two barriers).
template <typename T, typename W, int MODE>
__global__ void __launch_bounds__(kRingThreads, 1) block_norm_ring_kernel(const BlockNormArgs p, const __grid_constant__ RingArrays r) {
  constexpr int R = sizeof(T) == 2 ? 2 : 1;
  extern __shared__ __align__(128) uint8_t memory[];
  __shared__ uint64_t full[kRingStages];
  __shared__ __align__(16) float buf[2][R][16];
  const Row at{(int)threadIdx.x, (int)blockDim.x, p.H};
  RowSum<R, 16> sum{buf};
  const Ring<R> ring(r, memory, full);
  sum.init();
  if (threadIdx.x == 0) {
    for (int i = 0; i < r.stages; ++i) mbar_init(&full[i], 1);
    fence_barrier_init();
  }
  __syncthreads();
  pdl_wait();
  const int64_t step = (int64_t)R * gridDim.x;
  int64_t ahead = (int64_t)R * blockIdx.x;  // the next rows to copy
  for (int i = 0; i < r.stages && ahead < p.T; ++i, ahead += step) ring.fill(i, ahead);
  Eight q[2], v[2];
  load_weights<W, 2>(q, v, at, p.post_w, p.gate_kind == kGateChannel ? p.gate : nullptr, p.pre_w);
  const float inv = 1.f / (float)p.H;
  int s = 0, before = -1;
  uint32_t phase = 0, limit = kWaitLimit;
  for (int64_t first = (int64_t)R * blockIdx.x; first < p.T; first += step) {
    bool ok = mbar_wait(&full[s], phase, limit);
    if (!ok) limit = 1;
    // every thread is past the rows before: their stage takes the next copies
    ok = __syncthreads_and(ok);
    if (before >= 0 && ahead < p.T) {
      ring.fill(before, ahead);
      ahead += step;
    }
    int64_t row[R];
    bool there[R];
    RingRows<T, R> in;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      there[i] = first + i < p.T;
      row[i] = first + i;
      in.set(ring, i, s, there[i] ? i : 0);  // a row that is not there: another's values, not stored
    }
    norm_rows<T, 2, R, MODE>(p, at, in, row, there, sum, q, v, inv, ok ? 0.f : __uint_as_float(0x7fffffffu));
    before = s;
    if (++s == r.stages) {
      s = 0;
      phase ^= 1;
    }
  }
  if (limit == 1)  // a wait ran out: copies in flight land before the block leaves
    for (int i = 0; i < r.stages; ++i) (void)mbar_wait(&full[i], i < s ? phase : phase ^ 1);
}

template <typename T, typename W, int MODE>
__global__ void __launch_bounds__(kRingThreads, 1) block_norm_grad_ring_kernel(const BlockNormGradArgs p, const __grid_constant__ RingArrays r, float* part) {
  extern __shared__ __align__(128) uint8_t memory[];
  __shared__ uint64_t full[kRingStages];
  __shared__ __align__(16) float buf[2][8][16];
  const Row at{(int)threadIdx.x, (int)blockDim.x, p.H};
  RowSum<8, 16> sum{buf};
  const Ring<1> ring(r, memory, full);
  sum.init();
  if (threadIdx.x == 0) {
    for (int i = 0; i < r.stages; ++i) mbar_init(&full[i], 1);
    fence_barrier_init();
  }
  __syncthreads();
  pdl_wait();
  let_columns_start(p);
  int64_t ahead = blockIdx.x;
  for (int i = 0; i < r.stages && ahead < p.T; ++i, ahead += gridDim.x) ring.fill(i, ahead);
  Eight dq[2], dv[2], q[2], v[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) dq[i] = dv[i] = all_of(0.f);
  load_weights<W, 2>(q, v, at, p.post_w, p.gate_kind == kGateChannel ? p.gate : nullptr, p.pre_w);
  const float inv = 1.f / (float)p.H;
  int s = 0, before = -1;
  uint32_t phase = 0, limit = kWaitLimit;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
    const bool ok = mbar_wait(&full[s], phase, limit);
    if (!ok) limit = 1;
    RingGradRow<T> in;
    in.set(ring, 0, s, 0);
    grad_row<T, 2, MODE>(p, at, in, row, sum, q, v, dq, dv, inv, ok, [&] {
      // behind the sums' barrier every thread is past the row before
      if (before >= 0 && ahead < p.T) {
        ring.fill(before, ahead);
        ahead += gridDim.x;
      }
    });
    before = s;
    if (++s == r.stages) {
      s = 0;
      phase ^= 1;
    }
  }
  if (limit == 1)  // a wait ran out: copies in flight land before the block leaves
    for (int i = 0; i < r.stages; ++i) (void)mbar_wait(&full[i], i < s ? phase : phase ^ 1);
  put_columns<2>(p, at, part, blockIdx.x, gridDim.x, dq, dv);
}

// ---- rows of any length and alignment --------------------------------------------
// A block a row, value by value, in loops that stay small (unrolled over all of
// a thread's values they did not fit the instruction cache, which took most of
// the time). Four values' loads go out together, before the first store, which
// they could not pass. The second pass over a row finds it in L1 or L2. What a
// thread keeps of a row (h) or over its rows (the column sums) is in shared
// memory, at places that no other thread touches; longer rows' column sums in
// global. Issue slots bound it (66%: a value a load): the gradient of 1023 x 2049
// fp32 21 us, 2.4 TB/s, 53 with the loops unrolled.
constexpr int kOddThreads = 256, kOddUnroll = 4;

// Values c, c + kOddThreads, ... (kOddUnroll of them) of a row that may be
// absent (0, or `absent`).
template <typename T>
__device__ __forceinline__ void load_odd(float (&v)[kOddUnroll], const T* p, int c, int H, float absent = 0.f) {
#pragma unroll
  for (int i = 0; i < kOddUnroll; ++i) v[i] = p && c + i * kOddThreads < H ? f32_of<T>(p[c + i * kOddThreads]) : absent;
}
template <typename T>
__device__ __forceinline__ void store_odd(T* p, const float (&v)[kOddUnroll], int c, int H) {
#pragma unroll
  for (int i = 0; i < kOddUnroll; ++i)
    if (c + i * kOddThreads < H) p[c + i * kOddThreads] = T(v[i]);
}
#define DFM_ODD _Pragma("unroll") for (int i = 0; i < kOddUnroll; ++i)
#define DFM_ODD_ROW _Pragma("unroll 1") for (int c = threadIdx.x; c < H; c += kOddUnroll * kOddThreads)
template <typename T>
__device__ __forceinline__ const T* row_of(const void* p, int64_t row, int64_t ld) {
  return p ? static_cast<const T*>(p) + row * ld : nullptr;
}

template <typename T, typename W>
__global__ void __launch_bounds__(kOddThreads) block_norm_odd_kernel(const BlockNormArgs p) {
  extern __shared__ float kept[];  // h [H]
  __shared__ __align__(16) float buf[2][1][16];
  RowSum<1, 16> sum{buf};
  sum.init();
  __syncthreads();
  pdl_wait();
  const int64_t row = blockIdx.x;
  const int H = p.H;
  const T *u = row_of<T>(p.u, row, p.ldu), *res = row_of<T>(p.residual, row, p.ldr);
  const T* full = p.gate_kind == kGateFull ? row_of<T>(p.gate, row, p.ldg) : nullptr;
  const W *post_w = static_cast<const W*>(p.post_w), *pre_w = static_cast<const W*>(p.pre_w);
  const W* channel = p.gate_kind == kGateChannel ? static_cast<const W*>(p.gate) : nullptr;
  const float inv = 1.f / (float)H;
  float factor = 1.f, x[kOddUnroll], y[kOddUnroll], w[kOddUnroll], g[kOddUnroll];
  if (u && p.post) {
    float small = 1.f, s[1];
#pragma unroll 1
    for (int again = 0;; ++again) {
      s[0] = 0.f;
      DFM_ODD_ROW {
        load_odd(x, u, c, H);
        DFM_ODD s[0] = fmaf(x[i] * small, x[i] * small, s[0]);
      }
      sum(s, kOddThreads);
      if (again || s[0] + p.eps < INFINITY) break;
      small = kSmall;
    }
    factor = rms_of(s[0], inv, p.eps, small) * small;
  }
  if (p.gate_kind == kGateToken) factor *= static_cast<const float*>(p.gate)[row];
  float s[1] = {0.f}, small = 1.f;
  T* h = p.h ? static_cast<T*>(p.h) + row * p.ldh : nullptr;
  DFM_ODD_ROW {
    load_odd(x, u, c, H);
    load_odd(y, res, c, H);
    load_odd(w, post_w, c, H, 1.f);
    load_odd(g, channel, c, H, 1.f);
    if (full) load_odd(g, full, c, H);
    DFM_ODD {
      y[i] = fmaf(p.scale, y[i], u ? x[i] * factor * w[i] * g[i] : 0.f);
      s[0] = fmaf(y[i], y[i], s[0]);
      if (c + i * kOddThreads < H) kept[c + i * kOddThreads] = y[i];
    }
    if (h) store_odd(h, y, c, H);
  }
  if (!p.n) return;
  sum(s, kOddThreads);
  if (!(s[0] + p.eps < INFINITY)) {
    small = kSmall;
    s[0] = 0.f;
    DFM_ODD_ROW {
      load_odd(x, (const float*)kept, c, H);
      DFM_ODD s[0] = fmaf(x[i] * small, x[i] * small, s[0]);
    }
    sum(s, kOddThreads);
  }
  factor = rms_of(s[0], inv, p.eps, small) * small;
  T* n = static_cast<T*>(p.n) + row * p.ldn;
  DFM_ODD_ROW {
    load_odd(x, (const float*)kept, c, H);
    load_odd(w, pre_w, c, H, 1.f);
    DFM_ODD x[i] = x[i] * factor * w[i];
    store_odd(n, x, c, H);
  }
}

template <typename T, typename W>
__global__ void __launch_bounds__(kOddThreads) block_norm_grad_odd_kernel(const BlockNormGradArgs p, float* part, int in_shared) {
  extern __shared__ float kept[];  // the column sums [2][H], where they fit
  __shared__ __align__(16) float buf[2][8][16];
  RowSum<8, 16> sum{buf};
  sum.init();
  const int H = p.H;
  const bool want_q = wants_dq(p), want_v = p.dpre_w != nullptr;
  float* out_q = part + (int64_t)blockIdx.x * H;
  float* out_v = out_q + (want_q ? (int64_t)gridDim.x * H : 0);
  float *dq = in_shared ? kept : out_q, *dv = in_shared ? kept + H : out_v;
  __syncthreads();
  pdl_wait();
  let_columns_start(p);
  for (int c = threadIdx.x; c < H; c += kOddThreads) {
    if (want_q) dq[c] = 0.f;
    if (want_v) dv[c] = 0.f;
  }
  const float inv = 1.f / (float)H;
  const W *post_w = static_cast<const W*>(p.post_w), *pre_w = static_cast<const W*>(p.pre_w);
  const W* channel = p.gate_kind == kGateChannel ? static_cast<const W*>(p.gate) : nullptr;
  const bool by_token = p.gate_kind == kGateToken;
  const void* gates = p.gate_kind == kGateFull ? p.gate : nullptr;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
    const T *dh = row_of<T>(p.dh, row, p.lddh), *dn = row_of<T>(p.dn, row, p.lddn), *u = row_of<T>(p.u, row, p.ldu);
    const T *h = p.dn ? row_of<T>(p.h, row, p.ldh) : nullptr, *full = row_of<T>(gates, row, p.ldg);
    const float token = by_token ? static_cast<const float*>(p.gate)[row] : 1.f;
    RowFactors f;
    float sh = 1.f, su = 1.f, s[8], a[kOddUnroll], b[kOddUnroll], x[kOddUnroll], y[kOddUnroll], q[kOddUnroll], g[kOddUnroll], v[kOddUnroll];
#pragma unroll 1
    for (int again = 0;; ++again) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = 0.f;
      DFM_ODD_ROW {
        load_odd(a, h, c, H);
        load_odd(y, dn, c, H);
        load_odd(x, u, c, H);
        load_odd(b, dh, c, H);
        load_odd(q, post_w, c, H, 1.f);
        load_odd(v, pre_w, c, H, 1.f);
        load_odd(g, channel, c, H, 1.f);
        if (full) load_odd(g, full, c, H);
        DFM_ODD {
          a[i] *= sh, x[i] *= su, y[i] *= v[i];
          s[0] = fmaf(a[i], a[i], s[0]);
          if (p.post || again) s[1] = fmaf(x[i], x[i], s[1]);
          s[2] = fmaf(a[i], y[i], s[2]);
          x[i] *= q[i] * g[i];
          s[3] = fmaf(x[i], b[i], s[3]);
          s[4] = fmaf(x[i], y[i], s[4]);
          s[5] = fmaf(x[i], a[i], s[5]);
        }
      }
      sum(s, kOddThreads);
      f = row_factors(s, sh, su, p.dn != nullptr, p.post != 0, token, inv, p.eps);
      if (again == 3 || summed(s, f, sh, su, inv, p.eps)) break;
    }
    if (by_token && p.dgate && threadIdx.x == 0) static_cast<float*>(p.dgate)[row] = f.dtoken;
    T* dr = p.dresidual ? static_cast<T*>(p.dresidual) + row * p.lddr : nullptr;
    T* du = p.du ? static_cast<T*>(p.du) + row * p.lddu : nullptr;
    T* dg = gates && p.dgate ? static_cast<T*>(p.dgate) + row * p.lddg : nullptr;
    DFM_ODD_ROW {
      load_odd(a, h, c, H);
      load_odd(y, dn, c, H);
      load_odd(x, u, c, H);
      load_odd(b, dh, c, H);
      load_odd(q, post_w, c, H, 1.f);
      load_odd(v, pre_w, c, H, 1.f);
      load_odd(g, channel, c, H, 1.f);
      DFM_ODD {
        const int at = c + i * kOddThreads;
        a[i] *= f.rh;
        if (want_v && at < H) dv[at] = fmaf(y[i], a[i], dv[at]);
        b[i] = fmaf(f.rh, fmaf(-a[i], f.along, y[i] * v[i]), b[i]);  // G
        y[i] = p.scale * b[i];
      }
      if (full) load_odd(v, full, c, H);  // (before the stores)
      if (dr) store_odd(dr, y, c, H);
      if (!u) continue;
      DFM_ODD {
        const int at = c + i * kOddThreads;
        x[i] *= f.ru;
        q[i] *= g[i];
        y[i] = b[i] * (x[i] * q[i]);  // G a
        b[i] *= full ? v[i] : token;
        if (want_q && at < H) dq[at] = fmaf(b[i], x[i], dq[at]);
        b[i] *= q[i];
        if (p.post) b[i] = f.ru * fmaf(-x[i], f.mean, b[i]);
      }
      if (dg) store_odd(dg, y, c, H);
      if (du) store_odd(du, b, c, H);
    }
  }
  if (!in_shared) return;
  for (int c = threadIdx.x; c < H; c += kOddThreads) {
    if (want_q) out_q[c] = dq[c];
    if (want_v) out_v[c] = dv[c];
  }
}

// The workers' sums, in order of 16 interleaved parts. The first array's (G U)
// give two gradients, each times the other's factor.
template <typename W>
struct ColumnOuts {
  float *dpost_w, *dgate, *dpre_w;
  const W *post_w, *gate;  // null: 1
  int first;               // which array has dn H
};
constexpr int kColThreads = 512;
template <typename W>
__global__ void __launch_bounds__(kColThreads) norm_columns_kernel(const float* part, const ColumnOuts<W> o, int workers, int H) {
  constexpr int WARPS = kColThreads / 32;
  __shared__ float sums[WARPS][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  const float* in = part + (int64_t)blockIdx.y * workers * H;
  pdl_wait();
  float s = 0.f;
  if (c < H)
#pragma unroll 10
    for (int w = warp; w < workers; w += WARPS) s += in[(int64_t)w * H + c];
  sums[warp][lane] = s;
  __syncthreads();
  if (warp || c >= H) return;
  s = 0.f;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) s += sums[w][lane];
  if ((int)blockIdx.y == o.first) {
    o.dpre_w[c] = s;
  } else {
    if (o.dpost_w) o.dpost_w[c] = o.gate ? s * f32_of<W>(o.gate[c]) : s;
    if (o.dgate) o.dgate[c] = o.post_w ? s * f32_of<W>(o.post_w[c]) : s;
  }
}

// ---- host ------------------------------------------------------------------------
bool whole(const void* p, int64_t ld, int size) { return !p || !(((uintptr_t)p | (uint64_t)(ld * size)) & 15); }

// Threads of a row, threads of a block.
struct Shape {
  int tpr, threads;
};
Shape shape_of(int H, int each) {
  const int tpr = ((H + each - 1) / each + 31) / 32 * 32;
  return {tpr, tpr == 32 ? 128 : tpr};
}

constexpr int kRingBytes = 224 * 1024;  // of a block at most; an SM has 4 KB more, which each block needs beside it

// The ring's bytes for `blocks` blocks an SM of `rows` rows a stage; none
// (stages = 0) where two stages do not fit.
size_t ring_close(RingArrays& r, int rows, int blocks) {
  for (int a = 0; a < kArrays; ++a) r.arrays += r.base[a] != nullptr;
  const int stage = rows * r.arrays * r.bytes, n = ((kRingBytes + 4096) / blocks - 4096) / stage;
  r.stages = n < 2 ? 0 : n > kRingStages ? kRingStages : n;
  return (size_t)r.stages * stage;
}

// A kernel's dynamic shared memory, once a device.
template <typename K>
cudaError_t allow_shared(K kernel, std::atomic<uint64_t>& done) {
  int device = 0;
  (void)cudaGetDevice(&device);
  if (device < 64 && done.load() >> device & 1) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
  if (e == cudaSuccess && device < 64) done.fetch_or(1ull << device);
  return e;
}

// The kernel mode of a call that has all of its arrays.
int mode_of(int post, int gate_kind) {
  return (post ? kPost : 0) + (gate_kind == kGateToken ? kToken : gate_kind == kGateFull ? kFull : kPlain);
}

template <typename T, typename W, int MODE>
cudaError_t norm_ring(const BlockNormArgs& p, const RingArrays& r, int64_t blocks, int threads, size_t smem, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_shared(block_norm_ring_kernel<T, W, MODE>, done);
  if (e != cudaSuccess) return e;
  return launch_after_previous(block_norm_ring_kernel<T, W, MODE>, dim3((unsigned)blocks), dim3(threads), smem, s, p, r);
}

template <typename T, typename W>
cudaError_t norm_tw(const BlockNormArgs& p, int sms, cudaStream_t s) {
  constexpr int z = sizeof(T);
  const bool full = p.gate_kind == kGateFull;
  const bool vec = p.H % 8 == 0 && whole(p.u, p.ldu, z) && whole(p.residual, p.ldr, z) && whole(p.h, p.ldh, z) && whole(p.n, p.ldn, z) &&
                   whole(p.post_w, 0, 1) && whole(p.pre_w, 0, 1) &&
                   (p.gate_kind == kGateNone || p.gate_kind == kGateToken || whole(p.gate, full ? p.ldg : 0, z));
  if (!vec) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_shared(block_norm_odd_kernel<T, W>, done);
    if (e != cudaSuccess) return e;
    return launch_after_previous(block_norm_odd_kernel<T, W>, dim3((unsigned)p.T), dim3(kOddThreads), 4 * (size_t)p.H, s, p);
  }
  const Shape sh16 = shape_of(p.H, 16);
  const int each = kRingThreads / sh16.threads;  // blocks an SM of the ring
  // rows that all start at once gain nothing from a ring (152 x 7168 4.7 us straight
  // and 5.3, 304 8.5 and 6.3; 304 x 2048 4.4 and 4.7, 1000 8.0 and 6.2)
  if (p.H > 512 && p.H <= 16 * kRingThreads && p.T > (int64_t)sms * each) {
    const Shape sh = sh16;
    const int rows = z == 2 ? 2 : 1;  // rows a stage
    RingArrays r{};
    r.T = p.T;
    r.bytes = p.H * z;
    const void* base[3] = {p.u, p.residual, full ? p.gate : nullptr};
    const int64_t ld[3] = {p.ldu, p.ldr, p.ldg};
    for (int a = 0; a < 3; ++a) r.base[a] = static_cast<const char*>(base[a]), r.ld[a] = ld[a] * z;
    const size_t smem = ring_close(r, rows, each);
    if (r.stages) {
      const int64_t most = (int64_t)sms * each, steps = (p.T + rows - 1) / rows, blocks = steps < most ? steps : most;
      switch (p.u && p.residual && p.h && p.n ? mode_of(p.post, p.gate_kind) : kAny) {
        case kPlain: return norm_ring<T, W, kPlain>(p, r, blocks, sh.threads, smem, s);
        case kToken: return norm_ring<T, W, kToken>(p, r, blocks, sh.threads, smem, s);
        case kPost: return norm_ring<T, W, kPost>(p, r, blocks, sh.threads, smem, s);
        case kPost + kToken: return norm_ring<T, W, kPost + kToken>(p, r, blocks, sh.threads, smem, s);
        case kPost + kFull: return norm_ring<T, W, kPost + kFull>(p, r, blocks, sh.threads, smem, s);
        default: return norm_ring<T, W, kAny>(p, r, blocks, sh.threads, smem, s);
      }
    }
  }
  const Shape sh = shape_of(p.H, p.H <= 8192 ? 16 : 32);
  const int rows = sh.threads / sh.tpr;
  const dim3 grid((unsigned)((p.T + rows - 1) / rows));
  return p.H <= 8192 ? launch_after_previous(block_norm_kernel<T, W, 2, 512>, grid, dim3(sh.threads), 0, s, p, sh.tpr)
                     : launch_after_previous(block_norm_kernel<T, W, 4, 1024>, grid, dim3(sh.threads), 0, s, p, sh.tpr);
}

// Rows that are summed side by side, at most: about 1024 threads an SM of 8
// values each, 512 of 16, of at most 160 SMs.
int64_t grad_workers(int64_t T, int H) {
  const Shape sh = shape_of(H, H <= 8192 ? 8 : 32);
  const int64_t blocks = 160 * (1024 / sh.threads), rows = sh.threads / sh.tpr;
  return T < blocks * rows ? T : blocks * rows;
}

template <typename T, typename W, int MODE>
cudaError_t grad_ring(const BlockNormGradArgs& p, const RingArrays& r, float* part, int64_t workers, int threads, size_t smem, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_shared(block_norm_grad_ring_kernel<T, W, MODE>, done);
  if (e != cudaSuccess) return e;
  return launch_after_previous(block_norm_grad_ring_kernel<T, W, MODE>, dim3((unsigned)workers), dim3(threads), smem, s, p, r, part);
}

// The rows' kernel; `workers`: in how many parts the column sums are.
template <typename T, typename W>
cudaError_t grad_rows(const BlockNormGradArgs& p, float* part, int64_t* workers, int sms, cudaStream_t s) {
  constexpr int z = sizeof(T);
  const bool full = p.gate_kind == kGateFull;
  const bool vec = p.H % 8 == 0 && whole(p.dh, p.lddh, z) && whole(p.dn, p.lddn, z) && whole(p.h, p.ldh, z) && whole(p.u, p.ldu, z) &&
                   whole(p.du, p.lddu, z) && whole(p.dresidual, p.lddr, z) && whole(p.post_w, 0, 1) && whole(p.pre_w, 0, 1) &&
                   (p.gate_kind == kGateNone || p.gate_kind == kGateToken || whole(p.gate, full ? p.ldg : 0, z)) &&
                   (!full || whole(p.dgate, p.lddg, z));
  int64_t& n = *workers;
  n = grad_workers(p.T, p.H);
  const auto at_most = [&](int64_t most) { n = n < most ? n : most; };
  if (!vec) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_shared(block_norm_grad_odd_kernel<T, W>, done);
    if (e != cudaSuccess) return e;
    const int in_shared = 8 * p.H <= kRingBytes;
    const int each = !in_shared ? 4 : kRingBytes / (8 * p.H);  // blocks an SM
    at_most((int64_t)sms * (each < 4 ? each : 4));
    return launch_after_previous(block_norm_grad_odd_kernel<T, W>, dim3((unsigned)n), dim3(kOddThreads), in_shared ? 8 * (size_t)p.H : 0, s, p, part,
                                 in_shared);
  }
  // short rows: from some rows a worker on (304 x 1024 8.5 us straight and 9.7, 1000
  // 19 and 14; longer ones always: 1 x 7168 12 and 8.1)
  if (p.H > 512 && p.H <= 16 * kRingThreads && (p.H > 1024 || p.T > 4 * sms)) {
    const Shape sh = shape_of(p.H, 16);
    const int each = kRingThreads / sh.threads;  // blocks an SM
    RingArrays r{};
    r.T = p.T;
    r.bytes = p.H * z;
    const void* base[kArrays] = {p.dh, p.dn, p.dn ? p.h : nullptr, p.u, full ? p.gate : nullptr};
    const int64_t ld[kArrays] = {p.lddh, p.lddn, p.ldh, p.ldu, p.ldg};
    for (int a = 0; a < kArrays; ++a) r.base[a] = static_cast<const char*>(base[a]), r.ld[a] = ld[a] * z;
    const size_t smem = ring_close(r, 1, each);
    if (r.stages) {
      at_most((int64_t)sms * each);
      switch (p.u && p.dh && p.dn && p.du && p.dresidual ? mode_of(p.post, p.gate_kind) : kAny) {
        case kPlain: return grad_ring<T, W, kPlain>(p, r, part, n, sh.threads, smem, s);
        case kToken: return grad_ring<T, W, kToken>(p, r, part, n, sh.threads, smem, s);
        case kPost: return grad_ring<T, W, kPost>(p, r, part, n, sh.threads, smem, s);
        case kPost + kToken: return grad_ring<T, W, kPost + kToken>(p, r, part, n, sh.threads, smem, s);
        case kPost + kFull: return grad_ring<T, W, kPost + kFull>(p, r, part, n, sh.threads, smem, s);
        default: return grad_ring<T, W, kAny>(p, r, part, n, sh.threads, smem, s);
      }
    }
  }
  const Shape sh = shape_of(p.H, p.H <= 8192 ? 8 : 32);
  const int rows = sh.threads / sh.tpr;
  at_most((int64_t)sms * (1024 / sh.threads) * rows);
  const dim3 grid((unsigned)((n + rows - 1) / rows)), block(sh.threads);
  return p.H <= 1024   ? launch_after_previous(block_norm_grad_kernel<T, W, 1, 128>, grid, block, 0, s, p, sh.tpr, part, (int)n)
         : p.H <= 8192 ? launch_after_previous(block_norm_grad_kernel<T, W, 1, 1024>, grid, block, 0, s, p, sh.tpr, part, (int)n)
                       : launch_after_previous(block_norm_grad_kernel<T, W, 4, 1024>, grid, block, 0, s, p, sh.tpr, part, (int)n);
}

template <typename T, typename W>
cudaError_t grad_tw(const BlockNormGradArgs& p, float* part, int sms, cudaStream_t s) {
  int64_t workers = 0;
  const cudaError_t e = grad_rows<T, W>(p, part, &workers, sms, s);
  ColumnOuts<W> o{};
  const bool channel = p.gate_kind == kGateChannel;
  o.dpost_w = p.dpost_w;
  o.dgate = channel ? static_cast<float*>(p.dgate) : nullptr;
  o.dpre_w = p.dpre_w;
  o.post_w = static_cast<const W*>(p.post_w);
  o.gate = channel ? static_cast<const W*>(p.gate) : nullptr;
  o.first = o.dpost_w || o.dgate ? 1 : 0;
  const int arrays = o.first + (p.dpre_w ? 1 : 0);
  if (e != cudaSuccess || !arrays) return e;
  return launch_after_previous(norm_columns_kernel<W>, dim3((unsigned)((p.H + 31) / 32), arrays), dim3(kColThreads), 0, s, (const float*)part, o,
                               (int)workers, p.H);
}

template <typename T>
cudaError_t norm_t(const BlockNormArgs& p, int wtype, int sms, cudaStream_t s) {
  return wtype == 2 ? norm_tw<T, float>(p, sms, s) : norm_tw<T, T>(p, sms, s);
}
template <typename T>
cudaError_t grad_t(const BlockNormGradArgs& p, int wtype, float* part, int sms, cudaStream_t s) {
  return wtype == 2 ? grad_tw<T, float>(p, part, sms, s) : grad_tw<T, T>(p, part, sms, s);
}

}  // namespace
}  // namespace dfm
