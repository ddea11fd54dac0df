// k_norm.cu — the norms after and before a block, with its gate and the
// residual's scale, and their gradients. With rms(v) = 1 / sqrt(mean(v^2) + eps),
//
//   a = u rms(u) q   (post; else a = u)      u the block's output
//   h = s r + g a                            r the residual stream, g the gate
//   n = h rms(h) v                           the next block's input
//
//   G  = dh + rms(h) (v dn - H (mean over the row of v dn H)),   H = h rms(h)
//   dr = s G,  dg = G a,  dv = sum over the rows of dn H
//   du = rms(u) (q g G - U mean(q g G U)),   U = u rms(u)   (post; else g G)
//   dq = sum over the rows of g G U
//
// A row stays in registers between its sums and its outputs, so that every
// array is read and written once: HBM bounds the large calls. The gradient's
// sums of a row are all linear in G's three terms, so one reduction gives them
// (sum h^2, u^2, v dn h, and u q g times dh, v dn and h); its column sums stay
// in a block's registers over its rows and meet in a second kernel, in order.
// Sums are fp32. A row whose squares overflow fp32 is summed again at 2^-70.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <type_traits>

#include "internal.h"
#include "ops.h"
#include "pipeline.cuh"
#include "tcgen.cuh"

namespace dfm {
namespace {

constexpr float kSmall = 0x1p-70f;  // of rows whose squares overflow

template <typename T>
__device__ __forceinline__ float f32_of(T v);
template <>
__device__ __forceinline__ float f32_of(float v) { return v; }
template <>
__device__ __forceinline__ float f32_of(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float f32_of(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ void unpack_eight(float* v, const uint32_t (&u)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same<T, __half>::value) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      v[2 * i] = f.x, v[2 * i + 1] = f.y;
    } else {
      v[2 * i] = __uint_as_float(u[i] << 16), v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
}
template <typename T>
__device__ __forceinline__ void load_eight(float* v, const T* p, int i) {
  p += i;
  if constexpr (sizeof(T) == 4) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    unpack_eight<T>(v, u);
  }
}
// The same from shared memory, by its 32-bit address (generic addresses cost
// two more instructions a load).
template <typename T>
struct InShared {
  uint32_t at;
};
__device__ __forceinline__ void lds4(uint32_t (&w)[4], uint32_t at) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at));
}
template <typename T>
__device__ __forceinline__ void load_eight(float* v, InShared<T> p, int i) {
  uint32_t w[4];
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int h = 0; h < 8; h += 4) {
      lds4(w, p.at + 4 * (i + h));
#pragma unroll
      for (int j = 0; j < 4; ++j) v[h + j] = __uint_as_float(w[j]);
    }
  } else {
    lds4(w, p.at + 2 * i);
    unpack_eight<T>(v, w);
  }
}
template <typename T>
__device__ __forceinline__ float load_one(InShared<T> p, int i) {
  if constexpr (sizeof(T) == 4) {
    float f;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f) : "r"(p.at + 4 * i));
    return f;
  } else {
    unsigned short w;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(w) : "r"(p.at + 2 * i));
    if constexpr (std::is_same<T, __half>::value) return __half2float(__ushort_as_half(w));
    else return __uint_as_float((uint32_t)w << 16);
  }
}
template <typename T>
__device__ __forceinline__ float load_one(const T* p, int i) { return f32_of<T>(p[i]); }

template <typename T>
__device__ __forceinline__ void store_eight(T* p, const float* v) {
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack16<T>(v[0], v[1]), pack16<T>(v[2], v[3]), pack16<T>(v[4], v[5]), pack16<T>(v[6], v[7]));
  }
}

// A row's values as its threads hold them, in NV parts of eight: VEC: eight
// side by side, parts tpr such groups apart; else one by one, tpr apart. What
// lies behind the row is 0.
template <bool VEC>
struct Row {
  int t, tpr, H;
  __device__ __forceinline__ int col(int i, int j) const { return VEC ? 8 * (t + tpr * i) + j : t + tpr * (8 * i + j); }
  // from a const T* or InShared<T>
  template <typename P>
  __device__ __forceinline__ void load(float (&v)[8], P p, int i) const {
    if (VEC) {
      if (8 * (t + tpr * i) < H) {
        load_eight(v, p, 8 * (t + tpr * i));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.f;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = col(i, j) < H ? load_one(p, col(i, j)) : 0.f;
    }
  }
  template <typename T>
  __device__ __forceinline__ void store(T* p, const float (&v)[8], int i) const {
    if (VEC) {
      if (8 * (t + tpr * i) < H) store_eight(p + 8 * (t + tpr * i), v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (col(i, j) < H) p[col(i, j)] = T(v[j]);
    }
  }
};

// Sums of N values over a row's threads: a warp, or the whole block of `tpr`.
// Up to eight values share the shuffles: at each of three steps a lane keeps
// half of its values and hands the other half over, so that lane l ends with
// value l / 4 (nine shuffles, not forty). Alternating buffers: one barrier a
// sum. The order of the additions is fixed.
template <int N, int WARPS>
struct RowSum {
  static constexpr int S = WARPS == 32 ? 32 : 16;  // warps of a row at most
  float (*buf)[N][S];                              // [2], shared; zero where the row has no warp
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
    if (tpr > 32) {
      if (lane % G == 0) buf[which][lane / G][warp] = mine;
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
// What multiplies a thread's columns in every row: the weights behind the
// norms, `q` with a channel's gate. They stay in registers over a block's rows.
template <typename W, bool VEC, int NV>
__device__ __forceinline__ void load_weights(float (&q)[NV][8], float (&v)[NV][8], const Row<VEC>& at, const void* post_w,
                                             const void* channel, const void* pre_w) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[i][j] = v[i][j] = 1.f;
    if (post_w) at.load(q[i], static_cast<const W*>(post_w), i);
    if (channel) {
      at.load(w, static_cast<const W*>(channel), i);
#pragma unroll
      for (int j = 0; j < 8; ++j) q[i][j] *= w[j];
    }
    if (pre_w) at.load(v[i], static_cast<const W*>(pre_w), i);
  }
}

// sum v^2 over each of R rows, and of what factor the values are where that
// overflows: 1 / sqrt(mean + eps) of the values themselves.
template <int NV, int R, typename Sum>
__device__ __forceinline__ void rms_rows(float (&rms)[R], const float (&v)[R][NV][8], Sum& sum, int tpr, float inv, float eps) {
  float s[R], small[R];
  bool over = false;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    s[r] = 0.f, small[r] = 1.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) s[r] = fmaf(v[r][i][j], v[r][i][j], s[r]);
  }
  sum(s, tpr);
#pragma unroll
  for (int r = 0; r < R; ++r) over = over || !(s[r] < INFINITY);
  if (over) {
    float t[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      t[r] = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) t[r] = fmaf(v[r][i][j] * kSmall, v[r][i][j] * kSmall, t[r]);
    }
    sum(t, tpr);
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (!(s[r] < INFINITY)) s[r] = t[r], small[r] = kSmall;
  }
#pragma unroll
  for (int r = 0; r < R; ++r) rms[r] = rms_of(s[r], inv, eps, small[r]) * small[r];
}

// R rows side by side (their sums share the barriers). in.u(r), in.r(r),
// in.gate(r): where row r's arrays are; there[r]: whether it is one. `poison`
// is 0, or NaN for every output. Every thread of the rows runs this.
template <typename T, bool VEC, int NV, int R, typename In, typename Sum>
__device__ __forceinline__ void norm_rows(const BlockNormArgs& p, const Row<VEC>& at, const In& in, const int64_t (&row)[R],
                                          const bool (&there)[R], Sum& sum, const float (&q)[NV][8], const float (&v)[NV][8],
                                          float inv, float poison) {
  float h[R][NV][8], rms[R];
  if (p.u) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < NV; ++i) at.load(h[r][i], in.u(r), i);
#pragma unroll
    for (int r = 0; r < R; ++r) rms[r] = 1.f;
    if (p.post) rms_rows<NV, R>(rms, h, sum, at.tpr, inv, p.eps);
    if (p.gate_kind == kGateToken)
#pragma unroll
      for (int r = 0; r < R; ++r) rms[r] *= there[r] ? static_cast<const float*>(p.gate)[row[r]] : 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) h[r][i][j] = h[r][i][j] * rms[r] * q[i][j];
        float w[8];
        if (p.gate_kind == kGateFull) {
          at.load(w, in.gate(r), i);
#pragma unroll
          for (int j = 0; j < 8; ++j) h[r][i][j] *= w[j];
        }
        if (p.residual) {
          at.load(w, in.r(r), i);
#pragma unroll
          for (int j = 0; j < 8; ++j) h[r][i][j] = fmaf(p.scale, w[j], h[r][i][j]);
        }
      }
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        at.load(h[r][i], in.r(r), i);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[r][i][j] *= p.scale;
      }
  }
  if (poison != 0.f) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) h[r][i][j] = poison;
  }
  if (p.h) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (there[r])
#pragma unroll
        for (int i = 0; i < NV; ++i) at.store(static_cast<T*>(p.h) + row[r] * p.ldh, h[r][i], i);
  }
  if (!p.n) return;
  rms_rows<NV, R>(rms, h, sum, at.tpr, inv, p.eps);
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (there[r])
#pragma unroll
      for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) h[r][i][j] = h[r][i][j] * rms[r] * v[i][j];
        at.store(static_cast<T*>(p.n) + row[r] * p.ldn, h[r][i], i);
      }
}

// A row's gradients but the weights', whose terms are added to dq and dv:
//   dq += G U (times the token's or the full gate), dv += dn H.
// A channel's gate does not change from row to row: dpost_w is the gate times
// the sum of G U and the gate's gradient post_w times the same sum. `sums_done`
// runs behind the row's sums (whose barrier comes after the last read of an
// earlier row). ok: false in any thread makes the row NaN.
template <typename T, bool VEC, int NV, typename In, typename Sum, typename Done>
__device__ __forceinline__ void grad_row(const BlockNormGradArgs& p, const Row<VEC>& at, const In& in, int64_t row, Sum& sum,
                                         const float (&q)[NV][8], const float (&v)[NV][8], float (&dq)[NV][8], float (&dv)[NV][8],
                                         float inv, bool ok, Done sums_done) {
  const bool full = p.gate_kind == kGateFull;
  float token = p.gate_kind == kGateToken ? static_cast<const float*>(p.gate)[row] : 1.f;
  float sh = 1.f, su = 1.f, s[8];
  // the row's sums: h^2, u^2, h y, and u q g times dh, y and h (y = v dn, g without a token's)
  for (int again = 0;; ++again) {
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = 0.f;
    s[6] = ok ? 0.f : 1.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float h[8], y[8], x[8], w[8];
      if (p.dn) {
        at.load(h, in.h(), i);
        at.load(y, in.dn(), i);
        if (again) {
#pragma unroll
          for (int j = 0; j < 8; ++j) h[j] *= sh;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          y[j] *= v[i][j];
          s[0] = fmaf(h[j], h[j], s[0]);
          s[2] = fmaf(h[j], y[j], s[2]);
        }
      }
      if (!p.u || !(p.post || p.gate_kind == kGateToken)) continue;
      at.load(x, in.u(), i);
      if (again) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= su;
      }
      if (p.post) {
#pragma unroll
        for (int j = 0; j < 8; ++j) s[1] = fmaf(x[j], x[j], s[1]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= q[i][j];
      if (full) {
        at.load(w, in.gate(), i);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= w[j];
      }
      if (p.dh) {
        at.load(w, in.dh(), i);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[3] = fmaf(x[j], w[j], s[3]);
      }
      if (p.dn) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          s[4] = fmaf(x[j], y[j], s[4]);
          s[5] = fmaf(x[j], h[j], s[5]);
        }
      }
    }
    sum(s, at.tpr);
    if (again || (s[0] < INFINITY && s[1] < INFINITY)) break;
    if (!(s[0] < INFINITY)) sh = kSmall;
    if (!(s[1] < INFINITY)) su = kSmall;
  }
  // rms(h sh) = rh: H = h sh rh, rms(h) = sh rh; the same for u
  float rh = p.dn ? rms_of(s[0], inv, p.eps, sh) : 0.f, ru = p.post ? rms_of(s[1], inv, p.eps, su) : 1.f, scale = p.scale;
  if (s[6] != 0.f) rh = ru = token = scale = __uint_as_float(0x7fffffffu);
  const float along = rh * s[2] * inv, turned = along * rh * s[5];
  rh *= sh;
  // the sum over the row of G q g u su, then of q g G U over H
  const float gu = s[3] + rh * (s[4] - turned);
  const float mean = ru * (token * gu) * inv;
  if (p.dgate && p.gate_kind == kGateToken && at.t == 0) static_cast<float*>(p.dgate)[row] = ru * gu;
  ru *= su;
  sums_done();
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float G[8], h[8], y[8];
    if (p.dh) {
      at.load(G, in.dh(), i);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) G[j] = 0.f;
    }
    if (p.dn) {
      at.load(h, in.h(), i);
      at.load(y, in.dn(), i);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[j] *= rh;
        dv[i][j] = fmaf(y[j], h[j], dv[i][j]);
        G[j] = fmaf(rh, fmaf(-h[j], along, y[j] * v[i][j]), G[j]);
      }
    }
    if (p.dresidual) {
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = scale * G[j];
      at.store(static_cast<T*>(p.dresidual) + row * p.lddr, y, i);
    }
    if (!p.u) continue;
    at.load(h, in.u(), i);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] *= ru;  // U, or u
    if (full) {
      if (p.dgate) {  // G a
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = G[j] * (h[j] * q[i][j]);
        at.store(static_cast<T*>(p.dgate) + row * p.lddg, y, i);
      }
      at.load(y, in.gate(), i);
#pragma unroll
      for (int j = 0; j < 8; ++j) G[j] *= y[j];
    }
    if (p.gate_kind == kGateToken) {
#pragma unroll
      for (int j = 0; j < 8; ++j) G[j] *= token;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      dq[i][j] = fmaf(G[j], h[j], dq[i][j]);
      y[j] = q[i][j] * G[j];
    }
    if (p.du) {
      if (p.post) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = ru * fmaf(-h[j], mean, y[j]);
      }
      if (s[6] != 0.f) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = scale;  // NaN
      }
      at.store(static_cast<T*>(p.du) + row * p.lddu, y, i);
    }
  }
}

// The sums of a worker's rows, behind each other: part[array][worker][H].
template <bool VEC, int NV>
__device__ __forceinline__ void put_columns(const BlockNormGradArgs& p, const Row<VEC>& at, float* part, int worker, int workers,
                                            const float (&dq)[NV][8], const float (&dv)[NV][8]) {
  const int64_t array = (int64_t)workers * p.H;
  int k = 0;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if (which == 0 ? !(p.dpost_w || (p.dgate && p.gate_kind == kGateChannel)) : !p.dpre_w) continue;
    float* o = part + array * k++ + (int64_t)worker * p.H;
#pragma unroll
    for (int i = 0; i < NV; ++i) at.store(o, which == 0 ? dq[i] : dv[i], i);
  }
}

// ---- rows straight from global memory ------------------------------------------
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

template <typename T, typename W, bool VEC, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) block_norm_kernel(const BlockNormArgs p, int tpr) {
  __shared__ __align__(16) float buf[2][1][THREADS / 32 > 16 ? 32 : 16];
  const int rows = blockDim.x / tpr, g = threadIdx.x / tpr;
  const int64_t row[1] = {(int64_t)blockIdx.x * rows + g};
  const bool there[1] = {true};
  const Row<VEC> at{(int)threadIdx.x - g * tpr, tpr, p.H};
  RowSum<1, (THREADS / 32 > 16 ? 32 : 16)> sum{buf};
  sum.init();
  __syncthreads();
  pdl_wait();
  if (row[0] >= p.T) return;  // a whole warp: rows == 1 where a row has more
  float q[NV][8], v[NV][8];
  load_weights<W, VEC, NV>(q, v, at, p.post_w, p.gate_kind == kGateChannel ? p.gate : nullptr, p.pre_w);
  norm_rows<T, VEC, NV, 1>(p, at, GlobalRow<T>{p, row[0]}, row, there, sum, q, v, 1.f / (float)p.H, 0.f);
}

template <typename T, typename W, bool VEC, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) block_norm_grad_kernel(const BlockNormGradArgs p, int tpr, float* part, int workers) {
  __shared__ __align__(16) float buf[2][8][THREADS / 32 > 16 ? 32 : 16];
  const int rows = blockDim.x / tpr, g = threadIdx.x / tpr;
  const int worker = blockIdx.x * rows + g;
  const Row<VEC> at{(int)threadIdx.x - g * tpr, tpr, p.H};
  RowSum<8, (THREADS / 32 > 16 ? 32 : 16)> sum{buf};
  sum.init();
  __syncthreads();
  float dq[NV][8] = {}, dv[NV][8] = {}, q[NV][8], v[NV][8];
  const float inv = 1.f / (float)p.H;
  pdl_wait();
  if (worker >= workers) return;  // a whole warp: rows == 1 where a row has more
  load_weights<W, VEC, NV>(q, v, at, p.post_w, p.gate_kind == kGateChannel ? p.gate : nullptr, p.pre_w);
  for (int64_t row = worker; row < p.T; row += workers)
    grad_row<T, VEC, NV>(p, at, GlobalGradRow<T>{p, row}, row, sum, q, v, dq, dv, inv, true, [] {});
  put_columns<VEC, NV>(p, at, part, worker, workers, dq, dv);
}

// ---- rows through shared memory -------------------------------------------------
// Persistent blocks, a row at a time; bulk copies bring the arrays of the next
// rows into a ring of stages meanwhile, so that a row's sums and outputs do not
// stop the stream. Copies start and end on 16-byte boundaries: a row that does
// not is copied from the boundary before it to the one behind it (what lies
// between rows may be read), and starts inside its place. Before the first row
// and behind the last there is nothing that may be read: the bytes up to the
// first boundary and from the last are loaded one by one.
constexpr int kArrays = 5;
struct RingArrays {
  const char* base[kArrays];  // null: absent
  int64_t ld[kArrays];        // bytes
  int64_t T;
  int bytes;       // of a row
  int pitch;       // of an array's place in a stage
  int arrays;      // places
  int stages;
};
struct RingSmem {
  uint64_t full[8];
};

struct Window {
  const char *begin, *end;  // what is copied
  int lead;                 // the row starts this far behind its place's start
};
template <bool VEC>
__device__ __forceinline__ Window ring_window(const RingArrays& r, int a, int64_t row) {
  const char* p = r.base[a] + row * r.ld[a];
  if (VEC) return {p, p + r.bytes, 0};
  const uintptr_t at = (uintptr_t)p, lo = at & ~(uintptr_t)15, hi = (at + r.bytes + 15) & ~(uintptr_t)15;
  const uintptr_t first = ((uintptr_t)r.base[a] + 15) & ~(uintptr_t)15;
  const uintptr_t last = ((uintptr_t)r.base[a] + (r.T - 1) * r.ld[a] + r.bytes) & ~(uintptr_t)15;
  return {(const char*)(lo < first ? first : lo), (const char*)(hi > last ? last : hi), (int)(at & 15)};
}
// One thread: the copies of R rows (those there are) into stage s.
template <bool VEC, int R>
__device__ __forceinline__ void ring_fill(const RingArrays& r, uint8_t* ring, RingSmem* sm, int s, int64_t first) {
  const int rows = (int)min((int64_t)R, r.T - first);
  uint32_t bytes = 0;
  for (int i = 0; i < rows; ++i)
    for (int a = 0; a < kArrays; ++a)
      if (r.base[a]) {
        const Window w = ring_window<VEC>(r, a, first + i);
        bytes += (uint32_t)(w.end - w.begin);
      }
  if (!VEC) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // bytes that threads wrote there
  mbar_arrive_expect_tx(&sm->full[s], bytes);
  const uint64_t once = l2_evict_first_policy();
  for (int i = 0; i < rows; ++i) {
    uint8_t* place = ring + (size_t)(s * R + i) * r.arrays * r.pitch;
    for (int a = 0; a < kArrays; ++a)
      if (r.base[a]) {
        const Window w = ring_window<VEC>(r, a, first + i);
        const char* from = r.base[a] + (first + i) * r.ld[a] - w.lead;  // what the place's first byte is
        bulk_g2s(place + (w.begin - from), w.begin, (uint32_t)(w.end - w.begin), &sm->full[s], once);
        place += r.pitch;
      }
  }
}
// Where array a (the n-th there is) of a row starts, in the place of the i-th
// row of the ring.
template <bool VEC>
__device__ __forceinline__ uint32_t ring_row(const RingArrays& r, int i, int a, int n, int64_t row) {
  return (uint32_t)(i * r.arrays + n) * r.pitch + (VEC ? 0 : (uint32_t)((uintptr_t)(r.base[a] + row * r.ld[a]) & 15));
}
// The first and last row's bytes that no copy brings (all threads, then a barrier).
__device__ __forceinline__ void ring_patch(const RingArrays& r, uint8_t* ring, int i, int64_t row) {
  for (int a = 0, n = 0; a < kArrays; ++a)
    if (r.base[a]) {
      const Window w = ring_window<false>(r, a, row);
      const char* p = r.base[a] + row * r.ld[a];
      uint8_t* to = ring + (size_t)(i * r.arrays + n) * r.pitch + w.lead;
      const int head = (int)(w.begin - p), tail = (int)(p + r.bytes - w.end);
      if ((int)threadIdx.x < head) to[threadIdx.x] = p[threadIdx.x];
      if ((int)threadIdx.x < tail) to[r.bytes - 1 - threadIdx.x] = p[r.bytes - 1 - threadIdx.x];
      ++n;
    }
  __syncthreads();
}

constexpr int kRingThreads = 512;  // 16 values a thread: rows of up to 8192

// Where the arrays of the rows of a stage start.
template <typename T, int R>
struct RingRows {
  uint32_t at[R][kArrays];
  __device__ __forceinline__ InShared<T> get(int r, int a) const { return {at[r][a]}; }
  __device__ __forceinline__ InShared<T> u(int r) const { return get(r, 0); }
  __device__ __forceinline__ InShared<T> r(int r) const { return get(r, 1); }
  __device__ __forceinline__ InShared<T> gate(int r) const { return get(r, 2); }
};
template <typename T>
struct RingGradRow : RingRows<T, 1> {
  __device__ __forceinline__ InShared<T> dh() const { return this->get(0, 0); }
  __device__ __forceinline__ InShared<T> dn() const { return this->get(0, 1); }
  __device__ __forceinline__ InShared<T> h() const { return this->get(0, 2); }
  __device__ __forceinline__ InShared<T> u() const { return this->get(0, 3); }
  __device__ __forceinline__ InShared<T> gate() const { return this->get(0, 4); }
};

// R rows a stage (two of 16 bits: their sums share two barriers).
template <typename T, typename W, bool VEC>
__global__ void __launch_bounds__(kRingThreads, 1) block_norm_ring_kernel(const BlockNormArgs p, const RingArrays r) {
  constexpr int R = sizeof(T) == 2 ? 2 : 1;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ RingSmem sm;
  __shared__ __align__(16) float buf[2][R][16];
  const Row<VEC> at{(int)threadIdx.x, (int)blockDim.x, p.H};
  RowSum<R, 16> sum{buf};
  sum.init();
  const float inv = 1.f / (float)p.H;
  const uint32_t ring0 = smem_u32(ring);
  if (threadIdx.x == 0) {
    for (int i = 0; i < r.stages; ++i) mbar_init(&sm.full[i], 1);
    fence_barrier_init();
  }
  __syncthreads();
  pdl_wait();
  const int64_t step = (int64_t)R * gridDim.x;
  int64_t ahead = (int64_t)R * blockIdx.x;  // the next rows to copy
  if (threadIdx.x == 0)
    for (int i = 0; i < r.stages && ahead < p.T; ++i, ahead += step) ring_fill<VEC, R>(r, ring, &sm, i, ahead);
  float q[2][8], v[2][8];
  load_weights<W, VEC, 2>(q, v, at, p.post_w, p.gate_kind == kGateChannel ? p.gate : nullptr, p.pre_w);
  int s = 0, before = -1;
  uint32_t phase = 0, limit = kWaitLimit;
  for (int64_t first = (int64_t)R * blockIdx.x; first < p.T; first += step) {
    bool ok = mbar_wait(&sm.full[s], phase, limit);
    if (!ok) limit = 1;
    // every thread is past the rows before: their stage takes the next copies
    ok = __syncthreads_and(ok);
    if (threadIdx.x == 0 && before >= 0 && ahead < p.T) {
      ring_fill<VEC, R>(r, ring, &sm, before, ahead);
      ahead += step;
    }
    int64_t row[R];
    bool there[R];
    RingRows<T, R> in;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      there[i] = first + i < p.T;
      row[i] = there[i] ? first + i : first;  // a row that is not there: the one before it, not stored
      if (!VEC && there[i] && (row[i] == 0 || row[i] == p.T - 1)) ring_patch(r, ring, s * R + i, row[i]);
#pragma unroll
      for (int a = 0, n = 0; a < 3; ++a) {
        in.at[i][a] = ring0 + ring_row<VEC>(r, s * R + (there[i] ? i : 0), a, n, row[i]);
        n += r.base[a] != nullptr;
      }
    }
    norm_rows<T, VEC, 2, R>(p, at, in, row, there, sum, q, v, inv, ok ? 0.f : __uint_as_float(0x7fffffffu));
    before = s;
    if (++s == r.stages) {
      s = 0;
      phase ^= 1;
    }
  }
  if (limit == 1)  // a wait ran out: copies in flight land before the block leaves
    for (int i = 0; i < r.stages; ++i) (void)mbar_wait(&sm.full[i], i < s ? phase : phase ^ 1);
}

template <typename T, typename W, bool VEC>
__global__ void __launch_bounds__(kRingThreads, 1) block_norm_grad_ring_kernel(const BlockNormGradArgs p, const RingArrays r, float* part) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ RingSmem sm;
  __shared__ __align__(16) float buf[2][8][16];
  const Row<VEC> at{(int)threadIdx.x, (int)blockDim.x, p.H};
  RowSum<8, 16> sum{buf};
  sum.init();
  const float inv = 1.f / (float)p.H;
  const uint32_t ring0 = smem_u32(ring);
  if (threadIdx.x == 0) {
    for (int i = 0; i < r.stages; ++i) mbar_init(&sm.full[i], 1);
    fence_barrier_init();
  }
  __syncthreads();
  pdl_wait();
  int64_t ahead = blockIdx.x;
  if (threadIdx.x == 0)
    for (int i = 0; i < r.stages && ahead < p.T; ++i, ahead += gridDim.x) ring_fill<VEC, 1>(r, ring, &sm, i, ahead);
  float dq[2][8] = {}, dv[2][8] = {}, q[2][8], v[2][8];
  load_weights<W, VEC, 2>(q, v, at, p.post_w, p.gate_kind == kGateChannel ? p.gate : nullptr, p.pre_w);
  int s = 0, before = -1;
  uint32_t phase = 0, limit = kWaitLimit;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
    const bool ok = mbar_wait(&sm.full[s], phase, limit);
    if (!ok) limit = 1;
    if (!VEC && (row == 0 || row == p.T - 1)) {
      __syncthreads();
      ring_patch(r, ring, s, row);
    }
    RingGradRow<T> in;
#pragma unroll
    for (int a = 0, n = 0; a < kArrays; ++a) {
      in.at[0][a] = ring0 + ring_row<VEC>(r, s, a, n, row);
      n += r.base[a] != nullptr;
    }
    grad_row<T, VEC, 2>(p, at, in, row, sum, q, v, dq, dv, inv, ok, [&] {
      // behind the sums' barrier every thread is past the row before
      if (threadIdx.x == 0 && before >= 0 && ahead < p.T) {
        ring_fill<VEC, 1>(r, ring, &sm, before, ahead);
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
    for (int i = 0; i < r.stages; ++i) (void)mbar_wait(&sm.full[i], i < s ? phase : phase ^ 1);
  put_columns<VEC, 2>(p, at, part, blockIdx.x, gridDim.x, dq, dv);
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

bool vec_rows(const void* p, int64_t ld, int size) { return !(((uintptr_t)p | (uint64_t)(ld * size)) & 15); }

// Threads of a row, rows of a block.
struct Shape {
  int tpr, threads;
};
Shape shape_of(int H, int each) {
  const int tpr = ((H + each - 1) / each + 31) / 32 * 32;
  return {tpr, tpr == 32 ? 128 : tpr};
}

constexpr int kRingBytes = 224 * 1024;  // of a block at most; an SM has 4 KB more, which each block needs beside it

// The ring of a kernel for `blocks` blocks an SM: 0 stages where two do not fit.
RingArrays ring_of(int64_t T, int H, int size, int blocks) {
  RingArrays r{};
  r.T = T;
  r.bytes = H * size;
  r.pitch = (r.bytes + 15 + 15) / 16 * 16 + 16;
  r.stages = (kRingBytes + 4096) / blocks - 4096;  // bytes, until the arrays are known
  return r;
}
void ring_add(RingArrays& r, int a, const void* base, int64_t ld, int size) {
  r.base[a] = static_cast<const char*>(base);
  r.ld[a] = ld * size;
  if (base) ++r.arrays;
}
size_t ring_close(RingArrays& r, int rows) {
  const int stage = rows * r.arrays * r.pitch, n = r.stages / stage;
  r.stages = n < 2 ? 0 : n > 6 ? 6 : n;
  return (size_t)r.stages * stage;
}

template <typename K>
cudaError_t ring_configure(K kernel, std::atomic<uint64_t>& configured) {
  int device = 0;
  (void)cudaGetDevice(&device);
  if (device < 64 && configured.load() >> device & 1) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
  if (e == cudaSuccess && device < 64) configured.fetch_or(1ull << device);
  return e;
}

template <typename T, typename W, bool VEC>
cudaError_t norm_vec(const BlockNormArgs& p, int sms, cudaStream_t s) {
  const int z = sizeof(T);
  if (p.H > 1024 && p.H <= 16 * kRingThreads && p.T > 4 * sms) {
    const Shape sh = shape_of(p.H, 16);
    const int blocks = kRingThreads / sh.threads, rows = z == 2 ? 2 : 1;  // blocks an SM
    RingArrays r = ring_of(p.T, p.H, z, blocks);
    ring_add(r, 0, p.u, p.ldu, z);
    ring_add(r, 1, p.residual, p.ldr, z);
    ring_add(r, 2, p.gate_kind == kGateFull ? p.gate : nullptr, p.ldg, z);
    const size_t smem = ring_close(r, rows);
    if (r.stages) {
      static std::atomic<uint64_t> configured{0};
      const cudaError_t e = ring_configure(block_norm_ring_kernel<T, W, VEC>, configured);
      if (e != cudaSuccess) return e;
      const int64_t most = (int64_t)sms * blocks, steps = (p.T + rows - 1) / rows;
      return launch_after_previous(block_norm_ring_kernel<T, W, VEC>, dim3((unsigned)(steps < most ? steps : most)), dim3(sh.threads), smem, s, p, r);
    }
  }
  const Shape sh = shape_of(p.H, p.H <= 8192 ? 16 : 32);
  const int rows = sh.threads / sh.tpr;
  const dim3 grid((unsigned)((p.T + rows - 1) / rows));
  return p.H <= 8192 ? launch_after_previous(block_norm_kernel<T, W, VEC, 2, 512>, grid, dim3(sh.threads), 0, s, p, sh.tpr)
                     : launch_after_previous(block_norm_kernel<T, W, VEC, 4, 1024>, grid, dim3(sh.threads), 0, s, p, sh.tpr);
}
template <typename T, typename W>
cudaError_t norm_tw(const BlockNormArgs& p, int sms, cudaStream_t s) {
  const int z = sizeof(T);
  const bool vec = p.H % 8 == 0 && vec_rows(p.u, p.u ? p.ldu : 0, z) && vec_rows(p.residual, p.residual ? p.ldr : 0, z) &&
                   vec_rows(p.h, p.h ? p.ldh : 0, z) && vec_rows(p.n, p.n ? p.ldn : 0, z) && vec_rows(p.post_w, 0, 1) &&
                   vec_rows(p.pre_w, 0, 1) &&
                   (p.gate_kind == kGateNone || p.gate_kind == kGateToken || vec_rows(p.gate, p.gate_kind == kGateFull ? p.ldg : 0, z));
  return vec ? norm_vec<T, W, true>(p, sms, s) : norm_vec<T, W, false>(p, sms, s);
}

// Rows that are summed side by side: about 1024 threads an SM of 8 values each,
// 512 of 16, of at most 160 SMs.
int64_t grad_workers(int64_t T, int H) {
  const Shape sh = shape_of(H, H <= 8192 ? 8 : 32);
  const int64_t blocks = 160 * (1024 / sh.threads), rows = sh.threads / sh.tpr;
  return T < blocks * rows ? T : blocks * rows;
}

template <typename T, typename W, bool VEC>
cudaError_t grad_vec(const BlockNormGradArgs& p, float* part, int sms, cudaStream_t s) {
  const int z = sizeof(T);
  int64_t workers = grad_workers(p.T, p.H);
  cudaError_t e = cudaSuccess;
  bool ring = false;
  if (p.H > 1024 && p.H <= 16 * kRingThreads) {
    const Shape sh = shape_of(p.H, 16);
    const int blocks = kRingThreads / sh.threads;  // an SM
    RingArrays r = ring_of(p.T, p.H, z, blocks);
    ring_add(r, 0, p.dh, p.lddh, z);
    ring_add(r, 1, p.dn, p.lddn, z);
    ring_add(r, 2, p.dn ? p.h : nullptr, p.ldh, z);
    ring_add(r, 3, p.u, p.ldu, z);
    ring_add(r, 4, p.gate_kind == kGateFull ? p.gate : nullptr, p.ldg, z);
    const size_t smem = ring_close(r, 1);
    if (r.stages) {
      static std::atomic<uint64_t> configured{0};
      e = ring_configure(block_norm_grad_ring_kernel<T, W, VEC>, configured);
      if (e != cudaSuccess) return e;
      const int64_t most = (int64_t)sms * blocks;
      if (workers > most) workers = most;
      e = launch_after_previous(block_norm_grad_ring_kernel<T, W, VEC>, dim3((unsigned)workers), dim3(sh.threads), smem, s, p, r, part);
      ring = true;
    }
  }
  if (!ring) {
    const Shape sh = shape_of(p.H, p.H <= 8192 ? 8 : 32);
    const int rows = sh.threads / sh.tpr;
    const int64_t most = (int64_t)sms * (1024 / sh.threads) * rows;
    if (workers > most) workers = most;
    const dim3 grid((unsigned)((workers + rows - 1) / rows));
    e = p.H <= 1024   ? launch_after_previous(block_norm_grad_kernel<T, W, VEC, 1, 128>, grid, dim3(sh.threads), 0, s, p, sh.tpr, part, (int)workers)
        : p.H <= 8192 ? launch_after_previous(block_norm_grad_kernel<T, W, VEC, 1, 1024>, grid, dim3(sh.threads), 0, s, p, sh.tpr, part, (int)workers)
                      : launch_after_previous(block_norm_grad_kernel<T, W, VEC, 4, 1024>, grid, dim3(sh.threads), 0, s, p, sh.tpr, part, (int)workers);
  }
  ColumnOuts<W> o{};
  const bool channel = p.gate_kind == kGateChannel;
  o.dpost_w = p.dpost_w;
  o.dgate = channel ? static_cast<float*>(p.dgate) : nullptr;
  o.dpre_w = p.dpre_w;
  o.post_w = static_cast<const W*>(p.post_w);
  o.gate = channel ? static_cast<const W*>(p.gate) : nullptr;
  o.first = o.dpost_w || o.dgate ? 1 : 0;
  const int arrays = o.first + (p.dpre_w ? 1 : 0);
  if (e == cudaSuccess && arrays)
    e = launch_after_previous(norm_columns_kernel<W>, dim3((unsigned)((p.H + 31) / 32), arrays), dim3(kColThreads), 0, s, (const float*)part, o, (int)workers, p.H);
  return e;
}
template <typename T, typename W>
cudaError_t grad_tw(const BlockNormGradArgs& p, float* part, int sms, cudaStream_t s) {
  const int z = sizeof(T);
  const bool vec = p.H % 8 == 0 && vec_rows(p.dh, p.dh ? p.lddh : 0, z) && vec_rows(p.dn, p.dn ? p.lddn : 0, z) &&
                   vec_rows(p.h, p.h ? p.ldh : 0, z) && vec_rows(p.u, p.u ? p.ldu : 0, z) && vec_rows(p.du, p.du ? p.lddu : 0, z) &&
                   vec_rows(p.dresidual, p.dresidual ? p.lddr : 0, z) && vec_rows(p.post_w, 0, 1) && vec_rows(p.pre_w, 0, 1) &&
                   (p.gate_kind == kGateNone || p.gate_kind == kGateToken || vec_rows(p.gate, p.gate_kind == kGateFull ? p.ldg : 0, z)) &&
                   (p.gate_kind != kGateFull || vec_rows(p.dgate, p.dgate ? p.lddg : 0, z));
  return vec ? grad_vec<T, W, true>(p, part, sms, s) : grad_vec<T, W, false>(p, part, sms, s);
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormArgs& p, int dtype, int wtype, int sms, cudaStream_t s) {
  if (dtype == 0) return wtype == 2 ? norm_tw<__nv_bfloat16, float>(p, sms, s) : norm_tw<__nv_bfloat16, __nv_bfloat16>(p, sms, s);
  if (dtype == 1) return wtype == 2 ? norm_tw<__half, float>(p, sms, s) : norm_tw<__half, __half>(p, sms, s);
  return norm_tw<float, float>(p, sms, s);
}

size_t block_norm_grad_workspace_bytes(int64_t T, int H) { return 8 * (size_t)grad_workers(T, H) * (size_t)H; }

cudaError_t launch_block_norm_grad(const BlockNormGradArgs& p, int dtype, int wtype, void* workspace, int sms, cudaStream_t s) {
  float* part = static_cast<float*>(workspace);
  if (dtype == 0)
    return wtype == 2 ? grad_tw<__nv_bfloat16, float>(p, part, sms, s) : grad_tw<__nv_bfloat16, __nv_bfloat16>(p, part, sms, s);
  if (dtype == 1) return wtype == 2 ? grad_tw<__half, float>(p, part, sms, s) : grad_tw<__half, __half>(p, part, sms, s);
  return grad_tw<float, float>(p, part, sms, s);
}

}  // namespace dfm
