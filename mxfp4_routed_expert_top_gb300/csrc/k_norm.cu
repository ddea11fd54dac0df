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

#include <cstring>

#include "internal.h"
#include "ops.h"
#include "pipeline.cuh"

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
__device__ __forceinline__ void load_eight(float* v, const T* p) {
  T e[8];
  uint4 w[sizeof(T) / 2];
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
  memcpy(e, w, sizeof e);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = f32_of<T>(e[j]);
}
template <typename T>
__device__ __forceinline__ void store_eight(T* p, const float* v) {
  T e[8];
  uint4 w[sizeof(T) / 2];
#pragma unroll
  for (int j = 0; j < 8; ++j) e[j] = T(v[j]);
  memcpy(w, e, sizeof e);
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = w[i];
}

// A row's values as its threads hold them: VEC: eight side by side, tpr such
// groups apart; else one by one, tpr apart. What lies behind the row is 0.
template <bool VEC, int NV>
struct Row {
  int t, tpr, H;
  template <typename T>
  __device__ __forceinline__ void load(float (&v)[8 * NV], const T* p) const {
    if (VEC) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = 8 * (t + tpr * i);
        if (c < H) {
          load_eight(v + 8 * i, p + c);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[8 * i + j] = 0.f;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8 * NV; ++i) v[i] = t + tpr * i < H ? f32_of<T>(p[t + tpr * i]) : 0.f;
    }
  }
  template <typename T>
  __device__ __forceinline__ void store(T* p, const float (&v)[8 * NV]) const {
    if (VEC) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (8 * (t + tpr * i) < H) store_eight(p + 8 * (t + tpr * i), v + 8 * i);
    } else {
#pragma unroll
      for (int i = 0; i < 8 * NV; ++i)
        if (t + tpr * i < H) p[t + tpr * i] = T(v[i]);
    }
  }
};

// Sums over a row's threads: a warp, or the whole block. Alternating buffers,
// so that one barrier a sum is enough.
template <int N>
struct RowSum {
  float (*buf)[N][32];  // [2], shared
  int which = 0;
  __device__ __forceinline__ void operator()(float (&s)[N], int tpr) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int o = 16; o; o >>= 1) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
    if (tpr == 32) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = tpr >> 5;
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) buf[which][i][warp] = s[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      s[i] = lane < warps ? buf[which][i][lane] : 0.f;
#pragma unroll
      for (int o = 16; o; o >>= 1) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
    }
    which ^= 1;
  }
};

// 1 / sqrt(mean + eps), of values that were scaled by `small` (and is then of
// those too).
__device__ __forceinline__ float rms_of(float sum, int H, float eps, float small) {
  return __frsqrt_rn(sum / (float)H + eps * small * small);
}

template <typename T, typename W, bool VEC, int NV>
__global__ void __launch_bounds__(1024) block_norm_kernel(const BlockNormArgs p, int tpr) {
  __shared__ float buf[2][1][32];
  constexpr int E = 8 * NV;
  const int rows = blockDim.x / tpr, g = threadIdx.x / tpr;
  const int64_t row = (int64_t)blockIdx.x * rows + g;
  const Row<VEC, NV> at{(int)threadIdx.x - g * tpr, tpr, p.H};
  RowSum<1> sum{buf};
  pdl_wait();
  if (row >= p.T) return;  // a whole warp: rows == 1 where a row has more
  float a[E], h[E], w[E];
  if (p.u) at.load(a, static_cast<const T*>(p.u) + row * p.ldu);
  if (p.residual) at.load(h, static_cast<const T*>(p.residual) + row * p.ldr);
  if (p.u) {
    float scale = 1.f;
    if (p.post) {
      float s[1] = {0.f}, small = 1.f;
#pragma unroll
      for (int i = 0; i < E; ++i) s[0] = fmaf(a[i], a[i], s[0]);
      sum(s, tpr);
      if (!(s[0] < INFINITY)) {
        small = kSmall;
        s[0] = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) s[0] = fmaf(a[i] * small, a[i] * small, s[0]);
        sum(s, tpr);
      }
      const float rms = rms_of(s[0], p.H, p.eps, small);
#pragma unroll
      for (int i = 0; i < E; ++i) a[i] = a[i] * small * rms;
      if (p.post_w) {
        at.load(w, static_cast<const W*>(p.post_w));
#pragma unroll
        for (int i = 0; i < E; ++i) a[i] *= w[i];
      }
    }
    if (p.gate_kind == kGateToken) {
      scale = static_cast<const float*>(p.gate)[row];
#pragma unroll
      for (int i = 0; i < E; ++i) a[i] *= scale;
    } else if (p.gate_kind != kGateNone) {
      if (p.gate_kind == kGateChannel) at.load(w, static_cast<const W*>(p.gate));
      else at.load(w, static_cast<const T*>(p.gate) + row * p.ldg);
#pragma unroll
      for (int i = 0; i < E; ++i) a[i] *= w[i];
    }
  }
#pragma unroll
  for (int i = 0; i < E; ++i)
    h[i] = p.residual ? (p.u ? fmaf(p.scale, h[i], a[i]) : p.scale * h[i]) : a[i];
  if (p.h) at.store(static_cast<T*>(p.h) + row * p.ldh, h);
  if (!p.n) return;
  float s[1] = {0.f}, small = 1.f;
#pragma unroll
  for (int i = 0; i < E; ++i) s[0] = fmaf(h[i], h[i], s[0]);
  sum(s, tpr);
  if (!(s[0] < INFINITY)) {
    small = kSmall;
    s[0] = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) s[0] = fmaf(h[i] * small, h[i] * small, s[0]);
    sum(s, tpr);
  }
  const float rms = rms_of(s[0], p.H, p.eps, small);
#pragma unroll
  for (int i = 0; i < E; ++i) h[i] = h[i] * small * rms;
  if (p.pre_w) {
    at.load(w, static_cast<const W*>(p.pre_w));
#pragma unroll
    for (int i = 0; i < E; ++i) h[i] *= w[i];
  }
  at.store(static_cast<T*>(p.n) + row * p.ldn, h);
}

// Rows of a block, one after the other (blockDim.x / tpr at a time): the column
// sums stay in registers and go to part[array][worker][H].
template <typename T, typename W, bool VEC, int NV>
__global__ void __launch_bounds__(1024) block_norm_grad_kernel(const BlockNormGradArgs p, int tpr, float* part, int workers) {
  __shared__ float buf[2][6][32];
  constexpr int E = 8 * NV;
  const int rows = blockDim.x / tpr, g = threadIdx.x / tpr;
  const int worker = blockIdx.x * rows + g;
  const Row<VEC, NV> at{(int)threadIdx.x - g * tpr, tpr, p.H};
  RowSum<6> sum{buf};
  float dq[E], dv[E], dg[E];
#pragma unroll
  for (int i = 0; i < E; ++i) dq[i] = dv[i] = dg[i] = 0.f;
  pdl_wait();
  if (worker >= workers) return;  // a whole warp: rows == 1 where a row has more
  const float inv = 1.f / (float)p.H;
  for (int64_t row = worker; row < p.T; row += workers) {
    float h[E], y[E], G[E], u[E], q[E], w[E];  // y = v dn; q: the weights and gate of u but the token's
#pragma unroll
    for (int i = 0; i < E; ++i) h[i] = y[i] = G[i] = u[i] = 0.f, q[i] = 1.f;
    if (p.dn) {
      at.load(h, static_cast<const T*>(p.h) + row * p.ldh);
      at.load(y, static_cast<const T*>(p.dn) + row * p.lddn);
    }
    if (p.dh) at.load(G, static_cast<const T*>(p.dh) + row * p.lddh);
    if (p.u) at.load(u, static_cast<const T*>(p.u) + row * p.ldu);
    const float token = p.gate_kind == kGateToken ? static_cast<const float*>(p.gate)[row] : 1.f;
    if (p.post && p.post_w) at.load(q, static_cast<const W*>(p.post_w));
    if (p.gate_kind == kGateChannel || p.gate_kind == kGateFull) {
      if (p.gate_kind == kGateChannel) at.load(w, static_cast<const W*>(p.gate));
      else at.load(w, static_cast<const T*>(p.gate) + row * p.ldg);
#pragma unroll
      for (int i = 0; i < E; ++i) q[i] *= w[i];
    }
    if (p.pre_w) at.load(w, static_cast<const W*>(p.pre_w));
    float sh = 1.f, su = 1.f, s[6];
    for (int again = 0;; ++again) {
#pragma unroll
      for (int i = 0; i < 6; ++i) s[i] = 0.f;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float hs = h[i] * sh, us = u[i] * su, yw = p.pre_w ? y[i] * w[i] : y[i], uq = us * q[i];
        s[0] = fmaf(hs, hs, s[0]);
        s[1] = fmaf(us, us, s[1]);
        s[2] = fmaf(hs, yw, s[2]);
        s[3] = fmaf(uq, G[i], s[3]);
        s[4] = fmaf(uq, yw, s[4]);
        s[5] = fmaf(uq, hs, s[5]);
      }
      sum(s, tpr);
      if (again || (s[0] < INFINITY && (!p.post || s[1] < INFINITY))) break;
      if (!(s[0] < INFINITY)) sh = kSmall;
      if (p.post && !(s[1] < INFINITY)) su = kSmall;
    }
    // rms(h sh): H = h sh rh, rms(h) = sh rh; the same for u
    const float rh = p.dn ? rms_of(s[0], p.H, p.eps, sh) : 0.f, along = rh * s[2] * inv;
    const float ru = p.post ? rms_of(s[1], p.H, p.eps, su) : 1.f;
    // the sum over the row of G q u su
    const float gu = s[3] + rh * sh * (s[4] - along * rh * s[5]);
    const float mean = ru * (token * gu) * inv;
    float out[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float hat = h[i] * sh * rh;
      if (p.dn) {
        dv[i] = fmaf(y[i], hat, dv[i]);
        G[i] = fmaf(rh * sh, (p.pre_w ? y[i] * w[i] : y[i]) - hat * along, G[i]);
      }
      out[i] = p.scale * G[i];
    }
    if (p.dresidual) at.store(static_cast<T*>(p.dresidual) + row * p.lddr, out);
    if (!p.u) continue;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float hat = u[i] * su * ru;
      out[i] = p.post ? ru * su * (token * q[i] * G[i] - hat * mean) : token * q[i] * G[i];
    }
    if (p.du) at.store(static_cast<T*>(p.du) + row * p.lddu, out);
    if (p.dgate && p.gate_kind == kGateToken && at.t == 0) static_cast<float*>(p.dgate)[row] = ru * gu;
    // dq: G gate U; dg: G a. q holds both factors: taken apart again
    const bool channel = p.gate_kind == kGateChannel || p.gate_kind == kGateFull;
    float gate[E];
    if (channel) {
      if (p.gate_kind == kGateChannel) at.load(gate, static_cast<const W*>(p.gate));
      else at.load(gate, static_cast<const T*>(p.gate) + row * p.ldg);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) gate[i] = token;
    }
    if (p.dpost_w) {
#pragma unroll
      for (int i = 0; i < E; ++i) dq[i] = fmaf(gate[i] * G[i], u[i] * su * ru, dq[i]);
    }
    if (p.dgate && channel) {
      if (p.post && p.post_w) {
        at.load(w, static_cast<const W*>(p.post_w));
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) w[i] = 1.f;
      }
#pragma unroll
      for (int i = 0; i < E; ++i) {
        out[i] = G[i] * (u[i] * su * ru * w[i]);
        dg[i] += out[i];
      }
      if (p.gate_kind == kGateFull) at.store(static_cast<T*>(p.dgate) + row * p.lddg, out);
    }
  }
  const int64_t array = (int64_t)workers * p.H;
  int k = 0;
  for (int which = 0; which < 3; ++which) {
    const bool wanted = which == 0 ? p.dpost_w != nullptr : which == 1 ? p.dpre_w != nullptr : p.dgate && p.gate_kind == kGateChannel;
    if (!wanted) continue;
    float* o = part + array * k++ + (int64_t)worker * p.H;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int c = VEC ? 8 * (at.t + tpr * (i / 8)) + i % 8 : at.t + tpr * i;
      if (c < p.H) o[c] = which == 0 ? dq[i] : which == 1 ? dv[i] : dg[i];
    }
  }
}

// out[array][c] = the sum over the workers of part[array][worker][c], in order
// of 32 interleaved parts.
struct ColumnOuts {
  float* out[3];
};
__global__ void __launch_bounds__(1024) norm_columns_kernel(const float* part, const ColumnOuts outs, int workers, int H) {
  __shared__ float sums[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  const float* in = part + (int64_t)blockIdx.y * workers * H;
  pdl_wait();
  float s = 0.f;
  if (c < H)
#pragma unroll 4
    for (int w = warp; w < workers; w += 32) s += in[(int64_t)w * H + c];
  sums[warp][lane] = s;
  __syncthreads();
  if (warp) return;
  s = 0.f;
#pragma unroll
  for (int w = 0; w < 32; ++w) s += sums[w][lane];
  if (c < H) outs.out[blockIdx.y][c] = s;
}

bool vec_rows(const void* p, int64_t ld, int size) { return !(((uintptr_t)p | (uint64_t)(ld * size)) & 15); }

// Threads of a row, rows of a block.
struct Shape {
  int tpr, threads;
};
Shape shape_of(int H, int each) {
  const int tpr = ((H + each - 1) / each + 31) / 32 * 32;
  return {tpr, tpr == 32 ? 256 : tpr};
}

template <typename T, typename W, bool VEC>
cudaError_t norm_vec(const BlockNormArgs& p, cudaStream_t s) {
  const Shape sh = shape_of(p.H, p.H <= 16384 ? 16 : 32);
  const int rows = sh.threads / sh.tpr;
  const dim3 grid((unsigned)((p.T + rows - 1) / rows));
  return p.H <= 16384 ? launch_after_previous(block_norm_kernel<T, W, VEC, 2>, grid, dim3(sh.threads), 0, s, p, sh.tpr)
                      : launch_after_previous(block_norm_kernel<T, W, VEC, 4>, grid, dim3(sh.threads), 0, s, p, sh.tpr);
}
template <typename T, typename W>
cudaError_t norm_tw(const BlockNormArgs& p, cudaStream_t s) {
  const int z = sizeof(T);
  const bool vec = p.H % 8 == 0 && vec_rows(p.u, p.u ? p.ldu : 0, z) && vec_rows(p.residual, p.residual ? p.ldr : 0, z) &&
                   vec_rows(p.h, p.h ? p.ldh : 0, z) && vec_rows(p.n, p.n ? p.ldn : 0, z) && vec_rows(p.post_w, 0, 1) &&
                   vec_rows(p.pre_w, 0, 1) &&
                   (p.gate_kind == kGateNone || p.gate_kind == kGateToken || vec_rows(p.gate, p.gate_kind == kGateFull ? p.ldg : 0, z));
  return vec ? norm_vec<T, W, true>(p, s) : norm_vec<T, W, false>(p, s);
}

int grad_each(int H) { return H <= 8192 ? 8 : H <= 16384 ? 16 : 32; }
// Rows that are summed side by side: about 1024 threads an SM, of at most 160.
int64_t grad_workers(int64_t T, int H) {
  const Shape sh = shape_of(H, grad_each(H));
  const int64_t blocks = 160 * (1024 / sh.threads), rows = sh.threads / sh.tpr;
  return T < blocks * rows ? T : blocks * rows;
}

template <typename T, typename W, bool VEC>
cudaError_t grad_vec(const BlockNormGradArgs& p, float* part, int sms, cudaStream_t s) {
  const Shape sh = shape_of(p.H, grad_each(p.H));
  const int rows = sh.threads / sh.tpr;
  int64_t workers = grad_workers(p.T, p.H);
  const int64_t most = (int64_t)sms * (1024 / sh.threads) * rows;
  if (workers > most) workers = most;
  const dim3 grid((unsigned)((workers + rows - 1) / rows));
  const int w = (int)workers;
  cudaError_t e = p.H <= 8192    ? launch_after_previous(block_norm_grad_kernel<T, W, VEC, 1>, grid, dim3(sh.threads), 0, s, p, sh.tpr, part, w)
                  : p.H <= 16384 ? launch_after_previous(block_norm_grad_kernel<T, W, VEC, 2>, grid, dim3(sh.threads), 0, s, p, sh.tpr, part, w)
                                 : launch_after_previous(block_norm_grad_kernel<T, W, VEC, 4>, grid, dim3(sh.threads), 0, s, p, sh.tpr, part, w);
  ColumnOuts outs{};
  int n = 0;
  if (p.dpost_w) outs.out[n++] = p.dpost_w;
  if (p.dpre_w) outs.out[n++] = p.dpre_w;
  if (p.dgate && p.gate_kind == kGateChannel) outs.out[n++] = static_cast<float*>(p.dgate);
  if (e == cudaSuccess && n)
    e = launch_after_previous(norm_columns_kernel, dim3((unsigned)((p.H + 31) / 32), n), dim3(1024), 0, s, (const float*)part, outs, w, p.H);
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

cudaError_t launch_block_norm(const BlockNormArgs& p, int dtype, int wtype, cudaStream_t s) {
  if (dtype == 0) return wtype == 2 ? norm_tw<__nv_bfloat16, float>(p, s) : norm_tw<__nv_bfloat16, __nv_bfloat16>(p, s);
  if (dtype == 1) return wtype == 2 ? norm_tw<__half, float>(p, s) : norm_tw<__half, __half>(p, s);
  return norm_tw<float, float>(p, s);
}

size_t block_norm_grad_workspace_bytes(int64_t T, int H) { return 12 * (size_t)grad_workers(T, H) * (size_t)H; }

cudaError_t launch_block_norm_grad(const BlockNormGradArgs& p, int dtype, int wtype, void* workspace, int sms, cudaStream_t s) {
  float* part = static_cast<float*>(workspace);
  if (dtype == 0)
    return wtype == 2 ? grad_tw<__nv_bfloat16, float>(p, part, sms, s) : grad_tw<__nv_bfloat16, __nv_bfloat16>(p, part, sms, s);
  if (dtype == 1) return wtype == 2 ? grad_tw<__half, float>(p, part, sms, s) : grad_tw<__half, __half>(p, part, sms, s);
  return grad_tw<float, float>(p, part, sms, s);
}

}  // namespace dfm
