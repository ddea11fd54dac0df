// rowword.h — words of four values of arrays whose rows are not aligned to
// them. A word may hold values between two rows, or of the next one; nothing
// outside the array is read, whose neighbours belong to someone else.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define DFM_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define DFM_HOST_DEVICE inline
#endif

namespace dfm {

template <typename E>
struct alignas(4 * sizeof(E)) Four {
  E v[4];
};

// How an array is read: four values that are aligned in memory, or one.
template <typename E>
struct ArrayOf {
  const E* p;
  DFM_HOST_DEVICE Four<E> four(int64_t i) const { return *reinterpret_cast<const Four<E>*>(p + i); }
  DFM_HOST_DEVICE E one(int64_t i) const { return p[i]; }
};

// Values i .. i + 3 of an array of n, where value i is aligned to four: those
// outside [0, n) are zero.
template <typename E, typename Array>
DFM_HOST_DEVICE Four<E> array_four(const Array& a, int64_t i, int64_t n) {
  if (i >= 0 && i + 4 <= n) return a.four(i);
  Four<E> r{};
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (i + u >= 0 && i + u < n) r.v[u] = a.one(i + u);
  return r;
}

}  // namespace dfm
