// A row's two segments of rotated values: loads, stores and the rotation itself.
#pragma once
#include <cstdint>

namespace saf3r {

// N values of a row in a segment that is aligned to their size.
template <typename T, int N>
struct Segment {
  uint32_t w[N * sizeof(T) / 4];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (sizeof(w) == 8) {
      const uint2 x = *reinterpret_cast<const uint2*>(p);
      w[0] = x.x; w[1] = x.y;
    } else {
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(w) / 16); ++i) {
        const uint4 x = reinterpret_cast<const uint4*>(p)[i];
        w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
      }
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (sizeof(w) == 8) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(w) / 16); ++i)
        reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    return __uint_as_float((i & 1) ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
  }
  __device__ __forceinline__ void set2(int i, float a, float b) {  // values i (even) and i + 1
    if constexpr (sizeof(T) == 4) {
      w[i] = __float_as_uint(a);
      w[i + 1] = __float_as_uint(b);
    } else {
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i >> 1]) : "f"(b), "f"(a));
    }
  }
};

// The segments' values.
template <typename T, typename V, int N>
__device__ __forceinline__ void spread(const Segment<T, N>& u, const Segment<T, N>& w, V (&a)[N], V (&b)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    a[i] = u.get(i);
    b[i] = w.get(i);
  }
}

// A value as it is, or from 64 bits to fp32 to odd: cut off, with the last bit set where that was not exact.  It lies on the
// value's side of every border between two codes of fewer bits; rounded to nearest it could fall on the border itself and
// from there, a tie, to the wrong side.
template <typename V, typename T>
__device__ __forceinline__ V narrow(T x) {
  if constexpr (sizeof(T) == sizeof(V)) {
    return x;
  } else {
    const float f = __double2float_rz(x);
    return static_cast<double>(f) == x ? f : __uint_as_float(__float_as_uint(f) | 1u);
  }
}

// Turns the segments' N pairs: (a[i], b[i]), or neighbours inside each segment.  T: what the products are held in, V: the
// values.
template <typename V, typename T>
__device__ __forceinline__ void turn_pair(V& a, V& b, T s, T c) {
  const T x = a, y = b;
  a = narrow<V>(x * c - y * s);
  b = narrow<V>(x * s + y * c);
}
template <typename V, typename T, int N>
__device__ __forceinline__ void turn(V (&a)[N], V (&b)[N], const T (&s)[N], const T (&c)[N], bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      turn_pair(a[2 * i], a[2 * i + 1], s[i], c[i]);
      turn_pair(b[2 * i], b[2 * i + 1], s[N / 2 + i], c[N / 2 + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) turn_pair(a[i], b[i], s[i], c[i]);
  }
}

}  // namespace saf3r
