// Device helpers shared by the layer operators.
#pragma once

#include "device_common.h"

namespace comba {

// E consecutive elements as float32. V: the 16-byte path (16-byte aligned address, all E
// present); otherwise element by element, `n` of them (the rest 0).
template <typename T, int E, bool V> struct Pack;

template <int E> struct Pack<u16, E, true> {
  static_assert(E == 8, "16 bytes");
  __device__ static void load(const u16* p, float (&x)[E], int) {
    const uint4 t = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ static void store(u16* p, const float (&x)[E], int) {
    bf16x8 v;
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = to_bf16(x[i]);
    *reinterpret_cast<bf16x8*>(p) = v;
  }
};

template <int E> struct Pack<float, E, true> {
  static_assert(E % 4 == 0, "16-byte pieces");
  __device__ static void load(const float* p, float (&x)[E], int) {
#pragma unroll
    for (int i = 0; i < E; i += 4) {
      const f32x4 t = *reinterpret_cast<const f32x4*>(p + i);
      x[i] = t[0]; x[i + 1] = t[1]; x[i + 2] = t[2]; x[i + 3] = t[3];
    }
  }
  __device__ static void store(float* p, const float (&x)[E], int) {
#pragma unroll
    for (int i = 0; i < E; i += 4) *reinterpret_cast<f32x4*>(p + i) = f32x4{x[i], x[i + 1], x[i + 2], x[i + 3]};
  }
};

template <typename T, int E> struct Pack<T, E, false> {
  __device__ static void load(const T* p, float (&x)[E], int n) {
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = i < n ? Elem<T>::load(p, i) : 0.f;
  }
  __device__ static void store(T* p, const float (&x)[E], int n) {
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (i < n) Elem<T>::store(p, i, x[i]);
  }
};

constexpr float kLog2E = 1.44269504088896340736f;

// 1 / (1 + e^-x) from the hardware exponential and reciprocal (about 1 ulp each): relative
// error a few 2^-24, far below the rounding of a bf16 result and within float32's own.
// e^-x overflows to infinity for x < -88, where the result is 0, as it should be to float32.
__device__ __forceinline__ float sigmoid_fast(float x) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2E * x));
}

// Clamped bounds [t0, t1) of packed sequence n (see sequence_range); n < N.
__device__ __forceinline__ void packed_range(const int32_t* cu, int n, int T, int& t0, int& t1) {
  int b;
  sequence_range(cu, n, T, b, t0, t1);
}

// The last sequence that starts at or before token t (0 if none does): for t inside the batch
// the one that owns it, since empty sequences before it start at the same place.
__device__ __forceinline__ int find_sequence(const int32_t* cu, int N, int t) {
  int lo = 0, hi = N - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

}  // namespace comba
