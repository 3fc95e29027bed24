// Device helpers shared by the layer operators.
#pragma once

#include "bf16_tiles.h"
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

// A range of memory read and written through a buffer resource: loads past its end give 0, stores
// past its end are dropped, so that the ends of a tensor need no branches. Offsets are 32-bit byte
// offsets; kNowhere is past every end.
constexpr uint32_t kNowhere = 0x80000000u;
template <typename T> struct Range {
  __amdgpu_buffer_rsrc_t r;
  __device__ __forceinline__ Range(const T* base, int64_t bytes)
      : r(__builtin_amdgcn_make_buffer_rsrc(uniform_ptr(const_cast<T*>(base)), static_cast<short>(0),
                                            __builtin_amdgcn_readfirstlane(static_cast<int>(bytes)), kBufferWord3)) {}
  // The element's bits; value() makes them a float.
  __device__ __forceinline__ uint32_t load(uint32_t off) const {
    if constexpr (sizeof(T) == 2) return __builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0);
    else return __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
  }
  static __device__ __forceinline__ float value(uint32_t bits) { return __uint_as_float(sizeof(T) == 2 ? bits << 16 : bits); }
  __device__ __forceinline__ void store(uint32_t off, float x) const {
    if constexpr (sizeof(T) == 2) __builtin_amdgcn_raw_buffer_store_b16(float_to_bf16_bits(x), r, off, 0, 0);
    else __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x), r, off, 0, 0);
  }
};

// Keeps x where it is computed: the compiler neither moves its computation below this point nor
// turns a selection of it into a branch. No instruction.
__device__ __forceinline__ void pin(float& x) { asm volatile("" : "+v"(x)); }

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
