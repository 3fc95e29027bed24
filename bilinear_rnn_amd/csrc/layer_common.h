// Device helpers shared by the layer operators.
#pragma once

#include "bf16_tiles.h"
#include "device_common.h"

namespace comba {

// E consecutive elements as float32, at any address that is aligned to the element: the hardware
// takes 8- and 16-byte accesses off their natural alignment. V: all E are there; otherwise `n` of
// them (the rest 0).
template <typename Q> struct __attribute__((packed, aligned(2))) Loose { Q v; };

template <typename T, int E, bool V> struct Pack {
  static constexpr int W = E * sizeof(T) / 4;  // 32-bit words
  typedef uint32_t Words __attribute__((ext_vector_type(W)));
  static __device__ __forceinline__ Words fetch(const T* p, int n) {
    if (V || n == E) return reinterpret_cast<const Loose<Words>*>(p)->v;
    float x[E];
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = i < n ? Elem<T>::load(p, i) : 0.f;
    return words(x);
  }
  static __device__ __forceinline__ void unpack(const Words& w, float (&x)[E]) {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      if constexpr (sizeof(T) == 2) x[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
      else x[i] = __uint_as_float(w[i]);
    }
  }
  static __device__ __forceinline__ void load(const T* p, float (&x)[E], int n) { unpack(fetch(p, n), x); }
  static __device__ __forceinline__ Words words(const float (&x)[E]) {
    Words w;
    if constexpr (sizeof(T) == 2) {
      typedef __bf16 Half __attribute__((ext_vector_type(E)));
      Half h;
#pragma unroll
      for (int i = 0; i < E; ++i) h[i] = to_bf16(x[i]);
      w = __builtin_bit_cast(Words, h);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) w[i] = __float_as_uint(x[i]);
    }
    return w;
  }
  // STREAM: past the caches, for outputs that are written once and not read here.
  template <bool STREAM = false>
  static __device__ __forceinline__ void store(T* p, const float (&x)[E], int n) {
    if (V || n == E) {
      if constexpr (STREAM && W * 4 <= 16) {
        __builtin_nontemporal_store(words(x), &reinterpret_cast<Loose<Words>*>(p)->v);
      } else {
        reinterpret_cast<Loose<Words>*>(p)->v = words(x);
      }
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (i < n) Elem<T>::store(p, i, x[i]);
    }
  }
};

// A range of memory read and written through a buffer resource: loads past its end give 0, stores
// past its end are dropped, so that the ends of a tensor need no branches. Offsets are 32-bit byte
// offsets; kNowhere is past every end.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
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
  __device__ __forceinline__ u32x4 load16(uint32_t off) const { return __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0); }
  // Not kept in the caches on its way out (bit 1: nontemporal): a stream of outputs then leaves the
  // lines of the inputs alone.
  __device__ __forceinline__ void store16(uint32_t off, u32x4 v) const {
    __builtin_amdgcn_raw_buffer_store_b128(v, r, off, 0, 2);
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

// 1 / (1 + e^-x) from the hardware exponential and reciprocal (about 1 ulp, 2 2^-24, each). The
// exponential's argument, x log2(e), is rounded to float32 with the constant's own 0.2 2^-24, which
// e^-x shows as 1.3 |x| 2^-24: the relative error is up to (5 + 1.3 |x|) 2^-24 for negative x (31 2^-24 at
// -20) and 6 2^-24 for positive x, where e^-x is small beside the 1. Below the rounding of a bf16 result
// over the whole range, above that of a float32 one. e^-x overflows to infinity for x < -88, where
// the result is 0 instead of something below 6e-39.
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
