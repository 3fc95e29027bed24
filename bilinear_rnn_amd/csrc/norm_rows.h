// Rows held in registers by a part of a wavefront, a wavefront or a workgroup: shared by the block norms and
// the group norm of single tokens.
#pragma once

#include "layer_common.h"

namespace comba {

constexpr int kNormThreads = 256;

// Sum over the LPR lanes that share a row, in every one of them. `red`: LDS of one float per
// wavefront of the workgroup and value; the caller alternates between two such arrays, so that one barrier per
// reduction is enough.
template <int LPR, int K>
__device__ __forceinline__ void row_sums(float (&v)[K], float* red) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float x = v[k];
    x += dpp_flip<0>(x);
    x += dpp_flip<1>(x);
    x += dpp_flip<2>(x);
    if constexpr (LPR >= 16) x += dpp_flip<3>(x);
    if constexpr (LPR >= 32) {  // both halves of the pair of rows, then of the wavefront
      const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
      x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    if constexpr (LPR >= 64) {
      const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
      x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    v[k] = x;
  }
  if constexpr (LPR > 64) {
    constexpr int NW = LPR / 64;
    const int w = threadIdx.x % LPR / kWave;
    red += threadIdx.x / LPR * (K * NW);
    if ((threadIdx.x & (kWave - 1)) == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) red[k * NW + w] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < NW; ++i) s += red[k * NW + i];
      v[k] = s;
    }
  }
}

struct NormShape {
  int64_t rows;
  int D;
  float eps, inv;  // inv = 1 / D
};

// A lane's 8 elements number j of a row, in such columns that a load instruction reads neighbouring
// elements. V: one 16-byte piece of bf16 or two of float32, the second one LPR pieces behind the first
// (8192 rows of 2048 in fp32, gated norm: 37 -> 31.5 us against the two side by side); otherwise single elements,
// LPR apart.
template <typename T, bool V, int LPR> struct Eight {
  static constexpr int P = V ? 16 / sizeof(T) : 1;  // elements of a piece
  static __device__ __forceinline__ int col(int l, int j, int i) { return 8 * j * LPR + (i / P * LPR + l) * P + i % P; }
  uint32_t raw[V && sizeof(T) == 2 ? 4 : 8];
  // `at`: byte offset of the row in the range. Columns behind the row's end are read as 0.
  __device__ __forceinline__ void load(const Range<T>& m, uint32_t at, int l, int j, int D) {
    if constexpr (V) {
#pragma unroll
      for (int k = 0; k < sizeof(raw) / 16; ++k) {
        const u32x4 v = m.load16(col(l, j, k * P) < D ? at + col(l, j, k * P) * sizeof(T) : kNowhere);
#pragma unroll
        for (int i = 0; i < 4; ++i) raw[4 * k + i] = v[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) raw[i] = m.load(col(l, j, i) < D ? at + col(l, j, i) * sizeof(T) : kNowhere);
    }
  }
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (V && sizeof(T) == 2) return __uint_as_float(i & 1 ? raw[i / 2] & 0xffff0000u : raw[i / 2] << 16);
    else return Range<T>::value(raw[i]);
  }
  static __device__ __forceinline__ void store(const Range<T>& m, uint32_t at, int l, int j, int D, const float (&x)[8]) {
    if constexpr (V) {
      auto o = [&](int k) { return col(l, j, k * P) < D ? at + col(l, j, k * P) * static_cast<uint32_t>(sizeof(T)) : kNowhere; };
      if constexpr (sizeof(T) == 2) {
        bf16x8 v;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_bf16(x[i]);
        m.store16(o(0), __builtin_bit_cast(u32x4, v));
      } else {
        m.store16(o(0), __builtin_bit_cast(u32x4, f32x4{x[0], x[1], x[2], x[3]}));
        m.store16(o(1), __builtin_bit_cast(u32x4, f32x4{x[4], x[5], x[6], x[7]}));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) m.store(col(l, j, i) < D ? at + col(l, j, i) * sizeof(T) : kNowhere, x[i]);
    }
  }
  static __device__ __forceinline__ void params(const float* p, int l, int j, int D, float none, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = !p ? none : col(l, j, i) < D ? p[col(l, j, i)] : 0.f;
  }
};

// The rows of a workgroup's step as a range: RPB rows from `first` on, those behind the tensor's end
// missing; empty if the tensor is not given.
template <typename T, int RPB>
__device__ __forceinline__ Range<T> step_range(const T* base, int64_t first, const NormShape& s) {
  const int64_t left = s.rows - first, n = left < 0 ? 0 : (left < RPB ? left : RPB);
  return Range<T>(base + (base && n > 0 ? first * s.D : 0), base ? n * s.D * static_cast<int64_t>(sizeof(T)) : 0);
}

template <int LPR_, int NV_> struct NormTile {
  static constexpr int LPR = LPR_, NV = NV_;
};

// Calls f with the tile for rows of D columns: the smallest of 8 LPR NV columns that holds the row.
template <typename F>
static hipError_t with_tile(int D, F f) {
  if (D <= 64) return f(NormTile<8, 1>{});
  if (D <= 128) return f(NormTile<16, 1>{});
  if (D <= 256) return f(NormTile<32, 1>{});
  if (D <= 512) return f(NormTile<64, 1>{});
  if (D <= 1024) return f(NormTile<128, 1>{});
  if (D <= 2048) return f(NormTile<256, 1>{});
  if (D <= 4096) return f(NormTile<512, 1>{});
  if (D <= 8192) return f(NormTile<512, 2>{});
  return f(NormTile<1024, 2>{});
}

static bool norm_aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace comba
