// The norms after and before a block, fused with the block's gate, residual scale and residual sum.
// Per row of D elements:
//   u = y                      or  y k1 post_weight,  k1 = 1 / sqrt(mean(y^2) + eps)
//   u = u                      or  u gate sigmoid(gate)
//   r = scale u + residual     (either may be absent)
//   n = r k2 pre_weight,       k2 = 1 / sqrt(mean(r^2) + eps)   (if the next block's norm is asked for)
// n is formed from the float32 r, before r is rounded.
//
// Bound by HBM: every input is read once and every output written once, with the row in registers
// between the reductions. A row is spread over LPR lanes, 8 NV elements each: a part of a wavefront
// up to 512 columns (several rows per wavefront, reductions without LDS), a workgroup above 1024.
// Workgroups walk over many rows with the parameters in registers, and load the next row before they
// work on the present one. Parts that are not given read 0 from an empty range, without a branch.
// Measured, bf16, with inputs that change from call to call: gated norm of 524288 rows of 128 76 us
// (5.3 TB/s); the seam's backward with all parts, 8192 rows of 2048, 65 to 71 us with the parameter sums
// (3.8 to 4.1 TB/s); the seam for 33 rows of 2047 in fp32 4.2 us, of which a launch takes most. With the same
// inputs again, part of which the last-level cache then holds, 64 and 60 us (93 the former without the
// row ahead and the streaming stores); so were the comparisons below taken.
// Far from HBM's rate above 8192 columns, where 1024 threads may have 128 registers each: the backward
// spills 285 to 334 of them, and 1024 rows of 16384 with all parts take 430 us in bf16 and 487 in fp32 (0.6
// and 1.1 TB/s; forward 55 and 72 us). The backward of 4097 to 8192 columns spills where it takes single
// elements (78 registers in bf16, 48 in fp32) and 6 in fp32 with pieces: 2048 rows of 8192 89 us in bf16,
// 125 in fp32 (3.0 and 4.3 TB/s). Rows of odd widths, whose elements are read one by one, cost no more than
// their neighbours: 8192 rows of 2047 / 2048, all parts, forward 36 / 43 us in bf16, 64 / 64 in fp32,
// backward 66 / 68 and 118 / 114.
#include "column_sums.h"
#include "comba.h"
#include "launch.h"
#include "layer.h"
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

template <typename T, bool V, int LPR, int NV>
__global__ __launch_bounds__(LPR > kNormThreads ? LPR : kNormThreads) void norm_fwd_kernel(
    const T* __restrict__ y, const T* __restrict__ gate, const T* __restrict__ residual,
    const float* __restrict__ scale, const float* __restrict__ post, const float* __restrict__ pre, NormShape s,
    T* __restrict__ r_out, T* __restrict__ n_out) {
  constexpr int TH = LPR > kNormThreads ? LPR : kNormThreads, RPB = TH / LPR;
  constexpr bool PF = TH <= 512 && NV == 1;  // else there are no registers for a second row
  using E = Eight<T, V, LPR>;
  __shared__ float red[2][TH / 64];
  const int l = threadIdx.x % LPR, D = s.D;
  const uint32_t at = static_cast<uint32_t>(threadIdx.x / LPR) * D * sizeof(T);
  float wpost[NV][8], wpre[NV][8], sc[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    E::params(post, l, j, D, 1.f, wpost[j]);
    E::params(pre, l, j, D, 1.f, wpre[j]);
    E::params(scale, l, j, D, 1.f, sc[j]);
  }
  E yn[NV], gn[NV], rn[NV];
  auto fetch = [&](int64_t first) {
    const Range<T> ym = step_range<T, RPB>(y, first, s), gm = step_range<T, RPB>(gate, first, s),
                   rm = step_range<T, RPB>(residual, first, s);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      yn[j].load(ym, at, l, j, D);
      gn[j].load(gm, at, l, j, D);
      rn[j].load(rm, at, l, j, D);
    }
  };
  const int64_t stride = static_cast<int64_t>(gridDim.x) * RPB;
  int64_t first = static_cast<int64_t>(blockIdx.x) * RPB;
  if (PF) fetch(first);
  for (; first < s.rows; first += stride) {
    if (!PF) fetch(first);
    E yc[NV], gc[NV], rc[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      yc[j] = yn[j];
      gc[j] = gn[j];
      rc[j] = rn[j];
    }
    if (PF) fetch(first + stride);
    float k1 = 1.f;
    if (post) {
      float ss[1] = {0.f};
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss[0] = fmaf(yc[j][i], yc[j][i], ss[0]);
      row_sums<LPR, 1>(ss, red[0]);
      k1 = 1.f / sqrtf(fmaf(ss[0], s.inv, s.eps));
    }
    float u[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) u[j][i] = yc[j][i] * (k1 * wpost[j][i]);
    if (gate)
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) u[j][i] *= gc[j][i] * sigmoid_fast(gc[j][i]);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) u[j][i] = residual ? fmaf(u[j][i], sc[j][i], rc[j][i]) : u[j][i] * sc[j][i];
    const Range<T> ro = step_range<T, RPB>(r_out, first, s);
#pragma unroll
    for (int j = 0; j < NV; ++j) E::store(ro, at, l, j, D, u[j]);
    if (pre) {
      float ss[1] = {0.f};
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss[0] = fmaf(u[j][i], u[j][i], ss[0]);
      row_sums<LPR, 1>(ss, red[1]);
      const float k2 = 1.f / sqrtf(fmaf(ss[0], s.inv, s.eps));
      const Range<T> no = step_range<T, RPB>(n_out, first, s);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int i = 0; i < 8; ++i) u[j][i] *= k2 * wpre[j][i];
        E::store(no, at, l, j, D, u[j]);
      }
    }
    if constexpr (LPR > 64) {
      // one norm alone uses one array: the next row must not overwrite it while it is read
      if ((post != nullptr) != (pre != nullptr)) __syncthreads();
    }
  }
}

// Backward. With the row recomputed: given dr and dn,
//   d = dr + k2 (dn w - r k2^2 mean(dn w r)),  w = pre_weight;   dresidual = d
//   du = scale d;  dgate = du h s (1 + g (1 - s)),  h = the gated value, s = sigmoid(g);  dh = du g s
//   dy = k1 (dh w' - y k1^2 mean(dh w' y)),  w' = post_weight
// dscale = sum over rows of u d, dpre_weight of dn r k2, dpost_weight of dh y k1: float32 in
// registers over a workgroup's rows, then over its row groups through LDS, then over the workgroups
// by a second kernel, always in the same order. Mean: over the D columns.
template <typename T, bool V, int LPR, int NV>
__global__ __launch_bounds__(LPR > kNormThreads ? LPR : kNormThreads) void norm_bwd_kernel(
    const T* __restrict__ y, const T* __restrict__ gate, const T* __restrict__ residual,
    const float* __restrict__ scale, const float* __restrict__ post, const float* __restrict__ pre,
    const T* __restrict__ dr, const T* __restrict__ dn, NormShape s, T* __restrict__ dy, T* __restrict__ dgate,
    T* __restrict__ dres, float* __restrict__ part) {
  constexpr int TH = LPR > kNormThreads ? LPR : kNormThreads, RPB = TH / LPR;
  constexpr bool PF = TH <= 512 && NV == 1;  // else there are no registers for a second row
  using E = Eight<T, V, LPR>;
  __shared__ float red[3][2 * (TH / 64)];
  __shared__ float cols[RPB > 1 ? RPB : 1][RPB > 1 ? LPR * 8 : 1];
  const int l = threadIdx.x % LPR, D = s.D;
  const uint32_t at = static_cast<uint32_t>(threadIdx.x / LPR) * D * sizeof(T);
  float wpost[NV][8], wpre[NV][8], sc[NV][8], a_post[NV][8], a_pre[NV][8], a_sc[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    E::params(post, l, j, D, 1.f, wpost[j]);
    E::params(pre, l, j, D, 1.f, wpre[j]);
    E::params(scale, l, j, D, 1.f, sc[j]);
#pragma unroll
    for (int i = 0; i < 8; ++i) a_post[j][i] = a_pre[j][i] = a_sc[j][i] = 0.f;
  }
  E yn[NV], gn[NV], rn[NV], dn_[NV], en[NV];
  const T* res = dn ? residual : nullptr;  // the residual is needed for r alone
  auto fetch = [&](int64_t first) {
    const Range<T> ym = step_range<T, RPB>(y, first, s), gm = step_range<T, RPB>(gate, first, s),
                   rm = step_range<T, RPB>(res, first, s), dm = step_range<T, RPB>(dr, first, s),
                   em = step_range<T, RPB>(dn, first, s);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      yn[j].load(ym, at, l, j, D);
      gn[j].load(gm, at, l, j, D);
      rn[j].load(rm, at, l, j, D);
      en[j].load(em, at, l, j, D);
      dn_[j].load(dm, at, l, j, D);
    }
  };
  const int64_t stride = static_cast<int64_t>(gridDim.x) * RPB;
  int64_t first = static_cast<int64_t>(blockIdx.x) * RPB;
  if (PF) fetch(first);
  for (; first < s.rows; first += stride) {
    if (!PF) fetch(first);
    const bool live = first + threadIdx.x / LPR < s.rows;
    E yc[NV], gc[NV], rc[NV], dc[NV], ec[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      yc[j] = yn[j];
      gc[j] = gn[j];
      rc[j] = rn[j];
      dc[j] = dn_[j];
      ec[j] = en[j];
    }
    if (PF) fetch(first + stride);
    float k1 = 1.f;
    if (post) {
      float ss[1] = {0.f};
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss[0] = fmaf(yc[j][i], yc[j][i], ss[0]);
      row_sums<LPR, 1>(ss, red[0]);
      k1 = 1.f / sqrtf(fmaf(ss[0], s.inv, s.eps));
    }
    float d[NV][8], sg[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        d[j][i] = dc[j][i];
        sg[j][i] = gate ? sigmoid_fast(gc[j][i]) : 1.f;
      }
    // h: the value before the gate, gs: the gate's factor
    auto h = [&](int j, int i) { return yc[j][i] * (k1 * wpost[j][i]); };
    auto gs = [&](int j, int i) { return gate ? gc[j][i] * sg[j][i] : 1.f; };
    if (dn) {
      float ss[2] = {0.f, 0.f}, r[NV][8];
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          r[j][i] = fmaf(h(j, i) * gs(j, i), sc[j][i], rc[j][i]);
          ss[0] = fmaf(r[j][i], r[j][i], ss[0]);
          ss[1] = fmaf(ec[j][i] * wpre[j][i], r[j][i], ss[1]);
        }
      row_sums<LPR, 2>(ss, red[1]);
      const float k2 = 1.f / sqrtf(fmaf(ss[0], s.inv, s.eps)), m = ss[1] * s.inv * k2 * k2;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (live) a_pre[j][i] = fmaf(ec[j][i], r[j][i] * k2, a_pre[j][i]);
          d[j][i] += k2 * (ec[j][i] * wpre[j][i] - r[j][i] * m);
        }
    }
    if (dres) {
      const Range<T> o = step_range<T, RPB>(dres, first, s);
#pragma unroll
      for (int j = 0; j < NV; ++j) E::store(o, at, l, j, D, d[j]);
    }
    if (scale)
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (live) a_sc[j][i] = fmaf(h(j, i) * gs(j, i), d[j][i], a_sc[j][i]);
          d[j][i] *= sc[j][i];
        }
    if (gate) {
      const Range<T> o = step_range<T, RPB>(dgate, first, s);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float dg[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dg[i] = d[j][i] * h(j, i) * (sg[j][i] * fmaf(gc[j][i], 1.f - sg[j][i], 1.f));
          d[j][i] *= gs(j, i);
        }
        E::store(o, at, l, j, D, dg);
      }
    }
    if (post) {
      float ss[1] = {0.f};
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (live) a_post[j][i] = fmaf(d[j][i], yc[j][i] * k1, a_post[j][i]);
          d[j][i] *= wpost[j][i];
          ss[0] = fmaf(d[j][i], yc[j][i], ss[0]);
        }
      row_sums<LPR, 1>(ss, red[2]);
      const float m = ss[0] * s.inv * k1 * k1;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) d[j][i] = k1 * (d[j][i] - yc[j][i] * m);
    }
    const Range<T> o = step_range<T, RPB>(dy, first, s);
#pragma unroll
    for (int j = 0; j < NV; ++j) E::store(o, at, l, j, D, d[j]);
    if constexpr (LPR > 64) {
      if (!post && dn) __syncthreads();  // the one reduction's array is free for the next row
    }
  }
  // column sums of this workgroup: [block][scale, post, pre][D]
  float* out = part + static_cast<int64_t>(blockIdx.x) * 3 * D;
  auto emit = [&](int which, float (&a)[NV][8]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if constexpr (RPB > 1) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) cols[threadIdx.x / LPR][E::col(l, 0, i)] = a[j][i];
        __syncthreads();
        for (int k = threadIdx.x; k < LPR * 8; k += TH) {
          float t = 0.f;
          for (int q = 0; q < RPB; ++q) t += cols[q][k];
          const int col = j * LPR * 8 + k;
          if (col < D) out[which * static_cast<int64_t>(D) + col] = t;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (E::col(l, j, i) < D) out[which * static_cast<int64_t>(D) + E::col(l, j, i)] = a[j][i];
      }
    }
  };
  if (scale) emit(0, a_sc);
  if (post) emit(1, a_post);
  if (dn) emit(2, a_pre);
}

// --- launches -----------------------------------------------------------------------------------

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

static int64_t norm_blocks(int64_t rows, int rpb, int64_t most) {
  const int64_t want = (rows + rpb - 1) / rpb;
  return want < most ? want : most;
}

// 1024 threads per compute unit. With 512 / 1024 / 2048: 61 / 56 / 54 us for 524288 rows of 128 (gate
// and input the same tensor), 69 / 58 / 55 for 32768 of 2048, 36 / 32 / 31 for 8192 of 4096.
template <typename T, bool V>
static hipError_t norm_fwd_t(const NormArgs& a, hipStream_t st) {
  return with_tile(a.D, [&](auto tile) {
    constexpr int LPR = decltype(tile)::LPR, NV = decltype(tile)::NV, TH = LPR > kNormThreads ? LPR : kNormThreads;
    const int64_t grid = norm_blocks(a.rows, TH / LPR, 256 * (1024 / TH));
    const NormShape s{a.rows, a.D, a.eps, 1.f / a.D};
    norm_fwd_kernel<T, V, LPR, NV><<<static_cast<unsigned>(grid), TH, 0, st>>>(
        static_cast<const T*>(a.y), static_cast<const T*>(a.gate), static_cast<const T*>(a.residual), a.scale,
        a.post_weight, a.pre_weight, s, static_cast<T*>(a.r), static_cast<T*>(a.n));
    return hipGetLastError();
  });
}

hipError_t launch_norm(const NormArgs& a, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  const bool v = a.D % (a.dtype == COMBA_BF16 ? 8 : 4) == 0 && norm_aligned(a.y) && norm_aligned(a.gate) && norm_aligned(a.residual) &&
                 norm_aligned(a.r) && norm_aligned(a.n);
  if (a.dtype == COMBA_BF16) return v ? norm_fwd_t<u16, true>(a, st) : norm_fwd_t<u16, false>(a, st);
  return v ? norm_fwd_t<float, true>(a, st) : norm_fwd_t<float, false>(a, st);
}

// Two wavefronts per SIMD: at 8192 rows of 2048, bf16, all parts, 64 us against 66 with three and 79 with
// four (three are resident; more workgroups mean more partial sums and a second round).
constexpr int64_t kNormBwdThreads = 1 << 17;

template <typename Tile> static int64_t norm_bwd_grid(int64_t rows) {
  constexpr int TH = Tile::LPR > kNormThreads ? Tile::LPR : kNormThreads;
  return norm_blocks(rows, TH / Tile::LPR, kNormBwdThreads / TH);
}

int64_t norm_bwd_blocks(int64_t rows, int D) {
  int64_t n = 0;
  (void)with_tile(D, [&](auto tile) {
    n = norm_bwd_grid<decltype(tile)>(rows);
    return hipSuccess;
  });
  return n;
}

template <typename T, bool V>
static hipError_t norm_bwd_t(const NormBwdArgs& a, hipStream_t st) {
  const NormArgs& f = a.f;
  int64_t grid = 0;
  if (f.rows > 0) {
    const hipError_t e = with_tile(f.D, [&](auto tile) {
      constexpr int LPR = decltype(tile)::LPR, NV = decltype(tile)::NV, TH = LPR > kNormThreads ? LPR : kNormThreads;
      grid = norm_bwd_grid<decltype(tile)>(f.rows);
      const NormShape s{f.rows, f.D, f.eps, 1.f / f.D};
      norm_bwd_kernel<T, V, LPR, NV><<<static_cast<unsigned>(grid), TH, 0, st>>>(
          static_cast<const T*>(f.y), static_cast<const T*>(f.gate), static_cast<const T*>(f.residual), f.scale,
          f.post_weight, f.pre_weight, static_cast<const T*>(a.dr), static_cast<const T*>(a.dn), s,
          static_cast<T*>(a.dy), static_cast<T*>(a.dgate), static_cast<T*>(a.dresidual), a.part);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
  }
  // the parts that were summed; without dn the gradient of pre_weight is 0
  float* sc = a.dscale;
  float* post = a.dpost;
  float* pre = a.dpre;
  if (!sc && !post && !pre) return hipSuccess;
  const int D = f.D;
  const bool no_dn = a.dn == nullptr;
  return column_sums(a.part, grid, 3 * static_cast<int64_t>(D), 3 * D, st, [=] __device__(int col, float v) {
    const int k = col / D;
    float* to = k == 0 ? sc : k == 1 ? post : pre;
    if (to) to[col - k * D] = k == 2 && no_dn ? 0.f : v;
  });
}

hipError_t launch_norm_bwd(const NormBwdArgs& a, hipStream_t st) {
  const NormArgs& f = a.f;
  const bool v = f.D % (f.dtype == COMBA_BF16 ? 8 : 4) == 0 && norm_aligned(f.y) && norm_aligned(f.gate) && norm_aligned(f.residual) &&
                 norm_aligned(a.dr) && norm_aligned(a.dn) && norm_aligned(a.dy) && norm_aligned(a.dgate) &&
                 norm_aligned(a.dresidual);
  if (f.dtype == COMBA_BF16) return v ? norm_bwd_t<u16, true>(a, st) : norm_bwd_t<u16, false>(a, st);
  return v ? norm_bwd_t<float, true>(a, st) : norm_bwd_t<float, false>(a, st);
}

}  // namespace comba
