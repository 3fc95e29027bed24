// The norms after and before a block, fused with the block's gate, residual scale and residual sum.
// Per row of D elements:
//   u = y                      or  y k1 post_weight,  k1 = 1 / sqrt(mean(y^2) + eps)
//   u = u                      or  u gate sigmoid(gate)
//   r = scale u + residual     (either may be absent)
//   n = r k2 pre_weight,       k2 = 1 / sqrt(mean(r^2) + eps)   (if the next block's norm is asked for)
// n is formed from the float32 r, before r is rounded.
//
// Bound by HBM: every input is read once and every output written once, with the row in registers
// between the reductions. A row is spread over LPR lanes in pieces of 8 elements (piece j of lane l:
// columns 8 (j LPR + l)), a part of a wavefront up to 512 columns (several rows per wavefront,
// reductions without LDS), a workgroup above 1024. Workgroups walk over many rows with the
// parameters in registers.
#include "column_sums.h"
#include "comba.h"
#include "launch.h"
#include "layer.h"
#include "layer_common.h"

namespace comba {

constexpr int kNormThreads = 256;

// Sum over the LPR lanes that share a row, in every one of them. `red`: LDS of one float per
// wavefront and value; the caller alternates between two such arrays, so that one barrier per
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
    if constexpr (LPR >= 32) x += __shfl_xor(x, 16, kWave);
    if constexpr (LPR >= 64) x += __shfl_xor(x, 32, kWave);
    v[k] = x;
  }
  if constexpr (LPR > 64) {
    constexpr int NW = LPR / 64;
    const int w = threadIdx.x / kWave;
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

// 8 elements of column c of a row, with the pieces behind the row's end reading 0.
template <typename T, bool V>
__device__ __forceinline__ void load8(const T* row, int c, int D, float (&x)[8]) {
  if (c < D) {
    Pack<T, 8, V>::load(row + c, x, D - c);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
  }
}
template <typename T, bool V>
__device__ __forceinline__ void store8(T* row, int c, int D, const float (&x)[8]) {
  if (c < D) Pack<T, 8, V>::store(row + c, x, D - c);
}
__device__ __forceinline__ void load_param(const float* p, int c, int D, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = p && c + i < D ? p[c + i] : 0.f;
}

template <typename T, bool V, int LPR, int NV>
__global__ __launch_bounds__(LPR > kNormThreads ? LPR : kNormThreads) void norm_fwd_kernel(
    const T* __restrict__ y, const T* __restrict__ gate, const T* __restrict__ residual,
    const float* __restrict__ scale, const float* __restrict__ post, const float* __restrict__ pre, NormShape s,
    T* __restrict__ r_out, T* __restrict__ n_out) {
  constexpr int TH = LPR > kNormThreads ? LPR : kNormThreads, RPB = TH / LPR;
  __shared__ float red[2][LPR > 64 ? LPR / 64 : 1];
  const int l = threadIdx.x % LPR, D = s.D;
  float wpost[NV][8], wpre[NV][8], sc[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = 8 * (j * LPR + l);
    load_param(post, c, D, wpost[j]);
    load_param(pre, c, D, wpre[j]);
    load_param(scale, c, D, sc[j]);
  }
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * RPB + threadIdx.x / LPR;
       row - threadIdx.x / LPR < s.rows; row += static_cast<int64_t>(gridDim.x) * RPB) {
    const bool live = row < s.rows;  // rows of one workgroup share its barriers
    const int64_t at = (live ? row : s.rows - 1) * D;
    float u[NV][8], g[NV][8], r[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = 8 * (j * LPR + l);
      load8<T, V>(y + at, c, D, u[j]);
      if (gate) load8<T, V>(gate + at, c, D, g[j]);
      if (residual) load8<T, V>(residual + at, c, D, r[j]);
    }
    if (post) {
      float ss[1] = {0.f};
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss[0] = fmaf(u[j][i], u[j][i], ss[0]);
      row_sums<LPR, 1>(ss, red[0]);
      const float k1 = 1.f / sqrtf(fmaf(ss[0], s.inv, s.eps));
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) u[j][i] *= k1 * wpost[j][i];
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float v = u[j][i];
        if (gate) v *= g[j][i] * sigmoid_fast(g[j][i]);
        if (scale) v *= sc[j][i];
        u[j][i] = residual ? v + r[j][i] : v;
      }
    if (live)
#pragma unroll
      for (int j = 0; j < NV; ++j) store8<T, V>(r_out + at, 8 * (j * LPR + l), D, u[j]);
    if (pre) {
      float ss[1] = {0.f};
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss[0] = fmaf(u[j][i], u[j][i], ss[0]);
      row_sums<LPR, 1>(ss, red[1]);
      const float k2 = 1.f / sqrtf(fmaf(ss[0], s.inv, s.eps));
#pragma unroll
      for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int i = 0; i < 8; ++i) u[j][i] *= k2 * wpre[j][i];
        if (live) store8<T, V>(n_out + at, 8 * (j * LPR + l), D, u[j]);
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
  constexpr int TH = LPR > kNormThreads ? LPR : kNormThreads, RPB = TH / LPR, NW = LPR > 64 ? LPR / 64 : 1;
  __shared__ float red[3][2 * NW];
  __shared__ float cols[RPB > 1 ? RPB : 1][RPB > 1 ? LPR * 8 : 1];
  const int l = threadIdx.x % LPR, D = s.D;
  float wpost[NV][8], wpre[NV][8], sc[NV][8], a_post[NV][8], a_pre[NV][8], a_sc[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = 8 * (j * LPR + l);
    load_param(post, c, D, wpost[j]);
    load_param(pre, c, D, wpre[j]);
    load_param(scale, c, D, sc[j]);
#pragma unroll
    for (int i = 0; i < 8; ++i) a_post[j][i] = a_pre[j][i] = a_sc[j][i] = 0.f;
  }
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * RPB + threadIdx.x / LPR;
       row - threadIdx.x / LPR < s.rows; row += static_cast<int64_t>(gridDim.x) * RPB) {
    const bool live = row < s.rows;
    const int64_t at = (live ? row : s.rows - 1) * D;
    float yv[NV][8], g[NV][8], r[NV][8], d[NV][8], e[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = 8 * (j * LPR + l);
      load8<T, V>(y + at, c, D, yv[j]);
      if (gate) load8<T, V>(gate + at, c, D, g[j]);
      if (residual && dn) load8<T, V>(residual + at, c, D, r[j]);
      if (dr) load8<T, V>(dr + at, c, D, d[j]);
      if (dn) load8<T, V>(dn + at, c, D, e[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (!dr) d[j][i] = 0.f;
    }
    float k1 = 1.f;
    if (post) {
      float ss[1] = {0.f};
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss[0] = fmaf(yv[j][i], yv[j][i], ss[0]);
      row_sums<LPR, 1>(ss, red[0]);
      k1 = 1.f / sqrtf(fmaf(ss[0], s.inv, s.eps));
    }
    // h: the value before the gate; u = h (gate sigmoid(gate))
    auto value = [&](int j, int i) { return post ? yv[j][i] * k1 * wpost[j][i] : yv[j][i]; };
    if (dn) {
      float ss[2] = {0.f, 0.f};
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float v = value(j, i);
          if (gate) v *= g[j][i] * sigmoid_fast(g[j][i]);
          if (scale) v *= sc[j][i];
          if (residual) v += r[j][i];
          r[j][i] = v;
          ss[0] = fmaf(v, v, ss[0]);
          ss[1] = fmaf(e[j][i] * wpre[j][i], v, ss[1]);
        }
      row_sums<LPR, 2>(ss, red[1]);
      const float k2 = 1.f / sqrtf(fmaf(ss[0], s.inv, s.eps)), m = ss[1] * s.inv * k2 * k2;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (live) a_pre[j][i] = fmaf(e[j][i], r[j][i] * k2, a_pre[j][i]);
          d[j][i] += k2 * (e[j][i] * wpre[j][i] - r[j][i] * m);
        }
    }
    float ss[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = 8 * (j * LPR + l);
      if (dres && live) store8<T, V>(dres + at, c, D, d[j]);
      float dg[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float h = value(j, i);
        float sg = 1.f, gs = 1.f;
        if (gate) {
          sg = sigmoid_fast(g[j][i]);
          gs = g[j][i] * sg;
        }
        if (scale) {
          if (live) a_sc[j][i] = fmaf(h * gs, d[j][i], a_sc[j][i]);
          d[j][i] *= sc[j][i];
        }
        if (gate) {
          dg[i] = d[j][i] * h * (sg * fmaf(g[j][i], 1.f - sg, 1.f));
          d[j][i] *= gs;
        }
        if (post) {
          if (live) a_post[j][i] = fmaf(d[j][i], yv[j][i] * k1, a_post[j][i]);
          d[j][i] *= wpost[j][i];
          ss[0] = fmaf(d[j][i], yv[j][i], ss[0]);
        }
      }
      if (dgate && live) store8<T, V>(dgate + at, c, D, dg);
    }
    if (post) {
      row_sums<LPR, 1>(ss, red[2]);
      const float m = ss[0] * s.inv * k1 * k1;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) d[j][i] = k1 * (d[j][i] - yv[j][i] * m);
    }
    if (live)
#pragma unroll
      for (int j = 0; j < NV; ++j) store8<T, V>(dy + at, 8 * (j * LPR + l), D, d[j]);
    if constexpr (LPR > 64) {
      if (!post && dn) __syncthreads();  // the one reduction's array is free for the next row
    }
  }
  // column sums of this workgroup: [block][scale, post, pre][D]
  float* out = part + static_cast<int64_t>(blockIdx.x) * 3 * D;
  auto emit = [&](int which, float (&a)[NV][8]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = 8 * (j * LPR + l);
      if constexpr (RPB > 1) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) cols[threadIdx.x / LPR][l * 8 + i] = a[j][i];
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
          if (c + i < D) out[which * static_cast<int64_t>(D) + c + i] = a[j][i];
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
  if (D <= 1024) return f(NormTile<64, 2>{});
  if (D <= 2048) return f(NormTile<256, 1>{});
  if (D <= 4096) return f(NormTile<256, 2>{});
  if (D <= 8192) return f(NormTile<512, 2>{});
  return f(NormTile<1024, 2>{});
}

static bool norm_aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

static int64_t norm_blocks(int64_t rows, int rpb, int64_t most) {
  const int64_t want = (rows + rpb - 1) / rpb;
  return want < most ? want : most;
}

template <typename T, bool V>
static hipError_t norm_fwd_t(const NormArgs& a, hipStream_t st) {
  return with_tile(a.D, [&](auto tile) {
    constexpr int LPR = decltype(tile)::LPR, NV = decltype(tile)::NV, TH = LPR > kNormThreads ? LPR : kNormThreads;
    const int64_t grid = norm_blocks(a.rows, TH / LPR, 256 * (2048 / TH));
    const NormShape s{a.rows, a.D, a.eps, 1.f / a.D};
    norm_fwd_kernel<T, V, LPR, NV><<<static_cast<unsigned>(grid), TH, 0, st>>>(
        static_cast<const T*>(a.y), static_cast<const T*>(a.gate), static_cast<const T*>(a.residual), a.scale,
        a.post_weight, a.pre_weight, s, static_cast<T*>(a.r), static_cast<T*>(a.n));
    return hipGetLastError();
  });
}

hipError_t launch_norm(const NormArgs& a, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  const bool v = a.D % 8 == 0 && norm_aligned(a.y) && norm_aligned(a.gate) && norm_aligned(a.residual) &&
                 norm_aligned(a.r) && norm_aligned(a.n);
  if (a.dtype == COMBA_BF16) return v ? norm_fwd_t<u16, true>(a, st) : norm_fwd_t<u16, false>(a, st);
  return v ? norm_fwd_t<float, true>(a, st) : norm_fwd_t<float, false>(a, st);
}

// Four wavefronts per SIMD.
constexpr int64_t kNormBwdThreads = 1 << 18;

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
  float* to[3] = {a.dscale, a.dpost, a.dpre};
  const bool have[3] = {true, true, a.dn != nullptr};
  for (int k = 0; k < 3; ++k) {
    if (!to[k]) continue;
    const hipError_t e = launch_column_sums(a.part ? a.part + static_cast<int64_t>(k) * f.D : nullptr, have[k] ? grid : 0,
                                            3 * static_cast<int64_t>(f.D), f.D, to[k], st);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_norm_bwd(const NormBwdArgs& a, hipStream_t st) {
  const NormArgs& f = a.f;
  const bool v = f.D % 8 == 0 && norm_aligned(f.y) && norm_aligned(f.gate) && norm_aligned(f.residual) &&
                 norm_aligned(a.dr) && norm_aligned(a.dn) && norm_aligned(a.dy) && norm_aligned(a.dgate) &&
                 norm_aligned(a.dresidual);
  if (f.dtype == COMBA_BF16) return v ? norm_bwd_t<u16, true>(a, st) : norm_bwd_t<u16, false>(a, st);
  return v ? norm_bwd_t<float, true>(a, st) : norm_bwd_t<float, false>(a, st);
}

hipError_t launch_column_sums(const float* part, int64_t rows, int64_t stride, int cols, float* out, hipStream_t st) {
  return column_sums(part, rows, stride, cols, st, [=] __device__(int c, float s) { out[c] = s; });
}

}  // namespace comba
