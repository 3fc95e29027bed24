// Backward of the selective scan. With p_t = dy_t z sigmoid(z) and the forward's d, h, per channel
// (g_t: gradient of h_t, run from the end):
//   g_t[s]  = p_t C_t[s] + exp(d_{t+1} A[s]) g_{t+1}[s]      (behind the last token: d_final_state)
//   dC_t[s] = sum_c p_t h_t[s]          dB_t[s] = sum_c g_t[s] d_t x_t        (channels of the group)
//   dx_t    = skip p_t + d_t sum_s g_t[s] B_t[s]
//   dd_t    = x_t sum_s g_t[s] B_t[s] + sum_s A[s] k_t[s],  k_t = g_t exp(d_t A) h_{t-1};  ddt = dd sigmoid(dt + bias)
//   dA[s]   = sum_t d_t k_t[s],   dz, dskip, ddt_bias elementwise or summed over tokens,
//   d_initial_state = exp(d_0 A) g_0
//
// Every sequence is cut into segments of L tokens that run in parallel:
//   1. scan_bwd_ends: each segment's end state from 0, its gradient of its incoming state for no
//      gradient behind it, and its sum of step sizes (the map of both is exp(A sum d));
//   2. scan_bwd_carry: the true incoming states and outgoing gradients, along the segments;
//   3. scan_bwd: per segment the states at every CT-th token forward, then from its end the CT tokens
//      of each piece: states and decays recomputed into registers, then the reverse recurrence;
//   4. the sums over segments (dA, dskip, ddt_bias) and over channel blocks (dB, dC), in a fixed order.
// Nothing is kept from the forward. Bound by the vector ALU like the forward: three exponentials and
// about 25 instructions per (token, channel, state). The sums over the 16 channels of a wavefront
// halve the values at every step (permlane swaps: two instructions per pair of values).
#include "column_sums.h"
#include "comba.h"
#include "scan_common.h"

namespace comba {

template <int NPL> struct BwdTile {
  static constexpr int CT = NPL <= 4 ? 16 : 64 / NPL;        // tokens whose states are held in registers
  static constexpr int NSUB = NPL <= 8 ? 8 : 4;              // pieces of CT tokens per segment
  static constexpr int L = CT * NSUB;
};

template <typename T> struct ScanBwdK {
  const T* x;
  const T* dt;
  const float* A;
  const T* Bm;
  const T* Cm;
  const float* skip;
  const T* z;
  const float* dt_bias;
  const float* init;
  const int32_t* cu;
  const T* dy;
  const float* dfin;
  T* dx;
  T* ddt;
  T* dz;
  float* dinit;
  float* hseg;
  float* gseg;
  float* dsum;
  float* dApart;
  float* dDpart;
  float* dBCpart;
  int N, T_, D, S, G, L;
  bool softplus;
};

// B and C of the segment's tokens as float32 in LDS, [token][quad lane][NPL of B, NPL of C]; 0 where
// there is no token or state.
template <typename T, int NPL, int L>
__device__ __forceinline__ void stage_bc(const ScanBwdK<T>& a, const ScanPlace& p, float (*bc)[4][2 * NPL]) {
  constexpr int SP = 4 * NPL;
  const int64_t row0 = static_cast<int64_t>(p.b) * a.T_ + p.t0;
  for (int e = threadIdx.x; e < L * SP; e += kScanBlock) {
    const int t = e / SP, s = e % SP;
    const bool have = p.t0 + t < p.t1 && s < a.S;
    const int64_t o = ((row0 + t) * a.G + p.g) * a.S + s;
    bc[t][s / NPL][s % NPL] = have ? Elem<T>::load(a.Bm, o) : 0.f;
    bc[t][s / NPL][NPL + s % NPL] = have ? Elem<T>::load(a.Cm, o) : 0.f;
  }
}

// Sums v over the 16 channels of the wavefront (lane bits 2 .. 5). At lane bit 5, 4, 3, 2 a lane keeps
// the lower half of its values if the bit is clear, the upper half if it is set, while there are two
// or more; then all lanes add. Left: v[0 .. max(1, N/16) - 1].
template <int N>
__device__ __forceinline__ void channel_sums(float* v, int lane) {
  auto swap_add = [](float u, float w, auto wide) {
    const unsigned a = __float_as_uint(u), b = __float_as_uint(w);
    if constexpr (decltype(wide)::value) {
      auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
      return __uint_as_float(r[0]) + __uint_as_float(r[1]);
    } else {
      auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
      return __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
  };
  auto ror8 = [](float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x128, 0xf, 0xf, true));
  };
  // lane ^ 4: mirror the 8-lane half, then reverse the quad
  auto flip4 = [](float x) {
    const int m = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x141, 0xf, 0xf, true);
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, m, 0x1b, 0xf, 0xf, true));
  };
  constexpr int H5 = N >= 2 ? N / 2 : 1, H4 = H5 >= 2 ? H5 / 2 : 1, H3 = H4 >= 2 ? H4 / 2 : 1, H2 = H3 >= 2 ? H3 / 2 : 1;
#pragma unroll
  for (int i = 0; i < H5; ++i) v[i] = swap_add(v[i], v[N >= 2 ? i + H5 : i], std::true_type{});
#pragma unroll
  for (int i = 0; i < H4; ++i) v[i] = swap_add(v[i], v[H5 >= 2 ? i + H4 : i], std::false_type{});
  const bool b3 = lane & 8, b2 = lane & 4;
#pragma unroll
  for (int i = 0; i < H3; ++i) {
    if constexpr (H4 >= 2) {
      const float keep = b3 ? v[i + H3] : v[i], send = b3 ? v[i] : v[i + H3];
      v[i] = keep + ror8(send);
    } else {
      v[i] += ror8(v[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < H2; ++i) {
    if constexpr (H3 >= 2) {
      const float keep = b2 ? v[i + H2] : v[i], send = b2 ? v[i] : v[i + H2];
      v[i] = keep + flip4(send);
    } else {
      v[i] += flip4(v[i]);
    }
  }
}

// Index of the first value that channel_sums<N> leaves in this lane, and whether the lane is the one
// that writes it (where lanes hold the same value).
template <int N>
__device__ __forceinline__ int channel_sum_index(int lane, bool& writer) {
  int at = 0, n = N;
  writer = true;
#pragma unroll
  for (int b = 5; b >= 2; --b) {
    const int bit = (lane >> b) & 1;
    if (n >= 2) {
      n /= 2;
      at += bit * n;
    } else if (bit) {
      writer = false;
    }
  }
  return at;
}

template <typename T>
__device__ __forceinline__ float step_size(const ScanBwdK<T>& a, float raw, float bias) {
  const float u = raw + bias;
  return a.softplus ? softplus_f32(u) : u;
}

template <typename T, int NPL>
__global__ __launch_bounds__(kScanBlock) void scan_bwd_ends_kernel(ScanBwdK<T> a) {
  constexpr int SP = 4 * NPL, L = BwdTile<NPL>::L;
  __shared__ __align__(16) float bc[L][4][2 * NPL];
  const int tid = threadIdx.x, lane = tid & 63, q = lane & 3;
  const int cblocks = a.G * ((a.D / a.G + kScanChannels - 1) / kScanChannels);
  const ScanPlace p = scan_place<kScanChannels>(blockIdx.x / cblocks, blockIdx.x % cblocks, a.cu, a.N, a.T_, a.D, a.G, L);
  if (!p.ok) return;
  stage_bc<T, NPL, L>(a, p, bc);
  const int in = (tid >> 6) * 16 + (lane >> 2);
  const bool live = in < p.cl;
  const int c = p.c0 + (live ? in : p.cl - 1);
  float A2[NPL], h[NPL], gs[NPL], pr[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int s = q * NPL + i;
    A2[i] = s < a.S ? a.A[static_cast<int64_t>(c) * a.S + s] * kLog2E : 0.f;
    h[i] = gs[i] = 0.f;
    pr[i] = 1.f;
  }
  const float bias = a.dt_bias ? a.dt_bias[c] : 0.f;
  __syncthreads();
  const int64_t row0 = static_cast<int64_t>(p.b) * a.T_ + p.t0;
  const int len = p.t1 - p.t0;
  float dtot = 0.f;
  constexpr int U = 4;  // groups of four tokens fetched together
  for (int t = 0; t < len; t += 4 * U) {
    float rx[U], rd[U], rz[U], ry[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int64_t o = (row0 + min(t + 4 * j + q, len - 1)) * a.D + c;
      rx[j] = Elem<T>::load(a.x, o);
      rd[j] = Elem<T>::load(a.dt, o);
      ry[j] = Elem<T>::load(a.dy, o);
      rz[j] = a.z ? Elem<T>::load(a.z, o) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (t + 4 * j >= len) break;
      const bool have = t + 4 * j + q < len;
      const float dl = have ? step_size(a, rd[j], bias) : 0.f;
      const float dx = have ? dl * rx[j] : 0.f;
      float dyp = have ? ry[j] : 0.f;
      if (a.z && have) dyp *= rz[j] * sigmoid_fast(rz[j]);
      dtot += dl;
      auto token = [&](auto kc) {
        constexpr int K = decltype(kc)::value;
        const float dk = quad_bcast<K>(dl), xk = quad_bcast<K>(dx), yk = quad_bcast<K>(dyp);
        const float* r = bc[t + 4 * j + K][q];
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
          const float e = __builtin_amdgcn_exp2f(dk * A2[i]);
          h[i] = fmaf(e, h[i], xk * r[i]);
          pr[i] *= e;
          gs[i] = fmaf(pr[i], yk * r[NPL + i], gs[i]);
        }
      };
      token(std::integral_constant<int, 0>{});
      token(std::integral_constant<int, 1>{});
      token(std::integral_constant<int, 2>{});
      token(std::integral_constant<int, 3>{});
    }
  }
  if (!live) return;
  const int64_t at = (p.slot * a.D + c) * SP + q * NPL;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    a.hseg[at + i] = h[i];
    a.gseg[at + i] = gs[i];
  }
  dtot = lane_total<4>(dtot);
  if (q == 0) a.dsum[p.slot * a.D + c] = dtot;
}

// One thread per (direction, sequence, channel, state): hseg becomes the segments' incoming states,
// gseg the gradients at their ends; the gradient that leaves the first is d_initial_state.
__global__ __launch_bounds__(kScanBlock) void scan_bwd_carry_kernel(
    const float* __restrict__ A, const float* __restrict__ init, const float* __restrict__ dfin,
    const int32_t* __restrict__ cu, int N, int T, int64_t D, int S, int SP, int L, float* __restrict__ hseg,
    float* __restrict__ gseg, const float* __restrict__ dsum, float* __restrict__ dinit) {
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kScanBlock + threadIdx.x;
  const bool back = blockIdx.y == 1;
  const int s = static_cast<int>(id % SP);
  const int64_t nc = id / SP;
  const int n = static_cast<int>(nc / D);
  const int64_t c = nc - n * D;
  if (n >= N) return;
  int s0 = 0, s1 = T;
  if (cu) packed_range(cu, n, T, s0, s1);
  const int segs = segments_of(s1 - s0, L);
  const int64_t slot0 = cu ? static_cast<int64_t>(s0 / L) + n : static_cast<int64_t>(n) * ((T + L - 1) / L);
  const bool real = s < S;
  const float A2 = real ? A[c * S + s] * kLog2E : 0.f;
  const float* from = back ? dfin : init;
  float h = real && from ? from[(n * D + c) * S + s] : 0.f;
  float* hp = (back ? gseg : hseg) + (slot0 * D + c) * SP + s;
  const float* dp = dsum + slot0 * D + c;
  constexpr int U = 8;
  for (int k = 0; k < segs; k += U) {
    float own[U], d[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = min(k + u, segs - 1), at = back ? segs - 1 - i : i;
      own[u] = hp[at * D * SP];
      d[u] = dp[at * D];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k + u < segs) {
        hp[(back ? segs - 1 - k - u : k + u) * D * SP] = h;
        h = fmaf(__builtin_amdgcn_exp2f(A2 * d[u]), h, own[u]);
      }
    }
  }
  if (back && dinit && real) dinit[(n * D + c) * S + s] = h;
}

template <typename T, int NPL>
__global__ __launch_bounds__(kScanBlock) void scan_bwd_kernel(ScanBwdK<T> a) {
  constexpr int SP = 4 * NPL, CT = BwdTile<NPL>::CT, NSUB = BwdTile<NPL>::NSUB, L = BwdTile<NPL>::L, Q = CT / 4;
  constexpr int NV = 2 * NPL, LEFT = NV >= 16 ? NV / 16 : 1;
  __shared__ __align__(16) float bc[L][4][NV];
  __shared__ __align__(16) float held[NSUB][kScanBlock][NPL];   // states at the start of every piece
  __shared__ __align__(16) float red[2][4][CT][4][NV];          // dB, dC of a piece, per wavefront
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, q = lane & 3;
  const int dg = a.D / a.G, per = (dg + kScanChannels - 1) / kScanChannels, cblocks = a.G * per;
  const int cb = blockIdx.x % cblocks;
  const ScanPlace p = scan_place<kScanChannels>(blockIdx.x / cblocks, cb, a.cu, a.N, a.T_, a.D, a.G, L);
  const int in = wave * 16 + (lane >> 2);
  const bool live = in < p.cl;
  const int c = p.c0 + (live ? in : p.cl - 1);
  const int64_t at = (p.slot * a.D + c) * SP + q * NPL;
  const int64_t dpart = p.slot * 2 * a.D + c;
  if (!p.ok) {  // a slot between sequences adds nothing
    if (live) {
#pragma unroll
      for (int i = 0; i < NPL; ++i) a.dApart[at + i] = 0.f;
      if (q == 0) a.dDpart[dpart] = a.dDpart[dpart + a.D] = 0.f;
    }
    return;
  }
  stage_bc<T, NPL, L>(a, p, bc);
  float A2[NPL], h[NPL], gc[NPL], dA[NPL];  // gc: gradient that reaches the state before token t + 1
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int s = q * NPL + i;
    A2[i] = s < a.S ? a.A[static_cast<int64_t>(c) * a.S + s] * kLog2E : 0.f;
    h[i] = live ? a.hseg[at + i] : 0.f;
    gc[i] = live ? a.gseg[at + i] : 0.f;
    dA[i] = 0.f;
  }
  const float bias = a.dt_bias ? a.dt_bias[c] : 0.f, skip = a.skip ? a.skip[c] : 0.f;
  const int64_t row0 = static_cast<int64_t>(p.b) * a.T_ + p.t0;
  const int len = p.t1 - p.t0, nsub = (len + CT - 1) / CT;
  float dskip = 0.f, dbias = 0.f;
  __syncthreads();

  // states at the start of every piece
  for (int k = 0; k < nsub; ++k) {
#pragma unroll
    for (int i = 0; i < NPL; ++i) held[k][tid][i] = h[i];
    if (k == nsub - 1) break;
    float rx[Q], rd[Q];
#pragma unroll
    for (int j = 0; j < Q; ++j) {
      const int64_t o = (row0 + k * CT + 4 * j + q) * a.D + c;
      rx[j] = Elem<T>::load(a.x, o);
      rd[j] = Elem<T>::load(a.dt, o);
    }
#pragma unroll
    for (int j = 0; j < Q; ++j) {
      const float dl = live ? step_size(a, rd[j], bias) : 0.f;
      const float dx = live ? dl * rx[j] : 0.f;
      auto token = [&](auto kc) {
        constexpr int K = decltype(kc)::value;
        const float dk = quad_bcast<K>(dl), xk = quad_bcast<K>(dx);
        const float* r = bc[k * CT + 4 * j + K][q];
#pragma unroll
        for (int i = 0; i < NPL; ++i) h[i] = fmaf(__builtin_amdgcn_exp2f(dk * A2[i]), h[i], xk * r[i]);
      };
      token(std::integral_constant<int, 0>{});
      token(std::integral_constant<int, 1>{});
      token(std::integral_constant<int, 2>{});
      token(std::integral_constant<int, 3>{});
    }
  }

  bool writer;
  const int vat = channel_sum_index<NV>(lane, writer);
  const int cbg = cb - p.g * per;
  for (int k = nsub - 1, buf = 0; k >= 0; --k, buf ^= 1) {
    float xv[Q], ud[Q], zv[Q], yv[Q], dl[Q], dx[Q], dyp[Q], yr[Q];
#pragma unroll
    for (int j = 0; j < Q; ++j) {
      const int t = k * CT + 4 * j + q;
      const int64_t o = (row0 + min(t, len - 1)) * a.D + c;
      xv[j] = Elem<T>::load(a.x, o);
      ud[j] = Elem<T>::load(a.dt, o) + bias;
      yv[j] = Elem<T>::load(a.dy, o);
      zv[j] = a.z ? Elem<T>::load(a.z, o) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) h[i] = held[k][tid][i];
    float hs[CT][NPL], as[CT][NPL];
#pragma unroll
    for (int j = 0; j < Q; ++j) {
      const bool have = live && k * CT + 4 * j + q < len;
      dl[j] = have ? (a.softplus ? softplus_f32(ud[j]) : ud[j]) : 0.f;
      dx[j] = have ? dl[j] * xv[j] : 0.f;
      dyp[j] = have ? (a.z ? yv[j] * (zv[j] * sigmoid_fast(zv[j])) : yv[j]) : 0.f;
      float ys[4];
      auto token = [&](auto kc) {
        constexpr int K = decltype(kc)::value;
        const float dk = quad_bcast<K>(dl[j]), xk = quad_bcast<K>(dx[j]);
        const float* r = bc[k * CT + 4 * j + K][q];
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
          const float e = __builtin_amdgcn_exp2f(dk * A2[i]);
          const float prev = (4 * j + K) ? hs[(4 * j + K) ? 4 * j + K - 1 : 0][i] : h[i];
          as[4 * j + K][i] = e;
          hs[4 * j + K][i] = fmaf(e, prev, xk * r[i]);
          y = fmaf(hs[4 * j + K][i], r[NPL + i], y);
        }
        ys[K] = y;
      };
      token(std::integral_constant<int, 0>{});
      token(std::integral_constant<int, 1>{});
      token(std::integral_constant<int, 2>{});
      token(std::integral_constant<int, 3>{});
      yr[j] = lane_sums<4>(ys, lane);
    }
#pragma unroll
    for (int j = Q - 1; j >= 0; --j) {
      float sb[4], sa[4];
      auto token = [&](auto kc) {
        constexpr int K = decltype(kc)::value, t = K;
        const float dk = quad_bcast<K>(dl[j]), xk = quad_bcast<K>(dx[j]), yk = quad_bcast<K>(dyp[j]);
        const float* r = bc[k * CT + 4 * j + K][q];
        float v[NV], b = 0.f, d = 0.f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
          const float g = fmaf(yk, r[NPL + i], gc[i]);
          const float prev = (4 * j + t) ? hs[(4 * j + t) ? 4 * j + t - 1 : 0][i] : h[i];
          v[i] = g * xk;
          v[NPL + i] = hs[4 * j + t][i] * yk;
          b = fmaf(g, r[i], b);
          gc[i] = g * as[4 * j + t][i];
          const float kk = gc[i] * prev;
          dA[i] = fmaf(kk, dk, dA[i]);
          d = fmaf(kk, A2[i], d);
        }
        sb[K] = b;
        sa[K] = d;
        channel_sums<NV>(v, lane);
        if (writer)
#pragma unroll
          for (int i = 0; i < LEFT; ++i) red[buf][wave][4 * j + K][q][vat + i] = v[i];
      };
      token(std::integral_constant<int, 3>{});
      token(std::integral_constant<int, 2>{});
      token(std::integral_constant<int, 1>{});
      token(std::integral_constant<int, 0>{});
      const float b = lane_sums<4>(sb, lane), d = lane_sums<4>(sa, lane) * (1.f / kLog2E);
      if (live && k * CT + 4 * j + q < len) {
        const int64_t o = (row0 + k * CT + 4 * j + q) * a.D + c;
        Elem<T>::store(a.dx, o, fmaf(dl[j], b, skip * dyp[j]));
        float dd = fmaf(xv[j], b, d);
        if (a.softplus) dd *= sigmoid_fast(ud[j]);
        Elem<T>::store(a.ddt, o, dd);
        dbias += dd;
        dskip = fmaf(dyp[j], xv[j], dskip);
        if (a.z) {
          const float s = sigmoid_fast(zv[j]);
          Elem<T>::store(a.dz, o, yv[j] * fmaf(skip, xv[j], yr[j]) * (s * fmaf(zv[j], 1.f - s, 1.f)));
        }
      }
    }
    __syncthreads();  // the other buffer is written again only behind the next one
    for (int e = tid; e < CT * 2 * SP; e += kScanBlock) {
      const int t = e / (2 * SP), which = (e / SP) & 1, s = e % SP;
      if (k * CT + t < len) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) v += red[buf][w][t][s / NPL][which * NPL + s % NPL];
        const int64_t row = row0 + k * CT + t, rows = static_cast<int64_t>(a.cu ? 1 : a.N) * a.T_;
        a.dBCpart[((cbg * rows + row) * a.G + p.g) * (2 * SP) + which * SP + s] = v;
      }
    }
  }
  if (!live) return;
#pragma unroll
  for (int i = 0; i < NPL; ++i) a.dApart[at + i] = dA[i];
  dskip = lane_total<4>(dskip);
  dbias = lane_total<4>(dbias);
  if (q == 0) {
    a.dDpart[dpart] = dskip;
    a.dDpart[dpart + a.D] = dbias;
  }
}

// dB and dC: the partial sums of the group's channel blocks, added in order and rounded once.
// Tokens of no sequence are left alone.
template <typename T>
__global__ __launch_bounds__(kScanBlock) void scan_bwd_bc_kernel(const float* __restrict__ part, const int32_t* __restrict__ cu,
                                                                 int N, int64_t rows, int G, int S, int SP, int blocks,
                                                                 T* __restrict__ dB, T* __restrict__ dC) {
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kScanBlock + threadIdx.x, per = rows * G * 2 * SP;
  if (id >= per) return;
  const int s = static_cast<int>(id % SP), which = static_cast<int>(id / SP) & 1;
  const int64_t rg = id / (2 * SP);
  if (s >= S) return;
  if (cu) {
    const int64_t t = rg / G;
    if (t < cu[0] || t >= cu[N]) return;
  }
  float v = 0.f;
#pragma unroll 4
  for (int b = 0; b < blocks; ++b) v += part[b * per + id];
  Elem<T>::store(which ? dC : dB, rg * S + s, v);
}

int64_t scan_bwd_channel_blocks(int64_t D, int64_t G) { return G * ((D / G + kScanChannels - 1) / kScanChannels); }

ScanPlan scan_bwd_plan(int64_t B, int64_t T, int64_t N, int S, bool packed) {
  const int npl = scan_padded_states(S) / 4;
  const int L = npl <= 4 ? BwdTile<4>::L : npl == 8 ? BwdTile<8>::L : BwdTile<16>::L;
  static_assert(BwdTile<2>::L == BwdTile<4>::L, "one segment length up to 16 states");
  return ScanPlan{L, packed ? T / L + N + 1 : B * ((T + L - 1) / L)};
}

template <typename T, int NPL>
static hipError_t scan_bwd_t(const ScanBwdArgs& a, const ScanPlan& p, hipStream_t st) {
  const ScanArgs& f = a.f;
  constexpr int SP = 4 * NPL;
  const ScanBwdK<T> k{static_cast<const T*>(f.x), static_cast<const T*>(f.dt), f.A, static_cast<const T*>(f.Bm),
                      static_cast<const T*>(f.Cm), f.skip, static_cast<const T*>(f.z), f.dt_bias, f.init, f.cu_seqlens,
                      static_cast<const T*>(a.dy), a.dfin, static_cast<T*>(a.dx), static_cast<T*>(a.ddt),
                      static_cast<T*>(a.dz), a.dinit, a.hseg, a.gseg, a.dsum, a.dApart, a.dDpart, a.dBCpart,
                      f.N, f.T, f.D, f.S, f.G, p.L, f.softplus};
  const int64_t cb = scan_bwd_channel_blocks(f.D, f.G), rows = static_cast<int64_t>(f.B) * f.T;
  const unsigned grid = static_cast<unsigned>(p.slots * cb);
  hipError_t e;
  scan_bwd_ends_kernel<T, NPL><<<grid, kScanBlock, 0, st>>>(k);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const int64_t threads = static_cast<int64_t>(f.N) * f.D * SP;
  scan_bwd_carry_kernel<<<dim3(static_cast<unsigned>((threads + kScanBlock - 1) / kScanBlock), 2), kScanBlock, 0, st>>>(
      f.A, f.init, a.dfin, f.cu_seqlens, f.N, f.T, f.D, f.S, SP, p.L, a.hseg, a.gseg, a.dsum, a.dinit);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  scan_bwd_kernel<T, NPL><<<grid, kScanBlock, 0, st>>>(k);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (rows > 0) {
    const int64_t n = rows * f.G * 2 * SP;
    scan_bwd_bc_kernel<T><<<static_cast<unsigned>((n + kScanBlock - 1) / kScanBlock), kScanBlock, 0, st>>>(
        a.dBCpart, f.cu_seqlens, f.N, rows, f.G, f.S, SP, static_cast<int>(cb / f.G), static_cast<T*>(a.dBm),
        static_cast<T*>(a.dCm));
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  float* dA = a.dA;
  const int S = f.S;
  e = column_sums(a.dApart, p.slots, static_cast<int64_t>(f.D) * SP, f.D * SP, st, [=] __device__(int col, float v) {
    if (col % SP < S) dA[static_cast<int64_t>(col / SP) * S + col % SP] = v;
  });
  if (e != hipSuccess) return e;
  float* dk = a.dskip;
  float* db = a.ddt_bias;
  if (!dk && !db) return hipSuccess;
  const int D = f.D;
  return column_sums(a.dDpart, p.slots, 2 * static_cast<int64_t>(D), 2 * D, st, [=] __device__(int col, float v) {
    if (col < D) {
      if (dk) dk[col] = v;
    } else if (db) {
      db[col - D] = v;
    }
  });
}

hipError_t launch_scan_bwd(const ScanBwdArgs& a, const ScanPlan& p, hipStream_t st) {
  auto run = [&](auto npl) {
    constexpr int NPL = decltype(npl)::value;
    return a.f.dtype == COMBA_BF16 ? scan_bwd_t<u16, NPL>(a, p, st) : scan_bwd_t<float, NPL>(a, p, st);
  };
  switch (scan_padded_states(a.f.S)) {
    case 8: return run(std::integral_constant<int, 2>{});
    case 16: return run(std::integral_constant<int, 4>{});
    case 32: return run(std::integral_constant<int, 8>{});
    default: return run(std::integral_constant<int, 16>{});
  }
}

}  // namespace comba
