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
//      gradient behind it, and its sum of step sizes (the map of both is exp(A sum d)); a second time for
//      the gradients where the decays' product overflowed, as growing states make it;
//   2. scan_bwd_carry: the true incoming states and outgoing gradients, along the segments;
//   3. scan_bwd: per segment the states at every CT-th token forward, then from its end the CT tokens
//      of each piece: states and decays recomputed into registers, then the reverse recurrence;
//   4. scan_bwd_sums: over segments (dA, dskip, ddt_bias) and over channel blocks (dB, dC), in a fixed
//      order.
// Where no sequence can be longer than a segment (T <= L), 3 starts from the given states itself and
// writes d_initial_state: two launches instead of four, which is what a short batch's time is made of.
// Nothing is kept from the forward. Bound by the vector ALU like the forward: three exponentials and
// 38 instructions per (token, channel, state), 9 of them in 1 and 29 in 3. The sums over the 16 channels of a wavefront
// halve the values at every step. Through LDS instead (terms written, one sum per lane read back) the
// vector ALU has 12 % less to do, but the kernel waits for LDS longer than that: 316 us against 300 at
// B = 4, T = 2048, D = 2048, S = 16.
// Measured there, bf16, once the clock has settled: 356 to 369 us in all: 76 (1), 10 (2), 271 (3), 8.5 (4);
// in fp32 367 to 375. 8 x 4096 tokens 1370 us. 4 x 2048 tokens of 1024 channels with 32 states 506 us, with 64,
// at one wavefront per SIMD, 1370; of 2048 channels with 8 states 220 (two registers spilled for a
// third wavefront). The vector ALU is busy 79 to 83 % of 3's time, at two wavefronts per SIMD (240 registers: 16 tokens'
// states and decays; 61 KB of LDS). HBM moves 0.33 GB in 3.
#include <utility>

#include "column_sums.h"
#include "comba.h"
#include "scan_common.h"

namespace comba {

template <int NPL> struct BwdTile {
  static constexpr int CT = NPL <= 4 ? 16 : 64 / NPL;        // tokens whose states are held in registers
  static constexpr int NSUB = NPL <= 8 ? 8 : 4;              // pieces of CT tokens in the longest segment
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
  bool whole;  // no sequence is cut
};

// Sums v over the 16 channels of the wavefront (lane bits 2 .. 5). At lane bit 3, 2, 5, 4 a lane keeps
// the lower half of its values if the bit is clear, the upper half if it is set, while there are two
// or more; then all lanes add. Left: v[0 .. max(1, N/16) - 1]. The most values go through bits 3 and
// 2: 8 cycles a result there, 13 with a swap (4 x 2048 x 2048 x 16, all kernels: 373 -> 357 us).
template <int N>
__device__ __forceinline__ void channel_sums(float* v) {
  static_assert(N >= 4, "two states per lane at the least");
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
  constexpr int H2 = N / 4, H5 = H2 >= 2 ? H2 / 2 : 1, H4 = H5 >= 2 ? H5 / 2 : 1;
  halve_bits_3_2<H2>(v);
#pragma unroll
  for (int i = 0; i < H5; ++i) v[i] = swap_add(v[i], v[H2 >= 2 ? i + H5 : i], std::true_type{});
#pragma unroll
  for (int i = 0; i < H4; ++i) v[i] = swap_add(v[i], v[H5 >= 2 ? i + H4 : i], std::false_type{});
}

// Index of the first value that channel_sums<N> leaves in this lane. Lanes that differ in the bits
// behind the last halving hold the same value.
template <int N>
__device__ __forceinline__ int channel_sum_index(int lane) {
  constexpr int order[4] = {3, 2, 5, 4};
  int at = 0, n = N;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (n < 2) break;
    n /= 2;
    at += ((lane >> order[k]) & 1) * n;
  }
  return at;
}

// A piece of TT tokens for the 64 channels of a workgroup, worked on per (token, channel) with a lane
// per channel: thread (tk, ch) has tokens tk, tk + 4, ... of channel ch. Tokens behind the segment
// and channels behind the group's last read 0 and store nowhere.
template <typename T, int TT> struct Piece {
  static constexpr int R = TT / 4;
  uint32_t own[R];
  uint32_t rx[R], rd[R], rz[R], ry[R];
  float bias;
  int tk, ch;
  bool live;

  __device__ __forceinline__ void place(const ScanBwdK<T>& a, const ScanPlace& p) {
    ch = threadIdx.x % kScanChannels;
    tk = threadIdx.x / kScanChannels;
    live = ch < p.cl;
    const int c = p.c0 + (live ? ch : p.cl - 1);
    bias = a.dt_bias ? a.dt_bias[c] : 0.f;
#pragma unroll
    for (int j = 0; j < R; ++j)
      own[j] = live ? (static_cast<uint32_t>(tk + 4 * j) * a.D + c) * static_cast<uint32_t>(sizeof(T)) : kNowhere;
  }
  // The rows of the piece that starts at token t of the segment, as a range of `base`.
  static __device__ __forceinline__ Range<T> rows(const T* base, const ScanBwdK<T>& a, const ScanPlace& p, int t) {
    const int n = max(0, min(TT, p.t1 - p.t0 - t));
    return Range<T>(base + (base ? (static_cast<int64_t>(p.b) * a.T_ + p.t0 + t) * a.D : 0),
                    base ? static_cast<int64_t>(n) * a.D * sizeof(T) : 0);
  }
  template <bool ALL> __device__ __forceinline__ void fetch(const ScanBwdK<T>& a, const ScanPlace& p, int t) {
    const Range<T> x = rows(a.x, a, p, t), d = rows(a.dt, a, p, t);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      rx[j] = x.load(own[j]);
      rd[j] = d.load(own[j]);
    }
    if constexpr (ALL) {
      const Range<T> z = rows(a.z, a, p, t), y = rows(a.dy, a, p, t);
#pragma unroll
      for (int j = 0; j < R; ++j) {
        rz[j] = z.load(own[j]);
        ry[j] = y.load(own[j]);
      }
    }
  }
  __device__ __forceinline__ float step(const ScanBwdK<T>& a, const ScanPlace& p, int t, int j) const {
    const float u = Range<T>::value(rd[j]) + bias;
    float d = softplus_f32(u);
    pin(d);
    d = a.softplus ? d : u;
    return live && t + tk + 4 * j < p.t1 - p.t0 ? d : 0.f;  // elsewhere: decay 1, no input
  }
  // dy z sigmoid(z), the gradient of the ungated y; s: sigmoid(z)
  __device__ __forceinline__ float grad(const ScanBwdK<T>& a, int j, float& s) const {
    const float y = Range<T>::value(ry[j]), z = Range<T>::value(rz[j]);
    s = sigmoid_fast(z);
    float g = z * s;
    pin(g);
    return a.z ? y * g : y;
  }
};

// The piece's B and C: the thread's elements (token, state), 0 where there is none.
template <typename T, int TT, int SP> struct PieceBC {
  static constexpr int PT = (TT * SP + kScanBlock - 1) / kScanBlock;
  uint32_t off[PT], rb[PT], rc[PT];
  __device__ __forceinline__ void place(const ScanBwdK<T>& a) {
#pragma unroll
    for (int k = 0; k < PT; ++k) {
      const int e = threadIdx.x + k * kScanBlock, t = e / SP, s = e % SP;
      off[k] = t < TT && s < a.S ? (static_cast<uint32_t>(t) * a.G * a.S + s) * static_cast<uint32_t>(sizeof(T)) : kNowhere;
    }
  }
  __device__ __forceinline__ void fetch(const ScanBwdK<T>& a, const ScanPlace& p, int t) {
    const int n = max(0, min(TT, p.t1 - p.t0 - t));
    const int64_t at = ((static_cast<int64_t>(p.b) * a.T_ + p.t0 + t) * a.G + p.g) * a.S;
    const int64_t bytes = n ? (static_cast<int64_t>(n - 1) * a.G * a.S + a.S) * sizeof(T) : 0;
    const Range<T> B(a.Bm + at, bytes), C(a.Cm + at, bytes);
#pragma unroll
    for (int k = 0; k < PT; ++k) {
      rb[k] = B.load(off[k]);
      rc[k] = C.load(off[k]);
    }
  }
  // [token][quad lane][NPL of B, NPL of C]
  template <int NPL> __device__ __forceinline__ void put(float (*bc)[4][2 * NPL]) const {
#pragma unroll
    for (int k = 0; k < PT; ++k) {
      const int e = threadIdx.x + k * kScanBlock, t = e / SP, s = e % SP;
      if (PT * kScanBlock == TT * SP || t < TT) {
        bc[t][s / NPL][s % NPL] = Range<T>::value(rb[k]);
        bc[t][s / NPL][NPL + s % NPL] = Range<T>::value(rc[k]);
      }
    }
  }
};

template <typename T, int NPL>
__global__ __launch_bounds__(kScanBlock) void scan_bwd_ends_kernel(ScanBwdK<T> a) {
  constexpr int SP = 4 * NPL, TT = BwdTile<NPL>::CT;
  __shared__ __align__(16) float bc[2][TT][4][2 * NPL];
  __shared__ __align__(16) f32x4 st[2][TT][kScanChannels];  // step size, input, gradient of y
  __shared__ float tot[4][kScanChannels];
  const int tid = threadIdx.x, lane = tid & 63, q = lane & 3;
  const int cblocks = a.G * ((a.D / a.G + kScanChannels - 1) / kScanChannels);
  const ScanPlace p = scan_place<kScanChannels>(blockIdx.x / cblocks, blockIdx.x % cblocks, a.cu, a.N, a.T_, a.D, a.G, a.L);
  if (!p.ok) return;
  Piece<T, TT> pc;
  pc.place(a, p);
  PieceBC<T, TT, SP> pb;
  pb.place(a);
  pc.template fetch<true>(a, p, 0);
  pb.fetch(a, p, 0);
  const int in = tid / 4;
  const bool live = in < p.cl;
  const int c = p.c0 + (live ? in : p.cl - 1);
  float A2[NPL], h[NPL], gs[NPL], pr[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int s = q * NPL + i;
    A2[i] = s < a.S ? decay_rate(a.A[static_cast<int64_t>(c) * a.S + s]) : 0.f;
    h[i] = gs[i] = 0.f;
    pr[i] = 1.f;
  }
  const int len = p.t1 - p.t0;
  float dtot = 0.f;
  // Stages the segment piece by piece, the first one fetched before, and calls tokens(buffer) for each.
  auto pieces = [&](auto tokens) {
    for (int t = 0, buf = 0; t < len; t += TT, buf ^= 1) {
#pragma unroll
      for (int j = 0; j < pc.R; ++j) {
        float s;
        const float d = pc.step(a, p, t, j), g = pc.grad(a, j, s);
        dtot += d;
        st[buf][pc.tk + 4 * j][pc.ch] = f32x4{d, d * Range<T>::value(pc.rx[j]), g, 0.f};
      }
      pb.template put<NPL>(bc[buf]);
      pc.template fetch<true>(a, p, t + TT);
      pb.fetch(a, p, t + TT);
      __syncthreads();  // the other buffer is written only behind the next one
      tokens(buf);
    }
  };
  pieces([&](int buf) {
#pragma unroll
    for (int k = 0; k < TT; ++k) {
      const f32x4 e4 = st[buf][k][in];
      const float* r = bc[buf][k][q];
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        const float e = __builtin_amdgcn_exp2f(e4[0] * A2[i]);
        h[i] = fmaf(e, h[i], e4[1] * r[i]);
        pr[i] *= e;
        gs[i] = fmaf(pr[i], e4[2] * r[NPL + i], gs[i]);
      }
      if (k % 4 == 3)
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
          pin(h[i]);
          pin(gs[i]);
        }
    }
  });
  tot[pc.tk][pc.ch] = dtot;
  bool over = false;
#pragma unroll
  for (int i = 0; i < NPL; ++i) over |= !(pr[i] < INFINITY);
  over = __syncthreads_or(over);
  if (tid < kScanChannels && pc.live)
    a.dsum[p.slot * a.D + p.c0 + tid] = (tot[0][tid] + tot[1][tid]) + (tot[2][tid] + tot[3][tid]);
  const int64_t at = (p.slot * a.D + c) * SP + q * NPL;
  if (live)
#pragma unroll
    for (int i = 0; i < NPL; ++i) a.hseg[at + i] = h[i];
  if (over) {
    // A product of decays overflowed: a growing state. What it multiplies may be 0 or small enough for
    // a finite sum, so the sums are formed again with the products' exponents kept apart.
    int ex[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      gs[i] = 0.f;
      pr[i] = 1.f;
      ex[i] = 0;
    }
    pc.template fetch<true>(a, p, 0);
    pb.fetch(a, p, 0);
    pieces([&](int buf) {
#pragma unroll 1
      for (int k = 0; k < TT; ++k) {
        const f32x4 e4 = st[buf][k][in];
        const float* r = bc[buf][k][q];
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
          pr[i] *= __builtin_amdgcn_exp2f(e4[0] * A2[i]);
          ex[i] += __builtin_amdgcn_frexp_expf(pr[i]);
          pr[i] = __builtin_amdgcn_frexp_mantf(pr[i]);
          gs[i] += __builtin_amdgcn_ldexpf(pr[i] * (e4[2] * r[NPL + i]), ex[i]);
        }
      }
    });
  }
  if (live)
#pragma unroll
    for (int i = 0; i < NPL; ++i) a.gseg[at + i] = gs[i];
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
  const float A2 = real ? decay_rate(A[c * S + s]) : 0.f;
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
        h = carried(h, A2 * d[u], own[u]);
      }
    }
  }
  if (back && dinit && real) dinit[(n * D + c) * S + s] = h;
}

// Up to 8 states the registers are held to what three wavefronts per SIMD have.
template <typename T, int NPL>
__global__ __launch_bounds__(kScanBlock, NPL == 2 ? 3 : 1) void scan_bwd_kernel(ScanBwdK<T> a) {
  constexpr int SP = 4 * NPL, CT = BwdTile<NPL>::CT, NSUB = BwdTile<NPL>::NSUB;
  constexpr int NV = 2 * NPL;
  constexpr int LEFT = NV >= 16 ? NV / 16 : 1;
  __shared__ __align__(16) float bc[2][CT][4][NV];              // two pieces, then one
  __shared__ __align__(16) float held[NSUB][kScanBlock][NPL];   // states at the start of every piece
  __shared__ __align__(16) float red[4][CT][4][NV];             // dB, dC of a piece, per wavefront
  // Per (token, channel) of a piece: step size, input, gradient of y. The channel's quad replaces
  // them by what the token's thread needs: (sum g B, sum A k, , y).
  __shared__ __align__(16) f32x4 st[CT][kScanChannels];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, q = lane & 3;
  const int dg = a.D / a.G, per = (dg + kScanChannels - 1) / kScanChannels, cblocks = a.G * per;
  const int cb = blockIdx.x % cblocks;
  const ScanPlace p = scan_place<kScanChannels>(blockIdx.x / cblocks, cb, a.cu, a.N, a.T_, a.D, a.G, a.L);
  const int in = tid / 4;
  const bool live = in < p.cl;
  const int c = p.c0 + (live ? in : p.cl - 1);
  const int64_t at = (p.slot * a.D + c) * SP + q * NPL;
  if (!p.ok) {  // a slot between sequences adds nothing
    if (live) {
#pragma unroll
      for (int i = 0; i < NPL; ++i) a.dApart[at + i] = 0.f;
      if (q == 0) a.dDpart[p.slot * 2 * a.D + c] = a.dDpart[(p.slot * 2 + 1) * a.D + c] = 0.f;
    }
    return;
  }
  Piece<T, CT> pc;
  pc.place(a, p);
  PieceBC<T, CT, SP> pb;
  pb.place(a);
  pc.template fetch<false>(a, p, 0);
  pb.fetch(a, p, 0);
  float A2[NPL], h[NPL], gc[NPL], dA[NPL];  // gc: gradient that reaches the state before token t + 1
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int s = q * NPL + i;
    A2[i] = s < a.S ? decay_rate(a.A[static_cast<int64_t>(c) * a.S + s]) : 0.f;
    const int64_t given = (static_cast<int64_t>(p.n) * a.D + c) * a.S + s;
    if (a.whole) {
      h[i] = live && a.init && s < a.S ? a.init[given] : 0.f;
      gc[i] = live && a.dfin && s < a.S ? a.dfin[given] : 0.f;
    } else {
      h[i] = live ? a.hseg[at + i] : 0.f;
      gc[i] = live ? a.gseg[at + i] : 0.f;
    }
    dA[i] = 0.f;
  }
  const int lc = p.c0 + (pc.live ? pc.ch : p.cl - 1);
  const float skip = a.skip ? a.skip[lc] : 0.f;
  const int64_t row0 = static_cast<int64_t>(p.b) * a.T_ + p.t0;
  const int len = p.t1 - p.t0, nsub = (len + CT - 1) / CT;
  float dskip = 0.f, dbias = 0.f;

  // states at the start of every piece; the step sizes and inputs of two pieces share st
  f32x2(*sd)[CT][kScanChannels] = reinterpret_cast<f32x2(*)[CT][kScanChannels]>(&st[0][0]);
  for (int k = 0; k < nsub; ++k) {
#pragma unroll
    for (int i = 0; i < NPL; ++i) held[k][tid][i] = h[i];
    if (k == nsub - 1) break;
#pragma unroll
    for (int j = 0; j < pc.R; ++j) {
      const float d = pc.step(a, p, k * CT, j);
      sd[k & 1][pc.tk + 4 * j][pc.ch] = f32x2{d, d * Range<T>::value(pc.rx[j])};
    }
    pb.template put<NPL>(bc[k & 1]);
    pc.template fetch<false>(a, p, (k + 1) * CT);
    pb.fetch(a, p, (k + 1) * CT);
    __syncthreads();
#pragma unroll
    for (int t = 0; t < CT; ++t) {
      const f32x2 e2 = sd[k & 1][t][in];
      const float* r = bc[k & 1][t][q];
#pragma unroll
      for (int i = 0; i < NPL; ++i) h[i] = fmaf(__builtin_amdgcn_exp2f(e2[0] * A2[i]), h[i], e2[1] * r[i]);
      if (t % 4 == 3)
#pragma unroll
        for (int i = 0; i < NPL; ++i) pin(h[i]);
    }
  }

  const int vat = channel_sum_index<NV>(lane), cbg = cb - p.g * per;
  const int64_t rows = static_cast<int64_t>(a.cu ? 1 : a.N) * a.T_;
  pc.template fetch<true>(a, p, max(nsub - 1, 0) * CT);
  pb.fetch(a, p, max(nsub - 1, 0) * CT);
  for (int k = nsub - 1; k >= 0; --k) {
    __syncthreads();  // everything of the piece before is read
    pb.template put<NPL>(bc[0]);
    float xv[pc.R], uv[pc.R], zv[pc.R], yv[pc.R], dl[pc.R], dyp[pc.R], gz[pc.R];
#pragma unroll
    for (int j = 0; j < pc.R; ++j) {
      xv[j] = Range<T>::value(pc.rx[j]);
      uv[j] = Range<T>::value(pc.rd[j]) + pc.bias;
      zv[j] = Range<T>::value(pc.rz[j]);
      yv[j] = Range<T>::value(pc.ry[j]);
      dl[j] = pc.step(a, p, k * CT, j);
      dyp[j] = pc.grad(a, j, gz[j]);
      st[pc.tk + 4 * j][pc.ch] = f32x4{dl[j], dl[j] * xv[j], dyp[j], 0.f};
    }
    if (k > 0) {
      pc.template fetch<true>(a, p, (k - 1) * CT);
      pb.fetch(a, p, (k - 1) * CT);
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) h[i] = held[k][tid][i];
    __syncthreads();
    float hs[CT][NPL], as[CT][NPL];
#pragma unroll
    for (int j = 0; j < CT / 4; ++j) {
      float ys[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const f32x4 e4 = st[4 * j + t][in];
        const float* r = bc[0][4 * j + t][q];
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
          const float e = __builtin_amdgcn_exp2f(e4[0] * A2[i]);
          const float prev = (j || t) ? hs[4 * j + t - (j || t)][i] : h[i];
          as[4 * j + t][i] = e;
          hs[4 * j + t][i] = fmaf(e, prev, e4[1] * r[i]);
          y = i ? fmaf(hs[4 * j + t][i], r[NPL + i], y) : hs[4 * j + t][i] * r[NPL];
        }
        ys[t] = y;
      }
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < NPL; ++i) pin(hs[4 * j + t][i]);
      st[4 * j + q][in][3] = quad_sums(ys, lane);
    }
#pragma unroll
    for (int j = CT / 4 - 1; j >= 0; --j) {
      float sb[4], sa[4];
#pragma unroll
      for (int t = 3; t >= 0; --t) {
        const f32x4 e4 = st[4 * j + t][in];
        const float* r = bc[0][4 * j + t][q];
        float v[NV], b = 0.f, d = 0.f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
          const float g = fmaf(e4[2], r[NPL + i], gc[i]);
          const float prev = (j || t) ? hs[4 * j + t - (j || t)][i] : h[i];
          v[i] = g * e4[1];
          v[NPL + i] = hs[4 * j + t][i] * e4[2];
          b = i ? fmaf(g, r[i], b) : g * r[i];
          gc[i] = g * as[4 * j + t][i];
          const float kk = gc[i] * prev;
          dA[i] = fmaf(kk, e4[0], dA[i]);
          d = i ? fmaf(kk, A2[i], d) : kk * A2[i];
        }
        sb[t] = b;
        sa[t] = d;
        channel_sums<NV>(v);
#pragma unroll
        for (int i = 0; i < LEFT; ++i) red[wave][4 * j + t][q][vat + i] = v[i];
      }
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        pin(gc[i]);
        pin(dA[i]);
      }
      const float b = quad_sums(sb, lane), d = quad_sums(sa, lane) * (1.f / kLog2E);
      *reinterpret_cast<f32x2*>(&st[4 * j + q][in]) = f32x2{b, d};
    }
    __syncthreads();
    const Range<T> ox = Piece<T, CT>::rows(a.dx, a, p, k * CT), od = Piece<T, CT>::rows(a.ddt, a, p, k * CT),
                   oz = Piece<T, CT>::rows(a.dz, a, p, k * CT);
#pragma unroll
    for (int j = 0; j < pc.R; ++j) {
      const f32x4 e4 = st[pc.tk + 4 * j][pc.ch];
      ox.store(pc.own[j], fmaf(dl[j], e4[0], skip * dyp[j]));
      float dd = fmaf(xv[j], e4[0], e4[1]), s = sigmoid_fast(uv[j]);
      pin(s);
      dd = a.softplus ? dd * s : dd;
      od.store(pc.own[j], dd);
      oz.store(pc.own[j], yv[j] * fmaf(skip, xv[j], e4[3]) * (gz[j] * fmaf(zv[j], 1.f - gz[j], 1.f)));
      if (pc.live && k * CT + pc.tk + 4 * j < len) {
        dbias += dd;
        dskip = fmaf(dyp[j], xv[j], dskip);
      }
    }
    for (int e = tid; e < CT * 2 * SP; e += kScanBlock) {
      const int t = e / (2 * SP), which = (e / SP) & 1, s = e % SP;
      if (k * CT + t < len) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) v += red[w][t][s / NPL][which * NPL + s % NPL];
        a.dBCpart[((cbg * rows + row0 + k * CT + t) * a.G + p.g) * (2 * SP) + which * SP + s] = v;
      }
    }
  }
  // the four token groups' sums of a channel
  __syncthreads();
  st[pc.tk][pc.ch] = f32x4{dskip, dbias, 0.f, 0.f};
  __syncthreads();
  if (tid < kScanChannels && pc.live) {
    f32x4 t = st[0][tid];
#pragma unroll
    for (int w = 1; w < 4; ++w) t += st[w][tid];
    a.dDpart[p.slot * 2 * a.D + lc] = t[0];
    a.dDpart[(p.slot * 2 + 1) * a.D + lc] = t[1];
  }
  if (!live) return;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int s = q * NPL + i;
    a.dApart[at + i] = dA[i];
    if (a.whole && a.dinit && s < a.S) a.dinit[(static_cast<int64_t>(p.n) * a.D + c) * a.S + s] = gc[i];
  }
}

struct ScanSums {
  const float* dApart;
  const float* dDpart;
  const float* dBCpart;
  const int32_t* cu;
  float* dA;
  float* dskip;
  float* dbias;
  int64_t slots, rows;
  int N, D, S, SP, G, blocks;  // blocks: channel blocks of a group
};

constexpr int kSumThreads = kSumCols * kSumGroups;
static int64_t sum_blocks(int64_t columns) { return (columns + kSumCols - 1) / kSumCols; }

// One launch for all sums: the first workgroups take dA's columns, the next dskip's and ddt_bias's,
// the rest dB and dC, whose partial sums (one per channel block of the group) are added in order and
// rounded once. Tokens of no sequence are left alone.
template <typename T>
__global__ __launch_bounds__(kSumThreads) void scan_bwd_sums_kernel(ScanSums a, int ablocks, int dblocks, T* __restrict__ dB,
                                                                    T* __restrict__ dC) {
  int b = blockIdx.x;
  if (b < ablocks) {
    column_sums_block(a.dApart, a.slots, static_cast<int64_t>(a.D) * a.SP, a.D * a.SP, b, [&](int col, float v) {
      if (col % a.SP < a.S) a.dA[static_cast<int64_t>(col / a.SP) * a.S + col % a.SP] = v;
    });
    return;
  }
  b -= ablocks;
  if (b < dblocks) {
    column_sums_block(a.dDpart, a.slots, 2 * static_cast<int64_t>(a.D), 2 * a.D, b, [&](int col, float v) {
      float* to = col < a.D ? a.dskip : a.dbias;
      if (to) to[col < a.D ? col : col - a.D] = v;
    });
    return;
  }
  b -= dblocks;
  const int64_t id = static_cast<int64_t>(b) * kSumThreads + threadIdx.x, per = a.rows * a.G * 2 * a.SP;
  if (id >= per) return;
  const int s = static_cast<int>(id % a.SP), which = static_cast<int>(id / a.SP) & 1;
  const int64_t rg = id / (2 * a.SP);
  if (s >= a.S) return;
  if (a.cu) {
    const int64_t t = rg / a.G;
    if (t < a.cu[0] || t >= a.cu[a.N]) return;
  }
  float v = 0.f;
#pragma unroll 4
  for (int k = 0; k < a.blocks; ++k) v += a.dBCpart[k * per + id];
  Elem<T>::store(which ? dC : dB, rg * a.S + s, v);
}

int64_t scan_bwd_channel_blocks(int64_t D, int64_t G) { return G * ((D / G + kScanChannels - 1) / kScanChannels); }

// Segments are as long as LDS holds pieces of (128 tokens up to 16 states), shorter, down to one piece,
// where that leaves fewer than two workgroups per compute unit. At D = 2048, S = 16, bf16, with 128 /
// 64 / 32 / 16 tokens: 1 x 128 tokens 61 / 50 / 35 / 30 us, 1 x 1024 87 / 67 / 70 / 79, 1 x 4096
// 192 / 198 / 214 / 255; 1 x 500 of 512 channels 81 / 48 / 34 / 30.
ScanPlan scan_bwd_plan(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N, int S, bool packed) {
  const int npl = scan_padded_states(S) / 4;
  auto tile = [](auto t) { return std::pair<int64_t, int64_t>(decltype(t)::CT, decltype(t)::NSUB); };
  const auto [ct, most] = npl <= 4 ? tile(BwdTile<4>{}) : npl == 8 ? tile(BwdTile<8>{}) : tile(BwdTile<16>{});
  static_assert(BwdTile<2>::CT == BwdTile<4>::CT && BwdTile<2>::NSUB == BwdTile<4>::NSUB, "one length up to 16 states");
  const int64_t cb = scan_bwd_channel_blocks(D, G);
  int64_t L = ct * most;
  while (L > ct && (B * T / L + N) * cb < 512) L /= 2;
  return ScanPlan{static_cast<int>(L), packed ? T / L + N + 1 : B * ((T + L - 1) / L)};
}

template <typename T, int NPL>
static hipError_t scan_bwd_t(const ScanBwdArgs& a, const ScanPlan& p, hipStream_t st) {
  const ScanArgs& f = a.f;
  constexpr int SP = 4 * NPL;
  const ScanBwdK<T> k{static_cast<const T*>(f.x), static_cast<const T*>(f.dt), f.A, static_cast<const T*>(f.Bm),
                      static_cast<const T*>(f.Cm), f.skip, static_cast<const T*>(f.z), f.dt_bias, f.init, f.cu_seqlens,
                      static_cast<const T*>(a.dy), a.dfin, static_cast<T*>(a.dx), static_cast<T*>(a.ddt),
                      static_cast<T*>(a.dz), a.dinit, a.hseg, a.gseg, a.dsum, a.dApart, a.dDpart, a.dBCpart,
                      f.N, f.T, f.D, f.S, f.G, p.L, f.softplus, f.T <= p.L};
  const int64_t cb = scan_bwd_channel_blocks(f.D, f.G), rows = static_cast<int64_t>(f.B) * f.T;
  const unsigned grid = static_cast<unsigned>(p.slots * cb);
  hipError_t e;
  if (!k.whole) {
    scan_bwd_ends_kernel<T, NPL><<<grid, kScanBlock, 0, st>>>(k);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const int64_t threads = static_cast<int64_t>(f.N) * f.D * SP;
    scan_bwd_carry_kernel<<<dim3(static_cast<unsigned>((threads + kScanBlock - 1) / kScanBlock), 2), kScanBlock, 0, st>>>(
        f.A, f.init, a.dfin, f.cu_seqlens, f.N, f.T, f.D, f.S, SP, p.L, a.hseg, a.gseg, a.dsum, a.dinit);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  scan_bwd_kernel<T, NPL><<<grid, kScanBlock, 0, st>>>(k);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const ScanSums sums{a.dApart, a.dDpart, a.dBCpart, f.cu_seqlens, a.dA, a.dskip, a.ddt_bias, p.slots, rows,
                      f.N, f.D, f.S, SP, f.G, static_cast<int>(cb / f.G)};
  const int64_t ablocks = sum_blocks(static_cast<int64_t>(f.D) * SP), dblocks = sum_blocks(2ll * f.D);
  const int64_t bcblocks = (rows * f.G * 2 * SP + kSumThreads - 1) / kSumThreads;
  scan_bwd_sums_kernel<T><<<static_cast<unsigned>(ablocks + dblocks + bcblocks), kSumThreads, 0, st>>>(
      sums, static_cast<int>(ablocks), static_cast<int>(dblocks), static_cast<T*>(a.dBm), static_cast<T*>(a.dCm));
  return hipGetLastError();
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
