// Selective state space scan: a diagonal linear recurrence per channel with S states, whose decay,
// input and output vary with the token. Per channel c of group g and state s:
//   d_t = softplus(dt_t + dt_bias)           (or dt_t + dt_bias)
//   h_t[s] = exp(d_t A[s]) h_{t-1}[s] + d_t x_t B_t[g, s]
//   y_t = (sum_s C_t[g, s] h_t[s] + skip x_t) z_t sigmoid(z_t)
// The state and all sums are float32; y is rounded once.
//
// Per (token, channel, state) one exponential, three multiplications and two fused multiply-adds
// against 8 / S bytes of HBM per state (bf16): at S = 16 the vector ALU is the bound, not HBM, and
// since A differs per channel and state no matrix product can take the work over. The kernel
// therefore keeps everything but those six instructions out of the inner loop: B and C as float32 in
// LDS, one 16-byte read per four of them; step sizes and gates formed once per (token, channel);
// sums over the states transposed over the quad, four tokens at a time.
//
// Parallel over sequences and channels; a batch with too few of them for the chip is cut along time
// into segments of L tokens (scan_plan): every segment's end state from 0, a pass that carries the
// true states across (the state map of a segment is h -> exp(A sum d) h + end), and the scan of every
// segment from its true state.
#include "comba.h"
#include "scan_common.h"

namespace comba {

constexpr int kScanTile = 32;  // tokens per LDS tile

template <typename T> struct ScanK {
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
  T* y;
  float* fin;
  float* hseg;
  float* dsum;
  int N, T_, D, S, G, L;
  bool softplus;
};

// States s0 .. s0 + NPL - 1 of a channel from a row of S (or SP) states.
template <int NPL>
__device__ __forceinline__ void load_states(const float* row, int s0, int S, float (&h)[NPL]) {
#pragma unroll
  for (int i = 0; i < NPL; ++i) h[i] = s0 + i < S ? row[s0 + i] : 0.f;
}
template <int NPL>
__device__ __forceinline__ void store_states(float* row, int s0, int S, const float (&h)[NPL]) {
#pragma unroll
  for (int i = 0; i < NPL; ++i)
    if (s0 + i < S) row[s0 + i] = h[i];
}

// One workgroup: 64 channels over one segment. STATE: only the segment's end state from 0 and its
// sum of step sizes, for the carry.
template <typename T, int NPL, bool STATE>
__global__ __launch_bounds__(kScanBlock) void scan_fwd_kernel(ScanK<T> a) {
  constexpr int SP = 4 * NPL, TT = kScanTile, Q = TT / 4;
  constexpr int PT = (TT * SP + kScanBlock - 1) / kScanBlock;  // B (and C) elements staged per thread
  __shared__ __align__(16) float bc[2][TT][4][2 * NPL];
  const int tid = threadIdx.x, lane = tid & 63, q = lane & 3;
  const int cblocks = a.G * ((a.D / a.G + kScanChannels - 1) / kScanChannels);
  const int cb = blockIdx.x % cblocks;
  const ScanPlace p = scan_place(blockIdx.x / cblocks, cb, a.cu, a.N, a.T_, a.D, a.G, a.L);
  if (!p.ok) return;
  if (STATE && p.t1 >= p.s1) return;  // nothing follows the last segment
  const int in = (tid >> 6) * 16 + (lane >> 2);
  const bool live = in < p.cl;
  const int c = p.c0 + (live ? in : p.cl - 1);

  float A2[NPL], h[NPL];
  load_states<NPL>(a.A + static_cast<int64_t>(c) * a.S, q * NPL, a.S, A2);
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    A2[i] *= kLog2E;
    h[i] = 0.f;
  }
  if (!STATE) {
    if (a.L) load_states<NPL>(a.hseg + (p.slot * a.D + c) * SP, q * NPL, SP, h);
    else if (a.init) load_states<NPL>(a.init + (static_cast<int64_t>(p.n) * a.D + c) * a.S, q * NPL, a.S, h);
  }
  const float bias = a.dt_bias ? a.dt_bias[c] : 0.f, skip = !STATE && a.skip ? a.skip[c] : 0.f;

  // Elements of the tile that starts at token t: the lane's own token of each group of four, and the
  // thread's share of B and C. Rows of the batch row: 32-bit offsets from the tile's first row.
  const int64_t row0 = static_cast<int64_t>(p.b) * a.T_;
  T rx[Q], rd[Q], rz[Q] = {}, rb[PT], rc[PT] = {};
  auto fetch = [&](int t) {
    const T* x = a.x + (row0 + t) * a.D;
    const T* d = a.dt + (row0 + t) * a.D;
    const T* z = a.z ? a.z + (row0 + t) * a.D : nullptr;
#pragma unroll
    for (int j = 0; j < Q; ++j) {
      const uint32_t o = static_cast<uint32_t>(min(4 * j + q, p.t1 - 1 - t)) * static_cast<uint32_t>(a.D) + c;
      rx[j] = x[o];
      rd[j] = d[o];
      if (!STATE && z) rz[j] = z[o];
    }
    const int64_t bo = ((row0 + t) * a.G + p.g) * a.S;
    const T* B = a.Bm + bo;
    const T* C = a.Cm + bo;
#pragma unroll
    for (int k = 0; k < PT; ++k) {
      const int e = tid + k * kScanBlock, tt = e / SP, s = e % SP;
      const bool have = tt < TT && t + tt < p.t1 && s < a.S;
      const uint32_t o = have ? static_cast<uint32_t>(tt) * a.G * a.S + s : 0u;
      rb[k] = have ? B[o] : T(0);
      if (!STATE) rc[k] = have ? C[o] : T(0);
    }
  };

  float dtot = 0.f;
  int buf = 0;
  if (p.t0 < p.t1) fetch(p.t0);
  for (int t = p.t0; t < p.t1; t += TT, buf ^= 1) {
#pragma unroll
    for (int k = 0; k < PT; ++k) {
      const int e = tid + k * kScanBlock, tt = e / SP, s = e % SP;
      if (tt < TT) {
        bc[buf][tt][s / NPL][s % NPL] = Elem<T>::load(&rb[k], 0);
        if (!STATE) bc[buf][tt][s / NPL][NPL + s % NPL] = Elem<T>::load(&rc[k], 0);
      }
    }
    T cx[Q], cd[Q], cz[Q];
#pragma unroll
    for (int j = 0; j < Q; ++j) {
      cx[j] = rx[j];
      cd[j] = rd[j];
      cz[j] = rz[j];
    }
    if (t + TT < p.t1) fetch(t + TT);
    __syncthreads();  // one barrier per tile: the other buffer is written again only behind the next one
#pragma unroll
    for (int j = 0; j < Q; ++j) {
      const int mine = t + 4 * j + q;
      const bool in_seg = mine < p.t1;
      const float xv = Elem<T>::load(&cx[j], 0);
      float dl = Elem<T>::load(&cd[j], 0) + bias;
      if (a.softplus) dl = softplus_f32(dl);
      if (!in_seg) dl = 0.f;                       // tokens behind the segment: decay 1, no input
      const float dx = in_seg ? dl * xv : 0.f;
      if (STATE) dtot += dl;
      float ys[4];
      auto token = [&](auto kc) {
        constexpr int K = decltype(kc)::value;
        const float dk = quad_bcast<K>(dl), xk = quad_bcast<K>(dx);
        const float* r = bc[buf][4 * j + K][q];
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
          const float e = __builtin_amdgcn_exp2f(dk * A2[i]);
          h[i] = fmaf(e, h[i], xk * r[i]);
          if (!STATE) y = fmaf(h[i], r[NPL + i], y);
        }
        ys[K] = y;
      };
      token(std::integral_constant<int, 0>{});
      token(std::integral_constant<int, 1>{});
      token(std::integral_constant<int, 2>{});
      token(std::integral_constant<int, 3>{});
      if (!STATE) {
        float y = fmaf(skip, xv, quad_sums(ys, q));
        if (a.z) {
          const float zv = Elem<T>::load(&cz[j], 0);
          y *= zv * sigmoid_fast(zv);
        }
        if (in_seg && live) Elem<T>::store(a.y + (row0 + t) * a.D, static_cast<uint32_t>(4 * j + q) * static_cast<uint32_t>(a.D) + c, y);
      }
    }
  }
  if (!live) return;
  if (STATE) {
    store_states<NPL>(a.hseg + (p.slot * a.D + c) * SP, q * NPL, SP, h);
    dtot = quad_total(dtot);
    if (q == 0) a.dsum[p.slot * a.D + c] = dtot;
  } else if (a.fin && p.t1 >= p.s1) {
    store_states<NPL>(a.fin + (static_cast<int64_t>(p.n) * a.D + c) * a.S, q * NPL, a.S, h);
  }
}

// Carries the states across the segments of a sequence, one thread per (sequence, channel, state):
// hseg goes from every segment's end state from 0 to its incoming state.
__global__ __launch_bounds__(kScanBlock) void scan_carry_kernel(const float* __restrict__ A, const float* __restrict__ init,
                                                                const int32_t* __restrict__ cu, int N, int T, int64_t D,
                                                                int S, int SP, int L, float* __restrict__ hseg,
                                                                const float* __restrict__ dsum) {
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kScanBlock + threadIdx.x;
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
  float h = real && init ? init[(n * D + c) * S + s] : 0.f;
  float* hp = hseg + (slot0 * D + c) * SP + s;
  const float* dp = dsum + slot0 * D + c;
  constexpr int U = 8;
  for (int k = 0; k < segs; k += U) {
    float end[U], d[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {  // the last segment has no end state
      const bool have = k + u < segs - 1;
      end[u] = have ? hp[(k + u) * D * SP] : 0.f;
      d[u] = have ? dp[(k + u) * D] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k + u < segs) hp[(k + u) * D * SP] = h;
      h = fmaf(__builtin_amdgcn_exp2f(A2 * d[u]), h, end[u]);
    }
  }
}

// One token per sequence: the state is read once and written once, 8 S bytes per channel: bound by
// HBM. Lanes as above; a workgroup takes several sequences, with A in registers.
template <typename T, int NPL, bool V>
__global__ __launch_bounds__(kScanBlock) void scan_step_kernel(
    const T* __restrict__ x, const T* __restrict__ dt, const float* __restrict__ A, const T* __restrict__ Bm,
    const T* __restrict__ Cm, const float* __restrict__ skip, const T* __restrict__ z, const float* __restrict__ dt_bias,
    bool softplus, const float* init, int N, int64_t D, int S, int G, int per, T* __restrict__ y, float* fin) {
  const int lane = threadIdx.x & 63, q = lane & 3;
  const int cblocks = G * ((static_cast<int>(D) / G + kScanChannels - 1) / kScanChannels);
  const ScanPlace p = scan_place(0, blockIdx.x % cblocks, nullptr, 1, 1, static_cast<int>(D), G, 0);
  const int in = (threadIdx.x >> 6) * 16 + (lane >> 2);
  if (in >= p.cl) return;
  const int c = p.c0 + in, s0 = q * NPL;
  float A2[NPL];
  load_states<NPL>(A + static_cast<int64_t>(c) * S, s0, S, A2);
#pragma unroll
  for (int i = 0; i < NPL; ++i) A2[i] *= kLog2E;
  const float bias = dt_bias ? dt_bias[c] : 0.f, sk = skip ? skip[c] : 0.f;
  const int64_t first = static_cast<int64_t>(blockIdx.x / cblocks) * per;
  for (int64_t n = first; n < first + per && n < N; ++n) {
    float h[NPL];
    const int64_t at = (n * D + c) * S;
    if (!init) {
#pragma unroll
      for (int i = 0; i < NPL; ++i) h[i] = 0.f;
    } else if constexpr (V) {
#pragma unroll
      for (int i = 0; i < NPL; i += 4) {
        const f32x4 v = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(init + at + s0 + i));
        h[i] = v[0]; h[i + 1] = v[1]; h[i + 2] = v[2]; h[i + 3] = v[3];
      }
    } else {
      load_states<NPL>(init + at, s0, S, h);
    }
    const float xv = Elem<T>::load(x, n * D + c);
    float dl = Elem<T>::load(dt, n * D + c) + bias;
    if (softplus) dl = softplus_f32(dl);
    const float dx = dl * xv;
    const T* B = Bm + (n * G + p.g) * S;
    const T* C = Cm + (n * G + p.g) * S;
    float o = 0.f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const bool have = V || s0 + i < S;
      const float b = have ? Elem<T>::load(B, s0 + i) : 0.f, cc = have ? Elem<T>::load(C, s0 + i) : 0.f;
      h[i] = fmaf(__builtin_amdgcn_exp2f(dl * A2[i]), h[i], dx * b);
      o = fmaf(h[i], cc, o);
    }
    o = fmaf(sk, xv, quad_total(o));
    if (z) {
      const float zv = Elem<T>::load(z, n * D + c);
      o *= zv * sigmoid_fast(zv);
    }
    if (q == 0) Elem<T>::store(y, n * D + c, o);
    if (fin) {
      if constexpr (V) {
#pragma unroll
        for (int i = 0; i < NPL; i += 4)
          __builtin_nontemporal_store(f32x4{h[i], h[i + 1], h[i + 2], h[i + 3]},
                                      reinterpret_cast<f32x4*>(fin + at + s0 + i));
      } else {
        store_states<NPL>(fin + at, s0, S, h);
      }
    }
  }
}

// --- launches -----------------------------------------------------------------------------------

int scan_padded_states(int S) {
  int sp = 4;
  while (sp < S) sp *= 2;
  return sp;
}

int64_t scan_channel_blocks(int64_t D, int64_t G) { return G * ((D / G + kScanChannels - 1) / kScanChannels); }

// Cutting costs a second pass over the inputs and the exponentials (about 3/4 of a scan), so it pays
// where less than half of the 256 compute units would have a workgroup. Segments then make about
// 1024 workgroups (a wavefront per SIMD four times over), of 256 tokens at least. In a packed batch
// the lengths are unknown here: no sequence may run longer than the whole batch's share of a
// compute unit, at least 512 tokens.
ScanPlan scan_plan(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N, bool packed) {
  const int64_t cb = scan_channel_blocks(D, G);
  int64_t L;
  if (packed) {
    L = T * cb / 256;
    L = L < 512 ? 512 : L;
  } else {
    if (B * cb > 128) return ScanPlan{0, N};
    L = B * T * cb / 1024;
    L = L < 256 ? 256 : L;
  }
  L = (L + kScanTile - 1) / kScanTile * kScanTile;
  if (L >= T) return ScanPlan{0, N};
  return ScanPlan{static_cast<int>(L), packed ? T / L + N + 1 : B * ((T + L - 1) / L)};
}

template <typename T, int NPL>
static hipError_t scan_t(const ScanArgs& a, const ScanPlan& p, float* hseg, float* dsum, hipStream_t st) {
  const ScanK<T> k{static_cast<const T*>(a.x), static_cast<const T*>(a.dt), a.A, static_cast<const T*>(a.Bm),
                   static_cast<const T*>(a.Cm), a.skip, static_cast<const T*>(a.z), a.dt_bias, a.init, a.cu_seqlens,
                   static_cast<T*>(a.y), a.fin, hseg, dsum, a.N, a.T, a.D, a.S, a.G, p.L, a.softplus};
  const int64_t cb = scan_channel_blocks(a.D, a.G);
  const unsigned grid = static_cast<unsigned>(p.slots * cb);
  if (p.L) {
    scan_fwd_kernel<T, NPL, true><<<grid, kScanBlock, 0, st>>>(k);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t threads = static_cast<int64_t>(a.N) * a.D * 4 * NPL;
    scan_carry_kernel<<<static_cast<unsigned>((threads + kScanBlock - 1) / kScanBlock), kScanBlock, 0, st>>>(
        a.A, a.init, a.cu_seqlens, a.N, a.T, a.D, a.S, 4 * NPL, p.L, hseg, dsum);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  scan_fwd_kernel<T, NPL, false><<<grid, kScanBlock, 0, st>>>(k);
  return hipGetLastError();
}

template <typename T, int NPL>
static hipError_t scan_step_t(const ScanArgs& a, hipStream_t st) {
  const int64_t cb = scan_channel_blocks(a.D, a.G);
  // sequences per workgroup: up to 8 while eight workgroups per compute unit remain
  int64_t per = a.N * cb / 2048;
  per = per < 1 ? 1 : (per > 8 ? 8 : per);
  const unsigned grid = static_cast<unsigned>((a.N + per - 1) / per * cb);
  auto run = [&](auto v) {
    scan_step_kernel<T, NPL, decltype(v)::value><<<grid, kScanBlock, 0, st>>>(
        static_cast<const T*>(a.x), static_cast<const T*>(a.dt), a.A, static_cast<const T*>(a.Bm),
        static_cast<const T*>(a.Cm), a.skip, static_cast<const T*>(a.z), a.dt_bias, a.softplus, a.init, a.N, a.D, a.S,
        a.G, static_cast<int>(per), static_cast<T*>(a.y), a.fin);
    return hipGetLastError();
  };
  if constexpr (NPL % 4 == 0) {
    const bool v = a.S == 4 * NPL && (reinterpret_cast<uintptr_t>(a.init) & 15) == 0 &&
                   (reinterpret_cast<uintptr_t>(a.fin) & 15) == 0;
    if (v) return run(std::true_type{});
  }
  return run(std::false_type{});
}

template <typename F>
static hipError_t with_states(int S, F f) {
  if (S <= 4) return f(std::integral_constant<int, 1>{});
  if (S <= 8) return f(std::integral_constant<int, 2>{});
  if (S <= 16) return f(std::integral_constant<int, 4>{});
  if (S <= 32) return f(std::integral_constant<int, 8>{});
  return f(std::integral_constant<int, 16>{});
}

hipError_t launch_scan(const ScanArgs& a, const ScanPlan& p, float* hseg, float* dsum, hipStream_t st) {
  return with_states(a.S, [&](auto npl) {
    constexpr int NPL = decltype(npl)::value;
    return a.dtype == COMBA_BF16 ? scan_t<u16, NPL>(a, p, hseg, dsum, st) : scan_t<float, NPL>(a, p, hseg, dsum, st);
  });
}

hipError_t launch_scan_step(const ScanArgs& a, hipStream_t st) {
  return with_states(a.S, [&](auto npl) {
    constexpr int NPL = decltype(npl)::value;
    return a.dtype == COMBA_BF16 ? scan_step_t<u16, NPL>(a, st) : scan_step_t<float, NPL>(a, st);
  });
}

}  // namespace comba
