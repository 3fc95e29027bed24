// Selective state space scan: a diagonal linear recurrence per channel with S states, whose decay,
// input and output vary with the token. Per channel c of group g and state s:
//   d_t = softplus(dt_t + dt_bias)           (or dt_t + dt_bias)
//   h_t[s] = exp(d_t A[s]) h_{t-1}[s] + d_t x_t B_t[g, s]
//   y_t = (sum_s C_t[g, s] h_t[s] + skip x_t) z_t sigmoid(z_t)
// The state and all sums are float32; y is rounded once.
//
// Per (token, channel, state) one exponential, two multiplications and two fused multiply-adds
// against 8 / S bytes of HBM per state (bf16): at S = 16 the vector ALU is the bound, not HBM, and
// since A differs per channel and state no matrix product can take the work over. The kernel
// therefore keeps everything but those five instructions out of the inner loop: B, C, step sizes and
// inputs as float32 in LDS, formed once; sums over the states halved over the channel's lanes, eight
// tokens at a time.
//
// Measured, bf16, S = 16, D = 2048: 8 x 4096 tokens 350 to 357 us once the clock has settled, up to 380
// in the first fifty launches (3.0e12 states per second; HBM alone would take 87), 1 x 65536 tokens, cut,
// 882 to 945 us; 8 x 4096 with 4 states 281 us, with 16 in fp32 372. The uncut scan has the two wavefronts per
// SIMD that sequences and channels give, and the vector ALU is busy 75 to 78 % of the time; the cut one has four
// and runs at the rate of its instructions, 17.2 per token and wavefront: 10 of the recurrence, 2.1 of
// the sum over the lanes, 5 of the work per token. Not better: y summed by the matrix cores (16x16x4
// fp32 blocks hold the SIMD for 32 cycles each: 515 us against 421 then), the work per token spread
// between the recurrence's tokens, branches instead of selections in it (both flat).
//
// Parallel over sequences and channels; a batch with too few of them for the chip is cut along time
// into segments of L tokens (scan_plan): every segment's end state from 0, a pass that carries the
// true states across (the state map of a segment is h -> exp(A sum d) h + end), and the scan of every
// segment from its true state.
#include "comba.h"
#include "scan_common.h"

namespace comba {

// Tokens per LDS tile, channels per workgroup and lanes per channel of the forward. 32 channels make
// workgroups of four wavefronts whose phases do not line up, so that one's barrier and loads hide
// behind another's arithmetic; 8 lanes make twice the wavefronts of 4 for the same channels. Measured,
// all before the present sum over the lanes, at B = 8, T = 4096, D = 2048, S = 16, bf16 (8 lanes): 16 / 32 / 64 tokens 449 / 406 / 392 us at 32
// channels, 32 tokens at 16 / 64 channels 413 / 417 us; 4 lanes 595 us, 16 lanes (16 channels)
// 439 us. At B = 1, T = 65536, cut: 966 / 949 / 1028 us, 1055 / 952, 1140, 1089.
constexpr int kScanTile = 32, kFwdChannels = 32, kFwdLanes = 8;

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
  int64_t slots;
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

// v[k] summed over a channel's 8 lanes, lane bits 1 to 3, for the lane's own k: bits 3 and 2 are
// among them for their cheaper halvings (8 x 4096 x 2048 x 16: 387 -> 375 us, 1 x 65536: 913 -> 891).
__device__ __forceinline__ float lane_sums(float (&v)[8], int lane) {
  halve_bits_3_2<2>(v);
  halve_dpp<1, 1>(v, lane);
  return v[0];
}

// One workgroup: 32 channels over one segment. STATE: only the segment's end state from 0 and its
// sum of step sizes, for the carry.
//
// Work per (token, channel) is done with a lane per channel, so that loads and stores take pieces of
// rows: a thread forms the step size d and the input d x of its tokens and puts the pair into
// LDS. The recurrence then runs with 8 lanes per channel, which read the pair, B and C from there
// (a broadcast read costs the vector ALU nothing; taking them from a lane's register by DPP costs
// 5 to 7 cycles instead of 4 for every use), and leaves y, summed over the states, in LDS, where the
// channel's lane finds it behind the next barrier: one barrier per tile of TT tokens.
template <typename T, int NPL, bool STATE>
__global__ __launch_bounds__(kFwdChannels* kFwdLanes) void scan_fwd_kernel(ScanK<T> a) {
  constexpr int LPC = kFwdLanes, TT = kScanTile, CH = kFwdChannels, SP = LPC * NPL, TH = CH * LPC, TG = TH / CH, R = TT / TG;  // R: tokens per thread, TG apart
  constexpr int PT = (TT * SP + TH - 1) / TH;    // B (and C) elements staged per thread
  constexpr int YP = CH + 64 / LPC;              // row of y, padded: the tokens of a store hit different banks
  constexpr int AHEAD = NPL >= 16 ? 1 : 2;       // tokens read from LDS ahead
  __shared__ __align__(16) float bc[2][TT][LPC][STATE ? NPL : 2 * NPL];
  __shared__ __align__(16) f32x2 xd[2][TT][CH];
  __shared__ float yb[STATE ? 1 : 2][STATE ? 1 : TT][YP];
  const int tid = threadIdx.x, lane = tid & 63, q = (lane >> 1) & 7;
  // workgroups go round the 8 XCDs: neighbouring channels, which share lines, on one of them
  const int cblocks = a.G * ((a.D / a.G + CH - 1) / CH);
  const int per = (gridDim.x + 7) / 8, id = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  const int cb = id % cblocks;
  if (id >= a.slots * cblocks) return;
  const ScanPlace p = scan_place<CH>(id / cblocks, cb, a.cu, a.N, a.T_, a.D, a.G, a.L);
  if (!p.ok) return;
  if (STATE && p.t1 >= p.s1) return;  // nothing follows the last segment

  // the recurrence's channel and states
  const int in = tid / 64 * 8 + lane / 16 * 2 + (lane & 1);
  const bool live = in < p.cl;
  const int c = p.c0 + (live ? in : p.cl - 1);
  float A2[NPL], h[NPL];
  load_states<NPL>(a.A + static_cast<int64_t>(c) * a.S, q * NPL, a.S, A2);
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    A2[i] = decay_rate(A2[i]);
    h[i] = 0.f;
  }
  if (!STATE) {
    if (a.L) load_states<NPL>(a.hseg + (p.slot * a.D + c) * SP, q * NPL, SP, h);
    else if (a.init) load_states<NPL>(a.init + (static_cast<int64_t>(p.n) * a.D + c) * a.S, q * NPL, a.S, h);
  }

  // channel and first token for the work per token; threads behind the last channel read and write nowhere
  const int ch = tid % CH, tk = tid / CH;
  const bool have = ch < p.cl;
  const int lc = p.c0 + (have ? ch : p.cl - 1);
  const float bias = a.dt_bias ? a.dt_bias[lc] : 0.f, skip = !STATE && a.skip ? a.skip[lc] : 0.f;
  const bool gated = a.z != nullptr;
  const T* zp = gated ? a.z : a.x;  // without a gate x is loaded in its place, and not used
  const int64_t row0 = static_cast<int64_t>(p.b) * a.T_;
  uint32_t own[R], boff[PT];  // byte offsets from the tile's first row
#pragma unroll
  for (int j = 0; j < R; ++j)
    own[j] = have ? (static_cast<uint32_t>(tk + TG * j) * a.D + lc) * static_cast<uint32_t>(sizeof(T)) : kNowhere;
#pragma unroll
  for (int k = 0; k < PT; ++k) {
    const int e = tid + k * TH, tt = e / SP, s = e % SP;
    boff[k] = tt < TT && s < a.S ? (static_cast<uint32_t>(tt) * a.G * a.S + s) * static_cast<uint32_t>(sizeof(T)) : kNowhere;
  }
  uint32_t rx[R], rd[R], rz[R], rb[PT], rc[PT];
  auto fetch = [&](int t) {
    const int rows = max(0, min(TT, p.t1 - t));
    const int64_t at = (row0 + t) * a.D, bytes = static_cast<int64_t>(rows) * a.D * sizeof(T);
    const Range<T> x(a.x + at, bytes), d(a.dt + at, bytes), z(zp + at, STATE ? 0 : bytes);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      rx[j] = x.load(own[j]);
      rd[j] = d.load(own[j]);
      if (!STATE) rz[j] = z.load(own[j]);
    }
    const int64_t bat = ((row0 + t) * a.G + p.g) * a.S;
    const int64_t bbytes = rows ? (static_cast<int64_t>(rows - 1) * a.G * a.S + a.S) * sizeof(T) : 0;
    const Range<T> B(a.Bm + bat, bbytes), C(a.Cm + bat, STATE ? 0 : bbytes);
#pragma unroll
    for (int k = 0; k < PT; ++k) {
      rb[k] = B.load(boff[k]);
      if (!STATE) rc[k] = C.load(boff[k]);
    }
  };
  // The fetched elements become the next tile in LDS; x and the gate stay with the lane.
  float xv[R], zv[R], dtot = 0.f;
  auto stage = [&](int t, int buf) {
#pragma unroll
    for (int k = 0; k < PT; ++k) {
      const int e = tid + k * TH, tt = e / SP, s = e % SP;
      if (PT * TH == TT * SP || tt < TT) {
        bc[buf][tt][s / NPL][s % NPL] = Range<T>::value(rb[k]);
        if (!STATE) bc[buf][tt][s / NPL][NPL + s % NPL] = Range<T>::value(rc[k]);
      }
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
      xv[j] = Range<T>::value(rx[j]);
      const float u = Range<T>::value(rd[j]) + bias;
      float d = softplus_f32(u);
      pin(d);
      d = a.softplus ? d : u;
      if (t + tk + TG * j >= p.t1) d = 0.f;  // tokens behind the segment: decay 1, no input
      if (STATE) dtot += d;
      xd[buf][tk + TG * j][ch] = f32x2{d, d * xv[j]};
      if (!STATE) zv[j] = Range<T>::value(rz[j]);
    }
  };
  // Gate and store of the tile at t, whose y is complete in LDS; px, pz: its x and gate.
  auto finish = [&](int t, int buf, const float (&px)[R], const float (&pz)[R]) {
    const Range<T> out(a.y + (row0 + t) * a.D, static_cast<int64_t>(min(TT, p.t1 - t)) * a.D * sizeof(T));
#pragma unroll
    for (int j = 0; j < R; ++j) {
      float s = pz[j] * sigmoid_fast(pz[j]);
      pin(s);
      const float y = fmaf(skip, px[j], yb[buf][tk + TG * j][ch]);
      out.store(own[j], gated ? y * s : y);
    }
  };

  fetch(p.t0);
  stage(p.t0, 0);
  fetch(p.t0 + TT);
  int buf = 0;
  float px[R], pz[R];
  for (int t = p.t0; t < p.t1; t += TT, buf ^= 1) {
    __syncthreads();  // the tile is staged, the last one's y complete; the other buffers are free
    if (!STATE && t > p.t0) finish(t - TT, buf ^ 1, px, pz);
    if (!STATE)
#pragma unroll
      for (int j = 0; j < R; ++j) {
        px[j] = xv[j];
        pz[j] = zv[j];
      }
    // What the next AHEAD tokens need is read while the present ones are worked on: the scheduling
    // barrier keeps the compiler from moving the reads down to their use.
    f32x2 dn[AHEAD], dc[AHEAD];
    float bn[AHEAD][2 * NPL], bcur[AHEAD][2 * NPL];
    auto pull = [&](int tt) {
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        dn[k] = xd[buf][tt + k][in];
#pragma unroll
        for (int i = 0; i < (STATE ? NPL : 2 * NPL); ++i) bn[k][i] = bc[buf][tt + k][q][i];
      }
    };
    pull(0);
#pragma unroll
    for (int j = 0; j < TT / LPC; ++j) {
      float ys[LPC];
      each<LPC>([&](auto kc) {
        constexpr int K = decltype(kc)::value;
        if constexpr (K % AHEAD == 0) {
#pragma unroll
          for (int k = 0; k < AHEAD; ++k) {
            dc[k] = dn[k];
#pragma unroll
            for (int i = 0; i < (STATE ? NPL : 2 * NPL); ++i) bcur[k][i] = bn[k][i];
          }
          if (LPC * j + K + AHEAD < TT) pull(LPC * j + K + AHEAD);
          __builtin_amdgcn_sched_barrier(0);
        }
        const f32x2 dd = dc[K % AHEAD];
        const float(&r)[2 * NPL] = bcur[K % AHEAD];
        float o = 0.f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
          const float e = __builtin_amdgcn_exp2f(dd[0] * A2[i]);
          h[i] = fmaf(e, h[i], dd[1] * r[i]);
          if (!STATE) o = i ? fmaf(h[i], r[NPL + i], o) : h[i] * r[NPL];
        }
        if constexpr (K % AHEAD == AHEAD - 1)
#pragma unroll
          for (int i = 0; i < NPL; ++i) pin(h[i]);
        ys[K] = o;
      });
      if (!STATE) yb[buf][LPC * j + q][in] = lane_sums(ys, lane);
    }
    // Staged before the next tile's loads and behind no new store: the wait for the loads waits for
    // nothing else.
    stage(t + TT, buf ^ 1);
    fetch(t + 2 * TT);
  }
  if (!STATE && p.t0 < p.t1) {
    __syncthreads();
    finish(p.t0 + (p.t1 - 1 - p.t0) / TT * TT, buf ^ 1, px, pz);
  }
  if (STATE) {
    __shared__ float tot[TG][CH];
    tot[tk][ch] = dtot;
    __syncthreads();
    if (tk == 0 && have) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < TG; ++w) s += tot[w][ch];
      a.dsum[p.slot * a.D + lc] = s;
    }
    if (live) store_states<NPL>(a.hseg + (p.slot * a.D + c) * SP, q * NPL, SP, h);
  } else if (live && a.fin && p.t1 >= p.s1) {
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
  const float A2 = real ? decay_rate(A[c * S + s]) : 0.f;
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
      h = carried(h, A2 * d[u], end[u]);
    }
  }
}

// One token per sequence: the state is read once and written once, 8 S bytes per channel: bound by
// HBM. Four lanes per channel, a workgroup takes several sequences with A in registers, two
// sequences' loads in flight. Measured at D = 2048, S = 16, bf16, in place: 13.5 to 15 us for 256
// sequences (4.8 to 5.3 TB/s; 19.6 us with one sequence's loads in flight and B and C element by element),
// 101 to 117 us for 2048 (4.9 to 5.6 TB/s); 256 with 13 states, whose rows start anywhere, 16 us
// (24 element by element). States stored past the caches; loads that skip them too cost 16.8 us for 256.
template <typename T, int NPL>
__global__ __launch_bounds__(kScanBlock) void scan_step_kernel(
    const T* __restrict__ x, const T* __restrict__ dt, const float* __restrict__ A, const T* __restrict__ Bm,
    const T* __restrict__ Cm, const float* __restrict__ skip, const T* __restrict__ z, const float* __restrict__ dt_bias,
    bool softplus, const float* init, int N, int64_t D, int S, int G, int per, T* __restrict__ y, float* fin) {
  constexpr bool V = NPL % 4 == 0;  // a lane's states in 16-byte pieces, at any address of a float
  const int lane = threadIdx.x & 63, q = lane & 3;
  const int cblocks = G * ((static_cast<int>(D) / G + kScanChannels - 1) / kScanChannels);
  const ScanPlace p = scan_place<kScanChannels>(0, blockIdx.x % cblocks, nullptr, 1, 1, static_cast<int>(D), G, 0);
  const int in = (threadIdx.x >> 6) * 16 + (lane >> 2);
  if (in >= p.cl) return;
  const int c = p.c0 + in, s0 = q * NPL;
  const bool full = V && s0 + NPL <= S;
  float A2[NPL];
  load_states<NPL>(A + static_cast<int64_t>(c) * S, s0, S, A2);
#pragma unroll
  for (int i = 0; i < NPL; ++i) A2[i] = decay_rate(A2[i]);
  const float bias = dt_bias ? dt_bias[c] : 0.f, sk = skip ? skip[c] : 0.f;
  const int64_t first = static_cast<int64_t>(blockIdx.x / cblocks) * per;
  constexpr int U = 2;  // sequences whose loads are in flight together
  for (int64_t n0 = first; n0 < first + per && n0 < N; n0 += U) {
    float h[U][NPL], b[U][NPL], cc[U][NPL], xv[U], dl[U], zv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t n = min(n0 + u, static_cast<int64_t>(N) - 1), at = (n * D + c) * S;
      if (!init) {
#pragma unroll
        for (int i = 0; i < NPL; ++i) h[u][i] = 0.f;
      } else if (full) {
        if constexpr (V) Pack<float, NPL, true>::load(init + at + s0, h[u], NPL);
      } else {
        load_states<NPL>(init + at, s0, S, h[u]);
      }
      xv[u] = Elem<T>::load(x, n * D + c);
      dl[u] = Elem<T>::load(dt, n * D + c) + bias;
      zv[u] = z ? Elem<T>::load(z, n * D + c) : 0.f;
      const T* B = Bm + (n * G + p.g) * S + s0;
      const T* C = Cm + (n * G + p.g) * S + s0;
      if (full) {
        if constexpr (V) {
          Pack<T, NPL, true>::load(B, b[u], NPL);
          Pack<T, NPL, true>::load(C, cc[u], NPL);
        }
      } else {
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
          b[u][i] = s0 + i < S ? Elem<T>::load(B, i) : 0.f;
          cc[u][i] = s0 + i < S ? Elem<T>::load(C, i) : 0.f;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t n = n0 + u;
      if (n >= first + per || n >= N) break;
      const float d = softplus ? softplus_f32(dl[u]) : dl[u], dx = d * xv[u];
      float o = 0.f;
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        h[u][i] = fmaf(__builtin_amdgcn_exp2f(d * A2[i]), h[u][i], dx * b[u][i]);
        o = fmaf(h[u][i], cc[u][i], o);
      }
      o = fmaf(sk, xv[u], quad_total(o));
      if (z) o *= zv[u] * sigmoid_fast(zv[u]);
      if (q == 0) Elem<T>::store(y, n * D + c, o);
      if (fin) {
        const int64_t at = (n * D + c) * S;
        if (full) {
          if constexpr (V) {
#pragma unroll
            for (int i = 0; i < NPL; i += 4) {
              const float four[4] = {h[u][i], h[u][i + 1], h[u][i + 2], h[u][i + 3]};
              Pack<float, 4, true>::template store<true>(fin + at + s0 + i, four, 4);
            }
          }
        } else {
          store_states<NPL>(fin + at, s0, S, h[u]);
        }
      }
    }
  }
}

// --- launches -----------------------------------------------------------------------------------

int scan_padded_states(int S) {
  int sp = 8;
  while (sp < S) sp *= 2;
  return sp;
}

int64_t scan_channel_blocks(int64_t D, int64_t G) { return G * ((D / G + kFwdChannels - 1) / kFwdChannels); }

// Cutting costs a second pass over the inputs and the exponentials (about half a scan), so it pays
// where the uncut scan leaves SIMDs with one wavefront or none, 256 workgroups of four wavefronts.
// Measured at D = 2048, S = 16, T = 4096, bf16, uncut / cut: 261 / 79 us for B = 1, 265 / 136 for 2,
// 261 / 183 for 3, 271 / 237 for 4, 359 / 343 for 6; at B = 1, T = 65536 4640 / 874. Segments make
// 1024 workgroups, within 64 tokens (D = 512: T = 300 18 us, 22 with 128; T = 2048 23 us, 24 with 128,
// 27 with 32) and 1024 tokens (T = 65536: 874 us, 951 with 4096). Fewer than 256 tokens stay whole: two
// more launches cost as much (T = 200: 16 us whole, 18.5 cut; 256 with 32 states: 25 whole, 20 cut).
// A packed batch's lengths are not known here. Its long sequences are cut, to 512 tokens at the most
// (64 lognormal sequences, 47204 tokens: 742 us, 966 uncut), but where there are enough sequences to
// fill the chip not below their mean length, so that sequences of one length stay whole.
ScanPlan scan_plan(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N, bool packed) {
  const int64_t cb = scan_channel_blocks(D, G), most = packed ? 512 : 1024;
  if (T < 256 || (!packed && B * cb > 256)) return ScanPlan{0, N};
  int64_t L = B * T * cb / 2048;
  L = L < 64 ? 64 : (L > most ? most : L);
  if (packed && N * cb >= 512 && L < (T + N - 1) / N) L = (T + N - 1) / N;
  L = (L + kScanTile - 1) / kScanTile * kScanTile;
  if (L >= T) return ScanPlan{0, N};
  return ScanPlan{static_cast<int>(L), packed ? T / L + N + 1 : B * ((T + L - 1) / L)};
}

template <typename T, int NPL>
static hipError_t scan_t(const ScanArgs& a, const ScanPlan& p, float* hseg, float* dsum, hipStream_t st) {
  const ScanK<T> k{static_cast<const T*>(a.x), static_cast<const T*>(a.dt), a.A, static_cast<const T*>(a.Bm),
                   static_cast<const T*>(a.Cm), a.skip, static_cast<const T*>(a.z), a.dt_bias, a.init, a.cu_seqlens,
                   static_cast<T*>(a.y), a.fin, hseg, dsum, a.N, a.T, a.D, a.S, a.G, p.L, p.slots, a.softplus};
  constexpr int TH = kFwdChannels * kFwdLanes, SP = kFwdLanes * NPL;
  const unsigned grid = static_cast<unsigned>((p.slots * scan_channel_blocks(a.D, a.G) + 7) / 8 * 8);
  if (p.L) {
    scan_fwd_kernel<T, NPL, true><<<grid, TH, 0, st>>>(k);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t threads = static_cast<int64_t>(a.N) * a.D * SP;
    scan_carry_kernel<<<static_cast<unsigned>((threads + kScanBlock - 1) / kScanBlock), kScanBlock, 0, st>>>(
        a.A, a.init, a.cu_seqlens, a.N, a.T, a.D, a.S, SP, p.L, hseg, dsum);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  scan_fwd_kernel<T, NPL, false><<<grid, TH, 0, st>>>(k);
  return hipGetLastError();
}

static int64_t scan_step_channel_blocks(int64_t D, int64_t G) {
  return G * ((D / G + kScanChannels - 1) / kScanChannels);
}

// Sequences per workgroup: up to 16 while eight workgroups per compute unit remain. At D = 2048,
// S = 16, with 1 / 2 / 4 / 8 / 16 / 32: 177 / 128 / 114 / 105 / 101 / 106 us for 2048 sequences; for
// 256, 22 / 15 / 13.5 / 14.3 with 1 / 2 / 4 / 8.
static int64_t scan_step_per(int64_t N, int64_t cb) {
  const int64_t per = N * cb / 2048;
  return per < 1 ? 1 : (per > 16 ? 16 : per);
}

int64_t scan_step_blocks(int64_t N, int64_t D, int64_t G) {
  const int64_t cb = scan_step_channel_blocks(D, G), per = scan_step_per(N, cb);
  return (N + per - 1) / per * cb;
}

template <typename T, int NPL>
static hipError_t scan_step_t(const ScanArgs& a, hipStream_t st) {
  const int64_t per = scan_step_per(a.N, scan_step_channel_blocks(a.D, a.G));
  const unsigned grid = static_cast<unsigned>(scan_step_blocks(a.N, a.D, a.G));
  scan_step_kernel<T, NPL><<<grid, kScanBlock, 0, st>>>(
      static_cast<const T*>(a.x), static_cast<const T*>(a.dt), a.A, static_cast<const T*>(a.Bm),
      static_cast<const T*>(a.Cm), a.skip, static_cast<const T*>(a.z), a.dt_bias, a.softplus, a.init, a.N, a.D, a.S, a.G,
      static_cast<int>(per), static_cast<T*>(a.y), a.fin);
  return hipGetLastError();
}

hipError_t launch_scan(const ScanArgs& a, const ScanPlan& p, float* hseg, float* dsum, hipStream_t st) {
  auto run = [&](auto npl) {
    constexpr int NPL = decltype(npl)::value;
    return a.dtype == COMBA_BF16 ? scan_t<u16, NPL>(a, p, hseg, dsum, st) : scan_t<float, NPL>(a, p, hseg, dsum, st);
  };
  switch (scan_padded_states(a.S)) {
    case 8: return run(std::integral_constant<int, 1>{});
    case 16: return run(std::integral_constant<int, 2>{});
    case 32: return run(std::integral_constant<int, 4>{});
    default: return run(std::integral_constant<int, 8>{});
  }
}

template <typename F>
static hipError_t with_states(int S, F f) {
  if (S <= 4) return f(std::integral_constant<int, 1>{});
  if (S <= 8) return f(std::integral_constant<int, 2>{});
  if (S <= 16) return f(std::integral_constant<int, 4>{});
  if (S <= 32) return f(std::integral_constant<int, 8>{});
  return f(std::integral_constant<int, 16>{});
}

hipError_t launch_scan_step(const ScanArgs& a, hipStream_t st) {
  return with_states(a.S, [&](auto npl) {
    constexpr int NPL = decltype(npl)::value;
    return a.dtype == COMBA_BF16 ? scan_step_t<u16, NPL>(a, st) : scan_step_t<float, NPL>(a, st);
  });
}

}  // namespace comba
