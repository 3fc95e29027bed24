// Short causal depthwise convolution in front of a recurrence, with optional SiLU:
//   p[t, c] = bias[c] + sum_k weight[c, k] x[t - (W - 1) + k, c],   y = p or p sigmoid(p)
// where tokens before a sequence come from its state (its last W - 1 inputs) or are 0.
//
// A few operations per element: bound by HBM (one read of x, one write of y). A thread owns 16
// bytes of channels and walks along a tile of tokens with the last W - 1 inputs in registers, so
// that every input is loaded once per tile; eight loads are in flight before the first is used.
// Sums and the SiLU are float32, the output is rounded once. Measured, W = 4, bf16:
//   8 x 4096 tokens of 2048 channels: 56 to 59 us, 4.6 to 4.8 TB/s, of the 5.2 that a copy and the 6.2
//   that an elementwise sum reach; 45 to 47 us where the input is the one of the call before, part of
//   which the last-level cache then holds (56 so with loads only at natural alignment and stores
//   through the caches). fp32, W = 3, 15001 packed tokens of 1001 channels, whose rows start anywhere:
//   25 us, 4.8 TB/s (35 us with element loads);
//   one token for 256 sequences: 4.8 us, of which a launch takes most.
// The comparisons below were taken with the same inputs call after call.
#include "comba.h"
#include "column_sums.h"
#include "launch.h"
#include "layer.h"
#include "layer_common.h"

namespace comba {

constexpr int kConvBlock = 256;
constexpr int kConvAhead = 8;   // tokens loaded ahead; 4 and 16 are within 3 % (bf16, W = 4)

// Tokens per tile: 64 once that gives two wavefronts per SIMD (131072 threads); shorter for small
// batches, down to 4, where the threads count and not the W - 1 inputs read twice. With 2048 bf16
// channels, tiles of 4 / 16 / 32 / 64 / 128: 83 / 56 / 51 / 48 / 51 us for 8 x 4096 tokens, 22 / 15 /
// 15 / 23 / 39 for 4 x 2048, 4.5 / 7.4 / 11 / - / 35 for 256 tokens.
static int conv_tile(int64_t tokens, int64_t groups) {
  int t = 64;
  while (t > 4 && (tokens / t) * groups < 131072) t >>= 2;
  return t;
}

static int64_t tiles_of(int64_t B, int64_t T, bool packed, int TT) {
  const int64_t per = (T + TT - 1) / TT;
  return packed ? per : B * per;
}

struct ConvPos {  // one thread's place: a tile of tokens (or a sequence's state) and a channel group
  int tile, c, nc;
  bool done;
};

template <int E>
__device__ __forceinline__ ConvPos conv_pos(int D, int tiles) {
  const uint32_t groups = (D + E - 1) / E;
  const uint32_t item = blockIdx.x * static_cast<uint32_t>(kConvBlock) + threadIdx.x;
  ConvPos p;
  p.tile = static_cast<int>(item / groups);
  p.c = static_cast<int>(item % groups) * E;
  p.nc = min(E, D - p.c);
  p.done = p.tile >= tiles;
  return p;
}

// A ragged last group of channels moved back to whole pieces: some channels are then computed and
// stored twice, with the same bits, instead of a wavefront's going through element accesses (15001
// packed tokens of 1001 fp32 channels 28 -> 25 us; 8 x 2048 tokens of 1999 bf16 channels 67 -> 29, the
// backward 133 -> 44). Not where a state may be updated in place.
template <int E>
__device__ __forceinline__ int whole_group(int c, int64_t D) {
  return min(c, static_cast<int>(D) - E);
}

template <int E, bool V, int W>
__device__ __forceinline__ void load_weights(const float* weight, const float* bias, int c, int nc,
                                             float (&w)[W][E], float (&b)[E]) {
#pragma unroll
  for (int e = 0; e < E; ++e) {
#pragma unroll
    for (int k = 0; k < W; ++k) w[k][e] = V || e < nc ? weight[static_cast<int64_t>(c + e) * W + k] : 0.f;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) b[e] = bias && (V || e < nc) ? bias[c + e] : 0.f;
}

// The W - 1 inputs before token t of a sequence [s, ...) into win[0 .. W-2], oldest first. `x` is
// the row of token 0 of the batch row; `state` the sequence's first state row, or null.
template <typename T, int E, bool V, int W>
__device__ __forceinline__ void load_history(const T* x, const T* state, int64_t D, int s, int t, int nc,
                                             float (&win)[W][E]) {
#pragma unroll
  for (int k = 0; k < W - 1; ++k) {
    const int pos = t - (W - 1) + k;  // token of this place
    if (pos >= s) {
      Pack<T, E, V>::load(x + pos * D, win[k], nc);
    } else if (state) {
      Pack<T, E, V>::load(state + (W - 1 + pos - s) * D, win[k], nc);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) win[k][e] = 0.f;
    }
  }
}

template <int E, int W>
__device__ __forceinline__ void conv_dot(const float (&win)[W][E], const float (&w)[W][E], const float (&b)[E],
                                         float (&p)[E]) {
#pragma unroll
  for (int e = 0; e < E; ++e) {
    p[e] = b[e];
#pragma unroll
    for (int k = 0; k < W; ++k) p[e] = fmaf(w[k][e], win[k][e], p[e]);
  }
}

template <int E, int W>
__device__ __forceinline__ void shift_window(float (&win)[W][E]) {
#pragma unroll
  for (int k = 0; k < W - 1; ++k)
#pragma unroll
    for (int e = 0; e < E; ++e) win[k][e] = win[k + 1][e];
}

// Calls piece(n, s, e, m, mend) for the part [m, mend) of every sequence [s, e) that the tile holds.
template <typename F>
__device__ __forceinline__ void for_pieces(const int32_t* cu, int N, int T, int b, int m0, int m1, F piece) {
  if (!cu) {
    piece(b, 0, T, m0, m1);
    return;
  }
  for (int n = find_sequence(cu, N, m0); n < N; ++n) {
    int s, e;
    packed_range(cu, n, T, s, e);
    if (s >= m1) break;
    const int a = max(s, m0), z = min(e, m1);
    if (a < z) piece(n, s, e, a, z);
  }
}

template <typename T, int E, bool V, int W>
__global__ __launch_bounds__(kConvBlock) void conv_fwd_kernel(
    const T* __restrict__ x, const float* __restrict__ weight, const float* __restrict__ bias,
    const T* __restrict__ init, const int32_t* __restrict__ cu, int N, int Tn, int64_t D, int TT, int tiles,
    bool silu, T* __restrict__ y, T* __restrict__ fin) {
  const ConvPos p = conv_pos<E>(static_cast<int>(D), tiles + (fin ? N : 0));
  if (p.done) return;
  const int c = V ? whole_group<E>(p.c, D) : p.c, nc = V ? E : p.nc;
  if (p.tile >= tiles) {  // the last W - 1 inputs of sequence n: exact copies
    const int n = p.tile - tiles;
    int s = 0, e = Tn;
    if (cu) packed_range(cu, n, Tn, s, e);
    const T* xr = x + (cu ? 0 : static_cast<int64_t>(n) * Tn * D) + c;
    const T* st = init ? init + static_cast<int64_t>(n) * (W - 1) * D + c : nullptr;
    float win[W][E];
    load_history<T, E, V, W>(xr, st, D, s, e, nc, win);
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
      Pack<T, E, V>::store(fin + (static_cast<int64_t>(n) * (W - 1) + k) * D + c, win[k], nc);
    return;
  }
  const int per = (Tn + TT - 1) / TT;
  const int b = p.tile / per, m0 = (p.tile - b * per) * TT, m1 = min(m0 + TT, Tn);
  float w[W][E], bs[E];
  load_weights<E, V, W>(weight, bias, c, nc, w, bs);
  const T* xr = x + static_cast<int64_t>(b) * Tn * D + c;
  T* yr = y + static_cast<int64_t>(b) * Tn * D + c;
  for_pieces(cu, N, Tn, b, m0, m1, [&](int n, int s, int e, int m, int mend) {
    const T* st = init ? init + static_cast<int64_t>(n) * (W - 1) * D + c : nullptr;
    float win[W][E];
    load_history<T, E, V, W>(xr, st, D, s, m, nc, win);
    for (; m < mend; m += kConvAhead) {
      typename Pack<T, E, V>::Words in[kConvAhead];
#pragma unroll
      for (int u = 0; u < kConvAhead; ++u) in[u] = Pack<T, E, V>::fetch(xr + min(m + u, mend - 1) * D, nc);
#pragma unroll
      for (int u = 0; u < kConvAhead; ++u) {
        if (m + u < mend) {
          float o[E];
          Pack<T, E, V>::unpack(in[u], win[W - 1]);
          conv_dot<E, W>(win, w, bs, o);
          if (silu)
#pragma unroll
            for (int i = 0; i < E; ++i) o[i] *= sigmoid_fast(o[i]);
          Pack<T, E, V>::template store<true>(yr + (m + u) * D, o, nc);
          shift_window<E, W>(win);
        }
      }
    }
  });
}

// One token per sequence: the state is read, shifted by the token and written (in place if the
// caller asks for it: a thread reads its slots before it writes them). HBM-bound.
template <typename T, int E, bool V, int W>
__global__ __launch_bounds__(kConvBlock) void conv_step_kernel(
    const T* __restrict__ x, const float* __restrict__ weight, const float* __restrict__ bias, const T* init, int N,
    int64_t D, bool silu, T* __restrict__ y, T* fin) {
  const ConvPos p = conv_pos<E>(static_cast<int>(D), N);
  if (p.done) return;
  const int c = V ? whole_group<E>(p.c, D) : p.c, nc = V ? E : p.nc;
  const int64_t n = p.tile, so = n * (W - 1) * D + c;
  float win[W][E], w[W][E], bs[E], o[E];
  Pack<T, E, V>::load(x + n * D + c, win[W - 1], nc);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) {
    if (init) Pack<T, E, V>::load(init + so + k * D, win[k], nc);
    else
#pragma unroll
      for (int i = 0; i < E; ++i) win[k][i] = 0.f;
  }
  load_weights<E, V, W>(weight, bias, c, nc, w, bs);
  conv_dot<E, W>(win, w, bs, o);
  if (silu)
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] *= sigmoid_fast(o[i]);
  Pack<T, E, V>::store(y + n * D + c, o, nc);
  if (fin)
#pragma unroll
    for (int k = 0; k < W - 1; ++k) Pack<T, E, V>::store(fin + so + k * D, win[k + 1], nc);
}

// d loss / d p from d loss / d y: y = p sigmoid(p), y' = s (1 + p (1 - s)).
template <int E>
__device__ __forceinline__ void silu_grad(const float (&p)[E], float (&d)[E]) {
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const float s = sigmoid_fast(p[i]);
    d[i] *= s * fmaf(p[i], 1.f - s, 1.f);
  }
}

// Backward: dp as above from the recomputed p; dx[t] = sum_k weight[k] dp[t + W - 1 - k] (tokens of
// the same sequence), dweight[c, k] = sum_t dp[t] x[t - (W - 1) + k], dbias = sum_t dp. A thread
// walks its tile and the W - 1 tokens after it, whose dp it recomputes for its own dx. Parameter
// gradients: one float32 partial sum per four tiles, added up in a fixed order by a second kernel.
// The last N items form the gradients of the initial states from the first W - 1 tokens.
// Bound by HBM in principle (x and dy read, dx written); measured, 4 x 2048 tokens of 2048 bf16
// channels, W = 4: 35 us with the parameter sums, 2.9 TB/s, 27 us where the last-level cache holds part
// of the inputs; 93 us (4.3 TB/s) for 8 x 4096, in cache 83; 47 us (4.3 TB/s) for 4 x 2048 in fp32. The
// smaller one has two wavefronts per SIMD, each with eight loads in flight and none while it works on
// them: too few; four channels per thread and sums over four tiles in LDS took it from 48 to 28 us.
template <typename T, typename G, int E, bool V, int W>
__global__ __launch_bounds__(kConvBlock) void conv_bwd_kernel(
    const T* __restrict__ x, const float* __restrict__ weight, const float* __restrict__ bias,
    const T* __restrict__ init, const int32_t* __restrict__ cu, int N, int Tn, int64_t D, int TT, int tiles, bool silu,
    const G* __restrict__ dy, const T* __restrict__ dfin, T* __restrict__ dx, T* __restrict__ dinit,
    float* __restrict__ part) {
  // a workgroup: four tiles (or states) of 64 channel groups; one partial sum per four tiles
  __shared__ float sums[3][W + 1][E][kWave];
  const int groups = static_cast<int>((D + E - 1) / E), gblocks = (groups + kWave - 1) / kWave;
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int four = blockIdx.x / gblocks, g = (blockIdx.x - four * gblocks) * kWave + lane;
  const int sets = (tiles + 3) / 4, tile = four * 4 + wave;
  const bool here = g < groups;
  const int c = !here ? 0 : V ? whole_group<E>(g * E, D) : g * E;
  const int nc = !here ? 0 : V ? E : min(E, static_cast<int>(D) - c);
  float w[W][E], bs[E];
  if (here) load_weights<E, V, W>(weight, bias, c, nc, w, bs);
  if (four >= sets) {
    const int n = (four - sets) * 4 + wave;
    if (!here || n >= N) return;
    int s = 0, e = Tn;
    if (cu) packed_range(cu, n, Tn, s, e);
    const int64_t row = cu ? 0 : static_cast<int64_t>(n) * Tn * D;
    const int64_t so = static_cast<int64_t>(n) * (W - 1) * D + c;
    float win[W][E], acc[W][E];
    load_history<T, E, V, W>(x + row + c, init ? init + so : nullptr, D, s, s, nc, win);
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
      for (int i = 0; i < E; ++i) acc[j][i] = 0.f;
#pragma unroll
    for (int q = 0; q < W - 1; ++q) {
      if (s + q < e) {  // token q of the sequence sees slot j through weight j - q
        float p[E], d[E];
        Pack<T, E, V>::load(x + row + c + (s + q) * D, win[W - 1], nc);
        Pack<G, E, V>::load(dy + row + c + (s + q) * D, d, nc);
        conv_dot<E, W>(win, w, bs, p);
        if (silu) silu_grad<E>(p, d);
#pragma unroll
        for (int j = q; j < W - 1; ++j)
#pragma unroll
          for (int i = 0; i < E; ++i) acc[j][i] = fmaf(w[j - q][i], d[i], acc[j][i]);
        shift_window<E, W>(win);
      }
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      if (dfin && j >= e - s) {  // the slot is still in the final state, moved up by the length
        float f[E];
        Pack<T, E, V>::load(dfin + so + (j - (e - s)) * D, f, nc);
#pragma unroll
        for (int i = 0; i < E; ++i) acc[j][i] += f[i];
      }
      Pack<T, E, V>::store(dinit + so + j * D, acc[j], nc);
    }
    return;
  }
  const int per = (Tn + TT - 1) / TT;
  const int b = tile / per, m0 = (tile - b * per) * TT, m1 = min(m0 + TT, Tn);
  const int64_t row = static_cast<int64_t>(b) * Tn * D + c;
  float dw[W + 1][E];
#pragma unroll
  for (int k = 0; k <= W; ++k)
#pragma unroll
    for (int i = 0; i < E; ++i) dw[k][i] = 0.f;
  if (here && tile < tiles) for_pieces(cu, N, Tn, b, m0, m1, [&](int n, int s, int e, int m, int mend) {
    const int64_t so = static_cast<int64_t>(n) * (W - 1) * D + c;
    float win[W][E], ring[W][E];  // ring: dp of the last W tokens
    load_history<T, E, V, W>(x + row, init ? init + so : nullptr, D, s, m, nc, win);
#pragma unroll
    for (int k = 0; k < W; ++k)
#pragma unroll
      for (int i = 0; i < E; ++i) ring[k][i] = 0.f;
    const int first = m, stop = mend + W - 1, have = min(stop, e);
    constexpr int U = 4;
    for (; m < stop; m += U) {
      typename Pack<T, E, V>::Words in[U];
      typename Pack<G, E, V>::Words din[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = min(m + u, have - 1);
        in[u] = Pack<T, E, V>::fetch(x + row + t * D, nc);
        din[u] = Pack<G, E, V>::fetch(dy + row + t * D, nc);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = m + u;
        if (t < stop) {
          float d[E];
          Pack<T, E, V>::unpack(in[u], win[W - 1]);
          Pack<G, E, V>::unpack(din[u], d);
          if (t >= have) {
#pragma unroll
            for (int i = 0; i < E; ++i) d[i] = 0.f;
          } else if (silu) {
            float p[E];
            conv_dot<E, W>(win, w, bs, p);
            silu_grad<E>(p, d);
          }
          if (t < mend) {
#pragma unroll
            for (int i = 0; i < E; ++i) {
#pragma unroll
              for (int k = 0; k < W; ++k) dw[k][i] = fmaf(d[i], win[k][i], dw[k][i]);
              dw[W][i] += d[i];
            }
          }
          shift_window<E, W>(win);
#pragma unroll
          for (int i = 0; i < E; ++i) {
#pragma unroll
            for (int k = 0; k < W - 1; ++k) ring[k][i] = ring[k + 1][i];
            ring[W - 1][i] = d[i];
          }
          const int to = t - (W - 1);  // its dx is complete: ring[o] is dp[to + o]
          if (to >= first) {
            float g[E];
#pragma unroll
            for (int i = 0; i < E; ++i) {
              g[i] = 0.f;
#pragma unroll
              for (int o = 0; o < W; ++o) g[i] = fmaf(w[W - 1 - o][i], ring[o][i], g[i]);
            }
            const int slot = to - (e - (W - 1));
            if (dfin && slot >= 0) {
              float f[E];
              Pack<T, E, V>::load(dfin + so + slot * D, f, nc);
#pragma unroll
              for (int i = 0; i < E; ++i) g[i] += f[i];
            }
            Pack<T, E, V>::template store<true>(dx + row + to * D, g, nc);
          }
        }
      }
    }
  });
  if (wave > 0)
#pragma unroll
    for (int k = 0; k <= W; ++k)
#pragma unroll
      for (int i = 0; i < E; ++i) sums[wave - 1][k][i][lane] = dw[k][i];
  __syncthreads();
  if (wave == 0 && here)
#pragma unroll
    for (int k = 0; k <= W; ++k)
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (i < nc)
          part[(static_cast<int64_t>(four) * (W + 1) + k) * D + c + i] =
              ((dw[k][i] + sums[0][k][i][lane]) + sums[1][k][i][lane]) + sums[2][k][i][lane];
}

// --- launches -----------------------------------------------------------------------------------

static unsigned conv_grid(int64_t rows, int64_t groups) {
  return static_cast<unsigned>((rows * groups + kConvBlock - 1) / kConvBlock);
}

template <typename T, int E, bool V, int W>
static hipError_t conv_fwd_t(const ConvArgs& a, hipStream_t st) {
  const int64_t groups = (a.D + E - 1) / E;
  const int TT = conv_tile(static_cast<int64_t>(a.B) * a.T, groups);
  const int64_t tiles = tiles_of(a.B, a.T, a.cu_seqlens != nullptr, TT);
  const unsigned grid = conv_grid(tiles + (a.fin ? a.N : 0), groups);
  if (grid == 0) return hipSuccess;
  conv_fwd_kernel<T, E, V, W><<<grid, kConvBlock, 0, st>>>(
      static_cast<const T*>(a.x), a.weight, a.bias, static_cast<const T*>(a.init), a.cu_seqlens, a.N, a.T, a.D, TT,
      static_cast<int>(tiles), a.silu, static_cast<T*>(a.y), static_cast<T*>(a.fin));
  return hipGetLastError();
}

template <typename T, int E, bool V, int W>
static hipError_t conv_step_t(const ConvArgs& a, hipStream_t st) {
  conv_step_kernel<T, E, V, W><<<conv_grid(a.N, (a.D + E - 1) / E), kConvBlock, 0, st>>>(
      static_cast<const T*>(a.x), a.weight, a.bias, static_cast<const T*>(a.init), a.N, a.D, a.silu,
      static_cast<T*>(a.y), static_cast<T*>(a.fin));
  return hipGetLastError();
}

int64_t conv_tiles(int64_t B, int64_t T, int64_t D, bool packed) {
  return tiles_of(B, T, packed, conv_tile(B * T, (D + 7) / 8));
}

constexpr int kConvBwdPiece = 4;  // channels per thread: with 8 a thread needs more than 200 registers

// Tokens per tile of the backward: 64 once that gives two wavefronts per SIMD, down to 4. With 2048
// bf16 channels, tiles of 8 / 16 / 32 / 64 / 128: 106 / 89 / 81 / 78 / 86 us for 8 x 4096 tokens,
// 32 / 28 / 28 / 38 / 65 for 4 x 2048; for 256 tokens 8.5 with 4, 13 with 16, 31 with 64.
static int conv_bwd_tile(int64_t B, int64_t T, int64_t D) {
  const int64_t groups = (D + kConvBwdPiece - 1) / kConvBwdPiece;
  int t = 64;
  while (t > 4 && B * T / t * groups < 131072) t >>= 1;
  return t;
}

static int64_t conv_bwd_all_tiles(int64_t B, int64_t T, int64_t D, bool packed) {
  return tiles_of(B, T, packed, conv_bwd_tile(B, T, D));
}

int64_t conv_bwd_sets(int64_t B, int64_t T, int64_t D, bool packed) {
  return (conv_bwd_all_tiles(B, T, D, packed) + 3) / 4;
}

template <typename T, typename G, int E, bool V, int W>
static hipError_t conv_bwd_t(const ConvBwdArgs& a, hipStream_t st) {
  const ConvArgs& f = a.f;
  const int TT = conv_bwd_tile(f.B, f.T, f.D);
  const bool packed = f.cu_seqlens != nullptr;
  const int64_t tiles = conv_bwd_all_tiles(f.B, f.T, f.D, packed), sets = conv_bwd_sets(f.B, f.T, f.D, packed);
  const int64_t gblocks = ((f.D + E - 1) / E + kWave - 1) / kWave;
  const unsigned grid = static_cast<unsigned>((sets + (a.dinit ? (f.N + 3) / 4 : 0)) * gblocks);
  if (grid > 0) {
    conv_bwd_kernel<T, G, E, V, W><<<grid, kConvBlock, 0, st>>>(
        static_cast<const T*>(f.x), f.weight, f.bias, static_cast<const T*>(f.init), f.cu_seqlens, f.N, f.T, f.D, TT,
        static_cast<int>(tiles), f.silu, static_cast<const G*>(a.dy), static_cast<const T*>(a.dfin),
        static_cast<T*>(a.dx), static_cast<T*>(a.dinit), a.part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  // column k * D + c of the partial sums: dweight[c, k], the last D columns dbias
  float* dw = a.dweight;
  float* db = a.dbias;
  const int D = f.D;
  return column_sums(a.part, sets, static_cast<int64_t>(W + 1) * D, (W + (db ? 1 : 0)) * D, st,
                     [=] __device__(int col, float s) {
                       const int k = col / D, ch = col - k * D;
                       if (k < W) dw[static_cast<int64_t>(ch) * W + k] = s;
                       else db[ch] = s;
                     });
}

template <typename T, int E, bool V>
static hipError_t conv_w(const ConvArgs& a, bool step, hipStream_t st) {
  switch (a.W) {
    case 2: return step ? conv_step_t<T, E, V, 2>(a, st) : conv_fwd_t<T, E, V, 2>(a, st);
    case 3: return step ? conv_step_t<T, E, V, 3>(a, st) : conv_fwd_t<T, E, V, 3>(a, st);
    default: return step ? conv_step_t<T, E, V, 4>(a, st) : conv_fwd_t<T, E, V, 4>(a, st);
  }
}

static hipError_t conv_any(const ConvArgs& a, bool step, hipStream_t st) {
  const int E = a.dtype == COMBA_BF16 ? 8 : 4;
  // every thread has a whole piece of channels
  const bool v = a.D % E == 0 || (a.D >= E && !(step && a.fin && a.init == a.fin));
  if (a.dtype == COMBA_BF16) return v ? conv_w<u16, 8, true>(a, step, st) : conv_w<u16, 8, false>(a, step, st);
  return v ? conv_w<float, 4, true>(a, step, st) : conv_w<float, 4, false>(a, step, st);
}

hipError_t launch_conv(const ConvArgs& a, hipStream_t st) { return conv_any(a, false, st); }
hipError_t launch_conv_step(const ConvArgs& a, hipStream_t st) { return conv_any(a, true, st); }

template <typename T, typename G, bool V>
static hipError_t conv_bwd_w(const ConvBwdArgs& a, hipStream_t st) {
  switch (a.f.W) {
    case 2: return conv_bwd_t<T, G, kConvBwdPiece, V, 2>(a, st);
    case 3: return conv_bwd_t<T, G, kConvBwdPiece, V, 3>(a, st);
    default: return conv_bwd_t<T, G, kConvBwdPiece, V, 4>(a, st);
  }
}

hipError_t launch_conv_bwd(const ConvBwdArgs& a, hipStream_t st) {
  const bool v = a.f.D >= kConvBwdPiece;
  if (a.f.dtype == COMBA_FP32) return v ? conv_bwd_w<float, float, true>(a, st) : conv_bwd_w<float, float, false>(a, st);
  if (a.dy_dtype == COMBA_FP32) return v ? conv_bwd_w<u16, float, true>(a, st) : conv_bwd_w<u16, float, false>(a, st);
  return v ? conv_bwd_w<u16, u16, true>(a, st) : conv_bwd_w<u16, u16, false>(a, st);
}

}  // namespace comba
