// Linear attention with a decay for each head. Per value head, with S a V x K state:
//   S_t = e^{g_t} S_{t-1} + v_t k_t^T,    o_t = scale S_t q_t
// and over a chunk of tokens, with G_t the sum of g from the chunk's first token to t (C: its last):
//   o_t = scale (e^{G_t} S_0 q_t + sum_{s <= t} e^{G_t - G_s} (q_t . k_s) v_s)
//   S_C = e^{G_C} S_0 + sum_s e^{G_C - G_s} v_s k_s^T
// The gradients have the same form. With E the gradient of S at the chunk's end from what follows:
//   dq_t = scale (e^{G_t} S_0^T do_t + sum_{s <= t} e^{G_t - G_s} (do_t . v_s) k_s)
//   dk_s = e^{G_C - G_s} E^T v_s + scale sum_{t >= s} e^{G_t - G_s} (v_s . do_t) q_t
//   dv_s = e^{G_C - G_s} E k_s   + scale sum_{t >= s} e^{G_t - G_s} (k_s . q_t) do_t
//   E at the chunk's start = e^{G_C} E + scale sum_t e^{G_t} do_t q_t^T
// so one kernel, with the roles of the tensors exchanged and time run forwards or backwards, computes
// all of them:
//   out_u = f_u M^T x_u + sum_w D_uw (x_u . y_w) z_w,    M = decay M + sum_w r_w y_w z_w^T
// The gradient of g follows from dq and dk: all of the chunk's results depend on G_t through
// q_t . dq_t - k_t . dk_t, and S_C on G_C, so
//   dg_t = sum_{t' >= t, in the segment} (q . dq - k . dk)_{t'} + <E, S> at the segment's end.
#include "comba.h"
#include "linear_attn.h"
#include "attn_tiles.h"
#include "launch.h"
#include "scan_common.h"

namespace comba {

constexpr int kAttnThreads = 256;

// Logarithms of decays below this one are taken as it: its exponential is 0 in float32, and differences
// of sums stay finite.
constexpr float kLeastDecay = -200.f;

template <typename T> struct AttnRole {
  const T* x;                 // [tokens, xh heads, A]
  const T* y;                 // [tokens, yh heads, A]
  const T* z;                 // [tokens, zh heads, Z]
  T* out;                     // [tokens, H, Z], or null
  float* out32;               // the same in float32 (then out is null)
  const T* own;               // [tokens, own_h heads, Z]: its products with out's rows are wanted, or null
  float* rdot;                // [Z blocks, H, tokens]: those products
  float* state;               // [slots, H, V, K]: incoming states, or (state pass) where the segment's own go
  int xh, yh, zh, own_h, A, Z;
  bool back;                  // time runs from the segment's end
  bool a_is_k;                // A is the axis of K in a state, Z that of V; else the other way round
  float f_state, f_score, f_into;   // factors of M^T x, of the scores, of what goes into M
};

template <typename T> struct AttnK {
  AttnRole<T> role[3];
  const float* log_decay;
  const float* init;          // [N, H, V, K] or null: incoming state of sequences of one segment (forward)
  float* fin;                 // [N, H, V, K] or null
  const int32_t* cu_seqlens;
  double* decay;              // [slots, H]: the segment's sum of log2 decays (state pass)
  int N, Tn, H, K, V, L, roles;
  int64_t slots, tokens;
  bool per_token;
  bool whole_pass;            // backward: every segment has its states in role.state; state pass: the last one too
};

// Where a unit's workgroups find its column blocks and roles.
template <typename T> __host__ __device__ inline int attn_unit_blocks(const AttnK<T>& a) {
  int n = 0;
  for (int r = 0; r < a.roles; ++r) n += attn_blocks(a.role[r].Z);
  return n;
}

// Four elements a0 .. a0 + 3 of column z of M in a state [V, K].
struct StateMap {
  int K, A, Z;
  bool a_is_k;
  __device__ __forceinline__ f32x4 load(const float* s, int a0, int z) const {
    f32x4 r = {0.f, 0.f, 0.f, 0.f};
    if (z >= Z) return r;
    if (a_is_k && a0 + 4 <= A) return reinterpret_cast<const Loose<f32x4>*>(s + static_cast<int64_t>(z) * K + a0)->v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (a0 + i < A) r[i] = a_is_k ? s[z * K + a0 + i] : s[(a0 + i) * K + z];
    return r;
  }
  __device__ __forceinline__ void store(float* s, int a0, int z, const f32x4& x) const {
    if (z >= Z) return;
    if (a_is_k && a0 + 4 <= A) {
      reinterpret_cast<Loose<f32x4>*>(s + static_cast<int64_t>(z) * K + a0)->v = x;
      return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (a0 + i < A) s[a_is_k ? z * K + a0 + i : (a0 + i) * K + z] = x[i];
  }
};

// AP: A padded to 64, 128 or 256. NT: terms that float32 operands of a bf16 product are split into.
// STATE: the segment's own state alone (from 0, no outputs).
template <typename T, int AP, int NT, bool STATE>
__global__ __launch_bounds__(kAttnThreads) void attn_kernel(AttnK<T> a) {
  typedef Tiles<T> Ti;
  typedef typename Ti::Frag Frag;
  constexpr int CH = Ti::CH, BLK = Ti::BLK, E = Ti::PIECE, ZB = kAttnBlock;
  constexpr int NM = AP / 16, NA = AP / BLK, NS = CH / BLK, NU = CH / 16, EL = BLK / 4;
  constexpr int NTM = Ti::TERMS(NT), NTZ = Ti::TERMS(3);
  constexpr int XP = CH * AP / E / kAttnThreads, ZP = CH * ZB / E / kAttnThreads;  // pieces per thread
  typedef RowPiece<T> Piece;
  __shared__ __align__(16) T xs[STATE ? 8 : Ti::size(CH, AP)];
  __shared__ __align__(16) T ys[Ti::size(CH, AP)];
  __shared__ __align__(16) T zs[Ti::size(CH, ZB)];
  __shared__ __align__(16) typename Ti::P ps[STATE ? 8 : Ti::score_elems(NTM)];
  __shared__ double gs[CH];
  __shared__ __align__(16) float fs[CH], rs[CH];
  __shared__ float whole;
  __shared__ float dots[STATE ? 1 : 4][STATE ? 1 : CH];

  const int tid = threadIdx.x, w = tid >> 6, lane = tid & 63, g = lane >> 4, l16 = lane & 15;
  // the workgroups of one (segment, head) on one XCD, whose L2 they share
  const int per_unit = attn_unit_blocks(a);
  const int64_t unit = static_cast<int64_t>(blockIdx.x / (8 * per_unit)) * 8 + blockIdx.x % 8;
  if (unit >= a.slots * a.H) return;
  int zb = blockIdx.x / 8 % per_unit, ri = 0;
  const bool first_block = zb == 0;
  while (zb >= attn_blocks(a.role[ri].Z)) zb -= attn_blocks(a.role[ri++].Z);
  const AttnRole<T>& R = a.role[ri];
  const int64_t slot = unit / a.H;
  const int h = static_cast<int>(unit - slot * a.H);
  const ScanPlace pl = scan_place<1>(slot, 0, a.cu_seqlens, a.N, a.Tn, 1, 1, a.L);
  if (!pl.ok) return;
  const bool last = last_segment(pl), back = R.back;
  if (STATE && last && !a.whole_pass) return;
  const StateMap sm{a.K, R.A, R.Z, R.a_is_k};
  const int64_t KV = static_cast<int64_t>(a.K) * a.V;
  const int z0 = zb * ZB, zc = z0 + 16 * w + l16;  // first column of the block; this lane's column of M

  f32x4 m[NM];
  const float* from = nullptr;
  if (!STATE) {
    if (R.state && (a.whole_pass || segments_of(pl.s1 - pl.s0, a.L) > 1)) from = R.state + unit * KV;
    else if (a.init) from = a.init + (static_cast<int64_t>(pl.n) * a.H + h) * KV;
  }
#pragma unroll
  for (int j = 0; j < NM; ++j) m[j] = from ? sm.load(from, Ti::index(j, g, 0), zc) : f32x4{0.f, 0.f, 0.f, 0.f};
  double total = 0.0;

  const int chunks = (pl.t1 - pl.t0 + CH - 1) / CH;
  u32x4 xr[STATE ? 1 : XP], yr[XP], zr[ZP];
  float gr = 0.f;
  const int64_t row0 = static_cast<int64_t>(pl.b) * a.Tn;  // token 0 of the batch row
  const T* const xb = R.x + h / (a.H / R.xh) * static_cast<int64_t>(R.A);
  const T* const yb = R.y + h / (a.H / R.yh) * static_cast<int64_t>(R.A);
  const T* const zbase = R.z + h / (a.H / R.zh) * static_cast<int64_t>(R.Z);
  auto fetch = [&](int c) {
    const int t0 = pl.t0 + c * CH, n = min(CH, pl.t1 - t0);
#pragma unroll
    for (int i = 0; i < XP; ++i) {
      const int p = tid + i * kAttnThreads, r = min(p / (AP / E), n - 1), col = p % (AP / E) * E;
      if (!STATE) xr[i] = Piece::fetch(xb + (row0 + t0 + r) * R.xh * R.A, col, R.A);
      yr[i] = Piece::fetch(yb + (row0 + t0 + r) * R.yh * R.A, col, R.A);
    }
#pragma unroll
    for (int i = 0; i < ZP; ++i) {
      const int p = tid + i * kAttnThreads, r = min(p / (ZB / E), n - 1), col = z0 + p % (ZB / E) * E;
      zr[i] = Piece::fetch(zbase + (row0 + t0 + r) * R.zh * R.Z, col, R.Z);
    }
    if (w == 0) {
      const int r = min(lane, n - 1);
      gr = lane < n ? (a.per_token ? a.log_decay[(row0 + t0 + r) * a.H + h] : a.log_decay[h]) : 0.f;
    }
  };
  if (!STATE) {
    for (int i = tid; i < Ti::score_elems(NTM); i += kAttnThreads) ps[i] = 0;  // tiles beyond the diagonal stay 0
  }
  if (chunks > 0) fetch(back ? chunks - 1 : 0);

  for (int ci = 0; ci < chunks; ++ci) {
    const int c = back ? chunks - 1 - ci : ci;
    const int t0 = pl.t0 + c * CH, n = min(CH, pl.t1 - t0);
#pragma unroll
    for (int i = 0; i < XP; ++i) {
      const int p = tid + i * kAttnThreads, r = p / (AP / E), col = p % (AP / E) * E;
      if (!STATE) *reinterpret_cast<u32x4*>(xs + Ti::template at<AP>(r, col)) = Piece::place(xr[i], col, R.A, r < n);
      *reinterpret_cast<u32x4*>(ys + Ti::template at<AP>(r, col)) = Piece::place(yr[i], col, R.A, r < n);
    }
#pragma unroll
    for (int i = 0; i < ZP; ++i) {
      const int p = tid + i * kAttnThreads, r = p / (ZB / E), col = p % (ZB / E) * E;
      *reinterpret_cast<u32x4*>(zs + Ti::template at<ZB>(r, col)) = Piece::place(zr[i], z0 + col, R.Z, r < n);
    }
    if (w == 0) {
      // sums of log2 decays, in 64 bits: their differences are small beside them
      const float gl = gr < kLeastDecay ? kLeastDecay : gr;
      const double G = wave_inclusive_scan_f64(static_cast<double>(gl) * 1.4426950408889634, lane);
      const double all = __shfl(G, 63, kWave);
      const float since = __builtin_amdgcn_exp2f(static_cast<float>(G));
      const float rest = __builtin_amdgcn_exp2f(static_cast<float>(all - G));
      if (lane < CH) {
        gs[lane] = G;
        fs[lane] = R.f_state * (back ? rest : since);
        rs[lane] = R.f_into * (back ? since : rest);
      }
      if (lane == 0) whole = __builtin_amdgcn_exp2f(static_cast<float>(all));
      total += all;
    }
    __syncthreads();
    if (ci + 1 < chunks) fetch(back ? c - 1 : c + 1);

    if constexpr (!STATE) {
      // scores: tiles (target i, source j) on and below the diagonal, above it when time runs back
      for (int k = w; k < NU * (NU + 1) / 2; k += 4) {
        int i = 0;
        while ((i + 1) * (i + 2) / 2 <= k) ++i;
        int j = k - i * (i + 1) / 2;
        if (back) {
          i = NU - 1 - i;
          j = NU - 1 - j;
        }
        f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int p = 0; p < NA; ++p)
          s = Ti::mma(Ti::template along<AP>(ys, 16 * j + l16, p, g), Ti::template along<AP>(xs, 16 * i + l16, p, g), s);
        const int t = 16 * i + l16;
        const double Gt = gs[t];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int u = 16 * j + 4 * g + r;
          const double d = back ? gs[u] - Gt : Gt - gs[u];
          const bool in = back ? u >= t : u <= t;
          s[r] = in ? s[r] * (R.f_score * __builtin_amdgcn_exp2f(static_cast<float>(d))) : 0.f;
        }
        Ti::template put_scores<NTM>(ps, t, j, g, s);
      }
      __syncthreads();
    }

    Frag zf[NS];
#pragma unroll
    for (int b = 0; b < NS; ++b) zf[b] = Ti::template down<ZB>(zs, b, 16 * w, g, l16);

    if constexpr (!STATE) {
      Frag mf[NA][NTM];
#pragma unroll
      for (int p = 0; p < NA; ++p) Ti::template from_tiles<NTM>(m, p, mf[p]);
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        const int t = 16 * i + l16;
        f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int p = 0; p < NA; ++p) {
          const Frag x = Ti::template along<AP>(xs, t, p, g);
#pragma unroll
          for (int k = 0; k < NTM; ++k) o = Ti::mma(mf[p][k], x, o);
        }
        o *= fs[t];
#pragma unroll
        for (int b = 0; b < NS; ++b) {
          if (back ? BLK * (b + 1) <= 16 * i : BLK * b > 16 * i) continue;
#pragma unroll
          for (int k = 0; k < NTM; ++k) o = Ti::mma(zf[b], Ti::scores(ps, k, t, b, g), o);
        }
        // rows z0 + 16 w + 4 g .. + 3 of the output of token t
        const int z = z0 + 16 * w + 4 * g;
        const int left = t < n ? R.Z - z : 0;
        const int64_t tok = row0 + t0 + t;
        float ov[4] = {o[0], o[1], o[2], o[3]};
        if (left > 0) {
          if (R.out) Pack<T, 4, false>::store(R.out + (tok * a.H + h) * R.Z + z, ov, min(left, 4));
          else Pack<float, 4, false>::store(R.out32 + (tok * a.H + h) * R.Z + z, ov, min(left, 4));
        }
        if (R.own) {
          float d = 0.f;
          if (left > 0) {
            float own[4];
            Pack<T, 4, false>::load(R.own + (tok * R.own_h + h / (a.H / R.own_h)) * R.Z + z, own, min(left, 4));
#pragma unroll
            for (int r = 0; r < 4; ++r) d = fmaf(own[r], ov[r], d);
          }
          d += __shfl_xor(d, 16, kWave);
          d += __shfl_xor(d, 32, kWave);
          if (g == 0) dots[w][t] = d;
        }
      }
    }

    // into the state
    const float keep = whole;
#pragma unroll
    for (int j = 0; j < NM; ++j) m[j] *= keep;
#pragma unroll
    for (int b = 0; b < NS; ++b) {
      float zw[EL];
      Frag zt[NTZ];
#pragma unroll
      for (int e = 0; e < EL; ++e) zw[e] = Ti::value(zf[b], e) * rs[BLK * b + Ti::down_row(g, e)];
      Ti::template split<NTZ>(zw, zt);
#pragma unroll
      for (int j = 0; j < NM; ++j) {
        const Frag y = Ti::template down_index<AP>(ys, b, j, g, l16);
#pragma unroll
        for (int k = 0; k < NTZ; ++k) m[j] = Ti::mma(y, zt[k], m[j]);
      }
    }
    __syncthreads();
    if constexpr (!STATE) {
      if (R.own && tid < n)
        R.rdot[(static_cast<int64_t>(zb) * a.H + h) * a.tokens + row0 + t0 + tid] =
            (dots[0][tid] + dots[1][tid]) + (dots[2][tid] + dots[3][tid]);
    }
  }

  float* to = nullptr;
  if (STATE) to = R.state + unit * KV;
  else if (a.fin && last) to = a.fin + (static_cast<int64_t>(pl.n) * a.H + h) * KV;
  if (to)
#pragma unroll
    for (int j = 0; j < NM; ++j) sm.store(to, Ti::index(j, g, 0), zc, m[j]);
  if (STATE && first_block && tid == 0) a.decay[unit] = total;
}

// Carries the states across the segments of every sequence: state[slot] becomes the segment's incoming
// state. With `grad` (backward) also the gradients, from the last segment to the first: grad[slot] becomes
// the gradient at the segment's end, and inner[slot, h, block] its product with the state there.
template <bool BWD>
__global__ __launch_bounds__(256) void attn_carry_kernel(const float* __restrict__ init, const float* __restrict__ dfin,
                                                         const int32_t* __restrict__ cu, int N, int T, int H, int KV, int L,
                                                         float* __restrict__ state, float* __restrict__ grad,
                                                         const double* __restrict__ decay, double* __restrict__ inner,
                                                         float* __restrict__ dinit) {
  constexpr int EPT = kAttnScanElems / 256;
  __shared__ float red[4];
  const int blocks = (KV + kAttnScanElems - 1) / kAttnScanElems;
  const int eb = blockIdx.x % blocks;
  const int64_t nh = blockIdx.x / blocks;
  const int n = static_cast<int>(nh / H), h = static_cast<int>(nh - static_cast<int64_t>(n) * H);
  int b, t0, t1;
  sequence_range(cu, n, T, b, t0, t1);
  const int len = t1 - t0, nseg = segments_of(len, L);
  if (!BWD && nseg <= 1) return;
  const int64_t first = cu ? static_cast<int64_t>(t0 / L) + n : static_cast<int64_t>(n) * ((T + L - 1) / L);
  const int e0 = eb * kAttnScanElems + threadIdx.x;
  float S[EPT];
#pragma unroll
  for (int i = 0; i < EPT; ++i) S[i] = init && e0 + 256 * i < KV ? init[nh * KV + e0 + 256 * i] : 0.f;
  if (len == 0) {  // backward only: the gradient passes through
#pragma unroll
    for (int i = 0; i < EPT; ++i)
      if (dinit && e0 + 256 * i < KV) dinit[nh * KV + e0 + 256 * i] = dfin ? dfin[nh * KV + e0 + 256 * i] : 0.f;
    return;
  }
  for (int c = 0; c < nseg; ++c) {
    const int64_t unit = (first + c) * H + h;
    const float p = BWD || c + 1 < nseg ? static_cast<float>(decay[unit]) : 0.f;
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      const int e = e0 + 256 * i;
      if (e >= KV) continue;
      float* const at = state + unit * KV + e;
      const float add = BWD || c + 1 < nseg ? *at : 0.f;
      *at = S[i];
      S[i] = carried(S[i], p, add);
    }
  }
  if constexpr (BWD) {
    float G[EPT];
#pragma unroll
    for (int i = 0; i < EPT; ++i) G[i] = dfin && e0 + 256 * i < KV ? dfin[nh * KV + e0 + 256 * i] : 0.f;
    for (int c = nseg - 1; c >= 0; --c) {
      const int64_t unit = (first + c) * H + h;
      const float p = static_cast<float>(decay[unit]);
      float d = 0.f;
#pragma unroll
      for (int i = 0; i < EPT; ++i) {
        const int e = e0 + 256 * i;
        if (e >= KV) continue;
        float* const at = grad + unit * KV + e;
        const float add = *at;
        *at = G[i];
        d = fmaf(G[i], S[i], d);
        G[i] = carried(G[i], p, add);
        S[i] = state[unit * KV + e];
      }
      d = wave_sum(d);
      if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = d;
      __syncthreads();
      if (threadIdx.x == 0) inner[unit * blocks + eb] = (static_cast<double>(red[0]) + red[1]) + (static_cast<double>(red[2]) + red[3]);
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < EPT; ++i)
      if (dinit && e0 + 256 * i < KV) dinit[nh * KV + e0 + 256 * i] = G[i];
  }
}

// dlog_decay of a segment and head per wavefront: sums from the segment's end, in 64 bits.
__global__ __launch_bounds__(256) void attn_decay_grad_kernel(const float* __restrict__ rdot, const double* __restrict__ inner,
                                                              const int32_t* __restrict__ cu, int N, int T, int H, int L,
                                                              int64_t slots, int64_t tokens, int zblocks, int eblocks,
                                                              float* __restrict__ out, double* __restrict__ hsum) {
  const int lane = threadIdx.x & 63;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (unit >= slots * H) return;
  const int64_t slot = unit / H;
  const int h = static_cast<int>(unit - slot * H);
  const ScanPlace pl = scan_place<1>(slot, 0, cu, N, T, 1, 1, L);
  const bool some = pl.ok && pl.t1 > pl.t0;
  if (hsum && !some && lane == 0) hsum[unit] = 0.0;
  if (!some) return;
  double carry = 0.0, sum = 0.0;
  for (int i = 0; i < eblocks; ++i) carry += inner[unit * eblocks + i];
  const int64_t row0 = static_cast<int64_t>(pl.b) * T;
  for (int e = pl.t1; e > pl.t0; e -= 64) {  // lane l: the token l before the last of these 64
    const int t = e - 1 - lane;
    double r = 0.0;
    if (t >= pl.t0)
      for (int zb = 0; zb < zblocks; ++zb) {
        const int64_t at = (static_cast<int64_t>(zb) * H + h) * tokens + row0 + t;
        r += static_cast<double>(rdot[at]) - static_cast<double>(rdot[static_cast<int64_t>(zblocks) * H * tokens + at]);
      }
    const double s = wave_inclusive_scan_f64(r, lane) + carry;
    carry = __shfl(s, 63, kWave);
    if (t >= pl.t0) {
      sum += s;
      if (!hsum) out[(row0 + t) * H + h] = static_cast<float>(s);
    }
  }
  if (hsum) {
    sum = wave_inclusive_scan_f64(sum, lane);
    if (lane == 63) hsum[unit] = sum;
  }
}

// Constant decays: the heads' sums over all segments, in a fixed order.
__global__ __launch_bounds__(256) void attn_head_sum_kernel(const double* __restrict__ hsum, int64_t slots, int H,
                                                            float* __restrict__ out) {
  __shared__ double red[4];
  const int h = blockIdx.x, lane = threadIdx.x & 63;
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < slots; i += 256) s += hsum[i * H + h];
  s = wave_inclusive_scan_f64(s, lane);
  if (lane == 63) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) out[h] = static_cast<float>((red[0] + red[1]) + (red[2] + red[3]));
}

// dq and dk of shared heads: sums over the value heads of a group, of the tokens that belong to a sequence.
template <typename T>
__global__ __launch_bounds__(256) void attn_group_sum_kernel(const float* __restrict__ part, const int32_t* __restrict__ cu,
                                                             int N, int64_t tokens, int H, int Hk, int K, T* __restrict__ dq,
                                                             T* __restrict__ dk) {
  int64_t lo = 0, hi = tokens;
  if (cu) {
    int t0, t1;
    packed_range(cu, 0, static_cast<int>(tokens), t0, t1);
    lo = t0;
    packed_range(cu, N - 1, static_cast<int>(tokens), t0, t1);
    hi = t1;
  }
  const int rep = H / Hk;
  const int64_t row = static_cast<int64_t>(Hk) * K, count = (hi - lo) * row;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < 2 * count; i += static_cast<int64_t>(gridDim.x) * 256) {
    const bool second = i >= count;
    const int64_t e = i - (second ? count : 0), t = lo + e / row, x = e % row, hk = x / K, c = x - hk * K;
    const float* p = part + (second ? tokens * H * K : 0) + (t * H + hk * rep) * K + c;
    float s = 0.f;
    for (int r = 0; r < rep; ++r) s += p[r * K];
    Elem<T>::store(second ? dk : dq, t * row + x, s);
  }
}

// One token per sequence. A state row is spread over 16 lanes, 16-byte pieces at columns 4 j + 64 f; a wavefront
// holds four rows, a workgroup NP passes of 16.
template <typename T, int F, int NP>
__global__ __launch_bounds__(256) void attn_step_kernel(const T* __restrict__ q, const T* __restrict__ k,
                                                        const T* __restrict__ v, const float* __restrict__ log_decay,
                                                        bool per_token, float scale, const float* s0, int H, int Hk, int K,
                                                        int V, T* __restrict__ o, float* sf) {
  constexpr int VB = 16 * NP;
  const int vblocks = (V + VB - 1) / VB;
  const int vb = blockIdx.x % vblocks;
  const int64_t nh = blockIdx.x / vblocks, n = nh / H;
  const int h = static_cast<int>(nh - n * H);
  const int tid = threadIdx.x, j = tid & 15, r0 = vb * VB + (tid >> 4);
  const float* const S0 = s0 ? s0 + nh * K * V : nullptr;
  f32x4 S[NP][F];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int row = r0 + 16 * p;
#pragma unroll
    for (int f = 0; f < F; ++f) {
      const int c = 4 * j + 64 * f;
      f32x4 x = {0.f, 0.f, 0.f, 0.f};
      if (S0 && row < V && c < K) {
        if (c + 4 <= K) x = __builtin_nontemporal_load(&reinterpret_cast<const Loose<f32x4>*>(S0 + row * K + c)->v);
        else
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = c + i < K ? S0[row * K + c + i] : 0.f;
      }
      S[p][f] = x;
    }
  }
  const int64_t qk = (n * Hk + h / (H / Hk)) * K;
  float qv[F][4], kv[F][4];
#pragma unroll
  for (int f = 0; f < F; ++f) {
    const int c = 4 * j + 64 * f, left = K - c;
#pragma unroll
    for (int i = 0; i < 4; ++i) qv[f][i] = kv[f][i] = 0.f;
    if (left > 0) {
      Pack<T, 4, false>::load(q + qk + c, qv[f], min(left, 4));
      Pack<T, 4, false>::load(k + qk + c, kv[f], min(left, 4));
    }
  }
  const float a = expf(log_decay[per_token ? nh : h]);
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int row = r0 + 16 * p;
    const float vv = row < V ? Elem<T>::load(v, nh * V + row) : 0.f;
    float d = 0.f;
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        S[p][f][i] = fmaf(vv, kv[f][i], a * S[p][f][i]);
        d = fmaf(S[p][f][i], qv[f][i], d);
      }
    d = row16_sum(d);
    if (row < V) {
      if (j == 0) Elem<T>::store(o, nh * V + row, scale * d);
      if (sf)
#pragma unroll
        for (int f = 0; f < F; ++f) {
          const int c = 4 * j + 64 * f;
          float* const at = sf + nh * K * V + row * K + c;
          if (c + 4 <= K) __builtin_nontemporal_store(S[p][f], &reinterpret_cast<Loose<f32x4>*>(at)->v);
          else
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (c + i < K) at[i] = S[p][f][i];
        }
    }
  }
}

// --- launches ------------------------------------------------------------------------------------

AttnPlan attn_plan(int64_t B, int64_t T, int64_t H, int64_t V, int64_t N, bool packed) {
  const int64_t units = H * attn_blocks(static_cast<int>(V));
  int64_t L = B * T * units / 512;
  if (!packed && B * units >= 256) return AttnPlan{0, N};
  L = L < 256 ? 256 : L > 2048 ? 2048 : (L + 63) / 64 * 64;
  if (L >= T) return AttnPlan{0, N};
  return AttnPlan{static_cast<int>(L), packed ? T / L + N + 1 : B * ((T + L - 1) / L)};
}

AttnPlan attn_bwd_plan(int64_t B, int64_t T, int64_t H, int64_t N, bool packed) {
  int64_t L = B * T * H / 512;
  L = L < 256 ? 256 : L > 1024 ? 1024 : (L + 63) / 64 * 64;
  return AttnPlan{static_cast<int>(L), packed ? T / L + N + 1 : B * ((T + L - 1) / L)};
}

namespace {

template <typename T, int NT, bool STATE> hipError_t run_attn(const AttnK<T>& k, int A, hipStream_t st) {
  const int64_t units = (k.slots * k.H + 7) / 8 * 8;
  const unsigned grid = static_cast<unsigned>(units * attn_unit_blocks(k));
  if (A <= 64) attn_kernel<T, 64, NT, STATE><<<grid, kAttnThreads, 0, st>>>(k);
  else if (A <= 128) attn_kernel<T, 128, NT, STATE><<<grid, kAttnThreads, 0, st>>>(k);
  else attn_kernel<T, 256, NT, STATE><<<grid, kAttnThreads, 0, st>>>(k);
  return hipGetLastError();
}

int padded(int A) { return A <= 64 ? 64 : A <= 128 ? 128 : 256; }

template <typename T> AttnK<T> attn_args(const AttnArgs& f, const AttnPlan& p, double* decay) {
  AttnK<T> k{};
  k.log_decay = f.log_decay;
  k.cu_seqlens = f.cu_seqlens;
  k.decay = decay;
  k.N = f.N;
  k.Tn = f.T;
  k.H = f.H;
  k.K = f.K;
  k.V = f.V;
  k.L = p.L;
  k.slots = p.slots;
  k.tokens = static_cast<int64_t>(f.B) * f.T;
  k.per_token = f.per_token;
  return k;
}

template <typename T> hipError_t attn_t(const AttnArgs& f, const AttnPlan& p, const AttnWorkspace& w, hipStream_t st) {
  AttnK<T> k = attn_args<T>(f, p, w.decay);
  k.roles = 1;
  const T *q = static_cast<const T*>(f.q), *kk = static_cast<const T*>(f.k), *v = static_cast<const T*>(f.v);
  k.role[0] = AttnRole<T>{q, kk, v, static_cast<T*>(f.o), nullptr, nullptr, nullptr, w.state, f.Hk, f.Hk, f.H, 1,
                          f.K, f.V, false, true, f.scale, f.scale, 1.f};
  hipError_t e;
  if (p.L) {
    if ((e = run_attn<T, 2, true>(k, f.K, st)) != hipSuccess) return e;
    const int blocks = attn_inner_blocks(f.K, f.V);
    attn_carry_kernel<false><<<static_cast<unsigned>(static_cast<int64_t>(f.N) * f.H * blocks), 256, 0, st>>>(
        f.init, nullptr, f.cu_seqlens, f.N, f.T, f.H, f.K * f.V, p.L, w.state, nullptr, w.decay, nullptr, nullptr);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  k.init = f.init;
  k.fin = f.fin;
  return run_attn<T, 2, false>(k, f.K, st);
}

template <typename T> hipError_t attn_bwd_t(const AttnBwdArgs& a, const AttnPlan& p, hipStream_t st) {
  const AttnArgs& f = a.f;
  const int K = f.K, V = f.V, H = f.H, Hk = f.Hk;
  AttnK<T> k = attn_args<T>(f, p, a.decay);
  k.whole_pass = true;
  const T *q = static_cast<const T*>(f.q), *kk = static_cast<const T*>(f.k), *v = static_cast<const T*>(f.v),
          *dO = static_cast<const T*>(a.dO);
  // the segments' own states, and their parts of the gradients at their starts
  k.roles = 2;
  k.role[0] = AttnRole<T>{nullptr, kk, v, nullptr, nullptr, nullptr, nullptr, a.state, Hk, Hk, H, 1, K, V, false, true,
                          0.f, 0.f, 1.f};
  k.role[1] = AttnRole<T>{nullptr, q, dO, nullptr, nullptr, nullptr, nullptr, a.grad, Hk, Hk, H, 1, K, V, true, true,
                          0.f, 0.f, f.scale};
  hipError_t e;
  if ((e = run_attn<T, 2, true>(k, K, st)) != hipSuccess) return e;
  const int eblocks = attn_inner_blocks(K, V);
  attn_carry_kernel<true><<<static_cast<unsigned>(static_cast<int64_t>(f.N) * H * eblocks), 256, 0, st>>>(
      f.init, a.dfin, f.cu_seqlens, f.N, f.T, H, K * V, p.L, a.state, a.grad, a.decay, a.inner, a.dinit);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  T* const dq = a.dqk ? nullptr : static_cast<T*>(a.dq);
  T* const dk = a.dqk ? nullptr : static_cast<T*>(a.dk);
  float* const dk32 = a.dqk ? a.dqk + k.tokens * H * K : nullptr;
  const int zblocks = attn_blocks(K);
  float* const rk = a.rdot + static_cast<int64_t>(zblocks) * H * k.tokens;
  const AttnRole<T> rq_{dO, v, kk, dq, a.dqk, q, a.rdot, a.state, H, H, Hk, Hk, V, K, false, false, f.scale, f.scale, 1.f};
  const AttnRole<T> rk_{v, dO, q, dk, dk32, kk, rk, a.grad, H, H, Hk, Hk, V, K, true, false, 1.f, f.scale, f.scale};
  const AttnRole<T> rv_{kk, q, dO, static_cast<T*>(a.dv), nullptr, nullptr, nullptr, a.grad, Hk, Hk, H, 1, K, V, true, true,
                        1.f, f.scale, f.scale};
  k.role[0] = rq_;
  k.role[1] = rk_;
  k.role[2] = rv_;
  k.roles = padded(K) == padded(V) ? 3 : 2;
  if ((e = run_attn<T, 3, false>(k, V, st)) != hipSuccess) return e;
  if (k.roles == 2) {
    k.role[0] = rv_;
    k.roles = 1;
    if ((e = run_attn<T, 2, false>(k, K, st)) != hipSuccess) return e;
  }
  attn_decay_grad_kernel<<<static_cast<unsigned>((p.slots * H + 3) / 4), 256, 0, st>>>(
      a.rdot, a.inner, f.cu_seqlens, f.N, f.T, H, p.L, p.slots, k.tokens, zblocks, eblocks, a.dlog_decay,
      f.per_token ? nullptr : a.hsum);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (!f.per_token) {
    attn_head_sum_kernel<<<H, 256, 0, st>>>(a.hsum, p.slots, H, a.dlog_decay);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (a.dqk) {
    const int64_t want = (2 * k.tokens * Hk * K + 255) / 256;
    attn_group_sum_kernel<T><<<static_cast<unsigned>(want < 1 ? 1 : want > 16384 ? 16384 : want), 256, 0, st>>>(
        a.dqk, f.cu_seqlens, f.N, k.tokens, H, Hk, K, static_cast<T*>(a.dq), static_cast<T*>(a.dk));
    e = hipGetLastError();
  }
  return e;
}

template <typename T, int F, int NP> hipError_t step_np(const AttnArgs& a, hipStream_t st) {
  const int64_t grid = static_cast<int64_t>(a.N) * a.H * ((a.V + 16 * NP - 1) / (16 * NP));
  attn_step_kernel<T, F, NP><<<static_cast<unsigned>(grid), 256, 0, st>>>(
      static_cast<const T*>(a.q), static_cast<const T*>(a.k), static_cast<const T*>(a.v), a.log_decay, a.per_token, a.scale,
      a.init, a.H, a.Hk, a.K, a.V, static_cast<T*>(a.o), a.fin);
  return hipGetLastError();
}

template <typename T> hipError_t step_t(const AttnArgs& a, hipStream_t st) {
  if (a.K <= 64) return step_np<T, 1, 2>(a, st);
  if (a.K <= 128) return step_np<T, 2, 2>(a, st);
  return step_np<T, 4, 1>(a, st);
}

}  // namespace

int64_t attn_step_blocks(int64_t N, int64_t H, int64_t V) { return N * H * ((V + 15) / 16); }

hipError_t launch_attn(const AttnArgs& a, const AttnPlan& p, const AttnWorkspace& w, hipStream_t st) {
  return a.dtype == COMBA_BF16 ? attn_t<u16>(a, p, w, st) : attn_t<float>(a, p, w, st);
}

hipError_t launch_attn_step(const AttnArgs& a, hipStream_t st) {
  return a.dtype == COMBA_BF16 ? step_t<u16>(a, st) : step_t<float>(a, st);
}

hipError_t launch_attn_bwd(const AttnBwdArgs& a, const AttnPlan& p, hipStream_t st) {
  return a.f.dtype == COMBA_BF16 ? attn_bwd_t<u16>(a, p, st) : attn_bwd_t<float>(a, p, st);
}

}  // namespace comba
