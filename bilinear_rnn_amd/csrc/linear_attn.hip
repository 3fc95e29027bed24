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

constexpr int kAttnThreads = 512;

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
  int64_t rdot_inter;         // the same of f M^T x alone, so many floats behind
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

// Tokens per chunk: what the LDS holds twice.
template <typename T> __host__ __device__ constexpr int attn_chunk(int AP) {
  return (sizeof(T) == 2 ? 64 : 32) / (AP > 128 ? 2 : 1);
}

// One chunk's tensors, scores and decays in LDS.
template <typename T, int AP, int NT, bool STATE> struct AttnChunk {
  typedef Tiles<T> Ti;
  static constexpr int CH = attn_chunk<T>(AP);
  alignas(16) T xs[STATE ? 8 : Ti::size(CH, AP)];
  alignas(16) T ys[Ti::size(CH, AP)];
  alignas(16) T zs[Ti::size(CH, kAttnBlock)];
  alignas(16) T ps[STATE ? 8 : Ti::score_elems(CH, Ti::TERMS(NT))];
  alignas(16) float gh[CH];     // sums of log2 decays from the chunk's first token on, in two terms
  alignas(16) float gl[CH];
  alignas(16) float fs[CH];     // f_u, r_w and the whole chunk's decay
  alignas(16) float rs[CH];
  float whole;
};

// AP: A padded to 64, 128 or 256. NT: terms that float32 operands of a bf16 product are split into.
// STATE: the segment's own state alone (from 0, no outputs).
// Wavefronts 0 to 3 (consumers) hold 16 columns of M each and run the chunks; wavefronts 4 to 7 (producers)
// bring the next chunk into LDS and form its scores, which do not depend on M, and have the loads of the one
// behind that in flight.
// WHOLE: A and Z are multiples of a 16-byte piece.
template <typename T, int AP, int NT, bool STATE, bool WHOLE>
__global__ __launch_bounds__(kAttnThreads) __attribute__((amdgpu_waves_per_eu(2, STATE ? 4 : 2))) void attn_kernel(AttnK<T> a) {
  typedef Tiles<T> Ti;
  typedef typename Ti::Frag Frag;
  typedef AttnChunk<T, AP, NT, STATE> Chunk;
  constexpr int CH = Chunk::CH, BLK = Ti::BLK, E = Ti::PIECE, ZB = kAttnBlock;
  constexpr int NM = AP / 16, NA = AP / BLK, NS = CH / BLK, NU = CH / 16, EL = BLK / 4;
  constexpr int NTM = Ti::TERMS(NT), NTZ = Ti::TERMS(3);
  constexpr int PT = 256;  // producer threads
  constexpr int XP = CH * AP / E / PT, ZP = (CH * ZB / E + PT - 1) / PT;  // pieces per producer
  typedef Pieces<T, WHOLE> Piece;
  __shared__ Chunk chunk[2];
  __shared__ float dots[STATE ? 1 : 2][2][4][STATE ? 1 : CH];  // of two iterations: all, the states' part
  __shared__ int produced;
  static_assert(sizeof(chunk) + sizeof(dots) <= 160 * 1024, "LDS");

  const int tid = threadIdx.x, w = tid >> 6, lane = tid & 63, g = lane >> 4, l16 = lane & 15;
  const bool producer = w >= 4;
  // the workgroups of one (segment, head) on one XCD, whose L2 they share
  const int per_unit = attn_unit_blocks(a);
  const int64_t unit = static_cast<int64_t>(blockIdx.x / (8 * per_unit)) * 8 + blockIdx.x % 8;
  if (unit >= a.slots * a.H) return;
  int zb = blockIdx.x / 8 % per_unit, ri = 0;
  const bool first_block = zb == 0;
  while (zb >= attn_blocks(a.role[ri].Z)) zb -= attn_blocks(a.role[ri++].Z);
  const AttnRole<T> R = a.role[ri];
  const int64_t slot = unit / a.H;
  const int h = static_cast<int>(unit - slot * a.H);
  const ScanPlace pl = scan_place<1>(slot, 0, a.cu_seqlens, a.N, a.Tn, 1, 1, a.L);
  if (!pl.ok) return;
  const bool last = last_segment(pl), back = R.back;
  if (STATE && last && !a.whole_pass) return;
  const int chunks = (pl.t1 - pl.t0 + CH - 1) / CH;
  const int z0 = zb * ZB;                                   // first column of the block
  const int64_t row0 = static_cast<int64_t>(pl.b) * a.Tn;   // token 0 of the batch row
  const int64_t KV = static_cast<int64_t>(a.K) * a.V;
  auto first_token = [&](int it) { return pl.t0 + (back ? chunks - 1 - it : it) * CH; };

  if (!STATE) {  // score tiles beyond the diagonal stay 0
    for (int i = tid; i < 2 * Ti::score_elems(CH, NTM); i += kAttnThreads)
      chunk[i / Ti::score_elems(CH, NTM)].ps[i % Ti::score_elems(CH, NTM)] = 0;
    if (tid == 0) produced = 0;
  }

  if (producer) {
    const int pt = tid - 256, pw = w - 4;
    u32x4 xr[STATE ? 1 : XP], yr[XP], zr[ZP];
    float gr = 0.f;
    double total = 0.0;
    const int xs_ = R.xh * R.A, ys_ = R.yh * R.A, zs_ = R.zh * R.Z;  // elements from a token to the next
    const T* const xb = STATE ? nullptr : R.x + row0 * xs_ + h / (a.H / R.xh) * R.A;
    const T* const yb = R.y + row0 * ys_ + h / (a.H / R.yh) * R.A;
    const T* const zbase = R.z + row0 * zs_ + h / (a.H / R.zh) * R.Z;
    uint32_t xo[STATE ? 1 : XP], yo[XP], zo[ZP];
#pragma unroll
    for (int i = 0; i < XP; ++i) {
      const int p = pt + i * PT, r = p / (AP / E), col = p % (AP / E) * E;
      if (!STATE) xo[i] = Piece::offset(r, col, xs_, R.A);
      yo[i] = Piece::offset(r, col, ys_, R.A);
    }
#pragma unroll
    for (int i = 0; i < ZP; ++i) {
      const int p = pt + i * PT;
      zo[i] = Piece::offset(p / (ZB / E), z0 + p % (ZB / E) * E, zs_, R.Z);
    }
    auto fetch = [&](int it) {
      const int t0 = first_token(it), n = min(CH, pl.t1 - t0);
      const typename Piece::Rows xc{STATE ? nullptr : xb + static_cast<int64_t>(t0) * xs_, n, xs_, R.A},
          yc{yb + static_cast<int64_t>(t0) * ys_, n, ys_, R.A}, zc{zbase + static_cast<int64_t>(t0) * zs_, n, zs_, R.Z};
#pragma unroll
      for (int i = 0; i < XP; ++i) {
        const int r = (pt + i * PT) / (AP / E);
        if (!STATE) xr[i] = Piece::fetch(xc, xo[i], r);
        yr[i] = Piece::fetch(yc, yo[i], r);
      }
#pragma unroll
      for (int i = 0; i < ZP; ++i) zr[i] = Piece::fetch(zc, zo[i], (pt + i * PT) / (ZB / E));
      if (pw == 0) {
        const int r = min(lane, n - 1);
        gr = lane < n ? (a.per_token ? a.log_decay[(row0 + t0 + r) * a.H + h] : a.log_decay[h]) : 0.f;
      }
    };
    auto stage = [&](int it) {
      Chunk& ck = chunk[it & 1];
      const int t0 = first_token(it), n = min(CH, pl.t1 - t0);
#pragma unroll
      for (int i = 0; i < XP; ++i) {
        const int p = pt + i * PT, r = p / (AP / E), col = p % (AP / E) * E;
        if (!STATE) *reinterpret_cast<u32x4*>(ck.xs + Ti::template at<AP>(r, col)) = Piece::place(xr[i], r, n, col, R.A);
        *reinterpret_cast<u32x4*>(ck.ys + Ti::template at<AP>(r, col)) = Piece::place(yr[i], r, n, col, R.A);
      }
#pragma unroll
      for (int i = 0; i < ZP; ++i) {
        const int p = pt + i * PT, r = p / (ZB / E), col = p % (ZB / E) * E;
        if (CH * ZB / E % PT == 0 || r < CH)
          *reinterpret_cast<u32x4*>(ck.zs + Ti::template at<ZB>(r, col)) = Piece::place(zr[i], r, n, z0 + col, R.Z);
      }
      if (pw == 0) {
        // sums of log2 decays, in 64 bits: their differences are small beside them
        const float gl = gr < kLeastDecay ? kLeastDecay : gr;
        const double G = wave_scan_f64_dpp(static_cast<double>(gl) * 1.4426950408889634);
        const double all = __shfl(G, 63, kWave);
        const float since = __builtin_amdgcn_exp2f(static_cast<float>(G));
        const float rest = __builtin_amdgcn_exp2f(static_cast<float>(all - G));
        if (lane < CH) {
          ck.gh[lane] = static_cast<float>(G);
          ck.gl[lane] = static_cast<float>(G - static_cast<float>(G));
          ck.fs[lane] = R.f_state * (back ? rest : since);
          ck.rs[lane] = R.f_into * (back ? since : rest);
        }
        if (lane == 0) ck.whole = __builtin_amdgcn_exp2f(static_cast<float>(all));
        total += all;
      }
    };
    // tiles (target i, source j) on and below the diagonal, above it when time runs back
    auto scores = [&](int it) {
      Chunk& ck = chunk[it & 1];
      constexpr int tiles = NU * (NU + 1) / 2, TPW = (tiles + 3) / 4;
      int ti[TPW], tj[TPW];
      f32x4 s[TPW], d[TPW];
#pragma unroll
      for (int q = 0; q < TPW; ++q) {
        const int k = min(pw + 4 * q, tiles - 1);
        int i = 0;
#pragma unroll
        for (int n = 1; n < NU; ++n) i += k >= n * (n + 1) / 2;
        const int j = k - i * (i + 1) / 2;
        ti[q] = back ? NU - 1 - i : i;
        tj[q] = back ? NU - 1 - j : j;
        s[q] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
#pragma unroll
      for (int q = 0; q < TPW; ++q) {
        const int t = 16 * ti[q] + l16;
        const float sign = back ? -1.f : 1.f, h0 = sign * ck.gh[t], l0 = sign * ck.gl[t];
        const f32x4 h1 = *reinterpret_cast<const f32x4*>(ck.gh + 16 * tj[q] + 4 * g),
                    l1 = *reinterpret_cast<const f32x4*>(ck.gl + 16 * tj[q] + 4 * g);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          d[q][r] = R.f_score * __builtin_amdgcn_exp2f(fmaf(-sign, h1[r], h0) + fmaf(-sign, l1[r], l0));
      }
#pragma unroll
      for (int p = 0; p < NA; ++p)
#pragma unroll
        for (int q = 0; q < TPW; ++q)
          s[q] = Ti::mma(Ti::template along<AP>(ck.ys, 16 * tj[q] + l16, p, g),
                         Ti::template along<AP>(ck.xs, 16 * ti[q] + l16, p, g), s[q]);
#pragma unroll
      for (int q = 0; q < TPW; ++q) {
        if (pw + 4 * q >= tiles) continue;
        const int t = 16 * ti[q] + l16;
#pragma unroll
        for (int r = 0; r < 4; ++r) {  // a masked score is 0 whatever the product is
          const int since = t - (16 * tj[q] + 4 * g + r);
          float x = s[q][r] * d[q][r];
          pin(x);
          s[q][r] = (back ? -since : since) >= 0 ? x : 0.f;
        }
        Ti::template put_scores<CH, NTM>(ck.ps, t, tj[q], g, s[q]);
      }
    };
    auto put_dots = [&](int it) {
      if constexpr (STATE) return;
      const int t0 = first_token(it);
      if (R.own && pt < CH && pt < pl.t1 - t0) {
        const auto& d = dots[it & 1];
        float* const to = R.rdot + (static_cast<int64_t>(zb) * a.H + h) * a.tokens + row0 + t0 + pt;
        to[0] = (d[0][0][pt] + d[0][1][pt]) + (d[0][2][pt] + d[0][3][pt]);
        to[R.rdot_inter] = (d[1][0][pt] + d[1][1][pt]) + (d[1][2][pt] + d[1][3][pt]);
      }
    };
    int epoch = 0;
    // iteration `it` of the consumers, and two before their first
    for (int it = -2; it < chunks; ++it) {
      const bool next = it >= -1 && it + 1 < chunks;
      if (next) stage(it + 1);
      if (it + 2 < chunks) fetch(it + 2);
      if (it == -2) {
        if (!STATE) __syncthreads();  // the scores are cleared
        continue;
      }
      if constexpr (!STATE) {
        if (next) {
          producer_sync(&produced, epoch, lane);
          scores(it + 1);
        }
        if (it > 0) put_dots(it - 1);
      }
      __syncthreads();
    }
    if constexpr (!STATE) {
      if (chunks > 0) put_dots(chunks - 1);
    }
    if (STATE && first_block && pt == 0) a.decay[unit] = total;
    return;
  }

  // consumers
  const StateMap sm{a.K, R.A, R.Z, R.a_is_k};
  const int zc = z0 + 16 * w + l16;  // this lane's column of M
  f32x4 m[NM];
  const float* from = nullptr;
  if (!STATE) {
    if (R.state && (a.whole_pass || segments_of(pl.s1 - pl.s0, a.L) > 1)) from = R.state + unit * KV;
    else if (a.init) from = a.init + (static_cast<int64_t>(pl.n) * a.H + h) * KV;
  }
#pragma unroll
  for (int j = 0; j < NM; ++j) m[j] = from ? sm.load(from, Ti::index(j, g, 0), zc) : f32x4{0.f, 0.f, 0.f, 0.f};
  // waits for them here: a wait in the loop would be one for the stores of every chunk
#pragma unroll
  for (int j = 0; j < NM; ++j) asm volatile("" : "+v"(m[j]));
  const int z = z0 + 16 * w + 4 * g;  // this lane's first output column
  const int64_t first_out = ((row0 + pl.t0 + l16) * a.H + h) * R.Z + z, out_stride = static_cast<int64_t>(a.H) * R.Z;
  const T* const own = R.own ? R.own + ((row0 + pl.t0 + l16) * R.own_h + h / (a.H / R.own_h)) * R.Z + z : nullptr;
  const int64_t own_stride = static_cast<int64_t>(R.own_h) * R.Z;
  if (!STATE) __syncthreads();
  __syncthreads();
  for (int it = 0; it < chunks; ++it) {
    const Chunk& ck = chunk[it & 1];
    Frag zf[NS];
#pragma unroll
    for (int b = 0; b < NS; ++b) zf[b] = Ti::template down<ZB>(ck.zs, b, 16 * w, g, l16);
    if constexpr (!STATE) {
      const int t0 = first_token(it), n = min(CH, pl.t1 - t0);
      f32x4 o[NU];
#pragma unroll
      for (int i = 0; i < NU; ++i) o[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int p = 0; p < NA; ++p) {
        Frag mf[NTM];
        Ti::template from_tiles<NTM>(m, p, mf);
#pragma unroll
        for (int i = 0; i < NU; ++i) {
          const Frag x = Ti::template along<AP>(ck.xs, 16 * i + l16, p, g);
#pragma unroll
          for (int k = 0; k < NTM; ++k) o[i] = Ti::mma(mf[k], x, o[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        const int t = 16 * i + l16;
        o[i] *= ck.fs[t];
        const f32x4 inter = o[i];
#pragma unroll
        for (int b = 0; b < NS; ++b) {
          if (back ? BLK * (b + 1) <= 16 * i : BLK * b > 16 * i) continue;
#pragma unroll
          for (int k = 0; k < NTM; ++k) o[i] = Ti::mma(zf[b], Ti::template scores<CH>(ck.ps, k, t, b, g), o[i]);
        }
        const int left = t < n ? R.Z - z : 0, since = t0 - pl.t0 + 16 * i;
        float ov[4] = {o[i][0], o[i][1], o[i][2], o[i][3]};
        if (left > 0) {
          const int64_t at = first_out + since * out_stride;
          if (R.out) Pack<T, 4, WHOLE>::store(R.out + at, ov, min(left, 4));
          else Pack<float, 4, WHOLE>::store(R.out32 + at, ov, min(left, 4));
        }
        if (R.own) {
          float d = 0.f, di = 0.f;
          if (left > 0) {
            float x[4];
            Pack<T, 4, WHOLE>::load(own + since * own_stride, x, min(left, 4));
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              d = fmaf(x[r], ov[r], d);
              di = fmaf(x[r], inter[r], di);
            }
          }
          d += __shfl_xor(d, 16, kWave);
          d += __shfl_xor(d, 32, kWave);
          di += __shfl_xor(di, 16, kWave);
          di += __shfl_xor(di, 32, kWave);
          if (g == 0) {
            dots[it & 1][0][w][t] = d;
            dots[it & 1][1][w][t] = di;
          }
        }
      }
    }
    // into the state
    const float keep = ck.whole;
#pragma unroll
    for (int j = 0; j < NM; ++j) m[j] *= keep;
#pragma unroll
    for (int b = 0; b < NS; ++b) {
      float zw[EL];
      Frag zt[NTZ];
#pragma unroll
      for (int e = 0; e < EL; ++e) zw[e] = Ti::value(zf[b], e) * ck.rs[BLK * b + Ti::down_row(g, e)];
      Ti::template split<NTZ>(zw, zt);
#pragma unroll
      for (int j = 0; j < NM; ++j) {
        const Frag y = Ti::template down_index<AP>(ck.ys, b, j, g, l16);
#pragma unroll
        for (int k = 0; k < NTZ; ++k) m[j] = Ti::mma(y, zt[k], m[j]);
      }
    }
    __syncthreads();
  }

  float* to = nullptr;
  if (STATE) to = R.state + unit * KV;
  else if (a.fin && last) to = a.fin + (static_cast<int64_t>(pl.n) * a.H + h) * KV;
  if (to)
#pragma unroll
    for (int j = 0; j < NM; ++j) sm.store(to, Ti::index(j, g, 0), zc, m[j]);
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

// dlog_decay of a segment and head per wavefront: sums from the segment's end, in 64 bits. Over a whole
// chunk the scores' parts of q . dq and k . dk have the same sum, so only the parts that come from
// the states are carried from chunk to chunk: what is rounded in the others stays within the chunk.
// rdot: [q and k][all and states' part][Z blocks, H, tokens].
__global__ __launch_bounds__(256) void attn_decay_grad_kernel(const float* __restrict__ rdot, const double* __restrict__ inner,
                                                              const int32_t* __restrict__ cu, int N, int T, int H, int L,
                                                              int CH, int64_t slots, int64_t tokens, int zblocks,
                                                              int eblocks, float* __restrict__ out,
                                                              double* __restrict__ hsum) {
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
  const int64_t row0 = static_cast<int64_t>(pl.b) * T, one = static_cast<int64_t>(zblocks) * H * tokens;
  for (int c = (pl.t1 - pl.t0 - 1) / CH; c >= 0; --c) {  // lane l: the chunk's token CH - 1 - l
    const int t = pl.t0 + c * CH + CH - 1 - lane;
    double r = 0.0, ri = 0.0;
    if (lane < CH && t < pl.t1)
      for (int zb = 0; zb < zblocks; ++zb) {
        const float* const at = rdot + (static_cast<int64_t>(zb) * H + h) * tokens + row0 + t;
        r += static_cast<double>(at[0]) - static_cast<double>(at[2 * one]);
        ri += static_cast<double>(at[one]) - static_cast<double>(at[3 * one]);
      }
    const double s = wave_scan_f64_dpp(r) + carry;
    carry += __shfl(wave_scan_f64_dpp(ri), 63, kWave);
    if (lane < CH && t < pl.t1) {
      sum += s;
      if (!hsum) out[(row0 + t) * H + h] = static_cast<float>(s);
    }
  }
  if (hsum) {
    sum = wave_scan_f64_dpp(sum);
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
  s = wave_scan_f64_dpp(s);
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

template <typename T, int NT, bool STATE, bool WHOLE> hipError_t run_attn_w(const AttnK<T>& k, int A, hipStream_t st) {
  const int64_t units = (k.slots * k.H + 7) / 8 * 8;
  const unsigned grid = static_cast<unsigned>(units * attn_unit_blocks(k));
  if (A <= 64) attn_kernel<T, 64, NT, STATE, WHOLE><<<grid, kAttnThreads, 0, st>>>(k);
  else if (A <= 128) attn_kernel<T, 128, NT, STATE, WHOLE><<<grid, kAttnThreads, 0, st>>>(k);
  else attn_kernel<T, 256, NT, STATE, WHOLE><<<grid, kAttnThreads, 0, st>>>(k);
  return hipGetLastError();
}

// float32 products take values whole: one instance serves any number of terms.
template <typename T, int NT, bool STATE> hipError_t run_attn(const AttnK<T>& k, int A, hipStream_t st) {
  constexpr int E = Tiles<T>::PIECE, N = sizeof(T) == 2 ? NT : 2;
  bool whole = k.K % E == 0 && k.V % E == 0;
  for (int r = 0; r < k.roles; ++r)
    whole = whole && (reinterpret_cast<uintptr_t>(k.role[r].x) | reinterpret_cast<uintptr_t>(k.role[r].y) |
                      reinterpret_cast<uintptr_t>(k.role[r].z)) % 16 == 0;
  return whole ? run_attn_w<T, N, STATE, true>(k, A, st) : run_attn_w<T, N, STATE, false>(k, A, st);
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
  k.role[0] = AttnRole<T>{q, kk, v, static_cast<T*>(f.o), nullptr, nullptr, nullptr, 0, w.state, f.Hk, f.Hk, f.H, 1,
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
  k.role[0] = AttnRole<T>{nullptr, kk, v, nullptr, nullptr, nullptr, nullptr, 0, a.state, Hk, Hk, H, 1, K, V, false, true,
                          0.f, 0.f, 1.f};
  k.role[1] = AttnRole<T>{nullptr, q, dO, nullptr, nullptr, nullptr, nullptr, 0, a.grad, Hk, Hk, H, 1, K, V, true, true,
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
  const int64_t one = static_cast<int64_t>(zblocks) * H * k.tokens;
  float* const rk = a.rdot + 2 * one;
  const AttnRole<T> rq_{dO, v, kk, dq, a.dqk, q, a.rdot, one, a.state, H, H, Hk, Hk, V, K, false, false, f.scale, f.scale, 1.f};
  const AttnRole<T> rk_{v, dO, q, dk, dk32, kk, rk, one, a.grad, H, H, Hk, Hk, V, K, true, false, 1.f, f.scale, f.scale};
  const AttnRole<T> rv_{kk, q, dO, static_cast<T*>(a.dv), nullptr, nullptr, nullptr, 0, a.grad, Hk, Hk, H, 1, K, V, true, true,
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
      a.rdot, a.inner, f.cu_seqlens, f.N, f.T, H, p.L, attn_chunk<T>(padded(V)), p.slots, k.tokens, zblocks, eblocks, a.dlog_decay,
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
