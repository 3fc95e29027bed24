// Device code shared by the selective scan's forward and backward.
//
// A channel's SP states (S padded with states that stay 0) are spread over LPC lanes, NPL consecutive
// states each; a workgroup holds channels of one B / C group.
#pragma once

#include <type_traits>

#include "layer.h"
#include "layer_common.h"

namespace comba {

// Step and backward: 64 channels in quads per workgroup.
constexpr int kScanBlock = 256, kScanChannels = 64;

template <int CTRL>
__device__ __forceinline__ float dpp_move(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}

// Value of lane K of the quad.
template <int K>
__device__ __forceinline__ float quad_bcast(float x) {
  return dpp_move<K * 0x55>(x);
}

// f(integral_constant<int, 0>{}), ..., f(integral_constant<int, N - 1>{})
template <int N, int I = 0, typename F>
__device__ __forceinline__ void each(F f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    each<N, I + 1>(f);
  }
}

// Halves over lane bits 3 and 2: of 4 N values, the lane keeps numbers k + N (2 b3 + b2), k < N, in
// v[0 .. N - 1], each summed over lane ^ 4, ^ 8 and ^ 12. A DPP addition that writes only some banks of
// four lanes makes a halving two instructions per result; selecting what to keep and what to send
// makes it three, and the compiler has no form for the other. Inside the asm: two wait states (an
// instruction is one) between a register's write and its DPP read, before the first, between the
// two halvings and behind the last. The registers written are early clobbers: they are written before
// the last inputs are read, and without that the compiler gives equal values one register.
#define COMBA_BIT3(A, B)                                                      \
  "v_add_f32_dpp " A ", " A ", " A " row_ror:8 row_mask:0xf bank_mask:0xf\n\t" \
  "v_add_f32_dpp " A ", " B ", " B " row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
#define COMBA_BIT2(A, B, WAIT)                                                       \
  "v_add_f32_dpp " A ", " A ", " A " row_shl:4 row_mask:0xf bank_mask:0x5\n\t" WAIT   \
  "v_add_f32_dpp " A ", " B ", " B " row_shr:4 row_mask:0xf bank_mask:0xa\n\t"
template <int N> __device__ __forceinline__ void halve_bits_3_2(float* v) {
  if constexpr (N == 1) {
    asm("s_nop 1\n\t" COMBA_BIT3("%0", "%2") COMBA_BIT3("%1", "%3") COMBA_BIT2("%0", "%1", "s_nop 0\n\t") "s_nop 1"
        : "+&v"(v[0]), "+&v"(v[1])
        : "v"(v[2]), "v"(v[3]));
  } else {
    static_assert(N % 2 == 0, "1 or pairs");
#pragma unroll
    for (int i = 0; i < N; i += 2)
      asm("s_nop 1\n\t" COMBA_BIT3("%0", "%4") COMBA_BIT3("%1", "%5") COMBA_BIT3("%2", "%6") COMBA_BIT3("%3", "%7")
              COMBA_BIT2("%0", "%2", "") COMBA_BIT2("%1", "%3", "") "s_nop 1"
          : "+&v"(v[i]), "+&v"(v[i + 1]), "+&v"(v[i + N]), "+&v"(v[i + 1 + N])
          : "v"(v[i + 2 * N]), "v"(v[i + 1 + 2 * N]), "v"(v[i + 3 * N]), "v"(v[i + 1 + 3 * N]));
  }
}
#undef COMBA_BIT2
#undef COMBA_BIT3

// v[k] summed over the quad, for the lane's own k.
__device__ __forceinline__ float quad_sums(float (&v)[4], int lane) {
  halve_dpp<1, 2>(v, lane);
  halve_dpp<0, 1>(v, lane);
  return v[0];
}

// x summed over the quad.
__device__ __forceinline__ float quad_total(float x) {
  x += dpp_flip<0>(x);
  return x + dpp_flip<1>(x);
}

// log(1 + e^u), without cancellation where the result is small. With e = e^-|u| in (0, 1],
// log(1 + e) = 2 atanh(s), s = e / (2 + e) <= 1/3. 2 atanh(s) / s is an even function: a polynomial of
// degree 4 in s^2, fitted on [0, 1/9] for the least relative error (Remez exchange), is 4e-9 off. The
// relative error of the result is up to about (10 + 1.3 |u|) 2^-24 for negative u, the second part from the
// rounding of u log2(e) before the exponential (see sigmoid_fast), and 10 2^-24 for positive u.
__device__ __forceinline__ float softplus_f32(float u) {
  const float e = __builtin_amdgcn_exp2f(-kLog2E * fabsf(u));
  const float s = e * __builtin_amdgcn_rcpf(2.f + e), s2 = s * s;
  float p = 0.28178334f;
  p = fmaf(p, s2, 0.27960601f);
  p = fmaf(p, s2, 0.40024909f);
  p = fmaf(p, s2, 0.66666317f);
  p = fmaf(p, s2, 2.f);
  return fmaf(s, p, fmaxf(u, 0.f));
}

// A for the base-2 exponential, kept finite: a step size of 0 (tokens behind a segment have it) leaves
// the state as it is also where A is -infinity, which forgets it at every other token.
__device__ __forceinline__ float decay_rate(float A) {
  const float r = A * kLog2E;
  return r < -3.4028235e38f ? -3.4028235e38f : r;
}

// own + 2^p h: a state carried over a segment whose decays multiply to 2^p. Where that factor leaves
// float32's range, as it does for states that grow, h may be 0 or small enough for the product to be
// finite: it is then scaled by the factor's mantissa and exponent one after the other.
__device__ __forceinline__ float carried(float h, float p, float own) {
  if (fabsf(p) < 126.f) return fmaf(__builtin_amdgcn_exp2f(p), h, own);
  const float n = rintf(__builtin_amdgcn_fmed3f(p, -1e9f, 1e9f));
  return own + __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f(p - n) * h, static_cast<int>(n));
}

// A workgroup's place: segment [t0, t1) of sequence n in batch row b, channels from c0 on.
struct ScanPlace {
  int n, b, seg, t0, t1, s0, s1;   // s0, s1: the whole sequence
  int g, c0, cl;                   // group; first channel; channels here
  int64_t slot;
  bool ok;
};

__device__ __forceinline__ int segments_of(int len, int L) {
  return L && len > L ? (len - 1) / L + 1 : 1;
}

template <int CH>
__device__ __forceinline__ ScanPlace scan_place(int64_t slot, int cb, const int32_t* cu, int N, int T, int D, int G,
                                                int L) {
  ScanPlace p;
  const int dg = D / G, per = (dg + CH - 1) / CH;
  p.g = cb / per;
  const int in = (cb - p.g * per) * CH;
  p.c0 = p.g * dg + in;
  p.cl = min(CH, dg - in);
  p.slot = slot;
  if (!cu) {
    const int per_seq = L ? (T + L - 1) / L : 1;
    p.n = static_cast<int>(slot / per_seq);
    p.seg = static_cast<int>(slot - static_cast<int64_t>(p.n) * per_seq);
    p.b = p.n;
    p.s0 = 0;
    p.s1 = T;
  } else {
    p.b = 0;
    if (!L) {
      p.n = static_cast<int>(slot);
    } else {
      // the last sequence whose first slot, start / L + n, is at or before this one
      int lo = 0, hi = N - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        int s, e;
        packed_range(cu, mid, T, s, e);
        if (s / L + mid <= slot) lo = mid; else hi = mid - 1;
      }
      p.n = lo;
    }
    packed_range(cu, p.n, T, p.s0, p.s1);
    p.seg = L ? static_cast<int>(slot - (p.s0 / L + p.n)) : 0;
  }
  // an empty sequence has one, empty, segment; slots between sequences belong to none
  p.ok = p.seg >= 0 && p.seg < segments_of(p.s1 - p.s0, L);
  p.t0 = p.s0 + (p.ok ? p.seg * L : 0);
  p.t1 = L ? p.t0 + min(L, p.s1 - p.t0) : p.s1;
  return p;
}

__device__ __forceinline__ bool last_segment(const ScanPlace& p) { return p.t1 >= p.s1; }

}  // namespace comba
