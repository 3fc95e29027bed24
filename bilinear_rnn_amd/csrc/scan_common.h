// Device code shared by the selective scan's forward and backward.
//
// A channel's SP = 4 * NPL states (S padded with states that stay 0) are spread over the 4 lanes of a
// quad, NPL consecutive states each; a wavefront holds 16 channels, a workgroup 64 channels of one
// B / C group. Why quads: the sum over a channel's states is two DPP steps, values of one token reach
// the quad's other lanes as a DPP operand of the instruction that uses them (quad_perm costs
// nothing), and 16 channels per wavefront still give a wavefront per SIMD at 16384 channels. Each
// lane owns one of four consecutive tokens for the work per (token, channel): step size, gate, loads,
// stores.
#pragma once

#include "layer.h"
#include "layer_common.h"

namespace comba {

constexpr int kScanBlock = 256;     // 4 wavefronts
constexpr int kScanChannels = 64;   // channels per workgroup

// Value of lane K of the quad.
template <int K>
__device__ __forceinline__ float quad_bcast(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), K * 0x55, 0xf, 0xf, true));
}

// v[k] summed over the quad, for the lane's own k = lane & 3.
__device__ __forceinline__ float quad_sums(const float (&v)[4], int q) {
  const bool hi = q & 2, odd = q & 1;
  const float a = (hi ? v[2] : v[0]) + dpp_flip<1>(hi ? v[0] : v[2]);
  const float b = (hi ? v[3] : v[1]) + dpp_flip<1>(hi ? v[1] : v[3]);
  return (odd ? b : a) + dpp_flip<0>(odd ? a : b);
}

__device__ __forceinline__ float quad_total(float x) {
  x += dpp_flip<0>(x);
  return x + dpp_flip<1>(x);
}

// log(1 + e^u), to float32's accuracy also where the result is small. With e = e^-|u| in (0, 1],
// log(1 + e) = 2 atanh(s), s = e / (2 + e) <= 1/3, as the odd series s + s^3/3 + s^5/5 + ...: cut
// after s^15/15, the remainder is below s (1/9)^8 / 17 * 9/8 < 2^-29 of the value.
__device__ __forceinline__ float softplus_f32(float u) {
  const float e = __builtin_amdgcn_exp2f(-kLog2E * fabsf(u));
  const float s = e * __builtin_amdgcn_rcpf(2.f + e), s2 = s * s;
  float p = 2.f / 15.f;
  p = fmaf(p, s2, 2.f / 13.f);
  p = fmaf(p, s2, 2.f / 11.f);
  p = fmaf(p, s2, 2.f / 9.f);
  p = fmaf(p, s2, 2.f / 7.f);
  p = fmaf(p, s2, 2.f / 5.f);
  p = fmaf(p, s2, 2.f / 3.f);
  p = fmaf(p, s2, 2.f);
  return fmaf(s, p, fmaxf(u, 0.f));
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

__device__ __forceinline__ ScanPlace scan_place(int64_t slot, int cb, const int32_t* cu, int N, int T, int D, int G,
                                                int L) {
  ScanPlace p;
  const int dg = D / G, per = (dg + kScanChannels - 1) / kScanChannels;
  p.g = cb / per;
  const int in = (cb - p.g * per) * kScanChannels;
  p.c0 = p.g * dg + in;
  p.cl = min(kScanChannels, dg - in);
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
