// C ABI entry points of the layer operators (declared in include/comba.h): host-side validation,
// workspace carving and launches on the caller's stream.
#include <climits>
#include <cmath>
#include <initializer_list>

#include "comba.h"
#include "layer.h"

#define COMBA_API extern "C" __attribute__((visibility("default")))

namespace {

using comba::report;
using comba::report_launch;

constexpr int32_t kMaxWidth = 1 << 22;
// The kernels step through tokens in tiles with 32-bit counters, which run past the last token by
// less than two tiles.
constexpr int64_t kMaxTokens = INT_MAX - 0xffff;
constexpr int64_t kMaxThreads = UINT_MAX;               // of one launch
constexpr int64_t kMaxBlocks = kMaxThreads / 256 - 8;   // workgroups of 256, their number rounded up to 8

size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

bool known_dtype(int32_t d) { return d == COMBA_BF16 || d == COMBA_FP32; }
int64_t size_of(int32_t d) { return d == COMBA_BF16 ? 2 : 4; }

bool overlaps(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + static_cast<uintptr_t>(nb) && y < x + static_cast<uintptr_t>(na);
}

bool misaligned(const void* p, int64_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

// Batch sizes and packing, shared by the sequence operators; N is set to the number of sequences.
int32_t check_batch(const int32_t* cu, int32_t num_seqs, int32_t B, int32_t T, int64_t& N) {
  if (B < 1) return report(COMBA_ERR_INVALID_ARG, "B must be >= 1");
  if (cu) {
    if (B != 1) return report(COMBA_ERR_INVALID_ARG, "cu_seqlens requires B == 1");
    if (num_seqs < 1) return report(COMBA_ERR_INVALID_ARG, "cu_seqlens requires num_seqs >= 1");
    if (T < 0) return report(COMBA_ERR_INVALID_ARG, "T must be >= 0");
  } else if (T < 1) {
    return report(COMBA_ERR_INVALID_ARG, "T must be >= 1 without cu_seqlens");
  }
  N = cu ? num_seqs : B;
  if (static_cast<int64_t>(B) * T > kMaxTokens) return report(COMBA_ERR_UNSUPPORTED, "more than 2^31 - 2^16 tokens");
  return COMBA_OK;
}

int32_t check_workspace(const void* ws, size_t have, size_t need, const char* what) {
  if (need == 0) return COMBA_OK;
  if (!ws || have < need) return report(COMBA_ERR_WORKSPACE, what);
  if (misaligned(ws, 256)) return report(COMBA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  return COMBA_OK;
}

struct Span {  // a tensor, or nothing
  const void* p;
  int64_t bytes;
};

// Outputs lie apart from the inputs and from each other.
int32_t check_apart(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (auto o = outs.begin(); o != outs.end(); ++o) {
    for (const Span& i : ins)
      if (overlaps(o->p, o->bytes, i.p, i.bytes)) return report(COMBA_ERR_INVALID_ARG, "an output overlaps an input");
    for (auto u = o + 1; u != outs.end(); ++u)
      if (overlaps(o->p, o->bytes, u->p, u->bytes)) return report(COMBA_ERR_INVALID_ARG, "two outputs overlap");
  }
  return COMBA_OK;
}

// --- short convolution ---------------------------------------------------------------------------

int32_t check_conv(const void* x, const float* weight, int32_t D, int32_t W, int32_t dtype) {
  if (!x || !weight) return report(COMBA_ERR_INVALID_ARG, "x and weight must be non-NULL");
  if (!known_dtype(dtype)) return report(COMBA_ERR_INVALID_ARG, "dtype must be COMBA_BF16 or COMBA_FP32");
  if (D < 1 || W < 1) return report(COMBA_ERR_INVALID_ARG, "D and W must be >= 1");
  if (W < 2 || W > 4) return report(COMBA_ERR_UNSUPPORTED, "only convolutions of 2, 3 or 4 taps are implemented");
  if (D > kMaxWidth) return report(COMBA_ERR_UNSUPPORTED, "D above 2^22");
  return COMBA_OK;
}

// Threads of the largest launch: one per four channels of every tile and state.
int32_t check_conv_items(int64_t B, int64_t T, int64_t D, int64_t N, bool packed) {
  const int64_t fwd = comba::conv_tiles(B, T, D, packed), bwd = 4 * comba::conv_bwd_sets(B, T, D, packed);
  if (((fwd > bwd ? fwd : bwd) + N + 4) * ((D + 3) / 4 + 64) > INT_MAX)
    return report(COMBA_ERR_UNSUPPORTED, "too many (token tile, channel) pairs for one launch");
  return COMBA_OK;
}

}  // namespace

COMBA_API int32_t comba_short_conv_fwd(const void* x, const float* weight, const float* bias,
                                       const void* initial_state, const int32_t* cu_seqlens, int32_t num_seqs,
                                       int32_t B, int32_t T, int32_t D, int32_t W, int32_t dtype, int32_t silu,
                                       void* y, void* final_state, void* stream) {
  int32_t rc = check_conv(x, weight, D, W, dtype);
  if (rc != COMBA_OK) return rc;
  if (!y) return report(COMBA_ERR_INVALID_ARG, "y must be non-NULL");
  int64_t N = 0;
  if ((rc = check_batch(cu_seqlens, num_seqs, B, T, N)) != COMBA_OK) return rc;
  if ((rc = check_conv_items(B, T, D, N, cu_seqlens != nullptr)) != COMBA_OK) return rc;
  const int64_t state = N * (W - 1) * D * size_of(dtype);
  if (overlaps(initial_state, state, final_state, state))
    return report(COMBA_ERR_INVALID_ARG, "final_state overlaps initial_state (only the single-token form works in place)");
  const int64_t act = static_cast<int64_t>(B) * T * D * size_of(dtype);
  rc = check_apart({{y, act}, {final_state, state}},
                   {{x, act}, {weight, 4ll * D * W}, {bias, 4ll * D}, {initial_state, state},
                    {cu_seqlens, 4 * (N + 1)}});
  if (rc != COMBA_OK) return rc;
  const comba::ConvArgs a{x, weight, bias, initial_state, cu_seqlens, static_cast<int>(N), B, T, D, W, dtype,
                          silu != 0, y, final_state};
  return report_launch(comba::launch_conv(a, static_cast<hipStream_t>(stream)));
}

COMBA_API int32_t comba_short_conv_step(const void* x, const float* weight, const float* bias,
                                        const void* initial_state, int32_t N, int32_t D, int32_t W, int32_t dtype,
                                        int32_t silu, void* y, void* final_state, void* stream) {
  int32_t rc = check_conv(x, weight, D, W, dtype);
  if (rc != COMBA_OK) return rc;
  if (!y) return report(COMBA_ERR_INVALID_ARG, "y must be non-NULL");
  if (N < 1) return report(COMBA_ERR_INVALID_ARG, "N must be >= 1");
  if (static_cast<int64_t>(N) * D > INT_MAX)
    return report(COMBA_ERR_UNSUPPORTED, "too many (sequence, channel) pairs for one launch");
  const int64_t state = static_cast<int64_t>(N) * (W - 1) * D * size_of(dtype);
  if (initial_state != final_state && overlaps(initial_state, state, final_state, state))
    return report(COMBA_ERR_INVALID_ARG, "final_state partially overlaps initial_state");
  const Span in{x, static_cast<int64_t>(N) * D * size_of(dtype)}, w{weight, 4ll * D * W}, b{bias, 4ll * D};
  if ((rc = check_apart({{y, in.bytes}}, {in, w, b, {initial_state, state}, {final_state, state}})) != COMBA_OK ||
      (rc = check_apart({{final_state, state}}, {in, w, b})) != COMBA_OK)
    return rc;
  const comba::ConvArgs a{x, weight, bias, initial_state, nullptr, N, N, 1, D, W, dtype, silu != 0, y, final_state};
  return report_launch(comba::launch_conv_step(a, static_cast<hipStream_t>(stream)));
}

COMBA_API size_t comba_short_conv_bwd_workspace_size(int32_t B, int32_t T, int32_t D, int32_t W, int32_t num_seqs) {
  if (B < 1 || T < 0 || D < 1 || W < 2 || W > 4 || D > kMaxWidth) return 0;
  return up256(sizeof(float) * comba::conv_bwd_sets(B, T, D, num_seqs > 0) * (W + 1) * static_cast<size_t>(D));
}

COMBA_API int32_t comba_short_conv_bwd(const void* x, const float* weight, const float* bias,
                                       const void* initial_state, const int32_t* cu_seqlens, int32_t num_seqs,
                                       int32_t B, int32_t T, int32_t D, int32_t W, int32_t dtype, int32_t silu,
                                       const void* dy, int32_t dy_dtype, const void* d_final_state, void* dx,
                                       float* dweight, float* dbias, void* d_initial_state, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  int32_t rc = check_conv(x, weight, D, W, dtype);
  if (rc != COMBA_OK) return rc;
  if (!dy || !dx || !dweight) return report(COMBA_ERR_INVALID_ARG, "dy, dx and dweight must be non-NULL");
  if (!known_dtype(dy_dtype) || (dy_dtype == COMBA_BF16 && dtype != COMBA_BF16))
    return report(COMBA_ERR_INVALID_ARG, "dy_dtype must be dtype or COMBA_FP32");
  int64_t N = 0;
  if ((rc = check_batch(cu_seqlens, num_seqs, B, T, N)) != COMBA_OK) return rc;
  if ((rc = check_conv_items(B, T, D, N, cu_seqlens != nullptr)) != COMBA_OK) return rc;
  const size_t need = comba_short_conv_bwd_workspace_size(B, T, D, W, cu_seqlens ? num_seqs : 0);
  rc = check_workspace(workspace, workspace_bytes, need,
                       "workspace is NULL or smaller than comba_short_conv_bwd_workspace_size()");
  if (rc != COMBA_OK) return rc;
  const int64_t elems = static_cast<int64_t>(B) * T * D, act = elems * size_of(dtype);
  const int64_t state = N * (W - 1) * D * size_of(dtype);
  rc = check_apart({{dx, act}, {dweight, 4ll * D * W}, {dbias, 4ll * D}, {d_initial_state, state},
                    {workspace, static_cast<int64_t>(need)}},
                   {{x, act}, {weight, 4ll * D * W}, {bias, 4ll * D}, {initial_state, state},
                    {cu_seqlens, 4 * (N + 1)}, {dy, elems * size_of(dy_dtype)}, {d_final_state, state}});
  if (rc != COMBA_OK) return rc;
  const comba::ConvBwdArgs a{{x, weight, bias, initial_state, cu_seqlens, static_cast<int>(N), B, T, D, W, dtype,
                              silu != 0, nullptr, nullptr},
                             dy, dy_dtype, d_final_state, dx, dweight, dbias, d_initial_state,
                             static_cast<float*>(workspace)};
  return report_launch(comba::launch_conv_bwd(a, static_cast<hipStream_t>(stream)));
}

// --- selective scan ------------------------------------------------------------------------------

namespace {

int32_t check_scan(const void* x, const void* dt, const float* A, const void* Bm, const void* Cm, int32_t D, int32_t S,
                   int32_t G, int32_t dtype) {
  if (!x || !dt || !A || !Bm || !Cm) return report(COMBA_ERR_INVALID_ARG, "x, dt, A, Bm and Cm must be non-NULL");
  if (!known_dtype(dtype)) return report(COMBA_ERR_INVALID_ARG, "dtype must be COMBA_BF16 or COMBA_FP32");
  if (D < 1 || S < 1) return report(COMBA_ERR_INVALID_ARG, "D and S must be >= 1");
  if (G < 1 || D % G != 0) return report(COMBA_ERR_INVALID_ARG, "G must be >= 1 and divide D");
  if (S > comba::kScanMaxStates) return report(COMBA_ERR_UNSUPPORTED, "more than 64 states per channel");
  if (D > kMaxWidth) return report(COMBA_ERR_UNSUPPORTED, "D above 2^22");
  if (static_cast<int64_t>(G) * S > 1 << 23)  // a tile of B or C is addressed with 32-bit offsets
    return report(COMBA_ERR_UNSUPPORTED, "G * S above 2^23");
  return COMBA_OK;
}

// `carried`: the states that a launch with a thread each carries across segments.
int32_t check_scan_grid(int64_t slots, int64_t blocks, int64_t carried) {
  if (slots * blocks > kMaxBlocks || carried > kMaxThreads - 255)
    return report(COMBA_ERR_UNSUPPORTED, "too many (segment, channel) pairs for one launch");
  return COMBA_OK;
}

int32_t check_states(const float* s0, const float* sf, int64_t bytes) {
  if (s0 != sf && overlaps(s0, bytes, sf, bytes))
    return report(COMBA_ERR_INVALID_ARG, "final_state partially overlaps initial_state");
  return COMBA_OK;
}

struct ScanWorkspace {  // offsets of a cut forward's parts
  size_t dsum, total;
};
ScanWorkspace scan_workspace(const comba::ScanPlan& p, int64_t D, int64_t SP) {
  ScanWorkspace w{0, 0};
  if (!p.L) return w;
  w.dsum = up256(sizeof(float) * p.slots * D * SP);
  w.total = w.dsum + up256(sizeof(float) * p.slots * D);
  return w;
}

struct ScanBwdWorkspace {
  size_t gseg, dsum, dA, dD, dBC, total;
};
ScanBwdWorkspace scan_bwd_workspace(const comba::ScanPlan& p, int64_t rows, int64_t D, int64_t SP, int64_t G) {
  const size_t states = up256(sizeof(float) * p.slots * D * SP), f = sizeof(float);
  ScanBwdWorkspace w;
  w.gseg = states;
  w.dsum = 2 * states;
  w.dA = w.dsum + up256(f * p.slots * D);
  w.dD = w.dA + states;
  w.dBC = w.dD + up256(f * p.slots * 2 * D);
  w.total = w.dBC + up256(f * (comba::scan_bwd_channel_blocks(D, G) / G) * rows * G * 2 * SP);
  return w;
}

bool scan_sizes_ok(int32_t B, int32_t T, int32_t D, int32_t S, int32_t G) {
  return B >= 1 && T >= 0 && D >= 1 && D <= kMaxWidth && S >= 1 && S <= comba::kScanMaxStates && G >= 1 &&
         D % G == 0 && static_cast<int64_t>(B) * T <= kMaxTokens;
}

}  // namespace

COMBA_API size_t comba_selective_scan_workspace_size(int32_t B, int32_t T, int32_t D, int32_t S, int32_t G,
                                                     int32_t num_seqs) {
  if (!scan_sizes_ok(B, T, D, S, G)) return 0;
  const comba::ScanPlan p = comba::scan_plan(B, T, D, G, num_seqs > 0 ? num_seqs : B, num_seqs > 0);
  return scan_workspace(p, D, comba::scan_padded_states(S)).total;
}

COMBA_API int32_t comba_selective_scan_fwd(const void* x, const void* dt, const float* A, const void* Bm,
                                           const void* Cm, const float* skip, const void* z, const float* dt_bias,
                                           int32_t softplus, const float* initial_state, const int32_t* cu_seqlens,
                                           int32_t num_seqs, int32_t B, int32_t T, int32_t D, int32_t S, int32_t G,
                                           int32_t dtype, void* y, float* final_state, void* workspace,
                                           size_t workspace_bytes, void* stream) {
  int32_t rc = check_scan(x, dt, A, Bm, Cm, D, S, G, dtype);
  if (rc != COMBA_OK) return rc;
  if (!y) return report(COMBA_ERR_INVALID_ARG, "y must be non-NULL");
  int64_t N = 0;
  if ((rc = check_batch(cu_seqlens, num_seqs, B, T, N)) != COMBA_OK) return rc;
  if ((rc = check_states(initial_state, final_state, N * D * S * 4)) != COMBA_OK) return rc;
  const int64_t SP = comba::scan_padded_states(S);
  const comba::ScanPlan p = comba::scan_plan(B, T, D, G, N, cu_seqlens != nullptr);
  if ((rc = check_scan_grid(p.slots, comba::scan_channel_blocks(D, G), p.L ? N * D * SP : 0)) != COMBA_OK) return rc;
  const ScanWorkspace w = scan_workspace(p, D, SP);
  rc = check_workspace(workspace, workspace_bytes, w.total,
                       "workspace is NULL or smaller than comba_selective_scan_workspace_size()");
  if (rc != COMBA_OK) return rc;
  const int64_t rows = static_cast<int64_t>(B) * T, act = rows * D * size_of(dtype);
  const int64_t bc = rows * G * S * size_of(dtype), state = N * D * S * 4;
  const Span sx{x, act}, sd{dt, act}, sA{A, 4ll * D * S}, sB{Bm, bc}, sC{Cm, bc}, ss{skip, 4ll * D}, sz{z, act},
      sb{dt_bias, 4ll * D}, sc{cu_seqlens, 4 * (N + 1)}, sw{workspace, static_cast<int64_t>(w.total)};
  if ((rc = check_apart({{y, act}, sw}, {sx, sd, sA, sB, sC, ss, sz, sb, sc, {initial_state, state},
                                         {final_state, state}})) != COMBA_OK ||
      (rc = check_apart({{final_state, state}}, {sx, sd, sA, sB, sC, ss, sz, sb, sc})) != COMBA_OK)
    return rc;
  char* ws = static_cast<char*>(workspace);
  const comba::ScanArgs a{x, dt, A, Bm, Cm, skip, z, dt_bias, softplus != 0, initial_state, cu_seqlens,
                          static_cast<int>(N), B, T, D, S, G, dtype, y, final_state};
  return report_launch(comba::launch_scan(a, p, p.L ? reinterpret_cast<float*>(ws) : nullptr,
                                          p.L ? reinterpret_cast<float*>(ws + w.dsum) : nullptr,
                                          static_cast<hipStream_t>(stream)));
}

COMBA_API int32_t comba_selective_step(const void* x, const void* dt, const float* A, const void* Bm, const void* Cm,
                                       const float* skip, const void* z, const float* dt_bias, int32_t softplus,
                                       const float* initial_state, int32_t N, int32_t D, int32_t S, int32_t G,
                                       int32_t dtype, void* y, float* final_state, void* stream) {
  int32_t rc = check_scan(x, dt, A, Bm, Cm, D, S, G, dtype);
  if (rc != COMBA_OK) return rc;
  if (!y) return report(COMBA_ERR_INVALID_ARG, "y must be non-NULL");
  if (N < 1) return report(COMBA_ERR_INVALID_ARG, "N must be >= 1");
  if ((rc = check_states(initial_state, final_state, static_cast<int64_t>(N) * D * S * 4)) != COMBA_OK) return rc;
  if ((rc = check_scan_grid(comba::scan_step_blocks(N, D, G), 1, 0)) != COMBA_OK) return rc;
  const int64_t act = static_cast<int64_t>(N) * D * size_of(dtype), state = static_cast<int64_t>(N) * D * S * 4;
  const int64_t bc = static_cast<int64_t>(N) * G * S * size_of(dtype);
  const Span sx{x, act}, sd{dt, act}, sA{A, 4ll * D * S}, sB{Bm, bc}, sC{Cm, bc}, ss{skip, 4ll * D}, sz{z, act},
      sb{dt_bias, 4ll * D};
  if ((rc = check_apart({{y, act}}, {sx, sd, sA, sB, sC, ss, sz, sb, {initial_state, state}, {final_state, state}})) !=
          COMBA_OK ||
      (rc = check_apart({{final_state, state}}, {sx, sd, sA, sB, sC, ss, sz, sb})) != COMBA_OK)
    return rc;
  const comba::ScanArgs a{x, dt, A, Bm, Cm, skip, z, dt_bias, softplus != 0, initial_state, nullptr, N, N, 1, D, S, G,
                          dtype, y, final_state};
  return report_launch(comba::launch_scan_step(a, static_cast<hipStream_t>(stream)));
}

COMBA_API size_t comba_selective_scan_bwd_workspace_size(int32_t B, int32_t T, int32_t D, int32_t S, int32_t G,
                                                         int32_t num_seqs) {
  if (!scan_sizes_ok(B, T, D, S, G)) return 0;
  const comba::ScanPlan p = comba::scan_bwd_plan(B, T, D, G, num_seqs > 0 ? num_seqs : B, S, num_seqs > 0);
  return scan_bwd_workspace(p, static_cast<int64_t>(B) * T, D, comba::scan_padded_states(S), G).total;
}

COMBA_API int32_t comba_selective_scan_bwd(const void* x, const void* dt, const float* A, const void* Bm,
                                           const void* Cm, const float* skip, const void* z, const float* dt_bias,
                                           int32_t softplus, const float* initial_state, const int32_t* cu_seqlens,
                                           int32_t num_seqs, int32_t B, int32_t T, int32_t D, int32_t S, int32_t G,
                                           int32_t dtype, const void* dy, const float* d_final_state, void* dx,
                                           void* ddt, float* dA, void* dBm, void* dCm, float* dskip, void* dz,
                                           float* ddt_bias, float* d_initial_state, void* workspace,
                                           size_t workspace_bytes, void* stream) {
  int32_t rc = check_scan(x, dt, A, Bm, Cm, D, S, G, dtype);
  if (rc != COMBA_OK) return rc;
  if (!dy || !dx || !ddt || !dA || !dBm || !dCm)
    return report(COMBA_ERR_INVALID_ARG, "dy, dx, ddt, dA, dBm and dCm must be non-NULL");
  if ((z == nullptr) != (dz == nullptr)) return report(COMBA_ERR_INVALID_ARG, "dz is given exactly when z is");
  int64_t N = 0;
  if ((rc = check_batch(cu_seqlens, num_seqs, B, T, N)) != COMBA_OK) return rc;
  const int64_t SP = comba::scan_padded_states(S), rows = static_cast<int64_t>(B) * T;
  const comba::ScanPlan p = comba::scan_bwd_plan(B, T, D, G, N, S, cu_seqlens != nullptr);
  if ((rc = check_scan_grid(p.slots, comba::scan_bwd_channel_blocks(D, G), N * D * SP)) != COMBA_OK) return rc;
  if (rows * G * 2 * SP + 16 * (D * SP + 2 * D) > kMaxThreads - 4096)  // the sums: 16 threads per column
    return report(COMBA_ERR_UNSUPPORTED, "too many (token, group, state) triples for one launch");
  const ScanBwdWorkspace w = scan_bwd_workspace(p, rows, D, SP, G);
  rc = check_workspace(workspace, workspace_bytes, w.total,
                       "workspace is NULL or smaller than comba_selective_scan_bwd_workspace_size()");
  if (rc != COMBA_OK) return rc;
  const int64_t act = rows * D * size_of(dtype), bc = rows * G * S * size_of(dtype), state = N * D * S * 4;
  rc = check_apart({{dx, act}, {ddt, act}, {dA, 4ll * D * S}, {dBm, bc}, {dCm, bc}, {dskip, 4ll * D}, {dz, act},
                    {ddt_bias, 4ll * D}, {d_initial_state, state}, {workspace, static_cast<int64_t>(w.total)}},
                   {{x, act}, {dt, act}, {A, 4ll * D * S}, {Bm, bc}, {Cm, bc}, {skip, 4ll * D}, {z, act},
                    {dt_bias, 4ll * D}, {initial_state, state}, {cu_seqlens, 4 * (N + 1)}, {dy, act},
                    {d_final_state, state}});
  if (rc != COMBA_OK) return rc;
  char* ws = static_cast<char*>(workspace);
  auto at = [&](size_t o) { return reinterpret_cast<float*>(ws + o); };
  const comba::ScanBwdArgs a{{x, dt, A, Bm, Cm, skip, z, dt_bias, softplus != 0, initial_state, cu_seqlens,
                              static_cast<int>(N), B, T, D, S, G, dtype, nullptr, nullptr},
                             dy, d_final_state, dx, ddt, dA, dBm, dCm, dskip, dz, ddt_bias, d_initial_state,
                             at(0), at(w.gseg), at(w.dsum), at(w.dA), at(w.dD), at(w.dBC)};
  return report_launch(comba::launch_scan_bwd(a, p, static_cast<hipStream_t>(stream)));
}

// --- block norms ---------------------------------------------------------------------------------

namespace {

int32_t check_norm(const void* y, const void* gate, const void* residual, const float* scale, const float* post,
                   const float* pre, int64_t rows, int32_t D, float eps, int32_t dtype) {
  if (!y) return report(COMBA_ERR_INVALID_ARG, "y must be non-NULL");
  if (!known_dtype(dtype)) return report(COMBA_ERR_INVALID_ARG, "dtype must be COMBA_BF16 or COMBA_FP32");
  if (rows < 0 || D < 1) return report(COMBA_ERR_INVALID_ARG, "rows must be >= 0 and D >= 1");
  if (!(eps >= 0.f) || std::isinf(eps)) return report(COMBA_ERR_INVALID_ARG, "eps must be >= 0 and finite");
  if (!gate && !residual && !scale && !post && !pre)
    return report(COMBA_ERR_INVALID_ARG, "at least one of gate, residual, scale, post_weight and pre_weight is needed");
  if (D > comba::kNormMaxWidth) return report(COMBA_ERR_UNSUPPORTED, "rows of more than 16384 elements");
  if (rows > (static_cast<int64_t>(1) << 40)) return report(COMBA_ERR_UNSUPPORTED, "more than 2^40 rows");
  return COMBA_OK;
}

}  // namespace

COMBA_API int32_t comba_block_norm_fwd(const void* y, const void* gate, const void* residual, const float* scale,
                                       const float* post_weight, const float* pre_weight, int64_t rows, int32_t D,
                                       float eps, int32_t dtype, void* r, void* n, void* stream) {
  const int32_t rc = check_norm(y, gate, residual, scale, post_weight, pre_weight, rows, D, eps, dtype);
  if (rc != COMBA_OK) return rc;
  if (!r) return report(COMBA_ERR_INVALID_ARG, "r must be non-NULL");
  if ((n == nullptr) != (pre_weight == nullptr))
    return report(COMBA_ERR_INVALID_ARG, "n is given exactly when pre_weight is");
  const int64_t act = rows * D * size_of(dtype), par = 4ll * D;
  const int32_t apart = check_apart({{r, act}, {n, act}}, {{y, act}, {gate, act}, {residual, act}, {scale, par},
                                                           {post_weight, par}, {pre_weight, par}});
  if (apart != COMBA_OK) return apart;
  const comba::NormArgs a{y, gate, residual, scale, post_weight, pre_weight, rows, D, dtype, eps, r, n};
  return report_launch(comba::launch_norm(a, static_cast<hipStream_t>(stream)));
}

COMBA_API size_t comba_block_norm_bwd_workspace_size(int64_t rows, int32_t D) {
  if (rows < 1 || D < 1 || D > comba::kNormMaxWidth) return 0;
  return up256(sizeof(float) * 3 * static_cast<size_t>(comba::norm_bwd_blocks(rows, D)) * D);
}

COMBA_API int32_t comba_block_norm_bwd(const void* y, const void* gate, const void* residual, const float* scale,
                                       const float* post_weight, const float* pre_weight, int64_t rows, int32_t D,
                                       float eps, int32_t dtype, const void* dr, const void* dn, void* dy, void* dgate,
                                       void* dresidual, float* dscale, float* dpost_weight, float* dpre_weight,
                                       void* workspace, size_t workspace_bytes, void* stream) {
  int32_t rc = check_norm(y, gate, residual, scale, post_weight, pre_weight, rows, D, eps, dtype);
  if (rc != COMBA_OK) return rc;
  if (!dy) return report(COMBA_ERR_INVALID_ARG, "dy must be non-NULL");
  if (!dr && !dn) return report(COMBA_ERR_INVALID_ARG, "dr or dn must be given");
  if (dn && !pre_weight) return report(COMBA_ERR_INVALID_ARG, "dn needs pre_weight");
  if ((gate == nullptr) != (dgate == nullptr) || (residual == nullptr) != (dresidual == nullptr) ||
      (scale == nullptr) != (dscale == nullptr) || (post_weight == nullptr) != (dpost_weight == nullptr) ||
      (pre_weight == nullptr) != (dpre_weight == nullptr))
    return report(COMBA_ERR_INVALID_ARG, "a gradient is given exactly when its input is");
  const size_t need = comba_block_norm_bwd_workspace_size(rows, D);
  rc = check_workspace(workspace, workspace_bytes, need,
                       "workspace is NULL or smaller than comba_block_norm_bwd_workspace_size()");
  if (rc != COMBA_OK) return rc;
  const int64_t act = rows * D * size_of(dtype), par = 4ll * D;
  rc = check_apart({{dy, act}, {dgate, act}, {dresidual, act}, {dscale, par}, {dpost_weight, par}, {dpre_weight, par},
                    {workspace, static_cast<int64_t>(need)}},
                   {{y, act}, {gate, act}, {residual, act}, {scale, par}, {post_weight, par}, {pre_weight, par},
                    {dr, act}, {dn, act}});
  if (rc != COMBA_OK) return rc;
  const comba::NormBwdArgs a{{y, gate, residual, scale, post_weight, pre_weight, rows, D, dtype, eps, nullptr, nullptr},
                             dr, dn, dy, dgate, dresidual, dscale, dpost_weight, dpre_weight,
                             static_cast<float*>(workspace)};
  return report_launch(comba::launch_norm_bwd(a, static_cast<hipStream_t>(stream)));
}
