// Launchers of the layer operators around the recurrence (short convolution,
// selective scan, block norms). Arguments are already validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace comba {

// Records `what` as the calling thread's last error and returns `code` (abi.hip).
int32_t report(int32_t code, const char* what);
// Status of a launch sequence: COMBA_OK, or COMBA_ERR_HIP with the runtime's text (abi.hip).
int32_t report_launch(hipError_t e);

struct ConvArgs {
  const void* x;              // [B, T, D] (step: [N, D])
  const float* weight;        // [D, W]
  const float* bias;          // [D] or null
  const void* init;           // [N, W-1, D] or null
  const int32_t* cu_seqlens;  // [N + 1] or null
  int N, B, T, D, W, dtype;
  bool silu;
  void* y;
  void* fin;                  // [N, W-1, D] or null
};

struct ConvBwdArgs {
  ConvArgs f;                 // the forward's inputs; y and fin unused
  const void* dy;             // [B, T, D], dy_dtype
  int dy_dtype;
  const void* dfin;           // [N, W-1, D] x's type, or null
  void* dx;                   // [B, T, D] x's type
  float* dweight;             // [D, W]
  float* dbias;               // [D] or null
  void* dinit;                // [N, W-1, D] x's type, or null
  float* part;                // workspace: [sets of four tiles, W + 1, D]
};

hipError_t launch_conv(const ConvArgs& a, hipStream_t st);
hipError_t launch_conv_step(const ConvArgs& a, hipStream_t st);
hipError_t launch_conv_bwd(const ConvBwdArgs& a, hipStream_t st);
// Token tiles of the forward, and sets of four tiles of the backward.
int64_t conv_tiles(int64_t B, int64_t T, int64_t D, bool packed);
int64_t conv_bwd_sets(int64_t B, int64_t T, int64_t D, bool packed);

struct NormArgs {
  const void* y;              // [rows, D]
  const void* gate;           // [rows, D] or null
  const void* residual;       // [rows, D] or null
  const float* scale;         // [D] or null
  const float* post_weight;   // [D] or null
  const float* pre_weight;    // [D] or null
  int64_t rows;
  int D, dtype;
  float eps;
  void* r;                    // [rows, D]
  void* n;                    // [rows, D] or null (no pre_weight)
};

struct NormBwdArgs {
  NormArgs f;
  const void* dr;             // [rows, D] or null
  const void* dn;             // [rows, D] or null
  void* dy;
  void* dgate;                // or null
  void* dresidual;            // or null
  float* dscale;              // or null
  float* dpost;               // or null
  float* dpre;                // or null
  float* part;                // workspace: [blocks, 3, D]
};

constexpr int kNormMaxWidth = 16384;
// Workgroups of the backward: rows of the partial sums [blocks, 3, D] in its workspace.
int64_t norm_bwd_blocks(int64_t rows, int D);

hipError_t launch_norm(const NormArgs& a, hipStream_t st);
hipError_t launch_norm_bwd(const NormBwdArgs& a, hipStream_t st);

struct ScanArgs {
  const void* x;              // [B, T, D] (step: [N, D])
  const void* dt;
  const float* A;             // [D, S]
  const void* Bm;             // [B, T, G, S]
  const void* Cm;
  const float* skip;          // [D] or null
  const void* z;              // as x, or null
  const float* dt_bias;       // [D] or null
  bool softplus;
  const float* init;          // [N, D, S] or null
  const int32_t* cu_seqlens;  // [N + 1] or null
  int N, B, T, D, S, G, dtype;
  void* y;
  float* fin;                 // [N, D, S] or null
};

// Segments of a scan: sequence n's segment c (L tokens each) has slot
//   n * ceil(T / L) + c               (fixed-length batches)
//   cu_seqlens[n] / L + n + c         (packed batches; unique because starts increase)
struct ScanPlan {
  int L;                      // tokens per segment; 0: sequences are not cut
  int64_t slots;
};
ScanPlan scan_plan(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N, bool packed);
ScanPlan scan_bwd_plan(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N, int S, bool packed);
int scan_padded_states(int S);           // states per channel in the workspaces
int64_t scan_channel_blocks(int64_t D, int64_t G);      // workgroups per slot
int64_t scan_bwd_channel_blocks(int64_t D, int64_t G);
int64_t scan_step_blocks(int64_t N, int64_t D, int64_t G);  // workgroups of the step

struct ScanBwdArgs {
  ScanArgs f;                 // the forward's inputs; y and fin unused
  const void* dy;             // [B, T, D]
  const float* dfin;          // [N, D, S] or null
  void* dx;                   // [B, T, D]
  void* ddt;
  float* dA;                  // [D, S]
  void* dBm;                  // [B, T, G, S]
  void* dCm;
  float* dskip;               // [D] or null
  void* dz;                   // or null
  float* ddt_bias;            // [D] or null
  float* dinit;               // [N, D, S] or null
  // workspace
  float* hseg;                // [slots, D, SP]: every segment's end state from 0, then its incoming state
  float* gseg;                // [slots, D, SP]: its gradient sum, then the gradient at its end
  float* dsum;                // [slots, D]: sum of the step sizes
  float* dApart;              // [slots, D, SP]
  float* dDpart;              // [slots, 2, D]
  float* dBCpart;             // [channel blocks of a group, B * T, G, 2, SP]
};

constexpr int kScanMaxStates = 64;

// hseg [slots, D, SP] and dsum [slots, D]: workspace of a cut forward, null when not cut.
hipError_t launch_scan(const ScanArgs& a, const ScanPlan& p, float* hseg, float* dsum, hipStream_t st);
hipError_t launch_scan_step(const ScanArgs& a, hipStream_t st);
hipError_t launch_scan_bwd(const ScanBwdArgs& a, const ScanPlan& p, hipStream_t st);

}  // namespace comba
