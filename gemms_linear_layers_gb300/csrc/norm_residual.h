// norm_residual.h -- launchers of the norms around a block (norm_fwd.cu, norm_bwd.cu).
#pragma once
#include "tg_internal.h"

namespace tg {

constexpr int64_t NORM_MAX_D = 16384;

enum GateKind : int { GATE_NONE = 0, GATE_CHANNEL = 1, GATE_TOKEN = 2, GATE_FULL = 3 };

struct NormResidual {
  const void *B, *H, *w_post, *w_pre, *gate;  // H: the stream before (forward) or after (backward) the block
  const void *dH_out, *dN;                    // backward
  float *rstd_b, *rstd_h;                     // forward: outputs (may be null); backward: inputs
  void *H_out, *N;                            // forward
  void *dB, *dH, *dw_post, *dw_pre, *dgate;   // backward
  int64_t T, d;                               // both > 0
  float res_scale, eps;
  int gate_kind;
  int in_kind, res_kind, out_kind;
  float* ws;
  int num_sms;
  cudaStream_t stream;
  const char** rows;  // set to how the kernel takes its rows
};

cudaError_t norm_residual_fwd_launch(const NormResidual& a);
size_t norm_residual_bwd_ws_bytes(int64_t T, int64_t d, int num_sms);
cudaError_t norm_residual_bwd_launch(const NormResidual& a);

}  // namespace tg
