// layer_norm.h -- launchers of layer norm (layer_norm_fwd.cu, layer_norm_bwd.cu).
#pragma once
#include "norm_residual.h"

namespace tg {

struct LayerNorm {
  const void *X, *w, *b;   // b: may be null
  const void *dY, *dR;     // backward; dR: may be null
  void* Y;                 // forward
  float *mean, *rstd;      // forward: outputs (may be null); backward: inputs
  void *dX, *dw, *db;      // backward; db: may be null
  int64_t T, d;            // both > 0, d <= NORM_MAX_D
  float eps;
  int in_kind, out_kind;
  float* ws;
  int num_sms;
  cudaStream_t stream;
  const char** rows;       // set to how the kernel takes its rows
};

cudaError_t layer_norm_fwd_launch(const LayerNorm& a);
size_t layer_norm_bwd_ws_bytes(int64_t T, int64_t d, int num_sms);
cudaError_t layer_norm_bwd_launch(const LayerNorm& a);

}  // namespace tg
