// grad_clip.h -- launchers of the global gradient norm and clipping (grad_clip.cu).
#pragma once
#include "tg_internal.h"

namespace tg {

struct GradList {
  const void* const* grads;
  void* const* outs;  // null: no clipping, only the norm
  const int64_t* numels;
  const int* kinds;  // EK_*
  int64_t n;
  float max_norm;
  float* norm;  // device
  void* ws;
  int num_sms;
  cudaStream_t stream;
};

size_t grad_norm_ws_bytes(int64_t n, int num_sms);
cudaError_t grad_clip_launch(const GradList& g);

}  // namespace tg
