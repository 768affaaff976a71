// gated_few.h -- launcher of the gated block for few rows (gated_few.cu).
#pragma once
#include "gated.h"

namespace tg {

constexpr int64_t GATED_FEW = 128;  // most rows it takes

// A and W as TMA takes them: 16-byte aligned, rows `pitch` elements apart.
struct GatedFew {
  bool bwd;
  const void *A, *W, *GU;
  void *H, *out;
  int64_t T, f, d, pitch_x, pitch_w;  // all > 0
  int act, in_kind, num_sms;
  unsigned int* status;
  unsigned long long timeout_ns;
  cudaStream_t stream;
};
cudaError_t gated_few_launch(const GatedFew& g);

}  // namespace tg
