// gated_few.h -- launcher of the gated block for few rows (gated_few.cu).
#pragma once
#include "gated.h"

namespace tg {

// Most rows it takes: one limit for both directions and all widths, which fits none of them
// exactly.  Both sides (us, few rows and pairs): at the limit forward 2,304 -> 5,760 14.3 and
// 19.0, 576 -> 1,536 5.7 and 6.2, backward 14.1 and 18.2, but 576 -> 1,536 7.7 and 6.7.  Above it
// the few rows' kernel would still win with large weights (129 rows, 2,304 -> 5,760: forward
// 15.2 and 19.6, backward 14.3 and 17.4; 200 rows forward 18.1 and 19.7) and lose with others
// (200 rows, 576 -> 1,536: 7.7 and 6.6, backward 10.9 and 6.9; 256 rows, 1,024 -> 4,096: 14.7
// and 10.1).
constexpr int64_t GATED_FEW = 128;

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
