// grouped.h -- launcher of the products grouped by expert (grouped_tc.cu).
#pragma once
#include "tg_internal.h"

namespace tg {

constexpr int GROUPED_PER_LAUNCH = 256;  // experts of one launch (their offsets sit in shared memory)

struct GroupedCall {
  int op;  // 0 forward, 1 input gradient, 2 weight gradient
  const void* A;       // W [E, d_out, d_in]; weight gradient: dY [T, d_out]
  const void* B;       // X or dY [T, .]; weight gradient: X [T, d_in]
  const int* offsets;  // device, [E + 1]
  void* C;
  int64_t T, E, d_out, d_in;  // all > 0
  int in_kind, out_kind;
  void* ws;
  size_t ws_bytes;
  void* parts;  // set by the launcher
  int num_sms;
  unsigned int* status;
  unsigned long long timeout_ns;
  cudaStream_t stream;
};

// Bytes of the workspace; any_base: for bases that are not 16-byte aligned.
size_t grouped_ws_bytes(int op, int64_t T, int64_t E, int64_t d_out, int64_t d_in, bool any_base, int num_sms);
// *need: 0, or the workspace the call lacked (nothing was launched then).
cudaError_t grouped_launch(const GroupedCall& g, size_t* need);

}  // namespace tg
