// gated.h -- launchers of the gated feed-forward block (gated_tc.cu).
#pragma once
#include "tg_internal.h"

namespace tg {

enum ActKind : int { ACT_SILU = 0, ACT_GELU = 1, ACT_GELU_TANH = 2, ACT_RELU = 3 };

struct GatedCall {
  bool bwd;
  const void* A;  // X, or dY: [T, d]
  const void* W;  // [2 f, d] (gate rows, then up rows), or the down projection [d, f]
  const void* GU; // backward: [T, 2 f]
  void* H;        // [T, f]; backward: may be null
  void* out;      // forward: GU (may be null); backward: dGU
  int64_t T, f, d;  // T, f > 0
  int act, in_kind;
  void* ws;
  size_t ws_bytes;
  int num_sms;
  unsigned int* status;
  unsigned long long timeout_ns;
  cudaStream_t stream;
  const char** path;  // set to the kernel's name
};

// Bytes of the workspace; any_base: for bases that are not 16-byte aligned.
size_t gated_ws_bytes(bool bwd, int64_t T, int64_t f, int64_t d, bool any_base, int num_sms);
// *need: 0, or the workspace the call lacked (nothing was launched then).
cudaError_t gated_launch(const GatedCall& g, size_t* need);

}  // namespace tg
