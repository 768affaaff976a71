// orth.h -- launcher of the orthogonalised update (orth_tc.cu).
#pragma once
#include "tg_internal.h"

namespace tg {

// How a call was carried out.
struct OrthForm {
  int width;  // columns of a tile
  bool f16;   // parts in fp16
};
struct OrthCall {
  const void* G;
  void* O;
  int64_t batch, rows, cols;  // all > 0
  const double* coeffs;       // host, [steps][3]
  int64_t steps;
  float scale, eps;
  int in_kind, out_kind;
  void* ws;
  int num_sms;
  unsigned int* status;
  unsigned long long timeout_ns;
  cudaStream_t stream;
  OrthForm* form;  // set
};

// Whether the tiles of a call can be counted (2^30 in all, 2^27 of a matrix).
bool orth_fits(int64_t batch, int64_t rows, int64_t cols, int64_t steps);
size_t orth_ws_bytes(int64_t batch, int64_t rows, int64_t cols);
cudaError_t orth_launch(const OrthCall& g);

}  // namespace tg
