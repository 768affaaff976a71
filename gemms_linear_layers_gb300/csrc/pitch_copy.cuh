// pitch_copy.cuh -- 16-bit operands copied to rows that TMA can take.
#pragma once
#include "ptx.cuh"

namespace tg {

inline int64_t up8(int64_t n) { return (n + 7) / 8 * 8; }
inline size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Rows of `cols` 16-bit elements copied to rows of `pitch` (a multiple of 8)
// elements, the rest zero: what TMA needs of an operand whose rows are no
// multiple of 16 bytes or whose base is not 16-byte aligned.  Both operands of
// a call in one launch.
struct PitchCopy {
  const uint16_t* src;
  uint16_t* dst;
  long long rows;
  int cols, pitch;
};
// eight elements from column c of row r
__device__ __forceinline__ void pitch_word(const PitchCopy& p, long long r, int c) {
  const uint16_t* s = p.src + r * p.cols + c;
  uint32_t o[4];
  if (c + 8 <= p.cols && (reinterpret_cast<uintptr_t>(s) & 3) == 0) {
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = reinterpret_cast<const uint32_t*>(s)[j];
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = c + 2 * j < p.cols ? s[2 * j] : 0, hi = c + 2 * j + 1 < p.cols ? s[2 * j + 1] : 0;
      o[j] = lo | hi << 16;
    }
  }
  *reinterpret_cast<uint4*>(p.dst + r * p.pitch + c) = make_uint4(o[0], o[1], o[2], o[3]);
}
static __global__ void __launch_bounds__(256) pitch_copy_kernel(const PitchCopy a, const PitchCopy b) {
  pdl_wait();
  pdl_trigger();
  const long long first = a.rows * (a.pitch / 8), all = first + b.rows * (b.pitch / 8);
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < all;
       i += static_cast<long long>(gridDim.x) * blockDim.x) {
    const PitchCopy& p = i < first ? a : b;
    const long long k = i < first ? i : i - first;
    const int per = p.pitch / 8;
    const long long r = k / per;
    pitch_word(p, r, static_cast<int>(k - r * per) * 8);
  }
}

}  // namespace tg
