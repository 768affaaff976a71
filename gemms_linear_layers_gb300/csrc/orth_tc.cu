// orth_tc.cu -- the orthogonalised update of a weight from its gradient: with
// X = G / (|G| + eps) (Frobenius norm), `steps` times, m = min(rows, cols)
//   A = X X^T,  Q = a I + b A + c A A,  X = Q X          (rows <= cols)
//   A = X^T X,  Q = a I + b A + c A A,  X = X Q          (rows > cols)
// which takes every singular value s of X to a s + b s^3 + c s^5 and so all of
// them towards 1, and O = scale X.
//
// Everything between the launches is held as two bf16 parts, v = hi + lo to
// within 2^-17 |v|, and a product is the three products hi lo + lo hi + hi hi in
// one FP32 accumulator.  One 16-bit part would not do: rounding spreads over all
// directions alike, and a direction that the gradient barely has is multiplied
// by a^steps (485 for five steps of a = 3.44) on its way to 1, the rounding of the
// strong directions with it.  Relative to |X| = 1 the parts leave about
// 2^-18 |x|, or 5e-5 of a result's entries after that, below half a unit of fp16.
// A and Q are symmetric: only tiles that reach the diagonal or lie below it are
// computed and stored; an operand's block above it is loaded from below, where it is
// the same block MN-major, and the instruction is told so block by block.
// A tall G needs no transpose: its A is the product of MN-major operands, its
// X Q takes the symmetric Q as a K-major one.
#include <cmath>

#include "orth.h"

#include "pair_tc.cuh"
#include "pitch_copy.cuh"

namespace tg {
namespace {

// What a product makes of its sum.  EP_D, EP_E and EP_LAST are the last step's (see
// orth_launch), on one fp16 part each.
enum {
  EP_A = 0,     // A                                    two bf16 parts, symmetric
  EP_Q = 1,     // Q = a I + b A + c sum                two bf16 parts, symmetric
  EP_X = 2,     // X                                    two parts, bf16 or fp16
  EP_OUT = 3,   // scale X                              the result
  EP_D = 4,     // D = sum - I                          one fp16 part, symmetric
  EP_E = 5,     // E = (b + 2 c) D + c sum              one fp16 part, symmetric
  EP_LAST = 6   // scale ((a + b + c) X + sum)          the result; X two fp16 parts
};

// How an operand lies in memory.  OP_SYM: a symmetric matrix stored in part.  Row
// tile i (256 rows) of it holds its columns before 256 (i + 1), and the rest is taken
// from the other side of the diagonal, where a block lies MN-major.  When the last
// row tile has at most half its rows, these are stored, and computed, as the last
// columns of the tiles above (`strip` is the first of them), so that their products
// are narrow in N and not mostly empty in M.
enum { OP_K = 0, OP_MN = 1, OP_SYM = 2 };

struct OrthMaps {
  CUtensorMap A[2], B[2], C;  // operands: K-major boxes, MN-major boxes
};
struct OrthArgs {
  const uint16_t* in;  // EP_Q: A; EP_E: D; EP_LAST: X
  uint16_t* o;         // EP_OUT, EP_LAST
  long long in_pitch, in_part, in_matrix;  // elements from row to row, part to part, matrix to matrix
  int M, N;            // rows and columns of a result
  int batch, kbs, units, per, m_tiles, n_tiles, width;
  int strip;           // OP_SYM operands
  int main_units, out_strip;  // symmetric results: units before the strip's, first column of it
  float a, b, c;       // EP_Q: coefficients; EP_E: b, c; results: the factors of the sum (c) and of X (a)
  int wide, out_f16;
  uint32_t idesc;
  unsigned long long timeout_ns;
  unsigned int* status;
};
struct OrthUnit {
  int z, m0, n0, kb, nmma;
  int cols;  // that are stored (from n0 on, before clipping)
};

__device__ __forceinline__ void split2(float v, float* hi, float* lo) {
  *hi = __bfloat162float(__float2bfloat16_rn(v));
  *lo = v - *hi;
}
__device__ __forceinline__ void split2h(float v, float* hi, float* lo) {
  *hi = __half2float(__float2half_rn(v));
  *lo = v - *hi;
}

// Column tiles of a symmetric result's row tile i.
__host__ __device__ inline int sym_tiles(int i, int n_tiles, int width) {
  const int n = (i * 256 + 255) / width + 1;
  return n < n_tiles ? n : n_tiles;
}
__host__ __device__ inline int up64(int n) { return (n + 63) / 64 * 64; }

template <int A_OP, int B_OP, int EP, bool X16 = false>
struct OrthProduct {
  using Maps = OrthMaps;
  using Args = OrthArgs;
  using Unit = OrthUnit;
  using State = pt::NoState;
  static constexpr int A_KIND = A_OP, B_KIND = B_OP, EP_KIND = EP;
  static constexpr bool SYM = EP == EP_A || EP == EP_Q || EP == EP_D || EP == EP_E;
  static constexpr bool RESULT = EP == EP_OUT || EP == EP_LAST;
  static constexpr int PARTS = EP >= EP_D ? 1 : 2;
  static constexpr int OUT_PARTS = RESULT || PARTS == 1 ? 1 : 2;
  static constexpr int STAGES = PARTS == 2 ? 3 : 6, EPI_BLOCKS = 2;
  static constexpr unsigned SITE = 0x60;
  static __device__ __forceinline__ bool mn(const Args& a, int op, int row, int k0) {
    if (op != OP_SYM) return op == OP_MN;
    if (row >= a.strip) return k0 < a.strip;
    return k0 < a.strip && k0 >= ((row >> 8) + 1) << 8;
  }
  static __device__ __forceinline__ bool a_mn(const Args& a, const Unit& c, int kb) { return mn(a, A_OP, c.m0, kb * pt::BK); }
  static __device__ __forceinline__ bool b_mn(const Args& a, const Unit& c, int kb) { return mn(a, B_OP, c.n0, kb * pt::BK); }
  static __device__ __forceinline__ void prefetch(const Maps& m, const Args&) {
    prefetch_tmap(&m.A[A_OP == OP_MN]);
    prefetch_tmap(&m.B[B_OP == OP_MN]);
  }
  static __device__ __forceinline__ bool unit(const Args& a, int u, Unit& c) {
    c.kb = a.kbs;
    if (SYM && u >= a.main_units) {  // the strip: a tile of every row tile
      u -= a.main_units;
      c.z = u / a.m_tiles;
      c.m0 = (u - c.z * a.m_tiles) * 256;
      c.n0 = a.out_strip;
      c.cols = a.N - a.out_strip;
      c.nmma = up64(c.cols);
      return true;
    }
    c.z = u / a.per;
    int r = u - c.z * a.per;
    if (SYM) {
      int i = 0;
      for (int n; r >= (n = sym_tiles(i, a.n_tiles, a.width)); ++i) r -= n;
      c.m0 = i * 256;
      c.n0 = r * a.width;
      c.cols = min(a.width, c.m0 + 256 - c.n0);
    } else {
      const int j = r / a.m_tiles;
      c.m0 = (r - j * a.m_tiles) * 256;
      c.n0 = j * a.width;
      c.cols = a.width;
    }
    c.cols = min(c.cols, a.N - c.n0);
    c.nmma = up64(min(a.width, a.N - c.n0));
    return true;
  }
  // Boxes of a K-major B hold half a whole tile's rows.  One that may be either way comes
  // in whole 64 x 64 boxes, so that its bytes are the same.
  static __host__ __device__ __forceinline__ int b_rows(const Args& a) {
    return B_OP == OP_K ? a.width / 2 : up64(a.width / 2);
  }
  static __device__ __forceinline__ uint32_t bytes(const Args& a, const Unit&) {
    return PARTS * (pt::A_BYTES + b_rows(a) * pt::BK * 2);
  }
  static __device__ __forceinline__ void load(const Maps& m, const Args& a, const Unit& c, int kb, int rank,
                                              uint32_t a_dst, uint32_t b_dst, uint32_t bar) {
    const int k0 = kb * pt::BK;
    const int mrow = c.m0 + rank * 128, n = c.n0 + rank * (c.nmma / 2);
    const bool am = mn(a, A_OP, c.m0, k0), bm = mn(a, B_OP, c.n0, k0);
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
      const int z = c.z + p * a.batch;
      if (am) {
        tma_load_3d_pair(a_dst, &m.A[1], bar, mrow, k0, z);
        tma_load_3d_pair(a_dst + 8192, &m.A[1], bar, mrow + 64, k0, z);
      } else {
        tma_load_3d_pair(a_dst, &m.A[0], bar, k0, mrow, z);
      }
      if (bm) {
        for (int j = 0; j < b_rows(a); j += 64) tma_load_3d_pair(b_dst + j * 128, &m.B[1], bar, n + j, k0, z);
      } else {
        tma_load_3d_pair(b_dst, &m.B[0], bar, k0, n, z);
      }
      a_dst += pt::A_BYTES;
      b_dst += pt::B_BYTES;
    }
  }
  template <class Wait, class Release>
  static __device__ __forceinline__ void epilogue(const Maps& m, const Args& a, const Unit& c, const Unit*,
                                                  const pt::EpiWarp& at, pt::NoState&, Wait wait, Release release) {
    constexpr bool IN = EP == EP_Q || EP == EP_E || EP == EP_LAST, IN2 = IN && EP != EP_E;  // reads a matrix, of two parts
    constexpr bool IN16 = EP == EP_E || EP == EP_LAST;                                      // in fp16
    const int lane = threadIdx.x & 31;
    const int row0 = c.m0 + at.rank * 128 + at.q * 32;
    const int rows = min(32, a.M - row0);
    const int cols = rows > 0 ? c.cols : 0;
    uint8_t *b0 = at.blocks, *b1 = b0 + pt::BLOCK;
    pt::HalfRegs in0, in1;
    auto fetch = [&](int col) {
      const int n = c.n0 + col + 32 * at.h;
      const int left = (a.N - n + 7) & ~7;  // rows are whole words; what lies past the columns is not stored
      const uint16_t* p = a.in + c.z * a.in_matrix + row0 * a.in_pitch + n;
      pt::half_fetch(in0, p, a.in_pitch, rows, left, lane, true);
      if (IN2) pt::half_fetch(in1, p + a.in_part, a.in_pitch, rows, left, lane, true);
    };
    if (IN && cols > 0) fetch(0);
    if (!wait()) return;
    if (cols <= 0) release();
#pragma unroll 1
    for (int col = 0; col < cols; col += 64) {
      const int mine = col + 32 * at.h, n = c.n0 + mine;
      float v[32];
      tmem_ld_32x32b_x32(at.taddr + mine, reinterpret_cast<uint32_t*>(v));
      tmem_ld_wait();
      if (col + 64 >= cols) release();
      pt::blocks_free(at, lane);
      const int diagonal = row0 + lane - n;
      if constexpr (IN) {
        pt::half_put(in0, b0, at.h, lane);
        if (IN2) pt::half_put(in1, b1, at.h, lane);
        __syncwarp();
        if (col + 64 < cols) fetch(col + 64);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 h = *reinterpret_cast<uint4*>(pt::block_word(b0, lane, 4 * at.h + j));
          uint4 l = make_uint4(0, 0, 0, 0);
          if (IN2) l = *reinterpret_cast<uint4*>(pt::block_word(b1, lane, 4 * at.h + j));
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float2 x = pt::unpack16<IN16>(reinterpret_cast<const uint32_t*>(&h)[k]);
            if (IN2) {
              const float2 y = pt::unpack16<IN16>(reinterpret_cast<const uint32_t*>(&l)[k]);
              x.x += y.x;
              x.y += y.y;
            }
            const int e = 8 * j + 2 * k;
            if constexpr (EP == EP_Q) {
              v[e] = fmaf(a.c, v[e], fmaf(a.b, x.x, e == diagonal ? a.a : 0.f));
              v[e + 1] = fmaf(a.c, v[e + 1], fmaf(a.b, x.y, e + 1 == diagonal ? a.a : 0.f));
            } else {
              const float by = EP == EP_E ? a.b : a.a;
              v[e] = fmaf(a.c, v[e], by * x.x);
              v[e + 1] = fmaf(a.c, v[e + 1], by * x.y);
            }
          }
        }
      } else if constexpr (EP == EP_D) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] -= j == diagonal ? 1.f : 0.f;
      } else if constexpr (EP == EP_OUT) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] *= a.c;
      }
      if constexpr (RESULT) {
        if (a.out_f16) pt::put_row<true>(b0, lane, at.h, v);
        else pt::put_row<false>(b0, lane, at.h, v);
        if (!a.wide) {
          pt::half_store(b0, at.h, a.o + (static_cast<long long>(c.z) * a.M + row0) * a.N + n, a.N, rows, min(32, a.N - n), lane);
          continue;
        }
      } else if constexpr (OUT_PARTS == 1) {
        pt::put_row<true>(b0, lane, at.h, v);
      } else {
        float lo[32];
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if constexpr (X16) split2h(v[j], &v[j], &lo[j]);
          else split2(v[j], &v[j], &lo[j]);
        pt::put_row<X16>(b0, lane, at.h, v);
        pt::put_row<X16>(b1, lane, at.h, lo);
      }
      if (pt::blocks_full(at, lane)) {
        tma_store_3d(&m.C, smem_u32(b0), c.n0 + col, row0, c.z);
        if (OUT_PARTS == 2) tma_store_3d(&m.C, smem_u32(b1), c.n0 + col, row0, c.z + a.batch);
        bulk_commit();
      }
    }
  }
};

// ---------------------------------------------------------- the norm, X = G / (|G| + eps)
template <typename T>
__device__ __forceinline__ float to_float(T v) {
  if constexpr (sizeof(T) == 4) return v;
  else if constexpr (std::is_same<T, __half>::value) return __half2float(v);
  else return __bfloat162float(v);
}

constexpr int NORM_THREADS = 256;
constexpr int NORM_PARTS = 256;  // most partial sums of a matrix

// Eight elements from i on (zeros beyond n).
template <typename T>
__device__ __forceinline__ void eight(const T* p, long long i, long long n, bool wide, float* v) {
  if (wide) {  // n and i are multiples of 8, rows of 16 bytes
    alignas(16) T e[8];
    const uint4* s = reinterpret_cast<const uint4*>(p + i);
#pragma unroll
    for (int k = 0; k < static_cast<int>(sizeof(T)) / 2; ++k) reinterpret_cast<uint4*>(e)[k] = s[k];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = to_float<T>(e[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = i + j < n ? to_float<T>(p[i + j]) : 0.f;
  }
}

// part[z][k]: the sum of squares of range k of matrix z.  Squares are added in
// FP32 in groups of 32 and FP64 beyond; groups whose sum leaves FP32's range, or comes
// near its end, are added again in FP64.
template <typename T>
__global__ void __launch_bounds__(NORM_THREADS) orth_norm_kernel(const T* __restrict__ G, double* part, long long n, int parts,
                                                                 int wide) {
  __shared__ double s[NORM_THREADS / 32];
  pdl_wait();  // no early trigger: large batches make more CTAs than fit at once
  const long long z = blockIdx.x / parts;
  const int k = static_cast<int>(blockIdx.x - z * parts);
  const T* p = G + z * n;
  const long long step = static_cast<long long>(parts) * NORM_THREADS * 8;
  double sum = 0.;
  for (long long i = (static_cast<long long>(k) * NORM_THREADS + threadIdx.x) * 8; i < n; i += 4 * step) {
    float v[4][8], q = 0.f;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      if (i + g * step < n) {
        eight<T>(p, i + g * step, n, wide, v[g]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[g][j] = 0.f;
      }
    }
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
      for (int j = 0; j < 8; ++j) q = fmaf(v[g][j], v[g][j], q);
    if (q > 1e-30f && q < 1e38f) {
      sum += q;
    } else {
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += static_cast<double>(v[g][j]) * v[g][j];
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < NORM_THREADS / 32; ++i) sum += s[i];
    part[blockIdx.x] = sum;
  }
}

// X, two parts of [batch][rows][pitch], from G [batch][rows][cols].  `blocks` CTAs a matrix.
template <typename T>
__global__ void __launch_bounds__(256) orth_split_kernel(const T* G, const double* part, uint16_t* X, long long rows, int cols,
                                                         int pitch, int parts, int blocks, long long part_stride, float eps,
                                                         int wide) {
  __shared__ float factor[2];
  pdl_wait();
  const long long z = blockIdx.x / blocks;
  const int k = static_cast<int>(blockIdx.x - z * blocks);
  if (threadIdx.x < 32) {
    double sum = 0.;
    for (int i = threadIdx.x; i < parts; i += 32) sum += part[z * parts + i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    const double inv = 1. / (sqrt(sum) + static_cast<double>(eps));
    // in two factors, the first a power of two that keeps the second within FP32's range
    const double first = inv < 1e-36 ? 0x1p-64 : inv > 1e36 ? 0x1p64 : 1.;
    factor[0] = static_cast<float>(first);
    factor[1] = static_cast<float>(inv / first);
  }
  __syncthreads();
  const float f0 = factor[0], f1 = factor[1];
  const int per = pitch / 8;
  const long long words = rows * per;
  for (long long i = static_cast<long long>(k) * 256 + threadIdx.x; i < words; i += static_cast<long long>(blocks) * 256) {
    const long long r = i / per;
    const int c = static_cast<int>(i - r * per) * 8;
    float v[8];
    eight<T>(G + (z * rows + r) * cols, c, cols, wide, v);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float h[2], l[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) split2(v[2 * j + e] * f0 * f1, &h[e], &l[e]);
      hi[j] = pack_bf16x2(h[0], h[1]);
      lo[j] = pack_bf16x2(l[0], l[1]);
    }
    uint16_t* at = X + (z * rows + r) * pitch + c;
    *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(at + part_stride) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}

// ------------------------------------------------------------------ host side
constexpr int UNIT_COST = 64;  // of a tile beside its columns

struct Places {
  int64_t m, long_side, pitch_x, pitch_s;
  int64_t x_part, s_part;  // elements of one part of X, of A or Q
  int parts;
  size_t x[2], s, q, sums, bytes;  // offsets
};
Places places(int64_t batch, int64_t rows, int64_t cols) {
  Places l;
  l.m = rows < cols ? rows : cols;
  l.long_side = rows < cols ? cols : rows;
  l.pitch_x = up8(cols);
  l.pitch_s = up8(l.m);
  l.x_part = batch * rows * l.pitch_x;
  l.s_part = batch * l.m * l.pitch_s;
  const int64_t want = (rows * cols + 32 * NORM_THREADS - 1) / (32 * NORM_THREADS);
  l.parts = static_cast<int>(want < NORM_PARTS ? want : NORM_PARTS);
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t here = at;
    at += up256(n);
    return here;
  };
  l.x[0] = take(4 * l.x_part);
  l.x[1] = take(4 * l.x_part);
  l.s = take(4 * l.s_part);
  l.q = take(4 * l.s_part);
  l.sums = take(8 * static_cast<size_t>(batch) * l.parts);
  l.bytes = at;
  return l;
}

// One operand or result: two parts of [batch][rows][pitch].
struct Matrix {
  void* p;
  int64_t rows, cols, pitch;
};

// First column of a symmetric matrix's strip (m when it has none).
int strip_of(int64_t m) {
  const int rest = static_cast<int>(m % 256);
  return static_cast<int>(m > 256 && rest > 0 && rest <= 128 ? m - rest : m);
}

template <class P>
cudaError_t product(const OrthCall& g, const Matrix& A, const Matrix& B, const Matrix& C, OrthArgs a) {
  OrthMaps m = {};
  a.M = static_cast<int>(C.rows);
  a.N = static_cast<int>(C.cols);
  a.batch = static_cast<int>(g.batch);
  a.m_tiles = (a.M + 255) / 256;
  const int64_t K = P::A_KIND == OP_MN ? A.rows : A.cols;
  a.kbs = static_cast<int>((K + pt::BK - 1) / pt::BK);
  constexpr bool strips = P::SYM || P::A_KIND == OP_SYM || P::B_KIND == OP_SYM;
  a.strip = strip_of(P::SYM ? a.N : P::A_KIND == OP_SYM ? A.rows : B.rows);
  a.out_strip = a.strip;
  const bool split = strips && a.strip % 256 == 0 && a.strip < (P::SYM ? a.N : P::A_KIND == OP_SYM ? A.rows : B.rows);
  const int main_cols = P::SYM ? a.strip : a.N, main_rows = P::SYM && split ? a.strip / 256 : a.m_tiles;
  auto fit = [&](int w) {
    a.width = w;
    a.n_tiles = (main_cols + w - 1) / w;
    a.per = 0;
    if (P::SYM)
      for (int i = 0; i < main_rows; ++i) a.per += sym_tiles(i, a.n_tiles, w);
    else
      a.per = a.m_tiles * a.n_tiles;
    a.main_units = a.per * a.batch;
    a.units = a.main_units + (P::SYM && split ? a.m_tiles * a.batch : 0);
  };
  // The width with which the busiest pair has least to do: a unit costs its columns and
  // UNIT_COST more.  Where a symmetric operand or result has a strip, tiles must not
  // straddle its first column.
  const int pairs = g.num_sms / 2, rest = up64(a.N - a.strip);
  int best = 0;
  int64_t least = 0;
  for (int w = 64; w <= 256; w += 64) {
    if (split && (256 % w != 0 || (P::SYM && w < rest))) continue;
    fit(w);
    int64_t most = 0;
    for (int p = 0; p < pairs && p < a.units; ++p) {
      const int64_t mine = (a.units - p + pairs - 1) / pairs;
      const int64_t main = p < a.main_units ? (a.main_units - p + pairs - 1) / pairs : 0;
      const int64_t cost = main * (w + UNIT_COST) + (mine - main) * (rest + UNIT_COST);
      if (cost > most) most = cost;
    }
    if (best == 0 || most <= least) best = w, least = most;
  }
  fit(best);
  constexpr int in_kind = P::PARTS == 2 ? EK_BF16 : EK_F16;
  a.idesc = idesc_f16(in_kind == EK_BF16, false, false, 256, 0);
  a.timeout_ns = g.timeout_ns;
  a.status = g.status;
  const uint64_t planes = 2 * static_cast<uint64_t>(g.batch);
  auto map = [&](CUtensorMap* t, const Matrix& x, int op, int box_rows) {
    const uint64_t pitch = static_cast<uint64_t>(x.pitch) * 2;
    for (int mn = 0; mn < 2; ++mn)
      if ((op == OP_SYM || op == mn) &&
          !encode_tmap_3d(t + mn, x.p, in_kind, x.cols, x.rows, planes, pitch, x.rows * pitch, 64, mn ? 64 : box_rows, 128))
        return false;
    return true;
  };
  bool ok = map(m.A, A, P::A_KIND, 128) && map(m.B, B, P::B_KIND, P::b_rows(a));
  const uint64_t pc = static_cast<uint64_t>(C.pitch) * 2;
  if (P::RESULT) {
    a.wide = C.cols % 8 == 0 && reinterpret_cast<uintptr_t>(C.p) % 16 == 0;
    a.out_f16 = g.out_kind == EK_F16;
    a.o = static_cast<uint16_t*>(C.p);
    if (a.wide) ok = ok && encode_tmap_3d(&m.C, C.p, g.out_kind, C.cols, C.rows, g.batch, pc, C.rows * pc, 64, 32, 128);
  } else {
    ok = ok && encode_tmap_3d(&m.C, C.p, EK_BF16, C.cols, C.rows, planes, pc, C.rows * pc, 64, 32, 128);
  }
  if (!ok) return cudaErrorInvalidValue;
  return pt::pair_launch<P>(m, a, g.num_sms, g.stream);
}

template <typename T>
cudaError_t prepare(const OrthCall& g, const Places& l, double* sums, uint16_t* X) {
  const int64_t n = g.rows * g.cols;
  const T* G = static_cast<const T*>(g.G);
  const bool base = reinterpret_cast<uintptr_t>(G) % 16 == 0;
  cudaError_t e = launch_k(orth_norm_kernel<T>, dim3(static_cast<unsigned>(g.batch * l.parts)), dim3(NORM_THREADS), 0, g.stream, G,
                           sums, static_cast<long long>(n), l.parts, static_cast<int>(base && n % 8 == 0));
  if (e != cudaSuccess) return e;
  int64_t blocks = (g.rows * (l.pitch_x / 8) + 255) / 256;
  const int64_t most = (8 * g.num_sms + g.batch - 1) / g.batch;
  if (blocks > most) blocks = most;
  return launch_k(orth_split_kernel<T>, dim3(static_cast<unsigned>(g.batch * blocks)), dim3(256), 0, g.stream, G,
                  static_cast<const double*>(sums), X, static_cast<long long>(g.rows), static_cast<int>(g.cols),
                  static_cast<int>(l.pitch_x), l.parts, static_cast<int>(blocks), static_cast<long long>(l.x_part), g.eps,
                  static_cast<int>(base && g.cols % 8 == 0));
}

// Whether the last step may take one fp16 part (see orth_launch): its coefficients, and
// X's entries inside fp16's range by then: the steps before enlarge small singular values
// (entries start at 1 / sqrt(rows cols) in the mean square) and take none above 8.
bool light_last(const OrthCall& g) {
  const double* last = g.coeffs + 3 * (g.steps - 1);
  if (g.steps < 2 || fabs(last[1] + 2 * last[2]) + fabs(last[2]) > 3. || g.rows * g.cols > int64_t(1) << 30) return false;
  double slope = 1., top = 1.;
  for (int64_t i = 0; i + 1 < g.steps; ++i) {
    const double *k = g.coeffs + 3 * i, from = top;
    slope *= fabs(k[0]);
    top = 0.;
    for (int j = 1; j <= 64; ++j) {
      const double s = from * j / 64, v = fabs(s * (k[0] + s * s * (k[1] + s * s * k[2])));
      if (v > top) top = v;
    }
  }
  return slope >= 2. && top <= 8.;
}

}  // namespace

size_t orth_ws_bytes(int64_t batch, int64_t rows, int64_t cols) {
  return batch > 0 && rows > 0 && cols > 0 ? places(batch, rows, cols).bytes : 0;
}

cudaError_t orth_launch(const OrthCall& g) {
  const Places l = places(g.batch, g.rows, g.cols);
  char* ws = static_cast<char*>(g.ws);
  Matrix X[2] = {{ws + l.x[0], g.rows, g.cols, l.pitch_x}, {ws + l.x[1], g.rows, g.cols, l.pitch_x}};
  const Matrix S = {ws + l.s, l.m, l.m, l.pitch_s}, Q = {ws + l.q, l.m, l.m, l.pitch_s};
  const Matrix O = {g.O, g.rows, g.cols, g.cols};
  double* sums = reinterpret_cast<double*>(ws + l.sums);
  uint16_t* x0 = static_cast<uint16_t*>(X[0].p);
  cudaError_t e = g.in_kind == EK_BF16  ? prepare<__nv_bfloat16>(g, l, sums, x0)
                  : g.in_kind == EK_F16 ? prepare<__half>(g, l, sums, x0)
                                        : prepare<float>(g, l, sums, x0);
  const bool tall = g.rows > g.cols;
  // The last step of a bf16 result: written around 1, where the singular values are by
  // then, with D = A - I (X'X = I + D),
  //   (a + b + c) X + E X,  E = (b + 2 c) D + c D D,
  // D, E and the X of the products may be one fp16 part each: their rounding (2^-11 at most)
  // enters times |b + 2 c| + |c|, 2.7 with the usual coefficients (as a I + b A + c A A it
  // would be 7 and more), and the first term takes X in two parts.  Emulated in 64 bits it
  // leaves 2e-4 to 4e-4 of a result's size beside the 1.7e-3 of rounding to bf16 (1e-3
  // where X has directions of 1e-5), for a third of the products.
  const bool light = g.out_kind == EK_BF16 && light_last(g);
  for (int64_t i = 0; i < g.steps && e == cudaSuccess; ++i) {
    const Matrix &x = X[i & 1], &y = X[(i + 1) & 1];
    const double *k = g.coeffs + 3 * i, s = g.scale;
    const bool end = i + 1 == g.steps;
    OrthArgs sum = {}, poly = {}, out = {};
    poly.in = static_cast<const uint16_t*>(S.p);
    poly.in_pitch = l.pitch_s;
    poly.in_part = l.s_part;
    poly.in_matrix = l.m * l.pitch_s;
    poly.c = static_cast<float>(k[2]);
    if (end && light) {
      poly.b = static_cast<float>(k[1] + 2 * k[2]);
      out.in = static_cast<const uint16_t*>(x.p);
      out.in_pitch = l.pitch_x;
      out.in_part = l.x_part;
      out.in_matrix = g.rows * l.pitch_x;
      out.a = static_cast<float>(s * (k[0] + k[1] + k[2]));
      out.c = g.scale;
      e = tall ? product<OrthProduct<OP_MN, OP_MN, EP_D>>(g, x, x, S, sum) : product<OrthProduct<OP_K, OP_K, EP_D>>(g, x, x, S, sum);
      if (e == cudaSuccess) e = product<OrthProduct<OP_SYM, OP_SYM, EP_E>>(g, S, S, Q, poly);
      if (e == cudaSuccess)
        e = tall ? product<OrthProduct<OP_K, OP_SYM, EP_LAST>>(g, x, Q, O, out)
                 : product<OrthProduct<OP_SYM, OP_MN, EP_LAST>>(g, Q, x, O, out);
      break;
    }
    poly.a = static_cast<float>(k[0]);
    poly.b = static_cast<float>(k[1]);
    out.c = g.scale;
    e = tall ? product<OrthProduct<OP_MN, OP_MN, EP_A>>(g, x, x, S, sum) : product<OrthProduct<OP_K, OP_K, EP_A>>(g, x, x, S, sum);
    if (e == cudaSuccess) e = product<OrthProduct<OP_SYM, OP_SYM, EP_Q>>(g, S, S, Q, poly);
    if (e != cudaSuccess) break;
    if (end)
      e = tall ? product<OrthProduct<OP_K, OP_SYM, EP_OUT>>(g, x, Q, O, out) : product<OrthProduct<OP_SYM, OP_MN, EP_OUT>>(g, Q, x, O, out);
    else if (light && i + 2 == g.steps)  // X in fp16 parts for the last step
      e = tall ? product<OrthProduct<OP_K, OP_SYM, EP_X, true>>(g, x, Q, y, out)
               : product<OrthProduct<OP_SYM, OP_MN, EP_X, true>>(g, Q, x, y, out);
    else
      e = tall ? product<OrthProduct<OP_K, OP_SYM, EP_X>>(g, x, Q, y, out) : product<OrthProduct<OP_SYM, OP_MN, EP_X>>(g, Q, x, y, out);
  }
  return e;
}

}  // namespace tg
