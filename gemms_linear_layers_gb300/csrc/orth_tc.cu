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
// A and Q are symmetric: only tiles on and below the diagonal are computed, and
// each 32 x 32 block below it is stored twice, once turned.
// A tall G needs no transpose: its A is the product of MN-major operands, its
// X Q takes the symmetric Q as a K-major one.
#include "orth.h"

#include "pair_tc.cuh"
#include "pitch_copy.cuh"

namespace tg {
namespace {

enum { EP_SYM = 0, EP_POLY = 1, EP_X = 2, EP_OUT = 3 };

struct OrthMaps {
  CUtensorMap A, B, C;
};
struct OrthArgs {
  const uint16_t* s;  // EP_POLY: A of the iteration, two parts
  uint16_t* o;        // EP_OUT
  long long s_pitch, s_part, s_matrix;  // elements from row to row, part to part, matrix to matrix
  int M, N;           // rows and columns of a result
  int batch, kbs, units, per, m_tiles, n_tiles, width;
  float a, b, c;      // EP_POLY; EP_OUT: a is the scale
  int wide, out_f16;
  uint32_t idesc;
  unsigned long long timeout_ns;
  unsigned int* status;
};
struct OrthUnit {
  int z, m0, n0, kb, nmma;
};

__device__ __forceinline__ void split2(float v, float* hi, float* lo) {
  *hi = __bfloat162float(__float2bfloat16_rn(v));
  *lo = v - *hi;
}

// Column tiles of a symmetric result's row tile i that reach the diagonal or lie below it.
__host__ __device__ inline int sym_tiles(int i, int n_tiles, int width) {
  const int n = (i * 256 + 255) / width + 1;
  return n < n_tiles ? n : n_tiles;
}

template <bool AMN, bool BMN, int EP>
struct OrthProduct {
  using Maps = OrthMaps;
  using Args = OrthArgs;
  using Unit = OrthUnit;
  static constexpr int EP_KIND = EP;
  static constexpr bool SYM = EP == EP_SYM || EP == EP_POLY;
  static constexpr int STAGES = 5, EPI_WARP = (SYM ? 4 : 2) * pt::BLOCK;
  static constexpr bool A_MN = AMN, B_MN = BMN;
  static constexpr unsigned SITE = 0x60;
  static __device__ __forceinline__ void prefetch(const Maps& m, const Args&) {
    prefetch_tmap(&m.A);
    prefetch_tmap(&m.B);
  }
  static __device__ __forceinline__ bool unit(const Args& a, int u, Unit& c) {
    c.z = u / a.per;
    int r = u - c.z * a.per;
    c.kb = 3 * a.kbs;
    c.nmma = a.width;
    if (SYM) {
      int i = 0;
      for (int n; r >= (n = sym_tiles(i, a.n_tiles, a.width)); ++i) r -= n;
      c.m0 = i * 256;
      c.n0 = r * a.width;
    } else {
      const int j = r / a.m_tiles;
      c.m0 = (r - j * a.m_tiles) * 256;
      c.n0 = j * a.width;
    }
    return true;
  }
  static __device__ __forceinline__ int chunks64(const Args& a) { return (a.width / 2 + 63) / 64; }
  static __device__ __forceinline__ uint32_t bytes(const Args& a, const Unit&) {
    return pt::A_BYTES + (BMN ? chunks64(a) * 64 : a.width / 2) * pt::BK * 2;
  }
  static __device__ __forceinline__ void load(const Maps& m, const Args& a, const Unit& c, int kb, int rank,
                                              uint32_t a_dst, uint32_t b_dst, uint32_t bar) {
    // parts hi lo, lo hi, hi hi
    const int s = kb >= 2 * a.kbs ? 2 : kb >= a.kbs ? 1 : 0;
    const int k0 = (kb - s * a.kbs) * pt::BK;
    const int za = c.z + (s == 1 ? a.batch : 0), zb = c.z + (s == 0 ? a.batch : 0);
    const int mrow = c.m0 + rank * 128, n = c.n0 + rank * (a.width / 2);
    if (AMN) {
      tma_load_3d_pair(a_dst, &m.A, bar, mrow, k0, za);
      tma_load_3d_pair(a_dst + 8192, &m.A, bar, mrow + 64, k0, za);
    } else {
      tma_load_3d_pair(a_dst, &m.A, bar, k0, mrow, za);
    }
    if (BMN) {
      for (int j = 0; j < chunks64(a); ++j) tma_load_3d_pair(b_dst + j * 8192, &m.B, bar, n + 64 * j, k0, zb);
    } else {
      tma_load_3d_pair(b_dst, &m.B, bar, k0, n, zb);
    }
  }
  template <class Wait, class Release>
  static __device__ __forceinline__ void epilogue(const Maps& m, const Args& a, const Unit& c, int ew, int rank,
                                                  uint32_t taddr, uint8_t* slot, Wait wait, Release release) {
    const int lane = threadIdx.x & 31;
    const int row0 = c.m0 + rank * 128 + ((ew + 2) & 3) * 32;
    const int rows = min(32, a.M - row0);
    const int first = ew >> 2;  // the quadrant's warps take its 32-column blocks in turn
    // blocks of this warp: inside the result, and (symmetric) not above the diagonal
    int last = rows > 0 ? min(a.width, a.N - c.n0) : 0;
    if (SYM) last = min(last, row0 + 32 - c.n0);
    const int blocks = last > 32 * first ? (last - 32 * first + 63) / 64 : 0;
    pt::BlockRegs shi, slo;
    auto fetch = [&](int i) {
      const int n = c.n0 + (first + 2 * i) * 32;
      const uint16_t* p = a.s + c.z * a.s_matrix + row0 * a.s_pitch + n;
      pt::block_fetch(shi, p, a.s_pitch, rows, (min(32, a.N - n) + 7) & ~7, lane, true);
      pt::block_fetch(slo, p + a.s_part, a.s_pitch, rows, (min(32, a.N - n) + 7) & ~7, lane, true);
    };
    if (EP == EP_POLY && blocks > 0) fetch(0);
    if (!wait()) return;
    if (blocks == 0) release();
#pragma unroll 1
    for (int i = 0; i < blocks; ++i) {
      const int col = (first + 2 * i) * 32, n = c.n0 + col;
      float v[32];
      tmem_ld_32x32b_x32(taddr + col, reinterpret_cast<uint32_t*>(v));
      tmem_ld_wait();
      if (i == blocks - 1) release();
      if (lane == 0) bulk_wait_read<0>();
      __syncwarp();
      if constexpr (EP == EP_OUT) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] *= a.a;
        if (a.out_f16) pt::put_row<true>(slot, lane, v);
        else pt::put_row<false>(slot, lane, v);
        fence_async_smem();
        __syncwarp();
        if (a.wide) {
          if (lane == 0) tma_store_3d(&m.C, smem_u32(slot), n, row0, c.z);
        } else {
          pt::block_store(slot, a.o + (static_cast<long long>(c.z) * a.M + row0) * a.N + n, a.N, rows, min(32, a.N - n), lane);
        }
      } else {
        if constexpr (EP == EP_POLY) {
          pt::block_put(shi, slot, lane);
          pt::block_put(slo, slot + pt::BLOCK, lane);
          __syncwarp();
          if (i + 1 < blocks) fetch(i + 1);
          const int diagonal = row0 + lane - n;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 h = *reinterpret_cast<uint4*>(pt::block_word(slot, lane, j));
            const uint4 l = *reinterpret_cast<uint4*>(pt::block_word(slot + pt::BLOCK, lane, j));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 x = pt::unpack16<false>(reinterpret_cast<const uint32_t*>(&h)[k]);
              const float2 y = pt::unpack16<false>(reinterpret_cast<const uint32_t*>(&l)[k]);
              const int e = 8 * j + 2 * k;
              v[e] = fmaf(a.c, v[e], fmaf(a.b, x.x + y.x, e == diagonal ? a.a : 0.f));
              v[e + 1] = fmaf(a.c, v[e + 1], fmaf(a.b, x.y + y.y, e + 1 == diagonal ? a.a : 0.f));
            }
          }
          __syncwarp();
        }
        float lo[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) split2(v[j], &v[j], &lo[j]);
        pt::put_row<false>(slot, lane, v);
        pt::put_row<false>(slot + pt::BLOCK, lane, lo);
        const bool turned = SYM && row0 > n;  // below the diagonal (blocks on it hold both sides)
        if (turned) {
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            *pt::block_elem(slot + 2 * pt::BLOCK, j, lane) = __bfloat16_as_ushort(__float2bfloat16_rn(v[j]));
            *pt::block_elem(slot + 3 * pt::BLOCK, j, lane) = __bfloat16_as_ushort(__float2bfloat16_rn(lo[j]));
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_3d(&m.C, smem_u32(slot), n, row0, c.z);
          tma_store_3d(&m.C, smem_u32(slot + pt::BLOCK), n, row0, c.z + a.batch);
          if (turned) {
            tma_store_3d(&m.C, smem_u32(slot + 2 * pt::BLOCK), row0, n, c.z);
            tma_store_3d(&m.C, smem_u32(slot + 3 * pt::BLOCK), row0, n, c.z + a.batch);
          }
        }
      }
      if (lane == 0) bulk_commit();
      __syncwarp();
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
constexpr int NORM_PARTS = 64;  // most partial sums of a matrix

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
// FP32 eight at a time and FP64 beyond; eights whose sum leaves FP32's range, or
// comes near its end, are added again in FP64.
template <typename T>
__global__ void __launch_bounds__(NORM_THREADS) orth_norm_kernel(const T* G, double* part, long long n, int parts, int wide) {
  __shared__ double s[NORM_THREADS / 32];
  pdl_wait();  // no early trigger: large batches make more CTAs than fit at once
  const long long z = blockIdx.x / parts;
  const int k = static_cast<int>(blockIdx.x - z * parts);
  const T* p = G + z * n;
  const long long groups = (n + 7) / 8;
  double sum = 0.;
  for (long long g = static_cast<long long>(k) * NORM_THREADS + threadIdx.x; g < groups;
       g += static_cast<long long>(parts) * NORM_THREADS) {
    float v[8], q = 0.f;
    eight<T>(p, g * 8, n, wide, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) q = fmaf(v[j], v[j], q);
    if (q > 1e-30f && q < 1e38f) {
      sum += q;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += static_cast<double>(v[j]) * v[j];
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
  if (threadIdx.x == 0) {
    double sum = 0.;
    for (int i = 0; i < parts; ++i) sum += part[z * parts + i];
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
  const int64_t want = (rows * cols + 8 * NORM_THREADS - 1) / (8 * NORM_THREADS);
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

template <class P>
cudaError_t product(const OrthCall& g, const Matrix& A, const Matrix& B, const Matrix& C, OrthArgs a) {
  OrthMaps m = {};
  a.M = static_cast<int>(C.rows);
  a.N = static_cast<int>(C.cols);
  a.batch = static_cast<int>(g.batch);
  a.m_tiles = (a.M + 255) / 256;
  const int64_t K = P::A_MN ? A.rows : A.cols;
  a.kbs = static_cast<int>((K + pt::BK - 1) / pt::BK);
  auto fit = [&](int tiles) {  // columns in so many tiles of nearly equal width
    a.width = ((a.N + tiles - 1) / tiles + 31) / 32 * 32;
    a.n_tiles = (a.N + a.width - 1) / a.width;
    a.per = 0;
    if (P::SYM)
      for (int i = 0; i < a.m_tiles; ++i) a.per += sym_tiles(i, a.n_tiles, a.width);
    else
      a.per = a.m_tiles * a.n_tiles;
    a.units = a.per * a.batch;
  };
  int tiles = (a.N + 255) / 256;
  fit(tiles);
  // narrower tiles while there are pairs for twice as many
  while (a.units <= g.num_sms / 4 && a.width > 64) fit(tiles *= 2);
  a.idesc = idesc_f16(true, P::A_MN, P::B_MN, 256, 0);
  a.timeout_ns = g.timeout_ns;
  a.status = g.status;
  const uint64_t planes = 2 * static_cast<uint64_t>(g.batch);
  auto map = [&](CUtensorMap* t, const Matrix& x, bool mn, int box_rows) {
    const uint64_t pitch = static_cast<uint64_t>(x.pitch) * 2;
    return encode_tmap_3d(t, x.p, EK_BF16, x.cols, x.rows, planes, pitch, x.rows * pitch, 64, mn ? 64 : box_rows, 128);
  };
  bool ok = map(&m.A, A, P::A_MN, 128) && map(&m.B, B, P::B_MN, a.width / 2);
  const uint64_t pc = static_cast<uint64_t>(C.pitch) * 2;
  if (P::EP_KIND == EP_OUT) {
    a.wide = C.cols % 8 == 0 && reinterpret_cast<uintptr_t>(C.p) % 16 == 0;
    a.out_f16 = g.out_kind == EK_F16;
    a.o = static_cast<uint16_t*>(C.p);
    a.a = g.scale;
    if (a.wide) ok = ok && encode_tmap_3d(&m.C, C.p, g.out_kind, C.cols, C.rows, g.batch, pc, C.rows * pc, 32, 32, 64);
  } else {
    ok = ok && encode_tmap_3d(&m.C, C.p, EK_BF16, C.cols, C.rows, planes, pc, C.rows * pc, 32, 32, 64);
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
  for (int64_t i = 0; i < g.steps && e == cudaSuccess; ++i) {
    const Matrix &x = X[i & 1], &y = X[(i + 1) & 1];
    OrthArgs a = {};
    e = tall ? product<OrthProduct<true, true, EP_SYM>>(g, x, x, S, a) : product<OrthProduct<false, false, EP_SYM>>(g, x, x, S, a);
    if (e != cudaSuccess) break;
    a.s = static_cast<const uint16_t*>(S.p);
    a.s_pitch = l.pitch_s;
    a.s_part = l.s_part;
    a.s_matrix = l.m * l.pitch_s;
    a.a = static_cast<float>(g.coeffs[3 * i]);
    a.b = static_cast<float>(g.coeffs[3 * i + 1]);
    a.c = static_cast<float>(g.coeffs[3 * i + 2]);
    e = product<OrthProduct<false, false, EP_POLY>>(g, S, S, Q, a);
    if (e != cudaSuccess) break;
    a = {};
    if (i + 1 < g.steps)
      e = tall ? product<OrthProduct<false, false, EP_X>>(g, x, Q, y, a) : product<OrthProduct<false, true, EP_X>>(g, Q, x, y, a);
    else
      e = tall ? product<OrthProduct<false, false, EP_OUT>>(g, x, Q, O, a) : product<OrthProduct<false, true, EP_OUT>>(g, Q, x, O, a);
  }
  return e;
}

}  // namespace tg
