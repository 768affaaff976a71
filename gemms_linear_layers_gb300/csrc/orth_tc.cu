// orth_tc.cu -- the orthogonalised update of a weight from its gradient: with
// X = G / (|G| + eps) (Frobenius norm), `steps` times, m = min(rows, cols)
//   A = X X^T,  Q = a I + b A + c A A,  X = Q X          (rows <= cols)
//   A = X^T X,  Q = a I + b A + c A A,  X = X Q          (rows > cols)
// which takes every singular value s of X to a s + b s^3 + c s^5 and so all of
// them towards 1, and O = scale X.
//
// Everything between the products is held as two fp16 parts, v = hi + lo, and a product is
// the three products hi lo + lo hi + hi hi in one FP32 accumulator.  One 16-bit part would
// not do: rounding spreads over all directions alike, and a direction that the gradient
// barely has is multiplied by a^steps (485 for five steps of a = 3.44) on its way to 1, the
// rounding of the strong directions with it.  Two bf16 parts (2^-17) fell short too where eight
// strong directions stand beside others of 1e-3: 7e-4 of a result's size after five steps and
// 2.3e-3 after six (300 x 700), beside 2.1e-4 of rounding to fp16.  Two fp16 parts hold 22 bits
// where a value's size lets them, so X, A and Q are stored times powers of two that bring the
// largest they can be to 2^15 (see Ranges): what is lost is 2^-22 of a value or 2^-40 of that
// bound, 1.5e-5 and 4e-5 of those results when emulated with exact sums.  The rest is the tensor
// cores' FP32 sums, which cut off what lies below their last bit.  Measured, of a result's size
// beside its own rounding, others of 0.3 / 1e-3 after five steps: 300 x 700 1.2e-5 / 8e-5,
// 576 x 576 1.6e-5 / 1.4e-4, 2,304 x 2,304 2.7e-5 / 6e-4; after six, of 1e-3, 2.6e-4, 4.8e-4 and
// 1.9e-3.  (FP32 products: 2e-6 / 3e-5, 2e-6 / 4e-5, 3e-6 / 9e-5; 1.0e-4, 1.3e-4, 2.8e-4.  Against
// bf16 parts fp16 cost 6 % for four of 5,760 x 2,304, power, and 1 % and less below.  The sums of
// hi hi apart from the others' left no less after five steps; a X added beside the sum instead of
// a I within it left half, for 10 % of 8 x 1,536 x 576.)
// A and Q are symmetric: only tiles that reach the diagonal or lie below it are
// computed and stored; an operand's block above it is loaded from below, where it is
// the same block MN-major, and the instruction is told so block by block.
// A tall G needs no transpose: its A is the product of MN-major operands, its
// X Q takes the symmetric Q as a K-major one.
#include <cmath>
#include <type_traits>

#include "orth.h"

#include "pair_tc.cuh"
#include "pitch_copy.cuh"

namespace tg {
namespace {

// What a product makes of its sum.
enum {
  EP_A = 0,   // A, X                     two parts, A symmetric
  EP_Q = 1,   // Q = a I + b A + c sum    two parts, symmetric
  EP_OUT = 2  // scale X                  the result
};

constexpr int MAX_STEPS = 64;

// Powers of two that the parts are scaled with.  X of step i is stored times 2^(bits - e_i), A
// times 2^(bits - 2 e_i), Q times 2^(bits - q_i), where 2^e_i is not below X's spectral norm
// (which no entry exceeds) and 2^q_i not below |a + b s^2 + c s^4| for the s that X can have.
// e_0 is a matrix's own, from |G| / (|G| + eps); e_(i+1) = min(x_(i+1), e_i + q_i), x_i the
// bound that holds for every matrix.  Coefficients that let X's size move too far from its
// bound for fp16 (through a zero of the polynomial, or by growing without limit) take bf16
// parts, unscaled (bits = 0, all exponents 0), of 2^-17.
struct Ranges {
  int f16, bits;
  signed char x[MAX_STEPS + 1], q[MAX_STEPS];
};
__host__ __device__ inline int next_range(const Ranges& r, int i, int e) {
  const int grown = e + r.q[i];
  return grown < r.x[i + 1] ? grown : r.x[i + 1];
}
constexpr int LEAST_RANGE = -100;  // of a matrix that eps leaves next to nothing of

// How an operand lies in memory.  OP_SYM: a symmetric matrix stored in part.  Row
// tile i (256 rows) of it holds its columns before 256 (i + 1), and the rest is taken
// from the other side of the diagonal, where a block lies MN-major.  When the last
// row tile has at most half its rows, these are stored, and computed, as the last
// columns of the tiles above (`strip` is the first of them), so that their products
// are narrow in N and not mostly empty in M.
enum { OP_K = 0, OP_MN = 1, OP_SYM = 2 };

// All products of a call are one launch.  A unit is a tile of a product of a matrix; the
// units go product by product and, within one, matrix by matrix, dealt to the pairs in
// turn.  A matrix's next product begins when every tile of its last one has been stored
// (a counter of each matrix, in the workspace), whatever the other matrices are at, so
// only small batches wait at a product's end.  A unit waits for units before it only, and
// the launch is cooperative, so every wait ends.  (A launch a product made 24 matrices of
// 576 x 576 15 % slower and four of 5,760 x 2,304 1 %; one of 576 x 576 7 % faster, one of
// 2,304 x 2,304 4 %.)
//
// Measured: 24 of 576 x 576 314 us; four of 5,760 x 2,304 3.9 ms, 81 % of the MMA rate; one of
// 2,304 x 2,304 596 us; one of 576 x 576 118 us, one of 192 x 576 87 us: fifteen products in
// a row of 5 to 8 us, a third of it until a tile's stores are seen by others.  An epilogue
// step of 64 columns takes 3,000 to 4,300 cycles, as its stores wait behind the main loop's
// copies.  Stores straight from registers were slower still (24 of 576 x 576 26 %), stores by
// the lanes from shared memory, 64 bytes of a row at a time, too (3 %; 192 x 576 7 %, 100 of
// 64 x 64 5 %).
struct OrthMaps {
  // X (two buffers), A, Q, as loaded: K-major boxes of 128 rows, of half a tile's rows, MN-major boxes
  CUtensorMap k[4], kb[4], mn[4];
  CUtensorMap store[5];  // as stored, and the result
};
enum { BUF_S = 2, BUF_Q = 3, BUF_O = 4 };  // 0, 1: X

struct OrthArgs {
  const uint16_t* buf[4];
  int* done;           // [batch] blocks of 32 rows of tiles that have been stored: 8 a unit
  const int* range0;   // [batch] e_0
  uint16_t* o;
  long long x_pitch, x_part, s_pitch, s_part;  // elements from row to row, part to part
  int rows, cols, m;   // of X; min(rows, cols)
  int batch, steps, units;
  int sym_units, x_units;  // of a matrix: of a symmetric product, of the product with X
  int sym_main, sym_tiles_n, x_tiles_m, x_tiles_n, width;
  int strip;
  int kb_gram, kb_m;   // blocks of the reductions
  int wide, out_f16;
  float scale;
  unsigned long long timeout_ns;
  unsigned int* status;
  float coeffs[MAX_STEPS][3];  // a, b, c times 2^(bits - q), 2^-q, 2^(-bits - q)
  Ranges range;
};
struct OrthUnit {
  int step, kind;  // kind 0: A, 1: Q, 2: X
  int z, m0, n0, kb, nmma;
  int cols;        // that are stored (from n0 on)
  bool last;       // step
};

// Two values as two parts: the first parts packed, the values' rests packed.
template <bool F16>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t* hi, uint32_t* lo) {
  *hi = pt::pack16<F16>(x, y);
  const float2 h = pt::unpack16<F16>(*hi);
  *lo = pt::pack16<F16>(x - h.x, y - h.y);
}
// 2^n, 0 below FP32's normal range
__device__ __forceinline__ float power_of_two(int n) { return n < -126 ? 0.f : __int_as_float((n + 127) << 23); }
__device__ __forceinline__ int count_acquire(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// Column tiles of a symmetric result's row tile i.
__host__ __device__ inline int sym_tiles(int i, int n_tiles, int width) {
  const int n = (i * 256 + 255) / width + 1;
  return n < n_tiles ? n : n_tiles;
}
__host__ __device__ inline int up64(int n) { return (n + 63) / 64 * 64; }

// NARROW: tiles of up to 128 columns, whose part of B needs half the place: a stage more
// (8 of 1,536 x 576 6 us less, now 242; one of 576 x 576 5, now 118).  Stages of one part (five,
// and blocks for two epilogue steps beside them) cost these 13 us and 10.
template <bool TALL, bool NARROW>
struct OrthChain {
  using Maps = OrthMaps;
  using Args = OrthArgs;
  using Unit = OrthUnit;
  using State = pt::NoState;
  static constexpr bool COOPERATIVE = true;
  static constexpr int PARTS = 2, STAGES = NARROW ? 4 : 3, B_PART = NARROW ? pt::B_BYTES / 2 : pt::B_BYTES, EPI_BLOCKS = 2;
  static constexpr unsigned SITE = 0x60;

  static __device__ __forceinline__ uint32_t idesc(const Args& a, const Unit&) {
    return idesc_f16(!a.range.f16, false, false, 256, 0);
  }
  // How the operands of a product lie, and the buffers they are in.
  static __device__ __forceinline__ int a_op(const Unit& c) { return c.kind == 0 ? (TALL ? OP_MN : OP_K) : c.kind == 1 ? OP_SYM : TALL ? OP_K : OP_SYM; }
  static __device__ __forceinline__ int b_op(const Unit& c) { return c.kind == 0 ? (TALL ? OP_MN : OP_K) : c.kind == 1 ? OP_SYM : TALL ? OP_SYM : OP_MN; }
  static __device__ __forceinline__ int a_buf(const Unit& c) { return c.kind == 0 ? c.step & 1 : c.kind == 1 ? BUF_S : TALL ? c.step & 1 : BUF_Q; }
  static __device__ __forceinline__ int b_buf(const Unit& c) { return c.kind == 0 ? c.step & 1 : c.kind == 1 ? BUF_S : TALL ? BUF_Q : c.step & 1; }
  static __device__ __forceinline__ int c_buf(const Unit& c) { return c.kind == 0 ? BUF_S : c.kind == 1 ? BUF_Q : c.last ? BUF_O : (c.step + 1) & 1; }

  static __device__ __forceinline__ bool mn(const Args& a, int op, int row, int k0) {
    if (op != OP_SYM) return op == OP_MN;
    if (row >= a.strip) return k0 < a.strip;
    return k0 < a.strip && k0 >= ((row >> 8) + 1) << 8;
  }
  static __device__ __forceinline__ bool a_mn(const Args& a, const Unit& c, int kb) { return mn(a, a_op(c), c.m0, kb * pt::BK); }
  static __device__ __forceinline__ bool b_mn(const Args& a, const Unit& c, int kb) { return mn(a, b_op(c), c.n0, kb * pt::BK); }
  static __device__ __forceinline__ void prefetch(const Maps& m, const Args&) {
    prefetch_tmap(TALL ? &m.mn[0] : &m.k[0]);
    prefetch_tmap(TALL ? &m.mn[0] : &m.kb[0]);
  }
  static __device__ __forceinline__ bool unit(const Args& a, int u, Unit& c) {
    const int sym = a.sym_units * a.batch, step = 2 * sym + a.x_units * a.batch;
    c.step = u / step;
    int r = u - c.step * step;
    c.kind = r < sym ? 0 : r < 2 * sym ? 1 : 2;
    r -= c.kind * sym;
    c.last = c.step + 1 == a.steps;
    const int per = c.kind < 2 ? a.sym_units : a.x_units;
    c.z = r / per;
    r -= c.z * per;
    c.kb = c.kind == 0 ? a.kb_gram : a.kb_m;
    if (c.kind < 2) {
      if (r >= a.sym_main) {  // the strip: a tile of every row tile
        c.m0 = (r - a.sym_main) * 256;
        c.n0 = a.strip;
        c.cols = a.m - a.strip;
        c.nmma = up64(c.cols);
        return true;
      }
      int i = 0;
      for (int n; r >= (n = sym_tiles(i, a.sym_tiles_n, a.width)); ++i) r -= n;
      c.m0 = i * 256;
      c.n0 = r * a.width;
      c.cols = min(min(a.width, c.m0 + 256 - c.n0), a.m - c.n0);
      c.nmma = up64(min(a.width, a.m - c.n0));
    } else {
      const int N = TALL ? a.m : a.cols, j = r / a.x_tiles_m;
      c.m0 = (r - j * a.x_tiles_m) * 256;
      c.n0 = j * a.width;
      c.cols = min(a.width, N - c.n0);
      c.nmma = up64(c.cols);
    }
    return true;
  }
  // Units of this matrix that come before the product, times 8.
  static __device__ __forceinline__ int target(const Args& a, const Unit& c) {
    return 8 * (c.step * (2 * a.sym_units + a.x_units) + c.kind * a.sym_units);
  }
  static __device__ __forceinline__ bool ready(const Args& a, const Unit& c, volatile int* abort_flag) {
    const int want = target(a, c);
    if (want == 0) return true;
    const int* p = a.done + c.z;
    if (count_acquire(p) < want) {
      const uint64_t t0 = globaltimer_ns();
      for (uint32_t it = 1; count_acquire(p) < want; ++it) {
        if ((it & 31u) == 0u) {
          if (*abort_flag) return false;
          __nanosleep(20);
          if (globaltimer_ns() - t0 > a.timeout_ns) {
            *abort_flag = 1;
            atomicOr(a.status, TG_DEVSTAT_TIMEOUT | (SITE & TG_DEVSTAT_SITE_MASK));
            return false;
          }
        }
      }
    }
    asm volatile("fence.proxy.async;" ::: "memory");  // the copies that follow see what the counter stands for
    return true;
  }
  // Boxes of a K-major B hold half a whole tile's rows.  One that may be either way comes
  // in whole 64 x 64 boxes, so that its bytes are the same.
  static __device__ __forceinline__ int b_rows(const Args& a, int op) { return op == OP_K ? a.width / 2 : up64(a.width / 2); }
  static __device__ __forceinline__ uint32_t bytes(const Args& a, const Unit& c) {
    return PARTS * (pt::A_BYTES + b_rows(a, b_op(c)) * pt::BK * 2);
  }
  static __device__ __forceinline__ void load(const Maps& m, const Args& a, const Unit& c, int kb, int rank,
                                              uint32_t a_dst, uint32_t b_dst, uint32_t bar) {
    const int k0 = kb * pt::BK;
    const int mrow = c.m0 + rank * 128, n = c.n0 + rank * (c.nmma / 2);
    const bool am = a_mn(a, c, kb), bm = b_mn(a, c, kb);
    const int ab = a_buf(c), bb = b_buf(c), op = b_op(c), rows = b_rows(a, op);
    for (int p = 0; p < PARTS; ++p) {
      const int z = c.z + p * a.batch;
      if (am) {
        tma_load_3d_pair(a_dst, &m.mn[ab], bar, mrow, k0, z);
        tma_load_3d_pair(a_dst + 8192, &m.mn[ab], bar, mrow + 64, k0, z);
      } else {
        tma_load_3d_pair(a_dst, &m.k[ab], bar, k0, mrow, z);
      }
      if (bm) {
        for (int j = 0; j < rows; j += 64) tma_load_3d_pair(b_dst + j * 128, &m.mn[bb], bar, n + j, k0, z);
      } else {
        tma_load_3d_pair(b_dst, &m.kb[bb], bar, k0, n, z);
      }
      a_dst += pt::A_BYTES;
      b_dst += B_PART;
    }
  }

  // What EP makes of the accumulator's 64 columns from `col` on, into the quadrant's blocks.
  // k: what the unit matrix, A and the sum are taken times; without a polynomial the sum's factors.
  template <int EP, bool F16>
  static __device__ __forceinline__ void finish(const Args& a, const Unit& c, const pt::EpiWarp& at, int col, int row0,
                                                int rows, int lane, const float3& k, float* v) {
    uint8_t *b0 = at.blocks, *b1 = b0 + pt::BLOCK;
    const int n = c.n0 + col + 32 * at.h;
    if constexpr (EP == EP_Q) {  // A is in the blocks
      const int diagonal = row0 + lane - n;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 h = *reinterpret_cast<uint4*>(pt::block_word(b0, lane, 4 * at.h + j));
        const uint4 l = *reinterpret_cast<uint4*>(pt::block_word(b1, lane, 4 * at.h + j));
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float2 x = pt::unpack16<F16>(reinterpret_cast<const uint32_t*>(&h)[w]);
          const float2 y = pt::unpack16<F16>(reinterpret_cast<const uint32_t*>(&l)[w]);
          const int e = 8 * j + 2 * w;
          v[e] = fmaf(k.z, v[e], fmaf(k.y, x.x + y.x, e == diagonal ? k.x : 0.f));
          v[e + 1] = fmaf(k.z, v[e + 1], fmaf(k.y, x.y + y.y, e + 1 == diagonal ? k.x : 0.f));
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = EP == EP_OUT ? v[j] * k.x * k.y * k.z : v[j] * k.x;
    }
    if constexpr (EP == EP_OUT) {
      if (a.out_f16) pt::put_row<true>(b0, lane, at.h, v);
      else pt::put_row<false>(b0, lane, at.h, v);
      if (!a.wide)
        pt::half_store(b0, at.h, a.o + (static_cast<long long>(c.z) * a.rows + row0) * a.cols + n, a.cols, rows,
                       min(32, a.cols - n), lane);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split_pair<F16>(v[8 * j + 2 * e], v[8 * j + 2 * e + 1], &hi[e], &lo[e]);
        *reinterpret_cast<uint4*>(pt::block_word(b0, lane, 4 * at.h + j)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(pt::block_word(b1, lane, 4 * at.h + j)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
    }
  }
  template <class Wait, class Release>
  static __device__ __forceinline__ void epilogue(const Maps& m, const Args& a, const Unit& c, const Unit*,
                                                  const pt::EpiWarp& at, pt::NoState&, Wait wait, Release release) {
    const int lane = threadIdx.x & 31;
    volatile int* abort_flag = at.abort_flag;
    const bool result = c.kind == 2 && c.last;
    const int ep = c.kind == 1 ? EP_Q : result ? EP_OUT : EP_A;
    // the factors between what is stored: see Ranges
    const int bits = a.range.bits;
    float3 k = make_float3(power_of_two(-bits), 0.f, 0.f);
    if (c.kind > 0) {
      int e = a.range0[c.z];
      for (int i = 0; i < c.step; ++i) e = next_range(a.range, i, e);
      const int q = a.range.q[c.step];
      if (c.kind == 1) {
        const float* p = a.coeffs[c.step];
        k = make_float3(p[0], p[1] * power_of_two(2 * e), p[2] * power_of_two(4 * e));
      } else if (result) {  // X, then its scale: no product of factors may leave FP32's range
        k = make_float3(power_of_two(-2 * bits), power_of_two(q + e), a.scale);
      } else {
        k.x = power_of_two(e - next_range(a.range, c.step, e) + q - bits);
      }
    }
    const int M = c.kind == 2 && TALL ? a.rows : a.m;
    const int row0 = c.m0 + at.rank * 128 + at.q * 32;
    const int rows = min(32, M - row0);
    const int cols = rows > 0 ? c.cols : 0;
    uint8_t *b0 = at.blocks, *b1 = b0 + pt::BLOCK;
    pt::HalfRegs in0, in1;
    // the polynomial's A
    auto fetch = [&](int col) {
      const int n = c.n0 + col + 32 * at.h;
      const int left = (a.m - n + 7) & ~7;  // rows are whole words; what lies past the columns is not stored
      const uint16_t* p = a.buf[BUF_S] + (static_cast<long long>(c.z) * a.m + row0) * a.s_pitch + n;
      pt::half_fetch(in0, p, a.s_pitch, rows, left, lane, true);
      pt::half_fetch(in1, p + a.s_part, a.s_pitch, rows, left, lane, true);
    };
    // what this unit's copies wait for, the epilogue's first loads do too (one thread a quadrant looks: two
    // cost 8 matrices of 1,536 x 576 3 us); their lines are taken past L1
    if (ep == EP_Q && cols > 0) {
      if (pt::quadrant_all(at.q, lane != 0 || at.h != 0 || ready(a, c, abort_flag))) fetch(0);
    }
    if (!wait()) return;
    if (cols <= 0) release();
#pragma unroll 1
    for (int col = 0; col < cols; col += 64) {
      float v[32];
      tmem_ld_32x32b_x32(at.taddr + col + 32 * at.h, reinterpret_cast<uint32_t*>(v));
      tmem_ld_wait();
      if (col + 64 >= cols) release();
      pt::blocks_free(at, lane);
      if (ep == EP_Q) {
        pt::half_put(in0, b0, at.h, lane);
        pt::half_put(in1, b1, at.h, lane);
        __syncwarp();
        if (col + 64 < cols) fetch(col + 64);
      }
      auto parts = [&](auto f16) {
        constexpr bool F16 = decltype(f16)::value;
        if (ep == EP_Q) finish<EP_Q, F16>(a, c, at, col, row0, rows, lane, k, v);
        else finish<EP_A, F16>(a, c, at, col, row0, rows, lane, k, v);  // X too
      };
      if (result) finish<EP_OUT, true>(a, c, at, col, row0, rows, lane, k, v);
      else if (a.range.f16) parts(std::true_type());
      else parts(std::false_type());
      if (result && !a.wide) continue;
      if (pt::blocks_full(at, lane)) {
        const CUtensorMap* to = &m.store[c_buf(c)];
        tma_store_3d(to, smem_u32(b0), c.n0 + col, row0, c.z);
        if (!result) tma_store_3d(to, smem_u32(b1), c.n0 + col, row0, c.z + a.batch);
        bulk_commit();
      }
    }
    if (!result && at.h == 0 && lane == 0) {  // the thread that stored this quadrant's rows
      bulk_wait_all();
      asm volatile("fence.proxy.async;" ::: "memory");
      asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(a.done + c.z) : "memory");
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

// X, two parts of [batch][rows][pitch], from G [batch][rows][cols], and each matrix's e_0
// (see Ranges).  `blocks` CTAs a matrix.
template <typename T>
__global__ void __launch_bounds__(256) orth_split_kernel(const T* G, const double* part, uint16_t* X, long long rows, int cols,
                                                         int pitch, int parts, int blocks, long long part_stride, float eps,
                                                         int wide, int* done, int* range0, int f16, int bits) {
  __shared__ float factor[2];
  pdl_wait();
  const long long z = blockIdx.x / blocks;
  const int k = static_cast<int>(blockIdx.x - z * blocks);
  if (threadIdx.x < 32) {
    double sum = 0.;
    for (int i = threadIdx.x; i < parts; i += 32) sum += part[z * parts + i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    const double norm = sqrt(sum), under = norm + static_cast<double>(eps);
    int e = 0;
    if (bits > 0 && norm < under) {  // |X| = norm / under < 1, at most 2^e
      frexp(norm / under, &e);
      e = min(0, max(LEAST_RANGE, e));
    }
    if (k == 0 && threadIdx.x == 0) {
      done[z] = 0;
      range0[z] = e;
    }
    const double inv = ldexp(1., bits - e) / under;
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
      if (f16) split_pair<true>(v[2 * j] * f0 * f1, v[2 * j + 1] * f0 * f1, &hi[j], &lo[j]);
      else split_pair<false>(v[2 * j] * f0 * f1, v[2 * j + 1] * f0 * f1, &hi[j], &lo[j]);
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
  size_t x[2], s, q, sums, done, bytes;  // offsets
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
  l.done = take(8 * static_cast<size_t>(batch));  // and e_0
  l.bytes = at;
  return l;
}

// First column of a symmetric matrix's strip (m when it has none).
int strip_of(int64_t m) {
  const int rest = static_cast<int>(m % 256);
  return static_cast<int>(m > 256 && rest > 0 && rest <= 128 ? m - rest : m);
}

template <bool TALL>
cudaError_t chain(const OrthCall& g, const Places& l, OrthArgs a) {
  OrthMaps m = {};
  const int pairs = g.num_sms / 2, mt = (a.m + 255) / 256;
  a.strip = strip_of(a.m);
  const bool split = a.strip < a.m;
  const int main_rows = split ? a.strip / 256 : mt, rest = up64(a.m - a.strip);
  a.x_tiles_m = TALL ? (a.rows + 255) / 256 : mt;
  auto fit = [&](int w) {
    a.width = w;
    a.sym_tiles_n = (a.strip + w - 1) / w;
    a.sym_main = 0;
    for (int i = 0; i < main_rows; ++i) a.sym_main += sym_tiles(i, a.sym_tiles_n, w);
    a.sym_units = a.sym_main + (split ? mt : 0);
    a.x_tiles_n = ((TALL ? a.m : a.cols) + w - 1) / w;
    a.x_units = a.x_tiles_m * a.x_tiles_n;
  };
  // The width with which a step takes least: a unit costs its columns and UNIT_COST more,
  // rounds of units end together in a batch of one and run into each other in a large one.
  // Tiles must not straddle a strip's first column, and hold its columns.
  int best = 0;
  double least = 0.;
  for (int w = 64; w <= 256; w += 64) {
    if (split && (w < rest || 256 % w != 0)) continue;
    fit(w);
    auto rounds = [&](double units) { return units * g.batch > 4. * pairs ? units * g.batch / pairs : ceil(units * g.batch / pairs); };
    const double cost = (2. * a.kb_m + 2. * a.kb_gram) / 2. * rounds(a.sym_main) * (w + UNIT_COST) +
                        (split ? (a.kb_m + a.kb_gram) * rounds(mt) * (rest + UNIT_COST) : 0.) +
                        a.kb_m * rounds(a.x_units) * (w + UNIT_COST);
    if (best == 0 || cost <= least) best = w, least = cost;
  }
  fit(best);
  *g.form = {best, a.range.f16 != 0};
  const int64_t units = static_cast<int64_t>(a.steps) * g.batch * (2 * a.sym_units + a.x_units);
  if (units > (int64_t(1) << 30) || 8 * (units / g.batch) > (int64_t(1) << 30)) return cudaErrorInvalidValue;
  a.units = static_cast<int>(units);
  // a wait may last as long as everything before it
  const int64_t blocks = (units / pairs + 1) * (a.kb_gram > a.kb_m ? a.kb_gram : a.kb_m);
  a.timeout_ns = g.timeout_ns + static_cast<unsigned long long>(blocks) * 4000ull;
  const uint64_t planes = 2 * static_cast<uint64_t>(g.batch);
  bool ok = true;
  for (int i = 0; i < 4; ++i) {
    const bool x = i < 2;
    const uint64_t rows = x ? a.rows : a.m, cols = x ? a.cols : a.m, pitch = (x ? a.x_pitch : a.s_pitch) * 2;
    auto map = [&](CUtensorMap* t, int box_cols, int box_rows) {
      ok = ok && encode_tmap_3d(t, a.buf[i], EK_BF16, cols, rows, planes, pitch, rows * pitch, box_cols, box_rows, 128);
    };
    map(&m.k[i], 64, 128);
    map(&m.kb[i], 64, x ? a.width / 2 : up64(a.width / 2));
    map(&m.mn[i], 64, 64);
    map(&m.store[i], 64, 32);
  }
  a.wide = g.cols % 8 == 0 && reinterpret_cast<uintptr_t>(g.O) % 16 == 0;
  if (a.wide)
    ok = ok && encode_tmap_3d(&m.store[BUF_O], g.O, g.out_kind, g.cols, g.rows, g.batch, 2 * g.cols, g.rows * 2 * g.cols, 64, 32, 128);
  if (!ok) return cudaErrorInvalidValue;
  return a.width <= 128 ? pt::pair_launch<OrthChain<TALL, true>>(m, a, g.num_sms, g.stream)
                        : pt::pair_launch<OrthChain<TALL, false>>(m, a, g.num_sms, g.stream);
}

// The polynomial of a step where X's singular values s are at most t.
struct Span {
  double most;  // |a + b s^2 + c s^4|, at most
  double next;  // |a s + b s^3 + c s^5|, at most
  bool zero;    // somewhere
};
Span span_of(const double* k, double t) {
  const double a = k[0], b = k[1], c = k[2], end = t * t;
  Span r = {0., 0., false};
  bool above = false, below = false;
  auto look = [&](double u, bool turns) {
    if (!(u >= 0. && u <= end)) return;
    const double v = a + u * (b + u * c), size = fabs(v);
    above = above || v > 0.;
    below = below || v < 0.;
    r.zero = r.zero || v == 0.;
    if (turns) r.most = fmax(r.most, size);
    r.next = fmax(r.next, sqrt(u) * size);
  };
  look(0., true);
  look(end, true);
  if (c != 0.) look(-b / (2. * c), true);
  // where a s + b s^3 + c s^5 turns: a + 3 b u + 5 c u^2 = 0
  const double root = 9. * b * b - 20. * a * c;
  if (root >= 0.) {
    const double w = -(3. * b + copysign(sqrt(root), b)) / 2.;
    if (c != 0.) look(w / (5. * c), false);
    if (w != 0.) look(a / w, false);
  }
  r.zero = r.zero || (above && below);
  return r;
}
int exponent_above(double v) {  // 2^this >= v
  int e = 0;
  const double m = frexp(v, &e);
  return m == 0.5 ? e - 1 : e;
}
// fp16 parts where what they lose below their range (2^-25 an entry as stored, 2^-39 of the
// bound that the scale comes from) stays under about 2^-20 of |X| whatever the matrix: X's
// bound of each step beside what becomes of |X|, followed on singular values of four sizes an
// octave, for each e_0.
Ranges ranges_of(const OrthCall& g) {
  Ranges r = {1, 15, {}, {}};
  const int steps = static_cast<int>(g.steps);
  const double entries = sqrt(static_cast<double>(g.rows) * static_cast<double>(g.cols));
  double t = 1.;
  for (int i = 0; i < steps; ++i) {
    const Span s = span_of(g.coeffs + 3 * i, t);
    t = s.next * (1. + 0x1p-10);  // rounding adds a little
    if (s.zero || !(t > 0x1p-30 && t < 0x1p30 && s.most > 0x1p-30 && s.most < 0x1p30)) return Ranges{};
    r.q[i] = static_cast<signed char>(exponent_above(s.most));
    r.x[i + 1] = static_cast<signed char>(exponent_above(t));
  }
  double kept[MAX_STEPS];  // the least |X_i| / |X_0|
  for (int i = 0; i < steps; ++i) kept[i] = HUGE_VAL;
  const int smallest = -16;  // below, a alone counts
  for (int e0 = smallest; e0 <= 0; ++e0) {
    for (const double part : {1., 0.841, 0.707, 0.595}) {
      const double from = ldexp(part, e0);
      double s = from;
      for (int i = 0; i < steps; ++i) {
        const double* k = g.coeffs + 3 * i;
        kept[i] = fmin(kept[i], s / from);
        s = fabs(s * (k[0] + s * s * (k[1] + s * s * k[2])));
      }
    }
    const int from = e0 == smallest ? -100000 : e0;
    for (int i = 0, e = from; i < steps; ++i) {  // |X_0| is above 2^(e_0 - 1)
      if (!(ldexp(entries, e - from) <= 0x1p18 * kept[i])) return Ranges{};
      e = next_range(r, i, e);
    }
  }
  return r;
}

template <typename T>
cudaError_t prepare(const OrthCall& g, const Places& l, double* sums, uint16_t* X, int* done, const Ranges& range) {
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
                  static_cast<int>(base && g.cols % 8 == 0), done, done + g.batch, range.f16, range.bits);
}

}  // namespace

bool orth_fits(int64_t batch, int64_t rows, int64_t cols, int64_t steps) {
  if (batch <= 0 || rows <= 0 || cols <= 0) return true;
  const int64_t m = rows < cols ? rows : cols, n = rows < cols ? cols : rows, most = int64_t(1) << 27;
  auto tiles = [](int64_t a, int64_t b) { return ((a + 255) / 256 + 1) * ((b + 63) / 64); };
  const int64_t each = 2 * tiles(m, m) + tiles(n, m) + tiles(m, n);
  return each <= most / steps && each * steps <= 8 * most / batch;
}

size_t orth_ws_bytes(int64_t batch, int64_t rows, int64_t cols) {
  return batch > 0 && rows > 0 && cols > 0 ? places(batch, rows, cols).bytes : 0;
}

cudaError_t orth_launch(const OrthCall& g) {
  const Places l = places(g.batch, g.rows, g.cols);
  char* ws = static_cast<char*>(g.ws);
  OrthArgs a = {};
  uint16_t* x0 = reinterpret_cast<uint16_t*>(ws + l.x[0]);
  const size_t at[4] = {l.x[0], l.x[1], l.s, l.q};
  for (int i = 0; i < 4; ++i) a.buf[i] = reinterpret_cast<const uint16_t*>(ws + at[i]);
  a.done = reinterpret_cast<int*>(ws + l.done);
  a.o = static_cast<uint16_t*>(g.O);
  a.x_pitch = l.pitch_x;
  a.x_part = l.x_part;
  a.s_pitch = l.pitch_s;
  a.s_part = l.s_part;
  a.rows = static_cast<int>(g.rows);
  a.cols = static_cast<int>(g.cols);
  a.m = static_cast<int>(l.m);
  a.batch = static_cast<int>(g.batch);
  a.steps = static_cast<int>(g.steps);
  a.kb_gram = static_cast<int>((l.long_side + pt::BK - 1) / pt::BK);
  a.kb_m = static_cast<int>((l.m + pt::BK - 1) / pt::BK);
  a.out_f16 = g.out_kind == EK_F16;
  a.scale = g.scale;
  a.status = g.status;
  a.range0 = a.done + g.batch;
  a.range = ranges_of(g);
  for (int64_t i = 0; i < g.steps; ++i)
    for (int j = 0; j < 3; ++j)
      a.coeffs[i][j] = static_cast<float>(ldexp(g.coeffs[3 * i + j], (1 - j) * a.range.bits - a.range.q[i]));
  double* sums = reinterpret_cast<double*>(ws + l.sums);
  const cudaError_t e = g.in_kind == EK_BF16  ? prepare<__nv_bfloat16>(g, l, sums, x0, a.done, a.range)
                        : g.in_kind == EK_F16 ? prepare<__half>(g, l, sums, x0, a.done, a.range)
                                              : prepare<float>(g, l, sums, x0, a.done, a.range);
  if (e != cudaSuccess) return e;
  return g.rows > g.cols ? chain<true>(g, l, a) : chain<false>(g, l, a);
}

}  // namespace tg
