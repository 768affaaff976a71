// gated_tc.cu -- the gated feed-forward block on tcgen05 CTA pairs.
//
// Forward:   G = X Wg^T, U = X Wu^T, H = act(G) U, in one product over the weight
//            [Wg; Wu]: a pair's tile takes `width` gate rows into rank 0's half of B
//            and the same up rows into rank 1's, so that columns j and width + j of
//            each CTA's accumulator are G and U of one element and H needs no exchange.
// Backward:  dH = dY Wd (the down projection's input gradient), then in the epilogue
//            dG = dH U act'(G), dU = dH act(G), and H = act(G) U again for the down
//            projection's weight gradient.  dH never reaches memory.
// Everything of an element is FP32 until its one rounding.  The blocks of G and U that
// a backward epilogue needs are asked for before its accumulator is waited for.
//
// Measured, 2,304 -> 5,760, 4,096 rows, bf16: forward 121 us (1,790 TFLOP/s; without G and
// U 114), backward 83 us (1,310 TFLOP/s; without H 77, GELU 88); 576 -> 1,536, 1,001 rows,
// fp16 GELU 11.5 and 12.2 us (bf16 SiLU 10.3 and 10.7), 4,096 rows 19 and 25 us.
// Bound by what passes an SM's port, 64 bytes a cycle in and out together: a 64-deep block
// brings a CTA 32 KB for 512 cycles of MMA, all the port has, so what an epilogue reads
// and writes comes on top: 96 KB of a forward unit (19,900 cycles a unit, 18,400 of MMA),
// 320 KB of a backward one (25,500).  Hence the epilogue moves nothing twice; a ring of 4
// instead of 5 stages cost the backward 6 us, slots for two steps of G and U 7, G and U asked
// into L2 ahead 11.
#include "gated.h"

#include <type_traits>

#include "gated_act.cuh"
#include "gated_few.h"
#include "pair_tc.cuh"
#include "pitch_copy.cuh"

namespace tg {
namespace {

struct GatedMaps {
  CUtensorMap A, B, H, GU;
};
struct GatedArgs {
  const uint16_t* gu_in;  // backward: G and U [T, 2 f]
  uint16_t *h, *gu;       // outputs (h, or forward gu, may be null)
  long long T, f;
  int kb, units, m_tiles, width;  // width: columns of H of a tile
  int act;
  int wide;  // outputs through TMA, G and U by 16-byte words
  uint32_t idesc;
  unsigned long long timeout_ns;
  unsigned int* status;
};
struct GatedUnit {
  int m0, f0, kb, nmma;
};

__device__ __forceinline__ bool gated_unit(const GatedArgs& a, int u, GatedUnit& c, int per) {
  const int nt = u / a.m_tiles;
  c.m0 = (u - nt * a.m_tiles) * 256;
  c.f0 = nt * a.width;
  c.kb = a.kb;
  c.nmma = per * a.width;
  return true;
}

// Half a block's `cols` columns from f on to `to`, element by element.
__device__ __forceinline__ void gated_put(uint8_t* block, int h, uint16_t* to, long long pitch, int f, int row0, int rows,
                                          int cols, int lane) {
  pt::half_store(block, h, to + static_cast<long long>(row0) * pitch + f, pitch, rows, cols, lane);
}

template <class F>
__device__ __forceinline__ void with_act(int act, F apply) {
  switch (act) {
    case ACT_SILU: apply(std::integral_constant<int, ACT_SILU>()); break;
    case ACT_GELU: apply(std::integral_constant<int, ACT_GELU>()); break;
    case ACT_GELU_TANH: apply(std::integral_constant<int, ACT_GELU_TANH>()); break;
    default: apply(std::integral_constant<int, ACT_RELU>()); break;
  }
}

template <bool F16>
struct GatedFwd {
  using Maps = GatedMaps;
  using Args = GatedArgs;
  using Unit = GatedUnit;
  using State = pt::NoState;
  static constexpr int PARTS = 1, STAGES = 5, B_PART = pt::B_BYTES, EPI_BLOCKS = 3;
  static constexpr unsigned SITE = 0x50;
  static constexpr bool COOPERATIVE = false;
  static __device__ __forceinline__ uint32_t idesc(const Args& a, const Unit&) { return a.idesc; }
  static __device__ __forceinline__ bool ready(const Args&, const Unit&, volatile int*) { return true; }
  static __device__ __forceinline__ bool a_mn(const Args&, const Unit&, int) { return false; }
  static __device__ __forceinline__ bool b_mn(const Args&, const Unit&, int) { return false; }
  static __device__ __forceinline__ void prefetch(const Maps& m, const Args& a) {
    if (a.kb > 0) {
      prefetch_tmap(&m.A);
      prefetch_tmap(&m.B);
    }
  }
  static __device__ __forceinline__ bool unit(const Args& a, int u, Unit& c) { return gated_unit(a, u, c, 2); }
  static __device__ __forceinline__ uint32_t bytes(const Args& a, const Unit&) { return pt::A_BYTES + a.width * pt::BK * 2; }
  static __device__ __forceinline__ void load(const Maps& m, const Args&, const Unit& c, int kb, int rank, uint32_t a_dst,
                                              uint32_t b_dst, uint32_t bar) {
    tma_load_3d_pair(a_dst, &m.A, bar, kb * pt::BK, c.m0 + rank * 128, 0);
    tma_load_3d_pair(b_dst, &m.B, bar, kb * pt::BK, c.f0, rank);  // rank 0: gate rows, rank 1: up rows
  }
  template <class Wait, class Release>
  static __device__ __forceinline__ void epilogue(const Maps& m, const Args& a, const Unit& c, const Unit*,
                                                  const pt::EpiWarp& at, pt::NoState&, Wait wait, Release release) {
    const int lane = threadIdx.x & 31;
    const int row0 = c.m0 + at.rank * 128 + at.q * 32;
    const int rows = static_cast<int>(min(32ll, a.T - row0));
    uint8_t *bh = at.blocks, *bg = bh + pt::BLOCK, *bu = bg + pt::BLOCK;
    if (!wait()) return;
#pragma unroll 1
    for (int col = 0; col < a.width; col += 64) {
      const int mine = col + 32 * at.h;
      float g[32], u[32];
      if (c.kb > 0) {
        tmem_ld_32x32b_x32(at.taddr + mine, reinterpret_cast<uint32_t*>(g));
        tmem_ld_32x32b_x32(at.taddr + a.width + mine, reinterpret_cast<uint32_t*>(u));
        tmem_ld_wait();
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) g[j] = u[j] = 0.f;
      }
      if (col + 64 >= a.width) release();
      if (rows <= 0 || c.f0 + col >= a.f) continue;
      pt::blocks_free(at, lane);
      if (a.gu) {
        pt::put_row<F16>(bg, lane, at.h, g);
        pt::put_row<F16>(bu, lane, at.h, u);
      }
      with_act(a.act, [&](auto kind) {
#pragma unroll
        for (int j = 0; j < 32; ++j) g[j] = activation<decltype(kind)::value>(g[j]) * u[j];
      });
      pt::put_row<F16>(bh, lane, at.h, g);
      if (a.wide) {
        if (pt::blocks_full(at, lane)) {
          tma_store_3d(&m.H, smem_u32(bh), c.f0 + col, row0, 0);
          if (a.gu) {
            tma_store_3d(&m.GU, smem_u32(bg), c.f0 + col, row0, 0);
            tma_store_3d(&m.GU, smem_u32(bu), c.f0 + col, row0, 1);
          }
          bulk_commit();
        }
      } else {
        const int f = c.f0 + mine, cols = static_cast<int>(min(32ll, a.f - f));
        gated_put(bh, at.h, a.h, a.f, f, row0, rows, cols, lane);
        if (a.gu) {
          gated_put(bg, at.h, a.gu, 2 * a.f, f, row0, rows, cols, lane);
          gated_put(bu, at.h, a.gu + a.f, 2 * a.f, f, row0, rows, cols, lane);
        }
      }
    }
  }
};

// The backward's blocks of G and U are copied into shared memory one 64-column step
// ahead, across units too, by cp.async: loads into registers would hold lines of L1,
// of which little is left beside this much shared memory, and came late (4,096 rows,
// 2,304 -> 5,760: 83 us).  dG and dU take their places; H leaves from registers.
template <bool F16>
struct GatedBwd {
  using Maps = GatedMaps;
  using Args = GatedArgs;
  using Unit = GatedUnit;
  struct State {
    int slot;      // blocks of the step at work: 2 slot, 2 slot + 1
    bool fetched;  // its copies have been requested
  };
  static constexpr int PARTS = 1, STAGES = 5, B_PART = pt::B_BYTES, EPI_BLOCKS = 4;
  static constexpr unsigned SITE = 0x58;
  static constexpr bool COOPERATIVE = false;
  static __device__ __forceinline__ uint32_t idesc(const Args& a, const Unit&) { return a.idesc; }
  static __device__ __forceinline__ bool ready(const Args&, const Unit&, volatile int*) { return true; }
  static __device__ __forceinline__ bool a_mn(const Args&, const Unit&, int) { return false; }
  static __device__ __forceinline__ bool b_mn(const Args&, const Unit&, int) { return true; }
  static __device__ __forceinline__ void prefetch(const Maps& m, const Args& a) { GatedFwd<F16>::prefetch(m, a); }
  static __device__ __forceinline__ bool unit(const Args& a, int u, Unit& c) { return gated_unit(a, u, c, 1); }
  static __device__ __forceinline__ int chunks64(const Args& a) { return (a.width / 2 + 63) / 64; }
  static __device__ __forceinline__ uint32_t bytes(const Args& a, const Unit&) {
    return pt::A_BYTES + chunks64(a) * 64 * pt::BK * 2;
  }
  static __device__ __forceinline__ void load(const Maps& m, const Args& a, const Unit& c, int kb, int rank,
                                              uint32_t a_dst, uint32_t b_dst, uint32_t bar) {
    tma_load_3d_pair(a_dst, &m.A, bar, kb * pt::BK, c.m0 + rank * 128, 0);
    const int n = c.f0 + rank * (a.width / 2);
    for (int j = 0; j < chunks64(a); ++j) tma_load_3d_pair(b_dst + j * 8192, &m.B, bar, n + 64 * j, kb * pt::BK, 0);
  }
  template <class Wait, class Release>
  static __device__ __forceinline__ void epilogue(const Maps& m, const Args& a, const Unit& c, const Unit* next,
                                                  const pt::EpiWarp& at, State& st, Wait wait, Release release) {
    const int lane = threadIdx.x & 31;
    const int row_in = at.rank * 128 + at.q * 32;
    const int row0 = c.m0 + row_in;
    const int rows = static_cast<int>(min(32ll, a.T - row0));
    // this warp's half of the G and U of columns col.. of a unit, into slot s
    auto fetch = [&](const Unit& u, int col, int s) {
      const int f = u.f0 + col + 32 * at.h, r0 = u.m0 + row_in;
      const int n = static_cast<int>(min(32ll, a.T - r0)), cols = static_cast<int>(min(32ll, a.f - f));
      uint8_t *bg = at.blocks + 2 * s * pt::BLOCK, *bu = bg + pt::BLOCK;
      const bool any = n > 0 && cols > 0;
      const uint16_t* p = any ? a.gu_in + static_cast<long long>(r0) * 2 * a.f + f : a.gu_in;
      if (a.wide) {
        pt::half_copy(bg, at.h, p, 2 * a.f, any ? n : 0, cols, lane);
        pt::half_copy(bu, at.h, any ? p + a.f : p, 2 * a.f, any ? n : 0, cols, lane);
      } else {
        pt::HalfRegs r;
        pt::half_fetch(r, p, 2 * a.f, any ? n : 0, cols, lane, false);
        pt::half_put(r, bg, at.h, lane);
        pt::half_fetch(r, p + a.f, 2 * a.f, any ? n : 0, cols, lane, false);
        pt::half_put(r, bu, at.h, lane);
      }
      pt::copies_commit();
    };
    if (!st.fetched) fetch(c, 0, st.slot);  // the first unit's
    if (!wait()) return;
#pragma unroll 1
    for (int col = 0; col < a.width; col += 64) {
      const int mine = col + 32 * at.h;
      uint8_t *bg = at.blocks + 2 * st.slot * pt::BLOCK, *bu = bg + pt::BLOCK;
      pt::copies_wait();
      // the other slot's results have been read: the next step's G and U may come there
      pt::blocks_free(at, lane);
      if (col + 64 < a.width) fetch(c, col + 64, st.slot ^ 1);
      else if (next) fetch(*next, 0, st.slot ^ 1);
      float dh[32];
      if (c.kb > 0) {
        tmem_ld_32x32b_x32(at.taddr + mine, reinterpret_cast<uint32_t*>(dh));
        tmem_ld_wait();
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) dh[j] = 0.f;
      }
      if (col + 64 >= a.width) release();
      st.slot ^= 1;
      if (rows <= 0 || c.f0 + col >= a.f) continue;
      const int f = c.f0 + mine, cols = static_cast<int>(min(32ll, a.f - f));
      uint16_t* hrow = a.h + static_cast<long long>(row0 + lane) * a.f + f;
      // eight elements at a time, from the lane's rows of G and U into the same places
      with_act(a.act, [&](auto kind) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint4* pg = reinterpret_cast<uint4*>(pt::block_word(bg, lane, 4 * at.h + j));
          uint4* pu = reinterpret_cast<uint4*>(pt::block_word(bu, lane, 4 * at.h + j));
          const uint4 wg = *pg, wu = *pu;
          uint32_t og[4], ou[4], oh[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 x = pt::unpack16<F16>(reinterpret_cast<const uint32_t*>(&wg)[k]);
            const float2 y = pt::unpack16<F16>(reinterpret_cast<const uint32_t*>(&wu)[k]);
            const float d0 = dh[8 * j + 2 * k], d1 = dh[8 * j + 2 * k + 1];
            float a0, a1;
            const float b0 = activation_grad<decltype(kind)::value>(x.x, &a0);
            const float b1 = activation_grad<decltype(kind)::value>(x.y, &a1);
            og[k] = pt::pack16<F16>(d0 * y.x * b0, d1 * y.y * b1);
            ou[k] = pt::pack16<F16>(d0 * a0, d1 * a1);
            oh[k] = pt::pack16<F16>(a0 * y.x, a1 * y.y);
          }
          *pg = make_uint4(og[0], og[1], og[2], og[3]);
          *pu = make_uint4(ou[0], ou[1], ou[2], ou[3]);
          if (a.h && lane < rows) {
            if (a.wide) {
              if (8 * j < cols) *reinterpret_cast<uint4*>(hrow + 8 * j) = make_uint4(oh[0], oh[1], oh[2], oh[3]);
            } else {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                if (8 * j + k < cols) hrow[8 * j + k] = static_cast<uint16_t>(oh[k / 2] >> (k & 1 ? 16 : 0));
            }
          }
        }
      });
      if (a.wide) {
        if (pt::blocks_full(at, lane)) {
          tma_store_3d(&m.GU, smem_u32(bg), c.f0 + col, row0, 0);
          tma_store_3d(&m.GU, smem_u32(bu), c.f0 + col, row0, 1);
          bulk_commit();
        }
      } else {
        gated_put(bg, at.h, a.gu, 2 * a.f, f, row0, rows, cols, lane);
        gated_put(bu, at.h, a.gu + a.f, 2 * a.f, f, row0, rows, cols, lane);
      }
    }
    st.fetched = next != nullptr;
  }
};

// Operands as TMA takes them, and the copies that make them so.
struct Staged {
  const void* p[2];
  int64_t pitch[2];
  size_t bytes;
  bool copy[2];
};
struct Operand {
  const void* p;
  int64_t rows, cols;
};
Staged staged(const Operand* op, void* ws) {
  Staged s = {};
  for (int i = 0; i < 2; ++i) {
    s.p[i] = op[i].p;
    s.pitch[i] = up8(op[i].cols);
    s.copy[i] = op[i].cols > 0 && (op[i].cols % 8 != 0 || reinterpret_cast<uintptr_t>(op[i].p) % 16 != 0);
    if (s.copy[i]) {
      s.p[i] = static_cast<char*>(ws) + s.bytes;
      s.bytes += up256(static_cast<size_t>(op[i].rows) * s.pitch[i] * 2);
    }
  }
  return s;
}

template <class P>
cudaError_t launch_one(const GatedCall& g, const Staged& s) {
  const bool bwd = g.bwd;
  GatedMaps m = {};
  GatedArgs a = {};
  a.gu_in = static_cast<const uint16_t*>(g.GU);
  a.h = static_cast<uint16_t*>(g.H);
  a.gu = static_cast<uint16_t*>(g.out);
  a.T = g.T;
  a.f = g.f;
  a.kb = static_cast<int>((g.d + pt::BK - 1) / pt::BK);
  a.m_tiles = static_cast<int>((g.T + 255) / 256);
  a.act = g.act;
  a.idesc = idesc_f16(g.in_kind == EK_BF16, false, false, 256, 0);
  a.timeout_ns = g.timeout_ns;
  a.status = g.status;
  // whole tiles while they occupy more than half of the pairs, narrower ones below
  a.width = bwd ? 256 : 128;
  auto tiles = [&](int w) { return a.m_tiles * ((g.f + w - 1) / w); };
  while (a.width > 64 && tiles(a.width) <= g.num_sms / 4) a.width /= 2;
  a.units = static_cast<int>(tiles(a.width));
  const uint64_t f = g.f, T = g.T, d = g.d;
  a.wide = g.f % 8 == 0 && reinterpret_cast<uintptr_t>(g.H) % 16 == 0 && reinterpret_cast<uintptr_t>(g.out) % 16 == 0 &&
           reinterpret_cast<uintptr_t>(g.GU) % 16 == 0;
  bool ok = true;
  if (d > 0) {
    const uint64_t pa = s.pitch[0] * 2, pb = s.pitch[1] * 2;
    ok = encode_tmap_3d(&m.A, s.p[0], g.in_kind, d, T, 1, pa, 0, 64, 128, 128);
    ok = ok && (bwd ? encode_tmap_3d(&m.B, s.p[1], g.in_kind, f, d, 1, pb, 0, 64, 64, 128)
                    : encode_tmap_3d(&m.B, s.p[1], g.in_kind, d, f, 2, pb, f * pb, 64, a.width, 128));
  }
  if (a.wide && g.H) ok = ok && encode_tmap_3d(&m.H, g.H, g.in_kind, f, T, 1, f * 2, 0, 64, 32, 128);
  if (a.wide && g.out) ok = ok && encode_tmap_3d(&m.GU, g.out, g.in_kind, f, T, 2, 4 * f, 2 * f, 64, 32, 128);
  if (!ok) return cudaErrorInvalidValue;
  return pt::pair_launch<P>(m, a, g.num_sms, g.stream);
}

void operands(bool bwd, const void* A, const void* W, int64_t T, int64_t f, int64_t d, Operand* op) {
  op[0] = {A, T, d};
  op[1] = bwd ? Operand{W, d, f} : Operand{W, 2 * f, d};
}

}  // namespace

size_t gated_ws_bytes(bool bwd, int64_t T, int64_t f, int64_t d, bool any_base, int) {
  if (T <= 0 || f <= 0 || d <= 0) return 0;
  Operand op[2];
  operands(bwd, nullptr, nullptr, T, f, d, op);
  if (any_base)
    for (Operand& o : op) o.p = reinterpret_cast<const void*>(2);
  return staged(op, nullptr).bytes;
}

cudaError_t gated_launch(const GatedCall& g, size_t* need) {
  Operand op[2];
  operands(g.bwd, g.A, g.W, g.T, g.f, g.d, op);
  const Staged s = staged(op, g.ws);
  *need = s.bytes;
  if (s.bytes > 0 && (g.ws == nullptr || g.ws_bytes < s.bytes || reinterpret_cast<uintptr_t>(g.ws) % 16))
    return cudaSuccess;
  *need = 0;
  if (s.bytes > 0) {
    PitchCopy copy[2] = {};
    int64_t words = 0;
    for (int i = 0; i < 2; ++i)
      if (s.copy[i]) {
        copy[i] = {static_cast<const uint16_t*>(op[i].p), static_cast<uint16_t*>(const_cast<void*>(s.p[i])),
                   static_cast<long long>(op[i].rows), static_cast<int>(op[i].cols), static_cast<int>(s.pitch[i])};
        words += op[i].rows * (s.pitch[i] / 8);
      }
    int64_t grid = (words + 255) / 256;
    if (grid > 8 * g.num_sms) grid = 8 * g.num_sms;
    const cudaError_t e = launch_k(pitch_copy_kernel, dim3(static_cast<unsigned>(grid)), dim3(256), 0, g.stream, copy[0], copy[1]);
    if (e != cudaSuccess) return e;
  }
  if (g.T <= GATED_FEW && g.d > 0) {
    *g.path = "few rows";
    const GatedFew f = {g.bwd, s.p[0], s.p[1], g.GU, g.H, g.out, g.T, g.f, g.d, s.pitch[0], s.pitch[1], g.act, g.in_kind, g.num_sms,
                        g.status, g.timeout_ns, g.stream};
    return gated_few_launch(f);
  }
  *g.path = "pairs";
  if (g.in_kind == EK_F16) return g.bwd ? launch_one<GatedBwd<true>>(g, s) : launch_one<GatedFwd<true>>(g, s);
  return g.bwd ? launch_one<GatedBwd<false>>(g, s) : launch_one<GatedFwd<false>>(g, s);
}

}  // namespace tg
