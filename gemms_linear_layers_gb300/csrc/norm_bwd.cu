// norm_bwd.cu -- backward of norm_fwd.cu, for dH' and dN (means over the row):
//   hn = H' rstd_h, g1 = dN w_pre,  dh = dH' + rstd_h (g1 - hn mean(g1 hn))
//   bn = B rstd_b,  du = gate dh,   g2 = du w_post
//   dB = rstd_b (g2 - bn mean(g2 bn)),  dH = res_scale dh
//   dw_pre = sum_t dN hn,  dw_post = sum_t du bn,  dgate = dh bn w_post summed
//   over what the gate was broadcast along
// FP32 arithmetic, every output rounded once; the stored H' is what the
// derivative is taken at.  Bound by HBM: 4 values (5 with an element-wise
// gate) read and 2 (3) written an element, in one pass: the column sums build
// up in registers (while a thread has 8 columns; in shared memory beyond, where
// 16 or 32 would spill); the teams of a CTA are added in
// shared memory, the CTAs by a second launch, all in a fixed order.  The
// second mean is taken from sums that do not wait for the first (q and e
// below), so a row costs one exchange between its threads, not two.
//
// Measured: 8,192 x 2,304 bf16 with an FP32 stream 72 us, 4.7 TB/s, with a bf16
// one 55 us, 4.1 TB/s; with a channel gate 82 and 61, with a full one 87 and 63.  What
// stands before HBM is latency: neither issue (53 % of the slots) nor DRAM (52 %) is
// saturated, counted at 76 us; waiting for loads is the first stall (3.9 an issue), then
// the teams' barriers (2.5).  16,384 x 576 39 us; 8,192 x 2,300 with a bf16 stream 77 us;
// 2,048 x 576 15 us.
#include "norm_residual.cuh"

namespace tg {
namespace {
using namespace nr;

// Groups a thread: 1 while an SM's registers hold a row's threads (16,384 x 576
// takes 42 us with 1, 60 with 3: fewer warps); `many` beyond, 3, or 2 with an
// element-wise gate (column sums in registers: 128 of them for 512 threads);
// then 4 (sums in shared memory).  One CTA an SM (few partial sums): its threads.
constexpr int bwd_many(bool el) { return el ? 2 : 3; }
constexpr int BWD_WIDEST = 4;
constexpr int bwd_threads(bool el, int vpt) { return vpt > 1 ? 512 : el ? 576 : 864; }
constexpr int BWD_DEPTH = 2;      // rows in the ring

__device__ __forceinline__ void put_kind(void* p, long long i, float v, int kind) {
  if (kind == EK_F32) static_cast<float*>(p)[i] = v;
  else if (kind == EK_F16) static_cast<__half*>(p)[i] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// EL: the gate differs from element to element (full or channel); otherwise
// it is one value a row, or 1
template <typename IN, typename RES, int VPT, int FEED, bool EL>
__global__ void __launch_bounds__(bwd_threads(EL, VPT), 1) norm_bwd_kernel(const Args a) {
  constexpr bool RING = FEED == FEED_RING || FEED == FEED_SHIFT;
  constexpr int D = BWD_DEPTH;
  extern __shared__ __align__(16) uint8_t ring_smem[];  // the ring, then the column sums [3][d]
  __shared__ float4 slots[2][32];
  const int team_id = threadIdx.x / a.team, t = threadIdx.x - team_id * a.team;
  float4* slot = slots[0] + team_id * (a.team >> 5);
  const int d = a.d;
  const float inv_d = 1.f / static_cast<float>(d);
  const bool full = EL && a.gate_kind == GATE_FULL, channel = EL && a.gate_kind == GATE_CHANNEL;
  const int ring_words = VPT * (2 * Pack<RES>::WORDS + (full ? 3 : 2) * Pack<IN>::WORDS);
  const Ring ring = ring_of(ring_smem, ring_words);
  if (RING) ring_clear(ring, ring_words, D);
  pdl_wait();
  pdl_trigger();
  // rows: those congruent to `cls` modulo a.classes, dealt to the teams of the CTAs with that class in turn
  const int cls = blockIdx.x % a.classes;
  const long long step = static_cast<long long>(gridDim.x) * a.teams;
  const long long row0 = cls + static_cast<long long>(a.classes) * ((blockIdx.x / a.classes) * a.teams + team_id);
  const int shift = FEED == FEED_SHIFT ? static_cast<int>((static_cast<long long>(cls) * d) & 7) : 0;
  auto fetch = [&](long long row, int stage) {
    if (row < a.T) {
      const long long rest = (a.T - row) * d;
      const int left = rest < (1 << 30) ? static_cast<int>(rest) : 1 << 30;
      int w = 0;
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const Cols<FEED> c(v, t, a.team, d, shift);
        ring_copy<RES, FEED>(ring, stage, w, a.H, row, c, d, left);
        ring_copy<IN, FEED>(ring, stage, w, a.B, row, c, d, left);
        if (full) ring_copy<IN, FEED>(ring, stage, w, a.gate, row, c, d, left);
        ring_copy<IN, FEED>(ring, stage, w, a.dN, row, c, d, left);
        ring_copy<RES, FEED>(ring, stage, w, a.dH_out, row, c, d, left);
      }
    }
    ring_commit();
  };
  if (RING) {
#pragma unroll
    for (int i = 0; i < D - 1; ++i) fetch(row0 + i * step, i);
  }
  // 4 groups a thread (one team a CTA): column sum k of the thread's group v, half i at (((k * VPT + v) * 2 + i) * team + t)
  constexpr bool IN_SMEM = VPT == BWD_WIDEST;
  const int ring_bytes = RING ? D * static_cast<int>(ring.stage) : 0;
  float4* accs = reinterpret_cast<float4*>(ring_smem + ring_bytes) + t;
  auto at = [&](int k, int v, int i) -> float4& { return accs[((k * VPT + v) * 2 + i) * a.team]; };
  auto add8 = [&](int k, int v, const float2* x, float by) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float4 f = at(k, v, i);
      f.x = fmaf(x[2 * i].x, by, f.x);
      f.y = fmaf(x[2 * i].y, by, f.y);
      f.z = fmaf(x[2 * i + 1].x, by, f.z);
      f.w = fmaf(x[2 * i + 1].y, by, f.w);
      at(k, v, i) = f;
    }
  };
  if (IN_SMEM) {
    for (int k = 0; k < 3; ++k)
#pragma unroll
      for (int v = 0; v < VPT; ++v) at(k, v, 0) = at(k, v, 1) = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  // FEED_SHIFT: w_post, w_pre and a channel gate, beside the ring
  IN* sw = reinterpret_cast<IN*>(ring_smem + ring_bytes);
  const int groups = VPT * a.team;
  if (FEED == FEED_SHIFT) {
    lay_shifted<IN>(sw, 0, a.w_post, groups, d, shift);
    lay_shifted<IN>(sw, 1, a.w_pre, groups, d, shift);
    if (channel) lay_shifted<IN>(sw, 2, a.gate, groups, d, shift);
    __syncthreads();
  }
  auto vector = [&](int which, const void* from, int v, const Cols<FEED>& c) {
    if constexpr (FEED == FEED_SHIFT) return read_shifted<IN>(sw, which, groups, v * a.team + t);
    else return load8<IN, FEED>(from, 0, c, d);
  };
  constexpr int KEPT = IN_SMEM ? 1 : VPT;
  float2 acc_post[KEPT][4] = {}, acc_pre[KEPT][4] = {}, acc_gate[KEPT][4] = {};
  int which = 0, stage = 0;
  // a row's scalars are loaded a row ahead too
  const bool token = !EL && a.gate_kind == GATE_TOKEN;
  float rb_next = 0.f, rh_next = 0.f, gt_next = 1.f;
  auto scalars = [&](long long row) {
    if (row < a.T) {
      rb_next = a.rstd_b[row];
      rh_next = a.rstd_h[row];
      if (token) gt_next = to_f(static_cast<const IN*>(a.gate)[row]);
    }
  };
  scalars(row0);
  for (long long row = row0; row < a.T; row += step) {
    const float rb = rb_next, rh = rh_next, gt = gt_next;
    scalars(row + step);
    if (RING) {
      fetch(row + (D - 1) * step, stage + D - 1 < D ? stage + D - 1 : stage - 1);
      ring_wait<D - 1>();
    } else if (row + step < a.T) {
      prefetch_row<RES>(a.H, row + step, d, t, a.team);
      prefetch_row<IN>(a.B, row + step, d, t, a.team);
      prefetch_row<IN>(a.dN, row + step, d, t, a.team);
      prefetch_row<RES>(a.dH_out, row + step, d, t, a.team);
      if (full) prefetch_row<IN>(a.gate, row + step, d, t, a.team);
    }
    // Group v of the thread: everything for the sums; for the results H', B
    // and the gate are taken again (all of it kept between the two would spill).
    Pack<IN> b, dn, g, wpre, wpost;
    Pack<RES> h, dho;
    auto take = [&](int v, bool sums) {
      const Cols<FEED> c(v, t, a.team, d, shift);
      if (RING) {
        int w = v * (2 * Pack<RES>::WORDS + (full ? 3 : 2) * Pack<IN>::WORDS);
        h = ring_read<RES, FEED>(ring, stage, w, c, d);
        b = ring_read<IN, FEED>(ring, stage, w, c, d);
        if (full) g = ring_read<IN, FEED>(ring, stage, w, c, d);
        if (sums) dn = ring_read<IN, FEED>(ring, stage, w, c, d);
        if (sums) dho = ring_read<RES, FEED>(ring, stage, w, c, d);
      } else {
        h = load8<RES, FEED>(a.H, row, c, d);
        b = load8<IN, FEED>(a.B, row, c, d);
        if (full) g = load8<IN, FEED>(a.gate, row, c, d);
        if (sums) dn = load8<IN, FEED>(a.dN, row, c, d);
        if (sums) dho = load8<RES, FEED>(a.dH_out, row, c, d);
      }
      if (channel) g = vector(2, a.gate, v, c);
      if (sums) wpre = vector(1, a.w_pre, v, c);
      wpost = vector(0, a.w_post, v, c);
    };
    // With g1 = dN w_pre, q = B w_post (times an element-wise gate) and
    // e = dH' + rstd_h g1:  sum of g2 bn = rstd_b (sum of q e - rstd_h^2 mean(g1 H') (sum of q H'))
    float2 s1 = both(0.f), sa = both(0.f), sb = both(0.f);
    const float2 rh2 = both(rh);
    float2 e[VPT][4];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      float2 p[4];
      take(v, true);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 x = two(h, j), n = two(dn, j), g1 = mul2(n, two(wpre, j));
        s1 = fma2(g1, x, s1);
        p[j] = mul2(n, x);  // dw_pre's term, without rstd_h
        if constexpr (!IN_SMEM) acc_pre[v][j] = fma2(p[j], rh2, acc_pre[v][j]);
        float2 q = mul2(two(b, j), two(wpost, j));
        if (EL) q = mul2(q, two(g, j));
        e[v][j] = fma2(rh2, g1, two(dho, j));
        sa = fma2(q, e[v][j], sa);
        sb = fma2(q, x, sb);
      }
      if (IN_SMEM) add8(1, v, p, rh);
    }
    const float3 sum =
        team_sum3(make_float3(s1.x + s1.y, sa.x + sa.y, sb.x + sb.y), slot, which, team_id, a.team, t);
    which ^= 1;
    const float k1 = rh * (rh * (rh * sum.x * inv_d));  // rstd_h times rstd_h times mean(g1 hn)
    const float s2 = rb * (sum.y - k1 * sum.z);
    if (token && t == 0) put_kind(a.dgate, row, s2, a.out_kind);
    // dB = (rstd_b gate) dh w_post - (rstd_b^2 mean(g2 bn)) B
    const float2 mk1 = both(-k1), c1 = both(rb * gt), c2 = both(-rb * (rb * (gt * s2 * inv_d))), sc = both(a.res_scale);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const Cols<FEED> c(v, t, a.team, d, shift);
      float2 dh[4], o[4];
      take(v, false);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        dh[j] = fma2(mk1, two(h, j), e[v][j]);
        o[j] = mul2(sc, dh[j]);
      }
      store8<RES, FEED>(a.dH, row, c, d, o);
      float2 q[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 x = two(b, j), w = two(wpost, j);
        const float2 du = EL ? mul2(dh[j], two(g, j)) : dh[j];  // without a gate of one value a row: c1 holds it
        q[j] = mul2(du, x);
        if constexpr (!IN_SMEM) acc_post[v][j] = fma2(q[j], c1, acc_post[v][j]);
        o[j] = fma2(mul2(du, w), c1, mul2(c2, x));
        if (EL) {
          dh[j] = mul2(mul2(dh[j], x), mul2(w, c1));  // the gate's gradient, element by element
          if constexpr (!IN_SMEM) {
            if (channel) acc_gate[v][j] = add2(acc_gate[v][j], dh[j]);
          }
        }
      }
      store8<IN, FEED>(a.dB, row, c, d, o);
      if (EL && full) store8<IN, FEED>(a.dgate, row, c, d, dh);
      if (IN_SMEM) {
        add8(0, v, q, rb * gt);
        if (EL && channel) add8(2, v, dh, 1.f);
      }
    }
    stage = stage + 1 < D ? stage + 1 : 0;
  }
  if (RING) ring_wait<0>();
  const int sums = channel ? 3 : 2;
  float* out = a.part + static_cast<long long>(blockIdx.x) * 3 * d;
  if (IN_SMEM) {
    for (int k = 0; k < sums; ++k)
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const Cols<FEED> c(v, t, a.team, d, shift);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float4 f = at(k, v, i);
          if (c[4 * i] < d) out[k * d + c[4 * i]] = f.x;
          if (c[4 * i + 1] < d) out[k * d + c[4 * i + 1]] = f.y;
          if (c[4 * i + 2] < d) out[k * d + c[4 * i + 2]] = f.z;
          if (c[4 * i + 3] < d) out[k * d + c[4 * i + 3]] = f.w;
        }
      }
    return;
  }
  // the CTA's column sums: the teams one after the other, in the ring's place
  float* col = reinterpret_cast<float*>(ring_smem);
  for (int k = 0; k < a.teams; ++k) {
    __syncthreads();
    if (team_id == k) {
#pragma unroll
      for (int v = 0; v < KEPT; ++v) {
        const Cols<FEED> c(v, t, a.team, d, shift);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c[j] >= 0 && c[j] < d) {
            float* p = col + c[j];
            p[0] = (k ? p[0] : 0.f) + (j & 1 ? acc_post[v][j / 2].y : acc_post[v][j / 2].x);
            p[d] = (k ? p[d] : 0.f) + (j & 1 ? acc_pre[v][j / 2].y : acc_pre[v][j / 2].x);
            if (EL && channel) p[2 * d] = (k ? p[2 * d] : 0.f) + (j & 1 ? acc_gate[v][j / 2].y : acc_gate[v][j / 2].x);
          }
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < sums * d; i += blockDim.x) out[i] = col[i];
}

// Column sums of the CTAs' partials [ctas][3][d], a block of 32 columns per
// CTA: 32 threads a column add every 32nd partial in order, then a warp the
// 32 sums of a column (8 threads a column spent most of 8 us waiting for loads).
__global__ void __launch_bounds__(1024) norm_cols_kernel(const float* part, int ctas, int d, int sums, void* dw_post,
                                                         void* dw_pre, void* dgate, int kind) {
  __shared__ float s[32][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  int i = blockIdx.x * 32 + x;
  pdl_wait();  // no early trigger: wide rows make more CTAs than fit at once
  float v = 0.f;
  if (i < sums * d) {
#pragma unroll 5
    for (int c = y; c < ctas; c += 32) v += part[static_cast<long long>(c) * 3 * d + i];
  }
  s[y][x] = v;
  __syncthreads();
  v = s[x][y];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  i = blockIdx.x * 32 + y;
  if (x == 0 && i < sums * d) {
    const int which = i / d;
    put_kind(which == 0 ? dw_post : which == 1 ? dw_pre : dgate, i - which * d, v, kind);
  }
}

Geo bwd_geometry(int64_t T, int64_t d, bool shift, int sms, bool el) {
  int vpt = 1;
  for (const int v : {bwd_many(el), BWD_WIDEST})
    if (team_of(width_of(d, shift), vpt) > bwd_threads(el, vpt)) vpt = v;
  Geo g = geometry(T, d, shift, sms, vpt, bwd_threads(el, vpt), 1);
  if (vpt == BWD_WIDEST) {  // one row at a time
    g.teams = 1;
    g.ctas = static_cast<int>(T < sms ? T : sms);
  }
  return g;
}
// Bytes of the column sums, beside the rest (4 groups a thread) or in its
// place, and of shared memory in all.
int sum_bytes(const Geo& g, int64_t d) { return static_cast<int>(g.vpt == BWD_WIDEST ? 3 * g.vpt * g.team * 32 : 3 * d * 4); }
template <typename IN, typename RES>
int bwd_smem(const NormResidual& n, const Geo& g, int feed) {
  const int words = g.vpt * (2 * Pack<RES>::WORDS + (n.gate_kind == GATE_FULL ? 3 : 2) * Pack<IN>::WORDS);
  int rows = feed == FEED_RING || feed == FEED_SHIFT ? BWD_DEPTH * words * g.team * g.teams * 16 : 0;
  if (feed == FEED_SHIFT) rows += 3 * g.vpt * g.team * 8 * static_cast<int>(sizeof(IN));
  const int sums = sum_bytes(g, n.d);
  return g.vpt == BWD_WIDEST ? rows + sums : rows > sums ? rows : sums;
}

template <typename IN, typename RES, int VPT, int FEED, bool EL>
cudaError_t bwd_one(const NormResidual& n, const Geo& g) {
  const Args a = to_args(n, g);
  *n.rows = FEED_NAMES[FEED];
  auto kern = norm_bwd_kernel<IN, RES, VPT, FEED, EL>;
  const int smem = bwd_smem<IN, RES>(n, g, FEED);
  cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  e = launch_k(kern, dim3(g.ctas), dim3(g.team * g.teams), smem, n.stream, a);
  if (e != cudaSuccess) return e;
  const int sums = n.gate_kind == GATE_CHANNEL ? 3 : 2;
  return launch_k(norm_cols_kernel, dim3(static_cast<unsigned>((sums * n.d + 31) / 32)), dim3(1024), 0, n.stream,
                  static_cast<const float*>(n.ws), g.ctas, static_cast<int>(n.d), sums, n.dw_post, n.dw_pre, n.dgate,
                  n.out_kind);
}
template <typename IN, typename RES, bool EL>
cudaError_t bwd_gate(const NormResidual& n) {
  const bool full = n.gate_kind == GATE_FULL;
  const bool words = aligned16({n.B, n.H, n.w_post, n.w_pre, n.dH_out, n.dN, n.dB, n.dH, EL ? n.gate : nullptr,
                                full ? n.dgate : nullptr});
  constexpr int MANY = bwd_many(EL);
  // through the ring, with fewer rows at once (no fewer CTAs) where they do not fit
  auto fit = [&](bool shift, int feed, Geo* g) {
    *g = bwd_geometry(n.T, n.d, shift, n.num_sms, EL);
    while (g->teams > 1 && bwd_smem<IN, RES>(n, *g, feed) > SMEM_BYTES) --g->teams;
    return words && (n.d % 8 != 0) == shift && g->vpt != BWD_WIDEST && bwd_smem<IN, RES>(n, *g, feed) <= SMEM_BYTES;
  };
  Geo g;
  if (fit(true, FEED_SHIFT, &g))
    return g.vpt == 1 ? bwd_one<IN, RES, 1, FEED_SHIFT, EL>(n, g) : bwd_one<IN, RES, MANY, FEED_SHIFT, EL>(n, g);
  if (fit(false, FEED_RING, &g))
    return g.vpt == 1 ? bwd_one<IN, RES, 1, FEED_RING, EL>(n, g) : bwd_one<IN, RES, MANY, FEED_RING, EL>(n, g);
  g = bwd_geometry(n.T, n.d, false, n.num_sms, EL);
  // aligned rows of one group a thread always fit the ring (216 KB at most)
  if (g.vpt == 1) return bwd_one<IN, RES, 1, FEED_SCALAR, EL>(n, g);
  // Wider ones that do not: words of 16 bytes all the same (4,096 x 10,240 with an FP32
  // stream 174 us, element by element 509; 4,096 x 8,192 in FP32 208 and 463).  16-bit
  // streams always fit, and FP32 ones beside an element-wise gate on 16-bit values.
  const bool vec = words && n.d % 8 == 0;
  if constexpr (sizeof(RES) == 4 && (sizeof(IN) == 4 || !EL)) {
    if (g.vpt == MANY && vec) return bwd_one<IN, RES, MANY, FEED_VEC, EL>(n, g);
  }
  if (g.vpt == MANY) return bwd_one<IN, RES, MANY, FEED_SCALAR, EL>(n, g);
  return vec ? bwd_one<IN, RES, BWD_WIDEST, FEED_VEC, EL>(n, g) : bwd_one<IN, RES, BWD_WIDEST, FEED_SCALAR, EL>(n, g);
}
template <typename IN, typename RES>
cudaError_t bwd_types(const NormResidual& n) {
  return n.gate_kind == GATE_FULL || n.gate_kind == GATE_CHANNEL ? bwd_gate<IN, RES, true>(n) : bwd_gate<IN, RES, false>(n);
}

}  // namespace

size_t norm_residual_bwd_ws_bytes(int64_t T, int64_t d, int num_sms) {
  if (T <= 0 || d <= 0) return 0;
  return static_cast<size_t>((T < num_sms ? T : num_sms) + 7) * 3 * d * 4;  // of each CTA (whole rounds of up to 8 classes)
}

cudaError_t norm_residual_bwd_launch(const NormResidual& n) {
  const bool r32 = n.res_kind == EK_F32;
  switch (n.in_kind) {
    case EK_BF16: return r32 ? bwd_types<__nv_bfloat16, float>(n) : bwd_types<__nv_bfloat16, __nv_bfloat16>(n);
    case EK_F16: return r32 ? bwd_types<__half, float>(n) : bwd_types<__half, __half>(n);
    default: return bwd_types<float, float>(n);
  }
}

}  // namespace tg
