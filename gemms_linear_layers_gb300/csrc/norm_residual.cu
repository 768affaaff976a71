// norm_residual.cu -- the norm after a block, its gate, the residual sum and
// the norm before the next block, in one pass over the rows; and its backward.
//
//   u  = B rstd_b w_post             rstd_b = (mean_c B^2 + eps)^-1/2
//   H' = res_scale H + gate u
//   N  = H' rstd_h w_pre             rstd_h = (mean_c H'^2 + eps)^-1/2
// Backward, for dH' and dN (means over the row):
//   hn = H' rstd_h, g1 = dN w_pre,  dh = dH' + rstd_h (g1 - hn mean(g1 hn))
//   bn = B rstd_b,  du = gate dh,   g2 = du w_post
//   dB = rstd_b (g2 - bn mean(g2 bn)),  dH = res_scale dh
//   dw_pre = sum_t dN hn,  dw_post = sum_t du bn,  dgate = dh bn w_post summed
//   over what the gate was broadcast along
// All arithmetic in FP32; every output is rounded once.  N is taken from the
// unrounded H'; the backward takes the stored H'.
//
// Bound by HBM: forward reads 2 (3 with an element-wise gate) and writes 2
// values an element, backward reads 4 (5) and writes 2 (3).
//
// A team of 32..512 threads owns a row, thread t the 8-element groups t,
// t + team, ..; a CTA holds several teams when rows are short.  Columns stay
// with their thread from row to row, so the weights are loaded once and the
// column sums of the backward build up in registers; the teams of a CTA, then
// the CTAs (a second launch) are added in a fixed order.
#include <initializer_list>

#include "norm_residual.h"
#include "ptx.cuh"
#include "smem_attr.h"

namespace tg {
namespace {

constexpr int NR_MAX_TEAM = 512;
constexpr int NR_CTA = 512;  // most threads of a CTA

struct NrArgs {
  const void *B, *H, *w_post, *w_pre, *gate, *dH_out, *dN;
  float *rstd_b, *rstd_h;
  void *H_out, *N, *dB, *dH, *dgate;
  float* part;  // backward: [CTA][3][d]
  long long T;
  int d;
  int team, teams;  // threads of a team, teams of a CTA
  float res_scale, eps;
  int gate_kind;
};

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f(float v) { return v; }
template <>
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }

// Eight consecutive elements as they lie in memory.
template <typename T>
struct alignas(16) Pack {
  T v[8];
};

// c: first column; VEC: rows start at multiples of 16 bytes and d is a
// multiple of 8 (checked on the host); otherwise element by element
template <typename T, bool VEC>
__device__ __forceinline__ Pack<T> load8(const void* base, long long row, int c, int d) {
  Pack<T> r;
  const T* p = static_cast<const T*>(base) + row * d + c;
  if (VEC) {
    if (c < d) {
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
        reinterpret_cast<uint4*>(&r)[i] = reinterpret_cast<const uint4*>(p)[i];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) r.v[j] = from_f<T>(0.f);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) r.v[j] = c + j < d ? p[j] : from_f<T>(0.f);
  }
  return r;
}
template <typename T, bool VEC>
__device__ __forceinline__ void store8(void* base, long long row, int c, int d, const float* f) {
  T* p = static_cast<T*>(base) + row * d + c;
  Pack<T> r;
#pragma unroll
  for (int j = 0; j < 8; ++j) r.v[j] = from_f<T>(f[j]);
  if (VEC) {
    if (c < d) {
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
        reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<uint4*>(&r)[i];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j < d) p[j] = r.v[j];
  }
}

__device__ __forceinline__ void team_sync(int team_id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(team_id + 1), "r"(threads) : "memory");
}

// Sums of (x, y) over the team; every thread gets them, added in the same
// order.  `slot`: shared space for 2 x 16 pairs of this team; `which` alternates
// between its halves, so one barrier a call is enough.
__device__ __forceinline__ float2 team_sum(float2 v, float2* slot, int which, int team_id, int team) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(~0u, v.x, o);
    v.y += __shfl_xor_sync(~0u, v.y, o);
  }
  const int warps = team >> 5;
  if (warps == 1) return v;
  float2* s = slot + which * 16;
  const int t = threadIdx.x % team;
  if ((t & 31) == 0) s[t >> 5] = v;
  team_sync(team_id, team);
  float2 r = s[0];
  for (int i = 1; i < warps; ++i) {
    r.x += s[i].x;
    r.y += s[i].y;
  }
  return r;
}

template <typename IN, typename RES, int VPT, bool VEC>
__global__ void __launch_bounds__(NR_CTA) norm_residual_fwd_kernel(const NrArgs a) {
  __shared__ float2 slots[16][32];
  const int team_id = threadIdx.x / a.team, t = threadIdx.x % a.team;
  float2* slot = slots[team_id];
  const int d = a.d;
  const float inv_d = 1.f / static_cast<float>(d);
  pdl_wait();
  pdl_trigger();
  Pack<IN> wpost[VPT], wpre[VPT];
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = (v * a.team + t) * 8;
    wpost[v] = load8<IN, VEC>(a.w_post, 0, c, d);
    wpre[v] = load8<IN, VEC>(a.w_pre, 0, c, d);
  }
  const long long step = static_cast<long long>(gridDim.x) * a.teams;
  int which = 0;
  for (long long row = static_cast<long long>(blockIdx.x) * a.teams + team_id; row < a.T; row += step) {
    Pack<IN> b[VPT];
    Pack<RES> h[VPT];
    Pack<IN> g[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (v * a.team + t) * 8;
      b[v] = load8<IN, VEC>(a.B, row, c, d);
      h[v] = load8<RES, VEC>(a.H, row, c, d);
      if (a.gate_kind == GATE_FULL) g[v] = load8<IN, VEC>(a.gate, row, c, d);
      else if (a.gate_kind == GATE_CHANNEL) g[v] = load8<IN, VEC>(a.gate, 0, c, d);
    }
    const float gt = a.gate_kind == GATE_TOKEN ? to_f(static_cast<const IN*>(a.gate)[row]) : 1.f;
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = to_f(b[v].v[j]);
        s = fmaf(x, x, s);
      }
    s = team_sum(make_float2(s, 0.f), slot, which, team_id, a.team).x;
    which ^= 1;
    const float rb = rsqrtf(s * inv_d + a.eps);
    float x[VPT][8];
    s = 0.f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float u = to_f(b[v].v[j]) * rb * to_f(wpost[v].v[j]);
        if (a.gate_kind >= GATE_FULL || a.gate_kind == GATE_CHANNEL) u *= to_f(g[v].v[j]);
        else u *= gt;
        x[v][j] = fmaf(a.res_scale, to_f(h[v].v[j]), u);
        s = fmaf(x[v][j], x[v][j], s);
      }
      store8<RES, VEC>(a.H_out, row, (v * a.team + t) * 8, d, x[v]);
    }
    s = team_sum(make_float2(s, 0.f), slot, which, team_id, a.team).x;
    which ^= 1;
    const float rh = rsqrtf(s * inv_d + a.eps);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[v][j] *= rh * to_f(wpre[v].v[j]);
      store8<IN, VEC>(a.N, row, (v * a.team + t) * 8, d, x[v]);
    }
    if (t == 0) {
      if (a.rstd_b) a.rstd_b[row] = rb;
      if (a.rstd_h) a.rstd_h[row] = rh;
    }
  }
}

template <typename IN, typename RES, typename OUT, int VPT, bool VEC>
__global__ void __launch_bounds__(NR_CTA) norm_residual_bwd_kernel(const NrArgs a) {
  __shared__ float2 slots[16][32];
  const int team_id = threadIdx.x / a.team, t = threadIdx.x % a.team;
  float2* slot = slots[team_id];
  const int d = a.d;
  const float inv_d = 1.f / static_cast<float>(d);
  pdl_wait();
  pdl_trigger();
  float acc_post[VPT][8] = {}, acc_pre[VPT][8] = {}, acc_gate[VPT][8] = {};
  const long long step = static_cast<long long>(gridDim.x) * a.teams;
  int which = 0;
  for (long long row = static_cast<long long>(blockIdx.x) * a.teams + team_id; row < a.T; row += step) {
    Pack<IN> b[VPT], dn[VPT], g[VPT];
    Pack<RES> h[VPT], dho[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (v * a.team + t) * 8;
      h[v] = load8<RES, VEC>(a.H, row, c, d);
      dn[v] = load8<IN, VEC>(a.dN, row, c, d);
      dho[v] = load8<RES, VEC>(a.dH_out, row, c, d);
      b[v] = load8<IN, VEC>(a.B, row, c, d);
      if (a.gate_kind == GATE_FULL) g[v] = load8<IN, VEC>(a.gate, row, c, d);
      else if (a.gate_kind == GATE_CHANNEL) g[v] = load8<IN, VEC>(a.gate, 0, c, d);
    }
    const bool per_element = a.gate_kind == GATE_FULL || a.gate_kind == GATE_CHANNEL;
    const float gt = a.gate_kind == GATE_TOKEN ? to_f(static_cast<const IN*>(a.gate)[row]) : 1.f;
    const float rb = a.rstd_b[row], rh = a.rstd_h[row];
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const Pack<IN> wpre = load8<IN, VEC>(a.w_pre, 0, (v * a.team + t) * 8, d);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float p = to_f(dn[v].v[j]) * (to_f(h[v].v[j]) * rh);
        acc_pre[v][j] += p;
        s = fmaf(p, to_f(wpre.v[j]), s);
      }
    }
    s = team_sum(make_float2(s, 0.f), slot, which, team_id, a.team).x;
    which ^= 1;
    const float m1 = s * inv_d;
    float dh[VPT][8];
    float2 s2 = make_float2(0.f, 0.f);  // (sum of g2 bn, sum of dgate)
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (v * a.team + t) * 8;
      const Pack<IN> wpre = load8<IN, VEC>(a.w_pre, 0, c, d);
      const Pack<IN> wpost = load8<IN, VEC>(a.w_post, 0, c, d);
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float hn = to_f(h[v].v[j]) * rh;
        const float x = to_f(dho[v].v[j]) + rh * (to_f(dn[v].v[j]) * to_f(wpre.v[j]) - hn * m1);
        o[j] = a.res_scale * x;
        dh[v][j] = x;
      }
      store8<RES, VEC>(a.dH, row, c, d, o);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float bn = to_f(b[v].v[j]) * rb;
        const float e = dh[v][j] * bn;             // dw_post's term before the gate
        const float dg = e * to_f(wpost.v[j]);     // the gate's gradient, element by element
        const float gg = per_element ? to_f(g[v].v[j]) : gt;
        acc_post[v][j] = fmaf(gg, e, acc_post[v][j]);
        s2.x = fmaf(gg, dg, s2.x);
        s2.y += dg;
        if (a.gate_kind == GATE_CHANNEL) acc_gate[v][j] += dg;
        o[j] = dg;
      }
      if (a.gate_kind == GATE_FULL) store8<IN, VEC>(a.dgate, row, c, d, o);
    }
    s2 = team_sum(s2, slot, which, team_id, a.team);
    which ^= 1;
    if (a.gate_kind == GATE_TOKEN && t == 0) static_cast<OUT*>(a.dgate)[row] = from_f<OUT>(s2.y);
    const float m2 = s2.x * inv_d;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (v * a.team + t) * 8;
      const Pack<IN> wpost = load8<IN, VEC>(a.w_post, 0, c, d);
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float gg = per_element ? to_f(g[v].v[j]) : gt;
        const float bn = to_f(b[v].v[j]) * rb;
        o[j] = rb * (gg * dh[v][j] * to_f(wpost.v[j]) - bn * m2);
      }
      store8<IN, VEC>(a.dB, row, c, d, o);
    }
  }
  // the CTA's column sums: the teams one after the other
  extern __shared__ float col[];  // [3][d]
  const int sums = a.gate_kind == GATE_CHANNEL ? 3 : 2;
  for (int k = 0; k < a.teams; ++k) {
    __syncthreads();
    if (team_id == k) {
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int c = (v * a.team + t) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c + j < d) {
            float* p = col + c + j;
            p[0] = (k ? p[0] : 0.f) + acc_post[v][j];
            p[d] = (k ? p[d] : 0.f) + acc_pre[v][j];
            if (sums == 3) p[2 * d] = (k ? p[2 * d] : 0.f) + acc_gate[v][j];
          }
      }
    }
  }
  __syncthreads();
  float* out = a.part + static_cast<long long>(blockIdx.x) * 3 * d;
  for (int i = threadIdx.x; i < sums * d; i += blockDim.x) out[i] = col[i];
}

// Column sums of the CTAs' partials [ctas][3][d], a block of 32 columns per
// CTA: 8 threads a column add every eighth partial in order, then each other.
template <typename OUT>
__global__ void __launch_bounds__(256) norm_residual_cols_kernel(const float* part, int ctas, int d, int sums,
                                                                 void* dw_post, void* dw_pre, void* dgate) {
  __shared__ float s[8][32];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + x;
  pdl_wait();
  pdl_trigger();
  float v = 0.f;
  if (i < sums * d)
    for (int c = y; c < ctas; c += 8) v += part[static_cast<long long>(c) * 3 * d + i];
  s[y][x] = v;
  __syncthreads();
  if (y == 0 && i < sums * d) {
    for (int k = 1; k < 8; ++k) v += s[k][x];
    const int which = i / d;
    void* p = which == 0 ? dw_post : which == 1 ? dw_pre : dgate;
    static_cast<OUT*>(p)[i - which * d] = from_f<OUT>(v);
  }
}

struct Geo {
  int vpt, team, teams, ctas;
};
// Threads of a team: one per 8-element group up to 512, then 2 or 4 groups a
// thread; teams to fill CTAs of up to 512 threads (at most 15 named barriers).
Geo geometry(int64_t T, int64_t d, int sms) {
  Geo g;
  const int groups = static_cast<int>((d + 7) / 8);
  g.vpt = groups <= NR_MAX_TEAM ? 1 : groups <= 2 * NR_MAX_TEAM ? 2 : 4;
  g.team = ((groups + g.vpt - 1) / g.vpt + 31) / 32 * 32;
  g.teams = NR_CTA / g.team;
  if (g.teams > 8) g.teams = 8;
  const int64_t rows = (T + sms - 1) / sms;  // rows of an SM
  if (g.teams > rows) g.teams = static_cast<int>(rows);
  const int64_t most = (T + g.teams - 1) / g.teams;
  const int64_t want = static_cast<int64_t>(sms) * (g.vpt > 1 ? 1 : 2048 / (g.team * g.teams) > 4 ? 4 : 2);
  g.ctas = static_cast<int>(most < want ? most : want);
  return g;
}

bool vec_ok(std::initializer_list<const void*> ps, int64_t d) {
  if (d % 8) return false;
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) % 16) return false;
  return true;
}

NrArgs to_args(const NormResidual& n, const Geo& g) {
  NrArgs a = {};
  a.B = n.B;
  a.H = n.H;
  a.w_post = n.w_post;
  a.w_pre = n.w_pre;
  a.gate = n.gate;
  a.dH_out = n.dH_out;
  a.dN = n.dN;
  a.rstd_b = n.rstd_b;
  a.rstd_h = n.rstd_h;
  a.H_out = n.H_out;
  a.N = n.N;
  a.dB = n.dB;
  a.dH = n.dH;
  a.dgate = n.dgate;
  a.part = n.ws;
  a.T = n.T;
  a.d = static_cast<int>(n.d);
  a.team = g.team;
  a.teams = g.teams;
  a.res_scale = n.res_scale;
  a.eps = n.eps;
  a.gate_kind = n.gate_kind;
  return a;
}

template <typename IN, typename RES, int VPT>
cudaError_t fwd_one(const NormResidual& n, const Geo& g, bool vec) {
  const NrArgs a = to_args(n, g);
  auto kern = vec ? norm_residual_fwd_kernel<IN, RES, VPT, true> : norm_residual_fwd_kernel<IN, RES, VPT, false>;
  return launch_k(kern, dim3(g.ctas), dim3(g.team * g.teams), 0, n.stream, a);
}
template <typename IN, typename RES>
cudaError_t fwd_vpt(const NormResidual& n) {
  const Geo g = geometry(n.T, n.d, n.num_sms);
  // a gate of one value a row needs no alignment
  const bool wide_gate = n.gate_kind == GATE_FULL || n.gate_kind == GATE_CHANNEL;
  const bool vec = vec_ok({n.B, n.H, n.w_post, n.w_pre, n.H_out, n.N, wide_gate ? n.gate : nullptr}, n.d);
  switch (g.vpt) {
    case 1: return fwd_one<IN, RES, 1>(n, g, vec);
    case 2: return fwd_one<IN, RES, 2>(n, g, vec);
    default: return fwd_one<IN, RES, 4>(n, g, vec);
  }
}

template <typename IN, typename RES, typename OUT, int VPT>
cudaError_t bwd_one(const NormResidual& n, const Geo& g, bool vec) {
  const NrArgs a = to_args(n, g);
  auto kern = vec ? norm_residual_bwd_kernel<IN, RES, OUT, VPT, true> : norm_residual_bwd_kernel<IN, RES, OUT, VPT, false>;
  const size_t smem = static_cast<size_t>(3) * n.d * 4;
  cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kern), static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  e = launch_k(kern, dim3(g.ctas), dim3(g.team * g.teams), smem, n.stream, a);
  if (e != cudaSuccess) return e;
  const int sums = n.gate_kind == GATE_CHANNEL ? 3 : 2;
  return launch_k(norm_residual_cols_kernel<OUT>, dim3(static_cast<unsigned>((sums * n.d + 31) / 32)), dim3(256), 0,
                  n.stream, static_cast<const float*>(n.ws), g.ctas, static_cast<int>(n.d), sums, n.dw_post, n.dw_pre,
                  n.dgate);
}
template <typename IN, typename RES, typename OUT>
cudaError_t bwd_vpt(const NormResidual& n) {
  const Geo g = geometry(n.T, n.d, n.num_sms);
  const bool full = n.gate_kind == GATE_FULL, wide_gate = full || n.gate_kind == GATE_CHANNEL;
  const bool vec = vec_ok({n.B, n.H, n.w_post, n.w_pre, n.dH_out, n.dN, n.dB, n.dH, wide_gate ? n.gate : nullptr,
                           full ? n.dgate : nullptr},
                          n.d);
  switch (g.vpt) {
    case 1: return bwd_one<IN, RES, OUT, 1>(n, g, vec);
    case 2: return bwd_one<IN, RES, OUT, 2>(n, g, vec);
    default: return bwd_one<IN, RES, OUT, 4>(n, g, vec);
  }
}
template <typename IN>
cudaError_t bwd_types(const NormResidual& n) {
  const bool r32 = n.res_kind == EK_F32, o32 = n.out_kind == EK_F32;
  if (r32) return o32 ? bwd_vpt<IN, float, float>(n) : bwd_vpt<IN, float, IN>(n);
  return o32 ? bwd_vpt<IN, IN, float>(n) : bwd_vpt<IN, IN, IN>(n);
}

}  // namespace

cudaError_t norm_residual_fwd_launch(const NormResidual& n) {
  const bool r32 = n.res_kind == EK_F32;
  switch (n.in_kind) {
    case EK_BF16: return r32 ? fwd_vpt<__nv_bfloat16, float>(n) : fwd_vpt<__nv_bfloat16, __nv_bfloat16>(n);
    case EK_F16: return r32 ? fwd_vpt<__half, float>(n) : fwd_vpt<__half, __half>(n);
    default: return fwd_vpt<float, float>(n);
  }
}

size_t norm_residual_bwd_ws_bytes(int64_t T, int64_t d, int num_sms) {
  if (T <= 0 || d <= 0) return 0;
  return static_cast<size_t>(geometry(T, d, num_sms).ctas) * 3 * d * 4;
}

cudaError_t norm_residual_bwd_launch(const NormResidual& n) {
  switch (n.in_kind) {
    case EK_BF16: return bwd_types<__nv_bfloat16>(n);
    case EK_F16: return bwd_types<__half>(n);
    default: return bwd_vpt<float, float, float>(n);
  }
}

}  // namespace tg
