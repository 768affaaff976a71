// norm_residual.cuh -- what the forward and backward kernels of the norms
// around a block share: eight-element loads and stores, the ring of rows in
// flight, sums over the threads of a row, the launch geometry.
//
// A team of 32..1,024 threads owns a row, thread t the 8-element groups t,
// t + team, ..; a CTA holds several teams when rows are short.  Columns stay
// with their thread from row to row.
//
// The kernels are bound by HBM, and what feeds it is bytes in flight: about
// 50 KB an SM at its latency.  Each thread copies its own groups of the team's
// next row into shared memory with cp.async while it works on the present one
// (a warp reads only what it copied itself, so the ring needs no barrier).
// Rows in registers alone left the loads waiting behind each row's two sums:
// 16,384 x 2,304 forward ran at 2.7 TB/s that way.
#pragma once
#include <initializer_list>

#include "norm_residual.h"
#include "ptx.cuh"
#include "smem_attr.h"

namespace tg {
namespace nr {

// How a kernel takes its rows.
//   FEED_RING, FEED_VEC: rows start at multiples of 16 bytes and d is a
//     multiple of 8; through the ring, or straight into registers where two
//     rows do not fit shared memory.
//   FEED_SHIFT: the same ring for any d.  Row r starts s = (r d) % 8 elements
//     into an aligned group of eight, so the row is taken as the groups it
//     touches, columns -s .. -s + 7 first; what its first and last group hold
//     of the neighbouring rows is masked off.  A CTA takes rows of one s only
//     (the rows congruent to its index modulo 8 / gcd(8, d)), so columns stay
//     with their thread here too; the weights are laid out with the same shift
//     in shared memory.
//   FEED_SCALAR: bases off 16 bytes, and rows with such a d that do not fit: element by element.
enum Feed : int { FEED_SCALAR = 0, FEED_VEC = 1, FEED_RING = 2, FEED_SHIFT = 3 };

constexpr const char* FEED_NAMES[] = {"element", "vector", "ring", "shifted ring"};

constexpr int MAX_TEAMS = 15;     // named barriers 1..15
constexpr int SMEM_BYTES = 224 * 1024;  // dynamic, beside 1 KB of the warps' slots

struct Args {
  const void *B, *H, *w_post, *w_pre, *gate, *dH_out, *dN;
  float *rstd_b, *rstd_h;
  void *H_out, *N, *dB, *dH, *dgate;
  float* part;  // backward: [CTA][3][d]
  long long T;
  int d;
  int team, teams;  // threads of a team, teams of a CTA
  int classes;      // FEED_SHIFT: 8 / gcd(8, d), otherwise 1
  float res_scale, eps;
  int gate_kind, out_kind;
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
  static constexpr int WORDS = sizeof(T) / 2;  // of 16 bytes
};
template <typename T>
__device__ __forceinline__ Pack<T> zeros() {
  Pack<T> r;
#pragma unroll
  for (int j = 0; j < 8; ++j) r.v[j] = from_f<T>(0.f);
  return r;
}

// Two FP32 operations in one instruction (the kernels would otherwise be bound
// by instruction issue before HBM).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
  return reinterpret_cast<float2&>(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return reinterpret_cast<float2&>(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return reinterpret_cast<float2&>(r);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
// elements 2i, 2i + 1
template <typename T>
__device__ __forceinline__ float2 two(const Pack<T>& p, int i) {
  return make_float2(to_f(p.v[2 * i]), to_f(p.v[2 * i + 1]));
}

// The eight columns of group v of thread t: eight in a row, from -shift on,
// when rows are taken in groups of eight.  FEED_SCALAR with another d: one from
// each of eight runs of `team` columns, so that the lanes of a warp, element by
// element, still take neighbouring columns.
template <int FEED>
struct Cols {
  int first, step;
  __device__ __forceinline__ Cols(int v, int t, int team, int d, int shift) {
    const bool row = FEED != FEED_SCALAR || (d & 7) == 0;
    first = row ? (v * team + t) * 8 - (FEED == FEED_SHIFT ? shift : 0) : v * 8 * team + t;
    step = row ? 1 : team;
  }
  __device__ __forceinline__ int operator[](int j) const { return first + j * step; }
  // FEED_SHIFT: some of the eight are not of this row
  __device__ __forceinline__ bool edge(int d) const { return FEED == FEED_SHIFT && (first < 0 || first + 8 > d); }
};

template <typename T, int FEED>
__device__ __forceinline__ Pack<T> load8(const void* base, long long row, const Cols<FEED>& c, int d) {
  Pack<T> r = zeros<T>();
  const T* p = static_cast<const T*>(base) + row * d;
  if (FEED != FEED_SCALAR) {
    if (c.first < d) {
#pragma unroll
      for (int i = 0; i < Pack<T>::WORDS; ++i)
        reinterpret_cast<uint4*>(&r)[i] = reinterpret_cast<const uint4*>(p + c.first)[i];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c[j] < d) r.v[j] = p[c[j]];
  }
  return r;
}
template <typename T, int FEED>
__device__ __forceinline__ void store8(void* base, long long row, const Cols<FEED>& c, int d, const float2* f) {
  T* p = static_cast<T*>(base) + row * d;
  Pack<T> r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    r.v[2 * j] = from_f<T>(f[j].x);
    r.v[2 * j + 1] = from_f<T>(f[j].y);
  }
  // FP32: lanes 2i and 2i + 1 exchange a word, so that a store fills whole
  // sectors: words 0 and 1 of the even lane's group, then those of the odd lane's
  const int odd = threadIdx.x & 1;
  const int even = c.first - 8 * odd;  // the even lane's first column
  uint4 got = make_uint4(0, 0, 0, 0);
  if constexpr (FEED != FEED_SCALAR && sizeof(T) == 4) {
    const uint4* x = reinterpret_cast<const uint4*>(&r);
    const uint4 give = odd ? x[0] : x[1];
    got.x = __shfl_xor_sync(~0u, give.x, 1);
    got.y = __shfl_xor_sync(~0u, give.y, 1);
    got.z = __shfl_xor_sync(~0u, give.z, 1);
    got.w = __shfl_xor_sync(~0u, give.w, 1);
  }
  const bool edge = sizeof(T) == 4 ? FEED == FEED_SHIFT && (even < 0 || even + 16 > d) : c.edge(d);
  if (FEED == FEED_SCALAR || edge) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c[j] >= 0 && c[j] < d) p[c[j]] = r.v[j];
  } else if (sizeof(T) == 2) {
    if (c.first < d) *reinterpret_cast<uint4*>(p + c.first) = *reinterpret_cast<uint4*>(&r);
  } else {
    const uint4* x = reinterpret_cast<const uint4*>(&r);
    if (even < d) *reinterpret_cast<uint4*>(p + even + 4 * odd) = odd ? got : x[0];
    if (even + 8 < d) *reinterpret_cast<uint4*>(p + even + 8 + 4 * odd) = odd ? x[1] : got;
  }
}

// ------------------------------------------------------------ ring of rows
// A row in the ring is `words` planes of 16 bytes a thread: word w of stage s
// of thread `tid` sits at ((s * words + w) * threads + tid) * 16.  A group of
// 16-bit values is one word.  A group of FP32 values is two; a lane copies
// words `lane` and `lane + 32` of its warp's 64 instead of its own two, so that
// a copy takes whole 32-byte sectors (a lane's own words are 32 bytes apart
// from the next lane's: every sector would travel twice), and reads its own two
// from the two planes: word k of the warp's 64 is word (k ^ bit 3 of k) % 32 of
// plane k / 32, an order without bank conflicts.
struct Ring {
  uint32_t base;  // shared address of this thread's word 0 of stage 0
  uint32_t word, stage;  // bytes from one word to the next, one stage to the next
};
__device__ __forceinline__ Ring ring_of(const void* smem, int words) {
  Ring r;
  r.base = smem_u32(smem) + threadIdx.x * 16;
  r.word = blockDim.x * 16;
  r.stage = r.word * words;
  return r;
}
// `bytes` of 16 (the rest becomes zeros)
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// left: elements from the row's first to the tensor's end (FEED_SHIFT: the
// last group of the last row may end beyond it)
template <typename T, int FEED>
__device__ __forceinline__ void ring_copy(const Ring& r, int stage, int& w, const void* base, long long row,
                                          const Cols<FEED>& cols, int d, int left) {
  constexpr int N = 16 / sizeof(T);
  const T* p = static_cast<const T*>(base) + row * d;
  const uint32_t at = r.base + stage * r.stage + w * r.word;
  const int c = cols.first;
  auto copy = [&](uint32_t to, int col) {
    if (FEED == FEED_SHIFT) {
      if (col > -N && col < d) copy16(to, p + col, left - col >= N ? 16 : (left - col) * static_cast<int>(sizeof(T)));
    } else if (col < d) {
      copy16(to, p + col, 16);
    }
  };
  if constexpr (sizeof(T) == 2) {
    copy(at, c);
  } else {
    const int lane = threadIdx.x & 31;
    const int c0 = c - 8 * lane + 4 * lane;  // the warp's word `lane`
    const uint32_t to = at - 16 * lane + 16 * (lane ^ ((lane >> 3) & 1));
    copy(to, c0);
    copy(to + r.word, c0 + 128);
  }
  w += Pack<T>::WORDS;
}
__device__ __forceinline__ void ring_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// this thread's copies, and (FP32 planes) the other lanes', have landed
template <int N>
__device__ __forceinline__ void ring_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
  __syncwarp();
}
__device__ __forceinline__ uint4 read16(uint32_t at) {
  uint4 x;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "r"(at)
               : "memory");
  return x;
}
// Words of columns past the row's end are never copied: they are made zeros
// once, so that reading needs no test.
__device__ __forceinline__ void ring_clear(const Ring& r, int words, int stages) {
  for (int i = 0; i < words * stages; ++i)
    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(r.base + i * r.word), "r"(0) : "memory");
  __syncthreads();
}
template <typename T, int FEED>
__device__ __forceinline__ Pack<T> ring_read(const Ring& r, int stage, int& w, const Cols<FEED>& c, int d) {
  Pack<T> v;
  const uint32_t at = r.base + stage * r.stage + w * r.word;
  uint4* x = reinterpret_cast<uint4*>(&v);
  if constexpr (sizeof(T) == 2) {
    x[0] = read16(at);
  } else {
    // words 2 lane and 2 lane + 1 of the warp's 64
    const int lane = threadIdx.x & 31, k = 2 * lane & 31, flip = (k >> 3) & 1;
    const uint32_t plane = at - 16 * lane + (lane >> 4) * r.word;
    x[0] = read16(plane + 16 * (k ^ flip));
    x[1] = read16(plane + 16 * ((k + 1) ^ flip));
  }
  if (c.edge(d)) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c[j] < 0 || c[j] >= d) v.v[j] = from_f<T>(0.f);
  }
  w += Pack<T>::WORDS;
  return v;
}

// FEED_SHIFT: `n` vectors of d values each as the CTA's threads take them,
// [n][groups a thread * team] groups of eight, zeros outside the row.
template <typename T>
__device__ __forceinline__ void lay_shifted(T* to, int which, const void* from, int groups, int d, int shift) {
  for (int i = threadIdx.x; i < groups * 8; i += blockDim.x) {
    const int c = i - shift;
    to[which * groups * 8 + i] = c >= 0 && c < d ? static_cast<const T*>(from)[c] : from_f<T>(0.f);
  }
}
template <typename T>
__device__ __forceinline__ Pack<T> read_shifted(const T* at, int which, int groups, int group) {
  return reinterpret_cast<const Pack<T>*>(at)[which * groups + group];
}

// -------------------------------------------------------- sums over a team
__device__ __forceinline__ void team_sync(int team_id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(team_id + 1), "r"(threads) : "memory");
}

// Sums over the team; every thread gets them, added in the same order.
// `slot`: shared space of this team's warps in each of two arrays of 32;
// `which` alternates between them, so one barrier a call is enough.
__device__ __forceinline__ float team_sum(float v, float* slot, int which, int team_id, int team, int t) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  const int warps = team >> 5;
  if (warps == 1) return v;
  float* s = slot + which * 32;
  if ((t & 31) == 0) s[t >> 5] = v;
  team_sync(team_id, team);
  v = (t & 31) < warps ? s[t & 31] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}
__device__ __forceinline__ float3 team_sum3(float3 v, float4* slot, int which, int team_id, int team, int t) {
  auto warp_sum = [&] {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      v.x += __shfl_xor_sync(~0u, v.x, o);
      v.y += __shfl_xor_sync(~0u, v.y, o);
      v.z += __shfl_xor_sync(~0u, v.z, o);
    }
  };
  warp_sum();
  const int warps = team >> 5;
  if (warps == 1) return v;
  float4* s = slot + which * 32;
  if ((t & 31) == 0) s[t >> 5] = make_float4(v.x, v.y, v.z, 0.f);
  team_sync(team_id, team);
  const float4 x = (t & 31) < warps ? s[t & 31] : make_float4(0.f, 0.f, 0.f, 0.f);
  v = make_float3(x.x, x.y, x.z);
  warp_sum();
  return v;
}

// The next row's lines on their way to L2 while this one is worked on (rows
// that the ring cannot take): thread t asks for line t, t + team, ..
template <typename T>
__device__ __forceinline__ void prefetch_row(const void* base, long long row, int d, int t, int team) {
  const char* p = reinterpret_cast<const char*>(static_cast<const T*>(base) + row * d);
  for (int i = t * 128; i < d * static_cast<int>(sizeof(T)); i += team * 128)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p + i) : "memory");
}

__device__ __forceinline__ void put_kind(void* p, long long i, float v, int kind) {
  if (kind == EK_F32) static_cast<float*>(p)[i] = v;
  else if (kind == EK_F16) static_cast<__half*>(p)[i] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}


// Column sums of the CTAs' partials [ctas][planes][d], a block of 32 columns per
// CTA: 32 threads a column add every 32nd partial in order, then a warp the
// 32 sums of a column (8 threads a column spent most of 8 us waiting for loads).
static __global__ void __launch_bounds__(1024) norm_cols_kernel(const float* part, int ctas, int d, int planes, int sums,
                                                                void* dw_post, void* dw_pre, void* dgate, int kind) {
  __shared__ float s[32][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  int i = blockIdx.x * 32 + x;
  pdl_wait();  // no early trigger: wide rows make more CTAs than fit at once
  float v = 0.f;
  if (i < sums * d) {
#pragma unroll 5
    for (int c = y; c < ctas; c += 32) v += part[static_cast<long long>(c) * planes * d + i];
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

// ----------------------------------------------------------------- host side
struct Geo {
  int vpt, team, teams, ctas, classes;
};
// Threads of a team with v groups a thread, and the share of their lanes at work.
inline int team_of(int64_t d, int v) {
  const int groups = static_cast<int>((d + 7) / 8);
  return ((groups + v - 1) / v + 31) / 32 * 32;
}
inline double lanes_busy(int64_t d, int v) { return static_cast<double>((d + 7) / 8) / (v * team_of(d, v)); }

// Groups a thread: `many` where rows are many (a row's two exchanges, loop and
// addresses are paid once a thread: 16,384 x 576 forward 24.6 us with 1,
// 4,096 x 5,760 75 us), 1 where each SM has a row or two (a row's latency counts),
// or where `many` leaves more than a fifth more lanes idle.
inline int groups_a_thread(int64_t T, int64_t d, int sms, int many) {
  if (T <= 2 * static_cast<int64_t>(sms) || lanes_busy(d, many) < 0.8 * lanes_busy(d, 1)) return 1;
  return many;
}

// Columns to provide threads for: a shifted row touches up to seven more.
inline int64_t width_of(int64_t d, bool shift) { return shift ? d + 7 : d; }

// Teams to fill a CTA of `threads`; CTAs that an SM holds at once (`resident`
// threads: a CTA more would run as a second wave), in whole rounds of classes.
inline Geo geometry(int64_t T, int64_t d, bool shift, int sms, int vpt, int threads, int resident) {
  Geo g;
  g.vpt = vpt;
  g.team = team_of(width_of(d, shift), vpt);
  g.classes = 1;
  if (shift)
    for (int64_t k = d; k % 8; k *= 2) g.classes *= 2;
  g.teams = threads / g.team;
  if (g.teams < 1) g.teams = 1;
  if (g.teams > MAX_TEAMS) g.teams = MAX_TEAMS;
  const int64_t rows = (T + sms - 1) / sms;  // rows of an SM
  if (g.teams > rows) g.teams = static_cast<int>(rows);
  const int per_sm = resident / (g.team * g.teams) > 1 ? resident / (g.team * g.teams) : 1;
  const int64_t most = (T + g.teams - 1) / g.teams;
  int64_t want = static_cast<int64_t>(sms) * per_sm;
  if (most < want) want = most + g.classes - 1;
  g.ctas = static_cast<int>(want < g.classes ? g.classes : want / g.classes * g.classes);
  return g;
}

inline bool aligned16(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) % 16) return false;
  return true;
}

inline Args to_args(const NormResidual& n, const Geo& g) {
  Args a = {};
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
  a.classes = g.classes;
  a.res_scale = n.res_scale;
  a.eps = n.eps;
  a.gate_kind = n.gate_kind;
  a.out_kind = n.out_kind;
  return a;
}

}  // namespace nr
}  // namespace tg
