// The norms around the recurrence, forward and backward.
//
// Gated norm, over each head's D values (after the recurrence; with neither
// gate nor weight the L2 norm of q and k before it), a = act(gate):
//     n = x rstd, rstd = 1 / sqrt(mean(x^2) + eps)
//     y = scale w n a
// and with e = scale dy:
//     dgate = e w n a',  dw = sum over rows of e n a
//     g = e w a (the gradient of n),  dx = rstd (g - n mean(g n)).
//
// Residual norm, over rows of C values, f = scale s:
//     h = x + f r,  y = w h rstd(h)
// and with n = h rstd, g = dy w:
//     dx = dh + rstd (g - n mean(g n)),  dr = f dx
//     dw = sum of dy n,  ds = scale * sum of dx r.
//
// All of it is a few operations per element, so the kernels are laid out for
// HBM: every tensor is read and written once, in 16-byte pieces, a row lives
// in the registers of a group of L lanes between its statistics and its
// output, and the backward recomputes rstd from x (h), which it reads anyway.
// Statistics, products and weight gradients are fp32 (a mean is the sum times
// the rounded 1 / n); the outputs in the token type are rounded once.  The
// forward's y is formed from h before its rounding.
//
// In bf16 they run at or above a device copy's 5.1-5.5 TB/s: gated forward of
// 32,768 tokens x 16 heads x 128 (403 MB) 63.5 us, 6.3 TB/s; gated backward of
// 62,720 x 16 x 128 (1.28 GB) 216 us and 5 for the sum of dw, 5.8 TB/s;
// residual forward of 32,768 x 2048 (537 MB) 95 us, 5.6 TB/s, backward (805
// MB) 145 us and 5, 5.4 TB/s.  In fp32, gated forward of 32,768 x 16 x 128 (805
// MB) 137 us, 5.9 TB/s, backward (1.34 GB) 252 and 5, 5.2; residual backward of
// 16,384 x 8192 (3.22 GB) 606 and 5, 5.3, of 8192 x 16,384, whose two pieces a
// lane leave 32 bytes of spilled registers, 631 and 8, 5.0.  Counted HBM bytes
// are those of the tensors.
#pragma once
#include "gdn_kernels.hpp"

namespace sfgdn {

constexpr int NORM_V = 8;  // elements per lane and piece
constexpr int NORM_THREADS = 256;
// A launch holds fewer than 2^32 threads; with up to 1024 per workgroup.
constexpr long long NORM_MAX_GRID = 1 << 21;

// Eight elements of a token tensor as they are loaded (whole words, so that
// rows read ahead cost a register per word), and to floats.  STREAM: past the
// caches.
template <typename T> struct Raw8 {
  static constexpr int W = sizeof(T) / 2;
  f32x4 r[W];
  template <bool STREAM> __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const f32x4* s = reinterpret_cast<const f32x4*>(p) + i;
      r[i] = STREAM ? __builtin_nontemporal_load(s) : *s;
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < W; ++i) r[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  __device__ __forceinline__ void to(float (&f)[NORM_V]) const {
#pragma unroll
    for (int i = 0; i < NORM_V; ++i) {
      if (W == 1) {
        const unsigned u = __float_as_uint(r[0][i / 2]);
        f[i] = __uint_as_float(i % 2 ? u & 0xffff0000u : u << 16);
      } else {
        f[i] = r[i / 4 % W][i % 4];
      }
    }
  }
};
template <bool STREAM>
__device__ __forceinline__ void st8(bf16* p, const float (&f)[NORM_V]) {
  bf16x8 x;
#pragma unroll
  for (int i = 0; i < NORM_V; ++i) x[i] = (bf16)f[i];
  if (STREAM)
    __builtin_nontemporal_store(x, reinterpret_cast<bf16x8*>(p));
  else
    *reinterpret_cast<bf16x8*>(p) = x;
}
template <bool STREAM>
__device__ __forceinline__ void st8(float* p, const float (&f)[NORM_V]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f32x4 x = {f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]};
    if (STREAM)
      __builtin_nontemporal_store(x, reinterpret_cast<f32x4*>(p) + i);
    else
      reinterpret_cast<f32x4*>(p)[i] = x;
  }
}
// eight weights
__device__ __forceinline__ void ld8(const float* p, float (&f)[NORM_V]) {
  Raw8<float> r;
  r.load<false>(p);
  r.to(f);
}
__device__ __forceinline__ void fill8(float (&f)[NORM_V], float v) {
#pragma unroll
  for (int i = 0; i < NORM_V; ++i) f[i] = v;
}
__device__ __forceinline__ float dot8(const float (&a)[NORM_V], const float (&b)[NORM_V]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NORM_V; ++i) s += a[i] * b[i];
  return s;
}

// sum over the L lanes (8 .. 64, aligned) that hold one row, in every lane
template <int L>
__device__ __forceinline__ float sum_lanes(float x) {
  x += dpp_f<0xB1>(x);
  x += dpp_f<0x4E>(x);
  x += dpp_f<0x141>(x);
  if (L >= 16) x += dpp_f<0x140>(x);
  if (L >= 32) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  }
  if (L >= 64) {
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(b[0]) + __uint_as_float(b[1]);
  }
  return x;
}

// inv_n: 1 / n, rounded
__device__ __forceinline__ float rstd_of(float sum2, float inv_n, float eps) {
  return rsqrtf(sum2 * inv_n + eps);
}

// sigmoid(g) in the hardware's exponential and reciprocal (an ulp each, and
// the rounding of the exponent, which costs |g| / 2 ulps of a small result):
// the library forms' range handling and exact division cost twice the rest of
// the norm, and the ends are right as they are (exp(-g) = inf gives 0, and what
// is below 2^-126 may become 0).
__device__ __forceinline__ float sigmoid(float g) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(g * -1.44269504088896341f));
}
// act(g) and its derivative
__device__ __forceinline__ float gate_act(float g, int act) { return act ? g * sigmoid(g) : g; }
__device__ __forceinline__ void gate_act_d(float g, int act, float& a, float& d) {
  if (act) {
    const float s = sigmoid(g);
    a = g * s;
    d = s * (1.f + g * (1.f - s));
  } else {
    a = g;
    d = 1.f;
  }
}

// ---------------------------------------------------------------- gated norm
// Offset of head row i (token i / H, head i % H) in a tensor with ts elements
// between token rows.
__device__ __forceinline__ size_t head_row(unsigned i, const GatedNormArgs& a, long long ts) {
  if (ts == (long long)a.H * a.D) return (size_t)i * a.D;
  const unsigned n = i / (unsigned)a.H;
  return (size_t)n * ts + (size_t)(i - n * a.H) * a.D;
}

template <typename T, int L, bool STREAM>
__global__ __launch_bounds__(NORM_THREADS) void gated_norm_fwd_kernel(GatedNormArgs a) {
  constexpr int RB = NORM_THREADS / L;  // rows per workgroup
  const int c = threadIdx.x % L * NORM_V, grp = threadIdx.x / L;
  const unsigned M = (unsigned)(a.N * a.H);
  const float inv_d = 1.f / a.D;
  float w[NORM_V];
  fill8(w, 1.f);
  if (a.w && c < a.D) ld8(a.w + c, w);
#pragma unroll
  for (int j = 0; j < NORM_V; ++j) w[j] *= a.scale;
  for (unsigned i0 = blockIdx.x * RB; i0 < M; i0 += gridDim.x * RB) {
    const unsigned i = i0 + grp;
    const bool live = i < M && c < a.D;
    Raw8<T> rx, rg;
    rx.clear();
    rg.clear();
    if (live) {
      rx.template load<STREAM>(reinterpret_cast<const T*>(a.x) + head_row(i, a, a.xs) + c);
      if (a.gate)
        rg.template load<STREAM>(reinterpret_cast<const T*>(a.gate) + head_row(i, a, a.gs) + c);
    }
    float x[NORM_V];
    rx.to(x);
    const float rstd = rstd_of(sum_lanes<L>(dot8(x, x)), inv_d, a.eps);
    if (live) {
      float g[NORM_V];
      rg.to(g);
#pragma unroll
      for (int j = 0; j < NORM_V; ++j) {
        x[j] = x[j] * rstd * w[j];
        if (a.gate) x[j] *= gate_act(g[j], a.act);
      }
      st8<STREAM>(reinterpret_cast<T*>(a.y) + (size_t)i * a.D + c, x);
    }
  }
}

// The row groups' sums of a workgroup, v[j] for column c + j of group grp, to
// out[0 .. cols): one after another in LDS.  Every thread calls it.
template <int L, int TB>
__device__ __forceinline__ void join_groups(const float (&v)[NORM_V], int cols, float* out,
                                            float* lds) {
  __syncthreads();
#pragma unroll
  for (int j = 0; j < NORM_V; ++j) lds[threadIdx.x * NORM_V + j] = v[j];
  __syncthreads();
  for (int j = threadIdx.x; j < cols; j += TB) {
    float s = 0.f;
    for (int r = 0; r < TB / L; ++r) s += lds[r * L * NORM_V + j];
    out[j] = s;
  }
}

// Workgroups walk the rows with a fixed stride, a turn ahead with their loads,
// and keep their columns' weight gradient in registers.  Both row sums go
// through the lanes together: with t = e w a, mean(g n) is rstd mean(t x).
template <typename T, int L, bool STREAM>
__global__ __launch_bounds__(NORM_THREADS) void gated_norm_bwd_kernel(GatedNormArgs a) {
  constexpr int RB = NORM_THREADS / L;
  const int c = threadIdx.x % L * NORM_V, grp = threadIdx.x / L;
  const bool col = c < a.D;
  const float inv_d = 1.f / a.D;
  float w[NORM_V], dw[NORM_V];
  fill8(w, 1.f);
  fill8(dw, 0.f);
  if (a.w && col) ld8(a.w + c, w);
  const unsigned M = (unsigned)(a.N * a.H);
  Raw8<T> rx, rg, re;
  auto fetch = [&](unsigned i) {
    rx.clear();
    rg.clear();
    re.clear();
    if (i < M && col) {
      rx.template load<STREAM>(reinterpret_cast<const T*>(a.x) + head_row(i, a, a.xs) + c);
      if (a.gate)
        rg.template load<STREAM>(reinterpret_cast<const T*>(a.gate) + head_row(i, a, a.gs) + c);
      re.template load<STREAM>(reinterpret_cast<const T*>(a.dy) + (size_t)i * a.D + c);
    }
  };
  fetch(blockIdx.x * RB + grp);
  for (unsigned i0 = blockIdx.x * RB; i0 < M; i0 += gridDim.x * RB) {
    const unsigned i = i0 + grp;
    float x[NORM_V], g[NORM_V], e[NORM_V];
    rx.to(x);
    rg.to(g);
    re.to(e);
    fetch(i + gridDim.x * RB);
    float t[NORM_V], dact[NORM_V];
#pragma unroll
    for (int j = 0; j < NORM_V; ++j) {
      float act = 1.f;
      dact[j] = 0.f;
      if (a.gate) gate_act_d(g[j], a.act, act, dact[j]);
      e[j] *= a.scale;
      g[j] = act;
      t[j] = e[j] * w[j] * act;
    }
    float rstd = rstd_of(sum_lanes<L>(dot8(x, x)), inv_d, a.eps);
    if (i >= M) rstd = 0.f;  // no row: with eps = 0 it would be infinite, and dw NaN
    const float m = rstd * sum_lanes<L>(dot8(t, x)) * inv_d;
    const bool live = i < M && col;
#pragma unroll
    for (int j = 0; j < NORM_V; ++j) {
      x[j] *= rstd;
      const float en = e[j] * x[j];
      dw[j] += en * g[j];
      t[j] = rstd * (t[j] - x[j] * m);
      g[j] = en * w[j] * dact[j];
    }
    if (live) {
      st8<STREAM>(reinterpret_cast<T*>(a.dx) + (size_t)i * a.D + c, t);
      if (a.gate) st8<STREAM>(reinterpret_cast<T*>(a.dgate) + (size_t)i * a.D + c, g);
    }
  }
  if (!a.part) return;
  __shared__ float lds[NORM_THREADS * NORM_V];
  join_groups<L, NORM_THREADS>(dw, a.D, a.part + (size_t)blockIdx.x * a.D, lds);
}

// Column sums of part [np][cols] in a fixed order, the first C of them to
// out, the others (of a second gradient) to out2: 32 columns and 128 strided
// row sets per workgroup, joined pairwise in LDS.  np = 0 writes zeros.
constexpr int RED_COLS = 32, RED_THREADS = 1024, RED_SETS = RED_THREADS / (RED_COLS / 4);
__global__ __launch_bounds__(RED_THREADS) void norm_reduce_kernel(const float* part, int np,
                                                                  int cols, int C, float* out,
                                                                  float* out2) {
  __shared__ f32x4 sum[RED_SETS][RED_COLS / 4];
  const int q = threadIdx.x % (RED_COLS / 4), set = threadIdx.x / (RED_COLS / 4);
  const int c = blockIdx.x * RED_COLS + q * 4;
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  if (c < cols)
    for (int p = set; p < np; p += RED_SETS)
      s += *reinterpret_cast<const f32x4*>(part + (size_t)p * cols + c);
  sum[set][q] = s;
  for (int n = RED_SETS / 2; n > 0; n /= 2) {
    __syncthreads();
    if (set < n) sum[set][q] += sum[set + n][q];
  }
  if (set == 0 && c < cols)
    *reinterpret_cast<f32x4*>(c < C ? out + c : out2 + (c - C)) = sum[0][q];
}

static void norm_reduce(const float* part, int np, int cols, int C, float* out, float* out2,
                        hipStream_t st, Profiler* prof) {
  prof_begin(prof, "norm_reduce", st);
  hipLaunchKernelGGL(norm_reduce_kernel, dim3((cols + RED_COLS - 1) / RED_COLS), dim3(RED_THREADS),
                     0, st, part, np, cols, C, out, out2);
  prof_end(prof, st);
}

// Lanes per head row: the power of two that covers D in 8-element pieces.
static int norm_lanes(int D) {
  int L = 8;
  while (L * NORM_V < D) L *= 2;
  return L;
}

// Workgroups of the backward kernels: two per compute unit.  Their loads run a
// turn ahead, so that more do not hide more, and each leaves a row of partial
// weight gradients to write and read again (gated backward of 62,720 x 16 x
// 128: 384 workgroups 233 us, 512 223, 640 249, 768 224, 1024 243; residual
// backward of 1021 x 1536 in fp32, replayed from a graph with the sum over the
// partials: 512 13.5 us, 768 15.5, 1024 15.9).
constexpr int NORM_GROUPS = 512;

int gated_norm_groups(long long N, int H, int D) {
  const long long rb = NORM_THREADS / norm_lanes(D), need = (N * H + rb - 1) / rb;
  return (int)(need < NORM_GROUPS ? need : NORM_GROUPS);
}

template <typename T, int L, bool STREAM>
static hipError_t gated_fwd_l(const GatedNormArgs& a, hipStream_t st, Profiler* prof) {
  const long long rb = NORM_THREADS / L, need = (a.N * a.H + rb - 1) / rb;
  prof_begin(prof, "gated_norm_fwd", st);
  hipLaunchKernelGGL((gated_norm_fwd_kernel<T, L, STREAM>),
                     dim3((unsigned)(need < NORM_MAX_GRID ? need : NORM_MAX_GRID)),
                     dim3(NORM_THREADS), 0, st, a);
  prof_end(prof, st);
  return hipGetLastError();
}

template <typename T, int L, bool STREAM>
static hipError_t gated_bwd_l(const GatedNormArgs& a, hipStream_t st, Profiler* prof) {
  const int grid = gated_norm_groups(a.N, a.H, a.D);
  if (grid > 0) {
    prof_begin(prof, "gated_norm_bwd", st);
    hipLaunchKernelGGL((gated_norm_bwd_kernel<T, L, STREAM>), dim3(grid), dim3(NORM_THREADS), 0, st,
                       a);
    prof_end(prof, st);
  }
  if (a.dw) norm_reduce(a.part, grid, a.D, a.D, a.dw, nullptr, st, prof);
  return hipGetLastError();
}

template <typename T, bool STREAM>
static hipError_t gated_fwd(const GatedNormArgs& a, hipStream_t st, Profiler* prof) {
  switch (norm_lanes(a.D)) {
    case 8: return gated_fwd_l<T, 8, STREAM>(a, st, prof);
    case 16: return gated_fwd_l<T, 16, STREAM>(a, st, prof);
    case 32: return gated_fwd_l<T, 32, STREAM>(a, st, prof);
    case 64: return gated_fwd_l<T, 64, STREAM>(a, st, prof);
  }
  return hipErrorInvalidValue;
}
template <typename T, bool STREAM>
static hipError_t gated_bwd(const GatedNormArgs& a, hipStream_t st, Profiler* prof) {
  switch (norm_lanes(a.D)) {
    case 8: return gated_bwd_l<T, 8, STREAM>(a, st, prof);
    case 16: return gated_bwd_l<T, 16, STREAM>(a, st, prof);
    case 32: return gated_bwd_l<T, 32, STREAM>(a, st, prof);
    case 64: return gated_bwd_l<T, 64, STREAM>(a, st, prof);
  }
  return hipErrorInvalidValue;
}

// Tensors of more than 256 MB in all cannot be in the last-level cache when
// the next operation reads them, and go past the caches (gated forward of
// 32,768 x 16 x 128: 63.5 us instead of 71.7, 6.3 TB/s; residual forward of
// 32,768 x 2048: 95 instead of 100).  Not so in fp32, where a lane's eight
// elements are two pieces and each load takes half of every line (gated
// forward of 65,536 x 8 x 128: 151 us streamed, 139 not).
static bool norm_streams(long long elements, int tensors) {
  return (size_t)elements * tensors * sizeof(bf16) > (size_t)256 << 20;
}

template <typename T>
hipError_t launch_gated_norm_fwd(const GatedNormArgs& a, hipStream_t st, Profiler* prof) {
  if constexpr (sizeof(T) == 2)
    if (norm_streams(a.N * a.H * a.D, a.gate ? 3 : 2)) return gated_fwd<T, true>(a, st, prof);
  return gated_fwd<T, false>(a, st, prof);
}
template <typename T>
hipError_t launch_gated_norm_bwd(const GatedNormArgs& a, hipStream_t st, Profiler* prof) {
  if constexpr (sizeof(T) == 2)
    if (norm_streams(a.N * a.H * a.D, a.gate ? 5 : 3)) return gated_bwd<T, true>(a, st, prof);
  return gated_bwd<T, false>(a, st, prof);
}

// ------------------------------------------------------------- residual norm
// L lanes a row, NP pieces of 8 columns per lane.  Rows of up to 512 values
// lie in 16 or 64 lanes, several to a workgroup of 256; longer ones take a
// whole workgroup of 256 to 1024 lanes, whose waves' sums meet in LDS.
template <int L>
__device__ __forceinline__ void row_sums(float& x, float& y, float (*lds)[2]) {
  x = sum_lanes<(L < 64 ? L : 64)>(x);
  y = sum_lanes<(L < 64 ? L : 64)>(y);
  if (L <= 64) return;
  if (lane_id() == 0) {
    lds[wave_id()][0] = x;
    lds[wave_id()][1] = y;
  }
  __syncthreads();
  x = y = 0.f;
#pragma unroll
  for (int w = 0; w < L / 64; ++w) {
    x += lds[w][0];
    y += lds[w][1];
  }
}

template <int L> constexpr int row_threads() { return L < NORM_THREADS ? NORM_THREADS : L; }

template <typename T, int L, int NP, bool STREAM>
__global__ __launch_bounds__(row_threads<L>()) void residual_norm_fwd_kernel(ResidualNormArgs a) {
  constexpr int RB = row_threads<L>() / L;
  __shared__ float lds[2][L / 64 + 1][2];  // rows alternate, so that one barrier a row is enough
  const int l = threadIdx.x % L, grp = threadIdx.x / L;
  const float inv_c = 1.f / a.C;
  int par = 0;
  for (long long i0 = (long long)blockIdx.x * RB; i0 < a.N;
       i0 += (long long)gridDim.x * RB, par ^= 1) {
    const long long i = i0 + grp;
    const size_t base = (size_t)i * a.C;
    Raw8<T> rx[NP], rr[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int c = (p * L + l) * NORM_V;
      rx[p].clear();
      rr[p].clear();
      if (i < a.N && c < a.C) {
        rx[p].template load<STREAM>(reinterpret_cast<const T*>(a.x) + base + c);
        if (a.r) rr[p].template load<STREAM>(reinterpret_cast<const T*>(a.r) + base + c);
      }
    }
    float h[NP][NORM_V];
    float ss = 0.f, unused = 0.f;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int c = (p * L + l) * NORM_V;
      rx[p].to(h[p]);
      if (a.r && i < a.N && c < a.C) {
        float r[NORM_V], s[NORM_V];
        rr[p].to(r);
        fill8(s, 1.f);
        if (a.s) ld8(a.s + c, s);
#pragma unroll
        for (int j = 0; j < NORM_V; ++j) h[p][j] += a.scale * s[j] * r[j];
        st8<STREAM>(reinterpret_cast<T*>(a.h) + base + c, h[p]);
      }
      ss += dot8(h[p], h[p]);
    }
    row_sums<L>(ss, unused, lds[par]);
    const float rstd = rstd_of(ss, inv_c, a.eps);
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int c = (p * L + l) * NORM_V;
      if (i < a.N && c < a.C) {
        float w[NORM_V];
        fill8(w, 1.f);
        if (a.w) ld8(a.w + c, w);
#pragma unroll
        for (int j = 0; j < NORM_V; ++j) h[p][j] *= rstd * w[j];
        st8<STREAM>(reinterpret_cast<T*>(a.y) + base + c, h[p]);
      }
    }
  }
}

// As the gated backward: fixed strides over the rows, loads a turn ahead, the
// two row sums together (t = dy w, mean(g n) = rstd mean(t h)).
template <typename T, int L, int NP, bool STREAM>
__global__ __launch_bounds__(row_threads<L>()) void residual_norm_bwd_kernel(ResidualNormArgs a) {
  constexpr int TB = row_threads<L>(), RB = TB / L;
  __shared__ float lds[2][L / 64 + 1][2];
  const int l = threadIdx.x % L, grp = threadIdx.x / L;
  const float inv_c = 1.f / a.C;
  // Two pieces' rows ahead, or their weights, would not fit the registers.
  constexpr bool AHEAD = NP == 1;
  float w[NP][NORM_V], f[NP][NORM_V], dw[NP][NORM_V], ds[NP][NORM_V];
  auto weights = [&](const float* from, int p, float (&v)[NORM_V]) {
    const int c = (p * L + l) * NORM_V;
    fill8(v, 1.f);
    if (from && c < a.C) ld8(from + c, v);
  };
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    if (AHEAD) {
      weights(a.w, p, w[p]);
      weights(a.s, p, f[p]);
    }
    fill8(dw[p], 0.f);
    fill8(ds[p], 0.f);
  }
  Raw8<T> rh[NP], ry[NP], rd[NP], rr[NP];
  auto fetch = [&](long long i) {
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int c = (p * L + l) * NORM_V;
      rh[p].clear();
      ry[p].clear();
      rd[p].clear();
      rr[p].clear();
      if (i < a.N && c < a.C) {
        const size_t at = (size_t)i * a.C + c;
        rh[p].template load<STREAM>(reinterpret_cast<const T*>(a.x) + at);
        ry[p].template load<STREAM>(reinterpret_cast<const T*>(a.dy) + at);
        if (a.dh) rd[p].template load<STREAM>(reinterpret_cast<const T*>(a.dh) + at);
        if (a.ds) rr[p].template load<STREAM>(reinterpret_cast<const T*>(a.r) + at);
      }
    }
  };
  const long long step = (long long)gridDim.x * RB;
  if (AHEAD) fetch((long long)blockIdx.x * RB + grp);
  int par = 0;
  for (long long i0 = (long long)blockIdx.x * RB; i0 < a.N; i0 += step, par ^= 1) {
    const long long i = i0 + grp;
    const size_t base = (size_t)i * a.C;
    float h[NP][NORM_V], dy[NP][NORM_V], dx[NP][NORM_V], r[NP][NORM_V];
    float ss = 0.f, gn = 0.f;
    if (!AHEAD) fetch(i);
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      rh[p].to(h[p]);
      ry[p].to(dy[p]);
      rd[p].to(dx[p]);
      rr[p].to(r[p]);
    }
    if (AHEAD) fetch(i + step);
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      ss += dot8(h[p], h[p]);
      if (!AHEAD) weights(a.w, p, w[p]);
#pragma unroll
      for (int j = 0; j < NORM_V; ++j) gn += dy[p][j] * w[p][j] * h[p][j];
    }
    row_sums<L>(ss, gn, lds[par]);
    float rstd = rstd_of(ss, inv_c, a.eps);
    if (i >= a.N) rstd = 0.f;  // no row: with eps = 0 it would be infinite, and dw NaN
    const float m = rstd * gn * inv_c;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int c = (p * L + l) * NORM_V;
#pragma unroll
      for (int j = 0; j < NORM_V; ++j) {
        h[p][j] *= rstd;
        dw[p][j] += dy[p][j] * h[p][j];
        dx[p][j] += rstd * (dy[p][j] * w[p][j] - h[p][j] * m);
        ds[p][j] += dx[p][j] * r[p][j];
      }
      if (i < a.N && c < a.C) {
        st8<STREAM>(reinterpret_cast<T*>(a.dx) + base + c, dx[p]);
        if (a.dr) {
          if (!AHEAD) weights(a.s, p, f[p]);
#pragma unroll
          for (int j = 0; j < NORM_V; ++j) dx[p][j] *= a.scale * f[p][j];
          st8<STREAM>(reinterpret_cast<T*>(a.dr) + base + c, dx[p]);
        }
      }
    }
  }
  if (!a.dw && !a.ds) return;
  float* part = a.part + (size_t)blockIdx.x * a.C * (a.dw && a.ds ? 2 : 1);
  float* part2 = part + (a.dw ? a.C : 0);
#pragma unroll
  for (int p = 0; p < NP; ++p)
#pragma unroll
    for (int j = 0; j < NORM_V; ++j) ds[p][j] *= a.scale;
  if constexpr (RB > 1) {
    __shared__ float sum[TB * NORM_V];
    if (a.dw) join_groups<L, TB>(dw[0], a.C, part, sum);
    if (a.ds) join_groups<L, TB>(ds[0], a.C, part2, sum);
  } else {
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int c = (p * L + l) * NORM_V;
      if (c < a.C) {
        if (a.dw) st8<false>(part + c, dw[p]);
        if (a.ds) st8<false>(part2 + c, ds[p]);
      }
    }
  }
}

int residual_norm_groups(long long N, int C) {
  const long long rb = C <= 128 ? 16 : C <= 512 ? 4 : 1, need = (N + rb - 1) / rb;
  // Workgroups of 512 threads and more: one per compute unit (backward of
  // 16,384 x 4096 140 us instead of 150, of 3111 x 4744 in fp32 78 instead of
  // 84, of 8192 x 8192 144 instead of 147; at 1536, 82 instead of 71).
  const int most = C > 2048 ? NORM_GROUPS / 2 : NORM_GROUPS;
  return (int)(need < most ? need : most);
}

template <typename T, int L, int NP, bool STREAM>
static hipError_t residual_fwd_l(const ResidualNormArgs& a, hipStream_t st, Profiler* prof) {
  constexpr int RB = row_threads<L>() / L;
  const long long need = (a.N + RB - 1) / RB;
  prof_begin(prof, "residual_norm_fwd", st);
  hipLaunchKernelGGL((residual_norm_fwd_kernel<T, L, NP, STREAM>),
                     dim3((unsigned)(need < NORM_MAX_GRID ? need : NORM_MAX_GRID)),
                     dim3(row_threads<L>()), 0, st, a);
  prof_end(prof, st);
  return hipGetLastError();
}

template <typename T, int L, int NP, bool STREAM>
static hipError_t residual_bwd_l(const ResidualNormArgs& a, hipStream_t st, Profiler* prof) {
  const int grid = residual_norm_groups(a.N, a.C);
  if (grid > 0) {
    prof_begin(prof, "residual_norm_bwd", st);
    hipLaunchKernelGGL((residual_norm_bwd_kernel<T, L, NP, STREAM>), dim3(grid),
                       dim3(row_threads<L>()), 0, st, a);
    prof_end(prof, st);
  }
  if (a.dw || a.ds)
    norm_reduce(a.part, grid, a.C * (a.dw && a.ds ? 2 : 1), a.C, a.dw ? a.dw : a.ds, a.ds, st, prof);
  return hipGetLastError();
}

template <typename T, bool STREAM>
static hipError_t residual_fwd(const ResidualNormArgs& a, hipStream_t st, Profiler* prof) {
  if (a.C <= 128) return residual_fwd_l<T, 16, 1, STREAM>(a, st, prof);
  if (a.C <= 512) return residual_fwd_l<T, 64, 1, STREAM>(a, st, prof);
  if (a.C <= 2048) return residual_fwd_l<T, 256, 1, STREAM>(a, st, prof);
  if (a.C <= 4096) return residual_fwd_l<T, 512, 1, STREAM>(a, st, prof);
  if (a.C <= 8192) return residual_fwd_l<T, 1024, 1, STREAM>(a, st, prof);
  return residual_fwd_l<T, 1024, 2, STREAM>(a, st, prof);
}
template <typename T, bool STREAM>
static hipError_t residual_bwd(const ResidualNormArgs& a, hipStream_t st, Profiler* prof) {
  if (a.C <= 128) return residual_bwd_l<T, 16, 1, STREAM>(a, st, prof);
  if (a.C <= 512) return residual_bwd_l<T, 64, 1, STREAM>(a, st, prof);
  if (a.C <= 2048) return residual_bwd_l<T, 256, 1, STREAM>(a, st, prof);
  if (a.C <= 4096) return residual_bwd_l<T, 512, 1, STREAM>(a, st, prof);
  if (a.C <= 8192) return residual_bwd_l<T, 1024, 1, STREAM>(a, st, prof);
  return residual_bwd_l<T, 1024, 2, STREAM>(a, st, prof);
}

template <typename T>
hipError_t launch_residual_norm_fwd(const ResidualNormArgs& a, hipStream_t st, Profiler* prof) {
  if constexpr (sizeof(T) == 2)
    if (norm_streams(a.N * a.C, a.r ? 4 : 2)) return residual_fwd<T, true>(a, st, prof);
  return residual_fwd<T, false>(a, st, prof);
}
template <typename T>
hipError_t launch_residual_norm_bwd(const ResidualNormArgs& a, hipStream_t st, Profiler* prof) {
  if constexpr (sizeof(T) == 2) {
    const int tensors = 3 + (a.dh ? 1 : 0) + (a.dr ? 1 : 0) + (a.ds ? 1 : 0);
    if (norm_streams(a.N * a.C, tensors)) return residual_bwd<T, true>(a, st, prof);
  }
  return residual_bwd<T, false>(a, st, prof);
}

template hipError_t launch_gated_norm_fwd<bf16>(const GatedNormArgs&, hipStream_t, Profiler*);
template hipError_t launch_gated_norm_fwd<float>(const GatedNormArgs&, hipStream_t, Profiler*);
template hipError_t launch_gated_norm_bwd<bf16>(const GatedNormArgs&, hipStream_t, Profiler*);
template hipError_t launch_gated_norm_bwd<float>(const GatedNormArgs&, hipStream_t, Profiler*);
template hipError_t launch_residual_norm_fwd<bf16>(const ResidualNormArgs&, hipStream_t, Profiler*);
template hipError_t launch_residual_norm_fwd<float>(const ResidualNormArgs&, hipStream_t, Profiler*);
template hipError_t launch_residual_norm_bwd<bf16>(const ResidualNormArgs&, hipStream_t, Profiler*);
template hipError_t launch_residual_norm_bwd<float>(const ResidualNormArgs&, hipStream_t, Profiler*);

}  // namespace sfgdn
