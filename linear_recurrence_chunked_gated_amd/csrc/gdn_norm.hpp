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
// Statistics, products and weight gradients are fp32; the outputs in the
// token type are rounded once.  The forward's y is formed from h before its
// rounding.
#pragma once
#include "gdn_kernels.hpp"

namespace sfgdn {

constexpr int NORM_V = 8;  // elements per lane and piece
constexpr int NORM_THREADS = 256;
// A launch holds fewer than 2^32 threads; with up to 1024 per workgroup.
constexpr long long NORM_MAX_GRID = 1 << 21;

template <typename T>
__device__ __forceinline__ void ld8(const T* p, float (&f)[NORM_V]);
template <>
__device__ __forceinline__ void ld8<bf16>(const bf16* p, float (&f)[NORM_V]) {
  const bf16x8 x = *reinterpret_cast<const bf16x8*>(p);
#pragma unroll
  for (int i = 0; i < NORM_V; ++i) f[i] = (float)x[i];
}
template <>
__device__ __forceinline__ void ld8<float>(const float* p, float (&f)[NORM_V]) {
  const f32x4 x = *reinterpret_cast<const f32x4*>(p), y = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = x[i];
    f[4 + i] = y[i];
  }
}
__device__ __forceinline__ void st8(bf16* p, const float (&f)[NORM_V]) {
  bf16x8 x;
#pragma unroll
  for (int i = 0; i < NORM_V; ++i) x[i] = (bf16)f[i];
  *reinterpret_cast<bf16x8*>(p) = x;
}
__device__ __forceinline__ void st8(float* p, const float (&f)[NORM_V]) {
  f32x4 x, y;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = f[i];
    y[i] = f[4 + i];
  }
  *reinterpret_cast<f32x4*>(p) = x;
  *reinterpret_cast<f32x4*>(p + 4) = y;
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

__device__ __forceinline__ float rstd_of(float sum2, float n, float eps) {
  return 1.f / sqrtf(sum2 / n + eps);
}

// act(g) and its derivative
__device__ __forceinline__ float gate_act(float g, int act) {
  return act ? g / (1.f + expf(-g)) : g;
}
__device__ __forceinline__ void gate_act_d(float g, int act, float& a, float& d) {
  if (act) {
    const float s = 1.f / (1.f + expf(-g));
    a = g * s;
    d = s * (1.f + g * (1.f - s));
  } else {
    a = g;
    d = 1.f;
  }
}

// ---------------------------------------------------------------- gated norm
// Head row i (token i / H, head i % H) of a tensor with ts elements between
// token rows.
__device__ __forceinline__ size_t head_row(long long i, int H, int D, long long ts) {
  const long long n = i / H;
  return (size_t)n * ts + (size_t)(i - n * H) * D;
}

template <typename T, int L>
__global__ __launch_bounds__(NORM_THREADS) void gated_norm_fwd_kernel(GatedNormArgs a) {
  constexpr int RB = NORM_THREADS / L;  // rows per workgroup
  const int l = threadIdx.x % L, c = l * NORM_V;
  const long long M = a.N * a.H;
  float w[NORM_V];
  fill8(w, 1.f);
  if (a.w && c < a.D) ld8(a.w + c, w);
#pragma unroll
  for (int j = 0; j < NORM_V; ++j) w[j] *= a.scale;
  for (long long i0 = (long long)blockIdx.x * RB; i0 < M; i0 += (long long)gridDim.x * RB) {
    const long long i = i0 + threadIdx.x / L;
    const bool live = i < M && c < a.D;
    float x[NORM_V], g[NORM_V];
    fill8(x, 0.f);
    fill8(g, 0.f);
    if (live) {
      ld8(reinterpret_cast<const T*>(a.x) + head_row(i, a.H, a.D, a.xs) + c, x);
      if (a.gate) ld8(reinterpret_cast<const T*>(a.gate) + head_row(i, a.H, a.D, a.gs) + c, g);
    }
    const float rstd = rstd_of(sum_lanes<L>(dot8(x, x)), (float)a.D, a.eps);
    if (live) {
#pragma unroll
      for (int j = 0; j < NORM_V; ++j) {
        x[j] = x[j] * rstd * w[j];
        if (a.gate) x[j] *= gate_act(g[j], a.act);
      }
      st8(reinterpret_cast<T*>(a.y) + (size_t)i * a.D + c, x);
    }
  }
}

// Workgroups walk the rows with a fixed stride and keep their columns' weight
// gradient in registers; the row groups of a workgroup are joined in LDS.
template <typename T, int L>
__global__ __launch_bounds__(NORM_THREADS) void gated_norm_bwd_kernel(GatedNormArgs a) {
  constexpr int RB = NORM_THREADS / L;
  const int l = threadIdx.x % L, c = l * NORM_V, grp = threadIdx.x / L;
  const bool col = c < a.D;
  float w[NORM_V], dw[NORM_V];
  fill8(w, 1.f);
  fill8(dw, 0.f);
  if (a.w && col) ld8(a.w + c, w);
  const long long M = a.N * a.H;
  for (long long i0 = (long long)blockIdx.x * RB; i0 < M; i0 += (long long)gridDim.x * RB) {
    const long long i = i0 + grp;
    const bool live = i < M && col;
    float x[NORM_V], g[NORM_V], e[NORM_V];
    fill8(x, 0.f);
    fill8(g, 0.f);
    fill8(e, 0.f);
    if (live) {
      ld8(reinterpret_cast<const T*>(a.x) + head_row(i, a.H, a.D, a.xs) + c, x);
      if (a.gate) ld8(reinterpret_cast<const T*>(a.gate) + head_row(i, a.H, a.D, a.gs) + c, g);
      ld8(reinterpret_cast<const T*>(a.dy) + (size_t)i * a.D + c, e);
    }
    const float rstd = rstd_of(sum_lanes<L>(dot8(x, x)), (float)a.D, a.eps);
    float dn[NORM_V], dg[NORM_V];
#pragma unroll
    for (int j = 0; j < NORM_V; ++j) {
      float act = 1.f, dact = 0.f;
      if (a.gate) gate_act_d(g[j], a.act, act, dact);
      e[j] *= a.scale;
      x[j] *= rstd;
      dg[j] = e[j] * w[j] * x[j] * dact;
      dw[j] += e[j] * x[j] * act;
      dn[j] = e[j] * w[j] * act;
    }
    const float m = sum_lanes<L>(dot8(dn, x)) / (float)a.D;
    if (live) {
#pragma unroll
      for (int j = 0; j < NORM_V; ++j) dn[j] = rstd * (dn[j] - x[j] * m);
      st8(reinterpret_cast<T*>(a.dx) + (size_t)i * a.D + c, dn);
      if (a.gate) st8(reinterpret_cast<T*>(a.dgate) + (size_t)i * a.D + c, dg);
    }
  }
  if (!a.part) return;
  __shared__ float sum[NORM_THREADS * NORM_V];
#pragma unroll
  for (int j = 0; j < NORM_V; ++j) sum[(grp * L + l) * NORM_V + j] = dw[j];
  __syncthreads();
  for (int j = threadIdx.x; j < a.D; j += NORM_THREADS) {
    float s = 0.f;
    for (int r = 0; r < RB; ++r) s += sum[r * L * NORM_V + j];
    a.part[(size_t)blockIdx.x * a.D + j] = s;
  }
}

// out[c] = sum over p of part[p][c], in a fixed order: 32 columns and 128
// strided row sets per workgroup, joined pairwise in LDS.  np = 0 writes zeros.
constexpr int RED_COLS = 32, RED_THREADS = 1024, RED_SETS = RED_THREADS / (RED_COLS / 4);
__global__ __launch_bounds__(RED_THREADS) void norm_reduce_kernel(const float* part, int np, int C,
                                                                  float* out) {
  __shared__ f32x4 sum[RED_SETS][RED_COLS / 4];
  const int q = threadIdx.x % (RED_COLS / 4), set = threadIdx.x / (RED_COLS / 4);
  const int c = blockIdx.x * RED_COLS + q * 4;
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  if (c < C)
    for (int p = set; p < np; p += RED_SETS)
      s += *reinterpret_cast<const f32x4*>(part + (size_t)p * C + c);
  sum[set][q] = s;
  for (int n = RED_SETS / 2; n > 0; n /= 2) {
    __syncthreads();
    if (set < n) sum[set][q] += sum[set + n][q];
  }
  if (set == 0 && c < C) *reinterpret_cast<f32x4*>(out + c) = sum[0][q];
}

static void norm_reduce(const float* part, int np, int C, float* out, hipStream_t st,
                        Profiler* prof) {
  prof_begin(prof, "norm_reduce", st);
  hipLaunchKernelGGL(norm_reduce_kernel, dim3((C + RED_COLS - 1) / RED_COLS), dim3(RED_THREADS), 0,
                     st, part, np, C, out);
  prof_end(prof, st);
}

// Lanes per head row: the power of two that covers D in 8-element pieces.
static int norm_lanes(int D) {
  int L = 8;
  while (L * NORM_V < D) L *= 2;
  return L;
}

int gated_norm_groups(long long N, int H, int D) {
  const long long rb = NORM_THREADS / norm_lanes(D), need = (N * H + rb - 1) / rb;
  return (int)(need < 1024 ? need : 1024);
}

template <typename T, int L>
static hipError_t gated_fwd_l(const GatedNormArgs& a, hipStream_t st, Profiler* prof) {
  const long long rb = NORM_THREADS / L, need = (a.N * a.H + rb - 1) / rb;
  prof_begin(prof, "gated_norm_fwd", st);
  hipLaunchKernelGGL((gated_norm_fwd_kernel<T, L>),
                     dim3((unsigned)(need < NORM_MAX_GRID ? need : NORM_MAX_GRID)),
                     dim3(NORM_THREADS), 0, st, a);
  prof_end(prof, st);
  return hipGetLastError();
}

template <typename T, int L>
static hipError_t gated_bwd_l(const GatedNormArgs& a, hipStream_t st, Profiler* prof) {
  const int grid = gated_norm_groups(a.N, a.H, a.D);
  if (grid > 0) {
    prof_begin(prof, "gated_norm_bwd", st);
    hipLaunchKernelGGL((gated_norm_bwd_kernel<T, L>), dim3(grid), dim3(NORM_THREADS), 0, st, a);
    prof_end(prof, st);
  }
  if (a.dw) norm_reduce(a.part, grid, a.D, a.dw, st, prof);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_gated_norm_fwd(const GatedNormArgs& a, hipStream_t st, Profiler* prof) {
  switch (norm_lanes(a.D)) {
    case 8: return gated_fwd_l<T, 8>(a, st, prof);
    case 16: return gated_fwd_l<T, 16>(a, st, prof);
    case 32: return gated_fwd_l<T, 32>(a, st, prof);
    case 64: return gated_fwd_l<T, 64>(a, st, prof);
  }
  return hipErrorInvalidValue;
}
template <typename T>
hipError_t launch_gated_norm_bwd(const GatedNormArgs& a, hipStream_t st, Profiler* prof) {
  switch (norm_lanes(a.D)) {
    case 8: return gated_bwd_l<T, 8>(a, st, prof);
    case 16: return gated_bwd_l<T, 16>(a, st, prof);
    case 32: return gated_bwd_l<T, 32>(a, st, prof);
    case 64: return gated_bwd_l<T, 64>(a, st, prof);
  }
  return hipErrorInvalidValue;
}

// ------------------------------------------------------------- residual norm
// A workgroup per row, NP pieces of 8 columns per lane; LT lanes (64 .. 1024).
// Row sums go through LDS where the row spans waves.
template <int LT>
__device__ __forceinline__ float row_sum(float x, float* lds) {
  x = sum_lanes<64>(x);
  if (LT == 64) return x;
  if (lane_id() == 0) lds[wave_id()] = x;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < LT / 64; ++w) s += lds[w];
  return s;
}

template <typename T, int LT, int NP>
__global__ __launch_bounds__(LT) void residual_norm_fwd_kernel(ResidualNormArgs a) {
  __shared__ float lds[2][LT / 64];  // rows alternate, so that one barrier a row is enough
  int par = 0;
  for (long long i = blockIdx.x; i < a.N; i += gridDim.x, par ^= 1) {
    const size_t base = (size_t)i * a.C;
    float h[NP][NORM_V];
    float ss = 0.f;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int c = (p * LT + threadIdx.x) * NORM_V;
      fill8(h[p], 0.f);
      if (c < a.C) {
        ld8(reinterpret_cast<const T*>(a.x) + base + c, h[p]);
        if (a.r) {
          float r[NORM_V], s[NORM_V];
          ld8(reinterpret_cast<const T*>(a.r) + base + c, r);
          fill8(s, 1.f);
          if (a.s) ld8(a.s + c, s);
#pragma unroll
          for (int j = 0; j < NORM_V; ++j) h[p][j] += a.scale * s[j] * r[j];
          st8(reinterpret_cast<T*>(a.h) + base + c, h[p]);
        }
      }
      ss += dot8(h[p], h[p]);
    }
    const float rstd = rstd_of(row_sum<LT>(ss, lds[par]), (float)a.C, a.eps);
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int c = (p * LT + threadIdx.x) * NORM_V;
      if (c < a.C) {
        float w[NORM_V];
        fill8(w, 1.f);
        if (a.w) ld8(a.w + c, w);
#pragma unroll
        for (int j = 0; j < NORM_V; ++j) h[p][j] *= rstd * w[j];
        st8(reinterpret_cast<T*>(a.y) + base + c, h[p]);
      }
    }
  }
}

template <typename T, int LT, int NP>
__global__ __launch_bounds__(LT) void residual_norm_bwd_kernel(ResidualNormArgs a) {
  __shared__ float lds[4][LT / 64];
  float w[NP][NORM_V], f[NP][NORM_V], dw[NP][NORM_V], ds[NP][NORM_V];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int c = (p * LT + threadIdx.x) * NORM_V;
    fill8(w[p], 1.f);
    fill8(f[p], 1.f);
    fill8(dw[p], 0.f);
    fill8(ds[p], 0.f);
    if (c < a.C) {
      if (a.w) ld8(a.w + c, w[p]);
      if (a.s) ld8(a.s + c, f[p]);
    }
#pragma unroll
    for (int j = 0; j < NORM_V; ++j) f[p][j] *= a.scale;
  }
  int par = 0;
  for (long long i = blockIdx.x; i < a.N; i += gridDim.x, par ^= 2) {
    const size_t base = (size_t)i * a.C;
    float h[NP][NORM_V], dy[NP][NORM_V];
    float ss = 0.f;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int c = (p * LT + threadIdx.x) * NORM_V;
      fill8(h[p], 0.f);
      fill8(dy[p], 0.f);
      if (c < a.C) {
        ld8(reinterpret_cast<const T*>(a.x) + base + c, h[p]);
        ld8(reinterpret_cast<const T*>(a.dy) + base + c, dy[p]);
      }
      ss += dot8(h[p], h[p]);
    }
    const float rstd = rstd_of(row_sum<LT>(ss, lds[par]), (float)a.C, a.eps);
    float gn = 0.f;
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int j = 0; j < NORM_V; ++j) {
        h[p][j] *= rstd;
        dw[p][j] += dy[p][j] * h[p][j];
        dy[p][j] *= w[p][j];
        gn += dy[p][j] * h[p][j];
      }
    const float m = row_sum<LT>(gn, lds[par + 1]) / (float)a.C;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int c = (p * LT + threadIdx.x) * NORM_V;
      if (c < a.C) {
        float dx[NORM_V];
        fill8(dx, 0.f);
        if (a.dh) ld8(reinterpret_cast<const T*>(a.dh) + base + c, dx);
#pragma unroll
        for (int j = 0; j < NORM_V; ++j) dx[j] += rstd * (dy[p][j] - h[p][j] * m);
        st8(reinterpret_cast<T*>(a.dx) + base + c, dx);
        if (a.ds) {
          float r[NORM_V];
          ld8(reinterpret_cast<const T*>(a.r) + base + c, r);
#pragma unroll
          for (int j = 0; j < NORM_V; ++j) ds[p][j] += dx[j] * r[j];
        }
        if (a.dr) {
#pragma unroll
          for (int j = 0; j < NORM_V; ++j) dx[j] *= f[p][j];
          st8(reinterpret_cast<T*>(a.dr) + base + c, dx);
        }
      }
    }
  }
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int c = (p * LT + threadIdx.x) * NORM_V;
    if (c < a.C) {
      float* part = a.part + (size_t)blockIdx.x * a.C + c;
      if (a.dw) {
        st8(part, dw[p]);
        part += (size_t)gridDim.x * a.C;
      }
      if (a.ds) {
#pragma unroll
        for (int j = 0; j < NORM_V; ++j) ds[p][j] *= a.scale;
        st8(part, ds[p]);
      }
    }
  }
}

int residual_norm_groups(long long N, int C) { return (int)(N < 1024 ? N : 1024); }

template <typename T, int LT, int NP>
static hipError_t residual_fwd_l(const ResidualNormArgs& a, hipStream_t st, Profiler* prof) {
  prof_begin(prof, "residual_norm_fwd", st);
  hipLaunchKernelGGL((residual_norm_fwd_kernel<T, LT, NP>), dim3((unsigned)(a.N < NORM_MAX_GRID ? a.N : NORM_MAX_GRID)),
                     dim3(LT), 0, st, a);
  prof_end(prof, st);
  return hipGetLastError();
}

template <typename T, int LT, int NP>
static hipError_t residual_bwd_l(const ResidualNormArgs& a, hipStream_t st, Profiler* prof) {
  const int grid = residual_norm_groups(a.N, a.C);
  if (grid > 0) {
    prof_begin(prof, "residual_norm_bwd", st);
    hipLaunchKernelGGL((residual_norm_bwd_kernel<T, LT, NP>), dim3(grid), dim3(LT), 0, st, a);
    prof_end(prof, st);
  }
  if (a.dw) norm_reduce(a.part, grid, a.C, a.dw, st, prof);
  if (a.ds) norm_reduce(a.part + (a.dw ? (size_t)grid * a.C : 0), grid, a.C, a.ds, st, prof);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_residual_norm_fwd(const ResidualNormArgs& a, hipStream_t st, Profiler* prof) {
  if (a.C <= 512) return residual_fwd_l<T, 64, 1>(a, st, prof);
  if (a.C <= 2048) return residual_fwd_l<T, 256, 1>(a, st, prof);
  if (a.C <= 4096) return residual_fwd_l<T, 512, 1>(a, st, prof);
  if (a.C <= 8192) return residual_fwd_l<T, 1024, 1>(a, st, prof);
  return residual_fwd_l<T, 1024, 2>(a, st, prof);
}
template <typename T>
hipError_t launch_residual_norm_bwd(const ResidualNormArgs& a, hipStream_t st, Profiler* prof) {
  if (a.C <= 512) return residual_bwd_l<T, 64, 1>(a, st, prof);
  if (a.C <= 2048) return residual_bwd_l<T, 256, 1>(a, st, prof);
  if (a.C <= 4096) return residual_bwd_l<T, 512, 1>(a, st, prof);
  if (a.C <= 8192) return residual_bwd_l<T, 1024, 1>(a, st, prof);
  return residual_bwd_l<T, 1024, 2>(a, st, prof);
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
