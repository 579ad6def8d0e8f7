// The norm of every query and key head with the rotation by position in the
// same pass, forward and backward.
//
// Per head row x of D values, with a weight and a scale for the queries and
// another for the keys:
//     n = x rstd, rstd = 1 / sqrt(mean(x^2) + eps),   z = scale w n
//     y = R(pos) z: F pairs of z's first 2 F values turned by pos * freq[i]
//         (y1, y2) = (z1 c - z2 s, z2 c + z1 s), c = cos, s = sin
//     pairs (i, i + F) ("halves") or (2 i, 2 i + 1) ("neighbours")
// and backward with g = scale R(-pos) dy:
//     dw = sum over rows of g n,  t = g w,  dx = rstd (t - n mean(t n)).
//
// A few operations per element, so the kernels are laid out for HBM: 16-byte
// pieces, every tensor read and written once.  A row lies on L lanes of eight
// values; the other half of a pair of halves comes from another lane.  A wave
// takes whole tokens, so that a lane forms its angles' cosines and sines once
// for all the heads of the token.
//
// An angle far out loses its fraction in 32 bits (2^18 radians have steps of
// 2^-5), so pos * freq / (2 pi) is formed and reduced to a fraction of a turn
// in 64.
#pragma once
#include "gdn_norm.hpp"

namespace sfgdn {

constexpr int ROT_THREADS = 256;
constexpr int ROT_WAVES = ROT_THREADS / 64;

// Eight cosines and sines of a lane: for columns c .. c+7 of a row.
// NB (neighbours): columns 2i, 2i+1 share an angle.
template <bool NB>
__device__ __forceinline__ void lane_turns(const RotaryArgs& a, int c, long long token,
                                           float (&co)[NORM_V], float (&si)[NORM_V]) {
  const int pos = a.pos ? a.pos[token] : a.first + (int)(token % a.T);
#pragma unroll
  for (int j = 0; j < NORM_V; ++j) {
    if (NB && j % 2) {
      co[j] = co[j - 1];
      si[j] = si[j - 1];
      continue;
    }
    const int i = NB ? (c + j) / 2 : (c < a.F ? c : c - a.F) + j;
    const double turns = (double)pos * ((double)a.freq[i] * 0.15915494309189533577);
    const float f = (float)(turns - rint(turns));
    sincospif(2.f * f, &si[j], &co[j]);
  }
}

// v turned by the lane's angles (BACK: by the opposite ones).  `other`: the
// lane with the other halves of its pairs.  Lanes past the rotated columns
// (!in) keep theirs; every lane of the row calls it.
template <bool NB, bool BACK>
__device__ __forceinline__ void turn(float (&v)[NORM_V], const float (&co)[NORM_V],
                                     const float (&si)[NORM_V], bool in, bool second, int other) {
  float y[NORM_V];
#pragma unroll
  for (int j = 0; j < NORM_V; ++j) {
    const bool late = NB ? j % 2 : second;  // the second of its pair
    const float p = NB ? v[j ^ 1] : __shfl(v[j], other);
    const float s = late != BACK ? si[j] : -si[j];
    y[j] = v[j] * co[j] + p * s;
  }
#pragma unroll
  for (int j = 0; j < NORM_V; ++j) v[j] = in ? y[j] : v[j];
}

// What a lane is in a row.
struct RotLane {
  int c, grp, other;
  bool col, in, second;
};
template <int L>
__device__ __forceinline__ RotLane rot_lane(const RotaryArgs& a) {
  RotLane r;
  const int lane = lane_id();
  r.c = lane % L * NORM_V;
  r.grp = lane / L;
  r.col = r.c < a.D;
  r.in = r.c < 2 * a.F;
  r.second = r.c >= a.F;
  r.other = !r.in ? lane : r.second ? lane - a.F / NORM_V : lane + a.F / NORM_V;
  return r;
}

// Head row i of a token: its tensor (0 q, 1 k) and head there.
__device__ __forceinline__ int rot_side(const RotaryArgs& a, int& h) {
  if (h < a.H[0]) return 0;
  h -= a.H[0];
  return 1;
}

template <typename T, int L, bool NB, bool STREAM>
__global__ __launch_bounds__(ROT_THREADS) void rotary_fwd_kernel(RotaryArgs a, int split) {
  constexpr int G = 64 / L;  // rows of a wave at a time
  const RotLane r = rot_lane<L>(a);
  const float inv_d = 1.f / a.D;
  const int heads = a.H[0] + a.H[1];
  float w0[NORM_V], w1[NORM_V];
  fill8(w0, 1.f);
  fill8(w1, 1.f);
  if (a.w[0] && r.col) ld8(a.w[0] + r.c, w0);
  if (a.w[1] && r.col) ld8(a.w[1] + r.c, w1);
#pragma unroll
  for (int j = 0; j < NORM_V; ++j) {
    w0[j] *= a.scale[0];
    w1[j] *= a.scale[1];
  }
  // work units: a token's heads, or `split` shares of them
  const long long units = a.N * split, step = (long long)gridDim.x * ROT_WAVES;
  const int share = (heads + G * split - 1) / (G * split) * G;
  for (long long u = (long long)blockIdx.x * ROT_WAVES + wave_id(); u < units; u += step) {
    const long long n = u / split;
    const int h0 = (int)(u - n * split) * share, h1 = min(heads, h0 + share);
    float co[NORM_V], si[NORM_V];
    if (r.in) lane_turns<NB>(a, r.c, n, co, si);
    for (int hb = h0; hb < h1; hb += G) {
      int h = hb + r.grp;
      const bool live = h < h1 && r.col;
      const int side = h < h1 ? rot_side(a, h) : 0;
      Raw8<T> rx;
      rx.clear();
      if (live)
        rx.template load<STREAM>(reinterpret_cast<const T*>(a.x[side]) + n * a.xs[side] + h * a.D + r.c);
      float x[NORM_V];
      rx.to(x);
      const float rstd = rstd_of(sum_lanes<L>(dot8(x, x)), inv_d, a.eps);
#pragma unroll
      for (int j = 0; j < NORM_V; ++j) x[j] *= rstd * (side ? w1[j] : w0[j]);
      turn<NB, false>(x, co, si, r.in, r.second, r.other);
      if (live)
        st8<STREAM>(reinterpret_cast<T*>(a.y[side]) + (n * a.H[side] + h) * a.D + r.c, x);
    }
  }
}

// dw of both weights stays in the lanes' registers over all of a workgroup's
// tokens; its row groups meet in LDS at the end, and a row of partial sums for
// each workgroup in norm_reduce, in a fixed order.
template <typename T, int L, bool NB, bool STREAM>
__global__ __launch_bounds__(ROT_THREADS) void rotary_bwd_kernel(RotaryArgs a) {
  constexpr int G = 64 / L;
  const RotLane r = rot_lane<L>(a);
  const float inv_d = 1.f / a.D;
  const int heads = a.H[0] + a.H[1];
  float w0[NORM_V], w1[NORM_V], dw0[NORM_V], dw1[NORM_V];
  fill8(w0, 1.f);
  fill8(w1, 1.f);
  fill8(dw0, 0.f);
  fill8(dw1, 0.f);
  if (a.w[0] && r.col) ld8(a.w[0] + r.c, w0);
  if (a.w[1] && r.col) ld8(a.w[1] + r.c, w1);
  for (long long n = (long long)blockIdx.x * ROT_WAVES + wave_id(); n < a.N;
       n += (long long)gridDim.x * ROT_WAVES) {
    float co[NORM_V], si[NORM_V];
    if (r.in) lane_turns<NB>(a, r.c, n, co, si);
    for (int hb = 0; hb < heads; hb += G) {
      int h = hb + r.grp;
      const bool row = h < heads, live = row && r.col;
      const int side = row ? rot_side(a, h) : 0;
      Raw8<T> rx, re;
      rx.clear();
      re.clear();
      if (live) {
        rx.template load<STREAM>(reinterpret_cast<const T*>(a.x[side]) + n * a.xs[side] + h * a.D + r.c);
        re.template load<STREAM>(reinterpret_cast<const T*>(a.dy[side]) + (n * a.H[side] + h) * a.D + r.c);
      }
      float x[NORM_V], g[NORM_V], t[NORM_V];
      rx.to(x);
      re.to(g);
      turn<NB, true>(g, co, si, r.in, r.second, r.other);
#pragma unroll
      for (int j = 0; j < NORM_V; ++j) {
        g[j] *= side ? a.scale[1] : a.scale[0];
        t[j] = g[j] * (side ? w1[j] : w0[j]);
      }
      float rstd = rstd_of(sum_lanes<L>(dot8(x, x)), inv_d, a.eps);
      if (!row) rstd = 0.f;  // no row: with eps = 0 it would be infinite, and dw NaN
      const float m = rstd * sum_lanes<L>(dot8(t, x)) * inv_d;
#pragma unroll
      for (int j = 0; j < NORM_V; ++j) {
        x[j] *= rstd;
        const float gn = g[j] * x[j];
        dw0[j] += side ? 0.f : gn;
        dw1[j] += side ? gn : 0.f;
        t[j] = rstd * (t[j] - x[j] * m);
      }
      if (live)
        st8<STREAM>(reinterpret_cast<T*>(a.y[side]) + (n * a.H[side] + h) * a.D + r.c, t);
    }
  }
  if (!a.dw[0] && !a.dw[1]) return;
  __shared__ float lds[ROT_THREADS * NORM_V];
  const int two = a.dw[0] && a.dw[1];
  float* out = a.part + (size_t)blockIdx.x * (1 + two) * a.D;
  if (a.dw[0]) join_groups<L, ROT_THREADS>(dw0, a.D, out, lds);
  if (a.dw[1]) join_groups<L, ROT_THREADS>(dw1, a.D, out + two * a.D, lds);
}

// Workgroups of the backward kernel, each with a row of partial sums: fixed by
// the shape, so that the sums' order is too.
constexpr int ROT_GROUPS = 512;
int rotary_groups(long long N) {
  const long long need = (N + ROT_WAVES - 1) / ROT_WAVES;
  return (int)(need < ROT_GROUPS ? need : ROT_GROUPS);
}

template <typename T, int L, bool NB, bool STREAM>
static hipError_t rotary_fwd_l(const RotaryArgs& a, hipStream_t st, Profiler* prof) {
  // few tokens: their heads spread over several waves
  const int most = (a.H[0] + a.H[1] + 64 / L - 1) / (64 / L);
  int split = 1;
  while (split < most && a.N * split * 2 <= 2048) split *= 2;
  if (split > most) split = most;
  const long long need = (a.N * split + ROT_WAVES - 1) / ROT_WAVES;
  prof_begin(prof, "rotary_fwd", st);
  hipLaunchKernelGGL((rotary_fwd_kernel<T, L, NB, STREAM>),
                     dim3((unsigned)(need < NORM_MAX_GRID ? need : NORM_MAX_GRID)),
                     dim3(ROT_THREADS), 0, st, a, split);
  prof_end(prof, st);
  return hipGetLastError();
}
template <typename T, int L, bool NB, bool STREAM>
static hipError_t rotary_bwd_l(const RotaryArgs& a, hipStream_t st, Profiler* prof) {
  const int grid = rotary_groups(a.N);
  if (grid > 0) {
    prof_begin(prof, "rotary_bwd", st);
    hipLaunchKernelGGL((rotary_bwd_kernel<T, L, NB, STREAM>), dim3(grid), dim3(ROT_THREADS), 0, st, a);
    prof_end(prof, st);
  }
  if (a.dw[0] || a.dw[1])
    norm_reduce(a.part, grid, a.dw[0] && a.dw[1] ? 2 * a.D : a.D, a.D, a.dw[0] ? a.dw[0] : a.dw[1],
                a.dw[1], st, prof);
  return hipGetLastError();
}

template <typename T, bool NB, bool STREAM>
static hipError_t rotary_nb(const RotaryArgs& a, bool bwd, hipStream_t st, Profiler* prof) {
  switch (norm_lanes(a.D)) {
#define SF_CASE(L)                                                         \
  case L:                                                                  \
    return bwd ? rotary_bwd_l<T, L, NB, STREAM>(a, st, prof)               \
               : rotary_fwd_l<T, L, NB, STREAM>(a, st, prof);
    SF_CASE(8)
    SF_CASE(16)
    SF_CASE(32)
    SF_CASE(64)
#undef SF_CASE
  }
  return hipErrorInvalidValue;
}
template <typename T>
static hipError_t rotary(const RotaryArgs& a, bool nb, bool bwd, hipStream_t st, Profiler* prof) {
  if constexpr (sizeof(T) == 2) {
    if (norm_streams(a.N * (a.H[0] + a.H[1]) * a.D, bwd ? 3 : 2))
      return nb ? rotary_nb<T, true, true>(a, bwd, st, prof) : rotary_nb<T, false, true>(a, bwd, st, prof);
  }
  return nb ? rotary_nb<T, true, false>(a, bwd, st, prof) : rotary_nb<T, false, false>(a, bwd, st, prof);
}

template <typename T>
hipError_t launch_rotary_fwd(const RotaryArgs& a, bool neighbours, hipStream_t st, Profiler* prof) {
  return rotary<T>(a, neighbours, false, st, prof);
}
template <typename T>
hipError_t launch_rotary_bwd(const RotaryArgs& a, bool neighbours, hipStream_t st, Profiler* prof) {
  return rotary<T>(a, neighbours, true, st, prof);
}
template hipError_t launch_rotary_fwd<bf16>(const RotaryArgs&, bool, hipStream_t, Profiler*);
template hipError_t launch_rotary_fwd<float>(const RotaryArgs&, bool, hipStream_t, Profiler*);
template hipError_t launch_rotary_bwd<bf16>(const RotaryArgs&, bool, hipStream_t, Profiler*);
template hipError_t launch_rotary_bwd<float>(const RotaryArgs&, bool, hipStream_t, Profiler*);

}  // namespace sfgdn
