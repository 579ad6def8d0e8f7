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
//
// Measured (bf16, 16 + 16 heads of 128): forward of 32,768 tokens 99 us (5.4
// TB/s), backward of 62,720 tokens 266 us (5.8 TB/s), as fast as a copy of as
// many bytes; one token 5 to 6 us, its backward 7.5, what a launch (two) takes
// (3.2 us replayed from a graph).
#pragma once
#include "gdn_norm.hpp"

namespace sfgdn {

constexpr int ROT_THREADS = 256;
constexpr int ROT_WAVES = ROT_THREADS / 64;

// Cosines and sines of a token's F angles, one or a few per lane, to the
// wave's part of LDS: cs[0 .. F) and cs[MAX .. MAX + F).  (A lane needs eight,
// which several lanes share: formed where they are used they would cost eight
// times as much, half of the forward's arithmetic.)
constexpr int ROT_MAX = 256;
__device__ __forceinline__ void token_turns(const RotaryArgs& a, long long token, float* cs) {
  const int pos = a.pos ? a.pos[token] : a.first + (int)(token % a.T);
  // a wave's lanes go together: the compiler only has to keep the order
  __builtin_amdgcn_wave_barrier();
  for (int i = lane_id(); i < a.F; i += 64) {
    const double turns = (double)pos * ((double)a.freq[i] * 0.15915494309189533577);
    sincospif(2.f * (float)(turns - rint(turns)), &cs[ROT_MAX + i], &cs[i]);
  }
  __builtin_amdgcn_wave_barrier();
}

// What a lane is in a row of L lanes.
template <int L, bool NB> struct RotLane {
  int c, grp, other;   // first column, row of the wave, byte address of the pairs' other lane
  bool col, in, late;  // has columns, has rotated ones, the second half of its pairs
  int first;           // its first angle
  __device__ __forceinline__ explicit RotLane(const RotaryArgs& a) {
    const int lane = lane_id();
    c = lane % L * NORM_V;
    grp = lane / L;
    col = c < a.D;
    in = c < 2 * a.F;
    late = !NB && in && c >= a.F;
    other = 4 * (NB || !in ? lane : late ? lane - a.F / NORM_V : lane + a.F / NORM_V);
    first = !in ? 0 : NB ? c / 2 : late ? c - a.F : c;
  }
  // its angles' cosines and the sines that its values' partners are taken with
  __device__ __forceinline__ void angles(const float* cs, float (&co)[NORM_V], float (&si)[NORM_V],
                                         bool back) const {
#pragma unroll
    for (int j = 0; j < NORM_V; j += 4) {
      const float* p = cs + first + (NB ? j / 2 : j);
      float x[4], y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = p[NB ? e / 2 : e];
        y[e] = p[ROT_MAX + (NB ? e / 2 : e)];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        co[j + e] = in ? x[e] : 1.f;
        const bool second = NB ? e % 2 : late;
        si[j + e] = !in ? 0.f : second != back ? y[e] : -y[e];
      }
    }
  }
  __device__ __forceinline__ void turn(float (&v)[NORM_V], const float (&co)[NORM_V],
                                       const float (&si)[NORM_V]) const {
    float p[NORM_V];
#pragma unroll
    for (int j = 0; j < NORM_V; ++j)
      p[j] = NB ? v[j ^ 1]
                : __int_as_float(__builtin_amdgcn_ds_bpermute(other, __float_as_int(v[j])));
#pragma unroll
    for (int j = 0; j < NORM_V; ++j) {
      const float y = v[j] * co[j] + p[j] * si[j];
      v[j] = in ? y : v[j];  // (as it was: 0 times a value that is not finite is NaN)
    }
  }
};

// A wave takes a token: its query heads, then its key heads, 64 / L at a time,
// with the next ones' loads ahead.  `split`: heads of a token are spread over
// so many waves (few tokens).
template <typename T, int L, bool NB, bool STREAM>
__global__ __launch_bounds__(ROT_THREADS) void rotary_fwd_kernel(RotaryArgs a, int split) {
  constexpr int G = 64 / L;  // rows of a wave at a time
  __shared__ float turns[ROT_WAVES][2 * ROT_MAX];
  float* cs = turns[wave_id()];
  const RotLane<L, NB> r(a);
  const float inv_d = 1.f / a.D;
  float w[2][NORM_V];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    fill8(w[t], 1.f);
    if (a.w[t] && r.col) ld8(a.w[t] + r.c, w[t]);
#pragma unroll
    for (int j = 0; j < NORM_V; ++j) w[t][j] *= a.scale[t];
  }
  const long long units = a.N * split, step = (long long)gridDim.x * ROT_WAVES;
  for (long long u = (long long)blockIdx.x * ROT_WAVES + wave_id(); u < units; u += step) {
    const long long n = u / split;
    const int part = (int)(u - n * split) * G;
    float co[NORM_V], si[NORM_V];
    bool turned = false;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const T* x = reinterpret_cast<const T*>(a.x[t]) + n * a.xs[t] + r.c;
      T* y = reinterpret_cast<T*>(a.y[t]) + n * a.H[t] * a.D + r.c;
      Raw8<T> next;
      auto fetch = [&](int h) {
        next.clear();
        if (h < a.H[t] && r.col) next.template load<STREAM>(x + h * a.D);
      };
      if (part < a.H[t]) fetch(part + r.grp);
      if (!turned) {  // behind the first loads
        token_turns(a, n, cs);
        r.angles(cs, co, si, false);
        turned = true;
      }
      for (int hb = part; hb < a.H[t]; hb += G * split) {
        const int h = hb + r.grp;
        float v[NORM_V];
        next.to(v);
        fetch(h + G * split);
        const float rstd = rstd_of(sum_lanes<L>(dot8(v, v)), inv_d, a.eps);
#pragma unroll
        for (int j = 0; j < NORM_V; ++j) v[j] *= rstd * w[t][j];
        r.turn(v, co, si);
        if (h < a.H[t] && r.col) st8<STREAM>(y + h * a.D, v);
      }
    }
  }
}

// dw of both weights stays in the lanes' registers over all of a workgroup's
// tokens; its row groups meet in LDS at the end, and a row of partial sums for
// each workgroup in norm_reduce, in a fixed order.
template <typename T, int L, bool NB, bool STREAM>
__global__ __launch_bounds__(ROT_THREADS) void rotary_bwd_kernel(RotaryArgs a, int split) {
  constexpr int G = 64 / L;
  __shared__ float lds[ROT_THREADS * NORM_V];  // the waves' angles, then the sums
  static_assert(ROT_WAVES * 2 * ROT_MAX <= ROT_THREADS * NORM_V, "angles fit");
  float* cs = lds + wave_id() * 2 * ROT_MAX;
  const RotLane<L, NB> r(a);
  const float inv_d = 1.f / a.D;
  float w[2][NORM_V], dw[2][NORM_V];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    fill8(w[t], 1.f);
    fill8(dw[t], 0.f);
    if (a.w[t] && r.col) ld8(a.w[t] + r.c, w[t]);
  }
  const long long units = a.N * split, step = (long long)gridDim.x * ROT_WAVES;
  for (long long u = (long long)blockIdx.x * ROT_WAVES + wave_id(); u < units; u += step) {
    const long long n = u / split;
    const int part = (int)(u - n * split) * G;
    float co[NORM_V], si[NORM_V];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const T* x = reinterpret_cast<const T*>(a.x[t]) + n * a.xs[t] + r.c;
      const size_t flat = (size_t)n * a.H[t] * a.D + r.c;
      const T* dy = reinterpret_cast<const T*>(a.dy[t]) + flat;
      T* dx = reinterpret_cast<T*>(a.y[t]) + flat;
      const float scale = a.scale[t];
      Raw8<T> nx, ne;
      auto fetch = [&](int h) {
        nx.clear();
        ne.clear();
        if (h < a.H[t] && r.col) {
          nx.template load<STREAM>(x + h * a.D);
          ne.template load<STREAM>(dy + h * a.D);
        }
      };
      fetch(part + r.grp);
      if (t == 0) {  // behind the first loads
        token_turns(a, n, cs);
        r.angles(cs, co, si, true);
      }
      for (int hb = part; hb < a.H[t]; hb += G * split) {
        const int h = hb + r.grp;
        float v[NORM_V], g[NORM_V], e[NORM_V];
        nx.to(v);
        ne.to(g);
        fetch(h + G * split);
        r.turn(g, co, si);
#pragma unroll
        for (int j = 0; j < NORM_V; ++j) {
          g[j] *= scale;
          e[j] = g[j] * w[t][j];
        }
        float rstd = rstd_of(sum_lanes<L>(dot8(v, v)), inv_d, a.eps);
        if (h >= a.H[t]) rstd = 0.f;  // no row: with eps = 0 it would be infinite, and dw NaN
        const float m = rstd * sum_lanes<L>(dot8(e, v)) * inv_d;
#pragma unroll
        for (int j = 0; j < NORM_V; ++j) {
          v[j] *= rstd;
          dw[t][j] += g[j] * v[j];
          e[j] = rstd * (e[j] - v[j] * m);
        }
        if (h < a.H[t] && r.col) st8<STREAM>(dx + h * a.D, e);
      }
    }
  }
  if (!a.dw[0] && !a.dw[1]) return;
  const int two = a.dw[0] && a.dw[1];
  float* out = a.part + (size_t)blockIdx.x * (1 + two) * a.D;
  if (a.dw[0]) join_groups<L, ROT_THREADS>(dw[0], a.D, out, lds);
  if (a.dw[1]) join_groups<L, ROT_THREADS>(dw[1], a.D, out + two * a.D, lds);
}

// Few tokens: their heads are spread over several waves, as long as that makes
// no more than 2048 of them (backward of 254 tokens, 32 + 16 heads of 256, fp32:
// 23 us with a wave a token, 13.7 with eight, 17 with 16 or the 32 that there
// are heads; 2000 tokens of 16 + 16 heads of 128, bf16: 16.2 with one, 18 with
// two).
constexpr int ROT_SPLIT = 2048;
static int rotary_split(long long N, const int (&H)[2], int D) {
  const int G = 64 / norm_lanes(D), most = ((H[0] > H[1] ? H[0] : H[1]) + G - 1) / G;
  int split = 1;
  while (split < most && N * split * 2 <= ROT_SPLIT) split *= 2;
  return split > most ? most : split;
}
// Workgroups of the backward kernel, each with a row of partial sums: fixed by
// the shape, so that the sums' order is too.  (62,720 tokens of 16 + 16 heads of
// 128, bf16: 305 us with 512, 277 with 768, 272 with 1024 or 2048, whose rows
// take longer to add up: few and small ones lose what that gains.)
constexpr int ROT_GROUPS = 768;
int rotary_groups(long long N, const int (&H)[2], int D) {
  const long long need = (N * rotary_split(N, H, D) + ROT_WAVES - 1) / ROT_WAVES;
  return (int)(need < ROT_GROUPS ? need : ROT_GROUPS);
}

template <typename T, int L, bool NB, bool STREAM>
static hipError_t rotary_fwd_l(const RotaryArgs& a, hipStream_t st, Profiler* prof) {
  const int split = rotary_split(a.N, a.H, a.D);
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
  const int grid = rotary_groups(a.N, a.H, a.D);
  if (grid > 0) {
    prof_begin(prof, "rotary_bwd", st);
    hipLaunchKernelGGL((rotary_bwd_kernel<T, L, NB, STREAM>), dim3(grid), dim3(ROT_THREADS), 0, st, a,
                       rotary_split(a.N, a.H, a.D));
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
  // (past the caches: 99 us instead of 111 forward, 277 instead of 320 backward)
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
