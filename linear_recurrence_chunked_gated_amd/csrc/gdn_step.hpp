// The gated delta rule one token at a time over a pool of sequence states:
// the serving form beside the chunk kernels.
//
// Per sequence and value head, with a state S of D x D values (row v, column
// k), each new token does
//     p = S k,  s = S q                       (two dot products per row)
//     u = beta (v - alpha p)
//     o = alpha s + u (k . q)                 (= S' q, without a second pass)
//     S' = alpha S + u k^T
// Row v of the state meets only v's own entry of p, s, u and o, so rows are
// independent: eight lanes hold one row (D / 8 columns each, in 16-byte
// pieces so that a load instruction of a wave covers 128 consecutive bytes of
// eight rows), the two dot products end in three DPP steps among those lanes,
// and the state stays in registers over all of a sequence's tokens.
#pragma once
#include "gdn_kernels.hpp"

namespace sfgdn {

// What a sequence's entry of the batch says.  slot < 0 is padding (nothing is
// read or written).  An entry whose slot lies outside the pool, or (when the
// pool is written) repeats the slot of an earlier entry, is refused: its
// outputs become NaN and the pool is left alone.  Offsets are clamped to the
// token tensors, so no entry reaches outside them.
struct SeqEntry {
  int slot;
  int t0, t1;
  bool bad;
};
__device__ __forceinline__ SeqEntry seq_entry(const PoolBatch& b, int i) {
  SeqEntry e;
  e.slot = b.slots ? b.slots[i] : i;
  if (b.seq_start) {
    e.t0 = min(max(b.seq_start[i], 0), b.n_tok);
    e.t1 = min(b.seq_start[i + 1], b.n_tok);
  } else {
    e.t0 = i * b.uniform;
    e.t1 = e.t0 + b.uniform;
  }
  e.bad = e.slot >= b.n_slots;
  return e;
}
// Whether an earlier entry names the same slot (whole waves call this).
__device__ __forceinline__ bool slot_repeats(const PoolBatch& b, int i, int slot) {
  bool hit = false;
  for (int j = lane_id(); j < i; j += 64) hit |= b.slots[j] == slot;
  return __any(hit);
}

// sum over the 8 lanes of a half row; every lane ends with the total
__device__ __forceinline__ float sum_half_row8(float x) {
  x += dpp_f<0xB1>(x);
  x += dpp_f<0x4E>(x);
  x += dpp_f<0x141>(x);
  return x;
}

constexpr int STEP_THREADS = 256;

template <typename T> struct Row4 {
  typedef T vec __attribute__((ext_vector_type(4)));
};

// Workgroup: 4 waves, wave w rows r0 + 8 NR w .. of one (sequence, value
// head); NR row groups of 8 rows per wave.
template <typename T, int D, int NR>
__global__ __launch_bounds__(STEP_THREADS) void recurrent_step_kernel(StepArgs a) {
  typedef typename Row4<T>::vec vec4;
  constexpr int NE = D / 32;  // 4-column pieces per lane
  constexpr int PARTS = D / (32 * NR);
  const int part = blockIdx.x % PARTS;
  const int sh = blockIdx.x / PARTS;
  const int hv = sh % a.Hv, seq = sh / a.Hv;
  const SeqEntry e = seq_entry(a.b, seq);
  if (e.slot < 0 || e.t0 >= e.t1) return;
  const int lane = lane_id(), l8 = lane & 7;
  const int r0 = (part * 4 + wave_id()) * 8 * NR;  // first row of this wave
  const int row = r0 + (lane >> 3);                // row group r: row + 8 r
  T* __restrict__ o = reinterpret_cast<T*>(a.o) + (size_t)hv * D + r0;
  const size_t os = (size_t)a.Hv * D;
  // lane (group g = lane / 8, l8) writes output row 8 l8 + g, for l8 < NR
  const int orow = 8 * l8 + (lane >> 3);

  float4 S[NR][NE];
  float* Sp = a.state;
  if (!e.bad) {
    Sp += ((size_t)e.slot * a.Hv + hv) * D * D + (size_t)row * D + l8 * 4;
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int j = 0; j < NE; ++j) S[r][j] = *reinterpret_cast<const float4*>(Sp + r * 8 * D + j * 32);
  }
  const bool bad = e.bad || (a.update && a.b.slots && slot_repeats(a.b, seq, e.slot));
  if (bad) {
    if (l8 < NR)
      for (int t = e.t0; t < e.t1; ++t) o[t * os + orow] = (T)__builtin_nanf("");
    return;
  }
  const int hk = hv / a.group;
  const T* __restrict__ q = reinterpret_cast<const T*>(a.q) + (size_t)hk * D + l8 * 4;
  const T* __restrict__ k = reinterpret_cast<const T*>(a.k) + (size_t)hk * D + l8 * 4;
  const T* __restrict__ v = reinterpret_cast<const T*>(a.v) + (size_t)hv * D + row;

  vec4 kn[NE], qn[NE];
  T vn[NR];
  float an, bn;
  auto fetch = [&](int t) {
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      kn[j] = *reinterpret_cast<const vec4*>(k + (size_t)t * a.ks + j * 32);
      qn[j] = *reinterpret_cast<const vec4*>(q + (size_t)t * a.qs + j * 32);
    }
#pragma unroll
    for (int r = 0; r < NR; ++r) vn[r] = v[(size_t)t * a.vs + r * 8];
    an = a.alpha[(size_t)t * a.Hv + hv];
    bn = a.beta[(size_t)t * a.Hv + hv];
  };
  fetch(e.t0);
  for (int t = e.t0; t < e.t1; ++t) {
    float kf[NE][4], qf[NE][4], vf[NR];
#pragma unroll
    for (int j = 0; j < NE; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        kf[j][i] = (float)kn[j][i];
        qf[j][i] = (float)qn[j][i];
      }
#pragma unroll
    for (int r = 0; r < NR; ++r) vf[r] = (float)vn[r];
    const float al = an, be = bn;
    if (t + 1 < e.t1) fetch(t + 1);
    float kq = 0.f;
#pragma unroll
    for (int j = 0; j < NE; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) kq += kf[j][i] * qf[j][i];
    kq = sum_half_row8(kq);
    float out = 0.f;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      float p = 0.f, s = 0.f;
#pragma unroll
      for (int j = 0; j < NE; ++j) {
        const float4 x = S[r][j];
        p += x.x * kf[j][0] + x.y * kf[j][1] + x.z * kf[j][2] + x.w * kf[j][3];
        s += x.x * qf[j][0] + x.y * qf[j][1] + x.z * qf[j][2] + x.w * qf[j][3];
      }
      p = sum_half_row8(p);
      s = sum_half_row8(s);
      const float u = be * (vf[r] - al * p);
      const float y = al * s + u * kq;
      out = l8 == r ? y : out;
#pragma unroll
      for (int j = 0; j < NE; ++j) {
        S[r][j].x = al * S[r][j].x + u * kf[j][0];
        S[r][j].y = al * S[r][j].y + u * kf[j][1];
        S[r][j].z = al * S[r][j].z + u * kf[j][2];
        S[r][j].w = al * S[r][j].w + u * kf[j][3];
      }
    }
    if (l8 < NR) o[t * os + orow] = (T)out;
  }
  if (a.update) {
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int j = 0; j < NE; ++j) *reinterpret_cast<float4*>(Sp + r * 8 * D + j * 32) = S[r][j];
  }
}

template <typename T, int D, int NR>
static hipError_t step_nr(const StepArgs& a, hipStream_t st, Profiler* prof) {
  const unsigned grid = (unsigned)((size_t)a.b.n_seq * a.Hv * (D / (32 * NR)));
  prof_begin(prof, "recurrent_step", st);
  hipLaunchKernelGGL((recurrent_step_kernel<T, D, NR>), dim3(grid), dim3(STEP_THREADS), 0, st, a);
  prof_end(prof, st);
  return hipGetLastError();
}

template <typename T, int D>
hipError_t launch_recurrent_step(const StepArgs& a, hipStream_t st, Profiler* prof) {
  return step_nr<T, D, 1>(a, st, prof);
}

template hipError_t launch_recurrent_step<bf16, 64>(const StepArgs&, hipStream_t, Profiler*);
template hipError_t launch_recurrent_step<bf16, 128>(const StepArgs&, hipStream_t, Profiler*);
template hipError_t launch_recurrent_step<float, 64>(const StepArgs&, hipStream_t, Profiler*);
template hipError_t launch_recurrent_step<float, 128>(const StepArgs&, hipStream_t, Profiler*);

}  // namespace sfgdn
