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
//
// One token per sequence is bound by the states' traffic: 256 sequences of 32
// value heads at D = 128 (1.08 GB) take 182 us, 5.9 TB/s; a plain device copy
// of 1 GiB runs at 5.1 TB/s.  64 sequences of 1 to 8 tokens and 16 heads (139
// MB) take 27 us, 5.1 TB/s.  A long run is bound by a token's dependent
// arithmetic, 0.24 us at D = 128 and 0.2 at D = 64: one sequence of 256 tokens
// (16 heads, D = 128) takes 63 us, 7 of 33 tokens (6 heads, D = 64) 8.4.  Two
// tokens a reduction would shorten that chain (S_t k_{t+1} = alpha_t S_{t-1}
// k_{t+1} + u_t k_t . k_{t+1}), but would make a token's bits depend on which
// tokens came in the same call.
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
// Whether an earlier entry names the same slot: each wave scans up to 256
// entries by itself, a workgroup of several shares the work on more (4096
// sequences of 16 heads, D = 64: 381 us a call, 339 without slots, 655 with
// one load at a time and every wave for itself).  Every thread calls it.
template <int WAVES>
__device__ __forceinline__ bool slot_repeats(const PoolBatch& b, int i, int slot) {
  constexpr int U = 4;  // loads in flight
  const bool share = WAVES > 1 && i > 256;
  const int first = share ? threadIdx.x : lane_id(), step = share ? WAVES * 64 : 64;
  bool hit = false;
#pragma unroll 1
  for (int j = 0; j < i; j += U * step)
#pragma unroll
    for (int u = 0; u < U; ++u) hit |= b.slots[min(j + u * step + first, i - 1)] == slot;
  return share ? __syncthreads_or(hit) : __any(hit);
}

// Sums over a row's D columns come out the same, bit for bit, on 8 and on 16
// lanes and for a token that came alone or among others, so that a sequence's
// outputs do not depend on how it was batched: columns go in units of four,
// unit c of a row is summed with unit c + 16 (where D has it), that with unit
// c + 8's sum, and the eight results in a tree.  Which products are fused with
// an addition is written out, for the same reason.
//
// x: this lane's part, on 16 lanes the sum of units l and l + 16, on 8 lanes
// already joined with units l + 8 and l + 24; every lane gets the total.
template <int L>
__device__ __forceinline__ float sum_row_lanes(float x) {
  if (L == 16) x += dpp_f<0x128>(x);  // rotate by 8 within the 16 lanes
  x += dpp_f<0xB1>(x);
  x += dpp_f<0x4E>(x);
  x += dpp_f<0x141>(x);
  return x;
}
// S . k over the row, in every lane (NE is H or 2 H)
template <int NE, int L>
__device__ __forceinline__ float row_dot(const f32x4 (&S)[NE], const f32x4 (&k)[NE]) {
  constexpr int H = L == 8 ? 2 : 1;  // units summed apart in a lane
  float x[H];
#pragma unroll
  for (int h = 0; h < H; ++h) {
    if (NE == H) {
      x[h] = __builtin_fmaf(S[h][0], k[h][0], S[h][1] * k[h][1]) +
             __builtin_fmaf(S[h][2], k[h][2], S[h][3] * k[h][3]);
    } else {
      float s[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        s[i] = __builtin_fmaf(S[h + H][i], k[h + H][i], S[h][i] * k[h][i]);
      x[h] = (s[0] + s[1]) + (s[2] + s[3]);
    }
  }
  return sum_row_lanes<L>(H == 2 ? x[0] + x[H - 1] : x[0]);
}
// one unit of k . q
__device__ __forceinline__ float unit_dot(f32x4 k, f32x4 q) {
  return __builtin_fmaf(k[3], q[3],
                        __builtin_fmaf(k[2], q[2], __builtin_fmaf(k[1], q[1], k[0] * q[0])));
}

constexpr int STEP_THREADS = 256;
// Threads that stage a token, and tokens staged in LDS at a time (8 or 16): two
// buffers take about 20 KB, so that seven workgroups share a compute unit.
constexpr int step_token_threads(int D) { return D / 4; }
constexpr int step_tokens(int D) { return STEP_THREADS / step_token_threads(D); }

// Workgroup: 4 waves, each of 64 / L rows of one (sequence, value head)'s
// state, a row on L lanes.  SINGLE: one token per sequence, straight from
// global memory with the state.  Otherwise the tokens are staged through LDS
// a chunk ahead, as floats and with k . q beside them, since a token's
// arithmetic is far shorter than a load and each wave would repeat both.
// STREAM: the states bypass the caches (see launch_recurrent_step).
template <typename T, int D, int L, bool SINGLE, bool STREAM>
__global__ __launch_bounds__(STEP_THREADS) void recurrent_step_kernel(StepArgs a) {
  constexpr int NE = D / (4 * L);        // 4-column pieces per lane
  constexpr int WROWS = 64 / L;          // rows of a wave
  constexpr int ROWS = 4 * WROWS;        // rows of the workgroup
  constexpr int PARTS = D / ROWS;
  const int part = blockIdx.x % PARTS;
  const int sh = blockIdx.x / PARTS;
  const int hv = sh % a.Hv, seq = sh / a.Hv;
  const SeqEntry e = seq_entry(a.b, seq);
  if (e.slot < 0 || e.t0 >= e.t1) return;
  const int lane = lane_id(), l = lane % L;
  const int wrow = wave_id() * WROWS + lane / L;  // this lane's row in the workgroup
  const int r0 = part * ROWS;
  T* __restrict__ o = reinterpret_cast<T*>(a.o) + (size_t)hv * D + r0 + wrow;
  const size_t os = (size_t)a.Hv * D;

  f32x4 S[NE];
  float* Sp = a.state;
  if (!e.bad) {
    Sp += ((size_t)e.slot * a.Hv + hv) * D * D + (size_t)(r0 + wrow) * D + l * 4;
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      const f32x4* p = reinterpret_cast<const f32x4*>(Sp + j * 4 * L);
      S[j] = STREAM ? __builtin_nontemporal_load(p) : *p;
    }
  }
  const bool bad = e.bad || (a.update && a.b.slots && slot_repeats<4>(a.b, seq, e.slot));
  if (bad) {
    if (l == 0)
      for (int t = e.t0; t < e.t1; ++t) o[t * os] = (T)__builtin_nanf("");
    return;
  }
  const int hk = hv / a.group;
  const T* __restrict__ q = reinterpret_cast<const T*>(a.q) + (size_t)hk * D;
  const T* __restrict__ k = reinterpret_cast<const T*>(a.k) + (size_t)hk * D;
  const T* __restrict__ v = reinterpret_cast<const T*>(a.v) + (size_t)hv * D + r0;

  struct Token {
    f32x4 k[NE], q[NE];
    f32x4 g;  // alpha, beta, k . q
    float v;
  };
  auto token = [&](const Token& x) {
    const float p = row_dot<NE, L>(S, x.k), s = row_dot<NE, L>(S, x.q);
    const float u = x.g[1] * __builtin_fmaf(-x.g[0], p, x.v);
    const float y = __builtin_fmaf(u, x.g[2], x.g[0] * s);
#pragma unroll
    for (int j = 0; j < NE; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) S[j][i] = __builtin_fmaf(u, x.k[j][i], x.g[0] * S[j][i]);
    return y;
  };

  if constexpr (SINGLE) {
    typedef T vec4 __attribute__((ext_vector_type(4)));
    const size_t t = e.t0;
    Token x;
    float kq[NE];
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      x.k[j] = __builtin_convertvector(
          *reinterpret_cast<const vec4*>(k + t * a.ks + (j * L + l) * 4), f32x4);
      x.q[j] = __builtin_convertvector(
          *reinterpret_cast<const vec4*>(q + t * a.qs + (j * L + l) * 4), f32x4);
      kq[j] = unit_dot(x.k[j], x.q[j]);
    }
    constexpr int U = 16 / L;  // units l (and l + 8) of this lane, each with the one 16 on
#pragma unroll
    for (int j = U; j < NE; ++j) kq[j - U] += kq[j];
    if (U == 2) kq[0] += kq[1];
    x.v = (float)v[t * a.vs + wrow];
    x.g[0] = a.alpha[t * a.Hv + hv];
    x.g[1] = a.beta[t * a.Hv + hv];
    x.g[2] = sum_row_lanes<L>(kq[0]);
    const float y = token(x);
    if (l == 0) o[t * os] = (T)y;
  } else {
    // Staging: each thread of a token has a unit of four columns of k and q,
    // and the token's rows of v are spread over them.
    constexpr int TT = step_token_threads(D), TB = step_tokens(D);
    constexpr int VV = (ROWS + TT - 1) / TT;
    typedef T vec4 __attribute__((ext_vector_type(4)));
    struct Chunk {
      f32x4 k[TB][D / 4], q[TB][D / 4];
      float v[TB][VV * TT];
      f32x4 g[TB];  // alpha, beta, k . q
    };
    __shared__ Chunk lds[2];
    const int st = threadIdx.x / TT, sl = threadIdx.x % TT;  // token of the chunk, unit in it
    vec4 rk, rq;
    T rv[VV];
    float ra = 0.f, rb = 0.f;
    auto load = [&](int c) {
      const size_t t = min(c + st, e.t1 - 1);  // past the end: the last token again, not used
      rk = *reinterpret_cast<const vec4*>(k + t * a.ks + sl * 4);
      rq = *reinterpret_cast<const vec4*>(q + t * a.qs + sl * 4);
#pragma unroll
      for (int i = 0; i < VV; ++i) rv[i] = v[t * a.vs + min(i * TT + sl, ROWS - 1)];
      ra = a.alpha[t * a.Hv + hv];
      rb = a.beta[t * a.Hv + hv];
    };
    auto store = [&](Chunk& b) {
      const f32x4 kf = __builtin_convertvector(rk, f32x4), qf = __builtin_convertvector(rq, f32x4);
      float kq = unit_dot(kf, qf);
      if (D == 128) kq += __shfl_xor(kq, 16);
      kq = sum_row_lanes<16>(kq);
      b.k[st][sl] = kf;
      b.q[st][sl] = qf;
#pragma unroll
      for (int i = 0; i < VV; ++i) b.v[st][i * TT + sl] = (float)rv[i];
      if (sl == 0) b.g[st] = f32x4{ra, rb, kq, 0.f};
    };
    T* ot = o + e.t0 * os;
    load(e.t0);
#pragma unroll 1
    for (int c = e.t0, buf = 0; c < e.t1; c += TB, buf ^= 1) {
      // this buffer's readers (two chunks back) have passed the last barrier
      store(lds[buf]);
      __syncthreads();
      if (c + TB < e.t1) load(c + TB);
      const Chunk& b = lds[buf];
      const int m = min(TB, e.t1 - c);
      auto read = [&](int i, Token& x) {
#pragma unroll
        for (int j = 0; j < NE; ++j) {
          x.k[j] = b.k[i][j * L + l];
          x.q[j] = b.q[i][j * L + l];
        }
        x.g = b.g[i];
        x.v = b.v[i][wrow];
      };
      Token x;
      if constexpr (L == 16) {
        // Few workgroups, a wave or two per SIMD: what counts is a token's own
        // latency.  The next token is read from LDS ahead, four tokens run
        // without a branch between them, and lane i keeps token i's output to
        // store it after the chunk (33 tokens of a 64-wide fp32 state: 7.7 us
        // instead of 8.8).  With many workgroups the late stores cost more
        // than the branches (64 sequences of 4 tokens in fp32, 32 heads of
        // D = 128: 54 us instead of 51).
        static_assert(TB <= L, "a lane for each token's output");
        constexpr int U = 4;
        float out = 0.f;
        auto step = [&](int i) {
          Token y;
          read(min(i + 1, m - 1), y);
          const float r = token(x);
          out = l == i ? r : out;
          x = y;
        };
        read(0, x);
        int i = 0;
#pragma unroll 1
        for (; i + U <= m; i += U) {
#pragma unroll
          for (int u = 0; u < U; ++u) step(i + u);
        }
#pragma unroll 1
        for (; i < m; ++i) step(i);
        if (l < m) ot[l * os] = (T)out;
        ot += m * os;
      } else {
#pragma unroll 1
        for (int i = 0; i < m; ++i, ot += os) {
          read(i, x);
          const float y = token(x);
          if (l == 0) *ot = (T)y;
        }
      }
    }
  }
  if (a.update) {
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      f32x4* p = reinterpret_cast<f32x4*>(Sp + j * 4 * L);
      if (STREAM)
        __builtin_nontemporal_store(S[j], p);
      else
        *p = S[j];
    }
  }
}

template <typename T, int D, int L, bool SINGLE, bool STREAM>
static hipError_t step_launch(const StepArgs& a, hipStream_t st, Profiler* prof) {
  const unsigned grid = (unsigned)((size_t)a.b.n_seq * a.Hv * (D * L / 256));
  prof_begin(prof, "recurrent_step", st);
  hipLaunchKernelGGL((recurrent_step_kernel<T, D, L, SINGLE, STREAM>), dim3(grid),
                     dim3(STEP_THREADS), 0, st, a);
  prof_end(prof, st);
  return hipGetLastError();
}

// The variants, each against the other on an MI355X (bf16, D = 128, 16 heads):
//  - states of 128 MiB or more in one call cannot stay in the 256 MB last-level
//    cache until the next one: non-temporal loads and stores take 183 us
//    instead of 203 for 512 MiB and 50 instead of 53 for 128 MiB, but 37.3
//    instead of 36.2 for 96 MiB and 19.9 instead of 17.3 for 48 MiB;
//  - with several tokens and too few workgroups of eight-lane rows to give
//    every compute unit one, 16 lanes a row halve each token's arithmetic:
//    one sequence of 256 tokens 62 us instead of 83, two of 8 tokens 4.5
//    instead of 5.1; at 256 workgroups both take 5.4 and beyond, the eight
//    lanes are faster (8 sequences of 8 tokens 7.5 instead of 8.6).
template <typename T, int D>
hipError_t launch_recurrent_step(const StepArgs& a, hipStream_t st, Profiler* prof) {
  const size_t heads = (size_t)a.b.n_seq * a.Hv;
  const bool stream = heads * D * D * sizeof(float) >= (size_t)128 << 20;
  if (!a.b.seq_start && a.b.uniform == 1)
    return stream ? step_launch<T, D, 8, true, true>(a, st, prof)
                  : step_launch<T, D, 8, true, false>(a, st, prof);
  if (stream) return step_launch<T, D, 8, false, true>(a, st, prof);
  if (heads * (D / 32) < 256) return step_launch<T, D, 16, false, false>(a, st, prof);
  return step_launch<T, D, 8, false, false>(a, st, prof);
}

template hipError_t launch_recurrent_step<bf16, 64>(const StepArgs&, hipStream_t, Profiler*);
template hipError_t launch_recurrent_step<bf16, 128>(const StepArgs&, hipStream_t, Profiler*);
template hipError_t launch_recurrent_step<float, 64>(const StepArgs&, hipStream_t, Profiler*);
template hipError_t launch_recurrent_step<float, 128>(const StepArgs&, hipStream_t, Profiler*);

}  // namespace sfgdn
