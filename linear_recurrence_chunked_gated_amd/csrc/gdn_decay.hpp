// Linear attention with a fixed decay a for each head, over whole prompts or
// training chunks: sequences of one length or packed ones of different
// lengths, and the gradients.
//
//     S_t = a S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t
//
// In blocks of C = 64 tokens (n of them valid), r and s local, entry state E:
//     Y_r = sum_{s <= r} a^(r-s) (x_r . u_s) w_s + a^(r+1) E x_r
//     E'  = a^n E + sum_s a^(n-1-s) w_s u_s^T
// with x, u, w = q, k, v and E = S.  The backward is the same scan with its
// roles exchanged: with G_t = scale do_t q_t^T + a G_{t+1} (+ dS_out at the end)
//     dq_t = scale S_t^T do_t    forward,  x, u, w = do, v, k, E = S^T
//     dv_t = G_t k_t             reversed, x, u, w = k, q, do, E = G
//     dk_t = G_t^T v_t           reversed, x, u, w = v, do, q, E = G^T
// where the reversed scan has a^(s-r) over s >= r, a^(n-1-r) on E x_r and
// a^(s+1) on w_s u_s^T, from the last block to the first; dS_in is its exit.
//
// A sequence is cut into segments of L tokens (an item each) so that the items
// of all heads fill the GPU:
//   decay_sum     every inner boundary's sum over the segment before it (after
//                 it, reversed), from zero
//   decay_chain   those to the states at the boundaries, one after another
//   decay_scan    every item from its entry state: the outputs, and the last
//                 (first) item's exit state
#pragma once
#include "gdn_kernels.hpp"

namespace sfgdn {

constexpr int DECAY_NW = 4;  // waves per workgroup
constexpr int DECAY_NT = 64 * DECAY_NW;

// One item: a segment of a sequence.  prev, next: the boundary slots before
// and after it (-1 at the sequence's ends).
struct DecayItem {
  int seq, t0, n, prev, next;
};

__device__ __forceinline__ bool decay_item(const DecayPlan& p, int i, DecayItem& it) {
  if (p.table) {
    if (i >= p.table[0]) return false;
    const int* e = p.table + kDecayHead + i * kDecayItem;
    it = DecayItem{e[0], e[1], e[2], e[3], e[4]};
    return true;
  }
  const int seq = i / p.P, j = i - seq * p.P;
  it.seq = seq;
  it.t0 = seq * p.T + j * p.L;
  it.n = min(p.L, p.T - j * p.L);
  it.prev = j > 0 ? seq * (p.P - 1) + j - 1 : -1;
  it.next = j + 1 < p.P ? seq * (p.P - 1) + j : -1;
  return true;
}

// a^e for e >= 0, by squaring in 64 bits: exact to a rounding for every a,
// 0 and values near 1 among them.
__device__ __forceinline__ float decay_pow(float a, int e) {
  double r = 1.0, b = a;
  while (e > 0) {
    if (e & 1) r *= b;
    b *= b;
    e >>= 1;
  }
  return (float)r;
}

// ------------------------------------------------------------------ the plan
// Items and boundary slots of packed sequences, by one workgroup.  Offsets are
// taken as their running maximum, clamped to the token rows, so that items
// never overlap or reach outside them, whatever seq_start holds.
template <typename F>
__device__ __forceinline__ int scan1024(int x, int* lds, int ident, F join, int& total) {
  const int lane = lane_id(), w = wave_id();
  for (int d = 1; d < 64; d *= 2) {
    const int y = __shfl_up(x, d);
    if (lane >= d) x = join(x, y);
  }
  __syncthreads();
  if (lane == 63) lds[w] = x;
  __syncthreads();
  int before = ident;
  total = ident;
  for (int i = 0; i < 16; ++i) {
    if (i == w) before = total;
    total = join(total, lds[i]);
  }
  return join(before, x);
}

__global__ __launch_bounds__(1024) void decay_plan_kernel(const int* seq_start, int n_seq, int n_tok,
                                                          int L, int max_items, int* table) {
  __shared__ int lds[16];
  auto add = [](int a, int b) { return a + b; };
  auto most = [](int a, int b) { return max(a, b); };
  int* items = table + kDecayHead;
  int* multi = items + max_items * kDecayItem;
  int end = 0, n_items = 0, n_multi = 0;
  for (int base = 0; base < n_seq; base += 1024) {
    const int i = base + threadIdx.x;
    const bool live = i < n_seq;
    int x = live ? min(max(seq_start[i], 0), n_tok) : 0, top;
    const int t0 = max(end, scan1024(x, lds, 0, most, top));
    const int t1 = live ? max(t0, min(max(seq_start[i + 1], 0), n_tok)) : t0;
    end = max(end, top);
    const int len = t1 - t0;
    const int cnt = live ? max(1, (len + L - 1) / L) : 0;
    int sum, msum;
    const int at = n_items + scan1024(cnt, lds, 0, add, sum) - cnt;
    const int many = cnt > 1;
    const int m = n_multi + scan1024(many, lds, 0, add, msum) - many;
    // boundary slots before this sequence's: one less than items for each sequence
    const int slot0 = at - i;
    if (live)
      for (int j = 0; j < cnt; ++j) {
        int* e = items + (at + j) * kDecayItem;
        e[0] = i;
        e[1] = t0 + j * L;
        e[2] = min(L, len - j * L);
        e[3] = j > 0 ? slot0 + j - 1 : -1;
        e[4] = j + 1 < cnt ? slot0 + j : -1;
      }
    if (many) {
      int* e = multi + m * kDecayMulti;
      e[0] = i;
      e[1] = slot0;
      e[2] = cnt - 1;
      e[3] = len - (cnt - 1) * L;
    }
    n_items += sum;
    n_multi += msum;
  }
  if (threadIdx.x == 0) {
    table[0] = n_items;
    table[1] = n_multi;
    table[2] = n_seq > 0 ? min(max(seq_start[0], 0), n_tok) : 0;  // the rows that sequences have
    table[3] = max(end, n_seq > 0 ? min(max(seq_start[n_seq], 0), n_tok) : 0);
  }
}

// --------------------------------------------------------------------- tiles
// Operands are bf16: one plane for bf16 tensors; two for fp32 ones, x = hi +
// lo, with the three products hi hi + hi lo + lo hi summed in fp32 (what is
// left out is below 2^-16 of a term, and about 2e-6 of a sum; fp32 matrix
// instructions would take five times the time of the three).
template <typename T> constexpr int planes() { return sizeof(T) == 2 ? 1 : 2; }

template <int NA, int NB>
__device__ __forceinline__ f32x4 mma_planes(const bf16x8 (&a)[NA], const bf16x8 (&b)[NB], f32x4 c) {
  if constexpr (NA == 2) c = Mma<bf16>::mma(a[1], b[0], c);
  if constexpr (NB == 2) c = Mma<bf16>::mma(a[0], b[1], c);
  return Mma<bf16>::mma(a[0], b[0], c);
}

// Rows of D values, in planes of 64 x D bf16 (swizzled).
template <typename T, int D> struct DecayTile {
  static constexpr int NP = planes<T>();
  static constexpr int ELEMS = BLK * D;  // of a plane
  static constexpr int VEC = 16 / (int)sizeof(T), CPR = D / VEC, NCH = BLK * CPR / DECAY_NT;

  __device__ static __forceinline__ void load(uint4 (&r)[NCH], const T* g, size_t row_stride,
                                              int nvalid) {
#pragma unroll
    for (int it = 0; it < NCH; ++it) {
      const int c = threadIdx.x + DECAY_NT * it;
      const int row = min(c / CPR, nvalid - 1), ch = c % CPR;
      r[it] = *reinterpret_cast<const uint4*>(g + (size_t)row * row_stride + ch * VEC);
    }
  }
  __device__ static __forceinline__ void to_lds(const uint4 (&r)[NCH], bf16* s, int nvalid) {
#pragma unroll
    for (int it = 0; it < NCH; ++it) {
      const int c = threadIdx.x + DECAY_NT * it;
      const int row = c / CPR, ch = c % CPR;
      const bool ok = row < nvalid;
      uint4 v = r[it];
      v.x = ok ? v.x : 0u;
      v.y = ok ? v.y : 0u;
      v.z = ok ? v.z : 0u;
      v.w = ok ? v.w : 0u;
      bf16* p = lds_sw(s + row * D + ch * VEC, D);
      if constexpr (NP == 1) {
        *reinterpret_cast<uint4*>(p) = v;
      } else {
        const f32x4 f = __builtin_bit_cast(f32x4, v);
        bf16x4 hi, lo;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          hi[e] = (bf16)f[e];
          lo[e] = (bf16)(f[e] - (float)hi[e]);
        }
        *reinterpret_cast<bf16x4*>(p) = hi;
        *reinterpret_cast<bf16x4*>(p + ELEMS) = lo;
      }
    }
  }
  // operand rows from row0, contraction along the row
  template <int KO>
  __device__ static __forceinline__ void rows(const bf16* s, int row0, int step, bf16x8 (&f)[NP]) {
#pragma unroll
    for (int p = 0; p < NP; ++p)
      f[p] = frag_row<bf16, KO>(s + p * ELEMS + row0 * D, D, step);
  }
  // operand rows = columns from col0, contraction along the tokens
  __device__ static __forceinline__ void cols(const bf16* s, int col0, int step, bf16x8 (&f)[NP]) {
#pragma unroll
    for (int p = 0; p < NP; ++p) f[p] = frag_tr<bf16, STD>(s + p * ELEMS + col0, D, step);
  }
};

// Eight values to bf16 planes.
__device__ __forceinline__ void to_planes(const float (&x)[8], bf16x8 (&f)[1]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) f[0][j] = (bf16)x[j];
}
__device__ __forceinline__ void to_planes(const float (&x)[8], bf16x8 (&f)[2]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    f[0][j] = (bf16)x[j];
    f[1][j] = (bf16)(x[j] - (float)f[0][j]);
  }
}

// ------------------------------------------------------------------ the scan
// Workgroup: one item of one value head.  Wave w owns the state's columns
// (w_s' index) 16 NDV w .., held transposed in accumulators: tile [b][a] has
// m = the u index (16 a ..), n = the w index (16 (NDV w + b) ..).
//
// Roundings to fewer bits, for bf16 tensors: P and the state's copy that meets
// x, whose results are rounded to bf16 themselves; the state itself is summed
// from w scaled by its decay in two planes (2^-17), since it is an fp32 output
// and goes on from block to block.
template <typename T, int D, bool REV, bool OUT>
__global__ __launch_bounds__(DECAY_NT, 2) void decay_scan_kernel(DecayScanArgs a) {
  typedef DecayTile<T, D> Tl;
  constexpr int NP = planes<T>(), NDV = D / 16 / DECAY_NW, NDU = D / 16;
  constexpr int KD = D / 32, KT = BLK / 32;
  extern __shared__ __align__(16) unsigned char smem[];
  bf16* Us = reinterpret_cast<bf16*>(smem);
  bf16* Ws = Us + NP * Tl::ELEMS;
  bf16* Xs = Ws + NP * Tl::ELEMS;
  bf16* Ps = Xs + NP * Tl::ELEMS;
  float* pw = reinterpret_cast<float*>(OUT ? Ps + NP * BLK * BLK : Xs);  // a^0 .. a^64, [65] used
  float* dec = pw + 68;                                                // [64]

  const DecayRole& R = a.role[blockIdx.y];
  const int hv = blockIdx.x % a.Hv;
  DecayItem it;
  if (!decay_item(a.plan, blockIdx.x / a.Hv, it)) return;
  if (!OUT && (REV ? it.prev : it.next) < 0) return;  // no boundary behind this item
  const int hk = hv / a.group;
  const int w = wave_id(), lane = lane_id(), g = lane >> 4, li = lane & 15;
  const int w0 = 16 * NDV * w;  // this wave's first state column
  const float alpha = a.decay[hv];

  f32x4 St[NDV][NDU];
  {
    const int slot = REV ? it.next : it.prev;
    const float* E = nullptr;
    bool tr = R.tr_state;
    if (OUT) {
      if (slot >= 0) {
        E = R.bound + ((size_t)slot * a.Hv + hv) * D * D;
        tr = R.tr_bound;
      } else if (R.state) {
        E = R.state + ((size_t)it.seq * a.Hv + hv) * D * D;
      }
    }
#pragma unroll
    for (int b = 0; b < NDV; ++b)
#pragma unroll
      for (int c = 0; c < NDU; ++c) {
        const int m = 16 * c + 4 * g, n = w0 + 16 * b + li;
        f32x4 x = {0.f, 0.f, 0.f, 0.f};
        if (E && tr) {
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = E[(size_t)(m + e) * D + n];
        } else if (E) {
          x = *reinterpret_cast<const f32x4*>(E + (size_t)n * D + m);
        }
        St[b][c] = x;
      }
  }

  const T* xg = nullptr;
  if constexpr (OUT)
    xg = reinterpret_cast<const T*>(R.x.p) + (size_t)it.t0 * R.x.stride + (R.x.shared ? hk : hv) * D;
  const T* ug = reinterpret_cast<const T*>(R.u.p) + (size_t)it.t0 * R.u.stride + (R.u.shared ? hk : hv) * D;
  const T* wg = reinterpret_cast<const T*>(R.w.p) + (size_t)it.t0 * R.w.stride + (R.w.shared ? hk : hv) * D;

  const int nblk = (it.n + BLK - 1) / BLK;
  uint4 rx[OUT ? Tl::NCH : 1], ru[Tl::NCH], rw[Tl::NCH];
  auto fetch = [&](int b) {
    const int nv = min(BLK, it.n - b * BLK);
    const size_t t = (size_t)b * BLK;
    Tl::load(ru, ug + t * R.u.stride, R.u.stride, nv);
    if constexpr (OUT) Tl::load(rx, xg + t * R.x.stride, R.x.stride, nv);
    Tl::load(rw, wg + t * R.w.stride, R.w.stride, nv);
  };
  if (nblk > 0) fetch(REV ? nblk - 1 : 0);

  // powers; P tiles that the mask empties but a product of 32 tokens reads
  if (threadIdx.x <= BLK) pw[threadIdx.x] = decay_pow(alpha, threadIdx.x);
  if constexpr (OUT) {
    for (int i = threadIdx.x; i < NP * BLK * BLK / 8; i += DECAY_NT)
      reinterpret_cast<uint4*>(Ps)[i] = uint4{0, 0, 0, 0};
  }
  lds_barrier();
  float fd[4], fo[4], ft[3];  // a^|r-s| of a diagonal tile (masked), of the next one off, of 16 more
  if constexpr (OUT) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int d = REV ? 4 * g + e - li : li - 4 * g - e;
      fd[e] = d >= 0 ? R.s_pair * pw[d] : 0.f;
      fo[e] = R.s_pair * pw[16 + d];
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) ft[i] = pw[16 * i];
  }

  for (int i = 0; i < nblk; ++i) {
    const int blk = REV ? nblk - 1 - i : i;
    const int nv = min(BLK, it.n - blk * BLK);
    Tl::to_lds(ru, Us, nv);
    if constexpr (OUT) Tl::to_lds(rx, Xs, nv);
    Tl::to_lds(rw, Ws, nv);
    if (threadIdx.x < BLK)
      dec[threadIdx.x] = R.s_pair * pw[REV ? threadIdx.x + 1 : max(0, nv - 1 - (int)threadIdx.x)];
    lds_barrier();
    if (i + 1 < nblk) fetch(REV ? blk - 1 : blk + 1);

    f32x4 O[NDV][4];
    if constexpr (OUT) {
      // P: wave w has the pairs of s in its 16 tokens (m = s, n = r)
      const int r_lo = REV ? 0 : w, r_hi = REV ? w : 3;
      f32x4 p[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) p[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < KD; ++s) {
        bf16x8 fu[NP];
        Tl::template rows<STD>(Us, 16 * w, s, fu);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j >= r_lo && j <= r_hi) {
            bf16x8 fx[NP];
            Tl::template rows<STD>(Xs, 16 * j, s, fx);
            p[j] = mma_planes(fu, fx, p[j]);
          }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j >= r_lo && j <= r_hi) {
          const int off = REV ? w - j : j - w;
          float q[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            q[e] = p[j][e] * (off == 0 ? fd[e] : fo[e] * (off == 1 ? ft[0] : off == 2 ? ft[1] : ft[2]));
          bf16* d = lds_sw(Ps + (16 * j + li) * BLK + 16 * w + 4 * g, BLK);
          bf16x4 hi;
#pragma unroll
          for (int e = 0; e < 4; ++e) hi[e] = (bf16)q[e];
          *reinterpret_cast<bf16x4*>(d) = hi;
          if constexpr (NP == 2) {
            bf16x4 lo;
#pragma unroll
            for (int e = 0; e < 4; ++e) lo[e] = (bf16)(q[e] - (float)hi[e]);
            *reinterpret_cast<bf16x4*>(d + BLK * BLK) = lo;
          }
        }
      // E x
      zero_acc(O);
#pragma unroll
      for (int s = 0; s < KD; ++s) {
        bf16x8 fs[NDV][NP];
#pragma unroll
        for (int b = 0; b < NDV; ++b) {
          const f32x4 lo = St[b][2 * s], hi = St[b][2 * s + 1];
          const float x[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
          to_planes(x, fs[b]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          bf16x8 fx[NP];
          Tl::template rows<PERM>(Xs, 16 * j, s, fx);
#pragma unroll
          for (int b = 0; b < NDV; ++b) O[b][j] = mma_planes(fs[b], fx, O[b][j]);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = 16 * j + li;
        const float f = pw[REV ? max(0, nv - 1 - r) : r + 1];
#pragma unroll
        for (int b = 0; b < NDV; ++b) O[b][j] *= f;
      }
      lds_barrier();
    }
    // w of this wave's columns: for P w, and scaled for the state
    const float an = pw[nv];
#pragma unroll
    for (int b = 0; b < NDV; ++b)
#pragma unroll
      for (int c = 0; c < NDU; ++c) St[b][c] *= an;
#pragma unroll
    for (int s = 0; s < KT; ++s) {
      bf16x8 fw[NDV][NP], fd2[NDV][2];
      float dc[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) dc[j] = dec[32 * s + 8 * g + j];
#pragma unroll
      for (int b = 0; b < NDV; ++b) {
        Tl::cols(Ws, w0 + 16 * b, s, fw[b]);
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[j] = (float)fw[b][0][j];
          if constexpr (NP == 2) x[j] += (float)fw[b][1][j];
          x[j] *= dc[j];
        }
        to_planes(x, fd2[b]);
      }
      if constexpr (OUT) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (REV ? j < 2 * (s + 1) : j >= 2 * s) {
            bf16x8 fp[NP];
#pragma unroll
            for (int p = 0; p < NP; ++p)
              fp[p] = frag_row<bf16, STD>(Ps + p * BLK * BLK + 16 * j * BLK, BLK, s);
#pragma unroll
            for (int b = 0; b < NDV; ++b) O[b][j] = mma_planes(fw[b], fp, O[b][j]);
          }
      }
#pragma unroll
      for (int c = 0; c < NDU; ++c) {
        bf16x8 fu[NP];
        Tl::cols(Us, 16 * c, s, fu);
#pragma unroll
        for (int b = 0; b < NDV; ++b) St[b][c] = mma_planes(fu, fd2[b], St[b][c]);
      }
    }
    if constexpr (OUT) {
      const size_t t = (size_t)it.t0 + blk * BLK;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = 16 * j + li;
        if (r < nv) {
#pragma unroll
          for (int b = 0; b < NDV; ++b) {
            const f32x4 y = O[b][j] * R.s_out;
            const size_t at = ((t + r) * a.Hv + hv) * D + w0 + 16 * b + 4 * g;
            if (R.y_f32)
              *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(R.y) + at) = y;
            else
              st4(reinterpret_cast<T*>(R.y) + at, y[0], y[1], y[2], y[3]);
          }
        }
      }
    }
    lds_barrier();
  }

  // the exit state: of a sequence's end, or the sum at a boundary
  float* out = nullptr;
  if (!OUT)
    out = R.bound + ((size_t)(REV ? it.prev : it.next) * a.Hv + hv) * D * D;
  else if ((REV ? it.prev : it.next) < 0 && R.exit)
    out = R.exit + ((size_t)it.seq * a.Hv + hv) * D * D;
  if (out) {
#pragma unroll
    for (int b = 0; b < NDV; ++b)
#pragma unroll
      for (int c = 0; c < NDU; ++c)
        *reinterpret_cast<f32x4*>(out + (size_t)(w0 + 16 * b + li) * D + 16 * c + 4 * g) = St[b][c];
  }
}

template <typename T, int D, bool OUT> constexpr size_t decay_lds() {
  return (size_t)planes<T>() * 2 * ((OUT ? 3 : 2) * BLK * D + (OUT ? BLK * BLK : 0)) +
         (68 + BLK) * sizeof(float);
}

// ----------------------------------------------------------------- the chain
// Boundary sums to boundary states, in place: each thread four values of one
// head's state, from the sequence's entry (exit gradient, reversed) on.
template <int D>
__global__ __launch_bounds__(256) void decay_chain_kernel(DecayChainArgs a) {
  constexpr int PARTS = D * D / 1024;
  const DecayChainRole& R = a.role[blockIdx.y];
  const int part = blockIdx.x % PARTS, hv = blockIdx.x / PARTS % a.Hv;
  const int m = blockIdx.x / PARTS / a.Hv;
  int seq, slot0, cnt, last;
  if (a.plan.table) {
    if (m >= a.plan.table[1]) return;
    const int* e = a.plan.table + kDecayHead + a.plan.max_items * kDecayItem + m * kDecayMulti;
    seq = e[0], slot0 = e[1], cnt = e[2], last = e[3];
  } else {
    seq = m, cnt = a.plan.P - 1, slot0 = m * cnt, last = a.plan.T - cnt * a.plan.L;
  }
  const int at = part * 1024 + threadIdx.x * 4;
  const float alpha = a.decay[hv];
  const float aL = decay_pow(alpha, a.plan.L);
  float f = R.rev ? decay_pow(alpha, last) : aL;
  f32x4 X = {0.f, 0.f, 0.f, 0.f};
  if (R.state) {
    const float* E = R.state + ((size_t)seq * a.Hv + hv) * D * D;
    if (R.tr_state) {
#pragma unroll
      for (int e = 0; e < 4; ++e) X[e] = E[(size_t)((at + e) % D) * D + (at + e) / D];
    } else {
      X = *reinterpret_cast<const f32x4*>(E + at);
    }
  }
  const size_t pitch = (size_t)a.Hv * D * D;
  float* p = R.bound + (size_t)slot0 * pitch + (size_t)hv * D * D + at;
  constexpr int U = 8;  // boundaries in flight
  for (int j0 = 0; j0 < cnt; j0 += U) {
    f32x4 n[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = min(j0 + u, cnt - 1);
      n[u] = *reinterpret_cast<const f32x4*>(p + (size_t)(R.rev ? cnt - 1 - j : j) * pitch);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u;
      if (j >= cnt) break;
      X = X * f + n[u];
      f = aL;
      *reinterpret_cast<f32x4*>(p + (size_t)(R.rev ? cnt - 1 - j : j) * pitch) = X;
    }
  }
}

// ------------------------------------------------- gradients of shared heads
// y[row][hk] = the sum over its group of part[row][hk group + j], in order, for
// the rows that sequences have.
template <typename T>
__global__ __launch_bounds__(256) void decay_group_kernel(DecayGroupArgs a, int D4) {
  const float* part = a.part[blockIdx.y];
  T* y = reinterpret_cast<T*>(a.y[blockIdx.y]);
  long long i = 0, n4 = (long long)a.n_tok * a.Hk * D4;
  if (a.plan.table) {
    i = (long long)a.plan.table[2] * a.Hk * D4;
    n4 = (long long)a.plan.table[3] * a.Hk * D4;
  }
  for (i += (long long)blockIdx.x * 256 + threadIdx.x; i < n4; i += (long long)gridDim.x * 256) {
    const long long row = i / D4;
    const f32x4* p = reinterpret_cast<const f32x4*>(part) + row * a.group * D4 + (i - row * D4);
    f32x4 s = p[0];
    for (int j = 1; j < a.group; ++j) s += p[(size_t)j * D4];
    st4(y + 4 * i, s[0], s[1], s[2], s[3]);
  }
}

// -------------------------------------------------------------------- launch
static hipError_t decay_plan(const DecayPlan& p, const int* seq_start, int n_seq, int n_tok,
                             hipStream_t st, Profiler* prof) {
  if (!p.table) return hipSuccess;
  prof_begin(prof, "decay_plan", st);
  hipLaunchKernelGGL(decay_plan_kernel, dim3(1), dim3(1024), 0, st, seq_start, n_seq, n_tok, p.L,
                     p.max_items, p.table);
  prof_end(prof, st);
  return hipGetLastError();
}

template <typename T, int D, bool REV, bool OUT>
static hipError_t decay_scan(const DecayScanArgs& a, int roles, const char* name, hipStream_t st,
                             Profiler* prof) {
  constexpr size_t lds = decay_lds<T, D, OUT>();
  const void* fn = (const void*)decay_scan_kernel<T, D, REV, OUT>;
  hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  prof_begin(prof, name, st);
  hipLaunchKernelGGL((decay_scan_kernel<T, D, REV, OUT>),
                     dim3((unsigned)(a.plan.max_items * a.Hv), roles), dim3(DECAY_NT), lds, st, a);
  prof_end(prof, st);
  return hipGetLastError();
}

template <int D>
static hipError_t decay_chain(const DecayChainArgs& a, int roles, hipStream_t st, Profiler* prof) {
  prof_begin(prof, "decay_chain", st);
  hipLaunchKernelGGL((decay_chain_kernel<D>),
                     dim3((unsigned)(a.plan.max_multi * a.Hv * (D * D / 1024)), roles), dim3(256), 0,
                     st, a);
  prof_end(prof, st);
  return hipGetLastError();
}

template <typename T, int D>
hipError_t launch_decay_fwd(const DecayArgs& d, hipStream_t st, Profiler* prof) {
  hipError_t e;
  if ((e = decay_plan(d.plan, d.seq_start, d.n_seq, d.n_tok, st, prof)) != hipSuccess) return e;
  DecayScanArgs a{};
  a.plan = d.plan;
  a.decay = d.decay;
  a.Hv = d.Hv;
  a.group = d.group;
  DecayRole& r = a.role[0];
  r.x = {d.q, d.qs, 1};
  r.u = {d.k, d.ks, 1};
  r.w = {d.v, d.vs, 0};
  r.y = d.o;
  r.y_f32 = sizeof(T) == 4;
  r.bound = d.bound[0];
  r.state = d.S_in;
  r.exit = d.S_out;
  r.s_out = d.scale;
  r.s_pair = 1.f;
  if (d.plan.max_multi > 0) {
    if ((e = decay_scan<T, D, false, false>(a, 1, "decay_sum", st, prof)) != hipSuccess) return e;
    DecayChainArgs c{};
    c.plan = d.plan;
    c.decay = d.decay;
    c.Hv = d.Hv;
    c.role[0] = DecayChainRole{d.bound[0], d.S_in, 0, 0};
    if ((e = decay_chain<D>(c, 1, st, prof)) != hipSuccess) return e;
  }
  return decay_scan<T, D, false, true>(a, 1, "decay_scan", st, prof);
}

template <typename T, int D>
hipError_t launch_decay_bwd(const DecayArgs& d, hipStream_t st, Profiler* prof) {
  hipError_t e;
  if ((e = decay_plan(d.plan, d.seq_start, d.n_seq, d.n_tok, st, prof)) != hipSuccess) return e;
  const DecayTensor q{d.q, d.qs, 1}, k{d.k, d.ks, 1}, v{d.v, d.vs, 0},
      dO{d.dO, (long long)d.Hv * D, 0};
  const bool part = d.group > 1;
  const int f32 = part || sizeof(T) == 4;
  DecayScanArgs f{}, b{};
  f.plan = b.plan = d.plan;
  f.decay = b.decay = d.decay;
  f.Hv = b.Hv = d.Hv;
  f.group = b.group = d.group;
  // dq: the forward scan of S^T
  f.role[0] = DecayRole{dO, v, k, part ? (void*)d.part[0] : d.dq, f32, d.bound[0], d.S_in, nullptr,
                        d.scale, 1.f, 1, 0};
  // dv and dk: the reversed scan of G and of G^T, from the same boundaries
  b.role[0] = DecayRole{k, q, dO, d.dv, sizeof(T) == 4, d.bound[1], d.dS_out, d.dS_in, 1.f, d.scale,
                        0, 0};
  b.role[1] = DecayRole{v, dO, q, part ? (void*)d.part[1] : d.dk, f32, d.bound[1], d.dS_out, nullptr,
                        1.f, d.scale, 1, 1};
  if (d.plan.max_multi > 0) {
    if ((e = decay_scan<T, D, false, false>(f, 1, "decay_sum", st, prof)) != hipSuccess) return e;
    if ((e = decay_scan<T, D, true, false>(b, 1, "decay_sum_rev", st, prof)) != hipSuccess) return e;
    DecayChainArgs c{};
    c.plan = d.plan;
    c.decay = d.decay;
    c.Hv = d.Hv;
    c.role[0] = DecayChainRole{d.bound[0], d.S_in, 1, 0};
    c.role[1] = DecayChainRole{d.bound[1], d.dS_out, 0, 1};
    if ((e = decay_chain<D>(c, 2, st, prof)) != hipSuccess) return e;
  }
  if ((e = decay_scan<T, D, false, true>(f, 1, "decay_scan_dq", st, prof)) != hipSuccess) return e;
  if ((e = decay_scan<T, D, true, true>(b, 2, "decay_scan_dkv", st, prof)) != hipSuccess) return e;
  if (!part || d.n_tok == 0) return hipSuccess;
  DecayGroupArgs g{};
  g.plan = d.plan;
  g.part[0] = d.part[0];
  g.part[1] = d.part[1];
  g.y[0] = d.dq;
  g.y[1] = d.dk;
  g.n_tok = d.n_tok;
  g.Hk = d.Hv / d.group;
  g.group = d.group;
  const long long n = (long long)g.n_tok * g.Hk * (D / 4), blocks = (n + 255) / 256;
  prof_begin(prof, "decay_group", st);
  hipLaunchKernelGGL((decay_group_kernel<T>), dim3((unsigned)(blocks < 8192 ? blocks : 8192), 2),
                     dim3(256), 0, st, g, D / 4);
  prof_end(prof, st);
  return hipGetLastError();
}

#define SF_INST(T, D)                                                              \
  template hipError_t launch_decay_fwd<T, D>(const DecayArgs&, hipStream_t, Profiler*); \
  template hipError_t launch_decay_bwd<T, D>(const DecayArgs&, hipStream_t, Profiler*);
SF_INST(bf16, 64)
SF_INST(bf16, 128)
SF_INST(float, 64)
SF_INST(float, 128)
#undef SF_INST

}  // namespace sfgdn
