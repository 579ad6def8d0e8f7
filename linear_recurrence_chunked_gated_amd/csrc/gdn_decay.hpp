// Linear attention with a fixed decay a for each head, over whole prompts or
// training chunks: sequences of one length or packed ones of different
// lengths, and the gradients.
//
//     S_t = a S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t
//
// In blocks of C = 64 tokens (fp32: 32; n of them valid), r and s local, entry
// state E:
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
//   decay_chain   those to the states at the boundaries, one after another; where
//                 there are few, every item does that for its own boundary
//   decay_scan    every item from its entry state: the outputs, and the last
//                 (first) item's exit state
// with the scans of all roles in one launch, and so the sums (dv's and dk's
// boundaries are the same).
#pragma once
#include "gdn_kernels.hpp"

namespace sfgdn {

// One item: a segment of a sequence.  prev, next: the boundary slots before
// and after it (-1 at the sequence's ends).  Without a table: how many
// boundaries there are before and after it, and the last segment's tokens.
struct DecayItem {
  int seq, t0, n, prev, next, before, after, last;
};

// Packed sequences: offsets are taken as their running maximum, clamped to the
// token rows, so that items never overlap or reach outside them, whatever
// seq_start holds.
__device__ __forceinline__ int decay_offset(const DecayPlan& p, int i) {
  return min(max(p.seq_start[i], 0), p.n_tok);
}
// The last segments' rank falls with their blocks (by the power of two): the
// longer ones come first, so that no long item is left for the end.
__device__ __forceinline__ int decay_rank(int tokens) { return __clz((tokens + BLK - 1) / BLK); }

// x joined with the lanes before: rows of 16, then their ends to the next ones.
template <typename F> __device__ __forceinline__ int wave_scan(int x, int ident, F join) {
  x = join(x, __builtin_amdgcn_update_dpp(ident, x, 0x111, 0xF, 0xF, false));
  x = join(x, __builtin_amdgcn_update_dpp(ident, x, 0x112, 0xF, 0xF, false));
  x = join(x, __builtin_amdgcn_update_dpp(ident, x, 0x114, 0xF, 0xF, false));
  x = join(x, __builtin_amdgcn_update_dpp(ident, x, 0x118, 0xF, 0xF, false));
  x = join(x, __builtin_amdgcn_update_dpp(ident, x, 0x142, 0xA, 0xF, false));
  return join(x, __builtin_amdgcn_update_dpp(ident, x, 0x143, 0xC, 0xF, false));
}

// Up to 64 sequences, one a lane: every wave plans for itself, which takes less
// than a kernel before the others would (9 sequences, 4099 tokens in all, 6 heads
// at D = 64 in fp32: 33.6 us with one, 28.6 so; backward 51 and 47).
struct DecaySeqs {
  int t0, t1, cnt, slot0;  // its rows, its whole segments before the last, their first slot
  __device__ __forceinline__ DecaySeqs(const DecayPlan& p) {
    const int i = lane_id();
    const bool live = i < p.n_seq;
    const int x = live ? decay_offset(p, i) : 0, y = live ? decay_offset(p, i + 1) : 0;
    t0 = wave_scan(x, 0, [](int a, int b) { return max(a, b); });
    t1 = max(t0, y);
    cnt = live && t1 > t0 ? (t1 - t0 - 1) / p.L : 0;
    slot0 = wave_scan(cnt, 0, [](int a, int b) { return a + b; }) - cnt;
  }
};

// Item i (none: a negative sequence).  Packed: 0 .. max_slots-1 are the whole
// segments, by their boundary slot, then each sequence's last one, by its rank.
__device__ __forceinline__ DecayItem decay_item(const DecayPlan& p, int i) {
  if (p.table) {
    const int* e = p.table + kDecayHead + i * kDecayItem;
    return DecayItem{i >= p.table[0] && i < p.max_slots ? -1 : e[0], e[1], e[2], e[3], e[4], 0, 0, 0};
  }
  int seq, t0, len, first, cnt, j;
  if (p.seq_start) {
    const DecaySeqs s(p);
    unsigned long long in = __ballot(i >= s.slot0 && i < s.slot0 + s.cnt);
    if (i >= p.max_slots) {
      const int rank = lane_id() < p.n_seq ? decay_rank(s.t1 - s.t0 - s.cnt * p.L) : -1;
      int before = i - p.max_slots;
      for (int r = decay_rank(p.L); r <= 32; ++r) {
        in = __ballot(rank == r);
        const int n = __builtin_popcountll(in);
        if (before < n) break;
        before -= n;
      }
      for (; before > 0; --before) in &= in - 1;
    }
    seq = in ? __builtin_ctzll(in) : 0;
    t0 = __builtin_amdgcn_readlane(s.t0, seq);
    len = __builtin_amdgcn_readlane(s.t1, seq) - t0;
    first = __builtin_amdgcn_readlane(s.slot0, seq);
    cnt = __builtin_amdgcn_readlane(s.cnt, seq);
    j = i < p.max_slots ? i - first : cnt;
    if (!in) seq = -1;
  } else {
    seq = i / p.P;
    j = i - seq * p.P;
    t0 = seq * p.T;
    len = p.T;
    cnt = p.P - 1;
    first = seq * cnt;
  }
  const int last = len - cnt * p.L;
  return DecayItem{seq, t0 + j * p.L, j < cnt ? p.L : last, j > 0 ? first + j - 1 : -1,
                   j < cnt ? first + j : -1, j, cnt - j, last};
}

// a^e for e >= 0, by squaring in 64 bits: exact to a rounding for every a,
// 0 and values near 1 among them.
__device__ __forceinline__ double decay_pow64(float a, int e) {
  double r = 1.0, b = a;
  while (e > 0) {
    if (e & 1) r *= b;
    b *= b;
    e >>= 1;
  }
  return r;
}
__device__ __forceinline__ float decay_pow(float a, int e) { return (float)decay_pow64(a, e); }

// A segment's decay in 48 bits, and a boundary's state behind it: x a^n + sum.
// (In fp32 it is off to the same side at every boundary of a long chain.)
struct DecayFactor {
  float hi, lo;
  __device__ __forceinline__ DecayFactor(float a, int n) {
    const double p = decay_pow64(a, n);
    hi = (float)p;
    lo = (float)(p - (double)hi);
  }
  __device__ __forceinline__ f32x4 join(f32x4 x, f32x4 sum) const {
    f32x4 y;
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = __builtin_fmaf(x[e], hi, __builtin_fmaf(x[e], lo, sum[e]));
    return y;
  }
};

// ------------------------------------------------------------------ the plan
// Items and boundary slots of more packed sequences, by one workgroup.
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

__global__ __launch_bounds__(1024) void decay_plan_kernel(DecayPlan p) {
  __shared__ int lds[16];
  __shared__ int bucket[32];
  auto add = [](int a, int b) { return a + b; };
  auto most = [](int a, int b) { return max(a, b); };
  int* items = p.table + kDecayHead;
  int* multi = items + p.max_items * kDecayItem;
  const int n_seq = p.n_seq;
  if (threadIdx.x < 32) bucket[threadIdx.x] = 0;
  // once over the sequences to count the buckets, once to write
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    int end = 0, n_slots = 0, n_multi = 0;
    __syncthreads();
    if (pass == 1 && threadIdx.x == 0) {
      int at = p.max_slots;
      for (int i = 0; i < 32; ++i) {
        const int n = bucket[i];
        bucket[i] = at;
        at += n;
      }
    }
    __syncthreads();
    for (int base = 0; base < n_seq; base += 1024) {
      const int i = base + threadIdx.x;
      const bool live = i < n_seq;
      const int x = live ? decay_offset(p, i) : 0;
      int top, slots, multis;
      const int t0 = max(end, scan1024(x, lds, 0, most, top));
      const int t1 = live ? max(t0, decay_offset(p, i + 1)) : t0;
      end = max(end, top);
      const int len = t1 - t0, cnt = live && len > 0 ? (len - 1) / p.L : 0;
      const int last = len - cnt * p.L;
      if (pass == 0) {
        if (live) atomicAdd(&bucket[decay_rank(last) & 31], 1);
        continue;
      }
      const int slot0 = n_slots + scan1024(cnt, lds, 0, add, slots) - cnt;
      const int m = n_multi + scan1024(cnt > 0, lds, 0, add, multis) - (cnt > 0);
      for (int j = 0; j < cnt; ++j) {
        int* e = items + (slot0 + j) * kDecayItem;
        e[0] = i;
        e[1] = t0 + j * p.L;
        e[2] = p.L;
        e[3] = j > 0 ? slot0 + j - 1 : -1;
        e[4] = slot0 + j;
      }
      if (live) {
        int* e = items + atomicAdd(&bucket[decay_rank(last) & 31], 1) * kDecayItem;
        e[0] = i;
        e[1] = t0 + cnt * p.L;
        e[2] = last;
        e[3] = cnt > 0 ? slot0 + cnt - 1 : -1;
        e[4] = -1;
      }
      if (cnt > 0) {
        int* e = multi + m * kDecayMulti;
        e[0] = i;
        e[1] = slot0;
        e[2] = cnt;
        e[3] = last;
      }
      n_slots += slots;
      n_multi += multis;
    }
    if (pass == 1 && threadIdx.x == 0) {
      p.table[0] = n_slots;
      p.table[1] = n_multi;
      p.table[2] = n_seq > 0 ? decay_offset(p, 0) : 0;  // the rows that sequences have
      p.table[3] = max(end, n_seq > 0 ? decay_offset(p, n_seq) : 0);
    }
  }
}

// --------------------------------------------------------------------- tiles
// Operands are bf16 planes: a bf16 tensor is one, an fp32 tensor three, x = x0
// + x1 + x2 with what each plane leaves of the one before (24 bits).  Products
// run over the pairs of planes down to 2^-16 of the first, summed in fp32, the
// smallest first: six for two fp32 tensors, whose results differ from exact
// products of fp32 by less than the sums do (fp32 matrix instructions have a
// sixteenth of the rate).
template <typename T> struct DecayKind;
template <> struct DecayKind<bf16> {
  static constexpr int C = 64;  // tokens of a block
  static constexpr int NP = 1;  // planes of a tensor
  static constexpr int NY = 2;  // planes of P and of the state's copy, on the way to bf16 outputs
};
template <> struct DecayKind<float> {
  static constexpr int C = 32;
  static constexpr int NP = 3;
  static constexpr int NY = 3;
};

template <int NA, int NB>
__device__ __forceinline__ f32x4 mma_planes(const bf16x8 (&a)[NA], const bf16x8 (&b)[NB], f32x4 c) {
  constexpr int N = NA > NB ? NA : NB;
#pragma unroll
  for (int n = N - 1; n >= 0; --n)
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (n - i >= 0 && n - i < NB) c = Mma<bf16>::mma(a[i], b[n - i], c);
  return c;
}

// acc(i, j) += a[i] b[j] over all tiles, pair of planes by pair of planes, so
// that as many products as there are tiles lie between two into one of them.
template <int M, int N, int NA, int NB, typename F>
__device__ __forceinline__ void mma_grid(const bf16x8 (&a)[M][NA], const bf16x8 (&b)[N][NB], F acc) {
  constexpr int K = NA > NB ? NA : NB;
#pragma unroll
  for (int n = K - 1; n >= 0; --n)
#pragma unroll
    for (int p = 0; p < NA; ++p)
      if (n - p >= 0 && n - p < NB)
#pragma unroll
        for (int i = 0; i < M; ++i)
#pragma unroll
          for (int j = 0; j < N; ++j) acc(i, j) = Mma<bf16>::mma(a[i][p], b[j][n - p], acc(i, j));
}

// N values to planes, a pair at a time.
typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
template <int N, int K, typename V>
__device__ __forceinline__ void to_planes(const float (&x)[N], V (&f)[K]) {
#pragma unroll
  for (int j = 0; j < N; j += 2) {
    float a = x[j], b = x[j + 1];
#pragma unroll
    for (int p = 0; p < K; ++p) {
      const bf16x2 h = __builtin_convertvector((f32x2{a, b}), bf16x2);
      f[p][j] = h[0];
      f[p][j + 1] = h[1];
      if (p + 1 < K) {
        const unsigned u = __builtin_bit_cast(unsigned, h);
        a -= __uint_as_float(u << 16);
        b -= __uint_as_float(u & 0xffff0000u);
      }
    }
  }
}

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
template <typename V> __device__ __forceinline__ auto lds_at(unsigned at) {
  typedef __attribute__((address_space(3))) V lds_t;
  return (lds_t*)(size_t)at;
}
// 16-byte units of a lane's transpose read (see ds_tr4)
__device__ __forceinline__ bf16x4 lds_tr4(unsigned at) {
  return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(lds_at<i16x4>(at)));
}

constexpr int DECAY_NW = 4;  // waves of a workgroup

// A block's rows of D values in LDS, in planes of C x D bf16, each row's
// 16-byte units permuted as by lds_sw.
template <typename T, int D> struct DecayTile {
  static constexpr int C = DecayKind<T>::C, NP = DecayKind<T>::NP, NT = 64 * DECAY_NW;
  static constexpr int RB = 2 * D, BYTES = C * RB;  // of a plane's row, of a plane
  static constexpr int NW16 = sizeof(T) / 2;        // 16-byte loads for 16 bytes of a plane
  static constexpr int VEC = 16 / (int)sizeof(T), CPR = D / VEC, RPT = NT / CPR, NCH = C / RPT;
  static constexpr __host__ __device__ int swizzle(int row) {
    return D == 128 ? row & 15 : (row >> 1) & 7;
  }
  static_assert(C % RPT == 0, "a tile splits evenly over the workgroup");

  // A thread's first piece of a tile and the bytes to its next ones.
  struct Rows {
    unsigned at, step;
    __device__ __forceinline__ Rows(long long stride) {
      at = (unsigned)((threadIdx.x / CPR * stride + threadIdx.x % CPR * VEC) * sizeof(T));
      step = (unsigned)(RPT * stride * sizeof(T));
    }
  };
  // Rows 0 .. nv-1 of a block: past them a load gives zeros and a store is
  // dropped.  (A block spans less than 2^31 bytes: the strides are checked.)
  __device__ static __forceinline__ __amdgpu_buffer_rsrc_t block(const T* g, long long stride, int nv) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(g), 0,
                                             (int)(((nv - 1) * stride + D) * sizeof(T)), 0x00020000);
  }
  __device__ static __forceinline__ void load(u32x4 (&r)[NCH], const Rows& o, __amdgpu_buffer_rsrc_t g) {
#pragma unroll
    for (int it = 0; it < NCH; ++it)
      r[it] = __builtin_bit_cast(
          u32x4, __builtin_amdgcn_raw_buffer_load_b128(g, (int)(o.at + it * o.step), 0, 0));
  }
  // at: the tile's LDS address
  __device__ static __forceinline__ unsigned piece(unsigned at) {
    const int row = threadIdx.x / CPR, b = threadIdx.x % CPR * 16 / NW16;  // byte in a plane's row
    return at + row * RB + ((b & ~15) ^ (swizzle(row) << 4)) + (b & 15);
  }
  static __device__ __forceinline__ unsigned piece_of(unsigned p, int it) {
    static_assert(RPT >= 8 && (RPT & (RPT - 1)) == 0, "row + RPT it: bits of their own");
    return (p ^ swizzle(RPT * it) << 4) + it * RPT * RB;
  }
  __device__ static __forceinline__ void to_lds(const u32x4 (&r)[NCH], unsigned at) {
    const unsigned p = piece(at);
#pragma unroll
    for (int it = 0; it < NCH; ++it) {
      const unsigned q = piece_of(p, it);
      if constexpr (NP == 1) {
        *lds_at<u32x4>(q) = r[it];
      } else {
        const f32x4 f = __builtin_bit_cast(f32x4, r[it]);
        const float x[4] = {f[0], f[1], f[2], f[3]};
        bf16x4 h[NP];
        to_planes(x, h);
#pragma unroll
        for (int i = 0; i < NP; ++i) *lds_at<bf16x4>(q + i * BYTES) = h[i];
      }
    }
  }
  // The tile's first plane to a block's rows, each thread the pieces that it
  // writes itself in to_lds (so that needs no barrier after this).
  __device__ static __forceinline__ void rows_out(const Rows& o, __amdgpu_buffer_rsrc_t g, unsigned at) {
    const unsigned p = piece(at);
#pragma unroll
    for (int it = 0; it < NCH; ++it)
      __builtin_amdgcn_raw_buffer_store_b128(*lds_at<u32x4>(piece_of(p, it)), g,
                                             (int)(o.at + it * o.step), 0, 0);
  }
  // Operand reads.  The swizzle changes address bits that a lane's row decides,
  // the same for every tile of 16 rows, so a lane has one base for each form
  // of read and the rest is a constant to XOR and one to add (which the read
  // takes as its offset): without that, some hundred addresses would each
  // want a register.
  struct Lane {
    unsigned std, perm, col;
    __device__ __forceinline__ Lane() {
      const int l = lane_id(), g = l >> 4, i = l & 15, r = 8 * g + (i >> 2);
      std = i * RB + ((g ^ swizzle(i)) << 4);
      perm = i * RB + (((g >> 1) ^ swizzle(i)) << 4) + 8 * (g & 1);
      col = r * RB + (((i >> 1 & 1) ^ swizzle(r)) << 4) + 8 * (i & 1);
    }
    // not kept in registers per use over the blocks
    __device__ __forceinline__ void fresh() {
      __asm__ volatile("" : "+v"(std), "+v"(perm), "+v"(col));
    }
  };
  // operand rows from row0 (a multiple of 16), contraction along the row
  __device__ static __forceinline__ void rows_std(const Lane& l, unsigned at, int row0, int step,
                                                  bf16x8 (&f)[NP]) {
#pragma unroll
    for (int p = 0; p < NP; ++p)
      f[p] = *lds_at<bf16x8>((l.std ^ step << 6) + (at + p * BYTES + row0 * RB));
  }
  __device__ static __forceinline__ void rows_perm(const Lane& l, unsigned at, int row0, int step,
                                                   bf16x8 (&f)[NP]) {
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const unsigned o = at + p * BYTES + row0 * RB;
      const bf16x4 lo = *lds_at<bf16x4>((l.perm ^ step << 6) + o);
      const bf16x4 hi = *lds_at<bf16x4>((l.perm ^ step << 6 ^ 32) + o);
      f[p] = bf16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    }
  }
  // operand rows = columns 16 c .., contraction along the tokens
  __device__ static __forceinline__ void cols(const Lane& l, unsigned at, int c, int step,
                                              bf16x8 (&f)[NP]) {
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const unsigned o = at + p * BYTES + 32 * step * RB;
      const bf16x4 lo = lds_tr4((l.col ^ c << 5) + o);
      const bf16x4 hi = lds_tr4((l.col ^ c << 5 ^ swizzle(4) << 4) + (o + 4 * RB));
      f[p] = bf16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    }
  }
};

// P: rows r of C bf16, in planes.
template <int C> struct DecayP {
  static constexpr int RB = 2 * C, BYTES = C * RB;
  static_assert(C == 64 || C == 32, "rows of 128 bytes are swizzled, rows of 64 lie as they are");
  struct Lane {
    unsigned w, r;
    __device__ __forceinline__ Lane() {
      const int l = lane_id(), g = l >> 4, i = l & 15, x = C == 64 ? i >> 1 : 0;
      w = i * RB + (((g >> 1) ^ x) << 4) + 8 * (g & 1);
      r = i * RB + ((g ^ x) << 4);
    }
    __device__ __forceinline__ void fresh() { __asm__ volatile("" : "+v"(w), "+v"(r)); }
  };
  // four s from 16 st + 4 g of row r = 16 rt + lane
  template <int K>
  __device__ static __forceinline__ void store(const Lane& l, unsigned at, int rt, int st,
                                               const bf16x4 (&h)[K]) {
#pragma unroll
    for (int p = 0; p < K; ++p)
      *lds_at<bf16x4>((l.w ^ st << 5) + (at + p * BYTES + 16 * rt * RB)) = h[p];
  }
  template <int K>
  __device__ static __forceinline__ void rows(const Lane& l, unsigned at, int rt, int step,
                                              bf16x8 (&f)[K]) {
#pragma unroll
    for (int p = 0; p < K; ++p)
      f[p] = *lds_at<bf16x8>((l.r ^ step << 6) + (at + p * BYTES + 16 * rt * RB));
  }
};

// Workgroups go to the 8 XCDs in turn, each with an L2 of its own: the roles
// and the heads of a group, which read the same rows, are a key head's
// consecutive workgroups on one XCD.
__device__ __forceinline__ void decay_unit(const DecayScanArgs& a, int& role, int& hk, int& hv,
                                           int& item) {
  int y = blockIdx.x / kXcds;
  role = y % a.roles;
  y /= a.roles;
  const int i = y % a.group, Hk = a.Hv / a.group;
  y = y / a.group * kXcds + blockIdx.x % kXcds;
  hk = y % Hk;
  hv = hk * a.group + i;
  item = y / Hk;
}

// ------------------------------------------------------------------ the scan
// Workgroup: one item of one value head, four waves.  Wave w owns NB tiles of
// 16 columns of the state (its w index), held transposed in accumulators: tile
// [b][c] has m = the u index (16 c ..), n = the w index (16 (NB w + b) ..).
//
// Roundings to fewer bits, for bf16 tensors: P, the state's copy that meets x
// and w times its decay, which the state sums, go in two planes (2^-16), so that
// outputs are off by their own rounding to bf16 (2^-8) and no more; the last in
// a third (2^-24, all of an fp32 value; NS = 3) where the state ends as an fp32
// output, or in a boundary's sum on the way to one.  For fp32 tensors all of
// these are three planes.  (With P and the state's copy as plain bf16 the outputs
// of 65,536 tokens, 16 heads, D = 128 are 1.4 times as far off, 0.0023 relative
// rms for 0.0017; the scan takes 245 us then and 283 so, of a backward of 32,768
// tokens 310 and 357, of 24 packed prompts 131 and 151.)
//
// Four waves and two workgroups a compute unit, at up to 256 registers: the
// state, O and the next block's rows fill them (eight waves with half the columns
// each were slower, their operand reads twice as many; of the instances at
// D = 128 those whose items all end in an output spill 6 to 9 registers).
// Measured in bf16 at D = 128: 65,536 tokens of 16 heads take 137 us for the sums
// (4.2 TB/s) and 283 for the scan (3.9 TB/s); a block takes 8.9 us of a
// workgroup's time, with the matrix units busy for 37% of it (32% where 32 heads
// share 16 key heads: 3.1 TB/s), the vector units for 48% and LDS for 44%: the
// chain of steps between barriers bounds it, not one of them.  (A third of LDS's
// cycles are bank conflicts, most of them of the transpose reads, whose rows r and
// r + 1 meet; a swizzle that moves rows by pairs of units ends those, and with two
// more spilled registers was no faster: scan 243-247 us for 243-249, with P and
// the state's copy in one plane.)  fp32 (six products for one) 890 us for both,
// bound by the products.
//
// OUT: a scan; otherwise the sum for a boundary, which is the same whatever
// order its blocks come in.  They come in the opposite order of the scan's, so
// that what it reads first is what was read last and (256 MB of it) is still
// in the last-level cache.
template <typename T, int D, bool REV, bool OUT, int NS>
__device__ __forceinline__ void decay_scan_item(const DecayScanArgs& a, const DecayRole& R, int hk,
                                                int hv, int unit) {
  typedef DecayTile<T, D> Tl;
  constexpr int C = Tl::C, NP = Tl::NP, NY = DecayKind<T>::NY, NT = Tl::NT;
  constexpr int NW = NT / 64, NB = D / 16 / NW, NU = D / 16, KD = D / 32, KT = C / 32, NR = C / 16;
  typedef DecayP<C> Pl;
  // LDS (it starts at 0: there is no other): u, w, x, P, then the powers
  constexpr unsigned aU = 0, aW = NP * Tl::BYTES, aX = 2 * aW, aP = 3 * aW;
  constexpr unsigned aF = OUT ? aP + NY * Pl::BYTES : aX;
  extern __shared__ __align__(16) unsigned char smem[];
  float* pw = reinterpret_cast<float*>(smem + aF);  // a^0 .. a^C, and what a^C's rounding left
  float* dec = pw + C + 4;                          // [C]

  if (unit >= a.plan.max_items) return;
  const DecayItem it = decay_item(a.plan, unit);
  if (it.seq < 0) return;
  if (!OUT && (REV ? it.prev : it.next) < 0) return;  // no boundary behind this item
  const int w = wave_id(), lane = lane_id(), g = lane >> 4, li = lane & 15;
  const int w0 = 16 * NB * w;  // this wave's first state column
  const float alpha = a.decay[hv];

  const long long xst = R.x.stride, ust = R.u.stride, wst = R.w.stride;
  const T* xg = nullptr;
  if constexpr (OUT) xg = reinterpret_cast<const T*>(R.x.p) + it.t0 * xst + (R.x.shared ? hk : hv) * D;
  const T* ug = reinterpret_cast<const T*>(R.u.p) + it.t0 * ust + (R.u.shared ? hk : hv) * D;
  const T* wg = reinterpret_cast<const T*>(R.w.p) + it.t0 * wst + (R.w.shared ? hk : hv) * D;

  const int nblk = (it.n + C - 1) / C;
  const typename Tl::Rows ox(xst), ou(ust), ow(wst);
  u32x4 rx[OUT ? Tl::NCH : 1], ru[Tl::NCH], rw[Tl::NCH];
  auto fetch = [&](int b) {
    const int nv = min(C, it.n - b * C);
    const long long t = (long long)b * C;
    Tl::load(ru, ou, Tl::block(ug + t * ust, ust, nv));
    if constexpr (OUT) Tl::load(rx, ox, Tl::block(xg + t * xst, xst, nv));
    Tl::load(rw, ow, Tl::block(wg + t * wst, wst, nv));
  };
  constexpr bool DOWN = REV == OUT;  // from the last block to the first
  if (nblk > 0) fetch(DOWN ? nblk - 1 : 0);

  f32x4 St[NB][NU];
  {
    const int slot = REV ? it.next : it.prev;
    const float* E = nullptr;
    bool tr = R.tr_state;
    if (OUT) {
      if (slot >= 0 && !a.plan.direct) {
        E = R.bound + ((size_t)slot * a.Hv + hv) * D * D;
        tr = R.tr_bound;
      } else if (R.state) {
        E = R.state + ((size_t)it.seq * a.Hv + hv) * D * D;
      }
    }
    auto entry = [&](const float* E, bool tr, int b, int c) {
      const int m = 16 * c + 4 * g, n = w0 + 16 * b + li;
      f32x4 x = {0.f, 0.f, 0.f, 0.f};
      if (E && tr) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = E[(size_t)(m + e) * D + n];
      } else if (E) {
        x = *reinterpret_cast<const f32x4*>(E + (size_t)n * D + m);
      }
      return x;
    };
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int c = 0; c < NU; ++c) St[b][c] = entry(E, tr, b, c);
    if (OUT && slot >= 0 && a.plan.direct) {  // the chain up to this item's boundary
      const DecayFactor aL(alpha, a.plan.L);
      DecayFactor f = REV ? DecayFactor(alpha, it.last) : aL;
      const int n = REV ? it.after : it.before;
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        const float* B = R.bound + ((size_t)(REV ? slot + n - 1 - i : slot - n + 1 + i) * a.Hv + hv) * D * D;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int c = 0; c < NU; ++c) St[b][c] = f.join(St[b][c], entry(B, R.tr_bound, b, c));
        f = aL;
      }
    }
  }

  // powers; P tiles that the mask empties but a product of 32 tokens reads
  const float s_pair = R.s_pair, s_out = R.s_out;
  if (threadIdx.x <= C) {
    // (past the item's tokens none is used, but would meet the zeros behind them:
    // one that overflows would make those NaN)
    const double p = threadIdx.x <= it.n ? decay_pow64(alpha, threadIdx.x) : 0.0;
    pw[threadIdx.x] = (float)p;
    if (threadIdx.x == C) pw[C + 1] = (float)(p - (double)(float)p);
  }
  if constexpr (OUT) {
    for (int i = threadIdx.x; i < NY * Pl::BYTES / 16; i += NT)
      *lds_at<u32x4>(aP + 16 * i) = u32x4{0, 0, 0, 0};
  }
  lds_barrier();
  // a^(n-1-s) (reversed: a^(s+1)), of whole blocks
  if (threadIdx.x < C) dec[threadIdx.x] = s_pair * pw[REV ? threadIdx.x + 1 : C - 1 - threadIdx.x];
  // This wave's tiles of P that the mask leaves (m = s, n = r): of the operand
  // rows hi[.] (r; reversed: s) with lo[.] <= hi[.].  Of four rows of tiles, two
  // waves take the squares at the diagonal and two the rest, a column each, so
  // that a tile's operands serve two; of two rows a wave takes one tile.  (A
  // tile that a wave has no use for it does twice.)  pf: the factors, 0 where a
  // diagonal tile is masked.
  constexpr int TH = NR / 2, TPW = 2 * TH - 1;
  int hi[TH], lo[TH];
  float pf[TPW][4];
  auto tile_h = [](int i) { return TH == 1 ? 0 : i > 0; };
  auto tile_l = [](int i) { return i / 2; };
  if constexpr (OUT) {
    if constexpr (TH == 2) {
      hi[0] = w == 0 ? 0 : 2;
      lo[0] = w & 2;
      if (w & 1) lo[0] = w >> 1;
      hi[1] = hi[0] + 1;
      lo[1] = lo[0] + (w % 2 == 0);
    } else {
      hi[0] = w > 0;
      lo[0] = w > 1;
    }
#pragma unroll
    for (int i = 0; i < TPW; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d = 16 * (hi[tile_h(i)] - lo[tile_l(i)]) + (REV ? 4 * g + e - li : li - 4 * g - e);
        pf[i][e] = d >= 0 ? s_pair * s_out * pw[d] : 0.f;
      }
  }

  typename Tl::Lane ln;
  typename Pl::Lane lp;
  const double aC = OUT ? 0.0 : decay_pow64(alpha, C);
  const bool exact = R.exit && (REV ? it.prev : it.next) < 0;  // the state ends as an output
  // A scan's state is St times `frame`, which takes the blocks' decays until it
  // leaves 2^-20 .. 2^20 (a sum's block has the decay between it and the
  // boundary instead).  Both take a block's decay in 64 bits (48, in two floats,
  // for a scan: a double in registers makes the instances at D = 128 spill): rounded
  // to fp32 it is off to the same side in every block, over hundreds of them by
  // more than the sums' roundings.
  double frame = 1.0, far = 1.0;
  for (int i = 0; i < nblk; ++i) {
    const int blk = DOWN ? nblk - 1 - i : i;
    const int nv = min(C, it.n - blk * C);
    Tl::to_lds(ru, aU);
    if constexpr (OUT) Tl::to_lds(rx, aX);
    Tl::to_lds(rw, aW);
    ln.fresh();
    lp.fresh();
    if (!REV && nv < C && threadIdx.x < C)  // (w is zero past the end)
      dec[threadIdx.x] = s_pair * pw[max(0, nv - 1 - (int)threadIdx.x)];
    lds_barrier();
    if (i + 1 < nblk) fetch(DOWN ? blk - 1 : blk + 1);

    f32x4 O[NB][NR];
    if constexpr (OUT) {
      f32x4 p[TPW];
#pragma unroll
      for (int i = 0; i < TPW; ++i) p[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < KD; ++s) {
        bf16x8 fu[TH][NP], fx[TH][NP];
#pragma unroll
        for (int i = 0; i < TH; ++i) {
          Tl::rows_std(ln, aU, 16 * (REV ? hi : lo)[i], s, fu[i]);
          Tl::rows_std(ln, aX, 16 * (REV ? lo : hi)[i], s, fx[i]);
        }
#pragma unroll
        for (int i = 0; i < TPW; ++i)
          p[i] = mma_planes(fu[REV ? tile_h(i) : tile_l(i)], fx[REV ? tile_l(i) : tile_h(i)], p[i]);
      }
#pragma unroll
      for (int i = 0; i < TPW; ++i) {
        const float q[4] = {p[i][0] * pf[i][0], p[i][1] * pf[i][1], p[i][2] * pf[i][2],
                            p[i][3] * pf[i][3]};
        bf16x4 h[NY];
        to_planes(q, h);
        const int h_ = hi[tile_h(i)], l_ = lo[tile_l(i)];
        Pl::store(lp, aP, REV ? l_ : h_, REV ? h_ : l_, h);
      }
      // E x
      zero_acc(O);
#pragma unroll
      for (int s = 0; s < KD; ++s) {
        bf16x8 fs[NB][NY];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const f32x4 lo = St[b][2 * s], hi = St[b][2 * s + 1];
          const float x[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
          to_planes(x, fs[b]);
        }
        bf16x8 fx[NR][NP];
#pragma unroll
        for (int j = 0; j < NR; ++j) Tl::rows_perm(ln, aX, 16 * j, s, fx[j]);
        mma_grid(fs, fx, [&](int b, int j) -> f32x4& { return O[b][j]; });
      }
#pragma unroll
      for (int j = 0; j < NR; ++j) {
        const int r = 16 * j + li;
        const float f = s_out * (float)frame * pw[REV ? max(0, nv - 1 - r) : r + 1];
#pragma unroll
        for (int b = 0; b < NB; ++b) O[b][j] *= f;
      }
      lds_barrier();
    }
    // w of this wave's columns: for P w, and scaled for the state
    float fd;
    if constexpr (OUT) {
      frame *= (double)pw[nv] + (nv == C ? (double)pw[C + 1] : 0.0);
      if (!(frame > 0x1p-20 && frame < 0x1p20)) {
        const float f = (float)frame;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int c = 0; c < NU; ++c) St[b][c] *= f;
        frame = 1.0;
      }
      fd = (float)(1.0 / frame);
    } else {
      fd = (float)far;
      far *= aC;
    }
#pragma unroll
    for (int s = 0; s < KT; ++s) {
      bf16x8 fw[NB][NP], fs[NB][NS];
      const f32x4 d0 = fd * *reinterpret_cast<const f32x4*>(dec + 32 * s + 8 * g);
      const f32x4 d1 = fd * *reinterpret_cast<const f32x4*>(dec + 32 * s + 8 * g + 4);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        Tl::cols(ln, aW, NB * w + b, s, fw[b]);
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[j] = (float)fw[b][NP - 1][j];
#pragma unroll
          for (int n = NP - 2; n >= 0; --n) x[j] += (float)fw[b][n][j];
          x[j] *= j < 4 ? d0[j & 3] : d1[j & 3];
        }
        to_planes(x, fs[b]);
      }
      if constexpr (OUT) {
#pragma unroll
        for (int j = 0; j < NR; ++j)
          if (REV ? j < 2 * (s + 1) : j >= 2 * s) {
            bf16x8 fp[NY];
            Pl::rows(lp, aP, j, s, fp);
#pragma unroll
            for (int b = 0; b < NB; ++b) O[b][j] = mma_planes(fw[b], fp, O[b][j]);
          }
      }
      constexpr int CG = 4;  // column tiles at a time
#pragma unroll
      for (int c0 = 0; c0 < NU; c0 += CG) {
        bf16x8 fu[CG][NP];
#pragma unroll
        for (int c = 0; c < CG; ++c) Tl::cols(ln, aU, c0 + c, s, fu[c]);
        mma_grid(fu, fs, [&](int c, int b) -> f32x4& { return St[b][c0 + c]; });
      }
    }
    if constexpr (OUT && NS < 3) {
      if (exact) {  // what the two planes leave
#pragma unroll 1
        for (int s = 0; s < KT; ++s) {
          bf16x8 f3[NB][1];
          const float* dp = dec + 32 * s + 8 * g;
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            bf16x8 fw[NP];
            Tl::cols(ln, aW, NB * w + b, s, fw);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              float x = (float)fw[0][j] * (fd * dp[j]);
              x -= (float)(bf16)x;
              x -= (float)(bf16)x;
              f3[b][0][j] = (bf16)x;
            }
          }
#pragma unroll
          for (int c = 0; c < NU; ++c) {
            bf16x8 fu[1][NP];
            Tl::cols(ln, aU, c, s, fu[0]);
            mma_grid(fu, f3, [&](int, int b) -> f32x4& { return St[b][c]; });
          }
        }
      }
    }
    // y through the x tile to whole rows, or (fp32) straight from the lanes
    const long long yst = (long long)a.Hv * D;
    const size_t y0 = (((size_t)it.t0 + blk * C) * a.Hv + hv) * D;
    const bool rows = OUT && sizeof(T) == 2 && !R.y_f32;
    if constexpr (OUT) {
      if (rows) {
#pragma unroll
        for (int j = 0; j < NR; ++j)
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const f32x4 y = O[b][j];
            const float q[4] = {y[0], y[1], y[2], y[3]};
            bf16x4 h[1];
            to_planes(q, h);
            *lds_at<bf16x4>((ln.perm ^ (NB * w + b) << 5) + (aX + 16 * j * Tl::RB)) = h[0];
          }
      } else {
        const __amdgpu_buffer_rsrc_t yg = __builtin_amdgcn_make_buffer_rsrc(
            reinterpret_cast<float*>(R.y) + y0, 0, (int)(((nv - 1) * yst + D) * 4), 0x00020000);
#pragma unroll
        for (int j = 0; j < NR; ++j)
#pragma unroll
          for (int b = 0; b < NB; ++b)
            __builtin_amdgcn_raw_buffer_store_b128(
                __builtin_bit_cast(u32x4, O[b][j]), yg,
                (int)(4 * ((16 * j + li) * (unsigned)yst + w0 + 16 * b + 4 * g)), 0, 0);
      }
    }
    lds_barrier();
    if (rows)
      Tl::rows_out(typename Tl::Rows(yst), Tl::block(reinterpret_cast<const T*>(R.y) + y0, yst, nv), aX);
  }

  // the exit state: of a sequence's end, or the sum at a boundary
  float* out = nullptr;
  if (!OUT)
    out = R.bound + ((size_t)(REV ? it.prev : it.next) * a.Hv + hv) * D * D;
  else if ((REV ? it.prev : it.next) < 0 && R.exit)
    out = R.exit + ((size_t)it.seq * a.Hv + hv) * D * D;
  if (out) {
    const float f = (float)frame;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int c = 0; c < NU; ++c)
        *reinterpret_cast<f32x4*>(out + (size_t)(w0 + 16 * b + li) * D + 16 * c + 4 * g) = St[b][c] * f;
  }
}

// Roles that go forward have NSF planes for the state, reversed ones NSR (0:
// there are none).
template <typename T, int D, bool OUT, int NSF, int NSR>
__global__ __launch_bounds__(64 * DECAY_NW, 2) void decay_scan_kernel(DecayScanArgs a) {
  int role, hk, hv, unit;
  decay_unit(a, role, hk, hv, unit);
  const DecayRole& R = a.role[role];
  if constexpr (NSR > 0) {
    if (R.rev)
      decay_scan_item<T, D, true, OUT, NSR>(a, R, hk, hv, unit);
    else
      decay_scan_item<T, D, false, OUT, NSF>(a, R, hk, hv, unit);
  } else {
    decay_scan_item<T, D, false, OUT, NSF>(a, R, hk, hv, unit);
  }
}

template <typename T, int D, bool OUT> constexpr size_t decay_lds() {
  typedef DecayKind<T> K;
  return (size_t)2 * (K::NP * (OUT ? 3 : 2) * K::C * D + (OUT ? K::NY * K::C * K::C : 0)) +
         (2 * K::C + 4) * sizeof(float);
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
  } else if (a.plan.seq_start) {
    const DecaySeqs s(a.plan);
    unsigned long long in = __ballot(s.cnt > 0);
    if (m >= __builtin_popcountll(in)) return;
    for (int i = 0; i < m; ++i) in &= in - 1;
    seq = __builtin_ctzll(in);
    slot0 = __builtin_amdgcn_readlane(s.slot0, seq), cnt = __builtin_amdgcn_readlane(s.cnt, seq);
    last = __builtin_amdgcn_readlane(s.t1 - s.t0, seq) - cnt * a.plan.L;
  } else {
    seq = m, cnt = a.plan.P - 1, slot0 = m * cnt, last = a.plan.T - cnt * a.plan.L;
  }
  const int at = part * 1024 + threadIdx.x * 4;
  const float alpha = a.decay[hv];
  const DecayFactor aL(alpha, a.plan.L);
  DecayFactor f = R.rev ? DecayFactor(alpha, last) : aL;
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
  constexpr int U = 16;  // boundaries in flight
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
      X = f.join(X, n[u]);
      f = aL;
      if (j < cnt) *reinterpret_cast<f32x4*>(p + (size_t)(R.rev ? cnt - 1 - j : j) * pitch) = X;
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
  } else if (a.plan.seq_start) {
    const DecaySeqs s(a.plan);
    i = (long long)__builtin_amdgcn_readlane(s.t0, 0) * a.Hk * D4;
    n4 = (long long)__builtin_amdgcn_readlane(s.t1, a.plan.n_seq - 1) * a.Hk * D4;
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
static hipError_t decay_plan(const DecayPlan& p, hipStream_t st, Profiler* prof) {
  if (!p.table) return hipSuccess;
  prof_begin(prof, "decay_plan", st);
  hipLaunchKernelGGL(decay_plan_kernel, dim3(1), dim3(1024), 0, st, p);
  prof_end(prof, st);
  return hipGetLastError();
}

template <typename T, int D, bool OUT, int NSF, int NSR>
static hipError_t decay_scan(DecayScanArgs a, const char* name, hipStream_t st, Profiler* prof) {
  constexpr size_t lds = decay_lds<T, D, OUT>();
  const void* fn = (const void*)decay_scan_kernel<T, D, OUT, NSF, NSR>;
  hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  const long long units = (long long)a.plan.max_items * (a.Hv / a.group);
  prof_begin(prof, name, st);
  hipLaunchKernelGGL((decay_scan_kernel<T, D, OUT, NSF, NSR>),
                     dim3((unsigned)((units + kXcds - 1) / kXcds * kXcds * a.group * a.roles)),
                     dim3(64 * DECAY_NW), lds, st, a);
  prof_end(prof, st);
  return hipGetLastError();
}

// Planes of the state (bf16): three in sums for a state that is an output, and
// in scans where every item ends in one (no sequence is cut); where few do, they
// take the third by themselves and the others save it (backward of 32,768
// tokens, 16 heads, D = 128: 512 us, 547 with three).  A scan of dq ends in none.
template <typename T, int D>
static hipError_t decay_sums(const DecayScanArgs& a, bool bwd, bool exit, hipStream_t st, Profiler* prof) {
  if constexpr (sizeof(T) == 4)
    return bwd ? decay_scan<T, D, false, 3, 3>(a, "decay_sum_bwd", st, prof)
               : decay_scan<T, D, false, 3, 0>(a, "decay_sum", st, prof);
  else if (bwd)
    return exit ? decay_scan<T, D, false, 2, 3>(a, "decay_sum_bwd", st, prof)
                : decay_scan<T, D, false, 2, 2>(a, "decay_sum_bwd", st, prof);
  else
    return exit ? decay_scan<T, D, false, 3, 0>(a, "decay_sum", st, prof)
                : decay_scan<T, D, false, 2, 0>(a, "decay_sum", st, prof);
}
template <typename T, int D>
static hipError_t decay_scans(const DecayScanArgs& a, bool bwd, bool exit, hipStream_t st, Profiler* prof) {
  const bool third = exit && a.plan.max_multi == 0;
  if constexpr (sizeof(T) == 4)
    return bwd ? decay_scan<T, D, true, 3, 3>(a, "decay_scan_bwd", st, prof)
               : decay_scan<T, D, true, 3, 0>(a, "decay_scan", st, prof);
  else if (bwd)
    return third ? decay_scan<T, D, true, 2, 3>(a, "decay_scan_bwd", st, prof)
                 : decay_scan<T, D, true, 2, 2>(a, "decay_scan_bwd", st, prof);
  else
    return third ? decay_scan<T, D, true, 3, 0>(a, "decay_scan", st, prof)
                 : decay_scan<T, D, true, 2, 0>(a, "decay_scan", st, prof);
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
  if ((e = decay_plan(d.plan, st, prof)) != hipSuccess) return e;
  DecayScanArgs a{};
  a.plan = d.plan;
  a.decay = d.decay;
  a.Hv = d.Hv;
  a.group = d.group;
  a.roles = 1;
  a.role[0] = DecayRole{{d.q, d.qs, 1}, {d.k, d.ks, 1}, {d.v, d.vs, 0}, d.o, sizeof(T) == 4,
                        d.bound[0],     d.S_in,         d.S_out,        d.scale, 1.f, 0, 0, 0};
  if (d.plan.max_multi > 0) {
    if ((e = decay_sums<T, D>(a, false, d.S_out, st, prof)) != hipSuccess) return e;
    DecayChainArgs c{};
    c.plan = d.plan;
    c.decay = d.decay;
    c.Hv = d.Hv;
    c.role[0] = DecayChainRole{d.bound[0], d.S_in, 0, 0};
    if (!d.plan.direct && (e = decay_chain<D>(c, 1, st, prof)) != hipSuccess) return e;
  }
  return decay_scans<T, D>(a, false, d.S_out, st, prof);
}

template <typename T, int D>
hipError_t launch_decay_bwd(const DecayArgs& d, hipStream_t st, Profiler* prof) {
  hipError_t e;
  if ((e = decay_plan(d.plan, st, prof)) != hipSuccess) return e;
  const DecayTensor q{d.q, d.qs, 1}, k{d.k, d.ks, 1}, v{d.v, d.vs, 0},
      dO{d.dO, (long long)d.Hv * D, 0};
  const bool part = d.group > 1;
  const int f32 = part || sizeof(T) == 4;
  DecayScanArgs a{};
  a.plan = d.plan;
  a.decay = d.decay;
  a.Hv = d.Hv;
  a.group = d.group;
  // dv and dk: the reversed scan of G and of G^T, from the same boundaries
  a.role[0] = DecayRole{k, q, dO, d.dv, sizeof(T) == 4, d.bound[1], d.dS_out, d.dS_in, 1.f, d.scale,
                        0, 0, 1};
  a.role[2] = DecayRole{v, dO, q, part ? (void*)d.part[1] : d.dk, f32, d.bound[1], d.dS_out, nullptr,
                        1.f, d.scale, 1, 1, 1};
  // dq: the forward scan of S^T
  a.role[1] = DecayRole{dO, v, k, part ? (void*)d.part[0] : d.dq, f32, d.bound[0], d.S_in, nullptr,
                        d.scale, 1.f, 1, 0, 0};
  if (d.plan.max_multi > 0) {
    a.roles = 2;
    if ((e = decay_sums<T, D>(a, true, d.dS_in, st, prof)) != hipSuccess) return e;
    DecayChainArgs c{};
    c.plan = d.plan;
    c.decay = d.decay;
    c.Hv = d.Hv;
    c.role[0] = DecayChainRole{d.bound[0], d.S_in, 1, 0};
    c.role[1] = DecayChainRole{d.bound[1], d.dS_out, 0, 1};
    if (!d.plan.direct && (e = decay_chain<D>(c, 2, st, prof)) != hipSuccess) return e;
  }
  a.roles = 3;
  if ((e = decay_scans<T, D>(a, true, d.dS_in, st, prof)) != hipSuccess) return e;
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
