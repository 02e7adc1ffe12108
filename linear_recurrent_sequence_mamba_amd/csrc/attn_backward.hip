// attn_backward.hip -- the gradients of causal attention over packed sequences
// (gfx950).
//
//   p = exp(s - lse),  dp_ij = <do_i, v_j>,  D_i = <o_i, do_i>,
//   ds_ij = p_ij (dp_ij - D_i),
//   dv_j = sum_i p_ij do_i,  dk_j = scale sum_i ds_ij q_i,
//   dq_i = scale sum_j ds_ij k_j
//
// k_attn_dq takes queries as lanes and walks over keys; it also turns (o, do,
// lse) into one pair per row and head for k_attn_dkv, which takes keys as lanes
// and walks over queries.  Both recompute s from q and k, so no sum is shared
// between workgroups: there are no atomics, and equal calls give equal bits.
// The heads of a group add up in one workgroup, or, where that would leave
// too few, in parts that k_attn_sum adds in order.
#include "attn_common.h"

namespace m3 {
namespace {
typedef int i4 __attribute__((ext_vector_type(4)));
struct Yes { static constexpr bool value = true; };
struct No { static constexpr bool value = false; };

// ---------------------------------------------------------------------------
// One step of the sums over tiles of 32 rows:
//   kDq   lanes are queries, rows keys: sum += ds k
//   kDkv  lanes are keys, rows queries: sum (dk) += ds^T q, sum2 (dv) += p^T do
// A tile holds the rows that s is formed of (k; q) and, from row 32 on, the
// others (v; do); x and y are the lanes' own (q do; k v).  From s of the tile
// `cur` the step forms the weights, dp and ds, the products into the sums, and
// s of the tile `nxt`.  It is laid out product by product, each with its share
// of the softmax and the operand of a product some steps on: dp's products
// beside the exponentials, those of the next s beside the rest of ds.  Scores
// that do not count are -inf (hide_*).
enum { kDq = 0, kDkv = 1 };

template <typename T, int D, int KIND>
struct Grad {
  using L = Tile<T, D>;
  static constexpr int N1 = D / 16;                  // products of each kind
  static constexpr int A = N1, B = A + N1;           // first product of s2, of the first sum
  static constexpr int C = KIND == kDkv ? B + N1 : B;        // ... of dk's
  static constexpr int N = C + N1;
  // operands are read so many products before they are used (dk and dv of 128
  // channels have a SIMD to themselves; two everywhere: 2% slower)
  static constexpr int AHEAD = D == 128 && KIND == kDkv ? 4 : 3, R = AHEAD + 1;
  // steps over which the weights are spread: beside dp's products, or until
  // dv's sum needs them; and those of ds, which follows dp
  static constexpr int SW = KIND == kDkv ? B + N1 / 2 : A, SD = C + N1 / 2 - A - 1;

  static __device__ __forceinline__ Frag<T> operand(const char* cur, const char* nxt, int n, int lane) {
    if (n < A) return L::frag(cur, 32, n, lane);
    if (n < B) return L::frag(nxt, 0, n - A, lane);
    const int m = (n - B) % N1;
    return L::frag_t(cur, (n >= C ? 0 : 32) + 16 * (m / (N1 / 2)), 32 * (m % (N1 / 2)), lane);
  }
  // lse (which = 0) or -D (1) of the rows 8 b + 4 half + 0 .. 3; of queries as
  // lanes they are the lane's own
  static __device__ __forceinline__ f4 stats(const float* stat, float lse, int which, int b, int lane) {
    if (KIND == kDq) return f4{lse, lse, lse, lse};
    const int at = 32 * which + 8 * b + 4 * (lane >> 5);
    return *reinterpret_cast<const f4*>(stat + at);
  }
  static __device__ __forceinline__ void step(f16v* sum, f16v* sum2, f16v& s, f16v& s2, const Frag<T>* x,
                                              const Frag<T>* y, const char* cur, const char* nxt,
                                              const float* stat, float lse, float nd, float c,
                                              int lane) {
    f16v dp;   // - D from the start: the products are added to it
    if (KIND == kDq) {
      float z = nd;   // (a vector of it would be kept in 16 registers)
      asm volatile("" : "+v"(z));
#pragma unroll
      for (int e = 0; e < 16; ++e) dp[e] = z;
    } else {
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const f4 d = stats(stat, 0.0f, 1, b, lane);
#pragma unroll
        for (int j = 0; j < 4; ++j) dp[4 * b + j] = d[j];
      }
    }
    s2 = f16v{};
    Frag<T> op[R], f[2], fw[2];
    f4 l4[2];
    l4[0] = stats(stat, lse, 0, 0, lane);
#pragma unroll
    for (int n = 0; n < AHEAD; ++n) op[n] = operand(cur, nxt, n, lane);
    float w8[8], v8[8];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      if (n + AHEAD < N) op[(n + AHEAD) % R] = operand(cur, nxt, n + AHEAD, lane);
      if (n < A) {
        dp = mma(op[n % R], y[n], dp);
      } else if (n < B) {
        s2 = mma(op[n % R], x[n - A], s2);
      } else {
        const int m = (n - B) % N1, w = m / (N1 / 2), d = m % (N1 / 2);
        if (n < C) sum2[d] = mma(op[n % R], fw[w], sum2[d]);
        else sum[d] = mma(op[n % R], f[w], sum[d]);
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        if (e * SW / 16 == n) {
          if (e % 4 == 0 && e < 12) l4[(e / 4 + 1) & 1] = stats(stat, lse, 0, e / 4 + 1, lane);
          const float w = __builtin_amdgcn_exp2f(fmaf(s[e], c, -l4[(e / 4) & 1][e % 4]));
          s[e] = w;
          if (KIND == kDkv) {
            v8[e % 8] = w;
            if (e % 8 == 7) frag_from(fw[e / 8], v8);
          }
        }
        if (A + 1 + e * SD / 16 == n) {
          w8[e % 8] = s[e] * dp[e];
          if (e % 8 == 7) frag_from(f[e / 8], w8);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
};

// Only the rows before `edge`, or from it on, count.  (Called for the few tiles
// on the diagonal: in every step it would be a fifth of the vector instructions.)
__device__ __forceinline__ void hide_after(f16v& s, int edge, int lane) {
  edge -= 4 * (opaque(lane) >> 5);
#pragma unroll
  for (int e = 0; e < 16; ++e) s[e] = row_of(e, 0) < edge ? s[e] : -INFINITY;
}
__device__ __forceinline__ void hide_before(f16v& s, int edge, int lane) {
  edge -= 4 * (opaque(lane) >> 5);
#pragma unroll
  for (int e = 0; e < 16; ++e) s[e] = row_of(e, 0) >= edge ? s[e] : -INFINITY;
}

// D_i = <o_i, do_i> takes o as it was rounded, from weights that were.  Over n
// keys of like weight that moves dq and dk by sqrt(2 / n) of their own
// rounding, which only counts where n is small: blocks that see at most this
// many keys sum p dp instead, before anything else, and leave it to dk.  (All
// blocks would cost a sixth of the gradients' time; a long row whose weight is
// on a few keys keeps the larger error, up to 1.9 roundings.)
constexpr int kExactD = 512;

// ---------------------------------------------------------------------------
// dq: 32 queries a wave, tiles of 32 keys in LDS (8192 packed rows, 16 heads of
// 128 on 2: 166 us, 0.95 PFLOP/s, matrix cores busy 48%, vector units 35%)
template <typename T, int D, int WAVES>
__global__ __launch_bounds__(64 * WAVES, sizeof(T) * D == 512 ? 1 : 2) void k_attn_dq(AttnArgs a) {
  using L = Tile<T, D>;
  static_assert(WAVES == 4, "128 columns");
  constexpr int BN = 32;
  // Tiles t, t + 1 (its s), t + 2 and t + 3 (arriving).  Variables of their own,
  // used by name: of one array the compiler takes every read to follow the loads
  // that are on their way, and waits for them.
  __shared__ __align__(16) char sT0[L::BYTES], sT1[L::BYTES], sT2[L::BYTES], sT3[L::BYTES];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Columns col(a);
  const int64_t all = static_cast<int64_t>(a.Tq) * a.Hq;
  if (blockIdx.x == 0 && threadIdx.x == 0) {   // behind all rows' numbers
    a.stat[2 * all] = INFINITY;
    a.stat[2 * all + 1] = 0.0f;
  }
  const Slot sl = col.slot(a, lane);
  if (sl.s < 0) return;
  const int q0 = clamp_row(a.cuq[sl.s], a.Tq), q1 = clamp_row(a.cuq[sl.s + 1], a.Tq);
  const int k0 = clamp_row(a.cuk[sl.s], a.Tk), k1 = clamp_row(a.cuk[sl.s + 1], a.Tk);
  const int Lq = q1 - q0, Lk = max(0, k1 - k0);
  const int i0 = sl.tile * col.queries;
  if (i0 >= Lq) return;
  const int off = Lk - Lq, hk = col.hk, h = col.head(lane), half = lane >> 5;
  const int iw = i0 + col.first(wave), i = iw + col.query(lane);
  const int64_t row = q0 + min(i, Lq - 1);
  Frag<T> q[D / 16], g[D / 16];
  {
    const T* p = static_cast<const T*>(a.q) + row * a.ldq + h * D + 8 * half;
    const T* d = static_cast<const T*>(a.dout) + row * a.lddo + h * D + 8 * half;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      frag_load(q[kk], p + 16 * kk);
      frag_load(g[kk], d + 16 * kk);
    }
  }
  float lse = a.clse[row * a.Hq + h] * kLog2eA, dd = 0.0f;
  {
    // D = <o, do>; the other half of the row is in lane ^ 32
    const T* p = static_cast<const T*>(a.co) + row * a.ldo + h * D + 8 * half;
    Frag<T> o[D / 16];
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) frag_load(o[kk], p + 16 * kk);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) dd = frag_dot(o[kk], g[kk], dd);
    dd = half_sum(dd);
  }
  if (lse == -INFINITY) lse = INFINITY;   // no key: every weight 0
  float* st = a.stat + static_cast<int64_t>(h) * a.Tq + row;
  if (half == 0 && i < Lq) {
    st[0] = lse;
    st[all] = -dd;
  }
  f16v dq[D / 32];
#pragma unroll
  for (int d = 0; d < D / 32; ++d) dq[d] = f16v{};
  const float c = a.scale * kLog2eA;
  const int sees = min(i, Lq - 1) + off + 1;
  const int most = min(min(i0 + col.queries, Lq) + off, Lk);
  const int ntile = most <= 0 ? 0 : (most + BN - 1) / BN;
  const T* kp = static_cast<const T*>(a.k) + static_cast<int64_t>(k0) * a.ldk + hk * D;
  const T* vp = static_cast<const T*>(a.v) + static_cast<int64_t>(k0) * a.ldv + hk * D;
  f16v s, s2;
  if (most > 0 && most <= kExactD) {
    // D = sum_j p_ij dp_ij instead of <o, do>, for dk as well
    float r = 0.0f;
#pragma unroll 1
    for (int t = 0; t < ntile; ++t) {
      L::template load2<WAVES>(sT0, kp, a.ldk, vp, a.ldv, t * BN, Lk - 1, wave, lane);
      lds_loads_done();
      __syncthreads();
      s = f16v{};
      s2 = f16v{};
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        s = mma(L::frag(sT0, 0, kk, lane), q[kk], s);
        s2 = mma(L::frag(sT0, 32, kk, lane), g[kk], s2);
      }
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (t * BN + row_of(e, half) < sees)
          r = fmaf(__builtin_amdgcn_exp2f(fmaf(s[e], c, -lse)), s2[e], r);
      __syncthreads();
    }
    dd = half_sum(r);
    if (half == 0 && i < Lq) st[all] = -dd;
  }
  const auto pr = L::pair(kp, a.ldk, vp, a.ldv, wave, lane);
  auto fetch = [&](char* to, int t) __attribute__((always_inline)) {
    L::template load2<WAVES>(to, pr, kp, a.ldk, vp, a.ldv, 0, t * BN, Lk - 1, wave, lane);
  };
  const int all_see = min(iw, Lq - 1) + off + 1;   // keys that every query of the wave sees
  if (ntile > 0) {
    fetch(sT0, 0);
    lds_loads_done();
    __syncthreads();
    if (ntile > 1) fetch(sT1, 1);
    if (ntile > 2) fetch(sT2, 2);
    s = f16v{};
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) s = mma(L::frag(sT0, 0, kk, lane), q[kk], s);
  }
  // (in the loop's body all loads are made, so that the compiler, too, knows
  // which are still on their way)
  auto step = [&](auto in, int t, char* cur, char* nxt, char* aft, f16v& s, f16v& s2)
                  __attribute__((always_inline)) {
    if (in.value || t + 2 < ntile) lds_loads_but<L::NG / WAVES>(); else lds_loads_done();
    tiles_barrier();   // tile t + 1 is there; every wave is done with t - 1
    if (in.value || t + 3 < ntile) fetch(aft, t + 3);
    if ((t + 1) * BN > all_see) hide_after(s, sees - t * BN, lane);
    Grad<T, D, kDq>::step(dq, nullptr, s, s2, q, g, cur, nxt, nullptr, lse, -dd, c, lane);
  };
  int t = 0;
  for (; t + 6 < ntile; t += 4) {   // the scores change places, the buffers go round
    step(Yes{}, t, sT0, sT1, sT3, s, s2);
    step(Yes{}, t + 1, sT1, sT2, sT0, s2, s);
    step(Yes{}, t + 2, sT2, sT3, sT1, s, s2);
    step(Yes{}, t + 3, sT3, sT0, sT2, s2, s);
  }
  for (; t < ntile; t += 4) {
    step(No{}, t, sT0, sT1, sT3, s, s2);
    if (t + 1 < ntile) step(No{}, t + 1, sT1, sT2, sT0, s2, s);
    if (t + 2 < ntile) step(No{}, t + 2, sT2, sT3, sT1, s, s2);
    if (t + 3 < ntile) step(No{}, t + 3, sT3, sT0, sT2, s2, s);
  }
  if (i >= Lq) return;
  T* o = static_cast<T*>(a.dq) + (row * a.Hq + h) * D + 4 * half;
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      put4(o + 32 * d + 8 * e, dq[d][4 * e] * a.scale, dq[d][4 * e + 1] * a.scale,
           dq[d][4 * e + 2] * a.scale, dq[d][4 * e + 3] * a.scale);
}

// ---------------------------------------------------------------------------
// dk and dv: 32 keys a wave, tiles of 32 queries of the group's heads in LDS.
// At head dimension 128 keys, values, both sums and a tile's scores are more
// than 256 registers, which leaves one wave a SIMD; two kernels of two waves
// each need a quarter more products (one row of 8192, 16 heads of 128 on 2, all
// gradients: 1.06 ms, one kernel 0.95; fp32, two rows of 2048: 1.29 and 1.10).
// 8192 packed rows: 268 us, 0.78 PFLOP/s, matrix cores busy 37%, vector units 30%.
template <typename T, int D, int WAVES>
__global__ __launch_bounds__(64 * WAVES, D == 128 ? 1 : 2) void k_attn_dkv(AttnArgs a) {
  using L = Tile<T, D>;
  constexpr int BK = 32 * WAVES, BQ = 32;
  static_assert(BK == 128, "1 << 7 keys");
  // tiles t, t + 1 (its s), t + 2 and t + 3 (arriving), as in k_attn_dq
  __shared__ __align__(16) char sT0[L::BYTES], sT1[L::BYTES], sT2[L::BYTES], sT3[L::BYTES];
  __shared__ __align__(16) float sS0[2 * BQ], sS1[2 * BQ], sS2[2 * BQ], sS3[2 * BQ];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int per = a.Hk * a.gsplit;
  const int part = blockIdx.x % a.gsplit, hk = blockIdx.x % per / a.gsplit;
  // early keys are seen by most queries: they start first
  const Slot sl = key_slot(a, 7, static_cast<int>(blockIdx.x / per), lane);
  if (sl.s < 0) return;
  const int q0 = clamp_row(a.cuq[sl.s], a.Tq), q1 = clamp_row(a.cuq[sl.s + 1], a.Tq);
  const int k0 = clamp_row(a.cuk[sl.s], a.Tk), k1 = clamp_row(a.cuk[sl.s + 1], a.Tk);
  const int Lq = max(0, q1 - q0), Lk = k1 - k0;
  const int j0 = sl.tile * BK;
  if (j0 >= Lk) return;
  const int off = Lk - Lq, half = lane >> 5, grp = a.Hq / a.Hk, gper = grp / a.gsplit;
  const int jw = j0 + 32 * wave, j = jw + (lane & 31);
  const int64_t row = k0 + min(j, Lk - 1);
  Frag<T> k[D / 16], v[D / 16];
  {
    const T* p = static_cast<const T*>(a.k) + row * a.ldk + hk * D + 8 * half;
    const T* r = static_cast<const T*>(a.v) + row * a.ldv + hk * D + 8 * half;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      frag_load(k[kk], p + 16 * kk);
      frag_load(v[kk], r + 16 * kk);
    }
  }
  f16v sum[D / 32], sum2[D / 32];
#pragma unroll
  for (int d = 0; d < D / 32; ++d) sum[d] = sum2[d] = f16v{};
  const float c = a.scale * kLog2eA;
  // the first query that sees the block's first key, in whole tiles
  const int first = max(0, j0 - off) / BQ;
  const int nt = max(0, (Lq + BQ - 1) / BQ - first), all = nt * gper;
  // the tiles run over the queries of one head after the other
  int fh = hk * grp + part * gper, fi = first;   // of the next fetch
  const T* qp = static_cast<const T*>(a.q) + static_cast<int64_t>(q0) * a.ldq;
  const T* gp = static_cast<const T*>(a.dout) + static_cast<int64_t>(q0) * a.lddo;
  const auto pr = L::pair(qp, a.ldq, gp, a.lddo, wave, lane);
  constexpr int kLoads = L::NG / WAVES + 1;   // of a wave for one tile
  auto fetch = [&](char* to, float* st) __attribute__((always_inline)) {
    L::template load2<WAVES>(to, pr, qp, a.ldq, gp, a.lddo, fh * D, fi * BQ, Lq - 1, wave, lane);
    // lse of 32 rows, then -D of them; past the last row infinity and 0.  (Every
    // wave loads the same, so that all count the same number of loads.)
    const int i = fi * BQ + (lane & 31);
    const float* src = a.stat + (i < Lq ? (static_cast<int64_t>(half) * a.Hq + fh) * a.Tq + q0 + i
                                        : 2 * static_cast<int64_t>(a.Hq) * a.Tq + half);
    __builtin_amdgcn_global_load_lds((const M3_GLB void*)src, (M3_LDS void*)st, 4, 0, 0);
    if (++fi == first + nt) {
      fi = first;
      ++fh;
    }
  };
  f16v s, s2;
  if (all > 0) {
    fetch(sT0, sS0);
    lds_loads_done();
    __syncthreads();
    if (all > 1) fetch(sT1, sS1);
    if (all > 2) fetch(sT2, sS2);
    s = f16v{};
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) s = mma(L::frag(sT0, 0, kk, lane), k[kk], s);
  }
  int ci = first;   // the tile at hand
  auto step = [&](auto in, int n, char* cur, char* nxt, char* aft, float* st, float* sa, f16v& s,
                  f16v& s2) __attribute__((always_inline)) {
    if (in.value || n + 2 < all) lds_loads_but<kLoads>(); else lds_loads_done();
    tiles_barrier();   // tile n + 1 is there; every wave is done with n - 1
    if (in.value || n + 3 < all) fetch(aft, sa);
    const int i0 = ci * BQ;
    if constexpr (D == 128 && sizeof(T) == 2) {
      // k and v in the other half of the registers, from where products take
      // them as well, so that the sums and scores do not have to be moved there
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        i4 kx = __builtin_bit_cast(i4, k[kk]), vx = __builtin_bit_cast(i4, v[kk]);
        asm volatile("" : "+a"(kx), "+a"(vx));
        k[kk] = __builtin_bit_cast(Frag<T>, kx);
        v[kk] = __builtin_bit_cast(Frag<T>, vx);
      }
    }
    // rows i >= j - off count
    if (i0 < jw + 31 - off) hide_before(s, j - off - i0, lane);
    Grad<T, D, kDkv>::step(sum, sum2, s, s2, k, v, cur, nxt, st, 0.0f, 0.0f, c, lane);
    if (++ci == first + nt) ci = first;
  };
  int n = 0;
  for (; n + 6 < all; n += 4) {
    step(Yes{}, n, sT0, sT1, sT3, sS0, sS3, s, s2);
    step(Yes{}, n + 1, sT1, sT2, sT0, sS1, sS0, s2, s);
    step(Yes{}, n + 2, sT2, sT3, sT1, sS2, sS1, s, s2);
    step(Yes{}, n + 3, sT3, sT0, sT2, sS3, sS2, s2, s);
  }
  for (; n < all; n += 4) {
    step(No{}, n, sT0, sT1, sT3, sS0, sS3, s, s2);
    if (n + 1 < all) step(No{}, n + 1, sT1, sT2, sT0, sS1, sS0, s2, s);
    if (n + 2 < all) step(No{}, n + 2, sT2, sT3, sT1, sS2, sS1, s, s2);
    if (n + 3 < all) step(No{}, n + 3, sT3, sT0, sT2, sS3, sS2, s2, s);
  }
  if (j >= Lk) return;
  const int64_t at = (row * a.Hk + hk) * D + 4 * half;
  const int64_t to = static_cast<int64_t>(part) * a.Tk * a.Hk * D + at;
  // parts are scaled where they are added
  auto store = [&](const f16v* x, void* o, float* parts, float f) __attribute__((always_inline)) {
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x0 = x[d][4 * e], x1 = x[d][4 * e + 1], x2 = x[d][4 * e + 2], x3 = x[d][4 * e + 3];
        if (a.gsplit == 1)
          put4(static_cast<T*>(o) + at + 32 * d + 8 * e, x0 * f, x1 * f, x2 * f, x3 * f);
        else
          put4(parts + to + 32 * d + 8 * e, x0, x1, x2, x3);
      }
  };
  store(sum, a.dk, a.pk, a.scale);
  store(sum2, a.dv, a.pv, 1.0f);
}

// adds the parts of a group in order, for the rows that belong to a sequence
template <typename T>
__global__ __launch_bounds__(256) void k_attn_sum(AttnArgs a) {
  const int first = clamp_row(a.cuk[0], a.Tk), last = clamp_row(a.cuk[a.S], a.Tk);
  const int64_t w = static_cast<int64_t>(a.Hk) * a.D, size = a.Tk * w;
  const int64_t n = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (n < first * w || n >= last * w) return;
  f4 k = f4{0, 0, 0, 0}, v = f4{0, 0, 0, 0};
  for (int p = 0; p < a.gsplit; ++p) {
    k += *reinterpret_cast<const f4*>(a.pk + p * size + n);
    v += *reinterpret_cast<const f4*>(a.pv + p * size + n);
  }
  put4(static_cast<T*>(a.dk) + n, k.x * a.scale, k.y * a.scale, k.z * a.scale, k.w * a.scale);
  put4(static_cast<T*>(a.dv) + n, v.x, v.y, v.z, v.w);
}

// Parts of a group of heads: workgroups of 128 keys for twice the chip where the
// group has the heads for it, in equal parts.  Resident are one a CU (D = 128)
// or two; with half as many the uneven ends of a batch show, with twice as many
// the sums of the parts (all gradients of 4 sequences of 2048, 16 heads of 128
// on 2: from 256 workgroups on 381 us, 512 305, 1024 335; of 3 uneven ones of
// 8192 rows together, 16 heads of 64 on 2: 512 278, 1024 244).
int group_parts(int Tk, int S, int Hq, int Hk, int D) {
  const int g = Hq / Hk;
  const int64_t blocks = (static_cast<int64_t>(Tk) / 128 + S / 2 + 1) * Hk;   // a sequence ends inside a tile
  for (int n = 1; n < g; ++n)
    if (g % n == 0 && blocks * n >= (D == 128 ? 512 : 1024)) return n;
  return g;
}

template <typename T, int D>
hipError_t run(const AttnArgs& a, hipStream_t s) {
  constexpr int W = 4, B = 32 * W;
  const int64_t nk = (static_cast<int64_t>(a.Tk) / B + a.S) * a.Hk * a.gsplit;
  const int64_t nq = attn_query_workgroups(a.Tq, a.S, a.Hq, a.Hk);
  k_attn_dq<T, D, W><<<static_cast<unsigned>(nq), 64 * W, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // after dq, which leaves them lse and D
  k_attn_dkv<T, D, W><<<static_cast<unsigned>(nk), 64 * W, 0, s>>>(a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (a.gsplit > 1) {
    const int64_t n = static_cast<int64_t>(a.Tk) * a.Hk * D / 4;
    k_attn_sum<T><<<static_cast<unsigned>((n + 255) / 256), 256, 0, s>>>(a);
    e = hipGetLastError();
  }
  return e;
}

constexpr size_t up256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

size_t attn_backward_workspace_bytes(int Tq, int Tk, int S, int Hq, int Hk, int D) {
  const int g = group_parts(Tk, S, Hq, Hk, D);
  size_t n = up256(2 * sizeof(float) * (Tq * static_cast<size_t>(Hq) + 1));
  if (g > 1) n += 2 * up256(sizeof(float) * g * static_cast<size_t>(Tk) * Hk * D);
  return n;
}

hipError_t launch_attn_backward(AttnArgs& a, int bf16, void* ws, hipStream_t s) {
  a.lp = attn_log_pack(a.Hq, a.Hk);
  a.gsplit = group_parts(a.Tk, a.S, a.Hq, a.Hk, a.D);
  char* c = static_cast<char*>(ws);
  a.stat = reinterpret_cast<float*>(c);
  c += up256(2 * sizeof(float) * (a.Tq * static_cast<size_t>(a.Hq) + 1));
  a.pk = reinterpret_cast<float*>(c);
  c += up256(sizeof(float) * a.gsplit * static_cast<size_t>(a.Tk) * a.Hk * a.D);
  a.pv = reinterpret_cast<float*>(c);
  if (bf16) return a.D == 64 ? run<bf16_t, 64>(a, s) : run<bf16_t, 128>(a, s);
  return a.D == 64 ? run<float, 64>(a, s) : run<float, 128>(a, s);
}

}  // namespace m3
