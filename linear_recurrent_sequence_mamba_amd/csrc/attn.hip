// attn.hip -- causal attention over packed sequences, and one token against a
// cache (gfx950).
//
//   s = scale <q_i, k_j> for keys j <= i + (Lk - Lq),  p = softmax(s),
//   o_i = sum_j p_ij v_j,  lse_i = log sum_j exp(s_ij)
//
// Head h of q reads head h / (Hq / Hk) of k and v.  A row that sees no key
// has o = 0 and lse = -inf.
//
// The tiles are transposed (keys by queries), so that a query is a lane: the
// running maximum and sum of the softmax are one number per lane, a row of
// scores is reduced inside the lane and one exchange, and the weights are the
// B operand of the second product as they stand.
#include "attn_common.h"

namespace m3 {
namespace {

// ---------------------------------------------------------------------------
// The state of 32 queries: o transposed, maximum and sum (this lane's keys)
template <int D>
struct Rows {
  f16v o[D / 32];
  float m, l;
  __device__ __forceinline__ void init() {
#pragma unroll
    for (int d = 0; d < D / 32; ++d) o[d] = f16v{};
    m = -INFINITY;
    l = 0.0f;
  }
};

// Infinities and NaN of a tile of V in LDS become 0; returns whether this
// thread found any.  (The zero weights of keys that a query does not see would
// make NaN of them; they are added afterwards where they are seen.)
__device__ __forceinline__ bool special(bf16_t v) { return (v.bits & 0x7f80u) == 0x7f80u; }
__device__ __forceinline__ bool special(float v) {
  return (__float_as_uint(v) & 0x7f800000u) == 0x7f800000u;
}
template <typename T, int D, int THREADS>
__device__ __forceinline__ bool drop_special(char* V) {
  using L = Tile<T, D>;
  bool found = false;
  const int tid = opaque(threadIdx.x);
#pragma unroll 1
  for (int n = 0; n < 64 * L::NG / THREADS; ++n) {
    const int at = n * THREADS + tid;
    uint4* p = reinterpret_cast<uint4*>(V + L::place(at / 64) + 16 * (at % 64));
    uint4 u = *p;
    uint32_t w[4] = {u.x, u.y, u.z, u.w};
    bool bad = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (sizeof(T) == 2) {
        const bool lo = (w[j] & 0x7f80u) == 0x7f80u, hi = (w[j] & 0x7f800000u) == 0x7f800000u;
        w[j] &= (lo ? 0u : 0xffffu) | (hi ? 0u : 0xffff0000u);
        bad |= lo | hi;
      } else {
        const bool b = (w[j] & 0x7f800000u) == 0x7f800000u;
        if (b) w[j] = 0u;
        bad |= b;
      }
    }
    if (bad) *p = uint4{w[0], w[1], w[2], w[3]};
    found |= bad;
  }
  return found;
}

// Rows 32 + n .. 63 of a wave's own tile become 0.  What was loaded there behind
// the end of a cache repeats its last row, and the weights there are 0: a zero
// times a value that is infinite would be NaN.
template <typename T, int D>
__device__ __forceinline__ void clear_rows(char* KV, int n, int lane) {
  using L = Tile<T, D>;
  lane = opaque(lane);
  char* const at = KV + 16 * lane;
  n += 32 - L::lane_row(lane);
#pragma unroll
  for (int g = 0; g < L::NG; ++g)
    if (L::group_row(g) >= n) *reinterpret_cast<uint4*>(at + L::place(g)) = uint4{0u, 0u, 0u, 0u};
  lds_reads_done();   // (and writes)
}

// Scores of 32 queries against NB x 32 keys
template <typename T, int D, int NB>
__device__ __forceinline__ void score(f16v* s, const Frag<T>* q, const char* K, int lane) {
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    s[b] = f16v{};
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) s[b] = mma(Tile<T, D>::frag(K, 32 * b, kk, lane), q[kk], s[b]);
  }
}

// Only the first `seen` keys of a tile count (may be <= 0)
template <int NB>
__device__ __forceinline__ void hide(f16v* s, int seen, int lane) {
  seen -= 4 * (opaque(lane) >> 5);
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 16; ++i)
      s[b][i] = 32 * b + row_of(i, 0) < seen ? s[b][i] : -INFINITY;
}

template <int NB>
__device__ __forceinline__ float max_of(const f16v* s) {
  float mx = s[0][0];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[b][i]);
  return mx;
}

// The maximum that the weights are taken against, from the tile's (this
// lane's keys).  It moves only when it has to: weights up to 2^8 lose nothing
// in fp32 sums or bf16 products, and most tiles then leave o as it is.
template <int D>
__device__ __forceinline__ void raise_max(Rows<D>& st, float mx, float c) {
  mx = half_max(mx) * c;
  if (__ballot(mx > st.m + 8.0f)) {
    const float m = fmaxf(st.m, mx);
    const float f = m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(st.m - m);
    st.m = m;
    st.l *= f;
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) st.o[d][i] *= f;
  }
}

// Weights of a tile's scores, added to the sums
template <typename T, int D, int NB, int ROW0 = 0>
__device__ __forceinline__ void weigh(Rows<D>& st, f16v* s, const char* V, float c, int lane) {
  const float m0 = st.m == -INFINITY ? 0.0f : st.m;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      s[b][i] = __builtin_amdgcn_exp2f(fmaf(s[b][i], c, -m0));
      st.l += s[b][i];
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      Frag<T> p;
      float e8[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) e8[j] = s[b][8 * w + j];
      frag_from(p, e8);
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
        st.o[d] = mma(Tile<T, D>::frag_t(V, ROW0 + 32 * b + 16 * w, 32 * d, lane), p, st.o[d]);
    }
  }
}

// The same with the scores of the next tile formed meanwhile: they depend on
// nothing here, so the matrix cores work while the exponentials run.  The
// instructions are laid out step by step, each with one product (first those
// of the next scores, then those with V), its share of the exponentials, and
// the operand of the product two steps on, read from LDS.  Returns the maximum
// of the next scores, taken while the products with V run.
template <typename T, int D, int NB>
__device__ __forceinline__ float weigh_ahead(Rows<D>& st, f16v* s, f16v* next, const Frag<T>* q,
                                            const char* Knext, const char* V, float c, int lane) {
  using L = Tile<T, D>;
  constexpr int NM = NB * D / 16;          // products of each kind
  constexpr int F = 2 * NB, E = 16 * NB;   // fragments of weights, elements
  constexpr int S = NM + NM * (F - 1) / F; // steps until the last weight is needed
  const float m0 = st.m == -INFINITY ? 0.0f : st.m;
  auto operand = [&](int n) __attribute__((always_inline)) -> Frag<T> {
    if (n < NM) return L::frag(Knext, 32 * (n / (D / 16)), n % (D / 16), lane);
    const int m = n - NM;
    return L::frag_t(V, 16 * (m / (D / 32)), 32 * (m % (D / 32)), lane);
  };
#pragma unroll
  for (int b = 0; b < NB; ++b) next[b] = f16v{};
  float mx = -INFINITY;
  Frag<T> op[3], p[F];
  op[0] = operand(0);
  op[1] = operand(1);
#pragma unroll
  for (int n = 0; n < 2 * NM; ++n) {
    if (n + 2 < 2 * NM) op[(n + 2) % 3] = operand(n + 2);
    if (n < NM) {
      const int b = n / (D / 16);
      next[b] = mma(op[n % 3], q[n % (D / 16)], next[b]);
    } else {
      const int m = n - NM, d = m % (D / 32);
      st.o[d] = mma(op[n % 3], p[m / (D / 32)], st.o[d]);
    }
#pragma unroll
    for (int j = 0; j < (E + S - 1) / S; ++j) {
      const int e = (n * E + S - 1) / S + j;
      if (e >= E || e * S / E != n) continue;
      const float v = __builtin_amdgcn_exp2f(fmaf(s[e / 16][e % 16], c, -m0));
      s[e / 16][e % 16] = v;
      st.l += v;
      asm volatile("" : "+v"(st.l));   // added here, not after the loop
      if (e % 8 == 7) {
        float e8[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) e8[x] = s[e / 16][e % 16 - 7 + x];
        frag_from(p[e / 8], e8);
      }
    }
    // the last quarter of the next scores is still on its way at step NM
    constexpr int M0 = NM + 3, MS = 2 * NM - M0;
    // two at a time: one instruction takes the maximum of three
#pragma unroll
    for (int j = 0; j < (E / 2 + MS - 1) / MS; ++j) {
      const int e = 2 * (((n - M0) * (E / 2) + MS - 1) / MS + j);
      if (n >= M0 && e < E && M0 + e / 2 * MS / (E / 2) == n)
        mx = fmaxf(fmaxf(mx, next[e / 16][e % 16]), next[e / 16][e % 16 + 1]);
    }
    if (n >= M0) asm volatile("" : "+v"(mx));
    __builtin_amdgcn_sched_barrier(0);
  }
  return mx;
}

// 32 keys (rows 0 .. 31 of a tile) and their values (rows 32 .. 63)
template <typename T, int D, bool MASK>
__device__ __forceinline__ void attend(Rows<D>& st, const Frag<T>* q, const char* KV, float c,
                                       int seen, int lane) {
  f16v s[1];
  score<T, D, 1>(s, q, KV, lane);
  if (MASK) hide<1>(s, seen, lane);
  raise_max<D>(st, max_of<1>(s), c);
  weigh<T, D, 1, 32>(st, s, KV, c, lane);
}

// ---------------------------------------------------------------------------
// The prompt: a workgroup takes 128 (query, head) columns; K and V tiles of BN
// keys are double-buffered in LDS.  Two waves a SIMD (D = 64: three), so
// that one's softmax runs beside another's products as well.  16384 tokens, 16
// heads of 128: 1.02 ms, 1.08 PFLOP/s, matrix cores busy 56% and vector units
// 49% of the cycles; packed rows of 32 heads of 64: 242 us, 0.81 PFLOP/s, 40%
// and 70%.
template <typename T, int D, int WAVES, bool SPLIT>
__global__ __launch_bounds__(64 * WAVES, sizeof(T) * D == 512 ? 1 : 2) void k_attn(AttnArgs a) {
  using L = Tile<T, D>;
  static_assert(WAVES == 4, "128 columns");
  constexpr int BN = 64, NB = 2;
  // (variables of their own, used by name: of one array the compiler takes every
  // read to follow the loads that are on their way, and waits for them)
  __shared__ __align__(16) char sK0[L::BYTES], sK1[L::BYTES], sV0[L::BYTES], sV1[L::BYTES];
  __shared__ int sSpecial;
  if (threadIdx.x == 0) sSpecial = 0;   // read after the tiles' barriers
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Columns col(a);
  // late tiles of a sequence see most keys: they start first
  const Slot sl = col.slot(a, lane);
  if (sl.s < 0) return;
  const int q0 = clamp_row(a.cuq[sl.s], a.Tq), q1 = clamp_row(a.cuq[sl.s + 1], a.Tq);
  const int k0 = clamp_row(a.cuk[sl.s], a.Tk), k1 = clamp_row(a.cuk[sl.s + 1], a.Tk);
  const int Lq = q1 - q0, Lk = max(0, k1 - k0);
  const int i0 = sl.tile * col.queries;
  if (i0 >= Lq) return;
  const int off = Lk - Lq, hk = col.hk, h = col.head(lane);

  const int half = lane >> 5;
  const int iw = i0 + col.first(wave);         // the wave's first query
  const int i = iw + col.query(lane);          // the lane's
  const int64_t row = q0 + min(i, Lq - 1);
  Frag<T> q[D / 16];
  {
    const T* p = static_cast<const T*>(a.q) + row * a.ldq + h * D + 8 * half;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) frag_load(q[kk], p + 16 * kk);
  }
  Rows<D> st;
  st.init();
  const float c = a.scale * kLog2eA;
  int sees = min(i, Lq - 1) + off + 1;   // keys that the lane's query sees
  int most = min(min(i0 + col.queries, Lq) + off, Lk);   // that any query of the block sees
  int ntile = most <= 0 ? 0 : (most + BN - 1) / BN;
  // from here on some query of the block does not see the whole tile
  int tmask = max(0, min(i0, Lq - 1) + off + 1) / BN;
  const int wmost = min(min(iw + col.per_wave(), Lq) + off, Lk);
  int nw = (max(wmost, 0) + BN - 1) / BN;   // tiles that the wave sees
  int last = Lk - 1;
  const T* kp = static_cast<const T*>(a.k) + static_cast<int64_t>(k0) * a.ldk + hk * D;
  const T* vp = static_cast<const T*>(a.v) + static_cast<int64_t>(k0) * a.ldv + hk * D;
  if (SPLIT) {   // this workgroup's tiles, counted from its first key
    const int per = (ntile + a.nsplit - 1) / a.nsplit, t0 = min(static_cast<int>(blockIdx.y) * per, ntile);
    ntile = min(per, ntile - t0);
    kp += static_cast<int64_t>(t0 * BN) * a.ldk;
    vp += static_cast<int64_t>(t0 * BN) * a.ldv;
    sees -= t0 * BN;
    last -= t0 * BN;
    most = min(most - t0 * BN, ntile * BN);
    tmask = max(0, tmask - t0);
    nw = min(max(0, nw - t0), ntile);
  }
  // K runs one tile ahead of V.  Tiles that every query of the block sees
  // whole come first, in pairs (the two sets of scores change places): while
  // a tile's weights are formed the next tile's scores are.
  f16v s[NB], next[NB];
  const int npipe = max(0, min(tmask, ntile - 1)) & ~1;   // (no tile: none)
  auto arrive = [&](int t, char* K, char* V) __attribute__((always_inline)) {
    lds_loads_done();
    __syncthreads();   // V of t and K of t + 1 are there; every wave is done with t - 1
    if (t + 2 < ntile) L::template load<WAVES>(K, kp, a.ldk, (t + 2) * BN, last, wave, lane);
    if (t + 1 < ntile) L::template load<WAVES>(V, vp, a.ldv, (t + 1) * BN, last, wave, lane);
    // At D = 128 it is faster to let the loads end before the tiles at hand are
    // read (16384 tokens, 16 heads: 1042 us, not waiting 1061), at D = 64 not to
    // (packed rows of 32 heads: 264 and 255 us).
    if (D == 128) lds_loads_done();
  };
  if (ntile > 0) {
    L::template load<WAVES>(sK0, kp, a.ldk, 0, last, wave, lane);
    lds_loads_done();
    __syncthreads();
    L::template load<WAVES>(sV0, vp, a.ldv, 0, last, wave, lane);
    if (ntile > 1) L::template load<WAVES>(sK1, kp, a.ldk, BN, last, wave, lane);
    score<T, D, NB>(s, q, sK0, lane);
  }
  float mx = npipe > 0 ? max_of<NB>(s) : 0.0f;
  for (int t = 0; t < npipe; t += 2) {
    arrive(t, sK0, sV1);
    raise_max<D>(st, mx, c);
    mx = weigh_ahead<T, D, NB>(st, s, next, q, sK1, sV0, c, lane);
    arrive(t + 1, sK1, sV0);
    raise_max<D>(st, mx, c);
    mx = weigh_ahead<T, D, NB>(st, next, s, q, sK0, sV1, c, lane);
  }
#pragma unroll 1
  for (int t = npipe; t < ntile; ++t) {
    char* const V = t & 1 ? sV1 : sV0;
    arrive(t, t & 1 ? sK1 : sK0, t & 1 ? sV0 : sV1);
    if (t >= tmask) {
      if (drop_special<T, D, 64 * WAVES>(V)) sSpecial = 1;
      __syncthreads();
    }
    if (t >= nw) continue;
    hide<NB>(s, sees - t * BN, lane);
    raise_max<D>(st, max_of<NB>(s), c);
    weigh<T, D, NB>(st, s, V, c, lane);
    if (t + 1 < nw) score<T, D, NB>(s, q, t & 1 ? sK0 : sK1, lane);
  }
  if (ntile > 0 && sSpecial) {
    for (int key = tmask * BN; key < most; ++key) {
      const T* r = vp + key * a.ldv + 4 * half;
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const T v = r[32 * d + row_of(e, 0)];
          if (key < sees && special(v)) st.o[d][e] += to_f32(v);
        }
    }
  }
  const float l = half_sum(st.l);
  if (i >= Lq) return;
  if constexpr (SPLIT) {
    const int64_t at = (row * a.Hq + h) * a.nsplit + blockIdx.y;
    float* o = a.po + at * D + 4 * half;
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        put4(o + 32 * d + 8 * e, st.o[d][4 * e], st.o[d][4 * e + 1], st.o[d][4 * e + 2], st.o[d][4 * e + 3]);
    if (half == 0) *reinterpret_cast<f2*>(a.pm + 2 * at) = f2{st.m, l};
    return;
  }
  const float inv = l > 0.0f ? 1.0f / l : (l == l ? 0.0f : l);   // a NaN stays
  T* o = static_cast<T*>(a.o) + row * a.ldo + h * D + 4 * half;
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      put4(o + 32 * d + 8 * e, st.o[d][4 * e] * inv, st.o[d][4 * e + 1] * inv,
           st.o[d][4 * e + 2] * inv, st.o[d][4 * e + 3] * inv);
  if (half == 0 && a.lse)
    a.lse[row * a.Hq + h] = l == 0.0f ? -INFINITY : (st.m + __builtin_amdgcn_logf(l)) * kLn2A;
}

// ---------------------------------------------------------------------------
// One token: the queries of a group of heads (at most 32 at a time) are the
// tile's columns.  A workgroup takes a part of one sequence's cache, its
// waves every WAVES-th tile of 32 keys each, without barriers; the waves'
// sums are joined in LDS and the parts by k_attn_join.  Bound by reading the
// cache: 65536 keys of 16 heads of 64 in 49 us when called again and again (5.5
// TB/s: the last-level cache holds part of it), the join 4.6 us; 32 caches of 4096,
// 8 heads of 128, in a graph over 16 different ones 112 us (4.8 TB/s), in fp32
// 244 us (4.4), of 64 65 us (4.2) and 113 us (4.8).
template <typename T, int D, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_attn_decode(AttnArgs a) {
  using L = Tile<T, D>;
  // A wave's tile (32 rows of K, 32 of V); afterwards its o [32][D] in fp32.  One
  // buffer, as the other waves' loads fill the time (32 caches of 4096, 8 heads,
  // in fp32: 244 us at D = 128, 110 at 64; with two buffers half as many waves
  // fit, 402 and 145 us; in bf16 the same within 3%).  Resident are two workgroups
  // a CU at D = 64 and, with 348 registers and more, one at D = 128.
  constexpr int BN = 32;
  __shared__ __align__(16) char sKV[WAVES][L::BYTES];
  __shared__ float sM[WAVES][32], sL[WAVES][32];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = lane >> 5, g = a.Hq / a.Hk, ng = (g + 31) / 32;
  int n = blockIdx.x;
  const int part = n % a.nsplit;
  n /= a.nsplit;
  const int gb = n % ng;
  n /= ng;
  const int hk = n % a.Hk, s = n / a.Hk;
  const int len = max(0, min(a.len[s], a.cap));
  // the part's keys, in whole tiles
  const int tiles = (len + BN - 1) / BN;
  const int per = (tiles + a.nsplit - 1) / a.nsplit;
  const int t0 = part * per, t1 = min(t0 + per, tiles);
  const int hl = min(gb * 32 + (lane & 31), g - 1);   // the lane's head in the group
  const int h = hk * g + hl;
  Frag<T> q[D / 16];
  {
    const T* p = static_cast<const T*>(a.q) + s * a.ldq + h * D + 8 * half;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) frag_load(q[kk], p + 16 * kk);
  }
  Rows<D> st;
  st.init();
  const float c = a.scale * kLog2eA;
  const T* kp = static_cast<const T*>(a.k) + s * a.bk + hk * D;
  const T* vp = static_cast<const T*>(a.v) + s * a.bv + hk * D;
  auto fetch = [&](int t) __attribute__((always_inline)) {
    L::template load2<1>(sKV[wave], kp, a.ldk, vp, a.ldv, t * BN, len - 1, 0, lane);
  };
  int t = t0 + wave;
  if (t < t1) fetch(t);
  for (; t < t1; t += WAVES) {
    lds_loads_done();
    if ((t + 1) * BN <= len) {
      attend<T, D, false>(st, q, sKV[wave], c, BN, lane);
    } else {   // keys past the end are hidden, their values cleared
      clear_rows<T, D>(sKV[wave], len - t * BN, lane);
      attend<T, D, true>(st, q, sKV[wave], c, len - t * BN, lane);
    }
    if (t + WAVES < t1) {
      lds_reads_done();
      fetch(t + WAVES);
    }
  }
  const float l = half_sum(st.l);
  if (half == 0) {
    sM[wave][lane] = st.m;
    sL[wave][lane] = l;
  }
  // o of this wave, over its own tiles (of which it is done reading)
  static_assert(L::BYTES >= static_cast<int>(sizeof(float)) * 32 * D, "room for o");
  float* so = reinterpret_cast<float*>(sKV[wave]);
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) so[(lane & 31) * D + 32 * d + row_of(e, half)] = st.o[d][e];
  __syncthreads();
  const int rows = min(32, g - gb * 32);
  for (int x = threadIdx.x; x < rows * (D / 4); x += 64 * WAVES) {
    const int r = x / (D / 4), d = 4 * (x % (D / 4));
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) m = fmaxf(m, sM[w][r]);
    float ls = 0.0f;
    f4 v = f4{0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      const float f = sM[w][r] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(sM[w][r] - m);
      const float lw = sL[w][r];
      // a wave that saw no key has l = 0 and o = 0
      if (lw != 0.0f) {
        ls = fmaf(f, lw, ls);
        const f4 ow = *reinterpret_cast<const f4*>(reinterpret_cast<const float*>(sKV[w]) + r * D + d);
        v.x = fmaf(f, ow.x, v.x);
        v.y = fmaf(f, ow.y, v.y);
        v.z = fmaf(f, ow.z, v.z);
        v.w = fmaf(f, ow.w, v.w);
      }
    }
    const int hh = hk * g + gb * 32 + r;
    if (a.nsplit == 1) {
      const float inv = ls > 0.0f ? 1.0f / ls : (ls == ls ? 0.0f : ls);
      put4(static_cast<T*>(a.o) + static_cast<int64_t>(s) * a.ldo + hh * D + d, v.x * inv, v.y * inv,
           v.z * inv, v.w * inv);
      if (d == 0 && a.lse)
        a.lse[static_cast<int64_t>(s) * a.Hq + hh] =
            ls == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(ls)) * kLn2A;
    } else {
      const int64_t at = (static_cast<int64_t>(s) * a.Hq + hh) * a.nsplit + part;
      *reinterpret_cast<f4*>(a.po + at * D + d) = v;
      if (d == 0) *reinterpret_cast<f2*>(a.pm + 2 * at) = f2{m, ls};
    }
  }
}

// Joins the parts of one (sequence or query, head) per workgroup: 256 / (D / 4) groups
// of threads take every so manieth part each, four channels a thread.
template <typename T, int D>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a) {
  constexpr int NG = 1024 / D;
  __shared__ f4 sv[NG][D / 4];
  __shared__ float sl[NG];
  const int64_t n = blockIdx.x;
  if (a.cuq) {   // of queries: those that belong to a sequence
    const int64_t row = n / a.Hq;
    if (row < clamp_row(a.cuq[0], a.Tq) || row >= clamp_row(a.cuq[a.S], a.Tq)) return;
  }
  const int dl = threadIdx.x % (D / 4), g = threadIdx.x / (D / 4), lane = threadIdx.x & 63;
  const f2* pm = reinterpret_cast<const f2*>(a.pm) + n * a.nsplit;
  float m = -INFINITY;
  for (int p = lane; p < a.nsplit; p += 64) m = fmaxf(m, pm[p].x);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
  float l = 0.0f;
  f4 v = f4{0, 0, 0, 0};
#pragma unroll 2
  for (int p = g; p < a.nsplit; p += NG) {
    const f2 ml = pm[p];
    const f4 o = *reinterpret_cast<const f4*>(a.po + (n * a.nsplit + p) * D + 4 * dl);
    if (ml.y == 0.0f) continue;
    const float f = ml.x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(ml.x - m);
    l = fmaf(f, ml.y, l);
    v.x = fmaf(f, o.x, v.x);
    v.y = fmaf(f, o.y, v.y);
    v.z = fmaf(f, o.z, v.z);
    v.w = fmaf(f, o.w, v.w);
  }
  sv[g][dl] = v;
  if (dl == 0) sl[g] = l;
  __syncthreads();
  if (g != 0) return;
  l = 0.0f;
  v = f4{0, 0, 0, 0};
#pragma unroll
  for (int k = 0; k < NG; ++k) {
    l += sl[k];
    v += sv[k][dl];
  }
  const float inv = l > 0.0f ? 1.0f / l : (l == l ? 0.0f : l);
  const int64_t s = n / a.Hq;
  const int h = static_cast<int>(n % a.Hq);
  put4(static_cast<T*>(a.o) + s * a.ldo + h * D + 4 * dl, v.x * inv, v.y * inv, v.z * inv, v.w * inv);
  if (dl == 0 && a.lse) a.lse[n] = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2A;
}

template <typename T, int D>
hipError_t run_attn(const AttnArgs& a, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(attn_query_workgroups(a.Tq, a.S, a.Hq, a.Hk)),
                  static_cast<unsigned>(a.nsplit));
  if (a.nsplit == 1) {
    k_attn<T, D, 4, false><<<grid, 256, 0, s>>>(a);
    return hipGetLastError();
  }
  k_attn<T, D, 4, true><<<grid, 256, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_attn_join<T, D><<<static_cast<unsigned>(static_cast<int64_t>(a.Tq) * a.Hq), 256, 0, s>>>(a);
  return hipGetLastError();
}

// Parts of the keys where queries are so few that four would still not fill the
// chip (two workgroups a CU), each with 512 keys at the least of a sequence of
// mean length, in fp32, whose products take longer, 256.  16 queries of 16384
// keys, 16 heads of 128 on 2: 340 us whole, 26 split; 256 of 8192: 170 and 42; 2048
// of 2048, 4 heads of 128: 43 and 32; but 1024 of 1024, 16 heads on 2, in two: 27
// and 41, as the parts of so many rows have to be joined.  fp32, 2 of 1400, 64
// heads of 64 on 8: 98, 55 with 512 keys, 30 with 256.
int prompt_parts(int Tq, int Tk, int S, int Hq, int Hk, int bf16) {
  const int64_t blocks = attn_query_workgroups(Tq, S, Hq, Hk);
  const int n = static_cast<int>(512 / blocks), most = Tk / S / (bf16 ? 512 : 256);
  if (n < 4 || most < 2) return 1;
  return n < most ? n : most;
}

template <typename T, int D, int WAVES>
hipError_t run_decode(const AttnArgs& a, hipStream_t s) {
  const int g = a.Hq / a.Hk, ng = (g + 31) / 32;
  const int64_t grid = static_cast<int64_t>(a.S) * a.Hk * ng * a.nsplit;
  k_attn_decode<T, D, WAVES><<<static_cast<unsigned>(grid), 64 * WAVES, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.nsplit == 1) return e;
  k_attn_join<T, D><<<static_cast<unsigned>(a.S * a.Hq), 256, 0, s>>>(a);
  return hipGetLastError();
}

// Parts of a cache: two workgroups for every CU (at D = 128 they follow each other),
// each with 512 keys at the least, four tiles of 32 for each of four waves.
int decode_parts(int S, int cap, int Hq, int Hk) {
  const int64_t blocks = static_cast<int64_t>(S) * Hk * ((Hq / Hk + 31) / 32);
  int64_t n = (512 + blocks - 1) / blocks;
  const int64_t most = (cap + 511) / 512;
  if (n > most) n = most;
  return n < 1 ? 1 : static_cast<int>(n);
}

}  // namespace

bool attn_supported(int D) { return D == 64 || D == 128; }

size_t attn_workspace_bytes(int Tq, int Tk, int S, int Hq, int Hk, int D, int bf16) {
  const int n = prompt_parts(Tq, Tk, S, Hq, Hk, bf16);
  return n == 1 ? 0 : sizeof(float) * (static_cast<size_t>(D) + 2) * Tq * Hq * n;
}

hipError_t launch_attn(AttnArgs& a, int bf16, void* ws, hipStream_t s) {
  a.lp = attn_log_pack(a.Hq, a.Hk);
  a.nsplit = prompt_parts(a.Tq, a.Tk, a.S, a.Hq, a.Hk, bf16);
  a.po = static_cast<float*>(ws);
  a.pm = a.po + static_cast<size_t>(a.D) * a.Tq * a.Hq * a.nsplit;
  if (bf16) return a.D == 64 ? run_attn<bf16_t, 64>(a, s) : run_attn<bf16_t, 128>(a, s);
  return a.D == 64 ? run_attn<float, 64>(a, s) : run_attn<float, 128>(a, s);
}

size_t attn_decode_workspace_bytes(int S, int cap, int Hq, int Hk, int D) {
  const int n = decode_parts(S, cap, Hq, Hk);
  return n == 1 ? 0 : sizeof(float) * (static_cast<size_t>(D) + 2) * S * Hq * n;
}

hipError_t launch_attn_decode(AttnArgs& a, int bf16, void* ws, hipStream_t s) {
  a.nsplit = decode_parts(a.S, a.cap, a.Hq, a.Hk);
  a.po = static_cast<float*>(ws);
  a.pm = a.po + static_cast<size_t>(a.D) * a.S * a.Hq * a.nsplit;
  if (bf16) return a.D == 64 ? run_decode<bf16_t, 64, 4>(a, s) : run_decode<bf16_t, 128, 4>(a, s);
  return a.D == 64 ? run_decode<float, 64, 4>(a, s) : run_decode<float, 128, 4>(a, s);
}

}  // namespace m3
