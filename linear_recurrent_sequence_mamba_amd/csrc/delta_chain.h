// delta_chain.h -- the chain of the gated delta rule over a sequence's chunks, and
// what passes states through its segments (gfx950).  Not part of the public ABI.
#pragma once

#include "delta_common.h"

namespace m3 {
namespace {

// The chain.  A wave holds 16 columns of a head's state, so that nothing of it
// is ever exchanged; the NW waves of a workgroup share K, Q and the chunk's
// matrix in LDS.  The next chunk is on its way in registers meanwhile.
//
// Where sequences and heads are too few to fill the chip, a sequence's chunks
// are cut into segments.  A segment maps the state before it as S -> E + F S.
// kEnds gives E (a state that starts from zero), kMaps F (the columns of the
// identity as a state, without values), k_delta_join passes the states through
// the segments, and the segments then run at once.
//
// Parts (bf16): what reaches the state has three, so that it keeps fp32's
// accuracy, a map and the state that it is applied to among it: where a segment's
// keys overwrite the state, d S + F S cancels (with two parts a state behind slow
// decays is off by 2.7e-6 of itself, with three by 3e-7).  P and U, which only reach
// outputs in bf16, have two.
//
// With room for two of a chunk's tiles (NBUF = 2) the next chunk's are written
// while waves still read this one's, and one barrier a chunk is enough.
//
// What bounds it: each product needs the one before it.  A chunk takes 5.3 us
// (Dk = Dv = 128, bf16; 1.37 ms for 256 chunks) with a wave on each SIMD, 7.3 us
// with two: 730 vector and 182 matrix instructions on one path, with the states
// saved 800.  There (4 x 2048 tokens, 32 heads of 128 x 64, a wave on each SIMD)
// 46% of a wave's cycles issue, 39% wait for the matrix unit or a slot and 15% for
// LDS and barriers.  A second wave fills some of that, which is why segments pay
// although they do most of the work twice; but saved states (48 KB a chunk of
// 128 x 64) bring them to HBM's rate: in four segments each the chain alone
// takes 95 us for 480 MB, whole 184.
enum { kFull = 0, kEnds = 1, kMaps = 2, kMapsT = 3 };   // (kMapsT: the map's transpose, for the gradients)

template <typename T, int DK, int NT, bool FULL>
struct ChainTiles {
  using X = Rows64<DK>;
  using M = Rows64<64>;
  static constexpr int NI = DeltaParts<T>::IN, NO = DeltaParts<T>::OUT;
  static constexpr int BK = NI * X::PLANE, BQ = FULL ? BK : 0, BM = 3 * M::PLANE, BUF = BK + BQ + BM + 768;
  static constexpr int NG = (192 + NT - 1) / NT;
  Stage<T, DK, NT> k, q;
  Stage<float, 64, NT> m;
  float g[NG];
  __device__ __forceinline__ void store(char* b) const {
    k.store(b);
    if constexpr (FULL) q.store(b + BK);
    m.store(b + BK + BQ);
#pragma unroll
    for (int i = 0; i < NG; ++i)
      if (threadIdx.x + i * NT < 192) reinterpret_cast<float*>(b + BK + BQ + BM)[threadIdx.x + i * NT] = g[i];
  }
};

template <typename T, int DK, int NW, int NBUF, int MODE>
__device__ __forceinline__ void chain(const DeltaArgs& a, const DeltaSeg& seg, int h, int slice, char* smem) {
  using X = Rows64<DK>;
  constexpr bool FULL = MODE == kFull, MAPS = MODE == kMaps || MODE == kMapsT;
  constexpr int NT = 64 * NW, KS = DK / 32, DT = DK / 16;
  using Tiles = ChainTiles<T, DK, NT, FULL>;
  constexpr int NI = Tiles::NI, NO = Tiles::NO, NS = 3;
  constexpr int BK = Tiles::BK, BQ = Tiles::BQ, BM = Tiles::BM, BUF = Tiles::BUF;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4, hk = h / (a.Hv / a.Hk);
  const int cs = slice * NW + w, col = 16 * cs + r;   // of the values, or of the map
  const Triangle tri(lane);
  const typename X::Lane xl(lane);
  const Rows64<64>::Lane ml(lane);
  const int64_t head = static_cast<int64_t>(seg.s) * a.Hv + h, shead = static_cast<int64_t>(seg.n) * a.Hv + h;
  const int64_t dd = static_cast<int64_t>(DK) * a.Dv;
  const uint32_t at = static_cast<uint32_t>(8 * g * a.Dv + col);   // of a state
  const uint32_t end_at = (cs * DT * 64 + lane) * 4;               // of a segment's

  f4 S[DT];
#pragma unroll
  for (int t = 0; t < DT; ++t) S[t] = f4{0, 0, 0, 0};
  if constexpr (MAPS) {
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[t][e] = tile_row(t, e) + 8 * g == col ? 1.0f : 0.0f;
  } else if (FULL && (seg.j > 0 || (a.h0 && !seg.last))) {
    const float* p = seg.j > 0 ? a.ends + (shead - a.Hv) * dd : a.firsts + (static_cast<int64_t>(seg.place(a)) * a.Hv + h) * dd;
#pragma unroll
    for (int t = 0; t < DT; ++t) S[t] = *reinterpret_cast<const f4*>(p + end_at + t * 256);
  } else if (a.h0 && seg.j == 0) {
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[t][e] = (a.h0 + head * dd + tile_row(t, e) * a.Dv)[at];
    if constexpr (MODE == kEnds) {   // (hT may be h0, and is written while the first segment runs)
      float* p = a.firsts + (static_cast<int64_t>(seg.place(a)) * a.Hv + h) * dd;
#pragma unroll
      for (int t = 0; t < DT; ++t) *reinterpret_cast<f4*>(p + end_at + t * 256) = S[t];
    }
  }

  Tiles st;
  Cols<T> stV;
  const int c1 = seg.c0 + seg.nch;
  auto rows = [&](int c) __attribute__((always_inline)) { return min(kDeltaChunk, seg.len - c * kDeltaChunk); };
  auto first = [&](int c) __attribute__((always_inline)) { return seg.row0 + static_cast<int64_t>(c) * kDeltaChunk; };
  // (behind the last chunk the last one again, unused)
  auto fetch = [&](int c) __attribute__((always_inline)) {
    c = min(c, c1 - 1);
    const int64_t m = static_cast<int64_t>(seg.slot0 + c) * a.Hv + h;
    st.k.load(static_cast<const T*>(a.k) + first(c) * a.ldk + hk * DK, a.ldk, rows(c));
    st.m.load(a.pm + m * a.ldpm, 64, 64);
#pragma unroll
    for (int i = 0; i < Tiles::NG; ++i) st.g[i] = (a.pm + m * a.ldpm + kDeltaMatrix)[min(threadIdx.x + i * NT, 191u)];
    if constexpr (FULL) st.q.load(static_cast<const T*>(a.q) + first(c) * a.ldq + hk * DK, a.ldq, rows(c));
  };
  auto fetch_v = [&](int c) __attribute__((always_inline)) {
    c = min(c, c1 - 1);
    if constexpr (!MAPS) stV.load(static_cast<const T*>(a.v) + first(c) * a.ldv + h * a.Dv, a.ldv, rows(c), col, g);
  };
  if (seg.nch > 0) {
    fetch(seg.c0);
    fetch_v(seg.c0);
    st.store(smem);
    if constexpr (NBUF == 2) fetch(seg.c0 + 1);
  }
  char* buf = smem;
  float decay = 1.0f;   // of the segment
  for (int c = seg.c0; c < c1; ++c) {
    const char *sK = buf, *sQ = buf + BK, *sM = buf + BK + BQ;
    const float* sGate = reinterpret_cast<const float*>(buf + BK + BQ + BM);
    tiles_barrier();
    if (FULL && a.states) {
      float* p = a.states + (static_cast<int64_t>(seg.slot0 + c) * a.Hv + h) * a.ldpm;
#pragma unroll
      for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) (p + tile_row(t, e) * a.Dv)[at] = S[t][e];
    }
    // K S0 and Q S0, the next operands read ahead of their products
    f4 ks[4], qs[4];
    Parts<NI> ka[2][4], qa[2][4];
    Parts<NS> sp[2];
    auto read = [&](int x) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) ka[x & 1][i] = X::template by_row<NI>(sK, xl, i, x);
      if constexpr (FULL)
#pragma unroll
        for (int i = 0; i < 4; ++i) qa[x & 1][i] = X::template by_row<NI>(sQ, xl, i, x);
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) ks[i] = qs[i] = f4{0, 0, 0, 0};
    read(0);
    split_d<NS>(sp[0], S[0], S[1]);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int x = 0; x < KS; ++x) {
      if (x + 1 < KS) {
        read(x + 1);
        split_d<NS>(sp[(x + 1) & 1], S[2 * x + 2], S[2 * x + 3]);
      }
      mmp<NS>(ks, ka[x & 1], sp[x & 1]);
      if constexpr (FULL) mmp<NO>(qs, qa[x & 1], sp[x & 1]);
      if constexpr (NI == 1) interleave<FULL ? 8 : 4, FULL ? 20 : 4 * NS, FULL ? 3 : 4>();
      __builtin_amdgcn_sched_barrier(0);
    }
    // R = beta (V - exp(G) K S0) in place of K S0
    Parts<1> ta[2][6];
    tri.t6(ta[0], sM, ml, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f4 st = *reinterpret_cast<const f4*>(&sGate[tile_row(i, 0) + 8 * g]);
      const f4 bt = *reinterpret_cast<const f4*>(&sGate[128 + tile_row(i, 0) + 8 * g]);
#pragma unroll
      for (int e = 0; e < 4; ++e) ks[i][e] = bt[e] * fmaf(-st[e], ks[i][e], MAPS ? 0.0f : stV.v[4 * i + e].f());
    }
    Parts<NS> rp[2];
    split_d<NS>(rp[0], ks[0], ks[1]);
    split_d<NS>(rp[1], ks[2], ks[3]);
    __builtin_amdgcn_sched_barrier(0);
    // U = T R: R itself for the diagonal
    f4 u[6] = {ks[0], ks[1], ks[2], ks[3], f4{0, 0, 0, 0}, f4{0, 0, 0, 0}};
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      if (n + 1 < NS) tri.t6(ta[(n + 1) & 1], sM, ml, n + 1);
      mm6<NS>(u, ta[n & 1], rp, n);
      if (n == 0 && NBUF == 2) {
        buf = buf == smem ? smem + BUF : smem;
        st.store(buf);   // (the last time unread)
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    u[2] += u[4];
    u[3] += u[5];
    if constexpr (NBUF == 1) fetch(c + 1);   // (in few registers until then)
    // O = scale exp(G) Q S0 + P U
    if constexpr (FULL) {
      if (a.states) {
        float* p = a.states + (static_cast<int64_t>(seg.slot0 + c) * a.Hv + h) * a.ldpm + dd;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) (p + tile_row(i, e) * a.Dv)[at] = u[i][e];
      }
      Parts<1> pa[2][6];
      tri.p6(pa[0], sM, ml, 0);
      f4 y[6];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f4 st = *reinterpret_cast<const f4*>(&sGate[tile_row(i, 0) + 8 * g]);
#pragma unroll
        for (int e = 0; e < 4; ++e) y[i][e] = a.scale * st[e] * qs[i][e];
      }
      y[4] = y[5] = f4{0, 0, 0, 0};
      Parts<NO> up[2];
      split_d<NO>(up[0], u[0], u[1]);
      split_d<NO>(up[1], u[2], u[3]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int n = 0; n < NO; ++n) {
        if (n + 1 < NO) tri.p6(pa[(n + 1) & 1], sM, ml, n + 1);
        mm6<NO>(y, pa[n & 1], up, n);
        __builtin_amdgcn_sched_barrier(0);
      }
      y[2] += y[4];
      y[3] += y[5];
      const int ldo = a.Hv * a.Dv;
      const ChunkRows o(static_cast<T*>(a.o) + first(c) * ldo + h * a.Dv, ldo, rows(c));
      const uint32_t orow = static_cast<uint32_t>(ldo) * static_cast<uint32_t>(sizeof(T));
      const uint32_t oat = 8 * g * orow + col * static_cast<uint32_t>(sizeof(T));
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o.store1(T{}, oat + tile_row(i, e) * orow, y[i][e]);
    }
    fetch_v(c + 1);
    // S1 = exp(G_end) S0 + K^T (exp(G_end - G) U)
    Parts<NI> kc[2][4];
    auto read_t = [&](int n) __attribute__((always_inline)) {   // four tiles of S, 32 rows
#pragma unroll
      for (int t = 0; t < 4; ++t)
        kc[n & 1][t] = X::template by_col<NI>(sK, xl, 4 * (n % (DT / 4)) + t, n / (DT / 4));
    };
    Parts<NS> ep[2];
    read_t(0);
    const float last = sGate[63];
    decay *= last;
#pragma unroll
    for (int i = 0; i < 2; ++i) u[i] *= *reinterpret_cast<const f4*>(&sGate[64 + tile_row(i, 0) + 8 * g]);
    split_d<NS>(ep[0], u[0], u[1]);
#pragma unroll
    for (int t = 0; t < DT; ++t) S[t] *= last;
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 0; n < DT / 2; ++n) {
      if (n + 1 < DT / 2) read_t(n + 1);
      if (n == 0) {
#pragma unroll
        for (int i = 2; i < 4; ++i) u[i] *= *reinterpret_cast<const f4*>(&sGate[64 + tile_row(i, 0) + 8 * g]);
        split_d<NS>(ep[1], u[2], u[3]);
      }
      mmp<NS>(*reinterpret_cast<f4(*)[4]>(&S[4 * (n % (DT / 4))]), kc[n & 1], ep[n / (DT / 4)]);
      if constexpr (NI == 1)
        if (n == 0) interleave<10, 4 * NS, 4>();
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (NBUF == 1) {
      tiles_barrier();
      st.store(buf);
    } else {
      fetch(c + 2);
    }
  }
  if constexpr (MAPS) {   // less its decay, as the A operand of a product over its columns (or rows)
    uint16_t* p = a.maps + shead * NS * DK * DK;
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[t][e] -= tile_row(t, e) + 8 * g == col ? decay : 0.0f;
    if constexpr (MODE == kMaps) {
      const uint32_t to = col / 32 * 512 + (col % 32 / 8 * 16 + 4 * g) * 8 + col % 8;
#pragma unroll
      for (int t = 0; t < DT; ++t) {
        Parts<NS> f;
        split_d<NS>(f, S[t], S[t]);
#pragma unroll
        for (int n = 0; n < NS; ++n) {
          const uint4 u = __builtin_bit_cast(uint4, f.p[n]);
          const uint32_t i = to + (n * DT + t) * KS * 512;
          p[i] = static_cast<uint16_t>(u.x);
          p[i + 8] = static_cast<uint16_t>(u.x >> 16);
          p[i + 16] = static_cast<uint16_t>(u.y);
          p[i + 24] = static_cast<uint16_t>(u.y >> 16);
        }
      }
    } else {   // row col of the transpose: row 4 (col / 8) + col % 4 of tile 2 (col / 32) + col / 4 % 2
      const uint32_t to = (2 * (col >> 5) + ((col >> 2) & 1)) * KS * 512 + (16 * g + 4 * ((col >> 3) & 3) + (col & 3)) * 8;
#pragma unroll
      for (int x = 0; x < KS; ++x) {
        Parts<NS> f;
        split_d<NS>(f, S[2 * x], S[2 * x + 1]);
#pragma unroll
        for (int n = 0; n < NS; ++n) *reinterpret_cast<bh8*>(p + to + n * DT * KS * 512 + x * 512) = f.p[n];
      }
    }
    if (cs == 0 && lane == 0) a.decays[shead] = decay;
  } else if constexpr (MODE == kEnds) {
#pragma unroll
    for (int t = 0; t < DT; ++t) *reinterpret_cast<f4*>(a.ends + shead * dd + end_at + t * 256) = S[t];
  } else if (seg.last && a.hT) {
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) (a.hT + head * dd + tile_row(t, e) * a.Dv)[at] = S[t][e];
  }
}

// The states before the segments: S_{j+1} = E_j + d_j S_j + F_j S_j, with the
// decay d_j apart from the map.  E_j lies where S_{j+1} goes, with segment j; S_1
// is there already.  BACK: the gradients of the states behind them, from the last
// to the first, with the maps' transposes.  A workgroup has 16 columns of a sequence's
// head, a wave 32 rows of them; the rows of the next two maps are on their way
// in its registers, and the waves exchange the parts of the state in LDS.  1.8 us
// a map of 128 x 128, whose six products of parts follow each other (with two
// parts, three products: 1.4, and a wave for all rows, with maps in LDS, which
// reads four times as many operands in a row, 2.6).
template <int DK, bool BACK>
__global__ __launch_bounds__(2 * DK, 1) void k_delta_join(DeltaArgs a) {
  constexpr int KS = DK / 32, DT = DK / 16, NP = 3;
  __shared__ bh8 sS[2][KS][NP][64];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // (a head's workgroups on one XCD where the heads are a multiple of 8, as they
  // read the same maps)
  const uint32_t heads = static_cast<uint32_t>(min(a.B, a.inner)) * a.Hv, b = blockIdx.x % heads;
  const int slice = blockIdx.x / heads, h = b % a.Hv, c = b / a.Hv;
  int len, n0;   // the sequence's rows, the number of its first segment
  if (a.B > a.inner) {   // by segments, a sequence with its first
    const DeltaSeg seg(a, c, lane, false);
    if (seg.s < 0 || seg.j > 0) return;
    len = seg.len;
    n0 = c;
  } else if (a.cu) {
    const int row = clamp_row(a.cu[c], a.T);
    len = max(0, clamp_row(a.cu[c + 1], a.T) - row);
    n0 = row >> (6 + a.lseg);
  } else {
    len = a.T;
    n0 = c * (a.nseg / a.B - 1);
  }
  const int nmap = ((((len + kDeltaChunk - 1) / kDeltaChunk) + (1 << a.lseg) - 1) >> a.lseg) - 2;
  if (nmap <= 0) return;
  const int64_t next_seg = BACK ? -a.Hv : a.Hv;
  const int64_t from = static_cast<int64_t>(n0 + (BACK ? nmap : 0)) * a.Hv + h, step = next_seg * DK * a.Dv;
  const int64_t by = static_cast<int64_t>(n0 + (BACK ? nmap : 1)) * a.Hv + h;
  float* p = a.ends + from * DK * a.Dv + ((slice * DT + 2 * w) * 64 + lane) * 4;
  const uint16_t* f = a.maps + by * NP * DK * DK + (2 * w * KS * 64 + lane) * 8;
  const float* d = a.decays + by;
  struct Map {
    Parts<NP> f[2][KS];
    f4 e[2];
    float d;
  } map[2];
  auto fetch = [&](Map& m, int j) __attribute__((always_inline)) {   // (behind the last one the last again, unused)
    j = min(j, nmap - 1);
    const uint16_t* m0 = f + j * next_seg * NP * DK * DK;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      m.e[t] = *reinterpret_cast<const f4*>(p + (j + 1) * step + t * 256);
#pragma unroll
      for (int x = 0; x < KS; ++x)
#pragma unroll
        for (int n = 0; n < NP; ++n) m.f[t][x].p[n] = *reinterpret_cast<const bh8*>(m0 + ((n * DT + t) * KS + x) * 512);
    }
    m.d = d[j * next_seg];
  };
  f4 S[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) S[t] = *reinterpret_cast<const f4*>(p + t * 256);
  fetch(map[0], 0);
  fetch(map[1], 1);
  // (the state is waited for here: in the loop its wait would be one for all that
  // is on its way, in every turn)
  asm volatile("" : "+v"(S[0]), "+v"(S[1]));
  for (int j0 = 0; j0 < nmap; j0 += 2)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int j = j0 + q;
      if (j >= nmap) break;
      Map& m = map[q];
      Parts<NP> sp[KS];
      split_d<NP>(sp[0], S[0], S[1]);
#pragma unroll
      for (int n = 0; n < NP; ++n) sS[q][w][n][lane] = sp[0].p[n];
      tiles_barrier();
#pragma unroll
      for (int x = 0; x < KS; ++x)
#pragma unroll
        for (int n = 0; n < NP; ++n) sp[x].p[n] = sS[q][x][n][lane];
      f4 c[4];   // (four sums, not to wait for each product)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        c[2 + t] = f4{0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < 4; ++e) c[t][e] = fmaf(m.d, S[t][e], m.e[t][e]);
      }
#pragma unroll
      for (int x = 0; x < KS; x += 2)
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
          for (int k = 0; i + k < NP; ++k)
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
              for (int t = 0; t < 2; ++t)
                c[2 * y + t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(m.f[t][x + y].p[i], sp[x + y].p[k], c[2 * y + t], 0, 0, 0);
      fetch(m, j + 2);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        S[t] = c[t] + c[2 + t];
        *reinterpret_cast<f4*>(p + (j + 1) * step + t * 256) = S[t];
      }
    }
}

}  // namespace
}  // namespace m3
