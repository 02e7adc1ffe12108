// delta_backward.hip -- the gradients of the gated delta rule (gfx950).
//
// With dO the gradient of the outputs, dS1 that of the state behind a chunk,
// and the chunk's T, P and U as in the scan (P with the scale in it):
//   dU = P^T dO + exp(G_end - G) K dS1,   dR = T^T dU,   dV = beta dR,
//   dS0 = exp(G_end) dS1 + Q^T (scale exp(G) dO) - K^T (exp(G) dV)
// is a chain over the chunks from the last to the first; and with
//   dP = scale dO U^T (j <= i),  dA = -dR U^T (j < i),  Gamma_ij = exp(G_i - G_j),
//   F = dP Gamma,  M = beta_i dA Gamma,  X1 = dO S0^T,  X2 = dR S0^T,  X3 = U dS1^T:
//   dQ = scale exp(G) X1 + F K
//   dK = F^T Q + (M + M^T) K - exp(G) beta X2 + exp(G_end - G) X3
//   dbeta_i = dR_i.Y_i + sum_j dA_ij Gamma_ij k_i.k_j,   Y = V - exp(G) K S0
// for each chunk by itself.  dR_i.Y_i is dR_i.v_i - exp(G_i) k_i.X2_i.  With
// C_ij = F_ij q_i.k_j + M_ij k_i.k_j (j < i) and z_j = exp(G_end - G_j) k_j.X3_j
//   dG_i = sum_j C_ij - sum_j C_ji + scale exp(G_i) q_i.X1_i - exp(G_i) beta_i k_i.X2_i - z_i,
// to which the chunk's last row adds sum_j z_j + exp(G_end) <S0, dS1>; and dg_t =
// sum_{i >= t} dG_i.  (dG_i is also q_i.dq_i - k_i.dk_i + 2 (dR_i.U_i - dV_i.v_i),
// but there the pairs of rows behind t, which are in dg_t twice with opposite
// signs, come from sums that are rounded apart: 2 to 5 times the error in fp32.)
#include "delta_chain.h"

namespace m3 {
namespace {

// ---------------------------------------------------------------------------
// The chain, as the scan's and with its segments: a wave holds 16 columns of dS.
// FULL false: only the gradient of the state before the segment, from none
// behind it (the last segment: from dhT).  Bound as the scan's: 5.5 us a chunk
// of 128 x 64.
template <typename T, int DK, int NW, int NBUF, bool FULL>
__device__ __forceinline__ void back_chain(const DeltaArgs& a, const DeltaSeg& seg, int h, int slice, char* smem) {
  using X = Rows64<DK>;
  using M = Rows64<64>;
  constexpr int NT = 64 * NW, KS = DK / 32, DT = DK / 16, NI = DeltaParts<T>::IN;
  using Tiles = ChainTiles<T, DK, NT, true>;
  constexpr int BK = Tiles::BK, BM = Tiles::BM, BUF = Tiles::BUF;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4, hk = h / (a.Hv / a.Hk);
  const int cs = slice * NW + w, col = 16 * cs + r;
  const Triangle tri(lane);
  const typename X::Lane xl(lane);
  const M::Lane ml(lane);
  const int64_t head = static_cast<int64_t>(seg.s) * a.Hv + h, shead = static_cast<int64_t>(seg.n) * a.Hv + h;
  const int64_t dd = static_cast<int64_t>(DK) * a.Dv;
  const uint32_t at = static_cast<uint32_t>(8 * g * a.Dv + col), end_at = (cs * DT * 64 + lane) * 4;
  const int ldo = a.Hv * a.Dv;

  f4 S[DT];
#pragma unroll
  for (int t = 0; t < DT; ++t) S[t] = f4{0, 0, 0, 0};
  if (!seg.last) {
    if constexpr (FULL)
#pragma unroll
      for (int t = 0; t < DT; ++t) S[t] = *reinterpret_cast<const f4*>(a.ends + shead * dd + end_at + t * 256);
  } else if (a.dhT) {
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[t][e] = (a.dhT + head * dd + tile_row(t, e) * a.Dv)[at];
  }

  Tiles st;
  Cols<T> stO;
  const int c0 = seg.c0, c1 = seg.c0 + seg.nch;
  auto rows = [&](int c) __attribute__((always_inline)) { return min(kDeltaChunk, seg.len - c * kDeltaChunk); };
  auto first = [&](int c) __attribute__((always_inline)) { return seg.row0 + static_cast<int64_t>(c) * kDeltaChunk; };
  auto fetch = [&](int c) __attribute__((always_inline)) {
    c = max(c, c0);
    const int64_t m = static_cast<int64_t>(seg.slot0 + c) * a.Hv + h;
    st.k.load(static_cast<const T*>(a.k) + first(c) * a.ldk + hk * DK, a.ldk, rows(c));
    st.m.load(a.pm + m * a.ldpm, 64, 64);
#pragma unroll
    for (int i = 0; i < Tiles::NG; ++i) st.g[i] = (a.pm + m * a.ldpm + kDeltaMatrix)[min(threadIdx.x + i * NT, 191u)];
    st.q.load(static_cast<const T*>(a.q) + first(c) * a.ldq + hk * DK, a.ldq, rows(c));
  };
  auto fetch_o = [&](int c) __attribute__((always_inline)) {
    c = max(c, c0);
    stO.load(static_cast<const T*>(a.dout) + first(c) * ldo + h * a.Dv, ldo, rows(c), col, g);
  };
  if (seg.nch > 0) {
    fetch(c1 - 1);
    fetch_o(c1 - 1);
    st.store(smem);
    if constexpr (NBUF == 2) fetch(c1 - 2);
  }
  char* buf = smem;
  for (int c = c1 - 1; c >= c0; --c) {
    const char *sK = buf, *sQ = buf + BK, *sM = buf + 2 * BK;
    const float* sGate = reinterpret_cast<const float*>(buf + 2 * BK + BM);
    const int64_t m = static_cast<int64_t>(seg.slot0 + c) * a.Hv + h;
    tiles_barrier();
    if constexpr (FULL)
#pragma unroll
      for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) (a.after + m * dd + tile_row(t, e) * a.Dv)[at] = S[t][e];
    // K dS1
    f4 ks[4];
    Parts<NI> ka[2][4];
    Parts<3> sp[2];
    auto read = [&](int x) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) ka[x & 1][i] = X::template by_row<NI>(sK, xl, i, x);
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) ks[i] = f4{0, 0, 0, 0};
    read(0);
    split_d<3>(sp[0], S[0], S[1]);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int x = 0; x < KS; ++x) {
      if (x + 1 < KS) {
        read(x + 1);
        split_d<3>(sp[(x + 1) & 1], S[2 * x + 2], S[2 * x + 3]);
      }
      mmp<3>(ks, ka[x & 1], sp[x & 1]);
      if constexpr (NI == 1) interleave<4, 12, 4>();
      __builtin_amdgcn_sched_barrier(0);
    }
    // dU = P^T dO + exp(G_end - G) K dS1
    Parts<1> ta[2][6];
    tri.pt6(ta[0], sM, ml, 0);
    f4 u[6], o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f4 en = *reinterpret_cast<const f4*>(&sGate[64 + tile_row(i, 0) + 8 * g]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        o[i][e] = stO.v[4 * i + e].f();
        u[i][e] = en[e] * ks[i][e];
      }
    }
    u[4] = u[5] = f4{0, 0, 0, 0};
    Parts<NI> op[2];
    split_d<NI>(op[0], o[0], o[1]);
    split_d<NI>(op[1], o[2], o[3]);
    fetch_o(c - 1);
    __builtin_amdgcn_sched_barrier(0);
    Parts<3> ep[2];
#pragma unroll
    for (int n = 0; n < 3; ++n) {
      if (n < 2) tri.pt6(ta[(n + 1) & 1], sM, ml, n + 1);
      mmt6<3>(u, ta[n & 1], op, n);
      // (in the products' time) scale exp(G) dO, for dS0
      if (n < 2) {
#pragma unroll
        for (int i = 2 * n; i < 2 * n + 2; ++i) o[i] *= a.scale * *reinterpret_cast<const f4*>(&sGate[tile_row(i, 0) + 8 * g]);
        split_d<3>(ep[n], o[2 * n], o[2 * n + 1]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    u[0] += u[4];
    u[1] += u[5];
    // dS0 = exp(G_end) dS1 + Q^T (scale exp(G) dO) ...
    const float last = sGate[63];
#pragma unroll
    for (int t = 0; t < DT; ++t) S[t] *= last;
    Parts<NI> kc[2][4];
    auto read_t = [&](const char* tile, int n) __attribute__((always_inline)) {   // four tiles of dS, 32 rows
#pragma unroll
      for (int t = 0; t < 4; ++t)
        kc[n & 1][t] = X::template by_col<NI>(tile, xl, 4 * (n % (DT / 4)) + t, n / (DT / 4));
    };
    auto add = [&](const char* tile) __attribute__((always_inline)) {
#pragma unroll
      for (int n = 0; n < DT / 2; ++n) {
        if (n + 1 < DT / 2) read_t(tile, n + 1);
        mmp<3>(*reinterpret_cast<f4(*)[4]>(&S[4 * (n % (DT / 4))]), kc[n & 1], ep[n / (DT / 4)]);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    read_t(sQ, 0);
    // dR = T^T dU: dU itself for the diagonal
    Parts<3> up[2];
    split_d<3>(up[0], u[0], u[1]);
    split_d<3>(up[1], u[2], u[3]);
    add(sQ);
    tri.tt6(ta[0], sM, ml, 0);
    u[4] = u[5] = f4{0, 0, 0, 0};
#pragma unroll
    for (int n = 0; n < 3; ++n) {
      if (n < 2) tri.tt6(ta[(n + 1) & 1], sM, ml, n + 1);
      mmt6<3>(u, ta[n & 1], up, n);
      if (n == 0 && NBUF == 2) {
        buf = buf == smem ? smem + BUF : smem;
        st.store(buf);   // (the last time unread)
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    u[0] += u[4];
    u[1] += u[5];
    read_t(sK, 0);
    // dV = beta dR
    {
      const ChunkRows dv(static_cast<T*>(a.dv) + first(c) * ldo + h * a.Dv, ldo, rows(c));
      const uint32_t orow = static_cast<uint32_t>(ldo) * static_cast<uint32_t>(sizeof(T));
      const uint32_t oat = 8 * g * orow + col * static_cast<uint32_t>(sizeof(T));
      float* dr = a.dr + m * 64 * a.Dv;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f4 st = *reinterpret_cast<const f4*>(&sGate[tile_row(i, 0) + 8 * g]);
        const f4 bt = *reinterpret_cast<const f4*>(&sGate[128 + tile_row(i, 0) + 8 * g]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (FULL) (dr + tile_row(i, e) * a.Dv)[at] = u[i][e];
          u[i][e] *= bt[e];
          if constexpr (FULL) dv.store1(T{}, oat + tile_row(i, e) * orow, u[i][e]);
          u[i][e] *= -st[e];
        }
      }
    }
    // ... - K^T (exp(G) dV)
    split_d<3>(ep[0], u[0], u[1]);
    split_d<3>(ep[1], u[2], u[3]);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (NBUF == 1) fetch(c - 1);   // (in few registers until then)
    add(sK);
    if constexpr (NBUF == 1) {
      tiles_barrier();
      st.store(buf);
    } else {
      fetch(c - 2);
    }
  }
  if constexpr (!FULL) {   // to where the segment before ends
#pragma unroll
    for (int t = 0; t < DT; ++t) *reinterpret_cast<f4*>(a.ends + (shead - a.Hv) * dd + end_at + t * 256) = S[t];
  } else if (seg.j == 0 && a.dh0) {
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) (a.dh0 + head * dd + tile_row(t, e) * a.Dv)[at] = S[t][e];
  }
}

template <typename T, int DK, int NW, int NBUF>
__global__ __launch_bounds__(64 * NW, sizeof(T) == 2 ? 2 : 1) void k_delta_back_chain(DeltaArgs a) {
  __shared__ __align__(16) char smem[NBUF * ChainTiles<T, DK, 64 * NW, true>::BUF];
  const int nsl = a.Dv / (16 * NW), n = blockIdx.x / nsl;
  const DeltaSeg seg(a, n / a.Hv, threadIdx.x & 63);
  if (seg.s >= 0) back_chain<T, DK, NW, NBUF, true>(a, seg, n % a.Hv, blockIdx.x % nsl, smem);
}

// the gradients before all segments but the first, and the maps of those between
template <typename T, int DK, int NW, int NBUF>
__global__ __launch_bounds__(64 * NW, sizeof(T) == 2 ? 2 : 1) void k_delta_back_segments(DeltaArgs a) {
  __shared__ __align__(16) char smem[NBUF * ChainTiles<T, DK, 64 * NW, true>::BUF];
  const int nv = a.Dv / (16 * NW), nsl = nv + DK / (16 * NW);
  const int n = blockIdx.x / nsl, slice = blockIdx.x % nsl;
  const DeltaSeg seg(a, n / a.Hv, threadIdx.x & 63, true);
  if (seg.s < 0) return;
  if (slice < nv) back_chain<T, DK, NW, NBUF, false>(a, seg, n % a.Hv, slice, smem);
  else if (!seg.last) chain<T, DK, NW, NBUF, kMapsT>(a, seg, n % a.Hv, slice - nv, smem);
}

// ---------------------------------------------------------------------------
// The gradients of q, k, g and beta of a chunk and a head of k, its value heads
// one after another (MULTI: more than one).  Wave w has the 16 channels
// tile_row(w, ..) of q and k, so it reads 16 rows of S0 and dS1 straight from
// memory; the products over value channels (X1, X2, X3, dP, dA) go by 64 of them
// with dO, dR and U in LDS, where K, Q, F^T and M^T follow: the transposes, as a
// lane has four consecutive rows of a tile's column.  dP and dA have twelve
// tiles (of two blocks of 32 by 32 on and one below the diagonal), which the
// waves share.
//
// 128 chunks of 32 heads of 128 x 64, bf16: 203 us for 780 MB, 3.8 TB/s.  Its
// registers leave room for one workgroup a CU, so that what a workgroup asks for
// first and its products do not overlap with another's; two (128 registers) spill:
// 400 us.  The next slab's rows are asked for as soon as the last one's are split.
// AHEAD: a workgroup goes on to another chunk and head, whose first rows it asks
// for before the products over tokens (without it 230 us); with 128 value channels
// or fp32 the registers for it are not there (a packed batch of 8192 tokens, 16
// heads on 8 of 128 x 128: 246 us with it, 226 without).  Some spill without it: 15
// registers of bf16 with shared heads of 128 x 128, 29 and 90 of fp32 with shared
// heads of 128 x 64 and 128 x 128, at most 11 of the others (4 x 2048 tokens, 32
// heads on 16 of 128 x 128, fp32: 652 us, 540 of the 672 MB that it writes are
// scratch).
template <typename T, int DK, bool KEEP>   // KEEP: K and Q stay for all heads
struct GradTiles {
  using M = Rows64<64>;
  static constexpr int NI = DeltaParts<T>::IN, NO = DeltaParts<T>::OUT;
  static constexpr int ONE = (NI + 2 * NO) * M::PLANE;
  static constexpr int KQ = 2 * NI * Rows64<DK>::PLANE, TWO = KQ + 2 * NO * M::PLANE;
  static constexpr int BYTES = KEEP ? KQ + ONE : ONE > TWO ? ONE : TWO;
};

// tiles (i, j) of the lower half, n = 0 .. 11
__device__ __forceinline__ constexpr int tile_i(int n) { return n < 4 ? n >> 1 : 2 + ((n - 4) >> 2); }
__device__ __forceinline__ constexpr int tile_j(int n) { return n < 4 ? n & 1 : (n - 4) & 3; }

template <typename T, int DK, int DV, bool MULTI>
__global__ __launch_bounds__(4 * DK, sizeof(T) == 2 ? 2 : 1) void k_delta_grads(DeltaArgs a) {
  using X = Rows64<DK>;
  using M = Rows64<64>;
  using G = GradTiles<T, DK, MULTI && sizeof(T) == 2>;
  constexpr int NI = G::NI, NO = G::NO, NW = DK / 16, NT = 64 * NW, NTILE = (12 + NW - 1) / NW, VN = 512 / NT;
  // where there is room, the sums over heads wait in LDS (in registers they spill),
  // and K and Q stay there
  constexpr bool PARK = MULTI && sizeof(T) == 2, AHEAD = DV == 64 && sizeof(T) == 2;
  __shared__ float sAcc[PARK ? 32 : 1][PARK ? NT : 1];
  __shared__ __align__(16) char smem[G::BYTES];
  __shared__ __align__(16) float sGate[kDeltaGates];
  __shared__ float sRow[2][NW][64], sE[4][64], sW[4][64], sC[4][64], sV[64], sEnd[NW];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g0 = lane >> 4;
  const int group = MULTI ? a.Hv / a.Hk : 1, items = a.nslot * a.Hk;
  auto seek = [&](int n) {   // the next chunk and head that there is
    while (n < items && DeltaSlot(a, n / a.Hk, lane).n <= 0) n += AHEAD ? static_cast<int>(gridDim.x) : items;
    return n;
  };
  int item = seek(blockIdx.x);
  if (item >= items) return;
  const typename X::Lane xl(lane);
  const M::Lane ml(lane);
  const int ldo = a.Hv * DV;
  char *sO = smem + (PARK ? G::KQ : 0), *sR = sO + NI * M::PLANE, *sUt = sR + NO * M::PLANE;
  char *sK = smem, *sQ = smem + NI * X::PLANE, *sF = smem + G::KQ, *sN = sF + NO * M::PLANE;
  const int wcol = X::tile_col(w, lane);   // the wave's channels in K and Q
  const int dkr = 32 * (w >> 1) + 8 * (r >> 2) + 4 * (w & 1) + (r & 3);   // the lane's channel of q and k
  const int64_t dd = static_cast<int64_t>(DK) * DV;
  const uint32_t sat0 = static_cast<uint32_t>(dkr * DV + 8 * g0);
  Stage<T, 64, NT> so, sv;
  Stage<float, 64, NT> sr, su;
  Vec8<float> vs[2], vd[2];
  float gate = 0.0f, gate2 = 0.0f;
  // 64 columns of a chunk's rows, and of its states
  auto fetch = [&](const DeltaSlot& sl, int64_t m, int h, int c0, int tid) __attribute__((always_inline)) {
    so.load(static_cast<const T*>(a.dout) + sl.row0 * ldo + h * DV + c0, ldo, sl.n, tid);
    sv.load(static_cast<const T*>(a.v) + sl.row0 * a.ldv + h * DV + c0, a.ldv, sl.n, tid);
    sr.load(a.dr + m * 64 * DV + c0, DV, 64, tid);
    su.load(a.cstates + m * a.ldpm + dd + c0, DV, 64, tid);
  };
  auto fetch_s = [&](int64_t m, int c0, int x, uint32_t sat) __attribute__((always_inline)) {
    vs[x].load(a.cstates + m * a.ldpm + c0 + 32 * x + sat);
    vd[x].load(a.after + m * dd + c0 + 32 * x + sat);
  };
  auto fetch_first = [&](const DeltaSlot& sl, int64_t m, int h, int tid, uint32_t sat) __attribute__((always_inline)) {
    const float* p = a.pm + m * a.ldpm + kDeltaMatrix;
    gate = p[min(tid, kDeltaGates - 1)];
    if (NT < kDeltaGates) gate2 = p[min(tid + NT, kDeltaGates - 1)];
    fetch(sl, m, h, 0, tid);
    fetch_s(m, 0, 0, sat);
    fetch_s(m, 0, 1, sat);
  };
  auto head_of = [&](int n, int h) { return static_cast<int64_t>(n / a.Hk) * a.Hv + h; };
  if constexpr (AHEAD) {
    const DeltaSlot sl(a, item / a.Hk, lane);
    const int h = item % a.Hk * group;
    fetch_first(sl, head_of(item, h), h, threadIdx.x, sat0);
  }
  for (;;) {
    const int hk = item % a.Hk, slot = item / a.Hk;
    const DeltaSlot sl(a, slot, lane);
    // (behind the last one itself again, unused)
    int next = AHEAD ? seek(item + gridDim.x) : items;
    const bool more = next < items;
    if (!more) next = item;
    f4 dq[4], dk[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) dq[i] = dk[i] = f4{0, 0, 0, 0};

    auto fetch_kq = [&](Stage<T, DK, NT>& k, Stage<T, DK, NT>& q, int tid) __attribute__((always_inline)) {
      k.load(static_cast<const T*>(a.k) + sl.row0 * a.ldk + hk * DK, a.ldk, sl.n, tid);
      q.load(static_cast<const T*>(a.q) + sl.row0 * a.ldq + hk * DK, a.ldq, sl.n, tid);
    };
    if constexpr (PARK) {
      Stage<T, DK, NT> k, q;
      fetch_kq(k, q, threadIdx.x);
      k.store(sK);
      q.store(sQ);
    }

    for (int h = hk * group; h < (hk + 1) * group; ++h) {
      // (opaque: addresses are made again for each head, not kept over the loop)
      const int tid = MULTI || AHEAD ? opaque(threadIdx.x) : threadIdx.x, g = MULTI || AHEAD ? opaque(g0) : g0;
      const int64_t m = static_cast<int64_t>(slot) * a.Hv + h;
      const uint32_t sat = static_cast<uint32_t>(dkr * DV + 8 * g);
      f4 x1[4], x2[4], x3[4], dp[NTILE], da[NTILE];
#pragma unroll
      for (int i = 0; i < 4; ++i) x1[i] = x2[i] = x3[i] = f4{0, 0, 0, 0};
#pragma unroll
      for (int n = 0; n < NTILE; ++n) dp[n] = da[n] = f4{0, 0, 0, 0};
      float both = 0.0f;   // of <S0, dS1>
      float vdot[VN];
#pragma unroll
      for (int n = 0; n < VN; ++n) vdot[n] = 0.0f;
      if constexpr (!AHEAD) fetch_first(sl, m, h, tid, sat);
      Stage<T, DK, NT> stK, stQ;
      tiles_barrier();
      if (tid < kDeltaGates) sGate[tid] = gate;
      if (NT < kDeltaGates && tid + NT < kDeltaGates) sGate[tid + NT] = gate2;
      if (threadIdx.x < 256) {
        const int n = threadIdx.x / 64, i = threadIdx.x % 64;
        sE[n][i] = sW[n][i] = sC[n][i] = 0.0f;
      }
#pragma unroll
      for (int c0 = 0; c0 < DV; c0 += 64) {
        if (c0 > 0) tiles_barrier();
        so.store(sO, tid);
#pragma unroll
        for (int n = 0; n < VN; ++n) {
          const int row = tid / 8 + n * (NT / 8), c = tid % 8 * 8;
          float f[8], v[8];
          sr.v[n].get(f);
          sv.v[n].get(v);
#pragma unroll
          for (int j = 0; j < 8; ++j) vdot[n] = fmaf(f[j], v[j], vdot[n]);
          M::put<NO>(sR, row, c, f);
          su.v[n].get(f);
          M::put<NO>(sUt, row, c, f);
        }
        if (c0 + 64 < DV) {
          fetch(sl, m, h, c0 + 64, tid);
        } else {
          if constexpr (!PARK) fetch_kq(stK, stQ, tid);
        }
        tiles_barrier();
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          Parts<NO> ps, pd;
          {
            float f[8], d[8];
            vs[x].get(f);
            vd[x].get(d);
#pragma unroll
            for (int j = 0; j < 8; ++j) both = fmaf(f[j], d[j], both);
            split8<NO>(ps, f);
            split8<NO>(pd, d);
            if (c0 + 64 < DV) fetch_s(m, c0 + 64, x, sat);
          }
          {
            Parts<NI> oa[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) oa[i] = M::by_row<NI>(sO, ml, i, x);
            mmp<NO>(x1, oa, ps);
          }
          __builtin_amdgcn_sched_barrier(0);
          {
            Parts<NO> ra[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) ra[i] = M::by_row<NO>(sR, ml, i, x);
            mmp<NO>(x2, ra, ps);
          }
          __builtin_amdgcn_sched_barrier(0);
          {
            Parts<NO> ua[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) ua[i] = M::by_row<NO>(sUt, ml, i, x);
            mmp<NO>(x3, ua, pd);
          }
          __builtin_amdgcn_sched_barrier(0);
          // the wave's own tiles of dP and dA
#pragma unroll
          for (int n = 0; n < NTILE; ++n) {
            const int t = w + n * NW;
            if (t < 12) {
              const Parts<NO> ub = M::by_row<NO>(sUt, ml, tile_j(t), x);
              dp[n] = mmp<NO>(M::by_row<NI>(sO, ml, tile_i(t), x), ub, dp[n]);
              da[n] = mmp<NO>(M::by_row<NO>(sR, ml, tile_i(t), x), ub, da[n]);
            }
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
#pragma unroll
      for (int n = 0; n < VN; ++n) {
        const float d = group_sum<8>(vdot[n]);
        if (tid % 8 == 0) sV[tid / 8 + n * (NT / 8)] = d;
      }
      both = group_sum<64>(both);
      tiles_barrier();
      if constexpr (!PARK) {
        stK.store(sK, tid);
        stQ.store(sQ, tid);
        tiles_barrier();
      }
      if constexpr (AHEAD) {
        const bool same = MULTI && h + 1 < (hk + 1) * group;
        const int n = same ? item : next, nh = same ? h + 1 : next % a.Hk * group;
        const DeltaSlot nsl(a, n / a.Hk, lane);
        fetch_first(nsl, head_of(n, nh), nh, tid, sat);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int n = 0; n < NTILE; ++n) {
        const int t = w + n * NW;
        if (t < 12) {
          const int ti = tile_i(t), tj = tile_j(t), j = tile_row(tj, 0) + 8 * (r >> 2) + (r & 3);
          const int i0 = tile_row(ti, 0) + 8 * g;
          f4 kk = f4{0, 0, 0, 0}, qk = f4{0, 0, 0, 0};
#pragma unroll
          for (int x = 0; x < DK / 32; ++x) {
            const Parts<NI> kb = X::template by_row<NI>(sK, xl, tj, x);
            kk = mmp<3>(X::template by_row<NI>(sK, xl, ti, x), kb, kk);
            qk = mmp<3>(X::template by_row<NI>(sQ, xl, ti, x), kb, qk);
          }
          const float gh = sGate[192 + j], gl = sGate[256 + j];
          const f4 hi = *reinterpret_cast<const f4*>(&sGate[192 + i0]), lo = *reinterpret_cast<const f4*>(&sGate[256 + i0]);
          const f4 bt = *reinterpret_cast<const f4*>(&sGate[128 + i0]);
          float col = 0.0f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float gam = i0 + e >= j ? __builtin_amdgcn_exp2f((hi[e] - gh) + (lo[e] - gl)) : 0.0f;
            // (a product that is not finite stays out of the half that is not there)
            const float ag = i0 + e > j ? -da[n][e] * gam : 0.0f, ak = ag == 0.0f ? 0.0f : ag * kk[e];
            dp[n][e] = i0 + e >= j ? a.scale * dp[n][e] * gam : 0.0f;
            da[n][e] = bt[e] * ag;
            // (the diagonal does not depend on G)
            const float c = fmaf(bt[e], ak, i0 + e == j || dp[n][e] == 0.0f ? 0.0f : dp[n][e] * qk[e]);
            col += c;
            const float es = group_sum<16>(ak), cs = group_sum<16>(c);
            if (r == 0) {
              sE[tj][i0 + e] = es;
              sW[tj][i0 + e] = cs;
            }
          }
          col += __shfl_xor(col, 16, 64);
          col += __shfl_xor(col, 32, 64);
          if (g == 0) sC[ti][j] = col;
          Parts<NO> pf;
          split_d<NO>(pf, dp[n], da[n]);
          char* to = smem + 2 * NI * X::PLANE + M::at(j, i0 & ~7) + 2 * (i0 & 7);
#pragma unroll
          for (int q = 0; q < NO; ++q) {
            const uint4 u = __builtin_bit_cast(uint4, pf.p[q]);
            *reinterpret_cast<uint2*>(to + q * M::PLANE) = uint2{u.x, u.y};
            *reinterpret_cast<uint2*>(to + (NO + q) * M::PLANE) = uint2{u.z, u.w};
          }
        }
      }
      tiles_barrier();
      // dQ = scale exp(G) X1 + F K,  dK = F^T Q + (M + M^T) K - exp(G) beta X2 + exp(G_end - G) X3
      float re = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f4 st = *reinterpret_cast<const f4*>(&sGate[tile_row(i, 0) + 8 * g]);
        const f4 en = *reinterpret_cast<const f4*>(&sGate[64 + tile_row(i, 0) + 8 * g]);
        const f4 bt = *reinterpret_cast<const f4*>(&sGate[128 + tile_row(i, 0) + 8 * g]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = tile_row(i, e) + 8 * g;
          const float k = X::template get<NI>(sK, row, dkr), q = X::template get<NI>(sQ, row, dkr);
          const float x = x3[i][e] * en[e], y = st[e] * bt[e] * x2[i][e];
          x1[i][e] *= a.scale * st[e];
          const float d = group_sum<16>(fmaf(q, x1[i][e], -k * (x + y))), kx = group_sum<16>(k * x2[i][e]);
          if (r == 0) {
            sRow[0][w][row] = d;
            sRow[1][w][row] = kx;
          }
          re = fmaf(k, x, re);
          x2[i][e] = x - y;
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const Parts<NI> kb = X::template by_col<NI>(sK, wcol, x), qb = X::template by_col<NI>(sQ, wcol, x);
        Parts<NO> f[4];
        // columns of block x and rows of its and later blocks; by_col: of the
        // transpose's rows, which are its columns
#pragma unroll
        for (int i = 2 * x; i < 4; ++i) f[i] = M::by_col<NO>(sF, ml, i, x);
#pragma unroll
        for (int i = 2 * x; i < 4; ++i) x1[i] = mmp<NO>(f[i], kb, x1[i]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 2 * x; i < 4; ++i) f[i] = M::by_col<NO>(sN, ml, i, x);
#pragma unroll
        for (int i = 2 * x; i < 4; ++i) x2[i] = mmp<NO>(f[i], kb, x2[i]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 2 * x + 2; ++i) f[i] = M::by_row<NO>(sF, ml, i, x);
#pragma unroll
        for (int i = 0; i < 2 * x + 2; ++i) x2[i] = mmp<NO>(f[i], qb, x2[i]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 2 * x + 2; ++i) f[i] = M::by_row<NO>(sN, ml, i, x);
#pragma unroll
        for (int i = 0; i < 2 * x + 2; ++i) x2[i] = mmp<NO>(f[i], kb, x2[i]);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (PARK) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float *q = &sAcc[4 * i + e][tid], *k = &sAcc[16 + 4 * i + e][tid];
            *q = h > hk * group ? *q + x1[i][e] : x1[i][e];
            *k = h > hk * group ? *k + x2[i][e] : x2[i][e];
          }
        } else if constexpr (MULTI) {
          dq[i] += x1[i];
          dk[i] += x2[i];
        }
      }
      re = group_sum<64>(re);
      if (lane == 0) sEnd[w] = fmaf(sGate[63], both, re);
      tiles_barrier();
      if (w == 0) {
        float d = 0.0f, x = 0.0f, end = 0.0f;
#pragma unroll
        for (int n = 0; n < NW; ++n) {
          d += sRow[0][n][lane];
          x += sRow[1][n][lane];
          end += sEnd[n];
        }
        const float db = sV[lane] - sGate[lane] * x + (sE[0][lane] + sE[1][lane]) + (sE[2][lane] + sE[3][lane]);
        float dG = d;
#pragma unroll
        for (int n = 0; n < 4; ++n) dG += sW[n][lane] - sC[n][lane];
        if (lane == 63) dG += end;
        // sums of the rows from here on
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
          const float y = __shfl_down(dG, o, 64);
          if (lane + o < 64) dG += y;
        }
        if (lane < sl.n) {
          const int64_t at = (sl.row0 + lane) * a.Hv + h;
          static_cast<T*>(a.dg)[at] = from_f32<T>(dG);
          static_cast<T*>(a.dbeta)[at] = from_f32<T>(db);
        }
      }
      if constexpr (!MULTI) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          dq[i] = x1[i];
          dk[i] = x2[i];
        }
      }
    }
    const int ldq = a.Hk * DK;
    const ChunkRows oq(static_cast<T*>(a.dq) + sl.row0 * ldq + hk * DK, ldq, sl.n);
    const ChunkRows ok(static_cast<T*>(a.dk) + sl.row0 * ldq + hk * DK, ldq, sl.n);
    const uint32_t orow = static_cast<uint32_t>(ldq) * static_cast<uint32_t>(sizeof(T));
    const uint32_t oat = 8 * g0 * orow + dkr * static_cast<uint32_t>(sizeof(T));
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        oq.store1(T{}, oat + tile_row(i, e) * orow, PARK ? sAcc[4 * i + e][threadIdx.x] : dq[i][e]);
        ok.store1(T{}, oat + tile_row(i, e) * orow, PARK ? sAcc[16 + 4 * i + e][threadIdx.x] : dk[i][e]);
      }
    if (!more) break;
    item = next;
  }
}

template <typename T, int DK, int NW>
hipError_t run_back_chain(const DeltaArgs& a, hipStream_t s) {
  constexpr int NBUF = sizeof(T) == 2 && NW == 8 ? 2 : 1;
  const int64_t heads = static_cast<int64_t>(a.nseg) * a.Hv;
  if (a.lseg < 30) {
    k_delta_back_segments<T, DK, NW, NBUF>
        <<<static_cast<unsigned>(static_cast<int64_t>(a.inner) * a.Hv * ((a.Dv + DK) / (16 * NW))), 64 * NW, 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    k_delta_join<DK, true>
        <<<static_cast<unsigned>(static_cast<int64_t>(a.B < a.inner ? a.B : a.inner) * a.Hv * (a.Dv / 16)), 2 * DK, 0, s>>>(a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  k_delta_back_chain<T, DK, NW, NBUF><<<static_cast<unsigned>(heads * (a.Dv / (16 * NW))), 64 * NW, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T, int DK>
hipError_t run_backward(const DeltaArgs& a, hipStream_t s) {
  hipError_t e;
  if constexpr (DK == 128 && sizeof(T) == 2)
    e = a.Dv == 128 ? run_back_chain<T, DK, 8>(a, s) : run_back_chain<T, DK, 4>(a, s);
  else
    e = run_back_chain<T, DK, 4>(a, s);
  if (e != hipSuccess) return e;
  const int64_t items = static_cast<int64_t>(a.nslot) * a.Hk;
  const bool multi = a.Hv != a.Hk, ahead = a.Dv == 64 && sizeof(T) == 2;
  const int most = 256 * (multi || DK == 128 ? 1 : 2);   // as many as are resident
  const unsigned grid = static_cast<unsigned>(ahead && items > most ? most : items);
  if (a.Dv == 64) {
    if (a.Hv == a.Hk) k_delta_grads<T, DK, 64, false><<<grid, 4 * DK, 0, s>>>(a);
    else k_delta_grads<T, DK, 64, true><<<grid, 4 * DK, 0, s>>>(a);
  } else {
    if (a.Hv == a.Hk) k_delta_grads<T, DK, 128, false><<<grid, 4 * DK, 0, s>>>(a);
    else k_delta_grads<T, DK, 128, true><<<grid, 4 * DK, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace

size_t delta_backward_workspace_bytes(int B, int T, int Hv, int Dk, int Dv, bool packed) {
  return sizeof(float) * static_cast<size_t>(delta_slots(B, T, packed)) * Hv * (Dk + kDeltaChunk) * Dv +
         delta_segment_bytes(delta_plan(B, T, Hv, Dk, Dv, packed, true), B, Hv, Dk, Dv, true);
}

void delta_backward_carve(DeltaArgs& a, void* ws) {
  const size_t chunks = static_cast<size_t>(delta_slots(a.B, a.T, a.cu != nullptr)) * a.Hv;
  a.ldpm = delta_state_floats(a.Dk, a.Dv);
  a.pm = const_cast<float*>(a.cstates) + static_cast<size_t>(a.Dk + kDeltaChunk) * a.Dv;   // (only read)
  a.after = static_cast<float*>(ws);
  a.dr = a.after + static_cast<size_t>(a.Dk) * a.Dv * chunks;
  delta_carve_segments(a, delta_plan(a.B, a.T, a.Hv, a.Dk, a.Dv, a.cu != nullptr, true),
                       a.dr + static_cast<size_t>(kDeltaChunk) * a.Dv * chunks, true);
}

hipError_t launch_delta_backward(DeltaArgs& a, int bf16, hipStream_t s) {
  if (bf16) return a.Dk == 64 ? run_backward<bf16_t, 64>(a, s) : run_backward<bf16_t, 128>(a, s);
  return a.Dk == 64 ? run_backward<float, 64>(a, s) : run_backward<float, 128>(a, s);
}

}  // namespace m3
