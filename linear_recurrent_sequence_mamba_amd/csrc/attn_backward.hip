// attn_backward.hip -- the gradients of causal attention over packed sequences
// (gfx950).
//
//   p = exp(s - lse),  dp_ij = <do_i, v_j>,  D_i = <o_i, do_i>,
//   ds_ij = p_ij (dp_ij - D_i),
//   dv_j = sum_i p_ij do_i,  dk_j = scale sum_i ds_ij q_i,
//   dq_i = scale sum_j ds_ij k_j
//
// k_attn_stat turns (o, do, lse) into one pair per row and head; k_attn_dq
// takes queries as lanes and walks over keys, k_attn_dkv takes keys as lanes
// and walks over queries.  Both recompute s from q and k, so no sum is shared
// between workgroups: there are no atomics, and equal calls give equal bits.
// The heads of a group add up in one workgroup, or, where that would leave
// too few, in parts that k_attn_sum adds in order.
#include "attn_common.h"

namespace m3 {
namespace {

// D / 4 lanes to a row and head
template <typename T, int D>
__global__ __launch_bounds__(256) void k_attn_stat(AttnArgs a) {
  constexpr int G = D / 8;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * (256 / G) + threadIdx.x / G;
  const int64_t all = static_cast<int64_t>(a.Tq) * a.Hq;
  const int64_t m = n < all ? n : all - 1;
  const int64_t t = m / a.Hq;
  const int h = static_cast<int>(m % a.Hq), e = 8 * (threadIdx.x % G);
  float o[8], g[8], s = 0.0f;
  ld8(static_cast<const T*>(a.co), t * a.ldo + h * D + e, o);
  ld8(static_cast<const T*>(a.dout), t * a.lddo + h * D + e, g);
#pragma unroll
  for (int j = 0; j < 8; ++j) s = fmaf(o[j], g[j], s);
  s = group_sum<G>(s);
  if (n < all && e == 0)
    a.stat[static_cast<int64_t>(h) * a.Tq + t] = float2{a.clse[m] * kLog2eA, s};
}

// ---------------------------------------------------------------------------
// dq: 32 queries a wave, tiles of 32 keys in LDS
template <typename T, int D, int WAVES>
__global__ __launch_bounds__(64 * WAVES, sizeof(T) * D == 512 ? 1 : 2) void k_attn_dq(AttnArgs a) {
  using L = Tile<T, D>;
  constexpr int BM = 32 * WAVES, BN = 32;
  __shared__ __align__(16) char sKV[2][L::BYTES];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nslot = gridDim.x / a.Hq;
  const int h = blockIdx.x % a.Hq;
  const Slot sl = slot_of<BM>(a.cuq, a.S, a.Tq, nslot - 1 - static_cast<int>(blockIdx.x / a.Hq), lane);
  if (sl.s < 0) return;
  const int q0 = clamp_row(a.cuq[sl.s], a.Tq), q1 = clamp_row(a.cuq[sl.s + 1], a.Tq);
  const int k0 = clamp_row(a.cuk[sl.s], a.Tk), k1 = clamp_row(a.cuk[sl.s + 1], a.Tk);
  const int Lq = q1 - q0, Lk = max(0, k1 - k0);
  const int i0 = sl.tile * BM;
  if (i0 >= Lq) return;
  const int off = Lk - Lq, hk = h / (a.Hq / a.Hk), half = lane >> 5;
  const int iw = i0 + 32 * wave, i = iw + (lane & 31);
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
  const float2 st = a.stat[static_cast<int64_t>(h) * a.Tq + row];
  const float lse = st.x == -INFINITY ? INFINITY : st.x;   // no key: every weight 0
  f16v dq[D / 32];
#pragma unroll
  for (int d = 0; d < D / 32; ++d) dq[d] = f16v{};
  const float c = a.scale * kLog2eA;
  const int sees = min(i, Lq - 1) + off + 1;
  const int most = min(min(i0 + BM, Lq) + off, Lk);
  const int ntile = most <= 0 ? 0 : (most + BN - 1) / BN;
  const int wmost = min(min(iw + 32, Lq) + off, Lk);
  const T* kp = static_cast<const T*>(a.k) + static_cast<int64_t>(k0) * a.ldk + hk * D;
  const T* vp = static_cast<const T*>(a.v) + static_cast<int64_t>(k0) * a.ldv + hk * D;
  if (ntile > 0) {
    L::template load2<WAVES>(sKV[0], kp, a.ldk, vp, a.ldv, 0, Lk - 1, wave, lane);
  }
  for (int t = 0; t < ntile; ++t) {
    lds_loads_done();
    __syncthreads();
    if (t + 1 < ntile) {
      L::template load2<WAVES>(sKV[(t + 1) & 1], kp, a.ldk, vp, a.ldv, (t + 1) * BN, Lk - 1, wave, lane);
    }
    const int j0 = t * BN;
    if (j0 >= wmost) continue;
    const char* KV = sKV[t & 1];
    f16v s = f16v{}, dp = f16v{};
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      s = mma(L::frag(KV, 0, kk, lane), q[kk], s);
      dp = mma(L::frag(KV, 32, kk, lane), g[kk], dp);
    }
    float ds[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float p = __builtin_amdgcn_exp2f(fmaf(s[e], c, -lse));
      ds[e] = j0 + row_of(e, half) < sees ? p * (dp[e] - st.y) : 0.0f;
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      Frag<T> f;
      frag_from(f, ds + 8 * w);
#pragma unroll
      for (int d = 0; d < D / 32; ++d) dq[d] = mma(L::frag_t(KV, 16 * w, 32 * d, lane), f, dq[d]);
    }
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
// dk, dv: 32 keys a wave, tiles of 32 queries of the group's heads in LDS
template <typename T, int D, int WAVES>
__global__ __launch_bounds__(64 * WAVES, 1) void k_attn_dkv(AttnArgs a) {
  using L = Tile<T, D>;
  constexpr int BK = 32 * WAVES, BQ = 32;
  __shared__ __align__(16) char sQG[2][L::BYTES];
  __shared__ __align__(16) float sL[2][BQ], sD[2][BQ];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int per = a.Hk * a.gsplit;
  const int part = blockIdx.x % a.gsplit, hk = blockIdx.x % per / a.gsplit;
  // early keys are seen by most queries: they start first
  const Slot sl = slot_of<BK>(a.cuk, a.S, a.Tk, static_cast<int>(blockIdx.x / per), lane);
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
  f16v dk[D / 32], dv[D / 32];
#pragma unroll
  for (int d = 0; d < D / 32; ++d) dk[d] = dv[d] = f16v{};
  const float c = a.scale * kLog2eA;
  // the first query that sees the block's first key, in whole tiles
  const int first = max(0, j0 - off) / BQ;
  const int nt = max(0, (Lq + BQ - 1) / BQ - first), all = nt * gper;
  const int wfirst = jw - off;   // the first query that sees the wave's first key
  auto fetch = [&](int n, int buf) {
    const int h = hk * grp + part * gper + n / nt, i0 = (first + n % nt) * BQ;
    const T* qp = static_cast<const T*>(a.q) + static_cast<int64_t>(q0) * a.ldq + h * D;
    const T* gp = static_cast<const T*>(a.dout) + static_cast<int64_t>(q0) * a.lddo + h * D;
    L::template load2<WAVES>(sQG[buf], qp, a.ldq, gp, a.lddo, i0, Lq - 1, wave, lane);
    if (threadIdx.x < BQ) {
      const int i = i0 + threadIdx.x;
      const float2 st = a.stat[static_cast<int64_t>(h) * a.Tq + q0 + min(i, Lq - 1)];
      // rows without keys and rows past the end: every weight 0
      sL[buf][threadIdx.x] = i < Lq && st.x != -INFINITY ? st.x : INFINITY;
      sD[buf][threadIdx.x] = st.y;
    }
  };
  if (all > 0) fetch(0, 0);
  for (int n = 0; n < all; ++n) {
    lds_loads_done();
    __syncthreads();
    const int buf = n & 1;
    if (n + 1 < all) fetch(n + 1, buf ^ 1);
    const int i0 = (first + n % nt) * BQ;
    if (i0 + BQ <= wfirst) continue;
    const char* QG = sQG[buf];
    f16v s = f16v{}, dp = f16v{};
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      s = mma(L::frag(QG, 0, kk, lane), k[kk], s);
      dp = mma(L::frag(QG, 32, kk, lane), v[kk], dp);
    }
    float p[16], ds[16];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const f4 l4 = *reinterpret_cast<const f4*>(&sL[buf][8 * b + 4 * half]);
      const f4 d4 = *reinterpret_cast<const f4*>(&sD[buf][8 * b + 4 * half]);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int e = 4 * b + x;
        const float w = __builtin_amdgcn_exp2f(fmaf(s[e], c, -l4[x]));
        const bool on = i0 + 8 * b + 4 * half + x + off >= j && l4[x] != INFINITY;
        p[e] = on ? w : 0.0f;
        ds[e] = on ? w * (dp[e] - d4[x]) : 0.0f;
      }
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      Frag<T> fp, fd;
      frag_from(fp, p + 8 * w);
      frag_from(fd, ds + 8 * w);
#pragma unroll
      for (int d = 0; d < D / 32; ++d) {
        dv[d] = mma(L::frag_t(QG, 32 + 16 * w, 32 * d, lane), fp, dv[d]);
        dk[d] = mma(L::frag_t(QG, 16 * w, 32 * d, lane), fd, dk[d]);
      }
    }
  }
  if (j >= Lk) return;
  const int64_t at = (row * a.Hk + hk) * D + 4 * half;
  if (a.gsplit == 1) {
    T *ok = static_cast<T*>(a.dk) + at, *ov = static_cast<T*>(a.dv) + at;
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        put4(ok + 32 * d + 8 * e, dk[d][4 * e] * a.scale, dk[d][4 * e + 1] * a.scale,
             dk[d][4 * e + 2] * a.scale, dk[d][4 * e + 3] * a.scale);
        put4(ov + 32 * d + 8 * e, dv[d][4 * e], dv[d][4 * e + 1], dv[d][4 * e + 2], dv[d][4 * e + 3]);
      }
  } else {
    const int64_t to = static_cast<int64_t>(part) * a.Tk * a.Hk * D + at;
    float *ok = a.pk + to, *ov = a.pv + to;
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        put4(ok + 32 * d + 8 * e, dk[d][4 * e], dk[d][4 * e + 1], dk[d][4 * e + 2], dk[d][4 * e + 3]);
        put4(ov + 32 * d + 8 * e, dv[d][4 * e], dv[d][4 * e + 1], dv[d][4 * e + 2], dv[d][4 * e + 3]);
      }
  }
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

// Parts of a group of heads: enough workgroups of 128 keys to fill the chip
// twice, in equal parts.
int group_parts(int Tk, int S, int Hq, int Hk) {
  const int g = Hq / Hk;
  const int64_t blocks = (static_cast<int64_t>(Tk) / 128 + 1) * Hk;
  for (int n = 1; n < g; ++n)
    if (g % n == 0 && blocks * n >= 512) return n;
  return g;
}

template <typename T, int D>
hipError_t run(const AttnArgs& a, hipStream_t s) {
  constexpr int W = 4, B = 32 * W;
  const int64_t rows = static_cast<int64_t>(a.Tq) * a.Hq, per = 256 / (D / 8);
  k_attn_stat<T, D><<<static_cast<unsigned>((rows + per - 1) / per), 256, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t nk = (static_cast<int64_t>(a.Tk) / B + a.S) * a.Hk * a.gsplit;
  k_attn_dkv<T, D, W><<<static_cast<unsigned>(nk), 64 * W, 0, s>>>(a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (a.gsplit > 1) {
    const int64_t n = static_cast<int64_t>(a.Tk) * a.Hk * D / 4;
    k_attn_sum<T><<<static_cast<unsigned>((n + 255) / 256), 256, 0, s>>>(a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  const int64_t nq = (static_cast<int64_t>(a.Tq) / B + a.S) * a.Hq;
  k_attn_dq<T, D, W><<<static_cast<unsigned>(nq), 64 * W, 0, s>>>(a);
  return hipGetLastError();
}

constexpr size_t up256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

size_t attn_backward_workspace_bytes(int Tq, int Tk, int S, int Hq, int Hk, int D) {
  const int g = group_parts(Tk, S, Hq, Hk);
  size_t n = up256(sizeof(float2) * Tq * static_cast<size_t>(Hq));
  if (g > 1) n += 2 * up256(sizeof(float) * g * static_cast<size_t>(Tk) * Hk * D);
  return n;
}

hipError_t launch_attn_backward(AttnArgs& a, int bf16, void* ws, hipStream_t s) {
  a.gsplit = group_parts(a.Tk, a.S, a.Hq, a.Hk);
  char* c = static_cast<char*>(ws);
  a.stat = reinterpret_cast<float2*>(c);
  c += up256(sizeof(float2) * a.Tq * static_cast<size_t>(a.Hq));
  a.pk = reinterpret_cast<float*>(c);
  c += up256(sizeof(float) * a.gsplit * static_cast<size_t>(a.Tk) * a.Hk * a.D);
  a.pv = reinterpret_cast<float*>(c);
  if (bf16) return a.D == 64 ? run<bf16_t, 64>(a, s) : run<bf16_t, 128>(a, s);
  return a.D == 64 ? run<float, 64>(a, s) : run<float, 128>(a, s);
}

}  // namespace m3
