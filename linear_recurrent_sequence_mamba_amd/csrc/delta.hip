// delta.hip -- the gated delta rule (gfx950): the scan over a prompt (dense or
// packed) and one decode step.
//
// Per value head, with a state S [Dk, Dv] in fp32:
//   S' = exp(g_t) S_{t-1},  u_t = beta_t (v_t - S'^T k_t),
//   S_t = S' + k_t u_t^T,   o_t = scale S_t^T q_t
//
// Over a chunk of 64 tokens, with G the running sum of g inside it and S0 the
// state before it, the u of all tokens solve a triangular system:
//   E_ij = exp(G_i - G_j) k_i.k_j (j < i),  T = (1 + diag(beta) E)^-1,
//   U = T beta (V - exp(G) K S0),           P_ij = exp(G_i - G_j) q_i.k_j (j <= i),
//   O = scale (exp(G) Q S0 + P U),          S1 = exp(G_end) S0 + K^T (exp(G_end - G) U)
//
// k_delta_chunk makes T and P of every chunk and head at once; k_delta_chain
// walks each sequence's chunks with the state in registers.
#include "delta_common.h"

namespace m3 {
namespace {

// ---------------------------------------------------------------------------
// T, P and the gates of a chunk of one head.  The products K K^T and Q K^T are
// formed tile by tile, wave w those of rows 16 w ..; T by blocks of 16 in fp32:
// the diagonal's by substitution, a column a lane, then, diagonal by diagonal,
//   T_IJ = -T_II sum_{J <= K < I} A_IK T_KJ.
// Differences of G are taken in fp64, as G may be large where its differences
// are small.
template <typename T, int DK>
__global__ __launch_bounds__(256) void k_delta_chunk(DeltaArgs a) {
  using X = Rows64<DK>;
  constexpr int NI = DeltaParts<T>::IN, LM = 68;
  // K and Q, then the matrices A and [T \ P^T]
  constexpr int TILES = 2 * NI * X::PLANE, MATS = 2 * 64 * LM * static_cast<int>(sizeof(float));
  __shared__ __align__(16) char smem[TILES > MATS ? TILES : MATS];
  __shared__ double sG[64];
  __shared__ float sB[64];
  char *sK = smem, *sQ = smem + NI * X::PLANE;
  float(*sA)[LM] = reinterpret_cast<float(*)[LM]>(smem);
  float(*sM)[LM] = reinterpret_cast<float(*)[LM]>(smem + MATS / 2);
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int h = blockIdx.x % a.Hv, slot = blockIdx.x / a.Hv, hk = h / (a.Hv / a.Hk);
  const DeltaSlot sl(a, slot, lane);
  if (sl.n <= 0) return;
  Stage<T, DK, 256> stage;
  stage.load(static_cast<const T*>(a.k) + sl.row0 * a.ldk + hk * DK, a.ldk, sl.n);
  Stage<T, DK, 256> stage_q;
  stage_q.load(static_cast<const T*>(a.q) + sl.row0 * a.ldq + hk * DK, a.ldq, sl.n);
  if (w == 0) {
    const int64_t row = sl.row0 + min(lane, sl.n - 1);
    float gt = ld1(static_cast<const T*>(a.g), row * a.ldg + h);
    float bt = ld1(static_cast<const T*>(a.beta), row * a.ldb + h);
    if (lane >= sl.n) gt = bt = 0.0f;
    gt = gt < -128.0f ? -128.0f : gt;   // exp is 0 there, and -inf has no differences
    double G = gt;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const double o = __shfl_up(G, d, 64);
      if (lane >= d) G += o;
    }
    sG[lane] = G;
    sB[lane] = bt;
    const double end = __shfl(G, 63, 64);
    float* p = a.gates + (static_cast<int64_t>(slot) * a.Hv + h) * 192 + lane;
    p[0] = expf(static_cast<float>(G));
    p[64] = expf(static_cast<float>(end - G));
    p[128] = bt;
  }
  stage.store(sK, sl.n);
  stage_q.store(sQ, sl.n);
  __syncthreads();

  f4 kk[4], qk[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) kk[j] = qk[j] = f4{0, 0, 0, 0};
#pragma unroll
  for (int c = 0; c < DK; c += 32) {
    const Parts<NI> ka = X::template by_row<NI>(sK, 16 * w, c, lane);
    const Parts<NI> qa = X::template by_row<NI>(sQ, 16 * w, c, lane);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j <= w) {
        const Parts<NI> kb = X::template by_row<NI>(sK, 16 * j, c, lane);
        kk[j] = mmp<3>(ka, kb, kk[j]);
        qk[j] = mmp<3>(qa, kb, qk[j]);
      }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j <= w) {
      const double Gj = sG[16 * j + r];
      f4 p;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = 16 * w + 4 * g + e;
        const bool in = j < w || r <= 4 * g + e, strict = j < w || r < 4 * g + e;
        const float d = in ? expf(static_cast<float>(sG[i] - Gj)) : 0.0f;
        sA[i][16 * j + r] = strict ? sB[i] * d * kk[j][e] : 0.0f;
        p[e] = in ? a.scale * d * qk[j][e] : 0.0f;
      }
      // P^T on and above the diagonal
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (j < w || r <= 4 * g + e) sM[16 * j + r][16 * w + 4 * g + e] = p[e];
    }
  __syncthreads();
  {   // the diagonal's blocks: x = column r of (1 + A_ww)^-1
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = i == r ? 1.0f : 0.0f;
#pragma unroll
      for (int j = 0; j < i; ++j) s = fmaf(-sA[16 * w + i][16 * w + j], x[j], s);
      x[i] = s;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (g == i / 4 && r < i) sM[16 * w + i][16 * w + r] = x[i];
  }
#pragma unroll
  for (int d = 1; d < 4; ++d) {
    __syncthreads();
    if (w + d < 4) {
      const int I = w + d;
      f4 m = f4{0, 0, 0, 0};
#pragma unroll
      for (int K = 0; K < 3; ++K)
        if (K >= w && K < I) {
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const float av = sA[16 * I + r][16 * K + 4 * n + g];
            float tv = sM[16 * K + 4 * n + g][16 * w + r];
            if (K == w) tv = r < 4 * n + g ? tv : r == 4 * n + g ? 1.0f : 0.0f;
            m = __builtin_amdgcn_mfma_f32_16x16x4f32(av, tv, m, 0, 0, 0);
          }
        }
      f4 t = f4{0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < 4; ++e) {   // k slot g is row 4 g + e of m
        const int c = 4 * g + e;
        float tv = sM[16 * I + r][16 * I + c];
        tv = c < r ? tv : c == r ? 1.0f : 0.0f;
        t = __builtin_amdgcn_mfma_f32_16x16x4f32(-tv, m[e], t, 0, 0, 0);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) sM[16 * I + 4 * g + e][16 * w + r] = t[e];
    }
  }
  __syncthreads();
  float* out = a.pm + (static_cast<int64_t>(slot) * a.Hv + h) * 4096;
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const int x = threadIdx.x + 256 * n;
    *reinterpret_cast<f4*>(out + 4 * x) = *reinterpret_cast<const f4*>(&sM[x / 16][x % 16 * 4]);
  }
}

// ---------------------------------------------------------------------------
// The chain.  A wave holds 16 columns of a head's state, so that nothing of it
// is ever exchanged; the NW waves of a workgroup share K, Q and the chunk's
// matrix in LDS.  The next chunk is on its way in registers meanwhile.
template <typename T, int DK, int NW>
__global__ __launch_bounds__(64 * NW) void k_delta_chain(DeltaArgs a) {
  using X = Rows64<DK>;
  using M = Rows64<64>;
  constexpr int NI = DeltaParts<T>::IN, NO = DeltaParts<T>::OUT, NT = 64 * NW, KS = DK / 32, DT = DK / 16;
  __shared__ __align__(16) char sK[NI * X::PLANE], sQ[NI * X::PLANE], sM[3 * M::PLANE];
  __shared__ __align__(16) float sGate[192];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int nsl = a.Dv / (16 * NW);
  int n = blockIdx.x;
  const int slice = n % nsl;
  n /= nsl;
  const int h = n % a.Hv, s = n / a.Hv, hk = h / (a.Hv / a.Hk);
  const int col = (slice * NW + w) * 16 + r;
  const DeltaSeq seq(a, s);
  const Triangle tri(lane);
  const int64_t state = (static_cast<int64_t>(s) * a.Hv + h) * DK * a.Dv + col;

  f4 S[DT];
#pragma unroll
  for (int t = 0; t < DT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) S[t][e] = a.h0 ? a.h0[state + static_cast<int64_t>(16 * t + 4 * g + e) * a.Dv] : 0.0f;

  const int nch = (seq.len + kDeltaChunk - 1) / kDeltaChunk;
  Stage<T, DK, NT> stK, stQ;
  Stage<float, 64, NT> stM;
  float stG[(192 + NT - 1) / NT];
  Raw1<T> stV[16];
  auto fetch = [&](int c) __attribute__((always_inline)) {
    const int64_t row0 = seq.row0 + static_cast<int64_t>(c) * kDeltaChunk;
    const int cnt = min(kDeltaChunk, seq.len - c * kDeltaChunk);
    const int64_t at = static_cast<int64_t>(seq.slot0 + c) * a.Hv + h;
    stK.load(static_cast<const T*>(a.k) + row0 * a.ldk + hk * DK, a.ldk, cnt);
    stM.load(a.pm + at * 4096, 64, 64);
#pragma unroll
    for (int i = 0; i < (192 + NT - 1) / NT; ++i)
      stG[i] = a.gates[at * 192 + min(static_cast<int>(threadIdx.x) + i * NT, 191)];
    const T* v = static_cast<const T*>(a.v) + row0 * a.ldv + h * a.Dv + col;
#pragma unroll
    for (int i = 0; i < 16; ++i) stV[i].load(v, min(16 * (i / 4) + 4 * g + i % 4, cnt - 1) * a.ldv);
    stQ.load(static_cast<const T*>(a.q) + row0 * a.ldq + hk * DK, a.ldq, cnt);
  };
  if (nch > 0) fetch(0);
  for (int c = 0; c < nch; ++c) {
    const int cnt = min(kDeltaChunk, seq.len - c * kDeltaChunk);
    stK.store(sK, cnt);
    stQ.store(sQ, cnt);
#pragma unroll
    for (int i = 0; i < Stage<float, 64, NT>::N; ++i) {
      const int x = threadIdx.x + i * NT;
      float f[8];
      stM.v[i].get(f);
      M::template put<3>(sM, x / 8, x % 8 * 8, f);
    }
#pragma unroll
    for (int i = 0; i < (192 + NT - 1) / NT; ++i)
      if (threadIdx.x + i * NT < 192) sGate[threadIdx.x + i * NT] = stG[i];
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 16 * (i / 4) + 4 * g + i % 4 < cnt ? stV[i].f() : 0.0f;
    __syncthreads();
    if (c + 1 < nch) fetch(c + 1);
    const int64_t slot = static_cast<int64_t>(seq.slot0 + c) * a.Hv + h;
    if (a.states) {
      float* p = a.states + slot * DK * a.Dv + col;
#pragma unroll
      for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) p[static_cast<int64_t>(16 * t + 4 * g + e) * a.Dv] = S[t][e];
    }
    // K S0 and Q S0
    f4 ks[4], qs[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) ks[i] = qs[i] = f4{0, 0, 0, 0};
#pragma unroll
    for (int x = 0; x < KS; ++x) {
      Parts<3> sp;
      split_d<3>(sp, S[2 * x], S[2 * x + 1]);
#pragma unroll
      for (int i = 0; i < 4; ++i) ks[i] = mmp<3>(X::template by_row<NI>(sK, 16 * i, 32 * x, lane), sp, ks[i]);
#pragma unroll
      for (int i = 0; i < 4; ++i) qs[i] = mmp<NO>(X::template by_row<NI>(sQ, 16 * i, 32 * x, lane), sp, qs[i]);
    }
    // R = beta (V - exp(G) K S0) in place of K S0
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f4 st = *reinterpret_cast<const f4*>(&sGate[16 * i + 4 * g]);
      const f4 bt = *reinterpret_cast<const f4*>(&sGate[128 + 16 * i + 4 * g]);
#pragma unroll
      for (int e = 0; e < 4; ++e) ks[i][e] = bt[e] * fmaf(-st[e], ks[i][e], v[4 * i + e]);
    }
    // U = T R: R itself for the diagonal
    Parts<3> rp[2];
    split_d<3>(rp[0], ks[0], ks[1]);
    split_d<3>(rp[1], ks[2], ks[3]);
    f4 u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u[i] = ks[i];
#pragma unroll
      for (int x = 0; x <= i / 2; ++x) u[i] = mmp<3>(tri.t<3>(sM, i, x, lane), rp[x], u[i]);
    }
    // O = scale exp(G) Q S0 + P U
    {
      Parts<NO> up[2];
      split_d<NO>(up[0], u[0], u[1]);
      split_d<NO>(up[1], u[2], u[3]);
      T* o = static_cast<T*>(a.o) + (seq.row0 + static_cast<int64_t>(c) * kDeltaChunk) * a.Hv * a.Dv + h * a.Dv + col;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f4 st = *reinterpret_cast<const f4*>(&sGate[16 * i + 4 * g]);
        f4 y;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = a.scale * st[e] * qs[i][e];
#pragma unroll
        for (int x = 0; x <= i / 2; ++x) y = mmp<NO>(tri.p<NO>(sM, i, x, lane), up[x], y);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = 16 * i + 4 * g + e;
          if (row < cnt) o[static_cast<int64_t>(row) * a.Hv * a.Dv] = from_f32<T>(y[e]);
        }
      }
    }
    // S1 = exp(G_end) S0 + K^T (exp(G_end - G) U)
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] *= *reinterpret_cast<const f4*>(&sGate[64 + 16 * i + 4 * g]);
    split_d<3>(rp[0], u[0], u[1]);
    split_d<3>(rp[1], u[2], u[3]);
    const float last = sGate[63];
#pragma unroll
    for (int t = 0; t < DT; ++t) {
      S[t] *= last;
#pragma unroll
      for (int x = 0; x < 2; ++x) S[t] = mmp<3>(X::template by_col<NI>(sK, 32 * x, 16 * t, lane), rp[x], S[t]);
    }
    __syncthreads();
  }
  if (a.hT)
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) a.hT[state + static_cast<int64_t>(16 * t + 4 * g + e) * a.Dv] = S[t][e];
}

// ---------------------------------------------------------------------------
// One token.  A workgroup takes 64 columns of a head's state, a thread four of
// them in every sixteenth row.  With o = scale (exp(g) S^T q + (k.q) u) one
// round of sums, over S^T k, S^T q and k.q, is enough, and the state is read
// and written once: bound by HBM.
template <typename T, int DK>
__global__ __launch_bounds__(256) void k_delta_step(DeltaArgs a, float* hp) {
  constexpr int N = DK / 16;
  __shared__ f4 sk[4][16], sq[4][16];
  __shared__ float sd[4];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, c = lane & 15;
  const int nsl = a.Dv / 64;
  int n = blockIdx.x;
  const int slice = n % nsl;
  n /= nsl;
  const int h = n % a.Hv, hk = h / (a.Hv / a.Hk);
  const int64_t b = n / a.Hv;
  const int row = threadIdx.x >> 4, col = 64 * slice + 4 * c;
  float* p = hp + (b * a.Hv + h) * DK * a.Dv + static_cast<int64_t>(row) * a.Dv + col;
  const T* kp = static_cast<const T*>(a.k) + b * a.ldk + hk * DK + row;
  const T* qp = static_cast<const T*>(a.q) + b * a.ldq + hk * DK + row;
  Raw1<T> kr[N], qr[N], gr, br;
  RawVec<T, 4> vr;
  gr.load(static_cast<const T*>(a.g), b * a.ldg + h);
  br.load(static_cast<const T*>(a.beta), b * a.ldb + h);
  vr.load(static_cast<const T*>(a.v) + b * a.ldv + h * a.Dv + col);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    kr[i].load(kp, 16 * i);
    qr[i].load(qp, 16 * i);
  }
  f4 S[N];
#pragma unroll
  for (int i = 0; i < N; ++i) S[i] = ld4_state(p + static_cast<int64_t>(16 * i) * a.Dv);
  f4 ak = f4{0, 0, 0, 0}, aq = f4{0, 0, 0, 0};
  float dot = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float kv = kr[i].f(), qv = qr[i].f();
    dot = fmaf(kv, qv, dot);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      ak[e] = fmaf(S[i][e], kv, ak[e]);
      aq[e] = fmaf(S[i][e], qv, aq[e]);
    }
  }
#pragma unroll
  for (int o = 16; o < 64; o <<= 1) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      ak[e] += __shfl_xor(ak[e], o, 64);
      aq[e] += __shfl_xor(aq[e], o, 64);
    }
    dot += __shfl_xor(dot, o, 64);
  }
  if (lane < 16) {
    sk[w][c] = ak;
    sq[w][c] = aq;
    if (lane == 0) sd[w] = dot;
  }
  __syncthreads();
  ak = sk[0][c] + sk[1][c] + sk[2][c] + sk[3][c];
  const float decay = expf(gr.f()), bt = br.f();
  float v[4];
  vr.get(v);
  f4 u;
#pragma unroll
  for (int e = 0; e < 4; ++e) u[e] = bt * fmaf(-decay, ak[e], v[e]);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    f4 x;
    const float kv = kr[i].f();
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = fmaf(kv, u[e], decay * S[i][e]);
    st4_stream(p + static_cast<int64_t>(16 * i) * a.Dv, x);
  }
  if (threadIdx.x < 16) {
    aq = sq[0][c] + sq[1][c] + sq[2][c] + sq[3][c];
    dot = sd[0] + sd[1] + sd[2] + sd[3];
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = a.scale * fmaf(dot, u[e], decay * aq[e]);
    put4(static_cast<T*>(a.o) + (b * a.Hv + h) * a.Dv + col, y[0], y[1], y[2], y[3]);
  }
}

template <typename T, int DK>
hipError_t run_scan(const DeltaArgs& a, hipStream_t s) {
  k_delta_chunk<T, DK><<<static_cast<unsigned>(static_cast<int64_t>(a.nslot) * a.Hv), 256, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t heads = static_cast<int64_t>(a.B) * a.Hv;
  k_delta_chain<T, DK, 4><<<static_cast<unsigned>(heads * (a.Dv / 64)), 256, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t run_step(const DeltaArgs& a, float* h, hipStream_t s) {
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(a.B) * a.Hv * (a.Dv / 64));
  if (a.Dk == 64) k_delta_step<T, 64><<<grid, 256, 0, s>>>(a, h);
  else k_delta_step<T, 128><<<grid, 256, 0, s>>>(a, h);
  return hipGetLastError();
}

}  // namespace

bool delta_supported(int Dk, int Dv) { return (Dk == 64 || Dk == 128) && (Dv == 64 || Dv == 128); }

int64_t delta_slots(int B, int T, bool packed) {
  if (packed) return static_cast<int64_t>(T) / kDeltaChunk + B;
  return static_cast<int64_t>(B) * ((T + kDeltaChunk - 1) / kDeltaChunk);
}

size_t delta_workspace_bytes(int B, int T, int Hv, int, int, bool packed) {
  return sizeof(float) * (4096 + 192) * static_cast<size_t>(delta_slots(B, T, packed)) * Hv;
}

void delta_carve(DeltaArgs& a, void* ws) {
  a.nslot = static_cast<int>(delta_slots(a.B, a.T, a.cu != nullptr));
  a.pm = static_cast<float*>(ws);
  a.gates = a.pm + static_cast<size_t>(4096) * a.nslot * a.Hv;
}

hipError_t launch_delta_scan(DeltaArgs& a, int bf16, hipStream_t s) {
  if (bf16) return a.Dk == 64 ? run_scan<bf16_t, 64>(a, s) : run_scan<bf16_t, 128>(a, s);
  return a.Dk == 64 ? run_scan<float, 64>(a, s) : run_scan<float, 128>(a, s);
}

hipError_t launch_delta_step(const DeltaArgs& a, float* h, int bf16, hipStream_t s) {
  return bf16 ? run_step<bf16_t>(a, h, s) : run_step<float>(a, h, s);
}

}  // namespace m3
