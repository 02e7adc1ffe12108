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
// walks each sequence's chunks with the state in registers, in segments where
// sequences are few and long.
//
// 64 tokens a chunk: half of them would double the states that a training step
// keeps and the steps of the chain, each with the same latency; twice as many, the
// work of T and P, which is quadratic, and the LDS for it.
#include "delta_chain.h"

namespace m3 {
namespace {

// ---------------------------------------------------------------------------
// T, P and the gates of a chunk of one head.  The products K K^T and Q K^T are
// formed tile by tile, wave w those of rows 16 w ..; T by blocks of 16 in fp32:
// the diagonal's by substitution, a column a lane, then, diagonal by diagonal,
//   T_IJ = -T_II sum_{J <= K < I} A_IK T_KJ.
// Differences of G are taken in fp64, as G may be large where its differences
// are small.  256 chunks of 16 heads of 128, bf16: 56 us for 204 MB, 3.6 TB/s, of
// the 4.9 that a copy reaches: four workgroups a CU, whose barriers wait for loads
// and for the substitution.
template <typename T, int DK>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 4 : 2) void k_delta_chunk(DeltaArgs a) {
  using X = Rows64<DK, true>;
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
  const typename X::Lane xl(lane);
  Stage<T, DK, 256, true> stage;
  stage.load(static_cast<const T*>(a.k) + sl.row0 * a.ldk + hk * DK, a.ldk, sl.n);
  Stage<T, DK, 256, true> stage_q;
  stage_q.load(static_cast<const T*>(a.q) + sl.row0 * a.ldq + hk * DK, a.ldq, sl.n);
  if (w == 0) {
    const int64_t row = sl.row0 + min(lane, sl.n - 1);
    float gt = ld1(static_cast<const T*>(a.g), row * a.ldg + h);
    float bt = ld1(static_cast<const T*>(a.beta), row * a.ldb + h);
    if (lane >= sl.n) gt = bt = 0.0f;
    gt = gt < -128.0f ? -128.0f : gt;   // exp is 0 there, and -inf has no differences
    double G = gt * 1.4426950408889634;   // powers of 2 from here on
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const double o = __shfl_up(G, d, 64);
      if (lane >= d) G += o;
    }
    sG[lane] = G;
    sB[lane] = bt;
    const double end = __shfl(G, 63, 64);
    float* p = a.pm + (static_cast<int64_t>(slot) * a.Hv + h) * a.ldpm + kDeltaMatrix + lane;
    p[0] = __builtin_amdgcn_exp2f(static_cast<float>(G));
    p[64] = __builtin_amdgcn_exp2f(static_cast<float>(end - G));
    p[128] = bt;
    const float hi = static_cast<float>(G);
    p[192] = hi;
    p[256] = static_cast<float>(G - hi);
  }
  stage.store(sK);
  stage_q.store(sQ);
  __syncthreads();

  f4 kk[4], qk[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) kk[j] = qk[j] = f4{0, 0, 0, 0};
#pragma unroll
  for (int x = 0; x < DK / 32; ++x) {
    const Parts<NI> ka = X::template by_row<NI>(sK, xl, w, x);
    const Parts<NI> qa = X::template by_row<NI>(sQ, xl, w, x);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j <= w) {
        const Parts<NI> kb = X::template by_row<NI>(sK, xl, j, x);
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
        const float d = in ? __builtin_amdgcn_exp2f(static_cast<float>(sG[i] - Gj)) : 0.0f;
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
      float s[4] = {i == r ? 1.0f : 0.0f, 0.0f, 0.0f, 0.0f};   // (four sums, not to wait for each term)
#pragma unroll
      for (int j = 0; j < i; ++j) s[j & 3] = fmaf(-sA[16 * w + i][16 * w + j], x[j], s[j & 3]);
      x[i] = (s[0] + s[1]) + (s[2] + s[3]);
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
  float* out = a.pm + (static_cast<int64_t>(slot) * a.Hv + h) * a.ldpm;
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const int x = threadIdx.x + 256 * n;
    *reinterpret_cast<f4*>(out + 4 * x) = *reinterpret_cast<const f4*>(&sM[x / 16][x % 16 * 4]);
  }
}

// ---------------------------------------------------------------------------
// The chain (delta_chain.h)
template <typename T, int DK, int NW, int NBUF>
__global__ __launch_bounds__(64 * NW, sizeof(T) == 2 ? 2 : 1) void k_delta_chain(DeltaArgs a) {
  __shared__ __align__(16) char smem[NBUF * ChainTiles<T, DK, 64 * NW, true>::BUF];
  const int nsl = a.Dv / (16 * NW), n = blockIdx.x / nsl;
  const DeltaSeg seg(a, n / a.Hv, threadIdx.x & 63);
  if (seg.s >= 0) chain<T, DK, NW, NBUF, kFull>(a, seg, n % a.Hv, blockIdx.x % nsl, smem);
}

// E and F of all segments but the last, F of none before the second
template <typename T, int DK, int NW, int NBUF>
__global__ __launch_bounds__(64 * NW, sizeof(T) == 2 ? 2 : 1) void k_delta_segments(DeltaArgs a) {
  __shared__ __align__(16) char smem[NBUF * ChainTiles<T, DK, 64 * NW, false>::BUF];
  const int nv = a.Dv / (16 * NW), nsl = nv + DK / (16 * NW);
  const int n = blockIdx.x / nsl, slice = blockIdx.x % nsl;
  const DeltaSeg seg(a, n / a.Hv, threadIdx.x & 63, false);
  if (seg.s < 0) return;
  if (slice < nv) chain<T, DK, NW, NBUF, kEnds>(a, seg, n % a.Hv, slice, smem);
  else if (seg.j > 0) chain<T, DK, NW, NBUF, kMaps>(a, seg, n % a.Hv, slice - nv, smem);
}

// ---------------------------------------------------------------------------
// One token.  A workgroup takes 64 columns of a head's state, a thread four of
// them in every sixteenth row.  With o = scale (exp(g) S^T q + (k.q) u) one
// round of sums, over S^T k, S^T q and k.q, is enough, and the state is read
// and written once: bound by HBM.  128 sequences of 64 heads of 128 x 64: 90 us
// for 546 MB, 6.1 TB/s (the state's writes do not wait for HBM); a single sequence
// is bound by the launch.
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

template <typename T, int DK, int NW>
hipError_t run_chain(const DeltaArgs& a, bool split, hipStream_t s) {
  constexpr int NBUF = sizeof(T) == 2 && NW == 8 ? 2 : 1;
  const int64_t heads = static_cast<int64_t>(a.nseg) * a.Hv;
  if (split) {
    k_delta_segments<T, DK, NW, NBUF>
        <<<static_cast<unsigned>(static_cast<int64_t>(a.inner) * a.Hv * ((a.Dv + DK) / (16 * NW))), 64 * NW, 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    k_delta_join<DK, false>
        <<<static_cast<unsigned>(static_cast<int64_t>(a.B < a.inner ? a.B : a.inner) * a.Hv * (a.Dv / 16)), 2 * DK, 0, s>>>(a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  k_delta_chain<T, DK, NW, NBUF><<<static_cast<unsigned>(heads * (a.Dv / (16 * NW))), 64 * NW, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T, int DK>
hipError_t run_chunks(const DeltaArgs& a, hipStream_t s) {
  k_delta_chunk<T, DK><<<static_cast<unsigned>(static_cast<int64_t>(a.nslot) * a.Hv), 256, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T, int DK>
hipError_t run_scan(const DeltaArgs& a, bool split, hipStream_t s) {
  const hipError_t e = run_chunks<T, DK>(a, s);
  if (e != hipSuccess) return e;
  if constexpr (DK == 128 && sizeof(T) == 2)
    if (a.Dv == 128) return run_chain<T, DK, 8>(a, split, s);
  return run_chain<T, DK, 4>(a, split, s);
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

// The chain takes about the same time for a chunk whether a SIMD has one wave or
// two (6 us; half the waves' instructions wait for another's), so in such units
// it costs a sequence's chunks, times the waves beyond 2048.  The length of the
// longest of a packed batch is not known here; twice the mean is what uniform
// lengths give.  Segments cost their chunks twice, without outputs 3/4, for as
// many columns as the values and a state have together, and what joins them
// 0.2 for each.  They are taken where that is less than 3/4 (in a training step
// both are held by memory before that).  16384 tokens of 16 heads of 128: 1.43 ms
// whole, in 32 segments of 8 chunks 381 us with the rest, 16 of 16 333, 8 of 32
// 382.  What the estimate costs: 16 sequences of 1024 rows, 8 heads of 64 x 64 in
// fp32, are cut and take 172 us, whole 125; 24, the longest of 14000 of 16300, 16
// heads of 128, 401, whole 1257.
//
// A packed batch that would stay whole may still have one sequence that is much
// longer than the others: then segments no shorter than what uniform lengths give,
// so that those have one each and only such a sequence has more.  (60 sequences of
// 64 tokens and one of 4000, 8 heads of 128 x 64: 123 us instead of 272, with
// gradients 322 instead of 655.  64 of 128, 32 heads: 149 and 145, 526 and 505;
// 1000 of 16, 16 heads of 128: 803 and 791, 2721 and 2691.)
DeltaPlan delta_plan(int B, int T, int Hv, int Dk, int Dv, bool packed, bool back) {
  const double rows = packed ? T : static_cast<double>(B) * T;
  const double longest = (packed && B > 1 ? 2.0 * T / B : T) / kDeltaChunk, cols = Hv * (Dv / 16.0);
  auto rounds = [](double waves) { return waves > 2048 ? waves / 2048 : 1.0; };
  DeltaPlan p{30, B, false, 0};
  double best = 0.75 * longest * rounds(B * cols);
  for (int l = 3; l < 10 && longest / (1 << l) >= 2; ++l) {
    const double n = rows / (kDeltaChunk << l) + (packed ? B : 0);
    const double cost = (1 << l) * ((back ? 1.0 : 0.75) * rounds(n * cols * (1.0 + static_cast<double>(Dk) / Dv)) + rounds(n * cols)) +
                        0.2 * longest / (1 << l);
    if (cost < best) {
      best = cost;
      p = DeltaPlan{l, 0, true, 0};
    }
  }
  if (!p.split && packed && B > 1) {
    const DeltaPlan one = delta_plan(1, T, Hv, Dk, Dv, false, back);
    int l = one.lseg;
    while (one.split && l < 30 && static_cast<double>(1 << l) < longest) ++l;
    if (one.split && (static_cast<int64_t>(T) >> (6 + l)) >= 4) p = DeltaPlan{l, 0, true, 0};
  }
  if (p.split) {
    p.nseg = packed ? (static_cast<int64_t>(T) >> (6 + p.lseg)) + B
                    : B * ((static_cast<int64_t>(T) + (kDeltaChunk << p.lseg) - 1) / (kDeltaChunk << p.lseg));
    p.inner = p.nseg - B;
  }
  return p;
}

// A state, a map and a decay of each segment that may not be its sequence's last,
// and in the scan the states before sequences of several.
size_t delta_segment_bytes(const DeltaPlan& p, int B, int Hv, int Dk, int Dv, bool back) {
  const size_t inner = p.inner, firsts = back ? 0 : B < p.inner ? B : p.inner, state = static_cast<size_t>(Dk) * Dv;
  return Hv * (sizeof(float) * (state * (inner + firsts) + inner) + 3 * sizeof(uint16_t) * Dk * Dk * inner);
}

void delta_carve_segments(DeltaArgs& a, const DeltaPlan& p, void* ws, bool back) {
  a.lseg = p.lseg;
  a.nseg = static_cast<int>(p.nseg);
  a.nslot = static_cast<int>(delta_slots(a.B, a.T, a.cu != nullptr));
  a.inner = static_cast<int>(p.inner);
  const size_t heads = static_cast<size_t>(a.inner) * a.Hv;
  a.ends = static_cast<float*>(ws);
  a.maps = reinterpret_cast<uint16_t*>(a.ends + a.Dk * a.Dv * heads);
  a.firsts = reinterpret_cast<float*>(a.maps + 3 * a.Dk * a.Dk * heads);   // (backward: none)
  a.decays = a.firsts + static_cast<size_t>(a.Dk) * a.Dv * (back ? 0 : a.B < a.inner ? a.B : a.inner) * a.Hv;
}

size_t delta_workspace_bytes(int B, int T, int Hv, int Dk, int Dv, bool packed) {
  const size_t chunks = static_cast<size_t>(kDeltaMatrix + kDeltaGates) * delta_slots(B, T, packed) * Hv;
  return sizeof(float) * chunks + delta_segment_bytes(delta_plan(B, T, Hv, Dk, Dv, packed, false), B, Hv, Dk, Dv, false);
}

void delta_carve(DeltaArgs& a, void* ws) {
  a.pm = static_cast<float*>(ws);
  a.ldpm = kDeltaMatrix + kDeltaGates;
  delta_carve_segments(a, delta_plan(a.B, a.T, a.Hv, a.Dk, a.Dv, a.cu != nullptr, false),
                       a.pm + static_cast<size_t>(a.ldpm) * delta_slots(a.B, a.T, a.cu != nullptr) * a.Hv, false);
  if (a.states) {
    a.ldpm = delta_state_floats(a.Dk, a.Dv);
    a.pm = a.states + static_cast<size_t>(a.Dk + kDeltaChunk) * a.Dv;
  }
}

hipError_t launch_delta_scan(DeltaArgs& a, int bf16, hipStream_t s) {
  const bool split = a.lseg < 30;
  if (bf16) return a.Dk == 64 ? run_scan<bf16_t, 64>(a, split, s) : run_scan<bf16_t, 128>(a, split, s);
  return a.Dk == 64 ? run_scan<float, 64>(a, split, s) : run_scan<float, 128>(a, split, s);
}

hipError_t launch_delta_step(const DeltaArgs& a, float* h, int bf16, hipStream_t s) {
  return bf16 ? run_step<bf16_t>(a, h, s) : run_step<float>(a, h, s);
}

}  // namespace m3
