// qk_norm.hip -- RMS norms of queries and keys per head with the position
// rotation in the same pass, and the gradients (gfx950).
//
//   u = v / sqrt(mean v^2 + eps),  z = w u,  out = z with its pairs turned by
//   the angle pos * base^(-2j / rot)
//
// One pass reads and writes each element once and is bound by HBM.  A row
// (one head of one token) is spread over D / 8 lanes with four pairs each, so
// both members of a pair are in one lane for either pairing and the sum of
// squares needs log2(D / 8) lane steps.  A wave keeps its token's cosines and
// sines in registers for all the heads it handles; they cost one fp64 product
// and one hardware sine and cosine per pair and token.  Positions are int32:
// the product pos * freq is formed in turns in fp64 and reduced there, so
// that far positions lose no phase.
#include "m3_device.h"
#include "qk_norm.h"

namespace m3 {
namespace {

// Which elements of a row a lane's four pairs j = 4 l .. 4 l + 3 are.
//   kAdj:    (2j, 2j+1): eight consecutive elements
//   kHalf4:  (j, j + n) below n = rot / 2, n a multiple of 4: twice four
//            consecutive elements, or eight where nothing is rotated
//   kAny:    (j, j + n) for any n: element by element
enum { kAdj = 0, kHalf4 = 1, kAny = 2 };

template <typename T, int MODE>
struct RowIO {
  int n, j0;   // rotated pairs, the lane's first pair
  __device__ __forceinline__ RowIO(int l, int n_) : n(n_), j0(4 * l) {}
  __device__ __forceinline__ int first(int s) const {
    const int j = j0 + s;
    return MODE != kAdj && j < n ? j : 2 * j;
  }
  __device__ __forceinline__ int second(int s) const {
    const int j = j0 + s;
    return MODE != kAdj && j < n ? j + n : 2 * j + 1;
  }
  // A lane's pairs as loaded: eight consecutive elements, or twice four (kAny:
  // the members one by one), turned into floats only where they are used.
  struct Raw {
    RawVec<T, MODE == kAdj ? 8 : 4> lo, hi;   // kAdj: lo alone
    float a[MODE == kAny ? 4 : 1], b[MODE == kAny ? 4 : 1];
  };
  __device__ __forceinline__ void load(Raw& r, const T* p) const {
    if constexpr (MODE == kAny) {
#pragma unroll
      for (int s = 0; s < 4; ++s) { r.a[s] = to_f32(p[first(s)]); r.b[s] = to_f32(p[second(s)]); }
    } else if constexpr (MODE == kAdj) {
      r.lo.load(p + 2 * j0);
    } else {
      const bool split = j0 < n;
      r.lo.load(p + (split ? j0 : 2 * j0));
      r.hi.load(p + (split ? j0 + n : 2 * j0 + 4));
    }
  }
  // a[s], b[s]: the members of pair s
  __device__ __forceinline__ void get(const Raw& r, float* a, float* b) const {
    if constexpr (MODE == kAny) {
#pragma unroll
      for (int s = 0; s < 4; ++s) { a[s] = r.a[s]; b[s] = r.b[s]; }
    } else if constexpr (MODE == kAdj) {
      float x[8];
      r.lo.get(x);
#pragma unroll
      for (int s = 0; s < 4; ++s) { a[s] = x[2 * s]; b[s] = x[2 * s + 1]; }
    } else {
      float x[4], y[4];
      r.lo.get(x);
      r.hi.get(y);
      const bool split = j0 < n;
      a[0] = x[0];
      a[1] = split ? x[1] : x[2];
      a[2] = split ? x[2] : y[0];
      a[3] = split ? x[3] : y[2];
      b[0] = split ? y[0] : x[1];
      b[1] = split ? y[1] : x[3];
      b[2] = split ? y[2] : y[1];
      b[3] = y[3];
    }
  }
  static __device__ __forceinline__ uint32_t pack(float x, float y) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{x, y}, bh2));
  }
  static __device__ __forceinline__ void st4(float* p, f4 v) { *reinterpret_cast<f4*>(p) = v; }
  static __device__ __forceinline__ void st4(bf16_t* p, f4 v) {
    *reinterpret_cast<uint2*>(p) = uint2{pack(v.x, v.y), pack(v.z, v.w)};
  }
  static __device__ __forceinline__ void st8(float* p, const float* v) {
    st4(p, f4{v[0], v[1], v[2], v[3]});
    st4(p + 4, f4{v[4], v[5], v[6], v[7]});
  }
  static __device__ __forceinline__ void st8(bf16_t* p, const float* v) {
    *reinterpret_cast<uint4*>(p) =
        uint4{pack(v[0], v[1]), pack(v[2], v[3]), pack(v[4], v[5]), pack(v[6], v[7])};
  }
  __device__ __forceinline__ void store(T* p, const float* a, const float* b) const {
    if (MODE == kAdj || (MODE == kHalf4 && j0 >= n)) {
      float v[8];
#pragma unroll
      for (int s = 0; s < 4; ++s) { v[2 * s] = a[s]; v[2 * s + 1] = b[s]; }
      st8(p + 2 * j0, v);
    } else if (MODE == kHalf4) {
      st4(p + j0, f4{a[0], a[1], a[2], a[3]});
      st4(p + j0 + n, f4{b[0], b[1], b[2], b[3]});
    } else {
#pragma unroll
      for (int s = 0; s < 4; ++s) { p[first(s)] = from_f32<T>(a[s]); p[second(s)] = from_f32<T>(b[s]); }
    }
  }
};

// cos and sin of the lane's four pairs at position p (1 and 0 past rot / 2)
__device__ __forceinline__ void turns(const double* f, int p, float* c, float* s) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const double t = f[j] * static_cast<double>(p);
    const float r = static_cast<float>(t - __builtin_rint(t));
    c[j] = __builtin_amdgcn_cosf(r);
    s[j] = __builtin_amdgcn_sinf(r);
  }
}

// One tensor's rows g * ROWS + (lane group), g0 <= g < g1, of one token.
// U groups' rows are on their way together; groups past the last head repeat
// it without storing.
template <typename T, int D, int MODE, bool BWD>
struct Heads {
  static constexpr int G = D / 8, ROWS = 64 / G, U = BWD ? 2 : 4;
  using IO = RowIO<T, MODE>;
  static __device__ __forceinline__ void run(const IO& io, int grp, int g0, int g1, int H,
                                             const T* in, const T* gin, T* out, const float* w,
                                             const float* c, const float* sn, float eps,
                                             float* acc) {
    for (int gb = g0; gb < g1; gb += U) {
      typename IO::Raw rv[U], rg[BWD ? U : 1];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (gb + u >= g1) continue;
        const int h = min((gb + u) * ROWS + grp, H - 1);
        io.load(rv[u], in + h * D);
        if constexpr (BWD) io.load(rg[u], gin + h * D);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (gb + u >= g1) continue;
        const int h = (gb + u) * ROWS + grp;
        const bool on = h < H;
        float x[4], y[4];
        io.get(rv[u], x, y);
        float ss = 0.0f;
#pragma unroll
        for (int s = 0; s < 4; ++s) ss = fmaf(x[s], x[s], fmaf(y[s], y[s], ss));
        ss = group_sum<G>(ss);
        const float inv = __builtin_amdgcn_rsqf(fmaf(ss, 1.0f / D, eps));   // 1 ulp
        if constexpr (!BWD) {
          float ox[4], oy[4];
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            const float zx = x[s] * inv * w[s], zy = y[s] * inv * w[4 + s];
            ox[s] = fmaf(zx, c[s], -zy * sn[s]);
            oy[s] = fmaf(zx, sn[s], zy * c[s]);
          }
          if (on) io.store(out + h * D, ox, oy);
        } else {
          float gx[4], gy[4];
          io.get(rg[u], gx, gy);
          float dot = 0.0f, px[4], py[4];
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            const float ux = x[s] * inv, uy = y[s] * inv;
            const float rx = fmaf(gx[s], c[s], gy[s] * sn[s]);
            const float ry = fmaf(gy[s], c[s], -gx[s] * sn[s]);
            if (on) {
              acc[s] = fmaf(rx, ux, acc[s]);
              acc[4 + s] = fmaf(ry, uy, acc[4 + s]);
            }
            px[s] = rx * w[s];
            py[s] = ry * w[4 + s];
            dot = fmaf(px[s], ux, fmaf(py[s], uy, dot));
            x[s] = ux;
            y[s] = uy;
          }
          dot = group_sum<G>(dot) * (1.0f / D);
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            px[s] = inv * fmaf(-x[s], dot, px[s]);
            py[s] = inv * fmaf(-y[s], dot, py[s]);
          }
          if (on) io.store(out + h * D, px, py);
        }
      }
    }
  }
};

// A wave takes tokens, and of each the part blockIdx.y of the groups of heads
// (q's first, then k's).
template <typename T, int D, int MODE, bool BWD>
__global__ __launch_bounds__(256) void k_qk_norm(QkNormArgs a) {
  using K = Heads<T, D, MODE, BWD>;
  constexpr int G = K::G, ROWS = K::ROWS;
  const int lane = threadIdx.x & 63, l = lane % G, grp = lane / G;
  const int n = a.rot / 2;
  const typename K::IO io(l, n);
  float wq[8], wk[8];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    wq[s] = ld_or(a.wq, io.first(s), 1.0f);
    wq[4 + s] = ld_or(a.wq, io.second(s), 1.0f);
    wk[s] = ld_or(a.wk, io.first(s), 1.0f);
    wk[4 + s] = ld_or(a.wk, io.second(s), 1.0f);
  }
  double f[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) f[s] = 4 * l + s < n ? a.freq[4 * l + s] : 0.0;
  float accq[8], acck[8];
  if (BWD)
#pragma unroll
    for (int s = 0; s < 8; ++s) accq[s] = acck[s] = 0.0f;

  const int nq = (a.Hq + ROWS - 1) / ROWS, nk = (a.Hk + ROWS - 1) / ROWS;
  const int per = (nq + nk + a.split - 1) / a.split;
  const int g0 = static_cast<int>(blockIdx.y) * per, g1 = min(g0 + per, nq + nk);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int tt = blockIdx.x * 4 + wave; tt < a.T; tt += gridDim.x * 4) {
    const int64_t t = tt;
    float c[4], sn[4];
    turns(f, a.pos[t], c, sn);
    const int64_t oq = t * a.Hq * D, ok = t * a.Hk * D;
    K::run(io, grp, g0, min(g1, nq), a.Hq, static_cast<const T*>(a.q) + t * a.ldq,
           static_cast<const T*>(a.gq) + oq,
           BWD ? static_cast<T*>(a.dq) + t * a.ld_dq : static_cast<T*>(a.qo) + oq, wq, c, sn, a.eps, accq);
    K::run(io, grp, max(g0 - nq, 0), g1 - nq, a.Hk, static_cast<const T*>(a.k) + t * a.ldk,
           static_cast<const T*>(a.gk) + ok,
           BWD ? static_cast<T*>(a.dk) + t * a.ld_dk : static_cast<T*>(a.ko) + ok, wk, c, sn, a.eps, acck);
  }
  if constexpr (BWD) {
    // sums over the lane groups and the four waves, in a fixed order
    __shared__ float red[4][2][ROWS][D];
    const int w = threadIdx.x >> 6;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      red[w][0][grp][io.first(s)] = accq[s];
      red[w][0][grp][io.second(s)] = accq[4 + s];
      red[w][1][grp][io.first(s)] = acck[s];
      red[w][1][grp][io.second(s)] = acck[4 + s];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * D; e += 256) {
      float v = 0.0f;
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int r = 0; r < ROWS; ++r) v += red[q][e / D][r][e % D];
      a.part[(static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * 2 * D + e] = v;
    }
  }
}

// dw = the sum of the blocks' parts, in a fixed order: 64 threads of a channel
// take every 64th part each (four in flight) and are joined in LDS.
__global__ __launch_bounds__(1024) void k_qk_norm_dw(QkNormArgs a, int nblocks) {
  __shared__ float sum[64][17];
  const int cl = threadIdx.x & 15, k = threadIdx.x >> 4;
  const int e = blockIdx.x * 16 + cl;   // of 2 D
  float acc = 0.0f;
#pragma unroll 4
  for (int p = k; p < nblocks; p += 64) acc += a.part[static_cast<int64_t>(p) * 2 * a.D + e];
  sum[k][cl] = acc;
  __syncthreads();
  if (k == 0) {
    float v = 0.0f;
#pragma unroll
    for (int j = 0; j < 64; ++j) v += sum[j][cl];
    float* o = e < a.D ? a.dwq : a.dwk;
    if (o) o[e < a.D ? e : e - a.D] = v;
  }
}

// Workgroups of four waves: as many as are resident together, so that a wave
// reads the weights once for several tokens (16384 tokens of 18 heads of 128:
// 31 us; with one token a wave, 4096 workgroups, 42 us).  The gradients' grid
// also sets how many parts the weights' sums have (the same tokens: 42 us, 5.4
// TB/s, and 5 for the sums).
constexpr int kFwdBlocks = 2048, kBwdBlocks = 1024;

// Waves that share a token's heads: enough of them for every SIMD of the chip
// where tokens are few, one wave for all heads of a token (one set of cosines)
// where not.
int split_of(int T, int Hq, int Hk, int D) {
  const int rows = 64 / (D / 8);
  const int most = (Hq + rows - 1) / rows + (Hk + rows - 1) / rows;
  int s = (4096 + T - 1) / T;
  if (s > most) s = most;
  return s > 512 ? 512 : s;
}
dim3 grid_of(int T, int split, int most) {
  const int n = (T + 3) / 4, m = most / split;
  return dim3(static_cast<unsigned>(n < m ? n : m), static_cast<unsigned>(split));
}

template <typename T, int D, bool BWD>
void run_dim(const QkNormArgs& a, dim3 grid, hipStream_t s) {
  const int n = a.rot / 2;
  if (!a.half)
    k_qk_norm<T, D, kAdj, BWD><<<grid, 256, 0, s>>>(a);
  else if (n % 4 == 0)
    k_qk_norm<T, D, kHalf4, BWD><<<grid, 256, 0, s>>>(a);
  else
    k_qk_norm<T, D, kAny, BWD><<<grid, 256, 0, s>>>(a);
}
template <typename T, bool BWD>
void run_type(const QkNormArgs& a, dim3 grid, hipStream_t s) {
  switch (a.D) {
    case 32: run_dim<T, 32, BWD>(a, grid, s); break;
    case 64: run_dim<T, 64, BWD>(a, grid, s); break;
    case 128: run_dim<T, 128, BWD>(a, grid, s); break;
    case 256: run_dim<T, 256, BWD>(a, grid, s); break;
  }
}

}  // namespace

bool qk_norm_supported(int D) { return D == 32 || D == 64 || D == 128 || D == 256; }

size_t qk_norm_workspace_bytes(int T, int Hq, int Hk, int D) {
  const dim3 g = grid_of(T, split_of(T, Hq, Hk, D), kBwdBlocks);
  return sizeof(float) * 2 * D * g.x * g.y;
}

hipError_t launch_qk_norm(QkNormArgs& a, int bf16, hipStream_t s) {
  a.split = split_of(a.T, a.Hq, a.Hk, a.D);
  const dim3 grid = grid_of(a.T, a.split, kFwdBlocks);
  if (bf16) run_type<bf16_t, false>(a, grid, s);
  else run_type<float, false>(a, grid, s);
  return hipGetLastError();
}

hipError_t launch_qk_norm_backward(QkNormArgs& a, int bf16, hipStream_t s) {
  a.split = split_of(a.T, a.Hq, a.Hk, a.D);
  const dim3 grid = grid_of(a.T, a.split, kBwdBlocks);
  if (bf16) run_type<bf16_t, true>(a, grid, s);
  else run_type<float, true>(a, grid, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.dwq || a.dwk) {
    k_qk_norm_dw<<<2 * a.D / 16, 1024, 0, s>>>(a, static_cast<int>(grid.x * grid.y));
    e = hipGetLastError();
  }
  return e;
}

}  // namespace m3
