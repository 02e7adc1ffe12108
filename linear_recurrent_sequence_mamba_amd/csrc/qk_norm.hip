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
  int e0, n, j0;   // first pair, rotated pairs
  __device__ __forceinline__ RowIO(int l, int n_) : e0(0), n(n_), j0(4 * l) {}
  __device__ __forceinline__ int first(int s) const {
    const int j = j0 + s;
    return MODE != kAdj && j < n ? j : 2 * j;
  }
  __device__ __forceinline__ int second(int s) const {
    const int j = j0 + s;
    return MODE != kAdj && j < n ? j + n : 2 * j + 1;
  }
  // a[s], b[s]: the members of pair s
  __device__ __forceinline__ void load(const T* p, float* a, float* b) const {
    if (MODE == kAdj || (MODE == kHalf4 && j0 >= n)) {
      float v[8];
      ld8(p, 2 * j0, v);
#pragma unroll
      for (int s = 0; s < 4; ++s) { a[s] = v[2 * s]; b[s] = v[2 * s + 1]; }
    } else if (MODE == kHalf4) {
      const f4 x = ld4(p, j0), y = ld4(p, j0 + n);
#pragma unroll
      for (int s = 0; s < 4; ++s) { a[s] = x[s]; b[s] = y[s]; }
    } else {
#pragma unroll
      for (int s = 0; s < 4; ++s) { a[s] = to_f32(p[first(s)]); b[s] = to_f32(p[second(s)]); }
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

// A wave takes a token and the part blockIdx.y of its heads; its lane groups
// take rows h = group, group + 64 / G, ... of the part.
template <typename T, int D, int MODE, bool BWD>
__global__ __launch_bounds__(256) void k_qk_norm(QkNormArgs a) {
  constexpr int G = D / 8, ROWS = 64 / G;
  const int lane = threadIdx.x & 63, l = lane % G, grp = lane / G;
  const int n = a.rot / 2;
  const RowIO<T, MODE> io(l, n);
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

  const int H = a.Hq + a.Hk;
  const int per = (H + a.split - 1) / a.split;
  const int h0 = static_cast<int>(blockIdx.y) * per, h1 = min(h0 + per, H);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int tt = blockIdx.x * 4 + wave; tt < a.T; tt += gridDim.x * 4) {
    const int64_t t = tt;
    float c[4], sn[4];
    turns(f, a.pos[t], c, sn);
    for (int hb = h0; hb < h1; hb += ROWS) {
      const int hr = hb + grp;
      const bool on = hr < h1;
      const int h = on ? hr : h1 - 1;   // idle groups repeat the last row
      const bool isq = h < a.Hq;
      const int hh = isq ? h : h - a.Hq;
      const T* p = isq ? static_cast<const T*>(a.q) + t * a.ldq : static_cast<const T*>(a.k) + t * a.ldk;
      float x[4], y[4];
      io.load(p + hh * D, x, y);
      float ss = 0.0f;
#pragma unroll
      for (int s = 0; s < 4; ++s) ss = fmaf(x[s], x[s], fmaf(y[s], y[s], ss));
      ss = group_sum<G>(ss);
      const float inv = __builtin_amdgcn_rsqf(fmaf(ss, 1.0f / D, a.eps));   // 1 ulp
      const int64_t ro = (t * (isq ? a.Hq : a.Hk) + hh) * D;
      if constexpr (!BWD) {
        float ox[4], oy[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const float zx = x[s] * inv * (isq ? wq[s] : wk[s]);
          const float zy = y[s] * inv * (isq ? wq[4 + s] : wk[4 + s]);
          ox[s] = fmaf(zx, c[s], -zy * sn[s]);
          oy[s] = fmaf(zx, sn[s], zy * c[s]);
        }
        if (on) io.store((isq ? static_cast<T*>(a.qo) : static_cast<T*>(a.ko)) + ro, ox, oy);
      } else {
        float gx[4], gy[4];
        io.load((isq ? static_cast<const T*>(a.gq) : static_cast<const T*>(a.gk)) + ro, gx, gy);
        float dot = 0.0f, px[4], py[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const float ux = x[s] * inv, uy = y[s] * inv;
          const float rx = fmaf(gx[s], c[s], gy[s] * sn[s]);
          const float ry = fmaf(gy[s], c[s], -gx[s] * sn[s]);
          if (on && isq) {
            accq[s] = fmaf(rx, ux, accq[s]);
            accq[4 + s] = fmaf(ry, uy, accq[4 + s]);
          }
          if (on && !isq) {
            acck[s] = fmaf(rx, ux, acck[s]);
            acck[4 + s] = fmaf(ry, uy, acck[4 + s]);
          }
          px[s] = rx * (isq ? wq[s] : wk[s]);
          py[s] = ry * (isq ? wq[4 + s] : wk[4 + s]);
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
        T* o = isq ? static_cast<T*>(a.dq) + t * a.ld_dq : static_cast<T*>(a.dk) + t * a.ld_dk;
        if (on) io.store(o + hh * D, px, py);
      }
    }
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

constexpr int kFwdBlocks = 4096, kBwdBlocks = 1024;

// waves per token: enough units for every SIMD of the chip where tokens are
// few, one wave for all heads of a token (one set of cosines) where not
int split_of(int T, int H, int D) {
  const int rows = 64 / (D / 8);
  const int most = (H + rows - 1) / rows;
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
  const dim3 g = grid_of(T, split_of(T, Hq + Hk, D), kBwdBlocks);
  return sizeof(float) * 2 * D * g.x * g.y;
}

hipError_t launch_qk_norm(QkNormArgs& a, int bf16, hipStream_t s) {
  a.split = split_of(a.T, a.Hq + a.Hk, a.D);
  const dim3 grid = grid_of(a.T, a.split, kFwdBlocks);
  if (bf16) run_type<bf16_t, false>(a, grid, s);
  else run_type<float, false>(a, grid, s);
  return hipGetLastError();
}

hipError_t launch_qk_norm_backward(QkNormArgs& a, int bf16, hipStream_t s) {
  a.split = split_of(a.T, a.Hq + a.Hk, a.D);
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
