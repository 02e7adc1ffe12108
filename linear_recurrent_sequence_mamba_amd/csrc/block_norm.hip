// block_norm.hip -- the norms before and after a block, fused with its gate
// and residual scale (gfx950), and the gradients.
//
//   z = y / sqrt(mean y^2 + eps) * wy      (raw: y * wy)
//   h = x + scale act(gate) z,             n = h / sqrt(mean h^2 + eps) * wn
//
// One pass: each row is read and written once and everything between stays in
// registers, so the call is bound by HBM.  A workgroup takes a row at a time,
// eight elements a thread, and keeps the weights in registers over its rows
// (from L2 they would be more bytes than the row); the next row is on its way
// meanwhile.  The sums meet in LDS, one barrier each.
//
// Gradients, with u = y / rms(y), m = h / rms(h), gm = dn wn and
// gu = dH scale act(gate) wy:
//   dH = dh + (gm - m mean(gm m)) / rms(h) = dx
//   dy = (gu - u mean(gu u)) / rms(y)      (raw: gu)
//   dgate = dH scale z act'(gate),  dwn = sum dn m,
//   dwy = scale P, dscale = wy P, where P = sum dH act(gate) u
// u and h are formed again from the inputs, in fp32.  Three sums a row, since
// mean(h^2) and mean(gm h) are taken together.  P and dwn are summed over a
// workgroup's rows in registers, written once and joined in a fixed order.
#include "m3_device.h"
#include "block_norm.h"

namespace m3 {
namespace {

constexpr int kElems = 8;   // of a thread at a time

// A thread's elements of a row as loaded.  V = 8: NV times eight consecutive
// ones; V = 1 (a width or a row distance that no vector divides): elements a
// workgroup's threads apart.  Behind the row's end the first (last) are
// repeated and their values are 0.
template <typename T, int V, int NV>
struct RowPart;
template <typename T, int NV>
struct RowPart<T, 8, NV> {
  RawVec<T, 8> r[NV];
  static __device__ __forceinline__ int index(int j) {
    return ((j / kElems) * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x)) * kElems + j % kElems;
  }
  __device__ __forceinline__ void load(const T* row, int W) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = index(i * kElems);
      r[i].load(row + (e < W ? e : 0));
    }
  }
  __device__ __forceinline__ void get(float* v, int W) const {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      r[i].get(v + i * kElems);
      const bool on = index(i * kElems) < W;
#pragma unroll
      for (int j = 0; j < kElems; ++j) v[i * kElems + j] = on ? v[i * kElems + j] : 0.0f;
    }
  }
  static __device__ __forceinline__ void put8(float* p, const float* v) {
    *reinterpret_cast<f4*>(p) = f4{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<f4*>(p + 4) = f4{v[4], v[5], v[6], v[7]};
  }
  static __device__ __forceinline__ void put8(bf16_t* p, const float* v) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{v[2 * k], v[2 * k + 1]}, bh2));
    *reinterpret_cast<uint4*>(p) = uint4{w[0], w[1], w[2], w[3]};
  }
  static __device__ __forceinline__ void store(T* row, const float* v, int W) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = index(i * kElems);
      if (e < W) put8(row + e, v + i * kElems);
    }
  }
};
template <typename T, int NV>
struct RowPart<T, 1, NV> {
  Raw1<T> r[NV * kElems];
  static __device__ __forceinline__ int index(int j) {
    return j * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x);
  }
  __device__ __forceinline__ void load(const T* row, int W) {
#pragma unroll
    for (int j = 0; j < NV * kElems; ++j) r[j].load(row, min(index(j), W - 1));
  }
  __device__ __forceinline__ void get(float* v, int W) const {
#pragma unroll
    for (int j = 0; j < NV * kElems; ++j) v[j] = index(j) < W ? r[j].f() : 0.0f;
  }
  static __device__ __forceinline__ void store(T* row, const float* v, int W) {
#pragma unroll
    for (int j = 0; j < NV * kElems; ++j)
      if (index(j) < W) row[index(j)] = from_f32<T>(v[j]);
  }
};

// weights of a thread's elements (1 without any, 0 behind the end)
template <typename R, int E>
__device__ __forceinline__ void weights(float* w, const float* p, int W) {
#pragma unroll
  for (int j = 0; j < E; ++j) {
    const int e = R::index(j);
    w[j] = e < W ? ld_or(p, e, 1.0f) : 0.0f;
  }
}

// Sums over the workgroup, of its waves in order.  Two buffers take turns:
// whoever writes one again has passed the barrier of the other, before which
// everyone had read it.
struct Sums {
  f2 (*sh)[16];
  int turn;
  __device__ __forceinline__ f2 operator()(float a, float b) {
    a = group_sum<64>(a);
    b = group_sum<64>(b);
    const int nw = blockDim.x >> 6;
    if (nw == 1) return f2{a, b};
    f2* s = sh[turn];
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = f2{a, b};
    __syncthreads();
    f2 t = s[0];
    for (int w = 1; w < nw; ++w) t += s[w];
    return t;
  }
};

__device__ __forceinline__ float gate_sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * v));
}
// act(g), and its derivative in d
__device__ __forceinline__ float gate_act(int act, float g, float& d) {
  if (act == kGateLinear) {
    d = 1.0f;
    return g;
  }
  const float s = gate_sigmoid(g);
  if (act == kGateSigmoid) {
    d = s * (1.0f - s);
    return s;
  }
  d = fmaf(g * s, 1.0f - s, s);
  return g * s;
}

template <typename T, int V, int NV>
__global__ __launch_bounds__(1024) void k_block_norm(BlockNormArgs a) {
  using R = RowPart<T, V, NV>;
  constexpr int E = NV * kElems;
  __shared__ f2 sh[2][16];
  Sums sums{sh, 0};
  const int W = a.W;
  const float invW = 1.0f / static_cast<float>(W);
  float wz[E], wn[E];   // of y (with the scale) and of n
  weights<R, E>(wz, a.wy, W);
  weights<R, E>(wn, a.scale, W);
#pragma unroll
  for (int j = 0; j < E; ++j) wz[j] *= wn[j];
  weights<R, E>(wn, a.wn, W);
  const T* xp = static_cast<const T*>(a.x);
  const T* yp = static_cast<const T*>(a.y);
  const T* gp = static_cast<const T*>(a.gate);
  R rx, ry, rg;
  auto fetch = [&](int64_t t) __attribute__((always_inline)) {
    ry.load(yp + t * a.ldy, W);
    rx.load(xp + t * a.ldx, W);
    if (gp) rg.load(gp + t * a.ldg, W);
  };
  fetch(blockIdx.x);
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    float h[E], y[E], g[E];
    ry.get(y, W);
    rx.get(h, W);
    if (gp) {
      rg.get(g, W);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        float d;
        g[j] = gate_act(a.act, g[j], d);
      }
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) g[j] = 1.0f;
    }
    if (t + gridDim.x < a.T) fetch(t + gridDim.x);
    float iy = 1.0f;
    if (!a.raw) {
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < E; ++j) s = fmaf(y[j], y[j], s);
      iy = __builtin_amdgcn_rsqf(fmaf(sums(s, 0.0f).x, invW, a.eps));
    }
#pragma unroll
    for (int j = 0; j < E; ++j) h[j] = fmaf(g[j] * wz[j], y[j] * iy, h[j]);
    R::store(static_cast<T*>(a.h) + t * W, h, W);
    if (!a.n) continue;
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < E; ++j) s = fmaf(h[j], h[j], s);
    const float ih = __builtin_amdgcn_rsqf(fmaf(sums(s, 0.0f).x, invW, a.eps));
#pragma unroll
    for (int j = 0; j < E; ++j) h[j] *= ih * wn[j];
    R::store(static_cast<T*>(a.n) + t * W, h, W);
  }
}

template <typename T, int V, int NV>
__global__ __launch_bounds__(1024) void k_block_norm_bwd(BlockNormArgs a) {
  using R = RowPart<T, V, NV>;
  constexpr int E = NV * kElems;
  __shared__ f2 sh[2][16];
  Sums sums{sh, 0};
  const int W = a.W;
  const float invW = 1.0f / static_cast<float>(W);
  float wz[E], wn[E], pz[E], pn[E];
  weights<R, E>(wz, a.wy, W);
  weights<R, E>(wn, a.scale, W);
#pragma unroll
  for (int j = 0; j < E; ++j) {
    wz[j] *= wn[j];
    pz[j] = pn[j] = 0.0f;
  }
  weights<R, E>(wn, a.wn, W);
  const T* xp = static_cast<const T*>(a.x);
  const T* yp = static_cast<const T*>(a.y);
  const T* gp = static_cast<const T*>(a.gate);
  const T* hp = static_cast<const T*>(a.dh);
  const T* np = static_cast<const T*>(a.dn);
  R rx, ry, rg, rh, rn;
  auto fetch = [&](int64_t t) __attribute__((always_inline)) {
    ry.load(yp + t * a.ldy, W);
    rx.load(xp + t * a.ldx, W);
    if (gp) rg.load(gp + t * a.ldg, W);
    if (np) rn.load(np + t * W, W);
    if (hp) rh.load(hp + t * W, W);
  };
  fetch(blockIdx.x);
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    float h[E], u[E], act[E], da[E], dh[E], gm[E];
    ry.get(u, W);
    rx.get(h, W);
    if (gp) {
      rg.get(act, W);
#pragma unroll
      for (int j = 0; j < E; ++j) act[j] = gate_act(a.act, act[j], da[j]);
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) act[j] = 1.0f;
    }
    if (np) {
      rn.get(gm, W);
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) gm[j] = 0.0f;
    }
    if (hp) {
      rh.get(dh, W);
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) dh[j] = 0.0f;
    }
    if (t + gridDim.x < a.T) fetch(t + gridDim.x);
    float iy = 1.0f;
    if (!a.raw) {
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < E; ++j) s = fmaf(u[j], u[j], s);
      iy = __builtin_amdgcn_rsqf(fmaf(sums(s, 0.0f).x, invW, a.eps));
#pragma unroll
      for (int j = 0; j < E; ++j) u[j] *= iy;
    }
    if (np) {
      float s = 0.0f, d = 0.0f;
#pragma unroll
      for (int j = 0; j < E; ++j) {
        h[j] = fmaf(act[j] * wz[j], u[j], h[j]);
        s = fmaf(h[j], h[j], s);
        d = fmaf(gm[j] * wn[j], h[j], d);
      }
      const f2 sd = sums(s, d);
      const float ih = __builtin_amdgcn_rsqf(fmaf(sd.x, invW, a.eps));
      const float c = sd.y * invW * ih * ih;   // mean(gm m) / rms(h)
#pragma unroll
      for (int j = 0; j < E; ++j) {
        pn[j] = fmaf(gm[j], h[j] * ih, pn[j]);
        dh[j] += ih * fmaf(gm[j], wn[j], -h[j] * c);
      }
    }
    R::store(static_cast<T*>(a.dx) + t * W, dh, W);
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const float du = dh[j] * u[j];
      pz[j] = fmaf(du, act[j], pz[j]);
      if (gp) da[j] *= du * wz[j];        // the gate's gradient
      act[j] *= dh[j] * wz[j];            // gu
      s = fmaf(act[j], u[j], s);
    }
    if (gp) R::store(static_cast<T*>(a.dgate) + t * W, da, W);
    if (!a.raw) {
      const float c = sums(s, 0.0f).x * invW;
#pragma unroll
      for (int j = 0; j < E; ++j) act[j] = iy * fmaf(-u[j], c, act[j]);
    }
    R::store(static_cast<T*>(a.dy) + t * W, act, W);
  }
  RowPart<float, V, NV>::store(a.part + static_cast<int64_t>(blockIdx.x) * 2 * W, pz, W);
  RowPart<float, V, NV>::store(a.part + (static_cast<int64_t>(blockIdx.x) * 2 + 1) * W, pn, W);
}

// The parts of P and dwn of `nblk` workgroups, joined: 64 columns a workgroup,
// its sixteen waves every sixteenth part each.
__global__ __launch_bounds__(1024) void k_block_norm_join(BlockNormArgs a, int nblk) {
  __shared__ float sh[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int ncb = (a.W + 63) / 64;
  const bool second = static_cast<int>(blockIdx.x) >= ncb;
  const int c = (blockIdx.x - (second ? ncb : 0)) * 64 + lane;
  const float* p = a.part + (second ? a.W : 0) + min(c, a.W - 1);
  float s = 0.0f;
#pragma unroll 4
  for (int b = wave; b < nblk; b += 16) s += p[static_cast<int64_t>(b) * 2 * a.W];
  sh[wave][lane] = s;
  __syncthreads();
  if (wave != 0 || c >= a.W) return;
  s = 0.0f;
#pragma unroll
  for (int w = 0; w < 16; ++w) s += sh[w][lane];
  if (second) {
    if (a.dwn) a.dwn[c] = s;
  } else {
    if (a.dwy) a.dwy[c] = s * ld_or(a.scale, c, 1.0f);
    if (a.dscale) a.dscale[c] = s * ld_or(a.wy, c, 1.0f);
  }
}

// Threads of a workgroup: one for every eight elements, up to 1024.
int threads_of(int W) {
  const int n = ((W + kElems - 1) / kElems + 63) / 64 * 64;
  return n > 1024 ? 1024 : n;
}
// Workgroups: as many as are resident, each with several rows.
int groups_of(int T, int W, int threads_per_cu) {
  const int most = 256 * (threads_per_cu / threads_of(W));
  return T < most ? T : most;
}
constexpr int kFwdThreads = 2048, kBwdThreads = 1024;

// eight elements at a time: rows and their distances whole vectors
bool vectors(const BlockNormArgs& a) { return a.W % 8 == 0 && (a.ldx | a.ldy | a.ldg) % 8 == 0; }

template <typename T>
hipError_t run_fwd(const BlockNormArgs& a, hipStream_t s) {
  const int nt = threads_of(a.W), grid = groups_of(a.T, a.W, kFwdThreads);
  const bool two = a.W > 1024 * kElems;
  if (vectors(a)) {
    if (two) k_block_norm<T, 8, 2><<<grid, nt, 0, s>>>(a);
    else k_block_norm<T, 8, 1><<<grid, nt, 0, s>>>(a);
  } else {
    if (two) k_block_norm<T, 1, 2><<<grid, nt, 0, s>>>(a);
    else k_block_norm<T, 1, 1><<<grid, nt, 0, s>>>(a);
  }
  return hipGetLastError();
}

template <typename T>
hipError_t run_bwd(const BlockNormArgs& a, hipStream_t s) {
  const int nt = threads_of(a.W), grid = groups_of(a.T, a.W, kBwdThreads);
  const bool two = a.W > 1024 * kElems;
  if (vectors(a)) {
    if (two) k_block_norm_bwd<T, 8, 2><<<grid, nt, 0, s>>>(a);
    else k_block_norm_bwd<T, 8, 1><<<grid, nt, 0, s>>>(a);
  } else {
    if (two) k_block_norm_bwd<T, 1, 2><<<grid, nt, 0, s>>>(a);
    else k_block_norm_bwd<T, 1, 1><<<grid, nt, 0, s>>>(a);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || (!a.dwy && !a.dscale && !a.dwn)) return e;
  k_block_norm_join<<<2 * ((a.W + 63) / 64), 1024, 0, s>>>(a, grid);
  return hipGetLastError();
}

}  // namespace

size_t block_norm_workspace_bytes(int T, int W) {
  return sizeof(float) * 2 * static_cast<size_t>(groups_of(T, W, kBwdThreads)) * W;
}

hipError_t launch_block_norm(const BlockNormArgs& a, int bf16, hipStream_t s) {
  return bf16 ? run_fwd<bf16_t>(a, s) : run_fwd<float>(a, s);
}

hipError_t launch_block_norm_backward(const BlockNormArgs& a, int bf16, hipStream_t s) {
  return bf16 ? run_bwd<bf16_t>(a, s) : run_bwd<float>(a, s);
}

}  // namespace m3
