// block_norm.hip -- the norms before and after a block, fused with its gate
// and residual scale (gfx950), and the gradients.
//
//   z = y / sqrt(mean y^2 + eps) * wy      (raw: y * wy)
//   h = x + scale act(gate) z,             n = h / sqrt(mean h^2 + eps) * wn
//
// One pass: each row is read and written once and everything between stays in
// registers, so the call is bound by HBM.  A workgroup takes a row at a time,
// 16 bytes a thread, and keeps the weights in registers over its rows
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
//
// bf16, rows of 4096: 16384 124 us for 671 MB (5.4 TB/s), 8192 with gradients 64
// and 121 us for 872 MB (4.7 TB/s); 128 rows 4 us, less than the call takes the
// host.
#include "m3_device.h"
#include "block_norm.h"

namespace m3 {
namespace {

// A thread's E elements of a row as loaded: whole vectors of V, or (V = 1: a
// width or a row distance that no vector divides) single elements, both a
// workgroup's threads apart.  Behind the row's end the first (last) are repeated
// and their values are 0.
template <typename T, int V, int E>
struct RowPart {
  RawVec<T, V> r[E / V];
  static __device__ __forceinline__ int index(int j) {
    return ((j / V) * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x)) * V + j % V;
  }
  __device__ __forceinline__ void load(const T* row, int W) {
#pragma unroll
    for (int i = 0; i < E / V; ++i) {
      const int e = index(i * V);
      r[i].load(row + (V == 1 ? min(e, W - 1) : e < W ? e : 0));
    }
  }
  __device__ __forceinline__ void get(float* v, int W) const {
#pragma unroll
    for (int i = 0; i < E / V; ++i) {
      r[i].get(v + i * V);
      const bool on = index(i * V) < W;
#pragma unroll
      for (int j = 0; j < V; ++j) v[i * V + j] = on ? v[i * V + j] : 0.0f;
    }
  }
  // N of them from element i on, of one vector
  template <int N>
  __device__ __forceinline__ void some(float* v, int i, bool on) const {
    float f[V];
    r[i / V].get(f);
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = on ? f[i % V + j] : 0.0f;
  }
  // what is formed from them is formed anew from here on, not kept in registers
  __device__ __forceinline__ void renew() {
    constexpr int N = static_cast<int>(sizeof(r) / sizeof(uint32_t));
    uint32_t* u = reinterpret_cast<uint32_t*>(r);
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+v"(u[i]));
  }
  static __device__ __forceinline__ void put(float* p, const float* v) {
    if constexpr (V == 1) {
      p[0] = v[0];
    } else {
#pragma unroll
      for (int k = 0; k < V / 4; ++k) reinterpret_cast<f4*>(p)[k] = f4{v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]};
    }
  }
  static __device__ __forceinline__ void put(bf16_t* p, const float* v) {
    if constexpr (V == 1) {
      *reinterpret_cast<__bf16*>(p) = static_cast<__bf16>(v[0]);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{v[2 * k], v[2 * k + 1]}, bh2));
      *reinterpret_cast<uint4*>(p) = uint4{w[0], w[1], w[2], w[3]};
    }
  }
  // N values, of one vector
  template <int N>
  static __device__ __forceinline__ void put_some(float* p, const float* v) {
    if constexpr (N == 4) *reinterpret_cast<f4*>(p) = f4{v[0], v[1], v[2], v[3]};
    else if constexpr (N == 2) *reinterpret_cast<f2*>(p) = f2{v[0], v[1]};
    else p[0] = v[0];
  }
  template <int N>
  static __device__ __forceinline__ void put_some(bf16_t* p, const float* v) {
    if constexpr (N == 1) {
      put(p, v);
    } else {
      uint32_t w[N / 2];
#pragma unroll
      for (int k = 0; k < N / 2; ++k)
        w[k] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{v[2 * k], v[2 * k + 1]}, bh2));
      if constexpr (N == 4) *reinterpret_cast<uint2*>(p) = uint2{w[0], w[1]};
      else *reinterpret_cast<uint32_t*>(p) = w[0];
    }
  }
  template <typename O>
  static __device__ __forceinline__ void store(O* row, const float* v, int W) {
#pragma unroll
    for (int i = 0; i < E / V; ++i) {
      const int e = index(i * V);
      if (e < W) put(row + e, v + i * V);
    }
  }
};

// weights of a thread's elements (1 without any, 0 behind the end)
template <typename T, int V, int E>
__device__ __forceinline__ void weights(float* w, const float* p, int W) {
  if (p) {
    RowPart<float, V, E> r;
    r.load(p, W);
    r.get(w, W);
  } else {
#pragma unroll
    for (int j = 0; j < E; ++j) w[j] = RowPart<T, V, E>::index(j) < W ? 1.0f : 0.0f;
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

template <typename T, int V, int E>
__global__ __launch_bounds__(1024) void k_block_norm(BlockNormArgs a) {
  using R = RowPart<T, V, E>;
  __shared__ f2 sh[2][16];
  Sums sums{sh, 0};
  const int W = a.W;
  const float invW = 1.0f / static_cast<float>(W);
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
  float wz[E], wn[E];   // of y (with the scale) and of n
  weights<T, V, E>(wz, a.wy, W);
  weights<T, V, E>(wn, a.scale, W);
#pragma unroll
  for (int j = 0; j < E; ++j) wz[j] *= wn[j];
  weights<T, V, E>(wn, a.wn, W);
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

template <typename T, int V, int E>
__global__ __launch_bounds__(1024) void k_block_norm_bwd(BlockNormArgs a) {
  using R = RowPart<T, V, E>;
  __shared__ f2 sh[2][16];
  Sums sums{sh, 0};
  const int W = a.W;
  const float invW = 1.0f / static_cast<float>(W);
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
  float wz[E], wn[E], pz[E], pn[E];
  weights<T, V, E>(wz, a.wy, W);
  weights<T, V, E>(wn, a.scale, W);
#pragma unroll
  for (int j = 0; j < E; ++j) {
    wz[j] *= wn[j];
    pz[j] = pn[j] = 0.0f;
  }
  weights<T, V, E>(wn, a.wn, W);
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
  R::store(a.part + static_cast<int64_t>(blockIdx.x) * 2 * W, pz, W);
  R::store(a.part + (static_cast<int64_t>(blockIdx.x) * 2 + 1) * W, pn, W);
}

// The gradients where a thread has more elements than registers for all that the
// kernel above keeps of them: a row is not asked for ahead, what its passes need
// is formed from the loaded values each time, a few elements after the other, and
// P and dwn are summed in LDS.  4854 rows of 5473 bf16: 242 us with the forward
// call, in the kernel above, spilled, 627.
template <typename T, int V, int E>
__global__ __launch_bounds__(1024) void k_block_norm_bwd_lean(BlockNormArgs a) {
  using R = RowPart<T, V, E>;
  constexpr int N = V == 1 ? 1 : E == 16 ? 2 : 4;   // elements at a time
  __shared__ f2 sh[2][16];
  __shared__ __align__(16) float acc[2][1024 * E];
  Sums sums{sh, 0};
  const int W = a.W;
  const float invW = 1.0f / static_cast<float>(W);
  float wz[E], wn[E];
  weights<T, V, E>(wz, a.wy, W);
  weights<T, V, E>(wn, a.scale, W);
#pragma unroll
  for (int j = 0; j < E; ++j) {
    wz[j] *= wn[j];
    acc[0][R::index(j)] = acc[1][R::index(j)] = 0.0f;   // (only the thread's own elements, ever)
  }
  weights<T, V, E>(wn, a.wn, W);
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    R rx, ry, rg, rh, rn;
    ry.load(static_cast<const T*>(a.y) + t * a.ldy, W);
    rx.load(static_cast<const T*>(a.x) + t * a.ldx, W);
    if (a.gate) rg.load(static_cast<const T*>(a.gate) + t * a.ldg, W);
    if (a.dn) rn.load(static_cast<const T*>(a.dn) + t * W, W);
    if (a.dh) rh.load(static_cast<const T*>(a.dh) + t * W, W);
    float iy = 1.0f, ih = 0.0f, c = 0.0f;
    if (!a.raw) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < E; i += N) {
        float y[N];
        ry.template some<N>(y, i, R::index(i / V * V) < W);
#pragma unroll
        for (int j = 0; j < N; ++j) s = fmaf(y[j], y[j], s);
      }
      iy = __builtin_amdgcn_rsqf(fmaf(sums(s, 0.0f).x, invW, a.eps));
    }
    // of elements i ..: weights, act(gate) and its derivative, u and h
    struct Some {
      bool on;
      float act[N], da[N], u[N], h[N];
    };
    auto form = [&](Some& f, int i) __attribute__((always_inline)) {
      f.on = R::index(i / V * V) < W;
      ry.template some<N>(f.u, i, f.on);
      rx.template some<N>(f.h, i, f.on);
      if (a.gate) rg.template some<N>(f.act, i, f.on);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        f.u[j] *= iy;
        f.da[j] = 0.0f;
        f.act[j] = a.gate ? gate_act(a.act, f.act[j], f.da[j]) : 1.0f;
        f.h[j] = fmaf(f.act[j] * wz[i + j], f.u[j], f.h[j]);
      }
    };
    if (a.dn) {
      float s = 0.0f, d = 0.0f;
      ry.renew();
#pragma unroll
      for (int i = 0; i < E; i += N) {
        Some f;
        float gm[N];
        form(f, i);
        rn.template some<N>(gm, i, f.on);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          s = fmaf(f.h[j], f.h[j], s);
          d = fmaf(gm[j] * wn[i + j], f.h[j], d);
        }
        if (i % 4 == 0) __builtin_amdgcn_sched_barrier(0);
      }
      const f2 sd = sums(s, d);
      ih = __builtin_amdgcn_rsqf(fmaf(sd.x, invW, a.eps));
      c = sd.y * invW * ih * ih;
    }
    ry.renew();
    rx.renew();
    if (a.gate) rg.renew();
    if (a.dn) rn.renew();
    float gu[E], s = 0.0f;
#pragma unroll
    for (int i = 0; i < E; i += N) {
      Some f;
      float gm[N], dh[N];
      form(f, i);
#pragma unroll
      for (int j = 0; j < N; ++j) dh[j] = gm[j] = 0.0f;
      if (a.dh) rh.template some<N>(dh, i, f.on);
      if (a.dn) {
        rn.template some<N>(gm, i, f.on);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          dh[j] += ih * fmaf(gm[j], wn[i + j], -f.h[j] * c);
          gm[j] *= f.h[j] * ih;
        }
      }
      const int e = R::index(i);
      if (f.on) R::template put_some<N>(static_cast<T*>(a.dx) + t * W + e, dh);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float du = dh[j] * f.u[j], p = du * f.act[j];
        f.da[j] *= du * wz[i + j];
        gu[i + j] = f.act[j] * dh[j] * wz[i + j];
        s = fmaf(gu[i + j], f.u[j], s);
        acc[0][e + j] += p;
        acc[1][e + j] += gm[j];
      }
      if (a.gate && f.on) R::template put_some<N>(static_cast<T*>(a.dgate) + t * W + e, f.da);
      if (i % 4 == 0) __builtin_amdgcn_sched_barrier(0);
    }
    if (!a.raw) {
      const float m = sums(s, 0.0f).x * invW;
      ry.renew();
#pragma unroll
      for (int i = 0; i < E; i += N) {
        float y[N];
        ry.template some<N>(y, i, R::index(i / V * V) < W);
#pragma unroll
        for (int j = 0; j < N; ++j) gu[i + j] = iy * fmaf(-y[j] * iy, m, gu[i + j]);
      }
    }
    R::store(static_cast<T*>(a.dy) + t * W, gu, W);
  }
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * 2 * W;
#pragma unroll
  for (int j = 0; j < E; ++j)
    if (R::index(j) < W) {
      part[R::index(j)] = acc[0][R::index(j)];
      part[W + R::index(j)] = acc[1][R::index(j)];
    }
}

// Rows of more than 8192 elements where a thread would have 16 single or fp32 ones,
// for which there are no registers: nothing of a row is kept, each pass reads it
// again, from the caches (the rows under way are at most 320 KB a workgroup).
// 2000 rows of 16383 bf16: forward 148 us (in registers, spilled, 377), with
// gradients 444 (1602); 2000 of 16000 fp32 with gradients 477 (879).  In vectors of
// bf16 the kernels above are faster: 71 us forward, with gradients 344 (517 so).
//
// A thread's K elements of a turn: a vector, or four single ones; behind the
// row's end 0.
template <typename T, int V>
struct Turn {
  static constexpr int K = V == 1 ? 4 : V, STEP = 1024 * K;
  static __device__ __forceinline__ int first() { return threadIdx.x * V; }
  static __device__ __forceinline__ int at(int e, int j) { return V == 1 ? e + 1024 * j : e + j; }
  template <typename P>
  static __device__ __forceinline__ void take(float* v, const P* row, int e, int W) {
    if constexpr (V == 1) {
      RawVec<P, 1> r[K];
#pragma unroll
      for (int j = 0; j < K; ++j) r[j].load(row + min(at(e, j), W - 1));
#pragma unroll
      for (int j = 0; j < K; ++j) {
        r[j].get(v + j);
        v[j] = at(e, j) < W ? v[j] : 0.0f;
      }
    } else {
      RawVec<P, K> r;
      r.load(row + e);
      r.get(v);
    }
  }
  // weights, 1 without any
  static __device__ __forceinline__ void take_or(float* v, const float* p, int e, int W) {
    if (p) {
      take(v, p, e, W);
    } else {
#pragma unroll
      for (int j = 0; j < K; ++j) v[j] = 1.0f;
    }
  }
  template <typename P>
  static __device__ __forceinline__ void put(P* row, const float* v, int e, int W) {
    if constexpr (V == 1) {
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (at(e, j) < W) RowPart<T, 1, 1>::put(row + at(e, j), v + j);
    } else {
      RowPart<T, V, V>::put(row + e, v);
    }
  }
  // act(gate), its derivative, u and h
  float wz[K], act[K], da[K], u[K], h[K];
  __device__ __forceinline__ Turn(const BlockNormArgs& a, int64_t t, int e, float iy) {
    take(u, static_cast<const T*>(a.y) + t * a.ldy, e, a.W);
    take(h, static_cast<const T*>(a.x) + t * a.ldx, e, a.W);
    if (a.gate) take(act, static_cast<const T*>(a.gate) + t * a.ldg, e, a.W);
    float sc[K];
    take_or(wz, a.wy, e, a.W);
    take_or(sc, a.scale, e, a.W);
#pragma unroll
    for (int j = 0; j < K; ++j) {
      wz[j] *= sc[j];
      u[j] *= iy;
      da[j] = 0.0f;
      act[j] = a.gate ? gate_act(a.act, act[j], da[j]) : 1.0f;
      h[j] = fmaf(act[j] * wz[j], u[j], h[j]);
    }
  }
  static __device__ __forceinline__ float square(const BlockNormArgs& a, int64_t t) {
    float s = 0.0f;
#pragma unroll 2
    for (int e = first(); e < a.W; e += STEP) {
      float y[K];
      take(y, static_cast<const T*>(a.y) + t * a.ldy, e, a.W);
#pragma unroll
      for (int j = 0; j < K; ++j) s = fmaf(y[j], y[j], s);
    }
    return s;
  }
};

template <typename T, int V>
__global__ __launch_bounds__(1024) void k_block_norm_long(BlockNormArgs a) {
  using P = Turn<T, V>;
  __shared__ f2 sh[2][16];
  Sums sums{sh, 0};
  const float invW = 1.0f / static_cast<float>(a.W);
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const float iy = a.raw ? 1.0f : __builtin_amdgcn_rsqf(fmaf(sums(P::square(a, t), 0.0f).x, invW, a.eps));
    float ih = 0.0f;
    if (a.n) {   // (before h is written, which may be x or y)
      float s = 0.0f;
#pragma unroll 2
      for (int e = P::first(); e < a.W; e += P::STEP) {
        const P f(a, t, e, iy);
#pragma unroll
        for (int j = 0; j < P::K; ++j) s = fmaf(f.h[j], f.h[j], s);
      }
      ih = __builtin_amdgcn_rsqf(fmaf(sums(s, 0.0f).x, invW, a.eps));
    }
#pragma unroll 1
    for (int e = P::first(); e < a.W; e += P::STEP) {
      P f(a, t, e, iy);
      P::put(static_cast<T*>(a.h) + t * a.W, f.h, e, a.W);
      if (!a.n) continue;
      float wn[P::K];
      P::take_or(wn, a.wn, e, a.W);
#pragma unroll
      for (int j = 0; j < P::K; ++j) f.h[j] *= ih * wn[j];
      P::put(static_cast<T*>(a.n) + t * a.W, f.h, e, a.W);
    }
  }
}

// With q = act(gate) wy scale u, so that gu u = q dH:
//   sum gu u = sum q dh + (sum q gm - mean(gm m) / rms(h) sum q h) / rms(h)
// is there before dH is, and all outputs are formed in one pass.
template <typename T, int V>
__global__ __launch_bounds__(1024) void k_block_norm_bwd_long(BlockNormArgs a) {
  using P = Turn<T, V>;
  constexpr int K = P::K;
  __shared__ f2 sh[2][16];
  __shared__ __align__(16) float acc[2][kBlockNormMaxWidth];   // (a thread's own elements, never another's)
  Sums sums{sh, 0};
  const int W = a.W;
  const float invW = 1.0f / static_cast<float>(W);
  for (int e = P::first(); e < W; e += P::STEP)
#pragma unroll
    for (int j = 0; j < K; ++j)
      if (P::at(e, j) < W) acc[0][P::at(e, j)] = acc[1][P::at(e, j)] = 0.0f;
  const T* dhp = static_cast<const T*>(a.dh);
  const T* dnp = static_cast<const T*>(a.dn);
  auto grads = [&](float* d, float* g, float* wn, int64_t t, int e) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < K; ++j) d[j] = g[j] = 0.0f;
    if (dhp) P::take(d, dhp + t * W, e, W);
    if (dnp) P::take(g, dnp + t * W, e, W);
    P::take_or(wn, a.wn, e, W);
  };
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const float iy = a.raw ? 1.0f : __builtin_amdgcn_rsqf(fmaf(sums(P::square(a, t), 0.0f).x, invW, a.eps));
    float hh = 0.0f, gh = 0.0f, qd = 0.0f, qg = 0.0f, qh = 0.0f;
#pragma unroll 1
    for (int e = P::first(); e < W; e += P::STEP) {
      float d[K], g[K], wn[K];
      grads(d, g, wn, t, e);
      const P f(a, t, e, iy);
#pragma unroll
      for (int j = 0; j < K; ++j) {
        const float gm = g[j] * wn[j], q = f.act[j] * f.wz[j] * f.u[j];
        hh = fmaf(f.h[j], f.h[j], hh);
        gh = fmaf(gm, f.h[j], gh);
        qd = fmaf(q, d[j], qd);
        qg = fmaf(q, gm, qg);
        qh = fmaf(q, f.h[j], qh);
      }
    }
    const f2 s1 = sums(hh, gh), s2 = sums(qd, qg);
    const float sqh = sums(qh, 0.0f).x;
    // (without dn an h that is not finite reaches nothing)
    const float ih = dnp ? __builtin_amdgcn_rsqf(fmaf(s1.x, invW, a.eps)) : 0.0f;
    const float c = s1.y * invW * ih * ih;
    const float m = a.raw ? 0.0f : (dnp ? fmaf(ih, fmaf(-c, sqh, s2.y), s2.x) : s2.x) * invW;
#pragma unroll 1
    for (int e = P::first(); e < W; e += P::STEP) {
      float d[K], g[K], wn[K];
      grads(d, g, wn, t, e);
      P f(a, t, e, iy);
#pragma unroll
      for (int j = 0; j < K; ++j) {
        if (dnp) d[j] += ih * fmaf(g[j], wn[j], -f.h[j] * c);
        const float du = d[j] * f.u[j];
        if (V > 1 || P::at(e, j) < W) {
          acc[0][P::at(e, j)] += du * f.act[j];
          if (dnp) acc[1][P::at(e, j)] += g[j] * f.h[j] * ih;
        }
        f.da[j] *= du * f.wz[j];
        f.h[j] = iy * fmaf(-f.u[j], m, f.act[j] * d[j] * f.wz[j]);
      }
      P::put(static_cast<T*>(a.dx) + t * W, d, e, W);
      if (a.gate) P::put(static_cast<T*>(a.dgate) + t * W, f.da, e, W);
      P::put(static_cast<T*>(a.dy) + t * W, f.h, e, W);
    }
  }
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * 2 * W;
  for (int e = P::first(); e < W; e += P::STEP)
#pragma unroll
    for (int j = 0; j < K; ++j)
      if (P::at(e, j) < W) {
        part[P::at(e, j)] = acc[0][P::at(e, j)];
        part[W + P::at(e, j)] = acc[1][P::at(e, j)];
      }
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

// Elements of a thread: a vector of 16 bytes, or four single ones, twice or four
// times where 1024 threads are not enough for the row.  (Eight in fp32 spill the
// gradients: 5003 rows of 1021 with them 162 us, with four 67.)
int elems_of(int W, bool wide) {
  const int e = wide ? 8 : 4;
  return W <= 1024 * e ? e : W <= 2048 * e ? 2 * e : 4 * e;
}
int threads_of(int W, bool wide) {
  const int e = elems_of(W, wide);
  return ((W + e - 1) / e + 63) / 64 * 64;
}
// Workgroups: as many as are resident, each with several rows.
int groups_of(int T, int W, bool wide, int threads_per_cu) {
  const int most = 256 * (threads_per_cu / threads_of(W, wide));
  return T < most ? T : most;
}
constexpr int kFwdThreads = 2048, kBwdThreads = 1024;

// rows and their distances whole vectors of 16 bytes
template <typename T>
bool vectors(const BlockNormArgs& a) {
  return (a.W | a.ldx | a.ldy | a.ldg) % (16 / static_cast<int>(sizeof(T))) == 0;
}

// Elements of a thread decide: few stay in registers throughout, of more only the
// loaded values (gradients), of most nothing (figures at the kernels).
template <typename T, bool BWD, int V, int E>
hipError_t run(const BlockNormArgs& a, int grid, int nt, hipStream_t s) {
  if constexpr (BWD && E == 16 && V < 8) k_block_norm_bwd_long<T, V><<<grid, 1024, 0, s>>>(a);
  else if constexpr (E == 16 && V == 1) k_block_norm_long<T, V><<<grid, 1024, 0, s>>>(a);
  else if constexpr (BWD && (V == 8 ? E == 16 : E == 8)) k_block_norm_bwd_lean<T, V, E><<<grid, nt, 0, s>>>(a);
  else if constexpr (BWD) k_block_norm_bwd<T, V, E><<<grid, nt, 0, s>>>(a);
  else k_block_norm<T, V, E><<<grid, nt, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T, bool BWD>
hipError_t run_rows(const BlockNormArgs& a, int* grid, hipStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const bool vec = vectors<T>(a), wide = vec && V == 8;
  const int nt = threads_of(a.W, wide), e = elems_of(a.W, wide);
  *grid = groups_of(a.T, a.W, wide, BWD ? kBwdThreads : kFwdThreads);
  if (vec) {
    if (e == V) return run<T, BWD, V, V>(a, *grid, nt, s);
    if (e == 2 * V) return run<T, BWD, V, 2 * V>(a, *grid, nt, s);
    if constexpr (V == 4) return run<T, BWD, V, 4 * V>(a, *grid, nt, s);
  }
  if (e == 4) return run<T, BWD, 1, 4>(a, *grid, nt, s);
  return e == 8 ? run<T, BWD, 1, 8>(a, *grid, nt, s) : run<T, BWD, 1, 16>(a, *grid, nt, s);
}

template <typename T>
hipError_t run_fwd(const BlockNormArgs& a, hipStream_t s) {
  int grid;
  return run_rows<T, false>(a, &grid, s);
}

template <typename T>
hipError_t run_bwd(const BlockNormArgs& a, hipStream_t s) {
  int grid;
  const hipError_t e = run_rows<T, true>(a, &grid, s);
  if (e != hipSuccess || (!a.dwy && !a.dscale && !a.dwn)) return e;
  k_block_norm_join<<<2 * ((a.W + 63) / 64), 1024, 0, s>>>(a, grid);
  return hipGetLastError();
}

}  // namespace

size_t block_norm_workspace_bytes(int T, int W) {
  // (the more workgroups of the two kinds)
  const int n = groups_of(T, W, false, kBwdThreads), m = groups_of(T, W, true, kBwdThreads);
  return sizeof(float) * 2 * static_cast<size_t>(n > m ? n : m) * W;
}

hipError_t launch_block_norm(const BlockNormArgs& a, int bf16, hipStream_t s) {
  return bf16 ? run_fwd<bf16_t>(a, s) : run_fwd<float>(a, s);
}

hipError_t launch_block_norm_backward(const BlockNormArgs& a, int bf16, hipStream_t s) {
  return bf16 ? run_bwd<bf16_t>(a, s) : run_bwd<float>(a, s);
}

}  // namespace m3
