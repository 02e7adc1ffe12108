// gated.hip -- the gated linear recurrence (gfx950): the scan over a prompt
// (dense or packed), one decode step, and the gradients of the scan.
//
//   L_t = -c softplus(decay) sigmoid(r_t),   a_t = exp(L_t),
//   m_t = sqrt(1 - a_t^2),                   u_t = sigmoid(i_t) x_t,
//   h_t = a_t h_{t-1} + m_t u_t
//
// per channel, in fp32.  1 - a_t^2 is -expm1(2 L_t): a polynomial near zero,
// where 1 - a^2 would cancel.  The gradients follow the adjoint
// g_t = dy_t + a_{t+1} g_{t+1} (plus dhT at a sequence's end), carried here
// as q_t = a_t g_t; with d m / d L = -a^2 / m the gradient of L appears only
// as dL_t L_t, in which L / m has the limit 0 at a = 1.
#include "m3_device.h"
#include "gated.h"

namespace m3 {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
typedef unsigned long long u64;

// V consecutive elements (1 or 8) of a row
template <typename T, int V>
__device__ __forceinline__ void store_v(T* p, const float* v) {
  if constexpr (V == 1) {
    p[0] = from_f32<T>(v[0]);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int k = 0; k < V / 4; ++k)
      reinterpret_cast<f4*>(p)[k] = f4{v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]};
  } else {
    uint32_t w[V / 2];
#pragma unroll
    for (int k = 0; k < V / 2; ++k)
      w[k] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{v[2 * k], v[2 * k + 1]}, bh2));
    *reinterpret_cast<uint4*>(p) = uint4{w[0], w[1], w[2], w[3]};
  }
}

// one element of a row whose address is uniform, off bytes on (the hardware's
// conversion to bf16 rounds to nearest, as from_f32 does in six instructions)
__device__ __forceinline__ void put(float* row, uint32_t off, float v) {
  *reinterpret_cast<float*>(reinterpret_cast<char*>(row) + off) = v;
}
__device__ __forceinline__ void put(bf16_t* row, uint32_t off, float v) {
  *reinterpret_cast<__bf16*>(reinterpret_cast<char*>(row) + off) = static_cast<__bf16>(v);
}

// TOK rows from t0 on of the channel at ch.  Rows past the end repeat the
// last one.  The row's address is uniform: the lane adds a 32-bit offset.
template <typename T, int TOK>
__device__ __forceinline__ void load_rows(Raw1<T>* raw, const T* p, int64_t ld, int ch, int t0,
                                          int T_) {
  const uint32_t off = static_cast<uint32_t>(ch) * static_cast<uint32_t>(sizeof(T));
  const char* row = reinterpret_cast<const char*>(p + min(t0, T_ - 1) * ld);
  const int64_t step = ld * static_cast<int64_t>(sizeof(T));
#pragma unroll
  for (int j = 0; j < TOK; ++j) {
    raw[j].load(reinterpret_cast<const T*>(row + off), 0);
    row += t0 + j + 1 < T_ ? step : 0;
    __builtin_amdgcn_sched_barrier(0);   // one row address at a time
  }
}

// -c softplus(decay) log2(e), the factor of sigmoid(r) in log2(a)
__device__ __forceinline__ float decay_factor(float d, float c) {
  return -c * kLog2e * (fmaxf(d, 0.0f) + log1pf(expf(-fabsf(d))));
}

__device__ __forceinline__ float sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * v));
}

// a and 1 - a^2 from l = log2(a) <= 0.  With z = 2 L = 2 ln(2) l, the
// polynomial interpolates (1 - e^z) / l at Chebyshev points of z in
// [-0.35, 0] (relative error 1.5e-8); below that 1 - a^2 >= 0.3 loses nothing
// that fp32 keeps.
constexpr float kZ = 2.0f * kLn2;
__device__ __forceinline__ void decay_of(float l, float& a, float& m2) {
  a = __builtin_amdgcn_exp2f(l);
  float p = fmaf(l, -7.2112456e-03f * kZ * kZ * kZ * kZ * kZ, -4.1331873e-02f * kZ * kZ * kZ * kZ);
  p = fmaf(l, p, -1.6662531e-01f * kZ * kZ * kZ);
  p = fmaf(l, p, -4.9999820e-01f * kZ * kZ);
  p = fmaf(l, p, -0.99999999f * kZ);
  m2 = l > -0.35f / kZ ? l * p : fmaf(-a, a, 1.0f);
}

// ---------------------------------------------------------------------------
// Joining affine maps of a carry: after `h + p * c`.  In packed calls a row
// that starts (ends) a sequence cuts the carry off: its p is kReset, and what
// was carried up to there is dropped by a select, so that a NaN or an
// infinity of one sequence, or of rows that belong to none, stays there.  A
// decay is never negative, so -0 marks nothing else.
constexpr float kReset = -0.0f;
template <bool PACKED>
__device__ __forceinline__ bool is_reset(float p) {
  return PACKED && __float_as_uint(p) == 0x80000000u;
}
template <bool PACKED>
__device__ __forceinline__ float join(float p, float c, float h) {
  return is_reset<PACKED>(p) ? h : fmaf(p, c, h);
}
template <bool PACKED>
__device__ __forceinline__ float join_p(float p, float cp) {
  return is_reset<PACKED>(p) ? p : cp * p;
}

// The carry from time tile to time tile of one channel.  A tile is a map
// h -> H + P h.  Each publishes its map as soon as it has it; tiles come in
// groups of kGroup, and only the last tile of a group publishes the state
// after it.  A tile starts from the state before its group and applies the
// maps of the tiles before it in the group, always in that order, so results
// do not depend on timing, and the wait for a state passes from group to group
// instead of from tile to tile (about 0.8 us each).
//
// A workgroup takes a ticket when it starts; tickets run over the tiles in the
// order in which the carry moves, so whoever waits, waits for a workgroup that
// has started already and that waits, in turn, only for earlier tickets: every
// wait ends.  A slot is one 8-byte word, which needs no fence: a map's P and H
// (or 0 and a state), all ones until it is there (a NaN is published as the
// usual one, which has fewer).
constexpr int kGroup = 8;
constexpr u64 kNotYet = ~u64{0};
__device__ __forceinline__ void publish(u64* slot, float p, float h) {
  const uint32_t hi = p == p ? __float_as_uint(p) : 0x7fc00000u;
  __hip_atomic_store(slot, u64{hi} << 32 | __float_as_uint(h), __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ u64 peek(const u64* slot) {
  return __hip_atomic_load(slot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ bool ready(u64 w) { return static_cast<uint32_t>(w >> 32) != 0xffffffffu; }

// Slots of tile n (in the order of the carry) of a chain, for one lane.
struct Carry {
  u64 *maps, *states;   // of the first tile of its group; before its group
  int64_t stride;
  int r, n0;
  bool more;            // tiles follow
  __device__ __forceinline__ Carry(const GatedArgs& g, int n, int chain, int lane)
      : stride(static_cast<int64_t>(g.nchain) * 64), r(n % kGroup), n0(n - n % kGroup),
        more(n + 1 < g.ntile) {
    maps = g.slots + n0 * stride + chain * 64 + lane;
    states = g.slots + (g.ntile + n0 / kGroup - 1) * stride + chain * 64 + lane;
  }
  // the tile's own map
  __device__ __forceinline__ void give(float P, float H) const {
    if (r + 1 < kGroup && more) publish(maps + r * stride, P, H);
  }
  // wave w fetches the w-th map before the tile, the last one the state before the group
  __device__ __forceinline__ void fetch(u64 (*s)[64], int w, int lane) const {
    static_assert(kGroup <= 8, "a wave for each");
    const u64* slot = w < r ? maps + w * stride : states;
    if (w < r || (w == kGroup - 1 && n0 > 0)) {
      u64 m;
      while (!ready(m = peek(slot))) __builtin_amdgcn_s_sleep(1);
      s[w][lane] = m;
    }
  }
  // the state before the tile from what was fetched
  template <bool PACKED>
  __device__ __forceinline__ float take(const u64 (*s)[64], int lane, float first) const {
    float h = n0 > 0 ? __uint_as_float(static_cast<uint32_t>(s[kGroup - 1][lane])) : first;
    for (int k = 0; k < r; ++k) {
      const u64 m = s[k][lane];
      h = join<PACKED>(__uint_as_float(static_cast<uint32_t>(m >> 32)), h,
                       __uint_as_float(static_cast<uint32_t>(m)));
    }
    return h;
  }
  // the state after the tile, from the last of a group
  __device__ __forceinline__ void pass_on(float h) const {
    if (r + 1 == kGroup && more) publish(states + stride, 0.0f, h);
  }
};

// The last sequence that starts at or before row t (-1: none), by a search
// over the clean offsets.
__device__ __forceinline__ int seq_of(const int32_t* cu, int S, int t) {
  int lo = 0, hi = S + 1;   // first index with cu > t
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t) lo = mid + 1; else hi = mid;
  }
  return lo - 1;
}

// Offsets clamped into [0, T] and raised to the largest one before, by one
// workgroup: a thread takes `per` of them, and the threads' maxima are joined.
template <int THREADS>
__device__ __forceinline__ void clean_offsets(const int32_t* cu, int S, int T, int32_t* c) {
  __shared__ int top[THREADS];
  const int tid = threadIdx.x, per = S / THREADS + 1, k0 = tid * per, k1 = min(k0 + per, S + 1);
  int v = 0;
  for (int k = k0; k < k1; ++k) {
    v = max(v, min(cu[k], T));
    c[k] = v;
  }
  top[tid] = v;
  __syncthreads();
  for (int o = 1; o < THREADS; o <<= 1) {
    const int w = tid >= o ? top[tid - o] : 0;
    __syncthreads();
    top[tid] = max(top[tid], w);
    __syncthreads();
  }
  const int before = tid > 0 ? top[tid - 1] : 0;
  for (int k = k0; k < k1; ++k) c[k] = max(c[k], before);
  __syncthreads();
}

// Clears the ticket counter and the carry slots; for packed calls also writes
// the clean offsets and the windows, and gives the state rows of empty sequences
// their value (src row or 0).  Up to kInitSeqs offsets are cleaned by every
// workgroup for itself, more by k_gated_clean before.
constexpr int kInitSeqs = 8192;
__global__ __launch_bounds__(256) void k_gated_init(GatedArgs a, const float* src, float* dst,
                                                    int64_t nslot) {
  const int tid = threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * blockDim.x + tid;
  for (int64_t i = at; i < nslot / 2; i += step)
    reinterpret_cast<ulonglong2*>(a.slots)[i] = ulonglong2{kNotYet, kNotYet};   // 64 slots to a chain
  if (blockIdx.x == 0 && tid == 0) *a.ticket = 0;
  if (!a.cu) return;
  __shared__ int32_t own[kInitSeqs + 1];
  const int32_t* c = a.cuc;
  if (a.S <= kInitSeqs) {
    clean_offsets<256>(a.cu, a.S, a.T, own);
    if (blockIdx.x == 0)
      for (int k = tid; k <= a.S; k += 256) a.cuc[k] = own[k];
    c = own;
  }
  for (int64_t n = at; n * 32 < a.T; n += step) {
    const int t0 = static_cast<int>(n * 32);
    GatedWindow w{0u, 0u, 0u, 0, 0};
    w.s0 = max(0, seq_of(c, a.S, t0));
    w.s1 = min(max(0, seq_of(c, a.S, min(t0 + 32, a.T) - 1)), a.S - 1);
    for (int s = w.s0; s < a.S; ++s) {
      const int b = c[s] - t0, e = c[s + 1] - t0;
      if (b >= 32) break;
      if (e > b && e > 0) {
        if (b >= 0) w.start |= 1u << b;
        if (e <= 32) w.end |= 1u << (e - 1);
        const uint32_t upto = e >= 32 ? 0xffffffffu : (1u << e) - 1u;
        w.live |= upto & ~(b > 0 ? (1u << b) - 1u : 0u);
      }
    }
    a.win[n] = w;
  }
  if (dst)
    for (int k = blockIdx.x; k < a.S; k += gridDim.x)
      if (c[k + 1] <= c[k])
        for (int j = tid; j < a.D; j += blockDim.x)
          dst[static_cast<int64_t>(k) * a.D + j] = src ? src[static_cast<int64_t>(k) * a.D + j] : 0.0f;
}
__global__ __launch_bounds__(1024) void k_gated_clean(GatedArgs a) {
  clean_offsets<1024>(a.cu, a.S, a.T, a.cuc);
}

// A wave's TOK rows of a window: one 32-byte load where a search over the offsets
// would be a chain of them (16384 x 2048 in 64 sequences: fp32 124 us, with the
// search 145, bf16 86 and 98).
template <int TOK>
__device__ __forceinline__ GatedWindow window_of(const GatedArgs& g, int t0) {
  GatedWindow w{0u, 0u, 0u, 0, 0};
  if (t0 >= g.T) return w;
  w = g.win[t0 / 32];
  const uint32_t some = TOK == 32 ? 0xffffffffu : (1u << (TOK & 31)) - 1u;
  const int sh = TOK == 32 ? 0 : t0 % 32;
  w.start = w.start >> sh & some;
  w.end = w.end >> sh & some;
  w.live = w.live >> sh & some;
  return w;
}

__device__ __forceinline__ unsigned take_ticket(const GatedArgs& a) {
  if (a.ntile == 1) return blockIdx.x;
  __shared__ unsigned n;
  if (threadIdx.x == 0)
    n = __hip_atomic_fetch_add(a.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  return n;
}

// ---------------------------------------------------------------------------
// One workgroup: TOK * WAVES rows of 64 channels.  A wave scans its TOK
// rows from a zero state, keeping h and the running product of a; the waves'
// ends are joined through LDS, the tiles' through the carry slots, and
// y = h_local + product * carry.  x, r, i are read once and y written once, 8
// bytes an element in bf16: bound by HBM, closely followed by the six
// transcendental instructions an element (16384 x 4096: 123 to 127 us, 4.2 to
// 4.4 TB/s; 16 x 2048 x 4096: 226 us, 4.7 TB/s).  One channel a lane and 32
// rows a wave, timed before the carry went by groups: 127 us; 16 rows 136,
// 16 waves of 8 rows 205, two channels and 16 rows 135.
template <typename T, int TOK, int WAVES, bool PACKED>
__global__ __launch_bounds__(64 * WAVES, 4) void k_gated_scan(GatedArgs g) {
  constexpr int TILE = TOK * WAVES;
  static_assert(TOK <= 32 && 32 % TOK == 0 && kGatedChunk % TOK == 0, "rows in one window");
  static_assert(WAVES >= kGroup, "a wave for each slot before a tile");
  __shared__ float sH[WAVES][64], sP[WAVES][64], sC[64], sF[64];
  __shared__ u64 sM[kGroup][64];
  const unsigned n = take_ticket(g);
  const int tile = static_cast<int>(n / g.nchain), chain = static_cast<int>(n % g.nchain);
  const int b = chain / g.ncb, cb = chain % g.ncb;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ch = cb * 64 + lane;
  const bool on = ch < g.D;
  const int chc = on ? ch : g.D - 1;   // lanes past the end read the last channel
  const int t0 = tile * TILE + wave * TOK;
  const int64_t row0 = static_cast<int64_t>(b) * g.T;
  const T* x = static_cast<const T*>(g.x) + row0 * g.ldx;
  const T* r = static_cast<const T*>(g.r) + row0 * g.ldr;
  const T* gi = static_cast<const T*>(g.i) + row0 * g.ldi;
  T* y = static_cast<T*>(g.y) + row0 * g.D;

  const float dec = g.decay[chc];
  Raw1<T> rx[TOK], rr[TOK], ri[TOK];
  load_rows<T, TOK>(rr, r, g.ldr, chc, t0, g.T);
  load_rows<T, TOK>(rx, x, g.ldx, chc, t0, g.T);
  load_rows<T, TOK>(ri, gi, g.ldi, chc, t0, g.T);
  const Carry cr(g, tile, chain, lane);
  // h0 is read before the tile gives its map: hT may be the same memory, and
  // the last tile writes it as soon as it has the maps before it
  if (!PACKED && wave == 0)
    sF[lane] = cr.n0 == 0 && g.h0 ? g.h0[static_cast<int64_t>(b) * g.D + chc] : 0.0f;
  if (wave == 0) sC[lane] = decay_factor(dec, g.c);
  GatedWindow w{};
  if constexpr (PACKED) w = window_of<TOK>(g, t0);
  __syncthreads();
  const float k = sC[lane];

  float h = 0.0f, P = 1.0f, hl[TOK], pl[TOK];
  int s = w.s0;
#pragma unroll
  for (int j = 0; j < TOK; ++j) {
    const float vx = rx[j].f(), vr = rr[j].f(), vi = ri[j].f();
    if constexpr (PACKED) {
      if (w.start >> j & 1) {
        while (g.cuc[s] < t0 + j || g.cuc[s + 1] <= t0 + j) ++s;
        h = g.h0 ? g.h0[static_cast<int64_t>(s) * g.D + chc] : 0.0f;
        P = kReset;
      }
    }
    float a, m2;
    decay_of(k * sigmoid(vr), a, m2);
    const float bt = __builtin_amdgcn_sqrtf(m2) * (sigmoid(vi) * vx);
    h = fmaf(a, h, bt);
    P *= a;
    hl[j] = h;
    pl[j] = P;
  }
  sH[wave][lane] = h;
  sP[wave][lane] = P;
  __syncthreads();
  // the wave's entry state from the tile's: cH + cP * carry
  float cH = 0.0f, cP = 1.0f;
  for (int u = 0; u < wave; ++u) {
    const float p = sP[u][lane];
    cH = join<PACKED>(p, cH, sH[u][lane]);
    cP = join_p<PACKED>(p, cP);
  }
  const float tP = join_p<PACKED>(P, cP), tH = join<PACKED>(P, cH, h);
  if (wave == WAVES - 1) cr.give(tP, tH);   // the last wave's is the tile's
  cr.fetch(sM, wave, lane);
  __syncthreads();
  const float before = cr.take<PACKED>(sM, lane, PACKED ? 0.0f : sF[lane]);
  if (wave == WAVES - 1) cr.pass_on(join<PACKED>(tP, before, tH));
  const float carry = join<PACKED>(cP, before, cH);
  if (!on) return;
  if (g.states && t0 % kGatedChunk == 0 && t0 < g.T) {
    const int64_t nst = (g.T + kGatedChunk - 1) / kGatedChunk;
    g.states[(b * nst + t0 / kGatedChunk) * g.D + ch] = carry;
  }
  const uint32_t off = static_cast<uint32_t>(ch) * static_cast<uint32_t>(sizeof(T));
  s = w.s0;
#pragma unroll
  for (int j = 0; j < TOK; ++j) {
    const int t = t0 + j;
    if (t >= g.T) break;
    if (PACKED && !(w.live >> j & 1)) continue;
    const float o = join<PACKED>(pl[j], carry, hl[j]);
    put(y + static_cast<int64_t>(t) * g.D, off, o);
    if (PACKED) {
      if (w.end >> j & 1) {
        while (g.cuc[s + 1] <= t) ++s;   // the sequence whose last row this is
        if (g.hT) g.hT[static_cast<int64_t>(s) * g.D + ch] = o;
      }
    } else if (t == g.T - 1 && g.hT) {
      g.hT[static_cast<int64_t>(b) * g.D + ch] = o;
    }
  }
}

// ---------------------------------------------------------------------------
// Gradients.  Tiles run from the last to the first.  Each recomputes its h
// from the chunk state that the scan saved, scans q_t = a_t (dy_t + q_{t+1})
// backwards from zero with the running product of a, takes q of the next
// tile as its carry, and writes dx, dr, di and a partial sum of ddecay.
//
// A row keeps six numbers from pass to pass: a, dy and, first, m, sigmoid(r),
// sigmoid(i), x; these become the factors of g in dx, di, dL L and dr as soon
// as h is known, in place, so 16 rows fit 128 registers (four waves a SIMD).
// 14 bytes an element in bf16: 4 x 2048 x 4096 in 120 us, 3.9 TB/s.
template <typename T, int TOK, int WAVES, bool PACKED>
__global__ __launch_bounds__(64 * WAVES, 4) void k_gated_backward(GatedArgs g) {
  constexpr int TILE = TOK * WAVES;
  static_assert(TILE == kGatedChunk && 32 % TOK == 0, "one saved state per tile; rows in one window");
  static_assert(WAVES >= kGroup, "a wave for each slot before a tile");
  __shared__ float sH[WAVES][64], sP[WAVES][64], sC[64];
  __shared__ u64 sM[kGroup][64];
  const unsigned n = take_ticket(g);
  const int tile = g.ntile - 1 - static_cast<int>(n / g.nchain);
  const int chain = static_cast<int>(n % g.nchain);
  const int b = chain / g.ncb, cb = chain % g.ncb;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ch = cb * 64 + lane;
  const bool on = ch < g.D;
  const int chc = on ? ch : g.D - 1;
  const int t0 = tile * TILE + wave * TOK;
  const int nrow = min(TOK, g.T - t0);   // rows of this wave (may be <= 0)
  const int64_t row0 = static_cast<int64_t>(b) * g.T;

  const float dec = g.decay[chc];
  float entry = g.cstates[(b * static_cast<int64_t>(g.ntile) + tile) * g.D + chc];
  Raw1<T> rx[TOK], rr[TOK], ri[TOK], rd[TOK];
  load_rows<T, TOK>(rr, static_cast<const T*>(g.r) + row0 * g.ldr, g.ldr, chc, t0, g.T);
  load_rows<T, TOK>(rx, static_cast<const T*>(g.x) + row0 * g.ldx, g.ldx, chc, t0, g.T);
  load_rows<T, TOK>(ri, static_cast<const T*>(g.i) + row0 * g.ldi, g.ldi, chc, t0, g.T);
  load_rows<T, TOK>(rd, static_cast<const T*>(g.dy) + row0 * g.D, g.D, chc, t0, g.T);
  if (wave == 0) sC[lane] = decay_factor(dec, g.c);
  GatedWindow w{};
  if constexpr (PACKED) w = window_of<TOK>(g, t0);
  __syncthreads();
  const float k = sC[lane];

  // forward: the gates and the wave's scan from zero (rows past the end come
  // after those that count)
  float h = 0.0f, P = 1.0f, av[TOK], g1[TOK], g2[TOK], g3[TOK], g4[TOK];
  int s = w.s0;
#pragma unroll
  for (int j = 0; j < TOK; ++j) {
    const float vx = rx[j].f(), vr = rr[j].f(), vi = ri[j].f();
    if constexpr (PACKED) {
      if (w.start >> j & 1) {
        while (g.cuc[s] < t0 + j || g.cuc[s + 1] <= t0 + j) ++s;
        h = g.h0 ? g.h0[static_cast<int64_t>(s) * g.D + chc] : 0.0f;
        P = kReset;
      }
    }
    float a, m2;
    const float sr = sigmoid(vr), si = sigmoid(vi);
    decay_of(k * sr, a, m2);
    const float m = __builtin_amdgcn_sqrtf(m2);
    av[j] = a;
    g1[j] = m;
    g2[j] = sr;
    g3[j] = si;
    g4[j] = vx;
    h = fmaf(a, h, m * (si * vx));
    P *= a;
  }
  sH[wave][lane] = h;
  sP[wave][lane] = P;
  __syncthreads();
  for (int u = 0; u < wave; ++u) entry = join<PACKED>(sP[u][lane], entry, sH[u][lane]);
  __syncthreads();   // sH and sP are written again below

  // forward again, now with h: the factors of g
  s = w.s0;
#pragma unroll
  for (int j = 0; j < TOK; ++j) {
    if constexpr (PACKED) {
      if (w.start >> j & 1) {
        while (g.cuc[s] < t0 + j || g.cuc[s + 1] <= t0 + j) ++s;
        entry = g.h0 ? g.h0[static_cast<int64_t>(s) * g.D + chc] : 0.0f;
      }
    }
    // products of the first pass are formed anew, not kept in registers
    asm volatile("" : "+v"(g1[j]), "+v"(g2[j]), "+v"(g3[j]), "+v"(g4[j]));
    const float a = av[j], m = g1[j], sr = g2[j], si = g3[j];
    const float u = si * g4[j], L = kLn2 * (k * sr), ah = a * entry;
    // L / m where m is 0 (a = 1): the limit 0
    const float lm = m > 0.0f ? L * __builtin_amdgcn_rcpf(m) : 0.0f;
    const float mu = m * u;
    g1[j] = m * si;                                 // dx / g
    g3[j] = fmaf(-mu, si, mu);                      // di / g
    g4[j] = fmaf(ah, L, -(a * a) * (lm * u));      // dL L / g
    g2[j] = 1.0f - sr;
    entry = ah + mu;
  }

  // backward: q from zero and the product of a
  float q = 0.0f;
  P = 1.0f;
  int se = w.s1;   // the sequence of the wave's last row
  if constexpr (PACKED)
    while (se > 0 && g.cuc[se] >= min(t0 + TOK, g.T)) --se;
  int sb = se;
#pragma unroll
  for (int j = TOK - 1; j >= 0; --j) {
    if (j >= nrow) continue;
    if constexpr (PACKED) {
      if (w.end >> j & 1) {
        while (g.cuc[sb] > t0 + j || g.cuc[sb + 1] <= g.cuc[sb]) --sb;
        q = g.dhT ? g.dhT[static_cast<int64_t>(sb) * g.D + chc] : 0.0f;
        P = kReset;
      }
    }
    q = av[j] * (q + rd[j].f());
    P *= av[j];
  }
  sH[wave][lane] = q;
  sP[wave][lane] = P;
  __syncthreads();
  float cH = 0.0f, cP = 1.0f;
  for (int u = WAVES - 1; u > wave; --u) {
    const float p = sP[u][lane];
    cH = join<PACKED>(p, cH, sH[u][lane]);
    cP = join_p<PACKED>(p, cP);
  }
  const Carry cr(g, g.ntile - 1 - tile, chain, lane);
  const float tP = join_p<PACKED>(P, cP), tH = join<PACKED>(P, cH, q);
  if (wave == 0) cr.give(tP, tH);   // the first wave's is the tile's
  cr.fetch(sM, wave, lane);
  float last = 0.0f;
  if (!PACKED && cr.n0 == 0 && g.dhT) last = g.dhT[static_cast<int64_t>(b) * g.D + chc];
  __syncthreads();
  const float after = cr.take<PACKED>(sM, lane, last);
  if (wave == 0) {
    const float q0 = join<PACKED>(tP, after, tH);
    cr.pass_on(q0);
    if (!PACKED && tile == 0 && on && g.dh0) g.dh0[static_cast<int64_t>(b) * g.D + ch] = q0;
  }
  q = join<PACKED>(cP, after, cH);

  // backward again, now with q: the gradients
  float dk = 0.0f;
  const uint32_t off = static_cast<uint32_t>(ch) * static_cast<uint32_t>(sizeof(T));
  const int64_t step = g.ldg * static_cast<int64_t>(sizeof(T));
  const int64_t at = (row0 + t0 + TOK) * step;
  char* dx = static_cast<char*>(g.dx) + at;
  char* dr = static_cast<char*>(g.dr) + at;
  char* di = static_cast<char*>(g.di) + at;
  sb = se;
#pragma unroll
  for (int j = TOK - 1; j >= 0; --j) {
    dx -= step;
    dr -= step;
    di -= step;
    if (j >= nrow) continue;
    if constexpr (PACKED) {
      if (!(w.live >> j & 1)) continue;
      if (w.end >> j & 1) {
        while (g.cuc[sb] > t0 + j || g.cuc[sb + 1] <= g.cuc[sb]) --sb;
        q = g.dhT ? g.dhT[static_cast<int64_t>(sb) * g.D + chc] : 0.0f;
      }
    }
    const float gt = rd[j].f() + q, gl = gt * g4[j];
    dk += gl;
    q = av[j] * gt;
    if (on) {
      put(reinterpret_cast<T*>(dx), off, gt * g1[j]);
      put(reinterpret_cast<T*>(dr), off, gl * g2[j]);
      put(reinterpret_cast<T*>(di), off, gt * g3[j]);
      if (PACKED && (w.start >> j & 1) && g.dh0) g.dh0[static_cast<int64_t>(sb) * g.D + ch] = q;
    }
  }
  // the tile's part of the sum for ddecay, over its waves in order
  sH[wave][lane] = dk;
  __syncthreads();
  if (wave == 0 && on) {
    float acc = 0.0f;
#pragma unroll
    for (int u = 0; u < WAVES; ++u) acc += sH[u][lane];
    g.part[(b * static_cast<int64_t>(g.ntile) + tile) * g.D + ch] = acc;
  }
}

// ddecay = (sum of the tiles' parts) * sigmoid(decay) / softplus(decay), in a
// fixed order: 16 threads of a channel take every 16th part each.
__global__ __launch_bounds__(256) void k_gated_ddecay(GatedArgs g, int64_t nparts) {
  __shared__ float sum[16][17];
  const int cl = threadIdx.x & 15, k = threadIdx.x >> 4;
  const int ch = blockIdx.x * 16 + cl;
  float acc = 0.0f;
  if (ch < g.D)
    for (int64_t p = k; p < nparts; p += 16) acc += g.part[p * g.D + ch];
  sum[k][cl] = acc;
  __syncthreads();
  if (k == 0 && ch < g.D) {
    float v = 0.0f;
#pragma unroll
    for (int j = 0; j < 16; ++j) v += sum[j][cl];
    const float d = g.decay[ch];
    float ratio;
    if (d < -15.0f) {   // softplus(d) -> e^d: the ratio tends to 1
      ratio = 1.0f - 0.5f * expf(d);
    } else {
      const float e = expf(-fabsf(d));
      ratio = (d >= 0.0f ? 1.0f : e) / (1.0f + e) / (fmaxf(d, 0.0f) + log1pf(e));
    }
    g.ddecay[ch] = v * ratio;
  }
}

// ---------------------------------------------------------------------------
// One decode step: h is read and written once (1 x 4096 and 128 x 4096 in 4
// to 7 us: a launch and a round trip to memory).
template <typename T, int V>
__global__ __launch_bounds__(256) void k_gated_step(GatedArgs g, float* hs) {
  const int ncb = (g.D + V - 1) / V;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int b = static_cast<int>(n / ncb), ch = static_cast<int>(n % ncb) * V;
  if (b >= g.B) return;
  RawVec<T, V> rx, rr, ri;
  rr.load(static_cast<const T*>(g.r) + b * g.ldr + ch);
  rx.load(static_cast<const T*>(g.x) + b * g.ldx + ch);
  ri.load(static_cast<const T*>(g.i) + b * g.ldi + ch);
  RawVec<float, V> rh, rk;
  float* hp = hs + static_cast<int64_t>(b) * g.D + ch;
  rh.load(hp);
  rk.load(g.decay + ch);
  float x[V], r[V], i[V], h[V], d[V];
  rr.get(r);
  rx.get(x);
  ri.get(i);
  rh.get(h);
  rk.get(d);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float a, m2;
    decay_of(decay_factor(d[v], g.c) * sigmoid(r[v]), a, m2);
    h[v] = fmaf(a, h[v], __builtin_amdgcn_sqrtf(m2) * (sigmoid(i[v]) * x[v]));
  }
  store_v<float, V>(hp, h);
  store_v<T, V>(static_cast<T*>(g.y) + static_cast<int64_t>(b) * g.D + ch, h);
}

template <typename T, int TOK, int WAVES>
hipError_t run_scan(GatedArgs& g, hipStream_t s) {
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(g.ntile) * g.nchain);
  if (g.cu)
    k_gated_scan<T, TOK, WAVES, true><<<grid, 64 * WAVES, 0, s>>>(g);
  else
    k_gated_scan<T, TOK, WAVES, false><<<grid, 64 * WAVES, 0, s>>>(g);
  return hipGetLastError();
}
// 16 rows a wave just fit 128 registers in the dense bf16 kernel (4 x 2048 x
// 4096: 127 us, with 8 rows and twice the waves 166 us).  Windows of packed
// rows and fp32 inputs do not fit (fp32: 327 us, with 8 rows 199 us; packed
// 8192 x 2048 in bf16 155 and 110 us).  16 waves of 87 registers are one workgroup
// a CU, which waits as a whole at its barriers and for the carry, where the dense
// bf16 kernel has two: 16384 x 2048 in 64 sequences in bf16 204 us, 2.3 TB/s.
template <typename T>
hipError_t run_backward(GatedArgs& g, hipStream_t s) {
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(g.ntile) * g.nchain);
  if (g.cu)
    k_gated_backward<T, 8, kGatedChunk / 8, true><<<grid, 8 * kGatedChunk, 0, s>>>(g);
  else if constexpr (sizeof(T) == 4)
    k_gated_backward<T, 8, kGatedChunk / 8, false><<<grid, 8 * kGatedChunk, 0, s>>>(g);
  else
    k_gated_backward<T, 16, kGatedChunk / 16, false><<<grid, 4 * kGatedChunk, 0, s>>>(g);
  return hipGetLastError();
}

hipError_t run_init(const GatedArgs& g, const float* src, float* dst, int64_t nslot, hipStream_t s) {
  if (g.ntile == 1 && !g.cu) return hipSuccess;
  int64_t blocks = (nslot + 1023) / 1024;
  if (g.cu) {
    const int64_t windows = (static_cast<int64_t>(g.T) + 8191) / 8192, rows = g.S < 256 ? g.S : 256;
    if (blocks < windows) blocks = windows;
    if (blocks < rows) blocks = rows;
    if (g.S > kInitSeqs) k_gated_clean<<<1, 1024, 0, s>>>(g);
  }
  if (blocks > 4096) blocks = 4096;
  if (blocks < 1) blocks = 1;
  k_gated_init<<<static_cast<unsigned>(blocks), 256, 0, s>>>(g, src, dst, nslot);
  return hipGetLastError();
}

constexpr size_t up256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

// Tiles of the scan: 256 rows, or 512 where all workgroups of 256 would be
// resident at once (two a CU).  Then the time is that of a tile and of the
// carry passing on, and fewer, larger tiles take less: 16384 rows of 512
// channels 27 against 31 us, of 4096 channels 162 against 128 us.  (128 rows:
// 35 and 132 us.)
GatedPlan gated_plan(int B, int T, int D, bool packed, bool backward) {
  GatedPlan p;
  p.ncb = (D + 63) / 64;
  p.nchain = static_cast<int64_t>(p.ncb) * (packed ? 1 : B);
  p.tile = backward ? kGatedChunk : 256;
  if (!backward && T > 256 && (static_cast<int64_t>(T) + 255) / 256 * p.nchain <= 512) p.tile = 512;
  p.ntile = (T - 1) / p.tile + 1;
  return p;
}

// a word for every tile's map and for the state after every whole group
static int64_t gated_slots(const GatedPlan& p) {
  return 64 * p.nchain * (p.ntile + p.ntile / kGroup);
}

size_t gated_workspace_bytes(int B, int T, int D, bool packed, bool backward) {
  const GatedPlan p = gated_plan(B, T, D, packed, backward);
  size_t n = 256 + up256(sizeof(int32_t) * (static_cast<size_t>(B) + 1));
  if (packed) n += up256(sizeof(GatedWindow) * ((static_cast<size_t>(T) + 31) / 32));
  n += up256(sizeof(u64) * gated_slots(p));
  if (backward) n += up256(sizeof(float) * D * (packed ? 1 : B) * p.ntile);
  return n;
}

void gated_carve(GatedArgs& g, bool backward, void* ws) {
  const GatedPlan p = gated_plan(g.B, g.T, g.D, g.cu != nullptr, backward);
  g.ncb = p.ncb;
  g.nchain = static_cast<int>(p.nchain);
  g.ntile = p.ntile;
  char* c = static_cast<char*>(ws);
  g.ticket = reinterpret_cast<unsigned*>(c);
  c += 256;
  g.cuc = reinterpret_cast<int32_t*>(c);
  c += up256(sizeof(int32_t) * (static_cast<size_t>(g.B) + 1));
  g.win = reinterpret_cast<GatedWindow*>(c);
  if (g.cu) c += up256(sizeof(GatedWindow) * ((static_cast<size_t>(g.T) + 31) / 32));
  g.slots = reinterpret_cast<u64*>(c);
  c += up256(sizeof(u64) * gated_slots(p));
  g.part = reinterpret_cast<float*>(c);
  g.S = g.B;
}

hipError_t launch_gated_scan(GatedArgs& g, int bf16, hipStream_t s) {
  const GatedPlan p = gated_plan(g.B, g.T, g.D, g.cu != nullptr, false);
  hipError_t e = run_init(g, g.h0, g.hT, gated_slots(p), s);
  if (e != hipSuccess) return e;
  if (p.tile == 512) return bf16 ? run_scan<bf16_t, 32, 16>(g, s) : run_scan<float, 32, 16>(g, s);
  return bf16 ? run_scan<bf16_t, 32, 8>(g, s) : run_scan<float, 32, 8>(g, s);
}

hipError_t launch_gated_backward(GatedArgs& g, int bf16, hipStream_t s) {
  const GatedPlan p = gated_plan(g.B, g.T, g.D, g.cu != nullptr, true);
  hipError_t e = run_init(g, g.dhT, g.dh0, gated_slots(p), s);
  if (e != hipSuccess) return e;
  e = bf16 ? run_backward<bf16_t>(g, s) : run_backward<float>(g, s);
  if (e != hipSuccess) return e;
  const int64_t nparts = static_cast<int64_t>(g.cu ? 1 : g.B) * g.ntile;
  k_gated_ddecay<<<(g.D + 15) / 16, 256, 0, s>>>(g, nparts);
  return hipGetLastError();
}

hipError_t launch_gated_step(const GatedArgs& g, float* h, int bf16, hipStream_t s) {
  const bool wide = g.D % 8 == 0 && g.ldx % 8 == 0 && g.ldr % 8 == 0 && g.ldi % 8 == 0;
  const int64_t n = static_cast<int64_t>(g.B) * (wide ? g.D / 8 : g.D);
  const unsigned grid = static_cast<unsigned>((n + 255) / 256);
  if (bf16) {
    if (wide) k_gated_step<bf16_t, 8><<<grid, 256, 0, s>>>(g, h);
    else k_gated_step<bf16_t, 1><<<grid, 256, 0, s>>>(g, h);
  } else {
    if (wide) k_gated_step<float, 8><<<grid, 256, 0, s>>>(g, h);
    else k_gated_step<float, 1><<<grid, 256, 0, s>>>(g, h);
  }
  return hipGetLastError();
}

}  // namespace m3
