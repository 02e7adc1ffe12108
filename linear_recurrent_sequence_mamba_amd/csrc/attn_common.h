// attn_common.h -- tiles and matrix-core fragments of the attention kernels
// (gfx950).  Not part of the public ABI.
//
// Everything is built from 32x32 tiles.  A fragment holds, for row (or
// column) lane % 32, eight of sixteen k slots: slots 8 (lane / 32) + j.  bf16
// fragments feed one v_mfma_f32_32x32x16_bf16, fp32 ones eight
// v_mfma_f32_32x32x2_f32.  A result holds column lane % 32 and, in element i,
// row 8 (i / 4) + 4 (lane / 32) + i % 4; so elements 8 s .. 8 s + 7 are the B
// operand of a product over those rows, if the A operand takes its k slots in
// the order 16 s + 4 (lane / 32) + {0..3}, 16 s + 8 + 4 (lane / 32) + {0..3}:
// the softmax's result goes on to the next product without leaving its lanes.
#pragma once

#include "attn.h"
#include "m3_device.h"

namespace m3 {
namespace {

typedef float f16v __attribute__((ext_vector_type(16)));
typedef short s4v __attribute__((ext_vector_type(4)));
typedef short s8v __attribute__((ext_vector_type(8)));
#define M3_LDS __attribute__((address_space(3)))
#define M3_GLB __attribute__((address_space(1)))

template <typename T>
struct Frag;
template <>
struct Frag<bf16_t> {
  bh8 v;
};
template <>
struct Frag<float> {
  f4 a, b;
};

__device__ __forceinline__ f16v mma(const Frag<bf16_t>& a, const Frag<bf16_t>& b, f16v c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.v, b.v, c, 0, 0, 0);
}
__device__ __forceinline__ f16v mma(const Frag<float>& a, const Frag<float>& b, f16v c) {
#pragma unroll
  for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a.a[j], b.a[j], c, 0, 0, 0);
#pragma unroll
  for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a.b[j], b.b[j], c, 0, 0, 0);
  return c;
}

// eight consecutive elements of a row in memory
__device__ __forceinline__ void frag_load(Frag<bf16_t>& f, const bf16_t* p) {
  f.v = *reinterpret_cast<const bh8*>(p);
}
__device__ __forceinline__ void frag_load(Frag<float>& f, const float* p) {
  f.a = *reinterpret_cast<const f4*>(p);
  f.b = *reinterpret_cast<const f4*>(p + 4);
}
// sum + <a, b> over a lane's eight elements
__device__ __forceinline__ float frag_dot(const Frag<bf16_t>& a, const Frag<bf16_t>& b, float sum) {
#pragma unroll
  for (int j = 0; j < 8; ++j) sum = fmaf(static_cast<float>(a.v[j]), static_cast<float>(b.v[j]), sum);
  return sum;
}
__device__ __forceinline__ float frag_dot(const Frag<float>& a, const Frag<float>& b, float sum) {
#pragma unroll
  for (int j = 0; j < 4; ++j) sum = fmaf(a.a[j], b.a[j], fmaf(a.b[j], b.b[j], sum));
  return sum;
}
// elements 8 s .. 8 s + 7 of a result (bf16: rounded to nearest, off by at
// most 2^-8 of each weight before products that are summed in fp32)
__device__ __forceinline__ void frag_from(Frag<bf16_t>& f, const float* v) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const bh2 p = __builtin_convertvector(f2{v[2 * j], v[2 * j + 1]}, bh2);
    f.v[2 * j] = p[0];
    f.v[2 * j + 1] = p[1];
  }
}
__device__ __forceinline__ void frag_from(Frag<float>& f, const float* v) {
  f.a = f4{v[0], v[1], v[2], v[3]};
  f.b = f4{v[4], v[5], v[6], v[7]};
}

// row of element i of a result tile
__device__ __forceinline__ int row_of(int i, int half) { return 8 * (i >> 2) + 4 * half + (i & 3); }

// The same number, but what is derived from it in a rarely taken branch is not
// computed ahead of a loop and kept in registers there.
__device__ __forceinline__ int opaque(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// 64 rows of D elements in LDS (or twice 32 from two arrays).  Rows arrive by
// loads that go straight to LDS, where a wave's 64 lanes fill 1024 consecutive
// bytes; which rows those are, and where the 1024 bytes lie, is free.  Both
// are chosen so that neither sixteen rows' reads of one 16-byte chunk (frag)
// nor four rows' reads of 64 bytes (frag_t) meet in a bank: row r lies at
// 64 (r % 4) + 16 (r / 4 % 4) modulo the 256 bytes of all banks.  And since a
// row's place is a sum of terms of its index, every fragment is one lane
// address plus a constant (a permutation by exclusive or, as bank-free, costs
// an instruction for each fragment).
template <typename T, int D>
struct Tile {
  static constexpr int RB = D * sizeof(T);     // bytes of a row: 128, 256 or 512
  static constexpr int RPI = 1024 / RB;        // rows of one load instruction
  static constexpr int CPR = RB / 16;          // chunks of a row
  static constexpr int NG = 64 / RPI;          // load instructions of a tile
  static constexpr int EPC = 16 / sizeof(T);
  static constexpr int G1 = 1088;              // 64 bytes on
  static constexpr int G4 = RB == 128 ? 2320 : 4368;   // 16 bytes on
  static constexpr int HALF = 4 * 4368;        // 512-byte rows: from row 32 on
  static constexpr int BYTES = RB == 128 ? 4 * 2320 : RB == 256 ? 4 * 4368 : 2 * HALF;

  // load instruction g: where its bytes go, and its row beyond the lane's
  static __device__ __forceinline__ constexpr int place(int g) {
    return RB == 128 ? (g >> 1) * G4 + (g & 1) * G1
                     : (g >> 4) * HALF + ((g >> 2) & 3) * G4 + (g & 3) * G1;
  }
  static __device__ __forceinline__ constexpr int group_row(int g) {
    return RB == 128 ? 4 * (g >> 1) + 2 * (g & 1) : (g & 15) + 32 * (g >> 4);
  }
  static __device__ __forceinline__ int lane_row(int lane) {
    const int j = lane / CPR;
    return RB == 128 ? (j & 1) + 16 * (j >> 1) : 16 * j;
  }

  // Rows row0 .. row0 + 63 of p (rows ld elements apart), row indices clamped
  // to last; by NW waves, of which this is wave w.  A whole tile takes one
  // 32-bit lane offset (64 rows of less than 2^24 elements) and uniform bases.
  template <int NW>
  static __device__ __forceinline__ void load(char* lds, const T* p, int64_t ld, int row0, int last,
                                              int w, int lane) {
    if (row0 + 63 <= last) {
      const uint32_t off = static_cast<uint32_t>(lane_row(lane)) * static_cast<uint32_t>(ld) *
                               static_cast<uint32_t>(sizeof(T)) + 16 * (lane % CPR);
      const char* base = reinterpret_cast<const char*>(p + row0 * ld);
#pragma unroll
      for (int n = 0; n < NG / NW; ++n) {
        const int g = n * NW + w;
        __builtin_amdgcn_global_load_lds(
            (const M3_GLB void*)(base + group_row(g) * ld * static_cast<int64_t>(sizeof(T)) + off),
            (M3_LDS void*)(lds + place(g)), 16, 0, 0);
      }
    } else {
      lane = opaque(lane);
#pragma unroll
      for (int n = 0; n < NG / NW; ++n) {
        const int g = n * NW + w;
        const T* src = p + static_cast<int64_t>(min(row0 + group_row(g) + lane_row(lane), last)) * ld +
                       EPC * (lane % CPR);
        __builtin_amdgcn_global_load_lds((const M3_GLB void*)src, (M3_LDS void*)(lds + place(g)), 16, 0, 0);
      }
    }
  }
  // Rows row0 .. row0 + 31 of a as rows 0 .. 31 and of b as rows 32 .. 63
  template <int NW>
  static __device__ __forceinline__ void load2(char* lds, const T* a, int64_t lda, const T* b,
                                               int64_t ldb, int row0, int last, int w, int lane) {
    const int lr = lane_row(lane);
#pragma unroll
    for (int n = 0; n < NG / NW; ++n) {
      const int g = n * NW + w, r = group_row(g) + lr;
      const bool second = r >= 32;
      const int64_t row = min(row0 + (second ? r - 32 : r), last);
      const T* src = (second ? b + row * ldb : a + row * lda) + EPC * (lane % CPR);
      __builtin_amdgcn_global_load_lds((const M3_GLB void*)src, (M3_LDS void*)(lds + place(g)), 16, 0, 0);
    }
  }

  // The same for a loop over tiles: a lane's first row in a or b, and the bytes
  // to the next one.  A tile that is whole then takes one product and a few
  // additions instead of a clamp and two products for each load.
  struct Pair {
    const char* at;
    uint32_t ld;
  };
  static __device__ __forceinline__ Pair pair(const T* a, int64_t lda, const T* b, int64_t ldb, int w,
                                              int lane) {
    const int r = group_row(w) + lane_row(lane);
    const bool second = r >= 32;
    const int64_t ld = second ? ldb : lda;
    return Pair{reinterpret_cast<const char*>((second ? b : a) + (r & 31) * ld + EPC * (lane % CPR)),
                static_cast<uint32_t>(ld) * static_cast<uint32_t>(sizeof(T))};
  }
  // `by` elements beyond a and b
  template <int NW>
  static __device__ __forceinline__ void load2(char* lds, const Pair& p, const T* a, int64_t lda,
                                               const T* b, int64_t ldb, int64_t by, int row0, int last,
                                               int w, int lane) {
    if (RB == 512 || row0 + 31 > last) {   // (512: a and b are in loads of their own)
      load2<NW>(lds, a + by, lda, b + by, ldb, row0, last, w, opaque(lane));
      return;
    }
    // (opaque: one address now, not one for each load kept over the loop)
    const char* src = p.at + by * static_cast<int64_t>(sizeof(T)) +
                      static_cast<uint64_t>(static_cast<uint32_t>(opaque(row0))) * p.ld;
#pragma unroll
    for (int n = 0; n < NG / NW; ++n)
      __builtin_amdgcn_global_load_lds(
          (const M3_GLB void*)(src + static_cast<uint64_t>(p.ld) * group_row(n * NW)),
          (M3_LDS void*)(lds + place(n * NW + w)), 16, 0, 0);
  }

  // fragment kk (elements 16 kk ..) of rows row0 + lane % 32 (row0 0 or 32)
  static __device__ __forceinline__ Frag<T> frag(const char* lds, int row0, int kk, int lane) {
    const int r = lane & 31, h = lane >> 5;
    int at = static_cast<int>(sizeof(T)) * (8 * h + 16 * kk);
    if constexpr (RB == 128)
      at += ((r >> 2) & 3) * G4 + ((r >> 1) & 1) * G1 + ((r & 1) + 2 * (r >> 4)) * RB + 4 * RB * (row0 / 32);
    else
      at += ((r >> 2) & 3) * G4 + (r & 3) * G1 + (r >> 4) * RB + (RB == 256 ? 2 * RB : HALF) * (row0 / 32);
    const char* a = lds + at;
    Frag<T> f;
    if constexpr (sizeof(T) == 2) {
      f.v = *reinterpret_cast<const bh8*>(a);
    } else {
      f.a = *reinterpret_cast<const f4*>(a);
      f.b = *reinterpret_cast<const f4*>(a + 16);
    }
    return f;
  }
  // the transposed fragment: column d0 + lane % 32, k slots = rows
  // row0 + 4 h + {0..3}, row0 + 8 + 4 h + {0..3} (row0 a multiple of 16)
  static __device__ __forceinline__ Frag<T> frag_t(const char* lds, int row0, int d0, int lane) {
    const int h = lane >> 5, q = row0 / 16;
    const int far = RB == 128 ? q * 2 * RB : RB == 256 ? q * RB : (q & 1) * RB + (q >> 1) * HALF;
    Frag<T> f;
    if constexpr (sizeof(T) == 2) {
      // a transposing read: sixteen lanes point at four rows of sixteen
      // elements, each lane at four; lane i receives column i of the four
      const int i = lane & 15, c = i >> 2;
      const int at = h * G4 + (RB == 128 ? (c >> 1) * G1 + (c & 1) * RB : c * G1) +
                     32 * ((lane >> 4) & 1) + 8 * (i & 3) + far + 2 * d0;
      const char* a = lds + at;
      const s4v x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((M3_LDS s4v*)a);
      const s4v y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((M3_LDS s4v*)(a + 2 * G4));
      f.v = __builtin_bit_cast(bh8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      const int at = h * G4 + far + 4 * (d0 + (lane & 31));
      const char* a = lds + at;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f.a[j] = *reinterpret_cast<const float*>(a + j * G1);
        f.b[j] = *reinterpret_cast<const float*>(a + 2 * G4 + j * G1);
      }
    }
    return f;
  }
};

// the loads to LDS that this wave has issued are there
__device__ __forceinline__ void lds_loads_done() {
  __builtin_amdgcn_s_waitcnt(0x0f70);   // vmcnt(0)
}
// ... but for the last N of them
template <int N>
__device__ __forceinline__ void lds_loads_but() {
  static_assert(N < 16, "the low bits of the count");
  __builtin_amdgcn_s_waitcnt(0x0f70 | N);
}

// A barrier behind which the tiles are read that every wave has waited for by
// lds_loads_but, while later ones are still on their way (__syncthreads would
// wait for those, too): this wave's reads of LDS are done, and nothing moves
// over it.
__device__ __forceinline__ void tiles_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xc07f);   // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
// this wave's reads of LDS are done
__device__ __forceinline__ void lds_reads_done() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xc07f);
  asm volatile("" ::: "memory");
}

// Sequence and tile of a slot.  A sequence's tiles of B rows take the slots
// from cu[s] / B + s on: the next sequence's first slot is never before the
// last of them, and T / B + S slots hold every split of T rows into S
// sequences.  Offsets are clamped into [0, T], so whatever they hold, no row
// outside [0, T) is touched.
struct Slot {
  int s, tile;   // s = -1: none
};
__device__ __forceinline__ int clamp_row(int v, int T) { return max(0, min(v, T)); }
// (B = 1 << lb)
__device__ __forceinline__ Slot slot_of(const int32_t* cu, int S, int T, int lb, int slot, int lane) {
  int lo = 0, n = S;
  for (;;) {
    const int step = (n + 63) / 64;
    const int s = lo + lane * step;
    const bool le = s < lo + n && (clamp_row(cu[s < S ? s : S - 1], T) >> lb) + s <= slot;
    const int cnt = __popcll(__ballot(le));
    if (cnt == 0) return Slot{-1, 0};
    const int at = lo + (cnt - 1) * step;
    n = min(step, lo + n - at);
    lo = at;
    if (step == 1) break;
  }
  lo = __builtin_amdgcn_readfirstlane(lo);
  const int tile = slot - ((clamp_row(cu[lo], T) >> lb) + lo);
  return tile < 0 ? Slot{-1, 0} : Slot{lo, tile};
}

// The same for up to 64 sequences, in the order of the tiles' work, the largest
// first: a batch of few, uneven sequences then ends at once on all CUs.  A lane
// has a sequence of n tiles whose work grows by one from `a` on; the level at
// which the rank lies is found by bisection between 0 and `top`.  (Counts are
// below 2^24, so sums of floats are exact.)  `tile` is counted from the least
// work.
struct Ranked {
  int n, a;
  __device__ __forceinline__ Ranked(const int32_t* cu, int S, int T, int lb, int lane) : n(0), a(0) {
    if (lane < S)
      n = (max(0, clamp_row(cu[lane + 1], T) - clamp_row(cu[lane], T)) + (1 << lb) - 1) >> lb;
  }
  __device__ __forceinline__ int count(int x) const {   // tiles of level x and more
    return __builtin_amdgcn_readfirstlane(
        static_cast<int>(group_sum<64>(static_cast<float>(max(0, min(a + n - x, n))))));
  }
  __device__ __forceinline__ Slot at(int rank, int top, int lane) const {
    if (rank >= count(0)) return Slot{-1, 0};
    int lo = 0, hi = top;   // count(lo) > rank >= count(hi)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (count(mid) > rank) lo = mid; else hi = mid;
    }
    const int nth = rank - count(hi);   // by all lanes: not behind a condition
    const bool has = lo >= a && lo < a + n;
    const uint64_t mask = __ballot(has);
    const int before = __popcll(mask & ((uint64_t{1} << lane) - 1));
    const uint64_t one = __ballot(has && before == nth);
    if (one == 0) return Slot{-1, 0};
    const int s = __builtin_ctzll(one);
    return Slot{s, lo - __builtin_amdgcn_readlane(a, s)};
  }
};

// Whether workgroups are taken in the order of their work: where a wave has a
// lane for each sequence.  dk and dv always gain (8 sequences of 2048, 16 heads
// of 128 on 2: all gradients 802 -> 702 us).  The queries' tiles gain where the
// last workgroups weigh most, up to about four a CU (8192 rows in 3 uneven
// sequences, 16 heads of 128: 131 -> 122 us; 4 of 2048: 97 -> 85; but 32 of 256:
// 39 -> 43); with more of them several sequences' keys share the caches for
// nothing (8 of 2048, 32 heads of 64: 200 us, ranked 215).
__device__ __forceinline__ bool by_work(const AttnArgs& a) { return a.S > 1 && a.S <= kRankedSeqs; }

// the n-th tile of 1 << lb queries to start, of nslot
__device__ __forceinline__ Slot query_slot(const AttnArgs& a, int lb, int n, int nslot, int lane) {
  if (!by_work(a) || gridDim.x > kRankedWorkgroups) return slot_of(a.cuq, a.S, a.Tq, lb, nslot - 1 - n, lane);
  Ranked r(a.cuq, a.S, a.Tq, lb, lane);
  if (lane < a.S) {   // tiles of keys before the first query's own
    const int lk = clamp_row(a.cuk[lane + 1], a.Tk) - clamp_row(a.cuk[lane], a.Tk);
    const int lq = clamp_row(a.cuq[lane + 1], a.Tq) - clamp_row(a.cuq[lane], a.Tq);
    r.a = max(0, lk - lq) >> lb;
  }
  return r.at(n, (max(a.Tq, a.Tk) >> lb) + 3, lane);
}
// the n-th tile of 1 << lb keys to start: the first keys are seen by most queries
__device__ __forceinline__ Slot key_slot(const AttnArgs& a, int lb, int n, int lane) {
  if (!by_work(a)) return slot_of(a.cuk, a.S, a.Tk, lb, n, lane);
  const Ranked r(a.cuk, a.S, a.Tk, lb, lane);
  Slot s = r.at(n, (a.Tk >> lb) + 3, lane);
  if (s.s >= 0) s.tile = __builtin_amdgcn_readlane(r.n, s.s) - 1 - s.tile;
  return s;
}

// The (query, head) pairs of a workgroup's 128 columns: 128 >> lp queries of
// 1 << lp heads that share k and v.  So fewer keys are loaded for queries that do
// not see them, and short sequences fill a tile (packed rows of 32 heads of 64 on
// 8: 240 us, one head a tile 249; 1000 sequences of 16, 16 heads of 128 on 4: 71
// and 194).
struct Columns {
  int lp, queries, nslot, group, hk;   // queries of a workgroup; groups of heads, the own k and v
  __device__ __forceinline__ explicit Columns(const AttnArgs& a) : lp(a.lp), queries(128 >> a.lp) {
    const int ngroup = a.Hq >> lp;
    nslot = gridDim.x / ngroup;
    group = blockIdx.x % ngroup;
    hk = (group << lp) / (a.Hq / a.Hk);
  }
  __device__ __forceinline__ Slot slot(const AttnArgs& a, int lane) const {
    return query_slot(a, 7 - lp, static_cast<int>(blockIdx.x / (a.Hq >> lp)), nslot, lane);
  }
  __device__ __forceinline__ int first(int wave) const { return wave * (32 >> lp); }   // query of a wave
  __device__ __forceinline__ int per_wave() const { return 32 >> lp; }
  __device__ __forceinline__ int query(int lane) const { return (lane & 31) >> lp; }
  __device__ __forceinline__ int head(int lane) const {
    return (group << lp) + (lane & ((1 << lp) - 1));
  }
};

// maximum and sum of lanes l and l ^ 32, in both.  The swap exchanges the
// upper half of its first operand with the lower half of its second.
__device__ __forceinline__ float half_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// four consecutive elements of an output row
__device__ __forceinline__ void put4(float* p, float a, float b, float c, float d) {
  *reinterpret_cast<f4*>(p) = f4{a, b, c, d};
}
__device__ __forceinline__ void put4(bf16_t* p, float a, float b, float c, float d) {
  const bh2 x = __builtin_convertvector(f2{a, b}, bh2), y = __builtin_convertvector(f2{c, d}, bh2);
  *reinterpret_cast<uint2*>(p) =
      uint2{__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, y)};
}

constexpr float kLog2eA = 1.4426950408889634f;
constexpr float kLn2A = 0.6931471805599453f;

}  // namespace
}  // namespace m3
