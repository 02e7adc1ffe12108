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

// A tile of rows of D elements in LDS.  A row is CPR 16-byte chunks; chunk c
// of row r lies at position c ^ swz(r), so that neither sixteen rows' reads
// of one chunk (frag) nor four rows' reads of four chunks (frag_t) meet in a
// bank.  Rows arrive by loads that go straight to LDS: a wave's 64 lanes fill
// 64 consecutive positions, and the permutation is in the address each lane
// reads from.
template <typename T, int D>
struct Tile {
  static constexpr int EPC = 16 / sizeof(T);
  static constexpr int CPR = D / EPC;
  static constexpr int ROW = D;   // elements
  static __device__ __forceinline__ int swz(int r) {
    if constexpr (CPR == 8) return ((r >> 1) & 1) << 2 | ((r >> 2) & 3);
    return (r & 3) << 2 | ((r >> 2) & 3);
  }
  // Rows row0 .. row0 + ROWS of p (rows ld elements apart), row indices
  // clamped to last; by NW waves, of which this is wave w.  The rows of one
  // instruction are a multiple of 16 from those of the next, so their swizzle
  // is the same: a whole tile takes one 32-bit lane offset (64 rows of less
  // than 2^24 elements) and uniform bases.
  template <int ROWS, int NW>
  static __device__ __forceinline__ void load(T* lds, const T* p, int64_t ld, int row0, int last,
                                              int w, int lane) {
    static_assert(ROWS * CPR % (64 * NW) == 0, "whole waves");
    constexpr int N = ROWS * CPR / (64 * NW), STEP = 64 * NW / CPR;
    const int r0 = (w * 64 + lane) / CPR, c0 = ((w * 64 + lane) % CPR) ^ swz(r0);
    if (STEP % 16 == 0 && row0 + ROWS - 1 <= last) {
      const uint32_t off = (static_cast<uint32_t>(r0) * static_cast<uint32_t>(ld) + c0 * EPC) * sizeof(T);
      const char* base = reinterpret_cast<const char*>(p + row0 * ld);
#pragma unroll
      for (int n = 0; n < N; ++n) {
        __builtin_amdgcn_global_load_lds((const M3_GLB void*)(base + off),
                                         (M3_LDS void*)(lds + (n * NW + w) * 64 * EPC), 16, 0, 0);
        base += STEP * ld * static_cast<int64_t>(sizeof(T));
      }
    } else {
      lane = opaque(lane);
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int pos = (n * NW + w) * 64 + lane, r = pos / CPR, c = (pos % CPR) ^ swz(r);
        const T* src = p + static_cast<int64_t>(min(row0 + r, last)) * ld + c * EPC;
        __builtin_amdgcn_global_load_lds((const M3_GLB void*)src,
                                         (M3_LDS void*)(lds + (n * NW + w) * 64 * EPC), 16, 0, 0);
      }
    }
  }
  // fragment kk (elements 16 kk ..) of rows row0 + lane % 32
  static __device__ __forceinline__ Frag<T> frag(const T* lds, int row0, int kk, int lane) {
    const int r = row0 + (lane & 31), h = lane >> 5;
    Frag<T> f;
    if constexpr (sizeof(T) == 2) {
      f.v = *reinterpret_cast<const bh8*>(lds + r * ROW + (((2 * kk + h) ^ swz(r)) * EPC));
    } else {
      f.a = *reinterpret_cast<const f4*>(lds + r * ROW + (((4 * kk + 2 * h) ^ swz(r)) * EPC));
      f.b = *reinterpret_cast<const f4*>(lds + r * ROW + (((4 * kk + 2 * h + 1) ^ swz(r)) * EPC));
    }
    return f;
  }
  // the transposed fragment: column d0 + lane % 32, k slots = rows
  // row0 + 4 h + {0..3}, row0 + 8 + 4 h + {0..3}
  static __device__ __forceinline__ Frag<T> frag_t(const T* lds, int row0, int d0, int lane) {
    const int h = lane >> 5;
    Frag<T> f;
    if constexpr (sizeof(T) == 2) {
      // a transposing read: sixteen lanes point at four rows of sixteen
      // elements, each lane at four; lane i receives column i of the four
      const int i = lane & 15;
      const int c = (d0 >> 3) + 2 * ((lane >> 4) & 1) + ((i & 3) >> 1);
      s4v x[2];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int r = row0 + 8 * n + 4 * h + (i >> 2);
        const T* a = lds + r * ROW + ((c ^ swz(r)) * EPC) + (i & 1) * 4;
        x[n] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((M3_LDS s4v*)a);
      }
      const s8v y = __builtin_shufflevector(x[0], x[1], 0, 1, 2, 3, 4, 5, 6, 7);
      f.v = __builtin_bit_cast(bh8, y);
    } else {
      const int d = d0 + (lane & 31), c = d / EPC, e = d % EPC;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = row0 + 4 * h + j, r2 = r + 8;
        f.a[j] = lds[r * ROW + ((c ^ swz(r)) * EPC) + e];
        f.b[j] = lds[r2 * ROW + ((c ^ swz(r2)) * EPC) + e];
      }
    }
    return f;
  }
  // one element
  static __device__ __forceinline__ float at(const T* lds, int r, int d) {
    return to_f32(lds[r * ROW + (((d / EPC) ^ swz(r)) * EPC) + d % EPC]);
  }
};

// the loads to LDS that this wave has issued are there
__device__ __forceinline__ void lds_loads_done() {
  __builtin_amdgcn_s_waitcnt(0x0f70);   // vmcnt(0)
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
template <int B>
__device__ __forceinline__ Slot slot_of(const int32_t* cu, int S, int T, int slot, int lane) {
  int lo = 0, n = S;
  for (;;) {
    const int step = (n + 63) / 64;
    const int s = lo + lane * step;
    const bool le = s < lo + n && clamp_row(cu[s < S ? s : S - 1], T) / B + s <= slot;
    const int cnt = __popcll(__ballot(le));
    if (cnt == 0) return Slot{-1, 0};
    const int at = lo + (cnt - 1) * step;
    n = min(step, lo + n - at);
    lo = at;
    if (step == 1) break;
  }
  lo = __builtin_amdgcn_readfirstlane(lo);
  const int tile = slot - (clamp_row(cu[lo], T) / B + lo);
  return tile < 0 ? Slot{-1, 0} : Slot{lo, tile};
}

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
