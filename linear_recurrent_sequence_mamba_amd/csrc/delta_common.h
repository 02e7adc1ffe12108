// delta_common.h -- chunks, tiles and matrix-core operands of the gated delta
// rule (gfx950).  Not part of the public ABI.
//
// Operands.  Everything runs on v_mfma_f32_16x16x32_bf16.  A number in fp32 is
// a sum of bf16 parts, each the rounding of what the ones before it leave:
// three keep all 24 bits, two 16.  A product takes the pairs of parts (a, b)
// with a + b below the number of parts that are asked for.  Inputs in bf16 are
// one exact part.
//
// A result holds column lane % 16 and rows 4 (lane / 16) + {0..3} of a 16x16
// tile.  Two tiles below each other are the B operand of a product over their
// 32 rows if the A operand takes its k slots 8 g + j in the order
// 16 (j / 4) + 4 g + j % 4 (g = lane / 16): results go on to the next product
// without leaving their lanes, and a wave that holds some columns of the state
// never needs another wave's.
#pragma once

#include "delta.h"
#include "attn_common.h"

namespace m3 {
namespace {

template <int NP>
struct Parts {
  bh8 p[NP];
};

// eight floats as NP parts
template <int NP>
__device__ __forceinline__ void split8(Parts<NP>& f, const float* v) {
  float r[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) r[j] = v[j];
#pragma unroll
  for (int n = 0; n < NP; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bh2 h = __builtin_convertvector(f2{r[2 * j], r[2 * j + 1]}, bh2);
      f.p[n][2 * j] = h[0];
      f.p[n][2 * j + 1] = h[1];
      if (n + 1 < NP) {
        r[2 * j] -= static_cast<float>(h[0]);
        r[2 * j + 1] -= static_cast<float>(h[1]);
      }
    }
}
// two tiles of a result below each other
template <int NP>
__device__ __forceinline__ void split_d(Parts<NP>& f, f4 a, f4 b) {
  const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  split8<NP>(f, v);
}

// c + a b, of the products of parts (i, j) with i + j < N
template <int N, int NA, int NB>
__device__ __forceinline__ f4 mmp(const Parts<NA>& a, const Parts<NB>& b, f4 c) {
#pragma unroll
  for (int i = 0; i < NA; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
      if (i + j < N) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[i], b.p[j], c, 0, 0, 0);
  return c;
}

// 64 rows of C bf16 in LDS, one plane for each part.  Row r starts at
// r (2 C + 32) + 16 (r / 8) bytes, which is 32 (r % 8) + 16 (r / 8 % 2) modulo
// the 256 bytes of all banks: sixteen rows' reads of 8 bytes and eight rows'
// transposing reads of 32 bytes both fall on different banks.
template <int C>
struct Rows64 {
  static constexpr int ST = 2 * C + 32;
  static constexpr int PLANE = 64 * ST + 128;
  static __device__ __forceinline__ int at(int r, int c) { return r * ST + 16 * (r >> 3) + 2 * c; }

  // rows r, columns c .. c + 7 (c a multiple of 8)
  template <int NP>
  static __device__ __forceinline__ void put(char* lds, int r, int c, const float* v) {
    Parts<NP> f;
    split8<NP>(f, v);
#pragma unroll
    for (int n = 0; n < NP; ++n) *reinterpret_cast<bh8*>(lds + n * PLANE + at(r, c)) = f.p[n];
  }
  // operand with row (column) r0 + lane % 16 and k = columns c0 .. c0 + 31
  template <int NP>
  static __device__ __forceinline__ Parts<NP> by_row(const char* lds, int r0, int c0, int lane) {
    const char* a = lds + at(lane & 15, 4 * (lane >> 4)) + r0 * ST + 16 * (r0 >> 3) + 2 * c0;
    Parts<NP> f;
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      const uint2 x = *reinterpret_cast<const uint2*>(a + n * PLANE);
      const uint2 y = *reinterpret_cast<const uint2*>(a + n * PLANE + 32);
      f.p[n] = __builtin_bit_cast(bh8, uint4{x.x, x.y, y.x, y.y});
    }
    return f;
  }
  // operand with row (column) c0 + lane % 16 and k = rows r0 .. r0 + 31
  // (transposing reads: sixteen lanes point at four rows of sixteen elements,
  // four each, and lane i receives column i)
  template <int NP>
  static __device__ __forceinline__ Parts<NP> by_col(const char* lds, int r0, int c0, int lane) {
    const int i = lane & 15;
    const char* a = lds + at(4 * (lane >> 4) + (i >> 2), 4 * (i & 3)) + r0 * ST + 16 * (r0 >> 3) + 2 * c0;
    Parts<NP> f;
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      const s4v x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((M3_LDS s4v*)(a + n * PLANE));
      const s4v y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((M3_LDS s4v*)(a + n * PLANE + 16 * ST + 32));
      f.p[n] = __builtin_bit_cast(bh8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
    }
    return f;
  }
};

// A 64x64 matrix that holds two triangles: T strictly below the diagonal (its
// diagonal is 1) and P, transposed, on and above it.  An operand of one of them
// keeps its own side of the diagonal's tiles: masks for the lane's elements of
// such a tile.
struct Triangle {
  uint32_t low[2];    // by_row: columns before the lane's row
  uint32_t upto[2];   // by_col: rows up to the lane's column
  __device__ __forceinline__ explicit Triangle(int lane) {
    const int r = lane & 15, g = lane >> 4;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      low[p] = (4 * g + 2 * p < r ? 0xffffu : 0u) | (4 * g + 2 * p + 1 < r ? 0xffff0000u : 0u);
      upto[p] = (4 * g + 2 * p <= r ? 0xffffu : 0u) | (4 * g + 2 * p + 1 <= r ? 0xffff0000u : 0u);
    }
  }
  // the tile of the diagonal is the first (FIRST) or the second of the operand's
  // two; behind a first one nothing is left
  template <bool FIRST, int NP>
  static __device__ __forceinline__ void keep(Parts<NP>& f, const uint32_t* m) {
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      uint4 u = __builtin_bit_cast(uint4, f.p[n]);
      if (FIRST) {
        u.x &= m[0];
        u.y &= m[1];
        u.z = u.w = 0u;
      } else {
        u.z &= m[0];
        u.w &= m[1];
      }
      f.p[n] = __builtin_bit_cast(bh8, u);
    }
  }
  // rows 16 it .. of T, columns 32 s .. (s <= it / 2)
  template <int NP>
  __device__ __forceinline__ Parts<NP> t(const char* lds, int it, int s, int lane) const {
    Parts<NP> f = Rows64<64>::by_row<NP>(lds, 16 * it, 32 * s, lane);
    if (s == it / 2) {
      if (it & 1) keep<false, NP>(f, low);
      else keep<true, NP>(f, low);
    }
    return f;
  }
  // rows 16 it .. of P, columns 32 s ..
  template <int NP>
  __device__ __forceinline__ Parts<NP> p(const char* lds, int it, int s, int lane) const {
    Parts<NP> f = Rows64<64>::by_col<NP>(lds, 32 * s, 16 * it, lane);
    if (s == it / 2) {
      if (it & 1) keep<false, NP>(f, upto);
      else keep<true, NP>(f, upto);
    }
    return f;
  }
};

// parts of an input in T, and of a computed operand that only reaches outputs in T
template <typename T>
struct DeltaParts {
  static constexpr int IN = sizeof(T) == 2 ? 1 : 3;
  static constexpr int OUT = sizeof(T) == 2 ? 2 : 3;
};

// the rows of a sequence and its first slot
struct DeltaSeq {
  int64_t row0;
  int len, slot0;
  __device__ __forceinline__ DeltaSeq(const DeltaArgs& a, int s) {
    if (a.cu) {
      const int b = clamp_row(a.cu[s], a.T), e = clamp_row(a.cu[s + 1], a.T);
      row0 = b;
      len = max(0, e - b);
      slot0 = b / kDeltaChunk + s;
    } else {
      row0 = static_cast<int64_t>(s) * a.T;
      len = a.T;
      slot0 = s * ((a.T + kDeltaChunk - 1) / kDeltaChunk);
    }
  }
};
// the rows of a chunk; n = 0: the slot has none
struct DeltaSlot {
  int64_t row0;
  int n;
  __device__ __forceinline__ DeltaSlot(const DeltaArgs& a, int slot, int lane) {
    if (a.cu) {
      const Slot x = slot_of(a.cu, a.B, a.T, 6, slot, lane);
      n = 0;
      if (x.s < 0) return;
      const int b = clamp_row(a.cu[x.s], a.T), e = clamp_row(a.cu[x.s + 1], a.T);
      row0 = b + static_cast<int64_t>(x.tile) * kDeltaChunk;
      n = static_cast<int>(max(int64_t{0}, min(int64_t{kDeltaChunk}, e - row0)));
    } else {
      const int nch = (a.T + kDeltaChunk - 1) / kDeltaChunk, s = slot / nch, c = slot - s * nch;
      row0 = static_cast<int64_t>(s) * a.T + c * kDeltaChunk;
      n = min(kDeltaChunk, a.T - c * kDeltaChunk);
    }
  }
};

// 64 rows of C elements on their way to LDS through the registers of NT
// threads; rows from n on are zeros
template <typename T, int C, int NT>
struct Stage {
  static constexpr int N = 64 * C / 8 / NT;
  Vec8<T> v[N];
  __device__ __forceinline__ void load(const T* p, int64_t ld, int n) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int x = threadIdx.x + i * NT, r = x / (C / 8), c = x % (C / 8) * 8;
      v[i].load(p + min(r, n - 1) * ld + c);
    }
  }
  __device__ __forceinline__ void store(char* lds, int n) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int x = threadIdx.x + i * NT, r = x / (C / 8), c = x % (C / 8) * 8;
      float f[8];
      v[i].get(f, r < n);
      Rows64<C>::template put<DeltaParts<T>::IN>(lds, r, c, f);
    }
  }
};

}  // namespace
}  // namespace m3
