// gated.h -- host-side launch interface of the gated linear recurrence.  Not
// part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace m3 {

constexpr int kGatedChunk = 128;   // rows between the states saved for the backward pass

struct GatedArgs {
  const void *x, *r, *i;      // rows of D channels, ldx / ldr / ldi elements apart
  const float* decay;         // [D]
  const float* h0;            // [B, D] or null
  const int32_t* cu;          // packed: [B + 1] row offsets, else null
  void* y;                    // dense rows of D
  float* hT;                  // [B, D] or null
  float* states;              // [rows of chunks, D] or null
  // backward
  const void* dy;
  const float* dhT;
  const float* cstates;
  void *dx, *dr, *di;         // rows ldg elements apart
  float *ddecay, *dh0;
  // workspace
  unsigned* ticket;
  int32_t* cuc;               // clean offsets
  struct GatedWindow* win;    // what every 32 rows of a packed call hold
  unsigned long long* slots;  // carries [ntile, nchain, channels of a chain]
  float* part;                // parts of ddecay [chunks, D]
  int64_t ldx, ldr, ldi, ldg;
  int B, T, D, S;             // B sequences (packed: of T rows together)
  int ncb, nchain, ntile;
  float c;
};

// The rows t0 .. t0 + 31 of a packed batch as bit masks: bit j of `start` /
// `end`: row t0 + j is the first / last of its sequence; `live`: it belongs to
// one.  s0 is at or before the sequence of the first live row, s1 at or behind
// that of the last.
struct alignas(32) GatedWindow {
  uint32_t start, end, live;
  int32_t s0, s1;
};

struct GatedPlan {
  int tile, ncb, ntile;       // rows per tile, blocks of 64 channels, tiles
  int64_t nchain;             // independent chains of tiles
};
GatedPlan gated_plan(int B, int T, int D, bool packed, bool backward);
size_t gated_workspace_bytes(int B, int T, int D, bool packed, bool backward);
void gated_carve(GatedArgs& g, bool backward, void* ws);
hipError_t launch_gated_scan(GatedArgs& g, int bf16, hipStream_t s);
hipError_t launch_gated_backward(GatedArgs& g, int bf16, hipStream_t s);
hipError_t launch_gated_step(const GatedArgs& g, float* h, int bf16, hipStream_t s);

}  // namespace m3
