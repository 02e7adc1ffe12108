// delta.h -- host-side launch interface of the gated delta rule.  Not part of
// the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace m3 {

constexpr int kDeltaChunk = 64;   // tokens of a chunk
constexpr int kDeltaMatrix = 64 * 64;
constexpr int kDeltaGates = 5 * 64;   // floats of a chunk's gates: exp(G), exp(G_end - G), beta, G in two parts

struct DeltaArgs {
  const void *q, *k, *v, *g, *beta;   // token rows, ld* elements apart
  const float* h0;                    // [B, Hv, Dk, Dv] or null
  const int32_t* cu;                  // packed: [B + 1] row offsets, else null
  void* o;                            // dense rows
  float* hT;                          // [B, Hv, Dk, Dv] or null
  float* states;                      // [slots, Hv, delta_state_floats] or null: the state before a chunk
                                      // [Dk, Dv], its u [64, Dv], its matrix and its gates
  // backward
  const float *cstates, *dhT;
  const void* dout;                   // dense rows
  void *dq, *dk, *dv, *dg, *dbeta;    // dense rows
  float* dh0;                         // [B, Hv, Dk, Dv] or null
  // workspace
  float* pm;                          // T \ P^T [64, 64] and the gates of chunk and head n: from pm + n
  int64_t ldpm;                       // ldpm on (in `states` where those are saved)
  float* after;                       // backward: gradients of the state behind a chunk [slots, Hv, Dk, Dv]
  float* dr;                          // backward: those of R [slots, Hv, 64, Dv]
  // (of segments that are not their sequences' last, DeltaSeg's n-th at n)
  float* ends;                        // their ends from a zero state, then the states behind them, in
                                      // the order of results [inner, Hv, Dv / 16, Dk / 16, 64, 4]
  uint16_t* maps;                     // their maps of a state less their decay, in parts and in the
                                      // order of operands [inner, Hv, parts, Dk / 16, Dk / 32, 64, 8]
  float* decays;                      // their decays [inner, Hv]
  float* firsts;                      // scan: the states before sequences of several segments, as
                                      // `ends`, DeltaSeg's place() [min(B, inner), Hv, ..]
  int64_t ldq, ldk, ldv, ldg, ldb;
  int B, T, Hk, Hv, Dk, Dv;           // B sequences of T rows (packed: of T rows together)
  int nslot;
  int lseg, nseg;                     // log2 of a segment's chunks, segment slots
  int inner;                          // segments that may not be their sequences' last, at most
  float scale;
};

// Segments of the chain: how many chunks (log2) each has.
struct DeltaPlan {
  int lseg;
  int64_t nseg;   // slots of segments
  bool split;     // some sequence may have more than one
  int64_t inner;  // segments that may not be their sequences' last, at most
};
DeltaPlan delta_plan(int B, int T, int Hv, int Dk, int Dv, bool packed, bool back);
size_t delta_segment_bytes(const DeltaPlan& p, int B, int Hv, int Dk, int Dv, bool back);
void delta_carve_segments(DeltaArgs& a, const DeltaPlan& p, void* ws, bool back);

inline int64_t delta_state_floats(int Dk, int Dv) {
  return static_cast<int64_t>(Dk + kDeltaChunk) * Dv + kDeltaMatrix + kDeltaGates;
}
bool delta_supported(int Dk, int Dv);
int64_t delta_slots(int B, int T, bool packed);
size_t delta_workspace_bytes(int B, int T, int Hv, int Dk, int Dv, bool packed);
size_t delta_backward_workspace_bytes(int B, int T, int Hv, int Dk, int Dv, bool packed);
void delta_carve(DeltaArgs& a, void* ws);
void delta_backward_carve(DeltaArgs& a, void* ws);
hipError_t launch_delta_backward(DeltaArgs& a, int bf16, hipStream_t s);
hipError_t launch_delta_scan(DeltaArgs& a, int bf16, hipStream_t s);
hipError_t launch_delta_step(const DeltaArgs& a, float* h, int bf16, hipStream_t s);

}  // namespace m3
