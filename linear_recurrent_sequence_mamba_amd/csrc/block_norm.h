// block_norm.h -- host-side launch interface of the norms around a block.  Not
// part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace m3 {

enum { kGateLinear = 0, kGateSigmoid = 1, kGateSilu = 2 };
constexpr int kBlockNormMaxWidth = 16384;

struct BlockNormArgs {
  const void *x, *y, *gate;            // rows ldx / ldy / ldg elements apart; gate or null
  const float *wy, *scale, *wn;        // [W] or null (1)
  void *h, *n;                         // dense rows; n or null
  // backward
  const void *dh, *dn;                 // dense rows, one of them or null (0)
  void *dx, *dy, *dgate;
  float *dwy, *dscale, *dwn;           // [W] or null
  float* part;                         // workspace [workgroups, 2, W]
  int64_t ldx, ldy, ldg;
  int T, W;
  int act;                             // of the gate
  int raw;                             // y is taken as it is
  float eps;
};

size_t block_norm_workspace_bytes(int T, int W);
hipError_t launch_block_norm(const BlockNormArgs& a, int bf16, hipStream_t s);
hipError_t launch_block_norm_backward(const BlockNormArgs& a, int bf16, hipStream_t s);

}  // namespace m3
