// qk_norm.h -- host-side launch interface of the norms of queries and keys
// with the position rotation.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace m3 {

constexpr int kQkMaxDim = 256;

struct QkNormArgs {
  const void *q, *k;            // rows of H heads, ldq / ldk elements apart
  const float *wq, *wk;         // [D] or null (1)
  const int32_t* pos;           // [T]
  void *qo, *ko;                // dense [T, H, D]
  // backward
  const void *gq, *gk;          // dense [T, H, D]
  void *dq, *dk;                // rows ld_dq / ld_dk elements apart
  float *dwq, *dwk;             // [D] or null
  float* part;                  // workspace [blocks, 2, D]
  int64_t ldq, ldk, ld_dq, ld_dk;
  int T, Hq, Hk, D, rot;        // rot channels are rotated
  int half;                     // pairs (j, j + rot/2) instead of (2j, 2j+1)
  int split;                    // waves that share the heads of one token
  float eps;
  double freq[kQkMaxDim / 2];   // turns per position of each pair
};

bool qk_norm_supported(int D);
size_t qk_norm_workspace_bytes(int T, int Hq, int Hk, int D);
hipError_t launch_qk_norm(QkNormArgs& a, int bf16, hipStream_t s);
hipError_t launch_qk_norm_backward(QkNormArgs& a, int bf16, hipStream_t s);

}  // namespace m3
