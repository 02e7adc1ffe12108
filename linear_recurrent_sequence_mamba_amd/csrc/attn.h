// attn.h -- host-side launch interface of the causal attention kernels.  Not
// part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace m3 {

struct AttnArgs {
  const void *q, *k, *v;        // rows of H heads of D, ld* elements apart
  const int32_t *cuq, *cuk;     // [S + 1] row offsets of the sequences
  void* o;                      // rows ldo apart
  float* lse;                   // [Tq, Hq] (decode: [S, Hq])
  // backward
  const void *co, *dout;        // o and its gradient, rows ldo / lddo apart
  const float* clse;
  void *dq, *dk, *dv;           // dense rows
  float* stat;                  // workspace [2, Hq, Tq]: lse log2(e), then -<o, do>; infinity and 0
  float *pk, *pv;               // workspace [gsplit, Tk, Hk, D]: parts of dk, dv
  float *po, *pm;               // workspace: parts of o and their (max, sum)
  // decode
  const int32_t* len;           // [S] rows of each sequence's cache
  int64_t ldq, ldk, ldv, ldo, lddo;
  int64_t bk, bv;               // decode: elements from one sequence's cache to the next
  int Tq, Tk, S, Hq, Hk, D;
  int cap;                      // decode: rows a cache has room for
  int gsplit;                   // parts of a group of heads (backward of k, v)
  int lp;                       // log2 of the heads of a group that a tile of queries takes
  int nsplit;                   // parts of the keys (prompt) or of a cache (decode)
  float scale;
};

// Heads that share k and v and lie in one tile of 128 (query, head) pairs: the
// largest power of two that divides the group, up to 32.
inline int attn_log_pack(int Hq, int Hk) {
  int lp = 0;
  while (lp < 5 && (Hq / Hk) % (2 << lp) == 0) ++lp;
  return lp;
}
// Workgroups of a launch over queries: 128 pairs each, in as many slots as hold any
// split of Tq rows into S sequences.
inline int64_t attn_query_workgroups(int Tq, int S, int Hq, int Hk) {
  const int lp = attn_log_pack(Hq, Hk);
  return ((static_cast<int64_t>(Tq) >> (7 - lp)) + S) * (Hq >> lp);
}
// Up to so many of them are taken in the order of their work, by up to so many
// sequences.
constexpr int kRankedWorkgroups = 2048, kRankedSeqs = 64;
bool attn_supported(int D);
size_t attn_backward_workspace_bytes(int Tq, int Tk, int S, int Hq, int Hk, int D);
size_t attn_decode_workspace_bytes(int S, int cap, int Hq, int Hk, int D);
size_t attn_workspace_bytes(int Tq, int Tk, int S, int Hq, int Hk, int D, int bf16);
hipError_t launch_attn(AttnArgs& a, int bf16, void* ws, hipStream_t s);
hipError_t launch_attn_backward(AttnArgs& a, int bf16, void* ws, hipStream_t s);
hipError_t launch_attn_decode(AttnArgs& a, int bf16, void* ws, hipStream_t s);

}  // namespace m3
