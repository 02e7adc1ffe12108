// api.cpp -- the C ABI of libm3ssm (include/m3ssm.h): argument checks,
// workspace sizing and dispatch to the gfx950 kernels.  Every check runs on
// the host before anything is launched.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <mutex>

#include "../../include/m3ssm.h"
#include "attn.h"
#include "block_norm.h"
#include "delta.h"
#include "gated.h"
#include "m3_launch.h"
#include "qk_norm.h"
#include "rope_freq.h"

namespace {

thread_local int g_last_hip_error = 0;

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

m3_status hip_status(hipError_t e) {
  if (e == hipSuccess) return M3_OK;
  g_last_hip_error = static_cast<int>(e);
  return M3_ERR_HIP;
}

m3_status check_dims(const m3_dims* d, bool need_seqlen) {
  if (!d) return M3_ERR_NULL;
  if (d->batch <= 0 || d->nheads <= 0 || d->headdim <= 0 || d->dstate <= 0 || d->rank <= 0)
    return M3_ERR_SHAPE;
  if (need_seqlen && d->seqlen <= 0) return M3_ERR_SHAPE;
  if (d->dstate % 2 != 0) return M3_ERR_SHAPE;
  if (d->chunk < 0) return M3_ERR_SHAPE;
  if (d->in_dtype != M3_F32 && d->in_dtype != M3_BF16) return M3_ERR_DTYPE;
  if (d->out_dtype != M3_F32 && d->out_dtype != M3_BF16) return M3_ERR_DTYPE;
  if (d->flags & ~(M3_THETA_IS_ANGLE | M3_A_PER_TOKEN)) return M3_ERR_SHAPE;
  if (d->ngroups < 0 || d->ngroups > d->nheads) return M3_ERR_SHAPE;
  if (d->ngroups > 0 && d->nheads % d->ngroups != 0) return M3_ERR_SHAPE;
  return M3_OK;
}

int groups_of(const m3_dims* d) { return d->ngroups > 0 ? d->ngroups : d->nheads; }

// the B/C preparation of dims->bc into kernel arguments (off when absent)
m3_status bc_args(const m3_dims* d, m3::BCPrep* out) {
  *out = m3::BCPrep{};
  const m3_bc_prep* bc = d->bc;
  if (!bc) return M3_OK;
  if (!isfinite(bc->eps) || bc->eps < 0.0f) return M3_ERR_SHAPE;
  const void* ptrs[] = {bc->B_weight, bc->C_weight, bc->B_bias, bc->C_bias};
  for (const void* p : ptrs)
    if (p && misaligned(p)) return M3_ERR_ALIGN;
  out->Bw = bc->B_weight;
  out->Cw = bc->C_weight;
  out->Bb = bc->B_bias;
  out->Cb = bc->C_bias;
  out->eps = bc->eps;
  out->rms = bc->rms != 0;
  out->on = 1;
  return M3_OK;
}

// the angle projection of dims->tp into kernel arguments (off when absent)
m3_status tp_args(const m3_dims* d, m3::ThetaProj* out) {
  *out = m3::ThetaProj{};
  const m3_theta_proj* tp = d->tp;
  if (!tp) return M3_OK;
  if (tp->dim <= 0 || tp->dim % 32 != 0) return M3_ERR_SHAPE;
  if (!tp->u || !tp->W) return M3_ERR_NULL;
  if (misaligned(tp->u) || misaligned(tp->W)) return M3_ERR_ALIGN;
  out->u = tp->u;
  out->W = tp->W;
  out->dim = tp->dim;
  out->on = 1;
  return M3_OK;
}

// the backward's chunk length (64 unless the caller asks)
int chunk_of(const m3_dims* d) { return d->chunk > 0 ? d->chunk : 64; }
// a forward prefill's chunk length: the caller's, or the library's default
// for the shape
int prefill_chunk_of(const m3_dims* d) {
  return d->chunk > 0 ? d->chunk
                      : m3::prefill_default_chunk(d->headdim, d->dstate, d->rank,
                                                  d->in_dtype == M3_BF16);
}

// ---------------------------------------------------------------------------
// The scratch buffer of m3_scan_prefill_noalloc: one copy per GPU the library
// runs on, held until the process ends.  In host code `scratch` names a host
// stand-in, not device memory, so every host use goes through the device
// address that hipGetSymbolAddress returns for the current device, looked up
// once per device and kept.
static __device__ __align__(256) unsigned char scratch[M3_NOALLOC_SCRATCH_BYTES];

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices];   // this device's copy of `scratch`, or null until looked up

// the device address of `scratch` on the device of `stream` (the current
// device for the null stream), which must be the current device
hipError_t scratch_of_stream_device(void* stream, void** out) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (stream) {
    hipDevice_t sdev = 0;
    e = hipStreamGetDevice(static_cast<hipStream_t>(stream), &sdev);
    if (e != hipSuccess) return e;
    if (sdev != dev) return hipErrorInvalidDevice;
  }
  if (dev < 0 || dev >= kMaxDevices) return hipErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_ptr[dev]) {
    void* p = nullptr;
    e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (e != hipSuccess) return e;
    if (!p) return hipErrorInvalidSymbol;
    g_scratch_ptr[dev] = p;
  }
  *out = g_scratch_ptr[dev];
  return hipSuccess;
}

// m3_scan_prefill with the caller's workspace, or (noalloc) with this
// device's copy of `scratch`
m3_status scan_prefill(const m3_dims* d, const void* x, const void* dt, const float* A,
                       const void* lam, const void* theta, const void* B, const void* C,
                       const float* h0, const void* x_prev, const void* B_prev, void* y,
                       float* hT, void* ws, size_t ws_bytes, bool noalloc, void* stream) {
  m3_status st = check_dims(d, true);
  if (st != M3_OK) return st;
  m3::BCPrep bcp;
  if ((st = bc_args(d, &bcp)) != M3_OK) return st;
  m3::ThetaProj tpa;
  if ((st = tp_args(d, &tpa)) != M3_OK) return st;
  if (!x || !dt || !A || !lam || (!theta && !tpa.on) || !B || !C || !y) return M3_ERR_NULL;
  if ((x_prev == nullptr) != (B_prev == nullptr)) return M3_ERR_NULL;
  const void* ptrs[] = {x, dt, A, lam, theta, B, C, h0, x_prev, B_prev, y, hT, ws};
  for (const void* p : ptrs)
    if (p && misaligned(p)) return M3_ERR_ALIGN;
  const int Q = prefill_chunk_of(d);
  const int in_bf16 = d->in_dtype == M3_BF16;
  if (!m3::prefill_supported(d->headdim, d->dstate, d->rank, Q, in_bf16))
    return M3_ERR_UNSUPPORTED;
  const size_t need = m3::prefill_workspace_bytes(d->batch, d->seqlen, d->nheads, d->headdim,
                                                  d->dstate, d->rank, Q, bcp.on != 0);
  if (noalloc) {
    if (need > M3_NOALLOC_SCRATCH_BYTES) return M3_ERR_TOO_LARGE;
    hipError_t e = scratch_of_stream_device(stream, &ws);
    if (e != hipSuccess) return hip_status(e);
    ws_bytes = M3_NOALLOC_SCRATCH_BYTES;
  }
  if (!ws || ws_bytes < need) return M3_ERR_WORKSPACE;

  m3::PrefillArgs a{};
  a.x = x;
  a.dt = dt;
  a.A = A;
  a.lam = lam;
  a.theta = theta;
  a.B = B;
  a.C = C;
  a.h0 = h0;
  a.xp = x_prev;
  a.Bp = B_prev;
  a.y = y;
  a.hT = hT;
  a.Bsz = d->batch;
  a.T = d->seqlen;
  a.H = d->nheads;
  a.P = d->headdim;
  a.N = d->dstate;
  a.R = d->rank;
  a.Q = Q;
  a.nchunk = (d->seqlen + Q - 1) / Q;
  a.G = groups_of(d);
  a.flags = d->flags;
  a.has_prev = x_prev != nullptr;
  a.bc = bcp;
  a.tp = tpa;
  m3::prefill_carve(a, ws);
  hipError_t err = hipSuccess;
  if (m3::launch_prefill(a, in_bf16, d->out_dtype == M3_BF16,
                         static_cast<hipStream_t>(stream), &err) != 0)
    return M3_ERR_UNSUPPORTED;
  return hip_status(err);
}


// ---------------------------------------------------------------------------
// the other layers of a hybrid stack
bool misaligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }
// rows and tiles are counted in int, beyond the last one as well
constexpr int kMostRows = 0x7fff0000;
bool bad_dtype(int t) { return t != M3_F32 && t != M3_BF16; }
// a kernel's threads are counted in 32 bits
bool grid_fits(int64_t blocks, int threads) { return blocks <= int64_t{0xffffffff} / threads; }

template <size_t N>
bool any_misaligned(const void* const (&p)[N]) {
  for (const void* x : p)
    if (x && misaligned(x)) return true;
  return false;
}

m3_status check_gated(const m3_gated_dims* d, bool scan, bool packed) {
  if (!d) return M3_ERR_NULL;
  if (d->batch <= 0 || d->width <= 0 || (scan && d->seqlen <= 0)) return M3_ERR_SHAPE;
  if (d->batch > kMostRows || d->width > kMostRows || (scan && d->seqlen > kMostRows)) return M3_ERR_SHAPE;
  if (!isfinite(d->c) || d->c <= 0.0f) return M3_ERR_SHAPE;
  const int64_t lds[] = {d->ld_x, d->ld_r, d->ld_i, d->ld_g};
  for (int64_t ld : lds)
    if (ld != 0 && ld < d->width) return M3_ERR_SHAPE;
  if (bad_dtype(d->dtype)) return M3_ERR_DTYPE;
  if (scan) {
    const m3::GatedPlan p = m3::gated_plan(d->batch, d->seqlen, d->width, packed, true);
    if (p.nchain > 0x7fffffff || !grid_fits(p.nchain * p.ntile, 1024)) return M3_ERR_SHAPE;
  } else if (!grid_fits((static_cast<int64_t>(d->batch) * d->width + 255) / 256, 256)) {
    return M3_ERR_SHAPE;
  }
  return M3_OK;
}

m3::GatedArgs gated_args(const m3_gated_dims* d) {
  m3::GatedArgs g{};
  g.B = d->batch;
  g.T = d->seqlen;
  g.D = d->width;
  g.c = d->c;
  g.ldx = d->ld_x ? d->ld_x : d->width;
  g.ldr = d->ld_r ? d->ld_r : d->width;
  g.ldi = d->ld_i ? d->ld_i : d->width;
  g.ldg = d->ld_g ? d->ld_g : d->width;
  return g;
}

m3_status check_qk(const m3_qk_dims* d) {
  if (!d) return M3_ERR_NULL;
  if (d->tokens <= 0 || d->nheads_q <= 0 || d->nheads_k <= 0 || d->headdim <= 0) return M3_ERR_SHAPE;
  if (d->tokens > kMostRows) return M3_ERR_SHAPE;
  if (d->rotary_dim < 0 || d->rotary_dim > d->headdim || d->rotary_dim % 2) return M3_ERR_SHAPE;
  if (d->flags & ~M3_ROPE_HALF) return M3_ERR_SHAPE;
  if (!isfinite(d->eps) || d->eps < 0.0f) return M3_ERR_SHAPE;
  if (!isfinite(d->base) || d->base <= 0.0) return M3_ERR_SHAPE;
  if (bad_dtype(d->dtype)) return M3_ERR_DTYPE;
  const int64_t wq = static_cast<int64_t>(d->nheads_q) * d->headdim;
  const int64_t wk = static_cast<int64_t>(d->nheads_k) * d->headdim;
  if (wq > 0x3fffffff || wk > 0x3fffffff) return M3_ERR_SHAPE;
  if ((d->ld_q && d->ld_q < wq) || (d->ld_dq && d->ld_dq < wq) || (d->ld_k && d->ld_k < wk) ||
      (d->ld_dk && d->ld_dk < wk))
    return M3_ERR_SHAPE;
  if (!m3::qk_norm_supported(d->headdim)) return M3_ERR_UNSUPPORTED;
  if ((d->ld_q | d->ld_k | d->ld_dq | d->ld_dk) % 8) return M3_ERR_ALIGN;
  return M3_OK;
}

m3::QkNormArgs qk_args(const m3_qk_dims* d) {
  m3::QkNormArgs a{};
  a.T = d->tokens;
  a.Hq = d->nheads_q;
  a.Hk = d->nheads_k;
  a.D = d->headdim;
  a.rot = d->rotary_dim;
  a.half = (d->flags & M3_ROPE_HALF) != 0;
  a.eps = d->eps;
  const int64_t wq = static_cast<int64_t>(a.Hq) * a.D, wk = static_cast<int64_t>(a.Hk) * a.D;
  a.ldq = d->ld_q ? d->ld_q : wq;
  a.ldk = d->ld_k ? d->ld_k : wk;
  a.ld_dq = d->ld_dq ? d->ld_dq : wq;
  a.ld_dk = d->ld_dk ? d->ld_dk : wk;
  m3::rope_freq(d->base, a.rot, a.freq);
  return a;
}

m3_status check_delta(const m3_delta_dims* d, bool scan, bool packed) {
  if (!d) return M3_ERR_NULL;
  if (d->batch <= 0 || (scan && d->seqlen <= 0)) return M3_ERR_SHAPE;
  if (d->batch > kMostRows || (scan && d->seqlen > kMostRows)) return M3_ERR_SHAPE;
  if (d->nheads_k <= 0 || d->nheads_v <= 0 || d->headdim_k <= 0 || d->headdim_v <= 0)
    return M3_ERR_SHAPE;
  if (d->nheads_v % d->nheads_k) return M3_ERR_SHAPE;
  if (!isfinite(d->scale)) return M3_ERR_SHAPE;
  if (bad_dtype(d->dtype)) return M3_ERR_DTYPE;
  if (!m3::delta_supported(d->headdim_k, d->headdim_v)) return M3_ERR_UNSUPPORTED;
  const int64_t wk = static_cast<int64_t>(d->nheads_k) * d->headdim_k;
  const int64_t wv = static_cast<int64_t>(d->nheads_v) * d->headdim_v;
  const int64_t most = int64_t{1} << 24;   // a chunk's rows are 32-bit offsets apart
  if (wk >= most || wv >= most) return M3_ERR_SHAPE;
  const int64_t lds[][2] = {{d->ld_q, wk}, {d->ld_k, wk}, {d->ld_v, wv}, {d->ld_g, d->nheads_v}, {d->ld_beta, d->nheads_v}};
  for (const auto& l : lds)
    if (l[0] != 0 && (l[0] < l[1] || l[0] >= most)) return M3_ERR_SHAPE;
  if ((d->ld_q | d->ld_k | d->ld_v) % 8) return M3_ERR_ALIGN;
  // the step: 4 Dv threads for a sequence's head.  The scan: at most 4 (Dk + Dv)
  // for each chunk and head (what joins segments 2 Dk Dv / 16, once for at least
  // eight chunks)
  const int64_t slots = scan ? m3::delta_slots(d->batch, d->seqlen, packed) : d->batch;
  if (slots > 0x7fffffff || !grid_fits(slots * d->nheads_v, scan ? 1024 : 512)) return M3_ERR_SHAPE;
  return M3_OK;
}

static_assert(M3_DELTA_CHUNK == m3::kDeltaChunk &&
                  M3_DELTA_STATE_FLOATS(128, 64) == 192 * 64 + m3::kDeltaMatrix + m3::kDeltaGates,
              "the header's sizes");
// g and beta may be columns of any row
bool misaligned_gates(const m3_delta_dims* d, const void* g, const void* beta) {
  const uintptr_t m = d->dtype == M3_BF16 ? 1u : 3u;
  return ((reinterpret_cast<uintptr_t>(g) | reinterpret_cast<uintptr_t>(beta)) & m) != 0;
}

m3::DeltaArgs delta_args(const m3_delta_dims* d) {
  m3::DeltaArgs a{};
  a.B = d->batch;
  a.T = d->seqlen;
  a.Hk = d->nheads_k;
  a.Hv = d->nheads_v;
  a.Dk = d->headdim_k;
  a.Dv = d->headdim_v;
  a.scale = d->scale;
  const int64_t wk = static_cast<int64_t>(a.Hk) * a.Dk, wv = static_cast<int64_t>(a.Hv) * a.Dv;
  a.ldq = d->ld_q ? d->ld_q : wk;
  a.ldk = d->ld_k ? d->ld_k : wk;
  a.ldv = d->ld_v ? d->ld_v : wv;
  a.ldg = d->ld_g ? d->ld_g : a.Hv;
  a.ldb = d->ld_beta ? d->ld_beta : a.Hv;
  return a;
}

m3_status check_block(const m3_block_dims* d) {
  if (!d) return M3_ERR_NULL;
  if (d->tokens <= 0 || d->width <= 0 || d->tokens > kMostRows) return M3_ERR_SHAPE;
  if (d->flags & ~(M3_GATE_SIGMOID | M3_GATE_SILU | M3_BLOCK_RAW)) return M3_ERR_SHAPE;
  if ((d->flags & M3_GATE_SIGMOID) && (d->flags & M3_GATE_SILU)) return M3_ERR_SHAPE;
  if (!isfinite(d->eps) || d->eps < 0.0f) return M3_ERR_SHAPE;
  const int64_t lds[] = {d->ld_x, d->ld_y, d->ld_gate};
  for (int64_t ld : lds)
    if (ld != 0 && ld < d->width) return M3_ERR_SHAPE;
  if (bad_dtype(d->dtype)) return M3_ERR_DTYPE;
  if (d->width > m3::kBlockNormMaxWidth) return M3_ERR_UNSUPPORTED;
  return M3_OK;
}

m3::BlockNormArgs block_args(const m3_block_dims* d) {
  m3::BlockNormArgs a{};
  a.T = d->tokens;
  a.W = d->width;
  a.act = d->flags & M3_GATE_SILU      ? m3::kGateSilu
          : d->flags & M3_GATE_SIGMOID ? m3::kGateSigmoid
                                       : m3::kGateLinear;
  a.raw = (d->flags & M3_BLOCK_RAW) != 0;
  a.eps = d->eps;
  a.ldx = d->ld_x ? d->ld_x : d->width;
  a.ldy = d->ld_y ? d->ld_y : d->width;
  a.ldg = d->ld_gate ? d->ld_gate : d->width;
  return a;
}

m3_status check_attn(const m3_attn_dims* d, bool decode) {
  if (!d) return M3_ERR_NULL;
  if (d->nseq <= 0 || d->tokens_k <= 0 || (!decode && d->tokens_q <= 0)) return M3_ERR_SHAPE;
  if (d->tokens_k > kMostRows || (!decode && d->tokens_q > kMostRows)) return M3_ERR_SHAPE;
  if (d->nheads_q <= 0 || d->nheads_k <= 0 || d->headdim <= 0) return M3_ERR_SHAPE;
  if (d->nheads_q % d->nheads_k) return M3_ERR_SHAPE;
  // the maximum of the scores is that of the products, and a masked one's
  // scale * -inf has to stay -inf
  if (!isfinite(d->scale) || d->scale < 1.1754944e-38f) return M3_ERR_SHAPE;
  if (bad_dtype(d->dtype)) return M3_ERR_DTYPE;
  if (!m3::attn_supported(d->headdim)) return M3_ERR_UNSUPPORTED;
  const int64_t wq = static_cast<int64_t>(d->nheads_q) * d->headdim;
  const int64_t wk = static_cast<int64_t>(d->nheads_k) * d->headdim;
  const int64_t lq[] = {d->ld_q, d->ld_o, d->ld_do}, lk[] = {d->ld_k, d->ld_v};
  const int64_t most = int64_t{1} << 24;   // a tile's rows are 32-bit offsets apart
  if (wq >= most) return M3_ERR_SHAPE;
  for (int64_t ld : lq)
    if (ld != 0 && (ld < wq || ld >= most)) return M3_ERR_SHAPE;
  for (int64_t ld : lk)
    if (ld != 0 && (ld < wk || ld >= most)) return M3_ERR_SHAPE;
  if (d->stride_k < 0 || d->stride_v < 0) return M3_ERR_SHAPE;
  if ((d->ld_q | d->ld_o | d->ld_do | d->ld_k | d->ld_v | d->stride_k | d->stride_v) % 8)
    return M3_ERR_ALIGN;
  if (!decode) {
    // workgroups of the queries and of the keys; the kernels that join parts only
    // run where there are few of those
    const int64_t tiles = (static_cast<int64_t>(d->tokens_q > d->tokens_k ? d->tokens_q
                                                                          : d->tokens_k) >> 7) + d->nseq + 1;
    if (tiles > 0x7fffffff || !grid_fits(tiles * d->nheads_q, 256)) return M3_ERR_SHAPE;
  } else if (!grid_fits(static_cast<int64_t>(d->nseq) * d->nheads_q + 512, 256)) {   // 512: parts
    return M3_ERR_SHAPE;
  }
  return M3_OK;
}

m3::AttnArgs attn_args(const m3_attn_dims* d) {
  m3::AttnArgs a{};
  a.S = d->nseq;
  a.Tq = d->tokens_q;
  a.Tk = d->tokens_k;
  a.cap = d->tokens_k;
  a.Hq = d->nheads_q;
  a.Hk = d->nheads_k;
  a.D = d->headdim;
  a.scale = d->scale;
  const int64_t wq = static_cast<int64_t>(a.Hq) * a.D, wk = static_cast<int64_t>(a.Hk) * a.D;
  a.ldq = d->ld_q ? d->ld_q : wq;
  a.ldo = d->ld_o ? d->ld_o : wq;
  a.lddo = d->ld_do ? d->ld_do : wq;
  a.ldk = d->ld_k ? d->ld_k : wk;
  a.ldv = d->ld_v ? d->ld_v : wk;
  a.bk = d->stride_k ? d->stride_k : a.cap * a.ldk;
  a.bv = d->stride_v ? d->stride_v : a.cap * a.ldv;
  return a;
}

}  // namespace

extern "C" {

const char* m3_status_str(m3_status s) {
  // a C caller may pass any int; read its bits as an int, since a C++ load
  // of an enum value outside the enumerators' range is undefined
  int v;
  memcpy(&v, &s, sizeof v);
  switch (v) {
    case M3_OK: return "ok";
    case M3_ERR_NULL: return "required pointer is NULL";
    case M3_ERR_SHAPE: return "invalid shape or flags";
    case M3_ERR_DTYPE: return "unsupported dtype";
    case M3_ERR_UNSUPPORTED: return "no kernel for this (headdim, dstate, rank, chunk)";
    case M3_ERR_ALIGN: return "pointer not 16-byte aligned";
    case M3_ERR_WORKSPACE: return "workspace missing or too small";
    case M3_ERR_HIP: return "HIP launch failed";
    case M3_ERR_TOO_LARGE: return "call needs more than the built-in scratch buffer";
  }
  return "unknown status";
}

int m3_last_hip_error(void) { return g_last_hip_error; }

size_t m3_prefill_workspace_size(const m3_dims* d) {
  if (check_dims(d, true) != M3_OK) return 0;
  return m3::prefill_workspace_bytes(d->batch, d->seqlen, d->nheads, d->headdim, d->dstate,
                                     d->rank, prefill_chunk_of(d), d->bc != nullptr);
}

m3_status m3_scan_prefill(const m3_dims* d, const void* x, const void* dt, const float* A,
                          const void* lam, const void* theta, const void* B, const void* C,
                          const float* h0, const void* x_prev, const void* B_prev, void* y,
                          float* hT, void* ws, size_t ws_bytes, void* stream) {
  return scan_prefill(d, x, dt, A, lam, theta, B, C, h0, x_prev, B_prev, y, hT, ws, ws_bytes,
                      false, stream);
}

m3_status m3_scan_prefill_noalloc(const m3_dims* d, const void* x, const void* dt,
                                  const float* A, const void* lam, const void* theta,
                                  const void* B, const void* C, const float* h0,
                                  const void* x_prev, const void* B_prev, void* y, float* hT,
                                  void* stream) {
  return scan_prefill(d, x, dt, A, lam, theta, B, C, h0, x_prev, B_prev, y, hT, nullptr, 0, true,
                      stream);
}

size_t m3_prefill_backward_workspace_size(const m3_dims* d) {
  if (check_dims(d, true) != M3_OK) return 0;
  return m3::backward_workspace_bytes(d->batch, d->seqlen, d->nheads, d->headdim, d->dstate,
                                      d->rank, groups_of(d), chunk_of(d));
}

m3_status m3_scan_prefill_backward(const m3_dims* d, const void* x, const void* dt,
                                   const float* A, const void* lam, const void* theta,
                                   const void* B, const void* C, const float* h0,
                                   const void* x_prev, const void* B_prev, const void* dy,
                                   const float* dhT, float* dx, float* ddt, float* dA,
                                   float* dlam, float* dtheta, float* dB, float* dC, float* dh0,
                                   float* dx_prev, float* dB_prev, void* ws, size_t ws_bytes,
                                   void* stream) {
  m3_status st = check_dims(d, true);
  if (st != M3_OK) return st;
  if (d->bc || d->tp) return M3_ERR_UNSUPPORTED;
  if (!x || !dt || !A || !lam || !theta || !B || !C || !dy) return M3_ERR_NULL;
  if (!dx || !ddt || !dA || !dlam || !dtheta || !dB || !dC) return M3_ERR_NULL;
  if ((x_prev == nullptr) != (B_prev == nullptr)) return M3_ERR_NULL;
  const void* ptrs[] = {x, dt, A, lam, theta, B, C, h0, x_prev, B_prev, dy, dhT, dx, ddt, dA,
                        dlam, dtheta, dB, dC, dh0, dx_prev, dB_prev, ws};
  for (const void* p : ptrs)
    if (p && misaligned(p)) return M3_ERR_ALIGN;
  const int Q = chunk_of(d);
  const int in_bf16 = d->in_dtype == M3_BF16;
  if (!m3::prefill_supported(d->headdim, d->dstate, d->rank, Q, in_bf16) ||
      !m3::backward_supported(d->headdim, d->dstate, d->rank, Q))
    return M3_ERR_UNSUPPORTED;
  const size_t need = m3::backward_workspace_bytes(d->batch, d->seqlen, d->nheads, d->headdim,
                                                   d->dstate, d->rank, groups_of(d), Q);
  if (!ws || ws_bytes < need) return M3_ERR_WORKSPACE;

  m3::BackwardArgs g{};
  m3::PrefillArgs& a = g.f;
  a.x = x;
  a.dt = dt;
  a.A = A;
  a.lam = lam;
  a.theta = theta;
  a.B = B;
  a.C = C;
  a.h0 = h0;
  a.xp = x_prev;
  a.Bp = B_prev;
  a.Bsz = d->batch;
  a.T = d->seqlen;
  a.H = d->nheads;
  a.P = d->headdim;
  a.N = d->dstate;
  a.R = d->rank;
  a.Q = Q;
  a.nchunk = (d->seqlen + Q - 1) / Q;
  a.G = groups_of(d);
  a.flags = d->flags;
  a.has_prev = x_prev != nullptr;
  g.dy = dy;
  g.dhT = dhT;
  g.dx = dx;
  g.ddt = ddt;
  g.dA = dA;
  g.dlam = dlam;
  g.dtheta = dtheta;
  g.dB = dB;
  g.dC = dC;
  g.dh0 = dh0;
  g.dx_prev = x_prev ? dx_prev : nullptr;
  g.dB_prev = x_prev ? dB_prev : nullptr;
  m3::backward_carve(g, ws);
  hipError_t err = hipSuccess;
  if (m3::launch_backward(g, in_bf16, d->out_dtype == M3_BF16, static_cast<hipStream_t>(stream),
                          &err) != 0)
    return M3_ERR_UNSUPPORTED;
  return hip_status(err);
}

size_t m3_prefill_varlen_workspace_size(const m3_dims* d) {
  if (check_dims(d, true) != M3_OK) return 0;
  return m3::prefill_varlen_workspace_bytes(d->batch, d->seqlen, d->nheads, d->headdim, d->dstate,
                                            d->rank, prefill_chunk_of(d), d->bc != nullptr);
}

m3_status m3_scan_prefill_varlen(const m3_dims* d, const int32_t* cu_seqlens, const void* x,
                                 const void* dt, const float* A, const void* lam,
                                 const void* theta, const void* B, const void* C,
                                 const float* h0, const void* x_prev, const void* B_prev, void* y,
                                 float* hT, void* ws, size_t ws_bytes, void* stream) {
  m3_status st = check_dims(d, true);
  if (st != M3_OK) return st;
  m3::BCPrep bcp;
  if ((st = bc_args(d, &bcp)) != M3_OK) return st;
  m3::ThetaProj tpa;
  if ((st = tp_args(d, &tpa)) != M3_OK) return st;
  if (!cu_seqlens || !x || !dt || !A || !lam || (!theta && !tpa.on) || !B || !C || !y)
    return M3_ERR_NULL;
  if ((x_prev == nullptr) != (B_prev == nullptr)) return M3_ERR_NULL;
  const void* ptrs[] = {x, dt, A, lam, theta, B, C, h0, x_prev, B_prev, y, hT, ws};
  for (const void* p : ptrs)
    if (p && misaligned(p)) return M3_ERR_ALIGN;
  if (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) return M3_ERR_ALIGN;
  const int Q = prefill_chunk_of(d);
  const int in_bf16 = d->in_dtype == M3_BF16;
  if (!m3::prefill_supported(d->headdim, d->dstate, d->rank, Q, in_bf16) ||
      !m3::prefill_offsets_fit(d->nheads, d->headdim, d->dstate, d->rank, Q))
    return M3_ERR_UNSUPPORTED;
  const size_t need = m3::prefill_varlen_workspace_bytes(d->batch, d->seqlen, d->nheads,
                                                         d->headdim, d->dstate, d->rank, Q,
                                                         bcp.on != 0);
  if (!ws || ws_bytes < need) return M3_ERR_WORKSPACE;

  m3::PrefillArgs a{};
  a.x = x;
  a.dt = dt;
  a.A = A;
  a.lam = lam;
  a.theta = theta;
  a.B = B;
  a.C = C;
  a.h0 = h0;
  a.xp = x_prev;
  a.Bp = B_prev;
  a.y = y;
  a.hT = hT;
  a.Bsz = d->batch;
  a.T = d->seqlen;
  a.H = d->nheads;
  a.P = d->headdim;
  a.N = d->dstate;
  a.R = d->rank;
  a.Q = Q;
  a.nchunk = static_cast<int>(m3::varlen_slots(d->batch, d->seqlen, Q));
  a.G = groups_of(d);
  a.flags = d->flags;
  a.has_prev = x_prev != nullptr;
  a.bc = bcp;
  a.tp = tpa;
  m3::prefill_varlen_carve(a, ws);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t err = m3::launch_varlen_map(a, cu_seqlens, s);
  if (err != hipSuccess) return hip_status(err);
  if (m3::launch_prefill(a, in_bf16, d->out_dtype == M3_BF16, s, &err) != 0)
    return M3_ERR_UNSUPPORTED;
  return hip_status(err);
}

m3_status m3_decode_step(const m3_dims* d, float* h, const void* x_t, const void* x_prev,
                         const void* B_t, const void* B_prev, const void* C_t, const void* dt_t,
                         const float* A, const void* lam_t, const void* theta_t, void* y_t,
                         void* stream) {
  m3_status st = check_dims(d, false);
  if (st != M3_OK) return st;
  m3::BCPrep bcp;
  if ((st = bc_args(d, &bcp)) != M3_OK) return st;
  m3::ThetaProj tpa;
  if ((st = tp_args(d, &tpa)) != M3_OK) return st;
  if (!h || !x_t || !B_t || !C_t || !dt_t || !A || !lam_t || (!theta_t && !tpa.on) || !y_t)
    return M3_ERR_NULL;
  if ((x_prev == nullptr) != (B_prev == nullptr)) return M3_ERR_NULL;
  const void* ptrs[] = {h, x_t, x_prev, B_t, B_prev, C_t, dt_t, A, lam_t, theta_t, y_t};
  for (const void* p : ptrs)
    if (p && misaligned(p)) return M3_ERR_ALIGN;
  if (!m3::decode_supported(d->headdim, d->dstate, d->rank)) return M3_ERR_UNSUPPORTED;
  const int64_t units = static_cast<int64_t>(d->batch) * d->nheads;
  if (units > 0x7fffffff) return M3_ERR_SHAPE;

  m3::DecodeArgs a{};
  a.h = h;
  a.x = x_t;
  a.xp = x_prev;
  a.Bt = B_t;
  a.Bp = B_prev;
  a.Ct = C_t;
  a.dt = dt_t;
  a.A = A;
  a.lam = lam_t;
  a.theta = theta_t;
  a.y = y_t;
  a.H = d->nheads;
  a.P = d->headdim;
  a.N = d->dstate;
  a.R = d->rank;
  a.G = groups_of(d);
  a.K = 1;
  a.flags = d->flags;
  a.has_prev = x_prev != nullptr;
  a.bc = bcp;
  a.tp = tpa;
  hipError_t err = hipSuccess;
  if (m3::launch_decode(a, d->in_dtype == M3_BF16, d->out_dtype == M3_BF16,
                        static_cast<int>(units), static_cast<hipStream_t>(stream), &err) != 0)
    return M3_ERR_UNSUPPORTED;
  return hip_status(err);
}

m3_status m3_decode_tokens(const m3_dims* d, float* h, const void* x, const void* x_prev,
                           const void* B, const void* B_prev, const void* C, const void* dt,
                           const float* A, const void* lam, const void* theta, void* y,
                           void* stream) {
  m3_status st = check_dims(d, true);
  if (st != M3_OK) return st;
  m3::BCPrep bcp;
  if ((st = bc_args(d, &bcp)) != M3_OK) return st;
  if (d->tp) return M3_ERR_UNSUPPORTED;
  if (!h || !x || !B || !C || !dt || !A || !lam || !theta || !y) return M3_ERR_NULL;
  if ((x_prev == nullptr) != (B_prev == nullptr)) return M3_ERR_NULL;
  const void* ptrs[] = {h, x, x_prev, B, B_prev, C, dt, A, lam, theta, y};
  for (const void* p : ptrs)
    if (p && misaligned(p)) return M3_ERR_ALIGN;
  if (!m3::decode_tokens_supported(d->headdim, d->dstate, d->rank)) return M3_ERR_UNSUPPORTED;
  const int64_t units = static_cast<int64_t>(d->batch) * d->nheads;
  if (units > 0x7fffffff) return M3_ERR_SHAPE;

  m3::DecodeArgs a{};
  a.h = h;
  a.x = x;
  a.xp = x_prev;
  a.Bt = B;
  a.Bp = B_prev;
  a.Ct = C;
  a.dt = dt;
  a.A = A;
  a.lam = lam;
  a.theta = theta;
  a.y = y;
  a.H = d->nheads;
  a.P = d->headdim;
  a.N = d->dstate;
  a.R = d->rank;
  a.G = groups_of(d);
  a.K = d->seqlen;
  a.flags = d->flags;
  a.has_prev = x_prev != nullptr;
  a.bc = bcp;
  hipError_t err = hipSuccess;
  if (m3::launch_decode_tokens(a, d->in_dtype == M3_BF16, d->out_dtype == M3_BF16,
                               static_cast<int>(units), static_cast<hipStream_t>(stream), &err) != 0)
    return M3_ERR_UNSUPPORTED;
  return hip_status(err);
}

size_t m3_gated_scan_workspace_size(const m3_gated_dims* d, int packed) {
  if (check_gated(d, true, packed != 0) != M3_OK) return 0;
  return m3::gated_workspace_bytes(d->batch, d->seqlen, d->width, packed != 0, false);
}

size_t m3_gated_scan_backward_workspace_size(const m3_gated_dims* d, int packed) {
  if (check_gated(d, true, packed != 0) != M3_OK) return 0;
  return m3::gated_workspace_bytes(d->batch, d->seqlen, d->width, packed != 0, true);
}

m3_status m3_gated_scan(const m3_gated_dims* d, const int32_t* cu_seqlens, const void* x,
                        const void* r, const void* i, const float* decay, const float* h0, void* y,
                        float* hT, float* states, void* ws, size_t ws_bytes, void* stream) {
  const bool packed = cu_seqlens != nullptr;
  m3_status st = check_gated(d, true, packed);
  if (st != M3_OK) return st;
  if (!x || !r || !i || !decay || !y) return M3_ERR_NULL;
  const void* const ptrs[] = {x, r, i, decay, h0, y, hT, states, ws};
  if (any_misaligned(ptrs) || misaligned4(cu_seqlens)) return M3_ERR_ALIGN;
  if (!ws || ws_bytes < m3::gated_workspace_bytes(d->batch, d->seqlen, d->width, packed, false))
    return M3_ERR_WORKSPACE;
  m3::GatedArgs g = gated_args(d);
  g.cu = cu_seqlens;
  g.x = x;
  g.r = r;
  g.i = i;
  g.decay = decay;
  g.h0 = h0;
  g.y = y;
  g.hT = hT;
  g.states = states;
  m3::gated_carve(g, false, ws);
  return hip_status(m3::launch_gated_scan(g, d->dtype == M3_BF16, static_cast<hipStream_t>(stream)));
}

m3_status m3_gated_scan_backward(const m3_gated_dims* d, const int32_t* cu_seqlens, const void* x,
                                 const void* r, const void* i, const float* decay, const float* h0,
                                 const float* states, const void* dy, const float* dhT, void* dx,
                                 void* dr, void* di, float* ddecay, float* dh0, void* ws,
                                 size_t ws_bytes, void* stream) {
  const bool packed = cu_seqlens != nullptr;
  m3_status st = check_gated(d, true, packed);
  if (st != M3_OK) return st;
  if (!x || !r || !i || !decay || !states || !dy || !dx || !dr || !di || !ddecay)
    return M3_ERR_NULL;
  const void* const ptrs[] = {x, r, i, decay, h0, states, dy, dhT, dx, dr, di, ddecay, dh0, ws};
  if (any_misaligned(ptrs) || misaligned4(cu_seqlens)) return M3_ERR_ALIGN;
  if (!ws || ws_bytes < m3::gated_workspace_bytes(d->batch, d->seqlen, d->width, packed, true))
    return M3_ERR_WORKSPACE;
  m3::GatedArgs g = gated_args(d);
  g.cu = cu_seqlens;
  g.x = x;
  g.r = r;
  g.i = i;
  g.decay = decay;
  g.h0 = h0;
  g.cstates = states;
  g.dy = dy;
  g.dhT = dhT;
  g.dx = dx;
  g.dr = dr;
  g.di = di;
  g.ddecay = ddecay;
  g.dh0 = dh0;
  m3::gated_carve(g, true, ws);
  return hip_status(
      m3::launch_gated_backward(g, d->dtype == M3_BF16, static_cast<hipStream_t>(stream)));
}

m3_status m3_gated_step(const m3_gated_dims* d, float* h, const void* x, const void* r,
                        const void* i, const float* decay, void* y, void* stream) {
  m3_status st = check_gated(d, false, false);
  if (st != M3_OK) return st;
  if (!h || !x || !r || !i || !decay || !y) return M3_ERR_NULL;
  const void* const ptrs[] = {h, x, r, i, decay, y};
  if (any_misaligned(ptrs)) return M3_ERR_ALIGN;
  m3::GatedArgs g = gated_args(d);
  g.x = x;
  g.r = r;
  g.i = i;
  g.decay = decay;
  g.y = y;
  return hip_status(m3::launch_gated_step(g, h, d->dtype == M3_BF16, static_cast<hipStream_t>(stream)));
}

m3_status m3_qk_norm_rope(const m3_qk_dims* d, const void* q, const void* k, const float* q_weight,
                          const float* k_weight, const int32_t* positions, void* q_out, void* k_out,
                          void* stream) {
  m3_status st = check_qk(d);
  if (st != M3_OK) return st;
  if (!q || !k || !positions || !q_out || !k_out) return M3_ERR_NULL;
  const void* const ptrs[] = {q, k, q_weight, k_weight, q_out, k_out};
  if (any_misaligned(ptrs) || misaligned4(positions)) return M3_ERR_ALIGN;
  m3::QkNormArgs a = qk_args(d);
  a.q = q;
  a.k = k;
  a.wq = q_weight;
  a.wk = k_weight;
  a.pos = positions;
  a.qo = q_out;
  a.ko = k_out;
  return hip_status(m3::launch_qk_norm(a, d->dtype == M3_BF16, static_cast<hipStream_t>(stream)));
}

size_t m3_qk_norm_rope_backward_workspace_size(const m3_qk_dims* d) {
  if (check_qk(d) != M3_OK) return 0;
  return m3::qk_norm_workspace_bytes(d->tokens, d->nheads_q, d->nheads_k, d->headdim);
}

m3_status m3_qk_norm_rope_backward(const m3_qk_dims* d, const void* q, const void* k,
                                   const float* q_weight, const float* k_weight,
                                   const int32_t* positions, const void* dq_out, const void* dk_out,
                                   void* dq, void* dk, float* dq_weight, float* dk_weight, void* ws,
                                   size_t ws_bytes, void* stream) {
  m3_status st = check_qk(d);
  if (st != M3_OK) return st;
  if (!q || !k || !positions || !dq_out || !dk_out || !dq || !dk) return M3_ERR_NULL;
  const void* const ptrs[] = {q, k, q_weight, k_weight, dq_out, dk_out, dq, dk, dq_weight, dk_weight, ws};
  if (any_misaligned(ptrs) || misaligned4(positions)) return M3_ERR_ALIGN;
  if (!ws || ws_bytes < m3::qk_norm_workspace_bytes(d->tokens, d->nheads_q, d->nheads_k, d->headdim))
    return M3_ERR_WORKSPACE;
  m3::QkNormArgs a = qk_args(d);
  a.q = q;
  a.k = k;
  a.wq = q_weight;
  a.wk = k_weight;
  a.pos = positions;
  a.gq = dq_out;
  a.gk = dk_out;
  a.dq = dq;
  a.dk = dk;
  a.dwq = dq_weight;
  a.dwk = dk_weight;
  a.part = static_cast<float*>(ws);
  return hip_status(
      m3::launch_qk_norm_backward(a, d->dtype == M3_BF16, static_cast<hipStream_t>(stream)));
}

size_t m3_attn_prefill_varlen_workspace_size(const m3_attn_dims* d) {
  if (check_attn(d, false) != M3_OK) return 0;
  const size_t n = m3::attn_workspace_bytes(d->tokens_q, d->tokens_k, d->nseq, d->nheads_q,
                                            d->nheads_k, d->headdim, d->dtype == M3_BF16);
  return n ? n : 16;
}

m3_status m3_attn_prefill_varlen(const m3_attn_dims* d, const int32_t* cu_seqlens_q,
                                 const int32_t* cu_seqlens_k, const void* q, const void* k,
                                 const void* v, void* o, float* lse, void* ws, size_t ws_bytes,
                                 void* stream) {
  m3_status st = check_attn(d, false);
  if (st != M3_OK) return st;
  if (!cu_seqlens_q || !cu_seqlens_k || !q || !k || !v || !o) return M3_ERR_NULL;
  const void* const ptrs[] = {q, k, v, o, lse, ws};
  if (any_misaligned(ptrs) || misaligned4(cu_seqlens_q) || misaligned4(cu_seqlens_k))
    return M3_ERR_ALIGN;
  const size_t need = m3::attn_workspace_bytes(d->tokens_q, d->tokens_k, d->nseq, d->nheads_q,
                                               d->nheads_k, d->headdim, d->dtype == M3_BF16);
  if (need && (!ws || ws_bytes < need)) return M3_ERR_WORKSPACE;
  m3::AttnArgs a = attn_args(d);
  a.cuq = cu_seqlens_q;
  a.cuk = cu_seqlens_k;
  a.q = q;
  a.k = k;
  a.v = v;
  a.o = o;
  a.lse = lse;
  return hip_status(m3::launch_attn(a, d->dtype == M3_BF16, ws, static_cast<hipStream_t>(stream)));
}

size_t m3_attn_prefill_varlen_backward_workspace_size(const m3_attn_dims* d) {
  if (check_attn(d, false) != M3_OK) return 0;
  return m3::attn_backward_workspace_bytes(d->tokens_q, d->tokens_k, d->nseq, d->nheads_q,
                                           d->nheads_k, d->headdim);
}

m3_status m3_attn_prefill_varlen_backward(const m3_attn_dims* d, const int32_t* cu_seqlens_q,
                                          const int32_t* cu_seqlens_k, const void* q, const void* k,
                                          const void* v, const void* o, const float* lse,
                                          const void* d_o, void* dq, void* dk, void* dv, void* ws,
                                          size_t ws_bytes, void* stream) {
  m3_status st = check_attn(d, false);
  if (st != M3_OK) return st;
  if (!cu_seqlens_q || !cu_seqlens_k || !q || !k || !v || !o || !lse || !d_o || !dq || !dk || !dv)
    return M3_ERR_NULL;
  const void* const ptrs[] = {q, k, v, o, lse, d_o, dq, dk, dv, ws};
  if (any_misaligned(ptrs) || misaligned4(cu_seqlens_q) || misaligned4(cu_seqlens_k))
    return M3_ERR_ALIGN;
  if (!ws || ws_bytes < m3::attn_backward_workspace_bytes(d->tokens_q, d->tokens_k, d->nseq,
                                                          d->nheads_q, d->nheads_k, d->headdim))
    return M3_ERR_WORKSPACE;
  m3::AttnArgs a = attn_args(d);
  a.cuq = cu_seqlens_q;
  a.cuk = cu_seqlens_k;
  a.q = q;
  a.k = k;
  a.v = v;
  a.co = o;
  a.clse = lse;
  a.dout = d_o;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  return hip_status(
      m3::launch_attn_backward(a, d->dtype == M3_BF16, ws, static_cast<hipStream_t>(stream)));
}

size_t m3_attn_decode_workspace_size(const m3_attn_dims* d) {
  if (check_attn(d, true) != M3_OK) return 0;
  const size_t n = m3::attn_decode_workspace_bytes(d->nseq, d->tokens_k, d->nheads_q, d->nheads_k,
                                                   d->headdim);
  return n ? n : 16;
}

m3_status m3_attn_decode(const m3_attn_dims* d, const int32_t* lengths, const void* q,
                         const void* k, const void* v, void* o, float* lse, void* ws,
                         size_t ws_bytes, void* stream) {
  m3_status st = check_attn(d, true);
  if (st != M3_OK) return st;
  if (!lengths || !q || !k || !v || !o) return M3_ERR_NULL;
  const void* const ptrs[] = {q, k, v, o, lse, ws};
  if (any_misaligned(ptrs) || misaligned4(lengths)) return M3_ERR_ALIGN;
  const size_t need = m3::attn_decode_workspace_bytes(d->nseq, d->tokens_k, d->nheads_q,
                                                      d->nheads_k, d->headdim);
  if (need && (!ws || ws_bytes < need)) return M3_ERR_WORKSPACE;
  m3::AttnArgs a = attn_args(d);
  a.len = lengths;
  a.q = q;
  a.k = k;
  a.v = v;
  a.o = o;
  a.lse = lse;
  return hip_status(m3::launch_attn_decode(a, d->dtype == M3_BF16, ws, static_cast<hipStream_t>(stream)));
}

size_t m3_delta_scan_workspace_size(const m3_delta_dims* d, int packed) {
  if (check_delta(d, true, packed != 0) != M3_OK) return 0;
  return m3::delta_workspace_bytes(d->batch, d->seqlen, d->nheads_v, d->headdim_k, d->headdim_v,
                                   packed != 0);
}

m3_status m3_delta_scan(const m3_delta_dims* d, const int32_t* cu_seqlens, const void* q,
                        const void* k, const void* v, const void* g, const void* beta,
                        const float* h0, void* o, float* hT, float* states, void* ws,
                        size_t ws_bytes, void* stream) {
  const bool packed = cu_seqlens != nullptr;
  m3_status st = check_delta(d, true, packed);
  if (st != M3_OK) return st;
  if (!q || !k || !v || !g || !beta || !o) return M3_ERR_NULL;
  const void* const ptrs[] = {q, k, v, h0, o, hT, states, ws};
  if (any_misaligned(ptrs) || misaligned4(cu_seqlens) || misaligned_gates(d, g, beta)) return M3_ERR_ALIGN;
  if (!ws || ws_bytes < m3::delta_workspace_bytes(d->batch, d->seqlen, d->nheads_v, d->headdim_k,
                                                  d->headdim_v, packed))
    return M3_ERR_WORKSPACE;
  m3::DeltaArgs a = delta_args(d);
  a.cu = cu_seqlens;
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.beta = beta;
  a.h0 = h0;
  a.o = o;
  a.hT = hT;
  a.states = states;
  m3::delta_carve(a, ws);
  return hip_status(m3::launch_delta_scan(a, d->dtype == M3_BF16, static_cast<hipStream_t>(stream)));
}

size_t m3_delta_scan_backward_workspace_size(const m3_delta_dims* d, int packed) {
  if (check_delta(d, true, packed != 0) != M3_OK) return 0;
  return m3::delta_backward_workspace_bytes(d->batch, d->seqlen, d->nheads_v, d->headdim_k,
                                            d->headdim_v, packed != 0);
}

m3_status m3_delta_scan_backward(const m3_delta_dims* d, const int32_t* cu_seqlens, const void* q,
                                 const void* k, const void* v, const void* g, const void* beta,
                                 const float* states, const void* d_o, const float* dhT, void* dq,
                                 void* dk, void* dv, void* dg, void* dbeta, float* dh0, void* ws,
                                 size_t ws_bytes, void* stream) {
  const bool packed = cu_seqlens != nullptr;
  m3_status st = check_delta(d, true, packed);
  if (st != M3_OK) return st;
  if (!q || !k || !v || !g || !beta || !states || !d_o || !dq || !dk || !dv || !dg || !dbeta)
    return M3_ERR_NULL;
  const void* const ptrs[] = {q, k, v, states, d_o, dhT, dq, dk, dv, dg, dbeta, dh0, ws};
  if (any_misaligned(ptrs) || misaligned4(cu_seqlens) || misaligned_gates(d, g, beta)) return M3_ERR_ALIGN;
  if (!ws || ws_bytes < m3::delta_backward_workspace_bytes(d->batch, d->seqlen, d->nheads_v,
                                                           d->headdim_k, d->headdim_v, packed))
    return M3_ERR_WORKSPACE;
  m3::DeltaArgs a = delta_args(d);
  a.cu = cu_seqlens;
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.beta = beta;
  a.cstates = states;
  a.dout = d_o;
  a.dhT = dhT;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.dg = dg;
  a.dbeta = dbeta;
  a.dh0 = dh0;
  m3::delta_backward_carve(a, ws);
  return hip_status(
      m3::launch_delta_backward(a, d->dtype == M3_BF16, static_cast<hipStream_t>(stream)));
}

m3_status m3_delta_step(const m3_delta_dims* d, float* h, const void* q, const void* k,
                        const void* v, const void* g, const void* beta, void* o, void* stream) {
  m3_status st = check_delta(d, false, false);
  if (st != M3_OK) return st;
  if (!h || !q || !k || !v || !g || !beta || !o) return M3_ERR_NULL;
  const void* const ptrs[] = {h, q, k, v, o};
  if (any_misaligned(ptrs) || misaligned_gates(d, g, beta)) return M3_ERR_ALIGN;
  m3::DeltaArgs a = delta_args(d);
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.beta = beta;
  a.o = o;
  return hip_status(m3::launch_delta_step(a, h, d->dtype == M3_BF16, static_cast<hipStream_t>(stream)));
}

m3_status m3_block_norm(const m3_block_dims* d, const void* x, const void* y, const void* gate,
                        const float* y_weight, const float* scale, const float* n_weight, void* h,
                        void* n, void* stream) {
  m3_status st = check_block(d);
  if (st != M3_OK) return st;
  if (!x || !y || !h) return M3_ERR_NULL;
  const void* const ptrs[] = {x, y, gate, y_weight, scale, n_weight, h, n};
  if (any_misaligned(ptrs)) return M3_ERR_ALIGN;
  m3::BlockNormArgs a = block_args(d);
  a.x = x;
  a.y = y;
  a.gate = gate;
  a.wy = y_weight;
  a.scale = scale;
  a.wn = n_weight;
  a.h = h;
  a.n = n;
  return hip_status(m3::launch_block_norm(a, d->dtype == M3_BF16, static_cast<hipStream_t>(stream)));
}

size_t m3_block_norm_backward_workspace_size(const m3_block_dims* d) {
  if (check_block(d) != M3_OK) return 0;
  return m3::block_norm_workspace_bytes(d->tokens, d->width);
}

m3_status m3_block_norm_backward(const m3_block_dims* d, const void* x, const void* y,
                                 const void* gate, const float* y_weight, const float* scale,
                                 const float* n_weight, const void* dh, const void* dn, void* dx,
                                 void* dy, void* dgate, float* dy_weight, float* dscale,
                                 float* dn_weight, void* ws, size_t ws_bytes, void* stream) {
  m3_status st = check_block(d);
  if (st != M3_OK) return st;
  if (!x || !y || (!dh && !dn) || !dx || !dy || (gate && !dgate)) return M3_ERR_NULL;
  const void* const ptrs[] = {x,  y,  gate,  y_weight,  scale,  n_weight,  dh, dn,
                              dx, dy, dgate, dy_weight, dscale, dn_weight, ws};
  if (any_misaligned(ptrs)) return M3_ERR_ALIGN;
  if (!ws || ws_bytes < m3::block_norm_workspace_bytes(d->tokens, d->width)) return M3_ERR_WORKSPACE;
  m3::BlockNormArgs a = block_args(d);
  a.x = x;
  a.y = y;
  a.gate = gate;
  a.wy = y_weight;
  a.scale = scale;
  a.wn = n_weight;
  a.dh = dh;
  a.dn = dn;
  a.dx = dx;
  a.dy = dy;
  a.dgate = dgate;
  a.dwy = dy_weight;
  a.dscale = dscale;
  a.dwn = dn_weight;
  a.part = static_cast<float*>(ws);
  return hip_status(
      m3::launch_block_norm_backward(a, d->dtype == M3_BF16, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
