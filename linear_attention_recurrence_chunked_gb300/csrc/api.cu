// api.cu -- the extern "C" entry points declared in include/la.h.
//
// Host side only: argument validation (before anything is launched), the
// N == 0 state pass-through, and dispatch to the kernel launchers.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "kernels.h"
#include "la.h"

namespace la {
namespace {
thread_local int t_last_cuda_error = 0;
}  // namespace
void note_cuda_error(int code) { t_last_cuda_error = code; }
int last_cuda_error() { return t_last_cuda_error; }
}  // namespace la

namespace {

// Device status word set by bounded waits that expire (LA_ERR_TIMEOUT).
__device__ unsigned g_la_device_status = 0;

unsigned* device_status_ptr() {
  void* p = nullptr;
  if (cudaGetSymbolAddress(&p, g_la_device_status) != cudaSuccess) return nullptr;
  return static_cast<unsigned*>(p);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int elem_bytes(la_dtype t) { return t == LA_DTYPE_BF16 ? 2 : 4; }

bool valid_dtype(la_dtype t) { return t == LA_DTYPE_F32 || t == LA_DTYPE_BF16; }

// A [B,H,N,d] view: non-null (unless empty), 16-byte aligned base and token
// stride, non-negative strides, and rows that do not overlap along t.
bool valid_view(const la_tensor& x, int64_t B, int64_t H, int64_t N, int64_t d, la_dtype dt) {
  if (B * H * N == 0) return true;
  if (x.ptr == nullptr || !aligned16(x.ptr)) return false;
  if (x.stride_b < 0 || x.stride_h < 0 || x.stride_t < 0) return false;
  if (N > 1 && x.stride_t < d) return false;
  if ((x.stride_t * elem_bytes(dt)) % 16 != 0) return false;
  if ((x.stride_h * elem_bytes(dt)) % 16 != 0 || (x.stride_b * elem_bytes(dt)) % 16 != 0) return false;
  return true;
}

bool valid_gate(const la_tensor& x, int64_t B, int64_t H, int64_t N) {
  if (B * H * N == 0) return true;
  if (x.ptr == nullptr || (reinterpret_cast<uintptr_t>(x.ptr) & 3u) != 0) return false;
  if (x.stride_b < 0 || x.stride_h < 0) return false;
  return x.stride_t == 1;
}

la::View4 view(const la_tensor& x) { return la::View4{x.ptr, x.stride_b, x.stride_h, x.stride_t}; }

la_status from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return LA_OK;
  la::note_cuda_error((int)e);
  return LA_ERR_CUDA;
}

// N == 0: the final state is the initial state (or zero).
la_status pass_state(float* out, const float* in, size_t n_floats, cudaStream_t s) {
  if (n_floats == 0) return LA_OK;
  if (in == out) return LA_OK;
  const size_t bytes = n_floats * sizeof(float);
  if (in) return from_cuda(cudaMemcpyAsync(out, in, bytes, cudaMemcpyDeviceToDevice, s));
  return from_cuda(cudaMemsetAsync(out, 0, bytes, s));
}

constexpr int64_t kTaylorF = 16, kTaylorDv = 64, kTaylorD = 1 + 16 + 16 * 16;
constexpr int64_t kGdnD = 128;
constexpr int64_t kMaxDim = int64_t(1) << 40;
constexpr int64_t kMaxElems = int64_t(1) << 44;  // elements of one state array (64 TiB of fp32)

la_status check_based(const la_based_prefill_args* a) {
  if (!a) return LA_ERR_INVALID_ARGUMENT;
  if (a->B < 0 || a->H < 0 || a->N < 0 || a->B > kMaxDim || a->H > kMaxDim || a->N > kMaxDim)
    return LA_ERR_INVALID_ARGUMENT;
  if (!valid_dtype(a->in_dtype) || !valid_dtype(a->out_dtype)) return LA_ERR_INVALID_ARGUMENT;
  if (a->d_feat != kTaylorF || a->d_v != kTaylorDv) return LA_ERR_UNSUPPORTED;
  if (a->B * a->H > (int64_t(1) << 31) - 1) return LA_ERR_UNSUPPORTED;
  if (a->N > INT32_MAX - 128) return LA_ERR_UNSUPPORTED;  // tile coordinates are 32-bit
  const int64_t B = a->B, H = a->H, N = a->N;
  if (!valid_view(a->q, B, H, N, kTaylorF, a->in_dtype) || !valid_view(a->k, B, H, N, kTaylorF, a->in_dtype) ||
      !valid_view(a->v, B, H, N, kTaylorDv, a->in_dtype) || !valid_view(a->y, B, H, N, kTaylorDv, a->out_dtype))
    return LA_ERR_INVALID_ARGUMENT;
  if (B * H > 0) {
    if (!a->s_out || !a->z_out) return LA_ERR_INVALID_ARGUMENT;
    if (!aligned16(a->s_out) || !aligned16(a->s_in) || (reinterpret_cast<uintptr_t>(a->z_out) & 3u) ||
        (reinterpret_cast<uintptr_t>(a->z_in) & 3u) || (reinterpret_cast<uintptr_t>(a->decay) & 3u))
      return LA_ERR_INVALID_ARGUMENT;
  }
  return LA_OK;
}

la_status check_gdn(const la_gdn_prefill_args* a) {
  if (!a) return LA_ERR_INVALID_ARGUMENT;
  if (a->B < 0 || a->H < 0 || a->N < 0 || a->B > kMaxDim || a->H > kMaxDim || a->N > kMaxDim)
    return LA_ERR_INVALID_ARGUMENT;
  if (!valid_dtype(a->in_dtype) || !valid_dtype(a->out_dtype)) return LA_ERR_INVALID_ARGUMENT;
  if (a->d_k != kGdnD || a->d_v != kGdnD) return LA_ERR_UNSUPPORTED;
  if (a->B * a->H > (int64_t(1) << 28)) return LA_ERR_UNSUPPORTED;
  if (a->N > INT32_MAX - 128) return LA_ERR_UNSUPPORTED;  // tile coordinates are 32-bit
  const int64_t B = a->B, H = a->H, N = a->N;
  if (!valid_view(a->q, B, H, N, kGdnD, a->in_dtype) || !valid_view(a->k, B, H, N, kGdnD, a->in_dtype) ||
      !valid_view(a->v, B, H, N, kGdnD, a->in_dtype) || !valid_view(a->o, B, H, N, kGdnD, a->out_dtype))
    return LA_ERR_INVALID_ARGUMENT;
  if (!valid_gate(a->alpha, B, H, N) || !valid_gate(a->beta, B, H, N)) return LA_ERR_INVALID_ARGUMENT;
  if (B * H > 0) {
    if (!a->S_out || !aligned16(a->S_out) || !aligned16(a->S_in)) return LA_ERR_INVALID_ARGUMENT;
  }
  return LA_OK;
}

}  // namespace

namespace {

// The GDN-family prefill: delta = 1 is the gated delta rule, delta = 0 the
// scalar gate A_t = alpha_t I; both share validation, workspace and kernels.
la_status gdn_family_prefill(const la_gdn_prefill_args* a, void* ws, size_t ws_bytes, void* stream, float delta) {
  const la_status st = check_gdn(a);
  if (st != LA_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t BH = a->B * a->H;
  if (BH == 0) return LA_OK;
  if (a->N == 0) return pass_state(a->S_out, a->S_in, (size_t)(BH * kGdnD * kGdnD), s);
  // bf16: the two-kernel scan when the workspace holds its per-chunk inverse
  // records, else the single-kernel scan, which needs the segment scratch only
  bool split = false;
  if (a->in_dtype == LA_DTYPE_BF16) {
    if (ws != nullptr && !aligned16(ws)) return LA_ERR_WORKSPACE;
    const int64_t nch = (a->N + 63) / 64;
    split = ws != nullptr && ws_bytes >= la::gdn_scan_workspace_bytes(a->B, a->H, a->N) && BH * nch <= INT32_MAX;
    const size_t need_min = la::gdn_segment_plan(a->B, a->H, a->N).ws_bytes;
    if (!split && need_min > 0 && (ws == nullptr || ws_bytes < need_min)) return LA_ERR_WORKSPACE;
  }
  la::GdnPrefillLaunch L{};
  L.B = a->B; L.H = a->H; L.N = a->N;
  L.in_bf16 = a->in_dtype == LA_DTYPE_BF16;
  L.out_bf16 = a->out_dtype == LA_DTYPE_BF16;
  L.q = view(a->q); L.k = view(a->k); L.v = view(a->v);
  L.o = a->o.ptr; L.o_sb = a->o.stride_b; L.o_sh = a->o.stride_h; L.o_st = a->o.stride_t;
  L.alpha = static_cast<const float*>(a->alpha.ptr); L.a_sb = a->alpha.stride_b; L.a_sh = a->alpha.stride_h;
  L.beta = static_cast<const float*>(a->beta.ptr); L.b_sb = a->beta.stride_b; L.b_sh = a->beta.stride_h;
  L.q_scale = a->q_scale;
  L.S_in = a->S_in; L.S_out = a->S_out;
  L.delta = delta;
  if (!L.in_bf16) return from_cuda(la::launch_gdn_prefill_recurrent(L, s));
  unsigned* status = device_status_ptr();
  if (!status) return LA_ERR_CUDA;
  const cudaError_t e = split ? la::launch_gdn_prefill_scan(L, ws, ws_bytes, status, s)
                              : la::launch_gdn_prefill_chunked(L, ws, ws_bytes, status, s);
  if (e == cudaErrorInvalidValue) return LA_ERR_UNSUPPORTED;  // strides TMA cannot describe
  return from_cuda(e);
}

}  // namespace

extern "C" {

int la_abi_version(void) { return LA_ABI_VERSION; }

int la_last_cuda_error(void) { return la::last_cuda_error(); }

const char* la_cuda_error_name(int code) {
  const char* n = cudaGetErrorName(static_cast<cudaError_t>(code));
  return n ? n : "unknown CUDA error";
}

const char* la_status_string(la_status s) {
  switch (s) {
    case LA_OK: return "ok";
    case LA_ERR_INVALID_ARGUMENT: return "invalid argument (null pointer, size, stride or alignment)";
    case LA_ERR_UNSUPPORTED: return "unsupported shape or dtype for the built kernels";
    case LA_ERR_WORKSPACE: return "workspace missing or too small";
    case LA_ERR_CUDA: return "CUDA call failed";
    case LA_ERR_TIMEOUT: return "a bounded device-side wait expired";
  }
  return "unknown status";
}

// The workspace queries depend on the problem's sizes and dtypes only (no
// pointer is inspected), so they may be asked before any buffer exists.
size_t la_based_prefill_workspace_size(const la_based_prefill_args* a) {
  (void)a;
  return 0;
}

// bf16 GDN problems the chunked kernels take (the fp32 path needs no scratch)
static bool gdn_chunked_shape(const la_gdn_prefill_args* a) {
  if (!a || a->B <= 0 || a->H <= 0 || a->N <= 0 || a->B > kMaxDim || a->H > kMaxDim || a->N > kMaxDim) return false;
  return a->d_k == kGdnD && a->d_v == kGdnD && a->in_dtype == LA_DTYPE_BF16;
}

size_t la_gdn_prefill_workspace_size(const la_gdn_prefill_args* a) {
  return gdn_chunked_shape(a) ? la::gdn_scan_workspace_bytes(a->B, a->H, a->N) : 0;
}

size_t la_gdn_prefill_workspace_size_min(const la_gdn_prefill_args* a) {
  return gdn_chunked_shape(a) ? la::gdn_segment_plan(a->B, a->H, a->N).ws_bytes : 0;
}

la_status la_based_prefill(const la_based_prefill_args* a, void* ws, size_t ws_bytes, void* stream) {
  const la_status st = check_based(a);
  if (st != LA_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t BH = a->B * a->H;
  if (BH == 0) return LA_OK;
  if (a->N == 0) {
    la_status r = pass_state(a->s_out, a->s_in, (size_t)(BH * kTaylorD * kTaylorDv), s);
    if (r != LA_OK) return r;
    return pass_state(a->z_out, a->z_in, (size_t)(BH * kTaylorD), s);
  }
  (void)ws;
  (void)ws_bytes;
  la::TaylorPrefillLaunch L{};
  L.B = a->B; L.H = a->H; L.N = a->N;
  L.in_bf16 = a->in_dtype == LA_DTYPE_BF16;
  L.out_bf16 = a->out_dtype == LA_DTYPE_BF16;
  L.q = view(a->q); L.k = view(a->k); L.v = view(a->v);
  L.y = a->y.ptr; L.y_sb = a->y.stride_b; L.y_sh = a->y.stride_h; L.y_st = a->y.stride_t;
  L.s_in = a->s_in; L.z_in = a->z_in; L.s_out = a->s_out; L.z_out = a->z_out;
  L.eps = a->eps;
  L.decay = a->decay;
  if (!L.in_bf16) return from_cuda(la::launch_taylor_prefill_recurrent(L, s));
  unsigned* status = device_status_ptr();
  if (!status) return LA_ERR_CUDA;
  const cudaError_t e = la::launch_taylor_prefill_chunked(L, status, s);
  if (e == cudaErrorInvalidValue) return LA_ERR_UNSUPPORTED;  // strides TMA cannot describe
  return from_cuda(e);
}


la_status la_gdn_prefill(const la_gdn_prefill_args* a, void* ws, size_t ws_bytes, void* stream) {
  return gdn_family_prefill(a, ws, ws_bytes, stream, 1.f);
}

la_status la_gated_prefill(const la_gdn_prefill_args* a, void* ws, size_t ws_bytes, void* stream) {
  return gdn_family_prefill(a, ws, ws_bytes, stream, 0.f);
}

la_status la_decode_step(const la_decode_args* a, void* stream) {
  if (!a) return LA_ERR_INVALID_ARGUMENT;
  if (a->S < 0 || a->H < 0 || a->S > kMaxDim || a->H > kMaxDim) return LA_ERR_INVALID_ARGUMENT;
  if (!valid_dtype(a->in_dtype) || !valid_dtype(a->out_dtype)) return LA_ERR_INVALID_ARGUMENT;
  if (a->variant != LA_VARIANT_TAYLOR && a->variant != LA_VARIANT_GDN && a->variant != LA_VARIANT_GATED)
    return LA_ERR_INVALID_ARGUMENT;
  const bool gdn_family = a->variant != LA_VARIANT_TAYLOR;
  if (gdn_family && (a->d_k != kGdnD || a->d_v != kGdnD)) return LA_ERR_UNSUPPORTED;
  if (a->variant == LA_VARIANT_TAYLOR && (a->d_k != kTaylorF || a->d_v != kTaylorDv)) return LA_ERR_UNSUPPORTED;
  const int64_t SH = a->S * a->H;
  if (SH == 0) return LA_OK;
  if (SH > (int64_t(1) << 31) - 1) return LA_ERR_UNSUPPORTED;
  if (!a->q || !a->k || !a->v || !a->out || !a->state) return LA_ERR_INVALID_ARGUMENT;
  const int in_align = a->in_dtype == LA_DTYPE_BF16 ? 8 : 16;
  if ((reinterpret_cast<uintptr_t>(a->q) % in_align) || (reinterpret_cast<uintptr_t>(a->k) % in_align) ||
      (reinterpret_cast<uintptr_t>(a->v) % in_align) || !aligned16(a->state))
    return LA_ERR_INVALID_ARGUMENT;
  if (gdn_family && (!a->alpha || !a->beta)) return LA_ERR_INVALID_ARGUMENT;
  if (a->variant == LA_VARIANT_TAYLOR &&
      (!a->z || (reinterpret_cast<uintptr_t>(a->z) & 3u) || (reinterpret_cast<uintptr_t>(a->decay) & 3u)))
    return LA_ERR_INVALID_ARGUMENT;
  la::DecodeLaunch L{};
  L.S = a->S; L.H = a->H;
  L.in_bf16 = a->in_dtype == LA_DTYPE_BF16;
  L.out_bf16 = a->out_dtype == LA_DTYPE_BF16;
  L.q = a->q; L.k = a->k; L.v = a->v; L.alpha = a->alpha; L.beta = a->beta;
  L.out = a->out; L.state = a->state; L.z = a->z; L.eps = a->eps; L.q_scale = a->q_scale;
  L.delta = a->variant == LA_VARIANT_GDN ? 1.f : 0.f;
  L.decay = a->variant == LA_VARIANT_TAYLOR ? a->decay : nullptr;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return from_cuda(gdn_family ? la::launch_gdn_decode(L, s) : la::launch_taylor_decode(L, s));
}

la_status la_state_rescale(float* states, int64_t n_states, int64_t elems_per_state, const float* lambda,
                           float lambda_all, void* stream) {
  if (n_states < 0 || elems_per_state < 0 || n_states > kMaxDim || elems_per_state > kMaxDim ||
      (elems_per_state > 0 && n_states > kMaxElems / elems_per_state))
    return LA_ERR_INVALID_ARGUMENT;
  if (n_states == 0 || elems_per_state == 0) return LA_OK;
  if (!states || (reinterpret_cast<uintptr_t>(states) & 3u)) return LA_ERR_INVALID_ARGUMENT;
  if (lambda && (reinterpret_cast<uintptr_t>(lambda) & 3u)) return LA_ERR_INVALID_ARGUMENT;
  return from_cuda(la::launch_state_rescale(states, n_states, elems_per_state, lambda, lambda_all,
                                            static_cast<cudaStream_t>(stream)));
}

la_status la_state_gather(float* dst, const float* src, const int64_t* index, int64_t n_dst, int64_t n_src,
                          int64_t elems_per_state, void* stream) {
  if (n_dst < 0 || n_src < 0 || elems_per_state < 0 || n_dst > kMaxDim || n_src > kMaxDim ||
      elems_per_state > kMaxDim ||
      (elems_per_state > 0 && (n_dst > kMaxElems / elems_per_state || n_src > kMaxElems / elems_per_state)))
    return LA_ERR_INVALID_ARGUMENT;
  if (n_dst == 0 || elems_per_state == 0) return LA_OK;
  if (!dst || !src || !index) return LA_ERR_INVALID_ARGUMENT;
  if ((reinterpret_cast<uintptr_t>(dst) & 3u) || (reinterpret_cast<uintptr_t>(src) & 3u) ||
      (reinterpret_cast<uintptr_t>(index) & 7u))
    return LA_ERR_INVALID_ARGUMENT;
  const uintptr_t d0 = reinterpret_cast<uintptr_t>(dst), d1 = d0 + (uintptr_t)(n_dst * elems_per_state) * 4u;
  const uintptr_t s0 = reinterpret_cast<uintptr_t>(src), s1 = s0 + (uintptr_t)(n_src * elems_per_state) * 4u;
  if (d0 < s1 && s0 < d1) return LA_ERR_INVALID_ARGUMENT;  // overlapping arrays
  unsigned* status = device_status_ptr();
  if (!status) return LA_ERR_CUDA;
  return from_cuda(la::launch_state_gather(dst, src, index, n_dst, n_src, elems_per_state, status,
                                           static_cast<cudaStream_t>(stream)));
}

la_status la_swa_decode_step(const la_swa_decode_args* a, void* stream) {
  if (!a) return LA_ERR_INVALID_ARGUMENT;
  if (a->S < 0 || a->H < 0 || a->S > kMaxDim || a->H > kMaxDim) return LA_ERR_INVALID_ARGUMENT;
  if (!valid_dtype(a->in_dtype) || !valid_dtype(a->out_dtype)) return LA_ERR_INVALID_ARGUMENT;
  if (a->d < 8 || a->d > 128 || a->d % 8 != 0 || a->window < 1 || a->window > 256) return LA_ERR_UNSUPPORTED;
  const int64_t SH = a->S * a->H;
  if (SH == 0) return LA_OK;
  if (SH > (int64_t(1) << 31) - 1) return LA_ERR_UNSUPPORTED;
  if (!a->q || !a->k || !a->v || !a->k_cache || !a->v_cache || !a->pos || !a->out) return LA_ERR_INVALID_ARGUMENT;
  if (!aligned16(a->q) || !aligned16(a->k) || !aligned16(a->v) || !aligned16(a->k_cache) ||
      !aligned16(a->v_cache) || !aligned16(a->out) || (reinterpret_cast<uintptr_t>(a->pos) & 7u))
    return LA_ERR_INVALID_ARGUMENT;
  unsigned* status = device_status_ptr();
  if (!status) return LA_ERR_CUDA;
  la::SwaDecodeLaunch L{};
  L.S = a->S; L.H = a->H; L.d = (int)a->d; L.window = (int)a->window;
  L.in_bf16 = a->in_dtype == LA_DTYPE_BF16;
  L.out_bf16 = a->out_dtype == LA_DTYPE_BF16;
  L.q = a->q; L.k = a->k; L.v = a->v; L.k_cache = a->k_cache; L.v_cache = a->v_cache;
  L.pos = a->pos; L.out = a->out; L.scale = a->scale; L.status = status;
  return from_cuda(la::launch_swa_decode(L, static_cast<cudaStream_t>(stream)));
}

la_status la_notebank_scores(const la_notebank_scores_args* a, void* stream) {
  if (!a) return LA_ERR_INVALID_ARGUMENT;
  if (a->L < 0 || a->H < 0 || a->N < 0 || a->L > kMaxDim || a->H > kMaxDim || a->N > kMaxDim)
    return LA_ERR_INVALID_ARGUMENT;
  if (!valid_dtype(a->in_dtype)) return LA_ERR_INVALID_ARGUMENT;
  if (a->d < 32 || a->d > 256 || a->d % 32 != 0) return LA_ERR_UNSUPPORTED;
  if (a->chunk < 1 || a->chunk > 1024 || a->window < 1 || a->window > 4096) return LA_ERR_INVALID_ARGUMENT;
  const int64_t J = a->L * a->H;
  if (J == 0 || a->N == 0) return LA_OK;
  if (J * ((a->N + a->chunk - 1) / a->chunk) > (int64_t(1) << 31) - 1) return LA_ERR_UNSUPPORTED;
  if (!valid_view(a->k, a->L, a->H, a->N, a->d, a->in_dtype)) return LA_ERR_INVALID_ARGUMENT;
  if (!a->d_ch || !a->d_mean || (reinterpret_cast<uintptr_t>(a->d_ch) & 3u) ||
      (reinterpret_cast<uintptr_t>(a->d_mean) & 3u) || (reinterpret_cast<uintptr_t>(a->w) & 3u))
    return LA_ERR_INVALID_ARGUMENT;
  la::NotebankScoresLaunch L{};
  L.L = a->L; L.H = a->H; L.N = a->N; L.d = a->d;
  L.in_bf16 = a->in_dtype == LA_DTYPE_BF16;
  L.k = view(a->k);
  L.chunk = a->chunk; L.window = a->window;
  L.d_ch = a->d_ch; L.d_mean = a->d_mean; L.w = a->N >= a->window ? a->w : nullptr;
  return from_cuda(la::launch_notebank_scores(L, static_cast<cudaStream_t>(stream)));
}

la_status la_notebank_address(const la_notebank_address_args* a, void* stream) {
  if (!a) return LA_ERR_INVALID_ARGUMENT;
  if (a->L < 0 || a->H < 0 || a->N < 0 || a->n_notes < 0 || a->L > kMaxDim || a->H > kMaxDim || a->N > kMaxDim ||
      a->n_notes > kMaxDim)
    return LA_ERR_INVALID_ARGUMENT;
  if (!valid_dtype(a->in_dtype)) return LA_ERR_INVALID_ARGUMENT;
  if (a->d < la::kNoteAddrDims || a->d > kMaxDim) return LA_ERR_UNSUPPORTED;
  const int64_t warps = a->n_notes * a->L * a->H;
  if (warps == 0) return LA_OK;
  if (warps > (int64_t(1) << 33)) return LA_ERR_UNSUPPORTED;  // grid of warps * 32 / 256 blocks
  if (a->N == 0) return LA_ERR_INVALID_ARGUMENT;  // no token to point at
  if (!valid_view(a->q, a->L, a->H, a->N, a->d, a->in_dtype)) return LA_ERR_INVALID_ARGUMENT;
  if (!a->d_ch || !a->coords || !a->spans || !a->t_star || !a->rho || (reinterpret_cast<uintptr_t>(a->d_ch) & 3u) ||
      (reinterpret_cast<uintptr_t>(a->coords) & 3u) || (reinterpret_cast<uintptr_t>(a->spans) & 7u) ||
      (reinterpret_cast<uintptr_t>(a->t_star) & 3u) || (reinterpret_cast<uintptr_t>(a->rho) & 1u))
    return LA_ERR_INVALID_ARGUMENT;
  unsigned* status = device_status_ptr();
  if (!status) return LA_ERR_CUDA;
  la::NotebankAddressLaunch L{};
  L.L = a->L; L.H = a->H; L.N = a->N; L.d = a->d; L.n_notes = a->n_notes;
  L.in_bf16 = a->in_dtype == LA_DTYPE_BF16;
  L.q = view(a->q);
  L.d_ch = a->d_ch; L.coords = a->coords; L.spans = a->spans; L.t_star = a->t_star; L.rho = a->rho;
  return from_cuda(la::launch_notebank_address(L, status, static_cast<cudaStream_t>(stream)));
}

la_status la_notebank_route(const la_notebank_route_args* a, void* stream) {
  if (!a) return LA_ERR_INVALID_ARGUMENT;
  if (a->n_notes < 0 || a->J < 0 || a->n_notes > (int64_t(1) << 31) - 2 || a->J > kMaxDim)
    return LA_ERR_INVALID_ARGUMENT;
  if (a->n_q < 1 || a->n_q > 512 || a->R < 1 || a->R > 64) return LA_ERR_UNSUPPORTED;
  if (a->J == 0) return LA_OK;
  if (!a->u || !a->winner || !a->top || !aligned16(a->u) || (reinterpret_cast<uintptr_t>(a->winner) & 3u) ||
      (reinterpret_cast<uintptr_t>(a->top) & 3u))
    return LA_ERR_INVALID_ARGUMENT;
  if (a->n_notes > 0 && (!a->rho || !a->votes || !aligned16(a->rho) || (reinterpret_cast<uintptr_t>(a->votes) & 3u) ||
                         (reinterpret_cast<uintptr_t>(a->s) & 3u) || (reinterpret_cast<uintptr_t>(a->positions) & 7u)))
    return LA_ERR_INVALID_ARGUMENT;
  la::NotebankRouteLaunch L{};
  L.n_notes = a->n_notes; L.J = a->J; L.n_q = a->n_q; L.R = a->R;
  L.rho = a->rho; L.u = a->u; L.positions = a->positions; L.s = a->s;
  L.winner = a->winner; L.votes = a->votes; L.top = a->top;
  return from_cuda(la::launch_notebank_route(L, static_cast<cudaStream_t>(stream)));
}

namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

// Whether the product of sizes in [0, kMaxDim] stays within `limit`.
bool within(int64_t limit, std::initializer_list<int64_t> sizes) {
  int64_t p = 1;
  for (const int64_t s : sizes) {
    if (s == 0) return true;
    if (p > limit / s) return false;
    p *= s;
  }
  return true;
}
bool valid_size(int64_t s) { return s >= 0 && s <= kMaxDim; }

constexpr int64_t kMaxBlocks = (int64_t(1) << 31) - 1;  // of a launch's grid
// Whether the padding of [B, H, N] rows fits one launch (64 rows a block).
bool paddable(int64_t B, int64_t H, int64_t N) { return within(kMaxBlocks, {B, H, (N + 63) / 64}); }

// Whether no two elements of a [B, H, N, d] view lie on one another, for views whose axes nest in some order.
bool distinct(const la_tensor& x, int64_t B, int64_t H, int64_t N, int64_t d) {
  struct Axis { int64_t stride, size; } ax[3] = {{x.stride_b, B}, {x.stride_h, H}, {x.stride_t, N}};
  std::sort(ax, ax + 3, [](const Axis& a, const Axis& b) { return a.stride < b.stride; });
  int64_t extent = d;  // elements from the first to the last of what the smaller axes span
  for (const Axis& a : ax) {
    if (a.size == 0) return true;
    if (a.size == 1) continue;
    if (a.stride < extent || a.stride > (INT64_MAX - extent) / (a.size - 1)) return false;
    extent += a.stride * (a.size - 1);
  }
  return true;
}

// [B, N, C] view: as a [B, 1, N, C] one
bool valid_rows(la_tensor x, int64_t B, int64_t N, int64_t C, la_dtype dt, bool output) {
  x.stride_h = 0;
  return valid_view(x, B, 1, N, C, dt) && !(output && !distinct(x, B, 1, N, C));
}

// Zeros and incoming states for what a call with lens leaves out, as its `fill` asks for.
la_status fill_padding(int32_t fill, int64_t B, int64_t H, int64_t N, int64_t max_len, int64_t offset, const int64_t* lens, const la_tensor& y,
                       int64_t row, la_dtype dt, const void* state_in, void* state_out, int64_t state_bytes, cudaStream_t stream) {
  if (!lens || !(fill & (LA_FILL_ROWS | LA_FILL_STATE))) return LA_OK;
  const int64_t e = elem_bytes(dt);
  la::PaddingLaunch p{};
  p.B = B; p.H = H; p.N = N; p.max_len = max_len; p.offset = offset; p.lens = lens;
  p.rows = fill & LA_FILL_ROWS ? y.ptr : nullptr;
  p.sb = y.stride_b * e; p.sh = y.stride_h * e; p.st = y.stride_t * e; p.row_bytes = row * e;
  p.state_in = state_in; p.state_out = fill & LA_FILL_STATE ? state_out : nullptr; p.state_bytes = state_bytes;
  return from_cuda(la::launch_fill_padding(p, stream));
}

// 0, or a cap whose ratios to the scale and to log2(e) are far from fp32's ends
bool valid_cap(float softcap, float scale) {
  return softcap == 0.f || (softcap > 0.f && softcap <= 1e37f && std::fabs(scale / softcap) <= 1e37f);
}
bool valid_elem(const void* p, la_dtype dt) { return p && (reinterpret_cast<uintptr_t>(p) % elem_bytes(dt)) == 0; }
// strides of a bf16 view that a tensor map can hold: below 2^40 bytes
bool mappable(const la_tensor& x, int64_t B, int64_t H, int64_t N) {
  constexpr int64_t kEnd = int64_t(1) << 39;
  return (B <= 1 || x.stride_b < kEnd) && (H <= 1 || x.stride_h < kEnd) && (N <= 1 || x.stride_t < kEnd);
}
bool valid_strides(const la_tensor& x) { return x.stride_b >= 0 && x.stride_h >= 0 && x.stride_t >= 0; }

}  // namespace

la_status la_conv_prefill(const la_conv_prefill_args* a, void* stream) {
  if (!a) return LA_ERR_INVALID_ARGUMENT;
  if (!valid_size(a->B) || !valid_size(a->N) || !valid_size(a->C)) return LA_ERR_INVALID_ARGUMENT;
  if (!valid_dtype(a->in_dtype) || !valid_dtype(a->out_dtype) || !valid_dtype(a->w_dtype)) return LA_ERR_INVALID_ARGUMENT;
  if (a->W < 2 || a->W > 4) return LA_ERR_UNSUPPORTED;
  if (a->B == 0 || a->C == 0) return LA_OK;
  if (!within(kMaxBlocks * 256, {a->B, a->N + 1, a->C}) || !paddable(a->B, 1, a->N)) return LA_ERR_UNSUPPORTED;
  if (!valid_rows(a->x, a->B, a->N, a->C, a->in_dtype, false) || !valid_rows(a->y, a->B, a->N, a->C, a->out_dtype, true))
    return LA_ERR_INVALID_ARGUMENT;
  if (a->N > 0 && a->x.ptr == a->y.ptr) return LA_ERR_INVALID_ARGUMENT;  // a run's history may be overwritten
  if (!a->w || !a->state_out || !aligned16(a->w) || !aligned16(a->bias) || !aligned16(a->state_in) ||
      !aligned16(a->state_out) || !aligned8(a->lens))
    return LA_ERR_INVALID_ARGUMENT;
  unsigned* status = device_status_ptr();
  if (!status) return LA_ERR_CUDA;
  la::ConvLaunch L{};
  L.B = a->B; L.N = a->N; L.C = a->C; L.W = (int)a->W;
  L.in_bf16 = a->in_dtype == LA_DTYPE_BF16; L.out_bf16 = a->out_dtype == LA_DTYPE_BF16;
  L.w_bf16 = a->w_dtype == LA_DTYPE_BF16;
  L.x = a->x.ptr; L.x_sb = a->x.stride_b; L.x_st = a->x.stride_t;
  L.y = a->y.ptr; L.y_sb = a->y.stride_b; L.y_st = a->y.stride_t;
  L.w = a->w; L.bias = a->bias; L.state_in = a->state_in; L.state_out = a->state_out;
  L.lens = a->lens; L.silu = a->silu; L.status = status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  la_tensor y = a->y;
  y.stride_h = 0;
  const la_status st = fill_padding(a->fill, a->B, 1, a->N, a->N, 0, a->lens, y, a->C, a->out_dtype, a->state_in, a->state_out,
                                    (a->W - 1) * a->C * elem_bytes(a->in_dtype), s);
  return st != LA_OK ? st : from_cuda(la::launch_conv_prefill(L, s));
}

la_status la_conv_decode_step(const la_conv_decode_args* a, void* stream) {
  if (!a) return LA_ERR_INVALID_ARGUMENT;
  if (!valid_size(a->S) || !valid_size(a->C)) return LA_ERR_INVALID_ARGUMENT;
  if (!valid_dtype(a->in_dtype) || !valid_dtype(a->out_dtype) || !valid_dtype(a->w_dtype)) return LA_ERR_INVALID_ARGUMENT;
  if (a->W < 2 || a->W > 4) return LA_ERR_UNSUPPORTED;
  if (a->S == 0 || a->C == 0) return LA_OK;
  if (!within(kMaxBlocks * 256, {a->S, a->C})) return LA_ERR_UNSUPPORTED;
  const la_tensor x{const_cast<void*>(a->x), 0, 0, a->x_stride}, y{a->out, 0, 0, a->out_stride};
  if (!valid_rows(x, 1, a->S, a->C, a->in_dtype, false) || !valid_rows(y, 1, a->S, a->C, a->out_dtype, true))
    return LA_ERR_INVALID_ARGUMENT;
  if (!a->w || !a->state_in || !a->state_out || !aligned16(a->w) || !aligned16(a->bias) || !aligned16(a->state_in) ||
      !aligned16(a->state_out))
    return LA_ERR_INVALID_ARGUMENT;
  la::ConvLaunch L{};
  L.B = a->S; L.N = 1; L.C = a->C; L.W = (int)a->W;
  L.in_bf16 = a->in_dtype == LA_DTYPE_BF16; L.out_bf16 = a->out_dtype == LA_DTYPE_BF16;
  L.w_bf16 = a->w_dtype == LA_DTYPE_BF16;
  L.x = a->x; L.x_sb = a->x_stride;
  L.y = a->out; L.y_sb = a->out_stride;
  L.w = a->w; L.bias = a->bias; L.state_in = a->state_in; L.state_out = a->state_out;
  L.silu = a->silu;
  return from_cuda(la::launch_conv_decode(L, static_cast<cudaStream_t>(stream)));
}

static bool ssm_shape(const la_ssm_prefill_args* a) {
  return a && a->B > 0 && a->C > 0 && a->G > 0 && a->B <= 65535 && a->C % a->G == 0 && valid_size(a->N) && a->n >= 1 && a->n <= 64 &&
         a->C <= INT32_MAX / 64 && a->N <= INT32_MAX / 2 && within(kMaxElems, {a->B, a->C, a->n}) && within(kMaxElems, {a->B, a->N + 1, a->C});
}

size_t la_ssm_prefill_workspace_size(const la_ssm_prefill_args* a) {
  return ssm_shape(a) ? la::ssm_workspace_bytes(a->B, a->N, a->C, (int)a->n, a->G) : 0;
}

la_status la_ssm_prefill(const la_ssm_prefill_args* a, void* ws, size_t ws_bytes, void* stream) {
  if (!a) return LA_ERR_INVALID_ARGUMENT;
  if (!valid_size(a->B) || !valid_size(a->N) || !valid_size(a->C) || a->G < 1 || a->C % a->G != 0) return LA_ERR_INVALID_ARGUMENT;
  if (!valid_dtype(a->in_dtype) || !valid_dtype(a->out_dtype)) return LA_ERR_INVALID_ARGUMENT;
  if (a->n < 1 || a->n > 64) return LA_ERR_UNSUPPORTED;
  if (a->B == 0 || a->C == 0) return LA_OK;
  if (!ssm_shape(a) || !paddable(a->B, 1, a->N)) return LA_ERR_UNSUPPORTED;
  const int64_t B = a->B, N = a->N, C = a->C;
  if (!valid_rows(a->u, B, N, C, a->in_dtype, false) || !valid_rows(a->delta, B, N, C, a->in_dtype, false) ||
      (a->z.ptr && !valid_rows(a->z, B, N, C, a->in_dtype, false)) || !valid_rows(a->y, B, N, C, a->out_dtype, true))
    return LA_ERR_INVALID_ARGUMENT;
  if (N > 0 && (!valid_elem(a->Bm.ptr, a->in_dtype) || !valid_elem(a->Cm.ptr, a->in_dtype) || !valid_strides(a->Bm) || !valid_strides(a->Cm)))
    return LA_ERR_INVALID_ARGUMENT;
  if (!a->A || !a->h_out || !aligned4(a->A) || !aligned4(a->D) || !aligned4(a->delta_bias) || !aligned16(a->h_in) ||
      !aligned16(a->h_out) || !aligned8(a->lens))
    return LA_ERR_INVALID_ARGUMENT;
  const size_t need = la_ssm_prefill_workspace_size(a);
  if (need > 0 && (!ws || !aligned16(ws) || ws_bytes < need)) return LA_ERR_WORKSPACE;
  unsigned* status = device_status_ptr();
  if (!status) return LA_ERR_CUDA;
  la::SsmLaunch L{};
  L.B = B; L.N = N; L.C = C; L.G = a->G; L.n = (int)a->n;
  L.in_bf16 = a->in_dtype == LA_DTYPE_BF16; L.out_bf16 = a->out_dtype == LA_DTYPE_BF16;
  L.u = a->u.ptr; L.u_sb = a->u.stride_b; L.u_st = a->u.stride_t;
  L.delta = a->delta.ptr; L.d_sb = a->delta.stride_b; L.d_st = a->delta.stride_t;
  L.z = a->z.ptr; L.z_sb = a->z.stride_b; L.z_st = a->z.stride_t;
  L.y = a->y.ptr; L.y_sb = a->y.stride_b; L.y_st = a->y.stride_t;
  L.Bm = view(a->Bm); L.Cm = view(a->Cm);
  L.A = a->A; L.D = a->D; L.delta_bias = a->delta_bias; L.h_in = a->h_in; L.h_out = a->h_out;
  L.lens = a->lens; L.softplus = a->delta_softplus; L.status = status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  la_tensor y = a->y;
  y.stride_h = 0;
  const la_status st = fill_padding(a->fill, B, 1, N, N, 0, a->lens, y, C, a->out_dtype, a->h_in, a->h_out, C * a->n * (int64_t)sizeof(float), s);
  return st != LA_OK ? st : from_cuda(la::launch_ssm_prefill(L, ws, ws_bytes, s));
}

la_status la_ssm_decode_step(const la_ssm_decode_args* a, void* stream) {
  if (!a) return LA_ERR_INVALID_ARGUMENT;
  if (!valid_size(a->S) || !valid_size(a->C) || a->G < 1 || a->C % a->G != 0) return LA_ERR_INVALID_ARGUMENT;
  if (!valid_dtype(a->in_dtype) || !valid_dtype(a->out_dtype)) return LA_ERR_INVALID_ARGUMENT;
  if (a->n < 1 || a->n > 64) return LA_ERR_UNSUPPORTED;
  if (a->S == 0 || a->C == 0) return LA_OK;
  if (a->S > 4 * 65535 || a->C > INT32_MAX / 64 || !within(kMaxElems, {a->S, a->C, a->n})) return LA_ERR_UNSUPPORTED;
  for (const la_tensor* t : {&a->u, &a->delta, &a->Bm, &a->Cm})
    if (!valid_elem(t->ptr, a->in_dtype) || !valid_strides(*t)) return LA_ERR_INVALID_ARGUMENT;
  if (a->z.ptr && (!valid_elem(a->z.ptr, a->in_dtype) || !valid_strides(a->z))) return LA_ERR_INVALID_ARGUMENT;
  if (!valid_elem(a->out.ptr, a->out_dtype) || !valid_strides(a->out) || (a->S > 1 && a->out.stride_b < a->C))
    return LA_ERR_INVALID_ARGUMENT;
  if (!a->A || !a->state_in || !a->state_out || !aligned4(a->A) || !aligned4(a->D) || !aligned4(a->delta_bias) ||
      !aligned16(a->state_in) || !aligned16(a->state_out))
    return LA_ERR_INVALID_ARGUMENT;
  la::SsmLaunch L{};
  L.B = a->S; L.N = 1; L.C = a->C; L.G = a->G; L.n = (int)a->n;
  L.in_bf16 = a->in_dtype == LA_DTYPE_BF16; L.out_bf16 = a->out_dtype == LA_DTYPE_BF16;
  L.u = a->u.ptr; L.u_sb = a->u.stride_b;
  L.delta = a->delta.ptr; L.d_sb = a->delta.stride_b;
  L.z = a->z.ptr; L.z_sb = a->z.stride_b;
  L.y = a->out.ptr; L.y_sb = a->out.stride_b;
  L.Bm = view(a->Bm); L.Cm = view(a->Cm);
  L.A = a->A; L.D = a->D; L.delta_bias = a->delta_bias; L.h_in = a->state_in; L.h_out = a->state_out;
  L.softplus = a->delta_softplus;
  return from_cuda(la::launch_ssm_decode(L, static_cast<cudaStream_t>(stream)));
}

la_status la_swa_prefill(const la_swa_prefill_args* a, void* stream) {
  if (!a) return LA_ERR_INVALID_ARGUMENT;
  if (!valid_size(a->B) || !valid_size(a->H) || !valid_size(a->Nq) || !valid_size(a->Nk) || !valid_size(a->window) || a->H_kv < 1 ||
      a->H % a->H_kv != 0 || a->q_pos0 < 0 || a->q_pos0 > a->Nk || a->Nq > a->Nk - a->q_pos0)
    return LA_ERR_INVALID_ARGUMENT;
  if (!valid_dtype(a->in_dtype) || !valid_dtype(a->out_dtype)) return LA_ERR_INVALID_ARGUMENT;
  if (!valid_cap(a->softcap, a->scale) || (a->k_cache == nullptr) != (a->v_cache == nullptr))
    return LA_ERR_INVALID_ARGUMENT;
  if (a->d < 8 || a->d > 128 || a->d % 8 != 0) return LA_ERR_UNSUPPORTED;
  if (a->k_cache && (a->window < 1 || a->window > 256)) return LA_ERR_UNSUPPORTED;
  if (a->Nk > INT32_MAX - 512) return LA_ERR_UNSUPPORTED;  // key positions are 32-bit
  if (a->B == 0 || a->H == 0 || a->Nk == 0) return LA_OK;
  if (!within((int64_t(1) << 31) - 1024, {a->B, a->H, (a->Nq + 63) / 64}) ||
      (a->k_cache && !within((int64_t(1) << 34) - 8, {a->B, a->H_kv, a->window})))
    return LA_ERR_UNSUPPORTED;
  if (!valid_view(a->q, a->B, a->H, a->Nq, a->d, a->in_dtype) || !valid_view(a->k, a->B, a->H_kv, a->Nk, a->d, a->in_dtype) ||
      !valid_view(a->v, a->B, a->H_kv, a->Nk, a->d, a->in_dtype) || !valid_view(a->o, a->B, a->H, a->Nq, a->d, a->out_dtype))
    return LA_ERR_INVALID_ARGUMENT;
  if (!distinct(a->o, a->B, a->H, a->Nq, a->d)) return LA_ERR_INVALID_ARGUMENT;
  if (a->in_dtype == LA_DTYPE_BF16 && !(mappable(a->q, a->B, a->H, a->Nq) && mappable(a->k, a->B, a->H_kv, a->Nk) && mappable(a->v, a->B, a->H_kv, a->Nk)))
    return LA_ERR_UNSUPPORTED;
  if (!aligned4(a->slopes) || !aligned4(a->key_lo) || !aligned4(a->key_hi) || !aligned8(a->lens) || !aligned16(a->k_cache) ||
      !aligned16(a->v_cache))
    return LA_ERR_INVALID_ARGUMENT;
  unsigned* status = device_status_ptr();
  if (!status) return LA_ERR_CUDA;
  la::SwaPrefillLaunch L{};
  L.B = a->B; L.H = a->H; L.Hkv = a->H_kv; L.Nq = a->Nq; L.Nk = a->Nk; L.d = (int)a->d;
  L.window = a->window; L.q_pos0 = a->q_pos0;
  L.in_bf16 = a->in_dtype == LA_DTYPE_BF16; L.out_bf16 = a->out_dtype == LA_DTYPE_BF16;
  L.q = view(a->q); L.k = view(a->k); L.v = view(a->v);
  L.o = a->o.ptr; L.o_sb = a->o.stride_b; L.o_sh = a->o.stride_h; L.o_st = a->o.stride_t;
  L.scale = a->scale; L.softcap = a->softcap; L.slopes = a->slopes; L.key_lo = a->key_lo; L.key_hi = a->key_hi;
  L.lens = a->lens; L.k_cache = a->k_cache; L.v_cache = a->v_cache; L.status = status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->Nq > 0) {
    const la_status st = fill_padding(a->fill & LA_FILL_ROWS, a->B, a->H, a->Nq, a->Nk, a->q_pos0, a->lens, a->o, a->d, a->out_dtype, nullptr,
                                      nullptr, 0, s);
    if (st != LA_OK) return st;
    const cudaError_t e = L.in_bf16 ? la::launch_swa_prefill_tc(L, s) : la::launch_swa_prefill_simt(L, s);
    if (e != cudaSuccess) return from_cuda(e);
  }
  return a->k_cache ? from_cuda(la::launch_swa_fill_rings(L, s)) : LA_OK;
}

la_status la_swa_biased_decode_step(const la_swa_biased_decode_args* args, void* stream) {
  if (!args) return LA_ERR_INVALID_ARGUMENT;
  const la_swa_decode_args* a = &args->base;
  if (a->S < 0 || a->H < 0 || a->S > kMaxDim || a->H > kMaxDim || args->H_kv < 1 || a->H % args->H_kv != 0) return LA_ERR_INVALID_ARGUMENT;
  if (!valid_dtype(a->in_dtype) || !valid_dtype(a->out_dtype)) return LA_ERR_INVALID_ARGUMENT;
  if (!valid_cap(args->softcap, a->scale)) return LA_ERR_INVALID_ARGUMENT;
  if (a->d < 8 || a->d > 128 || a->d % 8 != 0 || a->window < 1 || a->window > 256 || a->H / args->H_kv > 16) return LA_ERR_UNSUPPORTED;
  if (a->S == 0 || a->H == 0) return LA_OK;
  if (!within((int64_t(1) << 31) - 1, {a->S, a->H})) return LA_ERR_UNSUPPORTED;
  if (!a->q || !a->k || !a->v || !a->k_cache || !a->v_cache || !a->pos || !a->out) return LA_ERR_INVALID_ARGUMENT;
  if (!aligned16(a->q) || !aligned16(a->k) || !aligned16(a->v) || !aligned16(a->k_cache) || !aligned16(a->v_cache) ||
      !aligned16(a->out) || !aligned8(a->pos) || !aligned4(args->slopes))
    return LA_ERR_INVALID_ARGUMENT;
  unsigned* status = device_status_ptr();
  if (!status) return LA_ERR_CUDA;
  la::SwaBiasedDecodeLaunch L{};
  L.base.S = a->S; L.base.H = a->H; L.base.d = (int)a->d; L.base.window = (int)a->window;
  L.base.in_bf16 = a->in_dtype == LA_DTYPE_BF16;
  L.base.out_bf16 = a->out_dtype == LA_DTYPE_BF16;
  L.base.q = a->q; L.base.k = a->k; L.base.v = a->v; L.base.k_cache = a->k_cache; L.base.v_cache = a->v_cache;
  L.base.pos = a->pos; L.base.out = a->out; L.base.scale = a->scale; L.base.status = status;
  L.Hkv = args->H_kv; L.softcap = args->softcap; L.slopes = args->slopes;
  return from_cuda(la::launch_swa_biased_decode(L, static_cast<cudaStream_t>(stream)));
}

// ---- queries' and keys' norms, paged caches

extern "C++" {
namespace {

// Rotation tables of `positions` rows for the first `rot` of d elements
bool valid_tables(const float* cos, const float* sin, int64_t rot, int64_t positions) {
  return rot == 0 || (cos && sin && aligned16(cos) && aligned16(sin) && positions >= 0 && positions <= kMaxDim);
}

template <typename Args>
la_status check_pages(const Args* a, int64_t B) {
  if (!valid_size(a->H_kv) || !valid_size(a->pages) || !valid_size(a->width) || !valid_dtype(a->in_dtype) || (a->bits != 0 && a->bits != 4))
    return LA_ERR_INVALID_ARGUMENT;
  if (a->bits == 4 ? a->in_dtype != LA_DTYPE_BF16 || (a->d != 64 && a->d != 128) : a->d < 8 || a->d > 128 || a->d % 8 != 0) return LA_ERR_UNSUPPORTED;
  if (a->page < 16 || a->page > 4096 || a->page % 16 != 0 || a->pages > INT32_MAX) return LA_ERR_UNSUPPORTED;
  if (!within(INT32_MAX - 8192, {a->width, a->page}) || !within(kMaxElems, {a->pages, a->H_kv, a->page, a->d}) ||
      !within(kMaxElems, {B, a->width}))
    return LA_ERR_UNSUPPORTED;
  return LA_OK;
}

template <typename Args>
bool valid_pools(const Args* a, int64_t B) {
  if (a->pages > 0 && a->H_kv > 0 && (!a->k_pages || !a->v_pages)) return false;
  return aligned16(a->k_pages) && aligned16(a->v_pages) && aligned4(a->table) && (a->table || B == 0 || a->width == 0);
}

template <typename Args>
la::PagedCache cache_of(const Args* a, unsigned* status) {
  la::PagedCache c{};
  c.Hkv = a->H_kv; c.pages = a->pages; c.width = a->width; c.d = (int)a->d; c.page = (int)a->page;
  c.bf16 = a->in_dtype == LA_DTYPE_BF16; c.four = a->bits == 4;
  c.k = const_cast<void*>(static_cast<const void*>(a->k_pages)); c.v = const_cast<void*>(static_cast<const void*>(a->v_pages));
  c.table = a->table; c.status = status;
  return c;
}

// Strides that 16 bytes times 32 bits hold
bool spannable(const la_tensor& x, int64_t B, int64_t H, int64_t N, la_dtype dt) {
  const int64_t end = (int64_t(1) << 36) / elem_bytes(dt);
  return (B <= 1 || x.stride_b < end) && (H <= 1 || x.stride_h < end) && (N <= 1 || x.stride_t < end);
}
la::Span4 span(const la_tensor& x, int64_t B, int64_t H, int64_t N, la_dtype dt) {  // a spannable one; strides of single entries do not count
  const int e = elem_bytes(dt);
  return la::Span4{x.ptr, (uint32_t)(B > 1 ? x.stride_b * e / 16 : 0), (uint32_t)(H > 1 ? x.stride_h * e / 16 : 0), (uint32_t)(N > 1 ? x.stride_t * e / 16 : 0)};
}

// Whether an output at its input's address may be it: rows in the same places, or other places altogether
bool in_place(const la_tensor& x, const la_tensor& y, int64_t B, int64_t H, int64_t N, la_dtype in, la_dtype out) {
  if (H == 0 || x.ptr != y.ptr) return true;
  return in == out && (B <= 1 || x.stride_b == y.stride_b) && (H <= 1 || x.stride_h == y.stride_h) && (N <= 1 || x.stride_t == y.stride_t);
}

}  // namespace
}  // extern "C++"

la_status la_qk_norm_rope(const la_qk_norm_rope_args* a, void* stream) {
  if (!a) return LA_ERR_INVALID_ARGUMENT;
  if (!valid_size(a->B) || !valid_size(a->H) || !valid_size(a->H_kv) || !valid_size(a->N)) return LA_ERR_INVALID_ARGUMENT;
  if (!valid_dtype(a->in_dtype) || !valid_dtype(a->out_dtype) || !valid_dtype(a->w_dtype)) return LA_ERR_INVALID_ARGUMENT;
  if (a->norm < LA_NORM_NONE || a->norm > LA_NORM_L2 || (a->norm != LA_NORM_NONE && !(a->eps > 0.f && a->eps <= 1e37f)) ||
      (a->norm == LA_NORM_NONE && (a->q_weight || a->k_weight)))
    return LA_ERR_INVALID_ARGUMENT;
  if (a->d < 8 || a->d > 256 || a->d % 8 != 0) return LA_ERR_UNSUPPORTED;
  if (a->rot < 0 || a->rot > a->d) return LA_ERR_INVALID_ARGUMENT;
  if (a->rot % 16 != 0) return LA_ERR_UNSUPPORTED;
  if (a->B == 0 || a->N == 0 || (a->H == 0 && a->H_kv == 0)) return LA_OK;
  if (a->H + a->H_kv > (int64_t(1) << 30) || !within(kMaxElems, {a->B, a->N, a->H + a->H_kv}) || la::qk_norm_rope_blocks(a->B, a->H, a->H_kv, a->N, (int)a->d) > kMaxBlocks / 4)
    return LA_ERR_UNSUPPORTED;
  if (!valid_view(a->q, a->B, a->H, a->N, a->d, a->in_dtype) || !valid_view(a->q_out, a->B, a->H, a->N, a->d, a->out_dtype) ||
      !valid_view(a->k, a->B, a->H_kv, a->N, a->d, a->in_dtype) || !valid_view(a->k_out, a->B, a->H_kv, a->N, a->d, a->out_dtype) ||
      (a->H > 0 && !distinct(a->q_out, a->B, a->H, a->N, a->d)) || (a->H_kv > 0 && !distinct(a->k_out, a->B, a->H_kv, a->N, a->d)))
    return LA_ERR_INVALID_ARGUMENT;
  if (!in_place(a->q, a->q_out, a->B, a->H, a->N, a->in_dtype, a->out_dtype) ||
      !in_place(a->k, a->k_out, a->B, a->H_kv, a->N, a->in_dtype, a->out_dtype))
    return LA_ERR_INVALID_ARGUMENT;
  if (!spannable(a->q, a->B, a->H, a->N, a->in_dtype) || !spannable(a->k, a->B, a->H_kv, a->N, a->in_dtype) ||
      !spannable(a->q_out, a->B, a->H, a->N, a->out_dtype) || !spannable(a->k_out, a->B, a->H_kv, a->N, a->out_dtype))
    return LA_ERR_UNSUPPORTED;
  if (!valid_tables(a->cos, a->sin, a->rot, a->positions) || !aligned16(a->q_weight) || !aligned16(a->k_weight) || !aligned8(a->pos) ||
      !aligned8(a->lens))
    return LA_ERR_INVALID_ARGUMENT;
  unsigned* status = device_status_ptr();
  if (!status) return LA_ERR_CUDA;
  la::QkNormRopeLaunch L{};
  L.B = a->B; L.H = a->H; L.Hkv = a->H_kv; L.N = a->N; L.positions = a->positions;
  L.d = (int)a->d; L.rot = (int)a->rot; L.norm = a->norm;
  L.in_bf16 = a->in_dtype == LA_DTYPE_BF16; L.out_bf16 = a->out_dtype == LA_DTYPE_BF16; L.w_bf16 = a->w_dtype == LA_DTYPE_BF16;
  L.q = span(a->q, a->B, a->H, a->N, a->in_dtype); L.k = span(a->k, a->B, a->H_kv, a->N, a->in_dtype);
  L.q_out = span(a->q_out, a->B, a->H, a->N, a->out_dtype); L.k_out = span(a->k_out, a->B, a->H_kv, a->N, a->out_dtype);
  L.q_weight = a->q_weight; L.k_weight = a->k_weight; L.cos = a->cos; L.sin = a->sin; L.pos = a->pos; L.lens = a->lens;
  L.eps = a->eps; L.interleaved = a->interleaved != 0; L.pos_each = a->pos_each != 0; L.fill = (a->fill & LA_FILL_ROWS) != 0;
  L.status = status;
  return from_cuda(la::launch_qk_norm_rope(L, static_cast<cudaStream_t>(stream)));
}

la_status la_paged_append(const la_paged_append_args* a, void* stream) {
  if (!a) return LA_ERR_INVALID_ARGUMENT;
  if (!valid_size(a->B) || !valid_size(a->N)) return LA_ERR_INVALID_ARGUMENT;
  const la_status st = check_pages(a, a->B);
  if (st != LA_OK) return st;
  if (a->rot < 0 || a->rot > a->d) return LA_ERR_INVALID_ARGUMENT;
  if (a->rot % 16 != 0) return LA_ERR_UNSUPPORTED;
  if (a->B == 0 || a->N == 0 || a->H_kv == 0) return LA_OK;
  if (!within((int64_t(1) << 31) - 8, {a->B, a->N, a->H_kv})) return LA_ERR_UNSUPPORTED;
  if (!valid_view(a->k, a->B, a->H_kv, a->N, a->d, a->in_dtype) || !valid_view(a->v, a->B, a->H_kv, a->N, a->d, a->in_dtype) ||
      !valid_pools(a, a->B) || !valid_tables(a->cos, a->sin, a->rot, a->positions) || !a->seen || !aligned8(a->seen) || !aligned8(a->lens))
    return LA_ERR_INVALID_ARGUMENT;
  if (!spannable(a->k, a->B, a->H_kv, a->N, a->in_dtype) || !spannable(a->v, a->B, a->H_kv, a->N, a->in_dtype)) return LA_ERR_UNSUPPORTED;
  unsigned* status = device_status_ptr();
  if (!status) return LA_ERR_CUDA;
  la::PagedAppendLaunch L{};
  L.c = cache_of(a, status);
  L.B = a->B; L.N = a->N; L.positions = a->positions; L.rot = (int)a->rot;
  L.k = span(a->k, a->B, a->H_kv, a->N, a->in_dtype); L.v = span(a->v, a->B, a->H_kv, a->N, a->in_dtype); L.cos = a->cos; L.sin = a->sin; L.seen = a->seen; L.lens = a->lens;
  L.interleaved = a->interleaved != 0;
  return from_cuda(la::launch_paged_append(L, static_cast<cudaStream_t>(stream)));
}

la_status la_paged_read(const la_paged_read_args* a, void* stream) {
  if (!a) return LA_ERR_INVALID_ARGUMENT;
  if (!valid_size(a->B) || !valid_size(a->N) || !valid_dtype(a->out_dtype)) return LA_ERR_INVALID_ARGUMENT;
  const la_status st = check_pages(a, a->B);
  if (st != LA_OK) return st;
  if (a->B == 0 || a->N == 0 || a->H_kv == 0) return LA_OK;
  if (a->N > INT32_MAX - 8192 || !within((int64_t(1) << 31) - 8, {a->B, (a->N + 15) / 16, a->H_kv, 2})) return LA_ERR_UNSUPPORTED;
  if (!valid_view(a->k, a->B, a->H_kv, a->N, a->d, a->out_dtype) || !valid_view(a->v, a->B, a->H_kv, a->N, a->d, a->out_dtype) ||
      !distinct(a->k, a->B, a->H_kv, a->N, a->d) || !distinct(a->v, a->B, a->H_kv, a->N, a->d) || !valid_pools(a, a->B) || !aligned8(a->lens))
    return LA_ERR_INVALID_ARGUMENT;
  if (!spannable(a->k, a->B, a->H_kv, a->N, a->out_dtype) || !spannable(a->v, a->B, a->H_kv, a->N, a->out_dtype)) return LA_ERR_UNSUPPORTED;
  unsigned* status = device_status_ptr();
  if (!status) return LA_ERR_CUDA;
  la::PagedReadLaunch L{};
  L.c = cache_of(a, status);
  L.B = a->B; L.N = a->N; L.out_bf16 = a->out_dtype == LA_DTYPE_BF16; L.fill = (a->fill & LA_FILL_ROWS) != 0;
  L.k = span(a->k, a->B, a->H_kv, a->N, a->out_dtype); L.v = span(a->v, a->B, a->H_kv, a->N, a->out_dtype);
  L.lens = a->lens;
  return from_cuda(la::launch_paged_read(L, static_cast<cudaStream_t>(stream)));
}

// LA_OK where the sizes say how often a sequence is split
static la_status paged_decode_shape(const la_paged_decode_args* a) {
  if (!a) return LA_ERR_INVALID_ARGUMENT;
  if (!valid_size(a->S) || !valid_size(a->H) || !valid_size(a->window) || a->H_kv < 1 || a->H % a->H_kv != 0) return LA_ERR_INVALID_ARGUMENT;
  const la_status st = check_pages(a, a->S);
  if (st != LA_OK) return st;
  if (a->H / a->H_kv > 16 || !within((int64_t(1) << 24) - 1, {a->S, a->H})) return LA_ERR_UNSUPPORTED;
  return LA_OK;
}

static int paged_decode_plan(const la_paged_decode_args* a) {
  const int64_t tokens = a->width * a->page;
  return la::paged_decode_splits(a->S, a->H_kv, a->window > 0 ? std::min(tokens, a->window + 16) : tokens);
}

size_t la_paged_decode_workspace_size(const la_paged_decode_args* a) {
  if (paged_decode_shape(a) != LA_OK || a->S == 0 || a->H == 0) return 0;
  const int splits = paged_decode_plan(a);
  return splits > 1 ? (size_t)a->S * a->H * splits * (a->d + 2) * sizeof(float) : 0;
}

la_status la_paged_decode_step(const la_paged_decode_args* a, void* ws, size_t ws_bytes, void* stream) {
  la_status st = paged_decode_shape(a);
  if (st != LA_OK) return st;
  if (!valid_dtype(a->out_dtype) || !valid_cap(a->softcap, a->scale)) return LA_ERR_INVALID_ARGUMENT;
  if (a->S == 0 || a->H == 0) return LA_OK;
  la_tensor q = a->q, o = a->out;
  q.stride_t = o.stride_t = a->d;
  if (!valid_view(q, a->S, a->H, 1, a->d, a->in_dtype) || !valid_view(o, a->S, a->H, 1, a->d, a->out_dtype) ||
      !distinct(o, a->S, a->H, 1, a->d) || !valid_pools(a, a->S) || !a->lens || !aligned8(a->lens) || !aligned4(a->slopes))
    return LA_ERR_INVALID_ARGUMENT;
  const size_t need = la_paged_decode_workspace_size(a);
  if (need > 0 && (!ws || !aligned16(ws) || ws_bytes < need)) return LA_ERR_WORKSPACE;
  unsigned* status = device_status_ptr();
  if (!status) return LA_ERR_CUDA;
  la::PagedDecodeLaunch L{};
  L.c = cache_of(a, status);
  L.S = a->S; L.H = a->H; L.window = a->window; L.out_bf16 = a->out_dtype == LA_DTYPE_BF16;
  L.scale = a->scale; L.softcap = a->softcap; L.q = view(q); L.out = o.ptr; L.o_sb = o.stride_b; L.o_sh = o.stride_h;
  L.lens = a->lens; L.slopes = a->slopes;
  L.splits = paged_decode_plan(a); L.parts = static_cast<float*>(ws);
  return from_cuda(la::launch_paged_decode(L, static_cast<cudaStream_t>(stream)));
}

la_status la_selftest_bounded_wait(int arrive, int64_t limit_ns, void* stream) {
  if (limit_ns < 1000000 || limit_ns > 2000000000) return LA_ERR_INVALID_ARGUMENT;
  unsigned* status = device_status_ptr();
  if (!status) return LA_ERR_CUDA;
  return from_cuda(la::launch_bounded_wait_selftest(arrive, (uint64_t)limit_ns, status, static_cast<cudaStream_t>(stream)));
}

la_status la_device_status(void* stream, int clear) {
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return LA_ERR_CUDA;
  unsigned v = 0;
  if (cudaMemcpyFromSymbol(&v, g_la_device_status, sizeof v) != cudaSuccess) return LA_ERR_CUDA;
  if (clear && v != 0) {
    const unsigned zero = 0;
    if (cudaMemcpyToSymbol(g_la_device_status, &zero, sizeof zero) != cudaSuccess) return LA_ERR_CUDA;
  }
  if (v & la::kStatusTimeout) return LA_ERR_TIMEOUT;
  return v ? LA_ERR_INVALID_ARGUMENT : LA_OK;  // kStatusBadIndex
}

}  // extern "C"
