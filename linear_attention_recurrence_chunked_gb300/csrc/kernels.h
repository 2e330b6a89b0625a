// kernels.h -- internal launch descriptors shared by the C ABI layer and the
// kernel translation units.  Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace la {

// Bits of the device status word (read back by la_device_status).
constexpr unsigned kStatusTimeout = 1u;   // a bounded wait expired
constexpr unsigned kStatusBadIndex = 2u;  // a state index outside its array was skipped

// The cudaError_t behind the latest LA_ERR_CUDA returned to the calling
// thread (api.cu); noted by every path that maps a CUDA failure to it.
void note_cuda_error(int code);
int last_cuda_error();

struct View4 {        // strided [B, H, N, d] view, element strides
  const void* ptr;
  int64_t sb, sh, st;
};

struct DecodeLaunch {
  int64_t S, H;
  bool in_bf16, out_bf16;
  const void *q, *k, *v;
  const float *alpha, *beta;
  void* out;
  float* state;
  float* z;
  float eps, q_scale;
  float delta;  // GDN-family decode: 1 = gated delta rule, 0 = scalar gate (A_t = alpha_t I)
  const float* decay;  // Taylor decode: per-head retention [H] or null
};

struct TaylorPrefillLaunch {
  int64_t B, H, N;
  bool in_bf16, out_bf16;
  View4 q, k, v;
  void* y;
  int64_t y_sb, y_sh, y_st;
  const float* s_in;
  const float* z_in;
  float* s_out;
  float* z_out;
  float eps;
  const float* decay;  // per-head retention [H] or null (no decay)
};

struct GdnPrefillLaunch {
  int64_t B, H, N;
  bool in_bf16, out_bf16;
  View4 q, k, v;
  void* o;
  int64_t o_sb, o_sh, o_st;
  const float* alpha;
  int64_t a_sb, a_sh;
  const float* beta;
  int64_t b_sb, b_sh;
  float q_scale;
  const float* S_in;
  float* S_out;
  float delta;  // 1 = gated delta rule, A_t = alpha_t (I - beta_t k_t k_t^T); 0 = scalar gate, A_t = alpha_t I
};

// Sequence-segment plan of the gated-delta-rule prefill (see gdn_chunked.cu):
// G segments of seg_len tokens per (b,h); G == 1 runs the plain chunk scan.
struct GdnSegPlan {
  int G;
  int64_t seg_len;
  size_t ws_bytes;  // workspace: segment maps then segment entry states
};
GdnSegPlan gdn_segment_plan(int64_t B, int64_t H, int64_t N);

cudaError_t launch_gdn_decode(const DecodeLaunch& a, cudaStream_t stream);
cudaError_t launch_taylor_decode(const DecodeLaunch& a, cudaStream_t stream);
// fp32 inputs: token-serial CUDA-core kernels (fp32 arithmetic throughout).
cudaError_t launch_taylor_prefill_recurrent(const TaylorPrefillLaunch& a, cudaStream_t stream);
cudaError_t launch_gdn_prefill_recurrent(const GdnPrefillLaunch& a, cudaStream_t stream);
// bf16 inputs: chunked tcgen05 kernels.  The single-kernel scan needs the
// segment scratch of gdn_segment_plan only; the two-kernel scan (per-chunk
// inverse records, then the warp-specialized state scan) needs
// gdn_scan_workspace_bytes.
cudaError_t launch_gdn_prefill_chunked(const GdnPrefillLaunch& a, void* ws, size_t ws_bytes, unsigned* dev_status,
                                       cudaStream_t stream);
size_t gdn_scan_workspace_bytes(int64_t B, int64_t H, int64_t N);
cudaError_t launch_gdn_prefill_scan(const GdnPrefillLaunch& a, void* ws, size_t ws_bytes, unsigned* dev_status,
                                    cudaStream_t stream);
cudaError_t launch_taylor_prefill_chunked(const TaylorPrefillLaunch& a, unsigned* dev_status, cudaStream_t stream);
struct SwaDecodeLaunch {
  int64_t S, H;
  int d, window;
  bool in_bf16, out_bf16;
  const void *q, *k, *v;
  void *k_cache, *v_cache;
  const int64_t* pos;
  void* out;
  float scale;
  unsigned* status;  // device status word (a negative position sets kStatusBadIndex)
};
cudaError_t launch_swa_decode(const SwaDecodeLaunch& a, cudaStream_t stream);

// State operations between calls (state_ops.cu).  per = fp32 elements per state.
cudaError_t launch_state_rescale(float* states, int64_t n_states, int64_t per, const float* lambda, float lambda_all,
                                 cudaStream_t stream);
cudaError_t launch_state_gather(float* dst, const float* src, const int64_t* index, int64_t n_dst, int64_t n_src,
                                int64_t per, unsigned* dev_status, cudaStream_t stream);
cudaError_t launch_bounded_wait_selftest(int arrive, uint64_t limit_ns, unsigned* dev_status, cudaStream_t stream);

// NoteBank write side and routing (notebank.cu).
constexpr int kNoteAddrDims = 16;  // d_rho: query coordinates stored per channel and note
struct NotebankScoresLaunch {
  int64_t L, H, N, d;   // channels = L x H; key width d (multiple of 32, <= 256)
  bool in_bf16;
  View4 k;              // [L, H, N, d]
  int64_t chunk, window;
  float* d_ch;          // [L, H, N]
  float* d_mean;        // [N]
  float* w;             // [N - window + 1] or null
};
struct NotebankAddressLaunch {
  int64_t L, H, N, d, n_notes;
  bool in_bf16;
  View4 q;                // [L, H, N, d]
  const float* d_ch;      // [L, H, N]
  const int32_t* coords;  // [L, H, 16]
  const int64_t* spans;   // [n_notes, 2]: start, length
  int32_t* t_star;        // [n_notes, L, H]
  void* rho;              // [n_notes, L, H, 16] bf16
};
struct NotebankRouteLaunch {
  int64_t n_notes, J, n_q, R;
  const void* rho;           // [n_notes, J, 16] bf16
  const void* u;             // [J, n_q, 16] bf16
  const int64_t* positions;  // [n_notes] or null
  float* s;                  // [n_notes, J] or null
  int32_t* winner;           // [J]
  int32_t* votes;            // [n_notes]
  int32_t* top;              // [R]
};
cudaError_t launch_notebank_scores(const NotebankScoresLaunch& a, cudaStream_t stream);
cudaError_t launch_notebank_address(const NotebankAddressLaunch& a, unsigned* status, cudaStream_t stream);
cudaError_t launch_notebank_route(const NotebankRouteLaunch& a, cudaStream_t stream);

// What a call with lens leaves out (padding.cu): rows [B, H, N] of row_bytes (strides in bytes, 16-byte aligned; null:
// none) from lens[b] - offset on become zeros, and where lens[b] is outside [0, max_len] all of the sequence's rows
// and its state_out (null: none) becomes state_in (null: zeros).
struct PaddingLaunch {
  int64_t B, H, N, max_len, offset;
  const int64_t* lens;
  void* rows;
  int64_t sb, sh, st, row_bytes;
  const void* state_in;
  void* state_out;
  int64_t state_bytes;  // of one sequence
};
cudaError_t launch_fill_padding(const PaddingLaunch& a, cudaStream_t stream);

// Short causal convolution (conv.cu).  The step is the prompt form's data with one token per sequence.
struct ConvLaunch {
  int64_t B, N, C;
  int W;
  bool in_bf16, out_bf16, w_bf16;
  const void* x;
  int64_t x_sb, x_st;
  void* y;
  int64_t y_sb, y_st;
  const void *w, *bias, *state_in;
  void* state_out;
  const int64_t* lens;  // [B] or null
  int silu;
  unsigned* status;     // device status word (a length out of range sets kStatusBadIndex)
};
cudaError_t launch_conv_prefill(const ConvLaunch& a, cudaStream_t stream);
cudaError_t launch_conv_decode(const ConvLaunch& a, cudaStream_t stream);  // N = 1, no lens

// Selective state space scan (ssm.cu).  The step has N = 1 and no lens.
struct SsmLaunch {
  int64_t B, N, C, G;
  int n;
  bool in_bf16, out_bf16;
  const void *u, *delta, *z;
  int64_t u_sb, u_st, d_sb, d_st, z_sb, z_st;
  void* y;
  int64_t y_sb, y_st;
  View4 Bm, Cm;         // [B, G, N, n]
  const float *A, *D, *delta_bias, *h_in;
  float* h_out;
  const int64_t* lens;
  int softplus;
  unsigned* status;
};
size_t ssm_workspace_bytes(int64_t B, int64_t N, int64_t C, int n, int64_t G);
cudaError_t launch_ssm_prefill(const SsmLaunch& a, void* ws, size_t ws_bytes, cudaStream_t stream);
cudaError_t launch_ssm_decode(const SsmLaunch& a, cudaStream_t stream);

// Masked window attention over a prompt (swa_prefill.cu: fp32 and the rings; swa_prefill_tc.cu: bf16).
struct SwaPrefillLaunch {
  int64_t B, H, Hkv, Nq, Nk;
  int d;
  int64_t window, q_pos0;
  bool in_bf16, out_bf16;
  View4 q, k, v;
  void* o;
  int64_t o_sb, o_sh, o_st;
  float scale, softcap;
  const float* slopes;
  const int32_t *key_lo, *key_hi;
  const int64_t* lens;
  void *k_cache, *v_cache;
  unsigned* status;
  uint64_t wait_ns;  // limit of a wait (bf16)
};
cudaError_t launch_swa_prefill_tc(const SwaPrefillLaunch& a, cudaStream_t stream);    // bf16 inputs, strides below 2^40 bytes
cudaError_t launch_swa_prefill_simt(const SwaPrefillLaunch& a, cudaStream_t stream);  // fp32 inputs
cudaError_t launch_swa_fill_rings(const SwaPrefillLaunch& a, cudaStream_t stream);

struct SwaBiasedDecodeLaunch {
  SwaDecodeLaunch base;
  int64_t Hkv;
  float softcap;
  const float* slopes;
};
cudaError_t launch_swa_biased_decode(const SwaBiasedDecodeLaunch& a, cudaStream_t stream);

// A [B, H, N, d] view whose strides are counted in 16 bytes: an element's place takes 32-bit products.
struct Span4 {
  void* ptr;
  uint32_t sb, sh, st;
#ifdef __CUDACC__
  template <typename T>
  __device__ __forceinline__ T* at(uint32_t b, uint32_t h, uint32_t n) const {
    return reinterpret_cast<T*>(static_cast<uint4*>(ptr) + ((uint64_t)b * sb + (uint64_t)h * sh + (uint64_t)n * st));
  }
  template <typename T>
  __device__ __forceinline__ int64_t step() const { return (int64_t)sh * (16 / (int)sizeof(T)); }  // elements from head to head
#endif
};

// Norms and position rotation of queries and keys (heads.cu).
struct QkNormRopeLaunch {
  int64_t B, H, Hkv, N, positions;
  int d, rot, norm;
  bool in_bf16, out_bf16, w_bf16;
  Span4 q, k, q_out, k_out;
  const void *q_weight, *k_weight;
  const float *cos, *sin;
  const int64_t *pos, *lens;
  float eps;
  bool interleaved, pos_each, fill;
  unsigned* status;
};
int64_t qk_norm_rope_blocks(int64_t B, int64_t H, int64_t Hkv, int64_t N, int d);  // of the launch's grid
cudaError_t launch_qk_norm_rope(const QkNormRopeLaunch& a, cudaStream_t stream);

// Paged caches (paged.cu): what a token's place follows from.
struct PagedCache {
  int64_t Hkv, pages, width;
  int d, page;
  bool bf16, four;       // type of the rows; four: 4 bits of bf16 rows
  void *k, *v;
  const int32_t* table;  // [B, width]
  unsigned* status;
};
struct PagedAppendLaunch {
  PagedCache c;
  int64_t B, N, positions;
  int rot;
  Span4 k, v;
  const float *cos, *sin;
  const int64_t *seen, *lens;
  bool interleaved;
};
struct PagedReadLaunch {
  PagedCache c;
  int64_t B, N;
  bool out_bf16, fill;
  Span4 k, v;
  const int64_t* lens;
};
cudaError_t launch_paged_append(const PagedAppendLaunch& a, cudaStream_t stream);
cudaError_t launch_paged_read(const PagedReadLaunch& a, cudaStream_t stream);

// One token's attention over a paged cache (paged_decode.cu).
struct PagedDecodeLaunch {
  PagedCache c;
  int64_t S, H, window;
  bool out_bf16;
  float scale, softcap;
  View4 q;
  void* out;
  int64_t o_sb, o_sh;
  const int64_t* lens;
  const float* slopes;
  int splits;    // of a sequence's tokens; more than one: the parts meet in `parts`
  float* parts;  // [S, H, splits, d + 2]: sums of weighted values, their greatest score, the sum of weights
};
int paged_decode_splits(int64_t S, int64_t Hkv, int64_t tokens);
cudaError_t launch_paged_decode(const PagedDecodeLaunch& a, cudaStream_t stream);

}  // namespace la
