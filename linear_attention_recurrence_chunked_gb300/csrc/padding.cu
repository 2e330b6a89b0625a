// padding.cu -- what a prompt call with sequence lengths leaves out of outputs that were made for it: zeros into the
// rows of padding, and the incoming state (or zeros) into the state of a sequence whose length is out of range.
// One launch that touches those rows only, in place of a fill of the whole output and a copy of the whole state
// in front of the call (5 ragged sequences of up to 1001 x 520 fp32 with a state: 19 us a call against 27).
#include "layers.cuh"

namespace la {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerBlock = 64;

__global__ void __launch_bounds__(kThreads)
fill_padding_kernel(const PaddingLaunch a, int64_t chunks) {
  const int64_t bh = blockIdx.x / chunks, chunk = blockIdx.x - bh * chunks, b = bh / a.H, h = bh - b * a.H;
  const int64_t n = a.lens[b];
  const bool bad = n < 0 || n > a.max_len;
  if (a.state_out && bad && h == 0) {
    const int64_t per = (a.state_bytes + chunks - 1) / chunks;  // bytes: every block of the sequence takes some
    const uint8_t* from = static_cast<const uint8_t*>(a.state_in) + b * a.state_bytes;
    uint8_t* to = static_cast<uint8_t*>(a.state_out) + b * a.state_bytes;
    for (int64_t i = chunk * per + threadIdx.x; i < min((chunk + 1) * per, a.state_bytes); i += kThreads) to[i] = a.state_in ? from[i] : 0;
  }
  if (!a.rows) return;
  const int64_t first = max(chunk * kRowsPerBlock, bad ? 0 : max((int64_t)0, n - a.offset));
  const int64_t last = min((chunk + 1) * kRowsPerBlock, a.N);
  if (first >= last) return;
  uint8_t* y = static_cast<uint8_t*>(a.rows) + b * a.sb + h * a.sh;  // strides in bytes, rows 16-byte aligned
  const int vecs = (int)((a.row_bytes + 15) / 16);
  for (int64_t e = threadIdx.x; e < (last - first) * vecs; e += kThreads) {
    const int64_t r = e / vecs, at = (e - r * vecs) * 16;
    uint8_t* p = y + (first + r) * a.st + at;
    if (at + 16 <= a.row_bytes) {
      *reinterpret_cast<uint4*>(p) = make_uint4(0u, 0u, 0u, 0u);
    } else {
      for (int64_t i = 0; i < a.row_bytes - at; i += 2) *reinterpret_cast<uint16_t*>(p + i) = 0;
    }
  }
}

}  // namespace

cudaError_t launch_fill_padding(const PaddingLaunch& a, cudaStream_t stream) {
  const int64_t chunks = a.N > kRowsPerBlock ? (a.N + kRowsPerBlock - 1) / kRowsPerBlock : 1;
  fill_padding_kernel<<<(unsigned)(a.B * a.H * chunks), kThreads, 0, stream>>>(a, chunks);
  return cudaGetLastError();
}

}  // namespace la
