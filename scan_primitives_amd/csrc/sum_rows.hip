// sum_rows.hip: sums over the rows of f32 arrays: the workgroups'
// shares of gradients that all tokens add to (weights, biases, rates).
//
// A workgroup takes 64 columns, its waves every 16th row each; the waves' sums
// meet in LDS. Always in the same order (no atomics), in 64 bits, for the rows
// may be many thousand and the kernel waits for memory either way.
#include "sx_state_space.hpp"

namespace sx {
namespace {

constexpr int kCols = 64, kSlices = 16;

__global__ __launch_bounds__(kCols* kSlices) void sum_rows(SumRows p) {
  __shared__ double l[kSlices][kCols];
  const auto& s = p.s[blockIdx.y];
  const int64_t first = int64_t(blockIdx.x) * kCols;
  if (first >= s.cols) return;
  const int lane = int(threadIdx.x) % kCols, slice = int(threadIdx.x) / kCols;
  const int64_t c = first + lane;
  double v = 0.0;
  if (c < s.cols) {
#pragma unroll 4
    for (int64_t r = slice; r < s.rows; r += kSlices) v += double(s.src[r * s.stride + c]);
  }
  l[slice][lane] = v;
  __syncthreads();
  if (slice == 0 && c < s.cols) {
    v = 0.0;
#pragma unroll
    for (int i = 0; i < kSlices; ++i) v += l[i][lane];
    const int64_t run = s.cols / s.inner;
    s.out[s.inner > 1 ? c % run * s.inner + c / run : c] = float(v);
  }
}

}  // namespace

hipError_t launch_sum_rows(const SumRows& p, hipStream_t stream) {
  SumRows q{};
  int64_t most = 0;
  for (int i = 0; i < p.count; ++i) {
    if (!p.s[i].out || p.s[i].cols == 0) continue;
    q.s[q.count++] = p.s[i];
    most = most > p.s[i].cols ? most : p.s[i].cols;
  }
  if (q.count == 0) return hipSuccess;
  sum_rows<<<dim3(unsigned((most + kCols - 1) / kCols), unsigned(q.count)), kCols * kSlices, 0, stream>>>(q);
  return hipGetLastError();
}

}  // namespace sx
