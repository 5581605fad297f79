// scan_march.hpp: what the selective scan's kernels share: tiles of tokens and
// channels on their way into LDS, and rows of b and c as operands of every lane.
#pragma once

#include <utility>

#include "sx_state_space.hpp"

namespace sx {

// Lane j of each row of 16 lanes holds token j's value; this is token J's, in every lane. The compiler joins it
// with the instruction that takes it (a DPP operand), so it costs nothing.
template <int J>
__device__ __forceinline__ float of_token(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x150 + J, 0xf, 0xf, true));
}

// f(integral_constant<int, 0>) ... f(integral_constant<int, N - 1>), or last to first.
template <int N, typename F>
__device__ __forceinline__ void each(F&& f) {
  [&]<int... I>(std::integer_sequence<int, I...>) { (f(std::integral_constant<int, I>{}), ...); }
  (std::make_integer_sequence<int, N>{});
}

// Four channels of one token. WIDE: they lie next to each other and exist all; else an element at a time, those
// behind the last (`left` of them exist) read as the last.
template <bool BF, bool WIDE>
__device__ __forceinline__ typename Piece<BF, 4>::Raw four_channels(const TokenView& v, int64_t at, int left) {
  using P = Piece<BF, 4>;
  using E = typename P::E;
  const E* p = static_cast<const E*>(v.p) + at;
  if constexpr (WIDE) {
    return P::load(p);
  } else {
    return P::of(p[0], p[min(1, left - 1) * v.sd], p[min(2, left - 1) * v.sd], p[min(3, left - 1) * v.sd]);
  }
}

// Four channels of a contiguous result.
template <bool BF, bool WIDE>
__device__ __forceinline__ void put_channels(void* out, int64_t at, int left, const float (&v)[4]) {
  using P = Piece<BF, 4>;
  using E = typename P::E;
  E* p = static_cast<E*>(out) + at;
  if constexpr (WIDE) {
    P::store(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) Piece<BF, 1>::store(p + i, {v[i]});
  }
}

// States n0 .. n0 + 3 of a token's row of b or c, zero where there are none.
template <bool BF>
struct RowRaw {
  typename Piece<BF, 1>::E e[kScanStates];
  __device__ __forceinline__ void load(const RowView& v, int64_t at, int n0, int N, bool live) {
    using E = typename Piece<BF, 1>::E;
    const E* p = static_cast<const E*>(v.p) + at;
#pragma unroll
    for (int i = 0; i < kScanStates; ++i) e[i] = live && n0 + i < N ? p[(n0 + i) * v.sn] : E(0);
  }
  __device__ __forceinline__ void open(float (&f)[kScanStates]) const {
#pragma unroll
    for (int i = 0; i < kScanStates; ++i) {
      float one[1];
      Piece<BF, 1>::open(e[i], one);
      f[i] = one[0];
    }
  }
};

// a[d, n0 .. n0 + 3] for exp2: times log2(e), zero where there are none.
__device__ __forceinline__ void rates(const float* a, int64_t d, int n0, int N, bool is, float (&r)[kScanStates]) {
#pragma unroll
  for (int i = 0; i < kScanStates; ++i) r[i] = is && n0 + i < N ? a[d * N + n0 + i] * kLog2e : 0.0f;
}

// h[n0 .. n0 + 3] of one channel in [.., D, N].
__device__ __forceinline__ void read_states(const float* p, int64_t row, int n0, int N, bool is,
                                            float (&h)[kScanStates]) {
#pragma unroll
  for (int i = 0; i < kScanStates; ++i) h[i] = p && is && n0 + i < N ? p[row * N + n0 + i] : 0.0f;
}
__device__ __forceinline__ void write_states(float* p, int64_t row, int n0, int N, bool is,
                                             const float (&h)[kScanStates]) {
#pragma unroll
  for (int i = 0; i < kScanStates; ++i)
    if (is && n0 + i < N) p[row * N + n0 + i] = h[i];
}

// The four states of channel d in an array [..][waves][D][4].
__device__ __forceinline__ int64_t packed_at(const SsParams& p, int64_t row, int wave, int64_t d) {
  return ((row * p.waves + wave) * p.D + d) * kScanStates;
}

}  // namespace sx
