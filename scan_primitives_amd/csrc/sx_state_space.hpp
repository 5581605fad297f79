// sx_state_space.hpp: descriptors and device helpers of the state-space layer's
// operators, shared by the host dispatch (sx_api.cpp) and their kernels
// (causal_conv.hip, selective_scan.hip, selective_scan_grad.hip, group_norm.hip).
// Internal to libsx_scan.so.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ms_mfma.hpp"
#include "sx_common.hpp"
#include "sx_scan.h"

namespace sx {

// [B, T, D] with element strides.
struct TokenView {
  const void* p;
  int64_t sb, st, sd;
};

// [B, T, G, N] with element strides.
struct RowView {
  const void* p;
  int64_t sb, st, sg, sn;
};

// Sums over the rows of up to four f32 arrays, one launch: out[c] = sum over r of
// src[r * stride + c]. With `inner` m > 1 the columns are m runs of cols / m, and
// run j's column d goes to out[d * m + j].
struct SumRows {
  struct {
    const float* src;
    float* out;       // nullptr: not wanted
    int64_t rows, stride, cols, inner;
  } s[4];
  int count;
};
hipError_t launch_sum_rows(const SumRows& p, hipStream_t stream);

// ---------------------------------------------------------------- causal convolution

struct CcParams {
  int B, T, D, K;
  TokenView x, go;         // go: the gradient of out (gradient only)
  const float* w;          // [D, K]
  const float* bias;       // [D] or nullptr
  const void* initial;     // [B, K - 1, D] or nullptr (zero)
  const void* grad_state;  // gradient of the last state, or nullptr
  const int32_t* lengths;  // [B] or nullptr
  int silu, bf16;
  int chunk, chunks;       // tokens a thread marches over, and how many such there are (set by the split)
  void* out;               // [B, T, D]: the result, or the gradient of x
  void* last;              // [B, K - 1, D]: the last state, or the gradient of the initial one; or nullptr
  float* partial;          // gradient: [B * chunks][K + 1][D]
  float* gw;               // [D, K]
  float* gbias;            // [D] or nullptr
};
void causal_conv_split(CcParams& p, bool gradient);
double causal_conv_workgroups(const CcParams& p, bool gradient);  // of 256
hipError_t launch_causal_conv(const CcParams& p, hipStream_t stream);
hipError_t launch_causal_conv_backward(const CcParams& p, hipStream_t stream);

struct CcStep {
  int B, D, K;
  const void* x;
  int64_t sb, sd;
  const float* w;
  const float* bias;
  void* state;             // slot s at s * ss, [K - 1, D] row-major
  int64_t ss, pool;
  const int32_t* slots;
  int silu, bf16;
  void* out;
};
double causal_conv_step_workgroups(const CcStep& p);  // of 256
hipError_t launch_causal_conv_step(const CcStep& p, hipStream_t stream);

// ---------------------------------------------------------------- selective scan

constexpr int kScanStates = 4;  // states a wave holds of each of its channels

struct SsParams {
  int B, T, D, G, N;
  int waves;               // of a workgroup: ceil(N / 4), eight above four
  TokenView x, delta, z;   // z.p nullptr: no gate
  RowView b, c;
  const float* a;          // [D, N]
  const float* skip;       // [D] or nullptr (zero)
  const float* delta_bias; // [D] or nullptr
  int softplus, bf16;
  const float* initial;    // [B, D, N] or nullptr (zero)
  const int32_t* lengths;  // [B] or nullptr
  void* out;               // [B, T, D]
  float* last;             // [B, D, N] or nullptr
  int segments, seg_tokens;
  float* seg_state;        // [segments][B][waves][D][4]: of a segment alone; the gradient's carry leaves the start's
  float* seg_steps;        // [segments][B][D]: sum of dt
  // gradient
  TokenView go;
  const float* grad_state; // [B, D, N] or nullptr
  float* seg_adjoint;      // as seg_state: of a segment alone at its start; the carry leaves the one at its end
  float* marks;            // [B][marks a row][waves][D][4]: the state before every kMarkTokens-th token
  float* mark_steps;       // [B][marks a row][D]: sum of dt from the segment's start on
  int row_marks;           // marks a row
  float* rows_partial;     // [B][G][T][blocks][2][4 waves]: gradients of b and c, a workgroup each
  float* a_partial;        // [B * segments][D][N]
  float* skip_partial;     // [B * segments][D]
  float* bias_partial;     // [B * segments][D]
  void *gx, *gdelta, *gz;  // [B, T, D]
  void *gb, *gc;           // [B, T, G, N]
  float *ga, *gskip, *gbias, *ginitial;
};
constexpr int kMarkTokens = 8;
constexpr int kGradChannels = 128;  // of a workgroup of the gradient's march
int selective_scan_grad_blocks(const SsParams& p);  // workgroups a group's channels make
void selective_scan_split(SsParams& p, bool gradient);
hipError_t launch_selective_scan(const SsParams& p, hipStream_t stream);
hipError_t launch_selective_scan_backward(const SsParams& p, hipStream_t stream);

struct SsStep {
  int B, D, G, N;
  TokenView x, delta, z;   // st unused
  RowView b, c;
  const float *a, *skip, *delta_bias;
  int softplus, bf16;
  float* state;            // slot s at s * ss, [D, N] row-major
  int64_t ss, pool;
  const int32_t* slots;
  void* out;
};
int selective_scan_step_lanes(int N);  // that a channel takes
hipError_t launch_selective_scan_step(const SsStep& p, hipStream_t stream);

// ---------------------------------------------------------------- group norm

struct GnParams {
  int64_t n, s;            // samples, and positions of a sample
  int c, g;                // channels and groups
  const void* x;           // [n, s, c], channels next to each other
  int64_t xn, xs;          // its strides
  const void* go;          // gradient of out (gradient only), the same
  int64_t gon, gos;
  const float* w;
  const float* bias;
  float eps;
  int silu, bf16;
  int64_t chunk;           // positions a workgroup takes (set by the split)
  int chunks;
  float* stats;            // [n][chunks][g][3]: count, mean and squared distance of a chunk
  float* sums;             // gradient: [n][chunks][2][c]
  void* out;               // contiguous
  float* gw;
  float* gbias;
};
void group_norm_split(GnParams& p, bool gradient);
double group_norm_workgroups(const GnParams& p, bool gradient);  // of its largest launch; infinite where none takes it
// Floats of workspace: stats, then sums (rows of the channels' gradients).
int64_t group_norm_stats_floats(const GnParams& p);
int64_t group_norm_sums_floats(const GnParams& p);
hipError_t launch_group_norm(const GnParams& p, hipStream_t stream);
hipError_t launch_group_norm_backward(const GnParams& p, hipStream_t stream);

// ---------------------------------------------------------------- device helpers

constexpr float kLog2e = 1.4426950408889634f;

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x4_any2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_any4 __attribute__((ext_vector_type(4), aligned(4)));

// V elements next to each other in memory, at any alignment of theirs.
template <bool BF, int V>
struct Piece;
template <>
struct Piece<true, 1> {
  using E = uint16_t;
  using Raw = uint16_t;
  static __device__ __forceinline__ Raw load(const E* p) { return *p; }
  static __device__ __forceinline__ Raw zero() { return 0; }
  static __device__ __forceinline__ void open(Raw r, float (&v)[1]) { v[0] = bf16_to_f32(r); }
  static __device__ __forceinline__ void store(E* p, const float (&v)[1]) { *p = f32_to_bf16_rne(v[0]); }
  static __device__ __forceinline__ void put(E* p, Raw r) { *p = r; }
};
template <>
struct Piece<false, 1> {
  using E = float;
  using Raw = float;
  static __device__ __forceinline__ Raw load(const E* p) { return *p; }
  static __device__ __forceinline__ Raw zero() { return 0.0f; }
  static __device__ __forceinline__ void open(Raw r, float (&v)[1]) { v[0] = r; }
  static __device__ __forceinline__ void store(E* p, const float (&v)[1]) { *p = v[0]; }
  static __device__ __forceinline__ void put(E* p, Raw r) { *p = r; }
};
typedef uint32_t u32_any2 __attribute__((aligned(2)));
typedef uint32_t u32x2_any4 __attribute__((ext_vector_type(2), aligned(4)));
template <>
struct Piece<true, 2> {
  using E = uint16_t;
  using Raw = uint32_t;
  static __device__ __forceinline__ Raw load(const E* p) { return *reinterpret_cast<const u32_any2*>(p); }
  static __device__ __forceinline__ Raw zero() { return 0; }
  static __device__ __forceinline__ void open(Raw r, float (&v)[2]) {
    v[0] = __uint_as_float(r << 16);
    v[1] = __uint_as_float(r & 0xffff0000u);
  }
  static __device__ __forceinline__ void store(E* p, const float (&v)[2]) { put(p, pack_bf16x2(v[0], v[1])); }
  static __device__ __forceinline__ void put(E* p, Raw r) { *reinterpret_cast<u32_any2*>(p) = r; }
};
template <>
struct Piece<false, 2> {
  using E = float;
  using Raw = u32x2;
  static __device__ __forceinline__ Raw load(const E* p) { return *reinterpret_cast<const u32x2_any4*>(p); }
  static __device__ __forceinline__ Raw zero() { return Raw{0, 0}; }
  static __device__ __forceinline__ void open(Raw r, float (&v)[2]) {
    v[0] = __uint_as_float(r[0]);
    v[1] = __uint_as_float(r[1]);
  }
  static __device__ __forceinline__ void store(E* p, const float (&v)[2]) {
    put(p, Raw{__float_as_uint(v[0]), __float_as_uint(v[1])});
  }
  static __device__ __forceinline__ void put(E* p, Raw r) { *reinterpret_cast<u32x2_any4*>(p) = r; }
};
template <>
struct Piece<true, 4> {
  using E = uint16_t;
  using Raw = u32x2;
  static __device__ __forceinline__ Raw load(const E* p) { return *reinterpret_cast<const u32x2_any*>(p); }
  static __device__ __forceinline__ Raw zero() { return Raw{0, 0}; }
  static __device__ __forceinline__ Raw of(E a, E b, E c, E d) {
    return Raw{uint32_t(a) | uint32_t(b) << 16, uint32_t(c) | uint32_t(d) << 16};
  }
  static __device__ __forceinline__ void open(Raw r, float (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[2 * i] = __uint_as_float(r[i] << 16);
      v[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(E* p, const float (&v)[4]) {
    put(p, Raw{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])});
  }
  static __device__ __forceinline__ void put(E* p, Raw r) { *reinterpret_cast<u32x2_any*>(p) = r; }
};
template <>
struct Piece<false, 4> {
  using E = float;
  using Raw = u32x4_t;
  static __device__ __forceinline__ Raw load(const E* p) { return *reinterpret_cast<const u32x4_any4*>(p); }
  static __device__ __forceinline__ Raw zero() { return Raw{0, 0, 0, 0}; }
  static __device__ __forceinline__ Raw of(E a, E b, E c, E d) {
    return Raw{__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d)};
  }
  static __device__ __forceinline__ void open(Raw r, float (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
  }
  static __device__ __forceinline__ void store(E* p, const float (&v)[4]) { put(p, of(v[0], v[1], v[2], v[3])); }
  static __device__ __forceinline__ void put(E* p, Raw r) { *reinterpret_cast<u32x4_any4*>(p) = r; }
};
template <>
struct Piece<true, 8> {
  using E = uint16_t;
  using Raw = u32x4_t;
  static __device__ __forceinline__ Raw load(const E* p) { return *reinterpret_cast<const u32x4_any2*>(p); }
  static __device__ __forceinline__ Raw zero() { return Raw{0, 0, 0, 0}; }
  static __device__ __forceinline__ void open(Raw r, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(r[i] << 16);
      v[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(E* p, const float (&v)[8]) {
    put(p, Raw{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])});
  }
  static __device__ __forceinline__ void put(E* p, Raw r) { *reinterpret_cast<u32x4_any2*>(p) = r; }
};

// A result that nothing reads again, past the caches where it is 16 bytes: what the L2s still held at a kernel's end
// would have to be written then (16384 rows of 2048 channels normed in bf16: 25.0 us, 26.2 through them).
template <bool BF, int V>
__device__ __forceinline__ void store_stream(typename Piece<BF, V>::E* p, const float (&v)[V]) {
  if constexpr (BF && V == 8) {
    const u32x4_any2 r = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                          pack_bf16x2(v[6], v[7])};
    __builtin_nontemporal_store(r, reinterpret_cast<u32x4_any2*>(p));
  } else if constexpr (!BF && V == 4) {
    const u32x4_any4 r = Piece<BF, V>::of(v[0], v[1], v[2], v[3]);
    __builtin_nontemporal_store(r, reinterpret_cast<u32x4_any4*>(p));
  } else {
    Piece<BF, V>::store(p, v);
  }
}

__device__ __forceinline__ float exp2_of(float v) { return __builtin_amdgcn_exp2f(v); }

// 1 / (1 + exp(-v)): the exponential's infinity makes it 0.
__device__ __forceinline__ float sigmoid_of(float v) {
  return __builtin_amdgcn_rcpf(1.0f + exp2_of(-kLog2e * v));
}

// log(1 + exp(v)) = max(v, 0) + log1p(e), e = exp(-|v|), to f32's accuracy also where it is small: with
// s = e / (2 + e) <= 1/3, log1p(e) = 2 atanh(s) = s p(s^2), p(q) = 2 (1 + q/3 + q^2/5 + ...). The coefficients are those
// of the polynomial of degree four that is nearest to p on [0, 1/9]: off by at most 8e-9 of it (the series' own need
// degree seven; 8192 tokens of 4096 channels take 270 us, 278 with those).
__device__ __forceinline__ float softplus_of(float v) {
  const float e = exp2_of(-kLog2e * fabsf(v));
  const float s = e * __builtin_amdgcn_rcpf(2.0f + e), q = s * s;
  float p = fmaf(q, 0.2817833423614502f, 0.27960601449012756f);
  p = fmaf(q, p, 0.40024909377098083f);
  p = fmaf(q, p, 0.6666631698608398f);
  p = fmaf(q, p, 2.0f);
  return fmaf(s, p, fmaxf(v, 0.0f));
}

// silu(u) = u sigmoid(u), and its slope.
__device__ __forceinline__ float silu_of(float u) { return u * sigmoid_of(u); }
__device__ __forceinline__ float silu_slope(float u) {
  const float p = sigmoid_of(u);
  return p * fmaf(u, 1.0f - p, 1.0f);
}

// Tokens of row b that exist.
__device__ __forceinline__ int row_length(const int32_t* lengths, int b, int T) {
  return lengths ? min(max(lengths[b], 0), T) : T;
}

}  // namespace sx
