// head_rotate.hip: the norm of each head of the queries and keys and the
// rotation by position, in one pass, with its gradient.
//
//   r = 1 / sqrt(mean(x^2) + eps),  u = x r w,  y = u with the pairs of its first
//   `rot` components turned by 2 pi position turns[i]
// and back, with gu the gradient turned the other way,
//   gw += gu x r,   gx = r (gu w - x r^2 mean(gu w x))
//
// A row (one head of one token) is cut into units of two components that turn
// together: (i, i + rot/2) or (2i, 2i+1), and neighbours behind `rot` that do not
// turn. A lane holds U units of a row, so a pair never leaves its lane: U
// consecutive ones (two 16-byte pieces a row, at any alignment) where elements
// are next to each other, else every G-th one. The gradient of 7 x 2481 tokens
// of 4 + 2 heads of 194, 12 of them turned, in bf16 takes 51 us in pieces, 112
// by elements. A workgroup takes some tokens of the queries or of the keys;
// their cosines and sines are formed once for all its heads, through LDS, while
// its first rows are on their way.
// The angle is reduced in 64 bits: position times turns, its nearest whole
// number taken off; 32 bits would lose the angle of far positions.
//
// Bound by memory: 4 x 4096 tokens of 16 + 16 heads of 128 in bf16 take 59.0 us,
// 4.6 TB/s, where a copy of this size reaches 4.8; the gradient of 2 x 2048 tokens of
// 16 + 4 heads 19 us, 3.3 TB/s, of which the weights' sums over the workgroups
// are 4.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "ms_mfma.hpp"
#include "sx_attention.hpp"
#include "sx_common.hpp"

namespace sx {
namespace {

constexpr int kThreads = 256;
constexpr int kMostTokens = 16;  // tokens of a workgroup at a time
constexpr int kMaxUnits = 128;   // d <= 256
// Workgroups of queries (and of keys) a compute unit: each forms its tokens' angles before it has rows to
// store, so few are better than many. 4 x 4096 tokens of 16 + 16 heads forward: 59.3, 58.5, 60.3, 68.6 us at
// 2, 4, 8, 16; 2 x 2048 of 16 + 4 backward, with the weights' sums: 21.7, 22.3, 28.8 us at 1, 2, 4.
constexpr int kForwardPerCu = 4, kGradPerCu = 1;
constexpr int kSumRows = 64;     // partial sums of a weight's gradient that are read at once

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t words_t __attribute__((ext_vector_type(2), aligned(2)));  // of a row of any alignment
typedef uint32_t word_t __attribute__((aligned(2)));

template <bool BF>
struct El;
template <>
struct El<true> {
  using E = uint16_t;
  static constexpr int U = 8;  // units a lane
  typedef uint32_t piece_t __attribute__((ext_vector_type(4), aligned(2)));  // of a row of any alignment
  static __device__ __forceinline__ float get(E v) { return bf16_to_f32(v); }
  static __device__ __forceinline__ E put(float v) { return f32_to_bf16_rne(v); }
  static __device__ __forceinline__ void open(u32x4 a, float* v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
    }
  }
  // a piece without its first n elements
  static __device__ __forceinline__ u32x4 shifted(u32x4 v, int n) {
    if (n & 4) v = u32x4{v[2], v[3], 0, 0};
    if (n & 2) v = u32x4{v[1], v[2], v[3], 0};
    if (n & 1) v = u32x4{v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16, v[3] >> 16};
    return v;
  }
  static __device__ __forceinline__ u32x4 close(const float* v) {
    return u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
  }
};
template <>
struct El<false> {
  using E = float;
  static constexpr int U = 4;
  typedef uint32_t piece_t __attribute__((ext_vector_type(4), aligned(4)));
  static __device__ __forceinline__ float get(E v) { return v; }
  static __device__ __forceinline__ E put(float v) { return v; }
  static __device__ __forceinline__ void open(u32x4 a, float* v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(a[i]);
  }
  static __device__ __forceinline__ u32x4 shifted(u32x4 v, int n) {
    if (n & 2) v = u32x4{v[2], v[3], 0, 0};
    if (n & 1) v = u32x4{v[1], v[2], v[3], 0};
    return v;
  }
  static __device__ __forceinline__ u32x4 close(const float* v) {
    return u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
  }
};

// Which components of a row a lane holds: every G-th unit, an element at a time (Elements); or two pieces of U
// consecutive components (16 bytes), of U units that are either halves apart or neighbours. The last pieces of
// either kind may hold fewer, and are read early where the row ends (Cut). Where none does (Whole) the gradient
// of 2 x 2048 tokens of 16 + 4 heads of 128 takes 19.0 us, 20.4 with the cuts looked for.
enum class Rows { Elements, Cut, Whole };

template <bool BF, int G, Rows R>
struct Lane {
  static constexpr bool WIDE = R != Rows::Elements, whole = R == Rows::Whole;
  using T = El<BF>;
  using E = typename T::E;
  static constexpr int U = T::U;
  using piece_t = typename T::piece_t;
  int lr, half, d;
  bool split;   // pairs are halves apart, not neighbours
  // WIDE:
  bool apart;   // ... and so are this lane's
  int unit0;    // its first unit
  int at[2], count[2];

  __device__ __forceinline__ Lane(const HrParams& p, int lane_in_row)
      : lr(lane_in_row), half(p.rot / 2), d(p.d), split(!p.neighbours) {
    const int turned = split ? (half + U - 1) / U : 0;  // lanes of units halves apart
    apart = lr < turned;
    unit0 = apart ? U * lr : (split ? half : 0) + U * (lr - turned);
    at[0] = apart ? unit0 : 2 * unit0;
    at[1] = at[0] + (apart ? half : U);
    const int end0 = apart ? half : d;
    count[0] = min(max(end0 - at[0], 0), U);
    count[1] = apart ? count[0] : min(max(d - at[1], 0), U);
  }
  __device__ __forceinline__ int unit(int i) const { return WIDE ? unit0 + i : lr + G * i; }
  // where its angle is, if it turns
  __device__ __forceinline__ int angle(int i) const {
    return WIDE ? min(unit0, kMaxUnits - U) + i : min(unit(i), kMaxUnits - 1);
  }
  // component of the first (j = 0) or second of unit i, d and more where there is none
  __device__ __forceinline__ int component(int i, int j) const {
    const int k = unit(i);
    if (WIDE && apart) return i < count[0] ? k + j * half : d;
    return !WIDE && split && k < half ? k + j * half : 2 * k + j;
  }

  struct Raw {
    u32x4 v[2];          // WIDE
    E x[U], y[U];        // not
  };
  // STREAM: past the caches, which a forward pass gains by (4 x 4096 tokens of 16 + 16 heads: 59.1 us, 60.7
  // without) and a backward one does not.
  template <bool STREAM>
  __device__ __forceinline__ void load(const E* row, int64_t sd, Raw& r) const {
    if constexpr (WIDE) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const piece_t* from = reinterpret_cast<const piece_t*>(row + min(at[j], d - U));
        const u32x4 none = {0, 0, 0, 0};
        r.v[j] = count[j] > 0 ? u32x4(STREAM ? __builtin_nontemporal_load(from) : *from) : none;
      }
    } else {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        r.x[i] = component(i, 0) < d ? row[component(i, 0) * sd] : E(0);
        r.y[i] = component(i, 1) < d ? row[component(i, 1) * sd] : E(0);
      }
    }
  }
  __device__ __forceinline__ void open(const Raw& r, float (&x)[U], float (&y)[U]) const {
    if constexpr (WIDE) {
      float v[2][U];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        u32x4 w = r.v[j];
        if constexpr (!whole) w = T::shifted(w, max(at[j] - (d - U), 0) % U);
        T::open(w, v[j]);
        if constexpr (!whole) {
#pragma unroll
          for (int i = 0; i < U; ++i) v[j][i] = i < count[j] ? v[j][i] : 0.0f;
        }
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        x[i] = apart ? v[0][i] : v[2 * i / U][2 * i % U];
        y[i] = apart ? v[1][i] : v[2 * i / U][2 * i % U + 1];
      }
    } else {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        x[i] = T::get(r.x[i]);
        y[i] = T::get(r.y[i]);
      }
    }
  }
  __device__ __forceinline__ void store(E* row, const float (&x)[U], const float (&y)[U]) const {
    if constexpr (WIDE) {
      float v[2][U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        v[0][i] = apart ? x[i] : (i & 1 ? y[i / 2] : x[i / 2]);
        v[1][i] = apart ? y[i] : (i & 1 ? y[(U + i) / 2] : x[(U + i) / 2]);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        // streamed where rows end on 16-byte borders: what the L2s still held at the kernel's end would have to
        // be written then (63.1 us without). Others write parts of lines, which the caches join (3 x 2947 tokens
        // of 8 + 8 heads of 228: 46.3 us, 49.9 streamed), the last components by words (48.4 one by one).
        if (count[j] == U) {
          piece_t* to = reinterpret_cast<piece_t*>(row + at[j]);
          if constexpr (whole) __builtin_nontemporal_store(piece_t(T::close(v[j])), to);
          else *to = T::close(v[j]);
        } else if constexpr (!whole) {
          constexpr int W = 4 / sizeof(E);  // elements a word
          u32x4 w = T::close(v[j]);
          E* to = row + at[j];
          if (count[j] & 2 * W) {
            *reinterpret_cast<words_t*>(to) = words_t{w[0], w[1]};
            to += 2 * W;
            w[0] = w[2];
            w[1] = w[3];
          }
          if (count[j] & W) {
            *reinterpret_cast<word_t*>(to) = w[0];
            to += W;
            w[0] = w[1];
          }
          if (W > 1 && (count[j] & 1)) *to = E(w[0]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (component(i, 0) < d) row[component(i, 0)] = T::put(x[i]);
        if (component(i, 1) < d) row[component(i, 1)] = T::put(y[i]);
      }
    }
  }
  __device__ __forceinline__ void weights(const float* w, float (&x)[U], float (&y)[U]) const {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      x[i] = component(i, 0) < d ? (w ? w[component(i, 0)] : 1.0f) : 0.0f;
      y[i] = component(i, 1) < d ? (w ? w[component(i, 1)] : 1.0f) : 0.0f;
    }
  }
};

// Sum over the G lanes of a row, the same in each.
template <int G>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int d = 1; d < G; d *= 2) v += __shfl_xor(v, d);
  return v;
}

// Cosine and sine of `count` tokens' units that turn, from token tok0 on, into cs[token][unit].
__device__ __forceinline__ void angles(const HrParams& p, uint32_t tok0, int count, float2 (*cs)[kMaxUnits]) {
  const int half = p.rot / 2;
  for (int q = int(threadIdx.x); q < count * half; q += kThreads) {
    const int t = q / half, i = q % half;
    const uint32_t tok = tok0 + uint32_t(t), b = tok / uint32_t(p.T);
    const int64_t at = int64_t(b) * p.pb + int64_t(tok - b * uint32_t(p.T)) * p.pt;
    const double pos = p.pos64 ? double(static_cast<const int64_t*>(p.positions)[at])
                               : double(static_cast<const int32_t*>(p.positions)[at]);
    const double turn = pos * p.turns[i];
    const float f = float(turn - rint(turn));
    cs[t][i] = make_float2(cospif(2.0f * f), sinpif(2.0f * f));
  }
}

// Row q of a group: head q % heads of token tok0 + q / heads.
template <typename E>
__device__ __forceinline__ const E* row_of(const HrParams& p, const HeadView& v, uint32_t tok0, int heads, int q) {
  const uint32_t t = uint32_t(q) / uint32_t(heads), h = uint32_t(q) - t * uint32_t(heads);
  const uint32_t tok = tok0 + t, b = tok / uint32_t(p.T);
  return static_cast<const E*>(v.p) + int64_t(b) * v.sb + int64_t(tok - b * uint32_t(p.T)) * v.st + int64_t(h) * v.sh;
}

// blockIdx.y: queries or keys. G lanes a row.
template <bool BF, int G, Rows R>
__global__ __launch_bounds__(kThreads) void rotate_forward(HrParams p) {
  using L = Lane<BF, G, R>;
  using E = typename L::E;
  constexpr int U = L::U, kSlots = kThreads / G;
  __shared__ float2 cs[kMostTokens][kMaxUnits];
  const bool isq = blockIdx.y == 0;
  const HeadView& v = isq ? p.q : p.k;
  const int heads = isq ? p.hq : p.hk, tokens = isq ? p.tokens_q : p.tokens_k;
  const uint32_t all = uint32_t(p.B) * uint32_t(p.T);
  const int64_t first = int64_t(blockIdx.x) * tokens;
  if (first >= all || heads == 0) return;
  const uint32_t tok0 = uint32_t(first);
  const int count = int(min(uint32_t(tokens), all - tok0)), rows = count * heads;
  const int slot = int(threadIdx.x) / G;
  const L l(p, int(threadIdx.x) % G);
  typename L::Raw raw;
  if (slot < rows) l.template load<true>(row_of<E>(p, v, tok0, heads, slot), v.sd, raw);
  float w0[U], w1[U];
  l.weights(isq ? p.qw : p.kw, w0, w1);
  angles(p, tok0, count, cs);
  __syncthreads();
  const float inv = 1.0f / float(p.d);
  E* out = static_cast<E*>(isq ? p.out_q : p.out_k) + int64_t(tok0) * heads * p.d;
  for (int q = slot; q < rows; q += kSlots) {
    float x[U], y[U];
    l.open(raw, x, y);
    if (q + kSlots < rows) l.template load<true>(row_of<E>(p, v, tok0, heads, q + kSlots), v.sd, raw);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < U; ++i) s = fmaf(x[i], x[i], fmaf(y[i], y[i], s));
    const float r = rsqrtf(row_sum<G>(s) * inv + p.eps);
    const float2* turn = cs[q / heads];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const float2 z = turn[l.angle(i)];
      const bool turns = l.unit(i) < l.half;
      const float a = x[i] * r * w0[i], c = y[i] * r * w1[i];
      x[i] = turns ? a * z.x - c * z.y : a;
      y[i] = turns ? a * z.y + c * z.x : c;
    }
    l.store(out + int64_t(q) * p.d, x, y);
  }
}

// A workgroup takes every gridDim.x-th group of tokens and leaves one partial sum of the weight's gradient.
template <bool BF, int G, Rows R>
__global__ __launch_bounds__(kThreads) void rotate_backward(HrParams p) {
  using L = Lane<BF, G, R>;
  using E = typename L::E;
  constexpr int U = L::U, kSlots = kThreads / G;
  __shared__ union {
    float2 cs[kMostTokens][kMaxUnits];
    float sums[kSlots][2 * U * G];
  } lds;
  const bool isq = blockIdx.y == 0;
  const HeadView& v = isq ? p.q : p.k;
  const HeadView& gv = isq ? p.gq : p.gk;
  const int heads = isq ? p.hq : p.hk, tokens = isq ? p.tokens_q : p.tokens_k;
  const uint32_t all = uint32_t(p.B) * uint32_t(p.T);
  const int slot = int(threadIdx.x) / G;
  const L l(p, int(threadIdx.x) % G);
  float w0[U], w1[U], g0[U], g1[U];
  l.weights(isq ? p.qw : p.kw, w0, w1);
#pragma unroll
  for (int i = 0; i < U; ++i) g0[i] = g1[i] = 0.0f;
  const float inv = 1.0f / float(p.d);
  for (int64_t first = int64_t(blockIdx.x) * tokens; first < all && heads > 0; first += int64_t(gridDim.x) * tokens) {
    const uint32_t tok0 = uint32_t(first);
    const int count = int(min(uint32_t(tokens), all - tok0)), rows = count * heads;
    typename L::Raw raw, graw;
    if (slot < rows) {
      l.template load<false>(row_of<E>(p, v, tok0, heads, slot), v.sd, raw);
      l.template load<false>(row_of<E>(p, gv, tok0, heads, slot), gv.sd, graw);
    }
    __syncthreads();
    angles(p, tok0, count, lds.cs);
    __syncthreads();
    E* out = static_cast<E*>(isq ? p.out_q : p.out_k) + int64_t(tok0) * heads * p.d;
    for (int q = slot; q < rows; q += kSlots) {
      float x[U], y[U], a[U], c[U];
      l.open(raw, x, y);
      l.open(graw, a, c);
      if (q + kSlots < rows) {
        l.template load<false>(row_of<E>(p, v, tok0, heads, q + kSlots), v.sd, raw);
        l.template load<false>(row_of<E>(p, gv, tok0, heads, q + kSlots), gv.sd, graw);
      }
      const float2* turn = lds.cs[q / heads];
      float s = 0.0f, dot = 0.0f;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const float2 z = turn[l.angle(i)];
        const bool turns = l.unit(i) < l.half;
        const float e = a[i], f = c[i];
        a[i] = turns ? e * z.x + f * z.y : e;  // the gradient of u
        c[i] = turns ? f * z.x - e * z.y : f;
        s = fmaf(x[i], x[i], fmaf(y[i], y[i], s));
        dot = fmaf(a[i] * w0[i], x[i], fmaf(c[i] * w1[i], y[i], dot));
      }
      const float r = rsqrtf(row_sum<G>(s) * inv + p.eps);
      const float along = row_sum<G>(dot) * inv * r * r;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        g0[i] = fmaf(a[i], x[i] * r, g0[i]);
        g1[i] = fmaf(c[i], y[i] * r, g1[i]);
        x[i] = (a[i] * w0[i] - x[i] * along) * r;
        y[i] = (c[i] * w1[i] - y[i] * along) * r;
      }
      l.store(out + int64_t(q) * p.d, x, y);
    }
  }
  if (!(isq ? p.gqw : p.gkw)) return;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < U; ++i) {
    lds.sums[slot][2 * U * l.lr + i] = g0[i];
    lds.sums[slot][2 * U * l.lr + U + i] = g1[i];
  }
  __syncthreads();
  float* partial = p.partial + (int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * p.d;
  for (int q = int(threadIdx.x); q < 2 * U * G; q += kThreads) {
    float s = 0.0f;
    for (int i = 0; i < kSlots; ++i) s += lds.sums[i][q];
    const L w(p, q / (2 * U));
    const int col = w.component(q % U, q % (2 * U) < U ? 0 : 1);
    if (col < p.d) partial[col] = s;
  }
}

// The workgroups' partial sums, in a fixed order: a workgroup takes 4 columns, kSumRows partial sums at once.
__global__ __launch_bounds__(kThreads) void weight_sum(HrParams p, int groups) {
  __shared__ float l[kSumRows][4];
  const int which = blockIdx.y, c = int(threadIdx.x) & 3, part = int(threadIdx.x) >> 2;
  const int col = int(blockIdx.x) * 4 + c;
  float* to = which ? p.gkw : p.gqw;
  if (!to) return;
  const float* from = p.partial + int64_t(which) * groups * p.d;
  float s = 0.0f;
  if (col < p.d) {
#pragma unroll 4
    for (int i = part; i < groups; i += kSumRows) s += from[int64_t(i) * p.d + col];
  }
  l[part][c] = s;
  __syncthreads();
  for (int d = kSumRows / 2; d > 0; d /= 2) {
    if (part < d) l[part][c] += l[part + d][c];
    __syncthreads();
  }
  if (part == 0 && col < p.d) to[col] = l[0][c];
}

// Tokens of a workgroup at a time: about 256 rows, but four workgroups a compute unit where there are so many.
int tokens_of(int64_t all, int heads, int per_cu) {
  const int64_t rows = std::max<int64_t>(1, 256 / std::max(heads, 1));
  const int64_t spread = std::max<int64_t>(1, all / (per_cu * device_cu_count()));
  return int(std::min<int64_t>({rows, spread, kMostTokens}));
}

int64_t groups_of(const HrParams& p) {
  const int64_t all = int64_t(p.B) * p.T;
  return std::max((all + p.tokens_q - 1) / p.tokens_q, (all + p.tokens_k - 1) / p.tokens_k);
}

HrParams with_tokens(const HrParams& given, int per_cu) {
  HrParams p = given;
  const int64_t all = int64_t(p.B) * p.T;
  p.tokens_q = tokens_of(all, p.hq, per_cu);
  p.tokens_k = tokens_of(all, p.hk, per_cu);
  return p;
}

template <bool BF, int G, Rows R>
void launch_rows(const HrParams& p, dim3 grid, bool gradient, hipStream_t stream) {
  if (gradient) rotate_backward<BF, G, R><<<grid, kThreads, 0, stream>>>(p);
  else rotate_forward<BF, G, R><<<grid, kThreads, 0, stream>>>(p);
}

template <bool BF, int G>
void launch_lanes(const HrParams& p, dim3 grid, bool gradient, hipStream_t stream) {
  bool wide = p.q.unit && (p.hk == 0 || p.k.unit);
  if (gradient) wide = wide && p.gq.unit && (p.hk == 0 || p.gk.unit);
  constexpr int U = El<BF>::U;
  const bool whole = p.d % U == 0 && (p.neighbours || p.rot / 2 % U == 0);
  if (!wide) return launch_rows<BF, G, Rows::Elements>(p, grid, gradient, stream);
  if constexpr (G * U <= kMaxUnits)  // else only cut rows take so many lanes
    if (whole) return launch_rows<BF, G, Rows::Whole>(p, grid, gradient, stream);
  launch_rows<BF, G, Rows::Cut>(p, grid, gradient, stream);
}

template <bool BF>
void launch_width(const HrParams& p, dim3 grid, bool gradient, hipStream_t stream) {
  constexpr int U = El<BF>::U;
  const int half = p.neighbours ? 0 : p.rot / 2;
  const int need = (half + U - 1) / U + (p.d - 2 * half + 2 * U - 1) / (2 * U);
  if (need <= 2) launch_lanes<BF, 2>(p, grid, gradient, stream);
  else if (need <= 4) launch_lanes<BF, 4>(p, grid, gradient, stream);
  else if (need <= 8) launch_lanes<BF, 8>(p, grid, gradient, stream);
  else if (need <= 16) launch_lanes<BF, 16>(p, grid, gradient, stream);
  else if (BF || need <= 32) launch_lanes<BF, 32>(p, grid, gradient, stream);
  else if constexpr (!BF) launch_lanes<BF, 64>(p, grid, gradient, stream);
}

}  // namespace

int head_rotate_backward_groups(const HrParams& given) {
  return int(std::min<int64_t>(groups_of(with_tokens(given, kGradPerCu)), 4 * int64_t(device_cu_count())));
}

hipError_t launch_head_rotate(const HrParams& given, hipStream_t stream) {
  const HrParams p = with_tokens(given, kForwardPerCu);
  const dim3 grid(unsigned(groups_of(p)), p.hk > 0 ? 2 : 1);
  if (p.bf16) launch_width<true>(p, grid, false, stream);
  else launch_width<false>(p, grid, false, stream);
  return hipGetLastError();
}

hipError_t launch_head_rotate_backward(const HrParams& given, hipStream_t stream) {
  const HrParams p = with_tokens(given, kGradPerCu);
  const int groups = head_rotate_backward_groups(p);
  if (groups > 0) {
    const dim3 grid(unsigned(groups), 2);
    if (p.bf16) launch_width<true>(p, grid, true, stream);
    else launch_width<false>(p, grid, true, stream);
  }
  if (p.gqw || p.gkw) weight_sum<<<dim3((p.d + 3) / 4, 2), kThreads, 0, stream>>>(p, groups);
  return hipGetLastError();
}

}  // namespace sx
