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
// turn. A lane holds four consecutive units of a row, so a pair never leaves its
// lane. A token's cosines and sines are formed once for all its heads, through
// LDS. The angle is reduced in 64 bits: position times turns, its nearest whole
// number taken off; 32 bits would lose the angle of far positions.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "ms_mfma.hpp"
#include "sx_attention.hpp"
#include "sx_common.hpp"

namespace sx {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 4;       // tokens a workgroup takes at a time where there are many
constexpr int kMaxUnits = 128;   // d <= 256

template <bool BF>
struct El {
  using E = uint16_t;
  static __device__ __forceinline__ float get(E v) { return bf16_to_f32(v); }
  static __device__ __forceinline__ E put(float v) { return f32_to_bf16_rne(v); }
  static __device__ __forceinline__ f32x4 get4(const E* p) {
    const uint2 a = *reinterpret_cast<const uint2*>(p);
    return f32x4{__uint_as_float(a.x << 16), __uint_as_float(a.x & 0xffff0000u), __uint_as_float(a.y << 16),
                 __uint_as_float(a.y & 0xffff0000u)};
  }
  static __device__ __forceinline__ void put4(E* p, f32x4 v) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  }
};
template <>
struct El<false> {
  using E = float;
  static __device__ __forceinline__ float get(E v) { return v; }
  static __device__ __forceinline__ E put(float v) { return v; }
  static __device__ __forceinline__ f32x4 get4(const E* p) { return *reinterpret_cast<const f32x4*>(p); }
  static __device__ __forceinline__ void put4(E* p, f32x4 v) { *reinterpret_cast<f32x4*>(p) = v; }
};

// The components of a lane's four units.
struct Units {
  int first[4], second[4];
  bool four;   // first[] and second[] are each four consecutive components, or eight in a row
  bool joint;  // units are neighbours: first, second alternate
};

__device__ __forceinline__ Units units_of(const HrParams& p, int lane_in_row) {
  Units u;
  const int half = p.rot / 2, i0 = 4 * lane_in_row;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = i0 + i;
    const bool split = k < half && !p.neighbours;
    u.first[i] = split ? k : 2 * k;
    u.second[i] = split ? k + half : 2 * k + 1;
  }
  u.joint = !(i0 < half && !p.neighbours);
  u.four = (half & 3) == 0 || p.neighbours;
  return u;
}

// A lane's components of a row (zero where there are none): x[i] the firsts, y[i] the seconds.
template <bool BF>
__device__ __forceinline__ void load_units(const typename El<BF>::E* row, int64_t sd, bool vec, int d, const Units& u,
                                           f32x4& x, f32x4& y) {
  using T = El<BF>;
  x = y = zero4();
  if (vec && u.four) {
    if (u.joint) {
      if (u.first[0] < d) {
        const f32x4 a = T::get4(row + u.first[0]), b = T::get4(row + u.first[0] + 4);
        x = f32x4{a[0], a[2], b[0], b[2]};
        y = f32x4{a[1], a[3], b[1], b[3]};
      }
    } else {
      x = T::get4(row + u.first[0]);
      y = T::get4(row + u.second[0]);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (u.first[i] < d) x[i] = T::get(row[u.first[i] * sd]);
    if (u.second[i] < d) y[i] = T::get(row[u.second[i] * sd]);
  }
}

template <bool BF>
__device__ __forceinline__ void store_units(typename El<BF>::E* row, bool vec, int d, const Units& u, f32x4 x,
                                            f32x4 y) {
  using T = El<BF>;
  if (vec && u.four) {
    if (u.joint) {
      if (u.first[0] < d) {
        T::put4(row + u.first[0], f32x4{x[0], y[0], x[1], y[1]});
        T::put4(row + u.first[0] + 4, f32x4{x[2], y[2], x[3], y[3]});
      }
    } else {
      T::put4(row + u.first[0], x);
      T::put4(row + u.second[0], y);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (u.first[i] < d) row[u.first[i]] = T::put(x[i]);
    if (u.second[i] < d) row[u.second[i]] = T::put(y[i]);
  }
}

template <int G>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int d = 1; d < G; d *= 2) v += __shfl_xor(v, d);
  return v;
}

__device__ __forceinline__ double position_of(const HrParams& p, int64_t tok) {
  const int64_t at = tok / p.T * p.pb + tok % p.T * p.pt;
  return p.pos64 ? double(static_cast<const int64_t*>(p.positions)[at])
                 : double(static_cast<const int32_t*>(p.positions)[at]);
}

// Cosine and sine of `count` tokens' units into cs[token][unit].
__device__ __forceinline__ void angles(const HrParams& p, int64_t tok0, int count, float2 (*cs)[kMaxUnits]) {
  const int half = p.rot / 2, units = (p.d + 1) / 2;
  for (int q = int(threadIdx.x); q < count * units; q += kThreads) {
    const int t = q / units, i = q % units;
    float2 v = make_float2(1.0f, 0.0f);
    if (i < half) {
      const double turn = position_of(p, tok0 + t) * p.turns[i];
      const float f = float(turn - rint(turn));
      v = make_float2(cospif(2.0f * f), sinpif(2.0f * f));
    }
    cs[t][i] = v;
  }
}

__device__ __forceinline__ void load_weights(const float* w, int d, const Units& u, f32x4& x, f32x4& y) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = u.first[i] < d ? (w ? w[u.first[i]] : 1.0f) : 0.0f;
    y[i] = u.second[i] < d ? (w ? w[u.second[i]] : 1.0f) : 0.0f;
  }
}

// G lanes a row.
template <bool BF, int G>
__global__ __launch_bounds__(kThreads) void rotate_forward(HrParams p, int tokens) {
  using E = typename El<BF>::E;
  __shared__ float2 cs[kTokens][kMaxUnits];
  const int lr = int(threadIdx.x) % G, slot = int(threadIdx.x) / G, heads = p.hq + p.hk;
  const int64_t all = int64_t(p.B) * p.T, tok0 = int64_t(blockIdx.x) * tokens;
  const int count = int(min(int64_t(tokens), all - tok0));
  const int units = (p.d + 1) / 2;
  const Units u = units_of(p, lr);
  f32x4 wq0, wq1, wk0, wk1;
  load_weights(p.qw, p.d, u, wq0, wq1);
  load_weights(p.kw, p.d, u, wk0, wk1);
  angles(p, tok0, count, cs);
  __syncthreads();
  const float inv = 1.0f / float(p.d);
  for (int q = slot; q < count * heads; q += kThreads / G) {
    const int t = q / heads, hh = q % heads;
    const bool isq = hh < p.hq;
    const int h = isq ? hh : hh - p.hq, nh = isq ? p.hq : p.hk;
    const HeadView& v = isq ? p.q : p.k;
    const int64_t tok = tok0 + t, b = tok / p.T, tt = tok % p.T;
    f32x4 x, y;
    load_units<BF>(static_cast<const E*>(v.p) + b * v.sb + tt * v.st + h * v.sh, v.sd, v.vec, p.d, u, x, y);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) s = fmaf(x[i], x[i], fmaf(y[i], y[i], s));
    const float r = rsqrtf(row_sum<G>(s) * inv + p.eps);
    const f32x4 a = x * r * (isq ? wq0 : wk0), c = y * r * (isq ? wq1 : wk1);
    f32x4 o0, o1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 z = 4 * lr + i < units ? cs[t][4 * lr + i] : make_float2(1.0f, 0.0f);
      o0[i] = a[i] * z.x - c[i] * z.y;
      o1[i] = a[i] * z.y + c[i] * z.x;
    }
    E* to = static_cast<E*>(isq ? p.out_q : p.out_k) + (tok * nh + h) * p.d;
    store_units<BF>(to, (p.d & 7) == 0, p.d, u, o0, o1);
  }
}

template <bool BF, int G>
__global__ __launch_bounds__(kThreads) void rotate_backward(HrParams p, int tokens, int64_t groups) {
  using E = typename El<BF>::E;
  __shared__ float2 cs[kTokens][kMaxUnits];
  __shared__ float sums[kThreads / G][2][2 * 4 * G];
  const int lr = int(threadIdx.x) % G, slot = int(threadIdx.x) / G, heads = p.hq + p.hk;
  const int64_t all = int64_t(p.B) * p.T;
  const int units = (p.d + 1) / 2;
  const Units u = units_of(p, lr);
  f32x4 wq0, wq1, wk0, wk1;
  load_weights(p.qw, p.d, u, wq0, wq1);
  load_weights(p.kw, p.d, u, wk0, wk1);
  f32x4 gq0 = zero4(), gq1 = zero4(), gk0 = zero4(), gk1 = zero4();
  const float inv = 1.0f / float(p.d);
  for (int64_t grp = blockIdx.x; grp < groups; grp += gridDim.x) {
    const int64_t tok0 = grp * tokens;
    const int count = int(min(int64_t(tokens), all - tok0));
    __syncthreads();
    angles(p, tok0, count, cs);
    __syncthreads();
    for (int q = slot; q < count * heads; q += kThreads / G) {
      const int t = q / heads, hh = q % heads;
      const bool isq = hh < p.hq;
      const int h = isq ? hh : hh - p.hq, nh = isq ? p.hq : p.hk;
      const HeadView& v = isq ? p.q : p.k;
      const HeadView& gv = isq ? p.gq : p.gk;
      const int64_t tok = tok0 + t, b = tok / p.T, tt = tok % p.T;
      f32x4 x, y, e, f;
      load_units<BF>(static_cast<const E*>(v.p) + b * v.sb + tt * v.st + h * v.sh, v.sd, v.vec, p.d, u, x, y);
      load_units<BF>(static_cast<const E*>(gv.p) + b * gv.sb + tt * gv.st + h * gv.sh, gv.sd, gv.vec, p.d, u, e, f);
      f32x4 a, c;  // the gradient of u
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 z = 4 * lr + i < units ? cs[t][4 * lr + i] : make_float2(1.0f, 0.0f);
        a[i] = e[i] * z.x + f[i] * z.y;
        c[i] = f[i] * z.x - e[i] * z.y;
      }
      const f32x4 n0 = a * (isq ? wq0 : wk0), n1 = c * (isq ? wq1 : wk1);
      float s = 0.0f, dot = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s = fmaf(x[i], x[i], fmaf(y[i], y[i], s));
        dot = fmaf(n0[i], x[i], fmaf(n1[i], y[i], dot));
      }
      const float r = rsqrtf(row_sum<G>(s) * inv + p.eps);
      const float along = row_sum<G>(dot) * inv * r * r;
      if (isq) {
        gq0 += a * x * r;
        gq1 += c * y * r;
      } else {
        gk0 += a * x * r;
        gk1 += c * y * r;
      }
      E* to = static_cast<E*>(isq ? p.out_q : p.out_k) + (tok * nh + h) * p.d;
      store_units<BF>(to, (p.d & 7) == 0, p.d, u, (n0 - x * along) * r, (n1 - y * along) * r);
    }
  }
  if (!p.gqw && !p.gkw) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sums[slot][0][8 * lr + i] = gq0[i];
    sums[slot][0][8 * lr + 4 + i] = gq1[i];
    sums[slot][1][8 * lr + i] = gk0[i];
    sums[slot][1][8 * lr + 4 + i] = gk1[i];
  }
  __syncthreads();
  for (int q = int(threadIdx.x); q < 2 * 8 * G; q += kThreads) {
    const int which = q / (8 * G), at = q % (8 * G);
    float s = 0.0f;
    for (int i = 0; i < kThreads / G; ++i) s += sums[i][which][at];
    const Units w = units_of(p, at / 8);
    int col = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (at % 8 == i) col = w.first[i];
      if (at % 8 == 4 + i) col = w.second[i];
    }
    if (col < p.d) p.partial[(int64_t(blockIdx.x) * 2 + which) * p.d + col] = s;
  }
}

// The workgroups' partial weight gradients, in their order: one workgroup a 64 columns.
__global__ __launch_bounds__(kThreads) void weight_sum(HrParams p, int groups) {
  __shared__ float l[kThreads / 64][64];
  const int which = blockIdx.y, lane = int(threadIdx.x) & 63, part = int(threadIdx.x) >> 6;
  const int col = int(blockIdx.x) * 64 + lane;
  float* to = which ? p.gkw : p.gqw;
  if (!to) return;
  float s = 0.0f;
  if (col < p.d)
    for (int i = part; i < groups; i += kThreads / 64) s += p.partial[(int64_t(i) * 2 + which) * p.d + col];
  l[part][lane] = s;
  __syncthreads();
  if (part == 0 && col < p.d) {
    for (int i = 1; i < kThreads / 64; ++i) s += l[i][lane];
    to[col] = s;
  }
}

int lanes_of(int d) {
  const int need = ((d + 1) / 2 + 3) / 4;
  int g = 4;
  while (g < need) g *= 2;
  return g;
}

int tokens_of(const HrParams& p) { return int64_t(p.B) * p.T >= 2048 ? kTokens : 1; }

template <bool BF>
hipError_t forward(const HrParams& p, hipStream_t stream) {
  const int tokens = tokens_of(p);
  const unsigned grid = unsigned((int64_t(p.B) * p.T + tokens - 1) / tokens);
  if (grid == 0) return hipSuccess;
  switch (lanes_of(p.d)) {
    case 4: rotate_forward<BF, 4><<<grid, kThreads, 0, stream>>>(p, tokens); break;
    case 8: rotate_forward<BF, 8><<<grid, kThreads, 0, stream>>>(p, tokens); break;
    case 16: rotate_forward<BF, 16><<<grid, kThreads, 0, stream>>>(p, tokens); break;
    default: rotate_forward<BF, 32><<<grid, kThreads, 0, stream>>>(p, tokens); break;
  }
  return hipGetLastError();
}

template <bool BF>
hipError_t backward(const HrParams& p, hipStream_t stream) {
  const int tokens = tokens_of(p), grid = head_rotate_backward_groups(p);
  const int64_t groups = (int64_t(p.B) * p.T + tokens - 1) / tokens;
  if (groups > 0) switch (lanes_of(p.d)) {
    case 4: rotate_backward<BF, 4><<<grid, kThreads, 0, stream>>>(p, tokens, groups); break;
    case 8: rotate_backward<BF, 8><<<grid, kThreads, 0, stream>>>(p, tokens, groups); break;
    case 16: rotate_backward<BF, 16><<<grid, kThreads, 0, stream>>>(p, tokens, groups); break;
    default: rotate_backward<BF, 32><<<grid, kThreads, 0, stream>>>(p, tokens, groups); break;
  }
  if (p.gqw || p.gkw) weight_sum<<<dim3((p.d + 63) / 64, 2), kThreads, 0, stream>>>(p, grid);
  return hipGetLastError();
}

}  // namespace

int head_rotate_backward_groups(const HrParams& p) {
  const int tokens = tokens_of(p);
  const int64_t groups = (int64_t(p.B) * p.T + tokens - 1) / tokens;
  return int(std::min<int64_t>(groups, 4 * int64_t(device_cu_count())));
}

hipError_t launch_head_rotate(const HrParams& p, hipStream_t stream) {
  return p.bf16 ? forward<true>(p, stream) : forward<false>(p, stream);
}

hipError_t launch_head_rotate_backward(const HrParams& p, hipStream_t stream) {
  return p.bf16 ? backward<true>(p, stream) : backward<false>(p, stream);
}

}  // namespace sx
