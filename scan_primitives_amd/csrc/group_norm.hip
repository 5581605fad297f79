// group_norm.hip: the norm of groups of channels, channels last, with an
// optional SiLU, and its gradient.
//
//   n = (x - mean) / sqrt(variance + eps) over a sample's positions and a group's channels,
//   u = n w + bias,  y = u or u sigmoid(u)
//   gu = gy, or gy times SiLU's slope at u;  gw = sum of gu n,  gb = sum of gu,
//   gx = r (gu w - mean(gu w) - n mean(gu w n)),  r = 1 / sqrt(variance + eps)
//
// Two ways. Where a sample is one position (each token normed on its own), L lanes
// hold a group in registers, x is read once, and the variance is of the
// differences from the mean; a lane keeps its channels from row to row, so the weights
// are read once and their gradients stay in registers (rows_*).
// Else the positions are cut into chunks: one launch leaves each chunk's count, mean and
// squared distance from it (joined pair by pair, so no large mean cancels), the next
// joins the chunks' and normalises; the gradient has one more for its two sums (map_*).
// Bound by memory.
#include <algorithm>

#include "sx_state_space.hpp"

namespace sx {
namespace {

constexpr int kThreads = 256;

template <bool BF, int V>
struct Chan {  // V channels' weights
  float w[V], bias[V];
  __device__ __forceinline__ void load(const GnParams& p, int c, bool is) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      w[v] = is ? (p.w ? p.w[c + v] : 1.0f) : 0.0f;
      bias[v] = is && p.bias ? p.bias[c + v] : 0.0f;
    }
  }
};

// ---------------------------------------------------------------- rows

// Sum over the L lanes of a group, the same in each. `l` holds a value a wave; two calls in a row take one each.
template <int L>
__device__ __forceinline__ float lanes_sum(float v, float* l) {
#pragma unroll
  for (int m = 1; m < (L < kWave ? L : kWave); m *= 2) v += __shfl_xor(v, m);
  if constexpr (L > kWave) {
    if (threadIdx.x % kWave == 0) l[threadIdx.x / kWave] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < L / kWave; ++i) v += l[i];
  }
  return v;
}

// Which row and group a thread has, of the first iteration.
template <int L>
struct Slot {
  int group, lane;
  int64_t row, step;
  bool any;
  __device__ __forceinline__ Slot(const GnParams& p) {
    constexpr int S = kThreads / L;
    const int slot = int(threadIdx.x) / L;
    lane = int(threadIdx.x) % L;
    const int rows = p.g >= S ? 1 : S / p.g;  // at once
    const int off = p.g >= S ? 0 : slot / p.g;
    group = p.g >= S ? int(blockIdx.y) * S + slot : slot % p.g;
    any = group < p.g && off < rows;
    row = int64_t(blockIdx.x) * rows + off;
    step = int64_t(gridDim.x) * rows;
    if (!any) row = p.n;
  }
};

template <bool BF, int V, int L, int M>
__global__ __launch_bounds__(kThreads) void rows_forward(GnParams p) {
  using P = Piece<BF, V>;
  using E = typename P::E;
  __shared__ float l[2][kThreads / kWave];
  const Slot<L> s(p);
  const int per = p.c / p.g, pieces = per / V;
  const float inv = 1.0f / float(per);
  Chan<BF, V> ch[M];
  int c[M];
  bool is[M];
#pragma unroll
  for (int m = 0; m < M; ++m) {
    is[m] = s.any && s.lane + L * m < pieces;
    c[m] = s.group * per + (s.lane + L * m) * V;
    ch[m].load(p, c[m], is[m]);
  }
  const E* x = static_cast<const E*>(p.x);
  typename P::Raw raw[M];
  const auto read = [&](int64_t row) {
#pragma unroll
    for (int m = 0; m < M; ++m) raw[m] = is[m] && row < p.n ? P::load(x + row * p.xn + c[m]) : P::zero();
  };
  read(s.row);
  // every thread takes part in the sums of as many rows
  const int64_t first = int64_t(blockIdx.x) * (s.step / gridDim.x);
  for (int64_t at = first, row = s.row; at < p.n; at += s.step, row += s.step) {
    float v[M][V], sum = 0.0f;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      P::open(raw[m], v[m]);
#pragma unroll
      for (int k = 0; k < V; ++k) sum += v[m][k];
    }
    read(row + s.step);
    const float mean = lanes_sum<L>(sum, l[0]) * inv;
    float sq = 0.0f;
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int k = 0; k < V; ++k) {
        v[m][k] -= mean;
        sq = is[m] ? fmaf(v[m][k], v[m][k], sq) : sq;
      }
    const float r = rsqrtf(fmaf(lanes_sum<L>(sq, l[1]), inv, p.eps));
#pragma unroll
    for (int m = 0; m < M; ++m) {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        v[m][k] = fmaf(v[m][k] * r, ch[m].w[k], ch[m].bias[k]);
        if (p.silu) v[m][k] = silu_of(v[m][k]);
      }
      if (is[m] && row < p.n) P::store(static_cast<E*>(p.out) + row * p.c + c[m], v[m]);
    }
  }
}

template <bool BF, int V, int L, int M>
__global__ __launch_bounds__(kThreads) void rows_backward(GnParams p) {
  using P = Piece<BF, V>;
  using E = typename P::E;
  __shared__ float l[4][kThreads / kWave];
  const Slot<L> s(p);
  const int per = p.c / p.g, pieces = per / V;
  const float inv = 1.0f / float(per);
  Chan<BF, V> ch[M];
  int c[M];
  bool is[M];
  float gw[M][V] = {}, gb[M][V] = {};
#pragma unroll
  for (int m = 0; m < M; ++m) {
    is[m] = s.any && s.lane + L * m < pieces;
    c[m] = s.group * per + (s.lane + L * m) * V;
    ch[m].load(p, c[m], is[m]);
  }
  const E* x = static_cast<const E*>(p.x);
  const E* go = static_cast<const E*>(p.go);
  typename P::Raw raw[M], graw[M];
  const auto read = [&](int64_t row) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      raw[m] = is[m] && row < p.n ? P::load(x + row * p.xn + c[m]) : P::zero();
      graw[m] = is[m] && row < p.n ? P::load(go + row * p.gon + c[m]) : P::zero();
    }
  };
  read(s.row);
  const int64_t first = int64_t(blockIdx.x) * (s.step / gridDim.x);
  for (int64_t at = first, row = s.row; at < p.n; at += s.step, row += s.step) {
    float v[M][V], g[M][V], sum = 0.0f;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      P::open(raw[m], v[m]);
      P::open(graw[m], g[m]);
#pragma unroll
      for (int k = 0; k < V; ++k) sum += v[m][k];
    }
    read(row + s.step);
    const float mean = lanes_sum<L>(sum, l[0]) * inv;
    float sq = 0.0f;
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int k = 0; k < V; ++k) {
        v[m][k] -= mean;
        sq = is[m] ? fmaf(v[m][k], v[m][k], sq) : sq;
      }
    const float r = rsqrtf(fmaf(lanes_sum<L>(sq, l[1]), inv, p.eps));
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float n = v[m][k] * r;
        if (p.silu) g[m][k] *= silu_slope(fmaf(n, ch[m].w[k], ch[m].bias[k]));
        gw[m][k] = fmaf(g[m][k], n, gw[m][k]);
        gb[m][k] += g[m][k];
        g[m][k] *= ch[m].w[k];
        s1 += g[m][k];
        s2 = fmaf(g[m][k], n, s2);
        v[m][k] = n;
      }
    s1 = lanes_sum<L>(s1, l[2]) * inv;
    s2 = lanes_sum<L>(s2, l[3]) * inv;
#pragma unroll
    for (int m = 0; m < M; ++m) {
#pragma unroll
      for (int k = 0; k < V; ++k) v[m][k] = r * (g[m][k] - s1 - v[m][k] * s2);
      if (is[m] && row < p.n) P::store(static_cast<E*>(p.out) + row * p.c + c[m], v[m]);
    }
  }
  if (s.any) {
    const int rows = int(s.step / gridDim.x);
    float* part = p.sums + (int64_t(blockIdx.x) * rows + (s.row - int64_t(blockIdx.x) * rows)) * 2 * p.c;
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (is[m]) {
          part[c[m] + k] = gw[m][k];
          part[p.c + c[m] + k] = gb[m][k];
        }
  }
}

// ---------------------------------------------------------------- maps

// How a sample's channels are spread over workgroups: blocks of whole groups, or of a part of one wide group.
struct Blocks {
  int pieces;     // of a group
  int parts;      // blocks a group takes (1: a block takes `groups` of them)
  int groups;
  int width;      // pieces of a block
  int count;      // blocks
  int rows;       // positions at once
};
template <int V>
__host__ __device__ __forceinline__ Blocks blocks_of(const GnParams& p) {
  Blocks k;
  k.pieces = p.c / p.g / V;
  if (k.pieces <= kThreads) {
    k.parts = 1;
    k.groups = kThreads / k.pieces < p.g ? kThreads / k.pieces : p.g;
    k.width = k.groups * k.pieces;
    k.count = (p.g + k.groups - 1) / k.groups;
  } else {
    k.parts = (k.pieces + kThreads - 1) / kThreads;
    k.groups = 1;
    k.width = kThreads;
    k.count = p.g * k.parts;
  }
  k.rows = kThreads / k.width;
  return k;
}

// A thread of a block: its piece and first position.
template <int V>
struct Place {
  Blocks k;
  int64_t sample, p0, p1;
  int chunk, block, piece, off, group, part, c;  // group: of the first of the block; c: first channel
  bool any;
  __device__ __forceinline__ Place(const GnParams& p) : k(blocks_of<V>(p)) {
    uint32_t at = blockIdx.x;
    block = int(at % uint32_t(k.count));
    at /= uint32_t(k.count);
    chunk = int(at % uint32_t(p.chunks));
    sample = at / uint32_t(p.chunks);
    p0 = chunk * p.chunk;
    p1 = p0 + p.chunk < p.s ? p0 + p.chunk : p.s;
    piece = int(threadIdx.x) % k.width;
    off = int(threadIdx.x) / k.width;
    group = k.parts == 1 ? block * k.groups : block / k.parts;
    part = k.parts == 1 ? 0 : block % k.parts;
    const int first = part * kThreads + piece;  // from the group's first piece on
    c = group * (p.c / p.g) + first * V;
    any = off < k.rows && (k.parts == 1 ? group + piece / k.pieces < p.g : first < k.pieces);
  }
  __device__ __forceinline__ int groups_here(const GnParams& p) const { return min(k.groups, p.g - group); }
};

struct Moments {  // of `n` values: their mean and squared distances from it
  float n, mean, m2;
  __device__ __forceinline__ void join(const Moments& o) {
    const float all = n + o.n, part = all > 0.0f ? o.n / all : 0.0f, off = o.mean - mean;
    mean = fmaf(off, part, mean);
    m2 += o.m2 + off * off * n * part;
    n = all;
  }
  __device__ __forceinline__ void over_wave() {
#pragma unroll
    for (int m = 1; m < kWave; m *= 2) join({__shfl_xor(n, m), __shfl_xor(mean, m), __shfl_xor(m2, m)});
  }
};

template <bool BF, int V>
__global__ __launch_bounds__(kThreads) void map_stats(GnParams p) {
  using P = Piece<BF, V>;
  using E = typename P::E;
  __shared__ Moments l[kThreads];
  const Place<V> a(p);
  const E* x = static_cast<const E*>(p.x) + a.sample * p.xn + a.c;
  // differences from the thread's first value
  float shift = 0.0f, sum = 0.0f, sq = 0.0f, n = 0.0f;
  if (a.any && a.p0 + a.off < a.p1) {
    float first[V];
    P::open(P::load(x + (a.p0 + a.off) * p.xs), first);
    shift = first[0];
#pragma unroll 4
    for (int64_t t = a.p0 + a.off; t < a.p1; t += a.k.rows) {
      float v[V];
      P::open(P::load(x + t * p.xs), v);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float d = v[k] - shift;
        sum += d;
        sq = fmaf(d, d, sq);
      }
      n += float(V);
    }
  }
  const float off = n > 0.0f ? sum / n : 0.0f;
  l[threadIdx.x] = {n, shift + off, fmaxf(sq - sum * off, 0.0f)};
  __syncthreads();
  // a wave a group: its threads' values, of `pieces` pieces next to each other in each of the rows
  const int lane = int(threadIdx.x) % kWave, per = a.k.parts == 1 ? a.k.pieces : a.k.width;
  for (int g = int(threadIdx.x) / kWave; g < a.groups_here(p); g += kThreads / kWave) {
    Moments m{0.0f, 0.0f, 0.0f};
    for (int i = lane; i < per * a.k.rows; i += kWave) m.join(l[i / per * a.k.width + g * per + i % per]);
    m.over_wave();
    if (lane == 0) {
      float* to = p.stats + ((((a.sample * p.chunks + a.chunk) * p.g) + a.group + g) * a.k.parts + a.part) * 3;
      to[0] = m.n;
      to[1] = m.mean;
      to[2] = m.m2;
    }
  }
}

// Mean and 1 / sqrt(variance + eps) of the block's groups, from all chunks, into lm and lr.
template <int V>
__device__ __forceinline__ void joined_stats(const GnParams& p, const Place<V>& a, float* lm, float* lr) {
  const int lane = int(threadIdx.x) % kWave, entries = p.chunks * a.k.parts;
  for (int g = int(threadIdx.x) / kWave; g < a.groups_here(p); g += kThreads / kWave) {
    Moments m{0.0f, 0.0f, 0.0f};
    for (int i = lane; i < entries; i += kWave) {
      const float* from = p.stats + (((a.sample * p.chunks + i / a.k.parts) * p.g + a.group + g) * a.k.parts +
                                     i % a.k.parts) * 3;
      m.join({from[0], from[1], from[2]});
    }
    m.over_wave();
    if (lane == 0) {
      lm[g] = m.mean;
      lr[g] = rsqrtf(m.m2 / m.n + p.eps);
    }
  }
  __syncthreads();
}

template <bool BF, int V>
__global__ __launch_bounds__(kThreads) void map_forward(GnParams p) {
  using P = Piece<BF, V>;
  using E = typename P::E;
  __shared__ float lm[kThreads], lr[kThreads];
  const Place<V> a(p);
  joined_stats<V>(p, a, lm, lr);
  if (!a.any) return;
  Chan<BF, V> ch;
  ch.load(p, a.c, true);
  const int g = a.k.parts == 1 ? a.piece / a.k.pieces : 0;
  const float mean = lm[g], r = lr[g];
  const E* x = static_cast<const E*>(p.x) + a.sample * p.xn + a.c;
  E* out = static_cast<E*>(p.out) + a.sample * p.s * p.c + a.c;
#pragma unroll 4
  for (int64_t t = a.p0 + a.off; t < a.p1; t += a.k.rows) {
    float v[V];
    P::open(P::load(x + t * p.xs), v);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      v[k] = fmaf((v[k] - mean) * r, ch.w[k], ch.bias[k]);
      if (p.silu) v[k] = silu_of(v[k]);
    }
    P::store(out + t * p.c, v);
  }
}

// Each channel's sums of gu n and gu over a chunk, and each group's of gu w n and gu w (behind them, [parts][2]).
template <bool BF, int V>
__global__ __launch_bounds__(kThreads) void map_sums(GnParams p, float* group_sums) {
  using P = Piece<BF, V>;
  using E = typename P::E;
  __shared__ float lm[kThreads], lr[kThreads], l[2][kThreads][V];
  const Place<V> a(p);
  joined_stats<V>(p, a, lm, lr);
  Chan<BF, V> ch;
  ch.load(p, a.c, a.any);
  float gw[V] = {}, gb[V] = {};
  if (a.any) {
    const int g = a.k.parts == 1 ? a.piece / a.k.pieces : 0;
    const float mean = lm[g], r = lr[g];
    const E* x = static_cast<const E*>(p.x) + a.sample * p.xn + a.c;
    const E* go = static_cast<const E*>(p.go) + a.sample * p.gon + a.c;
#pragma unroll 4
    for (int64_t t = a.p0 + a.off; t < a.p1; t += a.k.rows) {
      float v[V], gu[V];
      P::open(P::load(x + t * p.xs), v);
      P::open(P::load(go + t * p.gos), gu);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float n = (v[k] - mean) * r;
        if (p.silu) gu[k] *= silu_slope(fmaf(n, ch.w[k], ch.bias[k]));
        gw[k] = fmaf(gu[k], n, gw[k]);
        gb[k] += gu[k];
      }
    }
  }
#pragma unroll
  for (int k = 0; k < V; ++k) {
    l[0][threadIdx.x][k] = gw[k];
    l[1][threadIdx.x][k] = gb[k];
  }
  __syncthreads();
  const int64_t row = a.sample * p.chunks + a.chunk;
  if (a.any && a.off == 0) {
    for (int i = 1; i < a.k.rows; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) {
        gw[k] += l[0][i * a.k.width + a.piece][k];
        gb[k] += l[1][i * a.k.width + a.piece][k];
      }
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      p.sums[row * 2 * p.c + a.c + k] = gw[k];
      p.sums[(row * 2 + 1) * p.c + a.c + k] = gb[k];
      s1 = fmaf(ch.w[k], gb[k], s1);
      s2 = fmaf(ch.w[k], gw[k], s2);
    }
    lm[a.piece] = s1;
    lr[a.piece] = s2;
  } else if (a.off == 0) {
    lm[a.piece] = 0.0f;
    lr[a.piece] = 0.0f;
  }
  __syncthreads();
  const int lane = int(threadIdx.x) % kWave, per = a.k.parts == 1 ? a.k.pieces : a.k.width;
  for (int g = int(threadIdx.x) / kWave; g < a.groups_here(p); g += kThreads / kWave) {
    float s1 = 0.0f, s2 = 0.0f;
    for (int i = lane; i < per; i += kWave) {
      s1 += lm[g * per + i];
      s2 += lr[g * per + i];
    }
#pragma unroll
    for (int m = 1; m < kWave; m *= 2) {
      s1 += __shfl_xor(s1, m);
      s2 += __shfl_xor(s2, m);
    }
    if (lane == 0) {
      float* to = group_sums + ((row * p.g + a.group + g) * a.k.parts + a.part) * 2;
      to[0] = s1;
      to[1] = s2;
    }
  }
}

template <bool BF, int V>
__global__ __launch_bounds__(kThreads) void map_backward(GnParams p, const float* group_sums) {
  using P = Piece<BF, V>;
  using E = typename P::E;
  __shared__ float lm[kThreads], lr[kThreads], l1[kThreads], l2[kThreads];
  const Place<V> a(p);
  const int lane = int(threadIdx.x) % kWave, entries = p.chunks * a.k.parts;
  const float inv = 1.0f / (float(p.s) * float(p.c / p.g));
  for (int g = int(threadIdx.x) / kWave; g < a.groups_here(p); g += kThreads / kWave) {
    float s1 = 0.0f, s2 = 0.0f;
    for (int i = lane; i < entries; i += kWave) {
      const float* from = group_sums + (((a.sample * p.chunks + i / a.k.parts) * p.g + a.group + g) * a.k.parts +
                                        i % a.k.parts) * 2;
      s1 += from[0];
      s2 += from[1];
    }
#pragma unroll
    for (int m = 1; m < kWave; m *= 2) {
      s1 += __shfl_xor(s1, m);
      s2 += __shfl_xor(s2, m);
    }
    if (lane == 0) {
      l1[g] = s1 * inv;
      l2[g] = s2 * inv;
    }
  }
  joined_stats<V>(p, a, lm, lr);
  if (!a.any) return;
  Chan<BF, V> ch;
  ch.load(p, a.c, true);
  const int g = a.k.parts == 1 ? a.piece / a.k.pieces : 0;
  const float mean = lm[g], r = lr[g], s1 = l1[g], s2 = l2[g];
  const E* x = static_cast<const E*>(p.x) + a.sample * p.xn + a.c;
  const E* go = static_cast<const E*>(p.go) + a.sample * p.gon + a.c;
  E* out = static_cast<E*>(p.out) + a.sample * p.s * p.c + a.c;
#pragma unroll 4
  for (int64_t t = a.p0 + a.off; t < a.p1; t += a.k.rows) {
    float v[V], gu[V];
    P::open(P::load(x + t * p.xs), v);
    P::open(P::load(go + t * p.gos), gu);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const float n = (v[k] - mean) * r;
      if (p.silu) gu[k] *= silu_slope(fmaf(n, ch.w[k], ch.bias[k]));
      v[k] = r * (gu[k] * ch.w[k] - s1 - n * s2);
    }
    P::store(out + t * p.c, v);
  }
}

// ---------------------------------------------------------------- which

// Channels of a piece: 16 bytes where groups are whole pieces, else one.
int piece_channels(const GnParams& p) {
  const int v = p.bf16 ? 8 : 4;
  return p.c / p.g % v == 0 ? v : 1;
}

constexpr int kMostPieces = 4;  // of a lane that holds a row's group

// Lanes that hold a group of a row; 0: too wide, or samples of several positions.
int row_lanes(const GnParams& p) {
  if (p.s != 1) return 0;
  const int pieces = p.c / p.g / piece_channels(p);
  for (int l : {4, 16, 64, 256})
    if (pieces <= 2 * l) return l;
  return pieces <= kMostPieces * 256 ? 256 : 0;
}

// Workgroups in x, and rows each takes at once.
struct RowGrid {
  int rows, x, y;
};
RowGrid row_grid(const GnParams& p, int lanes, bool gradient) {
  const int slots = kThreads / lanes;
  RowGrid r;
  r.rows = p.g >= slots ? 1 : slots / p.g;
  r.y = p.g >= slots ? (p.g + slots - 1) / slots : 1;
  const int64_t want = std::max<int64_t>(1, int64_t(device_cu_count()) * (gradient ? 4 : 8) / r.y);
  r.x = int(std::max<int64_t>(1, std::min(want, (p.n + r.rows - 1) / r.rows)));
  return r;
}

template <bool BF, int V, int L, int M>
void rows_kernel(const GnParams& p, dim3 grid, bool gradient, hipStream_t stream) {
  if (gradient) rows_backward<BF, V, L, M><<<grid, kThreads, 0, stream>>>(p);
  else rows_forward<BF, V, L, M><<<grid, kThreads, 0, stream>>>(p);
}

template <bool BF, int V, int L>
void rows_pieces(const GnParams& p, dim3 grid, bool gradient, hipStream_t stream) {
  const int pieces = p.c / p.g / V;
  if (pieces <= L) rows_kernel<BF, V, L, 1>(p, grid, gradient, stream);
  else if (pieces <= 2 * L) rows_kernel<BF, V, L, 2>(p, grid, gradient, stream);
  else if constexpr (L == 256) rows_kernel<BF, V, L, kMostPieces>(p, grid, gradient, stream);
}

template <bool BF, int V>
hipError_t launch(const GnParams& p, bool gradient, hipStream_t stream) {
  const int lanes = row_lanes(p);
  if (lanes) {
    const RowGrid r = row_grid(p, lanes, gradient);
    const dim3 grid(unsigned(r.x), unsigned(r.y));
    switch (lanes) {
      case 4: rows_pieces<BF, V, 4>(p, grid, gradient, stream); break;
      case 16: rows_pieces<BF, V, 16>(p, grid, gradient, stream); break;
      case 64: rows_pieces<BF, V, 64>(p, grid, gradient, stream); break;
      default: rows_pieces<BF, V, 256>(p, grid, gradient, stream);
    }
    return hipGetLastError();
  }
  const unsigned grid = unsigned(p.n * p.chunks * blocks_of<V>(p).count);
  map_stats<BF, V><<<grid, kThreads, 0, stream>>>(p);
  if (!gradient) {
    map_forward<BF, V><<<grid, kThreads, 0, stream>>>(p);
  } else {
    float* group_sums = p.sums + p.n * p.chunks * 2 * p.c;
    map_sums<BF, V><<<grid, kThreads, 0, stream>>>(p, group_sums);
    map_backward<BF, V><<<grid, kThreads, 0, stream>>>(p, group_sums);
  }
  return hipGetLastError();
}

hipError_t launch_any(const GnParams& p, bool gradient, hipStream_t stream) {
  const bool wide = piece_channels(p) > 1;
  if (p.bf16) return wide ? launch<true, 8>(p, gradient, stream) : launch<true, 1>(p, gradient, stream);
  return wide ? launch<false, 4>(p, gradient, stream) : launch<false, 1>(p, gradient, stream);
}

Blocks blocks_for(const GnParams& p) {
  switch (piece_channels(p)) {
    case 8: return blocks_of<8>(p);
    case 4: return blocks_of<4>(p);
    default: return blocks_of<1>(p);
  }
}

}  // namespace

void group_norm_split(GnParams& p, bool gradient) {
  p.chunks = 1;
  p.chunk = p.s;
  if (row_lanes(p)) {
    const RowGrid r = row_grid(p, row_lanes(p), gradient);
    p.chunks = r.x * r.rows;  // rows of the channels' sums
    return;
  }
  const Blocks k = blocks_for(p);
  // Four workgroups a compute unit, of eight positions a thread at least.
  const int64_t want = std::max<int64_t>(1, int64_t(device_cu_count()) * 4 / std::max<int64_t>(1, p.n * k.count));
  const int64_t chunk = std::max<int64_t>(int64_t(k.rows) * 8, (p.s + want - 1) / want);
  p.chunk = chunk;
  p.chunks = int(std::max<int64_t>(1, (p.s + chunk - 1) / chunk));
}

double group_norm_workgroups(const GnParams& p) {
  return row_lanes(p) ? double(p.chunks) : double(p.n) * double(p.chunks) * blocks_for(p).count;
}

int64_t group_norm_stats_floats(const GnParams& p) {
  return row_lanes(p) ? 0 : p.n * p.chunks * p.g * blocks_for(p).parts * 3;
}

int64_t group_norm_sums_floats(const GnParams& p) {
  if (row_lanes(p)) return int64_t(p.chunks) * 2 * p.c;
  return p.n * p.chunks * (2 * int64_t(p.c) + int64_t(p.g) * blocks_for(p).parts * 2);
}

hipError_t launch_group_norm(const GnParams& p, hipStream_t stream) { return launch_any(p, false, stream); }

hipError_t launch_group_norm_backward(const GnParams& p, hipStream_t stream) {
  const hipError_t err = p.n * p.s > 0 ? launch_any(p, true, stream) : hipSuccess;
  if (err != hipSuccess) return err;
  const int64_t rows = p.n * p.s == 0 ? 0 : row_lanes(p) ? p.chunks : p.n * p.chunks, c = p.c;
  SumRows s{};
  s.count = 2;
  s.s[0] = {p.sums, p.gw, rows, 2 * c, c, 1};
  s.s[1] = {p.sums + c, p.gbias, rows, 2 * c, c, 1};
  return launch_sum_rows(s, stream);
}

}  // namespace sx
