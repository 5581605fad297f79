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
// squared distance from it (joined so that no large mean cancels), the next
// joins the chunks' and normalises; the gradient has one more for its two sums (map_*).
// Bound by memory: 16384 rows of 2048 channels in bf16 take 23 to 25 us (5.5 TB/s), the gradient of
// 8 x 4096 positions of 512 channels 58 to 60 us: three launches, of which the first two read what the third reads again.
#include <algorithm>
#include <cmath>

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
      w[v] = is ? 1.0f : 0.0f;
      bias[v] = 0.0f;
    }
    if (is && p.w) {
#pragma unroll
      for (int v = 0; v < V; ++v) w[v] = p.w[c + v];
    }
    if (is && p.bias) {
#pragma unroll
      for (int v = 0; v < V; ++v) bias[v] = p.bias[c + v];
    }
  }
  // gu = gy silu'(u), of n. One branch for all channels, here and in silu_all: one each forms them one after the
  // other (gradient of 8 x 4096 positions of 512 channels in bf16: 71 us, 59 so).
  __device__ __forceinline__ void pass_silu(const float (&n)[V], float (&gu)[V]) const {
#pragma unroll
    for (int v = 0; v < V; ++v) gu[v] *= silu_slope(fmaf(n[v], w[v], bias[v]));
  }
};

template <int V>
__device__ __forceinline__ void silu_all(float (&u)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) u[v] = silu_of(u[v]);
}

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
      for (int k = 0; k < V; ++k) v[m][k] = fmaf(v[m][k] * r, ch[m].w[k], ch[m].bias[k]);
      if (p.silu) silu_all<V>(v[m]);
      if (is[m] && row < p.n) store_stream<BF, V>(static_cast<E*>(p.out) + row * p.c + c[m], v[m]);
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
    for (int m = 0; m < M; ++m) {
      // a lane without channels or behind the last row adds zeros, also where r is infinite (no eps, no variance)
      const float scale = is[m] && row < p.n ? r : 0.0f;
#pragma unroll
      for (int k = 0; k < V; ++k) v[m][k] *= scale;
      if (p.silu) ch[m].pass_silu(v[m], g[m]);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        gw[m][k] = fmaf(g[m][k], v[m][k], gw[m][k]);
        gb[m][k] += g[m][k];
        g[m][k] *= ch[m].w[k];
        s1 += g[m][k];
        s2 = fmaf(g[m][k], v[m][k], s2);
      }
    }
    s1 = lanes_sum<L>(s1, l[2]) * inv;
    s2 = lanes_sum<L>(s2, l[3]) * inv;
#pragma unroll
    for (int m = 0; m < M; ++m) {
#pragma unroll
      for (int k = 0; k < V; ++k) v[m][k] = r * (g[m][k] - s1 - v[m][k] * s2);
      if (is[m] && row < p.n) store_stream<BF, V>(static_cast<E*>(p.out) + row * p.c + c[m], v[m]);
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

// A thread's positions of x (and of the result's gradient, GO), kAtOnce ahead of what is done with them: the first are
// on their way from the constructor on, which stands before the chunks' values are joined. 10 x 3000 positions of 333
// channels in bf16: 32 us, 41 with four at a time that are waited for.
constexpr int kAtOnce = 4;
template <bool BF, int V, bool GO>
struct Ahead {
  using P = Piece<BF, V>;
  using E = typename P::E;
  const E *x, *go;        // the thread's first position, then the one after each kAtOnce
  int64_t x_step, g_step; // to its next
  int left, rows;         // positions of the chunk from there on (a chunk of 2^31 would not fit the memory)
  typename P::Raw xin[kAtOnce], gin[GO ? kAtOnce : 1];
  __device__ __forceinline__ Ahead(const GnParams& p, const Place<V>& a)
      : x(static_cast<const E*>(p.x) + a.sample * p.xn + (a.p0 + a.off) * p.xs + a.c),
        go(GO ? static_cast<const E*>(p.go) + a.sample * p.gon + (a.p0 + a.off) * p.gos + a.c : nullptr),
        x_step(a.k.rows * p.xs), g_step(a.k.rows * p.gos), left(a.any ? int(a.p1 - a.p0) - a.off : 0), rows(a.k.rows) {
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      xin[i] = P::zero();
      if constexpr (GO) gin[i] = P::zero();
      read(i, 0);
    }
  }
  __device__ __forceinline__ void read(int i, int ahead) {
    if (left <= (i + ahead) * rows) return;
    xin[i] = P::load(x + (i + ahead) * x_step);
    if constexpr (GO) gin[i] = P::load(go + (i + ahead) * g_step);
  }
  // f(how many positions of the thread's before, x, gradient)
  template <typename F>
  __device__ __forceinline__ void each(F&& f) {
    for (int64_t n = 0; left > 0; n += kAtOnce) {
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        if (left <= i * rows) break;
        float v[V], gu[V] = {};
        P::open(xin[i], v);
        if constexpr (GO) P::open(gin[i], gu);
        read(i, kAtOnce);
        f(n + i, v, gu);
      }
      x += kAtOnce * x_step;
      if constexpr (GO) go += kAtOnce * g_step;
      left -= kAtOnce * rows;
    }
  }
};

// Sums of K values a thread over the threads of its group, in every thread: a wave takes a group at a time. `v` are
// zero in threads without a piece. Ends with l free again.
template <int K, int V>
__device__ __forceinline__ void group_sums_of(const GnParams& p, const Place<V>& a, float (*l)[kThreads], float (&v)[K]) {
  const int tid = int(threadIdx.x), lane = tid % kWave, per = a.k.parts == 1 ? a.k.pieces : a.k.width;
#pragma unroll
  for (int k = 0; k < K; ++k) l[k][tid] = v[k];
  __syncthreads();
  for (int g = tid / kWave; g < a.groups_here(p); g += kThreads / kWave) {
    float sum[K] = {};
    for (int i = lane; i < per * a.k.rows; i += kWave) {
      const int at = i / per * a.k.width + g * per + i % per;
#pragma unroll
      for (int k = 0; k < K; ++k) sum[k] += l[k][at];
    }
#pragma unroll
    for (int m = 1; m < kWave; m *= 2)
#pragma unroll
      for (int k = 0; k < K; ++k) sum[k] += __shfl_xor(sum[k], m);
    // the group's own first slot: no other wave reads it
    if (lane == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) l[k][g * per] = sum[k];
    }
  }
  __syncthreads();
  const int g = a.any && a.k.parts == 1 ? a.piece / a.k.pieces : 0;
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = l[k][g * per];
  __syncthreads();
}

struct Moments {  // of n values: their mean and squared distances from it
  float n, mean, m2;
};
struct Norm {
  float mean, r;
};

// 1 / n of a count, to 2^-44 of it: an instruction's 2^-22, refined.
__device__ __forceinline__ double inverse_of(float n) {
  const double r = __builtin_amdgcn_rcpf(n);
  return r * fma(-double(n), r, 2.0);
}

// Squared distance from the mean of n values with these sums. Below zero by rounding it is zero; what is not finite
// stays so: the mean of a group with an infinity is infinite, and only an infinite or lost variance turns all to NaN.
__device__ __forceinline__ float spread_of(float squares, float sum, float n) {
  const float d = fmaf(-sum, sum / n, squares);
  return d < 0.0f ? 0.0f : d;
}
__device__ __forceinline__ double spread_of(double squares, double sum, float n) {
  const double d = fma(-sum, sum * inverse_of(n), squares);
  return d < 0.0 ? 0.0 : d;
}

// The moments of a block's part of a thread's group. A thread sums differences from the mean of its first four
// positions, and the threads differences from the mean of a few of theirs, so that no large mean cancels, and no outlier
// among the first (4096 positions of 16 channels a group, the first position off by 300: 2e-7 of a result's size, 3e-6
// with differences from the very first).
template <bool BF, int V>
__device__ __forceinline__ Moments block_stats(const GnParams& p, const Place<V>& a, float (*l)[kThreads]) {
  using P = Piece<BF, V>;
  Ahead<BF, V, false> in(p, a);
  float shift = 0.0f, sum = 0.0f, sq = 0.0f, n = 0.0f;
  {
    const int count = in.left > 3 * in.rows ? 4 : in.left > in.rows ? 2 : 1;
    const float share = 1.0f / float(count * V);
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      float v[V];
      P::open(in.xin[i], v);
#pragma unroll
      for (int k = 0; k < V; ++k) shift = i < count ? fmaf(v[k], share, shift) : shift;
    }
  }
  in.each([&](int64_t, const float(&v)[V], const float(&)[V]) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const float d = v[k] - shift;
      sum += d;
      sq = fmaf(d, d, sq);
    }
    n += float(V);
  });
  const float mean = n > 0.0f ? shift + sum / n : 0.0f, m2 = n > 0.0f ? spread_of(sq, sum, n) : 0.0f;
  l[0][threadIdx.x] = mean;
  __syncthreads();
  const int g = a.any && a.k.parts == 1 ? a.piece / a.k.pieces : 0;
  float about = 0.0f;
  {
    const int per = a.k.parts == 1 ? a.k.pieces : a.k.width;
    const int here = a.k.parts == 1 ? a.k.pieces : min(kThreads, a.k.pieces - a.part * kThreads);
    // rows of threads that have positions; else pieces of the first, far from each other
    const bool rows = a.k.rows >= 4 && a.p1 - a.p0 >= 4;
    const int bits = rows ? 2 : here >= 8 ? 3 : here >= 4 ? 2 : here >= 2 ? 1 : 0;
    const int step = rows ? a.k.width : here >> bits;
    const float share = ldexpf(1.0f, -bits);  // of each first: their sum may pass the range
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // (all on their way at once)
      const bool is = i < 1 << bits;
      about = fmaf(l[0][g * per + (is ? i * step : 0)], is ? share : 0.0f, about);
    }
  }
  __syncthreads();
  const float off = mean - about;
  float v[3] = {n, n * off, n > 0.0f ? fmaf(n * off, off, m2) : 0.0f};
  group_sums_of<3>(p, a, l, v);
  return {v[0], about + v[1] / v[0], spread_of(v[2], v[1], v[0])};
}

// The first thread of each of the block's groups.
template <int V>
__device__ __forceinline__ bool first_of_group(const Place<V>& a) {
  return a.any && a.off == 0 && (a.k.parts == 1 ? a.piece % a.k.pieces == 0 : a.piece == 0);
}

// Where the values of a thread's group and a chunk are, of an array [samples][chunks][groups][parts].
template <int V>
__device__ __forceinline__ int64_t own_entry(const GnParams& p, const Place<V>& a) {
  const int g = a.k.parts == 1 ? a.piece / a.k.pieces : 0;
  return ((a.sample * p.chunks + a.chunk) * p.g + a.group + g) * a.k.parts + a.part;
}

template <bool BF, int V>
__global__ __launch_bounds__(kThreads) void map_stats(GnParams p) {
  __shared__ float l[3][kThreads];
  const Place<V> a(p);
  const Moments m = block_stats<BF, V>(p, a, l);
  if (first_of_group(a)) {
    float* to = p.stats + own_entry(p, a) * 3;
    to[0] = m.n;
    to[1] = m.mean;
    to[2] = m.m2;
  }
}

// Sums of K values over a block's groups' entries (chunks, and parts of wide groups), into l[..][group]: thread t has
// group t % groups and every (threads / groups)-th entry, value(group, entry, v).
template <int K, typename T, int V, typename F>
__device__ __forceinline__ void entry_sums(const GnParams& p, const Place<V>& a, T (*l)[kThreads], F&& value) {
  const int groups = a.groups_here(p), slots = kThreads / groups, entries = p.chunks * a.k.parts;
  const int tid = int(threadIdx.x), g = tid % groups, slot = tid / groups;
  T sum[K] = {};
  if (slot < slots) {
#pragma unroll 4
    for (int i = slot; i < entries; i += slots) {
      T v[K];
      value(g, i, v);
#pragma unroll
      for (int k = 0; k < K; ++k) sum[k] += v[k];
    }
  }
#pragma unroll
  for (int k = 0; k < K; ++k) l[k][tid] = sum[k];
  __syncthreads();
  for (int have = slots; have > 1;) {
    const int half = (have + 1) / 2;
    if (slot < have - half) {
#pragma unroll
      for (int k = 0; k < K; ++k) l[k][tid] += l[k][tid + half * groups];
    }
    have = half;
    __syncthreads();
  }
}

// Where the values of a block's group and entry are, of an array [samples][chunks][groups][parts].
template <int V>
__device__ __forceinline__ int64_t entry_at(const GnParams& p, const Place<V>& a, int g, int i) {
  return ((a.sample * p.chunks + i / a.k.parts) * p.g + a.group + g) * a.k.parts + i % a.k.parts;
}

// Mean and 1 / sqrt(variance + eps) of a thread's group, from all chunks: sums about the first entry's mean, in 64 bits,
// which a first chunk far from the others needs (of 200000 positions, off by 300: 1e-7 of a result's size, 1.5e-5 in 32).
template <int V>
__device__ __forceinline__ Norm joined_stats(const GnParams& p, const Place<V>& a, double (*l)[kThreads]) {
  const auto first = [&](int g) { return p.stats[entry_at(p, a, g, 0) * 3 + 1]; };
  entry_sums<3>(p, a, l, [&](int g, int i, double (&v)[3]) {
    const float* from = p.stats + entry_at(p, a, g, i) * 3;
    const double off = double(from[1]) - double(first(g));
    v[0] = from[0];
    v[1] = v[0] * off;
    v[2] = fma(v[1], off, double(from[2]));
  });
  const int g = a.any && a.k.parts == 1 ? a.piece / a.k.pieces : 0;
  const float count = float(l[0][g]);
  const Norm n{float(double(first(g)) + l[1][g] * inverse_of(count)),
               rsqrtf(float(spread_of(l[2][g], l[1][g], count)) / count + p.eps)};
  __syncthreads();
  return n;
}

template <bool BF, int V>
__device__ __forceinline__ void normalise(const GnParams& p, const Place<V>& a, Ahead<BF, V, false>& in, const Norm& n) {
  using E = typename Piece<BF, V>::E;
  Chan<BF, V> ch;
  ch.load(p, a.c, a.any);
  E* out = static_cast<E*>(p.out) + (a.sample * p.s + a.p0 + a.off) * p.c + a.c;
  const int64_t step = int64_t(a.k.rows) * p.c;
  in.each([&](int64_t t, float(&v)[V], const float(&)[V]) {
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] = fmaf((v[k] - n.mean) * n.r, ch.w[k], ch.bias[k]);
    if (p.silu) silu_all<V>(v);
    store_stream<BF, V>(out + t * step, v);
  });
}

// Each channel's sums of gu n and gu over a chunk, into p.sums; and those of gu w n (s2) and gu w (s1) of a thread's
// group over it.
template <bool BF, int V>
__device__ __forceinline__ void block_sums(const GnParams& p, const Place<V>& a, Ahead<BF, V, true>& in, const Norm& n,
                                           float (*l)[kThreads], float (*share)[kThreads][V], float* s1, float* s2) {
  Chan<BF, V> ch;
  ch.load(p, a.c, a.any);
  float gw[V] = {}, gb[V] = {};
  in.each([&](int64_t, float(&v)[V], float(&gu)[V]) {
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] = (v[k] - n.mean) * n.r;
    if (p.silu) ch.pass_silu(v, gu);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      gw[k] = fmaf(gu[k], v[k], gw[k]);
      gb[k] += gu[k];
    }
  });
  float v[2] = {0.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < V; ++k) {
    share[0][threadIdx.x][k] = gw[k];
    share[1][threadIdx.x][k] = gb[k];
    v[0] = fmaf(ch.w[k], gb[k], v[0]);
    v[1] = fmaf(ch.w[k], gw[k], v[1]);
  }
  group_sums_of<2>(p, a, l, v);
  *s1 = v[0];
  *s2 = v[1];
  if (a.any && a.off == 0) {
    for (int i = 1; i < a.k.rows; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) {
        gw[k] += share[0][i * a.k.width + a.piece][k];
        gb[k] += share[1][i * a.k.width + a.piece][k];
      }
    float* to = p.sums + (a.sample * p.chunks + a.chunk) * 2 * p.c + a.c;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      to[k] = gw[k];
      to[p.c + k] = gb[k];
    }
  }
}

template <bool BF, int V>
__device__ __forceinline__ void pass_back(const GnParams& p, const Place<V>& a, Ahead<BF, V, true>& in, const Norm& n,
                                          float s1, float s2) {
  using E = typename Piece<BF, V>::E;
  const float inv = 1.0f / (float(p.s) * float(p.c / p.g));
  s1 *= inv;
  s2 *= inv;
  Chan<BF, V> ch;
  ch.load(p, a.c, a.any);
  E* out = static_cast<E*>(p.out) + (a.sample * p.s + a.p0 + a.off) * p.c + a.c;
  const int64_t step = int64_t(a.k.rows) * p.c;
  in.each([&](int64_t t, float(&v)[V], float(&gu)[V]) {
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] = (v[k] - n.mean) * n.r;
    if (p.silu) ch.pass_silu(v, gu);
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] = n.r * (gu[k] * ch.w[k] - s1 - v[k] * s2);
    store_stream<BF, V>(out + t * step, v);
  });
}

template <bool BF, int V>
__global__ __launch_bounds__(kThreads) void map_forward(GnParams p) {
  __shared__ double l[3][kThreads];
  const Place<V> a(p);
  Ahead<BF, V, false> in(p, a);
  normalise<BF, V>(p, a, in, joined_stats<V>(p, a, l));
}

template <bool BF, int V>
__global__ __launch_bounds__(kThreads) void map_sums(GnParams p, float* group_sums) {
  __shared__ double joined[3][kThreads];
  __shared__ float l[2][kThreads], share[2][kThreads][V];
  const Place<V> a(p);
  Ahead<BF, V, true> in(p, a);
  const Norm n = joined_stats<V>(p, a, joined);
  float s1, s2;
  block_sums<BF, V>(p, a, in, n, l, share, &s1, &s2);
  if (first_of_group(a)) {
    float* to = group_sums + own_entry(p, a) * 2;
    to[0] = s1;
    to[1] = s2;
  }
}

template <bool BF, int V>
__global__ __launch_bounds__(kThreads) void map_backward(GnParams p, const float* group_sums) {
  __shared__ double joined[3][kThreads];
  __shared__ float l[2][kThreads];
  const Place<V> a(p);
  Ahead<BF, V, true> in(p, a);
  entry_sums<2>(p, a, l, [&](int g, int i, float (&v)[2]) {
    const float* from = group_sums + entry_at(p, a, g, i) * 2;
    v[0] = from[0];
    v[1] = from[1];
  });
  const int g = a.any && a.k.parts == 1 ? a.piece / a.k.pieces : 0;
  const float s1 = l[0][g], s2 = l[1][g];
  __syncthreads();
  pass_back<BF, V>(p, a, in, joined_stats<V>(p, a, joined), s1, s2);
}

// A block that has its groups whole (one chunk, no wide groups) does all of it in one launch: 4 positions of 256
// channels take 7.4 us, 11.4 in two.
template <bool BF, int V>
__global__ __launch_bounds__(kThreads) void map_alone(GnParams p, int gradient) {
  __shared__ float l[3][kThreads], share[2][kThreads][V];
  const Place<V> a(p);
  const Moments m = block_stats<BF, V>(p, a, l);
  const Norm n{m.mean, rsqrtf(m.m2 / m.n + p.eps)};
  if (!gradient) {
    Ahead<BF, V, false> in(p, a);
    normalise<BF, V>(p, a, in, n);
    return;
  }
  float s1, s2;
  {
    Ahead<BF, V, true> in(p, a);
    block_sums<BF, V>(p, a, in, n, l, share, &s1, &s2);
  }
  Ahead<BF, V, true> in(p, a);
  pass_back<BF, V>(p, a, in, n, s1, s2);
}

// ---------------------------------------------------------------- which

// Channels of a piece: up to 16 bytes, as many as groups are whole pieces of.
int piece_channels(const GnParams& p) {
  const int per = p.c / p.g;
  return p.bf16 && per % 8 == 0 ? 8 : per % 4 == 0 ? 4 : per % 2 == 0 ? 2 : 1;
}

constexpr int kMostPieces = 4;  // of a lane that holds a row's group
constexpr int kMapPerCu = 2, kMostEntries = 4096;

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
  // 16384 rows of 2048 channels in bf16: 29.5, 27.6, 25.4, 25.0 us with 3, 4, 6, 8 workgroups a compute unit; the
  // gradient of 16000 rows of 1024: 49.4, 39.1, 39.5, 42.9 with 1, 2, 3, 4, of 2000 rows of 370 in f32 21.3, 14.5,
  // 13.6, 13.4
  const int64_t want = std::max<int64_t>(1, int64_t(device_cu_count()) * (gradient ? 3 : 8) / r.y);
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
  if (p.chunks == 1 && blocks_of<V>(p).parts == 1) {
    map_alone<BF, V><<<grid, kThreads, 0, stream>>>(p, gradient ? 1 : 0);
    return hipGetLastError();
  }
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

template <bool BF>
hipError_t launch_any(const GnParams& p, bool gradient, hipStream_t stream) {
  switch (piece_channels(p)) {
    case 8:
      if constexpr (BF) return launch<BF, 8>(p, gradient, stream);
      return hipErrorInvalidValue;  // f32 pieces have four channels
    case 4: return launch<BF, 4>(p, gradient, stream);
    case 2: return launch<BF, 2>(p, gradient, stream);
    default: return launch<BF, 1>(p, gradient, stream);
  }
}

hipError_t launch_any(const GnParams& p, bool gradient, hipStream_t stream) {
  return p.bf16 ? launch_any<true>(p, gradient, stream) : launch_any<false>(p, gradient, stream);
}

Blocks blocks_for(const GnParams& p) {
  switch (piece_channels(p)) {
    case 8: return blocks_of<8>(p);
    case 4: return blocks_of<4>(p);
    case 2: return blocks_of<2>(p);
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
  const int bytes = piece_channels(p) * (p.bf16 ? 2 : 4), per_cu = std::min(8, kMapPerCu * 16 / bytes);
  // Two workgroups a compute unit (more where a piece is narrow: 10 x 3000 positions of 333 channels in bf16 take 32 us
  // with eight, 43 with two; the gradient of 8 x 4096 of 512 59, 59, 65, 72 with 1, 2, 3, 4), of eight positions a
  // thread at least, and as few chunks as a workgroup joins by the way (every workgroup joins those of its sample).
  const int64_t want = std::max<int64_t>(1, int64_t(device_cu_count()) * per_cu / std::max<int64_t>(1, p.n * k.count));
  const int64_t most = std::max<int64_t>(1, kMostEntries / (int64_t(k.groups) * k.parts));
  const int64_t split = std::min(want, most);
  const int64_t chunk = std::max<int64_t>(int64_t(k.rows) * 8, (p.s + split - 1) / split);
  p.chunk = chunk;
  p.chunks = int(std::max<int64_t>(1, (p.s + chunk - 1) / chunk));
}

double group_norm_workgroups(const GnParams& p, bool gradient) {
  if (!row_lanes(p)) return double(p.n) * double(p.chunks) * blocks_for(p).count;
  const RowGrid r = row_grid(p, row_lanes(p), gradient);
  return r.y > 65535 ? HUGE_VAL : double(r.x) * r.y;  // a grid has no more rows of workgroups
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
