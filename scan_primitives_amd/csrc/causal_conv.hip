// causal_conv.hip: a short causal convolution along the tokens, a channel at a
// time, with an optional SiLU; its gradient and its single-token form.
//
//   u[t] = bias + sum over j < K of w[j] x[t - (K - 1) + j],   y = u or u sigmoid(u)
//   gu = gy, or gy times the slope of SiLU at u
//   gx[s] = sum over j of w[j] gu[s + (K - 1) - j],  gw[j] = sum over t of gu[t] x[t - (K - 1) + j],  gb = sum of gu
//
// Channels lie last, so a lane takes V of them next to each other (16 bytes, or
// one element where rows are narrower or strided) and marches over a run of tokens with the
// last K - 1 inputs in registers; the run's first K - 1 are read again from the run before
// (from `initial` at the start). The last piece of a row starts early enough to
// be whole: the channels it shares with the piece before get the same values from both.
// Bound by memory: 8 ragged rows of 2048 tokens of 4096 channels in bf16 take 45.5 us; their bytes at a copy's rate
// would take 41.
#include <algorithm>
#include <cmath>

#include "sx_state_space.hpp"

namespace sx {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;  // tokens read ahead

template <bool BF, int V, int K>
struct Conv {
  using P = Piece<BF, V>;
  using E = typename P::E;
  using Raw = typename P::Raw;
  static constexpr int kPast = K > 1 ? K - 1 : 1;
  float w[K][V], bias[V];

  __device__ __forceinline__ Conv(const float* wp, const float* bp, int d0) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int j = 0; j < K; ++j) w[j][v] = wp[int64_t(d0 + v) * K + j];
      bias[v] = 0.0f;
    }
    if (bp) {
#pragma unroll
      for (int v = 0; v < V; ++v) bias[v] = bp[d0 + v];
    }
  }
  // u from the inputs before and the present one
  __device__ __forceinline__ void apply(const float (&past)[kPast][V], const float (&x)[V], float (&u)[V]) const {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      u[v] = bias[v];
#pragma unroll
      for (int j = 0; j < K - 1; ++j) u[v] = fmaf(w[j][v], past[j][v], u[v]);
      u[v] = fmaf(w[K - 1][v], x[v], u[v]);
    }
  }
  static __device__ __forceinline__ void shift(float (&past)[kPast][V], const float (&x)[V]) {
    if constexpr (K > 1) {
#pragma unroll
      for (int j = 0; j + 1 < K - 1; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) past[j][v] = past[j + 1][v];
#pragma unroll
      for (int v = 0; v < V; ++v) past[K - 2][v] = x[v];
    }
  }
};

// One thread's run of tokens and channels.
struct Run {
  int b, chunk, d0, n, t0, t1;
  bool any;
};
template <int V>
__device__ __forceinline__ Run run_of(const CcParams& p) {
  const uint32_t pieces = uint32_t((p.D + V - 1) / V);
  const int64_t idx = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t q = idx / pieces;
  Run r;
  r.any = q < int64_t(p.B) * p.chunks;
  r.b = int(q / p.chunks);
  r.chunk = int(q % p.chunks);
  r.d0 = min(int(idx % pieces) * V, p.D - V);
  r.n = r.any ? row_length(p.lengths, r.b, p.T) : 0;
  r.t0 = r.chunk * p.chunk;
  r.t1 = min(r.t0 + p.chunk, p.T);
  return r;
}

// The input at a position of row b that exists, the ones before the first from `initial`.
template <bool BF, int V>
__device__ __forceinline__ typename Piece<BF, V>::Raw input_at(const CcParams& p, const Run& r, int t) {
  using P = Piece<BF, V>;
  using E = typename P::E;
  if (t >= 0)
    return P::load(static_cast<const E*>(p.x.p) + int64_t(r.b) * p.x.sb + int64_t(t) * p.x.st + int64_t(r.d0) * p.x.sd);
  if (!p.initial) return P::zero();
  return P::load(static_cast<const E*>(p.initial) + (int64_t(r.b) * (p.K - 1) + (t + p.K - 1)) * p.D + r.d0);
}

template <bool BF, int V, int K>
__device__ __forceinline__ void read_past(const CcParams& p, const Run& r,
                                          float (&past)[Conv<BF, V, K>::kPast][V]) {
#pragma unroll
  for (int j = 0; j < K - 1; ++j) {
    const int t = r.t0 - (K - 1) + j;
    Piece<BF, V>::open(t < r.n ? input_at<BF, V>(p, r, t) : Piece<BF, V>::zero(), past[j]);
  }
}

template <bool BF, int V, int K>
__global__ __launch_bounds__(kThreads) void conv_forward(CcParams p) {
  using C = Conv<BF, V, K>;
  using P = typename C::P;
  using E = typename C::E;
  const Run r = run_of<V>(p);
  if (!r.any) return;
  const int end = min(r.t1, r.n);  // tokens there are
  const E* x = static_cast<const E*>(p.x.p) + int64_t(r.b) * p.x.sb + int64_t(r.d0) * p.x.sd;
  E* out = static_cast<E*>(p.out) + int64_t(r.b) * p.T * p.D + r.d0;
  typename P::Raw raw[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) raw[i] = r.t0 + i < end ? P::load(x + int64_t(r.t0 + i) * p.x.st) : P::zero();
  const C c(p.w, p.bias, r.d0);
  float past[C::kPast][V];
  read_past<BF, V, K>(p, r, past);
  for (int t = r.t0; t < end; t += kAhead) {
    float v[kAhead][V];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) P::open(raw[i], v[i]);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int at = t + kAhead + i;
      raw[i] = at < end ? P::load(x + int64_t(at) * p.x.st) : P::zero();
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      float u[V];
      c.apply(past, v[i], u);
      if (p.silu) {
#pragma unroll
        for (int k = 0; k < V; ++k) u[k] = silu_of(u[k]);
      }
      if (t + i < end) store_stream<BF, V>(out + int64_t(t + i) * p.D, u);
      C::shift(past, v[i]);
    }
  }
  for (int t = max(end, r.t0); t < r.t1; ++t) P::put(out + int64_t(t) * p.D, P::zero());
  if (r.chunk == 0 && p.last) {
    E* last = static_cast<E*>(p.last) + int64_t(r.b) * (K - 1) * p.D + r.d0;
#pragma unroll
    for (int j = 0; j < K - 1; ++j) P::put(last + int64_t(j) * p.D, input_at<BF, V>(p, r, r.n - (K - 1) + j));
  }
}

// The march goes K - 1 tokens past the run, whose gu the run's last inputs need; those tokens' own shares of
// gw and gb are the next run's.
template <bool BF, int V, int K>
__global__ __launch_bounds__(kThreads) void conv_backward(CcParams p) {
  using C = Conv<BF, V, K>;
  using P = typename C::P;
  using E = typename C::E;
  const Run r = run_of<V>(p);
  if (!r.any) return;
  const C c(p.w, p.bias, r.d0);
  float past[C::kPast][V], gpast[C::kPast][V] = {}, gw[K][V] = {}, gb[V] = {};
  read_past<BF, V, K>(p, r, past);
  const E* x = static_cast<const E*>(p.x.p) + int64_t(r.b) * p.x.sb + int64_t(r.d0) * p.x.sd;
  const E* g = static_cast<const E*>(p.go.p) + int64_t(r.b) * p.go.sb + int64_t(r.d0) * p.go.sd;
  E* gx = static_cast<E*>(p.out) + int64_t(r.b) * p.T * p.D + r.d0;
  const E* gs = static_cast<const E*>(p.grad_state);
  if (gs) gs += int64_t(r.b) * (K - 1) * p.D + r.d0;
  E* gi = p.last ? static_cast<E*>(p.last) + int64_t(r.b) * (K - 1) * p.D + r.d0 : nullptr;
  const int stop = r.t1 + K - 1;
  typename P::Raw xr[kAhead], gr[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    const int at = r.t0 + i;
    const bool is = at < min(stop, r.n);
    xr[i] = is ? P::load(x + int64_t(at) * p.x.st) : P::zero();
    gr[i] = is ? P::load(g + int64_t(at) * p.go.st) : P::zero();
  }
  for (int t = r.t0; t < stop; t += kAhead) {
    float xv[kAhead][V], gv[kAhead][V];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      P::open(xr[i], xv[i]);
      P::open(gr[i], gv[i]);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int at = t + kAhead + i;
      const bool is = at < min(stop, r.n);
      xr[i] = is ? P::load(x + int64_t(at) * p.x.st) : P::zero();
      gr[i] = is ? P::load(g + int64_t(at) * p.go.st) : P::zero();
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int at = t + i, s = at - (K - 1);
      float gu[V];
#pragma unroll
      for (int v = 0; v < V; ++v) gu[v] = gv[i][v];
      if (p.silu) {
        float u[V];
        c.apply(past, xv[i], u);
        // behind the row's end gy is zero, and the inputs before it may be anything
#pragma unroll
        for (int v = 0; v < V; ++v) gu[v] = at < r.n ? gu[v] * silu_slope(u[v]) : 0.0f;
      }
      if (at < min(r.t1, r.n)) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
          for (int j = 0; j < K - 1; ++j) gw[j][v] = fmaf(gu[v], past[j][v], gw[j][v]);
          gw[K - 1][v] = fmaf(gu[v], xv[i][v], gw[K - 1][v]);
          gb[v] += gu[v];
        }
      }
      float o[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        o[v] = c.w[0][v] * gu[v];
        // gu of s + (K - 1) - j, j taps on: gpast holds those of the K - 1 tokens before `at`
#pragma unroll
        for (int j = 1; j < K; ++j) o[v] = fmaf(c.w[j][v], gpast[K - 1 - j][v], o[v]);
      }
      if (at < stop && (s >= r.t0 || (r.chunk == 0 && s < 0))) {
        // the last K - 1 inputs are the last state
        const int j = s - (r.n - (K - 1));
        if (gs && j >= 0 && j < K - 1) {
          float e[V];
          P::open(P::load(gs + int64_t(j) * p.D), e);
#pragma unroll
          for (int v = 0; v < V; ++v) o[v] += e[v];
        }
        if (s >= r.n && s >= 0) P::put(gx + int64_t(s) * p.D, P::zero());
        else if (s >= 0) P::store(gx + int64_t(s) * p.D, o);
        else if (gi) P::store(gi + int64_t(s + K - 1) * p.D, o);
      }
      C::shift(past, xv[i]);
      C::shift(gpast, gu);
    }
  }
  float* part = p.partial + (int64_t(r.b) * p.chunks + r.chunk) * (K + 1) * p.D + r.d0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int j = 0; j < K; ++j) part[int64_t(j) * p.D + v] = gw[j][v];
    part[int64_t(K) * p.D + v] = gb[v];
  }
}

// One token of each row. Pieces never share a channel here: the state is read and written in place.
template <bool BF, int V, int K>
__global__ __launch_bounds__(kThreads) void conv_step(CcStep p) {
  using C = Conv<BF, V, K>;
  using P = typename C::P;
  using E = typename C::E;
  const uint32_t pieces = uint32_t(p.D / V);
  const int64_t idx = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t b = idx / pieces;
  if (b >= p.B) return;
  const int d0 = int(idx % pieces) * V;
  E* out = static_cast<E*>(p.out) + b * p.D + d0;
  const int64_t slot = p.slots ? p.slots[b] : b;
  if (slot < 0 || slot >= p.pool) {
    P::put(out, P::zero());
    return;
  }
  E* state = static_cast<E*>(p.state) + slot * p.ss + d0;
  typename P::Raw raw[C::kPast];
#pragma unroll
  for (int j = 0; j < K - 1; ++j) raw[j] = P::load(state + int64_t(j) * p.D);
  const auto now = P::load(static_cast<const E*>(p.x) + b * p.sb + int64_t(d0) * p.sd);
  const C c(p.w, p.bias, d0);
  float past[C::kPast][V], x[V], u[V];
#pragma unroll
  for (int j = 0; j < K - 1; ++j) P::open(raw[j], past[j]);
  P::open(now, x);
  c.apply(past, x, u);
  if (p.silu) {
#pragma unroll
    for (int v = 0; v < V; ++v) u[v] = silu_of(u[v]);
  }
  P::store(out, u);
  if constexpr (K > 1) {
#pragma unroll
    for (int j = 0; j + 1 < K - 1; ++j) P::put(state + int64_t(j) * p.D, raw[j + 1]);
    P::put(state + int64_t(K - 2) * p.D, now);
  }
}

constexpr int kForward = 0, kBackward = 1;

int64_t run_threads(const CcParams& p, int v) { return int64_t((p.D + v - 1) / v) * p.chunks * p.B; }

template <bool BF, int V, int K>
hipError_t launch_run(const CcParams& p, int which, hipStream_t stream) {
  const int64_t threads = run_threads(p, V);
  const unsigned grid = unsigned((threads + kThreads - 1) / kThreads);
  if (which == kForward) conv_forward<BF, V, K><<<grid, kThreads, 0, stream>>>(p);
  else conv_backward<BF, V, K><<<grid, kThreads, 0, stream>>>(p);
  return hipGetLastError();
}

template <bool BF, int V>
hipError_t launch_taps(const CcParams& p, int which, hipStream_t stream) {
  switch (p.K) {
    case 1: return launch_run<BF, V, 1>(p, which, stream);
    case 2: return launch_run<BF, V, 2>(p, which, stream);
    case 3: return launch_run<BF, V, 3>(p, which, stream);
    case 4: return launch_run<BF, V, 4>(p, which, stream);
    case 5: return launch_run<BF, V, 5>(p, which, stream);
    case 6: return launch_run<BF, V, 6>(p, which, stream);
    case 7: return launch_run<BF, V, 7>(p, which, stream);
    default: return launch_run<BF, V, 8>(p, which, stream);
  }
}

template <bool BF, int V, int K>
hipError_t step_run(const CcStep& p, hipStream_t stream) {
  const int64_t threads = int64_t(p.D / V) * p.B;
  conv_step<BF, V, K><<<unsigned((threads + kThreads - 1) / kThreads), kThreads, 0, stream>>>(p);
  return hipGetLastError();
}

template <bool BF, int V>
hipError_t step_taps(const CcStep& p, hipStream_t stream) {
  switch (p.K) {
    case 1: return step_run<BF, V, 1>(p, stream);
    case 2: return step_run<BF, V, 2>(p, stream);
    case 3: return step_run<BF, V, 3>(p, stream);
    case 4: return step_run<BF, V, 4>(p, stream);
    case 5: return step_run<BF, V, 5>(p, stream);
    case 6: return step_run<BF, V, 6>(p, stream);
    case 7: return step_run<BF, V, 7>(p, stream);
    default: return step_run<BF, V, 8>(p, stream);
  }
}

// Channels a lane takes: 16 bytes of them (the gradient holds three values a tap and channel, and takes four of
// either type).
int piece_channels(const CcParams& p, bool gradient) {
  const int v = p.bf16 && !gradient ? 8 : 4;
  const bool unit = p.x.sd == 1 && (!gradient || p.go.sd == 1);
  return unit && p.D >= v ? v : 1;
}
int step_channels(const CcStep& p) {
  const int v = p.bf16 ? 8 : 4;
  return p.sd == 1 && p.D % v == 0 ? v : 1;
}
double workgroups(double threads) { return std::ceil(threads / kThreads); }

}  // namespace

double causal_conv_workgroups(const CcParams& p, bool gradient) {
  return workgroups(double(run_threads(p, piece_channels(p, gradient))));
}
double causal_conv_step_workgroups(const CcStep& p) { return workgroups(double(p.D / step_channels(p)) * p.B); }

void causal_conv_split(CcParams& p, bool gradient) {
  // whatever the strides, for the workspace goes by it
  const int64_t v = p.bf16 && !gradient ? 8 : 4, pieces = (p.D + v - 1) / v;
  // Two waves a SIMD (8 ragged rows of 2048 tokens of 4096 channels in bf16: 48, 47, 46, 49 us with 4, 3, 2, 1; the
  // gradient of 4 x 2048 x 2048 42, 36, 35, 47), of 8 tokens at least, 16 of a gradient, whose first
  // and last are read twice.
  const int64_t want = std::max<int64_t>(1, int64_t(device_cu_count()) * 4 * 2 * kWave / std::max<int64_t>(1, pieces * p.B));
  const int64_t chunk = std::max<int64_t>(gradient ? 16 : 8, (p.T + want - 1) / want);
  p.chunk = int(std::min<int64_t>((chunk + kAhead - 1) / kAhead * kAhead, 1 << 20));
  p.chunks = int(std::max<int64_t>(1, (int64_t(p.T) + p.chunk - 1) / p.chunk));
}

hipError_t launch_causal_conv(const CcParams& p, hipStream_t stream) {
  const int v = piece_channels(p, false);
  if (p.bf16) return v == 1 ? launch_taps<true, 1>(p, kForward, stream) : launch_taps<true, 8>(p, kForward, stream);
  return v == 1 ? launch_taps<false, 1>(p, kForward, stream) : launch_taps<false, 4>(p, kForward, stream);
}

hipError_t launch_causal_conv_backward(const CcParams& p, hipStream_t stream) {
  const int v = piece_channels(p, true);
  hipError_t err = hipSuccess;
  if (p.B > 0 && p.bf16) err = v == 1 ? launch_taps<true, 1>(p, kBackward, stream) : launch_taps<true, 4>(p, kBackward, stream);
  else if (p.B > 0) err = v == 1 ? launch_taps<false, 1>(p, kBackward, stream) : launch_taps<false, 4>(p, kBackward, stream);
  if (err != hipSuccess) return err;
  SumRows s{};
  const int64_t rows = int64_t(p.B) * p.chunks, D = p.D;
  s.count = 2;
  s.s[0] = {p.partial, p.gw, rows, (p.K + 1) * D, p.K * D, p.K};
  s.s[1] = {p.partial + p.K * D, p.gbias, rows, (p.K + 1) * D, D, 1};
  return launch_sum_rows(s, stream);
}

hipError_t launch_causal_conv_step(const CcStep& p, hipStream_t stream) {
  const int v = step_channels(p);
  if (p.bf16) return v == 1 ? step_taps<true, 1>(p, stream) : step_taps<true, 8>(p, stream);
  return v == 1 ? step_taps<false, 1>(p, stream) : step_taps<false, 4>(p, stream);
}

}  // namespace sx
