// selective_scan.hip: the scan of a selective state space, over prompts and for
// single tokens.
//
//   dt = softplus(delta + delta_bias),  h[t] = exp(dt a) h[t-1] + dt x[t] b[t]
//   y[t] = c[t] . h[t] + skip x[t],     out = y silu(z)
//
// with N states h a channel, a rate a for each, and rows b[t], c[t] of N that
// the channels of a group share. Channels lie last: a lane is a channel, a wave
// holds four states of 64 channels, and a workgroup's waves share the states of
// those channels, so that few channels already fill the device.
//
// A workgroup goes through tiles of 16 tokens. All its threads turn the tile's x and
// delta into dt and dt x (LDS), four channels of a token each; each wave then
// marches its states over the tile, leaving its part of y in LDS; and the threads that
// read x and z sum the parts, gate and store. One barrier a tile: the next
// tile's dt are formed before it, its loads are on their way since the tile before.
// b and c are operands of no cost: lane j of each row of 16 lanes holds token j's
// values, and an instruction reads them from there (DPP row_newbcast).
//
// Long sequences of few channels are split into segments. A first pass marches each from
// zero, its state and sum of dt kept; the second starts segment m from the ones before it:
// h <- exp(a sum of dt) h + state.
#include <algorithm>

#include "scan_march.hpp"

namespace sx {
namespace {

constexpr int kTile = 16, kChannels = 64;
constexpr int kPieces = kTile * kChannels / 4;  // of a tile, four channels each

template <int W>
struct Lds {
  float dt[2][kTile][kChannels];
  float dx[2][kTile][kChannels];
  float y[2][W][kTile][kChannels];
};

template <bool BF, int W, bool WIDE, bool OUT>
__global__ __launch_bounds__(kWave* W) void scan_march(SsParams p) {
  using P = Piece<BF, 4>;
  using Raw = typename P::Raw;
  constexpr int kPasses = (kPieces + kWave * W - 1) / (kWave * W);
  __shared__ Lds<W> l;
  const int tid = int(threadIdx.x), lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int n0 = wave * kScanStates;
  // where the workgroup is
  const int per_group = p.D / p.G, blocks = (per_group + kChannels - 1) / kChannels;
  uint32_t at = blockIdx.x;
  const int cb = int(at % uint32_t(blocks));
  at /= uint32_t(blocks);
  const int g = int(at % uint32_t(p.G));
  at /= uint32_t(p.G);
  const int b = int(at % uint32_t(p.B)), seg = int(at / uint32_t(p.B));
  const int d0 = g * per_group + cb * kChannels, channels = min(kChannels, per_group - cb * kChannels);
  const int s0 = seg * p.seg_tokens, s1 = min(s0 + p.seg_tokens, p.T);
  const int end = min(s1, row_length(p.lengths, b, p.T));  // tokens there are
  const int tiles = end > s0 ? (end - s0 + kTile - 1) / kTile : 0;

  // this thread's pieces of a tile: token q0 + pass * step, channels c4 .. c4 + 3
  const int q0 = tid / (kChannels / 4), c4 = tid % (kChannels / 4) * 4, left = channels - c4;
  constexpr int kStep = W * kWave / (kChannels / 4), kAtOnce = kStep < kTile ? kStep : kTile;
  const bool mine = left > 0 && q0 < kTile;
  float bias[4], skip[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool is = mine && i < left;
    bias[i] = is && p.delta_bias ? p.delta_bias[d0 + c4 + i] : 0.0f;
    skip[i] = is && p.skip ? p.skip[d0 + c4 + i] : 0.0f;
  }
  const int64_t xo = int64_t(b) * p.x.sb + int64_t(d0 + c4) * p.x.sd;
  const int64_t deltao = int64_t(b) * p.delta.sb + int64_t(d0 + c4) * p.delta.sd;
  const int64_t zo = int64_t(b) * p.z.sb + int64_t(d0 + c4) * p.z.sd;
  Raw xin[kPasses], din[kPasses], zin[kPasses];     // on their way
  Raw xnext[kPasses], znext[kPasses], xnow[kPasses], znow[kPasses];
  const auto read = [&](int tile) {
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
      const int t = s0 + tile * kTile + q0 + k * kStep;
      const bool live = mine && q0 + k * kStep < kTile && t < end;
      xin[k] = live ? four_channels<BF, WIDE>(p.x, xo + int64_t(t) * p.x.st, left) : P::zero();
      din[k] = live ? four_channels<BF, WIDE>(p.delta, deltao + int64_t(t) * p.delta.st, left) : P::zero();
      if (OUT && p.z.p) zin[k] = live ? four_channels<BF, WIDE>(p.z, zo + int64_t(t) * p.z.st, left) : P::zero();
    }
  };
  const auto convert = [&](int tile) {
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
      const int q = q0 + k * kStep, t = s0 + tile * kTile + q;
      xnext[k] = xin[k];
      if (OUT) znext[k] = zin[k];
      if (!mine || q >= kTile) continue;
      float x[4], v[4];
      P::open(xin[k], x);
      P::open(din[k], v);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] += bias[i];
        if (p.softplus) v[i] = softplus_of(v[i]);
        v[i] = t < end ? v[i] : 0.0f;  // a token that does not exist changes no state
        x[i] *= v[i];
      }
      *reinterpret_cast<f32x4*>(&l.dt[tile & 1][q][c4]) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4*>(&l.dx[tile & 1][q][c4]) = f32x4{x[0], x[1], x[2], x[3]};
    }
  };

  // the wave's rows of b and c: lane j of 16 has token j's
  RowRaw<BF> brow, crow;
  const int64_t bo = int64_t(b) * p.b.sb + int64_t(g) * p.b.sg, co = int64_t(b) * p.c.sb + int64_t(g) * p.c.sg;
  const auto read_rows = [&](int tile) {
    const int t = s0 + tile * kTile + lane % kTile;
    const bool live = t < end;
    brow.load(p.b, bo + int64_t(live ? t : 0) * p.b.st, n0, p.N, live);
    if (OUT) crow.load(p.c, co + int64_t(live ? t : 0) * p.c.st, n0, p.N, live);
  };

  const bool is = lane < channels;
  const int64_t d = d0 + lane;
  float rate[kScanStates], h[kScanStates], steps = 0.0f;
  rates(p.a, d, n0, p.N, is, rate);
  if (OUT) {
    read_states(p.initial, int64_t(b) * p.D + d, n0, p.N, is, h);
    for (int m = 0; m < seg; ++m) {
      const int64_t row = int64_t(m) * p.B + b;
      const f32x4 own = is ? *reinterpret_cast<const f32x4*>(p.seg_state + packed_at(p, row, wave, d)) : zero4();
      const float sum = is ? p.seg_steps[row * p.D + d] : 0.0f;
#pragma unroll
      for (int i = 0; i < kScanStates; ++i) h[i] = fmaf(exp2_of(sum * rate[i]), h[i], own[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kScanStates; ++i) h[i] = 0.0f;
  }

  if (tiles > 0) {
    read(0);
    read_rows(0);
    convert(0);
    if (tiles > 1) read(1);
  }
  __syncthreads();
  for (int tile = 0; tile < tiles; ++tile) {
    const int buf = tile & 1;
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
      xnow[k] = xnext[k];
      if (OUT) znow[k] = znext[k];
    }
    float bv[kScanStates], cv[kScanStates];
    brow.open(bv);
    if (OUT) crow.open(cv);
    if (tile + 1 < tiles) read_rows(tile + 1);
    each<kTile>([&](auto J) {
      constexpr int j = decltype(J)::value;
      const float dt = l.dt[buf][j][lane], dx = l.dx[buf][j][lane];
      float y = 0.0f;
#pragma unroll
      for (int i = 0; i < kScanStates; ++i) {
        h[i] = fmaf(exp2_of(dt * rate[i]), h[i], of_token<j>(bv[i]) * dx);
        if (OUT) y = fmaf(of_token<j>(cv[i]), h[i], y);
      }
      if (OUT) l.y[buf][wave][j][lane] = y;
      else steps += dt;
    });
    if (tile + 1 < tiles) {
      convert(tile + 1);
      if (tile + 2 < tiles) read(tile + 2);
    }
    __syncthreads();
    if constexpr (OUT) {
#pragma unroll
      for (int k = 0; k < kPasses; ++k) {
        const int q = q0 + k * kStep, t = s0 + tile * kTile + q;
        if (!mine || q >= kTile || t >= end) continue;
        float x[4], y[4];
        P::open(xnow[k], x);
        f32x4 sum = *reinterpret_cast<const f32x4*>(&l.y[buf][0][q][c4]);
#pragma unroll
        for (int w = 1; w < W; ++w) sum += *reinterpret_cast<const f32x4*>(&l.y[buf][w][q][c4]);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = fmaf(skip[i], x[i], sum[i]);
        if (p.z.p) {
          float z[4];
          P::open(znow[k], z);
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] *= silu_of(z[i]);
        }
        put_channels<BF, WIDE>(p.out, (int64_t(b) * p.T + t) * p.D + d0 + c4, left, y);
      }
    }
  }
  if constexpr (OUT) {
    if (mine) {
      const float none[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int t = max(end, s0) + q0; t < s1; t += kAtOnce)
        put_channels<BF, WIDE>(p.out, (int64_t(b) * p.T + t) * p.D + d0 + c4, left, none);
    }
    if (p.last && seg == p.segments - 1) write_states(p.last, int64_t(b) * p.D + d, n0, p.N, is, h);
  } else if (is) {
    const int64_t row = int64_t(seg) * p.B + b;
    *reinterpret_cast<f32x4*>(p.seg_state + packed_at(p, row, wave, d)) = f32x4{h[0], h[1], h[2], h[3]};
    if (wave == 0) p.seg_steps[row * p.D + d] = steps;
  }
}

// One token of each row: a lane holds four states of a channel, L lanes (a power of two) a channel.
template <bool BF, int L, bool VEC>
__global__ __launch_bounds__(256) void scan_step(SsStep p) {
  using E = typename Piece<BF, 1>::E;
  const int64_t idx = (int64_t(blockIdx.x) * 256 + threadIdx.x) / L;
  const int n0 = int(threadIdx.x) % L * kScanStates;
  const int64_t b = idx / p.D;
  if (b >= p.B) return;
  const int d = int(idx % p.D), g = d / (p.D / p.G);
  const int64_t slot = p.slots ? p.slots[b] : b;
  E* out = static_cast<E*>(p.out) + b * p.D + d;
  if (slot < 0 || slot >= p.pool) {
    if (n0 == 0) Piece<BF, 1>::put(out, Piece<BF, 1>::zero());
    return;
  }
  float* state = p.state + slot * p.ss + int64_t(d) * p.N + n0;
  f32x4 h = zero4();
  if constexpr (VEC) {
    if (n0 < p.N) h = *reinterpret_cast<const f32x4*>(state);
  } else {
#pragma unroll
    for (int i = 0; i < kScanStates; ++i)
      if (n0 + i < p.N) h[i] = state[i];
  }
  const auto one = [&](const TokenView& v) {
    float f[1];
    Piece<BF, 1>::open(static_cast<const E*>(v.p)[b * v.sb + int64_t(d) * v.sd], f);
    return f[0];
  };
  const float x = one(p.x), z = p.z.p ? one(p.z) : 0.0f;
  float dt = one(p.delta) + (p.delta_bias ? p.delta_bias[d] : 0.0f);
  if (p.softplus) dt = softplus_of(dt);
  float rate[kScanStates], bv[kScanStates], cv[kScanStates];
  rates(p.a, d, n0, p.N, true, rate);
  RowRaw<BF> rows;
  rows.load(p.b, b * p.b.sb + int64_t(g) * p.b.sg, n0, p.N, true);
  rows.open(bv);
  rows.load(p.c, b * p.c.sb + int64_t(g) * p.c.sg, n0, p.N, true);
  rows.open(cv);
  float y = 0.0f;
#pragma unroll
  for (int i = 0; i < kScanStates; ++i) {
    h[i] = fmaf(exp2_of(dt * rate[i]), h[i], dt * x * bv[i]);
    y = fmaf(cv[i], h[i], y);
  }
  if constexpr (VEC) {
    if (n0 < p.N) *reinterpret_cast<f32x4*>(state) = h;
  } else {
#pragma unroll
    for (int i = 0; i < kScanStates; ++i)
      if (n0 + i < p.N) state[i] = h[i];
  }
#pragma unroll
  for (int m = 1; m < L; m *= 2) y += __shfl_xor(y, m);
  y = fmaf(p.skip ? p.skip[d] : 0.0f, x, y);
  if (p.z.p) y *= silu_of(z);
  if (n0 == 0) Piece<BF, 1>::store(out, {y});
}

template <bool BF, int W, bool WIDE>
hipError_t launch_waves(const SsParams& p, hipStream_t stream) {
  const int64_t per_group = p.D / p.G, blocks = (per_group + kChannels - 1) / kChannels;
  const int64_t units = blocks * p.G * p.B;
  if (p.segments > 1)
    scan_march<BF, W, WIDE, false><<<unsigned(units * (p.segments - 1)), kWave * W, 0, stream>>>(p);
  scan_march<BF, W, WIDE, true><<<unsigned(units * p.segments), kWave * W, 0, stream>>>(p);
  return hipGetLastError();
}

template <bool BF, bool WIDE>
hipError_t launch_states(const SsParams& p, hipStream_t stream) {
  switch (p.waves) {
    case 1: return launch_waves<BF, 1, WIDE>(p, stream);
    case 2: return launch_waves<BF, 2, WIDE>(p, stream);
    case 4: return launch_waves<BF, 4, WIDE>(p, stream);
    default: return launch_waves<BF, 8, WIDE>(p, stream);
  }
}

template <bool BF, int L>
void launch_step(const SsStep& p, bool vec, hipStream_t stream) {
  const unsigned grid = unsigned((int64_t(p.B) * p.D * L + 255) / 256);
  if (vec) scan_step<BF, L, true><<<grid, 256, 0, stream>>>(p);
  else scan_step<BF, L, false><<<grid, 256, 0, stream>>>(p);
}

template <bool BF>
void launch_step_states(const SsStep& p, bool vec, hipStream_t stream) {
  if (p.N <= 4) launch_step<BF, 1>(p, vec, stream);
  else if (p.N <= 8) launch_step<BF, 2>(p, vec, stream);
  else if (p.N <= 16) launch_step<BF, 4>(p, vec, stream);
  else launch_step<BF, 8>(p, vec, stream);
}

}  // namespace

hipError_t launch_selective_scan(const SsParams& p, hipStream_t stream) {
  const bool wide = p.x.sd == 1 && p.delta.sd == 1 && (!p.z.p || p.z.sd == 1) && (p.D / p.G) % 4 == 0;
  if (p.bf16) return wide ? launch_states<true, true>(p, stream) : launch_states<true, false>(p, stream);
  return wide ? launch_states<false, true>(p, stream) : launch_states<false, false>(p, stream);
}

void selective_scan_split(SsParams& p, bool gradient) {
  const int64_t per_group = p.D / p.G;
  p.waves = p.N <= 4 ? 1 : p.N <= 8 ? 2 : p.N <= 16 ? 4 : 8;
  const int64_t waves = (per_group + kChannels - 1) / kChannels * p.G * p.B * p.waves;
  const int64_t tiles = (int64_t(p.T) + kTile - 1) / kTile;
  // Two waves a SIMD; segments of four tiles at least.
  int64_t segments = std::max<int64_t>(1, std::min(int64_t(device_cu_count()) * 8 / std::max<int64_t>(waves, 1), tiles / 4));
  const int64_t per = std::max<int64_t>(1, (tiles + segments - 1) / segments);
  p.seg_tokens = int(std::min<int64_t>(per * kTile, int64_t(1) << 30));
  p.segments = int(std::max<int64_t>(1, (tiles + per - 1) / per));
  p.row_marks = int((int64_t(p.T) + kMarkTokens - 1) / kMarkTokens);
}

hipError_t launch_selective_scan_step(const SsStep& p, hipStream_t stream) {
  const bool vec = p.N % 4 == 0 && p.ss % 4 == 0 && (reinterpret_cast<uintptr_t>(p.state) & 15u) == 0;
  if (p.bf16) launch_step_states<true>(p, vec, stream);
  else launch_step_states<false>(p, vec, stream);
  return hipGetLastError();
}

}  // namespace sx
