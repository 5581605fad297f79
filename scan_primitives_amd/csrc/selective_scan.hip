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
// read x and z sum the parts, gate and store. The next
// tile's dt are formed before the barrier, its loads are on their way since the tile before.
// b and c are operands of no cost: lane j of each row of 16 lanes holds token j's
// values, and an instruction reads them from there (DPP row_newbcast).
//
// Long sequences of few channels are split into segments. A first pass marches each from
// zero, its state and sum of dt kept; the second starts segment m from the ones before it:
// h <- exp(a sum of dt) h + state.
//
// Bound by the issue of vector instructions. A state of a token takes an exponential (two slots) with its argument, a
// product with b, a sum and a product with c: 6 slots (5 in the first pass), and a channel of a token some 25 more for
// softplus, the gate and conversions. 8192 tokens of 4096 channels of 16 states in bf16: 269 to 273 us (under a profiler
// 122 the first pass and 181 the second); the bytes alone would take 52. The vector pipes issue in 75% of the cycles; a
// wave stands at a wait or a barrier a third of its time in the first pass and 41% in the second, with four on a SIMD.
#include <algorithm>

#include "scan_march.hpp"

namespace sx {
namespace {

// One token of each row: a lane holds 4 S states of a channel, L lanes (a power of two) a channel. VEC: states, rates, b
// and c by fours. Bound by memory: the states are read and written once. What bounded it before was the number of
// loads: with eight states a lane and all by fours, 128 requests of 4096 channels of 16 states take 16.1 us, 4.2 TB/s;
// 28.7 with four states and by elements. Four rows a lane, their rates read once, gain nothing (16.2).
template <bool BF, int L, int S, bool VEC>
__global__ __launch_bounds__(256) void scan_step(SsStep p) {
  using E = typename Piece<BF, 1>::E;
  using P4 = Piece<BF, 4>;
  const int64_t idx = (int64_t(blockIdx.x) * 256 + threadIdx.x) / L;
  const int n0 = int(threadIdx.x) % L * 4 * S;
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
  const float* a = p.a + int64_t(d) * p.N + n0;
  const E* brow = static_cast<const E*>(p.b.p) + b * p.b.sb + int64_t(g) * p.b.sg + n0 * p.b.sn;
  const E* crow = static_cast<const E*>(p.c.p) + b * p.c.sb + int64_t(g) * p.c.sg + n0 * p.c.sn;
  const int left = p.N - n0;  // states from the lane's first on
  f32x4 h[S], rate[S];
  typename P4::Raw braw[S], craw[S];
#pragma unroll
  for (int i = 0; i < S; ++i) {
    if constexpr (VEC) {
      const bool is = 4 * i < left;
      h[i] = is ? *reinterpret_cast<const f32x4*>(state + 4 * i) : zero4();
      rate[i] = is ? *reinterpret_cast<const f32x4*>(a + 4 * i) : zero4();
      braw[i] = is ? P4::load(brow + 4 * i) : P4::zero();
      craw[i] = is ? P4::load(crow + 4 * i) : P4::zero();
    } else {
      const auto one = [&](const E* row, int64_t sn, int k) { return 4 * i + k < left ? row[(4 * i + k) * sn] : E(0); };
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        h[i][k] = 4 * i + k < left ? state[4 * i + k] : 0.0f;
        rate[i][k] = 4 * i + k < left ? a[4 * i + k] : 0.0f;
      }
      braw[i] = P4::of(one(brow, p.b.sn, 0), one(brow, p.b.sn, 1), one(brow, p.b.sn, 2), one(brow, p.b.sn, 3));
      craw[i] = P4::of(one(crow, p.c.sn, 0), one(crow, p.c.sn, 1), one(crow, p.c.sn, 2), one(crow, p.c.sn, 3));
    }
  }
  const auto value = [&](const TokenView& v) {
    float f[1];
    Piece<BF, 1>::open(static_cast<const E*>(v.p)[b * v.sb + int64_t(d) * v.sd], f);
    return f[0];
  };
  const float x = value(p.x), z = p.z.p ? value(p.z) : 0.0f, skip = p.skip ? p.skip[d] : 0.0f;
  float dt = value(p.delta) + (p.delta_bias ? p.delta_bias[d] : 0.0f), y = 0.0f;
  if (p.softplus) dt = softplus_of(dt);
  const bool still = dt == 0.0f;  // whatever the rate (one times log2(e) may be infinite)
#pragma unroll
  for (int i = 0; i < S; ++i) {
    float bv[4], cv[4];
    P4::open(braw[i], bv);
    P4::open(craw[i], cv);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      h[i][k] = fmaf(still ? 1.0f : exp2_of(dt * (rate[i][k] * kLog2e)), h[i][k], dt * x * bv[k]);
      y = fmaf(cv[k], h[i][k], y);
    }
    if constexpr (VEC) {
      if (4 * i < left) *reinterpret_cast<f32x4*>(state + 4 * i) = h[i];
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (4 * i + k < left) state[4 * i + k] = h[i][k];
    }
  }
#pragma unroll
  for (int m = 1; m < L; m *= 2) y += __shfl_xor(y, m);
  y = fmaf(skip, x, y);
  if (p.z.p) y *= silu_of(z);
  if (n0 == 0) Piece<BF, 1>::store(out, {y});
}

template <bool BF, int W, Rows R>
hipError_t launch_waves(const SsParams& p, hipStream_t stream) {
  const int64_t per_group = p.D / p.G, blocks = (per_group + kChannels - 1) / kChannels;
  const int64_t units = blocks * p.G * p.B;
  if (p.segments > 1)
    scan_march<BF, W, R, March::Segments><<<unsigned(units * (p.segments - 1)), kWave * W, 0, stream>>>(p);
  scan_march<BF, W, R, March::Out><<<unsigned(units * p.segments), kWave * W, 0, stream>>>(p);
  return hipGetLastError();
}

template <bool BF, Rows R>
hipError_t launch_states(const SsParams& p, hipStream_t stream) {
  switch (p.waves) {
    case 1: return launch_waves<BF, 1, R>(p, stream);
    case 2: return launch_waves<BF, 2, R>(p, stream);
    case 3: return launch_waves<BF, 3, R>(p, stream);
    case 4: return launch_waves<BF, 4, R>(p, stream);
    default: return launch_waves<BF, 8, R>(p, stream);
  }
}

template <bool BF, int L, int S>
void launch_step(const SsStep& p, bool vec, hipStream_t stream) {
  const unsigned grid = unsigned((int64_t(p.B) * p.D * L + 255) / 256);
  if (vec) scan_step<BF, L, S, true><<<grid, 256, 0, stream>>>(p);
  else scan_step<BF, L, S, false><<<grid, 256, 0, stream>>>(p);
}

template <bool BF>
void launch_step_states(const SsStep& p, bool vec, hipStream_t stream) {
  switch (selective_scan_step_lanes(p.N)) {
    case 1: p.N <= 4 ? launch_step<BF, 1, 1>(p, vec, stream) : launch_step<BF, 1, 2>(p, vec, stream); break;
    case 2: launch_step<BF, 2, 2>(p, vec, stream); break;
    default: launch_step<BF, 4, 2>(p, vec, stream);
  }
}

}  // namespace

hipError_t launch_selective_scan(const SsParams& p, hipStream_t stream) {
  switch (scan_rows(p, false, kChannels)) {
    case Rows::Whole: return p.bf16 ? launch_states<true, Rows::Whole>(p, stream) : launch_states<false, Rows::Whole>(p, stream);
    case Rows::Early: return p.bf16 ? launch_states<true, Rows::Early>(p, stream) : launch_states<false, Rows::Early>(p, stream);
    default: return p.bf16 ? launch_states<true, Rows::Any>(p, stream) : launch_states<false, Rows::Any>(p, stream);
  }
}

void selective_scan_split(SsParams& p, bool gradient) {
  const int64_t per_group = p.D / p.G;
  p.waves = p.N <= 16 ? (p.N + kScanStates - 1) / kScanStates : 8;
  const int64_t width = gradient ? kGradChannels : kChannels;
  const int64_t waves = (per_group + width - 1) / width * p.G * p.B * p.waves;
  const int64_t tiles = (int64_t(p.T) + kTile - 1) / kTile;
  // Four waves a SIMD (of the gradient two, which its registers leave). Segments of a tile at least (333 tokens of
  // 3 x 210 channels: the gradient takes 48 us, 116 with four tiles; the result of 100 tokens of 2048 12.5, 17), of two
  // in a result of more than eight, whose segments each join all before (400 tokens of 1536 channels: 18.4 us, 21 with
  // one); up to four tiles cost less than a second launch (37 tokens of 2048 channels: 10.1 us, 11.8 in segments).
  const int64_t most = gradient ? tiles : tiles > 8 ? tiles / 2 : tiles > 4 ? tiles : 1;
  const int64_t want = int64_t(device_cu_count()) * (gradient ? 8 : 16) / std::max<int64_t>(waves, 1);
  const int64_t segments = std::max<int64_t>(1, std::min(want, most));
  const int64_t per = std::max<int64_t>(1, (tiles + segments - 1) / segments);
  p.seg_tokens = int(std::min<int64_t>(per * kTile, int64_t(1) << 30));
  p.segments = int(std::max<int64_t>(1, (tiles + per - 1) / per));
  p.row_marks = int((int64_t(p.T) + kMarkTokens - 1) / kMarkTokens);
}

int selective_scan_step_lanes(int N) { return N <= 8 ? 1 : N <= 16 ? 2 : 4; }

hipError_t launch_selective_scan_step(const SsStep& p, hipStream_t stream) {
  const bool vec = p.N % 4 == 0 && p.ss % 4 == 0 && (reinterpret_cast<uintptr_t>(p.state) & 15u) == 0 &&
                   (reinterpret_cast<uintptr_t>(p.a) & 15u) == 0 && p.b.sn == 1 && p.c.sn == 1;
  if (p.bf16) launch_step_states<true>(p, vec, stream);
  else launch_step_states<false>(p, vec, stream);
  return hipGetLastError();
}

}  // namespace sx
