// selective_scan_grad.hip: the gradient of the selective scan.
//
// With gy = gout silu(z), lam[t] the adjoint of h[t] and mu[t] = exp(dt a) lam[t] what it passes back,
//   lam[t] = c[t] gy + mu[t + 1]  (the last state's gradient behind the last token)
//   gc[t] = sum over channels of gy h[t],   gb[t] = sum over channels of dt x lam[t]
//   q = mu[t] h[t-1],  ga = sum over t of dt q,  gdt = sum over n of (a q) + x sum over n of (lam b)
//   gx = dt sum over n of (lam b) + skip gy,  gdelta = gdt sigmoid(delta + delta_bias)
//   gz = gout y silu'(z),  gskip = sum of gy x,  gbias = sum of gdelta,  ginitial = mu of the first token
//
// Three passes. mark_states marches forward and leaves the state before every
// eighth token; where the tokens are split into segments each marches from zero,
// with its adjoint: lam at its start is a sum over its tokens of the decays up to them, c and gy.
// carry joins the segments, states forward and adjoints back. grad_march then takes
// the eight tokens between two marks, last to first: it runs their states
// forward again from the mark into registers, decays too, and the adjoint back over them.
// What is left is sums over workgroups (sum_rows, token_rows).
//
// grad_march: a lane has two channels and four states of each, so that what is
// summed over channels is summed over two for nothing; over the lanes, 64 values
// at a time (eight tokens of four states of b and of c) fold into one a lane: each
// step adds halves of a pair of registers to one, 141 instructions for 64 sums.
#include <algorithm>

#include "scan_march.hpp"

namespace sx {
namespace {

constexpr int kTile = 2 * kMarkTokens, kChannels = 64;

// The marks of row b, and the segments' own states, sums of dt and adjoints (JOIN: more than one segment).
template <bool BF, int W, bool WIDE, bool JOIN>
__global__ __launch_bounds__(kWave* W) void mark_states(SsParams p) {
  using P = Piece<BF, 4>;
  using Raw = typename P::Raw;
  constexpr int kPieces = kTile * kChannels / 4, kPasses = (kPieces + kWave * W - 1) / (kWave * W);
  __shared__ float ldt[2][kTile][kChannels], ldx[2][kTile][kChannels], lgy[JOIN ? 2 : 1][JOIN ? kTile : 1][kChannels];
  const int tid = int(threadIdx.x), lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int n0 = wave * kScanStates;
  const int per_group = p.D / p.G, blocks = (per_group + kChannels - 1) / kChannels;
  uint32_t at = blockIdx.x;
  const int cb = int(at % uint32_t(blocks));
  at /= uint32_t(blocks);
  const int g = int(at % uint32_t(p.G));
  at /= uint32_t(p.G);
  const int b = int(at % uint32_t(p.B)), seg = int(at / uint32_t(p.B));
  const int d0 = g * per_group + cb * kChannels, channels = min(kChannels, per_group - cb * kChannels);
  const int s0 = seg * p.seg_tokens, s1 = min(s0 + p.seg_tokens, p.T);
  const int end = min(s1, row_length(p.lengths, b, p.T));
  const int tiles = end > s0 ? (end - s0 + kTile - 1) / kTile : 0;
  const int q0 = tid / (kChannels / 4), c4 = tid % (kChannels / 4) * 4, left = channels - c4;
  constexpr int kStep = W * kWave / (kChannels / 4);
  const bool mine = left > 0 && q0 < kTile;
  float bias[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) bias[i] = mine && i < left && p.delta_bias ? p.delta_bias[d0 + c4 + i] : 0.0f;
  const int64_t xo = int64_t(b) * p.x.sb + int64_t(d0 + c4) * p.x.sd;
  const int64_t deltao = int64_t(b) * p.delta.sb + int64_t(d0 + c4) * p.delta.sd;
  const int64_t zo = int64_t(b) * p.z.sb + int64_t(d0 + c4) * p.z.sd;
  const int64_t goo = int64_t(b) * p.go.sb + int64_t(d0 + c4) * p.go.sd;
  Raw xin[kPasses], din[kPasses], zin[kPasses], gin[kPasses];
  const auto read = [&](int tile) {
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
      const int t = s0 + tile * kTile + q0 + k * kStep;
      const bool live = mine && q0 + k * kStep < kTile && t < end;
      xin[k] = live ? four_channels<BF, WIDE>(p.x, xo + int64_t(t) * p.x.st, left) : P::zero();
      din[k] = live ? four_channels<BF, WIDE>(p.delta, deltao + int64_t(t) * p.delta.st, left) : P::zero();
      if (JOIN) gin[k] = live ? four_channels<BF, WIDE>(p.go, goo + int64_t(t) * p.go.st, left) : P::zero();
      if (JOIN && p.z.p) zin[k] = live ? four_channels<BF, WIDE>(p.z, zo + int64_t(t) * p.z.st, left) : P::zero();
    }
  };
  const auto convert = [&](int tile) {
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
      const int q = q0 + k * kStep, t = s0 + tile * kTile + q;
      if (!mine || q >= kTile) continue;
      float x[4], v[4];
      P::open(xin[k], x);
      P::open(din[k], v);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] += bias[i];
        if (p.softplus) v[i] = softplus_of(v[i]);
        v[i] = t < end ? v[i] : 0.0f;
        x[i] *= v[i];
      }
      *reinterpret_cast<f32x4*>(&ldt[tile & 1][q][c4]) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4*>(&ldx[tile & 1][q][c4]) = f32x4{x[0], x[1], x[2], x[3]};
      if constexpr (JOIN) {
        float gy[4], z[4];
        P::open(gin[k], gy);
        if (p.z.p) {
          P::open(zin[k], z);
#pragma unroll
          for (int i = 0; i < 4; ++i) gy[i] *= silu_of(z[i]);
        }
        *reinterpret_cast<f32x4*>(&lgy[tile & 1][q][c4]) = f32x4{gy[0], gy[1], gy[2], gy[3]};
      }
    }
  };
  RowRaw<BF> brow, crow;
  const int64_t bo = int64_t(b) * p.b.sb + int64_t(g) * p.b.sg, co = int64_t(b) * p.c.sb + int64_t(g) * p.c.sg;
  const auto read_rows = [&](int tile) {
    const int t = s0 + tile * kTile + lane % kTile;
    const bool live = t < end;
    brow.load(p.b, bo + int64_t(live ? t : 0) * p.b.st, n0, p.N, live);
    if (JOIN) crow.load(p.c, co + int64_t(live ? t : 0) * p.c.st, n0, p.N, live);
  };
  const bool is = lane < channels;
  const int64_t d = d0 + lane;
  float rate[kScanStates], h[kScanStates], through[kScanStates], adj[kScanStates], steps = 0.0f;
  rates(p.a, d, n0, p.N, is, rate);
  read_states(JOIN ? nullptr : p.initial, int64_t(b) * p.D + d, n0, p.N, is, h);
#pragma unroll
  for (int i = 0; i < kScanStates; ++i) {
    through[i] = 1.0f;
    adj[i] = 0.0f;
  }
  const auto mark = [&](int t) {
    if (!is) return;
    const int64_t row = int64_t(b) * p.row_marks + t / kMarkTokens;
    *reinterpret_cast<f32x4*>(p.marks + packed_at(p, row, wave, d)) = f32x4{h[0], h[1], h[2], h[3]};
    if (JOIN && wave == 0) p.mark_steps[row * p.D + d] = steps;
  };
  if (tiles > 0) {
    read(0);
    read_rows(0);
    convert(0);
    if (tiles > 1) read(1);
  }
  __syncthreads();
  for (int tile = 0; tile < tiles; ++tile) {
    const int buf = tile & 1, t0 = s0 + tile * kTile;
    float bv[kScanStates], cv[kScanStates];
    brow.open(bv);
    if (JOIN) crow.open(cv);
    if (tile + 1 < tiles) read_rows(tile + 1);
    each<kTile>([&](auto J) {
      constexpr int j = decltype(J)::value;
      if (j == 0) mark(t0);
      if (j == kMarkTokens && t0 + kMarkTokens < end) mark(t0 + kMarkTokens);
      const float dt = ldt[buf][j][lane], dx = ldx[buf][j][lane];
#pragma unroll
      for (int i = 0; i < kScanStates; ++i) {
        const float e = exp2_of(dt * rate[i]);
        h[i] = fmaf(e, h[i], of_token<j>(bv[i]) * dx);
        if constexpr (JOIN) {
          through[i] *= e;
          adj[i] = fmaf(through[i], of_token<j>(cv[i]) * lgy[buf][j][lane], adj[i]);
        }
      }
      steps += dt;
    });
    if (tile + 1 < tiles) {
      convert(tile + 1);
      if (tile + 2 < tiles) read(tile + 2);
    }
    __syncthreads();
  }
  if (JOIN && is) {
    const int64_t row = int64_t(seg) * p.B + b;
    *reinterpret_cast<f32x4*>(p.seg_state + packed_at(p, row, wave, d)) = f32x4{h[0], h[1], h[2], h[3]};
    *reinterpret_cast<f32x4*>(p.seg_adjoint + packed_at(p, row, wave, d)) = f32x4{adj[0], adj[1], adj[2], adj[3]};
    if (wave == 0) p.seg_steps[row * p.D + d] = steps;
  }
}

// A segment's own state becomes the one at its start (blockIdx.y 0), its own adjoint the one that enters at its
// end (1).
__global__ __launch_bounds__(256) void carry(SsParams p) {
  const int64_t idx = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t row = int64_t(p.waves) * p.D;  // of one batch row
  if (idx >= p.B * row) return;
  const int64_t b = idx / row, d = idx % p.D;
  const int n0 = int(idx % row / p.D) * kScanStates;
  const bool back = blockIdx.y == 1;
  float rate[kScanStates], h[kScanStates];
  rates(p.a, d, n0, p.N, true, rate);
  read_states(back ? p.grad_state : p.initial, b * p.D + d, n0, p.N, true, h);
  f32x4* at = reinterpret_cast<f32x4*>(back ? p.seg_adjoint : p.seg_state) + idx;
  const float* steps = p.seg_steps + b * p.D + d;
  constexpr int A = 4;  // segments read ahead of the chain
  for (int m = 0; m < p.segments; m += A) {
    f32x4 own[A];
    float sum[A];
#pragma unroll
    for (int k = 0; k < A; ++k) {
      const int s = min(m + k, p.segments - 1), j = back ? p.segments - 1 - s : s;
      own[k] = at[j * p.B * row];
      sum[k] = steps[int64_t(j) * p.B * p.D];
    }
#pragma unroll
    for (int k = 0; k < A; ++k) {
      if (m + k >= p.segments) break;
      const int j = back ? p.segments - 1 - (m + k) : m + k;
      at[j * p.B * row] = f32x4{h[0], h[1], h[2], h[3]};
#pragma unroll
      for (int i = 0; i < kScanStates; ++i) h[i] = fmaf(exp2_of(sum[k] * rate[i]), h[i], own[k][i]);
    }
  }
}

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}

// v[k] summed over the wave's lanes, in lane k. Registers k and k + H become one whose lanes with bit H of their
// number clear hold k's sum so far, the others that of k + H.
__device__ __forceinline__ float fold64(float (&v)[64], int lane) {
#pragma unroll
  for (int k = 0; k < 32; ++k) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[k]), __float_as_uint(v[k + 32]), false, false);
    v[k] = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v[k]), __float_as_uint(v[k + 16]), false, false);
    v[k] = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  // within a row of 16 the partner is the mirrored lane of the row, of its half, then two and one lanes away
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const bool up = lane & 8;
    v[k] = (up ? v[k + 8] : v[k]) + dpp<0x140>(up ? v[k] : v[k + 8]);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const bool up = lane & 4;
    v[k] = (up ? v[k + 4] : v[k]) + dpp<0x141>(up ? v[k] : v[k + 4]);
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const bool up = lane & 2;
    v[k] = (up ? v[k + 2] : v[k]) + dpp<0x4e>(up ? v[k] : v[k + 2]);
  }
  const bool up = lane & 1;
  return (up ? v[1] : v[0]) + dpp<0xb1>(up ? v[0] : v[1]);
}

constexpr int kWide = 128;  // channels of a workgroup of grad_march

template <int W>
struct GradLds {
  float dt[kMarkTokens][kWide], x[kMarkTokens][kWide], gy[kMarkTokens][kWide];
  float y[W][kMarkTokens][kWide], source[W][kMarkTokens][kWide], decay[W][kMarkTokens][kWide];
};

template <bool BF, int W, bool WIDE, bool JOIN>
__global__ __launch_bounds__(kWave* W) void grad_march(SsParams p) {
  using P = Piece<BF, 4>;
  using Raw = typename P::Raw;
  constexpr int M = kMarkTokens;
  constexpr int kPieces = M * kWide / 4, kPasses = (kPieces + kWave * W - 1) / (kWave * W);
  __shared__ GradLds<W> l;
  const int tid = int(threadIdx.x), lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int n0 = wave * kScanStates;
  const int per_group = p.D / p.G, blocks = (per_group + kWide - 1) / kWide;
  uint32_t at = blockIdx.x;
  const int cb = int(at % uint32_t(blocks));
  at /= uint32_t(blocks);
  const int g = int(at % uint32_t(p.G));
  at /= uint32_t(p.G);
  const int b = int(at % uint32_t(p.B)), seg = int(at / uint32_t(p.B));
  const int d0 = g * per_group + cb * kWide, channels = min(kWide, per_group - cb * kWide);
  const int s0 = seg * p.seg_tokens, s1 = min(s0 + p.seg_tokens, p.T);
  const int end = min(s1, row_length(p.lengths, b, p.T));
  const int spans = end > s0 ? (end - s0 + M - 1) / M : 0;
  const int q0 = tid / (kWide / 4), c4 = tid % (kWide / 4) * 4, left = channels - c4;
  constexpr int kStep = W * kWave / (kWide / 4), kAtOnce = kStep < M ? kStep : M;
  const bool mine = left > 0 && q0 < M;
  float bias[4], skip[4], gskip[4] = {}, gbias[4] = {};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool is = mine && i < left;
    bias[i] = is && p.delta_bias ? p.delta_bias[d0 + c4 + i] : 0.0f;
    skip[i] = is && p.skip ? p.skip[d0 + c4 + i] : 0.0f;
  }
  const int64_t xo = int64_t(b) * p.x.sb + int64_t(d0 + c4) * p.x.sd;
  const int64_t deltao = int64_t(b) * p.delta.sb + int64_t(d0 + c4) * p.delta.sd;
  const int64_t zo = int64_t(b) * p.z.sb + int64_t(d0 + c4) * p.z.sd;
  const int64_t goo = int64_t(b) * p.go.sb + int64_t(d0 + c4) * p.go.sd;
  Raw xin[kPasses], din[kPasses], zin[kPasses], gin[kPasses];
  Raw xnow[kPasses], dnow[kPasses], znow[kPasses], gnow[kPasses];
  const auto read = [&](int span) {
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
      const int t = s0 + span * M + q0 + k * kStep;
      const bool live = mine && q0 + k * kStep < M && t < end;
      xin[k] = live ? four_channels<BF, WIDE>(p.x, xo + int64_t(t) * p.x.st, left) : P::zero();
      din[k] = live ? four_channels<BF, WIDE>(p.delta, deltao + int64_t(t) * p.delta.st, left) : P::zero();
      gin[k] = live ? four_channels<BF, WIDE>(p.go, goo + int64_t(t) * p.go.st, left) : P::zero();
      if (p.z.p) zin[k] = live ? four_channels<BF, WIDE>(p.z, zo + int64_t(t) * p.z.st, left) : P::zero();
    }
  };
  const auto step_of = [&](float v) { return p.softplus ? softplus_of(v) : v; };

  // lanes 0 .. 7 of each row of 16 have the tokens' rows of b, 8 .. 15 those of c
  RowRaw<BF> rows;
  const bool second = lane & M;
  const RowView& rv = second ? p.c : p.b;
  const int64_t ro = int64_t(b) * rv.sb + int64_t(g) * rv.sg;
  const auto read_rows = [&](int span) {
    const int t = s0 + span * M + lane % M;
    const bool live = t < end;
    rows.load(rv, ro + int64_t(live ? t : 0) * rv.st, n0, p.N, live);
  };

  // two channels a lane
  const int64_t d = d0 + 2 * lane;
  bool is[2];
  float rate[2][kScanStates], start[2][kScanStates], mu[2][kScanStates], ga[2][kScanStates] = {};
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    is[c] = 2 * lane + c < channels;
    rates(p.a, d + c, n0, p.N, is[c], rate[c]);
    if constexpr (JOIN) {
      const int64_t row = int64_t(seg) * p.B + b;
#pragma unroll
      for (int i = 0; i < kScanStates; ++i) {
        start[c][i] = is[c] ? p.seg_state[packed_at(p, row, wave, d + c) + i] : 0.0f;
        mu[c][i] = is[c] ? p.seg_adjoint[packed_at(p, row, wave, d + c) + i] : 0.0f;
      }
    } else {
      read_states(p.grad_state, int64_t(b) * p.D + d + c, n0, p.N, is[c], mu[c]);
    }
  }
  f32x4 marks[2];
  float mark_steps[2];
  const auto read_marks = [&](int span) {
    const int64_t row = int64_t(b) * p.row_marks + s0 / M + span;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      marks[c] = is[c] ? *reinterpret_cast<const f32x4*>(p.marks + packed_at(p, row, wave, d + c)) : zero4();
      if (JOIN) mark_steps[c] = is[c] ? p.mark_steps[row * p.D + d + c] : 0.0f;
    }
  };

  // channels that do not exist add nothing to the sums over channels
  for (int i = tid; i < M * kWide; i += kWave * W) {
    (&l.dt[0][0])[i] = 0.0f;
    (&l.x[0][0])[i] = 0.0f;
    (&l.gy[0][0])[i] = 0.0f;
  }
  if (spans > 0) {
    read(spans - 1);
    read_rows(spans - 1);
    read_marks(spans - 1);
  }
  __syncthreads();
  for (int span = spans - 1; span >= 0; --span) {
    const int t0 = s0 + span * M;
    // dt, x and gy of the tokens
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
      const int q = q0 + k * kStep;
      xnow[k] = xin[k];
      dnow[k] = din[k];
      gnow[k] = gin[k];
      znow[k] = zin[k];
      if (!mine || q >= M) continue;
      float x[4], v[4], gy[4], z[4];
      P::open(xin[k], x);
      P::open(din[k], v);
      P::open(gin[k], gy);
      if (p.z.p) {
        P::open(zin[k], z);
#pragma unroll
        for (int i = 0; i < 4; ++i) gy[i] *= silu_of(z[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = t0 + q < end && i < left ? step_of(v[i] + bias[i]) : 0.0f;
      if (!WIDE) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] = i < left ? x[i] : 0.0f;
          gy[i] = i < left ? gy[i] : 0.0f;
        }
      }
      *reinterpret_cast<f32x4*>(&l.dt[q][c4]) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4*>(&l.x[q][c4]) = f32x4{x[0], x[1], x[2], x[3]};
      *reinterpret_cast<f32x4*>(&l.gy[q][c4]) = f32x4{gy[0], gy[1], gy[2], gy[3]};
    }
    float rowv[kScanStates];  // of b and of c
    rows.open(rowv);
    // the states before each token, from the mark on; and the decays
    float hs[M + 1][2][kScanStates], es[M][2][kScanStates];
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int i = 0; i < kScanStates; ++i) {
        hs[0][c][i] = marks[c][i];
        if constexpr (JOIN) hs[0][c][i] = fmaf(exp2_of(mark_steps[c] * rate[c][i]), start[c][i], hs[0][c][i]);
      }
    if (span > 0) {
      read(span - 1);
      read_rows(span - 1);
      read_marks(span - 1);
    }
    __syncthreads();
    each<M>([&](auto J) {
      constexpr int j = decltype(J)::value;
      float y[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float dt = l.dt[j][2 * lane + c], dx = dt * l.x[j][2 * lane + c];
        y[c] = 0.0f;
#pragma unroll
        for (int i = 0; i < kScanStates; ++i) {
          es[j][c][i] = exp2_of(dt * rate[c][i]);
          hs[j + 1][c][i] = fmaf(es[j][c][i], hs[j][c][i], of_token<j>(rowv[i]) * dx);
          y[c] = fmaf(of_token<M + j>(rowv[i]), hs[j + 1][c][i], y[c]);
        }
      }
      if (p.z.p) *reinterpret_cast<float2*>(&l.y[wave][j][2 * lane]) = make_float2(y[0], y[1]);
    });
    float sums[64];  // token, b or c, state
    each<M>([&](auto J) {
      constexpr int j = M - 1 - decltype(J)::value;
      float source[2], decay[2];
#pragma unroll
      for (int i = 0; i < 8; ++i) sums[8 * j + i] = 0.0f;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float dt = l.dt[j][2 * lane + c], dx = dt * l.x[j][2 * lane + c], gy = l.gy[j][2 * lane + c];
        source[c] = decay[c] = 0.0f;
#pragma unroll
        for (int i = 0; i < kScanStates; ++i) {
          const float lam = fmaf(of_token<M + j>(rowv[i]), gy, mu[c][i]);
          sums[8 * j + i] = fmaf(lam, dx, sums[8 * j + i]);
          sums[8 * j + 4 + i] = fmaf(gy, hs[j + 1][c][i], sums[8 * j + 4 + i]);
          source[c] = fmaf(of_token<j>(rowv[i]), lam, source[c]);
          mu[c][i] = es[j][c][i] * lam;
          const float q = mu[c][i] * hs[j][c][i];
          ga[c][i] = fmaf(dt, q, ga[c][i]);
          decay[c] = fmaf(rate[c][i], q, decay[c]);
        }
      }
      *reinterpret_cast<float2*>(&l.source[wave][j][2 * lane]) = make_float2(source[0], source[1]);
      *reinterpret_cast<float2*>(&l.decay[wave][j][2 * lane]) = make_float2(decay[0], decay[1]);
    });
    const float sum = fold64(sums, lane);
    {
      const int t = t0 + lane / 8, which = lane / 4 % 2, n = n0 + lane % 4;
      if (t < end)
        p.rows_partial[(((int64_t(b) * p.G + g) * p.T + t) * blocks + cb) * (8 * W) + which * 4 * W + n] = sum;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
      const int q = q0 + k * kStep, t = t0 + q;
      if (!mine || q >= M || t >= end) continue;
      float x[4], v[4], go[4], z[4], gx[4], gd[4], gz[4];
      P::open(xnow[k], x);
      P::open(dnow[k], v);
      P::open(gnow[k], go);
      if (p.z.p) P::open(znow[k], z);
      f32x4 y = zero4(), source = zero4(), decay = zero4();
#pragma unroll
      for (int w = 0; w < W; ++w) {
        if (p.z.p) y += *reinterpret_cast<const f32x4*>(&l.y[w][q][c4]);
        source += *reinterpret_cast<const f32x4*>(&l.source[w][q][c4]);
        decay += *reinterpret_cast<const f32x4*>(&l.decay[w][q][c4]);
      }
      const f32x4 dt = *reinterpret_cast<const f32x4*>(&l.dt[q][c4]);
      const f32x4 gy = *reinterpret_cast<const f32x4*>(&l.gy[q][c4]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        gx[i] = fmaf(dt[i], source[i], skip[i] * gy[i]);
        gskip[i] = fmaf(gy[i], x[i], gskip[i]);
        // the rates stand times log2(e)
        gd[i] = fmaf(decay[i], 1.0f / kLog2e, x[i] * source[i]);
        if (p.softplus) gd[i] *= sigmoid_of(v[i] + bias[i]);
        gbias[i] += gd[i];
        if (p.z.p) gz[i] = go[i] * fmaf(skip[i], x[i], y[i]) * silu_slope(z[i]);
      }
      const int64_t o = (int64_t(b) * p.T + t) * p.D + d0 + c4;
      put_channels<BF, WIDE>(p.gx, o, left, gx);
      put_channels<BF, WIDE>(p.gdelta, o, left, gd);
      if (p.z.p) put_channels<BF, WIDE>(p.gz, o, left, gz);
    }
    // the next span's dt, x and gy go where these were read
    __syncthreads();
  }
  // tokens that do not exist
  if (mine) {
    const float none[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int t = max(end, s0) + q0; t < s1; t += kAtOnce) {
      const int64_t o = (int64_t(b) * p.T + t) * p.D + d0 + c4;
      put_channels<BF, WIDE>(p.gx, o, left, none);
      put_channels<BF, WIDE>(p.gdelta, o, left, none);
      if (p.z.p) put_channels<BF, WIDE>(p.gz, o, left, none);
    }
  }
  const int64_t row = int64_t(seg) * p.B + b;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    write_states(p.a_partial, row * p.D + d + c, n0, p.N, is[c], ga[c]);
    if (seg == 0 && p.ginitial) write_states(p.ginitial, int64_t(b) * p.D + d + c, n0, p.N, is[c], mu[c]);
  }
  // the threads' shares of a channel's sums over tokens meet in LDS
  __syncthreads();
  if (mine) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      l.source[0][q0][c4 + i] = gskip[i];
      l.decay[0][q0][c4 + i] = gbias[i];
    }
  }
  __syncthreads();
  for (int c = tid; c < channels; c += kWave * W) {
    float a = 0.0f, v = 0.0f;
#pragma unroll
    for (int q = 0; q < kAtOnce; ++q) {
      a += l.source[0][q][c];
      v += l.decay[0][q][c];
    }
    p.skip_partial[row * p.D + d0 + c] = a;
    p.bias_partial[row * p.D + d0 + c] = v;
  }
}

// The gradients of b and c: the workgroups' sums of a token's rows, together. A thread has one value.
template <bool BF>
__global__ __launch_bounds__(256) void token_rows(SsParams p, int blocks) {
  using E = typename Piece<BF, 1>::E;
  const int cols = 8 * p.waves;  // b's, then c's
  const int64_t idx = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t row = idx / cols;  // (b, g, t)
  if (row >= int64_t(p.B) * p.G * p.T) return;
  const int col = int(idx % cols), n = col % (4 * p.waves);
  if (n >= p.N) return;
  const int t = int(row % p.T), g = int(row / p.T % p.G), b = int(row / p.T / p.G);
  float v = 0.0f;
  if (t < row_length(p.lengths, b, p.T)) {
    const float* at = p.rows_partial + row * blocks * cols + col;
#pragma unroll 4
    for (int k = 0; k < blocks; ++k) v += at[int64_t(k) * cols];
  }
  E* out = static_cast<E*>(col < 4 * p.waves ? p.gb : p.gc);
  Piece<BF, 1>::store(out + ((int64_t(b) * p.T + t) * p.G + g) * p.N + n, {v});
}

template <bool BF, int W, bool WIDE, bool JOIN>
hipError_t launch_join(const SsParams& p, hipStream_t stream) {
  const int64_t per_group = p.D / p.G;
  const int64_t units = int64_t(p.G) * p.B * p.segments;
  mark_states<BF, W, WIDE, JOIN>
      <<<unsigned((per_group + kChannels - 1) / kChannels * units), kWave * W, 0, stream>>>(p);
  if (JOIN) {
    const int64_t n = int64_t(p.B) * p.waves * p.D;
    carry<<<dim3(unsigned((n + 255) / 256), 2), 256, 0, stream>>>(p);
  }
  grad_march<BF, W, WIDE, JOIN><<<unsigned((per_group + kWide - 1) / kWide * units), kWave * W, 0, stream>>>(p);
  return hipGetLastError();
}

template <bool BF, int W, bool WIDE>
hipError_t launch_waves(const SsParams& p, hipStream_t stream) {
  return p.segments > 1 ? launch_join<BF, W, WIDE, true>(p, stream) : launch_join<BF, W, WIDE, false>(p, stream);
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

}  // namespace

int selective_scan_grad_blocks(const SsParams& p) { return (p.D / p.G + kWide - 1) / kWide; }

hipError_t launch_selective_scan_backward(const SsParams& p, hipStream_t stream) {
  const bool wide = p.x.sd == 1 && p.delta.sd == 1 && p.go.sd == 1 && (!p.z.p || p.z.sd == 1) &&
                    (p.D / p.G) % 4 == 0;
  hipError_t err = hipSuccess;
  if (p.B > 0) {
    if (p.bf16) err = wide ? launch_states<true, true>(p, stream) : launch_states<true, false>(p, stream);
    else err = wide ? launch_states<false, true>(p, stream) : launch_states<false, false>(p, stream);
    if (err != hipSuccess) return err;
    const int64_t n = int64_t(p.B) * p.G * p.T * 8 * p.waves;
    const int blocks = selective_scan_grad_blocks(p);
    if (n > 0) {
      const unsigned grid = unsigned((n + 255) / 256);
      if (p.bf16) token_rows<true><<<grid, 256, 0, stream>>>(p, blocks);
      else token_rows<false><<<grid, 256, 0, stream>>>(p, blocks);
    }
  }
  SumRows s{};
  const int64_t rows = int64_t(p.B) * p.segments, D = p.D;
  s.count = 3;
  s.s[0] = {p.a_partial, p.ga, rows, D * p.N, D * p.N, 1};
  s.s[1] = {p.skip_partial, p.gskip, rows, D, D, 1};
  s.s[2] = {p.bias_partial, p.gbias, rows, D, D, 1};
  return launch_sum_rows(s, stream);
}

}  // namespace sx
