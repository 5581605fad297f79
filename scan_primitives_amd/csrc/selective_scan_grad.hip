// selective_scan_grad.hip: the gradient of the selective scan.
//
// With gy = gout silu(z), lam[t] the adjoint of h[t] and mu[t] = exp(dt a) lam[t] what it passes back,
//   lam[t] = c[t] gy + mu[t + 1]  (the last state's gradient behind the last token)
//   gc[t] = sum over channels of gy h[t],   gb[t] = sum over channels of dt x lam[t]
//   q = mu[t] h[t-1],  ga = sum over t of dt q,  gdt = sum over n of (a q) + x sum over n of (lam b)
//   gx = dt sum over n of (lam b) + skip gy,  gdelta = gdt sigmoid(delta + delta_bias)
//   gz = gout y silu'(z),  gskip = sum of gy x,  gbias = sum of gdelta,  ginitial = mu of the first token
//
// Three passes. scan_march goes forward and leaves the state before every
// eighth token; where the tokens are split into segments each marches from zero,
// with its adjoint: lam at its start is a sum over its tokens of the decays up to them, c and gy.
// carry joins the segments, states forward and adjoints back. grad_march then takes
// the eight tokens between two marks, last to first: it runs their states
// forward again from the mark into registers, decays too, and the adjoint back over them.
// What is left is sums over workgroups (sum_rows, token_rows).
//
// grad_march: a lane has two channels and four states of each, so that what is
// summed over channels is summed over two for nothing; over the lanes, 64 sums at
// a time (eight tokens of four states of b and of c) fold into one a lane, in 140 additions.
//
// Bound by the issue of vector instructions (75% of the cycles of grad_march, which leaves two waves a SIMD: its
// registers hold the states before eight tokens). 4 x 2048 tokens of 2048 channels of 16 states in bf16: 354 us; the
// bytes alone would take 46. Under a profiler, where a launch costs some more, 114 scan_march, 7 carry, 272 grad_march
// and 11 the sums.
#include <algorithm>

#include "scan_march.hpp"

namespace sx {
namespace {

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
  struct Runs {
    f32x4 own[A];
    float sum[A];
  } next;
  const auto read = [&](int m) {
#pragma unroll
    for (int k = 0; k < A; ++k) {
      const int s = min(m + k, p.segments - 1), j = back ? p.segments - 1 - s : s;
      next.own[k] = at[j * p.B * row];
      next.sum[k] = steps[int64_t(j) * p.B * p.D];
    }
  };
  read(0);
  const auto chain = [&](auto grows) {
    for (int m = 0; m < p.segments; m += A) {
      const Runs now = next;
      if (m + A < p.segments) read(m + A);
#pragma unroll
      for (int k = 0; k < A; ++k) {
        if (m + k >= p.segments) break;
        const int j = back ? p.segments - 1 - (m + k) : m + k;
        at[j * p.B * row] = f32x4{h[0], h[1], h[2], h[3]};
        carry_over(grows, now.sum[k], rate, now.own[k], h);
      }
    }
  };
  if (may_grow(p, rate)) chain(std::true_type());
  else chain(std::false_type());
}

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}

// Sums over lanes: a step adds two registers into one whose lanes with a bit of their number clear hold the first's
// sum so far and the others the second's. Bit 3's partner is the mirrored lane of the row of 16, bit 2's that of its
// half, and which register a lane takes is the instruction's bank mask. Of the eight sums of a token: four in each
// of two registers. The waits are for a sum that was written just before, and for a swap that takes one just behind.
__device__ __forceinline__ void fold_token(const float (&v)[8], float (&s)[2]) {
  float r[4];
#define SX_PAIR(O, A, B, HOW, LOW, HIGH)                                            \
  "v_add_f32_dpp %" O ", %" A ", %" A " " HOW " row_mask:0xf bank_mask:" LOW "\n\t" \
  "v_add_f32_dpp %" O ", %" B ", %" B " " HOW " row_mask:0xf bank_mask:" HIGH "\n\t"
#define SX_ROW(O, A, B) SX_PAIR(O, A, B, "row_mirror", "0x3", "0xc")
#define SX_HALF(O, A, B) SX_PAIR(O, A, B, "row_half_mirror", "0x5", "0xa")
  asm("s_nop 1\n\t" SX_ROW("2", "6", "10") SX_ROW("3", "7", "11") SX_ROW("4", "8", "12") SX_ROW("5", "9", "13")
          SX_HALF("0", "2", "4") SX_HALF("1", "3", "5") "s_nop 1"
      : "=&v"(s[0]), "=&v"(s[1]), "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3])
      : "v"(v[0]), "v"(v[1]), "v"(v[2]), "v"(v[3]), "v"(v[4]), "v"(v[5]), "v"(v[6]), "v"(v[7]));
#undef SX_HALF
#undef SX_ROW
#undef SX_PAIR
}

// ... and of eight tokens: rows of 16 lanes (bits 5 and 4) take the tokens apart, quads are summed whole, and lane k
// of a quad keeps the fourth register k. The lane's sum is of token 4 bit5 + 2 bit4 + bit1, of b (bit 3 clear) or c,
// state 2 bit2 + bit0.
__device__ __forceinline__ float fold_tokens(float (&s)[8][2], int lane) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(s[j][m]), __float_as_uint(s[j + 4][m]), false, false);
      s[j][m] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(s[j][m]), __float_as_uint(s[j + 2][m]), false, false);
      s[j][m] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
      s[j][m] += dpp<0xb1>(s[j][m]);
      s[j][m] += dpp<0x4e>(s[j][m]);
    }
  const float even = lane & 1 ? s[0][1] : s[0][0], odd = lane & 1 ? s[1][1] : s[1][0];
  return lane & 2 ? odd : even;
}

// lam = mu + c gy in place of mu, and source = sum over states of b lam, of token J's rows in two channels: lane J of
// each row of 16 has b, lane 8 + J c (see read_out).
template <int J>
__device__ __forceinline__ void adjoints(const float (&rows)[kScanStates], const float (&gy)[2],
                                         float (&mu)[2][kScanStates], float (&source)[2]) {
#define SX_AT(N) " row_newbcast:%" N " row_mask:0xf bank_mask:0xf\n\t"
#define SX_LAM(G, M0, M1, M2, M3)                                                    \
  "v_fmac_f32_dpp %" M0 ", %10, %" G SX_AT("17") "v_fmac_f32_dpp %" M1 ", %11, %" G SX_AT("17") \
      "v_fmac_f32_dpp %" M2 ", %12, %" G SX_AT("17") "v_fmac_f32_dpp %" M3 ", %13, %" G SX_AT("17")
#define SX_SOURCE(O, M0, M1, M2, M3)                                                 \
  "v_mul_f32_dpp %" O ", %10, %" M0 SX_AT("16") "v_fmac_f32_dpp %" O ", %11, %" M1 SX_AT("16") \
      "v_fmac_f32_dpp %" O ", %12, %" M2 SX_AT("16") "v_fmac_f32_dpp %" O ", %13, %" M3 SX_AT("16")
  asm("s_nop 1\n\t" SX_LAM("14", "0", "1", "2", "3") SX_LAM("15", "4", "5", "6", "7")
          SX_SOURCE("8", "0", "1", "2", "3") SX_SOURCE("9", "4", "5", "6", "7")
      : "+v"(mu[0][0]), "+v"(mu[0][1]), "+v"(mu[0][2]), "+v"(mu[0][3]), "+v"(mu[1][0]), "+v"(mu[1][1]),
        "+v"(mu[1][2]), "+v"(mu[1][3]), "=&v"(source[0]), "=&v"(source[1])
      : "v"(rows[0]), "v"(rows[1]), "v"(rows[2]), "v"(rows[3]), "v"(gy[0]), "v"(gy[1]), "n"(J), "n"(J + 8));
#undef SX_SOURCE
#undef SX_LAM
#undef SX_AT
}

constexpr int kWide = kGradChannels;

template <int W>
struct alignas(16) GradLds {
  float dt[kMarkTokens][kWide], x[kMarkTokens][kWide], gy[kMarkTokens][kWide];
  float bias[kWide], skip[kWide];
  // the waves' parts of y, of sum b lam and of sum a q
  float y[W][kMarkTokens][kWide], source[W][kMarkTokens][kWide], decay[W][kMarkTokens][kWide];
};

// Two waves a SIMD, but where a thread has so many pieces of a span that the registers do not suffice for it (4 x 1024
// tokens of 2048 channels of 4 states in f32: 156 us, 306 with two).
constexpr int grad_waves_per_simd(bool bf16, int W) { return W == 1 || (W == 2 && !bf16) ? 1 : 2; }

template <bool BF, int W, Rows R, bool JOIN>
__global__ __launch_bounds__(kWave* W, grad_waves_per_simd(BF, W)) void grad_march(SsParams p) {
  using P = Piece<BF, 4>;
  using Raw = typename P::Raw;
  constexpr int M = kMarkTokens, kThreads = kWave * W;
  static_assert(M == 8, "the sums over lanes take eight tokens");
  constexpr int kPieces = M * kWide / 4, kPasses = (kPieces + kThreads - 1) / kThreads;
  constexpr int kStep = kThreads / (kWide / 4), kAtOnce = kStep < M ? kStep : M;
  constexpr bool WHOLE = R != Rows::Any;
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
  const int last = end - s0 - 1, spans = last >= 0 ? last / M + 1 : 0;
  const int q0 = tid / (kWide / 4), c0 = tid % (kWide / 4) * 4;
  const int c4 = R == Rows::Early ? min(c0, channels - 4) : c0, left = channels - c4;
  const bool mine = left > 0 && q0 < M, working = kThreads <= kPieces || q0 < M;
  float gskip[4] = {}, gbias[4] = {};
  for (int c = tid; c < kWide; c += kThreads) {
    l.bias[c] = c < channels && p.delta_bias ? p.delta_bias[d0 + c] : 0.0f;
    l.skip[c] = c < channels && p.skip ? p.skip[d0 + c] : 0.0f;
  }
  const TileReader<BF, R> xr(p.x, b, s0, d0, c4, channels), dr(p.delta, b, s0, d0, c4, channels);
  const TileReader<BF, R> zr(p.z, b, s0, d0, c4, channels), gr(p.go, b, s0, d0, c4, channels);
  const bool gated = p.z.p;
  struct Pieces {
    Raw x[kPasses], delta[kPasses], z[kPasses], go[kPasses];
  };
  const auto read = [&](int span, Pieces& to) {
    if (!working) return;
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
      const int q = q0 + k * kStep;
      to.x[k] = xr.read(p.x, span * M, q, last, left);
      to.delta[k] = dr.read(p.delta, span * M, q, last, left);
      to.go[k] = gr.read(p.go, span * M, q, last, left);
      if (gated) to.z[k] = zr.read(p.z, span * M, q, last, left);
    }
  };
  Pieces in;

  // lanes 0 .. 7 of each row of 16 have the tokens' rows of b, 8 .. 15 those of c
  RowReader<BF, false> rows(lane & M ? p.c : p.b, b, g, s0, n0, p.N);
  const int j8 = lane % M;

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
  for (int i = tid; i < M * kWide; i += kThreads) {
    (&l.dt[0][0])[i] = 0.0f;
    (&l.x[0][0])[i] = 0.0f;
    (&l.gy[0][0])[i] = 0.0f;
  }
  if (spans > 0) {
    read(spans - 1, in);
    rows.read((spans - 1) * M, j8, last);
    read_marks(spans - 1);
  }
  const bool grows = JOIN && (may_grow(p, rate[0]) || may_grow(p, rate[1]));
  __syncthreads();
  for (int span = spans - 1; span >= 0; --span) {
    const int t0 = span * M, room = last - t0;  // room: the last token of the span there is
    // dt, x and gy of the tokens
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
      const int q = q0 + k * kStep;
      if (!mine || (kPasses * kStep > M && q >= M)) continue;
      float x[4], v[4], gy[4], z[4];
      P::open(in.x[k], x);
      P::open(in.delta[k], v);
      P::open(in.go[k], gy);
      if (gated) {
        P::open(in.z[k], z);
#pragma unroll
        for (int i = 0; i < 4; ++i) gy[i] *= silu_of(z[i]);
      }
      lds_add<R>(l.bias, c4, v);
      if (p.softplus) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = softplus_of(v[i]);
      }
      if (!WHOLE || room < M - 1) {  // a token or channel that does not exist
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool there = q <= room && i < left;
          v[i] = there ? v[i] : 0.0f;
          x[i] = there ? x[i] : 0.0f;
          gy[i] = there ? gy[i] : 0.0f;
        }
      }
      lds_put<R>(l.dt[q], c4, v);
      lds_put<R>(l.x[q], c4, x);
      lds_put<R>(l.gy[q], c4, gy);
    }
    float rowv[kScanStates];  // of b and of c
    rows.open(t0, j8, last, M, rowv);
    // the states before each token, from the mark on; the decays are formed again on the way back, which their
    // registers are worth
    float hs[M + 1][2][kScanStates];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int i = 0; i < kScanStates; ++i) hs[0][c][i] = JOIN ? start[c][i] : marks[c][i];
      if constexpr (JOIN) carry_over(grows, mark_steps[c], rate[c], marks[c], hs[0][c]);
    }
    __syncthreads();
    each<2>([&](auto Q) {
      constexpr int j4 = 4 * decltype(Q)::value;
      float dx[4][2], es[4][2][kScanStates];
      each<4>([&](auto J) {
        constexpr int k = decltype(J)::value, j = j4 + k;
        const float2 dt = *reinterpret_cast<const float2*>(&l.dt[j][2 * lane]);
        const float2 x = *reinterpret_cast<const float2*>(&l.x[j][2 * lane]);
        dx[k][0] = dt.x * x.x;
        dx[k][1] = dt.y * x.y;
#pragma unroll
        for (int i = 0; i < kScanStates; ++i) {
          es[k][0][i] = exp2_of(dt.x * rate[0][i]);
          es[k][1][i] = exp2_of(dt.y * rate[1][i]);
        }
      });
      __builtin_amdgcn_sched_barrier(0);
      each<4>([&](auto J) {
        constexpr int k = decltype(J)::value, j = j4 + k;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int i = 0; i < kScanStates; ++i) hs[j + 1][c][i] = fmaf(es[k][c][i], hs[j][c][i], of_token<j>(rowv[i]) * dx[k][c]);
      });
      if (gated) {
        float y[2][4];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float after[4][kScanStates] = {
              {hs[j4 + 1][c][0], hs[j4 + 1][c][1], hs[j4 + 1][c][2], hs[j4 + 1][c][3]},
              {hs[j4 + 2][c][0], hs[j4 + 2][c][1], hs[j4 + 2][c][2], hs[j4 + 2][c][3]},
              {hs[j4 + 3][c][0], hs[j4 + 3][c][1], hs[j4 + 3][c][2], hs[j4 + 3][c][3]},
              {hs[j4 + 4][c][0], hs[j4 + 4][c][1], hs[j4 + 4][c][2], hs[j4 + 4][c][3]}};
          read_out<M + j4>(rowv, after, y[c]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<float2*>(&l.y[wave][j4 + k][2 * lane]) = make_float2(y[0][k], y[1][k]);
      }
    });
    float sums[M][2];
    Pieces now;
    each<M>([&](auto J) {
      constexpr int j = M - 1 - decltype(J)::value;
      // half of the states are done with: their registers take this span's operands once more, for the results, and
      // the next one's
      if constexpr (j == M / 2 - 1) {
        read(span, now);
        if (span > 0) {
          read(span - 1, in);
          rows.read(t0 - M, j8, last);
          read_marks(span - 1);
        }
      }
      const float2 dt2 = *reinterpret_cast<const float2*>(&l.dt[j][2 * lane]);
      const float2 x2 = *reinterpret_cast<const float2*>(&l.x[j][2 * lane]);
      const float2 gy2 = *reinterpret_cast<const float2*>(&l.gy[j][2 * lane]);
      const float dt[2] = {dt2.x, dt2.y}, x[2] = {x2.x, x2.y}, gy[2] = {gy2.x, gy2.y};
      float source[2], decay[2] = {0.0f, 0.0f}, shares[8];
      adjoints<j>(rowv, gy, mu, source);  // mu is lam here
#pragma unroll
      for (int i = 0; i < kScanStates; ++i) {
        shares[i] = fmaf(mu[1][i], dt[1] * x[1], mu[0][i] * (dt[0] * x[0]));
        shares[4 + i] = fmaf(gy[1], hs[j + 1][1][i], gy[0] * hs[j + 1][0][i]);
      }
      fold_token(shares, sums[j]);
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < kScanStates; ++i) {
          mu[c][i] *= exp2_of(dt[c] * rate[c][i]);
          const float q = mu[c][i] * hs[j][c][i];
          ga[c][i] = fmaf(dt[c], q, ga[c][i]);
          decay[c] = fmaf(rate[c][i], q, decay[c]);
        }
      *reinterpret_cast<float2*>(&l.source[wave][j][2 * lane]) = make_float2(source[0], source[1]);
      *reinterpret_cast<float2*>(&l.decay[wave][j][2 * lane]) = make_float2(decay[0], decay[1]);
      // no more than two tokens' operands at a time: with all eight's the wave's registers do not suffice
      if constexpr (j % 2 == 0) __builtin_amdgcn_sched_barrier(0);
    });
    {
      const float sum = fold_tokens(sums, lane);
      const int q = (lane >> 5 & 1) * 4 + (lane >> 4 & 1) * 2 + (lane >> 1 & 1), which = lane >> 3 & 1;
      const int n = n0 + (lane >> 2 & 1) * 2 + (lane & 1);
      if (q <= room)
        p.rows_partial[(((int64_t(b) * p.G + g) * p.T + s0 + t0 + q) * blocks + cb) * (8 * W) + which * 4 * W + n] = sum;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
      const int q = q0 + k * kStep;
      if (!mine || q > room || (kPasses * kStep > M && q >= M)) continue;
      float x[4], v[4], go[4], z[4], gx[4], gd[4], gz[4];
      P::open(now.x[k], x);
      P::open(now.delta[k], v);
      P::open(now.go[k], go);
      if (gated) P::open(now.z[k], z);
      float y[4], source[4] = {}, decay[4] = {}, dt[4] = {}, gy[4] = {}, skip[4] = {};
      lds_add<R>(l.bias, c4, v);
      lds_add<R>(l.skip, c4, skip);
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = skip[i] * x[i];
#pragma unroll
      for (int w = 0; w < W; ++w) {
        lds_add<R>(l.source[w][q], c4, source);
        lds_add<R>(l.decay[w][q], c4, decay);
      }
      if (gated) {
#pragma unroll
        for (int w = 0; w < W; ++w) lds_add<R>(l.y[w][q], c4, y);
      }
      lds_add<R>(l.dt[q], c4, dt);
      lds_add<R>(l.gy[q], c4, gy);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        gx[i] = fmaf(dt[i], source[i], skip[i] * gy[i]);
        gskip[i] = fmaf(gy[i], x[i], gskip[i]);
        // the rates stand times log2(e)
        gd[i] = fmaf(decay[i], 1.0f / kLog2e, x[i] * source[i]);
      }
      if (p.softplus) {  // once for the four, which are formed side by side so
#pragma unroll
        for (int i = 0; i < 4; ++i) gd[i] *= sigmoid_of(v[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) gbias[i] += gd[i];
      const int64_t o = (int64_t(b) * p.T + s0 + t0) * p.D + d0 + (int64_t(q) * p.D + c4);
      put_channels<BF, WHOLE>(p.gx, o, left, gx);
      put_channels<BF, WHOLE>(p.gdelta, o, left, gd);
      if (gated) {
#pragma unroll
        for (int i = 0; i < 4; ++i) gz[i] = go[i] * y[i] * silu_slope(z[i]);
        put_channels<BF, WHOLE>(p.gz, o, left, gz);
      }
    }
    // the next span's dt, x and gy go where these were read
    __syncthreads();
  }
  // tokens that do not exist
  if (mine) {
    const float none[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int t = max(end, s0) + q0; t < s1; t += kAtOnce) {
      const int64_t o = (int64_t(b) * p.T + t) * p.D + d0 + c4;
      put_channels<BF, WHOLE>(p.gx, o, left, none);
      put_channels<BF, WHOLE>(p.gdelta, o, left, none);
      if (gated) put_channels<BF, WHOLE>(p.gz, o, left, none);
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
  for (int c = tid; c < channels; c += kThreads) {
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

template <bool BF, int W, Rows R, bool JOIN>
hipError_t launch_join(const SsParams& p, hipStream_t stream) {
  const int64_t per_group = p.D / p.G;
  const int64_t units = int64_t(p.G) * p.B * p.segments;
  scan_march<BF, W, R, JOIN ? March::JoinedMarks : March::Marks>
      <<<unsigned((per_group + kChannels - 1) / kChannels * units), kWave * W, 0, stream>>>(p);
  if (JOIN) {
    const int64_t n = int64_t(p.B) * p.waves * p.D;
    carry<<<dim3(unsigned((n + 255) / 256), 2), 256, 0, stream>>>(p);
  }
  grad_march<BF, W, R, JOIN><<<unsigned((per_group + kWide - 1) / kWide * units), kWave * W, 0, stream>>>(p);
  return hipGetLastError();
}

template <bool BF, int W, Rows R>
hipError_t launch_waves(const SsParams& p, hipStream_t stream) {
  return p.segments > 1 ? launch_join<BF, W, R, true>(p, stream) : launch_join<BF, W, R, false>(p, stream);
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

}  // namespace

int selective_scan_grad_blocks(const SsParams& p) { return (p.D / p.G + kWide - 1) / kWide; }

hipError_t launch_selective_scan_backward(const SsParams& p, hipStream_t stream) {
  hipError_t err = hipSuccess;
  if (p.B > 0) {
    // both passes': workgroups of 64 and of 128 channels have four at least
    const Rows rows = scan_rows(p, true, kWide);
    const Rows r = rows == Rows::Any ? rows : scan_rows(p, true, kChannels);
    if (r == Rows::Whole) err = p.bf16 ? launch_states<true, Rows::Whole>(p, stream) : launch_states<false, Rows::Whole>(p, stream);
    else if (r == Rows::Early) err = p.bf16 ? launch_states<true, Rows::Early>(p, stream) : launch_states<false, Rows::Early>(p, stream);
    else err = p.bf16 ? launch_states<true, Rows::Any>(p, stream) : launch_states<false, Rows::Any>(p, stream);
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
