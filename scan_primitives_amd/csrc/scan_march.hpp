// scan_march.hpp: what the selective scan's kernels share: tiles of tokens and
// channels on their way into LDS, and rows of b and c as operands of every lane.
#pragma once

#include <utility>

#include "sx_state_space.hpp"

namespace sx {

// Lane j of each row of 16 lanes holds token j's value; this is token J's, in every lane. The compiler joins it
// with the instruction that takes it (a DPP operand), so it costs nothing.
template <int J>
__device__ __forceinline__ float of_token(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x150 + J, 0xf, 0xf, true));
}

// f(integral_constant<int, 0>) ... f(integral_constant<int, N - 1>).
template <int N, typename F>
__device__ __forceinline__ void each(F&& f) {
  [&]<int... I>(std::integer_sequence<int, I...>) { (f(std::integral_constant<int, I>{}), ...); }
  (std::make_integer_sequence<int, N>{});
}

// Four channels of one token, an element at a time: those behind the last (`left` of them exist) read as the last.
template <bool BF>
__device__ __forceinline__ typename Piece<BF, 4>::Raw four_channels(const TokenView& v, int64_t at, int left) {
  const auto* p = static_cast<const typename Piece<BF, 4>::E*>(v.p) + at;
  return Piece<BF, 4>::of(p[0], p[min(1, left - 1) * v.sd], p[min(2, left - 1) * v.sd], p[min(3, left - 1) * v.sd]);
}

// Four channels of a contiguous result. WIDE: all exist; else `left` of them.
template <bool BF, bool WIDE>
__device__ __forceinline__ void put_channels(void* out, int64_t at, int left, const float (&v)[4]) {
  using P = Piece<BF, 4>;
  using E = typename P::E;
  E* p = static_cast<E*>(out) + at;
  if constexpr (WIDE) {
    P::store(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) Piece<BF, 1>::store(p + i, {v[i]});
  }
}

// A rate for exp2: a log2(e), never infinite, for a step of zero (a token that does not exist has one) leaves the state
// as it is.
__device__ __forceinline__ float rate_of(float a) {
  constexpr float kMost = 3.4028234663852886e38f;
  const float r = a * kLog2e;
  return r < -kMost ? -kMost : r > kMost ? kMost : r;
}

// a[d, n0 .. n0 + 3] for exp2, zero where there are none.
__device__ __forceinline__ void rates(const float* a, int64_t d, int n0, int N, bool is, float (&r)[kScanStates]) {
#pragma unroll
  for (int i = 0; i < kScanStates; ++i) r[i] = is && n0 + i < N ? rate_of(a[d * N + n0 + i]) : 0.0f;
}

// Whether a wave's states may grow: a positive rate, or steps of any sign. It waits for the rates: asked for behind the
// first loads that do not.
__device__ __forceinline__ bool may_grow(const SsParams& p, const float (&rate)[kScanStates]) {
  bool any = !p.softplus;
#pragma unroll
  for (int i = 0; i < kScanStates; ++i) any |= !(rate[i] <= 0.0f);
  return __any(any);
}

// exp2(e) v, where exp2(e) alone may lie outside f32's range: 2^300 turns the least value there is to infinity.
__device__ __forceinline__ float times_exp2(float v, float e) {
  const float in = e > 300.0f ? 300.0f : e < -300.0f ? -300.0f : e, whole = floorf(in);
  return ldexpf(v * exp2_of(in - whole), int(whole));
}

// States (or adjoints) over tokens whose dt add up to `steps`: exp2(steps rate) h + own in place of h. Where states
// grow, the decay alone may be infinite while its product is not: a zero stays zero, a small state comes out as token
// by token.
constexpr float kMostExponent = 127.0f;
__device__ __forceinline__ void carry_over(bool grows, float steps, const float (&rate)[kScanStates], const f32x4& own,
                                           float (&h)[kScanStates]) {
  if (!grows) {
#pragma unroll
    for (int i = 0; i < kScanStates; ++i) h[i] = fmaf(exp2_of(steps * rate[i]), h[i], own[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kScanStates; ++i) {
      const float e = steps * rate[i];
      h[i] = e <= kMostExponent ? fmaf(exp2_of(e), h[i], own[i]) : times_exp2(h[i], e) + own[i];
    }
  }
}

// h[n0 .. n0 + 3] of one channel in [.., D, N].
__device__ __forceinline__ void read_states(const float* p, int64_t row, int n0, int N, bool is,
                                            float (&h)[kScanStates]) {
#pragma unroll
  for (int i = 0; i < kScanStates; ++i) h[i] = p && is && n0 + i < N ? p[row * N + n0 + i] : 0.0f;
}
__device__ __forceinline__ void write_states(float* p, int64_t row, int n0, int N, bool is,
                                             const float (&h)[kScanStates]) {
#pragma unroll
  for (int i = 0; i < kScanStates; ++i)
    if (is && n0 + i < N) p[row * N + n0 + i] = h[i];
}

// The four states of channel d in an array [..][waves][D][4].
__device__ __forceinline__ int64_t packed_at(const SsParams& p, int64_t row, int wave, int64_t d) {
  return ((row * p.waves + wave) * p.D + d) * kScanStates;
}

// ---------------------------------------------------------------- the march

constexpr int kTile = 16, kChannels = 64;  // tokens and channels of a workgroup's tile

// What a march is for: the result; the state and the sum of dt of segments on their own; the marks of the
// gradient; and those of segments on their own, with their states, sums of dt and adjoints.
enum class March { Out, Segments, Marks, JoinedMarks };

// How x, delta, z and out are read and written, four channels of a token a thread: an element at a time; four next
// to each other; or these at any channel, where the last of a workgroup start early enough to be whole and both
// threads that have a channel do the same to it.
enum class Rows { Any, Whole, Early };

// Four values of a row of LDS, from channel c on (a multiple of four but for Early).
template <Rows R>
__device__ __forceinline__ void lds_put(float* row, int c, const float (&v)[4]) {
  if constexpr (R == Rows::Early) {
#pragma unroll
    for (int i = 0; i < 4; ++i) row[c + i] = v[i];
  } else {
    *reinterpret_cast<f32x4*>(row + c) = f32x4{v[0], v[1], v[2], v[3]};
  }
}
template <Rows R>
__device__ __forceinline__ void lds_add(const float* row, int c, float (&v)[4]) {
  if constexpr (R == Rows::Early) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += row[c + i];
  } else {
    const f32x4 o = *reinterpret_cast<const f32x4*>(row + c);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += o[i];
  }
}

// One array's pieces of a tile. But for Any, by 32-bit offsets from the tile's start.
template <bool BF, Rows R>
struct TileReader {
  using P = Piece<BF, 4>;
  using E = typename P::E;
  const E* base;      // the segment's first token, the workgroup's first channel
  uint32_t off, row;  // of the thread's piece, and of a token
  int64_t at, st;     // Any
  __device__ __forceinline__ TileReader(const TokenView& v, int b, int s0, int d0, int c4, int channels) {
    if constexpr (R != Rows::Any) {
      base = static_cast<const E*>(v.p) + int64_t(b) * v.sb + int64_t(s0) * v.st + d0;
      row = uint32_t(v.st);
      off = uint32_t(min(c4, channels - 4));  // threads without channels read the last again
    } else {
      at = int64_t(b) * v.sb + int64_t(s0) * v.st + int64_t(d0 + c4) * v.sd;
      st = v.st;
    }
  }
  // the piece of token `q` from token `t` of the segment on; `last`: the last token of the segment there is
  __device__ __forceinline__ typename P::Raw read(const TokenView& v, int t, int q, int last, int left) const {
    if constexpr (R != Rows::Any) {
      const E* from = base + int64_t(t) * row;
      return P::load(from + (off + uint32_t(min(q, last - t)) * row));
    } else {
      return left > 0 && t + q <= last ? four_channels<BF>(v, at + int64_t(t + q) * st, left) : P::zero();
    }
  }
};

// A token's row of b or c for the wave: lane j of each `count` lanes has token j's states n0 .. n0 + 3, four at once
// where they lie next to each other. NEAR: by a 32-bit offset from the tile's first token, the same view in all lanes.
template <bool BF, bool NEAR>
struct RowReader {
  using P4 = Piece<BF, 4>;
  using E = typename P4::E;
  const E* base;
  int64_t st, sn;
  int n0, left;  // left: how many states there are from n0 on
  bool whole;
  typename P4::Raw four;
  E one[kScanStates];
  __device__ __forceinline__ RowReader(const RowView& v, int b, int g, int s0, int n, int N)
      : st(v.st), sn(v.sn), n0(n), left(N - n), whole(v.sn == 1 && N % kScanStates == 0) {
    base = static_cast<const E*>(v.p) + int64_t(b) * v.sb + int64_t(g) * v.sg + int64_t(s0) * v.st;
    if (left > 0) base += n0 * sn;  // a wave without states reads the first
  }
  // token `q` from token `t` of the segment on
  __device__ __forceinline__ void read(int t, int q, int last) {
    const E* from = NEAR ? base + int64_t(t) * st + uint32_t(min(q, last - t)) * uint32_t(st)
                         : base + int64_t(t + min(q, last - t)) * st;
    if (whole) {
      four = P4::load(from);
    } else {
#pragma unroll
      for (int i = 0; i < kScanStates; ++i) one[i] = from[min(i, max(left - 1, 0)) * sn];
    }
  }
  // zero where a token or state does not exist: the memory may hold anything
  __device__ __forceinline__ void open(int t, int q, int last, int count, float (&f)[kScanStates]) const {
    if (whole) {
      P4::open(four, f);
    } else {
#pragma unroll
      for (int i = 0; i < kScanStates; ++i) {
        float v[1];
        Piece<BF, 1>::open(one[i], v);
        f[i] = v[0];
      }
    }
    if (left < kScanStates) {
#pragma unroll
      for (int i = 0; i < kScanStates; ++i) f[i] = i < left ? f[i] : 0.0f;
    }
    if (last - t < count - 1) {
#pragma unroll
      for (int i = 0; i < kScanStates; ++i) f[i] = q <= last - t ? f[i] : 0.0f;
    }
  }
};

// y[k] = sum over i of token J + k's c[i] h[k][i], for four tokens: the products take c by DPP, which the compiler
// does only for products without a sum. The wait is for a c that was written just before.
template <int J>
__device__ __forceinline__ void read_out(const float (&c)[kScanStates], const float (&h)[4][kScanStates],
                                         float (&y)[4]) {
#define SX_ROW(N) " row_newbcast:%" N " row_mask:0xf bank_mask:0xf\n\t"
#define SX_TOKEN(O, H0, H1, H2, H3, T)                                        \
  "v_mul_f32_dpp %" O ", %4, %" H0 SX_ROW(T) "v_fmac_f32_dpp %" O ", %5, %" H1 SX_ROW(T) \
      "v_fmac_f32_dpp %" O ", %6, %" H2 SX_ROW(T) "v_fmac_f32_dpp %" O ", %7, %" H3 SX_ROW(T)
  asm("s_nop 1\n\t" SX_TOKEN("0", "8", "9", "10", "11", "24") SX_TOKEN("1", "12", "13", "14", "15", "25")
          SX_TOKEN("2", "16", "17", "18", "19", "26") SX_TOKEN("3", "20", "21", "22", "23", "27")
      : "=&v"(y[0]), "=&v"(y[1]), "=&v"(y[2]), "=&v"(y[3])
      : "v"(c[0]), "v"(c[1]), "v"(c[2]), "v"(c[3]), "v"(h[0][0]), "v"(h[0][1]), "v"(h[0][2]), "v"(h[0][3]),
        "v"(h[1][0]), "v"(h[1][1]), "v"(h[1][2]), "v"(h[1][3]), "v"(h[2][0]), "v"(h[2][1]), "v"(h[2][2]),
        "v"(h[2][3]), "v"(h[3][0]), "v"(h[3][1]), "v"(h[3][2]), "v"(h[3][3]), "n"(J), "n"(J + 1), "n"(J + 2),
        "n"(J + 3));
#undef SX_TOKEN
#undef SX_ROW
}

// u[k] = token J + k's b[i] times dx[k], for four tokens, in the same way.
template <int J>
__device__ __forceinline__ void sources(const float (&b)[kScanStates], const float (&dx)[4],
                                        float (&u)[4][kScanStates]) {
#define SX_ROW(N) " row_newbcast:%" N " row_mask:0xf bank_mask:0xf\n\t"
#define SX_TOKEN(U0, U1, U2, U3, D, T)                                                  \
  "v_mul_f32_dpp %" U0 ", %16, %" D SX_ROW(T) "v_mul_f32_dpp %" U1 ", %17, %" D SX_ROW(T) \
      "v_mul_f32_dpp %" U2 ", %18, %" D SX_ROW(T) "v_mul_f32_dpp %" U3 ", %19, %" D SX_ROW(T)
  asm("s_nop 1\n\t" SX_TOKEN("0", "1", "2", "3", "20", "24") SX_TOKEN("4", "5", "6", "7", "21", "25")
          SX_TOKEN("8", "9", "10", "11", "22", "26") SX_TOKEN("12", "13", "14", "15", "23", "27")
      : "=&v"(u[0][0]), "=&v"(u[0][1]), "=&v"(u[0][2]), "=&v"(u[0][3]), "=&v"(u[1][0]), "=&v"(u[1][1]),
        "=&v"(u[1][2]), "=&v"(u[1][3]), "=&v"(u[2][0]), "=&v"(u[2][1]), "=&v"(u[2][2]), "=&v"(u[2][3]),
        "=&v"(u[3][0]), "=&v"(u[3][1]), "=&v"(u[3][2]), "=&v"(u[3][3])
      : "v"(b[0]), "v"(b[1]), "v"(b[2]), "v"(b[3]), "v"(dx[0]), "v"(dx[1]), "v"(dx[2]), "v"(dx[3]), "n"(J), "n"(J + 1),
        "n"(J + 2), "n"(J + 3));
#undef SX_TOKEN
#undef SX_ROW
}

// A wave's adjoints of its segment once more, by the exponents' sums and an element at a time: the sum over the tokens
// of c gy times the decays up to each. What it needs is formed again from the block's number, and all of it behind the
// march: in the march the same costs every call registers (4 x 2048 tokens of 2048 channels in bf16: 395 us, 354).
template <bool BF>
__device__ __forceinline__ void adjoint_again(const SsParams& p) {
  using E = typename Piece<BF, 1>::E;
  uint32_t at = blockIdx.x;
  asm volatile("" : "+s"(at));  // nothing of it is kept over the march
  const int per_group = p.D / p.G, blocks = (per_group + kChannels - 1) / kChannels;
  const int cb = int(at % uint32_t(blocks));
  at /= uint32_t(blocks);
  const int g = int(at % uint32_t(p.G));
  at /= uint32_t(p.G);
  const int64_t b = at % uint32_t(p.B), seg = at / uint32_t(p.B);
  const int lane = int(threadIdx.x) % kWave, wave = int(threadIdx.x) / kWave, n0 = wave * kScanStates;
  if (lane >= min(kChannels, per_group - cb * kChannels)) return;
  const int64_t d = int64_t(g) * per_group + cb * kChannels + lane;
  const int s0 = int(seg) * p.seg_tokens, end = min(min(s0 + p.seg_tokens, p.T), row_length(p.lengths, int(b), p.T));
  const auto element = [](const void* from, int64_t i) {
    float v[1];
    Piece<BF, 1>::open(static_cast<const E*>(from)[i], v);
    return v[0];
  };
  const auto token = [&](const TokenView& v, int64_t t) { return element(v.p, b * v.sb + t * v.st + d * v.sd); };
  float rate[kScanStates], adj[kScanStates] = {}, steps = 0.0f;
  rates(p.a, d, n0, p.N, true, rate);
  const float bias = p.delta_bias ? p.delta_bias[d] : 0.0f;
#pragma unroll 1
  for (int t = s0; t < end; ++t) {
    const float v = token(p.delta, t) + bias;
    float gy = token(p.go, t);
    if (p.z.p) gy *= silu_of(token(p.z, t));
    steps += p.softplus ? softplus_of(v) : v;
#pragma unroll
    for (int i = 0; i < kScanStates; ++i) {
      if (n0 + i >= p.N) break;
      const float c = element(p.c.p, b * p.c.sb + int64_t(t) * p.c.st + g * p.c.sg + (n0 + i) * p.c.sn);
      adj[i] += times_exp2(c * gy, steps * rate[i]);
    }
  }
  *reinterpret_cast<f32x4*>(p.seg_adjoint + packed_at(p, seg * p.B + b, wave, d)) = f32x4{adj[0], adj[1], adj[2], adj[3]};
}

template <int W, March KIND>
struct alignas(16) MarchLds {
  float dt[2][kTile][kChannels];
  float dx[2][kTile][kChannels];
  float y[KIND == March::JoinedMarks ? 2 : 1]                               // Out: the waves' parts of y;
         [KIND == March::Out ? W : 1][KIND == March::Out || KIND == March::JoinedMarks ? kTile : 1]  // JoinedMarks: gy
         [kChannels];
};

// Waves a SIMD that the registers are to leave (of few waves, whose threads have more pieces of a tile each, LDS does
// not hold more).
constexpr int march_waves_per_simd(int W) { return W == 1 ? 2 : W == 2 ? 3 : 4; }

template <bool BF, int W, Rows R, March KIND>
__global__ __launch_bounds__(kWave* W, march_waves_per_simd(W)) void scan_march(SsParams p) {
  using P = Piece<BF, 4>;
  using Raw = typename P::Raw;
  constexpr bool OUT = KIND == March::Out, MARK = KIND == March::Marks || KIND == March::JoinedMarks,
                 ADJOINT = KIND == March::JoinedMarks, SUMS = KIND == March::Segments || ADJOINT;
  constexpr int kPieces = kTile * kChannels / 4, kThreads = kWave * W;
  constexpr int kPasses = (kPieces + kThreads - 1) / kThreads, kStep = kThreads / (kChannels / 4);
  constexpr int kAtOnce = kStep < kTile ? kStep : kTile;
  __shared__ MarchLds<W, KIND> l;
  __shared__ int back;  // JoinedMarks without softplus: a step is negative
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
  const int last = end - s0 - 1, tiles = last >= 0 ? last / kTile + 1 : 0;

  // this thread's pieces of a tile: token q0 + pass * step, channels c4 .. c4 + 3
  const int q0 = tid / (kChannels / 4), c0 = tid % (kChannels / 4) * 4;
  const int c4 = R == Rows::Early ? min(c0, channels - 4) : c0, left = channels - c4;
  const bool mine = left > 0 && q0 < kTile;
  const bool working = kThreads <= kPieces || q0 < kTile;  // uniform: more than four waves share a tile's pieces
  float bias[4], skip[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool is = mine && i < left;
    bias[i] = is && p.delta_bias ? p.delta_bias[d0 + c4 + i] : 0.0f;
    skip[i] = OUT && is && p.skip ? p.skip[d0 + c4 + i] : 0.0f;
  }
  const TileReader<BF, R> xr(p.x, b, s0, d0, c4, channels), dr(p.delta, b, s0, d0, c4, channels);
  const TileReader<BF, R> zr(p.z, b, s0, d0, c4, channels), gr(p.go, b, s0, d0, c4, channels);
  const bool gated = (OUT || ADJOINT) && p.z.p;
  Raw xin[kPasses], din[kPasses], gin[kPasses], zin[kPasses], xout[kPasses];
  const auto read = [&](int tile) {
    if (!working) return;
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
      const int q = q0 + k * kStep;
      xin[k] = xr.read(p.x, tile * kTile, q, last, left);
      din[k] = dr.read(p.delta, tile * kTile, q, last, left);
      if (ADJOINT) gin[k] = gr.read(p.go, tile * kTile, q, last, left);
      if (ADJOINT && gated) zin[k] = zr.read(p.z, tile * kTile, q, last, left);
    }
  };
  const auto convert = [&](int tile) {
    if (!working) return;
    const int room = last - tile * kTile;  // the last token of the tile there is
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
      const int q = q0 + k * kStep;
      if (kPasses * kStep > kTile && q >= kTile) continue;
      float x[4], v[4];
      P::open(xin[k], x);
      P::open(din[k], v);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += bias[i];
      if (p.softplus) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = softplus_of(v[i]);
      }
      if (room < kTile - 1) {  // a token that does not exist changes no state
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = q <= room ? v[i] : 0.0f;
          x[i] = q <= room ? x[i] : 0.0f;
        }
      }
      if (ADJOINT && !p.softplus) {
        if (fminf(fminf(v[0], v[1]), fminf(v[2], v[3])) < 0.0f) back = 1;
      }
      lds_put<R>(l.dt[tile & 1][q], c4, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] *= v[i];
      lds_put<R>(l.dx[tile & 1][q], c4, x);
      if constexpr (ADJOINT) {
        float gy[4], z[4];
        P::open(gin[k], gy);
        if (gated) {
          P::open(zin[k], z);
#pragma unroll
          for (int i = 0; i < 4; ++i) gy[i] *= silu_of(z[i]);
        }
        if (room < kTile - 1) {
#pragma unroll
          for (int i = 0; i < 4; ++i) gy[i] = q <= room ? gy[i] : 0.0f;
        }
        lds_put<R>(l.y[tile & 1][0][q], c4, gy);
      }
    }
  };
  RowReader<BF, R != Rows::Any> brow(p.b, b, g, s0, n0, p.N), crow(p.c, b, g, s0, n0, p.N);
  const int j16 = lane % kTile;
  const auto read_rows = [&](int tile) {
    brow.read(tile * kTile, j16, last);
    if (OUT || ADJOINT) crow.read(tile * kTile, j16, last);
  };

  const bool is = lane < channels;
  const int64_t d = d0 + lane;
  float rate[kScanStates], h[kScanStates], through[kScanStates], adj[kScanStates], steps = 0.0f;
  rates(p.a, d, n0, p.N, is, rate);
  read_states(OUT || KIND == March::Marks ? p.initial : nullptr, int64_t(b) * p.D + d, n0, p.N, is, h);
  if constexpr (OUT) {
    constexpr int A = 8;  // segments read ahead of the chain
    for (int m = 0; m < seg; m += A) {
      f32x4 own[A];
      float sum[A];
#pragma unroll
      for (int k = 0; k < A; ++k) {
        const int64_t row = int64_t(min(m + k, seg - 1)) * p.B + b;
        own[k] = is ? *reinterpret_cast<const f32x4*>(p.seg_state + packed_at(p, row, wave, d)) : zero4();
        sum[k] = is ? p.seg_steps[row * p.D + d] : 0.0f;
      }
      // one look at all of them: few have grown so far
      bool apart = false;
      if (may_grow(p, rate)) {
        float most = 0.0f;
#pragma unroll
        for (int k = 0; k < A; ++k)
#pragma unroll
          for (int i = 0; i < kScanStates; ++i) most = fmaxf(most, sum[k] * rate[i]);
        apart = __any(most > kMostExponent);
      }
      const auto chain = [&](auto grown) {
#pragma unroll
        for (int k = 0; k < A; ++k) {
          if (m + k >= seg) break;
          carry_over(grown, sum[k], rate, own[k], h);
        }
      };
      if (apart) chain(std::true_type());
      else chain(std::false_type());
    }
  }
#pragma unroll
  for (int i = 0; i < kScanStates; ++i) {
    through[i] = 1.0f;
    adj[i] = 0.0f;
  }
  const auto mark = [&](int t, float before) {
    if (!is) return;
    const int64_t row = int64_t(b) * p.row_marks + t / kMarkTokens;
    *reinterpret_cast<f32x4*>(p.marks + packed_at(p, row, wave, d)) = f32x4{h[0], h[1], h[2], h[3]};
    if (ADJOINT && wave == 0) p.mark_steps[row * p.D + d] = before;
  };

  if (ADJOINT && !p.softplus) {
    if (tid == 0) back = 0;
    __syncthreads();
  }
  if (tiles > 0) {
    read(0);
    read_rows(0);
    convert(0);
    if (tiles > 1) read(1);
  }
  __syncthreads();
  for (int tile = 0; tile < tiles; ++tile) {
    const int buf = tile & 1, t0 = tile * kTile;
    if (OUT && working) {
#pragma unroll
      for (int k = 0; k < kPasses; ++k) {
        const int q = q0 + k * kStep;
        xout[k] = xr.read(p.x, t0, q, last, left);
        if (gated) zin[k] = zr.read(p.z, t0, q, last, left);
      }
    }
    float bv[kScanStates], cv[kScanStates];
    brow.open(t0, j16, last, kTile, bv);
    if (OUT || ADJOINT) crow.open(t0, j16, last, kTile, cv);
    if (tile + 1 < tiles) read_rows(tile + 1);
    // four tokens at a time, the next four's dt and dt x on their way: all their exponentials first, which a
    // chain of one state after the other would wait for
    float dt[4], dx[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      dt[k] = l.dt[buf][k][lane];
      dx[k] = l.dx[buf][k][lane];
    }
    each<kTile / 4>([&](auto Q) {
      constexpr int j4 = 4 * decltype(Q)::value;
      float e[4][kScanStates], u[4][kScanStates], gy[4], read[4][kScanStates], before = 0.0f;  // read: c gy
      each<4>([&](auto J) {
        constexpr int k = decltype(J)::value;
#pragma unroll
        for (int i = 0; i < kScanStates; ++i) e[k][i] = exp2_of(dt[k] * rate[i]);
      });
      sources<j4>(bv, dx, u);
      if constexpr (SUMS) {
        before = steps;
#pragma unroll
        for (int k = 0; k < 4; ++k) steps += dt[k];
      }
      if constexpr (j4 + 4 < kTile) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          dt[k] = l.dt[buf][j4 + 4 + k][lane];
          dx[k] = l.dx[buf][j4 + 4 + k][lane];
        }
      }
      if constexpr (ADJOINT) {
#pragma unroll
        for (int k = 0; k < 4; ++k) gy[k] = l.y[buf][0][j4 + k][lane];
        sources<j4>(cv, gy, read);
      }
      __builtin_amdgcn_sched_barrier(0);
      if (MARK && j4 == 0) mark(s0 + t0, before);
      if (MARK && j4 == kMarkTokens && kMarkTokens <= last - t0) mark(s0 + t0 + kMarkTokens, before);
      float hs[4][kScanStates], y[4];
      each<4>([&](auto J) {
        constexpr int k = decltype(J)::value;
#pragma unroll
        for (int i = 0; i < kScanStates; ++i) {
          h[i] = fmaf(e[k][i], h[i], u[k][i]);
          if constexpr (OUT) hs[k][i] = h[i];
          if constexpr (ADJOINT) {
            through[i] *= e[k][i];
            adj[i] = fmaf(through[i], read[k][i], adj[i]);
          }
        }
      });
      if constexpr (OUT) {
        read_out<j4>(cv, hs, y);
#pragma unroll
        for (int k = 0; k < 4; ++k) l.y[0][wave][j4 + k][lane] = y[k];
      }
      // the states are here now: the compiler would form them behind what follows, apart from the rows of b and c,
      // which then take a register and a move each
#pragma unroll
      for (int i = 0; i < kScanStates; ++i) {
        asm volatile("" : "+v"(h[i]));
        if constexpr (ADJOINT) asm volatile("" : "+v"(through[i]), "+v"(adj[i]));
      }
      __builtin_amdgcn_sched_barrier(0);
    });
    if (tile + 1 < tiles) {
      convert(tile + 1);
      if (tile + 2 < tiles) read(tile + 2);
    }
    __syncthreads();
    if (OUT && working) {
#pragma unroll
      for (int k = 0; k < kPasses; ++k) {
        const int q = q0 + k * kStep;
        if (kPasses * kStep > kTile && q >= kTile) continue;
        float x[4], y[4];
        P::open(xout[k], x);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = skip[i] * x[i];
#pragma unroll
        for (int w = 0; w < (OUT ? W : 1); ++w) lds_add<R>(l.y[0][w][q], c4, y);
        if (gated) {
          float z[4];
          P::open(zin[k], z);
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] *= silu_of(z[i]);
        }
        if (left > 0 && t0 + q <= last)
          put_channels<BF, R != Rows::Any>(p.out, (int64_t(b) * p.T + s0 + t0) * p.D + d0 + (uint32_t(q) * uint32_t(p.D) + c4),
                                 left, y);
      }
    }
    if (OUT) __syncthreads();  // the next tile's parts go where these were read: two buffers would cost a fourth wave
  }
  if constexpr (OUT) {
    if (mine) {
      const float none[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int t = max(end, s0) + q0; t < s1; t += kAtOnce)
        put_channels<BF, R != Rows::Any>(p.out, (int64_t(b) * p.T + t) * p.D + d0 + c4, left, none);
    }
    if (p.last && seg == p.segments - 1) write_states(p.last, int64_t(b) * p.D + d, n0, p.N, is, h);
  }
  if (SUMS && is) {
    const int64_t row = int64_t(seg) * p.B + b;
    *reinterpret_cast<f32x4*>(p.seg_state + packed_at(p, row, wave, d)) = f32x4{h[0], h[1], h[2], h[3]};
    if (ADJOINT)
      *reinterpret_cast<f32x4*>(p.seg_adjoint + packed_at(p, row, wave, d)) = f32x4{adj[0], adj[1], adj[2], adj[3]};
    if (wave == 0) p.seg_steps[row * p.D + d] = steps;
  }
  if constexpr (ADJOINT) {
    // Where states grow, the decays' product may have left f32's range, and with steps of both signs come back: what
    // it multiplied may be zero or small. (Lanes without a channel hold what LDS held.)
    bool lost = !p.softplus && back;
#pragma unroll
    for (int i = 0; i < kScanStates; ++i) lost |= !(through[i] < INFINITY);
    if (__any(lost && is)) adjoint_again<BF>(p);
  }
}

// How a call's arrays can be read: 8192 tokens of 4096 channels of 16 states in bf16 take 247 us by fours, of 4095
// channels 258 (Early), of 4096 that lie two apart 324 by elements (one operand over and over).
inline Rows scan_rows(const SsParams& p, bool gradient, int channels) {
  const int64_t most = int64_t(1) << 24, per_group = p.D / p.G;
  bool unit = per_group % channels == 0 || per_group % channels >= 4;  // a workgroup has four channels at least
  for (const TokenView* v : {&p.x, &p.delta, &p.z, gradient ? &p.go : &p.x})
    unit = unit && (!v->p || (v->sd == 1 && v->st >= 0 && v->st < most));
  for (const RowView* v : {&p.b, &p.c}) unit = unit && v->st >= 0 && v->st < most;
  return !unit ? Rows::Any : per_group % 4 == 0 ? Rows::Whole : Rows::Early;
}

}  // namespace sx
