// decay_attention.hip: linear attention with a decay for each head, its
// gradient and its single-token form.
//
//   S[t] = exp(g[t]) S[t-1] + k[t] v[t]^T,   o[t] = scale S[t]^T q[t]
//
// Prompts and gradients run as marches (DaMarch in sx_attention.hpp) over
// chunks of C tokens. With G the running sum of g inside a chunk, and S the
// state the chunk is entered with,
//   out_i = scale (exp(G_i) S^T x_i + sum_{j <= i} exp(G_i - G_j) (x_i . y_j) z_j)
//   S    <- exp(G_C) S + sum_j exp(G_C - G_j) y_j z_j^T
// Every exponent is the log decay between two tokens, never its two halves
// apart, so nothing overflows however strong the decay, and a decay of zero
// (g = -inf) cuts exactly. A workgroup keeps S in its accumulators: the wave
// layout of a 16x16 MFMA result (four rows of one column a lane) is the layout
// of an operand contracted over those rows, so S feeds x S without leaving the
// registers.
//
// Long sequences with few heads are split into segments: a first pass forms
// each segment's state from its own tokens, a carry joins them, and the second
// pass marches all segments at once from their true states.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "ms_mfma.hpp"
#include "sx_attention.hpp"
#include "sx_common.hpp"

namespace sx {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
// Log decays are taken into [-200, 200]: exp(-200) is zero and exp(200) infinite in
// f32, so the results are those of the whole range, and -inf leaves no inf - inf.
constexpr float kMostLog = 200.0f;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

template <bool BF>
struct Op;

// bf16 operands. A Frag is four values along the contraction at one row (or
// column), a Pair two of them (one per 16-wide tile): v_mfma_f32_16x16x32_bf16
// contracts both tiles at once. Its own order of the 32 does not matter, as
// both operands use the same one.
template <>
struct Op<true> {
  using E = uint16_t;
  using Pair = uint4;
  static constexpr int C = 64;      // tokens a chunk
  static constexpr int kPiece = 8;  // elements of a 16-byte piece
  static constexpr int kPad = 8;
  // f32 values enter a product as bf16 parts: three carry all 24 bits, two carry
  // 16, enough where the result is rounded to bf16 (8 bits) on store.
  static constexpr int kState = 3;
  static constexpr int kScore = 2;
  static __device__ __forceinline__ f32x4 mma(Pair a, Pair b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  }
  // NP parts of eight f32 values (truncated to bf16 one after the other; the last
  // of three is what is left, exactly).
  template <int NP>
  static __device__ __forceinline__ void split(f32x4 a, f32x4 b, Pair (&out)[NP]) {
    float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      uint32_t u[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        u[i] = __float_as_uint(v[i]);
        if (p + 1 < NP) v[i] -= __uint_as_float(u[i] & 0xffff0000u);
      }
      out[p] = make_uint4(upper_halves(u[0], u[1]), upper_halves(u[2], u[3]), upper_halves(u[4], u[5]),
                          upper_halves(u[6], u[7]));
    }
  }
  // rows 16-wide tiles t and t + 1 of the contraction, columns 4g.. of each
  static __device__ __forceinline__ Pair row_pair(const E* row, int g) {
    const uint2 a = *reinterpret_cast<const uint2*>(row + 4 * g);
    const uint2 b = *reinterpret_cast<const uint2*>(row + 16 + 4 * g);
    return make_uint4(a.x, a.y, b.x, b.y);
  }
  // the same 32 columns in the other order both operands may share: eight in a row a lane
  static __device__ __forceinline__ Pair row_pair_any(const E* row, int g) {
    return *reinterpret_cast<const uint4*>(row + 8 * g);
  }
  // contraction over rows j0 + 4g .. of tile j0 and of tile j0 + 16, at column col0 + c
  static __device__ __forceinline__ Pair column_pair(const E* tile, int stride, int j0, int col0, int g, int c) {
    typedef s16x4_t __attribute__((address_space(3))) * lds4;
    const E* p = tile + (j0 + 4 * g + (c >> 2)) * stride + col0 + 4 * (c & 3);
    const uint2 a = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(p)));
    const uint2 b = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(p + 16 * stride)));
    return make_uint4(a.x, a.y, b.x, b.y);
  }
  static __device__ __forceinline__ f32x4 low(Pair a) {
    return f32x4{__uint_as_float(a.x << 16), __uint_as_float(a.x & 0xffff0000u), __uint_as_float(a.y << 16),
                 __uint_as_float(a.y & 0xffff0000u)};
  }
  static __device__ __forceinline__ f32x4 high(Pair a) { return low(make_uint4(a.z, a.w, 0, 0)); }
  static __device__ __forceinline__ f32x4 four(const E* p) {
    const uint2 a = *reinterpret_cast<const uint2*>(p);
    return low(make_uint4(a.x, a.y, 0, 0));
  }
  static __device__ __forceinline__ float one(E v) { return bf16_to_f32(v); }
  static __device__ __forceinline__ bool finite(uint4 v) {
    auto bad = [](uint32_t u) { return (u & 0x7f800000u) == 0x7f800000u || (u & 0x7f80u) == 0x7f80u; };
    return !(bad(v.x) || bad(v.y) || bad(v.z) || bad(v.w));
  }
  // infinities and NaN taken out
  static __device__ __forceinline__ Pair finite_part(Pair v) {
    auto f = [](uint32_t u) {
      if ((u & 0x7f800000u) == 0x7f800000u) u &= 0xffffu;
      if ((u & 0x7f80u) == 0x7f80u) u &= 0xffff0000u;
      return u;
    };
    return make_uint4(f(v.x), f(v.y), f(v.z), f(v.w));
  }
  static __device__ __forceinline__ void put4(E* p, f32x4 v) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  }
  static __device__ __forceinline__ E round(float v) { return f32_to_bf16_rne(v); }
};

// f32 operands on v_mfma_f32_16x16x4_f32, four contracted at a time.
template <>
struct Op<false> {
  using E = float;
  struct Pair {
    f32x4 a, b;
  };
  static constexpr int C = 32;
  static constexpr int kPiece = 4;
  static constexpr int kPad = 4;
  static constexpr int kState = 1;
  static constexpr int kScore = 1;
  static __device__ __forceinline__ f32x4 mma(Pair a, Pair b, f32x4 c) {
    c = mfma_16x16x16(a.a, b.a, c);
    return mfma_16x16x16(a.b, b.b, c);
  }
  template <int NP>
  static __device__ __forceinline__ void split(f32x4 a, f32x4 b, Pair (&out)[NP]) {
    static_assert(NP == 1, "f32 operands are whole");
    out[0] = Pair{a, b};
  }
  static __device__ __forceinline__ Pair row_pair(const E* row, int g) {
    return Pair{*reinterpret_cast<const f32x4*>(row + 4 * g), *reinterpret_cast<const f32x4*>(row + 16 + 4 * g)};
  }
  static __device__ __forceinline__ Pair row_pair_any(const E* row, int g) { return row_pair(row, g); }
  static __device__ __forceinline__ Pair column_pair(const E* tile, int stride, int j0, int col0, int g, int c) {
    const E* p = tile + (j0 + 4 * g) * stride + col0 + c;
    const E* q = p + 16 * stride;
    return Pair{f32x4{p[0], p[stride], p[2 * stride], p[3 * stride]},
                f32x4{q[0], q[stride], q[2 * stride], q[3 * stride]}};
  }
  static __device__ __forceinline__ f32x4 low(Pair a) { return a.a; }
  static __device__ __forceinline__ f32x4 high(Pair a) { return a.b; }
  static __device__ __forceinline__ f32x4 four(const E* p) { return *reinterpret_cast<const f32x4*>(p); }
  static __device__ __forceinline__ float one(E v) { return v; }
  static __device__ __forceinline__ bool finite(uint4 v) {
    auto bad = [](uint32_t u) { return (u & 0x7f800000u) == 0x7f800000u; };
    return !(bad(v.x) || bad(v.y) || bad(v.z) || bad(v.w));
  }
  static __device__ __forceinline__ Pair finite_part(Pair v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if ((__float_as_uint(v.a[i]) & 0x7f800000u) == 0x7f800000u) v.a[i] = 0.0f;
      if ((__float_as_uint(v.b[i]) & 0x7f800000u) == 0x7f800000u) v.b[i] = 0.0f;
    }
    return v;
  }
  static __device__ __forceinline__ void put4(E* p, f32x4 v) { *reinterpret_cast<f32x4*>(p) = v; }
  static __device__ __forceinline__ E round(float v) { return v; }
};

template <bool BF, int NKT, int NV>
struct Shape {
  using O = Op<BF>;
  using E = typename O::E;
  static constexpr int C = O::C, CT = C / 16;
  static constexpr int DX = 16 * NKT;       // widest x and y
  static constexpr int BV = 64 * NV;        // columns of z a workgroup holds: 16 NV a wave
  static constexpr int SX = DX + O::kPad, SZ = BV + O::kPad, SP = C + O::kPad;
  static constexpr int NX = C * DX / O::kPiece / kThreads;  // 16-byte pieces a thread of a tile
  static constexpr int NZ = C * BV / O::kPiece / kThreads;
  struct Lds {
    alignas(16) E x[C * SX];
    alignas(16) E y[C * SX];
    alignas(16) E z[C * SZ];
    alignas(16) E score[O::kScore][C * SP];
    alignas(16) E w[C * SZ];
    float pairs[C * (C + 1)];
    alignas(16) float2 g[C];   // running log2 decay, high and low part
    alignas(16) float row[C];  // decay between the row and the state
    alignas(16) float src[C];  // decay between the source and the next state, times scale_src
    float part[kWaves][C];
    float rect[kThreads];
    float total;
    int odd[2];                // a chunk's z holds an infinity or NaN
  };
  static_assert(NX >= 1 && NZ >= 1, "tiles smaller than a workgroup");
};

// Base of head h of batch row b, at token 0.
template <typename E>
__device__ __forceinline__ const E* head_base(const HeadView& v, int b, int h) {
  return static_cast<const E*>(v.p) + int64_t(b) * v.sb + int64_t(h / v.rep) * v.sh;
}

// A thread's pieces of the tile of C tokens from tb and W columns from c0; zero
// where a token (from `end` on) or a column (from `d` on) does not exist.
template <bool BF, int W, int N>
__device__ __forceinline__ void load_tile(const HeadView& v, const typename Op<BF>::E* base, int d, int c0, int tb,
                                          int end, uint4 (&r)[N]) {
  using E = typename Op<BF>::E;
  constexpr int P = Op<BF>::kPiece, PR = W / P;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int q = int(threadIdx.x) + n * kThreads;
    const int t = tb + q / PR, col = c0 + q % PR * P;
    r[n] = make_uint4(0, 0, 0, 0);
    if (t < end && col < d) {
      const E* p = base + int64_t(t) * v.st + int64_t(col) * v.sd;
      if (v.vec) {
        r[n] = *reinterpret_cast<const uint4*>(p);
      } else {
        uint32_t u[4] = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < P; ++e) {
          if (col + e < d) {
            if constexpr (BF) u[e / 2] |= uint32_t(p[e * v.sd]) << (16 * (e & 1));
            else u[e] = __float_as_uint(p[e * v.sd]);
          }
        }
        r[n] = make_uint4(u[0], u[1], u[2], u[3]);
      }
    }
  }
}

template <bool BF, int W, int N>
__device__ __forceinline__ void store_tile(typename Op<BF>::E* tile, int stride, const uint4 (&r)[N]) {
  constexpr int P = Op<BF>::kPiece, PR = W / P;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int q = int(threadIdx.x) + n * kThreads;
    *reinterpret_cast<uint4*>(tile + q / PR * stride + q % PR * P) = r[n];
  }
}

__device__ __forceinline__ double shfl_up_f64(double v, int d) {
  const long long u = __double_as_longlong(v);
  const int lo = __shfl_up(int(uint32_t(u)), d), hi = __shfl_up(int(u >> 32), d);
  return __longlong_as_double((static_cast<long long>(hi) << 32) | uint32_t(lo));
}

__device__ __forceinline__ float exp2_hw(float v) { return __builtin_amdgcn_exp2f(v); }

// A chunk's decays from a lane's log decay gv (wave 0; token tb + lane).
template <bool REV, int C, typename Lds>
__device__ __forceinline__ void chunk_decays(Lds& l, float gv, float scale_src, int lane) {
  gv = gv < -kMostLog ? -kMostLog : gv > kMostLog ? kMostLog : gv;
  // 64 bits: the difference of two running sums is the log decay between two tokens, and has to be
  // exact to f32 also behind a token that cut the state.
  double s = double(gv) * 1.4426950408889634;
#pragma unroll
  for (int d = 1; d < C; d *= 2) {
    const double u = shfl_up_f64(s, d);
    if (lane >= d) s += u;
  }
  const long long all = __double_as_longlong(s);
  const int tlo = __shfl(int(uint32_t(all)), C - 1), thi = __shfl(int(all >> 32), C - 1);
  const double total = __longlong_as_double((static_cast<long long>(thi) << 32) | uint32_t(tlo));
  if (lane < C) {
    const float hi = float(s);
    l.g[lane] = make_float2(hi, float(s - double(hi)));
    const float from_start = exp2_hw(hi), to_end = exp2_hw(float(total - s));
    l.row[lane] = REV ? to_end : from_start;
    l.src[lane] = (REV ? from_start : to_end) * scale_src;
    if (lane == 0) l.total = exp2_hw(float(total));
  }
}

// One workgroup's march. MASS: 0 none, 1 the rows' part of the decay's gradient
// (forward), 2 the sources' part (reverse). OUT false: the segment's own state only.
template <bool BF, int NKT, int NV, bool REV, int MASS, bool OUT>
__device__ __forceinline__ void march(const DaParams& p, const DaMarch& m, int block,
                                      typename Shape<BF, NKT, NV>::Lds& l) {
  using S = Shape<BF, NKT, NV>;
  using O = Op<BF>;
  using E = typename O::E;
  using Pair = typename O::Pair;
  constexpr int C = S::C, CT = S::CT;
  const int tid = int(threadIdx.x), lane = tid & 63, wave = tid >> 6, g = lane >> 4, c = lane & 15;

  const int ncb = (m.dz + S::BV - 1) / S::BV, BH = p.B * p.H;
  const int cb = block % ncb, bh = block / ncb % BH, seg_m = block / ncb / BH;
  if (seg_m >= (OUT ? p.segments : p.segments - 1)) return;
  const int b = bh / p.H, h = bh % p.H;
  const int seg = REV ? p.segments - 1 - seg_m : seg_m;
  const int t0 = seg * p.seg_tokens, t1 = min(p.T, t0 + p.seg_tokens);
  int len = p.T;
  if (p.lengths) len = min(max(p.lengths[b], 0), p.T);
  const int live = max(min(len, t1) - t0, 0);
  const int nc = (live + C - 1) / C;
  const int c0 = cb * S::BV, wc0 = 16 * NV * wave;  // first column of the workgroup, and of the wave within it
  const int nkt = (m.dx + 15) / 16;                 // tiles of x that exist
  const int64_t state = int64_t(p.dk) * p.dv;

  const E* xb = OUT ? head_base<E>(m.x, b, h) : nullptr;
  const E* yb = head_base<E>(m.y, b, h);
  const E* zb = head_base<E>(m.z, b, h);
  const E* wb = MASS ? head_base<E>(m.w, b, h) : nullptr;
  const float* gb = p.g + int64_t(b) * p.gb + int64_t(h) * p.gh;

  // The state: tile kt, rows 16 kt + 4 g + r, column c0 + wc0 + 16 n + c.
  f32x4 st[NKT][NV];
  {
    const float* from = !OUT ? nullptr : seg_m == 0 ? (m.first ? m.first + bh * state : nullptr)
                                                    : m.seg + (int64_t(seg_m - 1) * BH + bh) * state;
#pragma unroll
    for (int kt = 0; kt < NKT; ++kt)
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * kt + 4 * g + r, col = c0 + wc0 + 16 * n + c;
          st[kt][n][r] = from && row < m.dx && col < m.dz ? from[row * m.sr + col * m.sc] : 0.0f;
        }
  }

  uint4 rx[OUT ? S::NX : 1], ry[S::NX], rz[S::NZ], rw[MASS ? S::NZ : 1];
  float rg = 0.0f;
  auto fetch = [&](int ci) {
    const int tb = t0 + (REV ? nc - 1 - ci : ci) * C, end = min(len, t1);
    if constexpr (OUT) load_tile<BF, S::DX>(m.x, xb, m.dx, 0, tb, end, rx);
    load_tile<BF, S::DX>(m.y, yb, m.dx, 0, tb, end, ry);
    load_tile<BF, S::BV>(m.z, zb, m.dz, c0, tb, end, rz);
    if constexpr (MASS != 0) load_tile<BF, S::BV>(m.w, wb, m.dz, c0, tb, end, rw);
    if (wave == 0) rg = lane < C && tb + lane < end ? gb[int64_t(tb + lane) * p.gt] : 0.0f;
  };

  if (tid < 2) l.odd[tid] = 0;
  float decays = 1.0f;
  if (nc > 0) fetch(0);
  for (int ci = 0; ci < nc; ++ci) {
    const int chunk = REV ? nc - 1 - ci : ci, tb = t0 + chunk * C;
    __syncthreads();
    if constexpr (OUT) store_tile<BF, S::DX>(l.x, S::SX, rx);
    store_tile<BF, S::DX>(l.y, S::SX, ry);
    store_tile<BF, S::BV>(l.z, S::SZ, rz);
    if constexpr (MASS != 0) store_tile<BF, S::BV>(l.w, S::SZ, rw);
    if constexpr (OUT) {
      bool fine = true;
#pragma unroll
      for (int n = 0; n < S::NZ; ++n) fine = fine && O::finite(rz[n]);
      if (!fine) l.odd[ci & 1] = 1;
    }
    if (wave == 0) chunk_decays<REV, C>(l, rg, m.scale_src, lane);
    __syncthreads();
    if (ci + 1 < nc) fetch(ci + 1);
    const bool odd = OUT && l.odd[ci & 1] != 0;
    const float total = l.total;

    f32x4 acc[OUT ? NV : 1][OUT ? CT : 1];  // out transposed: column wc0 + 16 n + 4 g + r, row 16 it + c
    if constexpr (OUT) {
      // scores: the tiles on and on one side of the diagonal, in turn over the waves, as [row][source]
      for (int q = wave; q < CT * (CT + 1) / 2; q += kWaves) {
        int hi = 0, lo = q;
        while (lo > hi) lo -= ++hi;
        const int it = REV ? lo : hi, jt = REV ? hi : lo;
        const int row = 16 * it + c;
        f32x4 s = zero4();
#pragma unroll
        for (int k2 = 0; k2 < NKT / 2; ++k2)
          if (2 * k2 < nkt)
            s = O::mma(O::row_pair_any(l.y + (16 * jt + c) * S::SX + 32 * k2, g),
                       O::row_pair_any(l.x + row * S::SX + 32 * k2, g), s);
        const float2 gi = l.g[row];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = 16 * jt + 4 * g + r;
          const float2 gj = l.g[j];
          const float d = (gi.x - gj.x) + (gi.y - gj.y);
          const bool seen = REV ? j >= row : j <= row;
          s[r] = seen ? s[r] * m.scale_src * exp2_hw(REV ? -d : d) : 0.0f;
        }
        if constexpr (BF) {
          Pair parts[O::kScore];
          O::template split<O::kScore>(s, s, parts);
#pragma unroll
          for (int n = 0; n < O::kScore; ++n)
            *reinterpret_cast<uint2*>(l.score[n] + row * S::SP + 16 * jt + 4 * g) = make_uint2(parts[n].x, parts[n].y);
        } else {
          O::put4(l.score[0] + row * S::SP + 16 * jt + 4 * g, s);
        }
        if constexpr (MASS == 1) {
          // what a row takes from a source: decay (x_i . y_j) (w_i . z_j), this workgroup's columns of the second
          f32x4 a = zero4();
#pragma unroll
          for (int k2 = 0; k2 < S::BV / 32; ++k2)
            a = O::mma(O::row_pair_any(l.z + (16 * jt + c) * S::SZ + 32 * k2, g),
                       O::row_pair_any(l.w + row * S::SZ + 32 * k2, g), a);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int j = 16 * jt + 4 * g + r;
            l.pairs[row * (C + 1) + j] = j < row ? a[r] * s[r] * m.scale_out : 0.0f;
          }
        }
      }
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int it = 0; it < CT; ++it) acc[n][it] = zero4();
      // rows against the state
#pragma unroll
      for (int k2 = 0; k2 < NKT / 2; ++k2) {
        if (2 * k2 < nkt) {
          Pair sp[NV][O::kState];
#pragma unroll
          for (int n = 0; n < NV; ++n) O::template split<O::kState>(st[2 * k2][n], st[2 * k2 + 1][n], sp[n]);
#pragma unroll
          for (int it = 0; it < CT; ++it) {
            const Pair x = O::row_pair(l.x + (16 * it + c) * S::SX + 32 * k2, g);
#pragma unroll
            for (int n = 0; n < NV; ++n)
#pragma unroll
              for (int q = O::kState - 1; q >= 0; --q) acc[n][it] = O::mma(sp[n][q], x, acc[n][it]);
          }
        }
      }
#pragma unroll
      for (int it = 0; it < CT; ++it) {
        const float f = l.row[16 * it + c];
        float mass = 0.0f;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
          acc[n][it] *= f;
          if constexpr (MASS != 0) {
            const f32x4 w = O::four(l.w + (16 * it + c) * S::SZ + wc0 + 16 * n + 4 * g);
#pragma unroll
            for (int r = 0; r < 4; ++r) mass += acc[n][it][r] * w[r];
          }
        }
        if constexpr (MASS != 0) {
          mass += __shfl_xor(mass, 16);
          mass += __shfl_xor(mass, 32);
          if (g == 0) l.part[wave][16 * it + c] = mass * m.scale_out;
        }
      }
      __syncthreads();
      if (tid == 0) l.odd[(ci + 1) & 1] = 0;
    }

    // sources: into the rows of the chunk, and into the state
#pragma unroll
    for (int kt = 0; kt < NKT; ++kt)
#pragma unroll
      for (int n = 0; n < NV; ++n) st[kt][n] *= total;
    decays *= total;
#pragma unroll
    for (int j2 = 0; j2 < CT / 2; ++j2) {
      Pair z[NV], zs[NV][O::kState];
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        z[n] = O::column_pair(l.z, S::SZ, 32 * j2, wc0 + 16 * n, g, c);
        const f32x4 f0 = *reinterpret_cast<const f32x4*>(l.src + 32 * j2 + 4 * g);
        const f32x4 f1 = *reinterpret_cast<const f32x4*>(l.src + 32 * j2 + 16 + 4 * g);
        O::template split<O::kState>(O::low(z[n]) * f0, O::high(z[n]) * f1, zs[n]);
      }
      if constexpr (OUT) {
        // An infinity or NaN in z times a score of zero would reach rows that do not see its token: such
        // values are left out here and added below to the rows that do.
        if (odd)
          for (int n = 0; n < NV; ++n) z[n] = O::finite_part(z[n]);
#pragma unroll
        for (int it = 0; it < CT; ++it) {
          if (REV ? it <= 2 * j2 + 1 : it >= 2 * j2) {
            // the one tile of a pair beyond the diagonal was not written
            const bool half = REV ? it == 2 * j2 + 1 : it == 2 * j2;
#pragma unroll
            for (int q = O::kScore - 1; q >= 0; --q) {
              Pair s = O::row_pair(l.score[q] + (16 * it + c) * S::SP + 32 * j2, g);
              if (half) {
                if constexpr (BF) {
                  if (REV) s.x = s.y = 0; else s.z = s.w = 0;
                } else {
                  if (REV) s.a = zero4(); else s.b = zero4();
                }
              }
#pragma unroll
              for (int n = 0; n < NV; ++n) acc[n][it] = O::mma(z[n], s, acc[n][it]);
            }
          }
        }
      }
#pragma unroll
      for (int kt = 0; kt < NKT; ++kt) {
        if (kt < nkt) {
          const Pair y = O::column_pair(l.y, S::SX, 32 * j2, 16 * kt, g, c);
#pragma unroll
          for (int n = 0; n < NV; ++n)
#pragma unroll
            for (int q = O::kState - 1; q >= 0; --q) st[kt][n] = O::mma(y, zs[n][q], st[kt][n]);
        }
      }
    }

    if constexpr (OUT) {
      if (odd) {
        for (int j = 0; j < C; ++j)
#pragma unroll
          for (int n = 0; n < NV; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float v = O::one(l.z[j * S::SZ + wc0 + 16 * n + 4 * g + r]);
              if ((__float_as_uint(v) & 0x7f800000u) != 0x7f800000u) continue;
#pragma unroll
              for (int it = 0; it < CT; ++it) {
                const int row = 16 * it + c;
                if (REV ? j >= row : j <= row) acc[n][it][r] += O::one(l.score[0][row * S::SP + j]) * v;
              }
            }
      }
      const bool whole = (m.dz & 3) == 0;
#pragma unroll
      for (int it = 0; it < CT; ++it) {
        const int t = tb + 16 * it + c;
        if (t < t1) {
          const int64_t at = ((int64_t(b) * p.T + t) * p.H + h) * m.dz;
#pragma unroll
          for (int n = 0; n < NV; ++n) {
            const int col = c0 + wc0 + 16 * n + 4 * g;
            f32x4 v = acc[n][it] * m.scale_out;
            if (t >= len) v = zero4();
            if (whole && col < m.dz) {
              if (!BF || m.out_f32) *reinterpret_cast<f32x4*>(static_cast<float*>(m.out) + at + col) = v;
              else Op<true>::put4(static_cast<uint16_t*>(m.out) + at + col, v);
            } else {
#pragma unroll
              for (int r = 0; r < 4; ++r)
                if (col + r < m.dz) {
                  if (!BF || m.out_f32) static_cast<float*>(m.out)[at + col + r] = v[r];
                  else static_cast<uint16_t*>(m.out)[at + col + r] = f32_to_bf16_rne(v[r]);
                }
            }
          }
        }
      }
      if constexpr (MASS != 0) {
        const int64_t mb = (int64_t(cb) * BH + bh);
        float rect = 0.0f;
        if constexpr (MASS == 1) {
          // a token's decay carries every pair of a source before it and a row from it on: sum the
          // sources of each row, then the rows of each token. Both sums are taken outright, not as
          // differences of running totals, so a cut leaves an exact zero.
          constexpr int PARTS = kThreads / C, N = C / PARTS;
          const int row = tid / PARTS, part = tid % PARTS;
          float v[N], sum = 0.0f;
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const int j = part * N + i;
            v[i] = sum;
            if (j < row) sum += l.pairs[row * (C + 1) + j];
          }
          float before = sum;
#pragma unroll
          for (int d = 1; d < PARTS; d *= 2) {
            const float u = __shfl_up(before, d);
            if (part >= d) before += u;
          }
          before = __shfl_up(before, 1);
          if (part == 0) before = 0.0f;
#pragma unroll
          for (int i = 0; i < N; ++i) l.pairs[row * (C + 1) + part * N + i] = before + v[i];
          __syncthreads();
          const int t = tid % C, from = tid / C;
          float s = 0.0f;
          for (int i = from * N; i < from * N + N; ++i)
            if (i >= t) s += l.pairs[i * (C + 1) + t];
          l.rect[tid] = s;
          __syncthreads();
          if (tid < C)
            for (int q = 0; q < PARTS; ++q) rect += l.rect[q * C + tid];
        }
        if (wave == 0) {
          float v = 0.0f;
          if (lane < C)
            for (int q = 0; q < kWaves; ++q) v += l.part[q][lane];
          const int tok = tb + lane;
          // rows from the token on (MASS 1), or sources before it (MASS 2)
          float run = v;
#pragma unroll
          for (int d = 1; d < C; d *= 2) {
            const float u = MASS == 1 ? __shfl_down(run, d) : __shfl_up(run, d);
            if (MASS == 1 ? lane + d < C : lane >= d) run += u;
          }
          const float all = __shfl(run, MASS == 1 ? 0 : C - 1);
          float mine = run;
          if (MASS == 2) {
            mine = __shfl_up(run, 1);
            if (lane == 0) mine = 0.0f;
          }
          if (lane < C && tok < t1) m.mass[mb * p.T + tok] = mine + rect;
          if (lane == 0) {
            const int chunks = (p.T + C - 1) / C;
            m.mass_chunk[mb * chunks + tb / C] = all;
            if (m.chunk_decay && cb == 0) m.chunk_decay[int64_t(bh) * chunks + tb / C] = total;
          }
        }
      }
    }
  }

  if constexpr (OUT) {
    // tokens past the row's length, in chunks that were not marched
    const int from = t0 + nc * C;
    const int width = min(S::BV, m.dz - c0), rest = max(t1 - from, 0);
    for (int q = tid; q < rest * width; q += kThreads) {
      const int64_t at = ((int64_t(b) * p.T + from + q / width) * p.H + h) * m.dz + c0 + q % width;
      if (!BF || m.out_f32) static_cast<float*>(m.out)[at] = 0.0f;
      else static_cast<uint16_t*>(m.out)[at] = 0;
    }
    if constexpr (MASS != 0) {
      const int64_t mb = (int64_t(cb) * BH + bh);
      const int chunks = (p.T + C - 1) / C;
      for (int q = tid; q < rest; q += kThreads) m.mass[mb * p.T + from + q] = 0.0f;
      for (int q = tid; q < (rest + C - 1) / C; q += kThreads) {
        m.mass_chunk[mb * chunks + from / C + q] = 0.0f;
        if (m.chunk_decay && cb == 0) m.chunk_decay[int64_t(bh) * chunks + from / C + q] = 1.0f;
      }
    }
  }

  float* to = OUT ? (seg_m == p.segments - 1 && m.last ? m.last + bh * state : nullptr)
                  : m.seg + (int64_t(seg_m) * BH + bh) * state;
  if (to) {
#pragma unroll
    for (int kt = 0; kt < NKT; ++kt)
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * kt + 4 * g + r, col = c0 + wc0 + 16 * n + c;
          if (row < m.dx && col < m.dz) to[row * m.sr + col * m.sc] = st[kt][n][r];
        }
  }
  if (!OUT && tid == 0 && cb == 0) m.seg_decay[int64_t(seg_m) * BH + bh] = decays;
}

// blockIdx.y picks the march of a gradient: 0 grad_q, 1 grad_k, 2 grad_v.
template <bool BF, int NKT, int NV>
__global__ __launch_bounds__(kThreads) void march_forward(DaParams p) {
  __shared__ typename Shape<BF, NKT, NV>::Lds l;
  march<BF, NKT, NV, false, 0, true>(p, p.m[0], blockIdx.x, l);
}

template <bool BF, int NKT, int NV>
__global__ __launch_bounds__(kThreads) void march_gradient(DaParams p) {
  __shared__ typename Shape<BF, NKT, NV>::Lds l;
  if (blockIdx.y == 0) march<BF, NKT, NV, false, 1, true>(p, p.m[0], blockIdx.x, l);
  else if (blockIdx.y == 1) march<BF, NKT, NV, true, 2, true>(p, p.m[1], blockIdx.x, l);
  else march<BF, NKT, NV, true, 0, true>(p, p.m[2], blockIdx.x, l);
}

// Each segment's own state. A gradient needs two: the state (march 0's) and its
// adjoint (march 1's, which march 2 shares).
template <bool BF, int NKT, int NV>
__global__ __launch_bounds__(kThreads) void march_local(DaParams p) {
  __shared__ typename Shape<BF, NKT, NV>::Lds l;
  if (blockIdx.y == 0) march<BF, NKT, NV, false, 0, false>(p, p.m[0], blockIdx.x, l);
  else march<BF, NKT, NV, true, 0, false>(p, p.m[1], blockIdx.x, l);
}

// Segment m's entry, its own state so far, becomes the state at the start of segment m + 1.
__global__ __launch_bounds__(kThreads) void carry(DaParams p) {
  const DaMarch& m = p.m[blockIdx.y];
  const int64_t state = int64_t(p.dk) * p.dv, BH = int64_t(p.B) * p.H;
  const int64_t e = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (e >= BH * state) return;
  const int64_t bh = e / state;
  float s = m.first ? m.first[e] : 0.0f;
  for (int i = 0; i < p.segments - 1; ++i) {
    float* at = m.seg + i * BH * state + e;
    s = fmaf(m.seg_decay[i * BH + bh], s, *at);
    *at = s;
  }
}

// ---------------------------------------------------------------- the decay's gradient

__device__ __forceinline__ double block_sum(double v, double* l) {
  const int tid = int(threadIdx.x);
  l[tid] = v;
  __syncthreads();
  for (int d = kThreads / 2; d > 0; d /= 2) {
    if (tid < d) l[tid] += l[tid + d];
    __syncthreads();
  }
  v = l[0];
  __syncthreads();
  return v;
}

// What passes a chunk from before to after it, Y, from what crosses the border
// before it, Z: Y = Z - (its rows' mass), the next Z = Y + (its sources' mass), and
// Y is zero outright where the chunk's decays multiply to zero. One workgroup a
// head; the chunks are scanned as maps Z -> keep Z + add.
__global__ __launch_bounds__(kThreads) void decay_grad(DaDecayGrad p) {
  __shared__ double la[kThreads];
  __shared__ int lk[kThreads];
  const int bh = blockIdx.x, tid = int(threadIdx.x), b = bh / p.H, h = bh % p.H;
  const int64_t BH = int64_t(p.B) * p.H, state = int64_t(p.dk) * p.dv;
  int len = p.T;
  if (p.lengths) len = min(max(p.lengths[b], 0), p.T);
  auto sum_of = [&](const float* v, int64_t n, int64_t i) {
    double s = 0.0;
    for (int k = 0; k < p.blocks; ++k) s += double(v[(k * BH + bh) * n + i]);
    return s;
  };
  double z0 = 0.0;
  if (p.initial) {
    double s = 0.0;
    for (int64_t i = tid; i < state; i += kThreads)
      s += double(p.initial[bh * state + i]) * double(p.grad_initial[bh * state + i]);
    z0 = block_sum(s, la);
  }
  const int per = (p.chunks + kThreads - 1) / kThreads;
  const int first = min(tid * per, p.chunks), last = min(first + per, p.chunks);
  double add = 0.0;
  int keep = 1;
  for (int i = first; i < last; ++i) {
    const bool cut = p.chunk_decay[int64_t(bh) * p.chunks + i] == 0.0f;
    add = (cut ? 0.0 : add - sum_of(p.rows_chunk, p.chunks, i)) + sum_of(p.sources_chunk, p.chunks, i);
    if (cut) keep = 0;
  }
  la[tid] = add;
  lk[tid] = keep;
  __syncthreads();
  for (int d = 1; d < kThreads; d *= 2) {
    double a = 0.0;
    int k = 1;
    if (tid >= d) {
      a = la[tid - d];
      k = lk[tid - d];
    }
    __syncthreads();
    if (tid >= d) {
      if (lk[tid]) la[tid] += a;
      lk[tid] &= k;
    }
    __syncthreads();
  }
  double z = tid == 0 ? z0 : la[tid - 1] + (lk[tid - 1] ? z0 : 0.0);
  __syncthreads();
  double all = 0.0;
  for (int i = first; i < last; ++i) {
    const bool cut = p.chunk_decay[int64_t(bh) * p.chunks + i] == 0.0f;
    const double y = cut ? 0.0 : z - sum_of(p.rows_chunk, p.chunks, i);
    z = y + sum_of(p.sources_chunk, p.chunks, i);
    for (int t = i * p.chunk; t < min((i + 1) * p.chunk, p.T); ++t) {
      double v = 0.0;
      if (t < len) {
        const float gv = p.g[int64_t(b) * p.gb + int64_t(t) * p.gt + int64_t(h) * p.gh];
        // exp(g) = 0: nothing passes, and neither does a gradient
        if (!(gv <= -kMostLog)) v = y + sum_of(p.rows, p.T, t) + sum_of(p.sources, p.T, t);
      }
      if (p.per_head) all += v;
      else p.grad_g[(int64_t(b) * p.T + t) * p.H + h] = float(v);
    }
  }
  if (p.per_head) {
    all = block_sum(all, la);
    if (tid == 0) p.partial[bh] = all;
  }
}

__global__ void decay_grad_heads(DaDecayGrad p) {
  const int h = blockIdx.x * blockDim.x + threadIdx.x;
  if (h >= p.H) return;
  double s = 0.0;
  for (int b = 0; b < p.B; ++b) s += p.partial[int64_t(b) * p.H + h];
  p.grad_g[h] = float(s);
}

__global__ __launch_bounds__(kThreads) void share_sum(DaShare p) {
  const int64_t n = p.rows * p.d;
  for (int64_t e = int64_t(blockIdx.x) * kThreads + threadIdx.x; e < n; e += int64_t(gridDim.x) * kThreads) {
    const int64_t row = e / p.d, d = e % p.d;
    float s = 0.0f;
    for (int r = 0; r < p.rep; ++r) s += p.src[(row * p.rep + r) * p.d + d];
    if (p.bf16) static_cast<uint16_t*>(p.out)[e] = f32_to_bf16_rne(s);
    else static_cast<float*>(p.out)[e] = s;
  }
}

// ---------------------------------------------------------------- one token

// One workgroup a request, head and block of kStepCols columns: 8 threads of 4
// columns, 32 rows at a time.
constexpr int kStepCols = 32;

template <bool BF>
__global__ __launch_bounds__(kThreads) void step_kernel(DaStep p) {
  using O = Op<BF>;
  using E = typename O::E;
  __shared__ float sum[kThreads / 8][kStepCols];
  const int tid = int(threadIdx.x), cols = (p.dv + kStepCols - 1) / kStepCols;
  const int cb = blockIdx.x % cols, bh = blockIdx.x / cols, b = bh / p.H, h = bh % p.H;
  const int64_t slot = p.slots ? int64_t(p.slots[b]) : int64_t(b);
  const bool used = slot >= 0 && slot < p.slots_in_pool;
  const int col = cb * kStepCols + (tid & 7) * 4, r0 = tid >> 3;
  f32x4 o = zero4();
  if (used) {
    const E* q = head_base<E>(p.q, b, h);
    const E* k = head_base<E>(p.k, b, h);
    const E* v = head_base<E>(p.v, b, h);
    const float decay = expf(p.g[int64_t(b) * p.gb + int64_t(h) * p.gh]);
    f32x4 vv = zero4();
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (col + e < p.dv) vv[e] = O::one(v[int64_t(col + e) * p.v.sd]);
    float* s = p.state + slot * p.ss + int64_t(h) * p.sh;
    for (int r = r0; r < p.dk; r += kThreads / 8) {
      const float kr = O::one(k[int64_t(r) * p.k.sd]), qr = O::one(q[int64_t(r) * p.q.sd]);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (col + e < p.dv) {
          const float n = fmaf(decay, s[int64_t(r) * p.dv + col + e], kr * vv[e]);
          s[int64_t(r) * p.dv + col + e] = n;
          o[e] = fmaf(qr, n, o[e]);
        }
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) sum[r0][(tid & 7) * 4 + e] = o[e];
  __syncthreads();
  if (tid < kStepCols && cb * kStepCols + tid < p.dv) {
    float t = 0.0f;
    for (int r = 0; r < kThreads / 8; ++r) t += sum[r][tid];
    const int64_t at = int64_t(bh) * p.dv + cb * kStepCols + tid;
    static_cast<E*>(p.out)[at] = O::round(t * p.scale);
  }
}

// ---------------------------------------------------------------- launches

int tile_class(int d) { return d <= 32 ? 2 : d <= 64 ? 4 : d <= 128 ? 8 : 16; }

template <bool BF, int NKT, int NV>
hipError_t run_marches(const DaParams& p, hipStream_t stream) {
  const int64_t BH = int64_t(p.B) * p.H;
  int ncb = 1;
  for (int i = 0; i < p.marches; ++i) ncb = std::max(ncb, (p.m[i].dz + 64 * NV - 1) / (64 * NV));
  const int states = p.marches == 1 ? 1 : 2;
  if (p.segments > 1) {
    march_local<BF, NKT, NV><<<dim3(unsigned(ncb * BH * (p.segments - 1)), states), kThreads, 0, stream>>>(p);
    const int64_t n = BH * p.dk * p.dv;
    carry<<<dim3(unsigned((n + kThreads - 1) / kThreads), states), kThreads, 0, stream>>>(p);
  }
  const dim3 grid(unsigned(ncb * BH * p.segments), p.marches);
  if (p.marches == 1) march_forward<BF, NKT, NV><<<grid, kThreads, 0, stream>>>(p);
  else march_gradient<BF, NKT, NV><<<grid, kThreads, 0, stream>>>(p);
  return hipGetLastError();
}

template <bool BF>
hipError_t run_widths(const DaParams& p, hipStream_t stream) {
  const int wide = std::max(p.dk, p.dv);
  switch (tile_class(wide)) {
    case 2: return run_marches<BF, 2, 1>(p, stream);
    case 4: return run_marches<BF, 4, 1>(p, stream);
    case 8: return run_marches<BF, 8, 2>(p, stream);
    default: return run_marches<BF, 16, 1>(p, stream);
  }
}

}  // namespace

int decay_attention_chunk(bool bf16) { return bf16 ? Op<true>::C : Op<false>::C; }

int decay_attention_column_blocks(int dx, int dz) {
  const int bv = tile_class(std::max(dx, dz)) == 8 ? 128 : 64;
  return (dz + bv - 1) / bv;
}

void decay_attention_split(DaParams& p) {
  const int C = decay_attention_chunk(p.bf16 != 0);
  const int64_t chunks = (int64_t(p.T) + C - 1) / C;
  const int64_t groups = std::max<int64_t>(1, int64_t(p.B) * p.H * decay_attention_column_blocks(p.dk, p.dv));
  // two workgroups a compute unit, segments of two chunks at least
  const int64_t want = (2 * device_cu_count() + groups - 1) / groups;
  const int64_t segments = std::max<int64_t>(1, std::min(want, chunks / 2));
  const int64_t per = std::max<int64_t>(1, (chunks + segments - 1) / segments);
  p.seg_tokens = int(per * C);
  p.segments = int(std::max<int64_t>(1, (chunks + per - 1) / per));
}

hipError_t launch_decay_attention(const DaParams& p, hipStream_t stream) {
  return p.bf16 ? run_widths<true>(p, stream) : run_widths<false>(p, stream);
}

hipError_t launch_decay_grad(const DaDecayGrad& p, hipStream_t stream) {
  if (p.B > 0) decay_grad<<<unsigned(int64_t(p.B) * p.H), kThreads, 0, stream>>>(p);
  if (p.per_head) decay_grad_heads<<<(p.H + 63) / 64, 64, 0, stream>>>(p);
  return hipGetLastError();
}

hipError_t launch_share_sum(const DaShare& p, hipStream_t stream) {
  const int64_t n = p.rows * p.d;
  if (n == 0) return hipSuccess;
  const int64_t blocks = std::min<int64_t>((n + kThreads - 1) / kThreads, int64_t(device_cu_count()) * 16);
  share_sum<<<unsigned(blocks), kThreads, 0, stream>>>(p);
  return hipGetLastError();
}

hipError_t launch_decay_step(const DaStep& p, hipStream_t stream) {
  const unsigned grid = unsigned(int64_t(p.B) * p.H * ((p.dv + kStepCols - 1) / kStepCols));
  if (p.bf16) step_kernel<true><<<grid, kThreads, 0, stream>>>(p);
  else step_kernel<false><<<grid, kThreads, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace sx
