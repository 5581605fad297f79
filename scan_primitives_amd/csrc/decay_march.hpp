// decay_march.hpp: the march of decay attention: chunks of C tokens with one
// head's state in a workgroup's accumulators, forward or reverse, for the
// operator and its gradients. Included once for each operand type and way of
// reading operands, so that they compile side by side.
//
// With G the running sum of g inside a chunk, and S the state the chunk is
// entered with,
//   out_i = scale (exp(G_i) S^T x_i + sum_{j <= i} exp(G_i - G_j) (x_i . y_j) z_j)
//   S    <- exp(G_C) S + sum_j exp(G_C - G_j) y_j z_j^T
// Every exponent is the log decay between two tokens, never its two halves
// apart, so nothing overflows however strong the decay, and a decay of zero
// (g = -inf) cuts exactly. A workgroup keeps S in its accumulators, 16 columns a
// wave: the wave layout of a 16x16 MFMA result (four rows of one column a lane)
// is the layout of an operand contracted over those rows, so S feeds x S without
// leaving the registers.
//
// A chunk has two halves between barriers: scores and rows against the state,
// then sources into the rows and into the state. y and z stand in LDS twice, so
// the next chunk's arrive during the second half; x is read in the first alone.
//
// What bounds it (gfx950, 8192 tokens, 16 heads of 128 x 128 in bf16, one
// workgroup of eight waves a compute unit, 8 chunks each, 50.5 us): of a
// chunk's share, 12 100 cycles of a busy compute unit, the matrix pipes take
// 3 100, the vector pipes 4 600, LDS 5 400 (2 400 of them bank conflicts), and
// memory would take 5 500 at the rate of a copy. Two waves a SIMD go through the
// same phases between the barriers and overlap these only in part. Two such
// workgroups do not fit a compute unit: 130 KB of LDS, 220 registers a wave.
// Measured and not taken, in earlier forms: two smaller ones (128 registers a
// wave spill, and the loads ahead with them: 107 us for 97 at 512 heads of 512
// tokens), four waves of 32 columns (spills as well), segments of half the
// length (61 to 69 us, eight ragged rows of 2048 tokens, 16 heads of 64 x 64: a
// workgroup's start costs as much as two chunks).
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "ms_mfma.hpp"
#include "sx_attention.hpp"
#include "sx_common.hpp"

namespace sx {

// v_mul_legacy_f32: the product, but zero where either factor is, whatever the other.
__device__ float mul_legacy(float, float) __asm("llvm.amdgcn.fmul.legacy");

namespace {

// Log decays are taken into [-200, 200]: exp(-200) is zero and exp(200) infinite in
// f32, so the results are those of the whole range, and -inf leaves no inf - inf.
constexpr float kMostLog = 200.0f;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

template <bool BF>
struct Op;

// bf16 operands. A Pair is what a lane brings to a product contracted over 32 on
// v_mfma_f32_16x16x32_bf16: in lane group g the values 4g .. 4g + 3 of each of two
// 16-wide tiles. The instruction's own order of the 32 does not matter, as both
// operands use the same one.
template <>
struct Op<true> {
  using E = uint16_t;
  using Pair = uint4;
  static constexpr int C = 64;      // tokens a chunk
  static constexpr int kPiece = 8;  // elements of a 16-byte piece
  // f32 values enter a product as bf16 parts: three carry all 24 bits, two carry
  // 17, enough where the result is rounded to bf16 (8 bits) on store.
  static constexpr int kState = 3;
  static constexpr int kRead = 2;
  static constexpr int kScore = 2;
  static __device__ __forceinline__ f32x4 mma(Pair a, Pair b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  }
  // NP parts of eight f32 values. Of three, each but the last is truncated and the last is what is
  // left, exactly; of two, both are rounded to nearest, 2^-18 of the value off at most.
  template <int NP>
  static __device__ __forceinline__ void split(f32x4 a, f32x4 b, Pair (&out)[NP]) {
    float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    uint32_t w[4];
    if constexpr (NP == 2) {
#pragma unroll
      for (int p = 0; p < 2; ++p) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
          if (p == 0) {
            v[2 * i] -= __uint_as_float(w[i] << 16);
            v[2 * i + 1] -= __uint_as_float(w[i] & 0xffff0000u);
          }
        }
        out[p] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    } else {
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
  }
  // 32 columns of a row from two tiles
  static __device__ __forceinline__ Pair row_pair(const E* row, int g) {
    const uint2 a = *reinterpret_cast<const uint2*>(row + 4 * g);
    const uint2 b = *reinterpret_cast<const uint2*>(row + 16 + 4 * g);
    return make_uint4(a.x, a.y, b.x, b.y);
  }
  // Where column `col` of x and of the scores stands in LDS: a lane's two fours side by side, so that a
  // row is read by 16 bytes.
  static __device__ __forceinline__ int paired(int col) {
    return (col & ~31) | (col >> 2 & 3) * 8 | (col >> 4 & 1) * 4 | (col & 3);
  }
  static __device__ __forceinline__ void store_paired(E* row, int col, uint4 v) {
    E* p = row + paired(col);
    *reinterpret_cast<uint2*>(p) = make_uint2(v.x, v.y);
    *reinterpret_cast<uint2*>(p + 8) = make_uint2(v.z, v.w);
  }
  static __device__ __forceinline__ Pair paired_row(const E* row, int g) { return row_eight(row, g); }
  // 32 columns in the other order two rows may share: eight in a row a lane
  static __device__ __forceinline__ Pair row_eight(const E* row, int g) {
    return *reinterpret_cast<const uint4*>(row + 8 * g);
  }
  // Rows 4g .. of the tiles at j0 and j0 + 16, column col0 + c, through the transposing read: lane c of a
  // group addresses four columns of one row and receives column c of four rows.
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
  // the larger magnitudes of what was seen and of a piece, half by half, as bit patterns
  typedef uint16_t halves __attribute__((ext_vector_type(2)));
  static __device__ __forceinline__ uint32_t larger(uint32_t seen, uint4 v) {
    auto most = [](uint32_t a, uint32_t b) {
      return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(halves, a),
                                                                    __builtin_bit_cast(halves, b & 0x7fff7fffu)));
    };
    return most(most(most(most(seen, v.x), v.y), v.z), v.w);
  }
  static __device__ __forceinline__ bool finite(uint32_t seen) {
    return (seen & 0xffffu) < 0x7f80u && seen < 0x7f800000u;
  }
  // a piece without its first n elements, zeros behind
  static __device__ __forceinline__ uint4 shifted(uint4 v, int n) {
    if (n & 4) v = make_uint4(v.z, v.w, 0, 0);
    if (n & 2) v = make_uint4(v.y, v.z, v.w, 0);
    if (n & 1)
      v = make_uint4(v.x >> 16 | v.y << 16, v.y >> 16 | v.z << 16, v.z >> 16 | v.w << 16, v.w >> 16);
    return v;
  }
  // infinities and NaN taken out
  static __device__ __forceinline__ uint4 finite_part(uint4 v) {
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
  static constexpr int kState = 1;
  static constexpr int kRead = 1;
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
  static __device__ __forceinline__ int paired(int col) { return col; }
  static __device__ __forceinline__ void store_paired(E* row, int col, uint4 v) {
    *reinterpret_cast<uint4*>(row + col) = v;
  }
  static __device__ __forceinline__ Pair paired_row(const E* row, int g) { return row_pair(row, g); }
  static __device__ __forceinline__ Pair row_eight(const E* row, int g) { return row_pair(row, g); }
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
  static __device__ __forceinline__ uint32_t larger(uint32_t seen, uint4 v) {
    auto most = [](uint32_t a, uint32_t b) { return max(a, b & 0x7fffffffu); };
    return most(most(most(most(seen, v.x), v.y), v.z), v.w);
  }
  static __device__ __forceinline__ bool finite(uint32_t seen) { return seen < 0x7f800000u; }
  static __device__ __forceinline__ uint4 shifted(uint4 v, int n) {
    if (n & 2) v = make_uint4(v.z, v.w, 0, 0);
    if (n & 1) v = make_uint4(v.y, v.z, v.w, 0);
    return v;
  }
  static __device__ __forceinline__ uint4 finite_part(uint4 v) {
    auto f = [](uint32_t u) { return (u & 0x7f800000u) == 0x7f800000u ? 0u : u; };
    return make_uint4(f(v.x), f(v.y), f(v.z), f(v.w));
  }
  static __device__ __forceinline__ void put4(E* p, f32x4 v) { *reinterpret_cast<f32x4*>(p) = v; }
  static __device__ __forceinline__ E round(float v) { return v; }
};

// W waves hold a state of up to 16 NKT rows and 16 NV W columns. (NV is 1: two tiles of columns a wave spill. Written
// without it the same code comes in another order of instructions: 37 tokens of 4 heads of 64 8.4 us for 7.2.)
template <bool BF, int NKT, int NV, int W>
struct Shape {
  using O = Op<BF>;
  using E = typename O::E;
  static constexpr int kThreads = W * kWave;
  static constexpr int C = O::C, CT = C / 16;
  static constexpr int TILES = CT * (CT + 1) / 2;  // tiles of scores on and on one side of the diagonal
  static constexpr int DX = 16 * NKT;              // widest x and y
  static constexpr int BV = 16 * NV * W;           // columns of z a workgroup holds: 16 NV a wave
  // Row strides in elements. 64 banks of 4 bytes: with rows 4 banks past a multiple of 64, 16 rows read by
  // 16 bytes meet no bank twice; with bf16 rows 8 past, neither do the eight rows of 32 bytes that half a
  // wave's transposing read touches.
  static constexpr int kRowPad = O::kPiece, kColPad = BF ? 16 : 4;
  static constexpr int SX = DX + kRowPad, SY = DX + kColPad, SZ = BV + kColPad, SW = BV + kRowPad, SP = C + kRowPad;
  // y and z of two chunks at once, where they fit: the next chunk's arrive while this one's are read
  static constexpr int NB = NKT == 16 ? 1 : 2;
  struct Decays {
    alignas(16) float2 g[C];   // running log2 decay, high and low part
    alignas(16) float row[C];  // decay between the row and the state, times scale_out
    alignas(16) float src[C];  // decay between the source and the next state, times scale_src
    float total;
  };
  struct Local {  // what a segment's own state takes
    alignas(16) E y[NB][C * SY];
    alignas(16) E z[NB][C * SZ];
    Decays dec[2];
  };
  struct Out : Local {
    int odd[2];       // a chunk's z holds an infinity or NaN:
    int from[2][BV];  // the first token of each column that does (in the march's order; C and more: none)
    alignas(16) E x[C * SX];
    alignas(16) E score[O::kScore][C * SP];
    alignas(16) E out[C * SW];  // a chunk's rows of out, on their way to memory
  };
  struct Mass : Out {
    alignas(16) E w[C * SW];
    float part[2][W][C];        // a wave's columns of the rows against the state, and w
    float row_tile[2][CT][C];   // pairs of a row with the sources of a tile, summed
    float col_tile[2][TILES][16];  // pairs of a tile with their source before the column and their row from it on
    double cross[W];
  };
  template <bool OUT, int MASS>
  using Lds = std::conditional_t<MASS != 0, Mass, std::conditional_t<OUT, Out, Local>>;
};

// The same value, as if new: what is formed from it is formed where it is used, not
// ahead of the loop around it, where it would hold registers through every chunk.
__device__ __forceinline__ int anew(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// Base of head h of batch row b, at token 0.
template <typename E>
__device__ __forceinline__ const E* head_base(const HeadView& v, int b, int h) {
  return static_cast<const E*>(v.p) + int64_t(b) * v.sb + int64_t(h / v.rep) * v.sh;
}

// A workgroup's tile of C tokens and W columns from c0, on its way from memory to LDS: a thread's
// share of it in registers. Zero where a token or a column (from `d` on) does not exist: there the
// load reads the last token or the first columns instead, and `store` writes zero. (A load under a
// condition would have to be waited for where its lanes join the others again.) Rows of unit stride are
// read in 16-byte pieces at any alignment, at 32-bit offsets from the tile's first token; where the last is
// not whole (Cut), it is read up to the row's end and shifted into place, which other rows need not pay for
// (the gradient of 4 x 4096 tokens of 8 heads of 128 took 2.5% longer as Cut). Else one element at a time.
enum class Rows { Elements, Cut, Whole };

template <bool BF, int W, int THREADS, Rows R>
struct Tile {
  using O = Op<BF>;
  using E = typename O::E;
  static constexpr bool VEC = R != Rows::Elements, CUT = R == Rows::Cut;
  using Held = std::conditional_t<VEC, uint4, E>;
  static constexpr int PIECE = VEC ? O::kPiece : 1, PR = W / PIECE, STEP = THREADS / PR;
  static constexpr int N = (O::C + STEP - 1) / STEP;
  static_assert(THREADS % PR == 0);
  const char* base;
  int64_t st;        // bytes a token
  int64_t col_any;   // bytes to the thread's column
  int row, col;      // of the thread's first piece in the tile
  bool ok;           // its columns exist
  int shift;         // CUT: elements that the thread's piece is read early
  Held r[N];

  __device__ __forceinline__ void init(const HeadView& v, int b, int h, int d, int c0) {
    base = reinterpret_cast<const char*>(head_base<E>(v, b, h));
    st = v.st * int64_t(sizeof(E));
    row = int(threadIdx.x) / PR;
    col = int(threadIdx.x) % PR * PIECE;
    ok = c0 + col < d;
    const int from = CUT ? min(c0 + col, d - PIECE) : c0 + col;
    if constexpr (CUT) shift = ok ? c0 + col - from : 0;
    col_any = ok ? int64_t(from) * (VEC ? 1 : v.sd) * int64_t(sizeof(E)) : 0;
  }
  // tokens tb .. of which `left` > 0 exist
  __device__ __forceinline__ void fetch(int tb, int left) {
    const char* at = base + tb * st;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int t = min(row + n * STEP, left - 1);
      if constexpr (VEC) __builtin_memcpy(&r[n], at + (uint32_t(t) * uint32_t(st) + uint32_t(col_any)), 16);
      else r[n] = *reinterpret_cast<const Held*>(at + t * st + col_any);
    }
  }
  // `columns`: the tile is wider than the tensor; `part`: the tensor's width is no whole number of pieces
  __device__ __forceinline__ void mend(int left, bool columns, bool part) {
    if constexpr (CUT) {
      if (part) {
#pragma unroll
        for (int n = 0; n < N; ++n) r[n] = O::shifted(r[n], shift);
      }
    }
    if (left < O::C || columns) {
#pragma unroll
      for (int n = 0; n < N; ++n)
        if (!ok || row + n * STEP >= left) r[n] = Held{};
    }
  }
  template <bool PAIRED = false>
  __device__ __forceinline__ void store(E* tile, int stride) const {
#pragma unroll
    for (int n = 0; n < N; ++n)
      if (O::C % STEP == 0 || row + n * STEP < O::C) {
        E* to = tile + (row + n * STEP) * stride;
        if constexpr (PAIRED && VEC) O::store_paired(to, col, r[n]);
        else *reinterpret_cast<Held*>(to + (PAIRED ? O::paired(col) : col)) = r[n];
      }
  }
  __device__ __forceinline__ bool finite() const {
    uint32_t seen = 0;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      if constexpr (VEC) seen = O::larger(seen, r[n]);
      else seen = max(seen, __float_as_uint(O::one(r[n])) & 0x7fffffffu);
    }
    return VEC ? O::finite(seen) : seen < 0x7f800000u;
  }
  // Infinities and NaN taken out; `from` of their columns holds the first token of each (the last: `rev`).
  __device__ __forceinline__ void keep_finite(int* from, bool rev) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int t = row + n * STEP;
#pragma unroll
      for (int e = 0; e < PIECE; ++e) {
        uint32_t u;
        if constexpr (!VEC) u = __float_as_uint(O::one(r[n]));
        else if constexpr (BF) u = (e & 1) ? word(n, e / 2) : word(n, e / 2) << 16;
        else u = word(n, e);
        if ((u & 0x7f800000u) == 0x7f800000u) atomicMin(from + col + e, rev ? O::C - 1 - t : t);
      }
      if constexpr (VEC) r[n] = O::finite_part(r[n]);
      else if ((__float_as_uint(O::one(r[n])) & 0x7f800000u) == 0x7f800000u) r[n] = E(0);
    }
  }
  __device__ __forceinline__ uint32_t word(int n, int i) const {
    if constexpr (VEC) return i == 0 ? r[n].x : i == 1 ? r[n].y : i == 2 ? r[n].z : r[n].w;
    else return 0;
  }
};

__device__ __forceinline__ float exp2_hw(float v) { return __builtin_amdgcn_exp2f(v); }

// v times a decay: nothing is left where that is zero, of a state that is not finite either. (A comparison and a
// selection instead cost 8192 tokens of 16 heads of 128 x 128 in bf16 3.7%.)
__device__ __forceinline__ f32x4 decayed(f32x4 v, float decay) {
#pragma unroll
  for (int r = 0; r < 4; ++r) v[r] = mul_legacy(v[r], decay);
  return v;
}

// v of the lane that CTRL names (DPP), zero where there is none
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const long long u = __double_as_longlong(v);
  const int lo = __builtin_amdgcn_update_dpp(0, int(uint32_t(u)), CTRL, 0xF, 0xF, false);
  const int hi = __builtin_amdgcn_update_dpp(0, int(u >> 32), CTRL, 0xF, 0xF, false);
  return __longlong_as_double((static_cast<long long>(hi) << 32) | uint32_t(lo));
}
__device__ __forceinline__ float lane_of(float v, int i) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), i));
}
__device__ __forceinline__ double lane_of(double v, int i) {
  const long long u = __double_as_longlong(v);
  const int lo = __builtin_amdgcn_readlane(int(uint32_t(u)), i), hi = __builtin_amdgcn_readlane(int(u >> 32), i);
  return __longlong_as_double((static_cast<long long>(hi) << 32) | uint32_t(lo));
}

// Sum of the lanes up to this one.
template <typename T>
__device__ __forceinline__ T prefix_sum(T v, int lane) {
  v += dpp<0x111>(v);
  v += dpp<0x112>(v);
  v += dpp<0x114>(v);
  v += dpp<0x118>(v);
  const T a = lane_of(v, 15), b = a + lane_of(v, 31), c = b + lane_of(v, 47);
  return lane < 16 ? v : v + (lane < 32 ? a : lane < 48 ? b : c);
}
// Sum of the lanes from this one on.
__device__ __forceinline__ float suffix_sum(float v, int lane) {
  v += dpp<0x101>(v);
  v += dpp<0x102>(v);
  v += dpp<0x104>(v);
  v += dpp<0x108>(v);
  const float c = lane_of(v, 48), b = lane_of(v, 32) + c, a = lane_of(v, 16) + b;
  return lane >= 48 ? v : v + (lane >= 32 ? c : lane >= 16 ? b : a);
}
// v of the even and of the odd one of a pair of lane groups, and of the lower and upper half of the wave.
struct Two {
  float a, b;
};
__device__ __forceinline__ Two of_pair(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return {__uint_as_float(r[0]), __uint_as_float(r[1])};
}
__device__ __forceinline__ Two of_halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return {__uint_as_float(r[0]), __uint_as_float(r[1])};
}
// Sum over the four lanes, one a group, of a column.
__device__ __forceinline__ float groups_sum(float v) {
  const Two p = of_pair(v), h = of_halves(p.a + p.b);
  return h.a + h.b;
}
// Sum over the 16 lanes of a group, in its last lane.
__device__ __forceinline__ float group_sum(float v) {
  v += dpp<0x111>(v);
  v += dpp<0x112>(v);
  v += dpp<0x114>(v);
  return v + dpp<0x118>(v);
}

// A chunk's decays from a lane's log decay gv (one wave; token tb + lane).
template <bool REV, int C, typename Decays>
__device__ __forceinline__ void chunk_decays(Decays& l, float gv, float scale_out, float scale_src, int lane) {
  gv = gv < -kMostLog ? -kMostLog : gv > kMostLog ? kMostLog : gv;
  // 64 bits: the difference of two running sums is the log decay between two tokens, and has to be
  // exact to f32 also behind a token that cut the state.
  const double s = prefix_sum(double(gv) * 1.4426950408889634, lane);
  const double total = lane_of(s, C - 1);
  if (lane < C) {
    const float hi = float(s);
    l.g[lane] = make_float2(hi, float(s - double(hi)));
    const float from_start = exp2_hw(hi), to_end = exp2_hw(float(total - s));
    l.row[lane] = (REV ? to_end : from_start) * scale_out;
    l.src[lane] = (REV ? from_start : to_end) * scale_src;
    if (lane == 0) l.total = exp2_hw(float(total));
  }
}

// A chunk's share of the decay's gradient, from the sums its rows and pairs left (one wave).
// MASS 1: what the rows from a token on take from the state and from sources before the token.
// MASS 2: what the sources before it give. The sums are taken outright, not as differences of running
// totals, so a cut leaves an exact zero.
template <bool REV, int MASS, int CT, int TILES, typename Lds>
__device__ __forceinline__ void chunk_mass(const DaParams& p, const DaMarch& m, const Lds& l, int buf, int waves,
                                           int tb, int t1, int cb, int bh, int lane) {
  constexpr int C = 16 * CT;
  const int64_t mb = int64_t(cb) * p.B * p.H + bh;
  float v = 0.0f;
  if (lane < C)
    for (int q = 0; q < waves; ++q) v += l.part[buf][q][lane];
  float mine, all;
  if constexpr (MASS == 1) {
    mine = suffix_sum(v, lane);
    all = lane_of(mine, 0);
    // pairs: the sources of whole tiles before the token's own ...
    float before = 0.0f;
#pragma unroll
    for (int bt = 1; bt < CT; ++bt) {
      if (lane < C) before += l.row_tile[buf][bt - 1][lane];
      const float s = suffix_sum(lane >= 16 * bt ? before : 0.0f, lane);
      if (lane / 16 == bt) mine += s;
    }
    // ... and those of its own
    if (lane < C) {
      const int bt = lane / 16;
      for (int it = bt; it < CT; ++it) mine += l.col_tile[buf][it * (it + 1) / 2 + bt][lane % 16];
    }
  } else {
    const float run = prefix_sum(v, lane);
    all = lane_of(run, C - 1);
    mine = __shfl_up(run, 1);
    if (lane == 0) mine = 0.0f;
  }
  const int tok = tb + lane;
  if (lane < C && tok < t1) m.mass[mb * p.T + tok] = mine;
  if (lane == 0) m.mass_chunk[mb * ((p.T + C - 1) / C) + tb / C] = all;
}

// One workgroup's march. MASS: 0 none, 1 the rows' part of the decay's gradient
// (forward), 2 the sources' part (reverse). OUT false: the segment's own state only.
template <typename S, bool BF, int NKT, int NV, int W, Rows R, bool REV, int MASS, bool OUT>
__device__ __forceinline__ void march(const DaParams& p, const DaMarch& m, int block,
                                      typename S::template Lds<OUT, MASS>& l) {
  constexpr bool VEC = R != Rows::Elements, CUT = R == Rows::Cut;
  using O = Op<BF>;
  using E = typename O::E;
  using Pair = typename O::Pair;
  constexpr int C = S::C, CT = S::CT, THREADS = S::kThreads;
  constexpr int kRead = MASS == 0 ? O::kRead : O::kState;  // the decay's gradient is f32
  constexpr int kDecayWave = W - 1, kMassWave = W - 2;     // they have the fewest tiles of scores
  const int tid = int(threadIdx.x), lane = tid & 63, g = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  const int ncb = (m.dz + S::BV - 1) / S::BV, BH = p.B * p.H;
  const int cb = block % ncb, bh = block / ncb % BH, seg_m = block / ncb / BH;
  if (seg_m >= (OUT ? p.segments : p.segments - 1)) return;
  const int b = bh / p.H, h = bh % p.H;
  const int seg = REV ? p.segments - 1 - seg_m : seg_m;
  const int t0 = seg * p.seg_tokens, t1 = min(p.T, t0 + p.seg_tokens);
  int len = p.T;
  if (p.lengths) len = min(max(p.lengths[b], 0), p.T);
  const int live = max(min(len, t1) - t0, 0), end = min(len, t1);
  const int nc = (live + C - 1) / C;
  const int c0 = cb * S::BV, wc0 = 16 * NV * wave;  // first column of the workgroup, and of the wave within it
  const int64_t state = int64_t(p.dk) * p.dv;
  // Tiles of x, y and the state that hold nothing, and waves without columns, are left out where a product
  // is dear (f32: 32 cycles a 16x16x4; 333 tokens of 48 x 80: gradient 25 us, 32 without); with bf16 the
  // branches cost more than the products (8192 tokens of 128 x 128: 53 us, 56 with).
  const int pairs = BF ? NKT / 2 : (m.dx + 31) / 32;
  const int busy = BF ? W : min(W, (m.dz - c0 + 16 * NV - 1) / (16 * NV));
  const bool mine = BF || wave < busy;

  const float* gb = p.g + int64_t(b) * p.gb + int64_t(h) * p.gh;

  // The state: tile kt holds rows 16 kt + 4 g + r, column c0 + wc0 + 16 n + c.
  auto state_row = [&](int kt, int r) { return 16 * kt + 4 * g + r; };
  const uint32_t sr = uint32_t(m.sr), sc = uint32_t(m.sc);  // of at most 256 x 256 floats
  const uint32_t st_at = 4 * uint32_t(g) * sr + uint32_t(c0 + wc0 + c) * sc;
  auto state_at = [&](int kt, int n, int r) { return st_at + (16 * kt + r) * sr + 16 * n * sc; };
  auto state_is = [&](int kt, int n, int r) { return state_row(kt, r) < m.dx && c0 + wc0 + 16 * n + c < m.dz; };
  f32x4 st[NKT][NV];
  {
    const float* from = !OUT ? nullptr : seg_m == 0 ? (m.first ? m.first + bh * state : nullptr)
                                                    : m.seg + (int64_t(seg_m - 1) * BH + bh) * state;
#pragma unroll
    for (int kt = 0; kt < NKT; ++kt)
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) st[kt][n][r] = from && state_is(kt, n, r) ? from[state_at(kt, n, r)] : 0.0f;
  }

  Tile<BF, S::DX, THREADS, R> tx, ty;
  Tile<BF, S::BV, THREADS, R> tz, tw;
  if constexpr (OUT) tx.init(m.x, b, h, m.dx, 0);
  ty.init(m.y, b, h, m.dx, 0);
  tz.init(m.z, b, h, m.dz, c0);
  if constexpr (MASS != 0) tw.init(m.w, b, h, m.dz, c0);
  float rg = 0.0f;
  auto first_token = [&](int ci) { return t0 + (REV ? nc - 1 - ci : ci) * C; };
  auto fetch = [&](int ci) {
    const int tb = first_token(ci), left = end - tb;
    if constexpr (OUT) tx.fetch(tb, left);
    ty.fetch(tb, left);
    tz.fetch(tb, left);
    if constexpr (MASS != 0) tw.fetch(tb, left);
  };
  auto fetch_decay = [&](int ci) {
    const int t = first_token(ci) + lane;
    rg = lane < C && t < end ? gb[int64_t(t) * p.gt] : 0.0f;
  };

  // The state at the start of span k of the segment, to be met by its adjoint there (marches 0 and 1 hold both
  // alike, transposed: a lane's four rows are next to each other).
  auto mark = [&](int k) {
    if constexpr (MASS != 0) {
      const int pitch = (m.dx + 3) & ~3, col = c0 + wc0 + c;
      float* to = m.marks + ((int64_t(bh) * p.segments + seg) * (p.spans - 1) + (k - 1)) * mark_floats(p.dk, p.dv);
#pragma unroll
      for (int kt = 0; kt < NKT; ++kt)
#pragma unroll
        for (int n = 0; n < NV; ++n)
          if (16 * kt + 4 * g < pitch && col + 16 * n < m.dz)
            *reinterpret_cast<f32x4*>(to + (col + 16 * n) * pitch + 16 * kt + 4 * g) = st[kt][n];
    }
  };
  // What a decay carries in all at a segment's border: the state against its adjoint there, `adj`.
  auto carried = [&](const float* adj, int border) {
    if constexpr (MASS == 1) {
      double s = 0.0;
      if (adj) {
#pragma unroll
        for (int kt = 0; kt < NKT; ++kt)
#pragma unroll
          for (int n = 0; n < NV; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (state_is(kt, n, r)) s += double(st[kt][n][r]) * double(adj[state_at(kt, n, r)]);
      }
      s = lane_of(prefix_sum(s, lane), 63);
      if (lane == 0) l.cross[wave] = s;
      __syncthreads();
      if (tid == 0) {
        s = 0.0;
        for (int i = 0; i < W; ++i) s += l.cross[i];
        m.cross[(int64_t(cb) * BH + bh) * (int64_t(p.segments) * p.spans + 1) + border] = s;
      }
      __syncthreads();
    }
  };

  if (nc > 0) {
    fetch(0);
    if (wave == kDecayWave) fetch_decay(0);
  }
  if constexpr (MASS == 1) {
    // Between here and the segment's end the carried sum is kept by differences.
    if (seg_m > 0) carried(p.m[1].seg + (int64_t(p.segments - 1 - seg_m) * BH + bh) * state, seg * p.spans);
  }
  // chunk ci's tiles from registers to LDS: x and w, which only the first half of a chunk reads, and y and z
  auto put = [&](int ci) {
    const int left = end - first_token(ci), buf = ci % S::NB;
    if constexpr (OUT) {
      tx.mend(left, m.dx < S::DX, m.dx % O::kPiece != 0);
      tx.template store<true>(l.x, S::SX);
    }
    ty.mend(left, m.dx < S::DX, m.dx % O::kPiece != 0);
    ty.store(l.y[buf], S::SY);
    tz.mend(left, m.dz < c0 + S::BV, m.dz % O::kPiece != 0);
    if constexpr (OUT) {
      // An infinity or NaN in z times a score of zero would reach rows that do not see its token: such
      // values are left out of the products, and what does see them turns into NaN at the end.
      if (__builtin_expect(!tz.finite(), 0)) {
        l.odd[ci & 1] = 1;
        tz.keep_finite(l.from[ci & 1], REV);
      }
    }
    tz.store(l.z[buf], S::SZ);
    if constexpr (MASS != 0) {
      tw.mend(left, m.dz < c0 + S::BV, m.dz % O::kPiece != 0);
      tw.store(l.w, S::SW);
    }
  };
  // Results of the operands' type leave through LDS, a chunk late, by whole rows and past the caches: a
  // wave's 16 columns alone are 32 bytes of a bf16 row, and lines the L2s still held at the kernel's end
  // would have to be written then (8192 tokens of 128 x 128: 78.0 us, 81.8 straight from the accumulators).
  constexpr int PR = S::BV / O::kPiece, STEP = THREADS / PR, NO = (C + STEP - 1) / STEP;
  const bool staged = VEC && OUT && !(BF && m.out_f32);
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  u32x4 held[NO];
  auto out_read = [&] {
    if constexpr (OUT) {
      if (!staged) return;
#pragma unroll
      for (int n = 0; n < NO; ++n)
        held[n] = *reinterpret_cast<const u32x4*>(l.out + min(tid / PR + n * STEP, C - 1) * S::SW +
                                                  tid % PR * O::kPiece);
    }
  };
  auto out_write = [&](int ci) {
    if constexpr (OUT) {
      const int tb = first_token(ci), col = tid % PR * O::kPiece;
      if (!staged || c0 + col >= m.dz) return;
      const int64_t row_bytes = int64_t(p.H) * m.dz * int64_t(sizeof(E));
      char* to = static_cast<char*>(m.out) + (((int64_t(b) * p.T + tb) * p.H + h) * m.dz + c0) * int64_t(sizeof(E));
      const uint32_t off = uint32_t(tid / PR) * uint32_t(row_bytes) + uint32_t(col) * uint32_t(sizeof(E));
#pragma unroll
      for (int n = 0; n < NO; ++n) {
        const int t = tid / PR + n * STEP;
        if (tb + C > end && t >= end - tb) held[n] = u32x4{0, 0, 0, 0};
        if (t >= C || tb + t >= t1) continue;
        char* at = to + n * STEP * row_bytes + off;
        const int exist = m.dz - (c0 + col);
        if (!CUT || m.dz % O::kPiece == 0) {
          st_stream(reinterpret_cast<u32x4*>(at), held[n]);
        } else if (exist >= O::kPiece) {
          __builtin_memcpy(at, &held[n], 16);  // at any alignment
        } else {
#pragma unroll
          for (int e = 0; e < O::kPiece - 1; ++e) {
            const uint32_t w = BF ? held[n][e / 2] >> 16 * (e & 1) : held[n][e];
            if (e < exist) reinterpret_cast<E*>(at)[e] = BF ? E(uint16_t(w)) : E(__uint_as_float(w));
          }
        }
      }
    }
  };
  if constexpr (OUT) {
    if (tid < 2) l.odd[tid] = 0;
    for (int i = tid; i < 2 * S::BV; i += THREADS) l.from[i / S::BV][i % S::BV] = C;
  }
  float decays = 1.0f;
  int next_k = REV ? p.spans - 1 : 1;  // the next span's border on the way, and its chunk
  if constexpr (MASS == 2) {  // (those behind the row's last token)
    for (; next_k > 0 && next_k * p.span_chunks >= nc; --next_k) mark(next_k);
  }
  int next_mark = next_k > 0 && next_k < p.spans ? next_k * p.span_chunks : -1;
  __syncthreads();
  if (nc > 0) {
    if (wave == kDecayWave) {
      chunk_decays<REV, C>(l.dec[0], rg, m.scale_out, m.scale_src, lane);
      if (nc > 1) fetch_decay(1);
    }
    put(0);
    if (nc > 1) fetch(1);
    __syncthreads();
  }
  for (int ci = 0; ci < nc; ++ci) {
    const int tb = first_token(ci);
    typename S::Decays& dec = l.dec[ci & 1];
    E* const ly = l.y[ci % S::NB];
    E* const lz = l.z[ci % S::NB];
    const float total = dec.total;

    f32x4 acc[OUT ? NV : 1][OUT ? CT : 1];  // out transposed: column wc0 + 16 n + 4 g + r, row 16 it + c
    if constexpr (OUT) {
      if (tid == 0) l.odd[(ci + 1) & 1] = 0;
      if (ci > 0) out_read();
      // scores: the tiles on and on one side of the diagonal, in turn over the waves, as [row][source]; a
      // wave's tiles side by side
      constexpr int kTurns = (S::TILES + W - 1) / W;
      auto tiles = [&](auto count) {
        constexpr int N = decltype(count)::value;
        int it[N], jt[N];
        f32x4 s[N], a[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
          int hi = 0, lo = wave + i * W;
          while (lo > hi) lo -= ++hi;
          it[i] = REV ? lo : hi;
          jt[i] = REV ? hi : lo;
          s[i] = a[i] = zero4();
        }
        float2 gi[N];
        f32x4 gj[N][2];
#pragma unroll
        for (int i = 0; i < N; ++i) {
          gi[i] = dec.g[16 * it[i] + c];
          gj[i][0] = *reinterpret_cast<const f32x4*>(&dec.g[16 * jt[i] + 4 * g]);
          gj[i][1] = *reinterpret_cast<const f32x4*>(&dec.g[16 * jt[i] + 4 * g + 2]);
        }
        constexpr int A = NKT / 2 < 4 ? NKT / 2 : N == 1 ? 4 : 2;  // products whose operands are read at once
#pragma unroll
        for (int k2 = 0; k2 < NKT / 2; k2 += A) {
          if (!BF && k2 >= pairs) continue;
          Pair y[A][N], x[A][N];
#pragma unroll
          for (int k = 0; k < A; ++k)
#pragma unroll
            for (int i = 0; i < N; ++i) {
              y[k][i] = O::row_pair(ly + (16 * jt[i] + c) * S::SY + 32 * (k2 + k), g);
              x[k][i] = O::paired_row(l.x + (16 * it[i] + c) * S::SX + 32 * (k2 + k), g);
            }
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int k = 0; k < A; ++k)
#pragma unroll
            for (int i = 0; i < N; ++i) s[i] = O::mma(y[k][i], x[k][i], s[i]);
        }
        if constexpr (MASS == 1) {
          // what a row takes from a source: decay (x_i . y_j) (w_i . z_j), this workgroup's columns of the second
#pragma unroll
          for (int k2 = 0; k2 < S::BV / 32; k2 += 2) {
            if (!BF && c0 + 32 * k2 >= m.dz) continue;
            Pair z[2][N], w[2][N];
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int i = 0; i < N; ++i) {
                z[k][i] = O::row_eight(lz + (16 * jt[i] + c) * S::SZ + 32 * (k2 + k), g);
                w[k][i] = O::row_eight(l.w + (16 * it[i] + c) * S::SW + 32 * (k2 + k), g);
              }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int i = 0; i < N; ++i) a[i] = O::mma(z[k][i], w[k][i], a[i]);
          }
        }
        const float scale = m.scale_src * m.scale_out;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int row = 16 * it[i] + c, j0 = 16 * jt[i] + 4 * g;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float d = (gi[i].x - gj[i][r / 2][2 * (r & 1)]) + (gi[i].y - gj[i][r / 2][2 * (r & 1) + 1]);
            s[i][r] *= scale * exp2_hw(REV ? -d : d);
          }
          if (it[i] == jt[i]) {  // the tiles on the diagonal: sources a row does not see
#pragma unroll
            for (int r = 0; r < 4; ++r) s[i][r] = (REV ? j0 + r >= row : j0 + r <= row) ? s[i][r] : 0.0f;
          }
          if constexpr (BF) {
            Pair parts[O::kScore];
            O::template split<O::kScore>(s[i], s[i], parts);
#pragma unroll
            for (int n = 0; n < O::kScore; ++n)
              *reinterpret_cast<uint2*>(l.score[n] + row * S::SP + O::paired(j0)) = make_uint2(parts[n].x, parts[n].y);
          } else {
            O::put4(l.score[0] + row * S::SP + O::paired(j0), s[i]);
          }
          if constexpr (MASS == 1) {
            float sum = 0.0f, before[4];  // of the lane's sources, and of those before each
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              before[r] = sum;
              sum += j0 + r < row ? a[i][r] * s[i][r] : 0.0f;
            }
            // ... of the lane groups before this one
            const Two two = of_pair(sum), halves = of_halves(two.a + two.b);
            const float groups = (g & 1 ? two.a : 0.0f) + (g >= 2 ? halves.a : 0.0f);
            if (g == 3) l.row_tile[ci & 1][jt[i]][row] = halves.a + halves.b;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float v = group_sum(j0 + r <= row ? groups + before[r] : 0.0f);
              if (c == 15) l.col_tile[ci & 1][wave + i * W][4 * g + r] = v;
            }
          }
        }
      };
      if (wave + (kTurns - 1) * W < S::TILES) tiles(std::integral_constant<int, kTurns>{});
      else if constexpr (kTurns > 1) tiles(std::integral_constant<int, kTurns - 1>{});
      if (ci > 0) out_write(ci - 1);
      if (wave == kDecayWave && ci + 1 < nc) {
        chunk_decays<REV, C>(l.dec[(ci + 1) & 1], rg, m.scale_out, m.scale_src, lane);
        if (ci + 2 < nc) fetch_decay(ci + 2);
      }
      if constexpr (MASS != 0) {
        if (wave == kMassWave && ci > 0)
          chunk_mass<REV, MASS, CT, S::TILES>(p, m, l, (ci - 1) & 1, busy, first_token(ci - 1), t1, cb, bh, lane);
        if (m.chunk_decay && cb == 0 && tid == 0)
          m.chunk_decay[int64_t(bh) * ((p.T + C - 1) / C) + tb / C] = total;
      }
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int it = 0; it < CT; ++it) acc[n][it] = zero4();
      // rows against the state, each product's rows read ahead of the one before
      if (mine) {
        Pair x[2][CT];
        auto rows_of = [&](int k2) {
#pragma unroll
          for (int it = 0; it < CT; ++it) x[k2 & 1][it] = O::paired_row(l.x + (16 * it + c) * S::SX + 32 * k2, g);
        };
        rows_of(0);
#pragma unroll
        for (int k2 = 0; k2 < NKT / 2; ++k2) {
          if (!BF && k2 >= pairs) continue;
          if (k2 + 1 < NKT / 2) rows_of(k2 + 1);
          __builtin_amdgcn_sched_barrier(0);
          Pair sp[NV][kRead];
#pragma unroll
          for (int n = 0; n < NV; ++n) O::template split<kRead>(st[2 * k2][n], st[2 * k2 + 1][n], sp[n]);
#pragma unroll
          for (int q = kRead - 1; q >= 0; --q)
#pragma unroll
            for (int it = 0; it < CT; ++it)
#pragma unroll
              for (int n = 0; n < NV; ++n) acc[n][it] = O::mma(sp[n][q], x[k2 & 1][it], acc[n][it]);
        }
#pragma unroll
        for (int it = 0; it < CT; ++it) {
          const float f = dec.row[16 * it + c];
          float mass = 0.0f;
#pragma unroll
          for (int n = 0; n < NV; ++n) {
            acc[n][it] = decayed(acc[n][it], f);
            if constexpr (MASS != 0) {
              const f32x4 w = O::four(l.w + (16 * it + c) * S::SW + wc0 + 16 * n + 4 * g);
#pragma unroll
              for (int r = 0; r < 4; ++r) mass += acc[n][it][r] * w[r];
            }
          }
          if constexpr (MASS != 0) {
            mass = groups_sum(mass);
            if (g == 0) l.part[ci & 1][wave][16 * it + c] = mass;
          }
        }
      }
      __syncthreads();
    } else if (wave == kDecayWave && ci + 1 < nc) {
      chunk_decays<REV, C>(l.dec[(ci + 1) & 1], rg, m.scale_out, m.scale_src, lane);
      if (ci + 2 < nc) fetch_decay(ci + 2);
    }

    // sources: into the rows of the chunk, and into the state, half a chunk at a time; what a product
    // reads is on its way while the ones before it run
    constexpr int YA = NKT < 4 ? NKT : 4;  // columns of y read at once
    decays *= total;
#pragma unroll
    for (int j2 = 0; j2 < CT / 2; ++j2) {
      if (mine) {
        Pair z[NV], zs[NV][O::kState], y[2][YA];
        Pair sc[OUT ? CT : 1][O::kScore];
        f32x4 f0, f1;
        auto columns_of = [&](int kt) {
#pragma unroll
          for (int i = 0; i < YA; ++i) y[kt / YA & 1][i] = O::column_pair(ly, S::SY, 32 * j2, 16 * (kt + i), g, c);
        };
#pragma unroll
        for (int n = 0; n < NV; ++n) z[n] = O::column_pair(lz, S::SZ, 32 * j2, wc0 + 16 * n, g, c);
        f0 = *reinterpret_cast<const f32x4*>(dec.src + 32 * j2 + 4 * g);
        f1 = *reinterpret_cast<const f32x4*>(dec.src + 32 * j2 + 16 + 4 * g);
        if constexpr (OUT) {
#pragma unroll
          for (int it = 0; it < CT; ++it)
            if (REV ? it <= 2 * j2 + 1 : it >= 2 * j2) {
#pragma unroll
              for (int q = 0; q < O::kScore; ++q)
                sc[it][q] = O::paired_row(l.score[q] + (16 * it + c) * S::SP + 32 * j2, g);
            }
        }
        columns_of(0);
        __builtin_amdgcn_sched_barrier(0);
        if (j2 == 0) {
#pragma unroll
          for (int kt = 0; kt < NKT; ++kt)
#pragma unroll
            for (int n = 0; n < NV; ++n) {
              // (not where a segment's own state is formed: it starts from zero, and this product cost 52 us for 44
              // in the gradient of 4 x 4096 tokens of 8 heads of 128)
              if constexpr (OUT) st[kt][n] = decayed(st[kt][n], total);
              else st[kt][n] *= total;
            }
        }
#pragma unroll
        for (int n = 0; n < NV; ++n) O::template split<O::kState>(O::low(z[n]) * f0, O::high(z[n]) * f1, zs[n]);
        if constexpr (OUT) {
#pragma unroll
          for (int q = O::kScore - 1; q >= 0; --q)
#pragma unroll
            for (int it = 0; it < CT; ++it) {
              if (REV ? it <= 2 * j2 + 1 : it >= 2 * j2) {
                // the one tile of a pair beyond the diagonal was not written
                if (REV ? it == 2 * j2 + 1 : it == 2 * j2) {
                  if constexpr (BF) {
                    if (REV) sc[it][q].x = sc[it][q].y = 0; else sc[it][q].z = sc[it][q].w = 0;
                  } else {
                    if (REV) sc[it][q].a = zero4(); else sc[it][q].b = zero4();
                  }
                }
#pragma unroll
                for (int n = 0; n < NV; ++n) acc[n][it] = O::mma(z[n], sc[it][q], acc[n][it]);
              }
            }
        }
#pragma unroll
        for (int kt = 0; kt < NKT; kt += YA) {
          if (!BF && kt / 2 >= pairs) continue;
          if (kt + YA < NKT) columns_of(kt + YA);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int q = O::kState - 1; q >= 0; --q)
#pragma unroll
            for (int i = 0; i < YA; ++i)
#pragma unroll
              for (int n = 0; n < NV; ++n) st[kt + i][n] = O::mma(y[kt / YA & 1][i], zs[n][q], st[kt + i][n]);
        }
      }
      if (j2 == 0 && S::NB == 2 && ci + 1 < nc) {
        put(ci + 1);
        if (ci + 2 < nc) fetch(ci + 2);
      }
    }

    if constexpr (OUT) {
      if (__builtin_expect(l.odd[ci & 1] != 0, 0)) {
        int* from = l.from[ci & 1] + wc0;  // this wave's own columns
#pragma unroll
        for (int n = 0; n < NV; ++n) {
          const bool lost = from[16 * n + c] < C;
#pragma unroll
          for (int kt = 0; kt < NKT; ++kt)
#pragma unroll
            for (int r = 0; r < 4; ++r) st[kt][n][r] = lost ? NAN : st[kt][n][r];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int first = from[16 * n + 4 * g + r];
#pragma unroll
            for (int it = 0; it < CT; ++it) {
              const int row = REV ? C - 1 - (16 * it + c) : 16 * it + c;
              acc[n][it][r] = row >= first ? NAN : acc[n][it][r];
            }
          }
        }
        for (int i = lane; i < 16 * NV; i += kWave) from[i] = C;
      }
      if constexpr (MASS != 0) {
        if ((REV ? nc - 1 - ci : ci + 1) == next_mark) {
          mark(next_k);
          next_k += REV ? -1 : 1;
          next_mark = next_k > 0 && next_k < p.spans ? next_k * p.span_chunks : -1;
        }
      }
      // a token's rows of out
      if (staged) {
#pragma unroll
        for (int it = 0; it < CT; ++it)
#pragma unroll
          for (int n = 0; n < NV; ++n) O::put4(l.out + (16 * it + c) * S::SW + wc0 + 16 * n + 4 * g, acc[n][it]);
      } else {
        const int again = anew(tid), c = again & 15, g = again >> 4 & 3;
#pragma unroll
        for (int it = 0; it < CT; ++it) {
          const int t = tb + 16 * it + c;
          const int64_t row = ((int64_t(b) * p.T + t) * p.H + h) * m.dz + c0;
#pragma unroll
          for (int n = 0; n < NV; ++n) {
            const int at = wc0 + 16 * n + 4 * g;
            const f32x4 v = t >= len ? zero4() : acc[n][it];
            // (VEC: f32 results of bf16 operands, for a sum over the heads that share them)
            if (VEC && (!CUT || m.dz % 4 == 0)) {
              if (t < t1 && c0 + at < m.dz) *reinterpret_cast<f32x4*>(static_cast<float*>(m.out) + row + at) = v;
              continue;
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              if (t < t1 && c0 + at + r < m.dz) {
                if (!BF || m.out_f32) static_cast<float*>(m.out)[row + at + r] = v[r];
                else static_cast<uint16_t*>(m.out)[row + at + r] = f32_to_bf16_rne(v[r]);
              }
            }
          }
        }
      }
    }
    __syncthreads();
    if (S::NB == 1 && ci + 1 < nc) {
      put(ci + 1);
      if (ci + 2 < nc) fetch(ci + 2);
      __syncthreads();
    }
  }

  if (OUT && nc > 0) {
    out_read();
    out_write(nc - 1);
  }
  if constexpr (OUT) {
    // tokens past the row's length, in chunks that were not marched
    const int from = t0 + nc * C;
    const int width = min(S::BV, m.dz - c0), rest = max(t1 - from, 0);
    for (int q = tid; q < rest * width; q += THREADS) {
      const int64_t at = ((int64_t(b) * p.T + from + q / width) * p.H + h) * m.dz + c0 + q % width;
      if (!BF || m.out_f32) static_cast<float*>(m.out)[at] = 0.0f;
      else static_cast<uint16_t*>(m.out)[at] = 0;
    }
    if constexpr (MASS != 0) {
      const int64_t mb = (int64_t(cb) * BH + bh);
      const int chunks = (p.T + C - 1) / C;
      if (nc > 0 && wave == kMassWave)
        chunk_mass<REV, MASS, CT, S::TILES>(p, m, l, (nc - 1) & 1, busy, first_token(nc - 1), t1, cb, bh, lane);
      for (int q = tid; q < rest; q += THREADS) m.mass[mb * p.T + from + q] = 0.0f;
      for (int q = tid; q < (rest + C - 1) / C; q += THREADS) {
        m.mass_chunk[mb * chunks + from / C + q] = 0.0f;
        if (m.chunk_decay && cb == 0) m.chunk_decay[int64_t(bh) * chunks + from / C + q] = 1.0f;
      }
    }
  }

  if constexpr (MASS == 1) {
    for (int k = p.spans - 1; k > 0 && k * p.span_chunks > nc; --k) mark(k);  // (those behind the row's last token)
  }
  if (MASS == 1 && seg == p.segments - 1)
    carried(p.m[1].first ? p.m[1].first + bh * state : nullptr, p.segments * p.spans);
  float* to = OUT ? (seg_m == p.segments - 1 && m.last ? m.last + bh * state : nullptr)
                  : m.seg + (int64_t(seg_m) * BH + bh) * state;
  if (to) {
#pragma unroll
    for (int kt = 0; kt < NKT; ++kt)
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (state_is(kt, n, r)) to[state_at(kt, n, r)] = st[kt][n][r];
  }
  if (!OUT && tid == 0 && cb == 0) m.seg_decay[int64_t(seg_m) * BH + bh] = decays;
}

template <bool BF, int NKT, int NV, int W, Rows R>
__global__ __launch_bounds__(W * kWave) void march_forward(DaParams p) {
  using S = Shape<BF, NKT, NV, W>;
  __shared__ typename S::Out l;
  march<S, BF, NKT, NV, W, R, false, 0, true>(p, p.m[0], blockIdx.x, l);
}

// first + blockIdx.y is the march of a gradient: 0 grad_q, 1 grad_k, 2 grad_v.
template <bool BF, int NKT, int NV, int W, Rows R>
__global__ __launch_bounds__(W * kWave) void march_gradient(DaParams p, int first) {
  using S = Shape<BF, NKT, NV, W>;
  __shared__ typename S::Mass l;
  const int which = first + int(blockIdx.y);
  if (which == 0) march<S, BF, NKT, NV, W, R, false, 1, true>(p, p.m[0], blockIdx.x, l);
  else if (which == 1) march<S, BF, NKT, NV, W, R, true, 2, true>(p, p.m[1], blockIdx.x, l);
  else march<S, BF, NKT, NV, W, R, true, 0, true>(p, p.m[2], blockIdx.x, l);
}

// Each segment's own state. A gradient needs two: the state (march 0's) and its
// adjoint (march 1's, which march 2 shares).
template <bool BF, int NKT, int NV, int W, Rows R>
__global__ __launch_bounds__(W * kWave) void march_local(DaParams p) {
  using S = Shape<BF, NKT, NV, W>;
  __shared__ typename S::Local l;
  if (blockIdx.y == 0) march<S, BF, NKT, NV, W, R, false, 0, false>(p, p.m[0], blockIdx.x, l);
  else march<S, BF, NKT, NV, W, R, true, 0, false>(p, p.m[1], blockIdx.x, l);
}

// Marches first .. first + count - 1 of one shape (local: their segments' own states).
template <bool BF, int NKT, int W, Rows R>
void launch_shape(const DaParams& p, int first, int count, bool local, hipStream_t stream) {
  constexpr int BV = 16 * W;
  int64_t columns = 0;
  for (int i = first; i < first + count; ++i) columns = std::max<int64_t>(columns, (p.m[i].dz + BV - 1) / BV);
  const int64_t blocks = columns * p.B * p.H * (local ? p.segments - 1 : p.segments);
  const dim3 grid{unsigned(blocks), unsigned(count), 1};
  if (local) march_local<BF, NKT, 1, W, R><<<grid, W * kWave, 0, stream>>>(p);
  else if (p.marches == 1) march_forward<BF, NKT, 1, W, R><<<grid, W * kWave, 0, stream>>>(p);
  else march_gradient<BF, NKT, 1, W, R><<<grid, W * kWave, 0, stream>>>(p, first);
}

template <bool BF, Rows R>
hipError_t launch_marches(const DaParams& p, int first, int count, bool local, hipStream_t stream) {
  // the class of the widest: marches launched together may differ
  int dx = 0, dz = 0;
  for (int i = first; i < first + count; ++i) {
    dx = std::max(dx, p.m[i].dx);
    dz = std::max(dz, p.m[i].dz);
  }
  const int tiles = march_tiles(dx);
  if (march_waves(dz) == 4) {
    if (tiles == 2) launch_shape<BF, 2, 4, R>(p, first, count, local, stream);
    else if (tiles == 4) launch_shape<BF, 4, 4, R>(p, first, count, local, stream);
    else if (tiles == 8) launch_shape<BF, 8, 4, R>(p, first, count, local, stream);
    else launch_shape<BF, 16, 4, R>(p, first, count, local, stream);
  } else {
    if (tiles == 2) launch_shape<BF, 2, 8, R>(p, first, count, local, stream);
    else if (tiles == 4) launch_shape<BF, 4, 8, R>(p, first, count, local, stream);
    else if (tiles == 8) launch_shape<BF, 8, 8, R>(p, first, count, local, stream);
    else launch_shape<BF, 16, 8, R>(p, first, count, local, stream);
  }
  return hipGetLastError();
}

}  // namespace
}  // namespace sx
