// sx_attention.hpp: descriptors of the linear-attention operators, shared by the
// host dispatch (sx_api.cpp) and their kernels (decay_attention.hip,
// head_rotate.hip). Internal to libsx_scan.so.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sx_scan.h"

namespace sx {

// One tensor of per-head rows, [B, T, heads, D] with element strides. Head h of
// the call reads head h / rep of it.
struct HeadView {
  const void* p;
  int64_t sb, st, sh, sd;
  int rep;
  int unit;  // unit sd, and a row holds 16 bytes at least: pieces of it can be read at any alignment
};

// ---------------------------------------------------------------- decay attention

// A march along the tokens with the state S [Dx, Dz] of one head: for each token
// in march order
//   S = decay S + scale_src y z^T,   out = scale_out S^T x
// where y has the width of x (Dx) and out the width of z (Dz). The forward
// operator is (x, y, z) = (q, k, v); its gradients are marches as well:
//   grad_q: (grad_out, v, k), forward, on the transposed state
//   grad_k: (v, grad_out, q), reverse, on the transposed adjoint
//   grad_v: (k, q, grad_out), reverse, on the adjoint
// In a reverse march a token's decay is applied after its output is read, so
// out at t sees source s >= t through the decays of t+1 .. s.
struct DaMarch {
  HeadView x, y, z;
  HeadView w;           // grad_q: q; grad_k: k: the row each output meets in the decay's gradient (p == nullptr: none)
  int dx, dz;
  float scale_out, scale_src;
  void* out;            // element (b, t, h, d) at ((b * T + t) * H + h) * dz + d; nullptr: states only
  int out_f32;          // out is f32 whatever the inputs' type
  int64_t sr, sc;       // element (r, c) of a state [Dx, Dz] in memory
  const float* first;   // state the march starts from, one per (b, h), [Dk, Dv] (nullptr: zero)
  float* last;          // state it ends with (nullptr: not wanted)
  float* seg;           // segment states, [segments - 1][B * H][Dk, Dv]: of segment m's sources alone after the
                        // local pass, at the start of segment m + 1 after the carry
  float* seg_decay;     // [segments - 1][B * H]: product of a segment's decays
  float* mass;          // [column blocks][B * H][T]: the part of the decay's gradient that this march sees
  float* mass_chunk;    // [column blocks][B * H][chunks]: a chunk's mass against the state it entered with
  double* cross;        // [column blocks][B * H][segments * spans + 1]: the state against its adjoint at the spans'
                        // borders (but the first)
  float* marks;         // [B * H][segments][spans - 1][dz][dx, to a multiple of 4]: the state at the spans' borders
                        // within segments (grad_q, grad_k)
  float* chunk_decay;   // [B * H][chunks]: product of a chunk's decays (written by column block 0; nullptr: no)
};

struct DaParams {
  int B, T, H;
  int dk, dv;
  const float* g;       // log decay, strides below (gb = gt = 0: one value a head)
  int64_t gb, gt, gh;
  const int32_t* lengths;  // [B] or nullptr
  int bf16;
  int segments;         // the tokens split into this many segments of seg_tokens
  int seg_tokens;       // a multiple of the chunk
  int spans;            // and a segment into this many spans of span_chunks chunks (a gradient)
  int span_chunks;
  int marches;          // 1 (forward) or 3 (gradient)
  DaMarch m[3];
};

int decay_attention_chunk(bool bf16);
// Floats of a state in DaMarch::marks.
__host__ __device__ inline int64_t mark_floats(int dk, int dv) { return int64_t(dk) * ((dv + 3) & ~3); }
// Workgroups a head needs for `dz` columns.
int decay_attention_column_blocks(int dz);
// A march's shape: 16-row tiles of the state (2, 4, 8 or 16), and waves of 16 columns (4 or 8).
int march_tiles(int dx);
int march_waves(int dz);
hipError_t launch_marches_bf16(const DaParams& p, int first, int count, bool local, hipStream_t stream);
hipError_t launch_marches_bf16_cut(const DaParams& p, int first, int count, bool local, hipStream_t stream);
hipError_t launch_marches_bf16_any(const DaParams& p, int first, int count, bool local, hipStream_t stream);
hipError_t launch_marches_f32(const DaParams& p, int first, int count, bool local, hipStream_t stream);
hipError_t launch_marches_f32_cut(const DaParams& p, int first, int count, bool local, hipStream_t stream);
hipError_t launch_marches_f32_any(const DaParams& p, int first, int count, bool local, hipStream_t stream);
// How the tokens are split: sets segments and seg_tokens, spans and span_chunks.
void decay_attention_split(DaParams& p);
hipError_t launch_decay_attention(const DaParams& p, hipStream_t stream);

// The decay's gradient from the masses of the grad_q march (rows) and the grad_k
// march (sources): grad_g [B, T, H], or [H] summed over tokens when per_head.
struct DaDecayGrad {
  int B, T, H, dk, dv;
  int chunk, chunks, blocks;   // blocks: column blocks of both marches
  const float* g;
  int64_t gb, gt, gh;
  const int32_t* lengths;
  const float* rows;           // [blocks][B * H][T]
  const float* sources;
  const float* rows_chunk;     // [blocks][B * H][chunks]
  const float* sources_chunk;
  const float* chunk_decay;    // [B * H][chunks]
  int segments, seg_tokens, spans, span_chunks;
  double* cross;               // [blocks][B * H][segments * spans + 1], but of the first border
  const float* states;         // marks of the grad_q march and of the grad_k march
  const float* adjoints;
  const float* initial;        // nullptr: zero
  const float* grad_initial;
  double* partial;             // per_head: [segments * spans][B * H]
  float* grad_g;
  int per_head;
};
hipError_t launch_decay_grad(const DaDecayGrad& p, hipStream_t stream);

// out[b, t, i, d] = sum over the rep heads that share head i of src[b, t, i * rep + r, d].
struct DaShare {
  const float* src;
  void* out;
  int64_t rows;   // B * T * shared heads
  int rep, d;
  int bf16;
};
struct DaShares {
  DaShare s[3];
  int count;
};
hipError_t launch_share_sums(const DaShares& p, hipStream_t stream);

// One token of many requests.
struct DaStep {
  int B, H, dk, dv;
  HeadView q, k, v;     // st unused
  const float* g;
  int64_t gb, gh;
  float* state;         // slot s, head h at s * ss + h * sh, [dk, dv] row-major
  int64_t ss, sh, slots_in_pool;
  const int32_t* slots; // [B] or nullptr (row b uses slot b)
  float scale;
  int bf16;
  void* out;            // [B, H, dv] contiguous
};
hipError_t launch_decay_step(const DaStep& p, hipStream_t stream);

// ---------------------------------------------------------------- head norm and rotation

struct HrParams {
  int B, T, hq, hk, d, rot;
  HeadView q, k;        // inputs; rep = 1
  HeadView gq, gk;      // gradients of the outputs (backward only)
  const void* positions;
  int pos64;
  int64_t pb, pt;       // position strides (elements)
  const double* turns;  // [rot / 2], turns per position
  const float* qw;      // [d] or nullptr (ones)
  const float* kw;
  float eps;
  int neighbours;
  int bf16;
  void* out_q;          // contiguous [B, T, heads, d]: results, or gradients of q and k
  void* out_k;
  float* partial;       // backward: [2][workgroups][d]
  float* gqw;           // [d] or nullptr
  float* gkw;
  int tokens_q, tokens_k;  // tokens of a workgroup at a time (set by the launch)
};
int head_rotate_backward_groups(const HrParams& p);
hipError_t launch_head_rotate(const HrParams& p, hipStream_t stream);
hipError_t launch_head_rotate_backward(const HrParams& p, hipStream_t stream);

}  // namespace sx
