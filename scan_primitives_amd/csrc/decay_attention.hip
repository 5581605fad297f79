// decay_attention.hip: linear attention with a decay for each head, its
// gradient and its single-token form.
//
//   S[t] = exp(g[t]) S[t-1] + k[t] v[t]^T,   o[t] = scale S[t]^T q[t]
//
// Prompts and gradients run as marches over chunks of tokens (decay_march.hpp).
// Long sequences with few heads are split into segments: a first pass forms
// each segment's state from its own tokens, a carry joins them, and the second
// pass marches all segments at once from their true states.
#include "decay_march.hpp"

namespace sx {
namespace {

constexpr int kThreads = 256;
// Chunks over which the gradient of a decay is carried by differences. Of one decay a head, summed over 4096 tokens of
// 8 rows of 64 heads of 16 x 16 in f32, 3.8e-7 is lost against 64 bits, 8.7e-6 where spans are whole segments (128
// chunks); the marks cost 32 x 4096 tokens of 8 heads of 128 in bf16 1285 us for 1217.
constexpr int kSpanChunks = 8;

// Segment m's entry, its own state so far, becomes the state at the start of segment m + 1. Bound by
// memory: each entry is read and written once, eight read ahead of the chain (15 entries of 16 states of
// 128 x 128: 6.9 us).
__global__ __launch_bounds__(kThreads) void carry(DaParams p) {
  const DaMarch& m = p.m[blockIdx.y];
  const int64_t state = int64_t(p.dk) * p.dv, BH = int64_t(p.B) * p.H;
  const int64_t e = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (e >= BH * state) return;
  const int64_t bh = e / state;
  const int n = p.segments - 1;
  float s = m.first ? m.first[e] : 0.0f;
  constexpr int A = 8;  // entries read ahead of the chain
  for (int i = 0; i < n; i += A) {
    float v[A], d[A];
#pragma unroll
    for (int k = 0; k < A; ++k) {
      const int j = min(i + k, n - 1);
      v[k] = m.seg[j * BH * state + e];
      d[k] = m.seg_decay[j * BH + bh];
    }
#pragma unroll
    for (int k = 0; k < A; ++k) {
      if (i + k >= n) break;
      s = d[k] == 0.0f ? v[k] : fmaf(d[k], s, v[k]);  // nothing is left, of a state that is not finite either
      m.seg[(i + k) * BH * state + e] = s;
    }
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

// The state against its adjoint at the spans' borders within segments, from the marks that two marches left of
// them. One workgroup a border.
__global__ __launch_bounds__(kThreads) void span_cross(DaDecayGrad p) {
  __shared__ double l[kThreads];
  const int inner = p.segments * (p.spans - 1), tid = int(threadIdx.x);
  const int64_t at = blockIdx.x, bh = at / inner, BH = int64_t(p.B) * p.H, n = mark_floats(p.dk, p.dv);
  const int seg = int(at % inner) / (p.spans - 1), k = int(at % inner) % (p.spans - 1) + 1;
  const f32x4* s = reinterpret_cast<const f32x4*>(p.states + at * n);
  const f32x4* a = reinterpret_cast<const f32x4*>(p.adjoints + at * n);
  double v = 0.0;
#pragma unroll 4
  for (int64_t i = tid; i < n / 4; i += kThreads) {
    const f32x4 x = s[i], y = a[i];
#pragma unroll
    for (int e = 0; e < 4; ++e) v += double(x[e]) * double(y[e]);
  }
  v = block_sum(v, l);
  if (tid < p.blocks)
    p.cross[(tid * BH + bh) * (int64_t(p.segments) * p.spans + 1) + seg * p.spans + k] = tid == 0 ? v : 0.0;
}

// What passes a chunk from before to after it, Y, from what crosses the border
// before it, Z: Y = Z - (its rows' mass), the next Z = Y + (its sources' mass), and
// Y is zero outright where the chunk's decays multiply to zero. One workgroup a
// head and span, from the span's own Z. A span is few chunks (kSpanChunks), for
// what the two sums are rounded by adds up in Z, and stays when the state that
// it was rounded in has long decayed.
__global__ __launch_bounds__(kThreads) void decay_grad(DaDecayGrad p) {
  __shared__ double la[kThreads];
  __shared__ double ly[kSpanChunks];
  __shared__ double lw[kSpanChunks];
  __shared__ bool cuts[kSpanChunks];
  const int bh = blockIdx.x % (p.B * p.H), span = blockIdx.x / (p.B * p.H), tid = int(threadIdx.x);
  const int b = bh / p.H, h = bh % p.H, spans = p.segments * p.spans;
  const int64_t BH = int64_t(p.B) * p.H, state = int64_t(p.dk) * p.dv;
  int len = p.T;
  if (p.lengths) len = min(max(p.lengths[b], 0), p.T);
  auto sum_of = [&](const float* v, int64_t n, int64_t i) {
    double s = 0.0;
    for (int k = 0; k < p.blocks; ++k) s += double(v[(k * BH + bh) * n + i]);
    return s;
  };
  // its chunks (none, where the last segment is shorter)
  const int seg_chunks = p.seg_tokens / p.chunk, seg = span / p.spans;
  const int first = min(p.chunks, seg * seg_chunks + span % p.spans * p.span_chunks);
  const int last = min(p.chunks, min((seg + 1) * seg_chunks, first + p.span_chunks)), n = last - first;
  const int t0 = first * p.chunk, t1 = min(last * p.chunk, p.T);
  // What a token's decay carries within its chunk, and whether anything passes at all: where exp(g) = 0
  // neither does a gradient.
  struct Within {
    double v;
    bool passes;
  };
  auto within = [&](int t) {
    if (t >= len) return Within{0.0, false};
    const float gv = p.g[int64_t(b) * p.gb + int64_t(t) * p.gt + int64_t(h) * p.gh];
    return Within{sum_of(p.rows, p.T, t) + sum_of(p.sources, p.T, t), !(gv <= -kMostLog)};
  };
  // the first tokens' on their way before anything is waited for
  constexpr int A = 2;
  Within ahead[A];
#pragma unroll
  for (int i = 0; i < A; ++i) {
    const int t = t0 + i * kThreads + tid;
    ahead[i] = t < t1 ? within(t) : Within{0.0, false};
  }
  // cross: [blocks][B * H][spans + 1], at the start of each span but the first, and at the end
  double z = 0.0, end = 0.0;
  for (int k = 0; k < p.blocks; ++k) {
    const double* at = p.cross + (k * BH + bh) * (spans + 1);
    if (span > 0 && n > 0) z += at[span];
    if (n > 0) end += at[last == p.chunks ? spans : span + 1];
  }
  if (span == 0 && p.initial) {
    double s = 0.0;
    for (int64_t i = tid; i < state; i += kThreads)
      s += double(p.initial[bh * state + i]) * double(p.grad_initial[bh * state + i]);
    z = block_sum(s, la);
  }
  if (tid < n) {
    la[tid] = sum_of(p.sources_chunk, p.chunks, first + tid);
    ly[tid] = sum_of(p.rows_chunk, p.chunks, first + tid);
    cuts[tid] = p.chunk_decay[int64_t(bh) * p.chunks + first + tid] == 0.0f;
  }
  __syncthreads();
  if (tid == 0) {
    // `sum`: what was added up since the last cut, the scale of the rounding errors in z
    double sum = fabs(z);
    int from = 0;
    for (int i = 0; i < n; ++i) {
      if (cuts[i]) {
        from = i;
        sum = 0.0;
      } else {
        sum += fabs(ly[i]);
      }
      const double y = cuts[i] ? 0.0 : z - ly[i];
      lw[i] = sum;
      ly[i] = y;
      z = y + la[i];
      sum += fabs(la[i]);
    }
    // The carried sum at the span's end is known outright as well: what rounding has put between
    // the two is taken off again, in proportion to what had been added up.
    const double off = z - end;
    if (sum > 0.0 && fabs(off) <= 1e-4 * sum) {
      const double share = off / sum;
      for (int i = from; i < n; ++i) ly[i] -= cuts[i] ? 0.0 : share * lw[i];
    }
  }
  __syncthreads();
  double all = 0.0;
  auto put = [&](int t, Within in) {
    const double v = in.passes ? ly[t / p.chunk - first] + in.v : 0.0;
    if (p.per_head) all += v;
    else p.grad_g[(int64_t(b) * p.T + t) * p.H + h] = float(v);
  };
  int t = t0 + tid;
#pragma unroll
  for (int i = 0; i < A; ++i, t += kThreads)
    if (t < t1) put(t, ahead[i]);
  for (; t < t1; t += kThreads) put(t, within(t));
  if (p.per_head) {
    all = block_sum(all, la);
    if (tid == 0) p.partial[int64_t(span) * BH + bh] = all;
  }
}

// One wave a head.
__global__ __launch_bounds__(kWave) void decay_grad_heads(DaDecayGrad p) {
  const int h = blockIdx.x, lane = int(threadIdx.x);
  double s = 0.0;
  for (int64_t i = lane; i < int64_t(p.B) * p.segments * p.spans; i += kWave) s += p.partial[i * p.H + h];
  s = lane_of(prefix_sum(s, lane), 63);
  if (lane == 0) p.grad_g[h] = float(s);
}

// blockIdx.y: the tensor. A thread sums one element, or four side by side where d allows it.
__global__ __launch_bounds__(kThreads) void share_sum(DaShares all) {
  const DaShare p = all.s[blockIdx.y];
  const int e = p.d % 4 == 0 ? 4 : 1;
  const int64_t n = p.rows * p.d / e;
  for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < n; i += int64_t(gridDim.x) * kThreads) {
    const int64_t row = i * e / p.d, d = i * e % p.d;
    const float* from = p.src + row * p.rep * p.d + d;
    if (e == 4) {
      f32x4 s = zero4();
      for (int r = 0; r < p.rep; ++r) s += *reinterpret_cast<const f32x4*>(from + int64_t(r) * p.d);
      if (p.bf16) Op<true>::put4(static_cast<uint16_t*>(p.out) + i * 4, s);
      else *reinterpret_cast<f32x4*>(static_cast<float*>(p.out) + i * 4) = s;
    } else {
      float s = 0.0f;
      for (int r = 0; r < p.rep; ++r) s += from[int64_t(r) * p.d];
      if (p.bf16) static_cast<uint16_t*>(p.out)[i] = f32_to_bf16_rne(s);
      else static_cast<float*>(p.out)[i] = s;
    }
  }
}

// ---------------------------------------------------------------- one token

// Bound by memory: a state is read and written once. 64 requests of 16 heads of 128 x 128 from a pool of 80
// take 20.9 us, 6.0 TB/s (36 us by single elements, a row at a time).
// One workgroup a request, head and block of 4 CG columns: CG threads of four columns, kThreads / CG
// rows at a time, and of a thread's rows kStepRows on their way at once. VEC: the state by 16 bytes.
constexpr int kStepRows = 8;

template <bool BF, int CG, bool VEC>
__global__ __launch_bounds__(kThreads) void step_kernel(DaStep p) {
  using O = Op<BF>;
  using E = typename O::E;
  constexpr int RG = kThreads / CG;
  __shared__ float lq[256], lk[256];
  __shared__ alignas(16) float sum[RG][4 * CG];
  const int tid = int(threadIdx.x), blocks = (p.dv + 4 * CG - 1) / (4 * CG);
  const int cb = blockIdx.x % blocks, bh = blockIdx.x / blocks, b = bh / p.H, h = bh % p.H;
  const int64_t slot = p.slots ? int64_t(p.slots[b]) : int64_t(b);
  const bool used = slot >= 0 && slot < p.slots_in_pool;
  const int cg = tid % CG, r0 = tid / CG, col = 4 * (cb * CG + cg);
  f32x4 o = zero4();
  if (used) {
    float* s = p.state + slot * p.ss + int64_t(h) * p.sh + col;
    const E* v = head_base<E>(p.v, b, h);
    f32x4 old[kStepRows], vv = zero4();
    auto load = [&](int r1) {
#pragma unroll
      for (int i = 0; i < kStepRows; ++i) {
        // rows and columns that do not exist: an existing one, not written back
        const float* from = s + int64_t(min(r1 + i * RG, p.dk - 1)) * p.dv;
        if constexpr (VEC) {
          old[i] = *reinterpret_cast<const f32x4*>(col < p.dv ? from : from - col);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) old[i][e] = from[col + e < p.dv ? e : -col];
        }
      }
    };
    load(r0);
    if (tid < p.dk) {
      lq[tid] = O::one(head_base<E>(p.q, b, h)[int64_t(tid) * p.q.sd]);
      lk[tid] = O::one(head_base<E>(p.k, b, h)[int64_t(tid) * p.k.sd]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (col + e < p.dv) vv[e] = O::one(v[int64_t(col + e) * p.v.sd]);
    const float decay = expf(p.g[int64_t(b) * p.gb + int64_t(h) * p.gh]);
    const bool clears = decay == 0.0f;  // nothing of the state is left, whatever it holds
    __syncthreads();
    for (int r1 = r0; r1 < p.dk; r1 += kStepRows * RG) {
      if (r1 != r0) load(r1);
#pragma unroll
      for (int i = 0; i < kStepRows; ++i) {
        const int r = r1 + i * RG;
        if (r < p.dk) {
          const float kr = lk[r], qr = lq[r];
          f32x4 n;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            n[e] = fmaf(decay, clears ? 0.0f : old[i][e], kr * vv[e]);
            o[e] = fmaf(qr, n[e], o[e]);
          }
          float* to = s + int64_t(r) * p.dv;
          if constexpr (VEC) {
            if (col < p.dv) *reinterpret_cast<f32x4*>(to) = n;
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (col + e < p.dv) to[e] = n[e];
          }
        }
      }
    }
  }
  *reinterpret_cast<f32x4*>(&sum[r0][4 * cg]) = o;
  __syncthreads();
  const int at = 4 * CG * cb + tid;
  if (tid < 4 * CG && at < p.dv) {
    float t = 0.0f;
#pragma unroll
    for (int r = 0; r < RG; ++r) t += sum[r][tid];
    static_cast<E*>(p.out)[int64_t(bh) * p.dv + at] = O::round(t * p.scale);
  }
}

template <bool BF, int CG>
void launch_step(const DaStep& p, bool vec, hipStream_t stream) {
  const unsigned grid = unsigned(int64_t(p.B) * p.H * ((p.dv + 4 * CG - 1) / (4 * CG)));
  if (vec) step_kernel<BF, CG, true><<<grid, kThreads, 0, stream>>>(p);
  else step_kernel<BF, CG, false><<<grid, kThreads, 0, stream>>>(p);
}

}  // namespace

int decay_attention_chunk(bool bf16) { return bf16 ? Op<true>::C : Op<false>::C; }

int march_tiles(int dx) { return dx <= 32 ? 2 : dx <= 64 ? 4 : dx <= 128 ? 8 : 16; }
int march_waves(int dz) { return dz <= 64 ? 4 : 8; }

int decay_attention_column_blocks(int dz) {
  const int bv = 16 * march_waves(dz);
  return (dz + bv - 1) / bv;
}

void decay_attention_split(DaParams& p) {
  const int C = decay_attention_chunk(p.bf16 != 0);
  const int64_t chunks = (int64_t(p.T) + C - 1) / C;
  const int64_t groups = std::max<int64_t>(1, int64_t(p.B) * p.H * decay_attention_column_blocks(p.dv));
  // One workgroup a compute unit (two of four waves), rounded down so that all run at once, and segments
  // of two chunks at least: more segments cost more in starts and states than they spread (eight ragged
  // rows of 2048 tokens, 16 heads of 64 x 64: 60.7, 69.4, 68.4, 81.5 us at 2, 3, 4, 8 a compute unit).
  const int64_t resident = march_waves(p.dv) == 8 ? 1 : 2;
  const int64_t want = resident * device_cu_count() / groups;
  const int64_t segments = std::max<int64_t>(1, std::min(want, chunks / 2));
  const int64_t per = std::max<int64_t>(1, (chunks + segments - 1) / segments);
  p.seg_tokens = int(per * C);
  p.segments = int(std::max<int64_t>(1, (chunks + per - 1) / per));
  const int64_t spans = (per + kSpanChunks - 1) / kSpanChunks;
  p.span_chunks = int((per + spans - 1) / spans);
  p.spans = int((per + p.span_chunks - 1) / p.span_chunks);
}

hipError_t launch_decay_attention(const DaParams& p, hipStream_t stream) {
  // 16-byte pieces at 32-bit offsets within a chunk
  const int64_t e = p.bf16 ? 2 : 4, chunk = decay_attention_chunk(p.bf16 != 0), most = int64_t(1) << 31;
  bool vec = true, whole = true;  // whole: rows that are whole pieces cost the least
  for (int i = 0; i < p.marches; ++i) {
    for (const HeadView* v : {&p.m[i].x, &p.m[i].y, &p.m[i].z, &p.m[i].w})
      vec = vec && (!v->p || (v->unit && v->st >= 0 && v->st < most / (chunk * e)));
    whole = whole && p.m[i].dx * e % 16 == 0 && p.m[i].dz * e % 16 == 0;
    vec = vec && int64_t(p.H) * p.m[i].dz < most / (chunk * 4);
  }
  const auto launch = p.bf16 ? (!vec ? launch_marches_bf16_any : whole ? launch_marches_bf16 : launch_marches_bf16_cut)
                             : (!vec ? launch_marches_f32_any : whole ? launch_marches_f32 : launch_marches_f32_cut);
  hipError_t err = hipSuccess;
  if (p.segments > 1) {
    const int states = p.marches == 1 ? 1 : 2;
    err = launch(p, 0, states, true, stream);
    const int64_t n = int64_t(p.B) * p.H * p.dk * p.dv;
    if (err == hipSuccess) carry<<<dim3(unsigned((n + kThreads - 1) / kThreads), states), kThreads, 0, stream>>>(p);
  }
  if (err != hipSuccess) return err;
  if (p.marches == 1) return launch(p, 0, 1, false, stream);
  // grad_v's march holds the state the other way round: the same launch where keys and values are of one
  // class, or where the device has room for all three marches at once (the larger class then costs less
  // than a second launch: 333 tokens of 48 x 80 in f32, 28 us for the three when this was chosen, 44 in turn; 25 now)
  const bool alike = march_tiles(p.dk) == march_tiles(p.dv) && march_waves(p.dk) == march_waves(p.dv);
  if (alike || 3 * int64_t(p.B) * p.H * p.segments <= device_cu_count()) return launch(p, 0, 3, false, stream);
  err = launch(p, 0, 2, false, stream);
  return err == hipSuccess ? launch(p, 2, 1, false, stream) : err;
}

hipError_t launch_decay_grad(const DaDecayGrad& p, hipStream_t stream) {
  const int64_t BH = int64_t(p.B) * p.H;
  if (BH > 0) {
    if (p.spans > 1) span_cross<<<unsigned(BH * p.segments * (p.spans - 1)), kThreads, 0, stream>>>(p);
    decay_grad<<<unsigned(BH * p.segments * p.spans), kThreads, 0, stream>>>(p);
  }
  if (p.per_head) decay_grad_heads<<<p.H, kWave, 0, stream>>>(p);
  return hipGetLastError();
}

hipError_t launch_share_sums(const DaShares& p, hipStream_t stream) {
  int64_t n = 0;
  for (int i = 0; i < p.count; ++i) n = std::max(n, p.s[i].rows * p.s[i].d / (p.s[i].d % 4 == 0 ? 4 : 1));
  if (n == 0) return hipSuccess;
  const int64_t blocks = std::min<int64_t>((n + kThreads - 1) / kThreads, int64_t(device_cu_count()) * 16);
  share_sum<<<dim3(unsigned(blocks), unsigned(p.count)), kThreads, 0, stream>>>(p);
  return hipGetLastError();
}

hipError_t launch_decay_step(const DaStep& p, hipStream_t stream) {
  const bool vec = p.dv % 4 == 0 && p.ss % 4 == 0 && p.sh % 4 == 0 && (reinterpret_cast<uintptr_t>(p.state) & 15u) == 0;
  // 128 columns a workgroup where that fills the device, else 32
  const bool wide = p.dv > 32 && int64_t(p.B) * p.H * ((p.dv + 127) / 128) >= 2 * int64_t(device_cu_count());
  if (p.bf16) {
    if (wide) launch_step<true, 32>(p, vec, stream);
    else launch_step<true, 8>(p, vec, stream);
  } else {
    if (wide) launch_step<false, 32>(p, vec, stream);
    else launch_step<false, 8>(p, vec, stream);
  }
  return hipGetLastError();
}

}  // namespace sx
