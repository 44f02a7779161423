// Per-head RMS norm of queries and keys with the position rotation in the same
// pass, and its gradient.
//
// Mathematics. For a token t and a head h with gain g (none: 1),
//     r = 1 / sqrt(mean_d x_d^2 + eps),  y_d = x_d r g_d,
// then every pair (a, b) of y -- elements (2 i, 2 i + 1) or (i, i + dim / 2) --
// turns by the angle pos[t, axis_i] * freq_i: (a cos - b sin, a sin + b cos).
// Backward of L = sum <out, d>: z = d turned back by the same angle, w = z g,
// xn = x r, dx = r (w - xn mean(w xn)), dg = sum over tokens (and, for a shared
// gain, heads) of z xn.
//
// The angle is taken in turns in 64 bits, position times frequency / 2 pi, and
// reduced to [-1/2, 1/2] there before it is rounded to 32 bits. Two roundings of
// 2^-53 are on the way: while position times frequency is below 2^28 their error
// (9e-9 turns at most) is less than the 32-bit rounding's (1.5e-8); near 2^31 it
// is 7e-8 turns.
//
// Layout. A row (token, head) of dim elements is held by dim / (2 E) lanes (the
// group; E = 4 elements): lane c holds elements [c E, c E + E) of either half of
// the row, so both pairings have their pairs inside one lane. (E = 8 halves the
// lanes' instructions but holds five waves a SIMD, backward three, instead of
// eight and five: forward 128 us for 122 at the first size below, backward the
// same.) A wave holds 64 / group rows: the same token's
// consecutive heads. Its heads stay the same over the tokens that it walks, so
// a lane's gains (and the backward's sums of their gradients) live in
// registers. The sines and cosines of a token are computed once a wave, one
// pair a lane, and handed out through LDS that only this wave uses.
//
// What bounds it: memory, each element read and written once (backward: two
// read). bf16, 73,881 tokens x 32 heads of 64: 605 MB in 122 us, 4.96 TB/s, the
// rate of a large copy (5.03 TB/s). fp32, 16,219 x 16 heads of 72: 150 MB in
// 29.9 us, 5.0 TB/s. Backward, bf16, 15,800 x 24 heads of 128: 291 MB in 61 to 66
// us with the gains' sums, 4.4 to 4.8 TB/s; vector instructions are busy for most
// of it. The same in fp16: 61 us, in fp32: 122.
// 32 tokens: 4.3 us, one launch.
#include "common.h"
#include "token_types.h"
#include "tokens.h"

namespace trsc {
namespace {

constexpr int kWaves = 4;
constexpr int E = 4;  // elements of either half of a row in a lane
constexpr int kNormThreads = kWaves * 64;

template <class T>
struct SidePtrs {  // this lane's head
  const typename T::elt* x;
  const typename T::elt* dy;
  typename T::elt* y;
  int64_t xts, dts, yts;
  const float* gain;
};

template <class T>
__device__ __forceinline__ SidePtrs<T> side_ptrs(const NormArgs& a, int head, int off) {
  typedef typename T::elt elt;
  const bool isq = head < a.q.heads;
  const NormSide& s = isq ? a.q : a.k;
  const int h = isq ? head : head - a.q.heads;
  SidePtrs<T> p;
  p.x = static_cast<const elt*>(s.x) + h * s.xhs + off;
  p.dy = s.dy ? static_cast<const elt*>(s.dy) + h * s.dhs + off : nullptr;
  p.y = static_cast<elt*>(s.y) + h * s.yhs + off;
  p.xts = s.xts;
  p.dts = s.dts;
  p.yts = s.yts;
  p.gain = s.gain ? s.gain + (s.gain_rows > 1 ? h * a.dim : 0) + off : nullptr;
  return p;
}

// (cos, sin) of this lane's pair at token t into the wave's table.
__device__ __forceinline__ void turn_table(const NormArgs& a, int32_t p, double freq_turns, bool turns, int lane,
                                           float2* table) {
  float2 cs = make_float2(1.f, 0.f);
  if (turns) {
    const double t = double(p) * freq_turns;
    const float f = float(t - rint(t));
    sincospif(2.f * f, &cs.y, &cs.x);
  }
  table[lane] = cs;
}

__device__ __forceinline__ float group_sum(float v, int group) {
  for (int o = group >> 1; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

template <class T, bool IL, bool BWD>
__global__ __launch_bounds__(kNormThreads) void norm_rope_kernel(NormArgs a, int group) {
  typedef typename T::elt elt;
  __shared__ float2 s_turn[kWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int per = 64 / group;               // heads of a wave
  const int c = lane & (group - 1);         // chunk of the row
  const int lanes = a.dim / (2 * E);        // lanes of a row that hold elements
  const int heads = a.q.heads + a.k.heads;
  const int head = blockIdx.y * per + lane / group;
  const bool on = c < lanes && head < heads;
  const int off = on ? c * E : 0, half = a.dim / 2;
  const SidePtrs<T> p = side_ptrs<T>(a, head < heads ? head : 0, off);
  float g0[E], g1[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    g0[e] = on && p.gain ? p.gain[e] : 1.f;
    g1[e] = on && p.gain ? p.gain[half + e] : 1.f;
  }
  // the pair whose angle this lane computes
  const int axis = lane < a.c1 ? 0 : lane < a.c2 ? 1 : 2;
  const bool turns = lane < a.c3 && lane < half;
  const double freq = turns ? double(a.freqs[lane]) * 0.15915494309189533577 : 0.0;
  const float inv_dim = 1.f / float(a.dim);
  float d0[E], d1[E];  // sums of the gain's gradient
#pragma unroll
  for (int e = 0; e < E; ++e) d0[e] = d1[e] = 0.f;

  const int64_t step = int64_t(gridDim.x) * kWaves;
  int64_t t = int64_t(blockIdx.x) * kWaves + wave;
  Chunk<T, E> x0{}, x1{}, u0{}, u1{};
  int32_t pos = 0;
  auto fetch = [&](int64_t tt) {
    if (on) {
      x0.load(p.x + tt * p.xts);
      x1.load(p.x + tt * p.xts + half);
      if constexpr (BWD) {
        u0.load(p.dy + tt * p.dts);
        u1.load(p.dy + tt * p.dts + half);
      }
    }
    if (turns) pos = a.pos[tt * a.pos_ts + axis];
  };
  if (t < a.tokens) fetch(t);
  for (; t < a.tokens; t += step) {
    float x[2][E], u[2][E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      x[0][e] = x0.get(e);
      x[1][e] = x1.get(e);
      if constexpr (BWD) {
        u[0][e] = u0.get(e);
        u[1][e] = u1.get(e);
      }
    }
    turn_table(a, pos, freq, turns, lane, s_turn[wave]);
    if (t + step < a.tokens) fetch(t + step);
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) ss += x[0][e] * x[0][e] + x[1][e] * x[1][e];
    if (!on) ss = 0.f;
    ss = group_sum(ss, group);
    const float r = rsqrtf(ss * inv_dim + a.eps);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the table is the wave's own
    float2 cs[E];  // IL: E / 2 pairs of the first chunk, then E / 2 of the second; else pair e
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int pair = IL ? (e < E / 2 ? off / 2 + e : half / 2 + off / 2 + e - E / 2) : off + e;
      cs[e] = s_turn[wave][pair];
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    float o[2][E];
    auto turn = [&](float a0, float b0, float2 w, float& ra, float& rb) {
      const float sn = BWD ? -w.y : w.y;
      ra = a0 * w.x - b0 * sn;
      rb = a0 * sn + b0 * w.x;
    };
    if constexpr (!BWD) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        x[0][e] *= r * g0[e];
        x[1][e] *= r * g1[e];
      }
    }
    float(&in)[2][E] = BWD ? u : x;
    if constexpr (IL) {
#pragma unroll
      for (int hh = 0; hh < 2; ++hh)
#pragma unroll
        for (int e = 0; e < E; e += 2)
          turn(in[hh][e], in[hh][e + 1], cs[hh * (E / 2) + e / 2], o[hh][e], o[hh][e + 1]);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) turn(in[0][e], in[1][e], cs[e], o[0][e], o[1][e]);
    }
    if constexpr (BWD) {
      float dot = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        x[0][e] *= r;
        x[1][e] *= r;
        d0[e] += o[0][e] * x[0][e];
        d1[e] += o[1][e] * x[1][e];
        o[0][e] *= g0[e];
        o[1][e] *= g1[e];
        dot += o[0][e] * x[0][e] + o[1][e] * x[1][e];
      }
      if (!on) dot = 0.f;
      dot = group_sum(dot, group) * inv_dim;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        o[0][e] = r * (o[0][e] - x[0][e] * dot);
        o[1][e] = r * (o[1][e] - x[1][e] * dot);
      }
    }
    if (on) {
      Chunk<T, E> w0, w1;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        w0.set(e, o[0][e]);
        w1.set(e, o[1][e]);
      }
      w0.store(p.y + t * p.yts);
      w1.store(p.y + t * p.yts + half);
    }
  }
  if constexpr (BWD) {
    // the four waves' sums, joined in wave order, are this workgroup's partial
    __shared__ float s_sum[kWaves - 1][64][2 * E + 1];
    if (wave > 0) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        s_sum[wave - 1][lane][e] = d0[e];
        s_sum[wave - 1][lane][E + e] = d1[e];
      }
    }
    __syncthreads();
    if (wave == 0 && on) {
      float* dst = a.partials + (int64_t(blockIdx.x) * heads + head) * a.dim + off;
#pragma unroll
      for (int e = 0; e < E; ++e) {
#pragma unroll
        for (int w = 0; w < kWaves - 1; ++w) {
          d0[e] += s_sum[w][lane][e];
          d1[e] += s_sum[w][lane][E + e];
        }
        dst[e] = d0[e];
        dst[half + e] = d1[e];
      }
    }
  }
}

// dgain[row, d] = the sum, in a fixed order, of the workgroups' partials
// [splits][heads][dim] over the splits and, for a shared gain, the heads of
// that side. blockIdx.y: side. Two lanes of four columns each by 128 slices of
// the splits, joined in a tree (15,800 tokens x 24 heads of 128, 208 splits: 5 us;
// one thread a column walked all of them in 19).
__global__ __launch_bounds__(256) void gain_sum(NormArgs a, int splits) {
  constexpr int L = 2, kSlices = 256 / L;
  const NormSide& s = blockIdx.y == 0 ? a.q : a.k;
  if (s.dgain == nullptr) return;
  const int h0 = blockIdx.y == 0 ? 0 : a.q.heads, heads = a.q.heads + a.k.heads;
  const int cols = s.gain_rows * a.dim, inner = s.gain_rows == 1 ? s.heads : 1;
  const int lane = threadIdx.x % L, slice = threadIdx.x / L;
  const int col = (blockIdx.x * L + lane) * 4;
  __shared__ float4 s_part[256];
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](const float4& x) {
    v.x += x.x;
    v.y += x.y;
    v.z += x.z;
    v.w += x.w;
  };
  if (col < cols) {
    const float* src = a.partials + int64_t(h0) * a.dim + col;
    for (int i = slice; i < splits; i += kSlices) {
      const float* p = src + int64_t(i) * heads * a.dim;
#pragma unroll 4
      for (int h = 0; h < inner; ++h) add(*reinterpret_cast<const float4*>(p + h * a.dim));
    }
  }
  s_part[threadIdx.x] = v;
  __syncthreads();
#pragma unroll
  for (int n = kSlices / 2; n > 0; n >>= 1) {
    if (slice < n) {
      add(s_part[(slice + n) * L + lane]);
      s_part[threadIdx.x] = v;
    }
    __syncthreads();
  }
  if (slice == 0 && col < cols) *reinterpret_cast<float4*>(s.dgain + col) = v;
}

int group_lanes(int dim) {
  const int lanes = dim / (2 * E);
  int g = 1;
  while (g < lanes) g <<= 1;
  return g;
}

// Workgroups over the tokens: `fill` in all, fewer where a wave would have no
// token, and evened out so that every wave walks as many. Forward: four a CU
// (eight fit; 132 us for 122 with them at the first size above). Backward: the
// five a CU that fit (three: 59 us for 52 at 15,800 x 24 heads of 72).
constexpr int kForwardFill = 1024, kBackwardFill = 1280;
int token_blocks(int64_t tokens, int head_blocks, int fill) {
  const int64_t n = fill / head_blocks > 1 ? fill / head_blocks : 1;
  const int64_t walk = (tokens + n * kWaves - 1) / (n * kWaves);
  return walk == 0 ? 0 : int((tokens + walk * kWaves - 1) / (walk * kWaves));
}

template <class T, bool BWD>
void launch_pairs(const NormArgs& a, dim3 grid, hipStream_t st) {
  const int group = group_lanes(a.dim);
  if (a.interleaved)
    norm_rope_kernel<T, true, BWD><<<grid, kNormThreads, 0, st>>>(a, group);
  else
    norm_rope_kernel<T, false, BWD><<<grid, kNormThreads, 0, st>>>(a, group);
}

template <bool BWD>
void launch_typed(const NormArgs& a, dim3 grid, hipStream_t st) {
  if (a.dtype == TR_SC_BF16)
    launch_pairs<TBF16, BWD>(a, grid, st);
  else if (a.dtype == TR_SC_F16)
    launch_pairs<TF16, BWD>(a, grid, st);
  else
    launch_pairs<TF32, BWD>(a, grid, st);
}

int head_blocks(int heads, int dim) {
  const int per = 64 / group_lanes(dim);
  return (heads + per - 1) / per;
}

}  // namespace

hipError_t launch_norm_rope(const NormArgs& a, hipStream_t st) {
  if (a.tokens == 0) return hipSuccess;
  const int hb = head_blocks(a.q.heads + a.k.heads, a.dim);
  launch_typed<false>(a, dim3(token_blocks(a.tokens, hb, kForwardFill), hb), st);
  return hipGetLastError();
}

static int backward_blocks(int64_t tokens, int heads, int dim) {
  return token_blocks(tokens, head_blocks(heads, dim), kBackwardFill);
}

int64_t norm_rope_partials(int64_t tokens, int heads, int dim) {
  return int64_t(backward_blocks(tokens, heads, dim)) * heads * dim;
}

hipError_t launch_norm_rope_backward(const NormArgs& a, hipStream_t st) {
  const int heads = a.q.heads + a.k.heads;
  const int splits = backward_blocks(a.tokens, heads, a.dim);
  if (splits > 0) {
    launch_typed<true>(a, dim3(splits, head_blocks(heads, a.dim)), st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.q.dgain || a.k.dgain) {
    const int cols = (a.q.gain_rows > a.k.gain_rows ? a.q.gain_rows : a.k.gain_rows) * a.dim;
    gain_sum<<<dim3((cols + 7) / 8, 2), 256, 0, st>>>(a, splits);
  }
  return hipGetLastError();
}

}  // namespace trsc
