// Norm and rotation of new tokens' queries and keys, the keys and values
// straight to their places in a paged cache.
//
// Mathematics. As in norm_rope.hip: y = x / sqrt(mean(x^2) + eps) * gain (or
// x itself), its pairs turned by position times frequency. Token t, the i-th of
// the Lq tokens of sequence b, is the sequence's key j = len[b] - Lq + i; its
// place is slot j % page of page table[b][j / page].
//
// Layout. Rows in lanes as in norm_rope.hip, the heads of q, k and v side by
// side, so that the values' copy is the same loads and stores without the
// arithmetic. The places of a wave's next 64 tokens are looked up at once, one a
// lane (search in the offsets, length, table: three dependent reads), and read
// back lane by lane.
//
// What bounds it: memory. bf16, 73,881 tokens x 48 heads of 64 to empty caches:
// 909 MB in 191 us, 4.76 TB/s (a large copy: 5.03). fp32, 2,877 tokens x 20 heads of
// 72: 33 MB in 9.6 us, 3.5 TB/s, the look-up of places before the first store. 32
// tokens: 4.6 to 5.4 us, one launch.
#include "common.h"
#include "paged.h"
#include "rotate.h"
#include "token_types.h"

namespace trsc {
namespace {

constexpr int kWaves = 4;
constexpr int E = kRowElts;
constexpr int kThreads = kWaves * 64;

struct Place {
  int page, slot;  // page: kNoPage where the token's key has none, kNoSequence where the token is in no sequence
};
constexpr int kNoPage = -1, kNoSequence = -2;

__device__ __forceinline__ Place place_of(const AppendArgs& a, int64_t t) {
  Place p{kNoSequence, 0};
  if (t >= a.tokens) return p;
  int b;
  int64_t end;  // of the sequence's tokens
  if (a.seqs.cu == nullptr) {
    b = int(t) / a.seqs.each;
    end = int64_t(b + 1) * a.seqs.each;
  } else {
    if (t < a.seqs.cu[0]) return p;
    int lo = 0, n = a.seqs.batch;  // the last sequence that starts at t or before
    while (n > 1) {
      const int h = n >> 1;
      if (a.seqs.cu[lo + h] <= t) {
        lo += h;
        n -= h;
      } else {
        n = h;
      }
    }
    b = lo;
    end = a.seqs.cu[b + 1];
    if (t >= end) return p;
  }
  const int64_t j = int64_t(a.pool.len[b]) - (end - t);
  p.page = kNoPage;
  if (j < 0 || j >= int64_t(a.pool.table_pages) << a.pool.log2) return p;
  const int page = a.pool.table[b * a.pool.table_ts + (j >> a.pool.log2)];
  if (page >= 0 && page < a.pool.pages) p.page = page;
  p.slot = int(j) & ((1 << a.pool.log2) - 1);
  return p;
}

template <class T, bool IL>
__global__ __launch_bounds__(kThreads) void append_kernel(AppendArgs a, int group) {
  typedef typename T::elt elt;
  __shared__ float2 s_turn[kWaves][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int per = 64 / group;         // heads of a wave
  const int c = lane & (group - 1);   // chunk of the row
  const int hq = a.q.heads, hk = a.k.heads;
  const int head = blockIdx.y * per + lane / group;  // q's, then k's, then v's
  const bool on = c < a.dim / (2 * E) && head < hq + 2 * hk;
  const bool isq = head < hq, isv = head >= hq + hk;
  const int off = on ? c * E : 0, half = a.dim / 2;
  const int h = !on || isq ? (on ? head : 0) : isv ? head - hq - hk : head - hq;
  const NormSide& side = isq ? a.q : a.k;
  const elt* const x = static_cast<const elt*>(isv ? a.v.p : side.x) + h * (isv ? a.v.hs : side.xhs) + off;
  const int64_t xts = isv ? a.v.ts : side.xts;
  elt* const y = static_cast<elt*>(isq ? a.q.y : isv ? a.pool.v : a.pool.k) +
                 h * (isq ? a.q.yhs : isv ? a.pool.vhs : a.pool.khs) + off;
  const int64_t ps = isv ? a.pool.vps : a.pool.kps, ss = isv ? a.pool.vss : a.pool.kss;
  const float* const gain = isv || side.gain == nullptr ? nullptr : side.gain + (side.gain_rows > 1 ? h * a.dim : 0) + off;
  float g0[E], g1[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    g0[e] = on && gain ? gain[e] : 1.f;
    g1[e] = on && gain ? gain[half + e] : 1.f;
  }
  const int axis = lane < a.c1 ? 0 : lane < a.c2 ? 1 : 2;  // of the pair whose angle this lane computes
  const bool turns = lane < a.c3 && lane < half;
  const double freq = turns ? double(a.freqs[lane]) * 0.15915494309189533577 : 0.0;
  const float inv_dim = 1.f / float(a.dim);

  const int64_t step = int64_t(gridDim.x) * kWaves;
  int64_t t = int64_t(blockIdx.x) * kWaves + wave;
  Chunk<T, E> x0{}, x1{};
  int32_t pos = 0;
  auto fetch = [&](int64_t tt) {
    if (on) {
      x0.load(x + tt * xts);
      x1.load(x + tt * xts + half);
    }
    if (turns) pos = a.pos[tt * a.pos_ts + axis];
  };
  if (t < a.tokens) fetch(t);
  Place mine{};
  for (int n = 0; t < a.tokens; t += step, ++n) {
    if (n % 64 == 0) mine = place_of(a, t + lane * step);
    const int page = __builtin_amdgcn_readlane(mine.page, n % 64), slot = __builtin_amdgcn_readlane(mine.slot, n % 64);
    Chunk<T, E> w0 = x0, w1 = x1;
    turn_table(pos, freq, turns, lane, s_turn[wave]);
    if (t + step < a.tokens) fetch(t + step);
    float v[2][E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      v[0][e] = w0.get(e);
      v[1][e] = w1.get(e);
    }
    if (a.norm) {
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) sum += v[0][e] * v[0][e] + v[1][e] * v[1][e];
      if (!on) sum = 0.f;
      const float r = rsqrtf(group_sum(sum, group) * inv_dim + a.eps);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        v[0][e] *= r * g0[e];
        v[1][e] *= r * g1[e];
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the table is the wave's own
    float2 cs[E];  // IL: E / 2 pairs of the first chunk, then E / 2 of the second; else pair e
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int pair = IL ? (e < E / 2 ? off / 2 + e : half / 2 + off / 2 + e - E / 2) : off + e;
      cs[e] = s_turn[wave][pair];
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (!isv) {
      auto turn = [&](float p, float q, float2 w, float& rp, float& rq) {
        rp = p * w.x - q * w.y;
        rq = p * w.y + q * w.x;
      };
      float o[2][E];
      if constexpr (IL) {
#pragma unroll
        for (int hh = 0; hh < 2; ++hh)
#pragma unroll
          for (int e = 0; e < E; e += 2)
            turn(v[hh][e], v[hh][e + 1], cs[hh * (E / 2) + e / 2], o[hh][e], o[hh][e + 1]);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) turn(v[0][e], v[1][e], cs[e], o[0][e], o[1][e]);
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        w0.set(e, o[0][e]);
        w1.set(e, o[1][e]);
      }
    }
    if (on && (isq ? page != kNoSequence : page >= 0)) {
      elt* const to = y + (isq ? t * a.q.yts : page * ps + slot * ss);
      w0.store(to);
      w1.store(to + half);
    }
  }
}

template <class T>
void launch_pairs(const AppendArgs& a, dim3 grid, hipStream_t st) {
  const int group = group_lanes(a.dim);
  if (a.interleaved)
    append_kernel<T, true><<<grid, kThreads, 0, st>>>(a, group);
  else
    append_kernel<T, false><<<grid, kThreads, 0, st>>>(a, group);
}

}  // namespace

hipError_t launch_norm_rope_append(const AppendArgs& a, hipStream_t st) {
  if (a.tokens == 0) return hipSuccess;
  const int per = 64 / group_lanes(a.dim);
  const int head_blocks = (a.q.heads + 2 * a.k.heads + per - 1) / per;
  // seven workgroups a CU (eight fit), evened out so that every wave walks as many tokens: 73,881 tokens x 48 heads of 64
  // take 192 us, with eight or six 194, with four 228
  const int64_t n = 1792 / head_blocks > 1 ? 1792 / head_blocks : 1;
  const int64_t walk = (a.tokens + n * kWaves - 1) / (n * kWaves);
  const dim3 grid(unsigned((a.tokens + walk * kWaves - 1) / (walk * kWaves)), head_blocks);
  if (a.dtype == TR_SC_BF16)
    launch_pairs<TBF16>(a, grid, st);
  else if (a.dtype == TR_SC_F16)
    launch_pairs<TF16>(a, grid, st);
  else
    launch_pairs<TF32>(a, grid, st);
  return hipGetLastError();
}

}  // namespace trsc
