// The forward's rows on their way over the keys: scores, running maximum, weights
// and weighted sums of 32 rows a wave (attn_fwd.hip, paged_attn.hip).
#pragma once
#include "attn_common.h"

namespace trsc {

constexpr float kLog2e = 1.4426950408889634f;

// The running maximum need not be the true one: the weights only have to stay
// representable. A tile is weighed with the maximum so far, and only where its
// sum leaves [0, kMostSum) is the maximum taken again, the sums rescaled and the
// tile weighed anew. (fp16 holds weights up to 65504.) With the maximum of every
// tile taken a causal prompt of 32,768 tokens (bf16, 16 heads of 128 over 4, 4096 keys back)
// took 1.24 ms for 0.99, 73,881 tokens (16 heads of 64, 512 keys either way) 622 us for 411.
constexpr float kMostSum = 16384.f;
// fp16 holds weights from 2^-14 (its smallest normal) to 65504, so the base moves down as well: where a lane's sum
// of up to 32 keys falls below kLeastSum16 (a leading key before them, a sink say), the tile's own largest weight
// becomes 2^kBase16 and the sums grow instead, which fp32 has room for. So the weights of every tile keep the type's
// precision among themselves, and a row gets a share of 2^-30 as exactly as a large one. (With the base fixed by
// the leading key, keys 16 nats below it had 2 to 4 bits left.) Right after, a tile's sum is 2^2 to 2^7: it may
// rise by 8 powers of two and more, or fall by 11, before the base moves again, so scores that spread by a few nats
// seldom move it (2^6 in place of 2^2: 33.8 us for 30.5, the forward of 4,616 tokens, 16 heads of 64 over 4; with a
// base that only rises 31.1). In a tile that itself spreads further the largest weight goes up to 2^kTop16: keys up
// to 20 nats under it stay normal. No growing past sums of kMostL: what could still come is below 2^-64 of what was.
constexpr float kMostSum16 = 49152.f, kLeastSum16 = 1.f / 512.f, kBase16 = 2.f, kTop16 = 15.f, kMostL = 1.8446744e19f;

// The scores of 32 keys j0 + 8 g + 4 (lane / 32) + i: hidden ones become -inf.
__device__ __forceinline__ void hide(f32x16& s, int j0, int lo, int hi, int sinks, int lane) {
  const int base = j0 + 4 * (lane >> 5);
  const int a0 = lo - base, a1 = hi - base, a2 = sinks - base;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int j = 8 * (e >> 2) + (e & 3);
    const bool sees = j <= a1 && (j >= a0 || j < a2);
    s[e] = sees ? s[e] : -INFINITY;
  }
}

// A wave's 32 rows on their way over the keys: lane l and l + 32 hold row l.
template <class E, int NB, int KB>
struct RowState {
  typedef Tile<E, NB> T;
  typedef AttnType<E> A;
  typedef typename A::frag frag;
  static constexpr int ST = NB * 2, kAhead = A::wide ? 1 : 4;
  static constexpr bool kNarrow = A::narrow;
  frag qf[ST];     // the queries
  f32x16 acc[NB];  // O^T
  float mc, l;     // scaled maximum (base 2) and sum of the weights
  f32x16 s[KB];    // scores of a tile of 32 KB keys
  frag pf[KB][2];  // its weights

  __device__ __forceinline__ void start(const E* qp, bool on, int dim, int lane) {
#pragma unroll
    for (int st = 0; st < ST; ++st) qf[st] = row_from<E>(qp, on, st, dim, lane);
#pragma unroll
    for (int d = 0; d < NB; ++d)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[d][e] = 0.f;
    mc = -INFINITY;
    l = 0.f;
  }
  __device__ __forceinline__ void scores(const unsigned char* ks, int steps, const typename T::Lane& at) {
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int e = 0; e < 16; ++e) s[kb][e] = 0.f;
    products<KB * ST, kAhead, frag>([&](int i, frag& f) { f = T::row(ks, 32 * (i / ST), i % ST, at); },
                                    [&](int i, const frag& f) {
                                      // fp32: a last step of zeros (heads of 16 past 32's multiples) costs a branch less
                                      if (!A::wide || i % ST < ST - 1 || steps == ST)
                                        s[i / ST] = A::mma(f, qf[i % ST], s[i / ST]);
                                    });
  }
  // weights 2^(s c - m), their sum, and the fragments that multiply V
  __device__ __forceinline__ float weigh_by(float c, float m) {
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int ss = 0; ss < 2; ++ss)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float w = __builtin_amdgcn_exp2f(fmaf(s[kb][8 * ss + e], c, -m));
          sum[e & 1] += w;
          pf[kb][ss][e] = static_cast<E>(w);
        }
    return sum[0] + sum[1];
  }
  // whether the tile's weights are in range
  static __device__ __forceinline__ bool in_range(float sum) {
    if constexpr (kNarrow) return __builtin_amdgcn_fmed3f(sum, kLeastSum16, kMostSum16) == sum;
    return sum < kMostSum;
  }
  __device__ __forceinline__ void weigh(float c) {
    float sum = weigh_by(c, mc);
    const bool out = !in_range(sum);  // also where the row has seen nothing before (mc = -inf: the sum is NaN)
    if (__any(out) && (!kNarrow || __any(out && sum != 0.f))) {  // a row that sees none of the tile has the sum 0
      float mx = -INFINITY;
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int e = 0; e < 16; ++e) mx = fmaxf(mx, s[kb][e]);
      const float2 mh = both_halves(mx);
      mx = fmaxf(mh.x, mh.y) * c;
      if constexpr (kNarrow) {
        float mn = INFINITY;  // of the scores that the row sees
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
          for (int e = 0; e < 16; ++e) mn = fminf(mn, s[kb][e] == -INFINITY ? INFINITY : s[kb][e]);
        const float2 nh = both_halves(mn), lh = both_halves(l);
        const float to = mx - fminf(fmaxf(mx - fminf(nh.x, nh.y) * c - 14.f, kBase16), kTop16);
        if (mx == -INFINITY)
          mx = mc;
        else if (to < mc)  // down, at most 30 a tile: l stays under 2^95
          mx = lh.x + lh.y < kMostL ? fmaxf(to, mc - 30.f) : mc;
        else
          mx = to;
      } else {
        mx = fmaxf(mx, mc);
      }
      const float f = mx == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(mc - mx);
      l *= f;
#pragma unroll
      for (int d = 0; d < NB; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[d][e] *= f;
      mc = mx;
      sum = weigh_by(c, mx == -INFINITY ? 0.f : mx);
    }
    l += sum;
  }
  __device__ __forceinline__ void multiply(const unsigned char* vs, const typename T::Lane& at) {
    products<KB * 2 * NB, kAhead, frag>(
        [&](int i, frag& f) { f = T::col(vs, 32 * (i / (2 * NB)), i / NB % 2, i % NB, at); },
        [&](int i, const frag& f) { acc[i % NB] = A::mma(f, pf[i / (2 * NB)][i / NB % 2], acc[i % NB]); });
  }
  __device__ __forceinline__ void join_halves() {
    const float2 lh = both_halves(l);
    l = lh.x + lh.y;
  }
};

}  // namespace trsc
