// Gradients of the windowed attention with sinks.
//
// Mathematics. With P_ij = e^{scale q_i.k_j - lse_i} over the keys that row i
// sees and delta_i = o_i . do_i,
//     dV_j = sum_i P_ij do_i,   dP_ij = do_i . v_j,   dS_ij = P_ij (dP_ij - delta_i),
//     dq_i = scale sum_j dS_ij k_j,   dk_j = scale sum_i dS_ij q_i.
// Two kernels recompute P from q, k and lse: one walks the keys for 128 rows
// (dq, and delta on the way), one walks the rows for 128 keys (dk, dv). Seven
// products of the tile sizes instead of the five that one kernel with atomic
// sums would need, but every sum has one owner and a fixed order: the same bits
// on every call, and the gradients of a key-value head that several query heads
// share are summed in the registers.
//
// Rows, tiles and products are the forward's (attn_fwd.hip): S^T = K Q^T and
// dP^T = V dO^T give dS^T in the layout that dQ^T += K^T dS^T takes; in the
// other kernel S = Q K^T and dP = dO V^T (rows down, keys across) give P and dS
// as dV^T += dO^T P and dK^T += Q^T dS take them.
//
// Precision. The weights and dS are rounded to the tensors' type for the
// products (fp16: raised into its range first, whatever the size of dout and of
// the weights); either costs a sum about as much as its own last rounding does. The
// given o is rounded too, which would shift all dS of a row by the same share
// of P: sum_j P_ij dP_ij, exact where o is not, comes with the walk over the
// keys, so the dk, dv kernel takes that for delta, and dq is mended by a
// second product (see attn_dq). Without either, dq and dk of windows of 32
// keys were 1.8 times as far from the exact gradient as rounding once (now 1.5
// at most); the second product is 4 % of the gradient's time. fp16's ranges take
// 8 us of the 150 below.
//
// What bounds it. bf16, 15,800 tokens, 12 heads of 128, 512 keys either way: 495
// to 510 us for 0.25 TFLOP (10 flops a pair and element; 16 with what is computed
// twice and the second product, 780 TFLOP/s): matrix units and the LDS reads that
// feed them, one fragment a product, at two workgroups a CU (registers). fp16,
// 4,616 tokens in two sequences, 16 heads of 64 over 4, 1023 back: 150 us,
// latencies: each SIMD has two waves, and a wave's products, exponentials and
// packings follow one another.
//
// Sinks. All later rows see the sinks, so the tile that holds them would walk
// all rows. Its rows past the band go to workgroups of their own, in chunks;
// their partial sums and the tile's own are joined in a fixed order.
#include "attn_common.h"

namespace trsc {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kRowsWg = 128, kKeysWg = 128;
constexpr int kKeyTile = 64;      // keys of a tile of the dq kernel
constexpr int kRowTile = 32;      // rows of a tile of the dk, dv kernel
constexpr int kSinkChunk = 512;   // rows of a sink workgroup (256, 1024: 2 % either way, the sizes differing)
constexpr int kWantWgs = 512;     // workgroups that fill the chip: two on each of 256 CUs

// Powers of two that a weight of the dk, dv kernel is raised by before it is rounded: weights reach 1, so fp16 would
// have 14 powers of two for them and holds 29 this way (without, dv of keys 15 nats and more below a row's leading
// one were off by their own size). Taken off with the sums' last factor; the rows' stored lse has it.
template <class A>
constexpr float kWeightShift = A::narrow ? 15.f : 0.f;
template <class A>
constexpr float kWeightBack = A::narrow ? 1.f / 32768.f : 1.f;

// The score gradients dS = P (dP - delta) are as large as dout is and as small as P: fp16 would hold them for a dout
// of about one and windows of about a thousand keys (with dout of 1e-4, or a leading key, dq and dk were 3 to 6 times
// as far off as one rounding). So they are raised by a power of two before they are rounded. In dq it is each row's
// own: one that makes |dout|, as a vector, about 2^kScoreShift. That is a guess of dS from half of its factors, so
// the largest |dS| of a row is kept, and where it left [kLeastScore, kMostScore) the workgroup walks again with what
// it is now known to be. So it does for rows whose outputs are near or below the type's smallest normal, which give no
// usable delta, where dS is small enough for that to show (dq of heads past 64 was up to 280 roundings off). In dk it
// is one for the rows that a workgroup walks, from their largest |dS|, which the dq kernel leaves for it: a row far
// below the others adds little to the same sums. No |dS| counts as less than kScoreNoise (|lse| + 16) |o| |dout|, the
// error of P delta: where one key has all the weight dS is that noise, another in either kernel, and raised to the
// range's top in one it would overflow in the other (scores that spread by 60 nats: 660 us for 110, in a gradient of
// 8192 tokens, 8 heads of 64).
constexpr int kScoreShift = 9, kNoScore = -1000;
constexpr float kLeastScore = 1.f / 512.f, kMostScore = 32768.f, kDeltaScore = 2.f, kLeastOut = 1.f / 2048.f;
constexpr float kScoreNoise = 1.f / (1 << 20);
__device__ __forceinline__ int exponent_of(float v) { return __builtin_amdgcn_frexp_expf(v); }  // 0 if not finite
__device__ __forceinline__ float power_of_two(int n) { return __builtin_ldexpf(1.f, n); }

template <class E, int NB>
__device__ __forceinline__ void store_rows(E* p, const f32x16 (&acc)[NB], float f, int dim, int h) {
  typedef E out4 __attribute__((ext_vector_type(4)));
#pragma unroll
  for (int d = 0; d < NB; ++d)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int at = 32 * d + 8 * g + 4 * h;
      if (at < dim) {
        out4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = static_cast<E>(acc[d][4 * g + i] * f);
        *reinterpret_cast<out4*>(p + at) = v;
      }
    }
}

// Where a key tile stands to the rows at positions p0 .. p1 (of a wave): seen by any, or by all.
__device__ __forceinline__ bool any_sees(const AttnArgs& a, int p0, int p1, int j0, int j1, int lk) {
  return j0 < lk && j0 <= p1 + a.right && (j1 >= p0 - a.left || j0 < a.sinks);
}
__device__ __forceinline__ bool all_see(const AttnArgs& a, int p0, int p1, int j0, int j1, int lk) {
  return j1 <= p0 + a.right && j1 < lk && (j0 >= p1 - a.left || j1 < a.sinks);
}

// dq (not scaled) of a wave's rows at positions p0 .. p1 again, adding only what each sees (attn_common.h); p: this
// lane's position; qp, gp: its query and dout. lds: 4 KB of the wave's own.
template <class E, int NB>
__device__ void safe_dq(const AttnArgs& a, const Seq& q, const KeyTiles& kt, int p0, int p1, int p, bool on,
                        const E* qp, const E* gp, int kvh, float lse2, float delta, float* lds, int lane,
                        f32x16 (&acc)[NB]) {
  constexpr int ST = NB * 2;
  const float c = a.scale * kLog2e;
  const int lo = p - a.left, hi = min(p + a.right, q.lk - 1);
  const E* kbase = static_cast<const E*>(a.k.p) + int64_t(q.k0) * a.k.ts + kvh * a.k.hs;
  const E* vbase = static_cast<const E*>(a.v.p) + int64_t(q.k0) * a.v.ts + kvh * a.v.hs;
  typename AttnType<E>::frag qf[ST], gf[ST];
#pragma unroll
  for (int s = 0; s < ST; ++s) {
    qf[s] = row_from<E>(qp, on, s, a.dim, lane);
    gf[s] = row_from<E>(gp, on, s, a.dim, lane);
  }
#pragma unroll
  for (int d = 0; d < NB; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[d][e] = 0.f;
  for (int it = 0; it < kt.n * (kKeyTile / 32); ++it) {
    const int j0 = kt.at(it / (kKeyTile / 32)) * kKeyTile + it % (kKeyTile / 32) * 32;
    if (!any_sees(a, p0, p1, j0, j0 + 31, q.lk)) continue;
    const int mine = j0 + (lane & 31);
    f32x16 s = scores_from<E, ST>(kbase + mine * a.k.ts, mine < q.lk, qf, a.dim, lane);
    const f32x16 dp = scores_from<E, ST>(vbase + mine * a.v.ts, mine < q.lk, gf, a.dim, lane);
#pragma unroll
    for (int e = 0; e < 16; ++e) s[e] = __builtin_amdgcn_exp2f(fmaf(s[e], c, -lse2)) * (dp[e] - delta);
    put_factors(lds, s, lane);
    wave_fence();
    add_rows<E, NB>(
        acc, lds, [&](int i) { return kbase + min(j0 + i, q.lk - 1) * a.k.ts; },
        [&](int i) { return j0 + i <= hi && (j0 + i >= lo || j0 + i < a.sinks); }, 0, a.dim, lane);
    wave_fence();
  }
}

// dk (not scaled) and dv of a wave's 32 keys from jw over the rows [r0, r1) again, adding only rows that see them.
// key_on: this lane's key is one. lds: 8 KB of the wave's own.
template <class E, int NB>
__device__ void safe_dkv(const AttnArgs& a, const Seq& q, int r0, int r1, int jw, bool key_on, int kvh, float* lds,
                         int lane, f32x16 (&dk)[NB], f32x16 (&dv)[NB]) {
  constexpr int ST = NB * 2;
  const int group = a.hq / a.hk, shift = q.lk - q.lq, key = jw + (lane & 31);
  const float c = a.scale * kLog2e;
  const int64_t at = q.k0 + (key_on ? key : 0);
  const E* kp = static_cast<const E*>(a.k.p) + at * a.k.ts + kvh * a.k.hs;
  const E* vp = static_cast<const E*>(a.v.p) + at * a.v.ts + kvh * a.v.hs;
  const float2* stat = a.stat + (int64_t(kvh) * a.nq + q.q0) * group;
  auto q_row = [&](int r) {
    const int tok = r / group;
    return static_cast<const E*>(a.q.p) + int64_t(q.q0 + tok) * a.q.ts + (kvh * group + r - tok * group) * a.q.hs;
  };
  auto g_row = [&](int r) {
    const int tok = r / group;
    return static_cast<const E*>(a.dout.p) + int64_t(q.q0 + tok) * a.dout.ts +
           (kvh * group + r - tok * group) * a.dout.hs;
  };
  typename AttnType<E>::frag kf[ST], vf[ST];
#pragma unroll
  for (int s = 0; s < ST; ++s) {
    kf[s] = row_from<E>(kp, key_on, s, a.dim, lane);
    vf[s] = row_from<E>(vp, key_on, s, a.dim, lane);
  }
#pragma unroll
  for (int d = 0; d < NB; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) dk[d][e] = dv[d][e] = 0.f;
  for (int t0 = r0; t0 < r1; t0 += 32) {
    if (!any_sees(a, t0 / group + shift, min(t0 + 31, r1 - 1) / group + shift, jw, jw + 31, q.lk)) continue;
    const int mine = min(t0 + (lane & 31), r1 - 1);
    const bool on = t0 + (lane & 31) < r1;
    f32x16 s = scores_from<E, ST>(q_row(mine), on, kf, a.dim, lane);
    f32x16 dp = scores_from<E, ST>(g_row(mine), on, vf, a.dim, lane);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float2 st = stat[min(t0 + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3), r1 - 1)];
      s[e] = __builtin_amdgcn_exp2f(fmaf(s[e], c, -st.x)) * kWeightBack<AttnType<E>>;
      dp[e] = s[e] * (dp[e] - st.y);
    }
    put_factors(lds, s, lane);
    put_factors(lds + 1024, dp, lane);
    wave_fence();
    auto sees = [&](int i) {
      const int p = (t0 + i) / group + shift;
      return key_on && t0 + i < r1 && key <= p + a.right && (key >= p - a.left || key < a.sinks);
    };
    add_rows<E, NB>(dv, lds, [&](int i) { return g_row(min(t0 + i, r1 - 1)); }, sees, 0, a.dim, lane);
    add_rows<E, NB>(dk, lds + 1024, [&](int i) { return q_row(min(t0 + i, r1 - 1)); }, sees, 0, a.dim, lane);
    wave_fence();
  }
}

// dq and delta: 128 rows a workgroup, 32 a wave.
template <class E, int NB>
__global__ __launch_bounds__(256, sizeof(E) == 4 ? 1 : 2) void attn_dq(AttnArgs a, int tiles) {
  typedef Tile<E, NB> T;
  typedef AttnType<E> A;
  typedef typename A::frag frag;
  constexpr int KB = kKeyTile / 32, ST = NB * 2, kAhead = A::wide ? 1 : 4;
  // The half types' second product. Heads of 64 and less: sum_j P_ij k_j,
  // which the error of delta is taken off with at the end. Wider ones have no
  // registers for it: what rounding left of dS goes through the product as well,
  // which makes up for delta's error.
  constexpr bool kMean = !A::wide && NB <= 2;
  constexpr int kTileBytes = kKeyTile * T::kPitch;
  __shared__ __attribute__((aligned(1024))) unsigned char s_mem[4 * kTileBytes];
  const int lane = threadIdx.x & 63, l32 = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = a.hq / a.hk;
  const int w = xcd_remap(blockIdx.x, gridDim.x);
  const int tile = w % tiles, kvh = w / tiles;
  int inside;
  const int b = find_sequence(a.cu_q, a.batch, group, kRowsWg, tile, &inside);
  const Seq q = sequence(a, b);
  const int rows = q.lq * group;
  if (inside < 0 || inside > rows / kRowsWg) return;
  const int r0 = inside * kRowsWg;
  if (r0 >= rows) return;
  const int last = min(rows - 1, r0 + kRowsWg - 1) / group;
  const int shift = q.lk - q.lq;
  const KeyTiles kt = key_tiles<kKeyTile>(a, r0 / group + shift, last + shift, q.lk);
  const int wrow = r0 + 32 * wave, row = wrow + l32;
  const bool on = row < rows, wave_on = wrow < rows;
  const int tok = on ? row / group : last, head = kvh * group + (on ? row - tok * group : 0);
  const int p = tok + shift, lo = p - a.left, hi = min(p + a.right, q.lk - 1);
  const int pw0 = min(wrow, rows - 1) / group + shift, pw1 = min(wrow + 31, rows - 1) / group + shift;
  const int64_t q_at = q.q0 + tok;
  frag qf[ST], df[ST];
  float delta = 0.f, squares = 0.f, out_squares = 0.f, out_most = 0.f;  // o . do, do . do, o . o, largest |o|
  {
    const E* qp = static_cast<const E*>(a.q.p) + q_at * a.q.ts + head * a.q.hs;
    const E* dp = static_cast<const E*>(a.dout.p) + q_at * a.dout.ts + head * a.dout.hs;
    const E* op = static_cast<const E*>(a.o.p) + q_at * a.o.ts + head * a.o.hs;
#pragma unroll
    for (int s = 0; s < ST; ++s) {
      qf[s] = row_from<E>(qp, on, s, a.dim, lane);
      df[s] = row_from<E>(dp, on, s, a.dim, lane);
      const frag of = row_from<E>(op, on, s, a.dim, lane);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        delta = fmaf(float(of[e]), float(df[s][e]), delta);
        if constexpr (A::narrow) {
          squares = fmaf(float(df[s][e]), float(df[s][e]), squares);
          out_squares = fmaf(float(of[e]), float(of[e]), out_squares);
          out_most = fmaxf(out_most, fabsf(float(of[e])));
        }
      }
    }
  }
  delta += __shfl_xor(delta, 32);
  int up = 0;  // dS is raised by 2^up
  bool low_out = false;
  if constexpr (A::narrow) {
    squares += __shfl_xor(squares, 32);
    out_squares += __shfl_xor(out_squares, 32);
    up = kScoreShift - (exponent_of(squares) >> 1);
    low_out = fmaxf(out_most, __shfl_xor(out_most, 32)) < kLeastOut;
  }
  const float lse = on ? a.lse[int64_t(head) * a.nq + q_at] : 0.f;
  const float lse2 = lse == -INFINITY ? 0.f : lse * kLog2e;
  // fp16: weights raised by 2^15 where they are rounded too (for the mean), else by 2^up at once
  float lse_w = A::narrow ? lse2 - (kMean ? 15.f : float(up)) : lse2;
  float ds_factor = A::narrow && kMean ? power_of_two(up - 15) : 1.f;
  const E* kbase = static_cast<const E*>(a.k.p) + int64_t(q.k0) * a.k.ts + kvh * a.k.hs;
  const E* vbase = static_cast<const E*>(a.v.p) + int64_t(q.k0) * a.v.ts + kvh * a.v.hs;
  const typename T::Lane at = T::lane_of(lane);
  f32x16 acc[NB], mean[kMean ? NB : 1];
  float sum[2], most;  // sum of P dP; largest |dS| of fp16
  auto clear = [&]() {
#pragma unroll
    for (int d = 0; d < NB; ++d)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[d][e] = 0.f;
#pragma unroll
    for (int d = 0; d < (kMean ? NB : 1); ++d)
#pragma unroll
      for (int e = 0; e < 16; ++e) mean[d][e] = 0.f;
    sum[0] = sum[1] = most = 0.f;
  };
  const float c = a.scale * kLog2e;

  typename T::template Copy<kKeyTile, 4> kc, vc;
  kc.start(a.k.ts, a.dim, wave, lane);
  vc.start(a.v.ts, a.dim, wave, lane);
  auto fetch = [&](int it, int buf) {
    const int t0 = kt.at(it) * kKeyTile;
    unsigned char* dst = s_mem + buf * 2 * kTileBytes;
    kc.run(dst, kbase + t0 * a.k.ts, a.k.ts, q.lk - t0);
    vc.run(dst + kTileBytes, vbase + t0 * a.v.ts, a.v.ts, q.lk - t0);
  };
  auto compute = [&](int it, int buf) {
    const unsigned char* ks = s_mem + buf * 2 * kTileBytes;
    const unsigned char* vs = ks + kTileBytes;
    const int jt = kt.at(it) * kKeyTile;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      const int j0 = jt + 32 * kb, j1 = j0 + 31;
      if (!wave_on || !any_sees(a, pw0, pw1, j0, j1, q.lk)) continue;
      const bool all = all_see(a, pw0, pw1, j0, j1, q.lk);
      f32x16 s, dp;
#pragma unroll
      for (int e = 0; e < 16; ++e) s[e] = dp[e] = 0.f;
      products<2 * ST, kAhead, frag>(
          [&](int i, frag& f) { f = T::row(i < ST ? ks : vs, 32 * kb, i % ST, at); },
          [&](int i, const frag& f) {
            if (i < ST)
              s = A::mma(f, qf[i], s);
            else
              dp = A::mma(f, df[i - ST], dp);
          });
      if (!all) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int j = j0 + 4 * h + 8 * (e >> 2) + (e & 3);
          const bool sees = j <= hi && (j >= lo || j < a.sinks);
          s[e] = sees ? s[e] : -INFINITY;
          dp[e] = sees ? dp[e] : 0.f;
        }
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float w = __builtin_amdgcn_exp2f(fmaf(s[e], c, -lse_w)), wd = w * dp[e];
        sum[e & 1] += wd;
        s[e] = fmaf(-w, delta, wd);
        if constexpr (A::narrow && kMean) s[e] *= ds_factor;
        if constexpr (A::narrow) most = fmaxf(most, fabsf(s[e]));
        if constexpr (kMean) dp[e] = w;
      }
      const frag sf[2] = {pack_frag8<E>(s, 0), pack_frag8<E>(s, 1)};
      if constexpr (A::wide) {
        products<2 * NB, kAhead, frag>(
            [&](int i, frag& f) { f = T::col(ks, 32 * kb, i / NB, i % NB, at); },
            [&](int i, const frag& f) { acc[i % NB] = A::mma(f, sf[i / NB], acc[i % NB]); });
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) s[e] = kMean ? dp[e] : s[e] - float(sf[e / 8][e % 8]);
        const frag rest[2] = {pack_frag8<E>(s, 0), pack_frag8<E>(s, 1)};
        products<2 * NB, kAhead, frag>(
            [&](int i, frag& f) { f = T::col(ks, 32 * kb, i / NB, i % NB, at); },
            [&](int i, const frag& f) {
              acc[i % NB] = A::mma(f, sf[i / NB], acc[i % NB]);
              f32x16& to = kMean ? mean[i % (kMean ? NB : 1)] : acc[i % NB];
              to = A::mma(f, rest[i / NB], to);
            });
      }
    }
  };
  float2 half;
  for (int pass = 0;; ++pass) {
    clear();
    if (kt.n > 0) fetch(0, 0);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    for (int it = 0; it < kt.n; ++it) {
      if (it + 1 < kt.n) fetch(it + 1, (it & 1) ^ 1);
      compute(it, it & 1);
      __builtin_amdgcn_s_waitcnt(0);
      bare_barrier();
    }
    half = both_halves(sum[0] + sum[1]);
    if constexpr (A::narrow) {
      const float back = power_of_two(kMean ? -15 : -up);
      half.x *= back;
      half.y *= back;
      const float noise = sqrtf(squares * out_squares) * (fabsf(lse2) + 16.f) * kScoreNoise;
      most = fmaxf(fmaxf(most, __shfl_xor(most, 32)), noise * power_of_two(up));
      if (pass > 0) break;
      const bool redo = on && most > 0.f && most < INFINITY &&
                        (most >= kMostScore || most < kLeastScore || (low_out && most < kDeltaScore));
      // the whole workgroup walks again, or none of it (all reads of the tiles are done)
      uint32_t* flags = reinterpret_cast<uint32_t*>(s_mem);
      const bool mine = __any(redo);
      if (lane == 0) flags[wave] = mine;
      __syncthreads();
      const uint32_t again = flags[0] | flags[1] | flags[2] | flags[3];
      __syncthreads();
      if (again == 0) break;
      if (redo) {
        up = min(up + 13 - exponent_of(most), 100);
        lse_w = lse2 - (kMean ? 15.f : float(up));
        ds_factor = kMean ? power_of_two(up - 15) : 1.f;
        delta = half.x + half.y;
      }
    } else {
      break;
    }
  }
  if constexpr (A::narrow) {
    int largest = on && most > 0.f ? exponent_of(most) - up : kNoScore;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) largest = max(largest, __shfl_xor(largest, o));
    if (wave_on && lane == 0) a.score_exp[(int64_t(kvh) * tiles + tile) * 4 + wave] = largest;
  }
  if constexpr (kMean) {
    const float off = (half.x + half.y - delta) * ds_factor;  // as acc and mean are raised
#pragma unroll
    for (int d = 0; d < NB; ++d)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[d][e] = fmaf(-off, mean[d][e], acc[d][e]);
  }
  delta = half.x + half.y;
  if (on && h == 0)
    a.stat[(int64_t(kvh) * a.nq + q.q0) * group + row] = make_float2(lse2 - kWeightShift<A>, delta);
  const uint32_t bad = bad_rows(on ? zero_if_finite<NB>(acc) : 0.f);
  E* const dqp = static_cast<E*>(a.dq) + (q_at * a.hq + head) * a.dim;
  const bool mine = (bad >> l32) & 1u;
  if (on && !mine) store_rows<E, NB>(dqp, acc, A::narrow ? __builtin_ldexpf(a.scale, -up) : a.scale, a.dim, h);
  if (bad != 0) {
    safe_dq<E, NB>(a, q, kt, pw0, pw1, p, on, static_cast<const E*>(a.q.p) + q_at * a.q.ts + head * a.q.hs,
                   static_cast<const E*>(a.dout.p) + q_at * a.dout.ts + head * a.dout.hs, kvh, lse2, delta,
                   reinterpret_cast<float*>(s_mem) + wave * 1024, lane, acc);
    if (on && mine) store_rows<E, NB>(dqp, acc, a.scale, a.dim, h);
  }
}

// Token `t` as a bound of a sequence's tokens [0, lq].
__device__ __forceinline__ int token_at(int64_t t, int lq) { return t < 0 ? 0 : t > lq ? lq : int(t); }

// What a tile's rows need besides their elements.
template <int ROWS>
struct alignas(16) RowStats {
  float2 stat[ROWS];  // base-2 lse (0 for a row that sees nothing) less the weights' shift, and delta
  int pos[ROWS];      // position, or far below every window for a row that is not there
};
constexpr int kNoRow = -(1 << 30);  // kNoRow + right < 0, and kNoRow - left does not wrap

// dk and dv of 32 keys a wave. SINK = false: 128 keys a workgroup, the four
// waves take 32 each and share the row tiles. SINK = true: 32 keys (of the
// sinks) a workgroup, the rows past the band, one chunk; every wave walks row
// tiles of its own, and the four sums are joined at the end.
template <class E, int NB, bool SINK>
__global__ __launch_bounds__(256, sizeof(E) == 4 ? 1 : 2) void attn_dkv(AttnArgs a, int tiles, int parts) {
  typedef Tile<E, NB> T;
  typedef AttnType<E> A;
  typedef typename A::frag frag;
  constexpr int ST = NB * 2, kAhead = A::wide ? 1 : SINK ? 2 : 4;
  // Rows between two barriers: heads of 64 and less have the LDS for twice as many (the fp16 size above 182 us with
  // its forward, 187 without).
  constexpr int kRows = SINK || A::wide || NB > 2 ? kRowTile : 2 * kRowTile;
  typedef RowStats<kRows> Stats;
  constexpr int kTileBytes = kRows * T::kPitch;
  constexpr int kSets = SINK ? 4 : 1;                       // LDS tile sets: a wave's own, or shared
  constexpr int kBuffers = SINK ? 1 : 2;                    // a sink workgroup's other half waits on the CU instead
  constexpr int kLds = kSets * kBuffers * 2 * kTileBytes;
  constexpr int kJoin = SINK ? 3 * NB * 16 * 64 * 4 : 0;  // the waves' sums at the end
  // heads of 128: V's fragments stay in LDS (in registers, with K's and the sums, they would spill)
  constexpr bool kKeepV = NB < 4;
  constexpr int kV = kKeepV ? 0 : (SINK ? 32 : kKeysWg) * T::kPitch;
  // one array: with two, every copy to LDS is tracked by the array it goes to,
  // and a tile's reads wait for the next tile's copies
  constexpr int kTiles = kLds > kJoin ? kLds : kJoin;
  __shared__ __attribute__((aligned(1024))) unsigned char s_mem[kTiles + kV + kSets * kBuffers * sizeof(Stats)];
  unsigned char* const s_v = s_mem + kTiles;
  Stats* const s_stat = reinterpret_cast<Stats*>(s_mem + kTiles + kV);
  const int lane = threadIdx.x & 63, l32 = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = a.hq / a.hk;
  const int sink_blocks = (a.sinks + 31) / 32;
  const int w = xcd_remap(blockIdx.x, gridDim.x);
  const int tile = w % tiles, kvh = (w / tiles) % a.hk;
  const int sink_block = SINK ? w / tiles / a.hk : 0, part = SINK ? 0 : w / tiles / a.hk;
  int inside;
  const int b = SINK ? find_sequence(a.cu_q, a.batch, group, kSinkChunk, tile, &inside)
                     : find_sequence(a.cu_k, a.batch, 1, kKeysWg, tile, &inside);
  const Seq q = sequence(a, b);
  const int shift = q.lk - q.lq, rows = q.lq * group;
  if (inside < 0) return;
  int j0, r_begin, r_end, cap = 0;
  // rows that see a key of the tile [0, kKeysWg) inside the band end here
  const int band_end = token_at(int64_t(kKeysWg) + a.left - shift, q.lq) * group;
  if constexpr (SINK) {
    if (inside > rows / kSinkChunk) return;
    j0 = 32 * sink_block;
    r_begin = max(inside * kSinkChunk, band_end);
    r_end = min((inside + 1) * kSinkChunk, rows);
    if (r_begin >= r_end) return;  // a chunk that nothing reads
  } else {
    cap = a.cu_k ? clamp_to(a.cu_k[b + 1], q.k0, a.nk) - q.k0 : a.nk;
    if (inside > cap / kKeysWg) return;
    j0 = inside * kKeysWg;
    if (j0 >= cap) return;
    const int last = min(j0 + kKeysWg, q.lk) - 1;
    r_begin = token_at(int64_t(j0) - a.right - shift, q.lq) * group;
    r_end = token_at(int64_t(last) + a.left - shift + 1, q.lq) * group;
    if (j0 == 0 && a.sinks > 0) r_end = band_end;
    if (j0 >= q.lk) r_end = r_begin;
    if (parts > 1 && r_end > r_begin) {  // this workgroup's part of the row tiles
      const int n = (r_end - r_begin + kRowTile * group - 1) / (kRowTile * group);  // whole tokens
      const int from = r_begin, unit = kRowTile * group;
      r_begin = from + int(int64_t(n) * part / parts) * unit;
      r_end = min(r_end, from + int(int64_t(n) * (part + 1) / parts) * unit);
    }
  }
  const int jw = SINK ? j0 : j0 + 32 * wave, key = jw + l32;  // this wave's keys, this lane's
  const bool key_on = key < q.lk && (!SINK || key < a.sinks);
  frag kf[ST], vf[kKeepV ? ST : 1];
  {
    const int64_t at = q.k0 + (key_on ? key : 0);
    const E* kp = static_cast<const E*>(a.k.p) + at * a.k.ts + kvh * a.k.hs;
    const E* vp = static_cast<const E*>(a.v.p) + at * a.v.ts + kvh * a.v.hs;
#pragma unroll
    for (int s = 0; s < ST; ++s) {
      kf[s] = row_from<E>(kp, key_on, s, a.dim, lane);
      if constexpr (kKeepV) vf[s] = row_from<E>(vp, key_on, s, a.dim, lane);
    }
  }
  if constexpr (!kKeepV) {
    typename T::template Copy<SINK ? 32 : kKeysWg, 4> vc;
    vc.start(a.v.ts, a.dim, wave, lane);
    vc.run(s_v, static_cast<const E*>(a.v.p) + int64_t(q.k0 + j0) * a.v.ts + kvh * a.v.hs, a.v.ts, q.lk - j0);
  }
  const typename T::Lane lanes = T::lane_of(lane);
  f32x16 dk[NB], dv[NB];
#pragma unroll
  for (int d = 0; d < NB; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) dk[d][e] = dv[d][e] = 0.f;
  const float c = a.scale * kLog2e;
  int up = 0;  // dS is raised by 2^up, 2^15 of them by its weight
  if constexpr (A::narrow) {
    if (r_end > r_begin) {
      const int dq_tiles = int(int64_t(a.nq) * group / kRowsWg) + a.batch;  // as launched
      const int first = (a.cu_q ? first_tile(a.cu_q, b, group, kRowsWg) : 0) * 4;
      const int32_t* exponents = a.score_exp + int64_t(kvh) * dq_tiles * 4;
      int largest = kNoScore;
      for (int i = r_begin / 32 + lane; i <= (r_end - 1) / 32; i += 64)
        largest = max(largest, exponents[clamp_to(first + i, 0, dq_tiles * 4 - 1)]);
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) largest = max(largest, __shfl_xor(largest, o));
      up = clamp_to(14 - __builtin_amdgcn_readfirstlane(largest), -60, 100);
    }
  }
  const float ds_factor = power_of_two(up - 15);
  const float dk_factor = A::narrow ? __builtin_ldexpf(a.scale, -up) : a.scale;
  const int n_tiles = r_end > r_begin ? (r_end - r_begin + kRows - 1) / kRows : 0;
  const E* qbase = static_cast<const E*>(a.q.p) + int64_t(q.q0) * a.q.ts + int64_t(kvh) * group * a.q.hs;
  const E* dbase = static_cast<const E*>(a.dout.p) + int64_t(q.q0) * a.dout.ts + int64_t(kvh) * group * a.dout.hs;

  const float2* stat = a.stat + (int64_t(kvh) * a.nq + q.q0) * group;

  // The rows of a tile as copies: offsets from the tile's first token, the same
  // for every tile where the group divides the tile.
  constexpr int kCopies = kRows / T::kRowsPerCopy, kStep = SINK ? 1 : 4, kMine = (kCopies + kStep - 1) / kStep;
  const bool even = kRowTile % group == 0;
  const int tok_begin = r_begin / group, tok_step = kRowTile / group;
  // of the block of kRowTile rows n
  auto first_token = [&](int n) { return even ? tok_begin + n * tok_step : (r_begin + n * kRowTile) / group; };
  uint32_t oq[kMine], od[kMine];
  auto offsets = [&](int it) {
    const int t0 = r_begin + it * kRows, tok0 = first_token(it * (kRows / kRowTile));
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
      const int rr = (SINK ? j : j * 4 + wave) * T::kRowsPerCopy + lane / T::kChunks;
      const int chunk = (lane % T::kChunks) ^ T::key(rr);
      const int tok = (t0 + rr) / group, g = t0 + rr - tok * group;
      const bool in = chunk * T::kPer < a.dim;
      oq[j] = in ? uint32_t(tok - tok0) * uint32_t(a.q.ts * T::kElt) + uint32_t(g) * uint32_t(a.q.hs * T::kElt) +
                       chunk * 16
                 : 0x80000000u;
      od[j] = in ? uint32_t(tok - tok0) * uint32_t(a.dout.ts * T::kElt) +
                       uint32_t(g) * uint32_t(a.dout.hs * T::kElt) + chunk * 16
                 : 0x80000000u;
    }
  };
  if (even) offsets(0);
  auto fetch = [&](int it, int set) {
    unsigned char* dst = s_mem + set * 2 * kTileBytes;
    const int t0 = r_begin + it * kRows, tok0 = first_token(it * (kRows / kRowTile));
    const buffer_t bq = buffer_of(qbase + tok0 * a.q.ts, 0x7fffffffu);
    const buffer_t bd = buffer_of(dbase + tok0 * a.dout.ts, 0x7fffffffu);
    if (!even) offsets(it);
    // Past the rows: out of the buffer. (In place, in the last tile: a register
    // that a copy's offset was in is not reused before the copy has landed.)
    if (t0 + kRows > r_end) {
#pragma unroll
      for (int j = 0; j < kMine; ++j) {
        const bool in = t0 + (SINK ? j : j * 4 + wave) * T::kRowsPerCopy + lane / T::kChunks < r_end;
        oq[j] = in ? oq[j] : 0x80000000u;
        od[j] = in ? od[j] : 0x80000000u;
      }
    }
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
      const int n = SINK ? j : j * 4 + wave;
      if (kCopies % kStep != 0 && n >= kCopies) break;
      copy_lds16(bq, oq[j], dst + n * 1024);
      copy_lds16(bd, od[j], dst + kTileBytes + n * 1024);
    }
    if (SINK || wave == 3) {
      const buffer_t bs = buffer_of(stat + t0, uint32_t(min(kRows, r_end - t0)) * 8);
#pragma unroll
      for (int i = 0; i < kRows / 32; ++i)
        copy_lds4(bs, 256 * i + lane * 4, reinterpret_cast<unsigned char*>(s_stat[set].stat) + 256 * i);
      if (lane < kRows) s_stat[set].pos[lane] = t0 + lane < r_end ? (t0 + lane) / group + shift : kNoRow;
    }
  };
  auto block = [&](int it, int set, int rb) {  // rows 32 rb .. of tile `it`
    typename T::Lane at = lanes;
    if constexpr (!kKeepV) at.fresh();
    const unsigned char* qs = s_mem + set * 2 * kTileBytes + rb * kRowTile * T::kPitch;
    const unsigned char* ds_ = qs + kTileBytes;
    const int t0 = r_begin + it * kRows + rb * kRowTile;
    if (kRows > kRowTile && t0 >= r_end) return;
    const int p0 = first_token(it * (kRows / kRowTile) + rb) + shift;
    const int p1 = (even ? min(p0 + max(tok_step, 1) - 1, (r_end - 1) / group + shift)
                         : min(t0 + kRowTile - 1, r_end - 1) / group + shift);
    const int j1 = jw + 31;
    if (!any_sees(a, p0, p1, jw, j1, q.lk)) return;
    const bool all = t0 + kRowTile <= r_end && all_see(a, p0, p1, jw, j1, q.lk);
    f32x16 s, dp;
#pragma unroll
    for (int e = 0; e < 16; ++e) s[e] = dp[e] = 0.f;
    struct Pair {
      frag row, v;
    };
    products<ST, kAhead, frag>([&](int i, frag& f) { f = T::row(qs, 0, i, at); },
                               [&](int i, const frag& f) { s = A::mma(f, kf[i], s); });
    if constexpr (kKeepV)
      products<ST, kAhead, frag>([&](int i, frag& f) { f = T::row(ds_, 0, i, at); },
                                 [&](int i, const frag& f) { dp = A::mma(f, vf[i], dp); });
    else
      products<ST, (kAhead + 1) / 2, Pair>(
          [&](int i, Pair& f) {
            f.row = T::row(ds_, 0, i, at);
            f.v = T::row(s_v, SINK ? 0 : 32 * wave, i, at);
          },
          [&](int i, const Pair& f) { dp = A::mma(f.row, f.v, dp); });
    const float2* const stats = s_stat[set].stat + rb * kRowTile;
    const int* const at_pos = s_stat[set].pos + rb * kRowTile;
    // weights into s, score gradients into dp; of what a row does not see, zero.
    // Both branches end with their fragments, so that the products are a block
    // of their own and their reads can be put in order.
    frag pf[2], sf[2];
    auto pack = [&]() {
#pragma unroll
      for (int ss = 0; ss < 2; ++ss) {
        pf[ss] = pack_frag8<E>(s, ss);
        sf[ss] = pack_frag8<E>(dp, ss);
      }
    };
    if (all) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float4 s0 = read_lds<float4>(&stats[8 * g + 4 * h]), s1 = read_lds<float4>(&stats[8 * g + 4 * h + 2]);
        const float lv[4] = {s0.x, s0.z, s1.x, s1.z}, ev[4] = {s0.y, s0.w, s1.y, s1.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = 4 * g + i;
          s[e] = __builtin_amdgcn_exp2f(fmaf(s[e], c, -lv[i]));
          dp[e] = s[e] * (dp[e] - ev[i]);
          if constexpr (A::narrow) dp[e] *= ds_factor;
        }
      }
      pack();
    } else {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float4 s0 = read_lds<float4>(&stats[8 * g + 4 * h]), s1 = read_lds<float4>(&stats[8 * g + 4 * h + 2]);
        const int4 po = read_lds<int4>(&at_pos[8 * g + 4 * h]);
        const float lv[4] = {s0.x, s0.z, s1.x, s1.z}, ev[4] = {s0.y, s0.w, s1.y, s1.w};
        const int pv[4] = {po.x, po.y, po.z, po.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = 4 * g + i;
          const int from = key < a.sinks ? 0 : pv[i] - a.left, to = key_on ? pv[i] + a.right : -1;
          const bool sees = (key <= to) & (key >= from);
          const float pr = __builtin_amdgcn_exp2f(fmaf(s[e], c, -lv[i]));
          float d = pr * (dp[e] - ev[i]);
          if constexpr (A::narrow) d *= ds_factor;
          s[e] = sees ? pr : 0.f;
          dp[e] = sees ? d : 0.f;
        }
      }
      pack();
    }
    products<4 * NB, kAhead, frag>(
        [&](int i, frag& f) { f = T::col(i < 2 * NB ? ds_ : qs, 0, i / NB % 2, i % NB, at); },
        [&](int i, const frag& f) {
          if (i < 2 * NB)
            dv[i % NB] = A::mma(f, pf[i / NB], dv[i % NB]);
          else
            dk[i % NB] = A::mma(f, sf[i / NB - 2], dk[i % NB]);
        });
  };
  auto compute = [&](int it, int set) {
#pragma unroll
    for (int rb = 0; rb < kRows / kRowTile; ++rb) block(it, set, rb);
  };
  if constexpr (!SINK) {
    if (n_tiles > 0) fetch(0, 0);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    for (int it = 0; it < n_tiles; ++it) {
      if (it + 1 < n_tiles) fetch(it + 1, (it & 1) ^ 1);
      compute(it, it & 1);
      __builtin_amdgcn_s_waitcnt(0);
      bare_barrier();
    }
    const uint32_t bad = bad_rows(key < cap ? zero_if_finite<NB>(dk) + zero_if_finite<NB>(dv) : 0.f);
    // where a key's sums go: to the sinks' slots (joined with the later rows'),
    // to this part's (joined with the other parts'), or out
    auto slot = [&](int j) -> float* {
      if (j < a.sinks) return a.sink_part + (((int64_t(b) * parts + part) * a.hk + kvh) * a.sinks + j) * 2 * a.dim;
      if (parts > 1) return a.dkv_part + ((int64_t(part) * a.nk + q.k0 + j) * a.hk + kvh) * 2 * a.dim;
      return nullptr;
    };
    auto store = [&](bool which, float k_factor, float v_factor) {
      if (key >= cap || !which) return;
      if (float* dst = slot(key)) {
        store_rows<float, NB>(dst, dk, k_factor, a.dim, h);
        store_rows<float, NB>(dst + a.dim, dv, v_factor, a.dim, h);
      } else {
        const int64_t at = (int64_t(q.k0 + key) * a.hk + kvh) * a.dim;
        store_rows<E, NB>(static_cast<E*>(a.dk) + at, dk, k_factor, a.dim, h);
        store_rows<E, NB>(static_cast<E*>(a.dv) + at, dv, v_factor, a.dim, h);
      }
    };
    const bool mine = (bad >> l32) & 1u;
    store(!mine, dk_factor, kWeightBack<A>);
    if (bad != 0) {
      safe_dkv<E, NB>(a, q, r_begin, r_end, jw, key_on, kvh, reinterpret_cast<float*>(s_mem) + wave * 2048, lane, dk,
                      dv);
      store(mine, a.scale, 1.f);
    }
  } else {
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    for (int it = wave; it < n_tiles; it += 4) {
      __builtin_amdgcn_s_waitcnt(0);  // the last tile's reads are done
      asm volatile("" ::: "memory");
      fetch(it, wave);
      __builtin_amdgcn_s_waitcnt(0);
      asm volatile("" ::: "memory");
      compute(it, wave);
    }
    // waves 1 - 3 hand over, first dk, then dv; wave 0 adds in wave order
    float* red = reinterpret_cast<float*>(s_mem);
    auto join = [&](f32x16 (&x)[NB]) {
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
      if (wave > 0) {
#pragma unroll
        for (int d = 0; d < NB; ++d)
#pragma unroll
          for (int e = 0; e < 16; ++e) red[(((wave - 1) * NB + d) * 16 + e) * 64 + lane] = x[d][e];
      }
      __syncthreads();
      if (wave == 0) {
#pragma unroll
        for (int i = 0; i < 3; ++i)
#pragma unroll
          for (int d = 0; d < NB; ++d)
#pragma unroll
            for (int e = 0; e < 16; ++e) x[d][e] += red[((i * NB + d) * 16 + e) * 64 + lane];
      }
    };
    join(dk);
    join(dv);
    if (wave == 0) {
      float* const slot = a.sink_part + (int64_t(a.batch) * parts + tile) * a.hk * a.sinks * 2 * a.dim +
                          int64_t(kvh) * a.sinks * 2 * a.dim;
      const uint32_t bad = bad_rows(key < a.sinks ? zero_if_finite<NB>(dk) + zero_if_finite<NB>(dv) : 0.f);
      auto store = [&](bool which, float k_factor, float v_factor) {
        if (key >= a.sinks || !which) return;
        float* dst = slot + int64_t(key) * 2 * a.dim;
        store_rows<float, NB>(dst, dk, k_factor, a.dim, h);
        store_rows<float, NB>(dst + a.dim, dv, v_factor, a.dim, h);
      };
      const bool mine = (bad >> l32) & 1u;
      store(!mine, dk_factor, kWeightBack<A>);
      if (bad != 0) {
        safe_dkv<E, NB>(a, q, r_begin, r_end, jw, key_on, kvh, red, lane, dk, dv);
        store(mine, a.scale, 1.f);
      }
    }
  }
}

// dk, dv of the sinks: the tile's own sums plus the chunks' in chunk order. One
// workgroup a (sequence, kv head, sink), one thread an element of dk or dv.
template <class E>
__global__ __launch_bounds__(256) void attn_sinks(AttnArgs a, int chunks, int parts) {
  const int64_t i = blockIdx.x;
  const int key = int(i % a.sinks), kvh = int(i / a.sinks % a.hk), b = int(i / a.sinks / a.hk), d = threadIdx.x;
  const Seq q = sequence(a, b);
  const int cap = a.cu_k ? clamp_to(a.cu_k[b + 1], q.k0, a.nk) - q.k0 : a.nk;
  if (key >= cap || d >= 2 * a.dim) return;
  const int group = a.hq / a.hk, rows = q.lq * group;
  const int shift = q.lk - q.lq;
  const int band_end = token_at(int64_t(kKeysWg) + a.left - shift, q.lq) * group;
  const int base = a.cu_q ? first_tile(a.cu_q, b, group, kSinkChunk) : 0;
  const int c0 = band_end / kSinkChunk, c1 = rows > band_end ? (rows + kSinkChunk - 1) / kSinkChunk : c0;
  const int64_t slot = int64_t(a.hk) * a.sinks * 2 * a.dim;
  const float* src = a.sink_part + (int64_t(kvh) * a.sinks + key) * 2 * a.dim + d;
  float v = 0.f;
  for (int t = 0; t < parts; ++t) v += src[(int64_t(b) * parts + t) * slot];
  src += int64_t(a.batch) * parts * slot;
#pragma unroll 8
  for (int t = c0; t < c1; ++t) v += src[clamp_to(base + t, 0, chunks - 1) * slot];
  E* dst = static_cast<E*>(d < a.dim ? a.dk : a.dv);
  dst[(int64_t(q.k0 + key) * a.hk + kvh) * a.dim + (d < a.dim ? d : d - a.dim)] = static_cast<E>(v);
}

// dk, dv of every (key, kv head) from the parts of the row walk, in part order:
// one thread four elements.
template <class E>
__global__ __launch_bounds__(256) void attn_parts(AttnArgs a, int parts) {
  const int64_t per = a.dim / 2, n = int64_t(a.nk) * a.hk * per;  // float4s of a part
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= n) return;
  const float4* src = reinterpret_cast<const float4*>(a.dkv_part) + i;
  float4 v = src[0];
  for (int t = 1; t < parts; ++t) {
    const float4 x = src[t * n];
    v.x += x.x;
    v.y += x.y;
    v.z += x.z;
    v.w += x.w;
  }
  const int64_t row = i / per;
  const int d = int(i - row * per) * 4;
  typedef E out4 __attribute__((ext_vector_type(4)));
  E* dst = static_cast<E*>(d < a.dim ? a.dk : a.dv) + row * a.dim + (d < a.dim ? d : d - a.dim);
  *reinterpret_cast<out4*>(dst) = out4{static_cast<E>(v.x), static_cast<E>(v.y), static_cast<E>(v.z),
                                       static_cast<E>(v.w)};
}

// Parts of the row walk of a key tile: few key tiles with many rows each (short
// sequences, many query heads to a kv head) would leave most of the chip idle
// (the fp16 size above: 182 us with its forward and four parts, 244 with one).
int row_parts(const AttnArgs& a) {
  const int64_t wgs = tiles_of(a.nk, a.batch, 1, kKeysWg) * a.hk, group = a.hq / a.hk;
  const int64_t reach = int64_t(a.left) + a.right + 1 + kKeysWg;
  const int64_t units = (reach < a.nq ? reach : a.nq) / kRowTile;  // tiles of a part are a multiple of the group
  int64_t p = kWantWgs / wgs;
  if (p > units * group / 16) p = units * group / 16;  // 16 row tiles a part at least
  if (p > units) p = units;
  return p < 2 ? 1 : p > 8 ? 8 : int(p);
}

template <class E, int NB>
hipError_t launch_shape(const AttnArgs& a, hipStream_t st) {
  const int group = a.hq / a.hk;
  if (a.nq > 0) {
    const int64_t tiles = tiles_of(a.nq, a.batch, group, kRowsWg);
    if (tiles * a.hk >= (int64_t(1) << 31)) return hipErrorInvalidValue;
    attn_dq<E, NB><<<unsigned(tiles * a.hk), 256, 0, st>>>(a, int(tiles));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.nk == 0) return hipSuccess;
  const int64_t tiles = tiles_of(a.nk, a.batch, 1, kKeysWg);
  if (tiles * a.hk >= (int64_t(1) << 31)) return hipErrorInvalidValue;
  const int parts = row_parts(a);
  attn_dkv<E, NB, false><<<unsigned(tiles * a.hk * parts), 256, 0, st>>>(a, int(tiles), parts);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (parts > 1) {
    const int64_t n = int64_t(a.nk) * a.hk * (a.dim / 2);
    attn_parts<E><<<unsigned((n + 255) / 256), 256, 0, st>>>(a, parts);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.sinks == 0) return hipSuccess;
  if (a.nq > 0) {
    const int64_t chunks = tiles_of(a.nq, a.batch, group, kSinkChunk);
    const int64_t wgs = chunks * a.hk * ((a.sinks + 31) / 32);
    if (wgs >= (int64_t(1) << 31)) return hipErrorInvalidValue;
    attn_dkv<E, NB, true><<<unsigned(wgs), 256, 0, st>>>(a, int(chunks), parts);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int64_t n = int64_t(a.batch) * a.hk * a.sinks;  // < 2^31: see the caller
  attn_sinks<E><<<unsigned(n), 256, 0, st>>>(a, int(tiles_of(a.nq, a.batch, group, kSinkChunk)), parts);
  return hipGetLastError();
}

template <class E>
hipError_t launch_type(const AttnArgs& a, hipStream_t st) {
  switch ((a.dim + 31) / 32) {
    case 1: return launch_shape<E, 1>(a, st);
    case 2: return launch_shape<E, 2>(a, st);
    case 3: return launch_shape<E, 3>(a, st);
    default: return launch_shape<E, 4>(a, st);
  }
}

}  // namespace

size_t attention_backward_stat_floats(const AttnArgs& a) { return size_t(a.hq) * a.nq * 2; }

size_t attention_backward_exponents(const AttnArgs& a) {
  return a.dtype == TR_SC_F16 ? size_t(tiles_of(a.nq, a.batch, a.hq / a.hk, kRowsWg)) * a.hk * 4 : 0;
}

size_t attention_backward_sink_floats(const AttnArgs& a) {
  if (a.sinks == 0) return 0;
  const int64_t slots = int64_t(a.batch) * row_parts(a) + tiles_of(a.nq, a.batch, a.hq / a.hk, kSinkChunk);
  return size_t(slots) * a.hk * a.sinks * 2 * a.dim;
}

size_t attention_backward_part_floats(const AttnArgs& a) {
  const int parts = row_parts(a);
  return parts > 1 ? size_t(parts) * a.nk * a.hk * 2 * a.dim : 0;
}

hipError_t launch_attention_backward(const AttnArgs& a, hipStream_t st) {
  if (a.dtype == TR_SC_BF16) return launch_type<__bf16>(a, st);
  if (a.dtype == TR_SC_F16) return launch_type<_Float16>(a, st);
  return launch_type<float>(a, st);
}

}  // namespace trsc
