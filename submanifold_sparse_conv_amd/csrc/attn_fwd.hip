// Windowed attention with sinks, forward: prompts and packed objects, and
// single tokens against a cache.
//
// Mathematics. Row i of a sequence (Lq queries, Lk keys) stands at
// p = i + Lk - Lq and sees key j when j <= p + right and (j >= p - left or
// j < sinks). o = sum_j e^{scale q.k_j - lse} v_j over the keys it sees, lse the
// log of the sum of the exponentials. One pass over the keys with the running
// maximum m and sum l: e^{scale (s - m)} is taken as 2^{(s - m) c},
// c = scale log2 e.
//
// Rows. The queries of the heads that share a key-value head are one matrix:
// row r of a sequence is token r / G, head r % G of the group (G = q heads / kv
// heads). A workgroup takes 128 consecutive rows of one kv head, 32 a wave.
//
// Products. S^T = K Q^T (keys down, queries across), so a lane holds scores of
// one query only: the maximum and the sum need one exchange between the two
// halves of the wave, the rescaling none. The registers of S^T are, as they
// are, fragments of P^T for O^T += V^T P^T when V's keys are taken in the same
// order, which the transposed LDS read of V gives (attn_common.h).
//
// Rounding. Scores, maxima, sums and the result's sums are fp32. The weights are
// rounded to the tensors' type for the product with V (the matrix units take
// half types; for fp32 tensors nothing is rounded), their sum takes them
// unrounded: the result is off by that rounding's average and its own last one.
// fp16's range is kept by a base that moves with the tiles (kMostSum16).
//
// What bounds it (ranges: cards and their clocks differ). bf16, 32,768 tokens, 16
// query and 4 kv heads of 128, 4096 keys back: 1.03 TFLOP in 0.99 to 1.05 ms, 0.98
// to 1.04 PFLOP/s, of 1.19 that a large library product reaches (both on clocks
// that power lowers): matrix units, one LDS fragment a product; fp16 1.05 to 1.09
// ms. bf16, 73,881 tokens, 16 heads of 64, 512 keys either way: 0.31 TFLOP in 411
// to 436 us, 708 to 750 TFLOP/s: vector instructions in 68 % of cycles (16
// exponentials, sums and packings to every 8 products, and the window's edges) and
// matrix units in 42 %, hardly at the same time; fp16 437 to 454 us. fp32, 2,877
// tokens in four sequences, 6 heads of 80 over 2, 255 either way: 54.5 us, four
// splits a row tile to reach the chip, the products' padding (80 of 96) and the
// join. Token form: bytes; 32 caches of up to 4100 keys, 4 kv heads of 128: 257 MB
// in 58.5 us, 4.4 TB/s (fp32 513 MB in 118); one cache of 65,540 keys: 134 MB in
// 35.6 us, 3.8 TB/s (fp32 72.5 us), the join's launch (5 us) included; 48 and 31 us
// where the last call has left part of them in the caches.
#include "attn_rows.h"

namespace trsc {
namespace {

// A lane's row of the output: `count` blocks of 32 columns from block `first`.
template <class E, int NB>
__device__ __forceinline__ void store_tile_row(const AttnArgs& a, int splits, int split, int head, int64_t q_at,
                                               const f32x16 (&acc)[NB], float mc, float l, int first, int count,
                                               bool with_sum, int h) {
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const float lg = l == 0.f ? -INFINITY : mc + __builtin_amdgcn_logf(l);  // base 2
  const int64_t at_row = (int64_t(split) * a.hq + head) * a.nq + q_at;
  typedef E out4 __attribute__((ext_vector_type(4)));
  E* const op = static_cast<E*>(const_cast<void*>(a.o.p)) + q_at * a.o.ts + head * a.o.hs;
  float* const pp = a.part + at_row * a.dim;
#pragma unroll
  for (int d = 0; d < NB; ++d) {
    if (d >= count) break;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int col = 32 * (first + d) + 8 * g + 4 * h;
      if (col >= a.dim) continue;
      if (splits == 1) {
        out4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = static_cast<E>(acc[d][4 * g + i] * inv);
        *reinterpret_cast<out4*>(op + col) = v;
      } else {
        *reinterpret_cast<float4*>(pp + col) = make_float4(acc[d][4 * g] * inv, acc[d][4 * g + 1] * inv,
                                                           acc[d][4 * g + 2] * inv, acc[d][4 * g + 3] * inv);
      }
    }
  }
  if (!with_sum) return;
  if (splits > 1)
    a.part[int64_t(splits) * a.hq * a.nq * a.dim + at_row] = lg;
  else if (a.lse != nullptr)
    a.lse[int64_t(head) * a.nq + q_at] = lg * 0.6931471805599453f;
}

// Where a workgroup of `rows_wg` rows and each of its waves' rows lie.
struct RowTile {
  Seq q;
  int rows, r0, last, shift;  // rows of the sequence; first row; last token; position of token 0
};
__device__ __forceinline__ bool row_tile(const AttnArgs& a, int tile, int rows_wg, RowTile* t) {
  const int group = a.hq / a.hk;
  int inside;
  const int b = find_sequence(a.cu_q, a.batch, group, rows_wg, tile, &inside);
  t->q = sequence(a, b);
  t->rows = t->q.lq * group;  // < 2^31 - 2^10 (checked by the caller)
  if (inside < 0 || inside > t->rows / rows_wg) return false;
  t->r0 = inside * rows_wg;
  if (t->r0 >= t->rows) return false;
  t->last = min(t->rows - 1, t->r0 + rows_wg - 1) / group;
  t->shift = t->q.lk - t->q.lq;
  return true;
}
struct WaveRows {
  bool any, on;       // the wave has rows; this lane has one
  int first;          // the wave's first row
  int tok, head;      // this lane's
  int lo, hi;         // keys that it sees: [lo, hi] (and the sinks up to hi)
  int p0, p1;         // positions of the wave's rows
};
__device__ __forceinline__ WaveRows wave_rows(const AttnArgs& a, const RowTile& t, int first, int kvh, int l32) {
  const int group = a.hq / a.hk;
  WaveRows w;
  w.first = first;
  const int row = first + l32;
  w.any = first < t.rows;
  w.on = row < t.rows;
  w.tok = w.on ? row / group : t.last;
  w.head = kvh * group + (w.on ? row - w.tok * group : 0);
  const int p = w.tok + t.shift;
  w.lo = p - a.left;
  w.hi = min(p + a.right, t.q.lk - 1);
  w.p0 = min(first, t.rows - 1) / group + t.shift;
  w.p1 = min(first + 31, t.rows - 1) / group + t.shift;
  return w;
}
// A tile of keys j0 .. j1 as the wave's rows see it.
__device__ __forceinline__ bool tile_seen(const AttnArgs& a, const WaveRows& w, int j0, int j1) {
  return w.any && j0 <= w.p1 + a.right && (j1 >= w.p0 - a.left || j0 < a.sinks);
}
__device__ __forceinline__ bool tile_whole(const AttnArgs& a, const WaveRows& w, int j0, int j1, int lk) {
  return j1 <= w.p0 + a.right && j1 < lk && (j0 >= w.p1 - a.left || j1 < a.sinks);
}

// A wave's rows again over the key tiles [first, end), adding only what each sees (attn_common.h): blocks d0 ..
// d0 + DN of O^T, the scaled maximum and the sum. lds: 4 KB of the wave's own.
template <class E, int NB, int KT, int DN>
__device__ void safe_rows(const AttnArgs& a, const RowTile& t, const KeyTiles& kt, int first, int end,
                          const WaveRows& w, int kvh, int d0, float* lds, int lane, f32x16 (&acc)[NB], float& mc,
                          float& l) {
  constexpr int ST = NB * 2;
  const Seq& q = t.q;
  const E* qp = static_cast<const E*>(a.q.p) + int64_t(q.q0 + w.tok) * a.q.ts + w.head * a.q.hs;
  const E* kbase = static_cast<const E*>(a.k.p) + int64_t(q.k0) * a.k.ts + kvh * a.k.hs;
  const E* vbase = static_cast<const E*>(a.v.p) + int64_t(q.k0) * a.v.ts + kvh * a.v.hs;
  const float c = a.scale * kLog2e;
  typename AttnType<E>::frag qf[ST];
#pragma unroll
  for (int st = 0; st < ST; ++st) qf[st] = row_from<E>(qp, w.on, st, a.dim, lane);
#pragma unroll
  for (int d = 0; d < DN; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[d][e] = 0.f;
  float m = -INFINITY;
  l = 0.f;
  for (int it = first * (KT / 32); it < end * (KT / 32); ++it) {
    const int j0 = kt.at(it / (KT / 32)) * KT + it % (KT / 32) * 32;
    if (!tile_seen(a, w, j0, j0 + 31)) continue;
    const int mine = j0 + (lane & 31);
    f32x16 s = scores_from<E, ST>(kbase + mine * a.k.ts, mine < q.lk, qf, a.dim, lane);
    hide(s, j0, w.lo, w.hi, a.sinks, lane);
    float mx = m;
#pragma unroll
    for (int e = 0; e < 16; ++e) mx = fmaxf(mx, s[e]);
    const float2 mh = both_halves(mx);
    mx = fmaxf(mh.x, mh.y);
    const float ms = mx == -INFINITY ? 0.f : mx, f = __builtin_amdgcn_exp2f((m - ms) * c);
    m = mx;
    l *= f;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      s[e] = __builtin_amdgcn_exp2f((s[e] - ms) * c);
      l += s[e];
    }
    if (f != 1.f) {
#pragma unroll
      for (int d = 0; d < DN; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[d][e] *= f;
    }
    put_factors(lds, s, lane);
    wave_fence();
    add_rows<E, DN>(
        acc, lds, [&](int i) { return vbase + min(j0 + i, q.lk - 1) * a.v.ts; },
        [&](int i) { return j0 + i <= w.hi && (j0 + i >= w.lo || j0 + i < a.sinks); }, d0, a.dim, lane);
    wave_fence();
  }
  mc = m * c;
  const float2 lh = both_halves(l);
  l = lh.x + lh.y;
}

template <class E, int NB, bool TOKEN>
struct FwdShape {
  typedef Tile<E, NB> T;
  // fp32 products are sixteen times the half types' time: smaller tiles waste less of them at the window's edges
  // (the fp32 size above: 85 us with tiles of 64 keys, 60 with 32)
  static constexpr int kKeys = TOKEN || sizeof(E) == 4 ? 32 : 64;
  static constexpr int kTileBytes = kKeys * T::kPitch;
  // token form: every wave has its own tiles
  static constexpr int kBuffers = (TOKEN && sizeof(E) == 4 && NB > 2) ? 1 : 2;
  static constexpr int kWaveSets = TOKEN ? 4 : 1;
  static constexpr int kLds = kBuffers * 2 * kTileBytes * kWaveSets;
  static constexpr int kRows = TOKEN ? 32 : 128;
};

template <class E, int NB, bool TOKEN>
__global__ __launch_bounds__(256, sizeof(E) == 4 && NB == 4                ? 1
                                  : sizeof(E) == 2 && NB <= 2 && !TOKEN ? 4
                                                                        : 2) void attn_fwd(AttnArgs a, int tiles,
                                                                                           int splits) {
  typedef FwdShape<E, NB, TOKEN> F;
  typedef Tile<E, NB> T;
  // 32-key blocks whose scores are held at once. Heads of 64 and less: one block, and four waves a SIMD (the size
  // above 426 us, with two blocks and fewer waves 455). Wider heads: two blocks (1.00 ms, with one 1.03).
  constexpr int KB = NB <= 2 ? 1 : F::kKeys / 32;
  __shared__ __attribute__((aligned(1024))) unsigned char s_mem[F::kLds];
  const int lane = threadIdx.x & 63, l32 = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = a.hq / a.hk;
  const int w = xcd_remap(blockIdx.x, gridDim.x);
  const int tile = w % tiles, kvh = (w / tiles) % a.hk, split = w / tiles / a.hk;
  RowTile t;
  if (!row_tile(a, tile, F::kRows, &t)) return;
  const Seq& q = t.q;
  const KeyTiles kt = key_tiles<F::kKeys>(a, t.r0 / group + t.shift, t.last + t.shift, q.lk);
  const WaveRows wr = wave_rows(a, t, t.r0 + (TOKEN ? 0 : 32 * wave), kvh, l32);
  const typename T::Lane at = T::lane_of(lane);
  RowState<E, NB, KB> st;
  st.start(static_cast<const E*>(a.q.p) + int64_t(q.q0 + wr.tok) * a.q.ts + wr.head * a.q.hs, wr.on, a.dim, lane);
  const E* kbase = static_cast<const E*>(a.k.p) + int64_t(q.k0) * a.k.ts + kvh * a.k.hs;
  const E* vbase = static_cast<const E*>(a.v.p) + int64_t(q.k0) * a.v.ts + kvh * a.v.hs;
  const float c = a.scale * kLog2e;

  const int first = int(int64_t(kt.n) * split / splits), end = int(int64_t(kt.n) * (split + 1) / splits);
  unsigned char* const mem = s_mem + (TOKEN ? wave * F::kBuffers * 2 * F::kTileBytes : 0);
  typename T::template Copy<F::kKeys, TOKEN ? 1 : 4> kc, vc;
  kc.start(a.k.ts, a.dim, TOKEN ? 0 : wave, lane);
  vc.start(a.v.ts, a.dim, TOKEN ? 0 : wave, lane);
  auto fetch = [&](int it, int buf) {
    const int t0 = kt.at(it) * F::kKeys;
    unsigned char* dst = mem + buf * 2 * F::kTileBytes;
    kc.run(dst, kbase + t0 * a.k.ts, a.k.ts, q.lk - t0);
    vc.run(dst + F::kTileBytes, vbase + t0 * a.v.ts, a.v.ts, q.lk - t0);
  };
  auto compute = [&](int it, int buf) {
    const unsigned char* ks = mem + buf * 2 * F::kTileBytes;
#pragma unroll
    for (int part = 0; part < F::kKeys / (32 * KB); ++part) {
      const int j0 = kt.at(it) * F::kKeys + part * 32 * KB, j1 = j0 + 32 * KB - 1;
      if (!tile_seen(a, wr, j0, j1)) continue;
      st.scores(ks + part * 32 * KB * T::kPitch, (a.dim + 15) / 16, at);
      if (!tile_whole(a, wr, j0, j1, q.lk)) {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) hide(st.s[kb], j0 + 32 * kb, wr.lo, wr.hi, a.sinks, lane);
      }
      st.weigh(c);
      st.multiply(ks + F::kTileBytes + part * 32 * KB * T::kPitch, at);
    }
  };

  if constexpr (!TOKEN) {
    if (first < end) fetch(first, 0);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    for (int it = first; it < end; it += 2) {  // two tiles a round: the buffers' addresses are constants
#pragma unroll
      for (int buf = 0; buf < 2; ++buf) {
        if (it + buf >= end) break;
        if (it + buf + 1 < end) fetch(it + buf + 1, buf ^ 1);
        compute(it + buf, buf);
        __builtin_amdgcn_s_waitcnt(0);
        bare_barrier();
      }
    }
  } else {
    // each wave its own tiles and LDS: no barrier in the loop
    constexpr int NBUF = F::kBuffers;
    int it = first + wave, buf = 0;
    if (NBUF == 2 && it < end) fetch(it, 0);
    for (; it < end; it += 4) {
      if constexpr (NBUF == 2) {
        __builtin_amdgcn_s_waitcnt(0);
        asm volatile("" ::: "memory");
        if (it + 4 < end) fetch(it + 4, buf ^ 1);
        compute(it, buf);
        buf ^= 1;
      } else {
        __builtin_amdgcn_s_waitcnt(0);  // the last tile's reads are done
        fetch(it, 0);
        __builtin_amdgcn_s_waitcnt(0);
        asm volatile("" ::: "memory");
        compute(it, 0);
      }
    }
  }
  st.join_halves();
  float mc = st.mc, l = st.l;
  bool writer = true;
  if constexpr (TOKEN) {
    // the four waves hold the same rows over different keys: join them in wave
    // order; wave w sums the blocks d = w, w + 4, ...
    float* red = reinterpret_cast<float*>(s_mem);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (lane < 32) {
      red[wave * 64 + lane] = mc;
      red[wave * 64 + 32 + lane] = l;
    }
    __syncthreads();
    float mm = -INFINITY;
#pragma unroll
    for (int i = 0; i < 4; ++i) mm = fmaxf(mm, red[i * 64 + l32]);
    float f[4], ll = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float mi = red[i * 64 + l32];
      f[i] = mi == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mi - mm);
      ll += f[i] * red[i * 64 + 32 + l32];
    }
    const float mine = f[0] * (wave == 0) + f[1] * (wave == 1) + f[2] * (wave == 2) + f[3] * (wave == 3);
    const bool any = mc != -INFINITY;
    mc = mm;
    l = ll;
    __syncthreads();
#pragma unroll
    for (int d = 0; d < NB; ++d)
#pragma unroll
      for (int e = 0; e < 16; ++e) red[((wave * NB + d) * 16 + e) * 64 + lane] = any ? st.acc[d][e] * mine : 0.f;
    __syncthreads();
    writer = wave < NB;
    if (writer) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) v += red[((i * NB + wave) * 16 + e) * 64 + lane];
        st.acc[0][e] = v;
      }
    }
  }
  // rows whose sums are not finite, again without what they do not see
  {
    float zero = 0.f;
    if (writer && wr.on) {
      if constexpr (TOKEN) {
#pragma unroll
        for (int e = 0; e < 16; ++e) zero = fmaf(st.acc[0][e], 0.f, zero);
      } else {
        zero = zero_if_finite<NB>(st.acc);
      }
    }
    uint32_t bad = bad_rows(zero);
    if constexpr (TOKEN) {  // each wave has seen some of the columns: the rows of all four
      uint32_t* flags = reinterpret_cast<uint32_t*>(s_mem);
      __syncthreads();
      if (lane == 0) flags[wave] = bad;
      __syncthreads();
      bad = flags[0] | flags[1] | flags[2] | flags[3];
    }
    auto store = [&](bool which) {
      if (wr.on && writer && which)
        store_tile_row<E, NB>(a, splits, split, wr.head, q.q0 + wr.tok, st.acc, mc, l, TOKEN ? wave : 0,
                              TOKEN ? 1 : NB, h == 0 && (!TOKEN || wave == 0), h);
    };
    const bool mine = (bad >> l32) & 1u;
    store(!mine);
    if (bad != 0) {
      if constexpr (TOKEN) __syncthreads();  // the flags are read
      if (!writer) return;
      safe_rows<E, NB, F::kKeys, TOKEN ? 1 : NB>(a, t, kt, first, end, wr, kvh, TOKEN ? wave : 0,
                                                 reinterpret_cast<float*>(s_mem) + wave * 1024, lane, st.acc, mc, l);
      store(mine);
    }
  }
}

// Joins the splits of a row: o = sum_s 2^{l_s - l} o_s, l = log2 sum_s 2^{l_s}.
// WPR waves a (token, head); a lane has four elements, and the splits are dealt
// to the lanes' groups in turn, whose sums are added in a fixed order.
template <class E, int WPR>
__global__ __launch_bounds__(256) void attn_join(AttnArgs a, int splits) {
  constexpr int kRows = 4 / WPR;
  __shared__ float s_max[4], s_sum[4];
  __shared__ float4 s_out[4][32];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, tw = wave % WPR;
  const int64_t n = int64_t(a.hq) * a.nq;
  const int64_t row = int64_t(blockIdx.x) * kRows + wave / WPR;  // head * nq + token
  if (row >= n) return;                                          // the whole team
  const float* stat = a.part + int64_t(splits) * n * a.dim + row;
  float mx = -INFINITY;
  for (int s = tw * 64 + lane; s < splits; s += WPR * 64) mx = fmaxf(mx, stat[s * n]);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o));
  if constexpr (WPR > 1) {
    if (lane == 0) s_max[wave] = mx;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < WPR; ++i) mx = fmaxf(mx, s_max[i]);
  }
  const float ms = mx == -INFINITY ? 0.f : mx;
  const int width = a.dim <= 64 ? 16 : 32;  // lanes of a group
  const int groups = 64 / width, e4 = lane % width;
  const bool on = 4 * e4 < a.dim;
  const float* src = a.part + row * a.dim + 4 * (on ? e4 : 0);
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
#pragma unroll 4
  for (int s = tw * groups + lane / width; s < splits; s += WPR * groups) {
    const float w = __builtin_amdgcn_exp2f(stat[s * n] - ms);
    const float4 x = *reinterpret_cast<const float4*>(src + s * n * a.dim);
    sum += w;
    v.x += w * x.x;
    v.y += w * x.y;
    v.z += w * x.z;
    v.w += w * x.w;
  }
  for (int o = width; o < 64; o <<= 1) {
    sum += __shfl_xor(sum, o);
    v.x += __shfl_xor(v.x, o);
    v.y += __shfl_xor(v.y, o);
    v.z += __shfl_xor(v.z, o);
    v.w += __shfl_xor(v.w, o);
  }
  if constexpr (WPR > 1) {
    if (lane < 32) s_out[wave][lane] = v;
    if (lane == 0) s_sum[wave] = sum;
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int i = 1; i < WPR; ++i) {
      const float4 x = s_out[i][lane & 31];
      sum += s_sum[i];
      v.x += x.x;
      v.y += x.y;
      v.z += x.z;
      v.w += x.w;
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int head = int(row / a.nq);
  const int64_t tok = row - int64_t(head) * a.nq;
  if (on && lane < width) {
    typedef E out4 __attribute__((ext_vector_type(4)));
    E* op = static_cast<E*>(const_cast<void*>(a.o.p)) + tok * a.o.ts + head * a.o.hs + 4 * e4;
    *reinterpret_cast<out4*>(op) = out4{static_cast<E>(v.x * inv), static_cast<E>(v.y * inv),
                                        static_cast<E>(v.z * inv), static_cast<E>(v.w * inv)};
  }
  if (a.lse != nullptr && lane == 0)
    a.lse[row] = sum == 0.f ? -INFINITY : (ms + __builtin_amdgcn_logf(sum)) * 0.6931471805599453f;
}

template <class E, int NB, bool TOKEN>
hipError_t launch_shape(const AttnArgs& a, const AttnPlan& plan, hipStream_t st) {
  typedef FwdShape<E, NB, TOKEN> F;
  const int64_t tiles = tiles_of(a.nq, a.batch, a.hq / a.hk, F::kRows);
  const int64_t wgs = tiles * a.hk * plan.splits;
  if (wgs >= (int64_t(1) << 31)) return hipErrorInvalidValue;
  attn_fwd<E, NB, TOKEN><<<unsigned(wgs), 256, 0, st>>>(a, int(tiles), plan.splits);
  return hipGetLastError();
}

template <class E>
hipError_t launch_type(const AttnArgs& a, const AttnPlan& plan, hipStream_t st) {
  const int nb = (a.dim + 31) / 32;
  hipError_t e;
  if (plan.token_form)
    e = nb == 1   ? launch_shape<E, 1, true>(a, plan, st)
        : nb == 2 ? launch_shape<E, 2, true>(a, plan, st)
        : nb == 3 ? launch_shape<E, 3, true>(a, plan, st)
                  : launch_shape<E, 4, true>(a, plan, st);
  else
    e = nb == 1   ? launch_shape<E, 1, false>(a, plan, st)
        : nb == 2 ? launch_shape<E, 2, false>(a, plan, st)
        : nb == 3 ? launch_shape<E, 3, false>(a, plan, st)
                  : launch_shape<E, 4, false>(a, plan, st);
  if (e != hipSuccess || plan.splits == 1) return e;
  const int64_t rows = int64_t(a.hq) * a.nq;
  // many splits of few rows (one cache: 128 of 16 rows): four waves a row, the call 31 us for 33; few splits of many
  // rows (the fp32 size: 4 of 17 k): one, 57 us for 68
  if (plan.splits > 8)
    attn_join<E, 4><<<unsigned(rows), 256, 0, st>>>(a, plan.splits);
  else
    attn_join<E, 1><<<unsigned((rows + 3) / 4), 256, 0, st>>>(a, plan.splits);
  return hipGetLastError();
}

}  // namespace

AttnPlan plan_attention(const AttnArgs& a) {
  AttnPlan p{};
  const int group = a.hq / a.hk;
  p.splits = 1;
  // up to 32 rows a sequence on average: the token form
  p.token_form = int64_t(a.nq) * group <= int64_t(32) * a.batch;
  const int64_t tiles = tiles_of(a.nq, a.batch, group, p.token_form ? 32 : 128) * a.hk;
  const int keys = p.token_form || a.dtype == TR_SC_F32 ? 32 : 64;
  // keys that one row tile can see at most
  const int64_t reach = int64_t(a.left) + a.right + 1 + a.sinks + (p.token_form ? 32 : 128) / group;
  const int64_t span = reach < a.nk ? reach : a.nk;
  const int64_t per = p.token_form ? 4 : 1;  // tiles that a workgroup takes at once
  const int64_t key_rounds = (span + keys * per - 1) / (keys * per);
  // workgroups that the chip holds at once (by LDS: one a CU in the token form of wide heads, else two). Twice that
  // in the token form: 62 us for 60 and 43 for 37; half or more than that of the others was no faster.
  const int64_t want = p.token_form && (a.dim > 64 || a.dtype == TR_SC_F32) ? 256 : 512;
  int64_t s = (want + tiles - 1) / tiles;
  // Rounds that a split has at least. The join and its launch are worth 5 us: eight rounds (512 keys) of the half
  // types (450 tokens, 8 heads of 64, 64 keys either way: 17.4 us in two splits, 13.5 in one; all 450 keys: 17.3 and
  // 13.3), two of fp32 (700 tokens, 6 heads of 80: 21 us for 36) or of a workgroup whose waves take four tiles.
  const int64_t least = p.token_form || a.dtype == TR_SC_F32 ? 2 : 8;
  if (s > key_rounds / least) s = key_rounds / least;
  if (s > 256) s = 256;
  if (s > 1) p.splits = int(s);
  if (p.splits > 1) p.part_floats = size_t(p.splits) * a.hq * a.nq * (a.dim + 1);
  return p;
}

hipError_t launch_attention(const AttnArgs& a, const AttnPlan& plan, hipStream_t st) {
  if (a.nq == 0) return hipSuccess;
  if (a.dtype == TR_SC_BF16) return launch_type<__bf16>(a, plan, st);
  if (a.dtype == TR_SC_F16) return launch_type<_Float16>(a, plan, st);
  return launch_type<float>(a, plan, st);
}

}  // namespace trsc
