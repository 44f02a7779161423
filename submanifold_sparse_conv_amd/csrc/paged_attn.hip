// Windowed attention over a paged cache, with or without a prefix that the
// batch's sequences share.
//
// Mathematics. As in attn_fwd.hip; key j of a sequence is slot j % page of page
// table[j / page]. Behind a prefix of P keys the softmax goes over both: the
// prefix and a sequence's own keys are walked by different workgroups, each
// with the statistics of its part, and joined,
// o = sum_s 2^{l_s - l} o_s, l = log2 sum_s 2^{l_s}.
//
// Rows. A sequence's own keys: row r is its token r / G, head r % G of the
// group, tiles of 128 rows (32 a wave) or, for few rows, 32 that the four waves
// share. The prefix: the rows of all sequences are one matrix, so its keys are
// read once for 128 rows, whatever sequence they belong to; each row has its own
// position. A query that is i-th of Lq stands at i + P + Lk - Lq.
//
// Pages. A copy to LDS of a wave takes 2 to 8 rows, which lie in one page: a
// page holds a multiple of 8. The pages of a tile's rows are read a tile ahead,
// one a lane, and taken from there as scalars.
#include "attn_rows.h"
#include "paged.h"

namespace trsc {
namespace {

// A run of keys: a sequence's own, or the prefix.
struct Keys {
  const int32_t* table;
  int n;      // keys
  int sinks;  // of them
};

template <class E, int NB, int ROWS, int STEP>
struct PagedCopy {
  typedef Tile<E, NB> T;
  static constexpr int kRows = T::kRowsPerCopy, kCopies = ROWS / kRows, kN = (kCopies + STEP - 1) / STEP;
  uint32_t off[kN], row_bytes;
  int first;
  __device__ __forceinline__ void start(int64_t stride, int dim, int first_, int lane) {
    first = first_;
    row_bytes = uint32_t(dim * T::kElt);
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const int row = lane / T::kChunks;  // of the copy
      const int chunk = (lane % T::kChunks) ^ T::key((first + j * STEP) * kRows + row);
      off[j] = chunk * T::kPer < dim ? uint32_t(row) * uint32_t(stride * T::kElt) + chunk * 16 : 0x80000000u;
    }
  }
  // base: the head's first element in the pool; ids: page of row l of the tile in lane l, -1 for none; slot: the
  // first row's slot in its page; left: rows from the tile's first to the last key's. Rows without a page and past
  // the end read as zero.
  __device__ __forceinline__ void run(unsigned char* lds, const E* base, int64_t ps, int64_t ss, int ids, int page_mask,
                                      int t0, int left) const {
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const int copy = first + j * STEP;
      if (!((j + 1) * STEP <= kCopies || copy < kCopies)) continue;
      const int row = copy * kRows;
      const int page = __builtin_amdgcn_readlane(ids, row);
      const int n = left - row > kRows ? kRows : left - row;
      const uint32_t bytes = page < 0 || n <= 0 ? 0u : uint32_t(n - 1) * uint32_t(ss * T::kElt) + row_bytes;
      const E* from = base + (page < 0 ? 0 : page) * ps + ((t0 + row) & page_mask) * ss;
      copy_lds16(buffer_of(from, bytes), off[j], lds + copy * 1024);
    }
  }
};

// The page of key j, -1 where there is none.
__device__ __forceinline__ int page_of(const PagedArgs& a, const Keys& keys, int j) {
  if (j >= keys.n) return -1;
  const int page = keys.table[j >> a.pool.log2];
  return page >= 0 && page < a.pool.pages ? page : -1;
}

// The sequence of token t: the last that starts at or before it. One load per lane and level.
__device__ __forceinline__ int sequence_of(const Packed& s, int t) {
  const int lane = threadIdx.x & 63;
  int lo = 0, n = s.batch;
  while (n > 1) {
    const int step = (n + 63) / 64;
    const int c = __popcll(__ballot(lane * step < n && s.cu[lo + lane * step] <= t));
    const int at = (c > 0 ? c - 1 : 0) * step;
    lo += at;
    n = n - at < step ? n - at : step;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

struct OwnSeq {
  int q0, lq, lk;
};
__device__ __forceinline__ OwnSeq paged_sequence(const PagedArgs& a, int b) {
  OwnSeq s;
  if (a.seqs.cu != nullptr) {
    s.q0 = clamp_to(a.seqs.cu[b], 0, a.nq);
    s.lq = clamp_to(a.seqs.cu[b + 1], s.q0, a.nq) - s.q0;
  } else {
    s.q0 = b * a.seqs.each;
    s.lq = a.seqs.each;
  }
  s.lk = clamp_to(a.pool.len[b], 0, a.pool.table_pages << a.pool.log2);
  return s;
}

// The rows of a wave, lanes l and l + 32 row l. Positions are those of the run of keys.
struct Rows {
  bool any, on;
  int tok, head;
  int lo, hi;  // keys that the lane's row sees: [lo, hi], and the sinks up to hi
  int p0, p1;  // least and largest position of the wave's rows
};
__device__ __forceinline__ void see(const PagedArgs& a, const Keys& keys, int p, Rows& r) {
  r.lo = p - a.left;
  r.hi = min(p + a.right, keys.n - 1);
}
// Rows first .. first + 31 of a sequence against its own keys.
__device__ __forceinline__ Rows own_rows(const PagedArgs& a, const OwnSeq& s, const Keys& keys, int first, int kvh, int l32) {
  const int group = a.hq / a.hk, rows = s.lq * group, row = first + l32, shift = s.lk - s.lq;
  Rows r;
  r.any = first < rows;
  r.on = row < rows;
  const int i = (r.on ? row : rows - 1) / group;
  r.tok = s.q0 + i;
  r.head = kvh * group + (r.on ? row - i * group : 0);
  see(a, keys, i + shift, r);
  r.p0 = min(first, rows - 1) / group + shift;
  r.p1 = min(first + 31, rows - 1) / group + shift;
  return r;
}
// Rows first .. first + 31 of all sequences against the prefix.
__device__ __forceinline__ Rows prefix_rows(const PagedArgs& a, const Keys& keys, int first, int kvh, int l32) {
  const int group = a.hq / a.hk, rows = a.nq * group, row = first + l32;
  Rows r;
  r.tok = min(row, rows - 1) / group;
  r.head = kvh * group + (row < rows ? row - r.tok * group : 0);
  int p = 0;
  r.on = row < rows;
  if (a.seqs.cu == nullptr) {
    const OwnSeq s = paged_sequence(a, r.tok / a.seqs.each);
    p = r.tok - s.q0 + s.lk - s.lq;
  } else {
    // tokens of the wave's rows in order, a sequence at a time
    int b = sequence_of(a.seqs, __builtin_amdgcn_readfirstlane(r.tok));
    bool found = false;
    for (; b < a.seqs.batch; ++b) {
      const OwnSeq s = paged_sequence(a, b);
      if (!found && r.tok >= s.q0 && r.tok < s.q0 + s.lq) {
        found = true;
        p = r.tok - s.q0 + s.lk - s.lq;
      }
      if (!__any(r.on && !found && r.tok >= s.q0 + s.lq)) break;
    }
    r.on = r.on && found;
  }
  p += a.prefix_len;
  see(a, keys, p, r);
  int p0 = r.on ? p : 0x7fffffff, p1 = r.on ? p : -0x7fffffff;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    p0 = min(p0, __shfl_xor(p0, o));
    p1 = max(p1, __shfl_xor(p1, o));
  }
  r.p0 = __builtin_amdgcn_readfirstlane(p0);
  r.p1 = __builtin_amdgcn_readfirstlane(p1);
  r.any = r.p0 <= r.p1;
  return r;
}
__device__ __forceinline__ bool tile_seen(const PagedArgs& a, const Keys& keys, const Rows& r, int j0, int j1) {
  return r.any && j0 <= r.p1 + a.right && (j1 >= r.p0 - a.left || j0 < keys.sinks);
}
__device__ __forceinline__ bool tile_whole(const PagedArgs& a, const Keys& keys, const Rows& r, int j0, int j1) {
  return j1 <= r.p0 + a.right && j1 < keys.n && (j0 >= r.p1 - a.left || j1 < keys.sinks);
}

// A lane's row: blocks first .. first + count of 32 columns, and the statistic if `with_sum`, to the output or, of a
// part of the keys, to slot `slot` of `parts`.
template <class E, int NB>
__device__ __forceinline__ void store_row(const PagedArgs& a, int parts, int slot, const Rows& r, const f32x16 (&acc)[NB],
                                          float mc, float l, int first, int count, bool with_sum, int h) {
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const float lg = l == 0.f ? -INFINITY : mc + __builtin_amdgcn_logf(l);  // base 2
  const int64_t n = int64_t(a.hq) * a.nq, at_row = slot * n + int64_t(r.head) * a.nq + r.tok;
  typedef E out4 __attribute__((ext_vector_type(4)));
  E* const op = static_cast<E*>(const_cast<void*>(a.o.p)) + r.tok * a.o.ts + r.head * a.o.hs;
  float* const pp = a.part + at_row * a.dim;
#pragma unroll
  for (int d = 0; d < NB; ++d) {
    if (d >= count) break;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int col = 32 * (first + d) + 8 * g + 4 * h;
      if (col >= a.dim) continue;
      if (parts == 1) {
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
  if (parts > 1)
    a.part[parts * n * a.dim + at_row] = lg;
  else if (a.lse != nullptr)
    a.lse[int64_t(r.head) * a.nq + r.tok] = lg * 0.6931471805599453f;
}

// A wave's rows again over the key tiles [first, end), adding only what each sees (attn_common.h): blocks d0 ..
// d0 + DN of O^T, the scaled maximum and the sum. lds: 4 KB of the wave's own.
template <class E, int NB, int KT, int DN>
__device__ void safe_rows(const PagedArgs& a, const Keys& keys, const KeyTiles& kt, int first, int end, const Rows& r,
                          int kvh, int d0, float* lds, int lane, f32x16 (&acc)[NB], float& mc, float& l) {
  constexpr int ST = NB * 2;
  const E* qp = static_cast<const E*>(a.q.p) + r.tok * a.q.ts + r.head * a.q.hs;
  const E* kbase = static_cast<const E*>(a.pool.k) + kvh * a.pool.khs;
  const E* vbase = static_cast<const E*>(a.pool.v) + kvh * a.pool.vhs;
  const int mask = (1 << a.pool.log2) - 1;
  const float c = a.scale * kLog2e;
  typename AttnType<E>::frag qf[ST];
#pragma unroll
  for (int st = 0; st < ST; ++st) qf[st] = row_from<E>(qp, r.on, st, a.dim, lane);
#pragma unroll
  for (int d = 0; d < DN; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[d][e] = 0.f;
  float m = -INFINITY;
  l = 0.f;
  for (int it = first * (KT / 32); it < end * (KT / 32); ++it) {
    const int j0 = kt.at(it / (KT / 32)) * KT + it % (KT / 32) * 32;
    if (!tile_seen(a, keys, r, j0, j0 + 31)) continue;
    const int mine = j0 + (lane & 31), page = page_of(a, keys, mine);
    f32x16 s = scores_from<E, ST>(kbase + max(page, 0) * a.pool.kps + (mine & mask) * a.pool.kss, page >= 0, qf, a.dim,
                                  lane);
    hide(s, j0, r.lo, r.hi, keys.sinks, lane);
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
    // a key without a page has the value zero: nothing to add
    add_rows<E, DN>(
        acc, lds,
        [&](int i) {
          const int j = min(j0 + i, keys.n - 1);
          return vbase + max(__builtin_amdgcn_readlane(page, j - j0), 0) * a.pool.vps + (j & mask) * a.pool.vss;
        },
        [&](int i) {
          return __builtin_amdgcn_readlane(page, i) >= 0 && j0 + i <= r.hi && (j0 + i >= r.lo || j0 + i < keys.sinks);
        },
        d0, a.dim, lane);
    wave_fence();
  }
  mc = m * c;
  const float2 lh = both_halves(l);
  l = lh.x + lh.y;
}

template <class E, int NB, bool TOKEN>
struct PagedShape {  // as the contiguous kernels' (attn_fwd.hip)
  typedef Tile<E, NB> T;
  static constexpr int kKeys = TOKEN || sizeof(E) == 4 ? 32 : 64;
  static constexpr int kTileBytes = kKeys * T::kPitch;
  static constexpr int kBuffers = (TOKEN && sizeof(E) == 4 && NB > 2) ? 1 : 2;
  static constexpr int kWaveSets = TOKEN ? 4 : 1;
  static constexpr int kLds = kBuffers * 2 * kTileBytes * kWaveSets;
  static constexpr int kRows = TOKEN ? 32 : 128;
};

// Workgroups of one run of keys: tiles row tiles by kv heads by splits; slot0, parts: the first split's slot, and
// slots in all.
template <class E, int NB, bool TOKEN, bool PREFIX>
__global__ __launch_bounds__(256, TOKEN || sizeof(E) == 4 ? 1 : NB <= 2 ? 4 : 2) void paged_attn(PagedArgs a, int tiles,
                                                                                                int splits, int slot0,
                                                                                                int parts) {
  typedef PagedShape<E, NB, TOKEN> F;
  typedef Tile<E, NB> T;
  constexpr int KB = NB <= 2 ? 1 : F::kKeys / 32;
  __shared__ __attribute__((aligned(1024))) unsigned char s_mem[F::kLds];
  const int lane = threadIdx.x & 63, l32 = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = a.hq / a.hk;
  const int w = xcd_remap(blockIdx.x, gridDim.x);
  const int tile = w % tiles, kvh = (w / tiles) % a.hk, split = w / tiles / a.hk;
  Keys keys;
  Rows r;
  KeyTiles kt;
  if constexpr (PREFIX) {
    keys = Keys{a.prefix, a.prefix_len, min(a.sinks, a.prefix_len)};
    r = prefix_rows(a, keys, tile * F::kRows + (TOKEN ? 0 : 32 * wave), kvh, l32);
    int p0 = r.p0, p1 = r.p1;
    if constexpr (!TOKEN) {  // of the workgroup's rows
      int* const red = reinterpret_cast<int*>(s_mem);
      if (lane == 0) red[wave] = p0, red[4 + wave] = p1;
      __syncthreads();
      p0 = min(min(red[0], red[1]), min(red[2], red[3]));
      p1 = max(max(red[4], red[5]), max(red[6], red[7]));
      __syncthreads();
    }
    if (p0 > p1) return;
    kt = key_tiles<F::kKeys>(a.left, a.right, keys.sinks, p0, p1, keys.n);
  } else {
    int inside, b;
    if (a.seqs.cu == nullptr) {
      const int per = (a.seqs.each * group + F::kRows - 1) / F::kRows;
      b = tile / per;
      inside = tile - b * per;
    } else {
      b = find_sequence(a.seqs.cu, a.seqs.batch, group, F::kRows, tile, &inside);
    }
    const OwnSeq s = paged_sequence(a, b);
    const int rows = s.lq * group;
    if (inside < 0 || inside > rows / F::kRows || inside * F::kRows >= rows) return;
    const int r0 = inside * F::kRows, last = min(rows - 1, r0 + F::kRows - 1) / group, shift = s.lk - s.lq;
    keys = Keys{a.pool.table + b * a.pool.table_ts, s.lk, max(0, a.sinks - a.prefix_len)};
    kt = key_tiles<F::kKeys>(a.left, a.right, keys.sinks, r0 / group + shift, last + shift, s.lk);
    r = own_rows(a, s, keys, r0 + (TOKEN ? 0 : 32 * wave), kvh, l32);
  }
  const typename T::Lane at = T::lane_of(lane);
  RowState<E, NB, KB> st;
  st.start(static_cast<const E*>(a.q.p) + r.tok * a.q.ts + r.head * a.q.hs, r.on, a.dim, lane);
  const E* kbase = static_cast<const E*>(a.pool.k) + kvh * a.pool.khs;
  const E* vbase = static_cast<const E*>(a.pool.v) + kvh * a.pool.vhs;
  const float c = a.scale * kLog2e;
  const int mask = (1 << a.pool.log2) - 1;

  const int first = int(int64_t(kt.n) * split / splits), end = int(int64_t(kt.n) * (split + 1) / splits);
  unsigned char* const mem = s_mem + (TOKEN ? wave * F::kBuffers * 2 * F::kTileBytes : 0);
  PagedCopy<E, NB, F::kKeys, TOKEN ? 1 : 4> kc, vc;
  kc.start(a.pool.kss, a.dim, TOKEN ? 0 : wave, lane);
  vc.start(a.pool.vss, a.dim, TOKEN ? 0 : wave, lane);
  auto pages = [&](int it) { return it < end && lane < F::kKeys ? page_of(a, keys, kt.at(it) * F::kKeys + lane) : -1; };
  auto fetch = [&](int it, int buf, int ids) {
    const int t0 = kt.at(it) * F::kKeys;
    unsigned char* dst = mem + buf * 2 * F::kTileBytes;
    kc.run(dst, kbase, a.pool.kps, a.pool.kss, ids, mask, t0, keys.n - t0);
    vc.run(dst + F::kTileBytes, vbase, a.pool.vps, a.pool.vss, ids, mask, t0, keys.n - t0);
  };
  auto compute = [&](int it, int buf) {
    const unsigned char* ks = mem + buf * 2 * F::kTileBytes;
#pragma unroll
    for (int part = 0; part < F::kKeys / (32 * KB); ++part) {
      const int j0 = kt.at(it) * F::kKeys + part * 32 * KB, j1 = j0 + 32 * KB - 1;
      if (!tile_seen(a, keys, r, j0, j1)) continue;
      st.scores(ks + part * 32 * KB * T::kPitch, (a.dim + 15) / 16, at);
      if (!tile_whole(a, keys, r, j0, j1)) {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) hide(st.s[kb], j0 + 32 * kb, r.lo, r.hi, keys.sinks, lane);
      }
      st.weigh(c);
      st.multiply(ks + F::kTileBytes + part * 32 * KB * T::kPitch, at);
    }
  };

  if constexpr (!TOKEN) {
    if (first < end) fetch(first, 0, pages(first));
    int ids = pages(first + 1);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    for (int it = first; it < end; it += 2) {  // two tiles a round: the buffers' addresses are constants
#pragma unroll
      for (int buf = 0; buf < 2; ++buf) {
        if (it + buf >= end) break;
        if (it + buf + 1 < end) {
          fetch(it + buf + 1, buf ^ 1, ids);
          ids = pages(it + buf + 2);
        }
        compute(it + buf, buf);
        __builtin_amdgcn_s_waitcnt(0);
        bare_barrier();
      }
    }
  } else {
    // each wave its own tiles and LDS: no barrier in the loop
    constexpr int NBUF = F::kBuffers;
    int it = first + wave, buf = 0, ids = pages(it);
    if (NBUF == 2 && it < end) {
      fetch(it, 0, ids);
      ids = pages(it + 4);
    }
    for (; it < end; it += 4) {
      if constexpr (NBUF == 2) {
        __builtin_amdgcn_s_waitcnt(0);
        asm volatile("" ::: "memory");
        if (it + 4 < end) {
          fetch(it + 4, buf ^ 1, ids);
          ids = pages(it + 8);
        }
        compute(it, buf);
        buf ^= 1;
      } else {
        __builtin_amdgcn_s_waitcnt(0);  // the last tile's reads are done
        fetch(it, 0, ids);
        ids = pages(it + 4);
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
  float zero = 0.f;
  if (writer && r.on) {
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
    if (r.on && writer && which)
      store_row<E, NB>(a, parts, slot0 + split, r, st.acc, mc, l, TOKEN ? wave : 0, TOKEN ? 1 : NB,
                       h == 0 && (!TOKEN || wave == 0), h);
  };
  const bool mine = (bad >> l32) & 1u;
  store(!mine);
  if (bad != 0) {
    if constexpr (TOKEN) __syncthreads();  // the flags are read
    if (!writer) return;
    safe_rows<E, NB, F::kKeys, TOKEN ? 1 : NB>(a, keys, kt, first, end, r, kvh, TOKEN ? wave : 0,
                                               reinterpret_cast<float*>(s_mem) + wave * 1024, lane, st.acc, mc, l);
    store(mine);
  }
}

// Joins the parts of a row: WPR waves a (token, head); a lane has four
// elements, and the parts are dealt to the lanes' groups in turn, whose sums are
// added in a fixed order. Rows of no sequence are left.
template <class E, int WPR>
__global__ __launch_bounds__(256) void paged_join(PagedArgs a, int parts) {
  constexpr int kRows = 4 / WPR;
  __shared__ float s_max[4], s_sum[4];
  __shared__ float4 s_out[4][32];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, tw = wave % WPR;
  const int64_t n = int64_t(a.hq) * a.nq;
  const int64_t row = int64_t(blockIdx.x) * kRows + wave / WPR;  // head * nq + token
  if (row >= n) return;                                          // the whole team
  const int head = int(row / a.nq), tok = int(row - int64_t(head) * a.nq);
  if (a.seqs.cu != nullptr && (tok < a.seqs.cu[0] || tok >= a.seqs.cu[a.seqs.batch])) return;
  const float* stat = a.part + parts * n * a.dim + row;
  float mx = -INFINITY;
  for (int s = tw * 64 + lane; s < parts; s += WPR * 64) mx = fmaxf(mx, stat[s * n]);
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
  for (int s = tw * groups + lane / width; s < parts; s += WPR * groups) {
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
  if (on && lane < width) {
    typedef E out4 __attribute__((ext_vector_type(4)));
    E* op = static_cast<E*>(const_cast<void*>(a.o.p)) + tok * a.o.ts + head * a.o.hs + 4 * e4;
    *reinterpret_cast<out4*>(op) = out4{static_cast<E>(v.x * inv), static_cast<E>(v.y * inv),
                                        static_cast<E>(v.z * inv), static_cast<E>(v.w * inv)};
  }
  if (a.lse != nullptr && lane == 0)
    a.lse[row] = sum == 0.f ? -INFINITY : (ms + __builtin_amdgcn_logf(sum)) * 0.6931471805599453f;
}

int64_t own_tiles(const PagedArgs& a, int rows) {
  const int group = a.hq / a.hk;
  if (a.seqs.cu == nullptr) return int64_t(a.seqs.batch) * ((int64_t(a.seqs.each) * group + rows - 1) / rows);
  return tiles_of(a.nq, a.seqs.batch, group, rows);
}
int64_t prefix_tiles(const PagedArgs& a, int rows) { return (int64_t(a.nq) * (a.hq / a.hk) + rows - 1) / rows; }

template <class E, int NB, bool TOKEN, bool PREFIX>
hipError_t launch_run(const PagedArgs& a, int splits, int slot0, int parts, hipStream_t st) {
  constexpr int kRows = PagedShape<E, NB, TOKEN>::kRows;
  const int64_t tiles = PREFIX ? prefix_tiles(a, kRows) : own_tiles(a, kRows);
  const int64_t wgs = tiles * a.hk * splits;
  if (wgs >= (int64_t(1) << 31)) return hipErrorInvalidValue;
  paged_attn<E, NB, TOKEN, PREFIX><<<unsigned(wgs), 256, 0, st>>>(a, int(tiles), splits, slot0, parts);
  return hipGetLastError();
}

template <class E, int NB>
hipError_t launch_shape(const PagedArgs& a, const PagedPlan& p, hipStream_t st) {
  const int parts = p.prefix_splits + p.splits;
  hipError_t e = hipSuccess;
  if (p.prefix_splits > 0)
    e = p.prefix_token_form ? launch_run<E, NB, true, true>(a, p.prefix_splits, 0, parts, st)
                            : launch_run<E, NB, false, true>(a, p.prefix_splits, 0, parts, st);
  if (e != hipSuccess) return e;
  return p.token_form ? launch_run<E, NB, true, false>(a, p.splits, p.prefix_splits, parts, st)
                      : launch_run<E, NB, false, false>(a, p.splits, p.prefix_splits, parts, st);
}

template <class E>
hipError_t launch_type(const PagedArgs& a, const PagedPlan& p, hipStream_t st) {
  const int nb = (a.dim + 31) / 32;
  const hipError_t e = nb == 1   ? launch_shape<E, 1>(a, p, st)
                       : nb == 2 ? launch_shape<E, 2>(a, p, st)
                       : nb == 3 ? launch_shape<E, 3>(a, p, st)
                                 : launch_shape<E, 4>(a, p, st);
  const int parts = p.prefix_splits + p.splits;
  if (e != hipSuccess || parts == 1) return e;
  const int64_t rows = int64_t(a.hq) * a.nq;
  if (parts > 8)
    paged_join<E, 4><<<unsigned(rows), 256, 0, st>>>(a, parts);
  else
    paged_join<E, 1><<<unsigned((rows + 3) / 4), 256, 0, st>>>(a, parts);
  return hipGetLastError();
}

// Splits of a walk over `span` keys by `tiles` row tiles.
int splits_for(const PagedArgs& a, int64_t tiles, int64_t span, bool token) {
  const int keys = token || a.dtype == TR_SC_F32 ? 32 : 64;
  const int64_t rounds = (span + keys * (token ? 4 : 1) - 1) / (keys * (token ? 4 : 1));
  const int64_t want = token && (a.dim > 64 || a.dtype == TR_SC_F32) ? 256 : 512;
  const int64_t least = token || a.dtype == TR_SC_F32 ? 2 : 8;
  int64_t s = (want + tiles - 1) / tiles;
  if (s > rounds / least) s = rounds / least;
  return s > 256 ? 256 : s < 1 ? 1 : int(s);
}

}  // namespace

PagedPlan plan_paged_attention(const PagedArgs& a) {
  PagedPlan p{};
  p.splits = 1;
  if (a.nq == 0) return p;
  const int group = a.hq / a.hk;
  p.token_form = int64_t(a.nq) * group <= int64_t(32) * a.seqs.batch;
  const int64_t reach = int64_t(a.left) + a.right + 1 + a.sinks + (p.token_form ? 32 : 128) / group;
  const int64_t room = int64_t(a.pool.table_pages) << a.pool.log2;
  p.splits = splits_for(a, own_tiles(a, p.token_form ? 32 : 128) * a.hk, reach < room ? reach : room, p.token_form);
  if (a.prefix_len > 0) {
    p.prefix_token_form = int64_t(a.nq) * group <= 32;
    const int64_t tiles = prefix_tiles(a, p.prefix_token_form ? 32 : 128) * a.hk;
    p.prefix_splits = splits_for(a, tiles, a.prefix_len, p.prefix_token_form);
  }
  const int parts = p.splits + p.prefix_splits;
  if (parts > 1) p.part_floats = size_t(parts) * a.hq * a.nq * (a.dim + 1);
  return p;
}

hipError_t launch_paged_attention(const PagedArgs& a, const PagedPlan& p, hipStream_t st) {
  if (a.nq == 0) return hipSuccess;
  if (a.dtype == TR_SC_BF16) return launch_type<__bf16>(a, p, st);
  if (a.dtype == TR_SC_F16) return launch_type<_Float16>(a, p, st);
  return launch_type<float>(a, p, st);
}

}  // namespace trsc
