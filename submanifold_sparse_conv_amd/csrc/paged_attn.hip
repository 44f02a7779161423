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
// group, in tiles of 32 (few rows: one wave holds them) or 128 rows (four waves
// that share the key tiles). The prefix: the rows of all sequences are one
// matrix, so its keys are read once for a tile, whatever sequence its rows
// belong to (small calls: for each sequence's tile); each row has its own
// position. A query that is i-th of Lq stands at i + P + Lk - Lq.
//
// Work. An item is a row tile with all key tiles that it sees; a unit is one of
// those. The units of all items in a row are dealt out evenly, each wave (32
// rows) or workgroup (128) taking one contiguous run of them for one kv head:
// lengths differ and only the device knows them, so every wave sums them up and
// finds its run. A lane sums batch / 64 sequences, tile of rows by tile of rows, and
// where an item begins its sequence is searched from its lane's first one: short
// for a few hundred sequences or tiles; 4096 sequences of 50 keys take 597 us where
// 256 of 800 take 83 (4 kv heads of 128), one prompt of 16,384 tokens, 8 heads over
// 1 of 128, 1023 keys back, 567 us for a floor of 53, and behind a prefix, where
// there is no form without runs, 65,536 tokens of 8 heads over 1 of 64 2.8 ms for
// 128 us without one. An item that two runs share leaves
// parts in the workspace that the join adds up in order. The heads' runs are cut
// at the same places and lie in neighbouring waves, which so read neighbouring
// memory at the same time.
//
// Pages. A copy to LDS of a wave takes 2 to 8 rows, which lie in one page: a
// page holds a multiple of 8. The pages of a tile's rows are read a tile ahead,
// one a lane, and taken from there as scalars.
//
// Rounding. As in attn_fwd.hip: fp32 but for the weights, rounded to the tensors'
// type before they multiply V. Parts and their statistics are fp32.
//
// What bounds it. Single tokens: HBM reads. 32 caches of 1 to 4100 keys in a
// window, 4 kv heads of 128, bf16, pages of 16: 257 MB in 61 us, 4.2 TB/s; the
// kernel's 56 are 15 tiles a wave at 5.9 TB/s and 13 to 15 us before the first and
// after the last (lengths, table, tile: three dependent reads of memory, and code
// read for the first time), the join 5. One cache of 99,000 keys, fp16: 204 MB in
// 54 us, 45 and 9. Parts of prompts (1401 rows, 4 heads of 128 over up to 8192 keys,
// 16 query heads): 76.7 GFLOP in 110 us, 100 and the join of 45 MB of parts, matrix
// units busy in a third of the cycles: 36 units a workgroup, two workgroups a CU,
// which start and end a run 1.4 times on average. 256 sequences behind 8192 common
// keys: 77 to 79 us, where the prefix's half of the chip has one workgroup a CU, since a
// wave's own tiles take 128 KB of LDS. Small calls: latency; 8 caches of up to 450
// keys 7.8 us, 4 sequences behind 1369 keys 16.
#include <type_traits>

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

// A value that all lanes hold alike, in a scalar register. What comes from a division, a load or a 64-bit comparison is
// in vector registers otherwise, and with it all that is computed from it, down to the copies' descriptors, which then
// cost a loop over the lanes each.
__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Copies rows [0, ROWS) of a tile of keys from their pages to LDS: this wave's copies first, first + STEP, ... of 64
// lanes x 16 bytes. Offsets in the pool are taken in units of 16 bytes, 32 bits a factor.
template <class E, int NB, int ROWS, int STEP>
struct PagedCopy {
  typedef Tile<E, NB> T;
  static constexpr int kRows = T::kRowsPerCopy, kCopies = ROWS / kRows, kN = (kCopies + STEP - 1) / STEP;
  uint32_t off[kN], page16, slot16, full;
  int first;
  __device__ __forceinline__ void start(int64_t page_stride, int64_t stride, int dim, int first_, int lane) {
    first = first_;
    page16 = uni(uint32_t(page_stride / T::kPer));
    slot16 = uni(uint32_t(stride / T::kPer));
    full = uint32_t(kRows - 1) * slot16 * 16 + uint32_t(dim * T::kElt);
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const int row = lane / T::kChunks;  // of the copy
      const int chunk = (lane % T::kChunks) ^ T::key((first + j * STEP) * kRows + row);
      off[j] = chunk * T::kPer < dim ? uint32_t(row) * slot16 * 16 + chunk * 16 : 0x80000000u;
    }
  }
  // base: the head's first element in the pool; ids: page of row l of the tile in lane l, -1 for none; t0: the tile's
  // first key, left: keys from there on. Rows without a page read as zero; ZEROS: rows past the end too, in a page that
  // goes on behind them. (What lies there would spoil a product with a weight of zero; a score is hidden as it is.)
  template <bool ZEROS>
  __device__ __forceinline__ void run(unsigned char* lds, const E* base, int ids, int page_mask, int t0, int left) const {
    const uint64_t at = reinterpret_cast<uint64_t>(base);
    const uint64_t from = (uint64_t(uint32_t(uni(int(at >> 32)))) << 32) | uint32_t(uni(int(at)));
    page_mask = uni(page_mask);
    t0 = uni(t0);
    left = uni(left);
    uint64_t p = 0;
    uint32_t most = 0;
    const uint32_t step = uint32_t(STEP * kRows * 16) * slot16;
    if (page_mask >= ROWS - 1 && left >= ROWS) {  // one page, no end in it: tiles begin at multiples of ROWS
      const int page = __builtin_amdgcn_readlane(ids, 0);
      most = page < 0 ? 0u : full;
      p = from + ((uint64_t(uint32_t(page < 0 ? 0 : page)) * page16 + uint32_t((t0 & page_mask) + first * kRows) * slot16) << 4);
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        const int copy = first + j * STEP;
        if (!((j + 1) * STEP <= kCopies || copy < kCopies)) continue;
        copy_lds16(buffer_of(reinterpret_cast<const void*>(p), most), off[j], lds + copy * 1024);
        p += step;
      }
      return;
    }
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const int copy = first + j * STEP;
      if (!((j + 1) * STEP <= kCopies || copy < kCopies)) continue;
      const int row = copy * kRows, slot = (t0 + row) & page_mask;
      if (j == 0 || slot < STEP * kRows) {  // another page than the copy before
        const int page = __builtin_amdgcn_readlane(ids, row);
        most = page < 0 ? 0u : full;  // a row past the end has no page unless one before it has
        p = from + ((uint64_t(uint32_t(page < 0 ? 0 : page)) * page16 + uint32_t(slot) * slot16) << 4);
      } else {
        p += step;
      }
      uint32_t bytes = most;
      if constexpr (ZEROS) {
        if (left - row < kRows) bytes = left <= row ? 0u : most - uint32_t(kRows - (left - row)) * slot16 * 16;
        if (most == 0) bytes = 0;
      }
      copy_lds16(buffer_of(reinterpret_cast<const void*>(p), bytes), off[j], lds + copy * 1024);
    }
  }
};

// The table's entry for key j, -1 past the last; and whether it is a page of the pool. Apart, since the comparison
// waits for the entry and with it for the copies in flight.
__device__ __forceinline__ int entry_of(const PagedArgs& a, const Keys& keys, int j) {
  int page = -1;
  if (j < keys.n) page = keys.table[j >> a.pool.log2];
  return page;
}
__device__ __forceinline__ int checked(const PagedArgs& a, int page) {
  return uint32_t(page) < uint32_t(a.pool.pages) ? page : -1;
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
  int any, on;  // truth values
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
  r.p0 = uni(min(first, rows - 1) / group + shift);
  r.p1 = uni(min(first + 31, rows - 1) / group + shift);
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
    // a sequence at a time: that of the first row which has none yet (256 single tokens of 4 heads behind 8192 keys, 32
    // sequences a wave: 152 us with offsets, 49 without)
    bool found = false;
    uint64_t open = __ballot(r.on);
    while (open != 0) {
      const int first_open = __ffsll(static_cast<unsigned long long>(open)) - 1;
      const OwnSeq s = paged_sequence(a, sequence_of(a.seqs, __builtin_amdgcn_readlane(r.tok, first_open)));
      if (r.on && !found && r.tok >= s.q0 && r.tok < s.q0 + s.lq) {
        found = true;
        p = r.tok - s.q0 + s.lk - s.lq;
      }
      open &= ~(1ull << first_open) & ~__ballot(found);
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

// Where the parts of a call lie (bytes from the workspace's start).
struct PartMap {
  int64_t head, table, whole[2], slots[2];  // [0]: the sequences' own keys, [1]: the prefix
  int rows[2];                              // rows of a slot
  int64_t slot_count[2];
};
// A run of the work list in the workspace: T units in W runs. [0]: own, [1]: prefix (the same list where one kind of
// worker takes both; own units then follow the prefix's `before`).
struct Lists {
  int32_t units[2], runs[2];
  int32_t pre_n;  // units of an item of the prefix
};
struct Entry {  // of the table: a row tile's first unit and its units
  int32_t first, n;
};

// Where a lane puts its row: `out`, or a part of `rows` rows with the statistics behind the elements.
struct Target {
  float* part;
  int64_t row, rows;
};

// A lane's row: blocks first .. first + count of 32 columns, and the statistic if `with_sum`.
template <class E, int NB>
__device__ __forceinline__ void store_row(const PagedArgs& a, const Target& to, const Rows& r, const f32x16 (&acc)[NB],
                                          float mc, float l, int first, int count, bool with_sum, int h) {
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const float lg = l == 0.f ? -INFINITY : mc + __builtin_amdgcn_logf(l);  // base 2
  typedef E out4 __attribute__((ext_vector_type(4)));
  E* const op = static_cast<E*>(const_cast<void*>(a.o.p)) + r.tok * a.o.ts + r.head * a.o.hs;
  float* const pp = to.part + to.row * a.dim;
#pragma unroll
  for (int d = 0; d < NB; ++d) {
    if (d >= count) break;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int col = 32 * (first + d) + 8 * g + 4 * h;
      if (col >= a.dim) continue;
      if (to.part == nullptr) {
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
  if (to.part != nullptr)
    to.part[to.rows * a.dim + to.row] = lg;
  else if (a.lse != nullptr)
    a.lse[int64_t(r.head) * a.nq + r.tok] = lg * 0.6931471805599453f;
}

// A wave's rows again over the key tiles [first, end), adding only what each sees (attn_common.h): blocks d0 ..
// d0 + DN of O^T, the scaled maximum and the sum, from the start or (MORE) on top of another run of keys. lds: 4 KB of
// the wave's own.
template <class E, int NB, int KT, int DN, bool MORE = false>
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
  float m = -INFINITY;
  if constexpr (!MORE) {
#pragma unroll
    for (int d = 0; d < DN; ++d)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[d][e] = 0.f;
    l = 0.f;
  } else {  // both halves of the wave hold the whole sum
    m = mc / c;
    l *= 0.5f;
  }
  for (int it = first * (KT / 32); it < end * (KT / 32); ++it) {
    const int j0 = kt.at(it / (KT / 32)) * KT + it % (KT / 32) * 32;
    if (!tile_seen(a, keys, r, j0, j0 + 31)) continue;
    const int mine = j0 + (lane & 31), page = checked(a, entry_of(a, keys, mine));
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

// ---------------------------------------------------------------------------
// The work list: first the prefix's items, row tile by row tile, then the
// sequences'.
// ---------------------------------------------------------------------------
struct List {
  int pre_units, units;  // the prefix's; all (below 2^31, checked by the caller)
  int pre_tiles;         // row tiles of the prefix in this list
  KeyTiles pre;          // its key tiles, of all rows together
  // In LDS, for every lane: the units of the sequences before its own, behind the prefix's, and the first of those
  // sequences. (Not in registers, which the loops over the keys need.)
  struct Lane {
    int start;
    OwnSeq s;
  };
  Lane* lanes;
};
// No member smaller than 32 bits: the compiler puts the copied padding into LDS, and finds its place there by a read of
// the dispatch packet in host memory, 8 us of the kernel's time.
struct Item {
  int prefix;     // truth value
  int b, inside;  // sequence; row tile (of the prefix: of all rows)
  OwnSeq s;
  Keys keys;
  KeyTiles kt;
  int n;  // units: an item without keys has one, which writes its zeros
};
__device__ __forceinline__ OwnSeq uniform_sequence(const PagedArgs& a, int b) {
  const OwnSeq s = paged_sequence(a, b);
  return OwnSeq{uni(s.q0), uni(s.lq), uni(s.lk)};
}
// Row tile `inside` of a sequence.
template <int R, int KT>
__device__ __forceinline__ void own_tile(const PagedArgs& a, int b, const OwnSeq& s, int inside, Item& it) {
  const int group = a.hq / a.hk, rows = s.lq * group, r0 = inside * R, shift = s.lk - s.lq;
  it.prefix = false;
  it.b = b;
  it.inside = inside;
  it.s = s;
  it.keys = Keys{a.pool.table + b * a.pool.table_ts, s.lk, max(0, a.sinks - a.prefix_len)};
  it.kt = key_tiles<KT>(a.left, a.right, it.keys.sinks, r0 / group + shift, min(rows - 1, r0 + R - 1) / group + shift,
                        s.lk);
  it.n = max(it.kt.n, 1);
}
template <int R>
__device__ __forceinline__ int row_tiles(const PagedArgs& a, const OwnSeq& s) {
  return (s.lq * (a.hq / a.hk) + R - 1) / R;
}
template <int R>  // number of a sequence's first row tile in the table (find_sequence)
__device__ __forceinline__ int first_entry(const PagedArgs& a, int b, const OwnSeq& s) {
  const int group = a.hq / a.hk;
  return a.seqs.cu == nullptr ? b * ((a.seqs.each * group + R - 1) / R) : s.q0 * group / R + b;
}

// Sums up the list: every wave for itself, each lane over batch / 64 sequences. The prefix's positions are those of
// all sequences: what a tile of its rows does not see costs no products. (A sum by the whole workgroup takes three
// barriers, and an array in LDS; where that is not part of the tiles' array, the compiler has every read of a tile wait
// for the next tile's copies: 32 caches of up to 4100 keys, 72 us for 67.)
__device__ __forceinline__ int lane_sequences(const PagedArgs& a) { return uni((a.seqs.batch + 63) / 64); }
template <int R, int KT, int PR, int PKT>
__device__ __forceinline__ List sum_up(const PagedArgs& a, bool with_prefix, Entry* table, List::Lane* lanes) {
  const int lane = threadIdx.x & 63;
  const int per = lane_sequences(a), from = lane * per, to = min(a.seqs.batch, from + per);
  List l{};
  l.lanes = lanes;
  OwnSeq own{0, 0, 0};
  int mine = 0, p0 = 0x7fffffff, p1 = -0x7fffffff;
#pragma unroll 2
  for (int b = from; b < to; ++b) {
    const OwnSeq s = paged_sequence(a, b);
    if (b == from) own = s;
    const int tiles = row_tiles<R>(a, s);
    for (int i = 0; i < tiles; ++i) {
      Item it;
      own_tile<R, KT>(a, b, s, i, it);
      mine += it.n;
    }
    if (tiles > 0) {
      p0 = min(p0, s.lk - s.lq + a.prefix_len);
      p1 = max(p1, s.lk - 1 + a.prefix_len);
    }
  }
  int sum = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int x = __shfl_up(sum, o);
    if (lane >= o) sum += x;
  }
  lanes[lane] = List::Lane{sum - mine, own};  // every wave the same
  if (a.prefix_len > 0) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      p0 = min(p0, __shfl_xor(p0, o));
      p1 = max(p1, __shfl_xor(p1, o));
    }
    l.pre = key_tiles<PKT>(a.left, a.right, min(a.sinks, a.prefix_len), uni(p0), uni(p1), a.prefix_len);
    l.pre = KeyTiles{uni(l.pre.sink), uni(l.pre.band), uni(l.pre.n)};
    if (with_prefix) {
      l.pre_tiles = uni((a.nq * (a.hq / a.hk) + PR - 1) / PR);
      l.pre_units = l.pre_tiles * max(l.pre.n, 1);
    }
  }
  l.units = l.pre_units + __builtin_amdgcn_readlane(sum, 63);
  if (table != nullptr) {
    int at = l.pre_units + sum - mine;
    for (int b = from; b < to; ++b) {
      const OwnSeq s = paged_sequence(a, b);
      const int tiles = row_tiles<R>(a, s), first = first_entry<R>(a, b, s);
      for (int i = 0; i < tiles; ++i) {
        Item it;
        own_tile<R, KT>(a, b, s, i, it);
        table[first + i] = Entry{at, it.n};
        at += it.n;
      }
    }
  }
  return l;
}

// First unit of run w, floor(units w / runs), and the run of unit u. In 64-bit floats: the products, below 2^31 units
// times 2^16 runs, are exact, and a quotient that is no whole number is 2^-47 of itself from the next one at least, more
// than the division's rounding. (64-bit integer divisions are loops of a few hundred instructions.)
__device__ __forceinline__ int run_start(int units, int runs, int w) { return uni(int(double(units) * w / runs)); }
__device__ __forceinline__ int owner(int units, int runs, int u) {
  return int(((double(u) + 1.0) * runs - 1.0) / units);
}

__device__ __forceinline__ void prefix_item(const PagedArgs& a, const List& l, int tile, Item& it) {
  it.prefix = true;
  it.inside = tile;
  it.keys = Keys{a.prefix, a.prefix_len, min(a.sinks, a.prefix_len)};
  it.kt = l.pre;
  it.n = max(l.pre.n, 1);
}
__device__ __forceinline__ void to_scalars(const PagedArgs& a, Item& it) {
  it.b = uni(it.b);
  it.inside = uni(it.inside);
  it.s = OwnSeq{uni(it.s.q0), uni(it.s.lq), uni(it.s.lk)};
  it.prefix = uni(it.prefix);
  it.keys = Keys{it.prefix ? a.prefix : a.pool.table + it.b * a.pool.table_ts, uni(it.keys.n), uni(it.keys.sinks)};
  it.kt = KeyTiles{uni(it.kt.sink), uni(it.kt.band), uni(it.kt.n)};
  it.n = uni(it.n);
}
// The item of unit u, and the unit's number in it.
template <int R, int KT>
__device__ __forceinline__ int locate(const PagedArgs& a, const List& l, int u, Item& it) {
  if (u < l.pre_units) {
    const int n = max(l.pre.n, 1), item = uni(u / n);
    prefix_item(a, l, item, it);
    it.b = 0;
    it.s = OwnSeq{0, 0, 0};
    return u - item * n;
  }
  u -= l.pre_units;
  // the last lane whose sequences start at u or before: u is less than their units
  const int t = uni(__popcll(__ballot(l.lanes[threadIdx.x & 63].start <= u))) - 1;
  const List::Lane from = l.lanes[t];
  u -= uni(from.start);
  const int per = lane_sequences(a), last = min(a.seqs.batch, (t + 1) * per);
  for (int b = t * per; b < last; ++b) {
    OwnSeq s;
    if (b == t * per)
      s = OwnSeq{uni(from.s.q0), uni(from.s.lq), uni(from.s.lk)};
    else
      s = uniform_sequence(a, b);
    const int tiles = uni(row_tiles<R>(a, s));
    for (int i = 0; i < tiles; ++i) {
      own_tile<R, KT>(a, b, s, i, it);
      const int n = uni(it.n);
      if (u < n) {
        to_scalars(a, it);
        return u;
      }
      u -= n;
    }
  }
  it.n = 0;
  return 0;
}
// The item after `it`, whose first unit is u.
template <int R, int KT>
__device__ __forceinline__ void advance(const PagedArgs& a, const List& l, int u, Item& it) {
  if (it.prefix && it.inside + 1 < l.pre_tiles) {
    ++it.inside;
  } else if (!it.prefix && it.inside + 1 < uni(row_tiles<R>(a, it.s))) {
    own_tile<R, KT>(a, it.b, it.s, it.inside + 1, it);
    to_scalars(a, it);
  } else {
    locate<R, KT>(a, l, u, it);
  }
}

// The target of a lane's row after units [t0, t1) of an item by run w of kv head kvh.
__device__ __forceinline__ Target target_of(const PagedArgs& a, const PartMap& m, const Item& it, const Rows& r, int w, int kvh,
                                            int t0, int t1, int row_in_tile) {
  Target t{nullptr, 0, 0};
  char* const ws = reinterpret_cast<char*>(a.part);
  const int kind = it.prefix;
  if (t0 == 0 && t1 == it.n) {
    if (a.prefix_len == 0) return t;
    t.part = reinterpret_cast<float*>(ws + (kind ? m.whole[1] : m.whole[0]));
    t.row = int64_t(r.head) * a.nq + r.tok;
    t.rows = int64_t(a.hq) * a.nq;
  } else {  // an item that goes on in the next run: its second slot
    const int rows = kind ? m.rows[1] : m.rows[0];
    t.part = reinterpret_cast<float*>(ws + (kind ? m.slots[1] : m.slots[0]));
    t.row = ((int64_t(w) * a.hk + kvh) * 2 + (t0 == 0)) * rows + row_in_tile;
    t.rows = (kind ? m.slot_count[1] : m.slot_count[0]) * rows;
  }
  return t;
}

template <class E, int NB, int KEYS, int KB>
__device__ __forceinline__ void compute_tile(const PagedArgs& a, const Keys& keys, const KeyTiles& kt, const Rows& r,
                                             RowState<E, NB, KB>& st, const unsigned char* ks, int it, float c,
                                             const typename Tile<E, NB>::Lane& at, int lane) {
  typedef Tile<E, NB> T;
#pragma unroll
  for (int part = 0; part < KEYS / (32 * KB); ++part) {
    const int j0 = kt.at(it) * KEYS + part * 32 * KB, j1 = j0 + 32 * KB - 1;
    if (!tile_seen(a, keys, r, j0, j1)) continue;
    st.scores(ks + part * 32 * KB * T::kPitch, (a.dim + 15) / 16, at);
    if (!tile_whole(a, keys, r, j0, j1)) {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) hide(st.s[kb], j0 + 32 * kb, r.lo, r.hi, keys.sinks, lane);
    }
    st.weigh(c);
    st.multiply(ks + KEYS * T::kPitch + part * 32 * KB * T::kPitch, at);
  }
}

// The arguments of a kernel that takes StreamArgs alone, read again where they are used: held in scalar registers from
// the kernel's start on they crowd out what the loops need (200 spills a kernel).
struct StreamArgs {
  PagedArgs a;
  PartMap m;
};
__device__ __forceinline__ const StreamArgs& arguments() {
  typedef __attribute__((address_space(4))) const StreamArgs* Ptr;
  Ptr p = (Ptr)(__builtin_amdgcn_kernarg_segment_ptr());
  asm volatile("" : "+s"(p));
  return *(const StreamArgs*)(p);
}

// Run w of the list for one kv head, one wave: items of 32 rows, the next tile always on its way to LDS, over items'
// borders too. There is one place that begins an item, one that fetches and one that computes: code that runs once is
// read from memory, cache line by cache line.
template <class E, int NB>
__device__ __forceinline__ void token_run(const List& l, int kvh, int w, int runs, unsigned char* mem) {
  typedef PagedShape<E, NB, true> F;
  typedef Tile<E, NB> T;
  constexpr int KB = 1, NBUF = F::kBuffers;
  const int lane = threadIdx.x & 63, l32 = lane & 31, h = lane >> 5;
  const int u_end = run_start(l.units, runs, w + 1);
  int u = run_start(l.units, runs, w);  // next unit to fetch
  if (u >= u_end) return;
  const typename T::Lane at = T::lane_of(lane);
  PagedCopy<E, NB, F::kKeys, 1> kc, vc;
  Item item, next;  // of the tile in work, and of the one to fetch
  int t, tn, ids;   // their numbers, the pages of the latter
  auto pages = [&](const PagedArgs& a, const Item& i, int tile) {
    return tile < i.kt.n && lane < F::kKeys ? entry_of(a, i.keys, i.kt.at(tile) * F::kKeys + lane) : -1;
  };
  auto fetch = [&](const PagedArgs& a, int buf) {
    if (tn < next.kt.n) {
      const int t0 = next.kt.at(tn) * F::kKeys, mask = (1 << a.pool.log2) - 1;
      unsigned char* dst = mem + buf * 2 * F::kTileBytes;
      const int of = checked(a, ids);
      kc.template run<false>(dst, static_cast<const E*>(a.pool.k) + kvh * a.pool.khs, of, mask, t0, next.keys.n - t0);
      vc.template run<true>(dst + F::kTileBytes, static_cast<const E*>(a.pool.v) + kvh * a.pool.vhs, of, mask, t0,
                            next.keys.n - t0);
    }
    ++u;
    if (++tn < next.n) ids = pages(a, next, tn);
  };
  {
    const PagedArgs& a = arguments().a;
    kc.start(a.pool.kps, a.pool.kss, a.dim, 0, lane);
    vc.start(a.pool.vps, a.pool.vss, a.dim, 0, lane);
    t = tn = uni(locate<F::kRows, F::kKeys>(a, l, u, next));
    to_scalars(a, next);
    ids = pages(a, next, tn);
  }
  RowState<E, NB, KB> st;
  Rows r;
  int t0 = t, t1 = t, buf = 0, left = next.n > 0 ? u_end - u : 0;  // units to compute
  bool waiting = NBUF == 2;  // for the run's first tile: nothing to compute yet
  while (left > 0) {
    const PagedArgs& a = arguments().a;
    if (t == t1) {  // an item begins: the one whose tile was fetched last, or is fetched first
      item = next;
      t0 = t;
      t1 = min(item.n, t + left);
      r = item.prefix ? prefix_rows(a, item.keys, item.inside * F::kRows, kvh, l32)
                      : own_rows(a, item.s, item.keys, item.inside * F::kRows, kvh, l32);
      st.start(static_cast<const E*>(a.q.p) + r.tok * a.q.ts + r.head * a.q.hs, r.on, a.dim, lane);
    }
    __builtin_amdgcn_s_waitcnt(0);  // the tile, and the queries before the next tile's copies
    asm volatile("" ::: "memory");
    if (u < u_end) {
      if (tn == next.n) {
        advance<F::kRows, F::kKeys>(a, l, u, next);
        to_scalars(a, next);
        tn = 0;
        ids = pages(a, next, 0);
        __builtin_amdgcn_s_waitcnt(0);  // here, not where they are next set, behind the copies
      }
      fetch(a, buf);
    }
    buf ^= NBUF - 1;
    if (waiting) {
      waiting = false;
      continue;
    }
    if constexpr (NBUF == 1) {
      __builtin_amdgcn_s_waitcnt(0);
      asm volatile("" ::: "memory");
    }
    if (t < item.kt.n)
      compute_tile<E, NB, F::kKeys, KB>(a, item.keys, item.kt, r, st, mem + buf * 2 * F::kTileBytes, t,
                                        a.scale * kLog2e, at, lane);
    --left;
    if (++t < t1) continue;
    st.join_halves();
    const StreamArgs& sa = arguments();
    const Target to = target_of(a, sa.m, item, r, w, kvh, t0, t1, l32);
    const uint32_t bad = bad_rows(r.on ? zero_if_finite<NB>(st.acc) : 0.f);
    const bool mine = (bad >> l32) & 1u;
    if (r.on && !mine) store_row<E, NB>(a, to, r, st.acc, st.mc, st.l, 0, NB, h == 0, h);
    if (bad != 0) {  // again without what the rows do not see; the tile just used is free
      float* const lds = reinterpret_cast<float*>(mem + buf * 2 * F::kTileBytes);
      safe_rows<E, NB, F::kKeys, NB>(a, item.keys, item.kt, t0, min(t1, item.kt.n), r, kvh, 0, lds, lane, st.acc,
                                     st.mc, st.l);
      if (r.on && mine) store_row<E, NB>(a, to, r, st.acc, st.mc, st.l, 0, NB, h == 0, h);
    }
    t = t1 = 0;
    if (NBUF == 1 && left > 0) {
      advance<F::kRows, F::kKeys>(a, l, u, next);
      to_scalars(a, next);
      tn = 0;
      ids = pages(a, next, 0);
    }
  }
}

// Units u .. u_end of the list by one workgroup, from unit t of `item` on: items of 128 rows, 32 a wave. WHOLE: one
// item, straight to out.
template <class E, int NB, bool WHOLE>
__device__ __forceinline__ void tile_run(const List& l, int kvh, Item item, int t, int u, int u_end,
                                         int w, unsigned char* mem) {
  typedef PagedShape<E, NB, false> F;
  typedef Tile<E, NB> T;
  constexpr int KB = NB <= 2 ? 1 : F::kKeys / 32;
  const int lane = threadIdx.x & 63, l32 = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const typename T::Lane at = T::lane_of(lane);
  PagedCopy<E, NB, F::kKeys, 4> kc, vc;
  {
    const PagedArgs& a = arguments().a;
    kc.start(a.pool.kps, a.pool.kss, a.dim, wave, lane);
    vc.start(a.pool.vps, a.pool.vss, a.dim, wave, lane);
  }
  RowState<E, NB, KB> st;
  while (u < u_end && item.n > 0) {
    const int t0 = uni(t), t1 = uni(min(item.n, t + (u_end - u))), end = min(t1, item.kt.n);
    u += t1 - t0;
    auto pages = [&](const PagedArgs& a, int i) {
      return i < end && lane < F::kKeys ? entry_of(a, item.keys, item.kt.at(i) * F::kKeys + lane) : -1;
    };
    Rows r;
    int first_ids, ids;
    {
      const PagedArgs& a = arguments().a;
      first_ids = pages(a, t0);  // on their way while the rows are worked out
      ids = pages(a, t0 + 1);
      r = item.prefix ? prefix_rows(a, item.keys, item.inside * F::kRows + 32 * wave, kvh, l32)
                      : own_rows(a, item.s, item.keys, item.inside * F::kRows + 32 * wave, kvh, l32);
      st.start(static_cast<const E*>(a.q.p) + r.tok * a.q.ts + r.head * a.q.hs, r.on, a.dim, lane);
    }
    {
      const PagedArgs& a = arguments().a;
      const E* kbase = static_cast<const E*>(a.pool.k) + kvh * a.pool.khs;
      const E* vbase = static_cast<const E*>(a.pool.v) + kvh * a.pool.vhs;
      const float c = a.scale * kLog2e;
      const int mask = (1 << a.pool.log2) - 1;
      auto fetch = [&](int i, int buf, int ids) {
        const int j0 = item.kt.at(i) * F::kKeys;
        unsigned char* dst = mem + buf * 2 * F::kTileBytes;
        ids = checked(a, ids);
        kc.template run<false>(dst, kbase, ids, mask, j0, item.keys.n - j0);
        vc.template run<true>(dst + F::kTileBytes, vbase, ids, mask, j0, item.keys.n - j0);
      };
      if (t0 < end) fetch(t0, 0, first_ids);
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
      for (int i = t0; i < end; i += 2) {  // two tiles a round: the buffers' addresses are constants
#pragma unroll
        for (int buf = 0; buf < 2; ++buf) {
          if (i + buf >= end) break;
          if (i + buf + 1 < end) {
            fetch(i + buf + 1, buf ^ 1, ids);
            ids = pages(a, i + buf + 2);
          }
          compute_tile<E, NB, F::kKeys, KB>(a, item.keys, item.kt, r, st, mem + buf * 2 * F::kTileBytes, i + buf, c, at,
                                            lane);
          __builtin_amdgcn_s_waitcnt(0);
          bare_barrier();
        }
      }
    }
    st.join_halves();
    const StreamArgs& sa = arguments();
    const PagedArgs& a = sa.a;
    const Target to = WHOLE ? Target{nullptr, 0, 0} : target_of(a, sa.m, item, r, w, kvh, t0, t1, 32 * wave + l32);
    const uint32_t bad = bad_rows(r.on ? zero_if_finite<NB>(st.acc) : 0.f);
    const bool mine = (bad >> l32) & 1u;
    if (r.on && !mine) store_row<E, NB>(a, to, r, st.acc, st.mc, st.l, 0, NB, h == 0, h);
    if (bad != 0) {
      safe_rows<E, NB, F::kKeys, NB>(a, item.keys, item.kt, t0, end, r, kvh, 0,
                                     reinterpret_cast<float*>(mem) + wave * 1024, lane, st.acc, st.mc, st.l);
      if (r.on && mine) store_row<E, NB>(a, to, r, st.acc, st.mc, st.l, 0, NB, h == 0, h);
    }
    if constexpr (WHOLE) return;
    if (u < u_end) {
      advance<F::kRows, F::kKeys>(a, l, u, item);
      to_scalars(a, item);
      t = 0;
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();  // the tiles are read
    }
  }
}

// How many runs `units` are dealt to: `most`, or fewer of `least` units.
__device__ __forceinline__ int runs_of(int units, int most, int least) {
  const int r = units / least;
  return uni(r < 1 ? 1 : r < most ? r : most);
}
template <class E>
constexpr int kLeastTokenUnits = sizeof(E) == 4 ? 1 : 2;
template <class E>
constexpr int kLeastTileUnits = sizeof(E) == 4 ? 1 : 2;

// Waves take the whole list, or workgroups do, or the first workgroups the prefix and the others' waves the sequences'
// own keys. The launch has a wave (token runs) or workgroup (tile runs) at least for every kv head.
enum { kTokens = 0, kTiles = 1, kMixed = 2 };
template <class E, int NB, int MODE>
struct ModeShape {
  typedef PagedShape<E, NB, true> FT;
  typedef PagedShape<E, NB, false> FP;
  static constexpr int kLds = MODE == kTokens  ? FT::kLds
                              : MODE == kTiles ? FP::kLds
                                               : (FT::kLds > FP::kLds ? FT::kLds : FP::kLds);
  // Workgroups that a CU holds. (Tile runs, 16 heads of 64, 1401 rows over up to 8192 keys: three 96 us, four 111, two
  // 99; the kernel without runs holds four. Three spill 2 vector registers; two at half heads of 128 9, at fp32 heads of 96
  // 37.)
  static constexpr int kWhole = sizeof(E) == 4 ? (NB == 4 ? 1 : 2) : NB <= 2 ? 4 : 2;
  static constexpr int kPerCu = MODE == kTiles ? (sizeof(E) == 2 && NB <= 2 ? 3 : kWhole)
                                               : (kLds > 80 * 1024 ? 1 : 2);
  static constexpr int kGrid = 256 * kPerCu;
};
// Time of a prefix unit of a workgroup, in those of a wave's own. Swept at one shape, bf16 heads of 128, 256 sequences
// behind 8192 keys: 0.7 77.6 us, 0.55 92, 0.86 85. Other types and widths, whose units and workgroups a CU differ, use
// the same.
constexpr float kPrefixCost = 0.7f;

template <class E, int NB, int MODE>
__global__ __launch_bounds__(256, (ModeShape<E, NB, MODE>::kPerCu)) void paged_stream(StreamArgs) {
  typedef ModeShape<E, NB, MODE> M;
  typedef typename M::FT FT;
  typedef typename M::FP FP;
  __shared__ __attribute__((aligned(1024))) unsigned char s_mem[M::kLds + 64 * sizeof(List::Lane)];
  List::Lane* const lanes = reinterpret_cast<List::Lane*>(s_mem + M::kLds);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int grid = gridDim.x, block = blockIdx.x;
  const StreamArgs& sa = arguments();
  const PagedArgs& a = sa.a;
  char* const ws = reinterpret_cast<char*>(a.part);
  Entry* const table = block == 0 && wave == 0 ? reinterpret_cast<Entry*>(ws + sa.m.table) : nullptr;
  Lists* const lists = reinterpret_cast<Lists*>(ws + sa.m.head);
  if constexpr (MODE == kTokens) {
    const List l = sum_up<FT::kRows, FT::kKeys, FT::kRows, FT::kKeys>(a, true, table, lanes);
    const int runs = runs_of(l.units, 4 * grid / a.hk, kLeastTokenUnits<E>);
    if (block == 0 && threadIdx.x == 0) *lists = Lists{{l.units, l.units}, {runs, runs}, max(l.pre.n, 1)};
    const int at = block * 4 + wave, w = uni(at / a.hk);
    if (w < runs) token_run<E, NB>(l, at - w * a.hk, w, runs, s_mem + wave * (FT::kLds / 4));
  } else if constexpr (MODE == kTiles) {
    const List l = sum_up<FP::kRows, FP::kKeys, FP::kRows, FP::kKeys>(a, true, table, lanes);
    const int runs = runs_of(l.units, grid / a.hk, kLeastTileUnits<E>);
    if (block == 0 && threadIdx.x == 0) *lists = Lists{{l.units, l.units}, {runs, runs}, max(l.pre.n, 1)};
    if (block >= runs * a.hk) return;
    const int at = xcd_remap(block, runs * a.hk), kvh = uni(at / runs), w = at - kvh * runs;
    const int u = run_start(l.units, runs, w);
    Item item;
    const int t = uni(locate<FP::kRows, FP::kKeys>(a, l, u, item));
    to_scalars(a, item);
    tile_run<E, NB, false>(l, kvh, item, t, u, run_start(l.units, runs, w + 1), w, s_mem);
  } else {
    const List l = sum_up<FT::kRows, FT::kKeys, FP::kRows, FP::kKeys>(a, false, table, lanes);
    List p = l;
    p.pre_tiles = uni((a.nq * (a.hq / a.hk) + FP::kRows - 1) / FP::kRows);
    p.pre_units = p.units = p.pre_tiles * max(l.pre.n, 1);
    const float cost = kPrefixCost * float(p.units), own = 0.25f * float(l.units);
    int share = int(float(grid) * cost / (cost + own) + 0.5f);
    share = min(max(share, a.hk), grid - (a.hk + 3) / 4);
    const int pre_runs = runs_of(p.units, share / a.hk, kLeastTileUnits<E>), pre_blocks = pre_runs * a.hk;
    const int runs = runs_of(l.units, 4 * (grid - pre_blocks) / a.hk, kLeastTokenUnits<E>);
    if (block == 0 && threadIdx.x == 0) *lists = Lists{{l.units, p.units}, {runs, pre_runs}, max(l.pre.n, 1)};
    if (block < pre_blocks) {
      const int at = xcd_remap(block, pre_blocks), kvh = uni(at / pre_runs), w = at - kvh * pre_runs;
      const int u = run_start(p.units, pre_runs, w);
      Item item;
      const int t = uni(locate<FP::kRows, FP::kKeys>(a, p, u, item));
      to_scalars(a, item);
      tile_run<E, NB, false>(p, kvh, item, t, u, run_start(p.units, pre_runs, w + 1), w, s_mem);
    } else {
      const int at = (block - pre_blocks) * 4 + wave, w = uni(at / a.hk);
      if (w < runs) token_run<E, NB>(l, at - w * a.hk, w, runs, s_mem + wave * (FT::kLds / 4));
    }
  }
}

// One item a workgroup, straight to out: prompts of many rows.
template <class E, int NB>
__global__ __launch_bounds__(256, (ModeShape<E, NB, kTiles>::kWhole)) void paged_tiles(StreamArgs, int tiles) {
  typedef PagedShape<E, NB, false> F;
  __shared__ __attribute__((aligned(1024))) unsigned char s_mem[F::kLds];
  const PagedArgs& a = arguments().a;
  const int group = a.hq / a.hk, w = xcd_remap(blockIdx.x, gridDim.x), tile = w % tiles;
  int inside, b;
  if (a.seqs.cu == nullptr) {
    const int per = (a.seqs.each * group + F::kRows - 1) / F::kRows;
    b = tile / per;
    inside = tile - b * per;
  } else {
    b = find_sequence(a.seqs.cu, a.seqs.batch, group, F::kRows, tile, &inside);
  }
  const OwnSeq s = uniform_sequence(a, b);
  if (inside < 0 || inside >= row_tiles<F::kRows>(a, s)) return;
  Item item;
  own_tile<F::kRows, F::kKeys>(a, b, s, inside, item);
  to_scalars(a, item);
  tile_run<E, NB, true>(List{}, uni(w / tiles), item, 0, 0, item.n, 0, s_mem);
}

// Few rows over few keys: one row tile and kv head a workgroup, whose waves share its rows and split its keys, the
// prefix's and its own, straight to out. Eight waves where their tiles fit: a call of this size is as long as one
// wave's tiles, one after another.
template <class E, int NB>
struct ShortShape {
  typedef Tile<E, NB> T;
  static constexpr int kRows = 32, kKeys = 32, kTileBytes = kKeys * T::kPitch;
  static constexpr int kWaves = 16 * kTileBytes <= 128 * 1024 ? 8 : 4;
  static constexpr int kBuffers = kWaves * 4 * kTileBytes <= 128 * 1024 ? 2 : 1;
  static constexpr int kLds = kWaves * kBuffers * 2 * kTileBytes;
  static_assert(kLds >= kWaves * NB * 4096 && kLds >= kWaves * 4096, "the waves' sums and factors");
};
template <class E, int NB>
__global__ __launch_bounds__((64 * ShortShape<E, NB>::kWaves)) void paged_short(PagedArgs a, int tiles) {
  typedef ShortShape<E, NB> F;
  typedef Tile<E, NB> T;
  constexpr int KB = 1, NBUF = F::kBuffers, W = F::kWaves;
  __shared__ __attribute__((aligned(1024))) unsigned char s_mem[F::kLds];
  const int lane = threadIdx.x & 63, l32 = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = a.hq / a.hk, tile = blockIdx.x % tiles, kvh = uni(blockIdx.x / tiles);
  int inside, b;
  if (a.seqs.cu == nullptr) {
    const int per = (a.seqs.each * group + F::kRows - 1) / F::kRows;
    b = tile / per;
    inside = tile - b * per;
  } else {
    b = find_sequence(a.seqs.cu, a.seqs.batch, group, F::kRows, tile, &inside);
  }
  const OwnSeq s = uniform_sequence(a, b);
  if (inside < 0 || inside >= row_tiles<F::kRows>(a, s)) return;
  Item item;
  own_tile<F::kRows, F::kKeys>(a, b, s, inside, item);
  to_scalars(a, item);
  // the prefix as this tile's rows see it
  const Keys pre_keys{a.prefix, a.prefix_len, min(a.sinks, a.prefix_len)};
  KeyTiles pre_kt{0, 0, 0};
  if (a.prefix_len > 0) {
    const int rows = s.lq * group, p = a.prefix_len + s.lk - s.lq;
    pre_kt = key_tiles<F::kKeys>(a.left, a.right, pre_keys.sinks, inside * F::kRows / group + p,
                                 (min(rows, (inside + 1) * F::kRows) - 1) / group + p, a.prefix_len);
    pre_kt = KeyTiles{uni(pre_kt.sink), uni(pre_kt.band), uni(pre_kt.n)};
  }
  const int end = pre_kt.n + item.kt.n;
  // tile i: of the prefix, then of the own keys
  auto keys_of = [&](int i) { return i < pre_kt.n ? pre_keys : item.keys; };
  auto key_of = [&](int i) { return (i < pre_kt.n ? pre_kt.at(i) : item.kt.at(i - pre_kt.n)) * F::kKeys; };
  auto pages = [&](int i) { return i < end && lane < F::kKeys ? entry_of(a, keys_of(i), key_of(i) + lane) : -1; };
  int i = wave, buf = 0, ids = pages(i);  // on their way while the rows are worked out
  const Rows own = own_rows(a, s, item.keys, inside * F::kRows, kvh, l32);
  Rows pre = own;
  see(a, pre_keys, own.lo + a.left + a.prefix_len, pre);
  pre.p0 += a.prefix_len;
  pre.p1 += a.prefix_len;
  const typename T::Lane at = T::lane_of(lane);
  RowState<E, NB, KB> st;
  st.start(static_cast<const E*>(a.q.p) + own.tok * a.q.ts + own.head * a.q.hs, own.on, a.dim, lane);
  const E* kbase = static_cast<const E*>(a.pool.k) + kvh * a.pool.khs;
  const E* vbase = static_cast<const E*>(a.pool.v) + kvh * a.pool.vhs;
  const float c = a.scale * kLog2e;
  const int mask = (1 << a.pool.log2) - 1;
  unsigned char* const mem = s_mem + wave * NBUF * 2 * F::kTileBytes;
  PagedCopy<E, NB, F::kKeys, 1> kc, vc;
  kc.start(a.pool.kps, a.pool.kss, a.dim, 0, lane);
  vc.start(a.pool.vps, a.pool.vss, a.dim, 0, lane);
  auto fetch = [&](int i, int buf, int ids) {
    const int j0 = key_of(i), left = keys_of(i).n - j0;
    unsigned char* dst = mem + buf * 2 * F::kTileBytes;
    ids = checked(a, ids);
    kc.template run<false>(dst, kbase, ids, mask, j0, left);
    vc.template run<true>(dst + F::kTileBytes, vbase, ids, mask, j0, left);
  };
  auto compute = [&](int i, int buf) {
    const bool p = i < pre_kt.n;
    Rows r = own;
    r.lo = p ? pre.lo : own.lo;
    r.hi = p ? pre.hi : own.hi;
    r.p0 = p ? pre.p0 : own.p0;
    r.p1 = p ? pre.p1 : own.p1;
    const KeyTiles kt{0, p ? pre_kt.at(i) : item.kt.at(i - pre_kt.n), 1};
    compute_tile<E, NB, F::kKeys, KB>(a, keys_of(i), kt, r, st, mem + buf * 2 * F::kTileBytes, 0, c, at, lane);
  };
  // each wave its own tiles and LDS: no barrier in the loop
  if (NBUF == 2 && i < end) {
    fetch(i, 0, ids);
    ids = pages(i + W);
  }
  for (; i < end; i += W) {
    if constexpr (NBUF == 2) {
      __builtin_amdgcn_s_waitcnt(0);
      asm volatile("" ::: "memory");
      if (i + W < end) {
        fetch(i + W, buf ^ 1, ids);
        ids = pages(i + 2 * W);
      }
      compute(i, buf);
      buf ^= 1;
    } else {
      __builtin_amdgcn_s_waitcnt(0);  // the last tile's reads are done
      fetch(i, 0, ids);
      ids = pages(i + W);
      __builtin_amdgcn_s_waitcnt(0);
      asm volatile("" ::: "memory");
      compute(i, 0);
    }
  }
  st.join_halves();
  // the waves hold the same rows over different keys: join them in wave order; wave w sums block w
  float* red = reinterpret_cast<float*>(s_mem);
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  if (lane < 32) {
    red[wave * 64 + lane] = st.mc;
    red[wave * 64 + 32 + lane] = st.l;
  }
  __syncthreads();
  float mc = -INFINITY;
#pragma unroll
  for (int w = 0; w < W; ++w) mc = fmaxf(mc, red[w * 64 + l32]);
  float l = 0.f, mine = 0.f;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    const float mw = red[w * 64 + l32];
    const float f = mw == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mw - mc);
    l += f * red[w * 64 + 32 + l32];
    if (w == wave) mine = f;
  }
  const bool any = st.mc != -INFINITY;
  __syncthreads();
#pragma unroll
  for (int d = 0; d < NB; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) red[((wave * NB + d) * 16 + e) * 64 + lane] = any ? st.acc[d][e] * mine : 0.f;
  __syncthreads();
  const bool writer = wave < NB;
  float zero = 0.f;
  if (writer) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) v += red[((w * NB + wave) * 16 + e) * 64 + lane];
      st.acc[0][e] = v;
      if (own.on) zero = fmaf(v, 0.f, zero);
    }
  }
  // rows whose sums are not finite, again without what they do not see; each wave has seen some of the columns: the
  // rows of all
  uint32_t bad = bad_rows(zero);
  uint32_t* flags = reinterpret_cast<uint32_t*>(s_mem);
  __syncthreads();
  if (lane == 0) flags[wave] = bad;
  __syncthreads();
  bad = 0;
#pragma unroll
  for (int w = 0; w < NB; ++w) bad |= flags[w];
  const Target to{nullptr, 0, 0};
  const bool again = (bad >> l32) & 1u;
  if (own.on && writer && !again) store_row<E, NB>(a, to, own, st.acc, mc, l, wave, 1, h == 0 && wave == 0, h);
  if (bad != 0) {
    __syncthreads();  // the flags are read
    if (!writer) return;
    float* const lds = reinterpret_cast<float*>(s_mem) + wave * 1024;
    safe_rows<E, NB, F::kKeys, 1>(a, pre_keys, pre_kt, 0, pre_kt.n, pre, kvh, wave, lds, lane, st.acc, mc, l);
    safe_rows<E, NB, F::kKeys, 1, true>(a, item.keys, item.kt, 0, item.kt.n, own, kvh, wave, lds, lane, st.acc, mc, l);
    if (own.on && again) store_row<E, NB>(a, to, own, st.acc, mc, l, wave, 1, h == 0 && wave == 0, h);
  }
}

// Joins the parts of the rows of an item (own row tile `tile`, kv head): `rows` rows a wave, or (WPR > 1) one by WPR
// waves; a lane has four elements, and the parts are dealt to the lanes' groups in turn, whose sums are added in a
// fixed order. R: rows of a tile of the own keys, PR: of the prefix.
template <class E, int WPR, int R, int PR>
__global__ __launch_bounds__(WPR > 4 ? 64 * WPR : 256) void paged_join(PagedArgs a, PartMap m, int tiles, int chunks, int rows) {
  __shared__ float s_max[WPR], s_sum[WPR];
  __shared__ float4 s_out[WPR][32];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, tw = WPR > 1 ? wave : 0;
  const int group = a.hq / a.hk;
  const int chunk = blockIdx.x % chunks, tile = (blockIdx.x / chunks) % tiles, kvh = blockIdx.x / chunks / tiles;
  int inside, b;
  if (a.seqs.cu == nullptr) {
    const int per = (a.seqs.each * group + R - 1) / R;
    b = tile / per;
    inside = tile - b * per;
  } else {
    b = find_sequence(a.seqs.cu, a.seqs.batch, group, R, tile, &inside);
  }
  char* const ws = reinterpret_cast<char*>(a.part);
  const Lists lists = *reinterpret_cast<const Lists*>(ws + m.head);
  const Entry entry = reinterpret_cast<const Entry*>(ws + m.table)[tile];
  const OwnSeq s = paged_sequence(a, b);
  if (inside < 0 || inside >= row_tiles<R>(a, s)) return;
  // The runs that hold parts, [0] the own keys', [1] the prefix's: no table of a malformed batch leads out of them.
  int first[2] = {0, 0}, n[2] = {0, 0};
  auto find = [&](int kind, int u, int units) {
    if (lists.units[kind] <= 0) return;
    first[kind] = clamp_to(owner(lists.units[kind], lists.runs[kind], u), 0, lists.runs[kind] - 1);
    n[kind] = clamp_to(owner(lists.units[kind], lists.runs[kind], u + units - 1) - first[kind] + 1, 0,
                       lists.runs[kind] - first[kind]);
  };
  find(0, entry.first, entry.n);
  if (a.prefix_len == 0 && n[0] == 1) return;  // stored
  const int64_t all = int64_t(a.hq) * a.nq;
  for (int i = 0; i < rows; ++i) {
    const int in_tile = WPR > 1 ? chunk : (chunk * 4 + wave) * rows + i;
    const int row = inside * R + in_tile;
    if (in_tile >= R || row >= s.lq * group) return;  // WPR > 1: the whole workgroup
    const int tok = s.q0 + row / group, head = kvh * group + row % group;
    const int64_t out_row = int64_t(head) * a.nq + tok;
    int pre_in_tile = 0;
    if (a.prefix_len > 0) {
      const int pre_row = tok * group + row % group, pre_tile = pre_row / PR;
      pre_in_tile = pre_row - pre_tile * PR;
      find(1, pre_tile * lists.pre_n, lists.pre_n);
    }
    const int parts = n[0] + n[1];
    // part p: its elements' row and its statistic
    auto part = [&](int p, const float*& stat) -> const float* {
      const int kind = p >= n[0];
      if (kind) p -= n[0];
      const float* base;
      int64_t at, count;
      if (n[kind] == 1) {
        base = reinterpret_cast<const float*>(ws + m.whole[kind]);
        at = out_row;
        count = all;
      } else {
        base = reinterpret_cast<const float*>(ws + m.slots[kind]);
        at = ((int64_t(first[kind] + p) * a.hk + kvh) * 2 + (p == 0)) * m.rows[kind] + (kind ? pre_in_tile : in_tile);
        count = m.slot_count[kind] * m.rows[kind];
      }
      stat = base + count * a.dim + at;
      return base + at * a.dim;
    };
    const int width = a.dim <= 64 ? 16 : 32;  // lanes of a group
    const int groups = 64 / width, e4 = lane % width;
    const bool on = 4 * e4 < a.dim;
    // this group's parts, kParts at a time: their largest statistic, the sum of their weights, the weighted sum
    float mx = -INFINITY, sum = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kParts = WPR > 1 ? 8 : 4;
    for (int p = tw * groups + lane / width; p < parts; p += kParts * WPR * groups) {
      float lg[kParts];
      float4 x[kParts];
#pragma unroll
      for (int i = 0; i < kParts; ++i) {
        const int pi = p + i * WPR * groups;
        lg[i] = -INFINITY;
        x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (pi < parts) {
          const float* stat;
          x[i] = *reinterpret_cast<const float4*>(part(pi, stat) + 4 * (on ? e4 : 0));
          lg[i] = *stat;
        }
      }
      float top = mx;
#pragma unroll
      for (int i = 0; i < kParts; ++i) top = fmaxf(top, lg[i]);
      const float ms = top == -INFINITY ? 0.f : top, f = __builtin_amdgcn_exp2f(mx - ms);
      sum *= f;
      v.x *= f;
      v.y *= f;
      v.z *= f;
      v.w *= f;
      mx = top;
#pragma unroll
      for (int i = 0; i < kParts; ++i) {
        const float w = __builtin_amdgcn_exp2f(lg[i] - ms);
        sum += w;
        v.x += w * x[i].x;
        v.y += w * x[i].y;
        v.z += w * x[i].z;
        v.w += w * x[i].w;
      }
    }
    auto add = [&](float omx, float osum, const float4& o) {
      const float top = fmaxf(mx, omx), ms = top == -INFINITY ? 0.f : top;
      const float f = __builtin_amdgcn_exp2f(mx - ms), g = __builtin_amdgcn_exp2f(omx - ms);
      mx = top;
      sum = sum * f + osum * g;
      v.x = v.x * f + o.x * g;
      v.y = v.y * f + o.y * g;
      v.z = v.z * f + o.z * g;
      v.w = v.w * f + o.w * g;
    };
    for (int o = width; o < 64; o <<= 1)
      add(__shfl_xor(mx, o), __shfl_xor(sum, o),
          make_float4(__shfl_xor(v.x, o), __shfl_xor(v.y, o), __shfl_xor(v.z, o), __shfl_xor(v.w, o)));
    if constexpr (WPR > 1) {
      if (lane < 32) s_out[wave][lane] = v;
      if (lane == 0) s_max[wave] = mx, s_sum[wave] = sum;
      __syncthreads();
      if (wave > 0) return;
      for (int w = 1; w < WPR; ++w) add(s_max[w], s_sum[w], s_out[w][lane & 31]);
    }
    const float ms = mx == -INFINITY ? 0.f : mx;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    if (on && lane < width) {
      typedef E out4 __attribute__((ext_vector_type(4)));
      E* op = static_cast<E*>(const_cast<void*>(a.o.p)) + tok * a.o.ts + head * a.o.hs + 4 * e4;
      *reinterpret_cast<out4*>(op) = out4{static_cast<E>(v.x * inv), static_cast<E>(v.y * inv),
                                          static_cast<E>(v.z * inv), static_cast<E>(v.w * inv)};
    }
    if (a.lse != nullptr && lane == 0)
      a.lse[out_row] = sum == 0.f ? -INFINITY : (ms + __builtin_amdgcn_logf(sum)) * 0.6931471805599453f;
  }
}

// Whether a workgroup takes a row tile alone (one launch) or the chip's waves share the units (two, and the work list
// first). Measured, GPU time of a call, alone / shared: bf16, 8 sequences, 8 heads of 64, 1024 keys 12.0 / 17.2 us, 2048
// 17.8 / 19.0, 4096 24.6 / 22.9; 32, 4 heads of 128, 2048 keys 25.0 / 31.5, 4096 60 / 46; 128 (512 tiles) 1024 keys
// 46 / 51; 128, 8 heads of 64 (1024 tiles) 256 keys 27 / 23. fp32, 8 sequences, 8 heads of 64, 512 keys 14.1 / 14.0, 1024
// 27 / 23; 4 heads of 128, 256 keys 18.7 / 19.9, 512 25 / 20.5. Behind a prefix, which each tile reads for itself: bf16, 4
// sequences, 16 heads of 64, 1280 keys 13.5 / 17.9, 2304 19.4 / 18.4; 4 heads of 128, 1280 keys 18.0 / 21.9, 2304 27 / 22;
// 32, 16 heads of 64 (512 tiles) 768 keys 21.1 / 20.7.
bool takes_alone(const PagedArgs& a, int64_t tiles, int64_t span) {
  const bool wide = a.dim > 64, prefix = a.prefix_len > 0;
  const int64_t most = a.dtype == TR_SC_F32 ? (wide ? 256 : 512) : wide && prefix ? 1536 : 2048;
  return tiles <= (prefix ? 256 : 512) && span <= most;
}

int64_t own_tiles(const PagedArgs& a, int rows) {
  const int group = a.hq / a.hk;
  if (a.seqs.cu == nullptr) return int64_t(a.seqs.batch) * ((int64_t(a.seqs.each) * group + rows - 1) / rows);
  return tiles_of(a.nq, a.seqs.batch, group, rows);
}

// f(E{}, width in blocks of 32) for the call's type and head size.
template <class E, class F>
hipError_t with_width(const PagedArgs& a, const F& f) {
  switch ((a.dim + 31) / 32) {
    case 1: return f(E(), std::integral_constant<int, 1>());
    case 2: return f(E(), std::integral_constant<int, 2>());
    case 3: return f(E(), std::integral_constant<int, 3>());
    default: return f(E(), std::integral_constant<int, 4>());
  }
}
template <class F>
hipError_t with_shape(const PagedArgs& a, const F& f) {
  if (a.dtype == TR_SC_BF16) return with_width<__bf16>(a, f);
  if (a.dtype == TR_SC_F16) return with_width<_Float16>(a, f);
  return with_width<float>(a, f);
}

PartMap part_map(const PagedArgs& a, const PagedPlan& p) {
  PartMap m{};
  const bool tiles = p.form == PagedForm::tiles, mixed = p.form == PagedForm::mixed;
  const int64_t rows = int64_t(a.nq) * (a.hq / a.hk), each = int64_t(a.seqs.each) * (a.hq / a.hk);
  const auto least = [](int64_t x, int64_t y) { return x < y ? x : y; };
  int64_t at = 256;
  const auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at = (at + bytes + 255) / 256 * 256;
    return here;
  };
  m.table = take(own_tiles(a, tiles ? 128 : 32) * int64_t(sizeof(Entry)));
  if (a.prefix_len > 0)
    for (int i = 0; i < 2; ++i) m.whole[i] = take(int64_t(a.hq) * a.nq * (a.dim + 1) * 4);
  // two slots a run; where one list holds both kinds they share them
  m.rows[0] = int(least(tiles ? 128 : 32, a.seqs.cu == nullptr && (a.prefix_len == 0 || mixed) ? each : rows));
  m.slot_count[0] = int64_t(2) * p.grid * (tiles ? 1 : 4);
  m.slots[0] = take(m.slot_count[0] * m.rows[0] * (a.dim + 1) * 4);
  m.rows[1] = mixed ? int(least(128, rows)) : m.rows[0];
  m.slot_count[1] = mixed ? int64_t(2) * p.grid : m.slot_count[0];
  m.slots[1] = mixed ? take(m.slot_count[1] * m.rows[1] * (a.dim + 1) * 4) : m.slots[0];
  m.head = 0;
  return m;
}
int64_t part_bytes(const PagedArgs& a, const PartMap& m, bool mixed) {
  const int last = mixed ? 1 : 0;
  return m.slots[last] + m.slot_count[last] * m.rows[last] * (a.dim + 1) * 4;
}

template <class E, int R, int PR>
hipError_t launch_join(const PagedArgs& a, const PagedPlan& p, const PartMap& m, hipStream_t st) {
  const int64_t tiles = own_tiles(a, R), items = tiles * a.hk;
  const int64_t in_tile = a.seqs.cu == nullptr && int64_t(a.seqs.each) * (a.hq / a.hk) < R
                              ? int64_t(a.seqs.each) * (a.hq / a.hk)
                              : R;
  // parts of a row, on average: its item's runs, and the prefix's
  const int64_t workers = int64_t(p.grid) * (R == 32 ? 4 : 1), heads = a.hk;
  int64_t parts = workers / (items > 0 ? items : 1) + 1;
  if (a.prefix_len > 0) {
    const int64_t pre_tiles = (int64_t(a.nq) * (a.hq / a.hk) + PR - 1) / PR;
    parts += (PR == 128 ? p.grid / 2 : workers / 2) / (pre_tiles * heads) + 1;
  }
  // Many parts of few rows: sixteen waves a row, or four. Whole calls with 16 / 4 / 1, us: one cache of 99,000 keys, 8
  // heads over 2 of 128 (takes 16) 37.5 / 42 / 91; 32 sequences of 16 heads behind 16,219 keys (4) 35 / 31 / 33; 256 behind
  // 8192 (1) 116 / 82 / 75; parts of prompts, 1401 rows of 16 heads (1) 354 / 151 / 118; 30 rows of 6 heads, fp32 (16) 17.9 /
  // 17.2 / 17.3. The borders lie between these sizes; nearer to them nothing is measured.
  const int64_t rows_all = int64_t(a.hq) * a.nq;
  const int wpr = parts > 48 && rows_all <= 1024 ? 16 : parts > 8 && rows_all <= 16384 ? 4 : 1;
  const int rows = R == 32 ? 1 : 2;
  const int64_t chunks = wpr > 1 ? in_tile : (in_tile + 4 * rows - 1) / (4 * rows);
  if (items * chunks >= (int64_t(1) << 31)) return hipErrorInvalidValue;
  const unsigned grid = unsigned(items * chunks);
  if (wpr == 16)
    paged_join<E, 16, R, PR><<<grid, 1024, 0, st>>>(a, m, int(tiles), int(chunks), 1);
  else if (wpr == 4)
    paged_join<E, 4, R, PR><<<grid, 256, 0, st>>>(a, m, int(tiles), int(chunks), 1);
  else
    paged_join<E, 1, R, PR><<<grid, 256, 0, st>>>(a, m, int(tiles), int(chunks), rows);
  return hipGetLastError();
}

}  // namespace

PagedPlan plan_paged_attention(const PagedArgs& a) {
  PagedPlan p{};
  p.form = PagedForm::shorts;
  p.fits = true;
  if (a.nq == 0) return p;
  const int group = a.hq / a.hk;
  const bool few = int64_t(a.nq) * group <= int64_t(32) * a.seqs.batch;  // rows a sequence
  const int64_t room = int64_t(a.pool.table_pages) << a.pool.log2;
  const int64_t reach = int64_t(a.left) + a.right + 1 + a.sinks + 32 / group;
  const int64_t span = reach < room + a.prefix_len ? reach : room + a.prefix_len;  // keys that a row tile sees at most
  if (few && takes_alone(a, own_tiles(a, 32) * a.hk, span))
    p.form = PagedForm::shorts;
  else if (!few)
    p.form = PagedForm::tiles;
  else
    p.form = a.prefix_len == 0 || int64_t(a.nq) * group <= 32 ? PagedForm::tokens : PagedForm::mixed;
  (void)with_shape(a, [&](auto e, auto nb) {
    typedef decltype(e) E;
    constexpr int NB = decltype(nb)::value;
    p.grid = p.form == PagedForm::tiles   ? ModeShape<E, NB, kTiles>::kGrid
             : p.form == PagedForm::mixed ? ModeShape<E, NB, kMixed>::kGrid
                                          : ModeShape<E, NB, kTokens>::kGrid;
    return hipSuccess;
  });
  const int heads = p.form == PagedForm::tiles ? a.hk : p.form == PagedForm::mixed ? 2 * a.hk : (a.hk + 3) / 4;
  if (p.grid < heads) p.grid = heads;
  // items enough for the chip to even them out by itself: no parts
  if (p.form == PagedForm::tiles && a.prefix_len == 0 && own_tiles(a, 128) * a.hk >= int64_t(4) * p.grid)
    p.form = PagedForm::whole_tiles;
  if (p.form == PagedForm::tokens || p.form == PagedForm::tiles || p.form == PagedForm::mixed)
    p.part_floats = size_t(part_bytes(a, part_map(a, p), p.form == PagedForm::mixed)) / 4;
  if (p.part_floats > 0) {  // the units of the list, each 32 keys at least, are counted in 32 bits
    const int rows = p.form == PagedForm::tiles ? 128 : 32, keys = rows == 128 && a.dtype != TR_SC_F32 ? 64 : 32;
    const int64_t pre = (int64_t(a.nq) * group + rows - 1) / rows * (a.prefix_len / 32 + 3);
    p.fits = pre + own_tiles(a, rows) * (room / keys + 4) < (int64_t(1) << 31);
  }
  return p;
}

hipError_t launch_paged_attention(const PagedArgs& a, const PagedPlan& p, hipStream_t st) {
  if (a.nq == 0) return hipSuccess;
  return with_shape(a, [&](auto e, auto nb) -> hipError_t {
    typedef decltype(e) E;
    constexpr int NB = decltype(nb)::value;
    if (p.form == PagedForm::shorts || p.form == PagedForm::whole_tiles) {
      const int64_t tiles = own_tiles(a, p.form == PagedForm::shorts ? 32 : 128), n = tiles * a.hk;
      if (n >= (int64_t(1) << 31)) return hipErrorInvalidValue;
      if (p.form == PagedForm::shorts)
        paged_short<E, NB><<<unsigned(n), 64 * ShortShape<E, NB>::kWaves, 0, st>>>(a, int(tiles));
      else
        paged_tiles<E, NB><<<unsigned(n), 256, 0, st>>>(StreamArgs{a, PartMap{}}, int(tiles));
      return hipGetLastError();
    }
    const PartMap m = part_map(a, p);
    if (p.form == PagedForm::tokens)
      paged_stream<E, NB, kTokens><<<p.grid, 256, 0, st>>>(StreamArgs{a, m});
    else if (p.form == PagedForm::tiles)
      paged_stream<E, NB, kTiles><<<p.grid, 256, 0, st>>>(StreamArgs{a, m});
    else
      paged_stream<E, NB, kMixed><<<p.grid, 256, 0, st>>>(StreamArgs{a, m});
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    return p.form == PagedForm::tokens  ? launch_join<E, 32, 32>(a, p, m, st)
           : p.form == PagedForm::tiles ? launch_join<E, 128, 128>(a, p, m, st)
                                        : launch_join<E, 32, 128>(a, p, m, st);
  });
}

}  // namespace trsc
