// Shared device parts of the windowed attention kernels: element traits, the
// LDS tile layout, the sequence search and the window's tiles.
//
// Matrix products use 32x32 tiles: v_mfma_f32_32x32x16 for the half types, and
// eight v_mfma_f32_32x32x2_f32 for fp32. In both, a lane's fragment is eight
// elements: of row (or column) lane % 32, at k = 8 (lane / 32) + 0..7 of a
// 16-deep step (the fp32 instruction i of a step takes element i of either
// half). An accumulator's register 4 g + i of lane l holds row
// 8 g + 4 (l / 32) + i, column l % 32.
#pragma once
#include "common.h"
#include "tokens.h"

namespace trsc {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// LDS reads. The restrict gives each an alias scope of its own: without one the
// compiler waits for every copy to LDS in flight before it, the next tile's too.
// Transposing: of 16 lanes, lane i gets element i % 4 of the 8 bytes that lanes
// i / 4, i / 4 + 4, i / 4 + 8 and i / 4 + 12 name.
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
template <class V>
__device__ __forceinline__ V read_lds(const void* __restrict p) { return *static_cast<const V*>(p); }
__device__ __forceinline__ s16x4 read_tr(lds_s16x4* __restrict p) { return __builtin_amdgcn_ds_read_tr16_b64_v4i16(p); }

template <class E>
struct AttnType;  // wide: products in fp32; narrow: the type's exponents do not reach what fp32 sums hold
template <>
struct AttnType<__bf16> {
  typedef __bf16 elt;
  typedef __bf16 frag __attribute__((ext_vector_type(8)));
  static constexpr bool wide = false, narrow = false;
  static __device__ __forceinline__ f32x16 mma(frag a, frag b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
};
template <>
struct AttnType<_Float16> {
  typedef _Float16 elt;
  typedef _Float16 frag __attribute__((ext_vector_type(8)));
  static constexpr bool wide = false, narrow = true;
  static __device__ __forceinline__ f32x16 mma(frag a, frag b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
};
template <>
struct AttnType<float> {
  typedef float elt;
  typedef float frag __attribute__((ext_vector_type(8)));
  static constexpr bool wide = true, narrow = false;
  static __device__ __forceinline__ f32x16 mma(frag a, frag b, f32x16 c) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i], b[i], c, 0, 0, 0);
    return c;
  }
};

// Memory as a bounded buffer (wave-uniform; offsets from `bytes` on read as
// zero), and its direct copy to LDS: lane l of the wave fills lds + 16 l.
typedef __amdgpu_buffer_rsrc_t buffer_t;
__device__ __forceinline__ buffer_t buffer_of(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, int(bytes), 0x00027000);
}
__device__ __forceinline__ void copy_lds16(buffer_t b, uint32_t off, unsigned char* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (__attribute__((address_space(3))) void*)(lds), 16, int(off), 0, 0, 0);
}
__device__ __forceinline__ void copy_lds4(buffer_t b, uint32_t off, unsigned char* lds) {  // lds + 4 l
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (__attribute__((address_space(3))) void*)(lds), 4, int(off), 0, 0, 0);
}
// LDS tile of token rows, NB * 32 elements wide: rows of kPitch bytes in
// 16-byte chunks; chunk c of row r sits at chunk position c ^ key(r). The keys
// spread both reads over the banks: one chunk of 16 consecutive rows (row
// fragments), and four chunks of four consecutive rows (transposed fragments).
template <class E, int NB>
struct Tile {
  typedef AttnType<E> A;
  typedef typename A::frag frag;
  static constexpr int kElt = sizeof(E);
  static constexpr int kPitch = (NB <= 2 ? 64 : 128) * kElt;
  static constexpr int kChunks = kPitch / 16;       // chunk positions of a row
  static constexpr int kPer = 16 / kElt;            // elements of a chunk
  static constexpr int kRowsPerCopy = 64 / kChunks; // rows that one wave-wide copy fills
  static __device__ __forceinline__ int key(int r) {
    if constexpr (kElt == 4) return r & 15;
    if constexpr (kPitch == 256) return ((r & 3) << 2) | ((r >> 2) & 3);
    return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
  }
  static __device__ __forceinline__ int at(int r, int chunk) { return r * kPitch + ((chunk ^ key(r)) << 4); }

  // Copies rows [0, ROWS) of a tile from memory to LDS, this wave's part of it:
  // copies first, first + STEP, ... of ROWS / kRowsPerCopy, 64 lanes x 16 bytes
  // each. A lane's offsets from the tile's first row stay the same from tile to
  // tile; what lies past the tensor's end or a head's width reads as zero (the
  // buffer's bound). Buffer loads, not global ones: with a flat-encoded copy in
  // flight the compiler waits for all LDS reads where it needs one.
  template <int ROWS, int STEP>
  struct Copy {
    static constexpr int kN = (ROWS / kRowsPerCopy + STEP - 1) / STEP;
    uint32_t off[kN], row_bytes;
    int first;
    __device__ __forceinline__ void start(int64_t stride, int dim, int first_, int lane) {
      first = first_;
      row_bytes = uint32_t(dim * kElt);
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        const int row = (first + j * STEP) * kRowsPerCopy + lane / kChunks;
        const int chunk = (lane % kChunks) ^ key(row);
        off[j] = chunk * kPer < dim ? uint32_t(row) * uint32_t(stride * kElt) + chunk * 16 : 0x80000000u;
      }
    }
    // base: the tile's first row (wave-uniform); left: rows from there to the end
    __device__ __forceinline__ void run(unsigned char* lds, const E* base, int64_t stride, int left) const {
      const int rows = left < 0 ? 0 : left > ROWS ? ROWS : left;
      const buffer_t b = buffer_of(base, rows == 0 ? 0 : uint32_t(rows - 1) * uint32_t(stride * kElt) + row_bytes);
#pragma unroll
      for (int j = 0; j < kN; ++j)
        if ((j + 1) * STEP <= ROWS / kRowsPerCopy || first + j * STEP < ROWS / kRowsPerCopy)
          copy_lds16(b, off[j], lds + (first + j * STEP) * 1024);
    }
  };
  // A lane's byte offsets in a tile. key(r) is the same for rows 16 apart, and
  // the chunk's higher bits are the caller's constants, so a fragment's address
  // is one of these, the constants in by XOR and the tile's rows by addition.
  static constexpr int kCols = kElt == 2 ? 2 : 8;
  struct Lane {
    int row, col[kCols];
    // Addresses made from these are made again, not kept in registers (which
    // would be spilled) from before a loop.
    __device__ __forceinline__ void fresh() {
      asm volatile("" : "+v"(row));
#pragma unroll
      for (int e = 0; e < kCols; ++e) asm volatile("" : "+v"(col[e]));
    }
  };
  static __device__ __forceinline__ Lane lane_of(int lane) {
    Lane o;
    const int h = lane >> 5;
    if constexpr (kElt == 2) {
      o.row = at(lane & 31, h);
      const int i = lane & 15, chunk = 2 * ((lane >> 4) & 1) + ((i & 3) >> 1);
      o.col[0] = at(4 * h + (i >> 2), chunk) + 8 * (i & 1);
      o.col[1] = at(4 * h + (i >> 2) + 8, chunk) + 8 * (i & 1);
    } else {
      o.row = at(lane & 31, 2 * h);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        o.col[e] = at(4 * h + (e & 3) + 8 * (e >> 2), (lane & 31) / kPer) + (lane % kPer) * 4;
    }
    return o;
  }
  // Row fragment: rows r0 + lane % 32 (r0 a multiple of 32), elements 16 s + 8 (lane / 32) + 0..7.
  static __device__ __forceinline__ frag row(const unsigned char* lds, int r0, int s, const Lane& o) {
    if constexpr (kElt == 2) {
      return read_lds<frag>(lds + r0 * kPitch + (o.row ^ (s << 5)));
    } else {
      typedef float f4 __attribute__((ext_vector_type(4)));
      const f4 a = read_lds<f4>(lds + r0 * kPitch + (o.row ^ (s << 6)));
      const f4 b = read_lds<f4>(lds + r0 * kPitch + (o.row ^ (s << 6) ^ 16));
      return frag{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    }
  }
  // Transposed fragment: column 32 b + lane % 32, at the rows that the
  // accumulator registers 8 s .. 8 s + 7 of a 32-row block stand for:
  // r0 + 16 s + 4 (lane / 32) + 0..3 and those + 8.
  static __device__ __forceinline__ frag col(const unsigned char* lds, int r0, int s, int b, const Lane& o) {
    const unsigned char* const from = lds + (r0 + 16 * s) * kPitch;
    if constexpr (kElt == 2) {
      union {
        s16x4 half[2];
        frag f;
      } u;
      u.half[0] = read_tr((lds_s16x4*)(from + (o.col[0] ^ (b << 6))));
      u.half[1] = read_tr((lds_s16x4*)(from + (o.col[1] ^ (b << 6))));
      return u.f;
    } else {
      frag f;
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = read_lds<float>(from + (o.col[e] ^ (b << 7)));
      return f;
    }
  }
};

// Row fragment straight from memory: elements 16 s + 8 (lane / 32) + 0..7 of
// the lane's row, zeros past dim.
template <class E>
__device__ __forceinline__ typename AttnType<E>::frag row_from(const E* p, bool on, int s, int dim, int lane) {
  typedef typename AttnType<E>::frag frag;
  const int d = 16 * s + 8 * (lane >> 5);
  frag f;
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = E(0.f);
  if (on && d < dim) f = *reinterpret_cast<const frag*>(p + d);
  return f;
}

template <class E>
__device__ __forceinline__ typename AttnType<E>::frag pack_frag8(const f32x16& a, int s) {
  typename AttnType<E>::frag f;
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = static_cast<E>(a[8 * s + e]);
  return f;
}

// The value of lane ^ 32 and its own, as (lower half's, upper half's).
__device__ __forceinline__ float2 both_halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return make_float2(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// N products in order, the fragments of each read from LDS `AHEAD` products
// before it: load(i, f) and use(i, f). The scheduling barriers hold the order,
// which the compiler's own schedule gives up for fewer registers (every product
// then waits for its own reads).
template <int N, int AHEAD, class Frags, class Load, class Use>
__device__ __forceinline__ void products(const Load& load, const Use& use) {
  constexpr int kSlots = AHEAD < N ? AHEAD : N;
  Frags f[kSlots];
#pragma unroll
  for (int i = 0; i < kSlots; ++i) load(i, f[i]);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    use(i, f[i % kSlots]);
    if (i + kSlots < N) load(i + kSlots, f[i % kSlots]);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// A sequence of the packed batch. Offsets and lengths from the device are
// clamped to the tensors, so that no table can lead outside them.
struct Seq {
  int q0, lq, k0, lk;
};
__device__ __forceinline__ int clamp_to(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }
__device__ __forceinline__ Seq sequence(const AttnArgs& a, int b) {
  Seq s;
  s.q0 = a.cu_q ? clamp_to(a.cu_q[b], 0, a.nq) : 0;
  s.lq = (a.cu_q ? clamp_to(a.cu_q[b + 1], s.q0, a.nq) : a.nq) - s.q0;
  s.k0 = a.cu_k ? clamp_to(a.cu_k[b], 0, a.nk) : 0;
  s.lk = (a.cu_k ? clamp_to(a.cu_k[b + 1], s.k0, a.nk) : a.nk) - s.k0;
  if (a.k_len) s.lk = clamp_to(a.k_len[b], 0, s.lk);
  return s;
}

// Tiles of `size` units over sequences whose starts, in units, are mul * cu[b]:
// sequence b has the tile numbers from floor(mul cu[b] / size) + b to the next
// sequence's first, at least as many as it needs whatever the lengths, and the
// launch covers floor(mul total / size) + batch. No length is needed on the
// host, and no table is built. Returns the sequence of tile `t` and the tile's
// number inside it; one load per lane and level, 64 sequences a level.
__device__ __forceinline__ int first_tile(const int32_t* cu, int b, int mul, int size) {
  return int(uint32_t(cu[b]) * uint32_t(mul) / uint32_t(size)) + b;  // cu * mul < 2^31 (checked by the caller)
}
__device__ __forceinline__ int find_sequence(const int32_t* cu, int batch, int mul, int size, int t,
                                             int* inside) {
  if (cu == nullptr || batch == 1) {
    *inside = t - (cu ? first_tile(cu, 0, mul, size) : 0);
    return 0;
  }
  const int lane = threadIdx.x & 63;
  int lo = 0, n = batch;
  while (n > 1) {
    const int step = (n + 63) / 64;
    const int b = lo + lane * step;
    const bool le = lane * step < n && first_tile(cu, b, mul, size) <= t;
    const int c = __popcll(__ballot(le));
    const int at = (c > 0 ? c - 1 : 0) * step;
    lo += at;
    n = n - at < step ? n - at : step;
  }
  lo = __builtin_amdgcn_readfirstlane(lo);
  *inside = t - first_tile(cu, lo, mul, size);
  return lo;
}
inline int64_t tiles_of(int64_t total, int batch, int64_t mul, int size) { return total * mul / size + batch; }

// The key tiles (of KT keys, aligned to KT inside the sequence) that rows at
// positions p0 .. p1 see: first those of the sinks, then the band's.
struct KeyTiles {
  int sink, band, n;  // tiles of the sinks; first tile of the band; tiles in all
  __device__ __forceinline__ int at(int i) const { return i < sink ? i : band + i - sink; }
};
template <int KT>
__device__ __forceinline__ KeyTiles key_tiles(int left, int right, int most_sinks, int p0, int p1, int lk) {
  KeyTiles t;
  const int hi = min(lk, p1 + right + 1);  // positions and sides are within 2^30 each
  if (hi <= 0) {
    t.sink = t.band = t.n = 0;
    return t;
  }
  const int lo = max(0, p0 - left);
  const int sinks = min(most_sinks, min(lo, hi));
  t.sink = (sinks + KT - 1) / KT;
  t.band = max(lo / KT, t.sink);
  const int end = (hi + KT - 1) / KT;
  t.n = t.sink + max(0, end - t.band);
  return t;
}
template <int KT>
__device__ __forceinline__ KeyTiles key_tiles(const AttnArgs& a, int p0, int p1, int lk) {
  return key_tiles<KT>(a.left, a.right, a.sinks, p0, p1, lk);
}

// ---------------------------------------------------------------------------
// Non-finite elements that a row does not see. A weight of zero times such an
// element is NaN in the products that sum over keys (or rows), so where a
// result of a wave is not finite, the wave walks again: scores by products from
// memory, which keep what is not finite to its own key and row, and sums key by
// key in vector instructions, each lane adding only what it sees. No cost where
// all is finite but one check of the result. Where something is not, the waves
// that it reaches take 10 to 30 times their time (32,768 tokens, 16 heads of 128
// over 4, 4096 keys back, NaN in a sink's value, which all rows see: forward 32
// ms, gradient 132; a row or key at a time by a whole wave took 500 times).
// ---------------------------------------------------------------------------
template <int NB>
__device__ __forceinline__ float zero_if_finite(const f32x16 (&acc)[NB]) {  // NaN if any element is not finite
  float t = 0.f;
#pragma unroll
  for (int d = 0; d < NB; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) t = fmaf(acc[d][e], 0.f, t);
  return t;
}
// Lanes l and l + 32 hold the same row: bit l of the result.
__device__ __forceinline__ uint32_t bad_rows(float t) {
  const uint64_t m = __ballot(t != t);
  return uint32_t(m) | uint32_t(m >> 32);
}
// Scores of 32 rows of `a` (this lane's: pa, if on) against the fragments b: rows down, columns across.
template <class E, int ST>
__device__ __forceinline__ f32x16 scores_from(const E* pa, bool on, const typename AttnType<E>::frag (&b)[ST], int dim,
                                              int lane) {
  f32x16 s;
#pragma unroll
  for (int e = 0; e < 16; ++e) s[e] = 0.f;
#pragma unroll
  for (int st = 0; st < ST; ++st) s = AttnType<E>::mma(row_from<E>(pa, on, st, dim, lane), b[st], s);
  return s;
}
// 32 x 32 factors to the wave's own LDS, row by row, and one of them back as every row's of this lane's column.
__device__ __forceinline__ void put_factors(float* lds, const f32x16& s, int lane) {
#pragma unroll
  for (int e = 0; e < 16; ++e) lds[(8 * (e >> 2) + 4 * (lane >> 5) + (e & 3)) * 32 + (lane & 31)] = s[e];
}
__device__ __forceinline__ void wave_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }
// acc += factor i * row(i) for the 32 rows i of which sees(i), blocks d0 .. d0 + DN of 32 elements: the factors in
// LDS as put_factors laid them; row(i) can be read whether seen or not, and the next is on its way meanwhile.
template <class E, int DN, int NB, class Row, class Sees>
__device__ __forceinline__ void add_rows(f32x16 (&acc)[NB], const float* lds, const Row& row, const Sees& sees, int d0,
                                         int dim, int lane) {
  typedef E elt4 __attribute__((ext_vector_type(4)));
  elt4 x[2][DN][4];
  auto load = [&](int i, elt4 (&to)[DN][4]) {
    const E* from = row(i);
#pragma unroll
    for (int d = 0; d < DN; ++d)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int col = 32 * (d0 + d) + 8 * g + 4 * (lane >> 5);
        if (col < dim) to[d][g] = *reinterpret_cast<const elt4*>(from + col);
      }
  };
  load(0, x[0]);
  for (int i = 0; i < 32; i += 2) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      if (i + b + 1 < 32) load(i + b + 1, x[b ^ 1]);
      if (!sees(i + b)) continue;
      const float w = lds[(i + b) * 32 + (lane & 31)];
#pragma unroll
      for (int d = 0; d < DN; ++d)
#pragma unroll
        for (int g = 0; g < 4; ++g)  // columns past dim: not stored
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[d][4 * g + e] = fmaf(w, static_cast<float>(x[b][d][g][e]), acc[d][4 * g + e]);
    }
  }
}

}  // namespace trsc
