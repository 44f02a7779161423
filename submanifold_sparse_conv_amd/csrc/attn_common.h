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

template <class E>
struct AttnType;
template <>
struct AttnType<__bf16> {
  typedef __bf16 elt;
  typedef __bf16 frag __attribute__((ext_vector_type(8)));
  static constexpr bool wide = false;
  static __device__ __forceinline__ f32x16 mma(frag a, frag b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
};
template <>
struct AttnType<_Float16> {
  typedef _Float16 elt;
  typedef _Float16 frag __attribute__((ext_vector_type(8)));
  static constexpr bool wide = false;
  static __device__ __forceinline__ f32x16 mma(frag a, frag b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
};
template <>
struct AttnType<float> {
  typedef float elt;
  typedef float frag __attribute__((ext_vector_type(8)));
  static constexpr bool wide = true;
  static __device__ __forceinline__ f32x16 mma(frag a, frag b, f32x16 c) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i], b[i], c, 0, 0, 0);
    return c;
  }
};

// 16 bytes that stand for what lies past a sequence's end or a head's width.
__device__ __attribute__((aligned(16))) const uint32_t g_attn_zeros[4] = {0, 0, 0, 0};

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

  // Rows [0, ROWS) of the tile from tokens t0 + row (zeros from token `end`
  // on, and past `dim`): copies first, first + step, ... of ROWS / kRowsPerCopy.
  template <int ROWS, int STEP>
  static __device__ __forceinline__ void copy(unsigned char* lds, const E* base, int64_t stride, int t0, int end,
                                              int dim, int first, int lane) {
#pragma unroll
    for (int j = 0; j < ROWS / kRowsPerCopy; j += STEP) {
      const int n = j + first;
      const int row = n * kRowsPerCopy + lane / kChunks;
      const int chunk = (lane % kChunks) ^ key(row);
      const int t = t0 + row;
      const bool in = t < end && chunk * kPer < dim;
      const void* g = in ? static_cast<const void*>(base + int64_t(t) * stride + chunk * kPer)
                         : static_cast<const void*>(g_attn_zeros);
      copy16_to_lds(g, lds + n * 1024);
    }
  }
  // Row fragment: rows r0 + lane % 32, elements 16 s + 8 (lane / 32) + 0..7.
  static __device__ __forceinline__ frag row(const unsigned char* lds, int r0, int s, int lane) {
    const int r = r0 + (lane & 31), h = lane >> 5;
    if constexpr (kElt == 2) {
      return *reinterpret_cast<const frag*>(lds + at(r, 2 * s + h));
    } else {
      typedef float f4 __attribute__((ext_vector_type(4)));
      const f4 a = *reinterpret_cast<const f4*>(lds + at(r, 4 * s + 2 * h));
      const f4 b = *reinterpret_cast<const f4*>(lds + at(r, 4 * s + 2 * h + 1));
      return frag{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    }
  }
  // Transposed fragment: column 32 b + lane % 32, at the rows that the
  // accumulator registers 8 s .. 8 s + 7 of a 32-row block stand for:
  // r0 + 16 s + 4 (lane / 32) + 0..3 and those + 8.
  static __device__ __forceinline__ frag col(const unsigned char* lds, int r0, int s, int b, int lane) {
    const int h = lane >> 5;
    if constexpr (kElt == 2) {
      const int i = lane & 15;
      const int r = r0 + 16 * s + 4 * h + (i >> 2);
      const int chunk = 4 * b + 2 * ((lane >> 4) & 1) + ((i & 3) >> 1);
      typedef __attribute__((address_space(3))) s16x4* lptr;
      union {
        s16x4 half[2];
        frag f;
      } u;
      u.half[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lptr)(lds + at(r, chunk) + 8 * (i & 1)));
      u.half[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lptr)(lds + at(r + 8, chunk) + 8 * (i & 1)));
      return u.f;
    } else {
      const int d = 32 * b + (lane & 31);
      frag f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int r = r0 + 16 * s + 4 * h + (e & 3) + (e >> 2) * 8;
        f[e] = *reinterpret_cast<const float*>(lds + at(r, d / kPer) + (d % kPer) * 4);
      }
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
__device__ __forceinline__ KeyTiles key_tiles(const AttnArgs& a, int p0, int p1, int lk) {
  KeyTiles t;
  const int hi = min(lk, p1 + a.right + 1);  // positions and sides are within 2^30 each
  if (hi <= 0) {
    t.sink = t.band = t.n = 0;
    return t;
  }
  const int lo = max(0, p0 - a.left);
  const int sinks = min(a.sinks, min(lo, hi));
  t.sink = (sinks + KT - 1) / KT;
  t.band = max(lo / KT, t.sink);
  const int end = (hi + KT - 1) / KT;
  t.n = t.sink + max(0, end - t.band);
  return t;
}

// ---------------------------------------------------------------------------
// Non-finite elements that a row does not see. A weight of zero times such an
// element is NaN in the matrix products, so a result that is not finite is
// computed again, one row (or key) at a time by a whole wave that only touches
// what is seen; lane l has the elements 2 l and 2 l + 1. No cost where all is
// finite but one check of the result.
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
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
template <class E>
__device__ __forceinline__ float2 pair_of(const E* row, int dim, int lane) {
  return 2 * lane < dim ? make_float2(float(row[2 * lane]), float(row[2 * lane + 1])) : make_float2(0.f, 0.f);
}
__device__ __forceinline__ bool sees_key(const AttnArgs& a, int p, int j, int lk) {
  return j < lk && j <= p + a.right && (j >= p - a.left || j < a.sinks);
}

}  // namespace trsc
