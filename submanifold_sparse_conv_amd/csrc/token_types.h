// Element types of the token operators: 16-byte chunk loads and stores as
// floats. Arithmetic is fp32; a store rounds once, to nearest even.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

namespace trsc {

struct TF32 {
  typedef float elt;
};
struct TBF16 {
  typedef __bf16 elt;
};
struct TF16 {
  typedef _Float16 elt;
};

// E consecutive elements (E * sizeof(elt) a multiple of 8 bytes, aligned to
// 16 bytes where that large) as raw words, and their values.
template <class T, int E>
struct Chunk {
  typedef typename T::elt elt;
  typedef elt vec __attribute__((ext_vector_type(E)));
  vec v;
  __device__ __forceinline__ void load(const elt* p) { v = *reinterpret_cast<const vec*>(p); }
  __device__ __forceinline__ float get(int i) const { return static_cast<float>(v[i]); }
  __device__ __forceinline__ void set(int i, float f) { v[i] = static_cast<elt>(f); }
  __device__ __forceinline__ void store(elt* p) const { *reinterpret_cast<vec*>(p) = v; }
};

}  // namespace trsc
