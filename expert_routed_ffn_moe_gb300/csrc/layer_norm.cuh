// The layer norm's chunks of neighbouring columns: 8 where rows are aligned, else one.
#pragma once

#include "ops_internal.h"
#include "rows_common.cuh"

namespace moe {

template <typename T, int VEC>
struct Chunk;
template <typename T>
struct Chunk<T, 1> {
  T v;
  MOE_DEV void zero() { put(&v, 0.f); }
  MOE_DEV void load(const T* p) { v = *p; }
  MOE_DEV float get(int) const { return to_f(v); }
  static MOE_DEV void store(T* p, const float (&f)[1]) { put(p, f[0]); }
};
template <typename T>
struct Chunk<T, 8> {
  Raw<T> r;
  MOE_DEV void zero() { r.zero(); }
  MOE_DEV void load(const T* p) { r.load(p); }
  MOE_DEV float get(int i) const { return r.get().v[i]; }
  static MOE_DEV void store(T* p, const float (&f)[8]) {
    store8(p, F8{{f[0], f[1], f[2], f[3], f[4], f[5], f[6], f[7]}});
  }
};
// Columns c .. c + VEC - 1 of weight or bias; `otherwise` without one.
template <int VEC>
MOE_DEV void load_param(float (&f)[VEC], const void* p, int dtype, int c, float otherwise) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = otherwise;
  } else if (dtype == MOE_BF16) {
    Chunk<__nv_bfloat16, VEC> t;
    t.load(static_cast<const __nv_bfloat16*>(p) + c);
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = t.get(i);
  } else {
    Chunk<float, VEC> t;
    t.load(static_cast<const float*>(p) + c);
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = t.get(i);
  }
}

}  // namespace moe
