// Typed access to rows that may start on any element: rows of an odd number
// of 16-bit elements do.  gfx950 serves 16-byte global accesses at any
// address, so a lane always moves whole vectors and only the last, partial
// vector of a row goes element by element.
#pragma once

#include "common.hpp"

namespace rar {

typedef u32x4 u32x4_any __attribute__((aligned(2)));

__device__ __forceinline__ u32x4 ld16_any(const char* p) { return *(const u32x4_any*)p; }
template <bool NT>
__device__ __forceinline__ void st16_any(char* p, u32x4 v) {
  if constexpr (NT) __builtin_nontemporal_store(v, (u32x4_any*)p);
  else *(u32x4_any*)p = v;
}

// Eight consecutive elements as binary32.
template <int DT>
__device__ __forceinline__ G8 load8_any(const char* base, uint64_t elem) {
  const char* p = base + elem * DtypeSize<DT>::value;
  Raw8<DT> r;
  r.w[0] = ld16_any(p);
  if constexpr (DT == DT_F32) r.w[1] = ld16_any(p + 16);
  return unpack8<DT>(r);
}
template <int DT, bool NT>
__device__ __forceinline__ void store8_any(char* base, uint64_t elem, const G8& g) {
  char* p = base + elem * DtypeSize<DT>::value;
  const Raw8<DT> r = pack8<DT>(g);
  st16_any<NT>(p, r.w[0]);
  if constexpr (DT == DT_F32) st16_any<NT>(p + 16, r.w[1]);
}

// The same for the first n <= 8 elements (missing ones read as +0).
template <int DT>
__device__ __forceinline__ G8 load8_upto(const char* base, uint64_t elem, int n) {
  return n >= 8 ? load8_any<DT>(base, elem) : load_part8<DT>(base, elem, n);
}
template <int DT, bool NT>
__device__ __forceinline__ void store8_upto(char* base, uint64_t elem, int n, const G8& g) {
  if (n >= 8) store8_any<DT, NT>(base, elem, g);
  else store_part8<DT>(base, elem, n, g);
}

// One element of a type known at run time (uniform over the launch).
__device__ __forceinline__ float load_elem_dt(const char* base, uint64_t i, int dt) {
  if (dt == DT_F32) return load_elem<DT_F32>(base, i);
  return dt == DT_F16 ? load_elem<DT_F16>(base, i) : load_elem<DT_BF16>(base, i);
}
__device__ __forceinline__ void store_elem_dt(char* base, uint64_t i, int dt, float x) {
  if (dt == DT_F32) store_elem<DT_F32>(base, i, x);
  else if (dt == DT_F16) store_elem<DT_F16>(base, i, x);
  else store_elem<DT_BF16>(base, i, x);
}

// Sums over the 64 lanes of a wavefront; every lane receives the result.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

}  // namespace rar
