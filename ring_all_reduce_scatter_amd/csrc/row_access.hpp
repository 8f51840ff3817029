// Typed access to rows that may start on any element: rows of an odd number
// of 16-bit elements do.  gfx950 serves 8- and 16-byte global accesses at
// any address, so a lane always moves whole vectors and only the last,
// partial vector of a row goes element by element.
//
// A lane's vector is E consecutive elements: 8 when every type involved has
// 16 bits, 4 as soon as one is binary32, so that each load or store
// instruction of a wavefront covers one contiguous range in both types.
// (Eight binary32 elements a lane would be two instructions that each touch
// every other 16 bytes: streaming stores then reach memory as half lines.)
#pragma once

#include "common.hpp"

namespace rar {

typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));

template <int A, int B>
constexpr int vec_elems() {
  return A == DT_F32 || B == DT_F32 ? 4 : 8;
}

template <int E>
struct VecF {
  float v[E];
};

// A vector as stored: E elements of type DT.
template <int DT, int E>
struct VecRaw {
  static constexpr int W = E * DtypeSize<DT>::value / 4;
  static_assert(W == 2 || W == 4, "8 or 16 bytes");
  uint32_t w[W];
};

// NT: a streaming (nontemporal) load, for data that the launch reads once.
template <int DT, int E, bool NT = false>
__device__ __forceinline__ VecRaw<DT, E> load_raw(const char* base, uint64_t elem) {
  const char* p = base + elem * DtypeSize<DT>::value;
  VecRaw<DT, E> r;
  if constexpr (VecRaw<DT, E>::W == 4) {
    u32x4 x;
    if constexpr (NT) x = __builtin_nontemporal_load((const u32x4_any*)p);
    else x = *(const u32x4_any*)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = x[i];
  } else {
    u32x2 x;
    if constexpr (NT) x = __builtin_nontemporal_load((const u32x2_any*)p);
    else x = *(const u32x2_any*)p;
    r.w[0] = x[0];
    r.w[1] = x[1];
  }
  return r;
}

template <int DT, int E>
__device__ __forceinline__ VecF<E> unpack(const VecRaw<DT, E>& r) {
  VecF<E> f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    if constexpr (DT == DT_F32) f.v[i] = __uint_as_float(r.w[i]);
    else f.v[i] = widen16<DT>(i & 1 ? r.w[i / 2] >> 16 : r.w[i / 2] & 0xffffu);
  }
  return f;
}

template <int DT, int E>
__device__ __forceinline__ VecF<E> load_vec(const char* base, uint64_t elem) {
  return unpack<DT, E>(load_raw<DT, E>(base, elem));
}

// Four binary32 or eight 16-bit elements as stored.
template <int DT, int E>
__device__ __forceinline__ u32x4 pack_vec(const VecF<E>& f) {
  static_assert(E * DtypeSize<DT>::value == 16, "16 bytes");
  u32x4 x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == DT_F32) x[i] = __float_as_uint(f.v[i]);
    else x[i] = pack_pair<DT>(f.v[2 * i], f.v[2 * i + 1]);
  }
  return x;
}

template <int DT>
__device__ __forceinline__ u32x2 pack_vec_half(const VecF<4>& f) {
  return (u32x2){pack_pair<DT>(f.v[0], f.v[1]), pack_pair<DT>(f.v[2], f.v[3])};
}

// Streaming stores (nontemporal): an output that is not read back soon.
template <int DT, int E>
__device__ __forceinline__ void store_vec(char* base, uint64_t elem, const VecF<E>& f) {
  char* p = base + elem * DtypeSize<DT>::value;
  if constexpr (VecRaw<DT, E>::W == 4) __builtin_nontemporal_store(pack_vec<DT, E>(f), (u32x4_any*)p);
  else __builtin_nontemporal_store(pack_vec_half<DT>(f), (u32x2_any*)p);
}
// The same write-through (st16_wt), off bytes into a range; both must be
// multiples of the vector's size.
template <int DT, int E>
__device__ __forceinline__ void store_vec_wt(WtRange range, uint32_t off, const VecF<E>& f) {
  if constexpr (VecRaw<DT, E>::W == 4) st16_wt(range, off, pack_vec<DT, E>(f));
  else st8_wt(range, off, pack_vec_half<DT>(f));
}

// The same for the first n elements; missing ones read as +0.
template <int DT, int E>
__device__ __forceinline__ VecF<E> load_vec_upto(const char* base, uint64_t elem, int n) {
  if (n >= E) return load_vec<DT, E>(base, elem);
  VecF<E> f;
#pragma unroll
  for (int i = 0; i < E; ++i) f.v[i] = i < n ? load_elem<DT>(base, elem + i) : 0.0f;
  return f;
}
template <int DT, int E>
__device__ __forceinline__ void store_vec_upto(char* base, uint64_t elem, int n, const VecF<E>& f) {
  if (n >= E) {
    store_vec<DT, E>(base, elem, f);
    return;
  }
#pragma unroll
  for (int i = 0; i < E; ++i)
    if (i < n) store_elem<DT>(base, elem + i, f.v[i]);
}

// Elements of [col, dim) in a vector of E, for any col.
template <int E>
__device__ __forceinline__ int vec_count(uint64_t dim, uint64_t col) {
  return col >= dim ? 0 : (dim - col < (uint64_t)E ? (int)(dim - col) : E);
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

// This wavefront's stores have been acknowledged.
__device__ __forceinline__ void stores_done() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
}

// Sums over a DPP row of 16 lanes, and over the 64 lanes of a wavefront (all
// active); every lane receives its own.  The four rows of a wavefront are
// joined by scalar reads.
template <int CTRL>
__device__ __forceinline__ float dpp_f32(float v) {
  return __uint_as_float(dpp_u32<CTRL>(__float_as_uint(v)));
}
__device__ __forceinline__ float lane_f32(float v, int lane) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
}
__device__ __forceinline__ float dpp_row_sum(float v) {
  v += dpp_f32<kDppQuad1032>(v);
  v += dpp_f32<kDppQuad2301>(v);
  v += dpp_f32<kDppRowHalfMirror>(v);
  v += dpp_f32<kDppRowMirror>(v);
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
  v = dpp_row_sum(v);
  return (lane_f32(v, 0) + lane_f32(v, 16)) + (lane_f32(v, 32) + lane_f32(v, 48));
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

}  // namespace rar
