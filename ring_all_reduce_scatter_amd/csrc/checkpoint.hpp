// Activation checkpoints in 8 bits: the library's block floating point
// (bfp_scale, bfp_q in common.hpp) over the rows of a matrix, in blocks of 32
// columns.
//
//   E = max |x| >> 23 as binary32 bits,  e = max(E, 1) - 127,  k = 6 - e
//   q = clamp(rne(x 2^k), +-127),  value = q 2^-k;  E = 255: NaN, q = 0
//
// The scale is a power of two, so x 2^k and q 2^-k are exact and a checkpoint
// holds the same bytes whichever kernel writes it.  Blocks are as short as
// that because activations have single columns far above their neighbours,
// which cost a block its bits; the exponents take 1/32 of the codes' bytes.
//
// Layout of rows x dim with nb = ceil(dim / 32) blocks a row: the codes, 32 nb
// bytes a row (zeros past dim), then the exponents, nb bytes a row.  Rows of
// codes begin on 32 bytes at any dim, so codes move in whole vectors where
// the matrix itself cannot.
#pragma once

#include <algorithm>

#include "row_access.hpp"

namespace rar {

constexpr uint32_t kCkptBlock = 32;

struct Checkpoint {
  uint8_t* codes;
  uint8_t* exps;
  uint64_t nb;
  __host__ __device__ Checkpoint() : codes(nullptr), exps(nullptr), nb(0) {}
  __host__ __device__ Checkpoint(void* p, uint64_t rows, uint64_t dim)
      : codes((uint8_t*)p), exps((uint8_t*)p + rows * ((dim + 31) / 32 * 32)), nb((dim + 31) / 32) {}
  __device__ __forceinline__ uint8_t* code_row(uint64_t r) const { return codes + r * nb * kCkptBlock; }
  __device__ __forceinline__ uint8_t* exp_row(uint64_t r) const { return exps + r * nb; }
};

// 2^-k, NaN for E = 255: every value of a block is its code times this, exactly
// (the least step, 2^-132, is a subnormal that binary32 still holds).
__device__ __forceinline__ float ckpt_step(uint32_t E) {
  const float s = __builtin_amdgcn_ldexpf(1.0f, (int)(E < 1 ? 1 : E) - 133);
  return E == 255 ? __builtin_nanf("") : s;
}

// How a block of largest bits m is encoded.  Adding 1.5 * 2^23 to x 2^k in one
// fused step rounds to a whole number, to even on ties, and leaves it in the
// sum's low bits; values that would round to 128 are held at 127 before that.
// Nine instructions for two values then become five.  2^k passes binary32 for
// the smallest exponents, which go the plain way.
struct CkptScale {
  float s, most;  // 2^k, 127 * 2^-k
  BfpScale plain;
  bool tiny;
};
__device__ __forceinline__ CkptScale ckpt_scale(uint32_t m) {
  CkptScale c;
  c.plain = bfp_scale(m, 8);
  c.tiny = c.plain.k > 127;
  c.s = __builtin_amdgcn_ldexpf(1.0f, c.plain.k);
  c.most = __builtin_amdgcn_ldexpf(127.0f, -c.plain.k);
  return c;
}

// Four codes of a block, packed.
__device__ __forceinline__ uint32_t ckpt_encode4(const float* x, const CkptScale& c) {
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    q[i] = __float_as_uint(__builtin_fmaf(__builtin_amdgcn_fmed3f(x[i], -c.most, c.most), c.s, 12582912.0f));
  if (c.tiny) {
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = (uint32_t)(int)bfp_q(x[i], c.plain.k, 127.0f);
  }
  const uint32_t lo = __builtin_amdgcn_perm(q[1], q[0], 0x0c0c0400), hi = __builtin_amdgcn_perm(q[3], q[2], 0x04000c0c);
  return c.plain.nan ? 0 : lo | hi;
}
__device__ __forceinline__ float ckpt_code(uint32_t w, int i) { return (float)(int8_t)(w >> (8 * i)); }

template <int E>
__device__ __forceinline__ uint32_t vec_absmax(const VecF<E>& x) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < E; ++i) m = max(m, absbits(x.v[i]));
  return m;
}

// A vector of E codes as stored, with its block's exponent.
template <int E>
struct CkptRaw {
  uint32_t w[E / 4];
  uint32_t e;
};
template <int E>
__device__ __forceinline__ CkptRaw<E> ckpt_load(const uint8_t* codes, const uint8_t* exps, uint32_t col) {
  static_assert(E == 4 || E == 8, "");
  CkptRaw<E> r;
  if constexpr (E == 8) {
    const u32x2 x = __builtin_nontemporal_load((const u32x2*)(codes + col));
    r.w[0] = x[0];
    r.w[1] = x[1];
  } else {
    r.w[0] = __builtin_nontemporal_load((const uint32_t*)(codes + col));
  }
  r.e = exps[col / kCkptBlock];
  return r;
}
template <int E>
__device__ __forceinline__ VecF<E> ckpt_unpack(const CkptRaw<E>& r) {
  VecF<E> f;
  const float step = ckpt_step(r.e);
#pragma unroll
  for (int i = 0; i < E; ++i) f.v[i] = ckpt_code(r.w[i / 4], i % 4) * step;
  return f;
}
__device__ __forceinline__ float ckpt_elem(const uint8_t* codes, const uint8_t* exps, uint64_t col) {
  return (float)(int8_t)codes[col] * ckpt_step(exps[col / kCkptBlock]);
}

// Stores a lane's E values as codes, and by the first lane of each block its
// exponent.  m: the block's largest absolute bits, over the 32 / E lanes that
// hold it.
template <int E>
__device__ __forceinline__ void ckpt_store(uint8_t* codes, uint8_t* exps, uint32_t col, uint32_t m,
                                           const VecF<E>& x) {
  const CkptScale sc = ckpt_scale(m);
  if constexpr (E == 8)
    __builtin_nontemporal_store((u32x2){ckpt_encode4(x.v, sc), ckpt_encode4(x.v + 4, sc)}, (u32x2*)(codes + col));
  else
    __builtin_nontemporal_store(ckpt_encode4(x.v, sc), (uint32_t*)(codes + col));
  if (col % kCkptBlock == 0) exps[col / kCkptBlock] = (uint8_t)(m >> 23);
}

// n / d for n < 2^31: with s = ceil(log2 d) and m = ceil(2^(31 + s) / d) the
// quotient is n m >> (31 + s).
struct FastDiv {
  uint32_t m, s, d;
  explicit FastDiv(uint32_t by) : s(0), d(by) {
    while (((uint64_t)1 << s) < by) ++s;
    m = (uint32_t)((((uint64_t)1 << (31 + s)) + by - 1) / by);
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (uint32_t)((uint64_t)n * m >> (31 + s)); }
};

// A walk over blocks of rows, U vectors of E elements a lane: where its k-th
// vector lies.  Block numbers of a launch stay within 31 bits.
struct CkptPlace {
  uint32_t block, row, col;
  bool live;
};
template <int E, int U>
__device__ __forceinline__ CkptPlace ckpt_place(uint32_t k, uint32_t blocks, const FastDiv& nb) {
  constexpr uint32_t LB = kCkptBlock / E;  // lanes a block
  CkptPlace p;
  p.block = (blockIdx.x * U + k) * (kThreads / LB) + threadIdx.x / LB;
  p.live = p.block < blocks;
  p.row = nb.div(p.block);
  p.col = (p.block - p.row * nb.d) * kCkptBlock + threadIdx.x % LB * E;
  return p;
}

// Calls f with the first row, the rows and the grid of each launch.
template <int E, int U, class F>
hipError_t by_ckpt_rows(uint64_t rows, uint64_t nb, F f) {
  const uint64_t per = std::max<uint64_t>(1, ((uint64_t)1 << 30) / nb);
  for (uint64_t r = 0; r < rows; r += per) {
    const uint64_t n = std::min(per, rows - r), wg = U * kThreads / (kCkptBlock / E);
    const hipError_t e = f(r, (uint32_t)(n * nb), dim3((unsigned)((n * nb + wg - 1) / wg)));
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace rar
