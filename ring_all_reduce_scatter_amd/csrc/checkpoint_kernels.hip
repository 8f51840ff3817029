// Packing and unpacking of 8-bit activation checkpoints (checkpoint.hpp) for
// gfx950.  Both are one pass over memory and bound by it.
//
// The codes of a checkpoint are one flat array of 32-byte blocks, so lanes are
// dealt out over blocks, not rows: 4 lanes of 8 elements, or 8 lanes of 4 in
// binary32, take a block, and rows of any length fill every wavefront.  Only
// the matrix's address needs the row (one multiplication by a reciprocal that
// the host prepares).  16,384 x 4096 bfloat16, inputs cold: 34.5 us packing and
// 35 unpacking (203 MB, 5.8 TB/s); 67 x 1001 binary32 3.2 us each, latency.
#include <algorithm>

#include "checkpoint.hpp"
#include "operator_launch.hpp"

namespace rar {
namespace {

constexpr int kUnroll = 4;  // vectors a lane has in flight
template <int DT>
__global__ __launch_bounds__(kThreads) void ckpt_pack_kernel(Rows x, uint64_t dim, FastDiv nb, uint32_t blocks,
                                                              uint8_t* __restrict__ codes, uint8_t* __restrict__ exps) {
  constexpr int E = vec_elems<DT, DT>(), ES = DtypeSize<DT>::value;
  CkptPlace p[kUnroll];
  VecF<E> v[kUnroll];
#pragma unroll
  for (int k = 0; k < kUnroll; ++k) {
    p[k] = ckpt_place<E, kUnroll>(k, blocks, nb);
    v[k] = {};
    if (p[k].live) {
      const char* row = x.p + p[k].row * x.stride * ES;
      const int n = vec_count<E>(dim, p[k].col);
      if (n == E) v[k] = unpack<DT, E>(load_raw<DT, E, true>(row, p[k].col));
      else v[k] = load_vec_upto<DT, E>(row, p[k].col, n);
    }
  }
#pragma unroll
  for (int k = 0; k < kUnroll; ++k) {
    const uint32_t m = group_max_u32<kCkptBlock / E>(vec_absmax(v[k]));
    if (p[k].live)
      ckpt_store<E>(codes + (uint64_t)p[k].block * kCkptBlock, exps + p[k].block,
                    threadIdx.x % (kCkptBlock / E) * E, m, v[k]);
  }
}

template <int DT>
__global__ __launch_bounds__(kThreads) void ckpt_unpack_kernel(const uint8_t* __restrict__ codes,
                                                                const uint8_t* __restrict__ exps, FastDiv nb,
                                                                uint32_t blocks, Rows out, uint64_t dim) {
  constexpr int E = vec_elems<DT, DT>(), ES = DtypeSize<DT>::value;
  CkptPlace p[kUnroll];
  CkptRaw<E> raw[kUnroll];
#pragma unroll
  for (int k = 0; k < kUnroll; ++k) {
    p[k] = ckpt_place<E, kUnroll>(k, blocks, nb);
    raw[k] = {};
    if (p[k].live)
      raw[k] = ckpt_load<E>(codes + (uint64_t)p[k].block * kCkptBlock, exps + p[k].block,
                            threadIdx.x % (kCkptBlock / E) * E);
  }
#pragma unroll
  for (int k = 0; k < kUnroll; ++k)
    if (p[k].live)
      store_vec_upto<DT, E>(out.p + p[k].row * out.stride * ES, p[k].col, vec_count<E>(dim, p[k].col),
                            ckpt_unpack<E>(raw[k]));
}

template <int DT>
hipError_t pack_dt(const Rows& x, uint64_t rows, uint64_t dim, const Checkpoint& c, hipStream_t stream) {
  return by_ckpt_rows<vec_elems<DT, DT>(), kUnroll>(rows, c.nb, [&](uint64_t r, uint32_t blocks, dim3 grid) {
    Rows part = x;
    part.p += r * x.stride * DtypeSize<DT>::value;
    hipLaunchKernelGGL((ckpt_pack_kernel<DT>), grid, dim3(kThreads), 0, stream, part, dim, FastDiv((uint32_t)c.nb),
                       blocks, c.codes + r * c.nb * kCkptBlock, c.exps + r * c.nb);
    return launch_status(stream);
  });
}

template <int DT>
hipError_t unpack_dt(const Checkpoint& c, uint64_t rows, uint64_t dim, const Rows& out, hipStream_t stream) {
  return by_ckpt_rows<vec_elems<DT, DT>(), kUnroll>(rows, c.nb, [&](uint64_t r, uint32_t blocks, dim3 grid) {
    Rows part = out;
    part.p += r * out.stride * DtypeSize<DT>::value;
    hipLaunchKernelGGL((ckpt_unpack_kernel<DT>), grid, dim3(kThreads), 0, stream, c.codes + r * c.nb * kCkptBlock,
                       c.exps + r * c.nb, FastDiv((uint32_t)c.nb), blocks, part, dim);
    return launch_status(stream);
  });
}

}  // namespace

hipError_t launch_ckpt_pack(const Rows& x, uint64_t rows, uint64_t dim, void* ckpt, hipStream_t stream) {
  const Checkpoint c(ckpt, rows, dim);
  switch (x.dt) {
    case DT_F32: return pack_dt<DT_F32>(x, rows, dim, c, stream);
    case DT_F16: return pack_dt<DT_F16>(x, rows, dim, c, stream);
    default: return pack_dt<DT_BF16>(x, rows, dim, c, stream);
  }
}

hipError_t launch_ckpt_unpack(const void* ckpt, uint64_t rows, uint64_t dim, const Rows& out, hipStream_t stream) {
  const Checkpoint c((void*)ckpt, rows, dim);
  switch (out.dt) {
    case DT_F32: return unpack_dt<DT_F32>(c, rows, dim, out, stream);
    case DT_F16: return unpack_dt<DT_F16>(c, rows, dim, out, stream);
    default: return unpack_dt<DT_BF16>(c, rows, dim, out, stream);
  }
}

}  // namespace rar
