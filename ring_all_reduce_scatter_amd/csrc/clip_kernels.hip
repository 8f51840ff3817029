// Global norm of a set of gradient tensors, and clipping by it, for gfx950.
//
//   norm = |s| * sqrt(sum g^2)   or   |s| * max |g|        over all tensors
//   out  = round(g * f),   f = s * min(1, max_norm / (norm + 1e-6))
//
// The set is cut into tiles of kClipTile elements of one tensor, each with
// a descriptor written once when the set is prepared, so a workgroup finds
// its elements with one scalar load.  Squares and their sums are binary64:
// the square of any finite binary32 is then finite and not zero, the sum of
// a billion of them is right to the last bit of the binary32 result, and the
// vector units have the rate to spare (one 64-bit FMA an element against at
// least 2 bytes of memory).  Partial sums are added in a fixed order, so a
// result depends on the set alone.
#include "operator_launch.hpp"
#include "row_access.hpp"

namespace rar {
namespace {

constexpr int kNormMax = 1;

// The tensors' addresses arrive as integers; as global pointers they give
// global memory instructions.
__device__ __forceinline__ char* gaddr(uint64_t a) { return (char*)(__attribute__((address_space(1))) char*)a; }

struct ClipDesc {  // kClipDescBytes
  uint64_t in, out;
  uint32_t n, types;
  uint64_t unused;
};

__global__ __launch_bounds__(kThreads) void clip_desc_kernel(const uint64_t* __restrict__ tab, uint64_t nt,
                                                              uint64_t ntiles, ClipDesc* __restrict__ descs) {
  const uint64_t g = (uint64_t)blockIdx.x * kThreads + threadIdx.x;
  if (g >= ntiles) return;
  // largest t with first[t] <= g (a tensor without elements has no tile)
  uint64_t lo = 0, hi = nt;
  while (hi - lo > 1) {
    const uint64_t mid = (lo + hi) / 2;
    if (tab[mid] <= g) lo = mid;
    else hi = mid;
  }
  const uint64_t* in = tab + nt + 1;
  const uint64_t* out = in + nt;
  const uint64_t* count = out + nt;
  const uint64_t* types = count + nt;
  const uint64_t e0 = (g - tab[lo]) * kClipTile, left = count[lo] - e0;
  const uint32_t ty = (uint32_t)types[lo];
  ClipDesc d;
  d.in = in[lo] + e0 * ((ty & 0xff) == DT_F32 ? 4 : 2);
  d.out = out[lo] + e0 * ((ty >> 8) == DT_F32 ? 4 : 2);
  d.n = left < kClipTile ? (uint32_t)left : kClipTile;
  d.types = ty;
  d.unused = 0;
  descs[g] = d;
}

// The set's running norm in one lane: the sum of squares, or the largest
// absolute value as a bit pattern (which orders NaN above infinity).
template <int KIND>
struct Acc {
  double s = 0.0;
  uint32_t m = 0;
  __device__ __forceinline__ void add(float x) {
    if constexpr (KIND == kNormMax) m = max(m, absbits(x));
    else s = __builtin_fma((double)x, (double)x, s);
  }
  __device__ __forceinline__ void join(const Acc& o) {
    if constexpr (KIND == kNormMax) m = max(m, o.m);
    else s += o.s;
  }
};

// Sum over the workgroup; every lane receives it.  lds: one Acc per wave.
template <int KIND>
__device__ __forceinline__ Acc<KIND> block_join(Acc<KIND> a, double* lds) {
  if constexpr (KIND == kNormMax) a.m = group_max_u32<64>(a.m);
  else a.s = wave_sum(a.s);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = KIND == kNormMax ? (double)a.m : a.s;
  __syncthreads();
  Acc<KIND> r;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) {
    Acc<KIND> o;
    if constexpr (KIND == kNormMax) o.m = (uint32_t)lds[w];
    else o.s = lds[w];
    r.join(o);
  }
  return r;
}

template <int DT, int KIND>
__device__ __forceinline__ void norm_tile(const char* in, uint32_t n, Acc<KIND>& acc) {
  constexpr int E = vec_elems<DT, DT>();
  for (uint32_t e = threadIdx.x * E; e < n; e += kThreads * E) {
    const VecF<E> g = load_vec_upto<DT, E>(in, e, vec_count<E>(n, e));
#pragma unroll
    for (int i = 0; i < E; ++i) acc.add(g.v[i]);
  }
}

template <int KIND>
__global__ __launch_bounds__(kThreads) void grad_norm_kernel(const ClipDesc* __restrict__ descs, uint64_t ntiles,
                                                              double* __restrict__ partials) {
  extern __shared__ double lds[];
  Acc<KIND> acc;
  for (uint64_t t = blockIdx.x; t < ntiles; t += gridDim.x) {
    const ClipDesc d = descs[t];
    switch (d.types & 0xff) {
      case DT_F32: norm_tile<DT_F32>(gaddr(d.in), d.n, acc); break;
      case DT_F16: norm_tile<DT_F16>(gaddr(d.in), d.n, acc); break;
      default: norm_tile<DT_BF16>(gaddr(d.in), d.n, acc); break;
    }
  }
  acc = block_join(acc, lds);
  if (threadIdx.x == 0) partials[blockIdx.x] = KIND == kNormMax ? (double)acc.m : acc.s;
}

template <int KIND>
__global__ __launch_bounds__(kThreads) void norm_finish_kernel(const double* __restrict__ partials, uint32_t nparts,
                                                                double scale, double max_norm,
                                                                float* __restrict__ norm, float* __restrict__ factor) {
  extern __shared__ double lds[];
  Acc<KIND> acc;
  for (uint32_t i = threadIdx.x; i < nparts; i += kThreads) {
    Acc<KIND> o;
    if constexpr (KIND == kNormMax) o.m = (uint32_t)partials[i];
    else o.s = partials[i];
    acc.join(o);
  }
  acc = block_join(acc, lds);
  if (threadIdx.x != 0) return;
  double total;
  if constexpr (KIND == kNormMax) total = (double)__uint_as_float(acc.m);
  else total = __builtin_sqrt(acc.s);
  total *= __builtin_fabs(scale);
  *norm = (float)total;
  double c = max_norm / (total + 1e-6);
  if (c > 1.0) c = 1.0;  // a NaN norm stays a NaN factor
  *factor = (float)(scale * c);
}

template <int DI, int DO>
__device__ __forceinline__ void clip_tile(const char* in, char* out, uint32_t n, float f) {
  constexpr int E = vec_elems<DI, DO>();
  for (uint32_t e = threadIdx.x * E; e < n; e += kThreads * E) {
    const int k = vec_count<E>(n, e);
    VecF<E> g = load_vec_upto<DI, E>(in, e, k);
#pragma unroll
    for (int i = 0; i < E; ++i) g.v[i] *= f;
    store_vec_upto<DO, E>(out, e, k, g);
  }
}

template <int DI>
__device__ __forceinline__ void clip_tile_from(const ClipDesc& d, float f) {
  const char* in = gaddr(d.in);
  char* out = gaddr(d.out);
  switch (d.types >> 8) {
    case DT_F32: clip_tile<DI, DT_F32>(in, out, d.n, f); break;
    case DT_F16: clip_tile<DI, DT_F16>(in, out, d.n, f); break;
    default: clip_tile<DI, DT_BF16>(in, out, d.n, f); break;
  }
}

__global__ __launch_bounds__(kThreads) void grad_clip_kernel(const ClipDesc* __restrict__ descs,
                                                              const float* __restrict__ factor) {
  const ClipDesc d = descs[blockIdx.x];
  const float f = *factor;
  switch (d.types & 0xff) {
    case DT_F32: clip_tile_from<DT_F32>(d, f); break;
    case DT_F16: clip_tile_from<DT_F16>(d, f); break;
    default: clip_tile_from<DT_BF16>(d, f); break;
  }
}

template <int KIND>
hipError_t norm_launches(const ClipSet& set, double scale, double max_norm, float* norm, hipStream_t stream) {
  const size_t lds = kThreads / 64 * sizeof(double);
  const uint32_t grid = set.ntiles < kClipMaxBlocks ? (uint32_t)set.ntiles : kClipMaxBlocks;
  if (grid) {
    hipLaunchKernelGGL((grad_norm_kernel<KIND>), dim3(grid), dim3(kThreads), lds, stream,
                       (const ClipDesc*)set.descs, set.ntiles, (double*)set.partials);
    const hipError_t e = launch_status(stream);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((norm_finish_kernel<KIND>), dim3(1), dim3(kThreads), lds, stream, (const double*)set.partials,
                     grid, scale, max_norm, norm, (float*)set.result);
  return launch_status(stream);
}

}  // namespace

hipError_t launch_clip_desc(const uint64_t* table, void* descs, uint64_t ntensors, uint64_t ntiles,
                            hipStream_t stream) {
  if (ntiles == 0) return hipSuccess;
  hipLaunchKernelGGL(clip_desc_kernel, dim3((unsigned)((ntiles + kThreads - 1) / kThreads)), dim3(kThreads), 0, stream,
                     table, ntensors, ntiles, (ClipDesc*)descs);
  return launch_status(stream);
}

hipError_t launch_grad_norm(const ClipSet& set, int kind, double scale, float* norm, hipStream_t stream) {
  return kind == kNormMax ? norm_launches<kNormMax>(set, scale, 0.0, norm, stream)
                          : norm_launches<0>(set, scale, 0.0, norm, stream);
}

hipError_t launch_grad_clip(const ClipSet& set, int kind, double scale, double max_norm, float* norm,
                            hipStream_t stream) {
  const hipError_t e = kind == kNormMax ? norm_launches<kNormMax>(set, scale, max_norm, norm, stream)
                                        : norm_launches<0>(set, scale, max_norm, norm, stream);
  if (e != hipSuccess || set.ntiles == 0) return e;
  hipLaunchKernelGGL(grad_clip_kernel, dim3((unsigned)set.ntiles), dim3(kThreads), 0, stream,
                     (const ClipDesc*)set.descs, (const float*)set.result);
  return launch_status(stream);
}

}  // namespace rar
