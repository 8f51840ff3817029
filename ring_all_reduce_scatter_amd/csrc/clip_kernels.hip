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
#include <algorithm>

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

// The norm's workgroups: one per CU, of four tile groups.  (Every workgroup
// adds one to a common count at its end, about 10 ns each one after the
// other: 58.8 MB of f32 took 35 us with 2048 workgroups of 256 threads.)
constexpr int kNormThreads = 1024, kNormWaves = kNormThreads / 64, kNormGroups = kNormThreads / kThreads;

// Sum over the workgroup; every lane receives it.  lds: one value per wave.
template <int KIND>
__device__ __forceinline__ Acc<KIND> block_join(Acc<KIND> a, double* lds) {
  if constexpr (KIND == kNormMax) a.m = group_max_u32<64>(a.m);
  else a.s = wave_sum(a.s);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = KIND == kNormMax ? (double)a.m : a.s;
  __syncthreads();
  Acc<KIND> r;
#pragma unroll
  for (int w = 0; w < kNormWaves; ++w) {
    Acc<KIND> o;
    if constexpr (KIND == kNormMax) o.m = (uint32_t)lds[w];
    else o.s = lds[w];
    r.join(o);
  }
  return r;
}

// This wavefront's stores have been acknowledged.
__device__ __forceinline__ void stores_done() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
}

// Vectors of a whole tile per lane, in batches that are loaded at once.
template <int E>
constexpr int tile_vecs() {
  return (int)kClipTile / (kThreads * E);
}

// Tiles are taken by groups of kThreads threads (four wavefronts).
__device__ __forceinline__ uint32_t tile_lane() { return threadIdx.x % kThreads; }

template <int DT, int KIND, bool NT>
__device__ __forceinline__ void norm_tile(const char* in, uint32_t n, Acc<KIND>& acc) {
  constexpr int E = vec_elems<DT, DT>(), V = tile_vecs<E>();
  if (n == kClipTile) {
    VecRaw<DT, E> raw[V];
#pragma unroll
    for (int j = 0; j < V; ++j) raw[j] = load_raw<DT, E, NT>(in, (j * kThreads + tile_lane()) * E);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const VecF<E> g = unpack<DT, E>(raw[j]);
#pragma unroll
      for (int i = 0; i < E; ++i) acc.add(g.v[i]);
    }
    return;
  }
  for (uint32_t e = tile_lane() * E; e < n; e += kThreads * E) {
    const VecF<E> g = load_vec_upto<DT, E>(in, e, vec_count<E>(n, e));
#pragma unroll
    for (int i = 0; i < E; ++i) acc.add(g.v[i]);
  }
}

// Where the workgroups of one launch meet: each stores its partial result
// and counts itself; the last one adds the partial results, in their order,
// and sets the count back for the next launch.  Partial results and count
// are accessed at device scope, past the XCD's L2, and a store has been
// acknowledged before its workgroup counts itself, so the last one reads
// what all have stored.  (Acquire and release operations would order the
// same by writing back and invalidating whole caches: with them in every
// workgroup the norm of 378 million bf16 elements took 219 us, not 122.)
struct NormMeeting {
  double* partials;
  uint32_t* arrived;
  float* norm;
  float* factor;
  double scale, max_norm;
};

// NT: streaming loads, unless a clip of a set that the caches can hold follows.
template <int KIND, bool NT>
__global__ __launch_bounds__(kNormThreads) void grad_norm_kernel(const ClipDesc* __restrict__ descs, uint32_t ntiles,
                                                                  NormMeeting m) {
  extern __shared__ double lds[];
  Acc<KIND> acc;
  // consecutive tiles to different workgroups: few tiles reach many CUs
  const uint32_t group = (uint32_t)__builtin_amdgcn_readfirstlane(threadIdx.x / kThreads);
  for (uint32_t t = group * gridDim.x + blockIdx.x; t < ntiles; t += gridDim.x * kNormGroups) {
    const ClipDesc d = descs[t];
    switch (d.types & 0xff) {
      case DT_F32: norm_tile<DT_F32, KIND, NT>(gaddr(d.in), d.n, acc); break;
      case DT_F16: norm_tile<DT_F16, KIND, NT>(gaddr(d.in), d.n, acc); break;
      default: norm_tile<DT_BF16, KIND, NT>(gaddr(d.in), d.n, acc); break;
    }
  }
  acc = block_join(acc, lds);
  if (gridDim.x > 1) {
    uint32_t* last = (uint32_t*)(lds + kNormWaves);
    if (threadIdx.x == 0) {
      __hip_atomic_store(&m.partials[blockIdx.x], KIND == kNormMax ? (double)acc.m : acc.s, __ATOMIC_RELAXED,
                         __HIP_MEMORY_SCOPE_AGENT);
      stores_done();
      *last = __hip_atomic_fetch_add(m.arrived, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (*last != gridDim.x - 1) return;
    acc = Acc<KIND>{};
    for (uint32_t i = threadIdx.x; i < gridDim.x; i += kNormThreads) {
      const double p = __hip_atomic_load(&m.partials[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      Acc<KIND> o;
      if constexpr (KIND == kNormMax) o.m = (uint32_t)p;
      else o.s = p;
      acc.join(o);
    }
    acc = block_join(acc, lds);
  }
  if (threadIdx.x != 0) return;
  double total;
  if constexpr (KIND == kNormMax) total = (double)__uint_as_float(acc.m);
  else total = __builtin_sqrt(acc.s);
  total *= __builtin_fabs(m.scale);
  *m.norm = (float)total;
  double c = m.max_norm / (total + 1e-6);
  if (c > 1.0) c = 1.0;  // a NaN norm stays a NaN factor
  *m.factor = (float)(m.scale * c);
  *m.arrived = 0;
}

template <int DI, int DO>
__device__ __forceinline__ void clip_tile(const char* in, char* out, uint32_t n, float f) {
  constexpr int E = vec_elems<DI, DO>(), V = tile_vecs<E>();
  if (n == kClipTile && ((uint64_t)out & 15) == 0) {  // uniform
    const WtRange range = wt_range(out, kClipTile * DtypeSize<DO>::value);
    VecRaw<DI, E> raw[V];
#pragma unroll
    for (int j = 0; j < V; ++j) raw[j] = load_raw<DI, E, true>(in, (j * kThreads + threadIdx.x) * E);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      VecF<E> g = unpack<DI, E>(raw[j]);
#pragma unroll
      for (int i = 0; i < E; ++i) g.v[i] *= f;
      store_vec_wt<DO, E>(range, (j * kThreads + threadIdx.x) * E * DtypeSize<DO>::value, g);
    }
    return;
  }
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

// The tiles go in the reverse of the norm's order: the last ones it read are
// the ones that the memory-side cache still holds.
__global__ __launch_bounds__(kThreads) void grad_clip_kernel(const ClipDesc* __restrict__ descs,
                                                              const float* __restrict__ factor) {
  const ClipDesc d = descs[gridDim.x - 1 - blockIdx.x];
  const float f = *factor;
  switch (d.types & 0xff) {
    case DT_F32: clip_tile_from<DT_F32>(d, f); break;
    case DT_F16: clip_tile_from<DT_F16>(d, f); break;
    default: clip_tile_from<DT_BF16>(d, f); break;
  }
}

// Sets up to this many tiles (128 MiB of binary32) are read into the caches
// by the norm, for the clip to find; larger ones would only sweep them.
constexpr uint64_t kClipCachedTiles = 4096;

template <int KIND>
hipError_t norm_launch(const ClipSet& set, bool reread, double scale, double max_norm, float* norm,
                       hipStream_t stream) {
  const uint32_t grid = (uint32_t)std::min<uint64_t>(std::max<uint64_t>(set.ntiles, 1), kClipMaxBlocks);
  const NormMeeting m{(double*)set.partials, (uint32_t*)set.result + 1, norm, (float*)set.result, scale, max_norm};
  const size_t lds = (kNormWaves + 1) * sizeof(double);
  const ClipDesc* descs = (const ClipDesc*)set.descs;
  if (reread)
    hipLaunchKernelGGL((grad_norm_kernel<KIND, false>), dim3(grid), dim3(kNormThreads), lds, stream, descs,
                       (uint32_t)set.ntiles, m);
  else
    hipLaunchKernelGGL((grad_norm_kernel<KIND, true>), dim3(grid), dim3(kNormThreads), lds, stream, descs,
                       (uint32_t)set.ntiles, m);
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
  return kind == kNormMax ? norm_launch<kNormMax>(set, false, scale, 0.0, norm, stream)
                          : norm_launch<0>(set, false, scale, 0.0, norm, stream);
}

hipError_t launch_grad_clip(const ClipSet& set, int kind, double scale, double max_norm, float* norm,
                            hipStream_t stream) {
  const bool reread = set.ntiles <= kClipCachedTiles;
  const hipError_t e = kind == kNormMax ? norm_launch<kNormMax>(set, reread, scale, max_norm, norm, stream)
                                        : norm_launch<0>(set, reread, scale, max_norm, norm, stream);
  if (e != hipSuccess || set.ntiles == 0) return e;
  hipLaunchKernelGGL(grad_clip_kernel, dim3((unsigned)set.ntiles), dim3(kThreads), 0, stream,
                     (const ClipDesc*)set.descs, (const float*)set.result);
  return launch_status(stream);
}

}  // namespace rar
