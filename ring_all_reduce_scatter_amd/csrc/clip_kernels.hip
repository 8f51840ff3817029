// Global norm of a set of gradient tensors, and clipping by it, for gfx950.
//
//   norm = |s| * sqrt(sum g^2)   or   |s| * max |g|        over all tensors
//   out  = round(g * f),   f = s * min(1, max_norm / (norm + 1e-6))
//
// The set is cut into tiles of kClipTileBytes of one tensor, each with a
// descriptor written once when the set is prepared, so four wavefronts find
// their elements with one scalar load.  Squares and their sums are binary64:
// the square of any finite binary32 is then finite and not zero, the sum of
// a billion of them is right to the last bit of the binary32 result, and the
// vector units have the rate to spare (one 64-bit FMA an element against at
// least 2 bytes of memory).  Partial sums are added in a fixed order, so a
// result depends on the set alone.
//
// Bound by memory: the norm reads the set once, a clip once more beside its
// writes.  Times on one MI355X, inputs cold: norm of 378 million bf16
// elements 115 us (6.6 TB/s), clip of the same list 354 us (norm 114, clip
// 237 at 6.4 TB/s); 40 tensors of 19.6 million f32 elements in all 36 us
// (three passes of 78 MB at the copy rate: 37).  One cooperative launch that
// held the set on the chip between the norm and the product would spare the
// second read, but such a launch alone takes 19.5 us here against 2.5, more
// than that read costs for any set that fits.
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
  const uint32_t ty = (uint32_t)types[lo], tile = clip_tile_elems(ty & 0xff);
  const uint64_t e0 = (g - tab[lo]) * tile, left = count[lo] - e0;
  ClipDesc d;
  d.in = in[lo] + e0 * ((ty & 0xff) == DT_F32 ? 4 : 2);
  d.out = out[lo] + e0 * ((ty >> 8) == DT_F32 ? 4 : 2);
  d.n = left < tile ? (uint32_t)left : tile;
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

// The norm's workgroups: one per CU, of four tile groups.  (2048 workgroups of
// 256 threads take 17 us for 78 MB of f32 and 123 us for 378 million bf16
// elements, these 16 and 115.)
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

// Tiles are taken by groups of kThreads threads (four wavefronts).
__device__ __forceinline__ uint32_t tile_lane() { return threadIdx.x % kThreads; }

// A lane's share of a tile as loaded, whatever its type: kTileVecs vectors,
// kThreads vectors apart, as far as the tile has whole vectors, and one of
// the elements after them; zeros where there is nothing.
constexpr int kTileVecs = kClipTileBytes / 16 / kThreads;
struct TileRaw {
  u32x4 v[kTileVecs];
  float t;
};

template <bool NT>
__device__ __forceinline__ TileRaw load_tile(const ClipDesc& d) {
  const char* in = gaddr(d.in);
  const uint32_t type = d.types & 0xff, lane = tile_lane();
  const uint32_t per = type == DT_F32 ? 4 : 8, nvec = d.n / per, ntail = d.n % per;
  auto vector = [&](int j) -> u32x4 {
    const u32x4_any* p = (const u32x4_any*)(in + (j * kThreads + lane) * 16);
    if constexpr (NT) return __builtin_nontemporal_load(p);
    else return *p;
  };
  TileRaw x;
  x.t = 0.0f;
  if (nvec == kTileVecs * kThreads) {  // uniform: the loads need no masks
#pragma unroll
    for (int j = 0; j < kTileVecs; ++j) x.v[j] = vector(j);
    return x;
  }
#pragma unroll
  for (int j = 0; j < kTileVecs; ++j) {
    x.v[j] = u32x4{0u, 0u, 0u, 0u};
    if (j * kThreads + lane < nvec) x.v[j] = vector(j);
  }
  if (lane < ntail) x.t = load_elem_dt(in, nvec * per + lane, (int)type);
  return x;
}

template <int DT, int KIND>
__device__ __forceinline__ void norm_tile(const TileRaw& x, Acc<KIND>& acc) {
#pragma unroll
  for (int j = 0; j < kTileVecs; ++j) {
    const Vec<DT> g = unpack16<DT>(x.v[j]);
#pragma unroll
    for (int i = 0; i < Vec<DT>::E; ++i) acc.add(g.v[i]);
  }
  acc.add(x.t);
}

// The norm and the factor from the whole set's sum.
struct NormResult {
  float* norm;
  float* factor;  // NULL: not wanted
  double scale, max_norm;
};
template <int KIND>
__device__ __forceinline__ float finish_norm(const Acc<KIND>& acc, const NormResult& m) {
  double total;
  if constexpr (KIND == kNormMax) total = (double)__uint_as_float(acc.m);
  else total = __builtin_sqrt(acc.s);
  total *= __builtin_fabs(m.scale);
  double c = m.max_norm / (total + 1e-6);
  // a NaN norm stays a NaN factor; infinity over infinity is no limit either
  if (!(c <= 1.0) && total == total) c = 1.0;
  const float f = (float)(m.scale * c);
  if (threadIdx.x == 0) {
    *m.norm = (float)total;
    if (m.factor) *m.factor = f;
  }
  return f;
}

// Where the workgroups of one launch meet: each stores its partial result
// and counts itself, and the last one adds the partial results in their
// order.  The count has two levels, since adds to one address go one after
// the other, about 9 ns each: for 78 MB of f32 one count took 36 us with 2048
// workgroups, where two levels took 17, and 17.1 us with 256, where they take
// 16.3.  Workgroup b counts at word b mod kMeetWays, and the last to arrive
// there at the top word.  The last workgroup sets the words back for the next
// launch.  Partial results and counts are accessed at device scope, past the XCD's L2, and a store
// has been acknowledged before its workgroup counts itself, so the last one
// reads what all have stored.  (Acquire and release operations would order
// the same by writing back and invalidating whole caches: with them in every
// workgroup the norm of 378 million bf16 elements took 219 us, not 112.)
constexpr uint32_t kMeetWays = 16, kMeetStride = 16;  // words 64 bytes apart
static_assert((kMeetWays + 1) * kMeetStride * sizeof(uint32_t) <= kClipCountBytes, "count words");
struct Meeting {
  double* partials;
  uint32_t* counts;  // kMeetWays words, then the top word
};

// Whether this workgroup is the last (of gridDim.x > 1); one lane calls it.
__device__ __forceinline__ bool arrive(const Meeting& m, double partial) {
  __hip_atomic_store(&m.partials[blockIdx.x], partial, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  stores_done();
  const uint32_t way = blockIdx.x % kMeetWays, here = (gridDim.x - way + kMeetWays - 1) / kMeetWays;
  if (__hip_atomic_fetch_add(&m.counts[way * kMeetStride], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) != here - 1)
    return false;
  const uint32_t ways = gridDim.x < kMeetWays ? gridDim.x : kMeetWays;
  return __hip_atomic_fetch_add(&m.counts[kMeetWays * kMeetStride], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
         ways - 1;
}

// NT: streaming loads, unless a clip of a set that the caches can hold follows.
template <int KIND, bool NT>
__global__ __launch_bounds__(kNormThreads) void grad_norm_kernel(const ClipDesc* __restrict__ descs, uint32_t ntiles,
                                                                  Meeting m, NormResult result) {
  extern __shared__ double lds[];
  Acc<KIND> acc;
  // consecutive tiles to different workgroups: few tiles reach many CUs
  const uint32_t group = (uint32_t)__builtin_amdgcn_readfirstlane(threadIdx.x / kThreads);
  const uint32_t step = gridDim.x * kNormGroups;
  uint32_t t = group * gridDim.x + blockIdx.x;
  if (t < ntiles) {
    // the next tile is loaded while this one is added, its descriptor a tile earlier
    ClipDesc d = descs[t], next = descs[t + step < ntiles ? t + step : t];
    TileRaw x = load_tile<NT>(d);
    for (;;) {
      const uint32_t type = d.types & 0xff;
      const bool more = t + step < ntiles;
      TileRaw y;
      if (more) {
        y = load_tile<NT>(next);
        d = next;
        t += step;
        if (t + step < ntiles) next = descs[t + step];
      }
      if (type == DT_F32) norm_tile<DT_F32>(x, acc);
      else if (type == DT_F16) norm_tile<DT_F16>(x, acc);
      else norm_tile<DT_BF16>(x, acc);
      if (!more) break;
      x = y;
    }
  }
  acc = block_join(acc, lds);
  if (gridDim.x > 1) {
    uint32_t* last = (uint32_t*)(lds + kNormWaves);
    if (threadIdx.x == 0) *last = arrive(m, KIND == kNormMax ? (double)acc.m : acc.s);
    __syncthreads();
    if (!*last) return;
    if (threadIdx.x <= kMeetWays) m.counts[threadIdx.x * kMeetStride] = 0;
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
  finish_norm(acc, result);
}

template <int DI, int DO, bool NT>
__device__ __forceinline__ void clip_tile(const char* in, char* out, uint32_t n, float f) {
  constexpr int E = vec_elems<DI, DO>(), V = kClipTileBytes / DtypeSize<DI>::value / (kThreads * E);
  const uint32_t lane = threadIdx.x, nvec = n / E, ntail = n % E;
  VecRaw<DI, E> raw[V];
  if (nvec == V * kThreads && ((uint64_t)out & 15) == 0) {  // uniform: a whole tile, no masks
    const WtRange range = wt_range(out, V * kThreads * E * DtypeSize<DO>::value);
#pragma unroll
    for (int j = 0; j < V; ++j) raw[j] = load_raw<DI, E, NT>(in, (j * kThreads + lane) * E);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      VecF<E> g = unpack<DI, E>(raw[j]);
#pragma unroll
      for (int i = 0; i < E; ++i) g.v[i] *= f;
      store_vec_wt<DO, E>(range, (j * kThreads + lane) * E * DtypeSize<DO>::value, g);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const uint32_t i = j * kThreads + lane;
    raw[j] = VecRaw<DI, E>{};
    if (i < nvec) raw[j] = load_raw<DI, E, NT>(in, i * E);
  }
  float t = 0.0f;
  if (lane < ntail) t = load_elem<DI>(in, nvec * E + lane);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const uint32_t i = j * kThreads + lane;
    VecF<E> g = unpack<DI, E>(raw[j]);
#pragma unroll
    for (int k = 0; k < E; ++k) g.v[k] *= f;
    if (i < nvec) store_vec<DO, E>(out, i * E, g);
  }
  if (lane < ntail) store_elem<DO>(out, nvec * E + lane, t * f);
}

template <int DI, bool NT>
__device__ __forceinline__ void clip_tile_from(const ClipDesc& d, float f) {
  const char* in = gaddr(d.in);
  char* out = gaddr(d.out);
  switch (d.types >> 8) {
    case DT_F32: clip_tile<DI, DT_F32, NT>(in, out, d.n, f); break;
    case DT_F16: clip_tile<DI, DT_F16, NT>(in, out, d.n, f); break;
    default: clip_tile<DI, DT_BF16, NT>(in, out, d.n, f); break;
  }
}

// The tiles go in the reverse of the norm's order, eight by eight: the last
// ones it read are the ones that the L2s still hold (32 MiB of eight), and
// tile t goes to the XCD (t mod 8, as workgroups are dealt) whose L2 the norm
// read it through.  Norm and clip of 78 MB of f32 take 38.9 us so, 42.6 in
// reverse without regard to the XCD (the memory-side cache alone), 42.3 in the
// norm's own order; in place 37.6, 48.1 and 39.4; up to 24 MB the norm's order
// does as well.  NT: streaming loads, for a set that the norm has not read
// into the caches.
constexpr uint32_t kXcds = 8;
template <bool NT>
__global__ __launch_bounds__(kThreads) void grad_clip_kernel(const ClipDesc* __restrict__ descs, uint32_t ntiles,
                                                              const float* __restrict__ factor) {
  const uint32_t t = (gridDim.x - blockIdx.x - 1) / kXcds * kXcds + blockIdx.x % kXcds;
  if (t >= ntiles) return;
  const ClipDesc d = descs[t];
  const float f = *factor;
  switch (d.types & 0xff) {
    case DT_F32: clip_tile_from<DT_F32, NT>(d, f); break;
    case DT_F16: clip_tile_from<DT_F16, NT>(d, f); break;
    default: clip_tile_from<DT_BF16, NT>(d, f); break;
  }
}

// A set of up to kFewTiles tiles in one launch: a workgroup keeps them in
// its registers from the norm to the stores.
constexpr uint32_t kFewPerGroup = 2, kFewTiles = kFewPerGroup * kNormGroups;

template <int DI, int DO>
__device__ __forceinline__ void store_tile(const TileRaw& x, const ClipDesc& d, float f) {
  constexpr int E = Vec<DI>::E, S = vec_elems<DI, DO>();  // loaded and stored at once
  char* out = gaddr(d.out);
  const uint32_t lane = tile_lane(), nvec = d.n / E;
#pragma unroll
  for (int j = 0; j < kTileVecs; ++j) {
    const uint32_t i = j * kThreads + lane;
    if (i >= nvec) continue;
    const Vec<DI> g = unpack16<DI>(x.v[j]);
#pragma unroll
    for (int h = 0; h < E; h += S) {
      VecF<S> o;
#pragma unroll
      for (int k = 0; k < S; ++k) o.v[k] = g.v[h + k] * f;
      store_vec<DO, S>(out, i * E + h, o);
    }
  }
  if (lane < d.n % E) store_elem<DO>(out, nvec * E + lane, x.t * f);
}
template <int DI>
__device__ __forceinline__ void store_tile_from(const TileRaw& x, const ClipDesc& d, float f) {
  if (d.types >> 8 == DT_F32) store_tile<DI, DT_F32>(x, d, f);
  else if (d.types >> 8 == DT_F16) store_tile<DI, DT_F16>(x, d, f);
  else store_tile<DI, DT_BF16>(x, d, f);
}

template <int KIND>
__global__ __launch_bounds__(kNormThreads) void grad_clip_few_kernel(const ClipDesc* __restrict__ descs,
                                                                      uint32_t ntiles, NormResult result) {
  extern __shared__ double lds[];
  const uint32_t group = (uint32_t)__builtin_amdgcn_readfirstlane(threadIdx.x / kThreads);
  TileRaw x[kFewPerGroup];
  Acc<KIND> acc;
#pragma unroll
  for (uint32_t k = 0; k < kFewPerGroup; ++k)
    if (k * kNormGroups + group < ntiles) x[k] = load_tile<false>(descs[k * kNormGroups + group]);
#pragma unroll
  for (uint32_t k = 0; k < kFewPerGroup; ++k) {
    if (k * kNormGroups + group >= ntiles) break;
    const uint32_t type = descs[k * kNormGroups + group].types & 0xff;
    if (type == DT_F32) norm_tile<DT_F32>(x[k], acc);
    else if (type == DT_F16) norm_tile<DT_F16>(x[k], acc);
    else norm_tile<DT_BF16>(x[k], acc);
  }
  const float f = finish_norm(block_join(acc, lds), result);
#pragma unroll
  for (uint32_t k = 0; k < kFewPerGroup; ++k) {
    if (k * kNormGroups + group >= ntiles) break;
    const ClipDesc d = descs[k * kNormGroups + group];
    const uint32_t type = d.types & 0xff;
    if (type == DT_F32) store_tile_from<DT_F32>(x[k], d, f);
    else if (type == DT_F16) store_tile_from<DT_F16>(x[k], d, f);
    else store_tile_from<DT_BF16>(x[k], d, f);
  }
}

// Sets up to this many tiles (128 MiB) are read into the caches
// by the norm, for the clip to find; larger ones would only sweep them.
constexpr uint64_t kClipCachedTiles = 8192;

template <int KIND>
hipError_t norm_launch(const ClipSet& set, bool reread, const NormResult& result, hipStream_t stream) {
  const uint32_t grid = (uint32_t)std::min<uint64_t>(std::max<uint64_t>(set.ntiles, 1), kClipMaxBlocks);
  const Meeting m{(double*)set.partials, (uint32_t*)set.counts};
  const size_t lds = (kNormWaves + 1) * sizeof(double);
  const ClipDesc* descs = (const ClipDesc*)set.descs;
  if (reread)
    hipLaunchKernelGGL((grad_norm_kernel<KIND, false>), dim3(grid), dim3(kNormThreads), lds, stream, descs,
                       (uint32_t)set.ntiles, m, result);
  else
    hipLaunchKernelGGL((grad_norm_kernel<KIND, true>), dim3(grid), dim3(kNormThreads), lds, stream, descs,
                       (uint32_t)set.ntiles, m, result);
  return launch_status(stream);
}

template <int KIND>
hipError_t clip_launch(const ClipSet& set, const NormResult& result, hipStream_t stream) {
  const ClipDesc* descs = (const ClipDesc*)set.descs;
  if (set.ntiles <= kFewTiles) {
    hipLaunchKernelGGL(grad_clip_few_kernel<KIND>, dim3(1), dim3(kNormThreads), kNormWaves * sizeof(double), stream,
                       descs, (uint32_t)set.ntiles, result);
    return launch_status(stream);
  }
  const bool reread = set.ntiles <= kClipCachedTiles;
  const hipError_t e = norm_launch<KIND>(set, reread, result, stream);
  if (e != hipSuccess) return e;
  const uint32_t ntiles = (uint32_t)set.ntiles;
  const dim3 grid((ntiles + kXcds - 1) / kXcds * kXcds), block(kThreads);
  const float* factor = result.factor;
  if (reread) hipLaunchKernelGGL(grad_clip_kernel<false>, grid, block, 0, stream, descs, ntiles, factor);
  else hipLaunchKernelGGL(grad_clip_kernel<true>, grid, block, 0, stream, descs, ntiles, factor);
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
  const NormResult r{norm, nullptr, scale, 0.0};
  return kind == kNormMax ? norm_launch<kNormMax>(set, false, r, stream) : norm_launch<0>(set, false, r, stream);
}

hipError_t launch_grad_clip(const ClipSet& set, int kind, double scale, double max_norm, float* norm,
                            hipStream_t stream) {
  const NormResult r{norm, (float*)set.factor, scale, max_norm};
  return kind == kNormMax ? clip_launch<kNormMax>(set, r, stream) : clip_launch<0>(set, r, stream);
}

}  // namespace rar
