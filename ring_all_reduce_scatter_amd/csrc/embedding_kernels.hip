// Embedding lookup with scaling, and its gradient by sorted tokens, for gfx950.
//
//   out[t]     = round(a * W[id[t]])                 (a zero row for an id outside the table)
//   dW[v]      = round(a * sum of dout[t] over the tokens t with id[t] = v)   [+ dW[v]]
//
// The gradient is a sum over the tokens of each table row.  The tokens are
// sorted by row first (token_sort_kernel), keeping their order within a
// row, so that every row's sum is formed in binary32 in an order that the
// ids alone fix (ascending, in pieces), without atomics on the sums: the
// same inputs give the same bits.
//
// All of it is bound by memory for batches and by latency for a few tokens.
// Times on one MI355X, inputs cold: lookup of 16,383 rows of 4096 bf16 29.7
// us (6.2 TB/s of its 185 MB); gradient of 32,768 x 2048 bf16 tokens into
// 50,021 f32 rows 125 us: sort 13, sums and zero rows 113 (4.9 TB/s of 549
// MB; 95 where the memory-side cache holds the inputs), the second launch
// following the first without a gap; 509 x 512 f32 tokens into 8192 rows 8.6
// us, one launch of 9.4 with cold inputs in a kernel trace (8.2 warm).
#include <algorithm>

#include "operator_launch.hpp"
#include "row_access.hpp"

namespace rar {
namespace {

constexpr int kSeg = 64 * 8;  // columns of a row that a wavefront takes

// A wavefront's number in the grid, the same register for all its lanes.
__device__ __forceinline__ uint32_t grid_wave() {
  return blockIdx.x * (blockDim.x / 64) + (uint32_t)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
}

// A lane's share of kSeg columns from c0 on: V vectors, 64 * E columns apart.
template <int E>
struct SegCols {
  static constexpr int V = 8 / E;
  VecF<E> x[V];
  __device__ __forceinline__ void add(const SegCols& o) {
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int i = 0; i < E; ++i) x[j].v[i] += o.x[j].v[i];
  }
};
template <int E>
__device__ __forceinline__ uint64_t seg_col(uint64_t c0, int j) {
  return c0 + (uint32_t)(j * 64 + (int)(threadIdx.x & 63)) * E;
}
template <int DT, int E>
__device__ __forceinline__ SegCols<E> load_seg(const char* base, uint64_t row, uint64_t c0, uint64_t dim) {
  SegCols<E> s;
#pragma unroll
  for (int j = 0; j < SegCols<E>::V; ++j) {
    const uint64_t c = seg_col<E>(c0, j);
    s.x[j] = load_vec_upto<DT, E>(base, row + c, vec_count<E>(dim, c));
  }
  return s;
}
// WT: segments on cache-line boundaries are stored write-through.  (Elsewhere
// that costs: 32,768 x 1000 f32 tokens into 65,536 rows took 113.6 us with
// all segments on 16-byte boundaries so, 105.3 us this way.)
template <int DT, int E, bool WT>
__device__ __forceinline__ void store_seg(char* base, uint64_t row, uint64_t c0, uint64_t dim, const SegCols<E>& s) {
  constexpr int ES = DtypeSize<DT>::value;
  const char* seg = base + (row + c0) * ES;  // the same in all lanes
  if (WT && ((uint64_t)seg & 127) == 0) {
    const WtRange range = wt_range(seg, kSeg * ES);
#pragma unroll
    for (int j = 0; j < SegCols<E>::V; ++j) {
      const uint64_t c = seg_col<E>(c0, j);
      const int n = vec_count<E>(dim, c);
      if (n == E) store_vec_wt<DT, E>(range, (uint32_t)(c - c0) * ES, s.x[j]);
      else store_vec_upto<DT, E>(base, row + c, n, s.x[j]);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < SegCols<E>::V; ++j) {
    const uint64_t c = seg_col<E>(c0, j);
    store_vec_upto<DT, E>(base, row + c, vec_count<E>(dim, c), s.x[j]);
  }
}

// ------------------------------------------------------------------ lookup
// A wavefront per token and kSeg columns: each instruction moves a contiguous
// kilobyte, and a batch has enough wavefronts to need no loop.  Rows of the
// table go through the caches (frequent tokens are read again); the output is
// stored nontemporal (write-through was 2 % slower).

template <int DW, int DO, typename ID>
__global__ __launch_bounds__(kThreads) void embedding_kernel(Rows weight, uint64_t vocab, uint64_t dim,
                                                              const ID* __restrict__ ids, uint32_t units,
                                                              uint32_t segs, float scale, Rows out) {
  constexpr int E = vec_elems<DW, DO>();
  for (uint64_t w = grid_wave(); w < units; w += (uint64_t)gridDim.x * (kThreads / 64)) {
    const uint32_t u = (uint32_t)w;
    const uint64_t t = u / segs, c = (uint64_t)(u - (uint32_t)t * segs) * kSeg;
    const int64_t id = ids[t];
    SegCols<E> g = {};
    if ((uint64_t)id < vocab) {
      g = load_seg<DW, E>(weight.p, (uint64_t)id * weight.stride, c, dim);
#pragma unroll
      for (int j = 0; j < SegCols<E>::V; ++j)
#pragma unroll
        for (int i = 0; i < E; ++i) g.x[j].v[i] *= scale;
    }
    store_seg<DO, E, false>(out.p, t * out.stride, c, dim, g);
  }
}

template <int DW, int DO, typename ID>
hipError_t embedding_typed(const Rows& w, uint64_t vocab, uint64_t dim, const void* ids, uint64_t tokens, float scale,
                           const Rows& out, hipStream_t stream) {
  const uint32_t segs = (uint32_t)((dim + kSeg - 1) / kSeg);
  const uint32_t units = (uint32_t)(tokens * segs);
  constexpr uint32_t waves = kThreads / 64;
  // a wavefront each, as far as one launch holds them (2^32 threads)
  const uint32_t groups = std::min<uint32_t>(units / waves + (units % waves != 0), 1u << 23);
  hipLaunchKernelGGL((embedding_kernel<DW, DO, ID>), dim3(groups), dim3(kThreads), 0, stream, w, vocab, dim,
                     (const ID*)ids, units, segs, scale, out);
  return launch_status(stream);
}

template <int DW, typename ID>
hipError_t embedding_to(const Rows& w, uint64_t vocab, uint64_t dim, const void* ids, uint64_t tokens, float scale,
                        const Rows& out, hipStream_t stream) {
  switch (out.dt) {
    case DT_F32: return embedding_typed<DW, DT_F32, ID>(w, vocab, dim, ids, tokens, scale, out, stream);
    case DT_F16: return embedding_typed<DW, DT_F16, ID>(w, vocab, dim, ids, tokens, scale, out, stream);
    default: return embedding_typed<DW, DT_BF16, ID>(w, vocab, dim, ids, tokens, scale, out, stream);
  }
}

template <typename ID>
hipError_t embedding_ids(const Rows& w, uint64_t vocab, uint64_t dim, const void* ids, uint64_t tokens, float scale,
                         const Rows& out, hipStream_t stream) {
  switch (w.dt) {
    case DT_F32: return embedding_to<DT_F32, ID>(w, vocab, dim, ids, tokens, scale, out, stream);
    case DT_F16: return embedding_to<DT_F16, ID>(w, vocab, dim, ids, tokens, scale, out, stream);
    default: return embedding_to<DT_BF16, ID>(w, vocab, dim, ids, tokens, scale, out, stream);
  }
}

// ------------------------------------------------------------------ token sort
// Workgroup b owns the R table rows from lo = b*R.  Its 16 wavefronts each
// walk one sixteenth of the tokens: they count the tokens of every owned row
// (and those of rows before lo, which is where the workgroup's part of the
// order begins) and keep the owned tokens in LDS.  With the counts turned
// into positions (row by row, within a row wavefront by wavefront) they
// place the kept tokens, or, where a wavefront met more than it can keep,
// walk the ids again.  Tokens that share a row and a wavefront iteration are
// ranked by their lanes.  Every workgroup reads all ids: 256 workgroups read
// them from the L2, and no pass over memory or launch is added.  It is bound
// by the latency of its phases: 7 us for 1100 ids, 13 us for 32,768 (30 us
// before the owned tokens were kept, each iteration of the second walk then
// waiting for its ids and, in the workgroup of a frequent token, its ranks).

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr uint32_t kSortKeep = 256;      // owned tokens that a wavefront keeps from the first walk
constexpr uint32_t kSortMaxRows = 1792;  // counters of 112 KiB, kept tokens of 32: of the CU's 160
constexpr int kSortAhead = 16;           // ids in flight per lane

// Table rows of the tokens t, t + 64, ... below end; kNoRow for a token that
// counts for none.
constexpr uint32_t kNoRow = 0xffffffffu;
template <typename ID>
__device__ __forceinline__ void load_rows(const ID* ids, uint32_t t, uint32_t end, uint32_t vocab, int64_t padding,
                                          uint32_t* row) {
  ID id[kSortAhead];
#pragma unroll
  for (int k = 0; k < kSortAhead; ++k) {
    const uint32_t i = t + 64 * k;
    id[k] = ids[i < end ? i : end - 1];
  }
#pragma unroll
  for (int k = 0; k < kSortAhead; ++k) {
    const int64_t v = id[k];
    row[k] = t + 64 * k < end && (uint64_t)v < vocab && v != padding ? (uint32_t)v : kNoRow;
  }
}

// Lanes with the same r (below 2^rbits) as this one, among those of `in`.
__device__ __forceinline__ uint64_t lanes_alike(bool in, uint32_t r, int rbits) {
  uint64_t alike = __ballot(in);
  for (int j = 0; j < rbits; ++j) {
    const bool bit = (r >> j) & 1u;
    const uint64_t set = __ballot(bit);
    alike &= bit ? set : ~set;
  }
  return alike;
}
// Bits of the lanes before this one.
__device__ __forceinline__ uint64_t lanes_before() { return (1ull << (threadIdx.x & 63)) - 1ull; }

template <typename ID>
__global__ __launch_bounds__(kSortThreads) void token_sort_kernel(const ID* __restrict__ ids, uint32_t tokens,
                                                                   uint32_t vocab, int64_t padding, uint32_t R,
                                                                   int rbits, TokenSort sort) {
  extern __shared__ uint32_t sm[];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  uint32_t* wsum = sm;                                               // [kSortWaves]
  TokenEntry* keep = (TokenEntry*)(sm + kSortWaves) + w * kSortKeep;  // [kSortWaves][kSortKeep]
  uint32_t* cnt = sm + kSortWaves + 2 * kSortWaves * kSortKeep;      // [kSortWaves][R]
  const uint32_t lo = blockIdx.x * R;
  const uint32_t rows = vocab - lo < R ? vocab - lo : R;
  for (uint32_t i = tid; i < kSortWaves * R; i += kSortThreads) cnt[i] = 0;
  for (uint64_t i = (uint64_t)blockIdx.x * kSortThreads + tid; i < sort.ncounts; i += (uint64_t)gridDim.x * kSortThreads)
    sort.counts[i] = 0;
  __syncthreads();
  const uint32_t part = ((tokens + kSortWaves - 1) / kSortWaves + 63) / 64 * 64;
  const uint32_t t0 = (uint32_t)w * part;  // at most tokens + 1024: below 2^32
  const uint32_t t1 = t0 + part < tokens ? t0 + part : tokens;
  uint32_t before = 0, kept = 0;
  for (uint32_t b = t0; b < t1; b += 64 * kSortAhead) {
    uint32_t id[kSortAhead];
    load_rows(ids, b + lane, t1, vocab, padding, id);
#pragma unroll
    for (int k = 0; k < kSortAhead; ++k) {
      if (id[k] < lo) ++before;
      const uint32_t r = id[k] - lo;
      const bool in = id[k] >= lo && r < rows;
      const uint64_t owned = __ballot(in);
      if (owned == 0) continue;  // uniform over the wavefront
      if (in) {
        atomicAdd(&cnt[w * R + r], 1u);
        const uint32_t at = kept + (uint32_t)__popcll(owned & lanes_before());
        if (at < kSortKeep) keep[at] = TokenEntry{b + 64 * k + lane, r};
      }
      kept += (uint32_t)__popcll(owned);
    }
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) before += (uint32_t)__shfl_xor((int)before, d, 64);
  if (lane == 0) wsum[w] = before;
  __syncthreads();
  uint32_t base = 0;
#pragma unroll
  for (int k = 0; k < kSortWaves; ++k) base += wsum[k];
  __syncthreads();
  // exclusive scan of the rows' totals: each thread takes `per` consecutive rows
  const uint32_t per = (R + kSortThreads - 1) / kSortThreads;
  uint32_t mine = 0;
  for (uint32_t j = 0; j < per; ++j) {
    const uint32_t r = (uint32_t)tid * per + j;
    if (r >= rows) break;
#pragma unroll
    for (int k = 0; k < kSortWaves; ++k) mine += cnt[k * R + r];
  }
  uint32_t incl = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t y = (uint32_t)__shfl_up((int)incl, d, 64);
    if (lane >= d) incl += y;
  }
  if (lane == 63) wsum[w] = incl;
  __syncthreads();
  uint32_t pos = base + incl - mine;
#pragma unroll
  for (int k = 0; k < kSortWaves; ++k)
    if (k < w) pos += wsum[k];
  for (uint32_t j = 0; j < per; ++j) {
    const uint32_t r = (uint32_t)tid * per + j;
    if (r >= rows) break;
    sort.start[lo + r] = pos;
    uint32_t c[kSortWaves];
#pragma unroll
    for (int k = 0; k < kSortWaves; ++k) c[k] = cnt[k * R + r];
#pragma unroll
    for (int k = 0; k < kSortWaves; ++k) {
      cnt[k * R + r] = pos;
      pos += c[k];
    }
    if (lo + r + 1 == vocab) sort.start[vocab] = pos;
  }
  __syncthreads();
  auto place = [&](bool in, uint32_t r, uint32_t token) {
    const uint64_t alike = lanes_alike(in, r, rbits);
    if (in) {
      const uint32_t at = cnt[w * R + r];
      const uint64_t below = alike & lanes_before();
      sort.entries[at + (uint32_t)__popcll(below)] = TokenEntry{token, lo + r};
      if (below == 0) cnt[w * R + r] = at + (uint32_t)__popcll(alike);
    }
  };
  if (kept <= kSortKeep) {  // uniform over the wavefront
    for (uint32_t i = 0; i < kept; i += 64) {
      const bool in = i + lane < kept;
      const TokenEntry e = keep[in ? i + lane : i];
      place(in, in ? e.row : 0, e.token);
    }
    return;
  }
  for (uint32_t b = t0; b < t1; b += 64 * kSortAhead) {
    uint32_t id[kSortAhead];
    load_rows(ids, b + lane, t1, vocab, padding, id);
#pragma unroll
    for (int k = 0; k < kSortAhead; ++k) {
      const uint32_t r = id[k] - lo;
      const bool in = id[k] >= lo && r < rows;
      if (__ballot(in) != 0) place(in, in ? r : 0, b + 64 * k + lane);
    }
  }
}

hipError_t token_sort(const void* ids, bool ids64, uint64_t tokens, uint64_t vocab, int64_t padding,
                      const TokenSort& sort, hipStream_t stream) {
  uint32_t R = (uint32_t)((vocab + 255) / 256);
  if (R < 16) R = 16;
  if (R > kSortMaxRows) R = kSortMaxRows;
  int rbits = 1;
  while ((1u << rbits) < R) ++rbits;
  const uint32_t grid = (uint32_t)((vocab + R - 1) / R);
  const size_t lds = ((size_t)kSortWaves * R + kSortWaves + 2 * kSortWaves * kSortKeep) * sizeof(uint32_t);
  if (ids64)
    hipLaunchKernelGGL(token_sort_kernel<int64_t>, dim3(grid), dim3(kSortThreads), lds, stream, (const int64_t*)ids,
                       (uint32_t)tokens, (uint32_t)vocab, padding, R, rbits, sort);
  else
    hipLaunchKernelGGL(token_sort_kernel<int32_t>, dim3(grid), dim3(kSortThreads), lds, stream, (const int32_t*)ids,
                       (uint32_t)tokens, (uint32_t)vocab, padding, R, rbits, sort);
  return launch_status(stream);
}

// ------------------------------------------------------------------ gradient
// The sorted tokens are cut into pieces of CH entries whatever rows they
// belong to, so that a row with very many tokens (a few tokens make up most
// of any text) is shared by many wavefronts.  A wavefront takes one piece
// and kSeg columns, adds the gradients of each run of equal rows, and stores
// a run that lies inside its piece straight to the table's gradient.  A run
// cut by the piece's beginning goes to the piece's head partial, one that
// begins here and is cut by its end to its tail partial (binary32).
// The last wavefront to leave a part of a run adds them, the tail and the
// heads that follow it in order, in two levels so that a row with very many
// parts is not added by one wavefront alone: first the parts of each group
// of kGroup pieces, then the groups.  Parts and counts are accessed at
// device scope, past the XCD's L2, and a part's store has been acknowledged
// before it is counted, so the last wavefront reads what all have stored.
// The pieces are the launch's first wavefronts, so these waits pass under the
// zeroing of the table's other rows (a further launch for the cut runs took
// 10 us and its start).
// (A wavefront per table row took 1827 us where this takes 125: the most
// frequent of 32,768 natural tokens makes up 6 % of them.)
// Rows without tokens are zeroed by further wavefronts of the same launch,
// whose stores overlap the others' loads; done by the sort's workgroups the
// call took 12 us more.

struct Pieces {
  uint32_t tokens;
  uint32_t ch;      // entries per piece (a power of two, at most 64)
  uint32_t n;       // pieces
  uint32_t segs;    // column segments of kSeg
  uint64_t dim;
  uint32_t zrows;   // rows that one wavefront looks through for empty ones (at most 16)
  float* partials;  // [n][2][segs * kSeg]: head, tail
  uint32_t* counts; // [2][n][segs]: arrived parts of the group, groups of the run, that begin in a piece
};
constexpr uint32_t kGroup = 16, kPartBatch = 4;

// Rounds a finished sum into the table's gradient.
template <int DO, int E, bool WT = true>
__device__ __forceinline__ void finish_row(const Rows& dw, uint64_t row, uint64_t c0, uint64_t dim, float scale,
                                           bool accumulate, SegCols<E> acc) {
#pragma unroll
  for (int j = 0; j < SegCols<E>::V; ++j)
#pragma unroll
    for (int i = 0; i < E; ++i) acc.x[j].v[i] *= scale;
  if (accumulate) acc.add(load_seg<DO, E>(dw.p, row * dw.stride, c0, dim));
  store_seg<DO, E, WT>(dw.p, row * dw.stride, c0, dim, acc);
}

// Partial sums: a lane's eight values as two vectors 256 columns apart, in a
// row of kSeg floats (so no column is missing) of the workspace or of LDS.
template <int E>
__device__ __forceinline__ u32x4 partial_half(const SegCols<E>& s, int h) {
  u32x4 x;
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = __float_as_uint(s.x[(4 * h) / E].v[(4 * h) % E + i]);
  return x;
}
template <int E>
__device__ __forceinline__ void set_partial_half(SegCols<E>& s, int h, u32x4 x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) s.x[(4 * h) / E].v[(4 * h) % E + i] = __uint_as_float(x[i]);
}
// In LDS: p the lane's place.
template <int E>
__device__ __forceinline__ void store_partial(float* p, const SegCols<E>& s) {
#pragma unroll
  for (int h = 0; h < 2; ++h) *(u32x4*)(p + h * 256) = partial_half(s, h);
}
template <int E>
__device__ __forceinline__ SegCols<E> load_partial(const float* p) {
  SegCols<E> s;
#pragma unroll
  for (int h = 0; h < 2; ++h) set_partial_half(s, h, *(const u32x4*)(p + h * 256));
  return s;
}
// In the workspace, at device scope.
constexpr int kSc1 = 16;  // cache-policy operand
__device__ __forceinline__ WtRange part_range(const Pieces& pc, uint32_t piece, uint32_t tail, uint64_t c0) {
  return wt_range((const char*)(pc.partials + ((uint64_t)piece * 2 + tail) * pc.segs * kSeg + c0), kSeg * 4);
}
template <int E>
__device__ __forceinline__ void store_part(WtRange r, const SegCols<E>& s) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
    __builtin_amdgcn_raw_buffer_store_b128(partial_half(s, h), r, (int)((threadIdx.x & 63) * 16 + h * 1024), 0, kSc1);
}
template <int E>
__device__ __forceinline__ SegCols<E> load_part(WtRange r) {
  SegCols<E> s;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    set_partial_half(s, h,
                     __builtin_amdgcn_raw_buffer_load_b128(r, (int)((threadIdx.x & 63) * 16 + h * 1024), 0, kSc1));
  return s;
}

constexpr uint32_t kBatch = 8;  // rows of dout in flight per wavefront

// Counts this wavefront; how many came before it.  The loads that follow in
// the program stay after it (the fence is the compiler's alone).
__device__ __forceinline__ uint32_t arrive(uint32_t* count) {
  uint32_t before = 0;
  if ((threadIdx.x & 63) == 0) before = __hip_atomic_fetch_add(count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  before = (uint32_t)__builtin_amdgcn_readfirstlane(before);
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  return before;
}

// Adds the parts of the pieces a, a + step, ... below z, in order, of a run
// that begins in piece `first`; a batch of loads is in flight at a time, the
// last one repeated at its end.
template <int E>
__device__ __forceinline__ void add_parts(const Pieces& pc, uint32_t a, uint32_t z, uint32_t step, uint32_t first,
                                          uint64_t c0, SegCols<E>& sum) {
  for (uint32_t k0 = a; k0 < z; k0 += kPartBatch * step) {
    SegCols<E> part[kPartBatch];
#pragma unroll
    for (uint32_t i = 0; i < kPartBatch; ++i) {
      const uint32_t k = k0 + i * step < z ? k0 + i * step : k0;
      part[i] = load_part<E>(part_range(pc, k, k == first, c0));
    }
#pragma unroll
    for (uint32_t i = 0; i < kPartBatch; ++i)
      if (k0 + i * step < z) sum.add(part[i]);
  }
}

template <int DI, int DO>
__global__ __launch_bounds__(kThreads) void embedding_grad_kernel(Rows dout, uint64_t vocab,
                                                                   const uint32_t* __restrict__ start,
                                                                   const TokenEntry* __restrict__ entries, Pieces pc,
                                                                   float scale, bool accumulate, Rows dw) {
  constexpr int E = vec_elems<DI, DO>();
  const uint32_t u = grid_wave();
  const uint32_t units = pc.n * pc.segs;
  if (u >= units) {  // zero those of pc.zrows rows that have no tokens
    const uint32_t lane = threadIdx.x & 63;
    const uint64_t v0 = (uint64_t)(u - units) * pc.zrows;
    if (accumulate || v0 >= vocab) return;
    const uint64_t mine = v0 + lane;
    const bool empty = lane < pc.zrows && mine < vocab && start[mine] == start[mine + 1];
    for (uint64_t left = __ballot(empty); left != 0; left &= left - 1) {
      const uint64_t v = v0 + (uint32_t)__builtin_ctzll(left);
      for (uint32_t k = 0; k < pc.segs; ++k)
        store_seg<DO, vec_elems<DO, DO>(), true>(dw.p, v * dw.stride, (uint64_t)k * kSeg, pc.dim, {});
    }
    return;
  }
  const uint32_t p = u / pc.segs;
  const uint32_t seg = u - p * pc.segs;
  const uint64_t c0 = (uint64_t)seg * kSeg;
  const uint32_t total = start[vocab];
  const uint32_t i0 = p * pc.ch;
  // the piece's entries, one a lane, and the rows beside it; past the used
  // entries the buffer holds anything, which is not looked at
  const uint32_t lane = threadIdx.x & 63, last = pc.tokens - 1;
  const TokenEntry own = entries[lane < pc.ch && i0 + lane < last ? i0 + lane : last];
  const uint32_t row_before = entries[i0 > 0 ? i0 - 1 : 0].row;
  const uint32_t row_after = entries[i0 + pc.ch < last ? i0 + pc.ch : last].row;
  if (i0 >= total) return;
  const uint32_t m = i0 + pc.ch < total ? pc.ch : total - i0;
  auto entry_token = [&](uint32_t i) { return (uint32_t)__builtin_amdgcn_readlane(own.token, i); };
  auto entry_row = [&](uint32_t i) { return (uint32_t)__builtin_amdgcn_readlane(own.row, i); };
  uint32_t row = entry_row(0);
  const bool began = i0 > 0 && row_before == row;  // the first run began in an earlier piece
  const bool cut = i0 + m < total && row_after == entry_row(m - 1);
  bool head = began;
  SegCols<E> acc = {};
  for (uint32_t b = 0; b < m; b += kBatch) {
    SegCols<E> g[kBatch];
#pragma unroll
    for (uint32_t k = 0; k < kBatch; ++k)
      g[k] = load_seg<DI, E>(dout.p, (uint64_t)entry_token(b + k < m ? b + k : b) * dout.stride, c0, pc.dim);
#pragma unroll
    for (uint32_t k = 0; k < kBatch; ++k) {
      if (b + k >= m) break;
      const uint32_t r = entry_row(b + k);
      if (r != row) {  // uniform
        if (head) store_part(part_range(pc, p, 0, c0), acc);
        else finish_row<DO, E>(dw, row, c0, pc.dim, scale, accumulate, acc);
        head = false;
        row = r;
        acc = SegCols<E>{};
      }
      acc.add(g[k]);
    }
  }
  const bool tail = cut && !head;
  if (head) store_part(part_range(pc, p, 0, c0), acc);
  else if (cut) store_part(part_range(pc, p, 1, c0), acc);
  else finish_row<DO, E>(dw, row, c0, pc.dim, scale, accumulate, acc);
  if (!began && !tail) return;
  stores_done();
  // the run of the head part, then the run of the tail part
  for (uint32_t part = 0; part < 2; ++part) {
    if (!(part ? tail : began)) continue;
    const uint32_t to = part ? entry_row(m - 1) : entry_row(0);
    const uint32_t first = start[to] / pc.ch, end = (start[to + 1] - 1) / pc.ch;  // the run's pieces
    const uint32_t group = p / kGroup * kGroup;
    const uint32_t a = first > group ? first : group, z = end < group + kGroup - 1 ? end : group + kGroup - 1;
    SegCols<E> sum = {};
    if (z > a) {  // the group's last part adds them
      if (arrive(&pc.counts[(uint64_t)a * pc.segs + seg]) != z - a) continue;
      add_parts(pc, a, z + 1, 1, first, c0, sum);
    }
    if (end / kGroup != first / kGroup) {  // the run's last group adds them
      if (z > a) {
        store_part(part_range(pc, a, a == first, c0), sum);
        stores_done();
      }
      if (arrive(&pc.counts[((uint64_t)pc.n + first) * pc.segs + seg]) != end / kGroup - first / kGroup) continue;
      sum = load_part<E>(part_range(pc, first, 1, c0));
      add_parts(pc, (first / kGroup + 1) * kGroup, end + 1, kGroup, first, c0, sum);
    }
    finish_row<DO, E>(dw, to, c0, pc.dim, scale, accumulate, sum);
  }
}

// ------------------------------------------------------------------ gradient of few tokens
// Up to kFewTokens tokens are sorted, added and stored by one launch.  A
// workgroup of W wavefronts takes R table rows and kSeg columns: it picks its
// rows' tokens out of all ids (one a thread), zeroes the rows that have none,
// sorts the others in LDS by counting for each how many come before it (an
// entry is row << 10 | token, so they are ordered as numbers), and adds them
// in W pieces as above, with the partial sums in LDS.  Against three launches
// (sort, sums, cut runs): 8.6 us instead of 16.5 for 509 x 512 f32 tokens
// into 8192 rows.  Four wavefronts are enough for 256 tokens, and more of
// these workgroups fit a CU: 100 x 512 f32 tokens into 32,768 rows take 12.9
// us so, 14.1 with sixteen.
constexpr uint32_t kFewTokens = 1024, kFewRows = 1024;

template <int DI, int DO, typename ID, uint32_t W>
__global__ __launch_bounds__(W * 64) void embedding_grad_few_kernel(Rows dout, const ID* __restrict__ ids,
                                                                         uint32_t tokens, uint32_t vocab, uint64_t dim,
                                                                         int64_t padding, uint32_t R, float scale,
                                                                         bool accumulate, Rows dw) {
  constexpr int E = vec_elems<DI, DO>();
  extern __shared__ uint32_t sm[];
  uint32_t* count = sm;                      // [W]
  uint32_t* used = sm + W;                   // [kFewRows / 32] bits
  uint32_t* list = used + kFewRows / 32;     // [W * 64]
  uint32_t* sorted = list + W * 64;          // [W * 64]
  float* part = (float*)(sorted + W * 64);   // [W][2][kSeg]
  const uint32_t tid = threadIdx.x, lane = tid & 63;
  const uint32_t w = (uint32_t)__builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t lo = blockIdx.x * R, rows = vocab - lo < R ? vocab - lo : R;
  const uint64_t c0 = (uint64_t)blockIdx.y * kSeg;
  const int64_t id = ids[tid < tokens ? tid : 0];
  const bool in = tid < tokens && id != padding && id >= (int64_t)lo && id < (int64_t)lo + rows;
  const uint64_t mask = __ballot(in);
  if (tid < kFewRows / 32) used[tid] = 0;
  if (lane == 0) count[w] = (uint32_t)__popcll(mask);
  __syncthreads();
  uint32_t at = (uint32_t)__popcll(mask & lanes_before()), total = 0;
#pragma unroll
  for (uint32_t k = 0; k < W; ++k) {
    if (k < w) at += count[k];
    total += count[k];
  }
  total = (uint32_t)__builtin_amdgcn_readfirstlane(total);
  if (in) {
    const uint32_t r = (uint32_t)id - lo;
    list[at] = r << 10 | tid;
    atomicOr(&used[r >> 5], 1u << (r & 31));
  }
  __syncthreads();
  if (tid < total) {
    const uint32_t e = list[tid];
    uint32_t rank = 0;
#pragma unroll 4
    for (uint32_t k = 0; k < total; ++k) rank += list[k] < e;
    sorted[rank] = e;
  }
  if (!accumulate)
    // whole rows, shared out among the workgroups of these rows
    for (uint32_t r = w * gridDim.y + blockIdx.y; r < rows; r += W * gridDim.y)
      if (!(used[r >> 5] >> (r & 31) & 1u))
        for (uint32_t k = 0; k < gridDim.y; ++k)
          store_seg<DO, vec_elems<DO, DO>(), false>(dw.p, (uint64_t)(lo + r) * dw.stride, (uint64_t)k * kSeg, dim, {});
  if (total == 0) return;
  __syncthreads();
  // pieces of ch entries, the w-th this wavefront's
  const uint32_t ch = (total + W - 1) / W;
  const uint32_t i0 = w * ch, i1 = i0 + ch < total ? i0 + ch : total;
  float* mine = part + lane * 4;
  bool begins = false;  // a run begins in this piece and goes on in the next
  uint32_t row = 0;
  if (i0 < i1) {
    row = sorted[i0] >> 10;
    bool head = i0 > 0 && sorted[i0 - 1] >> 10 == row;
    const bool cut = i1 < total && sorted[i1] >> 10 == sorted[i1 - 1] >> 10;
    SegCols<E> acc = {};
    for (uint32_t b = i0; b < i1; b += kBatch) {
      const uint32_t m = i1 - b < kBatch ? i1 - b : kBatch;
      uint32_t e[kBatch];
      SegCols<E> g[kBatch];
#pragma unroll
      for (uint32_t k = 0; k < kBatch; ++k) e[k] = (uint32_t)__builtin_amdgcn_readfirstlane(sorted[b + (k < m ? k : 0)]);
#pragma unroll
      for (uint32_t k = 0; k < kBatch; ++k)
        if (k < m) g[k] = load_seg<DI, E>(dout.p, (uint64_t)(e[k] & 1023u) * dout.stride, c0, dim);
#pragma unroll
      for (uint32_t k = 0; k < kBatch; ++k) {
        if (k >= m) break;
        if (e[k] >> 10 != row) {  // uniform
          if (head) store_partial(mine + w * 2 * kSeg, acc);
          else finish_row<DO, E, false>(dw, lo + row, c0, dim, scale, accumulate, acc);
          head = false;
          row = e[k] >> 10;
          acc = SegCols<E>{};
        }
        acc.add(g[k]);
      }
    }
    begins = cut && !head;
    if (head) store_partial(mine + w * 2 * kSeg, acc);
    else if (cut) store_partial(mine + (w * 2 + 1) * kSeg, acc);
    else finish_row<DO, E, false>(dw, lo + row, c0, dim, scale, accumulate, acc);
  }
  __syncthreads();
  if (!begins) return;
  SegCols<E> acc = load_partial<E>(mine + (w * 2 + 1) * kSeg);
  for (uint32_t k = w + 1; k * ch < total && sorted[k * ch] >> 10 == row; ++k)
    acc.add(load_partial<E>(mine + k * 2 * kSeg));
  finish_row<DO, E, false>(dw, lo + row, c0, dim, scale, accumulate, acc);
}

template <int DI, int DO, uint32_t W>
hipError_t embedding_grad_few(const EmbeddingGrad& a, hipStream_t stream) {
  const uint64_t segs = (a.dim + kSeg - 1) / kSeg;
  // 32 wavefronts per CU, each workgroup of at least a row per wavefront
  constexpr uint64_t groups = 256 * 32 / W;
  const uint64_t R = std::min<uint64_t>(std::max<uint64_t>((a.vocab * segs + groups - 1) / groups, W), kFewRows);
  const dim3 grid((unsigned)((a.vocab + R - 1) / R), (unsigned)segs), block(W * 64);
  const size_t lds = (W + kFewRows / 32 + 2 * W * 64 + W * 2 * kSeg) * sizeof(uint32_t);
  if (a.ids64)
    hipLaunchKernelGGL((embedding_grad_few_kernel<DI, DO, int64_t, W>), grid, block, lds, stream, a.dout,
                       (const int64_t*)a.ids, (uint32_t)a.tokens, (uint32_t)a.vocab, a.dim, a.padding, (uint32_t)R,
                       a.scale, a.accumulate, a.dweight);
  else
    hipLaunchKernelGGL((embedding_grad_few_kernel<DI, DO, int32_t, W>), grid, block, lds, stream, a.dout,
                       (const int32_t*)a.ids, (uint32_t)a.tokens, (uint32_t)a.vocab, a.dim, a.padding, (uint32_t)R,
                       a.scale, a.accumulate, a.dweight);
  return launch_status(stream);
}

// Rows that one zeroing wavefront looks through, about 8 KiB: one row of 2048
// f32 (with 16 rows the whole call takes 9 us more), 16 rows of 128 bf16 (with
// one, each wavefront waits for its row's starts for a store of 256 bytes).
uint32_t zero_rows(uint64_t dim, int dt) {
  const uint64_t row_bytes = dim * (dt == DT_F32 ? 4 : 2);
  return row_bytes >= 8192 ? 1 : (uint32_t)std::min<uint64_t>(8192 / row_bytes, 16);
}

template <int DI, int DO>
hipError_t embedding_grad_typed(const EmbeddingGrad& a, hipStream_t stream) {
  if (a.tokens == 0 && a.accumulate) return hipSuccess;
  if (a.tokens > 0 && a.tokens <= kFewTokens && a.dim <= (uint64_t)kSeg * 65535)
    return a.tokens <= 256 ? embedding_grad_few<DI, DO, 4>(a, stream) : embedding_grad_few<DI, DO, 16>(a, stream);
  hipError_t e = token_sort(a.ids, a.ids64, a.tokens, a.vocab, a.padding, a.sort, stream);
  if (e != hipSuccess) return e;
  const uint64_t ch = embedding_piece(a.tokens, a.dim);
  const uint32_t zrows = zero_rows(a.dim, DO);
  const Pieces pc{(uint32_t)a.tokens, (uint32_t)ch, (uint32_t)((a.tokens + ch - 1) / ch), (uint32_t)((a.dim + kSeg - 1) / kSeg), a.dim,
                  zrows, a.partials, a.sort.counts};
  const uint64_t units = (uint64_t)pc.n * pc.segs + (a.accumulate ? 0 : embedding_zero_waves(a.vocab, a.dim, DO));
  constexpr int waves = kThreads / 64;
  hipLaunchKernelGGL((embedding_grad_kernel<DI, DO>), dim3((unsigned)((units + waves - 1) / waves)), dim3(kThreads), 0,
                     stream, a.dout, a.vocab, a.sort.start, a.sort.entries, pc, a.scale, a.accumulate, a.dweight);
  return launch_status(stream);
}

template <int DI>
hipError_t embedding_grad_to(const EmbeddingGrad& a, hipStream_t stream) {
  switch (a.dweight.dt) {
    case DT_F32: return embedding_grad_typed<DI, DT_F32>(a, stream);
    case DT_F16: return embedding_grad_typed<DI, DT_F16>(a, stream);
    default: return embedding_grad_typed<DI, DT_BF16>(a, stream);
  }
}

}  // namespace

hipError_t launch_embedding(const Rows& weight, uint64_t vocab, uint64_t dim, const void* ids, bool ids64,
                            uint64_t tokens, float scale, const Rows& out, hipStream_t stream) {
  if (tokens == 0) return hipSuccess;
  return ids64 ? embedding_ids<int64_t>(weight, vocab, dim, ids, tokens, scale, out, stream)
               : embedding_ids<int32_t>(weight, vocab, dim, ids, tokens, scale, out, stream);
}

uint64_t embedding_piece(uint64_t tokens, uint64_t dim) {
  // short pieces while that gives wavefronts to fill the chip (16 per CU),
  // longer ones for long batches: fewer partials
  const uint64_t segs = (dim + kSeg - 1) / kSeg;
  uint64_t ch = kBatch;
  while (ch < 64 && (tokens + ch - 1) / ch * segs > 4096) ch *= 2;
  return ch;
}

uint64_t embedding_zero_waves(uint64_t vocab, uint64_t dim, int dt) {
  const uint64_t rows = zero_rows(dim, dt);
  return (vocab + rows - 1) / rows;
}

hipError_t launch_embedding_grad(const EmbeddingGrad& a, hipStream_t stream) {
  switch (a.dout.dt) {
    case DT_F32: return embedding_grad_to<DT_F32>(a, stream);
    case DT_F16: return embedding_grad_to<DT_F16>(a, stream);
    default: return embedding_grad_to<DT_BF16>(a, stream);
  }
}

}  // namespace rar
