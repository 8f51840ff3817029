// Embedding lookup with scaling, and its gradient by sorted tokens, for gfx950.
//
//   out[t]     = round(a * W[id[t]])                 (a zero row for an id outside the table)
//   dW[v]      = round(a * sum of dout[t] over the tokens t with id[t] = v)   [+ dW[v]]
//
// The gradient is a sum over the tokens of each table row.  The tokens are
// sorted by row first (token_sort_kernel), keeping their order within a
// row, so that every row's sum is formed in ascending token order in
// binary32, without atomics: the same inputs give the same bits.
#include "operator_launch.hpp"
#include "row_access.hpp"

namespace rar {
namespace {

constexpr int kSeg = 64 * 8;  // columns of a row that a wavefront takes

__device__ __forceinline__ int64_t load_id(const void* ids, bool ids64, uint64_t t) {
  return ids64 ? ((const int64_t*)ids)[t] : (int64_t)((const int32_t*)ids)[t];
}

// ------------------------------------------------------------------ lookup

template <int DW, int DO>
__global__ __launch_bounds__(kThreads) void embedding_kernel(Rows weight, uint64_t vocab, uint64_t dim,
                                                              const void* __restrict__ ids, bool ids64,
                                                              uint64_t units, uint32_t segs, float scale, Rows out) {
  const uint64_t u = ((uint64_t)blockIdx.x * kThreads + threadIdx.x) >> 6;
  if (u >= units) return;
  const uint64_t t = u / segs, c = (u - t * segs) * kSeg + (threadIdx.x & 63) * 8;
  if (c >= dim) return;
  const int n = dim - c < 8 ? (int)(dim - c) : 8;
  const int64_t id = load_id(ids, ids64, t);
  G8 g = {};
  if ((uint64_t)id < vocab) {
    g = load8_upto<DW>(weight.p, (uint64_t)id * weight.stride + c, n);
#pragma unroll
    for (int i = 0; i < 8; ++i) g.v[i] *= scale;
  }
  store8_upto<DO, true>(out.p, t * out.stride + c, n, g);
}

template <int DW>
hipError_t embedding_to(const Rows& w, uint64_t vocab, uint64_t dim, const void* ids, bool ids64, uint64_t tokens,
                        float scale, const Rows& out, hipStream_t stream) {
  const uint32_t segs = (uint32_t)((dim + kSeg - 1) / kSeg);
  const uint64_t units = tokens * segs;
  const dim3 grid((unsigned)((units + kThreads / 64 - 1) / (kThreads / 64))), block(kThreads);
  switch (out.dt) {
    case DT_F32:
      hipLaunchKernelGGL((embedding_kernel<DW, DT_F32>), grid, block, 0, stream, w, vocab, dim, ids, ids64, units,
                         segs, scale, out);
      break;
    case DT_F16:
      hipLaunchKernelGGL((embedding_kernel<DW, DT_F16>), grid, block, 0, stream, w, vocab, dim, ids, ids64, units,
                         segs, scale, out);
      break;
    default:
      hipLaunchKernelGGL((embedding_kernel<DW, DT_BF16>), grid, block, 0, stream, w, vocab, dim, ids, ids64, units,
                         segs, scale, out);
  }
  return launch_status(stream);
}

// ------------------------------------------------------------------ token sort
// Workgroup b owns the R table rows from lo = b*R.  Its 16 wavefronts each
// walk one sixteenth of the tokens twice: first they count the tokens of
// every owned row (and those of rows before lo, which is where the
// workgroup's part of the order begins), then, with the counts turned into
// positions (row by row, within a row wavefront by wavefront), they place
// them.  Tokens that share a row and a wavefront iteration are ranked by
// their lanes.  Every workgroup reads all ids: 256 workgroups read them
// from the L2, and no pass over memory or launch is added.

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr uint32_t kSortMaxRows = 2048;  // 16 x 2048 counters: 128 of the 160 KiB of LDS

__global__ __launch_bounds__(kSortThreads) void token_sort_kernel(const void* __restrict__ ids, bool ids64,
                                                                   uint32_t tokens, uint32_t vocab, int64_t padding,
                                                                   uint32_t R, int rbits, TokenSort sort) {
  extern __shared__ uint32_t sm[];
  uint32_t* cnt = sm;                          // [kSortWaves][R]
  uint32_t* wsum = sm + kSortWaves * R;        // [kSortWaves]
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const uint32_t lo = blockIdx.x * R;
  const uint32_t rows = vocab - lo < R ? vocab - lo : R;
  for (uint32_t i = tid; i < kSortWaves * R; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
  const uint32_t part = ((tokens + kSortWaves - 1) / kSortWaves + 63) / 64 * 64;
  const uint64_t t0 = (uint64_t)w * part;
  const uint64_t t1 = t0 + part < tokens ? t0 + part : tokens;
  uint32_t before = 0;
  for (uint64_t b = t0; b < t1; b += 64) {
    const uint64_t t = b + lane;
    int64_t id = -1;
    if (t < t1) id = load_id(ids, ids64, t);
    const bool ok = (uint64_t)id < vocab && id != padding;
    if (ok && (uint32_t)id < lo) ++before;
    if (ok && (uint32_t)id >= lo && (uint32_t)id - lo < rows) atomicAdd(&cnt[w * R + ((uint32_t)id - lo)], 1u);
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
    if (r < rows)
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
    for (int k = 0; k < kSortWaves; ++k) {
      const uint32_t c = cnt[k * R + r];
      cnt[k * R + r] = pos;
      pos += c;
    }
    if (lo + r + 1 == vocab) sort.start[vocab] = pos;
  }
  __syncthreads();
  for (uint64_t b = t0; b < t1; b += 64) {
    const uint64_t t = b + lane;
    int64_t id = -1;
    if (t < t1) id = load_id(ids, ids64, t);
    const bool in = (uint64_t)id < vocab && id != padding && (uint32_t)id >= lo && (uint32_t)id - lo < rows;
    uint64_t peers = __ballot(in);
    if (peers == 0) continue;  // uniform over the wavefront
    const uint32_t r = in ? (uint32_t)id - lo : 0;
    for (int k = 0; k < rbits; ++k) {
      const bool bit = (r >> k) & 1u;
      const uint64_t set = __ballot(bit);
      peers &= bit ? set : ~set;
    }
    if (in) {
      const uint32_t at = cnt[w * R + r];
      const uint64_t below = peers & ((1ull << lane) - 1ull);
      sort.entries[at + (uint32_t)__popcll(below)] = TokenEntry{(uint32_t)t, (uint32_t)id};
      if (below == 0) cnt[w * R + r] = at + (uint32_t)__popcll(peers);
    }
  }
}

// ------------------------------------------------------------------ gradient
// The sorted tokens are cut into pieces of CH entries whatever rows they
// belong to, so that a row with very many tokens (a few tokens make up most
// of any text) is shared by many wavefronts.  A wavefront takes one piece
// and kSeg columns, adds the gradients of each run of equal rows, and stores
// a run that lies inside its piece straight to the table's gradient.  A run
// cut by the piece's beginning goes to the piece's head partial, one that
// begins here and is cut by its end to its tail partial (binary32); after
// the launch the tail and the heads that follow it are added in order.
// Rows without tokens are zeroed by further wavefronts of the same launch.

struct Pieces {
  uint32_t ch;      // entries per piece (a power of two)
  uint32_t n;       // pieces
  uint32_t segs;    // column segments of kSeg
  uint64_t dim;
  float* partials;  // [n][2][dim]: head, tail
};

// Rounds a finished sum into the table's gradient.
template <int DO>
__device__ __forceinline__ void store_row(const Rows& dw, uint64_t row, uint64_t c, int n, float scale,
                                          bool accumulate, G8 acc) {
  const uint64_t at = row * dw.stride + c;
#pragma unroll
  for (int k = 0; k < 8; ++k) acc.v[k] *= scale;
  if (accumulate) {
    const G8 old = load8_upto<DO>(dw.p, at, n);
#pragma unroll
    for (int k = 0; k < 8; ++k) acc.v[k] += old.v[k];
  }
  store8_upto<DO, true>(dw.p, at, n, acc);
}

constexpr int kBatch = 8;  // rows of dout in flight per wavefront

template <int DI, int DO>
__global__ __launch_bounds__(kThreads) void embedding_grad_kernel(Rows dout, uint64_t vocab, TokenSort sort,
                                                                   Pieces pc, float scale, bool accumulate, Rows dw) {
  const int lane = threadIdx.x & 63;
  const uint64_t u = (uint64_t)blockIdx.x * (kThreads / 64) + (uint32_t)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint64_t units = (uint64_t)pc.n * pc.segs;
  if (u >= units) {  // zero the rows without tokens
    const uint64_t v = u - units;
    if (accumulate || v >= vocab || sort.start[v] != sort.start[v + 1]) return;
    for (uint64_t c = lane * 8; c < pc.dim; c += kSeg)
      store8_upto<DO, true>(dw.p, v * dw.stride + c, pc.dim - c < 8 ? (int)(pc.dim - c) : 8, G8{});
    return;
  }
  const uint32_t p = (uint32_t)(u / pc.segs);
  const uint64_t c = (u - (uint64_t)p * pc.segs) * kSeg + lane * 8;
  const uint32_t total = sort.start[vocab];
  const uint32_t i0 = p * pc.ch;
  if (i0 >= total) return;
  const uint32_t i1 = i0 + pc.ch < total ? i0 + pc.ch : total;
  const int n = c >= pc.dim ? 0 : (pc.dim - c < 8 ? (int)(pc.dim - c) : 8);
  uint32_t row = sort.entries[i0].row;
  bool head = i0 > 0 && sort.entries[i0 - 1].row == row;  // the run began in an earlier piece
  const bool cut = i1 < total && sort.entries[i1].row == sort.entries[i1 - 1].row;
  float* part = pc.partials + (uint64_t)p * 2 * pc.dim;
  G8 acc = {};
  for (uint32_t b = i0; b < i1; b += kBatch) {
    const int m = i1 - b < (uint32_t)kBatch ? (int)(i1 - b) : kBatch;
    TokenEntry e[kBatch];
    G8 g[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) e[k] = sort.entries[b + (k < m ? k : 0)];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) g[k] = load8_upto<DI>(dout.p, (uint64_t)e[k].token * dout.stride + c, n);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (k >= m) break;
      if (e[k].row != row) {  // uniform
        if (head) store8_upto<DT_F32, false>((char*)part, c, n, acc);
        else store_row<DO>(dw, row, c, n, scale, accumulate, acc);
        head = false;
        row = e[k].row;
        acc = G8{};
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) acc.v[i] += g[k].v[i];
    }
  }
  if (head) store8_upto<DT_F32, false>((char*)part, c, n, acc);
  else if (cut) store8_upto<DT_F32, false>((char*)part, pc.dim + c, n, acc);
  else store_row<DO>(dw, row, c, n, scale, accumulate, acc);
}

// Adds up the runs that were cut: the workgroup of the piece in which such a
// run begins (and of kSeg columns) adds the piece's tail and the heads of
// the pieces up to the run's end, each wavefront a consecutive share of
// them, the shares in order.
constexpr int kJoinWaves = 8;

template <int DO>
__global__ __launch_bounds__(kJoinWaves * 64) void embedding_join_kernel(uint64_t vocab, TokenSort sort, Pieces pc,
                                                                          float scale, bool accumulate, Rows dw) {
  extern __shared__ float share[];  // [kJoinWaves][kSeg]
  const uint32_t p = blockIdx.x / pc.segs;
  const uint32_t total = sort.start[vocab];
  const uint32_t i0 = p * pc.ch, i1 = i0 + pc.ch;
  if (i1 >= total) return;
  const uint32_t row = sort.entries[i1].row;
  if (sort.entries[i1 - 1].row != row || sort.start[row] < i0) return;
  const uint32_t q = (sort.start[row + 1] - 1) / pc.ch;  // the run's last piece, after p
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const uint64_t c = (uint64_t)(blockIdx.x - p * pc.segs) * kSeg + lane * 8;
  const int n = c >= pc.dim ? 0 : (pc.dim - c < 8 ? (int)(pc.dim - c) : 8);
  const uint32_t count = q - p + 1, per = (count + kJoinWaves - 1) / kJoinWaves;
  const uint32_t a = p + w * per, z = a + per < q + 1 ? a + per : q + 1;
  G8 acc = {};
  for (uint32_t k = a; k < z; ++k) {
    const G8 g = load8_upto<DT_F32>((const char*)pc.partials, ((uint64_t)k * 2 + (k == p)) * pc.dim + c, n);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc.v[i] += g.v[i];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) share[w * kSeg + lane * 8 + i] = acc.v[i];
  __syncthreads();
  if (w != 0) return;
  for (int k = 1; k < kJoinWaves; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc.v[i] += share[k * kSeg + lane * 8 + i];
  store_row<DO>(dw, row, c, n, scale, accumulate, acc);
}

template <int DI, int DO>
hipError_t embedding_grad_typed(const Rows& dout, uint64_t vocab, const TokenSort& sort, const Pieces& pc, float scale,
                                bool accumulate, const Rows& dw, hipStream_t stream) {
  const uint64_t units = (uint64_t)pc.n * pc.segs + (accumulate ? 0 : vocab);
  constexpr int waves = kThreads / 64;
  if (units) {
    hipLaunchKernelGGL((embedding_grad_kernel<DI, DO>), dim3((unsigned)((units + waves - 1) / waves)), dim3(kThreads),
                       0, stream, dout, vocab, sort, pc, scale, accumulate, dw);
    const hipError_t e = launch_status(stream);
    if (e != hipSuccess || pc.n < 2) return e;
  }
  hipLaunchKernelGGL((embedding_join_kernel<DO>), dim3((pc.n - 1) * pc.segs), dim3(kJoinWaves * 64),
                     kJoinWaves * kSeg * sizeof(float), stream, vocab, sort, pc, scale, accumulate, dw);
  return launch_status(stream);
}

template <int DI>
hipError_t embedding_grad_to(const Rows& dout, uint64_t vocab, const TokenSort& sort, const Pieces& pc, float scale,
                             bool accumulate, const Rows& dw, hipStream_t stream) {
  switch (dw.dt) {
    case DT_F32: return embedding_grad_typed<DI, DT_F32>(dout, vocab, sort, pc, scale, accumulate, dw, stream);
    case DT_F16: return embedding_grad_typed<DI, DT_F16>(dout, vocab, sort, pc, scale, accumulate, dw, stream);
    default: return embedding_grad_typed<DI, DT_BF16>(dout, vocab, sort, pc, scale, accumulate, dw, stream);
  }
}

}  // namespace

hipError_t launch_embedding(const Rows& weight, uint64_t vocab, uint64_t dim, const void* ids, bool ids64,
                            uint64_t tokens, float scale, const Rows& out, hipStream_t stream) {
  if (tokens == 0) return hipSuccess;
  switch (weight.dt) {
    case DT_F32: return embedding_to<DT_F32>(weight, vocab, dim, ids, ids64, tokens, scale, out, stream);
    case DT_F16: return embedding_to<DT_F16>(weight, vocab, dim, ids, ids64, tokens, scale, out, stream);
    default: return embedding_to<DT_BF16>(weight, vocab, dim, ids, ids64, tokens, scale, out, stream);
  }
}

hipError_t launch_token_sort(const void* ids, bool ids64, uint64_t tokens, uint64_t vocab, int64_t padding,
                             const TokenSort& sort, hipStream_t stream) {
  uint32_t R = (uint32_t)((vocab + 255) / 256);
  if (R < 16) R = 16;
  if (R > kSortMaxRows) R = kSortMaxRows;
  int rbits = 1;
  while ((1u << rbits) < R) ++rbits;
  const uint32_t grid = (uint32_t)((vocab + R - 1) / R);
  const size_t lds = ((size_t)kSortWaves * R + kSortWaves) * sizeof(uint32_t);
  hipLaunchKernelGGL(token_sort_kernel, dim3(grid), dim3(kSortThreads), lds, stream, ids, ids64, (uint32_t)tokens,
                     (uint32_t)vocab, padding, R, rbits, sort);
  return launch_status(stream);
}

uint64_t embedding_piece(uint64_t tokens, uint64_t dim) {
  // short pieces while that gives wavefronts to fill the chip (16 per CU),
  // longer ones for long batches: fewer partials
  const uint64_t segs = (dim + kSeg - 1) / kSeg;
  uint64_t ch = kBatch;
  while (ch < 64 && (tokens + ch - 1) / ch * segs > 4096) ch *= 2;
  return ch;
}

hipError_t launch_embedding_grad(const Rows& dout, uint64_t tokens, uint64_t vocab, uint64_t dim,
                                 const TokenSort& sort, float* partials, float scale, bool accumulate,
                                 const Rows& dweight, hipStream_t stream) {
  const uint64_t ch = embedding_piece(tokens, dim);
  const Pieces pc{(uint32_t)ch, (uint32_t)((tokens + ch - 1) / ch), (uint32_t)((dim + kSeg - 1) / kSeg), dim, partials};
  if (accumulate && tokens == 0) return hipSuccess;
  switch (dout.dt) {
    case DT_F32: return embedding_grad_to<DT_F32>(dout, vocab, sort, pc, scale, accumulate, dweight, stream);
    case DT_F16: return embedding_grad_to<DT_F16>(dout, vocab, sort, pc, scale, accumulate, dweight, stream);
    default: return embedding_grad_to<DT_BF16>(dout, vocab, sort, pc, scale, accumulate, dweight, stream);
  }
}

}  // namespace rar
