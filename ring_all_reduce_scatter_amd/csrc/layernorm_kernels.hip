// Layer norm forward and backward for gfx950.
//
//   mu = mean x,  r = 1 / sqrt(mean (x - mu)^2 + eps),  h = (x - mu) r,  y = round(h w + b)
//   g = dy w,     dx = round(r (g - mean g - h mean(g h)))
//   dw = round(sum over rows of dy h [+ dw]),   db = round(sum over rows of dy [+ db])
//
// All statistics and sums are binary32; the variance is taken about the
// mean, not as a difference of moments.  The sums over rows are formed in a
// fixed order: each of the row groups on its own, then the groups in order.
//
// A row stays in the registers of NT lanes, V vectors a lane, from its load
// to its store, so memory is read and written once: 16 lanes for short rows,
// a wavefront, or two, four or eight of them.  Rows too long for that go
// through the loops at the end of this file, which read a row once per pass.
// The lanes per row follow from the row's length alone.  Both directions are
// bound by memory for batches, by launch latency for few rows.  Times on one
// MI355X, inputs cold: forward 16,384 x 4096 f16 46 us (5.8 TB/s of 268 MB),
// one row of 4096 bf16 3.1 us; 16,384 x 4096 bf16 with its checkpoint 61 to 66 us
// (336 MB, 5.4 TB/s), backward from it 67 to 76 and 4.3 (340 MB, 5.0 TB/s);
// backward 16,384 x 8192 bf16 144 us (139 and 5 for the partial rows; 5.8 TB/s of
// 839 MB), 2047 x 1001 f32 7.3 and 3.5 us.
// Measured and left out: a contiguous range of rows per workgroup instead of
// every n-th (forward 55 us, backward 151), ordinary loads instead of
// streaming ones (50 and 153), 16 wavefronts of half the columns backward
// (156).  The loops for longer rows are far from that: forward 2048 x 32,768
// bf16 218 us (42 at the copy rate), backward 366 (63), backward 4096 x 12,288
// f32 295 (95).
#include <algorithm>
#include <type_traits>

#include "checkpoint.hpp"
#include "operator_launch.hpp"
#include "row_access.hpp"

namespace rar {
namespace {

constexpr int kWaves = kThreads / 64;

// ------------------------------------------------------------------ rows in registers

// K sums over the NT lanes of a row; every lane receives them.  16 lanes are
// a DPP row, 64 a wavefront.  Of more, lds holds 2 * (NT / 64) * K floats of
// the row's own; consecutive calls alternate between its halves (turn), so
// one barrier a call is enough: a wavefront writes a half again only after a
// barrier that all readers of its last contents have passed.
template <int NT, int K>
__device__ __forceinline__ void row_sums(float* v, float* lds, int& turn) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = NT == 16 ? dpp_row_sum(v[k]) : wave_sum(v[k]);
  if constexpr (NT > 64) {
    constexpr int NW = NT / 64;
    float* half = lds + (turn & 1) * NW * K;
    ++turn;
    const int lane = threadIdx.x & 63, w = (int)(threadIdx.x >> 6) % NW;
    if (lane == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) half[w * K + k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float s = half[k];
#pragma unroll
      for (int i = 1; i < NW; ++i) s += half[i * K + k];
      v[k] = s;
    }
  }
}

// A row's number in its workgroup: the same register for all lanes of a
// wavefront, unless the wavefront carries several rows.
template <int NT>
__device__ __forceinline__ uint32_t row_slot() {
  const uint32_t slot = threadIdx.x / NT;
  return NT < 64 ? slot : (uint32_t)__builtin_amdgcn_readfirstlane(slot);
}

// A lane's share of a row of dim elements: V vectors of E, NT vectors
// apart, as far as the row has whole vectors, and one of the dim % E
// elements after them.  A lane without a vector (or element) holds zeros in
// its place; valid() and tail() tell.
template <int DT, int NT, int V>
struct RowShape {
  static constexpr int E = vec_elems<DT, DT>();
  uint32_t lane;  // among the row's NT
  uint32_t nvec, ntail;
  __device__ __forceinline__ RowShape(uint32_t l, uint64_t dim)
      : lane(l), nvec((uint32_t)(dim / E)), ntail((uint32_t)(dim % E)) {}
  __device__ __forceinline__ bool valid(int j) const { return j * NT + lane < nvec; }
  __device__ __forceinline__ uint32_t col(int j) const { return (j * NT + lane) * E; }
  __device__ __forceinline__ bool tail() const { return lane < ntail; }
  __device__ __forceinline__ uint32_t tail_col() const { return nvec * E + lane; }
};

// A row as loaded, and as binary32.
template <int DT, int V>
struct RowRaw {
  VecRaw<DT, vec_elems<DT, DT>()> v[V];
  float t;
};
template <int E, int V>
struct RowF {
  VecF<E> v[V];
  float t;
};

template <int DT, int NT, int V>
__device__ __forceinline__ void load_row(const RowShape<DT, NT, V>& sh, const char* row, RowRaw<DT, V>& x) {
  constexpr int E = RowShape<DT, NT, V>::E;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (sh.valid(j)) x.v[j] = load_raw<DT, E, true>(row, sh.col(j));
    else x.v[j] = VecRaw<DT, E>{};
  }
  x.t = 0.0f;
  if (sh.tail()) x.t = load_elem<DT>(row, sh.tail_col());
}
// Whether every row begins on a cache line.  Such rows are stored
// write-through (st16_wt), others with nontemporal stores: on 65,536 rows
// the forward pass of 1000 f32 columns takes 97 us so, 108 with all rows on
// 16-byte boundaries write-through; on 16,384 rows the backward pass of 8192
// bf16 columns 140 against 146 with nontemporal stores alone.
template <int DT>
__device__ __forceinline__ bool rows_on_lines(const Rows& r) {
  return (((uint64_t)r.p | r.stride * DtypeSize<DT>::value) & 127) == 0;
}
template <int DT, int NT, int V>
__device__ __forceinline__ void store_row(const RowShape<DT, NT, V>& sh, char* row, bool lines,
                                          const RowF<vec_elems<DT, DT>(), V>& x) {
  constexpr int E = RowShape<DT, NT, V>::E;
  if (NT >= 64 && lines) {  // uniform, as is the row
    const WtRange range = wt_range(row, sh.nvec * 16);
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (sh.valid(j)) st16_wt(range, sh.col(j) * DtypeSize<DT>::value, pack_vec<DT, E>(x.v[j]));
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (sh.valid(j)) store_vec<DT, E>(row, sh.col(j), x.v[j]);
  }
  if (sh.tail()) store_elem<DT>(row, sh.tail_col(), x.t);
}
template <int DT, int V>
__device__ __forceinline__ RowF<vec_elems<DT, DT>(), V> unpack_row(const RowRaw<DT, V>& x) {
  RowF<vec_elems<DT, DT>(), V> f;
#pragma unroll
  for (int j = 0; j < V; ++j) f.v[j] = unpack<DT, vec_elems<DT, DT>()>(x.v[j]);
  f.t = x.t;
  return f;
}

// A weight or bias vector of type WT in a row's shape.
template <int WT, int DT, int NT, int V>
__device__ __forceinline__ void load_weight_as(const RowShape<DT, NT, V>& sh, const char* w,
                                               RowF<vec_elems<DT, DT>(), V>& f) {
  constexpr int E = RowShape<DT, NT, V>::E;
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (sh.valid(j))
#pragma unroll
      for (int h = 0; h < E; h += 4) {
        const VecF<4> q = load_vec<WT, 4>(w, sh.col(j) + h);
#pragma unroll
        for (int i = 0; i < 4; ++i) f.v[j].v[h + i] = q.v[i];
      }
  if (sh.tail()) f.t = load_elem<WT>(w, sh.tail_col());
}
template <int DT, int NT, int V>
__device__ __forceinline__ void load_weight(const RowShape<DT, NT, V>& sh, const void* w, int wdt, float missing,
                                            RowF<vec_elems<DT, DT>(), V>& f) {
  f = {};
  if (w == nullptr) {
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int i = 0; i < RowShape<DT, NT, V>::E; ++i) f.v[j].v[i] = missing;
    f.t = missing;
  } else if (wdt == DT_F32) {
    load_weight_as<DT_F32>(sh, (const char*)w, f);
  } else if (wdt == DT_F16) {
    load_weight_as<DT_F16>(sh, (const char*)w, f);
  } else {
    load_weight_as<DT_BF16>(sh, (const char*)w, f);
  }
}

// Writes a row's checkpoint from its registers, called by all lanes of the
// wavefront.  A block of 32 columns is 32 / E consecutive lanes' vectors, so
// its largest value is a maximum over them; lanes past the row's vectors hold
// zeros and fill the last block up.  Where elements follow the last vector,
// the block that holds them goes to the first 16 lanes, two elements each,
// which read it again (from the cache).
template <int DT, int NT, int V>
__device__ __forceinline__ void checkpoint_row(const RowShape<DT, NT, V>& sh, const char* x, uint64_t dim, bool live,
                                               const RowF<vec_elems<DT, DT>(), V>& v, uint8_t* codes, uint8_t* exps) {
  constexpr int E = RowShape<DT, NT, V>::E;
  static_assert(NT % (kCkptBlock / E) == 0, "a block lies in one turn of the row's lanes");
  // columns of the blocks made of vectors
  const uint32_t whole = (uint32_t)(sh.ntail ? dim / kCkptBlock : (dim + kCkptBlock - 1) / kCkptBlock) * kCkptBlock;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const uint32_t m = group_max_u32<kCkptBlock / E>(vec_absmax(v.v[j]));
    uint32_t col = sh.col(j);
    asm volatile("" : "+v"(col));  // compared anew for each row: the masks of all vectors take too many registers
    if (live && col < whole) ckpt_store<E>(codes, exps, col, m, v.v[j]);
  }
  if (sh.ntail) {  // uniform
    const uint32_t c = whole + sh.lane;
    float a = 0.0f, b = 0.0f;
    if (sh.lane < 16 && c < dim) a = load_elem<DT>(x, c);
    if (sh.lane < 16 && c + 16 < dim) b = load_elem<DT>(x, c + 16);
    const uint32_t m = group_max_u32<16>(max(absbits(a), absbits(b)));
    if (live && sh.lane < 16) {
      const BfpScale sc = bfp_scale(m, 8);
      codes[c] = (uint8_t)(sc.nan ? 0 : (int)bfp_q(a, sc.k, 127.0f));
      codes[c + 16] = (uint8_t)(sc.nan ? 0 : (int)bfp_q(b, sc.k, 127.0f));
      if (sh.lane == 0) exps[whole / kCkptBlock] = (uint8_t)(m >> 23);
    }
  }
}

// Forward: a workgroup of NT * RB lanes carries RB rows at a time and
// strides over the rows; the next row's loads are issued before this one's
// sums.  CK: the rows' checkpoints are written too.
template <int DT, int NT, int V, int RB, bool CK>
__global__ __launch_bounds__(NT * RB) void layernorm_row_kernel(Rows x, const void* __restrict__ weight,
                                                                      const void* __restrict__ bias, int wdt,
                                                                      uint64_t rows, uint64_t dim, float eps, Rows y,
                                                                      float* __restrict__ mean,
                                                                      float* __restrict__ rstd, Checkpoint ck) {
  extern __shared__ float lds[];
  constexpr int E = vec_elems<DT, DT>(), ES = DtypeSize<DT>::value;
  const uint32_t slot = row_slot<NT>();
  const RowShape<DT, NT, V> sh(threadIdx.x % NT, dim);
  float* red = lds + slot * (2 * NT / 64);
  int turn = 0;
  const uint64_t step = (uint64_t)gridDim.x * RB;
  const bool lines = rows_on_lines<DT>(y);
  uint64_t r = (uint64_t)blockIdx.x * RB + slot;
  RowRaw<DT, V> raw;
  load_row(sh, x.p + (r < rows ? r : rows - 1) * x.stride * ES, raw);
  RowF<E, V> w, b;
  load_weight(sh, weight, wdt, 1.0f, w);
  load_weight(sh, bias, wdt, 0.0f, b);
  // every wavefront of the workgroup makes the same number of turns
  for (uint64_t r0 = (uint64_t)blockIdx.x * RB; r0 < rows; r0 += step, r += step) {
    RowF<E, V> v = unpack_row<DT, V>(raw);
    if (r0 + step < rows) load_row(sh, x.p + (r + step < rows ? r + step : rows - 1) * x.stride * ES, raw);
    if constexpr (CK) {
      const uint64_t q = r < rows ? r : rows - 1;
      checkpoint_row(sh, x.p + q * x.stride * ES, dim, r < rows, v, ck.code_row(q), ck.exp_row(q));
    }
    float s = v.t;
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int i = 0; i < E; ++i) s += v.v[j].v[i];
    row_sums<NT, 1>(&s, red, turn);
    const float mu = s / (float)dim;
    v.t -= mu;
    float q = sh.tail() ? v.t * v.t : 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
#pragma unroll
      for (int i = 0; i < E; ++i) v.v[j].v[i] -= mu;
      if (sh.valid(j))
#pragma unroll
        for (int i = 0; i < E; ++i) q = __builtin_fmaf(v.v[j].v[i], v.v[j].v[i], q);
    }
    row_sums<NT, 1>(&q, red, turn);
    const float rs = 1.0f / __builtin_sqrtf(q / (float)dim + eps);
    if (r < rows) {
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < E; ++i) v.v[j].v[i] = __builtin_fmaf(v.v[j].v[i] * rs, w.v[j].v[i], b.v[j].v[i]);
      v.t = __builtin_fmaf(v.t * rs, w.t, b.t);
      store_row(sh, y.p + r * y.stride * ES, lines, v);
      if (sh.lane == 0) {
        if (mean) mean[r] = mu;
        if (rstd) rstd[r] = rs;
      }
    }
  }
}

// An element of the backward pass's x, from its rows or from its checkpoint.
template <int DT, bool CK>
__device__ __forceinline__ float x_elem(const LayernormGrad& a, uint64_t r, uint64_t c) {
  if constexpr (CK) return ckpt_elem(a.ck.code_row(r), a.ck.exp_row(r), c);
  else return load_elem<DT>(a.x.p, r * a.x.stride + c);
}

// A row of x as loaded from its checkpoint.
template <int DT, int V>
struct CkptRow {
  CkptRaw<vec_elems<DT, DT>()> v[V];
  float t;
};
template <int DT, int NT, int V>
__device__ __forceinline__ void load_ckpt_row(const RowShape<DT, NT, V>& sh, const Checkpoint& ck, uint64_t r,
                                              CkptRow<DT, V>& x) {
  constexpr int E = RowShape<DT, NT, V>::E;
  const uint8_t *codes = ck.code_row(r), *exps = ck.exp_row(r);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (sh.valid(j)) x.v[j] = ckpt_load<E>(codes, exps, sh.col(j));
    else x.v[j] = CkptRaw<E>{};
  }
  x.t = 0.0f;
  if (sh.tail()) x.t = ckpt_elem(codes, exps, sh.tail_col());
}
template <int DT, int V>
__device__ __forceinline__ RowF<vec_elems<DT, DT>(), V> unpack_row(const CkptRow<DT, V>& x) {
  RowF<vec_elems<DT, DT>(), V> f;
#pragma unroll
  for (int j = 0; j < V; ++j) f.v[j] = ckpt_unpack(x.v[j]);
  f.t = x.t;
  return f;
}

// Sums of dy h and dy over all rows for 64 columns, a column a lane, each
// wavefront of the workgroup every W-th row, the wavefronts in order; the
// result goes straight to dw and db.
template <int DT, bool CK>
__device__ __forceinline__ void grad_columns(const LayernormGrad& a, uint64_t rows, uint64_t dim, uint64_t c0,
                                             uint32_t W, float* lds) {
  const uint32_t lane = threadIdx.x & 63, w = (uint32_t)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint64_t c = c0 + lane;
  float dw = 0.0f, db = 0.0f;
  if (c < dim) {
#pragma unroll 8
    for (uint64_t r = w; r < rows; r += W) {
      const float dy = load_elem<DT>(a.dy.p, r * a.dy.stride + c);
      const float h = (x_elem<DT, CK>(a, r, c) - a.mean[r]) * a.rstd[r];
      dw = __builtin_fmaf(dy, h, dw);
      db += dy;
    }
  }
  lds[w * 128 + lane] = dw;
  lds[w * 128 + 64 + lane] = db;
  __syncthreads();
  if (w > 1) return;  // wavefront 0 finishes dw, wavefront 1 db
  void* out = w ? a.dbias : a.dweight;
  if (!out || c >= dim) return;
  float v = 0.0f;
  for (uint32_t k = 0; k < W; ++k) v += lds[k * 128 + w * 64 + lane];
  if (a.accumulate) v += load_elem_dt((const char*)out, c, a.wdt);
  store_elem_dt((char*)out, c, a.wdt, v);
}

// Backward: the same walk over the rows with the sums of dy h and dy over
// the workgroup's rows kept in registers; at the end the RB row slots are
// added (through LDS) and stored as the workgroup's partial sums.
// Of few rows the workgroups carry only dx (`partial` false), and those past
// `groups` take the sums column by column, in the same launch.
// CK: x comes from its checkpoint, a byte an element and one more for 32.
template <int DT, int NT, int V, int RB, bool CK>
__global__ __launch_bounds__(NT * RB) void layernorm_grad_row_kernel(LayernormGrad a, uint64_t rows,
                                                                       uint64_t dim, uint32_t groups, bool partial) {
  extern __shared__ float lds[];
  if (blockIdx.x >= groups) {
    grad_columns<DT, CK>(a, rows, dim, (uint64_t)(blockIdx.x - groups) * 64, NT * RB / 64, lds);
    return;
  }
  constexpr int E = vec_elems<DT, DT>(), ES = DtypeSize<DT>::value;
  const uint32_t slot = row_slot<NT>();
  const RowShape<DT, NT, V> sh(threadIdx.x % NT, dim);
  float* red = lds + slot * (4 * NT / 64);
  int turn = 0;
  const uint64_t step = (uint64_t)groups * RB;
  const bool lines = rows_on_lines<DT>(a.dx);
  uint64_t r = (uint64_t)blockIdx.x * RB + slot;
  std::conditional_t<CK, CkptRow<DT, V>, RowRaw<DT, V>> rx;
  RowRaw<DT, V> ry;
  float mu_next, rs_next;
  auto fetch = [&](uint64_t row) {
    const uint64_t q = row < rows ? row : rows - 1;
    if constexpr (CK) load_ckpt_row(sh, a.ck, q, rx);
    else load_row(sh, a.x.p + q * a.x.stride * ES, rx);
    load_row(sh, a.dy.p + q * a.dy.stride * ES, ry);
    mu_next = a.mean[q];
    rs_next = a.rstd[q];
  };
  fetch(r);
  RowF<E, V> w, dw = {}, db = {};
  load_weight(sh, a.weight, a.wdt, 1.0f, w);
  for (uint64_t r0 = (uint64_t)blockIdx.x * RB; r0 < rows; r0 += step, r += step) {
    const float mu = mu_next, rs = rs_next;
    const bool live = r < rows;
    // where the row has no element dy is zero, so it adds to no sum
    RowF<E, V> h = unpack_row<DT, V>(rx), g = unpack_row<DT, V>(ry);
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int i = 0; i < E; ++i) h.v[j].v[i] = (h.v[j].v[i] - mu) * rs;
    h.t = (h.t - mu) * rs;
    if (live) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (sh.valid(j))
#pragma unroll
          for (int i = 0; i < E; ++i) {
            dw.v[j].v[i] = __builtin_fmaf(g.v[j].v[i], h.v[j].v[i], dw.v[j].v[i]);
            db.v[j].v[i] += g.v[j].v[i];
          }
      dw.t = __builtin_fmaf(g.t, h.t, dw.t);
      db.t += g.t;
    }
    g.t *= w.t;
    float s[2] = {g.t, sh.tail() ? g.t * h.t : 0.0f};
#pragma unroll
    for (int j = 0; j < V; ++j) {
#pragma unroll
      for (int i = 0; i < E; ++i) g.v[j].v[i] *= w.v[j].v[i];
      if (sh.valid(j))
#pragma unroll
        for (int i = 0; i < E; ++i) {
          s[0] += g.v[j].v[i];
          s[1] = __builtin_fmaf(g.v[j].v[i], h.v[j].v[i], s[1]);
        }
    }
    if (r0 + step < rows) fetch(r + step);
    if (a.dx.p == nullptr) continue;  // uniform
    row_sums<NT, 2>(s, red, turn);
    const float mg = s[0] / (float)dim, mgh = s[1] / (float)dim;
    if (live) {
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < E; ++i) g.v[j].v[i] = rs * __builtin_fmaf(-h.v[j].v[i], mgh, g.v[j].v[i] - mg);
      g.t = rs * __builtin_fmaf(-h.t, mgh, g.t - mg);
      store_row(sh, a.dx.p + r * a.dx.stride * ES, lines, g);
    }
  }
  if (!partial) return;
  // the row slots' sums, halving the slots each time: the upper half hands
  // its sums to the lower through LDS (in a fixed order like any other)
  if constexpr (RB > 1) {
    constexpr int kCols = NT * (V * E + 1);
    float* sum = lds + RB * 4 * NT / 64;  // [RB / 2][2][kCols]
#pragma unroll
    for (int half = RB / 2; half >= 1; half /= 2) {
      const bool gives = slot >= (uint32_t)half && slot < 2u * half;
      // consecutive lanes, consecutive banks
      float* at = sum + (slot % half) * 2 * kCols + sh.lane;
      if (gives) {
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
          for (int i = 0; i < E; ++i) {
            at[(j * E + i) * NT] = dw.v[j].v[i];
            at[(j * E + i) * NT + kCols] = db.v[j].v[i];
          }
        at[V * E * NT] = dw.t;
        at[V * E * NT + kCols] = db.t;
      }
      __syncthreads();
      if (slot < (uint32_t)half) {
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
          for (int i = 0; i < E; ++i) {
            dw.v[j].v[i] += at[(j * E + i) * NT];
            db.v[j].v[i] += at[(j * E + i) * NT + kCols];
          }
        dw.t += at[V * E * NT];
        db.t += at[V * E * NT + kCols];
      }
      __syncthreads();
    }
  }
  if (slot != 0) return;
  float* out = a.partials + (uint64_t)blockIdx.x * 2 * dim;
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (sh.valid(j))
#pragma unroll
      for (int h = 0; h < E; h += 4) {
        u32x4 x, y;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] = __float_as_uint(dw.v[j].v[h + i]);
          y[i] = __float_as_uint(db.v[j].v[h + i]);
        }
        *(u32x4_any*)(out + sh.col(j) + h) = x;
        *(u32x4_any*)(out + dim + sh.col(j) + h) = y;
      }
  if (sh.tail()) {
    out[sh.tail_col()] = dw.t;
    out[dim + sh.tail_col()] = db.t;
  }
}

// Adds the partial rows: 64 columns of dw (blockIdx.y = 0) or db per
// workgroup, each wavefront every kJoinWaves-th partial row, the wavefronts
// in order.  The workgroups of more columns than one grid dimension holds
// (2^32 threads) lie in blockIdx.z.
constexpr int kJoinWaves = 16;
constexpr uint64_t kJoinGridX = 1 << 20;

__global__ __launch_bounds__(kJoinWaves * 64) void layernorm_join_kernel(LayernormGrad a, uint64_t splits,
                                                                          uint64_t dim) {
  extern __shared__ float lds[];  // [kJoinWaves][64]
  void* out = blockIdx.y ? a.dbias : a.dweight;
  if (!out) return;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const uint64_t c = (blockIdx.z * kJoinGridX + blockIdx.x) * 64 + lane;
  const float* p = a.partials + blockIdx.y * dim + c;
  float v = 0.0f;
  if (c < dim)
#pragma unroll 8
    for (uint64_t k = w; k < splits; k += kJoinWaves) v += p[k * 2 * dim];
  lds[w * 64 + lane] = v;
  __syncthreads();
  if (w != 0 || c >= dim) return;
#pragma unroll
  for (int k = 1; k < kJoinWaves; ++k) v += lds[k * 64 + lane];
  if (a.accumulate) v += load_elem_dt((const char*)out, c, a.wdt);
  store_elem_dt((char*)out, c, a.wdt, v);
}

// ------------------------------------------------------------------ rows of any length

// Sum over the workgroup; every lane receives it.
__device__ __forceinline__ float block_sum(float v, float* lds) {
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) s += lds[w];
  return s;
}

__device__ __forceinline__ float weight_at(const void* w, int wdt, uint64_t i, float missing) {
  return w ? load_elem_dt((const char*)w, i, wdt) : missing;
}

template <int DT>
__global__ __launch_bounds__(kThreads) void layernorm_kernel(Rows x, const void* __restrict__ weight,
                                                              const void* __restrict__ bias, int wdt, uint64_t rows,
                                                              uint64_t dim, float eps, Rows y,
                                                              float* __restrict__ mean, float* __restrict__ rstd) {
  extern __shared__ float red[];
  for (uint64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const char* xr = x.p + r * x.stride * DtypeSize<DT>::value;
    char* yr = y.p + r * y.stride * DtypeSize<DT>::value;
    float s = 0.0f;
    for (uint64_t c = threadIdx.x; c < dim; c += kThreads) s += load_elem<DT>(xr, c);
    const float mu = block_sum(s, red) / (float)dim;
    float q = 0.0f;
    for (uint64_t c = threadIdx.x; c < dim; c += kThreads) {
      const float d = load_elem<DT>(xr, c) - mu;
      q = __builtin_fmaf(d, d, q);
    }
    const float rs = 1.0f / __builtin_sqrtf(block_sum(q, red) / (float)dim + eps);
    for (uint64_t c = threadIdx.x; c < dim; c += kThreads) {
      const float h = (load_elem<DT>(xr, c) - mu) * rs;
      store_elem<DT>(yr, c, __builtin_fmaf(h, weight_at(weight, wdt, c, 1.0f), weight_at(bias, wdt, c, 0.0f)));
    }
    if (threadIdx.x == 0) {
      if (mean) mean[r] = mu;
      if (rstd) rstd[r] = rs;
    }
  }
}

// Sums over one row group of dy h and dy, a column per lane.
template <int DT, bool CK>
__global__ __launch_bounds__(kThreads) void layernorm_dw_part_kernel(LayernormGrad a, uint64_t rows, uint64_t dim,
                                                                      uint64_t per) {
  const uint64_t c = (uint64_t)blockIdx.x * kThreads + threadIdx.x;
  if (c >= dim) return;
  const uint64_t r0 = blockIdx.y * per, r1 = r0 + per < rows ? r0 + per : rows;
  float dw = 0.0f, db = 0.0f;
  for (uint64_t r = r0; r < r1; ++r) {
    const float dy = load_elem<DT>(a.dy.p, r * a.dy.stride + c);
    const float h = (x_elem<DT, CK>(a, r, c) - a.mean[r]) * a.rstd[r];
    dw = __builtin_fmaf(dy, h, dw);
    db += dy;
  }
  a.partials[(uint64_t)blockIdx.y * 2 * dim + c] = dw;
  a.partials[((uint64_t)blockIdx.y * 2 + 1) * dim + c] = db;
}

template <int DT, bool CK>
__global__ __launch_bounds__(kThreads) void layernorm_dx_kernel(LayernormGrad a, uint64_t rows, uint64_t dim) {
  extern __shared__ float red[];
  for (uint64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const char* yr = a.dy.p + r * a.dy.stride * DtypeSize<DT>::value;
    char* dr = a.dx.p + r * a.dx.stride * DtypeSize<DT>::value;
    const float mu = a.mean[r], rs = a.rstd[r];
    float sg = 0.0f, sgh = 0.0f;
    for (uint64_t c = threadIdx.x; c < dim; c += kThreads) {
      const float g = load_elem<DT>(yr, c) * weight_at(a.weight, a.wdt, c, 1.0f);
      sg += g;
      sgh = __builtin_fmaf(g, (x_elem<DT, CK>(a, r, c) - mu) * rs, sgh);
    }
    const float mg = block_sum(sg, red) / (float)dim;
    const float mgh = block_sum(sgh, red) / (float)dim;
    for (uint64_t c = threadIdx.x; c < dim; c += kThreads) {
      const float g = load_elem<DT>(yr, c) * weight_at(a.weight, a.wdt, c, 1.0f);
      const float h = (x_elem<DT, CK>(a, r, c) - mu) * rs;
      store_elem<DT>(dr, c, rs * (g - mg - h * mgh));
    }
  }
}

unsigned row_grid(uint64_t rows) { return (unsigned)(rows < 65536 ? rows : 65536); }

// ------------------------------------------------------------------ launches

// Workgroups of the backward pass: one per CU, since each leaves a partial
// row of 2 * dim floats, as far as there are rows for its slots.
constexpr uint64_t kGradGroups = 256;
constexpr uint64_t kFewRows = 512, kFewBytes = 2 << 20;
// From a checkpoint fewer: its bytes come from memory, and a column's rows wait
// for one another (forward and backward of 512 x 1024 bf16 34 us by columns, 20
// with partial rows; 128 x 512 f32 17.6 and 20.6).
constexpr uint64_t kFewHeldRows = 128;
uint64_t grad_groups(uint64_t rows, int rb) { return std::min<uint64_t>(kGradGroups, (rows + rb - 1) / rb); }

template <int DT, int NT, int V, int RB, bool CK>
hipError_t forward_rows(const Rows& x, const void* weight, const void* bias, int wdt, uint64_t rows, uint64_t dim,
                        float eps, const Rows& y, float* mean, float* rstd, void* ckpt, hipStream_t stream) {
  // twelve wavefronts per CU: 46.6 us for 16,384 x 4096 in binary16, against
  // 50.6 with eight and 48.8 with sixteen
  constexpr uint64_t waves = NT * RB / 64, per_cu = waves < 12 ? 12 / waves : 1;
  const uint64_t groups = std::min<uint64_t>((rows + RB - 1) / RB, 256 * per_cu);
  hipLaunchKernelGGL((layernorm_row_kernel<DT, NT, V, RB, CK>), dim3((unsigned)groups), dim3(NT * RB),
                     RB * 2 * NT / 64 * sizeof(float), stream, x, weight, bias, wdt, rows, dim, eps, y, mean, rstd,
                     CK ? Checkpoint(ckpt, rows, dim) : Checkpoint());
  return launch_status(stream);
}

template <int DT, bool CK>
hipError_t layernorm_dt(const Rows& x, const void* weight, const void* bias, int wdt, uint64_t rows, uint64_t dim,
                        float eps, const Rows& y, float* mean, float* rstd, void* ckpt, hipStream_t stream) {
  const uint64_t vecs = dim / vec_elems<DT, DT>();
#define RAR_FORWARD(NT, V, RB) \
  return forward_rows<DT, NT, V, RB, CK>(x, weight, bias, wdt, rows, dim, eps, y, mean, rstd, ckpt, stream)
  if (vecs <= 16) RAR_FORWARD(16, 1, 16);
  if (vecs <= 32) RAR_FORWARD(16, 2, 16);
  if (vecs <= 64) RAR_FORWARD(16, 4, 16);
  if (vecs <= 128) RAR_FORWARD(64, 2, 4);
  if (vecs <= 256) RAR_FORWARD(64, 4, 4);
  // Between, three vectors on each of two wavefronts' lanes: 67 million values
  // in rows of 2560 bf16 46.7 us (60 with 256 lanes, whose second vectors most
  // lanes lack), of 2816 46.8 (56).  In binary32 the gain ends sooner: 1200
  // columns 91 us (98), 1344 91.7 (92.8), 1440 93 (90).
  if (vecs <= (DT == DT_F32 ? 340 : 384)) RAR_FORWARD(128, 3, 2);
  if (vecs <= 512) RAR_FORWARD(256, 2, 1);
  if (vecs <= 1024) RAR_FORWARD(256, 4, 1);
  if (vecs <= 2048) RAR_FORWARD(512, 4, 1);
  if constexpr (CK) {
    // Longer rows leave no registers for the blocks: they are packed on their
    // own, before y, which may be written over x.
    const hipError_t e = launch_ckpt_pack(x, rows, dim, ckpt, stream);
    if (e != hipSuccess) return e;
    return layernorm_dt<DT, false>(x, weight, bias, wdt, rows, dim, eps, y, mean, rstd, nullptr, stream);
  } else {
    if constexpr (DT == DT_F32)
      if (vecs <= 4096) RAR_FORWARD(512, 8, 1);
    hipLaunchKernelGGL((layernorm_kernel<DT>), dim3(row_grid(rows)), dim3(kThreads), kWaves * sizeof(float), stream, x,
                       weight, bias, wdt, rows, dim, eps, y, mean, rstd);
    return launch_status(stream);
  }
#undef RAR_FORWARD
}

hipError_t join_partials(const LayernormGrad& a, uint64_t splits, uint64_t dim, hipStream_t stream) {
  if (!a.dweight && !a.dbias) return hipSuccess;
  const uint64_t groups = (dim + 63) / 64;
  const dim3 grid((unsigned)std::min(groups, kJoinGridX), 2, (unsigned)((groups + kJoinGridX - 1) / kJoinGridX));
  hipLaunchKernelGGL(layernorm_join_kernel, grid, dim3(kJoinWaves * 64), kJoinWaves * 64 * sizeof(float), stream, a,
                     splits, dim);
  return launch_status(stream);
}

template <int DT, int NT, int V, int RB, bool CK>
hipError_t backward_rows(const LayernormGrad& a, uint64_t rows, uint64_t dim, hipStream_t stream) {
  const uint64_t groups = grad_groups(rows, RB);
  const size_t lds = (RB * 4 * NT / 64 + RB / 2 * 2 * NT * (V * vec_elems<DT, DT>() + 1)) * sizeof(float);
  const size_t column_lds = NT * RB / 64 * 128 * sizeof(float);
  const bool sums = a.dweight || a.dbias;
  auto launch = [&](uint64_t row_groups, uint64_t columns, bool partial) {
    hipLaunchKernelGGL((layernorm_grad_row_kernel<DT, NT, V, RB, CK>), dim3((unsigned)(row_groups + columns)),
                       dim3(NT * RB), std::max(lds, column_lds), stream, a, rows, dim, (uint32_t)row_groups, partial);
    return launch_status(stream);
  };
  if (rows > (CK ? kFewHeldRows : kFewRows) || rows * dim * DtypeSize<DT>::value > kFewBytes || !sums) {
    const hipError_t e = launch(groups, 0, sums);
    return e != hipSuccess ? e : join_partials(a, groups, dim, stream);
  }
  // Few rows: a second reading of x and dy (from the caches) by columns costs
  // less than a second launch that adds partial rows (256 x 1024 bf16 9.5 us
  // against 12.0), while a column's rows are few (512 x 8192: 37 us against
  // 16).  It comes first where dx is written over dy or x.
  const uint64_t columns = (dim + 63) / 64;
  if (!a.dx.p) return launch(0, columns, false);
  if (a.dx.p != a.dy.p && a.dx.p != a.x.p) return launch(groups, columns, false);
  const hipError_t e = launch(0, columns, false);
  return e != hipSuccess ? e : launch(groups, 0, false);
}

template <int DT, bool CK>
hipError_t layernorm_grad_dt(const LayernormGrad& a, uint64_t rows, uint64_t dim, hipStream_t stream) {
  if (rows == 0) return join_partials(a, 0, dim, stream);
  const uint64_t vecs = dim / vec_elems<DT, DT>();
  if (vecs <= 16) return backward_rows<DT, 16, 1, 64, CK>(a, rows, dim, stream);
  // (with codes and exponents to unpack, 64 rows do not fit the registers)
  if (vecs <= 32) return backward_rows<DT, 16, 2, CK ? 32 : 64, CK>(a, rows, dim, stream);
  if (vecs <= 64) return backward_rows<DT, 16, 4, 32, CK>(a, rows, dim, stream);
  if (vecs <= 128) return backward_rows<DT, 64, 2, 8, CK>(a, rows, dim, stream);
  if (vecs <= 256) return backward_rows<DT, 64, 4, 8, CK>(a, rows, dim, stream);
  // 2560 bf16 columns 74 us (87 with 256 lanes), 1200 binary32 140 (148).
  if (vecs <= 384) return backward_rows<DT, 128, 3, 4, CK>(a, rows, dim, stream);
  if (vecs <= 512) return backward_rows<DT, 256, 2, 2, CK>(a, rows, dim, stream);
  if (vecs <= 1024) return backward_rows<DT, 256, 4, 2, CK>(a, rows, dim, stream);
  if (vecs <= 2048) return backward_rows<DT, 512, 4, 1, CK>(a, rows, dim, stream);
  hipError_t e = hipSuccess;
  // dw and db first: dx may be written over dy or x
  if (a.dweight || a.dbias) {
    const uint64_t splits = std::min(layernorm_splits(rows), (rows + 63) / 64);
    hipLaunchKernelGGL((layernorm_dw_part_kernel<DT, CK>), dim3((unsigned)((dim + kThreads - 1) / kThreads), (unsigned)splits),
                       dim3(kThreads), 0, stream, a, rows, dim, (rows + splits - 1) / splits);
    if ((e = launch_status(stream)) != hipSuccess) return e;
    if ((e = join_partials(a, splits, dim, stream)) != hipSuccess) return e;
  }
  if (a.dx.p) {
    hipLaunchKernelGGL((layernorm_dx_kernel<DT, CK>), dim3(row_grid(rows)), dim3(kThreads), kWaves * sizeof(float), stream,
                       a, rows, dim);
    e = launch_status(stream);
  }
  return e;
}

}  // namespace

namespace {

template <bool CK>
hipError_t forward_any(const Rows& x, const void* weight, const void* bias, int wdt, uint64_t rows, uint64_t dim,
                       float eps, const Rows& y, float* mean, float* rstd, void* ckpt, hipStream_t stream) {
  switch (x.dt) {
    case DT_F32: return layernorm_dt<DT_F32, CK>(x, weight, bias, wdt, rows, dim, eps, y, mean, rstd, ckpt, stream);
    case DT_F16: return layernorm_dt<DT_F16, CK>(x, weight, bias, wdt, rows, dim, eps, y, mean, rstd, ckpt, stream);
    default: return layernorm_dt<DT_BF16, CK>(x, weight, bias, wdt, rows, dim, eps, y, mean, rstd, ckpt, stream);
  }
}

template <bool CK>
hipError_t backward_any(const LayernormGrad& a, uint64_t rows, uint64_t dim, hipStream_t stream) {
  switch (a.dy.dt) {
    case DT_F32: return layernorm_grad_dt<DT_F32, CK>(a, rows, dim, stream);
    case DT_F16: return layernorm_grad_dt<DT_F16, CK>(a, rows, dim, stream);
    default: return layernorm_grad_dt<DT_BF16, CK>(a, rows, dim, stream);
  }
}

}  // namespace

hipError_t launch_layernorm(const Rows& x, const void* weight, const void* bias, int wdt, uint64_t rows, uint64_t dim,
                            float eps, const Rows& y, float* mean, float* rstd, void* ckpt, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  return ckpt ? forward_any<true>(x, weight, bias, wdt, rows, dim, eps, y, mean, rstd, ckpt, stream)
              : forward_any<false>(x, weight, bias, wdt, rows, dim, eps, y, mean, rstd, nullptr, stream);
}

uint64_t layernorm_splits(uint64_t rows) {
  return std::max<uint64_t>(1, std::min<uint64_t>(kGradGroups, rows));
}

hipError_t launch_layernorm_grad(const LayernormGrad& a, uint64_t rows, uint64_t dim, hipStream_t stream) {
  return a.ck.codes ? backward_any<true>(a, rows, dim, stream) : backward_any<false>(a, rows, dim, stream);
}

}  // namespace rar
