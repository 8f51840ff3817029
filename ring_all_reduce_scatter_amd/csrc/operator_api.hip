// C-ABI of the operators next to the rings (argument checks, workspace
// layout, launches): global gradient norm and clipping, embedding lookup
// and gradient, layer norm forward and backward.  Kernels live in
// clip_kernels.hip, embedding_kernels.hip and layernorm_kernels.hip.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <vector>

#include "operator_launch.hpp"
#include "rar.h"

using namespace rar;

namespace {

constexpr size_t kAlign = 256;
// A launch holds fewer than 2^32 threads.
constexpr uint64_t kMaxTiles = (1ull << 24) - 16;  // workgroups of 256
constexpr uint64_t kMaxUnits = (1ull << 26) - 16;  // wavefronts
constexpr size_t kMaxTokens = (size_t)1 << 30, kMaxDim = 0x7fffffff;

size_t es_of(int dt) { return dt == RAR_F32 ? 4 : 2; }
bool dt_ok(int dt) { return dt == RAR_F32 || dt == RAR_F16 || dt == RAR_BF16; }
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
int hip_rc(hipError_t e) { return e == hipSuccess ? RAR_OK : RAR_EHIP; }

// A byte range, or (stride not 0) rows of `row` bytes every `stride` bytes in
// it; an output may coincide with inputs of the same `same` tag (not 0),
// element for element.
struct Range {
  uintptr_t p;
  size_t bytes;
  bool written;
  int same;
  size_t stride = 0, row = 0;
};

// Whether the rows of one range lie in the gaps between the other's: columns
// of one matrix.
bool in_gaps(const Range& a, const Range& b) {
  if (a.stride == 0 || a.stride != b.stride) return false;
  const size_t off = a.p < b.p ? (b.p - a.p) % a.stride : (a.p - b.p) % a.stride;
  const size_t first = a.p < b.p ? a.row : b.row, second = a.p < b.p ? b.row : a.row;
  return first <= off && second <= a.stride - off;
}

// Every written range apart from every other one, but for those of equal
// tag, address and length.  The ranges are few: one call's tensors.
int check_ranges(const Range* a, int n) {
  for (int i = 0; i < n; ++i)
    for (int j = 0; j < i; ++j) {
      if (!a[i].written && !a[j].written) continue;
      if (a[i].bytes == 0 || a[j].bytes == 0) continue;
      if (a[i].p >= a[j].p + a[j].bytes || a[j].p >= a[i].p + a[i].bytes) continue;
      if (a[i].same && a[i].same == a[j].same && a[i].p == a[j].p && a[i].bytes == a[j].bytes) continue;
      if (in_gaps(a[i], a[j])) continue;
      return RAR_EOVERLAP;
    }
  return RAR_OK;
}

// Elements from the first of the first row to the last of the last; false
// if the byte range does not fit the address space.
bool rows_bytes(size_t rows, size_t dim, size_t stride, size_t es, size_t* bytes) {
  *bytes = 0;
  if (rows == 0) return true;
  size_t span = 0;
  if (__builtin_mul_overflow(rows - 1, stride, &span) || __builtin_add_overflow(span, dim, &span) ||
      __builtin_mul_overflow(span, es, bytes))
    return false;
  return *bytes < ((size_t)1 << 48);
}

int check_ptr(const void* p, size_t align) {
  if (!p) return RAR_EOVERLAP;
  return (uintptr_t)p & (align - 1) ? RAR_EALIGN : RAR_OK;
}

// ------------------------------------------------------------------ norm and clip

// Workspace: table, descriptors, partial sums, then the counts of arrived
// workgroups and the factor.
uint64_t clip_tiles(size_t count, int dt) { return (count + clip_tile_elems(dt) - 1) / clip_tile_elems(dt); }
struct ClipLayout {
  size_t descs, partials, result, bytes;
};
bool clip_layout(const size_t* counts, size_t nt, ClipLayout* l) {
  uint64_t ntiles = 0;  // at most: as if every tensor were binary32
  for (size_t t = 0; t < nt; ++t) {
    if (counts[t] >= (size_t)1 << 43) return false;
    ntiles += clip_tiles(counts[t], RAR_F32);
  }
  if (nt >= (size_t)1 << 24 || ntiles > 0x7fffffffull) return false;
  l->descs = round_up((5 * nt + 1) * sizeof(uint64_t), kAlign);
  l->partials = l->descs + round_up((size_t)ntiles * kClipDescBytes, kAlign);
  l->result = l->partials + kClipMaxBlocks * sizeof(double);
  l->bytes = l->result + kClipCountBytes + kAlign;
  return true;
}

ClipSet clip_set(const rar_grad_plan* p) {
  char* ws = (char*)p->workspace;
  char* result = ws + p->result_offset;
  return ClipSet{ws + p->desc_offset, ws + p->partial_offset, result, result + kClipCountBytes, p->ntiles};
}

// Whether norm lies among the tensors of a set.
bool in_set(const rar_grad_set& s, const float* norm) {
  const uintptr_t a = (uintptr_t)norm;
  auto meets = [a](const void* p, size_t bytes) {
    return a < (uintptr_t)p + bytes && (uintptr_t)p < a + sizeof(float);
  };
  for (size_t t = 0; t < s.ntensors; ++t) {
    if (s.counts[t] == 0) continue;
    if (meets(s.grads[t], s.counts[t] * es_of(s.dtypes[t])) ||
        (s.outs && meets(s.outs[t], s.counts[t] * es_of(s.out_dtypes[t]))))
      return true;
  }
  return false;
}

// The norm is written while the workspace is read and before a clip reads the
// tensors, so it has to lie apart from them.  (The plan holds the tensors'
// addresses in the workspace, which the host does not read: they are compared
// where the caller keeps them.)
int check_plan(const rar_grad_plan* p, int norm_type, double scale, const float* norm) {
  if (!p || !p->workspace || ((uintptr_t)p->workspace & 15u) || p->ntiles > kMaxTiles) return RAR_EINVAL;
  if (p->desc_offset == 0 || (p->desc_offset | p->partial_offset | p->result_offset) & 15u) return RAR_EINVAL;
  if (norm_type != RAR_NORM_L2 && norm_type != RAR_NORM_MAX) return RAR_EINVAL;
  if (!std::isfinite(scale)) return RAR_EINVAL;
  const int rc = check_ptr(norm, sizeof(float));
  if (rc) return rc;
  const Range r[] = {{(uintptr_t)norm, sizeof(float), true, 0},
                     {(uintptr_t)p->workspace, p->result_offset + kClipCountBytes + kAlign, true, 0}};
  if (check_ranges(r, 2)) return RAR_EOVERLAP;
  return p->set && in_set(*p->set, norm) ? RAR_EOVERLAP : RAR_OK;
}

// clips: the set is written, to outs or (NULL) in place; without, its tensors
// are only read and may overlap.
int grad_prepare(void* const* grads, bool clips, void* const* outs, const size_t* counts, const int* dtypes,
                 const int* out_dtypes, size_t nt, void* workspace, size_t ws_bytes, rar_grad_plan* plan,
                 hipStream_t st) {
  if (!plan || (nt && (!grads || !counts || !dtypes)) || (outs && !out_dtypes)) return RAR_EINVAL;
  ClipLayout l;
  if (!clip_layout(counts, nt, &l)) return RAR_EINVAL;
  struct Out {
    uintptr_t p;
    size_t bytes, t;
  };
  std::vector<Out> o;
  for (size_t t = 0; t < nt; ++t) {
    const int odt = outs ? out_dtypes[t] : dtypes[t];
    if (!dt_ok(dtypes[t]) || !dt_ok(odt)) return RAR_EDTYPE;
    if (counts[t] == 0) continue;
    const void* out = outs ? outs[t] : grads[t];
    int rc = check_ptr(grads[t], es_of(dtypes[t]));
    if (!rc) rc = check_ptr(out, es_of(odt));
    if (rc) return rc;
    if (clips) o.push_back(Out{(uintptr_t)out, counts[t] * es_of(odt), t});
  }
  if (!workspace || ws_bytes < l.bytes) return RAR_EWORKSPACE;
  if ((uintptr_t)workspace & 15u) return RAR_EALIGN;
  // outputs apart from one another and from the workspace; an input apart
  // from the workspace and from every output, but for its own in place
  o.push_back(Out{(uintptr_t)workspace, l.bytes, nt});
  std::sort(o.begin(), o.end(), [](const Out& a, const Out& b) { return a.p < b.p; });
  for (size_t i = 0; i + 1 < o.size(); ++i)
    if (o[i + 1].p - o[i].p < o[i].bytes) return RAR_EOVERLAP;
  for (size_t t = 0; t < nt; ++t) {
    if (counts[t] == 0) continue;
    const uintptr_t a = (uintptr_t)grads[t], b = a + counts[t] * es_of(dtypes[t]);
    // the outputs are apart, so those that reach past a end in order too
    auto it = std::lower_bound(o.begin(), o.end(), a,
                               [](const Out& x, uintptr_t v) { return x.p + x.bytes <= v; });
    for (; it != o.end() && it->p < b; ++it) {
      const bool own = it->t == t && it->p == a && (!outs || out_dtypes[t] == dtypes[t]);
      if (!own) return RAR_EOVERLAP;
    }
  }
  std::vector<uint64_t> tab(5 * nt + 1);
  uint64_t tiles = 0;
  for (size_t t = 0; t < nt; ++t) {
    tab[t] = tiles;
    tiles += clip_tiles(counts[t], dtypes[t]);
    tab[nt + 1 + t] = (uint64_t)(uintptr_t)grads[t];
    tab[2 * nt + 1 + t] = (uint64_t)(uintptr_t)(outs ? outs[t] : grads[t]);
    tab[3 * nt + 1 + t] = counts[t];
    tab[4 * nt + 1 + t] = (uint64_t)dtypes[t] | (uint64_t)(outs ? out_dtypes[t] : dtypes[t]) << 8;
  }
  if (tiles > kMaxTiles) return RAR_ENOTSUP;
  tab[nt] = tiles;
  rar_grad_plan p{};
  p.workspace = workspace;
  p.desc_offset = l.descs;
  p.partial_offset = l.partials;
  p.result_offset = l.result;
  p.ntiles = tiles;
  p.clips = clips;
  if (tiles) {
    const uint64_t none[kClipCountBytes / sizeof(uint64_t)] = {};  // no workgroup has arrived
    int rc = hip_rc(launch_fill_u64((uint64_t*)((char*)workspace + l.result), none,
                                    (int)(kClipCountBytes / sizeof(uint64_t)), st));
    if (!rc) rc = hip_rc(launch_fill_u64((uint64_t*)workspace, tab.data(), (int)tab.size(), st));
    if (!rc) rc = hip_rc(launch_clip_desc((const uint64_t*)workspace, (char*)workspace + l.descs, nt, tiles, st));
    if (rc) return rc;
  }
  *plan = p;
  return RAR_OK;
}

}  // namespace

extern "C" {

size_t rar_grad_workspace_bytes(const size_t* counts, size_t ntensors) {
  ClipLayout l;
  if ((ntensors && !counts) || !clip_layout(counts, ntensors, &l)) return 0;
  return l.bytes;
}

int rar_grad_prepare(void* const* grads, void* const* outs, const size_t* counts, const int* dtypes,
                     const int* out_dtypes, size_t ntensors, void* workspace, size_t ws_bytes, rar_grad_plan* plan,
                     void* stream) {
  try {
    return grad_prepare(grads, true, outs, counts, dtypes, out_dtypes, ntensors, workspace, ws_bytes, plan,
                        (hipStream_t)stream);
  } catch (...) {  // host memory for the checks or the table
    return RAR_EHIP;
  }
}

int rar_grad_prepare_norm(void* const* grads, const size_t* counts, const int* dtypes, size_t ntensors,
                          void* workspace, size_t ws_bytes, rar_grad_plan* plan, void* stream) {
  try {
    return grad_prepare(grads, false, nullptr, counts, dtypes, nullptr, ntensors, workspace, ws_bytes, plan,
                        (hipStream_t)stream);
  } catch (...) {
    return RAR_EHIP;
  }
}

int rar_grad_norm(const rar_grad_plan* plan, int norm_type, double scale, float* norm, void* stream) {
  const int rc = check_plan(plan, norm_type, scale, norm);
  if (rc) return rc;
  return hip_rc(launch_grad_norm(clip_set(plan), norm_type, scale, norm, (hipStream_t)stream));
}

int rar_grad_clip(const rar_grad_plan* plan, int norm_type, double scale, double max_norm, float* norm,
                  void* stream) {
  const int rc = check_plan(plan, norm_type, scale, norm);
  if (rc) return rc;
  if (!plan->clips || !(max_norm >= 0.0)) return RAR_EINVAL;
  return hip_rc(launch_grad_clip(clip_set(plan), norm_type, scale, max_norm, norm, (hipStream_t)stream));
}

// ------------------------------------------------------------------ embedding

namespace {

int embedding_sizes(size_t tokens, size_t vocab, size_t dim) {
  if (vocab == 0 || dim == 0) return RAR_EINVAL;
  if (tokens > kMaxTokens || vocab > 0x7fffffff || dim > kMaxDim) return RAR_ENOTSUP;
  return RAR_OK;
}

// Workspace: row starts, sorted tokens, partial sums, counts.
struct EmbeddingLayout {
  size_t entries, partials, counts, ncounts, bytes;
};
EmbeddingLayout embedding_layout(size_t tokens, size_t vocab, size_t dim) {
  EmbeddingLayout l;
  const size_t ch = embedding_piece(tokens, dim);
  l.entries = round_up((vocab + 1) * sizeof(uint32_t), kAlign);
  l.partials = l.entries + round_up(tokens * sizeof(TokenEntry), kAlign);
  const size_t pieces = (tokens + ch - 1) / ch, columns = round_up(dim, 512);
  l.counts = l.partials + pieces * 2 * columns * sizeof(float);
  l.ncounts = pieces * 2 * (columns / 512);
  l.bytes = l.counts + round_up(l.ncounts * sizeof(uint32_t), kAlign);
  return l;
}

}  // namespace

int rar_embedding_forward(const void* weight, size_t weight_stride, int weight_dtype, size_t vocab, size_t dim,
                          const void* ids, int id_type, size_t tokens, float scale, void* out, size_t out_stride,
                          int out_dtype, void* stream) {
  int rc = embedding_sizes(tokens, vocab, dim);
  if (rc) return rc;
  if (!dt_ok(weight_dtype) || !dt_ok(out_dtype) || (id_type != RAR_I32 && id_type != RAR_I64)) return RAR_EDTYPE;
  size_t wb, ob;
  if (weight_stride < dim || out_stride < dim || !rows_bytes(vocab, dim, weight_stride, es_of(weight_dtype), &wb) ||
      !rows_bytes(tokens, dim, out_stride, es_of(out_dtype), &ob))
    return RAR_EINVAL;
  if (tokens == 0) return RAR_OK;
  const size_t ib = id_type == RAR_I64 ? 8 : 4;
  if ((rc = check_ptr(weight, es_of(weight_dtype))) || (rc = check_ptr(ids, ib)) ||
      (rc = check_ptr(out, es_of(out_dtype))))
    return rc;
  const size_t oe = es_of(out_dtype), we = es_of(weight_dtype);
  const Range r[] = {{(uintptr_t)out, ob, true, 0, out_stride * oe, dim * oe},
                     {(uintptr_t)weight, wb, false, 0, weight_stride * we, dim * we},
                     {(uintptr_t)ids, ib * tokens, false, 0}};
  if ((rc = check_ranges(r, 3))) return rc;
  if (tokens * ((dim + 511) / 512) > 0xfffffff0ull) return RAR_ENOTSUP;  // numbered in 32 bits
  return hip_rc(launch_embedding(Rows{(char*)weight, weight_stride, weight_dtype}, vocab, dim, ids,
                                 id_type == RAR_I64, tokens, scale, Rows{(char*)out, out_stride, out_dtype},
                                 (hipStream_t)stream));
}

size_t rar_embedding_workspace_bytes(size_t tokens, size_t vocab, size_t dim) {
  if (embedding_sizes(tokens, vocab, dim)) return 0;
  return embedding_layout(tokens, vocab, dim).bytes;
}

int rar_embedding_backward(const void* dout, size_t dout_stride, int dout_dtype, const void* ids, int id_type,
                           size_t tokens, size_t vocab, size_t dim, float scale, int64_t padding_id, int accumulate,
                           void* dweight, size_t dweight_stride, int dweight_dtype, void* workspace, size_t ws_bytes,
                           void* stream) {
  int rc = embedding_sizes(tokens, vocab, dim);
  if (rc) return rc;
  if (!dt_ok(dout_dtype) || !dt_ok(dweight_dtype) || (id_type != RAR_I32 && id_type != RAR_I64)) return RAR_EDTYPE;
  size_t db, wb;
  if (dweight_stride < dim || !rows_bytes(tokens, dim, dout_stride, es_of(dout_dtype), &db) ||
      !rows_bytes(vocab, dim, dweight_stride, es_of(dweight_dtype), &wb))
    return RAR_EINVAL;
  const size_t ib = id_type == RAR_I64 ? 8 : 4;
  if (tokens && ((rc = check_ptr(dout, es_of(dout_dtype))) || (rc = check_ptr(ids, ib)))) return rc;
  if ((rc = check_ptr(dweight, es_of(dweight_dtype)))) return rc;
  const size_t need = rar_embedding_workspace_bytes(tokens, vocab, dim);
  if (!workspace || ws_bytes < need) return RAR_EWORKSPACE;
  if ((uintptr_t)workspace & 15u) return RAR_EALIGN;
  const size_t we = es_of(dweight_dtype), de = es_of(dout_dtype);
  const Range r[] = {{(uintptr_t)dweight, wb, true, 0, dweight_stride * we, dim * we},
                     {(uintptr_t)workspace, need, true, 0},
                     {(uintptr_t)dout, db, false, 0, dout_stride * de, dim * de},
                     {(uintptr_t)ids, ib * tokens, false, 0}};
  if ((rc = check_ranges(r, 4))) return rc;
  const EmbeddingLayout l = embedding_layout(tokens, vocab, dim);
  const size_t pieces = (tokens + embedding_piece(tokens, dim) - 1) / embedding_piece(tokens, dim);
  if (pieces * ((dim + 511) / 512) + embedding_zero_waves(vocab, dim, dweight_dtype) > kMaxUnits) return RAR_ENOTSUP;
  char* base = (char*)workspace;
  EmbeddingGrad a{};
  a.dout = Rows{(char*)dout, dout_stride, dout_dtype};
  a.dweight = Rows{(char*)dweight, dweight_stride, dweight_dtype};
  a.ids = ids;
  a.tokens = tokens;
  a.vocab = vocab;
  a.dim = dim;
  a.padding = padding_id;
  a.sort = TokenSort{(uint32_t*)base, (TokenEntry*)(base + l.entries), (uint32_t*)(base + l.counts), l.ncounts};
  a.partials = (float*)(base + l.partials);
  a.scale = scale;
  a.ids64 = id_type == RAR_I64;
  a.accumulate = accumulate != 0;
  return hip_rc(launch_embedding_grad(a, (hipStream_t)stream));
}

// ------------------------------------------------------------------ layer norm

int rar_layernorm_forward(const void* x, size_t x_stride, const void* weight, const void* bias, size_t rows,
                          size_t dim, int dtype, int weight_dtype, float eps, void* y, size_t y_stride, float* mean,
                          float* rstd, void* stream) {
  if (!dt_ok(dtype) || !dt_ok(weight_dtype)) return RAR_EDTYPE;
  if (dim > kMaxDim) return RAR_ENOTSUP;
  size_t xb, yb;
  if (dim == 0 || y_stride < dim || !(eps >= 0.0f) || !rows_bytes(rows, dim, x_stride, es_of(dtype), &xb) ||
      !rows_bytes(rows, dim, y_stride, es_of(dtype), &yb))
    return RAR_EINVAL;
  if (rows == 0) return RAR_OK;
  int rc;
  const size_t ws = es_of(weight_dtype);
  if ((rc = check_ptr(x, es_of(dtype))) || (rc = check_ptr(y, es_of(dtype))) ||
      (weight && (rc = check_ptr(weight, ws))) || (bias && (rc = check_ptr(bias, ws))) ||
      (mean && (rc = check_ptr(mean, 4))) || (rstd && (rc = check_ptr(rstd, 4))))
    return rc;
  const size_t es = es_of(dtype);
  const Range r[] = {{(uintptr_t)y, yb, true, 1, y_stride * es, dim * es},
                     {(uintptr_t)x, xb, false, x_stride == y_stride ? 1 : 0, x_stride * es, dim * es},
                     {(uintptr_t)weight, weight ? dim * ws : 0, false, 0},
                     {(uintptr_t)bias, bias ? dim * ws : 0, false, 0},
                     {(uintptr_t)mean, mean ? rows * 4 : 0, true, 0},
                     {(uintptr_t)rstd, rstd ? rows * 4 : 0, true, 0}};
  if ((rc = check_ranges(r, 6))) return rc;
  return hip_rc(launch_layernorm(Rows{(char*)x, x_stride, dtype}, weight, bias, weight_dtype, rows, dim, eps,
                                 Rows{(char*)y, y_stride, dtype}, mean, rstd, (hipStream_t)stream));
}

size_t rar_layernorm_workspace_bytes(size_t rows, size_t dim) {
  if (dim == 0 || dim > kMaxDim) return 0;
  return round_up(layernorm_splits(rows) * 2 * dim * sizeof(float), kAlign);
}

int rar_layernorm_backward(const void* dy, size_t dy_stride, const void* x, size_t x_stride, const void* weight,
                           const float* mean, const float* rstd, size_t rows, size_t dim, int dtype,
                           int weight_dtype, void* dx, size_t dx_stride, void* dweight, void* dbias, int accumulate,
                           void* workspace, size_t ws_bytes, void* stream) {
  if (!dt_ok(dtype) || !dt_ok(weight_dtype)) return RAR_EDTYPE;
  size_t yb, xb, db = 0;
  const size_t es = es_of(dtype), ws = es_of(weight_dtype);
  if (dim > kMaxDim) return RAR_ENOTSUP;
  if (dim == 0 || !rows_bytes(rows, dim, dy_stride, es, &yb) ||
      !rows_bytes(rows, dim, x_stride, es, &xb) || (dx && (dx_stride < dim || !rows_bytes(rows, dim, dx_stride, es, &db))))
    return RAR_EINVAL;
  int rc;
  if (rows && ((rc = check_ptr(dy, es)) || (rc = check_ptr(x, es)) || (rc = check_ptr(mean, 4)) ||
               (rc = check_ptr(rstd, 4))))
    return rc;
  if ((weight && (rc = check_ptr(weight, ws))) || (dx && (rc = check_ptr(dx, es))) ||
      (dweight && (rc = check_ptr(dweight, ws))) || (dbias && (rc = check_ptr(dbias, ws))))
    return rc;
  const bool sums = dweight || dbias;
  const size_t need = sums ? rar_layernorm_workspace_bytes(rows, dim) : 0;
  if (sums && (!workspace || ws_bytes < need)) return RAR_EWORKSPACE;
  if (sums && ((uintptr_t)workspace & 15u)) return RAR_EALIGN;
  const Range r[] = {{(uintptr_t)dx, db, true, 1, dx_stride * es, dim * es},
                     {(uintptr_t)dy, yb, false, dy_stride == dx_stride ? 1 : 0, dy_stride * es, dim * es},
                     {(uintptr_t)x, xb, false, x_stride == dx_stride ? 1 : 0, x_stride * es, dim * es},
                     {(uintptr_t)weight, weight ? dim * ws : 0, false, 0},
                     {(uintptr_t)mean, rows * 4, false, 0},
                     {(uintptr_t)rstd, rows * 4, false, 0},
                     {(uintptr_t)dweight, dweight ? dim * ws : 0, true, 0},
                     {(uintptr_t)dbias, dbias ? dim * ws : 0, true, 0},
                     {(uintptr_t)workspace, need, true, 0}};
  if ((rc = check_ranges(r, 9))) return rc;
  LayernormGrad a{};
  a.dy = Rows{(char*)dy, dy_stride, dtype};
  a.x = Rows{(char*)x, x_stride, dtype};
  a.dx = Rows{(char*)dx, dx_stride, dtype};
  a.weight = weight;
  a.mean = mean;
  a.rstd = rstd;
  a.dweight = dweight;
  a.dbias = dbias;
  a.partials = (float*)workspace;
  a.wdt = weight_dtype;
  a.accumulate = accumulate != 0;
  return hip_rc(launch_layernorm_grad(a, rows, dim, (hipStream_t)stream));
}

}  // extern "C"
