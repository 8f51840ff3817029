// Host-side launchers of the operators next to the rings: global gradient
// norm and clipping, embedding, activation checkpoints, layer norm, gated
// feed-forward (internal to librar.so).  As in
// launch.hpp every launcher enqueues asynchronously on `stream`.
#pragma once

#include "checkpoint.hpp"
#include "launch.hpp"

namespace rar {

struct Rows {  // rows of `dim` elements, `stride` elements apart
  char* p;
  uint64_t stride;
  int dt;
};

// -------------------------------------------------------------- norm and clip (clip_kernels.hip)

// A prepared tensor set: where its pieces lie in the workspace.
struct ClipSet {
  const void* descs;   // one 32-byte descriptor per tile
  void* partials;      // kClipMaxBlocks doubles
  void* counts;        // kClipCountBytes: arrived workgroups, zero between launches
  void* factor;        // the last clip's factor (binary32)
  uint64_t ntiles;
};
constexpr uint32_t kClipTileBytes = 16384;  // of input per tile
__host__ __device__ constexpr uint32_t clip_tile_elems(int dt) { return kClipTileBytes / (dt == DT_F32 ? 4 : 2); }
constexpr uint32_t kClipMaxBlocks = 256;   // workgroups of the norm launch
constexpr uint32_t kClipDescBytes = 32;
constexpr uint32_t kClipCountBytes = 2048;
// Words of the table that launch_clip_desc reads: per tensor its first tile
// (and, after the last, the tile count), then per tensor the input address,
// the output address, the count and the types (input | output << 8).
hipError_t launch_clip_desc(const uint64_t* table, void* descs, uint64_t ntensors, uint64_t ntiles,
                            hipStream_t stream);
// *norm <- |scale| * norm of the whole set.
hipError_t launch_grad_norm(const ClipSet& set, int kind, double scale, float* norm, hipStream_t stream);
// The same, then every output <- round(input * scale * min(1, max_norm / (norm + 1e-6))).
hipError_t launch_grad_clip(const ClipSet& set, int kind, double scale, double max_norm, float* norm,
                            hipStream_t stream);

// -------------------------------------------------------------- embedding (embedding_kernels.hip)

hipError_t launch_embedding(const Rows& weight, uint64_t vocab, uint64_t dim, const void* ids, bool ids64,
                            uint64_t tokens, float scale, const Rows& out, hipStream_t stream);

// The tokens sorted by table row, ascending within a row: row v's are
// entries[start[v] .. start[v+1]) (start holds vocab + 1 words).
struct TokenEntry {
  uint32_t token, row;
};
// The sort also clears the counts that the gradient's launch begins with.
struct TokenSort {
  uint32_t* start;
  TokenEntry* entries;
  uint32_t* counts;
  uint64_t ncounts;
};
// Entries that one wavefront of the gradient takes; partials holds two rows
// of dim floats, rounded up to 512, for each such piece, counts two words
// for each piece and 512 columns.
uint64_t embedding_piece(uint64_t tokens, uint64_t dim);
// Wavefronts that zero the rows without tokens.
uint64_t embedding_zero_waves(uint64_t vocab, uint64_t dim, int dt);
struct EmbeddingGrad {
  Rows dout, dweight;
  const void* ids;
  uint64_t tokens, vocab, dim;
  int64_t padding;
  TokenSort sort;
  float* partials;
  float scale;
  bool ids64, accumulate;
};
hipError_t launch_embedding_grad(const EmbeddingGrad& a, hipStream_t stream);

// -------------------------------------------------------------- activation checkpoints (checkpoint_kernels.hip)

hipError_t launch_ckpt_pack(const Rows& x, uint64_t rows, uint64_t dim, void* ckpt, hipStream_t stream);
hipError_t launch_ckpt_unpack(const void* ckpt, uint64_t rows, uint64_t dim, const Rows& out, hipStream_t stream);

// -------------------------------------------------------------- layer norm (layernorm_kernels.hip)

// ckpt: where x's checkpoint is written, or NULL.
hipError_t launch_layernorm(const Rows& x, const void* weight, const void* bias, int wdt, uint64_t rows, uint64_t dim,
                            float eps, const Rows& y, float* mean, float* rstd, void* ckpt, hipStream_t stream);
// Row groups whose sums of the weight's and bias's gradients are kept apart
// in the workspace (2 * splits * dim floats) before they are added.
uint64_t layernorm_splits(uint64_t rows);
struct LayernormGrad {
  Rows dy, x, dx;
  Checkpoint ck;  // of x, in place of x
  const void* weight;
  const float* mean;
  const float* rstd;
  void* dweight;
  void* dbias;
  float* partials;
  int wdt;
  bool accumulate;
};
hipError_t launch_layernorm_grad(const LayernormGrad& a, uint64_t rows, uint64_t dim, hipStream_t stream);

// -------------------------------------------------------------- gated feed-forward (gated_ff_kernels.hip)

// saved: 0 nothing, 1 the projections in the activations' type (gate, up), 2
// their checkpoints (cgate, cup).
struct FfForward {
  Rows x, wgate, wup, h, gate, up;
  Checkpoint cgate, cup;
  uint64_t rows, dim, hidden;
  int dt, act, saved;
};
hipError_t launch_gated_ff(const FfForward& f, hipStream_t stream);

// Workspace of the backward pass: dg, du (rows x pitch elements each), copies
// of x and the weights (rows of copy_pitch; 0: none), then the partial sums of
// split products.
struct FfWorkspace {
  uint64_t pitch, du, x, copy_pitch, wgate, wup, partials, bytes;
};
FfWorkspace ff_workspace(uint64_t rows, uint64_t dim, uint64_t hidden, int dt);
struct FfBackward {
  Rows dh, x, wgate, wup, gate, up, dx, dwgate, dwup;
  Checkpoint cgate, cup;
  char* ws;
  uint64_t rows, dim, hidden;
  int dt, wdt, act, saved;
  bool accumulate;
};
hipError_t launch_gated_ff_grad(const FfBackward& b, hipStream_t stream);
// Workgroups of the smallest tiles over m x n outputs: what launches have to hold.
uint64_t ff_tile_count(uint64_t m, uint64_t n);

}  // namespace rar
