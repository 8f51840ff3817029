// The matrix products of the gated feed-forward block on gfx950's matrix
// instructions: C[q][p] = sum over k of Q(q, k) P(p, k), where each operand
// lies in memory either by rows of k (KC) or by rows of its own index (the
// weights in dx, x and dg in dW).
//
// A workgroup computes TP columns by TQ rows; a stage of both operands is 128
// bytes of k a row (64 16-bit terms, 32 in binary32), so every type has the
// same layout in LDS.  Two stages alternate: while the wavefronts multiply one,
// the other is on its way.  A wavefront holds TP / WP columns by TQ / WQ
// rows in blocks of 16 x 16: the instructions for them multiply random values
// at 2.08 PFLOP/s where those of 32 x 32 reach 1.79 (power holds the clock down;
// both have 2.46 on zeros).
//
// P is the matrix instruction's first operand, whose index runs over a lane's
// accumulators: 4 (lane / 16) + i for accumulator i.  Forward, two such blocks
// of the weights' rows are read in the order that makes this a lane's 8
// consecutive columns of 32 (from 8 (lane / 16) on), so that a checkpoint's
// codes are whole vectors.
//
// LDS positions are 16-byte chunks.  The chunks of a row are stored under an
// XOR of the row's low bits, so that the lanes of one read hit different
// banks; the loads apply it to their source, since direct loads write LDS in
// lane order.  Rows of the operand's own index are read by the transposing
// LDS load (16 bits), which hands lane i of 16 the i-th of 16 columns and
// four consecutive k.
//
// Bound by the matrix units' rate under power and what the loads leave of it.
// 8192 x 4096 x 11,264 bfloat16 (1.51 TFLOP a pass of two products): forward 1149
// us without kept projections (1.32 PFLOP/s) and 1212 with checkpoints, dx 1201,
// dW 1312, medians; large library products of these layouts reach 1.33-1.53, 1.20-1.40
// and 0.98-1.08 PFLOP/s.  Measured and left out: instructions of 32 x 32 (power),
// stages of 64 bytes a row in four turns (their loads move at half the rate:
// 1418 us where two of 128 took 1319), three to five stages, four wavefronts of
// 128 x 128, tiles of 256 x 128 (1937 us forward: half the products for three
// quarters of the loads; 511 x 2048 x 5632 42 instead of 36), loads of the next
// rows into the L2 ahead (1262-1281 against 1213), a different first k for each
// XCD (no change).
#pragma once

#include <algorithm>
#include <type_traits>
#include <utility>

#include "gated_ff.hpp"

namespace rar {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 h16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 b16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_char;

constexpr int kRow = 128;  // bytes of k a row of a stage

// Stages of binary32 (32 terms each) that are added up one by one; the sums of
// so many are added up after that.  A chain's error grows with the root of its
// length: 4096 random terms are off by 4.1e-7 of their size, in one chain by
// 1.15e-6, for 1.3 % of the time (2048 x 2048 x 5632 forward 802 us instead of
// 796; every 4 stages 2.3e-7 and 828).  In 16 bits the operands' own rounding is a
// thousand times a chain's.
constexpr uint32_t kFoldStages = 16;

// A chunk's terms in binary32 take four instructions, of one term in each of a
// lane quarter's chunks; in 16 bits one takes them all.
template <int DT>
__host__ __device__ constexpr int ff_turns() {
  return DT == DT_F32 ? 4 : 1;
}
template <int DT>
__device__ __forceinline__ f32x4 ff_mfma(u32x4 p, u32x4 q, f32x4 c, int turn) {
  if constexpr (DT == DT_BF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b16x8, p), __builtin_bit_cast(b16x8, q), c, 0, 0,
                                                   0);
  } else if constexpr (DT == DT_F16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h16x8, p), __builtin_bit_cast(h16x8, q), c, 0, 0,
                                                  0);
  } else {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(p[turn]), __uint_as_float(q[turn]), c, 0, 0, 0);
  }
}

// Direct loads are written as assembly because the compiler, which cannot tell
// the two stages apart, would wait for them before the next transposing read
// of LDS (dx of 8192 x 4096 x 11,264 bf16 took 1640 us instead of 1290 when both
// were tried).  They have no output register; the wait for them is ff_meet's.  The nop keeps the five wait
// states that a buffer access needs after a vector instruction wrote its
// scalar registers.
__device__ __forceinline__ void ff_load_lds(u32x4 range, uint32_t off, uint32_t to) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 4\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
               :
               : "v"(off), "s"(range), "s"(to)
               : "memory", "m0");
}
// This wavefront's loads into LDS have landed and its reads of LDS are done,
// and so are all others'.
__device__ __forceinline__ void ff_meet() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" : : : "memory");
}

// f(constant 0) ... f(constant N - 1): array indexes that stay constants.
template <class F, int... I>
__device__ __forceinline__ void ff_each(F f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>()), ...);
}
template <int N, class F>
__device__ __forceinline__ void ff_each(F f) {
  ff_each(f, std::make_integer_sequence<int, N>());
}

// 16 bytes of a row of `total` elements from element e on, zeros past the end:
// read where the row still has 16 bytes and shifted.
template <int ES>
__device__ __forceinline__ u32x4 ff_load_edge(const char* row, uint32_t e, uint32_t total) {
  constexpr uint32_t EC = 16 / ES;
  if (total < EC) {  // uniform: a matrix narrower than a chunk
    u32x4 x = {0, 0, 0, 0};
#pragma unroll
    for (uint32_t j = 0; j < EC; ++j)
      if (e + j < total) {
        if constexpr (ES == 4) x[j] = ((const uint32_t*)row)[e + j];
        else x[j / 2] |= (uint32_t)((const uint16_t*)row)[e + j] << (16 * (j & 1));
      }
    return x;
  }
  const uint32_t at = e < total - EC ? e : total - EC;
  const u32x4 x = *(const u32x4_any*)(row + (uint64_t)at * ES);
  const uint32_t words = (e - at) * ES / 4;  // by which the chunk lies behind what was read
  u32x4 y;
#pragma unroll
  for (uint32_t i = 0; i < 4; ++i) {
    y[i] = 0;
#pragma unroll
    for (uint32_t j = i; j < 4; ++j) y[i] = words == j - i ? x[j] : y[i];
  }
  if constexpr (ES == 2) {
    const uint32_t odd = (e - at) & 1;
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = odd ? y[i] >> 16 | (i < 3 ? y[i + 1] << 16 : 0) : y[i];
  }
  return y;
}

// One operand's share of a stage.  T: rows (KC) or columns of the operand's
// index in the tile.  PAIR: the 32-row halves of each 64 rows belong to two
// matrices (gate and up).  PERM: read in P's order.
//
// Rows of the operand's index past its last are read as its last one, columns
// past the last as anything that may be read: what comes of them is not
// stored.  Terms past the last are zeros in both operands.
template <int DT, bool KC, int T, int NTHR, bool DIRECT, bool PAIR, bool PERM>
struct FfLoader {
  static constexpr int ES = DtypeSize<DT>::value, EC = 16 / ES;  // elements of a chunk
  static constexpr int BK = kRow / ES;
  static constexpr int NI = T * kRow / 16 / NTHR;          // chunks a thread
  static constexpr int CPR = KC ? 8 : T * ES / 16;         // chunks a row of the stage
  static constexpr int RPI = NTHR / CPR;           // rows between a thread's chunks
  static constexpr uint32_t kOut = 0x80000000u;    // past every buffer range: reads as zeros
  static_assert(!PAIR || (KC && (RPI == 32 || RPI % 64 == 0)), "which matrix a chunk belongs to");
  static_assert(KC || CPR >= 16, "chunks that the XOR may exchange");

  // XOR of the chunks of a stage row.  KC: the rows that 16 lanes read (r ... r +
  // 15, or in P's order four each of r, r + 8, r + 16 and r + 24) have 16
  // different places in the 256 bytes of banks: even and odd rows, with eight
  // values of the XOR each.  Otherwise the eight k that 32 lanes of a
  // transposing read take 32 bytes of, or in binary32 two of the lane quarters.
  static __device__ __forceinline__ uint32_t swizzle(uint32_t row) {
    if constexpr (KC) return PERM ? (row >> 1 & 1) | (row >> 2 & 6) : row >> 1 & 7;
    else return ES == 2 ? (row & 3) << 2 | (row >> 2 & 2) : (row >> 2 & 1) << 3;
  }

  uint32_t row;       // of the thread's first chunk
  uint32_t chunk;     // of a KC operand's row, the same for all of the thread's
  uint32_t off[NI];   // bytes from the tile's first row or column
  u32x4 hold[DIRECT ? 1 : NI];

  // Which matrix the thread's i-th chunk belongs to (the same for the whole
  // wavefront), and its row there.
  static __device__ __forceinline__ uint32_t matrix_of(int i) {
    if constexpr (!PAIR) return 0;
    // (64 / CPR rows a wavefront)
    return RPI == 32 ? i & 1 : (uint32_t)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * (64 / CPR) / 32 & 1;
  }
  static __device__ __forceinline__ uint32_t local(uint32_t r) { return PAIR ? (r >> 6) * 32 + (r & 31) : r; }

  // limit: rows (KC) or columns that exist from the tile's first on.
  __device__ __forceinline__ void init(uint64_t limit, uint32_t stride0, uint32_t stride1) {
    row = threadIdx.x / CPR;
    chunk = threadIdx.x % CPR ^ swizzle(row);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const uint32_t r = row + i * RPI, stride = matrix_of(i) ? stride1 : stride0;
      if constexpr (KC) {
        const uint32_t l = local(r);
        off[i] = (l < limit ? l : (uint32_t)limit - 1) * stride + chunk * 16;
      } else {
        const uint32_t e = (threadIdx.x % CPR ^ swizzle(r)) * EC;
        off[i] = r * stride + (e < limit ? e * ES : 0);
      }
    }
  }

  // Asks for the thread's I-th chunk of a stage.  base: the tile's first row (KC)
  // or column at the stage's first term, of either matrix; left: terms from
  // there on (direct: 0 for none of it).  edge: (not direct) chunks may reach
  // past the last column, which is `limit` from the tile's first; before it are
  // `before` columns (KC: terms of the row before the stage).
  template <int I>
  __device__ __forceinline__ void load(const char* base0, const char* base1, uint32_t left, uint32_t stage, bool edge,
                                       uint32_t limit, uint32_t before) {
    const char* b = PAIR && matrix_of(I) ? base1 : base0;
    if constexpr (DIRECT) {
      const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
      const u32x4 range = {(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(uint64_t)b),
                           (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)b >> 32)), 0x7fffffffu,
                           0x00020000u};
      // no branch: the products go on around it
      const uint32_t o = (KC ? chunk * EC : row + I * RPI) < left ? off[I] : kOut;
      ff_load_lds(range, o, stage + (I * NTHR + wave * 64) * 16);
    } else if (left >= BK && !edge) {  // uniform
      hold[I] = *(const u32x4_any*)(b + off[I]);
    } else if constexpr (KC) {
      // the row's terms from `back` before the stage on
      const uint32_t n = left < BK ? left : BK, back = before < EC ? before : EC;
      const char* at = b + off[I] - chunk * 16 - back * ES;
      const u32x4 x = ff_load_edge<ES>(at, chunk * EC + back, n + back);
      hold[I] = chunk * EC < n ? x : (u32x4){0, 0, 0, 0};
    } else {
      const uint32_t r = row + I * RPI, e = (threadIdx.x % CPR ^ swizzle(r)) * EC;
      const uint32_t back = before < EC ? before : EC;
      const uint32_t step = e < limit ? e : 0;
      // past the last term: the stage's first row, made zeros
      const char* at = b + (r < left ? off[I] - step * ES : 0) - back * ES;
      const u32x4 x = ff_load_edge<ES>(at, step + back, limit + back);
      hold[I] = r < left ? x : (u32x4){0, 0, 0, 0};
    }
  }

  // Puts a stage that went through registers into LDS.
  __device__ __forceinline__ void put(lds_char* stage) {
    if constexpr (!DIRECT) {
#pragma unroll
      for (int i = 0; i < NI; ++i)
        *(__attribute__((address_space(3))) u32x4*)(stage + (i * NTHR + threadIdx.x) * 16) = hold[i];
    }
  }

  // Where this lane's fragments begin in a stage, for the tile's rows or
  // columns from `first` (a multiple of 32) on.
  static __device__ __forceinline__ uint32_t fragment_at(uint32_t first) {
    static_assert(!PERM || KC, "P's order is the weights' rows' forward");
    const uint32_t lane = threadIdx.x & 63, p = lane & 15, g = lane >> 4;
    if constexpr (KC) {
      const uint32_t r = PERM ? (p >> 2) * 8 + (p & 3) : p;
      return (first + r) * kRow + (g ^ swizzle(r)) * 16;
    } else if constexpr (ES == 2) {
      // the lane's place among 16 is a k (of four) and four columns (of 16)
      const uint32_t c = lane & 3, k = g * 8 + (p >> 2);
      return k * (T * 2) + ((first / 8 + c / 2) ^ swizzle(k)) * 16 + (c & 1) * 8;
    } else {
      const uint32_t n = first + p, k = g * 4;
      return k * (T * 4) + (n / 4 ^ swizzle(k)) * 16 + (n & 3) * 4;
    }
  }
  // The fragment of the wavefront's `block`-th 16 rows or columns, step ks (four
  // chunks of k).  In P's order block 2 b + 1 is four rows on from block 2 b.
  static __device__ __forceinline__ u32x4 fragment(const lds_char* stage, uint32_t at, int block, int ks) {
    if constexpr (KC) {
      // rows of the same XOR: it depends on bits that this does not change
      const int rows = PERM ? block / 2 * 32 + block % 2 * 4 : block * 16;
      return *(const __attribute__((address_space(3))) u32x4*)(stage + ((at ^ (ks * 64)) + rows * kRow));
    } else if constexpr (ES == 2) {
      // 16 columns are two chunks, on whose bits the XOR acts too; k advances by
      // 32, which it does not see
      typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
      lds_char* p = (lds_char*)stage + ((at ^ block * 32) + ks * 32 * (T * 2));
      const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p));
      const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * (T * 2))));
      return (u32x4){a[0], a[1], b[0], b[1]};
    } else {
      const lds_char* p = stage + ((at ^ block * 64) + ks * 16 * (T * 4));
      u32x4 x;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = *(const __attribute__((address_space(3))) uint32_t*)(p + i * (T * 4));
      return x;
    }
  }
};

// The kernel's one argument where the launch left it.  What only the turn from
// one item to the next and an item's outputs need is read anew from there: kept
// in scalar registers through the products it would not leave enough of them.
typedef const __attribute__((address_space(4))) FfProduct* FfArguments;
__device__ __forceinline__ FfArguments ff_arguments() {
  FfArguments a = (FfArguments)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(a));
  return a;
}

// What a workgroup makes at a time: a tile of an output, over all terms or one
// split of them.
struct FfItem {
  uint64_t m0, n0;
  uint32_t z, part, k_begin, k_end;  // output (dW), output and split, stages
};
// Order of the items: consecutive workgroups go to the 8 XCDs in turn, so each
// XCD gets a contiguous range of the order, which its workgroups go through
// side by side; in it, tiles come in bands of 8 tiles of rows, columns
// slowest, so that the 32 tiles an XCD works on at once share their operands
// through its L2.
struct FfOrder {
  uint32_t next, end, step;
  __device__ __forceinline__ explicit FfOrder(uint32_t items) {
    const uint32_t x = blockIdx.x % 8, base = items / 8, extra = items % 8;
    const uint32_t first = x * base + (x < extra ? x : extra);
    next = first + blockIdx.x / 8;
    end = first + base + (x < extra);
    step = (gridDim.x + 7 - x) / 8;
  }
};
template <int KIND, int ROWS, int COLS>
__device__ __forceinline__ FfItem ff_item(uint32_t id) {
  constexpr uint32_t kBand = 8;
  const FfArguments a = ff_arguments();
  const uint32_t tiles_m = a->tiles_m, tiles_n = a->tiles_n, splits = a->splits, per_split = a->per_split;
  const uint32_t tiles = tiles_m * tiles_n, part = id / tiles, t = id - part * tiles;
  const uint32_t z = KIND == FF_DW ? part / splits : 0;
  const uint32_t band = t / (kBand * tiles_n), first = band * kBand;
  const uint32_t height = tiles_m - first < kBand ? tiles_m - first : kBand;
  const uint32_t in = t - first * tiles_n, n = in / height;
  const uint32_t k = (part - z * splits) * per_split, ktiles = a->ktiles;
  return FfItem{(uint64_t)(first + in - n * height) * ROWS, (uint64_t)n * COLS, z, part, k,
                k + per_split < ktiles ? k + per_split : ktiles};
}

// A wavefront's place in LDS for the order of its outputs: 16 rows of 128 bytes.
constexpr uint32_t kScratch = 16 * 128;

// Tiles of TP columns (forward: half of them gate's, half up's) by TQ rows on
// WP x WQ wavefronts.
template <int TP_, int TQ_, int WP_, int WQ_>
struct FfShape {
  static constexpr int TP = TP_, TQ = TQ_, WP = WP_, WQ = WQ_;
  static constexpr int threads = WP * WQ * 64;
  static constexpr uint32_t stages = 2 * (TP + TQ) * kRow;
  static constexpr uint32_t lds = stages + WP * WQ * kScratch;
};

// Stores 16 rows of NB blocks of 32 columns, rounded to OT, through the
// wavefront's place in LDS: a lane's 8 columns would be 16 bytes here and there
// of 16 rows, so it takes 16-byte chunks of whole rows of 64 or 128 bytes
// instead.  value(b, e): element e of the lane's 8 of block b, consecutive
// columns (PERM) or twice four.  rows, cols: what exists from the first row and
// column on.  adds: (in binary32) what the output, of type DT, holds is added.
template <int DT, int OT, int NB, bool PERM, class V>
__device__ __forceinline__ void ff_store_rows(lds_char* scratch, char* out, uint64_t stride, int64_t rows, int64_t cols,
                                              V value, bool adds) {
  constexpr int ES = DtypeSize<OT>::value, E = 16 / ES, CPR = NB * 32 / E, W = CPR * 16;  // W: bytes of a row
  static_assert(W == 64 || W == 128, "whole rows in the wavefront's place");
  auto place = [](uint32_t row, uint32_t chunk) {
    return row * W + (chunk ^ (W == 128 ? row >> 1 & 7 : row >> 2 & 3)) * 16;
  };
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t r = lane & 15, g = lane >> 4;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    if constexpr (PERM) {
#pragma unroll
      for (int c = 0; c < 8 / E; ++c) {
        VecF<E> f;
#pragma unroll
        for (int e = 0; e < E; ++e) f.v[e] = value(b, c * E + e);
        *(__attribute__((address_space(3))) u32x4*)(scratch + place(r, b * (32 / E) + g * (8 / E) + c)) =
            pack_vec<OT, E>(f);
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // four columns from 16 h + 4 g on
        VecF<4> f;
#pragma unroll
        for (int e = 0; e < 4; ++e) f.v[e] = value(b, h * 4 + e);
        const uint32_t c = b * 32 + h * 16 + g * 4;
        lds_char* to = scratch + place(r, c / E) + c % E * ES;
        if constexpr (ES == 4) *(__attribute__((address_space(3))) u32x4*)to = pack_vec<OT, 4>(f);
        else *(__attribute__((address_space(3))) u32x2*)to = pack_vec_half<OT>(f);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < 16 * CPR / 64; ++t) {
    const uint32_t row = t * (64 / CPR) + lane / CPR, chunk = lane % CPR;
    const u32x4 x = *(__attribute__((address_space(3))) u32x4*)(scratch + place(row, chunk));
    const int64_t left = cols - (int64_t)(chunk * E);
    if ((int64_t)row >= rows || left <= 0) continue;
    if (OT == DT_F32 && adds) {  // uniform
      char* p = out + row * stride;
      VecF<E> f;
#pragma unroll
      for (int e = 0; e < E; ++e) f.v[e] = __uint_as_float(x[e]);
      const int n = left < E ? (int)left : E;
      const VecF<E> o = load_vec_upto<DT, E>(p, chunk * E, n);
#pragma unroll
      for (int e = 0; e < E; ++e) f.v[e] += o.v[e];
      store_vec_upto<DT, E>(p, chunk * E, n, f);
      continue;
    }
    char* p = out + row * stride + chunk * 16;
    if (left >= E) {
      *(u32x4_any*)p = x;
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (e < left) {
          if constexpr (ES == 4) ((uint32_t*)p)[e] = x[e];
          else ((uint16_t*)p)[e] = (uint16_t)(x[e / 2] >> (16 * (e & 1)));
        }
    }
  }
}

// Stores N such blocks of type DT, by as many at once as make a line.
template <int DT, int N, bool PERM, class V>
__device__ __forceinline__ void ff_store_blocks(lds_char* scratch, char* out, uint64_t stride, int64_t rows,
                                                int64_t cols, V value) {
  constexpr int NB = N % 2 == 0 && DT != DT_F32 ? 2 : 1;
#pragma unroll
  for (int b = 0; b < N; b += NB)
    ff_store_rows<DT, DT, NB, PERM>(scratch, out + b * 32 * DtypeSize<DT>::value, stride, rows, cols - b * 32,
                              [&](int i, int e) { return value(b + i, e); }, false);
}

// The outputs of an item from its sums.
template <int DT, int KIND, class SH, int NP, int NQ>
__device__ __forceinline__ void ff_finish(const FfItem& it, uint32_t wp, uint32_t wq, lds_char* scratch,
                                          f32x4 (&acc)[NP][NQ]) {
  constexpr int ES = DtypeSize<DT>::value;
  const uint32_t lane = threadIdx.x & 63, g = lane >> 4;
#pragma unroll
  for (int j = 0; j < NQ; ++j) {  // 16 rows
    const FfArguments args = ff_arguments();
    const uint64_t r0 = it.m0 + wq * (SH::TQ / SH::WQ) + j * 16;
    const uint64_t c0 = it.n0 + wp * (KIND == FF_FORWARD ? SH::TP / SH::WP / 2 : SH::TP / SH::WP);
    const int64_t rows = (int64_t)(args->m - r0), cols = (int64_t)(args->n - c0);
    if (rows <= 0 || cols <= 0) continue;  // uniform
    // the lane's 8 of the wavefront's b-th 32 columns
    auto at = [&](int b, int e) -> float { return acc[2 * b + e / 4][j][e % 4]; };
    if constexpr (KIND == FF_FORWARD) {
      const int act = args->act, saved = args->saved;
      // blocks 2 b and 2 b + 1 are columns 32 b ... 32 b + 31 of gate and up
      if (saved == 2) {
        const uint64_t nb = args->cgate.nb;
#pragma unroll
        for (int b = 0; b < NP / 2; ++b) {
          const int64_t left = cols - b / 2 * 32;
          VecF<8> v;
#pragma unroll
          for (int e = 0; e < 8; ++e) v.v[e] = at(b, e);
          // columns past the last were made of other rows: the block must not
          // see them
          if (left < 32) {
            const int n = (int)left - (int)g * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) v.v[e] = e < n ? v.v[e] : 0.0f;
          }
          uint32_t m = vec_absmax(v);
          m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
          m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
          if ((int64_t)(lane & 15) < rows && left > 0) {
            const uint64_t r = r0 + (lane & 15), c = c0 + b / 2 * 32;
            const CkptScale sc = ckpt_scale(m);
            *(u32x2*)((b & 1 ? args->cup.codes : args->cgate.codes) + r * nb * kCkptBlock + c + g * 8) =
                (u32x2){ckpt_encode4(v.v, sc), ckpt_encode4(v.v + 4, sc)};
            if (g == 0) (b & 1 ? args->cup.exps : args->cgate.exps)[r * nb + c / kCkptBlock] = (uint8_t)(m >> 23);
          }
        }
      } else if (saved == 1) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint64_t stride = (i ? args->up.stride : args->gate.stride) * ES;
          ff_store_blocks<DT, NP / 4, true>(scratch, (i ? args->up.p : args->gate.p) + r0 * stride + c0 * ES, stride, rows,
                                      cols, [&](int b, int e) { return at(2 * b + i, e); });
        }
      }
      const uint64_t stride = args->out_stride[0];
      ff_store_blocks<DT, NP / 4, true>(
          scratch, args->out[0] + r0 * stride + c0 * ES, stride, rows, cols,
          [&](int b, int e) { return ff_act<DT, false>(at(2 * b, e), act, nullptr) * at(2 * b + 1, e); });
    } else {
      const bool second = KIND == FF_DW && it.z;
      const uint64_t stride = second ? args->out_stride[1] : args->out_stride[0];
      char* out = (second ? args->out[1] : args->out[0]) + r0 * stride;
      const int out_dt = args->out_dt;
      if (args->splits > 1 || (DT != DT_F32 && out_dt == DT_F32) || (KIND == FF_DW && args->accumulate)) {
        const bool split = args->splits > 1, adds = KIND == FF_DW && args->accumulate && !split;
        float* part = args->partials + ((uint64_t)it.part * args->m + r0) * args->pitch;
        const uint64_t step = split ? args->pitch * 4 : stride;
        const int oes = split || out_dt == DT_F32 ? 4 : ES;
#pragma unroll
        for (int i = 0; i < NP / 2; ++i) {
          char* to = (split ? (char*)part : out) + (c0 + i * 32) * oes;
          auto value = [&](int, int e) { return at(i, e); };
          // (the type is the one that is added to: rounded sums are stored by it)
          if (DT != DT_F32 && adds && out_dt != DT_F32)
            ff_store_rows<DT, DT_F32, 1, false>(scratch, to, step, rows, cols - i * 32, value, true);
          else if (DT == DT_F32 || split || out_dt == DT_F32)
            ff_store_rows<DT_F32, DT_F32, 1, false>(scratch, to, step, rows, cols - i * 32, value, adds);
        }
      } else {
        ff_store_blocks<DT, NP / 2, false>(scratch, out + c0 * ES, stride, rows, cols, at);
      }
    }
  }
}

// A workgroup goes through its items as one stream of stages: the stages of
// the next item are asked for while the last ones of this item are
// multiplied and its outputs are stored.
template <int DT, int KIND, class SH, bool DIRECT>
__global__ __launch_bounds__(SH::threads) void ff_product_kernel(FfProduct a) {
  constexpr int TP = SH::TP, TQ = SH::TQ, WP = SH::WP, WQ = SH::WQ;
  constexpr int NTHR = SH::threads, ES = DtypeSize<DT>::value, BK = kRow / ES;
  constexpr int NP = TP / WP / 16, NQ = TQ / WQ / 16;  // 16 x 16 blocks of a wavefront
  // A stage is 2 steps of k, each of GROUPS groups of QN of Q's blocks.
  constexpr int QN = NQ < 2 ? NQ : 2, GROUPS = NQ / QN, STEPS = 2 * GROUPS;
  constexpr bool FWD = KIND == FF_FORWARD;
  static_assert(NP % 2 == 0 && (!FWD || NP % 4 == 0), "of each 64 columns 32 are gate's and 32 up's");
  using LP = FfLoader<DT, FWD, TP, NTHR, DIRECT, FWD, FWD>;
  using LQ = FfLoader<DT, KIND != FF_DW, TQ, NTHR, DIRECT, false, false>;
  constexpr uint32_t kStageP = TP * kRow, kStage = (TP + TQ) * kRow;
  constexpr int kLoads = LP::NI + LQ::NI;
  constexpr int kCols = FWD ? TP / 2 : TP;  // output columns of a tile
  extern __shared__ char smem[];
  lds_char* lds = (lds_char*)smem;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wp = wave % WP, wq = wave / WP;

  // ---- what is asked for next
  const uint32_t items = a.tiles_m * a.tiles_n * a.splits * (KIND == FF_DW ? 2 : 1);
  FfOrder ask(items);
  FfItem want;
  LP lp;
  LQ lq;
  bool going = false;  // there was a stage to ask for last
  uint32_t left = 0;   // terms of it
  uint32_t want_kt = 0, ahead = 0;  // stages of `want` asked for; asked for and not yet read, in all
  uint32_t slot_in = 0, slot = 0;   // where the next goes, where the one being read is
  const char *pcur, *pcur1 = nullptr, *qcur;
  uint64_t done;  // terms of the segment before the next stage
  uint32_t seg;
  const uint32_t seg_tiles = KIND == FF_DX ? a.ktiles / 2 : a.ktiles;
  uint64_t pstep = FWD ? kRow : (uint64_t)BK * a.pstride[0];  // dx: of the segment
  const uint64_t qstep = KIND == FF_DW ? (uint64_t)BK * a.qstride : kRow;
  // the operands of the item's stage kt (dx: gate's terms, then up's)
  auto aim = [&](uint32_t kt) __attribute__((always_inline)) {
    const FfArguments args = ff_arguments();
    seg = KIND == FF_DX && kt >= seg_tiles;
    const uint32_t k = kt - (seg ? seg_tiles : 0);
    done = (uint64_t)k * BK;
    if constexpr (KIND == FF_DX) {
      // the weights' rows may lie differently far apart
      const uint32_t stride = seg ? args->pstride[1] : args->pstride[0];
      pstep = (uint64_t)BK * stride;
      lp.init(args->n - want.n0, stride, stride);
    }
    const uint64_t prow = FWD ? want.n0 * args->pstride[0] : want.n0 * ES;
    pcur = (seg ? args->p[1] : args->p[0]) + prow + k * pstep;
    if (FWD) pcur1 = args->p[1] + want.n0 * args->pstride[1] + k * pstep;
    qcur = (seg || (KIND == FF_DW && want.z) ? args->q[1] : args->q[0]) +
           (KIND == FF_DW ? want.m0 * ES : want.m0 * args->qstride) + k * qstep;
  };
  auto begin = [&]() __attribute__((always_inline)) {
    want = ff_item<KIND, TQ, kCols>(ask.next);
    const FfArguments args = ff_arguments();
    if constexpr (KIND != FF_DX) lp.init(args->n - want.n0, args->pstride[0], args->pstride[1]);
    lq.init(args->m - want.m0, args->qstride, args->qstride);
    want_kt = want.k_begin;
    aim(want_kt);
  };
  // On to the stage after the one that was asked for last (here, and not when
  // that is done, since the products leave no registers for it).
  auto advance = [&]() __attribute__((always_inline)) {
    if (!going) return;
    done += BK;
    pcur += pstep;
    if (FWD) pcur1 += pstep;
    qcur += qstep;
    if (++want_kt == want.k_end) {
      ask.next += ask.step;
      if (ask.next < ask.end) begin();
    } else if (KIND == FF_DX && want_kt == seg_tiles) {
      aim(want_kt);
    }
  };
  // Asks for a part of the next stage, if there is one.  A wavefront's loads
  // queue up behind one another and hold back what it issues after them, so
  // they are spread over PARTS steps of products (all at once, the matrix units
  // idle for about 1000 of 3100 cycles a stage).
  constexpr int PARTS = !DIRECT ? 1 : STEPS < 4 ? STEPS : 4;
  auto fetch_part = [&](auto part) __attribute__((always_inline)) {
    constexpr int kPart = decltype(part)::value, kFirst = kPart * kLoads / PARTS;
    if (kPart == 0) {
      advance();
      going = ask.next < ask.end;
      left = !going ? 0 : a.k - done < BK ? (uint32_t)(a.k - done) : BK;
    }
    if (!DIRECT && !going) return;
    const uint32_t stage = (uint32_t)(uintptr_t)lds + slot_in * kStage;
    ff_each<(kPart + 1) * kLoads / PARTS - kFirst>([&](auto n) __attribute__((always_inline)) {
      constexpr int I = kFirst + decltype(n)::value;
      const uint32_t nlimit = (uint32_t)(a.n - want.n0), mlimit = (uint32_t)(a.m - want.m0);
      if constexpr (I < LP::NI)
        lp.template load<I>(pcur, pcur1, left, stage, !FWD && nlimit < TP, nlimit, (uint32_t)(FWD ? done : want.n0));
      else
        lq.template load<I - LP::NI>(qcur, qcur, left, stage + kStageP, KIND == FF_DW && mlimit < TQ, mlimit,
                                     (uint32_t)(KIND == FF_DW ? want.m0 : done));
    });
    if (kPart + 1 < PARTS || !going) return;
    ++ahead;
    slot_in ^= 1;
  };
  auto fetch = [&]() __attribute__((always_inline)) { ff_each<PARTS>(fetch_part); };
  auto put = [&](uint32_t to) __attribute__((always_inline)) {
    lp.put(lds + to * kStage);
    lq.put(lds + to * kStage + kStageP);
  };

  // ---- what is multiplied
  FfOrder mine(items);
  f32x4 acc[NP][NQ];
  const uint32_t pat = LP::fragment_at(wp * (TP / WP)), qat = LQ::fragment_at(wq * (TQ / WQ));
  u32x4 fp[2][NP], fq[2][QN];
  auto read = [&](auto step) __attribute__((always_inline)) {
    constexpr int ks = decltype(step)::value / GROUPS, group = decltype(step)::value % GROUPS;
    const lds_char *sp = lds + slot * kStage, *sq = sp + kStageP;
    if constexpr (group == 0)
#pragma unroll
      for (int i = 0; i < NP; ++i) fp[ks][i] = LP::fragment(sp, pat, i, ks);
#pragma unroll
    for (int j = 0; j < QN; ++j) fq[decltype(step)::value & 1][j] = LQ::fragment(sq, qat, group * QN + j, ks);
  };
  auto multiply = [&](auto step) __attribute__((always_inline)) {
    constexpr int ks = decltype(step)::value / GROUPS, group = decltype(step)::value % GROUPS;
#pragma unroll
    for (int t = 0; t < ff_turns<DT>(); ++t)
#pragma unroll
      for (int j = 0; j < QN; ++j)
#pragma unroll
        for (int i = 0; i < NP; ++i)
          acc[i][group * QN + j] = ff_mfma<DT>(fp[ks][i], fq[decltype(step)::value & 1][j], acc[i][group * QN + j], t);
  };
  constexpr std::integral_constant<int, 0> kFirstStep;
  constexpr std::integral_constant<int, STEPS - 1> kLastStep;
  auto most_of_a_stage = [&]() __attribute__((always_inline)) {
    ff_each<STEPS - 1>([&](auto step) __attribute__((always_inline)) {
      constexpr std::integral_constant<int, decltype(step)::value + 1> next;
      read(next);
      // the rest of the stage that was begun when this one's slot got free
      if constexpr (next < PARTS) fetch_part(next);
      multiply(step);
      // reads of further steps would take more registers than there are
      __builtin_amdgcn_sched_barrier(0);
    });
    --ahead;
  };
  auto next_stage = [&]() __attribute__((always_inline)) {
    slot ^= 1;
    put(slot);
    ff_meet();
  };

  if (mine.next >= mine.end) return;  // the whole workgroup
  begin();
  fetch();
  put(0);
  ff_meet();
  fetch_part(kFirstStep);  // as after every stage; the rest comes with the products
  // Each step's fragments are read while the step before multiplies, across
  // stages too: the wavefronts meet when the last step's fragments are in
  // registers, so that its products run while the next stage's first
  // fragments come and a further stage is asked for.
  for (; mine.next < mine.end; mine.next += mine.step) {
    const FfItem it = ff_item<KIND, TQ, kCols>(mine.next);
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
      for (int j = 0; j < NQ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.0f;
    f32x4 total[DT == DT_F32 ? NP : 1][DT == DT_F32 ? NQ : 1] = {};  // of the stages before acc's
    read(kFirstStep);
    for (uint32_t kt = it.k_begin + 1;;) {
      const uint32_t stop = DT == DT_F32 && kt + kFoldStages < it.k_end ? kt + kFoldStages : it.k_end;
      for (; kt < stop; ++kt) {
        most_of_a_stage();
        next_stage();
        fetch_part(kFirstStep);
        read(kFirstStep);
        multiply(kLastStep);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (kt >= it.k_end) break;
      if constexpr (DT == DT_F32) {
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
          for (int j = 0; j < NQ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              total[i][j][e] += acc[i][j][e];
              acc[i][j][e] = 0.0f;
            }
      }
    }
    // the last stage; the next item's first fragments come after this one's
    // outputs, which need the registers
    most_of_a_stage();
    if (ahead) {
      next_stage();
      fetch_part(kFirstStep);
    }
    multiply(kLastStep);
    if constexpr (DT == DT_F32) {
#pragma unroll
      for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int j = 0; j < NQ; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] += total[i][j][e];
    }
    ff_finish<DT, KIND, SH, NP, NQ>(it, wp, wq, lds + SH::stages + wave * kScratch, acc);
  }
  // the parts of a stage that was not there are loads too: none may be on its
  // way when this workgroup's LDS becomes another's
  asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
}

template <int DT, int KIND, class SH, bool DIRECT>
hipError_t ff_launch(FfProduct& a, hipStream_t stream) {
  constexpr uint64_t kCols = KIND == FF_FORWARD ? SH::TP / 2 : SH::TP;
  a.tiles_m = (uint32_t)((a.m + SH::TQ - 1) / SH::TQ);
  a.tiles_n = (uint32_t)((a.n + kCols - 1) / kCols);
  constexpr uint64_t kTerms = kRow / DtypeSize<DT>::value;
  a.ktiles = (uint32_t)((a.k + kTerms - 1) / kTerms) * (KIND == FF_DX ? 2 : 1);
  a.per_split = (a.ktiles + a.splits - 1) / a.splits;
  // a split without work would leave its partial sums unwritten
  a.splits = (a.ktiles + a.per_split - 1) / a.per_split;
  const uint64_t items = (uint64_t)a.tiles_m * a.tiles_n * a.splits * (KIND == FF_DW ? 2 : 1);
  const uint64_t resident = 256 * std::max<uint64_t>(1, std::min<uint64_t>(163840 / SH::lds, 1024 / SH::threads));
  hipLaunchKernelGGL((ff_product_kernel<DT, KIND, SH, DIRECT>), dim3((unsigned)std::min(items, resident)),
                     dim3(SH::threads), SH::lds, stream, a);
  return launch_status(stream);
}

// Tiles of 256 x 256 for many outputs (of direct loads in 16 bits), or smaller
// ones.
template <int DT, int KIND>
hipError_t ff_launch_dt(FfProduct& a, bool wide, bool direct, hipStream_t stream) {
  if constexpr (DT == DT_F32) {
    // In binary32 the matrix instructions take sixteen times as long for a
    // stage, so that small tiles cost little and fill the CUs evenly: forward of
    // 65 x 1024 x 2816 33 us (43 by 64 rows), 513 x 1024 x 2816 66 (75).  Many
    // tokens would take the larger ones: 2048 x 2048 x 5632 795 (729).  The
    // backward products are split, which fills the CUs for tiles of 64 rows.
    constexpr int TP = KIND == FF_FORWARD ? 128 : 64, TQ = KIND == FF_FORWARD ? 32 : 64;
    return direct ? ff_launch<DT, KIND, FfShape<TP, TQ, 2, 2>, true>(a, stream)
                  : ff_launch<DT, KIND, FfShape<TP, TQ, 2, 2>, false>(a, stream);
  } else {
    if (wide) return ff_launch<DT, KIND, FfShape<256, 256, 4, 2>, true>(a, stream);
    return direct ? ff_launch<DT, KIND, FfShape<128, 128, 2, 4>, true>(a, stream)
                  : ff_launch<DT, KIND, FfShape<128, 128, 2, 4>, false>(a, stream);
  }
}

template <int KIND>
hipError_t ff_launch_kind(int dt, FfProduct& a, bool wide, bool direct, hipStream_t stream) {
  switch (dt) {
    case DT_F32: return ff_launch_dt<DT_F32, KIND>(a, wide, direct, stream);
    case DT_F16: return ff_launch_dt<DT_F16, KIND>(a, wide, direct, stream);
    default: return ff_launch_dt<DT_BF16, KIND>(a, wide, direct, stream);
  }
}

}  // namespace
}  // namespace rar
