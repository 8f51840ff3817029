// The matrix products of the gated feed-forward block on gfx950's matrix
// instructions: C[q][p] = sum over k of Q(q, k) P(p, k), where each operand
// lies in memory either by rows of k (KC) or by rows of its own index (the
// weights in dx, x and dg in dW).
//
// A workgroup computes TP columns by TQ rows; a stage of both operands is 128
// bytes of k a row (64 16-bit terms, 32 in binary32), so every type has the
// same layout in LDS.  Two stages alternate: while the wavefronts multiply
// one, the next is on its way.  A wavefront holds 64 columns by TQ / WQ rows
// in 32 x 32 blocks.
//
// P is the matrix instruction's first operand, whose index runs over a lane's
// accumulators: p = 8 (i / 4) + 4 (lane / 32) + i % 4 for accumulator i.  Its
// rows are read in the order that makes this a lane's 16 consecutive columns
// (half = lane / 32: columns 16 half ... 16 half + 15), so an epilogue stores
// whole vectors and finds a checkpoint's block of 32 in two lanes.
//
// LDS positions are 16-byte chunks.  The chunks of a row are stored under an
// XOR of the row's low bits, so that the lanes of one read hit different
// banks; the loads apply it to their source, since direct loads write LDS in
// lane order.  Rows of the operand's own index are read by the transposing
// LDS load (16 bits), which hands lane i of 16 the i-th of 16 columns and
// four consecutive k.
#pragma once

#include <type_traits>

#include "gated_ff.hpp"

namespace rar {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef _Float16 h16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 b16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_char;

constexpr uint32_t kStageRow = 128;  // bytes of k a row of a stage

template <int DT>
__device__ __forceinline__ f32x16 ff_mfma(u32x4 p, u32x4 q, f32x16 c) {
  if constexpr (DT == DT_BF16) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b16x8, p), __builtin_bit_cast(b16x8, q), c, 0, 0,
                                                   0);
  } else if constexpr (DT == DT_F16) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h16x8, p), __builtin_bit_cast(h16x8, q), c, 0, 0,
                                                  0);
  } else {
    // four terms a lane: the i-th of each chunk pair make one instruction's two
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(p[i]), __uint_as_float(q[i]), c, 0, 0, 0);
    return c;
  }
}

// One operand's share of a stage.  T: rows (KC) or columns of the operand's
// index in the tile.  PAIR: the 32-row halves of each 64 rows belong to two
// matrices (gate and up).  PERM: read in P's order.
template <int DT, bool KC, int T, int NTHR, bool DIRECT, bool PAIR, bool PERM>
struct FfLoader {
  static constexpr int ES = DtypeSize<DT>::value, EC = 16 / ES;  // elements of a chunk
  static constexpr int BK = kStageRow / ES;
  static constexpr int NI = T * 8 / NTHR;          // chunks a thread
  static constexpr int CPR = KC ? 8 : T * ES / 16;  // chunks a row of the stage
  static constexpr int RPI = NTHR / CPR;           // rows between a thread's chunks
  static constexpr uint32_t kOut = 0x80000000u;    // past every buffer range: reads as zeros
  static_assert(!PAIR || (KC && (RPI == 32 || (RPI == 64 && DIRECT))), "which matrix a chunk belongs to");

  // XOR of the chunks of a stage row.  KC: the rows that neighbouring lanes
  // read (r ... r + 7, or in P's order r ... r + 3 and r + 16 ... r + 19) take
  // eight different values.  Otherwise the four k of a transposing read, or
  // in binary32 the two of the lane halves.
  static __device__ __forceinline__ uint32_t swizzle(uint32_t row) {
    if constexpr (KC) return PERM ? (row & 3) | (row >> 2 & 4) : row & 7;
    else return ES == 2 ? (row & 3) << 2 : (row >> 2 & 1) << 3;
  }

  uint32_t row, chunk;          // of the thread's first chunk; chunk after the XOR
  uint32_t off[DIRECT ? NI : 1];
  u32x4 hold[DIRECT ? 1 : NI];
  uint32_t limit;               // rows (KC) or columns of the tile that exist

  // Which matrix the thread's i-th chunk belongs to (the same for the whole
  // wavefront), and its row there.
  static __device__ __forceinline__ uint32_t matrix_of(int i) {
    if constexpr (!PAIR) return 0;
    return RPI == 32 ? i & 1 : (uint32_t)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6) / 4 & 1;
  }
  static __device__ __forceinline__ uint32_t local(uint32_t r) { return PAIR ? (r >> 6) * 32 + (r & 31) : r; }
  static __device__ __forceinline__ uint32_t chunk_of(uint32_t pos, uint32_t r) { return pos ^ swizzle(r); }

  __device__ __forceinline__ void init(uint32_t lim, uint64_t stride0, uint64_t stride1) {
    limit = lim;
    row = threadIdx.x / CPR;
    chunk = chunk_of(threadIdx.x % CPR, row);
    if constexpr (DIRECT) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const uint32_t r = row + i * RPI, stride = (uint32_t)(matrix_of(i) ? stride1 : stride0);
        if constexpr (KC) off[i] = local(r) < lim ? local(r) * stride + chunk * 16 : kOut;
        else off[i] = r * stride + chunk_of(threadIdx.x % CPR, r) * 16;
      }
    }
  }

  // Asks for the stage that begins at term k0 of `terms`.  base: the tile's
  // first row (KC) or column at term 0 of either matrix, end: past the last
  // byte of each.
  __device__ __forceinline__ void load(const char* const* base, const char* const* end, const uint64_t* stride,
                                       uint64_t k0, uint64_t terms, lds_char* stage) {
    const uint64_t left = terms - k0;
    if constexpr (DIRECT) {
      const bool last = left < BK;
      const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
      __amdgpu_buffer_rsrc_t range[PAIR ? 2 : 1];
#pragma unroll
      for (int m = 0; m < (PAIR ? 2 : 1); ++m) {
        const char* b = base[m] + (KC ? k0 * ES : k0 * stride[m]);
        const uint64_t bytes = (uint64_t)(end[m] - b);
        range[m] = wt_range(b, bytes < 0x7fffffffu ? (uint32_t)bytes : 0x7fffffffu);
      }
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        uint32_t o = off[i];
        if (last) {  // uniform
          if constexpr (KC) o = chunk * EC < left ? o : kOut;
          else o = row + i * RPI < left ? o : kOut;
        }
        lds_char* to = stage + (i * NTHR + wave * 64) * 16;
        if constexpr (PAIR) {
          if (matrix_of(i)) __builtin_amdgcn_raw_ptr_buffer_load_lds(range[PAIR], to, 16, (int)o, 0, 0, 0);
          else __builtin_amdgcn_raw_ptr_buffer_load_lds(range[0], to, 16, (int)o, 0, 0, 0);
        } else {
          __builtin_amdgcn_raw_ptr_buffer_load_lds(range[0], to, 16, (int)o, 0, 0, 0);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const uint32_t r = row + i * RPI;
        const uint32_t m = matrix_of(i);  // a constant here
        const char* b = m ? base[PAIR] : base[0];
        const uint64_t st = m ? stride[PAIR] : stride[0];
        const char* at;
        uint32_t have;  // elements of the chunk that exist
        if constexpr (KC) {
          const uint32_t e = chunk * EC;
          at = b + local(r) * st + (k0 + e) * ES;
          have = local(r) < limit && e < left ? (left - e < EC ? (uint32_t)(left - e) : EC) : 0;
        } else {
          const uint32_t e = chunk_of(threadIdx.x % CPR, r) * EC;
          at = b + (k0 + r) * st + (uint64_t)e * ES;
          have = r < left && e < limit ? (limit - e < EC ? limit - e : EC) : 0;
        }
        u32x4 x = {0, 0, 0, 0};
        if (have == EC) {
          x = *(const u32x4_any*)at;
        } else if (have) {
#pragma unroll
          for (int j = 0; j < EC; ++j)
            if ((uint32_t)j < have) {
              if constexpr (ES == 4) x[j] = ((const uint32_t*)at)[j];
              else x[j / 2] |= (uint32_t)((const uint16_t*)at)[j] << (16 * (j & 1));
            }
        }
        hold[i] = x;
      }
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

  // Where this lane's fragments begin in a stage.
  static __device__ __forceinline__ uint32_t fragment_at(uint32_t first) {
    const uint32_t lane = threadIdx.x & 63, half = lane >> 5;
    if constexpr (KC) {
      const uint32_t p = lane & 31;
      const uint32_t r = PERM ? (p >> 2 & 1) * 16 + (p >> 3) * 4 + (p & 3) : p;
      return (first + r) * kStageRow + (half ^ swizzle(r)) * 16;
    } else if constexpr (ES == 2) {
      const uint32_t l = lane & 3, g = lane >> 4 & 1, k = half * 8 + (lane >> 2 & 3);
      const uint32_t c = first / 8 + (PERM ? (l & 1) * 2 + g : g * 2 + (l >> 1)), h = PERM ? l >> 1 : l & 1;
      return k * (T * 2) + (c ^ swizzle(k)) * 16 + h * 8;
    } else {
      const uint32_t p = lane & 31;
      const uint32_t n = first + (PERM ? (p >> 2 & 1) * 16 + (p >> 3) * 4 + (p & 3) : p);
      // the swizzle is that of k = 4 half + 8 ks, the same for every ks
      return half * 4 * (T * 4) + (n / 4 ^ swizzle(half * 4)) * 16 + (n & 3) * 4;
    }
  }
  // The fragment of 32 rows or columns `tile` of the wavefront's, terms step
  // ks (two chunks of k).
  static __device__ __forceinline__ u32x4 fragment(const lds_char* stage, uint32_t at, int tile, int ks) {
    if constexpr (KC) {
      return *(const __attribute__((address_space(3))) u32x4*)(stage + ((at ^ (ks * 32)) + tile * 32 * kStageRow));
    } else if constexpr (ES == 2) {
      // k advances by 16: the XOR stays, and 32 columns are four chunks, above
      // whose bits it acts too
      typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
      lds_char* p = (lds_char*)stage + ((at ^ tile * 64) + ks * 16 * (T * 2));
      const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p));
      const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * (T * 2))));
      return (u32x4){a[0], a[1], b[0], b[1]};
    } else {
      const lds_char* p = stage + ((at ^ tile * 128) + ks * 8 * (T * 4));
      u32x4 x;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = *(const __attribute__((address_space(3))) uint32_t*)(p + i * (T * 4));
      return x;
    }
  }
};

// Order of the tiles: consecutive workgroups go to the 8 XCDs in turn, so
// each XCD gets a contiguous range of the order; in it, tiles come in bands
// of 8 tiles of rows, columns slowest, so that the 32 tiles an XCD works on
// at once share their operands through its L2.
struct FfTile {
  uint32_t m, n;
};
__device__ __forceinline__ uint32_t ff_order(uint32_t id, uint32_t count) {
  const uint32_t x = id % 8, base = count / 8, extra = count % 8;
  return x * base + (x < extra ? x : extra) + id / 8;
}
__device__ __forceinline__ FfTile ff_tile(uint32_t t, uint32_t tiles_m, uint32_t tiles_n) {
  constexpr uint32_t kBand = 8;
  const uint32_t band = t / (kBand * tiles_n), first = band * kBand;
  const uint32_t height = tiles_m - first < kBand ? tiles_m - first : kBand;
  const uint32_t in = t - band * kBand * tiles_n;
  return FfTile{first + in % height, in / height};
}

template <int DT, int KIND, int TP, int TQ, int WP, int WQ, bool DIRECT>
__global__ __launch_bounds__(WP* WQ * 64) void ff_product_kernel(FfProduct a) {
  constexpr int NTHR = WP * WQ * 64, ES = DtypeSize<DT>::value, BK = kStageRow / ES;
  constexpr int NP = TP / WP / 32, NQ = TQ / WQ / 32;  // 32 x 32 blocks of a wavefront
  constexpr bool FWD = KIND == FF_FORWARD;
  static_assert(NP == 2, "a wavefront's 64 columns: 32 of gate and 32 of up forward");
  using LP = FfLoader<DT, FWD, TP, NTHR, DIRECT, FWD, true>;
  using LQ = FfLoader<DT, KIND != FF_DW, TQ, NTHR, DIRECT, false, false>;
  constexpr uint32_t kStageP = TP * kStageRow, kStage = (TP + TQ) * kStageRow;
  extern __shared__ char smem[];
  lds_char* lds = (lds_char*)smem;

  const uint32_t tiles = a.tiles_m * a.tiles_n;
  uint32_t id = ff_order(blockIdx.x, gridDim.x);
  const uint32_t part = id / tiles;  // output (dW) and split
  id -= part * tiles;
  const uint32_t z = KIND == FF_DW ? part / a.splits : 0, split = KIND == FF_DW ? part - z * a.splits : part;
  const FfTile t = ff_tile(id, a.tiles_m, a.tiles_n);
  constexpr uint32_t kCols = FWD ? TP / 2 : TP;  // output columns of the tile
  const uint64_t n0 = (uint64_t)t.n * kCols, m0 = (uint64_t)t.m * TQ;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wp = wave % WP, wq = wave / WP;

  // a segment's terms: a row's for KC operands, the rows' count otherwise
  auto p_rows = [&]() { return FWD ? a.n : a.k; };
  auto q_rows = [&]() { return KIND == FF_DW ? a.k : a.m; };
  const char *pbase[2], *pend[2], *qbase[2], *qend[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    pbase[s] = a.p[s] + (FWD ? n0 * a.pstride[s] : n0 * ES);
    pend[s] = a.p[s] + (p_rows() - 1) * a.pstride[s] + (FWD ? a.k : a.n) * ES;
    qbase[s] = a.q[s] + (KIND == FF_DW ? m0 * ES : m0 * a.qstride[s]);
    qend[s] = a.q[s] + (q_rows() - 1) * a.qstride[s] + (KIND == FF_DW ? a.m : a.k) * ES;
  }
  LP lp;
  LQ lq;
  lp.init((uint32_t)(a.n - n0 < kCols ? a.n - n0 : kCols), a.pstride[0], a.pstride[1]);
  lq.init((uint32_t)(a.m - m0 < TQ ? a.m - m0 : TQ), a.qstride[0], a.qstride[1]);

  const uint32_t seg_tiles = KIND == FF_DX ? a.ktiles / 2 : a.ktiles;
  auto fetch = [&](uint32_t kt, uint32_t buf) {
    const uint32_t s = KIND == FF_DX ? (kt >= seg_tiles) : z;
    const uint64_t k0 = (uint64_t)(kt - (KIND == FF_DX && s ? seg_tiles : 0)) * BK;
    const char* pb[2] = {FWD ? pbase[0] : pbase[s], pbase[1]};
    const char* pe[2] = {FWD ? pend[0] : pend[s], pend[1]};
    const char* qb[1] = {qbase[s]};
    const char* qe[1] = {qend[s]};
    const uint64_t ps[2] = {FWD ? a.pstride[0] : a.pstride[s], a.pstride[1]};
    const uint64_t qs[1] = {a.qstride[s]};
    lp.load(pb, pe, ps, k0, a.k, lds + buf * kStage);
    lq.load(qb, qe, qs, k0, a.k, lds + buf * kStage + kStageP);
  };
  auto put = [&](uint32_t buf) {
    lp.put(lds + buf * kStage);
    lq.put(lds + buf * kStage + kStageP);
  };

  f32x16 acc[NP][NQ];
#pragma unroll
  for (int i = 0; i < NP; ++i)
#pragma unroll
    for (int j = 0; j < NQ; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
  const uint32_t pat = LP::fragment_at(wp * 64), qat = LQ::fragment_at(wq * (TQ / WQ));

  const uint32_t k_begin = split * a.per_split;
  const uint32_t k_end = k_begin + a.per_split < a.ktiles ? k_begin + a.per_split : a.ktiles;
  if (k_begin < k_end) {
    fetch(k_begin, 0);
    put(0);
  }
  for (uint32_t kt = k_begin; kt < k_end; ++kt) {
    const uint32_t buf = (kt - k_begin) & 1;
    // this stage's loads have landed, and nobody reads the other any more
    if constexpr (DIRECT) __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
    __syncthreads();
    if (kt + 1 < k_end) fetch(kt + 1, buf ^ 1);
    const lds_char *sp = lds + buf * kStage, *sq = sp + kStageP;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      u32x4 fp[NP], fq[NQ];
#pragma unroll
      for (int i = 0; i < NP; ++i) fp[i] = LP::fragment(sp, pat, i, ks);
#pragma unroll
      for (int j = 0; j < NQ; ++j) fq[j] = LQ::fragment(sq, qat, j, ks);
#pragma unroll
      for (int j = 0; j < NQ; ++j)
#pragma unroll
        for (int i = 0; i < NP; ++i) acc[i][j] = ff_mfma<DT>(fp[i], fq[j], acc[i][j]);
    }
    if (kt + 1 < k_end) put(buf ^ 1);
  }

  // epilogue: a lane's 16 columns of each block
  const uint32_t lane = threadIdx.x & 63, half = lane >> 5;
#pragma unroll
  for (int j = 0; j < NQ; ++j) {
    const uint64_t r = m0 + wq * (TQ / WQ) + j * 32 + (lane & 31);
    if constexpr (FWD) {
      const uint64_t c = n0 + wp * 32 + half * 16;
      const int n = c >= a.n ? 0 : (a.n - c < 16 ? (int)(a.n - c) : 16);
      float g[16], u[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        // columns past the last were multiplied with zeros, which an infinite
        // or NaN x makes NaN: a checkpoint's block must not see them
        g[e] = e < n ? acc[0][j][e] : 0.0f;
        u[e] = e < n ? acc[1][j][e] : 0.0f;
      }
      if (a.saved == 2) {
        auto save = [&](const Checkpoint& ck, const float* v) {
          uint32_t m = 0;
#pragma unroll
          for (int e = 0; e < 16; ++e) m = max(m, absbits(v[e]));
          m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
          if (r < a.m && c - half * 16 < a.n) {
            const BfpScale sc = bfp_scale(m, 8);
            u32x4 w;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = ckpt_encode4(v + 4 * i, sc);
            *(u32x4*)(ck.code_row(r) + c) = w;
            if (half == 0) ck.exp_row(r)[c / kCkptBlock] = (uint8_t)(m >> 23);
          }
        };
        save(a.cgate, g);
        save(a.cup, u);
      }
      if (r < a.m && n > 0) {
        if (a.saved == 1) {
          ff_store16<DT>(a.gate.p + r * a.gate.stride * ES, c, n, g);
          ff_store16<DT>(a.up.p + r * a.up.stride * ES, c, n, u);
        }
        float h[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) h[e] = ff_act<false>(g[e], a.act, nullptr) * u[e];
        ff_store16<DT>(a.out[0] + r * a.out_stride[0], c, n, h);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const uint64_t c = n0 + wp * 64 + i * 32 + half * 16;
        const int n = c >= a.n ? 0 : (a.n - c < 16 ? (int)(a.n - c) : 16);
        if (r >= a.m || n == 0) continue;
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = acc[i][j][e];
        if (a.splits > 1) {
          float* row = a.partials + ((uint64_t)part * a.m + r) * a.pitch;
          ff_store16<DT_F32>((char*)row, c, n, v);
          continue;
        }
        char* row = KIND == FF_DW && z ? a.out[1] + r * a.out_stride[1] : a.out[0] + r * a.out_stride[0];
        if (KIND == FF_DW && a.accumulate) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (e < n) v[e] += load_elem_dt(row, c + e, a.out_dt);
        }
        if (DT != DT_F32 && a.out_dt == DT_F32) ff_store16<DT_F32>(row, c, n, v);
        else ff_store16<DT>(row, c, n, v);
      }
    }
  }
}

template <int DT, int KIND, int TP, int TQ, int WP, int WQ, bool DIRECT>
hipError_t ff_launch(const FfProduct& a, hipStream_t stream) {
  constexpr size_t lds = 2 * (TP + TQ) * kStageRow;
  const uint64_t grid = (uint64_t)a.tiles_m * a.tiles_n * a.splits * (KIND == FF_DW ? 2 : 1);
  auto* kernel = &ff_product_kernel<DT, KIND, TP, TQ, WP, WQ, DIRECT>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(WP * WQ * 64), lds, stream, a);
  return launch_status(stream);
}

// wide: tiles of 256 x 256 (only of direct loads in 16 bits), else 128 x 128.
template <int DT, int KIND>
hipError_t ff_launch_dt(const FfProduct& a, bool wide, bool direct, hipStream_t stream) {
  if constexpr (DT != DT_F32)
    if (wide) return ff_launch<DT, KIND, 256, 256, 4, 2, true>(a, stream);
  return direct ? ff_launch<DT, KIND, 128, 128, 2, 2, true>(a, stream)
                : ff_launch<DT, KIND, 128, 128, 2, 2, false>(a, stream);
}

template <int KIND>
hipError_t ff_launch_kind(int dt, const FfProduct& a, bool wide, bool direct, hipStream_t stream) {
  switch (dt) {
    case DT_F32: return ff_launch_dt<DT_F32, KIND>(a, wide, direct, stream);
    case DT_F16: return ff_launch_dt<DT_F16, KIND>(a, wide, direct, stream);
    default: return ff_launch_dt<DT_BF16, KIND>(a, wide, direct, stream);
  }
}

}  // namespace
}  // namespace rar
