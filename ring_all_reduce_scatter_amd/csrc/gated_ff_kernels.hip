// Gated feed-forward block: the kernels around its tiled products
// (gated_ff_tile.hpp), and which of them a call takes.
#include <algorithm>

#include "gated_ff.hpp"

namespace rar {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 h16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 b16x8 __attribute__((ext_vector_type(8)));

uint64_t up_div(uint64_t a, uint64_t b) { return (a + b - 1) / b; }

// ------------------------------------------------------------------ few tokens

// Forward for at most 64 tokens: the weights' bytes are all that counts.

// A 16-byte chunk of a row from element e on; elements past dim are zeros.
template <int DT>
__device__ __forceinline__ u32x4 few_chunk(const char* row, uint64_t e, uint64_t dim) {
  constexpr int ES = DtypeSize<DT>::value, EC = 16 / ES;
  const char* at = row + e * ES;
  if (e + EC <= dim) return *(const u32x4_any*)at;
  u32x4 x = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < EC; ++j)
    if (e + j < dim) {
      if constexpr (ES == 4) x[j] = ((const uint32_t*)at)[j];
      else x[j / 2] |= (uint32_t)((const uint16_t*)at)[j] << (16 * (j & 1));
    }
  return x;
}

// One element of h and, if asked for, of the projections, from its two sums.
template <int DT>
__device__ __forceinline__ void few_store(const FfProduct& a, uint64_t token, uint64_t col, float g, float u) {
  constexpr int ES = DtypeSize<DT>::value;
  if (a.saved == 1) {
    store_elem<DT>(a.gate.p + token * a.gate.stride * ES, col, g);
    store_elem<DT>(a.up.p + token * a.up.stride * ES, col, u);
  }
  store_elem<DT>(a.out[0] + token * a.out_stride[0], col, ff_act<DT, false>(g, a.act, nullptr) * u);
}

template <int DT>
__device__ __forceinline__ f32x4 few_mfma(u32x4 w, u32x4 x, f32x4 c) {
  if constexpr (DT == DT_BF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b16x8, w), __builtin_bit_cast(b16x8, x), c, 0, 0,
                                                   0);
  } else if constexpr (DT == DT_F16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h16x8, w), __builtin_bit_cast(h16x8, x), c, 0, 0,
                                                  0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(w[i]), __uint_as_float(x[i]), c, 0, 0, 0);
    return c;
  }
}

// On the matrix units, straight from memory.  A workgroup has NR blocks of
// 16 hidden columns and NT blocks of 16 tokens, and its W wavefronts share the terms, 128-byte pieces of a row in turn; their sums are added through
// LDS in order.  An instruction's 16 rows take halves of each 128-byte line, the
// next instruction the others, so these loads must not be streaming ones (72 us
// for 64 tokens, 67 with these).
template <int DT, int NT, int NR, int W>
__global__ __launch_bounds__(W * 64) void ff_few_kernel(FfProduct a) {
  constexpr int ES = DtypeSize<DT>::value, EC = 16 / ES;
  extern __shared__ float sums[];  // [wavefront][gate, up][NR][NT][256]
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t r = lane & 15, quad = lane >> 4;
  const uint64_t c0 = (uint64_t)blockIdx.x * (16 * NR);
  // columns and tokens past the last read the last one's row; what comes of
  // them is not stored
  const char *w[2][NR], *x[NT];
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    const uint64_t c = c0 + n * 16 + r < a.n ? c0 + n * 16 + r : a.n - 1;
    w[0][n] = a.p[0] + c * a.pstride[0];
    w[1][n] = a.p[1] + c * a.pstride[1];
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
    x[t] = a.q[0] + (uint64_t)(t * 16 + r < a.m ? t * 16 + r : a.m - 1) * a.qstride;
  f32x4 acc[2][NR][NT];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[h][n][t] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
  // a piece is 128 bytes of a row, two steps of four chunks
  const uint32_t whole = (uint32_t)(a.k / (8 * EC)), pieces = (uint32_t)((a.k + 8 * EC - 1) / (8 * EC));
  uint32_t k = wave;
  for (; k < whole; k += W) {
    u32x4 pw[2][2][NR], px[2][NT];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint32_t at = k * 128 + quad * 32 + s * 16;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int n = 0; n < NR; ++n) pw[s][h][n] = *(const u32x4_any*)(w[h][n] + at);
#pragma unroll
      for (int t = 0; t < NT; ++t) px[s][t] = *(const u32x4_any*)(x[t] + at);
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int t = 0; t < NT; ++t) acc[h][n][t] = few_mfma<DT>(pw[s][h][n], px[s][t], acc[h][n][t]);
  }
  for (; k < pieces; k += W)
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint64_t e = ((uint64_t)k * 8 + quad * 2 + s) * EC;
      u32x4 q[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) q[t] = few_chunk<DT>(x[t], e, a.k);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int n = 0; n < NR; ++n) {
          const u32x4 p = few_chunk<DT>(w[h][n], e, a.k);
#pragma unroll
          for (int t = 0; t < NT; ++t) acc[h][n][t] = few_mfma<DT>(p, q[t], acc[h][n][t]);
        }
    }
  constexpr uint32_t kPlane = NR * NT * 256;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          sums[(wave * 2 + h) * kPlane + (t * 16 + r) * (16 * NR) + n * 16 + quad * 4 + i] = acc[h][n][t][i];
  __syncthreads();
  for (uint32_t o = threadIdx.x; o < kPlane; o += W * 64) {
    float vg = 0.0f, vu = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      vg += sums[i * 2 * kPlane + o];
      vu += sums[(i * 2 + 1) * kPlane + o];
    }
    const uint64_t token = o / (16 * NR), col = c0 + o % (16 * NR);
    if (token >= a.m || col >= a.n) continue;
    few_store<DT>(a, token, col, vg, vu);
  }
}

template <int DT, int NT, int NR, int W>
hipError_t few_launch(const FfProduct& a, hipStream_t stream) {
  hipLaunchKernelGGL((ff_few_kernel<DT, NT, NR, W>), dim3((unsigned)((a.n + 16 * NR - 1) / (16 * NR))),
                     dim3(W * 64), W * 2 * NR * NT * 256 * sizeof(float), stream, a);
  return launch_status(stream);
}

// The same for at most 32 tokens, with whole lines an instruction: its 16 rows
// are two halves of 8 columns, so that 8 lanes have the 128 bytes of a column's
// piece, each lane the chunk 2 quad + half.  A matrix instruction with the even
// chunks of x is then right for the first half's rows, one with the odd chunks
// for the second's, and the others are never stored: twice the products, which
// have time, for streaming loads of whole lines.  16 tokens of 4096 x 11264
// bfloat16 take 37.6 us, 24 44, the kernel above 47 and 53; 64 tokens have no
// registers left for it (86 to 104 us, 67 above).
template <int DT, int NT, int W, int PIECES>
__global__ __launch_bounds__(W * 64) void ff_lines_kernel(FfProduct a) {
  constexpr int ES = DtypeSize<DT>::value, EC = 16 / ES;
  extern __shared__ float sums[];  // [wavefront][gate, up][2][NT][16][16]
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t r = lane & 15, quad = lane >> 4;
  const uint64_t c0 = (uint64_t)blockIdx.x * 16;
  const char *w[2][2], *x[NT];
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const uint64_t c = c0 + n * 8 + (r & 7) < a.n ? c0 + n * 8 + (r & 7) : a.n - 1;
    w[0][n] = a.p[0] + c * a.pstride[0];
    w[1][n] = a.p[1] + c * a.pstride[1];
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
    x[t] = a.q[0] + (uint64_t)(t * 16 + r < a.m ? t * 16 + r : a.m - 1) * a.qstride;
  f32x4 acc[2][2][2][NT];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[h][n][s][t] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
  const uint32_t wq = quad * 2 + (r >> 3);
  const uint32_t whole = (uint32_t)(a.k / (8 * EC)), pieces = (uint32_t)((a.k + 8 * EC - 1) / (8 * EC));
  uint32_t k = wave;
  for (; k + W * (PIECES - 1) < whole; k += W * PIECES) {
    u32x4 pw[PIECES][2][2], px[PIECES][2][NT];
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const uint32_t at = (k + i * W) * 128;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int n = 0; n < 2; ++n) pw[i][h][n] = __builtin_nontemporal_load((const u32x4_any*)(w[h][n] + (at + wq * 16)));
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int t = 0; t < NT; ++t) px[i][s][t] = *(const u32x4_any*)(x[t] + (at + quad * 32 + s * 16));
    }
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[h][n][s][t] = few_mfma<DT>(pw[i][h][n], px[i][s][t], acc[h][n][s][t]);
  }
  for (; k < pieces; k += W) {
    u32x4 q[2][NT];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int t = 0; t < NT; ++t) q[s][t] = few_chunk<DT>(x[t], ((uint64_t)k * 8 + quad * 2 + s) * EC, a.k);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const u32x4 p = few_chunk<DT>(w[h][n], ((uint64_t)k * 8 + wq) * EC, a.k);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int t = 0; t < NT; ++t) acc[h][n][s][t] = few_mfma<DT>(p, q[s][t], acc[h][n][s][t]);
      }
  }
  constexpr uint32_t kPlane = NT * 512;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          sums[(wave * 2 + h) * kPlane + (quad >> 1) * (NT * 256) + (t * 16 + r) * 16 + n * 8 + (quad & 1) * 4 + i] =
              quad < 2 ? acc[h][n][0][t][i] : acc[h][n][1][t][i];
  __syncthreads();
  for (uint32_t o = threadIdx.x; o < NT * 256; o += W * 64) {
    float vg = 0.0f, vu = 0.0f;
#pragma unroll
    for (int i = 0; i < W * 2; ++i) {
      vg += sums[(i >> 1) * 2 * kPlane + (i & 1) * (NT * 256) + o];
      vu += sums[((i >> 1) * 2 + 1) * kPlane + (i & 1) * (NT * 256) + o];
    }
    const uint64_t token = o / 16, col = c0 + o % 16;
    if (token >= a.m || col >= a.n) continue;
    few_store<DT>(a, token, col, vg, vu);
  }
}

template <int DT, int NT, int W, int PIECES>
hipError_t lines_launch(const FfProduct& a, hipStream_t stream) {
  hipLaunchKernelGGL((ff_lines_kernel<DT, NT, W, PIECES>), dim3((unsigned)((a.n + 15) / 16)), dim3(W * 64),
                     W * 2 * NT * 512 * sizeof(float), stream, a);
  return launch_status(stream);
}

// Forward for one or two tokens, on the vector units: a row of a weight is read
// as 1 KiB an instruction, the pattern that reaches the rate of a copy, and each
// lane multiplies what it loaded.  A wavefront has one hidden column, which it
// finishes alone.  Two columns a wavefront share what is read of x and were
// slower (30.5 and 28.5 us): half as many wavefronts take turns waiting.  The
// weights' loads are streaming ones; lines of x stay.
constexpr int kVectorSteps = 4;  // instructions a row on their way; 8 measured the same

template <int DT, int T>
__global__ __launch_bounds__(kThreads) void ff_vector_kernel(FfProduct a) {
  constexpr int EC = 16 / DtypeSize<DT>::value, U = kVectorSteps;
  using Raw = VecRaw<DT, EC>;
  const uint32_t lane = threadIdx.x & 63;
  const uint64_t col = (uint64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  if (col >= a.n) return;
  const char* const w[2] = {a.p[0] + col * a.pstride[0], a.p[1] + col * a.pstride[1]};
  float sum[2][T] = {};
  auto add = [&](const u32x4 (&pw)[2], const u32x4 (&px)[T]) __attribute__((always_inline)) {
    const VecF<EC> g = unpack<DT, EC>(__builtin_bit_cast(Raw, pw[0])), u = unpack<DT, EC>(__builtin_bit_cast(Raw, pw[1]));
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const VecF<EC> x = unpack<DT, EC>(__builtin_bit_cast(Raw, px[t]));
#pragma unroll
      for (int e = 0; e < EC; ++e) {
        sum[0][t] = __builtin_fmaf(g.v[e], x.v[e], sum[0][t]);
        sum[1][t] = __builtin_fmaf(u.v[e], x.v[e], sum[1][t]);
      }
    }
  };
  const uint32_t whole = (uint32_t)(a.k / (64 * EC)), steps = (uint32_t)((a.k + 64 * EC - 1) / (64 * EC));
  uint32_t k = 0;
  for (; k + U <= whole; k += U) {
    u32x4 pw[U][2], px[U][T];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t at = ((k + i) * 64 + lane) * 16;
#pragma unroll
      for (int h = 0; h < 2; ++h) pw[i][h] = __builtin_nontemporal_load((const u32x4_any*)(w[h] + at));
#pragma unroll
      for (int t = 0; t < T; ++t) px[i][t] = *(const u32x4_any*)(a.q[0] + (uint64_t)t * a.qstride + at);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) add(pw[i], px[i]);
  }
  for (; k < steps; ++k) {
    const uint64_t e = ((uint64_t)k * 64 + lane) * EC;
    u32x4 pw[2], px[T];
#pragma unroll
    for (int h = 0; h < 2; ++h) pw[h] = few_chunk<DT>(w[h], e, a.k);
#pragma unroll
    for (int t = 0; t < T; ++t) px[t] = few_chunk<DT>(a.q[0] + (uint64_t)t * a.qstride, e, a.k);
    add(pw, px);
  }
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const float g = wave_sum(sum[0][t]), u = wave_sum(sum[1][t]);
    if (lane == 0) few_store<DT>(a, t, col, g, u);
  }
}

template <int DT, int T>
hipError_t vector_launch(const FfProduct& a, hipStream_t stream) {
  constexpr uint64_t wg = kThreads / 64;
  hipLaunchKernelGGL((ff_vector_kernel<DT, T>), dim3((unsigned)((a.n + wg - 1) / wg)), dim3(kThreads), 0, stream, a);
  return launch_status(stream);
}

// One and two tokens go to the vector units: 28.3 and 30.9 us at 4096 x 11264
// bfloat16 (184 MB, 29 us at the rate of a large copy), 32 and 32 by whole lines;
// at four tokens the rows of x cost more than that saves (37 to 41, and 33).  The
// shapes, us: 16 tokens 37.6, and 38 to 39.6 with 2 or 8 wavefronts, 2 or 8
// pieces; 24 tokens 44, and 46 to 58 with 8 wavefronts or 4 pieces; 64 tokens 67,
// and 78 to 83 with one block of columns, where x is read twice as often.  In
// binary32 the doubled products of whole lines do not have time beyond 16 tokens:
// 24 tokens 143 us so, 108 with each product once (16 tokens 85 and 108).
template <int DT>
hipError_t few_dt(const FfProduct& a, hipStream_t stream) {
  if (a.m == 1) return vector_launch<DT, 1>(a, stream);
  if (a.m == 2) return vector_launch<DT, 2>(a, stream);
  if (a.m <= 16) return lines_launch<DT, 1, 4, 4>(a, stream);
  if constexpr (DT == DT_F32) {
    if (a.m <= 32) return few_launch<DT, 2, 1, 8>(a, stream);
  } else {
    if (a.m <= 32) return lines_launch<DT, 2, 4, 2>(a, stream);
  }
  return few_launch<DT, 4, 2, 4>(a, stream);
}

// ------------------------------------------------------------------ gradients of the product

// dg and du from dh and the kept projections, two vectors a lane over blocks of
// 32 columns.  dg and du lie in the workspace with rows of whole blocks; the
// columns past hidden are made zeros, since dx's product reads whole chunks.
// Bound by memory: 8192 x 11,264 bfloat16 from checkpoints 118 us (744 MB, 6.3
// TB/s), 2048 x 5632 from rows 26 (115 MB, 4.4 TB/s).  dg and du are rounded to
// the activations' type because the products' matrix instructions take that
// type; as the two halves of a split sum they would cost twice the products.
constexpr int kGradUnroll = 2;

template <int DT, bool CK>
__global__ __launch_bounds__(kThreads) void ff_act_grad_kernel(FfBackward a, uint64_t row0, uint32_t blocks, FastDiv nb,
                                                                uint64_t du_at) {
  constexpr int E = vec_elems<DT, DT>(), ES = DtypeSize<DT>::value;
  const uint64_t pitch = (uint64_t)nb.d * kCkptBlock;
  CkptPlace p[kGradUnroll];
  VecF<E> dh[kGradUnroll], g[kGradUnroll], u[kGradUnroll];
#pragma unroll
  for (int k = 0; k < kGradUnroll; ++k) {
    p[k] = ckpt_place<E, kGradUnroll>(k, blocks, nb);
    dh[k] = g[k] = u[k] = {};
    if (!p[k].live) continue;
    const uint64_t row = row0 + p[k].row;
    const int n = vec_count<E>(a.hidden, p[k].col);
    dh[k] = load_vec_upto<DT, E>(a.dh.p + row * a.dh.stride * ES, p[k].col, n);
    if constexpr (CK) {
      g[k] = ckpt_unpack<E>(ckpt_load<E>(a.cgate.code_row(row), a.cgate.exp_row(row), p[k].col));
      u[k] = ckpt_unpack<E>(ckpt_load<E>(a.cup.code_row(row), a.cup.exp_row(row), p[k].col));
    } else {
      g[k] = load_vec_upto<DT, E>(a.gate.p + row * a.gate.stride * ES, p[k].col, n);
      u[k] = load_vec_upto<DT, E>(a.up.p + row * a.up.stride * ES, p[k].col, n);
    }
  }
#pragma unroll
  for (int k = 0; k < kGradUnroll; ++k) {
    if (!p[k].live) continue;
    const int n = vec_count<E>(a.hidden, p[k].col);
    VecF<E> dg = {}, du = {};
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (i < n) {
        float d;
        const float h = ff_act<DT, true>(g[k].v[i], a.act, &d);
        dg.v[i] = dh[k].v[i] * u[k].v[i] * d;
        du.v[i] = dh[k].v[i] * h;
      }
    const uint64_t at = ((row0 + p[k].row) * pitch + p[k].col) * ES;
    *(u32x4*)(a.ws + at) = pack_vec<DT, E>(dg);
    *(u32x4*)(a.ws + du_at + at) = pack_vec<DT, E>(du);
  }
}

template <int DT>
hipError_t act_grad_dt(const FfBackward& a, hipStream_t stream) {
  const uint64_t nb = (a.hidden + kCkptBlock - 1) / kCkptBlock;
  const uint64_t du_at = ff_workspace(a.rows, a.dim, a.hidden, DT).du;
  return by_ckpt_rows<vec_elems<DT, DT>(), kGradUnroll>(a.rows, nb, [&](uint64_t r, uint32_t blocks, dim3 grid) {
    const FastDiv by((uint32_t)nb);
    if (a.saved == 2)
      hipLaunchKernelGGL((ff_act_grad_kernel<DT, true>), grid, dim3(kThreads), 0, stream, a, r, blocks, by, du_at);
    else
      hipLaunchKernelGGL((ff_act_grad_kernel<DT, false>), grid, dim3(kThreads), 0, stream, a, r, blocks, by, du_at);
    return launch_status(stream);
  });
}

// ------------------------------------------------------------------ sums of splits

// Adds the splits of a product in order and rounds; blockIdx.y is the output.
// (2048 x 2048 of four splits 13 us, 71 MB: 5.4 TB/s)
template <int DT>
__global__ __launch_bounds__(kThreads) void ff_join_kernel(FfProduct a) {
  const uint64_t vecs = a.pitch / 4, z = blockIdx.y, plane = a.m * a.pitch;
  for (uint64_t i = (uint64_t)blockIdx.x * kThreads + threadIdx.x; i < a.m * vecs;
       i += (uint64_t)gridDim.x * kThreads) {
    const uint64_t row = i / vecs, col = (i - row * vecs) * 4;
    const float* p = a.partials + z * a.splits * plane + row * a.pitch + col;
    const int n = vec_count<4>(a.n, col);
    VecF<4> v = {};
    for (uint32_t s = 0; s < a.splits; ++s) {
      const VecF<4> w = load_vec<DT_F32, 4>((const char*)(p + s * plane), 0);
#pragma unroll
      for (int e = 0; e < 4; ++e) v.v[e] += w.v[e];
    }
    char* out = a.out[z] + row * a.out_stride[z];
    if (a.accumulate)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < n) v.v[e] += load_elem_dt(out, col + e, a.out_dt);
    if (a.out_dt == DT_F32) store_vec_upto<DT_F32, 4>(out, col, n, v);
    else store_vec_upto<DT, 4>(out, col, n, v);
  }
}

// Sums of splits are few enough for a vector a thread; the zeros of gradients
// without rows can be more than a launch has threads, and go round.
template <int DT>
hipError_t join_dt(const FfProduct& a, int outputs, hipStream_t stream) {
  const uint64_t n = a.m * (a.pitch / 4), groups = std::min<uint64_t>(up_div(n, kThreads), 1 << 20);
  hipLaunchKernelGGL((ff_join_kernel<DT>), dim3((unsigned)groups, outputs), dim3(kThreads), 0, stream, a);
  return launch_status(stream);
}

// ------------------------------------------------------------------ aligned copies

// Rows of `dim` elements copied to rows of whole blocks, zeros after them: what
// direct loads read where the rows themselves begin off 16 bytes.  1021 x 1001
// and twice 2731 x 1001 float16: 6 us, for which dx's product and the weights'
// take direct loads (27 and 25 us; the forward pass, which has no workspace,
// takes 48 of as many operations through registers).
struct FfCopy {
  const char* from[3];
  uint64_t stride[3], rows[3];
  char* to[3];
};
template <int DT>
__global__ __launch_bounds__(kThreads) void ff_copy_kernel(FfCopy a, uint64_t dim, uint32_t nb) {
  constexpr int E = vec_elems<DT, DT>(), ES = DtypeSize<DT>::value, LB = kCkptBlock / E;
  const uint32_t m = blockIdx.y;
  for (uint64_t block = (uint64_t)blockIdx.x * (kThreads / LB) + threadIdx.x / LB; block < a.rows[m] * nb;
       block += (uint64_t)gridDim.x * (kThreads / LB)) {
    const uint64_t row = block / nb;
    const uint32_t col = (uint32_t)(block - row * nb) * kCkptBlock + threadIdx.x % LB * E;
    const VecF<E> v = load_vec_upto<DT, E>(a.from[m] + row * a.stride[m] * ES, col, vec_count<E>(dim, col));
    *(u32x4*)(a.to[m] + block * kCkptBlock * ES + threadIdx.x % LB * 16) = pack_vec<DT, E>(v);
  }
}

template <int DT>
hipError_t copy_dt(const FfCopy& a, uint64_t dim, hipStream_t stream) {
  constexpr uint64_t wg = kThreads / (kCkptBlock / vec_elems<DT, DT>());
  const uint64_t nb = (dim + kCkptBlock - 1) / kCkptBlock;
  const uint64_t most = std::max(a.rows[0], std::max(a.rows[1], a.rows[2])) * nb;
  const dim3 grid((unsigned)std::min<uint64_t>((most + wg - 1) / wg, 1 << 16), 3);
  hipLaunchKernelGGL((ff_copy_kernel<DT>), grid, dim3(kThreads), 0, stream, a, dim, (uint32_t)nb);
  return launch_status(stream);
}

// ------------------------------------------------------------------ which kernel

constexpr uint64_t kFewTokens = 64;
constexpr uint64_t kCus = 256;

uint64_t es_of(int dt) { return dt == DT_F32 ? 4 : 2; }
uint64_t blocks_pitch(uint64_t n) { return up_div(n, kCkptBlock) * kCkptBlock; }

// Direct loads move 16 bytes from a 16-byte boundary.
bool direct_ok(const char* p, uint64_t stride_bytes) { return (((uint64_t)p | stride_bytes) & 15) == 0; }

// How a product of the backward pass is cut: tiles of 256 x 256 (of direct loads
// only) or the smaller ones, and splits of its terms for CUs that the tiles leave
// without work, of at least eight stages each.  Both sides, us of bfloat16 with
// the gradients of the product before it:
//   large tiles where they give every CU one: 8192 x 4096 x 11,264 towards x
//   1337 (small ones 3266), towards the weights 1469 (1756);
//   large tiles, split as often as every CU gets one, where there are at least a
//   quarter as many tiles as CUs and the sum is long: towards x 64 tiles of 2048
//   x 2048 x 5632 120 (small ones, unsplit, 192), 72 of 2304 x 2048 x 5632 138
//   (344); unsplit above half as many, 130 of 2560 x 3328 x 2816 142 (250), 220
//   of 2816 x 5120 x 2816 155 (332), 240 of 3840 x 4096 x 2816 163 (339);
//   towards the weights 130 of 8192 x 3328 x 1280 198 (266), 220 of 8192 x 2816 x
//   2560 234 (310);
//   small ones otherwise: 1024 x 1024 x 2816 towards the weights 30.5 (large
//   44), towards x 38 (40.5);
//   splits: 1024 x 1024 x 2816 towards x 38 (unsplit 89), 65 x 4096 x 11,264 63
//   (337), binary32 513 x 1024 x 2816 76 (198).
// Small tiles of rows off 16 bytes are split by their own number, not the large
// ones': 1024 x 4096 x 4096 towards x 152 (split as the large ones 216).
struct FfCut {
  bool wide;
  uint32_t splits;
};
FfCut cut_of(uint64_t m, uint64_t n, uint64_t outputs, uint64_t ktiles, int dt, bool direct) {
  if (dt == DT_F32) {
    const uint64_t tiles = up_div(m, 64) * up_div(n, 64) * outputs;
    return {false, (uint32_t)std::max<uint64_t>(1, std::min(4 * kCus / std::max<uint64_t>(tiles, 1), ktiles / 8))};
  }
  const uint64_t wide = up_div(m, 256) * up_div(n, 256) * outputs, small = up_div(m, 128) * up_div(n, 128) * outputs;
  if (direct && wide >= kCus) return {true, 1};
  if (direct && wide >= kCus / 4 && ktiles >= 64) return {true, (uint32_t)(kCus / wide)};
  if (small >= kCus) return {false, 1};
  return {false, (uint32_t)std::max<uint64_t>(1, std::min(kCus / std::max<uint64_t>(small, 1), ktiles / 8))};
}
uint64_t stage_terms(int dt) { return 128 / es_of(dt); }
FfCut dx_cut(uint64_t rows, uint64_t dim, uint64_t hidden, int dt, bool direct) {
  return cut_of(rows, dim, 1, 2 * up_div(hidden, stage_terms(dt)), dt, direct);
}
FfCut dw_cut(uint64_t rows, uint64_t dim, uint64_t hidden, int dt, bool direct) {
  return cut_of(hidden, dim, 2, up_div(rows, stage_terms(dt)), dt, direct);
}
uint64_t partial_pitch(uint64_t n) { return up_div(n, 4) * 4; }

template <class F>
hipError_t by_type(int dt, F f) {
  switch (dt) {
    case DT_F32: return f(std::integral_constant<int, DT_F32>());
    case DT_F16: return f(std::integral_constant<int, DT_F16>());
    default: return f(std::integral_constant<int, DT_BF16>());
  }
}

}  // namespace

uint64_t ff_tile_count(uint64_t m, uint64_t n) { return up_div(m, 64) * up_div(n, 64); }

FfWorkspace ff_workspace(uint64_t rows, uint64_t dim, uint64_t hidden, int dt) {
  const uint64_t es = es_of(dt);
  auto room = [](uint64_t bytes) { return up_div(bytes, 256) * 256; };
  FfWorkspace w;
  w.pitch = blocks_pitch(hidden);
  w.du = room(rows * w.pitch * es);
  w.x = 2 * w.du;
  // odd widths: aligned copies of x and the weights
  const bool copies = rows && dim % (16 / es) != 0;
  w.copy_pitch = copies ? blocks_pitch(dim) : 0;
  w.wgate = w.x + room(rows * w.copy_pitch * es);
  w.wup = w.wgate + room(hidden * w.copy_pitch * es);
  w.partials = w.wup + room(hidden * w.copy_pitch * es);
  // whether the loads are direct ones is not known here: room for either cut
  uint64_t sx = 1, sw = 1;
  for (const bool direct : {false, true}) {
    sx = std::max<uint64_t>(sx, dx_cut(rows, dim, hidden, dt, direct).splits);
    sw = std::max<uint64_t>(sw, dw_cut(rows, dim, hidden, dt, direct).splits);
  }
  const uint64_t bx = sx > 1 ? sx * rows : 0, bw = sw > 1 ? sw * 2 * hidden : 0;
  w.bytes = w.partials + std::max(bx, bw) * partial_pitch(dim) * sizeof(float);
  return w;
}

hipError_t launch_gated_ff(const FfForward& f, hipStream_t stream) {
  const uint64_t es = es_of(f.dt);
  FfProduct a{};
  a.p[0] = f.wgate.p;
  a.p[1] = f.wup.p;
  a.pstride[0] = (uint32_t)(f.wgate.stride * es);
  a.pstride[1] = (uint32_t)(f.wup.stride * es);
  a.q[0] = a.q[1] = f.x.p;
  a.qstride = (uint32_t)(f.x.stride * es);
  a.m = f.rows;
  a.n = f.hidden;
  a.k = f.dim;
  a.splits = 1;
  a.act = f.act;
  a.saved = f.saved;
  a.out[0] = f.h.p;
  a.out_stride[0] = f.h.stride * es;
  a.gate = f.gate;
  a.up = f.up;
  a.cgate = f.cgate;
  a.cup = f.cup;
  // At 4096 x 11,264 bfloat16 64 tokens take 68 us, 65 in tiles 76; at 1024 x
  // 2816 15 and 17.6.  Kept as checkpoints few tokens go through the tiles too, 71
  // us for one and 77 for 64 (with kept rows 29 and 68): they find a block's
  // largest value in registers, the kernels of few tokens store their sums one by
  // one.
  if (f.rows <= kFewTokens && f.saved != 2)
    return by_type(f.dt, [&](auto t) { return few_dt<decltype(t)::value>(a, stream); });
  const bool direct = f.dim % (16 / es) == 0 && direct_ok(a.p[0], a.pstride[0]) && direct_ok(a.p[1], a.pstride[1]) &&
                      direct_ok(a.q[0], a.qstride);
  // large tiles where they give every CU one: 8192 x 4096 x 11,264 bfloat16 1150
  // us (small ones 1636), 2048 x 2048 x 5632 104 (103); where they do not: 511 x
  // 2048 x 5632 50 and 34, 1024 x 1024 x 2816 31 and 20.7
  const bool wide = direct && f.dt != DT_F32 && up_div(f.rows, 256) * up_div(f.hidden, 128) >= kCus;
  return launch_ff_forward_tiles(f.dt, a, wide, direct, stream);
}

hipError_t launch_gated_ff_grad(const FfBackward& b, hipStream_t stream) {
  const uint64_t es = es_of(b.dt);
  const FfWorkspace ws = ff_workspace(b.rows, b.dim, b.hidden, b.dt);
  hipError_t e = hipSuccess;
  Rows x = b.x, wgate = b.wgate, wup = b.wup;
  if (b.rows) {
    e = by_type(b.dt, [&](auto t) { return act_grad_dt<decltype(t)::value>(b, stream); });
    if (e != hipSuccess) return e;
  }
  if (ws.copy_pitch) {
    FfCopy c{};
    auto copy = [&](int i, Rows& m, uint64_t rows, uint64_t at) {
      c.from[i] = m.p;
      c.stride[i] = m.stride;
      c.rows[i] = rows;
      c.to[i] = b.ws + at;
      m.p = c.to[i];
      m.stride = ws.copy_pitch;
    };
    if (b.dwgate.p) copy(0, x, b.rows, ws.x);
    if (b.dx.p) {
      copy(1, wgate, b.hidden, ws.wgate);
      copy(2, wup, b.hidden, ws.wup);
    }
    e = by_type(b.dt, [&](auto t) { return copy_dt<decltype(t)::value>(c, b.dim, stream); });
    if (e != hipSuccess) return e;
  }
  auto product = [&](bool dx) {
    FfProduct a{};
    a.q[0] = b.ws;
    a.q[1] = b.ws + ws.du;
    a.qstride = (uint32_t)(ws.pitch * es);
    a.partials = (float*)(b.ws + ws.partials);
    a.pitch = partial_pitch(b.dim);
    a.n = b.dim;
    FfCut cut;
    bool direct;
    if (dx) {
      a.p[0] = wgate.p;
      a.p[1] = wup.p;
      a.pstride[0] = (uint32_t)(wgate.stride * es);
      a.pstride[1] = (uint32_t)(wup.stride * es);
      a.m = b.rows;
      a.k = b.hidden;
      a.out[0] = b.dx.p;
      a.out_stride[0] = b.dx.stride * es;
      a.out_dt = b.dt;
      direct = direct_ok(a.p[0], a.pstride[0]) && direct_ok(a.p[1], a.pstride[1]);
      cut = dx_cut(b.rows, b.dim, b.hidden, b.dt, direct);
    } else {
      a.p[0] = a.p[1] = x.p;
      a.pstride[0] = a.pstride[1] = (uint32_t)(x.stride * es);
      a.m = b.hidden;
      a.k = b.rows;
      const uint64_t oes = es_of(b.wdt);
      a.out[0] = b.dwgate.p;
      a.out[1] = b.dwup.p;
      a.out_stride[0] = b.dwgate.stride * oes;
      a.out_stride[1] = b.dwup.stride * oes;
      a.out_dt = b.wdt;
      a.accumulate = b.accumulate;
      direct = direct_ok(a.p[0], a.pstride[0]);
      cut = dw_cut(b.rows, b.dim, b.hidden, b.dt, direct);
    }
    hipError_t r = hipSuccess;
    if (a.k) {
      a.splits = cut.splits;
      r = dx ? launch_ff_dx(b.dt, a, cut.wide, direct, stream)
             : launch_ff_dw(b.dt, a, cut.wide, direct, stream);
      if (r != hipSuccess || a.splits == 1) return r;
    }
    // without rows the weights' gradients are sums of nothing
    return by_type(b.dt, [&](auto t) { return join_dt<decltype(t)::value>(a, dx ? 1 : 2, stream); });
  };
  if (b.dx.p && b.rows) e = product(true);
  if (e == hipSuccess && b.dwgate.p) e = product(false);
  return e;
}

}  // namespace rar
