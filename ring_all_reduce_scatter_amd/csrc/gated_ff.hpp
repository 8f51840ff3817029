// Gated feed-forward block: what its kernels share.
//
//   g = x Wg^T,  u = x Wu^T,  h = round(act(g) u)
//   dg = round(dh u act'(g)),  du = round(dh act(g))
//   dx = round(dg Wg + du Wu),  dWg = round(dg^T x [+ dWg]),  dWu the same of du
//
// x is rows x dim, Wg and Wu hidden x dim, everything else rows x hidden.
#pragma once

#include "operator_launch.hpp"
#include "row_access.hpp"

namespace rar {

enum FfAct : int { FF_SILU = 0, FF_GELU = 1, FF_GELU_TANH = 2 };

// The logistic function s = 1 / (1 + exp(-z)) and s (1 - s).  For 16 bits from
// the hardware's 2^x and reciprocal (1 ulp each): the rounding of z log2(e) adds
// |z| 2^-24 of the exponential, which no rounding to 16 bits shows, and below
// 2^-126 the result is 0.  In binary32 from exp(-|z|), which never overflows, so
// that far negative z keep their digits, down to the subnormals (1 % of the
// gradients of 2048 x 2048 x 5632, nothing that shows of the forward pass).
struct FfLogistic {
  float s, slope;
};
template <int DT>
__device__ __forceinline__ FfLogistic ff_logistic(float z) {
  if constexpr (DT == DT_F32) {
    const float t = expf(-__builtin_fabsf(z)), r = __builtin_amdgcn_rcpf(1.0f + t);
    return {z >= 0.0f ? r : t * r, t * r * r};
  } else {
    const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504f));
    return {s, s * (1.0f - s)};
  }
}

// act(g), for results of type DT, and (D) its derivative.  The tanh form of gelu
// is g s(2 z) with z = c (g + 0.044715 g^3): (1 + tanh z) / 2 is the logistic
// function of 2 z.  s (1 - s) first: it is zero where g is large.  The sum (1 +
// erf) / 2 loses its digits where erf is near -1, so in binary32 it is taken as
// erfc(-x) / 2; in 16 bits the sum's error, 2^-24, passes their rounding only
// where act(g) is below 2^-10, and erfc costs 3 us of 116 forward (2048 x 2048 x
// 5632).
template <int DT, bool D>
__device__ __forceinline__ float ff_act(float g, int act, float* d) {
  if (act == FF_GELU) {
    float p, e;
    if constexpr (DT == DT_F32) {
      p = 0.5f * erfcf(g * -0.70710678f);
      if constexpr (D) e = expf(g * g * -0.5f);
    } else {
      p = 0.5f + 0.5f * erff(g * 0.70710678f);
      if constexpr (D) e = __builtin_amdgcn_exp2f(g * g * -0.72134752f);
    }
    if constexpr (D) *d = p + g * 0.39894228f * e;
    return g * p;
  }
  if (act == FF_SILU) {
    const FfLogistic f = ff_logistic<DT>(g);
    if constexpr (D) *d = f.s + g * f.slope;
    return g * f.s;
  }
  // past 128 the logistic function is 0 or 1, and the square must not overflow
  const float g2 = __builtin_fminf(g * g, 16384.0f);
  const FfLogistic f = ff_logistic<DT>(1.59576912f * g * (1.0f + 0.044715f * g2));
  if constexpr (D) *d = f.s + g * f.slope * (1.59576912f * (1.0f + 3.0f * 0.044715f * g2));
  return g * f.s;
}

// One product's operands: P indexes the output's columns, Q its rows.
struct FfProduct {
  const char* p[2];
  const char* q[2];
  uint32_t pstride[2], qstride;  // bytes between rows
  uint64_t m, n, k;              // rows and columns of the output, terms of a segment
  uint32_t splits;                            // wanted; the launch makes it what there is work for
  uint32_t tiles_m, tiles_n, ktiles, per_split;  // set by the launch; stages of all segments, of a split
  int act, saved;
  char* out[2];
  uint64_t out_stride[2];  // bytes
  int out_dt;
  bool accumulate;
  Rows gate, up;
  Checkpoint cgate, cup;
  float* partials;  // [output][split][m][pitch]
  uint64_t pitch;
};

enum FfKind : int { FF_FORWARD = 0, FF_DX = 1, FF_DW = 2 };

// One product's launch (gated_ff_forward.hip, gated_ff_dx.hip,
// gated_ff_dw.hip), of at least one term.
hipError_t launch_ff_forward_tiles(int dt, FfProduct& a, bool wide, bool direct, hipStream_t stream);
hipError_t launch_ff_dx(int dt, FfProduct& a, bool wide, bool direct, hipStream_t stream);
hipError_t launch_ff_dw(int dt, FfProduct& a, bool wide, bool direct, hipStream_t stream);

}  // namespace rar
