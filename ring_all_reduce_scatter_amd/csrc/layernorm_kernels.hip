// Layer norm forward and backward for gfx950.
//
//   mu = mean x,  r = 1 / sqrt(mean (x - mu)^2 + eps),  h = (x - mu) r,  y = round(h w + b)
//   g = dy w,     dx = round(r (g - mean g - h mean(g h)))
//   dw = round(sum over rows of dy h [+ dw]),   db = round(sum over rows of dy [+ db])
//
// All statistics and sums are binary32; the variance is taken about the
// mean (two passes over the row), not as a difference of moments.  The sums
// over rows are formed in a fixed order: each of `splits` row groups on its
// own, then the groups in order.
#include "operator_launch.hpp"
#include "row_access.hpp"

namespace rar {
namespace {

constexpr int kWaves = kThreads / 64;

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
  const float inv = 1.0f / (float)dim;
  for (uint64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const char* xr = x.p + r * x.stride * DtypeSize<DT>::value;
    char* yr = y.p + r * y.stride * DtypeSize<DT>::value;
    float s = 0.0f;
    for (uint64_t c = threadIdx.x; c < dim; c += kThreads) s += load_elem<DT>(xr, c);
    const float mu = block_sum(s, red) * inv;
    float q = 0.0f;
    for (uint64_t c = threadIdx.x; c < dim; c += kThreads) {
      const float d = load_elem<DT>(xr, c) - mu;
      q = __builtin_fmaf(d, d, q);
    }
    const float rs = 1.0f / __builtin_sqrtf(block_sum(q, red) * inv + eps);
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
template <int DT>
__global__ __launch_bounds__(kThreads) void layernorm_dw_part_kernel(LayernormGrad a, uint64_t rows, uint64_t dim,
                                                                      uint64_t per) {
  const uint64_t c = (uint64_t)blockIdx.x * kThreads + threadIdx.x;
  if (c >= dim) return;
  const uint64_t r0 = blockIdx.y * per, r1 = r0 + per < rows ? r0 + per : rows;
  float dw = 0.0f, db = 0.0f;
  for (uint64_t r = r0; r < r1; ++r) {
    const float dy = load_elem<DT>(a.dy.p, r * a.dy.stride + c);
    const float h = (load_elem<DT>(a.x.p, r * a.x.stride + c) - a.mean[r]) * a.rstd[r];
    dw = __builtin_fmaf(dy, h, dw);
    db += dy;
  }
  a.partials[(uint64_t)blockIdx.y * 2 * dim + c] = dw;
  a.partials[((uint64_t)blockIdx.y * 2 + 1) * dim + c] = db;
}

__global__ __launch_bounds__(kThreads) void layernorm_dw_join_kernel(LayernormGrad a, uint64_t splits, uint64_t dim) {
  const uint64_t c = (uint64_t)blockIdx.x * kThreads + threadIdx.x;
  if (c >= dim) return;
  float dw = 0.0f, db = 0.0f;
  for (uint64_t s = 0; s < splits; ++s) {
    dw += a.partials[s * 2 * dim + c];
    db += a.partials[(s * 2 + 1) * dim + c];
  }
  if (a.dweight) {
    if (a.accumulate) dw += load_elem_dt((const char*)a.dweight, c, a.wdt);
    store_elem_dt((char*)a.dweight, c, a.wdt, dw);
  }
  if (a.dbias) {
    if (a.accumulate) db += load_elem_dt((const char*)a.dbias, c, a.wdt);
    store_elem_dt((char*)a.dbias, c, a.wdt, db);
  }
}

template <int DT>
__global__ __launch_bounds__(kThreads) void layernorm_dx_kernel(LayernormGrad a, uint64_t rows, uint64_t dim) {
  extern __shared__ float red[];
  const float inv = 1.0f / (float)dim;
  for (uint64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const char* xr = a.x.p + r * a.x.stride * DtypeSize<DT>::value;
    const char* yr = a.dy.p + r * a.dy.stride * DtypeSize<DT>::value;
    char* dr = a.dx.p + r * a.dx.stride * DtypeSize<DT>::value;
    const float mu = a.mean[r], rs = a.rstd[r];
    float sg = 0.0f, sgh = 0.0f;
    for (uint64_t c = threadIdx.x; c < dim; c += kThreads) {
      const float g = load_elem<DT>(yr, c) * weight_at(a.weight, a.wdt, c, 1.0f);
      sg += g;
      sgh = __builtin_fmaf(g, (load_elem<DT>(xr, c) - mu) * rs, sgh);
    }
    const float mg = block_sum(sg, red) * inv;
    const float mgh = block_sum(sgh, red) * inv;
    for (uint64_t c = threadIdx.x; c < dim; c += kThreads) {
      const float g = load_elem<DT>(yr, c) * weight_at(a.weight, a.wdt, c, 1.0f);
      const float h = (load_elem<DT>(xr, c) - mu) * rs;
      store_elem<DT>(dr, c, rs * (g - mg - h * mgh));
    }
  }
}

unsigned row_grid(uint64_t rows) { return (unsigned)(rows < 65536 ? rows : 65536); }

template <int DT>
hipError_t layernorm_grad_dt(const LayernormGrad& a, uint64_t rows, uint64_t dim, hipStream_t stream) {
  hipError_t e = hipSuccess;
  // dw and db first: dx may be written over dy or x
  if (a.dweight || a.dbias) {
    const uint64_t splits = layernorm_splits(rows, dim);
    const unsigned cols = (unsigned)((dim + kThreads - 1) / kThreads);
    if (rows) {
      hipLaunchKernelGGL((layernorm_dw_part_kernel<DT>), dim3(cols, (unsigned)splits), dim3(kThreads), 0, stream, a,
                         rows, dim, (rows + splits - 1) / splits);
      if ((e = launch_status(stream)) != hipSuccess) return e;
    }
    hipLaunchKernelGGL(layernorm_dw_join_kernel, dim3(cols), dim3(kThreads), 0, stream, a, rows ? splits : 0, dim);
    if ((e = launch_status(stream)) != hipSuccess) return e;
  }
  if (a.dx.p && rows) {
    hipLaunchKernelGGL((layernorm_dx_kernel<DT>), dim3(row_grid(rows)), dim3(kThreads), kWaves * sizeof(float), stream,
                       a, rows, dim);
    e = launch_status(stream);
  }
  return e;
}

}  // namespace

hipError_t launch_layernorm(const Rows& x, const void* weight, const void* bias, int wdt, uint64_t rows, uint64_t dim,
                            float eps, const Rows& y, float* mean, float* rstd, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  const dim3 grid(row_grid(rows)), block(kThreads);
  const size_t lds = kWaves * sizeof(float);
  switch (x.dt) {
    case DT_F32:
      hipLaunchKernelGGL((layernorm_kernel<DT_F32>), grid, block, lds, stream, x, weight, bias, wdt, rows, dim, eps, y,
                         mean, rstd);
      break;
    case DT_F16:
      hipLaunchKernelGGL((layernorm_kernel<DT_F16>), grid, block, lds, stream, x, weight, bias, wdt, rows, dim, eps, y,
                         mean, rstd);
      break;
    default:
      hipLaunchKernelGGL((layernorm_kernel<DT_BF16>), grid, block, lds, stream, x, weight, bias, wdt, rows, dim, eps,
                         y, mean, rstd);
  }
  return launch_status(stream);
}

uint64_t layernorm_splits(uint64_t rows, uint64_t dim) {
  (void)dim;
  const uint64_t s = (rows + 63) / 64;
  return s < 1 ? 1 : (s > 256 ? 256 : s);
}

hipError_t launch_layernorm_grad(const LayernormGrad& a, uint64_t rows, uint64_t dim, hipStream_t stream) {
  switch (a.x.dt) {
    case DT_F32: return layernorm_grad_dt<DT_F32>(a, rows, dim, stream);
    case DT_F16: return layernorm_grad_dt<DT_F16>(a, rows, dim, stream);
    default: return layernorm_grad_dt<DT_BF16>(a, rows, dim, stream);
  }
}

}  // namespace rar
