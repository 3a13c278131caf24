// Layer norm, forward and backward (mean and variance over each row, gain and bias).
//
//   mean = (1/d) sum_j x_j,  var = (1/d) sum_j (x_j - mean)^2,  rstd = 1 / sqrt(var + eps),
//   xh = (x - mean) rstd,  y = xh g + b;
//   u = dY g,  dX = rstd (u - mean(u) - xh mean(u xh)) (+ dres),
//   dg_j = sum_t dY_tj xh_tj,  db_j = sum_t dY_tj.
// All sums are fp32 in a fixed order; the variance is summed about the mean, not as
// E[x^2] - mean^2, which would cancel for rows whose mean is large.
#include "fp8q_common.cuh"
#include "fp8q_internal.h"

namespace fp8q {

namespace {

template <int F32>
__device__ __forceinline__ float ln_load(const void* p, int64_t i) {
  if (F32) return static_cast<const float*>(p)[i];
  return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
}
template <int F32>
__device__ __forceinline__ void ln_store(void* p, int64_t i, float v) {
  if (F32) static_cast<float*>(p)[i] = v;
  else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// Sum over the block in a fixed order; result valid in every thread.
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  __syncthreads();
  if (lane == 0) red[warp] = v;
  __syncthreads();
  float t = lane < nw ? red[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
  return t;
}

template <int F32>
__global__ void __launch_bounds__(256) k_layernorm_fwd(const void* x, const void* g, const void* b, int d, float eps,
                                                       void* y, float* mean, float* rstd) {
  __shared__ float red[32];
  const int64_t row = blockIdx.x, base = row * d;
  float s = 0.0f;
  for (int j = threadIdx.x; j < d; j += blockDim.x) s += ln_load<F32>(x, base + j);
  const float mu = block_sum(s, red) / (float)d;
  s = 0.0f;
  for (int j = threadIdx.x; j < d; j += blockDim.x) {
    const float c = ln_load<F32>(x, base + j) - mu;
    s += c * c;
  }
  const float rs = 1.0f / sqrtf(block_sum(s, red) / (float)d + eps);
  for (int j = threadIdx.x; j < d; j += blockDim.x) {
    const float xh = (ln_load<F32>(x, base + j) - mu) * rs;
    ln_store<F32>(y, base + j, xh * ln_load<F32>(g, j) + (b ? ln_load<F32>(b, j) : 0.0f));
  }
  if (threadIdx.x == 0) {
    mean[row] = mu;
    rstd[row] = rs;
  }
}

template <int F32>
__global__ void __launch_bounds__(256) k_layernorm_bwd_rows(const void* dY, const void* x, const void* g,
                                                            const float* mean, const float* rstd, const void* dres,
                                                            int d, void* dX) {
  __shared__ float red[32];
  const int64_t row = blockIdx.x, base = row * d;
  const float mu = mean[row], rs = rstd[row];
  float su = 0.0f, sux = 0.0f;
  for (int j = threadIdx.x; j < d; j += blockDim.x) {
    const float u = ln_load<F32>(dY, base + j) * ln_load<F32>(g, j);
    su += u;
    sux += u * ((ln_load<F32>(x, base + j) - mu) * rs);
  }
  const float mu_u = block_sum(su, red) / (float)d;
  const float mu_ux = block_sum(sux, red) / (float)d;
  for (int j = threadIdx.x; j < d; j += blockDim.x) {
    const float u = ln_load<F32>(dY, base + j) * ln_load<F32>(g, j);
    const float xh = (ln_load<F32>(x, base + j) - mu) * rs;
    const float v = rs * (u - mu_u - xh * mu_ux);
    ln_store<F32>(dX, base + j, dres ? v + ln_load<F32>(dres, base + j) : v);
  }
}

// Partial sums of dg and db over a run of kLnRows rows: part [blocks][2][d].
template <int F32>
__global__ void __launch_bounds__(256) k_layernorm_bwd_cols(const void* dY, const void* x, const float* mean,
                                                            const float* rstd, int64_t T, int d, float* part) {
  const int j = blockIdx.x * blockDim.x + threadIdx.x;
  if (j >= d) return;
  const int64_t t0 = (int64_t)blockIdx.y * kLnRows, t1 = t0 + kLnRows < T ? t0 + kLnRows : T;
  float sg = 0.0f, sb = 0.0f;
  for (int64_t t = t0; t < t1; ++t) {
    const float dy = ln_load<F32>(dY, t * d + j);
    sg += dy * ((ln_load<F32>(x, t * d + j) - mean[t]) * rstd[t]);
    sb += dy;
  }
  float* p = part + (int64_t)blockIdx.y * 2 * d;
  p[j] = sg;
  p[d + j] = sb;
}
__global__ void __launch_bounds__(256) k_layernorm_bwd_finish(const float* part, int nblk, int d, float* dg, float* db) {
  const int j = blockIdx.x * blockDim.x + threadIdx.x;
  if (j >= d) return;
  float sg = 0.0f, sb = 0.0f;
  for (int k = 0; k < nblk; ++k) {
    sg += part[(int64_t)k * 2 * d + j];
    sb += part[(int64_t)k * 2 * d + d + j];
  }
  dg[j] = sg;
  if (db) db[j] = sb;
}

cudaError_t launched(const Launch& L) {
  if (L.launches) ++*L.launches;
  return cudaGetLastError();
}

}  // namespace

int layernorm_bwd_blocks(int64_t T, int d) {
  (void)d;
  return (int)((T + kLnRows - 1) / kLnRows);
}

cudaError_t launch_layernorm_fwd(const void* x, int f32, const void* g, const void* b, int64_t T, int d, float eps,
                                 void* y, float* mean, float* rstd, const Launch& L) {
  if (f32) k_layernorm_fwd<1><<<(unsigned)T, 256, 0, L.stream>>>(x, g, b, d, eps, y, mean, rstd);
  else k_layernorm_fwd<0><<<(unsigned)T, 256, 0, L.stream>>>(x, g, b, d, eps, y, mean, rstd);
  return launched(L);
}

cudaError_t launch_layernorm_bwd(const void* dY, const void* x, int f32, const void* g, const float* mean,
                                 const float* rstd, const void* dres, int64_t T, int d, void* dX, float* dg, float* db,
                                 float* part, const Launch& L) {
  const int nblk = layernorm_bwd_blocks(T, d);
  const dim3 cols((d + 255) / 256, nblk);
  if (f32) {
    k_layernorm_bwd_cols<1><<<cols, 256, 0, L.stream>>>(dY, x, mean, rstd, T, d, part);
    k_layernorm_bwd_rows<1><<<(unsigned)T, 256, 0, L.stream>>>(dY, x, g, mean, rstd, dres, d, dX);
  } else {
    k_layernorm_bwd_cols<0><<<cols, 256, 0, L.stream>>>(dY, x, mean, rstd, T, d, part);
    k_layernorm_bwd_rows<0><<<(unsigned)T, 256, 0, L.stream>>>(dY, x, g, mean, rstd, dres, d, dX);
  }
  cudaError_t e = launched(L);
  if (e != cudaSuccess) return e;
  if (L.launches) ++*L.launches;
  k_layernorm_bwd_finish<<<(d + 255) / 256, 256, 0, L.stream>>>(part, nblk, d, dg, db);
  return launched(L);
}

}  // namespace fp8q
