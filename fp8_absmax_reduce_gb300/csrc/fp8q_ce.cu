// Softmax cross entropy of a linear head over a large vocabulary, without keeping the logits.
//
//   z = x W^T,  lse_t = log sum_v e^{z_tv},  loss_t = lse_t - z_{t,y_t} (0 for an ignored token);
//   G = dloss_t (e^{z - lse_t} - 1[v = y_t]) (0 for an ignored token),  dX = G W,  dW = G^T x.
// The vocabulary is walked in pieces; the backward computes each piece's logits again.  G is kept in
// bf16, the tensor cores' operand type, as G / s with s = max_t |dloss_t|: a mean's one weight for
// all tokens then leaves no rounding of its own in G's large entries (p - 1 near -1).  s joins the
// products in fp32.  An ignored token's row of x is replaced by zero before dW = G^T x, so that a
// padded row may hold anything (0 times a NaN would reach every row of dW).
#include "fp8q_common.cuh"
#include "fp8q_internal.h"

namespace fp8q {

namespace {

// A target outside [0, V) that is not ignore_index is a mistake of the caller: recorded, and ignored.
__device__ __forceinline__ int64_t ce_target(int64_t y, int64_t V, int64_t ignore, unsigned* status) {
  if (y == ignore) return -1;
  if (y < 0 || y >= V) {
    atomicOr(status, kStatusBadTarget);
    return -1;
  }
  return y;
}

__device__ __forceinline__ float ce_warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}
__device__ __forceinline__ float ce_warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// One warp per row: joins a piece's logits into the running maximum, sum and target logit.
__global__ void __launch_bounds__(256) k_ce_piece(const float* z, int64_t ldz, int64_t T, int v0, int n,
                                                  const int64_t* targets, int64_t V, int64_t ignore, float* run_m,
                                                  float* run_s, float* run_y, float* loss, float* lse, int last,
                                                  unsigned* status) {
  const int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (t >= T) return;
  const float* row = z + t * ldz;
  float m = -INFINITY;
  for (int j = lane; j < n; j += 32) m = fmaxf(m, row[j]);
  m = ce_warp_max(m);
  float s = 0.0f;
  for (int j = lane; j < n; j += 32) s += expf(row[j] - m);
  s = ce_warp_sum(s);
  if (lane == 0) {
    const int64_t y = ce_target(targets[t], V, ignore, status);
    float zy = v0 ? run_y[t] : 0.0f;
    if (y >= v0 && y < v0 + n) zy = row[y - v0];
    if (v0) {
      const float m0 = run_m[t], mm = fmaxf(m0, m);
      s = run_s[t] * expf(m0 - mm) + s * expf(m - mm);
      m = mm;
    }
    run_m[t] = m;
    run_s[t] = s;
    run_y[t] = zy;
    if (last) {
      const float l = m + logf(s);
      lse[t] = l;
      loss[t] = y >= 0 ? l - zy : 0.0f;
    }
  }
}

// s = max |dloss| over the tokens that count (1 where that is 0 or not finite); scale = {s, 1}.
__global__ void __launch_bounds__(1024) k_ce_scale(const float* dloss, const int64_t* targets, int64_t T, int64_t V,
                                                   int64_t ignore, float* scale, unsigned* status) {
  __shared__ uint32_t red[32];
  uint32_t m = 0;
  for (int64_t t = threadIdx.x; t < T; t += blockDim.x)
    if (ce_target(targets[t], V, ignore, status) >= 0) m = max(m, abs_bits(dloss[t]));
  m = block_max_u32(m, red);
  if (threadIdx.x == 0) {
    scale[0] = (m == 0 || m >= 0x7F800000u) ? 1.0f : __uint_as_float(m);
    scale[1] = 1.0f;
  }
}

// x with the rows of ignored tokens zeroed.
__global__ void __launch_bounds__(256) k_ce_mask_x(const uint16_t* x, const int64_t* targets, int64_t T, int d, int64_t V,
                                                   int64_t ignore, uint16_t* xz) {
  const int64_t n8 = T * d / 8;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n8; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t y = targets[i * 8 / d];
    const bool keep = y != ignore && y >= 0 && y < V;
    st_v4(xz + 8 * i, keep ? ld_v4(x + 8 * i) : make_uint4(0, 0, 0, 0));
  }
}

__global__ void __launch_bounds__(256) k_ce_grad(const float* z, int64_t ldz, int64_t T, int v0, int n,
                                                 const int64_t* targets, int64_t V, int64_t ignore, const float* lse,
                                                 const float* dloss, const float* scale, uint16_t* G, int64_t ldg) {
  const int64_t t = blockIdx.x;
  const int64_t y = targets[t];
  const bool keep = y != ignore && y >= 0 && y < V;
  const float w = keep ? dloss[t] / scale[0] : 0.0f, l = lse[t];
  for (int j = threadIdx.x; j < n; j += blockDim.x) {
    float p = expf(z[t * ldz + j] - l);
    if (v0 + j == y) p -= 1.0f;
    reinterpret_cast<__nv_bfloat16*>(G)[t * ldg + j] = __float2bfloat16_rn(keep ? w * p : 0.0f);
  }
}

__global__ void __launch_bounds__(256) k_ce_join(float* acc, const float* part, int64_t n, int first, uint16_t* out) {
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    const float v = first ? part[i] : acc[i] + part[i];
    acc[i] = v;
    if (out) reinterpret_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
  }
}

constexpr int64_t kPiece = 8192;

GemmProblem ce_gemm(int a_mn, int b_mn, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* B,
                    int64_t ldb, int64_t b_cols, int out_f32, void* C, int64_t ldc) {
  GemmProblem g{};
  g.op16 = 1;
  g.a_mn = a_mn;
  g.b_mn = b_mn;
  g.M = (int)M;
  g.N = (int)N;
  g.K = (int)K;
  g.A = static_cast<const uint8_t*>(A);
  g.lda = lda;
  g.B = static_cast<const uint8_t*>(B);
  g.ldb = ldb;
  g.b_cols = b_cols;
  g.epi = kEpiStore;
  g.out_f32 = out_f32;
  g.C = C;
  g.ldc = ldc;
  return g;
}

cudaError_t launched(const Launch& L) {
  if (L.launches) ++*L.launches;
  return cudaGetLastError();
}

struct CeWs {
  float *z, *m, *s, *y, *part, *acc, *scale;
  uint16_t *G, *xz;
};
size_t ce_layout(int64_t T, int64_t d, int64_t V, bool bwd, uint8_t* base, CeWs* w) {
  size_t off = 0;
  auto take = [&](int64_t bytes) {
    uint8_t* p = base + off;
    off += ((size_t)bytes + 255) & ~size_t(255);
    return p;
  };
  const int64_t ld = V < kPiece ? (V + 7) / 8 * 8 : kPiece;
  CeWs t{};
  t.z = (float*)take(T * ld * 4);
  if (bwd) {
    t.G = (uint16_t*)take(T * ld * 2);
    t.xz = (uint16_t*)take(T * d * 2);
    t.part = (float*)take(T * d * 4);
    t.acc = (float*)take(T * d * 4);
    t.scale = (float*)take(8);
  } else {
    t.m = (float*)take(T * 4);
    t.s = (float*)take(T * 4);
    t.y = (float*)take(T * 4);
  }
  if (w) *w = t;
  return off;
}

}  // namespace

size_t ce_workspace_bytes(int64_t T, int64_t d, int64_t V, int bwd) { return ce_layout(T, d, V, bwd != 0, nullptr, nullptr); }

cudaError_t launch_ce_fwd(const uint16_t* x, const uint16_t* W, const int64_t* targets, int64_t T, int d, int64_t V,
                          int64_t ignore, float* loss, float* lse, void* ws, const Launch& L) {
  CeWs w;
  ce_layout(T, d, V, false, static_cast<uint8_t*>(ws), &w);
  const int64_t ld = V < kPiece ? (V + 7) / 8 * 8 : kPiece;
  int P = 0;
  for (int64_t v0 = 0; v0 < V; v0 += kPiece) {
    const int n = (int)(V - v0 < kPiece ? V - v0 : kPiece);
    cudaError_t e = launch_gemm(ce_gemm(0, 0, T, n, d, x, d, W + v0 * d, d, n, 1, w.z, ld), &P, L);
    if (e != cudaSuccess) return e;
    k_ce_piece<<<(unsigned)((T + 7) / 8), 256, 0, L.stream>>>(w.z, ld, T, (int)v0, n, targets, V, ignore, w.m, w.s, w.y,
                                                              loss, lse, v0 + n == V, L.status);
    if ((e = launched(L)) != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_ce_bwd(const uint16_t* x, const uint16_t* W, const int64_t* targets, const float* lse,
                          const float* dloss, int64_t T, int d, int64_t V, int64_t ignore, uint16_t* dX, void* dW,
                          int dw_f32, void* ws, const Launch& L) {
  CeWs w;
  ce_layout(T, d, V, true, static_cast<uint8_t*>(ws), &w);
  const int64_t ld = V < kPiece ? (V + 7) / 8 * 8 : kPiece;
  int P = 0;
  cudaError_t e;
  k_ce_scale<<<1, 1024, 0, L.stream>>>(dloss, targets, T, V, ignore, w.scale, L.status);
  if ((e = launched(L)) != cudaSuccess) return e;
  k_ce_mask_x<<<L.num_sms * 4, 256, 0, L.stream>>>(x, targets, T, d, V, ignore, w.xz);
  if ((e = launched(L)) != cudaSuccess) return e;
  for (int64_t v0 = 0; v0 < V; v0 += kPiece) {
    const int n = (int)(V - v0 < kPiece ? V - v0 : kPiece);
    if ((e = launch_gemm(ce_gemm(0, 0, T, n, d, x, d, W + v0 * d, d, n, 1, w.z, ld), &P, L)) != cudaSuccess) return e;
    k_ce_grad<<<(unsigned)T, 256, 0, L.stream>>>(w.z, ld, T, (int)v0, n, targets, V, ignore, lse, dloss, w.scale, w.G, ld);
    if ((e = launched(L)) != cudaSuccess) return e;
    // dX += s G W[piece]
    GemmProblem gx = ce_gemm(0, 1, T, d, n, w.G, ld, W + v0 * d, d, d, 1, w.part, d);
    gx.sinvA = w.scale;
    gx.sinvB = w.scale + 1;
    if ((e = launch_gemm(gx, &P, L)) != cudaSuccess) return e;
    k_ce_join<<<L.num_sms * 4, 256, 0, L.stream>>>(w.acc, w.part, T * d, v0 == 0, v0 + n == V ? dX : nullptr);
    if ((e = launched(L)) != cudaSuccess) return e;
    // dW[piece] = s G^T x
    void* dst = dw_f32 ? (void*)(static_cast<float*>(dW) + v0 * d) : (void*)(static_cast<uint16_t*>(dW) + v0 * d);
    GemmProblem gw = ce_gemm(1, 1, n, d, T, w.G, ld, w.xz, d, d, dw_f32, dst, d);
    gw.sinvA = w.scale;
    gw.sinvB = w.scale + 1;
    if ((e = launch_gemm(gw, &P, L)) != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace fp8q
