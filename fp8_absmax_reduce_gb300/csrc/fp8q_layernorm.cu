// Layer norm, forward and backward (mean and variance over each row, gain and bias).
//
//   mean = (1/d) sum_j x_j,  var = (1/d) sum_j (x_j - mean)^2,  rstd = 1 / sqrt(var + eps),
//   xh = (x - mean) rstd,  y = xh g + b;
//   u = dY g,  dX = rstd (u - mean(u) - xh mean(u xh)) (+ dres),
//   dg_j = sum_t dY_tj xh_tj,  db_j = sum_t dY_tj.
// All sums are fp32 in a fixed order; the variance is summed about a mean, not as
// E[x^2] - mean^2, which would cancel for rows whose mean is large.  Bound by memory: every tensor
// is read or written once.
#include "fp8q_common.cuh"
#include "fp8q_internal.h"

namespace fp8q {

namespace {

// A piece of VEC consecutive elements of a row: 8 of them as one (bf16) or two (fp32) 16-byte vectors
// where a row's bytes are a multiple of 16 (VEC = 8), else single elements (VEC = 1).
template <int F32, int VEC>
struct Piece {
  static constexpr int kWords = VEC == 8 ? (F32 ? 8 : 4) : 1;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    if constexpr (VEC == 8) {
      const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + i * (F32 ? 4 : 2));
#pragma unroll
      for (int k = 0; k < kWords / 4; ++k) {
        const uint4 v = q[k];
        w[4 * k] = v.x; w[4 * k + 1] = v.y; w[4 * k + 2] = v.z; w[4 * k + 3] = v.w;
      }
    } else {
      w[0] = F32 ? static_cast<const uint32_t*>(p)[i] : (uint32_t)static_cast<const uint16_t*>(p)[i] << 16;
    }
  }
  __device__ __forceinline__ float at(int k) const {
    if constexpr (VEC == 8 && !F32) return (k & 1) ? bf16_hi(w[k >> 1]) : bf16_lo(w[k >> 1]);
    else return __uint_as_float(w[k]);
  }
  __device__ static void store(void* p, int64_t i, const float (&v)[VEC]) {
    if constexpr (VEC == 8) {
      if constexpr (F32) {
        float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
        q[0] = make_float4(v[0], v[1], v[2], v[3]);
        q[1] = make_float4(v[4], v[5], v[6], v[7]);
      } else {
        st_v4(static_cast<uint16_t*>(p) + i, make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                       pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
      }
    } else {
      if constexpr (F32) static_cast<float*>(p)[i] = v[0];
      else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v[0]);
    }
  }
};

__device__ __forceinline__ float ln_warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// ---------------------------------------------------------------------------
// Forward: W warps hold a row in registers, NP pieces a lane (piece k of lane l of warp w is piece
// (k W + w) 32 + l of the row); a block of max(W, 8) warps has 8 / W rows at a time and walks the rows with the
// grid's stride, the next row's pieces in flight while the current one is computed and written.  Each
// warp takes the mean and the sum of squares about it of its own elements, in two passes over its registers; the
// warps' (mean, M2) pairs are then joined with the parallel-variance formula
// M2 = M2_a + M2_b + delta^2 n_a n_b / n, so a row costs one block barrier and nothing cancels.
// ---------------------------------------------------------------------------
constexpr int ln_fwd_threads(int W) { return W < 8 ? 256 : 32 * W; }
// Resident blocks per SM: 1024 threads of 64 registers, or 512 of 128 where fp32 pieces fill more.
constexpr int ln_fwd_per_sm(int F32, int VEC, int W) {
  return (F32 && VEC == 8 ? 512 : 1024) / ln_fwd_threads(W) > 0 ? (F32 && VEC == 8 ? 512 : 1024) / ln_fwd_threads(W) : 1;
}

template <int F32, int VEC, int NP, int W>
__global__ void __launch_bounds__(ln_fwd_threads(W), ln_fwd_per_sm(F32, VEC, W))
    k_layernorm_fwd(const void* x, const void* __restrict__ g, const void* __restrict__ b, int64_t T, int d, float eps,
                    void* y, float* __restrict__ mean, float* __restrict__ rstd) {
  constexpr int kRows = W < 8 ? 8 / W : 1;
  __shared__ float sm[2][kRows][W], sv[2][kRows][W];
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % W, r = (threadIdx.x >> 5) / W;
  const int pieces = d / VEC;
  // elements of a warp: full groups of 32 pieces, and what the last one holds
  auto count = [&](int w) {
    int n = 0;
#pragma unroll
    for (int k = 0; k < NP; ++k) n += min(32, max(0, pieces - (k * W + w) * 32));
    return n * VEC;
  };
  const int n_own = count(warp);
  const float inv_own = n_own ? 1.0f / (float)n_own : 0.0f;
  Piece<F32, VEC> px[NP], nx[NP];
  auto load = [&](Piece<F32, VEC>(&p)[NP], int64_t row) {
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int i = (k * W + warp) * 32 + lane;
      if (row < T && i < pieces) p[k].load(x, row * d + (int64_t)i * VEC);
    }
  };
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t row = (int64_t)blockIdx.x * kRows + r;
  load(nx, row);
  int par = 0;
  for (int64_t first = (int64_t)blockIdx.x * kRows; first < T; first += step, row += step, par ^= 1) {
#pragma unroll
    for (int k = 0; k < NP; ++k) px[k] = nx[k];
    load(nx, row + step);
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < NP; ++k)
      if ((k * W + warp) * 32 + lane < pieces)
#pragma unroll
        for (int e = 0; e < VEC; ++e) s += px[k].at(e);
    float mu = ln_warp_sum(s) * inv_own;
    float m2 = 0.0f;
#pragma unroll
    for (int k = 0; k < NP; ++k)
      if ((k * W + warp) * 32 + lane < pieces)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float c = px[k].at(e) - mu;
          m2 += c * c;
        }
    m2 = ln_warp_sum(m2);
    if (W > 1) {
      if (lane == 0) { sm[par][r][warp] = mu; sv[par][r][warp] = m2; }
      __syncthreads();
      float n = (float)count(0);
      mu = sm[par][r][0];
      m2 = sv[par][r][0];
#pragma unroll
      for (int w = 1; w < W; ++w) {
        const float nf = (float)count(w), tot = n + nf, delta = sm[par][r][w] - mu, share = __fdividef(nf, tot);
        mu += delta * share;
        m2 += sv[par][r][w] + delta * delta * n * share;
        n = tot;
      }
    }
    if (row >= T) continue;
    const float rs = 1.0f / sqrtf(m2 / (float)d + eps);
    if (warp == 0 && lane == 0) {
      mean[row] = mu;
      rstd[row] = rs;
    }
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int i = (k * W + warp) * 32 + lane;
      if (i < pieces) {
        Piece<F32, VEC> pg, pb;
        pg.load(g, (int64_t)i * VEC);
        if (b) pb.load(b, (int64_t)i * VEC);
        float v[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = (px[k].at(e) - mu) * rs * pg.at(e) + (b ? pb.at(e) : 0.0f);
        Piece<F32, VEC>::store(y, row * d + (int64_t)i * VEC, v);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Backward: a block owns a run of consecutive rows, a thread the same NP pieces of every row, whose
// shares of dg and db it keeps in registers; k_layernorm_bwd_finish adds the blocks' partial rows.
// A row needs one exchange between its warps, of the two sums in one barrier.
//
// RING (rows of a multiple of 16 bytes): x, dY and dres rows arrive in shared memory through bulk copies
// up to S rows ahead, so the bytes in flight are set by the ring and not by registers.  Every wait is
// bounded; on expiry all threads leave together after the row's barrier and thread 0 waits for the
// copies in flight before the block exits.
// Without RING (odd widths) a thread loads its elements itself, and again for the second use where it
// has more than 8.
// ---------------------------------------------------------------------------
constexpr int kLnSlotsMax = 8;
constexpr int kLnThreads = 512;

template <int F32, int VEC, int NP, int RING>
__global__ void __launch_bounds__(kLnThreads, NP * VEC <= 8 ? 2 : 1)
    k_layernorm_bwd(const void* dY, const void* x, const void* __restrict__ g, const float* __restrict__ mean,
                    const float* __restrict__ rstd, const void* dres, int64_t T, int d, int rows, int S, void* dX,
                    float* __restrict__ part, unsigned* status) {
  constexpr int ES = F32 ? 4 : 2;
  constexpr bool kHold = RING || NP <= 8;
  extern __shared__ __align__(128) uint8_t ln_rows[];
  __shared__ uint64_t full[kLnSlotsMax];
  __shared__ float red[2][2][32];
  __shared__ int bad[2][32];
  __shared__ volatile int give_up;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, nwarps = blockDim.x >> 5;
  const int pieces = d / VEC;
  const int64_t r0 = (int64_t)blockIdx.x * rows;
  const int nrows = (int)(T - r0 < rows ? T - r0 : rows);
  const uint32_t row_bytes = (uint32_t)d * ES, slot_bytes = row_bytes * (dres ? 3u : 2u);
  auto issue = [&](int rr) {  // thread 0 only
    const int s = rr % S;
    uint8_t* slot = ln_rows + (size_t)s * slot_bytes;
    const int64_t off = (r0 + rr) * (int64_t)row_bytes;
    mbar_arrive_expect_tx(&full[s], slot_bytes);
    bulk_load(slot, static_cast<const uint8_t*>(dY) + off, row_bytes, &full[s]);
    bulk_load(slot + row_bytes, static_cast<const uint8_t*>(x) + off, row_bytes, &full[s]);
    if (dres) bulk_load(slot + 2 * row_bytes, static_cast<const uint8_t*>(dres) + off, row_bytes, &full[s]);
  };
  if (RING) {
    if (t == 0) {
      for (int s = 0; s < S; ++s) mbar_init(&full[s], 1);
      give_up = 0;
      fence_mbar_init();
    }
    __syncthreads();
    if (t == 0)
      for (int k = 0; k < S && k < nrows; ++k) issue(k);
  }
  float ag[NP][VEC], ab[NP][VEC];
#pragma unroll
  for (int k = 0; k < NP; ++k)
#pragma unroll
    for (int e = 0; e < VEC; ++e) ag[k][e] = ab[k][e] = 0.0f;
  Piece<F32, VEC> pg[NP];
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const int i = k * (int)blockDim.x + t;
    if (kHold && i < pieces) pg[k].load(g, (int64_t)i * VEC);
  }
  const float inv_d = 1.0f / (float)d;
  float mu_next = mean[r0], rs_next = rstd[r0];
  bool aborted = false;
  int rr = 0;
  for (; rr < nrows; ++rr) {
    const float mu = mu_next, rs = rs_next;
    if (rr + 1 < nrows) { mu_next = mean[r0 + rr + 1]; rs_next = rstd[r0 + rr + 1]; }
    const int64_t base = (r0 + rr) * d;
    const uint8_t* slot = nullptr;
    bool ok = true;
    if (RING) {
      const int s = rr % S;
      ok = mbar_wait(&full[s], (uint32_t)(rr / S) & 1u, &give_up);
      if (!ok) give_up = 1;
      slot = ln_rows + (size_t)s * slot_bytes;
    }
    Piece<F32, VEC> py[NP], px[NP], pr[NP];
    float su = 0.0f, sx = 0.0f;
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int i = k * (int)blockDim.x + t;
      if (i >= pieces) continue;
      const int64_t j = (int64_t)i * VEC;
      if (RING) {
        py[k].load(slot, j);
        px[k].load(slot + row_bytes, j);
        if (dres) pr[k].load(slot + 2 * row_bytes, j);
      } else {
        py[k].load(dY, base + j);
        px[k].load(x, base + j);
        if (kHold && dres) pr[k].load(dres, base + j);
        if (!kHold) pg[k].load(g, j);
      }
    }
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      if (k * (int)blockDim.x + t >= pieces) continue;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float dy = py[k].at(e), xh = (px[k].at(e) - mu) * rs, u = dy * pg[k].at(e);
        su += u;
        sx += u * xh;
        ag[k][e] += dy * xh;
        ab[k][e] += dy;
      }
    }
    su = ln_warp_sum(su);
    sx = ln_warp_sum(sx);
    const int warp_bad = RING ? __any_sync(0xFFFFFFFFu, !ok) : 0;
    if (lane == 0) {
      red[rr & 1][0][warp] = su;
      red[rr & 1][1][warp] = sx;
      if (RING) bad[rr & 1][warp] = warp_bad;
    }
    __syncthreads();
    su = ln_warp_sum(lane < nwarps ? red[rr & 1][0][lane] : 0.0f) * inv_d;
    sx = ln_warp_sum(lane < nwarps ? red[rr & 1][1][lane] : 0.0f) * inv_d;
    if (RING) {
      if (__any_sync(0xFFFFFFFFu, lane < nwarps && bad[rr & 1][lane] != 0)) {
        aborted = true;
        break;
      }
      // every thread has its values of row rr in registers: the slot takes row rr + S
      if (t == 0 && rr + S < nrows) issue(rr + S);
    }
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int i = k * (int)blockDim.x + t;
      if (i >= pieces) continue;
      const int64_t j = (int64_t)i * VEC;
      if (!kHold) {
        py[k].load(dY, base + j);
        px[k].load(x, base + j);
        pg[k].load(g, j);
        if (dres) pr[k].load(dres, base + j);
      }
      float v[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float xh = (px[k].at(e) - mu) * rs;
        v[e] = rs * (py[k].at(e) * pg[k].at(e) - su - xh * sx);
        if (dres) v[e] += pr[k].at(e);
      }
      Piece<F32, VEC>::store(dX, base + j, v);
    }
  }
  if (aborted) {
    if (t == 0) {
      atomicOr(status, kStatusTimeout);
      volatile int never = 0;
      for (int k = rr; k < rr + S && k < nrows; ++k) mbar_wait(&full[k % S], (uint32_t)(k / S) & 1u, &never);
    }
    return;
  }
  float* pgp = part + (int64_t)blockIdx.x * 2 * d;
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const int i = k * (int)blockDim.x + t;
    if (i >= pieces) continue;
    Piece<1, VEC>::store(pgp, (int64_t)i * VEC, ag[k]);
    Piece<1, VEC>::store(pgp + d, (int64_t)i * VEC, ab[k]);
  }
}

// Column sums of the blocks' partial rows part [nblk][2 d]: 32 columns a block, 32 row groups, then a tree.
__global__ void __launch_bounds__(1024) k_layernorm_bwd_finish(const float* __restrict__ part, int nblk, int d,
                                                               float* __restrict__ dg, float* __restrict__ db) {
  __shared__ float sum[32][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int j = blockIdx.x * 32 + tx;
  float s = 0.0f;
  if (j < 2 * d)
#pragma unroll 4
    for (int k = ty; k < nblk; k += 32) s += part[(int64_t)k * 2 * d + j];
  sum[ty][tx] = s;
  __syncthreads();
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) {
    if (ty < w) sum[ty][tx] += sum[ty + w][tx];
    __syncthreads();
  }
  if (ty == 0 && j < 2 * d) {
    if (j < d) dg[j] = sum[0][tx];
    else if (db) db[j - d] = sum[0][tx];
  }
}

cudaError_t launched(const Launch& L) {
  if (L.launches) ++*L.launches;
  return cudaGetLastError();
}

template <int F32, int VEC, int NP, int W>
cudaError_t fwd_go(const void* x, const void* g, const void* b, int64_t T, int d, float eps, void* y, float* mean,
                   float* rstd, const Launch& L) {
  constexpr int rows = W < 8 ? 8 / W : 1;
  const int64_t need = (T + rows - 1) / rows, wave = (int64_t)L.num_sms * ln_fwd_per_sm(F32, VEC, W);
  k_layernorm_fwd<F32, VEC, NP, W><<<(unsigned)(need < wave ? need : wave), ln_fwd_threads(W), 0, L.stream>>>(
      x, g, b, T, d, eps, y, mean, rstd);
  return launched(L);
}

// The fewest warps (a power of two) whose lanes hold the row: up to 4 pieces of 8 columns or 16 single
// columns a lane.  More than one warp is taken only past half of what it holds, so a lane then has 3 or 4
// pieces of 8 (up to 16 single columns).
template <int F32>
cudaError_t fwd_t(const void* x, const void* g, const void* b, int64_t T, int d, float eps, void* y, float* mean,
                  float* rstd, const Launch& L) {
#define FP8Q_LN_FWD(VEC, NP, W) return fwd_go<F32, VEC, NP, W>(x, g, b, T, d, eps, y, mean, rstd, L)
  if (d % 8 == 0) {
    if (d <= 256) FP8Q_LN_FWD(8, 1, 1);
    if (d <= 512) FP8Q_LN_FWD(8, 2, 1);
    if (d <= 768) FP8Q_LN_FWD(8, 3, 1);
    if (d <= 1024) FP8Q_LN_FWD(8, 4, 1);
    if (d <= 1536) FP8Q_LN_FWD(8, 3, 2);
    if (d <= 2048) FP8Q_LN_FWD(8, 4, 2);
    if (d <= 4096 - 1024) FP8Q_LN_FWD(8, 3, 4);
    if (d <= 4096) FP8Q_LN_FWD(8, 4, 4);
    if (d <= 6144) FP8Q_LN_FWD(8, 3, 8);
    if (d <= 8192) FP8Q_LN_FWD(8, 4, 8);
    if (d <= 12288) FP8Q_LN_FWD(8, 3, 16);
    FP8Q_LN_FWD(8, 4, 16);
  }
  if (d <= 128) FP8Q_LN_FWD(1, 4, 1);
  if (d <= 512) FP8Q_LN_FWD(1, 16, 1);
  if (d <= 1024) FP8Q_LN_FWD(1, 16, 2);
  if (d <= 2048) FP8Q_LN_FWD(1, 16, 4);
  if (d <= 4096) FP8Q_LN_FWD(1, 16, 8);
  if (d <= 8192) FP8Q_LN_FWD(1, 16, 16);
  FP8Q_LN_FWD(1, 16, 32);
#undef FP8Q_LN_FWD
}

// The backward's launch shape.  d is a multiple of 8: a thread has 1, 2 or 4 pieces of 8 columns (d up to
// 4096, 8192, 16384); otherwise 4, 8, 16 or 32 single columns.
struct BwdShape {
  int np, threads, per_sm, S;
};
constexpr size_t kLnSmemBudget = 200 * 1024;  // per SM
BwdShape bwd_shape(int d, int f32, bool dres) {
  BwdShape s{};
  const bool ring = d % 8 == 0;
  const int pieces = ring ? d / 8 : d;
  s.np = ring ? 1 : 4;
  while (pieces > kLnThreads * s.np) s.np *= 2;
  s.threads = ((pieces + s.np - 1) / s.np + 31) / 32 * 32;
  if (s.threads < 64 && !ring) s.threads = 64;
  s.per_sm = s.np * (ring ? 8 : 1) <= 8 ? 2 : 1;
  if (ring) {
    const size_t slot = (size_t)d * (f32 ? 4 : 2) * (dres ? 3 : 2);
    if (2 * 3 * slot > kLnSmemBudget) s.per_sm = 1;
    s.S = (int)(kLnSmemBudget / s.per_sm / slot);
    if (s.S > kLnSlotsMax) s.S = kLnSlotsMax;
  }
  return s;
}

template <int F32, int VEC, int NP, int RING>
cudaError_t bwd_go(const BwdShape& s, const void* dY, const void* x, const void* g, const float* mean, const float* rstd,
                   const void* dres, int64_t T, int d, void* dX, float* part, int nblk, int rows, const Launch& L) {
  auto* k = k_layernorm_bwd<F32, VEC, NP, RING>;
  size_t smem = 0;
  if (RING) {
    smem = (size_t)s.S * d * (F32 ? 4 : 2) * (dres ? 3 : 2);
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kLnSmemBudget);
    if (e != cudaSuccess) return e;
  }
  k<<<nblk, s.threads, smem, L.stream>>>(dY, x, g, mean, rstd, dres, T, d, rows, s.S, dX, part, L.status);
  return launched(L);
}

template <int F32>
cudaError_t bwd_t(const BwdShape& s, const void* dY, const void* x, const void* g, const float* mean, const float* rstd,
                  const void* dres, int64_t T, int d, void* dX, float* part, int nblk, int rows, const Launch& L) {
  if (d % 8 == 0) {
    if (s.np == 1) return bwd_go<F32, 8, 1, 1>(s, dY, x, g, mean, rstd, dres, T, d, dX, part, nblk, rows, L);
    if (s.np == 2) return bwd_go<F32, 8, 2, 1>(s, dY, x, g, mean, rstd, dres, T, d, dX, part, nblk, rows, L);
    return bwd_go<F32, 8, 4, 1>(s, dY, x, g, mean, rstd, dres, T, d, dX, part, nblk, rows, L);
  }
  if (s.np == 4) return bwd_go<F32, 1, 4, 0>(s, dY, x, g, mean, rstd, dres, T, d, dX, part, nblk, rows, L);
  if (s.np == 8) return bwd_go<F32, 1, 8, 0>(s, dY, x, g, mean, rstd, dres, T, d, dX, part, nblk, rows, L);
  if (s.np == 16) return bwd_go<F32, 1, 16, 0>(s, dY, x, g, mean, rstd, dres, T, d, dX, part, nblk, rows, L);
  return bwd_go<F32, 1, 32, 0>(s, dY, x, g, mean, rstd, dres, T, d, dX, part, nblk, rows, L);
}

}  // namespace

cudaError_t launch_layernorm_fwd(const void* x, int f32, const void* g, const void* b, int64_t T, int d, float eps,
                                 void* y, float* mean, float* rstd, const Launch& L) {
  return f32 ? fwd_t<1>(x, g, b, T, d, eps, y, mean, rstd, L) : fwd_t<0>(x, g, b, T, d, eps, y, mean, rstd, L);
}

// One wave of resident blocks, each with a run of consecutive rows.  The workspace holds kLnMaxBlocks
// partial rows (or T, where that is less): no more blocks than that run.
cudaError_t launch_layernorm_bwd(const void* dY, const void* x, int f32, const void* g, const float* mean,
                                 const float* rstd, const void* dres, int64_t T, int d, void* dX, float* dg, float* db,
                                 float* part, const Launch& L) {
  const BwdShape s = bwd_shape(d, f32, dres != nullptr);
  int64_t most = (int64_t)L.num_sms * s.per_sm;
  if (most > kLnMaxBlocks) most = kLnMaxBlocks;
  const int rows = (int)((T + most - 1) / most);
  const int nblk = (int)((T + rows - 1) / rows);
  cudaError_t e = f32 ? bwd_t<1>(s, dY, x, g, mean, rstd, dres, T, d, dX, part, nblk, rows, L)
                      : bwd_t<0>(s, dY, x, g, mean, rstd, dres, T, d, dX, part, nblk, rows, L);
  if (e != cudaSuccess) return e;
  k_layernorm_bwd_finish<<<(2 * d + 31) / 32, 1024, 0, L.stream>>>(part, nblk, d, dg, db);
  return launched(L);
}

}  // namespace fp8q
