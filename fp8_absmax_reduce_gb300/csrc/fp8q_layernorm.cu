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
  // unit k: elements 2 k and 2 k + 1 of 8, or the element
  __device__ __forceinline__ auto unit(int k) const {
    if constexpr (VEC == 1) return __uint_as_float(w[0]);
    else if constexpr (F32) return make_float2(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]));
    else return make_float2(bf16_lo(w[k]), bf16_hi(w[k]));
  }
  __device__ __forceinline__ static void store(void* p, int64_t i, const float2 (&v)[4]) {
    if constexpr (F32) {
      float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
      q[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
      q[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
    } else {
      st_v4(static_cast<uint16_t*>(p) + i, make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y),
                                                     pack_bf16x2(v[2].x, v[2].y), pack_bf16x2(v[3].x, v[3].y)));
    }
  }
  __device__ __forceinline__ static void store(void* p, int64_t i, const float (&v)[1]) {
    if constexpr (F32) static_cast<float*>(p)[i] = v[0];
    else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v[0]);
  }
};

// A thread's arithmetic is on pairs of columns (packed fp32 instructions) where VEC = 8, else on floats.
template <int VEC>
struct Unit { using T = float2; static constexpr int kCount = 4; };
template <>
struct Unit<1> { using T = float; static constexpr int kCount = 1; };
__device__ __forceinline__ float2 add(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float mul(float a, float b) { return a * b; }
__device__ __forceinline__ float fma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float sum(float2 v) { return v.x + v.y; }
__device__ __forceinline__ float sum(float v) { return v; }
__device__ __forceinline__ void fill(float2& v, float f) { v = make_float2(f, f); }
__device__ __forceinline__ void fill(float& v, float f) { v = f; }
template <int VEC>
__device__ __forceinline__ typename Unit<VEC>::T all(float f) {
  typename Unit<VEC>::T v;
  fill(v, f);
  return v;
}

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
// Resident blocks per SM: 768 threads of 80 registers, or 512 of 128
// for fp32 pieces of 8 (two rows of them: 64 registers a thread at 4 pieces).
constexpr int ln_fwd_per_sm(int F32, int VEC, int W) {
  const int n = (F32 && VEC == 8 ? 512 : 768) / ln_fwd_threads(W);
  return n > 0 ? n : 1;
}

template <int F32, int VEC, int NP, int W>
__global__ void __launch_bounds__(ln_fwd_threads(W), ln_fwd_per_sm(F32, VEC, W))
    k_layernorm_fwd(const void* x, const void* __restrict__ g, const void* __restrict__ b, int64_t T, int d, float eps,
                    void* y, float* __restrict__ mean, float* __restrict__ rstd) {
  using E = typename Unit<VEC>::T;
  constexpr int kUnits = Unit<VEC>::kCount;
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
    // x about the warp's mean, in registers
    E c[NP][kUnits];
    E s = all<VEC>(0.0f);
#pragma unroll
    for (int k = 0; k < NP; ++k)
      if ((k * W + warp) * 32 + lane < pieces)
#pragma unroll
        for (int e = 0; e < kUnits; ++e) {
          c[k][e] = px[k].unit(e);
          s = add(s, c[k][e]);
        }
    const float own_mu = ln_warp_sum(sum(s)) * inv_own;
    float mu = own_mu;
    E q = all<VEC>(0.0f);
#pragma unroll
    for (int k = 0; k < NP; ++k)
      if ((k * W + warp) * 32 + lane < pieces)
#pragma unroll
        for (int e = 0; e < kUnits; ++e) {
          c[k][e] = add(c[k][e], all<VEC>(-own_mu));
          q = fma(c[k][e], c[k][e], q);
        }
    float m2 = ln_warp_sum(sum(q));
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
        E v[kUnits];
#pragma unroll
        for (int e = 0; e < kUnits; ++e) {
          const E f = mul(pg.unit(e), all<VEC>(rs)), h = add(c[k][e], all<VEC>(own_mu - mu));
          v[e] = b ? fma(h, f, pb.unit(e)) : mul(h, f);
        }
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

// Sums of two values over the warp: lanes 0-15 end with a's, lanes 16-31 with b's (5 exchanges for both).
__device__ __forceinline__ float ln_warp_sum2(float a, float b, int lane) {
  float v = (lane < 16 ? a : b) + __shfl_xor_sync(0xFFFFFFFFu, lane < 16 ? b : a, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

template <int F32, int VEC, int NP, int RING>
__global__ void __launch_bounds__(kLnThreads, NP * VEC <= 8 ? 2 : 1)
    k_layernorm_bwd(const void* dY, const void* x, const void* __restrict__ g, const float* __restrict__ mean,
                    const float* __restrict__ rstd, const void* dres, int64_t T, int d, int rows, int S, void* dX,
                    float* __restrict__ part, unsigned* status) {
  static_assert(RING == (VEC == 8), "the ring's pieces are vectors");
  using E = typename Unit<VEC>::T;
  constexpr int kUnits = Unit<VEC>::kCount;
  constexpr int ES = F32 ? 4 : 2;
  constexpr bool kHold = RING || NP <= 8;  // a thread's inputs stay in registers for their second use
  constexpr bool kKeep = RING && NP <= 2;  // and so do u and xh
  extern __shared__ __align__(128) uint8_t ln_rows[];
  __shared__ uint64_t full[kLnSlotsMax];
  __shared__ float red[2][2][16];
  __shared__ volatile int give_up;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, nwarps = blockDim.x >> 5;
  const int pieces = d / VEC;
  const int64_t r0 = (int64_t)blockIdx.x * rows;
  const int nrows = (int)(T - r0 < rows ? T - r0 : rows);
  const uint32_t row_bytes = (uint32_t)d * ES, slot_bytes = row_bytes * (dres ? 3u : 2u);
  auto issue = [&](int rr, int s) {  // thread 0 only
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
      for (int k = 0; k < S && k < nrows; ++k) issue(k, k);
  }
  E ag[NP][kUnits], ab[NP][kUnits];
#pragma unroll
  for (int k = 0; k < NP; ++k)
#pragma unroll
    for (int e = 0; e < kUnits; ++e) ag[k][e] = ab[k][e] = all<VEC>(0.0f);
  Piece<F32, VEC> pg[NP];
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const int i = k * (int)blockDim.x + t;
    if (kHold && i < pieces) pg[k].load(g, (int64_t)i * VEC);
  }
  const float inv_d = 1.0f / (float)d;
  float mu_next = mean[r0], rs_next = rstd[r0];
  bool aborted = false;
  int rr = 0, s = 0;
  uint32_t par = 0;
  for (; rr < nrows; ++rr) {
    const float mu = mu_next, rs = rs_next;
    if (rr + 1 < nrows) { mu_next = mean[r0 + rr + 1]; rs_next = rstd[r0 + rr + 1]; }
    const int64_t base = (r0 + rr) * d;
    const uint8_t* slot = nullptr;
    bool ok = true;
    if (RING) {
      ok = mbar_wait(&full[s], par, &give_up);
      if (!ok) give_up = 1;
      slot = ln_rows + (size_t)s * slot_bytes;
    }
    Piece<F32, VEC> py[NP], px[NP], pr[NP];
    E u[kKeep ? NP : 1][kUnits], xh[kKeep ? NP : 1][kUnits];
    E su_t = all<VEC>(0.0f), sx_t = all<VEC>(0.0f);
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
      for (int e = 0; e < kUnits; ++e) {
        const E dy = py[k].unit(e), uu = mul(dy, pg[k].unit(e));
        const E h = mul(add(px[k].unit(e), all<VEC>(-mu)), all<VEC>(rs));
        su_t = add(su_t, uu);
        sx_t = fma(uu, h, sx_t);
        ag[k][e] = fma(dy, h, ag[k][e]);
        ab[k][e] = add(ab[k][e], dy);
        if (kKeep) { u[kKeep ? k : 0][e] = uu; xh[kKeep ? k : 0][e] = h; }
      }
    }
    const float both = ln_warp_sum2(sum(su_t), sum(sx_t), lane);
    if ((lane & 15) == 0) red[rr & 1][lane >> 4][warp] = both;
    // the row's one barrier; a wait that expired anywhere in the block is seen by all after it
    if (RING) aborted = __syncthreads_or(!ok);
    else __syncthreads();
    if (aborted) break;
    float tot = (lane & 15) < nwarps ? red[rr & 1][lane >> 4][lane & 15] : 0.0f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) tot += __shfl_xor_sync(0xFFFFFFFFu, tot, o);
    const float su = __shfl_sync(0xFFFFFFFFu, tot, 0) * inv_d, sx = __shfl_sync(0xFFFFFFFFu, tot, 16) * inv_d;
    if (RING) {
      // every thread has its values of row rr in registers: the slot takes row rr + S
      if (t == 0 && rr + S < nrows) issue(rr + S, s);
      if (++s == S) { s = 0; par ^= 1u; }
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
      E v[kUnits];
#pragma unroll
      for (int e = 0; e < kUnits; ++e) {
        const E h = kKeep ? xh[kKeep ? k : 0][e] : mul(add(px[k].unit(e), all<VEC>(-mu)), all<VEC>(rs));
        const E uu = kKeep ? u[kKeep ? k : 0][e] : mul(py[k].unit(e), pg[k].unit(e));
        const E w = add(fma(h, all<VEC>(-sx), uu), all<VEC>(-su));
        v[e] = dres ? fma(w, all<VEC>(rs), pr[k].unit(e)) : mul(w, all<VEC>(rs));
      }
      Piece<F32, VEC>::store(dX, base + j, v);
    }
  }
  if (aborted) {
    if (t == 0) {
      atomicOr(status, kStatusTimeout);
      volatile int never = 0;
      // rows rr .. rr + S - 1 may still have copies in flight into this block's ring
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
