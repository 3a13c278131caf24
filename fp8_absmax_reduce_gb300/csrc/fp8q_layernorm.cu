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
#include "fp8q_head.cuh"
#include "fp8q_internal.h"

#include <atomic>

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
__device__ __forceinline__ float first_of(float2 v) { return v.x; }
__device__ __forceinline__ float first_of(float v) { return v; }
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

// Sums of two values over the warp: lanes 0-15 end with a's, lanes 16-31 with b's (5 exchanges for both).
__device__ __forceinline__ float ln_warp_sum2(float a, float b, int lane) {
  float v = (lane < 16 ? a : b) + __shfl_xor_sync(0xFFFFFFFFu, lane < 16 ? b : a, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// ---------------------------------------------------------------------------
// Rows on their way in: bulk copies into a ring of slots in shared memory, completing on a slot's
// mbarrier, so that the bytes in flight are set by the ring and not by registers.
//
// A bulk copy moves whole 16-byte units.  Where a row's bytes are no multiple of 16 (odd widths), the copy starts at
// the unit that holds the first byte and the data lie `off & 15` bytes into their region; the last unit is
// copied whole too, unless it would pass the tensor's end, whose last elements thread 0 then copies itself.
// ---------------------------------------------------------------------------
constexpr int kLnSlotsMax = 8;
constexpr size_t kLnSmemBudget = 200 * 1024;  // per SM

__host__ __device__ inline uint32_t ln_region(uint32_t bytes) {
  return bytes % 16 == 0 ? bytes : (bytes + 15) / 16 * 16 + 16;
}
// The bytes of a copy of [off, off + bytes) of a tensor of `total` bytes.  EVEN: all are multiples of 16.
template <bool EVEN>
__device__ __forceinline__ uint32_t ln_copy_bytes(int64_t off, uint32_t bytes, int64_t total) {
  if (EVEN) return bytes;
  const int64_t begin = off & ~(int64_t)15, end = min((off + bytes + 15) & ~(int64_t)15, total & ~(int64_t)15);
  return end > begin ? (uint32_t)(end - begin) : 0u;
}
template <bool EVEN>
__device__ __forceinline__ void ln_copy(uint8_t* dst, const void* src, int64_t off, uint32_t bytes, uint32_t n,
                                        uint64_t* bar) {
  if (EVEN) {
    bulk_load(dst, static_cast<const uint8_t*>(src) + off, n, bar);
    return;
  }
  const uint8_t* from = static_cast<const uint8_t*>(src) + (off & ~(int64_t)15);
  if (n) bulk_load(dst, from, n, bar);
  const uint32_t mis = (uint32_t)(off & 15);
  for (uint32_t k = n; k < mis + bytes; k += 2)
    if (k >= mis) *reinterpret_cast<uint16_t*>(dst + k) = *reinterpret_cast<const uint16_t*>(from + k);
}

// ---------------------------------------------------------------------------
// Forward: W warps hold RT rows at once in registers, NP pieces of each row a lane (piece k of lane l of warp w
// is piece (k W + w) 32 + l); a block of 8 warps (W where that is no divisor of 8) takes kRows consecutive rows at a time (one slot of the
// ring, one copy) and walks them with the grid's stride.  Each warp takes the mean and the sum of
// squares about it of its own elements, in two passes over its registers; the warps' (mean, M2) pairs are then joined about
// the first one's mean m_0, mean = m_0 + sum n_w (m_w - m_0) / d and M2 = sum (M2_w + n_w (m_w - mean)^2), so a row costs one
// block barrier and nothing cancels.  A row of equal values has to end with M2 = 0, whatever the value: a mean one step off
// would make a variance of (2^-24 x)^2, which passes eps from |x| = 5e4 on.  So where a warp's first element is as near to its
// mean as the mean's own roundings (kNear), it is the centre.  In bf16 sums of equal values are exact (8 + 14 bits) and the
// division's two roundings are left; other rows come that near only by a mean that is the element, or beside elements half as
// large as the mean or more away from it (bf16 steps are 2^-8), whose deviation is 2^13 times the difference or more.  In
// fp32 the sum has up to 32 roundings and other rows' elements are as near, so the second pass also adds up x - centre, which
// corrects the mean and M2.  (T = 16384, d = 5120 61.4 -> 62.6 us cold, d = 2560 32.8 -> 34.4; fp32 8192 x 4096 equal.)
// bf16 rows go two at a time (RT = 2): what bounds them is instructions, and the
// second row shares the unpacking of gain and bias and the exchanges (T = 16384, d = 5120: 66 -> 60 us).
// ---------------------------------------------------------------------------
constexpr int ln_fwd_threads(int W) { return 8 % W == 0 ? 256 : 32 * W; }
// Resident blocks per SM by registers: 512 threads of 128 for pieces of 8, 768 of 80 for single columns.  They hold a
// thread's gain and bias too: read again for each row, those come from L2 (the ring leaves L1 too little).
constexpr int ln_fwd_per_sm(int VEC, int W) {
  const int n = (VEC == 8 ? (W == 10 ? 640 : 512) : 768) / ln_fwd_threads(W);
  return n > 0 ? n : 1;
}

// Sums of RT values over the warp, valid in every lane.
template <int RT>
__device__ __forceinline__ void ln_warp_sums(float (&v)[RT], int lane) {
  if constexpr (RT == 1) {
    v[0] = ln_warp_sum(v[0]);
  } else {
    const float t = ln_warp_sum2(v[0], v[1], lane);
    v[0] = __shfl_sync(0xFFFFFFFFu, t, 0);
    v[1] = __shfl_sync(0xFFFFFFFFu, t, 16);
  }
}

template <int F32, int VEC, int NP, int W, int RT>
__global__ void __launch_bounds__(ln_fwd_threads(W), ln_fwd_per_sm(VEC, W))
    k_layernorm_fwd(const void* x, const void* __restrict__ g, const void* __restrict__ b, int64_t T, int d, float eps,
                    int S, void* y, float* __restrict__ mean, float* __restrict__ rstd, unsigned* status) {
  using E = typename Unit<VEC>::T;
  constexpr int kUnits = Unit<VEC>::kCount, ES = F32 ? 4 : 2;
  constexpr int kRows = 8 % W == 0 ? RT * (8 / W) : RT;
  constexpr float kNear = F32 ? 0x1p-19f : 0x1p-22f;
  static_assert(RT == 1 || W <= 16, "two rows join in the warp's halves");
  constexpr int kJoin = W <= 1 ? 1 : W <= 2 ? 2 : W <= 4 ? 4 : W <= 8 ? 8 : W <= 16 ? 16 : 32;  // lanes that join W pairs
  extern __shared__ __align__(128) uint8_t ln_rows[];
  __shared__ uint64_t full[kLnSlotsMax];
  __shared__ float2 pairs[2][kRows][W];
  __shared__ volatile int give_up;
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % W, r = (threadIdx.x >> 5) / W * RT;  // r: its first row
  const int pieces = d / VEC;
  const uint32_t row_bytes = (uint32_t)d * ES, slot_bytes = ln_region(kRows * row_bytes);
  const int64_t total = T * (int64_t)row_bytes, groups = (T + kRows - 1) / kRows;
  auto issue = [&](int64_t group, int s) {  // thread 0 only
    const int64_t first = group * kRows, off = first * row_bytes;
    const uint32_t bytes = (uint32_t)min((int64_t)kRows, T - first) * row_bytes, n = ln_copy_bytes<VEC == 8>(off, bytes, total);
    uint8_t* slot = ln_rows + (size_t)s * slot_bytes;
    ln_copy<VEC == 8>(slot, x, off, bytes, n, &full[s]);
    mbar_arrive_expect_tx(&full[s], n);
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) mbar_init(&full[s], 1);
    give_up = 0;
    fence_mbar_init();
    for (int s = 0; s < S && blockIdx.x + s * (int64_t)gridDim.x < groups; ++s) issue(blockIdx.x + s * (int64_t)gridDim.x, s);
  }
  __syncthreads();
  // elements of a warp: full groups of 32 pieces, and what the last one holds
  auto count = [&](int w) {
    int n = 0;
#pragma unroll
    for (int k = 0; k < NP; ++k) n += min(32, max(0, pieces - (k * W + w) * 32));
    return n * VEC;
  };
  const float inv_own = 1.0f / (float)count(warp), inv_d = 1.0f / (float)d;  // every warp has a piece
  const int of_warp = lane & (kJoin - 1);
  const float lane_count = of_warp < W ? (float)count(of_warp) : 0.0f, lane_share = lane_count * inv_d;
  Piece<F32, VEC> pg[NP], pb[NP];
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const int i = (k * W + warp) * 32 + lane;
    if (i < pieces) {
      pg[k].load(g, (int64_t)i * VEC);
      if (b) pb[k].load(b, (int64_t)i * VEC);
    }
  }
  int s = 0, turn = 0;
  uint32_t par = 0;
  bool aborted = false;
  int64_t group = blockIdx.x;
  for (; group < groups; group += gridDim.x, turn ^= 1) {
    const int64_t row = group * kRows + r;
    const bool ok = mbar_wait(&full[s], par, &give_up);
    if (!ok) give_up = 1;
    // x about the warp's mean, in registers.  A row past the end (or given up) holds what the slot held: it is not written
    E c[RT][NP][kUnits];
    float own_mu[RT], mu[RT], m2[RT];
    const uint8_t* slot = ln_rows + (size_t)s * slot_bytes + (VEC == 8 ? 0 : (int)((group * kRows * row_bytes) & 15));
#pragma unroll
    for (int q = 0; q < RT; ++q) {
      E sum_t = all<VEC>(0.0f);
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        const int i = (k * W + warp) * 32 + lane;
        if (i < pieces) {
          Piece<F32, VEC> px;
          px.load(slot, (r + q) * d + i * VEC);
#pragma unroll
          for (int e = 0; e < kUnits; ++e) {
            c[q][k][e] = px.unit(e);
            sum_t = add(sum_t, c[q][k][e]);
          }
        }
      }
      own_mu[q] = sum(sum_t);
    }
    ln_warp_sums<RT>(own_mu, lane);
#pragma unroll
    for (int q = 0; q < RT; ++q) {
      const float x0 = __shfl_sync(0xFFFFFFFFu, first_of(c[q][0][0]), 0);
      own_mu[q] *= inv_own;
      if (fabsf(x0 - own_mu[q]) < kNear * fabsf(own_mu[q])) own_mu[q] = x0;
      mu[q] = own_mu[q];
      E sq = all<VEC>(0.0f), off = all<VEC>(0.0f);
#pragma unroll
      for (int k = 0; k < NP; ++k)
        if ((k * W + warp) * 32 + lane < pieces)
#pragma unroll
          for (int e = 0; e < kUnits; ++e) {
            c[q][k][e] = add(c[q][k][e], all<VEC>(-own_mu[q]));
            sq = fma(c[q][k][e], c[q][k][e], sq);
            if (F32) off = add(off, c[q][k][e]);
          }
      m2[q] = sum(sq);
      if (F32) {
        const float both = ln_warp_sum2(m2[q], sum(off), lane);
        const float s1 = __shfl_sync(0xFFFFFFFFu, both, 16), more = s1 * inv_own;
        mu[q] += more;
        m2[q] = fmaf(-s1, more, __shfl_sync(0xFFFFFFFFu, both, 0));
        if (m2[q] < 0.0f) m2[q] = 0.0f;  // (a NaN stays)
      }
    }
    if (!F32) ln_warp_sums<RT>(m2, lane);
    if (W > 1 && lane == 0)
#pragma unroll
      for (int q = 0; q < RT; ++q) pairs[turn][r + q][warp] = make_float2(mu[q], m2[q]);
    // the one barrier: the pairs are there, and every thread has its part of the slot, which takes the group S
    // turns ahead; a wait that expired anywhere in the block is seen by all
    aborted = __syncthreads_or(!ok);
    if (aborted) break;
    if (threadIdx.x == 0 && group + S * (int64_t)gridDim.x < groups) issue(group + S * (int64_t)gridDim.x, s);
    if (++s == S) { s = 0; par ^= 1u; }
    if (W > 1) {
      // lanes 0-15 join the first row's pairs, 16-31 the second's
      float2 of = make_float2(0.0f, 0.0f);
      const auto& row_pairs = pairs[turn][r + (RT == 2 ? lane >> 4 : 0)];
      const float m0 = row_pairs[0].x;
      if (of_warp < W) of = row_pairs[of_warp];
      of.x = of_warp < W ? of.x - m0 : 0.0f;
      float m = of.x * lane_share;
#pragma unroll
      for (int o = kJoin / 2; o > 0; o >>= 1) m += __shfl_xor_sync(0xFFFFFFFFu, m, o);
      const float off = of_warp < W ? of.x - m : 0.0f;  // (lanes past W count for nothing, even where m m overflows)
      float v = fmaf(off * off, lane_count, of.y);
#pragma unroll
      for (int o = kJoin / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
      m += m0;
#pragma unroll
      for (int q = 0; q < RT; ++q) {
        mu[q] = RT == 1 ? m : __shfl_sync(0xFFFFFFFFu, m, 16 * q);
        m2[q] = RT == 1 ? v : __shfl_sync(0xFFFFFFFFu, v, 16 * q);
      }
    }
    float rs[RT], shift[RT];
#pragma unroll
    for (int q = 0; q < RT; ++q) {
      rs[q] = rsqrtf(fmaf(m2[q], inv_d, eps));
      shift[q] = own_mu[q] - mu[q];
      if (warp == 0 && lane == 0 && row + q < T) {
        mean[row + q] = mu[q];
        rstd[row + q] = rs[q];
      }
    }
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int i = (k * W + warp) * 32 + lane;
      if (i < pieces) {
        E gu[kUnits], bu[kUnits];
#pragma unroll
        for (int e = 0; e < kUnits; ++e) {
          gu[e] = pg[k].unit(e);
          bu[e] = b ? pb[k].unit(e) : all<VEC>(0.0f);
        }
#pragma unroll
        for (int q = 0; q < RT; ++q) {
          E v[kUnits];
#pragma unroll
          for (int e = 0; e < kUnits; ++e) v[e] = fma(add(c[q][k][e], all<VEC>(shift[q])), mul(gu[e], all<VEC>(rs[q])), bu[e]);
          if (row + q < T) Piece<F32, VEC>::store(y, (row + q) * d + (int64_t)i * VEC, v);
        }
      }
    }
  }
  if (aborted && threadIdx.x == 0) {
    atomicOr(status, kStatusTimeout);
    volatile int never = 0;
    // the copies still in flight: this turn's and those of the next S - 1 turns
    for (int k = 0; k < S && group + k * (int64_t)gridDim.x < groups; ++k) {
      mbar_wait(&full[s], par, &never);
      if (++s == S) { s = 0; par ^= 1u; }
    }
  }
}

// ---------------------------------------------------------------------------
// Backward of the other rows (odd widths, wider ones): a block owns a run of consecutive rows, a thread the same NP pieces
// of every row, whose shares of dg and db it keeps in registers; k_layernorm_bwd_finish adds the blocks' partial rows.
// A row needs one exchange between its warps, of the two sums in one barrier.
//
// dY, x and dres rows come through the ring, up to S rows ahead.  Every wait is bounded; on expiry all
// threads leave together after the row's barrier and thread 0 waits for the copies in flight before the block exits.
// ---------------------------------------------------------------------------
constexpr int kLnThreads = 512, kLnWide = 1024;
// The threads of a block at most.
constexpr int ln_bwd_most(int np, int stride) { return stride ? stride : np == 1 ? kLnWide : kLnThreads; }

template <int F32, int VEC, int NP, int STRIDE>
__global__ void __launch_bounds__(ln_bwd_most(NP, STRIDE), (NP * VEC <= 8 ? kLnWide : kLnThreads) / ln_bwd_most(NP, STRIDE))
    k_layernorm_bwd(const void* dY, const void* x, const void* __restrict__ g, const float* __restrict__ mean,
                    const float* __restrict__ rstd, const void* dres, int64_t T, int d, int rows, int S, void* dX,
                    float* __restrict__ part, unsigned* status) {
  using E = typename Unit<VEC>::T;
  constexpr int kUnits = Unit<VEC>::kCount;
  constexpr int ES = F32 ? 4 : 2;
  constexpr bool kKeep = NP * VEC <= 16;  // u and xh stay in registers for their second use, else the inputs
  extern __shared__ __align__(128) uint8_t ln_rows[];
  __shared__ uint64_t full[kLnSlotsMax];
  __shared__ float red[2][2][32];
  __shared__ volatile int give_up;
  start_dependents();
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, nwarps = blockDim.x >> 5;
  const int pieces = d / VEC;
  const int stride = STRIDE ? STRIDE : (int)blockDim.x;  // a constant lets single columns use immediate offsets
  const int64_t r0 = (int64_t)blockIdx.x * rows;
  const int nrows = (int)(T - r0 < rows ? T - r0 : rows);
  const uint32_t row_bytes = (uint32_t)d * ES, region = ln_region(row_bytes), slot_bytes = region * (dres ? 3u : 2u);
  const int64_t total = T * (int64_t)row_bytes;
  auto issue = [&](int rr, int s) {  // thread 0 only
    uint8_t* slot = ln_rows + (size_t)s * slot_bytes;
    const int64_t off = (r0 + rr) * (int64_t)row_bytes;
    const uint32_t n = ln_copy_bytes<VEC == 8>(off, row_bytes, total);
    ln_copy<VEC == 8>(slot, dY, off, row_bytes, n, &full[s]);
    ln_copy<VEC == 8>(slot + region, x, off, row_bytes, n, &full[s]);
    if (dres) ln_copy<VEC == 8>(slot + 2 * region, dres, off, row_bytes, n, &full[s]);
    mbar_arrive_expect_tx(&full[s], n * (dres ? 3u : 2u));
  };
  if (t == 0) {
    for (int s = 0; s < S; ++s) mbar_init(&full[s], 1);
    give_up = 0;
    fence_mbar_init();
    for (int k = 0; k < S && k < nrows; ++k) issue(k, k);
  }
  __syncthreads();
  E ag[NP][kUnits], ab[NP][kUnits];
#pragma unroll
  for (int k = 0; k < NP; ++k)
#pragma unroll
    for (int e = 0; e < kUnits; ++e) ag[k][e] = ab[k][e] = all<VEC>(0.0f);
  Piece<F32, VEC> pg[NP];
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const int i = k * stride + t;
    if (i < pieces) pg[k].load(g, (int64_t)i * VEC);
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
    const bool ok = mbar_wait(&full[s], par, &give_up);
    if (!ok) give_up = 1;
    const uint8_t* slot = ln_rows + (size_t)s * slot_bytes + (VEC == 8 ? 0 : (int)((base * ES) & 15));
    Piece<F32, VEC> py[NP], px[NP], pr[NP];
    E u[kKeep ? NP : 1][kUnits], xh[kKeep ? NP : 1][kUnits];
    E su_t = all<VEC>(0.0f), sx_t = all<VEC>(0.0f);
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int i = k * stride + t;
      if (i >= pieces) continue;
      const int j = i * VEC;
      py[k].load(slot, j);
      px[k].load(slot + region, j);
      if (dres) pr[k].load(slot + 2 * region, j);
    }
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      if (k * stride + t >= pieces) continue;
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
    aborted = __syncthreads_or(!ok);
    if (aborted) break;
    float tot = (lane & 15) < nwarps ? red[rr & 1][lane >> 4][lane & 15] : 0.0f;
    if ((lane & 15) + 16 < nwarps) tot += red[rr & 1][lane >> 4][(lane & 15) + 16];
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) tot += __shfl_xor_sync(0xFFFFFFFFu, tot, o);
    const float su = __shfl_sync(0xFFFFFFFFu, tot, 0) * inv_d, sx = __shfl_sync(0xFFFFFFFFu, tot, 16) * inv_d;
    // every thread has its values of row rr in registers: the slot takes row rr + S
    if (t == 0 && rr + S < nrows) issue(rr + S, s);
    if (++s == S) { s = 0; par ^= 1u; }
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int i = k * stride + t;
      if (i >= pieces) continue;
      const int64_t j = (int64_t)i * VEC;
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
    const int i = k * stride + t;
    if (i >= pieces) continue;
    Piece<1, VEC>::store(pgp, (int64_t)i * VEC, ag[k]);
    Piece<1, VEC>::store(pgp + d, (int64_t)i * VEC, ab[k]);
  }
}

// Backward of rows of whole 16-byte vectors, up to 8192 bf16 or 4096 fp32 columns: W warps own a run of consecutive rows, a
// lane NP vectors of each (vector k of lane l of warp w is vector (k W + w) 32 + l).  A lane copies its own vectors of the
// next D - 1 rows into its own part of shared memory meanwhile, so a row waits for no one's copies but its own, and only the
// two sums cross the W warps (one barrier among them).  An SM's 16 warps hold 16 / W rows at once; their shares of
// dg and db are added in shared memory at the end, so that the second launch reads one row an SM (four for the narrowest).
// Against one block a row with a ring of bulk copies (as below), with dres: bf16 T = 8192, d = 3584: 48 -> 45 us; d = 5120:
// 72 -> 62; T = 16384, d = 1024: 36 -> 29; T = 65536, d = 256: 45 -> 32; fp32 T = 16384, d = 512: 38 -> 28; T = 4096,
// d = 4096: 56 -> 49; T = 1000, d = 1024: 13 -> 7.  Bound by memory: 0.84 of the measured copy rate at 8192 x 5120.
template <int NP, int W>
struct RunPlan {
  static constexpr int kPerSm = NP == 1 ? 4 : 1;
  static constexpr int kWarps = NP == 1 ? 8 : 16 / W * W;
  static constexpr int kDepth = 4;
  static constexpr int kBytes = kWarps * kDepth * 3 * NP * 512;
};
// One vector of 16 bytes: 8 bf16 or 4 fp32 columns, taken in pairs.
template <int F32>
struct Vec16 {
  static constexpr int kUnits = F32 ? 2 : 4, kCols = 2 * kUnits;
  uint4 w;
  __device__ __forceinline__ void load(const void* p) { w = *static_cast<const uint4*>(p); }
  __device__ __forceinline__ float2 unit(int e) const {
    if constexpr (F32) return e == 0 ? make_float2(__uint_as_float(w.x), __uint_as_float(w.y)) : make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
    const uint32_t v = e == 0 ? w.x : e == 1 ? w.y : e == 2 ? w.z : w.w;
    return make_float2(bf16_lo(v), bf16_hi(v));
  }
  __device__ __forceinline__ static void store(void* p, const float2 (&v)[kUnits]) {
    if constexpr (F32) *static_cast<float4*>(p) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    else st_v4(static_cast<uint16_t*>(p), make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y),
                                                    pack_bf16x2(v[2].x, v[2].y), pack_bf16x2(v[3].x, v[3].y)));
  }
};

template <int F32, int NP, int W>
__global__ void __launch_bounds__(32 * RunPlan<NP, W>::kWarps, RunPlan<NP, W>::kPerSm)
    k_layernorm_bwd_runs(const uint8_t* dY, const uint8_t* x, const uint8_t* __restrict__ g, const float* __restrict__ mean,
                         const float* __restrict__ rstd, const uint8_t* dres, int64_t T, int d, int run, uint8_t* dX,
                         float* __restrict__ part) {
  using P = Vec16<F32>;
  constexpr int kWarps = RunPlan<NP, W>::kWarps, D = RunPlan<NP, W>::kDepth, kUnits = P::kUnits;
  extern __shared__ __align__(128) uint8_t ln_rows[];  // [warps][D][3][NP][32] pieces
  __shared__ float red[2][kWarps][2];
  start_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, pieces = d / P::kCols;
  const int group = warp / W, first = warp % W * 32 + lane;
  uint8_t* own = ln_rows + (warp * D * 3 * NP * 32 + lane) * 16;
  float2 ag[NP][kUnits], ab[NP][kUnits];
  P pg[NP];
#pragma unroll
  for (int k = 0; k < NP; ++k) {
#pragma unroll
    for (int e = 0; e < kUnits; ++e) ag[k][e] = ab[k][e] = all<8>(0.0f);
    if (32 * W * k + first < pieces) pg[k].load(g + 16 * (32 * W * k + first));
  }
  const int64_t r0 = ((int64_t)blockIdx.x * (kWarps / W) + group) * run, row_bytes = (int64_t)pieces * 16;
  const int n = (int)(T - r0 < run ? (T > r0 ? T - r0 : 0) : run);
  auto fetch = [&](int i, int slot) {
    if (i < n) {
#pragma unroll
      for (int w = 0; w < 3; ++w) {
        const uint8_t* src = w == 0 ? dY : w == 1 ? x : dres;
        if (!src) continue;
#pragma unroll
        for (int k = 0; k < NP; ++k)
          if (32 * W * k + first < pieces)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(own + ((slot * 3 + w) * NP + k) * 512)),
                         "l"(src + (r0 + i) * row_bytes + 16 * (32 * W * k + first))
                         : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto take = [&](int slot, int w, int k) {
    P v;
    v.load(own + ((slot * 3 + w) * NP + k) * 512);
    return v;
  };
  const float inv_d = 1.0f / (float)d;
#pragma unroll
  for (int i = 0; i < D - 1; ++i) fetch(i, i);
  float mus = 0.0f, rss = 0.0f;  // lane l's: of row l of the 32 at hand
  int slot = 0;
  for (int i = 0; i < n; ++i) {
    if ((i & 31) == 0 && i + lane < n) { mus = mean[r0 + i + lane]; rss = rstd[r0 + i + lane]; }
    const float mu = __shfl_sync(0xFFFFFFFFu, mus, i & 31), rs = __shfl_sync(0xFFFFFFFFu, rss, i & 31);
    fetch(i + D - 1, slot == 0 ? D - 1 : slot - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(D - 1) : "memory");
    P py[NP], px[NP];
    float2 su_t = all<8>(0.0f), sx_t = all<8>(0.0f);
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      if (32 * W * k + first >= pieces) continue;
      py[k] = take(slot, 0, k);
      px[k] = take(slot, 1, k);
#pragma unroll
      for (int e = 0; e < kUnits; ++e) {
        const float2 dy = py[k].unit(e), u = mul(dy, pg[k].unit(e));
        const float2 h = mul(add(px[k].unit(e), all<8>(-mu)), all<8>(rs));
        su_t = add(su_t, u);
        sx_t = fma(u, h, sx_t);
        ag[k][e] = fma(dy, h, ag[k][e]);
        ab[k][e] = add(ab[k][e], dy);
      }
    }
    const float both = ln_warp_sum2(sum(su_t), sum(sx_t), lane) * inv_d;
    float su, sx;
    if (W == 1) {
      su = __shfl_sync(0xFFFFFFFFu, both, 0);
      sx = __shfl_sync(0xFFFFFFFFu, both, 16);
    } else {  // the next row's pairs take the other buffer, so one barrier a row is enough
      if ((lane & 15) == 0) red[i & 1][warp][lane >> 4] = both;
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(32 * W) : "memory");
      su = sx = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        su += red[i & 1][group * W + w][0];
        sx += red[i & 1][group * W + w][1];
      }
    }
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      if (32 * W * k + first >= pieces) continue;
      P pr;
      if (dres) pr = take(slot, 2, k);
      float2 v[kUnits];
#pragma unroll
      for (int e = 0; e < kUnits; ++e) {
        const float2 h = mul(add(px[k].unit(e), all<8>(-mu)), all<8>(rs)), u = mul(py[k].unit(e), pg[k].unit(e));
        const float2 w = add(fma(h, all<8>(-sx), u), all<8>(-su));
        v[e] = dres ? fma(w, all<8>(rs), pr.unit(e)) : mul(w, all<8>(rs));
      }
      P::store(dX + (r0 + i) * row_bytes + 16 * (32 * W * k + first), v);
    }
    slot = slot + 1 == D ? 0 : slot + 1;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  float* rows = reinterpret_cast<float*>(ln_rows);  // [groups][d]
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < NP; ++k)
      if (32 * W * k + first < pieces)
#pragma unroll
        for (int e = 0; e < kUnits; e += 2) {
          const float2 a = which ? ab[k][e] : ag[k][e], b = which ? ab[k][e + 1] : ag[k][e + 1];
          *reinterpret_cast<float4*>(rows + group * d + P::kCols * (32 * W * k + first) + 2 * e) = make_float4(a.x, a.y, b.x, b.y);
        }
    __syncthreads();
    for (int j = threadIdx.x; j < d; j += 32 * kWarps) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps / W; ++w) v += rows[w * d + j];
      part[((int64_t)blockIdx.x * 2 + which) * d + j] = v;
    }
  }
}

// Column sums of the blocks' partial rows part [nblk][2 d]: 16 columns a block, 16 row groups, then a tree.  A block is small
// enough to become resident beside the kernel before it (against 1024 threads: T = 8192, d = 5120 in bf16 62 -> 60 us,
// T = 4096, d = 256 7.4 -> 6.8).
constexpr int kFinishCols = 16, kFinishThreads = 256;
__global__ void __launch_bounds__(kFinishThreads) k_layernorm_bwd_finish(const float* __restrict__ part, int nblk, int d,
                                                                         float* __restrict__ dg, float* __restrict__ db) {
  constexpr int kGroups = kFinishThreads / kFinishCols;
  __shared__ float sum[kGroups][kFinishCols + 1];
  wait_for_previous();
  const int tx = threadIdx.x % kFinishCols, ty = threadIdx.x / kFinishCols;
  const int j = blockIdx.x * kFinishCols + tx;
  float s = 0.0f;
  if (j < 2 * d)
    for (int k = ty; k < nblk; k += kGroups * 10) {
      float v[10];  // 10 loads in flight
#pragma unroll
      for (int q = 0; q < 10; ++q) v[q] = k + kGroups * q < nblk ? part[(int64_t)(k + kGroups * q) * 2 * d + j] : 0.0f;
#pragma unroll
      for (int q = 0; q < 10; ++q) s += v[q];
    }
  sum[ty][tx] = s;
  __syncthreads();
#pragma unroll
  for (int w = kGroups / 2; w > 0; w >>= 1) {
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

// The kernel's shared memory limit, raised once per device.
template <class Kernel>
cudaError_t ring_limit(Kernel* k, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (done.load(std::memory_order_relaxed) >> (dev & 63) & 1)) return e;
  e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kLnSmemBudget);
  if (e == cudaSuccess) done.fetch_or(1ull << (dev & 63));
  return e;
}

// Slots of a ring, at least one, within a block's share of the shared memory; fewer blocks per SM where that leaves
// each fewer than three.
int ring_slots(size_t slot, int* per_sm) {
  while (*per_sm > 1 && kLnSmemBudget / *per_sm < 3 * slot) --*per_sm;
  const int n = (int)(kLnSmemBudget / *per_sm / slot);
  return n < kLnSlotsMax ? n : kLnSlotsMax;
}

template <int F32, int VEC, int NP, int W>
cudaError_t fwd_go(const void* x, const void* g, const void* b, int64_t T, int d, float eps, void* y, float* mean,
                   float* rstd, const Launch& L) {
  constexpr int RT = VEC == 8 && !F32 && NP <= 3 ? 2 : 1, rows = 8 % W == 0 ? RT * (8 / W) : RT;
  auto* k = k_layernorm_fwd<F32, VEC, NP, W, RT>;
  const size_t slot = ln_region((uint32_t)(rows * d * (F32 ? 4 : 2)));
  int per_sm = ln_fwd_per_sm(VEC, W);
  const int S = ring_slots(slot, &per_sm);
  static std::atomic<uint64_t> done{0};
  cudaError_t e = ring_limit(k, done);
  if (e != cudaSuccess) return e;
  const int64_t need = (T + rows - 1) / rows, wave = (int64_t)L.num_sms * per_sm;
  k<<<(unsigned)(need < wave ? need : wave), ln_fwd_threads(W), S * slot, L.stream>>>(x, g, b, T, d, eps, S, y, mean,
                                                                                      rstd, L.status);
  return launched(L);
}

// The fewest warps (a power of two) whose lanes hold the row: in fp32 up to 4 pieces of 8 columns a lane, in bf16
// up to 3 (two rows of 4 do not fit in the registers: T = 16384, d = 4096 takes 70 us so, one such row at a time 51, and
// 42 with twice the warps), in odd widths up to 16 single columns.  In bf16 five or ten warps where they fit the row better
// (T = 16384, d = 2560: 36 us with four, 30 with five).
template <int F32>
cudaError_t fwd_t(const void* x, const void* g, const void* b, int64_t T, int d, float eps, void* y, float* mean,
                  float* rstd, const Launch& L) {
#define FP8Q_LN_FWD(VEC, NP, W) return fwd_go<F32, VEC, NP, W>(x, g, b, T, d, eps, y, mean, rstd, L)
  constexpr int kCols = 256;  // of a warp's lanes with a piece each
  if (d % 8 == 0) {
    if (d <= kCols) FP8Q_LN_FWD(8, 1, 1);
    if (d <= 2 * kCols) FP8Q_LN_FWD(8, 2, 1);
    if (d <= 3 * kCols) FP8Q_LN_FWD(8, 3, 1);
    if constexpr (F32) {
      if (d <= 4 * kCols) FP8Q_LN_FWD(8, 4, 1);
      if (d <= 6 * kCols) FP8Q_LN_FWD(8, 3, 2);
      if (d <= 8 * kCols) FP8Q_LN_FWD(8, 4, 2);
      if (d <= 12 * kCols) FP8Q_LN_FWD(8, 3, 4);
      if (d <= 16 * kCols) FP8Q_LN_FWD(8, 4, 4);
      if (d <= 24 * kCols) FP8Q_LN_FWD(8, 3, 8);
      if (d <= 32 * kCols) FP8Q_LN_FWD(8, 4, 8);
    } else {
      if (d <= 4 * kCols) FP8Q_LN_FWD(8, 2, 2);
      if (d <= 6 * kCols) FP8Q_LN_FWD(8, 3, 2);
      if (d <= 8 * kCols) FP8Q_LN_FWD(8, 2, 4);
      if (d <= 10 * kCols) FP8Q_LN_FWD(8, 2, 5);
      if (d <= 12 * kCols) FP8Q_LN_FWD(8, 3, 4);
      if (d <= 16 * kCols) FP8Q_LN_FWD(8, 2, 8);
      if (d <= 20 * kCols) FP8Q_LN_FWD(8, 2, 10);
      if (d <= 24 * kCols) FP8Q_LN_FWD(8, 3, 8);
      if (d <= 32 * kCols) FP8Q_LN_FWD(8, 2, 16);
    }
    if (d <= 48 * kCols) FP8Q_LN_FWD(8, 3, 16);
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

// The launch shape of a block a row.  d is a multiple of 8 (the widest, and fp32 above 4096): a thread has one piece of 8
// columns up to d = 8192, else 4.
// Otherwise 1 to 32 single columns, of 128 threads up to d = 1024 and of 512 above.
constexpr int kLnNarrow = 128;
constexpr int bwd_np(int d) {
  if (d % 8 == 0) return d <= 8 * kLnWide ? 1 : 4;
  const int threads = d > 8 * kLnNarrow ? kLnThreads : kLnNarrow;
  int np = 1;
  while (d > np * threads) np *= 2;
  return np;
}
constexpr int bwd_threads(int d) {
  if (d % 8 != 0) return d > 8 * kLnNarrow ? kLnThreads : kLnNarrow;
  return ((d / 8 + bwd_np(d) - 1) / bwd_np(d) + 31) / 32 * 32;
}
// Resident blocks per SM: 1024 threads of 64 registers (up to 16 narrow blocks: a row is a chain of
// dependent steps of about 0.8 us, so narrow rows need many blocks at work), or 512 of 128.
constexpr int bwd_per_sm(int d) {
  if (bwd_np(d) * (d % 8 == 0 ? 8 : 1) > 8) return 1;
  const int n = 1024 / bwd_threads(d);
  return n < 16 ? n : 16;
}
constexpr int kLnPlanSms = 152;
static_assert(bwd_per_sm(4104) == 1 && bwd_per_sm(8192) == 1, "fp32 widths that the bf16 runs' workspace holds too");

template <int F32, int VEC, int NP, int STRIDE>
cudaError_t bwd_go(const void* dY, const void* x, const void* g, const float* mean, const float* rstd, const void* dres,
                   int64_t T, int d, void* dX, float* part, int* nblk, const Launch& L) {
  auto* k = k_layernorm_bwd<F32, VEC, NP, STRIDE>;
  const size_t slot = (size_t)ln_region((uint32_t)(d * (F32 ? 4 : 2))) * (dres ? 3 : 2);
  int per_sm = bwd_per_sm(d);
  const int S = ring_slots(slot, &per_sm);
  static std::atomic<uint64_t> done{0};
  cudaError_t e = ring_limit(k, done);
  if (e != cudaSuccess) return e;
  // one wave of resident blocks, each with a run of consecutive rows (at most layernorm_bwd_blocks of them)
  const int64_t most = (int64_t)(L.num_sms < kLnPlanSms ? L.num_sms : kLnPlanSms) * per_sm;
  const int rows = (int)((T + most - 1) / most);
  *nblk = (int)((T + rows - 1) / rows);
  k<<<*nblk, bwd_threads(d), S * slot, L.stream>>>(dY, x, g, mean, rstd, dres, T, d, rows, S, dX, part, L.status);
  return launched(L);
}

constexpr int kRunsNarrow = 256, kRunsMost = 8192;  // bf16 columns of a warp with one vector a lane; of 16 with two

template <int F32, int NP, int W>
cudaError_t runs_go(const void* dY, const void* x, const void* g, const float* mean, const float* rstd, const void* dres,
                    int64_t T, int d, void* dX, float* part, int* nblk, const Launch& L) {
  using R = RunPlan<NP, W>;
  static_assert(R::kBytes * R::kPerSm <= (int)kLnSmemBudget, "shared memory per SM");
  auto* k = k_layernorm_bwd_runs<F32, NP, W>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = ring_limit(k, done);
  if (e != cudaSuccess) return e;
  // a wave of resident blocks, each group of warps with a run of consecutive rows
  constexpr int kGroups = R::kWarps / W;
  const int64_t groups = (int64_t)(L.num_sms < kLnPlanSms ? L.num_sms : kLnPlanSms) * R::kPerSm * kGroups;
  const int run = (int)((T + groups - 1) / groups), block_rows = run * kGroups;
  *nblk = (int)((T + block_rows - 1) / block_rows);
  auto bytes = [](const void* p) { return static_cast<const uint8_t*>(p); };
  k<<<*nblk, 32 * R::kWarps, R::kBytes, L.stream>>>(bytes(dY), bytes(x), bytes(g), mean, rstd, bytes(dres), T, d, run,
                                                    static_cast<uint8_t*>(dX), part);
  return launched(L);
}

template <int F32>
cudaError_t bwd_t(const void* dY, const void* x, const void* g, const float* mean, const float* rstd, const void* dres,
                  int64_t T, int d, void* dX, float* part, int* nblk, const Launch& L) {
#define FP8Q_LN_BWD(VEC, NP, STRIDE) \
  return bwd_go<F32, VEC, NP, STRIDE>(dY, x, g, mean, rstd, dres, T, d, dX, part, nblk, L)
  if (d % 8 == 0) {
#define FP8Q_LN_RUNS(NP, W) return runs_go<F32, NP, W>(dY, x, g, mean, rstd, dres, T, d, dX, part, nblk, L)
    constexpr int kCols = 2 * kRunsNarrow / (F32 ? 2 : 1);  // of a warp with two
    static_assert(F32 || 16 * kCols == kRunsMost, "widths in runs");
    if (2 * d <= kCols) FP8Q_LN_RUNS(1, 1);
    if (d <= kCols) FP8Q_LN_RUNS(2, 1);
    if (d <= 2 * kCols) FP8Q_LN_RUNS(2, 2);
    if (d <= 3 * kCols) FP8Q_LN_RUNS(2, 3);
    if (d <= 4 * kCols) FP8Q_LN_RUNS(2, 4);
    if (d <= 5 * kCols) FP8Q_LN_RUNS(2, 5);
    if (d <= 6 * kCols) FP8Q_LN_RUNS(2, 6);
    if (d <= 7 * kCols) FP8Q_LN_RUNS(2, 7);
    if (d <= 8 * kCols) FP8Q_LN_RUNS(2, 8);
    if (d <= 10 * kCols) FP8Q_LN_RUNS(2, 10);
    if (d <= 12 * kCols) FP8Q_LN_RUNS(2, 12);
    if (d <= 16 * kCols) FP8Q_LN_RUNS(2, 16);
#undef FP8Q_LN_RUNS
    if constexpr (F32) {
      if (d <= 8 * kLnWide) FP8Q_LN_BWD(8, 1, 0);
    }
    FP8Q_LN_BWD(8, 4, 0);
  }
  if (d <= kLnNarrow) FP8Q_LN_BWD(1, 1, kLnNarrow);
  if (d <= 2 * kLnNarrow) FP8Q_LN_BWD(1, 2, kLnNarrow);
  if (d <= 4 * kLnNarrow) FP8Q_LN_BWD(1, 4, kLnNarrow);
  if (d <= 8 * kLnNarrow) FP8Q_LN_BWD(1, 8, kLnNarrow);
  if (d <= 4 * kLnThreads) FP8Q_LN_BWD(1, 4, kLnThreads);
  if (d <= 8 * kLnThreads) FP8Q_LN_BWD(1, 8, kLnThreads);
  if (d <= 16 * kLnThreads) FP8Q_LN_BWD(1, 16, kLnThreads);
  FP8Q_LN_BWD(1, 32, kLnThreads);
#undef FP8Q_LN_BWD
}

}  // namespace

// Blocks of the first launch at most, of either type: those of k_layernorm_bwd_runs for the widths that it takes in bf16
// (in fp32 the wider ones of them have a block a row and an SM).
int layernorm_bwd_blocks(int64_t T, int d) {
  const bool runs = d % 8 == 0 && d <= kRunsMost;
  const int64_t n = (int64_t)kLnPlanSms * (!runs ? bwd_per_sm(d) : d <= kRunsNarrow ? RunPlan<1, 1>::kPerSm : RunPlan<2, 1>::kPerSm);
  return (int)(T < n ? T : n);
}

cudaError_t launch_layernorm_fwd(const void* x, int f32, const void* g, const void* b, int64_t T, int d, float eps,
                                 void* y, float* mean, float* rstd, const Launch& L) {
  return f32 ? fwd_t<1>(x, g, b, T, d, eps, y, mean, rstd, L) : fwd_t<0>(x, g, b, T, d, eps, y, mean, rstd, L);
}

cudaError_t launch_layernorm_bwd(const void* dY, const void* x, int f32, const void* g, const float* mean,
                                 const float* rstd, const void* dres, int64_t T, int d, void* dX, float* dg, float* db,
                                 float* part, const Launch& L) {
  int nblk = 0;
  cudaError_t e = f32 ? bwd_t<1>(dY, x, g, mean, rstd, dres, T, d, dX, part, &nblk, L)
                      : bwd_t<0>(dY, x, g, mean, rstd, dres, T, d, dX, part, &nblk, L);
  if (e != cudaSuccess) return e;
  e = launch_dependent(k_layernorm_bwd_finish, (unsigned)((2 * d + kFinishCols - 1) / kFinishCols), kFinishThreads, 0, L.stream, part, nblk, d, dg, db);
  if (L.launches) ++*L.launches;
  return e;
}

}  // namespace fp8q
