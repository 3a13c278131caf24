// Softmax cross entropy of a linear head over a large vocabulary, without keeping the logits.
//
//   z = x W^T,  lse_t = log sum_v e^{z_tv},  loss_t = lse_t - z_{t,y_t} (0 for an ignored token);
//   G = dloss_t (e^{z - lse_t} - 1[v = y_t]) (0 for an ignored token),  dX = G W,  dW = G^T x.
// The forward is one product whose epilogue keeps, of each 128-column piece of a row, the maximum and
// the sum of exponentials below it; a second kernel joins them.  The backward walks the vocabulary
// in pieces: the piece's logits again, turned into G in the epilogue, then its share of dX and its rows
// of dW.  All products are bf16 on the tensor cores with fp32 sums, and bound by them.
// (Up to 128 tokens with a small vocabulary, the logits do come to memory: in parts of K, see tok_logit_splits.)
//
// G is kept in bf16, the tensor cores' operand type, as G / s with s = max_t |dloss_t|: a mean's
// one weight for all tokens then leaves no rounding of its own in G's large entries (p - 1 near -1).
// s joins the products in fp32.  With few tokens (up to kTwoParts, where the products wait for memory) nothing
// averages the rounding of a token's largest entry, so G is kept there as two bf16 parts, the value and what its rounding
// lost, 2 Tp rows in all (Tp = T in whole blocks of 32): dX adds the two parts' products, dW runs over both with x twice
// (T = 2, d = 4080, V = 1686: dW's error 3.5e-3 of its norm with one part, as the plain fp32 form's 2.2e-3 with two;
// d = 2048, V = 32000: 89 -> 90 us for 24 tokens, 89 -> 95 for 60, but 97 -> 111 for 100).  An ignored
// token's row of x is replaced by zero before dW = G^T x, so
// that a padded row may hold anything (0 times a NaN would reach every row of dW).
#include "fp8q_common.cuh"
#include "fp8q_head.cuh"
#include "fp8q_internal.h"

#include <atomic>
#include <mutex>

namespace fp8q {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ce_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---------------------------------------------------------------------------
// The product: two SMs per 256 x 256 tile (tcgen05.mma cta_group::2), persistent, warp-specialised.
//
// A pair of CTAs (a cluster of two) computes C[256, 256] += A[256, K] B[256, K]^T in steps of 64 of K: each
// CTA loads its 128 rows of A and its 128 columns of B (32 KB a stage, where one SM with a
// 128 x 256 tile would load 48 KB for the same work: the operand bytes that reach an SM are what
// bounds the 128 x 256 kernel of the block's products), the even CTA issues the MMAs for both, and
// each CTA's tensor memory receives its 128 rows.  Two accumulators (2 x 256 columns) let a tile's
// epilogue run under the next tile's MMAs.
//   warp 0      TMA producer of its CTA; both signal the even CTA's full barrier;
//   warp 1      the even CTA's MMA issuer; its commits free the stage, and hand over the
//               accumulator, in both CTAs;
//   warp 2      tensor memory;
//   warps 3-10  epilogue: warp w reads lanes 32 (w % 4) ..; the first four take columns 0-127, the others 128-255.
// The tensor cores' fp32 sums drop what falls below the sum's last place at each step of 16 of K, so a logit's error grows
// with the steps (products of one sign, parts of 1024: 12 2^-23 of the logit on average); the loss's logits are therefore
// summed over K in parts that the epilogue adds in registers, the accumulators changing hands after each.  Parts of 1024
// with many tokens (T = 4096, d = 3584, V = 50257: the loss's error 2.7e-6 -> 0.7e-6 of its norm, 868 -> 888 us).  Up to 128
// tokens nothing averages a token's error (T = 1, d = 2048, V = 32000: 6.3e-6 so), and the parts are of 128, 0.7 2^-23 of
// the logit, with as many accumulators as tensor memory has room for, up to 8 (T = 24, d = 4096, V = 100000 141 -> 146 us,
// T = 120 147 -> 155, d = 2048, V = 32000 38.9 -> 39.4, cold; parts of 64: 161, 179, 40.3; of 192: 144, 151, 39.1).
// Up to 128 tokens the operands trade places (kTok*): the 256 rows of a pair's tile are rows of W (of W^T for
// dX) and its NT = 32, 64 or 128 columns the tokens, so that W streams at HBM's rate and the tensor cores do not
// work on padding.  The softmax statistics then run down the tile's lanes: each warp turns its 32 x 32 blocks
// in shared memory and keeps a running pair for each token over all its tiles.  Measured against the
// padded tiles (d = 2048, V = 32000): forward 42 against 54 us for one token, 42 / 46 for 24, 45 / 46 for 100;
// backward 90 / 112, 89 / 94, 97 / 100 (when it was made; now 39, 39, 43 and 87, 89, 93).
//
// Every wait is bounded.  On expiry a CTA records the time-out and stops; once all its roles have, its copies in flight, which
// signal the other CTA, get kCopyDrainNs to land; the pair meets at a cluster barrier and frees its tensor memory.
// ---------------------------------------------------------------------------
constexpr int PM = 256, PN = 256, PK = 64;
constexpr int kHalfTile = 128 * 128;  // bytes: 128 rows (or columns) x 64 bf16
constexpr int kEpiWarp = 3;           // the first of the 8 epilogue warps
constexpr int kPairThreads = 32 * (kEpiWarp + 8);
constexpr int kTokMax = 128;  // tokens up to which the operands trade places
constexpr int kTwoParts = 64; // tokens up to which the backward keeps G in two parts
// K of a partial sum of the logits, in blocks of 64, and the accumulators that take turns: up to 128 tokens and above.
constexpr int kSegTok = 2, kSegWide = 16;
constexpr int acc_count(int NT) { return NT == 256 ? 2 : NT == 128 ? 4 : 8; }
constexpr int kPartBlocks = 16; // K of a part of the logits that comes to memory, at most

enum PairMode {
  kPairLse = 0,   // per row and 128 columns: log2-domain maximum and sum; the target's logit
  kPairGrad = 1,  // G / s as bf16
  kPairDx = 2,    // dX: fp32 store, fp32 add or bf16 of the joined sum
  kPairDw = 3,    // dW: bf16 or fp32
  kTokLse = 4,    // the same three with the tokens as columns: statistics of a CTA's rows of W
  kTokGrad = 5,   //   G / s in two parts, stored by token
  kTokDx = 6,     //   dX's sum in fp32, by token, the parts of K and of G apart
  kTokLogits = 7, // the logits of few tokens in fp32, by token, the parts of K apart
};
enum PairOut { kOutF32Store = 0, kOutF32Add = 1, kOutBf16 = 2, kOutBf16Join = 3 };

// The shared memory of a CTA for tiles of NT columns.  dW's products are short where there are few
// tokens, and bound by its stores: it trades a stage for staging buffers of two blocks of 4 KB a warp.
template <int MODE, int NT>
struct PairPlan {
  static constexpr int kB = NT / 2 * 128;  // bytes of its share of B in a stage
  static constexpr int kStage = kHalfTile + kB;
  static constexpr int kStages = MODE == kPairDw ? 5 : NT == 256 ? 6 : NT == 128 ? 7 : NT == 64 ? 9 : 10;
  static constexpr int kStaging = MODE == kPairDw ? 8192 : 4096;  // per epilogue warp
  static constexpr int kStagingOffset = kStages * kStage;
  static constexpr int kTokOffset = kStagingOffset + 8 * kStaging;
  static constexpr int kBarOffset = kTokOffset + (MODE == kTokGrad ? NT * 16 : 0);
  static constexpr int kAcc = acc_count(NT);
  static constexpr int kSmem = kBarOffset + 512 + 1024;
  static_assert(kSmem <= 232448, "shared memory per CTA");
  static_assert(kStage % 1024 == 0, "swizzle atoms");
};
constexpr uint64_t kCopyDrainNs = 5000000ull;  // far beyond any copy in flight

// Division of n < 2^31 by a number known at the launch: n m >> s with m = ceil(2^s / d), s = 31 + ceil(log2 d).
// (Roles walk short tiles in less time than a chain of integer divisions takes.)
struct Divisor {
  uint32_t d, m, s;
};
Divisor divisor(int d) {
  uint32_t l = 0;
  while ((1ull << l) < (uint64_t)d) ++l;
  return Divisor{(uint32_t)d, (uint32_t)(((1ull << (31 + l)) + (uint32_t)d - 1) / (uint32_t)d), 31 + l};
}
__device__ __forceinline__ int divide(int n, const Divisor& d) { return (int)(((uint64_t)(uint32_t)n * d.m) >> d.s); }

struct PairArgs {
  int M, N, K;
  int m_tiles, n_tiles, k_blocks, group;
  int splits, split_blocks;  // parts of K, and the blocks of 64 in each (the last may have fewer)
  int num_tiles;             // m_tiles n_tiles splits
  Divisor by_part, by_span, by_group, by_last;  // tiles of a part, of a group; M tiles of a group, of the last group
  uint32_t idesc;
  int out;                  // PairOut; with splits > 1 fp32, split i at rows i 256 m_tiles of C
  const float* scale;       // s, or null: the sum as it is
  float* acc;               // kOutBf16Join: the sum so far [M, N]
  int v0;                   // kPairGrad, kTokGrad: the piece's first column
  int half_rows;            // rows of A in each CTA's half of a tile: 128, or fewer (kTokLse: tok_half_rows)
  int rows_lo;              // kTokGrad: the first row of G's second part, or 0: it has one
  const int64_t* targets;   // kPairLse, kTokLse
  int V;                    // kPairLse, kTokLse
  float2* part;             // (maximum log2e, sum) pairs: kPairLse [2 n_tiles][M], kTokLse [CTAs][N]
  float* zy;                // kPairLse, kTokLse: each token's target logit
  const float4* rows;       // kPairGrad, kTokGrad: each token's {lse log2e, dloss / s, target or -1 (int bits), 0}
  unsigned* status;
  uint64_t wait_ns;         // the self-test's limit of every wait of the pipeline, or 0 (issued MMAs keep kWaitLimitNs)
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t map_to_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A 2D tile into this CTA's shared memory; the bytes are counted on `bar`, a barrier of either CTA.
__device__ __forceinline__ void pair_load_2d(void* dst, const CUtensorMap* tm, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], "
      "[%2];" ::"r"(smem_addr(dst)),
      "l"(tm), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on the barrier at this offset in the CTAs of `mask` once the MMAs issued so far are done.
__device__ __forceinline__ void pair_commit(uint64_t* bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_addr(bar)),
      "h"(mask)
      : "memory");
}
// No memory but tensor memory changes hands here, and the tcgen05 fences order that: an arrival that releases at cluster
// scope would wait for all of the warp's stores (0.9 us a tile where a tile takes 2.3).
__device__ __forceinline__ void remote_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void out_store_2d(const CUtensorMap* tm, uint32_t src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(tm), "r"(src), "r"(x),
               "r"(y)
               : "memory");
}
// fp32 addition in global memory.  Each element is added to once per launch, so the order is fixed.
__device__ __forceinline__ void out_add_2d(const CUtensorMap* tm, uint32_t src, int x, int y) {
  asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(tm),
               "r"(src), "r"(x), "r"(y)
               : "memory");
}
__device__ __forceinline__ void out_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void sts_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// A warp's block of a tile on its way out: staged in the layout of the tensor map's swizzle and stored by
// lane 0, the blocks taking the warp's BYTES of staging in turn.  Rows of 64 bytes: 32 bf16; of 128: 64 bf16 or 32 fp32.
template <int BYTES>
struct PairStager {
  uint32_t buf;
  int lane, turn = 0;
  __device__ __forceinline__ PairStager(uint32_t b, int l) : buf(b), lane(l) {}
  template <int BLOCK>
  __device__ __forceinline__ uint32_t acquire() {
    constexpr int n = BYTES / BLOCK;
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(n - 1) : "memory");
    __syncwarp();
    const uint32_t b = buf + BLOCK * turn;
    turn = turn + 1 == n ? 0 : turn + 1;
    return b;
  }
  __device__ __forceinline__ void publish(const CUtensorMap* tm, uint32_t b, int x, int y, bool add = false) {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) {
      if (add) out_add_2d(tm, b, x, y);
      else out_store_2d(tm, b, x, y);
      out_commit();
    }
  }
  __device__ __forceinline__ void bf16(const CUtensorMap* tm, const float (&v)[32], int x, int y) {
    const uint32_t b = acquire<2048>();
#pragma unroll
    for (int q = 0; q < 4; ++q)
      sts_v4(b + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4), pack_bf16x2(v[8 * q], v[8 * q + 1]),
             pack_bf16x2(v[8 * q + 2], v[8 * q + 3]), pack_bf16x2(v[8 * q + 4], v[8 * q + 5]),
             pack_bf16x2(v[8 * q + 6], v[8 * q + 7]));
    publish(tm, b, x, y);
  }
  __device__ __forceinline__ void bf16_wide(const CUtensorMap* tm, const uint32_t (&a)[32], const uint32_t (&c)[32],
                                            float f, int x, int y) {
    const uint32_t b = acquire<4096>();
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int j = 8 * (q & 3) + 2 * k;
        w[k] = pack_bf16x2(f * __uint_as_float(q < 4 ? a[j] : c[j]), f * __uint_as_float(q < 4 ? a[j + 1] : c[j + 1]));
      }
      sts_v4(b + lane * 128 + ((q ^ (lane & 7)) << 4), w[0], w[1], w[2], w[3]);
    }
    publish(tm, b, x, y);
  }
  __device__ __forceinline__ void f32(const CUtensorMap* tm, const uint32_t (&a)[32], float f, int x, int y, bool add) {
    const uint32_t b = acquire<4096>();
#pragma unroll
    for (int q = 0; q < 8; ++q)
      sts_v4(b + lane * 128 + ((q ^ (lane & 7)) << 4), __float_as_uint(f * __uint_as_float(a[4 * q])),
             __float_as_uint(f * __uint_as_float(a[4 * q + 1])), __float_as_uint(f * __uint_as_float(a[4 * q + 2])),
             __float_as_uint(f * __uint_as_float(a[4 * q + 3])));
    publish(tm, b, x, y, add);
  }
};

// (maximum, sum) of logits in log2 units, brought together; a pair that holds nothing is (-inf, 0).
__device__ __forceinline__ float2 ce_join2(float2 a, float2 b) {
  const float m = fmaxf(a.x, b.x);
  if (m == -INFINITY) return make_float2(m, a.y + b.y);
  return make_float2(m, a.y * ce_exp2(a.x - m) + b.y * ce_exp2(b.x - m));
}
// lse - zy of a row's pair, about the maximum in log2 units: where the target is the likeliest entry, that difference is
// exact, while lse itself is rounded to 2^-24 of its size, which a small loss may not be far above.
__device__ __forceinline__ float ce_loss(float2 r, float zy) { return kLn2 * (fmaf(-zy, kLog2e, r.x) + log2f(r.y)); }
// 16 columns of this thread's tensor-memory lane, added to z.
__device__ __forceinline__ void ce_tmem_add16(uint32_t taddr, float* z) {
  uint32_t a[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]), "=r"(a[7]), "=r"(a[8]),
        "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]), "=r"(a[14]), "=r"(a[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int j = 0; j < 16; ++j) z[j] += __uint_as_float(a[j]);
}

// The pair of N logits.  Where all of them are -inf (masked columns; a mask of the type's lowest value gets there in
// log2 units), their sum is 0: about a maximum of -inf it would be NaN, and reach the whole row.
template <int N>
__device__ __forceinline__ float2 ce_pair(const float (&z)[N]) {
  float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int j = 0; j < N; ++j) mx[j & 3] = fmaxf(mx[j & 3], z[j]);
  const float m = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * kLog2e;
  const float about = m == -INFINITY ? 0.0f : m;
  float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int j = 0; j < N; ++j) sum[j & 3] += ce_exp2(fmaf(z[j], kLog2e, -about));
  return make_float2(m, (sum[0] + sum[1]) + (sum[2] + sum[3]));
}

// Tile -> (part of K, M tile, N tile): a part's tiles in groups of p.group M tiles, all N tiles of a group,
// M fastest inside it.  Its blocks of K are [k0, k1).
__device__ __forceinline__ int pair_coords(int tile, const PairArgs& p, int& mb, int& nb, int& k0, int& k1) {
  const int part = divide(tile, p.by_part);
  tile -= part * (int)p.by_part.d;
  k0 = part * p.split_blocks;
  k1 = min(k0 + p.split_blocks, p.k_blocks);
  const int grp = divide(tile, p.by_span), first = grp * p.group, local = tile - grp * (int)p.by_span.d;
  const bool full = first + p.group <= p.m_tiles;  // the last group may have fewer rows
  nb = divide(local, full ? p.by_group : p.by_last);
  mb = first + local - nb * (int)(full ? p.by_group.d : p.by_last.d);
  return part;
}

// SHORT: the self-test, whose waits poll, so that limits of nanoseconds are honoured (as a branch of one kernel: 741 -> 867 us
// at T = 4096, d = 3584, V = 50257).
template <int A_MN, int B_MN, int MODE, int NT, int SHORT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    k_ce_gemm(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
              const __grid_constant__ CUtensorMap tmC, const PairArgs p) {
  using PL = PairPlan<MODE, NT>;
  constexpr bool kSeg = MODE == kPairLse || MODE == kTokLse || MODE == kTokLogits;  // the sum over K comes in parts
  constexpr bool kTok = MODE >= kTokLse;
  constexpr int kSegBlocks = kTok ? kSegTok : kSegWide;
  static_assert(!(kTok && B_MN), "the tokens are a K-major operand");
  extern __shared__ uint8_t pair_smem[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(pair_smem) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + PL::kBarOffset);
  uint64_t* empty = full + PL::kStages;
  uint64_t* tfull = empty + PL::kStages;  // [kAcc]
  uint64_t* tempty = tfull + PL::kAcc;    // [kAcc]
  uint64_t* drain = tempty + PL::kAcc;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  const int first = (int)(blockIdx.x >> 1), step = (int)(gridDim.x >> 1);
  const int half_rows = MODE == kTokLse ? p.half_rows : 128;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if constexpr (SHORT) return mbar_poll(bar, parity, abort_flag, p.wait_ns);
    else return mbar_wait_held(bar, parity, abort_flag);
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < PL::kStages; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    for (int a = 0; a < PL::kAcc; ++a) { mbar_init(&tfull[a], 1); mbar_init(&tempty[a], 16); }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    if (MODE != kPairLse && MODE != kTokLse && MODE != kTokDx && MODE != kTokLogits) tma_prefetch_desc(&tmC);
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  wait_for_previous();
  start_dependents();
  // kTokGrad: the tokens' rows (kTokLse: their targets) where every lane can read them
  float4* tok = reinterpret_cast<float4*>(smem + PL::kTokOffset);
  if (MODE == kTokGrad && threadIdx.x < NT)
    tok[threadIdx.x] = (int)threadIdx.x < p.N ? p.rows[threadIdx.x] : make_float4(0.0f, 0.0f, __int_as_float(-1), 0.0f);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers exist, both have their tensor memory
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer ----------------
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = first; tile < p.num_tiles && ok; tile += step) {
        int mb, nb, kb0, kb1;
        pair_coords(tile, p, mb, nb, kb0, kb1);
        const int m0 = (2 * mb + rank) * half_rows, n0 = nb * NT + NT / 2 * rank;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!wait(&empty[stage], phase ^ 1u)) { ok = false; break; }
          uint8_t* sA = smem + stage * PL::kStage;
          uint8_t* sB = sA + kHalfTile;
          const uint32_t bar = map_to_rank(smem_addr(&full[stage]), 0);
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * (half_rows * 128 + PL::kB));
          const int k0 = kb * PK;
          if (A_MN) {  // two 64-element-wide boxes of 64 rows of K
            pair_load_2d(sA, &tmA, bar, m0, k0);
            pair_load_2d(sA + kHalfTile / 2, &tmA, bar, m0 + 64, k0);
          } else {
            pair_load_2d(sA, &tmA, bar, k0, m0);
          }
          if (B_MN) {
            pair_load_2d(sB, &tmB, bar, n0, k0);
            pair_load_2d(sB + kHalfTile / 2, &tmB, bar, n0 + 64, k0);
          } else {
            pair_load_2d(sB, &tmB, bar, k0, n0);
          }
          if (++stage == PL::kStages) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok) {
        atomicOr(p.status, kStatusTimeout);
        *abort_flag = 1;
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      // ---------------- MMA issuer ----------------
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int tile = first; tile < p.num_tiles && ok; tile += step) {
        int mb, nb, kb0, kb1;
        pair_coords(tile, p, mb, nb, kb0, kb1);
        for (int kb = kb0; kb < kb1 && ok;) {
          const int begin = kb, end = kSeg ? min(kb + kSegBlocks, kb1) : kb1;
          if (!wait(&tempty[acc], acc_phase ^ 1u)) { ok = false; break; }
          tc_fence_after();
          const uint32_t d = tmem_base + (uint32_t)(acc * NT);
          for (; kb < end; ++kb) {
            if (!wait(&full[stage], phase)) { ok = false; break; }
            tc_fence_after();
            const uint32_t sA = smem_addr(smem + stage * PL::kStage), sB = sA + kHalfTile;
#pragma unroll
            for (int kk = 0; kk < PK / 16; ++kk) {
              // K-major: 32 bytes further inside the 128-byte swizzle row; MN-major: 16 rows of K further,
              // the second 64-element block of MN 8 KB on
              const uint64_t ad = A_MN ? smem_desc_sw128(sA + kk * 2048, kHalfTile / 2, 1024) : smem_desc_sw128(sA + kk * 32, 16, 1024);
              const uint64_t bd = B_MN ? smem_desc_sw128(sB + kk * 2048, kHalfTile / 2, 1024) : smem_desc_sw128(sB + kk * 32, 16, 1024);
              pair_mma(d, ad, bd, p.idesc, (kb - begin) | kk ? 1u : 0u);
            }
            pair_commit(&empty[stage], 3);
            if (++stage == PL::kStages) { stage = 0; phase ^= 1u; }
          }
          if (!ok) break;
          pair_commit(&tfull[acc], 3);
          if (++acc == PL::kAcc) { acc = 0; acc_phase ^= 1u; }
        }
      }
      if (!ok) {
        atomicOr(p.status, kStatusTimeout);
        *abort_flag = 1;
      }
      // every MMA issued is done before tensor memory is released
      pair_commit(drain, 1);
      int dummy = 0;
      mbar_wait_held(drain, 0, &dummy);
    }
  } else if (warp >= kEpiWarp) {
    // ---------------- epilogue ----------------
    const int sub = warp & 3, half = (warp - kEpiWarp) >> 2;
    PairStager<PL::kStaging> out(smem_addr(smem + PL::kStagingOffset + (warp - kEpiWarp) * PL::kStaging), lane);
    const uint32_t tempty0 = map_to_rank(smem_addr(tempty), 0);
    const float alpha = p.scale ? *p.scale : 1.0f;
    // kTok*: warpgroup `half` takes the 32-token blocks half, half + 2, ...; lane = token after the turn
    constexpr int kBlocks = NT >= 64 ? NT / 64 : 1;
    float2 tp[kBlocks];
    int ty[kBlocks];
    if (MODE == kTokLse)
#pragma unroll
      for (int i = 0; i < kBlocks; ++i) {
        const int t = 32 * (half + 2 * i) + lane;
        tp[i] = make_float2(-INFINITY, 0.0f);
        const int64_t y = t < p.N ? p.targets[t] : -1;
        ty[i] = y >= 0 && y < p.V ? (int)y : -1;
      }
    int acc = 0;
    uint32_t acc_phase = 0;
    // lane 0 waits for the accumulator and the warp follows its result (what comes is warp-collective)
    auto take = [&]() -> bool {
      int ok = 0;
      if (lane == 0) ok = wait(&tfull[acc], acc_phase) ? 1 : 0;
      ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
      if (!ok) {
        atomicOr(p.status, kStatusTimeout);
        *abort_flag = 1;
      }
      tc_fence_after();
      return ok != 0;
    };
    auto release = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) remote_arrive(tempty0 + 8 * acc);
      if (++acc == PL::kAcc) { acc = 0; acc_phase ^= 1u; }
    };
    for (int tile = first; tile < p.num_tiles; tile += step) {
      int mb, nb, kb0, kb1;
      const int part = pair_coords(tile, p, mb, nb, kb0, kb1);
      const int row0 = (2 * mb + rank) * half_rows + sub * 32, row = row0 + lane;
      const bool row_ok = row < p.M && sub * 32 + lane < half_rows, warp_ok = row0 < p.M && sub * 32 < half_rows;
      const uint32_t lanes = tmem_base + ((uint32_t)(sub * 32) << 16);
      if constexpr (MODE == kPairLse) {
        const int col0 = nb * NT + 128 * half;
        int y = -1;
        if (row_ok) {
          const int64_t t = p.targets[row];
          if (t >= 0 && t < p.V) y = (int)t;
        }
        float z[128];
#pragma unroll
        for (int j = 0; j < 128; ++j) z[j] = 0.0f;
        bool ok = true;
#pragma unroll 1
        for (int kb = kb0; kb < kb1; kb += kSegBlocks) {
          if (!(ok = take())) break;
          if (warp_ok)
#pragma unroll
            for (int c = 0; c < 8; ++c)
              ce_tmem_add16(lanes + (uint32_t)(acc * NT + 128 * half + 16 * c), z + 16 * c);
          release();
        }
        if (!ok) break;
        if (row_ok && col0 < p.N) {
          if ((unsigned)(y - col0) < 128u) {
            float zy = 0.0f;
#pragma unroll
            for (int j = 0; j < 128; ++j)
              if (y - col0 == j) zy = z[j];
            p.zy[row] = zy;
          }
          if (col0 + 128 > p.N)
#pragma unroll
            for (int j = 0; j < 128; ++j)
              if (col0 + j >= p.N) z[j] = -INFINITY;
          p.part[(int64_t)(2 * nb + half) * p.M + row] = ce_pair(z);
        }
        __syncwarp();
      } else if constexpr (MODE == kTokLse || MODE == kTokLogits) {
        float z[kBlocks][32];
#pragma unroll
        for (int i = 0; i < kBlocks; ++i)
#pragma unroll
          for (int j = 0; j < 32; ++j) z[i][j] = 0.0f;
        bool ok = true;
#pragma unroll 1
        for (int kb = kb0; kb < kb1; kb += kSegBlocks) {
          if (!(ok = take())) break;
#pragma unroll
          for (int i = 0; i < kBlocks; ++i) {
            const int c = half + 2 * i;
            if (32 * c >= NT || !warp_ok) continue;
            uint32_t a[32];  // lane: row of W, register: token
            tmem_ld32(lanes + (uint32_t)(acc * NT + 32 * c), a);
#pragma unroll
            for (int j = 0; j < 32; ++j) z[i][j] += __uint_as_float(a[j]);
          }
          release();
        }
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
          const int c = half + 2 * i;
          if (32 * c >= NT || 32 * c >= p.N || !warp_ok) continue;
          if constexpr (MODE == kTokLogits) {
            if (!row_ok) continue;
            float* dst = p.acc + ((int64_t)part * p.N + 32 * c) * p.M + row;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (32 * c + j < p.N) dst[(int64_t)j * p.M] = z[i][j];
            continue;
          }
          // element (row r, token j) at word 32 r + (r ^ j): rows and columns are both free of bank conflicts
          const uint32_t stage = out.buf;
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 32; ++j)
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(stage + 4 * (32 * lane + (lane ^ j))), "f"(row_ok ? z[i][j] : -INFINITY)
                         : "memory");
          __syncwarp();
#pragma unroll
          for (int r = 0; r < 32; ++r)
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(z[i][r]) : "r"(stage + 4 * (32 * r + (r ^ lane))) : "memory");
          const int at = ty[i] - row0;
          if ((unsigned)at < 32u && sub * 32 + at < half_rows) {
            float zy;
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(zy) : "r"(stage + 4 * (32 * at + (at ^ lane))) : "memory");
            p.zy[32 * c + lane] = zy;
          }
          tp[i] = ce_join2(tp[i], ce_pair(z[i]));
        }
      } else {
        float4 rw = make_float4(0.0f, 0.0f, __int_as_float(-1), 0.0f);  // kPairGrad
        if (MODE == kPairGrad && row_ok) rw = p.rows[row];
        if (!take()) break;
        if constexpr (kTok) {
#pragma unroll 1
          for (int i = 0; i < kBlocks; ++i) {
            const int c = half + 2 * i;
            if (32 * c >= NT || 32 * c >= p.N || !warp_ok) continue;
            __syncwarp();
            uint32_t a[32];
            tmem_ld32(lanes + (uint32_t)(acc * NT + 32 * c), a);  // lane: row of W (column of dX), register: token
            if (MODE == kTokGrad) {
              // G by token: 32 tokens x 32 rows of W, 64 bytes a token, and as much for what the rounding lost
              if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
              __syncwarp();
              const uint32_t hi = out.buf, lo = out.buf + 2048;
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                const float4 r = tok[32 * c + j];
                const int ry = __float_as_int(r.z);
                float q = ce_exp2(fmaf(__uint_as_float(a[j]), kLog2e, -r.x));
                if (ry == p.v0 + row) q -= 1.0f;
                q = ry >= 0 ? r.y * q : 0.0f;
                const __nv_bfloat16 g = __float2bfloat16_rn(q), e = __float2bfloat16_rn(q - __bfloat162float(g));
                asm volatile("st.shared.u16 [%0], %1;" ::"r"(hi + 64 * j + 2 * lane), "h"(__bfloat16_as_ushort(g)) : "memory");
                asm volatile("st.shared.u16 [%0], %1;" ::"r"(lo + 64 * j + 2 * lane), "h"(__bfloat16_as_ushort(e)) : "memory");
              }
              out.publish(&tmC, hi, row0, 32 * c);
              if (p.rows_lo) out.publish(&tmC, lo, row0, p.rows_lo + 32 * c);
            } else if (row_ok) {
              float* dst = p.acc + ((int64_t)part * p.N + 32 * c) * p.M + row;
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (32 * c + j < p.N) {
                  float* q = dst + (int64_t)j * p.M;
                  *q = p.out == kOutF32Add ? *q + __uint_as_float(a[j]) : __uint_as_float(a[j]);
                }
            }
          }
        } else {
          const int col0 = nb * NT + 128 * half;
          const int row_c = part * p.m_tiles * PM + row0;  // of C, whose parts of K lie one after another
          const uint32_t cols = lanes + (uint32_t)(acc * NT + 128 * half);
          if (MODE == kPairDw && p.out == kOutBf16) {
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
              const int col = col0 + c * 64;
              if (!warp_ok || col >= p.N) break;
              __syncwarp();
              uint32_t a[32], b[32];
              tmem_ld32x2(cols + c * 64, cols + c * 64 + 32, a, b);
              out.bf16_wide(&tmC, a, b, alpha, col, row_c);
            }
          } else {
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              const int col = col0 + c * 32;
              if (!warp_ok || col >= p.N) break;
              __syncwarp();
              uint32_t a[32];
              tmem_ld32(cols + c * 32, a);
              float v[32];
              if (MODE == kPairGrad) {
                const int y = __float_as_int(rw.z), yc = y - p.v0 - col;
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                  float q = ce_exp2(fmaf(__uint_as_float(a[j]), kLog2e, -rw.x));
                  if (j == yc) q -= 1.0f;
                  v[j] = y >= 0 ? rw.y * q : 0.0f;
                }
                out.bf16(&tmC, v, col, row0);
              } else if (MODE == kPairDx && p.out == kOutBf16Join) {
                const float* old = p.acc + (int64_t)row * p.N + col;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                  if (row_ok && col + 4 * q < p.N) o = *reinterpret_cast<const float4*>(old + 4 * q);
                  v[4 * q] = alpha * (__uint_as_float(a[4 * q]) + o.x);
                  v[4 * q + 1] = alpha * (__uint_as_float(a[4 * q + 1]) + o.y);
                  v[4 * q + 2] = alpha * (__uint_as_float(a[4 * q + 2]) + o.z);
                  v[4 * q + 3] = alpha * (__uint_as_float(a[4 * q + 3]) + o.w);
                }
                out.bf16(&tmC, v, col, row0);
              } else if (MODE == kPairDx && p.out == kOutBf16) {
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = alpha * __uint_as_float(a[j]);
                out.bf16(&tmC, v, col, row0);
              } else {
                out.f32(&tmC, a, alpha, col, row_c, p.out == kOutF32Add);
              }
            }
          }
        }
        release();
      }
    }
    if (MODE == kTokLse) {
      // the four warps that share a warpgroup's tokens bring their pairs together (the abort path has partial
      // ones: its results are incomplete anyway)
      __syncwarp();  // every lane has read its last block
#pragma unroll
      for (int i = 0; i < kBlocks; ++i)
        asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(out.buf + 8 * (32 * i + lane)), "f"(tp[i].x), "f"(tp[i].y) : "memory");
      if (half == 0) asm volatile("bar.sync 1, 128;" ::: "memory");
      else asm volatile("bar.sync 2, 128;" ::: "memory");
      if (sub == 0)
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
          const int c = half + 2 * i, t = 32 * c + lane;
          float2 r = make_float2(-INFINITY, 0.0f);
          for (int k = 0; k < 4; ++k) {
            float2 q;
            const uint32_t at = smem_addr(smem + PL::kStagingOffset + (4 * half + k) * PL::kStaging) + 8 * (32 * i + lane);
            asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(q.x), "=f"(q.y) : "r"(at) : "memory");
            r = ce_join2(r, q);
          }
          if (32 * c < NT && t < p.N) p.part[(int64_t)blockIdx.x * p.N + t] = r;
        }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }

  tc_fence_before();
  __syncwarp();
  __syncthreads();
  // Where any role of the CTA gave up, copies may be in flight, its producer's among them though that finished: no one waits
  // for their barriers any more.  (The other CTA's roles then run into their own limits, so both wait here.)
  if (*abort_flag) {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < kCopyDrainNs) {}
    __syncwarp();
  }
  cluster_sync_all();  // neither CTA's memory or barriers are in use by the other any more
  tc_fence_after();
  if (warp == 2) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(512) : "memory");
}

// ---------------------------------------------------------------------------
// The small kernels around it
// ---------------------------------------------------------------------------
// Joins the pieces of a row: 32 rows a block, lane = row, warp w takes pieces w, w + 32, ... four at a
// time; then the warps' pairs.  lse = ln 2 (m2 + log2 s).  A target outside [0, V) that is not ignore_index is a
// mistake of the caller: recorded, and ignored.
__global__ void __launch_bounds__(1024) k_ce_finish(const float2* __restrict__ part, int pieces, int64_t T,
                                                    const int64_t* __restrict__ targets, int64_t V, int64_t ignore,
                                                    const float* __restrict__ zy, float* __restrict__ loss,
                                                    float* __restrict__ lse, unsigned* status) {
  __shared__ float2 sh[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * 32 + lane;
  const float2 none = make_float2(-INFINITY, 0.0f);
  float2 r = none;
  wait_for_previous();
  start_dependents();
  if (t < T)
    for (int i = warp; i < pieces; i += 128) {
      float2 q[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) q[k] = i + 32 * k < pieces ? part[(int64_t)(i + 32 * k) * T + t] : none;
      r = ce_join2(r, ce_join2(ce_join2(q[0], q[1]), ce_join2(q[2], q[3])));
    }
  sh[warp][lane] = r;
  __syncthreads();
  // warp w joins row w of the block: a butterfly over the 32 warps' pairs
  r = sh[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float2 q = make_float2(__shfl_xor_sync(0xFFFFFFFFu, r.x, o), __shfl_xor_sync(0xFFFFFFFFu, r.y, o));
    r = (lane & o) ? ce_join2(q, r) : ce_join2(r, q);
  }
  const int64_t row = (int64_t)blockIdx.x * 32 + warp;
  if (lane != 0 || row >= T) return;
  const float l = kLn2 * (r.x + log2f(r.y));
  lse[row] = l;
  const int64_t y = targets[row];
  const bool in = y >= 0 && y < V;
  if (y != ignore && !in) atomicOr(status, kStatusBadTarget);
  loss[row] = y != ignore && in ? ce_loss(r, zy[row]) : 0.0f;
}

// Few tokens and a small vocabulary: the logits themselves, [splits][T][V] in fp32, one part of K each (tok_logit_splits).
__device__ __forceinline__ float ce_logit(const float* __restrict__ z, int splits, int64_t T, int64_t V, int64_t t, int64_t v) {
  float sum = 0.0f;
  for (int k = 0; k < splits; ++k) sum += z[(k * T + t) * V + v];
  return sum;
}
// Forward: a block a token.
__global__ void __launch_bounds__(1024) k_ce_logits_fwd(const float* __restrict__ z, int splits, int64_t T,
                                                        const int64_t* __restrict__ targets, int64_t V, int64_t ignore,
                                                        float* __restrict__ loss, float* __restrict__ lse, unsigned* status) {
  __shared__ float2 sh[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = blockIdx.x;
  wait_for_previous();
  start_dependents();
  float2 r = make_float2(-INFINITY, 0.0f);
  for (int64_t v0 = threadIdx.x; v0 < V; v0 += 8 * 1024) {
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = v0 + 1024 * i < V ? ce_logit(z, splits, T, V, t, v0 + 1024 * i) : -INFINITY;
    r = ce_join2(r, ce_pair(q));
  }
  auto join = [&]() {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float2 q = make_float2(__shfl_xor_sync(0xFFFFFFFFu, r.x, o), __shfl_xor_sync(0xFFFFFFFFu, r.y, o));
      r = (lane & o) ? ce_join2(q, r) : ce_join2(r, q);
    }
  };
  join();
  if (lane == 0) sh[warp] = r;
  __syncthreads();
  if (warp != 0) return;
  r = sh[lane];
  join();
  if (lane != 0) return;
  const float l = kLn2 * (r.x + log2f(r.y));
  lse[t] = l;
  const int64_t y = targets[t];
  const bool in = y >= 0 && y < V;
  if (y != ignore && !in) atomicOr(status, kStatusBadTarget);
  loss[t] = y != ignore && in ? ce_loss(r, ce_logit(z, splits, T, V, t, y)) : 0.0f;
}
// Backward: G / s in `copies` parts (rows T .. pad - 1 zero), as kTokGrad stores it.
__global__ void __launch_bounds__(256) k_ce_logits_grad(const float* __restrict__ z, int splits, int64_t T, int64_t V,
                                                        const float4* __restrict__ rows, uint16_t* __restrict__ G,
                                                        int64_t pitch, int64_t pad, int copies) {
  wait_for_previous();
  start_dependents();
  const int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x, t = blockIdx.y;
  if (v >= V) return;
  float q = 0.0f;
  if (t < T) {
    const float4 r = rows[t];
    const int y = __float_as_int(r.z);
    if (y >= 0) {
      q = ce_exp2(fmaf(ce_logit(z, splits, T, V, t, v), kLog2e, -r.x));
      if (y == v) q -= 1.0f;
      q *= r.y;
    }
  }
  const __nv_bfloat16 g = __float2bfloat16_rn(q);
  G[t * pitch + v] = __bfloat16_as_ushort(g);
  if (copies == 2) G[(pad + t) * pitch + v] = __bfloat16_as_ushort(__float2bfloat16_rn(q - __bfloat162float(g)));
}

// The largest |dloss| over the tokens that count (1 where that is 0 or not finite), valid in every thread.
__device__ __forceinline__ float ce_block_scale(const float* __restrict__ dloss, const int64_t* __restrict__ targets,
                                                int64_t T, int64_t V, int64_t ignore, unsigned* status, uint32_t* red) {
  uint32_t m = 0;
  bool bad = false;
#pragma unroll 8
  for (int64_t t = threadIdx.x; t < T; t += blockDim.x) {
    const int64_t y = targets[t];
    const uint32_t v = abs_bits(dloss[t]);
    const bool in = y >= 0 && y < V;
    if (y != ignore && in) m = max(m, v);
    bad |= y != ignore && !in;
  }
  if (bad) atomicOr(status, kStatusBadTarget);
  m = block_max_u32(m, red);
  return (m == 0 || m >= 0x7F800000u) ? 1.0f : __uint_as_float(m);
}
__global__ void __launch_bounds__(1024) k_ce_scale(const float* __restrict__ dloss, const int64_t* __restrict__ targets,
                                                   int64_t T, int64_t V, int64_t ignore, float* scale, unsigned* status) {
  __shared__ uint32_t red[32];
  start_dependents();
  const float s = ce_block_scale(dloss, targets, T, V, ignore, status, red);
  if (threadIdx.x == 0) *scale = s;
}

// Per token: {lse log2e, dloss / s, its target or -1 where it is ignored}, and x with ignored rows zeroed.
// OWN: every block finds s itself (up to kCeOwnScale tokens, which saves a launch), and block 0 stores it.
constexpr int64_t kCeOwnScale = 2048;
template <int OWN>
__global__ void __launch_bounds__(256) k_ce_rows(const uint16_t* __restrict__ x, const int64_t* __restrict__ targets,
                                                 const float* __restrict__ lse, const float* __restrict__ dloss, int64_t T,
                                                 int d, int64_t V, int64_t ignore, float* scale,
                                                 float4* __restrict__ rows, uint16_t* __restrict__ xz, int64_t pad, int copies,
                                                 unsigned* status) {
  __shared__ uint32_t red[32];
  if (!OWN) wait_for_previous();
  start_dependents();
  float s;
  if (OWN) {
    s = ce_block_scale(dloss, targets, T, V, ignore, status, red);
    if (blockIdx.x == 0 && threadIdx.x == 0) *scale = s;
  } else {
    s = *scale;
  }
  // rows T .. pad - 1 are zero; `copies` copies of the pad rows
  for (int64_t t = blockIdx.x; t < pad; t += gridDim.x) {
    const int64_t y = t < T ? targets[t] : ignore;
    const bool keep = y != ignore && y >= 0 && y < V;
    if (threadIdx.x == 0 && t < T)
      rows[t] = make_float4(lse[t] * kLog2e, keep ? dloss[t] / s : 0.0f, __int_as_float(keep ? (int)y : -1), 0.0f);
    for (int j = 8 * threadIdx.x; j < d; j += 8 * blockDim.x) {
      const uint4 v = keep ? ld_v4(x + t * d + j) : make_uint4(0, 0, 0, 0);
      for (int c = 0; c < copies; ++c) st_v4(xz + (c * pad + t) * d + j, v);
    }
  }
}

// out = s (sum of the parts of K), part i at rows i `rows_pad` of part; N a multiple of 8.
__global__ void __launch_bounds__(256) k_ce_join(const float* __restrict__ part, int splits, int64_t rows_pad, int64_t M,
                                                 int N, const float* __restrict__ scale, void* out, int f32) {
  wait_for_previous();
  start_dependents();
  const int64_t n4 = M * N / 4, stride = rows_pad * N / 4;
  const float alpha = *scale;
  const float4* p = reinterpret_cast<const float4*>(part);
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n4; i += (int64_t)gridDim.x * blockDim.x) {
    float4 s = p[i];
#pragma unroll 4
    for (int k = 1; k < splits; ++k) {
      const float4 q = p[k * stride + i];
      s.x += q.x; s.y += q.y; s.z += q.z; s.w += q.w;
    }
    s.x *= alpha; s.y *= alpha; s.z *= alpha; s.w *= alpha;
    if (f32) reinterpret_cast<float4*>(out)[i] = s;
    else reinterpret_cast<uint2*>(out)[i] = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
  }
}

cudaError_t launched(const Launch& L) {
  if (L.launches) ++*L.launches;
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encode_fn() {
  static EncodeFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(ptr);
  });
  return fn;
}
bool make_map(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t ld, int es, int box_cols, int box_rows,
              CUtensorMapSwizzle sw) {
  EncodeFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(ld * es)};
  const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
  const cuuint32_t one[2] = {1, 1};
  return enc(m, es == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base),
             dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// op(A) [M, K] op(B) [N, K]^T: a K-major operand is stored [M or N, K], an MN-major one [K, M or N].
struct PairProblem {
  int64_t M, N, K;
  const void* A;
  int64_t lda;
  const void* B;
  int64_t ldb;
  void* C;
  int64_t ldc;
};

// The M tiles of a rasterisation group: every one of them while A fits in L2 beside the streamed B, one
// (N fastest) while B does instead, else 4096 rows (the forward at T = 8192, d = 3584, V = 32000, back to back: 1146 us with
// 1024 rows, 1094 with 2048, 1068 with 4096, 1082 with 8192; the backward 3484, 3398, 3398, 3540).
int pair_group(const PairProblem& q, int m_tiles) {
  constexpr int64_t kResident = 48ll << 20;
  const int64_t a = 2 * q.M * q.K, b = 2 * q.N * q.K;
  if (a <= b && a <= kResident) return m_tiles;
  if (b < a && b <= kResident) return 1;
  return 4096 / PM;
}

constexpr int kPlanPairs = 76;
int pair_grid(const Launch& L, int64_t tiles) {
  const int most = L.num_sms / 2 < kPlanPairs ? L.num_sms / 2 : kPlanPairs;
  return tiles < most ? (int)tiles : most;
}

// Parts of K for a product with few tiles.  A block of 64 of K takes a pair about 0.33 us (25 TFLOP/s), a
// tile's fill and epilogue about 2 us, and joining the parts a launch (3 us) and a read and a write of each
// part at about 6 TB/s; the tiles run in waves of one per pair.  E.g. T = 1003, d = 2048, V = 50257: dX has 32 tiles
// for 76 pairs, 245 us in one part.
int pair_splits(int64_t M, int64_t N, int64_t K) {
  const int64_t m_pad = (M + PM - 1) / PM * PM, tiles = m_pad / PM * ((N + PN - 1) / PN), kb = (K + PK - 1) / PK;
  if (tiles >= 4 * kPlanPairs) return 1;
  int best = 1;
  double least = 0.0;
  for (int s = 1; s <= 32 && s <= kb; ++s) {
    const int64_t each = (kb + s - 1) / s;
    if ((kb + each - 1) / each != s) continue;  // fewer parts hold the same blocks
    if (s > 1 && s * m_pad * N * 4 > (256ll << 20)) break;
    const double waves = (double)((tiles * s + kPlanPairs - 1) / kPlanPairs);
    const double us = waves * (0.33 * (double)each + 2.0) + (s > 1 ? 3.0 + (double)(s * M * N) * 8.0 / 6e6 : 0.0);
    if (s == 1 || us < least) { best = s; least = us; }
  }
  return best;
}

// Rows of W in each half of a tile of the forward of few tokens, a multiple of 8 up to 128: as many tiles as the pairs take
// in the waves of full ones, so that all pairs stream for the same time (T = 24 and 120, d = 4096, V = 100000, 391 full
// tiles: 153 -> 143 and 158 -> 148 us, with K in parts of 1024; nothing is gained where one wave holds them, nor in the backward's logits, which
// write G).  The MMAs work on 128 rows all the same: what the stage held beyond makes sums that are not read back.
int tok_half_rows(int64_t V, const Launch& L) {
  const int64_t pairs = pair_grid(L, 0x7FFFFFFF), waves = ((V + PM - 1) / PM + pairs - 1) / pairs;
  if (waves == 1) return PM / 2;
  return (int)(((V + 2 * pairs * waves - 1) / (2 * pairs * waves) + 7) / 8 * 8);
}

// Parts of K for the logits of few tokens, stored in fp32 and joined by another kernel; 0: in one launch (kTokLse, kTokGrad).
// A block of 64 of K takes a pair 0.25 us whatever the tokens and rows (an MMA of 256 rows takes as long for 32 columns as for
// 256), so where a small vocabulary has few tiles for the pairs, the pairs share K, in one wave.  The parts are of at
// most 1024 of K, each summed in parts of 128 as above.  T = 5, d = 4656, V = 2476, forward 29 -> 21 us and backward 49 -> 39; T = 2, d = 4080, V = 1686
// 27 -> 20 and 45 -> 33; T = 60, d = 3584, V = 4000 26 -> 22 and 49 -> 42 (in three waves T = 1, d = 5120, V = 9000 took 41 for 36).
int tok_logit_splits(int64_t T, int64_t d, int64_t V) {
  const int64_t tiles = (V + PM - 1) / PM, kb = (d + PK - 1) / PK;
  if (T > kTokMax) return 0;
  int best = 0;
  double least = 0.25 * (double)kb - 2.0;  // one launch; the parts cost the backward a launch more
  for (int64_t s = (kb + kPartBlocks - 1) / kPartBlocks; s <= kb && s <= 64 && tiles * s <= kPlanPairs; ++s) {
    const int64_t each = (kb + s - 1) / s;
    if (s < 2 || (kb + each - 1) / each != s) continue;
    if (s * T * V * 4 > (32ll << 20)) break;
    const double us = 0.25 * (double)each + 2.0 + (double)(s * T * V) * 8.0 / 3e6;
    if (us < least) { best = (int)s; least = us; }
  }
  return best;
}

template <int A_MN, int B_MN, int MODE, int NT, int SHORT>
cudaError_t launch_pair_kernel(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tc, const PairArgs& a,
                               const Launch& L, bool dependent) {
  auto* k = k_ce_gemm<A_MN, B_MN, MODE, NT, SHORT>;
  constexpr int kSmem = PairPlan<MODE, NT>::kSmem;
  static std::atomic<uint64_t> configured{0};  // a bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(configured.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    configured.fetch_or(1ull << dev);
  }
  const int pairs = pair_grid(L, a.num_tiles);
  if (!dependent) {  // comes first in its call
    k<<<2 * pairs, kPairThreads, kSmem, L.stream>>>(ta, tb, tc, a);
    e = cudaGetLastError();
  } else {
    e = launch_dependent(k, 2 * pairs, kPairThreads, kSmem, L.stream, ta, tb, tc, a);
  }
  if (L.launches) ++*L.launches;
  return e;
}

template <int A_MN, int B_MN, int MODE, int NT = 256>
cudaError_t launch_pair(const PairProblem& q, int splits, PairArgs a, const Launch& L, bool dependent = true) {
  constexpr bool kTok = MODE >= kTokLse;
  a.M = (int)q.M;
  a.N = (int)q.N;
  a.K = (int)q.K;
  a.half_rows = MODE == kTokLse ? tok_half_rows(q.M, L) : PM / 2;
  a.m_tiles = (int)((q.M + 2 * a.half_rows - 1) / (2 * a.half_rows));
  a.n_tiles = (a.N + NT - 1) / NT;
  a.k_blocks = (a.K + PK - 1) / PK;
  if ((int64_t)a.m_tiles * a.n_tiles * splits > 0x7FFFFFFF) return cudaErrorInvalidValue;
  // a shorter last piece of the vocabulary may need fewer parts; the others then get nothing added
  a.split_blocks = (a.k_blocks + splits - 1) / splits;
  a.splits = (a.k_blocks + a.split_blocks - 1) / a.split_blocks;
  a.num_tiles = a.m_tiles * a.n_tiles * a.splits;
  a.group = kTok ? a.m_tiles : pair_group(q, a.m_tiles);
  if (a.group > a.m_tiles) a.group = a.m_tiles;
  a.by_part = divisor(a.m_tiles * a.n_tiles);
  a.by_span = divisor(a.group * a.n_tiles);
  a.by_group = divisor(a.group);
  a.by_last = divisor(a.m_tiles % a.group ? a.m_tiles % a.group : a.group);
  // fp32 sums, bf16 operands and their majors, N / 8 and M / 16 of the pair's tile
  a.idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)A_MN << 15) | ((uint32_t)B_MN << 16) |
            ((uint32_t)(NT >> 3) << 17) | ((uint32_t)(PM >> 4) << 24);
  a.status = L.status;
  a.wait_ns = L.wait_ns;
  CUtensorMap ta, tb, tc;
  bool ok = A_MN ? make_map(&ta, q.A, q.M, q.K, q.lda, 2, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B)
                 : make_map(&ta, q.A, q.K, q.M, q.lda, 2, 64, a.half_rows, CU_TENSOR_MAP_SWIZZLE_128B);
  ok = ok && (B_MN ? make_map(&tb, q.B, q.N, q.K, q.ldb, 2, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B)
                   : make_map(&tb, q.B, q.K, q.N, q.ldb, 2, 64, NT / 2, CU_TENSOR_MAP_SWIZZLE_128B));
  tc = ta;
  if (MODE == kTokGrad) {  // by token: [2 Tp, M] or [N, M]
    ok = ok && make_map(&tc, q.C, q.M, a.rows_lo ? 2 * a.rows_lo : q.N, q.ldc, 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_NONE);
  } else if (!kTok && MODE != kPairLse) {
    const bool f32 = MODE != kPairGrad && (a.out == kOutF32Store || a.out == kOutF32Add);
    const bool wide = MODE == kPairDw && !f32;  // rows of 128 bytes, as fp32's
    ok = ok && make_map(&tc, q.C, q.N, splits > 1 ? (int64_t)splits * a.m_tiles * PM : q.M, q.ldc, f32 ? 4 : 2,
                        wide ? 64 : 32, 32, f32 || wide ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
  }
  if (!ok) return cudaErrorInvalidValue;
  if (a.wait_ns) return launch_pair_kernel<A_MN, B_MN, MODE, NT, 1>(ta, tb, tc, a, L, dependent);
  return launch_pair_kernel<A_MN, B_MN, MODE, NT, 0>(ta, tb, tc, a, L, dependent);
}

// Rows of G: its two parts of whole blocks of 32 tokens, or T.
int64_t ce_g_rows(int64_t T) { return T <= kTwoParts ? 2 * ((T + 31) / 32 * 32) : T; }
// Columns of a backward piece: all rows of G in about 256 MB (more than 131072 of them: 1024 columns), in whole tiles, the
// pieces alike.
int64_t ce_piece(int64_t T, int64_t V) {
  constexpr int64_t kPieceBytes = 256ll << 20;
  int64_t most = kPieceBytes / (2 * ce_g_rows(T)) / PN * PN;
  if (most < 4 * PN) most = 4 * PN;
  const int64_t n = (V + most - 1) / most;
  return ((V + n - 1) / n + PN - 1) / PN * PN;
}

// The backward's plan: the piece, and the parts of K of its two products.
struct CePlan {
  int64_t piece;
  int dx_splits, dw_splits;
  int z_splits;  // of the logits' K, or 0
};
CePlan ce_plan(int64_t T, int64_t d, int64_t V) {
  CePlan p{};
  p.piece = ce_piece(T, V);
  const int64_t n = p.piece < V ? p.piece : V;
  p.dx_splits = T <= kTokMax ? pair_splits(d, ce_g_rows(T), n) : pair_splits(T, d, n);
  p.dw_splits = pair_splits(n, d, ce_g_rows(T));
  p.z_splits = n == V ? tok_logit_splits(T, d, V) : 0;
  return p;
}

struct CeWs {
  float2* part;
  float4* rows;
  float *zy, *acc, *dw_part, *scale, *z;
  uint16_t *G, *xz;
};
size_t ce_layout(int64_t T, int64_t d, int64_t V, bool bwd, uint8_t* base, CeWs* w) {
  size_t off = 0;
  auto take = [&](int64_t bytes) {
    uint8_t* p = base + off;
    off += ((size_t)bytes + 255) & ~size_t(255);
    return p;
  };
  CeWs t{};
  if (bwd) {
    const CePlan p = ce_plan(T, d, V);
    const int64_t g_rows = ce_g_rows(T);
    t.G = (uint16_t*)take(g_rows * p.piece * 2);
    t.xz = (uint16_t*)take(g_rows * d * 2);
    const int64_t m_pad = (T + PM - 1) / PM * PM;
    if (T <= kTokMax) t.acc = (float*)take(p.dx_splits * g_rows * d * 4);
    else if (p.dx_splits > 1) t.acc = (float*)take(p.dx_splits * m_pad * d * 4);
    else if (p.piece < V) t.acc = (float*)take(T * d * 4);
    if (p.dw_splits > 1) t.dw_part = (float*)take(p.dw_splits * p.piece * d * 4);
    t.rows = (float4*)take(T * 16);
    t.scale = (float*)take(4);
    if (p.z_splits) t.z = (float*)take(p.z_splits * T * V * 4);
  } else if (const int z_splits = tok_logit_splits(T, d, V)) {
    t.z = (float*)take(z_splits * T * V * 4);
  } else {
    t.part = (float2*)take(T <= kTokMax ? 2 * kPlanPairs * T * 8 : 2 * ((V + PN - 1) / PN) * T * 8);
    t.zy = (float*)take(T * 4);
  }
  if (w) *w = t;
  return off;
}

// The logits of few tokens, in parts of K.
cudaError_t launch_tok_logits(const uint16_t* x, const uint16_t* W, int64_t T, int64_t d, int64_t V, int splits, float* z,
                              const Launch& L, bool dependent) {
  const PairProblem q{V, T, d, W, d, x, d, nullptr, 0};
  PairArgs a{};
  a.acc = z;
  return T <= 32   ? launch_pair<0, 0, kTokLogits, 32>(q, splits, a, L, dependent)
         : T <= 64 ? launch_pair<0, 0, kTokLogits, 64>(q, splits, a, L, dependent)
                   : launch_pair<0, 0, kTokLogits, 128>(q, splits, a, L, dependent);
}

}  // namespace

size_t ce_workspace_bytes(int64_t T, int64_t d, int64_t V, int bwd) { return ce_layout(T, d, V, bwd != 0, nullptr, nullptr); }

cudaError_t launch_ce_fwd(const uint16_t* x, const uint16_t* W, const int64_t* targets, int64_t T, int d, int64_t V,
                          int64_t ignore, float* loss, float* lse, void* ws, const Launch& L) {
  CeWs w;
  ce_layout(T, d, V, false, static_cast<uint8_t*>(ws), &w);
  cudaError_t e;
  if (const int splits = tok_logit_splits(T, d, V)) {
    if ((e = launch_tok_logits(x, W, T, d, V, splits, w.z, L, false)) != cudaSuccess) return e;
    e = launch_dependent(k_ce_logits_fwd, (unsigned)T, 1024, 0, L.stream, w.z, splits, T, targets, V, ignore, loss, lse, L.status);
    if (L.launches) ++*L.launches;
    return e;
  }
  PairArgs a{};
  a.targets = targets;
  a.V = (int)V;
  a.part = w.part;
  a.zy = w.zy;
  int pieces;
  if (T <= kTokMax) {
    const PairProblem q{V, T, d, W, d, x, d, nullptr, 0};
    e = T <= 32 ? launch_pair<0, 0, kTokLse, 32>(q, 1, a, L, false)
        : T <= 64 ? launch_pair<0, 0, kTokLse, 64>(q, 1, a, L, false) : launch_pair<0, 0, kTokLse, 128>(q, 1, a, L, false);
    const int half = tok_half_rows(V, L);
    pieces = 2 * pair_grid(L, (V + 2 * half - 1) / (2 * half));
  } else {
    e = launch_pair<0, 0, kPairLse>(PairProblem{T, V, d, x, d, W, d, nullptr, 0}, 1, a, L, false);
    pieces = (int)((V + 127) / 128);
  }
  if (e != cudaSuccess) return e;
  e = launch_dependent(k_ce_finish, (unsigned)((T + 31) / 32), 1024, 0, L.stream, w.part, pieces, T, targets, V, ignore,
                       w.zy, loss, lse, L.status);
  if (L.launches) ++*L.launches;
  return e;
}

cudaError_t launch_ce_bwd(const uint16_t* x, const uint16_t* W, const int64_t* targets, const float* lse,
                          const float* dloss, int64_t T, int d, int64_t V, int64_t ignore, uint16_t* dX, void* dW,
                          int dw_f32, void* ws, const Launch& L) {
  CeWs w;
  ce_layout(T, d, V, true, static_cast<uint8_t*>(ws), &w);
  const CePlan plan = ce_plan(T, d, V);
  const int64_t piece = plan.piece;
  const int join_blocks = 4 * L.num_sms;
  cudaError_t e;
  const int64_t g_rows = ce_g_rows(T);
  const int copies = T <= kTwoParts ? 2 : 1;
  const int64_t pad = g_rows / copies;
  const unsigned row_blocks = (unsigned)(pad < 8 * L.num_sms ? pad : 8 * L.num_sms);
  if (T <= kCeOwnScale) {
    k_ce_rows<1><<<row_blocks, 256, 0, L.stream>>>(x, targets, lse, dloss, T, d, V, ignore, w.scale, w.rows, w.xz, pad, copies,
                                                   L.status);
  } else {
    k_ce_scale<<<1, 1024, 0, L.stream>>>(dloss, targets, T, V, ignore, w.scale, L.status);
    if ((e = launched(L)) != cudaSuccess) return e;
    e = launch_dependent(k_ce_rows<0>, row_blocks, 256, 0, L.stream, x, targets, lse, dloss, T, d, V, ignore, w.scale, w.rows,
                         w.xz, pad, copies, L.status);
    if (e != cudaSuccess) return e;
  }
  if ((e = launched(L)) != cudaSuccess) return e;
  for (int64_t v0 = 0; v0 < V; v0 += piece) {
    const int64_t n = V - v0 < piece ? V - v0 : piece;
    const bool first = v0 == 0, last = v0 + n == V;
    PairArgs a{}, ax{};
    a.v0 = (int)v0;
    a.rows = w.rows;
    ax.acc = w.acc;
    const int xs = plan.dx_splits;
    if (T <= kTokMax) {
      const PairProblem q{n, T, d, W + v0 * d, d, x, d, w.G, piece};
      const PairProblem qx{d, g_rows, n, W + v0 * d, d, w.G, piece, nullptr, 0};
      a.rows_lo = copies == 2 ? (int)pad : 0;
      ax.out = first ? kOutF32Store : kOutF32Add;
      if (plan.z_splits) {
        if ((e = launch_tok_logits(x, W, T, d, V, plan.z_splits, w.z, L, true)) != cudaSuccess) return e;
        e = launch_dependent(k_ce_logits_grad, dim3((unsigned)((V + 255) / 256), (unsigned)pad), 256, 0, L.stream, w.z,
                             plan.z_splits, T, V, w.rows, w.G, piece, pad, copies);
        if (L.launches) ++*L.launches;
      } else {
        e = T <= 32   ? launch_pair<0, 0, kTokGrad, 32>(q, 1, a, L)
            : T <= 64 ? launch_pair<0, 0, kTokGrad, 64>(q, 1, a, L) : launch_pair<0, 0, kTokGrad, 128>(q, 1, a, L);
      }
      if (e != cudaSuccess) return e;
      e = T <= 32 ? launch_pair<1, 0, kTokDx, 64>(qx, xs, ax, L) : launch_pair<1, 0, kTokDx, 128>(qx, xs, ax, L);
      if (e != cudaSuccess) return e;
    } else {
      e = launch_pair<0, 0, kPairGrad>(PairProblem{T, n, d, x, d, W + v0 * d, d, w.G, piece}, 1, a, L);
      if (e != cudaSuccess) return e;
      // dX (+)= G W[piece]: the sum so far stays in fp32 (its parts of K apart), s joins it at the end
      ax.out = xs > 1 || !last ? (first ? kOutF32Store : kOutF32Add) : (first ? kOutBf16 : kOutBf16Join);
      if (xs == 1 && last) ax.scale = w.scale;
      void* to = xs > 1 || !last ? (void*)w.acc : (void*)dX;
      e = launch_pair<0, 1, kPairDx>(PairProblem{T, d, n, w.G, piece, W + v0 * d, d, to, d}, xs, ax, L);
      if (e != cudaSuccess) return e;
    }
    if (last && (xs > 1 || T <= kTokMax)) {
      const bool few = T <= kTokMax;
      e = launch_dependent(k_ce_join, join_blocks, 256, 0, L.stream, w.acc, few ? copies * xs : xs,
                           few ? pad : (T + PM - 1) / PM * PM, T, d, w.scale, dX, 0);
      if (e == cudaSuccess) e = launched(L);
      if (e != cudaSuccess) return e;
    }
    // dW[piece] = s G^T x
    PairArgs aw{};
    const int wsp = plan.dw_splits;
    if (wsp == 1) aw.scale = w.scale;
    aw.out = wsp > 1 || dw_f32 ? kOutF32Store : kOutBf16;
    void* dst = dw_f32 ? (void*)(static_cast<float*>(dW) + v0 * d) : (void*)(static_cast<uint16_t*>(dW) + v0 * d);
    e = launch_pair<1, 1, kPairDw>(PairProblem{n, d, g_rows, w.G, piece, w.xz, d, wsp > 1 ? (void*)w.dw_part : dst, d}, wsp, aw, L);
    if (e != cudaSuccess) return e;
    if (wsp > 1) {
      e = launch_dependent(k_ce_join, join_blocks, 256, 0, L.stream, w.dw_part, wsp, (n + PM - 1) / PM * PM, n, d, w.scale, dst, dw_f32);
      if (e == cudaSuccess) e = launched(L);
      if (e != cudaSuccess) return e;
    }
  }
  return cudaSuccess;
}

}  // namespace fp8q
