// Causal attention over the 8-bit key/value cache for many rows a sequence (pieces of prompts): on the 5th-generation tensor
// cores, bound by the chain of a tile's products and exponentials.  Two pieces of 512 tokens of 40 + 8 heads of 128 over 8192 and 6471: 192 us
// with the join, 771 TFLOP/s; the tensor pipe is active for 35 % of it, a block of 128 keys takes about 4500 cycles, whether the tiles' rows exist or
// not.  (Below: "2 x 512 over 8192"; other sizes are the largest of a batch, too.  Times of variants that were tried are beside that of the
// kernel as it then was.)
//
// The products are tcgen05 kind::f16 ones, fp16 operands and fp32 accumulators in tensor memory: FP8 codes are fp16 numbers, and q is
// one over a power of two of its row, so the scores lose nothing.  (FP8 operands would need q and P in several 4-bit parts.)
// A CTA has 256 rows of one K/V head, two tiles of 128 (token, query head) pairs, A and B, which share what is
// made of each block of 128 keys; its 16 warps (two have no work: a warp's number modulo 4 says which quarter of tensor memory's lanes it reads):
//   warp 5       pages, bulk copies of a block's codes of K and V into shared memory, and its scales, a block ahead;
//   warps 0-3    K's codes into a swizzled fp16 tile, then V's.  (V's by two warps of its own made two of an SM's four schedulers, and
//                the rows that run there, the last: 2 x 512 tokens over 8192 take 184 us either way, 64 x 104 over 1000 325 and 301);
//   warp 4       the products, one thread: O_A += P_A V of the block before, S_A = Q_A K^T, then B's;
//   warps 8-15   a row a thread (A, then B): q into shared memory; per block the row's maximum from S, P = 2^(s - m) as fp16
//                in tensor memory, and at the end O over the sum.
// P lies over S: S and O fill tensor memory, so a tile's S waits for its P V; meanwhile the other tile's rows work.  P in shared memory, and S a
// block ahead, was slower (195 us against 185 for 2 x 512 tokens over 8192): shared memory carries the products' operands (Q and K alone
// its full width while S is made), the codes and what is made of them.  Products with different accumulators may run in another order than
// they were issued in, so S over P waits for the product that reads P (1 to 2 % at head_dim 96 and 128); at head_dim 64 P lies beside O, which
// has half of its columns to spare, and nothing waits (1 % faster than over S).
// P's window is that of the few rows' kernel: p 2^11 in fp16, the reference maximum moving when it is exceeded by 2^4, and V's scales
// relative to the largest that the row has seen so far.  Both are a row's own: what it does not see does not move a bit of it.  (One reference for
// all rows of a unit's part, known before its first block, took 186 us where this takes 189, and scores of any size 191.)
// The keys of all (sequence, row tile, K/V head) units are cut into equal parts, one a CTA, as there.
//
// Every mbarrier wait is bounded; on expiry the CTA records FP8Q_STATUS_TIMEOUT, stops issuing, waits for the products and copies that it
// issued, whichever role gave up, frees tensor memory and exits.
#include <type_traits>

#include "fp8q_kvline.cuh"

namespace fp8q {

namespace {

constexpr int kConvertThreads = 128, kMmaWarp = 4, kCopyWarp = 5, kFirstRowWarp = 8, kThreads = 512;
constexpr int kTileRows = 128, kRows = 2 * kTileRows;
constexpr int kAtom = 16384;       // 128 rows x 128 bytes: 64 fp16 columns of a swizzled tile
constexpr int kTile = 2 * kAtom;   // a tile of 128 columns
constexpr int kQ = 0;              // [2 tiles]
constexpr int kK = kQ + 2 * kTile;
constexpr int kV = kK + kTile;
constexpr int kCodes = kV + kTile; // the next block's codes: K, V
constexpr int kBars = kCodes + kTile;
constexpr int kMisc = kBars + 256;
constexpr float kOffset = 11.0f, kSlack = 4.0f;
constexpr int kNothing = -45;      // V's exponent over the reference, at least: nothing is left of 2^(11 + 4 - 45) in fp16
constexpr int kAll = 0x7FFFFFFF;
// What a unit costs besides its keys, in blocks: q, the first pages, the results.  (2 x 512 tokens of 40 heads over 8192: 197, 195, 193, 192
// and 193 us with 3, 5, 7, 10 and 14; 16 x 104 over 4096: 217, 209, 193, 195, 199; 16 x 16: 77, 73, 74, 78, 85.)
constexpr int kUnitCost = 7;

// A block's scales as the rows need them, 16 keys each: 2^X of K; X of V, and dx, 2^-dx, its exponent over the block's largest.
struct BlockScales {
  float k[8], dx[8], back[8];
  int v[8];  // -1000: no page
  int none;  // bit g: keys 16 g .. have no page
  int vmax;  // the largest of v
};
// What is to be seen of a block's codes.
struct BlockKeys {
  int rows;   // keys that some row sees: 128 but in the last block
  int have;   // bit g: keys 16 g .. have a page
  int check;  // some row does not see all of them: V is looked at for what is not finite
};
struct Misc {
  BlockScales scales[2];  // by block
  BlockKeys keys[4];      // by block
  int odd;                // some V was NaN or infinite, and is 0 in its tile
  uint32_t tmem;
  int abort;
};
constexpr int kSmem = kMisc + (int)sizeof(Misc) + 1024;
static_assert(kSmem <= 232448, "shared memory per CTA");

__host__ __device__ constexpr uint32_t idesc_f16(int n, int b_mn) {
  return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}
// D[tmem] (+)= A[tmem] B[shared], fp16 operands.
__device__ __forceinline__ void umma_f16_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// S = Q K^T over DH: both K-major tiles of 128 rows.
template <int DH>
__device__ __forceinline__ void mma_scores(uint32_t d, uint32_t a, uint32_t b) {
#pragma unroll
  for (int i = 0; i < DH / 16; ++i) {
    const uint32_t off = (uint32_t)((i >> 2) * kAtom + (i & 3) * 32);
    umma_bf16(d, smem_desc_sw128(a + off, 16, 1024), smem_desc_sw128(b + off, 16, 1024), idesc_f16(128, 0), i ? 1u : 0u);
  }
}
// O (+)= P V over 128 keys: P in tensor memory, V MN-major (a row a key), N = 64 or 128 columns.
template <int N>
__device__ __forceinline__ void mma_values(uint32_t d, uint32_t a, uint32_t b, bool accumulate) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    umma_f16_ts(d, a + i * 8, smem_desc_sw128(b + i * 2048, kAtom, 1024), idesc_f16(N, 1), (accumulate || i) ? 1u : 0u);
}
// SHORT: the self-test's waits, which poll and give up after limit_ns (a kernel of its own: the choice at every wait cost a tenth).
template <bool SHORT>
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
  return SHORT ? mbar_poll(bar, parity, abort, limit_ns) : mbar_wait(bar, parity, abort);
}
template <bool SHORT>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
  return __all_sync(0xFFFFFFFFu, wait<SHORT>(bar, parity, abort, limit_ns)) != 0;
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// 16-byte piece j (8 fp16) of row r of a swizzled tile.
__device__ __forceinline__ uint32_t piece(uint32_t tile, int r, int j) {
  return tile + (uint32_t)((j >> 3) * kAtom + r * 128 + (((j ^ r) & 7) << 4));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};\n\t"
      "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
      "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A sequence's units: row tile by row tile, each for every K/V head.
struct Tiles {
  int pairs, before, G;  // (token, head) pairs; tokens before the call's; query heads of a K/V head
  uint32_t inv;          // 2^32 / G, rounded up: r inv / 2^32 is r / G for r below 2^22 (G at most 1024)
  __device__ __forceinline__ int token(int r) const { return G == 1 ? r : r < 1 << 22 ? (int)__umulhi((uint32_t)r, inv) : r / G; }
  __device__ __forceinline__ int count() const { return (int)((pairs + (int64_t)(kRows - 1)) / kRows); }
  __device__ __forceinline__ int rows(int rt) const { return min(kRows, pairs - rt * kRows); }
  // the keys that pair r sees
  __device__ __forceinline__ int limit(int r) const { return max(0, before + token(r) + 1); }
  __device__ __forceinline__ int blocks(int rt) const { return (limit(rt * kRows + rows(rt) - 1) + kBlockKeys - 1) / kBlockKeys; }
  __device__ __forceinline__ int cost(int rt) const {
    const int nb = blocks(rt);
    return nb ? nb + kUnitCost : 1;
  }
};
__device__ __forceinline__ Tiles tiles_of(const AttendArgs& p, const KvSeq& q) {
  const int G = p.n_heads / p.kv.hkv;
  return Tiles{q.n * G, q.len - q.n, G, 0xFFFFFFFFu / (uint32_t)G + 1u};
}
__device__ __forceinline__ int64_t seq_cost(const AttendArgs& p, const KvSeq& q) {
  const Tiles t = tiles_of(p, q);
  int64_t sum = 0;
  for (int rt = 0; rt < t.count(); ++rt) sum += t.cost(rt);
  return sum * p.kv.hkv;
}

// One part of the line after the other: what all roles walk through alike.  next() is a function of its own, and a Walk lies in
// local memory: inlined into every role, its code and its registers were in the way of the loops over the blocks.
struct Walk {
  const AttendArgs* p;
  int s, rt;       // sequence, row tile
  KvSeq q;
  Tiles t;
  int64_t base;    // first block of the row tile's units
  int64_t at, end;
  // of the segment
  int h, r0, n_rows, nb, b0, b1;
  int64_t unit0, cost;
  __device__ __noinline__ bool next() {
    const KvArgs& kv = p->kv;
    while (at < end) {
      if (rt >= t.count()) {
        if (++s >= kv.n_seqs) return false;
        q = kv_seq(kv, s);
        t = tiles_of(*p, q);
        rt = 0;
        continue;
      }
      const int c = t.cost(rt);
      const int64_t here = (int64_t)c * kv.hkv;
      if (at >= base + here) {
        base += here;
        ++rt;
        continue;
      }
      h = here < (int64_t)1 << 32 ? (int)((uint32_t)(at - base) / (uint32_t)c) : (int)((at - base) / c);
      const int v0 = (int)((at - base) - (int64_t)h * c), v1 = (int)min((int64_t)c, v0 + (end - at));
      unit0 = base + (int64_t)h * c;
      cost = c;
      nb = t.blocks(rt);
      at += v1 - v0;
      b0 = max(0, v0 - kUnitCost);
      b1 = min(nb, max(0, v1 - kUnitCost));
      if (b0 == b1 && nb) continue;
      r0 = rt * kRows;
      n_rows = t.rows(rt);
      return true;
    }
    return false;
  }
  // blocks of this segment that tile `side` sees
  __device__ __forceinline__ int blocks_of(int side) const {
    const int rows = min(kTileRows, n_rows - side * kTileRows);
    if (rows <= 0) return 0;
    return max(0, min(b1, (t.limit(r0 + side * kTileRows + rows - 1) + kBlockKeys - 1) / kBlockKeys) - b0);
  }
};

// What a row's scores of keys 16 g .. of a block are multiplied by.
__device__ __forceinline__ float factor_of(float rowf, const BlockScales& sc, int g) {
  return fminf(fmaxf(rowf * sc.k[g], 0x1p-100f), 0x1p126f);
}
// Where a row's scores are large: this thread's row of S becomes the differences from its reference m, over what they are multiplied by later.
__device__ __noinline__ void take_reference(uint32_t tS, const BlockScales& sc, float rowf, float m) {
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t z[32];
    tmem_ld32(tS + c * 32, z);
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const float f = factor_of(rowf, sc, 2 * c + (k >> 4));
      if (is_large(m)) z[k] = __float_as_uint(__fsub_rn(__fmul_rn(__uint_as_float(z[k]), f), m) * rcp(f));
    }
    tmem_st32(tS + c * 32, z);
  }
}

template <int FMT, int DH, bool SHORT>
__global__ void __launch_bounds__(kThreads, 1) k_kv_attend_many(const __grid_constant__ AttendArgs p) {
  constexpr int N = DH == 64 ? 64 : 128;  // columns of V's tile and of O: 96 are filled up with zeros
  constexpr int kP = DH == 64 ? 256 + 64 : 0;  // columns from S to P: beside O where that leaves room
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kBars);
  uint64_t* q_full = bars + 0;    // [2] per tile, once a segment
  uint64_t* k_full = bars + 2;
  uint64_t* k_empty = bars + 3;   // both S of the block are computed
  uint64_t* sc_full = bars + 4;   // [2] a block's scales (every other block's: a row may still read the one before)
  uint64_t* v_full = bars + 6;
  uint64_t* v_empty = bars + 7;   // both P V of the block are computed
  uint64_t* s_full = bars + 8;    // [2] per tile; O holds every product before it
  uint64_t* o_full = bars + 10;   // [2] O is complete
  uint64_t* p_full = bars + 12;   // [2]
  uint64_t* pv_done = bars + 14;  // [2] P V has read P, and S may be written over it
  uint64_t* drain = bars + 16;
  uint64_t* code_full = bars + 17;   // K's, V's codes of the next block
  uint64_t* code_free = bars + 19;   // [2] they have been read
  Misc& misc = *reinterpret_cast<Misc*>(smem + kMisc);
  volatile int* abort_flag = &misc.abort;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  start_dependents();

  // ---- the line, and this CTA's part of it (the sums lie where Q will)
  int64_t* warp_sums = reinterpret_cast<int64_t*>(smem);
  Line* line_s = reinterpret_cast<Line*>(smem + 256);
  const int per = (p.kv.n_seqs + kThreads - 1) / kThreads;
  int64_t total = 0, before = 0, own = 0;
  KvSeq mine{0, 0, 0};  // the last of this thread's sequences
  for (int s = t * per; s < min((t + 1) * per, p.kv.n_seqs); ++s) {
    mine = kv_seq(p.kv, s);
    own += seq_cost(p, mine);
  }
  {
    int64_t upto = own;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const int64_t v = __shfl_up_sync(0xFFFFFFFFu, upto, k);
      if (lane >= k) upto += v;
    }
    if (lane == 31) warp_sums[warp] = upto;
    __syncthreads();
    for (int w = 0; w < kThreads / 32; ++w) {
      before += w < warp ? warp_sums[w] : 0;
      total += warp_sums[w];
    }
    before += upto - own;
  }
  const int ctas = (int)min((int64_t)gridDim.x, total);
  const int j = blockIdx.x;
  if (t == 0) p.cuts[j].first = p.cuts[j].end = 0;
  if (j >= ctas) return;
  const int64_t begin = part(total, j, ctas), end = part(total, j + 1, ctas);
  if (begin >= before && begin < before + own) {
    int64_t base = before;
    int s = t * per;
    if (per > 1) {
      mine = kv_seq(p.kv, s);
      for (; s < p.kv.n_seqs - 1; ++s) {
        const int64_t n = seq_cost(p, mine);
        if (begin < base + n) break;
        base += n;
        mine = kv_seq(p.kv, s + 1);
      }
    }
    line_s->s = s;
    line_s->q = mine;
    line_s->base = base;
  }
  if (t == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], kTileRows);
      mbar_init(&sc_full[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&o_full[i], 1);
      mbar_init(&p_full[i], kTileRows);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(k_full, kConvertThreads);
    mbar_init(k_empty, 1);
    mbar_init(v_full, kConvertThreads);
    mbar_init(v_empty, 1);
    mbar_init(drain, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&code_full[i], 1);
      mbar_init(&code_free[i], kConvertThreads);
    }
    misc.abort = misc.odd = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) { tmem_alloc(&misc.tmem, 512); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc.tmem;
  const Line line = *line_s;
  __syncthreads();  // Q may be written
  const uint32_t sbase = smem_addr(smem);
  if (DH == 96) {
    for (int i = t; i < 128 * 4; i += kThreads) st_shared_v4(piece(sbase + kV, i >> 2, 12 + (i & 3)), make_uint4(0, 0, 0, 0));
    __syncthreads();
  }
  Walk w;
  w.p = &p;
  w.s = line.s;
  w.rt = 0;
  w.q = line.q;
  w.t = tiles_of(p, line.q);
  w.base = line.base;
  w.at = begin;
  w.end = end;
  int tile = 0;  // blocks so far
  bool ok = true;

  // ---------------- codes to fp16: THREADS threads, `lt` this one's number ----------------
  constexpr int kPieces = DH / 16;  // of 16 codes, of a key
  auto convert = [&](auto threads, int lt, uint32_t dst, uint32_t from, bool values, const BlockKeys& keys) {
    constexpr int kN = decltype(threads)::value, kMine = kBlockKeys * kPieces / kN, kBatch = kMine % 4 ? 3 : 4;
    // Piece i of this thread: codes 16 ch .. of key row `row`.  Rows of 128: eight neighbouring threads take the first half of a row
    // and the second of the next, so that what they read, and the two 16-byte pieces that each writes, touch every bank once; i moves
    // the row by a multiple of 8, so neither offset depends on it.
    auto place = [&](int i, int& row, int& ch) {
      if (DH == 128) {
        row = i * (kN / 8) + (((lt >> 4) << 1) | ((lt >> 2) & 1));
        ch = (lt & 3) | (((lt >> 2) ^ (lt >> 3)) & 1) << 2;
      } else {
        const int idx = i * kN + lt;
        row = idx / kPieces;
        ch = idx - row * kPieces;
      }
    };
    const int rows = keys.rows, have = keys.have, check = keys.check && values;
    const bool whole = rows == kBlockKeys && have == 0xFF;
    // A batch is read before its first piece is written: a write holds the reads behind it back.
#pragma unroll 1
    for (int i0 = 0; i0 < kMine; i0 += kBatch) {
      uint4 x[kBatch];
      int row[kBatch], ch[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        place(i0 + k, row[k], ch[k]);
        x[k] = ld_shared_v4(from + (uint32_t)(row[k] * DH + ch[k] * 16));
      }
      if (!whole) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          if (row[k] >= rows || !(have >> (row[k] >> 4) & 1)) x[k] = make_uint4(0, 0, 0, 0);
      }
      if (check) {
        uint32_t odd = 0;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) odd |= nonfinite4<FMT>(x[k].x) | nonfinite4<FMT>(x[k].y) | nonfinite4<FMT>(x[k].z) | nonfinite4<FMT>(x[k].w);
        if (odd) {  // a weight of 0 times it would be NaN in rows that do not see it: 0 here, and the rows look for themselves
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            x[k].x &= ~((nonfinite4<FMT>(x[k].x) >> 7) * 0xFFu);
            x[k].y &= ~((nonfinite4<FMT>(x[k].y) >> 7) * 0xFFu);
            x[k].z &= ~((nonfinite4<FMT>(x[k].z) >> 7) * 0xFFu);
            x[k].w &= ~((nonfinite4<FMT>(x[k].w) >> 7) * 0xFFu);
          }
          misc.odd = 1;
        }
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const uint4 v = x[k];
        st_shared_v4(piece(dst, row[k], 2 * ch[k]),
                     make_uint4(f16x2_of<FMT>(v.x), f16x2_of<FMT>(v.x >> 16), f16x2_of<FMT>(v.y), f16x2_of<FMT>(v.y >> 16)));
        st_shared_v4(piece(dst, row[k], 2 * ch[k] + 1),
                     make_uint4(f16x2_of<FMT>(v.z), f16x2_of<FMT>(v.z >> 16), f16x2_of<FMT>(v.w), f16x2_of<FMT>(v.w >> 16)));
      }
    }
  };
  if (t < kConvertThreads) {
    while (ok && w.next()) {
      const int n = max(w.blocks_of(0), w.blocks_of(1));
      for (int b = 0; b < n && ok; ++b, ++tile) {
        const uint32_t par = (uint32_t)tile & 1u;
#pragma unroll 1
        for (int is_v = 0; is_v < 2; ++is_v) {
          if (!warp_wait<SHORT>(is_v ? v_empty : k_empty, par ^ 1u, abort_flag, p.wait_ns) ||
              !warp_wait<SHORT>(&code_full[is_v], par, abort_flag, p.wait_ns)) { ok = false; break; }
          convert(std::integral_constant<int, kConvertThreads>{}, t, sbase + (is_v ? kV : kK), sbase + kCodes + is_v * kAtom, is_v, misc.keys[tile & 3]);
          mbar_arrive(&code_free[is_v]);
          fence_async_shared();
          mbar_arrive(is_v ? v_full : k_full);
        }
      }
    }
    if (!ok) {
      atomicOr(p.kv.status, kStatusTimeout);
      *abort_flag = 1;
    }
  } else if (warp == kCopyWarp) {
    // ---------------- pages, copies, scales ----------------
    uint32_t fetched[2] = {0, 0};  // blocks whose codes were asked for
    while (ok && w.next()) {
      const int n = max(w.blocks_of(0), w.blocks_of(1));
      if (n == 0) continue;
      const int first = w.t.limit(w.r0), klim = w.t.limit(w.r0 + w.n_rows - 1), stop = w.b0 + n;
      const int32_t* table = p.kv.pages + (int64_t)w.s * p.kv.max_pages;
      const int mask = (1 << p.kv.page_shift) - 1, step = min(1 << p.kv.page_shift, kBlockKeys) >> 4;  // groups of 16 keys of a copy
      // Lanes 0 .. 7: the page of keys 16 lane .. of block b.  Read a block before it is looked at, and its scales a block before
      // they are: a load under a condition, or looked at at once, would hold this warp for its latency.
      auto seen = [&](int b) { return lane < 8 && b < stop && b * kBlockKeys + 16 * lane < klim; };
      auto read_page = [&](int b) { return table[seen(b) ? (b * kBlockKeys + 16 * lane) >> p.kv.page_shift : 0]; };
      auto page_of = [&](int b, int id) {  // -1: none
        if (!seen(b)) return -1;
        if (id >= 0 && id < p.kv.n_pages) return id;
        atomicOr(p.kv.status, kStatusBadCache);
        return -1;
      };
      auto read_scale = [&](const uint8_t* scales, int id) { return (int)scales[(int64_t)max(id, 0) * p.kv.hkv + w.h]; };
      // Lanes 0 .. 7 copy block b's codes of K (0) or V (1), a page (or 128 keys) each.  Slots behind the last key come along.
      auto fetch = [&](int which, int b, int id) {
        ++fetched[which];
        const bool mine = lane < 8 && lane % step == 0 && id >= 0;
        const uint32_t bytes = (uint32_t)(step * 16 * DH);
        const unsigned copies = __popc(__ballot_sync(0xFFFFFFFFu, mine));
        if (lane == 0) {
          if (copies) mbar_arrive_expect_tx(&code_full[which], copies * bytes);
          else mbar_arrive(&code_full[which]);
        }
        __syncwarp();
        if (mine) {
          const int64_t at = ((((int64_t)id * p.kv.hkv + w.h) << p.kv.page_shift) + ((b * kBlockKeys + 16 * lane) & mask)) * DH;
          bulk_load(smem + kCodes + which * kAtom + lane * 16 * DH, (which ? p.kv.v : p.kv.k) + at, bytes, &code_full[which]);
        }
        __syncwarp();
      };
      int here = read_page(w.b0), next = read_page(w.b0 + 1);
      here = page_of(w.b0, here);
      int xk = read_scale(p.kv.k_scale, here), xv = read_scale(p.kv.v_scale, here);
      for (int b = w.b0; b < stop; ++b, ++tile) {
        const uint32_t par = (uint32_t)tile & 1u;
        const unsigned have = __ballot_sync(0xFFFFFFFFu, here >= 0) & 0xFFu;
        // K's codes of the block before have been read
        if (!warp_wait<SHORT>(&code_free[0], par ^ 1u, abort_flag, p.wait_ns)) { ok = false; break; }
        if (lane == 0) misc.keys[tile & 3] = BlockKeys{min(kBlockKeys, klim - b * kBlockKeys), (int)have, (b + 1) * kBlockKeys > first};
        __syncwarp();
        fetch(0, b, here);
        // V's too, whose tile was written when P V of the one before it was done: that one's scales have been read
        if (!warp_wait<SHORT>(&code_free[1], par ^ 1u, abort_flag, p.wait_ns)) { ok = false; break; }
        fetch(1, b, here);
        BlockScales& sc = misc.scales[par];
        if (lane < 8) {
          sc.k[lane] = pow2(here < 0 ? 0 : xk - 127);
        }
        const int v = here < 0 ? -1000 : xv - 127, vmax = __reduce_max_sync(0xFFFFFFFFu, v);  // (lanes from 8 on have none)
        if (lane < 8) {
          const int dx = max(v - vmax, kNothing);
          sc.v[lane] = v;
          sc.dx[lane] = (float)dx;
          sc.back[lane] = pow2i(-dx);
        }
        if (lane == 0) {
          sc.none = (int)(~have & 0xFFu);
          sc.vmax = vmax;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sc_full[par]);
        here = page_of(b + 1, next);
        next = read_page(b + 2);
        xk = read_scale(p.kv.k_scale, here);
        xv = read_scale(p.kv.v_scale, here);
      }
    }
    if (!ok) {
      atomicOr(p.kv.status, kStatusTimeout);
      *abort_flag = 1;
    }
    // The copies in flight, before the memory is given back.  This warp may have asked for its last block and left its loop in order
    // where another role gives up and nobody waits for the block any more; when none did, they have landed.
    int never = 0;
    for (int i = 0; i < 2; ++i)
      if (fetched[i]) warp_wait<false>(&code_full[i], (fetched[i] - 1) & 1u, &never, 0);
  } else if (warp == kMmaWarp) {
    if (lane == 0) {
      // ---------------- the products ----------------
      uint32_t nq[2] = {0, 0}, ns[2] = {0, 0}, np[2] = {0, 0};  // segments, blocks and waits for P V of each tile so far
      while (ok && w.next()) {
        const int na = w.blocks_of(0), nb = w.blocks_of(1), n = max(na, nb);
        const int nx[2] = {na, nb};
        if (n == 0) continue;
        for (int side = 0; side < 2 && ok; ++side)
          if (nx[side]) {
            ok = wait<SHORT>(&q_full[side], nq[side] & 1u, abort_flag, p.wait_ns);
            ++nq[side];
          }
        for (int b = 0; b <= n && ok; ++b) {
          for (int side = 0; side < 2; ++side) {
            if (b > 0 && b - 1 < nx[side]) {
              if (!wait<SHORT>(v_full, (uint32_t)(tile + b - 1) & 1u, abort_flag, p.wait_ns) ||
                  !wait<SHORT>(&p_full[side], (ns[side] + (uint32_t)(b - 1)) & 1u, abort_flag, p.wait_ns)) { ok = false; break; }
              tc_fence_after();
              mma_values<N>(tmem + 256 + side * 128, tmem + side * 128 + kP, sbase + kV, b > 1);
              if (b == nx[side]) umma_commit(&o_full[side]);
              else if (kP == 0) umma_commit(&pv_done[side]);
            }
            if (side == 1 && b > 0) umma_commit(v_empty);
            if (b < nx[side]) {
              if (!wait<SHORT>(k_full, (uint32_t)(tile + b) & 1u, abort_flag, p.wait_ns)) { ok = false; break; }
              if (kP == 0 && b > 0 && !wait<SHORT>(&pv_done[side], np[side]++ & 1u, abort_flag, p.wait_ns)) { ok = false; break; }
              tc_fence_after();
              mma_scores<DH>(tmem + side * 128, sbase + kQ + side * kTile, sbase + kK);
              umma_commit(&s_full[side]);
            }
          }
          if (ok && b < n) umma_commit(k_empty);
        }
        tile += n;
        ns[0] += (uint32_t)na;
        ns[1] += (uint32_t)nb;
      }
      if (!ok) {
        atomicOr(p.kv.status, kStatusTimeout);
        *abort_flag = 1;
      }
      umma_commit(drain);
      int dummy = 0;
      mbar_wait(drain, 0, &dummy);
    }
  } else if (warp >= kFirstRowWarp) {
    // ---------------- a row a thread ----------------
    const int side = (warp - kFirstRowWarp) >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + (uint32_t)(side * 128) + lane_off, tO = tS + 256;
    const uint32_t qtile = sbase + kQ + side * kTile;
    uint32_t done = 0, n_segs = 0;  // blocks of this tile so far, and segments that had some
    while (ok && w.next()) {
      const int nx = w.blocks_of(side), n = max(w.blocks_of(0), w.blocks_of(1));
      const int i = side * kTileRows + r, pair = w.r0 + i;
      const bool real = i < w.n_rows;
      const int G = w.t.G, tok = w.t.token(real ? pair : w.r0), hd = w.h * G + (real ? pair : w.r0) - tok * G;
      const int64_t row = w.q.first + tok;
      const int limit = real ? w.t.limit(pair) : kAll;
      const int kmin = __reduce_min_sync(0xFFFFFFFFu, limit);
      float m = -INFINITY, l = 0.0f;
      int xr = -1000;
      bool large = false;  // some row's reference is above kLarge
      if (nx) {
        // q over a power of two of its row, as fp16: a warp reads its 32 rows at once, 16 bytes a lane and row (a thread that read its own
        // row took 15000 cycles for it).  A row that does not exist reads the unit's first.
        constexpr int kLanes = DH == 64 ? 8 : 16, kStep = 32 / kLanes, kSteps = 32 / kStep;
        const int sub = lane / kLanes, col = lane % kLanes, r0 = w.r0, first = w.q.first, n_rows = w.n_rows, head0 = w.h * G;
        const int64_t width = (int64_t)(p.n_heads + 2 * p.kv.hkv) * DH;
        const uint16_t* base = p.qkv + (col * 8 < DH ? col * 8 : 0);
        int ex = -110;
        uint4 v[kSteps];
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          const int other = i - lane + k * kStep + sub, pr = r0 + (other < n_rows ? other : 0), tk = w.t.token(pr);
          v[k] = ld_nc_v4(base + (first + tk) * width + (head0 + pr - tk * G) * DH);
        }
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          uint32_t big = max(max(absmax_bf16x2(v[k].x), absmax_bf16x2(v[k].y)), max(absmax_bf16x2(v[k].z), absmax_bf16x2(v[k].w)));
#pragma unroll
          for (int m = 1; m < kLanes; m <<= 1) big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, m));
          const int e = max((int)(big >> 23) - 127, -110);
          const float fq = pow2i(14 - e);
          if (col * 8 < DH)
            st_shared_v4(piece(qtile, (warp & 3) * 32 + k * kStep + sub, col),
                         make_uint4(pack_half2(bf16_lo(v[k].x) * fq, bf16_hi(v[k].x) * fq), pack_half2(bf16_lo(v[k].y) * fq, bf16_hi(v[k].y) * fq),
                                    pack_half2(bf16_lo(v[k].z) * fq, bf16_hi(v[k].z) * fq), pack_half2(bf16_lo(v[k].w) * fq, bf16_hi(v[k].w) * fq)));
          const int mine = __shfl_sync(0xFFFFFFFFu, e, (lane % kStep) * kLanes);
          if (lane / kStep == k) ex = mine;
        }
        const float rowf = p.scale_log2 * pow2i(ex - 14);
        fence_async_shared();
        mbar_arrive(&q_full[side]);

        for (int b = 0; b < nx && ok; ++b, ++done) {
          const int kpar = (tile + b) & 1;
          if (!warp_wait<SHORT>(&s_full[side], done & 1u, abort_flag, p.wait_ns)) { ok = false; break; }
          if (!warp_wait<SHORT>(&sc_full[kpar], (uint32_t)((tile + b) >> 1) & 1u, abort_flag, p.wait_ns)) { ok = false; break; }
          tc_fence_after();
          const BlockScales& sc = misc.scales[kpar];
          const int key0 = (w.b0 + b) * kBlockKeys, none = sc.none;
          const bool edge = key0 + kBlockKeys > kmin || none;
          auto factor = [&](int g) { return factor_of(rowf, sc, g); };
          auto hidden = [&](int col) { return key0 + col >= limit || (none >> (col >> 4) & 1); };
          float mx = -INFINITY;
          int xnew = max(xr, sc.vmax);
          if (edge) {
            xnew = xr;
            for (int g = 0; g < 8; ++g)
              if (!hidden(16 * g)) xnew = max(xnew, sc.v[g]);
          }
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t z[32];
            tmem_ld32(tS + c * 32, z);
            if (edge) {
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (hidden(c * 32 + k)) z[k] = 0xFF800000u;
            }
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              float y[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) y[k] = __uint_as_float(z[g * 16 + k]);
#pragma unroll
              for (int k = 4; k < 16; ++k) y[k & 3] = fmaxf(y[k & 3], __uint_as_float(z[g * 16 + k]));
              mx = fmaxf(mx, fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])) * factor(2 * c + g));
            }
          }
          bool up = mx - m > kSlack;
          if (__any_sync(0xFFFFFFFFu, up || xnew != xr)) {
            up |= !edge && mx > m;  // (what rows do not all see moves only those that see it)
            const float alpha = up ? ex2(m - mx) : 1.0f, fo = alpha * pow2(xr - xnew);
            if (b > 0) {
#pragma unroll 1
              for (int c = 0; c < N / 32; ++c) {
                uint32_t o[32];
                tmem_ld32(tO + c * 32, o);
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * fo);
                tmem_st32(tO + c * 32, o);
              }
            }
            l *= alpha;
            if (up) m = mx;
            xr = xnew;
            large = __any_sync(0xFFFFFFFFu, is_large(m));
          }
          const float ref = fabsf(m) >= kLarge ? 0.0f : m;  // (a large one is taken before; a row that has seen nothing has none)
          // 2^(s - m + 11 + dx), dx the exponent of the page's V over xr; the sum takes 2^dx back, so it holds for pages of any V.  Where all
          // rows see the block dx is the block's own and one shift a row; elsewhere a page that the row does not see may be above xr.
          const int shift = max(sc.vmax - xr, kNothing);
          const float off = kOffset + (float)shift - ref;
          if (large) take_reference(tS, sc, rowf, m);
          float sum_b = 0.0f;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t z[32];
            tmem_ld32(tS + c * 32, z);
            float add[2] = {sc.dx[2 * c] + off, sc.dx[2 * c + 1] + off}, back[2] = {sc.back[2 * c], sc.back[2 * c + 1]};
            if (edge) {
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (hidden(c * 32 + k)) z[k] = 0xFF800000u;
#pragma unroll
              for (int g = 0; g < 2; ++g) {
                const int dx = max(min(sc.v[2 * c + g] - xr, 0), kNothing);
                add[g] = kOffset + (float)dx - ref;
                back[g] = pow2i(-dx);
              }
            }
            uint32_t yy[16];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              uint32_t* y = yy + 8 * g;
              const float fg = factor(2 * c + g);
              const float2 f2 = make_float2(fg, fg), c2 = make_float2(add[g], add[g]);
              float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const int col = g * 16 + 2 * k;
                const float2 e = __ffma2_rn(make_float2(__uint_as_float(z[col]), __uint_as_float(z[col + 1])), f2, c2);
                const float2 pr = make_float2(ex2(e.x), ex2(e.y));
                sum[k & 1] = __fadd2_rn(sum[k & 1], pr);
                y[k] = pack_half2(pr.x, pr.y);
              }
              sum[0] = __fadd2_rn(sum[0], sum[1]);
              sum_b = __fmaf_rn(sum[0].x + sum[0].y, back[g], sum_b);
            }
            tmem_st16(tS + kP + c * 16, yy);
          }
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&p_full[side]);
          l = __fmaf_rn(sum_b, edge ? 1.0f : pow2i(-shift), l);
        }
        // the last product
        if (ok && !warp_wait<SHORT>(&o_full[side], n_segs++ & 1u, abort_flag, p.wait_ns)) ok = false;
        if (!ok) break;
        tc_fence_after();
      }
      // ---- the row's result: O over the sum
      const bool starts = w.b0 == 0, whole = starts && w.b1 == w.nb;
      const int slot = 2 * j + (starts ? 1 : 0);
      const float inv = l == 0.0f ? 0.0f : 1.0f / l, fx = pow2(xr);
      const float lse2 = l == 0.0f ? -INFINITY : m + (log2f(l) - kOffset);
      // Where V held NaN or infinite values: each column's first key with one, into this warp's rows of Q, which the last S has read.
      const bool odd = nx && *(volatile int*)&misc.odd;
      int* bad = reinterpret_cast<int*>(smem + kQ + side * kTile + (warp & 3) * 4096);
      if (odd) {
        for (int k = lane; k < DH; k += 32) bad[k] = kAll;
        __syncwarp();
        const int last = min((w.b0 + nx) * kBlockKeys, w.t.limit(w.r0 + min(w.n_rows, (side + 1) * kTileRows) - 1));
        // (the blocks that V was looked at in: from the first that not all rows see)
        for (int key = max(w.b0, w.t.limit(w.r0) / kBlockKeys) * kBlockKeys + lane; key < last; key += 32) {
          const int id = p.kv.pages[(int64_t)w.s * p.kv.max_pages + (key >> p.kv.page_shift)];
          if (id < 0 || id >= p.kv.n_pages) continue;
          const uint8_t* codes = p.kv.v + ((((int64_t)id * p.kv.hkv + w.h) << p.kv.page_shift) + (key & ((1 << p.kv.page_shift) - 1))) * DH;
          for (int k = 0; k < DH; ++k)
            if (nonfinite4<FMT>(codes[k]) & 0x80u) atomicMin(&bad[k], key);
        }
        __syncwarp();
      }
      // Through this warp's rows of Q's second half (4 KB of its own behind `bad`), so that neighbouring lanes write a row's neighbouring bytes.
      const uint32_t stage = qtile + (uint32_t)((warp & 3) * 4096) + kAtom;
      const int to = real ? (int)(row * p.n_heads + hd) : -1;  // below 2^31
      const int64_t to_part = ((int64_t)slot * kRows + i - lane) * DH;
      const int there = w.n_rows - (i - lane);  // rows of this warp
#pragma unroll 1
      for (int c = 0; c < DH / 32; ++c) {
        uint32_t o[32];
        __syncwarp();
        if (nx) tmem_ld32(tO + c * 32, o);
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          float v = l == 0.0f ? 0.0f : __uint_as_float(nx ? o[k] : 0u) * inv * fx;
          if (odd && bad[c * 32 + k] < limit) v = __uint_as_float(0x7FC00000u);
          o[k] = __float_as_uint(v);
        }
        if (whole) {  // four lanes a row
          const int col = lane & 3;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            st_shared_v4(stage + lane * 64 + ((k ^ (lane >> 1)) & 3) * 16,
                         make_uint4(pack_bf16x2(__uint_as_float(o[8 * k]), __uint_as_float(o[8 * k + 1])),
                                    pack_bf16x2(__uint_as_float(o[8 * k + 2]), __uint_as_float(o[8 * k + 3])),
                                    pack_bf16x2(__uint_as_float(o[8 * k + 4]), __uint_as_float(o[8 * k + 5])),
                                    pack_bf16x2(__uint_as_float(o[8 * k + 6]), __uint_as_float(o[8 * k + 7]))));
          __syncwarp();
          uint4 x[4];
          int at[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int from = k * 8 + (lane >> 2);
            x[k] = ld_shared_v4(stage + from * 64 + ((col ^ (from >> 1)) & 3) * 16);
            at[k] = __shfl_sync(0xFFFFFFFFu, to, from);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (at[k] >= 0) *reinterpret_cast<uint4*>(p.att + (int64_t)at[k] * DH + c * 32 + col * 8) = x[k];
        } else {  // eight lanes a row
          const int col = lane & 7;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            st_shared_v4(stage + lane * 128 + ((k ^ lane) & 7) * 16, make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]));
          __syncwarp();
          uint4 x[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int from = k * 4 + (lane >> 3);
            x[k] = ld_shared_v4(stage + from * 128 + ((col ^ from) & 7) * 16);
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int from = k * 4 + (lane >> 3);
            if (from < there) *reinterpret_cast<uint4*>(p.part_o + to_part + from * DH + c * 32 + col * 4) = x[k];
          }
        }
      }
      if (real) {
        if (whole) p.lse[(int64_t)hd * p.kv.T + row] = lse2 * kLn2;
        else p.part_sum[slot * kRows + i] = make_float2(m, l * 0x1p-11f);
      }
      if (t == 32 * kFirstRowWarp && starts && !whole)
        p.cuts[j] = Cut{w.unit0, w.unit0 + w.cost, total, ctas, w.h, w.q.first, w.n_rows, w.r0};
      tc_fence_before();
      tile += n;
    }
    if (!ok) {
      atomicOr(p.kv.status, kStatusTimeout);
      *abort_flag = 1;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// Block (j, y): rows 32 y .. of the unit that CTA j began and did not end, four a warp at a time; its parts in order.
constexpr int kJoinWarps = 8, kJoinRows = 4;
template <int DH>
__global__ void __launch_bounds__(32 * kJoinWarps) k_kv_join_many(const AttendArgs p) {
  wait_for_previous();
  const int j = blockIdx.x, r0 = (blockIdx.y * kJoinWarps + (threadIdx.x >> 5)) * kJoinRows, lane = threadIdx.x & 31;
  const Cut cut = p.cuts[j];
  if (cut.first == cut.end || r0 >= cut.rows) return;
  const int n = (int)((cut.end * cut.ctas + cut.total - 1) / cut.total) - j;
  auto slot = [&](int i) { return i == 0 ? 2 * j + 1 : 2 * (j + i); };
  float M[kJoinRows], sum[kJoinRows], acc[kJoinRows][DH / 32];
#pragma unroll
  for (int q = 0; q < kJoinRows; ++q) {
    M[q] = -INFINITY;
    sum[q] = 0.0f;
#pragma unroll
    for (int k = 0; k < DH / 32; ++k) acc[q][k] = 0.0f;
  }
  // (rows behind the tile's last hold what an earlier call left; they are not written)
  for (int i = 0; i < n; ++i) {
    float2 e[kJoinRows];
    float v[kJoinRows][DH / 32];
#pragma unroll
    for (int q = 0; q < kJoinRows; ++q) {
      e[q] = p.part_sum[slot(i) * kRows + r0 + q];
      const float* src = p.part_o + ((int64_t)slot(i) * kRows + r0 + q) * DH + lane;
#pragma unroll
      for (int k = 0; k < DH / 32; ++k) v[q][k] = src[32 * k];
    }
#pragma unroll
    for (int q = 0; q < kJoinRows; ++q) {
      const float mn = fmaxf(M[q], e[q].x), fade = mn == M[q] ? 1.0f : ex2(M[q] - mn);
      const float wgt = e[q].y * (e[q].x == mn ? 1.0f : ex2(e[q].x - mn));  // (the sum of a part that saw nothing is 0)
      sum[q] = sum[q] * fade + wgt;
#pragma unroll
      for (int k = 0; k < DH / 32; ++k) acc[q][k] = acc[q][k] * fade + (e[q].y == 0.0f ? 0.0f : wgt * v[q][k]);
      M[q] = mn;
    }
  }
  const int G = p.n_heads / p.kv.hkv;
#pragma unroll
  for (int q = 0; q < kJoinRows; ++q) {
    const int r = r0 + q;
    if (r >= cut.rows) break;
    const int tok = (cut.group_row + r) / G, hd = cut.head * G + (cut.group_row + r) - tok * G;
    __nv_bfloat16* to = reinterpret_cast<__nv_bfloat16*>(p.att) + ((int64_t)(cut.row0 + tok) * p.n_heads + hd) * DH + lane;
#pragma unroll
    for (int k = 0; k < DH / 32; ++k) to[32 * k] = __float2bfloat16_rn(sum[q] == 0.0f ? 0.0f : acc[q][k] / sum[q]);
    if (lane == 0) p.lse[(int64_t)hd * p.kv.T + cut.row0 + tok] = sum[q] == 0.0f ? -INFINITY : (M[q] + log2f(sum[q])) * kLn2;
  }
}

template <int FMT, int DH, bool SHORT = false>
cudaError_t launch(const AttendArgs& p, int ctas, cudaStream_t s) {
  static std::atomic<uint64_t> configured{0};
  cudaError_t e = kv_smem(k_kv_attend_many<FMT, DH, SHORT>, kSmem, configured);
  if (e != cudaSuccess) return e;
  k_kv_attend_many<FMT, DH, SHORT><<<ctas, kThreads, kSmem, s>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_dependent(k_kv_join_many<DH>, dim3((unsigned)ctas, kRows / (kJoinRows * kJoinWarps)), 32 * kJoinWarps, 0, s, p);
}

}  // namespace

int kv_attend_many_rows() { return kRows; }

cudaError_t launch_kv_attend_many(const AttendArgs& p, int ctas, cudaStream_t s) {
  if (p.wait_ns && p.kv.fmt == 0 && p.kv.dh == 128) return launch<0, 128, true>(p, ctas, s);
  if (p.kv.fmt)
    return p.kv.dh == 128 ? launch<1, 128>(p, ctas, s) : p.kv.dh == 96 ? launch<1, 96>(p, ctas, s) : launch<1, 64>(p, ctas, s);
  return p.kv.dh == 128 ? launch<0, 128>(p, ctas, s) : p.kv.dh == 96 ? launch<0, 96>(p, ctas, s) : launch<0, 64>(p, ctas, s);
}

}  // namespace fp8q
