// Causal attention of a call's last tokens over the 8-bit key/value cache.
//
// The cache is read once, and each byte of it meets the rows of its K/V head: the query heads that share it, times the call's tokens, 1 to 64 of
// them, two operations each: bound by memory.  Tensor memory's accumulators of 128 rows would stand mostly empty, and their operands
// would have to go through shared memory a second time as fp16; so the products are warp-level
// m16n8k16 ones, whose operands are made in registers, and FP8 codes become fp16 (exactly) on the way from shared memory.
//
// A warp takes 32 keys at a time for 8 rows, or 16.  Keys are the products' long side (M = 16), rows the short one (N = 8), so the
// few rows of a token's query heads fill what they use.  Both products allow any order of their contraction, and the second of
// its rows, as long as both operands share it, and that decides the layout:
//   S^T = K Q^T: a thread's share of a key is head_dim / 4 consecutive bytes; word i of it is its operand of step i.
//   O^T = V^T P^T: rows g and g + 8 of tile i stand for elements g head_dim / 8 + 2 i and the next, so a thread's share of a key is
//   head_dim / 8 consecutive bytes, and so is its share of a row of O.
// P goes from the first product's accumulators to the second's operand through four 8 x 8 transposes.
//
// Precision.  Scores are fp32 in the log2 domain.  q is divided by a power of two of its row and so is exact in fp16 (elements
// below 2^-28 of the row's largest lose bits).  p = 2^(s - m) enters as fp16 times 2^15, so it has 11 bits down to 2^-29 of the
// row's largest and vanishes below 2^-39.  V's scales are relative to the largest that the row has seen so far (xr), which moves like the
// maximum does, and p times that ratio is what is rounded.  Both are a row's own: what it does not see does not move a bit of it.
//
// Work.  The keys of all (sequence, row tile, K/V head) units form one line of blocks of 128 keys, each unit preceded by what it costs
// besides; it is cut into equal parts, one a CTA.  A unit that is cut leaves fp32 partial results, which the second kernel joins in order.
//
// Measured (both kernels, out of a graph; lengths of batches differ, and sizes here are the largest): 64 sequences of up to 8192 tokens, 40 + 8
// heads of 128, 372 MB of cache: 69 us, 5.4 TB/s; 48 of up to 32768, 1.4 GB: 219 us, 6.4 TB/s; one of 250007, 28 + 4 heads: 54 us, 4.8
// TB/s; 24 of up to 3000 with up to 6 rows (83 in all), 12 + 12 heads of 64: 21.5 us.  A reference of V's scales for each row costs tiles of
// more than 8 rows 3 to 5 % (16 of up to 4096 with 5 rows: 45 us with one for a warp, 48 with its own for each).
// About 3 us go before the first byte of the cache arrives (the line, the pages), 3 to 4 for the second launch, a tenth for CTAs
// that end before the last.  Inside, with 12 warps an SM (their registers fill it) the
// issue slots are 45 % taken and shared memory 24 %: what holds the rest is the latency of a warp's own chain of instructions.
#include <atomic>

#include "fp8q_kvline.cuh"

namespace fp8q {

namespace {

constexpr int kThreads = 128, kWarps = 4;

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 16 bytes into shared memory; bytes = 0 writes zeros and reads nothing.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Offset of byte `b` (of a 16-byte piece) of a row in a tile of rows of DH codes.  Rows of 128: piece ^ row % 8; of 64: two rows to a
// line of 128, piece ^ twice the line % 4; with these, and with rows of 96 as they are, the K reads of a
// quarter of a warp, and the V reads of 128 and 64, touch every bank once.
template <int DH>
__device__ __forceinline__ uint32_t place(int row, int b) {
  if (DH == 128) return (uint32_t)(row * 128 + ((((b >> 4) ^ row) & 7) << 4) + (b & 15));
  if (DH == 64) {
    const int line = row >> 1, piece = (row & 1) * 4 + (b >> 4);
    return (uint32_t)(line * 128 + ((piece ^ ((line & 3) << 1)) << 4) + (b & 15));
  }
  return (uint32_t)(row * 96 + b);
}

// N / 4 words of a row from byte b on.
template <int DH, int N>
__device__ __forceinline__ void take(const uint8_t* tile, int row, int b, uint32_t (&w)[N / 4]) {
  if (N % 16 == 0) {
#pragma unroll
    for (int i = 0; i < N / 16; ++i) {
      const uint4 v = *reinterpret_cast<const uint4*>(tile + place<DH>(row, b + 16 * i));
      w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
    }
  } else if (N % 8 == 0) {
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
      const uint2 v = *reinterpret_cast<const uint2*>(tile + place<DH>(row, b + 8 * i));
      w[2 * i] = v.x; w[2 * i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) w[i] = *reinterpret_cast<const uint32_t*>(tile + place<DH>(row, b + 4 * i));
  }
}

template <int DH, int NT, int RW>
struct Shape {
  static constexpr int KW = kWarps / RW;      // groups of warps that share their keys
  static constexpr int GK = 32 * RW;          // keys of a group at a time
  static constexpr int RT = 8 * NT;           // rows of a warp
  static constexpr int R = RT * RW;           // rows of the CTA
  static constexpr int kTile = kBlockKeys * DH;
  static constexpr int kRing = 2 * 2 * kTile; // two stages of K and V
  static constexpr int kPitch = DH + 4;       // floats of a row of partial O
  static constexpr int kJoin = KW * R * kPitch * 4;
  static constexpr int kSmem = kRing > kJoin ? kRing : kJoin;
  // as many as shared memory and the registers of their accumulators allow
  static constexpr int kCtas = NT == 1 ? (DH == 128 ? 3 : DH == 96 ? 4 : 5) : (DH == 64 ? 4 : 3);
};

// What a unit costs besides its keys, in blocks of keys: its rows, its first page, joining the warps.  (64 sequences of up to 8192 tokens:
// 71.4, 69.3, 68.8, 69.5 and 72.3 us with 1, 2, 3, 4 and 6; 24 of up to 3000 with up to 6 rows: 21.2, 21.5, 21.5, 22.2, 23.3; 64 of up to
// 1000: 27.3, 26.1, 26.2, 25.6, 25.3.)
constexpr int kUnitCost = 3;

template <int R>
__device__ __forceinline__ int64_t seq_cost(const AttendArgs& p, const KvSeq& q, int& units, int& nb, int& cost) {
  const int pairs = q.n * (p.n_heads / p.kv.hkv);  // below 2^31 with T n_heads
  units = (int)((pairs + (int64_t)(R - 1)) / R) * p.kv.hkv;
  nb = (q.len + kBlockKeys - 1) / kBlockKeys;
  cost = nb ? nb + kUnitCost : 1;
  return (int64_t)units * cost;
}
// Transposes an 8 x 8 tile of 16-bit values over the warp: from (row lane / 4, columns 2 (lane % 4) and the next) to the same of its columns.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int FMT, int DH, int NT, int RW>
__global__ void __launch_bounds__(kThreads, Shape<DH, NT, RW>::kCtas) k_kv_attend(const AttendArgs p) {
  using C = Shape<DH, NT, RW>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t warp_sums[kWarps];
  __shared__ Line line_s;
  __shared__ int scales[2][kWarps][4];  // [stage][part of 32 keys][2 K, 2 V scales of 16 keys each]
  __shared__ float row_m[kWarps][C::RT], row_l[kWarps][C::RT];
  __shared__ int row_x[kWarps][C::RT];
  start_dependents();
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31, c = lane & 3, g8 = lane >> 2;
  const int kg = warp / RW, rw = warp % RW;
  const int G = p.n_heads / p.kv.hkv;

  // ---- the line, and this CTA's part of it
  const int per = (p.kv.n_seqs + kThreads - 1) / kThreads;
  int64_t total = 0, before = 0, own = 0;  // the line; the blocks of the sequences before this thread's, and of its own
  KvSeq mine{0, 0, 0};                     // the last of them
  for (int s = t * per; s < min((t + 1) * per, p.kv.n_seqs); ++s) {
    int units, nb, cost;
    mine = kv_seq(p.kv, s);
    own += seq_cost<C::R>(p, mine, units, nb, cost);
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
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
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
        int units, nb, cost;
        const int64_t n = seq_cost<C::R>(p, mine, units, nb, cost);
        if (begin < base + n) break;
        base += n;
        mine = kv_seq(p.kv, s + 1);
      }
    }
    line_s.s = s;
    line_s.q = mine;
    line_s.base = base;
  }
  __syncthreads();
  int s = line_s.s;
  KvSeq q = line_s.q;
  int64_t base = line_s.base, at = begin;

  while (at < end) {
    int units, nb, cost;
    const int64_t here = seq_cost<C::R>(p, q, units, nb, cost);
    if (at >= base + here) {
      base += here;
      if (++s >= p.kv.n_seqs) break;
      q = kv_seq(p.kv, s);
      continue;
    }
    // ---- one segment: blocks [b0, b1) of unit u, whose own cost comes before its blocks
    const int u = here < (int64_t)1 << 31 ? (int)((uint32_t)(at - base) / (uint32_t)cost) : (int)((at - base) / cost);
    const int v0 = (int)((at - base) - (int64_t)u * cost);
    const int v1 = (int)min((int64_t)cost, v0 + (end - at));
    const int64_t unit0 = base + (int64_t)u * cost;
    at += v1 - v0;
    const int b0 = max(0, v0 - kUnitCost), b1 = max(0, v1 - kUnitCost);
    if (b0 == b1 && nb) continue;
    const int rt = u / p.kv.hkv, h = u - rt * p.kv.hkv;
    const int r0 = rt * C::R, n_rows = min(C::R, q.n * G - r0);
    if (nb == 0) {  // an empty slot of a batch
      for (int i = t; i < n_rows * (DH / 4); i += kThreads) {
        const int r = i / (DH / 4), tok = (r0 + r) / G, hd = h * G + (r0 + r) - tok * G;
        *reinterpret_cast<uint2*>(p.att + ((int64_t)(q.first + tok) * p.n_heads + hd) * DH + (i - r * (DH / 4)) * 4) = make_uint2(0, 0);
        if (i == r * (DH / 4)) p.lse[(int64_t)hd * p.kv.T + q.first + tok] = -INFINITY;
      }
      continue;
    }
    // limit = the keys that a row sees; rows that do not exist see all and are dropped.  This thread's scores are of
    // rows 8 n + 2 c and the next of its warp.
    constexpr int kAll = 0x7FFFFFFF;
    const int before_rows = q.len - q.n;  // tokens before the call's
    int limit[NT][2], kmin = kAll, kmax = 0;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = rw * C::RT + 8 * n + 2 * c + e;
        limit[n][e] = r < n_rows ? before_rows + (r0 + r) / G + 1 : kAll;
        kmin = min(kmin, limit[n][e]);
        kmax = max(kmax, r < n_rows ? limit[n][e] : 0);
      }
    kmin = __reduce_min_sync(0xFFFFFFFFu, kmin);
    kmax = __reduce_max_sync(0xFFFFFFFFu, kmax);                                // of the warp
    const int klim = max(0, before_rows + (r0 + n_rows - 1) / G + 1);           // of the CTA
    const int stop = min(b1, (klim + kBlockKeys - 1) / kBlockKeys);

    // ---- the ring: this warp copies its part of 32 keys of its group's tile
    const int32_t* table = p.kv.pages + (int64_t)s * p.kv.max_pages;
    const int my_keys = kg * C::GK + rw * 32;  // within a block
    const int page_mask = (1 << p.kv.page_shift) - 1;
    const uint32_t ring = smem_addr(smem) + (uint32_t)(kg * C::GK * DH);
    // Lane k: the page of keys 16 (k % 2) .. of this warp's part of block b, and lanes 0 .. 3 its scales (K of both, V of both).  Read
    // a step before they are looked at: a load under a condition, or looked at at once, holds the warp for its latency.
    auto seen = [&](int b) { return b < stop && b * kBlockKeys + my_keys + 16 * (lane & 1) < klim; };
    auto read_page = [&](int b) { return table[seen(b) ? (b * kBlockKeys + my_keys + 16 * (lane & 1)) >> p.kv.page_shift : 0]; };
    auto page_of = [&](int b, int id) {  // -1: none, or behind the limit
      if (!seen(b)) return -1;
      if (id >= 0 && id < p.kv.n_pages) return id;
      atomicOr(p.kv.status, kStatusBadCache);
      return -1;
    };
    const uint8_t* scale_base = (lane & 2 ? p.kv.v_scale : p.kv.k_scale) + h;
    auto read_scale = [&](int id) { return (int)scale_base[(int64_t)max(id, 0) * p.kv.hkv]; };
    auto copy_tile = [&](int b, int id_lane, int sc, int stage) {
      const int key = b * kBlockKeys + my_keys;
      const uint32_t to = ring + (uint32_t)(stage * 2 * C::kTile);
      const bool full = key + 32 <= klim;
#pragma unroll
      for (int sub = 0; sub < 2; ++sub) {
        const int id = __shfl_sync(0xFFFFFFFFu, id_lane, sub);
        const int sl = (key + 16 * sub) & page_mask;
        const int64_t off = ((((int64_t)max(id, 0) * p.kv.hkv + h) << p.kv.page_shift) + sl) * DH;
        const uint8_t *ks = p.kv.k + off + lane * 16, *vs = p.kv.v + off + lane * 16;
        if (full && id >= 0) {
#pragma unroll
          for (int i = 0; i < DH / 32; ++i) {
            const int lin = (i * 32 + lane) * 16, row = lin / DH, byte = lin - row * DH;
            const uint32_t d = to + place<DH>(rw * 32 + 16 * sub + row, byte);
            copy16(d, ks + i * 512);
            copy16(d + C::kTile, vs + i * 512);
          }
        } else {  // rows that no row of the CTA sees become zero, and are not read
          const int rows = id < 0 ? 0 : min(16, klim - key - 16 * sub);
#pragma unroll 1
          for (int i = 0; i < DH / 32; ++i) {
            const int lin = (i * 32 + lane) * 16, row = lin / DH, byte = lin - row * DH;
            const uint32_t d = to + place<DH>(rw * 32 + 16 * sub + row, byte);
            const int bytes = row < rows ? 16 : 0;
            copy16(d, bytes ? ks + i * 512 : p.kv.k, bytes);
            copy16(d + C::kTile, bytes ? vs + i * 512 : p.kv.v, bytes);
          }
        }
      }
      if (lane < 4) scales[stage][warp][lane] = id_lane < 0 ? kNoPage : sc - 127;
    };
    auto group_sync = [&]() {
      if (RW == 1) __syncwarp();
      else asm volatile("bar.sync %0, %1;" ::"r"(1 + kg), "n"(32 * RW) : "memory");
    };

    // The chain that a segment begins with is a page's number, then its keys (and its scales, which are stored after
    // the copies are on their way); q is fetched beside it and made ready while the first keys arrive.
    int id_a = read_page(b0), id_b = read_page(b0 + 1);
    uint32_t qw[NT][DH / 8];  // row 8 n + lane / 4, elements c DH / 4 ..
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      // a row that does not exist reads the unit's first
      const int r = rw * C::RT + 8 * n + g8, pair = r0 + (r < n_rows ? r : 0), tok = pair / G;
      const uint16_t* src = p.qkv + (int64_t)(q.first + tok) * (p.n_heads + 2 * p.kv.hkv) * DH +
                            (int64_t)(h * G + pair - tok * G) * DH + c * (DH / 4);
#pragma unroll
      for (int i = 0; i < DH / 32; ++i) {
        const uint4 v = ld_nc_v4(src + 8 * i);
        qw[n][4 * i] = v.x; qw[n][4 * i + 1] = v.y; qw[n][4 * i + 2] = v.z; qw[n][4 * i + 3] = v.w;
      }
    }
    id_a = page_of(b0, id_a);
    int sc_a = read_scale(id_a);
    auto next = [&](int b) {  // copies block b's keys; a step ahead its successor's scales, two ahead the pages
      if (b < stop) copy_tile(b, id_a, sc_a, (b - b0) & 1);
      copies_commit();
      id_a = page_of(b + 1, id_b);
      sc_a = read_scale(id_a);
      id_b = read_page(b + 2);
    };
    next(b0);
    uint32_t qb[NT][DH / 16][2];
    int exq[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < DH / 8; ++i) m = max(m, absmax_bf16x2(qw[n][i]));
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
      const int ex = max((int)(m >> 23) - 127, -110);  // the row's largest |q| < 2^(ex + 1)
      const float f = pow2i(14 - ex);
#pragma unroll
      for (int i = 0; i < DH / 16; ++i) {
        qb[n][i][0] = pack_half2(bf16_lo(qw[n][2 * i]) * f, bf16_hi(qw[n][2 * i]) * f);
        qb[n][i][1] = pack_half2(bf16_lo(qw[n][2 * i + 1]) * f, bf16_hi(qw[n][2 * i + 1]) * f);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) exq[n][e] = __shfl_sync(0xFFFFFFFFu, ex - 14, (2 * c + e) * 4);
    }
    float o[DH / 16][NT][4], m[NT][2], l[NT][2];
    int xr[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < DH / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][n][e] = 0.0f;
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.0f;
      xr[n][0] = xr[n][1] = -1000;
    }
    bool large = false;  // some row's maximum is above kLarge

#pragma unroll 1
    for (int b = b0; b < stop; ++b) {
      next(b + 1);
      copies_wait<1>();
      group_sync();
      const int stage = (b - b0) & 1;
#pragma unroll 1
      for (int sub = 0; sub < RW; ++sub) {
        const int key0 = b * kBlockKeys + kg * C::GK + sub * 32;
        if (key0 >= kmax) break;
        const uint8_t* kt = smem + stage * 2 * C::kTile + kg * C::GK * DH;
        const uint8_t* vt = kt + C::kTile;
        const int row0 = sub * 32;
        const int* sc = scales[stage][kg * RW + sub];
        const int xk[2] = {sc[0], sc[1]}, xv[2] = {sc[2], sc[3]};
        // scores: [16 keys][8 rows][keys lane / 4 and 8 on, rows 2 c and the next]
        float z[2][NT][4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t wa[DH / 16], wb[DH / 16];
          take<DH, DH / 4>(kt, row0 + 16 * k + g8, c * (DH / 4), wa);
          take<DH, DH / 4>(kt, row0 + 16 * k + 8 + g8, c * (DH / 4), wb);
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) z[k][n][e] = 0.0f;
#pragma unroll
          for (int i = 0; i < DH / 16; ++i) {
            const uint32_t a[4] = {f16x2_of<FMT>(wa[i]), f16x2_of<FMT>(wb[i]), f16x2_of<FMT>(wa[i] >> 16), f16x2_of<FMT>(wb[i] >> 16)};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816(z[k][n], a, qb[n][i][0], qb[n][i][1]);
          }
        }
        const bool edge = key0 + 32 > kmin || xk[0] == kNoPage || xk[1] == kNoPage;
        if (edge) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (key0 + 16 * k + g8 + 8 * (e >> 1) >= limit[n][e & 1] || xk[k] == kNoPage) z[k][n][e] = -INFINITY;
        }
        // the row's maximum: a page's scale is positive, so it goes to the page's maximum alone
        float f[2][NT][2], mn[NT][2];
        bool moved = false;
        const int xv0 = xv[0] == kNoPage ? -1000 : xv[0], xv1 = xv[1] == kNoPage ? -1000 : xv[1];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = m[n][e];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              f[k][n][e] = p.scale_log2 * pow2i(max(exq[n][e] + xk[k], -100));
              x = fmaxf(x, fmaxf(z[k][n][e], z[k][n][e + 2]) * f[k][n][e]);
            }
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, w));
            mn[n][e] = x;
            moved |= x != m[n][e];
          }
        if (__any_sync(0xFFFFFFFFu, moved)) {
          large = false;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float fade = mn[n][e] == m[n][e] ? 1.0f : ex2(m[n][e] - mn[n][e]);
              l[n][e] *= fade;
#pragma unroll
              for (int i = 0; i < DH / 16; ++i) {
                o[i][n][e] *= fade;
                o[i][n][e + 2] *= fade;
              }
              m[n][e] = mn[n][e];
              large |= is_large(m[n][e]);
            }
          large = __any_sync(0xFFFFFFFFu, large);
        }
        if (large) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e)  // the difference, over what it is multiplied by below
                if (is_large(m[n][e & 1])) z[k][n][e] = __fsub_rn(__fmul_rn(z[k][n][e], f[k][n][e & 1]), m[n][e & 1]) * rcp(f[k][n][e & 1]);
        }
        // The largest scale of V that each row has seen.  Rows' differ only from the first step on that not all see, and what follows is such a
        // step; there a row may see one of the two groups of 16 keys, or none.
        auto largest = [&](int n, int e) {
          return max(xr[n][e], edge ? max(key0 < limit[n][e] ? xv0 : -1000, key0 + 16 < limit[n][e] ? xv1 : -1000) : max(xv0, xv1));
        };
        bool grew = false;
        if (edge) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) grew |= largest(n, e) != xr[n][e];
          grew = __any_sync(0xFFFFFFFFu, grew);
        } else {
          grew = largest(0, 0) != xr[0][0];
        }
        if (grew) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int x = largest(n, e);
              const float fx = pow2(xr[n][e] - x);
#pragma unroll
              for (int i = 0; i < DH / 16; ++i) {
                o[i][n][e] *= fx;
                o[i][n][e + 2] *= fx;
              }
              xr[n][e] = x;
            }
        }
        // 2^(s - m + 15 + dx), dx the exponent of the page's V over xr.  The sum takes 2^dx back, so it holds for pages of any V;
        // below 2^-60 nothing is left of one in fp16.  (A page that the row does not see may be above xr.)
        uint32_t pb[2][NT][2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float w[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int dx = max(min((k ? xv1 : xv0) - xr[n][e], 0), -60);
              const float add = (float)(15 + dx) - (fabsf(m[n][e]) >= kLarge ? 0.0f : m[n][e]), back = pow2i(-dx);
#pragma unroll
              for (int i = e; i < 4; i += 2) {
                w[i] = ex2(__fmaf_rn(z[k][n][i], f[k][n][e], add));
                l[n][e] = __fmaf_rn(w[i], back, l[n][e]);
              }
            }
            pb[k][n][0] = transposed(pack_half2(w[0], w[1]));
            pb[k][n][1] = transposed(pack_half2(w[2], w[3]));
          }
        }
        // the keys of step k: rows 2c, 2c + 1, 2c + 8, 2c + 9 of its 16
        uint32_t odd = 0;
        if (edge) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t w[DH / 32];
            take<DH, DH / 8>(vt, row0 + (i >> 2) * 16 + 2 * c + (i & 1) + (i & 2) * 4, g8 * (DH / 8), w);
#pragma unroll
            for (int k = 0; k < DH / 32; ++k) odd |= nonfinite4<FMT>(w[k]);
          }
          odd = __any_sync(0xFFFFFFFFu, odd != 0);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t w[4][DH / 32];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            take<DH, DH / 8>(vt, row0 + k * 16 + 2 * c + (i & 1) + (i >> 1) * 8, g8 * (DH / 8), w[i]);
          uint32_t ones[NT][2];
          if (odd) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int key = key0 + 16 * k + g8 + 8 * e;
                ones[n][e] = transposed(xk[k] == kNoPage ? 0u : (key < limit[n][0] ? 0x3C00u : 0u) | (key < limit[n][1] ? 0x3C000000u : 0u));
              }
          }
#pragma unroll
          for (int i = 0; i < DH / 16; ++i) {
            // bytes 2 i and 2 i + 1: the elements of rows lane / 4 and lane / 4 + 8 of tile i, for two pairs of keys
            const uint32_t sel = i & 1 ? 0x7362u : 0x5140u;
            const uint32_t x = __byte_perm(w[0][i >> 1], w[1][i >> 1], sel), y = __byte_perm(w[2][i >> 1], w[3][i >> 1], sel);
            uint32_t a[4] = {f16x2_of<FMT>(x), f16x2_of<FMT>(x >> 16), f16x2_of<FMT>(y), f16x2_of<FMT>(y >> 16)};
            if (odd) {
              // Some V is NaN or infinite, and some row does not see every key: a masked key's weight of 0 times it would be
              // NaN.  Such values become 0, and a second product, of ones, finds the rows that do see one.
              uint32_t bad[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t high = (((a[e] & 0x7FFF7FFFu) + 0x04000400u) & 0x80008000u) >> 15;
                a[e] &= ~(high * 0xFFFFu);
                bad[e] = high * 0x3C00u;
              }
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                float seen[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                mma16816(seen, bad, ones[n][0], ones[n][1]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (seen[e] != 0.0f) o[i][n][e] = __uint_as_float(0x7FC00000u);
              }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816(o[i][n], a, pb[k][n][0], pb[k][n][1]);
          }
        }
      }
      group_sync();
    }
    copies_wait<0>();

    // ---- join the groups' results: through the ring's memory
    __syncthreads();
    float* join = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * n + 2 * c + e;  // of the warp
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) l[n][e] += __shfl_xor_sync(0xFFFFFFFFu, l[n][e], w);
        if (g8 == 0) {
          row_m[warp][r] = m[n][e];
          row_l[warp][r] = l[n][e];
          row_x[warp][r] = xr[n][e];
        }
        if (rw * C::RT + r < n_rows) {
          float* to = join + (kg * C::R + rw * C::RT + r) * C::kPitch + g8 * (DH / 8);
#pragma unroll
          for (int i = 0; i < DH / 32; ++i)
            *reinterpret_cast<float4*>(to + 4 * i) = make_float4(o[2 * i][n][e], o[2 * i][n][e + 2], o[2 * i + 1][n][e], o[2 * i + 1][n][e + 2]);
        }
      }
    __syncthreads();
    const bool starts = b0 == 0, whole = starts && b1 == nb;
    const int slot = 2 * j + (starts ? 1 : 0);
    for (int i = t; i < n_rows * (DH / 4); i += kThreads) {
      const int r = i / (DH / 4), col = (i - r * (DH / 4)) * 4, w0 = r / C::RT, wr = r - w0 * C::RT;
      float M = -INFINITY;
      int X = -1000;
#pragma unroll
      for (int k = 0; k < C::KW; ++k) {
        M = fmaxf(M, row_m[k * RW + w0][wr]);
        X = max(X, row_x[k * RW + w0][wr]);
      }
      float L = 0.0f, a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < C::KW; ++k) {
        const int w = k * RW + w0;
        const float mk = row_m[w][wr], lk = row_l[w][wr];
        const float f = mk == M ? (M == -INFINITY ? 0.0f : 1.0f) : ex2(mk - M);
        L += lk * (lk != lk ? 1.0f : f);
        const float fo = f * pow2(row_x[w][wr] - X);
        const float4 v = *reinterpret_cast<const float4*>(join + (k * C::R + r) * C::kPitch + col);
        a[0] += v.x * fo; a[1] += v.y * fo; a[2] += v.z * fo; a[3] += v.w * fo;
      }
      const float inv = L == 0.0f ? 0.0f : 1.0f / L, fx = pow2(X);
#pragma unroll
      for (int k = 0; k < 4; ++k) a[k] = L == 0.0f ? 0.0f : a[k] * inv * fx;
      const float lse2 = L == 0.0f ? -INFINITY : M + (log2f(L) - 15.0f);
      if (whole) {
        const int tok = (r0 + r) / G, hd = h * G + (r0 + r) - tok * G;
        *reinterpret_cast<uint2*>(p.att + ((int64_t)(q.first + tok) * p.n_heads + hd) * DH + col) =
            make_uint2(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]));
        if (col == 0) p.lse[(int64_t)hd * p.kv.T + q.first + tok] = lse2 * kLn2;
      } else {
        *reinterpret_cast<float4*>(p.part_o + ((int64_t)slot * C::R + r) * DH + col) = make_float4(a[0], a[1], a[2], a[3]);
        if (col == 0) p.part_sum[slot * C::R + r] = make_float2(M, L * 0x1p-15f);
      }
    }
    if (t == 0 && starts && !whole)
      p.cuts[j] = Cut{unit0, unit0 + cost, total, ctas, h, q.first, n_rows, r0};
    __syncthreads();
  }
}

// Block (j, r): row r of the unit that CTA j began and did not end.  Its parts: CTA j's last, then the first of those after it; a warp
// takes every eighth, eight at a time in flight, and the warps' sums are added in order.  Most blocks have nothing to do, so what counts is how
// many an SM holds (16 x 5 rows over 4096: 48 us with five, 54 with three; 24 x 6 rows of heads of 64: 21.5 with six, 22.1 with five).
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;
template <int DH, int R>
__global__ void __launch_bounds__(kJoinThreads, DH == 64 ? 6 : 5) k_kv_join(const AttendArgs p) {
  __shared__ float acc_s[kJoinWarps][DH], max_s[kJoinWarps], sum_s[kJoinWarps];
  wait_for_previous();
  const int j = blockIdx.x, r = blockIdx.y, t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const Cut cut = p.cuts[j];
  if (cut.first == cut.end || r >= cut.rows) return;
  // the last CTA of the unit is the last whose part of the line begins before the unit's end: total i / ctas < end
  const int n = (int)((cut.end * cut.ctas + cut.total - 1) / cut.total) - j;
  auto slot = [&](int i) { return i == 0 ? 2 * j + 1 : 2 * (j + i); };
  float acc[DH / 32], sum = 0.0f, M = -INFINITY;
#pragma unroll
  for (int k = 0; k < DH / 32; ++k) acc[k] = 0.0f;
  for (int i0 = warp; i0 < n; i0 += 8 * kJoinWarps) {
    float v[8][DH / 32];
    float2 e[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {  // a part that does not exist is the warp's first, with no weight
      const int i = i0 + q * kJoinWarps, s = slot(i < n ? i : i0);
      e[q] = p.part_sum[s * R + r];
      const float* src = p.part_o + ((int64_t)s * R + r) * DH + lane;
#pragma unroll
      for (int k = 0; k < DH / 32; ++k) v[q][k] = src[32 * k];
      if (i >= n) e[q] = make_float2(-INFINITY, 0.0f);
    }
    float mn = M;
#pragma unroll
    for (int q = 0; q < 8; ++q) mn = fmaxf(mn, e[q].x);
    const float fade = mn == M ? 1.0f : ex2(M - mn);
    sum *= fade;
#pragma unroll
    for (int k = 0; k < DH / 32; ++k) acc[k] *= fade;
    M = mn;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float w = e[q].y * (e[q].x == M ? 1.0f : ex2(e[q].x - M));  // (the sum of a part that saw nothing is 0)
      sum += w;
#pragma unroll
      for (int k = 0; k < DH / 32; ++k) acc[k] += e[q].y == 0.0f ? 0.0f : w * v[q][k];
    }
  }
#pragma unroll
  for (int k = 0; k < DH / 32; ++k) acc_s[warp][lane + 32 * k] = acc[k];
  if (lane == 0) {
    max_s[warp] = M;
    sum_s[warp] = sum;
  }
  __syncthreads();
  if (t >= DH / 2) return;
  M = max_s[0];
#pragma unroll
  for (int k = 1; k < kJoinWarps; ++k) M = fmaxf(M, max_s[k]);
  float total = 0.0f, v[2] = {0.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < kJoinWarps; ++k) {  // (a warp whose rows are NaN has no maximum, and its sum is NaN)
    const float f = max_s[k] == M ? 1.0f : max_s[k] == -INFINITY ? (sum_s[k] == 0.0f ? 0.0f : 1.0f) : ex2(max_s[k] - M);
    total += f * sum_s[k];
    v[0] += f * acc_s[k][2 * t];
    v[1] += f * acc_s[k][2 * t + 1];
  }
  const int G = p.n_heads / p.kv.hkv, tok = (cut.group_row + r) / G, hd = cut.head * G + (cut.group_row + r) - tok * G;
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  *reinterpret_cast<uint32_t*>(p.att + ((int64_t)(cut.row0 + tok) * p.n_heads + hd) * DH + 2 * t) =
      total == 0.0f ? 0u : pack_bf16x2(v[0] * inv, v[1] * inv);
  if (t == 0) p.lse[(int64_t)hd * p.kv.T + cut.row0 + tok] = total == 0.0f ? -INFINITY : (M + log2f(total)) * kLn2;
}

// Rows of a CTA for the (token, head) pairs of a sequence and K/V head: 8 of one warp or 16; above, two or four warps share their keys
// for 16 rows each; and from kManyPairs on the kernel on tensor memory.  (2 sequences of up to 8192, 16 of up to 4096 and 64 of up to 1000,
// 40 + 8 heads of 128: 35 pairs 37, 74 and 84 us here and 51, 70, 98 there; 50 pairs 42, 78, 96 and 51, 63, 100; 80 pairs 54, 139, 149 and
// 52, 74, 103.)  Pairs are T / n_seqs rows times the heads, as the host does not know more: a batch that mixes a long piece of a prompt with single
// tokens is better split into two calls.
constexpr int kManyPairs = 65;
struct Rows {
  int nt, rw;
  bool many() const { return nt == 0; }
  int count() const { return many() ? kv_attend_many_rows() : 8 * nt * rw; }
  int ctas() const { return many() ? 152 : kMaxCtas; }
};
Rows rows_of(int64_t T, int n_seqs, int n_heads, int hkv) {
  const int64_t pairs = (T + n_seqs - 1) / n_seqs * (n_heads / hkv);
  return pairs <= 8 ? Rows{1, 1} : pairs <= 16 ? Rows{2, 1} : pairs <= 32 ? Rows{2, 2} : pairs < kManyPairs ? Rows{2, 4} : Rows{0, 0};
}
struct Pieces {
  size_t sum, cuts, all;
};
Pieces pieces(Rows r, int dh) {
  auto pad = [](size_t n) { return (n + 255) & ~size_t(255); };
  const size_t parts = 2 * (size_t)r.ctas();
  Pieces w;
  w.sum = pad(parts * r.count() * dh * 4);
  w.cuts = w.sum + pad(parts * r.count() * sizeof(float2));
  w.all = w.cuts + pad(sizeof(Cut) * r.ctas());
  return w;
}

template <int FMT, int DH, int NT, int RW>
cudaError_t launch(const AttendArgs& p, int sms, int64_t pairs, cudaStream_t s) {
  using C = Shape<DH, NT, RW>;
  static_assert(C::kCtas * 152 <= kMaxCtas, "parts of the workspace");
  const int ctas = min(kMaxCtas, sms * C::kCtas);
  static std::atomic<uint64_t> configured{0};
  cudaError_t e = kv_smem(k_kv_attend<FMT, DH, NT, RW>, C::kSmem, configured);
  if (e != cudaSuccess) return e;
  k_kv_attend<FMT, DH, NT, RW><<<ctas, kThreads, C::kSmem, s>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_dependent(k_kv_join<DH, C::R>, dim3((unsigned)ctas, (unsigned)min(pairs, (int64_t)C::R)), kJoinThreads, 0, s, p);
}
template <int FMT, int DH>
cudaError_t launch_rows(Rows r, const AttendArgs& p, int sms, int64_t pairs, cudaStream_t s) {
  if (r.nt == 1) return launch<FMT, DH, 1, 1>(p, sms, pairs, s);
  return r.rw == 1 ? launch<FMT, DH, 2, 1>(p, sms, pairs, s)
                   : r.rw == 2 ? launch<FMT, DH, 2, 2>(p, sms, pairs, s) : launch<FMT, DH, 2, 4>(p, sms, pairs, s);
}
template <int FMT>
cudaError_t launch_dh(Rows r, const AttendArgs& p, int sms, int64_t pairs, cudaStream_t s) {
  return p.kv.dh == 128 ? launch_rows<FMT, 128>(r, p, sms, pairs, s)
                        : p.kv.dh == 96 ? launch_rows<FMT, 96>(r, p, sms, pairs, s) : launch_rows<FMT, 64>(r, p, sms, pairs, s);
}

}  // namespace

size_t kv_attend_workspace_bytes(int64_t T, int n_seqs, int n_heads, int hkv, int dh) {
  return pieces(rows_of(T, n_seqs, n_heads, hkv), dh).all;
}

cudaError_t launch_kv_attend(const KvArgs& a, const uint16_t* qkv, int n_heads, uint16_t* att, float* lse, void* ws,
                             const Launch& L) {
  const Rows r = rows_of(a.T, a.n_seqs, n_heads, a.hkv);
  const Pieces w = pieces(r, a.dh);
  uint8_t* b = static_cast<uint8_t*>(ws);
  AttendArgs p{a, qkv, n_heads, kLog2e / sqrtf((float)a.dh), att, lse, reinterpret_cast<float*>(b),
               reinterpret_cast<float2*>(b + w.sum), reinterpret_cast<Cut*>(b + w.cuts), L.wait_ns};
  // rows of a unit at most, where the host knows them
  const int64_t pairs = a.row_start ? (int64_t)1 << 20 : (int64_t)a.rows * (n_heads / a.hkv);
  const cudaError_t e = r.many() ? launch_kv_attend_many(p, min(r.ctas(), L.num_sms), L.stream)
                        : a.fmt ? launch_dh<1>(r, p, L.num_sms, pairs, L.stream) : launch_dh<0>(r, p, L.num_sms, pairs, L.stream);
  if (e != cudaSuccess) return e;
  if (L.launches) *L.launches += 2;
  return cudaSuccess;
}

}  // namespace fp8q
