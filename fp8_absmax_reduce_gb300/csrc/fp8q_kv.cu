// Writing tokens into the 8-bit key/value cache, and reading them back.
//
// A page of one head has one power-of-two scale 2^X, X the smallest exponent at which its largest value is not clipped.  A
// page fills over many calls; when a later token is larger X grows by some k, and the codes that are there become
// rne(code 2^-k): an FP8 code over a power of two is a code again unless it becomes subnormal, so what the
// cache holds does not drift.
//
// Both are bound by memory (a long prompt) or by their chain of dependent loads (a few tokens).  Measured out of a graph: a token each of 16
// sequences, 8 heads of 128, 2.6 us; the prompts of four, 4096 tokens at most, 14.7 us (3.6 TB/s; 9.7 us with the caches warm); 39541
// rows of 8 heads of 96 read back as fp32 54 us (5.6 TB/s).
#include <cuda_fp16.h>

#include "fp8q_kv.cuh"

namespace fp8q {

namespace {

constexpr int kHeld = 8;  // vectors of 8 elements that a thread keeps between the absmax and the codes: a page's, of one head

template <int F32>
struct In8 {
  uint4 w[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + i * (F32 ? 4 : 2));
#pragma unroll
    for (int k = 0; k < (F32 ? 2 : 1); ++k) w[k] = q[k];
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
#pragma unroll
    for (int k = 0; k < (F32 ? 8 : 4); ++k) {
      if (F32) {
        v[k] = __uint_as_float(u[k]);
      } else {
        v[2 * k] = bf16_lo(u[k]);
        v[2 * k + 1] = bf16_hi(u[k]);
      }
    }
  }
};

constexpr uint32_t kInf = 0x7F800000u;

// The largest |v| of 8 as fp32 bits (a NaN's are above infinity's); bf16 values by twos.
template <int F32>
__device__ __forceinline__ uint32_t absmax8(const In8<F32>& x) {
  const uint32_t* u = reinterpret_cast<const uint32_t*>(x.w);
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < (F32 ? 8 : 4); ++k) m = F32 ? max(m, u[k] & 0x7FFFFFFFu) : __vmaxu2(m, u[k] & 0x7FFF7FFFu);
  return F32 ? m : max(m << 16, m & 0xFFFF0000u);
}
// The same over what is finite.
__device__ __forceinline__ uint32_t finite_absmax8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t b = abs_bits(v[k]);
    m = max(m, b >= kInf ? 0u : b);
  }
  return m;
}

// 2^d for d <= 0; below 2^-126 nothing of a code is left.
__device__ __forceinline__ float pow2_down(int d) { return __uint_as_float((uint32_t)(127 + max(d, -126)) << 23); }

template <int FMT>
__device__ __forceinline__ uint32_t shift4(uint32_t codes, float s) {
  const uint32_t lo = f16x2_of<FMT>(codes), hi = f16x2_of<FMT>(codes >> 16);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return cvt_fp8x4<FMT>(a.x * s, a.y * s, b.x * s, b.y * s);
}

// Group x of THREADS threads (a warp, or a block), head y, K or V z: the pieces of pages that begin in rows [x rows_per_group, ...).  A
// piece is what a call writes of one page; it begins at a sequence's first row or at a page's first token.  Its values are
// read once and kept in registers, where kHeld vectors a thread hold them.
constexpr int kAppendThreads = 128;  // of a block, at least
template <int F32, int FMT, int DH, int THREADS>
__global__ void __launch_bounds__(THREADS < kAppendThreads ? kAppendThreads : THREADS)
    k_kv_append(const KvArgs a, const void* __restrict__ qkv, int n_heads, int rows_per_group) {
  constexpr int kGroups = THREADS < kAppendThreads ? kAppendThreads / THREADS : 1;
  __shared__ uint32_t red[32];
  const int h = blockIdx.y, is_v = blockIdx.z, P = 1 << a.page_shift, tid = threadIdx.x % THREADS;
  constexpr int vecs = DH / 8;  // vectors of 8 of a token
  const int64_t width = (int64_t)(n_heads + 2 * a.hkv) * DH;
  const int64_t col = (int64_t)(n_heads + is_v * a.hkv + h) * DH;
  uint8_t* codes = is_v ? a.v : a.k;
  uint8_t* scales = is_v ? a.v_scale : a.k_scale;
  const int64_t r0 = ((int64_t)blockIdx.x * kGroups + threadIdx.x / THREADS) * rows_per_group;
  const int end = (int)min(r0 + rows_per_group, a.T);
  auto group_max = [&](uint32_t v) { return THREADS == 32 ? warp_max_u32(v) : block_max_u32(v, red); };
  bool nonfinite = false;
  int s = -1;
  KvSeq q{0, 0, 0};
  for (int row = (int)min(r0, a.T); row < end;) {
    if (row < q.first || row >= q.first + q.n) {
      s = kv_find_warp(a, row);
      if (s < 0) { ++row; continue; }
      q = kv_seq(a, s);
      if (row < q.first || row >= q.first + q.n) {  // behind the last sequence, or rows that are not in order
        ++row;
        continue;
      }
    }
    const int pos = q.pos(row);
    if (pos < 0) {  // padding
      row += min(-pos, q.first + q.n - row);
      continue;
    }
    const int slot = pos & (P - 1);
    const int m = min(P - slot, q.first + q.n - row);  // tokens of this page from here on
    if (row != q.first && slot != 0) {                 // the piece began before this group's rows
      row += m;
      continue;
    }
    const int first = row, n = m * vecs;
    row += m;
    const int id = kv_page(a, s, pos >> a.page_shift);
    const bool fits = THREADS > 32 || n <= kHeld * THREADS;  // a block's registers hold any piece
    auto load = [&](In8<F32>& x, int i) {
      const int t = i / vecs;
      x.load(qkv, (int64_t)(first + t) * width + col + (i - t * vecs) * 8);
    };
    In8<F32> held[kHeld];
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (tid + k * THREADS < n) load(held[k], tid + k * THREADS);
    if (id < 0) continue;
    const int64_t ph = (int64_t)id * a.hkv + h;
    const int was = slot ? (int)scales[ph] - 127 : 0;
    uint8_t* page = codes + (ph << a.page_shift) * DH;
    uint32_t amax = 0;
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (tid + k * THREADS < n) amax = max(amax, absmax8(held[k]));
    if (!fits)
#pragma unroll 1
      for (int i = tid + kHeld * THREADS; i < n; i += THREADS) {
        In8<F32> x;
        load(x, i);
        amax = max(amax, absmax8(x));
      }
    amax = group_max(amax);
    const bool odd = amax >= kInf;  // a value is NaN or infinite: those do not count, and become NaN codes
    if (odd) {
      amax = 0;
#pragma unroll 1
      for (int i = tid; i < n; i += THREADS) {
        In8<F32> x;
        load(x, i);
        float v[8];
        x.get(v);
        amax = max(amax, finite_absmax8(v));
      }
      amax = group_max(amax);
      nonfinite = true;
    }
    int X = mx_exponent<FMT>(amax);
    if (slot) X = max(X, was);
    const float scale = pow2_neg(X);
    auto store = [&](const In8<F32>& x, int i) {
      float v[8];
      x.get(v);
      if (odd) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = abs_bits(v[e]) >= kInf ? __uint_as_float(0x7FC00000u) : v[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __fmul_rn(v[e], scale);
      *reinterpret_cast<uint2*>(page + slot * DH + i * 8) =
          make_uint2(cvt_fp8x4<FMT>(v[0], v[1], v[2], v[3]), cvt_fp8x4<FMT>(v[4], v[5], v[6], v[7]));
    };
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (tid + k * THREADS < n) store(held[k], tid + k * THREADS);
    if (!fits)
#pragma unroll 1
      for (int i = tid + kHeld * THREADS; i < n; i += THREADS) {
        In8<F32> x;
        load(x, i);
        store(x, i);
      }
    if (slot && X > was) {  // the tokens that were there, to the new scale
      const float down = pow2_down(was - X);
      for (int i = tid; i < slot * vecs; i += THREADS) {
        uint2* p = reinterpret_cast<uint2*>(page + i * 8);
        const uint2 w = *p;
        *p = make_uint2(shift4<FMT>(w.x, down), shift4<FMT>(w.y, down));
      }
    }
    if (tid == 0 && (!slot || X != was)) scales[ph] = (uint8_t)(X + 127);
    if (THREADS == 32) __syncwarp();  // every lane has read the scale before a later piece's
  }
  if (nonfinite) atomicOr(a.status, kStatusNonfinite);
}

// A warp takes rows_per_warp rows, 16 bytes of output a lane and step, kReads steps in flight.
constexpr int kReadThreads = 256, kReads = 8;
template <int F32, int FMT, int DH>
__global__ void __launch_bounds__(kReadThreads) k_kv_read(const KvArgs a, void* __restrict__ kv, int rows_per_warp) {
  constexpr int N = F32 ? 4 : 8;  // codes of 16 bytes of output
  const int lane = threadIdx.x & 31, P = 1 << a.page_shift;
  const int vecs = 2 * a.hkv * DH / N;
  const int64_t r0 = ((int64_t)blockIdx.x * (kReadThreads / 32) + (threadIdx.x >> 5)) * rows_per_warp;
  const int end = (int)min(r0 + rows_per_warp, a.T);
  int s = -1;
  KvSeq q{0, 0, 0};
  for (int row = (int)r0; row < end; ++row) {
    if (row < q.first || row >= q.first + q.n) {
      s = kv_find_warp(a, row);
      if (s < 0) continue;
      q = kv_seq(a, s);
      if (row < q.first || row >= q.first + q.n) continue;
    }
    const int pos = q.pos(row);
    const int id = pos < 0 ? -1 : kv_page(a, s, pos >> a.page_shift);
    const int64_t ph0 = (int64_t)id * a.hkv;
    const int slot = pos & (P - 1);
    uint4* out = reinterpret_cast<uint4*>(kv) + (int64_t)row * vecs;
    if (id < 0) {  // padding, or no page
      for (int i = lane; i < vecs; i += 32) out[i] = make_uint4(0, 0, 0, 0);
      continue;
    }
    for (int i0 = lane; i0 < vecs; i0 += 32 * kReads) {
      uint32_t w[kReads][N / 4];
      uint32_t x[kReads];
#pragma unroll
      for (int k = 0; k < kReads; ++k) {  // (behind the row's end its last piece again, which is not written)
        const int e = min(i0 + 32 * k, vecs - 1) * N, head = e / DH, is_v = head >= a.hkv;
        const int64_t ph = ph0 + head - is_v * a.hkv;
        const uint8_t* src = (is_v ? a.v : a.k) + ((ph << a.page_shift) + slot) * DH + e - head * DH;
        x[k] = (is_v ? a.v_scale : a.k_scale)[ph];
        if (N == 8) {
          const uint2 u = *reinterpret_cast<const uint2*>(src);
          w[k][0] = u.x;
          w[k][N / 4 - 1] = u.y;
        } else {
          w[k][0] = *reinterpret_cast<const uint32_t*>(src);
        }
      }
#pragma unroll
      for (int k = 0; k < kReads; ++k) {
        const float scale = e8m0(x[k]);
        float v[N];
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
          const uint32_t h2 = f16x2_of<FMT>(w[k][j >> 1] >> (16 * (j & 1)));
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
          v[2 * j] = f.x * scale;
          v[2 * j + 1] = f.y * scale;
        }
        uint4 o;
        if (F32) o = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
        else o = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4 % N], v[5 % N]), pack_bf16x2(v[6 % N], v[7 % N]));
        if (i0 + 32 * k < vecs) out[i0 + 32 * k] = o;
      }
    }
  }
}

template <int F32, int FMT, int DH>
void append_threads(const KvArgs& a, const void* qkv, int n_heads, int sms, cudaStream_t s) {
  // A piece has a sequence's rows, or a page's tokens.  Where that is 16 at most (or what a warp's registers hold), a warp
  // takes it alone: nothing waits for a block, and four times as many pieces' loads are in flight (219 drafted rows 11.5 us by a block
  // and 5.8 by a warp, 200 single tokens 8.4 and 3.2, prompts in pages of 16 25.8 and 15.1).  Larger pieces do not fit a warp's registers and
  // would be read twice (prompts in pages of 64, caches warm: 20 us read twice, 9.7 once).  A group of threads gets a page's tokens of
  // rows, or fewer, down to one, until there are about as many groups as fit the GPU.
  const int P = 1 << a.page_shift;
  const int64_t piece = (a.T + a.n_seqs - 1) / a.n_seqs;
  const bool warp = (piece < P ? piece : P) <= 16 || P * DH <= 8 * kHeld * 32;
  const int64_t per = a.T * 2 * a.hkv / ((warp ? 64 : 8) * sms);
  const int rows = (int)(per < 1 ? 1 : 2 * per < P ? per : P);
  const int64_t groups = (a.T + rows - 1) / rows;
  const dim3 grid((unsigned)(warp ? (groups + 3) / 4 : groups), (unsigned)a.hkv, 2);
  if (warp) k_kv_append<F32, FMT, DH, 32><<<grid, kAppendThreads, 0, s>>>(a, qkv, n_heads, rows);
  else if (P * DH <= 8 * kHeld * 128) k_kv_append<F32, FMT, DH, 128><<<grid, 128, 0, s>>>(a, qkv, n_heads, rows);
  else k_kv_append<F32, FMT, DH, 256><<<grid, 256, 0, s>>>(a, qkv, n_heads, rows);
}
template <int F32, int FMT>
void append_dh(const KvArgs& a, const void* qkv, int n_heads, int sms, cudaStream_t s) {
  if (a.dh == 128) append_threads<F32, FMT, 128>(a, qkv, n_heads, sms, s);
  else if (a.dh == 96) append_threads<F32, FMT, 96>(a, qkv, n_heads, sms, s);
  else append_threads<F32, FMT, 64>(a, qkv, n_heads, sms, s);
}

template <int F32, int FMT>
void read_dh(const KvArgs& a, void* kv, unsigned grid, int rows, cudaStream_t s) {
  auto* k = a.dh == 128 ? k_kv_read<F32, FMT, 128> : a.dh == 96 ? k_kv_read<F32, FMT, 96> : k_kv_read<F32, FMT, 64>;
  k<<<grid, kReadThreads, 0, s>>>(a, kv, rows);
}

}  // namespace

cudaError_t launch_kv_append(const KvArgs& a, const void* qkv, int f32, int n_heads, const Launch& L) {
  if (f32) a.fmt ? append_dh<1, 1>(a, qkv, n_heads, L.num_sms, L.stream) : append_dh<1, 0>(a, qkv, n_heads, L.num_sms, L.stream);
  else a.fmt ? append_dh<0, 1>(a, qkv, n_heads, L.num_sms, L.stream) : append_dh<0, 0>(a, qkv, n_heads, L.num_sms, L.stream);
  if (L.launches) ++*L.launches;
  return cudaGetLastError();
}

cudaError_t launch_kv_read(const KvArgs& a, void* kv, int f32, const Launch& L) {
  // four rows a warp where that still gives every SM its 64 warps (a sequence's rows find it once); a row each below (333 rows: 2.75 us)
  const int warps = kReadThreads / 32;
  const int64_t per = a.T / (64 * (int64_t)L.num_sms);
  const int rows = (int)(per < 1 ? 1 : per > 4 ? 4 : per);
  const unsigned grid = (unsigned)((a.T + (int64_t)rows * warps - 1) / ((int64_t)rows * warps));
  if (f32) a.fmt ? read_dh<1, 1>(a, kv, grid, rows, L.stream) : read_dh<1, 0>(a, kv, grid, rows, L.stream);
  else a.fmt ? read_dh<0, 1>(a, kv, grid, rows, L.stream) : read_dh<0, 0>(a, kv, grid, rows, L.stream);
  if (L.launches) ++*L.launches;
  return cudaGetLastError();
}

}  // namespace fp8q
