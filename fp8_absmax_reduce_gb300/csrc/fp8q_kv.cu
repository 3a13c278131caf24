// Writing tokens into the 8-bit key/value cache, and reading them back.
//
// A page of one head has one power-of-two scale 2^X, X the smallest exponent at which its largest value is not clipped.  A
// page fills over many calls; when a later token is larger X grows by some k, and the codes that are there become
// rne(code 2^-k): an FP8 code over a power of two is a code again unless it becomes subnormal, so what the
// cache holds does not drift.
//
// Both are bound by memory (a long prompt) or by their chain of dependent loads (a few tokens).
#include <cuda_fp16.h>

#include "fp8q_kv.cuh"

namespace fp8q {

namespace {

constexpr int kAppendThreads = 128;
constexpr int kHeld = 8;  // vectors of 8 elements that a thread keeps between the absmax and the codes

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

// Bits of the largest finite |v|; values that are not finite are noted.
__device__ __forceinline__ uint32_t absmax8(const float (&v)[8], bool& nonfinite) {
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t b = abs_bits(v[k]);
    nonfinite |= b >= kInf;
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

// Block (c, h, kv) takes the pieces of pages that begin in rows [c rows_per_block, ...): a piece is what a call writes of one page,
// and begins at a sequence's first row or at a page's first token.
template <int F32, int FMT>
__global__ void __launch_bounds__(kAppendThreads) k_kv_append(const KvArgs a, const void* __restrict__ qkv, int n_heads,
                                                              int rows_per_block) {
  __shared__ uint32_t red[32];
  const int h = blockIdx.y, is_v = blockIdx.z, P = 1 << a.page_shift;
  const int vecs = a.dh >> 3;  // vectors of 8 of a token
  const int64_t width = (int64_t)(n_heads + 2 * a.hkv) * a.dh;
  const int64_t col = (int64_t)(n_heads + is_v * a.hkv + h) * a.dh;
  uint8_t* codes = is_v ? a.v : a.k;
  uint8_t* scales = is_v ? a.v_scale : a.k_scale;
  const int64_t r0 = (int64_t)blockIdx.x * rows_per_block;
  const int end = (int)min(r0 + rows_per_block, a.T);
  bool nonfinite = false;
  for (int row = (int)r0; row < end;) {
    const int s = kv_find(a, row);
    if (s < 0) { ++row; continue; }
    const KvSeq q = kv_seq(a, s);
    if (row < q.first || row >= q.first + q.n) {  // behind the last sequence, or rows that are not in order
      ++row;
      continue;
    }
    const int pos = q.pos(row);
    if (pos < 0) {  // padding
      row += min(-pos, q.first + q.n - row);
      continue;
    }
    const int slot = pos & (P - 1);
    const int m = min(P - slot, q.first + q.n - row);  // tokens of this page from here on
    if (row != q.first && slot != 0) {  // the piece began in an earlier block
      row += m;
      continue;
    }
    const int id = kv_page(a, s, pos >> a.page_shift);
    const int first = row;
    row += m;
    if (id < 0) continue;
    const int64_t ph = (int64_t)id * a.hkv + h;
    const int was = slot ? (int)scales[ph] - 127 : 0;
    uint8_t* page = codes + (ph << a.page_shift) * a.dh;
    const int n = m * vecs;
    In8<F32> held[kHeld];
    uint32_t amax = 0;
    for (int i = threadIdx.x, k = 0; i < n; i += kAppendThreads, ++k) {
      const int t = i / vecs;
      In8<F32> x;
      x.load(qkv, (int64_t)(first + t) * width + col + (i - t * vecs) * 8);
      float v[8];
      x.get(v);
      amax = max(amax, absmax8(v, nonfinite));
    }
    (void)held;
    amax = block_max_u32(amax, red);
    int X = mx_exponent<FMT>(amax);
    if (slot) X = max(X, was);
    const float scale = pow2_neg(X);
    for (int i = threadIdx.x; i < n; i += kAppendThreads) {
      const int t = i / vecs;
      In8<F32> x;
      x.load(qkv, (int64_t)(first + t) * width + col + (i - t * vecs) * 8);
      float v[8];
      x.get(v);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = abs_bits(v[k]) >= kInf ? __uint_as_float(0x7FC00000u) : __fmul_rn(v[k], scale);
      *reinterpret_cast<uint2*>(page + (int64_t)slot * a.dh + i * 8) =
          make_uint2(cvt_fp8x4<FMT>(v[0], v[1], v[2], v[3]), cvt_fp8x4<FMT>(v[4], v[5], v[6], v[7]));
    }
    if (slot && X > was) {  // the tokens that were there, to the new scale
      const float down = pow2_down(was - X);
      for (int i = threadIdx.x; i < slot * vecs; i += kAppendThreads) {
        uint2* p = reinterpret_cast<uint2*>(page + i * 8);
        const uint2 w = *p;
        *p = make_uint2(shift4<FMT>(w.x, down), shift4<FMT>(w.y, down));
      }
    }
    if (threadIdx.x == 0 && (!slot || X != was)) scales[ph] = (uint8_t)(X + 127);
  }
  if (nonfinite) atomicOr(a.status, kStatusNonfinite);
}

// One thread: 8 codes of one row.
template <int F32, int FMT>
__global__ void __launch_bounds__(256) k_kv_read(const KvArgs a, void* __restrict__ kv) {
  const int vecs = 2 * a.hkv * a.dh / 8;
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= a.T * vecs) return;
  const int row = (int)(i / vecs), e = (int)(i - (int64_t)row * vecs) * 8;
  const int s = kv_find(a, row);
  if (s < 0) return;
  const KvSeq q = kv_seq(a, s);
  if (row < q.first || row >= q.first + q.n) return;
  const int pos = q.pos(row);
  uint2 w = make_uint2(0u, 0u);
  float scale = 1.0f;
  if (pos >= 0) {
    const int id = kv_page(a, s, pos >> a.page_shift);
    if (id >= 0) {
      const int head = e / a.dh, is_v = head >= a.hkv;
      const int64_t ph = (int64_t)id * a.hkv + head - is_v * a.hkv;
      scale = e8m0((is_v ? a.v_scale : a.k_scale)[ph]);
      const int slot = pos & ((1 << a.page_shift) - 1);
      w = *reinterpret_cast<const uint2*>((is_v ? a.v : a.k) + ((ph << a.page_shift) + slot) * a.dh + e - head * a.dh);
    }
  }
  float v[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t h2 = f16x2_of<FMT>((k < 2 ? w.x : w.y) >> (16 * (k & 1)));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
    v[2 * k] = f.x * scale;
    v[2 * k + 1] = f.y * scale;
  }
  const int64_t o = (int64_t)row * (vecs * 8) + e;
  if (F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(kv) + o);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(kv) + o) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
}

}  // namespace

cudaError_t launch_kv_append(const KvArgs& a, const void* qkv, int f32, int n_heads, const Launch& L) {
  const int rows = 1 << a.page_shift;
  const dim3 grid((unsigned)((a.T + rows - 1) / rows), (unsigned)a.hkv, 2);
  auto* k = f32 ? (a.fmt ? k_kv_append<1, 1> : k_kv_append<1, 0>) : (a.fmt ? k_kv_append<0, 1> : k_kv_append<0, 0>);
  k<<<grid, kAppendThreads, 0, L.stream>>>(a, qkv, n_heads, rows);
  if (L.launches) ++*L.launches;
  return cudaGetLastError();
}

cudaError_t launch_kv_read(const KvArgs& a, void* kv, int f32, const Launch& L) {
  const int64_t n = a.T * (2 * a.hkv * a.dh / 8);
  const unsigned grid = (unsigned)((n + 255) / 256);
  auto* k = f32 ? (a.fmt ? k_kv_read<1, 1> : k_kv_read<1, 0>) : (a.fmt ? k_kv_read<0, 1> : k_kv_read<0, 0>);
  k<<<grid, 256, 0, L.stream>>>(a, kv);
  if (L.launches) ++*L.launches;
  return cudaGetLastError();
}

}  // namespace fp8q
