// Causal attention of a few rows a sequence over the 8-bit key/value cache.
#include <cuda_fp16.h>

#include "fp8q_kv.cuh"

namespace fp8q {

namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float block_reduce(float v, float* red, bool is_max) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float w = __shfl_xor_sync(0xFFFFFFFFu, v, o);
    v = is_max ? fmaxf(v, w) : v + w;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float r = red[0];
  for (int i = 1; i < kThreads / 32; ++i) r = is_max ? fmaxf(r, red[i]) : r + red[i];
  return r;
}

// One block: one row and one query head.  128 keys at a time: a key a thread for the scores, a column a thread for the sum.
template <int FMT>
__global__ void __launch_bounds__(kThreads) k_kv_attend_rows(const KvArgs a, const uint16_t* __restrict__ qkv, int n_heads,
                                                             float scale, uint16_t* att, float* lse) {
  __shared__ float q[128], p[kThreads], red[4];
  __shared__ int ids[kThreads];
  const int row = blockIdx.x, h = blockIdx.y, g = h / (n_heads / a.hkv), t = threadIdx.x;
  const int s = kv_find(a, row);
  if (s < 0) return;
  const KvSeq sq = kv_seq(a, s);
  if (row < sq.first || row >= sq.first + sq.n) return;
  const int keys = max(0, sq.pos(row) + 1);
  if (t < a.dh)
    q[t] = __uint_as_float((uint32_t)qkv[(int64_t)row * (n_heads + 2 * a.hkv) * a.dh + h * a.dh + t] << 16);
  float m = -INFINITY, l = 0.0f, o = 0.0f;
  for (int k0 = 0; k0 < keys; k0 += kThreads) {
    __syncthreads();
    const int key = k0 + t;
    float x = -INFINITY;
    int id = -1;
    if (key < keys) id = kv_page(a, s, key >> a.page_shift);
    if (id >= 0) {
      const int64_t ph = (int64_t)id * a.hkv + g;
      const uint8_t* kp = a.k + ((ph << a.page_shift) + (key & ((1 << a.page_shift) - 1))) * a.dh;
      x = 0.0f;
      for (int c = 0; c < a.dh; c += 2) {
        const uint32_t w = f16x2_of<FMT>(*reinterpret_cast<const uint16_t*>(kp + c));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
        x += f.x * q[c] + f.y * q[c + 1];
      }
      x *= e8m0(a.k_scale[ph]) * scale;
    }
    ids[t] = id;
    const float mn = fmaxf(m, block_reduce(x, red, true));
    const float ref = mn == -INFINITY ? 0.0f : mn;
    const float w = expf(x - ref), fade = expf(m - ref);
    p[t] = w;
    l = l * fade + block_reduce(w, red, false);
    o *= fade;
    m = mn;
    if (t < a.dh) {
      for (int k = 0; k < kThreads; ++k) {
        if (ids[k] < 0) continue;
        const int64_t ph = (int64_t)ids[k] * a.hkv + g;
        const uint32_t v = a.v[((ph << a.page_shift) + ((k0 + k) & ((1 << a.page_shift) - 1))) * a.dh + t];
        const uint32_t f = f16x2_of<FMT>(v);
        o += p[k] * __low2float(*reinterpret_cast<const __half2*>(&f)) * e8m0(a.v_scale[ph]);
      }
    }
  }
  if (t < a.dh) {
    const uint16_t bits = (uint16_t)pack_bf16x2(l == 0.0f ? 0.0f : o / l, 0.0f);
    att[((int64_t)row * n_heads + h) * a.dh + t] = bits;
  }
  if (t == 0) lse[(int64_t)h * a.T + row] = m + logf(l);
}

}  // namespace

size_t kv_attend_workspace_bytes(int64_t, int, int, int, int) { return 256; }

cudaError_t launch_kv_attend(const KvArgs& a, const uint16_t* qkv, int n_heads, uint16_t* att, float* lse, void*,
                             const Launch& L) {
  const dim3 grid((unsigned)a.T, (unsigned)n_heads);
  (a.fmt ? k_kv_attend_rows<1> : k_kv_attend_rows<0>)<<<grid, kThreads, 0, L.stream>>>(a, qkv, n_heads, 1.0f / sqrtf((float)a.dh),
                                                                                      att, lse);
  if (L.launches) ++*L.launches;
  return cudaGetLastError();
}

}  // namespace fp8q
