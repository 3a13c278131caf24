// What the two attention kernels over the 8-bit cache share (few rows a sequence: warp-level products; many: tensor memory):
// the line of work that they cut into equal parts, and the joining of units that were cut.
#pragma once

#include <cuda_fp16.h>

#include <atomic>

#include "fp8q_head.cuh"
#include "fp8q_kv.cuh"

namespace fp8q {

constexpr int kBlockKeys = 128;
constexpr int kMaxCtas = 152 * 5;
constexpr int kNoPage = 0x1000;   // in place of a scale: the keys are not seen
// A reference maximum (log2) from which on scores are rounded before it is taken from them.  One step, z f + (offset - m), rounds the offset
// away where m is large (half a unit of 2^-14 below 2^10), and leaves the maximum's own rounding in the exponent: from 2^24 on it
// would leave fp16's range upwards, or all weights would vanish.
constexpr float kLarge = 1024.0f;
__device__ __forceinline__ bool is_large(float m) { return fabsf(m) >= kLarge && m != -INFINITY; }
constexpr float kLn2 = 0.693147180559945309f, kLog2e = 1.44269504088896341f;

// What CTA j leaves behind when it begins a unit and does not end it.
struct Cut {
  int64_t first, end;  // the unit on the line; first = end: nothing
  int64_t total;       // of the line
  int ctas;            // parts of the line
  int head;            // K/V head
  int row0, rows;      // first row of the call, and rows (tokens times heads) of the tile
  int group_row;       // the tile's first (token, head) pair
};

struct AttendArgs {
  KvArgs kv;
  const uint16_t* qkv;
  int n_heads;
  float scale_log2;  // log2(e) / sqrt(head_dim)
  uint16_t* att;
  float* lse;
  float* part_o;     // [2 per CTA][R][DH]
  float2* part_sum;  // [2 per CTA][R]: the maximum (log2), and the sum over it; apart, as one would vanish in the other's rounding
  Cut* cuts;         // [CTAs]
  uint64_t wait_ns;  // limit of the waits of the kernel for many rows (0: 2 s)
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {  // to a unit in the last place
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^e, e between -126 and 127 or taken as the nearer of them: where what is below vanishes.
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(min(max(e, -126), 127) + 127) << 23); }
// 2^e down to the smallest subnormal number, and 0 below: a page's scale goes to 2^-127, the ratio of two to 2^-254.
__device__ __forceinline__ float pow2(int e) {
  return __uint_as_float(e >= -126 ? (uint32_t)(min(e, 127) + 127) << 23 : e < -149 ? 0u : 1u << (e + 149));
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Whether any of four codes is NaN or infinite.
template <int FMT>
__device__ __forceinline__ uint32_t nonfinite4(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + (FMT == 0 ? 0x01010101u : 0x04040404u)) & 0x80808080u;
}

// Where a CTA's part of the line begins: every CTA adds the line up by itself.
struct Line {
  int s;         // the sequence
  KvSeq q;
  int64_t base;  // its first block
};
// total j / ctas; a 64-bit division costs a third of a microsecond
__device__ __forceinline__ int64_t part(int64_t total, int j, int ctas) {
  return total < (1 << 21) ? (int64_t)((uint32_t)total * (uint32_t)j / (uint32_t)ctas) : total * j / ctas;
}

// A kernel's dynamic shared memory, once a device; `done` is that kernel's own.
template <class K>
cudaError_t kv_smem(K* kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (done.load(std::memory_order_relaxed) >> (dev & 63) & 1)) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(1ull << (dev & 63));
  return e;
}

// The kernel for many rows (fp8q_kvmany.cu): rows of its units, and its launch on `ctas` SMs.
int kv_attend_many_rows();
cudaError_t launch_kv_attend_many(const AttendArgs& p, int ctas, cudaStream_t s);

}  // namespace fp8q
