// Rotary positions of one or several axes on the packed qkv rows that the attention core reads.
//
// Pair i of a rotated head turns by the angle pos[axis(i)] freq(i).  The angle is kept as a phase in
// turns, a 64-bit fixed-point fraction: F = round(freq / (2 pi) 2^64) wraps modulo one turn, so
// pos * F modulo 2^64 is the phase's fraction for any 32-bit position (negative ones too), off by at
// most |pos| 2^-65 turns: no floating-point range reduction, and far positions lose nothing.  The
// top 32 bits, as a signed number of half-turns, go to sincospif.
#include "fp8q_common.cuh"
#include "fp8q_internal.h"

namespace fp8q {

namespace {

__device__ __forceinline__ void rope_sincos(int32_t pos, uint64_t F, float sign, float& s, float& c) {
  const uint64_t phase = (uint64_t)(int64_t)pos * F;
  const float half_turns = (float)(int32_t)(phase >> 32) * 4.656612873077392578125e-10f;  // 2^-31
  sincospif(half_turns, &s, &c);
  s *= sign;
}

template <int F32>
__global__ void __launch_bounds__(256) k_rope(const void* in, const RopePlan p, const int32_t* pos, int64_t T, int heads,
                                              int rot_heads, float sign, void* out) {
  const int64_t width = (int64_t)heads * p.dh;
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= T * width) return;
  const int64_t t = i / width;
  const int col = (int)(i - t * width), h = col / p.dh, c = col - h * p.dh;
  const int half = p.rot >> 1;
  if (h >= rot_heads || c >= p.rot) {
    if (in != out) {
      if (F32) static_cast<float*>(out)[i] = static_cast<const float*>(in)[i];
      else static_cast<uint16_t*>(out)[i] = static_cast<const uint16_t*>(in)[i];
    }
    return;
  }
  if (p.interleaved ? (c & 1) : (c >= half)) return;  // the pair's first element does both
  const int k = p.interleaved ? c >> 1 : c;
  const int64_t j = i + (p.interleaved ? 1 : half);
  float s, co;
  rope_sincos(pos[(int64_t)p.axis[k] * T + t], p.turn[k], sign, s, co);
  if (F32) {
    const float a = static_cast<const float*>(in)[i], b = static_cast<const float*>(in)[j];
    static_cast<float*>(out)[i] = a * co - b * s;
    static_cast<float*>(out)[j] = b * co + a * s;
  } else {
    const float a = __uint_as_float((uint32_t)static_cast<const uint16_t*>(in)[i] << 16);
    const float b = __uint_as_float((uint32_t)static_cast<const uint16_t*>(in)[j] << 16);
    static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(a * co - b * s);
    static_cast<__nv_bfloat16*>(out)[j] = __float2bfloat16_rn(b * co + a * s);
  }
}

}  // namespace

cudaError_t launch_rope(const void* in, int f32, const RopePlan& plan, const int32_t* pos, int64_t T, int n_heads,
                        int n_kv_heads, int inverse, void* out, const Launch& L) {
  const int heads = n_heads + 2 * n_kv_heads, rot_heads = n_heads + n_kv_heads;
  const int64_t n = T * heads * plan.dh;
  const float sign = inverse ? -1.0f : 1.0f;
  const unsigned grid = (unsigned)((n + 255) / 256);
  if (f32) k_rope<1><<<grid, 256, 0, L.stream>>>(in, plan, pos, T, heads, rot_heads, sign, out);
  else k_rope<0><<<grid, 256, 0, L.stream>>>(in, plan, pos, T, heads, rot_heads, sign, out);
  if (L.launches) ++*L.launches;
  return cudaGetLastError();
}

}  // namespace fp8q
