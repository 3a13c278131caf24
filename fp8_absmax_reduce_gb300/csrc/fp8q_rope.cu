// Rotary positions of one or several axes on the packed qkv rows that the attention core reads.
//
// Pair i of a rotated head turns by the angle pos[axis(i)] freq(i).  The angle is kept as a phase in
// turns, a 64-bit fixed-point fraction: F = round(freq / (2 pi) 2^64) wraps modulo one turn, so
// pos * F modulo 2^64 is the phase's fraction for any 32-bit position (negative ones too), off by at
// most |pos| 2^-65 turns: no floating-point range reduction, and far positions lose nothing.  As a
// signed number of half-turns, rounded to fp32 from all 64 bits (small angles keep their digits), it goes to sincospif.
//
// Bound by memory: every element is read and written once (in place: the rotated heads alone).  A
// thread keeps the sines and cosines of 8 pairs of one token in registers and applies them to its
// share of the token's heads, two vectors of 8 columns a head, four heads' loads in flight (fp32 two: with four, the registers
// leave too few blocks; T = 2000, 56 heads of 128, 64 turned: 24 us so and 20 with two).
#include "fp8q_common.cuh"
#include "fp8q_internal.h"

namespace fp8q {

namespace {

__device__ __forceinline__ void rope_sincos(int32_t pos, uint64_t F, float sign, float& s, float& c) {
  const uint64_t phase = (uint64_t)(int64_t)pos * F;
  const float half_turns = (float)(int64_t)phase * 0x1p-63f;
  sincospif(half_turns, &s, &c);
  s *= sign;
}

// 8 consecutive elements as one (bf16) or two (fp32) 16-byte vectors.
template <int F32>
struct Vec8 {
  uint4 w[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + i * (F32 ? 4 : 2));
#pragma unroll
    for (int k = 0; k < (F32 ? 2 : 1); ++k) w[k] = q[k];
  }
  __device__ __forceinline__ void store(void* p, int64_t i) const {
    uint4* q = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p) + i * (F32 ? 4 : 2));
#pragma unroll
    for (int k = 0; k < (F32 ? 2 : 1); ++k) q[k] = w[k];
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    if (F32) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint4 u = w[F32 ? k : 0];
        v[4 * k] = __uint_as_float(u.x); v[4 * k + 1] = __uint_as_float(u.y);
        v[4 * k + 2] = __uint_as_float(u.z); v[4 * k + 3] = __uint_as_float(u.w);
      }
    } else {
      const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) { v[2 * k] = bf16_lo(u[k]); v[2 * k + 1] = bf16_hi(u[k]); }
    }
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    if (F32) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        w[F32 ? k : 0] = make_uint4(__float_as_uint(v[4 * k]), __float_as_uint(v[4 * k + 1]), __float_as_uint(v[4 * k + 2]),
                                    __float_as_uint(v[4 * k + 3]));
    } else {
      w[0] = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    }
  }
};

constexpr int kRopeThreads = 128, kRopeShare = 8;  // threads of a block; heads of a thread, where tokens are many

// rot_dim a multiple of 16.  A token has `units` * `slots` threads: thread (u, s) turns pairs 8u .. 8u+7
// of heads s, s + slots, ...; then the token's threads copy what is not rotated.
template <int F32, int INTER>
__global__ void __launch_bounds__(kRopeThreads) k_rope_vec(const void* in, const __grid_constant__ RopePlan p,
                                                           const int32_t* __restrict__ pos, int64_t T, int heads,
                                                           int rot_heads, int units, int slots, int tokens, float sign,
                                                           void* out) {
  constexpr int kHeads = F32 ? 2 : 4;  // in flight
  const int group = units * slots;
  const int tok = threadIdx.x / group, r = threadIdx.x - tok * group;
  const int64_t t = (int64_t)blockIdx.x * tokens + tok;
  if (tok >= tokens || t >= T) return;
  const int slot = r / units, u = r - slot * units;
  const int64_t base = t * heads * p.dh;
  const int c0 = INTER ? 16 * u : 8 * u, c1 = INTER ? c0 + 8 : c0 + (p.rot >> 1);
  Vec8<F32> a[kHeads], b[kHeads];
  auto load = [&](int h0) {
#pragma unroll
    for (int q = 0; q < kHeads; ++q) {
      const int h = h0 + q * slots;
      if (h < rot_heads) {
        a[q].load(in, base + h * p.dh + c0);
        b[q].load(in, base + h * p.dh + c1);
      }
    }
  };
  load(slot);  // in flight while the angles are computed
  float s[8], c[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int i = 8 * u + k;
    rope_sincos(pos[(int64_t)p.axis[i] * T + t], p.turn[i], sign, s[k], c[k]);
  }
  for (int h0 = slot; h0 < rot_heads; h0 += kHeads * slots) {
    if (h0 != slot) load(h0);
#pragma unroll
    for (int q = 0; q < kHeads; ++q) {
      const int h = h0 + q * slots;
      if (h < rot_heads) {
        float x[8], y[8], xo[8], yo[8];
        a[q].get(x);
        b[q].get(y);
        if (INTER) {  // x = pairs 0..3 as (a, b) neighbours, y = pairs 4..7
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            xo[2 * k] = x[2 * k] * c[k] - x[2 * k + 1] * s[k];
            xo[2 * k + 1] = x[2 * k + 1] * c[k] + x[2 * k] * s[k];
            yo[2 * k] = y[2 * k] * c[4 + k] - y[2 * k + 1] * s[4 + k];
            yo[2 * k + 1] = y[2 * k + 1] * c[4 + k] + y[2 * k] * s[4 + k];
          }
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            xo[k] = x[k] * c[k] - y[k] * s[k];
            yo[k] = y[k] * c[k] + x[k] * s[k];
          }
        }
        a[q].set(xo);
        b[q].set(yo);
        a[q].store(out, base + h * p.dh + c0);
        b[q].store(out, base + h * p.dh + c1);
      }
    }
  }
  if (in == out) return;
  // the rest: the v heads, one run of the row, and the rotated heads' columns from rot on; kCopies vectors in flight
  constexpr int kCopies = F32 ? 4 : 8;
  const int v_vecs = (heads - rot_heads) * p.dh / 8, tail = (p.dh - p.rot) / 8, all = v_vecs + tail * rot_heads;
  for (int i0 = r; i0 < all; i0 += kCopies * group) {
    Vec8<F32> v[kCopies];
    int at[kCopies];
#pragma unroll
    for (int q = 0; q < kCopies; ++q) {
      const int i = i0 + q * group;
      if (i < v_vecs) {
        at[q] = rot_heads * p.dh + 8 * i;
      } else if (i < all) {
        const int h = (i - v_vecs) / tail;
        at[q] = h * p.dh + p.rot + 8 * (i - v_vecs - h * tail);
      }
      if (i < all) v[q].load(in, base + at[q]);
    }
#pragma unroll
    for (int q = 0; q < kCopies; ++q)
      if (i0 + q * group < all) v[q].store(out, base + at[q]);
  }
}

// Any even rot_dim: one thread per element; a pair's first element does both.
template <int F32>
__global__ void __launch_bounds__(kRopeThreads) k_rope_any(const void* in, const __grid_constant__ RopePlan p,
                                                           const int32_t* pos, int64_t T, int heads, int rot_heads,
                                                           float sign, void* out) {
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
  if (p.interleaved ? (c & 1) : (c >= half)) return;
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

cudaError_t launch_rope(const void* in, int f32, const RopePlan& p, const int32_t* pos, int64_t T, int n_heads,
                        int n_kv_heads, int inverse, void* out, const Launch& L) {
  const int heads = n_heads + 2 * n_kv_heads, rot_heads = n_heads + n_kv_heads;
  const float sign = inverse ? -1.0f : 1.0f;
  if (p.rot % 16 == 0) {
    // Threads per token: enough slots that each thread has at most kRopeShare heads and 16 vectors to copy (T = 16384, 24
    // heads of 96, 48 turned: 35 us with heads alone counted, 28 so), and for few tokens more (down to one head a thread),
    // until the grid holds about 512 threads per SM.
    const int units = p.rot / 16, most = kRopeThreads / units;
    int64_t slots = (rot_heads + kRopeShare - 1) / kRopeShare;
    const int copies = in == out ? 0 : (heads * p.dh - rot_heads * p.rot) / 8;
    if (slots * 16 * units < copies) slots = (copies + 16 * units - 1) / (16 * units);
    const int64_t fill = ((int64_t)L.num_sms * 512 + T * units - 1) / (T * units);
    if (slots < fill) slots = fill;
    if (slots > rot_heads) slots = rot_heads;
    if (slots > most) slots = most;
    const int group = units * (int)slots, tokens = kRopeThreads / group;
    const unsigned grid = (unsigned)((T + tokens - 1) / tokens);
    auto* k = f32 ? (p.interleaved ? k_rope_vec<1, 1> : k_rope_vec<1, 0>)
                  : (p.interleaved ? k_rope_vec<0, 1> : k_rope_vec<0, 0>);
    k<<<grid, kRopeThreads, 0, L.stream>>>(in, p, pos, T, heads, rot_heads, units, (int)slots, tokens, sign, out);
  } else {
    const int64_t n = T * heads * p.dh;
    const unsigned grid = (unsigned)((n + kRopeThreads - 1) / kRopeThreads);
    (f32 ? k_rope_any<1> : k_rope_any<0>)<<<grid, kRopeThreads, 0, L.stream>>>(in, p, pos, T, heads, rot_heads, sign, out);
  }
  if (L.launches) ++*L.launches;
  return cudaGetLastError();
}

}  // namespace fp8q
