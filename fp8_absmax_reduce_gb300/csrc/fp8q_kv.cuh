// What the kernels of the 8-bit key/value cache share: a call's rows by sequence, checked.
#pragma once

#include "fp8q_common.cuh"
#include "fp8q_internal.h"

namespace fp8q {

// The rows [first, first + n) of sequence s, and the tokens that it has in the cache (the call's included).  Values that
// leave their bounds are reported and taken as no rows, and as no tokens.
struct KvSeq {
  int first, n, len;
  __device__ __forceinline__ int pos(int row) const { return len - n + (row - first); }
};
__device__ __forceinline__ KvSeq kv_seq(const KvArgs& a, int s) {
  KvSeq q;
  if (a.row_start) {
    const int r0 = a.row_start[s], r1 = a.row_start[s + 1];
    const bool ok = r0 >= 0 && r1 >= r0 && r1 <= a.T;
    if (!ok) atomicOr(a.status, kStatusBadCache);
    q.first = ok ? r0 : 0;
    q.n = ok ? r1 - r0 : 0;
  } else {
    q.first = s * a.rows;
    q.n = a.rows;
  }
  q.len = a.lens[s];
  if (q.len < 0 || q.len > a.max_pages << a.page_shift) {
    atomicOr(a.status, kStatusBadCache);
    q.len = 0;
  }
  return q;
}

// The last sequence that starts at or before `row` (with rows never decreasing, the one that owns it); -1 if none does.  By a whole
// warp: 32 starts at a time, two steps for 1000 sequences instead of ten.
__device__ __forceinline__ int kv_find_warp(const KvArgs& a, int row) {
  if (!a.row_start) return row / a.rows;
  const int lane = threadIdx.x & 31;
  int lo = -1, hi = a.n_seqs;  // row_start[lo] <= row < row_start[hi]
  while (hi - lo > 1) {
    const int step = (hi - lo + 32) / 33, at = lo + (lane + 1) * step;
    const unsigned le = __ballot_sync(0xFFFFFFFFu, at < hi && a.row_start[at < hi ? at : 0] <= row);
    const int n = __ffs(~le) ? __ffs(~le) - 1 : 32;  // starts that are not behind the row
    lo += n * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// Page p of sequence s; -1, and reported, where the table names none.
__device__ __forceinline__ int kv_page(const KvArgs& a, int s, int p) {
  const int id = a.pages[s * a.max_pages + p];
  if (id >= 0 && id < a.n_pages) return id;
  atomicOr(a.status, kStatusBadCache);
  return -1;
}

// 2^(code - 127) of an E8M0 code.
__device__ __forceinline__ float e8m0(uint32_t code) {
  return __uint_as_float(code ? code << 23 : 0x00400000u);
}

// Two codes as fp16, exactly (both formats are subsets of fp16).
template <int FMT>
__device__ __forceinline__ uint32_t f16x2_of(uint32_t codes) {
  uint32_t r;
  if (FMT == 0) asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)codes));
  else asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(r) : "h"((uint16_t)codes));
  return r;
}

}  // namespace fp8q
