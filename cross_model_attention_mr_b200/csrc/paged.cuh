// Device side of the paged cache: page lookup and the row a position lives in.
#pragma once

#include "paged.h"

namespace mr {

__device__ __forceinline__ uint32_t fast_div(uint32_t n, const FastDiv& f) {
  return (__umulhi(n, f.mul) + n) >> f.shift;
}

// Detail codes recorded beside MR_ERR_DEVICE_CHECK.
constexpr uint32_t kBadPage = 0xD01;      // page number outside the pool
constexpr uint32_t kTableShort = 0xD02;   // kv_len beyond the table
constexpr uint32_t kBadPair = 0xD03;      // page pair outside the pool, or in conflict with another

// Pool row of (sequence s, kv head g, row j < capacity), or -1 for a page outside the pool.  Rows are
// numbered over the whole pool (the host keeps that below 2^31); row r starts at r * d elements.
__device__ __forceinline__ int pool_row(const PagedKv& kv, int s, int g, int j) {
  const int pi = (int)fast_div((uint32_t)j, kv.by_rows);
  const int page = __ldg(kv.table + (int64_t)s * kv.pages_per_seq + pi);
  if ((uint32_t)page >= (uint32_t)kv.n_pages) return -1;
  return (page * kv.H_kv + g) * kv.page_rows + (j - pi * kv.page_rows);
}

// Whether the new rows are worked on as tokens of their own.  Every CTA of both kernels comes to the same answer.  Whole CTA
// of NT threads; sums: shared memory for 2 * NT / 32 values.
template <int NT>
__device__ __noinline__ bool as_tokens(const PagedKv& kv, const int32_t* cu, int total_q, int window, int sinks,
                                       const FewRows& few, int64_t* sums) {
  int64_t once = 0, all = 0;  // keys that the sequences' last rows see; times their new rows
  for (int s = threadIdx.x; s < kv.n_seq; s += NT) {
    const int q0 = min(max(__ldg(cu + s), 0), total_q);
    const int n = min(max(__ldg(cu + s + 1), q0), total_q) - q0;
    if (n == 0) continue;
    const int len = max(__ldg(kv.kv_len + s), 0), held = min(len, kv.capacity);
    const int lo = window > 0 ? min(max(len - window, 0), held) : 0;
    const int64_t seen = min(sinks, lo) + (held - lo);
    once += seen;
    all += seen * n;
  }
#pragma unroll
  for (int w = 16; w; w >>= 1) {
    once += __shfl_xor_sync(0xffffffffu, once, w);
    all += __shfl_xor_sync(0xffffffffu, all, w);
  }
  if ((threadIdx.x & 31) == 0) {
    sums[threadIdx.x >> 5] = once;
    sums[NT / 32 + (threadIdx.x >> 5)] = all;
  }
  __syncthreads();
  once = all = 0;
  for (int w = 0; w < NT / 32; ++w) {
    once += sums[w];
    all += sums[NT / 32 + w];
  }
  __syncthreads();  // the sums' place is free again
  return all - once <= few.extra || all <= few.times * once;
}

// Mask of the bf16 halves of w that are infinite or NaN (an exponent of all ones carries into the bit above when one is
// added to it).
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  return ((((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u) >> 15) * 0xffffu;
}

// Sequence of packed row t: the s with cu[s] <= t < cu[s + 1]; n_seq behind the last one, -1 in front of the first.
__device__ __forceinline__ int sequence_of(const int32_t* cu, int n_seq, int t) {
  int lo = -1, hi = n_seq;  // cu[lo + 1] <= t or lo = -1; cu[hi] > t or hi = n_seq
  while (hi - lo > 1) {
    const int m = lo + (hi - lo) / 2;
    if (__ldg(cu + m) <= t)
      lo = m;
    else
      hi = m;
  }
  return lo < 0 ? -1 : (lo == n_seq - 1 && __ldg(cu + n_seq) <= t ? n_seq : lo);
}

}  // namespace mr
