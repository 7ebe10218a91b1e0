// Copying pages of the cache's pools: for every pair, one page of each pool.
//
// Bound by memory: a page is read and written once.  A block moves a chunk of one page of one pool with
// 16-byte loads, kUnroll in flight per thread.  Whether a pair may be copied depends on all the others (the
// copies count as simultaneous), so each block compares its pair with the whole list first: at a few
// thousand pairs that is 32 KB out of L2 per chunk of up to 64 KB, and needs no second launch and no memory.  It
// grows with the square of the list: 10000 pairs of 32 KB take 118 us (100 for the copies alone), of 2 KB 83 us (6),
// 50000 of 2 KB 1.8 ms (31).
#include "paged.cuh"
#include "profile.h"

namespace mr {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 8;
constexpr int kPoolsPerLaunch = 256;             // pool pointers passed by value

struct Pools {
  void* p[kPoolsPerLaunch];
};

__global__ void __launch_bounds__(kThreads)
    k_pages_copy(const __grid_constant__ Pools pools, int64_t vecs_per_page, int64_t chunk, int64_t n_pages,
                 const int32_t* __restrict__ pairs, int n_pairs, WsHeader* ws) {
  const int k = blockIdx.x;
  const int src = __ldg(pairs + 2 * (int64_t)k), dst = __ldg(pairs + 2 * (int64_t)k + 1);
  bool bad = (uint32_t)src >= (uint64_t)n_pages || (uint32_t)dst >= (uint64_t)n_pages;
  if (src == dst && !bad) return;
  for (int j = threadIdx.x; j < n_pairs; j += kThreads) {
    const int s = __ldg(pairs + 2 * (int64_t)j), d = __ldg(pairs + 2 * (int64_t)j + 1);
    bad |= s != d && (d == src || (j < k && d == dst));  // (d == src cannot be the pair itself)
  }
  if (__syncthreads_or(bad ? 1 : 0)) {
    if (threadIdx.x == 0) set_status(ws, MR_ERR_DEVICE_CHECK, kBadPair);
    return;
  }
  const int64_t v0 = (int64_t)blockIdx.z * chunk, v1 = min(v0 + chunk, vecs_per_page);
  char* base = (char*)pools.p[blockIdx.y];
  const uint4* from = reinterpret_cast<const uint4*>(base) + (int64_t)src * vecs_per_page;
  uint4* to = reinterpret_cast<uint4*>(base) + (int64_t)dst * vecs_per_page;
  for (int64_t v = v0 + threadIdx.x; v < v1; v += kThreads * kUnroll) {
    uint4 x[kUnroll];
#pragma unroll
    for (int w = 0; w < kUnroll; ++w)
      if (v + w * kThreads < v1) x[w] = __ldcs(from + v + w * kThreads);
#pragma unroll
    for (int w = 0; w < kUnroll; ++w)
      if (v + w * kThreads < v1) __stcs(to + v + w * kThreads, x[w]);
  }
}

}  // namespace

cudaError_t launch_pages_copy(void* const* pools, int n_pools, int64_t page_bytes, int64_t n_pages,
                              const int32_t* pairs, int n_pairs, WsHeader* ws, cudaStream_t st) {
  const int64_t vecs = page_bytes / 16;
  const int64_t round = kThreads * kUnroll;
  int64_t chunk = round * 2;
  while ((vecs + chunk - 1) / chunk > 65535) chunk *= 2;
  for (int p0 = 0; p0 < n_pools; p0 += kPoolsPerLaunch) {
    Pools g{};
    const int n = n_pools - p0 < kPoolsPerLaunch ? n_pools - p0 : kPoolsPerLaunch;
    for (int i = 0; i < n; ++i) g.p[i] = pools[p0 + i];
    const dim3 grid((unsigned)n_pairs, (unsigned)n, (unsigned)((vecs + chunk - 1) / chunk));
    ProfScope ps(kKPagesCopy, st);
    k_pages_copy<<<grid, kThreads, 0, st>>>(g, vecs, chunk, n_pages, pairs, n_pairs, ws);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace mr
