// Host-side launchers of the paged-cache operators (internal to the library; not part of the C-ABI).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace mr {

// Division by a host constant: n / d for 0 <= n < 2^31 (round-up multiplier of l + 32 bits, l =
// ceil(log2 d): Granlund and Montgomery, "Division by Invariant Integers using Multiplication", 1994).
struct FastDiv {
  uint32_t mul, shift, d;
};
inline FastDiv make_fastdiv(uint32_t d) {
  uint32_t l = 0;
  while (l < 32 && (1ull << l) < d) ++l;
  return FastDiv{(uint32_t)(((1ull << 32) * ((1ull << l) - d)) / d + 1), l, d};
}

// The cache and its sequences as the kernels see them.
struct PagedKv {
  void* k;
  void* v;
  const int32_t* table;
  const int32_t* kv_len;
  int H_kv, page_rows, d, n_pages, pages_per_seq, n_seq;
  int capacity;  // rows a table can hold: min(pages_per_seq * page_rows, 2^31 - 1)
  FastDiv by_rows;
};

// New rows of a chunk as tokens of their own (decode.cu) or in tiles (attn.cu, attn_tc.cu), decided on the device: as
// tokens where at most `extra` keys are read more often than once for each sequence, or `times` as many in all.
struct FewRows {
  int ask;  // 0: decided already
  int64_t extra, times;
};

struct AppendArgs {
  PagedKv kv;
  const mr_rope* rope;  // host; NULL = no rotation
  mr_rows q, q_out, k_new, v_new;  // q.ptr NULL: no queries
  int H_q;
  mr_dtype dt;
  const int32_t* cu_q;
  int total_q;
  WsHeader* ws;
  cudaStream_t stream;
};

struct RopeArgs {
  const mr_rope* rope;
  mr_rows x, y;
  mr_dtype dt;
  int H, n_rows;
  const int32_t* pos;
  int adjoint;
  cudaStream_t stream;
};

struct DecodeArgs {
  PagedKv kv;
  const int32_t* cu_q;  // NULL: one row per sequence; otherwise rows of a chunk, each as a token of its own
  int n_rows;
  mr_rows q, o;
  int H_q;
  mr_dtype dt;
  float scale;
  int window, sinks;
  float* lse;
  void* ws;  // decode_workspace_bytes: status header, join counters, partial results
  FewRows few;
  cudaStream_t stream;
};

struct AttnArgs {
  PagedKv kv;
  mr_rows q, o;
  int H_q;
  mr_dtype dt;
  const int32_t* cu_q;
  int total_q;
  float scale;
  int window, sinks;
  float* lse;
  void* ws;  // attn_workspace_bytes: status header, join counters, partial results
  cudaStream_t stream;
};

struct AttnParams;
constexpr int kAttnMaxCtas = 304;  // two per SM (148) at most; sizes counters and partial results

size_t attn_workspace_bytes(mr_dtype dt, int d);
size_t attn_tc_part_bytes(int d);  // partial results of the tensor-core kernel
// The tensor-core kernel, where it takes the call (false: it does not).
bool launch_attn_tc(const AttnArgs& a, AttnParams p, int sms, cudaError_t* result);
// chunks of at most max_heads query heads, and the new rows that a tile of `rows` query rows takes of each
void attn_split(AttnParams& p, int rows, int max_heads);
cudaError_t launch_attn(const AttnArgs& a);
size_t decode_workspace_bytes(int d);
cudaError_t launch_decode(const DecodeArgs& a);
cudaError_t launch_rope(const RopeArgs& a);
cudaError_t launch_append(const AppendArgs& a);
cudaError_t launch_pages_copy(void* const* pools, int n_pools, int64_t page_bytes, int64_t n_pages,
                              const int32_t* pairs, int n_pairs, WsHeader* ws, cudaStream_t st);

}  // namespace mr
