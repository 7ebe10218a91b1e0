// C-ABI of the paged-cache operators: argument validation and workspace layout.  Every check here runs on the
// host before anything is enqueued.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/mr.h"
#include "paged.h"

using namespace mr;

namespace {

mr_status from_cuda(cudaError_t e) { return e == cudaSuccess ? MR_OK : MR_ERR_CUDA; }

constexpr int kMaxHeads = 1024;

// An address that is there and that the kernels may read and write in steps of `bytes`.
bool aligned(const void* p, uintptr_t bytes) { return p && (uintptr_t)p % bytes == 0; }

mr_status cache_ok(const mr_kv_cache* c) {
  if (!c) return MR_ERR_INVALID_ARG;
  if (c->dt != MR_BF16 && c->dt != MR_F32) return MR_ERR_UNSUPPORTED;
  if (c->H_kv < 1 || c->page_rows < 1 || c->n_pages < 1) return MR_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128) return MR_ERR_UNSUPPORTED;
  if (c->H_kv > kMaxHeads) return MR_ERR_UNSUPPORTED;
  const int64_t most = ((int64_t)1 << 31) - 1;
  if (c->n_pages > most / c->H_kv / c->page_rows) return MR_ERR_UNSUPPORTED;
  return MR_OK;
}

mr_status pools_ok(const mr_kv_cache* c) {
  return aligned(c->k, 16) && aligned(c->v, 16) ? MR_OK : MR_ERR_INVALID_ARG;
}

mr_status seqs_ok(const mr_kv_seqs* s) {
  if (!s || !aligned(s->table, 4) || !aligned(s->kv_len, 4) || s->pages_per_seq < 1 || s->n_seq < 1)
    return MR_ERR_INVALID_ARG;
  return MR_OK;
}

// strides of a tensor of `heads` x `rows` rows of d elements; an output's rows must not overlap
bool rows_ok(const mr_rows* r, int heads, int64_t rows, int d, int esize, bool output) {
  if (!r || !r->ptr || r->head_stride < 0 || r->row_stride < 0) return false;
  if ((uintptr_t)r->ptr % (uintptr_t)esize) return false;
  // every byte offset stays far inside 64 bits
  const int64_t most = (int64_t)1 << 56;
  if (heads > 1 && r->head_stride > most / heads) return false;
  if (rows > 1 && r->row_stride > most / rows) return false;
  if (!output) return true;
  const int64_t hs = r->head_stride, rs = r->row_stride;
  if (heads > 1 && hs < d) return false;
  if (rows > 1 && rs < d) return false;
  if (heads > 1 && rows > 1 && hs < (rows - 1) * rs + d && rs < (int64_t)(heads - 1) * hs + d) return false;
  return true;
}

PagedKv view(const mr_kv_cache* c, const mr_kv_seqs* s) {
  PagedKv v;
  v.k = c->k;
  v.v = c->v;
  v.table = s->table;
  v.kv_len = s->kv_len;
  v.H_kv = c->H_kv;
  v.page_rows = c->page_rows;
  v.d = c->d;
  v.n_pages = (int)c->n_pages;
  v.pages_per_seq = s->pages_per_seq;
  v.n_seq = s->n_seq;
  const int64_t cap = (int64_t)s->pages_per_seq * c->page_rows;
  v.capacity = cap < INT32_MAX ? (int)cap : INT32_MAX;
  v.by_rows = make_fastdiv((uint32_t)c->page_rows);
  return v;
}

int esize(mr_dtype dt) { return dt == MR_BF16 ? 2 : 4; }

bool rope_ok(const mr_rope* r) {
  return r && r->d >= 8 && r->d <= 256 && r->d % 8 == 0 && r->rot_dim >= 2 && r->rot_dim <= r->d &&
         r->rot_dim % 2 == 0 && isfinite(r->mscale);
}

// the kernels work in base 2: scale * log2(e) has to be finite, too
bool scale_ok(float scale) { return isfinite(scale * 1.4426950408889634f); }

// the status word in front of a workspace, cleared in stream order
cudaError_t reset_header(void* ws, cudaStream_t st) { return cudaMemsetAsync(ws, 0, sizeof(WsHeader), st); }

}  // namespace

extern "C" {

mr_status mr_rope_apply(const mr_rope* rope, const mr_rows* X, const mr_rows* Y, mr_dtype dt, int H,
                        int n_rows, const int32_t* pos, int adjoint, void* stream) {
  if (dt != MR_BF16 && dt != MR_F32) return MR_ERR_UNSUPPORTED;
  if (!rope_ok(rope) || H < 1 || n_rows < 0) return MR_ERR_INVALID_ARG;
  if (H > kMaxHeads) return MR_ERR_UNSUPPORTED;
  if (n_rows == 0) return MR_OK;
  if (!aligned(pos, 4)) return MR_ERR_INVALID_ARG;
  if (!rows_ok(X, H, n_rows, rope->d, esize(dt), false) || !rows_ok(Y, H, n_rows, rope->d, esize(dt), true))
    return MR_ERR_INVALID_ARG;
  if (X->ptr == Y->ptr && ((H > 1 && X->head_stride != Y->head_stride) || (n_rows > 1 && X->row_stride != Y->row_stride)))
    return MR_ERR_INVALID_ARG;
  RopeArgs a{rope, *X, *Y, dt, H, n_rows, pos, adjoint, (cudaStream_t)stream};
  return from_cuda(launch_rope(a));
}

size_t mr_paged_workspace_bytes(const mr_kv_cache* cache, int H_q, int n_seq) {
  if (cache_ok(cache) != MR_OK || H_q < 1 || H_q > kMaxHeads || H_q % cache->H_kv || n_seq < 1) return 0;
  const size_t dec = decode_workspace_bytes(cache->d), att = attn_workspace_bytes(cache->dt, cache->d);
  return dec > att ? dec : att;
}

mr_status mr_kv_append(const mr_kv_cache* cache, const mr_kv_seqs* seqs, const mr_rope* rope,
                       const mr_rows* Q, const mr_rows* Q_out, int H_q, const mr_rows* K,
                       const mr_rows* V, const int32_t* cu_q, int total_q, void* ws, size_t ws_bytes,
                       void* stream) {
  mr_status e;
  if ((e = cache_ok(cache)) != MR_OK || (e = pools_ok(cache)) != MR_OK || (e = seqs_ok(seqs)) != MR_OK) return e;
  if (!aligned(ws, 16) || ws_bytes < kWsHeaderBytes || total_q < 0) return MR_ERR_INVALID_ARG;
  if (cu_q ? !aligned(cu_q, 4) : total_q != seqs->n_seq) return MR_ERR_INVALID_ARG;
  if (rope && (!rope_ok(rope) || rope->d != cache->d)) return MR_ERR_INVALID_ARG;
  if ((Q == nullptr) != (Q_out == nullptr)) return MR_ERR_INVALID_ARG;
  const int es = esize(cache->dt), d = cache->d;
  if (total_q > 0) {
    if (Q) {
      if (H_q < 1) return MR_ERR_INVALID_ARG;
      if (H_q > kMaxHeads) return MR_ERR_UNSUPPORTED;
      if (!rows_ok(Q, H_q, total_q, d, es, false) || !rows_ok(Q_out, H_q, total_q, d, es, true))
        return MR_ERR_INVALID_ARG;
      if (Q->ptr == Q_out->ptr && ((H_q > 1 && Q->head_stride != Q_out->head_stride) ||
                                   (total_q > 1 && Q->row_stride != Q_out->row_stride)))
        return MR_ERR_INVALID_ARG;
    }
    if (!rows_ok(K, cache->H_kv, total_q, d, es, false) || !rows_ok(V, cache->H_kv, total_q, d, es, false))
      return MR_ERR_INVALID_ARG;
  }
  cudaStream_t st = (cudaStream_t)stream;
  if (reset_header(ws, st) != cudaSuccess) return MR_ERR_CUDA;
  if (total_q == 0) return MR_OK;
  AppendArgs a;
  a.kv = view(cache, seqs);
  a.rope = rope;
  a.q = Q ? *Q : mr_rows{};
  a.q_out = Q ? *Q_out : mr_rows{};
  a.k_new = *K;
  a.v_new = *V;
  a.H_q = H_q;
  a.dt = cache->dt;
  a.cu_q = cu_q;
  a.total_q = total_q;
  a.ws = (WsHeader*)ws;
  a.stream = st;
  return from_cuda(launch_append(a));
}

mr_status mr_paged_decode(const mr_kv_cache* cache, const mr_kv_seqs* seqs, const mr_rows* Q, int H_q,
                          float scale, int window, int sinks, const mr_rows* O, float* lse, void* ws,
                          size_t ws_bytes, void* stream) {
  mr_status e;
  if ((e = cache_ok(cache)) != MR_OK || (e = pools_ok(cache)) != MR_OK || (e = seqs_ok(seqs)) != MR_OK) return e;
  if (H_q < 1 || H_q % cache->H_kv || window < 0 || sinks < 0 || !scale_ok(scale)) return MR_ERR_INVALID_ARG;
  if (H_q > kMaxHeads) return MR_ERR_UNSUPPORTED;
  const int es = esize(cache->dt), d = cache->d;
  if (!rows_ok(Q, H_q, seqs->n_seq, d, es, false) || !rows_ok(O, H_q, seqs->n_seq, d, es, true))
    return MR_ERR_INVALID_ARG;
  if (lse && !aligned(lse, 4)) return MR_ERR_INVALID_ARG;
  if (!aligned(ws, 16) || ws_bytes < mr_paged_workspace_bytes(cache, H_q, seqs->n_seq))
    return MR_ERR_INVALID_ARG;
  DecodeArgs a;
  a.kv = view(cache, seqs);
  a.cu_q = nullptr;
  a.n_rows = seqs->n_seq;
  a.q = *Q;
  a.o = *O;
  a.H_q = H_q;
  a.dt = cache->dt;
  a.scale = scale;
  a.window = window;
  a.sinks = sinks;
  a.lse = lse;
  a.ws = ws;
  a.few = FewRows{};
  a.stream = (cudaStream_t)stream;
  return from_cuda(launch_decode(a));
}

mr_status mr_paged_attn(const mr_kv_cache* cache, const mr_kv_seqs* seqs, const mr_rows* Q, int H_q,
                        const int32_t* cu_q, int total_q, float scale, int window, int sinks,
                        const mr_rows* O, float* lse, void* ws, size_t ws_bytes, void* stream) {
  mr_status e;
  if ((e = cache_ok(cache)) != MR_OK || (e = pools_ok(cache)) != MR_OK || (e = seqs_ok(seqs)) != MR_OK) return e;
  if (H_q < 1 || H_q % cache->H_kv || window < 0 || sinks < 0 || !scale_ok(scale)) return MR_ERR_INVALID_ARG;
  if (H_q > kMaxHeads) return MR_ERR_UNSUPPORTED;
  if (!aligned(cu_q, 4) || total_q < 0) return MR_ERR_INVALID_ARG;
  const int es = esize(cache->dt), d = cache->d;
  if (total_q > 0 && (!rows_ok(Q, H_q, total_q, d, es, false) || !rows_ok(O, H_q, total_q, d, es, true)))
    return MR_ERR_INVALID_ARG;
  if (lse && !aligned(lse, 4)) return MR_ERR_INVALID_ARG;
  if (!aligned(ws, 16) || ws_bytes < mr_paged_workspace_bytes(cache, H_q, seqs->n_seq))
    return MR_ERR_INVALID_ARG;
  AttnArgs a;
  a.kv = view(cache, seqs);
  a.q = total_q > 0 ? *Q : mr_rows{};
  a.o = total_q > 0 ? *O : mr_rows{};
  a.H_q = H_q;
  a.dt = cache->dt;
  a.cu_q = cu_q;
  a.total_q = total_q;
  a.scale = scale;
  a.window = window;
  a.sinks = sinks;
  a.lse = lse;
  a.ws = ws;
  a.stream = (cudaStream_t)stream;
  return from_cuda(launch_attn(a));
}

size_t mr_pages_copy_workspace_bytes(void) { return kWsHeaderBytes; }

mr_status mr_pages_copy(void* const* pools, int n_pools, int64_t page_bytes, int64_t n_pages,
                        const int32_t* pairs, int n_pairs, void* ws, size_t ws_bytes, void* stream) {
  if (!pools || n_pools < 1 || page_bytes < 16 || page_bytes % 16 || n_pages < 1 || n_pairs < 0)
    return MR_ERR_INVALID_ARG;
  if (!aligned(ws, 16) || ws_bytes < kWsHeaderBytes || (n_pairs > 0 && !aligned(pairs, 4))) return MR_ERR_INVALID_ARG;
  if (n_pages > INT32_MAX || page_bytes > ((int64_t)1 << 40)) return MR_ERR_UNSUPPORTED;
  for (int i = 0; i < n_pools; ++i)
    if (!aligned(pools[i], 16)) return MR_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  if (reset_header(ws, st) != cudaSuccess) return MR_ERR_CUDA;
  if (n_pairs == 0) return MR_OK;
  return from_cuda(launch_pages_copy(pools, n_pools, page_bytes, n_pages, pairs, n_pairs, (WsHeader*)ws, st));
}

}  // extern "C"
