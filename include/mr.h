/*
 * libmr: block-level top-p compression of causal attention maps and fused translated retrieval
 * for cross-model attention-map reuse, on NVIDIA B200 (sm_100a).
 *
 * The method is MapFlow ("Accelerating Cross-Model LLM Inference via Attention Map Reuse"):
 *   - a sender's per-head causal softmax maps are compressed once, per (layer, head, query
 *     block), to the smallest set of key blocks whose probability mass reaches p, and stored in
 *     Block Sparse Row form (sections 4 and 5.2, "Attention State Compressor");
 *   - a receiver head's map is a non-negative, normalised linear mix of sender heads' maps
 *     (section 3.3) and is applied to the receiver's values by one fused kernel that never writes
 *     the translated map to global memory (section 5.4, "Attention Retrieval with Fused Kernel").
 * mr_dense_ref is exact causal attention, softmax(QK^T/sqrt(d))V ("AttnCache Guide", section
 * "The Quadratic Self-Attention Cost"), for rows that are not reused and as the p = 1 reference.
 *
 * Conventions for every entry point:
 *   - All tensors are caller-owned device memory unless a parameter says "host".  The library
 *     allocates no memory and frees nothing.
 *   - Arguments are validated on the host before any launch; a rejected call returns
 *     MR_ERR_INVALID_ARG or MR_ERR_UNSUPPORTED and launches nothing.
 *   - Work is enqueued on `stream` (a cudaStream_t; NULL = the legacy default stream) with no
 *     host synchronisation.  Conditions found on the device (capacity overflow, a bounded wait
 *     that ran out, a failed device check) are recorded in a status word inside the workspace;
 *     read it with mr_sync_status.
 *   - No exception crosses the ABI.  Device code never traps or asserts.
 *   - Layouts are head-major and row-contiguous: element (h, row, c) of a [H][rows][dim]
 *     tensor is at ((h * rows) + row) * dim + c.
 */
#ifndef MR_H_
#define MR_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MR_OK = 0,
  MR_ERR_INVALID_ARG = 1,  /* null pointer, bad size or value (host check, nothing launched) */
  MR_ERR_UNSUPPORTED = 2,  /* well-formed but outside this build: dtype, head dim, block, length */
  MR_ERR_CAPACITY = 3,     /* the compressed map needs more tiles than capacity_tiles (device) */
  MR_ERR_CUDA = 4,         /* a CUDA runtime call or launch failed */
  MR_ERR_TIMEOUT = 5,      /* a bounded device-side wait ran out; the kernel returned early */
  MR_ERR_DEVICE_CHECK = 6, /* a device-side consistency check failed */
  MR_ERR_RANGE = 7         /* a row's logits span too wide a range for the fp32 exponent path */
} mr_status;

/*
 * Element types.  MR_FP8_E4M3 is a map value type only (inputs stay MR_BF16): MapFlow section 9,
 * "Compact representations for reusable attention state".  An fp8 map stores each value as e4m3
 * (IEEE-style, 4 exponent bits with bias 7, 3 mantissa bits) times a float scale per 32-row x 64-key
 * piece of a tile (mr_bsr.tile_scale).
 */
typedef enum { MR_BF16 = 0, MR_F32 = 1, MR_FP8_E4M3 = 2 } mr_dtype;

/*
 * Synthetic causal logit bias b(h, i, j), added to sigma * q_i.k_j for j <= i.  It stands in for
 * the attention-sink, local-window and retrieval-head patterns the AttnCache page describes
 * ("The Attention Map Redundancy Discovery").  b is the MAXIMUM of the terms that apply, 0 when
 * none applies:
 *   sink_bias    when j < sink_len                (sink_len = 0 disables it)
 *   window_bias  when i - j < window              (window = 0 disables it)
 *   kb_bias[h * n_kb + j / kb_block]  when that device float is finite (-inf = no bias).
 * For mr_dense_ref, i is the absolute position q_offset + row.  Pass NULL for "no bias".
 */
typedef struct {
  int32_t sink_len;
  float sink_bias;
  int32_t window;
  float window_bias;
  const float* kb_bias; /* device [n_heads][n_kb] or NULL */
  int32_t kb_block;     /* keys per kb_bias entry (> 0 when kb_bias != NULL) */
  int32_t n_kb;         /* entries per head row (>= ceil(keys / kb_block)) */
} mr_logit_bias;

/*
 * Block Sparse Row map of one layer's H_s sender heads (MapFlow section 4: "Block Sparse Row
 * format").  Rows are (head h, query block I), numbered u = h * nqb + I with nqb = L / block;
 * columns are key blocks J <= I, nkb = L / block, nkb_words = ceil(nkb / 32).
 * The caller fills H_s, L, block, val_dtype, capacity_tiles and the pointers; mr_compress fills
 * the arrays.
 *   row_ptr   int32  [H_s * nqb + 1]  exclusive prefix sum of kept counts (row_ptr[0] = 0)
 *   col_idx   int32  [capacity_tiles] kept key-block indices, ascending within each row
 *   vals      [capacity_tiles][block * block] probabilities in val_dtype; tile t belongs to
 *             the row u with row_ptr[u] <= t < row_ptr[u+1] and column col_idx[t]; element (a, b)
 *             of a tile is the probability of query I*block + a on key J*block + b; entries above
 *             the causal diagonal are 0.  Values are not renormalised.  Storage order inside a
 *             tile: panels of P = 128 / sizeof(element) columns, each panel holding its `block`
 *             rows of 128 bytes in turn; in row a, the 16-byte chunk c of the panel is stored at
 *             chunk position c ^ (a % 8).  So element (a, b) sits at
 *               (b / P) * block * P + a * P + E * (((b % P) / E) ^ (a % 8)) + b % E,
 *             E = 16 / sizeof(element).  (Each panel is a 128-byte-swizzled MMA operand.)
 *             MR_FP8_E4M3 tiles are stored in panels of 64 columns, each panel holding its `block`
 *             rows of 64 bytes in turn with no swizzle, and within every group of 4 columns the
 *             bytes ordered (0, 2, 1, 3): element (a, b) at
 *               (b / 64) * block * 64 + a * 64 + (b % 64) - (b % 4) + perm(b % 4), perm = {0, 2, 1, 3},
 *             and the value is e4m3(a, b) * tile_scale[t * S + (a / 32) * (block / 64) + b / 64],
 *             S = (block / 32) * (block / 64) scales per tile.
 *             mr_bsr_export converts tiles to plain row-major fp32.
 *   kept_mass float  [H_s * nqb]      mass of the kept blocks (fp64 sum, rounded to fp32)
 *   kept_bits uint32 [H_s * nqb][nkb_words]  bit (J % 32) of word J / 32 set iff block J kept
 *   mass      float  [H_s * nqb][nkb] optional block masses (NULL = not written); J > I is 0
 *   lse       float  [H_s][L]         optional natural-log row normaliser log(sum_j exp(s_ij))
 *   nnz       int64  [1]              number of kept tiles (may exceed capacity_tiles)
 *   tile_scale float [capacity_tiles][S]  MR_FP8_E4M3 maps only (else unused, may be NULL): the
 *             scale of each 32-row x 64-key piece, max(piece) / 448 (448 = largest e4m3 value)
 *   renormalised  set by the caller before mr_compress: 0 stores the kept probabilities as they
 *             are (each row of the map then sums to its kept mass, at most 1); 1 stores every row
 *             divided by its kept mass, so a head's kept probabilities of each query sum to 1 (the
 *             renormalised top-p map; the pages leave renormalisation open).  Masses, selection and
 *             lse are the same either way.
 */
typedef struct {
  int32_t H_s;
  int32_t L;
  int32_t block;
  mr_dtype val_dtype;
  int64_t capacity_tiles;
  int32_t* row_ptr;
  int32_t* col_idx;
  void* vals;
  float* kept_mass;
  uint32_t* kept_bits;
  float* mass;
  float* lse;
  int64_t* nnz;
  float* tile_scale;
  int32_t renormalised;
} mr_bsr;

/* Library version (major * 100 + minor). */
int mr_version(void);

/* Human-readable name of a status code (static string). */
const char* mr_status_string(mr_status s);

/* 1 when the current device is sm_100 (B200-class) and the kernels can run, else 0. */
int mr_device_supported(void);

/*
 * 1 in the bounds-checked build of the library (libmr_checked.so), else 0.  That build checks the
 * index of every global store of the tensor-core kernels, and of every map read whose index comes
 * from device data, against the extents passed in; a miss skips the access and records
 * MR_ERR_DEVICE_CHECK with a site code in the workspace status.  Same entry points and results.
 */
int mr_checked_build(void);

/*
 * Workspace bytes mr_compress needs for this shape (device memory, 256-byte aligned, contents
 * need no initialisation).  Returns 0 for an unsupported shape.
 */
size_t mr_compress_workspace_bytes(int H_s, int L, int d, int block);

/*
 * Worst-case tile count of a map of this shape: every causal tile kept,
 * H_s * nqb * (nqb + 1) / 2.  A capacity of this size can never overflow.
 */
int64_t mr_bsr_max_tiles(int H_s, int L, int block);

/*
 * Compress one layer: MapFlow sections 4 and 5.2.
 *   Q, K   [H_s][L][d] in dtype dt (MR_BF16: bf16; MR_F32: fp32)
 *   scale  logit scale sigma (pass 1/sqrt(d) for standard attention)
 *   p      top-p threshold in (0, 1]; p >= 1 keeps every causal block.  The kept set of row
 *          (h, I) is the first k blocks of J = 0..I ordered by block mass descending (ties: the
 *          smaller J first), k the least count whose cumulative mass (fp64) is >= p.
 *          Block mass M_IJ = (1/block) * sum over the block's B x B probabilities.
 *   bias   optional logit bias (NULL = none); kb_bias rows are per sender head.
 *   out    map descriptor (see mr_bsr); out->H_s, L, block must equal the arguments.
 *   ws     workspace of at least mr_compress_workspace_bytes(H_s, L, d, block) bytes.
 * Supported: d in {64, 128}; block in {64, 128}; L a positive multiple of block with
 * L / block <= 256; H_s <= 64.  MR_BF16 maps use bf16 vals; MR_F32 maps use fp32 vals; bf16 inputs
 * with d = 128 may also write an MR_FP8_E4M3 map (out->val_dtype = MR_FP8_E4M3, out->tile_scale
 * set), whose values carry the e4m3 rounding error (at most 2^-4 relative, plus 2^-10 of their
 * piece's scale below the normal range).
 * bf16 with d = 128 (and per-key-block biases, if any, on multiples of 32 keys) runs on the
 * tensor-core kernels; other shapes on the CUDA-core kernels.  Either way vals hold the tiles in
 * the 128-byte-panel layout described at mr_bsr.
 * If the map needs more than capacity_tiles tiles, the status word records MR_ERR_CAPACITY and
 * no tile at or beyond capacity_tiles is written (nnz still reports the full count).
 */
mr_status mr_compress(const void* Q, const void* K, mr_dtype dt, int H_s, int L, int d,
                      float scale, float p, const mr_logit_bias* bias, mr_bsr* out, void* ws,
                      size_t ws_bytes, void* stream);

/*
 * mr_compress restricted to the query blocks qb_begin <= I < qb_end of every head (all heads, all
 * key blocks J <= I): MapFlow section 6 ("Chunked Prefill"), and the per-rank share of one sequence
 * split across GPUs by query-block range.  Rows of *out outside the range are written as empty
 * (count 0, no kept bits, kept mass 0); their row_ptr entries repeat the running total, so the
 * map is a valid BSR map of the whole layer whose only non-empty rows are the range's.  Row
 * normalisers in out->lse are written for the range's rows (and, for block 64, possibly for the
 * other block of a 128-row pair).  Needs the same workspace as mr_compress.  Requires
 * 0 <= qb_begin < qb_end <= L / block; mr_compress is this call with the full range.
 */
mr_status mr_compress_blocks(const void* Q, const void* K, mr_dtype dt, int H_s, int L, int d,
                             float scale, float p, const mr_logit_bias* bias, int qb_begin,
                             int qb_end, mr_bsr* out, void* ws, size_t ws_bytes, void* stream);

/*
 * Allocation-free variant of mr_compress.  The paper has no counterpart: this is a deployment
 * convenience of this library.
 *
 * Who needs it: callers that cannot allocate device memory, and so cannot hand mr_compress a
 * workspace.  Examples are code running inside a framework whose memory pool already owns the
 * GPU's memory (a raw allocation there fails or fragments the pool), plug-ins held to a fixed,
 * pre-planned memory budget, and serving loops that must not call the allocator once running.
 *
 * It computes exactly what mr_compress computes, with the same arguments except the workspace.
 * The scratch comes from one fixed array compiled into the library, of
 * MR_COMPRESS_NOALLOC_SCRATCH_BYTES bytes.  Every GPU that loads the library holds that array
 * until the process exits.  The call allocates and frees nothing; the caller still owns Q, K and
 * every array of *out.
 *   - Limit: shapes with mr_compress_workspace_bytes(H_s, L, d, out->block) larger than the array
 *     are rejected with MR_ERR_UNSUPPORTED before any work is enqueued.  That allows
 *     H_s * L <= 1048576 rows and H_s * (L / block) <= 16384 query blocks, e.g. 32 heads of 32768
 *     tokens.
 *   - First call on a device: it looks up the array's device address with that device current.
 *     Make the first call on each device before any stream capture begins.
 *   - All calls share the one array, which keeps the last call's contents.  Each call clears the
 *     parts that must start at zero, in stream order.  Calls whose work can overlap on the GPU
 *     (other streams or other host threads without ordering between them) race on the array and
 *     corrupt each other's maps: order them.
 *   - There is no caller-visible workspace: read the status word of the most recent call with
 *     mr_compress_noalloc_status (capacity overflow, a bounded wait that ran out).
 *   - The array's device address is cached per device for the life of its CUDA context; after
 *     cudaDeviceReset the cached address is stale, so do not call this entry point again in a
 *     process that reset a device it used.
 */
#define MR_COMPRESS_NOALLOC_SCRATCH_BYTES (256 + 4194304 + 65536)
mr_status mr_compress_noalloc(const void* Q, const void* K, mr_dtype dt, int H_s, int L, int d,
                              float scale, float p, const mr_logit_bias* bias, mr_bsr* out,
                              void* stream);

/*
 * Synchronise `stream` and return the device-side status that the most recent
 * mr_compress_noalloc call on the current device recorded in the fixed scratch array (MR_OK if
 * nothing failed).  Calls on other streams without ordering to `stream` may overwrite it.
 */
mr_status mr_compress_noalloc_status(void* stream);

/*
 * Workspace bytes mr_retrieve needs (device memory, 256-byte aligned): the status header and one
 * progress counter per CTA, which the CTAs of a schedule group read to stay together (the ones
 * that read the same map tiles then find them in L2).  mr_retrieve zeroes it before its launch;
 * calls that overlap on the GPU need separate workspaces.
 */
size_t mr_retrieve_workspace_bytes(const mr_bsr* map, int H_r, int d_v, int n_req);

/*
 * Options of mr_retrieve (pass NULL for the defaults: every query block, one V head per receiver
 * head).
 *   qb_begin, qb_end  compute only the output rows of query blocks qb_begin <= I < qb_end
 *                     (MapFlow section 6, "Chunked Prefill"; also one rank's share of a sequence
 *                     split across GPUs).  Output rows outside the range are not written.  Both 0:
 *                     every query block.  Otherwise 0 <= qb_begin < qb_end <= L / block.
 *   v_group           receiver heads that share one value head (grouped-query attention): receiver
 *                     head r reads value head r / v_group.  0 or 1: one value head per receiver
 *                     head.  H_r must be a multiple of v_group.
 *   v_pages           paged values (MapFlow section 6, "PagedAttention"), or NULL: device int32
 *                     [n_req][pages_per_req] page numbers.  Token j of request q is row
 *                     j % page_rows of page v_pages[q * pages_per_req + j / page_rows], and V is a
 *                     pool of pages laid out [page][H_v][page_rows][d_v] (H_v = H_r / v_group), so
 *                     element (q, g, j, c) is at
 *                     V + ((page * H_v + g) * page_rows + j % page_rows) * d_v + c.
 *                     v_req_off, v_req_stride and v_head_stride are then ignored.  page_rows: a
 *                     positive multiple of 64; pages_per_req * page_rows >= L.  A page number whose
 *                     rows fall outside [0, v_elems) reads zeros and records MR_ERR_DEVICE_CHECK.
 */
typedef struct {
  int32_t qb_begin;
  int32_t qb_end;
  int32_t v_group;
  const int32_t* v_pages;
  int32_t page_rows;
  int32_t pages_per_req;
} mr_retrieve_opts;

/*
 * Fused translated retrieval: MapFlow sections 3.3 and 5.4.
 *   O_r[i] = sum_{j <= i} ( sum_s W[r][s] * A_s[i][j] * [key block of j kept for (s, block of i)] )
 *            * V_g(r)[j],   g(r) = r / v_group
 * for every receiver head r < H_r, query row i < map->L (or of the options' query-block range) and
 * request q < n_req.  The translated map is formed tile by tile on chip and never written to
 * global memory.
 *   map     a map filled by mr_compress (its vals dtype equals dt, or is MR_FP8_E4M3 with dt = MR_BF16;
 *           fp8 maps are mixed in half precision from their e4m3 values)
 *   W       device fp32 [H_r][H_s], row r = receiver head r's weights over sender heads
 *   V       values in dtype dt: element (q, g, j, c) of value head g at
 *           V + v_off(q) + g * v_head_stride + j * d_v + c,
 *           v_off(q) = v_req_off[q] (device int64 array) or q * v_req_stride when v_req_off is NULL
 *   v_elems number of elements of the V allocation.  Every value read stays below it: the host
 *           checks strided layouts before launch (MR_ERR_INVALID_ARG); with a device offset table,
 *           a request whose rows do not fit inside [0, v_elems) (or, on the tensor-core kernel,
 *           whose offset is not a multiple of d_v) reads zeros instead and records
 *           MR_ERR_DEVICE_CHECK in the status word.  The tensor-core mixing kernel (bf16 maps of
 *           128-key blocks, at most 32 sender heads) also records MR_ERR_DEVICE_CHECK, writing no
 *           output, if the device places its dynamic shared memory off a 1024-byte boundary.
 *   O       output in dtype dt: element (q, r, i, c) at O + q * H_r * L * d_v + (r * L + i) * d_v + c
 *   opts    NULL or mr_retrieve_opts
 *   ws      workspace of at least mr_retrieve_workspace_bytes(map, H_r, d_v, n_req) bytes
 * Supported: d_v in {64, 128}; H_r <= 256.  bf16 maps with d_v = 128, block 64 or 128 and
 * H_s <= 64 run on the tensor-core kernel; other shapes on the CUDA-core kernel.  Within the
 * tensor-core kernel, bf16 maps of 128-key blocks with H_s <= 32 and n_req <= 1 mix the sender
 * heads on the tensor core too (weights rounded to bf16, fp32 accumulation); other maps mix them
 * on the CUDA cores (bf16 maps in fp32, fp8 maps in half precision).
 * Tiles a map could not store (capacity overflow at compression) contribute nothing and set
 * MR_ERR_CAPACITY in the status word.
 */
mr_status mr_retrieve(const mr_bsr* map, const float* W, int H_r, const void* V, int64_t v_elems,
                      void* O, mr_dtype dt, int d_v, int n_req, const int64_t* v_req_off,
                      int64_t v_req_stride, int64_t v_head_stride, const mr_retrieve_opts* opts,
                      void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes mr_dense_ref needs (device memory). */
size_t mr_dense_ref_workspace_bytes(int n_seq);

/*
 * Exact causal attention over packed variable-length sequences ("AttnCache Guide": the
 * standard softmax(QK^T * scale)V), with the same logit bias rule:
 *   Q [H][total_q][d], K [H][total_k][d], V [H][total_k][d_v], O [H][total_q][d_v] (dtype dt)
 *   cu_q, cu_k  device int32 [n_seq + 1] row offsets of each sequence in Q/O and K/V
 *   q_offset    device int32 [n_seq] absolute position of each sequence's first query row
 *               within its keys (NULL = 0): row i of sequence s attends keys
 *               0 .. q_offset[s] + i, and requires q_offset[s] + len_q(s) <= len_k(s)
 *   total_q, total_k  host ints equal to cu_q[n_seq] and cu_k[n_seq] (the per-head row
 *               counts of the packed tensors; total_q also sizes the launch)
 * Supported: d, d_v in {64, 128}.  bf16 with d = d_v = 128 (and per-key-block biases, if any, on
 * multiples of 32 keys) runs on the tensor-core kernel; other shapes on the CUDA-core kernel.
 * Requires q_offset[s] + len_q(s) <= len_k(s) (not checked: device arrays).
 */
mr_status mr_dense_ref(const void* Q, const void* K, const void* V, void* O, mr_dtype dt, int H,
                       int d, int d_v, const int32_t* cu_q, const int32_t* cu_k,
                       const int32_t* q_offset, int n_seq, int total_q, int total_k, float scale,
                       const mr_logit_bias* bias, void* ws, size_t ws_bytes, void* stream);

/*
 * Synchronise `stream` and return the device-side status recorded in `ws` (MR_OK if nothing
 * failed).  Every entry point that takes a workspace clears its status word when it is enqueued,
 * so the result describes the most recent call that used `ws`.
 */
mr_status mr_sync_status(void* ws, void* stream);

/* Synchronise `stream` and copy the map's kept-tile count to *nnz_host (host pointer). */
mr_status mr_bsr_nnz(const mr_bsr* map, int64_t* nnz_host, void* stream);

/*
 * Convert the first n_tiles tiles of map->vals to fp32 row-major tiles
 * ([n_tiles][block][block], element (a, b) = probability of query a on key b of the tile),
 * whatever the internal storage order.  out is device memory.
 */
mr_status mr_bsr_export(const mr_bsr* map, int64_t n_tiles, float* out, void* stream);

/*
 * Prefix-hash block manager: MapFlow section 5.3 ("Block Manager") and section 1 (prefix-hash
 * indexing).  Host-side index from token prefixes to stored compressed maps.
 *
 * Row (h, I) of a layer's map depends only on the first (I + 1) * block tokens (the map is
 * causal), so the maps stored for one sequence serve the first k query blocks of every request
 * whose first k * block tokens are the same: retrieve those rows with mr_retrieve's query-block
 * range and compute the rest.  Prefixes are keyed by a chained 64-bit hash per block of tokens
 * and checked token by token, so a hash collision is never reported as a hit.
 *
 * The manager keeps copies of the mr_bsr descriptors, never the device arrays: the caller keeps
 * an entry's arrays alive until the manager reports the entry evicted (mr_bm_evicted), and frees
 * them then.  Entries carry reference counts (the insert and each successful lookup take one;
 * mr_bm_release drops one).  When the bytes of the held entries exceed the budget, the least
 * recently used entries without references are evicted.  All calls are thread-safe, host-only,
 * and touch no device memory.
 */
typedef struct mr_block_manager mr_block_manager;

/* New manager for maps of `block`-token blocks; budget_bytes 0 = no limit.  NULL on bad
 * arguments or when host memory runs out. */
mr_block_manager* mr_bm_create(int block, int64_t budget_bytes);
void mr_bm_destroy(mr_block_manager* bm);

/*
 * Register the maps of one sequence: tokens (host int32 [n_tokens]; whole blocks are indexed, a
 * partial last block is ignored) and one descriptor per layer (host array of n_layers, each with
 * this block size and L >= the indexed tokens).  map_bytes is what the entry counts against the
 * budget.  Returns the entry id (>= 0, holding one reference) or -mr_status.
 */
int64_t mr_bm_insert(mr_block_manager* bm, const int32_t* tokens, int n_tokens, const mr_bsr* maps,
                     int n_layers, int64_t map_bytes);

/*
 * Longest stored prefix of `tokens` in whole blocks: returns k, the number of leading query blocks
 * whose map rows can be reused (0 = none), and writes the entry that holds them to *entry (-1 when
 * k = 0), taking a reference on it.  Negative -mr_status on bad arguments.
 */
int mr_bm_lookup(mr_block_manager* bm, const int32_t* tokens, int n_tokens, int64_t* entry);

/* Copy of the descriptor of `layer` of an entry. */
mr_status mr_bm_map(mr_block_manager* bm, int64_t entry, int layer, mr_bsr* out);

/* Drop one reference of an entry (then evict to the budget if needed). */
mr_status mr_bm_release(mr_block_manager* bm, int64_t entry);

/* Ids of evicted entries not reported yet (oldest first, at most max_ids): their device arrays are
 * no longer referenced by the manager.  Returns how many were written. */
int mr_bm_evicted(mr_block_manager* bm, int64_t* ids, int max_ids);

/* out[5] = {entries, bytes held, lookups, lookups that hit, query blocks served by hits}. */
mr_status mr_bm_stats(mr_block_manager* bm, int64_t* out);

/*
 * ------------------------------------------------------------------------------------------------
 * The receiver's paged key-value cache: rotary positions, appending new rows, attention of new rows
 * over the cache (one token per sequence, or a chunk of rows), copying pages, and a host-side page
 * pool.  MapFlow section 6 ("PagedAttention", "Chunked Prefill", variable-length packing): a
 * receiver that reuses a prefix's maps still rotates and stores its own keys and values, computes
 * the rows behind the prefix exactly, and then decodes token by token.
 * ------------------------------------------------------------------------------------------------
 *
 * mr_rows: rows of a head-major tensor with explicit strides, in elements.  Element (h, row, c) is at
 * ptr + h * head_stride + row * row_stride + c, so both [H][rows][d] and [rows][H][d] buffers fit.
 * Strides must be >= 0; the heads and rows of an output must not overlap.
 */
typedef struct {
  void* ptr;
  int64_t head_stride;
  int64_t row_stride;
} mr_rows;

/*
 * A pool of pages, k and v each [n_pages][H_kv][page_rows][d] in dtype dt (the layout of
 * mr_retrieve's v_pages, so one value pool serves both).  k and v must be 16-byte aligned.
 * Supported: dt MR_BF16 or MR_F32; d in {64, 128}; H_kv >= 1; page_rows >= 1;
 * n_pages * H_kv * page_rows < 2^31.  (mr_retrieve needs page_rows to be a multiple of 64.)
 */
typedef struct {
  void* k;
  void* v;
  mr_dtype dt;
  int32_t H_kv;
  int32_t page_rows;
  int32_t d;
  int64_t n_pages;
} mr_kv_cache;

/*
 * The sequences of a call.  table: device int32 [n_seq][pages_per_seq]; row j of sequence s is row
 * j % page_rows of page table[s * pages_per_seq + j / page_rows].  kv_len: device int32 [n_seq], the
 * rows each sequence holds, the call's new rows included.  With n new rows, new row i has position
 * kv_len[s] - n + i.  Table entries behind the last row, and of pages whose rows are all outside the
 * window (and not among the sinks), are not used.
 * Conditions found on the device, all recorded as MR_ERR_DEVICE_CHECK: a used page number outside
 * [0, n_pages) (its rows read as zeros and are not written); kv_len beyond pages_per_seq * page_rows
 * (only the rows the table covers are read or written).  kv_len <= 0 is an empty sequence.
 */
typedef struct {
  const int32_t* table;
  const int32_t* kv_len;
  int32_t pages_per_seq;
  int32_t n_seq;
} mr_kv_seqs;

/*
 * Rotary positions.  The first rot_dim of a row's d elements are rotated in pairs, the rest are
 * copied: pair i (0 <= i < rot_dim / 2) is elements (i, i + rot_dim / 2), or (2i, 2i + 1) when
 * interleaved, and position p turns it by the angle p * f_i:
 *   y_a = mscale * (x_a cos(p f_i) - x_b sin(p f_i)),  y_b = mscale * (x_b cos(p f_i) + x_a sin(p f_i)).
 * turn[i] holds f_i / (2 pi) as a 64-bit binary fraction of a turn, so p * turn[i] modulo 2^64 is the
 * angle to 2^-32 turns at every 31-bit position.  Filled by mr_rope_init; plain data, copied freely.
 */
typedef struct {
  int32_t d;
  int32_t rot_dim;
  int32_t interleaved;
  float mscale;
  uint64_t turn[128];
} mr_rope;

/*
 * How f_i = base^(-2i / rot_dim) is changed for contexts longer than the model was trained on:
 *   MR_ROPE_LINEAR  f_i / factor
 *   MR_ROPE_BASE    base * factor^(rot_dim / (rot_dim - 2)) in place of base (rot_dim >= 4)
 *   MR_ROPE_RAMP    g_i f_i + (1 - g_i) f_i / factor, g_i = clamp((r_i - beta_slow) /
 *                   (beta_fast - beta_slow), 0, 1), r_i = orig_len f_i / (2 pi): pairs that turn more
 *                   than beta_fast times over orig_len positions stay, those below beta_slow turns
 *                   are stretched
 */
typedef enum { MR_ROPE_NONE = 0, MR_ROPE_LINEAR = 1, MR_ROPE_BASE = 2, MR_ROPE_RAMP = 3 } mr_rope_scaling;

/*
 * Fill *out (host).  d a positive multiple of 8, at most 256; rot_dim even, 2 <= rot_dim <= d; base > 1
 * and finite; factor > 0 (1 for MR_ROPE_NONE); MR_ROPE_RAMP: orig_len >= 1, beta_fast > beta_slow >= 0;
 * mscale finite.  inv_freq: NULL, or a host array of rot_dim / 2 finite angles per position in place
 * of base and scaling.  Every |f_i| must be below 2 pi (one turn per position).
 */
mr_status mr_rope_init(mr_rope* out, int d, int rot_dim, int interleaved, double base,
                       mr_rope_scaling scaling, double factor, int orig_len, double beta_slow,
                       double beta_fast, double mscale, const double* inv_freq);

/*
 * Y = rotation of X (dtype dt, H heads x n_rows rows of rope->d elements) by each row's position
 * pos[row] (device int32, 0 or more; a negative position turns the other way).  adjoint != 0 turns by
 * the opposite angle with the same mscale: the gradient with respect to X given Y's.  X == Y with
 * equal strides rotates in place; other overlaps are not allowed.  Arithmetic in fp32, one rounding
 * to dt.  Needs no workspace: it has no device-side conditions.
 */
mr_status mr_rope_apply(const mr_rope* rope, const mr_rows* X, const mr_rows* Y, mr_dtype dt, int H,
                        int n_rows, const int32_t* pos, int adjoint, void* stream);

/* Workspace bytes of mr_kv_append, mr_paged_decode and mr_paged_attn for a cache, H_q query heads and
 * n_seq sequences (device memory, 256-byte aligned; an address that is no multiple of 16 is refused).
 * 0 for an unsupported shape.  The contents need not be set before a call nor kept after it, but for
 * the status word; calls that can be under way at the same time (on other streams, or in graphs
 * replayed side by side) need a workspace each. */
size_t mr_paged_workspace_bytes(const mr_kv_cache* cache, int H_q, int n_seq);

/*
 * Append new rows to the cache: K rotated, V as it is, and rotate the queries into Q_out, in one
 * launch.  All tensors in cache->dt; K, V have H_kv heads, Q and Q_out H_q heads, total_q rows.
 *   rope   NULL: nothing is rotated (K copied; Q copied to Q_out).  Otherwise rope->d == cache->d.
 *   Q, Q_out  both NULL, or both given (the same tensor rotates in place)
 *   cu_q   device int32 [n_seq + 1] row offsets of each sequence in Q, K and V, ascending from 0, or
 *          NULL when every sequence has one new row (total_q == n_seq)
 *   total_q  host int, at least cu_q[n_seq]; rows at or behind cu_q[n_seq] are neither read nor
 *          written (their Q_out rows stay as they were)
 * Of the workspace only the first 256 bytes are used.
 * A new row whose position is negative (kv_len[s] below its new rows) is not stored, its Q_out row is
 * zero.  Sequences that share a page (after a fork) must not append into it: copy it first.
 */
mr_status mr_kv_append(const mr_kv_cache* cache, const mr_kv_seqs* seqs, const mr_rope* rope,
                       const mr_rows* Q, const mr_rows* Q_out, int H_q, const mr_rows* K,
                       const mr_rows* V, const int32_t* cu_q, int total_q, void* ws, size_t ws_bytes,
                       void* stream);

/*
 * Which rows a query at position p sees: row j when 0 <= j <= p and (window == 0, or j > p - window,
 * or j < sinks).  window 0: every earlier row.  sinks: first rows that stay visible outside the window.
 */

/*
 * Attention of one new token per sequence over its cached rows (its own included):
 *   O_h = sum_j softmax_j(scale * q_h.k_j) v_j over the rows j visible from position kv_len[s] - 1,
 * query head h reading key-value head h / (H_q / H_kv).  Q, O: H_q heads, row s for sequence s.
 *   lse  NULL or device fp32 [H_q][n_seq]: natural log of sum_j exp(scale * q.k_j)
 *   scale  finite, and so that scale * log2(e) is (up to 2.3e38 in magnitude)
 * A sequence without visible rows gets O = 0 and lse = -inf.  Rows that are not visible, stale rows of
 * the last page among them, do not influence the result whatever they hold (infinities and NaN too).
 * H_q must be a multiple of H_kv.  O may be Q (the same tensor).  Work is split along every sequence's length over the whole GPU
 * and joined in a fixed order: results do not vary from call to call.
 */
mr_status mr_paged_decode(const mr_kv_cache* cache, const mr_kv_seqs* seqs, const mr_rows* Q, int H_q,
                          float scale, int window, int sinks, const mr_rows* O, float* lse, void* ws,
                          size_t ws_bytes, void* stream);

/*
 * The same for a chunk of new rows per sequence (a prompt, or the rows behind a reused prefix), whose
 * keys and values are in the cache already.  cu_q: device int32 [n_seq + 1], ascending from 0; rows
 * cu_q[s] .. cu_q[s + 1] - 1 of Q and O belong to sequence s and have the positions kv_len[s] - n ..
 * kv_len[s] - 1.  total_q >= cu_q[n_seq]; rows of O and lse at or behind cu_q[n_seq] stay as they were.
 *   lse  NULL or device fp32 [H_q][total_q]
 * A row that sees nothing (a negative position) gets O = 0 and lse = -inf.  Rows of the cache that a new
 * row does not see do not influence its result, whatever they hold.  Probabilities enter the second
 * product in the cache's type (bf16: off by at most 2^-8 of themselves; calls of few rows, which run as
 * mr_paged_decode does: 2^-16); sums are fp32.  Scores are expected below 2^30 in magnitude.
 * Few rows (bf16: up to 16, fp32: up to 8, or 4 a sequence and 64 in all; in both, up to n_seq) run as
 * mr_paged_decode does where the lengths say that this reads little again; the choice depends on lengths, types and
 * heads only.
 * bf16 calls run on the tensor cores when page_rows is a multiple of 8, the rows of Q and O are 16-byte
 * aligned (addresses and strides) and Q's strides are above 0.  Others, and fp32, run on the CUDA cores, which
 * takes up to 30 times as long for many rows.
 * Q holds total_q rows; those at or behind cu_q[n_seq] may be read and do not count.  O may be Q (the same tensor).
 */
mr_status mr_paged_attn(const mr_kv_cache* cache, const mr_kv_seqs* seqs, const mr_rows* Q, int H_q,
                        const int32_t* cu_q, int total_q, float scale, int window, int sinks,
                        const mr_rows* O, float* lse, void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes mr_pages_copy needs (device memory, aligned as above). */
size_t mr_pages_copy_workspace_bytes(void);

/*
 * Copy pages: for every pair t, page pairs[2t + 1] <- page pairs[2t] in each of n_pools pools (the
 * k and v pools of every layer), all pools of n_pages pages of page_bytes bytes.  For forking (the
 * last page of a shared sequence before it is written) and for compacting a pool.
 *   pools   host array of n_pools device pointers, 16-byte aligned
 *   page_bytes  a positive multiple of 16
 *   pairs   device int32 [n_pairs][2]: source, destination
 * All pairs count as copied at once, so a pair is skipped and MR_ERR_DEVICE_CHECK recorded when its
 * source or destination lies outside [0, n_pages), when its source is another pair's destination or when
 * an earlier pair has the same destination.  A pair of a page with itself does nothing and counts for nothing.
 * One source may go to many destinations.  Every block compares its pair with the whole list: up to a few
 * thousand pairs this costs next to nothing, tens of thousands of small pages are quicker in several calls.
 */
mr_status mr_pages_copy(void* const* pools, int n_pools, int64_t page_bytes, int64_t n_pages,
                        const int32_t* pairs, int n_pairs, void* ws, size_t ws_bytes, void* stream);

/*
 * Page pool: which pages of a pool each sequence holds (host only; thread-safe; touches no device
 * memory).  Pages carry reference counts, so forked sequences share them until one of them writes.
 * Calls that return pairs give (source, destination) page numbers for mr_pages_copy, to be copied before
 * the pages are next read or written; until then the sources keep their content because the pool does
 * not hand them out again before the next call.  Functions that return a count or id return
 * -mr_status on an error, and change nothing then (MR_ERR_CAPACITY also when host memory runs out).
 */
typedef struct mr_page_pool mr_page_pool;

/* New pool of n_pages free pages of page_rows rows.  NULL on bad arguments or without host memory. */
mr_page_pool* mr_pp_create(int n_pages, int page_rows);
void mr_pp_destroy(mr_page_pool* pp);

/* New empty sequence: its id (>= 0). */
int64_t mr_pp_open(mr_page_pool* pp);

/* New sequence with the first `rows` rows of `seq`, sharing their pages: its id.  Refused as mr_pp_truncate is. */
int64_t mr_pp_fork(mr_page_pool* pp, int64_t seq, int rows);

/*
 * Make room for `rows` more rows of `seq`: takes free pages, and for a shared page that the new rows
 * would be written into a free page of its own.  Writes at most one pair to pair[2] (host int32) and
 * returns the number of pairs (0 or 1).  -MR_ERR_CAPACITY when there are too few free pages.
 */
int mr_pp_extend(mr_page_pool* pp, int64_t seq, int rows, int32_t* pair);

/*
 * Drop the last rows of `seq` so that `rows` remain; pages without rows are released.  Refused when
 * mr_pp_slide has given up a page that the next query (its position is `rows` or later) would see under
 * the window and sinks of the last mr_pp_slide, or the page of the last row that would remain.
 */
mr_status mr_pp_truncate(mr_page_pool* pp, int64_t seq, int rows);

/*
 * Release the pages of `seq` whose rows no later query sees under a window with sinks (window >= 1; the
 * next query's position is at least the rows held).  Their table entries become -1.  Returns how
 * many pages the sequence gave up.
 */
int mr_pp_slide(mr_page_pool* pp, int64_t seq, int window, int sinks);

/* End a sequence: its pages lose a reference each. */
mr_status mr_pp_close(mr_page_pool* pp, int64_t seq);

/*
 * Compact: renumber pages so that the pages in use are the first ones, and write the (source,
 * destination) pairs to pairs (host int32 [max_pairs][2]).  Returns the number of pairs, at most
 * max_pairs (the rest is left for a later call); sequences' tables change with it.
 */
int mr_pp_compact(mr_page_pool* pp, int32_t* pairs, int max_pairs);

/* Write the page numbers of `seq` to pages (host int32 [max_pages], the rest filled with -1) and its
 * rows to *rows (may be NULL).  Returns the sequence's page count; -MR_ERR_CAPACITY if max_pages is less. */
int mr_pp_table(mr_page_pool* pp, int64_t seq, int32_t* pages, int max_pages, int* rows);

/* out[4] = {pages, free pages, sequences, pages with more than one reference}. */
mr_status mr_pp_stats(mr_page_pool* pp, int64_t* out);

/*
 * Measurement hooks (not part of the method).  When profiling is enabled, every entry point
 * records a CUDA event on its stream before and after each kernel it launches; mr_profile_read
 * waits for the recorded events and reports, per kernel id, the summed elapsed milliseconds and
 * the launch count since profiling was enabled.  Kernel ids are stable small integers; their
 * names come from mr_kernel_name (NULL past the last id).
 */
int mr_profile_enable(int on);      /* returns the previous state; enabling clears the records */
int mr_profile_read(double* total_ms, int64_t* launches, int max_ids); /* host arrays; returns ids */
const char* mr_kernel_name(int id);
int64_t mr_kernel_launches(void);   /* kernels launched by this library in this process */

/*
 * Measurement kernel (not part of the method): the retrieval's map reads alone.  Walks `map` in
 * the retrieval's order (128-row blocks longest first; key blocks J <= I; the kept tile of every
 * sender head) and moves each stored tile into shared memory `readers` times (by `readers` CTAs
 * working on the same row block side by side, as the retrieval's receiver-head groups do) with
 * 16-byte asynchronous copies, doing no arithmetic; each of its 512 threads keeps up to
 * ring_slots copies in flight (even, 2 .. 24).  Time it on `stream`; bytes moved =
 * readers * stored tiles * tile bytes.  ws: at least 256 bytes (status header).
 */
mr_status mr_gather_probe(const mr_bsr* map, int readers, int ring_slots, void* ws, size_t ws_bytes,
                          void* stream);

/*
 * Failure-path test hook (not part of the method; process-wide, for tests).  Sets the limit of the
 * tensor-core dense kernel's protocol waits to wait_ns (0 = the default 2 s; its softmax
 * warpgroups wait twice as long, so the wait nearest a stall reports it) and, with
 * skip_arrive = 1, makes the softmax warpgroup of each CTA's first query tile withhold its first
 * "P ready" arrive, so the MMA warp's wait runs out: the call records MR_ERR_TIMEOUT (detail
 * 0x913) in the workspace's status word, drains its copies and MMAs, frees Tensor Memory and
 * returns, leaving the context usable.  mr_paged_attn's tensor-core kernel obeys the same two settings
 * (detail 0xA16).
 * mr_debug_set(0, 0) restores normal operation.  No GPU fault is involved.
 */
mr_status mr_debug_set(uint64_t wait_ns, int skip_arrive);

#ifdef __cplusplus
}
#endif

#endif /* MR_H_ */
