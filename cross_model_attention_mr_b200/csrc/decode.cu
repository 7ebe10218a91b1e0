// Attention of one new token per sequence over the paged cache: o_h = sum_j softmax_j(scale q_h.k_j) v_j.
//
// Bound by memory: each visible row of K and V is read once for all the query heads that share it, about
// 2 G operations a byte for groups of G heads, far below what the tensor cores do per byte read.  So the
// design is about keeping loads in flight and every SM equally busy:
//   * The visible rows of a sequence (first rows kept and the window) are numbered without the gap
//     between them and cut into tiles of 64.  The tiles of all (query row, kv head, chunk of up to 16 query
//     heads) units, one unit after the other, are split evenly over the CTAs, which need not begin or end
//     with a unit: ragged batches and single long sequences load the GPU alike.
//   * A CTA that holds a whole unit writes its output; the parts of a unit that several CTAs share go to the
//     workspace as (maximum, sum, unnormalised output), and the CTA that finishes last joins them, always in
//     the same order.  No CTA waits for another one.
//   * Within a CTA each of the 4 warps takes 16 rows of every tile and streams them through a ring of its own
//     with 16-byte asynchronous copies: no barrier between warps until the unit ends.  Rows that are not
//     visible are never read (zeros stand in for them), so nothing they hold can reach the result.
// bf16 uses the warp-level matrix instructions m16n8k16 (rows: query heads): a tile of 16 heads x 16 keys
// needs no more, and the 128-row tcgen05 tile would be filled to an eighth.  The scores' registers are the
// second product's operand as they are.  Probabilities are split into two bf16 parts (value and remainder)
// so that their rounding does not show beside the output's own; with up to 8 heads both parts share one
// instruction (rows 0-7 and 8-15).  A remainder may be 0 or negative, so an infinite value must not meet it: a warp
// whose sums come out infinite or NaN reads its rows a second time and leaves such values out of that product.  fp32
// runs on the CUDA cores.
// 8 sequences of 32768 rows, 64 heads in groups of 8 (1.07 GB): 177 to 182 us over several machines, 5.9 to 6.1 TB/s, 90 to
// 93% of a copy's rate; 16 sequences of 4608 to 6144 rows, 32 heads in groups of 4: 65 us, 5.4 TB/s.
#include <cuda_bf16.h>

#include "paged.cuh"
#include "profile.h"
#include "sm100.cuh"

namespace mr {
namespace {

using sm100::ex2_approx;
using sm100::smem_u32;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kSlice = 16;                 // rows a warp takes at a time
constexpr int kTile = kSlice * kWarps;
constexpr int kMaxRows = 16;               // query heads of a unit
constexpr int kMaxCtas = 304;              // two per SM (148) at most; sizes counters and partial slots
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Params {
  PagedKv kv;
  const void* q;
  void* o;
  int64_t q_head, q_row, o_head, o_row;  // strides in elements
  float* lse;
  const int32_t* cu;                     // NULL: row t is sequence t's
  int n_rows;
  int H_q, group, chunks, rows;          // chunks of `rows` query heads per kv head (the last may be shorter)
  int vec_q, vec_o;                      // rows aligned to 4 (Q) and 16 (O) bytes
  float a;                               // scale * log2(e)
  int window, sinks;
  FewRows few;
  WsHeader* ws;
  uint32_t* counters;                    // [kMaxCtas], zero at launch
  float* part;                           // [2 * kMaxCtas][kMaxRows * (d + 2)]
};

template <typename T, int D>
struct Cfg {
  static constexpr int kRowBytes = D * (int)sizeof(T);
  static constexpr int kChunks = kRowBytes / 16;               // 16-byte chunks of a row
  static constexpr int kRowsPerCopy = 32 / kChunks;            // rows a warp-wide copy covers
  static constexpr int kCopies = kSlice / kRowsPerCopy;
  static constexpr int kSliceBytes = 2 * kSlice * kRowBytes;   // K and V
  // slices on the way while one is worked on: 16 KB a warp (fp32 rows of 128: 32 KB)
  static constexpr int kStages = sizeof(T) == 2 && D == 64 ? 5 : 3;
  static constexpr int kRingBytes = kWarps * kStages * kSliceBytes;
};

// shared memory: [ring | q (fp32 only) | p (fp32 only)], the ring reused for merging and joining
template <typename T, int D>
constexpr int smem_bytes() {
  return Cfg<T, D>::kRingBytes + (sizeof(T) == 4 ? kMaxRows * D * 4 + kWarps * kMaxRows * (kSlice + 1) * 4 : 0);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&b);
}
// the part of (x, y) that pack2 rounds away
__device__ __forceinline__ uint32_t pack2_rest(float x, float y, uint32_t hi) {
  const float2 h = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&hi));
  return pack2(x - h.x, y - h.y);
}

// Query row t: its sequence (-1: none, the row is left alone) and how many cached rows it may see, itself included.
struct Query {
  int s, len;
};
__device__ __forceinline__ Query query(const Params& p, int t) {
  if (p.cu == nullptr) return Query{t, max(__ldg(p.kv.kv_len + t), 0)};
  const int s = sequence_of(p.cu, p.kv.n_seq, t);
  if (s < 0 || s >= p.kv.n_seq) return Query{-1, 0};
  const int64_t len = (int64_t)max(__ldg(p.kv.kv_len + s), 0) - (__ldg(p.cu + s + 1) - 1 - t);
  return Query{s, (int)min(max(len, (int64_t)0), (int64_t)INT32_MAX)};
}

// The cached rows a query sees: rows [0, first) and [lo, lo + n - first).
struct Visible {
  int n, first, lo;
};
__device__ __forceinline__ Visible visible(const Params& p, const Query& q) {
  const int held = min(q.len, p.kv.capacity);
  const int lo = p.window > 0 ? min(max(q.len - p.window, 0), held) : 0;
  const int first = min(p.sinks, lo);
  return Visible{first + held - lo, first, lo};
}

// A unit's part: tiles [t0, t1) of its nt.
struct Segment {
  int t;            // query row
  int s, g, chunk;  // sequence, kv head, chunk of query heads
  int rows, h0;     // its query heads
  int t0, t1, nt;
  Visible vis;
};

template <typename T, int D>
struct Stream {  // one warp's slices of a segment
  const Params& p;
  const Segment& sg;
  const int warp, lane;
  const uint32_t ring;  // shared address of this warp's ring
  int next_row;         // pool row of slice `ahead`, row (lane % 16)

  __device__ __forceinline__ int lookup(int t) const {
    const int x = t * kTile + warp * kSlice + (lane & 15);
    if (t >= sg.t1 || x >= sg.vis.n) return -1;
    const int j = x < sg.vis.first ? x : x - sg.vis.first + sg.vis.lo;
    const int r = pool_row(p.kv, sg.s, sg.g, j);
    if (r < 0) set_status(p.ws, MR_ERR_DEVICE_CHECK, kBadPage);
    return r;
  }
  // copy slice t into stage st with the row numbers looked up before, and look up the next slice's
  __device__ __forceinline__ void load(int t, int st) {
    using C = Cfg<T, D>;
    const int row = next_row;
    next_row = lookup(t + 1);
    if (t < sg.t1) {
      const uint32_t k_dst = ring + st * C::kSliceBytes, v_dst = k_dst + kSlice * C::kRowBytes;
      const int c = lane % C::kChunks;
#pragma unroll
      for (int i = 0; i < C::kCopies; ++i) {
        const int r = i * C::kRowsPerCopy + lane / C::kChunks;
        const int pr = __shfl_sync(0xffffffffu, row, r);
        const int64_t src = (int64_t)max(pr, 0) * C::kRowBytes + c * 16;
        const uint32_t off = r * C::kRowBytes + ((c ^ (r & 7)) << 4);
        cp_async16(k_dst + off, (const char*)p.kv.k + src, pr >= 0);
        cp_async16(v_dst + off, (const char*)p.kv.v + src, pr >= 0);
      }
    }
    cp_commit();
  }
};

// ---- bf16 ----------------------------------------------------------------------------------------
// A warp's slices of a segment: lane holds, of query heads lane / 4 (and + 8), maxima m, its share of the sums l, and the
// output columns 8 n + 2 (lane % 4) + {0, 1}.  Careful: values that are not finite meet the rounded probabilities only.
template <int D, bool Half, bool Careful>
__device__ __forceinline__ void slices_bf16(const Params& p, const Segment& sg, unsigned char* smem, float (&o)[D / 8][4],
                                            float (&m)[2], float (&l)[2]) {
  using T = __nv_bfloat16;
  using C = Cfg<T, D>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c2 = 2 * (lane & 3);
  Stream<T, D> st{p, sg, warp, lane, smem_u32(smem) + warp * C::kStages * C::kSliceBytes, 0};
  st.next_row = st.lookup(sg.t0);
#pragma unroll
  for (int i = 0; i < C::kStages - 1; ++i) st.load(sg.t0 + i, i);

  uint32_t qa[D / 16][4];
  {
    const T* q = (const T*)p.q + (int64_t)sg.t * p.q_row;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = g + 8 * (e & 1), col = 16 * kk + c2 + 8 * (e >> 1);
        qa[kk][e] = 0;
        if ((!Half || (e & 1) == 0) && r < sg.rows) {
          const T* x = q + (int64_t)(sg.h0 + r) * p.q_head + col;
          if (p.vec_q) {
            qa[kk][e] = *reinterpret_cast<const uint32_t*>(x);
          } else {
            const uint32_t lo = *reinterpret_cast<const unsigned short*>(x);
            const uint32_t hi = *reinterpret_cast<const unsigned short*>(x + 1);
            qa[kk][e] = lo | hi << 16;
          }
        }
      }
  }
#pragma unroll
  for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
  m[0] = m[1] = -INFINITY;
  l[0] = l[1] = 0.f;
  constexpr int NR = Half ? 1 : 2;

  const int mi = lane >> 3, mr = lane & 7;  // the 8x8 matrix and its row that this lane addresses
  for (int t = sg.t0, i = 0; t < sg.t1; ++t, ++i) {
    cp_wait<C::kStages - 2>();
    __syncwarp();
    st.load(t + C::kStages - 1, (i + C::kStages - 1) % C::kStages);
    const int x0 = t * kTile + warp * kSlice;
    if (x0 >= sg.vis.n) break;  // the last tile's end (uniform in the warp)
    const uint32_t kb = st.ring + (i % C::kStages) * C::kSliceBytes, vb = kb + kSlice * C::kRowBytes;
    float c[2][4] = {};
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      uint32_t b[4];
      const int r = (mi >> 1) * 8 + mr, ch = 2 * kk + (mi & 1);
      ldsm4(kb + r * C::kRowBytes + ((ch ^ (r & 7)) << 4), b);
      mma16816(c[0], qa[kk], b[0], b[1]);
      mma16816(c[1], qa[kk], b[2], b[3]);
    }
    // scores in base 2; keys behind the last one do not count
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 2 * NR; ++e)
        c[n][e] = x0 + 8 * n + c2 + (e & 1) < sg.vis.n ? c[n][e] * p.a : -INFINITY;
    bool moved = false;
    float f[2] = {1.f, 1.f}, ref[2];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      float mx = fmaxf(fmaxf(c[0][2 * r], c[0][2 * r + 1]), fmaxf(c[1][2 * r], c[1][2 * r + 1]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      if (mx > m[r]) {
        f[r] = ex2_approx(m[r] - mx);  // 0 at the first finite score
        m[r] = mx;
        moved = true;
      }
      ref[r] = m[r] == -INFINITY ? 0.f : m[r];
    }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int r = 0; r < NR; ++r) l[r] *= f[r];
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        o[n][0] *= f[0];
        o[n][1] *= f[0];
        o[n][2] *= f[Half ? 0 : 1];  // (Half: the remainders of the same heads)
        o[n][3] *= f[Half ? 0 : 1];
      }
    }
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 2 * NR; ++e) {
        c[n][e] = ex2_approx(c[n][e] - ref[e >> 1]);
        l[e >> 1] += c[n][e];
      }
    uint32_t pa[4], pl[4];
    pa[0] = pack2(c[0][0], c[0][1]);
    pa[2] = pack2(c[1][0], c[1][1]);
    if (Half) {
      pa[1] = pack2_rest(c[0][0], c[0][1], pa[0]);
      pa[3] = pack2_rest(c[1][0], c[1][1], pa[2]);
    } else {
      pa[1] = pack2(c[0][2], c[0][3]);
      pa[3] = pack2(c[1][2], c[1][3]);
      pl[0] = pack2_rest(c[0][0], c[0][1], pa[0]);
      pl[1] = pack2_rest(c[0][2], c[0][3], pa[1]);
      pl[2] = pack2_rest(c[1][0], c[1][1], pa[2]);
      pl[3] = pack2_rest(c[1][2], c[1][3], pa[3]);
    }
#pragma unroll
    for (int dd = 0; dd < D / 16; ++dd) {
      uint32_t b[4];
      const int r = (mi & 1) * 8 + mr, ch = 2 * dd + (mi >> 1);
      ldsm4_t(vb + r * C::kRowBytes + ((ch ^ (r & 7)) << 4), b);
      if (!Careful) {
        mma16816(o[2 * dd], pa, b[0], b[1]);
        mma16816(o[2 * dd + 1], pa, b[2], b[3]);
        if (!Half) {
          mma16816(o[2 * dd], pl, b[0], b[1]);
          mma16816(o[2 * dd + 1], pl, b[2], b[3]);
        }
      } else {
        const uint32_t hi[4] = {pa[0], Half ? 0u : pa[1], pa[2], Half ? 0u : pa[3]};
        const uint32_t rest[4] = {Half ? 0u : pl[0], Half ? pa[1] : pl[1], Half ? 0u : pl[2], Half ? pa[3] : pl[3]};
#pragma unroll
        for (int c8 = 0; c8 < 2; ++c8) {
          float(&x)[4] = o[2 * dd + c8];
          const uint32_t b0 = b[2 * c8], b1 = b[2 * c8 + 1];
          float y[4] = {x[0], x[1], Half ? 0.f : x[2], Half ? 0.f : x[3]};
          mma16816(y, hi, b0, b1);
          x[0] = y[0];
          x[1] = y[1];
          if (!Half) {
            x[2] = y[2];
            x[3] = y[3];
          }
          mma16816(x, rest, b0 & ~not_finite(b0), b1 & ~not_finite(b1));
        }
      }
    }
  }
  cp_wait<0>();
}

// (a function of its own, with results of its own: the ordinary pass keeps its registers)
template <int D, bool Half>
__device__ __noinline__ void slices_bf16_again(const Params& p, const Segment sg, unsigned char* smem,
                                               float (&o)[D / 8][4]) {
  float m[2], l[2];
  slices_bf16<D, Half, true>(p, sg, smem, o, m, l);
}

template <int D, bool Half>
__device__ void run_bf16(const Params& p, const Segment& sg, unsigned char* smem) {
  constexpr int NR = Half ? 1 : 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c2 = 2 * (lane & 3);
  float o[D / 8][4], m[2], l[2];
  slices_bf16<D, Half, false>(p, sg, smem, o, m, l);
  float zero[4] = {0.f, 0.f, 0.f, 0.f};  // stays 0 while every output is finite
#pragma unroll
  for (int n = 0; n < D / 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) zero[e] = fmaf(o[n][e], 0.f, zero[e]);
  if (__any_sync(0xffffffffu, !(zero[0] + zero[1] + zero[2] + zero[3] == 0.f))) {
    float again[D / 8][4];
    __syncwarp();
    slices_bf16_again<D, Half>(p, sg, smem, again);
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = again[n][e];
  }
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
  }
  __syncthreads();  // every warp has left its ring: it becomes [warp][row][d] outputs, then maxima and sums
  float* out = reinterpret_cast<float*>(smem);
  float* ml = out + kWarps * kMaxRows * D;
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const int row = g + 8 * r;
    if (row >= sg.rows) continue;
    float* dst = out + (warp * kMaxRows + row) * D + c2;
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
      *reinterpret_cast<float2*>(dst + 8 * n) = Half ? make_float2(o[n][0] + o[n][2], o[n][1] + o[n][3])
                                                     : make_float2(o[n][2 * r], o[n][2 * r + 1]);
    if ((lane & 3) == 0) {
      ml[warp * kMaxRows + row] = m[r];
      ml[(kWarps + warp) * kMaxRows + row] = l[r];
    }
  }
  __syncthreads();
}

// ---- fp32 ----------------------------------------------------------------------------------------
// R query heads (a power of two): scores by lanes (key lane % 16, heads of half lane / 16), outputs by lanes
// (4 columns each; at d = 64 two groups of lanes take 8 keys each).
template <int D, int R>
__device__ void run_f32(const Params& p, const Segment& sg, unsigned char* smem) {
  using C = Cfg<float, D>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* qs = reinterpret_cast<float*>(smem + C::kRingBytes);
  float* ps = qs + kMaxRows * D + warp * kMaxRows * (kSlice + 1);  // [R][16] probabilities, then R factors
  float* fs = ps + kMaxRows * kSlice;
  Stream<float, D> st{p, sg, warp, lane, smem_u32(smem) + warp * C::kStages * C::kSliceBytes, 0};
  st.next_row = st.lookup(sg.t0);
#pragma unroll
  for (int i = 0; i < C::kStages - 1; ++i) st.load(sg.t0 + i, i);
  for (int e = threadIdx.x; e < R * D; e += kThreads) {
    const int r = e / D;
    qs[e] = r < sg.rows ? ((const float*)p.q)[(int64_t)sg.t * p.q_row + (int64_t)(sg.h0 + r) * p.q_head + e % D] : 0.f;
  }
  __syncthreads();
  constexpr int NH = R >= 2 ? R / 2 : 1;  // heads of a lane
  const int key = lane & 15, half = lane >> 4;
  constexpr int kCols = D / 4, kKeyGroups = 32 / kCols;  // 1 or 2
  const int col = lane % kCols, kg = lane / kCols;
  float m[NH], l[NH], acc[R][4];
#pragma unroll
  for (int h = 0; h < NH; ++h) m[h] = -INFINITY, l[h] = 0.f;
#pragma unroll
  for (int h = 0; h < R; ++h) acc[h][0] = acc[h][1] = acc[h][2] = acc[h][3] = 0.f;

  for (int t = sg.t0, i = 0; t < sg.t1; ++t, ++i) {
    cp_wait<C::kStages - 2>();
    __syncwarp();
    st.load(t + C::kStages - 1, (i + C::kStages - 1) % C::kStages);
    const int x0 = t * kTile + warp * kSlice;
    if (x0 >= sg.vis.n) break;
    const unsigned char* kb = smem + (warp * C::kStages + i % C::kStages) * C::kSliceBytes;
    const unsigned char* vb = kb + kSlice * C::kRowBytes;
    float x[NH];
#pragma unroll
    for (int h = 0; h < NH; ++h) x[h] = 0.f;
    // one head: the lane halves take half of the columns each
    const int c_lo = R == 1 ? half * (D / 8) : 0, c_hi = R == 1 ? c_lo + D / 8 : D / 4;
#pragma unroll 8
    for (int c = c_lo; c < c_hi; ++c) {
      const float4 k4 = *reinterpret_cast<const float4*>(kb + key * C::kRowBytes + ((c ^ (key & 7)) << 4));
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        const float4 q4 = *reinterpret_cast<const float4*>(qs + (R == 1 ? 0 : half * NH + h) * D + 4 * c);
        x[h] = fmaf(q4.x, k4.x, x[h]);
        x[h] = fmaf(q4.y, k4.y, x[h]);
        x[h] = fmaf(q4.z, k4.z, x[h]);
        x[h] = fmaf(q4.w, k4.w, x[h]);
      }
    }
    if (R == 1) x[0] += __shfl_xor_sync(0xffffffffu, x[0], 16);
    bool moved = false;
    float f[NH];
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      x[h] = x0 + key < sg.vis.n ? x[h] * p.a : -INFINITY;
      float mx = x[h];
#pragma unroll
      for (int w = 1; w < 16; w *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      f[h] = 1.f;
      if (mx > m[h]) {
        f[h] = ex2_approx(m[h] - mx);
        m[h] = mx;
        moved = true;
      }
      x[h] = ex2_approx(x[h] - (m[h] == -INFINITY ? 0.f : m[h]));
      l[h] = l[h] * f[h] + x[h];
      if (R > 1 || half == 0) ps[(R == 1 ? 0 : half * NH + h) * kSlice + key] = x[h];
      if (key == 0 && (R > 1 || half == 0)) fs[R == 1 ? 0 : half * NH + h] = f[h];
    }
    moved = __any_sync(0xffffffffu, moved);
    __syncwarp();
    if (moved) {
#pragma unroll
      for (int h = 0; h < R; ++h) {
        const float w = fs[h];
        acc[h][0] *= w;
        acc[h][1] *= w;
        acc[h][2] *= w;
        acc[h][3] *= w;
      }
    }
#pragma unroll
    for (int j4 = 0; j4 < kSlice / kKeyGroups; j4 += 4) {
      const int j = kg * (kSlice / kKeyGroups) + j4;
      float4 v4[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v4[e] = *reinterpret_cast<const float4*>(vb + (j + e) * C::kRowBytes + ((col ^ ((j + e) & 7)) << 4));
#pragma unroll
      for (int h = 0; h < R; ++h) {
        const float4 w = *reinterpret_cast<const float4*>(ps + h * kSlice + j);
        const float we[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[h][0] = fmaf(we[e], v4[e].x, acc[h][0]);
          acc[h][1] = fmaf(we[e], v4[e].y, acc[h][1]);
          acc[h][2] = fmaf(we[e], v4[e].z, acc[h][2]);
          acc[h][3] = fmaf(we[e], v4[e].w, acc[h][3]);
        }
      }
    }
    __syncwarp();  // the probabilities have been read
  }
  cp_wait<0>();
#pragma unroll
  for (int h = 0; h < NH; ++h)
#pragma unroll
    for (int w = 1; w < 16; w *= 2) l[h] += __shfl_xor_sync(0xffffffffu, l[h], w);
  if (kKeyGroups == 2) {
#pragma unroll
    for (int h = 0; h < R; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[h][e] += __shfl_xor_sync(0xffffffffu, acc[h][e], 16);
  }
  __syncthreads();
  float* out = reinterpret_cast<float*>(smem);
  float* ml = out + kWarps * kMaxRows * D;
#pragma unroll
  for (int h = 0; h < R; ++h)
    if (h < sg.rows && kg == 0)
      *reinterpret_cast<float4*>(out + (warp * kMaxRows + h) * D + 4 * col) =
          make_float4(acc[h][0], acc[h][1], acc[h][2], acc[h][3]);
  if (key == 0 && (R > 1 || half == 0)) {
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      ml[warp * kMaxRows + half * NH + h] = m[h];
      ml[(kWarps + warp) * kMaxRows + half * NH + h] = l[h];
    }
  }
  __syncthreads();
}

// ---- merging, joining ----------------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ void store4(const Params& p, int64_t at, float4 x) {
  T* o = (T*)p.o + at;
  if (p.vec_o) {
    if (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(o) = x;
    } else {
      *reinterpret_cast<uint2*>(o) = make_uint2(pack2(x.x, x.y), pack2(x.z, x.w));
    }
  } else {
    o[0] = from_f32<T>(x.x);
    o[1] = from_f32<T>(x.y);
    o[2] = from_f32<T>(x.z);
    o[3] = from_f32<T>(x.w);
  }
}

// Natural log normaliser of a row with maximum m and sum l (base 2): -inf for a row without keys.
__device__ __forceinline__ float row_lse(float m, float l) { return l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2; }

// Combine n parts of the segment's rows: part_ml(i, row) gives part i's maximum and sum, part_out(i, row, c) four of its
// unnormalised outputs.  With `to` NULL the rows are finished and go to O, otherwise they become the part in that slot.
template <typename T, int D, typename M, typename F>
__device__ __forceinline__ void combine(const Params& p, const Segment& sg, int n, M part_ml, F part_out, float* to) {
  for (int e = threadIdx.x; e < sg.rows * (D / 4); e += kThreads) {
    const int row = e / (D / 4), c = 4 * (e % (D / 4));
    float M_ = -INFINITY;
    for (int i = 0; i < n; ++i) M_ = fmaxf(M_, part_ml(i, row).x);
    const float ref = M_ == -INFINITY ? 0.f : M_;
    float L = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float2 ml = part_ml(i, row);
      const float w = ex2_approx(ml.x - ref);
      const float4 y = part_out(i, row, c);
      L = fmaf(w, ml.y, L);
      x.x = fmaf(w, y.x, x.x);
      x.y = fmaf(w, y.y, x.y);
      x.z = fmaf(w, y.z, x.z);
      x.w = fmaf(w, y.w, x.w);
    }
    if (to != nullptr) {
      __stcg(reinterpret_cast<float4*>(to + 2 * kMaxRows + row * D + c), x);
      if (c == 0) __stcg(reinterpret_cast<float2*>(to) + row, make_float2(M_, L));
    } else {
      const float inv = L == 0.f ? 0.f : 1.f / L;
      store4<T>(p, (int64_t)(sg.h0 + row) * p.o_head + (int64_t)sg.t * p.o_row + c,
                make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
      if (c == 0 && p.lse) p.lse[(int64_t)(sg.h0 + row) * p.n_rows + sg.t] = row_lse(M_, L);
    }
  }
}

template <typename T, int D>
__device__ void run_segment(const Params& p, const Segment& sg, unsigned char* smem) {
  if constexpr (sizeof(T) == 2) {
    if (sg.rows <= 8)
      run_bf16<D, true>(p, sg, smem);
    else
      run_bf16<D, false>(p, sg, smem);
  } else {
    if (sg.rows == 1)
      run_f32<D, 1>(p, sg, smem);
    else if (sg.rows <= 4)
      run_f32<D, 4>(p, sg, smem);
    else if (sg.rows <= 8)
      run_f32<D, 8>(p, sg, smem);
    else
      run_f32<D, 16>(p, sg, smem);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) k_decode(const __grid_constant__ Params p) {
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ int sh_row, sh_last;
  __shared__ int64_t sh_sum[2 * kWarps], sh_before;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_rows = p.n_rows;
  if (p.few.ask && !as_tokens<kThreads>(p.kv, p.cu, n_rows, p.window, p.sinks, p.few, sh_sum)) return;
  // tiles in front of this thread's run of query rows
  const int per = (n_rows + kThreads - 1) / kThreads;
  const int t_lo = min(n_rows, (int)threadIdx.x * per), t_hi = min(n_rows, t_lo + per);
  int64_t mine = 0;
  for (int t = t_lo; t < t_hi; ++t) {
    const Query q = query(p, t);
    mine += (visible(p, q).n + kTile - 1) / kTile;
    if (blockIdx.x == 0 && q.len > p.kv.capacity) set_status(p.ws, MR_ERR_DEVICE_CHECK, kTableShort);
  }
  int64_t upto = mine;
#pragma unroll
  for (int w = 1; w < 32; w *= 2) {
    const int64_t y = __shfl_up_sync(0xffffffffu, upto, w);
    if (lane >= w) upto += y;
  }
  if (lane == 31) sh_sum[warp] = upto;
  __syncthreads();
  int64_t before = upto - mine;
  int64_t tiles = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sh_sum[w];
    tiles += sh_sum[w];
  }
  const int HC = p.kv.H_kv * p.chunks;
  const int64_t total = tiles * HC;
  const int64_t ctas = min((int64_t)gridDim.x, total);
  // query rows that see nothing
  for (int t = blockIdx.x; t < n_rows; t += gridDim.x) {
    const Query q = query(p, t);
    if (q.s < 0 || visible(p, q).n > 0) continue;
    for (int e = threadIdx.x; e < p.H_q * (D / 4); e += kThreads)
      store4<T>(p, (int64_t)(e / (D / 4)) * p.o_head + (int64_t)t * p.o_row + 4 * (e % (D / 4)),
                make_float4(0.f, 0.f, 0.f, 0.f));
    if (p.lse)
      for (int h = threadIdx.x; h < p.H_q; h += kThreads) p.lse[(int64_t)h * n_rows + t] = -INFINITY;
  }
  const int64_t k = blockIdx.x;
  if (k >= ctas) return;
  int64_t cur = k * total / ctas;
  const int64_t end = (k + 1) * total / ctas;
  if (cur >= before * HC && cur < (before + mine) * HC) {  // exactly one thread: the run that holds `cur`
    int t = t_lo;
    int64_t b = before;
    for (;; ++t) {
      const int nt = (visible(p, query(p, t)).n + kTile - 1) / kTile;
      if (cur < (b + nt) * HC) break;
      b += nt;
    }
    sh_row = t;
    sh_before = b;
  }
  __syncthreads();
  int t = sh_row;
  int64_t b = sh_before;
  while (cur < end) {
    Segment sg;
    const Query q = query(p, t);
    sg.vis = visible(p, q);
    sg.nt = (sg.vis.n + kTile - 1) / kTile;
    if (cur >= (b + sg.nt) * HC) {
      b += sg.nt;
      ++t;
      continue;
    }
    const int64_t r = cur - b * HC;
    const int hu = (int)(r / sg.nt);
    sg.t = t;
    sg.s = q.s;
    sg.t0 = (int)(r - (int64_t)hu * sg.nt);
    sg.t1 = (int)min((int64_t)sg.nt, sg.t0 + (end - cur));
    sg.g = hu / p.chunks;
    sg.chunk = hu - sg.g * p.chunks;
    sg.h0 = sg.g * p.group + sg.chunk * p.rows;
    sg.rows = min(p.rows, p.group - sg.chunk * p.rows);
    run_segment<T, D>(p, sg, smem);
    // [warp][row][D] outputs and their maxima and sums are in shared memory
    const float* out = reinterpret_cast<const float*>(smem);
    const float* ml = out + kWarps * kMaxRows * D;
    const auto warp_ml = [&](int i, int row) {
      return make_float2(ml[i * kMaxRows + row], ml[(kWarps + i) * kMaxRows + row]);
    };
    const auto warp_out = [&](int i, int row, int c) {
      return *reinterpret_cast<const float4*>(out + (i * kMaxRows + row) * D + c);
    };
    constexpr int kSlot = kMaxRows * (D + 2);
    if (sg.t0 == 0 && sg.t1 == sg.nt) {
      combine<T, D>(p, sg, kWarps, warp_ml, warp_out, nullptr);
    } else {
      // this CTA's slot: 2 k + 1 for a unit that begins here, 2 k for one that began before
      combine<T, D>(p, sg, kWarps, warp_ml, warp_out, p.part + (2 * k + (sg.t0 == 0 ? 1 : 0)) * kSlot);
      // the CTAs that hold the unit's first and last tile
      const int64_t u0 = cur - sg.t0, u1 = u0 + sg.nt - 1;
      const int first = (int)(((u0 + 1) * ctas - 1) / total), last = (int)(((u1 + 1) * ctas - 1) / total);
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) sh_last = atomicAdd(p.counters + first, 1u) == (uint32_t)(last - first);
      __syncthreads();
      if (sh_last) {
        __threadfence();
        const auto slot = [&](int i) { return p.part + (int64_t)(i == 0 ? 2 * first + 1 : 2 * (first + i)) * kSlot; };
        combine<T, D>(
            p, sg, last - first + 1, [&](int i, int row) { return __ldcg(reinterpret_cast<const float2*>(slot(i)) + row); },
            [&](int i, int row, int c) {
              return __ldcg(reinterpret_cast<const float4*>(slot(i) + 2 * kMaxRows + row * D + c));
            },
            nullptr);
      }
    }
    __syncthreads();  // shared memory is free again
    cur += sg.t1 - sg.t0;
  }
}

template <typename T, int D>
cudaError_t launch(const DecodeArgs& a, const Params& p, int sms) {
  constexpr int smem = smem_bytes<T, D>();
  cudaError_t e = cudaFuncSetAttribute(k_decode<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int per_sm = smem <= 113 * 1024 ? 2 : 1;
  // no more CTAs than there can be tiles
  const int64_t tiles = (int64_t)a.n_rows * p.kv.H_kv * p.chunks * (((int64_t)a.kv.capacity + kTile - 1) / kTile);
  int grid = sms * per_sm < kMaxCtas ? sms * per_sm : kMaxCtas;
  if (tiles < grid) grid = (int)tiles;
  ProfScope ps(kKDecode, a.stream);
  k_decode<T, D><<<grid, kThreads, smem, a.stream>>>(p);
  return cudaGetLastError();
}

constexpr size_t kCounterBytes = (kMaxCtas * sizeof(uint32_t) + 255) / 256 * 256;

}  // namespace

size_t decode_workspace_bytes(int d) {
  return kWsHeaderBytes + kCounterBytes + (size_t)2 * kMaxCtas * kMaxRows * (d + 2) * sizeof(float);
}

cudaError_t launch_decode(const DecodeArgs& a) {
  int dev = 0, sms = 0;
  cudaError_t e;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  if ((e = cudaMemsetAsync(a.ws, 0, kWsHeaderBytes + kCounterBytes, a.stream)) != cudaSuccess) return e;
  Params p;
  p.kv = a.kv;
  p.q = a.q.ptr;
  p.o = a.o.ptr;
  p.q_head = a.q.head_stride;
  p.q_row = a.q.row_stride;
  p.o_head = a.o.head_stride;
  p.o_row = a.o.row_stride;
  p.lse = a.lse;
  p.cu = a.cu_q;
  p.n_rows = a.n_rows;
  p.H_q = a.H_q;
  p.group = a.H_q / a.kv.H_kv;
  p.chunks = (p.group + kMaxRows - 1) / kMaxRows;
  p.rows = (p.group + p.chunks - 1) / p.chunks;
  const int es = a.dt == MR_BF16 ? 2 : 4;
  p.vec_q = ((uintptr_t)a.q.ptr | (uintptr_t)(a.q.head_stride * es) | (uintptr_t)(a.q.row_stride * es)) % 4 == 0;
  p.vec_o = ((uintptr_t)a.o.ptr | (uintptr_t)(a.o.head_stride * es) | (uintptr_t)(a.o.row_stride * es)) % 16 == 0;
  p.a = a.scale * kLog2e;
  p.window = a.window;
  p.sinks = a.sinks;
  p.few = a.few;
  p.ws = (WsHeader*)a.ws;
  p.counters = (uint32_t*)((char*)a.ws + kWsHeaderBytes);
  p.part = (float*)((char*)a.ws + kWsHeaderBytes + kCounterBytes);
  if (a.dt == MR_BF16)
    return a.kv.d == 64 ? launch<__nv_bfloat16, 64>(a, p, sms) : launch<__nv_bfloat16, 128>(a, p, sms);
  return a.kv.d == 64 ? launch<float, 64>(a, p, sms) : launch<float, 128>(a, p, sms);
}

}  // namespace mr
