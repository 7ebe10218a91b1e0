// Rotary positions, and appending rotated rows to a paged cache.
//
// Pair i of a row at position p turns by p f_i.  The angle is kept as a binary fraction of a turn in 64
// bits: turn_i = f_i / (2 pi) * 2^64, so p * turn_i in wrapping integer arithmetic drops the whole turns
// exactly, and a position of a million costs no accuracy (p * f_i in fp32 would be off by 0.06 rad
// there).  The fraction goes to sincospi, whose argument needs no further reduction.  The rotation
// itself is fp32 with one rounding to the tensor's type.
//
// Bound by memory: every element is read and written once, 3 operations each.  The sines cost far more than
// that (some 40 instructions a pair), so a block takes up to kMaxTokens tokens, computes their table
// once in shared memory, and uses it for every head of the query, key and (as a plain copy) value rows.
// A unit of work is two 16-byte vectors: the two halves of 8 (fp32: 4) pairs in the half layout, or
// neighbouring vectors in the interleaved one; the lanes of a warp cover whole rows.
#include <cuda_bf16.h>

#include "paged.cuh"
#include "profile.h"

namespace mr {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;    // tokens of a block
constexpr int kMaxPairs = 128;   // rot_dim / 2
constexpr int kUnroll = 4;       // units a thread loads before it stores the first

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Vec {
  T e[VEC];
};

struct RowsP {
  char* ptr;
  int64_t head, row;  // strides in bytes
};

struct Params {
  RowsP src[3], dst[3];  // query, key, value rows (dst of key and value: the pools)
  int heads[3];          // 0: absent
  int n_rows, d, rot, interleaved;
  float mscale;
  int sign;              // -1 turns the other way
  int tokens;            // tokens per block
  int heads_per_block;
  FastDiv by_units;      // units per row
  FastDiv by_tokens;
  const int32_t* pos;    // rope: position of each row
  const int32_t* cu;     // append: row offsets, or NULL for one row per sequence
  PagedKv kv;
  WsHeader* ws;
};

// where a token's rows go
struct Token {
  int live;  // 0: leave everything alone; 1: rotate; 2: zero the query row, store nothing
  int seq_row;  // position within the sequence (append)
  int base;  // pool row of kv head 0, or -1: not stored
};

template <typename T, int VEC, bool Append>
__global__ void __launch_bounds__(kThreads) k_rope(const __grid_constant__ mr_rope rope, const Params p) {
  __shared__ float2 cs[kMaxTokens][kMaxPairs];
  __shared__ Token tok[kMaxTokens];
  __shared__ int tok_pos[kMaxTokens];
  const int t0 = blockIdx.x * p.tokens;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nt = min(p.tokens, p.n_rows - t0);
  if (warp < nt) {  // one warp per token of the block
    const int t = t0 + warp;
    Token k{1, 0, -1};
    int at;
    if (Append) {
      const int s = p.cu ? find_sequence(p.cu, p.kv.n_seq, t, lane) : t;
      k.live = 0;
      at = 0;
      // (a row in front of cu[0] belongs to no sequence)
      if (s < p.kv.n_seq && (p.cu == nullptr || t >= __ldg(p.cu + s))) {
        const int behind = p.cu ? __ldg(p.cu + s + 1) - t : 1;  // rows from this one to the sequence's last
        const int64_t a = (int64_t)max(__ldg(p.kv.kv_len + s), 0) - behind;
        at = (int)a;
        k.live = a < 0 ? 2 : 1;
        if (a >= 0) {
          if (a < p.kv.capacity) {
            k.base = pool_row(p.kv, s, 0, at);
            if (k.base < 0 && lane == 0) set_status(p.ws, MR_ERR_DEVICE_CHECK, kBadPage);
          } else if (lane == 0) {
            set_status(p.ws, MR_ERR_DEVICE_CHECK, kTableShort);
          }
        }
      }
    } else {
      at = __ldg(p.pos + t);
    }
    if (lane == 0) {
      tok[warp] = k;
      tok_pos[warp] = at;
    }
  }
  __syncthreads();
  const int half = p.rot >> 1;
  for (int e = threadIdx.x; e < nt * half; e += kThreads) {
    const int t = e / half, i = e - t * half;
    const long long phase = (long long)((unsigned long long)(long long)tok_pos[t] * rope.turn[i]);
    float s, c;
    sincospif((float)phase * 1.0842021724855044e-19f, &s, &c);  // phase * 2^-63: half turns in [-1, 1]
    cs[t][i] = make_float2(c * p.mscale, s * p.mscale * (float)p.sign);
  }
  __syncthreads();

  const int upr = (int)p.by_units.d;
  const int rotated = half / VEC;
  const int h0 = blockIdx.y * p.heads_per_block;
  const int all = p.heads[0] + p.heads[1] + p.heads[2];
  const int n = min(p.heads_per_block, all - h0) * p.tokens * upr;
  using V = Vec<T, VEC>;
  for (int u0 = threadIdx.x; u0 < n; u0 += kThreads * kUnroll) {
    V a[kUnroll], b[kUnroll];
    char* dst[kUnroll];  // NULL: nothing to do
    int ia[kUnroll], ib[kUnroll], tt[kUnroll], ii[kUnroll];
#pragma unroll
    for (int w = 0; w < kUnroll; ++w) {
      const int u = u0 + w * kThreads;
      dst[w] = nullptr;
      if (u >= n) continue;
      const int row = (int)fast_div((uint32_t)u, p.by_units), i = u - row * upr;
      int h = (int)fast_div((uint32_t)row, p.by_tokens);
      const int t = row - h * p.tokens;
      h += h0;
      if (t >= nt || tok[t].live == 0) continue;
      const int kind = h < p.heads[0] ? 0 : h < p.heads[0] + p.heads[1] ? 1 : 2;
      h -= kind == 0 ? 0 : kind == 1 ? p.heads[0] : p.heads[0] + p.heads[1];
      const char* src = p.src[kind].ptr + h * p.src[kind].head + (int64_t)(t0 + t) * p.src[kind].row;
      if (Append && kind > 0) {
        if (tok[t].base < 0) continue;
        dst[w] = p.dst[kind].ptr + ((int64_t)tok[t].base + (int64_t)h * p.kv.page_rows) * p.d * (int)sizeof(T);
      } else {
        dst[w] = p.dst[kind].ptr + h * p.dst[kind].head + (int64_t)(t0 + t) * p.dst[kind].row;
      }
      const bool turn = i < rotated && kind < 2;
      // the unit's two vectors: the halves of its pairs, or neighbours
      ia[w] = i < rotated && !p.interleaved ? i * VEC : 2 * i * VEC;
      ib[w] = i < rotated && !p.interleaved ? half + i * VEC : (2 * i + 1) * VEC;
      tt[w] = t;
      ii[w] = turn ? i * VEC : -1;
      if (Append && tok[t].live == 2) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) a[w].e[e] = b[w].e[e] = from_f32<T>(0.f);
        ii[w] = -1;
      } else {
        a[w] = *reinterpret_cast<const V*>(src + ia[w] * (int)sizeof(T));
        b[w] = *reinterpret_cast<const V*>(src + ib[w] * (int)sizeof(T));
      }
    }
#pragma unroll
    for (int w = 0; w < kUnroll; ++w) {
      if (dst[w] == nullptr) continue;
      if (ii[w] >= 0) {
        if (p.interleaved) {  // 2 VEC consecutive elements hold VEC pairs
          float x[2 * VEC];
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            x[e] = to_f32<T>(a[w].e[e]);
            x[VEC + e] = to_f32<T>(b[w].e[e]);
          }
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float2 r = cs[tt[w]][ii[w] + e];
            const float y0 = x[2 * e] * r.x - x[2 * e + 1] * r.y, y1 = x[2 * e + 1] * r.x + x[2 * e] * r.y;
            x[2 * e] = y0;
            x[2 * e + 1] = y1;
          }
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            a[w].e[e] = from_f32<T>(x[e]);
            b[w].e[e] = from_f32<T>(x[VEC + e]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float2 r = cs[tt[w]][ii[w] + e];
            const float x0 = to_f32<T>(a[w].e[e]), x1 = to_f32<T>(b[w].e[e]);
            a[w].e[e] = from_f32<T>(x0 * r.x - x1 * r.y);
            b[w].e[e] = from_f32<T>(x1 * r.x + x0 * r.y);
          }
        }
      }
      *reinterpret_cast<V*>(dst[w] + ia[w] * (int)sizeof(T)) = a[w];
      *reinterpret_cast<V*>(dst[w] + ib[w] * (int)sizeof(T)) = b[w];
    }
  }
}

bool aligned(const mr_rows& r, int esize) {
  return ((uintptr_t)r.ptr & 15u) == 0 && (r.head_stride * esize) % 16 == 0 && (r.row_stride * esize) % 16 == 0;
}

RowsP bytes(const mr_rows& r, int esize) { return RowsP{(char*)r.ptr, r.head_stride * esize, r.row_stride * esize}; }

template <typename T, int VEC, bool Append>
cudaError_t launch(const mr_rope* rope, Params& p, cudaStream_t st) {
  static const mr_rope none{};
  const int all = p.heads[0] + p.heads[1] + p.heads[2];
  p.by_units = make_fastdiv((uint32_t)(p.d / 2 / VEC));
  // tokens per block: as many as leave two blocks for every SM; heads are split over blocks while there are
  // still fewer blocks than that and a block keeps a full round of units
  p.tokens = 1;
  while (p.tokens < kMaxTokens && p.n_rows / (2 * p.tokens) >= 296) p.tokens *= 2;
  p.by_tokens = make_fastdiv((uint32_t)p.tokens);
  const int blocks = (p.n_rows + p.tokens - 1) / p.tokens;
  int split = 1;
  while (blocks * split < 296 && (all / (2 * split)) * p.tokens * (int)p.by_units.d >= kThreads) split *= 2;
  p.heads_per_block = (all + split - 1) / split;
  const dim3 grid((unsigned)blocks, (unsigned)((all + p.heads_per_block - 1) / p.heads_per_block));
  ProfScope ps(Append ? kKAppend : kKRope, st);
  k_rope<T, VEC, Append><<<grid, kThreads, 0, st>>>(rope ? *rope : none, p);
  return cudaGetLastError();
}

template <bool Append>
cudaError_t dispatch(const mr_rope* rope, Params& p, mr_dtype dt, bool vec, cudaStream_t st) {
  const int wide = dt == MR_BF16 ? 8 : 4;
  // whole vectors on both sides of every pair, and of the elements that are copied
  vec = vec && p.rot % (2 * wide) == 0 && (p.d - p.rot) % (2 * wide) == 0;
  if (dt == MR_BF16)
    return vec ? launch<__nv_bfloat16, 8, Append>(rope, p, st) : launch<__nv_bfloat16, 1, Append>(rope, p, st);
  return vec ? launch<float, 4, Append>(rope, p, st) : launch<float, 1, Append>(rope, p, st);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a) {
  const int es = a.dt == MR_BF16 ? 2 : 4;
  Params p{};
  p.src[0] = bytes(a.x, es);
  p.dst[0] = bytes(a.y, es);
  p.heads[0] = a.H;
  p.n_rows = a.n_rows;
  p.d = a.rope->d;
  p.rot = a.rope->rot_dim;
  p.interleaved = a.rope->interleaved;
  p.mscale = a.rope->mscale;
  p.sign = a.adjoint ? -1 : 1;
  p.pos = a.pos;
  return dispatch<false>(a.rope, p, a.dt, aligned(a.x, es) && aligned(a.y, es), a.stream);
}

cudaError_t launch_append(const AppendArgs& a) {
  const int es = a.dt == MR_BF16 ? 2 : 4;
  Params p{};
  bool vec = aligned(a.k_new, es) && aligned(a.v_new, es);
  if (a.q.ptr) {
    p.src[0] = bytes(a.q, es);
    p.dst[0] = bytes(a.q_out, es);
    p.heads[0] = a.H_q;
    vec = vec && aligned(a.q, es) && aligned(a.q_out, es);
  }
  p.src[1] = bytes(a.k_new, es);
  p.src[2] = bytes(a.v_new, es);
  p.dst[1].ptr = (char*)a.kv.k;
  p.dst[2].ptr = (char*)a.kv.v;
  p.heads[1] = p.heads[2] = a.kv.H_kv;
  p.n_rows = a.total_q;
  p.d = a.kv.d;
  p.rot = a.rope ? a.rope->rot_dim : 0;
  p.interleaved = a.rope ? a.rope->interleaved : 0;
  p.mscale = a.rope ? a.rope->mscale : 1.f;
  p.sign = 1;
  p.cu = a.cu_q;
  p.kv = a.kv;
  p.ws = a.ws;
  return dispatch<true>(a.rope, p, a.dt, vec, a.stream);
}

}  // namespace mr
