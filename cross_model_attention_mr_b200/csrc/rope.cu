// Rotary positions, and appending rotated rows to a paged cache.
//
// Pair i of a row at position p turns by p f_i.  The angle is kept as a binary fraction of a turn in 64
// bits: turn_i = f_i / (2 pi) * 2^64, so p * turn_i in wrapping integer arithmetic drops the whole turns
// exactly, and a position of a million costs no accuracy (p * f_i in fp32 would be off by 0.06 rad
// there).  The fraction goes to sincospi, whose argument needs no further reduction.  The rotation
// itself is fp32 with one rounding to the tensor's type.
//
// Bound by memory: every element is read and written once, 3 operations each.  The sines cost more than that (some 30
// instructions a pair), so a thread keeps one unit of a token, two 16-byte vectors, for several heads: the two halves of
// 8 (fp32: 4) pairs in the half layout, or neighbouring vectors in the interleaved one.  Its loads do not depend on the
// position, so they are under way while the position is looked up and the sines are computed; nothing is shared between
// threads.  32 heads x 65536 rows of 128 in bf16 (1.07 GB): 168 us, 6.4 TB/s.  4096 rows: 11 to 13 us over several machines
// with the input in L2 from the call before (5.3 to 6.1 TB/s; a table of sines in shared memory, with the loads behind it,
// took 36 us), 15.4 us, 4.35 TB/s, with inputs that are not.  Appending 8192 rows of 28 + 2 x 4 heads: 35 us, 4.3 TB/s, from
// L2 or not.
#include <cuda_bf16.h>

#include "paged.cuh"
#include "profile.h"

namespace mr {
namespace {

constexpr int kThreads = 128;
constexpr int kMostHeads = 8;  // heads of a thread at most

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
  int heads_per_block;
  FastDiv by_units;      // units per row
  const int32_t* pos;    // rope: position of each row
  const int32_t* cu;     // append: row offsets, or NULL for one row per sequence
  PagedKv kv;
  WsHeader* ws;
};

template <typename T, int VEC, bool Append>
__global__ void __launch_bounds__(kThreads) k_rope(const __grid_constant__ mr_rope rope, const __grid_constant__ Params p) {
  using V = Vec<T, VEC>;
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int upr = (int)p.by_units.d;
  if (id >= (int64_t)p.n_rows * upr) return;
  // (ids stay below 2^31 for the division: rows are taken in slabs of 2^20)
  const int64_t slab = id / ((int64_t)upr << 20);
  const int within = (int)(id - slab * ((int64_t)upr << 20));
  const int t_in = (int)fast_div((uint32_t)within, p.by_units), i = within - t_in * upr;
  const int t = (int)(slab << 20) + t_in;
  // rows in front of the first sequence and behind the last one are not read
  if (Append && p.cu && (t < __ldg(p.cu) || t >= __ldg(p.cu + p.kv.n_seq))) return;
  const int half = p.rot >> 1, rotated = half / VEC;
  // the unit's two vectors: the halves of its pairs, or neighbours
  const bool split = i < rotated && !p.interleaved;
  const int ia = split ? i * VEC : 2 * i * VEC, ib = split ? half + i * VEC : (2 * i + 1) * VEC;
  const int all = p.heads[0] + p.heads[1] + p.heads[2];
  const int h0 = blockIdx.y * p.heads_per_block, h1 = min(h0 + p.heads_per_block, all);

  int live = 1, base = -1;  // live 0: leave everything alone; 1: rotate; 2: zero the query row, store nothing
  bool known = false;
  float c[VEC], s[VEC];
  for (int h = h0; h < h1; ++h) {
    const int kind = h < p.heads[0] ? 0 : h < p.heads[0] + p.heads[1] ? 1 : 2;
    const int hk = h - (kind == 0 ? 0 : kind == 1 ? p.heads[0] : p.heads[0] + p.heads[1]);
    const char* src = p.src[kind].ptr + hk * p.src[kind].head + (int64_t)t * p.src[kind].row;
    V a = *reinterpret_cast<const V*>(src + ia * (int)sizeof(T));
    V b = *reinterpret_cast<const V*>(src + ib * (int)sizeof(T));
    if (!known) {  // (once: the rows above are under way)
      known = true;
      int at;
      if (Append) {
        const int seq = p.cu ? sequence_of(p.cu, p.kv.n_seq, t) : t;
        live = 0;
        at = 0;
        if (seq >= 0 && seq < p.kv.n_seq) {
          const int behind = p.cu ? __ldg(p.cu + seq + 1) - t : 1;  // rows from this one to the sequence's last
          const int64_t q = (int64_t)max(__ldg(p.kv.kv_len + seq), 0) - behind;
          at = (int)q;
          live = q < 0 ? 2 : 1;
          if (q >= p.kv.capacity) {
            set_status(p.ws, MR_ERR_DEVICE_CHECK, kTableShort);
          } else if (q >= 0) {
            base = pool_row(p.kv, seq, 0, at);
            if (base < 0) set_status(p.ws, MR_ERR_DEVICE_CHECK, kBadPage);
          }
        }
      } else {
        at = __ldg(p.pos + t);
      }
      if (i < rotated) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const long long phase = (long long)((unsigned long long)(long long)at * rope.turn[i * VEC + e]);
          sincospif((float)phase * 1.0842021724855044e-19f, &s[e], &c[e]);  // phase * 2^-63: half turns in [-1, 1]
          c[e] *= p.mscale;
          s[e] *= p.mscale * (float)p.sign;
        }
      }
    }
    if (live == 0) continue;
    char* dst;
    if (Append && kind > 0) {
      if (base < 0) continue;
      dst = p.dst[kind].ptr + ((int64_t)base + (int64_t)hk * p.kv.page_rows) * p.d * (int)sizeof(T);
    } else {
      dst = p.dst[kind].ptr + hk * p.dst[kind].head + (int64_t)t * p.dst[kind].row;
    }
    if (Append && live == 2) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) a.e[e] = b.e[e] = from_f32<T>(0.f);
    } else if (i < rotated && kind < 2) {
      if (p.interleaved) {  // 2 VEC consecutive elements hold VEC pairs
        float x[2 * VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          x[e] = to_f32<T>(a.e[e]);
          x[VEC + e] = to_f32<T>(b.e[e]);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float y0 = x[2 * e] * c[e] - x[2 * e + 1] * s[e], y1 = x[2 * e + 1] * c[e] + x[2 * e] * s[e];
          x[2 * e] = y0;
          x[2 * e + 1] = y1;
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          a.e[e] = from_f32<T>(x[e]);
          b.e[e] = from_f32<T>(x[VEC + e]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float x0 = to_f32<T>(a.e[e]), x1 = to_f32<T>(b.e[e]);
          a.e[e] = from_f32<T>(x0 * c[e] - x1 * s[e]);
          b.e[e] = from_f32<T>(x1 * c[e] + x0 * s[e]);
        }
      }
    }
    *reinterpret_cast<V*>(dst + ia * (int)sizeof(T)) = a;
    *reinterpret_cast<V*>(dst + ib * (int)sizeof(T)) = b;
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
  // Heads of a thread: as many as leave 4 blocks for every SM, 8 at most.  (1024 blocks of 8 heads against 2048 of 4 for
  // 4096 rows x 32 heads: 10.7 and 11.6 us; 16 and 32 heads for 8192 rows x 36: 33 and 43 us.)
  const int64_t blocks = ((int64_t)p.n_rows * (p.d / 2 / VEC) + kThreads - 1) / kThreads;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  int each = 1;
  while (each < kMostHeads && blocks * ((all + 2 * each - 1) / (2 * each)) >= 4 * 148) each *= 2;
  p.heads_per_block = each;
  const dim3 grid((unsigned)blocks, (unsigned)((all + each - 1) / each));
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
