// Attention of a chunk of new rows per sequence over the paged cache, on the CUDA cores: fp32, and the bf16 calls whose
// alignment or page size the tensor-core kernel does not take.
//
// Bound by fp32 arithmetic: 4 d operations for a row and a key it sees.  A CTA holds a tile of 64 query rows (rows
// x the query heads that share a key head, so a tile of keys serves all of them) and walks key tiles of 64.  16 x 16
// threads own 4 x 4 scores and 4 x d/16 outputs each: 64 multiply-adds for 8 16-byte reads of shared memory.  Scores
// are turned into probabilities with a running maximum and sum per row, held by the 16 threads of the row.  Two CTAs an
// SM cover each other's loads.  2 x 4000 rows behind 1000, 8 heads of 128 in groups of 2: 1.82 ms, 36 TFLOP/s; a call of
// one key tile takes 23 us, most of it latency.
#include <cuda_bf16.h>

#include "attn_units.cuh"
#include "profile.h"
#include "sm100.cuh"

namespace mr {
namespace {

using sm100::ex2_approx;
using sm100::smem_u32;

constexpr int kThreads = 256;
constexpr int kRows = 64;   // query rows of a unit
constexpr int kKeys = 64;   // keys of a tile
constexpr int kMaxHeads = 32;
constexpr float kLn2 = 0.6931471805599453f;

template <int D>
struct Smem {
  static constexpr int kStride = D + 4;       // floats; shifts rows by 16 bytes in the banks
  static constexpr int kPStride = kKeys + 4;
  float q[kRows * kStride];
  float k[kKeys * kStride];                   // the probabilities take its place
  float v[kKeys * D];
  int rows[2][kKeys];                         // pool rows of this key tile and the next one (-1: zeros)
  PartitionSmem part;
  int last;
};
static_assert(Smem<64>::kPStride * kRows <= kKeys * Smem<64>::kStride, "probabilities fit");

// Rows of K or V from the pool into shared memory as fp32; rows[] < 0 become zeros.
template <typename T, int D>
__device__ __forceinline__ void load_rows(const void* pool, const int* rows, float* dst, int stride) {
  constexpr int V = 16 / sizeof(T);            // elements of a 16-byte load
  constexpr int kVecs = kKeys * (D / V);
#pragma unroll 4
  for (int e = threadIdx.x; e < kVecs; e += kThreads) {
    const int r = e / (D / V), c = (e % (D / V)) * V;
    float* d = dst + r * stride + c;
    const int row = rows[r];
    const T* src = (const T*)pool + (int64_t)max(row, 0) * D + c;
    if constexpr (sizeof(T) == 4) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(d)), "l"(src), "r"(row >= 0 ? 16 : 0)
                   : "memory");
    } else {
      uint4 x = make_uint4(0, 0, 0, 0);
      if (row >= 0) x = *reinterpret_cast<const uint4*>(src);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int i = 0; i < 4; i += 2)
        *reinterpret_cast<float4*>(d + 2 * i) =
            make_float4(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u),
                        __uint_as_float(w[i + 1] << 16), __uint_as_float(w[i + 1] & 0xffff0000u));
    }
  }
}

template <int D, bool Edge>
__device__ __forceinline__ void product(const float* pr, const float* v, float (&acc)[4][D / 16]) {
  // pr: this thread's 4 rows of probabilities (a masked one is -1), v: its columns 4 tx + 64 c
#pragma unroll 2
  for (int j = 0; j < kKeys; j += 4) {
    float4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(pr + i * Smem<D>::kPStride + j);
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const float4 x = *reinterpret_cast<const float4*>(v + (j + e) * D + 64 * c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float y = e == 0 ? w[i].x : e == 1 ? w[i].y : e == 2 ? w[i].z : w[i].w;
          if (!Edge || !(y < 0.f)) {  // what a masked row holds, infinities and NaN included, must not count
            acc[i][4 * c] = fmaf(y, x.x, acc[i][4 * c]);
            acc[i][4 * c + 1] = fmaf(y, x.y, acc[i][4 * c + 1]);
            acc[i][4 * c + 2] = fmaf(y, x.z, acc[i][4 * c + 2]);
            acc[i][4 * c + 3] = fmaf(y, x.w, acc[i][4 * c + 3]);
          }
        }
      }
  }
}

template <typename T>
__device__ __forceinline__ void store4(const AttnParams& p, int64_t at, float4 x) {
  T* o = (T*)p.o + at;
  if (sizeof(T) == 4 && p.vec_o) {
    *reinterpret_cast<float4*>(o) = x;
  } else {
    o[0] = from_f32<T>(x.x);
    o[1] = from_f32<T>(x.y);
    o[2] = from_f32<T>(x.z);
    o[3] = from_f32<T>(x.w);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 2) k_attn(const __grid_constant__ AttnParams p) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Smem<D>& s = *reinterpret_cast<Smem<D>*>(smem_raw);
  constexpr int kStride = Smem<D>::kStride, kPStride = Smem<D>::kPStride;
  constexpr int kSlot = kRows * (D + 2);  // floats of a part: 64 (maximum, sum), then outputs
  if (p.few.ask && as_tokens<kThreads>(p.kv, p.cu, p.total_q, p.window, p.sinks, p.few, s.part.sums)) return;
  empty_rows<T, D, kThreads>(p);
  Share sh;
  if (!make_share<kKeys, kThreads>(p, s.part, sh)) return;
  Segments<kKeys> walk(p, sh);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  Seg sg;
  while (walk.next(sg)) {
    const Unit& u = sg.u;
    // query rows: head r / tile_tokens, new row r % tile_tokens
    const auto query = [&](int r, int c) -> const T* {  // NULL: a row that does not exist
      const int hh = (int)fast_div((uint32_t)r, p.by_tile_tokens), t = r - hh * p.tile_tokens;
      return hh < sg.heads && t < u.n
                 ? (const T*)p.q + (int64_t)(sg.h0 + hh) * p.q_head + (int64_t)(u.q0 + t) * p.q_row + c
                 : nullptr;
    };
    if (sizeof(T) == 4 && p.vec_q) {
#pragma unroll
      for (int e = threadIdx.x; e < kRows * D / 4; e += kThreads) {
        const int r = e / (D / 4), c = 4 * (e % (D / 4));
        const T* x = query(r, c);
        *reinterpret_cast<float4*>(s.q + r * kStride + c) =
            x ? *reinterpret_cast<const float4*>(x) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    } else {
#pragma unroll 8
      for (int e = threadIdx.x; e < kRows * D; e += kThreads) {
        const T* x = query(e / D, e % D);
        s.q[e / D * kStride + e % D] = x ? to_f32<T>(*x) : 0.f;
      }
    }
    int hh[4], tok[4], pos[4], last[4];  // of this thread's rows: head, new row (-1: none), position, last row seen
    float m[4], l[4], acc[4][D / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * ty + i;
      hh[i] = (int)fast_div((uint32_t)r, p.by_tile_tokens);
      tok[i] = r - hh[i] * p.tile_tokens;
      if (hh[i] >= sg.heads || tok[i] >= u.n) tok[i] = -1;
      pos[i] = u.pos0 + max(tok[i], 0);
      last[i] = tok[i] < 0 ? -1 : min(pos[i], u.held - 1);
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) acc[i][c] = 0.f;
    }
    const int hi = min(u.pos0 + u.n - 1, u.held - 1);
    const int lo = p.window > 0 && u.pos0 >= p.window ? u.pos0 - p.window + 1 : 0;
    const int pos_last = u.pos0 + u.n - 1;
    // pool row of key tile j's key threadIdx.x, or -1 where no row of the unit sees it
    auto lookup = [&](int j) {
      const int key = tile_of(u, j) * kKeys + (int)threadIdx.x;
      if (threadIdx.x >= kKeys || j >= sg.j1 || key > hi || (key < lo && key >= p.sinks)) return -1;
      const int row = pool_row(p.kv, u.s, sg.g, key);
      if (row < 0) set_status(p.ws, MR_ERR_DEVICE_CHECK, kBadPage);
      return row;
    };
    if (threadIdx.x < kKeys) s.rows[0][threadIdx.x] = lookup(sg.j0);
    __syncthreads();
    for (int j = sg.j0; j < sg.j1; ++j) {
      const int key0 = tile_of(u, j) * kKeys, buf = (j - sg.j0) & 1;
      load_rows<T, D>(p.kv.k, s.rows[buf], s.k, kStride);
      asm volatile("cp.async.commit_group;" ::: "memory");
      load_rows<T, D>(p.kv.v, s.rows[buf], s.v, D);
      asm volatile("cp.async.commit_group;" ::: "memory");
      const int next = lookup(j + 1);  // (the table is read while the rows are under way)
      if (threadIdx.x < kKeys) s.rows[buf ^ 1][threadIdx.x] = next;
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncthreads();
      float x[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < 4; ++n) x[i][n] = 0.f;
#pragma unroll 4
      for (int c = 0; c < D; c += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(s.q + (4 * ty + i) * kStride + c);
#pragma unroll
        for (int n = 0; n < 4; ++n) b[n] = *reinterpret_cast<const float4*>(s.k + (tx + 16 * n) * kStride + c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            x[i][n] = fmaf(a[i].x, b[n].x, x[i][n]);
            x[i][n] = fmaf(a[i].y, b[n].y, x[i][n]);
            x[i][n] = fmaf(a[i].z, b[n].z, x[i][n]);
            x[i][n] = fmaf(a[i].w, b[n].w, x[i][n]);
          }
      }
      // some row of the tile may not see some key (pos0 < 0 included)
      const bool edge = key0 + kKeys - 1 > min(u.pos0, u.held - 1) ||
                        (p.window > 0 && pos_last >= p.window && key0 <= pos_last - p.window && key0 + kKeys > p.sinks);
      float f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float mx = -INFINITY;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const int key = key0 + tx + 16 * n;
          const bool seen = !edge || (key <= last[i] && (p.window == 0 || key > pos[i] - p.window || key < p.sinks));
          x[i][n] = seen ? x[i][n] * p.a : -INFINITY;
          mx = fmaxf(mx, x[i][n]);
        }
#pragma unroll
        for (int w = 1; w < 16; w *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
        f[i] = 1.f;
        if (mx > m[i]) {
          f[i] = ex2_approx(m[i] - mx);
          m[i] = mx;
        }
        const float ref = m[i] == -INFINITY ? 0.f : m[i];
        l[i] *= f[i];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const int key = key0 + tx + 16 * n;
          const bool seen = !edge || (key <= last[i] && (p.window == 0 || key > pos[i] - p.window || key < p.sinks));
          const float y = ex2_approx(x[i][n] - ref);
          x[i][n] = seen ? y : -1.f;
          l[i] += seen ? y : 0.f;
        }
#pragma unroll
        for (int c = 0; c < D / 16; ++c) acc[i][c] *= f[i];
      }
      __syncthreads();  // every thread has read the keys
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < 4; ++n) s.k[(4 * ty + i) * kPStride + tx + 16 * n] = x[i][n];
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncthreads();
      if (edge)
        product<D, true>(s.k + 4 * ty * kPStride, s.v + 4 * tx, acc);
      else
        product<D, false>(s.k + 4 * ty * kPStride, s.v + 4 * tx, acc);
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int w = 1; w < 16; w *= 2) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);

    bool finish = sg.whole();
    if (!finish) {
      int first, lastc;
      holders(sh, sg, first, lastc);
      float* mine = p.part + slot_of(blockIdx.x, first) * kSlot;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
        if (tx == 0) __stcg(reinterpret_cast<float2*>(mine) + r, make_float2(m[i], l[i]));
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          __stcg(reinterpret_cast<float4*>(mine + 2 * kRows + r * D + 4 * tx + 64 * c),
                 make_float4(acc[i][4 * c], acc[i][4 * c + 1], acc[i][4 * c + 2], acc[i][4 * c + 3]));
      }
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) s.last = atomicAdd(p.counters + first, 1u) == (uint32_t)(lastc - first);
      __syncthreads();
      finish = s.last != 0;
      if (finish) {
        __threadfence();
        // the thread's four rows together, part by part in the order of the keys
        float top[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          top[i] = -INFINITY;
          l[i] = 0.f;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) acc[i][c] = 0.f;
        }
#pragma unroll 2
        for (int b = first; b <= lastc; ++b) {
          const float2* ml = reinterpret_cast<const float2*>(p.part + slot_of(b, first) * kSlot) + 4 * ty;
#pragma unroll
          for (int i = 0; i < 4; ++i) top[i] = fmaxf(top[i], __ldcg(ml + i).x);
        }
#pragma unroll 2
        for (int b = first; b <= lastc; ++b) {
          const float* part = p.part + slot_of(b, first) * kSlot;
          float2 ml[4];
          float4 y[4][D / 64];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            ml[i] = __ldcg(reinterpret_cast<const float2*>(part) + 4 * ty + i);
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
              y[i][c] = __ldcg(reinterpret_cast<const float4*>(part + 2 * kRows + (4 * ty + i) * D + 4 * tx + 64 * c));
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float w = ex2_approx(ml[i].x - (top[i] == -INFINITY ? 0.f : top[i]));
            l[i] = fmaf(w, ml[i].y, l[i]);
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
              acc[i][4 * c] = fmaf(w, y[i][c].x, acc[i][4 * c]);
              acc[i][4 * c + 1] = fmaf(w, y[i][c].y, acc[i][4 * c + 1]);
              acc[i][4 * c + 2] = fmaf(w, y[i][c].z, acc[i][4 * c + 2]);
              acc[i][4 * c + 3] = fmaf(w, y[i][c].w, acc[i][4 * c + 3]);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) m[i] = top[i];
      }
    }
    if (finish) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (tok[i] < 0) continue;
        const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
        const int h = sg.h0 + hh[i], row = u.q0 + tok[i];
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          store4<T>(p, (int64_t)h * p.o_head + (int64_t)row * p.o_row + 4 * tx + 64 * c,
                    make_float4(acc[i][4 * c] * inv, acc[i][4 * c + 1] * inv, acc[i][4 * c + 2] * inv,
                                acc[i][4 * c + 3] * inv));
        if (tx == 0 && p.lse)
          p.lse[(int64_t)h * p.total_q + row] = l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * kLn2;
      }
    }
    __syncthreads();  // shared memory is free again
  }
}

template <typename T, int D>
cudaError_t launch(const AttnParams& p, int sms, cudaStream_t st) {
  constexpr int smem = (int)sizeof(Smem<D>);
  cudaError_t e = cudaFuncSetAttribute(k_attn<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int grid = 2 * sms < kAttnMaxCtas ? 2 * sms : kAttnMaxCtas;
  ProfScope ps(kKAttn, st);
  k_attn<T, D><<<grid, kThreads, smem, st>>>(p);
  return cudaGetLastError();
}

constexpr size_t kCounterBytes = (kAttnMaxCtas * sizeof(uint32_t) + 255) / 256 * 256;

// Few rows: each as a token of its own (ask 0), in tiles (-1), or as the lengths on the device say (1).  A row of its own
// reads its keys and values again, from L2 mostly, but no tile of query rows stands nearly empty, and P keeps its second
// part.  What decides is how much is read again, and that depends on how the rows are spread over the sequences, which the
// host does not know: 256 sequences of 1000 with one row each take 172 us as tokens and 333 in tiles, 256 of 4096 with all
// rows in one of them 391 and 141.  So where the host's bound leaves it open both kernels are launched, and one of them
// leaves at once (3 to 9 us more); calls of more than `most` rows, and more than sequences, run in tiles.  Measured, tokens
// / tiles in us, heads of 128:
//   bf16: up to 256 MB more.  32 heads in groups of 4: 1 sequence of 4096 with 8, 16 and 32 rows 27/33, 39/45 and 62/34; of
//   16384 with 2, 4 and 8 27/33, 39/39 and 62/47; 8 of 4096 with 1, 2 and 4 each 36/48, 51/47 and 85/49.  Groups of 1: 1 of
//   4096 with 2, 4 and 8 27/29, 39/31 and 62/36.
//   fp32: that, or 8 times as much, since the tiles are bound by their arithmetic.  1 of 65536 with 4, 8 and 16: 351/747,
//   683/747 and 1347/748; in groups of 8 431/747 and 841/749; 8 of 4096 with 1, 4 and 8 each: 63/271, 192/273 and 358/273.
FewRows few_rows(const AttnArgs& a) {
  const int n_seq = a.kv.n_seq;
  const int most = a.dt == MR_BF16 ? 16 : n_seq <= 2 ? 8 : n_seq < 16 ? 4 * n_seq : 64;
  if (a.total_q <= 0 || a.total_q > (most > n_seq ? most : n_seq)) return FewRows{-1, 0, 0};
  const int64_t key_bytes = (int64_t)a.kv.H_kv * a.kv.d * 2 * (a.dt == MR_BF16 ? 2 : 4);
  FewRows f{1, ((int64_t)256 << 20) / key_bytes, a.dt == MR_BF16 ? 1 : 8};
  int64_t seen = a.kv.capacity;  // keys that a row sees at most
  if (a.window > 0 && (int64_t)a.window + a.sinks < seen) seen = (int64_t)a.window + a.sinks;
  if (a.total_q <= f.times || (a.total_q - 1) * seen <= f.extra) f.ask = 0;
  return f;
}

}  // namespace

size_t attn_workspace_bytes(mr_dtype dt, int d) {
  const size_t simt = (size_t)2 * kAttnMaxCtas * kRows * (d + 2) * sizeof(float);
  const size_t tc = dt == MR_BF16 ? attn_tc_part_bytes(d) : 0;
  return kWsHeaderBytes + kCounterBytes + (simt > tc ? simt : tc);
}

void attn_split(AttnParams& p, int rows, int max_heads) {
  p.chunks = (p.group + max_heads - 1) / max_heads;
  p.hp = (p.group + p.chunks - 1) / p.chunks;
  p.tile_tokens = rows / p.hp;
  p.by_tile_tokens = make_fastdiv((uint32_t)p.tile_tokens);
}

cudaError_t launch_attn(const AttnArgs& a) {
  int dev = 0, sms = 0;
  cudaError_t e;
  const FewRows few = few_rows(a);
  if (few.ask >= 0) {
    DecodeArgs d;
    d.kv = a.kv;
    d.cu_q = a.cu_q;
    d.n_rows = a.total_q;
    d.q = a.q;
    d.o = a.o;
    d.H_q = a.H_q;
    d.dt = a.dt;
    d.scale = a.scale;
    d.window = a.window;
    d.sinks = a.sinks;
    d.lse = a.lse;
    d.ws = a.ws;
    d.few = few;
    d.stream = a.stream;
    if ((e = launch_decode(d)) != cudaSuccess || !few.ask) return e;
  }
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  // (behind the tokens' kernel the counters are zero: only one of the two uses them)
  if (few.ask < 0 && (e = cudaMemsetAsync(a.ws, 0, kWsHeaderBytes + kCounterBytes, a.stream)) != cudaSuccess) return e;
  if (a.total_q == 0) return cudaSuccess;
  AttnParams p{};
  p.few = FewRows{few.ask > 0, few.extra, few.times};
  p.kv = a.kv;
  p.q = a.q.ptr;
  p.o = a.o.ptr;
  p.q_head = a.q.head_stride;
  p.q_row = a.q.row_stride;
  p.o_head = a.o.head_stride;
  p.o_row = a.o.row_stride;
  p.lse = a.lse;
  p.cu = a.cu_q;
  p.total_q = a.total_q;
  p.H_q = a.H_q;
  p.group = a.H_q / a.kv.H_kv;
  const int es = a.dt == MR_BF16 ? 2 : 4;
  p.vec_q = ((uintptr_t)a.q.ptr | (uintptr_t)(a.q.head_stride * es) | (uintptr_t)(a.q.row_stride * es)) % 16 == 0;
  p.vec_o = ((uintptr_t)a.o.ptr | (uintptr_t)(a.o.head_stride * es) | (uintptr_t)(a.o.row_stride * es)) % 16 == 0;
  p.a = a.scale * 1.4426950408889634f;
  p.window = a.window;
  p.sinks = a.sinks;
  p.ws = (WsHeader*)a.ws;
  p.counters = (uint32_t*)((char*)a.ws + kWsHeaderBytes);
  p.part = (float*)((char*)a.ws + kWsHeaderBytes + kCounterBytes);
  if (launch_attn_tc(a, p, sms, &e)) return e;
  attn_split(p, kRows, kMaxHeads);
  p.tokens = p.tile_tokens;
  p.unit_cost = 1;
  p.min_steps = 1;
  p.max_parts = 24;
  if (a.dt == MR_BF16)
    return a.kv.d == 64 ? launch<__nv_bfloat16, 64>(p, sms, a.stream) : launch<__nv_bfloat16, 128>(p, sms, a.stream);
  return a.kv.d == 64 ? launch<float, 64>(p, sms, a.stream) : launch<float, 128>(p, sms, a.stream);
}

}  // namespace mr
