// How attention over the paged cache is cut into work: shared by the tensor-core and the CUDA-core kernel.
//
// A unit is (sequence, run of `tokens` new rows, kv head, chunk of `hp` query heads of its group); it reads a list of
// key tiles of KT rows: the tiles that hold first rows kept visible, then those from the first window's start to the
// last row's position.  All units' tiles, laid end to end (a run's heads next to one another, each with a few steps for
// beginning and ending it), are one range of steps that is split evenly over the CTAs: ragged batches, causal and windowed
// masks, and one long sequence with few new rows load the GPU alike.  A CTA's share may begin and end inside a unit; such
// parts are joined through the workspace by the CTA that finishes last, in the order of the keys.  No CTA waits for
// another one.
#pragma once

#include "paged.cuh"

namespace mr {

struct AttnParams {
  PagedKv kv;
  const void* q;
  void* o;
  int64_t q_head, q_row, o_head, o_row;  // strides in elements
  float* lse;
  const int32_t* cu;
  int total_q, H_q, group, chunks, hp;   // chunks of hp query heads per kv head (the last may be shorter)
  int tile_tokens, tokens;               // new rows of a tile of query rows, and of a unit
  FastDiv by_tile_tokens;
  int vec_q, vec_o;                      // rows aligned to 16 bytes (vec_o 2: to 32)
  float a;                               // scale * log2(e)
  int negate;                            // the scores' sign is changed (tensor-core kernel: a stays positive)
  int window, sinks;
  int unit_cost;                         // steps that beginning and ending a unit take
  // As many CTAs take part as leave each a share of about min_steps, or of about the longest unit's steps / max_parts if
  // that is more (rounding may halve a share, and so double a unit's parts).
  int min_steps, max_parts;
  WsHeader* ws;
  uint32_t* counters;                    // one per CTA, zero at launch
  float* part;                           // two slots per CTA
  uint64_t wait_ns;                      // (tensor-core kernel) limit of its waits
  FewRows few;
  int skip_arrive;                       // failure-path test: tile A's softmax keeps its first P back
};

struct Unit {
  int s, r;          // sequence, run
  int q0, n;         // first packed row, rows of the run
  int pos0, held;    // position of the first row; rows the table covers
  int lo_t, ns, nk;  // list of key tiles: 0 .. ns-1, then lo_t, lo_t + 1, ...; nk in all
};

__device__ __forceinline__ void seq_rows(const AttnParams& p, int s, int& q0, int& n) {
  q0 = min(max(__ldg(p.cu + s), 0), p.total_q);
  n = min(max(__ldg(p.cu + s + 1), q0), p.total_q) - q0;
}

__device__ __forceinline__ int runs_of(const AttnParams& p, int n) { return (n + p.tokens - 1) / p.tokens; }

// Run r of sequence s (its first row q0, n rows in all).
template <int KT>
__device__ __forceinline__ Unit make_unit(const AttnParams& p, int s, int r, int q0, int n) {
  Unit u;
  u.s = s;
  u.r = r;
  const int t = r * p.tokens;
  u.q0 = q0 + t;
  u.n = min(p.tokens, n - t);
  const int len = max(__ldg(p.kv.kv_len + s), 0);
  u.held = min(len, p.kv.capacity);
  u.pos0 = len - n + t;
  const int hi = min(u.pos0 + u.n - 1, u.held - 1);  // last row that is seen at all
  const int lo = p.window > 0 && u.pos0 >= p.window ? u.pos0 - p.window + 1 : 0;
  u.lo_t = lo / KT;
  u.ns = u.nk = 0;
  if (hi >= 0) {
    const int first = min(p.sinks, hi + 1);
    const int first_t = first > 0 ? (first - 1) / KT + 1 : 0;
    u.ns = min(first_t, lo <= hi ? u.lo_t : hi / KT + 1);
    u.nk = u.ns + (lo <= hi ? hi / KT - u.lo_t + 1 : 0);
  }
  return u;
}

// Steps of a unit: `unit_cost` in front for beginning and ending it, then its key tiles.
__device__ __forceinline__ int cost_of(const AttnParams& p, const Unit& u) { return u.nk > 0 ? u.nk + p.unit_cost : 0; }

// Entries of the unit's list that hold rows up to position hi.
template <int KT>
__device__ __forceinline__ int tiles_upto(const Unit& u, int hi) {
  if (hi < 0) return 0;
  const int t = hi / KT;
  return t >= u.lo_t ? min(u.nk, u.ns + t - u.lo_t + 1) : min(u.ns, t + 1);
}

__device__ __forceinline__ int tile_of(const Unit& u, int j) { return j < u.ns ? j : u.lo_t + (j - u.ns); }

// A CTA's share of the steps.
struct Share {
  int64_t cur, end;    // steps [cur, end)
  int64_t total, ctas;
  int s, r;            // the run that holds `cur`
  int64_t before;      // steps per head in front of that run
};

struct PartitionSmem {
  int64_t sums[32], all[32];
  int most[32];
  int64_t before;
  int s, r;
};

// Whole CTA of NT threads.  Returns false when there is nothing for this CTA.
template <int KT, int NT>
__device__ bool make_share(const AttnParams& p, PartitionSmem& sm, Share& sh) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n_seq = p.kv.n_seq;
  // walks the runs tid, tid + NT, ...: `base` runs lie in front of sequence s
  struct Walk {
    int s = -1, q0 = 0, n = 0, runs = 0;
    int64_t base = 0;
  };
  auto advance = [&](Walk& w, int64_t i) {
    while (w.s < n_seq && i >= w.base + w.runs) {
      w.base += w.runs;
      w.runs = 0;
      if (++w.s < n_seq) {
        seq_rows(p, w.s, w.q0, w.n);
        w.runs = runs_of(p, w.n);
      }
    }
    return w.s < n_seq;
  };
  auto cost_at = [&](Walk& w, int64_t i) {
    return advance(w, i) ? cost_of(p, make_unit<KT>(p, w.s, (int)(i - w.base), w.q0, w.n)) : 0;
  };
  // inclusive sum over the warp
  auto scan = [&](int64_t x) {
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    return x;
  };
  // the first NT runs are added up in order (often there are no more), the others only as a total
  Walk w;
  int cost = cost_at(w, tid), most = cost;
  int64_t upto = scan(cost), sum = cost;
  {
    Walk rest = w;
    for (int64_t i = (int64_t)tid + NT; advance(rest, i); i += NT) {
      const int c = cost_at(rest, i);
      sum += c;
      most = max(most, c);
    }
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, d);
    most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
  }
  if (lane == 31) {
    sm.sums[warp] = upto;
    sm.all[warp] = sum;
    sm.most[warp] = most;
  }
  __syncthreads();
  int64_t steps = 0;
#pragma unroll
  for (int i = 0; i < NT / 32; ++i) {
    steps += sm.all[i];
    most = max(most, sm.most[i]);
  }
  const int64_t HC = (int64_t)p.kv.H_kv * p.chunks;
  sh.total = steps * HC;
  const int64_t k = blockIdx.x;
  const int64_t least = max(p.min_steps, (most + p.max_parts - 1) / p.max_parts);
  sh.ctas = min((int64_t)gridDim.x, (sh.total + least - 1) / least);
  if (k >= sh.ctas) return false;
  sh.cur = k * sh.total / sh.ctas;
  sh.end = (k + 1) * sh.total / sh.ctas;
  int64_t front = 0;  // steps per head in front of the NT runs at hand
  for (int64_t i = tid;; i += NT) {
    if (i != tid) {
      cost = cost_at(w, i);
      upto = scan(cost);
      __syncthreads();
      if (lane == 31) sm.sums[warp] = upto;
      __syncthreads();
    }
    int64_t all = 0;
    upto += front;
#pragma unroll
    for (int v = 0; v < NT / 32; ++v) {
      if (v < warp) upto += sm.sums[v];
      all += sm.sums[v];
    }
    if (cost > 0 && sh.cur >= (upto - cost) * HC && sh.cur < upto * HC) {
      sm.s = w.s;
      sm.r = (int)(i - w.base);
      sm.before = upto - cost;
    }
    front += all;
    if (sh.cur < front * HC) break;  // (cur < total: the runs end no earlier)
  }
  __syncthreads();
  sh.s = sm.s;
  sh.r = sm.r;
  sh.before = sm.before;
  return true;
}

// The part of a unit that a CTA takes: entries [j0, j1) of its list, for one kv head and chunk of query heads.
struct Seg {
  Unit u;
  int g, h0, heads;    // kv head, first query head, query heads
  int j0, j1;
  int64_t first_step;  // of the unit's key tiles, among all steps

  __device__ __forceinline__ bool whole() const { return j0 == 0 && j1 == u.nk; }
};

// Walks the segments of a share; every warp that needs them keeps its own.
template <int KT>
struct Segments {
  const AttnParams& p;
  int64_t cur, end, before;
  int q0, n;  // the sequence's rows
  Unit u;

  __device__ __forceinline__ Segments(const AttnParams& pp, const Share& sh)
      : p(pp), cur(sh.cur), end(sh.end), before(sh.before) {
    seq_rows(p, sh.s, q0, n);
    u = make_unit<KT>(p, sh.s, sh.r, q0, n);
  }
  __device__ __forceinline__ bool next(Seg& sg) {
    const int64_t HC = (int64_t)p.kv.H_kv * p.chunks;
    while (cur < end) {
      int cost = cost_of(p, u);
      while (cur >= (before + cost) * HC) {  // to the next run that sees anything
        before += cost;
        int s = u.s, r = u.r + 1;
        while (r >= runs_of(p, n)) {
          seq_rows(p, ++s, q0, n);
          r = 0;
        }
        u = make_unit<KT>(p, s, r, q0, n);
        cost = cost_of(p, u);
      }
      const int64_t at = cur - before * HC;
      const int hu = (int)(at / cost);
      const int v0 = (int)(at - (int64_t)hu * cost), v1 = (int)min((int64_t)cost, v0 + (end - cur));
      sg.first_step = cur - v0 + p.unit_cost;
      cur += v1 - v0;
      sg.j0 = max(v0 - p.unit_cost, 0);
      sg.j1 = max(v1 - p.unit_cost, 0);
      if (sg.j0 >= sg.j1) continue;  // none of the unit's tiles
      sg.u = u;
      sg.g = hu / p.chunks;
      const int c = hu - sg.g * p.chunks;
      sg.h0 = sg.g * p.group + c * p.hp;
      sg.heads = min(p.hp, p.group - c * p.hp);
      return true;
    }
    return false;
  }
};

// CTAs that hold a unit's first and last key tile.
__device__ __forceinline__ void holders(const Share& sh, const Seg& sg, int& first, int& last) {
  first = (int)(((sg.first_step + 1) * sh.ctas - 1) / sh.total);
  last = (int)(((sg.first_step + sg.u.nk) * sh.ctas - 1) / sh.total);
}
// Slot of CTA c's part of a unit whose first step CTA `first` holds (a CTA has one unit that begins in it and goes on,
// and one that began before, at most).
__device__ __forceinline__ int64_t slot_of(int c, int first) { return 2 * (int64_t)c + (c == first ? 1 : 0); }

// Rows that see nothing, where no unit need take them: negative positions (the sequence holds fewer rows than its new
// ones), and without sinks those whose window begins behind the last row that the table covers.  Lengths beyond the table
// are recorded.
template <typename T, int D, int NT>
__device__ void empty_rows(const AttnParams& p) {
  for (int s = blockIdx.x; s < p.kv.n_seq; s += gridDim.x) {
    int q0, n;
    seq_rows(p, s, q0, n);
    const int len = max(__ldg(p.kv.kv_len + s), 0);
    const int held = min(len, p.kv.capacity);
    if (n > 0 && len > p.kv.capacity && threadIdx.x == 0) set_status(p.ws, MR_ERR_DEVICE_CHECK, kTableShort);
    // the first `front` rows and the last `behind` (a position from held + window - 1 on sees nothing)
    const int front = min(max(n - len, 0), n);
    const int64_t late = p.window > 0 && p.sinks == 0 ? (int64_t)len - held - p.window + 1 : 0;
    const int behind = (int)min(max(late, (int64_t)0), (int64_t)(n - front));
    const int64_t m = front + behind;
    const auto row_of = [&](int i) { return q0 + (i < front ? i : n - behind + (i - front)); };
    for (int64_t e = threadIdx.x; e < m * p.H_q * D; e += NT) {
      const int64_t hr = e / D;
      const int h = (int)(hr / m), row = row_of((int)(hr - (int64_t)h * m));
      ((T*)p.o)[(int64_t)h * p.o_head + (int64_t)row * p.o_row + e % D] = from_f32<T>(0.f);
    }
    if (p.lse)
      for (int64_t e = threadIdx.x; e < m * p.H_q; e += NT) {
        const int h = (int)(e / m);
        p.lse[(int64_t)h * p.total_q + row_of((int)(e - (int64_t)h * m))] = -INFINITY;
      }
  }
}

}  // namespace mr
