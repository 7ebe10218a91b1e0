// Attention of a chunk of new rows per sequence over the paged cache on the tensor cores (bf16; pages of a multiple of
// 8 rows; rows of Q and O aligned to 16 bytes).
//
// A unit is two tiles A and B of 128 query rows: runs of new rows times the query heads that share a key head, so a key
// tile serves the whole group, and one persistent CTA per SM walks its share of the units' key tiles (attn_units.cuh).
// Tensor Memory holds S and O of both tiles; P takes the place of S.
//   * producer warp: TMA loads of the query tiles (a box of rows x heads) and of key and value tiles page by page (a
//     lane per box; what nobody sees is asked for outside the pool, which TMA fills with zeros), K_0, K_1,
//     V_0, K_2, V_1, ... through a ring;
//   * an MMA warp for each tile.  The scores of a key tile come in two halves of 64 keys: S_1(j + 1) takes the place of
//     S_1(j) as soon as the softmax has read that, S_0(j + 1) the place of S_0(j) and P(j) behind O += P(j) V_j.  So the
//     softmax works on one half while the products that the other half waits for run.  S, P and O of a tile are ordered
//     by the tensor core's own order, so no barrier says that P has been read;
//   * two softmax warpgroups, a query row per thread: the mask only where some row does not see some key, a row reference
//     that moves when a score passes it by 2^8 (O is then rescaled in Tensor Memory), P = 2^(x - reference) rounded to bf16
//     once, the type that its product with V takes (off by at most 2^-8 of itself, as V is; the sums are of P before that.
//     A second part for what is rounded off, as in decoding, would be half as many products again);
//   * a fix-up warp looks after the values of key tiles that not every row sees: rows that nobody of the unit sees become
//     zeros (0 * NaN would not be 0); in rows that only some see, values that are not finite do, and the softmax warps
//     add them at the end to the rows that do see them.
// Bound by the chain S -> softmax -> P V -> S of each tile, two of which overlap: 16384 exponentials per tile at 16 a
// clock take as long as its two products, and neither alone fills the time.  4 suffixes of 512 to 2048 rows behind 4096,
// 32 heads of 128: 377 us replayed from a graph, 1.08 PFLOP/s, the tensor pipe 68% busy (53% its math, the rest operands
// from shared memory); 439 us as a call among others, under the power limit.  Heads of 64, pages of 16 rows: 295 us.
// Every wait is bounded (MR_ERR_TIMEOUT, then drain and free Tensor Memory).
#include <cuda_bf16.h>

#include "attn_ptx.cuh"
#include "attn_units.cuh"
#include "kernels.h"
#include "profile.h"
#include "sm100.cuh"
#include "tma_host.h"

namespace mr {
namespace {

using namespace sm100;

constexpr int kThreads = 384;
constexpr int kProducerWarp = 0;
constexpr int kMmaWarp0 = 1;      // tile A; tile B: warp 3
constexpr int kFixWarp = 2;
constexpr int kSoftmaxWarp0 = 4;
constexpr int kSoftmaxWarps = 8;  // a warpgroup for each tile
// Each SM sub-partition holds one warp of each warpgroup: 72 + 216 + 216 registers of the launch's 3 x 168.
constexpr int kLaunchRegs = 168;
constexpr int kRegsControl = 72;
constexpr int kRegsSoftmax = 216;
static_assert(kRegsControl + 2 * kRegsSoftmax == 3 * kLaunchRegs, "register split");
constexpr int kKeys = 128;
constexpr int kHalf = 64;         // keys whose scores and P are handed over at a time
constexpr int kMaxHeads = 32;     // query heads of a tile at most
constexpr int kMaxCtas = 152;     // one per SM
constexpr int kSlowRing = 16;     // segments that can be under way at once, and more
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr float kRescale = 8.0f;
constexpr float kLn2 = 0.6931471805599453f;

template <int D>
struct Smem {
  static constexpr int kHalves = D / 64;
  static constexpr int kSlots = D == 128 ? 5 : 8;
  static constexpr int kSlotBytes = kHalves * 128 * 128;
  __nv_bfloat16 q[2][kHalves][128 * 64];         // [tile][column half][row][64]
  __nv_bfloat16 kv[kSlots][kHalves][128 * 64];   // [slot][column half][key][64]
  uint64_t q_full, q_empty;
  uint64_t slot_full[kSlots], slot_empty[kSlots], slot_fixed[kSlots];
  uint64_t s_full[2][2], p_full[2][2];           // [tile][key half]
  uint64_t s_read[2];                            // the second half's scores are in registers
  uint64_t o_full[2], o_free[2];
  uint64_t part_done, join_go, mma_done;
  PartitionSmem part;
  uint32_t tmem_base;
  int abort;
  int slow[kSlowRing];  // segment number + 1 where values were taken out
  int join;
};

struct Maps {
  CUtensorMap q, k, v;
};

template <int D>
__device__ __forceinline__ void fail(Smem<D>& s, const AttnParams& p, uint32_t detail) {
  set_status(p.ws, MR_ERR_TIMEOUT, detail);
  s.abort = 1;
}

// Whether it holds in all lanes.  A vote alone does not say that the lanes go on together, and each has polled in a loop of
// its own before it; what follows a wait are instructions that a whole warp has to issue as one.
__device__ __forceinline__ bool warp_all(bool ok) {
  ok = __all_sync(0xffffffffu, ok);
  __syncwarp();
  return ok;
}

// mbar_wait by a whole warp for the phase with `n`'s parity: all lanes go on, or none.  All of them wait: a form in which
// one lane did and the others met it at the vote faulted.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t n, const volatile int* abort, uint64_t ns) {
  return warp_all(mbar_wait(bar, n & 1, abort, ns));
}

// Rows of positions first .. last: is there one of the N keys from key0 on that some row does not see?
template <int N>
__device__ __forceinline__ bool on_edge(int window, int sinks, int first, int last, int held, int key0) {
  return (key0 + N - 1 > min(first, held - 1)) |
         ((window > 0) & (last >= window) & (key0 <= last - window) & (key0 + N > sinks));
}

// Bits 0 .. n - 1, for any n.
__device__ __forceinline__ uint32_t below(int n) { return n >= 32 ? 0xffffffffu : (1u << max(n, 0)) - 1u; }

// Key tiles of the segment that tile x of the unit needs (a front part of them), 0 for a missing tile.
__device__ __forceinline__ int steps_of(const AttnParams& p, const Seg& sg, int x) {
  if (x * p.tile_tokens >= sg.u.n) return 0;
  const int hi = min(sg.u.pos0 + min((x + 1) * p.tile_tokens, sg.u.n) - 1, sg.u.held - 1);
  return min(max(tiles_upto<kKeys>(sg.u, hi) - sg.j0, 0), sg.j1 - sg.j0);
}

// ------------------------------------------------------------------------------------------------
template <int D>
__device__ void producer(Smem<D>& s, const AttnParams& p, const Share& sh, const Maps& maps, int box_rows) {
  constexpr int kSlots = Smem<D>::kSlots, kHalves = Smem<D>::kHalves;
  const int lane = threadIdx.x & 31;
  const int boxes = kKeys / box_rows;
  const int nowhere = p.kv.n_pages * p.kv.H_kv * p.kv.page_rows;  // the row behind the pool
  Segments<kKeys> walk(p, sh);
  Seg sg;
  uint32_t item = 0, segs = 0;
  bool ok = true;
  while (ok && walk.next(sg)) {
    const Unit& u = sg.u;
    if (segs > 0) ok = mbar_wait_sleep(&s.q_empty, (segs - 1) & 1, &s.abort, p.wait_ns, 64);
    ok = warp_all(ok);
    if (!ok) {
      if (lane == 0) fail(s, p, 0xA01);
      break;
    }
    if (lane == 0) {
      const int tiles = u.n > p.tile_tokens ? 2 : 1;
      mbar_arrive_expect_tx(&s.q_full, (uint32_t)(tiles * kHalves * p.hp * p.tile_tokens * 128));
      for (int x = 0; x < tiles; ++x)
        for (int c = 0; c < kHalves; ++c)
          tma_load_3d(&s.q[x][c][0], &maps.q, &s.q_full, 64 * c, u.q0 + x * p.tile_tokens, sg.h0);
    }
    ++segs;
    const int hi = min(u.pos0 + u.n - 1, u.held - 1);
    const int lo = p.window > 0 && u.pos0 >= p.window ? u.pos0 - p.window + 1 : 0;
    auto lookup = [&](int j) {
      const int key = tile_of(u, j) * kKeys + lane * box_rows;
      if (j >= sg.j1 || lane >= boxes || key > hi || (key >= p.sinks && key + box_rows - 1 < lo)) return nowhere;
      const int r = pool_row(p.kv, u.s, sg.g, key);
      if (r < 0) set_status(p.ws, MR_ERR_DEVICE_CHECK, kBadPage);
      return r < 0 ? nowhere : r;
    };
    // K_0, then K_{j+1} and V_j for each j
    int row = lookup(sg.j0), next_row = row;
    for (int j = sg.j0 - 1; j < sg.j1 && ok; ++j) {
      for (int kv = 0; kv < 2; ++kv) {
        if (kv == 0 ? j + 1 >= sg.j1 : j < sg.j0) continue;
        const int sl = item % kSlots;
        const uint32_t use = item / kSlots;
        ++item;
        if (use > 0) ok = mbar_wait_sleep(&s.slot_empty[sl], (use - 1) & 1, &s.abort, p.wait_ns, 64);
        ok = warp_all(ok);
        if (!ok) {
          --item;
          if (lane == 0) fail(s, p, 0xA02);
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(&s.slot_full[sl], Smem<D>::kSlotBytes);
        __syncwarp();
        if (lane < boxes)
          for (int c = 0; c < kHalves; ++c)
            tma_load_2d(&s.kv[sl][c][lane * box_rows * 64], kv ? &maps.v : &maps.k, &s.slot_full[sl], 64 * c,
                        kv ? row : next_row);
      }
      row = next_row;
      next_row = lookup(j + 2);
    }
  }
  // no load may land after the CTA releases its shared memory
  if (lane == 0) {
    const int never = 0;
    for (uint32_t i = item > (uint32_t)kSlots ? item - kSlots : 0; i < item; ++i)
      mbar_wait(&s.slot_full[i % kSlots], (i / kSlots) & 1, &never, kTimeoutNs);
    if (segs > 0) mbar_wait(&s.q_full, (segs - 1) & 1, &never, kTimeoutNs);
  }
}

// ------------------------------------------------------------------------------------------------
// A warp per tile.  The whole warp runs the loop, one elected lane issues: what the tensor core's instructions take
// (descriptors, Tensor Memory addresses) then stays in uniform registers.  (One lane that ran it alone spent 1.0 us on a
// tile's 16 products, which themselves take 0.54 us.)  Items of the ring that this tile does not need are passed on.
template <int D>
__device__ void mma_issuer(Smem<D>& s, const AttnParams& p, const Share& sh, int x) {
  constexpr int kSlots = Smem<D>::kSlots;
  constexpr uint32_t kSlotLo = Smem<D>::kSlotBytes >> 4;  // a slot further, in a descriptor's low word
  const uint32_t id_qk = idesc_bf16_f32(128, kHalf, false, false) | (p.negate ? kIdescNegateA : 0u);
  constexpr uint32_t id_pv = idesc_bf16_f32(128, D, false, true);
  const int lane = threadIdx.x & 31;
  const uint32_t s_col = __shfl_sync(0xffffffffu, s.tmem_base, 0) + 256 * x, o_col = s_col + 128;
  const bool leader = elect_one();
  // Q and K: K-major (distance of 8-row groups 1024); V: MN-major (column halves 16 KB apart)
  const uint64_t q_desc = sdesc_sw128(smem_u32(&s.q[x][0][0]), 16, 1024);
  const uint64_t k_desc = sdesc_sw128(smem_u32(&s.kv[0][0][0]), 16, 1024);
  const uint64_t v_desc = sdesc_sw128(smem_u32(&s.kv[0][0][0]), 128 * 128, 1024);
  Segments<kKeys> walk(p, sh);
  Seg sg;
  uint32_t segs = 0, fixed = 0;        // fixed: a parity bit per slot
  uint32_t slot = 0, round = 0;        // ring position of the next item, and its use's parity
  uint32_t pc = 0, oc = 0, where = 0;  // steps (P tiles) and outputs so far
  auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t code) {
    const bool ok = warp_wait(bar, parity, &s.abort, p.wait_ns);
    if (!ok) where = code;
    return ok;
  };
  auto advance = [&] {
    if (++slot == kSlots) slot = 0, round ^= 1;
  };
  // S of key half h = Q K^T, K in slot `sl`
  auto scores = [&](uint32_t sl, int h) {
    tc_fence_after();
    const uint64_t kd = k_desc + sl * kSlotLo + h * (kHalf * 128 >> 4);
    if (leader) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk >> 2) * 128 * 128 + 32 * (kk & 3)) >> 4;
        mma_bf16_ss(s_col + kHalf * h, q_desc + off, kd + off, id_qk, kk > 0 ? 1u : 0u);
      }
      mma_commit(&s.s_full[x][h]);
    }
  };
  // an item's slot is free again once this tile's products that read it are done (at once where there are none)
  auto release = [&](uint32_t sl, bool used) {
    if (used && leader) mma_commit(&s.slot_empty[sl]);
    if (!used && lane == 0) mbar_arrive(&s.slot_empty[sl]);
  };
  bool ok = true;
  while (ok && walk.next(sg)) {
    const Unit& u = sg.u;
    const int n = sg.j1 - sg.j0, nx = steps_of(p, sg, x);
    ok = wait(&s.q_full, segs++, 0xA11);
    if (ok && nx == 0 && lane == 0) mbar_arrive(&s.q_empty);
    ok = ok && wait(&s.slot_full[slot], round, 0xA12);
    if (!ok) break;
    if (nx > 0) {
      scores(slot, 1);
      scores(slot, 0);
    }
    release(slot, nx > 0);
    if (nx == 1 && leader) mma_commit(&s.q_empty);
    advance();
    for (int j = 0; j < n; ++j) {
      const bool use_v = j < nx, use_k = j + 1 < nx;
      const uint32_t k_slot = slot;
      if (j + 1 < n) {
        if (!(ok = wait(&s.slot_full[slot], round, 0xA13))) break;
        if (use_k) {  // the second half's scores are in registers: the next ones can take their place
          if (!(ok = wait(&s.s_read[x], pc, 0xA18))) break;
          scores(k_slot, 1);
        }
        advance();
      }
      if (!(ok = wait(&s.slot_full[slot], round, 0xA13))) break;
      if (on_edge<kKeys>(p.window, p.sinks, u.pos0, u.pos0 + u.n - 1, u.held, tile_of(u, sg.j0 + j) * kKeys)) {
        if (use_v && !(ok = wait(&s.slot_fixed[slot], fixed >> slot, 0xA14))) break;
        fixed ^= 1u << slot;
      }
      if (use_v) {
        if (j == 0 && oc > 0 && !(ok = wait(&s.o_free[x], oc - 1, 0xA15))) break;
        const uint64_t vd = v_desc + slot * kSlotLo;
#pragma unroll
        for (int h = 1; h >= 0; --h) {  // (P of keys 64 .. 127 comes first)
          if (ok) ok = wait(&s.p_full[x][h], pc, 0xA16);
          tc_fence_after();
          if (leader && ok) {
#pragma unroll
            for (int kk = 4 * h; kk < 4 * h + 4; ++kk)
              mma_bf16_ts(o_col, s_col + 8 * kk, vd + (2048 >> 4) * kk, id_pv, (j > 0 || kk != 4) ? 1u : 0u);
          }
        }
        if (!ok) break;
        ++pc;
        if (!use_k) {
          if (leader) mma_commit(&s.o_full[x]);
          ++oc;
        }
      }
      release(slot, use_v);
      if (use_k) scores(k_slot, 0);
      if (j + 1 < n) release(k_slot, use_k);
      if (j + 2 == nx && leader) mma_commit(&s.q_empty);
      advance();
    }
  }
  if (!ok && lane == 0) fail(s, p, where);
  // every MMA of this warp completes before Tensor Memory is released
  if (leader) mma_commit(&s.mma_done);
  __syncwarp();
  const int never = 0;
  mbar_wait(&s.mma_done, 0, &never, kTimeoutNs);
}

// ------------------------------------------------------------------------------------------------
// Follows the ring item by item, so that it never mistakes one use of a slot for another.
template <int D>
__device__ void fixer(Smem<D>& s, const AttnParams& p, const Share& sh) {
  constexpr int kSlots = Smem<D>::kSlots, kHalves = Smem<D>::kHalves;
  const int lane = threadIdx.x & 31;
  Segments<kKeys> walk(p, sh);
  Seg sg;
  uint32_t item = 0, segs = 0;
  while (walk.next(sg)) {
    const Unit& u = sg.u;
    const int last = u.pos0 + u.n - 1;
    const int hi = min(last, u.held - 1), all = min(u.pos0, u.held - 1);  // up to `all`: no row is too early
    const int lo = p.window > 0 && u.pos0 >= p.window ? u.pos0 - p.window + 1 : 0;
    const int from = p.window > 0 && last >= p.window ? last - p.window + 1 : 0;  // from here on: no window is past
    for (int j = sg.j0 - 1; j < sg.j1; ++j) {
      const int key0 = tile_of(u, max(j, sg.j0)) * kKeys;
      for (int kv = 0; kv < 2; ++kv) {
        if (kv == 0 ? j + 1 >= sg.j1 : j < sg.j0) continue;
        const int sl = item % kSlots;
        bool ok = mbar_wait_sleep(&s.slot_full[sl], (item / kSlots) & 1, &s.abort, 2 * p.wait_ns, 64);
        ++item;
        ok = warp_all(ok);
        if (!ok) {
          if (lane == 0) fail(s, p, 0xA21);
          return;
        }
        if (kv == 1 && on_edge<kKeys>(p.window, p.sinks, u.pos0, last, u.held, key0)) {
          // lane: 16 bytes of row 4 g + lane / 8 in each group g of 4 rows
          char* v = reinterpret_cast<char*>(&s.kv[sl][0][0]) + lane * 16;
          uint32_t bad = 0;
#pragma unroll 1
          for (int g0 = 0; g0 < 32; g0 += 4) {
            uint32_t dead = 0, look = 0;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const int key = key0 + 4 * (g0 + g) + (lane >> 3);
              const uint32_t first = key < p.sinks;
              const uint32_t d = (uint32_t)(key > hi) | ((uint32_t)(key < lo) & (first ^ 1u));
              const uint32_t full = (uint32_t)(key <= all) & ((uint32_t)(key >= from) | first);
              dead |= d << g;
              look |= ((d | full) ^ 1u) << g;
            }
            if (__any_sync(0xffffffffu, look != 0)) {
              uint4 y[4][kHalves];
#pragma unroll
              for (int g = 0; g < 4; ++g)
#pragma unroll
                for (int c = 0; c < kHalves; ++c)
                  y[g][c] = *reinterpret_cast<const uint4*>(v + c * 128 * 128 + (g0 + g) * 512);
#pragma unroll
              for (int g = 0; g < 4; ++g)
#pragma unroll
                for (int c = 0; c < kHalves; ++c) {
                  const uint32_t hit = (look >> g & 1u) ? not_finite(y[g][c].x) | not_finite(y[g][c].y) |
                                                              not_finite(y[g][c].z) | not_finite(y[g][c].w)
                                                        : 0u;
                  bad |= hit;
                  if (hit)
                    *reinterpret_cast<uint4*>(v + c * 128 * 128 + (g0 + g) * 512) =
                        make_uint4(y[g][c].x & ~not_finite(y[g][c].x), y[g][c].y & ~not_finite(y[g][c].y),
                                   y[g][c].z & ~not_finite(y[g][c].z), y[g][c].w & ~not_finite(y[g][c].w));
                }
            }
            if (__any_sync(0xffffffffu, dead != 0)) {
#pragma unroll
              for (int g = 0; g < 4; ++g)
#pragma unroll
                for (int c = 0; c < kHalves; ++c)
                  if (dead >> g & 1u) *reinterpret_cast<uint4*>(v + c * 128 * 128 + (g0 + g) * 512) = make_uint4(0, 0, 0, 0);
            }
          }
          fence_proxy_async_smem();
          if (__any_sync(0xffffffffu, bad != 0) && lane == 0) *(volatile int*)&s.slow[segs % kSlowRing] = (int)segs + 1;
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.slot_fixed[sl]);
        }
        if (lane == 0) mbar_arrive(&s.slot_empty[sl]);
      }
    }
    ++segs;
  }
}

// ------------------------------------------------------------------------------------------------
// Where a part of a unit goes: 256 (reference, sum) pairs, then outputs as [column / 4][row] float4.
template <int D>
__device__ __forceinline__ float* slot_ptr(const AttnParams& p, int64_t slot) {
  return p.part + slot * (256 * (D + 2));
}

template <int D>
__device__ __forceinline__ float4* slot_out(float* slot, int c4, int row) {
  return reinterpret_cast<float4*>(slot + 512) + c4 * 256 + row;
}

__device__ __forceinline__ uint32_t pack2(float x, float y) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// 32 bytes of a row: one store fills a sector of L2, two would write it in halves.
__device__ __forceinline__ void store32(void* dst, const uint32_t (&q)[8], bool aligned) {
  if (aligned) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(q[0]), "r"(q[1]), "r"(q[2]),
                 "r"(q[3]), "r"(q[4]), "r"(q[5]), "r"(q[6]), "r"(q[7])
                 : "memory");
  } else {
    *reinterpret_cast<uint4*>(dst) = make_uint4(q[0], q[1], q[2], q[3]);
    *(reinterpret_cast<uint4*>(dst) + 1) = make_uint4(q[4], q[5], q[6], q[7]);
  }
}

// Adds what the fix-up warp has taken out: p_j v_j for the elements of v_j that are not finite, where this lane's row
// sees key j.  The warp looks through the values of the segment's tiles that not every row sees; O is in Tensor Memory.
template <int D>
__device__ __noinline__ void put_back(const AttnParams& p, const Seg& sg, uint32_t o_addr, int pos, int last, float ref,
                                      const __nv_bfloat16* q) {
  constexpr int C = D / 32;
  const int lane = threadIdx.x & 31;
  const Unit& u = sg.u;
  const int u_last = u.pos0 + u.n - 1, hi = min(u_last, u.held - 1);
  const int lo = p.window > 0 && u.pos0 >= p.window ? u.pos0 - p.window + 1 : 0;
  const float a = p.negate ? -p.a : p.a;
  for (int j = sg.j0; j < sg.j1; ++j) {
    const int key0 = tile_of(u, j) * kKeys;
    if (!on_edge<kKeys>(p.window, p.sinks, u.pos0, u_last, u.held, key0)) continue;
    for (int key = key0; key < key0 + kKeys && key <= hi; ++key) {
      if (key < lo && key >= p.sinks) continue;
      const int at = pool_row(p.kv, u.s, sg.g, key);
      if (at < 0) continue;
      const __nv_bfloat16* v = (const __nv_bfloat16*)p.kv.v + (int64_t)at * D;
      uint32_t bad = 0;
#pragma unroll
      for (int c = 0; c < C; c += 2) bad |= not_finite(*reinterpret_cast<const uint32_t*>(v + C * lane + c));
      if (!__any_sync(0xffffffffu, bad != 0)) continue;
      const bool sees = key <= last && (p.window == 0 || pos < p.window || key > pos - p.window || key < p.sinks);
      float e = 0.f;
      if (sees) {
        const __nv_bfloat16* k = (const __nv_bfloat16*)p.kv.k + (int64_t)at * D;
        float x = 0.f;
        for (int c = 0; c < D; ++c) x = fmaf(__bfloat162float(q[c]), __bfloat162float(k[c]), x);
        e = ex2_approx(fmaf(x, a, ref == -INFINITY ? 0.f : -ref));
      }
      __syncwarp();
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        tmem_ld32(o_addr + c, o);
        tmem_wait_ld();
        tmem_ld32_done(o);
#pragma unroll
        for (int t = 0; t < 32; ++t) {
          const float y = __bfloat162float(v[c + t]);
          if (sees && !isfinite(y)) o[t] = __float_as_uint(fmaf(e, y, __uint_as_float(o[t])));
        }
        __syncwarp();
        tmem_st32(o_addr + c, o);
        tmem_wait_st();
      }
    }
  }
}

// The outputs of a warp's 32 rows from all parts of the unit; `own`: maximum and 1 / sum of this lane's row.  Where the
// warp has rows that do not exist, an item is 4 columns of a row, and up to 8 parts of it are under way at once.
template <int D>
__device__ __noinline__ void join_rows(const AttnParams& p, const Seg& sg, int x, int q4, int first, int lastc,
                                       float2 own) {
  const int lane = threadIdx.x & 31;
  // rows of the warp that exist, as a mask: head r / tile_tokens, new row r % tile_tokens
  const int r0 = 32 * q4 + lane;
  const int hh0 = (int)fast_div((uint32_t)r0, p.by_tile_tokens);
  const bool mine = hh0 < sg.heads && x * p.tile_tokens + r0 - hh0 * p.tile_tokens < sg.u.n;
  const uint32_t mask = __ballot_sync(0xffffffffu, mine);
  if (mask == 0xffffffffu) {
    // a full warp: a lane per row, 32 columns of it at a time from two parts
    const int at = 128 * x + r0, tok = x * p.tile_tokens + r0 - hh0 * p.tile_tokens;
    __nv_bfloat16* o = (__nv_bfloat16*)p.o + (int64_t)(sg.h0 + hh0) * p.o_head + (int64_t)(sg.u.q0 + tok) * p.o_row;
#pragma unroll 1
    for (int g = 0; g < D / 32; ++g) {
      float4 acc[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
      for (int c = first; c <= lastc; ++c) {
        float* part = slot_ptr<D>(p, slot_of(c, first));
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(part) + at);
        const float w = ex2_approx(ml.x - own.x) * own.y;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float4 y = __ldcg(slot_out<D>(part, 8 * g + e, at));
          acc[e].x = fmaf(w, y.x, acc[e].x);
          acc[e].y = fmaf(w, y.y, acc[e].y);
          acc[e].z = fmaf(w, y.z, acc[e].z);
          acc[e].w = fmaf(w, y.w, acc[e].w);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        uint32_t q[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          q[2 * i] = pack2(acc[e + i].x, acc[e + i].y);
          q[2 * i + 1] = pack2(acc[e + i].z, acc[e + i].w);
        }
        store32(o + 32 * g + 4 * e, q, p.vec_o == 2);
      }
    }
    return;
  }
  const int n = __popc(mask);
  const int kth = (int)__fns(mask, 0, lane + 1);  // the lane-th row that exists
  for (int e0 = 0; e0 < n * (D / 4); e0 += 32) {
    const int e = e0 + lane;
    const int c4 = e / n;
    const int i = __shfl_sync(0xffffffffu, kth, e - c4 * n);
    const float2 mi = make_float2(__shfl_sync(0xffffffffu, own.x, i), __shfl_sync(0xffffffffu, own.y, i));
    if (c4 >= D / 4) continue;
    const int r = 32 * q4 + i, at = 128 * x + r;
    const int hh = (int)fast_div((uint32_t)r, p.by_tile_tokens);
    const int tok = x * p.tile_tokens + r - hh * p.tile_tokens;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c0 = first; c0 <= lastc; c0 += 8) {
      float4 y[8];
      float2 ml[8];
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        ml[b] = make_float2(-INFINITY, 0.f);
        y[b] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c0 + b <= lastc) {
          float* part = slot_ptr<D>(p, slot_of(c0 + b, first));
          ml[b] = __ldcg(reinterpret_cast<const float2*>(part) + at);
          y[b] = __ldcg(slot_out<D>(part, c4, at));
        }
      }
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        const float w = ex2_approx(ml[b].x - mi.x) * mi.y;
        acc.x = fmaf(w, y[b].x, acc.x);
        acc.y = fmaf(w, y[b].y, acc.y);
        acc.z = fmaf(w, y[b].z, acc.z);
        acc.w = fmaf(w, y[b].w, acc.w);
      }
    }
    __nv_bfloat16* o = (__nv_bfloat16*)p.o + (int64_t)(sg.h0 + hh) * p.o_head + (int64_t)(sg.u.q0 + tok) * p.o_row + 4 * c4;
    *reinterpret_cast<uint2*>(o) = make_uint2(pack2(acc.x, acc.y), pack2(acc.z, acc.w));
  }
}

// Columns of O multiplied by f.
template <int N>
__device__ __forceinline__ void rescale(uint32_t addr, float f) {
#pragma unroll 1
  for (int c = 0; c < N; c += 16) {
    uint32_t o[16];
    tmem_ld16(addr + c, o);
    tmem_wait_ld();
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      asm volatile("" : "+r"(o[t]));  // (not read in front of the wait)
      o[t] = __float_as_uint(__uint_as_float(o[t]) * f);
    }
    tmem_st16(addr + c, o);
  }
  tmem_wait_st();
}

// A segment's softmax steps of one warp: what it needs, and nothing that the caller keeps across the segment (the call
// boundary keeps that out of the loop's registers).
struct Steps {
  float a;
  uint64_t wait_ns;
  int window, sinks;
  int x, n;                      // tile, key tiles
  int first_pos, last_pos;       // of the tile's rows
  int held, pos, last;           // rows the table covers; this row's position, the last row it sees
  int tile, ahead, lo_t;         // first key tile; after `ahead` of them the list goes on at tile lo_t
  uint32_t sc;                   // key tiles of this tile so far
  int skip;                      // failure-path test: the first P is not handed over
};

// Scores of keys 64 h .. at Tensor Memory column 256 x + 64 h, all of P in the first half's columns.  The second half
// is worked on first: its scores are computed while the previous step's P is still being made, so its exponentials run
// during the products that the first half's scores wait for.  They use the reference as it stands; where the first half
// then moves it (in a segment's first steps, hardly later), P of the second half is scaled.  That move goes by whole
// steps, so the factor is a power of two and P is not rounded a second time.
template <int D>
__device__ __noinline__ bool softmax_steps(Smem<D>& s, const Steps t, float& ref_out, float& l_out) {
  // (copies that no memory clobber makes the compiler read again)
  const int x = t.x, steps = t.n, last = t.last, sinks = t.sinks, ahead = t.ahead, lo_t = t.lo_t;
  const int win_lo = t.window > 0 && t.pos >= t.window ? t.pos - t.window + 1 : 0;  // the row's window
  const int full_hi = min(t.first_pos, t.held - 1) - (kHalf - 1);  // halves from here on: not every row sees all of them
  const int past = t.window > 0 ? t.last_pos - t.window : -1;      // halves up to here: neither ...
  const int from = t.sinks - kHalf;                                // ... unless they come before that
  const uint32_t sc = t.sc;
  const uint64_t wait_ns = t.wait_ns;
  const bool skip = t.skip != 0;
  const float a = t.a;
  const float2 a2 = make_float2(a, a);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t s_addr = s.tmem_base + ((uint32_t)(32 * (warp & 3)) << 16) + 256 * x;
  uint64_t* const s_full = s.s_full[x];
  uint64_t* const p_full = s.p_full[x];
  float ref = -INFINITY;  // row reference (base 2)
  float l = 0.f;          // row sum of 2^(x - ref)
  int tile = t.tile;
  uint32_t r[2][32];
  // the scores of 64 keys from k0 on, -infinity where this row does not see them; returns their maximum
  auto load = [&](int h, int k0) {
#pragma unroll
    for (int c = 0; c < 2; ++c) tmem_ld32(s_addr + kHalf * h + 32 * c, r[c]);
    tmem_wait_ld();
#pragma unroll
    for (int c = 0; c < 2; ++c) tmem_ld32_done(r[c]);
    if ((k0 > full_hi) | ((k0 <= past) & (k0 > from))) {
      const int hi = last + 1 - k0, lo = win_lo - k0, sk = sinks - k0;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint32_t seen = below(hi - 32 * c) & (~below(lo - 32 * c) | below(sk - 32 * c));
#pragma unroll
        for (int b = 0; b < 32; ++b) r[c][b] = (seen & (1u << b)) ? r[c][b] : 0xff800000u;
      }
    }
    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int e = 0; e < 64; e += 8)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        mx[c] = max3_nan(mx[c], __uint_as_float(r[e >> 5][(e & 31) + 2 * c]), __uint_as_float(r[e >> 5][(e & 31) + 2 * c + 1]));
    return max3_nan(max3_nan(mx[0], mx[1], mx[2]), mx[3], mx[3]) * a;
  };
  // P of the scores at hand as bf16 pairs, and its sum
  auto exponentials = [&](uint32_t (&pk)[32]) {
    const float neg = ref == -INFINITY ? 0.f : -ref;  // (a score of +infinity makes the row NaN)
    const float2 n2 = make_float2(neg, neg);
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const float2 y = fma2(make_float2(__uint_as_float(r[e >> 4][(2 * e) & 31]), __uint_as_float(r[e >> 4][(2 * e + 1) & 31])),
                            a2, n2);
      const float2 z = make_float2(ex2_approx(y.x), ex2_approx(y.y));
      sum[e & 1] = add2(sum[e & 1], z);
      pk[e] = pack2(z.x, z.y);
    }
    sum[0] = add2(sum[0], sum[1]);
    l += sum[0].x + sum[0].y;
  };
  // The reference moves to the row maximum at the first finite score (so a row that sees one key gives it exactly 1) and
  // whenever a score passes it by more than 2^8, with `whole` to the next whole step above that; returns whether one of the
  // warp's rows did, and what its sums have to be multiplied by.
  auto move = [&](float mt, float& f, bool whole) {
    const bool need = ref == -INFINITY ? mt > -INFINITY : mt - ref > kRescale;
    if (!__any_sync(0xffffffffu, need)) return false;
    f = 1.f;
    if (need) {
      const float by = ceilf(mt - ref);  // (infinite at the first finite score)
      if (whole && by < 126.f) {
        f = __int_as_float((127 - (int)by) << 23);
        ref += by;
      } else {
        f = ref == -INFINITY ? 0.f : ex2_approx(ref - mt);  // (where `whole`: too small to count, however it is rounded)
        ref = mt;
      }
    }
    __syncwarp();
    l *= f;
    return true;
  };
#pragma unroll 1
  for (int j = 0; j < steps; ++j) {
    const int key0 = tile * kKeys;
    tile = j + 1 == ahead ? lo_t : tile + 1;
    float f;
    uint32_t ph[32], pl[32];
    if (!warp_wait(&s_full[1], sc + j, &s.abort, wait_ns)) return false;
    tc_fence_after();
    const float mh = load(1, key0 + kHalf);
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.s_read[x]);
    if (move(mh, f, false) && j > 0) {
      // (the first half's scores are computed behind the last product that adds to O)
      if (!warp_wait(&s_full[0], sc + j, &s.abort, wait_ns)) return false;
      tc_fence_after();
      rescale<D>(s_addr + 128, f);
    }
    exponentials(ph);
    if (!warp_wait(&s_full[0], sc + j, &s.abort, wait_ns)) return false;
    tc_fence_after();
    const float ml = load(0, key0);
    if (move(ml, f, true)) {
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&ph[e]));
        ph[e] = pack2(y.x * f, y.y * f);
      }
      if (j > 0) rescale<D>(s_addr + 128, f);
    }
    tmem_st32(s_addr + 32, ph);
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0 && !(skip && j == 0)) mbar_arrive(&p_full[1]);
    exponentials(pl);
    tmem_st32(s_addr, pl);
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&p_full[0]);
  }
  ref_out = ref;
  l_out = l;
  return true;
}

// Softmax warpgroup of tile x: S_x and P_x at Tensor Memory column 256 x, O_x at 256 x + 128; a query row per thread.
template <int D>
__device__ void softmax_group(Smem<D>& s, const AttnParams& p, const Share& sh, int x) {
  const uint64_t wait_ns = 2 * p.wait_ns;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q4 = warp & 3;
  const int r = 32 * q4 + lane;  // row of the query tile
  const uint32_t o_addr = s.tmem_base + ((uint32_t)(32 * q4) << 16) + 256 * x + 128;
  const int hh = (int)fast_div((uint32_t)r, p.by_tile_tokens);
  const int tok = x * p.tile_tokens + r - hh * p.tile_tokens;
  Segments<kKeys> walk(p, sh);
  Seg sg;
  uint32_t sc = 0, oc = 0, segs = 0, joins = 0;
  for (; walk.next(sg); ++segs) {
    const Unit& u = sg.u;
    const bool whole = sg.whole();
    if (whole && x * p.tile_tokens >= u.n) continue;
    const bool row_ok = hh < sg.heads && tok < u.n;
    const int pos = u.pos0 + tok;
    const int last = row_ok ? min(pos, u.held - 1) : -1;  // last row seen
    const int first_pos = u.pos0 + x * p.tile_tokens;
    const int last_pos = u.pos0 + min((x + 1) * p.tile_tokens, u.n) - 1;
    const int nx = steps_of(p, sg, x);
    float ref = -INFINITY, l = 0.f;
    if (nx > 0 && !softmax_steps<D>(s, Steps{p.a, wait_ns, p.window, p.sinks, x, nx, first_pos, last_pos, u.held, pos, last,
                                   tile_of(u, sg.j0), u.ns - sg.j0, u.lo_t, sc,
                                   p.skip_arrive && x == 0 && sc == 0},
                          ref, l))
      return fail(s, p, 0xA31);
    sc += nx;
    if (nx > 0) {
      if (!warp_wait(&s.o_full[x], oc, &s.abort, wait_ns)) return fail(s, p, 0xA32);
      ++oc;
      tc_fence_after();
    }
    const bool slow = nx > 0 && *(volatile int*)&s.slow[segs % kSlowRing] == (int)segs + 1;
    const int row = u.q0 + tok, h = sg.h0 + hh;
    const int at = 128 * x + r;
    int first = 0, lastc = 0;
    float* slot = nullptr;
    if (!whole) {
      holders(sh, sg, first, lastc);
      if (!checked(p.ws, first >= 0 && lastc < kMaxCtas && (int)blockIdx.x <= lastc, 0xC53)) return fail(s, p, 0xC53);
      slot = slot_ptr<D>(p, slot_of(blockIdx.x, first));
    }
    if (slow)
      put_back<D>(p, sg, o_addr, pos, last, ref,
                  (const __nv_bfloat16*)p.q + (int64_t)(row_ok ? h : sg.h0) * p.q_head +
                      (int64_t)(row_ok ? row : u.q0) * p.q_row);
    {
      uint32_t o[D / 32][32];
      __syncwarp();
      if (nx > 0) {
#pragma unroll
        for (int c = 0; c < D / 32; ++c) tmem_ld32(o_addr + 32 * c, o[c]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < D / 32; ++c) tmem_ld32_done(o[c]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.o_free[x]);
      } else {
#pragma unroll
        for (int e = 0; e < D; ++e) o[e >> 5][e & 31] = 0;
      }
      if (row_ok && whole) {
        if (!checked(p.ws, h < p.H_q && row < p.total_q, 0xC51)) continue;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        if (p.lse) p.lse[(int64_t)h * p.total_q + row] = l == 0.f ? -INFINITY : (ref + log2f(l)) * kLn2;
        __nv_bfloat16* out = (__nv_bfloat16*)p.o + (int64_t)h * p.o_head + (int64_t)row * p.o_row;
#pragma unroll
        for (int g = 0; g < D / 16; ++g) {
          uint32_t q[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int k = 16 * g + 2 * e;
            q[e] = pack2(__uint_as_float(o[k >> 5][k & 31]) * inv, __uint_as_float(o[k >> 5][(k & 31) + 1]) * inv);
          }
          store32(out + 16 * g, q, p.vec_o == 2);
        }
      } else if (row_ok) {
        __stcg(reinterpret_cast<float2*>(slot) + at, make_float2(ref, l));
#pragma unroll
        for (int g = 0; g < D / 4; ++g) {
          const int k = 4 * g;
          __stcg(slot_out<D>(slot, g, at),
                 make_float4(__uint_as_float(o[k >> 5][k & 31]), __uint_as_float(o[k >> 5][(k & 31) + 1]),
                             __uint_as_float(o[k >> 5][(k & 31) + 2]), __uint_as_float(o[k >> 5][(k & 31) + 3])));
        }
      }
    }
    if (whole) continue;
    // the CTA that comes last joins the unit's parts
    __threadfence();
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.part_done);
    if (warp == kSoftmaxWarp0 && lane == 0) {
      if (!mbar_wait(&s.part_done, joins & 1, &s.abort, wait_ns)) {
        fail(s, p, 0xA33);
      } else {
        __threadfence();
        s.join = atomicAdd(p.counters + first, 1u) == (uint32_t)(lastc - first);
        mbar_arrive(&s.join_go);
      }
    }
    __syncwarp();
    if (!warp_wait(&s.join_go, joins, &s.abort, wait_ns)) return fail(s, p, 0xA34);
    const bool join = *(volatile int*)&s.join != 0;
    ++joins;
    if (!join) continue;
    __threadfence();
    // this thread's row: the maximum and the sum over all parts
    float2 own = make_float2(0.f, 0.f);
    if (row_ok) {
      float m = -INFINITY, sum = 0.f;
      for (int c0 = first; c0 <= lastc; c0 += 8) {
        float2 ml[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          ml[i] = c0 + i <= lastc ? __ldcg(reinterpret_cast<const float2*>(slot_ptr<D>(p, slot_of(c0 + i, first))) + at)
                                  : make_float2(-INFINITY, 0.f);
        float mm = m;
#pragma unroll
        for (int i = 0; i < 8; ++i) mm = fmaxf(mm, ml[i].x);
        const float m0 = mm == -INFINITY ? 0.f : mm;
        sum *= ex2_approx(m - m0);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(ex2_approx(ml[i].x - m0), ml[i].y, sum);
        m = mm;
      }
      own = make_float2(m == -INFINITY ? 0.f : m, sum == 0.f ? 0.f : 1.f / sum);
      if (p.lse) p.lse[(int64_t)h * p.total_q + row] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
    }
    __syncwarp();
    join_rows<D>(p, sg, x, q4, first, lastc, own);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn_tc(const __grid_constant__ Maps maps, const __grid_constant__ AttnParams p, int box_rows) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  Smem<D>& s = *reinterpret_cast<Smem<D>*>(smem_raw);
  if (smem_u32(smem_raw) & 1023u) {  // the swizzled tiles need it; there is no room to round up
    set_status(p.ws, MR_ERR_DEVICE_CHECK, 0xA41);
    return;
  }
  if (p.few.ask && as_tokens<kThreads>(p.kv, p.cu, p.total_q, p.window, p.sinks, p.few, s.part.sums)) return;
  empty_rows<__nv_bfloat16, D, kThreads>(p);
  Share sh;
  if (!make_share<kKeys, kThreads>(p, s.part, sh)) return;  // nothing for this CTA (all its threads leave)
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    mbar_init(&s.q_full, 1);
    mbar_init(&s.q_empty, 2);
    for (int i = 0; i < Smem<D>::kSlots; ++i) {
      mbar_init(&s.slot_full[i], 1);
      mbar_init(&s.slot_empty[i], 3);  // both tiles' MMAs, and the fix-up warp
      mbar_init(&s.slot_fixed[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      for (int h = 0; h < 2; ++h) {
        mbar_init(&s.s_full[i][h], 1);
        mbar_init(&s.p_full[i][h], 4);
      }
      mbar_init(&s.s_read[i], 4);
      mbar_init(&s.o_full[i], 1);
      mbar_init(&s.o_free[i], 4);
    }
    mbar_init(&s.part_done, kSoftmaxWarps);
    mbar_init(&s.join_go, 1);
    mbar_init(&s.mma_done, 2);
    s.abort = 0;
    for (int i = 0; i < kSlowRing; ++i) s.slow[i] = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp0) {
    tmem_alloc(&s.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp < kSoftmaxWarp0) {
    regs_dec<kRegsControl>();
    if (warp == kProducerWarp)
      producer<D>(s, p, sh, maps, box_rows);
    else if (warp == kFixWarp)
      fixer<D>(s, p, sh);
    else
      mma_issuer<D>(s, p, sh, (warp - kMmaWarp0) >> 1);
  } else {
    regs_inc<kRegsSoftmax>();
    softmax_group<D>(s, p, sh, (warp - kSoftmaxWarp0) >> 2);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp0) tmem_dealloc(s.tmem_base, 512);
}

template <int D>
cudaError_t launch(const Maps& maps, const AttnParams& p, int box_rows, int grid, cudaStream_t st) {
  // the register split assumes the launch allocation it was sized for; anything else could leave an increase waiting
  // for registers that do not exist
  cudaFuncAttributes fa;
  cudaError_t e = cudaFuncGetAttributes(&fa, k_attn_tc<D>);
  if (e != cudaSuccess) return e;
  if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
  constexpr size_t smem = sizeof(Smem<D>);
  static_assert(smem <= 227 * 1024, "shared memory of a block");
  e = cudaFuncSetAttribute(k_attn_tc<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  ProfScope ps(kKAttnTc, st);
  k_attn_tc<D><<<grid, kThreads, smem, st>>>(maps, p, box_rows);
  return cudaGetLastError();
}

}  // namespace

size_t attn_tc_part_bytes(int d) { return (size_t)2 * kMaxCtas * 256 * (d + 2) * sizeof(float); }

bool launch_attn_tc(const AttnArgs& a, AttnParams p, int sms, cudaError_t* result) {
  if (a.dt != MR_BF16 || a.kv.page_rows % 8 || !p.vec_q || !p.vec_o) return false;
  attn_split(p, 128, kMaxHeads);
  p.tokens = 2 * p.tile_tokens;
  p.unit_cost = 3;  // (about 7 us against 2.3 us for a key tile)
  p.min_steps = 4;
  p.max_parts = 24;
  int box = 8;  // rows of a page that one copy takes
  while (box < kKeys && a.kv.page_rows % (2 * box) == 0) box *= 2;
  const int d = a.kv.d;
  const uint64_t rows = (uint64_t)a.kv.n_pages * a.kv.H_kv * a.kv.page_rows;
  Maps maps;
  // a stride that is never taken may be anything
  const uint64_t q_row = a.total_q > 1 ? (uint64_t)a.q.row_stride * 2 : (uint64_t)d * 2;
  const uint64_t q_head = a.H_q > 1 ? (uint64_t)a.q.head_stride * 2 : (uint64_t)d * 2;
  if (q_row == 0 || q_head == 0) return false;
  if (!make_tmap_bf16_3d(&maps.q, a.q.ptr, d, a.total_q, a.H_q, q_row, q_head, 64, p.tile_tokens, p.hp) ||
      !make_tmap_bf16_2d(&maps.k, a.kv.k, d, rows, (uint64_t)d * 2, 64, box) ||
      !make_tmap_bf16_2d(&maps.v, a.kv.v, d, rows, (uint64_t)d * 2, 64, box))
    return false;
  // the running maximum is taken of the products before they are scaled, so the scale is kept positive (0 becomes so
  // small that no score counts; masked ones stay -infinity)
  p.negate = p.a < 0.f;
  p.a = p.a == 0.f ? 1e-30f : fabsf(p.a);
  if (((uintptr_t)a.o.ptr | (uintptr_t)(a.o.head_stride * 2) | (uintptr_t)(a.o.row_stride * 2)) % 32 == 0) p.vec_o = 2;
  debug_waits(&p.wait_ns, &p.skip_arrive);
  if (p.wait_ns == 0) p.wait_ns = kTimeoutNs;
  const int grid = sms < kMaxCtas ? sms : kMaxCtas;
  *result = d == 64 ? launch<64>(maps, p, box, grid, a.stream) : launch<128>(maps, p, box, grid, a.stream);
  return true;
}

}  // namespace mr
