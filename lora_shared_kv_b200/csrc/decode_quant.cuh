// Decode attention over a shared base K/V cache held in 8 bits, with per-agent
// low-rank value caches in bf16.
//
// For every (session s, agent i, query head h), with g = h / G and codes c and
// block scales s of the cache,
//     o = ( sum_t p_t sv c_v[t]  +  (p Umask_i) B_i,g ) / l
//     p_t = exp2(sk (q . c_k[t]) scale log2e - m)
// the same reordered form as over a bf16 cache: the rank-r product is accumulated
// per row and B_i applied once.
//
//  * What bounds it: the codes are read once from HBM, 2 d bytes a key and head, half
//    a bf16 cache's.  At that rate an SM gets a 64-key tile (16 KB at d = 128) every
//    730 cycles, and has to turn its 16 K codes into fp16: a conversion per two codes
//    at half rate, 128 cycles, and per 16 rows 128 MMAs of m16n8k16 at 2 cycles, 256
//    cycles.  (The warp-level fp8 MMA measured 6.2 cycles against 3.3 for fp16 MMA and
//    conversions together, and would round q and p to 4 bits.)  Measured (e4m3 / int8, in
//    brackets the decode over the same cache in bf16): 4 x 64k paged, 16 rows, 117.5 / 137
//    us (188; floor 85); 32 x 8k, 18 rows, 54.6 / 58.7 us (58.2; floor 21); 16 x 1k, 4
//    rows, 14.9 / 16.2 us (17.1; floor 5.3).  A tile without low-rank work takes 623 / 721
//    cycles at 8 rows on 128 CTAs (630 is the HBM rate there), 675 / 804 at 16, 993 /
//    1,156 at 18 and 1,210 / 1,493 at 32: up to 8 rows the HBM bounds, at 16 nearly so, from
//    17 on the consumers.  A launch takes about 7 us until its first tile has landed and 4 to
//    7 us from the last tile to the output, which is what separates the shorter ones
//    from their floor.
//  * A warp holds ALL rows of its row block (8, 16 or 16 + 8) and a slice of the
//    tile's keys, so that a code is converted once per tile.  The 16-row part
//    has rows as the MMA's M, the 8-row part has keys (or dims) as M; the
//    converted registers of K and V serve both as they are:
//      K (two 8-key fragments of 4 dims a lane) is B of S = Q K^T and A of S^T = K Q^T;
//      V (from ldmatrix's transposing byte form) is B of O += P V and A of O^T += V^T P^T.
//  * Key order inside 16 keys: MMA slot s is key s ^ ((s & 8) >> 1).  V's rows come
//    four consecutive per lane, slots (2t, 2t+1, 2t+8, 2t+9); with this order the
//    eight rows of every ldmatrix phase, K's and V's, lie in different 16-byte
//    banks of the swizzled tile.
//  * Softmax: running reference m per row, moved only when a tile beats it by 2^8.
//    The weights enter the value product as fp16, times the block's value scale:
//    p' = p 2^(m - w) sv, with a second reference w per row that keeps the largest
//    p' between 2^8 and 2^15 (fp16 ends at 2^16 and is full-precision down to
//    2^-14).  So p' carries 11 bits down to 2^-22 of the largest p' and 2^-33
//    absolute, whatever the scales; where the largest p' belongs to keys whose p is
//    under 2^-119 of the row's largest, it may be as low as 2^1 (the factor 2^(m - w) sv
//    ends at 2^127).  A p below 2^-126 is zero.  The low-rank product takes p as bf16.
//  * The items' tiles of the actual lengths, and what an item costs beside them, are
//    split evenly over the CTAs (each counts the sessions' tiles at its start), so
//    ragged batches are balanced; an item cut between CTAs is merged by the last one
//    to finish.
//  * Scores past seq_len and U rows before a_i are removed by selects on operands,
//    value codes past seq_len by zeroing them in shared memory.
#pragma once

#include <float.h>
#include <math.h>

#include "common.cuh"
#include "quant.h"
#include "quant_device.cuh"

namespace lrkv {

namespace {

constexpr float kNegInf = -INFINITY;

// The CTA's share of the work, found by warp 0.  Units (an item's kQItemUnits, then its
// tiles) are counted in 32 bits (checked on the host).
struct Range {
  int W, ctas;          // units of the launch; CTAs that take part
  int t_begin, t_end;   // this CTA's units
  int s, base, sl;      // session of t_begin, its first unit, its length
  int per_item;         // CTAs of every item (aligned shares), or 0
};

// First unit of CTA c when W units are split evenly: floor(c W / C), in 32 bits.
__device__ __forceinline__ int range_begin(int c, int W, int C) {
  const int q = W / C;
  return c * q + c * (W - q * C) / C;
}

// What the planner tells of a tile.
struct __align__(16) Entry {
  int key0;      // the tile's first key; kBadTile: not copied; kNoTile: the CTA's tiles end here
  int c3;        // page (paged) or session: the K/V copies' outermost coordinate
  int head;      // KV head | first agent << 16
  int session;
  float ks, vs;  // the block's scales
  int u;         // agents whose U tile is copied (16 bits) | U stage << 16 | its phase << 24; 0: none
  int pad;
};
constexpr int kBadTile = -1, kNoTile = -2;
constexpr int kPlan = 32;   // tiles of a planned chunk
constexpr int kPlans = 4;   // chunks of the table

__device__ __forceinline__ int clamp_len(const QDecodeParams& p, int sl) {
  sl = sl < 0 ? 0 : sl;
  sl = sl > p.max_seq_len ? p.max_seq_len : sl;
  return sl > p.u_rows ? p.u_rows : sl;
}
__device__ __forceinline__ int session_len(const QDecodeParams& p, int s) { return clamp_len(p, __ldg(p.seq_lens + s)); }
// An empty session keeps one (empty) tile per item, so that its rows are written.
__device__ __forceinline__ int tiles_of(int sl) { return sl > 0 ? (sl + kQBlock - 1) / kQBlock : 1; }
__device__ __forceinline__ int units_of(int sl) { return tiles_of(sl) + kQItemUnits; }

// Warp 0: count every session's units, then find this CTA's range.
__device__ __forceinline__ void find_range(const QDecodeParams& p, Range* out) {
  const int lane = threadIdx.x & 31;
  const int HR = p.Hkv * p.n_rg;
  int total = 0, nt_max = 0, sl = 0;
  bool bad = false;
  for (int s0 = 0; s0 < p.S; s0 += 32) {
    const int s = s0 + lane;
    if (s < p.S) {
      const int given = __ldg(p.seq_lens + s);
      sl = clamp_len(p, given);
      bad |= sl != given;
      total += units_of(sl);
      nt_max = max(nt_max, tiles_of(sl));
    }
  }
  if (blockIdx.x == 0 && __any_sync(0xFFFFFFFFu, bad) && lane == 0) atomicOr(p.flags, LRKV_DEVFLAG_SEQLEN);
  total = __reduce_add_sync(0xFFFFFFFFu, total);
  nt_max = __reduce_max_sync(0xFFFFFFFFu, nt_max);
  const int W = total * HR, items = p.S * HR, c = blockIdx.x;
  const int C = W < (int)gridDim.x ? W : (int)gridDim.x;
  Range r = {};
  r.W = W;
  r.per_item = q_item_ctas(items, C, nt_max, W);
  r.ctas = r.per_item ? items * r.per_item : C;
  if (c < r.ctas) {
    const int item = r.per_item ? c / r.per_item : 0;
    r.t_begin = r.per_item ? 0 : range_begin(c, W, C);
    r.t_end = r.per_item ? 0 : range_begin(c + 1, W, C);
    const int s_item = item / HR;
    // the session that holds the first unit (or the item), and its first unit
    for (int s0 = 0, base = 0; s0 < p.S; s0 += 32) {
      const int s = s0 + lane;
      if (p.S > 32) sl = s < p.S ? session_len(p, s) : 0;  // else still held from above
      const int nu = s < p.S ? units_of(sl) : 0;
      int incl = nu;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += up;
      }
      const int mine = base + (incl - nu) * HR;
      const bool here = s < p.S && (r.per_item ? s == s_item : (r.t_begin >= mine && r.t_begin < mine + nu * HR));
      const unsigned hit = __ballot_sync(0xFFFFFFFFu, here);
      if (hit) {
        const int src = __ffs(hit) - 1;
        r.s = s0 + src;
        r.base = __shfl_sync(0xFFFFFFFFu, mine, src);
        r.sl = __shfl_sync(0xFFFFFFFFu, sl, src);
        if (r.per_item) {  // this CTA's even part of its item
          const int tiles = tiles_of(r.sl), k = c - item * r.per_item;
          const int t0 = r.base + (item - s_item * HR) * units_of(r.sl) + kQItemUnits;
          const int parts = min(r.per_item, tiles);  // the last CTAs of a short item have none
          if (k < parts) {
            r.t_begin = t0 + range_begin(k, tiles, parts);
            r.t_end = t0 + range_begin(k + 1, tiles, parts);
          }
        }
        break;
      }
      base += __shfl_sync(0xFFFFFFFFu, incl, 31) * HR;
    }
  }
  if (lane == 0) *out = r;
}

// One CTA's stretch of one item.
struct Seg {
  int item, s, g, rg;
  int lo, hi;            // its tiles [lo, hi) of the item's nt
  int sl;                // session length
  int item_u0;           // the item's first unit
  int nt;
  int row_lo, rows;      // query rows [row_lo, row_lo + rows) of the N*G rows of this KV head
  int i_lo, n_ag;        // agents spanned by them
};

// Walks a CTA's range segment by segment.
struct Walk {
  int t, t_end, base, s, nu, sl;
  __device__ __forceinline__ void start(const Range& r) {
    t = r.t_begin;
    t_end = r.t_end;
    base = r.base;
    s = r.s;
    sl = r.sl;
    nu = units_of(sl);
  }
  __device__ __forceinline__ bool next(const QDecodeParams& p, Seg& sg) {
    const int HR = p.Hkv * p.n_rg;
    for (;;) {
      if (t >= t_end) return false;
      while (t >= base + nu * HR) {
        base += nu * HR;
        sl = session_len(p, ++s);
        nu = units_of(sl);
      }
      const int idx = (t - base) / nu, u0 = base + idx * nu;
      const int end = min(t_end, u0 + nu);
      sg.lo = max(t - u0 - kQItemUnits, 0);
      sg.hi = end - u0 - kQItemUnits;
      t = end;
      if (sg.hi <= sg.lo) continue;  // only units that stand for the item's own cost
      sg.s = s;
      sg.sl = sl;
      sg.nt = nu - kQItemUnits;
      sg.item = s * HR + idx;
      sg.item_u0 = u0;
      sg.g = idx / p.n_rg;
      sg.rg = idx - sg.g * p.n_rg;
      sg.row_lo = sg.rg * p.rows_per_group;
      const int row_hi = min(sg.row_lo + p.rows_per_group, p.rows_total);
      sg.rows = row_hi - sg.row_lo;
      sg.i_lo = sg.row_lo / p.G;
      sg.n_ag = (row_hi - 1) / p.G - sg.i_lo + 1;
      return true;
    }
  }
};

// Visiting order of an item's tiles.  Tiles past the agents' offsets carry the
// low-rank work, so runs of kTileRun tiles (contiguous in HBM) are visited in the
// order (j stride) mod runs with a stride near 0.618 of the run count and coprime to
// it: every contiguous stretch of the order then covers the item evenly, and so
// does every CTA's share.  A partial last run stays in place.
struct QOrder {
  int runs, stride;
  __device__ __forceinline__ void start(int nt, bool balance) {
    runs = nt / kTileRun;
    stride = 1;
    if (balance && runs > 2 && runs < 65536) {  // j * stride stays within 32 bits
      stride = (int)(0.618f * runs) | 1;
      for (;;) {
        int x = stride, y = runs;
        while (y) {
          const int z = x % y;
          x = y;
          y = z;
        }
        if (x == 1) break;
        stride += 2;
      }
      if (stride >= runs) stride = 1;
    }
  }
  __device__ __forceinline__ int tile(int k) const {  // the k-th tile visited
    const int j = k / kTileRun;
    return (stride > 1 && j < runs ? (int)((unsigned)j * (unsigned)stride % (unsigned)runs) : j) * kTileRun + k % kTileRun;
  }
};

__device__ __forceinline__ int load_offset(const QDecodeParams& p, int s, int agent, bool flag_errors) {
  if (p.offsets == nullptr) return 0;
  int a = __ldg(p.offsets + (size_t)s * p.N + agent);
  if (a < 0) {
    if (flag_errors) atomicOr(p.flags, LRKV_DEVFLAG_OFFSET);
    a = 0;
  }
  return a;
}

// ---------------------------------------------------------------------------
// producer warps
// ---------------------------------------------------------------------------
// Tile n of the CTA goes to ring stage n % stages.  Tiles that reach past an offset
// take a stage of the U ring too; tiles without one then do not hold its space.
// One warp plans: it walks the CTA's tiles, 32 at a time with one lane each, and
// writes their coordinates, scales and U stages into a table, several chunks ahead.
// One thread issues the K/V copies and one warp the U copies, reading the table: what
// stands between two copies is then short.  (One warp that walked, looked up and
// copied took 1,400 cycles a tile, three that each walked 960; a tile takes 730 at
// the HBM rate.)
// The stages of the K/V ring are a multiple of the consumer groups, so a stage always
// serves one group, which has seen every earlier phase of its barriers.  U stage g
// serves the groups that are g modulo their number; where several groups share one
// (large U tiles), useq holds the number of the stage's tile, and a group waits for
// its own tile's there before it waits on the barrier, lest an older phase of the same
// parity satisfy the wait.  A stage is released only by warps that saw its bytes land, so a
// copy is never issued into a stage whose last copy is still landing, abort or not.
struct QBars {
  uint64_t *full, *empty, *u_full, *u_empty;
  uint64_t *planned, *scaled, *used;  // chunks of the table: coordinates, scales written; every reader done
  Entry* table;
  volatile int* useq;
  volatile int* abort_flag;
};

__device__ __forceinline__ bool q_wait(const QDecodeParams& p, const QBars& bar, uint64_t* b, uint32_t phase) {
  return mbar_wait_bounded(b, phase, bar.abort_flag, p.flags, p.spin_cap, true);
}

// After an abort: wait (bounded) for the copies of the last `issued` stages to land.
__device__ __forceinline__ void q_drain(uint64_t* full, int stages, int issued, int stage, uint32_t phase) {
  for (int j = 0; j < (issued < stages ? issued : stages); ++j) {
    if (--stage < 0) {
      stage = stages - 1;
      phase ^= 1;
    }
    uint32_t spins = 0;
    while (!mbar_try_wait(&full[stage], phase) && ++spins < kSpinCap) {
    }
  }
}

// Chunk c of the table: its barriers' index and phase.
__device__ __forceinline__ int plan_slot(int n) { return n / kPlan % kPlans; }
__device__ __forceinline__ uint32_t plan_phase(int n) { return n / (kPlan * kPlans) & 1; }

template <int NG>
__device__ __forceinline__ void q_plan(const QDecodeParams& p, const QBars& bar, const Range& range) {
  const int lane = threadIdx.x & 31;
  const bool paged = p.page_table != nullptr;
  int n = 0;
  int uses = 0;  // lane u: how often U stage u was taken so far
  Walk walk;
  walk.start(range);
  Seg sg;
  // the lanes of a chunk are filled segment by segment; `open`: the chunk's slots are ours
  bool alive = true;
  auto open = [&] {  // before the first entry of a chunk
    if (n % kPlan == 0 && n >= kPlan * kPlans)
      alive = alive && !__any_sync(0xFFFFFFFFu, !q_wait(p, bar, &bar.used[plan_slot(n)], plan_phase(n) ^ 1));
    return alive;
  };
  while (walk.next(p, sg)) {
    if (sg.sl == 0) continue;  // nothing to read
    const int tiles = sg.hi - sg.lo;
    const int my_a = lane < sg.n_ag ? load_offset(p, sg.s, sg.i_lo + lane, false) : 0x7fffffff;
    const int32_t* pages = p.page_table + (size_t)sg.s * p.pt_stride;
    QOrder ord;
    ord.start(sg.nt, p.balance && range.per_item != 1);
    for (int k = 0; k < tiles;) {
      if (!open()) return;
      const int slot = n % kPlan, m = min(kPlan - slot, tiles - k);  // this pass: m tiles
      Entry* e = bar.table + plan_slot(n) * kPlan + slot + lane;
      const bool live = lane < m;
      int tile = 0, c3 = sg.s;
      bool ok = live;
      if (live) {
        tile = ord.tile(sg.lo + k + lane);
        if (paged) {
          c3 = __ldg(pages + tile);
          ok = c3 >= 0 && c3 < p.num_pages;
          if (!ok) atomicOr(p.flags, LRKV_DEVFLAG_PAGE);
        }
      }
      unsigned need = 0;
      for (int j = 0; j < sg.n_ag; ++j)
        need |= (tile + 1) * kQBlock > __shfl_sync(0xFFFFFFFFu, my_a, j) ? 1u << j : 0u;
      // the U stage of tile n + lane, and how often it was taken before
      const int us = (n + lane) % NG % p.u_stages;
      unsigned earlier = 0, same = 0;
      for (int u = 0; u < p.u_stages; ++u) {
        const unsigned takers = __ballot_sync(0xFFFFFFFFu, live && need && us == u);
        if (us == u) earlier = takers & ((1u << lane) - 1);
        if (lane == u) same = takers;
      }
      const int use = __shfl_sync(0xFFFFFFFFu, uses, us) + __popc(earlier);
      uses += __popc(same);
      if (live) {
        e->key0 = ok ? tile * kQBlock : kBadTile;
        e->c3 = c3;
        e->head = sg.g | sg.i_lo << 16;
        e->session = sg.s;
        e->u = need ? (int)need | us << 16 | (use & 1) << 24 : 0;
      }
      const bool filled = slot + m == kPlan;
      __syncwarp();
      if (filled && lane == 0) mbar_arrive(&bar.planned[plan_slot(n)]);
      if (ok) {
        const long long at = paged ? c3 * p.s_sp + sg.g * p.s_sh : sg.s * p.s_ss + sg.g * p.s_sh + tile;
        e->ks = __ldg(p.k_scale + at);
        e->vs = __ldg(p.v_scale + at);
      }
      __syncwarp();
      if (filled && lane == 0) mbar_arrive(&bar.scaled[plan_slot(n)]);
      k += m;
      n += m;
    }
  }
  if (!open()) return;
  if (lane == 0) {  // the end
    bar.table[plan_slot(n) * kPlan + n % kPlan].key0 = kNoTile;
    mbar_arrive(&bar.planned[plan_slot(n)]);
    mbar_arrive(&bar.scaled[plan_slot(n)]);
  }
}

template <int D>
__device__ __forceinline__ void q_produce_kv(const QDecodeParams& p, const CUtensorMap* tmK, const CUtensorMap* tmV,
                                             uint8_t* smem, const QDecodeSmem& lay, const QBars& bar) {
  const uint64_t policy = policy_evict_first();
  constexpr int KV_BYTES = kQBlock * D;
  const bool paged = p.page_table != nullptr;
  int stage = 0, n = 0;
  uint32_t phase = 0;
  for (;; ++n) {
    if (n % kPlan == 0) {
      if (n > 0) mbar_arrive(&bar.used[plan_slot(n - 1)]);
      if (!q_wait(p, bar, &bar.planned[plan_slot(n)], plan_phase(n))) break;
    }
    const int4 e = *reinterpret_cast<const int4*>(&bar.table[plan_slot(n) * kPlan + n % kPlan]);
    if (e.x == kNoTile) break;
    if (!q_wait(p, bar, &bar.empty[stage], phase ^ 1)) break;
    uint64_t* full = &bar.full[stage];
    if (e.x == kBadTile) {
      mbar_arrive(full);
    } else {
      uint8_t* st = smem + stage * lay.tile_bytes;
      const int c1 = paged ? 0 : e.x, g = e.z & 0xFFFF;
      mbar_arrive_expect_tx(full, 2 * KV_BYTES);
      tma_load_4d(st, tmK, full, 0, c1, g, e.y, policy);
      tma_load_4d(st + KV_BYTES, tmV, full, 0, c1, g, e.y, policy);
    }
    if (++stage == p.stages) {
      stage = 0;
      phase ^= 1;
    }
  }
  // no copy of this CTA may still be landing in shared memory when it exits
  if (*bar.abort_flag) q_drain(bar.full, p.stages, n, stage, phase);
}

template <int RK>
__device__ void q_produce_u(const QDecodeParams& p, const CUtensorMap* tmU, uint8_t* smem, const QDecodeSmem& lay,
                            const QBars& bar) {
  const int lane = threadIdx.x & 31;
  const uint64_t policy = policy_evict_last();
  constexpr int U_BYTES = kQBlock * RK * 2;
  const bool per_agent = p.mode == LRKV_BASE_SHARED;
  unsigned issued = 0, phases = 0;  // bit u: stage u was filled; the phase of its last filling
  for (int n = 0;; ++n) {
    if (n % kPlan == 0) {
      __syncwarp();
      if (n > 0 && lane == 0) mbar_arrive(&bar.used[plan_slot(n - 1)]);
      if (__any_sync(0xFFFFFFFFu, !q_wait(p, bar, &bar.planned[plan_slot(n)], plan_phase(n)))) break;
    }
    const Entry* e = &bar.table[plan_slot(n) * kPlan + n % kPlan];
    const int key0 = e->key0, u = e->u;
    if (key0 == kNoTile) break;
    if (!u) continue;
    const unsigned need = u & 0xFFFF, us = u >> 16 & 0xFF, phase = u >> 24;
    if (__any_sync(0xFFFFFFFFu, !q_wait(p, bar, &bar.u_empty[us], phase ^ 1))) break;
    issued |= 1u << us;
    phases = (phases & ~(1u << us)) | phase << us;
    uint64_t* full = &bar.u_full[us];
    if (lane == 0) {
      bar.useq[us] = n;
      if (key0 < 0) mbar_arrive(full);
      else mbar_arrive_expect_tx(full, (per_agent ? __popc(need) : 1) * U_BYTES);
    }
    __syncwarp();
    if (key0 >= 0 && (per_agent ? (need >> lane & 1) : lane == 0))  // one agent's tile per lane
      tma_load_4d(smem + lay.u_off + us * lay.u_bytes + lane * U_BYTES, tmU, full, 0, key0,
                  per_agent ? (e->head >> 16) + lane : 0, e->session, policy);
  }
  __syncwarp();
  if (*bar.abort_flag && lane < p.u_stages && (issued >> lane & 1))
    q_drain(&bar.u_full[lane], 1, 1, 0, (phases >> lane & 1) ^ 1);
}

// ---------------------------------------------------------------------------
// consumer warps
// ---------------------------------------------------------------------------
template <int D, int RK, int H16, int H8>
struct WarpRows {
  static constexpr int RPW = 16 * H16 + 8 * H8;  // rows of a row block
  static constexpr int KS = D / 16;
  static constexpr int MZ = RK >= 16 ? RK / 16 : 1;
  // 16-row part: this lane's rows are g8 and g8 + 8.  8-row part (rows 16 H16 ..):
  // rows 2 t4 and 2 t4 + 1.  Index 0, 1: the first; 2, 3: the second part's.
  static constexpr int NR = 2 * (H16 + H8);
  static constexpr int R8 = 2 * H16;             // first index of the 8-row part
  // A 24-row block keeps its query fragments in shared memory: its accumulators
  // leave no registers for them.
  static constexpr bool QS = H16 && H8;
  uint32_t q16[H16 && !QS ? KS : 1][4];
  uint32_t q8[H8 && !QS ? KS : 1][2];
  float c[NR];      // what turns a row's raw score into log2 units, without the block's key scale
  float m[NR];      // softmax reference (log2 units) of l and Z
  float w[NR];      // reference of O
  float l[NR];      // this lane's part of the row sum
  float o16[H16 ? D / 8 : 1][4];
  float o8[H8 ? D / 16 : 1][4];
  // Z^T of each eight rows: ranks 16 mz + g8 (+ 8), rows 8 x + 2 t4 (+ 1)
  static constexpr int OCT = 2 * H16 + H8;
  float z[OCT][MZ][4];
};

// Power of two that brings a row's largest |q| into [2^14, 2^15) (fp16 then holds
// every bf16 element down to 2^-28 of it exactly), and its inverse.
__device__ __forceinline__ void row_factor(float amax, float& f, float& inv) {
  int e = (int)(__float_as_uint(amax) >> 23) - 127;
  e = amax > 0.f && e < 128 ? min(14 - e, 113) : 0;  // at least 14 - 127 = -113
  f = __uint_as_float((uint32_t)(e + 127) << 23);
  inv = __uint_as_float((uint32_t)(127 - e) << 23);
}

__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

__device__ __forceinline__ const __nv_bfloat16* q_row(const QDecodeParams& p, const Seg& sg, int D, int row) {
  const int grow = sg.row_lo + row;
  return static_cast<const __nv_bfloat16*>(p.q) +
         (((size_t)sg.s * p.N + grow / p.G) * p.Hq + (size_t)sg.g * p.G + grow % p.G) * D;
}

// The row block's queries as fp16 fragments.  A lane's four dims of a 16-dim step
// are 4 t4 .. + 3 (the bytes that ldmatrix gives it of K), in the order of the codes'
// fp16 pairs.
template <int FMT, int D, int RK, int H16, int H8>
__device__ __forceinline__ void load_queries(const QDecodeParams& p, const Seg& sg, int rbase,
                                             WarpRows<D, RK, H16, H8>& st, uint32_t* qs) {
  using WR = WarpRows<D, RK, H16, H8>;
  constexpr int KS = D / 16;
  const int lane = threadIdx.x & 31, g8 = lane >> 2, t4 = lane & 3;
  constexpr int PARTS = 2 * H16 + H8;  // rows whose elements this lane holds
  uint2 raw[PARTS][KS];
  float f[PARTS], inv[PARTS];
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    const int row = rbase + 8 * i + g8;
    const bool live = row < sg.rows;
    const __nv_bfloat16* src = live ? q_row(p, sg, D, row) : nullptr;
    float amax = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      raw[i][ks] = live ? __ldg(reinterpret_cast<const uint2*>(src + 16 * ks + 4 * t4)) : make_uint2(0, 0);
    }
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
      amax = fmaxf(amax, fmaxf(fmaxf(fabsf(bf_lo(raw[i][ks].x)), fabsf(bf_hi(raw[i][ks].x))),
                               fmaxf(fabsf(bf_lo(raw[i][ks].y)), fabsf(bf_hi(raw[i][ks].y)))));
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
    row_factor(amax, f[i], inv[i]);
  }
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    uint32_t f16[4] = {}, f8[2] = {};
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
      const float d[4] = {bf_lo(raw[i][ks].x) * f[i], bf_hi(raw[i][ks].x) * f[i], bf_lo(raw[i][ks].y) * f[i],
                          bf_hi(raw[i][ks].y) * f[i]};
      const uint32_t lo = pack_f16x2(d[code_byte<FMT>(0)], d[code_byte<FMT>(1)]);
      const uint32_t hi = pack_f16x2(d[code_byte<FMT>(2)], d[code_byte<FMT>(3)]);
      if (H16 && i < 2) {
        f16[i] = lo;
        f16[i + 2] = hi;
      } else {
        f8[0] = lo;
        f8[1] = hi;
      }
    }
    if constexpr (WR::QS) {  // every warp of the block holds the same: one writes
      if (threadIdx.x < 32) {
        *reinterpret_cast<uint4*>(qs + (ks * 32 + lane) * 4) = make_uint4(f16[0], f16[1], f16[2], f16[3]);
        *reinterpret_cast<uint2*>(qs + KS * 128 + (ks * 32 + lane) * 2) = make_uint2(f8[0], f8[1]);
      }
    } else {
      if constexpr (H16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) st.q16[ks][i] = f16[i];
      }
      if constexpr (H8) {
        st.q8[ks][0] = f8[0];
        st.q8[ks][1] = f8[1];
      }
    }
  }
  if constexpr (H16) {
    st.c[0] = inv[0] * p.scale_log2;
    st.c[1] = inv[1] * p.scale_log2;
  }
  if constexpr (H8) {  // rows 2 t4, 2 t4 + 1 belong to the lanes with g8 = 2 t4, 2 t4 + 1
    const float mine = inv[PARTS - 1] * p.scale_log2;
    st.c[2 * H16] = __shfl_sync(0xFFFFFFFFu, mine, 8 * t4);
    st.c[2 * H16 + 1] = __shfl_sync(0xFFFFFFFFu, mine, 8 * t4 + 4);
  }
}

// Byte offset of 16-byte chunk c of key k in a swizzled tile (128-byte swizzle at
// d = 128, 64-byte at d = 64).
template <int D>
__device__ __forceinline__ uint32_t tile_at(int k, int c) {
  return D == 128 ? k * 128 + ((c ^ (k & 7)) << 4) : k * 64 + ((c ^ ((k >> 1) & 3)) << 4);
}
// Same for a U tile (rows of 2 RK bytes: no swizzle, 32-byte, 64-byte).
template <int RK>
__device__ __forceinline__ uint32_t u_at(int k, int c) {
  return RK == 8 ? k * 16 : RK == 16 ? k * 32 + ((c ^ ((k >> 2) & 1)) << 4) : k * 64 + ((c ^ ((k >> 1) & 3)) << 4);
}

__device__ __forceinline__ int slot_key(int s) { return s ^ ((s & 8) >> 1); }

// Scores, softmax and values of one warp's keys (kw .. of the tile) of one tile; the
// weights for the low-rank product are left in pz (of each 16 keys and eight rows, as
// a B fragment) if want_z.
// A tile that reaches past seq_len: its value codes past it are zeroed in shared memory
// first, and its scores past it selected out, so that one path serves every tile.
template <int FMT, int D, int RK, int H16, int H8>
__device__ __forceinline__ void q_tile(WarpRows<D, RK, H16, H8>& st, int sl, uint32_t Ks, float ks_scale,
                                       float vs_scale, int key0, int kw, const uint32_t* qs, bool want_z,
                                       uint32_t (*pz)[WarpRows<D, RK, H16, H8>::OCT][2]) {
  using WR = WarpRows<D, RK, H16, H8>;
  constexpr int KS = D / 16;
  constexpr int NB = kQWarpKeys / 16;  // blocks of 16 keys
  constexpr int NR = WR::NR;
  constexpr int R8 = WR::R8;
  const int lane = threadIdx.x & 31, g8 = lane >> 2, t4 = lane & 3;
  const uint32_t Vs = Ks + kQBlock * D;
  const bool last = key0 + kQBlock > sl;
  if (last) {
    for (int k = max(sl - key0, kw); k < kw + kQWarpKeys; ++k)
      if (lane < D / 16) st_shared_zero16(Vs + k * D + lane * 16);
    fence_proxy_async_smem();  // ahead of the copy that fills this stage next
    __syncwarp();
  }

  // ---- scores: S = Q K^T (16-row part), S^T = K Q^T (8-row part)
  float s16[H16 ? NB : 1][2][4], s8[H8 ? NB : 1][4];
  {
    // tiles are 1024-aligned and a row's chunk bits lie below its key bits, so
    // chunk 2 cc + c of a row is chunk c's address with bits 5 .. flipped by cc
    const int j = lane >> 3;
    const uint32_t at = Ks + tile_at<D>(kw + slot_key((j & 1) * 8 + (lane & 7)), j >> 1);
#pragma unroll
    for (int cc = 0; cc < KS / 2; ++cc) {
      uint32_t q16[H16 ? 2 : 1][4], q8[H8 ? 2 : 1][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int ks = 2 * cc + h;
        if constexpr (WR::QS) {
          const uint4 a = *reinterpret_cast<const uint4*>(qs + (ks * 32 + lane) * 4);
          const uint2 b = *reinterpret_cast<const uint2*>(qs + KS * 128 + (ks * 32 + lane) * 2);
          q16[h][0] = a.x;
          q16[h][1] = a.y;
          q16[h][2] = a.z;
          q16[h][3] = a.w;
          q8[h][0] = b.x;
          q8[h][1] = b.y;
        } else {
          if constexpr (H16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) q16[h][i] = st.q16[ks][i];
          }
          if constexpr (H8) {
            q8[h][0] = st.q8[ks][0];
            q8[h][1] = st.q8[ks][1];
          }
        }
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        uint32_t r[4];  // chunk 2cc: slots 0-7, 8-15; chunk 2cc + 1 likewise
        ldsm_x4(r[0], r[1], r[2], r[3], (at ^ (cc << 5)) + nb * 16 * D);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t a0, a2, b0, b2;
          codes_to_half2<FMT>(r[2 * h], a0, a2);
          codes_to_half2<FMT>(r[2 * h + 1], b0, b2);
          if (cc == 0 && h == 0) {
            if constexpr (H16) {
              mma_f16_16816_first(s16[nb][0], q16[h][0], q16[h][1], q16[h][2], q16[h][3], a0, a2);
              mma_f16_16816_first(s16[nb][1], q16[h][0], q16[h][1], q16[h][2], q16[h][3], b0, b2);
            }
            if constexpr (H8) mma_f16_16816_first(s8[nb], a0, b0, a2, b2, q8[h][0], q8[h][1]);
          } else {
            if constexpr (H16) {
              mma_f16_16816(s16[nb][0], q16[h][0], q16[h][1], q16[h][2], q16[h][3], a0, a2);
              mma_f16_16816(s16[nb][1], q16[h][0], q16[h][1], q16[h][2], q16[h][3], b0, b2);
            }
            if constexpr (H8) mma_f16_16816(s8[nb], a0, b0, a2, b2, q8[h][0], q8[h][1]);
          }
        }
      }
    }
  }

  // ---- softmax
  const int k_lo = key0 + kw + 2 * t4;                 // keys of slots 2 t4 (+ 1)
  const int k_hi = key0 + kw + 8 + ((2 * t4) ^ 4);     // keys of slots 2 t4 + 8 (+ 9)
  if (last) {  // keys at or past seq_len are selected out
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      if constexpr (H16) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s16[nb][0][e] = k_lo + 16 * nb + (e & 1) < sl ? s16[nb][0][e] : kNegInf;
          s16[nb][1][e] = k_hi + 16 * nb + (e & 1) < sl ? s16[nb][1][e] : kNegInf;
        }
      }
      if constexpr (H8) {
        const int ka = key0 + kw + 16 * nb + g8, kb = key0 + kw + 16 * nb + 8 + (g8 ^ 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) s8[nb][e] = (e < 2 ? ka : kb) < sl ? s8[nb][e] : kNegInf;
      }
    }
  }
  float sc[NR], mx[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    // A key scale may be zero, or take the product below fp32 (a block of zero keys is
    // written with 2^-100): the factor stays positive then, or the -inf of a masked score
    // would turn into NaN.  Raw scores end at 2^31, so they still come out under 2^-94.
    sc[i] = st.c[i] * ks_scale;
    sc[i] = sc[i] < FLT_MIN ? FLT_MIN : sc[i];
    mx[i] = kNegInf;
  }
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    if constexpr (H16) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        mx[i] = max3(max3(mx[i], s16[nb][0][2 * i], s16[nb][0][2 * i + 1]), s16[nb][1][2 * i],
                     s16[nb][1][2 * i + 1]);
    }
    if constexpr (H8) {
#pragma unroll
      for (int i = 0; i < 2; ++i) mx[R8 + i] = max3(mx[R8 + i], s8[nb][i], s8[nb][2 + i]);
    }
  }
  // The factor is > 0 and rounding monotonic: the scaled maximum is the maximum of
  // the scaled scores.  Each lane checks its own keys; the lanes of a row agree on
  // a new reference only on the few tiles that need one.
  const float lvs = __log2f(vs_scale);
  bool need = false;
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    mx[i] *= sc[i];
    const float a = st.w[i] - lvs;
    need |= mx[i] > (a < st.m[i] - 127.f ? st.m[i] - 126.f : fminf(st.m[i] + 8.f, a + 15.f));
  }
  if (__any_sync(0xFFFFFFFFu, need)) {
    float al[NR], be[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int lo = i < R8 ? 1 : 4, hi = i < R8 ? 2 : 16;  // lanes that share the row
#pragma unroll
      for (int o = lo; o <= hi; o <<= 1) mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xFFFFFFFFu, mx[i], o));
      const float mn = fmaxf(st.m[i], mx[i]);
      al[i] = mn == kNegInf ? 1.f : fast_exp2(st.m[i] - mn);
      st.m[i] = mn;
      // w: top is the tile's largest p' in log2 units; 2^(m - w) sv stays within 2^127.
      // Where m - w would pass that, the largest p' is still 2^1 or more (w <= top - 1,
      // since mx >= m - 126).  Weights below 2^-126 are zero and move nothing.
      const float top = mx[i] + lvs;
      float wn = st.w[i];
      if (mx[i] >= mn - 126.f) wn = fmaxf(top > wn + 15.f ? top - 8.f : wn, mn + lvs - 127.f);
      be[i] = wn == kNegInf ? 1.f : fast_exp2(st.w[i] - wn);
      st.w[i] = wn;
      st.l[i] *= al[i];
    }
    if constexpr (H16) {
#pragma unroll
      for (int x = 0; x < D / 8; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) st.o16[x][e] *= be[e >> 1];
#pragma unroll
      for (int x = 0; x < 2; ++x) {  // rows 2 t4, 2 t4 + 1 belong to the lanes with g8 = 2 t4, 2 t4 + 1
        const float a0 = __shfl_sync(0xFFFFFFFFu, al[x], 8 * t4), a1 = __shfl_sync(0xFFFFFFFFu, al[x], 8 * t4 + 4);
#pragma unroll
        for (int mz = 0; mz < WR::MZ; ++mz)
#pragma unroll
          for (int e = 0; e < 4; ++e) st.z[x][mz][e] *= e & 1 ? a1 : a0;
      }
    }
    if constexpr (H8) {
#pragma unroll
      for (int x = 0; x < D / 16; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) st.o8[x][e] *= be[R8 + (e & 1)];
#pragma unroll
      for (int x = 0; x < WR::MZ; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) st.z[2 * H16][x][e] *= al[R8 + (e & 1)];
    }
  }
  float mu[NR], f[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    mu[i] = st.m[i] == kNegInf ? 0.f : st.m[i];
    // 2^(m - w) sv; past 2^127 only where every weight of this row and tile is zero
    const float e = mu[i] - (st.w[i] == kNegInf ? 0.f : st.w[i]) + lvs;
    f[i] = fast_exp2(e > 127.f ? 127.f : e);
  }
  // weights: pz (bf16) for the low-rank product, pv (fp16, scaled) for the values
  uint32_t pv16[H16 ? NB : 1][4], pv8[H8 ? NB : 1][2];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    if constexpr (H16) {
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // A fragment: rows g8 + 8 i of slots 2 t4 + 8 x (+ 1)
          const float p0 = fast_exp2(fmaf(s16[nb][x][2 * i], sc[i], -mu[i]));
          const float p1 = fast_exp2(fmaf(s16[nb][x][2 * i + 1], sc[i], -mu[i]));
          st.l[i] += p0 + p1;
          if (want_z) pz[nb][i][x] = pack_bf16x2(p0, p1);  // of rows 8 i ..: the same layout
          pv16[nb][2 * x + i] = pack_f16x2(p0 * f[i], p1 * f[i]);
        }
    }
    if constexpr (H8) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {  // S^T: slots g8 + 8 x, rows 2 t4, + 1; transposed into a B fragment
        const float p0 = fast_exp2(fmaf(s8[nb][2 * x], sc[R8], -mu[R8]));
        const float p1 = fast_exp2(fmaf(s8[nb][2 * x + 1], sc[R8 + 1], -mu[R8 + 1]));
        st.l[R8] += p0;
        st.l[R8 + 1] += p1;
        if (want_z) pz[nb][2 * H16][x] = movmatrix_t(pack_bf16x2(p0, p1));
        pv8[nb][x] = movmatrix_t(pack_f16x2(p0 * f[R8], p1 * f[R8 + 1]));
      }
    }
  }

  // ---- values: O += P V, O^T += V^T P^T
  {
    // row 4 t + e of a 16 x 16 block becomes byte e of lane t: slots 2 t, 2 t + 1 (the
    // fp16 pair lo) and 2 t + 8, 2 t + 9 (hi)
    const int e = lane & 15;
    int i = 0;  // which element of the pairs byte e & 3 is
#pragma unroll
    for (int x = 0; x < 4; ++x) i = code_byte<FMT>(x) == (e & 3) ? x : i;
    const uint32_t at = Vs + tile_at<D>(kw + slot_key(2 * (e >> 2) + (i & 1) + 8 * (i >> 1)), lane >> 4);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int cc = 0; cc < KS / 2; ++cc) {
        uint32_t r[4];  // dims 32 cc + 8 x + g8
        ldsm_b8_x2_t(r[0], r[1], r[2], r[3], (at ^ (cc << 5)) + nb * 16 * D);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t a0, a1, b0, b1;
          codes_to_half2<FMT>(r[2 * h], a0, a1);
          codes_to_half2<FMT>(r[2 * h + 1], b0, b1);
          if constexpr (H16) {
            float* o = st.o16[4 * cc + 2 * h];
            mma_f16_16816(o, pv16[nb][0], pv16[nb][1], pv16[nb][2], pv16[nb][3], a0, a1);
            mma_f16_16816(o + 4, pv16[nb][0], pv16[nb][1], pv16[nb][2], pv16[nb][3], b0, b1);
          }
          if constexpr (H8) mma_f16_16816(st.o8[2 * cc + h], a0, b0, a1, b1, pv8[nb][0], pv8[nb][1]);
        }
      }
    }
  }

}

// Low-rank values of the same keys: Z^T += U_i^T P^T over each agent's own rows, eight
// rows at a time.  `agents` has a bit for every agent of this warp's rows whose U tile
// counts here; U rows before a_i or at or past seq_len are selected out (`clean`: there
// are none).  w_lo: the warp's first row, counted from the first agent's first.
template <int D, int RK, int H16, int H8>
__device__ __forceinline__ void q_low_rank(WarpRows<D, RK, H16, H8>& st,
                                           const uint32_t (*pz)[WarpRows<D, RK, H16, H8>::OCT][2], uint32_t Us,
                                           int slot_bytes, unsigned agents, bool one_pass, const int* my_ag, int G,
                                           int w_lo, bool clean, const int* a_sm, int key0, int kw, int sl) {
  using WR = WarpRows<D, RK, H16, H8>;
  constexpr int NB = kQWarpKeys / 16;
  const int lane = threadIdx.x & 31, t4 = lane & 3, j = lane >> 3;
  const uint32_t at = Us + u_at<RK>(kw + slot_key((j & 1) * 8 + (lane & 7)), RK == 8 ? 0 : j >> 1);
  while (agents) {
    const int ag = __ffs(agents) - 1;
    agents &= agents - 1;
    const uint32_t ub = at + ag * slot_bytes;
    uint32_t u[NB][WR::MZ][4];  // ranks 16 mz + g8: slots 0-7, 8-15; ranks + 8 likewise
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int mz = 0; mz < WR::MZ; ++mz) {
        uint32_t* r = u[nb][mz];
        r[2] = r[3] = 0;
        if constexpr (RK == 8) ldsm_x2_t(r[0], r[1], ub + nb * 256);
        else ldsm_x4_t(r[0], r[1], r[2], r[3], (ub ^ (mz << 5)) + nb * 32 * RK);
      }
    if (!clean) {
      const int a_i = one_pass ? 0 : a_sm[ag];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int x = key0 + kw + 16 * nb + 2 * t4, y = key0 + kw + 16 * nb + 8 + ((2 * t4) ^ 4);
        const uint32_t lo = (x >= a_i && x < sl ? 0xFFFFu : 0u) | (x + 1 >= a_i && x + 1 < sl ? 0xFFFF0000u : 0u);
        const uint32_t hi = (y >= a_i && y < sl ? 0xFFFFu : 0u) | (y + 1 >= a_i && y + 1 < sl ? 0xFFFF0000u : 0u);
#pragma unroll
        for (int mz = 0; mz < WR::MZ; ++mz) {
          u[nb][mz][0] &= lo;
          u[nb][mz][1] &= hi;
          u[nb][mz][2] &= lo;
          u[nb][mz][3] &= hi;
        }
      }
    }
    const int r_lo = one_pass ? 0 : ag * G - w_lo, r_hi = one_pass ? WR::RPW : r_lo + G;  // the agent's rows
#pragma unroll
    for (int x = 0; x < WR::OCT; ++x) {
      if (r_lo >= 8 * x + 8 || r_hi <= 8 * x) continue;  // warp-uniform
      const bool use = one_pass || my_ag[x] == ag;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const uint32_t b0 = use ? pz[nb][x][0] : 0u, b1 = use ? pz[nb][x][1] : 0u;
#pragma unroll
        for (int mz = 0; mz < WR::MZ; ++mz)
          mma_bf16_16816(st.z[x][mz], u[nb][mz][0], u[nb][mz][2], u[nb][mz][1], u[nb][mz][3], b0, b1);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// the end of a segment
// ---------------------------------------------------------------------------
constexpr int kQThreads = kQWarps * 32;  // consumer threads
__device__ __forceinline__ void q_sync() { named_bar_sync(1, kQThreads); }

// Two records per CTA: 0 for the segment that starts the CTA's range, 1 for a later
// one (only its last can be shared with the next CTA).
__device__ __forceinline__ size_t q_record_slot(int cta, int cta_begin, int item_u0) {
  return 2 * (size_t)cta + (item_u0 > cta_begin ? 1 : 0);
}

// Merge the warps' rows into the CTA's record rec = [m | l | O | Z] in shared
// memory.  The warps of a row block held the same rows over different keys, in the
// same fragment layout: they exchange whole fragments (a float4 a lane, no index
// arithmetic while the accumulators are live), a few at a time, and whoever sums one
// writes it to its place.  Sums run in warp order, so the result does not depend on
// timing.
template <int D, int RK, int H16, int H8, int NRB>
__device__ __forceinline__ void merge_warps(WarpRows<D, RK, H16, H8>& st, float* rec, float4* mb, float* ml, int rb,
                                            int peer) {
  using WR = WarpRows<D, RK, H16, H8>;
  constexpr int RPW = WR::RPW, RP = RPW * NRB, NR = WR::NR, R8 = WR::R8, MZ = WR::MZ;
  constexpr int PEERS = kQWarps / NRB;
  constexpr int N16 = H16 ? D / 8 : 0, N8 = H8 ? D / 16 : 0, NF = N16 + N8 + WR::OCT * MZ;  // fragments
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g8 = lane >> 2, t4 = lane & 3;
  int row[NR];  // this lane's rows within the block
#pragma unroll
  for (int i = 0; i < NR; ++i) row[i] = i < R8 ? 8 * i + g8 : 16 * H16 + 2 * t4 + (i - R8);
  float* my_ml = ml + warp * 2 * RPW;
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int lo = i < R8 ? 1 : 4, hi = i < R8 ? 2 : 16;
#pragma unroll
    for (int o = lo; o <= hi; o <<= 1) st.l[i] += __shfl_xor_sync(0xFFFFFFFFu, st.l[i], o);
    if ((i < R8 ? t4 : g8) == 0) {
      my_ml[row[i]] = st.m[i];
      my_ml[RPW + row[i]] = st.l[i];
    }
  }
  q_sync();
  // warp x of row block b is warp x * NRB + b
  float fo[NR], fz[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    float M = kNegInf;
#pragma unroll
    for (int x = 0; x < PEERS; ++x) M = fmaxf(M, ml[(x * NRB + rb) * 2 * RPW + row[i]]);
    fz[i] = st.m[i] == kNegInf ? 0.f : fast_exp2(st.m[i] - M);
    // O stands for weights 2^(w - m) times larger; in two factors, since w - m can pass 127
    fo[i] = st.m[i] == kNegInf || st.w[i] == kNegInf ? 0.f : fast_exp2(0.5f * (st.w[i] - M));
  }
  if (tid < RP) {
    const int b = tid / RPW, r = tid % RPW;
    float M = kNegInf, L = 0.f;
#pragma unroll
    for (int x = 0; x < PEERS; ++x) M = fmaxf(M, ml[(x * NRB + b) * 2 * RPW + r]);
#pragma unroll
    for (int x = 0; x < PEERS; ++x) {
      const float mm = ml[(x * NRB + b) * 2 * RPW + r];
      L += mm == kNegInf ? 0.f : ml[(x * NRB + b) * 2 * RPW + RPW + r] * fast_exp2(mm - M);
    }
    rec[tid] = M;
    rec[RP + tid] = L;
  }
  float zf[WR::OCT][2];  // fz of rows 2 t4, 2 t4 + 1 of each eight
#pragma unroll
  for (int x = 0; x < WR::OCT; ++x)
#pragma unroll
    for (int e = 0; e < 2; ++e)
      zf[x][e] = x < 2 * H16 ? __shfl_sync(0xFFFFFFFFu, fz[x], 8 * t4 + 4 * e) : fz[NR - 2 + e];
#pragma unroll
  for (int f0 = 0; f0 < NF; f0 += kQMergeFrags) {
#pragma unroll
    for (int f = f0; f < f0 + kQMergeFrags && f < NF; ++f) {
      float4 v;
      if (f < N16) {
        const float* o = st.o16[H16 ? f : 0];
        v = make_float4(o[0] * fo[0] * fo[0], o[1] * fo[0] * fo[0], o[2] * fo[1] * fo[1], o[3] * fo[1] * fo[1]);
      } else if (f < N16 + N8) {
        const float* o = st.o8[H8 ? f - N16 : 0];
        const float a = fo[NR - 2], b = fo[NR - 1];
        v = make_float4(o[0] * a * a, o[1] * b * b, o[2] * a * a, o[3] * b * b);
      } else {
        const int x = (f - N16 - N8) / MZ;
        const float* z = st.z[x][(f - N16 - N8) % MZ];
        v = make_float4(z[0] * zf[x][0], z[1] * zf[x][1], z[2] * zf[x][0], z[3] * zf[x][1]);
      }
      mb[(warp * kQMergeFrags + f - f0) * 32 + lane] = v;
    }
    q_sync();
    // a thread sums half a fragment's float4 of one row block over its warps
    for (int e = tid; e < NRB * kQMergeFrags * 64; e += kQThreads) {
      const int h = e & 1, ln = e >> 1 & 31, f = f0 + (e >> 6) % kQMergeFrags, b = (e >> 6) / kQMergeFrags;
      if (f >= NF) continue;
      const float2* src = reinterpret_cast<const float2*>(mb + (b * kQMergeFrags + f - f0) * 32 + ln) + h;
      float2 a = make_float2(0.f, 0.f);
#pragma unroll
      for (int x = 0; x < PEERS; ++x) {
        const float2 v = src[x * NRB * kQMergeFrags * 64];
        a.x += v.x;
        a.y += v.y;
      }
      const int g = ln >> 2, t = ln & 3;
      if (f < N16) {  // rows g (+ 8), columns 8 f + 2 t, + 1
        *reinterpret_cast<float2*>(rec + 2 * RP + (b * RPW + g + 8 * h) * D + 8 * f + 2 * t) = a;
      } else {        // rows 2 t, 2 t + 1 of an octet, one column
        const bool z = f >= N16 + N8;
        const int x = z ? f - N16 - N8 : f - N16;
        const int r = b * RPW + (z ? 8 * (x / MZ) : 16 * H16) + 2 * t, col = 16 * (z ? x % MZ : x) + 8 * h + g;
        float* dst = rec + 2 * RP + (z ? RP * D + r * RK : r * D) + col;
        if (!z || col < RK) {
          dst[0] = a.x;
          dst[z ? RK : D] = a.y;
        }
      }
    }
    q_sync();
  }
}

// Publish the record, or, as the last of the item's CTAs to get here (ticket), combine
// every record of the item; then out = (O + Z B_i,g) / l.  `table` holds kQMaxCtas x RP
// floats.
template <int D, int RK, int RP>
__device__ __forceinline__ void finish_item(const QDecodeParams& p, const Range& range, const Seg& sg, float* rec,
                                            float* table, int* bcast) {
  constexpr int THREADS = kQThreads;
  const int tid = threadIdx.x;
  constexpr int REC = RP * (D + RK + 2);
  constexpr int E4 = RP * (D + RK) / 4;
  constexpr int PER = (E4 + THREADS - 1) / THREADS;  // float4 elements of a thread
  constexpr int BATCH = 4;                            // records whose loads are in flight together
  const bool shared = sg.lo > 0 || sg.hi < sg.nt;
  // the B columns of the (agent, dim pair) units that this thread will write
  constexpr int D2 = D / 2;
  const int HD = p.Hkv * D, units = sg.n_ag * D2;
  auto b_at = [&](int u) {
    return reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p.b) +
                                             (size_t)(sg.i_lo + u / D2) * RK * HD + (size_t)sg.g * D + 2 * (u % D2));
  };
  if (tid < units) {  // into L1, while the record is published and merged
#pragma unroll
    for (int r = 0; r < RK; ++r) asm volatile("prefetch.global.L1 [%0];" ::"l"(b_at(tid) + (size_t)r * (HD / 2)));
  }
  if (shared) {
    // the CTAs that hold a part of the item
    const int C = range.ctas, W = range.W;
    int c_first, segs;
    if (range.per_item) {
      c_first = sg.item * range.per_item;
      segs = min(range.per_item, sg.nt);
    } else {
      c_first = (int)owner_cta(sg.item_u0 + kQItemUnits, W, C);
      segs = (int)owner_cta(sg.item_u0 + kQItemUnits + sg.nt - 1, W, C) - c_first + 1;
    }
    float* mine = p.partials + q_record_slot(blockIdx.x, range.t_begin, sg.item_u0) * REC;
    for (int e = 4 * tid; e < REC; e += 4 * THREADS)
      __stcg(reinterpret_cast<float4*>(mine + e), *reinterpret_cast<const float4*>(rec + e));
    q_sync();
    if (tid == 0) {
      __threadfence();
      unsigned* word = p.tickets + (c_first >> 2);  // c_first's byte of it
      const int at = 8 * (c_first & 3);
      const int last = (int)(atomicAdd(word, 1u << at) >> at & 0xFF) == segs - 1;
      if (last) atomicSub(word, (unsigned)segs << at);
      *bcast = last;
    }
    q_sync();
    if (!*bcast) return;
    __threadfence();
    // Only the item's first CTA can hold it in its second record slot.
    const float* first =
        p.partials + q_record_slot(c_first, range.per_item ? sg.item_u0 : range_begin(c_first, W, C), sg.item_u0) * REC;
    const float* rest = p.partials + 2 * (size_t)c_first * REC;
    auto record = [&](int j) { return j == 0 ? first : rest + (size_t)(2 * j) * REC; };
    for (int e = tid; e < segs * RP; e += THREADS) table[e] = __ldcg(record(e / RP) + e % RP);  // the records' m
    q_sync();
    if (tid < RP) {  // RP <= 32 <= THREADS
      float M = kNegInf, L = 0.f;
#pragma unroll 4
      for (int j = 0; j < segs; ++j) M = fmaxf(M, table[j * RP + tid]);
#pragma unroll 4
      for (int j = 0; j < segs; ++j) {
        const float mj = table[j * RP + tid], lj = __ldcg(record(j) + RP + tid);
        const float sc = mj == kNegInf ? 0.f : fast_exp2(mj - M);
        table[j * RP + tid] = sc;
        L += sc == 0.f ? 0.f : lj * sc;
      }
      rec[RP + tid] = L;
    }
    q_sync();
    {  // O and Z
      float4 acc[PER];
#pragma unroll
      for (int u = 0; u < PER; ++u) acc[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int jb = 0; jb < segs; jb += BATCH) {
        float4 v[BATCH][PER];
#pragma unroll
        for (int q = 0; q < BATCH; ++q) {
          const float4* src = reinterpret_cast<const float4*>(record(min(jb + q, segs - 1)) + 2 * RP);
#pragma unroll
          for (int u = 0; u < PER; ++u)
            if (tid + u * THREADS < E4) v[q][u] = __ldcg(src + tid + u * THREADS);
        }
#pragma unroll
        for (int q = 0; q < BATCH; ++q) {
          if (jb + q >= segs) break;
#pragma unroll
          for (int u = 0; u < PER; ++u) {
            const int e = 4 * (tid + u * THREADS);
            if (e >= 4 * E4) continue;
            const float sc = table[(jb + q) * RP + (e < RP * D ? e / D : (e - RP * D) / RK)];
            acc[u].x += v[q][u].x * sc;
            acc[u].y += v[q][u].y * sc;
            acc[u].z += v[q][u].z * sc;
            acc[u].w += v[q][u].w * sc;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < PER; ++u) {
        const int e4 = tid + u * THREADS;
        if (e4 < E4) *reinterpret_cast<float4*>(rec + 2 * RP + 4 * e4) = acc[u];
      }
    }
    q_sync();
  }
  // A thread takes (agent, two adjacent dims): the agent's B columns serve all its rows.
  const float* mL = rec + RP;
  const float* mO = rec + 2 * RP;
  const float* mZ = mO + RP * D;
  for (int u = tid; u < units; u += THREADS) {
    const int agent = sg.i_lo + u / D2, dim = 2 * (u % D2);
    const uint32_t* bp = b_at(u);
    uint32_t b[RK];
#pragma unroll
    for (int r = 0; r < RK; ++r) b[r] = __ldg(bp + (size_t)r * (HD / 2));
    const int r_end = min((agent + 1) * p.G - sg.row_lo, sg.rows);
    for (int row = max(agent * p.G - sg.row_lo, 0); row < r_end; ++row) {
      float2 o = *reinterpret_cast<const float2*>(mO + row * D + dim);
#pragma unroll
      for (int r = 0; r < RK; r += 4) {
        const float4 z = *reinterpret_cast<const float4*>(mZ + row * RK + r);
        o.x = fmaf(z.x, bf_lo(b[r]), o.x);
        o.y = fmaf(z.x, bf_hi(b[r]), o.y);
        o.x = fmaf(z.y, bf_lo(b[r + 1]), o.x);
        o.y = fmaf(z.y, bf_hi(b[r + 1]), o.y);
        o.x = fmaf(z.z, bf_lo(b[r + 2]), o.x);
        o.y = fmaf(z.z, bf_hi(b[r + 2]), o.y);
        o.x = fmaf(z.w, bf_lo(b[r + 3]), o.x);
        o.y = fmaf(z.w, bf_hi(b[r + 3]), o.y);
      }
      const float L = mL[row], il = L == 0.f ? 0.f : 1.f / L;
      o.x *= il;
      o.y *= il;
      const int grow = sg.row_lo + row;
      const size_t at = (((size_t)sg.s * p.N + agent) * p.Hq + (size_t)sg.g * p.G + grow % p.G) * D + dim;
      if (p.out_f32) *reinterpret_cast<float2*>(static_cast<float*>(p.out) + at) = o;
      else *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + at) = pack_bf16x2(o.x, o.y);
    }
  }
}

// Wait until a U stage that groups share holds tile number n's.
__device__ __forceinline__ bool q_wait_turn(const QDecodeParams& p, const QBars& bar, int us, int n) {
  uint32_t spins = 0;
  while (bar.useq[us] != n) {
    if (*bar.abort_flag) return false;
    if (++spins >= p.spin_cap) {
      *bar.abort_flag = 1;
      atomicOr(p.flags, LRKV_DEVFLAG_TIMEOUT);
      return false;
    }
  }
  return true;
}

template <int FMT, int D, int RK, int H16, int H8, int NRB>
__device__ void q_consumers(const QDecodeParams& p, uint8_t* smem, const QDecodeSmem& lay, const QBars& bar, int* bcast,
                            const Range& range) {
  using WR = WarpRows<D, RK, H16, H8>;
  constexpr int RPW = WR::RPW, RP = RPW * NRB, NR = WR::NR;
  constexpr int KW = kQBlock / kQWarpKeys;     // warps that share a tile's keys
  constexpr int NG = kQWarps / (KW * NRB);     // groups that take tiles in turn
  constexpr int NB = kQWarpKeys / 16;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g8 = lane >> 2;
  const int rb = warp % NRB, peer = warp / NRB;  // row block; place among the warps that hold its rows
  const int og = peer / KW, kw = (peer % KW) * kQWarpKeys;
  float* rec = reinterpret_cast<float*>(smem + lay.rec_off);
  float4* mb = reinterpret_cast<float4*>(smem + lay.mb_off);
  float* ml = reinterpret_cast<float*>(smem + lay.ml_off);
  uint32_t* qs = reinterpret_cast<uint32_t*>(smem + lay.q_off);
  int* a_sm = reinterpret_cast<int*>(smem + lay.a_off);
  const uint32_t ring = smem_u32(smem);
  // the group's next tile (number, stage, phase); the CTA's tiles before this segment
  int n = og, stage = og, before = 0;
  uint32_t phase = 0;
  bool alive = true;  // until a wait gives up: then nothing is read or released any more
  Walk walk;
  walk.start(range);
  Seg sg;
  WR st;
  while (walk.next(p, sg)) {
    if (tid < sg.n_ag) a_sm[tid] = load_offset(p, sg.s, sg.i_lo + tid, true);
    load_queries<FMT, D, RK, H16, H8>(p, sg, rb * RPW, st, qs);
    q_sync();
    // this lane's agent's offset (lane j: agent j), and the item's largest
    const int lane_a = lane < sg.n_ag ? a_sm[lane] : 0x7fffffff;
    const int a_max = __reduce_max_sync(0xFFFFFFFFu, lane < sg.n_ag ? lane_a : 0);
    // agents of this warp's rows, and of the rows whose weights this lane masks
    const int w_lo = sg.row_lo + rb * RPW, w_rows = min(RPW, sg.rows - rb * RPW);
    const int ag_lo = w_rows > 0 ? w_lo / p.G - sg.i_lo : 0;
    const int ag_hi = w_rows > 0 ? (w_lo + w_rows - 1) / p.G - sg.i_lo : -1;
    int my_ag[2 * H16 + H8];
#pragma unroll
    for (int i = 0; i < 2 * H16 + H8; ++i) my_ag[i] = 8 * i + g8 < w_rows ? (w_lo + 8 * i + g8) / p.G - sg.i_lo : -1;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      st.m[i] = st.w[i] = kNegInf;
      st.l[i] = 0.f;
    }
    if constexpr (H16) {
#pragma unroll
      for (int x = 0; x < D / 8; ++x) st.o16[x][0] = st.o16[x][1] = st.o16[x][2] = st.o16[x][3] = 0.f;
    }
    if constexpr (H8) {
#pragma unroll
      for (int x = 0; x < D / 16; ++x) st.o8[x][0] = st.o8[x][1] = st.o8[x][2] = st.o8[x][3] = 0.f;
    }
#pragma unroll
    for (int x = 0; x < WR::OCT; ++x)
#pragma unroll
      for (int mz = 0; mz < WR::MZ; ++mz) st.z[x][mz][0] = st.z[x][mz][1] = st.z[x][mz][2] = st.z[x][mz][3] = 0.f;

    before += sg.sl > 0 ? sg.hi - sg.lo : 0;  // an empty session has no tiles
    while (alive && n < before) {
      // the group's tiles of a chunk of the table are n % kPlan = og, og + NG, ..
      const int slot = plan_slot(n);
      if (n % kPlan < NG && __any_sync(0xFFFFFFFFu, !q_wait(p, bar, &bar.scaled[slot], plan_phase(n)))) {
        alive = false;
        break;
      }
      const Entry* e = &bar.table[slot * kPlan + n % kPlan];
      const int key0 = e->key0, u = e->u;
      const float ks = e->ks, vs = e->vs;
      if (__any_sync(0xFFFFFFFFu, !q_wait(p, bar, &bar.full[stage], phase))) {
        alive = false;
        break;
      }
      uint32_t pz[NB][WR::OCT][2];
      const uint32_t Ks = ring + stage * lay.tile_bytes;
      if (key0 >= 0) q_tile<FMT, D, RK, H16, H8>(st, sg.sl, Ks, ks, vs, key0, kw, qs, u != 0, pz);
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bar.empty[stage]);
        if (n % kPlan >= kPlan - NG) mbar_arrive(&bar.used[slot]);  // its last tile of the chunk
      }
      if (u) {
        const int us = u >> 16 & 0xFF;
        bool there = p.u_stages >= NG || q_wait_turn(p, bar, us, n);
        there = there && q_wait(p, bar, &bar.u_full[us], u >> 24);
        if (__any_sync(0xFFFFFFFFu, !there)) {
          alive = false;
          break;
        }
        if (key0 >= 0) {
          const bool last = key0 + kQBlock > sg.sl;
          const bool one_pass = p.mode == LRKV_BASE_LR_SHARED && !last && a_max <= key0;
          const unsigned mine = __ballot_sync(0xFFFFFFFFu, lane >= ag_lo && lane <= ag_hi && key0 + kQBlock > lane_a);
          const bool clean = !last && !__any_sync(0xFFFFFFFFu, (mine >> lane & 1) && lane_a > key0);
          q_low_rank<D, RK, H16, H8>(st, pz, ring + lay.u_off + us * lay.u_bytes,
                                     p.mode == LRKV_BASE_SHARED ? kQBlock * RK * 2 : 0,
                                     one_pass ? mine & (0u - mine) : mine, one_pass, my_ag, p.G,
                                     w_lo - sg.i_lo * p.G, clean, a_sm, key0, kw, sg.sl);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.u_empty[us]);
      }
      n += NG;
      stage += NG;
      if (stage >= p.stages) {
        stage = og;
        phase ^= 1;
      }
    }
    merge_warps<D, RK, H16, H8, NRB>(st, rec, mb, ml, rb, peer);
    finish_item<D, RK, RP>(p, range, sg, rec, reinterpret_cast<float*>(mb), bcast);
    q_sync();  // the record, the merge buffer and the offsets are free again
  }
}

// Three warpgroups: two of consumers, one of producers.  A thread is
// launched with 168 registers (65536 / 384); the producers' share goes to the
// consumers: 2 x 128 x 224 + 128 x 56 = 384 x 168.
constexpr int kQBlockThreads = (kQWarps + 4) * 32;
constexpr int kQConsumerRegs = 224, kQProducerRegs = 56;
static_assert(kQThreads * kQConsumerRegs + 128 * kQProducerRegs <= kQBlockThreads * 168, "register split");

template <int FMT, int D, int RK, int H16, int H8, int NRB>
__global__ void __launch_bounds__(kQBlockThreads, 1)
    decode_quant_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                        const __grid_constant__ CUtensorMap tmU, const QDecodeParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const QDecodeSmem lay = q_smem_plan(D, RK, 16 * H16 + 8 * H8, NRB, p.n_u_slots, p.stages, p.u_stages);
  QBars bar;
  bar.full = reinterpret_cast<uint64_t*>(smem + lay.bar_off);
  bar.empty = bar.full + p.stages;
  bar.u_full = bar.empty + p.stages;
  bar.u_empty = bar.u_full + p.u_stages;
  bar.planned = bar.u_empty + p.u_stages;
  bar.scaled = bar.planned + kPlans;
  bar.used = bar.scaled + kPlans;
  bar.table = reinterpret_cast<Entry*>(smem + lay.plan_off);
  bar.useq = reinterpret_cast<volatile int*>(smem + lay.useq_off);
  Range* range = reinterpret_cast<Range*>(smem + lay.misc_off);
  bar.abort_flag = reinterpret_cast<volatile int*>(range + 1);
  int* bcast = const_cast<int*>(bar.abort_flag) + 1;
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == kQWarps * 32) {
    constexpr int READERS = kQBlock / kQWarpKeys * NRB;  // warps that read a tile
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&bar.full[s], 1);
      mbar_init(&bar.empty[s], READERS);
    }
    for (int s = 0; s < p.u_stages; ++s) {
      mbar_init(&bar.u_full[s], 1);
      mbar_init(&bar.u_empty[s], READERS);
      bar.useq[s] = -1;
    }
    for (int s = 0; s < kPlans; ++s) {
      mbar_init(&bar.planned[s], 1);
      mbar_init(&bar.scaled[s], 1);
      mbar_init(&bar.used[s], kQWarps + 2);              // the consumers and the two copying warps
    }
    *bar.abort_flag = 0;
    *bcast = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmU);
  }
  pdl_wait();
  pdl_launch_dependents();
  if (warp == 0) find_range(p, range);
  __syncthreads();
  const Range r = *range;
  if (warp >= kQWarps) {
    setmaxnreg_dec<kQProducerRegs>();
    // the test hook (p.stall): nothing is copied, so the consumers' waits run out
    if (warp == kQWarps + 2) {
      q_plan<kQWarps / (kQBlock / kQWarpKeys) / NRB>(p, bar, r);
    } else if (warp == kQWarps && !p.stall) {
      if ((threadIdx.x & 31) == 0) q_produce_kv<D>(p, &tmK, &tmV, smem, lay, bar);
    } else if (warp == kQWarps + 1 && !p.stall) {
      q_produce_u<RK>(p, &tmU, smem, lay, bar);
    }
  } else {
    setmaxnreg_inc<kQConsumerRegs>();
    q_consumers<FMT, D, RK, H16, H8, NRB>(p, smem, lay, bar, bcast, r);
  }
}

template <int FMT, int D, int RK, int H16, int H8, int NRB>
lrkv_status launch_q(const QDecodeParams& p, const void* tmK, const void* tmV, const void* tmU, int smem, int ctas,
                     cudaStream_t stream) {
  auto kern = decode_quant_kernel<FMT, D, RK, H16, H8, NRB>;
  if (ensure_dynamic_smem<decode_quant_kernel<FMT, D, RK, H16, H8, NRB>>(smem) != cudaSuccess) return LRKV_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kQBlockThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const CUtensorMap& k = *static_cast<const CUtensorMap*>(tmK);
  const CUtensorMap& v = *static_cast<const CUtensorMap*>(tmV);
  const CUtensorMap& u = *static_cast<const CUtensorMap*>(tmU);
  return cudaLaunchKernelEx(&cfg, kern, k, v, u, p) == cudaSuccess ? LRKV_OK : LRKV_ERR_CUDA;
}

template <int FMT, int D, int RK>
lrkv_status dispatch_rows(const QDecodeParams& p, int rows, const void* tmK, const void* tmV, const void* tmU,
                          int smem, int ctas, cudaStream_t st) {
  if (rows <= 8) return launch_q<FMT, D, RK, 0, 1, 1>(p, tmK, tmV, tmU, smem, ctas, st);
  if (rows <= 16) return launch_q<FMT, D, RK, 1, 0, 1>(p, tmK, tmV, tmU, smem, ctas, st);
  if (rows <= 24) return launch_q<FMT, D, RK, 1, 1, 1>(p, tmK, tmV, tmU, smem, ctas, st);
  return launch_q<FMT, D, RK, 1, 0, 2>(p, tmK, tmV, tmU, smem, ctas, st);
}

}  // namespace

template <int FMT, int D>
lrkv_status launch_decode_quant_fd(const QDecodeParams& p, int RK, int rows, const void* tmK, const void* tmV,
                                   const void* tmU, int smem, int ctas, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (RK == 8) return dispatch_rows<FMT, D, 8>(p, rows, tmK, tmV, tmU, smem, ctas, st);
  if (RK == 16) return dispatch_rows<FMT, D, 16>(p, rows, tmK, tmV, tmU, smem, ctas, st);
  return dispatch_rows<FMT, D, 32>(p, rows, tmK, tmV, tmU, smem, ctas, st);
}

}  // namespace lrkv
