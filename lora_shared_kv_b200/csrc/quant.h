// Internal definitions of the operators on an 8-bit K/V cache.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "lrkv_internal.h"

namespace lrkv {

constexpr int kQBlock = LRKV_QUANT_BLOCK;  // tokens that share a scale, keys of a decode tile, tokens of a page
static_assert(kQBlock == kKeysPerTile, "a decode tile is one block of the cache");

// ---------------------------------------------------------------------------
// writing and reading back
// ---------------------------------------------------------------------------
struct QCacheParams {
  // the bf16 side (source of a write, destination of a read)
  uint16_t* x[2];            // K, V
  long long x_ss, x_sh, x_st, x_sp;
  const int32_t* x_table;    // null => dense
  long long x_pt;
  int x_pages;
  // the 8-bit side
  uint8_t* c[2];
  float* scale[2];
  long long c_ss, c_sh, c_st, c_sp;
  long long s_ss, s_sh, s_sp;
  const int32_t* c_table;
  long long c_pt;
  int c_pages;
  int rows;                  // row capacity of a session
  const int32_t* first;      // [S] or null
  const int32_t* count;      // [S] or null
  int S, Hkv, T;
  int nblk;                  // blocks that a session's rows can touch
  unsigned* flags;
};

lrkv_status launch_quantize(const QCacheParams& p, int D, int fmt, void* stream);
lrkv_status launch_dequantize(const QCacheParams& p, int D, int fmt, void* stream);

// ---------------------------------------------------------------------------
// decode
// ---------------------------------------------------------------------------
struct QDecodeParams {
  const void* q;             // bf16 [S, N, Hq, d]
  const void* b;             // bf16 [N, r, Hkv*d]
  const int32_t* seq_lens;   // [S]
  const int32_t* offsets;    // [S, N] or null
  const float* k_scale;
  const float* v_scale;
  long long s_ss, s_sh, s_sp;
  const int32_t* page_table; // null => dense
  long long pt_stride;
  void* out;
  int out_f32;
  int S, N, Hq, Hkv, G;
  int rows_total;            // N * G
  int rows_per_group;        // rows of one work item (<= kMaxRowsPerItem)
  int n_rg;                  // row groups per (session, KV head)
  int n_u_slots;             // U tiles staged per K/V tile
  int mode;
  int max_seq_len;
  int u_rows;
  int num_pages;
  int stages, u_stages;      // ring stages of K/V tiles and of U tiles
  int balance;               // visit an item's tiles in a low-discrepancy order (QOrder)
  float scale_log2;          // softmax_scale * log2(e)
  float* partials;           // two records per CTA: see q_record_slot
  unsigned* tickets;         // a byte per CTA: see kQTicketBytes
  unsigned* flags;
  unsigned spin_cap;         // failure-detection test hook, as in DecodeParams
  int stall;
};

// Consumer warps of the decode kernel.  A warp holds the query rows of one row
// block in one of three shapes: up to 8 rows (keys as the MMA's M), up to 16
// (rows as M), up to 24 (16 + 8).  Items of 25 to 32 rows take two row blocks of
// 16.  Two warps of a row block share a tile, 32 keys each.
constexpr int kQWarps = 8;
constexpr int kQWarpKeys = 32;

struct QShape {
  int h16, h8, nrb;          // 16-row part, 8-row part, row blocks
};

__host__ __device__ constexpr QShape q_shape(int rows) {
  return rows <= 8 ? QShape{0, 1, 1} : rows <= 16 ? QShape{1, 0, 1} : rows <= 24 ? QShape{1, 1, 1} : QShape{1, 0, 2};
}

// Groups of warps that take a CTA's tiles in turn.
__host__ __device__ constexpr int q_groups(int nrb) { return kQWarps / (kQBlock / kQWarpKeys) / nrb; }

// Accumulator fragments that the warps exchange per pass when their rows are merged.
constexpr int kQMergeFrags = 4;
constexpr int kQMaxCtas = 160;  // CTAs of a launch at most (and so partial records of an item)
// Tickets of the items that are cut between CTAs, between the status header and the
// records.  An item counts in the byte of its first CTA (no two cut items share that one:
// of two, the earlier would end in it), so their place depends on no shape, and a
// workspace that served other shapes holds zeros there.  The other operators' workspaces
// keep their first tickets at these bytes, zero between calls as well.
constexpr int kQTicketBytes = 256;
static_assert(kQMaxCtas <= kQTicketBytes && kQMaxCtas < 256, "a byte counts the CTAs of an item");
constexpr int kQPlanBytes = 4 * 32 * 32, kQPlanBarriers = 12;  // the planner's table of tiles

// Shared-memory plan (bytes from a 1024-aligned base).
struct QDecodeSmem {
  int tile_bytes, u_bytes, u_off, rec_off, mb_off, ml_off, q_off, plan_off, a_off, bar_off, useq_off, misc_off, total;
};

__host__ __device__ inline QDecodeSmem q_smem_plan(int D, int RK, int rows_block, int nrb, int n_u_slots, int stages,
                                                   int u_stages) {
  QDecodeSmem s;
  const int RP = rows_block * nrb;
  s.tile_bytes = 2 * kQBlock * D;                                        // K then V of one tile
  s.u_bytes = n_u_slots * kQBlock * RK * 2;
  s.u_off = stages * s.tile_bytes;
  s.rec_off = s.u_off + u_stages * s.u_bytes;                            // [m | l | O | Z] of RP rows
  s.mb_off = round_up(s.rec_off + RP * (D + RK + 2) * 4, 16);            // the warps' fragments; the records' scales
  const int mb_bytes = kQWarps * kQMergeFrags * 512, table_bytes = kQMaxCtas * RP * 4;
  s.ml_off = s.mb_off + (mb_bytes > table_bytes ? mb_bytes : table_bytes);  // the warps' m and l
  s.q_off = round_up(s.ml_off + kQWarps * rows_block * 2 * 4, 16);       // 24-row blocks: query fragments
  s.plan_off = s.q_off + (rows_block == 24 ? 24 * D * 2 : 0);            // the planner's table
  s.a_off = s.plan_off + kQPlanBytes;                                    // offsets of the item's agents
  s.bar_off = round_up(s.a_off + kMaxAgents * 4, 16);
  s.useq_off = s.bar_off + (2 * (stages + u_stages) + kQPlanBarriers) * 8;  // tile number of each U stage
  s.misc_off = round_up(s.useq_off + u_stages * 4, 16);                  // the CTA's range, abort word, broadcast word
  s.total = s.misc_off + 96;
  return s;
}

inline size_t q_record_floats(int RP, int D, int RK) { return (size_t)RP * (D + RK + 2); }

// What a stretch of an item costs a CTA beside its tiles (its queries, the merge of its
// warps, publishing, finishing), in tiles: 5 to 7 us against 0.37 us for a tile at the
// HBM rate.  The work is split in units: an item has its tiles and this many more.
// (Without them a CTA whose share of the tiles was a handful of short or empty sessions
// finished item after item long after the others: 24 ragged sessions 114 us.)
constexpr int kQItemUnits = 16;
// Tiles by which an aligned share may exceed the even one, which ends inside items more
// often than it counts (128 items of 128 tiles: 60.3 us aligned, 63.1 even).
constexpr int kQAlignTiles = 4;

// CTAs per item when every item takes the same number, or 0 for the even split of all
// units (W) over the CTAs.  Aligned shares end where items end: a CTA then has one
// stretch of one item, where the even split's CTAs mostly have two (and a CTA that holds
// a whole item has nothing to publish or merge).  They are taken when their longest is at
// most kQAlignTiles above the even share, which has its item's units in it; of them the
// fewest CTAs per item that lengthen the share by no more than another stretch costs.
__host__ __device__ inline int q_item_ctas(int items, int ctas, int nt_max, int W) {
  const int most = items > 0 ? ctas / items : 0;
  if (most == 0) return 0;
  const int share = (nt_max + most - 1) / most;
  if (share > (W + ctas - 1) / ctas + kQAlignTiles) return 0;
  return (nt_max + share + kQItemUnits - 1) / (share + kQItemUnits);
}

lrkv_status launch_decode_quant(const QDecodeParams& p, int D, int RK, int rows, int fmt, const void* tmK,
                                const void* tmV, const void* tmU, int smem_bytes, int ctas, void* stream);
// One translation unit per (format, head_dim), so that they compile in parallel.
template <int FMT, int D>
lrkv_status launch_decode_quant_fd(const QDecodeParams& p, int RK, int rows, const void* tmK, const void* tmV,
                                   const void* tmU, int smem_bytes, int ctas, void* stream);

}  // namespace lrkv
