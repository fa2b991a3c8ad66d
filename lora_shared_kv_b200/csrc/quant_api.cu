// C ABI of the 8-bit K/V cache: argument checks, work partition, launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include "api_common.h"
#include "quant.h"

using namespace lrkv::api;

namespace {

constexpr int kMaxRows = 1 << 30;  // row and key arithmetic stays within 32 bits

lrkv_status check_qkv(const lrkv_qkv_view* v, const lrkv_problem* p) {
  if (!v || !v->k || !v->v || !v->k_scale || !v->v_scale)
    return fail(LRKV_ERR_INVALID_ARGUMENT, "8-bit view or one of its k, v, k_scale, v_scale pointers is NULL");
  if (v->format != LRKV_Q_E4M3 && v->format != LRKV_Q_INT8) return fail(LRKV_ERR_INVALID_ARGUMENT, "8-bit format %d", v->format);
  if (!aligned16(v->k) || !aligned16(v->v)) return fail(LRKV_ERR_MISALIGNED, "8-bit k and v must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(v->k_scale) & 3u) || (reinterpret_cast<uintptr_t>(v->v_scale) & 3u))
    return fail(LRKV_ERR_MISALIGNED, "k_scale and v_scale must be 4-byte aligned");
  if (v->stride_token < p->head_dim || v->stride_head < 1 || v->scale_stride_head < 1)
    return fail(LRKV_ERR_INVALID_ARGUMENT, "8-bit view: strides too small");
  if (v->stride_token % 16 || v->stride_head % 16)
    return fail(LRKV_ERR_MISALIGNED, "8-bit view: token/head strides must be multiples of 16");
  if (v->page_table) {
    if (v->page_size != LRKV_QUANT_BLOCK) return fail(LRKV_ERR_UNSUPPORTED, "page_size %d (supported: %d)", v->page_size, LRKV_QUANT_BLOCK);
    if (v->num_pages < 1 || v->stride_page < 1 || v->stride_page % 16)
      return fail(LRKV_ERR_INVALID_ARGUMENT, "paged 8-bit view needs num_pages >= 1 and a stride_page that is a positive multiple of 16");
    if (v->page_table_stride < 1 || v->scale_stride_page < 1)
      return fail(LRKV_ERR_INVALID_ARGUMENT, "paged 8-bit view needs page_table_stride and scale_stride_page >= 1");
  } else if (p->num_sessions > 1) {
    if (v->stride_session < 1 || v->stride_session % 16)
      return fail(LRKV_ERR_MISALIGNED, "8-bit view: the session stride must be a positive multiple of 16");
    if (v->scale_stride_session < 1) return fail(LRKV_ERR_INVALID_ARGUMENT, "8-bit view: scale_stride_session must be >= 1");
  }
  return LRKV_OK;
}

// Checks and parameters (none if T is 0) shared by the write and the read.
lrkv_status cache_params(const lrkv_problem* p, const lrkv_kv_view* x, int32_t T, const lrkv_qkv_view* c, int32_t rows,
                         const int32_t* first, const int32_t* count, void* workspace, size_t workspace_bytes,
                         lrkv::QCacheParams* out) {
  lrkv_status s = check_problem(p);
  if (s != LRKV_OK) return s;
  if (T != 0 && (s = check_kv(x, p)) != LRKV_OK) return s;  // tensors of no rows have no address
  if ((s = check_qkv(c, p)) != LRKV_OK) return s;
  if (!workspace) return fail(LRKV_ERR_INVALID_ARGUMENT, "workspace must not be NULL");
  if (!aligned16(workspace)) return fail(LRKV_ERR_MISALIGNED, "workspace must be 16-byte aligned");
  if (workspace_bytes < LRKV_KV_QUANT_WORKSPACE_BYTES)
    return fail(LRKV_ERR_WORKSPACE_TOO_SMALL, "workspace %zu < %zu bytes", workspace_bytes, LRKV_KV_QUANT_WORKSPACE_BYTES);
  if (T < 0 || rows < 0) return fail(LRKV_ERR_INVALID_ARGUMENT, "need T >= 0 and a row capacity >= 0");
  if (rows > kMaxRows) return fail(LRKV_ERR_UNSUPPORTED, "more than %d rows a session", kMaxRows);
  if (T > rows && !count) return fail(LRKV_ERR_INVALID_ARGUMENT, "%d rows exceed the 8-bit cache's %d", T, rows);
  if (T > kMaxRows) return fail(LRKV_ERR_UNSUPPORTED, "T %d", T);
  if (T == 0) return LRKV_OK;
  if (c->page_table && ((long long)rows + LRKV_QUANT_BLOCK - 1) / LRKV_QUANT_BLOCK > c->page_table_stride)
    return fail(LRKV_ERR_INVALID_ARGUMENT, "%d rows exceed a page-table row of %lld pages", rows, (long long)c->page_table_stride);
  if (x->page_table && ((long long)T + LRKV_QUANT_BLOCK - 1) / LRKV_QUANT_BLOCK > x->page_table_stride)
    return fail(LRKV_ERR_INVALID_ARGUMENT, "%d rows exceed the bf16 view's page-table row of %lld pages", T, (long long)x->page_table_stride);
  lrkv::QCacheParams q = {};
  q.x[0] = static_cast<uint16_t*>(const_cast<void*>(x->k));
  q.x[1] = static_cast<uint16_t*>(const_cast<void*>(x->v));
  q.x_ss = x->stride_session;
  q.x_sh = x->stride_head;
  q.x_st = x->stride_token;
  q.x_sp = x->stride_page;
  q.x_table = x->page_table;
  q.x_pt = x->page_table_stride;
  q.x_pages = x->num_pages;
  q.c[0] = static_cast<uint8_t*>(c->k);
  q.c[1] = static_cast<uint8_t*>(c->v);
  q.scale[0] = c->k_scale;
  q.scale[1] = c->v_scale;
  q.c_ss = c->stride_session;
  q.c_sh = c->stride_head;
  q.c_st = c->stride_token;
  q.c_sp = c->stride_page;
  q.s_ss = c->scale_stride_session;
  q.s_sh = c->scale_stride_head;
  q.s_sp = c->scale_stride_page;
  q.c_table = c->page_table;
  q.c_pt = c->page_table_stride;
  q.c_pages = c->num_pages;
  q.rows = rows;
  q.first = first;
  q.count = count;
  q.S = p->num_sessions;
  q.Hkv = p->num_kv_heads;
  q.T = T;
  // blocks that T rows can touch: from a block's first row when no first row is given
  q.nblk = first ? (T + LRKV_QUANT_BLOCK - 2) / LRKV_QUANT_BLOCK + 1 : (T + LRKV_QUANT_BLOCK - 1) / LRKV_QUANT_BLOCK;
  q.flags = static_cast<unsigned*>(workspace);
  *out = q;
  return LRKV_OK;
}

struct QPlan {
  int G, R, n_rg, rows_per_group, n_u_slots, nt, ctas, stages, u_stages, smem, RP;
  long long items;
  size_t partials_off, bytes;
};

lrkv_status plan_decode_quant(const lrkv_problem* p, int max_seq_len, const DeviceInfo& dev, QPlan* pl) {
  lrkv_status s = check_problem(p);
  if (s != LRKV_OK) return s;
  if (max_seq_len < 0 || max_seq_len > kMaxRows) return fail(LRKV_ERR_INVALID_ARGUMENT, "max_seq_len %d", max_seq_len);
  pl->G = p->num_q_heads / p->num_kv_heads;
  const long long R = (long long)p->num_agents * pl->G;
  if (R > (1 << 20)) return fail(LRKV_ERR_UNSUPPORTED, "%lld query rows per KV head", R);
  pl->R = (int)R;
  pl->n_rg = (pl->R + lrkv::kMaxRowsPerItem - 1) / lrkv::kMaxRowsPerItem;
  pl->rows_per_group = (pl->R + pl->n_rg - 1) / pl->n_rg;
  pl->n_rg = (pl->R + pl->rows_per_group - 1) / pl->rows_per_group;  // no empty last group
  int max_ag = 1;
  for (int lo = 0; lo < pl->R; lo += pl->rows_per_group) {
    const int hi = lo + pl->rows_per_group < pl->R ? lo + pl->rows_per_group : pl->R;
    const int n = (hi - 1) / pl->G - lo / pl->G + 1;
    max_ag = n > max_ag ? n : max_ag;
  }
  pl->n_u_slots = p->mode == LRKV_BASE_SHARED ? max_ag : 1;
  pl->nt = max_seq_len > 0 ? (int)(((long long)max_seq_len + LRKV_QUANT_BLOCK - 1) / LRKV_QUANT_BLOCK) : 1;
  if (p->num_kv_heads > 0xFFFF) return fail(LRKV_ERR_UNSUPPORTED, "%d KV heads", p->num_kv_heads);
  const long long per_session = (long long)p->num_kv_heads * pl->n_rg;
  pl->items = p->num_sessions * per_session;
  if (pl->items > 0x3FFFFFF || pl->items * (pl->nt + lrkv::kQItemUnits) > 0x7FFF0000)
    return fail(LRKV_ERR_UNSUPPORTED, "too many (session, KV head, row group) items or tiles");
  const int sms = dev.sms < 1 ? 148 : dev.sms > lrkv::kQMaxCtas ? lrkv::kQMaxCtas : dev.sms;
  const long long W = pl->items * pl->nt;
  pl->ctas = (int)(W < sms ? W : sms);
  const lrkv::QShape sh = lrkv::q_shape(pl->rows_per_group);
  const int rows_block = 16 * sh.h16 + 8 * sh.h8;
  pl->RP = rows_block * sh.nrb;
  // One U stage per consumer group (fewer where U tiles are large), as long as two K/V
  // stages per group fit beside them; then as many K/V stages as fit, up to 16, in
  // multiples of the groups.
  const int optin = dev.smem_optin > 0 ? dev.smem_optin : 232448;
  const int groups = lrkv::q_groups(sh.nrb);
  auto smem_of = [&](int stages) {
    return lrkv::q_smem_plan(p->head_dim, p->rank, rows_block, sh.nrb, pl->n_u_slots, stages, pl->u_stages).total + 1024;
  };
  pl->u_stages = groups;
  while (pl->u_stages > 1 && smem_of(2 * groups) > optin) --pl->u_stages;
  int stages = 16;
  while (stages >= groups && smem_of(stages) > optin) stages -= groups;
  if (stages < groups) return fail(LRKV_ERR_UNSUPPORTED, "decode tiles do not fit in shared memory");
  pl->stages = stages;
  pl->smem = smem_of(stages);
  pl->partials_off = lrkv::kWsHeaderBytes + lrkv::kQTicketBytes;
  pl->bytes = pl->partials_off + (size_t)2 * pl->ctas * lrkv::q_record_floats(pl->RP, p->head_dim, p->rank) * 4;
  return LRKV_OK;
}

}  // namespace

namespace lrkv {

lrkv_status launch_decode_quant(const QDecodeParams& p, int D, int RK, int rows, int fmt, const void* tmK,
                                const void* tmV, const void* tmU, int smem, int ctas, void* stream) {
  if (fmt == LRKV_Q_E4M3)
    return D == 128 ? launch_decode_quant_fd<LRKV_Q_E4M3, 128>(p, RK, rows, tmK, tmV, tmU, smem, ctas, stream)
                    : launch_decode_quant_fd<LRKV_Q_E4M3, 64>(p, RK, rows, tmK, tmV, tmU, smem, ctas, stream);
  return D == 128 ? launch_decode_quant_fd<LRKV_Q_INT8, 128>(p, RK, rows, tmK, tmV, tmU, smem, ctas, stream)
                  : launch_decode_quant_fd<LRKV_Q_INT8, 64>(p, RK, rows, tmK, tmV, tmU, smem, ctas, stream);
}

}  // namespace lrkv

extern "C" {

lrkv_status lrkv_quantize_kv(const lrkv_problem* p, const lrkv_kv_view* src, int32_t T, const lrkv_qkv_view* dst,
                             int32_t dst_rows, const int32_t* first_rows, const int32_t* row_counts,
                             void* workspace, size_t workspace_bytes, lrkv_stream_t stream) {
  lrkv::QCacheParams q;
  lrkv_status s = cache_params(p, src, T, dst, dst_rows, first_rows, row_counts, workspace, workspace_bytes, &q);
  if (s != LRKV_OK || T == 0) return s;
  DeviceInfo dev;
  if ((s = device_info(&dev)) != LRKV_OK) return s;
  s = lrkv::launch_quantize(q, p->head_dim, dst->format, stream);
  if (s != LRKV_OK) return fail(s, "quantize launch failed: %s", cudaGetErrorString(cudaGetLastError()));
  return LRKV_OK;
}

lrkv_status lrkv_dequantize_kv(const lrkv_problem* p, const lrkv_qkv_view* src, int32_t src_rows, int32_t T,
                               const lrkv_kv_view* dst, const int32_t* first_rows, const int32_t* row_counts,
                               void* workspace, size_t workspace_bytes, lrkv_stream_t stream) {
  lrkv::QCacheParams q;
  lrkv_status s = cache_params(p, dst, T, src, src_rows, first_rows, row_counts, workspace, workspace_bytes, &q);
  if (s != LRKV_OK || T == 0) return s;
  DeviceInfo dev;
  if ((s = device_info(&dev)) != LRKV_OK) return s;
  s = lrkv::launch_dequantize(q, p->head_dim, src->format, stream);
  if (s != LRKV_OK) return fail(s, "dequantize launch failed: %s", cudaGetErrorString(cudaGetLastError()));
  return LRKV_OK;
}

size_t lrkv_decode_quant_workspace_bytes(const lrkv_problem* p, int32_t max_seq_len) {
  DeviceInfo dev;
  if (device_info(&dev) != LRKV_OK) {
    dev.sms = 148;
    dev.smem_optin = 232448;
  }
  QPlan pl;
  return plan_decode_quant(p, max_seq_len, dev, &pl) == LRKV_OK ? pl.bytes : 0;
}

lrkv_status lrkv_attn_decode_quant(const lrkv_problem* p, const void* q, const lrkv_qkv_view* kv,
                                   const int32_t* seq_lens, int32_t max_seq_len, const lrkv_u_view* u,
                                   const void* b, const int32_t* alora_offsets, void* out, int32_t out_dtype,
                                   void* workspace, size_t workspace_bytes, lrkv_stream_t stream) {
  lrkv_status s = check_problem(p);
  if (s != LRKV_OK) return s;
  if (!q || !seq_lens || !b || !out || !workspace)
    return fail(LRKV_ERR_INVALID_ARGUMENT, "q, seq_lens, b, out and workspace must not be NULL");
  if (!aligned16(q) || !aligned16(b) || !aligned16(out) || !aligned16(workspace))
    return fail(LRKV_ERR_MISALIGNED, "q, b, out and workspace must be 16-byte aligned");
  if (out_dtype != LRKV_BF16 && out_dtype != LRKV_F32) return fail(LRKV_ERR_INVALID_ARGUMENT, "out_dtype %d", out_dtype);
  if (max_seq_len < 0) return fail(LRKV_ERR_INVALID_ARGUMENT, "max_seq_len must be >= 0");
  if (max_seq_len > kMaxRows) return fail(LRKV_ERR_UNSUPPORTED, "max_seq_len %d", max_seq_len);
  if ((s = check_qkv(kv, p)) != LRKV_OK) return s;
  if ((s = check_u(u, p, max_seq_len)) != LRKV_OK) return s;
  if (kv->page_table && ((long long)max_seq_len + LRKV_QUANT_BLOCK - 1) / LRKV_QUANT_BLOCK > kv->page_table_stride)
    return fail(LRKV_ERR_INVALID_ARGUMENT, "max_seq_len %d exceeds a page-table row of %lld pages", max_seq_len, (long long)kv->page_table_stride);
  DeviceInfo dev;
  if ((s = device_info(&dev)) != LRKV_OK) return s;
  QPlan pl;
  if ((s = plan_decode_quant(p, max_seq_len, dev, &pl)) != LRKV_OK) return s;
  if (workspace_bytes < pl.bytes) return fail(LRKV_ERR_WORKSPACE_TOO_SMALL, "workspace %zu < %zu bytes", workspace_bytes, pl.bytes);

  const int D = p->head_dim, RK = p->rank;
  alignas(64) CUtensorMap tmK, tmV, tmU;
  {
    const CUtensorMapSwizzle swz = D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    const uint32_t box[4] = {(uint32_t)D, LRKV_QUANT_BLOCK, 1, 1};
    const bool paged = kv->page_table != nullptr;
    const uint64_t dims[4] = {(uint64_t)D, paged ? LRKV_QUANT_BLOCK : (uint64_t)(max_seq_len > 0 ? max_seq_len : 1),
                              (uint64_t)p->num_kv_heads, (uint64_t)(paged ? kv->num_pages : p->num_sessions)};
    const int64_t str[3] = {kv->stride_token, kv->stride_head, paged ? kv->stride_page : kv->stride_session};
    if ((s = make_map4(&tmK, kv->k, dims, str, box, swz, "8-bit K", CU_TENSOR_MAP_DATA_TYPE_UINT8, 1)) != LRKV_OK) return s;
    if ((s = make_map4(&tmV, kv->v, dims, str, box, swz, "8-bit V", CU_TENSOR_MAP_DATA_TYPE_UINT8, 1)) != LRKV_OK) return s;
  }
  {
    const CUtensorMapSwizzle swz = RK == 8 ? CU_TENSOR_MAP_SWIZZLE_NONE : RK == 16 ? CU_TENSOR_MAP_SWIZZLE_32B : CU_TENSOR_MAP_SWIZZLE_64B;
    const uint64_t dims[4] = {(uint64_t)RK, (uint64_t)(u->num_rows > 0 ? u->num_rows : 1),
                              (uint64_t)(p->mode == LRKV_BASE_SHARED ? p->num_agents : 1), (uint64_t)p->num_sessions};
    const int64_t str[3] = {u->stride_token, u->stride_agent, u->stride_session};
    const uint32_t box[4] = {(uint32_t)RK, LRKV_QUANT_BLOCK, 1, 1};
    if ((s = make_map4(&tmU, u->u, dims, str, box, swz, "U")) != LRKV_OK) return s;
  }
  lrkv::QDecodeParams dp = {};
  dp.q = q;
  dp.b = b;
  dp.seq_lens = seq_lens;
  dp.offsets = alora_offsets;
  dp.k_scale = kv->k_scale;
  dp.v_scale = kv->v_scale;
  dp.s_ss = kv->scale_stride_session;
  dp.s_sh = kv->scale_stride_head;
  dp.s_sp = kv->scale_stride_page;
  dp.page_table = kv->page_table;
  dp.pt_stride = kv->page_table_stride;
  dp.out = out;
  dp.out_f32 = out_dtype == LRKV_F32;
  dp.S = p->num_sessions;
  dp.N = p->num_agents;
  dp.Hq = p->num_q_heads;
  dp.Hkv = p->num_kv_heads;
  dp.G = pl.G;
  dp.rows_total = pl.R;
  dp.rows_per_group = pl.rows_per_group;
  dp.n_rg = pl.n_rg;
  dp.n_u_slots = pl.n_u_slots;
  dp.mode = p->mode;
  dp.max_seq_len = max_seq_len;
  dp.u_rows = u->num_rows;
  dp.num_pages = kv->page_table ? kv->num_pages : 0;
  dp.stages = pl.stages;
  dp.u_stages = pl.u_stages;
  dp.balance = p->mode == LRKV_BASE_SHARED;
  dp.scale_log2 = scale_of(p) * 1.4426950408889634f;
  char* ws = static_cast<char*>(workspace);
  dp.flags = reinterpret_cast<unsigned*>(ws);
  dp.tickets = reinterpret_cast<unsigned*>(ws + lrkv::kWsHeaderBytes);
  dp.partials = reinterpret_cast<float*>(ws + pl.partials_off);
  take_stall_hook(&dp.spin_cap, &dp.stall);
  s = lrkv::launch_decode_quant(dp, D, RK, pl.rows_per_group, kv->format, &tmK, &tmV, &tmU, pl.smem, pl.ctas, stream);
  if (s != LRKV_OK) return fail(s, "decode launch failed: %s", cudaGetErrorString(cudaGetLastError()));
  return LRKV_OK;
}

}  // extern "C"
