// Host side of the attention over the paged 8-bit cache: how a call is laid out,
// and its launches, for the two kinds of parameters.  Each kind's kernel
// instances live in a translation unit of their own (kv_attn.hip,
// kv_attn_more.hip), so that they compile in parallel.
#pragma once

#include <algorithm>
#include <cmath>

#include "kv_prompt_kernels.hpp"

namespace bq {

template <typename P, int D, int RT>
const void* kv_rows_kernel(int format) {
  return format == BQ_KV_I8 ? reinterpret_cast<const void*>(&kv_attn_rows_kernel<D, BQ_KV_I8, RT, P>)
                            : reinterpret_cast<const void*>(&kv_attn_rows_kernel<D, BQ_KV_E4M3, RT, P>);
}
template <typename P>
const void* kv_pick_rows(int D, int rows, int format) {
  if (rows == 32) return D == 64 ? kv_rows_kernel<P, 64, 2>(format) : kv_rows_kernel<P, 128, 2>(format);
  return D == 64 ? kv_rows_kernel<P, 64, 1>(format) : D == 128 ? kv_rows_kernel<P, 128, 1>(format)
       : D == 192 ? kv_rows_kernel<P, 192, 1>(format) : kv_rows_kernel<P, 256, 1>(format);
}

template <typename P, int D>
const void* kv_prompt_kernel(int format) {
  return format == BQ_KV_I8 ? reinterpret_cast<const void*>(&kv_attn_prompt_kernel<D, BQ_KV_I8, P>)
                            : reinterpret_cast<const void*>(&kv_attn_prompt_kernel<D, BQ_KV_E4M3, P>);
}
template <typename P>
const void* kv_pick_prompt(int D, int format) {
  return D == 64 ? kv_prompt_kernel<P, 64>(format) : D == 128 ? kv_prompt_kernel<P, 128>(format)
       : D == 192 ? kv_prompt_kernel<P, 192>(format) : kv_prompt_kernel<P, 256>(format);
}
template <typename P>
const void* kv_pick_join(int D) {
  return D == 64 ? reinterpret_cast<const void*>(&kv_attn_join_kernel<64, P>)
       : D == 128 ? reinterpret_cast<const void*>(&kv_attn_join_kernel<128, P>)
       : D == 192 ? reinterpret_cast<const void*>(&kv_attn_join_kernel<192, P>)
                  : reinterpret_cast<const void*>(&kv_attn_join_kernel<256, P>);
}

// Few rows: workgroups to aim at, one for each CU, whose registers one fills.
// Parts beyond that (twice, three times as many) measured slower on every
// batch: with one workgroup on a CU, its start (batch, table, first page) and
// its join, some 8 us, overlap with nobody's loads.  From kKvRowTiles workgroups
// on no tile is split.
constexpr int kKvTarget = 256, kKvRowTiles = 4096;
constexpr int kKvCounters = BQ_KV_ATTN_COUNTER_BYTES / 4;

// How a call is laid out: rows of a tile, tiles of a head at most, and the
// workgroups of a head to aim at (0: no tile is split).
struct KvAttnPlan {
  int rows;
  int64_t tiles, target;
  size_t bytes;
};
// One plan for both kinds of parameters: bq_kv_attn_workspace gives the size for either.
inline KvAttnPlan kv_attn_plan(const bq_kv_cache* c, int q_heads, int batch, int total, int64_t max_pages, size_t workspace_bytes) {
  KvAttnPlan p{};
  // By the rows of a sequence, on average; two row groups of wide heads do
  // not fit a wave's registers.  Tiles of 32 for up to 128 rows instead:
  // 6 x 77 rows over 1500 tokens, 16 heads of 64, 17.9 us against 16.1, 24
  // times 41.4 against 33.3, 8 x 96 rows over 4000, heads of 128, 31.7 against
  // 27.0; over 8000 tokens 34.3 against 37.4 (the length is not looked at).
  const int64_t rows = (int64_t)total * (q_heads / c->kv_heads);
  const bool narrow = c->head_dim <= 128;
  p.rows = rows <= 16 * (int64_t)batch ? 16 : narrow && rows <= 32 * (int64_t)batch ? 32 : kPromptRows;
  const bool prompt = p.rows == kPromptRows;
  const int wgs = prompt && narrow ? 2 * kKvTarget : kKvTarget;  // that run at once
  p.tiles = std::min(batch, total) + rows / p.rows;
  const size_t slot = (size_t)kv_part_floats(p.rows, c->head_dim) * 4;
  const size_t room = workspace_bytes > BQ_KV_ATTN_COUNTER_BYTES ? (workspace_bytes - BQ_KV_ATTN_COUNTER_BYTES) / slot : 0;
  const int each = std::clamp(wgs / c->kv_heads, 1, kKvMaxParts);
  // enough tiles of their own, or more pages than 31 bits count
  if (p.tiles * c->kv_heads >= (prompt ? wgs : kKvRowTiles) || p.tiles * max_pages > 0x3FFFFFFF) return p;
  // parts that the counters and the workspace hold, for each head
  p.target = std::min<int64_t>(each, (int64_t)((prompt ? room : std::min(room, (size_t)kKvCounters)) / c->kv_heads) - p.tiles);
  if (p.target < 2) p.target = 0;
  if (p.target > 0) p.bytes = BQ_KV_ATTN_COUNTER_BYTES + (size_t)((p.tiles + p.target) * c->kv_heads) * slot;
  return p;
}

inline int kv_check_attn(const bq_kv_cache* cache, int q_heads, int batch, int total) {
  const int st = kv_check_cache(cache);
  if (st != BQ_OK) return st;
  if (q_heads < 1 || q_heads > 65536 || q_heads % cache->kv_heads != 0) return BQ_ERR_SHAPE;
  if (batch < 1 || batch > (1 << 20) || total < 0 || total > (1 << 28) ||
      (int64_t)total * (q_heads / cache->kv_heads) > 0x7FFFFF00)
    return BQ_ERR_SHAPE;
  return BQ_OK;
}

// The launches of `wgs` shares of each head; a grid's y holds 65535 at most.
template <typename P>
int kv_launch_shares(const void* fn, int64_t wgs, int threads, P& p, void* stream) {
  constexpr int64_t kMost = 32768;
  for (int64_t at = 0; at < wgs; at += kMost) {
    p.item0 = (int)at;
    const int st = kv_launch(fn, dim3((unsigned)p.kv_heads, (unsigned)std::min(kMost, wgs - at)), dim3((unsigned)threads), 0,
                             stream, &p);
    if (st != BQ_OK) return st;
  }
  return BQ_OK;
}

// A call.  p holds what its kind of rows adds (mask, words, sinks); the rest is
// checked and filled in here.
template <typename P>
int kv_attn_run(P p, const bq_kv_cache* cache, int layer, const void* q, void* out, long long q_stride,
                long long out_stride, int q_heads, const int* cu, const int* lens, const int* table, int batch,
                int max_pages, int total, float scale, int window, int flags, void* workspace, size_t workspace_bytes,
                void* stream) {
  int st = kv_check_attn(cache, q_heads, batch, total);
  if (st != BQ_OK) return st;
  if (total > 0 && (!q || !out)) return BQ_ERR_NULL;
  if ((flags & ~BQ_KV_CAUSAL) != 0 || (window > 0 && !(flags & BQ_KV_CAUSAL))) return BQ_ERR_FLAGS;
  if (layer < 0 || layer >= cache->layers || window < 0 || !std::isfinite(scale)) return BQ_ERR_SHAPE;
  st = kv_check_batch(cu, lens, table, batch, max_pages, total);
  if (st != BQ_OK) return st;
  const int D = cache->head_dim;
  if (!kv_rows_ok(q, q_stride, q_heads * D) || !kv_rows_ok(out, out_stride, q_heads * D) || !kv_aligned(workspace, 16))
    return BQ_ERR_ALIGN;
  if (total == 0) return BQ_OK;
  const size_t at = (size_t)layer * kv_layer_heads(cache);
  p.k = static_cast<const uint8_t*>(cache->k) + at * kv_head_bytes(cache);
  p.v = static_cast<const uint8_t*>(cache->v) + at * kv_head_bytes(cache);
  p.ks = cache->k_scales + at * kKvBlocks;
  p.vs = cache->v_scales + at * kKvBlocks;
  p.q = static_cast<const _Float16*>(q);
  p.out = static_cast<_Float16*>(out);
  p.q_stride = q_stride;
  p.out_stride = out_stride;
  p.batch = KvBatch{cu, lens, table, batch, max_pages, cache->num_pages, total};
  p.kv_heads = cache->kv_heads;
  p.group = q_heads / cache->kv_heads;
  p.causal = flags & BQ_KV_CAUSAL;
  p.window = std::min(window, 1 << 30);  // no sequence is longer; a row's place may be negative
  p.scale = scale * 1.44269504f;
  const KvAttnPlan pl = kv_attn_plan(cache, q_heads, batch, total, max_pages, workspace ? workspace_bytes : 0);
  p.target = (int)pl.target;
  // (many rows, measured: parts of 4 pages are 17% faster than of 8 at D 64,
  // 13% slower at D 128.  Wide heads, 4 with 6 query heads each, us in parts of
  // 4, 8 and 16 pages: 40 rows of 2 sequences of up to 4000 tokens, D 256, 34.2,
  // 39.8 and 56.1, D 192 29.3, 33.5 and 47.2; 100 rows over 8000, D 256, 66.5,
  // 66.5 and 60.1; five rows of 8 sequences of up to 16000 67.5, 67.5 and 58.3)
  p.min_pages = pl.rows < kPromptRows ? 0 : std::is_same_v<P, KvAttnMore> ? 2 : D == 64 ? 4 : 8;
  p.counters = static_cast<unsigned*>(workspace);
  p.part = workspace ? reinterpret_cast<float*>(static_cast<char*>(workspace) + BQ_KV_ATTN_COUNTER_BYTES) : nullptr;
  const int64_t wgs = pl.tiles + pl.target;
  if (pl.rows < kPromptRows)
    return kv_launch_shares(kv_pick_rows<P>(D, pl.rows, cache->format), wgs, 64 * kv_waves(D), p, stream);
  st = kv_launch_shares(kv_pick_prompt<P>(D, cache->format), wgs, kPromptThreads, p, stream);
  if (st != BQ_OK || pl.target == 0) return st;
  // (tiles that are split are fewer than the workgroups to aim at)
  const int64_t joined = pl.tiles * (kPromptRows / 16);
  return kv_launch(kv_pick_join<P>(D), dim3((unsigned)cache->kv_heads, (unsigned)joined), dim3(256), 0, stream, &p);
}

}  // namespace bq
