// C entry points of the attention over the paged 8-bit cache.  Declarations
// are in include/bq.h.
#include <algorithm>
#include <cmath>

#include "kv_attn_kernels.hpp"

namespace {

using namespace bq;

template <int D, int RT>
const void* rows_kernel(int format) {
  return format == BQ_KV_I8 ? reinterpret_cast<const void*>(&kv_attn_rows_kernel<D, BQ_KV_I8, RT>)
                            : reinterpret_cast<const void*>(&kv_attn_rows_kernel<D, BQ_KV_E4M3, RT>);
}
template <int RT>
const void* pick_rows(int D, int format) {
  return D == 64 ? rows_kernel<64, RT>(format) : D == 128 ? rows_kernel<128, RT>(format)
       : D == 192 ? rows_kernel<192, RT>(format) : rows_kernel<256, RT>(format);
}

constexpr int kCounters = BQ_KV_ATTN_COUNTER_BYTES / 4;
constexpr int kTarget = 1024;   // workgroups of a call
constexpr int kMinPages = 4;    // one page for each wave of a part

// How a call is laid out: rows of a tile, tiles of a head at most, and the
// workgroups of a head to aim at (0: no tile is split).
struct Plan {
  int rows;
  int64_t tiles, target, slot;
};
Plan plan(const bq_kv_cache* c, int q_heads, int batch, int total, size_t workspace_bytes) {
  Plan p{};
  const int group = q_heads / c->kv_heads;
  p.rows = 16;
  p.tiles = std::min(batch, total) + (int64_t)total * group / p.rows;
  p.slot = (int64_t)kv_part_floats(p.rows, c->head_dim) * 4;
  // parts that the workspace holds, for each head
  const int64_t room = workspace_bytes > BQ_KV_ATTN_COUNTER_BYTES
                           ? ((int64_t)workspace_bytes - BQ_KV_ATTN_COUNTER_BYTES) / (p.slot * c->kv_heads) : 0;
  const int64_t items = std::min<int64_t>(room, kCounters / c->kv_heads);
  p.target = std::min<int64_t>(kTarget / c->kv_heads + 1, items - p.tiles);
  if (p.tiles * c->kv_heads >= kTarget || p.target < 2) p.target = 0;
  return p;
}

int check_attn(const bq_kv_cache* cache, int q_heads, int batch, int total) {
  const int st = kv_check_cache(cache);
  if (st != BQ_OK) return st;
  if (q_heads < 1 || q_heads > 65536 || q_heads % cache->kv_heads != 0) return BQ_ERR_SHAPE;
  if (batch < 1 || batch > (1 << 20) || total < 0 || total > (1 << 28) ||
      (int64_t)total * (q_heads / cache->kv_heads) > 0x7FFFFFFF)
    return BQ_ERR_SHAPE;
  return BQ_OK;
}

}  // namespace

extern "C" {

int bq_kv_attn_workspace(const bq_kv_cache* cache, int q_heads, int batch, int total, size_t* bytes) {
  if (!bytes) return BQ_ERR_NULL;
  *bytes = 0;
  const int st = check_attn(cache, q_heads, batch, total);
  if (st != BQ_OK) return st;
  const Plan p = plan(cache, q_heads, batch, total, SIZE_MAX / 4);
  if (p.target > 0) *bytes = BQ_KV_ATTN_COUNTER_BYTES + (size_t)((p.tiles + p.target) * cache->kv_heads * p.slot);
  return BQ_OK;
}

int bq_kv_attn(const bq_kv_cache* cache, int layer, const void* q, void* out, long long q_stride,
               long long out_stride, int q_heads, const int* cu, const int* lens, const int* table, int batch,
               int max_pages, int total, float scale, int window, int flags, void* workspace, size_t workspace_bytes,
               void* stream) {
  int st = check_attn(cache, q_heads, batch, total);
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
  KvAttnParams p{};
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
  p.window = window;
  p.scale = scale * 1.44269504f;
  const Plan pl = plan(cache, q_heads, batch, total, workspace ? workspace_bytes : 0);
  p.target = (int)pl.target;
  p.min_pages = kMinPages;
  p.counters = static_cast<unsigned*>(workspace);
  p.part = workspace ? reinterpret_cast<float*>(static_cast<char*>(workspace) + BQ_KV_ATTN_COUNTER_BYTES) : nullptr;
  if (pl.tiles + pl.target > 0x7FFFFFFF) return BQ_ERR_SHAPE;
  return kv_launch(pick_rows<1>(D, cache->format), dim3((unsigned)(pl.tiles + pl.target), (unsigned)cache->kv_heads),
                   dim3(256), 0, stream, &p);
}

}  // extern "C"
