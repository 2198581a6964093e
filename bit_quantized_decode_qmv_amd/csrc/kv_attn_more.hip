// C entry points of the attention with a window and sinks, and of a tree of
// drafted tokens, over the paged 8-bit cache.  Declarations are in
// include/bq.h.
#include "kv_attn_launch.hpp"

using namespace bq;

namespace {

// (no sequence is longer than this)
int sinks_of(int sinks) { return std::min(sinks, 1 << 30); }

}  // namespace

extern "C" {

int bq_kv_attn_sinks(const bq_kv_cache* cache, int layer, const void* q, void* out, long long q_stride,
                     long long out_stride, int q_heads, const int* cu, const int* lens, const int* table, int batch,
                     int max_pages, int total, float scale, int window, int sinks, void* workspace,
                     size_t workspace_bytes, void* stream) {
  if (sinks < 0) return BQ_ERR_SHAPE;
  KvAttnMore p{};
  p.sinks = sinks_of(sinks);
  return kv_attn_run(p, cache, layer, q, out, q_stride, out_stride, q_heads, cu, lens, table, batch, max_pages, total,
                     scale, window, BQ_KV_CAUSAL, workspace, workspace_bytes, stream);
}

int bq_kv_attn_tree(const bq_kv_cache* cache, int layer, const void* q, void* out, long long q_stride,
                    long long out_stride, int q_heads, const int* cu, const int* lens, const int* table, int batch,
                    int max_pages, int total, const void* mask, int mask_words, float scale, int window, int sinks,
                    void* workspace, size_t workspace_bytes, void* stream) {
  if (sinks < 0 || mask_words < 1 || mask_words > BQ_TREE_MAX_WORDS) return BQ_ERR_SHAPE;
  if (total > 0 && !mask) return BQ_ERR_NULL;
  if (!kv_aligned(mask, 8)) return BQ_ERR_ALIGN;
  KvAttnMore p{};
  p.mask = static_cast<const uint64_t*>(mask);
  p.words = mask_words;
  p.sinks = sinks_of(sinks);
  return kv_attn_run(p, cache, layer, q, out, q_stride, out_stride, q_heads, cu, lens, table, batch, max_pages, total,
                     scale, window, BQ_KV_CAUSAL, workspace, workspace_bytes, stream);
}

}  // extern "C"
