// C entry points of a tree of drafted tokens.  Declarations are in
// include/bq.h.
#include <algorithm>

#include "tree_kernels.hpp"

namespace {

using namespace bq;

int check_tree(const int* parent, const int* cu, const int* lens, int batch, int total) {
  if (!cu || !lens || (total > 0 && !parent)) return BQ_ERR_NULL;
  if (batch < 1 || batch > (1 << 20) || total < 0 || total > (1 << 28)) return BQ_ERR_SHAPE;
  return kv_aligned(parent, 4) && kv_aligned(cu, 4) && kv_aligned(lens, 4) ? BQ_OK : BQ_ERR_ALIGN;
}

}  // namespace

extern "C" {

int bq_tree_plan(const int* parent, const int* cu, const int* lens, int batch, int total, int mask_words, int window,
                 void* mask, int* pos, void* stream) {
  const int st = check_tree(parent, cu, lens, batch, total);
  if (st != BQ_OK) return st;
  if (total > 0 && !mask && !pos) return BQ_ERR_NULL;
  if (mask_words < 1 || mask_words > BQ_TREE_MAX_WORDS || window < 0) return BQ_ERR_SHAPE;
  if (!kv_aligned(mask, 8) || !kv_aligned(pos, 4)) return BQ_ERR_ALIGN;
  if (total == 0) return BQ_OK;
  TreePlanParams p{TreeBatch{parent, cu, lens, batch, total}, static_cast<uint64_t*>(mask), pos, mask_words, window};
  return kv_launch(reinterpret_cast<const void*>(&tree_plan_kernel), dim3((unsigned)batch), dim3(256), 0, stream, &p);
}

int bq_tree_accept(const int* target, const int* token, const int* parent, const int* cu, const int* lens, int batch,
                   int total, int max_path, int* path, int* kept, int* next_token, int* want, void* stream) {
  const int st = check_tree(parent, cu, lens, batch, total);
  if (st != BQ_OK) return st;
  if ((total > 0 && (!target || !token)) || !path || !kept || !next_token || !want) return BQ_ERR_NULL;
  if (max_path < 1 || max_path > BQ_TREE_MAX_ROWS) return BQ_ERR_SHAPE;
  for (const int* x : {target, token, (const int*)path, (const int*)kept, (const int*)next_token, (const int*)want})
    if (!kv_aligned(x, 4)) return BQ_ERR_ALIGN;
  TreeAcceptParams p{TreeBatch{parent, cu, lens, batch, total}, target, token, path, kept, next_token, want, max_path};
  return kv_launch(reinterpret_cast<const void*>(&tree_accept_kernel), dim3((unsigned)batch), dim3(256), 0, stream, &p);
}

int bq_kv_keep(const bq_kv_cache* cache, const int* cu, const int* lens, const int* table, int batch, int max_pages,
               const int* path, int max_path, const int* kept, void* stream) {
  int st = kv_check_cache(cache);
  if (st != BQ_OK) return st;
  st = kv_check_batch(cu, lens, table, batch, max_pages, 0);
  if (st != BQ_OK) return st;
  if (!path || !kept) return BQ_ERR_NULL;
  if (max_path < 1 || max_path > BQ_TREE_MAX_ROWS) return BQ_ERR_SHAPE;
  if (!kv_aligned(path, 4) || !kv_aligned(kept, 4)) return BQ_ERR_ALIGN;
  const int64_t items = 2 * (int64_t)batch * cache->kv_heads;
  if (items * 256 > 0xFFFFFFFF) return BQ_ERR_SHAPE;
  KvKeepParams p{};
  p.k = static_cast<uint8_t*>(cache->k);
  p.v = static_cast<uint8_t*>(cache->v);
  p.ks = cache->k_scales;
  p.vs = cache->v_scales;
  p.batch = KvBatch{cu, lens, table, batch, max_pages, cache->num_pages, INT32_MAX};  // (no array has a row of each)
  p.path = path;
  p.kept = kept;
  p.max_path = max_path;
  p.kv_heads = cache->kv_heads;
  p.head_dim = cache->head_dim;
  p.format = cache->format;
  return kv_launch(reinterpret_cast<const void*>(&kv_keep_kernel), dim3((unsigned)items, (unsigned)cache->layers),
                   dim3(256), 0, stream, &p);
}

}  // extern "C"
