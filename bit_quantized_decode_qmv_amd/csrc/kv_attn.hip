// C entry points of the attention over the paged 8-bit cache.  Declarations
// are in include/bq.h.
#include "kv_attn_launch.hpp"

using namespace bq;

extern "C" {

int bq_kv_attn_workspace(const bq_kv_cache* cache, int q_heads, int batch, int total, size_t* bytes) {
  if (!bytes) return BQ_ERR_NULL;
  *bytes = 0;
  const int st = kv_check_attn(cache, q_heads, batch, total);
  if (st != BQ_OK) return st;
  const KvAttnPlan p = kv_attn_plan(cache, q_heads, batch, total, 1, SIZE_MAX);
  *bytes = p.bytes;
  return BQ_OK;
}

int bq_kv_attn(const bq_kv_cache* cache, int layer, const void* q, void* out, long long q_stride,
               long long out_stride, int q_heads, const int* cu, const int* lens, const int* table, int batch,
               int max_pages, int total, float scale, int window, int flags, void* workspace, size_t workspace_bytes,
               void* stream) {
  return kv_attn_run(KvAttnParams{}, cache, layer, q, out, q_stride, out_stride, q_heads, cu, lens, table, batch,
                     max_pages, total, scale, window, flags, workspace, workspace_bytes, stream);
}

}  // extern "C"
