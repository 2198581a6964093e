// C entry points of the cache's pages.  Declarations are in include/bq.h.
#include <algorithm>

#include "kv_pages_kernels.hpp"

namespace {

using namespace bq;

KvPool pool_of(const bq_kv_cache* c) {
  KvPool p{};
  p.k = static_cast<uint8_t*>(c->k);
  p.v = static_cast<uint8_t*>(c->v);
  p.ks = c->k_scales;
  p.vs = c->v_scales;
  p.layers = c->layers;
  p.num_pages = c->num_pages;
  p.page_bytes = (int64_t)c->kv_heads * (int64_t)kv_head_bytes(c);
  p.page_scales = c->kv_heads * kKvBlocks;
  return p;
}

// Workgroups of the launch that copies, for `most` pairs at most: a unit of
// one pair each, up to sixteen for each CU, from where on they take several
// pairs.
dim3 copy_grid(const KvPool& p, int64_t most) {
  const int64_t units = p.page_bytes / kCopyUnit;
  const int64_t pairs = std::clamp<int64_t>(4096 / (units * p.layers * 2), 1, std::max<int64_t>(most, 1));
  return dim3((unsigned)(p.layers * 2), (unsigned)(units * pairs));
}

// entries: of the table, at most
int check_tables(const bq_kv_cache* cache, const int* table, const int* refs, int rows, int max_pages, const int* status,
                 const void* workspace, size_t workspace_bytes, int64_t entries = INT64_MAX) {
  const int st = kv_check_cache(cache);
  if (st != BQ_OK) return st;
  if (!table || !refs || !status) return BQ_ERR_NULL;
  if (rows < 1 || rows > (1 << 20) || max_pages < 1 || max_pages > (1 << 24) || (int64_t)rows * max_pages > entries)
    return BQ_ERR_SHAPE;
  if (!workspace || workspace_bytes < kv_plan_ints(cache->num_pages, rows) * 4) return BQ_ERR_WORKSPACE;
  if (!kv_aligned(table, 4) || !kv_aligned(refs, 4) || !kv_aligned(status, 4) || !kv_aligned(workspace, 16))
    return BQ_ERR_ALIGN;
  return BQ_OK;
}

KvPagesParams params_of(const bq_kv_cache* c, int* table, int* lens, int* refs, int rows, int max_pages, int* status,
                        void* workspace) {
  KvPagesParams p{};
  p.pool = pool_of(c);
  int* w = static_cast<int*>(workspace);
  p.plan.head = w;
  p.plan.src = w + kPlanHead;
  p.plan.dst = p.plan.src + c->num_pages;
  p.plan.take = p.plan.dst + c->num_pages;
  p.plan.row = p.plan.take + c->num_pages;
  p.table = table;
  p.lens = lens;
  p.refs = refs;
  p.status = status;
  p.rows = rows;
  p.max_pages = max_pages;
  return p;
}

int run(const void* plan, const void* carry, dim3 grid, KvPagesParams& p, void* stream) {
  const int st = kv_launch(plan, dim3(1), dim3(kPlanThreads), 0, stream, &p);
  return st != BQ_OK ? st : kv_launch(carry, grid, dim3(kCopyThreads), 0, stream, &p);
}

}  // namespace

extern "C" {

int bq_kv_pages_workspace(const bq_kv_cache* cache, int rows, size_t* bytes) {
  if (!bytes) return BQ_ERR_NULL;
  *bytes = 0;
  const int st = kv_check_cache(cache);
  if (st != BQ_OK) return st;
  if (rows < 1 || rows > (1 << 20)) return BQ_ERR_SHAPE;
  *bytes = kv_plan_ints(cache->num_pages, rows) * 4;
  return BQ_OK;
}

int bq_kv_fork(const bq_kv_cache* cache, int* table, int* lens, int* refs, int rows, int max_pages, const int* src,
               const int* dst, int n, int* status, void* workspace, size_t workspace_bytes, void* stream) {
  const int st = check_tables(cache, table, refs, rows, max_pages, status, workspace, workspace_bytes);
  if (st != BQ_OK) return st;
  if (!lens || !src || !dst) return BQ_ERR_NULL;
  if (n < 1 || n > rows) return BQ_ERR_SHAPE;
  if (!kv_aligned(lens, 4) || !kv_aligned(src, 4) || !kv_aligned(dst, 4)) return BQ_ERR_ALIGN;
  KvPagesParams p = params_of(cache, table, lens, refs, rows, max_pages, status, workspace);
  p.a = src;
  p.b = dst;
  p.n = n;
  return run(reinterpret_cast<const void*>(&kv_fork_plan_kernel), reinterpret_cast<const void*>(&kv_fork_kernel),
             copy_grid(p.pool, n), p, stream);
}

int bq_kv_resize(const bq_kv_cache* cache, int* table, int* lens, int* refs, int rows, int max_pages, const int* want,
                 int* status, void* workspace, size_t workspace_bytes, void* stream) {
  // the plan counts the pages that all rows ask for in 31 bits
  const int st = check_tables(cache, table, refs, rows, max_pages, status, workspace, workspace_bytes, INT32_MAX);
  if (st != BQ_OK) return st;
  if (!lens || !want) return BQ_ERR_NULL;
  if (!kv_aligned(lens, 4) || !kv_aligned(want, 4)) return BQ_ERR_ALIGN;
  KvPagesParams p = params_of(cache, table, lens, refs, rows, max_pages, status, workspace);
  p.a = want;
  return run(reinterpret_cast<const void*>(&kv_resize_plan_kernel), reinterpret_cast<const void*>(&kv_resize_kernel),
             copy_grid(p.pool, rows), p, stream);
}

int bq_kv_compact(const bq_kv_cache* cache, int* table, int* refs, int rows, int max_pages, int* status,
                  void* workspace, size_t workspace_bytes, void* stream) {
  const int st = check_tables(cache, table, refs, rows, max_pages, status, workspace, workspace_bytes);
  if (st != BQ_OK) return st;
  KvPagesParams p = params_of(cache, table, nullptr, refs, rows, max_pages, status, workspace);
  return run(reinterpret_cast<const void*>(&kv_compact_plan_kernel), reinterpret_cast<const void*>(&kv_compact_kernel),
             copy_grid(p.pool, cache->num_pages / 2 + 1), p, stream);
}

int bq_kv_copy_pages(const bq_kv_cache* cache, const int* src, const int* dst, int n, void* stream) {
  const int st = kv_check_cache(cache);
  if (st != BQ_OK) return st;
  if (!src || !dst) return BQ_ERR_NULL;
  if (n < 0) return BQ_ERR_SHAPE;
  if (!kv_aligned(src, 4) || !kv_aligned(dst, 4)) return BQ_ERR_ALIGN;
  if (n == 0) return BQ_OK;
  KvPagesParams p{};
  p.pool = pool_of(cache);
  p.a = src;
  p.b = dst;
  p.n = n;
  return kv_launch(reinterpret_cast<const void*>(&kv_copy_kernel), copy_grid(p.pool, n), dim3(kCopyThreads), 0,
                   stream, &p);
}

}  // extern "C"
