// C entry points of the rotary positions and of the paged 8-bit cache's
// writing and reading.  Declarations are in include/bq.h.
#include <algorithm>
#include <cmath>
#include <limits>

#include "kv_cache_kernels.hpp"

namespace {

using namespace bq;

// Arguments of a rotation: rot_dim 0 (nothing turns) needs no arrays.
int check_angles(const int* pos, const float* inv_freq, const int* axis, int rot_dim, int axes, int flags, int head_dim,
                 int total) {
  if ((flags & ~BQ_ROPE_ADJACENT) != 0) return BQ_ERR_FLAGS;
  if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 16 != 0 || axes < 1 || axes > BQ_ROPE_MAX_AXES) return BQ_ERR_SHAPE;
  if (rot_dim > 0 && total > 0 && (!pos || !inv_freq)) return BQ_ERR_NULL;
  if (!kv_aligned(pos, 4) || !kv_aligned(inv_freq, 4) || !kv_aligned(axis, 4)) return BQ_ERR_ALIGN;
  return BQ_OK;
}
RopeAngles angles(const int* pos, const float* inv_freq, const int* axis, int rot_dim, int axes, int flags, int total) {
  return RopeAngles{pos, inv_freq, axis, rot_dim, axes, (flags & BQ_ROPE_ADJACENT) ? 1 : 0, total};
}
// Tokens a workgroup rotates: one while the tokens are few, more once they
// fill the chip several times over, as far as the table of angles holds them;
// of these numbers the one whose units best fill the rounds of its threads.
int rope_tokens_per_wg(int tokens, int rot_dim, int units, int threads) {
  const int most = std::clamp(tokens / 512, 1, std::min(8, 2 * kRopeTable / std::max(rot_dim, 1)));
  const int64_t round = (int64_t)kRopeAtOnce * threads;
  const auto fill = [&](int t) { return (double)t * units / (double)(((int64_t)t * units + round - 1) / round); };
  int best = 1;
  for (int t = 2; t <= most; ++t)
    if (fill(t) >= fill(best)) best = t;
  return best;
}

// Arguments of a norm: w null is none.
int check_norm(const float* w, float eps) {
  if (!kv_aligned(w, 4)) return BQ_ERR_ALIGN;
  return std::isfinite(eps) && eps >= 0.f ? BQ_OK : BQ_ERR_SHAPE;
}

// The hardware's reciprocal root takes a number below the normal ones as 0, and
// a row of zeros times its infinity would be no number.  The mean of squares of
// any other fp16 row is at least 2^-58: such an eps is not seen in it.
NormWeight norm_of(const float* w, float eps) {
  return NormWeight{w, eps > 0.f ? std::max(eps, std::numeric_limits<float>::min()) : 0.f};
}

template <bool NORM>
const void* pick_append(int per) {
  return per == 4 ? reinterpret_cast<const void*>(&kv_append_kernel<4, NORM>)
       : per == 2 ? reinterpret_cast<const void*>(&kv_append_kernel<2, NORM>)
                  : reinterpret_cast<const void*>(&kv_append_kernel<1, NORM>);
}

int append(const bq_kv_cache* cache, int layer, const void* k, const void* v, long long k_stride,
           long long v_stride, const void* q, void* q_out, long long q_stride, long long q_out_stride,
           int q_heads, const int* cu, const int* lens, const int* table, int batch, int max_pages, int total,
           const int* pos, const float* inv_freq, const int* axis, int rot_dim, int axes, int flags,
           const NormWeight& k_norm, const NormWeight& q_norm, void* stream) {
  int st = kv_check_cache(cache);
  if (st != BQ_OK) return st;
  if (total > 0 && (!k || !v || (q && !q_out))) return BQ_ERR_NULL;
  if (layer < 0 || layer >= cache->layers) return BQ_ERR_SHAPE;
  st = kv_check_batch(cu, lens, table, batch, max_pages, total);
  if (st != BQ_OK) return st;
  const int D = cache->head_dim;
  if (q && (q_heads < 1 || q_heads > 65536)) return BQ_ERR_SHAPE;
  st = check_angles(pos, inv_freq, axis, rot_dim, axes, flags, D, total);
  if (st != BQ_OK) return st;
  if (!kv_rows_ok(k, k_stride, cache->kv_heads * D) || !kv_rows_ok(v, v_stride, cache->kv_heads * D)) return BQ_ERR_ALIGN;
  if (q && (!kv_rows_ok(q, q_stride, q_heads * D) || !kv_rows_ok(q_out, q_out_stride, q_heads * D))) return BQ_ERR_ALIGN;
  if (total == 0) return BQ_OK;
  KvAppendNormParams p{};
  const size_t at = (size_t)layer * kv_layer_heads(cache);
  p.k = static_cast<uint8_t*>(cache->k) + at * kv_head_bytes(cache);
  p.v = static_cast<uint8_t*>(cache->v) + at * kv_head_bytes(cache);
  p.ks = cache->k_scales + at * kKvBlocks;
  p.vs = cache->v_scales + at * kKvBlocks;
  p.nk = static_cast<const _Float16*>(k);
  p.nv = static_cast<const _Float16*>(v);
  p.nk_stride = k_stride;
  p.nv_stride = v_stride;
  p.q = RopeRows{static_cast<const _Float16*>(q), static_cast<_Float16*>(q_out), q_stride, q_out_stride, q_heads, D};
  p.a = angles(pos, inv_freq, axis, rot_dim, axes, flags, total);
  p.batch = KvBatch{cu, lens, table, batch, max_pages, cache->num_pages, total};
  p.kv_heads = cache->kv_heads;
  p.head_dim = D;
  p.format = cache->format;
  // n tokens lie in at most (n + 126) / 64 pages
  const int64_t items = ((int64_t)total + (int64_t)std::min(batch, total) * 126) / kKvPage * cache->kv_heads;
  // Blocks of a page a thread: one (two where heads are wide) while the pages
  // are fewer than half the CUs and written whole, else all four.  Measured, 8
  // heads of 128: 128 tokens 13.1 us with one and 16.8 with four, 1500 tokens
  // 26.0 and 23.4, 4093 tokens 50 and 38.7; 4 heads of 256: 300 tokens 17.7 us
  // with two and 20.6 with four, eight times 301 tokens 31.6 and 27.0.
  const int per = total < 16 * (int64_t)batch || items > 128 ? 4 : D <= 128 ? 1 : 2;
  const int threads = 2 * D * (kKvBlocks / per);
  const bool norm = k_norm.w || q_norm.w;
  p.k_norm = k_norm;
  p.q_norm = q_norm;
  p.q_tokens_per_wg = rope_tokens_per_wg(total, rot_dim, q_heads * (q_norm.w ? norm_lanes(D) : D / 16), threads);
  const int64_t q_wgs = q ? (total + p.q_tokens_per_wg - 1) / p.q_tokens_per_wg : 0;
  if (items + q_wgs > 0x7FFFFFFF) return BQ_ERR_SHAPE;
  p.items = (int)items;
  const void* fn = norm ? pick_append<true>(per) : pick_append<false>(per);
  return kv_launch(fn, dim3((unsigned)(items + q_wgs)), dim3((unsigned)threads), 0, stream, &p);
}

}  // namespace

extern "C" {

int bq_rope(const void* x, void* y, long long x_stride, long long y_stride, int tokens, int heads, int head_dim,
            const int* pos, const float* inv_freq, const int* axis, int rot_dim, int axes, int flags, void* stream) {
  if (tokens > 0 && (!x || !y)) return BQ_ERR_NULL;
  if (tokens < 0 || tokens > (1 << 28) || heads < 1 || heads > 65536 || head_dim < 16 || head_dim > 1024 ||
      head_dim % 16 != 0)
    return BQ_ERR_SHAPE;
  const int st = check_angles(pos, inv_freq, axis, rot_dim, axes, flags, head_dim, tokens);
  if (st != BQ_OK) return st;
  if (!kv_rows_ok(x, x_stride, heads * head_dim) || !kv_rows_ok(y, y_stride, heads * head_dim)) return BQ_ERR_ALIGN;
  if (tokens == 0) return BQ_OK;
  RopeParams p{};
  p.rows = RopeRows{static_cast<const _Float16*>(x), static_cast<_Float16*>(y), x_stride, y_stride, heads, head_dim};
  p.a = angles(pos, inv_freq, axis, rot_dim, axes, flags, tokens);
  p.tokens_per_wg = rope_tokens_per_wg(tokens, rot_dim, heads * head_dim / 16, 256);
  return kv_launch(reinterpret_cast<const void*>(&rope_kernel),
                   dim3((unsigned)((tokens + p.tokens_per_wg - 1) / p.tokens_per_wg)), dim3(256), 0, stream, &p);
}

int bq_norm_rope(const void* x, void* y, long long x_stride, long long y_stride, int tokens, int heads, int head_dim,
                 const float* weight, float eps, const int* pos, const float* inv_freq, const int* axis, int rot_dim,
                 int axes, int flags, void* stream) {
  if (tokens > 0 && (!x || !y)) return BQ_ERR_NULL;
  if (!weight) return BQ_ERR_NULL;
  if (tokens < 0 || tokens > (1 << 28) || heads < 1 || heads > 65536 || head_dim < 16 || head_dim > 1024 ||
      head_dim % 16 != 0)
    return BQ_ERR_SHAPE;
  int st = check_norm(weight, eps);
  if (st != BQ_OK) return st;
  st = check_angles(pos, inv_freq, axis, rot_dim, axes, flags, head_dim, tokens);
  if (st != BQ_OK) return st;
  if (!kv_rows_ok(x, x_stride, heads * head_dim) || !kv_rows_ok(y, y_stride, heads * head_dim)) return BQ_ERR_ALIGN;
  if (tokens == 0) return BQ_OK;
  NormRopeParams p{};
  p.rows = RopeRows{static_cast<const _Float16*>(x), static_cast<_Float16*>(y), x_stride, y_stride, heads, head_dim};
  p.a = angles(pos, inv_freq, axis, rot_dim, axes, flags, tokens);
  p.norm = norm_of(weight, eps);
  p.tokens_per_wg = rope_tokens_per_wg(tokens, rot_dim, heads * norm_lanes(head_dim), 256);
  return kv_launch(reinterpret_cast<const void*>(&norm_rope_kernel),
                   dim3((unsigned)((tokens + p.tokens_per_wg - 1) / p.tokens_per_wg)), dim3(256), 0, stream, &p);
}

int bq_kv_append(const bq_kv_cache* cache, int layer, const void* k, const void* v, long long k_stride,
                 long long v_stride, const void* q, void* q_out, long long q_stride, long long q_out_stride,
                 int q_heads, const int* cu, const int* lens, const int* table, int batch, int max_pages, int total,
                 const int* pos, const float* inv_freq, const int* axis, int rot_dim, int axes, int flags,
                 void* stream) {
  return append(cache, layer, k, v, k_stride, v_stride, q, q_out, q_stride, q_out_stride, q_heads, cu, lens, table,
                batch, max_pages, total, pos, inv_freq, axis, rot_dim, axes, flags, NormWeight{}, NormWeight{}, stream);
}

int bq_kv_append_norm(const bq_kv_cache* cache, int layer, const void* k, const void* v, long long k_stride,
                      long long v_stride, const void* q, void* q_out, long long q_stride, long long q_out_stride,
                      int q_heads, const int* cu, const int* lens, const int* table, int batch, int max_pages,
                      int total, const float* k_weight, const float* q_weight, float eps, const int* pos,
                      const float* inv_freq, const int* axis, int rot_dim, int axes, int flags, void* stream) {
  int st = check_norm(k_weight, eps);
  if (st == BQ_OK) st = check_norm(q_weight, eps);
  if (st != BQ_OK) return st;
  return append(cache, layer, k, v, k_stride, v_stride, q, q_out, q_stride, q_out_stride, q_heads, cu, lens, table,
                batch, max_pages, total, pos, inv_freq, axis, rot_dim, axes, flags, norm_of(k_weight, eps),
                norm_of(q ? q_weight : nullptr, eps), stream);
}

int bq_kv_read(const bq_kv_cache* cache, int layer, void* k, void* v, const int* cu, const int* lens, const int* table,
               int batch, int max_pages, int total, void* stream) {
  int st = kv_check_cache(cache);
  if (st != BQ_OK) return st;
  if (total > 0 && (!k || !v)) return BQ_ERR_NULL;
  if (layer < 0 || layer >= cache->layers) return BQ_ERR_SHAPE;
  st = kv_check_batch(cu, lens, table, batch, max_pages, total);
  if (st != BQ_OK) return st;
  if (!kv_aligned(k, 16) || !kv_aligned(v, 16)) return BQ_ERR_ALIGN;
  if (total == 0) return BQ_OK;
  KvReadParams p{};
  const size_t at = (size_t)layer * kv_layer_heads(cache);
  p.k = static_cast<const uint8_t*>(cache->k) + at * kv_head_bytes(cache);
  p.v = static_cast<const uint8_t*>(cache->v) + at * kv_head_bytes(cache);
  p.ks = cache->k_scales + at * kKvBlocks;
  p.vs = cache->v_scales + at * kKvBlocks;
  p.ok = static_cast<_Float16*>(k);
  p.ov = static_cast<_Float16*>(v);
  p.batch = KvBatch{cu, lens, table, batch, max_pages, cache->num_pages, total};
  p.kv_heads = cache->kv_heads;
  p.head_dim = cache->head_dim;
  p.format = cache->format;
  // as in the append, and one item more for a sequence shorter than its rows
  const int64_t seqs = std::min(batch, total);
  const int64_t items = (((int64_t)total + seqs * 126) / kKvPage + seqs) * cache->kv_heads;
  if (items > 0x7FFFFFFF) return BQ_ERR_SHAPE;
  return kv_launch(reinterpret_cast<const void*>(&kv_read_kernel), dim3((unsigned)items), dim3(256), 0, stream, &p);
}

}  // extern "C"
