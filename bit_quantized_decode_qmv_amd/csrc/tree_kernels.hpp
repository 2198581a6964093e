// A tree of drafted tokens: its masks and positions, the path that the target
// tokens take, and moving that path's keys and values behind the context.
//
// Rows of a sequence are its tree, a row's parent stands ahead of it.  All
// three are short chains of latency (a launch, the batch's arrays, one or two
// reads that depend on them); what they move is small.
#pragma once

#include "kv_common.hpp"

namespace bq {

constexpr int kTreeRows = BQ_TREE_MAX_ROWS;

struct TreeBatch {
  const int *parent, *cu, *lens;
  int batch, total;
};
// A sequence's rows, and the position of its first one.
struct TreeSeq {
  int q0, n, base;
};
__device__ __forceinline__ TreeSeq tree_seq(const TreeBatch& p, int b) {
  TreeSeq s;
  s.q0 = min(max(p.cu[b], 0), p.total);
  s.n = min(max(p.cu[b + 1], s.q0), p.total) - s.q0;
  s.base = max(max(p.lens[b], 0) - s.n, 0);
  return s;
}
__device__ __forceinline__ int tree_parent(int parent, int row) { return parent >= 0 && parent < row ? parent : -1; }

struct TreePlanParams {
  TreeBatch t;
  uint64_t* mask;
  int* pos;
  int words, window;
};

// One workgroup a sequence: parents in LDS, a thread walks up from its row.
// The rows above come in falling order, so a row's words are finished one
// after the other, from the last on.  Measured: 32 trees of 61 rows, 8 levels,
// 3.6 us; one tree of 13 rows 1.9.
__global__ __launch_bounds__(256) void tree_plan_kernel(TreePlanParams p) {
  __shared__ short parent[kTreeRows];
  const TreeSeq s = tree_seq(p.t, (int)blockIdx.x);
  const int rows = min(s.n, 64 * p.words);
  for (int i = (int)threadIdx.x; i < rows; i += 256) parent[i] = (short)tree_parent(p.t.parent[s.q0 + i], i);
  __syncthreads();
  for (int i = (int)threadIdx.x; i < s.n; i += 256) {
    uint64_t* out = p.mask ? p.mask + (int64_t)(s.q0 + i) * p.words : nullptr;
    int depth = 0, word = p.words - 1;
    uint64_t bits = 0;
    for (int at = i < rows ? i : -1; at >= 0; at = parent[at], ++depth) {
      if (!out || (p.window > 0 && depth >= p.window)) continue;
      for (; word > at >> 6; --word) {
        out[word] = bits;
        bits = 0;
      }
      bits |= 1ull << (at & 63);
    }
    for (; out && word >= 0; --word) {
      out[word] = bits;
      bits = 0;
    }
    if (p.pos) p.pos[s.q0 + i] = s.base + max(depth - 1, 0);
  }
}

struct TreeAcceptParams {
  TreeBatch t;
  const int *target, *token;
  int *path, *kept, *next_token, *want;
  int max_path;
};

// One workgroup a sequence.  Each row asks whether its token is its parent's
// target, and if so stands as that parent's child, the lowest row of several;
// then one thread follows the children from row 0.  Measured: 32 trees of 61
// rows 3.5 us, one of 13 rows 2.0.
__global__ __launch_bounds__(256) void tree_accept_kernel(TreeAcceptParams p) {
  __shared__ int target[kTreeRows], child[kTreeRows], path[kTreeRows];
  __shared__ int found;
  const int b = (int)blockIdx.x;
  const TreeSeq s = tree_seq(p.t, b);
  const int rows = min(s.n, kTreeRows);
  constexpr int EACH = kTreeRows / 256;
  int parent[EACH], token[EACH];
#pragma unroll
  for (int k = 0; k < EACH; ++k) {
    const int i = (int)threadIdx.x + 256 * k;
    parent[k] = -1;
    if (i >= rows) continue;
    parent[k] = tree_parent(p.t.parent[s.q0 + i], i);
    token[k] = p.token[s.q0 + i];
    target[i] = p.target[s.q0 + i];
    child[i] = kTreeRows;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < EACH; ++k)
    if (parent[k] >= 0 && token[k] == target[parent[k]]) atomicMin(&child[parent[k]], (int)threadIdx.x + 256 * k);
  __syncthreads();
  if (threadIdx.x == 0) {
    int n = 0, last = 0;
    for (int at = 0; at < rows && n < p.max_path; at = child[at]) path[n++] = last = at;
    found = n;
    p.kept[b] = n;
    p.next_token[b] = n > 0 ? target[last] : -1;
    p.want[b] = s.n > 0 ? min(s.base + n, max(p.t.lens[b], 0)) : p.t.lens[b];
  }
  __syncthreads();
  for (int i = (int)threadIdx.x; i < p.max_path; i += 256) p.path[(int64_t)b * p.max_path + i] = i < found ? path[i] : -1;
}

struct KvKeepParams {
  uint8_t *k, *v;
  float *ks, *vs;
  KvBatch batch;
  const int *path, *kept;
  int max_path, kv_heads, head_dim, format;
};

// Four codes under ratios of their own; a ratio of 1 leaves a code's bits.
__device__ __forceinline__ uint32_t kv_rescale4(int format, uint32_t w, const float (&ratio)[4]) {
  float x[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = kv_value(format, (w >> (8 * j)) & 255u) * ratio[j];
  const uint32_t made = kv_codes4(format, x[0], x[1], x[2], x[3]);
  uint32_t out = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) out |= (ratio[j] == 1.f ? w : made) & (255u << (8 * j));
  return out;
}

// One workgroup for the K or V of one head of one sequence and layer.  Rows go
// to places at or ahead of theirs, so the blocks that take rows are worked
// from the first on, each read whole (its own codes and its rows') before it
// is written; no later block's rows lie in it.  K's 16-byte units are 16
// dimensions of a token; V's dwords are four tokens of a dimension, each byte
// from where its token was.  A row that stays where it is asks for nothing.
// A block of V is a dword of each of its page's 16-byte units, so its lines are
// the whole page's.  Measured: 4 layers of 8 heads of 128, 32 sequences of 2 to
// 9 rows, 15.8 us (the places of a page's four blocks found together, and two
// blocks read at once: 19.4, with 92 registers for 49); two layers and one
// sequence 4.9.
__global__ __launch_bounds__(256) void kv_keep_kernel(KvKeepParams p) {
  __shared__ int path[kTreeRows];
  __shared__ int from_page[kKvBlock], from_at[kKvBlock];  // of the block's tokens: page (-1: stays), place in it
  __shared__ float ratio[kKvBlock];
  __shared__ int first_moved;
  const int D = p.head_dim, tid = (int)threadIdx.x;
  int item = (int)blockIdx.x;
  const bool is_v = item & 1;
  item >>= 1;
  const int head = item % p.kv_heads, b = item / p.kv_heads;
  const KvSeq s = kv_seq(p.batch, b);
  const int base = s.len - s.n;
  const int count = min(min(max(p.kept[b], 0), p.max_path), min(s.n, kTreeRows));
  if (count == 0 || base < 0) return;
  if (tid == 0) first_moved = count;
  for (int i = tid; i < count; i += 256) path[i] = p.path[(int64_t)b * p.max_path + i];
  __syncthreads();
  bool bad = false;
  for (int i = tid; i < count; i += 256) {
    const int at = path[i];
    bad = bad || at <= (i > 0 ? path[i - 1] : -1) || at >= s.n;
    if (at != i) atomicMin(&first_moved, i);
  }
  if (__syncthreads_or(bad) || first_moved == count) return;
  // the layer's arrays
  const int64_t layer = (int64_t)blockIdx.y * p.batch.num_pages * p.kv_heads;
  uint8_t* codes = (is_v ? p.v : p.k) + (layer + head) * kKvPage * D;
  float* scales = (is_v ? p.vs : p.ks) + (layer + head) * kKvBlocks;
  const int64_t page_codes = (int64_t)p.kv_heads * kKvPage * D, page_scales = (int64_t)p.kv_heads * kKvBlocks;
  for (int block = (base + first_moved) / kKvBlock; block <= (base + count - 1) / kKvBlock; ++block) {
    const int page = kv_page(p.batch, b, block / (kKvPage / kKvBlock)), in = block % kKvBlocks;
    if (page < 0) continue;  // (the same for all threads)
    float* mine = scales + page * page_scales + in;
    if (tid < 64) {
      // a lane a token: where it comes from, under which scale
      const int lane = tid & 15, i = block * kKvBlock + lane - base;  // the row whose place this is
      int page_of = -1, at = 0;
      float scale = 0.f;
      const float held = *mine;
      if (i >= first_moved && i < count && path[i] != i) {
        const int t = base + path[i];
        page_of = kv_page(p.batch, b, t / kKvPage);
        at = t % kKvPage;
        if (page_of >= 0) scale = scales[page_of * page_scales + at / kKvBlock];
      }
      float top = __builtin_fmaxf(held, scale);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, o, 64));
      if (tid < 16) {
        from_page[lane] = page_of;
        from_at[lane] = at;
        const float own = page_of >= 0 ? scale : held;
        ratio[lane] = own == top ? 1.f : top > 0.f ? own / top : 0.f;
      }
      // (read by the lanes above; written once their codes are at hand)
      if (tid == 0) *mine = top;
    }
    __syncthreads();
    uint8_t* dst = codes + page * page_codes;
    if (!is_v) {
      uint4 w = make_uint4(0, 0, 0, 0);
      const int t = tid & 15, g = tid >> 4;  // 16 dimensions from 16 g on
      const bool on = g < (D >> 4);
      const int to = kv_k_at(in * kKvBlock + t, 16 * g, D);
      if (on) {
        const uint8_t* src = from_page[t] >= 0 ? codes + from_page[t] * page_codes + kv_k_at(from_at[t], 16 * g, D) : dst + to;
        w = *reinterpret_cast<const uint4*>(src);
      }
      __syncthreads();
      if (on) {
        const float r[4] = {ratio[t], ratio[t], ratio[t], ratio[t]};
        *reinterpret_cast<uint4*>(dst + to) = make_uint4(kv_rescale4(p.format, w.x, r), kv_rescale4(p.format, w.y, r),
                                                         kv_rescale4(p.format, w.z, r), kv_rescale4(p.format, w.w, r));
      }
    } else {
      uint32_t w[4];
      const int g = tid & 3;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int dim = (tid >> 2) + 64 * k;
        w[k] = 0;
        if (dim >= D) continue;
        w[k] = *reinterpret_cast<const uint32_t*>(dst + kv_v_at(in * kKvBlock + 4 * g, dim));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = 4 * g + j;
          if (from_page[t] < 0) continue;
          const uint32_t c = codes[from_page[t] * page_codes + kv_v_at(from_at[t], dim)];
          w[k] = (w[k] & ~(255u << (8 * j))) | (c << (8 * j));
        }
      }
      __syncthreads();
      const float r[4] = {ratio[4 * g], ratio[4 * g + 1], ratio[4 * g + 2], ratio[4 * g + 3]};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int dim = (tid >> 2) + 64 * k;
        if (dim < D)
          *reinterpret_cast<uint32_t*>(dst + kv_v_at(in * kKvBlock + 4 * g, dim)) = kv_rescale4(p.format, w[k], r);
      }
    }
    __syncthreads();
  }
}

}  // namespace bq
