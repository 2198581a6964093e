// Rotary positions with several axes, writing tokens into the paged 8-bit
// cache, and reading them back.
//
// Rotation: pair r of a head's first rot dimensions turns by
// a = pos[axis[r]][token] * inv_freq[r],
//   y1 = x1 cos a - x2 sin a,  y2 = x2 cos a + x1 sin a,
// with x1, x2 the dimensions r and r + rot/2, or 2r and 2r + 1 (adjacent);
// the dimensions past rot pass through.  fp32 arithmetic, one rounding to
// fp16 (rotated q) or to a code (rotated k).
//
// Codes: value = scale * code with one scale for each block of 16 tokens and
// head.  A call that brings the tokens [start, len) of a sequence gives each
// block it touches the scale
//   s = max(max |new value| / 127 (e4m3: / 448), the block's scale if it
//       holds tokens before start),
// codes each new value as rne(x / s), brings the codes of older tokens of
// the block to the new scale (unchanged when the scale did not grow), and
// clears the block's tokens past len.
#pragma once

#include "kv_common.hpp"

namespace bq {

constexpr int kRopeAdjacent = BQ_ROPE_ADJACENT;

struct RopeAngles {
  const int* pos;         // [axes][total]
  const float* inv_freq;  // [rot / 2]
  const int* axis;        // [rot / 2], or null: axis 0
  int rot, axes, adjacent, total;
};

// A unit is 16 elements of one head's row, as two 16-byte pieces: in the
// rotated part the two halves of eight pairs (adjacent pairs: 16 consecutive
// elements), past it 16 consecutive elements.
__device__ __forceinline__ void rope_unit_at(const RopeAngles& a, int unit, int& lo, int& hi) {
  const int pairs = a.rot >> 4;
  if (unit < pairs && !a.adjacent) {
    lo = unit * 8;
    hi = (a.rot >> 1) + unit * 8;
  } else {
    lo = unit * 16;
    hi = lo + 8;
  }
}

// The 16 values of a unit, rotated, in the order of the two pieces.
__device__ __forceinline__ void rope_unit(const RopeAngles& a, int unit, int token, const half8_t& lo,
                                          const half8_t& hi, float (&y)[16]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    y[j] = (float)lo[j];
    y[8 + j] = (float)hi[j];
  }
  if (unit >= (a.rot >> 4)) return;
  float c[8], s[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int r = unit * 8 + j;
    int ax = a.axis ? a.axis[r] : 0;
    ax = min(max(ax, 0), a.axes - 1);
    rope_cos_sin(rope_freq(a.inv_freq[r]), a.pos[(int64_t)ax * a.total + token], c[j], s[j]);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int i1 = a.adjacent ? 2 * j : j, i2 = a.adjacent ? 2 * j + 1 : 8 + j;
    const float x1 = y[i1], x2 = y[i2];
    y[i1] = x1 * c[j] - x2 * s[j];
    y[i2] = x2 * c[j] + x1 * s[j];
  }
}

struct RopeRows {
  const _Float16* x;
  _Float16* y;
  int64_t x_stride, y_stride;  // elements from token to token
  int heads, head_dim;
};

// Thread `thread` of `threads` over the units of `tokens` rows from `token0`.
// Every unit is read whole before it is written, so y may be x.
__device__ __forceinline__ void rope_rows(const RopeRows& p, const RopeAngles& a, int token0, int tokens, int thread,
                                          int threads) {
  const int units = p.head_dim >> 4, per = p.heads * units;
  for (int i = thread; i < tokens * per; i += threads) {
    const int t = i / per, u = i - t * per, head = u / units, unit = u - head * units, token = token0 + t;
    int lo, hi;
    rope_unit_at(a, unit, lo, hi);
    const _Float16* x = p.x + (int64_t)token * p.x_stride + head * p.head_dim;
    float v[16];
    rope_unit(a, unit, token, *reinterpret_cast<const half8_t*>(x + lo), *reinterpret_cast<const half8_t*>(x + hi), v);
    half8_t o0, o1;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      o0[j] = (_Float16)v[j];
      o1[j] = (_Float16)v[8 + j];
    }
    _Float16* y = p.y + (int64_t)token * p.y_stride + head * p.head_dim;
    *reinterpret_cast<half8_t*>(y + lo) = o0;
    *reinterpret_cast<half8_t*>(y + hi) = o1;
  }
}

struct RopeParams {
  RopeRows rows;
  RopeAngles a;
  int tokens_per_wg;
};
__global__ __launch_bounds__(256) void rope_kernel(RopeParams p) {
  const int t0 = (int)blockIdx.x * p.tokens_per_wg;
  rope_rows(p.rows, p.a, t0, min(p.tokens_per_wg, p.a.total - t0), (int)threadIdx.x, 256);
}

struct KvAppendParams {
  uint8_t *k, *v;               // the layer's codes
  float *ks, *vs;               // and scales
  const _Float16 *nk, *nv;      // new rows [total][kv_heads][D]
  int64_t nk_stride, nv_stride;
  RopeRows q;                   // x null: no q
  RopeAngles a;
  KvBatch batch;
  int kv_heads, head_dim, format;
  int items, q_tokens_per_wg;   // page items (at most), then workgroups over q
};

// One workgroup per (page, head) that new tokens lie in; 2 * D threads, the
// first D take K and the others V.  A thread holds one unit of one token of
// the block at hand; the codes go through LDS to be written in page order.
__global__ __launch_bounds__(512) void kv_append_kernel(KvAppendParams p) {
  __shared__ float red[2][4];
  __shared__ __align__(16) uint8_t codes[2][kKvBlock * 256];
  const int D = p.head_dim, units = D >> 4;
  if ((int)blockIdx.x >= p.items) {
    const int t0 = ((int)blockIdx.x - p.items) * p.q_tokens_per_wg;
    rope_rows(p.q, p.a, t0, min(p.q_tokens_per_wg, p.batch.total - t0), (int)threadIdx.x, (int)blockDim.x);
    return;
  }
  const int item = (int)blockIdx.x / p.kv_heads, head = (int)blockIdx.x % p.kv_heads;
  int b, local;
  if (!kv_locate(item, p.batch.batch, [&](int i) { int f; return kv_touched(kv_seq(p.batch, i), f); }, b, local)) return;
  const KvSeq s = kv_seq(p.batch, b);
  int first;
  kv_touched(s, first);
  const int at = first + local;
  const int page = kv_page(p.batch, b, at);
  if (page < 0) return;
  const int start = max(s.len - s.n, 0);
  const int which = (int)threadIdx.x >= D ? 1 : 0, tid = (int)threadIdx.x - which * D;
  const int tok = tid / units, unit = tid - tok * units;
  const int wave = tid >> 6, waves = D >> 6;
  const int64_t head_at = (int64_t)page * p.kv_heads + head;
  uint8_t* dst = (which ? p.v : p.k) + head_at * kKvPage * D;
  float* scales = (which ? p.vs : p.ks) + head_at * kKvBlocks;
  const _Float16* src = which ? p.nv : p.nk;
  const int64_t stride = which ? p.nv_stride : p.nk_stride;
  RopeAngles a = p.a;
  if (which) a.rot = 0;
  int lo, hi;
  rope_unit_at(a, unit, lo, hi);
  for (int i = 0; i < kKvBlocks; ++i) {
    const int t0 = at * kKvPage + i * kKvBlock;  // the block's first token
    if (t0 + kKvBlock <= start || t0 >= s.len) continue;
    const int t = t0 + tok;
    const bool old = t < start, fresh = !old && t < s.len;
    float x[16];
    float top = 0.f;
    if (fresh) {
      const int row = s.q0 + t - (s.len - s.n);
      const _Float16* r = src + (int64_t)row * stride + head * D;
      rope_unit(a, unit, row, *reinterpret_cast<const half8_t*>(r + lo), *reinterpret_cast<const half8_t*>(r + hi), x);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float m = __builtin_fabsf(x[j]);
        top = m < __builtin_inff() ? __builtin_fmaxf(top, m) : top;  // finite values only
      }
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int dim = j < 8 ? lo + j : hi + j - 8, pt = i * kKvBlock + tok;
        x[j] = old ? kv_value(p.format, dst[which ? kv_v_at(pt, dim) : kv_k_at(pt, dim, D)]) : 0.f;
      }
    }
    const float held = t0 < start ? scales[i] : 0.f;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, o, 64));
    if ((tid & 63) == 0) red[which][wave] = top;
    __syncthreads();
    for (int w = 0; w < waves; ++w) top = __builtin_fmaxf(top, red[which][w]);
    const float scale = __builtin_fmaxf(top / kv_qmax(p.format), held);
    const float mul = scale > 0.f ? (old ? held / scale : 1.f / scale) : 0.f;
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
      const uint32_t w = kv_codes4(p.format, x[j] * mul, x[j + 1] * mul, x[j + 2] * mul, x[j + 3] * mul);
      *reinterpret_cast<uint32_t*>(&codes[which][tok * D + (j < 8 ? lo + j : hi + j - 8)]) = w;
    }
    __syncthreads();
    if (tid == 0) scales[i] = scale;
    if (!which) {
      // 16 bytes a thread: (c, g, t) of block i
      const int c = tid >> 6, g = (tid >> 4) & 3, tt = tid & 15;
      const uint4 w = *reinterpret_cast<const uint4*>(&codes[0][tt * D + c * 64 + g * 16]);
      *reinterpret_cast<uint4*>(dst + ((i * units / 4 + c) * 64 + g * 16 + tt) * 16) = w;
    } else {
      // four tokens of a dimension are a dword; four dwords a thread
      for (int e = tid; e < 4 * D; e += D) {
        const int g = e / D, dim = e - g * D;
        uint32_t w = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) w |= (uint32_t)codes[1][(4 * g + j) * D + dim] << (8 * j);
        *reinterpret_cast<uint32_t*>(dst + kv_v_at(i * kKvBlock + 4 * g, dim)) = w;
      }
    }
    __syncthreads();
  }
}

struct KvReadParams {
  const uint8_t *k, *v;
  const float *ks, *vs;
  _Float16 *ok, *ov;  // [total][kv_heads][D]
  KvBatch batch;
  int kv_heads, head_dim, format;
};

// One workgroup per (page, head) that the last tokens of a sequence lie in:
// the page's codes go to LDS as they are stored, and a thread writes 16
// values of a token.  Tokens that no page holds are written as zeros.
__global__ __launch_bounds__(256) void kv_read_kernel(KvReadParams p) {
  __shared__ __align__(16) uint8_t page_codes[2][kKvPage * 256];
  const int D = p.head_dim, units = D >> 4;
  const int item = (int)blockIdx.x / p.kv_heads, head = (int)blockIdx.x % p.kv_heads;
  int b, local;
  // a sequence shorter than its rows: its first rows are zeros, one item more
  const auto count = [&](int i) {
    const KvSeq s = kv_seq(p.batch, i);
    int f;
    return kv_touched(s, f) + (s.n > s.len ? 1 : 0);
  };
  if (!kv_locate(item, p.batch.batch, count, b, local)) return;
  const KvSeq s = kv_seq(p.batch, b);
  int first;
  const int pages = kv_touched(s, first);
  if (local == pages) {
    for (int i = (int)threadIdx.x; i < (s.n - s.len) * units * 2; i += 256) {
      const int which = i & 1, u = (i >> 1) % units, row = s.q0 + (i >> 1) / units;
      half8_t* o = reinterpret_cast<half8_t*>((which ? p.ov : p.ok) + ((int64_t)row * p.kv_heads + head) * D + u * 16);
      o[0] = o[1] = half8_t{};
    }
    return;
  }
  const int at = first + local, page = kv_page(p.batch, b, at);
  const int64_t head_at = (int64_t)max(page, 0) * p.kv_heads + head;
  for (int i = (int)threadIdx.x; i < 8 * D; i += 256) {
    const int which = i >= 4 * D, e = i - which * 4 * D;
    const uint4* src = reinterpret_cast<const uint4*>((which ? p.v : p.k) + head_at * kKvPage * D);
    reinterpret_cast<uint4*>(page_codes[which])[e] = src[e];
  }
  __syncthreads();
  const int t0 = max(s.len - s.n - at * kKvPage, 0), t1 = min(s.len - at * kKvPage, kKvPage);
  for (int i = (int)threadIdx.x; i < (t1 - t0) * units * 2; i += 256) {
    const int which = i & 1, u = (i >> 1) % units, t = t0 + (i >> 1) / units;
    const float scale = page < 0 ? 0.f : (which ? p.vs : p.ks)[head_at * kKvBlocks + t / kKvBlock];
    const int row = s.q0 + at * kKvPage + t - (s.len - s.n);
    half8_t o[2];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const uint32_t c = page_codes[which][which ? kv_v_at(t, u * 16 + j) : kv_k_at(t, u * 16 + j, D)];
      o[j >> 3][j & 7] = (_Float16)(page < 0 ? 0.f : kv_value(p.format, c) * scale);
    }
    half8_t* dst = reinterpret_cast<half8_t*>((which ? p.ov : p.ok) + ((int64_t)row * p.kv_heads + head) * D + u * 16);
    dst[0] = o[0];
    dst[1] = o[1];
  }
}

}  // namespace bq
