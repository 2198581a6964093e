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
//
// Norms: where a row is normed first, x is x * rsqrt(mean(x^2) + eps) * w over
// its head's dimensions, in fp32 and without a rounding of its own.  The root
// comes first: x times it is at most sqrt(head_dim), while the root of a small
// row times a weight may pass fp32's range, and where x is 0 be no number.
#pragma once

#include <type_traits>

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

// cos and sin of pair r at a token.
__device__ __forceinline__ float2 rope_pair(const RopeAngles& a, int r, int token) {
  int ax = a.axis ? a.axis[r] : 0;
  ax = min(max(ax, 0), a.axes - 1);
  float2 cs;
  rope_cos_sin(rope_freq(a.inv_freq[r]), a.pos[(int64_t)ax * a.total + token], cs.x, cs.y);
  return cs;
}

// A unit's two pieces turned by its eight (cos, sin), in fp32.
__device__ __forceinline__ void rope_turn(int adjacent, const float2 (&cs)[8], float (&y)[16]) {
  if (adjacent) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x1 = y[2 * j], x2 = y[2 * j + 1];
      y[2 * j] = x1 * cs[j].x - x2 * cs[j].y;
      y[2 * j + 1] = x2 * cs[j].x + x1 * cs[j].y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x1 = y[j], x2 = y[8 + j];
      y[j] = x1 * cs[j].x - x2 * cs[j].y;
      y[8 + j] = x2 * cs[j].x + x1 * cs[j].y;
    }
  }
}

struct RopeRows {
  const _Float16* x;
  _Float16* y;
  int64_t x_stride, y_stride;  // elements from token to token
  int heads, head_dim;
};

// (cos, sin) of the tokens at hand, formed once for all heads.
constexpr int kRopeTable = 2048;
constexpr int kRopeAtOnce = 4;  // units of a thread whose loads are in flight together

// A workgroup's `tokens` rows from `token0`: the angles of its tokens go to
// LDS once for all heads, then a thread turns units, four at a time with
// their loads in flight together.  Bound by HBM; the table costs one pair a
// thread for every token of 128 dimensions (angles formed by each unit
// instead: 85 us for 35 us).  Every unit is read whole before it is written,
// so y may be x.  Measured: 8191 tokens of 48 heads of 128, three axes, 35 us
// (5.8 TB/s read and written), 5 tokens 3.5 us.
__device__ __forceinline__ void rope_rows(const RopeRows& p, const RopeAngles& a, int token0, int tokens, int thread,
                                          int threads, float2* table) {
  const int half = a.rot >> 1;
  for (int i = thread; i < tokens * half; i += threads) {
    const int t = (int)((unsigned)i / (unsigned)half);
    table[i] = rope_pair(a, i - t * half, token0 + t);
  }
  __syncthreads();
  const int units = p.head_dim >> 4, per = p.heads * units, all = tokens * per;
  constexpr int AT_ONCE = kRopeAtOnce;
  for (int i0 = thread; i0 < all; i0 += AT_ONCE * threads) {
    half8_t v[AT_ONCE][2];
    int lo[AT_ONCE], hi[AT_ONCE], tok[AT_ONCE], unit[AT_ONCE], at[AT_ONCE];
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) {
      const int i = min(i0 + k * threads, all - 1);  // no branch: the last unit is read again
      tok[k] = (int)((unsigned)i / (unsigned)per);
      const int u = i - tok[k] * per, head = (int)((unsigned)u / (unsigned)units);
      unit[k] = u - head * units;
      at[k] = head * p.head_dim;
      rope_unit_at(a, unit[k], lo[k], hi[k]);
      const _Float16* x = p.x + (int64_t)(token0 + tok[k]) * p.x_stride + at[k];
      v[k][0] = *reinterpret_cast<const half8_t*>(x + lo[k]);
      v[k][1] = *reinterpret_cast<const half8_t*>(x + hi[k]);
    }
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) {
      if (i0 + k * threads >= all) break;
      if (unit[k] < (a.rot >> 4)) {
        float y[16];
        float2 cs[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          y[j] = (float)v[k][0][j];
          y[8 + j] = (float)v[k][1][j];
          cs[j] = table[tok[k] * half + unit[k] * 8 + j];
        }
        rope_turn(a.adjacent, cs, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[k][0][j] = (_Float16)y[j];
          v[k][1][j] = (_Float16)y[8 + j];
        }
      }
      _Float16* y = p.y + (int64_t)(token0 + tok[k]) * p.y_stride + at[k];
      *reinterpret_cast<half8_t*>(y + lo[k]) = v[k][0];
      *reinterpret_cast<half8_t*>(y + hi[k]) = v[k][1];
    }
  }
}

struct RopeParams {
  RopeRows rows;
  RopeAngles a;
  int tokens_per_wg;
};
__global__ __launch_bounds__(256) void rope_kernel(RopeParams p) {
  __shared__ float2 table[kRopeTable];
  const int t0 = (int)blockIdx.x * p.tokens_per_wg;
  rope_rows(p.rows, p.a, t0, min(p.tokens_per_wg, p.a.total - t0), (int)threadIdx.x, 256, table);
}

// A norm of each head's row ahead of the rotation.
struct NormWeight {
  const float* w;  // [head_dim], or null: no norm
  float eps;
};
// Lanes that a head's row takes where it is normed: its units, filled up to a
// power of two, so that a row's sum stays inside a wave.
__host__ __device__ inline int norm_lanes(int head_dim) {
  int lanes = 1;
  while (lanes * 16 < head_dim) lanes *= 2;
  return lanes;
}

// The sum over groups of `lanes` lanes, the same bits on each: within 16 by data
// parallel primitives (neighbours, pairs, then mirrors, whose lanes hold equal
// sums by then).
template <int CTL>
__device__ __forceinline__ float norm_add(float x) {
  return x + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTL, 0xF, 0xF, false));
}
__device__ __forceinline__ float norm_sum(float x, int lanes) {
  if (lanes >= 2) x = norm_add<0xB1>(x);    // quad_perm [1, 0, 3, 2]
  if (lanes >= 4) x = norm_add<0x4E>(x);    // quad_perm [2, 3, 0, 1]
  if (lanes >= 8) x = norm_add<0x141>(x);   // row_half_mirror
  if (lanes >= 16) x = norm_add<0x140>(x);  // row_mirror
  if (lanes >= 32) x += __shfl_xor(x, 16, 64);
  if (lanes >= 64) x += __shfl_xor(x, 32, 64);
  return x;
}

// rope_rows with a norm: a thread's unit is the same in all of its rounds
// (a round is a multiple of 64 threads), so its sixteen weights stay in
// registers, and a row's sum of squares is the work of `lanes` lanes side by
// side.  Bound by HBM like the rotation alone; the sum is hidden behind the
// loads of the other rounds.  Measured in a captured run, 48 heads of 128: 8191
// tokens 35.6 us (5.6 TB/s; the rotation alone 34.7), 5 tokens 3.7 (3.1).
__device__ __forceinline__ void norm_rope_rows(const RopeRows& p, const RopeAngles& a, const NormWeight& norm, int token0,
                                               int tokens, int thread, int threads, float2* table) {
  const int half = a.rot >> 1;
  for (int i = thread; i < tokens * half; i += threads) {
    const int t = (int)((unsigned)i / (unsigned)half);
    table[i] = rope_pair(a, i - t * half, token0 + t);
  }
  const int lanes = norm_lanes(p.head_dim), per = p.heads * lanes, all = tokens * per;
  const int unit = thread & (lanes - 1);
  const bool mine = unit < (p.head_dim >> 4), turns = unit < (a.rot >> 4);
  int lo, hi;
  rope_unit_at(a, mine ? unit : 0, lo, hi);
  float w[16];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    w[j] = norm.w[lo + j];
    w[8 + j] = norm.w[hi + j];
  }
  const float mean = 1.f / (float)p.head_dim;
  __syncthreads();
  constexpr int AT_ONCE = kRopeAtOnce;
  for (int i0 = thread; i0 < all; i0 += AT_ONCE * threads) {
    half8_t v[AT_ONCE][2];
    int tok[AT_ONCE], at[AT_ONCE];
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) {
      const int i = min(i0 + k * threads, all - 1);  // no branch: the last row is read again
      tok[k] = (int)((unsigned)i / (unsigned)per);
      at[k] = (int)((unsigned)(i - tok[k] * per) / (unsigned)lanes) * p.head_dim;
      const _Float16* x = p.x + (int64_t)(token0 + tok[k]) * p.x_stride + at[k];
      v[k][0] = *reinterpret_cast<const half8_t*>(x + lo);
      v[k][1] = *reinterpret_cast<const half8_t*>(x + hi);
    }
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) {
      float y[16], sum = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        y[j] = (float)v[k][0][j];
        y[8 + j] = (float)v[k][1][j];
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) sum = __builtin_fmaf(y[j], y[j], sum);
      sum = norm_sum(mine ? sum : 0.f, lanes);
      const float r = __builtin_amdgcn_rsqf(__builtin_fmaf(sum, mean, norm.eps));
      if (!mine || i0 + k * threads >= all) continue;
#pragma unroll
      for (int j = 0; j < 16; ++j) y[j] = y[j] * r * w[j];
      if (turns) {
        float2 cs[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) cs[j] = table[tok[k] * half + unit * 8 + j];
        rope_turn(a.adjacent, cs, y);
      }
      half8_t o[2];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        o[0][j] = (_Float16)y[j];
        o[1][j] = (_Float16)y[8 + j];
      }
      _Float16* to = p.y + (int64_t)(token0 + tok[k]) * p.y_stride + at[k];
      *reinterpret_cast<half8_t*>(to + lo) = o[0];
      *reinterpret_cast<half8_t*>(to + hi) = o[1];
    }
  }
}

struct NormRopeParams : RopeParams {
  NormWeight norm;
};
__global__ __launch_bounds__(256) void norm_rope_kernel(NormRopeParams p) {
  __shared__ float2 table[kRopeTable];
  const int t0 = (int)blockIdx.x * p.tokens_per_wg;
  norm_rope_rows(p.rows, p.a, p.norm, t0, min(p.tokens_per_wg, p.a.total - t0), (int)threadIdx.x, 256, table);
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
struct KvAppendNormParams : KvAppendParams {
  NormWeight k_norm, q_norm;
};

// Four dwords of four bytes each, transposed.
__device__ __forceinline__ void kv_transpose4(const uint32_t (&x)[4], uint32_t (&y)[4]) {
  const uint32_t a = __builtin_amdgcn_perm(x[1], x[0], 0x05010400u), b = __builtin_amdgcn_perm(x[1], x[0], 0x07030602u);
  const uint32_t c = __builtin_amdgcn_perm(x[3], x[2], 0x05010400u), d = __builtin_amdgcn_perm(x[3], x[2], 0x07030602u);
  y[0] = __builtin_amdgcn_perm(c, a, 0x05040100u);
  y[1] = __builtin_amdgcn_perm(c, a, 0x07060302u);
  y[2] = __builtin_amdgcn_perm(d, b, 0x05040100u);
  y[3] = __builtin_amdgcn_perm(d, b, 0x07060302u);
}

// One workgroup per (page, head) that new tokens lie in.  2 * D threads take
// PER of the page's four blocks, the first D of them K and the others V; a
// thread holds one unit of one token of each: all loads first, then the
// largest values of the blocks (one exchange through LDS), then the codes,
// which go through LDS to be written in page order.  The angles of a unit are
// formed by the thread that turns it, from frequencies and positions in LDS.
// Long calls are bound by HBM, short ones by the chain of latencies from the
// table to the page.  Measured, 8 heads of 128 and q of 48: 4093 tokens 30 us
// (4.2 TB/s), one token each of 32 sequences 7.7 us.
// NORM: a token's units lie on D / 16 threads side by side; where D is 192 they
// may be of two waves, and the sums of squares are exchanged through LDS ahead
// of the barrier that the angles' table needs anyway.  k's weights lie in LDS: a
// thread holds four tokens in registers already (weights in registers too: 35.4 us
// for 28.3).  Measured in a captured run, 8 heads of 128 and q of 48: 4093
// tokens 27.4 us (without norms 24.6), one token each of 32 sequences 7.7 (6.8).
template <int PER, bool NORM = false>
__global__ __launch_bounds__(PER == 4 ? 512 : 1024) void kv_append_kernel(
    std::conditional_t<NORM, KvAppendNormParams, KvAppendParams> p) {
  __shared__ float red[2][kKvBlocks][4];
  __shared__ __align__(16) uint8_t codes[2][kKvPage * 256];
  __shared__ RopeFreq freq[128];
  __shared__ int axis[128], pos[BQ_ROPE_MAX_AXES][kKvPage];
  __shared__ __align__(16) float weight[NORM ? 256 : 1];
  const int D = p.head_dim, units = D >> 4;
  if ((int)blockIdx.x >= p.items) {
    const int t0 = ((int)blockIdx.x - p.items) * p.q_tokens_per_wg;
    if constexpr (NORM) {
      if (p.q_norm.w) {
        norm_rope_rows(p.q, p.a, p.q_norm, t0, min(p.q_tokens_per_wg, p.batch.total - t0), (int)threadIdx.x,
                       (int)blockDim.x, reinterpret_cast<float2*>(codes));
        return;
      }
    }
    rope_rows(p.q, p.a, t0, min(p.q_tokens_per_wg, p.batch.total - t0), (int)threadIdx.x, (int)blockDim.x,
              reinterpret_cast<float2*>(codes));
    return;
  }
  const int item = (int)blockIdx.x / p.kv_heads, head = (int)blockIdx.x % p.kv_heads;
  KvSeq s;
  int b, local, first;
  if (!kv_locate(p.batch, item, [](const KvSeq& x) { int f; return kv_touched(x, f); }, s, b, local)) return;
  kv_touched(s, first);
  const int at = first + local;
  const int page = kv_page(p.batch, b, at);
  if (page < 0) return;
  const int start = max(s.len - s.n, 0), row0 = s.q0 - (s.len - s.n);  // row of token t: row0 + t
  const int part = (int)threadIdx.x / D, which = part & 1, tid = (int)threadIdx.x - part * D;
  const int i0 = (part >> 1) * PER;  // this thread's blocks: i0 .. i0 + PER - 1
  const int tok = tid / units, unit = tid - tok * units;
  const int wave = tid >> 6, waves = D >> 6;
  const int64_t head_at = (int64_t)page * p.kv_heads + head;
  uint8_t* dst = (which ? p.v : p.k) + head_at * kKvPage * D;
  float* scales = (which ? p.vs : p.ks) + head_at * kKvBlocks;
  const _Float16* src = which ? p.nv : p.nk;
  const int64_t stride = which ? p.nv_stride : p.nk_stride;
  // blocks with new tokens
  const int t00 = at * kKvPage;
  const int b0 = max(start - t00, 0) / kKvBlock, b1 = (min(s.len - t00, kKvPage) - 1) / kKvBlock + 1;
  int lo, hi;
  if (which) {
    lo = unit * 16;
    hi = lo + 8;
  } else {
    rope_unit_at(p.a, unit, lo, hi);
  }
  half8_t raw[PER][2];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int t = t00 + (i0 + i) * kKvBlock + tok;
    if (t < start || t >= s.len) continue;
    const _Float16* r = src + (int64_t)(row0 + t) * stride + head * D;
    raw[i][0] = *reinterpret_cast<const half8_t*>(r + lo);
    raw[i][1] = *reinterpret_cast<const half8_t*>(r + hi);
  }
  // what the first of these blocks holds of older tokens
  const bool older = t00 + b0 * kKvBlock < start, mine = t00 + b0 * kKvBlock + tok < start;
  const float held = older ? scales[b0] : 0.f;
  uint32_t old[4];
  if (older && mine && b0 >= i0 && b0 < i0 + PER) {
    const int in = b0 * kKvBlock + tok;
    if (which) {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const uint32_t c = dst[kv_v_at(in, lo + j)];
        old[j >> 2] = j & 3 ? old[j >> 2] | (c << (8 * (j & 3))) : c;
      }
    } else {
      const uint2 w0 = *reinterpret_cast<const uint2*>(dst + kv_k_at(in, lo, D));
      const uint2 w1 = *reinterpret_cast<const uint2*>(dst + kv_k_at(in, hi, D));
      old[0] = w0.x, old[1] = w0.y, old[2] = w1.x, old[3] = w1.y;
    }
  }
  const bool turns = !which && unit < (p.a.rot >> 4);
  [[maybe_unused]] float root[PER];  // a token's sum of squares
  [[maybe_unused]] float(*squares)[kKvBlock][17] = nullptr;  // [block][token][unit], in LDS that the codes take later
  [[maybe_unused]] bool norms = false;
  if constexpr (NORM) {
    norms = !which && p.k_norm.w;
    squares = reinterpret_cast<float(*)[kKvBlock][17]>(&codes[1][0]);
    if (p.k_norm.w)
      for (int i = (int)threadIdx.x; i < D; i += (int)blockDim.x) weight[i] = p.k_norm.w[i];
    if (norms) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int t = t00 + (i0 + i) * kKvBlock + tok;
        const bool fresh = t >= start && t < s.len;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float a = (float)raw[i][0][j], b = (float)raw[i][1][j];
          sum = __builtin_fmaf(a, a, __builtin_fmaf(b, b, sum));
        }
        if (units != 12) root[i] = norm_sum(fresh ? sum : 0.f, units);
        else if (fresh) squares[i0 + i][tok][unit] = sum;
      }
    }
  }
  if (p.a.rot > 0) {
    for (int i = (int)threadIdx.x; i < (p.a.rot >> 1); i += (int)blockDim.x) {
      freq[i] = rope_freq(p.a.inv_freq[i]);
      axis[i] = min(max(p.a.axis ? p.a.axis[i] : 0, 0), p.a.axes - 1);
    }
    for (int i = (int)threadIdx.x; i < p.a.axes * kKvPage; i += (int)blockDim.x) {
      const int t = t00 + i % kKvPage;
      if (t >= start && t < s.len) pos[i / kKvPage][i % kKvPage] = p.a.pos[(int64_t)(i / kKvPage) * p.a.total + row0 + t];
    }
  }
  __syncthreads();
  float x[PER][16];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (i0 + i < b0 || i0 + i >= b1) continue;
    const int in = (i0 + i) * kKvBlock + tok, t = t00 + in;
    float top = 0.f;
    if (t >= start && t < s.len) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[i][j] = (float)raw[i][0][j];
        x[i][8 + j] = (float)raw[i][1][j];
      }
      if constexpr (NORM) {
        if (norms) {
          float sum = root[i];
          if (units == 12) {
            sum = 0.f;
#pragma unroll
            for (int u = 0; u < 12; ++u) sum += squares[i0 + i][tok][u];
          }
          const float r = __builtin_amdgcn_rsqf(__builtin_fmaf(sum, 1.f / (float)D, p.k_norm.eps));
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const f32x4 w = *reinterpret_cast<const f32x4*>(&weight[j < 8 ? lo + j : hi + j - 8]);
#pragma unroll
            for (int k = 0; k < 4; ++k) x[i][j + k] = x[i][j + k] * r * w[k];
          }
        }
      }
      if (turns) {
        float2 cs[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) rope_cos_sin(freq[unit * 8 + j], pos[axis[unit * 8 + j]][in], cs[j].x, cs[j].y);
        rope_turn(p.a.adjacent, cs, x[i]);
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float m = __builtin_fabsf(x[i][j]);
        top = m < __builtin_inff() ? __builtin_fmaxf(top, m) : top;  // finite values only
      }
    } else {
      // an older token of the block, or none
#pragma unroll
      for (int j = 0; j < 16; ++j) x[i][j] = t < start ? kv_value(p.format, (old[j >> 2] >> (8 * (j & 3))) & 255u) : 0.f;
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, o, 64));
    if ((tid & 63) == 0) red[which][i0 + i][wave] = top;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (i0 + i < b0 || i0 + i >= b1) continue;
    const int in = (i0 + i) * kKvBlock + tok;
    float top = 0.f;
    for (int w = 0; w < waves; ++w) top = __builtin_fmaxf(top, red[which][i0 + i][w]);
    const float was = i0 + i == b0 ? held : 0.f;
    const float scale = __builtin_fmaxf(top / kv_qmax(p.format), was);
    const float mul = scale > 0.f ? (t00 + in < start ? was / scale : 1.f / scale) : 0.f;
    if (tid == 0) scales[i0 + i] = scale;
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
      const uint32_t w = kv_codes4(p.format, x[i][j] * mul, x[i][j + 1] * mul, x[i][j + 2] * mul, x[i][j + 3] * mul);
      *reinterpret_cast<uint32_t*>(&codes[which][in * D + (j < 8 ? lo + j : hi + j - 8)]) = w;
    }
  }
  __syncthreads();
  if (!which) {
    // 16 bytes a thread and block: (c, g, t)
    const int c = tid >> 6, g = (tid >> 4) & 3, tt = tid & 15;
    for (int i = max(b0, i0); i < min(b1, i0 + PER); ++i) {
      const uint4 w = *reinterpret_cast<const uint4*>(&codes[0][(i * kKvBlock + tt) * D + c * 64 + g * 16]);
      *reinterpret_cast<uint4*>(dst + ((i * units / 4 + c) * 64 + g * 16 + tt) * 16) = w;
    }
  } else if (i0 == 0) {
    // a thread takes four dimensions of the tokens 16i + 4g ..
    const int g = tid / (D >> 2), dim = (tid - g * (D >> 2)) * 4;
    uint32_t out[4][kKvBlocks];
#pragma unroll
    for (int i = 0; i < kKvBlocks; ++i) {
      if (i < b0 || i >= b1) continue;
      uint32_t w[4], y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = *reinterpret_cast<const uint32_t*>(&codes[1][(i * kKvBlock + 4 * g + j) * D + dim]);
      kv_transpose4(w, y);
#pragma unroll
      for (int d = 0; d < 4; ++d) out[d][i] = y[d];
    }
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      uint8_t* to = dst + kv_v_at(4 * g, dim + d);
      if (b0 == 0 && b1 == kKvBlocks) {
        *reinterpret_cast<uint4*>(to) = make_uint4(out[d][0], out[d][1], out[d][2], out[d][3]);
      } else {
#pragma unroll
        for (int i = 0; i < kKvBlocks; ++i)
          if (i >= b0 && i < b1) *reinterpret_cast<uint32_t*>(to + 4 * i) = out[d][i];
      }
    }
  }
}

struct KvReadParams {
  const uint8_t *k, *v;
  const float *ks, *vs;
  _Float16 *ok, *ov;  // [total][kv_heads][D]
  KvBatch batch;
  int kv_heads, head_dim, format;
};

// Sixteen codes' values as fp16.
__device__ __forceinline__ void kv_put16(int format, const uint4& c, float scale, _Float16* dst) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  half8_t o[2];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    half2_t a, b;
    if (format == BQ_KV_I8) kv_half4<BQ_KV_I8>(w[j], a, b);
    else kv_half4<BQ_KV_E4M3>(w[j], a, b);
    o[j >> 1][(j & 1) * 4] = (_Float16)((float)a.x * scale);
    o[j >> 1][(j & 1) * 4 + 1] = (_Float16)((float)a.y * scale);
    o[j >> 1][(j & 1) * 4 + 2] = (_Float16)((float)b.x * scale);
    o[j >> 1][(j & 1) * 4 + 3] = (_Float16)((float)b.y * scale);
  }
  reinterpret_cast<half8_t*>(dst)[0] = o[0];
  reinterpret_cast<half8_t*>(dst)[1] = o[1];
}

// One workgroup per (page, head) that the last tokens of a sequence lie in.
// K's 16-byte units are 16 dimensions of a token and go straight to their
// row; V's are four tokens of each block, turned into rows through LDS.
// Tokens that no page holds are written as zeros.  Bound by HBM once it fills
// the chip.  Measured: 4096 tokens of 8 heads of 128 8.4 us (3 TB/s).
__global__ __launch_bounds__(256) void kv_read_kernel(KvReadParams p) {
  __shared__ __align__(16) uint8_t rows[kKvPage * 256];
  const int D = p.head_dim, units = D >> 4;
  const int item = (int)blockIdx.x / p.kv_heads, head = (int)blockIdx.x % p.kv_heads;
  KvSeq s;
  int b, local, first;
  // a sequence shorter than its rows: its first rows are zeros, one item more
  const auto count = [](const KvSeq& x) {
    int f;
    return kv_touched(x, f) + (x.n > x.len ? 1 : 0);
  };
  if (!kv_locate(p.batch, item, count, s, b, local)) return;
  const int pages = kv_touched(s, first);
  if (local == pages) {
    // by rows: 2 units of each are more than 31 bits count
    const int at_once = 256 / (2 * units), first_row = (int)threadIdx.x / (2 * units);
    const int in = (int)threadIdx.x - first_row * 2 * units, which = in & 1, u = in >> 1;
    if (first_row >= at_once) return;
    for (int row = first_row; row < s.n - s.len; row += at_once) {
      half8_t* o = reinterpret_cast<half8_t*>((which ? p.ov : p.ok) + ((int64_t)(s.q0 + row) * p.kv_heads + head) * D + u * 16);
      o[0] = o[1] = half8_t{};
    }
    return;
  }
  const int at = first + local, page = kv_page(p.batch, b, at);
  const int64_t head_at = (int64_t)max(page, 0) * p.kv_heads + head;
  const uint4* k = reinterpret_cast<const uint4*>(p.k + head_at * kKvPage * D);
  const u32x4_t* v = reinterpret_cast<const u32x4_t*>(p.v + head_at * kKvPage * D);
  const int t0 = max(s.len - s.n - at * kKvPage, 0), t1 = min(s.len - at * kKvPage, kKvPage);
  const int64_t row0 = s.q0 + at * kKvPage - (s.len - s.n);  // row of the page's token t: row0 + t
  // K's units and the scales are requested ahead of V, D / 64 a thread
  const int all = (t1 - t0) * units;  // at least one: the page holds some of the rows
  uint4 kc[4];
  float ks[4], vs[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j * 64 >= D) continue;
    const int i = min((int)threadIdx.x + j * 256, all - 1), t = t0 + i / units;
    kc[j] = k[kv_k_at(t, i % units * 16, D) >> 4];
    ks[j] = p.ks[head_at * kKvBlocks + t / kKvBlock];
    vs[j] = p.vs[head_at * kKvBlocks + t / kKvBlock];
  }
  for (int i = (int)threadIdx.x; i < D; i += 256) {
    // four dimensions (dim ..) of the tokens 16i + 4g ..
    const int g = i / (D >> 2), dim = (i - g * (D >> 2)) * 4;
    u32x4_t c[4];
#pragma unroll
    for (int d = 0; d < 4; ++d) c[d] = v[kv_v_at(4 * g, dim + d) >> 4];
#pragma unroll
    for (int blk = 0; blk < kKvBlocks; ++blk) {
      const uint32_t w[4] = {c[0][blk], c[1][blk], c[2][blk], c[3][blk]};
      uint32_t y[4];
      kv_transpose4(w, y);
#pragma unroll
      for (int j = 0; j < 4; ++j) *reinterpret_cast<uint32_t*>(&rows[(blk * kKvBlock + 4 * g + j) * D + dim]) = y[j];
    }
  }
  __syncthreads();
  const uint32_t zero = p.format == BQ_KV_I8 ? 0x80808080u : 0u;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int i = (int)threadIdx.x + j * 256;
    if (i >= all) break;
    const int t = t0 + i / units, u = i % units;
    const int64_t to = ((row0 + t) * p.kv_heads + head) * D + u * 16;
    uint4 vc = *reinterpret_cast<const uint4*>(&rows[t * D + u * 16]);
    if (page < 0) {
      kc[j] = vc = make_uint4(zero, zero, zero, zero);
      ks[j] = vs[j] = 0.f;
    }
    kv_put16(p.format, kc[j], ks[j], p.ok + to);
    kv_put16(p.format, vc, vs[j], p.ov + to);
  }
}

}  // namespace bq
