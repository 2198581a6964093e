// Attention over the paged 8-bit cache.
//
//   o[r] = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale * q[r].k_j - max_j)
// over the tokens j that row r sees.  k_j = sk * code with sk constant over a
// block of 16 tokens, so the scale is taken out of the dot product; likewise
// p_j v_j = (p_j sv) * code.  Codes enter the matrix cores as fp16, exactly;
// scores, probabilities' sums and outputs are held in fp32; the probabilities
// are rounded to fp16 (nearest even) for the second product.
//
// The `group` query heads that share a key/value head and the tokens of a
// sequence's rows form one list of rows (token-major), taken 16 at a time as
// the columns of both products:
//   S^T [64 tokens][16 rows] = K [64][D] x Q^T,   O^T [D][16] += V^T [D][64] x P^T.
#pragma once

#include "kv_common.hpp"

namespace bq {

struct KvAttnParams {
  const uint8_t *k, *v;  // the layer's codes and scales
  const float *ks, *vs;
  const _Float16* q;
  _Float16* out;
  int64_t q_stride, out_stride;
  KvBatch batch;
  int kv_heads, group, causal, window;
  float scale;           // softmax scale * log2(e)
  unsigned* counters;    // workspace: parts done of each tile, zero between calls
  float* part;           // workspace: partial results
  int target;            // workgroups of a head to aim at; 0: tiles are not split
  int min_pages;         // pages of a part, at least
};

constexpr int kKvMaxParts = 256;

__device__ __forceinline__ float kv_exp2(float x) { return __builtin_amdgcn_exp2f(x); }

// max / sum over the four lanes of a column (lanes l, l ^ 16, l ^ 32, l ^ 48)
__device__ __forceinline__ float kv_col_max(float x) {
  x = __builtin_fmaxf(x, __shfl_xor(x, 16, 64));
  return __builtin_fmaxf(x, __shfl_xor(x, 32, 64));
}
__device__ __forceinline__ float kv_col_sum(float x) {
  x += __shfl_xor(x, 16, 64);
  return x + __shfl_xor(x, 32, 64);
}

// Values that other workgroups read: stores and loads at device scope, which
// do not stay in one XCD's L2.
__device__ __forceinline__ void kv_put2(float* p, float a, float b) {
  const uint64_t w = (uint64_t)__builtin_bit_cast(uint32_t, a) | ((uint64_t)__builtin_bit_cast(uint32_t, b) << 32);
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p), w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2 kv_get2(const float* p) {
  const uint64_t w =
      __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return make_float2(__builtin_bit_cast(float, (uint32_t)w), __builtin_bit_cast(float, (uint32_t)(w >> 32)));
}

// One workgroup's share: a tile of ROWS rows of one sequence, part `split` of
// `parts` of the pages that the tile sees.
struct KvWork {
  int b, tile, split, parts;
};
__device__ __forceinline__ int kv_first_page(const KvAttnParams& p, const KvSeq& s) {
  return p.causal && p.window > 0 ? max(s.len - s.n - p.window + 1, 0) / kKvPage : 0;
}
template <int ROWS>
__device__ __forceinline__ bool kv_attn_work(const KvAttnParams& p, int item, KvWork& w) {
  const auto pages = [&](const KvSeq& s) {
    return max((s.len + kKvPage - 1) / kKvPage - kv_first_page(p, s), 1);
  };
  const auto tiles = [&](const KvSeq& s) { return (s.n * p.group + ROWS - 1) / ROWS; };
  int chunk = 0x7FFFFFFF;
  if (p.target > 0) {
    // pages of a part: the batch's tiles times pages over the target, so a
    // long sequence gets as many more parts as it has more pages
    long long all = 0;
    for (int i = (int)(threadIdx.x & 63); i < p.batch.batch; i += 64) {
      const KvSeq s = kv_seq(p.batch, i);
      all += (long long)tiles(s) * pages(s);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) all += __shfl_xor(all, o, 64);
    chunk = (int)min(max((all + p.target - 1) / p.target, (long long)p.min_pages), (long long)0x7FFFFFFF);
  }
  const auto parts = [&](const KvSeq& s) {
    return p.target > 0 ? min((pages(s) + chunk - 1) / chunk, kKvMaxParts) : 1;
  };
  int local;
  if (!kv_locate(item, p.batch.batch, [&](int i) { const KvSeq s = kv_seq(p.batch, i); return tiles(s) * parts(s); },
                 w.b, local))
    return false;
  w.parts = __builtin_amdgcn_readfirstlane(parts(kv_seq(p.batch, w.b)));
  w.tile = local / w.parts;
  w.split = local - w.tile * w.parts;
  return true;
}

// Rows 16t + l % 16 of a tile: the tokens each sees are [lo, hi).
struct KvRowRange {
  int lo, hi;
};
__device__ __forceinline__ KvRowRange kv_row_range(const KvAttnParams& p, const KvSeq& s, int token) {
  KvRowRange r;
  const int pos = s.len - s.n + token;
  r.hi = p.causal ? max(pos + 1, 0) : s.len;
  r.lo = p.causal && p.window > 0 ? max(pos - p.window + 1, 0) : 0;
  return r;
}

// Floats of a part's partial result: (max, sum) of each row, then O [ROWS][D].
__host__ __device__ constexpr int kv_part_floats(int rows, int D) { return rows * (D + 2); }

// Few rows: four waves share a part's pages (every fourth), each with its own
// running maximum and sum; they are joined through LDS, and the parts of a
// tile by the workgroup that finishes last.
template <int D, int FMT, int RT>
__global__ __launch_bounds__(256) void kv_attn_rows_kernel(KvAttnParams p) {
  constexpr int C = D / 64, N = D / 16, ROWS = 16 * RT;
  __shared__ __align__(16) float lds[2 * 64 * RT * (4 * N + 2) > 2 * kKvMaxParts * ROWS ? 2 * 64 * RT * (4 * N + 2)
                                                                                     : 2 * kKvMaxParts * ROWS];
  __shared__ int last;
  const int lane = (int)threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int item = (int)blockIdx.x, head = (int)blockIdx.y;
  KvWork w;
  if (!kv_attn_work<ROWS>(p, item, w)) return;
  KvSeq s = kv_seq(p.batch, w.b);
  s.q0 = __builtin_amdgcn_readfirstlane(s.q0);
  s.n = __builtin_amdgcn_readfirstlane(s.n);
  s.len = __builtin_amdgcn_readfirstlane(s.len);
  const int rows = s.n * p.group, row0 = w.tile * ROWS;

  // Q as the B operand: column r, k = dims 64c + 16g + 8h .. + 7
  half8_t q[RT][2 * C];
  int lo[RT], hi[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int row = row0 + 16 * t + r;
    const bool ok = row < rows;
    const int token = ok ? row / p.group : 0, qh = head * p.group + (ok ? row - token * p.group : 0);
    const KvRowRange range = kv_row_range(p, s, token);
    lo[t] = range.lo;
    hi[t] = ok ? range.hi : 0;
    const _Float16* src = p.q + (int64_t)(s.q0 + token) * p.q_stride + qh * D + 16 * g;
#pragma unroll
    for (int c = 0; c < 2 * C; ++c)
      q[t][c] = ok ? *reinterpret_cast<const half8_t*>(src + (c >> 1) * 64 + (c & 1) * 8) : half8_t{};
  }
  // the tile's pages, and the tokens that all its rows see
  const int tok0 = row0 / p.group, tok1 = min((row0 + ROWS - 1) / p.group, s.n - 1);
  const KvRowRange r0 = kv_row_range(p, s, tok0), r1 = kv_row_range(p, s, tok1);
  const int pa = r0.lo / kKvPage, pages = max((r1.hi + kKvPage - 1) / kKvPage - pa, 0);
  const int begin = pa + (int)((int64_t)pages * w.split / w.parts);
  const int end = pa + (int)((int64_t)pages * (w.split + 1) / w.parts);

  f32x4 o[RT][N];
  float m[RT], l[RT];
  float R = 0x1p-100f, invR = 0x1p100f;  // o is in units of R, a power of two near the largest scale of V so far
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    m[t] = -__builtin_inff();
    l[t] = 0.f;
#pragma unroll
    for (int n = 0; n < N; ++n) o[t][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  for (int at = begin + wave; at < end; at += 4) {
    const int page = kv_page(p.batch, w.b, at);
    if (page < 0) continue;
    const int64_t head_at = (int64_t)page * p.kv_heads + head;
    const u32x4_t* kp = reinterpret_cast<const u32x4_t*>(p.k + head_at * (kKvPage * D)) + lane;
    const u32x4_t* vp = reinterpret_cast<const u32x4_t*>(p.v + head_at * (kKvPage * D)) + lane;
    u32x4_t kr[4][C], vr[N];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < C; ++c) kr[i][c] = kp[(i * C + c) * 64];
#pragma unroll
    for (int n = 0; n < N; ++n) vr[n] = vp[n * 64];
    float sk[4], sv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sk[i] = p.ks[head_at * kKvBlocks + i];
      sv[i] = p.vs[head_at * kKvBlocks + i];
    }
    const int j0 = at * kKvPage, left = s.len - j0;  // tokens of the page that are held
    if (left < kKvPage) {
      // what lies past the length is never used: neither a scale nor, in
      // e4m3, a code that is no number
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (16 * i >= left) sv[i] = 0.f;
        if constexpr (FMT == BQ_KV_E4M3) {
          const int keep = min(max(left - 16 * i - 4 * g, 0), 4);
          const uint32_t mask = keep == 4 ? 0xFFFFFFFFu : (1u << (8 * keep)) - 1u;
#pragma unroll
          for (int n = 0; n < N; ++n) vr[n][i] &= mask;
        }
      }
    }

    // scores, in units of log2
    f32x4 x[RT][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int t = 0; t < RT; ++t) x[t][i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const half8_t a0 = kv_half8<FMT>(kr[i][c][0], kr[i][c][1]), a1 = kv_half8<FMT>(kr[i][c][2], kr[i][c][3]);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          x[t][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a0, q[t][2 * c], x[t][i], 0, 0, 0);
          x[t][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a1, q[t][2 * c + 1], x[t][i], 0, 0, 0);
        }
      }
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = j0 + 16 * i + 4 * g + e;
          const float y = x[t][i][e] * (sk[i] * p.scale);
          x[t][i][e] = j >= lo[t] && j < hi[t] ? y : -__builtin_inff();
        }
    }

    // running maximum and units of o
    const float rmax = __builtin_fmaxf(__builtin_fmaxf(sv[0], sv[1]), __builtin_fmaxf(sv[2], sv[3]));
    float change = 1.f;
    if (rmax > R) {
      float up = R;
      const int ex = (int)((__builtin_bit_cast(uint32_t, rmax) >> 23) & 255u) + 1;  // the power of two above rmax
      up = __builtin_bit_cast(float, (uint32_t)min(ex, 253) << 23);
      change = R / up;
      R = up;
      invR = 1.f / up;
    }
    half8_t pb[RT][2];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      float mx = -__builtin_inff();
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) mx = __builtin_fmaxf(mx, x[t][i][e]);
      const float mn = __builtin_fmaxf(m[t], kv_col_max(mx));
      const float base = mn == -__builtin_inff() ? 0.f : mn;  // a row that has seen nothing yet
      const float alpha = kv_exp2(m[t] - base);
      m[t] = mn;
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float e2 = kv_exp2(x[t][i][e] - base);
          sum += e2;
          pb[t][i >> 1][(i & 1) * 4 + e] = (_Float16)(e2 * (sv[i] * invR));
        }
      l[t] = l[t] * alpha + sum;
#pragma unroll
      for (int n = 0; n < N; ++n) o[t][n] *= alpha * change;
    }
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const half8_t a = kv_half8<FMT>(vr[n][2 * h], vr[n][2 * h + 1]);
#pragma unroll
        for (int t = 0; t < RT; ++t) o[t][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, pb[t][h], o[t][n], 0, 0, 0);
      }
  }

  // o in its own units, the sum over a column's four lanes
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    l[t] = kv_col_sum(l[t]);
#pragma unroll
    for (int n = 0; n < N; ++n) o[t][n] *= R;
  }
  // waves 2, 3 into 0, 1, then 1 into 0
#pragma unroll
  for (int step = 2; step >= 1; step >>= 1) {
    float* box = lds + (wave & (step - 1)) * (64 * RT * (4 * N + 2));
    if (wave >= step && wave < 2 * step) {
#pragma unroll
      for (int t = 0; t < RT; ++t) {
#pragma unroll
        for (int n = 0; n < N; ++n) *reinterpret_cast<f32x4*>(box + ((t * N + n) * 64 + lane) * 4) = o[t][n];
        box[(RT * N * 4 + 2 * t) * 64 + lane] = m[t];
        box[(RT * N * 4 + 2 * t + 1) * 64 + lane] = l[t];
      }
    }
    __syncthreads();
    if (wave < step) {
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const float m2 = box[(RT * N * 4 + 2 * t) * 64 + lane], l2 = box[(RT * N * 4 + 2 * t + 1) * 64 + lane];
        const float mn = __builtin_fmaxf(m[t], m2), base = mn == -__builtin_inff() ? 0.f : mn;
        const float a1 = kv_exp2(m[t] - base), a2 = kv_exp2(m2 - base);
        m[t] = mn;
        l[t] = l[t] * a1 + l2 * a2;
#pragma unroll
        for (int n = 0; n < N; ++n)
          o[t][n] = o[t][n] * a1 + *reinterpret_cast<const f32x4*>(box + ((t * N + n) * 64 + lane) * 4) * a2;
      }
    }
    __syncthreads();
  }

  if (w.parts == 1) {
    if (wave == 0) {
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const int row = row0 + 16 * t + r;
        if (row >= rows) continue;
        const int token = row / p.group, qh = head * p.group + row - token * p.group;
        const float inv = l[t] > 0.f ? 1.f / l[t] : 0.f;  // nothing seen: zeros
        _Float16* dst = p.out + (int64_t)(s.q0 + token) * p.out_stride + qh * D + 4 * g;
#pragma unroll
        for (int n = 0; n < N; ++n) {
          const f32x4 y = o[t][n] * inv;
          *reinterpret_cast<half4_t*>(dst + 16 * n) =
              half4_t{(_Float16)y[0], (_Float16)y[1], (_Float16)y[2], (_Float16)y[3]};
        }
      }
    }
    return;
  }

  // The part's result goes to its slot; the workgroup that counts last joins
  // the tile's parts, in order (the same result on every call).
  constexpr int SLOT = kv_part_floats(ROWS, D);
  float* tile_part = p.part + ((int64_t)(item - w.split) * p.kv_heads + head) * SLOT;
  const int64_t next = (int64_t)p.kv_heads * SLOT;
  unsigned* counter = p.counters + (int64_t)(item - w.split) * p.kv_heads + head;
  if (wave == 0) {
    float* mine = tile_part + w.split * next;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int row = 16 * t + r;
      if (row0 + row >= rows) continue;
      if (g == 0) kv_put2(mine + 2 * row, m[t], l[t]);
      float* dst = mine + 2 * ROWS + row * D + 4 * g;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        kv_put2(dst + 16 * n, o[t][n][0], o[t][n][1]);
        kv_put2(dst + 16 * n + 2, o[t][n][2], o[t][n][3]);
      }
    }
    // the stores are performed at device scope before the count is
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    if (lane == 0)
      last = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (unsigned)(w.parts - 1);
  }
  __syncthreads();
  if (!last) return;
  const int some = min(ROWS, rows - row0);
  float *wm = lds, *wl = lds + kKvMaxParts * ROWS;
  for (int i = (int)threadIdx.x; i < w.parts * ROWS; i += 256) {
    const int part = i / ROWS, row = i % ROWS;
    float2 ml = make_float2(-__builtin_inff(), 0.f);
    if (row < some) ml = kv_get2(tile_part + part * next + 2 * row);
    wm[i] = ml.x;
    wl[i] = ml.y;
  }
  __syncthreads();
  {
    constexpr int PER = 256 / ROWS;  // consecutive lanes of a row
    const int row = (int)threadIdx.x / PER, sub = (int)threadIdx.x % PER;
    float mx = -__builtin_inff(), sum = 0.f;
    for (int i = sub; i < w.parts; i += PER) mx = __builtin_fmaxf(mx, wm[i * ROWS + row]);
#pragma unroll
    for (int d = PER / 2; d > 0; d >>= 1) mx = __builtin_fmaxf(mx, __shfl_xor(mx, d, 64));
    const float base = mx == -__builtin_inff() ? 0.f : mx;
    for (int i = sub; i < w.parts; i += PER) sum += wl[i * ROWS + row] * kv_exp2(wm[i * ROWS + row] - base);
#pragma unroll
    for (int d = PER / 2; d > 0; d >>= 1) sum += __shfl_xor(sum, d, 64);
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    for (int i = sub; i < w.parts; i += PER) wm[i * ROWS + row] = kv_exp2(wm[i * ROWS + row] - base) * inv;
  }
  __syncthreads();
  for (int i = (int)threadIdx.x; i < some * (D / 2); i += 256) {
    const int row = i / (D / 2), d2 = i % (D / 2);
    float a = 0.f, b = 0.f;
#pragma unroll 8
    for (int part = 0; part < w.parts; ++part) {
      const float2 v = kv_get2(tile_part + part * next + 2 * ROWS + row * D + 2 * d2);
      const float f = wm[part * ROWS + row];
      a += v.x * f;
      b += v.y * f;
    }
    const int token = (row0 + row) / p.group, qh = head * p.group + row0 + row - token * p.group;
    *reinterpret_cast<half2_t*>(p.out + (int64_t)(s.q0 + token) * p.out_stride + qh * D + 2 * d2) =
        half2_t{(_Float16)a, (_Float16)b};
  }
  if (threadIdx.x == 0) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

}  // namespace bq
