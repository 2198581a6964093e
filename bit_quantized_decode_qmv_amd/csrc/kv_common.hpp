// Shared pieces of the paged 8-bit key/value cache kernels: the layout of a
// page, code conversion, the rotary angle, and the mapping from a workgroup's
// index to a sequence of the batch.
//
// A page holds 64 tokens of one head.  Its codes are stored in the order in
// which a wave takes them as the A operand of v_mfma_f32_16x16x32_f16
// (lane l: row l % 16, eight consecutive k of group l / 16):
//   K  [i: 4][c: D/64][g: 4][t: 16][j: 16]  token 16i + t, dim 64c + 16g + j
//   V  [n: D/16][g: 4][d: 16][i: 4][j: 4]   token 16i + 4g + j, dim 16n + d
// so a 16-byte load per lane reads 1 KB of consecutive bytes, a lane's 16
// bytes are its operands of two matrix instructions, and the tokens of a V
// operand are those that the lane already holds of the score tile (C layout:
// row 4g + e, column l % 16): the probabilities go from the first product to
// the second without leaving their lane.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bq.h"

namespace bq {

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half4_t __attribute__((ext_vector_type(4)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kKvPage = BQ_KV_PAGE;    // tokens of a page
constexpr int kKvBlock = BQ_KV_BLOCK;  // tokens that share a scale
constexpr int kKvBlocks = kKvPage / kKvBlock;

__device__ __forceinline__ int kv_k_at(int token, int dim, int D) {
  return ((((token >> 4) * (D >> 6) + (dim >> 6)) * 4 + ((dim >> 4) & 3)) * 16 + (token & 15)) * 16 + (dim & 15);
}
__device__ __forceinline__ int kv_v_at(int token, int dim) {
  return ((((dim >> 4) * 4 + ((token >> 2) & 3)) * 16 + (dim & 15)) * 4 + (token >> 4)) * 4 + (token & 3);
}

// Four codes of a dword as fp16, exactly: an int8 code is held as the byte
// code + 128, which under the exponent byte 0x64 is the fp16 1024 + byte;
// every e4m3 number is an fp16 number.
template <int FMT>
__device__ __forceinline__ void kv_half4(uint32_t w, half2_t& lo, half2_t& hi) {
  if constexpr (FMT == BQ_KV_I8) {
    const half2_t off = {(_Float16)-1152.f, (_Float16)-1152.f};
    lo = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, w, 0x04010400u)) + off;
    hi = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, w, 0x04030402u)) + off;
  } else {
    lo = __builtin_bit_cast(half2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false));
    hi = __builtin_bit_cast(half2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true));
  }
}

template <int FMT>
__device__ __forceinline__ half8_t kv_half8(uint32_t a, uint32_t b) {
  half2_t x0, x1, y0, y1;
  kv_half4<FMT>(a, x0, x1);
  kv_half4<FMT>(b, y0, y1);
  return half8_t{x0.x, x0.y, x1.x, x1.y, y0.x, y0.y, y1.x, y1.y};
}

// Codes as operands of the matrix cores.  BYTES: the byte of an int8 code,
// code + 128, is as it stands the fp16 subnormal (code + 128) 2^-24, which the
// matrix cores take exactly; the product with 128 2^-24 is taken off the sums.
// That is two byte permutes for four codes, where the codes themselves cost
// two additions more.  Sums of V's bytes grow with all probabilities while
// those of its codes average out, so what the offset adds is taken off every
// few pages, not only at the end: every 64 pages of many rows, where it is
// done with the look at the maximum, and every 16 of a wave's pages of few
// rows.  Even weights over 131072 tokens, many rows: error 0.031% of the
// outputs (0.028% of it the rounding of probabilities and results), and 0.40%
// with one subtraction at the end; over 1048576 tokens 0.033% and 5.4%, few
// rows 0.023% and 0.47%.
template <bool BYTES>
constexpr float kKvOffset = BYTES ? 0x1p-17f : 0.f;
template <bool BYTES>
constexpr float kKvUnit = BYTES ? 0x1p24f : 1.f;  // of the sums
constexpr int kKvOffsetPages = 64, kKvOffsetRowPages = 16;
template <int FMT, bool BYTES>
__device__ __forceinline__ half8_t kv_operand8(uint32_t a, uint32_t b) {
  if constexpr (BYTES) {
    const u32x4_t w = {__builtin_amdgcn_perm(0u, a, 0x0C010C00u), __builtin_amdgcn_perm(0u, a, 0x0C030C02u),
                       __builtin_amdgcn_perm(0u, b, 0x0C010C00u), __builtin_amdgcn_perm(0u, b, 0x0C030C02u)};
    return __builtin_bit_cast(half8_t, w);
  } else {
    return kv_half8<FMT>(a, b);
  }
}

// One code's value.
__device__ __forceinline__ float kv_value(int format, uint32_t byte) {
  if (format == BQ_KV_I8) return (float)((int)byte - 128);
  return (float)__builtin_bit_cast(half2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(byte, 1.0f, false)).x;
}

__host__ __device__ inline float kv_qmax(int format) { return format == BQ_KV_I8 ? 127.f : 448.f; }

// Four values, in units of their block's scale, as four code bytes (round to
// nearest even).  A value past the largest code (an infinity) saturates; a
// NaN becomes 0, so the cache holds numbers only.
__device__ __forceinline__ uint32_t kv_codes4(int format, float a, float b, float c, float d) {
  const float top = kv_qmax(format);
  a = a == a ? __builtin_fminf(__builtin_fmaxf(a, -top), top) : 0.f;
  b = b == b ? __builtin_fminf(__builtin_fmaxf(b, -top), top) : 0.f;
  c = c == c ? __builtin_fminf(__builtin_fmaxf(c, -top), top) : 0.f;
  d = d == d ? __builtin_fminf(__builtin_fmaxf(d, -top), top) : 0.f;
  if (format == BQ_KV_I8) {
    const uint32_t x = (uint32_t)((int)__builtin_rintf(a) + 128), y = (uint32_t)((int)__builtin_rintf(b) + 128);
    const uint32_t z = (uint32_t)((int)__builtin_rintf(c) + 128), w = (uint32_t)((int)__builtin_rintf(d) + 128);
    return x | (y << 8) | (z << 16) | (w << 24);
  }
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
}

// cos and sin of pos * inv_freq.  The angle is taken in turns, the product
// with inv_freq / (2 pi) held as a sum of two floats.  A product with the
// first is formed as fma(p, hi, -whole turns): the exact product less an
// integer, rounded once, so the fraction that goes to the hardware functions
// is good to about 2^-24 turns for text positions and to 2^-20 at 2^31.
struct RopeFreq {
  float hi, lo;  // inv_freq / (2 pi)
};
__device__ __forceinline__ RopeFreq rope_freq(float inv_freq) {
  constexpr float kHi = 0.15915494f, kLo = 6.4206382e-09f;  // 1 / (2 pi)
  RopeFreq f;
  f.hi = inv_freq * kHi;
  f.lo = __builtin_fmaf(inv_freq, kHi, -f.hi) + inv_freq * kLo;
  return f;
}
__device__ __forceinline__ void rope_cos_sin(RopeFreq f, int pos, float& c, float& s) {
  const float p1 = (float)(pos & ~4095), p0 = (float)(pos & 4095);  // both exact
  float t = __builtin_fmaf(p1, f.hi, -__builtin_rintf(p1 * f.hi)) + __builtin_fmaf(p0, f.hi, -__builtin_rintf(p0 * f.hi));
  t += __builtin_fmaf(p1, f.lo, p0 * f.lo);
  t -= __builtin_rintf(t);
  c = __builtin_amdgcn_cosf(t);
  s = __builtin_amdgcn_sinf(t);
}

// The sequences of a call, as every cache kernel reads them.  Values that do
// not fit the arrays are brought into range here, so that no address depends
// on them unchecked.
struct KvBatch {
  const int* cu;     // [batch + 1] first row of each sequence
  const int* lens;   // [batch] tokens held, the call's own included
  const int* table;  // [batch][max_pages]
  int batch, max_pages, num_pages, total;
};
struct KvSeq {
  int q0, n, len;  // first row, rows, tokens held
};
__device__ __forceinline__ KvSeq kv_seq(const KvBatch& p, int b) {
  KvSeq s;
  s.q0 = min(max(p.cu[b], 0), p.total);
  s.n = min(max(p.cu[b + 1], s.q0), p.total) - s.q0;
  s.len = min(max(p.lens[b], 0), p.max_pages * kKvPage);
  return s;
}
// Page id at a place of a sequence's table, or -1 when it is not a page.
__device__ __forceinline__ int kv_page(const KvBatch& p, int b, int at) {
  const int id = p.table[(int64_t)b * p.max_pages + at];
  return (unsigned)id < (unsigned)p.num_pages ? id : -1;
}
// Pages that the last n tokens of a sequence lie in, and the first of them.
__device__ __forceinline__ int kv_touched(const KvSeq& s, int& first) {
  const int start = max(s.len - s.n, 0);
  first = start / kKvPage;
  return s.n > 0 && s.len > 0 ? (s.len - 1) / kKvPage - first + 1 : 0;
}

// Inclusive prefix sums over a wave's lanes, in six adds of lanes nearby (data
// parallel primitives: shifts within rows of 16, then broadcasts across rows).
__device__ __forceinline__ int kv_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast:15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast:31 into rows 2 and 3
  return v;
}

// Item `item` of a list in which a sequence has count(sequence) items: the
// sequence, its number and the item's place among its own.  Called by whole
// waves, a lane a sequence; every lane gets the same (scalar) answer; false
// past the list's end.
template <typename Count>
__device__ __forceinline__ bool kv_locate(const KvBatch& p, int item, Count count, KvSeq& s, int& b, int& local) {
  const int lane = threadIdx.x & 63;
  for (int base = 0; base < p.batch; base += 64) {
    const KvSeq mine = base + lane < p.batch ? kv_seq(p, base + lane) : KvSeq{};
    const int c = base + lane < p.batch ? count(mine) : 0;
    const int sum = kv_scan(c);
    const int all = __builtin_amdgcn_readlane(sum, 63);
    if (item < all) {
      const int at = __builtin_ctzll(__ballot(sum > item));
      b = base + at;
      local = item - __builtin_amdgcn_readlane(sum - c, at);
      s.q0 = __builtin_amdgcn_readlane(mine.q0, at);
      s.n = __builtin_amdgcn_readlane(mine.n, at);
      s.len = __builtin_amdgcn_readlane(mine.len, at);
      return true;
    }
    item -= all;
  }
  return false;
}

inline bool kv_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Checks of a cache description shared by the entry points.
inline int kv_check_cache(const bq_kv_cache* c) {
  if (!c || !c->k || !c->v || !c->k_scales || !c->v_scales) return BQ_ERR_NULL;
  if (c->format != BQ_KV_I8 && c->format != BQ_KV_E4M3) return BQ_ERR_BITS;
  if (c->layers < 1 || c->layers > 4096 || c->num_pages < 1 || c->num_pages > BQ_KV_MAX_PAGES || c->kv_heads < 1 || c->kv_heads > 1024 ||
      (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 192 && c->head_dim != 256))
    return BQ_ERR_SHAPE;
  if (!kv_aligned(c->k, 16) || !kv_aligned(c->v, 16) || !kv_aligned(c->k_scales, 16) || !kv_aligned(c->v_scales, 16))
    return BQ_ERR_ALIGN;
  return BQ_OK;
}
inline size_t kv_head_bytes(const bq_kv_cache* c) { return (size_t)kKvPage * c->head_dim; }
inline size_t kv_layer_heads(const bq_kv_cache* c) { return (size_t)c->num_pages * c->kv_heads; }

inline int kv_check_batch(const int* cu, const int* lens, const int* table, int batch, int max_pages, int total) {
  if (!cu || !lens || !table) return BQ_ERR_NULL;
  if (batch < 1 || batch > (1 << 20) || max_pages < 1 || max_pages > (1 << 24) || total < 0 || total > (1 << 28))
    return BQ_ERR_SHAPE;
  if (!kv_aligned(cu, 4) || !kv_aligned(lens, 4) || !kv_aligned(table, 4)) return BQ_ERR_ALIGN;
  return BQ_OK;
}
// rows of 16-byte units: pointer and row stride
inline bool kv_rows_ok(const void* p, long long stride, int row) {
  return kv_aligned(p, 16) && stride % 8 == 0 && stride >= row;
}

inline int kv_launch(const void* fn, dim3 grid, dim3 block, size_t shmem, void* stream, void* params) {
  if ((uint64_t)grid.x * block.x > 0xFFFFFFFFu || grid.y > 65535) return BQ_ERR_SHAPE;
  void* args[] = {params};
  return hipLaunchKernel(fn, grid, block, args, shmem, static_cast<hipStream_t>(stream)) == hipSuccess ? BQ_OK
                                                                                                       : BQ_ERR_HIP;
}

}  // namespace bq
