// Attention over the paged 8-bit cache.
//
//   o[r] = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale * q[r].k_j - max_j)
// over the tokens j that row r sees.  k_j = sk * code with sk constant over a
// block of 16 tokens, so the scale is taken out of the dot product; likewise
// p_j v_j = (p_j sv) * code.  Codes enter the matrix cores as fp16, exactly;
// scores, probabilities' sums and outputs are held in fp32; how the
// probabilities enter the second product is said at each kernel.
//
// The `group` query heads that share a key/value head and the tokens of a
// sequence's rows form one list of rows (token-major), taken 16 at a time as
// the columns of both products:
//   S^T [64 tokens][16 rows] = K [64][D] x Q^T,   O^T [D][16] += V^T [D][64] x P^T.
//
// Two more kinds of rows share these kernels (KvAttnMore): a window with
// sinks, where a row sees the first `sinks` tokens beside those of its window,
// and a tree of drafted tokens, where the sequence's last n tokens are seen by
// a row as its bits say and the context ahead of them as by a window.  A tile
// then walks the pages of the sinks and those from its first window on, as one
// run of numbers; what differs between its rows is the masking of the pages
// that some row does not see whole: a row's 64 bits of such a page instead of
// one range.  They are instances of their own, since what the plain ones hold in
// registers all along leaves no room (rows<128, e4m3, 2> spilled 15 registers
// with both in one; of their own one instance spills, rows<128, int8, 2>: 4
// registers, 20 bytes a lane, where the plain one spills 1).  Measured, 48 heads
// over 8 of 128, int8 unless said: one token each of
// eight sequences, a window of 4096 and 4 sinks 20 us (3.4 TB/s: two or three
// pages a wave do not hide the start and the join), drafts of 5 rows of them 31;
// 2047 rows with a window of 1024 86 (0.60 PFLOP/s: 768 workgroups for the 512
// that run at once, and two pages of 18 seen in part); a tree of 5 rows over 1003
// tokens 15 and over 16384 27, of 32 sequences of 1024 to 16384 133 (4.3 TB/s), of
// 13 rows over 1003 tokens 14 (a chain of latencies and the join's launch), of 64
// over 131001 235 (0.87 PFLOP/s); 16 trees of 61 rows over 1024 to 16384 tokens
// with a window of 1024 and 4 sinks 65, without 335 (0.62 PFLOP/s); with lengths
// spread over their logarithm, in e4m3, 199 (0.69 PFLOP/s: parts of a few pages,
// the codes' conversion, and 16 us of the join).
#pragma once

#include <type_traits>

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
  int min_pages;         // of a part; 0: by the number of pages
  int item0;             // share of the launch's first workgroups
};

struct KvAttnMore : KvAttnParams {
  const uint64_t* mask;  // [total][words]: the rows of its sequence's tree that a row sees; null: causal
  int words, sinks;
};

constexpr int kKvMaxParts = 128;  // of a tile
constexpr int kKvOnePage = 16;    // pages of tiles whose parts may be a page each

// Probabilities enter the second product as fp16 numbers.  They are formed as
// 2^(score - maximum + kKvLift) and, between two looks at the maximum, grow to
// 2^15: all of fp16's range lies below them, so a term's steps end at 2^-31 of
// the largest one (V's scale included) and not at 2^-24.  Where one token has
// most of the weight and no value, the result is the sum of terms near 2^-20.
// Sums carry the same factor, so it leaves with the division.
constexpr float kKvLift = 7.f;

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

__device__ __forceinline__ float kv_max3(float a, float b, float c) {
  float d;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(b), "v"(c));  // (without quieting each operand first)
  return d;
}
// The larger of each half (fp16, not negative) of three dwords; a half that
// is no number stays so.
__device__ __forceinline__ uint32_t kv_pk_max3(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("v_pk_maximum3_f16 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(b), "v"(c));
  return d;
}
__device__ __forceinline__ float kv_min4(f32x4 x) {
  return __builtin_fminf(__builtin_fminf(x[0], x[1]), __builtin_fminf(x[2], x[3]));
}
__device__ __forceinline__ float kv_max4(f32x4 x) {
  return __builtin_fmaxf(__builtin_fmaxf(x[0], x[1]), __builtin_fmaxf(x[2], x[3]));
}

// The outputs are in units of R, a power of two that follows V's scales from
// page to page: a term is formed as probability times scale / R, and what is
// lost of it goes by R.  A page whose scales lie in R's range is taken as it
// is.  For any other R is fitted to it: above its largest scale, or, where the
// scales differ by more than 4, above the page's largest term and four times
// its smallest scale above 0.  So R is at most 64 times that scale, or twice
// that term, and a block of large values that no row attends to, or sees,
// takes no bits from the terms beside it, and none from later pages.
// low, top: the least and the largest of a page's scales / R.
__device__ __forceinline__ bool kv_in_unit(float low, float top) { return low >= 0x1p-6f && top <= 1.f; }
// R is held as its exponent, biased by 127.  Below the least one a scale's
// values are 0 in fp16, whatever their weight.
constexpr int kKvLeastUnit = 127 - 48;
__device__ __forceinline__ float kv_exp_float(int ex) { return __builtin_bit_cast(float, (uint32_t)ex << 23); }
// Fits R to a page whose scales are unit * R and whose largest term is 2^most
// * R.  Brings unit along; what o is multiplied by.
template <typename Most>
__device__ __forceinline__ float kv_fit_unit(f32x4& unit, float low, float top, Most most, int& ex) {
  if (__builtin_expect(__builtin_amdgcn_readfirstlane(top > 4.f * low), 0)) {
    low = top;  // of those that are not 0
#pragma unroll
    for (int i = 0; i < 4; ++i) low = unit[i] > 0.f ? __builtin_fminf(low, unit[i]) : low;
    top = __builtin_fminf(top, __builtin_fmaxf(4.f * low, __builtin_amdgcn_exp2f(most())));
  }
  const int above = (int)((__builtin_bit_cast(uint32_t, top) >> 23) & 255u) + 1 - 127, was = ex;
  ex = __builtin_amdgcn_readfirstlane(min(max(ex + above, kKvLeastUnit), 253));
  const float change = __builtin_ldexpf(1.f, was - ex);
  unit *= change;
  return change;
}
// max over a wave's lanes, by shifts within rows of 16 and broadcasts across
// rows (no lane addresses, which would be held all along the page loop)
template <int STEP, int ROWS>
__device__ __forceinline__ float kv_max_step(float x) {
  const int bits = __builtin_bit_cast(int, x);
  return __builtin_fmaxf(x, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(bits, bits, STEP, ROWS, 0xF, false)));
}
__device__ __forceinline__ float kv_wave_max(float x) {
  x = kv_max_step<0x111, 0xF>(x);  // row_shr:1
  x = kv_max_step<0x112, 0xF>(x);  // row_shr:2
  x = kv_max_step<0x114, 0xF>(x);  // row_shr:4
  x = kv_max_step<0x118, 0xF>(x);  // row_shr:8
  x = kv_max_step<0x142, 0xA>(x);  // row_bcast:15 into rows 1 and 3
  x = kv_max_step<0x143, 0xC>(x);  // row_bcast:31 into rows 2 and 3
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 63));
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

// One workgroup's share: part `split` of the `parts` of a tile (ROWS rows of
// one sequence); the parts of a tile are `chunk` pages each, the last one
// what is left.  The list of a head's shares has the whole parts of all tiles
// first and their last parts after them, so that no workgroup begins a long
// part when others are done.
struct KvWork {
  KvSeq s;
  int b, tile, split, parts, chunk;
  int slot;  // place of the tile's part 0 when the parts are kept tile by tile
};
// Pages of a sequence's tiles, at most.
__device__ __forceinline__ int kv_pages(const KvAttnParams& p, const KvSeq& s) {
  const int first = p.causal && p.window > 0 ? max(s.len - s.n - p.window + 1, 0) / kKvPage : 0;
  return max((s.len + kKvPage - 1) / kKvPage - first, 1);
}
__device__ __forceinline__ int kv_pages(const KvAttnMore& p, const KvSeq& s) {
  // (a row of a tree that sees none of it sees the whole window of the context)
  const int first = p.window > 0 ? max(s.len - s.n - p.window + (p.mask ? 0 : 1), 0) / kKvPage : 0;
  const int front = min((min(p.sinks, s.len) + kKvPage - 1) / kKvPage, first);
  return max((s.len + kKvPage - 1) / kKvPage - first + front, 1);
}
// Every wave of the grid finds its share from the batch's arrays: a lane
// takes a sequence (64 at a time; the first 64 stay in its registers).
// JOIN: share `item` is the last part of tile `item`.
template <int ROWS, bool JOIN = false, typename P>
__device__ __forceinline__ bool kv_attn_work(const P& p, int item, KvWork& w) {
  const int lane = (int)threadIdx.x & 63, batch = p.batch.batch;
  const auto pages = [&](const KvSeq& s) { return kv_pages(p, s); };
  const auto tiles = [&](const KvSeq& s) { return (s.n * p.group + ROWS - 1) / ROWS; };
  // Offsets that fall would make the list longer than the launch and the
  // workspace are made for: then there is no work.
  bool falls = false;
  const auto load = [&](int b) {
    if (b >= batch) return KvSeq{};
    falls = falls || p.batch.cu[b + 1] < p.batch.cu[b];
    return kv_seq(p.batch, b);
  };
  const KvSeq first = load(lane);
  const auto seq = [&](int base) { return base == 0 ? first : load(base + lane); };
  w.chunk = 0x7FFFFFFF;
  if (p.target > 0) {
    // the batch's tiles times pages over the target: a long sequence gets as
    // many more parts as it has more pages
    int all = 0;
    [[maybe_unused]] int count = 0;     // tiles, of which
    [[maybe_unused]] uint64_t far = 0;  // some have more than kKvOnePage pages
    for (int base = 0; base < batch; base += 64) {
      if constexpr (ROWS > 32 && std::is_same_v<P, KvAttnMore>) {
        const KvSeq s = seq(base);
        const int n = tiles(s), each = pages(s);
        all += n * each;
        count += n;
        far |= __ballot(n > 0 && each > kKvOnePage);
      } else {
        all += tiles(seq(base)) * pages(seq(base));
      }
    }
    if (__ballot(falls) != 0) return false;
    all = __builtin_amdgcn_readlane(kv_scan(all), 63);
    // few rows: no part shorter than pays for joining it.  Measured, heads of
    // 128, us in parts of 16 pages at least and of 8:
    //   one sequence, 8 heads: 16 pages 9.5 and 12.0, 17 13.5 and 11.6, 32 13.8
    //   and 12.0, 64 13.8 and 12.2, 65 13.6 and 12.2, 128 15.2 and 14.7, 256
    //   16.4 and 18.9, 400 20.0 and 20.3;
    //   one head: 65 13.5 and 11.7, 128 13.6 and 11.7, 256 13.7 and 13.9, 400
    //   15.8 and 17.4;
    //   8 heads, two sequences of 16 pages 9.6 and 12.0, of 64 15.1 and 14.0,
    //   four of 64 15.9 and 16.0.
    // The rule goes by the pages of all tiles together, which is coarse: it
    // gives away some 2 us from 65 to about 128 pages, and where several
    // sequences of up to 16 pages are 64 together or fewer.
    const int least = p.min_pages > 0 ? p.min_pages : all <= 16 || all > 64 ? 16 : 8;
    // A quarter more than an even share, few rows: every tile's last part comes
    // on top of the whole ones, and would run in a second round.  Measured, 8
    // heads of 128, even shares and a quarter more: 4 sequences of up to 30000
    // tokens 31.4 us and 24.4, 16 of up to 16000 47.9 and 41.2, 64 of up to
    // 4100 44.6 and 41.7; five rows each of 32 of up to 16384 87.9 and 89.2.
    // (Where all shares fit one round there is nothing to gain: one head over
    // 2047 pages has parts of 20 pages, 103 of them, 26 us.)
    const unsigned share = ROWS <= 32 ? (unsigned)all + (unsigned)all / 4 : (unsigned)all;
    // Whatever sets the chunk, here and below, it is ceil(all / target) or more.
    // So there are `target` parts at most beyond one for each tile, which is what
    // the launch's grid and the workspace's slots are made for, and a tile has
    // no more than target <= kKvMaxParts, for which the joins have room: shorter
    // parts would be written behind the workspace, or not computed.
    w.chunk = max((int)((share + p.target - 1) / (unsigned)p.target), least);
    if constexpr (ROWS > 32 && std::is_same_v<P, KvAttnMore>) {
      // Many rows of a tree, or with sinks: no more than 32 parts of a tile on
      // average, and two pages each (min_pages).  Measured, us with parts of 2,
      // 4 and 8 pages: one tree of 13 rows of 48 heads over 1003 tokens 14.4,
      // 17.6 and 23.1, over 4000 17.9, 18.8 and 23.2, four trees over up to
      // 2000 17.8, 18.8 and 23.8; 61 rows of 16 heads of 64 over 16000 (250
      // pages) 27.4, 27.7 and 24.1.
      count = __builtin_amdgcn_readlane(kv_scan(count), 63);
      const unsigned most = 32u * (unsigned)max(count, 1);
      w.chunk = max(w.chunk, (int)(((unsigned)all + most - 1) / most));
      // One page each where no tile has more than 16 and all heads together have
      // half a chip's.  Measured, us with two pages and with one: 13 rows of 48
      // heads over 8 and 1003 tokens (16 pages) 14.2 and 13.7, over 17 to 19
      // pages 13.5 to 14.5 and 14.4 to 14.7, 26 over 500 tokens 16.1 and 14.7, 61
      // of 16 over 8 of 64 and 1003 14.1 and 12.6, 61 over 1003 19.5 and 22.6; 26
      // rows of 16 over 4 heads of 192 and 4, 8, 12 and 16 pages 17.8, 18.2, 18.9,
      // 19.1 and 16.3, 17.3, 18.1, 18.9, of 256 20.4, 20.9, 21.5, 22.1 and 18.7,
      // 19.9, 21.0, 22.3 (13 of 48 over 8 and 16 pages 20.3 and 21.3, the one side
      // on which it loses); four sequences of 61, 1, 1 and 1 pages, 12 over 2 heads
      // of 128, 17.7 and 21.3, which is why the longest counts.
      if (far == 0 && (unsigned)all * (unsigned)p.kv_heads <= 128u)
        w.chunk = max((int)(((unsigned)all + p.target - 1) / (unsigned)p.target), 1);
      // From 12 pages on somewhat longer parts, if all of them then run at
      // once.  Measured, us without and with that: 64 rows of 48 heads over
      // 131001 tokens 250 and 233, 61 rows over 60000 129 and 118, of eight
      // sequences of up to 30000 202 and 180, 13 rows of twelve of up to 16000
      // 74 and 59.
      if (w.chunk >= 12) {
        const int first = w.chunk;
        w.chunk = first + (first + 15) / 16;
        for (int i = 0; i < 6; ++i) {
          const int c = first + i * max(first / 48, 1);
          int parts = 0;
          for (int base = 0; base < batch; base += 64) {
            const KvSeq s = seq(base);
            parts += __builtin_amdgcn_readlane(kv_scan(tiles(s) * ((int)((unsigned)(pages(s) - 1) / (unsigned)c) + 1)), 63);
          }
          if (parts > p.target) continue;
          w.chunk = c;
          break;
        }
      }
    }
  }
  // whole parts ahead of a tile's last one
  const auto whole = [&](const KvSeq& s) { return (int)((unsigned)(pages(s) - 1) / (unsigned)w.chunk); };
  // sequence `at` of the 64 from `base`, its tile's part 0 after `before` others
  const auto take = [&](int base, int at, int before) {
    const KvSeq s = seq(base);
    w.b = base + at;
    w.s.q0 = __builtin_amdgcn_readlane(s.q0, at);
    w.s.n = __builtin_amdgcn_readlane(s.n, at);
    w.s.len = __builtin_amdgcn_readlane(s.len, at);
    w.parts = (p.target > 0 ? __builtin_amdgcn_readlane(whole(s), at) : 0) + 1;
    w.slot = before + w.tile * w.parts;
    w.tile = __builtin_amdgcn_readlane(tiles(s), at) - 1 - w.tile;  // the last rows see the most: they begin first
  };
  int wholes = 0;
  if (p.target > 0) {
    int before_tiles = 0;
    for (int base = 0; base < batch; base += 64) {
      const KvSeq s = seq(base);
      const int nt = tiles(s), nw = nt * whole(s);
      const int st = kv_scan(nt), sw = kv_scan(nw);
      const int all_w = __builtin_amdgcn_readlane(sw, 63);
      if (!JOIN && item < wholes + all_w) {
        const int at = __builtin_ctzll(__ballot(wholes + sw > item));
        const int from = wholes + __builtin_amdgcn_readlane(sw - nw, at);
        const int each = __builtin_amdgcn_readlane(whole(s), at);
        w.tile = (int)((unsigned)(item - from) / (unsigned)each);
        w.split = item - from - w.tile * each;
        take(base, at, from + before_tiles + __builtin_amdgcn_readlane(st - nt, at));
        return true;
      }
      wholes += all_w;
      before_tiles += __builtin_amdgcn_readlane(st, 63);
    }
  }
  if (JOIN) item += wholes;
  int before_tiles = 0, before_wholes = 0;
  for (int base = 0; base < batch; base += 64) {
    const KvSeq s = seq(base);
    if (__ballot(falls) != 0) return false;
    const int nt = tiles(s), nw = p.target > 0 ? nt * whole(s) : 0;
    const int st = kv_scan(nt), sw = p.target > 0 ? kv_scan(nw) : 0;
    const int mine = item - wholes - before_tiles, all_t = __builtin_amdgcn_readlane(st, 63);
    if (mine < all_t) {
      const int at = __builtin_ctzll(__ballot(st > mine));
      const int from = __builtin_amdgcn_readlane(st - nt, at);
      w.tile = mine - from;
      take(base, at, before_tiles + from + before_wholes + __builtin_amdgcn_readlane(sw - nw, at));
      w.split = w.parts - 1;
      return true;
    }
    before_tiles += all_t;
    before_wholes += __builtin_amdgcn_readlane(sw, 63);
  }
  return false;
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

// Of rows from token t0 to token t1 of a sequence's: no row sees tokens ahead
// of kv_first_range's lo (its sinks apart) or from kv_last_range's hi on; all
// see those from the last's lo to the first's hi.
__device__ __forceinline__ KvRowRange kv_first_range(const KvAttnParams& p, const KvSeq& s, int t0) { return kv_row_range(p, s, t0); }
__device__ __forceinline__ KvRowRange kv_last_range(const KvAttnParams& p, const KvSeq& s, int t1) { return kv_row_range(p, s, t1); }
__device__ __forceinline__ KvRowRange kv_first_range(const KvAttnMore& p, const KvSeq& s, int t0) {
  if (!p.mask) return kv_row_range(p, s, t0);
  const int base = s.len - s.n;
  return KvRowRange{p.window > 0 ? max(base - p.window, 0) : 0, max(base, 0)};
}
__device__ __forceinline__ KvRowRange kv_last_range(const KvAttnMore& p, const KvSeq& s, int t1) {
  if (!p.mask) return kv_row_range(p, s, t1);
  return KvRowRange{p.window > 0 ? max(s.len - s.n - max(p.window - s.n, 0), 0) : 0, s.len};
}
// A tile's pages where sinks may stand apart, as places 0, 1, ..: the first
// `front` are the sinks' pages, the others `gap` further.
struct KvPlaces {
  int front, gap;
  __device__ __forceinline__ int operator()(int at) const { return at < front ? at : at + gap; }
};
__device__ __forceinline__ KvPlaces kv_places(const KvAttnMore& p, const KvRowRange& r0, const KvRowRange& r1) {
  const int first = r0.lo / kKvPage, front = min((min(p.sinks, r1.hi) + kKvPage - 1) / kKvPage, first);
  return KvPlaces{front, first - front};
}
__device__ __forceinline__ int kv_sinks(const KvAttnMore& p, int hi) { return min(p.sinks, hi); }
__device__ __forceinline__ int kv_sinks(const KvAttnParams&, int) { return 0; }

// Bits from up to (not including) to, of 64.
__device__ __forceinline__ uint64_t kv_bits(int from, int to) {
  from = max(from, 0);
  to = min(to, 64);
  return from < to ? (~0ull >> (64 - to + from)) << from : 0ull;
}
// What a row sees: the context's tokens [lo, hi) and those ahead of sinks, and
// of a tree the rows that its words say.
struct KvRowMore {
  int lo, hi, sinks;
  const uint64_t* mask;  // null: no tree (or no row)
};
__device__ __forceinline__ KvRowMore kv_row_more(const KvAttnMore& p, const KvSeq& s, int token, bool ok) {
  KvRowMore r;
  if (p.mask) {
    const int base = s.len - s.n;
    r.mask = ok ? p.mask + (int64_t)(s.q0 + token) * p.words : nullptr;
    r.lo = 0;
    if (p.window > 0 && ok) {
      int seen = 0;
      for (int i = 0; i < p.words && 64 * i < s.n; ++i) seen += __builtin_popcountll(r.mask[i] & kv_bits(0, s.n - 64 * i));
      r.lo = max(base - max(p.window - seen, 0), 0);
    }
    r.hi = ok ? max(base, 0) : 0;
  } else {
    const KvRowRange x = kv_row_range(p, s, token);
    r.mask = nullptr;
    r.lo = x.lo;
    r.hi = ok ? x.hi : 0;
  }
  r.sinks = min(p.sinks, r.hi);
  return r;
}
// A row's bits of the page that begins at token j0 and holds `left` tokens.
// (Pages that need them are few: what the row sees is found anew for each, so
// that nothing of it is held all along the page loop.)
__device__ __forceinline__ uint64_t kv_row_bits(const KvAttnMore& p, const KvSeq& s, const KvRowMore r, int j0, int left) {
  uint64_t bits = kv_bits(r.lo - j0, r.hi - j0) | kv_bits(0, r.sinks - j0);
  const int off = j0 - (s.len - s.n);  // of the page's first token in the tree
  if (r.mask && off > -64 && off < s.n) {
    uint64_t tree;
    if (off < 0) {
      tree = r.mask[0] << -off;
    } else {
      const int word = off >> 6, shift = off & 63;
      tree = word < p.words ? r.mask[word] >> shift : 0ull;
      if (shift > 0 && word + 1 < p.words) tree |= r.mask[word + 1] << (64 - shift);
    }
    bits |= tree & kv_bits(-off, s.n - off);
  }
  return bits & kv_bits(0, left);
}
__device__ __forceinline__ uint64_t kv_row_bits(const KvAttnMore& p, const KvSeq& s, int row, int rows, int j0, int left) {
  asm volatile("" : "+v"(row));  // stays where it is called
  const bool ok = row < rows;
  return kv_row_bits(p, s, kv_row_more(p, s, ok ? row / p.group : 0, ok), j0, left);
}
// A score where its bit is set, else -infinity.
__device__ __forceinline__ float kv_seen(uint64_t bits, int bit, float y) {
  const uint32_t all = (uint32_t)__builtin_amdgcn_sbfe((int)(bit < 32 ? (uint32_t)bits : (uint32_t)(bits >> 32)), bit & 31, 1);
  return __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, y) & all) | (0xFF800000u & ~all));
}

// Floats of a part's result: (max, sum) of each row, then O [ROWS][D].
__host__ __device__ constexpr int kv_part_floats(int rows, int D) { return rows * (D + 2); }

// Buffer descriptor over the codes of one head's page; bytes 0: every load
// gives zeros and touches no memory.
typedef __amdgpu_buffer_rsrc_t kv_rsrc_t;
__device__ __forceinline__ kv_rsrc_t kv_rsrc(const void* base, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, bytes, 0x00020000);
}

// Table entries of pages at first, first + step, ..: a lane holds one of 64.
struct KvPages {
  int ids;
  // page id of entry k (asked for in order); -1 past `end` or where the table holds no page
  template <typename Real>
  __device__ __forceinline__ int at(const KvAttnParams& p, int b, int first, int step, int end, int k, Real real) {
    if ((k & 63) == 0) {
      const int place = first + step * (k + ((int)threadIdx.x & 63));
      ids = place < end ? kv_page(p.batch, b, real(place)) : -1;
    }
    return __builtin_amdgcn_readlane(ids, k & 63);
  }
};

// The offset of the codes of K, in a row's scores.
template <bool BYTES, int COUNT>
__device__ __forceinline__ float kv_query_offset(const half8_t (&q)[COUNT]) {
  if constexpr (!BYTES) return 0.f;
  float sum = 0.f;
#pragma unroll
  for (int c = 0; c < COUNT; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += (float)q[c][j];
  return -kKvOffset<BYTES> * kv_col_sum(sum);
}
// The offset of the codes of V as rows of an operand.
template <bool BYTES>
__device__ __forceinline__ half8_t kv_offset_operand() {
  half8_t v;
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = (_Float16)kKvOffset<BYTES>;
  return v;
}

// One page's codes in flight or at hand, as a wave holds them.
template <int D>
struct KvCodes {
  u32x4_t k[4][D / 64], v[D / 16];
};

// Waves of a workgroup: two for each SIMD as long as their registers allow.
constexpr int kv_waves(int D) { return D <= 128 ? 8 : 4; }

// Few rows: a workgroup's waves share a part's pages in turn, each with its
// own running maximum and sum; they are joined through LDS, and the parts of
// a tile by the workgroup that finishes last.
//
// Bound by HBM (each code is read once).  A wave's registers hold one page:
// the next page's K is requested as soon as the scores are formed, its V as
// soon as the outputs are, so a wave always has a page's worth of loads in
// flight while it computes.  Every load is issued (past the last page from an
// empty descriptor): a conditional load would make the compiler wait for all
// that are in flight.
//
// The running maximum is raised only when a score passes it by more than 8
// (in log2): then the four lanes of a column agree on a new one and the
// outputs are rescaled.  Otherwise a page costs no step across lanes, and the
// probabilities, at most 2^15 (kKvLift), stay inside fp16.  They are taken as
// the sum of two fp16 numbers: what is lost of a term is no more than 2^-22 of
// it, or 2^-32 of the outputs' unit (kv_in_unit).  The second product is cheap
// beside the loads.
//
// Measured, 8 heads of 128 with 6 query heads each: one row over 131001
// tokens 55 us (4.9 TB/s of codes), over 1003 tokens 9.6 us (a launch, the
// table, two pages a wave and the join); one row each of 16 sequences of 1000
// to 16000 tokens 41 us; five rows each of 32 sequences of 1024 to 16384
// tokens (e4m3) 88 us (4.3 TB/s).
template <int D, int FMT, int RT, typename P>
__global__ __launch_bounds__(64 * kv_waves(D)) void kv_attn_rows_kernel(P p) {
  constexpr bool MORE = std::is_same_v<P, KvAttnMore>;
  constexpr int C = D / 64, N = D / 16, ROWS = 16 * RT, NW = kv_waves(D), THREADS = 64 * NW;
  constexpr bool BYTES = FMT == BQ_KV_I8;
  constexpr int JOIN = NW * (N * 256 + 32);
  __shared__ __align__(16) float lds[JOIN > 2 * kKvMaxParts * ROWS ? JOIN : 2 * kKvMaxParts * ROWS];
  __shared__ int last;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int lane = (int)threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int item = p.item0 + (int)blockIdx.y, head = (int)blockIdx.x;
  KvWork w;
  if (!kv_attn_work<ROWS>(p, item, w)) return;
  const KvSeq s = w.s;
  const int rows = s.n * p.group, row0 = w.tile * ROWS;

  // the tile's pages, and the tokens that all its rows see
  const int tok0 = row0 / p.group, tok1 = min((row0 + ROWS - 1) / p.group, s.n - 1);
  const KvRowRange r0 = kv_first_range(p, s, tok0), r1 = kv_last_range(p, s, tok1);
  const auto real = [&] {
    if constexpr (MORE) return kv_places(p, r0, r1);
    else return [](int at) { return at; };
  }();
  int pa = r0.lo / kKvPage, pages = max((r1.hi + kKvPage - 1) / kKvPage - pa, 0);
  if constexpr (MORE) {
    pages = max((r1.hi + kKvPage - 1) / kKvPage - real.gap, 0);
    pa = 0;
  }
  const int begin = pa + (w.parts > 1 ? w.split * w.chunk : 0);
  const int end = pa + (w.split == w.parts - 1 ? pages : min((w.split + 1) * w.chunk, pages));

  // The wave's k-th page is at begin + wave + NW k.  A lane holds the table's
  // entry of one of 64 of them, so that no request waits for the table.
  KvPages pages_of;
  const auto place = [&](int k) -> int64_t {
    const int page = pages_of.at(p, w.b, begin + wave, NW, end, k, real);
    return page < 0 ? -1 : (int64_t)page * p.kv_heads + head;
  };
  const float scale = p.scale * kKvUnit<BYTES>;
  KvCodes<D> x;
  const auto load_k = [&](int64_t at) {
    const kv_rsrc_t rs = kv_rsrc(p.k + max(at, (int64_t)0) * (kKvPage * D), at < 0 ? 0 : kKvPage * D);
#pragma unroll
    for (int i = 0; i < 4 * C; ++i)
      x.k[i / C][i % C] = __builtin_amdgcn_raw_buffer_load_b128(rs, lane * 16, i * 1024, 0);
  };
  const auto load_v = [&](int64_t at) {
    const kv_rsrc_t rs = kv_rsrc(p.v + max(at, (int64_t)0) * (kKvPage * D), at < 0 ? 0 : kKvPage * D);
#pragma unroll
    for (int n = 0; n < N; ++n) x.v[n] = __builtin_amdgcn_raw_buffer_load_b128(rs, lane * 16, n * 1024, 0);
  };
  f32x4 sk, sv;
  const auto load_scales = [&](int64_t at) {
    sk = *reinterpret_cast<const f32x4*>(p.ks + max(at, (int64_t)0) * kKvBlocks);
    sv = *reinterpret_cast<const f32x4*>(p.vs + max(at, (int64_t)0) * kKvBlocks);
  };
  int64_t here = place(0);
  load_k(here);
  load_scales(here);
  load_v(here);

  // Q as the B operand: column r, k = dims 64c + 16g + 8h .. + 7
  half8_t q[RT][2 * C];
  int lo[RT], hi[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int row = row0 + 16 * t + r;
    const bool ok = row < rows;
    const int token = ok ? row / p.group : 0, qh = head * p.group + (ok ? row - token * p.group : 0);
    if constexpr (MORE) {
      lo[t] = 0;
      hi[t] = ok ? r1.hi : 0;  // (above 0: a row)
    } else {
      const KvRowRange range = kv_row_range(p, s, token);
      lo[t] = range.lo;
      hi[t] = ok ? range.hi : 0;
    }
    const _Float16* src = p.q + (int64_t)(s.q0 + token) * p.q_stride + qh * D + 16 * g;
#pragma unroll
    for (int c = 0; c < 2 * C; ++c)
      q[t][c] = ok ? *reinterpret_cast<const half8_t*>(src + (c >> 1) * 64 + (c & 1) * 8) : half8_t{};
  }

  // what the offset of the codes adds to every score of a row
  float q_off[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) q_off[t] = kv_query_offset<BYTES>(q[t]);
  const half8_t ones = kv_offset_operand<BYTES>();

  f32x4 o[RT][N], o_off[RT];  // o_off: what the codes' offset has added to each o since it was last taken off
  float m[RT], l[RT];
  int unit_ex = kKvLeastUnit;  // of R, the unit of o
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    m[t] = -__builtin_inff();
    l[t] = 0.f;
    o_off[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int n = 0; n < N; ++n) o[t][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  for (int at = begin + wave, k = 1; at < end; at += NW, ++k) {
    const int64_t next = place(k);
    const int j0 = real(at) * kKvPage;
    const int left = here < 0 ? 0 : s.len - j0;  // tokens of the page that are held

    // scores, in units of log2
    f32x4 y[RT][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int t = 0; t < RT; ++t) y[t][i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const half8_t a0 = kv_operand8<FMT, BYTES>(x.k[i][c][0], x.k[i][c][1]), a1 = kv_operand8<FMT, BYTES>(x.k[i][c][2], x.k[i][c][3]);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          y[t][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a0, q[t][2 * c], y[t][i], 0, 0, 0);
          y[t][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a1, q[t][2 * c + 1], y[t][i], 0, 0, 0);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float c = sk[i] * scale, off = q_off[t] * c;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[t][i][e] = BYTES ? __builtin_fmaf(y[t][i][e], c, off) : y[t][i][e] * c;
      }
    load_k(next);
    if (left < kKvPage || ((j0 + kKvPage > r0.hi || j0 < r1.lo) && (!MORE || j0 + kKvPage > kv_sinks(p, r0.hi)))) {
      // a page that some row does not see whole: the row's tokens [lo, hi)
      // as one unsigned comparison of each token, or by its bits
      if constexpr (MORE) {
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          const uint64_t bits = kv_row_bits(p, s, row0 + 16 * t + r, rows, j0, left) >> (4 * g);
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              y[t][i][e] = kv_seen(bits, 16 * i + e, y[t][i][e]);
        }
      } else {
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          const int from = max(lo[t] - j0, 0), count = max(min(hi[t] - j0, left) - from, 0);
          int in = 4 * g - from;
          // stays in this branch: computed ahead of it, it would cost every page
          asm volatile("" : "+v"(in));
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              y[t][i][e] = (unsigned)(in + 16 * i + e) < (unsigned)count ? y[t][i][e] : -__builtin_inff();
        }
      }
      // what lies past the length is never used: neither a scale (any in R's
      // range stands for it) nor, in e4m3, a code that is no number
      if (left < kKvPage) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (16 * i >= left) sv[i] = left > 0 ? sv[0] : kv_exp_float(unit_ex);
          if constexpr (FMT == BQ_KV_E4M3) {
            const int keep = min(max(left - 16 * i - 4 * g, 0), 4);
            const uint32_t mask = keep == 4 ? 0xFFFFFFFFu : (1u << (8 * keep)) - 1u;
#pragma unroll
            for (int n = 0; n < N; ++n) x.v[n][i] &= mask;
          }
        }
      }
    }

    // running maximum and unit of o
    f32x4 unit = sv * kv_exp_float(254 - unit_ex);
    const float low = kv_min4(unit), top = kv_max4(unit);
    const bool fine = kv_in_unit(low, top);
    float mx[RT];
    bool raise = !fine;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      mx[t] = y[t][0][0];
#pragma unroll
      for (int i = 0; i < 4; ++i) mx[t] = kv_max3(kv_max3(mx[t], y[t][i][0], y[t][i][1]), y[t][i][2], y[t][i][3]);
      raise = raise || mx[t] > m[t] + 8.f;
    }
    if (__ballot(raise) != 0) {
      float alpha[RT];
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const float mn = __builtin_fmaxf(m[t], kv_col_max(mx[t]));
        alpha[t] = mn == -__builtin_inff() ? 1.f : kv_exp2(m[t] - mn);
        m[t] = mn;
        l[t] *= alpha[t];
      }
      float change = 1.f;
      if (__builtin_amdgcn_readfirstlane(!fine))
        change = kv_fit_unit(
            unit, low, top,
            [&] {  // rows past the last one (hi 0) and those that have seen nothing have no terms
              float most = -__builtin_inff();
#pragma unroll
              for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float term = kv_max4(y[t][i]) + __builtin_amdgcn_logf(unit[i]) - m[t];
                  most = hi[t] > 0 && m[t] > -__builtin_inff() ? __builtin_fmaxf(most, term) : most;
                }
              return kv_wave_max(most);
            },
            unit_ex);
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const float f = alpha[t] * change;
        o_off[t] *= f;
#pragma unroll
        for (int n = 0; n < N; ++n) o[t][n] *= f;
      }
    }
    if (BYTES && k % kKvOffsetRowPages == 0) {
#pragma unroll
      for (int t = 0; t < RT; ++t) {
#pragma unroll
        for (int n = 0; n < N; ++n) o[t][n] -= o_off[t];
        o_off[t] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
    }
    half8_t ph_[RT][2], pl_[RT][2];
    load_scales(next);
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const float base = m[t] == -__builtin_inff() ? 0.f : m[t] - kKvLift;  // (0: a row that has seen nothing yet)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float e2 = kv_exp2(y[t][i][e] - base);
          l[t] += e2;
          const float f = e2 * unit[i];
          const _Float16 h = (_Float16)f;
          ph_[t][i >> 1][(i & 1) * 4 + e] = h;
          pl_[t][i >> 1][(i & 1) * 4 + e] = (_Float16)(f - (float)h);
        }
    }
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const half8_t a = kv_operand8<FMT, BYTES>(x.v[n][2 * h], x.v[n][2 * h + 1]);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          o[t][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, ph_[t][h], o[t][n], 0, 0, 0);
          o[t][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, pl_[t][h], o[t][n], 0, 0, 0);
        }
      }
    if constexpr (BYTES) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          o_off[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones, ph_[t][h], o_off[t], 0, 0, 0);
          o_off[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones, pl_[t][h], o_off[t], 0, 0, 0);
        }
    }
    load_v(next);
    here = next;
  }

  // The waves' results are joined through LDS, 16 rows at a time: a thread
  // adds up four values of a row.
  constexpr int SLOT = kv_part_floats(ROWS, D);
  const auto slot = [&](int part) { return p.part + ((int64_t)(w.slot + part) * p.kv_heads + head) * SLOT; };
  float *ml = lds + NW * N * 256;  // [wave][16 rows] (max, sum)
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const float sum = kv_col_sum(l[t]);
#pragma unroll
    for (int n = 0; n < N; ++n) *reinterpret_cast<f32x4*>(lds + ((wave * N + n) * 64 + lane) * 4) = (o[t][n] - o_off[t]) * (kv_exp_float(unit_ex) * kKvUnit<BYTES>);
    if (g == 0) *reinterpret_cast<float2*>(ml + (wave * 16 + r) * 2) = make_float2(m[t], sum);
    __syncthreads();
    const int row = 16 * t + r;  // of the tile; the same for all that a thread takes
    float2 of[NW];
    float mx = -__builtin_inff(), all = 0.f;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      of[i] = *reinterpret_cast<const float2*>(ml + (i * 16 + r) * 2);
      mx = __builtin_fmaxf(mx, of[i].x);
    }
    const float base = mx == -__builtin_inff() ? 0.f : mx;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      of[i].x = kv_exp2(of[i].x - base);
      all += of[i].y * of[i].x;
    }
    if (row0 + row < rows) {
      const int token = (row0 + row) / p.group, qh = head * p.group + row0 + row - token * p.group;
      _Float16* dst = p.out + (int64_t)(s.q0 + token) * p.out_stride + qh * D + 4 * g;
      float* mine = slot(w.split);
      const float inv = all > 0.f ? 1.f / all : 0.f;  // nothing seen: zeros
#pragma unroll
      for (int n = wave; n < N; n += NW) {
        f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NW; ++i) y += *reinterpret_cast<const f32x4*>(lds + ((i * N + n) * 64 + lane) * 4) * of[i].x;
        if (w.parts == 1) {
          y *= inv;
          *reinterpret_cast<half4_t*>(dst + 16 * n) =
              half4_t{(_Float16)y[0], (_Float16)y[1], (_Float16)y[2], (_Float16)y[3]};
        } else {
          float* to = mine + 2 * ROWS + row * D + 16 * n + 4 * g;
          kv_put2(to, y[0], y[1]);
          kv_put2(to + 2, y[2], y[3]);
        }
      }
      if (w.parts > 1 && wave == 0 && g == 0) kv_put2(mine + 2 * row, mx, all);
    }
    if (t + 1 < RT) __syncthreads();
  }
  if (w.parts == 1) return;

  // The part's result is in its slot; the workgroup that counts last joins
  // the tile's parts, in order (the same result on every call).
  unsigned* counter = p.counters + (int64_t)w.slot * p.kv_heads + head;
  // every wave's stores are performed at device scope before the count is
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0)
    last = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (unsigned)(w.parts - 1);
  __syncthreads();
  if (!last) return;
  // Two values of the tile a thread, or, where the tile has fewer, a share of
  // the parts of two values; AHEAD parts are requested at a time, the first
  // of them together with the maxima and sums.
  constexpr int AHEAD = 16;
  const int some = min(ROWS, rows - row0), pairs = some * (D / 2);
  const int groups = max(THREADS / pairs, 1);
  const int tid = (int)threadIdx.x, group = groups > 1 ? tid / pairs : 0;
  float *wm = lds, *wl = lds + kKvMaxParts * ROWS;
  float2 v[AHEAD];
  const auto request = [&](int at, int k0) {
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int part = min(group + (k0 + k) * groups, w.parts - 1);
      v[k] = kv_get2(slot(part) + 2 * ROWS + 2 * min(at, pairs - 1));  // no branch: all are in flight at once
    }
  };
  int at = groups > 1 ? (group < groups ? tid - group * pairs : pairs) : tid;
  request(at, 0);
  for (int i = tid; i < w.parts * ROWS; i += THREADS) {
    const int part = i / ROWS, row = i % ROWS;
    float2 ml = make_float2(-__builtin_inff(), 0.f);
    if (row < some) ml = kv_get2(slot(part) + 2 * row);
    wm[i] = ml.x;
    wl[i] = ml.y;
  }
  __syncthreads();
  {
    constexpr int PER = THREADS / ROWS;  // consecutive lanes of a row
    const int row = tid / PER, sub = tid % PER;
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
  for (bool fresh = true; __syncthreads_or(at < pairs); at += THREADS, fresh = false) {
    const int row = min(at, pairs - 1) / (D / 2);
    float2 sum = make_float2(0.f, 0.f);
    if (!fresh) request(at, 0);
    for (int k0 = 0; k0 * groups < w.parts; k0 += AHEAD) {
      if (k0 > 0) request(at, k0);
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const int part = group + (k0 + k) * groups;
        const float f = part < w.parts ? wm[part * ROWS + row] : 0.f;
        sum.x += v[k].x * f;
        sum.y += v[k].y * f;
      }
    }
    if (groups > 1) {
      if (at < pairs) reinterpret_cast<float2*>(wl)[group * pairs + at] = sum;
      __syncthreads();
      if (group == 0 && at < pairs)
        for (int i = 1; i < groups; ++i) {
          const float2 other = reinterpret_cast<const float2*>(wl)[i * pairs + at];
          sum.x += other.x;
          sum.y += other.y;
        }
    }
    if (group == 0 && at < pairs) {
      const int token = (row0 + row) / p.group, qh = head * p.group + row0 + row - token * p.group;
      *reinterpret_cast<half2_t*>(p.out + (int64_t)(s.q0 + token) * p.out_stride + qh * D + 2 * (at % (D / 2))) =
          half2_t{(_Float16)sum.x, (_Float16)sum.y};
    }
    if (groups > 1) break;
  }
  if (threadIdx.x == 0) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

}  // namespace bq
