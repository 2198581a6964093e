// Log probabilities of given tokens, entropy and the largest values of rows of
// logits, in one read of them.
//
//   log p[v] = x[v] - m - log s,  s = sum exp(x - m),
//   entropy = log s - sum (x - m) exp(x - m) / s.
// Terms of fp16 logits are formed as 2^(x log2(e) - B) with B = m log2(e)
// rounded to fp32; the rounding, fma(m, log2(e), -B), is taken out of the
// result again, so a term's error goes by its distance from the maximum and not
// by m.  With fp32 logits, of which there are half as many in a byte and whose
// product with log2(e) may pass fp32's range, B is m and the term
// 2^((x - B) log2(e)).  A wave keeps one running maximum, sums are fp32, four to
// a lane.
//
// The largest values: a value and its token make one 64-bit number, a larger
// value first, then a lower token, all different.  A wave collects numbers from
// a floor on, below which none is among the `top`, in LDS, unsorted: a lane
// compares its maximum, which the softmax needs anyway, and only where one
// passes are the values of its 16-byte blocks that pass looked at, side by side,
// a thread one (through LDS: a register has no number that a thread could
// choose).  The floor begins at what the maxima of a workgroup's first 1024
// blocks say (`top` lanes hold a value from it on, so as many values are), rises
// with the lanes' maxima over more of them, by a wave's maxima where most of its
// lanes pass, and when the room runs out: then the `top` largest are found by
// bisection, a count over the wave for each step, and the others leave.  A value
// equal to the floor's passes only with a lower token.  In the end each of the
// waves' numbers, then of the parts', finds its place by counting those above it.
// So ties and order change nothing but the time: 2047 rows of 151936 in fp16 with
// entropy, top 1, 20 and 64, take 118, 127 and 141 us with random values, 125, 128
// and 133 with equal ones, 116, 120 and 121 with values that fall all along, 144,
// 288 and 846 with values that rise: each pass then holds only new ones.
#pragma once

#include "kv_common.hpp"
#include "spec_kernels.hpp"

namespace bq {

constexpr int kLpWaves = 4, kLpThreads = 64 * kLpWaves;
constexpr int kLpLoads = 4;                              // 16-byte loads of a lane at a time
constexpr int kLpWaveBlocks = 64 * kLpLoads;             // 16-byte blocks a wave takes at a time
constexpr int kLpBlocks = kLpWaves * kLpWaveBlocks;      // and a workgroup
constexpr int kLpMaxSplit = 64;
constexpr int kLpCounterStride = 8;                      // 4-byte words between rows
constexpr int kLpSplitRows = BQ_LOGPROBS_COUNTER_BYTES / (4 * kLpCounterStride);
constexpr int kLpAhead = 3;                              // parts a wave asks for at a time
constexpr int kLpRoom = 64 * (1 + kLpAhead);             // numbers a wave collects
constexpr int kLpStage = 64;                             // blocks whose values it looks at

struct LogprobsParams {
  const void* logits;
  int64_t row_stride;
  const int* tokens;
  float *logprob, *entropy, *top_logprobs;
  int* top_tokens;
  unsigned* counters;  // workspace: parts done of each row, zero between calls
  uint64_t* part;      // workspace: what the parts found
  int rows, V, count, top;
  int split;           // workgroups of a row
  int passes;          // of kLpBlocks that one of them makes
};
// 8-byte words of a part: (m, B), (s, t), up to 64 numbers, the largest first
constexpr int lp_slot(int top) { return top > 0 ? 2 + 64 : 2; }

typedef unsigned long long lp_key_t;
typedef lp_key_t lp_pair_t __attribute__((ext_vector_type(2)));

// The largest t found that at least `want` of some numbers reach (0 where fewer
// reach 0), by distances below the largest of them: first powers of two, then
// between two of them, until exactly `want` reach it or the steps run out.  A
// step counts at three distances together: it is a chain of latencies, from the
// lanes' comparison to the next distance, whatever it counts.
template <typename Reach>
__device__ __forceinline__ uint32_t lp_search(uint32_t largest, int want, int steps, Reach reach) {
  const auto at = [&](uint32_t far) { return far < largest ? largest - far : 0u; };
  // exponents: fewer than `want` reach a power that is `low`; at `high` enough do, or it is 2^32
  int low = -1, high = 32;
  while (high - low > 1) {
    const int third = max((high - low) / 4, 1), a = low + third, b = min(a + third, high - 1), c = min(b + third, high - 1);
    const int na = reach(at(1u << a)), nb = reach(at(1u << b)), nc = reach(at(1u << c));
    if (na >= want) high = a;
    else if (nb >= want) low = a, high = b;
    else if (nc >= want) low = b, high = c;
    else low = c;
  }
  uint32_t near = low < 0 ? 0u : 1u << low, far = high == 32 ? 0xFFFFFFFFu : 1u << high;
  if (low < 0 && reach(largest) >= want) return largest;
  for (int i = 0; i < steps && far - near > 1; ++i) {
    const uint32_t part = max((far - near) >> 2, 1u), a = near + part, b = min(a + part, far - 1), c = min(b + part, far - 1);
    const int na = reach(at(a)), nb = reach(at(b)), nc = reach(at(c));
    int n = 0;
    if (na >= want) far = a, n = na;
    else if (nb >= want) near = a, far = b, n = nb;
    else if (nc >= want) near = b, far = c, n = nc;
    else near = c;
    if (n == want) break;
  }
  return at(far);
}
// A result over the wave's lanes in six steps of lanes nearby (data parallel
// primitives: shifts within rows of 16, then broadcasts across rows); each lane
// takes `none` where its neighbour lies outside.
template <typename Op>
__device__ __forceinline__ uint32_t lp_over_wave(uint32_t x, uint32_t none, Op op) {
  x = op(x, __builtin_amdgcn_update_dpp(none, x, 0x111, 0xF, 0xF, false));  // row_shr:1
  x = op(x, __builtin_amdgcn_update_dpp(none, x, 0x112, 0xF, 0xF, false));
  x = op(x, __builtin_amdgcn_update_dpp(none, x, 0x114, 0xF, 0xF, false));
  x = op(x, __builtin_amdgcn_update_dpp(none, x, 0x118, 0xF, 0xF, false));
  x = op(x, __builtin_amdgcn_update_dpp(none, x, 0x142, 0xA, 0xF, false));  // row_bcast:15 into rows 1 and 3
  x = op(x, __builtin_amdgcn_update_dpp(none, x, 0x143, 0xC, 0xF, false));  // row_bcast:31 into rows 2 and 3
  return __builtin_amdgcn_readlane(x, 63);
}
__device__ __forceinline__ uint32_t lp_wave_max(uint32_t x) {
  return lp_over_wave(x, 0u, [](uint32_t a, uint32_t b) { return max(a, b); });
}
__device__ __forceinline__ uint32_t lp_wave_min(uint32_t x) {
  return lp_over_wave(x, 0xFFFFFFFFu, [](uint32_t a, uint32_t b) { return min(a, b); });
}
template <typename Op>
__device__ __forceinline__ float lp_over_wave(float x, float none, Op op) {
  return __builtin_bit_cast(float, lp_over_wave(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, none), [&](uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, op(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)));
  }));
}
__device__ __forceinline__ float lp_wave_sum(float x) {
  return lp_over_wave(x, 0.f, [](float a, float b) { return a + b; });
}

__device__ __forceinline__ lp_key_t lp_lane(lp_key_t x, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)x, lane), hi = __builtin_amdgcn_readlane((uint32_t)(x >> 32), lane);
  return ((lp_key_t)hi << 32) | lo;
}

// A wave's numbers in LDS.
struct LpPicked {
  lp_key_t* room;   // [kLpRoom]
  int n;
  lp_key_t floor;   // numbers below it are not among the `top`
  float least;      // its value
  float above;      // and the next larger one, which a later token than the floor's needs (NaN: all pass)

  __device__ __forceinline__ void raise(lp_key_t to) {
    to = lp_lane(to, 0);  // (the same for all lanes)
    if (to <= floor) return;
    floor = to;
    const uint32_t key = (uint32_t)(to >> 32);
    least = __builtin_bit_cast(float, SpecBits<float>::value_of(key));
    above = __builtin_bit_cast(float, SpecBits<float>::value_of(key + 1));
  }
  // What a value of these tokens, the first of them `first`, has to reach.
  __device__ __forceinline__ float limit(int first) const { return (uint32_t)first > 0xFFFFFFFFu - (uint32_t)floor ? above : least; }
  // What lanes write others read; all in one wave.
  static __device__ __forceinline__ void settle() {
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
  __device__ __forceinline__ uint64_t found(lp_key_t key) const { return __ballot(key != 0 && key >= floor); }  // (0: none)
  // The lanes' numbers from the floor on join; there is room for them.
  __device__ __forceinline__ void add(lp_key_t key) {
    const uint64_t in = found(key);
    if (key != 0 && key >= floor)
      room[n + __builtin_amdgcn_mbcnt_hi((uint32_t)(in >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)in, 0))] = key;
    n += __builtin_popcountll(in);
  }
  // Their number, for others, who read them in twos.
  __device__ __forceinline__ void end(int& count) const {
    if ((threadIdx.x & 63) != 0) return;
    count = n;
    if (n & 1) room[n] = 0;
  }
  // All but the `top` largest leave.
  __device__ __forceinline__ void keep(int top) {
    constexpr int EACH = kLpRoom / 64;
    settle();
    if (n <= top) return;
    lp_key_t key[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const int at = (int)(threadIdx.x & 63) + 64 * i;
      key[i] = at < n ? room[at] : 0;
    }
    // by value, then, of those that have the last value, by token
    uint32_t largest = 0;
#pragma unroll
    for (int i = 0; i < EACH; ++i) largest = max(largest, (uint32_t)(key[i] >> 32));
    largest = lp_wave_max(largest);
    const uint32_t value = lp_search(largest, top, 32, [&](uint32_t at) {
      int reach = 0;
#pragma unroll
      for (int i = 0; i < EACH; ++i) reach += __builtin_popcountll(__ballot((uint32_t)(key[i] >> 32) >= at));
      return reach;
    });
    int above = 0, reach = 0;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      reach += __builtin_popcountll(__ballot((uint32_t)(key[i] >> 32) >= value));
      above += __builtin_popcountll(__ballot((uint32_t)(key[i] >> 32) > value));
    }
    uint32_t token = 0;
    if (reach > top) {
      uint32_t most = 0;
#pragma unroll
      for (int i = 0; i < EACH; ++i) most = max(most, (uint32_t)(key[i] >> 32) == value ? (uint32_t)key[i] : 0u);
      token = lp_search(lp_wave_max(most), top - above, 32, [&](uint32_t at) {
        int n = 0;
#pragma unroll
        for (int i = 0; i < EACH; ++i)
          n += __builtin_popcountll(__ballot((uint32_t)(key[i] >> 32) == value && (uint32_t)key[i] >= at));
        return n;
      });
    }
    const lp_key_t t = ((lp_key_t)value << 32) | token;
    settle();
    n = 0;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const uint64_t found = __ballot(key[i] >= t);
      if (key[i] >= t)
        room[n + __builtin_amdgcn_mbcnt_hi((uint32_t)(found >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)found, 0))] = key[i];
      n += __builtin_popcountll(found);
    }
    settle();
    raise(t);
  }
};

// Maxima that are no number where an operand is none.
__device__ __forceinline__ uint32_t lp_max3(uint32_t a, uint32_t b, uint32_t c, _Float16) {
  uint32_t d;
  asm("v_pk_maximum3_f16 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(b), "v"(c));
  return d;
}
__device__ __forceinline__ uint32_t lp_max3(uint32_t a, uint32_t b, uint32_t c, float) {
  uint32_t d;
  asm("v_maximum3_f32 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(b), "v"(c));
  return d;
}
// The largest of a dword's values.
__device__ __forceinline__ float lp_float(uint32_t w, float) { return __builtin_bit_cast(float, w); }
__device__ __forceinline__ float lp_float(uint32_t w, _Float16) {
  const half2_t h = __builtin_bit_cast(half2_t, w);
  const float a = (float)h.x, b = (float)h.y;
  return __builtin_bit_cast(float, lp_max3(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b),
                                           __builtin_bit_cast(uint32_t, b), 0.f));
}
template <typename T>
__device__ __forceinline__ float lp_value(const u32x4_t& w, int e) {
  const uint32_t bits = w[sizeof(T) == 2 ? e >> 1 : e];  // (a vector's element has no address to cast from)
  if constexpr (sizeof(T) == 2) return (float)__builtin_bit_cast(half2_t, bits)[e & 1];
  else return __builtin_bit_cast(float, bits);
}

constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f;

// A value's place below B, in log2; B of a maximum (0 where that is -inf); how
// far places move from one B to another; what of the sum's logarithm is B's
// rounding.
__device__ __forceinline__ float lp_place(float x, float b, _Float16) { return __builtin_fmaf(x, kLog2e, -b); }
__device__ __forceinline__ float lp_place(float x, float b, float) { return (x - b) * kLog2e; }
__device__ __forceinline__ float lp_base(float m, _Float16) { return m == -__builtin_inff() ? 0.f : m * kLog2e; }
__device__ __forceinline__ float lp_base(float m, float) { return m == -__builtin_inff() ? 0.f : m; }
__device__ __forceinline__ float lp_moved(float from, float to, _Float16) { return from - to; }
__device__ __forceinline__ float lp_moved(float from, float to, float) { return (from - to) * kLog2e; }
__device__ __forceinline__ float lp_rounding(float m, float b, _Float16) { return kLn2 * __builtin_fmaf(m, kLog2e, -b); }
__device__ __forceinline__ float lp_rounding(float, float, float) { return 0.f; }

// What a wave, a workgroup or a row has seen: the largest value, B, and the
// sums of 2^y and of y 2^y over the places y.
struct LpSums {
  float m, b, s, t;
};
// Sums under another B, `d` further; f = 2^d, 0 where there was nothing.
__device__ __forceinline__ void lp_scale(float& s, float& t, float d, float f) {
  t = f > 0.f ? f * __builtin_fmaf(d, s, t) : 0.f;
  s = f > 0.f ? s * f : 0.f;
}
__device__ __forceinline__ float lp_max(float a, float b) {  // no number where one is none
  return a != a ? a : b != b ? b : __builtin_fmaxf(a, b);
}
// Joins what the lanes hold (m -inf: nothing).
template <typename T>
__device__ __forceinline__ LpSums lp_join(LpSums x) {
  LpSums all;
  all.m = lp_over_wave(x.m, -__builtin_inff(), [](float a, float b) { return lp_max(a, b); });
  all.b = lp_base(all.m, T{});
  const float d = lp_moved(x.b, all.b, T{});
  lp_scale(x.s, x.t, d, x.m == -__builtin_inff() ? 0.f : __builtin_amdgcn_exp2f(d));
  all.s = lp_wave_sum(x.s);
  all.t = lp_wave_sum(x.t);
  return all;
}

// One workgroup for a part of a row (of the whole row where rows fill the
// chip); a row's parts are joined by the one that finishes last.  A wave takes
// 4 KB at a time; what hides its loads is the other waves of its SIMD.  Many
// rows are bound by HBM and, not far behind, by issue (a conversion, a
// product, an exponential and two sums for a value), few by the chain of
// latencies from the first load to the join.  Measured with entropy, us
// without alternatives and with 1, 5, 20 and 64: 2047 rows of 151936 in fp16
// 110, 118, 123, 127 and 141 (622 MB: 5.65 to 4.4 TB/s; without entropy 107,
// 113, 117, 124 and 138), 301 rows of it 20.9, 27.6, 30.6, 35.0 and 45.1, 5
// rows 5.4, 9.9, 10.9, 12.6 and 14.7; 301 rows of 32000 in fp32 11.0, 15.1,
// 16.7, 18.4 and 24.5.  Eight waves a SIMD with alternatives, which take some
// registers to memory: 127, 130, 133 and 142 us for the first of these, 30.3,
// 33.2, 37.8 and 48.9 for the second; five waves 115, 119, 124 and 139, but
// 2047 rows of 32000 take 36.2 for 34.6 (top 5).  The next pass's loads asked
// for a pass ahead: 132 us (top 5, 16 registers more).  Numbers are ranked by
// a thread each, and the finding of the `top` largest by bisection stands in
// three places only: with one wave that put them together first, and eight
// places, the code was 45 KB for 25, and 5 rows took 13.5 and 19.0 us (top 20
// and 64).
template <typename T, bool ENTROPY, bool TOP>
__global__ __launch_bounds__(kLpThreads, TOP ? 6 : 8) void logprobs_kernel(LogprobsParams p) {
  constexpr int EPV = 16 / (int)sizeof(T);  // values of a 16-byte block
  __shared__ __align__(16) lp_key_t room[TOP ? kLpWaves : 1][TOP ? kLpRoom : 1];
  __shared__ __align__(16) u32x4_t stage[TOP ? kLpWaves : 1][TOP ? kLpStage : 1];
  __shared__ short stage_of[TOP ? kLpWaves : 1][TOP ? kLpStage : 1];
  __shared__ lp_key_t bound;        // the highest of the waves' floors
  __shared__ uint32_t first[TOP ? kLpThreads : 1];
  __shared__ int counts[kLpWaves];
  __shared__ LpSums sums[kLpWaves];
  __shared__ int last;
  const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int row = (int)blockIdx.x / p.split, part = (int)blockIdx.x - row * p.split;
  const T* logits = static_cast<const T*>(p.logits) + row * p.row_stride;
  // the row in aligned 16-byte blocks: block q holds values q * EPV - lead ..
  const int lead = (int)(((uintptr_t)logits & 15) / sizeof(T));
  const u32x4_t* blocks = reinterpret_cast<const u32x4_t*>(logits - lead);
  const int all = (int)(((int64_t)lead + p.V + EPV - 1) / EPV);
  const int from = part * p.passes * kLpBlocks, to = min(from + p.passes * kLpBlocks, all);

  LpSums x{-__builtin_inff(), 0.f, 0.f, 0.f};  // (the same for all lanes)
  float s[kLpLoads] = {}, t[kLpLoads] = {};
  [[maybe_unused]] LpPicked picked{room[TOP ? wave : 0], 0, 0, -__builtin_inff(), -__builtin_inff()};
  [[maybe_unused]] float seen = -__builtin_inff();  // the largest that the lane has met
  [[maybe_unused]] int pass = 0;
  bool none = false;  // something is no number
  int q0 = from + wave * kLpWaveBlocks;
  const int q_first = q0;
  // (with TOP all waves make the first pass, which has a barrier; past the part it finds nothing)
  for (; q0 < to || (TOP && q0 == q_first); q0 += kLpBlocks) {
    u32x4_t w[kLpLoads];
#pragma unroll
    for (int j = 0; j < kLpLoads; ++j) w[j] = blocks[min(q0 + 64 * j + lane, all - 1)];
    const bool inside = q0 * EPV >= lead && (int64_t)(q0 + kLpWaveBlocks) * EPV - lead <= p.V && q0 + kLpWaveBlocks <= to;
    if (!inside) {
      // values outside the row, and blocks past the part, are -inf
#pragma unroll
      for (int j = 0; j < kLpLoads; ++j) {
        const int q = q0 + 64 * j + lane;
        const int64_t v0 = (int64_t)q * EPV - lead;
#pragma unroll
        for (int e = 0; e < EPV; ++e) {
          if (v0 + e >= 0 && v0 + e < p.V && q < to) continue;
          if constexpr (sizeof(T) == 2) w[j][e >> 1] = e & 1 ? (w[j][e >> 1] & 0xFFFFu) | 0xFC000000u : (w[j][e >> 1] & 0xFFFF0000u) | 0xFC00u;
          else w[j][e] = 0xFF800000u;
        }
      }
    }
    // the largest value of each block, and of all
    uint32_t most[kLpLoads];
#pragma unroll
    for (int j = 0; j < kLpLoads; ++j) most[j] = lp_max3(lp_max3(w[j][0], w[j][1], w[j][2], T{}), w[j][3], w[j][3], T{});
    static_assert(kLpLoads == 4);
    const float top = lp_float(lp_max3(lp_max3(most[0], most[1], most[2], T{}), most[3], most[3], T{}), T{});
    none = none || top != top;
    if (__ballot(top > x.m) != 0) {
      // (a NaN counts for nothing here)
      const float m = lp_over_wave(__builtin_fmaxf(x.m, top), -__builtin_inff(), [](float a, float b) { return __builtin_fmaxf(a, b); });
      const float b = lp_base(m, T{}), d = lp_moved(x.b, b, T{});
      const float f = x.m == -__builtin_inff() ? 0.f : __builtin_amdgcn_exp2f(d);
#pragma unroll
      for (int j = 0; j < kLpLoads; ++j) lp_scale(s[j], t[j], d, f);
      x.m = m;
      x.b = b;
    }
#pragma unroll
    for (int j = 0; j < kLpLoads; ++j)
#pragma unroll
      for (int e = 0; e < EPV; ++e) {
        float y = lp_place(lp_value<T>(w[j], e), x.b, T{});
        if constexpr (ENTROPY) y = __builtin_fmaxf(y, -0x1p20f);  // (-inf: 0 times it is 0)
        const float f = __builtin_amdgcn_exp2f(y);
        s[j] += f;
        if constexpr (ENTROPY) t[j] = __builtin_fmaf(y, f, t[j]);
      }
    if constexpr (TOP) {
      // `top` of the workgroup's lanes have met a value that reaches the floor;
      // found anew after 4, 8, .. passes, if some are left, then without waiting
      // for the others, of whom an older maximum is as true (2047 rows of 151936,
      // top 5, 127 -> 122 us; after the second pass too, 2047 rows of 32000 take
      // 39 for 36)
      seen = __builtin_fmaxf(seen, top);
      ++pass;
      if (pass == 1 || (pass >= 4 && (pass & (pass - 1)) == 0 && q0 + 4 * kLpBlocks < to)) {
        first[threadIdx.x] = q0 < to ? spec_key(seen) : 0u;
        if (pass == 1) {
          if (threadIdx.x == 0) bound = 0;
          __syncthreads();
        } else {
          LpPicked::settle();
        }
        uint32_t of[kLpWaves], largest = 0;
#pragma unroll
        for (int i = 0; i < kLpWaves; ++i) largest = max(largest, of[i] = first[64 * i + lane]);
        picked.raise((lp_key_t)lp_search(lp_wave_max(largest), p.top, 2, [&](uint32_t at) {
          int reach = 0;
#pragma unroll
          for (int i = 0; i < kLpWaves; ++i) reach += __builtin_popcountll(__ballot(of[i] >= at));
          return reach;
        }) << 32);
      }
      const int token0 = q0 * EPV - lead;  // (the first row's may be negative: then all tokens are in question)
      if (__ballot(!(top < picked.limit(max(token0, 0)))) != 0) {
        picked.raise(*(volatile lp_key_t*)&bound);
        const lp_key_t before = picked.floor;
        // many lanes: the floor rises to what `top` of their maxima reach
        // (without this, 2047 rows of values that rise took 1111 us for the
        // largest and 2423 for 64)
        if (__builtin_popcountll(__ballot(!(top < picked.limit(max(token0, 0))))) > min(max(p.top, 16), 48)) {
          const uint32_t mine = spec_key(top);
          picked.raise((lp_key_t)lp_search(lp_wave_max(mine), p.top, 2, [&](uint32_t at) { return __builtin_popcountll(__ballot(mine >= at)); }) << 32);
        }
        const float limit = picked.limit(max(token0, 0));
        // the blocks whose maximum passes go to LDS side by side, of all loads or, where they are many, of one
        bool pass[kLpLoads];
        uint64_t found[kLpLoads];
        int blocks_found = 0;
#pragma unroll
        for (int j = 0; j < kLpLoads; ++j) {
          pass[j] = !(lp_float(most[j], T{}) < limit);
          found[j] = __ballot(pass[j]);
          blocks_found += __builtin_popcountll(found[j]);
        }
        const int loads = blocks_found <= kLpStage ? kLpLoads : 1;
        for (int j0 = 0; j0 < kLpLoads; j0 += loads) {
          int n = 0;
#pragma unroll
          for (int j = 0; j < kLpLoads; ++j) {
            if (j < j0 || j >= j0 + loads) continue;
            if (pass[j]) {
              const int at = n + __builtin_amdgcn_mbcnt_hi((uint32_t)(found[j] >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)found[j], 0));
              stage[TOP ? wave : 0][at] = w[j];
              stage_of[TOP ? wave : 0][at] = 64 * j + lane;
            }
            n += __builtin_popcountll(found[j]);
          }
          LpPicked::settle();
          // their values, a thread one
          for (int i = lane / EPV; i - lane / EPV < n; i += 64 / EPV) {
            const int at = min(i, n - 1), q = q0 + stage_of[TOP ? wave : 0][at];
            const T value = reinterpret_cast<const T*>(&stage[TOP ? wave : 0][at])[lane % EPV];
            const int64_t v = (int64_t)q * EPV + lane % EPV - lead;
            const lp_key_t key = i < n && q < to && v >= 0 && v < p.V ? spec_pack(spec_key((float)value), (int)v) : 0ull;
            if (picked.found(key) == 0) continue;
            if (picked.n > kLpRoom - 64) picked.keep(p.top);
            picked.add(key);
          }
          LpPicked::settle();
        }
        if (picked.floor != before && lane == 0) atomicMax(&bound, picked.floor);
      }
    }
  }
  // the wave's sums, then the workgroup's
  x.s = lp_wave_sum((s[0] + s[1]) + (s[2] + s[3]));
  if constexpr (ENTROPY) x.t = lp_wave_sum((t[0] + t[1]) + (t[2] + t[3]));
  if (__ballot(none) != 0) x.m = __builtin_nanf("");
  if (lane == 0) sums[wave] = x;
  // A round for the part, and, where a row has several, one for the row.
  LpSums own;  // of the lane's wave, then of its part
  [[maybe_unused]] lp_key_t key;  // of the thread, of the n numbers that the waves collected
  [[maybe_unused]] int n, above;  // and how many of those are larger
  for (int round = 1;; ++round) {
    if constexpr (TOP) {
      picked.end(counts[wave]);
    }
    __syncthreads();
    if constexpr (TOP) {
      int of[kLpWaves];
      const auto count = [&] {
        n = 0;
#pragma unroll
        for (int i = 0; i < kLpWaves; ++i) n += of[i] = __builtin_amdgcn_readfirstlane(counts[i]);
      };
      count();
      if (n > kLpThreads) {
        __syncthreads();
        if (picked.n > 64) picked.keep(p.top);  // (64 at most)
        picked.end(counts[wave]);
        __syncthreads();
        count();
      }
      int at = (int)threadIdx.x;
      key = 0;
      above = 0;
#pragma unroll
      for (int i = 0; i < kLpWaves; ++i) {
        if (at >= 0 && at < of[i]) key = room[i][at];
        at -= of[i];
      }
      if (64 * wave < n)
        for (int i = 0; i < kLpWaves; ++i) {
          const int many = __builtin_amdgcn_readfirstlane(counts[i]);
#pragma unroll 8
          for (int k = 0; k < many; k += 2) {  // (the same for all lanes: one read)
            const lp_pair_t two = *reinterpret_cast<const lp_pair_t*>(&room[i][k]);
            above += (two[0] > key) + (two[1] > key);
          }
        }
    }
    if (round == 1) own = lane < kLpWaves ? sums[lane] : LpSums{-__builtin_inff(), 0.f, 0.f, 0.f};
    x = lp_join<T>(own);
    if (round == 2 || p.split == 1) break;
    const int slot = lp_slot(p.top);
    uint64_t* mine = p.part + (int64_t)blockIdx.x * slot;
    const auto pack = [](float a, float b) {
      return (uint64_t)__builtin_bit_cast(uint32_t, a) | ((uint64_t)__builtin_bit_cast(uint32_t, b) << 32);
    };
    const auto put = [](uint64_t* at, uint64_t v) {
      __hip_atomic_store(at, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    };
    const auto get = [](const uint64_t* at) { return __hip_atomic_load(at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); };
    unsigned* counter = p.counters + row * kLpCounterStride;
    if (threadIdx.x == 0) {
      put(mine, pack(x.m, x.b));
      put(mine + 1, pack(x.s, x.t));
    }
    if constexpr (TOP) {
      if (key != 0 && above < 64) put(mine + 2 + above, key);
      if ((int)threadIdx.x >= n && threadIdx.x < 64) put(mine + 2 + threadIdx.x, 0ull);
    }
    // every wave's stores are performed at device scope before the count is
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0)
      last = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (unsigned)(p.split - 1);
    __syncthreads();
    if (!last) return;
    // the row's parts, a lane each; their numbers, a wave every fourth
    const uint64_t* parts = p.part + (int64_t)row * p.split * slot;
    const uint64_t* of = parts + min(lane, p.split - 1) * slot;
    const uint64_t mb = get(of), st = get(of + 1);
    if constexpr (TOP) {
      // Each part but the last has `top` numbers at least, so `top` reach the lowest of their q-th ones.
      const int q = (p.top + p.split - 2) / (p.split - 1);
      const uint64_t qth = get(parts + min(lane, p.split - 2) * slot + 2 + q - 1);
      lp_key_t ahead[kLpAhead];
      picked = LpPicked{room[wave], 0, 0, -__builtin_inff(), -__builtin_inff()};
      for (int i0 = wave; i0 < p.split; i0 += kLpAhead * kLpWaves) {
#pragma unroll
        for (int k = 0; k < kLpAhead; ++k) ahead[k] = get(parts + min(i0 + k * kLpWaves, p.split - 1) * slot + 2 + lane);
        if (i0 == wave) picked.raise((lp_key_t)lp_wave_min((uint32_t)(qth >> 32)) << 32);
        int more = 0;
#pragma unroll
        for (int k = 0; k < kLpAhead; ++k) {
          if (i0 + k * kLpWaves >= p.split) ahead[k] = 0;
          more += __builtin_popcountll(picked.found(ahead[k]));
        }
        if (picked.n + more > kLpRoom) picked.keep(p.top);
#pragma unroll
        for (int k = 0; k < kLpAhead; ++k) picked.add(ahead[k]);
      }
    }
    own = LpSums{-__builtin_inff(), 0.f, 0.f, 0.f};
    if (lane < p.split) {
      own.m = __builtin_bit_cast(float, (uint32_t)mb);
      own.b = __builtin_bit_cast(float, (uint32_t)(mb >> 32));
      own.s = __builtin_bit_cast(float, (uint32_t)st);
      own.t = __builtin_bit_cast(float, (uint32_t)(st >> 32));
    }
    if (threadIdx.x == 0) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  // a row without probabilities: something is no number, +inf, or all is -inf
  const float nan = __builtin_nanf("");
  const bool fine = x.m > -__builtin_inff() && x.m < __builtin_inff();
  const float log_s = logf(x.s), shift = fine ? log_s - lp_rounding(x.m, x.b, T{}) : nan;
  if (ENTROPY && threadIdx.x == 0) p.entropy[row] = fine ? log_s - kLn2 * (x.t / x.s) : nan;
  if constexpr (TOP) {
    const auto tell = [&](int place, int token, float value) {
      p.top_tokens[(int64_t)row * p.top + place] = token;
      p.top_logprobs[(int64_t)row * p.top + place] = value;
    };
    if (key != 0 && above < p.top) {
      const float value = __builtin_bit_cast(float, SpecBits<float>::value_of((uint32_t)(key >> 32)));
      tell(above, (int)(0xFFFFFFFFu - (uint32_t)key), (value - x.m) - shift);
    }
    if ((int)threadIdx.x >= n && (int)threadIdx.x < p.top) tell((int)threadIdx.x, -1, -__builtin_inff());  // behind the vocabulary
  }
  for (int i = (int)threadIdx.x; i < p.count; i += kLpThreads) {
    const int token = p.tokens[(int64_t)row * p.count + i];
    float lp = -__builtin_inff();
    if (token >= 0 && token < p.V) lp = ((float)logits[token] - x.m) - shift;
    p.logprob[(int64_t)row * p.count + i] = fine ? lp : nan;
  }
}

}  // namespace bq
