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
// The largest values: a value and its token make one 64-bit number (a larger
// value first, then a lower token), all different.  A wave keeps its 64 largest
// sorted across its lanes, a lane one.  A new one is found by comparing the
// lane's maxima, which the softmax needs anyway, with the k-th largest that any
// wave of the workgroup has so far, and goes to its place by one shift across
// lanes; where many come at once (the first values, rows that rise) they are
// sorted and the two lists merged.  So ties and order change nothing but the
// time, and that by a bounded factor.
#pragma once

#include "kv_common.hpp"
#include "spec_kernels.hpp"

namespace bq {

constexpr int kLpWaves = 4, kLpThreads = 64 * kLpWaves;
constexpr int kLpLoads = 4;                              // 16-byte loads of a lane at a time
constexpr int kLpWaveBlocks = 64 * kLpLoads;             // 16-byte blocks a wave takes at a time
constexpr int kLpBlocks = kLpWaves * kLpWaveBlocks;      // and a workgroup
constexpr int kLpMaxSplit = 64;
constexpr int kLpCounterStride = 16;                     // 4-byte words: a line of its own for each row
constexpr int kLpSplitRows = BQ_LOGPROBS_COUNTER_BYTES / (4 * kLpCounterStride);
constexpr int kLpFew = 12;                               // new values that are put in one by one

struct LogprobsParams {
  const void* logits;
  int64_t row_stride;
  const int* tokens;
  float *logprob, *entropy, *top_logprobs;
  int* top_tokens;
  unsigned* counters;  // workspace: parts done of each row, zero between calls
  uint64_t* part;      // workspace: (m, B), (s, t), then `top` numbers, of each part
  int rows, V, count, top;
  int split;           // workgroups of a row
  int passes;          // of kLpBlocks that one of them makes
};
constexpr int lp_slot(int top) { return 2 + top; }  // 8-byte words of a part

typedef unsigned long long lp_key_t;

// Larger first across the wave's lanes: one step of a sorting network.
__device__ __forceinline__ lp_key_t lp_step(lp_key_t x, int d, bool up) {
  const lp_key_t y = __shfl_xor(x, d, 64);
  return (x > y) == up ? x : y;
}
// Sorts a sequence that rises and falls once (bitonic).
__device__ __forceinline__ lp_key_t lp_merge_steps(lp_key_t x) {
  const int lane = (int)threadIdx.x & 63;
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) x = lp_step(x, d, (lane & d) == 0);
  return x;
}
__device__ __forceinline__ lp_key_t lp_sort(lp_key_t x) {
  const int lane = (int)threadIdx.x & 63;
#pragma unroll
  for (int n = 2; n <= 64; n *= 2)
#pragma unroll
    for (int d = n >> 1; d > 0; d >>= 1) x = lp_step(x, d, ((lane & d) == 0) == ((lane & n) == 0 || n == 64));
  return x;
}
// The 64 largest of two sorted lists, sorted.
__device__ __forceinline__ lp_key_t lp_merge(lp_key_t a, lp_key_t b) {
  const lp_key_t r = __shfl(b, 63 - ((int)threadIdx.x & 63), 64);
  return lp_merge_steps(a > r ? a : r);
}
__device__ __forceinline__ lp_key_t lp_lane(lp_key_t x, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)x, lane), hi = __builtin_amdgcn_readlane((uint32_t)(x >> 32), lane);
  return ((lp_key_t)hi << 32) | lo;
}
// x (the same on all lanes) to its place in a sorted list; the last one leaves.
__device__ __forceinline__ lp_key_t lp_insert(lp_key_t list, lp_key_t x) {
  const int place = __builtin_popcountll(__ballot(list > x)), lane = (int)threadIdx.x & 63;
  // each lane's neighbour below (data parallel primitive: a shift over the wave)
  const uint32_t lo = __builtin_amdgcn_update_dpp(0u, (uint32_t)list, 0x138, 0xF, 0xF, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0u, (uint32_t)(list >> 32), 0x138, 0xF, 0xF, false);
  const lp_key_t up = ((lp_key_t)hi << 32) | lo;
  return lane < place ? list : lane == place ? x : up;
}

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
// Joins what `n` neighbouring lanes hold; the same result on each.
template <typename T>
__device__ __forceinline__ LpSums lp_join(LpSums x, int n) {
  float m = x.m;
  for (int d = n >> 1; d > 0; d >>= 1) m = lp_max(m, __shfl_xor(m, d, 64));
  const float b = lp_base(m, T{}), d = lp_moved(x.b, b, T{});
  lp_scale(x.s, x.t, d, x.m == -__builtin_inff() ? 0.f : __builtin_amdgcn_exp2f(d));
  x.m = m;
  x.b = b;
  for (int d = n >> 1; d > 0; d >>= 1) {
    x.s += __shfl_xor(x.s, d, 64);
    x.t += __shfl_xor(x.t, d, 64);
  }
  return x;
}

// One workgroup for a part of a row (of the whole row where rows fill the
// chip); a row's parts are joined by the one that finishes last.  The loads of
// a wave's next 4 KB are in flight while it works on the last.  Bound by HBM
// where rows are many, then by issue: of a value two conversions and sums, an
// exponential and a share of the maxima.  Measured: MEASURED_LP.
template <typename T, bool ENTROPY, bool TOP>
__global__ __launch_bounds__(kLpThreads) void logprobs_kernel(LogprobsParams p) {
  constexpr int EPV = 16 / (int)sizeof(T);  // values of a 16-byte block
  __shared__ lp_key_t lists[kLpWaves][64];
  __shared__ lp_key_t bound;  // no value below it is among the `top`
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

  LpSums x{-__builtin_inff(), 0.f, 0.f, 0.f};
  float s[kLpLoads] = {}, t[kLpLoads] = {};
  lp_key_t list = 0, own_bound = 0;
  float least = -__builtin_inff();  // the value of the bound
  bool none = false;                // something is no number
  if constexpr (TOP) {
    if (threadIdx.x == 0) bound = 0;
    __syncthreads();
  }
  u32x4_t next[kLpLoads];
  const auto request = [&](int q0) {
#pragma unroll
    for (int j = 0; j < kLpLoads; ++j) next[j] = blocks[min(q0 + 64 * j + lane, all - 1)];
  };
  int q0 = from + wave * kLpWaveBlocks;
  if (q0 < to) request(q0);
  for (; q0 < to; q0 += kLpBlocks) {
    u32x4_t w[kLpLoads];
#pragma unroll
    for (int j = 0; j < kLpLoads; ++j) w[j] = next[j];
    request(q0 + kLpBlocks);
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
      float m = __builtin_fmaxf(x.m, top);  // (a NaN counts for nothing here)
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) m = __builtin_fmaxf(m, __shfl_xor(m, d, 64));
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
      const lp_key_t others = *(volatile lp_key_t*)&bound;
      if (others > own_bound) {
        own_bound = others;
        least = __builtin_bit_cast(float, SpecBits<float>::value_of((uint32_t)(own_bound >> 32)));
      }
      if (__ballot(!(top < least)) != 0) {
        const lp_key_t before = own_bound;
        const auto raise = [&] {
          const lp_key_t k = lp_lane(list, p.top - 1);
          if (k > own_bound) {
            own_bound = k;
            least = __builtin_bit_cast(float, SpecBits<float>::value_of((uint32_t)(k >> 32)));
          }
        };
#pragma unroll
        for (int j = 0; j < kLpLoads; ++j) {
          if (__ballot(!(lp_float(most[j], T{}) < least)) == 0) continue;
          const int64_t v0 = (int64_t)(q0 + 64 * j + lane) * EPV - lead;
          const bool here = q0 + 64 * j + lane < to;
#pragma unroll
          for (int e = 0; e < EPV; ++e) {
            const float value = lp_value<T>(w[j], e);
            if (__ballot(!(value < least)) == 0) continue;
            const bool real = here && v0 + e >= 0 && v0 + e < p.V;
            lp_key_t key = real ? spec_pack(spec_key(value), (int)(v0 + e)) : 0ull;
            key = key > own_bound ? key : 0ull;
            uint64_t found = __ballot(key != 0);
            if (found == 0) continue;
            if (__builtin_popcountll(found) > kLpFew) {
              list = lp_merge(list, lp_sort(key));
              raise();
            } else {
              for (; found != 0; found &= found - 1) {
                const lp_key_t k = lp_lane(key, __builtin_ctzll(found));
                if (k <= own_bound) continue;
                list = lp_insert(list, k);
                raise();
              }
            }
          }
        }
        if (own_bound != before && lane == 0) atomicMax(&bound, own_bound);
      }
    }
  }
  // the wave's sums, then the workgroup's
  x.s = (s[0] + s[1]) + (s[2] + s[3]);
  if constexpr (ENTROPY) x.t = (t[0] + t[1]) + (t[2] + t[3]);
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    x.s += __shfl_xor(x.s, d, 64);
    if constexpr (ENTROPY) x.t += __shfl_xor(x.t, d, 64);
  }
  if (__ballot(none) != 0) x.m = __builtin_nanf("");
  if (lane == 0) sums[wave] = x;
  if constexpr (TOP) lists[wave][lane] = list;
  __syncthreads();
  if (wave == 0) {
    x = lp_join<T>(sums[lane & (kLpWaves - 1)], kLpWaves);
    if constexpr (TOP) {
      list = lists[0][lane];
#pragma unroll
      for (int i = 1; i < kLpWaves; ++i) list = lp_merge(list, lists[i][lane]);
    }
  }
  if (p.split > 1) {
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
    if (wave == 0) {
      if (lane == 0) {
        put(mine, pack(x.m, x.b));
        put(mine + 1, pack(x.s, x.t));
      }
      if (TOP && lane < p.top) put(mine + 2 + lane, list);
      // the stores are performed at device scope before the count is
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      if (lane == 0)
        last = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (unsigned)(p.split - 1);
    }
    __syncthreads();
    if (!last) return;
    // the row's parts, a lane each; their lists, a wave every fourth, in order
    const uint64_t* parts = p.part + (int64_t)row * p.split * slot;
    x = LpSums{-__builtin_inff(), 0.f, 0.f, 0.f};
    if (wave == 0 && lane < p.split) {
      const uint64_t a = get(parts + lane * slot), b = get(parts + lane * slot + 1);
      x.m = __builtin_bit_cast(float, (uint32_t)a);
      x.b = __builtin_bit_cast(float, (uint32_t)(a >> 32));
      x.s = __builtin_bit_cast(float, (uint32_t)b);
      x.t = __builtin_bit_cast(float, (uint32_t)(b >> 32));
    }
    if constexpr (TOP) {
      list = 0;
      for (int i = wave; i < p.split; i += kLpWaves) {
        const lp_key_t other = lane < p.top ? get(parts + i * slot + 2 + lane) : 0ull;
        list = i == wave ? other : lp_merge(list, other);
      }
      lists[wave][lane] = list;
      __syncthreads();
    }
    if (wave == 0) {
      x = lp_join<T>(x, 64);
      if constexpr (TOP) {
#pragma unroll
        for (int i = 1; i < kLpWaves; ++i) list = lp_merge(list, lists[i][lane]);
      }
    }
    if (threadIdx.x == 0) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (wave == 0 && lane == 0) sums[0] = x;
  __syncthreads();
  x = sums[0];
  // a row without probabilities: something is no number, +inf, or all is -inf
  const float nan = __builtin_nanf("");
  const bool fine = x.m > -__builtin_inff() && x.m < __builtin_inff();
  const float log_s = logf(x.s), shift = fine ? log_s - lp_rounding(x.m, x.b, T{}) : nan;
  if (ENTROPY && threadIdx.x == 0) p.entropy[row] = fine ? log_s - kLn2 * (x.t / x.s) : nan;
  if (TOP && wave == 0 && lane < p.top) {
    const float value = __builtin_bit_cast(float, SpecBits<float>::value_of((uint32_t)(list >> 32)));
    p.top_tokens[(int64_t)row * p.top + lane] = list != 0 ? (int)(0xFFFFFFFFu - (uint32_t)list) : -1;
    p.top_logprobs[(int64_t)row * p.top + lane] = list != 0 ? (value - x.m) - shift : -__builtin_inff();
  }
  for (int i = (int)threadIdx.x; i < p.count; i += kLpThreads) {
    const int token = p.tokens[(int64_t)row * p.count + i];
    float lp = -__builtin_inff();
    if (token >= 0 && token < p.V) lp = ((float)logits[token] - x.m) - shift;
    p.logprob[(int64_t)row * p.count + i] = fine ? lp : nan;
  }
}

}  // namespace bq
