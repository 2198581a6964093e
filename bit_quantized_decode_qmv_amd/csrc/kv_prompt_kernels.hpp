// Attention of many rows over the paged 8-bit cache: a prompt's chunk, a
// whole prompt, or queries over an encoder's states.
//
// The same products as for few rows (S^T = K Q^T, O^T += V^T P^T, 32 rows a
// wave).  What differs is the sharing: a workgroup's four waves take 128
// rows and walk the pages together, so that a page's codes are read and
// turned into fp16 once for all of them.  The fp16 operands go through LDS in
// the order in which the waves read them back (16 bytes a lane, consecutive:
// no bank is hit twice); the next page's codes are in flight meanwhile, and
// two workgroups share a CU where their registers and LDS allow, one in its
// products while the other is in its softmax.
//
// The probabilities are rounded to fp16 (nearest even) once, with V's block
// scale folded in: by up to 2^-11 of each, 2^-12 on average, as the rounding of
// the result, or by 2^-32 of the outputs' unit (kKvLift, kv_in_unit).
// Their sum is taken of the rounded ones, so that a row that sees few tokens
// does not keep the rounding of a common factor.
//
// Bound by issue: a wave's page of 128 dimensions is 68 matrix instructions
// (1090 cycles), some 220 vector instructions (1350, a quarter of them for
// the exponentials) and 32 reads of LDS (256 of the CU's), of two waves a
// SIMD.  Measured: 2047 rows of 48 heads (8 of them keys' and values') of 128
// over 10240 tokens 485 us, 0.96 PFLOP/s, in a run of calls (the first ten
// after a pause take up to 620, and the time falls over the next fifty); the
// matrix instructions alone 200, without the softmax 334.  One wave a SIMD with
// 64 rows reads LDS half as often, and took 714 us; eight waves with 256 rows
// 474 before other steps, but 10 to 40% more where prompts are short.
#pragma once

#include "kv_attn_kernels.hpp"

namespace bq {

// The order of a product whose operands come from LDS: AHEAD reads first,
// then one more after the two matrix instructions that share one, so that
// none waits for the read just issued.
// `more` matrix instructions that need none of the reads come first.
template <int READS, int MORE = 0>
__device__ __forceinline__ void kv_order_reads() {
  constexpr int AHEAD = READS < 16 ? READS / 2 : 8;
  __builtin_amdgcn_sched_group_barrier(0x100, AHEAD, 0);  // LDS reads
  if constexpr (MORE > 0) __builtin_amdgcn_sched_group_barrier(0x008, MORE, 0);
#pragma unroll
  for (int i = 0; i < READS - AHEAD; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);  // matrix instructions
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, 2 * AHEAD, 0);
}

// Wide heads, whose registers are two files: o stays in the accumulation
// registers and the scores (ACC false) in the others.  What only a rarely
// taken branch changes is otherwise copied to and fro on every page, and
// spills (head_dim 256, 500 rows over 4000 tokens: 124 us and 90).
template <int D, bool ACC = true>
__device__ __forceinline__ void kv_stay(f32x4& x) {
  if constexpr (D > 128) {
    if constexpr (ACC) asm volatile("" : "+a"(x));
    else asm volatile("" : "+v"(x));
  }
}

constexpr int kPromptWaves = 4, kPromptThreads = 64 * kPromptWaves;
constexpr int kPromptRows = 32 * kPromptWaves;

template <int D, int FMT>
__global__ __launch_bounds__(kPromptThreads, D <= 128 ? 2 : 1) void kv_attn_prompt_kernel(KvAttnParams p) {
  constexpr int C = D / 64, N = D / 16, UNITS = 4 * D / kPromptThreads;  // 16-byte units of K (or V) a thread
  constexpr bool BYTES = FMT == BQ_KV_I8;
  // [buffer][K, V][operand][lane][8]
  __shared__ __align__(16) half8_t lds[2][2][8 * C][64];
  const int lane = (int)threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int head = (int)blockIdx.x;
  const int item = p.item0 + (int)blockIdx.y;
  KvWork w;
  if (!kv_attn_work<kPromptRows>(p, item, w)) return;
  const KvSeq s = w.s;
  const int rows = s.n * p.group;
  const int row0 = w.tile * kPromptRows, row1 = min(row0 + kPromptRows, rows) - 1;
  const KvRowRange r0 = kv_row_range(p, s, row0 / p.group), r1 = kv_row_range(p, s, row1 / p.group);
  const int pa = r0.lo / kKvPage, pages = max((r1.hi + kKvPage - 1) / kKvPage - pa, 0);
  const int begin = pa + (w.parts > 1 ? w.split * w.chunk : 0);
  const int end = pa + (w.split == w.parts - 1 ? pages : min((w.split + 1) * w.chunk, pages));

  KvPages pages_of;
  const auto place = [&](int k) -> int64_t {
    const int page = pages_of.at(p, w.b, begin, 1, end, k);
    return page < 0 ? -1 : (int64_t)page * p.kv_heads + head;
  };
  // a page's scales are requested ahead of its codes: what waits for them
  // does not wait for the codes
  f32x4 sk_next, sv_next;
  u32x4_t raw[2][UNITS];
  const auto request = [&](int64_t at) {
    sk_next = *reinterpret_cast<const f32x4*>(p.ks + max(at, (int64_t)0) * kKvBlocks);
    sv_next = *reinterpret_cast<const f32x4*>(p.vs + max(at, (int64_t)0) * kKvBlocks);
    const kv_rsrc_t rk = kv_rsrc(p.k + max(at, (int64_t)0) * (kKvPage * D), at < 0 ? 0 : kKvPage * D);
    const kv_rsrc_t rv = kv_rsrc(p.v + max(at, (int64_t)0) * (kKvPage * D), at < 0 ? 0 : kKvPage * D);
#pragma unroll
    for (int j = 0; j < UNITS; ++j) {
      raw[0][j] = __builtin_amdgcn_raw_buffer_load_b128(rk, (int)threadIdx.x * 16, j * kPromptThreads * 16, 0);
      raw[1][j] = __builtin_amdgcn_raw_buffer_load_b128(rv, (int)threadIdx.x * 16, j * kPromptThreads * 16, 0);
    }
  };
  // codes at hand to buffer `to`; `left` tokens of the page are held
  const auto stage = [&](int to, int left) {
#pragma unroll
    for (int j = 0; j < UNITS; ++j) {
      const int unit = (int)threadIdx.x + j * kPromptThreads, op = unit >> 6, ln = unit & 63;
      if (FMT == BQ_KV_E4M3 && left < kKvPage) {
        // what lies past the length may be no number: cleared
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int keep = min(max(left - 16 * i - 4 * (ln >> 4), 0), 4);
          raw[1][j][i] &= keep == 4 ? 0xFFFFFFFFu : (1u << (8 * keep)) - 1u;
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        lds[to][x][2 * op][ln] = kv_operand8<FMT, BYTES>(raw[x][j][0], raw[x][j][1]);
        lds[to][x][2 * op + 1][ln] = kv_operand8<FMT, BYTES>(raw[x][j][2], raw[x][j][3]);
      }
    }
  };
  int64_t here = place(0);
  request(here);

  // this wave's rows
  half8_t q[2][2 * C];
  int lo[2], hi[2];
  int wave_lo = 0, wave_hi = 0;  // tokens that some row of the wave sees
  int all_lo = 0, all_hi = 0;    // that all of them see
  {
    const int first = row0 + 32 * wave, last = min(first + 31, rows - 1);
    if (first < rows) {
      const KvRowRange a = kv_row_range(p, s, first / p.group), b = kv_row_range(p, s, last / p.group);
      wave_lo = a.lo;
      wave_hi = b.hi;
      all_lo = b.lo;
      all_hi = a.hi;
    }
  }
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int row = row0 + 32 * wave + 16 * t + r;
    const bool ok = row < rows;
    const int token = ok ? row / p.group : 0, qh = head * p.group + (ok ? row - token * p.group : 0);
    const KvRowRange range = kv_row_range(p, s, token);
    lo[t] = range.lo;
    hi[t] = ok ? range.hi : 0;
    const _Float16* src = p.q + (int64_t)(s.q0 + token) * p.q_stride + qh * D + 16 * g;
#pragma unroll
    for (int c = 0; c < 2 * C; ++c) {
      q[t][c] = ok ? *reinterpret_cast<const half8_t*>(src + (c >> 1) * 64 + (c & 1) * 8) : half8_t{};
      if (p.scale < 0.f) q[t][c] = -q[t][c];
    }
  }
  const float scale = __builtin_fabsf(p.scale) * kKvUnit<BYTES>;
  f32x4 q_off[2];  // what the offset of the codes adds to every score: where the sums begin
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const float off = kv_query_offset<BYTES>(q[t]);
    q_off[t] = f32x4{off, off, off, off};
  }

  f32x4 o[2][N];
  // Sums over the rounded probabilities, by the matrix cores: rows 4g + e of
  // one more operand hold, e = 0, V's code offset (since it was last taken
  // off o) and, 1 and 2, the two fp16 terms of what takes V's scale out again.
  f32x4 sums[2];
  const int term = lane & 3;
  const float pick_all = term == 2 ? 1.f : 0.f, pick_hi = term == 1 ? 1.f : term == 2 ? -1.f : 0.f;
  const float pick_off = term == 0 ? kKvOffset<BYTES> : 0.f;
  float m[2], l[2], base[2];  // base: what is taken off a score, the maximum less kKvLift, 0 while there is none
  bool fresh = true;          // some row has seen nothing yet
  int unit_ex = kKvLeastUnit;  // of R, the unit of o
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    m[t] = row0 + 32 * wave + 16 * t + r < rows ? -__builtin_inff() : 0.f;
    l[t] = base[t] = 0.f;
    sums[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int n = 0; n < N; ++n) o[t][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  stage(0, here < 0 ? 0 : s.len - begin * kKvPage);
  __syncthreads();
  for (int at = begin; at < end; ++at) {
    const int buf = (at - begin) & 1;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int n = 0; n < N; ++n) kv_stay<D>(o[t][n]);
    const int64_t next = place(at + 1 - begin);
    const f32x4 sk = sk_next;
    f32x4 sv = sv_next;
    request(next);
    const int j0 = at * kKvPage, left = here < 0 ? 0 : s.len - j0;

    if (j0 < wave_hi && j0 + kKvPage > wave_lo) {
      f32x4 y[2][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[0][i] = q_off[0];
        y[1][i] = q_off[1];
#pragma unroll
        for (int c = 0; c < 2 * C; ++c) {
          const half8_t a = lds[buf][0][2 * C * i + c][lane];
          y[0][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, q[0][c], y[0][i], 0, 0, 0);
          y[1][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, q[1][c], y[1][i], 0, 0, 0);
        }
      }
      kv_order_reads<8 * C>();
#pragma unroll
      for (int i = 0; i < 4; ++i) kv_stay<D, false>(y[0][i]), kv_stay<D, false>(y[1][i]);
      f32x4 c = sk * scale;
      if (left < kKvPage || j0 + kKvPage > all_hi || j0 < all_lo) {
        // a page that some row does not see whole; a block past the length
        // has no scale (its probabilities are 0 under any)
        int held = left;
        asm volatile("" : "+s"(held));  // stays in this branch
        if (held < kKvPage) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (16 * i >= held) {
              c[i] = 0.f;
              sv[i] = held > 0 ? sv[0] : kv_exp_float(unit_ex);
            }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int from = max(lo[t] - j0, 0), count = max(min(hi[t] - j0, left) - from, 0);
          int in = 4 * g - from;
          asm volatile("" : "+v"(in));
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              y[t][i][e] = (unsigned)(in + 16 * i + e) < (unsigned)count ? y[t][i][e] * c[i] : -__builtin_inff();
        }
        c = f32x4{1.f, 1.f, 1.f, 1.f};  // a hidden score times 0 would be no number
      }
      // V's scales in units of R: they go into the exponent.
      f32x4 unit = sv * kv_exp_float(254 - unit_ex), log_unit;
#pragma unroll
      for (int i = 0; i < 4; ++i) log_unit[i] = __builtin_amdgcn_logf(unit[i]);
      half8_t pb[2][2];
      const auto weigh = [&] {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              pb[t][i >> 1][(i & 1) * 4 + e] = (_Float16)kv_exp2(__builtin_fmaf(y[t][i][e], c[i], log_unit[i] - base[t]));
      };
      // The maximum stays as it is unless a probability, in V's units, passes
      // 2^8 (2^15 as it is held): found on the packed ones, which are half as
      // many as the scores.
      // Where V's scales leave R's range (fine false) R is fitted to them and
      // the scores are looked at: a block of V far below the others would hide
      // how large the probability itself is.
      const float low = kv_min4(unit), most_unit = kv_max4(unit);
      bool fine = __builtin_amdgcn_readfirstlane(kv_in_unit(low, most_unit));
      // (Only then does o begin from what may be negative: until then it and
      // the offset's sum are rounded alike, and a value of 0 comes back as 0.)
      const bool take_off = BYTES && at % kKvOffsetPages == 0;
      bool raise = fresh || !fine || take_off;
      if (!raise) {
        weigh();
        uint32_t top = 0;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const u32x4_t w = __builtin_bit_cast(u32x4_t, pb[t][h]);
            top = kv_pk_max3(kv_pk_max3(top, w[0], w[1]), w[2], w[3]);
          }
        raise = __ballot(top > 0x7800FFFFu || (top & 0xFFFFu) > 0x7800u) != 0;
      }
      if (raise) {
        fresh = false;
        float alpha[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          float mx = -__builtin_inff();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float most = kv_max3(kv_max3(y[t][i][0], y[t][i][1], y[t][i][2]), y[t][i][3], y[t][i][3]);
            mx = __builtin_fmaxf(mx, most * c[i]);
          }
          const float mn = __builtin_fmaxf(m[t], kv_col_max(mx));
          alpha[t] = mn == -__builtin_inff() ? 1.f : kv_exp2(m[t] - mn);
          m[t] = mn;
          base[t] = mn == -__builtin_inff() ? 0.f : mn - kKvLift;
          fresh = fresh || __ballot(mn == -__builtin_inff()) != 0;
          l[t] *= alpha[t];
        }
        float change = 1.f;
        if (!fine) {
          change = kv_fit_unit(
              unit, low, most_unit,
              [&] {  // rows past the last one (hi 0) and those that have seen nothing have no terms
                float most = -__builtin_inff();
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const float term = kv_max4(y[t][i]) * c[i] + log_unit[i] - m[t];
                    most = hi[t] > 0 && m[t] > -__builtin_inff() ? __builtin_fmaxf(most, term) : most;
                  }
                return kv_wave_max(most);
              },
              unit_ex);
#pragma unroll
          for (int i = 0; i < 4; ++i) log_unit[i] = __builtin_amdgcn_logf(unit[i]);
          fine = __builtin_amdgcn_readfirstlane(kv_min4(unit) >= 0x1p-6f && kv_max4(unit) <= 0x1p6f);
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float f = alpha[t] * change, off = take_off ? sums[t][0] : 0.f;
#pragma unroll
          for (int n = 0; n < N; ++n) {
            kv_stay<D>(o[t][n]);
            o[t][n] = BYTES ? (o[t][n] - off) * f : o[t][n] * f;
            kv_stay<D>(o[t][n]);
          }
          sums[t] = f32x4{(sums[t][0] - off) * f, sums[t][1] * alpha[t], sums[t][2] * alpha[t], 0.f};
        }
        weigh();
      }
      // what the sums' operand holds for the tokens of block i
      u32x4_t per;
      if (fine) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float back = __builtin_amdgcn_rcpf(unit[i]);
          const float hi = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, back) & 0xFFFFE000u);
          const float v = __builtin_fmaf(back, pick_all, __builtin_fmaf(hi, pick_hi, pick_off));
          per[i] = __builtin_bit_cast(uint32_t, half2_t{(_Float16)v, (_Float16)v});
        }
      } else {
        // the rounded probabilities of such a block say too little of their sum
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) l[t] += kv_exp2(__builtin_fmaf(y[t][i][e], c[i], -base[t]));
        const uint32_t off = __builtin_bit_cast(uint32_t, half2_t{(_Float16)pick_off, (_Float16)pick_off});
        per = u32x4_t{off, off, off, off};
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const half8_t a = __builtin_bit_cast(half8_t, u32x4_t{per[2 * h], per[2 * h], per[2 * h + 1], per[2 * h + 1]});
        sums[0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, pb[0][h], sums[0], 0, 0, 0);
        sums[1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, pb[1][h], sums[1], 0, 0, 0);
      }
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const half8_t a = lds[buf][1][2 * n + h][lane];
          o[0][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, pb[0][h], o[0][n], 0, 0, 0);
          o[1][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, pb[1][h], o[1][n], 0, 0, 0);
        }
      kv_order_reads<2 * N, 4>();
    }
    stage(buf ^ 1, next < 0 ? 0 : s.len - j0 - kKvPage);
    here = next;
    __syncthreads();
  }

  constexpr int SLOT = kv_part_floats(kPromptRows, D);
  float* mine = p.part + ((int64_t)(w.slot + w.split) * p.kv_heads + head) * SLOT;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const float sum = kv_col_sum(l[t]) + (sums[t][1] + sums[t][2]);
    const float unit = kv_exp_float(unit_ex) * kKvUnit<BYTES>;  // of o
    const int in = 32 * wave + 16 * t + r, row = row0 + in;
    if (row >= rows) continue;
    if (w.parts == 1) {
      const int token = row / p.group, qh = head * p.group + row - token * p.group;
      const float inv = sum > 0.f ? unit / sum : 0.f;  // nothing seen: zeros
      _Float16* dst = p.out + (int64_t)(s.q0 + token) * p.out_stride + qh * D + 4 * g;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const f32x4 v = (o[t][n] - sums[t][0]) * inv;
        *reinterpret_cast<half4_t*>(dst + 16 * n) = half4_t{(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]};
      }
    } else {
      if (g == 0) *reinterpret_cast<float2*>(mine + 2 * in) = make_float2(m[t], sum);
#pragma unroll
      for (int n = 0; n < N; ++n) *reinterpret_cast<f32x4*>(mine + 2 * kPromptRows + in * D + 16 * n + 4 * g) =
            (o[t][n] - sums[t][0]) * unit;
    }
  }
}

// Joins the parts of the tiles that have several, in order; a workgroup takes
// 16 rows of a tile.
template <int D>
__global__ __launch_bounds__(256) void kv_attn_join_kernel(KvAttnParams p) {
  constexpr int SLOT = kv_part_floats(kPromptRows, D);
  __shared__ float f[kKvMaxParts][16];
  const int head = (int)blockIdx.x, item = (int)blockIdx.y / (kPromptRows / 16), first = (int)blockIdx.y % (kPromptRows / 16) * 16;
  KvWork w;
  if (!kv_attn_work<kPromptRows, true>(p, item, w) || w.parts == 1) return;
  const KvSeq s = w.s;
  const int row0 = w.tile * kPromptRows + first, some = min(16, s.n * p.group - row0);
  if (some <= 0) return;
  const int64_t next = (int64_t)p.kv_heads * SLOT;
  const float* part0 = p.part + ((int64_t)w.slot * p.kv_heads + head) * SLOT;
  // 16 lanes a row
  const int row = (int)threadIdx.x >> 4, sub = (int)threadIdx.x & 15;
  float mx = -__builtin_inff(), sum = 0.f;
  if (row < some) {
    for (int i = sub; i < w.parts; i += 16) mx = __builtin_fmaxf(mx, part0[i * next + 2 * (first + row)]);
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) mx = __builtin_fmaxf(mx, __shfl_xor(mx, d, 64));
    const float base = mx == -__builtin_inff() ? 0.f : mx;
    for (int i = sub; i < w.parts; i += 16) {
      const float2 ml = *reinterpret_cast<const float2*>(part0 + i * next + 2 * (first + row));
      const float e = kv_exp2(ml.x - base);
      f[i][row] = e;
      sum += ml.y * e;
    }
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) sum += __shfl_xor(sum, d, 64);
  }
  __syncthreads();
  if (row >= some) return;
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  const int token = (row0 + row) / p.group, qh = head * p.group + row0 + row - token * p.group;
  _Float16* dst = p.out + (int64_t)(s.q0 + token) * p.out_stride + qh * D;
#pragma unroll
  for (int d = 4 * sub; d < D; d += 64) {
    f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int i = 0; i < w.parts; ++i)
      y += *reinterpret_cast<const f32x4*>(part0 + i * next + 2 * kPromptRows + (first + row) * D + d) * f[i][row];
    y *= inv;
    *reinterpret_cast<half4_t*>(dst + d) = half4_t{(_Float16)y[0], (_Float16)y[1], (_Float16)y[2], (_Float16)y[3]};
  }
}

}  // namespace bq
