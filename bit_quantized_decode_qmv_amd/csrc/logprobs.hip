// C entry points of the log probabilities.  Declarations are in include/bq.h.
#include <algorithm>

#include "logprobs_kernels.hpp"

namespace {

using namespace bq;

template <typename T>
const void* pick(bool entropy, bool top) {
  return entropy ? top ? reinterpret_cast<const void*>(&logprobs_kernel<T, true, true>)
                       : reinterpret_cast<const void*>(&logprobs_kernel<T, true, false>)
                 : top ? reinterpret_cast<const void*>(&logprobs_kernel<T, false, true>)
                       : reinterpret_cast<const void*>(&logprobs_kernel<T, false, false>);
}

int check_sizes(int rows, int V, int logits_dtype, int top) {
  if (logits_dtype != BQ_DTYPE_F16 && logits_dtype != BQ_DTYPE_F32) return BQ_ERR_BITS;
  if (rows < 0 || rows >= (1 << 24) || V < 1 || V >= (1 << 28) || top < 0 || top > BQ_LOGPROBS_MAX_TOP) return BQ_ERR_SHAPE;
  return BQ_OK;
}

// Workgroups of a row, and the passes of each: as many as bring the call to
// kTarget workgroups, no more than a row has passes (a value may start
// anywhere in a 16-byte block) or `room` holds.  Measured, us with 512, 1024 and
// 2048: 301 rows of 151936 in fp16, top 5, 33.4, 30.6 and 30.8, 700 rows of 50000
// 23.4, 23.5 and 29.1 (a part costs its first pass's barrier, its list and its
// share of the join); 5 rows of 151936 and 301 of 32000 in fp32 alike.
constexpr int kTarget = 1024;
struct Split {
  int split, passes;
};
Split split_of(int rows, int V, int logits_dtype, int64_t room) {
  const int64_t blocks = ((int64_t)V * (logits_dtype == BQ_DTYPE_F16 ? 2 : 4) + 15 + 15) / 16;
  const int passes = (int)((blocks + kLpBlocks - 1) / kLpBlocks);
  int split = 1;
  if (rows > 0 && rows <= kLpSplitRows)
    split = (int)std::min<int64_t>({std::max((kTarget + rows / 2) / rows, 1), passes, kLpMaxSplit, std::max<int64_t>(room / rows, 1)});
  const int each = (passes + split - 1) / split;
  return Split{(passes + each - 1) / each, each};
}

}  // namespace

extern "C" {

int bq_logprobs_workspace(int rows, int V, int logits_dtype, int top, size_t* bytes) {
  if (!bytes) return BQ_ERR_NULL;
  *bytes = 0;
  const int st = check_sizes(rows, V, logits_dtype, top);
  if (st != BQ_OK) return st;
  const Split s = split_of(rows, V, logits_dtype, INT64_MAX);
  if (s.split > 1) *bytes = BQ_LOGPROBS_COUNTER_BYTES + (size_t)rows * s.split * lp_slot(top) * 8;
  return BQ_OK;
}

int bq_logprobs(const void* logits, int logits_dtype, long long row_stride, int rows, int V, const int* tokens,
                int count, float* logprob, float* entropy, int top, int* top_tokens, float* top_logprobs,
                void* workspace, size_t workspace_bytes, void* stream) {
  const int st = check_sizes(rows, V, logits_dtype, top);
  if (st != BQ_OK) return st;
  if (count < 0 || count > BQ_LOGPROBS_MAX_COUNT || row_stride < V || (count == 0 && !entropy && top == 0))
    return BQ_ERR_SHAPE;
  if (rows > 0 && (!logits || (count > 0 && (!tokens || !logprob)) || (top > 0 && (!top_tokens || !top_logprobs))))
    return BQ_ERR_NULL;
  if (!kv_aligned(logits, logits_dtype == BQ_DTYPE_F16 ? 2 : 4) || !kv_aligned(tokens, 4) || !kv_aligned(logprob, 4) ||
      !kv_aligned(entropy, 4) || !kv_aligned(top_tokens, 4) || !kv_aligned(top_logprobs, 4) || !kv_aligned(workspace, 16))
    return BQ_ERR_ALIGN;
  if (rows == 0) return BQ_OK;
  int64_t room = 0;
  if (workspace && workspace_bytes > BQ_LOGPROBS_COUNTER_BYTES)
    room = (int64_t)((workspace_bytes - BQ_LOGPROBS_COUNTER_BYTES) / (lp_slot(top) * 8));
  const Split s = split_of(rows, V, logits_dtype, room);
  LogprobsParams p{};
  p.logits = logits;
  p.row_stride = row_stride;
  p.tokens = tokens;
  p.logprob = logprob;
  p.entropy = entropy;
  p.top_logprobs = top_logprobs;
  p.top_tokens = top_tokens;
  p.counters = static_cast<unsigned*>(workspace);
  p.part = workspace ? reinterpret_cast<uint64_t*>(static_cast<char*>(workspace) + BQ_LOGPROBS_COUNTER_BYTES) : nullptr;
  p.rows = rows;
  p.V = V;
  p.count = count;
  p.top = top;
  p.split = s.split;
  p.passes = s.passes;
  const void* fn = logits_dtype == BQ_DTYPE_F16 ? pick<_Float16>(entropy != nullptr, top > 0) : pick<float>(entropy != nullptr, top > 0);
  return kv_launch(fn, dim3((unsigned)(rows * s.split)), dim3(kLpThreads), 0, stream, &p);
}

}  // extern "C"
