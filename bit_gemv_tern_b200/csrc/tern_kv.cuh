// Device helpers of the attention-side kernels: the sequences of a call, checked.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "tern_kernels.h"
#include "tern_kv.h"

namespace tern {

// The smallest block scale: a power of two far below any value in use, so that a block of zeros
// needs no case of its own (1/s is finite and the codes are 0).
constexpr float kKvScaleFloor = 8.673617379884035e-19f;      // 2^-60

// What a call reads may have been written by the kernel just before it, beside which programmatic dependent launch
// starts it: nothing of it goes through the non-coherent path (ld.global.nc).

// Sequence b's rows and tokens, and whether the call can use them.
struct SeqInfo {
  int start, n, len;
  bool ok;
};
__device__ __forceinline__ SeqInfo seq_info(const KvView& kv, int b) {
  SeqInfo s;
  const int e = kv.row_start[b + 1];
  s.start = kv.row_start[b];
  s.len = kv.kv_len[b];
  s.ok = s.start >= 0 && e >= s.start && e <= kv.rows && s.len >= 0 && s.len <= kv.max_pages * kv.page_size;
  s.n = s.ok ? e - s.start : 0;
  return s;
}

// seq[i] = the sequence that owns row w0 + i, or -1 (nobody's, or a sequence that is left out).
// need_tokens: every row must be a token of the cache (kv_len >= n). Ends with a barrier.
template <int kThreadsT>
__device__ __forceinline__ void locate_rows(const KvView& kv, int w0, int wn, bool need_tokens, int* seq) {
  for (int i = threadIdx.x; i < wn; i += kThreadsT) seq[i] = -1;
  __syncthreads();
  for (int b = threadIdx.x; b < kv.batch; b += kThreadsT) {
    const SeqInfo s = seq_info(kv, b);
    if (!s.ok || (need_tokens && s.len < s.n)) {
      if (kv.flag) *kv.flag = 1;
      continue;
    }
    for (int r = max(s.start, w0); r < min(s.start + s.n, w0 + wn); ++r) seq[r - w0] = b;
  }
  __syncthreads();
}

}  // namespace tern
