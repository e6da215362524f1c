// Launch interface of the attention-side kernels: per-head norm and rotation, the paged int8
// key/value cache, attention over it (declared for callers in include/tern.h).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/tern.h"

namespace tern {

// A cache and the sequences of a call, as the kernels take them.
struct KvView {
  int8_t* k;
  int8_t* v;
  float* ks;
  float* vs;
  int32_t pages, page_size, kv_heads;
  int32_t batch, rows, max_pages;
  const int32_t* row_start;
  const int32_t* kv_len;
  const int32_t* table;
  int32_t* flag;               // optional error flag
};

// Division of 0 <= n < 2^31 by a number fixed at launch: one multiply (Granlund and Montgomery, "Division
// by invariant integers using multiplication", PLDI 1994).
struct FastDiv {
  uint32_t d, mul, shift;
};
inline FastDiv fast_div(uint32_t d) {
  uint32_t lg = 0;
  while ((1ull << lg) < d) ++lg;
  // mul = floor(2^(31 + lg) / d) + 1, q = (n * mul) >> (31 + lg); d = 1: n * 2^31 / 2^31
  return FastDiv{d, (uint32_t)((1ull << (31 + lg)) / d) + (d > 1 ? 1u : 0u), lg};
}
#ifdef __CUDACC__
__device__ __forceinline__ int operator/(int n, const FastDiv& f) {
  return (int)(((unsigned long long)(uint32_t)n * f.mul) >> (31 + f.shift));
}
__device__ __forceinline__ int operator%(int n, const FastDiv& f) { return n - (n / f) * (int)f.d; }
#endif

struct QkvParams {
  const void* src;
  int64_t stride;              // elements
  int32_t q_heads, kv_heads;
  const uint16_t* q_gain;
  const uint16_t* k_gain;
  float eps;
  const double* freq;
  const int32_t* pos;          // without a cache
  uint16_t* q;
  uint16_t* k;                 // without a cache
  int32_t rows;
  KvView kv;                   // with a cache
};
// bf16: source type; append: into the cache, else to q and k rows.
cudaError_t launch_qkv(const QkvParams& p, int head_dim, bool bf16, bool append, bool pdl, cudaStream_t st);

struct KvReadParams {
  KvView kv;
  uint16_t* k;
  uint16_t* v;
  int32_t window;              // rows of a CTA, set by the launch
};
cudaError_t launch_kv_read(KvReadParams& p, int head_dim, cudaStream_t st);

struct AttnParams {
  KvView kv;
  const uint16_t* q;
  uint16_t* out;
  float* lse;                  // optional
  int32_t q_heads;
  FastDiv group, page, grid;   // q_heads / kv_heads, page_size, CTAs of the launch
  int32_t box;                 // tokens of a TMA box: the largest of 64, 32, 16 that divides page_size
  float scale;
  int32_t max_rows;
  uint8_t* ws;
};
size_t attn_workspace_bytes(int head_dim);
cudaError_t launch_attn(const AttnParams& p, int head_dim, bool pdl, cudaStream_t st);
cudaError_t read_and_clear_attn_latch(int* out);
cudaError_t read_and_clear_attn_tile_latch(int* out);

// One launch, optionally with programmatic stream serialisation (the kernel calls pdl_wait()).
template <typename P>
cudaError_t launch_maybe_pdl(void (*kern)(P), dim3 grid, dim3 block, size_t smem, bool pdl, cudaStream_t st, const P& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace tern
