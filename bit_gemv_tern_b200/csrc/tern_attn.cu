// Attention over the paged int8 cache (include/tern.h, tern_paged_attn).
//
// One warp per row and query head walks the row's tokens with the running maximum and sum of the
// softmax; a lane holds D/32 elements of the head.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "tern_device.cuh"
#include "tern_kv.cuh"
#include "tern_kv.h"

namespace tern {
namespace {

template <int D>
__global__ void __launch_bounds__(128) k_attn_rows(const __grid_constant__ AttnParams p) {
  constexpr int E = D / 32;
  __shared__ int seq[1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x;
  pdl_wait();
  locate_rows<128>(p.kv, row, 1, false, seq);
  const int b = seq[0];
  if (b < 0) return;
  const SeqInfo si = seq_info(p.kv, b);
  const int pos = si.len - (si.start + si.n - row);
  for (int h = blockIdx.y * 4 + warp; h < p.q_heads; h += gridDim.y * 4) {
    const int hk = h / p.group;
    float q[E], o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      q[e] = bf16_bits_to_float(p.q[((int64_t)row * p.q_heads + h) * D + lane * E + e]) * p.scale;
      o[e] = 0.0f;
    }
    float m = -INFINITY, l = 0.0f;
    for (int j = 0; j <= pos; ++j) {
      const int page = __ldg(p.kv.table + (int64_t)b * p.kv.max_pages + j / p.kv.page_size);
      if (page < 0 || page >= p.kv.pages) {
        if (p.kv.flag && lane == 0) *p.kv.flag = 1;
        continue;
      }
      const int place = j % p.kv.page_size;
      const int64_t head = (int64_t)page * p.kv.kv_heads + hk, at = (head * p.kv.page_size + place) * D + lane * E;
      const int64_t blk = head * (p.kv.page_size / TERN_KV_BLOCK) + place / TERN_KV_BLOCK;
      float s = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) s += q[e] * (float)p.kv.k[at + e];
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
      s *= p.kv.ks[blk];
      const float mn = fmaxf(m, s), f = expf(m - mn), w = expf(s - mn), vs = p.kv.vs[blk];
      l = l * f + w;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = o[e] * f + w * (vs * (float)p.kv.v[at + e]);
      m = mn;
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
      *reinterpret_cast<__nv_bfloat16*>(p.out + ((int64_t)row * p.q_heads + h) * D + lane * E + e) =
          __float2bfloat16_rn(l > 0.0f ? o[e] / l : 0.0f);
    if (p.lse && lane == 0) p.lse[(int64_t)row * p.q_heads + h] = m + logf(l);
  }
}

}  // namespace

size_t attn_workspace_bytes(int head_dim) { return 1024; }

cudaError_t launch_attn(const AttnParams& p, int head_dim, bool pdl, cudaStream_t st) {
  const dim3 grid(p.kv.rows, (p.q_heads + 3) / 4);
  return head_dim == 128 ? launch_maybe_pdl(k_attn_rows<128>, grid, dim3(128), 0, pdl, st, p)
                         : launch_maybe_pdl(k_attn_rows<64>, grid, dim3(128), 0, pdl, st, p);
}

}  // namespace tern
