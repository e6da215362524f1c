// C ABI of the attention-side operators (declared and documented in include/tern.h): argument
// checks and launches. No entry point allocates device memory or keeps state.
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/tern.h"
#include "tern_kv.h"

namespace {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline cudaStream_t cs(tern_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }
inline tern_status from_cuda(cudaError_t e) { return e == cudaSuccess ? TERN_OK : TERN_ECUDA; }

bool valid_heads(int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
  return kv_heads >= 1 && kv_heads <= 1024 && q_heads >= 1 && q_heads <= 4096 && q_heads % kv_heads == 0 &&
         (head_dim == 64 || head_dim == 128);
}
constexpr int32_t kMaxRows = 1 << 24;

// A call without rows takes null for the tensors of its rows: one of no elements has no address.
inline bool row_ptr(const void* p, int32_t rows, uintptr_t a) { return (p || rows == 0) && aligned(p, a); }

tern_status check_qkv(const tern_qkv* x, int32_t rows, int heads_per_kv) {
  if (!x || !x->freq_dev) return TERN_EINVAL;
  if (x->src_type != TERN_ELEM_F32 && x->src_type != TERN_ELEM_BF16) return TERN_EINVAL;
  if (!valid_heads(x->q_heads, x->kv_heads, x->head_dim)) return TERN_ESHAPE;
  if (x->row_stride < (int64_t)(x->q_heads + heads_per_kv * x->kv_heads) * x->head_dim || x->row_stride % 4 ||
      x->row_stride > (int64_t)1 << 32)
    return TERN_ESHAPE;
  if (!(x->eps >= 0.0f) || !std::isfinite(x->eps)) return TERN_EINVAL;
  if (!row_ptr(x->src_dev, rows, 16) || !aligned(x->freq_dev, 8) || !aligned(x->q_gain_dev, 4) || !aligned(x->k_gain_dev, 4))
    return TERN_EINVAL;
  return TERN_OK;
}

// The cache and the sequences; fills the kernels' view of them.
tern_status check_kv(const tern_kv_cache* c, const tern_kv_batch* b, int32_t* err_flag_dev, tern::KvView& v) {
  if (!c || !b || !c->k_dev || !c->v_dev || !c->k_scale_dev || !c->v_scale_dev) return TERN_EINVAL;
  if (!b->row_start_dev || !b->kv_len_dev || !b->page_table_dev) return TERN_EINVAL;
  if (c->pages < 1 || c->page_size < TERN_KV_BLOCK || c->page_size > 65536 || c->page_size % TERN_KV_BLOCK) return TERN_ESHAPE;
  if (!valid_heads(c->kv_heads, c->kv_heads, c->head_dim)) return TERN_ESHAPE;
  if (b->batch < 1 || b->batch > 65536 || b->rows < 0 || b->rows > kMaxRows || b->max_pages < 1 ||
      (int64_t)b->max_pages * c->page_size > INT32_MAX - 65536 || (int64_t)c->pages * c->kv_heads * c->page_size > INT32_MAX)
    return TERN_ESHAPE;
  if (!aligned(c->k_dev, 16) || !aligned(c->v_dev, 16) || !aligned(c->k_scale_dev, 4) || !aligned(c->v_scale_dev, 4) ||
      !aligned(b->row_start_dev, 4) || !aligned(b->kv_len_dev, 4) || !aligned(b->page_table_dev, 4) || !aligned(err_flag_dev, 4))
    return TERN_EINVAL;
  v = tern::KvView{c->k_dev, c->v_dev, c->k_scale_dev, c->v_scale_dev, c->pages, c->page_size, c->kv_heads,
                   b->batch, b->rows, b->max_pages, b->row_start_dev, b->kv_len_dev, b->page_table_dev, err_flag_dev};
  return TERN_OK;
}

tern::QkvParams qkv_params(const tern_qkv* x, int32_t rows, uint16_t* q) {
  tern::QkvParams p = {};
  p.src = x->src_dev;
  p.stride = x->row_stride;
  p.q_heads = x->q_heads;
  p.kv_heads = x->kv_heads;
  p.q_gain = x->q_gain_dev;
  p.k_gain = x->k_gain_dev;
  p.eps = x->eps;
  p.freq = x->freq_dev;
  p.q = q;
  p.rows = rows;
  return p;
}

}  // namespace

extern "C" {

tern_status tern_qk_norm_rope(const tern_qkv* x, int32_t rows, const int32_t* pos_dev, uint16_t* q_dev, uint16_t* k_dev,
                              uint32_t flags, tern_stream_t stream) {
  tern_status st = check_qkv(x, rows, 1);
  if (st != TERN_OK) return st;
  if (rows < 0 || rows > kMaxRows) return TERN_ESHAPE;
  if (!row_ptr(pos_dev, rows, 4) || !row_ptr(q_dev, rows, 16) || !row_ptr(k_dev, rows, 16) || (flags & ~TERN_FLAG_PDL))
    return TERN_EINVAL;
  if (rows == 0) return TERN_OK;
  tern::QkvParams p = qkv_params(x, rows, q_dev);
  p.pos = pos_dev;
  p.k = k_dev;
  return from_cuda(tern::launch_qkv(p, x->head_dim, x->src_type == TERN_ELEM_BF16, false, (flags & TERN_FLAG_PDL) != 0, cs(stream)));
}

tern_status tern_kv_append(const tern_qkv* x, const tern_kv_cache* cache, const tern_kv_batch* batch, uint16_t* q_dev,
                           int32_t* err_flag_dev, uint32_t flags, tern_stream_t stream) {
  if (!batch) return TERN_EINVAL;
  tern_status st = check_qkv(x, batch->rows, 2);
  if (st != TERN_OK) return st;
  tern::KvView v;
  st = check_kv(cache, batch, err_flag_dev, v);
  if (st != TERN_OK) return st;
  if (!row_ptr(q_dev, batch->rows, 16) || (flags & ~TERN_FLAG_PDL)) return TERN_EINVAL;
  if (x->kv_heads != cache->kv_heads || x->head_dim != cache->head_dim) return TERN_ESHAPE;
  if (batch->rows == 0) return TERN_OK;
  tern::QkvParams p = qkv_params(x, batch->rows, q_dev);
  p.kv = v;
  return from_cuda(tern::launch_qkv(p, x->head_dim, x->src_type == TERN_ELEM_BF16, true, (flags & TERN_FLAG_PDL) != 0, cs(stream)));
}

tern_status tern_kv_read(const tern_kv_cache* cache, const tern_kv_batch* batch, uint16_t* k_dev, uint16_t* v_dev,
                         int32_t* err_flag_dev, tern_stream_t stream) {
  tern::KvReadParams p = {};
  tern_status st = check_kv(cache, batch, err_flag_dev, p.kv);
  if (st != TERN_OK) return st;
  if (!row_ptr(k_dev, batch->rows, 16) || !row_ptr(v_dev, batch->rows, 16)) return TERN_EINVAL;
  if (batch->rows == 0) return TERN_OK;
  p.k = k_dev;
  p.v = v_dev;
  return from_cuda(tern::launch_kv_read(p, cache->head_dim, cs(stream)));
}

size_t tern_paged_attn_workspace_bytes(int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
  return valid_heads(q_heads, kv_heads, head_dim) ? tern::attn_workspace_bytes(head_dim) : 0;
}

tern_status tern_paged_attn(const uint16_t* q_dev, int32_t q_heads, float softmax_scale, const tern_kv_cache* cache,
                            const tern_kv_batch* batch, int32_t max_rows, uint16_t* out_dev, float* lse_dev,
                            void* workspace_dev, size_t workspace_bytes, int32_t* err_flag_dev, uint32_t flags,
                            tern_stream_t stream) {
  tern::AttnParams p = {};
  tern_status st = check_kv(cache, batch, err_flag_dev, p.kv);
  if (st != TERN_OK) return st;
  if (!workspace_dev || (flags & ~TERN_FLAG_PDL)) return TERN_EINVAL;
  if (!valid_heads(q_heads, cache->kv_heads, cache->head_dim) || max_rows < 1 || (int64_t)batch->rows * q_heads > INT32_MAX - 64)
    return TERN_ESHAPE;
  if (!row_ptr(q_dev, batch->rows, 16) || !row_ptr(out_dev, batch->rows, 16) || !aligned(lse_dev, 4) || !aligned(workspace_dev, 16))
    return TERN_EINVAL;
  if (!std::isfinite(softmax_scale)) return TERN_EINVAL;
  if (workspace_bytes < tern::attn_workspace_bytes(cache->head_dim)) return TERN_EINVAL;
  if (batch->rows == 0) return TERN_OK;
  p.q = q_dev;
  p.out = out_dev;
  p.lse = lse_dev;
  p.q_heads = q_heads;
  p.group = tern::fast_div(q_heads / cache->kv_heads);
  p.page = tern::fast_div(cache->page_size);
  p.scale = softmax_scale;
  p.max_rows = max_rows;
  p.ws = static_cast<uint8_t*>(workspace_dev);
  return from_cuda(tern::launch_attn(p, cache->head_dim, (flags & TERN_FLAG_PDL) != 0, cs(stream)));
}

}  // extern "C"
