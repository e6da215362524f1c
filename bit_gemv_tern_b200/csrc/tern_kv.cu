// Queries, keys and values between the q|k|v linear and attention: per-head RMSNorm, rotation, and
// the append to (and read-back from) the paged int8 cache. The formulas and the cache layout are in
// include/tern.h.
//
// k_qkv: one pass over the linear's output rows. A CTA takes a window of rows; a unit is the run of
// rows that fall into one 16-token block of one sequence (without a cache: the window itself).
// The unit's rotation angles are the same for every head, so the CTA computes their sines and
// cosines once into shared memory, and its warps then take heads in turn: a query head streams
// its rows through once, a key or value head twice, because the block's scale (an absmax over all of
// them) must be known before the first code. A half-warp takes a row; a lane holds the same
// D/32 elements of both halves of a head, so the rotation needs no exchange between lanes.
// One warp owns one (block, head): no atomics, and the result does not depend on the schedule.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "tern_device.cuh"
#include "tern_kv.cuh"
#include "tern_kv.h"

namespace tern {
namespace {

constexpr int kQkvThreads = 256;
constexpr int kWindow = 16;                     // rows of a window (decode batches take windows of one row)
constexpr int kReadWindow = 16;

// One head's elements of a lane: of its row's 16 lanes lane l holds l * V .. of the first half and of the second half.
template <int V>
struct Halves {
  float lo[V], hi[V];
};

template <int V, bool BF16>
__device__ __forceinline__ void load_some(float (&x)[V], const void* src, int64_t at) {
  if constexpr (BF16) {
    uint32_t w[V / 2];
    if constexpr (V == 4) {
      const uint2 y = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(src) + at);
      w[0] = y.x; w[1] = y.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(src) + at);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) x[e] = __uint_as_float(e & 1 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
  } else if constexpr (V == 4) {
    const float4 y = *reinterpret_cast<const float4*>(static_cast<const float*>(src) + at);
    x[0] = y.x; x[1] = y.y; x[2] = y.z; x[3] = y.w;
  } else {
    const float2 y = *reinterpret_cast<const float2*>(static_cast<const float*>(src) + at);
    x[0] = y.x; x[1] = y.y;
  }
}

template <int D, bool BF16>
__device__ __forceinline__ Halves<D / 32> load_head(const void* src, int64_t at, int l) {
  constexpr int V = D / 32;
  Halves<V> h;
  load_some<V, BF16>(h.lo, src, at + l * V);
  load_some<V, BF16>(h.hi, src, at + D / 2 + l * V);
  return h;
}

// Over the 16 lanes of a row.
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Norm (where there is a gain), then rotation by this lane's cosines and sines.
template <int D>
__device__ __forceinline__ void norm_rope(Halves<D / 32>& h, const Halves<D / 32>& g, bool norm, float eps,
                                          const float2* tab) {
  constexpr int V = D / 32;
  float r = 1.0f;
  if (norm) {
    float ss = 0.0f;
#pragma unroll
    for (int e = 0; e < V; ++e) ss += h.lo[e] * h.lo[e] + h.hi[e] * h.hi[e];
    ss = row_sum(ss);
    r = rsqrtf(ss * (1.0f / D) + eps);
  }
  float4 two;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    if (e % 2 == 0) two = *reinterpret_cast<const float4*>(tab + e);
    const float a = norm ? h.lo[e] * r * g.lo[e] : h.lo[e], b = norm ? h.hi[e] * r * g.hi[e] : h.hi[e];
    const float2 t = e & 1 ? make_float2(two.z, two.w) : make_float2(two.x, two.y);
    h.lo[e] = a * t.x - b * t.y;
    h.hi[e] = b * t.x + a * t.y;
  }
}

template <int V>
__device__ __forceinline__ void store_some_bf16(uint16_t* dst, const float (&x)[V]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[V - 2], x[V - 1]);
  const uint32_t u = *reinterpret_cast<const uint32_t*>(&a), w = *reinterpret_cast<const uint32_t*>(&b);
  if constexpr (V == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(u, w);
  else *reinterpret_cast<uint32_t*>(dst) = u;
}

template <int D>
__device__ __forceinline__ void store_bf16(uint16_t* dst, const Halves<D / 32>& h, int l) {
  store_some_bf16<D / 32>(dst + l * (D / 32), h.lo);
  store_some_bf16<D / 32>(dst + D / 2 + l * (D / 32), h.hi);
}

// Gains are aligned to 4 bytes only.
template <int D>
__device__ __forceinline__ Halves<D / 32> load_gain(const uint16_t* gain, int l) {
  Halves<D / 32> g{};
  if (gain) {
#pragma unroll
    for (int e = 0; e < D / 32; e += 2) {
      float x[2];
      load_some<2, true>(x, gain, l * (D / 32) + e);
      g.lo[e] = x[0]; g.lo[e + 1] = x[1];
      load_some<2, true>(x, gain, D / 2 + l * (D / 32) + e);
      g.hi[e] = x[0]; g.hi[e + 1] = x[1];
    }
  }
  return g;
}

// clamp(rint(x * inv), -127, 127) in the low byte: adding 1.5 * 2^23 rounds to an integer and leaves it in the low bits (the
// conversion instructions run at a quarter of the rate).
__device__ __forceinline__ uint32_t code_of(float x, float inv) {
  return __float_as_uint(fminf(fmaxf(x * inv, -127.0f), 127.0f) + 12582912.0f);
}

template <int V>
__device__ __forceinline__ void store_some_codes(int8_t* dst, const float (&x)[V], float inv) {
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < V; ++e) w |= (code_of(x[e], inv) & 0xFFu) << (8 * e);
  if constexpr (V == 4) *reinterpret_cast<uint32_t*>(dst) = w;
  else *reinterpret_cast<uint16_t*>(dst) = (uint16_t)w;
}

// The codes of one token in one block.
template <int D>
__device__ __forceinline__ void store_codes(int8_t* dst, const Halves<D / 32>& h, float inv, int l) {
  store_some_codes<D / 32>(dst + l * (D / 32), h.lo, inv);
  store_some_codes<D / 32>(dst + D / 2 + l * (D / 32), h.hi, inv);
}

// A key or value head of one unit: cnt rows from `row`, at places first .. first + cnt - 1 of the block. The rows are read
// twice, for the absmax and for the codes (the second time from the caches): holding 16 rows of a head would take 64
// registers a lane and leave half the warps.
template <int D, bool BF16>
__device__ __forceinline__ void append_head(const QkvParams& p, bool is_k, int hk, int row, int cnt, int first, int page,
                                            int place, const float2 (*tab)[D / 2], int lane) {
  constexpr int V = D / 32;
  const int l = lane & 15, sub = lane >> 4;
  const KvView& kv = p.kv;
  const int64_t src = (int64_t)row * p.stride + (int64_t)(p.q_heads + (is_k ? 0 : kv.kv_heads) + hk) * D;
  const int64_t blk = ((int64_t)page * kv.kv_heads + hk) * (kv.page_size / TERN_KV_BLOCK) + place / TERN_KV_BLOCK;
  float* scale = (is_k ? kv.ks : kv.vs) + blk;
  int8_t* codes = (is_k ? kv.k : kv.v) + blk * (TERN_KV_BLOCK * D);
  const float old = first ? *scale : 0.0f;
  const bool norm = is_k && p.k_gain;
  const Halves<V> g = load_gain<D>(norm ? p.k_gain : nullptr, l);
  auto value = [&](int j) {
    Halves<V> x = load_head<D, BF16>(p.src, src + j * p.stride, l);
    if (is_k) norm_rope<D>(x, g, norm, p.eps, &tab[j][l * V]);
    return x;
  };
  float top = 0.0f;
#pragma unroll 2
  for (int j = 0; j < cnt; j += 2) {                            // two rows at a time, the last alone by both half-warps
    const Halves<V> x = value(min(j + sub, cnt - 1));
#pragma unroll
    for (int e = 0; e < V; ++e) top = fmaxf(top, fmaxf(fabsf(x.lo[e]), fabsf(x.hi[e])));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  const float s = fmaxf(fmaxf(old, __fdiv_rn(top, 127.0f)), kKvScaleFloor);
  const float inv = __fdiv_rn(1.0f, s);
  if (first && s != old) {
    // the block's scale grows: its earlier codes move to the new one (D/32 bytes of a token per lane)
    const float f = __fdiv_rn(old, s);
    for (int j = 0; j < first; ++j) {
      int8_t* c = codes + j * D + lane * (D / 32);
#pragma unroll
      for (int e = 0; e < D / 32; ++e) c[e] = (int8_t)__float2int_rn((float)c[e] * f);
    }
  }
#pragma unroll 2
  for (int j = 0; j < cnt; j += 2) {
    const Halves<V> x = value(min(j + sub, cnt - 1));
    if (j + sub < cnt) store_codes<D>(codes + (first + j + sub) * D, x, inv, l);
  }
  if (lane == 0 && s != old) *scale = s;
}

// 64 registers a thread where it appends, 48 where not: 36.4 and 23.1 us (append of 2496 rows with read-back; rotation, 4095
// rows); with one CTA more on the SM 38.2 and 24.7, with one less 38.2 and 23.8.
template <int D, bool BF16, bool APPEND, int W>
__global__ void __launch_bounds__(kQkvThreads, APPEND ? 4 : 5) k_qkv(const __grid_constant__ QkvParams p) {
  constexpr int V = D / 32;
  __shared__ __align__(16) float2 tab[kWindow][D / 2];
  __shared__ int seq[W];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int w0 = blockIdx.x * W, wn = min(W, p.rows - w0);
  const int tasks = p.q_heads + (APPEND ? 2 : 1) * p.kv_heads;
  // source head of a warp's task: keys and values first (they take longest), then queries
  auto source_head = [&](int t) {
    if (!APPEND) return t;
    return t < 2 * p.kv_heads ? p.q_heads + t : t - 2 * p.kv_heads;
  };
  const int t0 = blockIdx.y * (kQkvThreads / 32) + warp;
  pdl_wait();
  pdl_launch_dependents();
  // the rows of the warp's first head are on their way while the sequences are looked up and the angles computed
  if (t0 < tasks) {
    constexpr int kLines = D * (BF16 ? 2 : 4) / 128;
    const char* src = static_cast<const char*>(p.src) + (int64_t)source_head(t0) * D * (BF16 ? 2 : 4);
    for (int l = lane; l < wn * kLines; l += 32)
      asm volatile("prefetch.global.L1 [%0];" ::"l"(src + (int64_t)(w0 + l / kLines) * p.stride * (BF16 ? 2 : 4) + l % kLines * 128));
  }
  if constexpr (APPEND) locate_rows<kQkvThreads>(p.kv, w0, wn, true, seq);
  for (int i = 0; i < wn; i += APPEND ? 1 : W) {
    int row = w0 + i, cnt = wn, pos0 = 0, b = 0;
    if constexpr (APPEND) {
      b = seq[i];
      if (b < 0) continue;
      const int start = p.kv.row_start[b], end = p.kv.row_start[b + 1];
      pos0 = p.kv.kv_len[b] - (end - row);
      if (row != start && pos0 % TERN_KV_BLOCK) continue;       // inside a unit that began earlier
      cnt = min(TERN_KV_BLOCK - pos0 % TERN_KV_BLOCK, end - row);
      __syncthreads();                                          // the last unit's table is done with
    }
    // angles in turns, reduced in fp64 to half a turn (three roundings: off by 3 * 2^-53 of the unreduced angle at most); the fast
    // sine and cosine are good to 2^-21 there
    for (int t = threadIdx.x; t < cnt * (D / 2); t += kQkvThreads) {
      const int j = t / (D / 2), e = t % (D / 2);
      const double pos = APPEND ? (double)(pos0 + j) : (double)p.pos[row + j];
      double turn = pos * (p.freq[e] * 0.15915494309189533577);
      turn -= rint(turn);
      float s, c;
      __sincosf(6.283185307179586f * (float)turn, &s, &c);
      tab[j][e] = make_float2(c, s);
    }
    __syncthreads();
    int page = 0, place = 0;
    if constexpr (APPEND) {
      page = p.kv.table[(int64_t)b * p.kv.max_pages + pos0 / p.kv.page_size];
      place = pos0 % p.kv.page_size;
      if (page < 0 || page >= p.kv.pages) {
        if (threadIdx.x == 0 && p.kv.flag) *p.kv.flag = 1;
        page = -1;
      }
    }
    for (int t = t0; t < tasks; t += gridDim.y * (kQkvThreads / 32)) {
      if constexpr (APPEND) {
        if (t < 2 * p.kv_heads) {
          if (page >= 0)
            append_head<D, BF16>(p, t < p.kv_heads, t % p.kv_heads, row, cnt, place % TERN_KV_BLOCK, page, place, tab, lane);
          continue;
        }
      }
      const int h = APPEND ? t - 2 * p.kv_heads : t;            // source head: queries, then keys
      const bool is_q = h < p.q_heads;
      const uint16_t* gain = is_q ? p.q_gain : p.k_gain;
      const int l = lane & 15, sub = lane >> 4;
      const Halves<V> g = load_gain<D>(gain, l);
      uint16_t* dst = is_q ? p.q + ((int64_t)row * p.q_heads + h) * D : p.k + ((int64_t)row * p.kv_heads + h - p.q_heads) * D;
      const int64_t step = (int64_t)(is_q ? p.q_heads : p.kv_heads) * D;
#pragma unroll 2
      for (int j0 = 0; j0 < cnt; j0 += 2) {
        const int j = min(j0 + sub, cnt - 1);
        Halves<V> x = load_head<D, BF16>(p.src, (int64_t)(row + j) * p.stride + (int64_t)h * D, l);
        norm_rope<D>(x, g, gain != nullptr, p.eps, &tab[j][l * V]);
        if (j0 + sub < cnt) store_bf16<D>(dst + j * step, x, l);
      }
    }
  }
}

// Sixteen elements of one token and head per thread and step: 16 code bytes in, 32 bytes out. Where a row's token
// lies is looked up once per row; the rows of a CTA are few where there are few in all.
template <int D>
__global__ void __launch_bounds__(256) k_kv_read(const __grid_constant__ KvReadParams p) {
  __shared__ int seq[kReadWindow];
  __shared__ int at[kReadWindow][2];              // page (-1: none), place
  const KvView& kv = p.kv;
  const int w0 = blockIdx.x * p.window, wn = min(p.window, kv.rows - w0);
  locate_rows<256>(kv, w0, wn, true, seq);
  if (threadIdx.x < wn) {
    const int b = seq[threadIdx.x], row = w0 + threadIdx.x;
    int page = -1, place = 0;
    if (b >= 0) {
      const int pos = kv.kv_len[b] - (kv.row_start[b + 1] - row);
      page = kv.table[(int64_t)b * kv.max_pages + pos / kv.page_size];
      place = pos % kv.page_size;
      if (page < 0 || page >= kv.pages) {
        page = -1;
        if (kv.flag) *kv.flag = 1;
      }
    }
    at[threadIdx.x][0] = page;
    at[threadIdx.x][1] = place;
  }
  __syncthreads();
  const int per_row = kv.kv_heads * (D / 16), all = wn * per_row;
#pragma unroll 2
  for (int t = threadIdx.x; t < 2 * all; t += 256) {
    const bool is_v = t >= all;
    const int u = is_v ? t - all : t;
    const int i = u / per_row, r = u - i * per_row, hk = r / (D / 16), c = r % (D / 16);
    const int page = at[i][0], place = at[i][1];
    if (page < 0) continue;
    const int64_t head = (int64_t)page * kv.kv_heads + hk;
    const float s = (is_v ? kv.vs : kv.ks)[head * (kv.page_size / TERN_KV_BLOCK) + place / TERN_KV_BLOCK];
    const uint4 w = *reinterpret_cast<const uint4*>((is_v ? kv.v : kv.k) + (head * kv.page_size + place) * D + c * 16);
    // a code as a float without the (slow) conversion: 0x4B0000uu is 2^23 + u, u = code + 128
    const uint32_t x[4] = {w.x ^ 0x80808080u, w.y ^ 0x80808080u, w.z ^ 0x80808080u, w.w ^ 0x80808080u};
    uint32_t o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float f0 = __uint_as_float(__byte_perm(x[e >> 1], 0x4B000000u, e & 1 ? 0x7442 : 0x7440)) - 8388736.0f;
      const float f1 = __uint_as_float(__byte_perm(x[e >> 1], 0x4B000000u, e & 1 ? 0x7443 : 0x7441)) - 8388736.0f;
      const __nv_bfloat162 v = __floats2bfloat162_rn(f0 * s, f1 * s);
      o[e] = *reinterpret_cast<const uint32_t*>(&v);
    }
    uint4* dst = reinterpret_cast<uint4*>((is_v ? p.v : p.k) + ((int64_t)(w0 + i) * kv.kv_heads + hk) * D + c * 16);
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

template <int D, bool BF16, bool APPEND>
cudaError_t launch_qkv_t(const QkvParams& p, bool pdl, cudaStream_t st) {
  // Appending: windows of one row while the sequences bring fewer than 16 rows each (decode, verify), so that every block is a
  // CTA's own; windows of 16 rows for longer runs, whose blocks fill up. Without a cache nothing ties rows together:
  // windows of 8 once there are enough of them (4095 rows: 10% faster than with 16), one row below.
  constexpr int kWide = APPEND ? kWindow : kWindow / 2;
  const bool wide = APPEND ? p.rows / p.kv.batch >= kWindow : p.rows >= 64 * kWindow;
  const int windows = wide ? (p.rows + kWide - 1) / kWide : p.rows;
  const int tasks = p.q_heads + (APPEND ? 2 : 1) * p.kv_heads;
  const int warps = kQkvThreads / 32;
  // The heads are split over CTAs until every SM has eight (of rows of 8: sixteen): one head a warp hides the look-ups and the
  // angles best (append of 2496 rows with read-back: 36.4 us, against 44.8 with five a SM; rotation 23.1 against 24.3 with ten).
  int split = ((APPEND ? 8 : 16) * device_sm_count() + windows - 1) / windows;
  if (split > (tasks + warps - 1) / warps) split = (tasks + warps - 1) / warps;
  // the fewest CTAs with as many rounds of heads
  const int rounds = (tasks + split * warps - 1) / (split * warps);
  split = (tasks + rounds * warps - 1) / (rounds * warps);
  const dim3 grid(windows, split);
  return wide ? launch_maybe_pdl(k_qkv<D, BF16, APPEND, kWide>, grid, dim3(kQkvThreads), 0, pdl, st, p)
              : launch_maybe_pdl(k_qkv<D, BF16, APPEND, 1>, grid, dim3(kQkvThreads), 0, pdl, st, p);
}

}  // namespace

cudaError_t launch_qkv(const QkvParams& p, int head_dim, bool bf16, bool append, bool pdl, cudaStream_t st) {
  if (head_dim == 128) {
    if (append) return bf16 ? launch_qkv_t<128, true, true>(p, pdl, st) : launch_qkv_t<128, false, true>(p, pdl, st);
    return bf16 ? launch_qkv_t<128, true, false>(p, pdl, st) : launch_qkv_t<128, false, false>(p, pdl, st);
  }
  if (append) return bf16 ? launch_qkv_t<64, true, true>(p, pdl, st) : launch_qkv_t<64, false, true>(p, pdl, st);
  return bf16 ? launch_qkv_t<64, true, false>(p, pdl, st) : launch_qkv_t<64, false, false>(p, pdl, st);
}

cudaError_t launch_kv_read(KvReadParams& p, int head_dim, cudaStream_t st) {
  // windows of 16 rows, fewer while the SMs would have less than two CTAs each
  p.window = p.kv.rows / (2 * device_sm_count());
  p.window = p.window < 1 ? 1 : p.window > kReadWindow ? kReadWindow : p.window;
  const int grid = (p.kv.rows + p.window - 1) / p.window;
  if (head_dim == 128) k_kv_read<128><<<grid, 256, 0, st>>>(p);
  else k_kv_read<64><<<grid, 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace tern
