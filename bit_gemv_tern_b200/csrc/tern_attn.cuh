// What the attention kernels share: the walk over a call's tiles and its cut into equal ranges, the conversion of
// codes, and the layout of partial results.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "tern_device.cuh"
#include "tern_kv.cuh"
#include "tern_kv.h"
#include "tern_mbar.cuh"

namespace tern {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kCounterBytes = 8192;               // the workspace's counters, before the partial results
// A row's probabilities p' = 2^(e - m) are rounded to fp16 for the second product while their sum stays in fp32. A term too small
// for fp16 is then missing from the output but not from the sum, and a long flat tail beside one strong token is made of such terms.
// So the reference m is set kLift below the row's largest exponent, and follows once that has risen kSlack further (no rescale of the
// output for every small rise): the largest p' lies between 2^7 and 2^15 (fp16 ends at 65504), and a rounding takes 2^-25 at
// most, 2^-32 of the largest. With m at the largest exponent itself it took 2^-25 of it: 3000 tokens of 2^-26.5 each were lost.
// m is common to a row's sum and output, so nothing else depends on it.
constexpr float kLift = 7.0f, kSlack = 8.0f;
// The reference of no token at all: finite, so that differences of it with itself and with minus infinity are not nan.
constexpr float kNoMax = -1e30f;


struct alignas(64) AttnMaps {
  CUtensorMap kmap, vmap;      // [pages * kv_heads * page_size][head_dim] bytes, boxes of p.box rows
  AttnParams p;
};

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Two fp16 codes from two bytes of x, which holds code + 128: SEL 0x4140 takes bytes 0 and 1, 0x4342
// bytes 2 and 3; 0x6400 | u is 1024 + u, and 1152 comes off again (all exact).
template <uint32_t SEL>
__device__ __forceinline__ uint32_t codes_f16(uint32_t x) {
  const uint32_t w = __byte_perm(x, 0x64646464u, SEL);
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&w), __half2half2(__ushort_as_half(0x6480)));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// A value block's scale as the exponents carry it: its logarithm and its reciprocal have to be finite, so that zero (a block of
// zeros by its scale) and what else lies below the smallest scale of an append counts as that. The tokens keep their weight; their
// values are then 127 * 2^-60 at most. A negative scale or nan stays one and shows as nan.
__device__ __forceinline__ float value_scale(float s) { return s >= 0.0f && s < kKvScaleFloor ? kKvScaleFloor : s; }

// R: rows of a tile, CH: tokens of a chunk, COST: what a tile costs beside its chunks, in chunks.

// The walk over tiles: sequence, key/value head, row tile; chunks of a tile.
template <int R, int CH, int COST>
struct Walk {
  SeqInfo s;
  int b, hk, qt, chunks, vis;
  __device__ __forceinline__ static int tiles_of(const SeqInfo& s, const FastDiv& group) { return (int)(((uint32_t)s.n * group.d + R - 1) / R); }
  // tokens that the last row of a row tile sees
  __device__ __forceinline__ static int visible(const SeqInfo& s, const FastDiv& group, int qt) {
    const int last = min(s.n - 1, ((qt + 1) * R - 1) / group);
    return max(0, s.len - s.n + last + 1);
  }
  __device__ __forceinline__ static int chunks_of(int vis) { return max(1, (vis + CH - 1) / CH); }
  // cost of one head's tiles
  __device__ __forceinline__ static long long cost_of_head(const SeqInfo& s, const FastDiv& group) {
    long long sum = 0;
    const int nt = tiles_of(s, group);
    for (int q = 0; q < nt; ++q) sum += chunks_of(visible(s, group, q)) + COST;
    return sum;
  }
  __device__ __forceinline__ void set(const FastDiv& group) {
    vis = visible(s, group, qt);
    chunks = chunks_of(vis);
  }
  __device__ __forceinline__ void next(const AttnParams& p) {
    if (++qt < tiles_of(s, p.group)) return set(p.group);
    qt = 0;
    if (++hk < p.kv.kv_heads) return set(p.group);
    hk = 0;
    for (++b; b < p.kv.batch; ++b) {
      s = seq_info(p.kv, b);
      if (s.n) return set(p.group);
    }
  }
};

// Where a CTA's range starts.
struct Plan {
  SeqInfo s;                   // of the tile's sequence
  int b, hk, qt, at;           // tile, and the place in its cost (COST, then its chunks)
};

// A CTA's segments: the pieces of tiles in its range, [seg chunks from chunk off of tile w].
template <int R, int CH, int COST>
struct Segments {
  Walk<R, CH, COST> w;
  int at, pos, count;          // place in the tile's cost; place in the range; the range's length
  int off, seg, tile;          // tile: the tile's start, relative to the range's
  // Moves to the next piece that has chunks; false at the end of the range.
  __device__ __forceinline__ bool next(const AttnParams& p, bool first) {
    for (;; first = false) {
      if (!first) {
        if (pos >= count) return false;
        w.next(p);
        at = 0;
      }
      tile = pos - at;
      const int take = min(w.chunks + COST - at, count - pos);
      off = max(0, at - COST);
      seg = max(0, at + take - COST) - off;
      pos += take;
      if (seg) return true;
    }
  }
};

// Cuts the call's cost into equal ranges and finds this CTA's: total cost, cost per CTA, start. Every
// thread takes part; ends with a barrier. One load and one scan where the batch fits the block.
template <int R, int CH, int COST, int kThreadsT>
__device__ __forceinline__ void make_plan(const AttnParams& p, Plan* plan, longlong2* warp_sums, long long& total, long long& per) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kWarps = kThreadsT / 32;
  auto load = [&](int b, SeqInfo& s) -> long long {
    s.n = 0;
    if (b >= p.kv.batch) return 0;
    s = seq_info(p.kv, b);
    if (!s.ok && p.kv.flag && blockIdx.x == 0) *p.kv.flag = 1;
    return s.n ? Walk<R, CH, COST>::cost_of_head(s, p.group) * p.kv.kv_heads : 0;
  };
  SeqInfo s;
  long long c = load(threadIdx.x, s), incl = c, more = 0;
  if (p.kv.batch > kThreadsT) {
    for (int b = threadIdx.x + kThreadsT; b < p.kv.batch; b += kThreadsT) {
      SeqInfo x;
      more += load(b, x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) more += __shfl_xor_sync(0xFFFFFFFFu, more, o);
  }
  long long s0 = 0, base = 0;                    // base: cost of the sequences before this round's
  for (int b0 = 0; b0 < p.kv.batch; b0 += kThreadsT) {
    if (b0) {
      incl = c = load(b0 + threadIdx.x, s);
      __syncthreads();
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sums[warp] = make_longlong2(more + incl, incl);
    __syncthreads();
    long long before = base + incl - c, sum = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const longlong2 v = warp_sums[w];
      sum += v.x;
      base += v.y;
      if (w < warp) before += v.y;
    }
    if (b0 == 0) {
      total = sum;
      const long long up = total + gridDim.x - 1;
      per = up < 0x7FFFFFFFll ? (int)up / p.grid : up / gridDim.x;
      s0 = per * blockIdx.x;
    }
    if (c && s0 >= before && s0 < before + c) {
      long long rem = s0 - before;
      const long long per_head = c / p.kv.kv_heads;
      plan->s = s;
      plan->b = b0 + threadIdx.x;
      if (c < 0x7FFFFFFFll) {
        plan->hk = (int)rem / (int)per_head;
        rem = (int)rem % (int)per_head;
      } else {
        plan->hk = (int)(rem / per_head);
        rem %= per_head;
      }
      int qt = 0;
      for (;; ++qt) {
        const int n = Walk<R, CH, COST>::chunks_of(Walk<R, CH, COST>::visible(s, p.group, qt)) + COST;
        if (rem < n) break;
        rem -= n;
      }
      plan->qt = qt;
      plan->at = (int)rem;
    }
    if (s0 < base || s0 >= total) break;         // the same for every thread
  }
  __syncthreads();
}

// A call whose ranges do not fit the kernels' 32-bit chunk counters (hours of work) is left out and reported.
__device__ __forceinline__ bool too_long(const AttnParams& p, long long per) {
  if (per < (1ll << 30)) return false;
  if (p.kv.flag && threadIdx.x == 0) *p.kv.flag = 1;
  return true;
}

// The kernel for tiles of many rows (tern_attn_tile.cu).
size_t attn_tile_workspace_bytes(int head_dim);
cudaError_t launch_attn_tile(AttnMaps& a, int head_dim, bool pdl, cudaStream_t st);

// The exponent E of an absmax a: a < 2^E (clamped to -100 .. 128), from its bits.
__device__ __forceinline__ int absmax_exponent(float a) {
  const int E = (int)(__float_as_uint(a) >> 23) - 126;
  return max(-100, min(E, 128));
}

}  // namespace tern
