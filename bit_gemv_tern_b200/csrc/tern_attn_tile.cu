// Attention over the paged int8 cache for many rows a sequence (prefill, long verify passes) on the
// 5th-generation tensor cores: include/tern.h, tern_paged_attn.
//
// Bound by the tensor cores and, as much, by the softmax: a tile of 256 query rows x 128 tokens is 16.8
// MFLOP, 2048 cycles of an SM's MMA rate at heads of 128, and 32768 exponentials, 2048 cycles of its
// special function units. So everything overlaps: one persistent CTA per SM, in four warpgroups:
//
//   warps 0..3, 4..7   softmax of the tile's two halves of 128 query rows (a row x head of the group,
//               flattened), one row per thread: S from TMEM, running maximum and sum in registers, P
//               back to TMEM as fp16 where S was, the output rescaled only when the maximum has risen by
//               more than 2^8; at a tile's end O / sum to the output (or a partial result to the workspace);
//   warps 8..11  codes to fp16 operand tiles: keys [token][element], values transposed
//               [element][token], both K-major with 128-byte swizzle;
//   warp 12     TMA of the raw codes (boxes of up to 64 tokens of a page), block scales;
//   warp 14     walks the CTA's range and hands the other warps their segments through a ring;
//   warps 13, 15  issue the tcgen05.mma kind::f16 of a half each: S = Q K^T (A = Q and B = K from shared
//               memory), O += P V (A = P from TMEM, B = V^T). While one half's softmax runs, the other
//               half's products do.
// TMEM: S of the two halves (128 columns each, P over them), O of the two halves (128 each): all 512.
// Token order: the key tile's row 8 o + j holds token 16 j + o of the chunk, so that the transposition of the
// values reads and writes shared memory without bank conflicts; column r of S is then of block r % 8, and the
// softmax takes its eight block scales as compile-time choices.
// Scales and splitting as in tern_attn.cu: the exponent carries log2 of the value scale, and the call's
// (tile, chunk) sequence is cut into equal ranges.
// Every mbarrier wait is bounded; a kernel that gives up latches TERN_ETIMEOUT, drains what it issued (bounded),
// frees its TMEM and returns.
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "tern_attn.cuh"
#include "tern_kernels.h"

namespace tern {

__device__ int g_attn_tile_latch = 0;

namespace {

constexpr int kRows = 256, kHalf = 128;           // rows of a tile, of an MMA
constexpr int kChunk = 128;                       // tokens of a chunk
constexpr int kBlocks = kChunk / TERN_KV_BLOCK;
// What a tile costs beside its chunks (queries in, results out), in chunks of about a microsecond.
constexpr int kTileCost = 2;
constexpr int kThreads = 512;
constexpr int kDecWarps = 4;
constexpr int kPanel = 128 * 128;                 // a swizzled panel of 128 rows x 64 fp16
// block scales of this many chunks: codes in flight, two expanded, one in the softmax and the one before it, whose sums
// a thread may still be scaling; a power of two
constexpr int kScaleSlots = 8;
// registers a thread of the softmax warpgroups and of the others: they add up to what the launch has
constexpr int kRegsSoftmax = 184, kRegsOther = 72;
static_assert((kRegsSoftmax + kRegsOther) * (kThreads / 2) == 128 * kThreads, "register split");

// A piece of a tile: what the warps need to know of it.
struct Segment {
  int seg, off;                // chunks, the first one (seg = 0: the end of the range)
  int start, first;            // the sequence's first row; its first row's token position
  int row0, rows;              // the tile's first flattened row, its rows
  int vis, b, hk;              // tokens seen, sequence, key/value head
  int c0, c1;                  // the CTAs that share the tile
  int pad;
};
constexpr int kSegments = 4;                      // ring of segments
constexpr int kSegWarps = 8 + kDecWarps + 3;      // warps that read it

template <int D>
struct Tile {
  static constexpr int kPanels = D / 64;
  static constexpr int kQ = kPanels * kPanel;                       // one half's queries
  static constexpr int kK = kPanels * kPanel;
  static constexpr int kVPanel = D * 128;                           // D rows x 64 tokens
  static constexpr int kV = 2 * kVPanel;
  static constexpr int kRaw = kChunk * D;                           // codes of a chunk's keys
  static constexpr int kOffK = 2 * kQ, kOffV = kOffK + 2 * kK, kOffRaw = kOffV + 2 * kV;
  static constexpr int kOffScale = kOffRaw + 2 * kRaw;           // [slot][ks, log2 vs, 1 / vs][block]
  static constexpr int kOffBar = kOffScale + kScaleSlots * 3 * kBlocks * 4;
  static constexpr int kBars = 1 + 1 + 1 + 1 + 2 + 2 + 2 + 2 + 2 + 2 + 4 + 2 + 2 + 2 * kSegments;
  static constexpr int kSmem = kOffBar + kBars * 8 + 16 + 1024;
  static constexpr int kPartFloats = kHalf * D + 2 * kHalf;         // a half's partial result
  static constexpr uint32_t kIdescS = (1u << 4) | ((uint32_t)(kChunk >> 3) << 17) | ((uint32_t)(kHalf >> 4) << 24);
  static constexpr uint32_t kIdescO = (1u << 4) | ((uint32_t)(D >> 3) << 17) | ((uint32_t)(kHalf >> 4) << 24);
};

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
// K-major operand with 128-byte swizzle: 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t umma_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(16u >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}
// One lane of the (converged) warp, chosen so that the compiler keeps the tensor-core operands of the code it guards in
// uniform registers: three instructions an MMA, against twelve behind a test of threadIdx.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
  return e;
}
// D[tmem] (+)= A[smem] B[smem], fp16 operands, fp32 accumulator.
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}
// D[tmem] (+)= A[tmem] B[smem].
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n"
      ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}
__device__ __forceinline__ void umma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// 32 consecutive columns of this thread's lane; the caller waits.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(__float_as_uint(x)), "r"(__float_as_uint(y)));
  return v;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& x, float& y) {
  uint32_t a, b;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(v));
  x = __uint_as_float(a);
  y = __uint_as_float(b);
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Keys of a chunk: raw codes (as TMA left them) to [row][element] fp16 panels. Neighbouring lanes take two rows and
// opposite panels, so that loads and stores meet every bank once.
template <int D>
__device__ __forceinline__ void expand_keys(uint32_t raw, uint32_t dst, int warp, int lane) {
  const int c4 = lane & 3, b = lane >> 2 & 1, r2 = lane >> 3;
#pragma unroll
  for (int it = 0; it < 4 * Tile<D>::kPanels; ++it) {
    const int panel = Tile<D>::kPanels == 2 ? b ^ (it & 1) : 0;
    const int pair = (warp * 4 + r2) * 4 + (Tile<D>::kPanels == 2 ? it >> 1 : it);
    const int row = 2 * pair + b, tok = 16 * (row & 7) + (row >> 3);
    const int chunk = D == 128 ? (c4 + 4 * panel) ^ (tok & 7) : c4 ^ (tok >> 1 & 3);
    const uint4 x = lds128(raw + tok * D + (chunk << 4));
    const uint32_t w[4] = {x.x ^ 0x80808080u, x.y ^ 0x80808080u, x.z ^ 0x80808080u, x.w ^ 0x80808080u};
    const uint32_t to = dst + panel * kPanel + row * 128;
    sts128(to + (((2 * c4) ^ (row & 7)) << 4), codes_f16<0x4140>(w[0]), codes_f16<0x4342>(w[0]), codes_f16<0x4140>(w[1]), codes_f16<0x4342>(w[1]));
    sts128(to + (((2 * c4 + 1) ^ (row & 7)) << 4), codes_f16<0x4140>(w[2]), codes_f16<0x4342>(w[2]), codes_f16<0x4140>(w[3]), codes_f16<0x4342>(w[3]));
  }
}
// Values of a chunk: transposed to [element][row order of the keys] fp16 panels. A lane takes eight tokens (one 16-byte
// piece of four elements' rows): eight lanes read eight neighbouring tokens and write eight pieces of a row.
template <int D>
__device__ __forceinline__ void expand_values(uint32_t raw, uint32_t dst, int warp, int lane) {
  const int o = lane & 7, wl = lane >> 3;
#pragma unroll
  for (int it = 0; it < D / 32; ++it) {
    const int oh = it & 1, wc = (D / 64) * warp + (it >> 1);         // half of the tokens, 16-element piece
    uint32_t v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int tok = 16 * j + 8 * oh + o;
      const int chunk = D == 128 ? wc ^ (tok & 7) : wc ^ (tok >> 1 & 3);
      v[j] = lds32(raw + tok * D + (chunk << 4) + 4 * wl) ^ 0x80808080u;
    }
    uint32_t e[4][4];                                                // [element][token pair]
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = __byte_perm(v[2 * j], v[2 * j + 1], 0x5140), hi = __byte_perm(v[2 * j], v[2 * j + 1], 0x7362);
      e[0][j] = codes_f16<0x4140>(lo);
      e[1][j] = codes_f16<0x4342>(lo);
      e[2][j] = codes_f16<0x4140>(hi);
      e[3][j] = codes_f16<0x4342>(hi);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d = 16 * wc + 4 * wl + i;
      sts128(dst + oh * Tile<D>::kVPanel + d * 128 + ((o ^ (d & 7)) << 4), e[i][0], e[i][1], e[i][2], e[i][3]);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) k_attn_tile(const __grid_constant__ AttnMaps a) {
  using SH = Tile<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw0 = smem_u32(smem_raw), base = (raw0 + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw0);
  float* sscale = reinterpret_cast<float*>(sm + SH::kOffScale);
  const uint32_t sQ = base, sK = base + SH::kOffK, sV = base + SH::kOffV, sRaw = base + SH::kOffRaw;
  const uint32_t kr_full = base + SH::kOffBar, kr_empty = kr_full + 8, vr_full = kr_empty + 8, vr_empty = vr_full + 8;
  const uint32_t k_full = vr_empty + 8, k_empty = k_full + 16;
  const uint32_t v_full = k_empty + 16, v_empty = v_full + 16, q_full = v_empty + 16;
  const uint32_t s_full = q_full + 16, p_full = s_full + 16;         // p_full: [half][half of the chunk]
  const uint32_t pv_done = p_full + 32, done_bar = pv_done + 16;
  const uint32_t seg_full = done_bar + 16, seg_empty = seg_full + 8 * kSegments, tmem_slot = seg_empty + 8 * kSegments;
  __shared__ Plan plan;
  __shared__ longlong2 warp_sums[kThreads / 32];
  __shared__ Segment segs[kSegments];
  const AttnParams& p = a.p;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

  if (threadIdx.x == 12 * 32) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full + 8 * i, kDecWarps);
      mbar_init(k_empty + 8 * i, 2);
      mbar_init(v_full + 8 * i, kDecWarps);
      mbar_init(v_empty + 8 * i, 2);
      mbar_init(q_full + 8 * i, 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + 8 * i, 1);
      mbar_init(pv_done + 8 * i, 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(p_full + 8 * i, 4);
    mbar_init(kr_full, 1);
    mbar_init(kr_empty, kDecWarps);
    mbar_init(vr_full, 1);
    mbar_init(vr_empty, kDecWarps);
    for (int i = 0; i < kSegments; ++i) {
      mbar_init(seg_full + 8 * i, 1);
      mbar_init(seg_empty + 8 * i, kSegWarps);
    }
    mbar_init(done_bar, 1);
    mbar_init(done_bar + 8, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  pdl_wait();
  pdl_launch_dependents();
  long long total, per;
  make_plan<kRows, kChunk, kTileCost, kThreads>(p, &plan, warp_sums, total, per);   // ends with a barrier
  const long long s0 = per * blockIdx.x;
  if (s0 >= total || too_long(p, per)) return;
  if (warp == 13) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tmem_slot), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<uint32_t*>(sm + (tmem_slot - base));
  // the segment of turn i (warp-uniform), given back when the warp is done with it
  auto take = [&](int i, bool& ok) -> const Segment* {
    ok = __all_sync(0xFFFFFFFFu, mbar_wait(seg_full + 8 * (i % kSegments), (i / kSegments) & 1));
    const Segment* g = &segs[i % kSegments];
    return ok && g->seg ? g : nullptr;
  };
  auto give = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(seg_empty + 8 * (i % kSegments));
  };
  bool ok = true;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp < 12) {
      // ---------------- codes to operand tiles ----------------
      const int wd = warp - 8;
      int i = 0;                                                     // chunk
      for (int turn = 0; ok; ++turn) {
        const Segment* g = take(turn, ok);
        if (!g) break;
        const int end = i + g->seg;
        give(turn);
        for (; i < end && ok; ++i) {
          const int s = i & 1;
          ok = mbar_wait(kr_full, i & 1) && (i < 2 || mbar_wait(k_empty + 8 * s, ((i >> 1) - 1) & 1));
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          expand_keys<D>(sRaw, sK + s * SH::kK, wd, lane);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(k_full + 8 * s);
            mbar_arrive(kr_empty);
          }
          ok = mbar_wait(vr_full, i & 1) && (i < 2 || mbar_wait(v_empty + 8 * s, ((i >> 1) - 1) & 1));
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          expand_values<D>(sRaw + SH::kRaw, sV + s * SH::kV, wd, lane);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(v_full + 8 * s);
            mbar_arrive(vr_empty);
          }
        }
      }
    } else if (warp == 12) {
      // ---------------- producer ----------------
      int n = 0, nk = 0;                                             // chunks issued: values, keys
      for (int turn = 0; ok; ++turn) {
        const Segment* g = take(turn, ok);
        if (!g) break;
        const int seg = g->seg, off = g->off, vis = g->vis, hk = g->hk;
        const int32_t* table = p.kv.table + (int64_t)g->b * p.kv.max_pages;
        give(turn);
        int row = -2;                                                // lane: block lane % 8 of chunk lane / 8 of a group
        float ks = 0.0f, vs = 0.0f;
        for (int c = 0; c < seg; ++c, ++n) {
          const int at = c & 3;
          if (at == 0) {
            const int t = (off + c) * kChunk + lane * TERN_KV_BLOCK;
            row = -2;
            if (t < vis) {
              const int page = table[t / p.page], place = t % p.page;
              row = -1;
              if (page >= 0 && page < p.kv.pages) {
                const int head = page * p.kv.kv_heads + hk;
                const int64_t blk = (int64_t)head * (p.kv.page_size / TERN_KV_BLOCK) + place / TERN_KV_BLOCK;
                row = head * p.kv.page_size + place;
                ks = p.kv.ks[blk];
                vs = value_scale(p.kv.vs[blk]);
              } else if (p.kv.flag) {
                *p.kv.flag = 1;
              }
            }
          }
          const int slot = n % kScaleSlots;
          if (n >= 1 && !(ok = __all_sync(0xFFFFFFFFu, mbar_wait(kr_empty, (n - 1) & 1)))) break;
          // blocks 0..7 of the chunk to lanes 0..7
          const int src = 8 * at + (lane & 7);
          const int r = __shfl_sync(0xFFFFFFFFu, row, src);
          const float k = __shfl_sync(0xFFFFFFFFu, ks, src), v = __shfl_sync(0xFFFFFFFFu, vs, src);
          const int step = p.box / TERN_KV_BLOCK;
          const bool copies = lane < kBlocks && r >= 0 && (lane & (step - 1)) == 0;
          const uint32_t have = __ballot_sync(0xFFFFFFFFu, copies);
          // the scales, ordered before the scores by kr_full, k_full and s_full; a block that is not there gets
          // scores of 0 * anything - infinity
          if (lane < kBlocks) {
            float* sc = sscale + slot * 3 * kBlocks + lane;
            sc[0] = r >= 0 ? k : 0.0f;
            sc[kBlocks] = r >= 0 ? __log2f(v) : -INFINITY;
            sc[2 * kBlocks] = r >= 0 ? __fdividef(1.0f, v) : 0.0f;
          }
          __syncwarp();
          const uint32_t bytes = __popc(have) * p.box * D, dst = sRaw + lane * TERN_KV_BLOCK * D;
          if (lane == 0) mbar_arrive_expect_tx(kr_full, bytes);
          __syncwarp();
          if (copies) tma_load_2d(dst, &a.kmap, 0, r, kr_full);
          ++nk;
          if (n >= 1 && !(ok = __all_sync(0xFFFFFFFFu, mbar_wait(vr_empty, (n - 1) & 1)))) break;
          if (lane == 0) mbar_arrive_expect_tx(vr_full, bytes);
          __syncwarp();
          if (copies) tma_load_2d(dst + SH::kRaw, &a.vmap, 0, r, vr_full);
        }
      }
      // do not leave with copies in flight (bounded, also after a give-up)
      if ((nk && !mbar_wait(kr_full, (nk - 1) & 1)) || (n && !mbar_wait(vr_full, (n - 1) & 1))) ok = false;
    } else if (warp == 13 || warp == 15) {
      // ---------------- MMA issue, a warp for each half ----------------
      const uint64_t dQ = umma_desc(sQ), dK = umma_desc(sK), dV = umma_desc(sV);     // + offset / 16: the address field
      const int q = warp == 15;
      const uint32_t tS = tmem + q * kChunk, tO = tmem + 2 * kChunk + q * D;
      // the scores of a chunk from key buffer `buf`
      auto scores = [&](int buf) {
        tc_fence_after();
        if (elect_one()) {
          const uint64_t a = dQ + (uint32_t)(q * (SH::kQ >> 4)), b = dK + (uint32_t)(buf * (SH::kK >> 4));
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            umma_ss(tS, a + (uint32_t)(((k >> 2) * kPanel + 32 * (k & 3)) >> 4), b + (uint32_t)(((k >> 2) * kPanel + 32 * (k & 3)) >> 4),
                    SH::kIdescS, k > 0);
          umma_commit(s_full + 8 * q);
          umma_commit(k_empty + 8 * buf);
        }
        __syncwarp();
      };
      // O += P V of half x of the chunk; more: O holds earlier products
      auto product = [&](int x, int buf, bool more) {
        tc_fence_after();
        if (elect_one()) {
          const uint64_t b = dV + (uint32_t)(buf * (SH::kV >> 4) + x * (SH::kVPanel >> 4));
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_ts(tO, tS + 32 * x + 8 * k, b + (uint32_t)(32 * k >> 4), SH::kIdescO, k > 0 ? 1u : (uint32_t)more);
          if (x) {
            umma_commit(pv_done + 8 * q);
            umma_commit(v_empty + 8 * buf);
          }
        }
        __syncwarp();
      };
      auto wait = [&](uint32_t bar, int phase) {
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar, phase & 1));
        return ok;
      };
      int n = 0, nq = 0, tiles = 0;                                  // chunks begun; chunks, tiles of this half
      for (int turn = 0; ok; ++turn) {
        const Segment* g = take(turn, ok);
        if (!g) break;
        const int seg = g->seg;
        const bool mine = g->rows > q * kHalf;
        give(turn);
        if (!mine) {                                                 // keep the buffers going for the other half
          for (int c = 0; c < seg && ok; ++c, ++n) {
            if (lane == 0) {
              mbar_arrive(k_empty + 8 * (n & 1));
              mbar_arrive(v_empty + 8 * (n & 1));
            }
            __syncwarp();
            if (wait(k_empty + 8 * (n & 1), n >> 1)) wait(v_empty + 8 * (n & 1), n >> 1);
          }
          continue;
        }
        // the queries are in, and the last tile's P (where S goes) has been multiplied
        if (!wait(k_full + 8 * (n & 1), n >> 1) || !wait(q_full + 8 * q, tiles++) || (nq && !wait(pv_done + 8 * q, nq - 1))) break;
        scores(n & 1);
        for (int c = 0; c < seg; ++c, ++n, ++nq) {
          const bool next = c + 1 < seg;
          if (!wait(v_full + 8 * (n & 1), n >> 1) || (next && !wait(k_full + 8 * ((n + 1) & 1), (n + 1) >> 1))) break;
          if (!wait(p_full + 16 * q, nq)) break;
          product(0, n & 1, c > 0);
          if (!wait(p_full + 16 * q + 8, nq)) break;
          product(1, n & 1, true);
          // the next scores go over P once that has been read
          if (next && !wait(pv_done + 8 * q, nq)) break;
          if (next) scores((n + 1) & 1);
        }
      }
      // every MMA issued has completed once done_bar flips
      __syncwarp();
      if (elect_one()) umma_commit(done_bar + 8 * q);
      __syncwarp();
      if (!mbar_wait(done_bar + 8 * q, 0)) ok = false;
    } else if (warp == 14) {
      // ---------------- the walk ----------------
      Segments<kRows, kChunk, kTileCost> sg;
      sg.w.s = plan.s;
      sg.w.b = plan.b;
      sg.w.hk = plan.hk;
      sg.w.qt = plan.qt;
      sg.w.set(p.group);
      sg.at = plan.at;
      sg.pos = 0;
      sg.count = (int)min(per, total - s0);
      const int per32 = (int)per;
      bool more = sg.next(p, true);
      for (int turn = 0;; ++turn) {
        const int s = turn % kSegments;
        if (turn >= kSegments && !(ok = __all_sync(0xFFFFFFFFu, mbar_wait(seg_empty + 8 * s, ((turn / kSegments) - 1) & 1)))) break;
        if (lane == 0) {
          Segment g;
          g.seg = more ? sg.seg : 0;
          g.off = sg.off;
          g.start = sg.w.s.start;
          g.first = sg.w.s.len - sg.w.s.n;
          g.row0 = sg.w.qt * kRows;
          g.rows = min(kRows, sg.w.s.n * (int)p.group.d - g.row0);
          g.vis = sg.w.vis;
          g.b = sg.w.b;
          g.hk = sg.w.hk;
          const int x0 = sg.tile + kTileCost, x1 = x0 + sg.w.chunks - 1;
          g.c0 = blockIdx.x - (x0 < 0 ? (per32 - 1 - x0) / per32 : 0);
          g.c1 = blockIdx.x + (x1 < per32 ? 0 : x1 / per32);
          g.pad = 0;
          segs[s] = g;
          mbar_arrive(seg_full + 8 * s);
        }
        __syncwarp();
        if (!more) break;
        more = sg.next(p, false);
      }
    }
  } else {
    // ---------------- softmax: thread = query row ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int q = warp >> 2, r = threadIdx.x & (kHalf - 1);
    const uint32_t tS = tmem + ((uint32_t)(warp & 3) << 21) + q * kChunk, tO = tmem + ((uint32_t)(warp & 3) << 21) + 2 * kChunk + q * D;
    int n = 0, nq = 0;                                               // chunks of the CTA, of this half
    for (int turn = 0;; ++turn) {
      bool there;
      const Segment* g = take(turn, there);
      ok = ok && there;
      if (!g) break;
      const int seg = g->seg, chunk0 = g->off;
      const int valid = g->rows - q * kHalf;                         // rows of this half
      if (valid <= 0) {
        n += seg;
        give(turn);
        continue;
      }
      // ---- the row's query: fp16, scaled by a power of two into [2^13, 2^14) ----
      const int fr = g->row0 + q * kHalf + (r < valid ? r : 0), qi = fr / p.group;
      const int64_t at = (int64_t)(g->start + qi) * p.q_heads + g->hk * (int)p.group.d + (fr - qi * (int)p.group.d);
      const int pos = g->first + qi;                                 // the row sees tokens 0 .. pos
      // tokens below this are seen by every row of the half
      const int clear = g->first + (g->row0 + q * kHalf) / p.group + 1;
      float rowf;
      {
        uint4 v[D / 8];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) v[i] = r < valid ? *reinterpret_cast<const uint4*>(p.q + at * D + 8 * i) : make_uint4(0u, 0u, 0u, 0u);
        __nv_bfloat162 top2 = __float2bfloat162_rn(0.0f);
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) top2 = __hmax2_nan(top2, __habs2(reinterpret_cast<const __nv_bfloat162*>(&v[i])[e]));
        const int E = absmax_exponent(fmaxf(__low2float(top2), __high2float(top2)));
        const __nv_bfloat162 up = __float2bfloat162_rn(exp2f_i(14 - E));             // a power of two: exact products
        rowf = p.scale * kLog2e * exp2f_i(E - 14);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          uint32_t h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = __bfloat1622float2(__hmul2(reinterpret_cast<const __nv_bfloat162*>(&v[i])[e], up));
            h[e] = pack_f16(f.x, f.y);
          }
          sts128(sQ + q * SH::kQ + (i >> 3) * kPanel + r * 128 + (((i & 7) ^ (r & 7)) << 4), h[0], h[1], h[2], h[3]);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full + 8 * q);
      }
      float m = -INFINITY, l = 0.0f;
#pragma unroll 1
      for (int c = 0; c < seg; ++c, ++n, ++nq) {
        const int t0 = (chunk0 + c) * kChunk;
        if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait(s_full + 8 * q, nq & 1));
        if (!ok) continue;
        tc_fence_after();
        uint32_t s[kChunk];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32(tS + 32 * i, s + 32 * i);
        const float* sc = sscale + (n % kScaleSlots) * 3 * kBlocks;
        uint64_t cf[kBlocks / 2], lv[kBlocks / 2];
#pragma unroll
        for (int j = 0; j < kBlocks / 2; ++j) {
          const float2 ks = *reinterpret_cast<const float2*>(sc + 2 * j), x = *reinterpret_cast<const float2*>(sc + kBlocks + 2 * j);
          cf[j] = pack2(rowf * ks.x, rowf * ks.y);
          lv[j] = pack2(x.x, x.y);
        }
        tmem_wait_ld();
        // the exponents (base 2) of the row's probabilities; pairs of columns, whose blocks repeat every eight columns
        uint64_t t[kChunk / 2];
#pragma unroll
        for (int i = 0; i < kChunk / 2; ++i)
          t[i] = fma2(pack2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), cf[i & 3], lv[i & 3]);
        if (t0 + kChunk > clear) {
          const int lim = pos - t0;                                  // the last visible token of the chunk
#pragma unroll
          for (int i = 0; i < kChunk / 2; ++i) {
            float x, y;
            unpack2(t[i], x, y);
            const int row = 2 * i, tok = 16 * (row & 7) + (row >> 3);
            t[i] = pack2(tok > lim ? -INFINITY : x, tok + 16 > lim ? -INFINITY : y);
          }
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < kChunk / 2; ++i) {
          float x, y;
          unpack2(t[i], x, y);
          asm("max.f32 %0, %1, %2, %3;" : "=f"(mx[i & 3]) : "f"(mx[i & 3]), "f"(x), "f"(y));
        }
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        if (__any_sync(0xFFFFFFFFu, top > m + (kLift + kSlack))) {
          const float nm = fmaxf(m, top - kLift), f = nm == -INFINITY ? 1.0f : exp2_approx(m - nm);
          m = nm;
          l *= f;
          if (c > 0) {                                               // the products so far are complete: the scores waited for them
#pragma unroll 1
            for (int i = 0; i < D / 16; ++i) {
              uint32_t o[16];
              tmem_ld16(tO + 16 * i, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st16(tO + 16 * i, o);
            }
          }
        }
        const float neg = m == -INFINITY ? 0.0f : -m;
        const uint64_t neg2 = pack2(neg, neg);
        uint64_t acc[kBlocks / 2];                                   // sums of p' of the blocks
#pragma unroll
        for (int j = 0; j < kBlocks / 2; ++j) acc[j] = 0;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float x, y;
            unpack2(add2(t[16 * h + i], neg2), x, y);
            x = exp2_approx(x);
            y = exp2_approx(y);
            acc[i & 3] = add2(acc[i & 3], pack2(x, y));
            pk[i] = pack_f16(x, y);
          }
          tmem_st16(tS + 16 * h, pk);
          if (h & 1) {                                               // a half of the chunk's probabilities is there
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full + 16 * q + 8 * (h >> 1));
          }
        }
#pragma unroll
        for (int j = 0; j < kBlocks / 2; ++j) {
          float x, y;
          unpack2(acc[j], x, y);
          const float2 iv = *reinterpret_cast<const float2*>(sc + 2 * kBlocks + 2 * j);
          l = fmaf(x, iv.x, fmaf(y, iv.y, l));
        }
      }
      // ---- the tile's end ----
      const int c0 = g->c0, c1 = g->c1;
      const bool whole = c0 == c1;
      if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait(pv_done + 8 * q, (nq - 1) & 1));
      tc_fence_after();
      // element d of row r of a partial result at [d / 4][r][d % 4]: neighbouring rows are neighbours
      float* parts = reinterpret_cast<float*>(p.ws + kCounterBytes) + (int64_t)q * SH::kPartFloats;
      auto part_of = [&](int cta) { return parts + (int64_t)(2 * cta + (cta == c0)) * 2 * SH::kPartFloats; };
      auto inv_of = [](float sum) { return sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum); };      // nan stays
      auto lse_of = [](float top, float sum) { return sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f; };
      const float inv = whole ? inv_of(l) : 1.0f;
      float* mine = part_of(blockIdx.x);
#pragma unroll 1
      for (int i = 0; i < D / 32; ++i) {
        uint32_t o[32];
        tmem_ld32(tO + 32 * i, o);
        tmem_wait_ld();
        if (r >= valid) continue;
        if (whole) {
          uint4* dst = reinterpret_cast<uint4*>(p.out + at * D + 32 * i);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const __nv_bfloat162 x = __floats2bfloat162_rn(__uint_as_float(o[8 * e + 2 * k]) * inv, __uint_as_float(o[8 * e + 2 * k + 1]) * inv);
              h[k] = *reinterpret_cast<const uint32_t*>(&x);
            }
            dst[e] = make_uint4(h[0], h[1], h[2], h[3]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<uint4*>(mine + ((8 * i + e) * kHalf + r) * 4) = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      }
      if (whole) {
        if (p.lse && r < valid) p.lse[at] = lse_of(m, l);
      } else {
        mine[kHalf * D + r] = m;
        mine[kHalf * D + kHalf + r] = l;
        // rows are a warp's own from here on: one counter per warp of the tile
        __threadfence();
        __syncwarp();
        int* counter = reinterpret_cast<int*>(p.ws) + 8 * c0 + warp;
        int arrived = 0;
        if (lane == 0) arrived = atomicAdd(counter, 1);
        if (__shfl_sync(0xFFFFFFFFu, arrived, 0) == c1 - c0) {
          __threadfence();
          if (lane == 0) *counter = 0;
          float top = -INFINITY, sum = 0.0f;
#pragma unroll 4
          for (int i = c0; i <= c1; ++i) top = fmaxf(top, __ldcg(part_of(i) + kHalf * D + r));
#pragma unroll 4
          for (int i = c0; i <= c1; ++i) {
            const float mi = __ldcg(part_of(i) + kHalf * D + r);
            sum = fmaf(__ldcg(part_of(i) + kHalf * D + kHalf + r), mi == -INFINITY ? 0.0f : exp2_approx(mi - top), sum);
          }
          const float iv = inv_of(sum);
          constexpr int kTake = 16;                                  // float4s of a partial result in flight
#pragma unroll 1
          for (int e = 0; e < D / 4; e += kTake) {
            float4 v[kTake];
#pragma unroll
            for (int k = 0; k < kTake; ++k) v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
            for (int i = c0; i <= c1; ++i) {
              const float* y = part_of(i);
              const float mi = __ldcg(y + kHalf * D + r), f = mi == -INFINITY ? 0.0f : exp2_approx(mi - top) * iv;
              float4 u[kTake];
#pragma unroll
              for (int k = 0; k < kTake; ++k) u[k] = __ldcg(reinterpret_cast<const float4*>(y + ((e + k) * kHalf + r) * 4));
#pragma unroll
              for (int k = 0; k < kTake; ++k) {
                v[k].x = fmaf(u[k].x, f, v[k].x); v[k].y = fmaf(u[k].y, f, v[k].y);
                v[k].z = fmaf(u[k].z, f, v[k].z); v[k].w = fmaf(u[k].w, f, v[k].w);
              }
            }
            if (r < valid) {
#pragma unroll
              for (int k = 0; k < kTake; k += 2) {
                const __nv_bfloat162 x0 = __floats2bfloat162_rn(v[k].x, v[k].y), x1 = __floats2bfloat162_rn(v[k].z, v[k].w);
                const __nv_bfloat162 x2 = __floats2bfloat162_rn(v[k + 1].x, v[k + 1].y), x3 = __floats2bfloat162_rn(v[k + 1].z, v[k + 1].w);
                *reinterpret_cast<uint4*>(p.out + at * D + 4 * (e + k)) =
                    make_uint4(*reinterpret_cast<const uint32_t*>(&x0), *reinterpret_cast<const uint32_t*>(&x1),
                               *reinterpret_cast<const uint32_t*>(&x2), *reinterpret_cast<const uint32_t*>(&x3));
              }
            }
          }
          if (p.lse && r < valid) p.lse[at] = lse_of(top, sum);
        }
      }
      give(turn);
    }
  }

  if (!ok) atomicExch(&g_attn_tile_latch, 5);
  tc_fence_before();
  __syncthreads();
  if (warp == 13) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

template <int D>
cudaError_t launch_tile_t(AttnMaps& a, bool pdl, cudaStream_t st) {
  static std::atomic<unsigned long long> smem_raised{0};
  cudaError_t e = allow_max_dynamic_smem(k_attn_tile<D>, smem_raised);
  if (e != cudaSuccess) return e;
  a.p.grid = fast_div(persistent_grid(kMaxGridCTAs));
  return launch_maybe_pdl(k_attn_tile<D>, dim3(a.p.grid.d), dim3(kThreads), Tile<D>::kSmem, pdl, st, a);
}

}  // namespace

size_t attn_tile_workspace_bytes(int head_dim) {
  return kCounterBytes + (size_t)4 * kMaxGridCTAs * (head_dim == 128 ? Tile<128>::kPartFloats : Tile<64>::kPartFloats) * 4;
}

cudaError_t launch_attn_tile(AttnMaps& a, int head_dim, bool pdl, cudaStream_t st) {
  return head_dim == 128 ? launch_tile_t<128>(a, pdl, st) : launch_tile_t<64>(a, pdl, st);
}

cudaError_t read_and_clear_attn_tile_latch(int* out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_attn_tile_latch, sizeof(int));
  if (e != cudaSuccess) return e;
  const int zero = 0;
  return cudaMemcpyToSymbol(g_attn_tile_latch, &zero, sizeof(int));
}

}  // namespace tern
