// Attention over the paged int8 cache for a few rows a sequence (decode tokens, draft-verify rows):
// include/tern.h, tern_paged_attn.
//
//   s_j = scale * q.k_j,  out = sum_j e^(s_j) v_j / sum_j e^(s_j)
//
// Bound by the cache's bytes: every key and value code is read once and used for the `group`
// query heads (times the sequence's rows) that share it. Persistent CTAs, two on an SM for few rows, stream the cache
// through a ring of shared-memory stages (TMA boxes of up to 64 tokens of one page, swizzled), whatever
// sequence, head and page the tokens belong to:
//
//   Work.   A tile is R query rows (row x head of the group, flattened) of one sequence and one
//           key/value head; its chunks are the 64-token stages that its last row sees. The chunks of all
//           tiles, in order, each tile with a fixed cost before its chunks, are cut into equal contiguous
//           ranges, one per CTA, found on the device from kv_len and row_start (a captured call follows
//           the lengths). A tile that spans CTAs
//           leaves a partial result (max, sum, unnormalised output) per CTA in the workspace; the last
//           CTA to arrive, by a counter, joins them in CTA order, so results do not depend on timing.
//   Warps.  One producer warp; each consumer warp takes whole 16-token blocks in turn and keeps a softmax
//           of its own (max, sum, output in registers); the warps' results are joined once per tile.
//   Math.   S^T = K Q^T and O^T = V^T P^T with mma.sync m16n8k16 f16: the 16 tokens of a block are the
//           M side of the first product, so a block's scale is one number per instruction, and the
//           query rows are the N side, 8 at a time (a decode token of a group of four wastes half of
//           it, not three quarters as on the M side). Codes become fp16 exactly (0x6400 | byte is
//           1024 + byte). tcgen05 would need M = 128 rows or tokens as the wide operand; at these row
//           counts the tensor pipe is mostly idle and the bytes bind.
//   Scales. The exponent of a probability carries the value block's scale, e = log2(e) s + log2(s_v):
//           p' = 2^(e - m), with m up to 2^7 below the largest e, is the fp16 operand of the second product and
//           never above 2^15, whatever the scales; the softmax's sum is sum p' / s_v in fp32.
#include <cstdint>
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "tern_attn.cuh"
#include "tern_kernels.h"

namespace tern {

__device__ int g_attn_latch = 0;

namespace {

constexpr int kChunk = 64;                        // tokens of a stage: four blocks
constexpr int kBlocks = kChunk / TERN_KV_BLOCK;
constexpr uint32_t kMaxPolls = 1u << 26;          // seconds, then a wait for a stage gives up
// What a tile costs beside its chunks (queries in, warps joined, result out), in chunks: measured 2.5 us of a
// CTA that streams a chunk in 0.7 us; with 32 rows and one CTA on the SM 6 to 8 us, of which the last CTA of a tile spends 4
// on joining the partial results (16 ragged sequences of 8 rows: 71.4 us with a cost of 4, 65.4 with 8, 65.7 with 10). With 16 rows 4 takes 1 to 2% longer
// than 7 (16 sequences of 4 rows 70.5 against 69.2 us), with 8 rows 6 does than 4 (64 ragged tokens 77.6 against 76.8).
template <int R>
constexpr int kTileCost = R == 32 ? 8 : R == 16 ? 7 : 4;

template <int D, int R>
struct Shape {
  // CTAs on an SM: while one joins its warps at the end of a tile, the other's stream goes on. 12 warps on the SM, three to
  // a register file partition (168 registers a thread), for 32 rows 8 (255 registers); 16 warps with 128 registers were
  // 2% slower for 8 rows. One warp of a CTA produces: a second one for 32 rows, a consumer less, was 9% slower (16 sequences of
  // 8 rows, 77.4 against 71.2 us).
  static constexpr int kPerSM = R == 32 ? 1 : 2;
  static constexpr int kCW = (R == 32 ? 8 : 12) / kPerSM - 1;     // consumer warps
  static constexpr int kThreads = (kCW + 1) * 32;
  static constexpr int kNT = R / 8;                               // 8-row column groups
  static constexpr int kTiles = D / 16;                           // 16-element tiles of a head
  static constexpr int kHalfStage = kChunk * D;                   // bytes of a stage's keys
  static constexpr int kStages = 4 * 128 / D;
  // floats of a row in the join buffer, and where its element d sits: a lane's D/8 elements of rows 2t and
  // 2t + 1 go out as 16-byte stores without bank conflicts
  static constexpr int kRowPitch = D == 128 ? 148 : 84;
  static __device__ __forceinline__ int place(int d) { return D == 128 ? d + 4 * (((d >> 4) + 1) >> 1) : d + 4 * (d >> 4); }
  // stages | join buffer [warp][R][pitch] | max, sum [warp][R] each | scales [stage][block][4] | masks, stage numbers | barriers
  static constexpr int kOffJoin = kStages * 2 * kHalfStage;
  // the join buffer also takes the max and sum of a tile's partial results, one of every CTA at most
  static constexpr int kJoinFloats = kCW * R * kRowPitch, kPartMaxima = 2 * kPerSM * kMaxGridCTAs * R;
  static constexpr int kOffMax = kOffJoin + (kJoinFloats > kPartMaxima ? kJoinFloats : kPartMaxima) * 4;
  static constexpr int kOffSum = kOffMax + kCW * R * 4;
  static constexpr int kOffScale = kOffSum + kCW * R * 4;
  static constexpr int kOffMask = kOffScale + kStages * 4 * kBlocks * 4;
  static constexpr int kOffQ = kOffMask + kStages * 8;            // R = 32: query fragments [step][NT / 2][32] x 16 B, row factors
  static constexpr int kOffBar = kOffQ + (R == 32 ? D / 16 * kNT * 256 + 4 * R : 0);
  static constexpr int kSmem = kOffBar + kStages * 16 + 1024;
  static constexpr int kPartFloats = R * D + 2 * R;               // a partial result in the workspace
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 8x8 16-bit transpose across the warp.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

template <int D, int R>
__global__ void __launch_bounds__(Shape<D, R>::kThreads, Shape<D, R>::kPerSM) k_attn_stream(const __grid_constant__ AttnMaps a) {
  using SH = Shape<D, R>;
  constexpr int CW = SH::kCW, NT = SH::kNT, T = SH::kTiles, ST = SH::kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  float* join = reinterpret_cast<float*>(sm + SH::kOffJoin);
  float* smax = reinterpret_cast<float*>(sm + SH::kOffMax);
  float* ssum = reinterpret_cast<float*>(sm + SH::kOffSum);
  float* sscale = reinterpret_cast<float*>(sm + SH::kOffScale);
  uint32_t* smask = reinterpret_cast<uint32_t*>(sm + SH::kOffMask);
  int* sstage = reinterpret_cast<int*>(smask + ST);                  // the stage a slot holds or is being filled with
  const uint32_t full = base + SH::kOffBar, empty = full + 8 * ST;
  __shared__ Plan plan;
  __shared__ longlong2 warp_sums[SH::kThreads / 32];
  __shared__ int s_last;
  const AttnParams& p = a.p;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

  if (threadIdx.x == CW * 32) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, kBlocks);
      sstage[s] = -1;
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  pdl_wait();
  pdl_launch_dependents();
  long long total, per;
  make_plan<R, kChunk, kTileCost<R>, SH::kThreads>(p, &plan, warp_sums, total, per);       // ends with a barrier
  const long long s0 = per * blockIdx.x;
  if (s0 >= total || too_long(p, per)) return;
  Segments<R, kChunk, kTileCost<R>> sg;                                                    // the CTA's segment at hand
  sg.w.s = plan.s;
  sg.w.b = plan.b;
  sg.w.hk = plan.hk;
  sg.w.qt = plan.qt;
  sg.w.set(p.group);
  sg.at = plan.at;
  sg.pos = 0;
  sg.count = (int)min(per, total - s0);
  bool ok = true;

  if (warp == CW) {
    // ---------------- producer: pages, scales and boxes, a group of 32 blocks looked up ahead ----------------
    struct Group {
      int row;                 // first row of the block in the tensor maps, -1: no such page, -2: past the end
      float ks, vs;
    };
    // lane: block lane % 4 of the chunk lane / 4 after chunk0
    auto look = [&](const auto& x, int chunk0) -> Group {
      Group g{-2, 0.0f, 0.0f};
      const int t = (chunk0 + lane / kBlocks) * kChunk + lane % kBlocks * TERN_KV_BLOCK;
      if (t < x.vis) {
        const int page = p.kv.table[(int64_t)x.b * p.kv.max_pages + t / p.page], place = t % p.page;
        g.row = -1;
        if (page >= 0 && page < p.kv.pages) {
          const int head = page * p.kv.kv_heads + x.hk;
          const int64_t blk = (int64_t)head * (p.kv.page_size / TERN_KV_BLOCK) + place / TERN_KV_BLOCK;
          g.row = head * p.kv.page_size + place;
          g.ks = p.kv.ks[blk];
          g.vs = p.kv.vs[blk];
        } else if (p.kv.flag) {
          *p.kv.flag = 1;
        }
      }
      return g;
    };
    constexpr int kAhead = 32 / kBlocks;         // chunks of a group
    // blocks of a chunk that begin a box
    const uint32_t boxes = p.box == 64 ? 1u : p.box == 32 ? 5u : 15u;
    int q0 = 0, last = -1;                       // ring position of the segment; of the last stage
    Group cur, nxt;
    bool ready = false;                          // nxt is the segment's first group
    for (bool more = sg.next(p, true); more && ok; more = sg.next(p, false)) {
      const int seg = sg.seg;
      if (!ready) nxt = look(sg.w, sg.off);
      ready = false;
      int at = 0;
      for (int c = 0; c < seg; ++c) {
        const int q = q0 + c, s = q % ST;
        if (at == 0) {                           // look the next group up while this one is copied
          cur = nxt;
          if (c + kAhead < seg) {
            nxt = look(sg.w, sg.off + c + kAhead);
          } else {
            Segments<R, kChunk, kTileCost<R>> x = sg;
            ready = x.next(p, false);
            if (ready) nxt = look(x.w, x.off);
          }
        }
        if (q >= ST && !(ok = __all_sync(0xFFFFFFFFu, mbar_wait(empty + 8 * s, ((q / ST) - 1) & 1)))) break;
        last = q;
        int row[kBlocks];
        uint32_t have = 0, bytes = 0;
#pragma unroll
        for (int j = 0; j < kBlocks; ++j) {
          row[j] = __shfl_sync(0xFFFFFFFFu, cur.row, at * kBlocks + j);
          if (row[j] >= 0) have |= 1u << j;
        }
        // the copies first: the block's scales may still be on their way
        if (lane == 0) {
#pragma unroll
          for (int j = 0; j < kBlocks; ++j)
            if ((boxes >> j & 1) && row[j] >= 0) {
              const uint32_t dst = base + s * 2 * SH::kHalfStage + j * TERN_KV_BLOCK * D;
              tma_load_2d(dst, &a.kmap, 0, row[j], full + 8 * s);
              tma_load_2d(dst + SH::kHalfStage, &a.vmap, 0, row[j], full + 8 * s);
              bytes += 2 * p.box * D;
            }
          smask[s] = have;
          *reinterpret_cast<volatile int*>(&sstage[s]) = q;
        }
        if (lane / kBlocks == at)                // ks, log2 vs, 1 / vs of the chunk's blocks
          *reinterpret_cast<float4*>(sscale + (s * kBlocks + lane % kBlocks) * 4) = make_float4(cur.ks, __log2f(value_scale(cur.vs)), __fdividef(1.0f, value_scale(cur.vs)), 0.0f);
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(full + 8 * s, bytes);
        if (++at == kAhead) at = 0;
      }
      q0 += seg;
    }
    // do not leave with copies in flight (bounded, also after a give-up)
    for (int r = last; r >= 0 && r > last - ST; --r)
      if (!mbar_wait(full + 8 * (r % ST), (r / ST) & 1)) { ok = false; break; }
    if (!ok && lane == 0) atomicExch(&g_attn_latch, 5);
    return;
  }

  // ---------------- consumers ----------------
  const int g = lane >> 2, t = lane & 3;
  const int swz = D == 128 ? (g & 7) : ((g >> 1) & 3);               // row g's (and g + 8's) chunk swizzle
  int q0 = 0;                                                        // ring position of the segment
  const auto& w = sg.w;
  for (bool more = sg.next(p, true); more; more = sg.next(p, false)) {
    const int seg = sg.seg, off = sg.off;
    const int rows = min(R, w.s.n * (int)p.group.d - w.qt * R);      // valid rows of the tile
    const int row0 = w.qt * R;                                       // flattened: row * group + head
    // queries as fp16 fragments, each row scaled by a power of two into [2^13, 2^14)
    uint32_t qf[R == 32 ? 1 : NT][R == 32 ? 1 : T][2];
    float rowf[NT][2], m[NT][2], l[NT][2], o[T][NT][4];
    // for 32 rows, 8 by each of four warps, which leave them in shared memory (every warp for itself: 65.4 against 62.5 us)
    static_assert(R < 32 || CW >= NT);
    float* srow = reinterpret_cast<float*>(sm + SH::kOffQ + D / 16 * NT * 256);
#pragma unroll
    for (int n = R == 32 ? warp : 0; n < NT; n += R == 32 ? NT : 1) {
      const int r = row0 + 8 * n + g;
      uint4 v[D / 32];
      float top = 0.0f;
      const bool live = 8 * n + g < rows;
      const uint16_t* src = p.q + ((int64_t)(w.s.start + (live ? r / p.group : 0)) * p.q_heads + w.hk * (int)p.group.d + (live ? r % p.group : 0)) * D + t * (D / 4);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        v[i] = live ? *reinterpret_cast<const uint4*>(src + 8 * i) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          top = fmaxf(top, fmaxf(fabsf(__uint_as_float(x[e] << 16)), fabsf(__uint_as_float(x[e] & 0xFFFF0000u))));
      }
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      const int E = absmax_exponent(top);
      const float up = exp2f_i(14 - E);
      const float f = p.scale * kLog2e * exp2f_i(E - 14);
      if constexpr (R == 32) {
        if (t == 0) srow[8 * n + g] = f;
      } else {
        rowf[n][0] = __shfl_sync(0xFFFFFFFFu, f, 8 * t);             // rows 2t, 2t + 1 of the group of eight
        rowf[n][1] = __shfl_sync(0xFFFFFFFFu, f, 8 * t + 4);
      }
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t h = pack_f16(__uint_as_float(x[e] << 16) * up, __uint_as_float(x[e] & 0xFFFF0000u) * up);
          if constexpr (R == 32) {
            uint32_t* sq = reinterpret_cast<uint32_t*>(sm + SH::kOffQ);      // step 2i + e/2 of the fragments
            sq[(((2 * i + (e >> 1)) * (NT / 2) + n / 2) * 32 + lane) * 4 + (n & 1) * 2 + (e & 1)] = h;
          } else {
            qf[n][2 * i + (e >> 1)][e & 1] = h;
          }
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = kNoMax;
      l[n][0] = l[n][1] = 0.0f;
#pragma unroll
      for (int i = 0; i < T; ++i) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.0f;
    }
    if constexpr (R == 32) {
      named_sync(1, CW * 32);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        rowf[n][0] = srow[8 * n + 2 * t];
        rowf[n][1] = srow[8 * n + 2 * t + 1];
      }
    }
    // tokens below this are seen by every row of the tile
    const int clear = max(0, w.s.len - w.s.n + row0 / p.group + 1);
    const int phase = q0 * kBlocks % CW;                             // the warp that takes the first block
    const int turn = (warp - phase + CW) % CW, used = min(CW, seg * kBlocks);

    for (int i = turn; i < seg * kBlocks; i += CW) {
      const int qs = q0 + i / kBlocks, s = qs % ST, j = i % kBlocks;
      const int t0 = (off + i / kBlocks) * kChunk + j * TERN_KV_BLOCK;
      // A wait tells the phases of a slot apart by parity alone, and a warp may skip stages, so that a slot whose last but
      // one stage is late would look like this one: the slot has to hold this stage before its phase means anything.
      if (ok) {
        uint32_t polls = 0;
        while (*reinterpret_cast<volatile int*>(&sstage[s]) != qs && ++polls < kMaxPolls) {}
        ok = __all_sync(0xFFFFFFFFu, polls < kMaxPolls && mbar_wait(full + 8 * s, (qs / ST) & 1));
      }
      if (ok && t0 < w.vis && (smask[s] >> j & 1)) {
        const uint32_t kb = base + s * 2 * SH::kHalfStage + j * TERN_KV_BLOCK * D, vb = kb + SH::kHalfStage;
        const float4 sc = *reinterpret_cast<const float4*>(sscale + (s * kBlocks + j) * 4);
        const float ks = sc.x, lv = sc.y, iv = sc.z;
        // keys: tokens g and g + 8, elements t * D/4 .. of the head
        float c[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) c[n][0] = c[n][1] = c[n][2] = c[n][3] = 0.0f;
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {                            // 16 bytes of both tokens: four steps
          const uint32_t chunk = (uint32_t)(((D == 128 ? 2 * t + h : t) ^ swz) << 4);
          const uint4 x = lds128(kb + g * D + chunk), y = lds128(kb + (g + 8) * D + chunk);
          const uint32_t xs[4] = {x.x ^ 0x80808080u, x.y ^ 0x80808080u, x.z ^ 0x80808080u, x.w ^ 0x80808080u};
          const uint32_t ys[4] = {y.x ^ 0x80808080u, y.y ^ 0x80808080u, y.z ^ 0x80808080u, y.w ^ 0x80808080u};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t a0 = codes_f16<0x4140>(xs[e]), a2 = codes_f16<0x4342>(xs[e]);
            const uint32_t a1 = codes_f16<0x4140>(ys[e]), a3 = codes_f16<0x4342>(ys[e]);
            if constexpr (R == 32) {
#pragma unroll
              for (int n = 0; n < NT; n += 2) {
                const uint4 b = lds128(base + SH::kOffQ + (((4 * h + e) * (NT / 2) + n / 2) * 32 + lane) * 16);
                mma_f16(c[n], a0, a1, a2, a3, b.x, b.y);
                mma_f16(c[n + 1], a0, a1, a2, a3, b.z, b.w);
              }
            } else {
#pragma unroll
              for (int n = 0; n < NT; ++n) mma_f16(c[n], a0, a1, a2, a3, qf[n][4 * h + e][0], qf[n][4 * h + e][1]);
            }
          }
        }
        const bool edge = t0 + TERN_KV_BLOCK > clear;
        bool rise = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float f0 = rowf[n][0] * ks, f1 = rowf[n][1] * ks;
          c[n][0] = fmaf(c[n][0], f0, lv);
          c[n][1] = fmaf(c[n][1], f1, lv);
          c[n][2] = fmaf(c[n][2], f0, lv);
          c[n][3] = fmaf(c[n][3], f1, lv);
          if (edge) {
            const int r = row0 + 8 * n + 2 * t, first = w.s.len - w.s.n;
            const int p0 = first + r / p.group, p1 = first + (r + 1) / p.group;   // positions of the two rows
            if (t0 + g > p0) c[n][0] = -INFINITY;
            if (t0 + g > p1) c[n][1] = -INFINITY;
            if (t0 + g + 8 > p0) c[n][2] = -INFINITY;
            if (t0 + g + 8 > p1) c[n][3] = -INFINITY;
          }
          rise |= fmaxf(c[n][0], c[n][2]) > m[n][0] + (kLift + kSlack) || fmaxf(c[n][1], c[n][3]) > m[n][1] + (kLift + kSlack);
        }
        // only where some row's maximum rises above the slack are the lanes' maxima joined and the sums rescaled
        if (__any_sync(0xFFFFFFFFu, rise)) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float x0 = fmaxf(c[n][0], c[n][2]), x1 = fmaxf(c[n][1], c[n][3]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
              x0 = fmaxf(x0, __shfl_xor_sync(0xFFFFFFFFu, x0, d));
              x1 = fmaxf(x1, __shfl_xor_sync(0xFFFFFFFFu, x1, d));
            }
            x0 = fmaxf(m[n][0], x0 - kLift);
            x1 = fmaxf(m[n][1], x1 - kLift);
            const float r0 = exp2_approx(m[n][0] - x0), r1 = exp2_approx(m[n][1] - x1);
            m[n][0] = x0;
            m[n][1] = x1;
            l[n][0] *= r0;
            l[n][1] *= r1;
#pragma unroll
            for (int k = 0; k < T; ++k) {
              o[k][n][0] *= r0;
              o[k][n][1] *= r1;
              o[k][n][2] *= r0;
              o[k][n][3] *= r1;
            }
          }
        }
        uint32_t pb[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float e0 = exp2_approx(c[n][0] - m[n][0]), e1 = exp2_approx(c[n][1] - m[n][1]);
          const float e2 = exp2_approx(c[n][2] - m[n][0]), e3 = exp2_approx(c[n][3] - m[n][1]);
          l[n][0] = fmaf(e0 + e2, iv, l[n][0]);
          l[n][1] = fmaf(e1 + e3, iv, l[n][1]);
          pb[n][0] = movmatrix_trans(pack_f16(e0, e1));
          pb[n][1] = movmatrix_trans(pack_f16(e2, e3));
        }
        // values: tokens 2t, 2t + 1, 2t + 8, 2t + 9, elements g * D/8 .. of the head
        constexpr int W = D / 32;                                     // words of D/8 bytes
        uint32_t v[4][W];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int tok = 2 * t + (e & 1) + 8 * (e >> 1);
          if constexpr (D == 128) {
            const uint4 x = lds128(vb + tok * D + ((g ^ (tok & 7)) << 4));
            v[e][0] = x.x; v[e][1] = x.y; v[e][2] = x.z; v[e][3] = x.w;
          } else {
            const uint2 x = lds64(vb + tok * D + ((((g >> 1) ^ ((tok >> 1) & 3)) << 4) | ((g & 1) << 3)));
            v[e][0] = x.x; v[e][1] = x.y;
          }
        }
#pragma unroll
        for (int k = 0; k < W; ++k) {
          const uint32_t lo0 = __byte_perm(v[0][k], v[1][k], 0x5140) ^ 0x80808080u, hi0 = __byte_perm(v[0][k], v[1][k], 0x7362) ^ 0x80808080u;
          const uint32_t lo1 = __byte_perm(v[2][k], v[3][k], 0x5140) ^ 0x80808080u, hi1 = __byte_perm(v[2][k], v[3][k], 0x7362) ^ 0x80808080u;
          const uint32_t a0 = codes_f16<0x4140>(lo0), a1 = codes_f16<0x4342>(lo0), a2 = codes_f16<0x4140>(lo1), a3 = codes_f16<0x4342>(lo1);
          const uint32_t b0 = codes_f16<0x4140>(hi0), b1 = codes_f16<0x4342>(hi0), b2 = codes_f16<0x4140>(hi1), b3 = codes_f16<0x4342>(hi1);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_f16(o[2 * k][n], a0, a1, a2, a3, pb[n][0], pb[n][1]);
            mma_f16(o[2 * k + 1][n], b0, b1, b2, b3, pb[n][0], pb[n][1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + 8 * s);
    }

    // ---- join the warps: a common maximum, then the scaled sums in warp order ----
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) {
        l[n][0] += __shfl_xor_sync(0xFFFFFFFFu, l[n][0], d);
        l[n][1] += __shfl_xor_sync(0xFFFFFFFFu, l[n][1], d);
      }
      if (g == 0) {
        smax[warp * R + 8 * n + 2 * t] = m[n][0];
        smax[warp * R + 8 * n + 2 * t + 1] = m[n][1];
      }
    }
    named_sync(1, CW * 32);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float n0 = kNoMax, n1 = kNoMax;
#pragma unroll
      for (int x = 0; x < CW; ++x) {
        n0 = fmaxf(n0, smax[x * R + 8 * n + 2 * t]);
        n1 = fmaxf(n1, smax[x * R + 8 * n + 2 * t + 1]);
      }
      const float f0 = exp2_approx(m[n][0] - n0), f1 = exp2_approx(m[n][1] - n1);
      if (g == 0) {
        ssum[warp * R + 8 * n + 2 * t] = l[n][0] * f0;
        ssum[warp * R + 8 * n + 2 * t + 1] = l[n][1] * f1;
      }
      if (turn >= used) continue;                                     // no block was this warp's
      // the lane's D/8 elements of rows 2t and 2t + 1
      float* j0 = join + (warp * R + 8 * n + 2 * t) * SH::kRowPitch + SH::place(g * (D / 8));
      float* j1 = j0 + SH::kRowPitch;
#pragma unroll
      for (int k = 0; k < T / 2; ++k) {
        *reinterpret_cast<float4*>(j0 + 4 * k) = make_float4(o[2 * k][n][0] * f0, o[2 * k][n][2] * f0, o[2 * k + 1][n][0] * f0, o[2 * k + 1][n][2] * f0);
        *reinterpret_cast<float4*>(j1 + 4 * k) = make_float4(o[2 * k][n][1] * f1, o[2 * k][n][3] * f1, o[2 * k + 1][n][1] * f1, o[2 * k + 1][n][3] * f1);
      }
    }
    named_sync(1, CW * 32);
    // the CTAs that share the tile's chunks, the first and the last of which lie x0 and x1 after the range's start
    const int x0 = sg.tile + kTileCost<R>, x1 = x0 + w.chunks - 1, per32 = (int)per;
    const int c0 = blockIdx.x - (x0 < 0 ? (per32 - 1 - x0) / per32 : 0), c1 = blockIdx.x + (x1 < per32 ? 0 : x1 / per32);
    const bool whole = c0 == c1;
    float* parts = reinterpret_cast<float*>(p.ws + kCounterBytes);
    float* part = parts + (int64_t)(2 * blockIdx.x + ((int)blockIdx.x == c0)) * SH::kPartFloats;
    auto write_out = [&](int r, int d, float4 v, float sum, float top) {
      const int fr = row0 + r;
      const int64_t at = (int64_t)(w.s.start + fr / p.group) * p.q_heads + w.hk * (int)p.group.d + fr % p.group;
      const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);      // nan stays
      const __nv_bfloat162 x = __floats2bfloat162_rn(v.x * inv, v.y * inv), y = __floats2bfloat162_rn(v.z * inv, v.w * inv);
      *reinterpret_cast<uint2*>(p.out + at * D + d) = make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
      if (p.lse && d == 0) p.lse[at] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
    };
    for (int x = warp * 32 + lane; x < rows * (D / 4); x += CW * 32) {
      const int r = x / (D / 4), d = x % (D / 4) * 4;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float sum = 0.0f, top = kNoMax;
#pragma unroll
      for (int y = 0; y < CW; ++y) {
        if ((y - phase + CW) % CW < used) {
          const float4 u = *reinterpret_cast<const float4*>(join + (y * R + r) * SH::kRowPitch + SH::place(d));
          v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
        }
        sum += ssum[y * R + r];
        top = fmaxf(top, smax[y * R + r]);
      }
      if (whole) {
        write_out(r, d, v, sum, top);
      } else {
        *reinterpret_cast<float4*>(part + r * D + d) = v;
        if (d == 0) {
          part[R * D + r] = top;
          part[R * D + R + r] = sum;
        }
      }
    }
    if (!whole) {
      __threadfence();
      named_sync(1, CW * 32);
      int* counter = reinterpret_cast<int*>(p.ws) + c0;
      if (threadIdx.x == 0) s_last = atomicAdd(counter, 1) == c1 - c0;
      named_sync(1, CW * 32);
      if (s_last) {
        __threadfence();
        if (threadIdx.x == 0) *counter = 0;
        // maxima and sums of all partial results first, then their outputs, every load on its own
        const int np = c1 - c0 + 1;
        float* pm = join;
        float* pl = join + np * R;
        for (int x = warp * 32 + lane; x < np * R; x += CW * 32) {
          const int c = c0 + x / R;
          const float* y = parts + (int64_t)(2 * c + (c == c0)) * SH::kPartFloats + R * D + x % R;
          const bool have = x % R < rows;
          pm[x] = have ? __ldcg(y) : kNoMax;
          pl[x] = have ? __ldcg(y + R) : 0.0f;
        }
        named_sync(1, CW * 32);
        for (int x = warp * 32 + lane; x < rows * (D / 4); x += CW * 32) {
          const int r = x / (D / 4), d = x % (D / 4) * 4;
          float top = kNoMax;
          for (int i = 0; i < np; ++i) top = fmaxf(top, pm[i * R + r]);
          float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          float sum = 0.0f;
#pragma unroll 8
          for (int i = 0; i < np; ++i) {
            const float f = exp2_approx(pm[i * R + r] - top);
            const float4 u = __ldcg(reinterpret_cast<const float4*>(parts + (int64_t)(2 * (c0 + i) + (i == 0)) * SH::kPartFloats + r * D + d));
            v.x = fmaf(u.x, f, v.x); v.y = fmaf(u.y, f, v.y); v.z = fmaf(u.z, f, v.z); v.w = fmaf(u.w, f, v.w);
            sum = fmaf(pl[i * R + r], f, sum);
          }
          write_out(r, d, v, sum, top);
        }
      }
    }
    named_sync(1, CW * 32);                      // the join buffers are free again
    q0 += seg;
  }
  if (!ok && lane == 0) atomicExch(&g_attn_latch, 5);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }
  return fn;
}

// The codes as rows of one token of one head; a box lies in one page.
bool block_map(CUtensorMap* m, int8_t* codes, const KvView& kv, int head_dim, int box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = encode_fn();
  if (!encode) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)head_dim, (cuuint64_t)kv.pages * kv.kv_heads * kv.page_size};
  const cuuint64_t strides[1] = {(cuuint64_t)head_dim};
  const cuuint32_t box[2] = {(cuuint32_t)head_dim, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, codes, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int R>
cudaError_t launch_stream_t(AttnMaps& a, bool pdl, cudaStream_t st) {
  static std::atomic<unsigned long long> smem_raised{0};
  cudaError_t e = allow_max_dynamic_smem(k_attn_stream<D, R>, smem_raised);
  if (e != cudaSuccess) return e;
  static_assert((Shape<D, R>::kSmem + 1024) * Shape<D, R>::kPerSM <= 228 * 1024, "the CTAs of an SM share its memory");
  a.p.grid = fast_div(persistent_grid(kMaxGridCTAs) * Shape<D, R>::kPerSM);
  return launch_maybe_pdl(k_attn_stream<D, R>, dim3(a.p.grid.d), dim3(Shape<D, R>::kThreads),
                          Shape<D, R>::kSmem, pdl, st, a);
}

template <int D>
cudaError_t launch_stream_d(AttnMaps& a, bool pdl, cudaStream_t st) {
  const long long rows = (long long)a.p.max_rows * a.p.group.d;        // of a sequence and head, if the caller is right
  // 33 to 64 rows are two tiles here, the cache read twice, and one of the tile kernel. Where the tiles are few beside the SMs both
  // wait on latency and the stream's is the shorter (one sequence of 16 rows, 16 tiles, over 100 / 1000 / 4000 / 30000 tokens:
  // 8.8 / 18.9 / 20.3 / 54.6 us against 11.2 / 20.5 / 27.8 / 71.1), with more the tile kernel's (4 sequences, 64 tiles, over 2000:
  // 27.4 against 24.3; 16 over 4096: 105 against 77).
  const long long tiles = ((long long)a.p.kv.rows * a.p.group.d + 31) / 32 * a.p.kv.kv_heads;
  if (rows > 64 || (rows > 32 && tiles * 8 > persistent_grid(kMaxGridCTAs))) return launch_attn_tile(a, D, pdl, st);
  if (rows <= 8) return launch_stream_t<D, 8>(a, pdl, st);
  if (rows <= 16) return launch_stream_t<D, 16>(a, pdl, st);
  return launch_stream_t<D, 32>(a, pdl, st);
}

}  // namespace

size_t attn_workspace_bytes(int head_dim) {
  const auto parts = [&](int rows, int per_sm) { return (size_t)2 * kMaxGridCTAs * per_sm * (rows * head_dim + 2 * rows) * 4; };
  const size_t a = parts(32, Shape<128, 32>::kPerSM), b = parts(16, Shape<128, 16>::kPerSM);
  const size_t c = kCounterBytes + (a > b ? a : b), t = attn_tile_workspace_bytes(head_dim);
  return c > t ? c : t;
}

cudaError_t launch_attn(const AttnParams& p, int head_dim, bool pdl, cudaStream_t st) {
  AttnMaps a;
  a.p = p;
  a.p.box = p.kv.page_size % 64 == 0 ? 64 : p.kv.page_size % 32 == 0 ? 32 : 16;
  if (!block_map(&a.kmap, p.kv.k, p.kv, head_dim, a.p.box) || !block_map(&a.vmap, p.kv.v, p.kv, head_dim, a.p.box))
    return cudaErrorInvalidValue;
  return head_dim == 128 ? launch_stream_d<128>(a, pdl, st) : launch_stream_d<64>(a, pdl, st);
}

cudaError_t read_and_clear_attn_latch(int* out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_attn_latch, sizeof(int));
  if (e != cudaSuccess) return e;
  const int zero = 0;
  return cudaMemcpyToSymbol(g_attn_latch, &zero, sizeof(int));
}

}  // namespace tern
