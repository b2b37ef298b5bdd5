// Attention over the paged 8-bit cache for more than a few rows a key/value
// head (prompts, drafted tokens of large groups); the mathematics, the order
// of the work and the join are those of rn_kv_attn.cu.
//
// Both products run on the tensor cores (tcgen05, f16 operands, fp32 sums) with
// 128 rows of queries as M.  Tensor memory holds all that belongs to rows: the
// queries (f16, the A operand of S = Q K^T), the scores S of one page (fp32, 64
// columns), the weights in their place (f16, the A operand of O = P V) and the
// output O (fp32); so shared memory holds keys and values only, as B operands
// in f16 (128-byte swizzle): K [64 positions, dim] and V^T [dim, 64 positions],
// both as the cache has them.
//
// Roles of a CTA (one an SM):
//   NG groups of 4 warps   softmax: a thread owns a row of a tile
//   4 warps                codes -> f16: pages are read two ahead into registers
//   1 warp of 4            issues the products (the others give their registers away)
// dim <= 128, NG = 2: two tiles of 128 rows take turns, so the tensor cores work
// on one while the other's scores become weights.  Where a (row tile, head)
// has 128 rows or fewer, the two groups take its even and odd pages instead and
// the first one adds both results up at the end.  dim > 128, NG = 1: the output
// takes half of the tensor memory; one tile, two buffers of scores.
//
// The weights' reference M is not raised for less than 2^8 (weights up to 2^8
// fit f16 as well), which leaves few rescalings of O in tensor memory.
#include <cuda_runtime.h>

#include "rn_device.cuh"
#include "rn_internal.h"
#include "rn_kv.cuh"
#include "rn_kv_plan.cuh"
#include "rn_tc.cuh"

namespace rn {
namespace {

__device__ unsigned g_err_kv_tile;

template <int D>
constexpr int kGroups = D <= 128 ? 2 : 1;
template <int D>
constexpr int kTileRows = 128 * kGroups<D>;
template <int D>
constexpr int kTileThreads = 128 * (kGroups<D> + 2);
// Registers a thread: the launch gives 65536 / threads, which the last group hands to the others
// (two groups: 2 * 160 + 128 + 64 = 4 * 128; one: 200 + 208 + 96 = 3 * 168)
template <int D>
constexpr int kRegsSoft = kGroups<D> == 2 ? 160 : 200;
template <int D>
constexpr int kRegsConv = kGroups<D> == 2 ? 128 : 208;
template <int D>
constexpr int kRegsMma = kGroups<D> == 2 ? 64 : 96;
// a stage: f16 keys and values of a page
template <int D>
constexpr int kStageBytesKv = 2 * 64 * D * 2;
template <int D>
constexpr int kStagesKv = D == 64 ? 8 : 196608 / kStageBytesKv<D>;

// tensor memory columns
template <int D>
struct Cols {
  static constexpr int kQ = D / 2;                            // of a tile's queries
  static constexpr int kS = kGroups<D> * kQ;                  // two score buffers of 64
  static constexpr int kO = kS + 128;
  static_assert(kO + kGroups<D> * D <= 512, "tensor memory");
};

__device__ __forceinline__ void tmem_alloc1(uint32_t smem_dst) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_dst) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free1(uint32_t taddr) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(taddr));
}

// D (+)= A B: A f16 in tensor memory, B f16 in shared memory; one elected lane of a converged warp issues it
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.u32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void mma_commit1(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}

template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// 32 columns of this thread's lane
__device__ __forceinline__ void tmem_store32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// f16 x f16 -> fp32, M = 128
__host__ __device__ constexpr uint32_t idesc_f16(int n) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ uint4 ldg_codes(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// what the converting warps say about a stage's page
struct PageInfo {
  int ek, ev;          // exponents; ek = kNoPage: no page
  uint32_t nan[2];     // positions whose values hold a NaN that is not in the stage
};
constexpr int kNoPage = 1 << 20;

struct Stats {
  float m, M, l;
};

template <int D, bool EXTRA>
__global__ void __launch_bounds__(kTileThreads<D>, 1) rn_kv_tile_kernel(const KvAttnParams p, int items) {
  constexpr int NG = kGroups<D>, R = kTileRows<D>, NT = kTileThreads<D>, NS = kStagesKv<D>;
  using C = Cols<D>;
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) uint64_t full_b[NS], empty_b[NS], s_b[2], p_b[2], q_b, o_b[2];
  __shared__ uint32_t tmem_at;
  __shared__ PageInfo info[NS];
  __shared__ Stats other[128];
  __shared__ Ranges<1, NT / 32> sh;
  const uint32_t ring = (smem_u32(raw) + 1023u) & ~1023u;
  const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
  constexpr int kConv = 4 * NG, kMma = kConv + 4;
  unsigned* err = &g_err_kv_tile;

  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(smem_u32(&full_b[s]), 4);   // the converting warps
      mbar_init(smem_u32(&empty_b[s]), 1);  // the products that read the stage
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s_b[i]), 1);      // scores
      mbar_init(smem_u32(&p_b[i]), 4);      // weights: a group's warps
      mbar_init(smem_u32(&o_b[i]), 1);      // a page's part of the output
    }
    mbar_init(smem_u32(&q_b), 4 * NG);      // queries: every softmax warp
    fence_barrier_init();
  }
  if (warp == kMma) tmem_alloc1(smem_u32(&tmem_at));
  tc_fence_before();
  pdl_launch_dependents();
  pdl_wait();
  Plan pl;
  const Dealt dealt = deal_pages<R, 1, NT>(p, items, sh, pl);  // has barriers
  tc_fence_after();
  const uint32_t tmem = tmem_at;
  const int me = (int)blockIdx.x;
  Desc* desc = static_cast<Desc*>(p.ws);
  if (me >= dealt.workers) {
    if (tid == 0) desc[me].parts = 0;
  } else if (warp >= kMma) {
    // ------------------------------------------------------ products
    regs_down<kRegsMma<D>>();
    Walk<R> at = walk_of<R>(pl, dealt, sh, p.c.heads, me, 0);
    constexpr uint32_t kIdS = idesc_f16(64), kIdO = idesc_f16(D);
    RingPos rs{0, 0}, ro{0, 0};          // stages of the scores' pages, and of the outputs'
    uint32_t p_ph[2] = {0, 0}, q_ph = 0;
    while (warp == kMma && at.left > 0) {
      const int cnt = at.segment();
      const bool both = NG == 2 && at.it.rows > 128;   // every page for both tiles
      const int tasks = both ? 2 * cnt : cnt;
      mbar_wait_warp(smem_u32(&q_b), q_ph, err, kErrReadyWait);
      q_ph ^= 1u;
      tc_fence_after();
      auto scores = [&](int i) {
        if (!both || (i & 1) == 0) mbar_wait_warp(smem_u32(&full_b[rs.slot]), rs.phase, err, kErrFullWait);
        tc_fence_after();
        const int x = i & 1;
        const uint32_t d = tmem + C::kS + 64 * x, q = tmem + (NG == 2 ? x * C::kQ : 0);
        const uint32_t kb = ring + rs.slot * kStageBytesKv<D>;
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
          mma_f16_ts(d, q + 8 * s, smem_desc(kb + (s / 4) * 8192, false) + 2 * (s % 4), kIdS, s > 0);
        mma_commit1(smem_u32(&s_b[x]));
        if (!both || x == 1) rs.advance(1, NS);
      };
      scores(0);
      if (tasks > 1) scores(1);
      for (int i = 0; i < tasks; ++i) {
        const int x = i & 1;
        mbar_wait_warp(smem_u32(&p_b[x]), p_ph[x], err, kErrStatsWait);
        p_ph[x] ^= 1u;
        tc_fence_after();
        const uint32_t a = tmem + C::kS + 64 * x, d = tmem + C::kO + (NG == 2 ? x * D : 0);
        const uint32_t vb = ring + ro.slot * kStageBytesKv<D> + 64 * D * 2;
        const bool begun = NG == 2 ? i > 1 : i > 0;
#pragma unroll
        for (int s = 0; s < 4; ++s) mma_f16_ts(d, a + 8 * s, smem_desc(vb, false) + 2 * s, kIdO, begun || s > 0);
        if (!both || x == 1) {
          mma_commit1(smem_u32(&empty_b[ro.slot]));
          ro.advance(1, NS);
        }
        mma_commit1(smem_u32(&o_b[x]));
        if (i + 2 < tasks) scores(i + 2);
      }
      at.advance(pl, p.c.heads, cnt);
    }
  } else if (warp >= kConv) {
    // ------------------------------------------------------ codes to f16
    if constexpr (NG == 1) regs_up<kRegsConv<D>>();
    Walk<R> at = walk_of<R>(pl, dealt, sh, p.c.heads, me, 0);
    const int ct = tid - 32 * kConv, cw = warp - kConv;
    constexpr int N = D / 32;          // 16-byte pieces a thread, of keys and of values
    constexpr int DEPTH = 2;           // pages read ahead
    // keys: a warp takes 8 positions x 64 dims (4 pieces each); values: 8 dims x 64 positions
    const int sub = lane & 3, row8 = lane >> 2;
    uint4 k[DEPTH][N], v[DEPTH][N];
    struct Ahead {
      int page, head, from, to, base;  // positions [from, to) of the page are seen
      bool some;                       // only some rows may see them all
      uint32_t ks, vs;
    } a[DEPTH];
    int pages = -1, batch = 0;
    auto fetch = [&]() {
      batch = at.blk;
      const int b = at.blk + lane;
      pages = b < at.it.nblk ? kv_page(p.q, p.c.pages, at.it.b, at.it.blk0 + b) : -1;
    };
    fetch();
    auto load = [&](int d) {
      if (at.left == 0) return;
      if (at.blk >= batch + 32) fetch();
      Ahead& x = a[d];
      x.page = __shfl_sync(0xFFFFFFFFu, pages, at.blk - batch);
      x.head = at.head;
      x.base = (at.it.blk0 + at.blk) * 64;
      x.from = max(at.it.lo - x.base, 0);
      x.to = min(at.it.hi - x.base, 64);
      const int i0 = at.it.r0 / p.group, i1 = (at.it.r0 + at.it.rows - 1) / p.group;
      x.some = i1 > i0 && (x.base + 64 > (p.causal ? at.it.p0 + i0 + 1 : at.it.len) ||
                           (p.window > 0 && x.base < at.it.p0 + i1 - p.window + 1));
      if (x.page >= 0) {
        const int64_t ph = (int64_t)x.page * p.c.heads + at.head;
        const uint8_t* kp = p.c.k + ph * 64 * D + sub * 16;
        const uint8_t* vp = p.c.v + ph * 64 * D + sub * 16;
        // piece i of the warp: keys: positions 8 (i % 2 + 2 cw) .., dims 64 (i / 2) ..; values: dims 8 (4 i + cw) ..
#pragma unroll
        for (int i = 0; i < N; ++i) k[d][i] = ldg_codes(kp + (8 * ((i & 1) + 2 * cw) + row8) * D + 64 * (i >> 1));
#pragma unroll
        for (int i = 0; i < N; ++i) v[d][i] = ldg_codes(vp + (8 * (4 * i + cw) + row8) * 64);
        x.ks = p.c.ks[ph];
        x.vs = p.c.vs[ph];
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) k[d][i] = v[d][i] = make_uint4(0, 0, 0, 0);
        x.ks = x.vs = 127;
      }
      const int item = at.item;
      if (at.advance(pl, p.c.heads, 1) && (batch != 0 || at.item != item)) fetch();
    };
    int64_t todo = at.left;
    load(0);
    load(1);
    RingPos r{0, 0};
    auto convert = [&](int d) {
      Ahead& x = a[d];
      mbar_wait(smem_u32(&empty_b[r.slot]), r.phase ^ 1u, err, kErrEmptyWait);
      const uint32_t kb = ring + r.slot * kStageBytesKv<D>, vb = kb + 64 * D * 2;
      if (ct == 0) {
        info[r.slot].ek = x.page >= 0 ? kv_exp(x.ks) : kNoPage;
        info[r.slot].ev = kv_exp(x.vs);
        info[r.slot].nan[0] = info[r.slot].nan[1] = 0;
      }
      if (x.from > 0 || x.to < 64 || x.some) {
        // what no row sees is not looked at; a NaN that only some rows see reaches those by their weight
        uint32_t keep[4], nan[4] = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          keep[j] = 0;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int pos = 16 * sub + 4 * j + q;
            if (pos >= x.from && pos < x.to) keep[j] |= 0xFFu << (8 * q);
          }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
          uint32_t* w = reinterpret_cast<uint32_t*>(&v[d][i]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            w[j] &= keep[j];
            if (x.some) {
              const uint32_t bad = ((w[j] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
              nan[j] |= bad;
              w[j] &= ~((bad >> 7) * 0xFFu);
            }
          }
        }
        // 16 positions of this lane as bits; then those of the warp
        uint32_t bits = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) bits |= (nan[j] >> (8 * q + 7) & 1u) << (4 * j + q);
        bits <<= 16 * (sub & 1);
        uint32_t lo = sub < 2 ? bits : 0u, hi = sub < 2 ? 0u : bits;
        lo = __reduce_or_sync(0xFFFFFFFFu, lo);
        hi = __reduce_or_sync(0xFFFFFFFFu, hi);
        asm volatile("bar.sync 2, 128;" ::: "memory");  // the stage's bits are clear
        if (lane == 0 && (lo | hi)) {
          atomicOr(&info[r.slot].nan[0], lo);
          atomicOr(&info[r.slot].nan[1], hi);
        }
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int row = 8 * ((i & 1) + 2 * cw) + row8;
        const uint32_t w[4] = {k[d][i].x, k[d][i].y, k[d][i].z, k[d][i].w};
        uint32_t h[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) e4m3x4_f16x4(w[j], h[2 * j], h[2 * j + 1]);
        const uint32_t o = kb + (i >> 1) * 8192 + row * 128;
        sts128(o + (((2 * sub) ^ row8) << 4), h[0], h[1], h[2], h[3]);
        sts128(o + (((2 * sub + 1) ^ row8) << 4), h[4], h[5], h[6], h[7]);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int row = 8 * (4 * i + cw) + row8;
        const uint32_t w[4] = {v[d][i].x, v[d][i].y, v[d][i].z, v[d][i].w};
        uint32_t h[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) e4m3x4_f16x4(w[j], h[2 * j], h[2 * j + 1]);
        const uint32_t o = vb + row * 128;
        sts128(o + (((2 * sub) ^ row8) << 4), h[0], h[1], h[2], h[3]);
        sts128(o + (((2 * sub + 1) ^ row8) << 4), h[4], h[5], h[6], h[7]);
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&full_b[r.slot]));
      r.advance(1, NS);
    };
    while (todo > 0) {
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) {
        if (todo > 0) {
          convert(d);
          load(d);
          --todo;
        }
      }
    }
  } else {
    // ------------------------------------------------------ softmax
    regs_up<kRegsSoft<D>>();
    Walk<R> at = walk_of<R>(pl, dealt, sh, p.c.heads, me, 0);
    const int x = warp >> 2;                             // the group
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tq = tmem + lanes + x * C::kQ, to = tmem + lanes + C::kO + x * D;
    const int in_tile = (warp & 3) * 32 + lane;
    uint32_t done[2] = {0, 0};                           // pages of each score buffer so far
    RingPos r{0, 0};
    while (at.left > 0) {
      const Item& it = at.it;
      const int head = at.head, cnt = at.segment();
      const bool begins = at.blk == 0, ends = at.blk + cnt == it.nblk;
      const bool both = NG == 2 && it.rows > 128, split = NG == 2 && !both;
      const int row_in = both ? x * 128 + in_tile : in_tile;
      const int rr = it.r0 + min(row_in, it.rows - 1);
      const int qi = rr / p.group, qh = head * p.group + rr % p.group;
      float qs;
      {
        // the query row in f16, its largest magnitude at 2^14
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.x) +
                                                          (int64_t)(it.s0 + qi) * p.stride + (int64_t)qh * D);
        const bool real = row_in < it.rows;
        uint32_t big = 0;
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
          const uint4 w4 = real ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t lo = w[j] & 0x7FFFu, hi = w[j] >> 16 & 0x7FFFu;
            if (lo < 0x7F80u) big = max(big, lo);
            if (hi < 0x7F80u) big = max(big, hi);
          }
        }
        const int up = max((int)(big >> 7) - 127 - 14, kKvExpMin);
        const float mul = pow2i(-up);
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
          uint32_t h[32];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint4 w4 = real ? __ldg(src + c * 8 + j) : make_uint4(0, 0, 0, 0);
            float f[8];
            bf16x8_to_f32(w4, f);
#pragma unroll
            for (int i = 0; i < 4; ++i) h[4 * j + i] = pack_f16x2(f[2 * i] * mul, f[2 * i + 1] * mul);
          }
          tmem_store32(tq + 32 * c, h);
        }
        tmem_store_wait();
        qs = EXTRA ? pow2i(up) * p.scale : pow2i(up) * (p.scale * kLog2e);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&q_b));
      const int pos0 = it.p0 + qi;
      const int row_hi = p.causal ? pos0 + 1 : it.len, row_lo = p.window > 0 ? pos0 - p.window + 1 : 0;
      const int i0 = it.r0 / p.group, i1 = (it.r0 + it.rows - 1) / p.group;
      const int all_hi = p.causal ? it.p0 + i0 + 1 : it.len, all_lo = p.window > 0 ? it.p0 + i1 - p.window + 1 : 0;
      float slope = 0.0f;
      if constexpr (EXTRA)
        if (p.slopes != nullptr) slope = __ldg(p.slopes + qh) * kLog2e;

      float m = -INFINITY, M = -INFINITY, l = 0.0f;
      const int step = split ? 2 : 1, first = split ? x : 0;
      if (split && x == 1) r.advance(1, NS);
#pragma unroll 1
      for (int c = first; c < cnt; c += step) {
        const int buf = NG == 2 ? x : c & 1;
        const uint32_t ts = tmem + lanes + C::kS + 64 * buf;
        mbar_wait_warp(smem_u32(&full_b[r.slot]), r.phase, err, kErrFullWait);
        const PageInfo& pg = info[r.slot];
        const int ek = pg.ek, base = (it.blk0 + at.blk + c) * 64;
        const float ev = (float)pg.ev;
        const bool there = ek != kNoPage;
        const float f = qs * pow2i(there ? ek : 0);
        const bool edge = !there || base < all_lo || base + 64 > all_hi;
        uint32_t nan[2] = {0, 0};
        if (edge) nan[0] = pg.nan[0], nan[1] = pg.nan[1];
        mbar_wait_warp(smem_u32(&s_b[buf]), done[buf] & 1, err, kErrStatsWait);
        ++done[buf];
        tc_fence_after();
        float s[64];
        tmem_load32(ts, reinterpret_cast<float(&)[32]>(s));
        tmem_load32(ts + 32, reinterpret_cast<float(&)[32]>(s[32]));
        tmem_load_wait();
        float mul = f;
        if (EXTRA || edge) {
          mul = 1.0f;
#pragma unroll
          for (int i = 0; i < 64; ++i) {
            const int pos = base + i;
            float z = s[i] * f;
            if constexpr (EXTRA) {
              if (p.softcap > 0.0f) z = capped(z, p.softcap, 2.0f * kLog2e / p.softcap);
              z = fmaf(slope, (float)(pos - pos0), z * kLog2e);
            }
            if (edge) {
              const bool sees = there && pos >= row_lo && pos < row_hi;
              if (nan[i >> 5] >> (i & 31) & 1) z = __uint_as_float(0x7FC00000u);
              if (!sees) z = -INFINITY;
            }
            s[i] = z;
          }
        }
        float top = s[0];
#pragma unroll
        for (int i = 1; i < 64; ++i) top = fmaxf(top, s[i]);
        if (top != top) top = -INFINITY;  // NaN everywhere: the weights carry it
        top *= mul;
        const float m2 = fmaxf(m, top);
        const float base_m = m2 == -INFINITY ? 0.0f : m2;
        const bool raise = top + ev > M + 8.0f;
        if (__any_sync(0xFFFFFFFFu, raise)) {
          const float M2 = raise ? top + ev : M;
          if (c != first) {
            // The output holds the pages before: two groups ask for a page's scores after its own page
            // before has been added; one group, only after the one before that.
            if constexpr (NG == 1)
              mbar_wait_warp(smem_u32(&o_b[buf ^ 1]), (done[buf ^ 1] - 1) & 1, err, kErrStatsWait);
            tc_fence_after();
            const float shrink = raise ? ex2(M - M2) : 1.0f;
#pragma unroll 1
            for (int d = 0; d < D / 32; ++d) {
              float o[32];
              tmem_load32(to + 32 * d, o);
              tmem_load_wait();
              uint32_t u[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(o[i] * shrink);
              tmem_store32(to + 32 * d, u);
            }
            tmem_store_wait();
          }
          M = M2;
        }
        const float sub = M == -INFINITY ? 0.0f : M - ev;  // 2^sub: the unit of this page's weights
        float sum0 = 0.0f, sum1 = 0.0f;
        uint32_t w[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float a = ex2(fmaf(s[2 * i], mul, -sub)), b = ex2(fmaf(s[2 * i + 1], mul, -sub));
          sum0 += a;
          sum1 += b;
          w[i] = pack_f16x2(a, b);
        }
        tmem_store32(ts, w);
        l = l * ex2(m - base_m) + (sum0 + sum1) * ex2(fminf(sub - base_m, 126.0f));
        m = m2;
        tmem_store_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&p_b[buf]));
        r.advance(step, NS);
      }
      // the stages of the other group's last pages
      if (split) {
        const int left = cnt - first, mine = left > 0 ? (left + 1) / 2 : 0;
        const int passed = first + 2 * mine;
        if (passed > cnt) {
          // one stage too far: back by one
          if (r.slot == 0) {
            r.slot = NS - 1;
            r.phase ^= 1u;
          } else {
            --r.slot;
          }
        }
      }

      // ---------------------------------------------------- the segment's end
      const bool any = !split || x < cnt;
      const int last = NG == 2 ? x : (cnt - 1) & 1;
      if (any) mbar_wait_warp(smem_u32(&o_b[last]), (done[last] - 1) & 1, err, kErrStatsWait);
      tc_fence_after();
      float mo = -INFINITY, Mo = -INFINITY, lo = 0.0f;   // of the odd pages
      if (split) {
        if (x == 1) other[in_tile] = Stats{m, M, l};
        tc_fence_before();
        asm volatile("bar.sync 1, 256;" ::: "memory");
        tc_fence_after();
        if (x == 0) mo = other[in_tile].m, Mo = other[in_tile].M, lo = other[in_tile].l;
      }
      if (!(split && x == 1)) {
        const bool odd = split && cnt > 1;
        const float mm = fmaxf(m, mo), MM = fmaxf(M, Mo);
        const float bm = mm == -INFINITY ? 0.0f : mm, bM = MM == -INFINITY ? 0.0f : MM;
        const float sum = l * ex2(m - bm) + lo * ex2(mo - bm);
        const float unit = sum == 0.0f ? 0.0f : ex2(bM - bm) / sum;
        const float fa = unit * ex2(M - bM), fb = unit * ex2(Mo - bM);
        const float log2s = sum == 0.0f ? -INFINITY : bm + log2f(sum);
        const int64_t row = (int64_t)(it.s0 + qi) * (p.c.heads * p.group) + qh;
        float* part = kv_part(p.ws, me, begins ? 1 : 0, R, D);
        const bool whole = begins && ends, real = row_in < it.rows;
#pragma unroll 1
        for (int d = 0; d < D / 32; ++d) {
          float o[32], u[32];
          tmem_load32(to + 32 * d, o);
          if (odd) tmem_load32(to + D + 32 * d, u);
          tmem_load_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            o[i] = sum == 0.0f ? 0.0f : o[i] * fa;
            if (odd) o[i] = sum == 0.0f ? 0.0f : fmaf(u[i], fb, o[i]);
          }
          if (!real) continue;
          if (whole) {
            uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + row * D + 32 * d);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              out[i] = make_uint4(pack_bf16x2(o[8 * i], o[8 * i + 1]), pack_bf16x2(o[8 * i + 2], o[8 * i + 3]),
                                  pack_bf16x2(o[8 * i + 4], o[8 * i + 5]), pack_bf16x2(o[8 * i + 6], o[8 * i + 7]));
          } else {
            float4* out = reinterpret_cast<float4*>(part + (int64_t)row_in * D + 32 * d);
#pragma unroll
            for (int i = 0; i < 8; ++i) out[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          }
        }
        if (real) {
          if (!whole) part[R * D + row_in] = log2s;
          else if (p.lse != nullptr) p.lse[row] = log2s * kLn2;
        }
      }
      tc_fence_before();
      if (at.left == cnt && tid == 0)
        desc[me] = desc_of(dealt, me, begins && !ends ? dealt.start(me + 1) + (it.nblk - at.blk - cnt) : 0, at.item,
                           it.rows, head);
      at.advance(pl, p.c.heads, cnt);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMma) tmem_free1(tmem);
}

template <int D, bool EXTRA>
rn_status launch_e(const KvAttnParams& p, int sms, cudaStream_t s) {
  constexpr size_t smem = (size_t)kStagesKv<D> * kStageBytesKv<D> + 1024;
  auto k = rn_kv_tile_kernel<D, EXTRA>;
  static std::atomic<int> kept[kMaxDevices];
  if (once_per_device(kept, [&] {
        return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) == cudaSuccess ? 1 : -1;
      }) < 1)
    return RN_ERR_CUDA;
  const int items = (int)((int64_t)p.q.tokens * p.group / kTileRows<D>) + p.q.B;
  const int grid = sms < kKvMaxCtas ? sms : kKvMaxCtas;
  rn_status st = launch_pdl<KvAttnParams, int>(k, dim3(grid), kTileThreads<D>, smem, s, p, items);
  if (st != RN_OK) return st;
  return launch_kv_join(p, D, kTileRows<D>, grid, s);
}

template <int D>
rn_status launch_d(const KvAttnParams& p, int sms, cudaStream_t s) {
  return p.softcap > 0.0f || p.slopes != nullptr ? launch_e<D, true>(p, sms, s) : launch_e<D, false>(p, sms, s);
}

}  // namespace

rn_status launch_kv_tile(const KvAttnParams& p, int dim, int sms, cudaStream_t s) {
  switch (dim) {
    case 64: return launch_d<64>(p, sms, s);
    case 128: return launch_d<128>(p, sms, s);
    case 192: return launch_d<192>(p, sms, s);
    default: return launch_d<256>(p, sms, s);
  }
}

rn_status read_clear_error_kv_tile(unsigned* code) {
  unsigned v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_kv_tile, sizeof(v)) != cudaSuccess) return RN_ERR_CUDA;
  if (cudaMemcpyToSymbol(g_err_kv_tile, &zero, sizeof(zero)) != cudaSuccess) return RN_ERR_CUDA;
  *code = v;
  return RN_OK;
}

}  // namespace rn
