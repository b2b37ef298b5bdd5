// Attention over the paged 8-bit cache for more than a few rows a key/value
// head (prompts, drafted tokens of large groups); the mathematics, the order
// of the work and the join are those of rn_kv_attn.cu.
//
// Both products run on the tensor cores (tcgen05, f16 operands, fp32 sums) with
// 128 rows of queries as M.  Tensor memory holds all that belongs to rows: the
// queries (f16, the A operand of S = Q K^T), the scores S of a page (fp32), the
// weights in their place (f16, the A operand of O = P V) and the output O (fp32);
// so shared memory holds keys and values only, as B operands in f16 (128-byte
// swizzle): K [64 positions, dim] and V^T [dim, 64 positions], as the cache has them.
//
// Roles of a CTA (one an SM):
//   1 warp                 issues the products
//   1 warp                 copies pages (bulk copies of 64 dim bytes) into a ring of codes
//   4 warps                codes -> f16
//   4 warps a tile         softmax: a thread owns a row
// dim <= 128, NG = 2: two tiles of 128 rows take turns, so the tensor cores work
// on one while the other's scores become weights.  Where a (row tile, head) has
// 128 rows or fewer, the two tiles' warps take its even and odd pages instead and
// the first ones add both results up at the end.  dim > 128, NG = 1: the output
// takes half of the tensor memory; one tile, two buffers of scores.
//
// What bounds it: 4096 new tokens on 8192, 64 query heads of 128 over 8: 1279 us,
// 1075 TFLOP/s, 0.56 of the measured bf16 rate; a page of two tiles takes 2200
// cycles, of which the products are 1024 (tensor pipe 46 % active).  The rest is
// latency: a tile's page goes products -> scores -> weights -> products in turn
// (reading scores 60 cycles, their maximum 270, the exponentials 450, storing and
// handing on 120, the products 512), the tensor memory has no room for more than
// one page of scores a tile, and the warps wait for instructions as much as they
// issue them (IPC 1.8).  Tried and slower: weights beside the scores, whose buffer
// both tiles share (1288 us); 8 softmax warps a tile with half the scores a thread
// (1829); the products issued by one thread (2074), by two warps (1288), or by
// several specialized instruction sequences (1477).  20 rows a head (32 x 4 tokens on
// 6000, groups of 5) 97 us where the cache's bytes take 38: a page takes the conversion
// 1080 cycles and the issuing warp 990 where memory would allow 700.
//
// The weights' reference M, whose weight is 2^9, is not raised for less than 2^6.5
// (f16 ends at 2^16), which leaves few rescalings of O in tensor memory and 11 bits
// to weights down to 2^-23 of it.  With 2^7 and 2^8 the prompt takes 0.4 % less, with
// 2^11 and 2^4 1 % more.
#include <cuda_runtime.h>

#include <type_traits>

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
// Registers a thread: the launch gives 128 (512 threads) or 168 (384); the products' and the converting group hand
// some to the softmax's (2 * 176 + 2 * 80 = 4 * 128, 248 + 2 * 128 = 3 * 168)
template <int D>
constexpr int kRegsSoft = kGroups<D> == 2 ? 176 : 248;
template <int D>
constexpr int kRegsRest = kGroups<D> == 2 ? 80 : 128;
// a stage: f16 keys and values of a page; a slot: its codes
template <int D>
constexpr int kStageBytesKv = 2 * 64 * D * 2;
template <int D>
constexpr int kSlotBytes = 2 * 64 * D;
template <int D>
constexpr int kStagesKv = D == 64 ? 6 : D == 128 ? 4 : 2;
template <int D>
constexpr int kSlotsKv = D == 64 ? 12 : D == 256 ? 2 : 4;

// tensor memory columns
template <int D>
struct Cols {
  static constexpr int kQ = D / 2;                            // of a tile's queries
  static constexpr int kS = kGroups<D> * kQ;                  // two buffers of scores
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

// f16 x f16 -> fp32, M = 128
__host__ __device__ constexpr uint32_t idesc_f16(int n) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

// What the products' warp issues for a page and tile, by one election: P V into the output (o, from the weights at
// p and the values at vd; add: not the first page), then its arrivals, then the scores of a later page (s, from the
// queries at q and the keys at kd) with theirs.  An election for each product took 94 cycles whatever its size; with
// one for all, nothing else on the SM, a product of N columns takes its N / 2 cycles.  What is left out is left out by
// predicates: a second copy of the sequence would cost more than it saves, the SM's instruction cache being what is
// short.
#define RN_PV(A, B, ACC) \
  "add.u32 ra, %1, " #A ";\n\tadd.u64 rb, %2, " #B ";\n\t" \
  "@po tcgen05.mma.cta_group::1.kind::f16 [%0], [ra], rb, %3, " ACC ";\n\t"
#define RN_QK(A, B, ACC) \
  "add.u32 ra, %5, " #A ";\n\tadd.u64 rb, %6, " #B ";\n\t" \
  "@ps tcgen05.mma.cta_group::1.kind::f16 [%4], [ra], rb, %7, " ACC ";\n\t"
#define RN_ARRIVE(P, BAR) "@" P " tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [" BAR "];\n\t"
#define RN_HEAD                                                                                                      \
  "{\n\t.reg .pred e, po, ps, pe, add, yes, no;\n\t.reg .b32 ra;\n\t.reg .b64 rb;\n\t"                               \
  "setp.ne.u32 add, %8, 0;\n\tsetp.ne.u32 po, %9, 0;\n\tsetp.ne.u32 ps, %10, 0;\n\tsetp.ne.u32 pe, %11, 0;\n\t"      \
  "setp.eq.u32 yes, %8, %8;\n\tsetp.ne.u32 no, %8, %8;\n\telect.sync _|e, 0xffffffff;\n\t"                           \
  "and.pred po, po, e;\n\tand.pred ps, ps, e;\n\tand.pred pe, pe, e;\n\t"                                            \
  RN_PV(0, 0, "add") RN_PV(8, 2, "yes") RN_PV(16, 4, "yes") RN_PV(24, 6, "yes")                                      \
  RN_ARRIVE("pe", "%12") RN_ARRIVE("po", "%13")                                                                      \
  RN_QK(0, 0, "no") RN_QK(8, 2, "yes") RN_QK(16, 4, "yes") RN_QK(24, 6, "yes")
#define RN_TAIL                                                                                                      \
  RN_ARRIVE("ps", "%14")                                                                                             \
  "}" ::"r"(o), "r"(p), "l"(vd), "r"(ido), "r"(s), "r"(q), "l"(kd), "r"(ids), "r"((uint32_t)add),                    \
      "r"((uint32_t)has_o), "r"((uint32_t)has_s), "r"((uint32_t)frees), "r"(empty), "r"(obar), "r"(sbar) : "memory"
#define RN_QK64(A0, A1, A2, A3, B0, B1, B2, B3) \
  RN_QK(A0, B0, "yes") RN_QK(A1, B1, "yes") RN_QK(A2, B2, "yes") RN_QK(A3, B3, "yes")
template <int D>
__device__ __forceinline__ void issue_task(bool has_o, uint32_t o, uint32_t p, uint64_t vd, bool add, bool frees,
                                           uint32_t empty, uint32_t obar, bool has_s, uint32_t s, uint32_t q,
                                           uint64_t kd, uint32_t sbar) {
  constexpr uint32_t ido = idesc_f16(D), ids = idesc_f16(64);
  if constexpr (D == 64)
    asm volatile(RN_HEAD RN_TAIL);
  else if constexpr (D == 128)
    asm volatile(RN_HEAD RN_QK64(32, 40, 48, 56, 512, 514, 516, 518) RN_TAIL);
  else if constexpr (D == 192)
    asm volatile(RN_HEAD RN_QK64(32, 40, 48, 56, 512, 514, 516, 518)
                     RN_QK64(64, 72, 80, 88, 1024, 1026, 1028, 1030) RN_TAIL);
  else
    asm volatile(RN_HEAD RN_QK64(32, 40, 48, 56, 512, 514, 516, 518) RN_QK64(64, 72, 80, 88, 1024, 1026, 1028, 1030)
                     RN_QK64(96, 104, 112, 120, 1536, 1538, 1540, 1542) RN_TAIL);
}
#undef RN_PV
#undef RN_QK
#undef RN_QK64
#undef RN_ARRIVE
#undef RN_HEAD
#undef RN_TAIL

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
// 16 columns of it, both ways
__device__ __forceinline__ void tmem_load16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_store16(uint32_t taddr, const float (&v)[16]) {
  uint32_t r[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i]);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// 16 codes -> two 16-byte units of a swizzled row of f16
__device__ __forceinline__ void store16_f16(uint32_t row_addr, int row8, int sub, const uint4& v) {
  uint32_t h[8];
  e4m3x4_f16x4(v.x, h[0], h[1]);
  e4m3x4_f16x4(v.y, h[2], h[3]);
  e4m3x4_f16x4(v.z, h[4], h[5]);
  e4m3x4_f16x4(v.w, h[6], h[7]);
  sts128(row_addr + (((2 * sub) ^ row8) << 4), h[0], h[1], h[2], h[3]);
  sts128(row_addr + (((2 * sub + 1) ^ row8) << 4), h[4], h[5], h[6], h[7]);
}

// the largest; NaN where all are
__device__ __forceinline__ float max_of3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// what the copying warp says about a slot's page
struct SlotInfo {
  int from, to;        // positions of it that any row sees; none where there is no page
  int some;            // some rows may see only some of those
};
// what the converting warps say about a stage's page
struct PageInfo {
  uint32_t nan[2];     // positions whose values hold a NaN that is not in the stage
};
constexpr int kNoPage = 0x7FFF;

struct Stats {
  float m, M, l;
};

// What a (row tile, head) costs besides its pages, in pages (its queries' way into tensor memory, the first page's
// latency, the output: 11 000 cycles and more; a page 2200, both at dim 128 without options, the only ones measured)
constexpr int kExtra = 6;

// log2 of the weight at the reference M, and how far weights may go above it before M is raised: f16 ends at 2^16,
// has 11 bits down to 2^-14 and nothing below 2^-25.
constexpr float kTopWeight = 9.0f, kSlack = 6.5f;

template <int D, bool EXTRA>
__global__ void __launch_bounds__(kTileThreads<D>, 1) rn_kv_tile_kernel(const KvAttnParams p, int items) {
  constexpr int NG = kGroups<D>, R = kTileRows<D>, NT = kTileThreads<D>, NS = kStagesKv<D>;
  using C = Cols<D>;
  extern __shared__ unsigned char raw[];
  constexpr int NC = kSlotsKv<D>;
  __shared__ __align__(8) uint64_t full_b[NS], empty_b[NS], in_b[NC], out_b[NC], s_b[2], p_b[2], q_b, o_b[2];
  __shared__ uint32_t tmem_at;
  __shared__ PageInfo info[NS];
  __shared__ SlotInfo slot_info[NC];
  __shared__ Stats other[2][128];
  __shared__ Ranges<1, NT / 32> sh;
  const uint32_t ring = (smem_u32(raw) + 1023u) & ~1023u;
  const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
  const uint32_t codes = ring + NS * kStageBytesKv<D>;
  constexpr int kMma = 0, kCopy = 1, kConv = 4, kSoft = 8;
  unsigned* err = &g_err_kv_tile;

  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(smem_u32(&full_b[s]), 4);   // the converting warps
      mbar_init(smem_u32(&empty_b[s]), 1);  // the products that read the stage
    }
    for (int s = 0; s < NC; ++s) {
      mbar_init(smem_u32(&in_b[s]), 1);
      mbar_init(smem_u32(&out_b[s]), 4);    // the converting warps
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s_b[i]), 1);      // scores
      mbar_init(smem_u32(&p_b[i]), 4);      // weights: a tile's warps
      mbar_init(smem_u32(&o_b[i]), 1);      // a page's part of the output
    }
    mbar_init(smem_u32(&q_b), 4 * NG);      // queries: 4 warps a tile
    fence_barrier_init();
  }
  if (warp == kMma) tmem_alloc1(smem_u32(&tmem_at));
  tc_fence_before();
  pdl_launch_dependents();
  pdl_wait();
  Plan pl;
  const Dealt dealt = deal_pages<R, kExtra, 1, NT>(p, items, sh, pl);  // has barriers
  tc_fence_after();
  const int me = (int)blockIdx.x;
  Desc* desc = static_cast<Desc*>(p.ws);
  if (me >= dealt.workers) {
    if (tid == 0) desc[me].parts = 0;
  } else if (warp < kConv) {
    regs_down<kRegsRest<D>>();
    Walk<R, kExtra> at = walk_of<R, kExtra>(pl, dealt, sh, p.c.heads, me, 0);
    if (warp == kCopy) {
      // ---------------------------------------------------- copies
      // page numbers are read 32 at a time, one a lane
      int page = -1, batch = 0;
      auto fetch = [&]() {
        batch = at.blk;
        const int b = at.blk + lane;
        page = b < at.it.nblk ? kv_page(p.q, p.c.pages, at.it.b, at.it.blk0 + b) : -1;
      };
      fetch();
      RingPos r{0, 0};
      while (at.left > 0) {
        if (at.blk >= batch + 32) fetch();
        const int pg = __shfl_sync(0xFFFFFFFFu, page, at.blk - batch);
        mbar_wait(smem_u32(&out_b[r.slot]), r.phase ^ 1u, err, kErrEmptyWait);
        if (lane == 0) {
          const Item& it = at.it;
          const int base = (it.blk0 + at.blk) * 64;
          const int i0 = quot(it.r0, p.group), i1 = quot(it.r0 + it.rows - 1, p.group);
          const bool some = i1 > i0 && (base + 64 > (p.causal ? it.p0 + i0 + 1 : it.len) ||
                                        base < first_seen(it.p0 + i1, p.window));
          slot_info[r.slot] = SlotInfo{max(it.lo - base, 0), pg >= 0 ? min(it.hi - base, 64) : 0, some};
          // a page that is none is masked: any other stands for it
          const int64_t ph = (int64_t)max(pg, 0) * p.c.heads + at.head;
          const uint32_t to = codes + r.slot * kSlotBytes<D>, bar = smem_u32(&in_b[r.slot]);
          mbar_arrive_expect_tx(bar, kSlotBytes<D>);
          bulk_g2s(to, p.c.k + ph * 64 * D, 64 * D, bar);
          bulk_g2s(to + 64 * D, p.c.v + ph * 64 * D, 64 * D, bar);
        }
        __syncwarp();
        r.advance(1, NC);
        const int item = at.item;
        if (at.advance(pl, p.c.heads, 1) && (batch != 0 || at.item != item)) fetch();
      }
    }
    // ------------------------------------------------------ products
    RingPos rs{0, 0}, ro{0, 0};          // stages of the scores' pages, and of the outputs'
    uint32_t p_ph0 = 0, p_ph1 = 0, q_ph = 0;
    const uint64_t kd0 = smem_desc(ring, false), vd0 = smem_desc(ring + 64 * D * 2, false);
    constexpr uint32_t kStep = kStageBytesKv<D> >> 4;  // of the descriptors, a stage
    while (warp == kMma && at.left > 0) {
      const int cnt = at.segment();
      const bool both = NG == 2 && at.it.rows > 128;   // every page for both tiles
      const int tasks = both ? 2 * cnt : cnt;
      mbar_wait_warp(smem_u32(&q_b), q_ph, err, kErrReadyWait);
      q_ph ^= 1u;
      // task i: a page and the tile (or score buffer) x = i & 1; its scores are asked for two tasks ahead
      auto task = [&](auto xc, int i) {
        constexpr int x = decltype(xc)::value;
        constexpr uint32_t kSx = C::kS + 64 * x, kOx = C::kO + (NG == 2 ? x * D : 0), kQx = NG == 2 ? x * C::kQ : 0;
        const bool has_o = i >= 0, has_s = i + 2 < tasks;
        const bool frees = has_o && (x == 1 || !both);
        auto issue = [&](bool outputs, bool scores) {
          tc_fence_after();
          issue_task<D>(outputs, kOx, kSx, vd0 + ro.slot * kStep, i >= NG, outputs && frees,
                        smem_u32(&empty_b[ro.slot]), smem_u32(&o_b[x]), scores, kSx, kQx,
                        kd0 + rs.slot * kStep, smem_u32(&s_b[x]));
        };
        if (has_o) {
          uint32_t& ph = x ? p_ph1 : p_ph0;
          mbar_wait_warp(smem_u32(&p_b[x]), ph, err, kErrStatsWait);
          ph ^= 1u;
          // with two stages the page that the scores wait for needs the one that this frees
          if (NS == 2) issue(true, false);
        }
        if (has_s && (x == 0 || !both)) mbar_wait_warp(smem_u32(&full_b[rs.slot]), rs.phase, err, kErrFullWait);
        if (NS > 2 || has_s) issue(NS > 2 && has_o, has_s);
        if (frees) ro.advance(1, NS);
        if (has_s && (x == 1 || !both)) rs.advance(1, NS);
      };
      for (int i = -2; i < tasks; i += 2) {
        task(std::integral_constant<int, 0>{}, i);
        if (i + 1 < tasks) task(std::integral_constant<int, 1>{}, i + 1);
      }
      at.advance(pl, p.c.heads, cnt);
    }
  } else if (warp < kSoft) {
    // ------------------------------------------------------ codes to f16
    regs_down<kRegsRest<D>>();
    const int cw = warp - kConv, sub = lane & 3, row8 = lane >> 2;
    RingPos r{0, 0}, in{0, 0};
    Walk<R, kExtra> at = walk_of<R, kExtra>(pl, dealt, sh, p.c.heads, me, 0);
    for (; at.left > 0; at.advance(pl, p.c.heads, 1)) {
      mbar_wait(smem_u32(&in_b[in.slot]), in.phase, err, kErrFullWait);
      const SlotInfo si = slot_info[in.slot];
      // Keys: a warp takes 8 positions x 64 dims at a time, values 8 dims x 64 positions: 8 lanes read 128 bytes of
      // different banks and write 128 bytes of different banks (of two rows; of two blocks of 64 dims where the
      // rows lie a multiple of 128 bytes apart).  All are read first: one after another, a page took 1300 cycles.
      const uint32_t kc = codes + in.slot * kSlotBytes<D> + sub * 16, vc = kc + 64 * D;
      uint4 kv[D / 32], vv[D / 32];
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const int blk = D % 128 == 0 ? (i >> 1) ^ (row8 & 1) : i >> 1;
        kv[i] = lds128(kc + (8 * (cw + 4 * (i & 1)) + row8) * D + blk * 64);
      }
#pragma unroll
      for (int i = 0; i < D / 32; ++i) vv[i] = lds128(vc + (8 * (4 * i + cw) + row8) * 64);
      mbar_wait(smem_u32(&empty_b[r.slot]), r.phase ^ 1u, err, kErrEmptyWait);
      const uint32_t kb = ring + r.slot * kStageBytesKv<D>, vb = kb + 64 * D * 2;
      const bool plain = si.from <= 0 && si.to >= 64 && !si.some;
      if (warp == kConv && lane == 0) info[r.slot] = PageInfo{{0u, 0u}};
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const int row = 8 * (cw + 4 * (i & 1)) + row8;
        const int blk = D % 128 == 0 ? (i >> 1) ^ (row8 & 1) : i >> 1;
        store16_f16(kb + blk * 8192 + row * 128, row8, sub, kv[i]);
      }
      if (plain) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) store16_f16(vb + (8 * (4 * i + cw) + row8) * 128, row8, sub, vv[i]);
      } else {
        // what no row sees is not looked at; a NaN that only some rows see reaches those by their weights
        uint32_t keep[4], nan[4] = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          keep[j] = 0;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int pos = 16 * sub + 4 * j + q;
            if (pos >= si.from && pos < si.to) keep[j] |= 0xFFu << (8 * q);
          }
        }
#pragma unroll 1
        for (int i = 0; i < D / 32; ++i) {
          const int row = 8 * (4 * i + cw) + row8;
          const uint4 v = lds128(vc + row * 64);
          uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            w[j] &= keep[j];
            if (si.some) {
              const uint32_t bad = ((w[j] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
              nan[j] |= bad;
              w[j] &= ~((bad >> 7) * 0xFFu);
            }
          }
          store16_f16(vb + row * 128, row8, sub, make_uint4(w[0], w[1], w[2], w[3]));
        }
        if (si.some) {
          // 16 positions of this lane as bits; then those of the warp
          uint32_t bits = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) bits |= (nan[j] >> (8 * q + 7) & 1u) << (4 * j + q);
          bits <<= 16 * (sub & 1);
          const uint32_t lo = __reduce_or_sync(0xFFFFFFFFu, sub < 2 ? bits : 0u);
          const uint32_t hi = __reduce_or_sync(0xFFFFFFFFu, sub < 2 ? 0u : bits);
          asm volatile("bar.sync 2, 128;" ::: "memory");  // the stage's bits are clear
          if (lane == 0 && (lo | hi) != 0) {
            atomicOr(&info[r.slot].nan[0], lo);
            atomicOr(&info[r.slot].nan[1], hi);
          }
        }
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(smem_u32(&full_b[r.slot]));
        mbar_arrive(smem_u32(&out_b[in.slot]));
      }
      r.advance(1, NS);
      in.advance(1, NC);
    }
  } else {
    // ------------------------------------------------------ softmax
    regs_up<kRegsSoft<D>>();
    Walk<R, kExtra> at = walk_of<R, kExtra>(pl, dealt, sh, p.c.heads, me, 0);
    const int x = (warp - kSoft) >> 2;                   // the tile
    if (warp == kSoft && lane == 0) desc[me].parts = 0;  // for a range without pages
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tq = lanes + x * C::kQ, to = lanes + C::kO + x * D;
    const int in_tile = (warp & 3) * 32 + lane;
    uint32_t done0 = 0, done1 = 0;                       // pages of the buffers so far (NG = 2: of the tile's)
    RingPos r{0, 0};
    // Whose turn it is of `other`: a segment of one page asks nothing of the odd warps, so they may be at the next
    // one's statistics before the even warps have read these; they wait for them at that one's barrier.
    int turn = 0;
    while (at.left > 0) {
      const Item& it = at.it;
      const int head = at.head, cnt = at.segment();
      const bool begins = at.blk == 0, ends = at.blk + cnt == it.nblk;
      const bool both = NG == 2 && it.rows > 128, split = NG == 2 && !both;
      const int row_in = both ? x * 128 + in_tile : in_tile;
      const int rr = it.r0 + min(row_in, it.rows - 1);
      const int qi = quot(rr, p.group), qh = head * p.group.d + rr - qi * p.group.d;
      float qs;
      {
        // the query row in f16, its largest magnitude at 2^14
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.x) +
                                                          (int64_t)(it.s0 + qi) * p.stride + (int64_t)qh * D);
        const bool real = row_in < it.rows;
        // the whole row at once: its loads are on their way together
        uint4 w4[D / 8];
#pragma unroll
        for (int c = 0; c < D / 8; ++c) w4[c] = real ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
        uint32_t big = 0;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint32_t w[4] = {w4[c].x, w4[c].y, w4[c].z, w4[c].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t lo = w[j] & 0x7FFFu, hi = w[j] >> 16 & 0x7FFFu;
            if (lo < 0x7F80u) big = max(big, lo);
            if (hi < 0x7F80u) big = max(big, hi);
          }
        }
        const int up = max((int)(big >> 7) - 127 - 14, kKvExpMin);
        const float mul = pow2i(-up);
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint32_t h[32];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float f[8];
            bf16x8_to_f32(w4[c * 8 + j], f);
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
      const int row_hi = p.causal ? pos0 + 1 : it.len, row_lo = first_seen(pos0, p.window);
      const int i0 = quot(it.r0, p.group), i1 = quot(it.r0 + it.rows - 1, p.group);
      const int all_hi = p.causal ? it.p0 + i0 + 1 : it.len, all_lo = first_seen(it.p0 + i1, p.window);
      float slope = 0.0f;
      if constexpr (EXTRA)
        if (p.slopes != nullptr) slope = __ldg(p.slopes + qh) * kLog2e;

      float m = -INFINITY, M = -INFINITY, l = 0.0f;
      const int step = split ? 2 : 1, first = split ? x : 0;
      if (split && x == 1) r.advance(1, NS);
      // the scales of 32 pages, one a lane: the keys' exponent in the low half (kNoPage: no page)
      int scales = 0, batch = first - 32;
#pragma unroll 1
      for (int c = first; c < cnt; c += step) {
        if (c >= batch + 32) {
          batch = c;
          const int b = at.blk + c + lane;
          const int pg = b < it.nblk ? kv_page(p.q, p.c.pages, it.b, it.blk0 + b) : -1;
          const int64_t ph = (int64_t)pg * p.c.heads + head;
          scales = pg >= 0 ? (kv_exp(p.c.vs[ph]) << 16) | (kv_exp(p.c.ks[ph]) & 0xFFFF) : kNoPage;
        }
        const int sc = __shfl_sync(0xFFFFFFFFu, scales, c - batch), ek = (int16_t)sc;
        const int base = (it.blk0 + at.blk + c) * 64;
        const bool there = ek != kNoPage;
        const float ev = (float)(sc >> 16);
        const float f = qs * pow2i(there ? ek : 0);
        const bool edge = !there || base < all_lo || base + 64 > all_hi;
        uint32_t nan[2] = {0, 0};
        if (edge) {
          mbar_wait(smem_u32(&full_b[r.slot]), r.phase, err, kErrFullWait);
          nan[0] = info[r.slot].nan[0];
          nan[1] = info[r.slot].nan[1];
        }
        const int buf = NG == 2 ? x : c & 1;
        const uint32_t ts = lanes + C::kS + 64 * buf;
        mbar_wait(smem_u32(&s_b[buf]), (NG == 2 || buf == 0 ? done0 : done1) & 1, err, kErrStatsWait);
        __syncwarp();
        tc_fence_after();
        if constexpr (EXTRA) {
          // Capped and biased 16 at a time, back where they were: as a part of the 64 below, this would be four times
          // the instructions, more than the SM's instruction cache holds (4 x 1024, groups of 4, biased 230 us, now 104;
          // 4096 on 8192 with a cap 5970, now 2577, without one 1279).
          const float inv_cap = 1.0f / p.softcap;
#pragma unroll 1
          for (int h = 0; h < 64; h += 16) {
            float z[16];
            tmem_load16(ts + h, z);
            tmem_load_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) z[i] *= f;
            if (p.softcap > 0.0f) cap_scores(z, p.softcap, inv_cap);
            const float away = (float)(base + h - pos0);
#pragma unroll
            for (int i = 0; i < 16; ++i) z[i] = fmaf(slope, away + (float)i, z[i] * kLog2e);
            tmem_store16(ts + h, z);
          }
          tmem_store_wait();
        }
        float s[64];
        tmem_load32(ts, reinterpret_cast<float(&)[32]>(s));
        tmem_load32(ts + 32, reinterpret_cast<float(&)[32]>(s[32]));
        tmem_load_wait();
        float mul = EXTRA ? 1.0f : f;
        if (edge) {
          mul = 1.0f;
#pragma unroll
          for (int i = 0; i < 64; ++i) {
            const int pos = base + i;
            float z = EXTRA ? s[i] : s[i] * f;
            const bool sees = there && pos >= row_lo && pos < row_hi;
            if (nan[i >> 5] >> (i & 31) & 1) z = __uint_as_float(0x7FC00000u);
            if (!sees) z = -INFINITY;
            s[i] = z;
          }
        }
        float top4[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) top4[i] = max_of3(s[3 * i], s[3 * i + 1], s[3 * i + 2]);
#pragma unroll
        for (int i = 12; i < 64; i += 2) top4[i / 2 & 3] = max_of3(top4[i / 2 & 3], s[i], s[i + 1]);
        float top = fmaxf(max_of3(top4[0], top4[1], top4[2]), top4[3]);
        if (top != top) top = -INFINITY;  // NaN everywhere: the weights carry it
        top *= mul;
        const float m2 = fmaxf(m, top);
        const float base_m = m2 == -INFINITY ? 0.0f : m2;
        const bool raise = top + ev > M + kSlack;
        if (__any_sync(0xFFFFFFFFu, raise)) {
          const float M2 = raise ? top + ev : M;
          if (c != first) {
            // The output holds the pages before: with two tiles, a page's scores were asked for after the tile's page
            // before had been added; with one, after the one before that.
            if constexpr (NG == 1)
              mbar_wait(smem_u32(&o_b[buf ^ 1]), ((buf == 0 ? done1 : done0) - 1) & 1, err, kErrStatsWait);
            __syncwarp();
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
        // 2^sub: the unit of this page's weights.  Where the values are so small that no weight reaches f16, a finer
        // one, in which the sum of the weights loses nothing.
        const float sub = top == -INFINITY ? 0.0f : fminf(M - ev - kTopWeight, top + 90.0f);
        uint32_t w[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float2 z = fma2(make_float2(s[2 * i], s[2 * i + 1]), splat2(mul), splat2(-sub));
          s[2 * i] = ex2(z.x);
          s[2 * i + 1] = ex2(z.y);
          w[i] = pack_f16x2(s[2 * i], s[2 * i + 1]);
        }
        tmem_store32(ts, w);
        tmem_store_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&p_b[buf]));
        if (NG == 2 || buf == 0) ++done0;
        else ++done1;
        // the sum is not waited for
        float2 sum[4] = {};
#pragma unroll
        for (int i = 0; i < 32; ++i) sum[i & 3] = add2(sum[i & 3], make_float2(s[2 * i], s[2 * i + 1]));
        sum[0] = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
        l = l * ex2(m - base_m) + (sum[0].x + sum[0].y) * ex2(fminf(sub - base_m, 126.0f));
        m = m2;
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
      if (!split || x < cnt) {
        const int b = NG == 2 ? x : (cnt - 1) & 1;
        mbar_wait(smem_u32(&o_b[b]), ((NG == 2 || b == 0 ? done0 : done1) - 1) & 1, err, kErrStatsWait);
      }
      __syncwarp();
      tc_fence_after();
      float mo = -INFINITY, Mo = -INFINITY, lo = 0.0f;   // of the odd pages
      if (split) {
        if (x == 1) other[turn][in_tile] = Stats{m, M, l};
        tc_fence_before();
        asm volatile("bar.sync 1, 256;" ::: "memory");
        tc_fence_after();
        if (x == 0) {
          const Stats odd_ones = other[turn][in_tile];
          mo = odd_ones.m, Mo = odd_ones.M, lo = odd_ones.l;
        }
        turn ^= 1;
      }
      if (!(split && x == 1)) {
        const bool odd = split && cnt > 1;
        const float mm = fmaxf(m, mo), MM = fmaxf(M, Mo);
        const float bm = mm == -INFINITY ? 0.0f : mm, bM = MM == -INFINITY ? 0.0f : MM;
        const float sum = l * ex2(m - bm) + lo * ex2(mo - bm);
        // 2^(M - 9 - m); in two halves where it may be below the normal floats, as the values of the pages are least
        float power = bM - kTopWeight - bm;
        const bool halves = __any_sync(0xFFFFFFFFu, power < -90.0f);
        if (halves) power *= 0.5f;
        const float unit = sum == 0.0f ? 0.0f : ex2(power) / sum;
        const float fa = unit * ex2(M - bM), fb = unit * ex2(Mo - bM);
        const float log2s = sum == 0.0f ? -INFINITY : bm + log2f(sum);
        const int64_t row = (int64_t)(it.s0 + qi) * (p.c.heads * p.group.d) + qh;
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
          if (halves) {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= ex2(power);
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
      if (at.is_last(cnt) && warp == kSoft && lane == 0)
        desc[me] = desc_of(dealt, 1, begins && !ends ? dealt.start(me + 1) + (it.nblk - at.blk - cnt) : 0, it.s0,
                           it.r0, it.rows, head);
      at.advance(pl, p.c.heads, cnt);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMma) tmem_free1(tmem_at);
}

template <int D, bool EXTRA>
rn_status launch_e(const KvAttnParams& p, int sms, cudaStream_t s) {
  constexpr size_t smem = (size_t)kStagesKv<D> * kStageBytesKv<D> + (size_t)kSlotsKv<D> * kSlotBytes<D> + 1024;
  auto k = rn_kv_tile_kernel<D, EXTRA>;
  static std::atomic<int> kept[kMaxDevices];
  if (once_per_device(kept, [&] {
        return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) == cudaSuccess ? 1 : -1;
      }) < 1)
    return RN_ERR_CUDA;
  const int items = (int)((int64_t)p.q.tokens * p.group.d / kTileRows<D>) + p.q.B;
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
