// Attention of a sequence's newest tokens with its positions in the paged
// 8-bit cache, for few rows a key/value head (decoding, drafted tokens).
//
//   s_ij = scale q_i . k_j        (then c tanh(s / c), then + slope (j - p_i))
//   out_i = sum_j exp(s_ij - m_i) v_j / sum_j exp(s_ij - m_i)
//
// One pass over the pages with running maxima and sums.  A page's key scale
// 2^eK multiplies its scores; its value scale 2^eV goes into the weights:
// besides the maximum m of the scores a second one, M, of the scores plus eV
// (in base 2) scales the weights w = 2^(s + eV - M + 15) <= 2^15 that multiply
// the value codes, so that no page's contribution is lost in 16 bits however far
// the pages' scales and scores lie apart.  The sum of exp(s - m) is kept in fp32.
//
// The products are mma.sync m16n8k16 on f16 with the cache as the 16 rows and
// the queries as the 8 columns: S^T = K Q^T, O^T = V^T P^T.  Codes become f16
// by one conversion a pair, exactly; a query row becomes f16 times the power of
// two that puts its largest magnitude at 2^14 (what is 2^28 below it loses
// bits: 2^-39 of the row's largest); weights are rounded to f16, half a step of
// 2^-11 down to 2^-29 of the largest, which the bf16 output's 2^-8 covers.  Sums
// are fp32.  m + eV and the like are exact up to |m| = 2^23: whole numbers on
// multiples of 1/2.
//
// Which positions the rows and which dims the reduction index of a fragment
// stand for is free as long as both operands agree, so a lane reads 16
// contiguous codes at a time: for lane (g, t), g = lane / 4, t = lane % 4, the
// 16 dims 64 c + 16 t .. of a key give four products' operands, and so do the 16
// positions 16 t .. of a dim of V.  Row r of product st of S^T stands for position
// 16 (r / 2 % 4) + 4 st + 2 (r / 8) + r % 2 then.  The weights come out as rows
// of positions and are wanted as columns: movmatrix turns 8 x 8 of them.
//
// A worker is one warp with a ring of slots of its own, filled by bulk copies
// of whole pages (keys and values of 64 positions are contiguous, 64 dim
// bytes each; half pages where dim > 128).  The (row tile, head, page) triples of
// the call, in this order, are dealt evenly to all workers, so ragged lengths
// cost nothing.  A (row tile, head) that several workers share is joined from
// their partial results in the workers' order: by their CTA, and where it goes
// beyond one CTA, by a second kernel.
//
// What bounds it: the cache's bytes, with about 15 us around them.  64 sequences
// of up to 16384, 8 heads of 128, groups of 8 (1.24 GB): 206 us, 6.02 TB/s, 0.90 of
// the measured copy rate; one of 131072 (268 MB, 40 us at that rate) 55 us, 4.9 TB/s:
// besides the bytes the launches, the dealing, the first pages' latency and two
// joins.  The rest of a small call (1000 positions: 9.4 us) is latency: the call's
// arrays, the page table, the page, the join.  9 to 16 rows double the products and
// exponentials of a page: 32 sequences of 8192, 4 heads, groups of 16 69 us (floor 40).
#include <cuda_runtime.h>

#include <type_traits>

#include "rn_device.cuh"
#include "rn_internal.h"
#include "rn_kv.cuh"
#include "rn_kv_plan.cuh"

namespace rn {
namespace {

__device__ unsigned g_err_kv;

// A CTA's warps have 192 KB of slots, each of a page's keys or values, or half of
// them (dim > 128: positions 0 .. 31 and 32 .. 63 of the keys, the dims' halves of
// the values).
constexpr int kWarps = 8;
template <int D>
constexpr int kHalves = D > 128 ? 2 : 1;
template <int D>
constexpr int kPiece = 64 * D / kHalves<D>;
template <int D>
constexpr int kSlots = 196608 / (kWarps * kPiece<D>);

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t turn8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// over the lanes whose numbers differ in the bits from FROM on
template <int FROM>
__device__ __forceinline__ float max_from(float v) {
#pragma unroll
  for (int o = FROM; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}
template <int FROM>
__device__ __forceinline__ float sum_from(float v) {
#pragma unroll
  for (int o = FROM; o < 32; o <<= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
// over the 8 lanes with the same t
__device__ __forceinline__ uint32_t or_g(uint32_t v) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) v |= __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// bytes [from, to) of a word's four, as ones
__device__ __forceinline__ uint32_t byte_range(int from, int to) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m |= (i >= from && i < to) ? 0xFFu << (8 * i) : 0u;
  return m;
}

// A row put together from partial results, which are normalized: the weighted
// mean and the log2 of the weights' sum (-infinity: none).  Lane i holds the dims
// 2 i + 64 c and the one behind.
template <int D>
struct Joined {
  float2 acc[D / 64];
  float top;
};

// The root of a part's share 2^(l - top), multiplied in twice: the share may be below the normal floats, and the part's
// values as far above 1.
__device__ __forceinline__ float share_root(float l, float top) {
  return ex2(0.5f * (l - (top == -INFINITY ? 0.0f : top)));
}
template <int D>
__device__ __forceinline__ void add_part(float2 (&acc)[D / 64], const float2 (&v)[D / 64], float root) {
#pragma unroll
  for (int c = 0; c < D / 64; ++c) {
    acc[c].x = fmaf(v[c].x * root, root, acc[c].x);
    acc[c].y = fmaf(v[c].y * root, root, acc[c].y);
  }
}
template <int D>
__device__ __forceinline__ void load_part(float2 (&v)[D / 64], const float* part, int row, int lane) {
#pragma unroll
  for (int c = 0; c < D / 64; ++c) v[c] = *reinterpret_cast<const float2*>(part + row * D + c * 64 + 2 * lane);
}
template <int D>
__device__ __forceinline__ Joined<D> finish(const float2 (&acc)[D / 64], float top, float sum) {
  Joined<D> j;
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int c = 0; c < D / 64; ++c) j.acc[c] = make_float2(acc[c].x * inv, acc[c].y * inv);
  j.top = sum == 0.0f ? -INFINITY : top + log2f(sum);
  return j;
}

// Row `row` of the parts i0, i0 + step .. of n, each R rows of D and then the rows' log2 sums; the loads of four
// parts are on their way together.
template <int D, class Part>
__device__ __forceinline__ Joined<D> join_parts(int n, int i0, int step, int lane, int row, int R, Part part) {
  float2 acc[D / 64] = {};
  float top = -INFINITY, sum = 0.0f;
  for (int i = i0; i < n; i += 4 * step) {
    float2 v[4][D / 64];
    float l[4], now = top;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float* at = part(min(i + k * step, n - 1));
      l[k] = at[R * D + row];
      load_part<D>(v[k], at, row, lane);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (i + k * step >= n) l[k] = -INFINITY;
      now = fmaxf(now, l[k]);
    }
    const float base = now == -INFINITY ? 0.0f : now, keep = ex2(0.5f * (top - base));
    top = now;
    sum *= keep * keep;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) acc[c] = make_float2(acc[c].x * keep * keep, acc[c].y * keep * keep);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (i + k * step >= n) continue;
      const float root = share_root(l[k], base);
      sum = fmaf(root, root, sum);
      add_part<D>(acc, v[k], root);
    }
  }
  return finish<D>(acc, top, sum);
}
// the row as a partial result again
template <int D>
__device__ __forceinline__ void store_part(const Joined<D>& j, float* part, int row, int R, int lane) {
#pragma unroll
  for (int c = 0; c < D / 64; ++c) *reinterpret_cast<float2*>(part + row * D + c * 64 + 2 * lane) = j.acc[c];
  if (lane == 0) part[R * D + row] = j.top;
}
template <int D>
__device__ __forceinline__ void store_joined(const KvAttnParams& p, const Joined<D>& j, int64_t row, int lane) {
  uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + row * D);
#pragma unroll
  for (int c = 0; c < D / 64; ++c) out[c * 32 + lane] = pack_bf16x2(j.acc[c].x, j.acc[c].y);
  if (p.lse != nullptr && lane == 0) p.lse[row] = j.top * kLn2;
}

// Rows row0 .. row0 + RB - 1 of n <= 8 parts at once, for one warp: the sums one a lane (of row lane % RB), the loads of
// a part's rows on their way together.
template <int D, int RB, class Part, class Store>
__device__ __forceinline__ void join_rows(int n, int lane, int row0, int rows, int R, Part part, Store store) {
  constexpr int kAtOnce = 32 / RB, kTimes = RB / 4;   // sums of kAtOnce parts at a time
  static_assert(kAtOnce * kTimes == 8 && kTimes <= 2, "8 parts");
  float2 v[RB][D / 64], acc[RB][D / 64] = {};
  auto load = [&](int i) {
#pragma unroll
    for (int k = 0; k < RB; ++k) load_part<D>(v[k], part(i), min(row0 + k, rows - 1), lane);
  };
  float root[kTimes], top = -INFINITY, sum = 0.0f;
#pragma unroll
  for (int h = 0; h < kTimes; ++h) {
    const int i = lane / RB + h * kAtOnce;
    root[h] = i < n ? part(i)[R * D + min(row0 + lane % RB, rows - 1)] : -INFINITY;
    top = fmaxf(top, root[h]);
  }
  load(0);
  top = max_from<RB>(top);
#pragma unroll
  for (int h = 0; h < kTimes; ++h) {
    root[h] = share_root(root[h], top);
    sum = fmaf(root[h], root[h], sum);
  }
  sum = sum_from<RB>(sum);
#pragma unroll 1
  for (int i = 0;;) {
    const float mine = i < kAtOnce ? root[0] : root[kTimes - 1];
#pragma unroll
    for (int k = 0; k < RB; ++k) add_part<D>(acc[k], v[k], __shfl_sync(0xFFFFFFFFu, mine, i % kAtOnce * RB + k));
    if (++i >= n) break;
    load(i);
  }
#pragma unroll
  for (int k = 0; k < RB; ++k) {
    const float t = __shfl_sync(0xFFFFFFFFu, top, k), of_row = __shfl_sync(0xFFFFFFFFu, sum, k);
    if (row0 + k >= rows) break;
    store(row0 + k, finish<D>(acc[k], t, of_row));
  }
}

constexpr int kNoScales = 256;  // no page

// log2 of the largest weight in f16, whose values end at 2^16: the others have 11 bits down to 2^-29 of it, and vanish
// below 2^-40.  With 2^0 they had them to 2^-14 and vanished below 2^-25, which lost the output of a row whose first
// position takes 0.995 of the weight and has values near 0.
constexpr float kTopWeight = 15.0f;

// what the join within the CTA has to know of a worker's range
struct WorkerEnd {
  int within, closes;        // it begins within a (row tile, head), and holds its last page
  int opens;                 // it begins one that it does not finish
  int s0, r0, rows, head;    // that one
  int64_t end;               // where its pages end
  int rows0;                 // of the one that it begins within
};

template <int D, int NB, bool EXTRA>
__global__ void __launch_bounds__(32 * kWarps, 1) rn_kv_attn_kernel(const KvAttnParams p, int items) {
  constexpr int R = 8 * NB, W = kWarps, S = kSlots<D>, PIECE = kPiece<D>, PH = kHalves<D>;
  extern __shared__ __align__(1024) unsigned char raw[];
  __shared__ __align__(8) uint64_t full_b[W][S];
  __shared__ Ranges<W, W> sh;
  __shared__ WorkerEnd ends_of[W];
  const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  if (lane == 0) {
    for (int s = 0; s < S; ++s) mbar_init(smem_u32(&full_b[warp][s]), 1);
    fence_barrier_init();
  }
  pdl_launch_dependents();
  pdl_wait();

  Plan pl;
  const Dealt dealt = deal_pages<R, 0, W, 32 * W>(p, items, sh, pl);
  const int me = (int)blockIdx.x * dealt.per_cta + warp;
  Desc* desc = static_cast<Desc*>(p.ws);
  if (me >= dealt.workers && warp == 0) {  // nothing for this CTA
    if (lane == 0) desc[blockIdx.x].parts = 0;
    return;  // as its other warps do, below
  }
  if ((int)blockIdx.x * dealt.per_cta >= dealt.workers) return;
  const bool works = warp < dealt.per_cta && me < dealt.workers;
  const uint32_t ring = smem_u32(raw) + warp * (S * PIECE);
  auto bar = [&](int s) { return smem_u32(&full_b[warp][s]); };

  // ------------------------------------------------------------- copies
  // Page numbers are read 32 at a time, one a lane, and the next ones while these are used; the scales of a slot's
  // page are in the lane with the slot's number.
  using Range = Walk<R, 0>;
  Range ld{};
  if (works) ld = walk_of<R, 0>(pl, dealt, sh, p.c.heads, me, warp);
  Range at = ld;
  int pages = -1, pages_next = -1, batch = 0, ks = 0, vs = 0;
  auto read_pages = [&](const Item& it, int blk) {
    const int b = blk + lane;
    return b < it.nblk ? kv_page(p.q, p.c.pages, it.b, it.blk0 + b) : -1;
  };
  // a batch begins at the cursor: asks for the one behind it
  auto look_ahead = [&]() {
    batch = ld.blk;
    if (batch + 32 < ld.it.nblk) {
      pages_next = read_pages(ld.it, batch + 32);
    } else {
      Range next = ld;
      if (next.advance(pl, p.c.heads, next.segment())) pages_next = read_pages(next.it, 0);
    }
  };
  if (works) {
    pages = read_pages(ld.it, ld.blk);
    look_ahead();
  }
  uint32_t slot_l = 0;
  int piece = 0, ld_page = -1;   // the next piece of the page: keys, then values
  auto issue = [&]() {
    if (ld.left == 0) return;
    if (piece == 0) ld_page = __shfl_sync(0xFFFFFFFFu, pages, ld.blk - batch);
    // a page that is none is masked: any other stands for it
    const int64_t ph = (int64_t)max(ld_page, 0) * p.c.heads + ld.head;
    if (lane == 0) {
      const uint8_t* from = (piece < PH ? p.c.k : p.c.v) + ph * 64 * D + (piece % PH) * PIECE;
      mbar_arrive_expect_tx(bar(slot_l), PIECE);
      bulk_g2s(ring + slot_l * PIECE, from, PIECE, bar(slot_l));
    }
    if (piece == 0 && lane == slot_l) {
      ks = ld_page >= 0 ? (int)p.c.ks[ph] : kNoScales;
      vs = p.c.vs[ph];
    }
    if (++slot_l == S) slot_l = 0;
    if (++piece == 2 * PH) {
      piece = 0;
      if (ld.advance(pl, p.c.heads, 1) || ld.blk == batch + 32) {
        pages = pages_next;
        look_ahead();
      }
    }
  };
#pragma unroll 1
  for (int i = 0; i < S; ++i) issue();
  __syncwarp();

  // ------------------------------------------------------------- the pages
  RingPos r{0, 0};
  auto wait_slots = [&](int n) {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const RingPos a = r.ahead(i, S);
      mbar_wait(bar(a.slot), a.phase, &g_err_kv, kErrFullWait);
    }
  };
  auto free_slots = [&](int n) {
    __syncwarp();
    r.advance(n, S);
#pragma unroll
    for (int i = 0; i < n; ++i) issue();
  };
  if (lane == 0) ends_of[warp] = WorkerEnd{};
  const float inv_cap = EXTRA ? 1.0f / p.softcap : 0.0f;
  while (at.left > 0) {
    const Item& it = at.it;
    const int head = at.head, blk = at.blk;
    // queries of the segment as operands: lane (g, t) holds row g's dims
    const int cnt = at.segment();
    const bool begins = blk == 0, ends = blk + cnt == it.nblk;
    uint32_t q[NB][D / 16][2];
    float qs[NB][2];      // scale of the scores of rows 2t, 2t + 1, without the page's
    int row_hi[NB][2], row_lo[NB][2];
    float slope[NB][2];
    int row_p[NB][2];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const int r = it.r0 + n * 8 + g, qi = quot(r, p.group);
      const bool real = n * 8 + g < it.rows;
      uint4 raw4[D / 64][2];
      uint32_t big = 0;
      const unsigned char* src =
          static_cast<const unsigned char*>(p.x) +
          ((int64_t)(it.s0 + qi) * p.stride + (int64_t)(head * p.group.d + r - qi * p.group.d) * D + 16 * t) * 2;
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          raw4[c][h] = real ? __ldg(reinterpret_cast<const uint4*>(src + c * 128 + h * 16)) : make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {raw4[c][h].x, raw4[c][h].y, raw4[c][h].z, raw4[c][h].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t a = w[i] & 0x7FFFu, b = w[i] >> 16 & 0x7FFFu;
            if (a < 0x7F80u) big = max(big, a);
            if (b < 0x7F80u) big = max(big, b);
          }
        }
      big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 1));
      big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 2));
      // largest magnitude's exponent - 14; rows below 2^-106 keep fewer bits
      const int up = max((int)(big >> 7) - 127 - 14, kKvExpMin);
      const float mul = pow2i(-up);
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float f[8];
          bf16x8_to_f32(raw4[c][h], f);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            q[n][4 * c + 2 * h + i / 2][i % 2] = pack_f16x2(f[2 * i] * mul, f[2 * i + 1] * mul);
        }
      const float own = EXTRA ? pow2i(up) * p.scale : pow2i(up) * (p.scale * kLog2e);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        qs[n][j] = __shfl_sync(0xFFFFFFFFu, own, (2 * t + j) * 4);
        const int rr = it.r0 + min(n * 8 + 2 * t + j, it.rows - 1), i = quot(rr, p.group);
        row_p[n][j] = it.p0 + i;
        row_hi[n][j] = p.causal ? row_p[n][j] + 1 : it.len;
        row_lo[n][j] = first_seen(row_p[n][j], p.window);
        if constexpr (EXTRA)
          slope[n][j] =
              p.slopes != nullptr ? __ldg(p.slopes + head * p.group.d + rr - i * p.group.d) * kLog2e : 0.0f;
      }
    }
    // every row sees [all_lo, all_hi)
    const int i0 = quot(it.r0, p.group), i1 = quot(it.r0 + it.rows - 1, p.group);
    const int all_hi = p.causal ? it.p0 + i0 + 1 : it.len;
    const int all_lo = first_seen(it.p0 + i1, p.window);
    const bool several = i1 > i0;

    float m[NB][2], M[NB][2], l[NB][2], o[NB][D / 16][4];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
#pragma unroll
      for (int j = 0; j < 2; ++j) m[n][j] = M[n][j] = -INFINITY, l[n][j] = 0.0f;
#pragma unroll
      for (int d = 0; d < D / 16; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[n][d][i] = 0.0f;
    }

#pragma unroll 1
    for (int c = 0; c < cnt; ++c) {
      const int base = (it.blk0 + blk + c) * 64;
      wait_slots(PH);
      const int kbyte = __shfl_sync(0xFFFFFFFFu, ks, r.slot), vbyte = __shfl_sync(0xFFFFFFFFu, vs, r.slot);
      const bool there = kbyte != kNoScales;
      // positions of the page that any row sees
      const int from = there ? max(it.lo - base, 0) : 64, to = there ? min(it.hi - base, 64) : 0;
      const bool edge = !there || base < all_lo || base + 64 > all_hi;

      float s[NB][4][4];
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int st = 0; st < 4; ++st)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[n][st][i] = 0.0f;
      {
        // dim > 128: the positions 16 (g / 2) .. of lanes g >= 4 are in the second slot
        const int key = 16 * (g >> 1) + (g & 1);
        const uint32_t from_slot = PH == 1 ? r.slot : (g < 4 ? r.slot : r.ahead(1, S).slot);
        const uint32_t at = ring + from_slot * PIECE + (PH == 1 ? key : key & 31) * D + 16 * t;
#pragma unroll
        for (int st = 0; st < 4; ++st)
#pragma unroll
          for (int d = 0; d < D / 64; ++d) {
            const uint4 k0 = lds128(at + (4 * st) * D + 64 * d), k1 = lds128(at + (4 * st + 2) * D + 64 * d);
            const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t a[4];
              e4m3x4_f16x4(w0[i], a[0], a[2]);
              e4m3x4_f16x4(w1[i], a[1], a[3]);
#pragma unroll
              for (int n = 0; n < NB; ++n) mma_f16(s[n][st], a, q[n][4 * d + i][0], q[n][4 * d + i][1]);
            }
          }
      }
      free_slots(PH);

      // scores in base 2, maxima, weights
      const float unit = pow2i(there ? kv_exp(kbyte) : 0), ev = (float)kv_exp(vbyte);
      uint32_t pw[NB][4][2];
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        float top[2] = {-INFINITY, -INFINITY}, score[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) score[i] = s[n][i >> 2][i & 3] * (qs[n][i & 1] * unit);
        if constexpr (EXTRA)
          if (p.softcap > 0.0f) cap_scores(score, p.softcap, inv_cap);
#pragma unroll
        for (int st = 0; st < 4; ++st)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = i & 1, pos = base + 16 * (g >> 1) + 4 * st + 2 * (i >> 1) + (g & 1);
            float z = score[4 * st + i];
            if constexpr (EXTRA) z = fmaf(slope[n][j], (float)(pos - row_p[n][j]), z * kLog2e);
            if (edge && !(there && pos >= row_lo[n][j] && pos < row_hi[n][j])) z = -INFINITY;
            s[n][st][i] = z;
            top[j] = fmaxf(top[j], z);
          }
        float unit_w[2], to_l[2], shrink[2], sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          top[j] = max_from<4>(top[j]);
          const float m2 = fmaxf(m[n][j], top[j]), M2 = fmaxf(M[n][j], top[j] + ev);
          const float base_m = m2 == -INFINITY ? 0.0f : m2, base_M = M2 == -INFINITY ? 0.0f : M2;
          l[n][j] *= ex2(m[n][j] - base_m);
          shrink[j] = ex2(M[n][j] - base_M);
          // 2^unit: the unit of this page's weights.  Where the values are so small that no weight reaches f16, a
          // finer one, in which the sum of the weights loses nothing.
          unit_w[j] = top[j] == -INFINITY ? 0.0f : fminf(M2 - ev - kTopWeight, top[j] + 90.0f);
          to_l[j] = ex2(fminf(unit_w[j] - base_m, 126.0f));
          m[n][j] = m2;
          M[n][j] = M2;
        }
        if (__any_sync(0xFFFFFFFFu, shrink[0] != 1.0f || shrink[1] != 1.0f)) {
#pragma unroll
          for (int d = 0; d < D / 16; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][d][i] *= shrink[i & 1];
        }
#pragma unroll
        for (int st = 0; st < 4; ++st) {
          float w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            w[i] = ex2(s[n][st][i] - unit_w[i & 1]);
            sum[i & 1] += w[i];
          }
          pw[n][st][0] = turn8x8(pack_f16x2(w[0], w[1]));
          pw[n][st][1] = turn8x8(pack_f16x2(w[2], w[3]));
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) l[n][j] = fmaf(sum[j], to_l[j], l[n][j]);
      }

      uint32_t keep[4];
      if (edge) {
        // what no row sees is not looked at: those codes may be anything
#pragma unroll
        for (int st = 0; st < 4; ++st) keep[st] = byte_range(from - 16 * t - 4 * st, to - 16 * t - 4 * st);
        if (several) {
          // a NaN that only some rows see: those get it by their weight
          wait_slots(PH);
          uint32_t nan[4] = {0, 0, 0, 0};
#pragma unroll 1
          for (int d = 0; d < D / 8; ++d) {
            const uint32_t slot = PH == 1 || d < D / 16 ? r.slot : r.ahead(1, S).slot;
            const uint4 v0 = lds128(ring + slot * PIECE + (PH == 1 ? d : d % (D / 16)) * 512 + g * 64 + 16 * t);
            const uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w};
#pragma unroll
            for (int st = 0; st < 4; ++st)
              nan[st] |= ((w0[st] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u & keep[st];
          }
#pragma unroll
          for (int st = 0; st < 4; ++st) {
            nan[st] = or_g(nan[st]);
            keep[st] &= ~((nan[st] >> 7) * 0xFFu);
          }
          if (__any_sync(0xFFFFFFFFu, (nan[0] | nan[1] | nan[2] | nan[3]) != 0)) {
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
              for (int st = 0; st < 4; ++st)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  uint32_t w = pw[n][st][h];
                  if ((nan[st] >> (16 * h) & 0x80u) && (w & 0xFFFFu)) w |= 0x7E00u;
                  if ((nan[st] >> (16 * h) & 0x8000u) && (w >> 16)) w |= 0x7E000000u;
                  pw[n][st][h] = w;
                }
          }
        }
      }
      auto add_values = [&](auto masked) {
#pragma unroll
        for (int part = 0; part < PH; ++part) {
          wait_slots(1);
          const uint32_t at = ring + r.slot * PIECE + g * 64 + 16 * t;
#pragma unroll
          for (int d = part * (D / 16 / PH); d < (part + 1) * (D / 16 / PH); ++d) {
            const int off = (d - part * (D / 16 / PH)) * 1024;
            const uint4 v0 = lds128(at + off), v1 = lds128(at + off + 512);
            uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w}, w1[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
            for (int st = 0; st < 4; ++st) {
              if constexpr (decltype(masked)::value) {
                w0[st] &= keep[st];
                w1[st] &= keep[st];
              }
              uint32_t a[4];
              e4m3x4_f16x4(w0[st], a[0], a[2]);
              e4m3x4_f16x4(w1[st], a[1], a[3]);
#pragma unroll
              for (int n = 0; n < NB; ++n) mma_f16(o[n][d], a, pw[n][st][0], pw[n][st][1]);
            }
          }
          free_slots(1);
        }
      };
      if (edge)
        add_values(std::true_type{});
      else
        add_values(std::false_type{});
    }

    // ----------------------------------------------------- the segment's end
    // 2^(M - 15 - m) in two halves, as it may be below the normal floats where the values of the pages are least
    float half[NB][2];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
#pragma unroll
      for (int j = 0; j < 2; ++j) half[n][j] = m[n][j] == -INFINITY ? 0.0f : ex2(0.5f * (M[n][j] - kTopWeight - m[n][j]));
#pragma unroll
      for (int d = 0; d < D / 16; ++d)
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const float2 v = mul2(make_float2(o[n][d][i], o[n][d][i + 1]), make_float2(half[n][0], half[n][1]));
          o[n][d][i] = v.x, o[n][d][i + 1] = v.y;
        }
    }
    float* part = dealt.per_cta == 1 ? kv_part(p.ws, blockIdx.x, begins ? 1 : 0, R, D)
                                     : kv_worker_part(p.ws, me, begins ? 1 : 0, R, D);
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float sum = sum_from<4>(l[n][j]);
        // the sum of the weights is never 0 where a row sees a position; NaN stays
        const float inv = sum == 0.0f ? 0.0f : __fdividef(half[n][j], sum);
        const float log2s = sum == 0.0f ? -INFINITY : m[n][j] + log2f(sum);
        const int r = n * 8 + 2 * t + j;
        if (r >= it.rows) continue;
        if (begins && ends) {
          const int64_t row = kv_row(p, it.s0, it.r0, head, r);
          uint16_t* out = static_cast<uint16_t*>(p.out) + row * D + g;
#pragma unroll
          for (int d = 0; d < D / 16; ++d)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              out[16 * d + 8 * i] = (uint16_t)pack_bf16x2(o[n][d][2 * i + j] * inv, 0.0f);
          if (p.lse != nullptr && g == 0) p.lse[row] = log2s * kLn2;
        } else {
#pragma unroll
          for (int d = 0; d < D / 16; ++d)
#pragma unroll
            for (int i = 0; i < 2; ++i) part[r * D + 16 * d + 8 * i + g] = o[n][d][2 * i + j] * inv;
          if (g == 0) part[R * D + r] = log2s;
        }
      }
    if (lane == 0) {
      WorkerEnd& e = ends_of[warp];
      if (!begins) {
        e.within = 1;
        e.closes = ends;
        e.rows0 = it.rows;
      } else if (!ends) {
        e.opens = 1;
        e.s0 = it.s0;
        e.r0 = it.r0;
        e.rows = it.rows;
        e.head = head;
        e.end = dealt.start(me + 1) + (it.nblk - blk - cnt);
      }
    }
    at.advance(pl, p.c.heads, cnt);
  }

  // ------------------------------------------------- the join within the CTA
  const int n_workers = min(dealt.per_cta, dealt.workers - (int)blockIdx.x * dealt.per_cta);
  if (dealt.per_cta == 1) {
    if (warp == 0 && lane == 0) {
      const WorkerEnd& e = ends_of[0];
      desc[blockIdx.x] = desc_of(dealt, 1, e.opens ? e.end : 0, e.s0, e.r0, e.rows, e.head);
    }
    return;
  }
  __syncthreads();
  const int w0 = (int)blockIdx.x * dealt.per_cta;
  if (tid == 0) {
    Desc d{};
    const int64_t cta_end = dealt.start(w0 + n_workers);
    for (int w = 0; w < n_workers; ++w) {
      const WorkerEnd& e = ends_of[w];
      if (e.opens && e.end > cta_end) d = desc_of(dealt, dealt.per_cta, e.end, e.s0, e.r0, e.rows, e.head);
    }
    desc[blockIdx.x] = d;
  }
  // The one that the CTA begins within: its rows go to the warps.
  if (ends_of[0].within) {
    int n = 1;
    while (n < n_workers && !ends_of[n - 1].closes) ++n;
    for (int row = warp; row < ends_of[0].rows0; row += W) {
      const Joined<D> j = join_parts<D>(n, 0, 1, lane, row, R, [&](int i) -> const float* {
        return kv_worker_part(p.ws, w0 + i, 0, R, D);
      });
      store_part<D>(j, kv_part(p.ws, blockIdx.x, 0, R, D), row, R, lane);
    }
  }
  // A warp joins the one that it opened, with the first parts of the warps behind it.
  if (warp < n_workers && ends_of[warp].opens) {
    const WorkerEnd& e = ends_of[warp];
    int last = warp;
    bool closed = false;
    while (!closed && last + 1 < n_workers) closed = ends_of[++last].closes != 0;
    constexpr int RB = D <= 128 ? 8 : 4;
    for (int row0 = 0; row0 < e.rows; row0 += RB)
      join_rows<D, RB>(
          last - warp + 1, lane, row0, e.rows, R,
          [&](int i) -> const float* { return kv_worker_part(p.ws, me + i, i == 0 ? 1 : 0, R, D); },
          [&](int row, const Joined<D>& j) {
            if (closed)
              store_joined<D>(p, j, kv_row(p, e.s0, e.r0, e.head, row), lane);
            else
              store_part<D>(j, kv_part(p.ws, blockIdx.x, 1, R, D), row, R, lane);
          });
  }
}

// Joins the parts of a (row tile, head) that several CTAs share: the second part
// of the CTA that begins it and the first parts of those behind it, in that
// order; SP warps of a CTA share the parts of a row.
template <int D, int R, int SP>
__global__ void __launch_bounds__(256) rn_kv_join_kernel(const KvAttnParams p) {
  __shared__ float part_s[8][D + 2];
  pdl_launch_dependents();
  pdl_wait();
  const int cta = blockIdx.x;
  const Desc d = static_cast<const Desc*>(p.ws)[cta];
  if (d.parts == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp % SP;
  constexpr int kRows = 8 / SP;
  for (int r0 = blockIdx.y * kRows; r0 < d.rows; r0 += kRows * gridDim.y) {
    const int row = r0 + warp / SP;
    Joined<D> j{};
    if (row < d.rows)
      j = join_parts<D>(d.parts, sub, SP, lane, row, R,
                        [&](int i) -> const float* { return kv_part(p.ws, cta + i, i == 0 ? 1 : 0, R, D); });
    if constexpr (SP > 1) {
      store_part<D>(j, part_s[warp], 0, 1, lane);
      __syncthreads();
      if (sub == 0) {
        j = join_parts<D>(SP, 0, 1, lane, 0, 1, [&](int i) -> const float* { return part_s[warp + i]; });
      }
      __syncthreads();
    }
    if (sub == 0 && row < d.rows) store_joined<D>(p, j, kv_row(p, d.s0, d.r0, d.head, row), lane);
  }
}

template <int D, int NB, bool EXTRA>
rn_status launch_all(const KvAttnParams& p, int sms, cudaStream_t s) {
  constexpr int R = 8 * NB, W = kWarps;
  constexpr size_t smem = (size_t)W * kSlots<D> * kPiece<D>;
  auto k = rn_kv_attn_kernel<D, NB, EXTRA>;
  static std::atomic<int> kept[kMaxDevices];
  if (once_per_device(kept, [&] {
        return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) == cudaSuccess ? 1 : -1;
      }) < 1)
    return RN_ERR_CUDA;
  const int items = (int)((int64_t)p.q.tokens * p.group.d / R) + p.q.B;
  const int grid = sms < kKvMaxCtas ? sms : kKvMaxCtas;
  rn_status st = launch_pdl<KvAttnParams, int>(k, dim3(grid), 32 * W, smem, s, p, items);
  if (st != RN_OK) return st;
  return launch_kv_join(p, D, R, grid, s);
}

template <int D>
rn_status join_d(const KvAttnParams& p, int rows, int ctas, cudaStream_t s) {
  switch (rows) {
    case 8: return launch_pdl<KvAttnParams>(rn_kv_join_kernel<D, 8, 4>, dim3(ctas, 4), 256, 0, s, p);
    case 16: return launch_pdl<KvAttnParams>(rn_kv_join_kernel<D, 16, 4>, dim3(ctas, 8), 256, 0, s, p);
    case 128: return launch_pdl<KvAttnParams>(rn_kv_join_kernel<D, 128, 1>, dim3(ctas, 8), 256, 0, s, p);
    default: return launch_pdl<KvAttnParams>(rn_kv_join_kernel<D, 256, 1>, dim3(ctas, 16), 256, 0, s, p);
  }
}

template <int D>
rn_status launch_d(const KvAttnParams& p, int sms, cudaStream_t s) {
  const bool extra = p.softcap > 0.0f || p.slopes != nullptr;
  // By the mean rows of a sequence and head; no more is known on the host.  us, this kernel against the tiles: 16 rows,
  // 32 x 8192, dim 64 86 / 128, dim 128 72 / 89, dim 192 134 / 141, dim 256 174 / 174; 20 rows, dim 128 105 / 99;
  // 24 rows, dim 64 147 / 132, dim 128 188 / 168; 32 rows, dim 128 191 / 168.  Those are batches of one kind; where both
  // are mixed, one kind gets the other's kernel (60 x 1 on up to 16384 and a prompt of 512, groups of 8: 697, apart 206
  // and 36; 512 x 1 on 1000 and a prompt of 4096, groups of 1: 666, apart 182 and 79).
  const int64_t rows = (int64_t)p.q.tokens * p.group.d;  // of a head, all sequences
  if (rows > (int64_t)16 * p.q.B) return launch_kv_tile(p, D, sms, s);
  const bool one = rows <= (int64_t)8 * p.q.B;
  if (one) return extra ? launch_all<D, 1, true>(p, sms, s) : launch_all<D, 1, false>(p, sms, s);
  return extra ? launch_all<D, 2, true>(p, sms, s) : launch_all<D, 2, false>(p, sms, s);
}

}  // namespace

rn_status launch_kv_attn(const KvAttnParams& p, int dim, int sms, cudaStream_t s) {
  switch (dim) {
    case 64: return launch_d<64>(p, sms, s);
    case 128: return launch_d<128>(p, sms, s);
    case 192: return launch_d<192>(p, sms, s);
    default: return launch_d<256>(p, sms, s);
  }
}

rn_status launch_kv_join(const KvAttnParams& p, int dim, int rows, int ctas, cudaStream_t s) {
  switch (dim) {
    case 64: return join_d<64>(p, rows, ctas, s);
    case 128: return join_d<128>(p, rows, ctas, s);
    case 192: return join_d<192>(p, rows, ctas, s);
    default: return join_d<256>(p, rows, ctas, s);
  }
}

size_t kv_attn_bytes(int dim) {
  // few rows: up to 16, and partial results of every warp; many: tiles of 256 rows, or 128 where dim > 128
  const int64_t few = (kKvMaxCtas + kKvMaxWorkers) * part_floats(16, dim);
  const int64_t many = kKvMaxCtas * part_floats(dim > 128 ? 128 : 256, dim);
  return sizeof(Desc) * kKvMaxCtas + sizeof(float) * 2 * (size_t)(few > many ? few : many);
}

rn_status read_clear_error_kv(unsigned* code) {
  unsigned v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_kv, sizeof(v)) != cudaSuccess) return RN_ERR_CUDA;
  if (cudaMemcpyToSymbol(g_err_kv, &zero, sizeof(zero)) != cudaSuccess) return RN_ERR_CUDA;
  *code = v;
  return RN_OK;
}

}  // namespace rn
