// Attention of a sequence's newest tokens with its positions in the paged
// 8-bit cache, for few rows a key/value head (decoding, drafted tokens).
//
//   s_ij = scale q_i . k_j        (then c tanh(s / c), then + slope (j - p_i))
//   out_i = sum_j exp(s_ij - m_i) v_j / sum_j exp(s_ij - m_i)
//
// One pass over the pages with running maxima and sums.  A page's key scale
// 2^eK multiplies its scores; its value scale 2^eV goes into the weights:
// besides the maximum m of the scores a second one, M, of the scores plus eV
// (in base 2) scales the weights w = 2^(s + eV - M) <= 1 that multiply the
// value codes, so that no page's contribution is lost in 16 bits however far
// the pages' scales lie apart.  The sum of exp(s - m) is kept in fp32.
//
// The products are mma.sync m16n8k16 on f16 with the cache as the 16 rows and
// the queries as the 8 columns: S^T = K Q^T, O^T = V^T P^T.  Codes become f16
// by one conversion a pair, exactly; a query row becomes f16 times the power of
// two that puts its largest magnitude at 2^14 (what is 2^28 below it loses
// bits: 2^-39 of the row's largest); weights are rounded to f16, half a step of
// 2^-11, which the bf16 output's 2^-8 covers.  Sums are fp32.
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
// bytes each).  The (row tile, head, page) triples of the call, in this order,
// are dealt evenly to all workers, so ragged lengths cost nothing; a (row
// tile, head) that several workers share is joined from their partial results
// by a second kernel, in the workers' order.
#include <cuda_runtime.h>

#include "rn_device.cuh"
#include "rn_internal.h"
#include "rn_kv.cuh"
#include "rn_kv_plan.cuh"

namespace rn {
namespace {

__device__ unsigned g_err_kv;

// warps of a CTA and slots of a warp: 192 KB of slots an SM
template <int D>
constexpr int kWarps = D <= 128 ? 8 : 4;
template <int D>
constexpr int kSlots = 196608 / (kWarps<D> * 64 * D);

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

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// over the 8 lanes with the same t
__device__ __forceinline__ float max_g(float v) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}
__device__ __forceinline__ float sum_g(float v) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
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

template <int D, int NB, bool EXTRA>
__global__ void __launch_bounds__(32 * kWarps<D>, 1) rn_kv_attn_kernel(const KvAttnParams p, int items) {
  constexpr int R = 8 * NB, W = kWarps<D>, S = kSlots<D>, SLOT = 64 * D;
  extern __shared__ __align__(1024) unsigned char raw[];
  __shared__ __align__(8) uint64_t full_b[W][S];
  __shared__ Ranges<W, W> sh;
  const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  if (lane == 0) {
    for (int s = 0; s < S; ++s) mbar_init(smem_u32(&full_b[warp][s]), 1);
    fence_barrier_init();
  }
  pdl_launch_dependents();
  pdl_wait();

  Plan pl;
  const Dealt dealt = deal_pages<R, W, 32 * W>(p, items, sh, pl);
  const int me = (int)blockIdx.x * dealt.per_cta + warp;
  Desc* desc = static_cast<Desc*>(p.ws);
  if (warp >= dealt.per_cta || me >= dealt.workers) {  // no worker
    const int rest = W - dealt.per_cta;
    if (lane == 0)
      desc[warp < dealt.per_cta ? me : (int)gridDim.x * dealt.per_cta + (int)blockIdx.x * rest + warp - dealt.per_cta]
          .parts = 0;
    return;
  }
  const uint32_t ring = smem_u32(raw) + warp * (S * SLOT);
  auto bar = [&](int s) { return smem_u32(&full_b[warp][s]); };

  // ------------------------------------------------------------- copies
  // page numbers are read 32 at a time, one a lane
  Walk<R> ld = walk_of<R>(pl, dealt, sh, p.c.heads, me, warp);
  Walk<R> at = ld;
  int pages = -1, batch = 0;
  auto fetch = [&]() {
    batch = ld.blk;
    const int b = ld.blk + lane;
    pages = b < ld.it.nblk ? kv_page(p.q, p.c.pages, ld.it.b, ld.it.blk0 + b) : -1;
  };
  fetch();
  uint32_t slot_l = 0;
  int ld_page = -1;
  bool ld_v = false;
  // the scale bytes of the last two pages begun: lane 0 the keys', lane 1 the values'
  uint32_t sc_new = 0, sc_cur = 0;
  // begins the copy of the next page's keys, or values
  auto issue = [&]() {
    if (!ld_v) {
      if (ld.left == 0) return;
      if (ld.blk >= batch + 32) fetch();
      ld_page = __shfl_sync(0xFFFFFFFFu, pages, ld.blk - batch);
    }
    const int64_t ph = (int64_t)max(ld_page, 0) * p.c.heads + ld.head;
    if (lane == 0) {
      mbar_arrive_expect_tx(bar(slot_l), SLOT);
      bulk_g2s(ring + slot_l * SLOT, (ld_v ? p.c.v : p.c.k) + ph * SLOT, SLOT, bar(slot_l));
    }
    if (!ld_v) {
      // 256: no page
      sc_new = 256;
      if (ld_page >= 0 && lane < 2) sc_new = lane == 0 ? p.c.ks[ph] : p.c.vs[ph];
    } else {
      const int item = ld.item;
      if (ld.advance(pl, p.c.heads, 1) && (batch != 0 || ld.item != item)) fetch();
    }
    ld_v = !ld_v;
    if (++slot_l == S) slot_l = 0;
  };
  // two or more slots ahead; the scales of a page are read while the one before is worked on
#pragma unroll 1
  for (int i = 0; i < 2; ++i) issue();

  // ------------------------------------------------------------- the pages
  uint32_t slot_c = 0, phase = 0;
  int ahead = 2;   // slots begun and not yet worked on
  auto wait_slot = [&]() { mbar_wait(bar(slot_c), phase, &g_err_kv, kErrFullWait); };
  auto free_slot = [&]() {
    __syncwarp();
    if (++slot_c == S) {
      slot_c = 0;
      phase ^= 1;
    }
    --ahead;
  };
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
      const int r = it.r0 + n * 8 + g;
      const bool real = n * 8 + g < it.rows;
      uint4 raw4[D / 64][2];
      uint32_t big = 0;
      const unsigned char* src =
          static_cast<const unsigned char*>(p.x) +
          ((int64_t)(it.s0 + r / p.group) * p.stride + (int64_t)(head * p.group + r % p.group) * D + 16 * t) * 2;
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
        const int rr = it.r0 + min(n * 8 + 2 * t + j, it.rows - 1), i = rr / p.group;
        row_p[n][j] = it.p0 + i;
        row_hi[n][j] = p.causal ? row_p[n][j] + 1 : it.len;
        row_lo[n][j] = p.window > 0 ? row_p[n][j] - p.window + 1 : 0;
        if constexpr (EXTRA)
          slope[n][j] = p.slopes != nullptr ? __ldg(p.slopes + head * p.group + rr % p.group) * kLog2e : 0.0f;
      }
    }
    // every row sees [all_lo, all_hi)
    const int i0 = it.r0 / p.group, i1 = (it.r0 + it.rows - 1) / p.group;
    const int all_hi = p.causal ? it.p0 + i0 + 1 : it.len;
    const int all_lo = p.window > 0 ? it.p0 + i1 - p.window + 1 : 0;
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
      // keep the ring full: this page's slots, then the next pages'
      sc_cur = sc_new;
      const int base = (it.blk0 + blk + c) * 64;
      const uint32_t kbyte = __shfl_sync(0xFFFFFFFFu, sc_cur, 0), vbyte = __shfl_sync(0xFFFFFFFFu, sc_cur, 1);
      const bool there = kbyte < 256;
      if (ahead < S && (ld.left > 0 || ld_v)) {
        issue();
        ++ahead;
      }
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
      wait_slot();
      {
        const uint32_t at = ring + slot_c * SLOT + (16 * (g >> 1) + (g & 1)) * D + 16 * t;
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
      free_slot();
      if (ld.left > 0 || ld_v) {
        issue();
        ++ahead;
      }

      // scores in base 2, maxima, weights
      const float ek = pow2i(there ? kv_exp(kbyte) : 0), ev = there ? (float)kv_exp(vbyte) : 0.0f;
      uint32_t pw[NB][4][2];
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int st = 0; st < 4; ++st)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = i & 1, pos = base + 16 * (g >> 1) + 4 * st + 2 * (i >> 1) + (g & 1);
            float z = s[n][st][i] * (qs[n][j] * ek);
            if constexpr (EXTRA) {
              if (p.softcap > 0.0f) z = capped(z, p.softcap, 2.0f * kLog2e / p.softcap);
              z = fmaf(slope[n][j], (float)(pos - row_p[n][j]), z * kLog2e);
            }
            if (edge && !(there && pos >= row_lo[n][j] && pos < row_hi[n][j])) z = -INFINITY;
            s[n][st][i] = z;
            top[j] = fmaxf(top[j], z);
          }
        float add[2], base_m[2], shrink[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          top[j] = max_g(top[j]);
          const float m2 = fmaxf(m[n][j], top[j]), M2 = fmaxf(M[n][j], top[j] + ev);
          base_m[j] = m2 == -INFINITY ? 0.0f : m2;
          const float base_M = M2 == -INFINITY ? 0.0f : M2;
          l[n][j] *= ex2(m[n][j] - base_m[j]);
          shrink[j] = ex2(M[n][j] - base_M);
          add[j] = ex2(fminf(base_m[j] + ev - base_M, 126.0f));
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
            w[i] = ex2(s[n][st][i] - base_m[i & 1]);
            l[n][i & 1] += w[i];
            w[i] *= add[i & 1];
          }
          pw[n][st][0] = turn8x8(pack_f16x2(w[0], w[1]));
          pw[n][st][1] = turn8x8(pack_f16x2(w[2], w[3]));
        }
      }

      wait_slot();
      {
        const uint32_t at = ring + slot_c * SLOT + g * 64 + 16 * t;
        if (!edge) {
#pragma unroll
          for (int d = 0; d < D / 16; ++d) {
            const uint4 v0 = lds128(at + d * 1024), v1 = lds128(at + d * 1024 + 512);
            const uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w}, w1[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
            for (int st = 0; st < 4; ++st) {
              uint32_t a[4];
              e4m3x4_f16x4(w0[st], a[0], a[2]);
              e4m3x4_f16x4(w1[st], a[1], a[3]);
#pragma unroll
              for (int n = 0; n < NB; ++n) mma_f16(o[n][d], a, pw[n][st][0], pw[n][st][1]);
            }
          }
        } else {
          // what no row sees is not looked at: those codes may be anything
          uint32_t keep[4];
#pragma unroll
          for (int st = 0; st < 4; ++st)
            keep[st] = byte_range(from - 16 * t - 4 * st, to - 16 * t - 4 * st);
          if (several) {
            // a NaN that only some rows see: those get it by their weight
            uint32_t nan[4] = {0, 0, 0, 0};
#pragma unroll
            for (int d = 0; d < D / 8; ++d) {
              const uint4 v0 = lds128(at + d * 512);
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
#pragma unroll
          for (int d = 0; d < D / 16; ++d) {
            const uint4 v0 = lds128(at + d * 1024), v1 = lds128(at + d * 1024 + 512);
            const uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w}, w1[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
            for (int st = 0; st < 4; ++st) {
              uint32_t a[4];
              e4m3x4_f16x4(w0[st] & keep[st], a[0], a[2]);
              e4m3x4_f16x4(w1[st] & keep[st], a[1], a[3]);
#pragma unroll
              for (int n = 0; n < NB; ++n) mma_f16(o[n][d], a, pw[n][st][0], pw[n][st][1]);
            }
          }
        }
      }
      free_slot();
    }
    // ----------------------------------------------------- the segment's end
    float* part = kv_part(p.ws, me, begins ? 1 : 0, R, D);
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float sum = sum_g(l[n][j]);
        // the sum of the weights is never 0 where a row sees a position; NaN stays
        const float inv = sum == 0.0f ? 0.0f : ex2(M[n][j] - m[n][j]) / sum;
        const float log2s = sum == 0.0f ? -INFINITY : m[n][j] + log2f(sum);
        const int r = n * 8 + 2 * t + j;
        if (r >= it.rows) continue;
        if (begins && ends) {
          const int64_t row = (int64_t)(it.s0 + (it.r0 + r) / p.group) * (p.c.heads * p.group) + head * p.group +
                              (it.r0 + r) % p.group;
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
    if (at.left == cnt && lane == 0)
      desc[me] = desc_of(dealt, me, begins && !ends ? dealt.start(me + 1) + (it.nblk - blk - cnt) : 0, at.item, it.rows,
                         head);
    at.advance(pl, p.c.heads, cnt);
  }
}

// Joins the parts of a (row tile, head): worker w's second part and the first
// parts of the workers behind it, in that order.
template <int D, int R>
__global__ void __launch_bounds__(256) rn_kv_join_kernel(const KvAttnParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int w = blockIdx.x;
  const Desc d = static_cast<const Desc*>(p.ws)[w];
  if (d.parts == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto part = [&](int i) -> const float* { return kv_part(p.ws, w + i, i == 0 ? 1 : 0, R, D); };
  const Plan pl{p.q.starts, p.q.lens, p.q.B, p.q.tokens, p.group, p.causal, p.window, p.q.width * 64};
  const Item it = item_at<R>(pl, d.item);
  for (int r = blockIdx.y * 8 + warp; r < d.rows; r += 8 * gridDim.y) {
    float top = -INFINITY;
    for (int i = lane; i < d.parts; i += 32) top = fmaxf(top, part(i)[R * D + r]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if (top == -INFINITY) top = 0.0f;
    float sum = 0.0f;
    float acc[D / 32] = {};
#pragma unroll 4
    for (int i = 0; i < d.parts; ++i) {
      const float wgt = ex2(part(i)[R * D + r] - top);
      sum += wgt;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) acc[c] = fmaf(wgt, part(i)[r * D + c * 32 + lane], acc[c]);
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const int64_t row = (int64_t)(it.s0 + (it.r0 + r) / p.group) * (p.c.heads * p.group) + d.head * p.group +
                        (it.r0 + r) % p.group;
    uint16_t* out = static_cast<uint16_t*>(p.out) + row * D + lane;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) out[c * 32] = (uint16_t)pack_bf16x2(acc[c] * inv, 0.0f);
    if (p.lse != nullptr && lane == 0) p.lse[row] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
  }
}

template <int D, int NB, bool EXTRA>
rn_status launch_all(const KvAttnParams& p, int sms, cudaStream_t s) {
  constexpr int R = 8 * NB, W = kWarps<D>;
  constexpr size_t smem = (size_t)W * kSlots<D> * 64 * D;
  auto k = rn_kv_attn_kernel<D, NB, EXTRA>;
  static std::atomic<int> kept[kMaxDevices];
  if (once_per_device(kept, [&] {
        return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) == cudaSuccess ? 1 : -1;
      }) < 1)
    return RN_ERR_CUDA;
  const int items = (int)((int64_t)p.q.tokens * p.group / R) + p.q.B;
  const int grid = sms < kKvMaxCtas ? sms : kKvMaxCtas;
  rn_status st = launch_pdl<KvAttnParams, int>(k, dim3(grid), 32 * W, smem, s, p, items);
  if (st != RN_OK) return st;
  return launch_kv_join(p, D, R, grid * W, s);
}

template <int D>
rn_status join_d(const KvAttnParams& p, int rows, int workers, cudaStream_t s) {
  switch (rows) {
    case 8: return launch_pdl<KvAttnParams>(rn_kv_join_kernel<D, 8>, dim3(workers), 256, 0, s, p);
    case 16: return launch_pdl<KvAttnParams>(rn_kv_join_kernel<D, 16>, dim3(workers, 2), 256, 0, s, p);
    case 128: return launch_pdl<KvAttnParams>(rn_kv_join_kernel<D, 128>, dim3(workers, 8), 256, 0, s, p);
    default: return launch_pdl<KvAttnParams>(rn_kv_join_kernel<D, 256>, dim3(workers, 8), 256, 0, s, p);
  }
}

template <int D>
rn_status launch_d(const KvAttnParams& p, int sms, cudaStream_t s) {
  const bool extra = p.softcap > 0.0f || p.slopes != nullptr;
  const int64_t rows = (int64_t)p.q.tokens * p.group;  // of a head, all sequences
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

rn_status launch_kv_join(const KvAttnParams& p, int dim, int rows, int workers, cudaStream_t s) {
  switch (dim) {
    case 64: return join_d<64>(p, rows, workers, s);
    case 128: return join_d<128>(p, rows, workers, s);
    case 192: return join_d<192>(p, rows, workers, s);
    default: return join_d<256>(p, rows, workers, s);
  }
}

size_t kv_attn_bytes(int dim) {
  const int64_t few = kKvMaxWorkers * part_floats(16, dim), tile = kKvMaxCtas * part_floats(256, dim);
  return sizeof(Desc) * kKvMaxWorkers + sizeof(float) * 2 * (size_t)(few > tile ? few : tile);
}

rn_status read_clear_error_kv(unsigned* code) {
  unsigned v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_kv, sizeof(v)) != cudaSuccess) return RN_ERR_CUDA;
  if (cudaMemcpyToSymbol(g_err_kv, &zero, sizeof(zero)) != cudaSuccess) return RN_ERR_CUDA;
  *code = v;
  return RN_OK;
}

}  // namespace rn
