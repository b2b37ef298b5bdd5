// Products of one or a few tokens with a weight matrix: NVFP4 weights (E2M1
// codes, an E4M3 scale per 16 elements, a tensor scale), plain or as a gated
// feed-forward block, and the bf16 gated block for few tokens.
//
// The weights' bytes are the cost: each is read once, straight from global
// memory into the registers of the lane whose matrix fragment it is, and
// multiplied by mma.sync m16n8k16 with the weights as the 16 rows and the
// tokens as the 8 columns (few tokens leave most of a tcgen05 tile empty, and
// its operands would have to pass through shared memory, NVFP4 ones
// expanded fourfold).  Which k a lane's registers stand for is free as long as
// both operands agree, so a lane takes 32 contiguous bytes of a row (64 NVFP4
// codes, 16 bf16): four lanes read 128 contiguous bytes, an "item" is that of
// 32 rows (16 gate and 16 linear rows, or 32 rows of a plain product), and each
// warp keeps kDepth items in flight.  (With 16 bytes a lane the L1 looked up
// twice the lines: NVFP4 1 x 8192 x 65536, N x K x R, 70 against 60 us.)
//
// The tokens stand in shared memory in the order the fragments want them
// (16-byte conflict-free reads).  NVFP4 weights become f16 with one
// conversion and one product a pair: E2M1 value x E4M3 scale has at most 6
// significant bits and lies in [2^-10, 2688], so it is exact in f16.  The
// tokens, bf16, become f16 too, times the power of two that puts their
// largest magnitude at 2^14: exact unless the magnitudes span more than 2^31;
// a CTA that finds an element that is not exact keeps its tokens in bf16 and
// expands the weights to bf16 (exact as well), which is slower.  Sums
// are fp32.
//
// A CTA's W warps split the reduction kw ways and the rows W / kw ways; where
// rows are few, clusters of CTAs split it further (each holds its part of the
// tokens); where the tokens are too many for the shared memory, the CTA takes
// them slab after slab and keeps its steps' sums.  The parts meet in shared
// memory and are added in a fixed order.
//
// What bounds it: for one token the weights' read, 5.0 TB/s at 1 x 8192 x 65536
// (59-61 us for 302 MB; the same loads with nothing computed took 49 us, the
// computation alone 33 us) and 5.3 TB/s in bf16 (1 x 4096 x 8192 gated, 134 MB,
// 25.1 us); for 8 to 32 tokens the expansion's instructions at 8 to 16 warps an
// SM and the staging of the tokens in every CTA (8 x 8192 x 65536 71 us, 16
// 112 us, 32 x 4096 x 32768 78 us).
#include <cuda_runtime.h>

#include "rn_act_math.cuh"
#include "rn_device.cuh"
#include "rn_internal.h"
#include "rn_matvec_plan.h"
#include "rn_tc.cuh"

namespace rn {
namespace {

__device__ unsigned g_err_mv;

constexpr int kWBytes = 128;     // of a row's weights in a chunk
constexpr int kSBytes = 16;      // of its scales (NVFP4)

// items in flight per warp: two only with 32 tokens, where a CTA is 8 warps of
// up to 255 registers
template <int T>
constexpr int kDepth = T == 4 ? 2 : 1;

enum WeightKind : int { kWBf16 = 0, kWNvfp4 = 1 };

// how the weights' rows can be read: in whole chunks and on 32 bytes, in
// whole 32-byte pieces of a lane, in whole 16-byte halves of one, or any
enum RowKind : int { kRowsChunks = 0, kRowsPieces = 1, kRowsHalves = 2, kRowsAny = 3 };

// weights: read once, so 32-byte loads (a whole sector) leave L1 alone; of
// narrower ones several share a sector, which L1 keeps for them (13 x 5136 x
// 8200, 8-byte loads: 22.8 us, 27.6 without)
__device__ __forceinline__ void ldg_w32(const void* p, uint4 (&v)[2]) {
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0].x), "=r"(v[0].y), "=r"(v[0].z), "=r"(v[0].w), "=r"(v[1].x), "=r"(v[1].y),
                 "=r"(v[1].z), "=r"(v[1].w)
               : "l"(p));
}
__device__ __forceinline__ uint4 ldg_w16(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ldg_w8(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.L2::256B.v2.u32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "l"(p));
  return v;
}

__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// D += A B, m16n8k16, fp32 sums
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// the four pairs of E2M1 codes of a word -> f16x2 (even element low)
__device__ __forceinline__ void e2m1x8_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// two E4M3 codes -> f16x2 (exact)
__device__ __forceinline__ uint32_t e4m3x2_f16(uint32_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)c));
  return r;
}

__device__ __forceinline__ float2 f16x2_f32(uint32_t h) {
  float2 f;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// an item of a lane: 32 bytes of rows g and g + 8 of two 16-row tiles, and
// for NVFP4 the four scale codes of each
struct Item {
  uint4 w[2][2][2];
  uint32_t s[2][2];
  // 9 to 16 tokens, rows whose scales lie on any byte: the word behind, and by
  // how many bits the four codes stand off (a byte for each row)
  uint32_t s_next[2][2], off;
};

__device__ __forceinline__ void sts16(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

// what a lane reads next: its bytes of rows g and g + 8 of two 16-row tiles
struct Rows {
  const uint8_t* w[2][2];
  const uint8_t* s[2][2];
};

template <int WK, int T>
struct Mv {
  static constexpr int CK = WK == kWNvfp4 ? 256 : 64;  // reduction elements of a chunk
  static constexpr int J = CK / 32;                    // 16-byte pieces of a token a lane reads per chunk

  // chunk `chunk` of row tile `rt`: a plain product's 32 rows, or 16 gate and
  // 16 linear ones; rows past the end read the last row (their sums are
  // dropped)
  template <bool GATED>
  __device__ __forceinline__ static void rows(const MvParams& p, int rt, int chunk, int lane, Rows& r) {
    const int g = lane >> 2, t = lane & 3;
    const int64_t pitch = WK == kWNvfp4 ? p.K / 2 : p.K * 2ll;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = min((GATED ? rt * 16 : rt * 32 + m * 16) + g + 8 * h, p.H - 1);
        const int64_t row = at + (GATED ? (int64_t)m * p.H : 0);
        r.w[m][h] = static_cast<const uint8_t*>(p.w) + row * pitch + (int64_t)chunk * kWBytes + t * 32;
        if constexpr (WK == kWNvfp4) r.s[m][h] = p.blocks + row * (p.K / 16) + chunk * kSBytes + t * 4;
      }
  }

  // the item `d` chunks after r, which stands at chunk `chunk`
  __device__ __forceinline__ static void load(const MvParams& p, const Rows& r, int chunk, int d, int lane,
                                              Item& it) {
    const int left = p.K - (chunk + d) * CK - (lane & 3) * (CK / 4);  // of the row, from this lane's piece on
    if (p.rows == kRowsChunks) {
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          ldg_w32(r.w[m][h] + d * kWBytes, it.w[m][h]);
          if constexpr (WK == kWNvfp4)
            it.s[m][h] = __ldg(reinterpret_cast<const unsigned*>(r.s[m][h] + d * kSBytes));
        }
    } else if constexpr (WK == kWBf16) {
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int f = 0; f < 2; ++f)
            it.w[m][h][f] =
                left > f * 8 ? ldg_w16(r.w[m][h] + d * kWBytes + f * 16) : make_uint4(0, 0, 0, 0);
    } else if (p.rows == kRowsPieces) {
      // past the row's end its last pieces are read again: the tokens are 0 there
      const int at = d * CK + min(0, left - 64);
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          ldg_w32(r.w[m][h] + at / 2, it.w[m][h]);
          it.s[m][h] = __ldg(reinterpret_cast<const unsigned*>(r.s[m][h] + at / 16));
        }
    } else if (T == 2 && left >= 128) {
      // The piece, and four blocks behind it, are in the row: its codes from
      // fixed offsets, its scales as the two words around them, put together
      // when they are used (against put together here, where the warp has to
      // wait for them: 9 x 5136 x 8200 19.2 / 20.9 us, 13 tokens 20.7 / 22.4, 16
      // 23.6 / 25.2, 16 x 8208 x 65536 177 / 199, 9 x 1040 x 8200 7.7 / 7.9).  Not with
      // other numbers of tokens, whose registers are all in use: 1 x 8192 x 65536
      // 64.5 us instead of 61.1, 5 x 2080 x 5000 gated 13.7 instead of 12.4.
      it.off = 0;
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint8_t* w = r.w[m][h] + d * kWBytes;
          if (p.rows == kRowsHalves) {
            it.w[m][h][0] = ldg_w16(w);
            it.w[m][h][1] = ldg_w16(w + 16);
          } else {
#pragma unroll
            for (int f = 0; f < 2; ++f) {
              const uint2 a = ldg_w8(w + f * 16), b = ldg_w8(w + f * 16 + 8);
              it.w[m][h][f] = make_uint4(a.x, a.y, b.x, b.y);
            }
          }
          const uintptr_t sc = reinterpret_cast<uintptr_t>(r.s[m][h] + d * kSBytes);
          const unsigned* at = reinterpret_cast<const unsigned*>(sc & ~(uintptr_t)3);
          it.s[m][h] = __ldg(at);
          it.s_next[m][h] = __ldg(at + 1);
          it.off |= (uint32_t)(sc & 3) << (3 + 8 * (m * 2 + h));
        }
    } else {
      // at the row's end: block after block, past it the last one again
      const bool whole = p.rows == kRowsHalves;
      it.off = 0;
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint8_t* w = r.w[m][h] + d * kWBytes;
          const uint8_t* sc = r.s[m][h] + d * kSBytes;
          it.s[m][h] = 0;
          it.s_next[m][h] = 0;
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            const int o0 = min(f * 32, left - 16), o1 = min(f * 32 + 16, left - 16);  // of two blocks
            if (whole) {
              it.w[m][h][f] = ldg_w16(w + min(f * 32, left - 32) / 2);
            } else {
              const uint2 lo = ldg_w8(w + o0 / 2), hi = ldg_w8(w + o1 / 2);
              it.w[m][h][f] = make_uint4(lo.x, lo.y, hi.x, hi.y);
            }
            it.s[m][h] |= (__ldg(sc + o0 / 16) | (uint32_t)__ldg(sc + o1 / 16) << 8) << (16 * f);
          }
        }
    }
  }
  __device__ __forceinline__ static void advance(Rows& r) {
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        r.w[m][h] += kDepth<T> * kWBytes;
        if constexpr (WK == kWNvfp4) r.s[m][h] += kDepth<T> * kSBytes;
      }
  }

  // where this lane's fragments of each group of 8 tokens start in a chunk (in bytes); columns
  // without a token read the last token's: their sums are dropped
  __device__ __forceinline__ static void lane_at(int n, int lane, int (&at)[T]) {
#pragma unroll
    for (int t = 0; t < T; ++t) at[t] = (min(t * 8 + (lane >> 2), n - 1) * 4 + (lane & 3)) * 16;
  }

  // acc += item x tokens; shifted: the item's scales are in two words; xs: the
  // chunk's fragments (a shared-memory address: through a pointer the compiler
  // had lost the address space, 72 against 62 us at 1 x 8192 x 65536), at: this
  // lane's offsets in them
  template <bool WIDE>
  __device__ __forceinline__ static void compute(const Item& it, bool shifted, uint32_t xs, int n,
                                                 const int (&at)[T], float (&acc)[2][T][4]) {
    if constexpr (WK == kWBf16) {
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        uint4 b[T];
#pragma unroll
        for (int t = 0; t < T; ++t) b[t] = lds16(xs + f * frag_row(n) + at[t]);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const uint4 &u = it.w[m][0][f], &v = it.w[m][1][f];
          const uint32_t a0[4] = {u.x, v.x, u.y, v.y};
          const uint32_t a1[4] = {u.z, v.z, u.w, v.w};
#pragma unroll
          for (int t = 0; t < T; ++t) {
            mma16816<false>(acc[m][t], a0, b[t].x, b[t].y);
            mma16816<false>(acc[m][t], a1, b[t].z, b[t].w);
          }
        }
      }
    } else {
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        uint32_t s2[2][2];  // the scales of two blocks
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t s4 = shifted ? __funnelshift_r(it.s[m][h], it.s_next[m][h], it.off >> (8 * (m * 2 + h)))
                                        : it.s[m][h];
            s2[m][h] = e4m3x2_f16(f == 0 ? s4 : s4 >> 16);
          }
#pragma unroll
        for (int q = 0; q < 4; ++q) {  // 8 codes of each row
          uint4 b[T];
#pragma unroll
          for (int t = 0; t < T; ++t) b[t] = lds16(xs + (f * 4 + q) * frag_row(n) + at[t]);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            uint32_t v[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint4& wq = it.w[m][h][f];
              const uint32_t w = q == 0 ? wq.x : q == 1 ? wq.y : q == 2 ? wq.z : wq.w;
              const uint32_t s = __byte_perm(s2[m][h], 0u, q < 2 ? 0x1010 : 0x3232);
              e2m1x8_f16(w, v[h]);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                v[h][i] = mul_f16x2(v[h][i], s);
                if constexpr (WIDE) {
                  const float2 g = f16x2_f32(v[h][i]);
                  v[h][i] = pack_bf16x2(g.x, g.y);
                }
              }
            }
            const uint32_t a0[4] = {v[0][0], v[1][0], v[0][1], v[1][1]};
            const uint32_t a1[4] = {v[0][2], v[1][2], v[0][3], v[1][3]};
#pragma unroll
            for (int t = 0; t < T; ++t) {
              mma16816<!WIDE>(acc[m][t], a0, b[t].x, b[t].y);
              mma16816<!WIDE>(acc[m][t], a1, b[t].z, b[t].w);
            }
          }
        }
      }
    }
  }
};

// y of one output column and token: stored as p.mode asks (kFfnMx: the warp
// holds the 32 columns of a block)
template <int ACT>
__device__ __forceinline__ void finish(const MvParams& p, int n, int col, float a, float b, float* amax) {
  const bool ok = col < p.H;
  float y = a;
  if constexpr (ACT != kActNone) {
    y = act_value<ACT>(a, b, p.limit, p.alpha) * (p.scales ? __ldg(p.scales + n) : 1.0f);
    if (p.pre != nullptr && ok) {
      uint16_t* pre = static_cast<uint16_t*>(p.pre) + (int64_t)n * 2 * p.H;
      const uint32_t v = pack_bf16x2(a, b);
      pre[col] = (uint16_t)v;
      pre[(int64_t)p.H + col] = (uint16_t)(v >> 16);
    }
  }
  const int64_t o = (int64_t)n * p.H + col;
  if (p.mode == kFfnMx) {
    const uint32_t code = e8m0_code(warp_max_nan(fabsf(y)));
    if (ok) {
      static_cast<uint8_t*>(p.out)[o] = (uint8_t)pack_e4m3x2(y * e8m0_inv_scale(code), 0.0f);
      if ((col & 31) == 0) p.row_scales[(int64_t)n * (p.H / 32) + col / 32] = (uint8_t)code;
    }
  } else if (ok) {
    if (p.mode == kFfnBf16) {
      static_cast<uint16_t*>(p.out)[o] = (uint16_t)pack_bf16x2(y, 0.0f);
    } else if (p.mode == kFfnF32) {
      static_cast<float*>(p.out)[o] = y;
    } else {
      *amax = amax_acc(*amax, y);
      static_cast<uint8_t*>(p.out)[o] = (uint8_t)pack_e4m3x2(y * __ldg(p.scale), 0.0f);
    }
  }
}

// Copies the tokens' elements of chunks lo .. hi - 1 into shared memory in
// fragment order (zeros past the row's end); returns the largest magnitude
// this thread saw, as bf16 bits (NVFP4).  A thread keeps to one 16-byte place of
// the row and walks over the tokens, kBatch loads at a time (1 x 8192 x 65536:
// 60.8 us with 2, 65.0 with 8; 32 x 4096 x 32768: 84.0 with 2, 77.6 with 8).
template <int WK, int T, int W>
__device__ __forceinline__ uint32_t copy_tokens(const MvParams& p, int lo, int hi, int n0, int n, uint32_t xs) {
  using M = Mv<WK, T>;
  constexpr int CP = M::CK / 8;  // pieces of a token in a chunk
  constexpr int kBatch = T == 1 ? 2 : 8;
  const int pieces = (hi - lo) * CP;  // per token, 8 elements each
  for (int i = threadIdx.x; i < (hi - lo) * M::J; i += 32 * W)  // the 16 bytes behind each fragment
    sts16(xs + i * frag_row(n) + n * 64, make_uint4(0, 0, 0, 0));
  uint32_t m = 0;
  // rows shorter than the threads: groups of threads share the tokens
  const int groups = pieces > 0 ? max(1, 32 * W / pieces) : 1;
  const int group = pieces >= 32 * W ? 0 : (int)threadIdx.x / max(1, pieces);
  if (group < groups) {
#pragma unroll 1
    for (int q = (int)threadIdx.x - group * pieces; q < pieces; q += 32 * W) {
      const uint32_t to = xs + (q / CP * M::J + q % M::J) * frag_row(n) + q % CP / M::J * 16;
      const uint16_t* x = static_cast<const uint16_t*>(p.x) + (int64_t)n0 * p.K + (int64_t)lo * M::CK + q * 8;
      const bool in = lo * M::CK + q * 8 < p.K;
#pragma unroll 1
      for (int tok = group; tok < n; tok += kBatch * groups) {
        uint4 v[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          v[u] = make_uint4(0, 0, 0, 0);
          if (in && tok + u * groups < n)
            v[u] = __ldg(reinterpret_cast<const uint4*>(x + (int64_t)(tok + u * groups) * p.K));
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          if (tok + u * groups < n) sts16(to + (tok + u * groups) * 64, v[u]);
          if constexpr (WK == kWNvfp4) {
            const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) m = max(m, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
          }
        }
      }
    }
  }
  return m;
}

// The tokens of a slab; returns what the sums are to be multiplied with.
// *wide: whether they had to stay bf16 (NVFP4).
template <int WK, int T, int W>
__device__ __forceinline__ float stage_tokens(const MvParams& p, int lo, int hi, int n0, int n, uint32_t xs,
                                              bool* wide) {
  uint32_t m = copy_tokens<WK, T, W>(p, lo, hi, n0, n, xs);
  if constexpr (WK == kWBf16) {
    __syncthreads();
    return 1.0f;
  } else {
    __shared__ uint32_t warp_max[W];
    const int count = (hi - lo) * Mv<WK, T>::J * (frag_row(n) / 16);  // 16-byte pieces
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < W; ++w) m = max(m, warp_max[w]);
    // 2^c puts it into [2^14, 2^15); c within what fp32 holds
    const int c = m == 0u ? 0 : min(126, max(-126, 14 - ((int)(m >> 7) - 127)));
    const float up = __uint_as_float((uint32_t)(c + 127) << 23);
    const float down = __uint_as_float((uint32_t)(127 - c) << 23);
    bool inexact = false;
#pragma unroll 1
    for (int i = threadIdx.x; i < count; i += 32 * W) {
      const uint4 v = lds16(xs + i * 16);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = bf16x2_f32(w[j]);
        h[j] = pack_f16x2(f.x * up, f.y * up);
        const float2 r = f16x2_f32(h[j]);
        inexact |= !(r.x * down == f.x && r.y * down == f.y);
      }
      sts16(xs + i * 16, make_uint4(h[0], h[1], h[2], h[3]));
    }
    *wide = __syncthreads_or(inexact);
    if (!*wide) return down;
    copy_tokens<WK, T, W>(p, lo, hi, n0, n, xs);
    __syncthreads();
    return 1.0f;
  }
}

// one step's sums over this warp's chunks c_lo .. c_hi - 1 of the slab that
// starts at chunk `lo`; x: the tokens of chunk c_lo.  The first items are
// under way (r stands at c_lo), and the first ones of tile next_tile (chunks
// n_lo .. n_hi - 1) are sent on theirs.
template <bool GATED, int WK, int T, bool WIDE>
__device__ __forceinline__ void step_sums(const MvParams& p, int next_tile, int lane, int n, uint32_t x,
                                          int c_lo, int c_hi, int n_lo, int n_hi,
                                          const int (&at)[T], Rows& r, Item (&it)[kDepth<T>],
                                          float (&acc)[2][T][4]) {
  using M = Mv<WK, T>;
  const int stride = M::J * frag_row(n);
  int c = c_lo;
  do {
    // a slot's next item: of this step, or the first ones of the next
    const bool last = c + kDepth<T> >= c_hi;
    if (last)
      M::template rows<GATED>(p, next_tile, n_lo, lane, r);
    else
      M::advance(r);
    const int from = last ? n_lo : c + kDepth<T>, to = last ? n_hi : c_hi;
#pragma unroll
    for (int d = 0; d < kDepth<T>; ++d) {
      if (c + d < c_hi)
        M::template compute<WIDE>(it[d], T == 2 && p.rows >= kRowsHalves, x + d * stride, n, at, acc);
      if (from + d < to) M::load(p, r, from, d, lane, it[d]);
    }
    c += kDepth<T>;
    x += kDepth<T> * stride;
  } while (c < c_hi);
}

// W warps a CTA; 8 warps and few tokens: two CTAs an SM.  CS: a cluster whose
// CTAs take their tokens slab after slab (compiled apart: in one kernel the
// others lost 1 to 3 %, 32 x 4096 x 32768 81.4 us instead of 78.7)
template <int ACT, int WK, int T, int W, bool CS>
__global__ void __launch_bounds__(32 * W, (T == 1 && W == 8) ? 2 : 1) rn_matvec_kernel(const MvParams p, const MvPlan pl) {
  using M = Mv<WK, T>;
  constexpr bool GATED = ACT != kActNone;
  extern __shared__ uint4 smem[];
  __shared__ __align__(8) uint64_t ready_b[2], free_b[2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = pl.split > 1 ? (int)cluster_rank() : 0;
  const int group = (int)blockIdx.x / pl.split, n_groups = (int)gridDim.x / pl.split;
  const int n0 = (int)blockIdx.y * 8 * T;
  const int n = min(8 * T, p.N - n0);
  const int rw = W / pl.kw, wr = warp / pl.kw, wk = warp % pl.kw;
  const int cols = rw * (GATED ? 16 : 32);  // outputs of a step
  // the tokens; the warps' sums of two steps
  // [2][warps][n][kPartStride]; in a cluster its CTAs' sums [split][rw][n][32]; with several slabs the steps'
  // sums of this CTA [batch][rw][n][32]
  const int kPart = W * n * kPartStride;  // floats of the warps' sums of a step
  uint4* xs = smem;
  float* part = reinterpret_cast<float*>(xs + pl.slab * M::J * (frag_row(n) / 16));
  float* parts = part + 2 * kPart;
  const int lo = rank * pl.part, hi = max(lo, min(lo + pl.part, pl.chunks));
  // (the same in every CTA of a cluster)
  const int slabs = CS ? (pl.part + pl.slab - 1) / pl.slab : max(1, (hi - lo + pl.slab - 1) / pl.slab);
  const int my_steps = (pl.steps - group + n_groups - 1) / n_groups;
  const int vals = rw * n * 32;
  // this warp's chunks of slab i: contiguous
  const auto chunk_at = [&](int i, int w) {
    const int a = min(lo + i * pl.slab, hi), b = min(a + pl.slab, hi);
    return a + (b - a) * w / pl.kw;
  };
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&ready_b[i]), W);
      mbar_init(smem_u32(&free_b[i]), W);
    }
    fence_barrier_init();
  }
  // every CTA of the cluster has to have started before the first sums go to
  // another one's shared memory; waited for behind the staging
  if (pl.split > 1) cluster_arrive();
  // nothing of the caller's memory is touched until the kernel before has completed
  pdl_launch_dependents();
  pdl_wait();
  int at[T];
  M::lane_at(n, lane, at);
  const float si = WK == kWNvfp4 ? __ldg(p.scale_inv) : 1.0f;
  float amax = 0.0f, inv = 1.0f;

  // The warps' sums of a step are added one step later, while the next
  // step's weights are on their way: the warps of a CTA meet on two
  // barriers a buffer (written, read) and may be a step apart.
  uint32_t used = 0;              // steps whose sums were written
  int held = -1, held_slab = 0;   // the one that waits to be added
  const auto add_up = [&]() {
    const uint32_t u = used - 1, buf = u & 1;
    mbar_wait(smem_u32(&ready_b[buf]), (u >> 1) & 1, &g_err_mv, kErrReadyWait);
    const float* from = part + buf * kPart;
    // one row's sum over the CTA's warps, times what the tokens were scaled by
    const auto cta_sum = [&](int tile, int tok, int row) {
      const float* q = from + (tile * pl.kw * n + tok) * kPartStride + row;
      float v = q[0];
      for (int w = 1; w < pl.kw; ++w) v += q[w * n * kPartStride];
      return v * inv;
    };
    const int step = group + held * n_groups;
    if (pl.split == 1) {
      // with several slabs each thread keeps its outputs' sums
      float* sums = parts + (size_t)(held % pl.batch) * vals;
      for (int i = threadIdx.x; i < cols * n; i += 32 * W) {
        const int tok = i / cols, col = i % cols;
        float a, b = 0.0f;
        if constexpr (GATED) {
          a = cta_sum(col / 16, tok, col % 16);
          b = cta_sum(col / 16, tok, 16 + col % 16);
        } else {
          a = cta_sum(col / 32, tok, col % 32);
        }
        if (slabs > 1) {
          if (held_slab > 0) {
            a += sums[i];
            if constexpr (GATED) b += sums[vals / 2 + i];
          }
          sums[i] = a;
          if constexpr (GATED) sums[vals / 2 + i] = b;
        }
        if (held_slab + 1 == slabs) finish<ACT>(p, n0 + tok, step * cols + col, a * si, b * si, &amax);
      }
    } else {
      // the steps' sums meet in the cluster's CTAs in turn
      const int leader = held % pl.split;
      const uint32_t to = map_to_rank(smem_u32(parts + rank * vals), leader);
      const bool whole = !CS || held_slab + 1 == slabs;
      if constexpr (CS) {
        // this CTA's sums of the slabs so far; the last slab's go out with them
        float* sums = parts + (size_t)(pl.split + held % pl.batch) * vals;
        for (int i = threadIdx.x; i < vals; i += 32 * W) {
          float v = cta_sum(i / (n * 32), i / 32 % n, i & 31);
          if (held_slab > 0) v += sums[i];
          sums[i] = v;
          if (whole) asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + i * 4), "f"(v) : "memory");
        }
      } else {
        for (int i = threadIdx.x; i < vals; i += 32 * W)
          asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + i * 4),
                       "f"(cta_sum(i / (n * 32), i / 32 % n, i & 31))
                       : "memory");
      }
      if (whole) cluster_sync();
      if (whole && rank == leader) {
        const auto sum = [&](int tile, int tok, int row) {
          const float* q = parts + (tile * n + tok) * 32 + row;
          float v = q[0];
          for (int s = 1; s < pl.split; ++s) v += q[s * vals];
          return v * si;
        };
        for (int i = threadIdx.x; i < cols * n; i += 32 * W) {
          const int tok = i / cols, col = i % cols;
          if constexpr (GATED)
            finish<ACT>(p, n0 + tok, step * cols + col, sum(col / 16, tok, col % 16),
                        sum(col / 16, tok, 16 + col % 16), &amax);
          else
            finish<ACT>(p, n0 + tok, step * cols + col, sum(col / 32, tok, col % 32), 0.0f, &amax);
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&free_b[buf]));
    held = -1;
  };

  Item it[kDepth<T>];
  Rows r;
  {
    const int c_lo = chunk_at(0, wk), c_hi = chunk_at(0, wk + 1);
    M::template rows<GATED>(p, group * rw + wr, c_lo, lane, r);
#pragma unroll
    for (int d = 0; d < kDepth<T>; ++d)
      if (c_lo + d < c_hi) M::load(p, r, c_lo, d, lane, it[d]);
  }
  bool wide = false;
  for (int b0 = 0; b0 < my_steps; b0 += pl.batch) {
    const int b1 = min(b0 + pl.batch, my_steps);
    for (int sl = 0; sl < slabs; ++sl) {
      if (slabs > 1 || b0 == 0) {
        if (held >= 0) add_up();  // it needs the scales of the slab before
        __syncthreads();
        const int s_lo = lo + sl * pl.slab;
        inv = stage_tokens<WK, T, W>(p, s_lo, max(s_lo, min(s_lo + pl.slab, hi)), n0, n, smem_u32(xs), &wide);
        if (pl.split > 1 && b0 == 0 && sl == 0) cluster_wait();
      }
      const int c_lo = chunk_at(sl, wk), c_hi = chunk_at(sl, wk + 1);
      const uint32_t x = smem_u32(xs) + (c_lo - lo - sl * pl.slab) * (M::J * frag_row(n));
      for (int j = b0; j < b1; ++j) {
        // what follows: the batch's next step, its first with the next slab, the next batch's first
        const bool wrap = j + 1 == b1;
        const int sl2 = wrap ? (sl + 1) % slabs : sl;
        const int j2 = wrap ? (sl + 1 < slabs ? b0 : b1) : j + 1;
        const int n_lo = chunk_at(sl2, wk), n_hi = j2 < my_steps ? chunk_at(sl2, wk + 1) : n_lo;
        const int next = (group + min(j2, my_steps - 1) * n_groups) * rw + wr;
        float acc[2][T][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int t = 0; t < T; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][t][i] = 0.0f;
        if (c_lo >= c_hi) {  // nothing of this slab for this warp
          M::template rows<GATED>(p, next, n_lo, lane, r);
#pragma unroll
          for (int d = 0; d < kDepth<T>; ++d)
            if (n_lo + d < n_hi) M::load(p, r, n_lo, d, lane, it[d]);
        } else if (WK == kWNvfp4 && wide) {
          step_sums<GATED, WK, T, true>(p, next, lane, n, x, c_lo, c_hi, n_lo, n_hi, at, r, it, acc);
        } else {
          step_sums<GATED, WK, T, false>(p, next, lane, n, x, c_lo, c_hi, n_lo, n_hi, at, r, it, acc);
        }
        // this warp's sums: [n][32 rows]
        const uint32_t buf = used & 1;
        mbar_wait(smem_u32(&free_b[buf]), ((used >> 1) & 1) ^ 1, &g_err_mv, kErrEmptyWait);
        float* mine = part + buf * kPart + warp * n * kPartStride;
        const int g = lane >> 2, t2 = (lane & 3) * 2;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int t = 0; t < T; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int tok = t * 8 + t2 + (i & 1);
              if (tok < n) mine[tok * kPartStride + m * 16 + g + (i >> 1) * 8] = acc[m][t][i];
            }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ready_b[buf]));
        if (held >= 0) add_up();
        ++used;
        held = j;
        held_slab = sl;
      }
    }
  }
  if (held >= 0) add_up();
  if (p.mode == kFfnFp8) {
    const float m = warp_max_nan(amax);
    if (lane == 0) atomicMax(reinterpret_cast<unsigned*>(p.amax), abs_bits(m));
  }
  if (pl.split > 1) cluster_sync();  // no CTA leaves while another writes to it
}

template <int ACT, int WK, int T, int W, bool CS>
rn_status launch_plan(const MvParams& p, const MvLaunch& l, cudaStream_t s) {
  auto k = rn_matvec_kernel<ACT, WK, T, W, CS>;
  const MvPlan& pl = l.plan;
  static std::atomic<int> kept[kMaxDevices];
  if (once_per_device(kept, [&] {
        return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMvSmem) == cudaSuccess
                   ? 1
                   : -1;
      }) < 1)
    return RN_ERR_CUDA;
  static_assert(kMvMaxN / 32 <= 65535, "groups of tokens are gridDim.y");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(l.groups * pl.split), (unsigned)l.ny);
  cfg.blockDim = dim3(32 * W);
  cfg.dynamicSmemBytes = l.smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  int na = 0;
  if (pl.split > 1) {
    attr[na].id = cudaLaunchAttributeClusterDimension;
    attr[na].val.clusterDim.x = (unsigned)pl.split;
    attr[na].val.clusterDim.y = 1;
    attr[na].val.clusterDim.z = 1;
    ++na;
  }
  attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[na].val.programmaticStreamSerializationAllowed = 1;
  ++na;
  cfg.attrs = attr;
  cfg.numAttrs = na;
  if (cudaLaunchKernelEx(&cfg, k, p, pl) != cudaSuccess) return RN_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? RN_OK : RN_ERR_CUDA;
}

template <int ACT, int WK, int T, int W>
rn_status launch_t(const MvParams& p, int sms, cudaStream_t s) {
  MvLaunch l{};
  if (!mv_plan({p.N, p.K, p.H, WK == kWNvfp4, ACT != kActNone, p.mode == kFfnMx, T, W}, sms, &l))
    return RN_ERR_UNSUPPORTED;
  if constexpr (T > 1)
    if (l.plan.split > 1 && l.plan.slab < l.plan.part) return launch_plan<ACT, WK, T, W, true>(p, l, s);
  return launch_plan<ACT, WK, T, W, false>(p, l, s);
}

template <int ACT, int WK>
rn_status launch_n(const MvParams& p, int sms, cudaStream_t s) {
  const MvVariant v = mv_variant(p.N, p.K);
  if (v.T == 1) return v.W == 8 ? launch_t<ACT, WK, 1, 8>(p, sms, s) : launch_t<ACT, WK, 1, 16>(p, sms, s);
  return v.T == 2 ? launch_t<ACT, WK, 2, 12>(p, sms, s) : launch_t<ACT, WK, 4, 8>(p, sms, s);
}

}  // namespace

rn_status launch_nvfp4_mv(int act, const MvParams& q, int sms, cudaStream_t s) {
  MvParams p = q;
  const bool on32 = reinterpret_cast<uintptr_t>(p.w) % 32 == 0;
  p.rows = on32 && p.K % 256 == 0  ? kRowsChunks
           : on32 && p.K % 64 == 0 ? kRowsPieces
           : p.K % 32 == 0         ? kRowsHalves
                                   : kRowsAny;
  switch (act) {
    case kActNone: return launch_n<kActNone, kWNvfp4>(p, sms, s);
    case kActSwiglu: return launch_n<kActSwiglu, kWNvfp4>(p, sms, s);
    default: return launch_n<kActClampedSwiglu, kWNvfp4>(p, sms, s);
  }
}

rn_status launch_bf16_mv(int act, const MvParams& q, int sms, cudaStream_t s) {
  MvParams p = q;
  p.rows = p.K % 64 == 0 && reinterpret_cast<uintptr_t>(p.w) % 32 == 0 ? kRowsChunks : kRowsAny;
  return act == kActSwiglu ? launch_n<kActSwiglu, kWBf16>(p, sms, s)
                           : launch_n<kActClampedSwiglu, kWBf16>(p, sms, s);
}

rn_status read_clear_error_mv(unsigned* code) {
  unsigned v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_mv, sizeof(v)) != cudaSuccess) return RN_ERR_CUDA;
  if (cudaMemcpyToSymbol(g_err_mv, &zero, sizeof(zero)) != cudaSuccess) return RN_ERR_CUDA;
  *code = v;
  return RN_OK;
}

}  // namespace rn
