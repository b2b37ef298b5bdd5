// How the attention over the paged cache deals its work: row tiles of the
// sequences, their pages, the workers' ranges, and where partial results lie.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "rn_internal.h"
#include "rn_kv.cuh"

namespace rn {

constexpr int kKvMaxCtas = 160;
constexpr int kKvMaxWorkers = kKvMaxCtas * 8;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// sequences whose rows and lengths are kept in shared memory
constexpr int kSeqsInSmem = 1024;

// the (row tile, head) that a CTA begins and does not finish
struct Desc {
  int parts;       // CTAs that share it, this one the first (0: none)
  int s0, r0, rows, head;
  int unused[3];
};

// a row tile of a sequence
struct Item {
  int b;
  int s0;          // first row of the sequence
  int r0, rows;    // its rows of (query, query head of the group), query-major
  int p0;          // position of query 0
  int len;
  int lo, hi;      // positions that any row sees
  int blk0, nblk;  // pages; one without positions where the rows see none
};

struct Plan {
  const int* starts;  // shared or global
  const int* lens;
  const int* bases;   // shared: item_base of every sequence, or NULL
  int B, tokens;
  FastDiv group;
  int causal, window;
  int reach;          // positions that the page table has room for
};

// the first position that a query at p sees
__device__ __forceinline__ int first_seen(int p, int window) { return window > 0 && p >= window ? p - window + 1 : 0; }

template <int R>
__device__ __forceinline__ int item_base(const Plan& a, int b) {
  return (int)((int64_t)min(max(a.starts[b], 0), a.tokens) * a.group.d / R) + b;
}

// item i of the call; nblk = 0 where it has no rows.  The sequence with r rows
// (times the group) has ceil(r / R) items, at most one more than base(b + 1) -
// base(b) - 1 counts.
template <int R>
__device__ __forceinline__ Item item_at(const Plan& a, int i) {
  int lo = 0, hi = a.B;  // the last b with base(b) <= i
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if ((a.bases != nullptr ? a.bases[mid] : item_base<R>(a, mid)) <= i) lo = mid;
    else hi = mid;
  }
  Item t;
  t.b = lo;
  const KvRows r = kv_rows(a.starts, lo, a.tokens);
  const int n = r.s1 - r.s0;
  const int64_t all = (int64_t)n * a.group.d, first = (int64_t)(i - item_base<R>(a, lo)) * R;
  t.s0 = r.s0;
  t.nblk = 0;
  t.rows = 0;
  if (first < 0 || first >= all) return t;
  t.r0 = (int)first;
  t.rows = (int)min((int64_t)R, all - first);
  t.len = max(a.lens[lo], 0);
  t.p0 = t.len - n;
  const int i0 = quot(t.r0, a.group), i1 = quot(t.r0 + t.rows - 1, a.group);
  t.hi = min(a.causal ? max(t.p0 + i1 + 1, 0) : t.len, a.reach);
  t.lo = first_seen(t.p0 + i0, a.window);
  t.blk0 = t.lo >> 6;
  t.nblk = t.hi > t.lo ? ((t.hi - 1) >> 6) - t.blk0 + 1 : 1;
  return t;
}

// A range of (row tile, head, page) triples, in this order, from its first on.
// Beginning a (row tile, head) costs as much as EXTRA pages (its queries, its
// output), so it is dealt with as many more; a range that would end or begin
// within those ends or begins in front of them.
template <int R, int EXTRA>
struct Walk {
  Item it;
  int item, head, blk;  // the next page
  int64_t left;         // pages, and extra ones, until the range's end

  // pages of the (row tile, head) that the range still has
  __device__ __forceinline__ int segment() const {
    return (int)min(left - (blk == 0 ? EXTRA : 0), (int64_t)(it.nblk - blk));
  }

  // n pages further, within a segment; true where that goes on to another (row tile, head)
  __device__ __forceinline__ bool advance(const Plan& a, int heads, int n) {
    left -= n + (blk == 0 ? EXTRA : 0);
    blk += n;
    if (blk < it.nblk) return false;
    if (left <= EXTRA) {
      left = 0;
      return false;
    }
    blk = 0;
    if (++head == heads) {
      head = 0;
      do {
        it = item_at<R>(a, ++item);
      } while (it.nblk == 0);  // pages are left, so an item with some follows
    }
    return true;
  }

  // whether the segment of cnt pages is the range's last
  __device__ __forceinline__ bool is_last(int cnt) const {
    const int64_t then = left - cnt - (blk == 0 ? EXTRA : 0);
    return blk + cnt < it.nblk || then <= EXTRA;
  }
};

// what the workers of a CTA find out about their ranges
template <int W, int WARPS>
struct Ranges {
  int64_t sums[WARPS];
  int64_t from[W];   // the first page of the worker's (row tile, ...), before it is dealt to heads
  int64_t base[W];   // where its item's pages begin
  int item[W];
  int seqs[3 * kSeqsInSmem + 1];
};

// `more` workers have one page more than the others.  They are spread over all (and so over the SMs: where the first
// ones had it, 8 SMs had 24 pages, the others 16, and 9 sequences of dim 256 took 34.4 us; now 31.9).
struct Dealt {
  int64_t total;     // pages of the call with the extra ones, times heads
  int64_t each;
  uint32_t step;     // 2^20 more / workers, a little more than that: workers step / 2^20 < more + 0.01
  int per_cta;       // workers of a CTA; all of them are `workers`
  int workers;
  __device__ __forceinline__ int64_t start(int w) const {
    return each * w + ((uint32_t)w * step >> 20);  // (w <= workers <= 1280, step <= 2^20)
  }
};

// Called by all NT threads: the call's plan, and the items that the CTA's
// workers begin in (up to W of them; fewer where pages are few, so that every
// SM has some, and a worker has one page at least).
template <int R, int EXTRA, int W, int NT>
__device__ __forceinline__ Dealt deal_pages(const KvAttnParams& p, int items, Ranges<W, NT / 32>& sh, Plan& pl) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pl = Plan{p.q.starts, p.q.lens, nullptr, p.q.B, p.q.tokens, p.group, p.causal, p.window, p.q.width * 64};
  if (p.q.B <= kSeqsInSmem) {
    int *starts = sh.seqs, *lens = starts + kSeqsInSmem + 1, *bases = lens + kSeqsInSmem;
    for (int i = tid; i <= p.q.B; i += NT) {
      starts[i] = p.q.starts[i];
      if (i < p.q.B) {
        lens[i] = p.q.lens[i];
        bases[i] = item_base<R>(pl, i);
      }
    }
    pl.starts = starts;
    pl.lens = lens;
    pl.bases = bases;
    __syncthreads();
  }
  // pages of this thread's items: of the first kKept rounds they are kept
  constexpr int kKept = 4;
  int kept[kKept];
  int64_t mine_all = 0;
  auto pages_of = [&](int i) {
    const int n = i < items ? item_at<R>(pl, i).nblk : 0;
    return n > 0 ? n + EXTRA : 0;
  };
#pragma unroll
  for (int k = 0; k < kKept; ++k) {
    kept[k] = pages_of(tid + k * NT);
    mine_all += kept[k];
  }
  for (int i = tid + kKept * NT; i < items; i += NT) mine_all += pages_of(i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine_all += __shfl_xor_sync(0xFFFFFFFFu, mine_all, o);
  if (lane == 0) sh.sums[warp] = mine_all;
  __syncthreads();
  Dealt d;
  d.total = 0;
#pragma unroll
  for (int i = 0; i < NT / 32; ++i) d.total += sh.sums[i];
  d.total *= p.c.heads;
  d.per_cta = (int)(d.total >= (int64_t)W * gridDim.x ? W : ((int)d.total + gridDim.x - 1) / gridDim.x);
  d.workers = (int)min((int64_t)d.per_cta * gridDim.x, d.total);
  d.each = d.step = 0;
  if (d.total == 0) return d;
  if (d.total < (int64_t(1) << 31)) {  // the usual case, without a division of 64 bits
    d.each = (uint32_t)d.total / (uint32_t)d.workers;
  } else {
    d.each = d.total / d.workers;
  }
  // the quotient is off by 2^-21 of 2^20 at most
  const int more = (int)(d.total - d.each * d.workers);
  d.step = (uint32_t)__fdividef((float)(more << 20), (float)d.workers) + 2;
  const int w0 = (int)blockIdx.x * d.per_cta, mine = min(d.per_cta, d.workers - w0);
  if (tid < mine) {
    const int64_t f = d.start(w0 + tid);
    sh.from[tid] = f < (int64_t(1) << 31) ? (int64_t)((uint32_t)f / (uint32_t)p.c.heads) : f / p.c.heads;
  }
  // where they begin, round after round of the items
  int64_t before = 0;
#pragma unroll 1
  for (int round = 0; round * NT < items; ++round) {
    const int i = round * NT + tid;
    int n;
    if (round < kKept)
      n = round == 0 ? kept[0] : round == 1 ? kept[1] : round == 2 ? kept[2] : kept[3];
    else
      n = pages_of(i);
    int64_t incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += v;
    }
    __syncthreads();
    if (lane == 31) sh.sums[warp] = incl;
    __syncthreads();
    int64_t all = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
      if (w < warp) incl += sh.sums[w];
      all += sh.sums[w];
    }
    incl += before;
    for (int w = 0; w < mine; ++w)
      if (incl - n <= sh.from[w] && sh.from[w] < incl) {
        sh.item[w] = i;
        sh.base[w] = incl - n;
      }
    before += all;
  }
  __syncthreads();
  return d;
}

// the range of worker `me`, the CTA's number w
template <int R, int EXTRA, int W, int WARPS>
__device__ __forceinline__ Walk<R, EXTRA> walk_of(const Plan& pl, const Dealt& d, const Ranges<W, WARPS>& sh, int heads,
                                                  int me, int w) {
  Walk<R, EXTRA> k;
  const int64_t f0 = d.start(me);
  k.item = sh.item[w];
  k.it = item_at<R>(pl, k.item);
  // pages within the item: at most heads * each
  const int64_t rel = f0 - sh.base[w] * heads;
  const int each = k.it.nblk + EXTRA;
  k.head = rel < (int64_t(1) << 31) ? (int)((uint32_t)rel / (uint32_t)each) : (int)(rel / each);
  const int at = (int)(rel - (int64_t)k.head * each);
  k.blk = max(at - EXTRA, 0);
  k.left = d.start(me + 1) - f0 + (k.blk == 0 ? at : 0);
  if (k.blk == 0 && k.left <= EXTRA) k.left = 0;
  return k;
}

// What a CTA leaves for the join: `end` is where the pages of the (row tile,
// head) that it began and did not finish end, 0 if it has none; `per_cta`
// workers of the deal are a CTA's.
__device__ __forceinline__ Desc desc_of(const Dealt& d, int per_cta, int64_t end, int s0, int r0, int rows, int head) {
  Desc r{0, s0, r0, rows, head};
  if (end > 0) {
    int c = (int)blockIdx.x + 1, hi = (int)gridDim.x - 1;  // the CTA that holds the last page
    while (c < hi) {
      const int mid = (c + hi) >> 1;
      if (d.start(min((mid + 1) * per_cta, d.workers)) < end) c = mid + 1;
      else hi = mid;
    }
    r.parts = c - (int)blockIdx.x + 1;
  }
  return r;
}

// Workspace: a Desc for every CTA, then two partial results each: of the (row
// tile, head) that its range begins within (0) and of the one that it begins and
// does not finish (1): R rows of dims, then their log2 sums.  Behind them the
// same for every worker, where a CTA has several.
__host__ __device__ inline int64_t part_floats(int rows, int dim) { return (int64_t)rows * dim + rows; }
__device__ __forceinline__ float* kv_part(void* ws, int cta, int which, int rows, int dim) {
  return reinterpret_cast<float*>(static_cast<Desc*>(ws) + kKvMaxCtas) +
         ((int64_t)cta * 2 + which) * part_floats(rows, dim);
}
__device__ __forceinline__ float* kv_worker_part(void* ws, int worker, int which, int rows, int dim) {
  return kv_part(ws, kKvMaxCtas + worker, which, rows, dim);
}

// a row of the output, as an index into [tokens, query heads]
__device__ __forceinline__ int64_t kv_row(const KvAttnParams& p, int s0, int r0, int head, int r) {
  const int rr = r0 + r, i = quot(rr, p.group), d = p.group.d;
  return ((int64_t)(s0 + i) * p.c.heads + head) * d + (rr - i * d);
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// c tanh(z / c), its error relative to the result.  From z / c = 1/4 on c - 2 c / (e^(2 z / c) + 1), off by c 2^-21 at
// most (e's 2^-22 and its argument's 3 2^-24, the quotient's 2^-22), 2^-19 of tanh(1/4).  Below, where that cancels,
// the series z (1 - y^2 / 3 + 2 y^4 / 15 - 17 y^6 / 315 + 62 y^8 / 2835) in y = z / c; its next term is 2^-26.
__device__ __forceinline__ float capped_near(float z, float inv_cap) {
  const float y = z * inv_cap, y2 = y * y;
  return fmaf(z, fmaf(y2, fmaf(y2, fmaf(y2, 62.0f / 2835.0f, -17.0f / 315.0f), 2.0f / 15.0f), -1.0f / 3.0f) * y2, z);
}
__device__ __forceinline__ float capped(float z, float cap, float inv_cap) {
  const float y = fabsf(z) * inv_cap, x = y * (2.0f * kLog2e);
  const float far = cap - __fdividef(2.0f * cap, ex2(x > 126.0f ? 126.0f : x) + 1.0f);
  return y < 0.25f ? capped_near(z, inv_cap) : copysignf(far, z);
}
// 16 scores of each lane of a converged warp; the series alone where that does for all
__device__ __forceinline__ void cap_scores(float (&z)[16], float cap, float inv_cap) {
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(z[i]));
  if (__any_sync(0xFFFFFFFFu, top * inv_cap >= 0.25f)) {
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = capped(z[i], cap, inv_cap);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = capped_near(z[i], inv_cap);
  }
}

// joins the partial results of tiles of `rows` rows left by `ctas` CTAs
rn_status launch_kv_join(const KvAttnParams& p, int dim, int rows, int ctas, cudaStream_t s);
// for more than a few rows a key/value head (rn_kv_tile.cu)
rn_status launch_kv_tile(const KvAttnParams& p, int dim, int sms, cudaStream_t s);

template <class... A>
rn_status launch_pdl(void (*k)(A...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, k, a...) != cudaSuccess) return RN_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? RN_OK : RN_ERR_CUDA;
}

}  // namespace rn
