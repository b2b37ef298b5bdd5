// How the few-token kernel (rn_matvec.cu) splits its work: host arithmetic
// only, no CUDA, so that it can be compiled and examined by itself.
#pragma once

#include <cstddef>
#include <cstdint>

#if defined(__CUDACC__)
#define RN_HOST_DEVICE __host__ __device__
#else
#define RN_HOST_DEVICE
#endif

namespace rn {

constexpr int kPartStride = 36;  // floats per token of a warp's sums (32 rows, no bank conflicts)

// Bytes of one fragment of n tokens: 4 lanes x 16 bytes each, and 16 that keep
// the staging of neighbouring fragments off the same banks (with 16 tokens its
// stores had taken 32 turns each).
RN_HOST_DEVICE constexpr int frag_row(int n) { return n * 64 + 16; }

constexpr size_t kMvSmem = 224 * 1024;  // shared memory of an SM's CTAs

struct MvPlan {
  int kw;       // warps along the reduction
  int split;    // CTAs of a cluster along the reduction
  int chunks;   // chunks (256 NVFP4 / 64 bf16 elements) of the reduction
  int part;     // chunks per CTA of the cluster
  int slab;     // chunks whose tokens are in shared memory at a time
  int steps;    // groups of W / kw row tiles
  int batch;    // steps whose sums are kept while the slabs change (slab < part)
};

// the problem as the kernel variant sees it
struct MvShape {
  int N, K, H;   // tokens, reduction, outputs
  bool nvfp4;    // else bf16 weights
  bool gated;    // a row tile is 16 gate and 16 linear rows (else 32 rows)
  bool mx;       // MXFP8 output
  int T, W;      // groups of 8 tokens a CTA holds, its warps
};

// Groups of 8 tokens a CTA holds and its warps, for N tokens.  Up to 8 tokens:
// two CTAs an SM of 8 warps while their tokens are small (each CTA stages its
// own), else one of 16.  9 to 16: 12 warps, what 65536 registers hold without
// spills (16 x 4096 x 8192 gated NVFP4 21.5 us, 24.2 with 8 warps, 24.4 with 8 of
// two items in flight; 13 x 5136 x 8200 27.5, 29.0, 29.2 with the loads of that
// time, 20.7 now).
struct MvVariant {
  int T, W;
};
inline MvVariant mv_variant(int N, int K) {
  if (N <= 8) return {1, (int64_t)N * K <= 40960 ? 8 : 16};
  if (N <= 16) return {2, 12};
  return {4, 8};
}

struct MvLaunch {
  MvPlan plan;
  int groups;    // clusters (or CTAs) a group of tokens gets
  int64_t ny;    // groups of tokens
  size_t smem;   // dynamic shared memory of a CTA
};

// The last halving of the warps along the reduction may leave fewer steps than
// SMs (12 warps go from 3 to 1).  Then more of them are taken if the warp with
// the most to do gets clearly less that way, a sixth: its chunks are those of a
// step times the rounds of steps, and with 9 tokens or more a step costs about
// a third of a chunk besides (its sums).  us, 12 / 6 / 4 / 3 / 2 / 1 warps along
// the reduction of 16 x 2048 x 20000: 18.9 / 19.3 / 18.0 / 21.5 / 17.4 / 24.4,
// 16 x 2048 x 32768: 23.9 / 24.0 / 24.0 / 22.0 / 28.2 / 25.6, 9 x 528 x 21128: 18.2 /
// 13.8 / 11.9 / 11.9 / 10.5 / 13.4; 8 / 4 / 2 / 1, 1 x 624 x 8797 gated: 8.2 / 6.8 /
// 8.0 / 10.8 and, kept at 1 with its 79 steps, 30 x 1040 x 20000: 26.1 / 28.3 / 29.1 /
// 26.0.
inline int mv_more_along(const MvShape& s, int tiles, int64_t ny, const MvPlan& pl, int sms, int per_sm) {
  const auto steps = [&](int kw) { return (tiles + s.W / kw - 1) / (s.W / kw) * ny * pl.split; };
  const auto work = [&](int kw) {
    const int64_t rounds = (steps(kw) + (int64_t)sms * per_sm - 1) / ((int64_t)sms * per_sm);
    return 3 * rounds * ((pl.part + kw - 1) / kw) + (s.T > 1 ? rounds : 0);
  };
  int best = pl.kw;
  if (steps(pl.kw) < sms)
    for (int kw = pl.kw + 1; kw <= s.W; ++kw)
      if (s.W % kw == 0 && !(s.mx && s.W / kw % 2 != 0) && work(kw) < work(best) && 6 * work(kw) < 5 * work(pl.kw))
        best = kw;
  return best;
}

// The plan whose reduction is split over clusters of pl.split CTAs, at most
// `clusters` of them a group of tokens; false: there is none.
inline bool mv_plan_split(const MvShape& s, int sms, MvPlan pl, int clusters, MvLaunch* out) {
  const int T = s.T, W = s.W;
  const int J = s.nvfp4 ? 8 : 2;     // 16-byte pieces of a token a lane reads per chunk
  const int RO = s.gated ? 16 : 32;  // outputs of a row tile
  const int n = s.N < 8 * T ? s.N : 8 * T;
  const int64_t ny = ((int64_t)s.N + 8 * T - 1) / (8 * T);
  const int tiles = (s.H + RO - 1) / RO;
  const int64_t chunk_bytes = (int64_t)J * frag_row(n);
  const int per_sm = T == 1 && W == 8 ? 2 : 1;
  const int64_t fixed_bytes = 2ll * W * n * kPartStride * 4;
  pl.part = (pl.chunks + pl.split - 1) / pl.split;
  // warps along the reduction: fewer where it is short and the rows are many
  // (an MXFP8 block needs two row tiles a step), or where its slabs are short
  const int long_ = T == 1 ? 1 : 4;  // chunks a warp should have of a step
  pl.kw = s.mx ? W / 2 : W;
  while (pl.kw > 1 && pl.part < long_ * pl.kw && (int64_t)tiles * ny * pl.split * pl.kw >= (int64_t)sms * W)
    pl.kw /= 2;
  pl.kw = mv_more_along(s, tiles, ny, pl, sms, per_sm);
  int64_t step_bytes = 0, cluster_bytes = 0;
  int per = 1;
  for (;; pl.kw /= 2) {
    const int rw = W / pl.kw;
    pl.steps = (tiles + rw - 1) / rw;
    step_bytes = (int64_t)rw * n * 32 * 4;
    cluster_bytes = pl.split > 1 ? pl.split * step_bytes : 0;
    per = clusters < pl.steps ? clusters : pl.steps;
    if (per < 1) per = 1;
    pl.batch = (pl.steps + per - 1) / per;
    // the tokens whole where there is room, else in slabs
    pl.slab = pl.part;
    const int64_t room = (int64_t)(kMvSmem / per_sm) - fixed_bytes - cluster_bytes;
    if (pl.slab * chunk_bytes <= room) break;
    // a third of the room at most for the steps' sums
    const int fit = room > 0 ? (int)(room / 3 / step_bytes) : 0;
    if (pl.batch > fit) pl.batch = fit;
    if (pl.batch < 1) return false;
    pl.slab = (int)((room - pl.batch * step_bytes) / chunk_bytes);
    if (pl.slab < 1) return false;
    const int slabs = (pl.part + pl.slab - 1) / pl.slab;
    pl.slab = (pl.part + slabs - 1) / slabs;
    if (pl.slab >= long_ * pl.kw || pl.kw == 1 || pl.steps < 2 * per) break;
  }
  out->smem = (size_t)(pl.slab * chunk_bytes + fixed_bytes + cluster_bytes);
  if (pl.slab < pl.part) out->smem += (size_t)(pl.batch * step_bytes);
  out->plan = pl;
  out->groups = per;
  out->ny = ny;
  return true;
}

// What a plan in slabs costs, in the time a CTA takes to stage the tokens of a
// chunk (32 tokens: 1.1 us): every batch of steps stages them again, a round of
// steps has in each slab the chunks of its busiest warp at about 2 and 1 for
// the sums, and in a cluster 2 a row tile to exchange them.  us against the
// cost, clusters of 1 / 2 / 4 / 8: 32 x 16384 x 1024 86 (88), 46 (46), 25 (24), 37
// (28); 32 x 16384 x 4096 87 (88), 66 (60), 60 (54); 20 x 16384 x 2048 57, 32 (44),
// 26 (30), 36 (42); 12 x 65536 x 40 121, 66, 34, 20.
inline int64_t mv_slab_cost(const MvShape& s, const MvLaunch& l) {
  const MvPlan& p = l.plan;
  const int64_t rounds = (p.steps + l.groups - 1) / l.groups;
  const int64_t slabs = (p.part + p.slab - 1) / p.slab;
  const int64_t batches = slabs > 1 ? (rounds + p.batch - 1) / p.batch : 1;
  return batches * p.part + rounds * slabs * (2 * ((p.slab + p.kw - 1) / p.kw) + 1) +
         (p.split > 1 ? 2 * rounds * (s.W / p.kw) : 0);
}

// false: no plan
inline bool mv_plan(const MvShape& s, int sms, MvLaunch* out) {
  const int CK = s.nvfp4 ? 256 : 64;
  const int RO = s.gated ? 16 : 32;
  const int64_t ny = ((int64_t)s.N + 8 * s.T - 1) / (8 * s.T);
  const int tiles = (s.H + RO - 1) / RO;
  const int per_sm = s.T == 1 && s.W == 8 ? 2 : 1;
  MvPlan pl{};
  pl.chunks = (s.K + CK - 1) / CK;
  // few row tiles: the reduction over a cluster, while its CTAs' warps keep
  // two chunks each
  pl.split = 1;
  while (pl.split < 8 && tiles * ny * pl.split < sms && pl.chunks >= 2 * s.W * pl.split) pl.split *= 2;
  const bool found = mv_plan_split(s, sms, pl, per_sm * sms / pl.split, out);
  if (pl.split == 1 || (found && out->plan.slab == out->plan.part)) return found;
  // The tokens of a cluster's CTA do not fit: in slabs, by the cheapest split
  // (up to 8 tokens fit a cluster of 8 up to K = 88064: no slabs in clusters for
  // them).  So many clusters of 1, 2, 4, 8 CTAs with an SM each run at a time on a
  // GB300 of 152 SMs.
  const int resident[4] = {sms, sms / 2, sms * 36 / 152, sms * 15 / 152};
  bool any = false;
  for (int i = 0; i < 4; ++i) {
    pl.split = 1 << i;
    MvLaunch l{};
    if (!mv_plan_split(s, sms, pl, resident[i] > ny ? (int)(resident[i] / ny) : 1, &l)) continue;
    if (s.T == 1 && i > 0 && l.plan.slab < l.plan.part) continue;
    if (!any || mv_slab_cost(s, l) < mv_slab_cost(s, *out)) *out = l;
    any = true;
  }
  return any;
}

}  // namespace rn
