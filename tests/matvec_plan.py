"""The few-token kernel's plan (csrc/rn_matvec_plan.h, host arithmetic only), compiled by itself."""
import ctypes
import os
import subprocess
import tempfile
from functools import lru_cache
from types import SimpleNamespace

import mxfp8_quantization_gb300 as rn

CSRC = os.path.join(os.path.dirname(os.path.abspath(rn.__file__)), "csrc")
FIELDS = ("T", "W", "kw", "split", "chunks", "part", "slab", "steps", "batch", "groups", "ny", "smem")

WRAPPER = """
#include "rn_matvec_plan.h"
extern "C" int plan(int N, int K, int H, int nvfp4, int gated, int mx, int sms, long long* o) {
  const rn::MvVariant v = rn::mv_variant(N, K);
  rn::MvLaunch l{};
  if (!rn::mv_plan({N, K, H, nvfp4 != 0, gated != 0, mx != 0, v.T, v.W}, sms, &l)) return 0;
  const rn::MvPlan& p = l.plan;
  const long long f[12] = {v.T, v.W, p.kw, p.split, p.chunks, p.part, p.slab, p.steps, p.batch, l.groups, l.ny,
                           (long long)l.smem};
  for (int i = 0; i < 12; ++i) o[i] = f[i];
  return 1;
}
"""


@lru_cache(maxsize=1)
def _lib():
    d = tempfile.mkdtemp()
    src, so = os.path.join(d, "plan.cc"), os.path.join(d, "plan.so")
    with open(src, "w") as f:
        f.write(WRAPPER)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, src, "-o", so], check=True)
    return ctypes.CDLL(so)


def plan(N, K, H, nvfp4=True, gated=False, mx=False, sms=152):
    """The plan for N tokens, K inputs and H outputs, with what follows from it; None if there is none."""
    o = (ctypes.c_longlong * 12)()
    if not _lib().plan(N, K, H, nvfp4, gated, mx, sms, o):
        return None
    p = SimpleNamespace(**dict(zip(FIELDS, o)))
    p.per_sm = 2 if (p.T, p.W) == (1, 8) else 1
    p.n = min(N, 8 * p.T)
    p.tiles = -(-H // (16 if gated else 32))
    p.rw = p.W // p.kw
    p.slabs = -(-p.part // p.slab)
    p.rounds = -(-p.steps // p.groups)
    p.batches = -(-p.rounds // p.batch) if p.slabs > 1 else 1
    p.ctas = p.groups * p.split * p.ny
    return p
