"""Cases that measure the paged 8-bit key/value cache and the attention that reads it.

Three operators, named by a case's "op":

  write   the keys and values of new tokens go into their sequences' pages, E4M3 with one power-of-two
          scale for each page of 64 positions and head; a page whose scale grows is scaled over
  read    positions of the cache as numbers again
  attend  softmax(scale q k^T) v of new tokens with the cached positions of their sequences, causal,
          with an optional window, cap of the scores (tanh) and bias by distance

B sequences; row starts[b] + i of the new tokens is position lens[b] - n_b + i of sequence b, which stands in
page table[b, position // 64].  Keys lie [pages, heads, 64, dim], values transposed [pages, heads, dim, 64].
"""
import math
import random

import torch

own = False

PAGE = 64
E_MIN, E_MAX = -120, 120
OPS = ("write", "read", "attend")


def _case(name, op, B, new, held, heads, dim, group=1, dtype="bf16", ragged=False, window=0, softcap=0.0,
          slopes=False, causal=True, mix=0):
    """new: tokens a sequence gets (write, attend) or gives back (read); held: positions before them."""
    c = {"op": op, "B": B, "new": new, "held": held, "heads": heads, "dim": dim, "group": group, "dtype": dtype,
         "ragged": ragged, "window": window, "softcap": softcap, "slopes": slopes, "causal": causal, "mix": mix}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one token of each of a few sequences joins its page while text is generated: all latency
        _case("write 32x1 h8 d128", "write", 32, 1, 1500, 8, 128, ragged=True, mix=1),
        # odd head count, a narrow head, fp32 keys and values, pages begun by earlier tokens
        _case("write 7x777 h5 d64 f32", "write", 7, 777, 100, 5, 64, dtype="f32", ragged=True, mix=2),
        # a batch of prompts of different lengths
        _case("write 16x4096 h8 d128", "write", 16, 4096, 0, 8, 128, ragged=True, mix=3),
        # one short sequence is taken out of the cache
        _case("read 1x1000 h4 d64", "read", 1, 1000, 0, 4, 64),
        # a batch of long sequences is taken out of the cache
        _case("read 24x16000 h8 d128", "read", 24, 16000, 0, 8, 128, ragged=True, mix=4),
        # one token of one short sequence: all latency
        _case("attend 1x1 len 1000", "attend", 1, 1, 999, 8, 128, 4),
        # one token of one very long sequence
        _case("attend 1x1 len 131072", "attend", 1, 1, 131071, 8, 128, 8),
        # one token of each of many sequences of different lengths
        _case("attend 64x1 len 16384", "attend", 64, 1, 16383, 8, 128, 8, ragged=True, mix=5),
        # every query head with keys of its own, a window and a bias by distance, narrow heads
        _case("attend 16x1 window h20 d64", "attend", 16, 1, 4001, 20, 64, 1, ragged=True, window=1000, slopes=True,
              mix=6),
        # wide heads and capped scores
        _case("attend 9x1 cap h4 d256", "attend", 9, 1, 8000, 4, 256, 4, ragged=True, softcap=50.0, mix=7),
        # a few drafted tokens of each sequence are checked at once, an odd number of heads to a key
        _case("attend 32x4 len 6000", "attend", 32, 4, 6000, 8, 128, 5, ragged=True, mix=8),
        # a part of a prompt meets what the cache holds of it
        _case("attend 1x4096 on 8192", "attend", 1, 4096, 8192, 8, 128, 8),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    most = [work(c) for c in listed()]
    bytes_, flops = max(w["bytes"] for w in most), max(w["flops"] for w in most)
    op = rng.choice(["write", "read", "attend", "attend", "attend"])
    while True:
        heads, dim = rng.randint(1, 16), rng.choice([64, 128, 128, 192, 256])
        dtype, mix = rng.choice(["bf16", "bf16", "f32"]), rng.randrange(1 << 30)
        if op == "write":
            c = _case("", op, _log(rng, 1, 256), _log(rng, 1, 4096), _log(rng, 1, 4096) - 1, heads, dim, dtype=dtype,
                      ragged=True, mix=mix)
        elif op == "read":
            c = _case("", op, _log(rng, 1, 64), _log(rng, 1, 16384), _log(rng, 1, 4096) - 1, heads, dim, dtype=dtype,
                      ragged=True, mix=mix)
        else:
            new = rng.choice([1, 1, 1, rng.randint(2, 8), _log(rng, 16, 4096)])
            c = _case("", op, _log(rng, 1, 128 if new <= 8 else 8), new, _log(rng, 1, 131072) - 1, heads, dim,
                      rng.choice([1, 2, 4, 5, 8, 16]), ragged=True,
                      window=_log(rng, 16, 8192) if rng.random() < 0.25 else 0,
                      softcap=rng.choice([0.0, 0.0, 0.0, 30.0, 50.0]), slopes=rng.random() < 0.2,
                      causal=rng.random() < 0.9, mix=mix)
        w = work(c)
        if w["bytes"] <= bytes_ and w["flops"] <= flops and _cached_bytes(c) <= 3 << 30:
            return c


def _sequences(case):
    """(new tokens, positions held with them) of each sequence."""
    rng = random.Random(case["mix"])
    out = []
    for _ in range(case["B"]):
        new, held = case["new"], case["held"]
        if case["ragged"]:
            held = rng.randint(held // 4, held)
            if new > 8:
                new = rng.randint(new // 2, new)
        out.append((new, held + new))
    return out


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _cached_bytes(case):
    return sum(_pages(n) for _, n in _sequences(case)) * PAGE * case["heads"] * case["dim"] * 2


def _seen(case, new, n, i):
    """The positions [lo, hi) that new token i of a sequence attends to."""
    p = n - new + i
    return (max(0, p - case["window"] + 1) if case["window"] else 0), (p + 1 if case["causal"] else n)


def work(case):
    H, D, G = case["heads"], case["dim"], case["group"]
    seqs = _sequences(case)
    rows = sum(new for new, _ in seqs)
    if case["op"] != "attend":
        esz = 4 if case["dtype"] == "f32" else 2
        pages = sum(_pages(n) - (n - new) // PAGE for new, n in seqs)
        return {"bytes": rows * H * D * 2 * (esz + 1) + 2 * pages * H, "flops": 2 * rows * H * D}
    held = pairs = 0
    for new, n in seqs:
        held += _seen(case, new, n, new - 1)[1] - _seen(case, new, n, 0)[0]
        for i in range(new):
            lo, hi = _seen(case, new, n, i)
            pairs += hi - lo
    return {"bytes": held * H * (2 * D) + 2 * (held // PAGE) * H + 4 * rows * H * G * D, "flops": 4 * pairs * H * G * D}


def _exponents(amax):
    """The smallest e with amax <= 448 2^e."""
    m, x = torch.frexp(amax)
    return (x - 9 + (m > 0.875).int()).clamp(E_MIN, E_MAX)


def _pow2(e):
    """2^e as the float with that exponent; no value of e beyond +-126 is used."""
    return ((e.clamp(-126, 127) + 127).int() << 23).view(torch.float32)


def _codes(x, dims):
    """E4M3 codes and E8M0 bytes of x, one scale over `dims`."""
    e = _exponents(x.abs().amax(dims))
    f = _pow2(-e)[(...,) + (None,) * len(dims)]
    return (x * f).to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    H, D, op = case["heads"], case["dim"], case["op"]
    seqs = _sequences(case)
    rows = sum(new for new, _ in seqs)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = {"case": case, "rows": rows, "seqs": seqs}
    width = max(_pages(n) for _, n in seqs)
    total = sum(_pages(n) for _, n in seqs)
    order = torch.randperm(total + 3, generator=g, device="cuda").int()  # pages lie in no order
    table = torch.zeros(len(seqs), width, dtype=torch.int32, device="cuda")
    at = 0
    for b, (_, n) in enumerate(seqs):
        table[b, :_pages(n)] = order[at:at + _pages(n)]
        at += _pages(n)
    s["table"] = table
    s["starts"] = torch.tensor([0] + [new for new, _ in seqs], device="cuda").cumsum(0).int()
    s["lens"] = torch.tensor([n for _, n in seqs], device="cuda").int()
    P = total + 3
    s["k"] = torch.empty(P, H, PAGE, D, dtype=torch.uint8, device="cuda")
    s["v"] = torch.empty(P, H, D, PAGE, dtype=torch.uint8, device="cuda")
    s["ks"] = torch.empty(P, H, dtype=torch.uint8, device="cuda")
    s["vs"] = torch.empty(P, H, dtype=torch.uint8, device="cuda")
    for a in range(0, P, 1024):
        n = min(1024, P - a)
        # channels of different size, pages of different size
        size = torch.exp(0.5 * randn(1, H, 1, D)) * torch.exp(0.3 * randn(n, H, 1, 1))
        s["k"][a:a + n], s["ks"][a:a + n] = _codes(randn(n, H, PAGE, D) * size, (2, 3))
        s["v"][a:a + n], s["vs"][a:a + n] = _codes(randn(n, H, D, PAGE) * torch.exp(0.3 * randn(n, H, 1, 1)), (2, 3))
    if op == "write":
        dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        s["new_k"], s["new_v"] = (randn(rows, H, D) * 2.0).to(dt), (randn(rows, H, D) * 1.5).to(dt)
    elif op == "attend":
        s["q"] = (randn(rows, H * case["group"], D) * 1.5).bfloat16()
        if case["slopes"]:
            n = H * case["group"]
            s["slopes"] = torch.exp2(-8.0 * torch.arange(1, n + 1, device="cuda") / n)
    return s


def _plain_write(s):
    """Pages of each sequence in turn: old values and new ones under the larger of both scales."""
    for b, (new, n) in enumerate(s["seqs"]):
        a = s["offsets"][b]
        first, p0 = (n - new) // PAGE, n - new
        ids = s["table"][b, first:_pages(n)].long()
        m = ids.numel()
        pos = torch.arange(m * PAGE, device="cuda") + first * PAGE
        fresh = ((pos >= p0) & (pos < n)).view(m, 1, PAGE, 1)
        kept = (pos < p0).view(m, 1, PAGE, 1)
        begun = (kept.any(2)[..., 0]).expand(m, s["ks"].shape[1])
        for name, codes, scales, swap in (("new_k", "k", "ks", False), ("new_v", "v", "vs", True)):
            x = s[name][a:a + new].float()
            full = torch.zeros(m * PAGE, *x.shape[1:], device="cuda")
            full[p0 - first * PAGE:n - first * PAGE] = x
            full = full.view(m, PAGE, *x.shape[1:]).transpose(1, 2)  # [m, H, PAGE, D]
            e = _exponents(full.abs().amax((2, 3)))
            old_e = s[scales][ids].int() - 127
            e = torch.where(begun, torch.maximum(e, old_e), e)
            old = s[codes][ids].view(torch.float8_e4m3fn).float()
            old = old.transpose(2, 3) if swap else old
            held = (old * _pow2(old_e - e)[..., None, None]).clamp(-448.0, 448.0)
            now = (full * _pow2(-e)[..., None, None]).clamp(-448.0, 448.0)
            out = torch.where(fresh, now, torch.where(kept, held, old)).to(torch.float8_e4m3fn).view(torch.uint8)
            s[codes][ids] = out.transpose(2, 3) if swap else out
            s[scales][ids] = (e + 127).to(torch.uint8)


def _values(codes, scales):
    return codes.view(torch.float8_e4m3fn).float() * _pow2(scales.int() - 127)[..., None, None]


def _plain_read(s):
    H, D = s["case"]["heads"], s["case"]["dim"]
    dt = torch.float32 if s["case"]["dtype"] == "f32" else torch.bfloat16
    k = torch.empty(s["rows"], H, D, dtype=dt, device="cuda")
    v = torch.empty_like(k)
    for b, (new, n) in enumerate(s["seqs"]):
        a, first = s["offsets"][b], (n - new) // PAGE
        ids = s["table"][b, first:_pages(n)].long()
        lo, hi = n - new - first * PAGE, n - first * PAGE
        k[a:a + new] = _values(s["k"][ids], s["ks"][ids]).transpose(1, 2).reshape(-1, H, D)[lo:hi].to(dt)
        v[a:a + new] = _values(s["v"][ids], s["vs"][ids]).permute(0, 3, 1, 2).reshape(-1, H, D)[lo:hi].to(dt)
    return k, v


def _plain_attend(s):
    case = s["case"]
    H, D, G = case["heads"], case["dim"], case["group"]
    out = torch.empty(s["rows"], H * G, D, dtype=torch.bfloat16, device="cuda")
    for b, (new, n) in enumerate(s["seqs"]):
        a = s["offsets"][b]
        ids = s["table"][b, :_pages(n)].long()
        k = _values(s["k"][ids], s["ks"][ids]).transpose(0, 1).reshape(H, -1, D)[:, :n]
        v = _values(s["v"][ids], s["vs"][ids]).permute(1, 0, 3, 2).reshape(H, -1, D)[:, :n]
        j = torch.arange(n, device="cuda")
        step = max(1, (1 << 28) // (n * H * G))
        for i in range(0, new, step):
            m = min(step, new - i)
            q = s["q"][a + i:a + i + m].float().view(m, H, G, D).permute(1, 2, 0, 3).reshape(H, G * m, D)
            z = (q @ k.transpose(1, 2)).view(H, G, m, n) * (1.0 / math.sqrt(D))
            if case["softcap"]:
                z = case["softcap"] * torch.tanh(z / case["softcap"])
            p = (torch.arange(i, i + m, device="cuda") + (n - new))[:, None]
            if case["slopes"]:
                z = z + s["slopes"].view(H, G, 1, 1) * (j - p).float()
            sees = (j <= p) if case["causal"] else (j >= 0).expand(m, n)
            if case["window"]:
                sees = sees & (j > p - case["window"])
            z = z.masked_fill(~sees, -math.inf)
            z = torch.exp(z - z.amax(-1, keepdim=True))
            z = z / z.sum(-1, keepdim=True)
            y = (z.view(H, G * m, n) @ v).view(H, G, m, D).permute(2, 0, 1, 3).reshape(m, H * G, D)
            out[a + i:a + i + m] = y.bfloat16()
    return out


def run(s):
    case, op = s["case"], s["case"]["op"]
    if own:
        import mxfp8_quantization_gb300 as rn
        cache = rn.KVCache(s["k"], s["v"], s["ks"], s["vs"])
        seqs = rn.KVSequences(s["table"], s["starts"], s["lens"])
        if op == "write":
            rn.kv_cache_write(cache, seqs, s["new_k"], s["new_v"])
        elif op == "read":
            return rn.kv_cache_read(cache, seqs, s["rows"],
                                    out_dtype=torch.float32 if case["dtype"] == "f32" else torch.bfloat16)
        else:
            return rn.kv_attention(s["q"], cache, seqs, causal=case["causal"], window=case["window"],
                                   softcap=case["softcap"], slopes=s.get("slopes"))
    else:
        s["offsets"] = [0]
        for new, _ in s["seqs"]:
            s["offsets"].append(s["offsets"][-1] + new)
        if op == "read":
            return _plain_read(s)
        if op == "attend":
            return _plain_attend(s)
        _plain_write(s)
    return {"k": s["k"].view(torch.float8_e4m3fn), "v": s["v"].view(torch.float8_e4m3fn),
            "k_scales": s["ks"].view(torch.float8_e8m0fnu), "v_scales": s["vs"].view(torch.float8_e8m0fnu)}


def exact(case, seed):
    s = prepare(case, seed)
    H, D, G, op = case["heads"], case["dim"], case["group"], case["op"]
    two = torch.tensor(2.0, dtype=torch.float64, device="cuda")

    def real(codes, scales, ids):
        return codes[ids].view(torch.float8_e4m3fn).double(), torch.pow(two, scales[ids].double() - 127.0)

    if op == "write":
        out = {"k": s["k"].view(torch.float8_e4m3fn).double(), "v": s["v"].view(torch.float8_e4m3fn).double(),
               "k_scales": torch.pow(two, s["ks"].double() - 127.0), "v_scales": torch.pow(two, s["vs"].double() - 127.0)}
        row = 0
        for b, (new, n) in enumerate(s["seqs"]):
            done = 0
            while done < new:  # page by page
                p = n - new + done
                off, take = p % PAGE, min(PAGE - p % PAGE, new - done)
                page = int(s["table"][b, p // PAGE])
                for name, codes, scales in (("new_k", "k", "k_scales"), ("new_v", "v", "v_scales")):
                    x = s[name][row + done:row + done + take].double().permute(1, 0, 2)  # [H, take, D]
                    top = x.abs().amax((1, 2))
                    unit = torch.pow(two, torch.ceil(torch.log2(top / 448.0)).clamp(E_MIN, E_MAX))
                    unit = torch.where(top > 448.0 * unit, 2 * unit, unit)
                    unit = torch.where(top <= 224.0 * unit, unit / 2, unit)
                    if off:
                        old = out[scales][page]
                        unit = torch.maximum(unit, old)
                        shrink = (old / unit)[:, None, None]
                        if codes == "k":
                            out[codes][page][:, :off] *= shrink
                        else:
                            out[codes][page][:, :, :off] *= shrink
                    x = (x / unit[:, None, None]).clamp(-448.0, 448.0)
                    if codes == "k":
                        out[codes][page][:, off:off + take] = x
                    else:
                        out[codes][page][:, :, off:off + take] = x.transpose(1, 2)
                    out[scales][page] = unit
                done += take
            row += new
        return out
    if op == "read":
        k, v = [], []
        for b, (new, n) in enumerate(s["seqs"]):
            pos = torch.arange(n - new, n, device="cuda")
            page, off = s["table"][b].long()[pos // PAGE], pos % PAGE
            unit = torch.pow(two, s["ks"][page].double() - 127.0)[..., None]
            k.append(s["k"][page, :, off].view(torch.float8_e4m3fn).double() * unit)
            unit = torch.pow(two, s["vs"][page].double() - 127.0)[..., None]
            v.append(s["v"][page, :, :, off].view(torch.float8_e4m3fn).double() * unit)
        return torch.cat(k), torch.cat(v)
    if work(case)["flops"] > 4e12:
        return None
    out = torch.empty(s["rows"], H * G, D, dtype=torch.float64, device="cuda")
    row = 0
    for b, (new, n) in enumerate(s["seqs"]):
        ids = s["table"][b, :(n + PAGE - 1) // PAGE].long()
        pos = torch.arange(n, dtype=torch.float64, device="cuda")
        for h in range(H):
            kc, ku = real(s["k"][:, h], s["ks"][:, h], ids)
            vc, vu = real(s["v"][:, h], s["vs"][:, h], ids)
            keys = (kc * ku[:, None, None]).reshape(-1, D)[:n]
            vals = (vc * vu[:, None, None]).transpose(1, 2).reshape(-1, D)[:n]
            for i in range(0, new, 2048):
                m = min(2048, new - i)
                mine = pos.new_tensor(range(n - new + i, n - new + i + m))[:, None]
                hidden = torch.zeros(m, n, dtype=torch.bool, device="cuda")
                if case["causal"]:
                    hidden |= pos > mine
                if case["window"]:
                    hidden |= pos <= mine - case["window"]
                for g in range(h * G, h * G + G):
                    t = s["q"][row + i:row + i + m, g].double() @ keys.T / D ** 0.5
                    if case["softcap"]:
                        t = torch.tanh(t / case["softcap"]) * case["softcap"]
                    if case["slopes"]:
                        t = t + s["slopes"][g].double() * (pos - mine)
                    t = t.masked_fill(hidden, -math.inf).softmax(-1)
                    out[row + i:row + i + m, g] = t @ vals
        row += new
    return out
