"""Seeded paged inputs for the attentions with modified scores, and their comparison.

What no query may see is poisoned: blocks that no table names, slots past a
sequence's length and keys before every row's first visible one hold NaN, and
table entries of blocks with no visible key hold an id outside the cache.
"""
import math

import torch

from oracle import scored

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16,
      "fp8": torch.float8_e4m3fn}


def poison(cache, blk, off, head=slice(None), dim=slice(None)):
    if cache.dtype == torch.float8_e4m3fn:
        cache.view(torch.uint8)[blk, off, head, dim] = 0x7F
    else:
        cache[blk, off, head, dim] = float("nan")


def make(cached, new, Hq, Hkv, D, bs, dt, cdt, softcap=0.0, alibi=False, window=0, key_start=None,
         prefix_lens=None, seed=0, q_scale=2.0, decode=False):
    """cached / new: tokens per sequence.  key_start: per new token (decode: per sequence)."""
    g = torch.Generator().manual_seed(seed)
    S = len(cached)
    n = [c + l for c, l in zip(cached, new)]
    nblk = [-(-x // bs) for x in n]
    MB = max(nblk + [1])
    used = sum(nblk)
    NB = used + 3
    perm = torch.randperm(NB, generator=g)
    tables = torch.full((S, MB), -1, dtype=torch.int32)
    at = 0
    for s in range(S):
        tables[s, :nblk[s]] = perm[at:at + nblk[s]]
        at += nblk[s]

    def cache():
        x = torch.randn(NB, bs, Hkv, D, generator=g)
        return (x * 40).clamp(-448, 448).to(DT[cdt]) if cdt == "fp8" else x.to(DT[cdt])
    kc, vc = cache(), cache()
    for b in perm[at:].tolist():
        poison(kc, b, slice(None))
        poison(vc, b, slice(None))
    qs = [0]
    for l in new:
        qs.append(qs[-1] + l)
    T = qs[-1]
    ks = None if key_start is None else torch.tensor(key_start, dtype=torch.int32)
    pl = None if prefix_lens is None else torch.tensor(prefix_lens, dtype=torch.int32)
    for s in range(S):
        for t in range(n[s], nblk[s] * bs):
            poison(kc, int(tables[s, t // bs]), t % bs)
            poison(vc, int(tables[s, t // bs]), t % bs)
        if new[s] == 0:
            continue
        p = torch.arange(cached[s], n[s])
        lo = torch.zeros_like(p)
        if window:
            lo = (p - window + 1).clamp(min=0)
        if ks is not None:
            lo = torch.maximum(lo, (ks[s:s + 1] if decode else ks[qs[s]:qs[s + 1]]).long())
        hi = p if pl is None else torch.maximum(p, (pl[s] - 1).clamp(max=n[s] - 1).long())
        some = lo <= hi
        first = int(lo[some].min()) if some.any() else n[s]
        for t in range(min(first, n[s])):
            poison(kc, int(tables[s, t // bs]), t % bs)
            poison(vc, int(tables[s, t // bs]), t % bs)
        tables[s, :(first // bs if first < n[s] else nblk[s])] = NB + 7
    q = (torch.randn(T, Hq, D, generator=g) * q_scale).to(DT[dt])
    slopes = torch.exp2(-8.0 * (torch.arange(Hq) + 1) / Hq).float() if alibi else None
    fp8 = cdt == "fp8"
    return {"q": q, "kc": kc, "vc": vc, "tables": tables,
            "lens": torch.tensor(n, dtype=torch.int32), "qs": torch.tensor(qs, dtype=torch.int32),
            "scale": 1.0 / math.sqrt(D), "softcap": softcap, "slopes": slopes, "window": window,
            "key_start": ks, "prefix_lens": pl, "k_scale": 0.025 if fp8 else 1.0,
            "v_scale": 0.03 if fp8 else 1.0, "max_ctx": max(n + [0]), "max_new": max(new + [0]),
            "decode": decode, "dt": dt, "cdt": cdt}


def oracle(c) -> scored.Bound:
    return scored.scored_attention(
        c["q"], c["kc"], c["vc"], c["tables"], c["lens"], None if c["decode"] else c["qs"],
        c["scale"], c["softcap"], c["slopes"], c["window"], c["key_start"], c["prefix_lens"],
        c["k_scale"], c["v_scale"])


def check(c, got, what, want=None):
    """Element by element: the same NaN pattern, the rest within the derived tolerance."""
    b = oracle(c) if want is None else want
    g = got.cpu().double()
    nan = torch.isnan(b.out)
    assert torch.equal(torch.isnan(g), nan), \
        f"{what}: NaN pattern differs at {torch.nonzero(torch.isnan(g) != nan)[:4].tolist()}"
    p_dt = {"f32": None, "fp8": torch.float16}.get(c["cdt"], DT[c["dt"]])
    fine = torch.isfinite(b.out)
    assert torch.equal(g[~fine & ~nan], b.out[~fine & ~nan]), f"{what}: infinities"
    tol = b.tolerance(DT[c["dt"]], p_dt, c["q"].shape[2])
    over = ((g - b.out).abs() - tol)[fine]
    assert over.numel() == 0 or (over <= 0).all(), \
        f"{what}: {int((over > 0).sum())} of {over.numel()} elements, {float(over.max()):.3g} over"
