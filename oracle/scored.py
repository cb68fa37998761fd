"""The fused norm / rotation / append and the attentions with modified scores, in 64 bits.

Plain statements from the formulas in include/pa.h, on CPU torch tensors in float64.
They share no code with the CUDA library.  Every attention result comes with the
sums its error bound needs (see ``Bound``).
"""
from __future__ import annotations

import dataclasses
import math
from typing import Optional

import torch


def stored(x: torch.Tensor) -> torch.Tensor:
    """The values a tensor of any storage dtype holds, in float64."""
    return x.float().double() if x.dtype == torch.float8_e4m3fn else x.double()


# ----------------------------------------------------------- norm, rotation, append

def norm_rope(x: torch.Tensor, weight: Optional[torch.Tensor], eps: float, weight_offset: float,
              cos_sin: Optional[torch.Tensor], positions, interleaved: bool):
    """x [T, H, D] -> (rows in float64, the magnitude |a| + |b| each element is made of)."""
    y = stored(x)
    if weight is not None:
        rms = torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
        y = y / rms * (stored(weight) + weight_offset)
    size = y.abs()
    if cos_sin is None or cos_sin.shape[1] == 0:
        return y, size
    out, osize = y.clone(), size.clone()
    r = cos_sin.shape[1]
    for j in range(r // 2):
        ia, ib = (2 * j, 2 * j + 1) if interleaved else (j, j + r // 2)
        c = cos_sin[positions, j].double()[:, None]
        s = cos_sin[positions, r // 2 + j].double()[:, None]
        a, b = y[..., ia], y[..., ib]
        out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
        osize[..., ia] = osize[..., ib] = size[..., ia] + size[..., ib]
    return out, osize


# ------------------------------------------------------------------------- attention

LOG2E = math.log2(math.e)


def _rounding(D: int) -> float:
    """fp32 arithmetic of one score, relative to the sum of its terms' magnitudes: D
    products and their sums, and the modifications, each within 2^-24."""
    return (D + 32) * 2.0 ** -24


@dataclasses.dataclass
class Bound:
    """out: the result; weighted: sum_i p_i |v_i| per output element; moved: how far
    the output moves, to first order, where every score z_i is off by its size,
    size_i = 1 + sum_d |q_d k_d| * scale + |what the cap leaves| + |bias| + |z_i - max z|
    (the last for the subtraction of the maximum).  With dz_i the scores' errors,
        d out = sum_i p_i dz_i (v_i - out),
    at most sum_i p_i |dz_i| |v_i| + (sum_i p_i |dz_i|) * weighted: a key that weighs
    nothing adds nothing, however large its bias.  spread: sum_i |v_i| over the visible
    keys."""
    out: torch.Tensor
    weighted: torch.Tensor
    moved: torch.Tensor
    spread: torch.Tensor

    def tolerance(self, out_dtype: torch.dtype, p_dtype: Optional[torch.dtype], D: int):
        """How far a kernel may be off: the output's own rounding, the rounding
        of each probability to p_dtype (in the numerator and in the sum), the fp32
        arithmetic of the scores, and the weighted sum in fp32.  A probability is taken
        against a maximum of 1, so below p_dtype's smallest normal number it is off by
        half that number's step whatever its size (f16: 2^-25 a key; the sum is 1 at
        least)."""
        half = lambda t: torch.finfo(t).eps / 2                          # noqa: E731
        up = half(p_dtype) if p_dtype is not None else 0.0
        low = up * torch.finfo(p_dtype).smallest_normal if p_dtype is not None else 0.0
        # (below its smallest normal number a type's steps stay what they are there)
        out = half(out_dtype) * self.out.abs().clamp(min=torch.finfo(out_dtype).smallest_normal)
        return (out + (2 * up + 2.0 ** -18) * self.weighted
                + _rounding(D) * self.moved + low * self.spread + 1e-30)


def scored_attention(q, key_cache, value_cache, block_tables, context_lens, query_start, scale,
                     softcap=0.0, slopes=None, window=0, key_start=None, prefix_lens=None,
                     k_scale=1.0, v_scale=1.0) -> Bound:
    """q [T, Hq, D]; query_start [S + 1] (None: one new token per sequence)."""
    T, Hq, D = q.shape
    NB, bs, Hkv, _ = key_cache.shape
    G = Hq // Hkv
    S = len(context_lens)
    qs = list(range(S + 1)) if query_start is None else [int(x) for x in query_start]
    out = torch.zeros(T, Hq, D, dtype=torch.float64)
    wtd, moved, spread = (torch.zeros_like(out) for _ in range(3))
    qd = stored(q)
    for s in range(S):
        a, b, n = qs[s], qs[s + 1], int(context_lens[s])
        L = b - a
        if L == 0:
            continue
        p = torch.arange(n - L, n)[:, None]
        i = torch.arange(n)[None, :]
        ahead = p if prefix_lens is None else torch.clamp(p, min=int(prefix_lens[s]) - 1)
        seen = i <= ahead
        if window:
            seen &= p - i < window
        if key_start is not None:
            ks = key_start[s:s + 1] if query_start is None else key_start[a:b]
            seen &= i >= ks[:, None]
        if not seen.any():
            continue
        # rows of keys nobody sees are left out: their blocks need not exist
        keys = torch.nonzero(seen.any(0))[:, 0]
        seen = seen[:, keys]
        dist = (p - keys[None, :]).abs().double()
        blk, off = block_tables[s][keys // bs].long(), keys % bs
        kk = stored(key_cache[blk, off]) * k_scale          # [n', Hkv, D]
        vv = stored(value_cache[blk, off]) * v_scale
        for h in range(Hq):
            z = scale * (qd[a:b, h] @ kk[:, h // G].T)
            # (infinite elements are exact: they add no rounding)
            q_fine, k_fine = (torch.where(torch.isfinite(x), x, 0.0).abs()
                              for x in (qd[a:b, h], kk[:, h // G]))
            size = abs(scale) * (q_fine @ k_fine.T)
            if softcap:
                # an error of the product passes with the tanh's slope, largest at the
                # end of its interval that is nearer to zero
                near = (z.abs() - _rounding(D) * size).clamp(min=0.0) / softcap
                z = softcap * torch.tanh(z / softcap)
                size = size * (1 - torch.tanh(near) ** 2) + z.abs()
            if slopes is not None:
                slope = abs(float(slopes[h]))
                z = z - float(slopes[h]) * dist
                # kernels may count the distance from their tile's first key, up to 128
                # away, where that loses little (slopes up to 64 in log2 units): four
                # roundings of it, where _rounding() has D + 32
                size = size + slope * (dist + (4 * 128 / (D + 32) if slope * LOG2E <= 64 else 0))
            z = z.masked_fill(~seen, -math.inf)
            some = seen.any(1)
            w = torch.zeros_like(z)
            w[some] = torch.softmax(z[some], -1)
            size = 1 + size + (z - z.amax(1, keepdim=True)).abs()
            share = torch.where(seen & (w != 0), w * size, 0.0)
            v = vv[:, h // G]
            bad = ~torch.isfinite(v)
            if bad.any():      # a value reaches the rows that see its key, and no other
                fine = w @ torch.where(bad, 0.0, v)
                for key, d in torch.nonzero(bad).tolist():
                    fine[seen[:, key], d] += v[key, d]
                out[a:b, h] = fine
            else:
                out[a:b, h] = w @ v
            v_size = torch.nan_to_num(v, 0.0, 0.0, 0.0).abs()
            wtd[a:b, h] = w @ v_size
            spread[a:b, h] = seen.double() @ v_size
            moved[a:b, h] = share @ v_size + share.sum(1, keepdim=True) * wtd[a:b, h]
    return Bound(out, wtd, moved, spread)
