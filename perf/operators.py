"""What the fused cache append and the attentions with modified scores are measured on.

Three operators of the library, each as a user's program calls it (``own`` true) and in its
plain form (``own`` false: elementary torch operations in 32 bits, rounded once at the end):

* ``append``   norm of every query and key head, rotation by position, and the write of the new
               tokens' keys and values into their cache slots (pa_norm_rope_append);
* ``decode``   single-token attention over the paged cache with capped scores, a distance bias,
               a sliding window and a first visible key per sequence (pa_decode_scored);
* ``chunk``    the same for a batch of new-token chunks, with a first visible key per new token
               and a bidirectional prefix per sequence (pa_prefill_scored).

``listed()`` gives the measured cases, ``draw`` more of the same ranges, ``prepare`` the tensors
a program holds before the call, ``run`` one pass, ``work`` what the pass cannot do without and
``exact`` the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16,
          "fp8": torch.float8_e4m3fn}
BYTES = {"f32": 4, "f16": 2, "bf16": 2, "fp8": 1}


# ------------------------------------------------------------------------------------- cases

def _append(name, T, Hq, Hkv, D, bs, dtype, cache, norm=True, rot=None, interleaved=False):
    return {"name": name, "op": "append", "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "bs": bs,
            "dtype": dtype, "cache": cache, "norm": norm, "rot": D if rot is None else rot,
            "interleaved": interleaved}


def _decode(name, S, Hq, Hkv, D, bs, dtype, cache, lo, hi, cap=0.0, alibi=False, window=0,
            starts=False):
    return {"name": name, "op": "decode", "S": S, "Hq": Hq, "Hkv": Hkv, "D": D, "bs": bs,
            "dtype": dtype, "cache": cache, "lo": lo, "hi": hi, "cap": cap, "alibi": alibi,
            "window": window, "starts": starts}


def _chunk(name, S, Hq, Hkv, D, bs, dtype, cache, qlo, qhi, clo, chi, cap=0.0, alibi=False,
           window=0, starts=False, prefix=False):
    return {"name": name, "op": "chunk", "S": S, "Hq": Hq, "Hkv": Hkv, "D": D, "bs": bs,
            "dtype": dtype, "cache": cache, "qlo": qlo, "qhi": qhi, "clo": clo, "chi": chi,
            "cap": cap, "alibi": alibi, "window": window, "starts": starts, "prefix": prefix}


def listed():
    return [
        # one decode step of a small batch: latency
        _append("append_step_8", 8, 32, 8, 128, 16, "bf16", "bf16"),
        # one decode step of a large batch into an 8-bit cache
        _append("append_step_256_fp8", 256, 32, 8, 128, 32, "bf16", "fp8"),
        # a ragged prompt, multi-head, no norm, a quarter of each head rotated in adjacent pairs
        _append("append_prompt_f16_mha", 1003, 32, 32, 64, 16, "f16", "f16", norm=False, rot=16,
                interleaved=True),
        # a step of chunked prefill: 16 chunks of 2048 tokens
        _append("append_chunks_bf16", 32768, 32, 8, 128, 16, "bf16", "bf16"),
        # one short conversation: latency
        _decode("decode_cap_single", 1, 32, 8, 128, 16, "bf16", "bf16", 501, 501, cap=50.0),
        # multi-head attention with a distance bias
        _decode("decode_alibi_mha_f16", 64, 32, 32, 128, 16, "f16", "f16", 512, 2048, alibi=True),
        # a sliding-window layer over an 8-bit cache, capped, many sequences
        _decode("decode_window_fp8", 256, 32, 8, 128, 32, "bf16", "fp8", 64, 8192, cap=30.0,
                window=1024, starts=True),
        # a full-attention layer with capped scores at the size of a serving batch
        _decode("decode_cap_batch128", 128, 32, 8, 128, 16, "bf16", "bf16", 1024, 8192, cap=50.0),
        # several prompts in one short call, documents packed behind each other, prefixes seen whole
        _chunk("chunk_documents_bf16", 6, 32, 8, 128, 16, "bf16", "bf16", 1, 333, 0, 700,
               starts=True, prefix=True),
        # a windowed layer with a distance bias, small heads, ragged prompts
        _chunk("chunk_alibi_window_f16", 4, 16, 16, 64, 8, "f16", "f16", 300, 1500, 0, 2500,
               alibi=True, window=512),
        # a few proposed tokens each on top of long contexts in an 8-bit cache
        _chunk("chunk_verify_fp8", 16, 32, 8, 128, 32, "bf16", "fp8", 1, 8, 2000, 32000, cap=30.0),
        # chunked prefill with capped scores
        _chunk("chunk_cap_bf16", 8, 32, 8, 128, 16, "bf16", "bf16", 2048, 2048, 0, 6144, cap=50.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "decode", "chunk"))
    dtype = rng.choice(("bf16", "f16"))
    bs = rng.choice((8, 16, 32))
    Hkv = rng.choice((1, 2, 4, 8, 16))
    G = rng.choice((1, 2, 4, 8, 16)) if Hkv <= 2 else rng.choice((1, 2, 4))
    Hq = G * Hkv
    cap = rng.choice((0.0, 15.0, 30.0, 50.0))
    if op == "append":
        D = rng.choice((64, 128, 256))
        dtype = rng.choice((dtype, "f32"))
        T = _log(rng, 1, 32768)
        T = max(1, min(T, (1 << 28) // ((Hq + 2 * Hkv) * D * BYTES[dtype] // 2)))
        c = _append("", T, Hq, Hkv, D, bs, dtype, rng.choice((dtype, "fp8")),
                    rng.random() < 0.7, rng.choice((D, D, D // 2, 16)), rng.random() < 0.3)
    elif op == "decode":
        D, cache = rng.choice(((128, dtype), (128, dtype), (64, dtype), (128, "fp8"),
                               (256, dtype), (64, "f32")))
        dtype = "f32" if cache == "f32" else dtype
        S = _log(rng, 1, 256)
        hi = _log(rng, 1, 100000)
        hi = max(1, min(hi, (1 << 30) // (S * Hkv * D)))   # tokens x heads of the padded batch
        c = _decode("", S, Hq, Hkv, D, bs, dtype, cache, max(1, hi // rng.choice((1, 3, 9))), hi,
                    cap, rng.random() < 0.3, rng.choice((0, 0, _log(rng, 1, 4096))),
                    rng.random() < 0.3)
    else:
        D, cache = rng.choice(((128, dtype), (128, dtype), (64, dtype), (128, "fp8")))
        S = _log(rng, 1, 32)
        qhi = _log(rng, 1, 2048)
        chi = _log(rng, 1, 32768)
        qhi = max(1, min(qhi, (1 << 28) // (S * Hq * (chi + qhi))))
        c = _chunk("", S, Hq, Hkv, D, bs, dtype, cache, max(1, qhi // rng.choice((1, 4))), qhi,
                   rng.choice((0, chi)), chi, cap, rng.random() < 0.3,
                   rng.choice((0, 0, _log(rng, 1, 4096))), rng.random() < 0.3, rng.random() < 0.3)
    del c["name"]
    return c


# ------------------------------------------------------------------------------------ inputs

def _randn(shape, name, g, scale=1.0):
    x = torch.randn(shape, generator=g, device="cuda")
    if name == "fp8":
        return (x * (448.0 / 5.0)).clamp_(-448.0, 448.0).to(DTYPES[name])
    return (x * scale).to(DTYPES[name])


def _scales(c):
    return (5.0 / 448.0, 5.0 / 448.0) if c["cache"] == "fp8" else (1.0, 1.0)


def _sizes(c):
    """The cached and the new tokens of every sequence, the same for every seed of a case."""
    g = torch.Generator().manual_seed(c["S"] * 7 + c["bs"])
    if c["op"] == "decode":
        n = torch.randint(c["lo"], c["hi"] + 1, (c["S"],), generator=g)
        return n - 1, torch.ones_like(n)
    new = torch.randint(c["qlo"], c["qhi"] + 1, (c["S"],), generator=g)
    return torch.randint(c["clo"], c["chi"] + 1, (c["S"],), generator=g), new


def _starts(c, n_old, new):
    """A first visible key per new token: documents packed behind each other end somewhere in
    the sequence, and every fifteenth row is padding that sees nothing."""
    seq = torch.repeat_interleave(torch.arange(c["S"]), new)
    row = torch.arange(len(seq)) - torch.repeat_interleave(torch.cumsum(new, 0) - new, new)
    pos = n_old[seq] + row
    length = 97 + 40 * (seq % 5) if c["op"] == "chunk" else 900 + 400 * (seq % 5)
    start = pos // length * length
    if c["op"] == "chunk":
        start = torch.where(torch.arange(len(seq)) % 15 == 7, pos + 1, start)
    return start.to(torch.int32)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.Generator().manual_seed(seed)
    ks, vs = _scales(c)
    st = {"case": c, "k_scale": ks, "v_scale": vs}
    Hq, Hkv, D, bs = c["Hq"], c["Hkv"], c["D"], c["bs"]
    if c["op"] == "append":
        T = c["T"]
        NB = (T + T // 4) // bs + 2
        # the projection's output: queries, keys and values of a token behind each other
        qkv = _randn((T, (Hq + 2 * Hkv) * D), c["dtype"], g)
        st["q"] = qkv[:, :Hq * D].view(T, Hq, D)
        st["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
        st["v"] = qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D)
        st["q_out"] = torch.empty((T, Hq, D), dtype=qkv.dtype, device="cuda")
        st["q_weight"] = st["k_weight"] = None
        if c["norm"]:
            st["q_weight"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(qkv.dtype)
            st["k_weight"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(qkv.dtype)
        P = 65536
        freq = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda") / c["rot"])
        angle = torch.arange(P, dtype=torch.float64, device="cuda")[:, None] * freq
        st["cos_sin"] = torch.cat((angle.cos(), angle.sin()), 1).float().contiguous()
        # chunks of up to 2048 tokens, each at positions of its own
        first = torch.randint(0, P - 2048, ((T + 2047) // 2048,), generator=h)
        t = torch.arange(T)
        st["positions"] = (first[t // 2048] + t % 2048).cuda()
        # slots: blocks in shuffled order, filled from their first token on; a few tokens are padding
        slots = torch.randperm(NB, generator=h)[t // bs] * bs + t % bs
        slots[11::97] = -1
        st["slots"] = slots.cuda()
        st["kept"] = (slots >= 0).nonzero()[:, 0].cuda()
        st["kept_slots"] = slots[slots >= 0].cuda()
        st["key_cache"] = _randn((NB, bs, Hkv, D), c["cache"], g)
        st["value_cache"] = _randn((NB, bs, Hkv, D), c["cache"], g)
        return st
    n_old, new = _sizes(c)
    n = n_old + new
    S, T = c["S"], int(new.sum())
    nblk = (n + bs - 1) // bs
    MB, used = int(nblk.max()), int(nblk.sum())
    NB = used + used // 10 + 1
    ids = torch.randperm(NB, generator=h)
    ends = torch.cumsum(nblk, 0)
    col = torch.arange(MB)[None, :]
    tables = torch.where(col < nblk[:, None], ids[((ends - nblk)[:, None] + col).clamp(max=NB - 1)], -1)
    st["block_tables"] = tables.to(torch.int32).cuda()
    st["context_lens"] = n.to(torch.int32).cuda()
    st["lens_host"], st["max_ctx"], st["max_new"] = n.to(torch.int32), int(n.max()), int(new.max())
    st["query_start"] = torch.cat((torch.zeros(1, dtype=torch.int64), torch.cumsum(new, 0))).to(torch.int32).cuda()
    seq = torch.repeat_interleave(torch.arange(S), new)
    row = torch.arange(T) - torch.repeat_interleave(torch.cumsum(new, 0) - new, new)
    st["row_seq"], st["row_at"] = seq.cuda(), row.cuda()
    st["q"] = _randn((T, Hq, D), c["dtype"], g, 3.0)
    st["key_cache"] = _randn((NB, bs, Hkv, D), c["cache"], g)
    st["value_cache"] = _randn((NB, bs, Hkv, D), c["cache"], g)
    st["out"] = torch.empty_like(st["q"])
    st["scale"] = 1.0 / math.sqrt(D)
    st["slopes"] = None
    if c["alibi"]:
        st["slopes"] = torch.exp2(-8.0 * (torch.arange(Hq, device="cuda") + 1) / Hq).float()
    st["key_start"] = _starts(c, n_old, new).cuda() if c["starts"] else None
    st["prefix_lens"] = None
    if c.get("prefix"):
        st["prefix_lens"] = (n * (torch.arange(S) % 3) // 3).to(torch.int32).cuda()
    return st


# -------------------------------------------------------------------------------------- runs

def run(state):
    op = state["case"]["op"]
    if op == "append":
        return _own_append(state) if own else _plain_append(state)
    if own:
        return _own_decode(state) if op == "decode" else _own_chunk(state)
    return _plain_attention(state)


def _own_append(st):
    import paged_kv_cache_338_b200 as pa
    pa.pa_norm_rope_append(st["q_out"], st["q"], st["k"], st["v"], st["q_weight"], st["k_weight"],
                           1e-6, st["cos_sin"], st["positions"], st["key_cache"],
                           st["value_cache"], st["slots"],
                           interleaved=st["case"]["interleaved"], k_scale=st["k_scale"],
                           v_scale=st["v_scale"])
    return {"q": st["q_out"], "key_cache": st["key_cache"], "value_cache": st["value_cache"]}


def _own_decode(st):
    import paged_kv_cache_338_b200 as pa
    c = st["case"]
    if "partition" not in st:               # a program's plan and workspace, made once
        lens = st["lens_host"]
        if c["window"]:
            lens = lens.clamp(max=c["window"])
        st["partition"] = pa.pa_decode_suggest_partition(c["Hkv"], c["bs"], lens)
        nbytes = pa.pa_decode_scored_workspace_size(c["S"], c["Hq"], c["D"], c["bs"], st["max_ctx"],
                                                    c["window"], st["partition"])
        st["workspace"] = torch.empty(max(nbytes, 16), dtype=torch.uint8, device="cuda")
    pa.pa_decode_scored(st["out"], st["q"], st["key_cache"], st["value_cache"], st["block_tables"],
                        st["context_lens"], st["max_ctx"], st["scale"], softcap=c["cap"],
                        slopes=st["slopes"], window=c["window"], key_start=st["key_start"],
                        k_scale=st["k_scale"], v_scale=st["v_scale"], partition=st["partition"],
                        workspace=st["workspace"])
    return st["out"]


def _own_chunk(st):
    import paged_kv_cache_338_b200 as pa
    c = st["case"]
    if "partition" not in st:               # a program's plan and workspace, made once
        st["partition"] = pa.pa_prefill_scored_suggest_partition(
            c["S"], c["Hq"], c["Hkv"], st["max_new"], st["max_ctx"], c["window"])
        nbytes = pa.pa_prefill_scored_workspace_size(
            c["S"], st["q"].shape[0], c["Hq"], c["D"], st["max_new"], st["max_ctx"], c["window"],
            st["partition"])
        st["workspace"] = torch.empty(max(nbytes, 16), dtype=torch.uint8, device="cuda")
    pa.pa_prefill_scored(st["out"], st["q"], st["key_cache"], st["value_cache"],
                         st["block_tables"], st["context_lens"], st["query_start"], st["max_new"],
                         st["max_ctx"], st["scale"], softcap=c["cap"], slopes=st["slopes"],
                         window=c["window"], key_start=st["key_start"],
                         prefix_lens=st["prefix_lens"], k_scale=st["k_scale"],
                         v_scale=st["v_scale"], partition=st["partition"],
                         workspace=st["workspace"])
    return st["out"]


def _plain_append(st):
    c = st["case"]
    r = c["rot"]
    table = st["cos_sin"][st["positions"]][:, None, :]
    cos, sin = table[..., :r // 2], table[..., r // 2:]

    def head(x, w):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w.float()
        a, b = (y[..., 0:r:2], y[..., 1:r:2]) if c["interleaved"] else (y[..., :r // 2], y[..., r // 2:r])
        a, b = a * cos - b * sin, b * cos + a * sin
        turned = torch.stack((a, b), -1).flatten(-2) if c["interleaved"] else torch.cat((a, b), -1)
        return torch.cat((turned, y[..., r:]), -1)

    def write(cache, x, scale):
        rows = x[st["kept"]]
        if c["cache"] == "fp8":
            rows = (rows / scale).clamp(-448.0, 448.0)
        raw = cache.view(torch.uint8 if c["cache"] == "fp8" else cache.dtype)
        raw.view(-1, c["Hkv"], c["D"])[st["kept_slots"]] = rows.to(cache.dtype).view(raw.dtype)

    st["q_out"].copy_(head(st["q"], st["q_weight"]))
    write(st["key_cache"], head(st["k"], st["k_weight"]), st["k_scale"])
    write(st["value_cache"], st["v"].float(), st["v_scale"])
    return {"q": st["q_out"], "key_cache": st["key_cache"], "value_cache": st["value_cache"]}


def _gathered(cache, tables, scale, dtype):
    """[S, Hkv, tokens, D]: every sequence's rows in order, through its table."""
    raw = cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache
    x = raw[tables.clamp(min=0).long()].view(cache.dtype).flatten(1, 2).to(dtype)
    return (x * scale if scale != 1.0 else x).transpose(1, 2)


def _plain_attention(st):
    c = st["case"]
    S, Hq, Hkv, D = c["S"], c["Hq"], c["Hkv"], c["D"]
    G, L = Hq // Hkv, st["max_new"]
    k = _gathered(st["key_cache"], st["block_tables"], st["k_scale"], torch.float32)
    v = _gathered(st["value_cache"], st["block_tables"], st["v_scale"], torch.float32)
    N = k.shape[2]
    at, seq = st["row_at"], st["row_seq"]
    q = torch.zeros((S, L, Hq, D), device="cuda")
    q[seq, at] = st["q"].float()
    q = q.view(S, L, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(S, Hkv, G * L, D)
    z = (q @ k.transpose(-1, -2)).view(S, Hkv, G, L, N).mul_(st["scale"])
    if c["cap"]:
        z.div_(c["cap"]).tanh_().mul_(c["cap"])
    new = (st["query_start"][1:] - st["query_start"][:-1]).long()
    n = st["context_lens"].long()
    i = torch.arange(N, device="cuda")
    pos = (n - new)[:, None] + torch.arange(L, device="cuda")
    if st["slopes"] is not None:
        far = (i - pos[:, :, None]).abs().float()
        z.sub_(st["slopes"].view(1, Hkv, G, 1, 1) * far[:, None, None])
    lo, hi = torch.zeros_like(pos), pos
    if c["window"]:
        lo = pos - c["window"] + 1
    if st["key_start"] is not None:
        start = torch.zeros_like(pos)
        start[seq, at] = st["key_start"].long()
        lo = torch.maximum(lo, start)
    if st["prefix_lens"] is not None:
        hi = torch.maximum(pos, st["prefix_lens"].long()[:, None] - 1)
    seen = (i >= lo[..., None]) & (i <= hi[..., None]) & (i < n[:, None, None])
    z.masked_fill_(~seen[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    p = z.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True).view(S, Hkv, G * L, 1)
    o = p.view(S, Hkv, G * L, N) @ v
    o = torch.where(total == 0, 0.0, o / total).view(S, Hkv, G, L, D)
    st["out"].copy_(o.permute(0, 3, 1, 2, 4).reshape(S, L, Hq, D)[seq, at])
    return st["out"]


# -------------------------------------------------------------------------------------- work

def work(case):
    c = case
    e, ec, D, Hq, Hkv = BYTES[c["dtype"]], BYTES[c["cache"]], c["D"], c["Hq"], c["Hkv"]
    if c["op"] == "append":
        T = c["T"]
        row = 2 * Hq * D * e + 2 * Hkv * D * (e + ec) + (4 * c["rot"] if c["rot"] else 0) + 16
        return {"bytes": T * row, "flops": T * (Hq + Hkv) * D * 8}
    n_old, new = _sizes(c)
    seq = torch.repeat_interleave(torch.arange(c["S"]), new)
    row = torch.arange(len(seq)) - torch.repeat_interleave(torch.cumsum(new, 0) - new, new)
    pos, n = n_old[seq] + row, (n_old + new)[seq]
    lo, hi = torch.zeros_like(pos), pos.clone()
    if c["window"]:
        lo = torch.maximum(lo, pos - c["window"] + 1)
    if c["starts"]:
        lo = torch.maximum(lo, _starts(c, n_old, new).long())
    if c.get("prefix"):
        hi = torch.maximum(hi, ((n_old + new) * (torch.arange(c["S"]) % 3) // 3)[seq] - 1)
    hi = torch.minimum(hi, n - 1)
    pairs = int((hi - lo + 1).clamp(min=0).sum())
    # keys of a sequence that at least one of its rows sees (the rows' ranges run into each other)
    some = hi >= lo
    first = torch.full((c["S"],), 1 << 40).scatter_reduce(0, seq[some], lo[some], "amin")
    last = torch.full((c["S"],), -1).scatter_reduce(0, seq[some], hi[some], "amax")
    keys = int((last - first + 1).clamp(min=0).sum())
    return {"bytes": keys * 2 * Hkv * D * ec + 2 * len(seq) * Hq * D * e, "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------------------------------- exact

def exact(case, seed):
    st = prepare(case, seed)
    return _exact_append(st) if case["op"] == "append" else _exact_attention(st)


def _exact_append(st):
    c = st["case"]
    T, D, r, half = c["T"], c["D"], c["rot"], c["rot"] // 2
    j = torch.arange(half, device="cuda")
    first, second = (2 * j, 2 * j + 1) if c["interleaved"] else (j, j + half)
    turn = st["cos_sin"].double()[st["positions"]]
    turn = torch.complex(turn[:, :half], turn[:, half:])[:, None, :]

    def head(x, w):
        y = x.double()
        if w is not None:
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / D + 1e-6) * w.double()
        z = torch.complex(y[..., first], y[..., second]) * turn
        y = y.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    out = {"q": head(st["q"], st["q_weight"])}
    for name, x, s in (("key_cache", head(st["k"], st["k_weight"]), st["k_scale"]),
                       ("value_cache", st["v"].double(), st["v_scale"])):
        x = (x / torch.tensor(s, dtype=torch.float32).double().item()).clamp(-448, 448) if c["cache"] == "fp8" else x
        rows = st[name].double().view(-1, c["Hkv"], D)
        rows[st["kept_slots"]] = x[st["kept"]]
        out[name] = rows.view(st[name].shape)
    return out


def _exact_attention(st):
    """One sequence and kv head at a time; every new token's visible keys by their indices."""
    c = st["case"]
    G, D = c["Hq"] // c["Hkv"], c["D"]
    qs, lens = st["query_start"].tolist(), st["lens_host"].tolist()
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for s in range(c["S"]):
        a, b, n = qs[s], qs[s + 1], lens[s]
        blocks = st["block_tables"][s, :(n + c["bs"] - 1) // c["bs"]].long()
        k, v = (x.view(torch.uint8)[blocks].view(x.dtype).reshape(-1, c["Hkv"], D)[:n].double() * f
                if c["cache"] == "fp8" else x[blocks].reshape(-1, c["Hkv"], D)[:n].double()
                for x, f in ((st["key_cache"], st["k_scale"]), (st["value_cache"], st["v_scale"])))
        i = torch.arange(n, device="cuda")
        p = torch.arange(n - (b - a), n, device="cuda")[:, None]
        hidden = i > p
        if st["prefix_lens"] is not None:
            hidden &= i >= st["prefix_lens"][s]
        if c["window"]:
            hidden |= p - i >= c["window"]
        if st["key_start"] is not None:
            hidden |= i < st["key_start"][a:b, None]
        for h in range(c["Hq"]):
            z = st["scale"] * (st["q"][a:b, h].double() @ k[:, h // G].T)
            if c["cap"]:
                z = c["cap"] * torch.tanh(z / c["cap"])
            if st["slopes"] is not None:
                z = z - st["slopes"][h].double() * (p - i).abs()
            z = z.masked_fill(hidden, -math.inf)
            w = torch.nan_to_num(torch.softmax(z, -1), nan=0.0)
            out[a:b, h] = w @ v[:, h // G]
    return out
