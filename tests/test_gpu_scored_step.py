"""The fused append and the attentions with modified scores as a serving loop uses them
together: the pool makes the tables, prompts come in chunks (append, then
pa_prefill_scored over the cache), then single tokens (append, then pa_decode_scored,
captured into one CUDA graph and replayed with new inputs), then a few proposed tokens
each (pa_prefill_scored with few rows).  A shadow keeps every sequence's rotated keys and
its values in the cache's own rounding; after every call the caches are those rows bit for
bit where they are not recomputed, and the outputs are the oracle's on them."""
import pytest
import torch

import paged_kv_cache_338_b200 as pa
import scored_cases as sc
from oracle import scored

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    pa.pa_device_status(clear=True)
    yield


class Layer:
    def __init__(self, cdt, bs, NB=256, Hq=16, Hkv=4, D=128, window=150, softcap=20.0):
        self.Hq, self.Hkv, self.D, self.bs, self.window, self.softcap = Hq, Hkv, D, bs, window, softcap
        self.g = torch.Generator().manual_seed(bs)
        self.cdt = cdt
        self.ks, self.vs = (0.02, 0.03) if cdt == "fp8" else (1.0, 1.0)
        self.pool = pa.BlockPool(NB, bs)
        z = lambda: torch.full((NB, bs, Hkv, D), float("nan")).to(sc.DT[cdt]).cuda()     # noqa: E731
        self.kc, self.vc = z(), z()
        self.qw, self.kw = ((1 + 0.2 * torch.randn(D, generator=self.g)).bfloat16().cuda() for _ in range(2))
        ang = torch.arange(4096, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, D, 2) / D)
        self.cs = torch.cat((ang.cos(), ang.sin()), 1).float().cuda()
        self.scale = D ** -0.5
        self.seqs = []

    def slots(self, new):
        """Room for the new tokens of every sequence: positions and slots in their order."""
        pos, slots = [], []
        for s, l in zip(self.seqs, new):
            for _ in range(l):
                pos.append(self.pool.seq_len(s))
                slot, src, dst = self.pool.seq_append(s)
                assert src < 0 or src == dst or dst < 0
                slots.append(slot)
        return torch.tensor(pos), torch.tensor(slots)

    def tables(self):
        n = torch.tensor([self.pool.seq_len(s) for s in self.seqs], dtype=torch.int32)
        blocks = [self.pool.seq_blocks(s) for s in self.seqs]
        t = torch.full((len(self.seqs), 64), -1, dtype=torch.int32)
        for i, b in enumerate(blocks):
            t[i, :len(b)] = torch.tensor(b, dtype=torch.int32)
        return t, n

    def project(self, T):
        qkv = torch.randn(T, (self.Hq + 2 * self.Hkv) * self.D, generator=self.g).bfloat16()
        return qkv

    def split(self, qkv):
        T, a, b = len(qkv), self.Hq * self.D, (self.Hq + self.Hkv) * self.D
        return (qkv[:, :a].view(T, self.Hq, self.D), qkv[:, a:b].view(T, self.Hkv, self.D),
                qkv[:, b:].view(T, self.Hkv, self.D))

    def append(self, qkv, pos, slots, q_out):
        q, k, v = self.split(qkv)
        pa.pa_norm_rope_append(q_out, q, k, v, self.qw, self.kw, 1e-6, self.cs, pos, self.kc, self.vc,
                               slots, k_scale=self.ks, v_scale=self.vs)

    def check(self, q_out, qkv, pos, slots, out, qs, tables, lens, decode, what):
        q, k, v = self.split(qkv.cpu())
        cs = self.cs.cpu()
        want, size = scored.norm_rope(q, self.qw.cpu(), 1e-6, 0.0, cs, pos, False)
        tol = 2.0 ** -8 * want.abs() + 2.0 ** -18 * size + 1e-30
        assert ((scored.stored(q_out.cpu()) - want).abs() <= tol).all(), what
        kw, ksz = scored.norm_rope(k, self.kw.cpu(), 1e-6, 0.0, cs, pos, False)
        half = 2.0 ** -4 if self.cdt == "fp8" else 2.0 ** -8
        for cache, x, sz, s in ((self.kc, kw, ksz, self.ks), (self.vc, scored.stored(v), 0 * ksz, self.vs)):
            raw = cache.cpu()
            rows = raw.view(torch.uint8).view(-1, self.Hkv, raw.view(torch.uint8).shape[-1])[slots].view(raw.dtype)
            s32 = float(torch.tensor(s, dtype=torch.float32))
            y = (x / s32).clamp(-448, 448) if self.cdt == "fp8" else x
            step = 2.0 ** -10 if self.cdt == "fp8" else 0.0          # half of E4M3's smallest step
            assert ((scored.stored(rows) - y).abs() <= half * y.abs() + 2.0 ** -18 * sz / s32 + step).all(), what
        c = {"q": q_out.cpu(), "kc": self.kc.cpu(), "vc": self.vc.cpu(), "tables": tables, "lens": lens,
             "qs": qs, "scale": self.scale, "softcap": self.softcap, "slopes": None, "window": self.window,
             "key_start": None, "prefix_lens": None, "k_scale": self.ks, "v_scale": self.vs,
             "decode": decode, "dt": "bf16", "cdt": self.cdt}
        sc.check(c, out, what)

    def chunk(self, new, what):
        T = sum(new)
        pos, slots = self.slots(new)
        tables, lens = self.tables()
        qkv = self.project(T).cuda()
        qs = torch.tensor([0] + list(torch.tensor(new).cumsum(0)), dtype=torch.int32)
        q = torch.empty(T, self.Hq, self.D, dtype=torch.bfloat16, device="cuda")
        out = torch.empty_like(q)
        self.append(qkv, pos.cuda(), slots.cuda(), q)
        mx, mc = max(new), int(lens.max())
        part = pa.pa_prefill_scored_suggest_partition(len(new), self.Hq, self.Hkv, mx, mc, self.window)
        nb = pa.pa_prefill_scored_workspace_size(len(new), T, self.Hq, self.D, mx, mc, self.window, part)
        ws = torch.empty(max(nb, 16), dtype=torch.uint8, device="cuda")
        pa.pa_prefill_scored(out, q, self.kc, self.vc, tables.cuda(), lens.cuda(), qs.cuda(), mx, mc,
                             self.scale, softcap=self.softcap, window=self.window, k_scale=self.ks,
                             v_scale=self.vs, partition=part, workspace=ws)
        self.check(q, qkv, pos, slots, out, qs, tables, lens, False, what)


@pytest.mark.parametrize("cdt,bs", [("bf16", 16), ("fp8", 32)])
def test_a_layer_over_prompts_steps_and_proposals(cdt, bs):
    m = Layer(cdt, bs)
    m.seqs = [m.pool.seq_new() for _ in range(4)]
    m.chunk([200, 1, 77, 130], "first chunk")
    m.chunk([50, 90, 1, 128], "second chunk")
    # single tokens: one graph, new inputs every step
    S, mc = 4, 512
    static = {"qkv": m.project(S).cuda(), "pos": torch.zeros(S, dtype=torch.int64, device="cuda"),
              "slots": torch.full((S,), -1, dtype=torch.int64, device="cuda"),
              "tables": torch.full((S, 64), -1, dtype=torch.int32, device="cuda"),
              "lens": torch.zeros(S, dtype=torch.int32, device="cuda")}
    q = torch.zeros(S, m.Hq, m.D, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    ws = torch.empty(pa.pa_decode_scored_workspace_size(S, m.Hq, m.D, bs, mc, m.window, 64), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        m.append(static["qkv"], static["pos"], static["slots"], q)
        pa.pa_decode_scored(out, q, m.kc, m.vc, static["tables"], static["lens"], mc, m.scale,
                            softcap=m.softcap, window=m.window, k_scale=m.ks, v_scale=m.vs, partition=64,
                            workspace=ws)
    for step in range(6):
        pos, slots = m.slots([1] * S)
        tables, lens = m.tables()
        for k, x in (("qkv", m.project(S)), ("pos", pos), ("slots", slots), ("tables", tables), ("lens", lens)):
            static[k].copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        m.check(q, static["qkv"], pos, slots, out, None, tables, lens, True, f"step {step}")
    # proposals: a few tokens each, on the few-row kernel
    m.chunk([5, 1, 8, 3], "proposals")
    m.chunk([1, 1, 1, 1], "one each")
    assert pa.pa_device_status() == 0
