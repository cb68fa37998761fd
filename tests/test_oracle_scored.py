"""The error bound of the modified-score oracle: tight enough that a wrong output fails.

A bound that grows with a key's bias or with the cap, whatever the key weighs, lets any
output pass; these cases pin what it may be."""
import pytest
import torch

import scored_cases as sc


def fails(c, want, out, what):
    with pytest.raises(AssertionError, match=what):
        sc.check(c, out.to(sc.DT[c["dt"]]), what, want)


@pytest.mark.parametrize("prefix", [False, True])
def test_a_steep_slope_leaves_the_bound_alone(prefix):
    """Slope 1e30: the query's own key has all the weight, whatever the others' biases."""
    c = sc.make([700], [20], 4, 4, 128, 16, "bf16", "bf16", alibi=True, seed=4,
                prefix_lens=[710] if prefix else None)
    c["slopes"] = torch.tensor([1e30, 1e-30, -0.01, 0.0])
    want = sc.oracle(c)
    p = 700 + torch.arange(20)
    own = c["vc"][c["tables"][0][p // 16].long(), p % 16, 0].double()
    assert torch.equal(want.out[:, 0], own)
    sc.check(c, want.out.to(torch.bfloat16), "itself", want)
    for head in range(4):
        for wrong in (0.0, 12345.0):
            out = want.out.clone()
            out[:, head] = wrong
            fails(c, want, out, f"head {head} {wrong}")


@pytest.mark.parametrize("mod", [{}, dict(alibi=True), dict(softcap=1e6), dict(softcap=30.0),
                                 dict(softcap=5.0, alibi=True, window=900)])
@pytest.mark.parametrize("dt,most", [("f32", 2.0 ** -10), ("f16", 2.0 ** -8), ("bf16", 2.0 ** -5)])
def test_the_bound_is_small_beside_the_values(dt, most, mod):
    """Relative to sum p |v|: three half steps of the type and the scores' arithmetic."""
    c = sc.make([1499], [1], 8, 2, 128, 16, dt, dt, seed=5, **mod)
    b = sc.oracle(c)
    p_dt = None if dt == "f32" else sc.DT[dt]
    assert (b.tolerance(sc.DT[dt], p_dt, 128) <= most * b.weighted).all()


def test_a_capped_score_is_bounded_by_its_own_size():
    """A score's error of 2^-23 of a cap of 1e6 must not pass for fp32 rounding."""
    c = sc.make([399], [1], 4, 2, 128, 16, "f32", "f32", softcap=1e6, seed=6)
    want = sc.oracle(c)
    g = torch.Generator().manual_seed(1)
    off = dict(c, softcap=0.0)
    z_err = 1e6 * 2.0 ** -23
    # the same attention with one key's score moved by that much: a bias on a head of its own
    assert torch.allclose(sc.oracle(off).out, want.out, atol=1e-6)     # (the cap does nothing here)
    w = want.out * (1 + z_err * torch.randn(want.out.shape, generator=g).double())
    fails(c, want, w, "cap")


def test_infinite_keys_add_nothing_to_the_bound():
    c = sc.make([63], [1], 4, 4, 128, 16, "f32", "f32", softcap=3.0, seed=3)
    c["kc"][int(c["tables"][0, 1]), 3, :, 0] = float("inf")
    c["q"][:, :, 0] = 1.0
    b = sc.oracle(c)
    assert torch.isfinite(b.out).all()
    assert (b.tolerance(torch.float32, None, 128) <= 2.0 ** -10 * b.weighted).all()


def test_subnormal_outputs_round_by_half_their_step():
    c = sc.make([39], [1], 2, 2, 128, 16, "f16", "f16", seed=8)
    c["vc"] = c["vc"] * 2.0 ** -22
    want = sc.oracle(c)
    assert (want.out.abs() < torch.finfo(torch.float16).smallest_normal).all()
    sc.check(c, want.out.to(torch.float16), "rounded", want)
    step = 2.0 ** -24
    fails(c, want, want.out + 2 * step, "off by two steps")
