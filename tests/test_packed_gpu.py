"""Attention over packed sequences against the plain 64-bit restatement (packed_ref)."""

import math

import pytest

import packed_ref as R

pytestmark = pytest.mark.gpu

DIMS = (64, 96, 128, 192, 256, 384)


def make(lengths, H, Hkv, d, seed=0, lead=0, tail=0, spread=1.0):
    """q, k, v as slices of a fused projection's rows, and cu; `lead` and `tail` rows of no sequence."""
    import torch
    g = torch.Generator(device="cuda:0").manual_seed(seed)
    T = lead + sum(lengths) + tail
    x = torch.randn((T, H + 2 * Hkv, d), generator=g, device="cuda:0")
    x[:, H:H + Hkv] *= spread
    x = x.to(torch.bfloat16)
    cu = [lead]
    for n in lengths:
        cu.append(cu[-1] + n)
    return x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:], torch.tensor(cu, dtype=torch.int32, device="cuda:0"), cu


def forward(lengths, H, Hkv, d, causal, scale=None, **kw):
    from tiled_attention_tmem_gb300 import api
    q, k, v, cu, host = make(lengths, H, Hkv, d, **kw)
    o, lse = api.packed_attention_forward(q, k, v, cu, scale, causal)
    api.check_device_error()
    r = R.attend(q, k, v, host, d ** -0.5 if scale is None else scale, causal)
    R.check_forward(o, lse, r, d, f"{lengths} {H}/{Hkv} d={d}")


@pytest.mark.parametrize("causal", (True, False))
@pytest.mark.parametrize("d", DIMS)
def test_forward_one_sequence(d, causal):
    forward([1], 1, 1, d, causal)
    forward([2], 2, 1, d, causal)
    forward([300], 4, 2, d, causal)


@pytest.mark.parametrize("d", DIMS)
@pytest.mark.parametrize("H,Hkv", [(1, 1), (4, 4), (8, 2), (3, 1), (14, 2), (5, 1), (32, 1), (24, 2)])
def test_forward_groups_and_ragged_lengths(d, H, Hkv):
    forward([1, 37, 0, 128, 129, 5, 400, 64], H, Hkv, d, True, seed=d + H)
    forward([63, 0, 257, 2], H, Hkv, d, False, seed=d + H + 1, spread=3.0)


def both(lengths, H, Hkv, d, causal, variants=(0, 7), scale=None, **kw):
    """Forward and backward in each form against the reference."""
    import torch
    from tiled_attention_tmem_gb300 import api
    q, k, v, cu, host = make(lengths, H, Hkv, d, **kw)
    g = torch.Generator(device="cuda:0").manual_seed(99)
    do = torch.randn(q.shape, generator=g, device="cuda:0").to(torch.bfloat16)
    what = f"{lengths} {H}/{Hkv} d={d} causal={causal}"
    o, lse = api.packed_attention_forward(q, k, v, cu, scale, causal)
    r = R.attend(q, k, v, host, d ** -0.5 if scale is None else scale, causal, do)
    R.check_forward(o, lse, r, d, what)
    for variant in variants:
        grads = api.packed_attention_backward(q, k, v, o, do, lse, cu, scale, causal, variant=variant)
        api.check_device_error()
        R.check_backward(grads, r, f"{what} variant={variant}")


@pytest.mark.parametrize("causal", (True, False))
@pytest.mark.parametrize("d", DIMS)
def test_backward_one_sequence(d, causal):
    both([2], 1, 1, d, causal)
    both([300], 4, 2, d, causal)


@pytest.mark.parametrize("d", DIMS)
@pytest.mark.parametrize("H,Hkv", [(1, 1), (4, 4), (8, 2), (3, 1), (14, 2), (5, 1), (32, 1), (24, 2)])
def test_backward_groups_and_ragged_lengths(d, H, Hkv):
    both([1, 37, 0, 128, 129, 5, 400, 64], H, Hkv, d, True, seed=d + H)
    both([63, 0, 257, 2], H, Hkv, d, False, seed=d + H + 1, spread=3.0)


@pytest.mark.parametrize("d", DIMS)
@pytest.mark.parametrize("H,Hkv", [(2, 2), (4, 1), (3, 1)])
def test_nothing_of_another_sequence_or_of_no_sequence_reaches_a_result(d, H, Hkv):
    """NaN and infinities in the rows before the first sequence, behind the last and in a whole
    sequence: the others' results are those of clean inputs, and rows of no sequence stay as they were."""
    import torch
    from tiled_attention_tmem_gb300 import api
    lengths, lead, tail, bad = [70, 33, 300, 1, 129], 5, 200, 1
    for causal in (True, False):
        q, k, v, cu, host = make(lengths, H, Hkv, d, seed=d + H, lead=lead, tail=tail)
        do = torch.randn(q.shape, generator=torch.Generator("cuda:0").manual_seed(3), device="cuda:0").to(torch.bfloat16)
        dirty = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda:0")
        dirty[:lead], dirty[host[-1]:], dirty[host[bad]:host[bad + 1]] = True, True, True
        poison = [t.clone() for t in (q, k, v, do)]
        for i, t in enumerate(poison):
            t[dirty] = (math.nan, math.inf, -math.inf, math.nan)[i]
        mark = dict(out=torch.full(q.shape, 5.0, device="cuda:0").to(torch.bfloat16),
                    lse=torch.full(q.shape[:2], 5.0, device="cuda:0"))
        o, lse = api.packed_attention_forward(q, k, v, cu, causal=causal)
        o2, lse2 = api.packed_attention_forward(*poison[:3], cu, causal=causal, **mark)
        assert o2 is mark["out"] and lse2 is mark["lse"]
        outside = torch.ones_like(dirty)
        outside[lead:host[-1]] = False
        assert bool((o2[outside] == 5).all()) and bool((lse2[outside] == 5).all())
        assert torch.equal(o2[~dirty], o[~dirty]) and torch.equal(lse2[~dirty], lse[~dirty])
        o2[dirty], lse2[dirty] = math.nan, math.nan
        r = R.attend(q, k, v, host, d ** -0.5, causal, do)
        for variant in (0, 7):
            grads = [torch.full(t.shape, 5.0, device="cuda:0").to(torch.bfloat16) for t in (q, k, v)]
            got = api.packed_attention_backward(*poison[:3], o2, poison[3], lse2, cu, causal=causal, variant=variant,
                                                grads=grads)
            assert all(a is b for a, b in zip(got, grads))
            api.check_device_error()
            assert not any(bool(t[outside].any()) for t in got)
            clean = {n: r[n].clone() for n in r}
            for n in ("dq", "dk", "dv"):
                clean[n][dirty] = math.nan
            R.check_backward(got, clean, f"d={d} {H}/{Hkv} causal={causal} variant={variant}")
