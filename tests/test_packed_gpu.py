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
