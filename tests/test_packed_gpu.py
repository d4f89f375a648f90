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


def _do(q, seed=7):
    import torch
    return torch.randn(q.shape, generator=torch.Generator("cuda:0").manual_seed(seed), device="cuda:0").to(torch.bfloat16)


@pytest.mark.parametrize("d", DIMS)
def test_strides_of_every_array(d):
    """Heads first, padded rows, slices of wider arrays: the same results as dense ones."""
    import torch
    from tiled_attention_tmem_gb300 import api
    q, k, v, cu, host = make([50, 140, 3], 6, 3, d, seed=1)
    do = _do(q)
    dense = [t.contiguous() for t in (q, k, v, do)]
    o, lse = api.packed_attention_forward(*dense[:3], cu)
    wide = torch.zeros((q.shape[0], 6, d + 24), dtype=torch.bfloat16, device="cuda:0")

    def first(t):
        return t.transpose(0, 1).contiguous().transpose(0, 1)

    o2, lse2 = api.packed_attention_forward(first(q), k, first(v), cu, out=wide[..., 16:16 + d])
    assert torch.equal(o2, o) and torch.equal(lse2, lse)
    assert not bool(wide[..., :16].any()) and not bool(wide[..., 16 + d:].any())
    ref = api.packed_attention_backward(*dense[:3], o, dense[3], lse, cu, variant=7)
    joint = torch.zeros((q.shape[0], 12, d + 8), dtype=torch.bfloat16, device="cuda:0")
    grads = joint[:, :6, :d], joint[:, 6:9, :d], joint[:, 9:, :d]
    got = api.packed_attention_backward(first(q), first(k), v, o2, first(do), lse, cu, variant=7, grads=grads)
    assert all(torch.equal(a, b) for a, b in zip(got, ref)) and not bool(joint[..., d:].any())


def test_refused_by_the_torch_layer():
    import torch
    from tiled_attention_tmem_gb300 import api
    from tiled_attention_tmem_gb300.binding import FaError
    q, k, v, cu, _ = make([10, 20], 4, 2, 64)
    o, lse = api.packed_attention_forward(q, k, v, cu)

    def refuse(kind, match, *args, f=api.packed_attention_forward, **kw):
        with pytest.raises(kind, match=match):
            f(*args, **kw)

    refuse(ValueError, "tokens and channels", q, k[:-1], v, cu)
    refuse(ValueError, "multiple", q[:, :3], k, v, cu)
    refuse(ValueError, "shape", q, k, v[:, :1], cu)
    refuse(ValueError, "positive", q, k[:, :1].expand(-1, 2, -1), v, cu)
    refuse(ValueError, "channels", q.transpose(1, 2), k, v, cu)
    refuse(ValueError, "cu", q, k, v, cu.long())
    refuse(ValueError, "cu", q, k, v, cu[:0])
    refuse(ValueError, "CUDA", q, k, v, cu.cpu())
    refuse(ValueError, "lse", q, k, v, cu, lse=lse[:, :3])
    refuse(ValueError, "overlap", q, k, v, cu, out=o[:, :1].expand(-1, 4, -1))
    small = torch.empty(16, dtype=torch.uint8, device="cuda:0")
    refuse(ValueError, "workspace", q, k, v, torch.zeros(42, dtype=torch.int32, device="cuda:0"), workspace=small)
    refuse(ValueError, "workspace", q, k, v, cu, workspace=small.float())
    refuse(ValueError, "workspace", q, k, v, o, o, lse, cu, f=api.packed_attention_backward, workspace=small)
    refuse(FaError, "invalid", q, k, v, cu, scale=0.0)
    refuse(FaError, "invalid", q, k, v, cu, scale=1e300)
    refuse(FaError, "aligned", q.as_strided(q.shape, (q.stride(0) + 4, 64, 1)), k, v, cu) if q.stride(0) % 8 == 0 else None
    back = api.packed_attention_backward
    refuse(ValueError, "lse", q, k, v, o, o, lse[:-1], cu, f=back)
    refuse(ValueError, "do", q, k, v, o, o.float(), lse, cu, f=back)
    refuse(ValueError, "grads", q, k, v, o, o, lse, cu, grads=(q, k), f=back)
    refuse(FaError, "invalid", q, k, v, o, o, lse, cu, variant=4, f=back)
    q, k, v, cu, _ = make([10], 4, 2, 192)
    o, lse = api.packed_attention_forward(q, k, v, cu)
    refuse(FaError, "unsupported", q, k, v, o, o, lse, cu, variant=5, f=back)
    q, k, v, cu, _ = make([10], 66, 2, 64)
    refuse(FaError, "unsupported", q, k, v, cu)


def test_calls_without_work():
    import torch
    from tiled_attention_tmem_gb300 import api
    q, k, v, cu, _ = make([5, 6], 4, 2, 64)
    mark = torch.full(q.shape, 3.0, device="cuda:0").to(torch.bfloat16)
    lse = torch.full(q.shape[:2], 3.0, device="cuda:0")
    api.packed_attention_forward(q, k, v, cu[:1], out=mark, lse=lse)  # no sequences
    assert bool((mark == 3).all()) and bool((lse == 3).all())
    grads = api.packed_attention_backward(q, k, v, mark, mark, lse, cu[:1])
    assert not any(bool(t.any()) for t in grads)
    assert api.packed_attention_forward(q[:0], k[:0], v[:0], cu * 0)[0].shape == (0, 4, 64)
    assert api.packed_attention_forward(q[:, :0], k[:, :0], v[:, :0], cu)[1].shape == (11, 0)
    none = api.packed_attention_backward(q[:0], k[:0], v[:0], q[:0], q[:0], lse[:0], cu * 0)
    assert [t.shape[0] for t in none] == [0, 0, 0]
    empty = torch.zeros(9, dtype=torch.int32, device="cuda:0")  # eight sequences of no token
    api.packed_attention_forward(q, k, v, empty, out=mark, lse=lse)
    assert bool((mark == 3).all())
    assert not any(bool(t.any()) for t in api.packed_attention_backward(q, k, v, mark, mark, lse, empty))
    api.check_device_error()


def test_gradients_of_keys_and_values_of_no_queries():
    """kv heads that serve no head: sums over none, zeros in new tensors and in given ones."""
    import torch
    from tiled_attention_tmem_gb300 import api
    q, k, v, cu, _ = make([5, 6], 4, 2, 64)
    none = q[:, :0]
    lse = torch.empty((11, 0), device="cuda:0")
    k_new = torch.full((12, 2, 72), 5.0, device="cuda:0").to(torch.bfloat16)
    given = torch.empty_like(none), k_new[:11, :, :64], torch.full_like(v, 5.0)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    for kw in (dict(grads=given), {}, dict(variant=7, stream=stream.cuda_stream)):
        dq, dk, dv = api.packed_attention_backward(none, k, v, none, none, lse, cu, **kw)
        torch.cuda.synchronize()
        assert dq.shape == (11, 0, 64) and dk.shape == dv.shape == (11, 2, 64)
        assert not bool(dk.any()) and not bool(dv.any())
    assert bool((k_new[11] == 5).all()) and bool((k_new[..., 64:] == 5).all())


def test_sequences_outside_the_tokens_have_none():
    import torch
    from tiled_attention_tmem_gb300 import api
    q, k, v, _, _ = make([40], 4, 2, 128)
    for bad in ([0, 10, 25, 41], [-3, 0, 25, 40], [0, 25, 2 ** 31 - 1], [-2 ** 31, 0, 25], [50, 60], [0, 25, 30, 12, 40]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda:0")
        mark = torch.full(q.shape, 3.0, device="cuda:0").to(torch.bfloat16)
        o, lse = api.packed_attention_forward(q, k, v, cu, out=mark, lse=torch.full(q.shape[:2], 3.0, device="cuda:0"))
        if bad == sorted(bad):
            r = R.attend(q, k, v, bad, 128 ** -0.5, True)
            R.check_forward(o, lse, r, 128, str(bad))
            assert bool((o[torch.isnan(r["lse"][:, 0])] == 3).all())
        for variant in (5, 7):
            api.packed_attention_backward(q, k, v, o, o, lse, cu, variant=variant)  # in bounds, whatever it holds
        api.check_device_error()


@pytest.mark.parametrize("d", (64, 128, 256))
@pytest.mark.parametrize("B", (3, 32, 40, 300, 2100))
def test_no_attention_where_sequences_overlap(d, B):
    """Sequences that overlap (all of the tokens again and again) would be many times the work of the tokens: without
    a plan, and in each way that a plan puts sequences in order, nothing is attended to, and the next call is as ever."""
    import torch
    from tiled_attention_tmem_gb300 import api
    T = 300
    q, k, v, whole, host = make([T], 4, 2, d)
    do = _do(q)
    again = [T * (i & 1) for i in range(B + 1)]
    for bad in (again, [0, 200, 100] + [T] * (B - 2), [0] * (B - 2) + [T, T - 1, T]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda:0")
        held = sum(n for _, n in R.bounds(bad, T))
        assert cu.numel() == B + 1 and held > T
        mark = torch.full(q.shape, 3.0, device="cuda:0").to(torch.bfloat16)
        lse = torch.full(q.shape[:2], 3.0, device="cuda:0")
        for causal in (True, False):
            api.packed_attention_forward(q, k, v, cu, causal=causal, out=mark, lse=lse)
            assert bool((mark == 3).all()) and bool((lse == 3).all())
            for variant in (0, 7):
                api.packed_attention_backward(q, k, v, mark, do, lse, cu, causal=causal, variant=variant)
        api.check_device_error()
    o, lse = api.packed_attention_forward(q, k, v, whole)
    r = R.attend(q, k, v, host, d ** -0.5, True, do)
    R.check_forward(o, lse, r, d)
    R.check_backward(api.packed_attention_backward(q, k, v, o, do, lse, whole), r)


@pytest.mark.parametrize("d,H,Hkv,T", [(64, 4, 2, 90), (128, 4, 1, 1500), (192, 2, 2, 90), (256, 8, 1, 1500), (384, 2, 1, 90)])
def test_gradients_of_rows_of_sequences_that_lie_outside(d, H, Hkv, T):
    """cu that does not decrease, with sequences that begin below 0 or end past T: those have no tokens, their
    rows' gradients are zeros, and the others are those of a call without them."""
    import torch
    from tiled_attention_tmem_gb300 import api
    q, k, v, _, _ = make([T], H, Hkv, d)
    do = _do(q)
    a, b = T // 5, T - T // 4
    for cu, rows in (([-3, a, b], (a, b)), ([0, a, b, T + 1], (0, b)), ([-2 ** 31, -1, a, b, 2 ** 31 - 1], (a, b)),
                     ([-5, T + 2], None), ([T + 1, T + 9], None), ([-9, -1], None), ([-4, 0, T], (0, T)),
                     ([a, b, b, T + 7, T + 7], (a, b))):
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda:0")
        o, lse = api.packed_attention_forward(q, k, v, cu)
        for variant in (5, 7) if d <= 128 else (7,):
            grads = [torch.full(t.shape, 5.0, device="cuda:0").to(torch.bfloat16) for t in (q, k, v)]
            api.packed_attention_backward(q, k, v, o, do, lse, cu, variant=variant, grads=grads)
            api.check_device_error()
            lo, hi = rows or (0, 0)
            assert not any(bool(t[:lo].any()) or bool(t[hi:].any()) for t in grads)
            if rows:
                at = slice(lo, hi)
                host = [x - lo for x in cu.tolist() if lo <= x <= hi]
                r = R.attend(q[at], k[at], v[at], host, d ** -0.5, True, do[at])
                R.check_backward([t[at] for t in grads], r, f"{cu.tolist()} variant={variant}")


@pytest.mark.parametrize("d,B", [(64, 3000), (128, 2048), (256, 2049)])
def test_very_many_sequences(d, B):
    """More than are put in order, and more than a block has threads."""
    import torch
    from tiled_attention_tmem_gb300 import api
    g = torch.Generator().manual_seed(B)
    lengths = torch.randint(0, 6, (B,), generator=g).tolist()
    lengths[B // 2] = 700
    q, k, v, cu, host = make(lengths, 2, 1, d, seed=B)
    do = _do(q)
    o, lse = api.packed_attention_forward(q, k, v, cu)
    grads = api.packed_attention_backward(q, k, v, o, do, lse, cu)
    api.check_device_error()
    some = list(range(0, B, 97)) + [B // 2, B - 1]
    for b in some:  # one sequence at a time against the reference
        at = slice(host[b], host[b + 1])
        n = host[b + 1] - host[b]
        if n:
            r = R.attend(q[at], k[at], v[at], [0, n], d ** -0.5, True, do[at])
            R.check_forward(o[at], lse[at], r, d, f"sequence {b}")
            R.check_backward([t[at] for t in grads], r, f"sequence {b}")


@pytest.mark.parametrize("H,Hkv,d,n", [(4, 1, 128, 5000), (2, 2, 64, 4099), (7, 1, 256, 2500), (2, 1, 384, 2100), (3, 1, 192, 2300)])
def test_long_sequences_beside_short_ones(H, Hkv, d, n):
    both([3, n, 130], H, Hkv, d, True, seed=n, spread=2.0)


def test_scores_of_minus_infinity():
    """A query whose scores are all -inf gets zeros and -inf; one -inf among others weighs nothing."""
    import torch
    from tiled_attention_tmem_gb300 import api
    for d in (64, 256):
        q, k, v, cu, host = make([40, 150], 2, 1, d)
        q, k = q.clone(), k.clone()
        k[..., 0] = k[..., 0].abs() + 0.5
        k[60:70, :, 0] *= -1
        q[5, 0, 0], q[100, 1, 0] = -math.inf, -math.inf  # sequence 0: every score -inf; sequence 1: +inf among them
        o, lse = api.packed_attention_forward(q, k, v, cu)
        assert bool((o[5, 0] == 0).all()) and float(lse[5, 0]) == -math.inf
        assert bool(torch.isnan(o[100, 1]).all())
        q[5, 0, 0], q[100, 1, 0] = 0, 0
        o2, lse2 = api.packed_attention_forward(q, k, v, cu)
        for t in (o, o2):
            t[5, 0], t[100, 1] = 0, 0
        assert torch.equal(o, o2)


def test_offsets_past_32_bits():
    import torch
    from tiled_attention_tmem_gb300 import api
    T, H, Hkv, d, step = 140_000, 4, 2, 64, 16384
    x = torch.empty((T, step), dtype=torch.bfloat16, device="cuda:0")
    lengths = [T - 900, 300, 600]
    host = [0, T - 900, T - 600, T]
    at = slice(T - 900, T)
    x[at, :(H + 2 * Hkv) * d] = torch.randn((900, (H + 2 * Hkv) * d), generator=torch.Generator("cuda:0").manual_seed(5),
                                            device="cuda:0").to(torch.bfloat16)
    x[:T - 900, :(H + 2 * Hkv) * d] = 0
    q, k, v = (x[:, a * d:b * d].unflatten(1, (b - a, d)) for a, b in ((0, H), (H, H + Hkv), (H + Hkv, H + 2 * Hkv)))
    cu = torch.tensor([0, 0, T - 600, T], dtype=torch.int32, device="cuda:0")
    cu[1] = T - 900
    out = torch.empty_strided((T, H, d), (step, d, 1), dtype=torch.bfloat16, device="cuda:0")
    cu[0] = T - 900  # (the first sequence would only cost time: it is left without tokens)
    o, lse = api.packed_attention_forward(q, k, v, cu, out=out)
    do = torch.zeros_like(out)
    do[at] = _do(q[at])
    grads = api.packed_attention_backward(q, k, v, o, do, lse, cu, grads=(
        torch.empty_strided((T, H, d), (step, d, 1), dtype=torch.bfloat16, device="cuda:0"),
        torch.empty((T, Hkv, d), dtype=torch.bfloat16, device="cuda:0"),
        torch.empty((T, Hkv, d), dtype=torch.bfloat16, device="cuda:0")))
    r = R.attend(q[at], k[at], v[at], [0, 300, 900], d ** -0.5, True, do[at])
    R.check_forward(o[at], lse[at], r, d)
    R.check_backward([t[at] for t in grads], r)
    assert not any(bool(t[:T - 900].any()) for t in grads) and len(lengths) + 1 == len(host)


@pytest.mark.parametrize("d", (64, 128, 256))
def test_the_same_bits_every_time(d):
    """The forward and the 7-GEMM backward, whatever order the items are claimed in."""
    import torch
    from tiled_attention_tmem_gb300 import api
    q, k, v, cu, _ = make([900, 3, 411, 700, 64], 8, 2, d, seed=4)
    do = _do(q)
    o, lse = api.packed_attention_forward(q, k, v, cu)
    grads = api.packed_attention_backward(q, k, v, o, do, lse, cu, variant=7)
    for _ in range(3):
        o2, lse2 = api.packed_attention_forward(q, k, v, cu)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        again = api.packed_attention_backward(q, k, v, o, do, lse, cu, variant=7)
        assert all(torch.equal(a, b) for a, b in zip(grads, again))


def test_graphs_with_other_lengths_and_one_workspace():
    """Two captured steps that share their workspaces, replayed in turn after inputs and lengths changed."""
    import torch
    from tiled_attention_tmem_gb300 import api
    steps = []
    ws_f = torch.empty(1 << 20, dtype=torch.uint8, device="cuda:0")
    ws_b = torch.empty(64 << 20, dtype=torch.uint8, device="cuda:0")
    stream = torch.cuda.Stream()
    for H, Hkv, d in ((8, 2, 128), (4, 4, 64)):
        q, k, v, cu, _ = make([100, 200, 50], H, Hkv, d)
        t = [x.contiguous() for x in (q, k, v)] + [_do(q)]
        with torch.cuda.stream(stream):
            for _ in range(2):
                o, lse = api.packed_attention_forward(*t[:3], cu, workspace=ws_f)
                api.packed_attention_backward(*t[:3], o, t[3], lse, cu, workspace=ws_b)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            o, lse = api.packed_attention_forward(*t[:3], cu, workspace=ws_f)
            grads = api.packed_attention_backward(*t[:3], o, t[3], lse, cu, workspace=ws_b)
        steps.append((graph, t, cu, o, lse, grads, d))
    for lengths in ([100, 200, 50], [1, 0, 349], [340, 9, 1]):
        host = [0, lengths[0], lengths[0] + lengths[1], 350]
        for graph, t, cu, o, lse, grads, d in steps:
            cu.copy_(torch.tensor(host, dtype=torch.int32))
            for x in t:
                x.copy_(torch.randn(x.shape, device="cuda:0").to(torch.bfloat16))
            graph.replay()
        torch.cuda.synchronize()
        for graph, t, cu, o, lse, grads, d in steps:
            r = R.attend(*t[:3], host, d ** -0.5, True, t[3])
            R.check_forward(o, lse, r, d, str(lengths))
            R.check_backward(grads, r, str(lengths))


def test_two_streams_at_once_and_a_stream_argument():
    import torch
    from tiled_attention_tmem_gb300 import api
    cases = [make([700, 300], 8, 2, 128, seed=1), make([512, 90, 11], 6, 3, 64, seed=2)]
    ref = [api.packed_attention_forward(*c[:4]) for c in cases]
    grads = [api.packed_attention_backward(*c[:3], *r[:1], r[0], r[1], c[3], variant=7) for c, r in zip(cases, ref)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(5):
        for i, (c, s) in enumerate(zip(cases, streams)):
            o, lse = api.packed_attention_forward(*c[:4], stream=s.cuda_stream)
            got[i].append((o, lse, *api.packed_attention_backward(*c[:3], o, o, lse, c[3], variant=7, stream=s.cuda_stream)))
    torch.cuda.synchronize()
    api.check_device_error()
    for i in range(2):
        for out in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(out, (*ref[i], *grads[i])))


def test_nothing_is_computed_while_the_error_word_is_set():
    import torch
    from tiled_attention_tmem_gb300 import api
    from tiled_attention_tmem_gb300 import binding as b
    q, k, v, cu, _ = make([60, 70], 4, 2, 128)
    o, lse = api.packed_attention_forward(q, k, v, cu)
    st = torch.cuda.current_stream().cuda_stream
    assert b.fa_watchdog_selftest(st) == b.FA_OK
    mark = torch.full(q.shape, 3.0, device="cuda:0").to(torch.bfloat16)
    api.packed_attention_forward(q, k, v, cu, out=mark)
    grads = [torch.full(t.shape, 3.0, device="cuda:0").to(torch.bfloat16) for t in (q, k, v)]
    for variant in (5, 7):
        api.packed_attention_backward(q, k, v, o, o, lse, cu, variant=variant, grads=grads)
    with pytest.raises(b.FaError):
        api.check_device_error()
    assert bool((mark == 3).all()) and all(bool((t == 3).all()) for t in grads)
    o2, _ = api.packed_attention_forward(q, k, v, cu)
    api.check_device_error()
    assert torch.equal(o, o2)


def test_profile_counts_the_kernels():
    from tiled_attention_tmem_gb300 import api
    from tiled_attention_tmem_gb300 import binding as b
    q, k, v, cu, _ = make([60, 70], 4, 2, 128)
    for variant, want in ((5, {"bwd_pre": 1, "bwd_kv5": 1, "bwd_conv": 1}), (7, {"bwd_pre": 1, "bwd_kv7": 1, "bwd_q7": 1})):
        b.fa_profile_start()
        o, lse = api.packed_attention_forward(q, k, v, cu)
        api.packed_attention_backward(q, k, v, o, o, lse, cu, variant=variant)
        counts = {n: c for n, (c, _) in b.fa_profile_stop().items() if c}
        assert counts == {"fwd": 1, **want}
    b.fa_profile_start()
    api.packed_attention_forward(*make([3] * 33, 4, 2, 128)[:4])
    assert {n: c for n, (c, _) in b.fa_profile_stop().items() if c} == {"packed_plan": 1, "fwd": 1}


@pytest.mark.parametrize("d", (64, 96, 128, 192, 256, 384))
def test_forward_with_and_without_a_plan(d):
    """The same sequences among empty ones, so many that their order is made by a kernel of its own: the same bits
    where the tiles are the same ones (at d = 96 and 128 they go by the mean length).  Lengths around a tile of keys, rows of no sequence that hold NaN, entries of cu that are out of range."""
    import torch
    from tiled_attention_tmem_gb300 import api
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    most = 64 * (sms // 2 - 2)  # in two sequences of 4 kv heads: two items an SM, so that an item has two tiles
    for H, Hkv in ((2, 2), (8, 2), (7, 1), (8, 4)):
        for lengths in ([1, 64, 65, 127, 128, 129, 300], [0, 0, 257, 0], [31] * 32, [700, 5]):
            if Hkv == 4:
                lengths = [most - 150 - 3 - 737, 737]
            q, k, v, cu, host = make(lengths, H, Hkv, d, seed=d + len(lengths), lead=3, tail=150)
            for t in (q, k, v):
                t[:3], t[host[-1]:] = math.nan, math.nan
            for bad in (None, -5, q.shape[0] + 1):
                host[-1] = host[-1] if bad is None else bad
                some = torch.tensor(host, dtype=torch.int32, device="cuda:0")
                many = torch.tensor([host[0]] * 40 + host, dtype=torch.int32, device="cuda:0")
                assert b_bytes(some, q, k) == 0 and b_bytes(many, q, k) > 0
                for causal in (True, False):
                    marks = [dict(out=torch.full(q.shape, 5.0, device="cuda:0").to(torch.bfloat16),
                                  lse=torch.full(q.shape[:2], 5.0, device="cuda:0")) for _ in range(2)]
                    api.packed_attention_forward(q, k, v, some, causal=causal, **marks[0])
                    api.packed_attention_forward(q, k, v, many, causal=causal, **marks[1])
                    api.check_device_error()
                    if d in (96, 128):
                        r = R.attend(q, k, v, host if bad is None else host[:-1], d ** -0.5, causal)
                        for m in marks:
                            R.check_forward(m["out"], m["lse"], r, d, f"{lengths} {H}/{Hkv} {bad} {causal}")
                    else:
                        assert all(torch.equal(marks[0][n], marks[1][n]) for n in ("out", "lse"))
                    assert not bool(torch.isnan(marks[0]["out"]).any())
                    assert bool((marks[0]["out"][:3] == 5).all()) and bool((marks[0]["lse"][-150:] == 5).all())


@pytest.mark.parametrize("d", (64, 96, 128))
def test_items_of_two_tiles_end_where_their_sequence_does(d):
    """NaN around the sequences and in one of them, where an item holds two query tiles."""
    import torch
    from tiled_attention_tmem_gb300 import api
    q, k, v, cu, host = make([1900, 37, 661, 100], 16, 2, d, seed=d, lead=2, tail=130)
    dirty = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda:0")
    dirty[:2], dirty[host[-1]:], dirty[host[1]:host[2]] = True, True, True
    poison = [t.clone() for t in (q, k, v)]
    for t in poison:
        t[dirty] = math.nan
    for causal in (True, False):
        o, lse = api.packed_attention_forward(q, k, v, cu, causal=causal)
        o2, lse2 = api.packed_attention_forward(*poison, cu, causal=causal)
        api.check_device_error()
        assert torch.equal(o[~dirty], o2[~dirty]) and torch.equal(lse[~dirty], lse2[~dirty])


@pytest.mark.parametrize("d", (64, 96, 128))
@pytest.mark.parametrize("causal", (True, False))
@pytest.mark.parametrize("lengths", ([2900, 1500, 37, 2200], [1400, 1100, 1270, 1], [640, 641, 639, 200, 900], [320, 300, 350, 290, 7], [170, 150, 160]))
def test_forward_on_both_sides_of_the_choice_of_tiles(lengths, causal, d):
    """Mean lengths around those at which the tiles change, many items a multiprocessor, NaN between two of the
    sequences; and the same sequences behind so many empty ones that the mean takes the other tiles."""
    import torch
    from tiled_attention_tmem_gb300 import api
    q, k, v, cu, host = make(lengths, 16, 4, d, seed=sum(lengths), spread=1.5)
    r = R.attend(q, k, v, host, d ** -0.5, causal)
    dirty = slice(host[1], host[2])
    poison = [t.clone() for t in (q, k, v)]
    for t in poison:
        t[dirty] = math.nan
    for before in (0, 40 * len(lengths)):
        many = torch.tensor([0] * before + host, dtype=torch.int32, device="cuda:0")
        o, lse = api.packed_attention_forward(q, k, v, many, causal=causal)
        api.check_device_error()
        R.check_forward(o, lse, r, d, f"{lengths} d={d} {before}")
        o2, lse2 = api.packed_attention_forward(*poison, many, causal=causal)
        api.check_device_error()
        for got, want in ((o2, o), (lse2, lse)):
            got[dirty] = want[dirty]
            assert torch.equal(got, want)


@pytest.mark.parametrize("causal", (True, False))
@pytest.mark.parametrize("d", (96, 128))
@pytest.mark.parametrize("H,Hkv,lengths", [(16, 4, [1504, 1473, 2900, 20, 2200, 1505]), (7, 1, [2900, 1501, 36, 2200, 19]),
                                           (8, 8, [1500, 1281, 100, 1408, 1200])])
def test_forward_in_items_of_two_tiles(H, Hkv, lengths, d, causal):
    """Mean lengths and items a multiprocessor well above those where items of two query tiles begin (packed_fwd.cu:
    two_ctas), with the second tile full, of one token and empty; rows of no sequence and one of the sequences hold NaN.  Behind many empty sequences
    the same ones run in items of one tile: other bits, so these were of two."""
    import torch
    from tiled_attention_tmem_gb300 import api
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert sum(lengths) / len(lengths) > 1.1 * 960 and sum(lengths) // (128 // (H // Hkv)) * Hkv > 2.1 * sms
    q, k, v, cu, host = make(lengths, H, Hkv, d, seed=H + d, lead=2, tail=130, spread=1.5)
    r = R.attend(q, k, v, host, d ** -0.5, causal)
    dirty = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda:0")
    dirty[:2], dirty[host[-1]:], dirty[host[2]:host[3]] = True, True, True
    poison = [t.clone() for t in (q, k, v)]
    for t in poison:
        t[dirty] = math.nan
    many = torch.tensor([2] * (40 * len(lengths)) + host, dtype=torch.int32, device="cuda:0")
    mine = ~torch.isnan(r["lse"][:, 0])
    got = []
    for some in (cu, many):
        o, lse = api.packed_attention_forward(q, k, v, some, causal=causal)
        o2, lse2 = api.packed_attention_forward(*poison, some, causal=causal)
        api.check_device_error()
        R.check_forward(o, lse, r, d, f"{lengths} {H}/{Hkv} d={d}")
        assert torch.equal(o[~dirty], o2[~dirty]) and torch.equal(lse[~dirty], lse2[~dirty])
        got.append(o[mine])
    assert not torch.equal(*got)


def b_bytes(cu, q, k):
    from tiled_attention_tmem_gb300 import api
    return api.packed_forward_workspace_bytes(cu.numel() - 1, q.shape[0], q.shape[1], k.shape[1], q.shape[2])


# ------------------------------------------------------------------ as they are used together

def test_a_training_step_through_all_of_them():
    """Norms and rotation, attention, and both gradients: each stage against the reference on what it was given."""
    import torch
    import rotary_ref as Y
    from tiled_attention_tmem_gb300 import api
    H, Hkv, d, lengths = 8, 2, 128, [90, 1, 260, 33]
    q, k, v, cu, host = make(lengths, H, Hkv, d, seed=9, tail=12)
    g = torch.Generator("cuda:0").manual_seed(10)
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=g, device="cuda:0")).to(torch.bfloat16) for _ in range(2))
    rotary = Y.table(512, d, device="cuda:0")
    pos = torch.full((q.shape[0],), -1, dtype=torch.int32, device="cuda:0")
    for a, n in zip(host, lengths):
        pos[a:a + n] = torch.arange(n, device="cuda:0", dtype=torch.int32)
    do = _do(q)
    tq, tk = api.qk_norm_rope(q, k, rotary, pos, wq, wk)
    o, lse = api.packed_attention_forward(tq, tk, v, cu)
    dtq, dtk, dv = api.packed_attention_backward(tq, tk, v, o, do, lse, cu)
    dq, dk, dwq, dwk = api.qk_norm_rope_backward(dtq, dtk, q, k, rotary, pos, wq, wk)
    api.check_device_error()
    mine = pos >= 0
    for y, x, w in ((tq, q, wq), (tk, k, wk)):
        ref, size = Y.forward(x, w, 1e-6, rotary, pos, False)
        Y.check(y[mine], ref[mine], size[mine])
    r = R.attend(tq, tk, v, host, d ** -0.5, True, do)
    R.check_forward(o, lse, r, d)
    R.check_backward((dtq, dtk, dv), r)
    for dx, dw, dy, x, w in ((dq, dwq, dtq, q, wq), (dk, dwk, dtk, k, wk)):
        ref, size, ref_w, size_w = Y.backward(dy, x, w, 1e-6, rotary, pos, False)
        Y.check(dx, ref, size)
        Y.check_weight(dw, ref_w, size_w, x.shape[0] * x.shape[1])
    assert not bool(dq[~mine].any()) and not bool(dv[~mine].any())


def test_serving_prompts_then_steps():
    """Pages, append, attention over the prompts' own rows, then decoding steps over the 4-bit cache."""
    import torch
    import rotary_ref as Y
    from tiled_attention_tmem_gb300 import api
    H, Hkv, d, page = 8, 2, 128, 16
    i32 = dict(dtype=torch.int32, device="cuda:0")
    cache = api.KV4Cache.empty(64, Hkv, page, d, 2.0 ** -6, 2.0 ** -6, device="cuda:0")
    table, held = torch.full((3, 16), -1, **i32), torch.zeros(3, **i32)
    free, count = torch.arange(64, **i32), torch.full((1,), 64, **i32)
    rotary = Y.table(1024, d, device="cuda:0")
    g = torch.Generator("cuda:0").manual_seed(3)
    for new in ([70, 5, 130], [1, 1, 1], [1, 1, 1]):
        T = sum(new)
        x = torch.randn((T, H + 2 * Hkv, d), generator=g, device="cuda:0").to(torch.bfloat16)
        q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
        before = held.tolist()
        pos = torch.cat([torch.arange(b, b + n, **i32) for b, n in zip(before, new)])
        slots, cu, held, count = api.page_grow(held, torch.tensor(new, **i32), table, free, count, page, T)
        turned = torch.empty_like(k)
        tq = api.kv4_append(q, k, v, rotary, pos, slots, cache, k_out=turned)
        if T > 3:  # prompts: their own rows, not yet rounded to 4 bits
            o, lse = api.packed_attention_forward(tq, turned, v, cu)
            r = R.attend(tq, turned, v, cu.tolist(), d ** -0.5, True)
            R.check_forward(o, lse, r, d)
            continue
        o, lse = api.kv4_attention(tq, cache, table, held, cu, max_q=1)
        for b, n in enumerate(held.tolist()):
            at, _ = api.page_slots(torch.zeros(1, **i32), held[b:b + 1].contiguous(), table[b:b + 1].contiguous(), page, n)
            kk, vv = (t.double().repeat_interleave(H // Hkv, 1) for t in api.kv4_load(at, cache))
            s = torch.einsum("hd,khd->hk", tq[b].double(), kk) * d ** -0.5
            ref = torch.einsum("hk,khd->hd", s.softmax(-1), vv)
            # Probabilities to f16, o to bf16: 2^-8 of what is summed bounds both (values are below 4 here).
            assert float((o[b].double() - ref).abs().max()) <= 2.0 ** -8 * 4
    api.check_device_error()


@pytest.mark.parametrize("causal", (True, False))
@pytest.mark.parametrize("d", DIMS)
@pytest.mark.parametrize("H,Hkv,lengths", [(4, 1, [1500, 3]), (2, 2, [1100, 1, 1300]), (7, 1, [900])])
def test_backward_of_few_key_tiles(H, Hkv, lengths, d, causal):
    """Query ranges in parts: fp32 partial sums, parts without query tiles beside short sequences."""
    from tiled_attention_tmem_gb300 import binding as b
    both(lengths, H, Hkv, d, causal, seed=H + d, lead=2, tail=9)
    b.fa_profile_start()
    both(lengths, H, Hkv, d, causal, variants=(0,))
    # Two parts at least where a mean sequence's rows give each 512.
    assert b.fa_profile_stop()["bwd_kvsum"][0] == (sum(lengths) // len(lengths) * (H // Hkv) >= 1024)


@pytest.mark.parametrize("d", (64, 96, 128))
def test_items_of_two_tiles(d):
    """More items than SMs: two query tiles each, the second of them empty at some ends."""
    both([1500, 700, 1500, 64, 1499, 1200, 33], 16, 4, d, True, seed=d, variants=(0,))
    both([1100, 20, 900, 1300, 1], 24, 8, d, False, seed=d, variants=(7,))
