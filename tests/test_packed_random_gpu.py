"""Attention over packed sequences, rotation and append on shapes drawn at random, against the 64-bit restatements."""

import math
import random

import pytest

import packed_ref as R
import rotary_ref as Y

pytestmark = pytest.mark.gpu


def draw(rng):
    d = rng.choice((64, 96, 128, 192, 256, 384))
    G = rng.choice((1, 1, 2, 3, 4, 5, 6, 7, 8, 12, 16, 32))
    Hkv = rng.choice((1, 1, 2, 3, 4, 8)) if G < 8 else rng.choice((1, 1, 2))
    B = rng.choice((1, 1, 2, 3, 5, 9, 17, 32, 33, 260, 2100))
    if B > 33:  # (the reference goes sequence by sequence and head by head)
        G, Hkv = rng.choice((1, 2)), 1
    longest = int(2 ** rng.uniform(0, 11 if B < 10 else 9 if B < 80 else 4))
    lengths = [rng.choice((0, 1, longest, rng.randint(0, longest), 64 * rng.randint(0, longest // 64 + 1))) for _ in range(B)]
    while sum(lengths) * G * Hkv * d > 2e7:
        lengths[rng.randrange(B)] //= 2
    return dict(d=d, H=G * Hkv, Hkv=Hkv, lengths=lengths, lead=rng.choice((0, 0, 3, 70)), tail=rng.choice((0, 1, 90)),
                causal=rng.random() < 0.6, scale=None if rng.random() < 0.7 else 10 ** rng.uniform(-3, 0.3), pad=rng.choice((0, 0, 8, 24)),
                heads_first=rng.random() < 0.2, dirty=rng.random() < 0.5, turned=32 * rng.randint(0, d // 32),
                interleaved=rng.random() < 0.5, positions=rng.choice((1, 7, 500)), weights=[rng.random() < 0.7 for _ in range(2)],
                page=rng.choice((16, 32, 64, 128)))


@pytest.mark.parametrize("seed", range(48))
def test_random_shapes(seed):
    import torch
    from tiled_attention_tmem_gb300 import api
    c = draw(random.Random(seed))
    what = str({n: (x[:12] if n == "lengths" else x) for n, x in c.items()})
    d, H, Hkv = c["d"], c["H"], c["Hkv"]
    host = [c["lead"]]
    for n in c["lengths"]:
        host.append(host[-1] + n)
    T = host[-1] + c["tail"]
    if T == 0:
        T = host[-1] + 5
    g = torch.Generator("cuda:0").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda:0").to(torch.bfloat16)

    def full(like, value):
        return torch.full(like.shape, value, device="cuda:0").to(torch.bfloat16)

    x = normal(T, H + 2 * Hkv, d + c["pad"])
    q, k, v = x[:, :H, :d], x[:, H:H + Hkv, :d], x[:, H + Hkv:, :d]
    if c["heads_first"]:
        q, k, v = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v))
    raw_q, raw_k, raw_v = (t.clone() for t in (q, k, v))
    inside = torch.zeros(T, dtype=torch.bool, device="cuda:0")
    inside[host[0]:host[-1]] = True
    if c["dirty"]:
        for t in (q, k, v):
            t[~inside] = math.nan
    cu = torch.tensor(host, dtype=torch.int32, device="cuda:0")
    do, scale = normal(T, H, d), d ** -0.5 if c["scale"] is None else c["scale"]
    o, lse = api.packed_attention_forward(q, k, v, cu, c["scale"], c["causal"], out=full(q, 3.0),
                                          lse=torch.full((T, H), 3.0, device="cuda:0"))
    api.check_device_error()
    r = R.attend(q, k, v, host, scale, c["causal"], do)
    R.check_forward(o, lse, r, d, what)
    assert bool((o[~inside] == 3).all()) and bool((lse[~inside] == 3).all()), what
    for variant in (5, 7) if d <= 128 else (7,):
        grads = [full(t, 5.0) for t in (q, k, v)]
        api.packed_attention_backward(q, k, v, o, do, lse, cu, c["scale"], c["causal"], variant=variant, grads=grads)
        api.check_device_error()
        assert not any(bool(t[~inside].any()) for t in grads), what
        R.check_backward(grads, r, f"{what} variant={variant}")

    # Norms, rotation and the append of the same rows.
    rotary = Y.table(c["positions"], c["turned"], device="cuda:0")
    pos = torch.randint(-1, c["positions"] + 1, (T,), generator=g, device="cuda:0", dtype=torch.int32)
    w = [(1 + 0.3 * torch.randn(d, generator=g, device="cuda:0")).to(torch.bfloat16) if one else None for one in c["weights"]]
    mine, how = Y.live(pos, rotary), (1e-5, c["interleaved"])
    y = api.qk_norm_rope(raw_q, raw_k, rotary, pos, *w, *how, out=(full(q, 7.0), full(k, 7.0)))
    dy = normal(T, H, d), normal(T, Hkv, d)
    back = api.qk_norm_rope_backward(*dy, raw_q, raw_k, rotary, pos, *w, *how)
    for i, t in enumerate((raw_q, raw_k)):
        ref, size = Y.forward(t, w[i], 1e-5, rotary, pos, c["interleaved"])
        Y.check(y[i][mine], ref[mine], size[mine], what)
        assert bool((y[i][~mine] == 7).all()), what
        ref, size, ref_w, size_w = Y.backward(dy[i], t, w[i], 1e-5, rotary, pos, c["interleaved"])
        Y.check(back[i], ref, size, what)
        if w[i] is not None:
            Y.check_weight(back[2 + i], ref_w, size_w, T * t.shape[1], what)
    page = c["page"]
    pages = -(-T // page) + 1
    slots = torch.randperm(pages * page, generator=g, device="cuda:0")[:T].contiguous()
    slots[::7] = -1
    one, two = (api.KV4Cache.empty(pages, Hkv, page, d, 2.0 ** -5, 2.0 ** -5) for _ in range(2))
    kept = full(k, 7.0)
    z = api.kv4_append(raw_q, raw_k, raw_v, rotary, pos, slots, one, *w, *how, out=full(q, 7.0), k_out=kept)
    assert torch.equal(z, y[0]) and torch.equal(kept, y[1]), what
    api.kv4_store(y[1], raw_v, torch.where(mine, slots, -1), two)
    assert all(torch.equal(getattr(one, n), getattr(two, n)) for n in ("k_codes", "k_scales", "v_codes", "v_scales")), what
