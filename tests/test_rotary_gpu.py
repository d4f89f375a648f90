"""Norms and rotation of queries and keys, and the rotated append to the 4-bit cache."""

import pytest

import rotary_ref as R

pytestmark = pytest.mark.gpu

DIMS = (64, 96, 128, 192, 256, 384)


def make(T, H, Hkv, d, turned, seed=0, weights=True, positions=512, loose=True, value=False):
    """q, k (and v) as slices of a fused projection's rows, a table, positions of which some are not in it."""
    import torch
    g = torch.Generator(device="cuda:0").manual_seed(seed)
    x = torch.randn((T, H + 2 * Hkv, d), generator=g, device="cuda:0").to(torch.bfloat16)
    pos = torch.randint(0, positions, (T,), generator=g, device="cuda:0", dtype=torch.int32)
    if loose and T > 4:
        pos[1], pos[T // 2], pos[-1] = -1, positions, -2 ** 31
    w = [(1 + 0.3 * torch.randn(d, generator=g, device="cuda:0")).to(torch.bfloat16) if weights else None for _ in range(2)]
    out = (x[:, :H], x[:, H:H + Hkv], R.table(positions, turned, device="cuda:0"), pos, *w)
    return out + (x[:, H + Hkv:],) if value else out


CASES = [(1, 1, 1), (7, 8, 2), (64, 32, 8), (33, 5, 3), (1000, 7, 1), (3000, 12, 4)]


@pytest.mark.parametrize("interleaved", (False, True))
@pytest.mark.parametrize("d", DIMS)
def test_forward_and_backward(d, interleaved):
    import torch
    from tiled_attention_tmem_gb300 import api
    for n, (T, H, Hkv) in enumerate(CASES):
        for weights in (True, False):
            turned = (d, 32, d - 32, 0)[(n + weights) % 4]
            q, k, rotary, pos, wq, wk = make(T, H, Hkv, d, turned, seed=n, weights=weights)
            what = f"T={T} {H}/{Hkv} d={d} turned={turned} weights={weights}"
            mine = R.live(pos, rotary)
            marked = [torch.full(t.shape, 7.0, device="cuda:0").to(torch.bfloat16) for t in (q, k)]
            got = api.qk_norm_rope(q, k, rotary, pos, wq, wk, 1e-5, interleaved, out=marked)
            assert got[0] is marked[0] and got[1] is marked[1]
            for y, x, w in zip(got, (q, k), (wq, wk)):
                ref, size = R.forward(x, w, 1e-5, rotary, pos, interleaved)
                R.check(y[mine], ref[mine], size[mine], what)
                assert bool((y[~mine] == 7).all()), what  # tokens without a position stay as they were
            g = torch.Generator(device="cuda:0").manual_seed(50 + n)
            dq, dk = (torch.randn(t.shape, generator=g, device="cuda:0").to(torch.bfloat16) for t in (q, k))
            back = api.qk_norm_rope_backward(dq, dk, q, k, rotary, pos, wq, wk, 1e-5, interleaved)
            for dx, dw, dy, x, w in zip(back[:2], back[2:], (dq, dk), (q, k), (wq, wk)):
                ref, size, ref_w, size_w = R.backward(dy, x, w, 1e-5, rotary, pos, interleaved)
                R.check(dx, ref, size, what + " gradient")
                assert (dw is None) == (w is None)
                if dw is not None:
                    R.check_weight(dw, ref_w, size_w, T * x.shape[1], what + " weight")
            again = api.qk_norm_rope_backward(dq, dk, q, k, rotary, pos, wq, wk, 1e-5, interleaved)
            assert all(a is b is None or torch.equal(a, b) for a, b in zip(back, again))  # a fixed order
            # In place, both ways.
            q2, k2 = q.clone(), k.clone()
            api.qk_norm_rope(q2, k2, rotary, pos, wq, wk, 1e-5, interleaved, out=(q2, k2))
            assert torch.equal(q2[mine], got[0][mine]) and torch.equal(k2[mine], got[1][mine])
            assert torch.equal(q2[~mine], q[~mine])
            api.qk_norm_rope_backward(dq, dk, q, k, rotary, pos, wq, wk, 1e-5, interleaved, grads=(dq, dk))
            assert torch.equal(dq, back[0]) and torch.equal(dk, back[1])


def test_one_weight_of_two_and_rows_of_zeros():
    import torch
    from tiled_attention_tmem_gb300 import api
    q, k, rotary, pos, wq, wk = make(40, 6, 2, 128, 64, weights=True)
    q = q.clone()
    q[3] = 0
    dq, dk = torch.ones_like(q), torch.ones_like(k)
    for a, b in ((wq, None), (None, wk)):
        y = api.qk_norm_rope(q, k, rotary, pos, a, b)
        back = api.qk_norm_rope_backward(dq, dk, q, k, rotary, pos, a, b)
        mine = R.live(pos, rotary)
        for i, (x, w, dy) in enumerate(((q, a, dq), (k, b, dk))):
            ref, size = R.forward(x, w, 1e-6, rotary, pos, False)
            R.check(y[i][mine], ref[mine], size[mine])
            ref, size, ref_w, size_w = R.backward(dy, x, w, 1e-6, rotary, pos, False)
            R.check(back[i], ref, size)
            assert (back[2 + i] is None) == (w is None)
            if w is not None:
                R.check_weight(back[2 + i], ref_w, size_w, 240)
    # eps = 0: tokens without a position, and steps that are not full, put no NaN into a sum.
    back = api.qk_norm_rope_backward(dq[:, :5], dk, q[:, :5].clone().fill_(1), k, rotary, pos, wq, wk, 0.0)
    assert all(bool(torch.isfinite(t).all()) for t in back)


def test_tokens_without_a_position_beside_weights_that_are_not_finite():
    """Their gradients are zeros all the same, and they put nothing into the weights' sums."""
    import math
    import torch
    from tiled_attention_tmem_gb300 import api
    for d in (64, 96, 384):
        for interleaved in (False, True):
            q, k, rotary, pos, wq, wk = make(40, 3, 2, d, 32, weights=True)
            mine = R.live(pos, rotary)
            ref = api.qk_norm_rope_backward(q, k, q, k, rotary, pos, wq, wk, interleaved=interleaved)
            bad = [wq.clone(), wk.clone()]
            bad[0][3], bad[0][d - 1], bad[1][0] = math.nan, math.inf, -math.inf
            grads = [torch.full(t.shape, 5.0, device="cuda:0").to(torch.bfloat16) for t in (q, k)]
            got = api.qk_norm_rope_backward(q, k, q, k, rotary, pos, *bad, interleaved=interleaved, grads=grads)
            for x, y in zip(got[:2], ref):
                assert not bool(x[~mine].any()) and not bool(torch.isfinite(x[mine]).all()) and bool((y[~mine] == 0).all())
            # The weights' gradients have no weight in them.
            assert torch.equal(got[2], ref[2]) and torch.equal(got[3], ref[3])


def test_far_positions_and_large_magnitudes():
    import torch
    from tiled_attention_tmem_gb300 import api
    q, k, _, _, wq, wk = make(64, 4, 2, 128, 128)
    rotary = R.table(1 << 20, 128, device="cuda:0")
    pos = torch.arange((1 << 20) - 64, 1 << 20, device="cuda:0", dtype=torch.int32)
    for scale in (2.0 ** -60, 1.0, 2.0 ** 60):
        x, z = q * scale, k * scale
        y = api.qk_norm_rope(x, z, rotary, pos, wq, wk, 0.0)
        for got, t, w in zip(y, (x, z), (wq, wk)):
            ref, size = R.forward(t, w, 0.0, rotary, pos, False)
            R.check(got, ref, size, f"scale {scale}")


def test_strides_empty_calls_and_tables_without_rows():
    import torch
    from tiled_attention_tmem_gb300 import api
    q, k, rotary, pos, wq, wk = make(50, 6, 3, 96, 96, loose=False)
    heads_first = q.transpose(0, 1).contiguous().transpose(0, 1)
    one = k[:, :1].expand(-1, 3, -1)  # a broadcast head
    y, z = api.qk_norm_rope(heads_first, one, rotary, pos, wq, wk)
    y2, z2 = api.qk_norm_rope(q.contiguous(), one.contiguous(), rotary, pos, wq, wk)
    assert torch.equal(y, y2) and torch.equal(z, z2)
    wide = torch.zeros((50, 6, 160), dtype=torch.bfloat16, device="cuda:0")
    api.qk_norm_rope(q, k, rotary, pos, wq, wk, out=(wide[..., 8:104], torch.empty_like(k)))
    assert torch.equal(wide[..., 8:104], y2) and not bool(wide[..., :8].any()) and not bool(wide[..., 104:].any())
    # No tokens, no heads, no positions.
    none = api.qk_norm_rope_backward(q[:0], k[:0], q[:0], k[:0], rotary, pos[:0], wq, wk)
    assert none[0].shape == (0, 6, 96) and not bool(none[2].any()) and not bool(none[3].any())
    assert api.qk_norm_rope(q[:0], k[:0], rotary, pos[:0])[0].shape == (0, 6, 96)
    y, z = api.qk_norm_rope(q[:, :0], k, rotary, pos, wq, wk)
    assert y.shape == (50, 0, 96) and torch.equal(z, api.qk_norm_rope(q, k, rotary, pos, wq, wk)[1])
    y, _ = api.qk_norm_rope(q, k, rotary[:0], pos, out=(torch.zeros_like(q), torch.zeros_like(k)))
    assert not bool(y.any())


@pytest.mark.parametrize("d,turned,interleaved", [(64, 64, False), (96, 32, True), (128, 128, False), (128, 64, True), (192, 160, False),
                                                  (256, 256, False), (384, 384, True)])
def test_each_product_and_sum_is_rounded_alone(d, turned, interleaved):
    """Without weights the results are those of fp32 products and sums taken one after the other, bit for bit, and so are the
    gradients and what an append gives.  (Taken together, two of 10^5 results come out otherwise.)"""
    import torch
    from tiled_attention_tmem_gb300 import api
    T, H, Hkv = 3001, 6, 2
    q, k, rotary, pos, _, _, v = make(T, H, Hkv, d, turned, seed=d, weights=False, positions=32768, loose=False, value=True)
    a, b = R.channels(turned, interleaved, "cuda:0")
    row = rotary[pos.long()][:, None]
    c, s = row[..., :turned // 2], row[..., turned // 2:]

    def turn(x, s):
        x = x.float()
        y = x.clone()
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        return y.to(torch.bfloat16)

    want = turn(q, s), turn(k, s)
    got = api.qk_norm_rope(q, k, rotary, pos, interleaved=interleaved)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    back = api.qk_norm_rope_backward(q, k, q, k, rotary, pos, interleaved=interleaved)
    assert torch.equal(back[0], turn(q, -s)) and torch.equal(back[1], turn(k, -s))
    cache, turned_k = api.KV4Cache.empty(-(-T // 16), Hkv, 16, d), torch.empty_like(k)
    y = api.kv4_append(q, k, v, rotary, pos, torch.arange(T, device="cuda:0"), cache, interleaved=interleaved, k_out=turned_k)
    assert torch.equal(y, want[0]) and torch.equal(turned_k, want[1])


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("d", DIMS)
def test_append_is_rotation_then_store(d):
    """The same bits as qk_norm_rope and kv4_store one after the other, in every layout."""
    import torch
    from tiled_attention_tmem_gb300 import api
    for n, (T, H, Hkv, page) in enumerate([(1, 1, 1, 16), (7, 8, 2, 64), (64, 32, 8, 64), (33, 5, 3, 32), (2500, 7, 1, 128),
                                           (1200, 12, 4, 16)]):
        for weights in (True, False):
            turned, interleaved = (d, 32, d - 32, 0)[(n + weights) % 4], bool(n & 1)
            q, k, rotary, pos, wq, wk, v = make(T, H, Hkv, d, turned, seed=n, weights=weights, value=True)
            pages = -(-T // page) + 3
            g = torch.Generator(device="cuda:0").manual_seed(n)
            slots = torch.randperm(pages * page, generator=g, device="cuda:0")[:T].contiguous()
            if T > 6:
                slots[2], slots[3] = -1, pages * page
            one, two = (api.KV4Cache.empty(pages, Hkv, page, d, 2.0 ** -6, 2.0 ** -7) for _ in range(2))
            mark = dict(out=torch.full(q.shape, 7.0, device="cuda:0").to(torch.bfloat16),
                        k_out=torch.full(k.shape, 7.0, device="cuda:0").to(torch.bfloat16))
            y = api.kv4_append(q, k, v, rotary, pos, slots, one, wq, wk, 1e-5, interleaved, **mark)
            assert y is mark["out"]
            ref = api.qk_norm_rope(q, k, rotary, pos, wq, wk, 1e-5, interleaved,
                                   out=tuple(torch.full(t.shape, 7.0, device="cuda:0").to(torch.bfloat16) for t in (q, k)))
            mine = R.live(pos, rotary)
            api.kv4_store(ref[1], v, torch.where(mine, slots, -1), two)
            what = f"T={T} {H}/{Hkv} d={d} turned={turned} weights={weights}"
            assert torch.equal(y, ref[0]) and torch.equal(mark["k_out"], ref[1]), what
            for a in ("k_codes", "k_scales", "v_codes", "v_scales"):
                assert torch.equal(getattr(one, a), getattr(two, a)), f"{what} {a}"
            # Without the keys' own rows, and in place.
            three = api.KV4Cache.empty(pages, Hkv, page, d, 2.0 ** -6, 2.0 ** -7)
            x = q.clone()
            api.kv4_append(x, k, v, rotary, pos, slots, three, wq, wk, 1e-5, interleaved, out=x)
            assert torch.equal(x[mine], y[mine]) and torch.equal(x[~mine], q[~mine])
            assert torch.equal(three.k_codes, one.k_codes) and torch.equal(three.v_codes, one.v_codes)


def test_append_without_queries_tokens_or_pages():
    import torch
    from tiled_attention_tmem_gb300 import api
    q, k, rotary, pos, wq, wk, v = make(40, 4, 2, 128, 128, value=True, loose=False)
    slots = torch.arange(40, device="cuda:0")
    one, two = (api.KV4Cache.empty(4, 2, 16, 128) for _ in range(2))
    api.kv4_append(q, k, v, rotary, pos, slots, one, wq, wk)
    api.kv4_append(q[:, :0], k, v, rotary, pos, slots, two, wq, wk)
    assert torch.equal(one.k_codes, two.k_codes) and torch.equal(one.v_scales, two.v_scales)
    assert api.kv4_append(q[:0], k[:0], v[:0], rotary, pos[:0], slots[:0], one).shape == (0, 4, 128)
    y = api.kv4_append(q, k, v, rotary, pos, slots, api.KV4Cache.empty(0, 2, 16, 128), wq, wk)
    assert torch.equal(y, api.qk_norm_rope(q, k, rotary, pos, wq, wk)[0])


def test_append_in_slots_given_twice_and_two_at_once():
    """A slot given twice ends up with bytes of either token, and no other slot with any; calls on two streams do not meet."""
    import torch
    from tiled_attention_tmem_gb300 import api
    q, k, rotary, pos, wq, wk, v = make(64, 4, 2, 128, 128, value=True, loose=False)
    slots = torch.arange(64, device="cuda:0")
    ref, twice = (api.KV4Cache.empty(8, 2, 16, 128) for _ in range(2))
    y = api.kv4_append(q, k, v, rotary, pos, slots, ref, wq, wk)
    both = slots.clone()
    both[9] = 8
    assert torch.equal(api.kv4_append(q, k, v, rotary, pos, both, twice, wq, wk), y)
    assert not bool(twice.k_codes[0, :, 9].any()) and not bool(twice.k_codes[4:].any())
    for c, r in ((twice.k_codes, ref.k_codes), (twice.v_codes, ref.v_codes)):
        assert torch.equal(c[1:4], r[1:4]) and torch.equal(c[0, :, :8], r[0, :, :8]) and torch.equal(c[0, :, 10:], r[0, :, 10:])
        assert bool(((c[0, :, 8] == r[0, :, 8]) | (c[0, :, 8] == r[0, :, 9])).all())
    # Two streams into one cache, each its own slots.
    cache = api.KV4Cache.empty(8, 2, 16, 128)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, s in enumerate(streams):
            at = slice(i, None, 2)
            api.kv4_append(q[at], k[at], v[at], rotary, pos[at].contiguous(), slots[at].contiguous(), cache, wq, wk,
                           stream=s.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(cache.k_codes, ref.k_codes) and torch.equal(cache.v_scales, ref.v_scales)


def test_offsets_past_32_bits():
    """Arrays of over 2^31 elements and a pool of over 2^32 bytes: the first and the last tokens are those of a short call."""
    import torch
    from tiled_attention_tmem_gb300 import api
    T, n = 530000, 40
    q, k, rotary, pos, wq, wk, v = make(n, 32, 1, 128, 128, value=True, loose=False)
    long = [torch.zeros((T, t.shape[1], 128), dtype=torch.bfloat16, device="cuda:0") for t in (q, k)]
    assert long[0].numel() > 2 ** 31
    at = torch.full((T,), -1, dtype=torch.int32, device="cuda:0")
    for part in (slice(0, n), slice(T - n, T)):
        long[0][part], long[1][part], at[part] = q, k, pos
    short = api.qk_norm_rope(q, k, rotary, pos, wq, wk)
    back = api.qk_norm_rope_backward(q, k, q, k, rotary, pos, wq, wk)
    got = api.qk_norm_rope(*long, rotary, at, wq, wk, out=[t.clone() for t in long])
    grads = api.qk_norm_rope_backward(*long, *long, rotary, at, wq, wk)
    for part in (slice(0, n), slice(T - n, T)):
        assert all(torch.equal(t[part], r) for t, r in zip(got, short))
        assert all(torch.equal(t[part], r) for t, r in zip(grads[:2], back[:2]))
    assert not bool(got[0][n:T - n].any()) and not bool(grads[0][n:T - n].any())
    for dw, x, w in zip(grads[2:], (q, k), (wq, wk)):  # twice the short call's sums
        _, _, ref_w, size_w = R.backward(x, x, w, 1e-6, rotary, pos, False)
        R.check_weight(dw, 2 * ref_w, 2 * size_w, 2 * n * x.shape[1])
    del got, grads, long
    torch.cuda.empty_cache()
    big, small = api.KV4Cache.empty(525000, 1, 128, 128), api.KV4Cache.empty(1, 1, 128, 128)
    assert big.k_codes.numel() > 2 ** 32
    slots = 524990 * 128 + torch.arange(n, device="cuda:0")
    y = api.kv4_append(q, k, v, rotary, pos, slots, big, wq, wk)
    assert torch.equal(y, api.kv4_append(q, k, v, rotary, pos, slots - 524990 * 128, small, wq, wk))
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(big, name)[524990], getattr(small, name)[0])
    assert not bool(big.k_codes[0].any()) and not bool(big.k_codes[524989].any())


# ------------------------------------------------------------------ calls

def test_refused_by_the_torch_layer():
    import torch
    from tiled_attention_tmem_gb300 import api
    from tiled_attention_tmem_gb300.binding import FaError
    q, k, rotary, pos, wq, wk, v = make(40, 4, 2, 128, 64, value=True, loose=False)
    slots = torch.arange(40, device="cuda:0")
    cache = api.KV4Cache.empty(4, 2, 16, 128)
    calls = {"pass": lambda q=q, k=k, t=rotary, p=pos, a=wq, b=wk, **kw: api.qk_norm_rope(q, k, t, p, a, b, **kw),
             "back": lambda q=q, k=k, t=rotary, p=pos, a=wq, b=wk, **kw: api.qk_norm_rope_backward(q, k, q, k, t, p, a, b, **kw),
             "append": lambda q=q, k=k, t=rotary, p=pos, a=wq, b=wk, **kw: api.kv4_append(q, k, v, t, p, slots, cache, a, b, **kw)}
    before = [t.clone() for t in (q, k, cache.k_codes)]

    def refuse(kind, match, only=calls, **kw):
        for name in only:
            with pytest.raises(kind, match=match):
                calls[name](**kw)

    refuse(TypeError, "tensor", q=None, only=("pass", "back"))
    refuse(ValueError, "CUDA", q=q.float())
    refuse(ValueError, "CUDA|cuda", q=q.cpu())
    refuse(ValueError, "tokens and channels", k=k[:-1], only=("pass", "back"))
    refuse(ValueError, "shape", k=k[:-1], only=("append",))
    refuse(ValueError, "shape", q=q[:-1], only=("append",))
    refuse(ValueError, "rotary", t=rotary.double())
    refuse(ValueError, "rotary", t=rotary[:, ::2])
    refuse(ValueError, "rotary", t=rotary[:, :48].contiguous())
    refuse(ValueError, "rotary", t=torch.zeros(8, 160, device="cuda:0"))
    refuse(ValueError, "positions", p=pos.long())
    refuse(ValueError, "positions", p=pos[:-1])
    refuse(ValueError, "q_weight", a=wq.float())
    refuse(ValueError, "k_weight", b=wk[:64])
    refuse(FaError, "invalid", eps=-1.0)
    refuse(FaError, "invalid", eps=float("nan"))
    refuse(FaError, "invalid", eps=1e300)
    refuse(ValueError, "overlap", out=(q[:, :1].expand(-1, 4, -1), torch.empty_like(k)), only=("pass",))
    refuse(ValueError, "overlap", out=q[:, :1].expand(-1, 4, -1), only=("append",))
    refuse(ValueError, "k_out", k_out=k[:, :1], only=("append",))
    refuse(ValueError, "pair", out=(q,), only=("pass",))
    refuse(ValueError, "pair", grads=(q, k, q), only=("back",))
    refuse(ValueError, "workspace", workspace=torch.empty(16, dtype=torch.uint8, device="cuda:0"), only=("back",))
    refuse(ValueError, "workspace", workspace=torch.empty(1 << 20, device="cuda:0"), only=("back",))
    with pytest.raises(ValueError, match="slots"):
        api.kv4_append(q, k, v, rotary, pos, slots.int(), cache)
    with pytest.raises(ValueError, match="v must|shape"):
        api.kv4_append(q, k, v[:, :1], rotary, pos, slots, cache)
    assert all(torch.equal(a, b) for a, b in zip(before, (q, k, cache.k_codes)))


def test_append_refuses_what_is_no_tensor():
    import torch
    from tiled_attention_tmem_gb300 import api
    q, k, rotary, pos, wq, wk, v = make(16, 4, 2, 64, 64, value=True, loose=False)
    slots, cache = torch.arange(16, device="cuda:0"), api.KV4Cache.empty(1, 2, 16, 64)
    for kw in (dict(k_out=5), dict(out=5), dict(k_out="k"), dict(k_out=k.tolist())):
        with pytest.raises(TypeError, match="must be a torch tensor"):
            api.kv4_append(q, k, v, rotary, pos, slots, cache, wq, wk, **kw)
    assert not bool(cache.k_codes.any())


def test_graphs_that_share_a_workspace():
    """Two captured steps, forward and backward, of different sizes and one workspace, replayed in turn after their
    inputs changed: each gives what an uncaptured call gives."""
    import torch
    from tiled_attention_tmem_gb300 import api
    stream, steps = torch.cuda.Stream(), []
    ws = torch.empty(4 << 20, dtype=torch.uint8, device="cuda:0")
    for T, H, Hkv, d, turned in ((300, 8, 2, 128, 128), (77, 5, 1, 96, 32)):
        q, k, rotary, pos, wq, wk = make(T, H, Hkv, d, turned, seed=T)
        t = [x.contiguous() for x in (q, k)]
        t += [torch.ones_like(x) for x in t]

        def step(t=t, at=(rotary, pos, wq, wk), **kw):
            return (*api.qk_norm_rope(t[0], t[1], *at, out=(torch.zeros_like(t[0]), torch.zeros_like(t[1]))),
                    *api.qk_norm_rope_backward(t[2], t[3], t[0], t[1], *at, **kw))
        assert api.qk_norm_rope_workspace_bytes(T, H, Hkv, d) <= ws.numel()
        with torch.cuda.stream(stream):
            step(workspace=ws)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = step(workspace=ws)
        steps.append((graph, t, out, step))
    for turn in range(3):
        for graph, t, out, step in steps:
            for x in t:
                x.copy_(torch.randn(x.shape, device="cuda:0"))
        torch.cuda.synchronize()
        for graph, t, out, step in steps:
            graph.replay()
            graph.replay()
        torch.cuda.synchronize()
        for graph, t, out, step in steps:
            assert all(torch.equal(a, b) for a, b in zip(out, step()))


def test_streams_and_the_profile():
    import torch
    from tiled_attention_tmem_gb300 import api
    from tiled_attention_tmem_gb300 import binding as b
    q, k, rotary, pos, wq, wk, v = make(2000, 8, 2, 128, 128, value=True)
    slots = torch.arange(2000, device="cuda:0")
    cache = api.KV4Cache.empty(125, 2, 16, 128)
    ref = api.qk_norm_rope(q, k, rotary, pos, wq, wk, out=(torch.zeros_like(q), torch.zeros_like(k)))
    back = api.qk_norm_rope_backward(q, k, q, k, rotary, pos, wq, wk)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(10):  # two at once, each with its own outputs and workspaces
        for s in streams:
            with torch.cuda.stream(s):
                y = api.qk_norm_rope(q, k, rotary, pos, wq, wk, out=(torch.zeros_like(q), torch.zeros_like(k)))
                got.append((y, api.qk_norm_rope_backward(q, k, q, k, rotary, pos, wq, wk)))
    torch.cuda.synchronize()
    for y, g in got:
        assert all(torch.equal(a, b) for a, b in zip((*y, *g), (*ref, *back)))
    b.fa_profile_start()
    api.qk_norm_rope(q, k, rotary, pos, wq, wk)
    api.qk_norm_rope_backward(q, k, q, k, rotary, pos, wq, wk)
    api.qk_norm_rope_backward(q, k, q, k, rotary, pos)
    api.kv4_append(q, k, v, rotary, pos, slots, cache, wq, wk)
    counts = {n: c for n, (c, _) in b.fa_profile_stop().items() if c}
    assert counts == {"rotate": 1, "rotate_bwd": 2, "rotate_sum": 1, "kv4_append": 1}
