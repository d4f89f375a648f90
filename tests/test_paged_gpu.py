"""Page tables, the 4-bit cache's store and load, and attention over it, against plain
64-bit restatements (kv4_ref)."""

import math

import numpy as np
import pytest

import kv4_ref as R
from helpers import to_dev, to_f64

pytestmark = pytest.mark.gpu

DIMS = (64, 96, 128, 192, 256, 384)


def _dev(x, dtype):
    import torch
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda:0")


def _i32(x):
    import torch
    return _dev(x, torch.int32)


# ------------------------------------------------------------------ page tables

def _grow_case(B, page, most, new, seed, free=None, width=None, T=None):
    rng = np.random.default_rng(seed)
    held = rng.integers(0, most + 1, B)
    add = rng.integers(0, new + 1, B)
    width = -(-(most + new) // page) if width is None else width
    owned = np.minimum(-(-held // page), width)
    ids = rng.permutation(int(owned.sum() + (-(-(held + add) // page)).sum()) + 7)
    table = np.full((B, width), -7)
    at = 0
    for b in range(B):
        table[b, :owned[b]] = ids[at:at + owned[b]]
        at += owned[b]
    stack = ids[at:]
    count = len(stack) if free is None else free
    return held, add, table, stack, count, int(add.sum()) + 3 if T is None else T


@pytest.mark.parametrize("B,page,most,new,kw", [
    (1, 16, 0, 1, {}), (1, 64, 100, 5000, {}), (3, 32, 70, 40, {}), (300, 16, 200, 1, {}), (777, 64, 900, 300, {}),
    (40, 128, 1000, 600, {}), (5, 16, 64, 64, dict(free=3)), (64, 16, 64, 64, dict(free=0)),
    (33, 16, 100, 60, dict(width=5)), (33, 16, 100, 60, dict(T=100)), (9, 32, 50, 50, dict(T=0)),
    (2000, 16, 40, 3, {}), (4, 16, 50, 0, {}),
], ids=str)
def test_page_grow(B, page, most, new, kw):
    import torch
    from tiled_attention_tmem_gb300 import api
    held, add, table, stack, count, T = _grow_case(B, page, most, new, seed=B + page, **kw)
    slots, cu, tab, hold, left = R.pages(held, add, table, stack, count, page, T)
    t = _i32(table)
    for _ in range(2):  # nothing but fresh table entries changes: a repeat gives the same
        got = api.page_grow(_i32(held), _i32(add), t, _i32(stack), _i32([count]), page, T)
        for g, r in zip(got, (slots, cu, hold, [left])):
            assert np.array_equal(g.cpu().numpy(), r)
        assert np.array_equal(t.cpu().numpy(), tab)
    # The slots of all that is now held, from the finished table.
    got, cu2 = api.page_slots(_i32(np.zeros(B, int)), _i32(hold), t, page, int(hold.sum()) + 2)
    ref = R.pages(np.zeros(B, int), hold, tab, [], None, page, int(hold.sum()) + 2)
    assert np.array_equal(got.cpu().numpy(), ref[0]) and np.array_equal(cu2.cpu().numpy(), ref[1])
    assert got.dtype == torch.int64


def test_page_grow_ignores_negative_counts_and_a_count_above_the_stack():
    from tiled_attention_tmem_gb300 import api
    held, add = [-5, 3, 20], [2, -4, 14]
    table = np.full((3, 4), 2)
    t = _i32(table)
    got = api.page_grow(_i32(held), _i32(add), t, _i32([11, 12]), _i32([1000]), 16, 20)
    ref = R.pages(held, add, table, [11, 12], 1000, 16, 20)
    for g, r in zip(got, (ref[0], ref[1], ref[3], [ref[4]])):
        assert np.array_equal(g.cpu().numpy(), r)
    assert np.array_equal(t.cpu().numpy(), ref[2])


@pytest.mark.parametrize("B", [466_700, 466_944, 1 << 21])
def test_page_grow_of_very_many_requests(B):
    """Block shares of about 48 KB of rows, and the most requests there can be."""
    from tiled_attention_tmem_gb300 import api
    rng = np.random.default_rng(B)
    held, add = rng.integers(0, 16, B), rng.integers(0, 3, B)
    owned = (held > 0).astype(int)
    table = np.where(np.arange(2) < owned[:, None], np.arange(B)[:, None], -7)
    stack = np.arange(B, 2 * B)
    t, T = _i32(table), B // 2
    got = api.page_grow(_i32(held), _i32(add), t, _i32(stack), _i32([B // 3]), 16, T)
    # Without a loop: one page at most is needed beyond those owned, or two tokens' first.
    cu = np.minimum(np.concatenate([[0], np.cumsum(add)]), T)
    add = np.diff(cu)
    need = -(-(held + add) // 16) - owned
    before = np.cumsum(need) - need
    src = B // 3 - 1 - before
    assert need.max() == 1
    fresh = np.where(src >= 0, stack[src], -1)
    tab = table.copy()
    take = need > 0
    tab[np.nonzero(take)[0], owned[take]] = fresh[take]
    req = np.repeat(np.arange(B), add)
    pos = held[req] + np.arange(len(req)) - cu[req]
    page = tab[req, pos // 16]
    slots = np.full(T, -1)
    slots[:len(req)] = np.where(page >= 0, page * 16 + pos % 16, -1)
    room = (owned + (take & (src >= 0))) * 16 - held
    for g, r in zip(got, (slots, cu, held + np.minimum(add, room), [max(B // 3 - need.sum(), 0)])):
        assert np.array_equal(g.cpu().numpy(), r)
    assert np.array_equal(t.cpu().numpy(), tab)


def test_page_calls_with_no_requests_and_no_width():
    import torch
    from tiled_attention_tmem_gb300 import api
    none = torch.empty(0, dtype=torch.int32, device="cuda:0")
    slots, cu, held, count = api.page_grow(none, none, none.view(0, 0), none, _i32([0]), 16, 3)
    assert slots.tolist() == [-1] * 3 and cu.tolist() == [0] and held.numel() == 0 and count.tolist() == [0]
    slots, cu = api.page_slots(_i32([0]), _i32([2]), none.view(1, 0), 16, 3)
    assert slots.tolist() == [-1] * 3 and cu.tolist() == [0, 2]


# ------------------------------------------------------------------ store and load

def _cache_arrays(cache):
    return [t.cpu().numpy() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]


@pytest.mark.parametrize("d", DIMS)
@pytest.mark.parametrize("page,heads,T", [(16, 1, 1), (32, 3, 37), (64, 2, 130), (128, 5, 300)])
def test_store_and_load(d, page, heads, T):
    import torch
    from tiled_attention_tmem_gb300 import api
    rng = np.random.default_rng(d + T)
    pool = -(-T // page) + 3
    x = rng.standard_normal((2, T, heads, d)) * np.exp(rng.standard_normal((2, T, heads, 1)) * 3)
    bits = R.bf16(x)
    # Slices of wider rows, as a fused projection leaves them.
    wide = torch.zeros((T, 2 * heads * d + 24), dtype=torch.bfloat16, device="cuda:0")
    k = wide[:, 8:8 + heads * d].unflatten(1, (heads, d))
    v = wide[:, 16 + heads * d:16 + 2 * heads * d].unflatten(1, (heads, d))
    k.copy_(to_dev(bits[0]))
    v.copy_(to_dev(bits[1]))
    slots = rng.permutation(pool * page)[:T].astype(np.int64)
    slots[rng.random(T) < 0.1] = -1
    if T > 3:
        slots[1], slots[2] = pool * page, -(1 << 40)  # outside the pool
    cache = api.KV4Cache.empty(pool, heads, page, d, 2.0 ** -5, 2.0 ** -6)
    for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales):
        t.fill_(0xA5)
    api.kv4_store(k, v, _dev(slots, torch.int64), cache)
    got = _cache_arrays(cache)
    fine = (slots >= 0) & (slots < pool * page)
    pg, off = slots[fine] // page, slots[fine] % page
    for i, gain in ((0, 2.0 ** -5), (1, 2.0 ** -6)):
        codes, scales = R.encode(to_f64(to_dev(bits[i])), gain)
        want_c, want_s = np.full_like(got[2 * i], 0xA5), np.full_like(got[2 * i + 1], 0xA5)
        want_c[pg, :, off], want_s[pg, :, off] = codes[fine], scales[fine]
        assert np.array_equal(got[2 * i + 1], want_s)
        same = got[2 * i] == want_c
        # A zero keeps its sign in the cache; the restatement has no signed zero.
        assert np.all(same | (R.e2m1_value(got[2 * i] & 15) == R.e2m1_value(want_c & 15))
                      & (R.e2m1_value(got[2 * i] >> 4) == R.e2m1_value(want_c >> 4)))
    lk, lv = api.kv4_load(_dev(slots, torch.int64), cache)
    for i, (t, gain) in enumerate(((lk, 2.0 ** -5), (lv, 2.0 ** -6))):
        want = np.zeros((T, heads, d))
        want[fine] = R.decode(got[2 * i][pg, :, off], got[2 * i + 1][pg, :, off], gain)
        assert np.array_equal(to_f64(t), want)  # gains that are powers of two: exact in bf16
    api.check_device_error()


def test_store_rounds_every_bf16_ratio_to_nearest_even():
    """Every scale a row can get against every bf16 mantissa: ties and their neighbours."""
    import torch
    from tiled_attention_tmem_gb300 import api
    tops, small = [], []
    for m in range(128, 256):  # the largest of a group sets the scale: amax / 6
        for k in (128 + np.arange(128)):
            tops.append(m / 128.0)
            small.append(k / 128.0)
    tops, small = np.array(tops), np.array(small)
    x = np.zeros((len(tops), 16))
    x[:, 0] = tops
    for j in range(1, 8):
        x[:, j] = np.minimum(small * 2.0 ** (1 - j), tops)
        x[:, 15 - j] = -x[:, j]
    x = np.concatenate([x, x * 2.0 ** -8, x * 2.0 ** 9])
    x = x.reshape(-1, 4, 1, 16).transpose(0, 2, 1, 3).reshape(-1, 1, 64)
    T = len(x)
    cache = api.KV4Cache.empty(-(-T // 64), 1, 64, 64)
    k = to_dev(R.bf16(x))
    slots = torch.arange(T, device="cuda:0")
    api.kv4_store(k, k, slots, cache)
    codes, scales = R.encode(x, 1.0)
    got = _cache_arrays(cache)
    n = T // 64 * 64
    assert np.array_equal(got[1].reshape(-1, 4)[:n], scales[:n, 0])
    both = np.stack([got[0] & 15, got[0] >> 4], -1).reshape(-1, 64)[:n]
    want = np.stack([codes & 15, codes >> 4], -1).reshape(-1, 64)[:n]
    assert np.array_equal(R.e2m1_value(both), R.e2m1_value(want))


def test_store_of_infinities_nan_and_zeros_stays_finite():
    import torch
    from tiled_attention_tmem_gb300 import api
    x = np.zeros((4, 1, 64), np.float32)
    x[0, 0, :4] = [np.inf, 1.0, -2.0, 3.0]
    x[0, 0, 16:20] = [-np.inf, 1e30, -1e30, 0]
    x[1, 0, :4] = [np.nan, 6.0, -3.0, 0.5]
    x[2, 0, 0] = 1e-30
    k = to_dev(R.bf16(x))
    cache = api.KV4Cache.empty(1, 1, 16, 64)
    slots = torch.arange(4, device="cuda:0")
    api.kv4_store(k, k, slots, cache)
    lk, _ = api.kv4_load(slots, cache)
    got = to_f64(lk)
    assert np.all(np.isfinite(got))
    assert got[0, 0, 0] == 2688 and list(got[0, 0, 16:20]) == [-2688, 2688, -2688, 0]
    assert list(got[1, 0, :4]) == [6, 6, -3, 0.5]  # NaN: code 6 under the scale of the others
    assert np.all(got[2:] == 0)


def test_load_of_every_byte():
    """All codes under all scale bytes, the sign bit of a scale and 0x7f included; a gain
    that is no power of two is rounded once."""
    import torch
    from tiled_attention_tmem_gb300 import api
    cache = api.KV4Cache.empty(16, 1, 16, 64, 0.3, 1.0)
    cache.k_codes.copy_(torch.arange(32, device="cuda:0").to(torch.uint8).mul_(8).add_(3).expand(16, 1, 16, 32))
    cache.v_codes.copy_(torch.arange(8, device="cuda:0").repeat(4).to(torch.uint8).mul_(16).add_(9).expand(16, 1, 16, 32))
    every = torch.arange(256, device="cuda:0").to(torch.uint8).view(16, 1, 16, 1).expand(16, 1, 16, 4)
    cache.k_scales.copy_(every)
    cache.v_scales.copy_(every)
    lk, lv = api.kv4_load(torch.arange(256, device="cuda:0"), cache)
    a = _cache_arrays(cache)
    assert np.array_equal(to_f64(lv), R.decode(a[2], a[3], 1.0).reshape(256, 1, 64))
    want = R.decode(a[0], a[1], float(np.float32(0.3))).reshape(256, 1, 64)
    # fp32 product (2^-24) and bf16 (2^-8), relative.
    assert np.all(np.abs(to_f64(lk) - want) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(want))


# ------------------------------------------------------------------ attention

def _problem(d, page, heads, kv, lengths, queries, seed, spread=1.0, spare=3, pad=0, gains=(2.0 ** -6, 2.0 ** -5)):
    """A pool with the requests' pages scattered, everything else filled with 0xff."""
    rng = np.random.default_rng(seed)
    need = [-(-max(n, 0) // page) for n in lengths]
    pool = sum(need) + spare
    ids = rng.permutation(pool)
    width = max(need + [1]) + 1
    table = np.full((len(lengths), width), -1)
    at = 0
    arrays = [np.full((pool, kv, page, d // 2), 0xFF, np.uint8), np.full((pool, kv, page, d // 16), 0xFF, np.uint8),
              np.full((pool, kv, page, d // 2), 0xFF, np.uint8), np.full((pool, kv, page, d // 16), 0xFF, np.uint8)]
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
        for i, gain in enumerate(gains):
            x = rng.standard_normal((n, kv, page, d)) * (spread if i == 0 else 1.0)
            codes, scales = R.encode(x, gain)
            last = max(lengths[b], 0) - (n - 1) * page
            if n:  # slots behind the last token keep their 0xff
                codes[-1, :, last:], scales[-1, :, last:] = 0xFF, 0xFF
            arrays[2 * i][table[b, :n]], arrays[2 * i + 1][table[b, :n]] = codes, scales
    cu = np.concatenate([[0], np.cumsum(queries)])
    q = R.bf16(rng.standard_normal((int(cu[-1]) + pad, heads, d)))
    return arrays, table, cu, q, gains


def _cache_of(arrays, gains):
    import torch
    from tiled_attention_tmem_gb300 import api
    return api.KV4Cache(*(torch.from_numpy(a).cuda() for a in arrays), *gains)


def _reference(arrays, gains, table, cu, q, lengths, max_q, scale):
    # Each byte pattern stands for a finite value, but slots behind a request's last
    # token are no keys, so the restatement never reads their 0xff.
    k = R.decode(arrays[0], arrays[1], gains[0])
    v = R.decode(arrays[2], arrays[3], gains[1])
    return R.attend(to_f64(to_dev(q, "cpu")), (k, v), table, lengths, cu, max_q, scale)


def _attend(problem, lengths, max_q, scale=None, **kw):
    from tiled_attention_tmem_gb300 import api
    arrays, table, cu, q, gains = problem
    d = q.shape[-1]
    cache = _cache_of(arrays, gains)
    o, lse = api.kv4_attention(to_dev(q), cache, _i32(table), _i32(lengths), _i32(cu), max_q, scale, **kw)
    api.check_device_error()
    ref = _reference(arrays, gains, table, cu, q, lengths, max_q, 1 / math.sqrt(d) if scale is None else scale)
    own = int(cu[-1])
    R.check(to_f64(o)[:own], to_f64(lse)[:own], tuple(x[:own] for x in ref), d)
    return o, lse


LENGTHS = [0, 1, 15, 16, 17, 63, 64, 65, 200, 333]


@pytest.mark.parametrize("d", DIMS)
@pytest.mark.parametrize("page,kv,group", [(16, 2, 1), (32, 1, 4), (64, 3, 8), (128, 1, 7)])
def test_attention_one_query(d, page, kv, group):
    problem = _problem(d, page, kv * group, kv, LENGTHS, [1] * len(LENGTHS), seed=d + page)
    _attend(problem, LENGTHS, 1)


@pytest.mark.parametrize("d", DIMS)
@pytest.mark.parametrize("page,kv,group,queries", [
    (16, 1, 1, [3, 0, 5, 1, 2, 8, 1, 4]), (64, 2, 4, [2, 6, 0, 3, 6, 6, 1, 5]), (32, 1, 16, [1, 2, 3, 3, 0, 2, 3, 1]),
    (128, 1, 5, [9, 1, 0, 7, 3, 9, 2, 4])])
def test_attention_several_queries(d, page, kv, group, queries):
    """Queries a request from none to more than its tokens (rows that see nothing)."""
    lengths = [2, 0, 5, 64, 65, 130, 1, 257]
    problem = _problem(d, page, kv * group, kv, lengths, queries, seed=7 * d + page, pad=3)
    _attend(problem, lengths, max(queries))


@pytest.mark.parametrize("d", DIMS)
@pytest.mark.parametrize("page,kv,group,queries", [
    (64, 1, 16, [9, 0, 1, 4, 9, 2]), (16, 2, 8, [6, 5, 2, 6, 1, 3]), (128, 1, 33, [2, 4, 1, 3, 4, 4]),
    (32, 1, 130, [1, 2, 1, 1, 2, 1])])
def test_attention_many_rows(d, page, kv, group, queries):
    """Rows enough for the tcgen05 kernel, up to more than one tile of 128, over contexts
    that begin and end inside a block's share of the units."""
    lengths = [2300, 0, 1, 700, 65, 129]
    problem = _problem(d, page, kv * group, kv, lengths, queries, seed=3 * d + page, pad=2)
    _attend(problem, lengths, max(queries))


@pytest.mark.parametrize("d,page,lengths", [(128, 64, [9000]), (384, 32, [5001]), (256, 16, [4000, 2]), (64, 128, [20000])])
def test_attention_many_rows_cut_over_all_blocks(d, page, lengths):
    problem = _problem(d, page, 20, 1, lengths, [3] * len(lengths), seed=d, spread=3.0, gains=(2.0 ** -4, 2.0 ** -5))
    _attend(problem, lengths, 3)


def test_attention_many_rows_skips_bad_pages_and_foreign_rows():
    import torch
    lengths = [2000, 1500]
    arrays, table, cu, q, gains = _problem(128, 16, 24, 1, lengths, [3, 2], seed=61, pad=2)
    table[0, 3], table[0, 60], table[1, 0], table[1, 17] = -1, 10 ** 6, len(arrays[0]), -9
    o = torch.full((7, 24, 128), 7.0, dtype=torch.bfloat16, device="cuda:0")
    lse = torch.full((7, 24), 7.0, device="cuda:0")
    _attend((arrays, table, cu, q, gains), lengths, 3, out=o, lse=lse)
    assert torch.all(o[5:] == 7) and torch.all(lse[5:] == 7)


def test_attention_many_rows_keeps_nan_in_its_row():
    import torch
    from tiled_attention_tmem_gb300 import api
    lengths = [3000, 900]
    arrays, table, cu, q, gains = _problem(128, 64, 40, 1, lengths, [2, 1], seed=67)
    x, cache = to_dev(q), _cache_of(arrays, gains)
    clean, _ = api.kv4_attention(x, cache, _i32(table), _i32(lengths), _i32(cu), 2)
    x[0, 1, 5], x[2, 20, 0] = float("nan"), float("inf")
    got, lse = api.kv4_attention(x, cache, _i32(table), _i32(lengths), _i32(cu), 2)
    bad = torch.zeros((3, 40), dtype=torch.bool, device="cuda:0")
    bad[0, 1] = bad[2, 20] = True
    assert torch.all(torch.isnan(got[bad])) and torch.all(torch.isnan(lse[bad]))
    assert torch.equal(got[~bad], clean[~bad])


@pytest.mark.parametrize("d,page", [(96, 16), (96, 128), (128, 32), (128, 64)])
@pytest.mark.parametrize("group,queries", [(6, 4), (17, 1), (7, 3)])
@pytest.mark.parametrize("lengths", [[0, 3, 64, 95, 170, 333], [9000, 2, 0, 1025]], ids=["short", "long"])
def test_attention_of_17_to_24_rows(d, page, group, queries, lengths):
    each = [max(1, queries - b % 2) for b in range(len(lengths))]
    problem = _problem(d, page, 2 * group, 2, lengths, each, seed=d + group, spread=2.0)
    _attend(problem, lengths, queries)


@pytest.mark.parametrize("heads,lengths", [(4, [30, 9, 100]), (64, [30, 9, 2000])])
def test_attention_of_more_queries_than_max_q(heads, lengths):
    """The first max_q queries of a request, at the positions that all of them give them;
    the rows of the others stay as they were."""
    import torch
    queries, max_q = [5, 2, 7], 3
    problem = _problem(64, 16, heads, 1, lengths, queries, seed=71)
    o = torch.full((14, heads, 64), 7.0, dtype=torch.bfloat16, device="cuda:0")
    _attend(problem, lengths, max_q, out=o)
    assert torch.all(o[3:5] == 7) and torch.all(o[10:] == 7)


def test_attention_in_place_and_on_two_streams_at_once():
    import torch
    from tiled_attention_tmem_gb300 import api
    runs = []
    for seed, (heads, lengths, queries) in enumerate([(8, [3000, 17, 400], [2, 1, 3]), (32, [40, 900], [4, 4]),
                                                      (80, [5000, 1200], [2, 1])]):
        arrays, table, cu, q, gains = _problem(128, 64, heads, 2 if heads < 80 else 1, lengths, queries, seed=seed)
        args = (_cache_of(arrays, gains), _i32(table), _i32(lengths), _i32(cu), max(queries))
        x = to_dev(q)
        want, lse = api.kv4_attention(x, *args)
        again = x.clone()
        got, lse2 = api.kv4_attention(again, *args, out=again)  # the output over the queries
        assert got is again and torch.equal(got, want) and torch.equal(lse, lse2)
        runs.append((x, args, want, lse))
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    outs = [[] for _ in runs]
    for _ in range(8):
        for s, (x, args, _, _), out in zip(streams, runs, outs):
            with torch.cuda.stream(s):
                out.append(api.kv4_attention(x, *args))
    torch.cuda.synchronize()
    for (_, _, want, lse), out in zip(runs, outs):
        for o, l in out:
            assert torch.equal(o, want) and torch.equal(l, lse)
    api.check_device_error()


def test_attention_of_scores_past_the_range_of_fp32():
    """A scale at the end of fp32: a zero query still weighs all keys alike."""
    import torch
    from tiled_attention_tmem_gb300 import api
    arrays, table, cu, q, gains = _problem(64, 16, 2, 1, [20], [1], seed=73)
    x = to_dev(q)
    x[0, 1] = 0
    o, lse = api.kv4_attention(x, _cache_of(arrays, gains), _i32(table), _i32([20]), scale=1e38)
    ref = _reference(arrays, gains, table, cu, R.bf16(to_f64(x)), [20], 1, 1.0)
    assert abs(float(lse[0, 1]) - math.log(20)) < 1e-5
    assert np.all(np.abs(to_f64(o)[0, 1] - ref[0][0, 1]) <= 2.0 ** -7 * ref[2][0, 1])


def test_attention_without_offsets_is_one_query_a_request():
    from tiled_attention_tmem_gb300 import api
    lengths = [5, 0, 77]
    arrays, table, cu, q, gains = _problem(64, 16, 4, 2, lengths, [1, 1, 1], seed=3)
    o, lse = api.kv4_attention(to_dev(q), _cache_of(arrays, gains), _i32(table), _i32(lengths))
    ref = _reference(arrays, gains, table, cu, q, lengths, 1, 1 / 8)
    R.check(to_f64(o), to_f64(lse), ref, 64)


@pytest.mark.parametrize("d,page,kv,group,lengths", [
    (128, 64, 1, 2, [30000]), (64, 16, 2, 4, [9000, 1, 4097]), (256, 32, 1, 1, [7001, 0, 50]), (384, 128, 1, 3, [5000]),
    (96, 64, 2, 1, [6000, 6000])], ids=str)
def test_attention_cut_over_many_warps(d, page, kv, group, lengths):
    """Few requests, many units: every triple is cut and its parts are merged."""
    problem = _problem(d, page, kv * group, kv, lengths, [1] * len(lengths), seed=d)
    _attend(problem, lengths, 1)


def test_attention_many_requests_share_warps():
    rng = np.random.default_rng(5)
    lengths = [int(n) for n in rng.integers(0, 90, 700)]
    queries = [int(n) for n in rng.integers(0, 3, 700)]
    problem = _problem(64, 16, 4, 2, lengths, queries, seed=6)
    _attend(problem, lengths, 2)


def test_attention_sharp_and_far_scores():
    """Keys far apart: running maxima that grow by more and by less than the threshold."""
    for spread, scale in ((8.0, 1.0), (0.001, None), (30.0, 0.5)):
        problem = _problem(128, 64, 8, 2, [1000, 129], [1, 2], seed=11, spread=spread, gains=(2.0 ** -3, 2.0 ** -5))
        _attend(problem, [1000, 129], 2, scale)


@pytest.mark.parametrize("power", [-100, -20, 12, 30])
def test_attention_queries_of_any_magnitude(power):
    arrays, table, cu, q, gains = _problem(64, 16, 4, 1, [50, 9], [1, 1], seed=13)
    q = R.bf16(np.ldexp(to_f64(to_dev(q, "cpu")), power))
    _attend((arrays, table, cu, q, gains), [50, 9], 1, scale=2.0 ** -power / 8)


def test_attention_skips_bad_pages_and_keeps_foreign_rows():
    import torch
    from tiled_attention_tmem_gb300 import api
    lengths = [200, 90, 64]
    arrays, table, cu, q, gains = _problem(64, 16, 4, 2, lengths, [1, 1, 1], seed=17, pad=5)
    table[0, 3], table[0, 12], table[1, 0] = -1, 10 ** 6, len(arrays[0])
    table[2, :] = -3  # no page at all: the row is empty
    o = torch.full((8, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda:0")
    lse = torch.full((8, 4), 7.0, device="cuda:0")
    _attend((arrays, table, cu, q, gains), lengths, 1, out=o, lse=lse)
    assert torch.all(o[3:] == 7) and torch.all(lse[3:] == 7)
    assert torch.all(o[2] == 0) and torch.all(torch.isinf(lse[2]))


def test_attention_lengths_past_the_table_and_offsets_outside_q():
    import torch
    from tiled_attention_tmem_gb300 import api
    lengths = [40, 20]
    arrays, table, cu, q, gains = _problem(64, 16, 2, 1, lengths, [1, 1], seed=19)
    table = np.ascontiguousarray(table[:, :2])  # 32 tokens fit
    _attend((arrays, table, cu, q, gains), lengths, 1)
    # Offsets that leave q, run backwards or ask for more than max_q.
    cache = _cache_of(arrays, gains)
    for bad in ([0, 5, 9], [-3, 1, 2], [2, 0, 1], [1 << 30, (1 << 30) + 1, 3]):
        o = torch.full((2, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda:0")
        api.kv4_attention(to_dev(q), cache, _i32(table), _i32(lengths), _i32(bad), 4, out=o)
        api.check_device_error()
        assert torch.all(torch.isfinite(o))


def test_attention_of_nan_and_infinite_queries_stays_in_its_row():
    import torch
    from tiled_attention_tmem_gb300 import api
    arrays, table, cu, q, gains = _problem(128, 16, 4, 1, [70, 33], [2, 1], seed=23)
    x = to_dev(q)
    clean, _ = api.kv4_attention(x, _cache_of(arrays, gains), _i32(table), _i32([70, 33]), _i32(cu), 2)
    x[0, 1, 5] = float("nan")
    x[2, 3, 0] = float("inf")
    got, lse = api.kv4_attention(x, _cache_of(arrays, gains), _i32(table), _i32([70, 33]), _i32(cu), 2)
    bad = torch.zeros((3, 4), dtype=torch.bool, device="cuda:0")
    bad[0, 1] = bad[2, 3] = True
    assert torch.all(torch.isnan(got[0, 1])) and torch.isnan(lse[0, 1]) and torch.all(torch.isnan(got[2, 3]))
    assert torch.equal(got[~bad], clean[~bad])


def test_attention_strided_query_and_output_match_dense_ones():
    import torch
    from tiled_attention_tmem_gb300 import api
    lengths, queries = [100, 7, 300], [2, 1, 3]
    arrays, table, cu, q, gains = _problem(128, 32, 8, 2, lengths, queries, seed=29)
    cache = _cache_of(arrays, gains)
    x = to_dev(q)
    dense, lse = api.kv4_attention(x, cache, _i32(table), _i32(lengths), _i32(cu), 3)
    wide = torch.randn((6, 8 * 128 + 512), device="cuda:0").to(torch.bfloat16)
    wide[:, 256:256 + 1024].copy_(x.view(6, -1))
    heads_first = torch.empty((8, 6, 128), dtype=torch.bfloat16, device="cuda:0")
    got, lse2 = api.kv4_attention(wide[:, 256:256 + 1024].unflatten(1, (8, 128)), cache, _i32(table), _i32(lengths),
                                  _i32(cu), 3, out=heads_first.transpose(0, 1))
    assert torch.equal(got, dense) and torch.equal(lse, lse2)
    with pytest.raises(RuntimeError, match="aligned"):
        api.kv4_attention(wide[:, 4:4 + 1024].unflatten(1, (8, 128)), cache, _i32(table), _i32(lengths), _i32(cu), 3)
    with pytest.raises(ValueError, match="dense"):
        api.kv4_attention(x.transpose(1, 2).contiguous().transpose(1, 2), cache, _i32(table), _i32(lengths), _i32(cu), 3)
    with pytest.raises(ValueError, match="channels"):
        api.kv4_attention(x[:, :7], cache, _i32(table), _i32(lengths), _i32(cu), 3)


def test_attention_is_reproducible_and_clean_of_its_workspace():
    import torch
    from tiled_attention_tmem_gb300 import api
    lengths = [5000, 3, 0, 900]
    arrays, table, cu, q, gains = _problem(128, 64, 8, 2, lengths, [1, 1, 1, 1], seed=31)
    cache = _cache_of(arrays, gains)
    args = (to_dev(q), cache, _i32(table), _i32(lengths))
    first = api.kv4_attention(*args)
    for fill in (0, 0xFF, 0x7F):
        ws = torch.full((api.kv4_attention_workspace_bytes(4, 8, cache, table.shape[1]),), fill, dtype=torch.uint8, device="cuda:0")
        again = api.kv4_attention(*args, workspace=ws)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    with pytest.raises(ValueError, match="workspace holds"):
        api.kv4_attention(*args, workspace=ws[:-1])


def test_cache_beyond_four_gigabytes():
    """Pages whose bytes lie past 2^32, written, read back and attended to."""
    import torch
    from tiled_attention_tmem_gb300 import api
    page, kv, d = 128, 2, 128
    pool = (1 << 32) // (page * kv * d // 2) + 40
    cache = api.KV4Cache(*(torch.empty((pool, kv, page, n), dtype=torch.uint8, device="cuda:0")
                           for n in (d // 2, d // 16, d // 2, d // 16)), 2.0 ** -6, 2.0 ** -6)
    rng = np.random.default_rng(37)
    n = 300
    ids = np.array([pool - 1, pool - 30, 2])
    slots = (ids[:, None] * page + np.arange(page)).reshape(-1)[:n]
    x = R.bf16(rng.standard_normal((2, n, kv, d)))
    api.kv4_store(to_dev(x[0]), to_dev(x[1]), _dev(slots, torch.int64), cache)
    lk, lv = api.kv4_load(_dev(slots, torch.int64), cache)
    k, v = (R.decode(*R.encode(to_f64(to_dev(y)), 2.0 ** -6), 2.0 ** -6) for y in x)
    assert np.array_equal(to_f64(lk), k) and np.array_equal(to_f64(lv), v)
    q = R.bf16(rng.standard_normal((1, 4, d)))
    o, lse = api.kv4_attention(to_dev(q), cache, _i32([ids]), _i32([n]))
    full = [np.zeros((3, kv, page, d)) for _ in range(2)]
    for f, y in zip(full, (k, v)):
        f.transpose(0, 2, 1, 3).reshape(-1, kv, d)[:n] = 0  # (a copy: fill below)
        g = f.transpose(0, 2, 1, 3).reshape(-1, kv, d).copy()
        g[:n] = y
        f[:] = g.reshape(3, page, kv, d).transpose(0, 2, 1, 3)
    ref = R.attend(to_f64(to_dev(q)), full, np.array([[0, 1, 2]]), [n], [0, 1], 1, 1 / math.sqrt(d))
    R.check(to_f64(o), to_f64(lse), ref, d)


def test_operands_beyond_two_to_the_31_elements():
    """Token strides that carry a query, an output, and a key past 2^31 elements."""
    import torch
    from tiled_attention_tmem_gb300 import api
    problem = _problem(64, 16, 4, 2, [40, 21, 33], [1, 1, 1], seed=79)
    arrays, table, cu, q, gains = problem
    cache, x = _cache_of(arrays, gains), to_dev(q)
    want, lse = api.kv4_attention(x, cache, _i32(table), _i32([40, 21, 33]))
    step = (1 << 30) + 64
    far = torch.empty(2 * step + 256, dtype=torch.bfloat16, device="cuda:0").as_strided((3, 4, 64), (step, 64, 1))
    far.copy_(x)
    got, lse2 = api.kv4_attention(far, cache, _i32(table), _i32([40, 21, 33]), out=far)
    assert torch.equal(got, want) and torch.equal(lse, lse2)
    slots = torch.arange(3, device="cuda:0")
    api.kv4_store(far[:, :2], far[:, 2:], slots, cache)
    near = api.KV4Cache(*(torch.zeros_like(t) for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)), *gains)
    api.kv4_store(want[:, :2].contiguous(), want[:, 2:].contiguous(), slots, near)
    for a, b in zip(api.kv4_load(slots, cache), api.kv4_load(slots, near)):
        assert torch.equal(a, b)


def test_store_and_load_at_the_ends_of_the_gains():
    """Groups that are zero but for one channel, under the smallest and largest gain."""
    import torch
    from tiled_attention_tmem_gb300 import api
    for power in (-100, 100):
        cache = api.KV4Cache.empty(1, 1, 16, 64, 2.0 ** power, 2.0 ** power)
        x = np.zeros((4, 1, 64))
        x[0, 0, 3], x[1, 0, 17], x[2, 0, 40], x[3, 0, 0] = 2.0 ** 120, 2.0 ** -120, 1.0, -2.0 ** 99
        slots = torch.arange(4, device="cuda:0")
        api.kv4_store(to_dev(R.bf16(x)), to_dev(R.bf16(-x)), slots, cache)
        a = _cache_arrays(cache)
        codes, scales = R.encode(x, 2.0 ** power)
        assert np.array_equal(a[0][0, 0, :4], codes[:, 0]) and np.array_equal(a[1][0, 0, :4], scales[:, 0])
        k, v = api.kv4_load(slots, cache)
        want = R.decode(codes, scales, 2.0 ** power)
        assert np.all(np.abs(to_f64(k) - want) <= 2.0 ** -8 * np.abs(want)) and torch.equal(v, -k)


def test_calls_with_nothing_to_do():
    """No tokens, no requests, no pages, no width, no cached token: shapes, zeros and
    nothing written."""
    import torch
    from tiled_attention_tmem_gb300 import api

    def bf16(*shape):
        return torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda:0")

    none = torch.empty(0, dtype=torch.int64, device="cuda:0")
    cache = api.KV4Cache.empty(3, 2, 16, 64)
    api.kv4_store(bf16(0, 2, 64), bf16(0, 2, 64), none, cache)
    k, v = api.kv4_load(none, cache)
    assert k.shape == v.shape == (0, 2, 64)
    o, lse = api.kv4_attention(bf16(0, 4, 64), cache, _i32([]).view(0, 5), _i32([]))
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
    o = bf16(3, 4, 64)
    api.kv4_attention(bf16(3, 4, 64), cache, _i32([[0, 1]] * 2), _i32([9, 9]), _i32([0, 0, 0]), 2, out=o)
    assert torch.all(o == 7)  # requests without queries
    for pool, width, length in ((3, 0, 9), (0, 2, 9), (3, 2, 0), (3, 2, -4)):
        o, lse = api.kv4_attention(bf16(2, 4, 64), api.KV4Cache.empty(pool, 2, 16, 64), _i32([[0] * width] * 2).view(2, width),
                                   _i32([length] * 2))
        assert torch.all(o == 0) and torch.all(lse == -math.inf)
    empty = api.KV4Cache.empty(0, 2, 16, 64)
    api.kv4_store(bf16(1, 2, 64), bf16(1, 2, 64), torch.zeros(1, dtype=torch.int64, device="cuda:0"), empty)
    k, v = api.kv4_load(torch.zeros(1, dtype=torch.int64, device="cuda:0"), empty)
    assert torch.all(k == 0) and torch.all(v == 0)
    api.check_device_error()


def test_profile_counts_the_serving_kernels():
    import torch
    from tiled_attention_tmem_gb300 import api, binding as b
    arrays, table, cu, q, gains = _problem(64, 16, 4, 2, [3000, 5], [1, 1], seed=83)
    cache, x = _cache_of(arrays, gains), to_dev(q)
    spare = _dev([len(arrays[0]) * 16], torch.int64)  # past the pool: nothing is stored
    b.fa_profile_start()
    api.page_slots(_i32([0, 0]), _i32([1, 1]), _i32(table), 16, 2)
    api.kv4_store(x[:1, :2], x[:1, 2:], spare, cache)
    api.kv4_load(spare, cache)
    api.kv4_attention(x, cache, _i32(table), _i32([3000, 5]))
    prof = b.fa_profile_stop()
    assert {k: n for k, (n, _) in prof.items() if n} == dict(page=1, kv4_store=1, kv4_load=1, kv4_attn=1, kv4_merge=1)


# ------------------------------------------------------------------ together

def _serve(api, torch, page, kv, group, d, prompts, steps, seed, stream=None):
    """Prompts admitted, stored and attended to, then decoding steps: the operators as a
    serving loop calls them.  Yields what each step attended with."""
    rng = np.random.default_rng(seed)
    B, H = len(prompts), kv * group
    pool = sum(-(-(n + steps) // page) for n in prompts) + 2
    width = -(-(max(prompts) + steps) // page)
    cache = api.KV4Cache.empty(pool, kv, page, d, 2.0 ** -6, 2.0 ** -6)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda:0")
    lengths = torch.zeros(B, dtype=torch.int32, device="cuda:0")
    free = _i32(rng.permutation(pool))
    count = _i32([pool])
    keys = [np.zeros((0, kv, d)) for _ in prompts]
    vals = [np.zeros((0, kv, d)) for _ in prompts]
    for step in range(steps + 1):
        new = prompts if step == 0 else [1] * B
        T = sum(new) + 2
        rows = R.bf16(rng.standard_normal((T, (H + 2 * kv) * d)))
        x = to_dev(rows)
        q, k, v = (t.unflatten(1, (-1, d)) for t in (x[:, :H * d], x[:, H * d:(H + kv) * d], x[:, (H + kv) * d:]))
        slots, cu, lengths, count = api.page_grow(lengths, _i32(new), table, free, count, page, T, stream=stream)
        api.kv4_store(k, v, slots, cache, stream=stream)
        o, lse = api.kv4_attention(q, cache, table, lengths, cu, max(new), stream=stream)
        kf, vf = (R.decode(*R.encode(to_f64(t.contiguous()), 2.0 ** -6), 2.0 ** -6) for t in (k, v))
        at = np.concatenate([[0], np.cumsum(new)])
        for b in range(B):
            keys[b] = np.concatenate([keys[b], kf[at[b]:at[b + 1]]])
            vals[b] = np.concatenate([vals[b], vf[at[b]:at[b + 1]]])
        yield to_f64(q.contiguous()), o, lse, new, at, keys, vals, (cache, table, lengths)


@pytest.mark.parametrize("page,kv,group,d", [(16, 2, 4, 64), (64, 1, 8, 128)])
def test_serving_loop(page, kv, group, d):
    import torch
    from tiled_attention_tmem_gb300 import api
    prompts = [5, 70, 1, 33]
    for q, o, lse, new, at, keys, vals, (cache, table, lengths) in _serve(api, torch, page, kv, group, d, prompts, 20, 41):
        for b in range(len(prompts)):
            n = len(keys[b])
            kk, vv = (x[b].transpose(1, 0, 2)[None] for x in (keys, vals))  # one page of n tokens
            ref = R.attend(q[at[b]:at[b + 1]], (kk, vv), np.array([[0]]), [n], [0, new[b]], new[b], 1 / math.sqrt(d))
            R.check(to_f64(o)[at[b]:at[b + 1]], to_f64(lse)[at[b]:at[b + 1]], ref, d)
    # What the cache holds comes back through its slots.
    total = int(lengths.sum())
    slots, cu = api.page_slots(torch.zeros_like(lengths), lengths, table, page, total)
    lk, lv = api.kv4_load(slots, cache)
    assert np.array_equal(to_f64(lk), np.concatenate(keys)) and np.array_equal(to_f64(lv), np.concatenate(vals))
    api.check_device_error()


def test_serving_on_another_stream_and_two_at_once():
    import torch
    from tiled_attention_tmem_gb300 import api
    want = [(o.clone(), l.clone()) for _, o, l, *_ in _serve(api, torch, 16, 2, 4, 64, [5, 70], 4, 43)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    runs = []
    for s in streams:
        with torch.cuda.stream(s):
            runs.append(_serve(api, torch, 16, 2, 4, 64, [5, 70], 4, 43))
    for i, ref in enumerate(want):
        for s, r in zip(streams, runs):
            with torch.cuda.stream(s):
                out = next(r)
            s.synchronize()
            assert torch.equal(out[1][:-2], ref[0][:-2]) and torch.equal(out[2][:-2], ref[1][:-2])
    # An explicit stream handle, with the current stream another one.
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    args = None
    for _, o, l, _, _, _, _, (cache, table, lengths) in _serve(api, torch, 16, 2, 4, 64, [5, 70], 4, 43):
        args = (cache, table, lengths)
    q = to_dev(R.bf16(np.random.default_rng(1).standard_normal((2, 8, 64))))
    torch.cuda.synchronize()
    ref = api.kv4_attention(q, *args)
    got = [api.kv4_attention(q, *args, stream=s.cuda_stream) for _ in range(5)]
    s.synchronize()
    for o, l in got:
        assert torch.equal(o, ref[0]) and torch.equal(l, ref[1])


def test_graph_capture_of_a_decoding_step():
    import torch
    from tiled_attention_tmem_gb300 import api
    page, kv, group, d, B = 16, 2, 4, 128, 3
    H, pool, width, T = kv * group, 40, 12, B
    rng = np.random.default_rng(47)
    cache = api.KV4Cache.empty(pool, kv, page, d, 2.0 ** -6, 2.0 ** -6)
    free, new = _i32(rng.permutation(pool)), _i32([1] * B)
    x = torch.zeros((T, (H + 2 * kv) * d), dtype=torch.bfloat16, device="cuda:0")
    state = dict(table=torch.full((B, width), -1, dtype=torch.int32, device="cuda:0"),
                 lengths=torch.zeros(B, dtype=torch.int32, device="cuda:0"), count=_i32([pool]))

    def step():
        q, k, v = (t.unflatten(1, (-1, d)) for t in (x[:, :H * d], x[:, H * d:(H + kv) * d], x[:, (H + kv) * d:]))
        slots, cu, held, count = api.page_grow(state["lengths"], new, state["table"], free, state["count"], page, T)
        api.kv4_store(k, v, slots, cache)
        out = api.kv4_attention(q, cache, state["table"], held)
        state["lengths"].copy_(held)
        state["count"].copy_(count)
        return out

    def reset():
        state["table"].fill_(-1)
        state["lengths"].zero_()
        state["count"].fill_(pool)
        for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales):
            t.zero_()

    rows = [to_dev(R.bf16(rng.standard_normal((T, (H + 2 * kv) * d)))) for _ in range(50)]
    want = []
    for r in rows:
        x.copy_(r)
        want.append(tuple(t.clone() for t in step()))
    reset()
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=s):
        out = step()
    reset()
    for r, ref in zip(rows, want):
        x.copy_(r)
        graph.replay()
        assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])
    api.check_device_error()


def test_a_set_error_word_stops_the_attention():
    """A kernel that gave up a wait leaves the error word set; attention then writes nothing."""
    import torch
    from tiled_attention_tmem_gb300 import api, binding as b
    arrays, table, cu, q, gains = _problem(64, 16, 4, 2, [300], [1], seed=53)
    o = torch.full((1, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda:0")
    assert b.lib().fa_watchdog_selftest(torch.cuda.current_stream().cuda_stream) == b.FA_OK
    api.kv4_attention(to_dev(q), _cache_of(arrays, gains), _i32(table), _i32([300]), out=o)
    st, _ = b.fa_get_device_error(torch.cuda.current_stream().cuda_stream)
    assert st == b.FA_ERR_DEVICE_TIMEOUT and torch.all(o == 7)
    api.kv4_attention(to_dev(q), _cache_of(arrays, gains), _i32(table), _i32([300]), out=o)
    api.check_device_error()
    assert not torch.any(o == 7)


@pytest.mark.parametrize("heads,lengths", [(4, [30000, 700]), (80, [9000, 700])], ids=["split", "many_rows"])
def test_a_set_error_word_stops_the_attention_and_its_merge(heads, lengths):
    import torch
    from tiled_attention_tmem_gb300 import api, binding as b
    arrays, table, cu, q, gains = _problem(64, 64, heads, 1, lengths, [2, 2], seed=59)
    args = (to_dev(q), _cache_of(arrays, gains), _i32(table), _i32(lengths), _i32(cu), 2)
    assert api.kv4_attention_workspace_bytes(2, heads, args[1], table.shape[1], 2) > 0
    want, lse = api.kv4_attention(*args)
    o, l = torch.full_like(want, 7.0), torch.full_like(lse, 7.0)
    assert b.lib().fa_watchdog_selftest(torch.cuda.current_stream().cuda_stream) == b.FA_OK
    api.kv4_attention(*args, out=o, lse=l)
    st, _ = b.fa_get_device_error(torch.cuda.current_stream().cuda_stream)
    assert st == b.FA_ERR_DEVICE_TIMEOUT and torch.all(o == 7) and torch.all(l == 7)
    api.kv4_attention(*args, out=o, lse=l)
    api.check_device_error()
    assert torch.equal(o, want) and torch.equal(l, lse)


@pytest.mark.parametrize("heads,kv,d", [(4, 2, 128), (20, 1, 96), (80, 1, 64), (40, 1, 384)],
                         ids=["split", "24_rows", "many_rows", "many_rows_384"])
def test_graphs_that_share_a_workspace_follow_new_lengths(heads, kv, d):
    """Two captured graphs over one workspace, replayed in turn while lengths change in place."""
    import torch
    from tiled_attention_tmem_gb300 import api
    lengths = [6000, 1200, 3]
    arrays, table, _, _, gains = _problem(d, 64, heads, kv, lengths, [1, 1, 1], seed=89)
    cache, tab, held = _cache_of(arrays, gains), _i32(table), _i32(lengths)
    qs = [torch.randn((3, heads, d), device="cuda:0").to(torch.bfloat16) for _ in range(2)]
    ws = torch.empty(max(api.kv4_attention_workspace_bytes(3, heads, cache, table.shape[1]), 1), dtype=torch.uint8, device="cuda:0")
    assert ws.numel() > 1
    api.kv4_attention(qs[0], cache, tab, held, workspace=ws)
    graphs, stream = [], torch.cuda.Stream()
    for q in qs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            out = api.kv4_attention(q, cache, tab, held, workspace=ws)
        graphs.append((g, out))
    for new in (lengths, [1, 0, 3], [6000, 1199, 2], [511, 64, 1]):
        held.copy_(_i32(new))
        for (g, out), q in zip(graphs, qs):
            g.replay()
            want = api.kv4_attention(q, cache, tab, held)
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    for g, _ in graphs * 10:  # back to back
        g.replay()
    for (_, out), q in zip(graphs, qs):
        want = api.kv4_attention(q, cache, tab, held)
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    api.check_device_error()


def test_stream_zero_is_the_default_stream(monkeypatch):
    """Handle 0 as the stream of every call, while another stream is current: each kernel is
    launched on the default stream, and what is allocated belongs to it."""
    import torch
    from tiled_attention_tmem_gb300 import api, binding as b, serving
    lengths = [3000, 40]
    arrays, table, cu, q, gains = _problem(64, 16, 4, 2, lengths, [1, 1], seed=97)
    cache, x, tab, held = _cache_of(arrays, gains), to_dev(q), _i32(table), _i32(lengths)
    free, count, slots = _i32([5]), _i32([1]), _dev([len(arrays[0]) * 16] * 2, torch.int64)
    streams = []

    class Lib:
        def __getattr__(self, name):
            call = getattr(real, name)
            if not name.startswith(("fa_page", "fa_kv4")) or name.endswith("_size"):
                return call
            return lambda *a: (streams.append(a[-1]), call(*a))[1]

    real = b.lib()
    monkeypatch.setattr(b, "lib", Lib)
    side = torch.cuda.Stream()
    assert torch.cuda.default_stream().cuda_stream == 0 and side.cuda_stream != 0
    want = api.kv4_attention(x, cache, tab, held)
    torch.cuda.synchronize()
    streams.clear()
    with torch.cuda.stream(side):
        api.page_grow(held, _i32([0, 0]), tab, free, count, 16, 2, stream=0)
        api.page_slots(held, _i32([0, 0]), tab, 16, 2, stream=0)
        api.kv4_store(x[:, :2], x[:, 2:], slots, cache, stream=0)
        api.kv4_load(slots, cache, stream=0)
        got = api.kv4_attention(x, cache, tab, held, stream=0)
        with serving._On(0, 0):
            assert torch.cuda.current_stream().cuda_stream == 0
        assert torch.cuda.current_stream() == side
    assert streams == [0] * 5
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("heads,kv,lengths,queries", [
    (4, 2, [30, 9, 100], [5, 2, 7]), (64, 1, [30, 9, 2000], [3, 0, 2]), (6, 1, [3000, 1, 700], [4, 1, 2])], ids=str)
def test_attention_with_offsets_alone_computes_every_query(heads, kv, lengths, queries):
    import torch
    from tiled_attention_tmem_gb300 import api
    arrays, table, cu, q, gains = _problem(64, 16, heads, kv, lengths, queries, seed=101, pad=2)
    o = torch.full((len(q), heads, 64), 7.0, dtype=torch.bfloat16, device="cuda:0")
    lse = torch.full((len(q), heads), 7.0, device="cuda:0")
    args = to_dev(q), _cache_of(arrays, gains), _i32(table), _i32(lengths), _i32(cu)
    api.kv4_attention(*args, out=o, lse=lse)
    api.check_device_error()
    ref = _reference(arrays, gains, table, cu, q, lengths, max(queries), 1 / 8)
    own = int(cu[-1])
    R.check(to_f64(o)[:own], to_f64(lse)[:own], tuple(x[:own] for x in ref), 64)
    assert torch.all(o[own:] == 7) and torch.all(lse[own:] == 7)


@pytest.mark.parametrize("page,T", [(16, 40), (64, 7)])
def test_page_grow_with_an_empty_stack(page, T):
    """No page is free: tokens that fit the last page owned get slots, the others none."""
    import torch
    from tiled_attention_tmem_gb300 import api
    held, add = [0, 5, page, 2 * page - 1, 3], [4, 2, 1, 9, 0]
    table = np.arange(15).reshape(5, 3) + 20
    none = torch.arange(4, dtype=torch.int32, device="cuda:0")[:0]
    assert none.data_ptr() == 0
    for count in (0, 5):
        t = _i32(table)
        got = api.page_grow(_i32(held), _i32(add), t, none, _i32([count]), page, T)
        ref = R.pages(held, add, table, [], 0, page, T)
        for g, r in zip(got, (ref[0], ref[1], ref[3], [0])):
            assert np.array_equal(g.cpu().numpy(), r)
        assert np.array_equal(t.cpu().numpy(), ref[2])


@pytest.mark.parametrize("heads,kv,lengths", [(2, 1, [40, 20]), (4, 2, [9000, 700]), (80, 1, [5000, 700])],
                         ids=["block", "split", "many_rows"])
def test_attention_of_offsets_that_leave_the_queries(heads, kv, lengths):
    """Offsets that leave q or run backwards: those requests have no queries, the others'
    rows are right, and every other byte of the buffers around q, o and lse is as it was."""
    import torch
    from tiled_attention_tmem_gb300 import api
    T, max_q, most, least = 6, 4, (1 << 31) - 1, -(1 << 31)
    arrays, table, _, q, gains = _problem(64, 16, heads, kv, lengths, [T, 0], seed=103, pad=6)
    cache, tab, held = _cache_of(arrays, gains), _i32(table), _i32(lengths)
    wide_q = to_dev(q)  # six rows between three and three more
    for cu, valid in (([0, 5, 9], [0]), ([-3, 1, 2], [1]), ([2, 0, 1], [1]), ([1 << 30, (1 << 30) + 1, 3], []),
                      ([0, 7, 7], []), ([0, 2, 7], [0]), ([1, 6, 6], [0]), ([0, 2, most], [0]), ([least, most, 3], []),
                      ([least, least, 6], []), ([most, least, 0], []), ([0, 0, 6], [1]), ([4, 6, 2], [0])):
        o = torch.full((T + 6, heads, 64), 7.0, dtype=torch.bfloat16, device="cuda:0")
        lse = torch.full((T + 6, heads), 7.0, device="cuda:0")
        api.kv4_attention(wide_q[3:3 + T], cache, tab, held, _i32(cu), max_q, out=o[3:3 + T], lse=lse[3:3 + T])
        api.check_device_error()
        mine = torch.zeros(T + 6, dtype=torch.bool, device="cuda:0")
        for b in valid:
            rows = slice(cu[b], min(cu[b + 1], cu[b] + max_q))
            mine[3 + rows.start:3 + rows.stop] = True
            ref = _reference(arrays, gains, table[b:b + 1], [cu[b], cu[b + 1]], q[3:3 + T], lengths[b:b + 1], max_q, 1 / 8)
            R.check(to_f64(o)[3:3 + T][rows], to_f64(lse)[3:3 + T][rows], tuple(x[rows] for x in ref), 64, str(cu))
        assert torch.all(o[~mine] == 7) and torch.all(lse[~mine] == 7), cu


def test_attention_refuses_a_max_q_past_31_bits():
    """2^32 + 1 would be cut to 1 on its way to the library: the first query of each request."""
    from tiled_attention_tmem_gb300 import api
    arrays, table, cu, q, gains = _problem(64, 16, 2, 1, [40, 20], [3, 2], seed=107)
    args = to_dev(q), _cache_of(arrays, gains), _i32(table), _i32([40, 20]), _i32(cu)
    for max_q in (1 << 31, (1 << 32) + 1):
        with pytest.raises(ValueError, match="max_q"):
            api.kv4_attention(*args, max_q)
    with pytest.raises(RuntimeError, match="invalid"):
        api.kv4_attention(*args, -1)


@pytest.mark.parametrize("heads,kv,lengths", [(4, 2, [50, 9]), (4, 2, [6000, 700]), (80, 1, [5000, 700])],
                         ids=["block", "split", "many_rows"])
@pytest.mark.parametrize("scale,gain,keys,power", [
    (1.5 * 2.0 ** 127, -100, -94, -35), (2.0 ** 62, 60, 58, -123), (2.0 ** -120, 0, 6, 112),
    (2.0 ** 30, -100, -94, 62)], ids=["scale", "product", "tiny_scale", "gain"])
def test_attention_of_ordinary_scores_from_extreme_factors(heads, kv, lengths, scale, gain, keys, power):
    """scale, k_gain and q at the ends of their ranges, with products that fp32 does not hold
    and scores of ordinary size."""
    arrays, table, cu, q, gains = _problem(64, 16, heads, kv, lengths, [2, 1], seed=109, spread=2.0 ** keys,
                                           gains=(2.0 ** gain, 2.0 ** -5))
    q = R.bf16(np.ldexp(to_f64(to_dev(q, "cpu")), power))
    _attend((arrays, table, cu, q, gains), lengths, 2, scale=scale)


# ------------------------------------------------------------------ many tokens, long shares

@pytest.mark.parametrize("heads", [1, 5])
@pytest.mark.parametrize("d", DIMS)
def test_store_and_load_of_many_tokens(d, heads):
    """Tokens enough for the kernels that keep four a warp in flight, with an end inside a
    batch: the same bytes as in calls too short for them, and the restatement's for a sample."""
    import torch
    from tiled_attention_tmem_gb300 import api
    pieces = heads * d // 8
    per_warp, chunks = max(1, 32 // pieces), -(-pieces // 32)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    T = -(-128 * sms // chunks) * per_warp  # T / per_warp * chunks tokens' rows: 128 an SM
    T += 8 * 4 * per_warp + 4 * per_warp + 1
    assert T % (8 * 4 * per_warp)
    page, rng = 64, np.random.default_rng(d + heads)
    pool = -(-T // page) + 2
    g = torch.Generator(device="cuda:0").manual_seed(d)
    x = torch.randn((T, 2 * heads, d), generator=g, device="cuda:0") * torch.exp(
        3 * torch.randn((T, 2 * heads, 1), generator=g, device="cuda:0"))
    x = x.to(torch.bfloat16)
    k, v = x[:, :heads], x[:, heads:]
    slots = rng.permutation(pool * page)[:T].astype(np.int64)
    slots[rng.random(T) < 0.1] = -1
    slots[rng.integers(0, T, 20)] = pool * page
    slots[rng.integers(0, T, 20)] = -(1 << 40)
    slots[-3:] = -1, slots[-2], slots[-1]
    where = _dev(slots, torch.int64)
    caches = []
    for step in (T, T // 4 + 1):
        cache = api.KV4Cache.empty(pool, heads, page, d, 2.0 ** -5, 2.0 ** -6)
        for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales):
            t.fill_(0xA5)
        for t in range(0, T, step):
            api.kv4_store(k[t:t + step], v[t:t + step], where[t:t + step], cache)
        caches.append(cache)
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(caches[0], name), getattr(caches[1], name)), name
    lk, lv = api.kv4_load(where, caches[0])
    parts = [api.kv4_load(where[t:t + T // 4 + 1], caches[0]) for t in range(0, T, T // 4 + 1)]
    for whole, part in ((lk, torch.cat([p[0] for p in parts])), (lv, torch.cat([p[1] for p in parts]))):
        assert torch.equal(whole, part)
    sample = np.unique(np.concatenate([np.arange(T - 70, T), rng.integers(0, T, 200)]))
    fine = (slots[sample] >= 0) & (slots[sample] < pool * page)
    for dense, out, gain in ((k, lk, 2.0 ** -5), (v, lv, 2.0 ** -6)):
        rows = to_f64(dense[torch.from_numpy(sample).cuda()].contiguous())
        want = np.where(fine[:, None, None], R.decode(*R.encode(rows, gain), gain), 0.0)
        assert np.array_equal(to_f64(out[torch.from_numpy(sample).cuda()].contiguous()), want)
    api.check_device_error()


def _long_problem(d, page, kv, heads, lengths, queries, seed, bad=0.02):
    """A cache of random codes and scales on the GPU, some entries of the table no page."""
    import torch
    from tiled_attention_tmem_gb300 import api
    g = torch.Generator(device="cuda:0").manual_seed(seed)
    need = [-(-n // page) for n in lengths]
    pool, width = sum(need) + 3, max(need)

    def random(n, low, high):
        return torch.randint(low, high, (pool, kv, page, n), generator=g, device="cuda:0", dtype=torch.uint8)

    # Scales from 1/4 to 2: scores with a deviation of about 3.
    cache = api.KV4Cache(random(d // 2, 0, 256), random(d // 16, 0x28, 0x41), random(d // 2, 0, 256),
                         random(d // 16, 0x28, 0x41), 1.0, 2.0 ** -5)
    ids = torch.randperm(pool, generator=g, device="cuda:0").int()
    table = torch.full((len(lengths), width), -1, dtype=torch.int32, device="cuda:0")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    hit = torch.rand((len(lengths), width), generator=g, device="cuda:0")
    table[hit < bad] = -1
    table[hit > 1 - bad / 2] = pool
    cu = np.concatenate([[0], np.cumsum(queries)])
    q = torch.randn((int(cu[-1]), heads, d), generator=g, device="cuda:0").to(torch.bfloat16)
    return cache, table, cu, q


def _long_reference(cache, table, cu, q, lengths, scale):
    """R.attend in torch's 64 bits, a request at a time."""
    import torch
    dev = "cuda:0"
    pair = torch.tensor([[R.e2m1_value(b & 15), R.e2m1_value(b >> 4)] for b in range(256)], dtype=torch.float64, device=dev)
    value = torch.tensor(R.e4m3_value(np.arange(256)), dtype=torch.float64, device=dev)
    kv, page, d = cache.kv_heads, cache.page_size, cache.head_dim
    T, H, _ = q.shape
    new = dict(dtype=torch.float64, device=dev)
    o, lse, pv, qk, sv = (torch.full((T, H, d), math.nan, **new), torch.full((T, H), math.nan, **new),
                          torch.zeros((T, H, d), **new), torch.zeros((T, H), **new), torch.zeros((T, H, d), **new))
    for b, n in enumerate(lengths):
        t0, t1 = int(cu[b]), int(cu[b + 1])
        if n == 0 or t0 == t1:
            o[t0:t1], lse[t0:t1] = 0.0, -math.inf
            continue
        ids = table[b, :-(-n // page)].long()
        fine = ((ids >= 0) & (ids < cache.pages)).repeat_interleave(page)[:n]
        ids = ids.clamp(0, cache.pages - 1)

        def rows(codes, scales, gain):
            x = pair[codes[ids].long()].flatten(-2) * value[scales[ids].long()].repeat_interleave(16, -1) * gain
            return x.transpose(0, 1).reshape(kv, -1, d)[:, :n]

        k, v = rows(cache.k_codes, cache.k_scales, cache.k_gain), rows(cache.v_codes, cache.v_scales, cache.v_gain)
        x = q[t0:t1].double().view(t1 - t0, kv, H // kv, d)
        see = fine & (torch.arange(n, device=dev) <= n - (t1 - t0) + torch.arange(t1 - t0, device=dev)[:, None])
        s = torch.einsum("ighd,gjd->ighj", x, k) * scale
        s.masked_fill_(~see[:, None, None], -math.inf)
        l = torch.logsumexp(s, -1)
        p = torch.where(torch.isneginf(s), 0.0, torch.exp(s - l[..., None]))
        lse[t0:t1] = l.reshape(t1 - t0, H)
        o[t0:t1] = torch.einsum("ighj,gjd->ighd", p, v).reshape(t1 - t0, H, d)
        pv[t0:t1] = torch.einsum("ighj,gjd->ighd", p, v.abs()).reshape(t1 - t0, H, d)
        size = torch.einsum("ighd,gjd->ighj", x.abs(), k.abs()) * scale
        qk[t0:t1] = torch.where(see[:, None, None], size, 0.0).amax(-1).reshape(t1 - t0, H)
        sv[t0:t1] = torch.einsum("ij,gjd->igd", see.double(), v.abs()).repeat_interleave(H // kv, 1)
    return tuple(t.cpu().numpy() for t in (o, lse, pv, qk, sv))


def _attend_long(d, page, kv, group, lengths, queries, seed, solo=False):
    from tiled_attention_tmem_gb300 import api
    cache, table, cu, q = _long_problem(d, page, kv, kv * group, lengths, queries, seed)
    need = api.kv4_attention_workspace_bytes(len(lengths), kv * group, cache, table.shape[1], max(queries))
    assert (need == 0) == solo
    args = q, cache, table, _i32(lengths), _i32(cu), max(queries)
    o, lse = api.kv4_attention(*args)
    api.check_device_error()
    R.check(to_f64(o), to_f64(lse), _long_reference(cache, table, cu, q, lengths, d ** -0.5), d)
    again = api.kv4_attention(*args)
    assert all(bool((a == b).all()) for a, b in zip((o, lse), again))


# 12 warps an SM and 152 of them, units of 64 tokens: eleven units a warp and more, where its
# ring holds four at most; past one of 256 units, a warp goes from request to request.
LONG = [16384, 1, 3001, 8192, 15000, 64, 12345, 7777, 11111, 9000, 16000, 500, 14001, 8191, 6000, 13000, 10240, 4097, 9999,
        15872]


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("d,group,queries", [
    (d, group, queries) for d in DIMS for group, queries, dims in (
        (4, 1, DIMS), (5, 3, (64, 96, 128, 192)), (9, 3, (64,)), (8, 3, (96, 128)), (11, 2, (64, 96, 128))) if d in dims],
    ids=str)
def test_attention_of_long_shares(d, group, queries, page):
    """Tiles of 8, 16, 24 and 32 rows, and several, whose warps run through their rings."""
    each = [queries if b % 3 else max(1, queries - 1) for b in range(len(LONG))]
    _attend_long(d, page, 8, group, LONG, each, seed=d + group)


@pytest.mark.parametrize("d", DIMS)
def test_attention_of_long_shares_with_a_few_prompts_among_single_queries(d):
    """One request of many queries: the others' rows decide the form, its rows take many tiles."""
    each = [1] * len(LONG)
    each[9] = 21
    _attend_long(d, 64, 8, 2, LONG, each, seed=d)


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("d", DIMS)
def test_attention_of_many_rows_over_long_shares(d, page):
    """tcgen05 kernel: 60 units a block and more, where its rings hold 14 and 32 units'
    page bits are kept; with two row tiles too."""
    _attend_long(d, page, 4, 24, LONG, [3 if b % 4 else 2 for b in range(len(LONG))], seed=d)
    _attend_long(d, page, 1, 70, LONG + LONG, [2] * 40, seed=d + 1)


@pytest.mark.parametrize("d,group,queries", [(d, 4, 1) for d in DIMS] + [(64, 8, 3), (64, 6, 2), (96, 6, 2), (128, 5, 3), (192, 16, 1)],
                         ids=str)
def test_attention_in_one_block_a_request_over_long_rings(d, group, queries):
    """A block per request and kv head with ten units a warp, where its ring holds four."""
    units = 40 if d <= 256 and group * queries <= 8 else 34  # of those that the form still takes
    unit = 64 if d <= 128 else 32
    batch = 38 if d <= 256 and group * queries <= 8 else 30
    rng = np.random.default_rng(d + group)
    lengths = [int(n) for n in rng.integers(1, units * unit + 1, batch)]
    lengths[:3] = [units * unit, 1, units * unit - 1]
    _attend_long(d, 16, 8, group, lengths, [queries] * batch, seed=d, solo=True)


@pytest.mark.parametrize("heads,kv,lengths", [(4, 2, [50, 9]), (4, 2, [6000, 700]), (80, 1, [5000, 700])],
                         ids=["block", "split", "many_rows"])
@pytest.mark.parametrize("power", [-10, -17, -20])
def test_attention_of_queries_with_one_channel_far_above_the_others(heads, kv, lengths, power):
    """A channel that no key has a part in sets the row's power of two, and the scores come
    from channels 2^power below it: exact to 2^-17 of the largest, and 2^-25 of it below that."""
    d, far = 64, 37
    arrays, table, cu, q, gains = _problem(d, 16, heads, kv, lengths, [2, 1], seed=113)
    arrays[0][..., far // 2] &= 0x0F if far % 2 else 0xF0  # the keys' codes of that channel: 0
    x = to_f64(to_dev(q, "cpu"))
    # Between 2^power and 2^(power + 1) in magnitude.
    x = np.where(x < 0, -1.0, 1.0) * (1 + np.abs(x) % 1.0) * 2.0 ** power
    x[..., far] = 1.5
    q = R.bf16(x)
    scale = 2.0 ** -power / 8
    problem = arrays, table, cu, q, gains
    if power >= -17:
        _attend(problem, lengths, 2, scale)
        return
    from tiled_attention_tmem_gb300 import api
    o, lse = api.kv4_attention(to_dev(q), _cache_of(arrays, gains), _i32(table), _i32(lengths), _i32(cu), 2, scale)
    api.check_device_error()
    ro, rl, pv, qk, sv = _reference(arrays, gains, table, cu, q, lengths, 2, scale)
    # sum_c |k_c| of the largest key times a channel's 2^-25 * 1.5: what a score is off by more;
    # a weight by twice that, as exp(2 e) - 1 <= 2 e + 4 e^2 for e below 1/2.
    k = np.abs(R.decode(arrays[0], arrays[1], gains[0])).sum(-1)
    seen = np.zeros(k.shape, bool)
    for b, n in enumerate(lengths):
        seen[table[b, :-(-n // 16)]] = True
    e = k[seen & (arrays[1] != 0xFF).all(-1)].max() * 1.5 * 2.0 ** -25 * scale
    assert e < 0.5
    tol_o, tol_l = R.tolerances(ro, rl, pv, qk, sv, d)
    assert np.all(np.abs(to_f64(lse) - rl) <= tol_l + e)
    assert np.all(np.abs(to_f64(o) - ro) <= tol_o * 2 + (2 * e + 4 * e * e) * 2 * pv)


@pytest.mark.parametrize("heads,length", [(2, 1), (2, 6000), (80, 6000)], ids=["block", "split", "many_rows"])
def test_attention_whose_scores_are_all_minus_infinity_is_an_empty_row(heads, length):
    import torch
    from tiled_attention_tmem_gb300 import api
    arrays, table, cu, q, gains = _problem(64, 16, heads, 1, [length], [1], seed=127)
    arrays[0][..., 2] = arrays[0][..., 2] & 0xF0 | 0x9  # channel 4 of every key: -1/2 of its scale,
    arrays[1][:] = 0x38                                 # which is 1
    x = to_dev(q)
    x[0, 0, 4], x[0, 1, 4] = math.inf, -math.inf
    o, lse = api.kv4_attention(x, _cache_of(arrays, gains), _i32(table), _i32([length]))
    api.check_device_error()
    assert torch.all(o[0, 0] == 0) and lse[0, 0] == -math.inf
    assert torch.all(torch.isnan(o[0, 1])) and torch.isnan(lse[0, 1])
    assert torch.all(torch.isfinite(o[0, 2:])) and torch.all(torch.isfinite(lse[0, 2:]))


def test_page_grow_of_negative_page_ids():
    """An id below 0 is a page to the lengths and the count, and none to the slots."""
    from tiled_attention_tmem_gb300 import api
    held, add, table, stack = [5, 16, 0], [20, 3, 40], [[-1, 8, 8, 8], [4, 8, 8, 8], [8, 8, 8, 8]], [7, -2, 9, -5, 11, 12]
    t = _i32(table)
    got = api.page_grow(_i32(held), _i32(add), t, _i32(stack), _i32([6]), 16, 70)
    ref = R.pages(held, add, table, stack, 6, 16, 70)
    assert list(ref[3]) == [25, 19, 40] and (ref[0][:63] < 0).any()
    for g, r in zip(got, (ref[0], ref[1], ref[3], [ref[4]])):
        assert np.array_equal(g.cpu().numpy(), r)
    assert np.array_equal(t.cpu().numpy(), ref[2])


FIRST_CALL = """
import sys
import torch
sys.path[:0] = {paths!r}
from tiled_attention_tmem_gb300 import api
dev = "cuda:0"
i32 = dict(dtype=torch.int32, device=dev)
cache = api.KV4Cache.empty(40, 1, 16, 64, device=dev)
cache.k_scales.fill_(0x38), cache.v_scales.fill_(0x38)
cache.v_codes.fill_(0x22)
q, table, lengths = torch.ones(1, 2, 64, device=dev).bfloat16(), torch.arange(40, **i32)[None], torch.full((1,), 600, **i32)
graph, out = torch.cuda.CUDAGraph(), torch.zeros(1, 2, 64, device=dev).bfloat16()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    api.kv4_attention(q, cache, table, lengths, out=out)
graph.replay()
api.check_device_error()
assert torch.all(out == 1), out
print("captured")
"""


def test_the_first_call_of_a_process_can_be_captured():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", FIRST_CALL.format(paths=[root])], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and "captured" in out.stdout, out.stdout + out.stderr[-2000:]


@pytest.mark.parametrize("heads,kv,width", [(4, 2, 4), (4, 2, 400), (80, 1, 300)], ids=["block", "split", "many_rows"])
def test_lengths_at_the_ends_of_their_type(heads, kv, width):
    """2^31 - 1 tokens over a table that holds fewer, and a most negative count: attention sees
    what the table holds, pages and slots past it are none."""
    from tiled_attention_tmem_gb300 import api
    most, least, page = (1 << 31) - 1, -(1 << 31), 16
    arrays, table, cu, q, gains = _problem(64, page, heads, kv, [width * page] * 2, [2, 1], seed=131)
    table, lengths = np.ascontiguousarray(table[:, :width]), [most, least]
    _attend((arrays, table, cu, q, gains), lengths, 2)
    held, add = [most, 0, width * page], [most, most, 3]
    three, stack = np.concatenate([table, table[:1]]), np.arange(8) + 5
    t = _i32(three)
    got = api.page_grow(_i32(held), _i32(add), t, _i32(stack), _i32([8]), page, 50)
    ref = R.pages(held, add, three, stack, 8, page, 50)
    for g, r in zip(got, (ref[0], ref[1], ref[3], [ref[4]])):
        assert np.array_equal(g.cpu().numpy(), r)
    assert np.array_equal(t.cpu().numpy(), ref[2])
    first, count = [most, least, width * page - 2], [9, 2, 7]
    got = api.page_slots(_i32(first), _i32(count), t, page, 20)
    ref = R.pages(first, count, ref[2], [], None, page, 20)
    assert np.array_equal(got[0].cpu().numpy(), ref[0]) and np.array_equal(got[1].cpu().numpy(), ref[1])
