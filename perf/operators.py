"""Cases of the paged 4-bit cache: page tables, storing, loading, attention.

Each case is one pass through one operator, either in its plain form (elementary
torch operations in 32 bits) or, with ``own``, through the calls a serving
program makes.  The cache holds keys and values as e2m1 codes (two channels a
byte, the even channel in the low half) with one e4m3 scale per 16 channels of a
token's head and one fp32 gain per tensor: value = gain * scale * code.
"""

import math
import random

import torch

own = False

BF16 = torch.bfloat16
GROUP = 16
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # A full batch of decoding requests, one new token each, small pages.
        dict(name="grow_decode", op="grow", batch=512, page=16, held=8192, new=1),
        # Prompts of very different lengths admitted together.
        dict(name="grow_prompts", op="grow", batch=256, page=64, held=1024, new=1024),
        # The new tokens of one decoding step, a slice of the fused projection.
        dict(name="store_decode", op="store", tokens=64, kv_heads=8, dim=128, page=64),
        # A long prompt written at once.
        dict(name="store_prompt", op="store", tokens=16384, kv_heads=8, dim=128, page=64),
        # A short prefix read back for the dense path, heads of 96 channels.
        dict(name="load_prefix", op="load", tokens=1021, kv_heads=4, dim=96, page=32),
        # A long prefix read back.
        dict(name="load_long", op="load", tokens=65536, kv_heads=4, dim=128, page=64),
        # One short chat request: the latency of a single small call.
        dict(name="attend_short", op="attend", batch=1, heads=8, kv_heads=2, dim=64, page=16, longest=517, ragged=False, query=1),
        # One very long document at batch one.
        dict(name="attend_long", op="attend", batch=1, heads=32, kv_heads=8, dim=128, page=64, longest=131071, ragged=False, query=1),
        # A serving batch of ragged requests, grouped queries.
        dict(name="attend_ragged", op="attend", batch=48, heads=64, kv_heads=8, dim=128, page=64, longest=8192, ragged=True, query=1),
        # A head for every query head, wide heads.
        dict(name="attend_mha", op="attend", batch=7, heads=16, kv_heads=16, dim=256, page=32, longest=4001, ragged=False, query=1),
        # Verification of drafted tokens: several queries a request.
        dict(name="attend_verify", op="attend", batch=16, heads=32, kv_heads=4, dim=128, page=64, longest=4096, ragged=True, query=5),
        # A full machine: many long requests.
        dict(name="attend_full", op="attend", batch=64, heads=32, kv_heads=8, dim=128, page=64, longest=16384, ragged=True, query=1),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("grow", "store", "load", "attend", "attend", "attend"))
    page = rng.choice((16, 32, 64, 128))
    if op == "grow":
        return dict(op=op, batch=_log(rng, 1, 512), page=page, held=_log(rng, 1, 8192), new=_log(rng, 1, 1024))
    dim = rng.choice((64, 96, 128, 192, 256, 384))
    if op != "attend":
        kv_heads = rng.choice((1, 2, 4, 8, 16))
        most = 16384 * 8 * 128 if op == "store" else 65536 * 4 * 128
        return dict(op=op, tokens=_log(rng, 1, most // (kv_heads * dim)), kv_heads=kv_heads, dim=dim, page=page)
    kv_heads = rng.choice((1, 2, 4, 8, 16))
    heads = kv_heads * rng.choice((1, 2, 4, 5, 7, 8, 16))
    query = rng.choice((1, 1, 1, 2, 3, 4, 8))
    longest = _log(rng, 1, 65536)
    # No more rows of keys, and no more products, than the largest listed case has.
    most = 2 ** 30 // (longest * kv_heads * dim)
    most = min(most, 2 ** 32 // (longest * heads * dim * query))
    return dict(op=op, batch=_log(rng, 1, max(1, min(128, most))), heads=heads, kv_heads=kv_heads, dim=dim, page=page, longest=longest,
                ragged=rng.random() < 0.7, query=query)


def _lengths(case):
    """Tokens of each request and new ones among them: a property of the case, so that its work is known."""
    rng = random.Random("%(batch)d %(longest)d %(query)d" % case)
    n = [case["longest"]] * case["batch"]
    q = [case["query"]] * case["batch"]
    if case["ragged"]:
        n = [case["longest"]] + [rng.randint(case["longest"] // 8, case["longest"]) for _ in n[1:]]
        q = [case["query"]] + [rng.randint(1, case["query"]) for _ in q[1:]]
    return n, q


def _held_new(case):
    rng = random.Random("%(batch)d %(held)d %(new)d" % case)
    held = [rng.randint(0, case["held"]) for _ in range(case["batch"])]
    new = [1 if case["new"] == 1 else rng.randint(0, case["new"]) for _ in range(case["batch"])]
    return held, new


def _pages(tokens, page):
    return -(-tokens // page)


# --------------------------------------------------------------- the inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    def order(n):
        return torch.randperm(n, generator=g, device="cuda")

    def ints(x, dtype=torch.int32):
        return torch.tensor(x, dtype=dtype, device="cuda")

    page = case["page"]
    if case["op"] == "grow":
        held, new = _held_new(case)
        width = _pages(case["held"] + case["new"], page)
        width = _pages(width, 8) * 8
        owned = [_pages(h, page) for h in held]
        total = sum(_pages(h + n, page) for h, n in zip(held, new))
        ids = order(total + 32).int()
        column = torch.arange(width, device="cuda")
        rows = ints(owned, torch.int64)
        first = rows.cumsum(0) - rows
        at = first[:, None] + column
        table = torch.where(column < rows[:, None], ids[at.clamp(max=len(ids) - 1)], -1)
        free = ids[sum(owned):].contiguous()
        return dict(case=case, lengths=ints(held), new=ints(new), table=table, free=free, count=ints([len(free)]),
                    page=page, tokens=sum(new) + 5)

    heads, dim = case["kv_heads"], case["dim"]
    gain = dict(key=2.0 ** -6, value=2.0 ** -7)
    # Keys have a few channels far above the others, as rotated keys do.
    wide = 1.0 + 4.0 * (torch.rand((1, heads, 1, dim), generator=g, device="cuda") < 0.03)

    def empty(pages):
        shape = (pages, heads, page)
        return dict(k=torch.zeros(shape + (dim // 2,), dtype=torch.uint8, device="cuda"),
                    ks=torch.zeros(shape + (dim // GROUP,), dtype=torch.uint8, device="cuda"),
                    v=torch.zeros(shape + (dim // 2,), dtype=torch.uint8, device="cuda"),
                    vs=torch.zeros(shape + (dim // GROUP,), dtype=torch.uint8, device="cuda"))

    def filled(pages):
        k, ks = _encode(normal(pages, heads, page, dim) * wide, gain["key"])
        v, vs = _encode(normal(pages, heads, page, dim), gain["value"])
        return dict(k=k, ks=ks, v=v, vs=vs)

    state = dict(case=case, page=page, key=gain["key"], value=gain["value"])
    if case["op"] in ("store", "load"):
        tokens = case["tokens"]
        pages = _pages(tokens, page) + 4
        where = order(pages)[:_pages(tokens, page)]
        slots = (where[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)[:tokens].contiguous()
        state["slots"] = slots
        if case["op"] == "load":
            state.update(filled(pages))
            return state
        # Keys and values as the fused projection leaves them: slices of its rows.
        fused = torch.cat([normal(tokens, 2 * heads * dim), (normal(tokens, heads, dim) * wide[:, :, 0]).reshape(tokens, -1),
                           normal(tokens, heads * dim)], 1).to(BF16)
        state["new_k"] = fused[:, 2 * heads * dim:3 * heads * dim].unflatten(1, (heads, dim))
        state["new_v"] = fused[:, 3 * heads * dim:].unflatten(1, (heads, dim))
        state.update(empty(pages))
        return state

    n, q = _lengths(case)
    needed = [_pages(x, page) for x in n]
    width = _pages(max(needed), 8) * 8
    pages = sum(needed) + 4
    ids = order(pages).int()
    rows = ints(needed, torch.int64)
    column = torch.arange(width, device="cuda")
    at = (rows.cumsum(0) - rows)[:, None] + column
    state["table"] = torch.where(column < rows[:, None], ids[at.clamp(max=pages - 1)], -1)
    state["lengths"] = ints(n)
    state["cu"] = ints([sum(q[:i]) for i in range(len(q) + 1)])
    state["most"] = max(q)
    state.update(filled(pages))
    fused = normal(sum(q), (case["heads"] + 2 * heads) * dim).to(BF16)
    state["q"] = fused[:, :case["heads"] * dim].unflatten(1, (case["heads"], dim))
    return state


# ----------------------------------------------------------- the plain form

def _encode(x, gain):
    """e2m1 codes and e4m3 scales of x [..., d]: scale = amax / 6 rounded to e4m3, codes rounded to nearest even."""
    y = (x.float() / gain).unflatten(-1, (-1, GROUP))
    a = y.abs()
    scale = (a.amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale.float()[..., None]
    r = torch.where(s > 0, a / s, 0.0)
    code = ((r > 0.25).byte() + (r >= 0.75).byte() + (r > 1.25).byte() + (r >= 1.75).byte()
            + (r > 2.5).byte() + (r >= 3.5).byte() + (r > 5.0).byte())
    code += torch.where(s > 0, torch.signbit(y), False).byte() * 8
    code = code.flatten(-2)
    return code[..., ::2] + code[..., 1::2] * 16, scale.view(torch.uint8)


def _decode(code, scale):
    """scale * code [..., d] of a cache's bytes, in 32 bits (exact)."""
    one = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=code.device)
    two = torch.stack([one.repeat(16), one.repeat_interleave(16)], 1)
    x = two.index_select(0, code.reshape(-1).int()).view(code.shape[:-1] + (-1, GROUP))
    return (x * scale.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _plain_grow(s):
    page, most, table = s["page"], s["tokens"], s["table"]
    batch, width = table.shape
    held = s["lengths"].long().clamp(min=0)
    new = s["new"].long().clamp(min=0)
    cu = torch.nn.functional.pad(new.cumsum(0), (1, 0)).clamp(max=most)
    new = cu[1:] - cu[:-1]
    owned = (held + page - 1) // page
    wanted = ((held + new + page - 1) // page).clamp(max=width)
    need = (wanted - owned).clamp(min=0)
    before = need.cumsum(0) - need
    count = s["count"].long()
    given = torch.minimum((count - before).clamp(min=0), need)
    column = torch.arange(width, device=table.device)
    source = count - 1 - (before[:, None] + column - owned[:, None])
    fresh = torch.where(source >= 0, s["free"][source.clamp(0, len(s["free"]) - 1)], -1)
    inside = (column >= owned[:, None]) & (column < wanted[:, None])
    table.copy_(torch.where(inside, fresh, table))
    placed = torch.minimum(torch.minimum(owned + given, torch.full_like(owned, width)) * page - held, new).clamp(min=0)
    token = torch.arange(most, device=table.device)
    of = torch.searchsorted(cu[1:].contiguous(), token, right=True).clamp(max=batch - 1)
    position = held[of] + token - cu[of]
    where = table[of, (position // page).clamp(max=width - 1)].long()
    fine = (token < cu[-1]) & (token - cu[of] < placed[of]) & (where >= 0)
    slots = torch.where(fine, where * page + position % page, -1)
    return slots, cu.int(), table, (held + placed).int(), (count - need.sum()).clamp(min=0).int()


def _plain_store(s):
    slots = s["slots"]
    page, offset = slots // s["page"], slots % s["page"]
    for_k, for_v = _encode(s["new_k"], s["key"]), _encode(s["new_v"], s["value"])
    s["k"][page, :, offset], s["ks"][page, :, offset] = for_k
    s["v"][page, :, offset], s["vs"][page, :, offset] = for_v


def _plain_load(s):
    slots = s["slots"]
    page, offset = slots // s["page"], slots % s["page"]
    k = _decode(s["k"][page, :, offset], s["ks"][page, :, offset]) * s["key"]
    v = _decode(s["v"][page, :, offset], s["vs"][page, :, offset]) * s["value"]
    return k.to(BF16), v.to(BF16)


def _plain_attend(s):
    case, page, cu = s["case"], s["page"], s["cu"].long()
    batch, kv, dim, most = case["batch"], case["kv_heads"], case["dim"], s["most"]
    each = case["heads"] // kv
    n = s["lengths"].long()
    q = cu[1:] - cu[:-1]
    pages = s["table"][:, :_pages(case["longest"], page)].long().clamp(min=0)

    def rows(code, scale):  # [batch, kv, tokens, dim]
        x = _decode(code[pages], scale[pages])
        return x.transpose(1, 2).reshape(batch, kv, -1, dim)

    token = torch.arange(most, device=n.device)
    at = (cu[:-1, None] + token).clamp(max=len(s["q"]) - 1)
    x = s["q"][at].float().view(batch, most, kv, each, dim).permute(0, 2, 3, 1, 4).reshape(batch, kv, -1, dim)
    score = (x @ rows(s["k"], s["ks"]).transpose(2, 3)) * (s["key"] / math.sqrt(dim))
    # Query i of a request is its token n - q + i and sees the tokens up to itself.
    last = (n - q)[:, None] + token
    seen = torch.arange(score.shape[-1], device=n.device) <= last[..., None]
    score = score.view(batch, kv, each, most, -1).masked_fill(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top.clamp(min=-3e38))
    total = p.sum(-1, keepdim=True)
    lse = (top + torch.log(total)).squeeze(-1)
    p = p / total.clamp(min=1e-37)
    o = (p.view(batch, kv, each * most, -1) @ rows(s["v"], s["vs"])) * s["value"]
    o = o.view(batch, kv, each, most, dim).permute(0, 3, 1, 2, 4).reshape(batch, most, kv * each, dim)
    lse = lse.permute(0, 3, 1, 2).reshape(batch, most, kv * each)
    mine = token < q[:, None]
    return o[mine].to(BF16), lse[mine]


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        from tiled_attention_tmem_gb300 import api
        if op == "grow":
            slots, cu, lengths, count = api.page_grow(s["lengths"], s["new"], s["table"], s["free"], s["count"], s["page"], s["tokens"])
            return slots, cu, s["table"], lengths, count
        if "cache" not in s:  # the handle that a program makes once with its pool
            s["cache"] = api.KV4Cache(s["k"], s["ks"], s["v"], s["vs"], s["key"], s["value"])
        cache = s["cache"]
        if op == "store":
            api.kv4_store(s["new_k"], s["new_v"], s["slots"], cache)
        if op != "attend":
            return api.kv4_load(s["slots"], cache)
        return api.kv4_attention(s["q"], cache, s["table"], s["lengths"], cu_q=s["cu"], max_q=s["most"])
    if op == "grow":
        return _plain_grow(s)
    if op == "store":
        _plain_store(s)
    if op != "attend":
        return _plain_load(s)
    return _plain_attend(s)


def work(case):
    if case["op"] == "grow":
        held, new = _held_new(case)
        fresh = sum(_pages(h + n, case["page"]) - _pages(h, case["page"]) for h, n in zip(held, new))
        # Lengths and counts in and out, fresh pages read and written, one slot a token; the page that a
        # request's last token sits in is read.
        return {"bytes": 16 * case["batch"] + 8 * fresh + 8 * (sum(new) + 5) + 4 * case["batch"], "flops": 0}
    row = case["kv_heads"] * (case["dim"] // 2 + case["dim"] // GROUP)
    wide = case["kv_heads"] * case["dim"] * 2
    if case["op"] in ("store", "load"):
        passes = 2 if case["op"] == "store" else 1  # written from the new rows, and read back
        return {"bytes": passes * case["tokens"] * (2 * row + 2 * wide + 8), "flops": 0}
    n, q = _lengths(case)
    io = sum(q) * case["heads"] * (4 * case["dim"] + 4)
    seen = sum(sum(max(0, x - y + 1 + i) for i in range(y)) for x, y in zip(n, q))
    table = 4 * sum(_pages(x, case["page"]) for x in n)
    return {"bytes": 2 * row * sum(n) + io + table, "flops": 4 * case["heads"] * case["dim"] * seen}


# ------------------------------------------------------------ in 64 bits

def exact(case, seed):
    """The definition in 64 bits; whole numbers (page tables) have nothing to round."""
    if case["op"] == "grow":
        return None
    s = prepare(case, seed)
    page = s["page"]

    def value(code, scale, gain):
        bits = torch.stack([code & 15, code >> 4], -1).flatten(-2)
        e, f = ((bits >> 1) & 3).double(), (bits & 1).double()
        x = torch.where(e == 0, f / 2, (1 + f / 2) * 2.0 ** (e - 1)) * (1 - 2 * (bits >> 3).double())
        e, f = ((scale >> 3) & 15).double(), (scale & 7).double()
        t = torch.where(e == 0, f * 2.0 ** -9, (1 + f / 8) * 2.0 ** (e - 7))
        return x * t.repeat_interleave(GROUP, -1) * gain

    def rounded(x, gain):
        y = x.double().unflatten(-1, (-1, GROUP)) / gain
        t = y.abs().amax(-1, keepdim=True) / 6
        step = 2.0 ** (torch.floor(torch.log2(t.clamp(min=2.0 ** -60))).clamp(min=-6) - 3)
        t = (torch.round(t / step) * step).clamp(max=448.0)
        grid = torch.tensor(MAGNITUDES, dtype=torch.float64, device="cuda")
        away = (y.abs()[..., None] - grid * t[..., None]).abs()
        # The nearest of the eight; of two as near, the one of even index.
        away = torch.where(away == away.amin(-1, keepdim=True), torch.tensor([0, 4, 1, 5, 2, 6, 3, 7], device="cuda"), 9)
        near = grid[away.argmin(-1)] * t
        return (torch.where(y < 0, -near, near) * gain).flatten(-2)

    if case["op"] == "store":
        return rounded(s["new_k"], s["key"]), rounded(s["new_v"], s["value"])
    if case["op"] == "load":
        at = s["slots"] // page, slice(None), s["slots"] % page
        return value(s["k"][at], s["ks"][at], s["key"]), value(s["v"][at], s["vs"][at], s["value"])
    n, q = _lengths(case)
    kv, dim, each, done, o, lse = case["kv_heads"], case["dim"], case["heads"] // case["kv_heads"], 0, [], []
    for b in range(case["batch"]):
        pages = s["table"][b, :_pages(n[b], page)].long()
        k, v = (value(s[c][pages], s[c + "s"][pages], s[x]).transpose(0, 1).reshape(kv, -1, dim)[:, :n[b]]
                for c, x in (("k", "key"), ("v", "value")))
        for i in range(q[b]):
            left = max(0, n[b] - q[b] + 1 + i)
            x = s["q"][done + i].double().view(kv, each, dim)
            score = x @ k[:, :left].transpose(1, 2) / math.sqrt(dim)
            lse.append(torch.logsumexp(score, -1).reshape(-1))
            o.append((torch.exp(score - lse[-1].view(kv, each, 1).clamp(min=-1e300)) @ v[:, :left]).reshape(-1, dim))
        done += q[b]
    return torch.stack(o), torch.stack(lse)
