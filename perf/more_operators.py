"""Cases of attention over packed sequences and of what stands around it: norms and rotation
of queries and keys, and the rotated append to the paged 4-bit cache.

Each case is one pass, either in its plain form (elementary torch operations in 32
bits) or, with ``own``, through the calls a program makes.  Sequences of different lengths lie
one behind the other: tokens cu[b] .. cu[b + 1] - 1 are sequence b, and kv head h / (heads /
kv_heads) serves head h.  Queries, keys and values are slices of the fused projection's rows.
"""

import math
import random

import torch

own = False

BF16 = torch.bfloat16
GROUP = 16
EPS = 1e-6
PLAIN_SCORES = 2 ** 30  # scores that the plain form holds at a time


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # A few short prompts admitted together: the latency of a small call.
        dict(name="prompt_short", op="prompt", batch=4, longest=77, heads=8, kv_heads=2, dim=64, causal=True),
        # A prefill batch of ragged prompts.
        dict(name="prompt_ragged", op="prompt", batch=16, longest=2048, heads=32, kv_heads=8, dim=128, causal=True),
        # One long document.
        dict(name="prompt_long", op="prompt", batch=1, longest=16384, heads=32, kv_heads=8, dim=128, causal=True),
        # Wide heads, seven to a kv head, odd lengths.
        dict(name="prompt_wide", op="prompt", batch=5, longest=1999, heads=14, kv_heads=2, dim=256, causal=True),
        # A small encoder's step, every token sees its whole sequence, a kv head for every head.
        dict(name="train_encoder", op="train", batch=3, longest=201, heads=4, kv_heads=4, dim=96, causal=False),
        # Documents packed into a training batch.
        dict(name="train_documents", op="train", batch=12, longest=4096, heads=32, kv_heads=8, dim=128, causal=True),
        # Many short documents, narrow heads.
        dict(name="train_short", op="train", batch=64, longest=512, heads=16, kv_heads=4, dim=64, causal=True),
        # Queries and keys of one decoding step.
        dict(name="rotate_step", op="rotate", tokens=64, heads=32, kv_heads=8, dim=128, turned=128, normed=True, interleaved=False,
             train=False),
        # Queries and keys of a training batch, forward and backward.
        dict(name="rotate_train", op="rotate", tokens=16384, heads=32, kv_heads=8, dim=128, turned=128, normed=True, interleaved=False,
             train=True),
        # An odd number of tokens, part of each head turned, neighbours paired.
        dict(name="rotate_part", op="rotate", tokens=4099, heads=12, kv_heads=4, dim=96, turned=32, normed=True, interleaved=True,
             train=True),
        # The new tokens of one decoding step.
        dict(name="append_step", op="append", tokens=64, heads=32, kv_heads=8, dim=128, turned=128, interleaved=False, page=64),
        # A long prompt at once.
        dict(name="append_prompt", op="append", tokens=16384, heads=32, kv_heads=8, dim=128, turned=128, interleaved=False, page=64),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("prompt", "prompt", "train", "train", "rotate", "append"))
    dim = rng.choice((64, 96, 128, 192, 256, 384))
    kv_heads = rng.choice((1, 2, 3, 4, 8))
    heads = kv_heads * rng.choice((1, 2, 3, 4, 5, 7, 8))
    if op in ("prompt", "train"):
        longest = _log(rng, 1, 8192) if op == "prompt" else _log(rng, 2, 2048)
        # No more tokens, and no more products, than the largest listed case of the kind has.
        most = min(2 ** 25 // (longest * (heads + 2 * kv_heads) * dim) if op == "train" else 2 ** 27 // (longest * heads * dim),
                   2 ** (39 if op == "prompt" else 37) // (longest ** 2 * heads * dim))
        return dict(op=op, batch=_log(rng, 1, max(1, min(64, most))), longest=longest, heads=heads, kv_heads=kv_heads, dim=dim,
                    causal=rng.random() < 0.75)
    most = 16384 * 48 * 128 // ((heads + 2 * kv_heads) * dim)
    case = dict(op=op, tokens=_log(rng, 1, min(16384, most)), heads=heads, kv_heads=kv_heads, dim=dim,
                turned=rng.choice((32, 64, dim, dim, dim)), interleaved=rng.random() < 0.3)
    if op == "append":
        return dict(case, page=rng.choice((16, 32, 64, 128)))
    return dict(case, normed=rng.random() < 0.8, train=rng.random() < 0.6)


def _lengths(case):
    """Tokens of each sequence: a property of the case, so that its work is known."""
    rng = random.Random("%(batch)d %(longest)d" % case)
    return [case["longest"]] + [rng.randint(max(1, case["longest"] // 16), case["longest"]) for _ in range(case["batch"] - 1)]


# --------------------------------------------------------------- the inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    heads, kv, dim = case["heads"], case["kv_heads"], case["dim"]
    # Keys have a few channels far above the others.
    wide = 1.0 + 4.0 * (torch.rand((kv, dim), generator=g, device="cuda") < 0.03)
    if case["op"] in ("prompt", "train"):
        n = _lengths(case)
        tokens = sum(n)
    else:
        tokens = case["tokens"]
    fused = torch.cat([normal(tokens, heads * dim), (normal(tokens, kv, dim) * wide).reshape(tokens, -1), normal(tokens, kv * dim)],
                      1).to(BF16)
    state = dict(case=case, q=fused[:, :heads * dim].unflatten(1, (heads, dim)),
                 k=fused[:, heads * dim:(heads + kv) * dim].unflatten(1, (kv, dim)),
                 v=fused[:, (heads + kv) * dim:].unflatten(1, (kv, dim)))
    if case["op"] in ("prompt", "train"):
        state["cu"] = torch.tensor([sum(n[:b]) for b in range(len(n) + 1)], dtype=torch.int32, device="cuda")
        if case["op"] == "train":
            state["do"] = normal(tokens, heads, dim).to(BF16)
        return state

    # Cosines and sines of every position, taken in 64 bits; tokens of several requests.
    turned = case["turned"]
    angle = torch.arange(32768, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
        -torch.arange(0, turned, 2, device="cuda", dtype=torch.float64) / turned)
    state["rotary"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    state["positions"] = torch.randint(0, 32768, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    if case["op"] == "append":
        page = case["page"]
        pages = -(-tokens // page) + 4
        where = torch.randperm(pages, generator=g, device="cuda")
        state["slots"] = (where[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)[:tokens].contiguous()
        state.update(page=page, key=2.0 ** -6, value=2.0 ** -7)
        for name, size in (("kc", dim // 2), ("ks", dim // GROUP), ("vc", dim // 2), ("vs", dim // GROUP)):
            state[name] = torch.zeros((pages, kv, page, size), dtype=torch.uint8, device="cuda")
        return state
    state["wq"] = (1.0 + 0.2 * normal(dim)).to(BF16) if case["normed"] else None
    state["wk"] = (1.0 + 0.2 * normal(dim)).to(BF16) if case["normed"] else None
    if case["train"]:
        state["dq"], state["dk"] = normal(tokens, heads, dim).to(BF16), normal(tokens, kv, dim).to(BF16)
    return state


# ----------------------------------------------------------- the plain form

def _plain_attention(s):
    """Sequences padded to the longest, and as many kv heads at a time as PLAIN_SCORES allows."""
    case, cu = s["case"], s["cu"].long()
    batch, longest, kv, dim = case["batch"], case["longest"], case["kv_heads"], case["dim"]
    each, scale, train = case["heads"] // kv, 1.0 / math.sqrt(dim), case["op"] == "train"
    place = torch.arange(longest, device=cu.device)
    n = cu[1:] - cu[:-1]
    mine = place < n[:, None]
    at = torch.where(mine, cu[:-1, None] + place, 0)
    hidden = ~mine[:, None, :].expand(-1, longest, -1)
    if case["causal"]:
        hidden = hidden | (place[None, :] > place[:, None])
    hidden = hidden[:, None, None]  # [batch, 1, 1, query, key]
    got = []
    step = max(1, min(kv, PLAIN_SCORES // (batch * each * longest * longest)))
    for h in range(0, kv, step):
        def queries(x):  # [batch, heads of kv, heads of each, longest, dim]
            x = x[:, h * each:(h + step) * each].float()[at] * mine[:, :, None, None]
            return x.unflatten(2, (-1, each)).permute(0, 2, 3, 1, 4)

        def rows(x):  # [batch, heads of kv, 1, longest, dim]
            return (x[:, h:h + step].float()[at] * mine[:, :, None, None]).transpose(1, 2)[:, :, None]

        q, k, v = queries(s["q"]), rows(s["k"]), rows(s["v"])
        score = (q @ k.transpose(-1, -2)).mul_(scale).masked_fill_(hidden, -math.inf)
        top = score.amax(-1, keepdim=True).clamp_(min=-3e38)
        p = score.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        p = p.div_(total)
        lse = (top + torch.log(total)).squeeze(-1)
        o = p @ v
        out = [o, lse]
        if train:
            do = queries(s["do"])
            dv = (p.transpose(-1, -2) @ do).sum(2)
            dp = do @ v.transpose(-1, -2)
            ds = dp.sub_((o * do).sum(-1, keepdim=True)).mul_(p).mul_(scale)
            out += [ds @ k, (ds.transpose(-1, -2) @ q).sum(2), dv]
        got.append(out)

    def packed(i):  # [tokens, heads, ...] of the padded results
        x = torch.cat([out[i] for out in got], 1)
        if i < 3:
            x = x.flatten(1, 2)
        return x.transpose(1, 2)[mine]

    o, lse = packed(0).to(BF16), packed(1)
    return (o, lse) + tuple(packed(i).to(BF16) for i in (2, 3, 4)) if train else (o, lse)


def _pairs(x, turned, interleaved):
    """The two channels of each pair, and the channels that stay."""
    t, rest = x[..., :turned], x[..., turned:]
    if interleaved:
        return t[..., ::2], t[..., 1::2], rest
    return t[..., :turned // 2], t[..., turned // 2:], rest


def _joined(a, b, rest, interleaved):
    t = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([t, rest], -1)


def _angles(s):
    half = s["case"]["turned"] // 2
    row = s["rotary"][s["positions"].long()][:, None]
    return row[..., :half], row[..., half:]


def _plain_turn(s, x, w):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
    cos, sin = _angles(s)
    a, b, rest = _pairs(x, s["case"]["turned"], s["case"]["interleaved"])
    return _joined(a * cos - b * sin, b * cos + a * sin, rest, s["case"]["interleaved"]).to(BF16)


def _plain_turn_back(s, dy, x, w):
    cos, sin = _angles(s)
    a, b, rest = _pairs(dy.float(), s["case"]["turned"], s["case"]["interleaved"])
    g = _joined(a * cos + b * sin, b * cos - a * sin, rest, s["case"]["interleaved"])
    if w is None:
        return g.to(BF16), None
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    unit = x * r
    wg = g * w.float()
    return (r * (wg - unit * (unit * wg).mean(-1, keepdim=True))).to(BF16), (g * unit).sum((0, 1))


def _encode(x, gain):
    """e2m1 codes and e4m3 scales of x [..., d]: scale = amax / 6 rounded to e4m3, codes rounded to nearest even."""
    y = (x.float() / gain).unflatten(-1, (-1, GROUP))
    a = y.abs()
    scale = (a.amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    t = scale.float()[..., None]
    r = torch.where(t > 0, a / t, 0.0)
    code = ((r > 0.25).byte() + (r >= 0.75).byte() + (r > 1.25).byte() + (r >= 1.75).byte()
            + (r > 2.5).byte() + (r >= 3.5).byte() + (r > 5.0).byte())
    code += torch.where(t > 0, torch.signbit(y), False).byte() * 8
    code = code.flatten(-2)
    return code[..., ::2] + code[..., 1::2] * 16, scale.view(torch.uint8)


def _decode(code, scale, gain):
    """gain * scale * code [..., d] of a cache's bytes, rounded once."""
    one = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=code.device)
    one = torch.cat([one, -one])
    x = one[torch.stack([code & 15, code >> 4], -1).flatten(-2).long()].unflatten(-1, (-1, GROUP))
    return ((x * scale.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2) * gain).to(BF16)


def _plain_append(s):
    at = s["slots"] // s["page"], slice(None), s["slots"] % s["page"]
    s["kc"][at], s["ks"][at] = _encode(_plain_turn(s, s["k"], None), s["key"])
    s["vc"][at], s["vs"][at] = _encode(s["v"], s["value"])
    return (_plain_turn(s, s["q"], None), _decode(s["kc"][at], s["ks"][at], s["key"]),
            _decode(s["vc"][at], s["vs"][at], s["value"]))


# ------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        from tiled_attention_tmem_gb300 import api
        if op in ("prompt", "train"):
            o, lse = api.packed_attention_forward(s["q"], s["k"], s["v"], s["cu"], causal=case["causal"])
            if op == "prompt":
                return o, lse
            return (o, lse) + tuple(api.packed_attention_backward(s["q"], s["k"], s["v"], o, s["do"], lse, s["cu"],
                                                                  causal=case["causal"]))
        if op == "append":
            if "cache" not in s:  # the handle that a program makes once with its pool
                s["cache"] = api.KV4Cache(s["kc"], s["ks"], s["vc"], s["vs"], s["key"], s["value"])
            q = api.kv4_append(s["q"], s["k"], s["v"], s["rotary"], s["positions"], s["slots"], s["cache"],
                               interleaved=case["interleaved"])
            return (q,) + tuple(api.kv4_load(s["slots"], s["cache"]))
        how = dict(q_weight=s["wq"], k_weight=s["wk"], eps=EPS, interleaved=case["interleaved"])
        q, k = api.qk_norm_rope(s["q"], s["k"], s["rotary"], s["positions"], **how)
        if not case["train"]:
            return q, k
        back = api.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["rotary"], s["positions"], **how)
        return (q, k) + tuple(x for x in back if x is not None)
    if op in ("prompt", "train"):
        return _plain_attention(s)
    if op == "append":
        return _plain_append(s)
    out = _plain_turn(s, s["q"], s["wq"]), _plain_turn(s, s["k"], s["wk"])
    if case["train"]:
        (dq, dwq), (dk, dwk) = _plain_turn_back(s, s["dq"], s["q"], s["wq"]), _plain_turn_back(s, s["dk"], s["k"], s["wk"])
        out += tuple(x for x in (dq, dk, dwq, dwk) if x is not None)
    return out


def work(case):
    heads, kv, dim = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] in ("prompt", "train"):
        n = _lengths(case)
        pairs = sum(x * (x + 1) // 2 if case["causal"] else x * x for x in n)
        # q, k, v in, o and lse out; with the gradients do in and dq, dk, dv out.
        row = 4 * heads * dim + 4 * kv * dim + 4 * heads
        if case["op"] == "train":
            row += 4 * heads * dim + 4 * kv * dim
        return {"bytes": sum(n) * row + 4 * (len(n) + 1), "flops": (14 if case["op"] == "train" else 4) * heads * dim * pairs}
    tokens, fixed = case["tokens"], 4 * case["turned"] + 4  # a token's row of cosines and sines, and its position
    if case["op"] == "append":
        held = 2 * kv * (dim // 2 + dim // GROUP)  # written, and read back to bf16
        return {"bytes": tokens * (4 * heads * dim + 4 * kv * dim + 2 * held + 4 * kv * dim + fixed + 16), "flops": 0}
    rows = 2 * (heads + kv) * dim
    return {"bytes": tokens * (rows * (4 if case["train"] else 2) + fixed), "flops": 0}


# ------------------------------------------------------------ in 64 bits

def exact(case, seed):
    """The definitions in 64 bits, one sequence and kv head after the other."""
    s = prepare(case, seed)
    heads, kv, dim = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] in ("prompt", "train"):
        each, outs = heads // kv, []
        start = 0
        for n in _lengths(case):
            take = slice(start, start + n)
            start += n
            parts = []
            for h in range(kv):
                q = s["q"][take, h * each:(h + 1) * each].double().transpose(0, 1)
                k, v = s["k"][take, h].double(), s["v"][take, h].double()
                x = torch.matmul(q, k.T) / math.sqrt(dim)
                if case["causal"]:
                    x = x.masked_fill(torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1), -math.inf)
                lse = torch.logsumexp(x, -1)
                p = torch.exp(x - lse[..., None])
                o = torch.matmul(p, v)
                one = [o.transpose(0, 1), lse.T]
                if case["op"] == "train":
                    do = s["do"][take, h * each:(h + 1) * each].double().transpose(0, 1)
                    dx = p * (torch.matmul(do, v.T) - (do * o).sum(-1, keepdim=True)) / math.sqrt(dim)
                    one += [torch.matmul(dx, k).transpose(0, 1), torch.einsum("gij,gid->jd", dx, q)[:, None],
                            torch.einsum("gij,gid->jd", p, do)[:, None]]
                parts.append(one)
            outs.append([torch.cat([one[i] for one in parts], 1) for i in range(len(parts[0]))])
        return tuple(torch.cat([o[i] for o in outs]) for i in range(len(outs[0])))

    turned, half = case["turned"], case["turned"] // 2
    row = s["rotary"].double()[s["positions"].long()]
    first = torch.arange(half, device="cuda") * (2 if case["interleaved"] else 1)
    second = first + (1 if case["interleaved"] else half)

    def turn(x, back=False):
        cos, sin = row[:, None, :half], row[:, None, half:] * (-1 if back else 1)
        y = x.clone()
        y[..., first] = x[..., first] * cos - x[..., second] * sin
        y[..., second] = x[..., second] * cos + x[..., first] * sin
        return y

    def root(x):
        return (x.pow(2).sum(-1, keepdim=True) / dim + EPS).sqrt()

    if case["op"] == "append":
        # What is held in 4 bits is not computed in 64: its borders are those of the rounded key.
        return turn(s["q"].double()), None, None
    out, back, weights = [], [], []
    for x, w, dy in ((s["q"].double(), s["wq"], s.get("dq")), (s["k"].double(), s["wk"], s.get("dk"))):
        out.append(turn(x if w is None else x / root(x) * w.double()))
        if dy is not None:
            g = turn(dy.double(), True)
            if w is None:
                back.append(g)
                continue
            z = g * w.double()
            back.append(z / root(x) - x * (x * z).sum(-1, keepdim=True) / (dim * root(x) ** 3))
            weights.append((g * x / root(x)).sum((0, 1)))
    return tuple(out + back + weights)
