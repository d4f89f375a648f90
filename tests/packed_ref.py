"""Plain 64-bit restatements of attention over packed sequences, for its tests (torch, any device)."""

import math

import torch


def bounds(cu, T):
    """(first token, tokens) of each sequence; none where its tokens do not lie in [0, T)."""
    return [(a, b - a) if 0 <= a <= b <= T else (0, 0) for a, b in zip(cu[:-1], cu[1:])]


def attend(q, k, v, cu, scale, causal, do=None):
    """q [T, H, d], k and v [T, Hkv, d] (any type).  Returns a dict of 64-bit results: o, lse, and with
    ``do`` (dq, dk, dv), with the sums that bound their errors; NaN in rows of no sequence."""
    T, H, d = q.shape
    G = H // k.shape[1]
    f = dict(dtype=torch.float64, device=q.device)
    r = dict(o=torch.full((T, H, d), math.nan, **f), lse=torch.full((T, H), math.nan, **f),
             pv=torch.zeros((T, H, d), **f), qk=torch.zeros((T, H), **f))
    if do is not None:
        r.update(dq=torch.full((T, H, d), math.nan, **f), dk=torch.full(k.shape, math.nan, **f),
                 dv=torch.full(k.shape, math.nan, **f), edq=torch.zeros((T, H, d), **f),
                 edk=torch.zeros(k.shape, **f), edv=torch.zeros(k.shape, **f))
    for start, n in bounds(cu, T):
        if n == 0:
            continue
        at = slice(start, start + n)
        hidden = torch.ones(n, n, dtype=torch.bool, device=q.device).triu(1) if causal else None
        for h in range(H):
            x, y, z = q[at, h].double(), k[at, h // G].double(), v[at, h // G].double()
            s = x @ y.T * scale
            if causal:
                s = s.masked_fill(hidden, -math.inf)
            top = s.amax(-1, keepdim=True)
            e = torch.exp(s - top.clamp(min=-1e300))
            total = e.sum(-1, keepdim=True)
            p = torch.where(total > 0, e / total, 0.0)
            r["lse"][at, h] = (top + torch.log(total))[:, 0]
            r["o"][at, h] = o = p @ z
            r["pv"][at, h] = p @ z.abs()
            qk = x.abs() @ y.abs().T * scale
            r["qk"][at, h] = (qk if hidden is None else qk.masked_fill(hidden, 0)).amax(-1)
            if do is None:
                continue
            g = do[at, h].double()
            dp = g @ z.T
            D = (g * o).sum(-1, keepdim=True)
            ds = p * (dp - D)
            # Bounds on the errors.  P is off by e of itself, sums over keys, queries and heads by `many`
            # of their terms, D by what o is off by, dP by its fp32 sums; dS and P are rounded to bf16.
            e = score_error(r["qk"][at, h], d)[:, None]
            many = n * G * 2.0 ** -23
            off_o = 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2 * e) * (1 + 2.0 ** -7) * r["pv"][at, h]
            off = (g.abs() * off_o).sum(-1, keepdim=True) + (d + 4) * 2.0 ** -23 * (g.abs() @ z.abs().T)
            ads = p * ((2.0 ** -8 + 2 * e + many) * (dp - D).abs() + (1 + 2 * e) * off) * (1 + 2.0 ** -7)
            ap = p * (2.0 ** -8 + 2 * e + many) * (1 + 2.0 ** -7)
            for name, value in (("dk", ds.T @ x * scale), ("dv", p.T @ g), ("edk", ads.T @ x.abs() * scale),
                                ("edv", ap.T @ g.abs())):
                t = r[name][at, h // G]
                t.copy_(value if h % G == 0 else t + value)
            r["dq"][at, h] = ds @ y * scale
            r["edq"][at, h] = ads @ y.abs() * scale
    return r


def score_error(qk, d):
    """Bound on the relative error of a probability: the scores are sums of d exact products in
    fp32 (2^-23 of the sum of magnitudes each, the tensor core may truncate), times one
    factor (two roundings of 2^-24), ex2.approx and the sums and logarithms 2^-17."""
    return (d + 4) * 2.0 ** -23 * qk + 2.0 ** -17


def check_forward(o, lse, r, d, what=""):
    """Probabilities are rounded to bf16 (2^-8 of the products' magnitudes), o to bf16 once."""
    mine = ~torch.isnan(r["lse"])
    e = score_error(r["qk"], d)
    full = mine & torch.isfinite(r["lse"])
    assert bool((o[mine & ~full] == 0).all()) and bool((lse[mine & ~full] == -math.inf).all()), what
    tol_l = e + 2.0 ** -22 * r["lse"].abs()
    tol_o = 2.0 ** -8 * r["o"].abs() + ((2.0 ** -8 + 2 * e)[..., None]) * r["pv"] * (1 + 2.0 ** -7) + 1e-30
    for name, got, ref, tol in (("lse", lse, r["lse"], tol_l), ("o", o, r["o"], tol_o)):
        got, ref, tol = got[full].double(), ref[full], tol[full]
        assert bool(torch.isfinite(got).all()), f"{what}: {name} is not finite"
        if got.numel():
            far = float(((got - ref).abs() / tol).max())
            assert far <= 1, f"{what}: {name} off by {far:.2f} of its bound"


def check_backward(grads, r, what=""):
    """The bounds of ``attend`` and the one rounding of a gradient to bf16."""
    for name, got in zip(("dq", "dk", "dv"), grads):
        mine = ~torch.isnan(r[name])
        ref, off, got = r[name][mine], r["e" + name][mine], got[mine].double()
        tol = 2.0 ** -8 * ref.abs() + (1 + 2.0 ** -8) * off + 1e-30
        assert bool(torch.isfinite(got).all()), f"{what}: {name} is not finite"
        far = float(((got - ref).abs() / tol).max()) if got.numel() else 0.0
        assert far <= 1, f"{what}: {name} off by {far:.2f} of its bound"
