"""Plain 64-bit restatements of the serving operators, for their tests (numpy, CPU)."""

from __future__ import annotations

import math

import numpy as np

from tiled_attention_tmem_gb300 import inputs as I

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_value(b) -> np.ndarray:
    """Scale bytes to values: the sign bit is ignored, 0x7f reads as 480."""
    b = np.asarray(b).astype(np.int64) & 0x7F
    e, m = b >> 3, b & 7
    return np.where(e == 0, m * 2.0 ** -9, (1 + m / 8.0) * 2.0 ** (e - 7.0))


def e2m1_value(code) -> np.ndarray:
    code = np.asarray(code).astype(np.int64)
    return np.where(code & 8, -1.0, 1.0) * GRID[code & 7]


def decode(codes, scales, gain) -> np.ndarray:
    """codes [..., d/2], scales [..., d/16] (uint8) to values [..., d]."""
    both = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[:-1] + (-1,))
    return e2m1_value(both) * np.repeat(e4m3_value(scales), 16, -1) * gain


def _nearest_even(x, grid):
    """Index of the grid value nearest to x >= 0, of two as near the even index."""
    away = np.abs(x[..., None] - grid)
    best = away.min(-1, keepdims=True)
    index = np.arange(len(grid))
    return np.where(away == best, np.where(index % 2 == 0, index, index + 1000), 10 ** 6).argmin(-1)


E4M3 = e4m3_value(np.arange(0x7F))  # 0 .. 448


def encode(x, gain):
    """(codes, scales) of x [..., d] by the definition: scale = e4m3(max|y|/6), code =
    e2m1(y/scale), both to nearest even and saturating."""
    y = (np.asarray(x, np.float64) / gain).reshape(x.shape[:-1] + (x.shape[-1] // 16, 16))
    top = np.minimum(np.abs(y).max(-1) / 6.0, 448.0)
    scale = _nearest_even(top, E4M3)
    s = E4M3[scale][..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        r = np.where(s > 0, np.minimum(np.abs(y) / s, 6.0), 0.0)
    code = _nearest_even(r, GRID) | np.where((y < 0) & (s > 0), 8, 0)
    code = code.reshape(x.shape).astype(np.uint8)
    return code[..., ::2] | (code[..., 1::2] << 4), scale.astype(np.uint8)


def pages(lengths, new, table, free, count, page, T):
    """page_grow by walking the requests one by one (count None: page_slots)."""
    table = np.array(table)
    width = table.shape[1]
    slots = np.full(T, -1, np.int64)
    cu, held = [0], []
    left = 0 if count is None else max(0, min(count, len(free)))
    for b, (n, a) in enumerate(zip(lengths, new)):
        n, a = max(int(n), 0), max(int(a), 0)
        a = min(a, T - cu[-1])
        owned = -(-n // page)
        room = 0
        wanted = min(-(-(n + a) // page), width)
        if count is not None:
            for c in range(owned, wanted):
                if left > 0:
                    left -= 1
                    table[b, c] = free[left]
                    room += 1
                else:
                    table[b, c] = -1
        placed = min(max(min(owned + room, width) * page - n, 0), a)
        for i in range(a):
            pos = n + i
            col = pos // page
            if col < width and table[b, col] >= 0:
                slots[cu[-1] + i] = int(table[b, col]) * page + pos % page
        held.append(n + placed)
        cu.append(cu[-1] + a)
    return slots, np.array(cu, np.int32), table, np.array(held, np.int32), left


def attend(q, cache, table, lengths, cu, max_q, scale):
    """q fp64 [T, H, d]; cache: (k, v) decoded, [pages, Hkv, page, d].  Returns o, lse and
    the sums that bound their errors: sum_j p_j |v_j|, max_j sum_c |q_c k_jc| scale and
    sum_j |v_j|; rows that no query owns are NaN."""
    k, v = cache
    npages, kv, page, d = k.shape
    T, H, _ = q.shape
    G = H // kv
    o = np.full((T, H, d), np.nan)
    lse = np.full((T, H), np.nan)
    pv, qk, sv = np.zeros((T, H, d)), np.zeros((T, H)), np.zeros((T, H, d))
    width = table.shape[1]
    for b, n in enumerate(lengths):
        n = max(int(n), 0)
        t0, t1 = int(cu[b]), int(cu[b + 1])
        nq = min(t1 - t0, max_q)
        cols = min(-(-n // page), width)
        ids = table[b, :cols]
        fine = np.repeat((ids >= 0) & (ids < npages), page)
        at = np.clip(ids, 0, max(npages - 1, 0))
        keys = k[at].transpose(1, 0, 2, 3).reshape(kv, -1, d)
        vals = v[at].transpose(1, 0, 2, 3).reshape(kv, -1, d)
        index = np.arange(cols * page)
        for i in range(nq):
            see = fine & (index <= n - (t1 - t0) + i) & (index < n)
            for h in range(H):
                kk, vv = keys[h // G][see], vals[h // G][see]
                if len(kk) == 0:
                    o[t0 + i, h], lse[t0 + i, h] = 0.0, -math.inf
                    continue
                s = kk @ q[t0 + i, h] * scale
                top = s.max()
                p = np.exp(s - top)
                lse[t0 + i, h] = top + math.log(p.sum())
                p /= p.sum()
                o[t0 + i, h] = p @ vv
                pv[t0 + i, h] = p @ np.abs(vv)
                sv[t0 + i, h] = np.abs(vv).sum(0)
                qk[t0 + i, h] = (np.abs(kk) @ np.abs(q[t0 + i, h])).max() * scale
    return o, lse, pv, qk, sv


def tolerances(o, lse, pv, qk, sv, d):
    """Bounds on |o - ref| and |lse - ref|.

    Scores: products of f16 factors that are exact, summed in fp32 over d terms (each
    sum off by at most 2^-23 of the partial sums, which sum |q k| bounds: the tensor
    core may truncate), then one fp32 factor (2^-23): e_s = (d + 2) 2^-23 max sum|qk|.
    exp2 of them: relative error e_s and 2^-21 for ex2.approx, log2 and the sums (fp32,
    a few hundred parts of a sum at most: 2^-17 is far above them).  Probabilities are
    rounded to f16 (2^-11, but 2^-25 absolute below f16's smallest normal: they are held
    times 2^7 or more of the row's largest, so that is 2^-32 of the row's sum a key), the
    output to bf16 (2^-8)."""
    e = (d + 2) * 2.0 ** -23 * qk + 2.0 ** -17
    tol_o = 2.0 ** -8 * np.abs(o) + (2.0 ** -11 + 2 * e)[..., None] * pv + 2.0 ** -32 * sv + 1e-30
    with np.errstate(invalid="ignore"):
        tol_l = e + 2.0 ** -22 * np.where(np.isfinite(lse), np.abs(lse), 0.0)
    return tol_o, tol_l


def check(o, lse, ref, d, what=""):
    ro, rl, pv, qk, sv = ref
    own = ~np.isnan(rl)
    tol_o, tol_l = tolerances(ro, rl, pv, qk, sv, d)
    assert np.array_equal(np.isinf(lse[own]), np.isinf(rl[own])), f"{what}: empty rows differ"
    full = own & np.isfinite(rl)
    assert np.all(o[own & np.isinf(rl)] == 0), f"{what}: an empty row is not zero"
    eo, el = np.abs(o[full] - ro[full]), np.abs(lse[full] - rl[full])
    assert np.all(np.isfinite(o[full])) and np.all(np.isfinite(lse[full])), what
    assert np.all(el <= tol_l[full]), f"{what}: lse off by {el.max():.3e}, {(el / tol_l[full]).max():.2f} of its bound"
    assert np.all(eo <= tol_o[full]), f"{what}: o off by {eo.max():.3e}, {(eo / tol_o[full]).max():.2f} of its bound"


def bf16(x) -> np.ndarray:
    return I.f32_to_bf16_bits(np.asarray(x, np.float32))
