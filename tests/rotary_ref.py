"""Plain 64-bit restatement of the norms and rotation of queries and keys (torch, any device)."""

import torch


def table(positions, turned, base=10000.0, device="cpu"):
    """fp32 [positions, turned]: cosines, then sines, taken in 64 bits."""
    i = torch.arange(0, turned, 2, dtype=torch.float64, device=device)
    a = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * base ** (-i / max(turned, 1))
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def channels(turned, interleaved, device):
    i = torch.arange(turned // 2, device=device)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + turned // 2)


def live(positions, rotary):
    return (positions >= 0) & (positions < rotary.shape[0])


def turn(x, rotary, positions, interleaved, back=False):
    """(turned x, the sums of magnitudes behind each value)."""
    turned = rotary.shape[1]
    at = positions.long().clamp(0, max(rotary.shape[0] - 1, 0))
    row = rotary.double()[at][:, None]
    c, s = row[..., :turned // 2], row[..., turned // 2:]
    if back:
        s = -s
    a, b = channels(turned, interleaved, x.device)
    y, size = x.clone(), x.abs()
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    size[..., a], size[..., b] = (x[..., a] * c).abs() + (x[..., b] * s).abs(), (x[..., b] * c).abs() + (x[..., a] * s).abs()
    return y, size


def forward(x, w, eps, rotary, positions, interleaved):
    """x [T, heads, d]: (y, sums of magnitudes), 64 bits."""
    n = x.double()
    if w is not None:
        n = n * (n.square().mean(-1, keepdim=True) + eps) ** -0.5 * w.double()
    return turn(n, rotary, positions, interleaved)


def backward(dy, x, w, eps, rotary, positions, interleaved):
    """(dx, its sums of magnitudes, dw, its sum of magnitudes); tokens without a position have none."""
    mine = live(positions, rotary)[:, None, None]
    g, size = turn(dy.double() * mine, rotary, positions, interleaved, back=True)
    if w is None:
        return g, size, None, None
    x = x.double()
    r = (x.square().mean(-1, keepdim=True) + eps) ** -0.5
    unit = x * r
    z = g * w.double()
    zs = size * w.double().abs()
    dx = r * (z - unit * (unit * z).mean(-1, keepdim=True))
    dxs = r * (zs + unit.abs() * (unit.abs() * zs).mean(-1, keepdim=True))
    unit, mask = torch.where(mine, unit, 0.0), mine.expand_as(dx)
    return (torch.where(mask, dx, 0.0), torch.where(mask, dxs, 0.0), (g * unit).sum((0, 1)),
            (size * unit.abs()).sum((0, 1)))


# A norm's factor: a sum of d <= 384 squares in 21 roundings at most (16 one after the other, then a
# tree), a product, a sum, rsqrtf to 2^-22: below 2^-19 of itself; its products with the channel and the
# weight, the rotation's products and sum add 2^-24 each; the mean of a gradient the like again.  2^-17
# of the sums of magnitudes bounds all of it, and the result is rounded to bf16 once.
OFF = 2.0 ** -17


def check(got, ref, size, what=""):
    tol = 2.0 ** -8 * (ref.abs() + OFF * size) + OFF * size + 1e-30
    far = ((got.double() - ref).abs() / tol)
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    assert got.numel() == 0 or float(far.max()) <= 1, f"{what}: off by {float(far.max()):.2f} of its bound"


def check_weight(got, ref, size, rows, what=""):
    """Sums of `rows` terms in fp32: 2^-24 of the magnitudes for each, at most."""
    far = (got.double() - ref).abs() / ((OFF + rows * 2.0 ** -24) * size + 1e-30)
    assert bool(torch.isfinite(got).all()) and float(far.max()) <= 1, f"{what}: off by {float(far.max()):.2f} of its bound"
