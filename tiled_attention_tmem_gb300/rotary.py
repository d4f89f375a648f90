"""Norms and rotation of queries and keys: torch-tensor wrappers over ``include/fa_packed.h``.

Marshalling only, like ``serving``, whose checks it shares (``api`` offers these names too).  Each is one
pass over q and k: as it is for training, with its gradients, and on the way into the paged 4-bit
cache for serving.
"""

from __future__ import annotations

import functools

from . import binding as _b
from .packed import _device_index, _f32, _workspace
from .serving import (_BF16, _F32, _I32, _MOST, KV4Cache, _On, _Tensor, _check, _check_sizes, _current_device,
                      _current_stream, _dense, _empty, _rows, _slot_count)


def _angles(rotary, positions, T, d, index):
    """Address and shape of the table, address of the positions."""
    if not (isinstance(rotary, _Tensor) and rotary.dtype is _F32 and rotary.dim() == 2 and rotary.get_device() == index
            and rotary.is_contiguous()):
        _dense(rotary, "rotary", _F32, (None, None), index)
    many, turned = rotary.shape
    if turned > d or turned % 32:
        raise ValueError(f"rotary has {turned} columns: a multiple of 32, at most {d}, can be turned")
    if many > _MOST:
        _check_sizes(many)
    if not (isinstance(positions, _Tensor) and positions.dtype is _I32 and positions.shape == (T,)
            and positions.get_device() == index and positions.is_contiguous()):
        _dense(positions, "positions", _I32, (T,), index)
    return rotary.data_ptr(), many, turned, positions.data_ptr()


def _weight(w, name, d, index):
    if w is None:
        return 0
    if not (isinstance(w, _Tensor) and w.dtype is _BF16 and w.shape == (d,) and w.get_device() == index
            and w.is_contiguous()):
        _dense(w, name, _BF16, (d,), index)
    return w.data_ptr()


def _pair(q, k, index):
    qs, ks = _rows(q, "q", None, index), _rows(k, "k", None, index)
    T, H, d = q.shape
    if k.shape[0] != T or k.shape[2] != d:
        raise ValueError(f"q is {tuple(q.shape)}, k {tuple(k.shape)}: tokens and channels must be equal")
    return T, H, k.shape[1], d, qs, ks


def _outputs(out, names, q, k, index):
    """(tensor, strides) of the results for q and k: those given, or new ones."""
    if out is None:
        q_out, k_out = _empty(q.shape, dtype=_BF16, device=q.device), _empty(k.shape, dtype=_BF16, device=q.device)
        d = q.shape[2]
        return q_out, (q.shape[1] * d, d), k_out, (k.shape[1] * d, d)
    if len(out) != 2:
        raise ValueError(f"{names[0]} and {names[1]} are a pair")
    q_out, k_out = out
    return (q_out, _rows(q_out, names[0], q.shape, index, written=True),
            k_out, _rows(k_out, names[1], k.shape, index, written=True))


def qk_norm_rope(q, k, rotary, positions, q_weight=None, k_weight=None, eps: float = 1e-6, interleaved: bool = False,
                 out=None, stream=None):
    """Norms each head of q and k and turns it by its token's position, in one pass.

    q bf16 [T, heads, d], k bf16 [T, kv_heads, d] (token and head strides free, in eights); rotary
    fp32 [positions, turned]: the cosines of each position's turned/2 angles, then the sines; the
    first ``turned`` channels (a multiple of 32) are turned, channel i with i + turned/2, or 2i with 2i + 1 if
    ``interleaved``; positions int32 [T].  ``q_weight`` and ``k_weight``: bf16 [d] (x / rms(x) * weight,
    before the rotation), or None: no norm.  Returns (q, k) in new tensors or in ``out``, a pair that may be
    (q, k) themselves.  Tokens whose position is not in the table are left as they were there."""
    index = _device_index(q, "q")
    if stream is not None or _current_device() != index:
        with _On(index, stream):
            return qk_norm_rope(q, k, rotary, positions, q_weight, k_weight, eps, interleaved, out)
    T, H, Hkv, d, (qt, qh), (kt, kh) = _pair(q, k, index)
    table, many, turned, at = _angles(rotary, positions, T, d, index)
    wq, wk = _weight(q_weight, "q_weight", d, index), _weight(k_weight, "k_weight", d, index)
    q_out, (qot, qoh), k_out, (kot, koh) = _outputs(out, ("q", "k"), q, k, index)
    st = _b.fa_qk_norm_rope(q.data_ptr(), qt, qh, k.data_ptr(), kt, kh, q_out.data_ptr(), qot, qoh, k_out.data_ptr(), kot,
                            koh, table, at, wq, wk, many, turned, _f32(eps), bool(interleaved), T, H, Hkv, d,
                            _current_stream(index))
    if st:
        _check(st, "fa_qk_norm_rope")
    return q_out, k_out


def qk_norm_rope_workspace_bytes(tokens, heads, kv_heads, head_dim) -> int:
    """What ``qk_norm_rope_backward`` needs where there is a weight (on the current device)."""
    _check_sizes(tokens, heads, kv_heads)
    return _b.fa_qk_norm_rope_bwd_workspace_size(tokens, heads, kv_heads, head_dim)


# By shape and device, whose multiprocessors it goes by.
_sum_bytes = functools.lru_cache(maxsize=1024)(lambda *shape_and_device: _b.fa_qk_norm_rope_bwd_workspace_size(
    *shape_and_device[:-1]))


def qk_norm_rope_backward(dq, dk, q, k, rotary, positions, q_weight=None, k_weight=None, eps: float = 1e-6,
                          interleaved: bool = False, grads=None, workspace=None, stream=None):
    """Gradients of ``qk_norm_rope``: dq and dk (bf16, of its results) to (dq, dk bf16 of its inputs q
    and k, dq_weight, dk_weight fp32 [d], None where there is no weight).  ``grads``: a pair of tensors for the
    first two (which may be (dq, dk) themselves), or None; ``workspace``: a uint8 CUDA tensor of
    ``qk_norm_rope_workspace_bytes``, not shared with a concurrent call, or None.  Tokens without a position have
    gradients of zero."""
    index = _device_index(dq, "dq")
    if stream is not None or _current_device() != index:
        with _On(index, stream):
            return qk_norm_rope_backward(dq, dk, q, k, rotary, positions, q_weight, k_weight, eps, interleaved, grads,
                                         workspace)
    T, H, Hkv, d, (qt, qh), (kt, kh) = _pair(q, k, index)
    (gqt, gqh), (gkt, gkh) = _rows(dq, "dq", q.shape, index), _rows(dk, "dk", k.shape, index)
    table, many, turned, at = _angles(rotary, positions, T, d, index)
    wq, wk = _weight(q_weight, "q_weight", d, index), _weight(k_weight, "k_weight", d, index)
    q_out, (qot, qoh), k_out, (kot, koh) = _outputs(grads, ("dq", "dk"), q, k, index)
    dwq = None if q_weight is None else _empty(d, dtype=_F32, device=q.device)
    dwk = None if k_weight is None else _empty(d, dtype=_F32, device=q.device)
    need = 0 if q_weight is None and k_weight is None else _sum_bytes(T, H, Hkv, d, index)
    workspace, ws, need = _workspace(workspace, need, index, q.device)
    st = _b.fa_qk_norm_rope_bwd(dq.data_ptr(), gqt, gqh, dk.data_ptr(), gkt, gkh, q.data_ptr(), qt, qh, k.data_ptr(), kt,
                                kh, q_out.data_ptr(), qot, qoh, k_out.data_ptr(), kot, koh, table, at, wq, wk,
                                0 if dwq is None else dwq.data_ptr(), 0 if dwk is None else dwk.data_ptr(), many,
                                turned, _f32(eps), bool(interleaved), T, H, Hkv, d, ws, need, _current_stream(index))
    if st:
        _check(st, "fa_qk_norm_rope_bwd")
    return q_out, k_out, dwq, dwk


def kv4_append(q, k, v, rotary, positions, slots, cache: KV4Cache, q_weight=None, k_weight=None, eps: float = 1e-6,
               interleaved: bool = False, out=None, k_out=None, stream=None):
    """``qk_norm_rope`` of q and k, and ``kv4_store`` of the turned keys and of v, in one pass.

    q bf16 [T, heads, d], k and v bf16 [T, kv_heads, d], slots int64 [T]; the rest as there.  Returns the
    turned q (in ``out``, which may be q, or a new tensor).  ``k_out``: a tensor for the turned keys too (it may be
    k), as a prompt's attention over its own rows wants them, or None.  Tokens whose position is not in
    the table are left out; those whose slot is outside the pool (-1) are turned and not stored."""
    c = cache
    index = c.index
    if stream is not None or _current_device() != index:
        with _On(index, stream):
            return kv4_append(q, k, v, rotary, positions, slots, cache, q_weight, k_weight, eps, interleaved, out, k_out)
    T = _slot_count(slots, index)
    shape = (T, c.kv_heads, c.head_dim)
    d = c.head_dim
    qt, qh = _rows(q, "q", None, index)
    if q.shape[0] != T or q.shape[2] != d:
        raise ValueError(f"q must have shape ({T}, heads, {d}), not {tuple(q.shape)}")
    H = q.shape[1]
    kt, kh = _rows(k, "k", shape, index)
    vt, vh = _rows(v, "v", shape, index)
    table, many, turned, at = _angles(rotary, positions, T, d, index)
    wq, wk = _weight(q_weight, "q_weight", d, index), _weight(k_weight, "k_weight", d, index)
    if out is None:
        out = _empty(q.shape, dtype=_BF16, device=q.device)
        ot, oh = H * d, d
    else:
        ot, oh = _rows(out, "out", q.shape, index, written=True)
    kot, koh = (0, 0) if k_out is None else _rows(k_out, "k_out", shape, index, written=True)
    ko = 0 if k_out is None else k_out.data_ptr()
    st = _b.fa_kv4_append(c.address, q.data_ptr(), qt, qh, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, out.data_ptr(), ot,
                          oh, ko, kot, koh, table, at, wq, wk, slots.data_ptr(), many, turned, _f32(eps),
                          bool(interleaved), T, H, _current_stream(index))
    if st:
        _check(st, "fa_kv4_append")
    return out
