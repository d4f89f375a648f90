"""Attention over packed sequences: torch-tensor wrappers over ``include/fa_packed.h``.

Marshalling only, like ``serving``, whose checks it shares (``api`` offers these names too).
Sequences of different lengths lie one behind the other in tensors [tokens, heads, d];
``cu`` (int32 [sequences + 1]) says where each begins, and stays on the GPU.
"""

from __future__ import annotations

import functools

from . import binding as _b
from .serving import (_BF16, _F32, _I32, _MOST, _U8, _On, _Tensor, _check, _check_sizes, _current_device,
                      _current_stream, _dense, _empty, _rows)


def _input(t, name, shape, index):
    """``_rows`` of an operand that is read by tiles: strides of 0 or below are refused."""
    st, sh = _rows(t, name, shape, index)
    if (st <= 0 and t.shape[0] > 1) or (sh <= 0 and t.shape[1] > 1):
        raise ValueError(f"{name}: the strides of tokens and heads must be positive")
    return st, sh


def _device_index(t, name):
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a CUDA bfloat16 tensor")
    return index


def _sequences(cu, index):
    if not (isinstance(cu, _Tensor) and cu.dtype is _I32 and cu.dim() == 1 and cu.get_device() == index
            and cu.is_contiguous()):
        _dense(cu, "cu", _I32, (None,), index)
    if not 1 <= cu.shape[0] <= _MOST:
        raise ValueError("cu must have an entry more than there are sequences")
    return cu.shape[0] - 1


def _f32(x):
    """A number to pass as fp32: one too large for it is an infinity, which the library refuses."""
    return x if -3e38 < x < 3e38 else float("inf")


def _workspace(workspace, need, index, device):
    """(tensor that keeps it alive, address, bytes) of the caller's workspace or of a new one."""
    if workspace is not None:
        _dense(workspace, "workspace", _U8, (None,), index)
        if workspace.numel() < need:
            raise ValueError(f"workspace holds {workspace.numel()} bytes, {need} are needed")
        return workspace, workspace.data_ptr(), workspace.numel()
    if need == 0:
        return None, 0, 0
    workspace = _empty(need, dtype=_U8, device=device)
    return workspace, workspace.data_ptr(), need


def packed_forward_workspace_bytes(sequences, tokens, heads, kv_heads, head_dim) -> int:
    """What ``packed_attention_forward`` needs on the current device (0: none)."""
    _check_sizes(sequences, tokens, heads, kv_heads)
    return _b.fa_packed_fwd_workspace_size(sequences, tokens, heads, kv_heads, head_dim)


# By shape and device, whose multiprocessors it goes by.
_forward_bytes = functools.lru_cache(maxsize=1024)(lambda *shape_and_device: packed_forward_workspace_bytes(
    *shape_and_device[:-1]))


def _shapes(q, k, v, index):
    qs = _input(q, "q", None, index)
    ks = _input(k, "k", None, index)
    T, H, d = q.shape
    Hkv = k.shape[1]
    if k.shape[0] != T or k.shape[2] != d or (H % Hkv if Hkv else H):
        raise ValueError(f"q is {tuple(q.shape)}, k {tuple(k.shape)}: tokens and channels must be equal, "
                         "the heads of q a multiple of those of k")
    vs = _input(v, "v", k.shape, index)
    _check_sizes(T, H)
    return T, H, Hkv, d, qs, ks, vs


def packed_attention_forward(q, k, v, cu, scale: float | None = None, causal: bool = True, out=None, lse=None,
                             workspace=None, stream=None):
    """Attention of packed sequences: token cu[b] + i of q sees the keys of its own sequence b (up to
    its own, if ``causal``).

    q bf16 [T, heads, d], k and v bf16 [T, kv_heads, d] (token and head strides free, in
    eights; heads a multiple of kv_heads, at most 32 times it); cu int32 [B + 1], not decreasing.  Returns
    (o bf16 [T, heads, d], lse fp32 [T, heads]).  Rows of no sequence are left as they were (in
    ``out`` and ``lse``, given or new), and nothing that the inputs hold there, or in another sequence,
    reaches a result.  ``workspace``: a uint8 CUDA tensor of ``packed_forward_workspace_bytes``,
    not shared with a concurrent call, or None."""
    index = _device_index(q, "q")
    if stream is not None or _current_device() != index:
        with _On(index, stream):
            return packed_attention_forward(q, k, v, cu, scale, causal, out, lse, workspace)
    T, H, Hkv, d, (qt, qh), (kt, kh), (vt, vh) = _shapes(q, k, v, index)
    B = _sequences(cu, index)
    if out is None:
        out = _empty(q.shape, dtype=_BF16, device=q.device)
        ot, oh = H * d, d
    else:
        ot, oh = _rows(out, "out", q.shape, index, written=True)
    if lse is None:
        lse = _empty((T, H), dtype=_F32, device=q.device)
    else:
        _dense(lse, "lse", _F32, (T, H), index)
    workspace, at, need = _workspace(workspace, _forward_bytes(B, T, H, Hkv, d, index), index, q.device)
    st = _b.fa_packed_fwd(q.data_ptr(), qt, qh, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, out.data_ptr(), ot, oh,
                          lse.data_ptr(), cu.data_ptr(), B, T, H, Hkv, d, d ** -0.5 if scale is None else _f32(scale),
                          bool(causal), at, need, _current_stream(index))
    if st:
        _check(st, "fa_packed_fwd")
    return out, lse


def packed_backward_workspace_bytes(sequences, tokens, heads, kv_heads, head_dim, variant=_b.FA_BWD_AUTO) -> int:
    """What ``packed_attention_backward`` needs (on the current device)."""
    _check_sizes(sequences, tokens, heads, kv_heads)
    return _b.fa_packed_bwd_workspace_size(sequences, tokens, heads, kv_heads, head_dim, variant)


_backward_bytes = functools.lru_cache(maxsize=1024)(lambda *shape_and_device: packed_backward_workspace_bytes(
    *shape_and_device[:-1]))


def packed_attention_backward(q, k, v, o, do, lse, cu, scale: float | None = None, causal: bool = True,
                              variant: int = _b.FA_BWD_AUTO, workspace=None, grads=None, stream=None):
    """Returns (dq, dk, dv) bf16 of ``packed_attention_forward``'s q, k and v, given its results o and
    lse and the gradient do (bf16 [T, heads, d], strides free like q's).  Rows of no sequence get zeros.
    ``grads``: three tensors to write, or None; ``workspace``: a uint8 CUDA tensor of
    ``packed_backward_workspace_bytes`` (of the same variant), not shared with a concurrent
    call, or None.  ``variant`` as in ``attention_backward``: the 7-GEMM form gives the same bits every time."""
    index = _device_index(q, "q")
    if stream is not None or _current_device() != index:
        with _On(index, stream):
            return packed_attention_backward(q, k, v, o, do, lse, cu, scale, causal, variant, workspace, grads)
    T, H, Hkv, d, (qt, qh), (kt, kh), (vt, vh) = _shapes(q, k, v, index)
    ot, oh = _input(o, "o", q.shape, index)
    gt, gh = _input(do, "do", q.shape, index)
    if not (isinstance(lse, _Tensor) and lse.dtype is _F32 and lse.shape == (T, H) and lse.get_device() == index
            and lse.is_contiguous()):
        _dense(lse, "lse", _F32, (T, H), index)
    B = _sequences(cu, index)
    if grads is None:
        dq = _empty(q.shape, dtype=_BF16, device=q.device)
        dk, dv = (_empty(k.shape, dtype=_BF16, device=q.device) for _ in range(2))
        (qgt, qgh), (kgt, kgh), (vgt, vgh) = (H * d, d), (Hkv * d, d), (Hkv * d, d)
    else:
        if len(grads) != 3:
            raise ValueError("grads must be (dq, dk, dv)")
        dq, dk, dv = grads
        (qgt, qgh), (kgt, kgh), (vgt, vgh) = (_rows(t, name, like.shape, index, written=True) for t, name, like in
                                              ((dq, "dq", q), (dk, "dk", k), (dv, "dv", v)))
    workspace, at, need = _workspace(workspace, _backward_bytes(B, T, H, Hkv, d, variant, index), index, q.device)
    st = _b.fa_packed_bwd(q.data_ptr(), qt, qh, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, o.data_ptr(), ot, oh,
                          do.data_ptr(), gt, gh, lse.data_ptr(), dq.data_ptr(), qgt, qgh, dk.data_ptr(), kgt, kgh,
                          dv.data_ptr(), vgt, vgh, cu.data_ptr(), B, T, H, Hkv, d,
                          d ** -0.5 if scale is None else _f32(scale), bool(causal), variant, at, need,
                          _current_stream(index))
    if st:
        _check(st, "fa_packed_bwd")
    if H == 0:  # (no work for the library: sums over no heads)
        dk.zero_(), dv.zero_()
    return dq, dk, dv
