"""Torch-tensor convenience wrappers over the C ABI (marshalling only).

PyTorch supplies device memory and the current stream; the computation runs in
the CUDA library through ``binding``.  Tensors must be CUDA, bf16 (LSE fp32),
C-contiguous and shaped [B, H, N, d].
"""

from __future__ import annotations

import math

from . import binding as _b


def _validate(specs, device=None):
    """Rejects any operand that is not a contiguous CUDA tensor of its dtype and
    shape on one device, before a pointer of it can reach the library.  specs:
    (tensor, name, dtype, shape or None); dtypes and shapes are checked first."""
    import torch
    for t, name, dtype, shape in specs:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch tensor")
        if t.dtype != dtype:
            raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor, not {t.dtype}")
        if shape is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    for t, name, dtype, _ in specs:
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor")
        dev = device if device is not None else specs[0][0].device
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the other operands on {dev}")


def _stream(stream):
    import torch
    return stream if stream is not None else torch.cuda.current_stream().cuda_stream


def attention_forward(q, k, v, scale: float | None = None, causal: bool = False,
                      out=None, lse=None, stream=None, splits: int | None = 1, workspace=None):
    """Returns (O bf16 [B,H,N,d], LSE fp32 [B,H,N]).

    ``splits`` > 1 runs the split-KV form (``fa_fwd_splitkv``) with that many key
    parts per query block; ``None`` takes ``fa_fwd_choose_splits``.  ``workspace``
    (a uint8 CUDA tensor of ``splitkv_workspace_bytes`` or more) is allocated when
    needed and not given."""
    import torch
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q, k, v must share one [B, H, N, d] shape")
    B, H, N, d = q.shape
    specs = [(q, "q", torch.bfloat16, None), (k, "k", torch.bfloat16, q.shape), (v, "v", torch.bfloat16, q.shape)]
    if out is not None:
        specs.append((out, "out", torch.bfloat16, q.shape))
    if lse is not None:
        specs.append((lse, "lse", torch.float32, (B, H, N)))
    _validate(specs)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o = torch.empty_like(q) if out is None else out
    l = torch.empty((B, H, N), dtype=torch.float32, device=q.device) if lse is None else lse
    if splits is None:
        splits = _b.fa_fwd_choose_splits(B, H, N, d, int(causal))
    if splits == 1:
        st = _b.fa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), l.data_ptr(),
                       B, H, N, d, scale, int(causal), _stream(stream))
        if st != _b.FA_OK:
            raise _b.FaError(st, "fa_fwd")
        return o, l
    need = _b.fa_fwd_splitkv_workspace_size(B, H, N, d, splits)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    else:
        _validate([(workspace, "workspace", torch.uint8, None)], q.device)
        if workspace.numel() < need:
            raise ValueError(f"workspace holds {workspace.numel()} bytes, {need} are needed")
    st = _b.fa_fwd_splitkv(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), l.data_ptr(),
                           B, H, N, d, scale, int(causal), splits, workspace.data_ptr(),
                           workspace.numel(), _stream(stream))
    if st != _b.FA_OK:
        raise _b.FaError(st, "fa_fwd_splitkv")
    return o, l


def splitkv_workspace_bytes(B, H, N, d, splits) -> int:
    return _b.fa_fwd_splitkv_workspace_size(B, H, N, d, splits)


def workspace_bytes(B, H, N, d, variant=_b.FA_BWD_AUTO) -> int:
    return _b.fa_bwd_workspace_size(B, H, N, d, variant)


def attention_backward(q, k, v, o, do, lse, scale: float | None = None, causal: bool = False,
                       variant: int = _b.FA_BWD_AUTO, workspace=None, grads=None, stream=None):
    """Returns (dQ, dK, dV) bf16 [B,H,N,d]; ``workspace`` is a uint8 CUDA tensor or None."""
    import torch
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q, k, v, o, do must share one [B, H, N, d] shape")
    B, H, N, d = q.shape
    if grads is not None and len(grads) != 3:
        raise ValueError("grads must be (dq, dk, dv)")
    specs = [(q, "q", torch.bfloat16, None)] + [(t, n, torch.bfloat16, q.shape)
                                                for t, n in ((k, "k"), (v, "v"), (o, "o"), (do, "do"))]
    specs.append((lse, "lse", torch.float32, (B, H, N)))
    if grads is not None:
        specs += [(t, n, torch.bfloat16, q.shape) for t, n in zip(grads, ("dq", "dk", "dv"))]
    if workspace is not None:
        specs.append((workspace, "workspace", torch.uint8, None))
    _validate(specs)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    need = _b.fa_bwd_workspace_size(B, H, N, d, variant)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    elif workspace.numel() < need:
        raise ValueError(f"workspace holds {workspace.numel()} bytes, {need} are needed")
    if grads is None:
        grads = (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v))
    dq, dk, dv = grads
    st = _b.fa_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(),
                   lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                   B, H, N, d, scale, int(causal), variant,
                   workspace.data_ptr(), workspace.numel(), _stream(stream))
    if st != _b.FA_OK:
        raise _b.FaError(st, "fa_bwd")
    return dq, dk, dv


# ------------------------------------------------- serving from a paged 4-bit cache

PAGE_SIZES = (16, 32, 64, 128)


class _Launch:
    """The device and stream of a call: allocations inside belong to the stream that
    the kernels run on (so a freed workspace is not reused before they end), and the
    tensors' device is current."""

    def __init__(self, device, stream):
        import torch
        self.device, self.stream, self.stack = device, stream, []
        if not torch.cuda.is_available():
            return
        if device.index != torch.cuda.current_device():
            self.stack.append(torch.cuda.device(device))
        if stream is not None:
            self.stack.append(torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device)))

    def __enter__(self):
        import torch
        for c in self.stack:
            c.__enter__()
        return self.stream if self.stream is not None else torch.cuda.current_stream().cuda_stream

    def __exit__(self, *exc):
        for c in reversed(self.stack):
            c.__exit__(*exc)


def _check(st, where):
    if st != _b.FA_OK:
        raise _b.FaError(st, where)


def _dense(t, name, dtype, shape, device):
    """A dense CUDA tensor of this dtype and shape (None in a shape: any size)."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor, not {t.dtype}")
    if t.dim() != len(shape) or any(b is not None and a != b for a, b in zip(t.shape, shape)):
        raise ValueError(f"{name} must have shape {tuple('any' if n is None else n for n in shape)}, not {tuple(t.shape)}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the other operands on {device}")


def _rows(t, name, shape, device):
    """bf16 [tokens, heads, d] with dense channels; returns its token and head strides.
    A dimension of one element or none has no stride that matters (0 is passed)."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != torch.bfloat16 or t.dim() != 3:
        raise ValueError(f"{name} must be a CUDA bfloat16 tensor of shape [tokens, heads, d]")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA bfloat16 tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the other operands on {device}")
    st, sh, sd = t.stride()
    if sd != 1 and t.shape[2] > 1:
        raise ValueError(f"{name}: the channels must be dense")
    return (st if t.shape[0] > 1 else 0), (sh if t.shape[1] > 1 else 0)


def _page_checks(per_request, table, page_size, num_tokens):
    import torch
    if page_size not in PAGE_SIZES:
        raise ValueError(f"page_size must be one of {PAGE_SIZES}")
    if num_tokens < 0:
        raise ValueError("num_tokens must not be negative")
    first = per_request[0][0]
    if not isinstance(first, torch.Tensor) or first.dim() != 1:
        raise ValueError(f"{per_request[0][1]} must be a 1-D int32 tensor")
    for t, name in per_request:
        _dense(t, name, torch.int32, first.shape, first.device)
    _dense(table, "table", torch.int32, (first.shape[0], None), first.device)


def page_grow(lengths, new_tokens, table, free_pages, free_count, page_size, num_tokens, stream=None):
    """Pages and slots for the next ``new_tokens[b]`` tokens of each request.

    lengths, new_tokens int32 [B]; table int32 [B, width]: the pages of each request,
    whose entries for pages taken now are written in place; free_pages int32 [n] and
    free_count int32 [1]: the stack of free pages (taken from its end).  Returns
    (slots int64 [num_tokens], cu int32 [B + 1], lengths int32 [B], free_count int32
    [1]): the slot of each new token in request order (-1: none, and past the last
    one), where each request's tokens begin, and the lengths and the count after it.
    A request that got fewer tokens than it asked for (pages, width or num_tokens ran
    out) shows it in its length.  Nothing but ``table`` is changed, so the call can be
    repeated; keep the returned lengths and count for the next one."""
    import torch
    _page_checks([(lengths, "lengths"), (new_tokens, "new_tokens")], table, page_size, num_tokens)
    dev = lengths.device
    _dense(free_pages, "free_pages", torch.int32, (None,), dev)
    _dense(free_count, "free_count", torch.int32, (1,), dev)
    B, width = table.shape
    with _Launch(dev, stream) as st:
        if B == 0:
            return (torch.full((num_tokens,), -1, dtype=torch.int64, device=dev),
                    torch.zeros(1, dtype=torch.int32, device=dev), torch.empty_like(lengths), free_count.clone())
        slots = torch.empty(num_tokens, dtype=torch.int64, device=dev)
        cu = torch.empty(B + 1, dtype=torch.int32, device=dev)
        held, count = torch.empty_like(lengths), torch.empty_like(free_count)
        _check(_b.fa_page_grow(lengths.data_ptr(), new_tokens.data_ptr(), table.data_ptr(), B, width, page_size,
                               free_pages.data_ptr(), free_pages.shape[0], free_count.data_ptr(), num_tokens,
                               slots.data_ptr(), cu.data_ptr(), held.data_ptr(), count.data_ptr(), st), "fa_page_grow")
    return slots, cu, held, count


def page_slots(first, count, table, page_size, num_tokens, stream=None):
    """Slots of the tokens first[b] .. first[b] + count[b] - 1 that each request holds.
    Returns (slots int64 [num_tokens], cu int32 [B + 1]) as ``page_grow`` does."""
    import torch
    _page_checks([(first, "first"), (count, "count")], table, page_size, num_tokens)
    dev = first.device
    B, width = table.shape
    with _Launch(dev, stream) as st:
        if B == 0:
            return (torch.full((num_tokens,), -1, dtype=torch.int64, device=dev),
                    torch.zeros(1, dtype=torch.int32, device=dev))
        slots = torch.empty(num_tokens, dtype=torch.int64, device=dev)
        cu = torch.empty(B + 1, dtype=torch.int32, device=dev)
        _check(_b.fa_page_slots(first.data_ptr(), count.data_ptr(), table.data_ptr(), B, width, page_size, num_tokens,
                                slots.data_ptr(), cu.data_ptr(), st), "fa_page_slots")
    return slots, cu


class KV4Cache:
    """A pool of pages of keys and values in 4 bits: per tensor, e2m1 codes uint8
    [pages, kv_heads, page_size, d/2] (even channel in the low half), e4m3 scales uint8
    [pages, kv_heads, page_size, d/16] and one gain; value = gain * scale * code.  Choose
    the gain so that max|x| / (6 * gain) stays below 448; a power of two loses nothing."""

    __slots__ = ("k_codes", "k_scales", "v_codes", "v_scales", "k_gain", "v_gain", "device", "pages", "kv_heads",
                 "page_size", "head_dim", "pointers")

    def __init__(self, k_codes, k_scales, v_codes, v_scales, k_gain: float = 1.0, v_gain: float = 1.0):
        import torch
        _dense(k_codes, "k_codes", torch.uint8, (None,) * 4, None)
        pages, heads, page, half = k_codes.shape
        if page not in PAGE_SIZES:
            raise ValueError(f"the page size must be one of {PAGE_SIZES}, not {page}")
        dev = k_codes.device
        _dense(v_codes, "v_codes", torch.uint8, k_codes.shape, dev)
        for t, name in ((k_scales, "k_scales"), (v_scales, "v_scales")):
            _dense(t, name, torch.uint8, (pages, heads, page, half // 8), dev)
        if half % 8 or 2 * half not in (64, 96, 128, 192, 256, 384):
            raise ValueError(f"unsupported head dimension {2 * half}")
        for x, name in ((k_gain, "k_gain"), (v_gain, "v_gain")):
            if not (math.isfinite(x) and x > 0):
                raise ValueError(f"{name} must be finite and positive")
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.k_gain, self.v_gain, self.device = float(k_gain), float(v_gain), dev
        self.pages, self.kv_heads, self.page_size, self.head_dim = pages, heads, page, 2 * half
        self.pointers = tuple(t.data_ptr() for t in (k_codes, k_scales, v_codes, v_scales))

    @classmethod
    def empty(cls, pages, kv_heads, page_size, head_dim, k_gain: float = 1.0, v_gain: float = 1.0, device="cuda"):
        """A cache of zeros."""
        import torch
        shape = (pages, kv_heads, page_size)
        parts = [torch.zeros(shape + (n,), dtype=torch.uint8, device=device)
                 for n in (head_dim // 2, head_dim // 16) * 2]
        return cls(*parts, k_gain, v_gain)


def _slots(slots, device):
    import torch
    _dense(slots, "slots", torch.int64, (None,), device)
    return slots.shape[0]


def kv4_store(k, v, slots, cache: KV4Cache, stream=None):
    """Writes k and v (bf16 [T, kv_heads, d]; token and head strides free, in eights)
    into the slots (int64 [T]) of ``cache``; tokens whose slot is outside the pool
    (-1) are skipped.  The other slots must be distinct."""
    c = cache
    T = _slots(slots, c.device)
    shape = (T, c.kv_heads, c.head_dim)
    kt, kh = _rows(k, "k", shape, c.device)
    vt, vh = _rows(v, "v", shape, c.device)
    with _Launch(c.device, stream) as st:
        kc, ks, vc, vs = c.pointers
        _check(_b.fa_kv4_store(k.data_ptr(), v.data_ptr(), kt, kh, vt, vh, slots.data_ptr(), T, c.kv_heads, c.head_dim,
                               kc, ks, vc, vs, c.pages, c.page_size, c.k_gain, c.v_gain, st), "fa_kv4_store")


def kv4_load(slots, cache: KV4Cache, stream=None):
    """Returns (k, v), bf16 [T, kv_heads, d]: what the cache holds in these slots
    (int64 [T]); zeros for a slot outside the pool (-1)."""
    import torch
    c = cache
    T = _slots(slots, c.device)
    with _Launch(c.device, stream) as st:
        k = torch.empty((T, c.kv_heads, c.head_dim), dtype=torch.bfloat16, device=c.device)
        v = torch.empty_like(k)
        _check(_b.fa_kv4_load(slots.data_ptr(), T, c.kv_heads, c.head_dim, *c.pointers, c.pages, c.page_size, c.k_gain,
                              c.v_gain, k.data_ptr(), v.data_ptr(), st), "fa_kv4_load")
    return k, v


def kv4_attention_workspace_bytes(batch, heads, kv_heads, head_dim, max_q=1) -> int:
    return _b.fa_kv4_attn_workspace_size(batch, heads, kv_heads, head_dim, max_q)


def kv4_attention(q, cache: KV4Cache, table, lengths, cu_q=None, max_q: int = 1, scale: float | None = None,
                  out=None, lse=None, workspace=None, stream=None):
    """Attention of each request's newest tokens over its cached keys and values.

    q bf16 [T, heads, d] (token and head strides free, in eights; heads a multiple of
    the cache's); table int32 [B, width]; lengths int32 [B]: tokens of each request in
    the cache, the queries' own included; cu_q int32 [B + 1]: where each request's
    queries begin in q (None: one each), at most ``max_q`` of them.  Query i of a
    request's n sees the tokens up to lengths - n + i.  Returns (o bf16 [T, heads, d],
    lse fp32 [T, heads]); a query that sees nothing gets o = 0 and lse = -inf, rows of
    no request are left as they were.  ``workspace``: a uint8 CUDA tensor of
    ``kv4_attention_workspace_bytes``, not shared with a concurrent call, or None."""
    import torch
    c = cache
    qt, qh = _rows(q, "q", None, c.device)
    T, H, d = q.shape
    if d != c.head_dim or H % c.kv_heads if c.kv_heads else H:
        raise ValueError(f"q has {H} heads of {d} channels, the cache {c.kv_heads} of {c.head_dim}")
    _dense(table, "table", torch.int32, (None, None), c.device)
    B, width = table.shape
    _dense(lengths, "lengths", torch.int32, (B,), c.device)
    if cu_q is not None:
        _dense(cu_q, "cu_q", torch.int32, (B + 1,), c.device)
    else:
        max_q = 1
        if T < B:
            raise ValueError(f"q has {T} tokens for {B} requests")
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    need = _b.fa_kv4_attn_workspace_size(B, H, c.kv_heads, d, max_q)
    with _Launch(c.device, stream) as st:
        if out is None:
            out = torch.empty((T, H, d), dtype=torch.bfloat16, device=c.device)
            ot, oh = H * d, d
        else:
            ot, oh = _rows(out, "out", (T, H, d), c.device)
        if lse is None:
            lse = torch.empty((T, H), dtype=torch.float32, device=c.device)
        else:
            _dense(lse, "lse", torch.float32, (T, H), c.device)
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=c.device)
        else:
            _dense(workspace, "workspace", torch.uint8, (None,), c.device)
            if workspace.numel() < need:
                raise ValueError(f"workspace holds {workspace.numel()} bytes, {need} are needed")
        _check(_b.fa_kv4_attn(q.data_ptr(), qt, qh, T, cu_q.data_ptr() if cu_q is not None else None, max_q,
                              *c.pointers, c.pages, c.page_size, table.data_ptr(), width, lengths.data_ptr(), B, H,
                              c.kv_heads, d, scale, c.k_gain, c.v_gain, out.data_ptr(), ot, oh, lse.data_ptr(),
                              workspace.data_ptr(), workspace.numel(), st), "fa_kv4_attn")
    return out, lse


def check_device_error(stream=None):
    """Synchronises the stream and raises if a bounded in-kernel wait expired."""
    st, site = _b.fa_get_device_error(_stream(stream))
    if st != _b.FA_OK:
        raise _b.FaError(st, f"device error (site 0x{site:x})")
