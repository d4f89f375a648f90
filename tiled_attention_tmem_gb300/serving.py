"""Serving from a paged 4-bit cache: torch-tensor wrappers over ``include/fa_paged.h``.

Marshalling only, like ``api`` (which offers these names too): PyTorch supplies device
memory and the stream, the CUDA library computes.  Every operand is a CUDA tensor on
the cache's (or the lengths') device, which need not be the current one.  A decoding
step makes several of these calls and each takes a few microseconds on the GPU, so the
usual case of each check is a handful of attribute reads, and only an operand that
fails it is looked at again for the reason.
"""

from __future__ import annotations

import functools

import torch

from . import binding as _b

PAGE_SIZES = (16, 32, 64, 128)
HEAD_DIMS = (64, 96, 128, 192, 256, 384)

_MOST = 2 ** 31 - 1  # (the binding would cut larger numbers to their low 32 bits)

_I32, _I64, _BF16, _F32, _U8 = torch.int32, torch.int64, torch.bfloat16, torch.float32, torch.uint8
_empty, _Tensor = torch.empty, torch.Tensor
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _current_device():
    return torch.cuda.current_device()


_current_device = getattr(torch._C, "_cuda_getDevice", None) or _current_device


class _On:
    """Makes a device and a stream current, so that what is allocated inside belongs to
    the stream that the kernels run on: a freed workspace is not reused before they end."""

    def __init__(self, index, stream):
        self.stack = [torch.cuda.device(index)]
        if stream is not None:
            # (0 is the default stream; ExternalStream(0) would be a new one.)
            s = torch.cuda.ExternalStream(stream, device=index) if stream else torch.cuda.default_stream(index)
            self.stack.append(torch.cuda.stream(s))

    def __enter__(self):
        for c in self.stack:
            c.__enter__()

    def __exit__(self, *exc):
        for c in reversed(self.stack):
            c.__exit__(*exc)


def _check(st, where):
    if st != _b.FA_OK:
        raise _b.FaError(st, where)


def _dense(t, name, dtype, shape, index=None):
    """Refuses all but a dense CUDA tensor of this dtype and shape (None: any size)."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor, not {t.dtype}")
    if t.dim() != len(shape) or any(n is not None and a != n for a, n in zip(t.shape, shape)):
        raise ValueError(f"{name} must have shape {tuple('any' if n is None else n for n in shape)}, "
                         f"not {tuple(t.shape)}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor")
    if index is not None and t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the other operands on cuda:{index}")


def _rows(t, name, shape, index, written=False):
    """Refuses all but a CUDA bf16 tensor [tokens, heads, d] with dense channels; returns its
    token and head strides (0 for a dimension of one element)."""
    if isinstance(t, _Tensor) and t.dtype is _BF16 and t.get_device() == index and t.dim() == 3:
        st, sh, sd = t.stride()
        if sd == 1 and st and sh and not (st | sh) & 7 and not written and (shape is None or t.shape == shape):
            return st, sh
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype is not _BF16 or t.dim() != 3:
        raise ValueError(f"{name} must be a CUDA bfloat16 tensor of shape [tokens, heads, d]")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.get_device() != index:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA bfloat16 tensor")
        raise ValueError(f"{name} is on {t.device}, the other operands on cuda:{index}")
    tokens, heads, d = t.shape
    st, sh, sd = t.stride()
    if sd != 1 and d > 1:
        raise ValueError(f"{name}: the channels must be dense")
    st, sh = st if tokens > 1 else 0, sh if heads > 1 else 0
    if written:
        reach = d  # elements that the dimensions inside this one span
        for stride, n in sorted(((st, tokens), (sh, heads))):
            if n > 1 and stride < reach:
                raise ValueError(f"{name}: its rows overlap")
            reach += stride * (n - 1)
    return st, sh


def _check_sizes(*sizes):
    if max(sizes) > _MOST:
        raise ValueError("sizes must be below 2^31")


def _check_pages(per_request, table, page_size, num_tokens):
    if page_size not in PAGE_SIZES:
        raise ValueError(f"page_size must be one of {PAGE_SIZES}")
    if not 0 <= num_tokens <= _MOST:
        raise ValueError("num_tokens must not be negative, nor 2^31 or more")
    first, name = per_request[0]
    if not isinstance(first, _Tensor) or first.dim() != 1:
        raise ValueError(f"{name} must be a 1-D int32 tensor")
    index = first.get_device() if first.is_cuda else None
    for t, name in per_request:
        _dense(t, name, _I32, first.shape, index)
    _dense(table, "table", _I32, (first.shape[0], None), index)
    _check_sizes(*table.shape)


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
    try:
        index = lengths.get_device()
        (B,), (rows, width) = lengths.shape, table.shape
        fine = (index >= 0 and rows == B and lengths.dtype is _I32 and new_tokens.dtype is _I32 and table.dtype is _I32
                and free_pages.dtype is _I32 and free_count.dtype is _I32 and new_tokens.shape == (B,)
                and free_count.shape == (1,) and free_pages.dim() == 1 and page_size in PAGE_SIZES and num_tokens >= 0
                and max(B, width, num_tokens, free_pages.shape[0]) <= _MOST
                and new_tokens.get_device() == index and table.get_device() == index
                and free_pages.get_device() == index and free_count.get_device() == index
                and lengths.is_contiguous() and new_tokens.is_contiguous() and table.is_contiguous()
                and free_pages.is_contiguous())
    except (AttributeError, TypeError, ValueError):
        fine = False
    if not fine:
        _check_pages([(lengths, "lengths"), (new_tokens, "new_tokens")], table, page_size, num_tokens)
        _dense(free_pages, "free_pages", _I32, (None,), lengths.get_device())
        _dense(free_count, "free_count", _I32, (1,), lengths.get_device())
        _check_sizes(free_pages.shape[0])
    if stream is not None or _current_device() != index:
        with _On(index, stream):
            return page_grow(lengths, new_tokens, table, free_pages, free_count, page_size, num_tokens)
    dev = lengths.device
    if B == 0:
        return (torch.full((num_tokens,), -1, dtype=_I64, device=dev), torch.zeros(1, dtype=_I32, device=dev),
                torch.empty_like(lengths), free_count.clone())
    slots = _empty(num_tokens, dtype=_I64, device=dev)
    cu = _empty(B + 1, dtype=_I32, device=dev)
    held = _empty(B, dtype=_I32, device=dev)
    count = _empty(1, dtype=_I32, device=dev)
    _check(_b.fa_page_grow(lengths.data_ptr(), new_tokens.data_ptr(), table.data_ptr(), B, width, page_size,
                           free_pages.data_ptr(), free_pages.shape[0], free_count.data_ptr(), num_tokens,
                           slots.data_ptr(), cu.data_ptr(), held.data_ptr(), count.data_ptr(),
                           _current_stream(index)), "fa_page_grow")
    return slots, cu, held, count


def page_slots(first, count, table, page_size, num_tokens, stream=None):
    """Slots of the tokens first[b] .. first[b] + count[b] - 1 that each request holds.
    Returns (slots int64 [num_tokens], cu int32 [B + 1]) as ``page_grow`` does."""
    _check_pages([(first, "first"), (count, "count")], table, page_size, num_tokens)
    index = first.get_device()
    if stream is not None or _current_device() != index:
        with _On(index, stream):
            return page_slots(first, count, table, page_size, num_tokens)
    B, width = table.shape
    dev = first.device
    if B == 0:
        return torch.full((num_tokens,), -1, dtype=_I64, device=dev), torch.zeros(1, dtype=_I32, device=dev)
    slots = _empty(num_tokens, dtype=_I64, device=dev)
    cu = _empty(B + 1, dtype=_I32, device=dev)
    _check(_b.fa_page_slots(first.data_ptr(), count.data_ptr(), table.data_ptr(), B, width, page_size, num_tokens,
                            slots.data_ptr(), cu.data_ptr(), _current_stream(index)), "fa_page_slots")
    return slots, cu


class KV4Cache:
    """A pool of pages of keys and values in 4 bits: per tensor, e2m1 codes uint8
    [pages, kv_heads, page_size, d/2] (even channel in the low half), e4m3 scales uint8
    [pages, kv_heads, page_size, d/16] and one gain (2^-100 to 2^100); value = gain * scale *
    code.  Choose the gain so that max|x| / (6 * gain) stays below 448; a power of two loses
    nothing.  The arrays' contents may change, the arrays and gains are those given here."""

    __slots__ = ("k_codes", "k_scales", "v_codes", "v_scales", "k_gain", "v_gain", "device", "index", "pages",
                 "kv_heads", "page_size", "head_dim", "descriptor", "address")

    def __init__(self, k_codes, k_scales, v_codes, v_scales, k_gain: float = 1.0, v_gain: float = 1.0):
        _dense(k_codes, "k_codes", _U8, (None,) * 4)
        index = k_codes.get_device()
        pages, heads, page, half = k_codes.shape
        _check_sizes(pages, heads)
        if page not in PAGE_SIZES:
            raise ValueError(f"the page size must be one of {PAGE_SIZES}, not {page}")
        if 2 * half not in HEAD_DIMS:
            raise ValueError(f"unsupported head dimension {2 * half}")
        _dense(v_codes, "v_codes", _U8, k_codes.shape, index)
        for t, name in ((k_scales, "k_scales"), (v_scales, "v_scales")):
            _dense(t, name, _U8, (pages, heads, page, half // 8), index)
        for x, name in ((k_gain, "k_gain"), (v_gain, "v_gain")):
            if not 2.0 ** -100 <= x <= 2.0 ** 100:
                raise ValueError(f"{name} must be from 2^-100 to 2^100")
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.k_gain, self.v_gain, self.device, self.index = float(k_gain), float(v_gain), k_codes.device, index
        self.pages, self.kv_heads, self.page_size, self.head_dim = pages, heads, page, 2 * half
        self.descriptor = _b.FaKv4Cache(*(t.data_ptr() for t in (k_codes, k_scales, v_codes, v_scales)), pages, page,
                                        heads, 2 * half, k_gain, v_gain)
        self.address = self.descriptor.address

    @classmethod
    def empty(cls, pages, kv_heads, page_size, head_dim, k_gain: float = 1.0, v_gain: float = 1.0, device="cuda"):
        """A cache of zeros."""
        if head_dim not in HEAD_DIMS:
            raise ValueError(f"unsupported head dimension {head_dim}")
        parts = [torch.zeros((pages, kv_heads, page_size, n), dtype=_U8, device=device)
                 for n in (head_dim // 2, head_dim // 16) * 2]
        return cls(*parts, k_gain, v_gain)


def _slot_count(slots, index):
    if not (isinstance(slots, _Tensor) and slots.dtype is _I64 and slots.dim() == 1 and slots.get_device() == index
            and slots.is_contiguous()):
        _dense(slots, "slots", _I64, (None,), index)
    T = slots.shape[0]
    if T > _MOST:
        _check_sizes(T)
    return T


def kv4_store(k, v, slots, cache: KV4Cache, stream=None):
    """Writes k and v (bf16 [T, kv_heads, d]; token and head strides free, in eights)
    into the slots (int64 [T]) of ``cache``; tokens whose slot is outside the pool
    (-1) are skipped.  The other slots must be distinct."""
    c = cache
    T = _slot_count(slots, c.index)
    shape = (T, c.kv_heads, c.head_dim)
    kt, kh = _rows(k, "k", shape, c.index)
    vt, vh = _rows(v, "v", shape, c.index)
    if stream is not None or _current_device() != c.index:
        with _On(c.index, stream):
            return kv4_store(k, v, slots, cache)
    _check(_b.fa_kv4_store(c.address, k.data_ptr(), v.data_ptr(), kt, kh, vt, vh, slots.data_ptr(), T,
                           _current_stream(c.index)), "fa_kv4_store")


def kv4_load(slots, cache: KV4Cache, stream=None):
    """Returns (k, v), bf16 [T, kv_heads, d]: what the cache holds in these slots
    (int64 [T]); zeros for a slot outside the pool (-1)."""
    c = cache
    T = _slot_count(slots, c.index)
    if stream is not None or _current_device() != c.index:
        with _On(c.index, stream):
            return kv4_load(slots, cache)
    shape = (T, c.kv_heads, c.head_dim)
    k = _empty(shape, dtype=_BF16, device=c.device)
    v = _empty(shape, dtype=_BF16, device=c.device)
    _check(_b.fa_kv4_load(c.address, slots.data_ptr(), T, k.data_ptr(), v.data_ptr(), _current_stream(c.index)),
           "fa_kv4_load")
    return k, v


def kv4_attention_workspace_bytes(batch, heads, cache: KV4Cache, width, max_q=1) -> int:
    """What ``kv4_attention`` needs for a table of ``width`` pages a request (0: none)."""
    _check_sizes(batch, heads, width, max_q)
    if _current_device() != cache.index:
        with _On(cache.index, None):
            return kv4_attention_workspace_bytes(batch, heads, cache, width, max_q)
    return _b.fa_kv4_attn_workspace_size(batch, heads, cache.kv_heads, cache.head_dim, max_q, cache.page_size, width)


# The same by shape and device (it is asked for in every call and depends on nothing else).
_workspace_bytes = functools.lru_cache(maxsize=1024)(lambda *shape_and_device: _b.fa_kv4_attn_workspace_size(
    *shape_and_device[:-1]))


def kv4_attention(q, cache: KV4Cache, table, lengths, cu_q=None, max_q: int | None = None,
                  scale: float | None = None, out=None, lse=None, workspace=None, stream=None):
    """Attention of each request's newest tokens over its cached keys and values.

    q bf16 [T, heads, d] (token and head strides free, in eights; heads a multiple of
    the cache's); table int32 [B, width]; lengths int32 [B]: tokens of each request in
    the cache, the queries' own included; cu_q int32 [B + 1]: where each request's
    queries begin in q (None: one each), of which the first ``max_q`` are computed (None:
    all; the most that a request has is the better bound).  Query
    i of a request's n sees the tokens up to lengths - n + i.  Returns (o bf16 [T, heads,
    d], lse fp32 [T, heads]); a query that sees nothing gets o = 0 and lse = -inf, rows of
    no request are left as they were (in ``out`` and ``lse``, given or new; ``out`` may be q).
    The table's width and ``max_q`` choose the kernel, so neither should be much larger than
    the longest request.  ``workspace``: a uint8 CUDA tensor of
    ``kv4_attention_workspace_bytes`` (of the same ``max_q``), not shared with a concurrent
    call, or None."""
    c = cache
    index = c.index
    if stream is not None or _current_device() != index:
        with _On(index, stream):
            return kv4_attention(q, cache, table, lengths, cu_q, max_q, scale, out, lse, workspace)
    qt, qh = _rows(q, "q", None, index)
    shape = T, H, d = q.shape
    kv = c.kv_heads
    if d != c.head_dim or (H % kv if kv else H):
        raise ValueError(f"q has {H} heads of {d} channels, the cache {kv} of {c.head_dim}")
    if not (isinstance(table, _Tensor) and table.dtype is _I32 and table.dim() == 2 and table.get_device() == index
            and table.is_contiguous()):
        _dense(table, "table", _I32, (None, None), index)
    B, width = table.shape
    if B > _MOST or width > _MOST:
        _check_sizes(B, width)
    if not (isinstance(lengths, _Tensor) and lengths.dtype is _I32 and lengths.shape == (B,)
            and lengths.get_device() == index and lengths.is_contiguous()):
        _dense(lengths, "lengths", _I32, (B,), index)
    if cu_q is not None:
        if not (isinstance(cu_q, _Tensor) and cu_q.dtype is _I32 and cu_q.shape == (B + 1,)
                and cu_q.get_device() == index and cu_q.is_contiguous()):
            _dense(cu_q, "cu_q", _I32, (B + 1,), index)
        offsets = cu_q.data_ptr()
        if max_q is None:
            max_q = T
        if max_q > _MOST:
            raise ValueError("max_q must be below 2^31")
    else:
        offsets, max_q = None, 1
        if T < B:
            raise ValueError(f"q has {T} tokens for {B} requests")
    need = _workspace_bytes(B, H, kv, d, max_q, c.page_size, width, index)
    if out is None:
        out = _empty(shape, dtype=_BF16, device=c.device)
        ot, oh = H * d, d
    else:
        ot, oh = _rows(out, "out", shape, index, written=True)
    if lse is None:
        lse = _empty((T, H), dtype=_F32, device=c.device)
    else:
        _dense(lse, "lse", _F32, (T, H), index)
    if workspace is not None:
        _dense(workspace, "workspace", _U8, (None,), index)
        if workspace.numel() < need:
            raise ValueError(f"workspace holds {workspace.numel()} bytes, {need} are needed")
        need, at = workspace.numel(), workspace.data_ptr()
    elif need:
        workspace = _empty(need, dtype=_U8, device=c.device)
        at = workspace.data_ptr()
    else:
        at = None
    st = _b.lib().fa_kv4_attn(c.address, q.data_ptr(), qt, qh, T, offsets, max_q, table.data_ptr(), width,
                              lengths.data_ptr(), B, H, d ** -0.5 if scale is None else scale, out.data_ptr(), ot, oh,
                              lse.data_ptr(), at, need, _current_stream(index))
    if st:
        _check(st, "fa_kv4_attn")
    return out, lse
