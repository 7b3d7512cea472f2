"""The softmax layers of a hybrid lightning-attention stack: binding of the
library's paged-cache operators (declared in ``include/lightning_attn.h``).

MiniMax-01 puts one softmax layer after every seven lightning layers.  A serving
step of such a layer is

    slots, positions, cu, served = paged_reserve(block_table, seq_lens, new_lens, ...)
    out = paged_step(q, k, v, positions, table, k_cache, v_cache, slots, block_table, seq_lens)

beside :func:`decode` of the lightning layers; a prompt enters the cache through
:func:`paged_append`.  :func:`qk_norm_rope` and its gradients also precede
:func:`prefill` and follow :func:`backward` in training.

As in the rest of the package, nothing is computed here and there is no
fallback: arguments are checked, turned into pointers, sizes and strides, and
the library's kernels are launched on ``stream`` (default: the current stream
of the tensors' device, whichever device is current).  Scratch memory and
outputs that a call allocates come from that stream's pool, so they are safe
on any stream and inside a CUDA graph.
"""
from __future__ import annotations

import ctypes

import torch

_CODES = {torch.bfloat16: 0, torch.float32: 1}
_INT32 = torch.int32


def declare(lib) -> None:
    """Argument types of the entry points this module calls."""
    p, i, l, f, c = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_int)
    rotary = [p, p, i, i, i, p, p, f]  # positions, table, rows, dim, interleaved, weights, eps
    shape = [i, i, i, i, c]            # tokens, heads, kv heads, head_dim, dtype
    cache = [p, l, p, l]
    for name, args in {
        "qk_norm_rope": [p, l, p, l] + rotary + shape + [p, l, p, l, p],
        "qk_norm_rope_backward": [p, l, p, l] + rotary + shape + [p, l] * 4 + [p, p, p, l, p],
        "paged_append": [p, l] * 3 + rotary + shape + [p, l] + cache + [p, i, i, p],
        "paged_decode": [p, l] + cache + [p, i, i, p, i, i] + shape + [f, p, p, p, l, p],
        "paged_step": [p, l] * 3 + rotary + cache + [p, p, i, i, p, i, i] + shape +
                      [f, p, p, p, l, p],
        "paged_reserve": [p, i, i, p, p, p, i, p, p, i, i, i, p, p, p, p, p, p, p],
    }.items():
        fn = getattr(lib, "lightning_attn_" + name)
        fn.argtypes, fn.restype = args, ctypes.c_int
    for name, args in {"qk_norm_rope_workspace_bytes": [i], "paged_decode_workspace_bytes": [i],
                       "paged_step_workspace_bytes": [i, i, i]}.items():
        fn = getattr(lib, "lightning_attn_" + name)
        fn.argtypes, fn.restype = args, ctypes.c_int64


class _Call:
    """Device and stream of one call: every tensor is on the device of the
    first; the call runs with that device current."""

    __slots__ = ("device", "stream", "handle", "given")

    def __init__(self, first, name, stream):
        if not isinstance(first, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if not first.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (got {first.device})")
        self.device, self.given = first.device, stream is not None
        if stream is None:
            stream = torch.cuda.current_stream(self.device)
        elif stream.device != self.device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {self.device}")
        self.stream, self.handle = stream, stream.cuda_stream

    def here(self, t, name):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.device != self.device:
            raise ValueError(f"{name} must be on {self.device} (got {t.device})")

    def empty(self, shape, dtype):
        if self.given:  # from the pool of the stream that will write it
            with torch.cuda.stream(self.stream):
                return torch.empty(shape, dtype=dtype, device=self.device)
        return torch.empty(shape, dtype=dtype, device=self.device)

    def workspace(self, workspace, need):
        """(pointer, bytes) of the scratch memory, and its tensor."""
        if workspace is None:
            workspace = self.empty(need, torch.uint8)
        else:
            self.here(workspace, "workspace")
            if not workspace.is_contiguous():
                raise ValueError("workspace must be contiguous")
        return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace

    def rows(self, t, name, tokens, heads, d, dtype):
        """(pointer, row stride) of a [tokens, heads, d] array whose tokens are
        contiguous blocks."""
        self.here(t, name)
        if t.dtype != dtype or tuple(t.shape) != (tokens, heads, d):
            raise ValueError(f"{name} must be {dtype} of shape {(tokens, heads, d)}, got {t.dtype} "
                             f"{tuple(t.shape)}")
        s0, s1, s2 = t.stride()
        if s2 != 1 or (heads > 1 and s1 != d):
            raise ValueError(f"{name}: the heads of a token must be contiguous")
        return t.data_ptr(), s0 if tokens > 1 else heads * d

    def ints(self, t, name, n):
        self.here(t, name)
        if t.dtype != _INT32 or t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 tensor of {n} elements")
        return t.data_ptr()

    def weight(self, t, name, d):
        if t is None:
            return None
        self.here(t, name)
        if t.dtype != torch.float32 or tuple(t.shape) != (d,) or not t.is_contiguous():
            raise ValueError(f"{name} must be fp32 [{d}]")
        return t.data_ptr()

    def rotary(self, positions, table, tokens):
        """positions, table pointer, rows and rotary_dim."""
        if table is None:
            if positions is not None:
                raise ValueError("positions without a rotary table")
            return None, None, 0, 0
        self.here(table, "table")
        if table.dtype != torch.float32 or table.dim() != 2 or not table.is_contiguous():
            raise ValueError("table must be a contiguous fp32 [positions, rotary_dim] tensor")
        return (self.ints(positions, "positions", tokens), table.data_ptr(), table.shape[0],
                table.shape[1])

    def cache(self, t, name, hk, d, dtype):
        """(pointer, page stride) of one half of the cache."""
        self.here(t, name)
        pages, h, page, dim = t.shape if t.dim() == 4 else (0, 0, 0, 0)
        if t.dtype != dtype or t.dim() != 4 or h != hk or dim != d:
            raise ValueError(f"{name} must be {dtype} [pages, {hk}, page_size, {d}], got {t.dtype} "
                             f"{tuple(t.shape)}")
        s0, s1, s2, s3 = t.stride()
        if s3 != 1 or (page > 1 and s2 != d) or (h > 1 and s1 != page * d):
            raise ValueError(f"{name}: a page must be contiguous")
        return t.data_ptr(), s0 if pages > 1 else h * page * d

    def table(self, t, batch):
        """(pointer, row stride, width) of the block table."""
        self.here(t, "block_table")
        if t.dtype != _INT32 or t.dim() != 2 or t.shape[0] != batch:
            raise ValueError(f"block_table must be int32 [{batch}, blocks]")
        s0, s1 = t.stride()
        if t.shape[1] > 1 and s1 != 1:
            raise ValueError("a row of block_table must be contiguous")
        return t.data_ptr(), s0 if batch > 1 else max(t.shape[1], 1), t.shape[1]

    def run(self, name, *args):
        from . import _check, load
        fn = getattr(load(), name)
        if self.device.index == torch.cuda.current_device():
            status = fn(*args, self.handle)
        else:
            with torch.cuda.device(self.device):
                status = fn(*args, self.handle)
        if status:
            _check(status, name)


def _bytes(name, *args) -> int:
    from . import load
    n = int(getattr(load(), name)(*args))
    if n < 0:
        raise ValueError("invalid sizes for the workspace")
    return n


def _dtype(t) -> int:
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype} (bf16 or fp32)")
    return code


def _shape(q, k):
    """(tokens, heads, kv heads, head_dim) of q and k (k may be None)."""
    if q.dim() != 3:
        raise ValueError("q must be [T, H, d]")
    if k is not None and (not isinstance(k, torch.Tensor) or k.dim() != 3):
        raise ValueError("k must be [T, Hkv, d]")
    t, h, d = q.shape
    return t, h, 0 if k is None else k.shape[1], d


def rotary_table(max_position: int, rotary_dim: int, *, base: float = 10000.0,
                 device=None) -> torch.Tensor:
    """fp32 [max_position, rotary_dim]: the cosines, then the sines, of
    position * base^(-2 i / rotary_dim), with the angles taken in 64 bits (at
    position 10^5 a 32-bit angle is off by up to 0.004).  Build it once per
    model; other frequency schedules make tables of the same layout."""
    if rotary_dim < 16 or rotary_dim % 16:
        raise ValueError("rotary_dim must be a multiple of 16")
    i = torch.arange(0, rotary_dim, 2, dtype=torch.float64, device=device)
    p = torch.arange(max_position, dtype=torch.float64, device=device)
    a = p[:, None] * torch.pow(torch.tensor(base, dtype=torch.float64, device=device),
                               -i / rotary_dim)
    return torch.cat([a.cos(), a.sin()], dim=1).to(torch.float32)


def qk_norm_rope(q, k, positions=None, table=None, *, q_weight=None, k_weight=None,
                 eps: float = 1e-6, interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """RMS norm of every query and key head and the position rotation, in one
    pass.  Returns ``(q_out, k_out)``.

    q: [T, H, d], k: [T, Hkv, d] or None (bf16 or fp32, d 64 or 128); the tokens of
    both may be strided (slices of one projection's output), a token's heads
    are contiguous.  positions: int32 [T]; table: :func:`rotary_table`, its
    width the rotated part of a head (both None: no rotation).  q_weight,
    k_weight: fp32 [d] (both None: no norm).  interleaved: elements 2 i and 2 i + 1
    are rotated together, instead of i and i + rotary_dim / 2.  ``q_out=q,
    k_out=k`` works in place.
    """
    call = _Call(q, "q", stream)
    t, h, hk, d = _shape(q, k)
    code = _dtype(q)
    q_in = call.rows(q, "q", t, h, d, q.dtype)
    k_in = (None, 0) if k is None else call.rows(k, "k", t, hk, d, q.dtype)
    rot = call.rotary(positions, table, t)
    w = call.weight(q_weight, "q_weight", d), call.weight(k_weight, "k_weight", d)
    if q_out is None:
        q_out = call.empty((t, h, d), q.dtype)
    if k is not None and k_out is None:
        k_out = call.empty((t, hk, d), q.dtype)
    call.run("lightning_attn_qk_norm_rope", *q_in, *k_in, *rot, int(interleaved), *w, eps,
             t, h, hk, d, code, *call.rows(q_out, "q_out", t, h, d, q.dtype),
             *((None, 0) if k is None else call.rows(k_out, "k_out", t, hk, d, q.dtype)))
    return q_out, (None if k is None else k_out)


def qk_norm_rope_backward(q, k, positions, table, dq_out, dk_out, *, q_weight=None, k_weight=None,
                          eps: float = 1e-6, interleaved: bool = False, dq=None, dk=None,
                          workspace=None, stream=None):
    """Gradients of :func:`qk_norm_rope`: ``(dq, dk, dq_weight, dk_weight)`` from its
    inputs and the gradients of its outputs.  dq and dk have the inputs' dtype
    (``dq=dq_out`` works in place; strided outputs, e.g. slices of a fused
    gradient, are taken too); the weights' gradients are fp32 [d], or None
    without weights, and the same bits on every call."""
    call = _Call(q, "q", stream)
    t, h, hk, d = _shape(q, k)
    code = _dtype(q)
    q_in = call.rows(q, "q", t, h, d, q.dtype)
    dq_in = call.rows(dq_out, "dq_out", t, h, d, q.dtype)
    k_in = dk_in = (None, 0)
    if k is not None:
        k_in = call.rows(k, "k", t, hk, d, q.dtype)
        dk_in = call.rows(dk_out, "dk_out", t, hk, d, q.dtype)
    rot = call.rotary(positions, table, t)
    w = call.weight(q_weight, "q_weight", d), call.weight(k_weight, "k_weight", d)
    if dq is None:
        dq = call.empty((t, h, d), q.dtype)
    if k is not None and dk is None:
        dk = call.empty((t, hk, d), q.dtype)
    dqw = dkw = None
    ws = (None, 0)
    if q_weight is not None:
        dqw = call.empty((d,), torch.float32)
        dkw = None if k is None else call.empty((d,), torch.float32)
        *ws, workspace = call.workspace(
            workspace, _bytes("lightning_attn_qk_norm_rope_workspace_bytes", d))
    call.run("lightning_attn_qk_norm_rope_backward", *q_in, *k_in, *rot, int(interleaved), *w, eps,
             t, h, hk, d, code, *dq_in, *dk_in, *call.rows(dq, "dq", t, h, d, q.dtype),
             *((None, 0) if k is None else call.rows(dk, "dk", t, hk, d, q.dtype)),
             None if dqw is None else dqw.data_ptr(), None if dkw is None else dkw.data_ptr(), *ws)
    return dq, (None if k is None else dk), dqw, dkw


def _qkv(call, q, k, v):
    t, h, hk, d = _shape(q, k)
    if k is None:
        raise ValueError("k must be [T, Hkv, d]")
    return (t, h, hk, d), (*call.rows(q, "q", t, h, d, q.dtype),
                           *call.rows(k, "k", t, hk, d, q.dtype),
                           *call.rows(v, "v", t, hk, d, q.dtype))


def _caches(call, k_cache, v_cache, hk, d, dtype):
    """Pointers and strides of both halves; pages and page size."""
    both = (*call.cache(k_cache, "k_cache", hk, d, dtype),
            *call.cache(v_cache, "v_cache", hk, d, dtype))
    if k_cache.shape != v_cache.shape:
        raise ValueError("k_cache and v_cache must have one shape")
    return both, k_cache.shape[0], k_cache.shape[2]


def paged_append(q, k, v, positions, table, k_cache, v_cache, slots, *, q_weight=None,
                 k_weight=None, eps: float = 1e-6, interleaved: bool = False, q_out=None,
                 stream=None):
    """:func:`qk_norm_rope` whose keys, and the values as they are, go into the
    paged cache.  Returns ``q_out``.

    v: [T, Hkv, d]; k_cache, v_cache: [pages, Hkv, page_size, d], each page
    contiguous (the two may be halves of one array); slots: int32 [T], token t
    into row slots[t] % page_size of page slots[t] // page_size.  A slot outside the
    pool (-1: padding) is skipped; the others are distinct.
    """
    call = _Call(q, "q", stream)
    code = _dtype(q)
    (t, h, hk, d), qkv = _qkv(call, q, k, v)
    rot = call.rotary(positions, table, t)
    caches, pages, page = _caches(call, k_cache, v_cache, hk, d, q.dtype)
    at = call.ints(slots, "slots", t)
    w = call.weight(q_weight, "q_weight", d), call.weight(k_weight, "k_weight", d)
    if q_out is None:
        q_out = call.empty((t, h, d), q.dtype)
    call.run("lightning_attn_paged_append", *qkv, *rot, int(interleaved), *w, eps, t, h, hk, d,
             code, *call.rows(q_out, "q_out", t, h, d, q.dtype), *caches, at, pages, page)
    return q_out


def _attention_outputs(call, out, lse, b, h, d, dtype):
    if out is None:
        out = call.empty((b, h, d), dtype)
    else:
        call.here(out, "out")
        if out.dtype != dtype or tuple(out.shape) != (b, h, d) or not out.is_contiguous():
            raise ValueError(f"out must be a contiguous {dtype} [{b}, {h}, {d}]")
    if lse is not None:
        call.here(lse, "lse")
        if lse.dtype != torch.float32 or tuple(lse.shape) != (b, h) or not lse.is_contiguous():
            raise ValueError(f"lse must be a contiguous fp32 [{b}, {h}]")
    return out, None if lse is None else lse.data_ptr()


def paged_decode_workspace_bytes(head_dim: int) -> int:
    """Bytes of workspace :func:`paged_decode` needs, whatever the batch."""
    return _bytes("lightning_attn_paged_decode_workspace_bytes", head_dim)


def paged_step_workspace_bytes(batch: int, num_heads: int, head_dim: int) -> int:
    """Bytes of workspace :func:`paged_step` needs."""
    return _bytes("lightning_attn_paged_step_workspace_bytes", batch, num_heads, head_dim)


def paged_decode(q, k_cache, v_cache, block_table, seq_lens, *, scale: float | None = None,
                 out=None, lse=None, workspace=None, stream=None):
    """Softmax attention of one new token per request over the paged cache.
    Returns out [B, H, d] in q's dtype.

    q: [B, H, d] (H a multiple of the cache's Hkv); k_cache, v_cache: [pages, Hkv,
    page_size, d]; block_table: int32 [B, blocks]; seq_lens: int32 [B], the tokens
    that request b attends to (the new one among them; 0 gives a row of zeros);
    scale: default d^-1/2; lse: optional fp32 [B, H], filled with the logarithms
    of the softmax sums; workspace: optional uint8 tensor of
    :func:`paged_decode_workspace_bytes` (a stream's calls may share one).
    """
    call = _Call(q, "q", stream)
    code = _dtype(q)
    if q.dim() != 3:
        raise ValueError("q must be [B, H, d]")
    b, h, d = q.shape
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [pages, Hkv, page_size, d]")
    hk = k_cache.shape[1]
    q_in = call.rows(q, "q", b, h, d, q.dtype)
    caches, pages, page = _caches(call, k_cache, v_cache, hk, d, q.dtype)
    bt = call.table(block_table, b)
    lens = call.ints(seq_lens, "seq_lens", b)
    out, lse_ptr = _attention_outputs(call, out, lse, b, h, d, q.dtype)
    *ws, workspace = call.workspace(workspace, paged_decode_workspace_bytes(d))
    call.run("lightning_attn_paged_decode", *q_in, *caches, *bt, lens, pages, page, b, h, hk, d,
             code, d ** -0.5 if scale is None else scale, out.data_ptr(), lse_ptr, *ws)
    return out


def paged_step(q, k, v, positions, table, k_cache, v_cache, slots, block_table, seq_lens, *,
               q_weight=None, k_weight=None, eps: float = 1e-6, interleaved: bool = False,
               scale: float | None = None, out=None, lse=None, workspace=None, stream=None):
    """One serving step of a softmax layer: :func:`paged_append` of each request's
    new token, then :func:`paged_decode` over the cache that now holds it (the
    queries stay fp32 in between, so out is rounded once).  q: [B, H, d], k, v:
    [B, Hkv, d]; ``seq_lens`` counts the new tokens.  Returns out [B, H, d]."""
    call = _Call(q, "q", stream)
    code = _dtype(q)
    (b, h, hk, d), qkv = _qkv(call, q, k, v)
    rot = call.rotary(positions, table, b)
    caches, pages, page = _caches(call, k_cache, v_cache, hk, d, q.dtype)
    at = call.ints(slots, "slots", b)
    bt = call.table(block_table, b)
    lens = call.ints(seq_lens, "seq_lens", b)
    w = call.weight(q_weight, "q_weight", d), call.weight(k_weight, "k_weight", d)
    out, lse_ptr = _attention_outputs(call, out, lse, b, h, d, q.dtype)
    *ws, workspace = call.workspace(workspace, paged_step_workspace_bytes(b, h, d))
    call.run("lightning_attn_paged_step", *qkv, *rot, int(interleaved), *w, eps, *caches, at, *bt,
             lens, pages, page, b, h, hk, d, code, d ** -0.5 if scale is None else scale,
             out.data_ptr(), lse_ptr, *ws)
    return out


def paged_reserve(block_table, seq_lens, new_lens, free_pages, free_count, page_size: int,
                  num_tokens: int, *, finished=None, seq_lens_out=None, free_count_out=None,
                  stream=None):
    """Page bookkeeping of one serving step on the GPU, from the requests' lengths.
    Returns ``(slots, positions, cu_seqlens, served)``.

    block_table: int32 [B, blocks], updated; seq_lens, new_lens: int32 [B], tokens so
    far and new ones; free_pages, free_count: int32 stack of free pages [pages] and
    its height [1]; finished: optional bool (or uint8) [B], requests whose pages go back
    to the stack first.  Requests are served in order as long as there are
    pages (a request that needs none always is); the tokens of the others get
    slot -1.  slots, positions: int32 [num_tokens] (past the last new token: -1
    and 0); cu_seqlens: int32 [B + 1]; served: bool [B].  The new lengths and the
    stack's height go to seq_lens_out and free_count_out: by default in place.
    """
    call = _Call(block_table, "block_table", stream)
    if block_table.dim() != 2:
        raise ValueError("block_table must be int32 [B, blocks]")
    b = block_table.shape[0]
    if free_pages.dim() != 1:
        raise ValueError("free_pages must be an int32 [pages] tensor")
    pages = free_pages.shape[0]
    bt = call.table(block_table, b)
    lens, new = call.ints(seq_lens, "seq_lens", b), call.ints(new_lens, "new_lens", b)
    stack = call.ints(free_pages, "free_pages", pages)
    count = call.ints(free_count, "free_count", 1)
    done = None
    if finished is not None:
        call.here(finished, "finished")
        if finished.dtype not in (torch.bool, torch.uint8) or tuple(finished.shape) != (b,) or \
                not finished.is_contiguous():
            raise ValueError(f"finished must be a contiguous bool tensor of {b} elements")
        done = finished.data_ptr()
    lens_to = lens if seq_lens_out is None else call.ints(seq_lens_out, "seq_lens_out", b)
    count_to = count if free_count_out is None else call.ints(free_count_out, "free_count_out", 1)
    # one allocation for the three int32 outputs, each on a 16-byte boundary
    # (cu_seqlens goes on to prefill(), which asks for one)
    n = (num_tokens + 3) // 4 * 4
    ints = call.empty((2 * n + b + 1,), _INT32)
    served = call.empty((b,), torch.bool)
    base = ints.data_ptr()
    call.run("lightning_attn_paged_reserve", *bt, lens, new, done, b, stack, count, pages,
             page_size, num_tokens, base, base + 4 * n, base + 8 * n, served.data_ptr(), lens_to,
             count_to)
    return ints[:num_tokens], ints[n:n + num_tokens], ints[2 * n:], served
