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
fallback: a native binding (``csrc/binding.cpp``) checks the arguments and
launches the library's kernels on ``stream`` (default: the current stream
of the tensors' device, whichever device is current).  Scratch memory and
outputs that a call allocates come from that stream's pool.  Where ``stream`` is
not the current one, its use of the inputs and the current stream's use of the
outputs are recorded with the allocator, so either may be dropped after the call;
a third stream's use is the caller's to record, and so is the order of the streams
(``wait_stream``).

Nothing here is recorded for autograd: outputs of inputs that require a gradient do
not (gradients come from :func:`qk_norm_rope_backward`, e.g. in an
``autograd.Function``).  What a call writes of the caller's has its version raised, so
autograd refuses a backward pass whose saved inputs were overwritten.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os

import torch


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


BINDING_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_build",
                            "_lightning_binding.so")
_binding = None


def _calls():
    """The native binding (``csrc/binding.cpp``), which checks a call's tensors
    and makes the library call; raises if it has not been built."""
    global _binding
    if _binding is None:
        if not os.path.exists(BINDING_PATH):
            raise RuntimeError(f"binding not found at {BINDING_PATH}; build it with "
                               "`python -m lightning_attention_attn_gb300.build`")
        from . import load
        load()
        name = "_lightning_binding"
        spec = importlib.util.spec_from_file_location(
            name, BINDING_PATH, loader=importlib.machinery.ExtensionFileLoader(name, BINDING_PATH))
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _binding = module
    return _binding


def _bytes(name, *args) -> int:
    from . import load
    n = int(getattr(load(), name)(*args))
    if n < 0:
        raise ValueError("invalid sizes for the workspace")
    return n


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
    return (_binding or _calls()).qk_norm_rope(q, k, positions, table, q_weight, k_weight, eps,
                                               interleaved, q_out, k_out, stream)


def qk_norm_rope_backward(q, k, positions, table, dq_out, dk_out, *, q_weight=None, k_weight=None,
                          eps: float = 1e-6, interleaved: bool = False, dq=None, dk=None,
                          workspace=None, stream=None):
    """Gradients of :func:`qk_norm_rope`: ``(dq, dk, dq_weight, dk_weight)`` from its
    inputs and the gradients of its outputs.  dq and dk have the inputs' dtype
    (``dq=dq_out`` works in place; strided outputs, e.g. slices of a fused
    gradient, are taken too); the weights' gradients are fp32 [d], or None
    without weights, and the same bits on every call."""
    return (_binding or _calls()).qk_norm_rope_backward(
        q, k, positions, table, dq_out, dk_out, q_weight, k_weight, eps, interleaved, dq, dk,
        workspace, stream)


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
    return (_binding or _calls()).paged_append(q, k, v, positions, table, k_cache, v_cache, slots,
                                               q_weight, k_weight, eps, interleaved, q_out, stream)


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
    return (_binding or _calls()).paged_decode(q, k_cache, v_cache, block_table, seq_lens, scale, out,
                                               lse, workspace, stream)


def paged_step(q, k, v, positions, table, k_cache, v_cache, slots, block_table, seq_lens, *,
               q_weight=None, k_weight=None, eps: float = 1e-6, interleaved: bool = False,
               scale: float | None = None, out=None, lse=None, workspace=None, stream=None):
    """One serving step of a softmax layer: :func:`paged_append` of each request's
    new token, then :func:`paged_decode` over the cache that now holds it (the
    queries are fp32 in between, not rounded to q's dtype).  q: [B, H, d], k, v:
    [B, Hkv, d]; ``seq_lens`` counts the new tokens.  Returns out [B, H, d]."""
    return (_binding or _calls()).paged_step(
        q, k, v, positions, table, k_cache, v_cache, slots, block_table, seq_lens, q_weight,
        k_weight, eps, interleaved, scale, out, lse, workspace, stream)


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
    and 0); cu_seqlens: int32 [B + 1] (2^31 - 1 from there on); served: bool [B].  The
    new lengths and the stack's height go to seq_lens_out and free_count_out: by
    default in place (new_lens is never an output).
    """
    return (_binding or _calls()).paged_reserve(
        block_table, seq_lens, new_lens, free_pages, free_count, page_size, num_tokens, finished,
        seq_lens_out, free_count_out, stream)
