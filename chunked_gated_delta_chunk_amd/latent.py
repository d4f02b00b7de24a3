"""Python binding of latent attention (cdr_latent_* of include/chunk_dr.h): the absorbed form over a
paged cache, for decoding.

Argument marshalling only, as in ops.py.
"""
import ctypes
from typing import Optional, Tuple

import torch

from . import ops
from .blocks import _gpu, _on, _ptr
from .ops import CDR_OK, _need, _raise, load_library

LATENT_DIM, LATENT_ROPE = 512, 64


def _part(t, name, shape):
    """A bf16 input read in place where its last dimension is dense, its other strides are
    multiples of 8 elements and its data is 16-byte aligned; else a contiguous copy."""
    _need(t, name, torch.bfloat16, shape)
    st = t.stride()
    if t.data_ptr() % 16 or (st[-1] != 1 and t.shape[-1] != 1) or any(s % 8 for s in st[:-1]):
        t = t.contiguous()
        if t.data_ptr() % 16:
            t = t.clone()
    return t


def _tokens(t):
    """t ([B, T, ...]) with its first two dimensions as one of packed tokens: (t, token stride)."""
    B, T = t.shape[:2]
    if B == 1 or T == 0:
        return t, t.stride(1)
    if T == 1:
        return t, t.stride(0)
    if t.stride(0) != T * t.stride(1):
        t = t.contiguous()
    return t, t.stride(1)


def latent_cache_write(c: torch.Tensor, k_rope: torch.Tensor, cache: torch.Tensor, slot_map: torch.Tensor) -> None:
    """Writes new tokens' latents into a paged cache, in place.

    ``c [..., 512]`` and ``k_rope [..., 64]`` bf16 of T tokens in all; ``cache [P, page, 576]`` bf16;
    ``slot_map`` int32 of T slots (:func:`build_page_tables` makes it): token t becomes row
    ``slot_map[t]`` of the cache's ``P * page`` rows, and slots outside them are skipped.  Two tokens
    with one slot give an undefined row.
    """
    lib = load_library()
    if c.dim() < 1 or k_rope.dim() < 1 or c.shape[-1] != LATENT_DIM or k_rope.shape[-1] != LATENT_ROPE:
        raise ValueError("c must be [..., 512] and k_rope [..., 64]")
    T = c.numel() // LATENT_DIM
    _need(c, "c", torch.bfloat16)
    _need(k_rope, "k_rope", torch.bfloat16, tuple(c.shape[:-1]) + (LATENT_ROPE,))
    _need(slot_map, "slot_map", torch.int32)
    if slot_map.numel() != T:
        raise ValueError(f"slot_map has {slot_map.numel()} slots for {T} tokens")
    P, page = _check_cache(cache)
    device = cache.device
    _on(device, c=c, k_rope=k_rope, slot_map=slot_map)
    stream, current = _gpu(device)
    c = _part(c.reshape(T, LATENT_DIM), "c", (T, LATENT_DIM))
    k_rope = _part(k_rope.reshape(T, LATENT_ROPE), "k_rope", (T, LATENT_ROPE))
    slot_map = slot_map.contiguous()
    with current:
        st = lib.cdr_latent_cache_write(T, P, page, _ptr(c), _ptr(k_rope), c.stride(0), k_rope.stride(0), _ptr(cache),
                                        _ptr(slot_map), stream)
    if st != CDR_OK:
        _raise(st, "latent_cache_write")


def _check_cache(cache):
    _need(cache, "cache", torch.bfloat16, dense=True)
    if cache.dim() != 3 or cache.shape[2] != LATENT_DIM + LATENT_ROPE or cache.numel() == 0:
        raise ValueError("cache must be [P, page, 576]")
    if cache.data_ptr() % 16:
        raise ValueError("cache must be 16-byte aligned")
    return cache.shape[0], cache.shape[1]


def latent_decode_workspace_bytes(N: int, T: int, H: int, varlen: bool = False) -> int:
    """Bytes of the scratch buffer that :func:`latent_decode_fwd` needs for q of N sequences with T
    tokens each (T in all when varlen) and H heads."""
    p = ops.cdr_latent_decode_problem(N, T, H, int(bool(varlen)), 1, 1, 1, 1.0)
    return load_library().cdr_latent_decode_workspace_bytes(ctypes.byref(p))


def latent_decode_fwd(q_latent: torch.Tensor, q_rope: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor,
                      seq_lens: torch.Tensor, scale: float, cu_seqlens: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None, lse_out: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Latent attention over a paged cache, in the absorbed form (the decode path).

    ``q_latent [N,T,H,512]`` (queries with the key's up-projection absorbed) and ``q_rope
    [N,T,H,64]`` bf16 of N sequences with T new tokens each, or ``[1,T,H,*]`` packed with
    ``cu_seqlens`` int32 ``[N+1]``; ``cache [P,page,576]`` bf16 (latent, then rope; page a power of
    two); ``block_table`` int32 ``[N,W]``; ``seq_lens`` int32 ``[N]``, the keys of each sequence, new
    tokens' included.  A sequence's new token i sees its first ``seq_lens - T + i + 1`` keys.  Keys
    whose page is not in the cache are masked; a row without keys gives zeros and -inf.  ``scale``
    has no default: it belongs to the width of the heads before absorption.

    Returns ``(o, lse)``: o ``[.., H, 512]`` bf16 (the weighted latents, before the value
    up-projection) and the log of the sum of exponentials ``[.., H]`` fp32.  ``out``, ``lse_out``
    and ``workspace`` (uint8, :func:`latent_decode_workspace_bytes`) optionally supply the buffers;
    rows behind the last packed sequence are left as they were in them.
    """
    lib = load_library()
    if not isinstance(q_latent, torch.Tensor) or q_latent.dim() != 4 or q_latent.shape[3] != LATENT_DIM:
        raise ValueError("q_latent must be [N, T, H, 512]")
    B, T, H = q_latent.shape[:3]
    P, page = _check_cache(cache)
    _need(block_table, "block_table", torch.int32)
    _need(seq_lens, "seq_lens", torch.int32)
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32)
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must be a 1-D tensor of N + 1 offsets")
        if B != 1:
            raise ValueError("cu_seqlens requires packed queries [1, T, H, 512]")
        N = cu_seqlens.numel() - 1
    else:
        N = B
    if block_table.dim() != 2 or block_table.shape[0] != N or block_table.shape[1] < 1:
        raise ValueError(f"block_table must be [{N}, W] with W >= 1")
    if tuple(seq_lens.shape) != (N,):
        raise ValueError(f"seq_lens must be [{N}]")
    if out is not None:
        _need(out, "out", torch.bfloat16, (B, T, H, LATENT_DIM), dense=True)
        if out.data_ptr() % 16:
            raise ValueError("out must be 16-byte aligned")
    if lse_out is not None:
        _need(lse_out, "lse_out", torch.float32, (B, T, H), dense=True)
    device = q_latent.device
    _on(device, q_rope=q_rope, cache=cache, block_table=block_table, seq_lens=seq_lens, cu_seqlens=cu_seqlens, out=out,
        lse_out=lse_out, workspace=workspace)
    qc, qct = _tokens(_part(q_latent, "q_latent", (B, T, H, LATENT_DIM)))
    qr, qrt = _tokens(_part(q_rope, "q_rope", (B, T, H, LATENT_ROPE)))
    p = ops.cdr_latent_decode_problem(N, T, H, int(cu_seqlens is not None), P, page, block_table.shape[1], float(scale))
    p.qc_stride[0], p.qc_stride[1] = qct, qc.stride(2)
    p.qr_stride[0], p.qr_stride[1] = qrt, qr.stride(2)
    ref = ctypes.byref(p)
    st = lib.cdr_latent_decode_check(ref)
    if st != CDR_OK:
        _raise(st, "latent_decode_fwd")
    stream, current = _gpu(device)
    need = lib.cdr_latent_decode_workspace_bytes(ref)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    elif workspace.numel() * workspace.element_size() < need:
        raise ValueError("workspace too small")
    elif not workspace.is_contiguous() or workspace.data_ptr() % 16:
        raise ValueError("workspace must be contiguous and 16-byte aligned")
    if out is None:
        out = torch.empty((B, T, H, LATENT_DIM), dtype=torch.bfloat16, device=device)
    if lse_out is None:
        lse_out = torch.empty((B, T, H), dtype=torch.float32, device=device)
    block_table, seq_lens = block_table.contiguous(), seq_lens.contiguous()
    cu = None if cu_seqlens is None else cu_seqlens.contiguous()
    with current:
        st = lib.cdr_latent_decode_fwd(ref, _ptr(qc), _ptr(qr), _ptr(cache), _ptr(block_table), _ptr(seq_lens),
                                       _ptr(cu), _ptr(out), _ptr(lse_out), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), stream)
    if st != CDR_OK:
        _raise(st, "latent_decode_fwd")
    return out, lse_out
