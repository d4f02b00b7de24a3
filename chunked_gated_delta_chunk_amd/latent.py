"""Python binding of latent attention (cdr_latent_* of include/chunk_dr.h): the absorbed form over a
paged cache, for decoding, and the expanded form with its gradients, for prefill and training.

Argument marshalling only, as in ops.py.
"""
import ctypes
import math
from typing import Optional, Tuple

import torch

from . import ops
from .blocks import _apart, _launch, _need_gpu, _on, _ptr
from .ops import CDR_OK, _need, _raise, load_library

LATENT_DIM, LATENT_ROPE = 512, 64
VARLEN_FILL = 2   # CDR_VARLEN_FILL of chunk_dr.h


_STRIDE_LIMIT = 1 << 23   # elements: the kernels step over a tile's rows in 32 bits


def _part(t, name, shape):
    """A bf16 input read in place where its last dimension is dense, its other strides are multiples
    of 8 elements and its data is 16-byte aligned; else a contiguous copy.  A stride along a dimension
    of one element means nothing."""
    _need(t, name, torch.bfloat16, shape)
    if t.is_contiguous() and t.data_ptr() % 16 == 0:
        return t
    odd = t.data_ptr() % 16 or (t.stride(-1) != 1 and t.shape[-1] != 1)
    if odd or any(n > 1 and (s % 8 or s >= _STRIDE_LIMIT) for s, n in zip(t.stride()[:-1], t.shape)):
        t = t.contiguous()
        if t.data_ptr() % 16:
            t = t.clone()
    return t


def _step(t, dim):
    return t.stride(dim) if t.shape[dim] > 1 else 0


def _tokens(t):
    """t ([B, T, ...]) with its first two dimensions as one of packed tokens: (t, token stride)."""
    B, T = t.shape[:2]
    if B <= 1 or T == 0:
        return t, _step(t, 1)
    if T == 1:
        return t, _step(t, 0)
    if t.stride(0) != T * t.stride(1):
        t = t.contiguous()
    return t, t.stride(1)


def _results(p, out, lse_out, shape, device):
    """The outputs of a forward.  What packed sequences do not hold becomes zeros and -inf in those made here,
    written by the kernels (VARLEN_FILL) where both are."""
    if p.varlen and (out is None) != (lse_out is None):
        if out is None:
            out = torch.zeros(shape, dtype=torch.bfloat16, device=device)
        else:
            lse_out = torch.full(shape[:3], -math.inf, dtype=torch.float32, device=device)
    elif out is None or lse_out is None:
        if p.varlen:
            p.varlen = VARLEN_FILL
        if out is None:
            out = torch.empty(shape, dtype=torch.bfloat16, device=device)
        if lse_out is None:
            lse_out = torch.empty(shape[:3], dtype=torch.float32, device=device)
    return out, lse_out


def latent_cache_write(c: torch.Tensor, k_rope: torch.Tensor, cache: torch.Tensor, slot_map: torch.Tensor) -> None:
    """Writes new tokens' latents into a paged cache, in place.

    ``c [..., 512]`` and ``k_rope [..., 64]`` bf16 of T tokens in all; ``cache [P, page, 576]`` bf16;
    ``slot_map`` int32 of T slots (:func:`build_page_tables` makes it): token t becomes row
    ``slot_map[t]`` of the cache's ``P * page`` rows, and slots outside them are skipped.  Two tokens
    with one slot give an undefined row.  c and k_rope may be rows of the cache itself, to copy pages,
    where no slot names one of them.
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
    _need_gpu(device)
    c = _part(c.reshape(T, LATENT_DIM), "c", (T, LATENT_DIM))
    k_rope = _part(k_rope.reshape(T, LATENT_ROPE), "k_rope", (T, LATENT_ROPE))
    slot_map = slot_map.contiguous()
    _launch(device, "latent_cache_write", lib.cdr_latent_cache_write, T, P, page, _ptr(c), _ptr(k_rope), _step(c, 0),
            _step(k_rope, 0), _ptr(cache), _ptr(slot_map))


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
    up-projection) and the log of the sum of exponentials ``[.., H]`` fp32; rows that no packed
    sequence holds are zeros and -inf.  ``out``, ``lse_out`` and ``workspace`` (uint8,
    :func:`latent_decode_workspace_bytes`) optionally supply the buffers, apart from the inputs; in the
    former two such rows are left as they were.
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
    p.qc_stride[0], p.qc_stride[1] = qct, _step(qc, 2)
    p.qr_stride[0], p.qr_stride[1] = qrt, _step(qr, 2)
    ref = ctypes.byref(p)
    st = lib.cdr_latent_decode_check(ref)
    if st != CDR_OK:
        _raise(st, "latent_decode_fwd")
    if out is not None or lse_out is not None:
        _apart(dict(q_latent=qc, q_rope=qr, cache=cache, block_table=block_table, seq_lens=seq_lens, cu_seqlens=cu_seqlens),
               dict(out=out, lse_out=lse_out))
    _need_gpu(device)
    need = lib.cdr_latent_decode_workspace_bytes(ref)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    elif workspace.numel() * workspace.element_size() < need:
        raise ValueError("workspace too small")
    elif not workspace.is_contiguous() or workspace.data_ptr() % 16:
        raise ValueError("workspace must be contiguous and 16-byte aligned")
    block_table, seq_lens = block_table.contiguous(), seq_lens.contiguous()
    cu = None if cu_seqlens is None else cu_seqlens.contiguous()
    out, lse_out = _results(p, out, lse_out, (B, T, H, LATENT_DIM), device)
    _launch(device, "latent_decode_fwd", lib.cdr_latent_decode_fwd, ref, _ptr(qc), _ptr(qr), _ptr(cache),
            _ptr(block_table), _ptr(seq_lens), _ptr(cu), _ptr(out), _ptr(lse_out), _ptr(workspace),
            workspace.numel() * workspace.element_size())
    return out, lse_out


NOPE_DIM, VALUE_DIM = 128, 128
QUERY_DIM = NOPE_DIM + LATENT_ROPE


class _LatentAttn:
    """The checked inputs of the expanded form: its problem struct and the tensors it points to."""

    def __init__(self, q, k_nope, k_rope, v, scale, cu_seqlens, cu_seqlens_k, what):
        self.lib = load_library()
        if not isinstance(q, torch.Tensor) or q.dim() != 4 or q.shape[3] != QUERY_DIM:
            raise ValueError("q must be [B, T, H, 192]")
        B, T, H = q.shape[:3]
        if not isinstance(k_nope, torch.Tensor) or k_nope.dim() != 4:
            raise ValueError("k_nope must be [B, Tk, H, 128]")
        Tk = k_nope.shape[1]
        q = _part(q, "q", (B, T, H, QUERY_DIM))
        k_nope = _part(k_nope, "k_nope", (B, Tk, H, NOPE_DIM))
        k_rope = _part(k_rope, "k_rope", (B, Tk, LATENT_ROPE))
        v = _part(v, "v", (B, Tk, H, VALUE_DIM))
        N = B
        if cu_seqlens is None and cu_seqlens_k is not None:
            raise ValueError("cu_seqlens_k needs cu_seqlens")
        if cu_seqlens is not None:
            if cu_seqlens_k is None:
                if Tk != T:
                    raise ValueError("cu_seqlens_k is required where keys and queries differ in number")
                cu_seqlens_k = cu_seqlens
            for name, t in (("cu_seqlens", cu_seqlens), ("cu_seqlens_k", cu_seqlens_k)):
                _need(t, name, torch.int32)
                if t.dim() != 1 or t.numel() < 2:
                    raise ValueError(f"{name} must be a 1-D tensor of N + 1 offsets")
            N = cu_seqlens.numel() - 1
            if cu_seqlens_k.numel() != N + 1:
                raise ValueError("cu_seqlens and cu_seqlens_k differ in length")
            if B != 1:
                raise ValueError("cu_seqlens requires B == 1")
            cu_seqlens, cu_seqlens_k = cu_seqlens.contiguous(), cu_seqlens_k.contiguous()
        self.device = q.device
        _on(self.device, k_nope=k_nope, k_rope=k_rope, v=v, cu_seqlens=cu_seqlens, cu_seqlens_k=cu_seqlens_k)
        q, qt = _tokens(q)
        k_nope, kt = _tokens(k_nope)
        k_rope, rt = _tokens(k_rope)
        v, vt = _tokens(v)
        self.B, self.T, self.Tk, self.H = B, T, Tk, H
        p = ops.cdr_latent_attn_problem(N, T, Tk, H, int(cu_seqlens is not None),
                                        QUERY_DIM ** -0.5 if scale is None else float(scale))
        p.q_stride[0], p.q_stride[1] = qt, _step(q, 2)
        p.k_stride[0], p.k_stride[1] = kt, _step(k_nope, 2)
        p.v_stride[0], p.v_stride[1] = vt, _step(v, 2)
        p.k_rope_stride = rt
        st = self.lib.cdr_latent_attn_check(ctypes.byref(p))
        if st != CDR_OK:
            _raise(st, what)
        self.p = p
        self.tensors = (q, k_nope, k_rope, v, cu_seqlens, cu_seqlens_k)
        self.inputs = tuple(_ptr(t) for t in self.tensors)


def latent_attn_fwd(q: torch.Tensor, k_nope: torch.Tensor, k_rope: torch.Tensor, v: torch.Tensor,
                    scale: Optional[float] = None, cu_seqlens: Optional[torch.Tensor] = None,
                    cu_seqlens_k: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                    lse_out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Causal latent attention in the expanded form (prefill and training).

    ``q [B,T,H,192]`` (nope, then rope part), ``k_nope [B,Tk,H,128]``, ``k_rope [B,Tk,64]`` (one for
    all heads), ``v [B,Tk,H,128]`` bf16; k_nope and v may be slices of one projection.  The last
    query sees all Tk keys, so ``Tk - T`` earlier keys are a context; a query without keys gives
    zeros and -inf.  Packed batches have B = 1, ``cu_seqlens`` int32 ``[N+1]`` for the queries and
    ``cu_seqlens_k`` for the keys (the same when None).  ``scale=None`` means ``192 ** -0.5``; it must
    be positive.  Returns ``(o, lse)``: ``[B,T,H,128]`` bf16 and ``[B,T,H]`` fp32; rows that no packed
    sequence holds are zeros and -inf.  ``out`` and ``lse_out`` optionally supply the buffers, apart from
    the inputs; in them such rows are left as they were.
    """
    c = _LatentAttn(q, k_nope, k_rope, v, scale, cu_seqlens, cu_seqlens_k, "latent_attn_fwd")
    if out is not None:
        _need(out, "out", torch.bfloat16, (c.B, c.T, c.H, VALUE_DIM), dense=True)
        if out.data_ptr() % 16:
            raise ValueError("out must be 16-byte aligned")
    if lse_out is not None:
        _need(lse_out, "lse_out", torch.float32, (c.B, c.T, c.H), dense=True)
    _on(c.device, out=out, lse_out=lse_out)
    if out is not None or lse_out is not None:
        _apart(dict(zip(("q", "k_nope", "k_rope", "v", "cu_seqlens", "cu_seqlens_k"), c.tensors)),
               dict(out=out, lse_out=lse_out))
    _need_gpu(c.device)
    out, lse_out = _results(c.p, out, lse_out, (c.B, c.T, c.H, VALUE_DIM), c.device)
    _launch(c.device, "latent_attn_fwd", c.lib.cdr_latent_attn_fwd, ctypes.byref(c.p), *c.inputs, _ptr(out),
            _ptr(lse_out))
    return out, lse_out


def latent_attn_bwd(q: torch.Tensor, k_nope: torch.Tensor, k_rope: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                    lse: torch.Tensor, do: torch.Tensor, scale: Optional[float] = None,
                    cu_seqlens: Optional[torch.Tensor] = None, cu_seqlens_k: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None):
    """Gradients of :func:`latent_attn_fwd`.

    Inputs as the forward, its ``o`` and ``lse``, and ``do [B,T,H,128]`` bf16, the gradient of o.
    Returns bf16 ``(dq, dk_nope, dk_rope, dv)`` with the shapes of the inputs; dk_rope is the sum
    over the heads, added in fp32.  Rows and keys that no packed sequence holds get zeros.  Repeated
    calls give the same bits.  ``workspace`` optionally supplies the scratch buffer (uint8, contiguous).
    """
    c = _LatentAttn(q, k_nope, k_rope, v, scale, cu_seqlens, cu_seqlens_k, "latent_attn_bwd")
    shape = (c.B, c.T, c.H, VALUE_DIM)
    _need(o, "o", torch.bfloat16, shape)
    _need(do, "do", torch.bfloat16, shape)
    _need(lse, "lse", torch.float32, shape[:3])
    _on(c.device, o=o, do=do, lse=lse, workspace=workspace)
    _need_gpu(c.device)
    o, lse, do = ops._aligned(o), lse.contiguous(), ops._aligned(do)
    need = c.lib.cdr_latent_attn_bwd_workspace_bytes(ctypes.byref(c.p))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=c.device)
    elif workspace.numel() * workspace.element_size() < need:
        raise ValueError("workspace too small")
    elif not workspace.is_contiguous() or workspace.data_ptr() % 16:
        raise ValueError("workspace must be contiguous and 16-byte aligned")
    empty = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=c.device)  # noqa: E731
    dq = empty(c.B, c.T, c.H, QUERY_DIM)
    dk, dv = empty(c.B, c.Tk, c.H, NOPE_DIM), empty(c.B, c.Tk, c.H, VALUE_DIM)
    dkr = empty(c.B, c.Tk, LATENT_ROPE)
    if c.p.varlen:
        c.p.varlen = VARLEN_FILL
    _launch(c.device, "latent_attn_bwd", c.lib.cdr_latent_attn_bwd, ctypes.byref(c.p), *c.inputs, _ptr(o), _ptr(lse),
            _ptr(do), _ptr(dq), _ptr(dk), _ptr(dkr), _ptr(dv), _ptr(workspace),
            workspace.numel() * workspace.element_size())
    return dq, dk, dkr, dv
