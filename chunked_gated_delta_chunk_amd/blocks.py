"""Python binding of what stands around the token mixer: the block boundary's norms, gate and
residual (cdr_block_norm_* of include/chunk_dr.h) and a serving step's offsets, page tables and
slots (cdr_build_page_tables).

Argument marshalling only, as in ops.py: dtype and shape checks, allocation of the outputs and the
workspace, one call into libchunkdr.so on the current stream of the tensors' device.
"""
import ctypes
from typing import NamedTuple, Optional, Tuple, Union

import torch

from . import ops
from .ops import CDR_OK, _need, _raise, load_library

_DTYPES = {torch.bfloat16: 0, torch.float32: 1}
_ACTS = {None: 0, "sigmoid": 1, "silu": 2}


# the raw handle of a device's current stream: what torch.cuda.current_stream(device).cuda_stream
# returns, without the stream object in between (0.1 us against 1.9 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _launch(device, what, entry, *args):
    """entry(*args, stream) on the device's current stream, with that device current."""
    index = device.index
    if index == torch.cuda.current_device():
        st = entry(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            st = entry(*args, _raw_stream(index))
    if st != CDR_OK:
        _raise(st, what)


def _span(t):
    """First byte and end of the memory between a tensor's first and last element."""
    a = t.data_ptr()
    last = -1 if t.numel() == 0 else sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
    return a, a + (last + 1) * t.element_size()


def _apart(inputs, outputs):
    """Raises where an output's memory overlaps that of an input read in place (both dicts, None for none)."""
    spans = [(m, *_span(i)) for m, i in inputs.items() if i is not None]
    for n, o in outputs.items():
        if o is None:
            continue
        a, e = _span(o)
        for m, b, f in spans:
            if a < f and b < e:
                raise ValueError(f"{n} overlaps {m}, which is read after it is written")


def _need_gpu(device):
    if device.type != "cuda":
        raise ValueError("inputs must be on a GPU device")


def _on(device, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")


def _dense_like(t):
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _rows(t, inner):
    """(t, outer stride, inner stride) of the rows of t ([..., D]); a copy of it where its rows do
    not start at i // inner * outer + i % inner * step, or its last dimension is strided."""
    if t.is_contiguous():
        D = t.shape[-1]
        return t, inner * D, D
    lead = t.shape[:-1]
    st = t.stride()
    if t.shape[-1] == 1 or st[-1] == 1:
        split = len(lead) - 1 if inner > 1 else len(lead)
        step = st[split] if inner > 1 else 0
        outer, size = None, 1      # of the leading dimensions, as one
        for n, s in zip(reversed(lead[:split]), reversed(st[:split])):
            if n == 1:
                continue
            if outer is None:
                outer, size = s, n
            elif s == outer * size:
                size *= n
            else:
                break
        else:
            return t, outer or 0, step
    t = t.contiguous()
    D = t.shape[-1]
    return t, inner * D, D


class _BlockNorm:
    """The checked arguments of a block norm: its problem struct and the tensors it points to."""

    def __init__(self, y, weight, gate, gate_act, residual, res_scale, next_weight, eps):
        if not isinstance(y, torch.Tensor):
            raise TypeError("y must be a torch.Tensor")
        if y.dtype not in _DTYPES:
            raise TypeError(f"y must be bfloat16 or float32, got {y.dtype}")
        if y.dim() < 1:
            raise ValueError("y must be [..., D]")
        shape, D = tuple(y.shape), y.shape[-1]
        if gate_act not in _ACTS:
            raise ValueError(f"gate_act must be 'sigmoid', 'silu' or None, got {gate_act!r}")
        if gate is not None:
            _need(gate, "gate", y.dtype, shape)
            if gate_act is None:
                raise ValueError("a gate needs gate_act")
        if residual is not None:
            if not isinstance(residual, torch.Tensor) or residual.dtype not in _DTYPES:
                raise TypeError("residual must be a bfloat16 or float32 tensor")
            _need(residual, "residual", residual.dtype, shape)
        for name, t in (("weight", weight), ("next_weight", next_weight)):
            if t is not None:
                _need(t, name, torch.float32, (D,))
        alpha = 1.0
        if isinstance(res_scale, torch.Tensor):
            _need(res_scale, "res_scale", torch.float32, (D,))
        elif res_scale is not None:
            alpha, res_scale = float(res_scale), None
        device = y.device
        _on(device, weight=weight, gate=gate, residual=residual, res_scale=res_scale, next_weight=next_weight)
        self.device, self.shape, self.D = device, shape, D
        self.dtype = y.dtype
        self.out_dtype = residual.dtype if residual is not None else y.dtype
        inner = shape[-2] if len(shape) > 2 else 1
        rows = y.numel() // D if D else 0
        if rows >= 2 ** 31 or D >= 2 ** 31:
            raise ValueError("y has more than 2^31 - 1 rows or columns")
        p = ops.cdr_block_norm_problem()
        p.rows, p.D, p.inner = rows, D, inner if rows else 1
        p.dtype = _DTYPES[y.dtype]
        p.res_dtype = _DTYPES[self.out_dtype]
        p.gate_act = 0 if gate is None else _ACTS[gate_act]
        p.has_weight, p.has_residual = weight is not None, residual is not None
        p.has_scale, p.has_next = res_scale is not None, next_weight is not None
        p.alpha, p.eps = alpha, float(eps)
        self.p = p
        self.lib = load_library()
        self.y, p.y_stride[0], p.y_stride[1] = _rows(y, p.inner)
        self.gate = self.residual = None
        if gate is not None:
            self.gate, p.gate_stride[0], p.gate_stride[1] = _rows(gate, p.inner)
        if residual is not None:
            self.residual, p.residual_stride[0], p.residual_stride[1] = _rows(residual, p.inner)
        self.weight = None if weight is None else weight.contiguous()
        self.scale = None if res_scale is None else res_scale.contiguous()
        self.next_weight = None if next_weight is None else next_weight.contiguous()
        self.inputs = (_ptr(self.y), _ptr(self.gate), _ptr(self.residual), _ptr(self.weight), _ptr(self.scale),
                       _ptr(self.next_weight))


def block_norm_fwd(y: torch.Tensor, weight: Optional[torch.Tensor] = None,
                   gate: Optional[torch.Tensor] = None, gate_act: Optional[str] = "sigmoid",
                   residual: Optional[torch.Tensor] = None,
                   res_scale: Union[torch.Tensor, float, None] = None,
                   next_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                   out: Optional[torch.Tensor] = None, next_out: Optional[torch.Tensor] = None,
                   ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The norm after a token mixer with its gate, the residual, and the norm before the next block.

    ``n = rmsnorm(y) * weight`` (n = y without weight), ``r = residual + res_scale * a(gate) * n``
    with a = sigmoid or silu, ``h = rmsnorm(r) * next_weight``, over the last dimension D (1 to
    8192); every part but y is optional.  y, gate ``[..., D]`` bf16 or fp32; residual ``[..., D]``
    bf16 or fp32 (r takes its type, else y's); weight, next_weight and a tensor res_scale ``[D]``
    fp32; a float res_scale multiplies.  Returns ``(r, h)``, h None without next_weight.  Slices of
    a wider projection are read in place; other strided inputs are copied first.  ``out`` and
    ``next_out`` (contiguous) optionally supply the results; ``out`` may be residual itself and
    ``next_out`` y itself, when those are contiguous.

    With D = 128 on o ``[B,T,HV,128]``, a gate and a weight it is the gated head norm that follows
    :func:`chunk_dr_fwd`.
    """
    c = _BlockNorm(y, weight, gate, gate_act, residual, res_scale, next_weight, eps)
    if out is not None:
        _need(out, "out", c.out_dtype, c.shape, dense=True)
    if next_out is not None:
        if next_weight is None:
            raise ValueError("next_out needs next_weight")
        _need(next_out, "next_out", c.dtype, c.shape, dense=True)
    _on(c.device, out=out, next_out=next_out)
    _need_gpu(c.device)
    if out is None:
        out = _dense_like(y if residual is None else residual)
    if next_out is None and next_weight is not None:
        next_out = _dense_like(y)
    _launch(c.device, "block_norm_fwd", c.lib.cdr_block_norm_fwd, ctypes.byref(c.p), *c.inputs, out.data_ptr(),
            _ptr(next_out))
    return out, next_out


def block_norm_bwd(y: torch.Tensor, d_out: Optional[torch.Tensor], d_next: Optional[torch.Tensor] = None,
                   weight: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                   gate_act: Optional[str] = "sigmoid", residual: Optional[torch.Tensor] = None,
                   res_scale: Union[torch.Tensor, float, None] = None,
                   next_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                   workspace: Optional[torch.Tensor] = None):
    """Gradients of :func:`block_norm_fwd`, which is recomputed from the same inputs.

    ``d_out`` (the type of r; None for zero, with next_weight) and ``d_next`` (y's type, with
    next_weight) are the gradients of r and h.  Returns ``(dy, dweight, dgate, dresidual,
    dres_scale, dnext_weight)``: dy, dgate in y's type, dresidual in residual's, the vectors' in
    fp32, None for what was not given (or is a float).  Repeated calls give the same bits.
    ``workspace`` optionally supplies the scratch buffer (uint8, contiguous).
    """
    c = _BlockNorm(y, weight, gate, gate_act, residual, res_scale, next_weight, eps)
    if d_out is not None:
        _need(d_out, "d_out", c.out_dtype, c.shape)
    elif next_weight is None:
        raise ValueError("d_out is required without next_weight")
    if (d_next is None) != (next_weight is None):
        raise ValueError("d_next and next_weight go together")
    if d_next is not None:
        _need(d_next, "d_next", c.dtype, c.shape)
    _on(c.device, d_out=d_out, d_next=d_next, workspace=workspace)
    _need_gpu(c.device)
    need = c.lib.cdr_block_norm_bwd_workspace_bytes(ctypes.byref(c.p))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=c.device)
    elif workspace.numel() * workspace.element_size() < need:
        raise ValueError("workspace too small")
    elif not workspace.is_contiguous() or workspace.data_ptr() % 16:
        raise ValueError("workspace must be contiguous and 16-byte aligned")
    like = lambda t: None if t is None else _dense_like(t)  # noqa: E731
    dense = lambda t: None if t is None else t.contiguous()  # noqa: E731
    d_out, d_next = dense(d_out), dense(d_next)
    dy, dgate, dres = _dense_like(y), like(gate), like(residual)
    dw, ds, dw2 = like(c.weight), like(c.scale), like(c.next_weight)
    _launch(c.device, "block_norm_bwd", c.lib.cdr_block_norm_bwd, ctypes.byref(c.p), *c.inputs, _ptr(d_out),
            _ptr(d_next), _ptr(dy), _ptr(dgate), _ptr(dres), _ptr(dw), _ptr(ds), _ptr(dw2), _ptr(workspace),
            workspace.numel() * workspace.element_size())
    return dy, dw, dgate, dres, ds, dw2


class PageTables(NamedTuple):
    """What :func:`build_page_tables` writes, int32 on the device."""
    cu_seqlens: torch.Tensor   # [N + 1]
    seq_lens: torch.Tensor     # [N], context and new tokens
    positions: torch.Tensor    # [max_tokens]
    slot_map: torch.Tensor     # [max_tokens], -1 for no slot
    free_head: torch.Tensor    # [1], the free list's head after the step
    shortage: torch.Tensor     # [1], pages wanted and not there


def build_page_tables(query_lens: torch.Tensor, context_lens: torch.Tensor, block_table: torch.Tensor,
                      free_pages: torch.Tensor, free_head: torch.Tensor, page_size: int, max_tokens: int,
                      free_head_out: Optional[torch.Tensor] = None,
                      out: Optional[PageTables] = None, workspace: Optional[torch.Tensor] = None) -> PageTables:
    """A serving step's offsets, positions, page table and slots, on the device (formulas at
    cdr_build_page_tables in chunk_dr.h).

    ``query_lens`` and ``context_lens`` int32 ``[N]``: each request's new tokens and tokens already
    cached; ``block_table`` int32 ``[N, W]``, updated in place with the new pages, which are taken
    from ``free_pages`` int32 ``[F]`` at ``free_head`` int32 ``[1]``.  ``free_head`` is advanced in
    place unless ``free_head_out`` is given.  ``max_tokens`` is the size of the token arrays (a
    captured step's): positions and slots behind the last request are 0 and -1.  ``cu_seqlens`` then ends
    below ``max_tokens``, which latent attention takes as it is; :func:`chunk_dr_fwd` and
    :func:`fused_recurrent_fwd` need offsets that end at their T.  Nothing is read
    back to the host; ``shortage`` says how many pages were missing.  ``out`` reuses the tensors of
    an earlier call, as a captured graph does (``free_head`` of it is ignored); they must not overlap
    the inputs, so an earlier call's ``seq_lens`` taken as ``context_lens`` is not also this call's.
    """
    lib = load_library()
    _need(query_lens, "query_lens", torch.int32)
    if query_lens.dim() != 1 or query_lens.numel() < 1:
        raise ValueError("query_lens must be [N] with N >= 1")
    N = query_lens.shape[0]
    _need(context_lens, "context_lens", torch.int32, (N,))
    _need(block_table, "block_table", torch.int32, dense=True)
    if block_table.dim() != 2 or block_table.shape[0] != N or block_table.shape[1] < 1:
        raise ValueError(f"block_table must be [{N}, W] with W >= 1")
    _need(free_pages, "free_pages", torch.int32)
    if free_pages.dim() != 1:
        raise ValueError("free_pages must be one-dimensional")
    _need(free_head, "free_head", torch.int32, (1,))
    page_size, max_tokens = int(page_size), int(max_tokens)
    if not 1 <= page_size < 2 ** 31 or not 0 <= max_tokens < 2 ** 31:
        raise ValueError("page_size must be positive and max_tokens not negative")
    if free_head_out is None:
        free_head_out = free_head
    else:
        _need(free_head_out, "free_head_out", torch.int32, (1,))
    device = query_lens.device
    need = lib.cdr_page_tables_workspace_bytes(N)
    _on(device, context_lens=context_lens, block_table=block_table, free_pages=free_pages, free_head=free_head,
        free_head_out=free_head_out, workspace=workspace)
    if out is not None:
        for name, t, n in (("cu_seqlens", out.cu_seqlens, N + 1), ("seq_lens", out.seq_lens, N),
                           ("positions", out.positions, max_tokens), ("slot_map", out.slot_map, max_tokens),
                           ("shortage", out.shortage, 1)):
            _need(t, "out." + name, torch.int32, (n,), dense=True)
            _on(device, **{"out." + name: t})
        ins = dict(query_lens=query_lens, context_lens=context_lens, block_table=block_table, free_pages=free_pages,
                   free_head=free_head)
        _apart({n: t for n, t in ins.items() if t.is_contiguous()},   # others are copied first
               {"out." + n: t for n, t in zip(out._fields, out) if n != "free_head"})
    _need_gpu(device)
    sizes = [N + 1, N, max_tokens, max_tokens, 1]
    if out is not None:
        cu, lens, pos, slot, short = out.cu_seqlens, out.seq_lens, out.positions, out.slot_map, out.shortage
    elif workspace is not None:
        cu, lens, pos, slot, short = torch.empty(sum(sizes), dtype=torch.int32, device=device).split_with_sizes(sizes)
    else:   # one allocation, the scratch space at its end
        sizes.append(need // 4)
        cu, lens, pos, slot, short, workspace = torch.empty(sum(sizes), dtype=torch.int32, device=device).split_with_sizes(sizes)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    elif workspace.numel() * workspace.element_size() < need or not workspace.is_contiguous() \
            or workspace.data_ptr() % 4:
        raise ValueError(f"workspace must be contiguous, 4-byte aligned and hold {need} bytes")
    query_lens, context_lens, free_pages = query_lens.contiguous(), context_lens.contiguous(), free_pages.contiguous()
    _launch(device, "build_page_tables", lib.cdr_build_page_tables, N, block_table.shape[1], free_pages.numel(),
            page_size, max_tokens, _ptr(query_lens), _ptr(context_lens), _ptr(block_table), _ptr(free_pages),
            _ptr(free_head), _ptr(free_head_out), _ptr(cu), _ptr(lens), _ptr(pos), _ptr(slot), _ptr(short),
            _ptr(workspace), workspace.numel() * workspace.element_size())
    return PageTables(cu, lens, pos, slot, free_head_out, short)
