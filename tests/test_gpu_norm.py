"""The block boundary's kernels against the fp64 oracle, on the GPU.

Tolerance of an element: half a step of its type relative to the value, plus 64 roundings of 2^-24
relative to its magnitude (the sum of the absolute terms, as the oracle gives it): a thread adds at
most 16 squares and a row's sum at most 8 + 4 more levels, whose relative error halves in the root;
each element then takes fewer than 16 products and sums, one exponential and one reciprocal (each
within 2 units), and the exponential's argument up to |z| log2(e) half units, |z| <= 8 here.  A column
sum adds at most rows / 512 + 16 terms in a thread and 128 + 4 partial rows.
"""
import pytest
import torch

import chunked_gated_delta_chunk_amd as cdr
from oracle.norm import block_norm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U32 = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


def make(shape, seed, dt=BF16, rdt=BF16, post=True, gate=True, res=True, scale=True, pre=True):
    g = torch.Generator().manual_seed(seed)
    D = shape[-1]
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    kw = dict(y=r(*shape).to(dt), weight=1 + 0.2 * r(D) if post else None,
              gate=(2 * r(*shape)).clamp(-8, 8).to(dt) if gate else None,
              residual=r(*shape).to(rdt) if res else None, res_scale=0.5 + 0.2 * r(D) if scale else None,
              next_weight=1 + 0.2 * r(D) if pre else None)
    return kw, r(*shape).to(rdt if res else dt), r(*shape).to(dt) if pre else None


def to_dev(kw):
    return {k: v.to(DEV) if isinstance(v, torch.Tensor) else v for k, v in kw.items()}


def check(name, got, ref, rows):
    value, mag = ref
    assert got is not None, name
    got64 = got.cpu().double()
    half = torch.finfo(got.dtype).eps / 2
    n = 64 + (rows // 512 + 16 + 132 if value.dim() == 1 else 0)
    tol = half * value.abs() + n * U32 * mag + 1e-30
    worst = float(((got64 - value).abs() / tol).max()) if value.numel() else 0.0
    assert worst <= 1.0, f"{name}: {worst:.3f} of the tolerance"


def run(kw, dr, dh, act, eps=1e-6):
    d = to_dev(kw)
    rows = kw["y"].numel() // kw["y"].shape[-1]
    r, h = cdr.block_norm_fwd(**d, gate_act=act, eps=eps)
    grads = cdr.block_norm_bwd(d_out=None if dr is None else dr.to(DEV), d_next=None if dh is None else dh.to(DEV),
                               **d, gate_act=act, eps=eps)
    ref = block_norm(**kw, gate_act=act, eps=eps, d_out=dr, d_next=dh)
    names = ("dy", "dweight", "dgate", "dresidual", "dres_scale", "dnext_weight")
    got = dict(zip(names, grads), r=r, h=h)
    assert {k for k, v in got.items() if v is not None} == set(ref)
    for name in ref:
        check(name, got[name], ref[name], rows)
    return got


PARTS = {"all": {}, "head gate": dict(res=False, scale=False, pre=False), "pre only": dict(post=False, gate=False, scale=False),
         "post only": dict(gate=False, res=False, scale=False, pre=False), "no norm": dict(post=False, pre=False),
         "no residual": dict(res=False)}


@pytest.mark.parametrize("parts", list(PARTS), ids=lambda p: p.replace(" ", "_"))
@pytest.mark.parametrize("dt,rdt", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_parts_and_types(parts, dt, rdt, act):
    kw, dr, dh = make((5, 3, 128), 1, dt, rdt, **PARTS[parts])
    run(kw, dr, dh, act)


@pytest.mark.parametrize("D", [1, 2, 7, 8, 127, 128, 129, 136, 511, 512, 520, 777, 2047, 2048, 2056, 4095, 4096, 4104,
                               8185, 8192])
@pytest.mark.parametrize("rows", [1, 37])
def test_widths(D, rows):
    kw, dr, dh = make((rows, D), D + rows)
    run(kw, dr, dh, "silu")


@pytest.mark.parametrize("rows,D", [(5000, 128), (1100, 512), (2100, 256), (700, 1024)])
def test_many_rows_and_same_bits(rows, D):
    """More rows than the workgroups take in one turn, and the column sums' order is fixed."""
    kw, dr, dh = make((rows, D), 3)
    a = run(kw, dr, dh, "sigmoid")
    b = run(kw, dr, dh, "sigmoid")
    for k in a:
        assert torch.equal(a[k], b[k]), k


def test_no_rows():
    kw, dr, dh = make((0, 64), 4)
    got = run(kw, dr, dh, "silu")
    assert (got["dweight"] == 0).all() and got["r"].shape == (0, 64)


def test_strided_slices_are_read_in_place():
    """y, gate and residual as slices of one projection [T, 2 HV D + ...], aligned and not."""
    g = torch.Generator().manual_seed(5)
    for T, HV, D, start in ((6, 4, 128, 0), (6, 4, 128, 8), (5, 3, 64, 3), (4, 2, 37, 5)):
        wide = torch.randn(T, 3 * HV * D + 11 + start, generator=g).to(BF16)
        cut = lambda w, i: w[:, start + i * HV * D:start + (i + 1) * HV * D].view(T, HV, D)  # noqa: E731
        kw, dr, dh = make((T, HV, D), 6)
        kw.update(y=cut(wide, 0), gate=cut(wide, 1), residual=cut(wide, 2))
        dev = wide.to(DEV)
        ref = block_norm(**kw, d_out=dr, d_next=dh)
        d = to_dev(kw)
        d.update(y=cut(dev, 0), gate=cut(dev, 1), residual=cut(dev, 2))
        assert not d["y"].is_contiguous()
        r, h = cdr.block_norm_fwd(**d)
        grads = cdr.block_norm_bwd(d_out=dr.to(DEV), d_next=dh.to(DEV), **d)
        check("r", r, ref["r"], T * HV)
        check("h", h, ref["h"], T * HV)
        for name, got in zip(("dy", "dweight", "dgate", "dresidual", "dres_scale", "dnext_weight"), grads):
            check(name, got, ref[name], T * HV)


def test_other_layouts_give_the_same():
    """Transposed, broadcast and one-dimensional inputs."""
    kw, dr, dh = make((4, 6, 32), 7)
    d = to_dev(kw)
    want = cdr.block_norm_fwd(**d)
    t = dict(d, y=d["y"].permute(2, 0, 1).contiguous().permute(1, 2, 0), gate=d["gate"].transpose(0, 1).contiguous()
             .transpose(0, 1))
    for a, b in zip(cdr.block_norm_fwd(**t), want):
        assert torch.equal(a, b)
    wide = dict(d, gate=d["gate"][:1].expand(4, 6, 32))
    for a, b in zip(cdr.block_norm_fwd(**wide), cdr.block_norm_fwd(**dict(d, gate=wide["gate"].contiguous()))):
        assert torch.equal(a, b)
    one = {k: v[0, 0] if v.dim() == 3 else v for k, v in d.items()}
    for a, b in zip(cdr.block_norm_fwd(**one), want):
        assert torch.equal(a, b[0, 0])


def test_in_place_and_given_outputs():
    kw, dr, dh = make((33, 256), 8, BF16, BF16)
    d = to_dev(kw)
    r, h = cdr.block_norm_fwd(**d)
    x, y = d["residual"].clone(), d["y"].clone()
    r2, h2 = cdr.block_norm_fwd(**dict(d, residual=x, y=y), out=x, next_out=y)
    assert r2 is x and h2 is y and torch.equal(r, x) and torch.equal(h, y)


def test_float_scale_and_gradient_of_next_alone():
    kw, dr, dh = make((9, 96), 9, scale=False)
    kw["res_scale"] = 0.22
    run(kw, dr, dh, "silu")
    run(kw, None, dh, "silu")


def test_zero_rows_and_large_values():
    """A row of zeros (the norm is eps alone) and rows whose squares are far from one."""
    kw, dr, dh = make((4, 128), 10, F32, F32, gate=False)
    kw["y"][0] = 0
    kw["residual"][0] = 0
    kw["y"][1] *= 1e12
    kw["y"][2] *= 1e-12
    run(kw, dr, dh, "sigmoid")


def test_gate_far_from_zero():
    kw, dr, dh = make((3, 64), 11, F32, F32)
    kw["gate"][0], kw["gate"][1] = 200.0, -200.0
    d = to_dev(kw)
    for act in ("sigmoid", "silu"):
        r, h = cdr.block_norm_fwd(**d, gate_act=act)
        grads = cdr.block_norm_bwd(d_out=dr.to(DEV), d_next=dh.to(DEV), **d, gate_act=act)
        assert torch.isfinite(r).all() and torch.isfinite(h).all()
        assert all(torch.isfinite(t).all() for t in grads)
        assert torch.equal(r[1], d["residual"][1])        # a closed gate leaves the residual as it was


def test_graph_replays():
    kw, dr, dh = make((300, 512), 12)
    d = to_dev(kw)
    dr, dh = dr.to(DEV), dh.to(DEV)
    step = lambda: cdr.block_norm_fwd(**d) + cdr.block_norm_bwd(d_out=dr, d_next=dh, **d)  # noqa: E731
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in (20, 21, 22):
        new, ndr, ndh = make((300, 512), seed)
        for k, v in new.items():
            d[k].copy_(v)
        dr.copy_(ndr)
        dh.copy_(ndh)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, step()):
            assert torch.equal(a, b)


def test_after_the_chunked_forward():
    """o of the chunked forward through the gated head norm, the residual and the next norm."""
    import oracle
    from chunked_gated_delta_chunk_amd.synth import make_inputs
    inp = make_inputs(1, 150, 2, seed=13, initial_state=True)
    d = inp.to(DEV)
    o, _ = cdr.chunk_dr_fwd(d.q, d.k, d.v, d.g, d.beta, initial_state=d.initial_state)
    kw, _, _ = make((1, 150, 2, 128), 14, pre=False, res=False, scale=False)
    kw["y"] = o
    dev = to_dev(kw)
    r, _ = cdr.block_norm_fwd(**dev)
    kw2, _, _ = make((1, 150, 256), 15, F32, F32, post=False, gate=False, scale=False)
    kw2["y"] = r.reshape(1, 150, 256).float()
    x, h = cdr.block_norm_fwd(**to_dev(kw2))
    check("r", r, block_norm(**dict(kw, y=o.cpu()))["r"], 300)
    ref = block_norm(**dict(kw2, y=kw2["y"].cpu()))
    check("x", x, ref["r"], 150)
    check("h", h, ref["h"], 150)
    o_ref, _ = oracle.recurrent_fwd(inp.q, inp.k, inp.v, inp.g, inp.beta, initial_state=inp.initial_state)
    assert (abs(o.float().cpu().numpy() - o_ref) <= 1e-2 + 1e-2 * abs(o_ref)).all()
