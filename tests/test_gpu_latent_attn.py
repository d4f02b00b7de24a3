"""Latent attention in the expanded form on the GPU against the fp64 oracle, forward and gradients.

Tolerances.  A score is 192 exact products of bf16 added in fp32 and scaled: an error of at most
e = (193 + 8) 2^-24 times the sum of its absolute terms (`size`).  Weights p have relative error
2 e + 2^-18 (e in the score and in the statistics; exponential, sum of at most 4096 in a lane and 8
levels of tree) before they are rounded to bf16 (2^-8).  With `mag` the sum of the absolute terms of an
output's last product:

  o, dv     (2^-8 + 2 e + 2^-16) mag + half a step of the value
  dq, dk    dS = p (dP - delta): p as above; dP has 2^-16 of its absolute terms, delta is formed from o
            as the forward rounded it, (2^-8 + 2^-8 + 2 e + 2^-16) of its absolute terms; dS is rounded
            to bf16: 2^-8; together (4 2^-8 + 4 e + 2^-14) mag + half a step
"""
import ctypes
import math

import pytest
import torch

import chunked_gated_delta_chunk_amd as cdr
from chunked_gated_delta_chunk_amd import latent
from oracle import latent as oracle_latent

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16
NAMES = ("dq", "dk_nope", "dk_rope", "dv")


def make(lq, lk, H, seed, packed=True, spare=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(BF16)  # noqa: E731
    if packed:
        B, T, Tk = 1, sum(lq) + spare, sum(lk) + spare
        cu = lambda x: torch.tensor([0] + list(x)).cumsum(0).to(torch.int32)  # noqa: E731
        more = dict(cu_seqlens=cu(lq), cu_seqlens_k=cu(lk))
    else:
        B, T, Tk, more = len(lq), lq[0], lk[0], {}
    kv = r(B, Tk, H, 256)
    return dict(q=r(B, T, H, 192), k_nope=kv[..., :128], k_rope=r(B, Tk, 64), v=kv[..., 128:], **more), r(B, T, H, 128)


def dev(kw):
    """On the GPU with the same strides."""
    out = {}
    for k, v in kw.items():
        if isinstance(v, torch.Tensor) and k in ("k_nope", "v") and not v.is_contiguous():
            base = torch.empty(v.shape[:3] + (256,), dtype=BF16, device=DEV)
            view = base[..., :128] if k == "k_nope" else base[..., 128:]
            view.copy_(v)
            out[k] = view
        else:
            out[k] = v.to(DEV) if isinstance(v, torch.Tensor) else v
    return out


def within(name, got, ref, tol, live):
    d = ((got.cpu().double() - ref).abs() / tol)[live]
    assert not d.numel() or float(d.max()) <= 1, f"{name}: {float(d.max()):.3f} of the tolerance"


def compare(kw, do, o, lse, grads, scale):
    ref = oracle_latent.attention(scale=scale, do=do, **kw)
    live = ~torch.isnan(ref["lse"])
    empty = live & torch.isinf(ref["lse"])
    full = live & ~empty
    assert torch.isfinite(o.cpu()[live]).all()
    assert (o.cpu()[empty] == 0).all() and (lse.cpu()[empty] == -math.inf).all()
    e = 201 * 2.0 ** -24 * ref["size"]
    within("lse", lse, ref["lse"], e + 2.0 ** -18 + 2.0 ** -22 * ref["lse"].abs(), full)
    top = float(e[live].max()) if live.any() else 0.0     # keys meet many rows: the largest of them
    tol = lambda n, f, x: (f * 2.0 ** -8 + x * top + 2.0 ** -14) * ref[n + "_mag"] \
        + 2.0 ** -8 * ref[n].abs() + 1e-30  # noqa: E731
    within("o", o, ref["o"], tol("o", 1, 2), live)
    if grads is None:
        return
    for name, g in zip(NAMES, grads):
        keys = ~torch.isnan(ref[name])
        assert torch.isfinite(g.cpu()[keys]).all(), name
        within(name, g, ref[name], tol(name, 1 if name == "dv" else 4, 2 if name == "dv" else 4), keys)


def run(kw, do, scale=192 ** -0.5):
    d = dev(kw)
    o, lse = cdr.latent_attn_fwd(**d, scale=scale)
    grads = cdr.latent_attn_bwd(**d, o=o, lse=lse, do=do.to(DEV), scale=scale)
    compare(kw, do, o, lse, grads, scale)
    return (o, lse) + grads


@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 257])
def test_one_sequence(T):
    run(*make([T], [T], 2, T, packed=False))


@pytest.mark.parametrize("H", [1, 3, 8])
def test_equal_lengths(H):
    run(*make([70] * 3, [70] * 3, H, H, packed=False))
    run(*make([40] * 2, [150] * 2, H, 10 + H, packed=False))        # a context of 110 keys


@pytest.mark.parametrize("lq,lk", [
    ((1, 130, 64, 3), (1, 130, 64, 3)), ((5, 0, 129, 0, 1), (5, 0, 129, 0, 1)),
    ((1, 1, 1, 1), (300, 64, 1, 65)), ((10, 128, 33), (200, 129, 1000)), ((0, 4), (70, 4)),
    ((64, 65), (0, 65)), ((200, 3), (100, 1)), ((130, 250), (129, 60)), ((1,) * 40, (2,) * 40)])
def test_packed(lq, lk):
    """Tails, empty sequences, contexts, rows without keys, keys that no row sees."""
    run(*make(lq, lk, 2, sum(lq) + 3 * sum(lk)))


def test_long_sequence():
    run(*make([1500], [1500], 1, 21))
    run(*make([700], [2100], 2, 22))


def test_behind_the_last_sequence_is_left_alone():
    kw, do = make([30, 41], [50, 41], 2, 23, spare=5)
    d = dev(kw)
    d["q"][:, 71:], d["k_rope"][:, 91:], d["v"][:, 91:] = math.nan, math.nan, math.inf   # no sequence's
    d["k_nope"][:, 91:] = math.nan
    out = torch.full((1, 76, 2, 128), 3.0, dtype=BF16, device=DEV)
    lse = torch.full((1, 76, 2), 3.0, device=DEV)
    cdr.latent_attn_fwd(**d, out=out, lse_out=lse)
    assert (out[:, 71:] == 3).all() and (lse[:, 71:] == 3).all()
    compare(kw, do, out, lse, None, 192 ** -0.5)
    out[:, 71:], lse[:, 71:] = math.nan, math.nan
    grads = cdr.latent_attn_bwd(**d, o=out, lse=lse, do=do.to(DEV))
    compare(kw, do, out, lse, grads, 192 ** -0.5)


def raw_bwd(kw, do, o, lse, varlen, fill=3.0):
    """cdr_latent_attn_bwd itself, over outputs and a workspace that hold `fill`."""
    c = latent._LatentAttn(kw["q"], kw["k_nope"], kw["k_rope"], kw["v"], None, kw["cu_seqlens"], kw["cu_seqlens_k"], "")
    c.p.varlen = varlen
    full = lambda *s: torch.full(s, fill, dtype=BF16, device=DEV)  # noqa: E731
    dq, dk, dv = full(1, c.T, c.H, 192), full(1, c.Tk, c.H, 128), full(1, c.Tk, c.H, 128)
    dkr = full(1, c.Tk, 64)
    need = c.lib.cdr_latent_attn_bwd_workspace_bytes(ctypes.byref(c.p))
    work = torch.full((need // 4,), fill, device=DEV)
    st = c.lib.cdr_latent_attn_bwd(ctypes.byref(c.p), *c.inputs, o.data_ptr(), lse.data_ptr(), do.data_ptr(),
                                   dq.data_ptr(), dk.data_ptr(), dkr.data_ptr(), dv.data_ptr(), work.data_ptr(), need,
                                   torch.cuda.current_stream().cuda_stream)
    assert st == 0
    return dq, dk, dkr, dv


def gaps(seed):
    """Two sequences with rows and keys in front of the first (7 and 9) and behind the last (5 each), NaN and infinite."""
    kw, do = make([7, 30, 41], [9, 50, 41], 2, seed, spare=5)
    kw["cu_seqlens"], kw["cu_seqlens_k"] = kw["cu_seqlens"][1:], kw["cu_seqlens_k"][1:]
    d, ddo = dev(kw), do.to(DEV)
    for name in ("q", "k_nope", "k_rope", "v"):
        a, b = (7, 78) if name == "q" else (9, 100)
        d[name][:, :a], d[name][:, b:] = math.nan, math.inf
    ddo[:, :7], ddo[:, 78:] = math.nan, math.nan
    return kw, do, d, ddo


def test_results_that_no_sequence_holds_are_empty_rows(monkeypatch):
    """Zeros and -inf in what the binding allocates, whatever memory it gets; supplied buffers keep theirs."""
    kw, do, d, _ = gaps(59)
    empty = torch.empty
    with monkeypatch.context() as m:
        m.setattr(torch, "empty", lambda *s, **k: empty(*s, **k).fill_(77))
        o, lse = cdr.latent_attn_fwd(**d)
        out, lse_out = torch.full_like(o, 3), torch.full_like(lse, 3)
        only_lse = cdr.latent_attn_fwd(**d, out=out)[1]
        only_o = cdr.latent_attn_fwd(**d, lse_out=lse_out)[0]
    compare(kw, do, o, lse, None, 192 ** -0.5)
    for x, y, z, value in ((o, only_o, out, 0), (lse, only_lse, lse_out, -math.inf)):
        for rows in (slice(0, 7), slice(78, 83)):
            assert (x[:, rows] == value).all() and (z[:, rows] == 3).all()
        assert torch.equal(x, y) and torch.equal(x[:, 7:78], z[:, 7:78])


def test_gradients_that_no_sequence_holds_are_left_alone():
    kw, do, d, ddo = gaps(60)
    o, lse = cdr.latent_attn_fwd(**d)
    grads = raw_bwd(d, ddo, o, lse, 1)
    compare(kw, do, o, lse, grads, 192 ** -0.5)
    for name, g in zip(NAMES, grads):
        a, b = (7, 78) if name == "dq" else (9, 100)
        assert (g[:, :a] == 3).all() and (g[:, b:] == 3).all(), name


def test_gradients_that_no_sequence_holds_are_zero(monkeypatch):
    """From the C entry over what the outputs held before, and from the binding, whatever memory it gets."""
    kw, do, d, ddo = gaps(61)
    o, lse = cdr.latent_attn_fwd(**d)
    filled = raw_bwd(d, ddo, o, lse, latent.VARLEN_FILL, fill=math.nan)
    empty = torch.empty
    with monkeypatch.context() as m:
        m.setattr(torch, "empty", lambda *s, **k: empty(*s, **k).fill_(77))
        grads = cdr.latent_attn_bwd(**d, o=o, lse=lse, do=ddo)
    compare(kw, do, o, lse, grads, 192 ** -0.5)
    for name, g, f in zip(NAMES, grads, filled):
        a, b = (7, 78) if name == "dq" else (9, 100)
        assert (g[:, :a] == 0).all() and (g[:, b:] == 0).all(), name
        assert torch.equal(g, f), name


def test_gradients_of_padding_alone_and_of_many_rows_of_it():
    """No sequence with a token, and a tail far longer than the launch has workgroups."""
    for lens, spare in (((0, 0), 300), ((3,), 9000)):
        kw, do = make(lens, lens, 1, 62, spare=spare)
        d = dev(kw)
        o, lse = cdr.latent_attn_fwd(**d)
        grads = cdr.latent_attn_bwd(**d, o=o, lse=lse, do=do.to(DEV))
        compare(kw, do, o, lse, grads, 192 ** -0.5)
        assert all((g[:, sum(lens):] == 0).all() for g in grads)


def test_neighbours_of_a_sequence_do_not_matter():
    """The same sequence between others that hold NaN, with the same bits."""
    kw, do = make([77], [90], 2, 24)
    alone = run(kw, do)
    big, _ = make([64, 77, 50], [70, 90, 50], 2, 25)
    d = dev(big)
    ddo = torch.full((1, 191, 2, 128), math.nan, dtype=BF16, device=DEV)
    for n in ("q", "k_nope", "k_rope", "v"):
        a, b = (64, 141) if n == "q" else (70, 160)
        d[n].fill_(math.nan)
        d[n][:, a:b] = kw[n].to(DEV)
    ddo[:, 64:141] = do.to(DEV)
    o, lse = cdr.latent_attn_fwd(**d)
    dq, dk, dkr, dv = cdr.latent_attn_bwd(**d, o=o, lse=lse, do=ddo)
    for got, want in zip((o, lse, dq), (alone[0], alone[1], alone[2])):
        assert torch.equal(got[:, 64:141], want)
    for got, want in zip((dk, dkr, dv), alone[3:]):
        assert torch.equal(got[:, 70:160], want)


def test_layouts_give_the_same():
    kw, do = make([60, 9], [60, 9], 3, 26)
    want = run(kw, do)
    dense = {k: v.contiguous().to(DEV) for k, v in kw.items()}
    turned = dict(dense, q=dense["q"].permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3))
    odd = torch.empty(69 * 3 * 128 + 1, dtype=BF16, device=DEV)[1:].view(1, 69, 3, 128)
    odd.copy_(dense["v"])
    for d in (dense, turned, dict(dense, v=odd), dict(dense, v=dense["v"].permute(0, 1, 3, 2).contiguous().permute(0, 1, 3, 2))):
        o, lse = cdr.latent_attn_fwd(**d)
        g = cdr.latent_attn_bwd(**d, o=o, lse=lse, do=do.to(DEV))
        for a, b in zip((o, lse) + g, want):
            assert torch.equal(a, b)


def test_strides_of_single_elements_and_far_rows():
    """One sequence of one token and head with odd strides there; rows further apart than the kernels step."""
    kw, do = make([1], [1], 1, 40, packed=False)
    d = {k: v.contiguous().to(DEV) for k, v in kw.items()}
    want = cdr.latent_attn_fwd(**d)
    odd = lambda t: torch.as_strided(t, t.shape, (3, 5, 7, 1)[-t.dim():])  # noqa: E731
    for a, b in zip(cdr.latent_attn_fwd(**{k: odd(v) for k, v in d.items()}), want):
        assert torch.equal(a, b)
    kw, do = make([3], [3], 1, 41, packed=False)
    d = {k: v.contiguous().to(DEV) for k, v in kw.items()}
    want = cdr.latent_attn_fwd(**d)
    far = torch.zeros(3 * (1 << 23), dtype=BF16, device=DEV).as_strided((1, 3, 1, 192), (0, 1 << 23, 192, 1))
    far.copy_(d["q"])
    for a, b in zip(cdr.latent_attn_fwd(**dict(d, q=far)), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("n", [2, 63, 64, 65])
def test_many_short_sequences_in_either_order(n):
    """Up to 64 packed sequences are taken by weight, more by slot."""
    g = torch.Generator().manual_seed(n)
    lens = torch.randint(0, 40, (n,), generator=g).tolist()
    lens[n // 2] = 300
    run(*make(lens, [x + (i % 3) * 50 for i, x in enumerate(lens)], 1, 50 + n))


@pytest.mark.parametrize("n,H", [(32, 2), (33, 2), (5, 76), (5, 77)])
def test_orders_of_the_forward(n, H):
    """The forward takes up to 32 packed sequences by weight, and up to 1536 blocks of 128 rows: 5 sequences of 2000
    rows make 20 a head."""
    g = torch.Generator().manual_seed(n + H)
    if n == 5:
        lens = [1100, 3, 400, 297, 200]
    else:
        lens = torch.randint(0, 60, (n,), generator=g).tolist()
        lens[3] = 290
    run(*make(lens, [x + (i % 2) * 9 for i, x in enumerate(lens)], H, 70 + n + H))


def test_dq_in_blocks_of_either_size():
    """256 blocks of 256 rows and more take the larger blocks."""
    kw, do = make([257, 30, 513], [257, 30, 600], 64, 44)
    run(kw, do)


@pytest.mark.parametrize("short", [53, 54, 58, 70])
def test_dq_of_long_sequences_on_both_sides_of_the_larger_blocks(short):
    """dq takes blocks of 256 rows from 512 of them on (T // 256 + N a head): with 53 short sequences beside three
    long ones 504 for 8 heads, with 54 just 512; with 70 the blocks go by slot, not by weight."""
    lq = [1100, 257, 513] + [3] * short
    run(*make(lq, [1100, 257, 600] + [3, 4, 2, 150, 0, 3, 3] * (short // 7) + [3] * (short % 7), 8, 47 + short))


def test_dq_in_the_larger_blocks_of_one_long_sequence():
    """2500 rows among 55 of one, 520 blocks of 256 for 8 heads."""
    run(*make([2500] + [1] * 55, [3001] + [1] * 55, 8, 49))


def test_dq_in_the_larger_blocks_of_equal_lengths():
    """11 sequences of 520 rows and 16 heads, 528 blocks: two full ones and a cut one, behind a context."""
    run(*make([520] * 11, [560] * 11, 16, 48, packed=False))


@pytest.mark.parametrize("H", [2, 80])
def test_rows_on_both_sides_of_128_keys(H):
    """Blocks of either size in which delta comes from the weights for some rows and from o for others, among
    them blocks that begin with rows without keys and contexts that end at the border."""
    run(*make([300, 256, 129, 257], [200, 383, 129, 130], H, 45))


def test_scales_and_large_scores():
    kw, do = make([100], [130], 2, 27)
    run(kw, do, scale=0.4)
    kw["q"] = (kw["q"].float() * 20).to(BF16)
    run(kw, do)


@pytest.mark.parametrize("rise", [0.5, 2.0, 8.0])
def test_scores_that_grow_along_the_keys(rise):
    """The running maximum is met again and again, by a little or by a lot."""
    kw, do = make([500], [640], 2, 46)
    kw["q"] = (kw["q"].float() * 0.1 + 1).to(BF16)
    step = torch.linspace(0, 1, 640).view(1, 640, 1, 1) * rise
    kw["k_nope"] = (kw["k_nope"].float() * 0.1 + step).to(BF16)
    kw["k_rope"] = (kw["k_rope"].float() * 0.1 + step[..., 0]).to(BF16)
    run(kw, do)


def test_no_tokens():
    kw, do = make([0], [0], 2, 28, packed=False)
    d = dev(kw)
    o, lse = cdr.latent_attn_fwd(**d)
    assert o.shape == (1, 0, 2, 128) and lse.shape == (1, 0, 2)
    assert all(g.numel() == 0 for g in cdr.latent_attn_bwd(**d, o=o, lse=lse, do=do.to(DEV)))
    run(*make([3], [0], 2, 29, packed=False))
    run(*make([0], [3], 2, 30, packed=False))


def test_graph_replays():
    kw, do = make([150, 40], [170, 40], 2, 31)
    d, do = dev(kw), do.to(DEV)

    def step():
        o, lse = cdr.latent_attn_fwd(**d)
        return (o, lse) + cdr.latent_attn_bwd(**d, o=o, lse=lse, do=do)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed, lq, lk in ((41, (150, 40), (170, 40)), (42, (10, 180), (10, 200)), (43, (190, 0), (200, 10))):
        new, ndo = make(lq, lk, 2, seed)
        for k, v in new.items():
            d[k].copy_(v)
        do.copy_(ndo)
        graph.replay()
        torch.cuda.synchronize()
        compare(new, ndo, held[0], held[1], held[2:], 192 ** -0.5)
        for a, b in zip(held, step()):
            assert torch.equal(a, b)


def test_padded_graph_replays():
    """A captured step of 200 rows and 230 keys that holds fewer: what the last replay held and this one does not
    is empty again."""
    kw, do = make([150, 40], [170, 40], 2, 51, spare=10)
    kw["k_rope"], kv = kw["k_rope"].new_zeros(1, 230, 64), torch.zeros(1, 230, 2, 256, dtype=BF16)
    kw["k_nope"], kw["v"] = kv[..., :128], kv[..., 128:]
    d, do = dev(kw), do.to(DEV)

    def step():
        o, lse = cdr.latent_attn_fwd(**d)
        return (o, lse) + cdr.latent_attn_bwd(**d, o=o, lse=lse, do=do)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed, lq, lk in ((52, (150, 40), (170, 40)), (53, (3, 0), (9, 2)), (54, (0, 199), (10, 220)), (55, (0, 0), (0, 0))):
        new, ndo = make(lq, lk, 2, seed)
        for k, v in new.items():
            if k.startswith("cu"):
                d[k].copy_(v)
            else:
                d[k].fill_(math.nan)
                d[k][:, :v.shape[1]] = v.to(DEV)
        do.fill_(math.nan)
        do[:, :sum(lq)] = ndo.to(DEV)
        graph.replay()
        torch.cuda.synchronize()
        cut = lambda t, n: t[:, :n]  # noqa: E731
        a, b = sum(lq), sum(lk)
        compare(new, ndo, cut(held[0], a), cut(held[1], a), (cut(held[2], a),) + tuple(cut(t, b) for t in held[3:]),
                192 ** -0.5)
        for t, n, empty in zip(held, (a, a, a, b, b, b), (0, -math.inf, 0, 0, 0, 0)):
            assert (t[:, n:] == empty).all()
        for x, y in zip(held, step()):
            assert torch.equal(x, y)


def test_gradients_match_differences():
    """Directional differences of the forward itself: o's change along the gradient's direction, in the
    fp64 oracle's step, against the gradient's product with it."""
    kw, do = make([90], [90], 2, 32)
    _, _, dq, dk, dkr, dv = run(kw, do)
    g = torch.Generator().manual_seed(33)
    for name, grad in (("q", dq), ("k_nope", dk), ("k_rope", dkr), ("v", dv)):
        u = torch.randn(kw[name].shape, generator=g, dtype=torch.float64)
        step = 1e-5
        loss = []
        for s in (step, -step):
            moved = {k: v.double() if v.is_floating_point() else v for k, v in kw.items()}
            moved[name] = moved[name] + s * u
            loss.append(float((oracle_latent.attention(**moved, scale=192 ** -0.5)["o"] * do.double()).sum()))
        want = (loss[0] - loss[1]) / (2 * step)
        got = float((grad.cpu().double() * u).sum())
        # rounding of the gradient: at most 5 * 2^-8 of its absolute terms, of random sign
        assert abs(got - want) <= 5 * 2.0 ** -8 * float((grad.cpu().double().square() * u.square()).sum().sqrt()) * 4


def test_prefill_agrees_with_decode():
    """The two forms of one layer: keys and values expanded from latents, and the query absorbed."""
    g = torch.Generator().manual_seed(34)
    H, T = 4, 70
    c, r = torch.randn(T, 512, generator=g).to(BF16), torch.randn(T, 64, generator=g).to(BF16)
    wk, wv = (torch.randn(H, 128, 512, generator=g) / 512 ** 0.5 for _ in range(2))
    k = torch.einsum("hdc,tc->thd", wk, c.float()).to(BF16)
    v = torch.einsum("hdc,tc->thd", wv, c.float()).to(BF16)
    q = torch.randn(T, H, 192, generator=g).to(BF16)
    o, lse = cdr.latent_attn_fwd(q[None].to(DEV), k[None].to(DEV), r[None].to(DEV), v[None].to(DEV))
    qc = torch.einsum("thd,hdc->thc", q[:, :, :128].float(), wk).to(BF16)
    cache = torch.zeros(5, 16, 576, dtype=BF16, device=DEV)
    cdr.latent_cache_write(c.to(DEV), r.to(DEV), cache, torch.arange(T, dtype=torch.int32, device=DEV))
    oc, lse2 = cdr.latent_decode_fwd(qc[None].to(DEV), q[None, :, :, 128:].to(DEV), cache,
                                     torch.arange(5, dtype=torch.int32, device=DEV)[None],
                                     torch.tensor([T], dtype=torch.int32, device=DEV), 192 ** -0.5)
    back = torch.einsum("thc,hdc->thd", oc[0].cpu().float(), wv)
    # bf16 roundings of k, v and the absorbed q (2^-9 each at random) move scores of size ~1 and weights alike
    assert (lse.cpu() - lse2.cpu()).abs().max() < 0.05
    assert (o[0].cpu().float() - back).abs().max() < 0.05
