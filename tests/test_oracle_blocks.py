"""The oracles of the block boundary and of the page tables, on the CPU: gradients against central
differences in fp64, tables against hand-written ones, and the binding's refusals."""
import ctypes

import pytest
import torch

import chunked_gated_delta_chunk_amd as cdr
from chunked_gated_delta_chunk_amd import ops
from oracle.norm import block_norm
from oracle.pages import build_page_tables


def _inputs(D=7, rows=3, seed=0, post=True, gate=True, res=True, scale=True, pre=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    return dict(y=r(rows, D), weight=r(D) if post else None, gate=r(rows, D) if gate else None,
                residual=r(rows, D) if res else None, res_scale=r(D) if scale else None,
                next_weight=r(D) if pre else None), r(rows, D), r(rows, D) if pre else None


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("parts", [(1, 1, 1, 1, 1), (1, 1, 0, 0, 0), (0, 0, 1, 1, 1), (1, 0, 1, 0, 1), (0, 1, 0, 1, 0)])
def test_norm_gradients_match_differences(act, parts):
    kw, dr, dh = _inputs(post=parts[0], gate=parts[1], res=parts[2], scale=parts[3], pre=parts[4])
    got = block_norm(**kw, gate_act=act, d_out=dr, d_next=dh)

    def loss(**k):
        o = block_norm(**k, gate_act=act)
        return float((o["r"][0] * dr).sum() + ((o["h"][0] * dh).sum() if dh is not None else 0))

    names = dict(y="dy", weight="dweight", gate="dgate", residual="dresidual", res_scale="dres_scale",
                 next_weight="dnext_weight")
    step = 1e-6
    for name, t in kw.items():
        if t is None:
            assert names[name] not in got
            continue
        flat = t.reshape(-1)
        for i in range(0, flat.numel(), 3):
            keep = float(flat[i])
            flat[i] = keep + step
            up = loss(**kw)
            flat[i] = keep - step
            down = loss(**kw)
            flat[i] = keep
            # central differences: step^2 times the third derivative, and rounding of the loss / step
            assert abs((up - down) / (2 * step) - float(got[names[name]][0].reshape(-1)[i])) < 1e-6


def test_norm_magnitudes_cover_the_values():
    kw, dr, dh = _inputs()
    for name, (value, mag) in block_norm(**kw, d_out=dr, d_next=dh).items():
        assert (value.abs() <= mag * (1 + 1e-12)).all(), name


def test_page_tables_by_hand():
    # two tokens a page; request 0 holds 3 tokens (one place left), request 1 none, request 2 takes no token
    got = build_page_tables([2, 3, 0], [3, 0, 2], [[7, 8, -1], [-1, -1, -1], [5, -1, -1]], [9, 4, 6, 1], 1, 2, 7)
    assert got["cu_seqlens"] == [0, 2, 5, 5] and got["seq_lens"] == [5, 3, 2]
    assert got["block_table"] == [[7, 8, 4], [6, 1, -1], [5, -1, -1]]
    assert got["positions"] == [3, 4, 0, 1, 2, 0, 0]
    assert got["slot_map"] == [17, 8, 12, 13, 2, -1, -1]
    assert got["free_head"] == 4 and got["shortage"] == 0
    # one page short, a full row, a cut at three tokens
    got = build_page_tables([9, 2], [0, 1], [[-1, -1], [3, -1]], [5], 0, 2, 3)
    assert got["cu_seqlens"] == [0, 3, 3] and got["block_table"] == [[5, -1], [3, -1]]
    assert got["slot_map"] == [10, 11, -1] and got["shortage"] == 1 and got["free_head"] == 1


# --------------------------------------------------------------------------------------- refusals

def test_norm_struct_matches_header():
    import os
    import re
    text = open(os.path.join(os.path.dirname(ops.__file__), "..", "include", "chunk_dr.h")).read()
    body = re.search(r"typedef struct \{([^{}]*)\} cdr_block_norm_problem;", text).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    fields = re.findall(r"(?:int32_t|int64_t|float)\s+(\w+)(?:\[2\])?;", body)
    assert fields == [f[0] for f in ops.cdr_block_norm_problem._fields_]


def _problem(**kw):
    p = ops.cdr_block_norm_problem()
    p.rows, p.D, p.alpha, p.eps = 4, 8, 1.0, 1e-6
    for k, v in kw.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("kw,status", [
    (dict(), 0), (dict(rows=0), 0), (dict(D=8192), 0), (dict(rows=-1), 2), (dict(D=0), 2), (dict(D=8193), 3),
    (dict(dtype=2), 3), (dict(has_residual=1, res_dtype=5), 3), (dict(gate_act=3), 3), (dict(inner=3), 2),
    (dict(inner=2), 0), (dict(inner=-1), 2), (dict(eps=-1.0), 2), (dict(eps=float("nan")), 2),
])
def test_norm_check_status(kw, status):
    assert cdr.load_library().cdr_block_norm_check(ctypes.byref(_problem(**kw))) == status


def test_norm_rejects_missing_pointers_without_touching_device():
    lib = cdr.load_library()
    fake = 1 << 20
    p = _problem(has_weight=1)
    assert lib.cdr_block_norm_fwd(ctypes.byref(p), fake, None, None, None, None, None, fake, None, None) == 1
    p = _problem(has_next=1)
    assert lib.cdr_block_norm_fwd(ctypes.byref(p), fake, None, None, None, None, fake, fake, None, None) == 1
    p = _problem()   # no gradient of r and no next norm
    assert lib.cdr_block_norm_bwd(ctypes.byref(p), fake, *([None] * 5), None, None, fake, *([None] * 5), fake,
                                  1 << 20, None) == 1
    p = _problem(has_weight=1)
    assert lib.cdr_block_norm_bwd(ctypes.byref(p), fake, None, None, fake, None, None, fake, None, fake, None, None,
                                  fake, None, None, None, 0, None) == 5


def test_norm_binding_errors():
    y = torch.zeros(3, 8, dtype=torch.bfloat16)
    w = torch.ones(8)
    for bad, kw in ((TypeError, dict(y=y.half())), (TypeError, dict(weight=w.double())),
                    (ValueError, dict(weight=w[:4])), (ValueError, dict(gate=y[:2])),
                    (TypeError, dict(gate=y.float())), (ValueError, dict(gate=y, gate_act="relu")),
                    (ValueError, dict(gate=y, gate_act=None)), (TypeError, dict(residual=y.half())),
                    (ValueError, dict(next_out=y)), (ValueError, dict(out=y.t().contiguous().t())),
                    (ValueError, dict())):          # host tensors: no CPU path exists
        with pytest.raises(bad):
            cdr.block_norm_fwd(**{"y": y, **kw})
    with pytest.raises(ValueError, match="d_out"):
        cdr.block_norm_bwd(y, None)
    with pytest.raises(ValueError, match="together"):
        cdr.block_norm_bwd(y, y, next_weight=w)
    with pytest.raises(ValueError):
        cdr.block_norm_fwd(torch.zeros(1, 8193))


def test_pages_rejects_bad_arguments_without_touching_device():
    lib = cdr.load_library()
    fake = 1 << 20
    ok = [2, 4, 8, 16, 32]
    for i, v in ((0, 0), (1, 0), (2, -1), (3, 0), (4, -1)):
        sizes = list(ok)
        sizes[i] = v
        assert lib.cdr_build_page_tables(*sizes, *([fake] * 12), 64, None) == 2
    for i in range(11):
        args = [fake] * 11
        args[i] = None
        assert lib.cdr_build_page_tables(*ok, *args, fake, 64, None) == 1, i
    assert lib.cdr_build_page_tables(*ok, *([fake] * 11), fake, 4, None) == 5
    assert lib.cdr_build_page_tables(*ok, *([fake] * 11), None, 64, None) == 5


def test_pages_binding_errors():
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    good = dict(query_lens=i32(3), context_lens=i32(3), block_table=i32(3, 4), free_pages=i32(9), free_head=i32(1),
                page_size=16, max_tokens=8)
    for bad, kw in ((TypeError, dict(query_lens=i32(3).long())), (ValueError, dict(query_lens=i32(0))),
                    (ValueError, dict(context_lens=i32(2))), (ValueError, dict(block_table=i32(4, 3).t())),
                    (ValueError, dict(block_table=i32(2, 4))), (ValueError, dict(free_head=i32(2))),
                    (ValueError, dict(page_size=0)), (ValueError, dict(max_tokens=-1)),
                    (ValueError, dict(free_pages=i32(3, 3))), (ValueError, dict())):
        with pytest.raises(bad):
            cdr.build_page_tables(**{**good, **kw})


# ------------------------------------------------------------------------------ latent attention

def test_latent_decode_oracle_matches_a_plain_softmax():
    """One sequence on pages in order is plain attention over [c, r] with values c."""
    from oracle import latent
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    qc, qr, cache = r(1, 2, 3, 512), r(1, 2, 3, 64), r(3, 4, 576)
    table = torch.arange(3, dtype=torch.int32)[None]
    o, lse, mag, _ = latent.decode(qc, qr, cache, table, torch.tensor([9], dtype=torch.int32), 0.1)
    keys = cache.reshape(12, 576)[:9]
    s = torch.einsum("thd,jd->thj", torch.cat([qc, qr], -1)[0], keys) * 0.1
    s[0, :, 8] = float("-inf")
    p = torch.softmax(s, -1)
    assert torch.allclose(o[0], p @ keys[:, :512]) and torch.allclose(lse[0], torch.logsumexp(s, -1))
    assert (o.abs() <= mag + 1e-12).all()


def test_latent_decode_struct_and_check():
    import os
    import re
    text = open(os.path.join(os.path.dirname(ops.__file__), "..", "include", "chunk_dr.h")).read()
    body = re.search(r"typedef struct \{([^{}]*)\} cdr_latent_decode_problem;", text).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    fields = re.findall(r"(?:int32_t|int64_t|float)\s+(\w+)(?:\[2\])?;", body)
    assert fields == [f[0] for f in ops.cdr_latent_decode_problem._fields_]
    lib = cdr.load_library()
    ok = dict(N=2, T=1, H=16, varlen=0, num_pages=8, page_size=16, table_cols=4, scale=1.0)
    for kw, status in ((dict(), 0), (dict(N=0), 2), (dict(T=-1), 2), (dict(H=0), 2), (dict(num_pages=0), 2),
                       (dict(page_size=0), 2), (dict(table_cols=0), 2), (dict(page_size=12), 3),
                       (dict(num_pages=2 ** 30), 2), (dict(T=2 ** 28), 2), (dict(T=0), 0)):
        p = ops.cdr_latent_decode_problem(*{**ok, **kw}.values())
        assert lib.cdr_latent_decode_check(ctypes.byref(p)) == status, kw
        assert (lib.cdr_latent_decode_workspace_bytes(ctypes.byref(p)) > 0) == (status == 0)
    p = ops.cdr_latent_decode_problem(*ok.values())
    fake = 1 << 20
    args = [fake] * 5 + [None, fake, None, fake]
    big = 1 << 40
    for i in (0, 1, 2, 3, 4, 6):
        bad = list(args)
        bad[i] = None
        assert lib.cdr_latent_decode_fwd(ctypes.byref(p), *bad, big, None) == 1, i
    assert lib.cdr_latent_decode_fwd(ctypes.byref(p), *args, 64, None) == 5
    bad = list(args)
    bad[2] = fake + 8
    assert lib.cdr_latent_decode_fwd(ctypes.byref(p), *bad, big, None) == 3
    p.qc_stride[1] = 4
    assert lib.cdr_latent_decode_fwd(ctypes.byref(p), *args, big, None) == 3
    p = ops.cdr_latent_decode_problem(*{**ok, "varlen": 1}.values())
    assert lib.cdr_latent_decode_fwd(ctypes.byref(p), *args, big, None) == 1     # no cu_seqlens
    assert lib.cdr_latent_cache_write(1, 0, 16, fake, fake, 512, 64, fake, fake, None) == 2
    assert lib.cdr_latent_cache_write(-1, 1, 16, fake, fake, 512, 64, fake, fake, None) == 2
    assert lib.cdr_latent_cache_write(1, 1, 16, fake, fake, 12, 64, fake, fake, None) == 3
    assert lib.cdr_latent_cache_write(1, 1, 16, None, fake, 512, 64, fake, fake, None) == 1
    assert lib.cdr_latent_cache_write(1, 1, 16, fake, fake + 2, 512, 64, fake, fake, None) == 3


def test_latent_decode_binding_errors():
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    good = dict(q_latent=b(2, 1, 4, 512), q_rope=b(2, 1, 4, 64), cache=b(3, 16, 576), block_table=i(2, 2),
                seq_lens=i(2), scale=0.1)
    for bad, kw in ((ValueError, dict(q_latent=b(2, 1, 4, 256))), (TypeError, dict(q_latent=b(2, 1, 4, 512).float())),
                    (ValueError, dict(q_rope=b(2, 1, 3, 64))), (ValueError, dict(cache=b(3, 16, 512))),
                    (ValueError, dict(cache=b(3, 12, 576))), (TypeError, dict(block_table=i(2, 2).long())),
                    (ValueError, dict(block_table=i(3, 2))), (ValueError, dict(seq_lens=i(3))),
                    (ValueError, dict(cu_seqlens=i(3))), (ValueError, dict(out=b(2, 1, 512, 4).transpose(2, 3))),
                    (TypeError, dict(lse_out=b(2, 1, 4))), (ValueError, dict())):
        with pytest.raises(bad):
            cdr.latent_decode_fwd(**{**good, **kw})
    for bad, args in ((ValueError, (b(3, 512), b(3, 64), b(3, 16, 576), i(2))),
                      (ValueError, (b(3, 256), b(3, 64), b(3, 16, 576), i(3))),
                      (ValueError, (b(3, 512), b(2, 64), b(3, 16, 576), i(3))),
                      (TypeError, (b(3, 512), b(3, 64), b(3, 16, 576), i(3).long())),
                      (ValueError, (b(3, 512), b(3, 64), b(3, 16, 576), i(3)))):
        with pytest.raises(bad):
            cdr.latent_cache_write(*args)


def test_latent_outputs_over_inputs_are_refused():
    """An output that lies over an input, whole or in part, also over a strided one; neighbours are none."""
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    T, H = 6, 2
    q, kr = b(1, T, H, 192), b(1, T, 64)
    buf = b(4 * T * H * 128)
    part = lambda at: buf[at * T * H * 128 // 2:][:T * H * 128].view(1, T, H, 128)  # noqa: E731
    v, k = part(0), b(1, T, H, 128)
    kv = buf[:2 * T * H * 128].view(1, T, H, 256)
    lse = torch.zeros(1, T, H)
    for kw in (dict(v=v, out=v), dict(v=v, out=part(1)), dict(k_nope=part(2), out=part(2)),
               dict(k_nope=kv[..., :128], v=kv[..., 128:], out=part(1)), dict(k_nope=kv[..., :128], out=part(3)),
               dict(lse_out=kr.view(-1)[:2 * T * H].view(torch.float32).view(1, T, H))):
        with pytest.raises(ValueError, match="overlaps"):
            cdr.latent_attn_fwd(**{**dict(q=q, k_nope=k, k_rope=kr, v=b(1, T, H, 128)), **kw})
    with pytest.raises(ValueError, match="GPU"):      # apart: refused for nothing else than the device
        cdr.latent_attn_fwd(q, k, kr, v, out=part(2), lse_out=lse)
    with pytest.raises(ValueError, match="GPU"):
        cdr.latent_attn_fwd(q, kv[..., :128], kr, kv[..., 128:], out=part(4))
    ql = b(2, 1, 4, 512)
    good = dict(q_latent=ql, q_rope=b(2, 1, 4, 64), cache=b(3, 16, 576), block_table=i(2, 2), seq_lens=i(2), scale=0.1)
    for kw in (dict(out=ql), dict(out=good["cache"].view(-1)[576:][:4096].view(2, 1, 4, 512))):
        with pytest.raises(ValueError, match="overlaps"):
            cdr.latent_decode_fwd(**{**good, **kw})
    with pytest.raises(ValueError, match="GPU"):
        cdr.latent_decode_fwd(**good, out=b(2, 1, 4, 512))


def test_latent_attention_oracle_gradients_match_differences():
    from oracle import latent
    g = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    H, lq, lk = 2, (3, 2), (5, 2)
    x = dict(q=r(1, 5, H, 192), k_nope=r(1, 7, H, 128), k_rope=r(1, 7, 64), v=r(1, 7, H, 128))
    cu = dict(cu_seqlens=torch.tensor([0, 3, 5]), cu_seqlens_k=torch.tensor([0, 5, 7]))
    do = r(1, 5, H, 128)
    got = latent.attention(**x, **cu, scale=0.1, do=do)
    step = 1e-6
    for name, grad in (("q", "dq"), ("k_nope", "dk_nope"), ("k_rope", "dk_rope"), ("v", "dv")):
        flat = x[name].reshape(-1)
        for i in range(0, flat.numel(), flat.numel() // 23):
            keep = float(flat[i])
            loss = []
            for v in (keep + step, keep - step):
                flat[i] = v
                loss.append(float((latent.attention(**x, **cu, scale=0.1)["o"] * do).sum()))
            flat[i] = keep
            assert abs((loss[0] - loss[1]) / (2 * step) - float(got[grad].reshape(-1)[i])) < 1e-7
        assert (got[grad].abs() <= got[grad + "_mag"] + 1e-12).all()


def test_latent_attention_oracle_rows_without_keys():
    from oracle import latent
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    got = latent.attention(r(1, 4, 1, 192), r(1, 2, 1, 128), r(1, 2, 64), r(1, 2, 1, 128), 0.1, do=r(1, 4, 1, 128))
    assert (got["o"][0, :2] == 0).all() and (got["lse"][0, :2] == float("-inf")).all()
    assert (got["dq"][0, :2] == 0).all() and torch.isfinite(got["dk_rope"]).all()


def test_latent_attn_struct_and_check():
    import os
    import re
    text = open(os.path.join(os.path.dirname(ops.__file__), "..", "include", "chunk_dr.h")).read()
    body = re.search(r"typedef struct \{([^{}]*)\} cdr_latent_attn_problem;", text).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    fields = re.findall(r"(?:int32_t|int64_t|float)\s+(\w+)(?:\[2\])?;", body)
    assert fields == [f[0] for f in ops.cdr_latent_attn_problem._fields_]
    lib = cdr.load_library()
    ok = dict(N=2, T=9, Tk=9, H=4, varlen=0, scale=0.1)

    def problem(**kw):
        p = ops.cdr_latent_attn_problem(*{**ok, **{k: v for k, v in kw.items() if k in ok}}.values())
        for n, v in (("q_stride", (768, 192)), ("k_stride", (512, 128)), ("v_stride", (512, 128))):
            getattr(p, n)[:] = kw.get(n, v)
        p.k_rope_stride = kw.get("k_rope_stride", 64)
        return p

    for kw, status in ((dict(), 0), (dict(N=0), 2), (dict(T=-1), 2), (dict(Tk=-1), 2), (dict(H=0), 2),
                       (dict(scale=0.0), 2), (dict(scale=-1.0), 2), (dict(scale=float("nan")), 2),
                       (dict(scale=float("inf")), 2), (dict(H=40000), 3), (dict(T=2 ** 30), 2), (dict(Tk=2 ** 30), 2),
                       (dict(T=0), 0), (dict(Tk=0), 0), (dict(q_stride=(768, 4)), 3), (dict(k_stride=(-8, 128)), 3),
                       (dict(v_stride=(2 ** 23, 128)), 3), (dict(k_rope_stride=68), 3)):
        assert lib.cdr_latent_attn_check(ctypes.byref(problem(**kw))) == status, kw
    p = problem()
    fake, big = 1 << 20, 1 << 40
    args = [fake] * 4 + [None, None] + [fake, fake]
    for i in (0, 1, 2, 3, 6, 7):
        bad = list(args)
        bad[i] = None
        assert lib.cdr_latent_attn_fwd(ctypes.byref(p), *bad, None) == 1, i
    bad = list(args)
    bad[3] = fake + 8
    assert lib.cdr_latent_attn_fwd(ctypes.byref(p), *bad, None) == 3
    assert lib.cdr_latent_attn_fwd(ctypes.byref(problem(varlen=1)), *args, None) == 1
    args = [fake] * 4 + [None, None] + [fake] * 7
    for i in [0, 1, 2, 3] + list(range(6, 13)):
        bad = list(args)
        bad[i] = None
        assert lib.cdr_latent_attn_bwd(ctypes.byref(p), *bad, fake, big, None) == 1, i
    assert lib.cdr_latent_attn_bwd(ctypes.byref(p), *args, fake, 64, None) == 5
    assert lib.cdr_latent_attn_bwd(ctypes.byref(p), *args, fake + 4, big, None) == 5


def test_latent_attn_binding_errors():
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    good = dict(q=b(1, 5, 2, 192), k_nope=b(1, 5, 2, 128), k_rope=b(1, 5, 64), v=b(1, 5, 2, 128))
    for bad, kw in ((ValueError, dict(q=b(1, 5, 2, 128))), (TypeError, dict(q=b(1, 5, 2, 192).float())),
                    (ValueError, dict(k_nope=b(1, 5, 3, 128))), (ValueError, dict(k_rope=b(1, 4, 64))),
                    (ValueError, dict(v=b(1, 5, 2, 64))), (ValueError, dict(cu_seqlens_k=i(2))),
                    (ValueError, dict(cu_seqlens=i(2), cu_seqlens_k=i(3))), (TypeError, dict(cu_seqlens=i(2).long())),
                    (ValueError, dict(cu_seqlens=i(2), q=b(1, 4, 2, 192))), (ValueError, dict(scale=-0.1)),
                    (ValueError, dict(out=b(1, 5, 128, 2).transpose(2, 3))), (ValueError, dict())):
        with pytest.raises(bad):
            cdr.latent_attn_fwd(**{**good, **kw})
    two = dict(q=b(2, 5, 2, 192), k_nope=b(2, 5, 2, 128), k_rope=b(2, 5, 64), v=b(2, 5, 2, 128), cu_seqlens=i(2))
    with pytest.raises(ValueError):
        cdr.latent_attn_fwd(**two)
    o, lse = b(1, 5, 2, 128), torch.zeros(1, 5, 2)
    for bad, kw in ((ValueError, dict(o=b(1, 5, 2, 64))), (TypeError, dict(lse=b(1, 5, 2))),
                    (TypeError, dict(do=o.float())), (ValueError, dict())):
        with pytest.raises(bad):
            cdr.latent_attn_bwd(**{**good, "o": o, "lse": lse, "do": o, **kw})
