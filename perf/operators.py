"""The operators around the chunked gated delta rule, as cases that can be timed and compared.

Four kinds of case:

  norm    the norm after a token mixer, its gate, the residual and the norm before the next block, in one pass
          (``block_norm_fwd``), and with ``train`` its gradients too (``block_norm_bwd``)
  pages   a serving step's offsets, positions, page tables and slots from request lengths (``build_page_tables``)
  decode  latent attention in the absorbed form: the new tokens' latents are written into a paged cache and attended
          with everything before them (``latent_cache_write``, ``latent_decode_fwd``)
  attn    latent attention in the expanded form over packed sequences (``latent_attn_fwd``), and with ``train`` its
          gradients too (``latent_attn_bwd``)

With ``own`` false ``run`` computes them from elementary torch operations in 32 bits, rounded once at the end.
"""
import math

import torch

own = False

DEV = "cuda:0"
DC, DR = 512, 64          # latent and rope widths of a cached key
DN, DV = 128, 128         # head widths of the expanded form (nope part, value)
EPS = 1e-6
BF16, F32 = torch.bfloat16, torch.float32


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step's gated head norm: 256 sequences x 16 heads of 128
        dict(name="gated head norm, decode", kind="norm", rows=256 * 16, D=128, post=True, gate="sigmoid",
             residual=False, pre=False, scale=False, dtype="bf16", res="bf16", train=False),
        # prefill of 8192 tokens at width 2048: norm, gate, learned residual scale, fp32 residual stream, next norm
        dict(name="block norm, 8192 x 2048", kind="norm", rows=8192, D=2048, post=True, gate="silu",
             residual=True, pre=True, scale=True, dtype="bf16", res="fp32", train=False),
        # the same block boundary in a training step
        dict(name="block norm train, 8192 x 2048", kind="norm", rows=8192, D=2048, post=True, gate="silu",
             residual=True, pre=True, scale=True, dtype="bf16", res="bf16", train=True),
        # an odd width and row count, everything in fp32, residual add and next norm without a gate
        dict(name="residual norm train, odd", kind="norm", rows=1021, D=1537, post=False, gate="none",
             residual=True, pre=True, scale=True, dtype="fp32", res="fp32", train=True),
        # a decode step of 256 requests, one token each
        dict(name="page tables, decode", kind="pages", n=256, context=8192, new=1, ragged=True, page=64, spare=0),
        # a ragged prefill of 64 requests, up to 2048 tokens each, padded to a captured size
        dict(name="page tables, prefill", kind="pages", n=64, context=1024, new=2048, ragged=True, page=16,
             spare=1000),
        # one user, one token: latency
        dict(name="latent decode, 1 x 8192", kind="decode", n=1, t=1, H=16, context=8192, ragged=False, page=64),
        # a full serving batch of ragged lengths, 16 heads a device
        dict(name="latent decode, 256 ragged", kind="decode", n=256, t=1, H=16, context=8192, ragged=True, page=64),
        # four draft tokens a sequence, 64 heads
        dict(name="latent decode, 64 x 4 drafts", kind="decode", n=64, t=4, H=64, context=4096, ragged=True, page=16),
        # a packed prefill, odd lengths, 16 heads
        dict(name="latent attention, packed", kind="attn", n=5, T=8168, H=16, context=0, ragged=True, train=False),
        # one long training sequence, forward and backward
        dict(name="latent attention train, 8192", kind="attn", n=1, T=8192, H=16, context=0, ragged=False,
             train=True),
        # a short ragged training batch
        dict(name="latent attention train, ragged", kind="attn", n=7, T=1001, H=8, context=0, ragged=True,
             train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "norm", "pages", "decode", "decode", "attn", "attn"])
    if kind == "norm":
        D = rng.choice([128, _log(rng, 32, 8192), 8 * _log(rng, 8, 1024)])
        rows = _log(rng, 1, max(2, min(131072, 16_000_000 // D)))
        post, pre = rng.choice([(True, True), (True, False), (False, True)])
        return dict(kind=kind, rows=rows, D=D, post=post, gate=rng.choice(["none", "sigmoid", "silu"]),
                    residual=pre or rng.random() < 0.5, pre=pre, scale=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "bf16", "fp32"]), res=rng.choice(["bf16", "fp32"]),
                    train=rng.random() < 0.5)
    if kind == "pages":
        return dict(kind=kind, n=_log(rng, 1, 1024), context=_log(rng, 1, 16384), new=_log(rng, 1, 512),
                    ragged=rng.random() < 0.7, page=rng.choice([1, 16, 32, 64, 128]), spare=rng.choice([0, 1, 333]))
    if kind == "decode":
        H = rng.choice([1, 4, 16, 20, 32, 64, 128])
        t = rng.choice([1, 1, 2, 4])
        context = _log(rng, 1, 16384)
        n = _log(rng, 1, max(2, min(256, 33_000_000 // (context * t * H))))
        return dict(kind=kind, n=n, t=t, H=H, context=context, ragged=rng.random() < 0.7,
                    page=rng.choice([1, 16, 32, 64, 128]))
    H = rng.choice([1, 3, 8, 16])
    T = _log(rng, 17, 4500)
    return dict(kind=kind, n=rng.choice([1, 1, 2, 5, 9]), T=T, H=H,
                context=rng.choice([0, 0, _log(rng, 1, 2000)]), ragged=rng.random() < 0.6,
                train=rng.random() < 0.5)


def _spread(n, top, ragged):
    """n lengths up to `top`: all `top`, or spread evenly over 1..top in a mixed order, the first the longest."""
    if not ragged:
        return [top] * n
    return [top if i == 0 else 1 + int((top - 1) * ((i * 0.6180339887498949) % 1.0)) for i in range(n)]


def _split(n, total, ragged):
    """`total` tokens over n sequences: evenly, or in the shares of _spread; the last takes what is left."""
    share = _spread(n, 1000, ragged)
    got = [total * s // sum(share) for s in share]
    got[-1] += total - sum(got)
    return got


def _offsets(lens):
    out = [0]
    for x in lens:
        out.append(out[-1] + x)
    return out


def _attn_lens(case):
    lq = _split(case["n"], case["T"], case["ragged"])
    ctx = _spread(case["n"], case["context"], case["ragged"]) if case["context"] else [0] * case["n"]
    return lq, [a + b for a, b in zip(lq, ctx)]


# ---------------------------------------------------------------------------------------- prepare

def prepare(case, seed):
    g = torch.Generator(DEV).manual_seed(int(seed))
    c = dict(case)

    def randn(*shape, dtype=BF16):
        return torch.randn(*shape, generator=g, device=DEV, dtype=F32).to(dtype)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device=DEV)

    if c["kind"] == "norm":
        dt, rdt = (BF16 if c["dtype"] == "bf16" else F32), (BF16 if c["res"] == "bf16" else F32)
        R, D = c["rows"], c["D"]
        c["y"] = randn(R, D, dtype=dt)
        c["z"] = randn(R, D, dtype=dt) if c["gate"] != "none" else None
        c["x"] = randn(R, D, dtype=rdt) if c["residual"] else None
        c["w"] = 1 + 0.1 * randn(D, dtype=F32) if c["post"] else None
        c["w2"] = 1 + 0.1 * randn(D, dtype=F32) if c["pre"] else None
        c["s"] = 0.3 + 0.1 * randn(D, dtype=F32) if c["scale"] else None
        c["dr"] = randn(R, D, dtype=rdt if c["residual"] else dt) if c["train"] else None
        c["dh"] = randn(R, D, dtype=dt) if c["train"] and c["pre"] else None
    elif c["kind"] == "pages":
        n, ps = c["n"], c["page"]
        roll = torch.randperm(n, generator=g, device=DEV).tolist()
        ctx = [_spread(n, c["context"], c["ragged"])[i] for i in roll]
        new = [_spread(n, c["new"], c["ragged"])[i] for i in roll[::-1]]
        cols = -(-(c["context"] + c["new"]) // ps)
        held = [-(-x // ps) for x in ctx]
        want = sum(-(-(x + y) // ps) for x, y in zip(ctx, new))
        pages = torch.randperm(want + 8, generator=g, device=DEV).to(torch.int32)
        at = torch.arange(cols, device=DEV)[None, :]
        mine = at < ints(held)[:, None]
        table = torch.full((n, cols), -1, dtype=torch.int32, device=DEV)
        table[mine] = pages[:sum(held)]
        c["table"], c["free"], c["page_count"] = table, pages, want + 8
        c["head"] = ints([sum(held)])
        c["context_lens"], c["query_lens"] = ints(ctx), ints(new)
        c["tokens"] = sum(new) + c["spare"]
    elif c["kind"] == "decode":
        n, t, H, ps = c["n"], c["t"], c["H"], c["page"]
        lens = [x + t for x in _spread(n, c["context"], c["ragged"])]
        roll = torch.randperm(n, generator=g, device=DEV).tolist()
        lens = [lens[i] for i in roll]
        cols = -(-max(lens) // ps)
        pages = sum(-(-x // ps) for x in lens)
        own_pages = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        mine = torch.arange(cols, device=DEV)[None, :] < ints([-(-x // ps) for x in lens])[:, None]
        table = torch.full((n, cols), -1, dtype=torch.int32, device=DEV)
        table[mine] = own_pages
        c["table"], c["seq_lens"] = table, ints(lens)
        c["longest"] = max(lens)
        c["cache"] = torch.randn(pages, ps, DC + DR, generator=g, device=DEV, dtype=BF16)
        c["qc"], c["qr"] = randn(n, t, H, DC), randn(n, t, H, DR)
        c["c_new"], c["r_new"] = randn(n * t, DC), randn(n * t, DR)
        pos = (ints(lens)[:, None] - t + torch.arange(t, device=DEV)[None, :]).long()
        c["slots"] = (table.long().gather(1, pos // ps) * ps + pos % ps).reshape(-1).to(torch.int32)
        c["scale"] = (DN + DR) ** -0.5
    else:
        lq, lk = _attn_lens(c)
        H = c["H"]
        c["cu_q"], c["cu_k"] = ints(_offsets(lq)), ints(_offsets(lk))
        Tq, Tk = sum(lq), sum(lk)
        c["q"] = randn(1, Tq, H, DN + DR)
        kv = randn(1, Tk, H, DN + DV)                  # one projection's output, read in place
        c["k"], c["v"] = kv[..., :DN], kv[..., DN:]
        c["kr"] = randn(1, Tk, DR)
        c["do"] = randn(1, Tq, H, DV) if c["train"] else None
        c["scale"] = (DN + DR) ** -0.5
    return c


# ---------------------------------------------------------------------------------- the calls

def run(c):
    if own:
        return {"norm": _own_norm, "pages": _own_pages, "decode": _own_decode, "attn": _own_attn}[c["kind"]](c)
    return {"norm": _norm, "pages": _pages, "decode": _decode, "attn": _attn}[c["kind"]](c)


def _named(**kw):
    return {k: v for k, v in kw.items() if v is not None}


def _own_norm(c):
    import chunked_gated_delta_chunk_amd as cdr
    kw = dict(weight=c["w"], gate=c["z"], gate_act=None if c["gate"] == "none" else c["gate"], residual=c["x"],
              res_scale=c["s"], next_weight=c["w2"], eps=EPS)
    r, h = cdr.block_norm_fwd(c["y"], **kw)
    if not c["train"]:
        return _named(r=r, h=h)
    dy, dw, dz, dx, ds, dw2 = cdr.block_norm_bwd(c["y"], c["dr"], c["dh"], **kw)
    return _named(r=r, h=h, dy=dy, dw=dw, dz=dz, dx=dx, ds=ds, dw2=dw2)


def _own_pages(c):
    import chunked_gated_delta_chunk_amd as cdr
    t = cdr.build_page_tables(c["query_lens"], c["context_lens"], c["table"], c["free"], c["head"], c["page"],
                              c["tokens"], free_head_out=c.setdefault("head_out", torch.empty_like(c["head"])))
    return dict(cu=t.cu_seqlens, seq_lens=t.seq_lens, positions=t.positions, slots=t.slot_map, table=c["table"],
                head=t.free_head, short=t.shortage)


def _own_decode(c):
    import chunked_gated_delta_chunk_amd as cdr
    cdr.latent_cache_write(c["c_new"], c["r_new"], c["cache"], c["slots"])
    o, lse = cdr.latent_decode_fwd(c["qc"], c["qr"], c["cache"], c["table"], c["seq_lens"], scale=c["scale"])
    return dict(o=o, lse=lse, cache=c["cache"])


def _own_attn(c):
    import chunked_gated_delta_chunk_amd as cdr
    kw = dict(scale=c["scale"], cu_seqlens=c["cu_q"], cu_seqlens_k=c["cu_k"])
    o, lse = cdr.latent_attn_fwd(c["q"], c["k"], c["kr"], c["v"], **kw)
    if not c["train"]:
        return dict(o=o, lse=lse)
    dq, dk, dkr, dv = cdr.latent_attn_bwd(c["q"], c["k"], c["kr"], c["v"], o, lse, c["do"], **kw)
    return dict(o=o, lse=lse, dq=dq, dk=dk, dkr=dkr, dv=dv)


# ---------------------------------------------------------------------------- the plain forms

def _norm(c):
    y = c["y"].float()
    D = c["D"]
    w = c["w"] if c["w"] is not None else torch.ones(D, device=DEV)
    s = c["s"] if c["s"] is not None else torch.ones(D, device=DEV)
    rs = torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) if c["post"] else torch.ones_like(y[:, :1])
    n = y * rs * w
    if c["gate"] == "none":
        a = torch.ones_like(y)
    else:
        z = c["z"].float()
        sg = 1 / (1 + torch.exp(-z))
        a = sg if c["gate"] == "sigmoid" else z * sg
    r = s * a * n
    if c["residual"]:
        r = r + c["x"].float()
    rt = c["x"].dtype if c["residual"] else c["y"].dtype
    out = dict(r=r.to(rt))
    if c["pre"]:
        rr = torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS)
        out["h"] = (r * rr * c["w2"]).to(c["y"].dtype)
    if not c["train"]:
        return out
    d = c["dr"].float()
    if c["pre"]:
        dh = c["dh"].float()
        hat = r * rr
        p = dh * c["w2"]
        d = d + rr * (p - hat * (p * hat).mean(-1, keepdim=True))
        out["dw2"] = (dh * hat).sum(0)
    if c["residual"]:
        out["dx"] = d.to(rt)
    if c["s"] is not None:
        out["ds"] = (d * a * n).sum(0)
    if c["gate"] != "none":
        slope = sg * (1 - sg) if c["gate"] == "sigmoid" else sg * (1 + z * (1 - sg))
        out["dz"] = (d * s * n * slope).to(c["z"].dtype)
    dn = d * s * a
    if c["post"]:
        hat = y * rs
        out["dw"] = (dn * hat).sum(0)
        p = dn * w
        dn = rs * (p - hat * (p * hat).mean(-1, keepdim=True))
    out["dy"] = dn.to(c["y"].dtype)
    return out


def _pages(c):
    ps, cap = c["page"], c["tokens"]
    table, free, head = c["table"], c["free"].long(), c["head"].long()
    n, cols = table.shape
    ctx = c["context_lens"].long()
    zero = torch.zeros(1, dtype=torch.long, device=DEV)
    cu = torch.cat([zero, c["query_lens"].long().cumsum(0)]).clamp(max=cap)
    lens = ctx + cu[1:] - cu[:-1]
    held, full = ((ctx + ps - 1) // ps).clamp(max=cols), (lens + ps - 1) // ps
    upto = full.clamp(max=cols)
    need = upto - held
    first = head + need.cumsum(0) - need
    at = torch.arange(cols, device=DEV)[None, :]
    src = first[:, None] + at - held[:, None]
    taken = torch.where(src < free.numel(), free[src.clamp(0, free.numel() - 1)], -1)
    new = torch.where((at >= held[:, None]) & (at < upto[:, None]), taken, table.long())
    t = torch.arange(cap, device=DEV)
    row = torch.bucketize(t, cu[1:].contiguous(), right=True)
    used = row < n
    row = row.clamp(max=n - 1)
    pos = torch.where(used, ctx[row] + t - cu[row], 0)
    j = pos // ps
    pg = new[row, j.clamp(max=cols - 1)]
    slot = torch.where(used & (j < cols) & (pg >= 0), pg * ps + pos % ps, -1)
    end = head + need.sum()
    short = (end - free.numel()).clamp(min=0) + (full - upto).sum()
    table.copy_(new)
    i32 = torch.int32
    return dict(cu=cu.to(i32), seq_lens=lens.to(i32), positions=pos.to(i32), slots=slot.to(i32), table=table,
                head=end.clamp(max=free.numel()).to(i32), short=short.to(i32))


def _decode(c):
    n, t, H, ps = c["n"], c["t"], c["H"], c["page"]
    cache = c["cache"]
    flat = cache.view(-1, DC + DR)
    flat[c["slots"].long()] = torch.cat([c["c_new"], c["r_new"]], 1)
    L = c["longest"]
    j = torch.arange(L, device=DEV)
    page = c["table"].long()[:, j // ps].clamp(min=0)
    keys = flat[page * ps + j % ps].float()                                        # [n, L, 576]
    q = torch.cat([c["qc"], c["qr"]], -1).float().reshape(n, t * H, DC + DR)
    s = torch.bmm(keys, q.transpose(1, 2).contiguous()).transpose(1, 2) * c["scale"]
    s = s.reshape(n, t, H, L)
    last = c["seq_lens"].long()[:, None] - t + torch.arange(t, device=DEV)[None, :]   # [n, t]
    s = torch.where(j[None, None, None, :] <= last[:, :, None, None], s, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    o = torch.bmm((p / l).reshape(n, t * H, L), keys[..., :DC].contiguous()).reshape(n, t, H, DC)
    return dict(o=o.to(BF16), lse=(m + torch.log(l))[..., 0], cache=cache)


def _attn(c):
    H, scale = c["H"], c["scale"]
    heads = lambda x: x[0].float().transpose(0, 1).contiguous()  # noqa: E731   [H, T, .]
    q, k, v = heads(c["q"]), heads(c["k"]), heads(c["v"])
    Tq, Tk = q.shape[1], k.shape[1]
    k = torch.cat([k, c["kr"][0].float()[None].expand(H, Tk, DR)], -1)
    cuq, cuk = c["cu_q"].long(), c["cu_k"].long()
    i, j = torch.arange(Tq, device=DEV), torch.arange(Tk, device=DEV)
    ni = torch.bucketize(i, cuq[1:].contiguous(), right=True)
    nj = torch.bucketize(j, cuk[1:].contiguous(), right=True)
    lq, lk = cuq[1:] - cuq[:-1], cuk[1:] - cuk[:-1]
    last = i - cuq[ni] + (lk - lq)[ni]
    seen = (ni[:, None] == nj[None, :]) & ((j - cuk[nj])[None, :] <= last[:, None])
    s = torch.bmm(q, k.transpose(1, 2).contiguous()).mul_(scale).masked_fill_(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    p = p.div_(l)
    o = torch.bmm(p, v)
    back = lambda x: x.transpose(0, 1)[None].to(BF16).contiguous()  # noqa: E731
    out = dict(o=back(o), lse=(m + torch.log(l))[..., 0].transpose(0, 1)[None].contiguous())
    if not c["train"]:
        return out
    do = heads(c["do"])
    delta = (do * o).sum(-1, keepdim=True)
    dv = torch.bmm(p.transpose(1, 2).contiguous(), do)
    ds = torch.bmm(do, v.transpose(1, 2).contiguous()).sub_(delta).mul_(p).mul_(scale)
    dq = torch.bmm(ds, k)
    dk = torch.bmm(ds.transpose(1, 2).contiguous(), q)
    return dict(out, dq=back(dq), dk=back(dk[..., :DN]), dkr=dk[..., DN:].sum(0)[None].to(BF16), dv=back(dv))


# ------------------------------------------------------------------------------------ work, exact

def work(case):
    c = case
    if c["kind"] == "norm":
        e, er = (2 if c["dtype"] == "bf16" else 4), (2 if c["res"] == "bf16" else 4)
        n = c["rows"] * c["D"]
        rt = er if c["residual"] else e
        each = e + e * (c["gate"] != "none") + er * c["residual"] + rt + e * c["pre"]
        if c["train"]:     # dr, dh in; dy, dz, dx out; y, z, x are there already
            each += rt + e * c["pre"] + e + e * (c["gate"] != "none") + er * c["residual"]
        vec = 4 * c["D"] * (c["post"] + c["pre"] + c["scale"]) * (2 if c["train"] else 1)
        return {"bytes": n * each + vec, "flops": n * (20 if not c["train"] else 60)}
    if c["kind"] == "pages":
        n, ps = c["n"], c["page"]
        ctx, new = _spread(n, c["context"], c["ragged"]), _spread(n, c["new"], c["ragged"])
        tokens = sum(new) + c["spare"]
        pages = sum(new) // ps + n
        return {"bytes": 4 * (3 * n + 2 * pages + n + 2 * tokens), "flops": 4 * tokens + 8 * n}
    if c["kind"] == "decode":
        n, t, H = c["n"], c["t"], c["H"]
        lens = [x + t for x in _spread(n, c["context"], c["ragged"])]
        keys = sum(lens)
        rows = n * t * H
        return {"bytes": 2 * (DC + DR) * (keys + 2 * n * t) + rows * (2 * (DC + DR) + 2 * DC + 4)
                + 4 * sum(-(-x // c["page"]) for x in lens),
                "flops": 2 * (2 * DC + DR) * H * t * keys}
    lq, lk = _attn_lens(c)
    H = c["H"]
    pairs = sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(lq, lk)) * H
    Tq, Tk = sum(lq), sum(lk)
    fwd_b = 2 * (Tq * H * (DN + DR + DV) + Tk * H * (DN + DV) + Tk * DR) + 4 * Tq * H
    fwd_f = 2 * (DN + DR + DV) * pairs
    if not c["train"]:
        return {"bytes": fwd_b, "flops": fwd_f}
    bwd_b = 2 * (Tq * H * (DN + DR + DV) + Tk * H * (DN + DV) + Tk * DR)
    return {"bytes": fwd_b + bwd_b, "flops": fwd_f + 2 * (3 * (DN + DR) + 2 * DV) * pairs}


def exact(case, seed):
    if case["kind"] == "pages":
        return None
    c = prepare(case, seed)
    return {"norm": _exact_norm, "decode": _exact_decode, "attn": _exact_attn}[case["kind"]](c)


def _leaf(x):
    return None if x is None else x.double().requires_grad_(True)


def _exact_norm(c):
    y, z, x, w, w2, s = (_leaf(c[k]) for k in ("y", "z", "x", "w", "w2", "s"))
    with torch.enable_grad():
        r = y
        if w is not None:
            r = w * r / torch.sqrt((r * r).sum(-1, keepdim=True) / c["D"] + EPS)
        if z is not None:
            r = r * torch.sigmoid(z) * (z if c["gate"] == "silu" else 1.0)
        if s is not None:
            r = r * s
        if x is not None:
            r = x + r
        h = None
        if w2 is not None:
            h = w2 * r / torch.sqrt((r * r).sum(-1, keepdim=True) / c["D"] + EPS)
        out = _named(r=r, h=h)
        if c["train"]:
            total = (r * c["dr"].double()).sum()
            if h is not None:
                total = total + (h * c["dh"].double()).sum()
            wanted = _named(dy=y, dw=w, dz=z, dx=x, ds=s, dw2=w2)
            out.update(zip(wanted, torch.autograd.grad(total, list(wanted.values()))))
    return {k: v.detach() for k, v in out.items()}


def _exact_decode(c):
    t, ps = c["t"], c["page"]
    cache = c["cache"].clone()
    flat = cache.view(-1, DC + DR)
    flat[c["slots"].long(), :DC] = c["c_new"]
    flat[c["slots"].long(), DC:] = c["r_new"]
    o = torch.empty(c["qc"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(o.shape[:3], dtype=torch.float64, device=DEV)
    for n, length in enumerate(c["seq_lens"].tolist()):
        pages = c["table"][n, :-(-length // ps)].long()
        keys = cache[pages].reshape(-1, DC + DR)[:length].double()
        for i in range(t):
            upto = length - t + i + 1
            s = c["scale"] * (c["qc"][n, i].double() @ keys[:upto, :DC].T + c["qr"][n, i].double() @ keys[:upto, DC:].T)
            lse[n, i] = torch.logsumexp(s, -1)
            o[n, i] = torch.softmax(s, -1) @ keys[:upto, :DC]
    return dict(o=o, lse=lse, cache=None)


def _exact_attn(c):
    names = ("q", "k", "kr", "v")
    q, k, kr, v = (c[x].double() for x in names)
    o = torch.zeros(q.shape[:3] + (DV,), dtype=torch.float64, device=DEV)
    lse = torch.full(q.shape[:3], -math.inf, dtype=torch.float64, device=DEV)
    grads = [torch.zeros_like(x) for x in (q, k, kr, v)]
    cuq, cuk = c["cu_q"].tolist(), c["cu_k"].tolist()
    for a, b, e, f in zip(cuq, cuq[1:], cuk, cuk[1:]):
        if a == b or e == f:
            continue
        hide = torch.ones(b - a, f - e, dtype=torch.bool, device=DEV).triu(f - e - (b - a) + 1)
        for h in range(c["H"]):
            with torch.enable_grad():
                x = [_leaf(q[0, a:b, h]), _leaf(k[0, e:f, h]), _leaf(kr[0, e:f]), _leaf(v[0, e:f, h])]
                s = c["scale"] * (x[0][:, :DN] @ x[1].T + x[0][:, DN:] @ x[2].T)
                s = s.masked_fill(hide, -math.inf)
                out = torch.softmax(s, -1) @ x[3]
                o[0, a:b, h] = out.detach()
                lse[0, a:b, h] = torch.logsumexp(s.detach(), -1)
                if c["train"]:
                    d = torch.autograd.grad((out * c["do"][0, a:b, h].double()).sum(), x)
                    grads[0][0, a:b, h] = d[0]
                    grads[1][0, e:f, h] = d[1]
                    grads[2][0, e:f] += d[2]
                    grads[3][0, e:f, h] = d[3]
    if not c["train"]:
        return dict(o=o, lse=lse)
    return dict(o=o, lse=lse, dq=grads[0], dk=grads[1], dkr=grads[2], dv=grads[3])
