"""fp64 oracle of latent attention, written from the formulas, one sequence (and head) at a time.

Absorbed form over a paged cache: ``s_j = scale (q_c . c_j + q_r . r_j)``, ``o = sum softmax(s)_j
c_j``.  Results come with the magnitude ``sum_j p_j |c_j|`` and the size of the scores' terms, which
is what rounding errors are relative to.
"""
import math

import torch


def decode(q_latent, q_rope, cache, block_table, seq_lens, scale, cu_seqlens=None):
    """(o, lse, magnitude of o, largest sum of absolute score terms) on the CPU, q as the binding takes it.
    Rows outside every sequence stay NaN."""
    qc, qr, cache = (t.detach().cpu().double() for t in (q_latent, q_rope, cache))
    table, lens = block_table.tolist(), seq_lens.tolist()
    B, T, H = qc.shape[:3]
    o = torch.full((B * T, H, 512), math.nan, dtype=torch.float64)
    mag = o.clone()
    lse = torch.full((B * T, H), math.nan, dtype=torch.float64)
    size = lse.clone()
    P, page = cache.shape[:2]
    qc, qr = qc.reshape(B * T, H, 512), qr.reshape(B * T, H, 64)
    cu = [n * T for n in range(B + 1)] if cu_seqlens is None else cu_seqlens.tolist()
    for n in range(len(cu) - 1):
        total = max(lens[n], 0)
        length = min(total, len(table[n]) * page)
        keys = torch.zeros(length, 576, dtype=torch.float64)
        there = torch.zeros(length, dtype=torch.bool)
        for j in range(length):
            at = table[n][j // page]
            if 0 <= at < P:
                keys[j] = cache[at, j % page]
                there[j] = True
        new = cu[n + 1] - cu[n]
        for i in range(new):
            t = cu[n] + i
            seen = there & (torch.arange(length) < total - new + i + 1)
            if not seen.any():
                o[t], mag[t], size[t], lse[t] = 0, 0, 0, -math.inf
                continue
            c, r = keys[seen, :512], keys[seen, 512:]
            s = scale * (qc[t] @ c.T + qr[t] @ r.T)
            p = torch.softmax(s, -1)
            o[t], mag[t] = p @ c, p @ c.abs()
            lse[t] = torch.logsumexp(s, -1)
            size[t] = (abs(scale) * (qc[t].abs() @ c.abs().T + qr[t].abs() @ r.abs().T)).amax(-1)
    return o.reshape(B, T, H, 512), lse.reshape(B, T, H), mag.reshape(B, T, H, 512), size.reshape(B, T, H)


def attention(q, k_nope, k_rope, v, scale, cu_seqlens=None, cu_seqlens_k=None, do=None):
    """The expanded form in fp64 on the CPU, a sequence and head at a time: a dict of o, lse and, with do,
    dq, dk_nope, dk_rope, dv from the formulas (dS = P (do v^T - rowsum(do o))).  For each the dict also
    holds, under the name + "_mag", the sum of the absolute terms of its last product, and under "size"
    the largest sum of absolute score terms of each row.  What no sequence holds stays NaN."""
    q, k, r, v = (t.detach().cpu().double() for t in (q, k_nope, k_rope, v))
    B, T, H = q.shape[:3]
    Tk = k.shape[1]
    flat = lambda t: t.reshape((t.shape[0] * t.shape[1],) + tuple(t.shape[2:]))  # noqa: E731
    cuq = [n * T for n in range(B + 1)] if cu_seqlens is None else cu_seqlens.tolist()
    cuk = [n * Tk for n in range(B + 1)] if cu_seqlens is None else \
        (cu_seqlens if cu_seqlens_k is None else cu_seqlens_k).tolist()
    shapes = dict(o=v.shape[3], lse=0, size=0)
    out = {n: torch.full((B * T, H) + ((d,) if d else ()), math.nan, dtype=torch.float64) for n, d in shapes.items()}
    out["o_mag"] = out["o"].clone()
    nope = k.shape[3]
    qf, kf, rf, vf = flat(q), flat(k), flat(r), flat(v)
    df = None
    if do is not None:
        df = flat(do.detach().cpu().double())
        out["dq"] = torch.full(qf.shape, math.nan, dtype=torch.float64)
        out["dk_nope"], out["dv"] = (torch.full(t.shape, math.nan, dtype=torch.float64) for t in (kf, vf))
        out["dk_rope"] = torch.full(rf.shape, math.nan, dtype=torch.float64)
        for n in ("dq", "dk_nope", "dk_rope", "dv"):
            out[n + "_mag"] = out[n].clone()
    for n in range(len(cuq) - 1):
        a, b, e, f = cuq[n], cuq[n + 1], cuk[n], cuk[n + 1]
        seen = torch.arange(f - e)[None, :] < (f - e) - (b - a) + torch.arange(b - a)[:, None] + 1
        if do is not None:
            for name in ("dk_rope", "dk_rope_mag"):
                out[name][e:f] = 0
        for h in range(H):
            key = torch.cat([kf[e:f, h], rf[e:f]], -1)
            s = scale * (qf[a:b, h] @ key.T)
            s = torch.where(seen, s, torch.full_like(s, -math.inf))
            m = s.amax(-1, keepdim=True) if f > e else torch.full((b - a, 1), -math.inf, dtype=torch.float64)
            m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
            p = torch.exp(s - m)
            total = p.sum(-1, keepdim=True)
            out["lse"][a:b, h] = (m + torch.log(total))[:, 0]
            p = p / torch.where(total > 0, total, torch.ones_like(total))
            o = p @ vf[e:f, h]
            out["o"][a:b, h], out["o_mag"][a:b, h] = o, p @ vf[e:f, h].abs()
            size = abs(scale) * torch.where(seen, qf[a:b, h].abs() @ key.abs().T, torch.zeros_like(s))
            out["size"][a:b, h] = size.amax(-1) if f > e else 0
            if do is None:
                continue
            d = df[a:b, h]
            dp = d @ vf[e:f, h].T
            delta = (d * o).sum(-1, keepdim=True)
            ds = p * (dp - delta)
            # absolute terms: dp and delta are sums themselves, delta from the rounded o
            dsm = p * (d.abs() @ vf[e:f, h].abs().T + (d.abs() * out["o_mag"][a:b, h]).sum(-1, keepdim=True))
            out["dv"][e:f, h], out["dv_mag"][e:f, h] = p.T @ d, p.T @ d.abs()
            out["dq"][a:b, h], out["dq_mag"][a:b, h] = scale * ds @ key, abs(scale) * dsm @ key.abs()
            dk, dkm = scale * ds.T @ qf[a:b, h], abs(scale) * dsm.T @ qf[a:b, h].abs()
            out["dk_nope"][e:f, h], out["dk_nope_mag"][e:f, h] = dk[:, :nope], dkm[:, :nope]
            out["dk_rope"][e:f] += dk[:, nope:]
            out["dk_rope_mag"][e:f] += dkm[:, nope:]
    wide = {"o": q, "o_mag": q, "lse": q, "size": q, "dq": q, "dq_mag": q}
    return {n: t.reshape((B, T if n in wide else Tk) + tuple(t.shape[1:])) for n, t in out.items()}
