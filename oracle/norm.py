"""fp64 oracle of the block boundary (norm, gate, residual scale, residual, next norm).

Written from the formulas: with ``R(x) = 1 / sqrt(mean x^2 + eps)`` over the last dimension,

    n = y R(y) w,   r = x + alpha s a(z) n,   h = r R(r) w2

The gradients use ``d(x R(x))/dx`` applied to p: ``R (p - x^ mean(p x^))``, ``x^ = x R``.  Every
result comes with a magnitude: the sum of the absolute values of the terms that make it up, which is
what fp32 rounding errors are relative to.
"""
import torch


def _f64(t):
    return None if t is None else t.detach().cpu().double()


def _act(z, act):
    sg = 1.0 / (1.0 + torch.exp(-z))
    if act == "sigmoid":
        return sg, sg * (1 - sg)
    return z * sg, sg * (1 + z * (1 - sg))


def block_norm(y, weight=None, gate=None, gate_act="sigmoid", residual=None, res_scale=None, next_weight=None,
               eps=1e-6, d_out=None, d_next=None):
    """``{name: (value, magnitude)}`` of r and h, and with d_out or d_next of dy, dweight, dgate, dresidual,
    dres_scale and dnext_weight (those that exist)."""
    y, w, z, x, w2 = (_f64(t) for t in (y, weight, gate, residual, next_weight))
    alpha, s = (1.0, _f64(res_scale)) if isinstance(res_scale, torch.Tensor) else \
        (1.0 if res_scale is None else float(res_scale), None)
    one = torch.ones(y.shape[-1], dtype=torch.float64)
    wf, sf = one if w is None else w, one if s is None else s
    rs = torch.rsqrt(y.square().mean(-1, keepdim=True) + eps) if w is not None else torch.ones_like(y[..., :1])
    hat = y * rs
    n = hat * wf
    a, slope = _act(z, gate_act) if z is not None else (torch.ones_like(y), torch.zeros_like(y))
    t = alpha * sf * a * n
    r = t if x is None else x + t
    rmag = t.abs() if x is None else x.abs() + t.abs()
    out = {"r": (r, rmag)}
    if w2 is not None:
        rr = torch.rsqrt(r.square().mean(-1, keepdim=True) + eps)
        rhat = r * rr
        # an error of r enters every element of its row through rr as well
        spread = (rmag * rhat.abs()).mean(-1, keepdim=True) * rr
        out["h"] = (rhat * w2, (rmag * rr + rhat.abs() * (1 + spread)) * w2.abs())
    if d_out is None and d_next is None:
        return out
    rows = tuple(range(y.dim() - 1))
    d = torch.zeros_like(y) if d_out is None else _f64(d_out)
    dmag = d.abs()
    if w2 is not None:
        dh = _f64(d_next)
        p = dh * w2
        m = (p * rhat).mean(-1, keepdim=True)
        hatmag = rmag * rr + rhat.abs() * (1 + spread)
        mmag = (p.abs() * hatmag).mean(-1, keepdim=True)
        d = d + rr * (p - rhat * m)
        dmag = dmag + rr * (1 + spread) * (p.abs() + hatmag * mmag)
        out["dnext_weight"] = ((dh * rhat).sum(rows), (dh.abs() * hatmag).sum(rows))
    if x is not None:
        out["dresidual"] = (d, dmag)
    k = abs(alpha)
    if s is not None:
        out["dres_scale"] = ((alpha * d * a * n).sum(rows), (k * dmag * (a * n).abs()).sum(rows))
    if z is not None:
        smag = (slope.abs() + 0.5)   # sigmoid's slope is formed as a difference of numbers near one
        out["dgate"] = (alpha * d * sf * n * slope, k * dmag * (sf * n).abs() * smag)
    p = alpha * d * sf * a
    pmag = k * dmag * (sf * a).abs()
    if w is None:
        out["dy"] = (p, pmag)
        return out
    out["dweight"] = ((p * hat).sum(rows), (pmag * hat.abs()).sum(rows))
    p, pmag = p * wf, pmag * wf.abs()
    m = (p * hat).mean(-1, keepdim=True)
    out["dy"] = (rs * (p - hat * m), rs * (pmag + hat.abs() * (pmag * hat.abs()).mean(-1, keepdim=True)))
    return out
