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
        length = min(max(lens[n], 0), len(table[n]) * page)
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
            seen = there & (torch.arange(length) < length - new + i + 1)
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
