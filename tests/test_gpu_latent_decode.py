"""Latent attention over a paged cache (absorbed form) on the GPU against the fp64 oracle.

Tolerances.  A score is 576 exact products of bf16 added in fp32: an error of at most 577 roundings
of 2^-24 of the sum of the absolute terms (`size`), and as much again for scale and base-2 steps;
call that e = (577 + 8) 2^-24 size.  The same e, plus the sum over at most 4096 weights (each lane
adds few, the rest is a tree: 64 + 8 roundings) and the logarithm, bounds lse's error.  The weights
exp(s - m) have relative error e + 4 2^-24 and are rounded to bf16 (2^-9 of nearest even, 2^-8 allowed)
in the numerator but not in the sum; o is then at most (2^-8 + 2 e + 2^-16) times the magnitude
sum p |c| away, plus its own half step.
"""
import math

import pytest
import torch

import chunked_gated_delta_chunk_amd as cdr
from oracle import latent as oracle_latent

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16
SCALE = 192 ** -0.5


def make(lens, T, H, page, seed, spare_cols=1, extra_pages=3, packed=None):
    """q, cache and tables: random distinct pages, everything outside the sequences' keys NaN."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(BF16)  # noqa: E731
    N = len(lens)
    shape = (N, T, H) if packed is None else (1, sum(packed) + 2, H)
    held = [-(-max(x, 0) // page) for x in lens]
    cols = max(max(held), 1) + spare_cols
    P = sum(held) + extra_pages
    pages = torch.randperm(P, generator=g).tolist()
    cache = torch.full((P, page, 576), math.nan, dtype=BF16)
    table = torch.full((N, cols), 2 ** 30, dtype=torch.int32)
    at = 0
    for n, k in enumerate(held):
        for j in range(k):
            table[n, j] = pages[at]
            fill = min(page, lens[n] - j * page)
            cache[pages[at], :fill] = r(fill, 576)
            at += 1
    cu = None
    if packed is not None:
        cu = torch.tensor([0] + list(packed)).cumsum(0).to(torch.int32)
    return dict(q_latent=r(*shape, 512), q_rope=r(*shape, 64), cache=cache, block_table=table,
                seq_lens=torch.tensor(lens, dtype=torch.int32), cu_seqlens=cu)


def dev(kw):
    return {k: v.to(DEV) if isinstance(v, torch.Tensor) else v for k, v in kw.items()}


def compare(kw, o, lse, scale=SCALE):
    o_ref, lse_ref, mag, size = oracle_latent.decode(scale=scale, **kw)
    o, lse = o.cpu().double(), lse.cpu().double()
    live = ~torch.isnan(lse_ref)
    assert torch.isfinite(o[live]).all()
    empty = live & torch.isinf(lse_ref)
    assert (o[empty] == 0).all() and (lse[empty] == -math.inf).all()
    full = live & ~empty
    e = 585 * 2.0 ** -24 * size + 80 * 2.0 ** -24
    d = ((lse - lse_ref).abs() / (e + 2.0 ** -22 * lse_ref.abs()))[full]
    assert not d.numel() or float(d.max()) <= 1, f"lse: {float(d.max()):.3f} of the tolerance"
    tol = (2.0 ** -8 + 2 * e + 2.0 ** -16)[..., None] * mag + 2.0 ** -8 * o_ref.abs() + 1e-30
    d = ((o - o_ref).abs() / tol)[full]
    assert not d.numel() or float(d.max()) <= 1, f"o: {float(d.max()):.3f} of the tolerance"


def run(kw, scale=SCALE, **more):
    o, lse = cdr.latent_decode_fwd(**dev(kw), scale=scale, **more)
    compare(kw, o, lse, scale)
    return o, lse


@pytest.mark.parametrize("H", [1, 3, 16, 17, 32, 33, 64, 128])
@pytest.mark.parametrize("T", [1, 2, 5])
def test_heads_and_tokens(H, T):
    run(make([T, 63 + T, 130], T, H, 16, 100 * H + T))


@pytest.mark.parametrize("page", [1, 2, 16, 64, 256])
def test_lengths_and_pages(page):
    run(make([1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 511], 1, 16, page, page))
    run(make([3, 64, 66, 300], 3, 24, page, page + 1))


def test_one_long_sequence_is_cut_and_joined():
    for H in (4, 24, 64):
        run(make([4097], 1, H, 64, H))
    run(make([5, 3000, 70, 1], 1, 16, 32, 7))


def test_more_sequences_than_workgroups():
    g = torch.Generator().manual_seed(8)
    lens = torch.randint(1, 90, (700,), generator=g).tolist()
    run(make(lens, 1, 8, 16, 9))


def test_rows_without_keys():
    """No keys at all, fewer keys than new tokens, a negative length, and pages that are not there."""
    kw = make([0, 2, 70, 64], 4, 6, 16, 10)
    run(kw)
    kw["seq_lens"] = torch.tensor([-3, 1, 70, 64], dtype=torch.int32)
    run(kw)
    kw["block_table"][2, 1] = -1              # a hole inside
    kw["block_table"][3, :] = 10 ** 6         # no page at all
    kw["block_table"][1, 0] = -2 ** 31
    o, lse = run(kw)
    assert (o[3] == 0).all() and torch.isinf(lse[3]).all()


def test_lengths_beyond_the_table_are_cut():
    kw = make([64, 40], 1, 16, 16, 11, spare_cols=0)
    want = cdr.latent_decode_fwd(**dev(kw), scale=SCALE)
    kw["seq_lens"] = torch.tensor([2 ** 31 - 1, 40], dtype=torch.int32)
    for a, b in zip(cdr.latent_decode_fwd(**dev(kw), scale=SCALE), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [2, 4, 70])
@pytest.mark.parametrize("H", [4, 16, 40])
def test_new_tokens_beyond_the_table(T, H):
    """New tokens that found no room in the table: those before them see what they would see in a longer
    table whose further pages are not there."""
    kw = make([63, 40, 0, 64], T, H, 16, 10 * T + H, spare_cols=0)
    kw["seq_lens"] = torch.tensor([63 + T, 40 + T, T, 64 + T], dtype=torch.int32)
    kw["cache"][torch.isnan(kw["cache"])] = 0.5      # the tail of a last page is a new token's now
    wider = dict(kw, block_table=torch.cat([kw["block_table"], torch.full((4, 5), -1, dtype=torch.int32)], 1))
    o, lse = cdr.latent_decode_fwd(**dev(kw), scale=SCALE)
    compare(wider, o, lse)
    compare(kw, o, lse)


def test_the_most_keys_a_sequence_can_have():
    """A length of 2^31 - 1 over a table with room for as many: only its first and last page are there, the last
    up to key 2^31 - 256, and both are one page of the cache."""
    page, cols = 2 ** 16, 2 ** 15
    g = torch.Generator().manual_seed(20)
    q = torch.randn(1, 1, 3, 576, generator=g).to(BF16)
    cache = torch.randn(1, page, 576, generator=g).to(BF16)
    table = torch.full((1, cols), -1, dtype=torch.int32)
    table[0, 0] = table[0, -1] = 0
    o, lse = cdr.latent_decode_fwd(q[..., :512].to(DEV), q[..., 512:].to(DEV), cache.to(DEV), table.to(DEV),
                                   torch.tensor([2 ** 31 - 1], dtype=torch.int32, device=DEV), SCALE)
    keys = cache[0].double()
    twice = torch.full((page,), math.log(2.0), dtype=torch.float64)
    twice[-256:] = 0
    s = SCALE * (q[0, 0].double() @ keys.T) + twice
    p = torch.softmax(s, -1)
    size = SCALE * (q[0, 0].double().abs() @ keys.abs().T).amax(-1)
    # as in compare(), the sums taken over the 1024 tiles of a page one after the other, two roundings each
    e = 585 * 2.0 ** -24 * size + (80 + 2 * 1024) * 2.0 ** -24
    lse_ref = torch.logsumexp(s, -1)
    assert ((lse[0, 0].cpu().double() - lse_ref).abs() <= e + 2.0 ** -22 * lse_ref.abs()).all()
    ref, mag = p @ keys[:, :512], p @ keys[:, :512].abs()
    tol = (2.0 ** -8 + 2 * e + 2.0 ** -16)[:, None] * mag + 2.0 ** -8 * ref.abs()
    assert ((o[0, 0].cpu().double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("H", [5, 16, 40])
def test_packed_queries(H):
    packed = [1, 4, 0, 2, 9]
    kw = make([30, 64, 50, 129, 9], 0, H, 16, H, packed=packed)
    total = sum(packed)
    out = torch.full((1, total + 2, H, 512), 7.0, dtype=BF16, device=DEV)
    lse = torch.full((1, total + 2, H), 7.0, device=DEV)
    o, l2 = cdr.latent_decode_fwd(**dev(kw), scale=SCALE, out=out, lse_out=lse)
    assert o is out and l2 is lse
    compare(kw, o, lse)
    assert (out[0, total:] == 7).all() and (lse[0, total:] == 7).all()    # behind the last sequence


@pytest.mark.parametrize("H,spare", [(5, 2), (40, 600)])
def test_rows_that_no_sequence_holds_are_empty(H, spare, monkeypatch):
    """Zeros and -inf in what the binding allocates, whatever memory it gets; supplied buffers keep theirs."""
    packed = [3, 1, 4, 0, 2]
    kw = make([9, 30, 64, 50, 129], 0, H, 16, H, packed=packed)
    wide = lambda t: torch.cat([t, torch.full((1, spare - 2) + t.shape[2:], math.nan, dtype=BF16)], 1)  # noqa: E731
    kw["q_latent"], kw["q_rope"] = wide(kw["q_latent"]), wide(kw["q_rope"])
    for n in ("seq_lens", "block_table", "cu_seqlens"):
        kw[n] = kw[n][1:]                      # the first three rows are nobody's
    empty, d = torch.empty, dev(kw)
    with monkeypatch.context() as m:
        m.setattr(torch, "empty", lambda *s, **k: empty(*s, **k).fill_(77))
        o, lse = cdr.latent_decode_fwd(**d, scale=SCALE)
        out, lse_out = torch.full_like(o, 3), torch.full_like(lse, 3)
        only_lse = cdr.latent_decode_fwd(**d, scale=SCALE, out=out)[1]
        only_o = cdr.latent_decode_fwd(**d, scale=SCALE, lse_out=lse_out)[0]
    compare(kw, o, lse)
    for x, y, z, value in ((o, only_o, out, 0), (lse, only_lse, lse_out, -math.inf)):
        for rows in (slice(0, 3), slice(10, 10 + spare)):
            assert (x[:, rows] == value).all() and (z[:, rows] == 3).all()
        assert torch.equal(x, y) and torch.equal(x[:, 3:10], z[:, 3:10])


def test_strided_queries_and_other_scales():
    kw = make([33, 100], 2, 8, 16, 12)
    g = dev(kw)
    wide = torch.zeros(2, 2, 8, 640, dtype=BF16, device=DEV)
    wide[..., :512], wide[..., 576:] = g["q_latent"], g["q_rope"]
    want = cdr.latent_decode_fwd(**g, scale=SCALE)
    for a, b in zip(cdr.latent_decode_fwd(**dict(g, q_latent=wide[..., :512], q_rope=wide[..., 576:]), scale=SCALE), want):
        assert torch.equal(a, b)
    turned = g["q_latent"].transpose(0, 1).contiguous().transpose(0, 1)
    odd = torch.zeros(2 * 2 * 8 * 64 + 1, dtype=BF16, device=DEV)[1:].view(2, 2, 8, 64)
    odd.copy_(g["q_rope"])
    for a, b in zip(cdr.latent_decode_fwd(**dict(g, q_latent=turned, q_rope=odd), scale=SCALE), want):
        assert torch.equal(a, b)
    run(kw, scale=-0.3)
    run(kw, scale=0.0)


def test_a_cache_beyond_32_bit_offsets():
    """Pages behind 2^31 elements (4.3 GB) of the cache, written and read."""
    kw = make([200, 33], 1, 16, 64, 19, extra_pages=0)
    far = 2 ** 31 // (64 * 576) + 5
    cache = torch.empty(far + kw["cache"].shape[0], 64, 576, dtype=BF16, device=DEV)
    cache[far:] = kw["cache"].to(DEV)
    g = dev(kw)
    table = g["block_table"].clone()
    table[table < 100] += far
    o, lse = cdr.latent_decode_fwd(**dict(g, cache=cache, block_table=table), scale=SCALE)
    compare(kw, o, lse)
    row = torch.randn(1, 576, generator=torch.Generator().manual_seed(1)).to(BF16).to(DEV)
    cdr.latent_cache_write(row[:, :512], row[:, 512:], cache,
                           torch.tensor([far * 64 + 7], dtype=torch.int32, device=DEV))
    assert torch.equal(cache[far, 7], row[0])


def test_strides_of_single_elements_mean_nothing():
    """One head, one token or one sequence, with strides there that no row could have."""
    kw = make([40], 1, 1, 16, 18)
    g = dev(kw)
    want = cdr.latent_decode_fwd(**g, scale=SCALE)
    odd = lambda t: torch.as_strided(t, t.shape, (3, 5, 7, 1))  # noqa: E731
    for a, b in zip(cdr.latent_decode_fwd(**dict(g, q_latent=odd(g["q_latent"]), q_rope=odd(g["q_rope"])), scale=SCALE), want):
        assert torch.equal(a, b)
    cache = torch.zeros(1, 16, 576, dtype=BF16, device=DEV)
    c = torch.as_strided(g["q_latent"].view(512), (1, 512), (3, 1))
    r = torch.as_strided(g["q_rope"].view(64), (1, 64), (5, 1))
    cdr.latent_cache_write(c, r, cache, torch.zeros(1, dtype=torch.int32, device=DEV))
    assert torch.equal(cache[0, 0], torch.cat([c[0], r[0]])) and (cache[0, 1:] == 0).all()


def test_large_scores_and_infinite_neighbours():
    """Scores of hundreds (one key carries all), and infinities in rows that no sequence holds."""
    kw = make([90, 64], 1, 16, 16, 13)
    kw["q_latent"] = (kw["q_latent"].float() * 30).to(BF16)
    kw["cache"][torch.isnan(kw["cache"])] = math.inf
    run(kw)


def test_same_bits_and_graph_replays_with_other_lengths():
    kw = make([500, 3, 64, 300], 1, 16, 16, 14)
    g = dev(kw)
    call = lambda: cdr.latent_decode_fwd(**g, scale=SCALE)  # noqa: E731
    a, b = call(), call()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    for lens in ([500, 3, 64, 300], [1, 2, 3, 4], [499, 0, 10, 65]):
        g["seq_lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        compare(dict(kw, seq_lens=torch.tensor(lens, dtype=torch.int32)), *held)
        for x, y in zip(held, call()):
            assert torch.equal(x, y)


def test_on_another_stream():
    kw = make([120, 7], 1, 16, 16, 15)
    g = dev(kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o, lse = cdr.latent_decode_fwd(**g, scale=SCALE)
    side.synchronize()
    compare(kw, o, lse)


# ------------------------------------------------------------------------------------ cache write

def test_cache_write():
    g = torch.Generator().manual_seed(16)
    for T in (1, 3, 257):
        cache = torch.randn(20, 16, 576, generator=g).to(BF16)
        c, r = torch.randn(T, 512, generator=g).to(BF16), torch.randn(T, 64, generator=g).to(BF16)
        slots = torch.randperm(320, generator=g)[:T].to(torch.int32)
        slots[T // 2] = -1 if T > 1 else slots[0]
        if T > 2:
            slots[0], slots[1] = 320, 2 ** 31 - 1
        want = cache.clone().view(320, 576)
        for t, s in enumerate(slots.tolist()):
            if 0 <= s < 320:
                want[s] = torch.cat([c[t], r[t]])
        got = cache.to(DEV)
        wide = torch.cat([c, r], 1).to(DEV)
        cdr.latent_cache_write(wide[:, :512], wide[:, 512:], got, slots.to(DEV))
        assert torch.equal(got.cpu().view(320, 576), want)


def test_cache_write_from_the_cache_itself():
    """Pages copied to others, as for a request that takes over another's beginning."""
    cache = torch.randn(9, 8, 576, generator=torch.Generator().manual_seed(21)).to(BF16).to(DEV)
    want = cache.clone()
    want[6:9] = cache[1:4]
    want[0, 3] = cache[4, 7]
    cdr.latent_cache_write(cache[1:4, :, :512], cache[1:4, :, 512:], cache,
                           torch.arange(48, 72, dtype=torch.int32, device=DEV))
    cdr.latent_cache_write(cache[4, 7:, :512], cache[4, 7:, 512:], cache, torch.tensor([3], dtype=torch.int32, device=DEV))
    assert torch.equal(cache, want)


def test_a_serving_step():
    """Three decode steps from request lengths: page tables, cache write, attention, all on the GPU,
    against attention over the plain history."""
    g = torch.Generator().manual_seed(17)
    N, H, page = 3, 16, 4
    ctx = [0, 6, 4]
    hist = [torch.randn(n, 576, generator=g).to(BF16) for n in ctx]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    cache = torch.full((40, page, 576), math.nan, dtype=BF16, device=DEV)
    table = torch.full((N, 8), -1, dtype=torch.int32, device=DEV)
    free, head = torch.randperm(40, generator=g).to(torch.int32).to(DEV), i32([0])
    first = cdr.build_page_tables(i32(ctx), i32([0] * N), table, free, head, page, sum(ctx))
    old = torch.cat(hist).to(DEV)
    cdr.latent_cache_write(old[:, :512], old[:, 512:], cache, first.slot_map)
    for step in range(3):
        new = torch.randn(N, 576, generator=g).to(BF16)
        q = torch.randn(N, 1, H, 576, generator=g).to(BF16)
        t = cdr.build_page_tables(i32([1] * N), i32([len(h) for h in hist]), table, free, head, page, N + 2)
        d = torch.cat([new, torch.zeros(2, 576).to(BF16)]).to(DEV)
        cdr.latent_cache_write(d[:, :512], d[:, 512:], cache, t.slot_map)
        qd = q.to(DEV)
        o, lse = cdr.latent_decode_fwd(qd[..., :512], qd[..., 512:], cache, table, t.seq_lens, SCALE)
        hist = [torch.cat([h, new[n:n + 1]]) for n, h in enumerate(hist)]
        plain = torch.full((N, 16, 576), math.nan, dtype=BF16)
        for n, h in enumerate(hist):
            plain[n, :len(h)] = h
        kw = dict(q_latent=q[..., :512], q_rope=q[..., 512:], cache=plain, block_table=torch.arange(N, dtype=torch.int32)[:, None],
                  seq_lens=torch.tensor([len(h) for h in hist], dtype=torch.int32))
        compare(kw, o, lse)
