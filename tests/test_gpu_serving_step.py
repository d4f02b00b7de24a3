"""What build_page_tables writes, passed on to the operators that take it: packed latent decode and prefill in steps
padded to a captured size, and the chunked and per-token delta rule in steps that are not.  The latent operators are
compared as in test_gpu_latent_decode.py and test_gpu_latent_attn.py, whose tolerances hold."""
import math

import pytest
import torch

import chunked_gated_delta_chunk_amd as cdr
import test_gpu_latent_attn as attn
import test_gpu_latent_decode as decode

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16
H, PAGE, POOL, COLS = 16, 4, 60, 12


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Service:
    """Requests with their history on the host, and the device's cache, page table and free list."""

    def __init__(self, N, cap, seed):
        self.g = torch.Generator().manual_seed(seed)
        self.N, self.cap = N, cap
        self.hist = [torch.zeros(0, 576, dtype=BF16) for _ in range(N)]
        self.cache = torch.full((POOL, PAGE, 576), math.nan, dtype=BF16, device=DEV)
        self.table = torch.full((N, COLS), -1, dtype=torch.int32, device=DEV)
        self.free, self.head = torch.randperm(POOL, generator=self.g).to(torch.int32).to(DEV), i32([0])
        self.query, self.context = i32([0] * N), i32([0] * N)
        self.c = torch.zeros(cap, 576, dtype=BF16, device=DEV)
        self.q = torch.zeros(1, cap, H, 576, dtype=BF16, device=DEV)

    def feed(self, new):
        """The next step's inputs; rows behind its tokens hold NaN."""
        r = lambda *s: torch.randn(*s, generator=self.g).to(BF16)  # noqa: E731
        rows, q = r(sum(new), 576), r(sum(new), H, 576)
        self.query.copy_(torch.tensor(new, dtype=torch.int32))
        self.context.copy_(torch.tensor([len(h) for h in self.hist], dtype=torch.int32))
        self.c.fill_(math.nan)
        self.q.fill_(math.nan)
        self.c[:sum(new)], self.q[0, :sum(new)] = rows.to(DEV), q.to(DEV)
        self.hist = [torch.cat([h, x]) for h, x in zip(self.hist, rows.split(new))]
        return q

    def step(self):
        t = cdr.build_page_tables(self.query, self.context, self.table, self.free, self.head, PAGE, self.cap)
        cdr.latent_cache_write(self.c[:, :512], self.c[:, 512:], self.cache, t.slot_map)
        o, lse = cdr.latent_decode_fwd(self.q[..., :512], self.q[..., 512:], self.cache, self.table, t.seq_lens,
                                       decode.SCALE, cu_seqlens=t.cu_seqlens)
        return t, o, lse

    def check(self, new, q, t, o, lse):
        total = sum(new)
        assert t.cu_seqlens.tolist() == torch.tensor([0] + new).cumsum(0).tolist() and t.shortage.tolist() == [0]
        plain = torch.full((self.N, COLS * PAGE, 576), math.nan, dtype=BF16)
        for n, h in enumerate(self.hist):
            plain[n, :len(h)] = h
        wide = torch.zeros(1, self.cap, H, 576, dtype=BF16)
        wide[0, :total] = q
        kw = dict(q_latent=wide[..., :512], q_rope=wide[..., 512:], cache=plain.view(self.N * COLS * PAGE, 1, 576),
                  block_table=torch.arange(self.N * COLS * PAGE, dtype=torch.int32).view(self.N, -1),
                  seq_lens=torch.tensor([len(h) for h in self.hist], dtype=torch.int32), cu_seqlens=t.cu_seqlens.cpu())
        decode.compare(kw, o, lse)
        assert (o[:, total:] == 0).all() and (lse[:, total:] == -math.inf).all()


STEPS = [[5, 0, 9, 3], [1, 1, 1, 1], [2, 7, 0, 1], [0, 0, 0, 0], [1, 4, 4, 4]]


def test_padded_packed_steps():
    s = Service(4, 20, 1)
    for new in STEPS:
        q = s.feed(new)
        s.check(new, q, *s.step())


def test_a_captured_padded_step():
    """The whole step in one graph, replayed with other lengths; the eager step of a twin in between."""
    s, twin = Service(4, 20, 2), Service(4, 20, 2)
    twin.feed([0, 0, 0, 0])
    twin.step()                       # loads the kernels; takes no page
    s.feed([0, 0, 0, 0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = s.step()
    for new in STEPS:
        q = s.feed(new)
        twin.feed(new)
        graph.replay()
        torch.cuda.synchronize()
        s.check(new, q, *held)
        t, o, lse = twin.step()
        assert torch.equal(o, held[1]) and torch.equal(lse, held[2]) and torch.equal(t.slot_map, held[0].slot_map)


def test_padded_prefill_in_the_expanded_form():
    """Chunked prefill: the step's offsets for the queries, those of seq_lens for the keys, and spare tokens."""
    new, ctx, spare = [70, 0, 130, 5], [30, 0, 64, 0], 9
    t = cdr.build_page_tables(i32(new), i32(ctx), torch.full((4, 20), -1, dtype=torch.int32, device=DEV),
                              torch.arange(80, dtype=torch.int32, device=DEV), i32([0]), 16, sum(new) + spare)
    kw, do = attn.make(new, [a + b for a, b in zip(new, ctx)], 2, 3, spare=spare)
    cu_k = torch.cat([torch.zeros_like(t.seq_lens[:1]), t.seq_lens.cumsum(0).to(torch.int32)])
    d = dict(attn.dev(kw), cu_seqlens=t.cu_seqlens, cu_seqlens_k=cu_k)
    assert torch.equal(t.cu_seqlens.cpu(), kw["cu_seqlens"]) and torch.equal(cu_k.cpu(), kw["cu_seqlens_k"])
    o, lse = cdr.latent_attn_fwd(**d)
    grads = cdr.latent_attn_bwd(**d, o=o, lse=lse, do=do.to(DEV))
    attn.compare(kw, do, o, lse, grads, 192 ** -0.5)
    assert all((x[:, -spare:] == 0).all() for x in (o,) + grads)


def test_the_delta_rule_takes_the_offsets_of_a_step_without_spare_tokens():
    from chunked_gated_delta_chunk_amd.synth import make_inputs
    import oracle
    new = [100, 0, 64, 30]
    T = sum(new)
    tables = lambda cap: cdr.build_page_tables(i32(new), i32([0] * 4), torch.full((4, 20), -1, dtype=torch.int32, device=DEV),  # noqa: E731
                                               torch.arange(80, dtype=torch.int32, device=DEV), i32([0]), 16, cap)
    cu = tables(T).cu_seqlens
    assert cdr.check_cu_seqlens(cu, T) == 0
    assert cdr.check_cu_seqlens(tables(T + 5).cu_seqlens, T + 5) == len(new) + 1     # a padded step's are refused there
    inp = make_inputs(1, T, 2, seed=4)
    d = inp.to(DEV)
    # bounds as in test_gpu_parity.py
    o_ref, S_ref = oracle.recurrent_fwd(inp.q, inp.k, inp.v, inp.g, inp.beta, cu_seqlens=cu.cpu())
    for fwd in (cdr.chunk_dr_fwd, cdr.fused_recurrent_fwd):
        o, S = fwd(d.q, d.k, d.v, d.g, d.beta, cu_seqlens=cu, output_final_state=True)
        assert (abs(o.float().cpu().numpy() - o_ref) <= 1e-2 + 1e-2 * abs(o_ref)).all()
        assert (abs(S.cpu().numpy() - S_ref) <= 1e-3 + 1e-3 * abs(S_ref)).all()
