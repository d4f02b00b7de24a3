"""The serving step's bookkeeping on the GPU against the integer oracle: equal everywhere."""
import random

import pytest
import torch

import chunked_gated_delta_chunk_amd as cdr
from oracle.pages import build_page_tables

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def run(q, c, table, free, head, page, cap, **kw):
    want = build_page_tables(q, c, table, free, head, page, cap)
    t, h = i32(table), i32([head])
    got = cdr.build_page_tables(i32(q), i32(c), t, i32(free) if free else torch.empty(0, dtype=torch.int32, device=DEV),
                                h, page, cap, **kw)
    assert got.cu_seqlens.tolist() == want["cu_seqlens"]
    assert got.seq_lens.tolist() == want["seq_lens"]
    assert got.positions.tolist() == want["positions"]
    assert got.slot_map.tolist() == want["slot_map"]
    assert t.tolist() == want["block_table"]
    assert got.free_head.tolist() == [want["free_head"]]
    assert got.shortage.tolist() == [want["shortage"]]
    return got, h


def draw(rng, n, page, ctx, new, cols, spare=0, short=0):
    c = [rng.randint(0, ctx) for _ in range(n)]
    q = [rng.randint(0, new) for _ in range(n)]
    held = [min(-(-x // page), cols) for x in c]
    pages = list(range(sum(held) + sum(-(-x // page) + 1 for x in q)))
    rng.shuffle(pages)
    table, at = [], 0
    for k in held:
        table.append(pages[at:at + k] + [rng.choice([-1, 123456]) for _ in range(cols - k)])
        at += k
    free = pages[at:len(pages) - short]
    return q, c, table, [99] * 2 + free, 2, page, sum(q) + spare


@pytest.mark.parametrize("n,page,ctx,new,cols", [
    (1, 1, 0, 1, 1), (1, 16, 100, 1, 7), (3, 64, 0, 200, 4), (5, 3, 50, 20, 30), (64, 16, 300, 1, 20),
    (257, 64, 500, 1, 9), (1025, 16, 40, 3, 4), (2500, 5, 20, 4, 6), (5000, 8, 30, 2, 5), (70, 16, 200, 300, 40)])
def test_lengths(n, page, ctx, new, cols):
    rng = random.Random(n * 1000 + page)
    for spare in (0, 13):
        run(*draw(rng, n, page, ctx, new, cols, spare=spare))


def test_one_token_each_and_none():
    run([1] * 8, [0, 1, 15, 16, 17, 31, 32, 33], [[i, 10 + i, 20 + i] for i in range(8)], list(range(40, 60)), 3, 16, 8)
    run([0, 0], [0, 5], [[-1], [3]], [], 0, 16, 0)
    run([0, 0], [0, 5], [[-1], [3]], [8], 0, 16, 5)


def test_shortage_full_rows_and_cut():
    rng = random.Random(3)
    run(*draw(rng, 40, 4, 20, 9, 6, short=15))                   # the free list ends early, rows too short
    q, c, table, free, head, page, cap = draw(rng, 40, 4, 20, 9, 8)
    run(q, c, table, free, head, page, cap // 2)                 # fewer tokens than asked for
    run(q, c, table, free, len(free) + 7, page, cap)             # a head behind the list
    run(q, c, table, free, -4, page, cap)


def test_negative_and_huge_values_stay_in_bounds():
    top = 2 ** 31 - 1
    run([-5, 3, 2], [4, -9, top - 1], [[1, 2], [-1, -1], [3, -7]], [4, 5, 6], 0, 4, 6)
    run([2], [10], [[-3, -3, -3, -3]], [top // 2, top], 0, 4, 4)  # slots beyond int32 are no slots


def test_many_tokens_take_the_second_kernel():
    rng = random.Random(4)
    run(*draw(rng, 9, 16, 1000, 2000, 200, spare=1000))
    run(*draw(rng, 4200, 16, 30, 4, 3, spare=5))


def test_head_in_place_and_apart_and_reused_outputs():
    args = draw(random.Random(5), 6, 8, 30, 12, 8, spare=3)
    got, head = run(*args)
    assert got.free_head.data_ptr() == head.data_ptr()
    other = i32([0])
    got2, head = run(*args, free_head_out=other)
    assert head.tolist() == [2] and got2.free_head is other
    got3, _ = run(*args, out=got2)
    assert got3.slot_map is got2.slot_map


def test_outputs_over_inputs_are_refused():
    """The natural next step, with the last step's lengths as context and its tensors as outputs."""
    n = 3
    table, free, head = i32([[-1] * 4] * n), i32(list(range(9))), i32([0])
    first = cdr.build_page_tables(i32([2] * n), i32([0] * n), table, free, head, 4, 6)
    with pytest.raises(ValueError, match="overlaps"):
        cdr.build_page_tables(i32([2] * n), first.seq_lens, table, free, head, 4, 6, out=first)
    again = cdr.build_page_tables(i32([2] * n), first.seq_lens, table, free, head, 4, 6)
    assert again.seq_lens.tolist() == [4] * n and again.positions.tolist() == [2, 3] * n


def test_graph_replays_advance_the_step():
    """A captured decode step: lengths grow by one and pages come from the list, replay after replay."""
    n, page, cols, cap = 5, 4, 6, 8
    ctx = [0, 3, 4, 7, 8]
    free = list(range(50, 90))
    table = [[10 * i + j for j in range(-(-c // page))] + [-1] * (cols + (-c // page)) for i, c in enumerate(ctx)]
    q, c, t, f, h = i32([1] * n), i32(ctx), i32(table), i32(free), i32([0])
    warm = cdr.build_page_tables(q, c, t.clone(), f, h.clone(), page, cap)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = cdr.build_page_tables(q, c, t, f, h, page, cap)
        c.add_(1)
    del warm
    head = 0
    for _ in range(5):
        want = build_page_tables([1] * n, ctx, table, free, head, page, cap)
        graph.replay()
        torch.cuda.synchronize()
        assert got.slot_map.tolist() == want["slot_map"] and got.positions.tolist() == want["positions"]
        assert t.tolist() == want["block_table"] and h.tolist() == [want["free_head"]]
        ctx, table, head = [x + 1 for x in ctx], want["block_table"], want["free_head"]
        cdr.build_page_tables(i32([3]), i32([2]), i32([[1, 2]]), f, i32([0]), page, 4)   # eager work in between
