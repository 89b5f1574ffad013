"""attn_sink_page_map: the argument checks on the CPU, every entry against the oracle's request-by-request
tables on the GPU."""
import numpy as np
import pytest
import torch

import gqa_softmax_attention_attn_b200 as attn
import oracle

INVALID, MISALIGNED = -1, -3
gpu = pytest.mark.gpu


def fake(n):
    return [0x7f0000000000 + 0x1000 * i for i in range(n)]


def test_host_checks():
    lib = attn.load()
    c, n, par, free, tab, sl, cu, pos, rows, st = fake(10)

    def call(c_=c, n_=n, par_=par, free_=free, tab_=tab, sl_=sl, cu_=cu, B=4, total=32, width=64, ps=16, pages=512,
             n_free=10, st_=st):
        return lib.attn_sink_page_map(c_, n_, par_, free_, tab_, sl_, cu_, pos, rows, st_, B, total, width, ps, pages,
                                      n_free, None)

    for bad in (dict(c_=None), dict(n_=None), dict(tab_=None), dict(sl_=None), dict(cu_=None), dict(st_=None),
                dict(free_=None), dict(B=0), dict(total=0), dict(width=0), dict(ps=0), dict(ps=24), dict(pages=0),
                dict(n_free=-1), dict(pages=1 << 28), dict(width=1 << 28), dict(B=1 << 20, width=1 << 12),
                dict(sl_=c), dict(cu_=n), dict(tab_=free), dict(st_=par)):
        assert call(**bad) == INVALID, bad
    assert call(par_=par + 4) == MISALIGNED
    assert call(sl_=sl + 4) == MISALIGNED


def test_oracle_map_by_hand():
    """Three requests over pages of 4 slots, one tree, one free page short."""
    table, lens, cu, pos, rows, stats = oracle.page_map([3, 0, 8], [3, 2, 0], [9, 5], [[1, -1, 7], [6, -1, -1], [2, 3, 0]],
                                                        7, 4, 10, parents=[-1, 0, 0, -1, -1, 0, 0])
    assert table.tolist() == [[1, 9, 7], [5, -1, -1], [2, 3, 0]]
    assert lens == [6, 2, 8] and cu == [0, 3, 5, 5] and stats == [5, 2, 0, 0]
    assert pos.tolist() == [3, 4, 4, 0, 0, 0, 0]
    assert rows.tolist() == [7, 36, 37, 20, 21, -1, -1]
    short = oracle.page_map([3, 0], [3, 2], [9], [[1, -1, 7], [6, -1, -1]], 5, 4, 10)
    assert short[0].tolist() == [[1, 9, 7], [-1, -1, -1]] and short[4].tolist() == [7, 36, 37, -1, -1]
    assert short[5] == [5, 2, 1, 0]


def run(cached, new, free, table, total, ps, pages, parents=None):
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    tab = i32(table)
    B = len(cached)
    outs = [torch.full((n,), -77, dtype=torch.int32, device="cuda") for n in (B, B + 1, total, total, 4)]
    attn.attn_sink_page_map(i32(cached), i32(new), i32(free) if free else None, tab, *outs, ps, pages,
                            parents=None if parents is None else i32(parents))
    torch.cuda.synchronize()
    return [tab.cpu().numpy()] + [o.cpu().numpy() for o in outs]


def check(cached, new, free, table, total, ps, pages, parents=None):
    got = run(cached, new, free, table, total, ps, pages, parents)
    ref = oracle.page_map(cached, new, free, table, total, ps, pages, parents)
    for name, g, r in zip(("page_table", "seqlens", "cu_seqlens", "positions", "kv_rows", "stats"), got, ref):
        assert np.array_equal(g, np.asarray(r)), name


def problem(B, cmax, nmax, ps, seed, zero=0.2, spare=8):
    g = np.random.default_rng(seed)
    cached, new = g.integers(0, cmax + 1, B), g.integers(0, nmax + 1, B)
    new[g.random(B) < zero] = 0
    cached[g.random(B) < zero] = 0
    have, need = -(-cached // ps), -(-(cached + new) // ps)
    width = max(int(need.max()), 1) + 1
    pages = int(need.sum()) + spare
    perm = g.permutation(pages)
    table = g.integers(-5, 2 * pages, (B, width))  # entries past a request's pages hold anything
    at = 0
    for b in range(B):
        table[b, :have[b]] = perm[at:at + have[b]]
        at += have[b]
    parents = [int(g.integers(-2, max(i, 1) + 1)) for n in new for i in range(n)]
    return cached.tolist(), new.tolist(), perm[at:].tolist(), table.tolist(), pages, parents


@gpu
@pytest.mark.parametrize("ps", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("B,nmax", [(1, 1), (1, 700), (3, 300), (64, 8), (1023, 3), (1025, 40), (5000, 2)])
def test_requests(B, nmax, ps):
    """One request to several scanned chunks of them, trees and chains (also past the tree limit), padding."""
    cached, new, free, table, pages, parents = problem(B, 900, nmax, ps, B + nmax)
    total = sum(new)
    for pad in (0, 1, 300):
        if total + pad:
            check(cached, new, free, table, total + pad, ps, pages)
            check(cached, new, free, table, total + pad, ps, pages, parents + [0] * pad)


@gpu
def test_a_chain_of_parents_is_no_parents():
    cached, new = [5, 0, 77], [256, 255, 3]
    parents = [i - 1 for n in new for i in range(n)]
    free, table = list(range(40)), [[50 + i for i in range(30)] for _ in range(3)]
    a = run(cached, new, free, table, sum(new), 16, 100, parents)
    b = run(cached, new, free, table, sum(new), 16, 100)
    for x, y in zip(a, b):
        assert np.array_equal(x, y)


@gpu
def test_shortages_and_bad_lengths():
    """Too few free pages, none at all, free pages outside the pool, tables too narrow, negative lengths,
    more tokens than rows, and lengths near 2^31."""
    check([10, 3, 30], [40, 20, 1], [7, 3], [[1, 2, 0, 0], [4, 0, 0, 0], [5, 6, 0, 0]], 61, 16, 9)
    check([10, 3, 30], [40, 20, 1], [], [[1, 2, 0, 0], [4, 0, 0, 0], [5, 6, 0, 0]], 61, 16, 9)
    check([10, 3, 30], [40, 20, 1], [99, -4, 8, 3], [[1, 2, 0, 0], [4, 0, 0, 0], [5, -6, 0, 0]], 61, 16, 9)
    check([10, 100, 0], [40, 20, 33], list(range(20)), [[1, 2], [4, 5], [6, 7]], 93, 16, 60)
    check([-5, 4, 0], [3, -2, 2], [1, 2, 3], [[0, 9], [8, 9], [7, 9]], 9, 8, 10)
    check([4, 4, 4], [30, 30, 30], list(range(10)), [[0] * 8] * 3, 50, 8, 70)
    # two requests of 2^31 - 1 cached tokens in a table of four pages
    got = run([2 ** 31 - 1, 2 ** 31 - 1], [2, 0], [1, 2], [[0] * 4] * 2, 2, 8, 10)
    assert got[1].tolist() == [2 ** 31 - 1] * 2 and got[4].tolist() == [-1, -1] and got[5].tolist() == [2, 0, 0, 2]
    got = run([0, 0, 0], [2 ** 31 - 1] * 3, [1, 2], [[0] * 4] * 3, 2, 8, 10)
    assert got[2].tolist() == [0, 2, 2, 2] and got[5].tolist() == [2 ** 31 - 1, 12, 10, 3]


@gpu
def test_captured_with_room_for_more():
    """A graph captured for 40 tokens replayed for other requests; the rows it does not need are empty."""
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    cached, new, free = i32([5, 0]), i32([4, 9]), i32(list(range(10, 30)))
    tab = i32([[0, 1, 2, 3, 4, 5]] * 2)
    outs = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (2, 3, 40, 40, 4)]
    call = lambda: attn.attn_sink_page_map(cached, new, free, tab, *outs, 8, 64)
    call()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        call()
    for c, n in (([5, 0], [4, 9]), ([13, 2], [0, 30]), ([0, 0], [0, 0])):
        start = [[0, 1, 2, 3, 4, 5], [6, 7, 8, 9, 8, 7]]
        cached.copy_(i32(c))
        new.copy_(i32(n))
        tab.copy_(i32(start))
        gr.replay()
        torch.cuda.synchronize()
        ref = oracle.page_map(c, n, list(range(10, 30)), start, 40, 8, 64)
        for g, r in zip([tab] + outs, ref):
            assert np.array_equal(g.cpu().numpy(), np.asarray(r))
