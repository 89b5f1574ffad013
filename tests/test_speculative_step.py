"""One verification step of a speculative decoder, as a server would run it: page map -> prologue with q/k
norms, appending to the paged cache -> attention of the drafted trees, twice in a row and from a captured
graph, against the same chain of the oracle."""
import numpy as np
import pytest
import torch

import gqa_softmax_attention_attn_b200 as attn
import oracle
from _harness import assert_close_bf16, assert_lse
from test_qk_norm import EPS, YARN, oracle_rope
from test_tree_decode import make_tree

pytestmark = pytest.mark.gpu
D, Hq, Hkv, PS = 64, 16, 2, 16
CAP = 40  # rows the step is captured for


class Server:
    """Device buffers of a small server: a page pool, its free list and a step's tables."""

    def __init__(self, B, pages, width, seed):
        g = torch.Generator().manual_seed(seed)
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
        bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
        self.B, self.pages = B, pages
        self.cached, self.new, self.parents = i32(B), i32(B), i32(CAP)
        self.free_host = torch.randperm(pages, generator=g).int()
        self.free = self.free_host.cuda()
        self.table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        self.lens, self.cu, self.pos, self.rows, self.stats = i32(B), i32(B + 1), i32(CAP), i32(CAP), i32(4)
        self.qkv, self.q, self.out = bf(CAP, (Hq + 2 * Hkv) * D), bf(CAP, Hq, D), bf(CAP, Hq, D)
        self.lse = torch.zeros(CAP, Hq, device="cuda")
        self.k, self.v = (torch.full((pages, PS, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda")
                          for _ in range(2))
        self.bias = (torch.randn((Hq + 2 * Hkv) * D, generator=g) * 0.1).cuda()
        self.qw, self.kw = (1 + 0.2 * torch.randn(D, generator=g)).cuda(), (1 + 0.2 * torch.randn(D, generator=g)).cuda()
        self.sinks = torch.randn(Hq, generator=g).cuda()
        self.ws = torch.empty(max(16, attn.attn_sink_decode_tree_workspace_size(
            B, CAP, CAP, Hq, Hkv, D, width * PS, 0, 0, attn.DTYPE_BF16)), dtype=torch.uint8, device="cuda")

    def step(self, window):
        attn.attn_sink_page_map(self.cached, self.new, self.free, self.table, self.lens, self.cu, self.pos, self.rows,
                                self.stats, PS, self.pages, parents=self.parents)
        attn.attn_sink_qk_norm_prologue(self.qkv, self.bias, self.qw, self.kw, self.pos, self.q,
                                        self.k.view(-1, Hkv, D), self.v.view(-1, Hkv, D), EPS, kv_rows=self.rows, **YARN)
        attn.attn_sink_decode_tree_paged(self.q, self.k, self.v, self.table, self.cu, self.parents, self.lens,
                                         self.sinks, self.out, self.lse, CAP, window, 0.125, 0, self.ws)


@pytest.mark.parametrize("window", [0, 24])
def test_steps_of_a_server(window):
    """A prompt of every request (a chain), then a step of drafted trees of which a part of one path is kept
    (its keys moved to the front, as a server does), then another, replayed from a graph of the first."""
    B = 3
    s = Server(B, 40, 8, 5)
    ref_k = [np.zeros((0, Hkv, D)) for _ in range(B)]
    ref_v = [np.zeros((0, Hkv, D)) for _ in range(B)]
    g = torch.Generator().manual_seed(9)
    graph = None
    used = 0
    for new in ([15, 0, 9], [7, 12, 1], [0, 16, 10]):
        trees = [make_tree(n, "random" if used else "chain", g) for n in new]
        cached = [len(k) for k in ref_k]
        qkv = (torch.randn(CAP, (Hq + 2 * Hkv) * D, generator=g)).bfloat16()
        s.cached.copy_(torch.tensor(cached))
        s.new.copy_(torch.tensor(new))
        flat = sum(trees, [])
        s.parents.copy_(torch.tensor(flat + [-1] * (CAP - len(flat))))
        s.qkv.copy_(qkv)
        s.free.copy_(torch.roll(s.free_host, -used))  # the pages taken so far are gone from the front
        if graph is None:
            s.step(window)  # (the first call on a device sets itself up)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                s.step(window)
        graph.replay()
        torch.cuda.synchronize()
        used += int(s.stats[1])
        assert s.stats[0] == sum(new) and s.stats[2:].tolist() == [0, 0]

        # the oracle's chain; its keys and values are bf16, as the cache is
        pos = [cached[b] + d for b, t in enumerate(trees) for d in oracle.tree_depths(t)]
        assert s.pos.tolist() == pos + [0] * (CAP - len(pos))
        n = len(pos)
        q, k, v = oracle.qk_norm_prologue(qkv[:n], s.bias, s.qw, s.kw, np.array(pos), Hq, Hkv, D, EPS,
                                          **oracle_rope(YARN))
        bf = lambda x: torch.from_numpy(x).bfloat16().double().numpy()
        q, k, v = bf(q), bf(k), bf(v)
        cu = np.concatenate([[0], np.cumsum(new)])
        for b in range(B):
            ref_k[b] = np.concatenate([ref_k[b], k[cu[b]:cu[b + 1]]])
            ref_v[b] = np.concatenate([ref_v[b], v[cu[b]:cu[b + 1]]])
        L = max(len(x) for x in ref_k)
        pad = lambda xs: np.stack([np.concatenate([x, np.zeros((L - len(x), Hkv, D))]) for x in xs])
        ro, rl = oracle.decode_tree(q, pad(ref_k), pad(ref_v), cu, np.array(flat), np.array([len(x) for x in ref_k]),
                                    s.sinks, window, 0.125)
        # (a bf16 rounding of q or k that falls the other way moves a score of size S by 2^-8 S: the framework's
        # bf16 bounds, as for the prologue chained into the forward)
        assert_close_bf16(s.out[:n], ro, f"out, new={new}")
        assert_lse(s.lse[:n], rl, f"lse, new={new}")
        # keep the path of each tree's last token
        for b, t in enumerate(trees):
            path, a = [], len(t) - 1
            while a >= 0:
                path.append(a)
                a = t[a]
            path = path[::-1]
            rows = s.table[b].long().repeat_interleave(PS) * PS + torch.arange(PS, device="cuda").repeat(s.table.shape[1])
            for pool in (s.k.view(-1, Hkv, D), s.v.view(-1, Hkv, D)):
                pool[rows[cached[b]:cached[b] + len(path)]] = pool[rows[[cached[b] + a for a in path]]]
            for ref in (ref_k, ref_v):
                ref[b] = np.concatenate([ref[b][:cached[b]], ref[b][cached[b]:][path]])
    assert attn.attn_sink_get_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_calls_in_line(dtype):
    """Every call's kernels may start while the grid ahead still runs: a line of calls that each read what the
    one before wrote, and write what it read, gives the bits of the same calls with a synchronisation after each,
    run eagerly and from a captured graph."""
    B, T, pages, width = 4, 10, 80, 20
    n = B * T
    g = torch.Generator().manual_seed(31)
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32).cuda()
    dev = dict(device="cuda")
    qkv0 = torch.randn(n, (Hq + 2 * Hkv) * D, generator=g).bfloat16().cuda()
    pool0 = torch.randn(2, pages, PS, Hkv, D, generator=g).to(dtype).cuda()
    bias = (torch.randn((Hq + 2 * Hkv) * D, generator=g) * 0.1).cuda()
    qw, kw = (1 + 0.2 * torch.randn(D, generator=g)).cuda(), (1 + 0.2 * torch.randn(D, generator=g)).cuda()
    sinks = torch.randn(Hq, generator=g).cuda()
    parents = i32(sum((make_tree(T, "random", g) for _ in range(B)), []))
    free = i32(torch.randperm(pages, generator=g))
    ws = torch.empty(max(16, attn.attn_sink_decode_tree_workspace_size(
        B, n, T, Hq, Hkv, D, width * PS, 0, 0, attn.DTYPE_BF16 if dtype == torch.bfloat16 else attn.DTYPE_F32)),
        dtype=torch.uint8, **dev)
    ws_bwd = torch.empty(attn.attn_sink_qk_norm_prologue_bwd_workspace_size(n, Hq, Hkv, D), dtype=torch.uint8, **dev)
    cached, new = i32([250, 0, 17, 100]), i32([T] * B)

    class State:
        pass

    def fresh():
        s = State()
        s.qkv, s.table = qkv0.clone(), torch.full((B, width), -1, dtype=torch.int32, **dev)
        have = [(c + PS - 1) // PS for c in cached.tolist()]
        for b in range(B):  # pages already held: the last ones of the list
            s.table[b, :have[b]] = free[pages - sum(have[:b + 1]):pages - sum(have[:b])]
        s.k, s.v = pool0[0].clone(), pool0[1].clone()
        s.kt, s.vt = (torch.empty(n, Hkv, D, dtype=torch.bfloat16, **dev) for _ in range(2))
        s.lens, s.cu, s.pos, s.rows, s.stats = (torch.zeros(x, dtype=torch.int32, **dev) for x in (B, B + 1, n, n, 4))
        s.q = torch.empty(n, Hq, D, dtype=torch.bfloat16, **dev)
        s.out, s.lse = torch.empty(n, Hq, D, dtype=dtype, **dev), torch.empty(n, Hq, **dev)
        s.dqkv, s.dbias = torch.empty_like(s.qkv), torch.empty_like(bias)
        s.dqw, s.dkw = torch.empty_like(qw), torch.empty_like(kw)
        return s

    def line(s, after=lambda: None):
        x, y = s.qkv, s.dqkv
        for _ in range(4):
            attn.attn_sink_page_map(cached, new, free, s.table, s.lens, s.cu, s.pos, s.rows, s.stats, PS, pages,
                                    parents=parents)
            after()
            if dtype == torch.bfloat16:
                attn.attn_sink_qk_norm_prologue(x, bias, qw, kw, s.pos, s.q, s.k.view(-1, Hkv, D),
                                                s.v.view(-1, Hkv, D), EPS, kv_rows=s.rows, **YARN)
                after()
            attn.attn_sink_qk_norm_prologue(x, bias, qw, kw, s.pos, s.q, s.kt, s.vt, EPS, **YARN)
            after()
            a, b = s.q if dtype == torch.bfloat16 else s.q.float(), s.out
            for _ in range(3):  # each on the output of the one before
                attn.attn_sink_decode_tree_paged(a, s.k, s.v, s.table, s.cu, parents, s.lens, sinks, b, s.lse, T, 0,
                                                 0.125, 0, ws)
                after()
                a, b = b, a
            attn.attn_sink_qk_norm_prologue_bwd(x, bias, qw, kw, s.pos, s.q, s.kt, s.vt, y, s.dbias, s.dqw, s.dkw, EPS,
                                                workspace=ws_bwd, **YARN)
            after()
            x, y = y, x
        return x, s.out, s.lse, s.k, s.v, s.dbias, s.dqw, s.dkw, s.pos, s.rows, s.table

    want = [t.clone() for t in line(fresh(), torch.cuda.synchronize)]
    assert all(bool(torch.isfinite(t.float()).all()) for t in want)
    for _ in range(3):
        for a, b in zip(line(fresh()), want):
            assert torch.equal(a, b)
    s = fresh()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = line(s)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert attn.attn_sink_get_device_status() == 0
