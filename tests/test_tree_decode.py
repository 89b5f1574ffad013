"""attn_sink_decode_tree and its paged form: the oracle's pins and the argument checks on the CPU, parity
with the fp64 oracle on the GPU."""
import itertools
import math

import numpy as np
import pytest
import torch

import gqa_softmax_attention_attn_b200 as attn
import oracle
from gqa_softmax_attention_attn_b200 import _native

D = 64
OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, -1, -2, -3, -5
gpu = pytest.mark.gpu


def make_tree(n, kind, g):
    if kind == "chain":
        return list(range(-1, n - 1))
    if kind == "star":  # one root, everything else its child
        return [-1] + [0] * (n - 1)
    if kind == "roots":
        return [-1] * n
    return [-1 if i == 0 or torch.rand((), generator=g) < 0.05 else int(torch.randint(max(0, i - 6), i, (), generator=g))
            for i in range(n)]


def make_case(lens_cached, ns, Hq, Hkv, dtype, kind="random", seed=0, pad_rows=0, std=1.0):
    """A contiguous problem whose cache rows behind each sequence are NaN."""
    g = torch.Generator().manual_seed(seed)
    B, total = len(ns), sum(ns) + pad_rows
    lens = [c + n for c, n in zip(lens_cached, ns)]
    Lmax = max(max(lens), 1)
    q = (torch.randn(total, Hq, D, generator=g) * std).to(dtype)
    k = (torch.randn(B, Lmax, Hkv, D, generator=g) * std).to(dtype)
    v = torch.randn(B, Lmax, Hkv, D, generator=g).to(dtype)
    for b, n in enumerate(lens):
        k[b, n:] = float("nan")
        v[b, n:] = float("nan")
    cu = torch.tensor([0] + list(itertools.accumulate(ns)), dtype=torch.int32)
    parents = torch.tensor(sum((make_tree(n, kind, g) for n in ns), []) + [7] * pad_rows, dtype=torch.int32)
    return dict(q=q, k=k, v=v, cu=cu, parents=parents, lens=torch.tensor(lens, dtype=torch.int32),
                sinks=torch.randn(Hq, generator=g), max_q=max(ns), total=sum(ns))


def paginate(c, page_size, seed=1):
    """The case's caches as pages in random order; unused pages NaN, unused table entries out of the pool."""
    g = torch.Generator().manual_seed(seed)
    B, Lmax, Hkv, _ = c["k"].shape
    lens = c["lens"].tolist()
    per = [-(-n // page_size) for n in lens]
    pages = sum(per) + 3
    perm = torch.randperm(pages, generator=g)
    kp = torch.full((pages, page_size, Hkv, D), float("nan"), dtype=c["k"].dtype)
    vp = kp.clone()
    table = torch.tensor([1 << 30, -1, -7, pages], dtype=torch.int32).repeat(B, -(-max(max(per), 1) // 4)).contiguous()
    at = 0
    for b, n in enumerate(per):
        for e in range(n):
            ph = int(perm[at])
            at += 1
            table[b, e] = ph
            m = min(lens[b], (e + 1) * page_size) - e * page_size
            kp[ph, :m] = c["k"][b, e * page_size:e * page_size + m]
            vp[ph, :m] = c["v"][b, e * page_size:e * page_size + m]
    return kp, vp, table


def run(c, window, page_size=0, num_splits=0, scale=0.125, pages=None):
    dev = "cuda"
    q = c["q"].to(dev)
    Hq, Hkv = q.shape[1], c["k"].shape[2]
    B, dt = len(c["lens"]), _native._dtype_code(c["q"])
    out = torch.full_like(q, 3.0)
    lse = torch.full((q.shape[0], Hq), 3.0, device=dev)
    cu, par, lens, sinks = (c[x].to(dev) for x in ("cu", "parents", "lens", "sinks"))
    if page_size:
        kp, vp, table = (x.to(dev) for x in (pages or paginate(c, page_size)))
        Lmax = table.shape[1] * page_size
    else:
        kc, vc = c["k"].to(dev), c["v"].to(dev)
        Lmax = kc.shape[1]
    n = attn.attn_sink_decode_tree_workspace_size(B, q.shape[0], c["max_q"], Hq, Hkv, D, Lmax, window, num_splits, dt)
    ws = torch.full((max(n, 16),), 255, dtype=torch.uint8, device=dev)  # NaN partials unless written
    if page_size:
        attn.attn_sink_decode_tree_paged(q, kp, vp, table, cu, par, lens, sinks, out, lse, c["max_q"], window, scale,
                                         num_splits, ws)
    else:
        attn.attn_sink_decode_tree(q, kc, vc, cu, par, lens, sinks, out, lse, c["max_q"], window, scale, num_splits,
                                   ws)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu()


def check(c, got, window, scale=0.125, oracle_case=None):
    """Bounds from the roundings.  With S = scale max_ij sum_d |q_id k_jd| the fp32 score is off by at most
    64 * 2^-24 S (a sum of 64 products), so a probability relatively by at most twice that plus the
    exponentials' 2^-21, and a sum of n terms by n * 2^-24: with A = sum_j p_j |v_j| (the operation on |v|)
        |out - ref| <= e A,  e = 2^-17 S + 2^-20 + n 2^-24 (fp32), and for bf16 inputs
    additionally 2^-8 A for p rounded to bf16 and 2^-8 (|ref| + the error so far) for the stored value."""
    o = oracle_case or c
    out, lse = got
    n = c["total"]
    assert (out[n:] == 3.0).all() and (lse[n:] == 3.0).all(), "rows behind the last sequence"
    args = (o["cu"], o["parents"], o["lens"], o["sinks"], window, scale)
    ro, rl = oracle.decode_tree(o["q"], o["k"], o["v"], *args)
    ra, _ = oracle.decode_tree(o["q"], o["k"], o["v"].abs(), *args)
    fin = lambda x: torch.nan_to_num(x.double(), nan=0.0)
    G = o["q"].shape[1] // o["k"].shape[2]
    S = 0.0
    for b in range(len(o["lens"])):
        qs = fin(o["q"][o["cu"][b]:o["cu"][b + 1]]).abs()
        if qs.numel():
            kk = fin(o["k"][b]).abs().repeat_interleave(G, 1)
            S = max(S, scale * float(torch.einsum("thd,jhd->thj", qs, kk).max()))
    keys = o["k"].shape[1]
    e = 2.0 ** -17 * S + 2.0 ** -20 + keys * 2.0 ** -24
    tol = e * ra[:n] + 1e-30
    if c["q"].dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * ra[:n]
        tol = tol + 2.0 ** -8 * (np.abs(ro[:n]) + tol)
    d = np.abs(out[:n].double().numpy() - ro[:n])
    assert (d <= tol).all(), f"out: worst {np.nanmax(d / tol):.3f} of the bound"
    # d lse = the probabilities' mean relative error, and log2's last bits
    fl = np.isfinite(rl[:n])
    assert np.array_equal(np.isfinite(lse[:n].numpy()), fl)
    dl = np.abs(lse[:n].double().numpy() - rl[:n])[fl]
    assert (dl <= e + 2.0 ** -21 * (1 + np.abs(rl[:n][fl]))).all(), f"lse: {dl.max():.3e}"


# ------------------------------------------------------------------ CPU: the oracle and the checks
def test_oracle_chain_is_the_prefill():
    """A chain over a cached prefix is the causal forward's last rows, dense and banded."""
    for window in (0, 5):
        c = make_case([13], [6], 4, 2, torch.float64, "chain", seed=3)
        out, lse = oracle.decode_tree(c["q"], c["k"], c["v"], c["cu"], c["parents"], c["lens"], c["sinks"], window, 0.2)
        ro, rl = oracle.fwd(c["q"][None], c["k"], c["v"], c["sinks"], window, 0.2)
        assert np.allclose(out, ro[0], atol=1e-13) and np.allclose(lse, rl[0].T, atol=1e-13)


def test_oracle_tree_against_masked_softmax():
    """Every path of a tree, by a mask built from matrix powers of the parent relation."""
    c = make_case([9], [12], 2, 1, torch.float64, "random", seed=4)
    par = c["parents"].tolist()
    up = np.zeros((12, 12))
    for i, a in enumerate(par):
        if a >= 0:
            up[i, a] = 1
    hops = [np.eye(12)]
    for _ in range(12):
        hops.append(hops[-1] @ up)
    depth = sum(h.sum(1) for h in hops[1:])
    for window in (0, 3):
        vis = np.zeros((12, 21), dtype=bool)
        for s, h in enumerate(hops):
            if window <= 0 or s < window:
                vis[:, 9:] |= h > 0
        for j in range(9):
            vis[:, j] = True if window <= 0 else j > 9 + depth - window
        out, lse = oracle.decode_tree(c["q"], c["k"], c["v"], c["cu"], c["parents"], c["lens"], c["sinks"], window, 0.2)
        for h in range(2):
            s = np.where(vis, (c["q"][:, h] @ c["k"][0, :, 0].T).numpy() * 0.2, -np.inf)
            z = np.exp(s).sum(1) + math.exp(float(c["sinks"][h]))
            assert np.allclose(lse[:, h], np.log(z), atol=1e-12)
            assert np.allclose(out[:, h], np.exp(s) / z[:, None] @ c["v"][0, :, 0].numpy(), atol=1e-12)


def fake(n):
    return [0x7f0000000000 + 0x1000 * i for i in range(n)]


def test_host_checks():
    lib = attn.load()
    q, k, v, cu, par, sl, s, o, l, ws, tab = fake(11)

    def call(q_=q, cu_=cu, par_=par, B=4, total=32, max_q=8, Lmax=4096, Hq=8, Hkv=2, D_=64, scale=0.125, splits=8,
             w=ws, wbytes=1 << 24, dtype=1):
        return lib.attn_sink_decode_tree(q_, k, v, cu_, par_, sl, s, o, l, B, total, max_q, Lmax, Hq, Hkv, D_, 0, scale,
                                         splits, w, wbytes, dtype, None)

    for bad in (dict(q_=None), dict(cu_=None), dict(par_=None), dict(B=0), dict(total=0), dict(max_q=0), dict(Lmax=0),
                dict(Hkv=3), dict(splits=129), dict(splits=-1)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(D_=128), dict(dtype=2), dict(max_q=257), dict(scale=0.0), dict(scale=float("inf"))):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(q_=q + 8) == MISALIGNED
    assert call(par_=par + 4) == MISALIGNED
    assert call(w=ws + 4) == MISALIGNED
    size = attn.attn_sink_decode_tree_workspace_size
    need = size(4, 32, 8, 8, 2, 64, 4096, 0, 8, 1)
    assert need > 0
    assert call(w=None) == WORKSPACE
    assert call(wbytes=need - 1) == WORKSPACE
    # fp32: 8 chunks of 512 keys; one chunk needs none
    assert size(4, 32, 8, 8, 2, 64, 4096, 0, 8, 0) == 32 * 8 * 8 * 66 * 4
    assert call(dtype=0, wbytes=32 * 8 * 8 * 66 * 4 - 1) == WORKSPACE
    assert size(4, 32, 8, 8, 2, 64, 4096, 0, 1, 0) == 0
    # a window of a few tiles is never cut; the bf16 workspace does not grow with the cache
    assert size(4, 32, 8, 8, 2, 64, 4096, 128, 0, 1) == 0
    assert size(64, 512, 8, 64, 8, 64, 32768, 0, 0, 1) == size(64, 512, 8, 64, 8, 64, 1 << 20, 0, 0, 1)
    # sizes that the calls refuse report none
    assert size(4, 32, 257, 8, 2, 64, 4096, 0, 8, 1) == 0
    assert size(4, 32, 8, 8, 2, 64, 4096, 0, 129, 1) == 0
    assert size(4, 32, 8, 8, 2, 64, (1 << 30) + 1, 0, 8, 1) == 0 and call(Lmax=(1 << 30) + 1) == UNSUPPORTED

    def paged(ps=16, pages=256, num=1024, dtype=1, t=tab, Hkv=2):
        return lib.attn_sink_decode_tree_paged(q, k, v, t, cu, par, sl, s, o, l, 4, 32, 8, pages, ps, num, 8, Hkv, 64, 0,
                                               0.125, 8, ws, 0, dtype, None)

    for bad in (dict(ps=12), dict(ps=0), dict(pages=0), dict(num=0), dict(t=None), dict(pages=1 << 27), dict(Hkv=3)):
        assert paged(**bad) == INVALID, bad
    assert paged(t=tab + 4) == MISALIGNED
    assert paged() == WORKSPACE and paged(dtype=0) == WORKSPACE


def test_wrapper_checks():
    c = make_case([3], [2], 4, 2, torch.bfloat16)
    out, lse = torch.empty_like(c["q"]), torch.empty(2, 4)
    args = lambda **kw: [{**dict(q=c["q"], k=c["k"], v=c["v"], cu=c["cu"], parents=c["parents"], lens=c["lens"],
                                 sinks=c["sinks"], out=out, lse=lse), **kw}[x]
                         for x in ("q", "k", "v", "cu", "parents", "lens", "sinks", "out", "lse")]
    with pytest.raises(ValueError, match="CUDA"):
        attn.attn_sink_decode_tree(*args(), 2, 0, 0.125)
    for name, bad in (("parents", c["parents"][:1]), ("lens", torch.zeros(3)), ("lse", torch.empty(4, 2)),
                      ("out", out[:1]), ("v", c["v"][:, :2]), ("sinks", torch.zeros(3))):
        with pytest.raises(ValueError, match="must be"):
            attn.attn_sink_decode_tree(*args(**{name: bad}), 2, 0, 0.125)


# ------------------------------------------------------------------ GPU parity
@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("window", [0, 1, 7, 128])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (3, 3), (10, 2), (16, 1)])
def test_ragged_batch(Hq, Hkv, window, dtype):
    """Caches from none to many tiles, a sequence without tokens, one token, odd trees."""
    c = make_case([0, 130, 5, 63, 700, 64], [5, 1, 0, 17, 9, 3], Hq, Hkv, dtype, seed=11, pad_rows=2)
    check(c, run(c, window), window)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("page_size", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("window", [0, 60])
def test_paged(page_size, window, dtype):
    c = make_case([0, 257, 31, 640], [4, 11, 1, 33], 8, 2, dtype, seed=12, pad_rows=1)
    got = run(c, window, page_size)
    check(c, got, window)
    if page_size == 16:
        flat = run(c, window)
        assert torch.equal(got[0], flat[0]) and torch.equal(got[1], flat[1])  # the same tiles and splits


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("splits", [1, 2, 5, 40, 128])
@pytest.mark.parametrize("window", [0, 300])
def test_splits(splits, window, dtype):
    c = make_case([0, 2900, 70], [6, 30, 2], 8, 2, dtype, seed=13)
    check(c, run(c, window, 0, splits), window)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,G", [(3, 8), (7, 8), (12, 8), (40, 8)])
@pytest.mark.parametrize("window", [0, 50])
def test_many_short_sequences(window, T, G, dtype):
    """More units of a tile or two than CTAs: every CTA walks several, some cut; some sequences without tokens
    or without a cache."""
    g = torch.Generator().manual_seed(21)
    B = 400
    cached = torch.randint(0, 150, (B,), generator=g).tolist()
    ns = torch.randint(0, T + 1, (B,), generator=g).tolist()
    cached[:5], ns[:5] = [0, 0, 600, 149, 149], [0, T, T, 0, 1]
    c = make_case(cached, ns, 2 * G, 2, dtype, seed=22)
    c["max_q"] = T
    check(c, run(c, window, 16), window)


@gpu
@pytest.mark.parametrize("kind", ["chain", "star", "roots", "random"])
@pytest.mark.parametrize("T,G", [(256, 1), (255, 3), (128, 8), (61, 5), (1, 40)])
def test_tree_shapes(T, G, kind):
    c = make_case([50, 0], [T, max(1, T // 3)], 2 * G, 2, torch.bfloat16, kind, seed=14)
    for window in (0, 20):
        check(c, run(c, window), window)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sink", [-math.inf, 60.0, -60.0, -1e30, -3.4e38])
def test_sinks_and_large_scores(sink, dtype):
    """No sink, a sink far above and far below the scores; scores that move the running maximum often."""
    c = make_case([400, 3], [9, 2], 8, 2, dtype, seed=15, std=4.0)
    c["sinks"] = torch.full((8,), sink)
    c["k"][0, :400] *= torch.linspace(0.01, 1, 400)[:, None, None].to(dtype)  # growing scores
    for splits in (1, 3):
        check(c, run(c, 0, 0, splits), 0)
    c["q"] *= 4  # scores in the hundreds: probabilities of one key
    check(c, run(c, 0), 0)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_empty_and_bad_entries(dtype):
    """Lengths of zero or below, lengths shorter than the draft and beyond the cache, parents that point
    at themselves, forward or nowhere, offsets that run past the rows."""
    c = make_case([20, 30, 0, 10], [4, 5, 3, 4], 8, 2, dtype, seed=16)
    c["parents"] = torch.tensor([0, 5, -9, 1 << 30] + [-1, 0, 2, 1, -5] + [-1, 0, 1] + [-1, 0, 0, 2], dtype=torch.int32)
    got_case = dict(c, lens=torch.tensor([-3, 35, 2, 99999], dtype=torch.int32))
    Lmax = c["k"].shape[1]
    c["k"][3], c["v"][3] = 1.0, 0.5  # the last sequence is clamped to the whole cache
    ref = dict(c, lens=torch.tensor([0, 35, 2, Lmax], dtype=torch.int32))
    # (of the third sequence's three drafted tokens, two have their keys in the cache)
    out = run(got_case, 0)
    check(got_case, out, 0, oracle_case=ref)
    assert (out[0][:4] == 0).all() and torch.allclose(out[1][:4], c["sinks"].expand(4, -1))
    # a token bound below the longest draft: the rest of its rows are left alone
    cut = dict(c, lens=ref["lens"], max_q=3)
    o, l = run(cut, 0)
    full = run(dict(c, lens=ref["lens"]), 0)
    for b, n in enumerate((4, 5, 3, 4)):
        r0 = int(c["cu"][b])
        assert torch.equal(o[r0:r0 + 3], full[0][r0:r0 + 3])
        assert (o[r0 + 3:r0 + n] == 3.0).all() and (l[r0 + 3:r0 + n] == 3.0).all()


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_pages_behind_the_window_hold_anything(dtype):
    """Cache rows in front of every token's window and behind the sequence are NaN or infinite."""
    c = make_case([500], [6], 8, 2, dtype, "chain", seed=17)
    ref = {x: c[x].clone() if torch.is_tensor(c[x]) else c[x] for x in c}
    first = 500 - 100 + 1
    c["k"][0, :first] = float("inf")
    c["v"][0, :first] = float("nan")
    ref["k"][0, :first] = 0
    ref["v"][0, :first] = 0
    check(c, run(c, 100), 100, oracle_case=ref)
    kp, vp, table = paginate(c, 16)
    table[0, :first // 64 * 4] = -1  # whole tiles in front of it are not mapped at all
    check(c, run(c, 100, 16, pages=(kp, vp, table)), 100, oracle_case=ref)


@gpu
def test_long_cache_offsets():
    """A cache whose rows lie past 2^31 elements, its last sequence against the oracle."""
    B, Lmax, Hkv = 3, 1 << 20, 16
    c = make_case([40], [5], 16, Hkv, torch.bfloat16, seed=18)
    k = torch.zeros(B, Lmax, Hkv, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    n = Lmax - 1000
    g = torch.Generator(device="cuda").manual_seed(5)
    k[2, n - 300:n] = torch.randn(300, Hkv, D, device="cuda", generator=g)
    v[2, n - 300:n] = torch.randn(300, Hkv, D, device="cuda", generator=g)
    cu = torch.tensor([0, 0, 0, 5], dtype=torch.int32)
    lens = torch.tensor([0, 0, n], dtype=torch.int32)
    q = c["q"].cuda()
    out, lse = torch.empty_like(q), torch.empty(5, 16, device="cuda")
    w = 256
    ws = torch.empty(max(16, attn.attn_sink_decode_tree_workspace_size(B, 5, 5, 16, Hkv, D, Lmax, w, 0, 1)),
                     dtype=torch.uint8, device="cuda")
    attn.attn_sink_decode_tree(q, k, v, cu.cuda(), c["parents"].cuda(), lens.cuda(), c["sinks"].cuda(), out, lse, 5, w,
                               0.125, 0, ws)
    torch.cuda.synchronize()
    small = dict(c, k=k[2:, n - 300:n].cpu(), v=v[2:, n - 300:n].cpu(), cu=torch.tensor([0, 5], dtype=torch.int32),
                 lens=torch.tensor([300], dtype=torch.int32))
    check(dict(c, total=5), (out.cpu(), lse.cpu()), w, oracle_case=small)


@gpu
def test_streams_graphs_and_repeats():
    """The same call twice, on a side stream, captured and replayed with new lengths, and two captured
    graphs replayed at once with their own workspaces: bit for bit."""
    c = make_case([900, 333, 20], [8, 8, 8], 8, 2, torch.bfloat16, seed=19)
    dev = "cuda"
    t = {x: c[x].to(dev) for x in ("q", "k", "v", "cu", "parents", "lens", "sinks")}
    n = attn.attn_sink_decode_tree_workspace_size(3, 24, 8, 8, 2, D, t["k"].shape[1], 0, 4, 1)
    outs = [(torch.zeros_like(t["q"]), torch.zeros(24, 8, device=dev), torch.empty(n, dtype=torch.uint8, device=dev))
            for _ in range(3)]

    def call(k):
        o, l, ws = outs[k]
        attn.attn_sink_decode_tree(t["q"], t["k"], t["v"], t["cu"], t["parents"], t["lens"], t["sinks"], o, l, 8, 0,
                                   0.125, 4, ws)

    call(0)
    torch.cuda.synchronize()
    graphs = []
    for k in (1, 2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            call(k)
        graphs.append(gr)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s1):
            graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
    torch.cuda.synchronize()
    for k in (1, 2):
        assert torch.equal(outs[k][0], outs[0][0]) and torch.equal(outs[k][1], outs[0][1])
    # shorter sequences replayed into the same graph
    t["lens"].copy_(torch.tensor([600, 100, 9], dtype=torch.int32))
    graphs[0].replay()
    torch.cuda.synchronize()
    check(c, (outs[1][0].cpu(), outs[1][1].cpu()), 0, oracle_case=dict(c, lens=torch.tensor([600, 100, 9])))


@gpu
def test_one_token_is_the_decode():
    """A draft of one token is attn_sink_decode's query."""
    c = make_case([100, 2000, 64], [1, 1, 1], 16, 2, torch.bfloat16, seed=20)
    out, lse = run(c, 0)
    q, kc, vc, sl, s = (c[x].cuda() for x in ("q", "k", "v", "lens", "sinks"))
    o2, l2 = torch.empty_like(q), torch.empty(3, 16, device="cuda")
    attn.attn_sink_decode(q, kc, vc, sl, s, o2, l2, 0, 0.125, 1)
    torch.cuda.synchronize()
    check(c, (o2.cpu(), l2.cpu()), 0)
    check(c, (out, lse), 0)
    assert attn.attn_sink_get_device_status() == 0


@gpu
@pytest.mark.parametrize("T", [1, 6, 16, 60])
def test_expired_waits_are_reported(T):
    """With a limit of 1 ns the waits that outlast the hardware's own suspension of a try expire (2 GB of cache
    that every CTA reads at once): the call winds down, the status says so once, and the next call with the
    default limit is right.  (480 rows a KV head are bound by arithmetic, and no wait need be that long.)"""
    B, L, Hkv = 64, 16384, 8
    k = torch.zeros(B, L, Hkv, D, dtype=torch.bfloat16, device="cuda")
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32).cuda()
    q = torch.zeros(B * T, 64, D, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(B * T, 64, device="cuda")
    ws = torch.empty(attn.attn_sink_decode_tree_workspace_size(B, B * T, T, 64, Hkv, D, L, 0, 0, 1), dtype=torch.uint8,
                     device="cuda")
    args = (q, k, k.clone(), i32(range(0, B * T + 1, T)), i32([-1] * (B * T)), i32([L] * B),
            torch.zeros(64, device="cuda"), out, lse, T, 0, 0.125, 0, ws)
    old = attn.attn_sink_set_wait_timeout_ns(1)
    try:
        attn.attn_sink_decode_tree(*args)
        status = attn.attn_sink_get_device_status()
    finally:
        attn.attn_sink_set_wait_timeout_ns(old)
    assert status == -7 or (T == 60 and status == 0)
    assert attn.attn_sink_get_device_status() == 0
    attn.attn_sink_decode_tree(*args)
    assert attn.attn_sink_get_device_status() == 0
    # zero keys: every one of L - T cached and one drafted key, and the sink, weighs the same
    assert (out == 0).all() and torch.allclose(lse, torch.tensor(math.log(L - T + 2.0), device="cuda"), atol=1e-5)
    c = make_case([300, 500, 100], [T, T, 1], 16, 2, torch.bfloat16, seed=23)
    check(c, run(c, 0), 0)
