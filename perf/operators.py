"""Measured cases of the speculative-decoding operators and of the QK-norm prologue.

Four operators: attention of a tree of drafted tokens over a KV cache (contiguous and paged), the page
tables and slot maps it needs, the QKV prologue with per-head norms of q and k, and that prologue's
backward.  ``run`` computes them in plain torch operations, or (``own``) through the library's calls.
"""
from __future__ import annotations

import math

import torch

own = False

D = 64
# gpt-oss's context extension: 4096 original positions scaled 32 times
YARN = dict(rope_theta=150000.0, rope_factor=32.0, rope_original_max_pos=4096, beta_fast=32.0, beta_slow=1.0)
EPS = 2.0 ** -20  # the norms' epsilon, exact in 32 bits (about 1e-6)


def listed():
    return [
        # ---- tree attention
        # a small server's verification step: 4 requests, a chain-like draft of 4 tokens, short contexts
        dict(op="tree", name="tree_paged_b4_t4", paged=True, page_size=16, B=4, T=4, lmin=300, lmax=1200, Hq=64, Hkv=8,
             window=0, dtype="bf16"),
        # the 64-sequence decode workload (lengths 1024 to 32768) with 8 drafted tokens each, 16-key pages
        dict(op="tree", name="tree_paged_b64_t8", paged=True, page_size=16, B=64, T=8, lmin=1024, lmax=32768, Hq=64,
             Hkv=8, window=0, dtype="bf16"),
        # the same sequences in a layer banded to 128 keys, 16 drafted tokens
        dict(op="tree", name="tree_paged_b64_t16_w128", paged=True, page_size=64, B=64, T=16, lmin=1024, lmax=32768,
             Hq=64, Hkv=8, window=128, dtype="bf16"),
        # one long context in a contiguous cache, a wide tree of 32
        dict(op="tree", name="tree_b1_t32_l131072", paged=False, page_size=0, B=1, T=32, lmin=131072, lmax=131072,
             Hq=64, Hkv=8, window=0, dtype="bf16"),
        # wide trees of 61 tokens over medium contexts: 488 rows per KV head, bound by arithmetic
        dict(op="tree", name="tree_b16_t61", paged=False, page_size=0, B=16, T=61, lmin=4001, lmax=8191, Hq=64, Hkv=8,
             window=0, dtype="bf16"),
        # the exact 32-bit path, odd sizes, groups of 3 heads
        dict(op="tree", name="tree_f32_b3_t7", paged=False, page_size=0, B=3, T=7, lmin=77, lmax=1025, Hq=6, Hkv=2,
             window=0, dtype="f32"),
        # ---- page tables and slot maps
        # a verification step of 64 requests with 8 drafted tokens each
        dict(op="map", name="map_b64_t8", B=64, nmin=8, nmax=8, cmin=1024, cmax=32700, page_size=16, tree=True, pad=0),
        # a mixed step: 1000 requests, decodes and prefill chunks, padded to a captured token count
        dict(op="map", name="map_b1000_mixed", B=1000, nmin=0, nmax=130, cmin=0, cmax=8000, page_size=16, tree=False,
             pad=999),
        # ---- prologue with per-head norms
        # 64 requests x 8 drafted tokens appended to a paged cache
        dict(op="norm", name="norm_append_t512", T=512, Hq=64, Hkv=8, bias=False, interleaved=False, scatter=True),
        # a prompt of 4096 tokens with projection biases
        dict(op="norm", name="norm_t4096", T=4096, Hq=64, Hkv=8, bias=True, interleaved=False, scatter=False),
        # ---- its backward
        # an odd small batch, interleaved pairs, groups of 5
        dict(op="norm_bwd", name="norm_bwd_t1003", T=1003, Hq=10, Hkv=2, bias=True, interleaved=True),
        # the training shape: 8 sequences of 8192 tokens
        dict(op="norm_bwd", name="norm_bwd_t65536", T=65536, Hq=64, Hkv=8, bias=True, interleaved=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "map", "norm", "norm_bwd"])
    if op == "tree":
        f32 = rng.random() < 0.2
        Hq, Hkv = rng.choice([(64, 8), (64, 8), (8, 2), (6, 2), (16, 1), (10, 2), (4, 4), (24, 1)])
        lmax = _log_int(rng, 1, 2048 if f32 else 131072)
        lmin = max(1, min(lmax, int(lmax * rng.choice([0.03, 0.3, 1.0]))))
        T = _log_int(rng, 1, 16 if f32 else 200)
        B = _log_int(rng, 1, 6 if f32 else 64)
        # no dearer than the listed 64-sequence case (tokens of cache) and the 61-token one (products)
        while B > 1 and (B * (lmin + lmax) * Hkv > 64 * 33792 * 8 or B * (lmin + lmax) * T * Hq > 16 * 12192 * 61 * 64):
            B = max(1, B // 2)
        while T > 1 and B * (lmin + lmax) * T * Hq > 16 * 12192 * 61 * 64:
            T = max(1, T // 2)
        return dict(op=op, paged=rng.random() < 0.5, page_size=rng.choice([8, 16, 32, 64, 128]), B=B, T=T, lmin=lmin,
                    lmax=lmax, Hq=Hq, Hkv=Hkv, window=rng.choice([0, 0, 128, rng.randint(1, 700)]),
                    dtype="f32" if f32 else "bf16")
    if op == "map":
        nmax = _log_int(rng, 1, 256)
        return dict(op=op, B=_log_int(rng, 1, 1000), nmin=rng.choice([0, nmax]), nmax=nmax, cmin=0,
                    cmax=_log_int(rng, 1, 32000), page_size=rng.choice([8, 16, 32, 64, 128]), tree=rng.random() < 0.5,
                    pad=rng.choice([0, 0, rng.randint(1, 500)]))
    Hq, Hkv = rng.choice([(64, 8), (8, 2), (10, 2), (16, 1), (4, 4), (40, 8)])
    c = dict(op=op, T=_log_int(rng, 1, 65536), Hq=Hq, Hkv=Hkv, bias=rng.random() < 0.5,
             interleaved=rng.random() < 0.3)
    if op == "norm":
        c["scatter"] = rng.random() < 0.5
    return c


# ------------------------------------------------------------------ inputs
def _spread(n, lo, hi):
    """n lengths evenly over [lo, hi] (a case's total work does not depend on the seed)."""
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _gens(seed):
    return torch.Generator().manual_seed(seed), torch.Generator(device="cuda").manual_seed(seed + 1)


def _tree(n, g):
    """Parents of n drafted tokens: token 0 the root, most of the others near the token before them."""
    back = torch.randint(0, 4, (n,), generator=g) * torch.randint(0, 3, (n,), generator=g)
    par = torch.arange(n) - 1 - back
    return torch.where(torch.arange(n) == 0, torch.full_like(par, -1), par.clamp_min(0)).to(torch.int32)


def _lens(case, g):
    lens = _spread(case["B"], case["lmin"], case["lmax"])
    return [lens[i] for i in torch.randperm(len(lens), generator=g).tolist()]


def _prepare_tree(case, seed):
    g, gd = _gens(seed)
    B, T, Hq, Hkv, ps = case["B"], case["T"], case["Hq"], case["Hkv"], case["page_size"]
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    cached = _lens(case, g)
    lens = [c + T for c in cached]
    lmax = max(lens)
    total = B * T
    st = dict(case=case, cached=cached, dt=dt, lens=lens)
    st["q"] = torch.randn(total, Hq, D, device="cuda", generator=gd).to(dt)
    if case["paged"]:
        per = [(n + ps - 1) // ps for n in lens]
        width = (max(per) + 3) // 4 * 4
        pages = sum(per) + 5
        perm = torch.randperm(pages, generator=g).to(torch.int32)
        table = torch.full((B, width), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(per):
            table[b, :n] = perm[at:at + n]
            at += n
        shape = (pages, ps, Hkv, D)
        st["table"] = table.cuda()
        bound = width * ps
    else:
        shape = (B, lmax, Hkv, D)
        bound = lmax
    st["k"] = torch.empty(shape, dtype=dt, device="cuda")
    st["v"] = torch.empty(shape, dtype=dt, device="cuda")
    for x in (st["k"], st["v"]):
        for part in torch.chunk(x, max(1, min(64, shape[0])), 0):
            part.copy_(torch.randn(part.shape, device="cuda", generator=gd, dtype=torch.float32))
    st["sinks"] = torch.randn(Hq, generator=g).cuda()
    st["seqlens"] = torch.tensor(lens, dtype=torch.int32).cuda()
    st["cu"] = (torch.arange(B + 1, dtype=torch.int32) * T).cuda()
    st["parents_host"] = [_tree(T, g) for _ in range(B)]
    st["parents"] = torch.cat(st["parents_host"]).cuda()
    st["out"] = torch.empty(total, Hq, D, dtype=dt, device="cuda")
    st["lse"] = torch.empty(total, Hq, device="cuda")
    if own:
        import gqa_softmax_attention_attn_b200 as attn

        n = attn.attn_sink_decode_tree_workspace_size(B, total, T, Hq, Hkv, D, bound, case["window"], 0,
                                                      attn.DTYPE_F32 if dt == torch.float32 else attn.DTYPE_BF16)
        st["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    return st


def _prepare_map(case, seed):
    g, _ = _gens(seed)
    B, ps = case["B"], case["page_size"]
    new = _spread(B, case["nmin"], case["nmax"])
    new = [new[i] for i in torch.randperm(B, generator=g).tolist()]
    cached = _spread(B, case["cmin"], case["cmax"])
    cached = [cached[i] for i in torch.randperm(B, generator=g).tolist()]
    have = [(c + ps - 1) // ps for c in cached]
    need = [(c + n + ps - 1) // ps for c, n in zip(cached, new)]
    width = (max(max(need), 1) + 3) // 4 * 4
    pages = sum(need) + 16
    perm = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(have):
        table[b, :n] = perm[at:at + n]
        at += n
    total = max(sum(new) + case["pad"], 1)
    st = dict(case=case, pages=pages, total=total)
    st["cached"] = torch.tensor(cached, dtype=torch.int32).cuda()
    st["new"] = torch.tensor(new, dtype=torch.int32).cuda()
    st["free"] = perm[at:].clone().cuda()
    st["table"] = table.cuda()
    st["parents"] = None
    if case["tree"]:
        par = torch.full((total,), -1, dtype=torch.int32)
        t = 0
        for n in new:
            if n:
                par[t:t + n] = _tree(n, g)
            t += n
        st["parents"] = par.cuda()
    for name, n in (("seqlens", B), ("cu", B + 1), ("positions", total), ("rows", total), ("stats", 4)):
        st[name] = torch.empty(n, dtype=torch.int32, device="cuda")
    return st


def _prepare_norm(case, seed):
    g, gd = _gens(seed)
    T, Hq, Hkv = case["T"], case["Hq"], case["Hkv"]
    W = (Hq + 2 * Hkv) * D
    bf = torch.bfloat16
    st = dict(case=case)
    st["qkv"] = torch.randn(T, W, device="cuda", generator=gd).to(bf)
    st["bias"] = torch.randn(W, device="cuda", generator=gd) * 0.1 if case["bias"] else None
    st["qw"] = 1.0 + 0.2 * torch.randn(D, device="cuda", generator=gd)
    st["kw"] = 1.0 + 0.2 * torch.randn(D, device="cuda", generator=gd)
    st["positions"] = torch.randint(0, 131072, (T,), generator=g, dtype=torch.int64).to(torch.int32).cuda()
    if case["op"] == "norm":
        rows = T
        st["kv_rows"] = None
        if case["scatter"]:
            rows = 2 * T + 3
            st["kv_rows"] = torch.randperm(rows, generator=g)[:T].to(torch.int32).cuda()
        st["q"] = torch.empty(T, Hq, D, dtype=bf, device="cuda")
        st["k"] = torch.zeros(rows, Hkv, D, dtype=bf, device="cuda")
        st["v"] = torch.zeros(rows, Hkv, D, dtype=bf, device="cuda")
        return st
    st["dq"] = (torch.randn(T, Hq, D, device="cuda", generator=gd) * 0.1).to(bf)
    st["dk"] = (torch.randn(T, Hkv, D, device="cuda", generator=gd) * 0.1).to(bf)
    st["dv"] = (torch.randn(T, Hkv, D, device="cuda", generator=gd) * 0.1).to(bf)
    st["dqkv"] = torch.empty(T, W, dtype=bf, device="cuda")
    st["dbias"] = torch.empty(W, device="cuda") if case["bias"] else None
    st["dqw"], st["dkw"] = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    if own:
        import gqa_softmax_attention_attn_b200 as attn

        n = attn.attn_sink_qk_norm_prologue_bwd_workspace_size(T, Hq, Hkv, D)
        st["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    return st


def prepare(case, seed):
    if case["op"] == "tree":
        return _prepare_tree(case, seed)
    if case["op"] == "map":
        return _prepare_map(case, seed)
    return _prepare_norm(case, seed)


# ------------------------------------------------------------------ one pass
def run(st):
    op = st["case"]["op"]
    return (_own if own else _plain)[op](st)


def _own_tree(st):
    import gqa_softmax_attention_attn_b200 as attn

    c = st["case"]
    if c["paged"]:
        attn.attn_sink_decode_tree_paged(st["q"], st["k"], st["v"], st["table"], st["cu"], st["parents"],
                                         st["seqlens"], st["sinks"], st["out"], st["lse"], c["T"], c["window"],
                                         0.125, 0, st["ws"])
    else:
        attn.attn_sink_decode_tree(st["q"], st["k"], st["v"], st["cu"], st["parents"], st["seqlens"], st["sinks"],
                                   st["out"], st["lse"], c["T"], c["window"], 0.125, 0, st["ws"])
    return st["out"], st["lse"]


def _own_map(st):
    import gqa_softmax_attention_attn_b200 as attn

    attn.attn_sink_page_map(st["cached"], st["new"], st["free"], st["table"], st["seqlens"], st["cu"],
                            st["positions"], st["rows"], st["stats"], st["case"]["page_size"], st["pages"],
                            parents=st["parents"])
    return st["table"], st["seqlens"], st["cu"], st["positions"], st["rows"], st["stats"]


def _own_norm(st):
    import gqa_softmax_attention_attn_b200 as attn

    attn.attn_sink_qk_norm_prologue(st["qkv"], st["bias"], st["qw"], st["kw"], st["positions"], st["q"], st["k"],
                                    st["v"], EPS, interleaved=st["case"]["interleaved"], kv_rows=st["kv_rows"], **YARN)
    return st["q"], st["k"], st["v"]


def _own_norm_bwd(st):
    import gqa_softmax_attention_attn_b200 as attn

    attn.attn_sink_qk_norm_prologue_bwd(st["qkv"], st["bias"], st["qw"], st["kw"], st["positions"], st["dq"],
                                        st["dk"], st["dv"], st["dqkv"], st["dbias"], st["dqw"], st["dkw"], EPS,
                                        workspace=st["ws"], interleaved=st["case"]["interleaved"], **YARN)
    return tuple(x for x in (st["dqkv"], st["dbias"], st["dqw"], st["dkw"]) if x is not None)


def _ancestors(par):
    """[B, T, T] truth values: token i descends from token j, or is it."""
    B, T = par.shape
    a = torch.eye(T, device=par.device).expand(B, T, T).clone()
    i = torch.arange(T, device=par.device)
    bb = torch.arange(B, device=par.device)[:, None].expand(B, T)
    ok = par >= 0
    a[bb[ok], i.expand(B, T)[ok], par.long()[ok]] = 1.0
    step = 1
    while step < T:
        a = ((a @ a) > 0).float()
        step *= 2
    return a > 0


def _plain_tree(st):
    c = st["case"]
    B, T, Hq, Hkv, w, ps = c["B"], c["T"], c["Hq"], c["Hkv"], c["window"], c["page_size"]
    G = Hq // Hkv
    anc = _ancestors(st["parents"].view(B, T))
    depth = anc.sum(-1) - 1
    if w > 0:
        anc = anc & (depth[:, :, None] - depth[:, None, :] < w)
    sink = st["sinks"].view(Hkv, 1, G, 1)
    for b in range(B):
        n, cached = st["lens"][b], st["cached"][b]
        lo = max(0, cached - w + 1) if w > 0 else 0
        if c["paged"]:
            j = torch.arange(lo, n, device="cuda")
            page = st["table"][b][j // ps].long()
            k, v = st["k"][page, j % ps], st["v"][page, j % ps]
        else:
            k, v = st["k"][b, lo:n], st["v"][b, lo:n]
        q = st["q"][b * T:(b + 1) * T].float().view(T, Hkv, G, D).permute(1, 0, 2, 3).reshape(Hkv, T * G, D)
        s = torch.matmul(q * 0.125, k.float().permute(1, 2, 0)).view(Hkv, T, G, n - lo)
        if w > 0:
            j = torch.arange(lo, cached, device="cuda")
            see = j[None, :] > (cached + depth[b])[:, None] - w
            s[..., :cached - lo].masked_fill_(~see[None, :, None, :], -math.inf)
        s[..., cached - lo:].masked_fill_(~anc[b][None, :, None, :], -math.inf)
        m = torch.maximum(s.amax(-1, keepdim=True), sink)
        p = s.sub_(m).exp_()
        z = p.sum(-1, keepdim=True) + (sink - m).exp()
        o = torch.matmul(p.view(Hkv, T * G, n - lo), v.float().permute(1, 0, 2)).view(Hkv, T, G, D) / z
        st["out"][b * T:(b + 1) * T] = o.permute(1, 0, 2, 3).reshape(T, Hq, D).to(st["dt"])
        st["lse"][b * T:(b + 1) * T] = (m + z.log()).permute(1, 0, 2, 3).reshape(T, Hq)
    return st["out"], st["lse"]


def _plain_map(st):
    c = st["case"]
    B, ps, total = c["B"], c["page_size"], st["total"]
    cached, new, table = st["cached"].long(), st["new"].long(), st["table"]
    dev = table.device
    have = (cached + ps - 1) // ps
    take = (cached + new + ps - 1) // ps - have
    first = torch.cumsum(take, 0) - take
    st["seqlens"].copy_(cached + new)
    st["cu"][0] = 0
    st["cu"][1:] = torch.cumsum(new, 0)
    cu = st["cu"].long()
    # the pages taken: entry e of request b is free page first[b] + e - have[b]
    e = torch.arange(table.shape[1], device=dev)[None, :]
    fresh = (e >= have[:, None]) & (e < (have + take)[:, None])
    at = (first[:, None] + e - have[:, None]).clamp(0, st["free"].numel() - 1)
    table.copy_(torch.where(fresh, st["free"][at], table))
    # token t belongs to the last request that starts at or before it
    t = torch.arange(total, device=dev)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    real = b < B
    b = b.clamp_max(B - 1)
    i = t - cu[b]
    if c["tree"]:
        # depths by doubling: each round hops twice as far towards the root
        par = st["parents"].long()
        up = torch.where((par >= 0) & real, cu[b] + par, torch.full_like(par, total))
        up = torch.cat([up, up.new_full((1,), total)])
        depth = (up < total).long()
        step = 1
        while step < max(c["nmax"], 2):
            depth = depth + depth[up]
            up = up[up]
            step *= 2
        depth = depth[:total]
    else:
        depth = i
    st["positions"].copy_(torch.where(real, cached[b] + depth, torch.zeros_like(t)))
    j = cached[b] + i
    page = table[b, torch.where(real, j // ps, torch.zeros_like(j))].long()
    st["rows"].copy_(torch.where(real, page * ps + j % ps, torch.full_like(t, -1)))
    st["stats"].copy_(torch.stack([new.sum(), take.sum(), torch.zeros_like(take[0]), torch.zeros_like(take[0])]))
    return st["table"], st["seqlens"], st["cu"], st["positions"], st["rows"], st["stats"]


def _angles(positions):
    """cos and sin of every (token, pair), the attention factor in them, formed in 64 bits."""
    base, factor, L0 = YARN["rope_theta"], YARN["rope_factor"], YARN["rope_original_max_pos"]
    i = torch.arange(D // 2, dtype=torch.float64, device=positions.device)
    f = base ** (-2.0 * i / D)
    lo, hi = (D * math.log(L0 / (2 * math.pi * n)) / (2 * math.log(base)) for n in (YARN["beta_fast"],
                                                                                   YARN["beta_slow"]))
    ramp = ((i - lo) / (hi - lo)).clamp(0, 1)
    f = f * (1 - ramp) + f / factor * ramp
    a = positions.double()[:, None] * f[None, :]
    m = 0.1 * math.log(factor) + 1.0
    return (a.cos() * m).float()[:, None, :], (a.sin() * m).float()[:, None, :]


def _pairs(x, interleaved):
    return (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :D // 2], x[..., D // 2:])


def _join(a, b, interleaved):
    return torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)


def _plain_norm(st):
    c = st["case"]
    T, Hq, Hkv, il = c["T"], c["Hq"], c["Hkv"], c["interleaved"]
    y = st["qkv"].float()
    if st["bias"] is not None:
        y = y + st["bias"]
    y = y.view(T, Hq + 2 * Hkv, D)
    cos, sin = _angles(st["positions"])
    outs = []
    for x, w in ((y[:, :Hq], st["qw"]), (y[:, Hq:Hq + Hkv], st["kw"])):
        n = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
        a, b = _pairs(n, il)
        outs.append(_join(a * cos - b * sin, b * cos + a * sin, il).to(torch.bfloat16))
    st["q"].copy_(outs[0])
    v = y[:, Hq + Hkv:].to(torch.bfloat16)
    if st["kv_rows"] is None:
        st["k"].copy_(outs[1])
        st["v"].copy_(v)
    else:
        rows = st["kv_rows"].long()
        st["k"][rows] = outs[1]
        st["v"][rows] = v
    return st["q"], st["k"], st["v"]


def _plain_norm_bwd(st):
    c = st["case"]
    T, Hq, Hkv, il = c["T"], c["Hq"], c["Hkv"], c["interleaved"]
    W = (Hq + 2 * Hkv) * D
    dbias = torch.zeros(W, dtype=torch.float64, device="cuda")
    dws = [torch.zeros(D, dtype=torch.float64, device="cuda") for _ in range(2)]
    step = 8192  # tokens at a time
    for t0 in range(0, T, step):
        sl = slice(t0, min(T, t0 + step))
        y = st["qkv"][sl].float()
        if st["bias"] is not None:
            y = y + st["bias"]
        y = y.view(-1, Hq + 2 * Hkv, D)
        cos, sin = _angles(st["positions"][sl])
        parts = []
        for k, (x, w, g) in enumerate(((y[:, :Hq], st["qw"], st["dq"][sl]),
                                       (y[:, Hq:Hq + Hkv], st["kw"], st["dk"][sl]))):
            ga, gb = _pairs(g.float(), il)
            g = _join(ga * cos + gb * sin, gb * cos - ga * sin, il)
            r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
            n = x * r
            dws[k] += (g * n).double().sum((0, 1))
            gw = g * w
            parts.append(r * (gw - n * (gw * n).mean(-1, keepdim=True)))
        parts.append(st["dv"][sl].float())
        dy = torch.cat(parts, 1).view(-1, W)
        dbias += dy.double().sum(0)
        st["dqkv"][sl] = dy.to(torch.bfloat16)
    if st["dbias"] is not None:
        st["dbias"].copy_(dbias)
    st["dqw"].copy_(dws[0])
    st["dkw"].copy_(dws[1])
    return tuple(x for x in (st["dqkv"], st["dbias"], st["dqw"], st["dkw"]) if x is not None)


_plain = dict(tree=_plain_tree, map=_plain_map, norm=_plain_norm, norm_bwd=_plain_norm_bwd)
_own = dict(tree=_own_tree, map=_own_map, norm=_own_norm, norm_bwd=_own_norm_bwd)


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    if case["op"] == "map":
        return None  # whole numbers only
    st = prepare(case, seed)
    if case["op"] == "tree":
        return _exact_tree(case, st)
    if case["op"] == "norm":
        return _exact_norm(case, st)
    return _exact_norm_bwd(case, st)


def _exact_tree(case, st):
    B, T, Hq, Hkv, w, ps = (case[x] for x in ("B", "T", "Hq", "Hkv", "window", "page_size"))
    G = Hq // Hkv
    out = torch.zeros(B * T, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B * T, Hq, dtype=torch.float64, device="cuda")
    sinks = st["sinks"].double()
    for b in range(B):
        n, cached = st["lens"][b], st["cached"][b]
        par = st["parents_host"][b].tolist()
        paths = []  # each token's ancestors, itself last
        for i in range(T):
            paths.append((paths[par[i]] if par[i] >= 0 else []) + [i])
        bias = torch.full((T, n), -math.inf, dtype=torch.float64)
        for i, path in enumerate(paths):
            pos = cached + len(path) - 1
            first = 0 if w <= 0 else max(0, pos - w + 1)
            bias[i, first:cached] = 0.0
            for e, a in enumerate(path):
                if w <= 0 or len(path) - 1 - e < w:
                    bias[i, cached + a] = 0.0
        lo = 0 if w <= 0 else max(0, cached - w + 1)
        bias = bias[:, lo:].cuda()
        if case["paged"]:
            idx = (st["table"][b].long()[:, None] * ps + torch.arange(ps, device="cuda")).flatten()[lo:n]
            kb, vb = st["k"].view(-1, Hkv, D)[idx], st["v"].view(-1, Hkv, D)[idx]
        else:
            kb, vb = st["k"][b, lo:n], st["v"][b, lo:n]
        for g in range(Hkv):
            kg, vg = kb[:, g].double(), vb[:, g].double()
            for h in range(g * G, (g + 1) * G):
                s = st["q"][b * T:(b + 1) * T, h].double() @ kg.T / 8.0 + bias
                z = torch.logaddexp(torch.logsumexp(s, -1), sinks[h].expand(T))
                out[b * T:(b + 1) * T, h] = torch.exp(s - z[:, None]) @ vg
                lse[b * T:(b + 1) * T, h] = z
    return out, lse


def _rotation(positions):
    """Unit complex numbers times the attention factor, [T, 1, D/2]."""
    b, s, L0 = YARN["rope_theta"], YARN["rope_factor"], YARN["rope_original_max_pos"]
    edge = [D / 2 * math.log(L0 / (2 * math.pi * n)) / math.log(b) for n in (YARN["beta_fast"], YARN["beta_slow"])]
    f = []
    for i in range(D // 2):
        keep = 1.0 - min(1.0, max(0.0, (i - edge[0]) / (edge[1] - edge[0])))
        f.append((keep + (1.0 - keep) / s) * b ** (-i / (D / 2)))
    ang = torch.outer(positions.double(), torch.tensor(f, dtype=torch.float64, device=positions.device))
    return torch.polar(torch.full_like(ang, 0.1 * math.log(s) + 1.0), ang)[:, None, :]


def _to_complex(x, interleaved):
    x = x.unflatten(-1, (D // 2, 2)) if interleaved else x.unflatten(-1, (2, D // 2)).transpose(-1, -2)
    return torch.view_as_complex(x.contiguous())


def _to_real(z, interleaved):
    x = torch.view_as_real(z)
    return (x if interleaved else x.transpose(-1, -2)).flatten(-2)


def _exact_norm(case, st):
    T, Hq, Hkv = case["T"], case["Hq"], case["Hkv"]
    q = torch.empty(T, Hq, D, dtype=torch.float64, device="cuda")
    k, v = torch.zeros(st["k"].shape, dtype=torch.float64, device="cuda"), torch.zeros(
        st["v"].shape, dtype=torch.float64, device="cuda")
    rows = torch.arange(T, device="cuda") if st["kv_rows"] is None else st["kv_rows"].long()
    for t0 in range(0, T, 4096):
        sl = slice(t0, min(T, t0 + 4096))
        y = st["qkv"][sl].double()
        if st["bias"] is not None:
            y += st["bias"].double()
        y = y.unflatten(-1, (-1, D))
        rot = _rotation(st["positions"][sl])

        def head(x, w):
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / D + EPS) * w.double()
            return _to_real(_to_complex(x, case["interleaved"]) * rot, case["interleaved"])

        q[sl] = head(y[:, :Hq], st["qw"])
        k[rows[sl]] = head(y[:, Hq:Hq + Hkv], st["kw"])
        v[rows[sl]] = y[:, Hq + Hkv:]
    return q, k, v


def _exact_norm_bwd(case, st):
    T, Hq, Hkv, il = case["T"], case["Hq"], case["Hkv"], case["interleaved"]
    W = (Hq + 2 * Hkv) * D
    dqkv = torch.empty(T, W, dtype=torch.float64, device="cuda")
    dw = [0.0, 0.0]
    for t0 in range(0, T, 4096):
        sl = slice(t0, min(T, t0 + 4096))
        y = st["qkv"][sl].double()
        if st["bias"] is not None:
            y += st["bias"].double()
        y = y.unflatten(-1, (-1, D))
        back = _rotation(st["positions"][sl]).conj()  # the transpose of the scaled rotation
        dst = dqkv[sl].view(-1, Hq + 2 * Hkv, D)
        for k, (h0, h1, w, g) in enumerate(((0, Hq, st["qw"], st["dq"]), (Hq, Hq + Hkv, st["kw"], st["dk"]))):
            x = y[:, h0:h1]
            g = _to_real(_to_complex(g[sl].double(), il) * back, il)
            rms = torch.sqrt(x.square().sum(-1, keepdim=True) / D + EPS)
            dw[k] = dw[k] + (g * x / rms).sum((0, 1))
            u = g * w.double()
            dst[:, h0:h1] = u / rms - x * ((u * x).sum(-1, keepdim=True) / (D * rms ** 3))
        dst[:, Hq + Hkv:] = st["dv"][sl].double()
    out = (dqkv, dqkv.sum(0) if case["bias"] else None, dw[0], dw[1])
    return tuple(x for x in out if x is not None)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "tree":
        B, T, Hq, Hkv, w = (case[x] for x in ("B", "T", "Hq", "Hkv", "window"))
        eb = 4 if case["dtype"] == "f32" else 2
        cached = _spread(B, case["lmin"], case["lmax"])
        keys = sum((min(c, w - 1) if w > 0 else c) + T for c in cached)
        # every row against the cached keys of its window (taken at the root's depth) and at least itself
        pairs = sum(T * ((min(c, w - 1) if w > 0 else c) + 1) for c in cached) * Hq
        rows = B * T * Hq
        return dict(bytes=keys * Hkv * D * 2 * eb + rows * (2 * D * eb + 4) + B * T * 4, flops=pairs * 4 * D)
    if op == "map":
        B, ps = case["B"], case["page_size"]
        new = _spread(B, case["nmin"], case["nmax"])
        total = max(sum(new) + case["pad"], 1)
        taken = sum(n // ps for n in new)
        # lengths in and out, a slot and a position for every token (its parent read), the fresh pages' entries
        return dict(bytes=4 * (4 * B + (3 if case["tree"] else 2) * total + 2 * taken), flops=2 * B + 4 * total)
    T, Hq, Hkv = case["T"], case["Hq"], case["Hkv"]
    W = (Hq + 2 * Hkv) * D
    if op == "norm":
        return dict(bytes=4 * T * W + 8 * T, flops=T * (Hq + Hkv) * D * 7)
    return dict(bytes=6 * T * W + 4 * T, flops=T * (Hq + Hkv) * D * 16)
