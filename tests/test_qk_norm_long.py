"""The QK-norm prologue and its backward in their steady state: slabs of several batches of rotations and many
turns of the rings, and the gradients summed over tokens held to the depth of the kernel's own sums."""
import numpy as np
import pytest
import torch

import gqa_softmax_attention_attn_b200 as attn
import oracle
from test_qk_norm import D, EPS, YARN, close, forward_bound, make, oracle_rope, run_bwd, up

gpu = pytest.mark.gpu
# (tokens, query heads, KV heads): 46 or 47 tokens a slab forward, 69 to 72 backward, the last steps and batches
# of a slab ragged; 300 heads leave the last group of 16 a quarter full
SHAPES = [(4099, 64, 8), (1003, 300, 4)]


def slabs_of(T, heads):
    """The backward's division of the work: groups of 16 heads, and the slabs of tokens that two CTAs an SM leave."""
    groups = -(-heads // 16)
    n = max(1, min(-(-T // 4), 2 * 148 // groups))
    return groups, [(T * s // n, T * (s + 1) // n) for s in range(n)]


class Sums:
    """dbias, dq_weight and dk_weight with a bound each.  With u the gradient rotated back and n = y r, a term u n
    is off by at most 2^-20 A |n| for the rotation's angle and roundings (A = a (|dz_a| + |dz_b|), a the attention
    factor: u = a (c dz_a + s dz_b)) and 2^-20 |u n| for n's and the product's; a term of dbias by 2^-18 of
    E = r (|w| A + |n| mean(|w| A |n|)), whose two summands hold every product that dy adds up.  A sum adds at most
    `depth` times one after the other (a lane's tokens, the 4 token lanes, times the 16 heads of a group for the
    weights, then a sixteenth of the slabs' partial rows, of every group for the weights, and the 16 parts), each
    addition rounding by 2^-24 of a partial sum of absolute values."""

    def __init__(self, c, Hq, Hkv, rope, interleaved):
        T, heads = len(c["qkv"]), Hq + 2 * Hkv
        kw = oracle_rope(rope)
        groups, self.slabs = slabs_of(T, heads)
        lane = -(-max(e - b for b, e in self.slabs) // 4)
        f, a = oracle.yarn_frequencies(D, kw["base"], kw.get("factor", 1.0), kw.get("original_max_pos", 0.0),
                                       kw.get("beta_fast", 32.0), kw.get("beta_slow", 1.0))
        y = c["qkv"].double().numpy() + c["bias"].double().numpy()
        y = y.reshape(T, heads, D)
        pos = c["pos"].double().numpy()
        self.dx = oracle.qk_norm_prologue_bwd(c["qkv"], c["bias"], c["qw"], c["kw"], c["pos"], c["dq"], c["dk"], c["dv"],
                                              EPS, interleaved=interleaved, **kw)[0]
        E = np.zeros((T, heads, D))
        self.un, weight_err = [], []
        for sl, w, g in ((slice(0, Hq), c["qw"], c["dq"]), (slice(Hq, Hq + Hkv), c["kw"], c["dk"])):
            x, w, g = y[:, sl], w.double().abs().numpy(), g.double().numpy()
            r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + EPS)
            n = x * r
            u = oracle.rotate(g, -pos, f, a, interleaved)
            pair = np.arange(D) ^ 1 if interleaved else (np.arange(D) + D // 2) % D
            A = a * (np.abs(g) + np.abs(g[..., pair]))
            n_abs = np.abs(n)
            E[:, sl] = r * (w * A + n_abs * (w * A * n_abs).mean(-1, keepdims=True))
            self.un.append(u * n)
            weight_err.append((A * n_abs).sum((0, 1)))
        depth = lane + 4 + -(-len(self.slabs) // 16) + 16
        depth_w = lane + 4 * 16 + -(-len(self.slabs) * groups // 16) + 16
        self.refs = [self.dx.sum(0)] + [x.sum((0, 1)) for x in self.un]
        self.tols = [2.0 ** -18 * E.reshape(T, -1).sum(0) + depth * 2.0 ** -24 * np.abs(self.dx).sum(0) + 1e-30]
        for x, e in zip(self.un, weight_err):
            s = np.abs(x).sum((0, 1))
            self.tols.append(2.0 ** -20 * (e + s) + depth_w * 2.0 ** -24 * s + 1e-30)

    NAMES = ("dbias", "dq_weight", "dk_weight")

    def check(self, got):
        for name, g, ref, tol in zip(self.NAMES, got, self.refs, self.tols):
            close(g, ref, tol, name)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv", SHAPES)
def test_the_bounds_notice_what_is_left_out(T, Hq, Hkv, interleaved):
    """Sums of zero, and sums without one slab, without one token lane of one slab, without one head: the bound
    refuses most of their columns."""
    s = Sums(make(T, Hq, Hkv, 81), Hq, Hkv, YARN, interleaved)
    (b, e), h = s.slabs[len(s.slabs) // 2], Hkv // 2
    missing = [
        ("everything", s.refs),
        ("a slab", [s.dx[b:e].sum(0)] + [x[b:e].sum((0, 1)) for x in s.un]),
        ("a token lane of a slab", [s.dx[b + 1:e:4].sum(0)] + [x[b + 1:e:4].sum((0, 1)) for x in s.un]),
        ("a head", [np.where(np.arange(s.dx.shape[1]) // D == h, s.refs[0], 0)] + [x[:, h].sum(0) for x in s.un]),
    ]
    for what, parts in missing:
        for name, part, tol in zip(s.NAMES, parts, s.tols):
            cols = part != 0  # (one head's columns of dbias)
            assert (np.abs(part) > tol)[cols].mean() > 0.5, (what, name)


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv", SHAPES)
def test_backward_many_batches_a_slab(T, Hq, Hkv, interleaved):
    c = make(T, Hq, Hkv, 81)
    dqkv, *sums = run_bwd(up(c), YARN, interleaved)
    s = Sums(c, Hq, Hkv, YARN, interleaved)
    s.check(sums)
    # an element of dy: its share of the bound above before the rounding to bf16 (2^-8 of the value)
    rope = oracle_rope(YARN)
    a = oracle.yarn_frequencies(D, rope["base"], rope["factor"], rope["original_max_pos"], 32.0, 1.0)[1]
    y = (c["qkv"].double().numpy() + c["bias"].double().numpy()).reshape(T, -1, D)[:, :Hq + Hkv]
    r = 1 / np.sqrt((y * y).mean(-1, keepdims=True) + EPS)
    n = np.abs(y * r)
    g = np.abs(np.concatenate([c["dq"].double().numpy(), c["dk"].double().numpy()], 1))
    w = np.concatenate([np.broadcast_to(c[x].double().abs().numpy(), (h, D)) for x, h in (("qw", Hq), ("kw", Hkv))])
    wA = w * a * (g + g[..., np.arange(D) ^ 1 if interleaved else (np.arange(D) + D // 2) % D])
    E = r * (wA + n * (wA * n).mean(-1, keepdims=True))
    E = 2.0 ** -18 * np.concatenate([E, np.zeros((T, Hkv, D))], 1).reshape(T, -1)
    close(dqkv, s.dx, E + 2.0 ** -8 * (np.abs(s.dx) + E) + 1e-30, "dqkv")


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv", SHAPES)
def test_forward_many_batches_a_slab(T, Hq, Hkv, interleaved):
    """In token order, and into a cache whose rows are taken in random order, every eighth token without one."""
    c = make(T, Hq, Hkv, 82)
    t = up(c)
    rq, rk, rv = oracle.qk_norm_prologue(c["qkv"], c["bias"], c["qw"], c["kw"], c["pos"], Hq, Hkv, D, EPS,
                                         interleaved=interleaved, **oracle_rope(YARN))
    kb, vb = forward_bound(c, rk, Hq, Hkv, c["kw"]), 2.0 ** -8 * np.abs(rv) + 2.0 ** -20
    qb = forward_bound(c, rq, Hq, Hkv, c["qw"])
    total = 2 * T + 5
    rows = torch.randperm(total, generator=torch.Generator().manual_seed(7))[:T]
    rows[::8] = -1
    kept = [i for i in range(T) if i % 8]
    for cache in (False, True):
        n = total if cache else T
        q = torch.full((T, Hq, D), 5.0, dtype=torch.bfloat16, device="cuda")
        k, v = (torch.full((n, Hkv, D), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        attn.attn_sink_qk_norm_prologue(t["qkv"], t["bias"], t["qw"], t["kw"], t["pos"], q, k, v, EPS,
                                        interleaved=interleaved, kv_rows=rows.int().cuda() if cache else None, **YARN)
        torch.cuda.synchronize()
        close(q, rq, qb, "q")
        if not cache:
            close(k, rk, kb, "k")
            close(v, rv, vb, "v")
            continue
        at = rows[kept].cuda()
        close(k[at], rk[kept], kb[kept], "k")
        close(v[at], rv[kept], vb[kept], "v")
        rest = torch.ones(n, dtype=torch.bool, device="cuda")
        rest[at] = False
        assert (k[rest] == 5.0).all() and (v[rest] == 5.0).all()
