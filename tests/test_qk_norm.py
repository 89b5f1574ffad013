"""attn_sink_qk_norm_prologue and its backward: the oracle's pins and the argument checks on the CPU, parity
with the fp64 oracle on the GPU."""
import numpy as np
import pytest
import torch

import gqa_softmax_attention_attn_b200 as attn
import oracle

D = 64
INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = -1, -2, -3, -5
gpu = pytest.mark.gpu
YARN = dict(rope_theta=150000.0, rope_factor=32.0, rope_original_max_pos=4096, beta_fast=32.0, beta_slow=1.0)
PLAIN = dict(rope_theta=10000.0, rope_factor=1.0)
EPS = 2.0 ** -20


def oracle_rope(kw):
    return {dict(rope_theta="base", rope_factor="factor", rope_original_max_pos="original_max_pos").get(k, k): v
            for k, v in kw.items()}


def make(T, Hq, Hkv, seed, bias=True, std=1.0):
    g = torch.Generator().manual_seed(seed)
    W = (Hq + 2 * Hkv) * D
    r = lambda *s: torch.randn(*s, generator=g)
    return dict(qkv=(r(T, W) * std).bfloat16(), bias=r(W) * 0.3 if bias else None, qw=1 + 0.5 * r(D), kw=1 + 0.5 * r(D),
                pos=torch.randint(0, 131072, (T,), generator=g).int(), dq=r(T, Hq, D).bfloat16(),
                dk=r(T, Hkv, D).bfloat16(), dv=r(T, Hkv, D).bfloat16())


# ------------------------------------------------------------------ CPU
def test_oracle_unit_weights_and_rms():
    """Heads come out with root mean square `factor`, weights and rotation undone; v keeps its values."""
    c = make(5, 4, 2, 1)
    one = torch.ones(D)
    q, k, v = oracle.qk_norm_prologue(c["qkv"], c["bias"], one, one, c["pos"], 4, 2, D, 0.0, **oracle_rope(YARN))
    a = 0.1 * np.log(32.0) + 1
    assert np.allclose((q ** 2).mean(-1), a * a) and np.allclose((k ** 2).mean(-1), a * a)
    plain = oracle.qkv_prologue(c["qkv"], c["bias"], c["pos"], 4, 2, D, **oracle_rope(YARN))
    assert np.array_equal(v, plain[2])
    # proportional to the head without the norm, unit weights commuting with the rotation
    cos = (q * plain[0]).sum(-1) / np.sqrt((q ** 2).sum(-1) * (plain[0] ** 2).sum(-1))
    assert np.allclose(cos, 1.0)


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_gradients_by_differences(interleaved):
    """Central differences of L = <q, dq> + <k, dk> + <v, dv> in a random direction of every input."""
    T, Hq, Hkv = 3, 4, 2
    c = make(T, Hq, Hkv, 2)
    kw = dict(interleaved=interleaved, **oracle_rope(YARN))
    x = {n: c[n].double() for n in ("qkv", "bias", "qw", "kw")}

    def loss(**d):
        y = {**x, **d}
        q, k, v = oracle.qk_norm_prologue(y["qkv"], y["bias"], y["qw"], y["kw"], c["pos"], Hq, Hkv, D, EPS, **kw)
        return (q * c["dq"].double().numpy()).sum() + (k * c["dk"].double().numpy()).sum() + (
            v * c["dv"].double().numpy()).sum()

    grads = oracle.qk_norm_prologue_bwd(c["qkv"], c["bias"], c["qw"], c["kw"], c["pos"], c["dq"], c["dk"], c["dv"], EPS,
                                        **kw)
    g = torch.Generator().manual_seed(3)
    for n, grad in zip(("qkv", "bias", "qw", "kw"), grads):
        dirn = torch.randn(x[n].shape, generator=g, dtype=torch.float64)
        h = 1e-5
        diff = (loss(**{n: x[n] + h * dirn}) - loss(**{n: x[n] - h * dirn})) / (2 * h)
        assert np.isclose(diff, (grad * dirn.numpy()).sum(), rtol=1e-6, atol=1e-6), n


def fake(n):
    return [0x7f0000000000 + 0x1000 * i for i in range(n)]


def test_host_checks():
    lib = attn.load()
    qkv, b, qw, kw, pos, rows, q, k, v = fake(9)

    def call(qkv_=qkv, qw_=qw, kw_=kw, pos_=pos, rows_=rows, T=10, Hq=8, Hkv=2, D_=64, nrows=10, eps=1e-6,
             theta=10000.0, factor=32.0, L0=4096, bf=32.0, bs=1.0, inter=0):
        return lib.attn_sink_qk_norm_prologue(qkv_, b, qw_, kw_, pos_, rows_, q, k, v, T, Hq, Hkv, D_, nrows, eps,
                                              theta, factor, L0, bf, bs, inter, None)

    for bad in (dict(qkv_=None), dict(qw_=None), dict(kw_=None), dict(pos_=None), dict(T=0), dict(Hkv=3), dict(nrows=0),
                dict(rows_=None, nrows=5), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
                dict(theta=1.0), dict(factor=0.0), dict(L0=0), dict(bf=1.0), dict(inter=2)):
        assert call(**bad) == INVALID, bad
    assert call(D_=128) == UNSUPPORTED
    assert call(qw_=qw + 4) == MISALIGNED and call(rows_=rows + 8) == MISALIGNED
    dq, dk, dv, dx, db, dqw, dkw, ws = fake(17)[9:]
    need = attn.attn_sink_qk_norm_prologue_bwd_workspace_size(10, 8, 2, 64)
    assert need > 0 and attn.attn_sink_qk_norm_prologue_bwd_workspace_size(10, 8, 3, 64) == 0

    def bwd(bias=b, dq_=dq, dx_=dx, db_=db, dqw_=dqw, T=10, Hkv=2, D_=64, eps=1e-6, theta=1e4, inter=0, w=ws,
            wbytes=need):
        return lib.attn_sink_qk_norm_prologue_bwd(qkv, bias, qw, kw, pos, dq_, dk, dv, dx_, db_, dqw_, dkw, T, 8, Hkv,
                                                  D_, eps, theta, 1.0, 0, 32.0, 1.0, inter, w, wbytes, None)

    for bad in (dict(dq_=None), dict(dx_=None), dict(dqw_=None), dict(bias=None), dict(T=0), dict(Hkv=3),
                dict(eps=-1.0), dict(theta=0.5), dict(inter=3), dict(dx_=qkv), dict(dx_=dk)):
        assert bwd(**bad) == INVALID, bad
    assert bwd(D_=32) == UNSUPPORTED
    assert bwd(db_=db + 4) == MISALIGNED and bwd(w=ws + 4) == MISALIGNED
    assert bwd(w=None) == WORKSPACE and bwd(wbytes=need - 1) == WORKSPACE


# ------------------------------------------------------------------ GPU
def up(c):
    return {k: v.cuda() if torch.is_tensor(v) else v for k, v in c.items()}


def close(got, ref, err, what):
    d = np.abs(got.double().cpu().numpy() - ref)
    assert d.shape == ref.shape and (d <= err).all(), f"{what}: worst {np.nanmax(d / err):.3f} of the bound"


def forward_bound(c, ref, Hq, Hkv, weights):
    """A normalised head's fp32 values carry a few roundings each and the angle 2^-24 of half a turn, so a
    rotated value is off by at most 2^-20 of its pair's size (at most a max|n w|, n = y / rms, in two
    terms); then 2^-8 of the value for its rounding to bf16."""
    y = c["qkv"].double().numpy().reshape(len(ref), -1, D)
    if c["bias"] is not None:
        y = y + c["bias"].double().numpy().reshape(1, -1, D)
    y = y[:, :Hq] if weights is c["qw"] else y[:, Hq:Hq + Hkv]
    n = y / np.sqrt((y * y).mean(-1, keepdims=True) + EPS) * weights.double().numpy()
    small = 2.0 ** -20 * 2 * 1.35 * np.abs(n).max(-1, keepdims=True)
    return small + 2.0 ** -8 * (np.abs(ref) + small) + 1e-30


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rope", [YARN, PLAIN], ids=["yarn", "plain"])
@pytest.mark.parametrize("T,Hq,Hkv,bias", [(1, 8, 2, True), (7, 3, 3, False), (333, 64, 8, True), (9, 10, 2, False),
                                           (8, 1, 1, True), (3, 300, 4, True)])
def test_forward(T, Hq, Hkv, bias, rope, interleaved):
    c = make(T, Hq, Hkv, 31 + T, bias)
    t = up(c)
    q = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    k = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    attn.attn_sink_qk_norm_prologue(t["qkv"], t["bias"], t["qw"], t["kw"], t["pos"], q, k, v, EPS,
                                    interleaved=interleaved, **rope)
    torch.cuda.synchronize()
    rq, rk, rv = oracle.qk_norm_prologue(c["qkv"], c["bias"], c["qw"], c["kw"], c["pos"], Hq, Hkv, D, EPS,
                                         interleaved=interleaved, **oracle_rope(rope))
    close(q, rq, forward_bound(c, rq, Hq, Hkv, c["qw"]), "q")
    close(k, rk, forward_bound(c, rk, Hq, Hkv, c["kw"]), "k")
    close(v, rv, 2.0 ** -8 * np.abs(rv) + 2.0 ** -20, "v")  # one fp32 add, one rounding to bf16


@gpu
def test_forward_into_a_cache():
    """k and v go to their cache rows; rows outside the cache are not written, the others keep their values."""
    T, Hq, Hkv = 6, 8, 2
    c = make(T, Hq, Hkv, 41)
    t = up(c)
    rows = torch.tensor([3, -1, 50, 0, 2 ** 31 - 1, 49], dtype=torch.int32)
    k = torch.full((50, Hkv, D), 7.0, dtype=torch.bfloat16, device="cuda")
    v = torch.full_like(k, -3.0)
    q = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    attn.attn_sink_qk_norm_prologue(t["qkv"], t["bias"], t["qw"], t["kw"], t["pos"], q, k, v, EPS, kv_rows=rows.cuda(),
                                    **YARN)
    torch.cuda.synchronize()
    rq, rk, rv = oracle.qk_norm_prologue(c["qkv"], c["bias"], c["qw"], c["kw"], c["pos"], Hq, Hkv, D, EPS,
                                         **oracle_rope(YARN))
    close(q, rq, forward_bound(c, rq, Hq, Hkv, c["qw"]), "q")
    at, src = [3, 0, 49], [0, 3, 5]
    close(k[at], rk[src], forward_bound(c, rk, Hq, Hkv, c["kw"])[src], "k")
    close(v[at], rv[src], 2.0 ** -8 * np.abs(rv[src]) + 2.0 ** -20, "v")
    rest = [r for r in range(50) if r not in at]
    assert (k[rest] == 7.0).all() and (v[rest] == -3.0).all()


@gpu
def test_zero_and_large_heads():
    """A head of zeros stays zero; heads near bf16's largest squares and far below one are normalised alike."""
    T, Hq, Hkv = 4, 4, 2
    c = make(T, Hq, Hkv, 42, bias=False)
    c["qkv"][0] = 0
    c["qkv"][1] *= 1e15
    c["qkv"][2] *= 1e-3
    t = up(c)
    q = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.empty(T, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    attn.attn_sink_qk_norm_prologue(t["qkv"], None, t["qw"], t["kw"], t["pos"], q, k, v, EPS, **YARN)
    torch.cuda.synchronize()
    rq, rk, _ = oracle.qk_norm_prologue(c["qkv"], None, c["qw"], c["kw"], c["pos"], Hq, Hkv, D, EPS, **oracle_rope(YARN))
    assert (q[0] == 0).all() and (k[0] == 0).all()
    close(q, rq, forward_bound(c, rq, Hq, Hkv, c["qw"]), "q")
    close(k, rk, forward_bound(c, rk, Hq, Hkv, c["kw"]), "k")


def run_bwd(t, rope, interleaved, bias=True):
    T, Hq, Hkv = t["dq"].shape[0], t["dq"].shape[1], t["dk"].shape[1]
    W = (Hq + 2 * Hkv) * D
    dqkv = torch.full((T, W), float("nan"), dtype=torch.bfloat16, device="cuda")
    db = torch.full((W,), float("nan"), device="cuda") if bias else None
    dqw, dkw = (torch.full((D,), float("nan"), device="cuda") for _ in range(2))
    ws = torch.full((attn.attn_sink_qk_norm_prologue_bwd_workspace_size(T, Hq, Hkv, D),), 255, dtype=torch.uint8,
                    device="cuda")
    attn.attn_sink_qk_norm_prologue_bwd(t["qkv"], t["bias"], t["qw"], t["kw"], t["pos"], t["dq"], t["dk"], t["dv"],
                                        dqkv, db, dqw, dkw, EPS, interleaved=interleaved, workspace=ws, **rope)
    torch.cuda.synchronize()
    return dqkv, db, dqw, dkw


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,bias,rope", [(1, 8, 2, True, YARN), (7, 3, 3, False, PLAIN), (333, 64, 8, True, YARN),
                                                (2500, 10, 2, True, YARN), (8, 1, 1, False, YARN),
                                                (17, 300, 4, True, PLAIN)])
def test_backward(T, Hq, Hkv, bias, rope, interleaved):
    """Bounds: u is off by at most 2^-20 a (|dz_a| + |dz_b|) (as the forward's rotation), so an element of dy by
    2^-18 of E = r (max|w u| + max|n| mean|w u n|) over its head, plus 2^-8 for its rounding to bf16; a sum of
    T terms of an fp32 column by 2^-18 of the sum of E and (T + 64) 2^-24 of the sum of |dy|."""
    c = make(T, Hq, Hkv, 51 + T, bias)
    t = up(c)
    dqkv, db, dqw, dkw = run_bwd(t, rope, interleaved, bias)
    rx, rb, rqw, rkw = oracle.qk_norm_prologue_bwd(c["qkv"], c["bias"], c["qw"], c["kw"], c["pos"], c["dq"], c["dk"],
                                                   c["dv"], EPS, interleaved=interleaved, **oracle_rope(rope))
    y = c["qkv"].double().numpy()
    if bias:
        y = y + c["bias"].double().numpy()
    y = y.reshape(T, -1, D)[:, :Hq + Hkv]
    r = 1 / np.sqrt((y * y).mean(-1, keepdims=True) + EPS)
    n = np.abs(y * r)
    g = np.concatenate([c["dq"].double().numpy(), c["dk"].double().numpy()], 1)
    w = np.concatenate([np.broadcast_to(c[x].double().abs().numpy(), (h, D)) for x, h in (("qw", Hq), ("kw", Hkv))])
    u = 2 * 1.35 * np.abs(g).max(-1, keepdims=True)  # a bound on every |u| of the head
    E = r * (u * w.max(-1)[None, :, None] + n.max(-1, keepdims=True) * (u * w[None] * n).mean(-1, keepdims=True))
    E = np.concatenate([np.broadcast_to(E, (T, Hq + Hkv, D)), np.zeros((T, Hkv, D))], 1).reshape(T, -1)
    close(dqkv, rx, 2.0 ** -18 * E + 2.0 ** -8 * (np.abs(rx) + 2.0 ** -18 * E) + 1e-30, "dqkv")
    if bias:
        close(db, rb, 2.0 ** -18 * E.sum(0) + (T + 64) * 2.0 ** -24 * np.abs(rx).sum(0) + 1e-30, "dbias")
    un = np.broadcast_to(u, n.shape) * n
    for name, got, ref, sl, heads in (("dq_weight", dqw, rqw, slice(0, Hq), Hq),
                                      ("dk_weight", dkw, rkw, slice(Hq, Hq + Hkv), Hkv)):
        s = un[:, sl].sum((0, 1))
        close(got, ref, (2.0 ** -18 + (T * heads + 64) * 2.0 ** -24) * s + 1e-30, name)


@gpu
def test_backward_by_differences():
    """The forward's own outputs, moved along a direction of the weights: every q value is linear in them, so
    the difference of <q, dq> + <k, dk> over a step is the gradient times the step, up to the roundings of the
    outputs to bf16 (2^-8 of each |q dq|, at both ends)."""
    T, Hq, Hkv = 64, 8, 2
    c = make(T, Hq, Hkv, 61)
    t = up(c)
    _, _, dqw, dkw = run_bwd(t, YARN, False)
    step = torch.randn(D, generator=torch.Generator().manual_seed(6)).cuda()
    for name, dw, grad, which in (("qw", dqw, t["dq"], 0), ("kw", dkw, t["dk"], 1)):
        vals, slack = [], 0.0
        for s in (1.0, -1.0):
            w = {**t, name: t[name] + s * step}
            q = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
            k, v = (torch.empty(T, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
            attn.attn_sink_qk_norm_prologue(w["qkv"], w["bias"], w["qw"], w["kw"], w["pos"], q, k, v, EPS, **YARN)
            z = (q, k)[which].double() * grad.double()
            vals.append(float(z.sum()))
            slack += float(z.abs().sum()) * 2.0 ** -8
        assert abs((vals[0] - vals[1]) / 2 - float((dw.double() * step.double()).sum())) <= slack / 2 * 1.01


@gpu
def test_backward_repeats_streams_and_graphs():
    """Twice, on a side stream and captured: the same bits; without dbias the rest is unchanged."""
    c = make(1000, 16, 2, 71)
    t = up(c)
    a = run_bwd(t, YARN, False)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = run_bwd(t, YARN, False)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    no = run_bwd(t, YARN, False, bias=False)
    assert torch.equal(no[0], a[0]) and torch.equal(no[2], a[2]) and torch.equal(no[3], a[3])
    outs = [torch.empty_like(x) for x in a]
    ws = torch.empty(attn.attn_sink_qk_norm_prologue_bwd_workspace_size(1000, 16, 2, D), dtype=torch.uint8,
                     device="cuda")
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        attn.attn_sink_qk_norm_prologue_bwd(t["qkv"], t["bias"], t["qw"], t["kw"], t["pos"], t["dq"], t["dk"], t["dv"],
                                            *outs, EPS, workspace=ws, **YARN)
    for _ in range(3):
        gr.replay()
    torch.cuda.synchronize()
    for x, y in zip(a, outs):
        assert torch.equal(x, y)
