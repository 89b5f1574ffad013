"""attn_sink_decode_tree where a team of CTAs has a part of the KV heads, over pages that are no power of two, and
beside the prefill's last rows."""
import numpy as np
import pytest
import torch

import gqa_softmax_attention_attn_b200 as attn
import oracle
from test_tree_decode import check, make_case, run

pytestmark = pytest.mark.gpu


# 64 query and 8 KV heads: 128 tokens are 8 row tiles, of which the GPU holds 9 teams with 4 of the KV heads each,
# 200 tokens 13 row tiles and 11 teams with 2 heads; (6, 6) heads and 256 tokens two row tiles and all heads in a team
@pytest.mark.parametrize("window", [0, 50, 600])  # (50: at most six tiles a sequence, which are never cut)
@pytest.mark.parametrize("splits", [0, 3, 17])
@pytest.mark.parametrize("Hq,Hkv,max_q", [(64, 8, 128), (64, 8, 200), (6, 6, 256)])
def test_groups_of_kv_heads(Hq, Hkv, max_q, splits, window):
    c = make_case([300, 0, 61, 700], [40, max_q, 0, 3], Hq, Hkv, torch.bfloat16, seed=31, pad_rows=1)
    check(c, run(c, window, 0, splits), window)


@pytest.mark.parametrize("page_size", [16, 192])
def test_groups_of_kv_heads_paged(page_size):
    """The draft of one sequence is as long as the bound, the others' are shorter; and a bound above all of them."""
    c = make_case([250, 1000, 0, 5], [6, 128, 0, 30], 64, 8, torch.bfloat16, seed=32)
    check(c, run(c, 0, page_size), 0)
    c = make_case([250, 1000, 0, 5], [6, 9, 0, 30], 64, 8, torch.bfloat16, seed=33)
    for bound in (40, 200, 256):
        loose = dict(c, max_q=bound)
        check(loose, run(loose, 0, page_size), 0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("page_size", [192, 320, 1024])
@pytest.mark.parametrize("window", [0, 60, 250])
def test_pages_of_odd_multiples(page_size, window, dtype):
    c = make_case([0, 257, 31, 640, 959], [4, 11, 1, 33, 2], 8, 2, dtype, seed=34, pad_rows=1)
    got = run(c, window, page_size)
    check(c, got, window)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("window", [0, 100])
@pytest.mark.parametrize("L,T", [(300, 7), (65, 64), (130, 130)])
def test_a_chain_is_the_prefill(L, T, window, dtype):
    """A chain of T tokens over L - T cached keys: attn_sink_fwd of the same T rows over all L keys.  Each is off by
    at most the bound of `check` from the definition; the prefill's probabilities by 2^-13 more each, numerator and
    denominator (a quarter of its exponentials is a polynomial, 7.5e-5 off)."""
    Hq, Hkv, scale = 16, 2, 0.125
    c = make_case([L - T], [T], Hq, Hkv, dtype, "chain", seed=35)
    got = run(c, window)
    check(c, got, window)
    q, k, v, sinks = (c[x].cuda() for x in ("q", "k", "v", "sinks"))
    out, lse = torch.empty_like(q[None]), torch.empty(1, Hq, T, device="cuda")
    attn.attn_sink_fwd(q[None].contiguous(), k, v, sinks, out, lse, window, scale)
    torch.cuda.synchronize()
    out, lse = out[0].cpu().double().numpy(), lse[0].T.cpu().double().numpy()
    ro, rl = oracle.fwd(c["q"][None], c["k"], c["v"], c["sinks"], window, scale)
    ra, _ = oracle.fwd(c["q"][None], c["k"], c["v"].abs(), c["sinks"], window, scale)
    ro, ra, rl = ro[0], ra[0], rl[0].T
    qk = torch.einsum("thd,jhd->thj", c["q"].double().abs(), c["k"][0].double().abs().repeat_interleave(Hq // Hkv, 1))
    e = 2.0 ** -17 * scale * float(qk.max()) + 2.0 ** -20 + L * 2.0 ** -24
    tree, fwd = e * ra + 1e-30, (e + 2.0 ** -12) * ra + 1e-30
    if dtype == torch.bfloat16:
        tree, fwd = ((t + 2.0 ** -8 * ra) * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ro) for t in (tree, fwd))
    d = np.abs(got[0].double().numpy() - out)
    assert (d <= tree + fwd).all(), f"out: worst {(d / (tree + fwd)).max():.3f} of the bound"
    dl = np.abs(got[1].double().numpy() - lse)
    assert (dl <= 2 * e + 2.0 ** -12 + 2.0 ** -20 * (1 + np.abs(rl))).all(), f"lse: {dl.max():.3e}"
