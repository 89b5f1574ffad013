"""attn_sink_decode_tree where a team of CTAs has a part of the KV heads, and over pages that are no power of two."""
import pytest
import torch

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
