"""The tree, page map and QK-norm calls captured behind nodes that are no kernels (a fill, a copy), behind two
streams that join, as the first node of a graph, and on a stream of their own beside the capturing one: every call
launches its kernels as dependents of the node ahead, whatever that is."""
import pytest
import torch

import gqa_softmax_attention_attn_b200 as attn
from test_qk_norm import EPS, YARN, make, up
from test_tree_decode import D, make_case

pytestmark = pytest.mark.gpu


def tree_call(dtype, num_splits=0, window=0):
    c = make_case([900, 333, 20], [8, 3, 8], 8, 2, dtype, seed=41)
    t = {x: c[x].cuda() for x in ("q", "k", "v", "cu", "parents", "lens", "sinks")}
    code = attn.DTYPE_F32 if dtype == torch.float32 else attn.DTYPE_BF16
    n = attn.attn_sink_decode_tree_workspace_size(3, 19, 8, 8, 2, D, t["k"].shape[1], window, num_splits, code)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    outs = (torch.empty_like(t["q"]), torch.empty(19, 8, device="cuda"))
    return t["q"], outs, lambda: attn.attn_sink_decode_tree(t["q"], t["k"], t["v"], t["cu"], t["parents"], t["lens"],
                                                            t["sinks"], *outs, 8, window, 0.125, num_splits, ws)


def map_call():
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    new, cached, free = i32([4, 0, 9]), i32([5, 8, 0]), i32(list(range(20, 40)))
    tab = i32([[0, 1, 2, 3]] * 3)
    outs = tuple(torch.empty(n, dtype=torch.int32, device="cuda") for n in (3, 4, 20, 20, 4))
    return new, outs, lambda: attn.attn_sink_page_map(cached, new, free, tab, *outs, 8, 64)


def norm_call():
    t = up(make(77, 8, 2, 42))
    outs = tuple(torch.empty(77, h, D, dtype=torch.bfloat16, device="cuda") for h in (8, 2, 2))
    return t["qkv"], outs, lambda: attn.attn_sink_qk_norm_prologue(t["qkv"], t["bias"], t["qw"], t["kw"], t["pos"],
                                                                   *outs, EPS, **YARN)


def norm_bwd_call():
    t = up(make(77, 8, 2, 43))
    outs = (torch.empty_like(t["qkv"]), torch.empty_like(t["bias"]), torch.empty_like(t["qw"]), torch.empty_like(t["kw"]))
    ws = torch.empty(attn.attn_sink_qk_norm_prologue_bwd_workspace_size(77, 8, 2, D), dtype=torch.uint8, device="cuda")
    return t["qkv"], outs, lambda: attn.attn_sink_qk_norm_prologue_bwd(
        t["qkv"], t["bias"], t["qw"], t["kw"], t["pos"], t["dq"], t["dk"], t["dv"], *outs, EPS, workspace=ws, **YARN)


CALLS = {
    "tree": lambda: tree_call(torch.bfloat16), "tree cut": lambda: tree_call(torch.bfloat16, 5),
    "tree banded": lambda: tree_call(torch.bfloat16, 0, 50), "tree fp32": lambda: tree_call(torch.float32, 5),
    "page map": map_call, "norm": norm_call, "norm backward": norm_bwd_call,
}


@pytest.mark.parametrize("name", CALLS)
def test_behind_any_node(name):
    src, outs, call = CALLS[name]()
    call()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    keep, pinned = src.clone(), src.cpu().pin_memory()
    other = torch.empty(1 << 22, device="cuda")  # something that takes its time on the second stream
    side = torch.cuda.Stream()

    def first():
        call()

    def fill():
        for o in outs:
            o.zero_()
        call()

    def copy():  # the input arrives by a copy node
        src.copy_(keep)
        call()

    def copy_from_host():
        src.copy_(pinned, non_blocking=True)
        call()

    def joined():  # the input is copied on one stream, a kernel runs on the other; the call waits for both
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            src.copy_(keep)
            src.add_(0)
        other.normal_()
        here.wait_stream(side)
        call()

    def forked():  # the call on the second stream, behind a join of its own
        here = torch.cuda.current_stream()
        src.copy_(keep)
        side.wait_stream(here)
        other.zero_()
        with torch.cuda.stream(side):
            call()
        here.wait_stream(side)
        other.add_(1)

    for how in (first, fill, copy, copy_from_host, joined, forked):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            how()
        for _ in range(3):
            for o in outs:
                o.fill_(7)
            if how not in (first, fill):
                src.zero_()
            graph.replay()
            torch.cuda.synchronize()
            for o, w in zip(outs, want):
                assert torch.equal(o, w), how.__name__
    assert attn.attn_sink_get_device_status() == 0


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("name", CALLS)
def test_between_two_calls_another_stream_writes(name, captured):
    """A call whose kernels let the next one in early, then a wait for another stream, whose copy of the input comes
    late, then the call again: the second reads what the other stream wrote."""
    src, outs, call = CALLS[name]()
    call()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    keep = src.clone()
    side = torch.cuda.Stream()

    def line():
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        call()  # on an input of zeros
        ready = torch.cuda.Event()
        ready.record()
        with torch.cuda.stream(side):
            side.wait_event(ready)  # (the first call reads the input)
            torch.cuda._sleep(400000)  # some 200 us
            src.copy_(keep)
        call()  # and once more, while the other stream sleeps
        for o in outs:
            o.fill_(7)
        call()
        here.wait_stream(side)
        call()

    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            line()
    for _ in range(5):
        src.zero_()
        torch.cuda.synchronize()
        graph.replay() if captured else line()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
    assert attn.attn_sink_get_device_status() == 0
