"""The mixture-of-experts operators with stream=: which stream's memory a call
allocates, and how long the tensors of a call are kept from reuse."""
import numpy as np
import pytest
import torch

import moe_plain as P
from int4_weight_only_gptq_b200 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from int4_weight_only_gptq_b200.build import build
    build()
    B.load()
    assert B.device_error() == 0
    yield
    assert B.device_error() == 0


def cu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def layer_on(stream, x, ids, w, q, s, E, G):
    """Every operator with stream= and its own outputs."""
    xs, offsets, dest = B.moe_sort(x, ids, E, stream=stream)
    y = B.gemm_experts(xs, q, s, offsets, G, stream=stream)
    out = B.moe_combine(y, dest, w, stream=stream)
    dy, dw = B.moe_combine_backward(out, y, dest, w, stream=stream)
    dx = B.gemm_experts_dx(dy, q, s, offsets, G, stream=stream)
    return xs, offsets, dest, y, out, dy, dw, dx


def layer_inputs(seed, M=300, E=6, K=512, N=512, G=64):
    rng = np.random.default_rng(seed)
    q, s = (cu(a) for a in P.make_weights(rng, E, K, N, G))
    x, ids = cu(P.make_rows(rng, M, K)), cu(P.make_ids(rng, M, E, 2))
    return x, ids, torch.rand((M, 2), device="cuda"), q, s, E, G


def span(t):
    return t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()


def test_a_raw_handle_takes_no_memory_that_the_callers_stream_still_uses():
    args = layer_inputs(21)
    want = layer_on(None, *args)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    freed = [torch.empty_like(t) for t in want for _ in range(3)]
    spans = [span(t) for t in freed]
    del freed
    got = layer_on(side.cuda_stream, *args)
    for t in got:
        lo, hi = span(t)
        assert all(hi <= a or lo >= b for a, b in spans)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("handle", [0, 1])
def test_the_legacy_default_stream_by_its_handles(handle):
    args = layer_inputs(22)
    want = layer_on(None, *args)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = layer_on(handle, *args)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("raw", [False, True])
def test_inputs_are_kept_until_the_other_stream_is_done(raw):
    """A caller may drop an input right after a call on another stream."""
    rng = np.random.default_rng(23)
    M, H, topk, E = 2048, 4096, 2, 4
    ids = P.make_ids(rng, M, E, topk)
    dest = cu(P.sort(ids, E)[1])
    rows = cu(P.make_rows(rng, M * topk, H))
    want = B.moe_combine(rows, dest)
    side, out = torch.cuda.Stream(), torch.empty_like(want)
    y, spare = rows.clone(), torch.empty_like(rows)
    torch.cuda.synchronize()
    del spare  # the only free block of y's size, so that the first of two takes it
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)  # about 50 ms
    got = B.moe_combine(y, dest, out=out, stream=side.cuda_stream if raw else side)
    lo = y.data_ptr()
    del y
    busy = not side.query()
    others = [torch.empty_like(rows) for _ in range(2)]
    assert busy, "the side stream had finished too early to show anything"
    assert all(t.data_ptr() != lo for t in others)
    for t in others:
        t.fill_(float("nan"))
    torch.cuda.synchronize()
    assert got is out and torch.equal(got, want)


def test_the_current_stream_by_name_or_handle_is_no_other_stream():
    args = layer_inputs(24)
    want = layer_on(None, *args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for stream in (side, side.cuda_stream):
            for a, b in zip(layer_on(stream, *args), want):
                assert torch.equal(a, b)
    torch.cuda.synchronize()


def test_captured_on_a_forked_raw_handle():
    args = layer_inputs(25, M=40)
    want = layer_on(None, *args)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = layer_on(side.cuda_stream, *args)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
