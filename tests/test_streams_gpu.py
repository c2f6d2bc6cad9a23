"""The layer's entries with stream=: what a call allocates on another stream is
that stream's memory, and the tensors of the call are kept until it is done."""
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


def calls(M, K=512, N=512, G=64, rank=32):
    """Every entry of a layer, by name: a call of (stream) with its own outputs."""
    rng = np.random.default_rng(M)
    q, s = (cu(a[0]) for a in P.make_weights(rng, 1, K, N, G))
    x, a, b = (cu(P.make_rows(rng, r, c)) for r, c in ((M, K), (rank, K), (N, rank)))
    zeros = cu(rng.integers(-2 ** 31, 2 ** 31, (K // G, N // 8)).astype(np.int32))
    g_idx = cu(rng.integers(0, K // G, K).astype(np.int32))
    return {
        "gemm": lambda st: B.gemm(x, q, s, G, stream=st),
        "gemm_grouped": lambda st: B.gemm_grouped(x, [q, q], [s, s], G, stream=st),
        "gemm_asym": lambda st: B.gemm_asym(x, q, s, zeros, G, stream=st),
        "gemm_gidx": lambda st: B.gemm_gidx(x, q, s, g_idx, stream=st),
        "gemm_lora": lambda st: B.gemm_lora(x, q, s, G, a, b, stream=st),
        "gemm_lora_noalloc": lambda st: B.gemm_lora_noalloc(x, q, s, G, a, b, stream=st),
        "dequant": lambda st: B.dequant(q, s, G, stream=st),
    }


@pytest.mark.parametrize("name", ["gemm", "gemm_grouped", "gemm_asym", "gemm_gidx", "gemm_lora",
                                  "gemm_lora_noalloc", "dequant"])
@pytest.mark.parametrize("M", [3, 200])
@pytest.mark.parametrize("raw", [False, True])
def test_what_a_call_allocates_is_its_streams_memory(name, M, raw, monkeypatch):
    call = calls(M)[name]
    want = call(None)
    side, seen = torch.cuda.Stream(), []
    torch.cuda.synchronize()
    empty = torch.empty

    def spy(*args, **kw):  # outputs and work tensors alike
        seen.append(torch.cuda.current_stream().cuda_stream)
        return empty(*args, **kw)

    monkeypatch.setattr(torch, "empty", spy)
    got = call(side.cuda_stream if raw else side)
    monkeypatch.undo()
    assert seen and all(s == side.cuda_stream for s in seen)
    torch.cuda.synchronize()
    for a, b in zip(B._tensors([got]), B._tensors([want])):
        assert torch.equal(a, b)


@pytest.mark.parametrize("raw", [False, True])
def test_inputs_are_kept_until_the_other_stream_is_done(raw):
    """Those in lists too."""
    rng = np.random.default_rng(7)
    K, N, G, M = 4096, 4096, 128, 2
    q, s = (cu(a[0]) for a in P.make_weights(rng, 1, K, N, G))
    x = cu(P.make_rows(rng, M, K))
    want = B.gemm(x, q, s, G)
    side, out = torch.cuda.Stream(), torch.empty_like(want)
    copy, spare = q.clone(), torch.empty_like(q)
    torch.cuda.synchronize()
    del spare  # the only free block of this size, so that the first of two takes it
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)  # about 50 ms
    B.gemm_grouped(x, [copy], [s], G, outs=[out], stream=side.cuda_stream if raw else side)
    lo = copy.data_ptr()
    del copy
    busy = not side.query()
    others = [torch.empty_like(q) for _ in range(2)]
    assert busy, "the side stream had finished too early to show anything"
    assert all(t.data_ptr() != lo for t in others)
    for t in others:
        t.zero_()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
