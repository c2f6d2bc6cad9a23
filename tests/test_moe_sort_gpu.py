"""The sort of tokens by expert in its forms for more pairs: one launch in which
every CTA counts all ids (up to 16,384 pairs and 48 MB of rows), and above that
the places by one cluster with the rows' launch behind it."""
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


@pytest.mark.parametrize("E", [1, 31, 33, 63, 65, 1023])
def test_places_of_any_number_of_experts(E):
    """The cluster's loops over the experts end at different trips within a
    warp where their number is no multiple of 32."""
    M, H, topk = 9001, 16, 2
    rng = np.random.default_rng(E)
    x, ids = P.make_rows(rng, M, H), rng.integers(-1, E + 1, (M, topk)).astype(np.int32)
    offsets, dest = P.sort(ids, E)
    tx, tids = cu(x), cu(ids)
    for _ in range(5):
        xs, got_offsets, got_dest = B.moe_sort(tx, tids, E)
        assert np.array_equal(got_offsets.cpu().numpy(), offsets)
        assert np.array_equal(got_dest.cpu().numpy(), dest)
        live = int(offsets[-1])
        want = P.sorted_rows(x, dest, np.zeros((M * topk, H), np.float16))
        assert np.array_equal(xs.cpu().numpy()[:live].view(np.uint16), want[:live].view(np.uint16))


# Sizes that take each form: (tokens, choices, H)
FORMS = {
    "few pairs": (900, 4, 1024),
    "every CTA counts": (3000, 4, 512),
    "cluster, by pairs": (6000, 4, 256),
    "cluster, by bytes": (2700, 2, 5120),
}
E_BEHIND = 40


def chain(M, topk, H, y, back, ids0, rows, x, steps):
    """Sorts, each right behind kernels that write its x and its ids and let it
    begin before they end: a combine of eight rows per token into x, and a sort
    whose places are the ids (most of them name no expert)."""
    results = []
    for i in range(steps):
        B.moe_combine(y[i], back[i], out=x)
        ids = B.moe_sort(rows, ids0[i], 3)[2]
        results.append(B.moe_sort(x, ids, E_BEHIND if i % 2 else 1024))
    return results


def chain_inputs(form, steps):
    M, topk, H = FORMS[form]
    rng = np.random.default_rng([M, H])
    y = [cu(P.make_rows(rng, 8 * M, H)) for _ in range(steps)]
    back = [cu(rng.permutation(8 * M).reshape(M, 8).astype(np.int32)) for _ in range(steps)]
    ids0 = [cu(rng.integers(0, 3, (M, topk)).astype(np.int32)) for _ in range(steps)]
    rows = cu(P.make_rows(rng, M, 8))
    x = torch.zeros((M, H), dtype=torch.float16, device="cuda")
    return M, topk, H, y, back, ids0, rows, x, steps


def chain_one_by_one(args):
    """The same with the device idle before every call."""
    *_, y, back, ids0, rows, x, steps = args
    results = []
    for i in range(steps):
        at = torch.empty_like(x)
        B.moe_combine(y[i], back[i], out=at)
        torch.cuda.synchronize()
        ids = B.moe_sort(rows, ids0[i], 3)[2]
        torch.cuda.synchronize()
        E = E_BEHIND if i % 2 else 1024
        results.append(B.moe_sort(at, ids, E))
        torch.cuda.synchronize()
        offsets, dest = P.sort(ids.cpu().numpy(), E)
        assert np.array_equal(results[-1][1].cpu().numpy(), offsets)
        assert np.array_equal(results[-1][2].cpu().numpy(), dest)
    return results


def same_live_rows(got, want):
    live = int(want[1][-1])
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    assert live > 0 and torch.equal(got[0][:live], want[0][:live])


@pytest.mark.parametrize("form", FORMS)
def test_sort_behind_unfinished_writers(form):
    args = chain_inputs(form, 6)
    want = chain_one_by_one(args)
    for _ in range(3):
        args[7].zero_()
        torch.cuda.synchronize()
        for got, ref in zip(chain(*args), want):
            same_live_rows(got, ref)


@pytest.mark.parametrize("form", FORMS)
def test_captured_sort_behind_unfinished_writers(form):
    args = chain_inputs(form, 4)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        chain(*args)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = chain(*args)
    rng = np.random.default_rng(1)
    for _ in range(3):
        for y, ids in zip(args[3], args[5]):  # new rows and new routings for every replay
            y.copy_(y.roll(1, 0))
            ids.copy_(cu(rng.integers(0, 3, tuple(ids.shape)).astype(np.int32)))
        graph.replay()
        torch.cuda.synchronize()
        got = [tuple(t.clone() for t in r) for r in captured]
        for a, b in zip(got, chain_one_by_one(args)):
            same_live_rows(a, b)


@pytest.mark.parametrize("form", FORMS)
def test_sort_behind_copies(form):
    """x and ids rewritten by copies directly before each sort."""
    M, topk, H = FORMS[form]
    rng = np.random.default_rng(M)
    sets = [(P.make_rows(rng, M, H), P.make_ids(rng, M, E_BEHIND, topk, 0.1)) for _ in range(4)]
    dev = [(cu(a), cu(b)) for a, b in sets]
    x, ids = (torch.empty_like(t) for t in dev[0])
    got = []
    for a, b in dev * 2:
        x.copy_(a)
        ids.copy_(b)
        got.append(B.moe_sort(x, ids, E_BEHIND))
    for (a, b), (xs, offsets, dest) in zip(sets * 2, got):
        want_offsets, want_dest = P.sort(b, E_BEHIND)
        assert np.array_equal(offsets.cpu().numpy(), want_offsets)
        assert np.array_equal(dest.cpu().numpy(), want_dest)
        live = int(want_offsets[-1])
        order = np.argsort(np.where(want_dest < 0, M * topk, want_dest).reshape(-1), kind="stable")
        assert np.array_equal(xs[:live].cpu().numpy().view(np.uint16),
                              a[order[:live] // topk].view(np.uint16))
