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
