"""The experts' products where their kernels' own paths differ: the short form
of the dequantisation against every scale that takes it, and walks over many
token tiles, in which rings and accumulators come round again and again."""
import numpy as np
import pytest
import torch

import moe_plain as P
import oracle
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
    a = np.ascontiguousarray(a)
    if a.dtype == np.float16:
        return torch.from_numpy(a.view(np.int16)).view(torch.float16).cuda()
    return torch.from_numpy(a).cuda()


def bits(a):
    return np.ascontiguousarray(a).view(np.uint16)


def scale_bits(rng, shape):
    """Scales of each kind, as FP16 bits; the short form takes a stage of a
    warp's 32 columns if all their scales have bits 0x0001 .. 0x27FF."""
    normal = rng.uniform(1e-3, 2e-2, shape).astype(np.float16).view(np.uint16)
    one_above = normal.copy()
    # one scale in a column of the first warp and the first group
    one_above[0, 5] = 0x2800
    return [
        rng.integers(0x0001, 0x0400, shape),  # subnormal
        rng.integers(0x03F0, 0x0420, shape),  # about the smallest normal one
        rng.integers(0x0001, 0x2800, shape),  # everything in the range
        np.full(shape, 0x27FF), np.full(shape, 0x2800),  # the border, from both sides
        normal, one_above,
        np.where(rng.random(shape) < 0.01, rng.choice([0x0000, 0x8000, 0xA000, 0x3C00], shape),
                 normal),             # some warps take one form, some the other
    ]


KERNELS = {
    "decode 16": dict(kernel=B.KERNEL_DECODE, tile=16),
    "decode 32": dict(kernel=B.KERNEL_DECODE, tile=32),
    "pairs": dict(kernel=B.KERNEL_PREFILL),
}


@pytest.mark.parametrize("G", [16, 32, 64, 128, -1])
@pytest.mark.parametrize("kernel,N", [("decode 16", 264), ("decode 32", 264), ("pairs", 264),
                                      ("pairs", 1416)])  # the last: tiles of 256 rows
def test_ordinary_scales_reproduce_weights(G, kernel, N):
    """Every weight of every expert, bit for bit: each expert's rows are the
    rows of a unit matrix, and each expert has scales of another kind."""
    K = 272  # a whole stage of 256 k and a part
    rng = np.random.default_rng(G + N)
    n_groups = 1 if G == -1 else -(-K // G)
    s = np.stack(scale_bits(rng, (n_groups, N))).astype(np.uint16).view(np.float16)
    E = len(s)
    q, _ = P.make_weights(rng, E, K, N, G)
    # K rows of each expert, more than 256: with six column pairs there is a tile
    # for every cluster, and the pair kernel takes tiles of 256 rows
    x = np.tile(np.eye(K, dtype=np.float16), (E, 1))
    got = B.gemm_experts(cu(x), cu(q), cu(s), cu(P.offsets_of([K] * E)), G,
                         **KERNELS[kernel]).cpu().numpy().reshape(E, K, N)
    for e in range(E):
        want = oracle.dequant(q[e], s[e], G)
        # a sum with zeros has no negative zero
        same = bits(got[e] + np.float16(0)) == bits(want + np.float16(0))
        assert same.all(), f"scales of kind {e}: {np.argwhere(~same)[:4].tolist()}"


def sampled(got, rows, q, s, offsets, G, gradient, picks):
    """Some rows against the oracle's weights."""
    expert = np.searchsorted(offsets, picks, side="right") - 1
    for r, e in zip(picks, expert):
        w = oracle.dequant(q[e], s[e], G).astype(np.float64)
        w = w.T if gradient else w
        x = rows[r].astype(np.float64)
        ref, size = x @ w, np.abs(x) @ np.abs(w)
        err = np.abs(got[r].cpu().numpy().astype(np.float64) - ref)
        tol = P.product_tol(ref, size, w.shape[0])
        assert (err <= tol).all(), f"row {r} of expert {e}: {(err - tol).max()} over the bound"


MIXED = [300, 1, 1500, 40, 129, 128, 513, 64, 2, 260, 700, 33]  # 306 on average
NARROW = [40, 1, 128, 129, 300, 200, 96, 0, 257, 31, 64, 8]     # 105 on average


@pytest.mark.parametrize("counts", [MIXED, NARROW], ids=["tiles of 256", "tiles of 128"])
@pytest.mark.parametrize("gradient", [False, True], ids=["y", "dx"])
@pytest.mark.parametrize("C,G", [(400, 64), (136 * 2, 16)])
def test_long_walks_over_mixed_tiles(counts, gradient, C, G):
    """Six and more tiles per cluster, wide ones and narrow ones in turn: both
    accumulators' hand-over, and the change between halves and the whole."""
    O = 9616  # 38 column pairs
    K, N = (O, C) if gradient else (C, O)
    rng = np.random.default_rng([C, len(counts), gradient])
    offsets = P.offsets_of(counts)
    q, s = P.make_weights(rng, len(counts), K, N, G)
    rows = P.make_rows(rng, int(offsets[-1]), C)
    args = (cu(rows), cu(q), cu(s), cu(offsets), G)
    run = (lambda: B.gemm_experts_dx(*args)) if gradient else (
        lambda: B.gemm_experts(*args, kernel=B.KERNEL_PREFILL))
    first = run()
    for _ in range(15):
        assert torch.equal(run(), first)
    edges = np.concatenate([offsets[:-1], offsets[1:] - 1, offsets[:-1] + 127, offsets[:-1] + 128])
    picks = np.unique(np.concatenate([edges[edges < offsets[-1]],
                                      rng.choice(len(rows), 12, replace=False)]))
    sampled(first, rows, q, s, offsets, G, gradient, picks)


@pytest.mark.parametrize("counts,O,gradient", [
    ([1] * 1024, 5120, False),               # tiles of 128 rows, 20,480 of them
    ([2, 0, 1, 1] * 256, 6928, True),        # (K is the output's width)
    ([257] * 8, 310000, False),              # tiles of 256 rows, 19,376
], ids=["128-y", "128-dx", "256-y"])
def test_more_tiles_than_a_cluster_lists(counts, O, gradient):
    """A cluster looks up its first 256 tiles once and the others one by one.
    Small whole numbers and scales that are powers of two: every sum is exact
    in FP32, and the whole output is compared."""
    C = 16
    E = len(counts)
    K, N = (O, C) if gradient else (C, O)
    gen = torch.Generator(device="cuda").manual_seed(O)
    q = torch.randint(-2 ** 31, 2 ** 31, (E, K // 8, N), generator=gen, device="cuda",
                      dtype=torch.int32)
    s = (2.0 ** torch.randint(-4, 1, (E, 1, N), generator=gen, device="cuda")).half()
    rows = torch.randint(-3, 4, (sum(counts), C), generator=gen, device="cuda").half()
    offsets = cu(P.offsets_of(counts))
    tiles = sum(-(-c // 128) if len(counts) > 8 else -(-c // 256) for c in counts)
    assert tiles * -(-O // 256) > 256 * 74
    got = (B.gemm_experts_dx(rows, q, s, offsets, -1) if gradient
           else B.gemm_experts(rows, q, s, offsets, -1, kernel=B.KERNEL_PREFILL))
    shifts = torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)
    lo = 0
    for e, c in enumerate(counts):
        # sums of at most 16 products of at most 3 * 8, in steps of 1/16, then
        # one rounding
        w = (((q[e, :, None, :] >> shifts[None, :, None]) & 15) - 8).reshape(K, N).float()
        w = w * s[e].float()
        want = (rows[lo:lo + c].float() @ (w.T if gradient else w)).half()
        assert torch.equal(got[lo:lo + c], want), f"expert {e}"
        lo += c
