"""The mixture-of-experts operators on the GPU against their definitions in 64
bits (moe_plain): tokens sorted by expert, combine and its gradients, the
experts' INT4 products and the gradient of their rows, alone and as the run of
a layer, forward and backward.

Bars: whole numbers and copied rows exactly; sums within the rounding of the
FP32 additions and the one rounding to FP16 (the bounds in moe_plain); bitwise
where the definition leaves no freedom (one-hot rows reproduce weights, w *
dout is one product and one rounding).  Outputs lie between guard bands, and
rows that belong to no expert must keep their bytes.
"""
import ctypes

import numpy as np
import pytest
import torch

import moe_plain as P
import oracle
from int4_weight_only_gptq_b200 import binding as B

pytestmark = pytest.mark.gpu
GUARD = 4096
ERR_INDEX = 10


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


class Guarded:
    """A [rows, cols] FP16 tensor of random bytes inside guard bands."""

    def __init__(self, rows, cols, seed=0):
        self.n = rows * cols * 2
        self.bytes = np.random.default_rng(seed).integers(0, 256, 2 * GUARD + self.n,
                                                          dtype=np.uint8)
        self.buf = torch.from_numpy(self.bytes.copy()).cuda()
        self.t = self.buf[GUARD:GUARD + self.n].view(torch.float16).view(rows, cols)
        self.shape = (rows, cols)

    def before(self):
        return self.bytes[GUARD:GUARD + self.n].view(np.float16).reshape(self.shape)

    def after(self):
        torch.cuda.synchronize()
        got = self.buf.cpu().numpy()
        assert np.array_equal(got[:GUARD], self.bytes[:GUARD]), "write before the output"
        assert np.array_equal(got[GUARD + self.n:], self.bytes[GUARD + self.n:]), \
            "write past the output"
        return got[GUARD:GUARD + self.n].view(np.float16).reshape(self.shape)


def bits(a):
    return np.ascontiguousarray(a).view(np.uint16)


def within(got, ref, tol, label):
    over = np.abs(got.astype(np.float64) - ref) - tol
    assert not np.isnan(got).any(), label
    assert over.max(initial=-1.0) <= 0, f"{label}: {over.max()} over the bound"
    used = np.max(np.abs(got.astype(np.float64) - ref) / np.maximum(tol, 1e-30), initial=0.0)
    print(f"[moe] {label}: {used:.3f} of the bound")


# ---- sort ----------------------------------------------------------------------

SORT = [  # (tokens, H, topk, E, drop)
    (1, 8, 1, 1, 0.0), (1, 2048, 8, 64, 0.0), (3, 72, 2, 5, 0.3), (37, 1048, 3, 12, 0.1),
    (512, 264, 8, 128, 0.0),      # as many pairs as the one-launch form for few takes
    (513, 264, 8, 128, 0.2),      # one more token: every CTA counts all ids
    (4096, 40, 4, 32, 0.1),       # as many pairs as that takes
    (4097, 40, 4, 33, 0.1),       # one more token: the cluster
    # more bytes than it takes, and fewer; each CTA's tokens in one step and more
    (8192, 1032, 2, 8, 0.5), (2500, 520, 5, 300, 0.3), (5000, 512, 3, 1000, 0.2),
    (2700, 5120, 2, 8, 0.3), (2100, 8200, 2, 3, 0.1), (1400, 12288, 4, 6, 0.6),
    (1200, 20000, 4, 5, 0.2), (300, 24584, 16, 20, 0.5), (9000, 1040, 1, 3, 1.0),
    (1500, 1024, 6, 1024, 0.5),   # the most experts
    (4099, 1032, 2, 8, 0.05), (70, 16, 64, 200, 0.0), (300, 40, 33, 100, 0.4),
    (5000, 8, 1, 3, 1.0),         # every pair dropped
    (9, 2056, 4, 4, 1.0),
]


@pytest.mark.parametrize("M,H,topk,E,drop", SORT)
@pytest.mark.parametrize("wide", [False, True])
def test_sort(M, H, topk, E, drop, wide):
    rng = np.random.default_rng([M, H, topk, E])
    x = P.make_rows(rng, M, H)
    ids = P.make_ids(rng, M, E, topk, drop)
    # what names no expert is dropped, whatever its value
    ids[ids < 0] = rng.choice([-1, -7, E, E + 5, 2 ** 31 - 1, -2 ** 31], size=(ids < 0).sum())
    dev_ids = ids.astype(np.int64) if wide else ids
    if wide and drop:
        dev_ids[(ids < 0) | (ids >= E)] += 2 ** 32 * E  # not an expert in 64 bits either
    offsets, dest = P.sort(ids, E)
    out = Guarded(M * topk, H, seed=M)
    _, got_offsets, got_dest = B.moe_sort(cu(x), cu(dev_ids), E, out=out.t)
    assert got_offsets.cpu().numpy().tolist() == offsets.tolist()
    assert np.array_equal(got_dest.cpu().numpy(), dest)
    assert np.array_equal(bits(out.after()), bits(P.sorted_rows(x, dest, out.before())))


@pytest.mark.parametrize("M", [6, 3000])
def test_sort_repeated_expert_of_a_token(M):
    rng = np.random.default_rng(M)
    x, ids = P.make_rows(rng, M, 24), rng.integers(0, 3, (M, 4)).astype(np.int32)
    offsets, dest = P.sort(ids, 3)
    xs, got_offsets, got_dest = B.moe_sort(cu(x), cu(ids), 3)
    assert got_offsets.cpu().numpy().tolist() == offsets.tolist()
    assert np.array_equal(got_dest.cpu().numpy(), dest)
    assert np.array_equal(bits(xs.cpu().numpy()), bits(P.sorted_rows(x, dest, np.zeros(xs.shape, np.float16))))


def test_sort_no_tokens():
    x = torch.empty((0, 64), dtype=torch.float16, device="cuda")
    xs, offsets, dest = B.moe_sort(x, torch.empty((0, 4), dtype=torch.int32, device="cuda"), 9)
    assert xs.shape == (0, 64) and dest.shape == (0, 4)
    assert offsets.cpu().tolist() == [0] * 10


# ---- combine -------------------------------------------------------------------

COMBINE = [  # (tokens, H, topk, E, drop)
    (1, 8, 1, 1, 0.0), (1, 5120, 8, 64, 0.0), (8, 2048, 8, 64, 0.0), (37, 1048, 3, 12, 0.2),
    (19, 520, 40, 64, 0.1), (700, 1032, 6, 32, 0.5), (3, 16, 2, 4, 1.0), (2000, 264, 2, 8, 0.0),
]


@pytest.mark.parametrize("M,H,topk,E,drop", COMBINE)
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(M, H, topk, E, drop, weighted):
    rng = np.random.default_rng([M, H, topk])
    ids = P.make_ids(rng, M, E, topk, drop)
    offsets, dest = P.sort(ids, E)
    y = P.make_rows(rng, M * topk, H)
    y[offsets[-1]:] = np.nan  # rows of no pair
    w = rng.random((M, topk)).astype(np.float32) if weighted else None
    if weighted:
        w[dest < 0] = np.nan  # weights of dropped pairs count for nothing
    ref, size = P.combine(y, dest, w)
    out = Guarded(M, H, seed=1)
    B.moe_combine(cu(y), cu(dest), None if w is None else cu(w), out=out.t)
    got = out.after()
    within(got, ref, P.combine_tol(ref, size, topk), f"combine M={M} H={H} topk={topk}")
    assert not got[(dest < 0).all(axis=1)].any()


@pytest.mark.parametrize("M,H,topk,E,drop", COMBINE)
def test_combine_backward(M, H, topk, E, drop):
    rng = np.random.default_rng([M, H, topk, 1])
    ids = P.make_ids(rng, M, E, topk, drop)
    offsets, dest = P.sort(ids, E)
    y, g = P.make_rows(rng, M * topk, H), P.make_rows(rng, M, H)
    y[offsets[-1]:] = np.nan
    w = rng.standard_normal((M, topk)).astype(np.float32)
    out = Guarded(M * topk, H, seed=2)
    _, dw = B.moe_combine_backward(cu(g), cu(y), cu(dest), cu(w), out=out.t)
    want = out.before().copy()
    for m in range(M):
        for j, d in enumerate(dest[m]):
            if d >= 0:  # one FP32 product, one rounding
                want[d] = (w[m, j] * g[m].astype(np.float32)).astype(np.float16)
    assert np.array_equal(bits(out.after()), bits(want))
    ref, size = P.dweights(g, y, dest)
    dw = dw.cpu().numpy()
    within(dw, ref, H * P.U32 * size, f"dweights M={M} H={H} topk={topk}")
    assert not dw[dest < 0].any()


def test_combine_special_values():
    # infinities and NaN travel as the sum's arithmetic has them
    y = np.array([[np.inf] * 8, [-np.inf] * 8, [1.0] * 8, [np.nan] * 8, [65504.0] * 8], np.float16)
    dest = np.array([[0, 2], [0, 1], [3, 2], [4, 4], [2, -1]], np.int32)
    out = B.moe_combine(cu(y), cu(dest)).cpu().numpy()[:, 0]
    assert out[0] == np.inf and np.isnan(out[1]) and np.isnan(out[2])
    assert out[3] == np.inf and out[4] == 1.0  # overflow rounds to infinity


def test_bad_places_are_reported_and_left_out():
    rng = np.random.default_rng(5)
    y, g = P.make_rows(rng, 4, 64), P.make_rows(rng, 2, 64)
    dest = np.array([[1, 4], [2 ** 31 - 1, 0]], np.int32)
    w = np.ones((2, 2), np.float32)
    out = B.moe_combine(cu(y), cu(dest)).cpu().numpy()
    assert B.device_error() == ERR_INDEX and B.device_error() == 0
    assert np.array_equal(bits(out), bits(y[[1, 0]]))
    buf = Guarded(4, 64)
    _, dw = B.moe_combine_backward(cu(g), cu(y), cu(dest), cu(w), out=buf.t)
    assert B.device_error() == ERR_INDEX
    got = buf.after()
    assert np.array_equal(bits(got[[1, 0]]), bits(g))
    assert np.array_equal(bits(got[2:]), bits(buf.before()[2:]))
    assert dw.cpu().numpy()[0, 1] == 0 and dw.cpu().numpy()[1, 0] == 0


# ---- the experts' products -------------------------------------------------------

PRODUCT = [  # (rows per expert, K, N, G, rows behind the last expert's)
    ([1], 16, 8, -1, 0),
    ([1, 1, 1, 1, 1, 1, 1, 1], 512, 256, 128, 0),
    ([0, 3, 0, 1, 0], 528, 136, 128, 5),
    ([2], 5120, 72, 128, 0),
    ([5, 17, 33, 0, 64, 1], 1040, 200, 16, 9),
    ([16, 0, 15], 2064, 264, 32, 1),
    ([257, 1, 100], 272, 264, 64, 3),
    ([300, 129, 128, 512, 31], 512, 512, 32, 0),
    ([2049], 128, 72, 1024, 40),
    ([33, 65, 97, 161, 193, 225, 255, 256], 192, 320, 256, 2),
    ([700, 0, 900], 256, 2600, 512, 0),
    ([8, 9, 7, 1, 30, 2] * 10, 1424, 392, 64, 11),
    ([0, 0, 0], 256, 128, 32, 6),
    ([1, 0, 2, 1] * 256, 64, 24, 32, 0),
]


def product_inputs(case, gradient):
    counts, K, N, G, tail = case
    rng = np.random.default_rng([len(counts), K, N])
    offsets = P.offsets_of(counts)
    q, s = P.make_weights(rng, len(counts), K, N, G)
    rows = P.make_rows(rng, int(offsets[-1]) + tail, N if gradient else K)
    rows[offsets[-1]:] = np.nan
    return rows, q, s, offsets


@pytest.mark.parametrize("case", PRODUCT, ids=lambda c: f"E{len(c[0])}-K{c[1]}-N{c[2]}-G{c[3]}")
@pytest.mark.parametrize("gradient", [False, True], ids=["y", "dx"])
def test_product(case, gradient):
    counts, K, N, G, tail = case
    rows, q, s, offsets = product_inputs(case, gradient)
    ref, size = P.product(rows, P.expert_weights(q, s, G), offsets, gradient)
    live = int(offsets[-1])
    out = Guarded(rows.shape[0], K if gradient else N, seed=3)
    kw = {} if gradient else dict(kernel=B.KERNEL_PREFILL)
    run = lambda *a, **k: (B.gemm_experts_dx if gradient else B.gemm_experts)(*a, **k, **kw)
    run(cu(rows), cu(q), cu(s), cu(offsets), G, out=out.t)
    got = out.after()
    assert np.array_equal(bits(got[live:]), bits(out.before()[live:]))
    within(got[:live], ref[:live],
           P.product_tol(ref[:live], size[:live], N if gradient else K),
           f"{'dx' if gradient else 'y'} E={len(counts)} K={K} N={N} G={G}")
    again = run(cu(rows), cu(q), cu(s), cu(offsets), G).cpu().numpy()
    assert np.array_equal(bits(again[:live]), bits(got[:live]))


DECODE = [  # more for the kernel of few rows: (rows per expert, K, N, G, rows behind)
    ([1], 4096, 72, 128, 0),              # a cluster of eight shares the item
    ([1, 0, 2], 1536, 264, 64, 1),        # ... of three stages' worth
    ([9, 20, 7], 784, 136, 16, 2),        # K no multiple of 64: boxes of 64 k
    ([64, 65, 31, 33, 17, 15, 128], 320, 1032, 32, 0),
    ([3] * 40, 512, 640, -1, 4),          # more items than SMs
    ([2] * 37, 64, 1024, 128, 0),         # one stage per item
    ([70, 1, 30] * 20, 208, 520, 32, 3),
]


@pytest.mark.parametrize("case", PRODUCT + DECODE,
                         ids=lambda c: f"E{len(c[0])}-K{c[1]}-N{c[2]}-G{c[3]}")
@pytest.mark.parametrize("tile", [16, 32])
def test_product_of_few_rows(case, tile):
    counts, K, N, G, tail = case
    rows, q, s, offsets = product_inputs(case, False)
    ref, size = P.product(rows, P.expert_weights(q, s, G), offsets)
    live = int(offsets[-1])
    out = Guarded(rows.shape[0], N, seed=4)
    args = (cu(rows), cu(q), cu(s), cu(offsets), G)
    B.gemm_experts(*args, out=out.t, kernel=B.KERNEL_DECODE, tile=tile)
    got = out.after()
    assert np.array_equal(bits(got[live:]), bits(out.before()[live:]))
    within(got[:live], ref[:live], P.product_tol(ref[:live], size[:live], K),
           f"tile {tile} E={len(counts)} K={K} N={N} G={G}")
    again = B.gemm_experts(*args, kernel=B.KERNEL_DECODE, tile=tile).cpu().numpy()
    assert np.array_equal(bits(again[:live]), bits(got[:live]))


@pytest.mark.parametrize("tile", [16, 32])
def test_few_rows_over_long_walks(tile):
    """Many items and stages per CTA, over and over: the ring, the A slots and
    the accumulators wrap around many times, with the same result each time
    and the other kernel's within the bound."""
    rng = np.random.default_rng(tile)
    K, N, G, E = 2048, 2048, 128, 48
    offsets = P.offsets_of(rng.integers(0, 2 * tile // 3 + 3, E))
    x, (q, s) = P.make_rows(rng, int(offsets[-1]), K), P.make_weights(rng, E, K, N, G)
    args = (cu(x), cu(q), cu(s), cu(offsets), G)
    first = B.gemm_experts(*args, kernel=B.KERNEL_DECODE, tile=tile)
    for _ in range(30):
        assert torch.equal(B.gemm_experts(*args, kernel=B.KERNEL_DECODE, tile=tile), first)
    assert B.device_error() == 0
    some = rng.choice(len(x), 24, replace=False)
    expert = np.searchsorted(offsets, some, side="right") - 1
    for r, e in zip(some, expert):
        w = oracle.dequant(q[e], s[e], G).astype(np.float64)
        ref = x[r].astype(np.float64) @ w
        size = np.abs(x[r].astype(np.float64)) @ np.abs(w)
        within(first[r].cpu().numpy(), ref, P.product_tol(ref, size, K), f"tile {tile} row {r}")


@pytest.mark.parametrize("counts", [[2, 3, 1], [40, 70, 20], [300, 5, 140]])
@pytest.mark.parametrize("G", [-1, 16, 32, 64, 128])
def test_one_hot_rows_reproduce_weights(counts, G):
    """Every scale (subnormal, negative, zero, large) and code: bit for bit.
    The middle expert's scales are NaN and infinite; nothing of it shows in
    the others' rows."""
    rng = np.random.default_rng(G + 7)
    K, N = 272, 200
    offsets = P.offsets_of(counts)
    q, s = P.make_weights(rng, 3, K, N, G)
    s = (s * 2.0 ** rng.integers(-18, 9, s.shape) * rng.choice([1, 1, 1, -1, 0], s.shape)
         ).astype(np.float16)
    s[1] = rng.choice([np.nan, np.inf, -np.inf], s[1].shape)
    w = np.stack([oracle.dequant(q[e], s[e], G) if e != 1 else np.zeros((K, N), np.float16)
                  for e in range(3)])
    args = (cu(q), cu(s), cu(offsets), G)
    R = int(offsets[-1])
    expert = np.searchsorted(offsets, np.arange(R), side="right") - 1
    keep = expert != 1
    decode = [dict(kernel=B.KERNEL_DECODE, tile=t) for t in (16, 32)]
    for kw in [{}, dict(kernel=B.KERNEL_PREFILL), *decode, None]:
        gradient = kw is None
        width = N if gradient else K
        hot = rng.integers(0, width, R)
        rows = np.zeros((R, width), np.float16)
        rows[np.arange(R), hot] = 1.0
        got = (B.gemm_experts_dx(cu(rows), *args) if gradient
               else B.gemm_experts(cu(rows), *args, **kw)).cpu().numpy()[keep]
        want = np.stack([w[e, :, h] if gradient else w[e, h] for e, h in zip(expert, hot)])[keep]
        # a sum with zeros has no negative zero
        assert np.array_equal(bits(got + np.float16(0)), bits(want + np.float16(0)))


@pytest.mark.parametrize("gradient", [False, True], ids=["y", "dx"])
@pytest.mark.parametrize("counts", [[3, 2], [150, 90]])
def test_a_row_with_nan_touches_no_other(counts, gradient):
    rng = np.random.default_rng(11)
    K, N, G = 512, 256, 128
    offsets = P.offsets_of(counts)
    q, s = P.make_weights(rng, 2, K, N, G)
    rows = P.make_rows(rng, int(offsets[-1]), N if gradient else K)
    bad = rows.copy()
    bad[1] = np.nan
    bad[offsets[1], 5] = np.inf
    run = B.gemm_experts_dx if gradient else B.gemm_experts
    args = (cu(q), cu(s), cu(offsets), G)
    a, b = run(cu(rows), *args).cpu().numpy(), run(cu(bad), *args).cpu().numpy()
    others = np.ones(len(rows), bool)
    others[[1, offsets[1]]] = False
    assert np.array_equal(bits(a[others]), bits(b[others]))
    assert np.isnan(b[1]).all() and not np.isfinite(b[offsets[1]]).any()


@pytest.mark.parametrize("kernel,tile", [(3, 0), (-1, 0), (1, 0), (1, 8), (2, 16), (0, 16)])
def test_bad_kernel_choices_are_refused(kernel, tile):
    rng = np.random.default_rng(1)
    q, s = P.make_weights(rng, 2, 64, 32, 32)
    with pytest.raises(B.GptqError) as e:
        B.gemm_experts(cu(P.make_rows(rng, 4, 64)), cu(q), cu(s), cu(P.offsets_of([2, 2])), 32,
                       kernel=kernel, tile=tile)
    assert e.value.status == 9


@pytest.mark.parametrize("offsets", [[0, 5, 3, 8], [0, 4, 9, 11], [-3, 2, 5, 8], [0, 8, 8, 4]])
def test_bad_offsets_are_reported(offsets):
    rng = np.random.default_rng(3)
    K, N, G = 256, 136, 64
    q, s = P.make_weights(rng, 3, K, N, G)
    off = cu(np.array(offsets, np.int32))
    for gradient in (False, True):
        out = Guarded(8, K if gradient else N)
        run = B.gemm_experts_dx if gradient else B.gemm_experts
        run(cu(P.make_rows(rng, 8, N if gradient else K)), cu(q), cu(s), off, G, out=out.t)
        out.after()
        assert B.device_error() == ERR_INDEX


def test_binding_refuses_mis_shaped_tensors():
    rng = np.random.default_rng(0)
    q, s = P.make_weights(rng, 2, 64, 32, 32)
    off, rows = cu(P.offsets_of([2, 2])), cu(P.make_rows(rng, 4, 64))
    ok = dict(x_sorted=rows, qweight=cu(q), scales=cu(s), offsets=off, group=32)
    half = lambda *shape: torch.zeros(shape, dtype=torch.float16, device="cuda")
    for kw, err in [(dict(out=half(4, 40)), ValueError), (dict(out=half(3, 32)), ValueError),
                    (dict(x_sorted=half(4, 32)), ValueError),
                    (dict(x_sorted=half(4, 128)[:, ::2]), ValueError),
                    (dict(x_sorted=rows.float()), TypeError),
                    (dict(offsets=off[:2]), ValueError), (dict(offsets=off.long()), TypeError),
                    (dict(scales=cu(s)[:, :1]), ValueError)]:
        with pytest.raises(err):
            B.gemm_experts(**{**ok, **kw})
    x, ids = half(3, 64), torch.zeros((3, 2), dtype=torch.int32, device="cuda")
    for args, kw, err in [((x, ids[:2], 4), {}, ValueError), ((x, ids.float(), 4), {}, TypeError),
                          ((x, ids[:, 0], 4), {}, ValueError), ((x, ids, 0), {}, B.GptqError),
                          ((x, ids, 1025), {}, B.GptqError), ((x, ids, 4), dict(out=half(5, 64)), ValueError)]:
        with pytest.raises(err):
            B.moe_sort(*args, **kw)
    y, w = half(6, 64), torch.zeros((3, 2), device="cuda")
    for args, err in [((y, ids, w[:2]), ValueError), ((y, ids, w.half()), TypeError),
                      ((y, ids.long(), w), TypeError), ((y.float(), ids, w), TypeError)]:
        with pytest.raises(err):
            B.moe_combine(*args)
    for args, err in [((x[:2], y, ids, w), ValueError), ((x, half(6, 32), ids, w), ValueError),
                      ((x, y, ids, None), TypeError)]:
        with pytest.raises(err):
            B.moe_combine_backward(*args)


# ---- a layer -----------------------------------------------------------------------

class Layer:
    """A layer's experts (gate and up side by side, then down) and its run."""

    def __init__(self, E, H, F, G, seed):
        rng = np.random.default_rng(seed)
        self.E, self.F, self.G = E, F, G
        up, down = P.make_weights(rng, E, H, 2 * F, G), P.make_weights(rng, E, F, H, G)
        self.host = [P.expert_weights(*up, G), P.expert_weights(*down, G)]
        self.up, self.down = [cu(a) for a in up], [cu(a) for a in down]

    def forward(self, x, ids, w):
        xs, offsets, dest = B.moe_sort(x, ids, self.E)
        gu = B.gemm_experts(xs, *self.up, offsets, self.G)
        gate, up = gu[:, :self.F].float(), gu[:, self.F:].float()
        h = (torch.nn.functional.silu(gate) * up).half()
        y = B.gemm_experts(h, *self.down, offsets, self.G)
        return B.moe_combine(y, dest, w), (offsets, dest, gate, up, y)

    def backward(self, dout, w, saved):
        offsets, dest, gate, up, y = saved
        dy, dw = B.moe_combine_backward(dout, y, dest, w)
        dh = B.gemm_experts_dx(dy, *self.down, offsets, self.G).float()
        sg = torch.sigmoid(gate)
        dgate = dh * up * sg * (1 + gate * (1 - sg))
        dgu = torch.cat([dgate, dh * gate * sg], dim=1).half()
        dxs = B.gemm_experts_dx(dgu, *self.up, offsets, self.G)
        return B.moe_combine(dxs, dest), dw

    def plain(self, x, ids, w):
        """The same layer in 64 bits, rounded to FP16 where it hands on rows;
        differentiable in x and w."""
        rows = lambda t: t + (t.detach().half().double() - t.detach())  # rounded, gradient 1
        out = torch.zeros_like(x)
        for m in range(x.shape[0]):
            for j in range(ids.shape[1]):
                e = int(ids[m, j])
                if 0 <= e < self.E:
                    gu = rows(x[m] @ torch.from_numpy(self.host[0][e].astype(np.float64)))
                    h = rows(torch.nn.functional.silu(gu[:self.F]) * gu[self.F:])
                    y = rows(h @ torch.from_numpy(self.host[1][e].astype(np.float64)))
                    out = out.index_add(0, torch.tensor([m]), (w[m, j] * y)[None])
        return out


@pytest.mark.parametrize("M,E,topk,H,F,G", [(1, 8, 2, 256, 192, 64), (24, 6, 3, 136 * 2, 96, 32)])
def test_layer_forward_and_backward(M, E, topk, H, F, G):
    layer = Layer(E, H, F, G, seed=M)
    rng = np.random.default_rng(M + 1)
    x = P.make_rows(rng, M, H)
    ids = P.make_ids(rng, M, E, topk, drop=0.1 if M > 1 else 0.0)
    w = rng.random((M, topk)).astype(np.float32)
    dout = P.make_rows(rng, M, H)
    out, saved = layer.forward(cu(x), cu(ids), cu(w))
    dx, dw = layer.backward(cu(dout), cu(w), saved)

    tx = torch.from_numpy(x.astype(np.float64)).requires_grad_()
    tw = torch.from_numpy(w.astype(np.float64)).requires_grad_()
    ref = layer.plain(tx, ids, tw)
    (ref * torch.from_numpy(dout.astype(np.float64))).sum().backward()
    # Each value passes three roundings to FP16 forward (gate/up, h, y) and
    # four more backward (dy, dh's and dgu's rows, dx), relative U16 each on
    # rows whose entries are comparable in size; sums of independent errors
    # grow like their root, so eight U16 of the result's RMS bound the RMS of
    # the error with a factor of two to spare.
    for got, want, label in ((out, ref.detach(), "out"), (dx, tx.grad, "dx"), (dw, tw.grad, "dw")):
        got, want = got.cpu().double().numpy(), want.numpy()
        rms = np.sqrt(np.mean((got - want) ** 2)) / np.sqrt(np.mean(want ** 2))
        print(f"[moe] layer M={M} {label}: RMS error {rms:.2e}")
        assert rms <= 8 * P.U16, label

    # against differences of the forward pass itself: dout . out along the
    # gradient's own direction, a step to each side; the values of out carry
    # three roundings each, at random sign
    d = dx.cpu().numpy().astype(np.float64)
    d = (d / np.sqrt(np.mean(d ** 2))).astype(np.float32)
    step = 2.0 ** -4
    ends = [layer.forward(cu((x.astype(np.float32) + t * d).astype(np.float16)), cu(ids),
                          cu(w))[0].cpu().double().numpy() for t in (step, -step)]
    xs = [(x.astype(np.float32) + t * d).astype(np.float16).astype(np.float64)
          for t in (step, -step)]
    g = dout.astype(np.float64)
    slope = (g * (ends[0] - ends[1])).sum()
    want = (dx.cpu().double().numpy() * (xs[0] - xs[1])).sum()
    noise = 4 * 3 * P.U16 * np.sqrt((g ** 2 * (ends[0] ** 2 + ends[1] ** 2)).sum())
    curve = step ** 2 * np.sqrt((g ** 2).sum() * (ends[0] ** 2).sum())
    print(f"[moe] layer M={M}: difference {slope:.4f}, gradient {want:.4f}, "
          f"noise {noise:.4f}, curvature {curve:.4f}")
    assert abs(slope - want) <= noise + curve


@pytest.mark.parametrize("gradient", [False, True], ids=["y", "dx"])
def test_product_is_linear_along_differences(gradient):
    """<g, F(x + d) - F(x)> = <F^T g, d>, both sides from the kernels."""
    rng = np.random.default_rng(21)
    K, N, G = 400, 264, 32
    offsets = P.offsets_of([7, 0, 70, 33])
    q, s = P.make_weights(rng, 4, K, N, G)
    args = (cu(q), cu(s), cu(offsets), G)
    fwd, bwd = (B.gemm_experts_dx, B.gemm_experts) if gradient else (B.gemm_experts, B.gemm_experts_dx)
    a, b = (N, K) if gradient else (K, N)
    x, d, g = (P.make_rows(rng, 110, n) for n in (a, a, b))
    f = lambda t: fwd(cu(t), *args).cpu().double().numpy()
    xd = (x.astype(np.float32) + d).astype(np.float16)
    f1, f0 = f(xd), f(x)
    ft = bwd(cu(g), *args).cpu().double().numpy()
    lhs = (g.astype(np.float64) * (f1 - f0)).sum()
    step = xd.astype(np.float64) - x
    rhs = (ft * step).sum()
    w = P.expert_weights(q, s, G)
    tol = 0.0
    for rows, out, grad, weight in ((xd, f1, gradient, g), (x, f0, gradient, g), (g, ft, not gradient, step)):
        ref, size = P.product(rows, w, offsets, grad)
        tol += (np.abs(weight) * P.product_tol(ref, size, rows.shape[1])).sum()
    assert abs(lhs - rhs) <= tol
    # the bound of every rounding at once is wide; at random signs the errors
    # stay within a few parts of its root-mean-square form
    assert abs(lhs - rhs) <= 6 * P.U16 * np.sqrt(sum(
        ((np.asarray(u, np.float64) * v) ** 2).sum() for u, v in ((g, f1), (g, f0), (ft, step))))


def test_captured_layer_sees_new_routings():
    """A captured run of the layer, forward and backward, replayed on new
    tokens and routings, equals the calls made one by one."""
    layer = Layer(8, 512, 256, 128, seed=9)
    M, topk = 40, 2
    rng = np.random.default_rng(2)
    draw = lambda: (cu(P.make_rows(rng, M, 512)), cu(P.make_ids(rng, M, 8, topk, 0.2)),
                    cu(rng.random((M, topk)).astype(np.float32)), cu(P.make_rows(rng, M, 512)))
    x, ids, w, dout = draw()

    def run():
        out, saved = layer.forward(x, ids, w)
        return (out, *layer.backward(dout, w, saved))

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        run()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run()
    for _ in range(3):
        for old, new in zip((x, ids, w, dout), draw()):
            old.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in captured]
        for a, b in zip(got, run()):
            assert torch.equal(a, b)


def test_calls_on_two_streams_at_once():
    rng = np.random.default_rng(4)
    K, N, G, E = 1024, 520, 64, 12
    sets = []
    for i in range(2):
        q, s = P.make_weights(rng, E, K, N, G)
        x, ids = P.make_rows(rng, 50 + 9 * i, K), P.make_ids(rng, 50 + 9 * i, E, 3)
        sets.append([cu(a) for a in (x, ids, q, s)])

    def run(x, ids, q, s, stream=None):
        xs, offsets, dest = B.moe_sort(x, ids, E, stream=stream)
        y = B.gemm_experts(xs, q, s, offsets, G, stream=stream)
        dx = B.gemm_experts_dx(y, q, s, offsets, G, stream=stream)
        return B.moe_combine(y, dest, stream=stream), B.moe_combine(dx, dest, stream=stream)

    want = [run(*a) for a in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for _ in range(5):
        for a, st in zip(sets, streams):
            with torch.cuda.stream(st):
                got.append(run(*a, stream=st))
    torch.cuda.synchronize()
    for i, pair in enumerate(got):
        for a, b in zip(pair, want[i % 2]):
            assert torch.equal(a, b)


def test_abi_takes_the_legacy_default_stream():
    rng = np.random.default_rng(6)
    x, ids = cu(P.make_rows(rng, 5, 64)), cu(P.make_ids(rng, 5, 4, 2))
    xs = torch.empty((10, 64), dtype=torch.float16, device="cuda")
    off = torch.empty(5, dtype=torch.int32, device="cuda")
    dest = torch.empty((5, 2), dtype=torch.int32, device="cuda")
    ptr = lambda t: ctypes.c_void_p(t.data_ptr())
    assert B.load().gptq_moe_sort(ptr(x), ptr(ids), 4, 5, 64, 2, 4, ptr(xs), ptr(off), ptr(dest),
                                  None) == 0
    torch.cuda.synchronize()
    a, b, c = B.moe_sort(x, ids, 4)
    assert torch.equal(a, xs) and torch.equal(b, off) and torch.equal(c, dest)


def layer_on(stream, x, ids, w, q, s, E, G):
    """Every operator with stream= and its own outputs."""
    xs, offsets, dest = B.moe_sort(x, ids, E, stream=stream)
    y = B.gemm_experts(xs, q, s, offsets, G, stream=stream)
    out = B.moe_combine(y, dest, w, stream=stream)
    dy, dw = B.moe_combine_backward(out, y, dest, w, stream=stream)
    dx = B.gemm_experts_dx(dy, q, s, offsets, G, stream=stream)
    return xs, offsets, dest, y, out, dy, dw, dx


def test_outputs_on_another_stream_take_no_memory_that_the_callers_still_uses():
    rng = np.random.default_rng(11)
    M, E, K, N, G = 300, 6, 512, 512, 64
    q, s = (cu(a) for a in P.make_weights(rng, E, K, N, G))
    x, ids = cu(P.make_rows(rng, M, K)), cu(P.make_ids(rng, M, E, 2))
    w = torch.rand((M, 2), device="cuda")
    want = layer_on(None, x, ids, w, q, s, E, G)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    # blocks of these sizes, freed while the caller's stream may still use them
    freed = [torch.empty_like(t) for t in want for _ in range(3)]
    spans = [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in freed]
    del freed
    got = layer_on(side, x, ids, w, q, s, E, G)
    for t in got:
        end = t.data_ptr() + t.numel() * t.element_size()
        assert all(end <= a or t.data_ptr() >= b for a, b in spans)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    out = torch.empty_like(want[4])
    assert B.moe_combine(want[3], want[2], w, out=out, stream=side) is out
    torch.cuda.synchronize()
    assert torch.equal(out, want[4])


def test_captured_on_a_forked_stream():
    rng = np.random.default_rng(12)
    M, E, K, N, G = 40, 6, 512, 512, 64
    q, s = (cu(a) for a in P.make_weights(rng, E, K, N, G))
    x, ids = cu(P.make_rows(rng, M, K)), cu(P.make_ids(rng, M, E, 2))
    w = torch.rand((M, 2), device="cuda")
    want = layer_on(None, x, ids, w, q, s, E, G)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = layer_on(side, x, ids, w, q, s, E, G)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("n", [0, -1, 1025, 10 ** 12])
def test_sort_refuses_numbers_of_experts(n):
    x = torch.zeros((4, 64), dtype=torch.float16, device="cuda")
    with pytest.raises(B.GptqError) as e:
        B.moe_sort(x, torch.zeros((4, 2), dtype=torch.int32, device="cuda"), n)
    assert e.value.status == 2  # GPTQ_ERR_SHAPE


@pytest.mark.parametrize("E,R,K,N", [(200, 64, 256, 136), (9, 3000, 2048, 264), (2, 5, 2048, 128)])
def test_offsets_that_overlap_are_reported(E, R, K, N):
    rng = np.random.default_rng(E)
    q, s = (cu(a) for a in P.make_weights(rng, E, K, N, 64))
    offsets = torch.arange(E + 1, device="cuda", dtype=torch.int32) % 2 * R  # 0, R, 0, R, ...
    if E == 2:
        offsets = torch.tensor([0, R, 2], device="cuda", dtype=torch.int32)
    for gradient in (False, True):
        rows = cu(P.make_rows(rng, R, N if gradient else K))
        out = Guarded(R, K if gradient else N)
        run = B.gemm_experts_dx if gradient else B.gemm_experts
        good = cu(P.offsets_of([R] + [0] * (E - 1)))
        want = run(rows, q, s, good, 64)
        run(rows, q, s, offsets, 64, out=out.t)
        out.after()
        assert B.device_error() == ERR_INDEX
        assert torch.equal(run(rows, q, s, good, 64), want)  # the next call works
        assert B.device_error() == 0


@pytest.mark.parametrize("counts,tile,gradient", [
    ([3, 0, 9], 16, False), ([3, 0, 30], 32, False), ([150, 0, 40], 0, False),
    ([150, 0, 40], 0, True)])
def test_longest_sums(counts, tile, gradient):
    K, N = (72 * 8, 65536) if gradient else (65536, 136)
    rows, q, s, offsets = product_inputs((counts, K, N, 128, 0), gradient)
    ref, size = P.product(rows, P.expert_weights(q, s, 128), offsets, gradient)
    kw = {} if gradient else dict(kernel=B.KERNEL_DECODE if tile else B.KERNEL_PREFILL, tile=tile)
    run = B.gemm_experts_dx if gradient else B.gemm_experts
    got = run(cu(rows), cu(q), cu(s), cu(offsets), 128, **kw).cpu().numpy()
    within(got, ref, P.product_tol(ref, size, 65536), f"{counts} {gradient}")
    within(got, ref, 1e-2 * (1 + np.abs(ref)), f"{counts} {gradient}, the library's bound")


@pytest.mark.parametrize("G", [16, 32, 64, 128, -1])
@pytest.mark.parametrize("gradient", [False, True], ids=["y", "dx"])
def test_product_of_many_rows(G, gradient):
    """Enough rows and columns for the tiles of 256 rows."""
    K, N = (5136, 200) if gradient else (208, 5128)
    rows, q, s, offsets = product_inputs(([700, 0, 333], K, N, G, 0), gradient)
    ref, size = P.product(rows, P.expert_weights(q, s, G), offsets, gradient)
    out = Guarded(1033, K if gradient else N, seed=5)
    run = B.gemm_experts_dx if gradient else B.gemm_experts
    run(cu(rows), cu(q), cu(s), cu(offsets), G, out=out.t)
    within(out.after(), ref, P.product_tol(ref, size, N if gradient else K),
           f"{'dx' if gradient else 'y'} K={K} N={N} G={G}")
