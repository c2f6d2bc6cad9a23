"""The mixture-of-experts entries on the host: every refusal of the C ABI and
of the binding, before a device is touched.  No call here launches a kernel."""
import ctypes

import numpy as np
import pytest
import torch

import moe_plain as P
from int4_weight_only_gptq_b200 import binding as B
from int4_weight_only_gptq_b200.build import build

NULL, SHAPE, GROUP, ALIGN, DEVICE, ALIAS = 1, 2, 3, 4, 5, 8

# fake, aligned addresses far apart: never dereferenced
A = [0x10000000 * (i + 1) for i in range(8)]


@pytest.fixture(scope="module")
def lib():
    build()
    return B.load()


def v(p):
    return ctypes.c_void_p(p) if p else None


def sort(lib, x=A[0], ids=A[1], nb=4, M=4, H=64, topk=2, E=8, xs=A[2], off=A[3], dest=A[4]):
    return lib.gptq_moe_sort(v(x), v(ids), nb, M, H, topk, E, v(xs), v(off), v(dest), None)


def combine(lib, y=A[0], dest=A[1], w=A[2], M=4, H=64, topk=2, R=8, out=A[3]):
    return lib.gptq_moe_combine(v(y), v(dest), v(w), M, H, topk, R, v(out), None)


def backward(lib, g=A[0], y=A[1], dest=A[2], w=A[3], M=4, H=64, topk=2, R=8, dy=A[4], dw=A[5]):
    return lib.gptq_moe_combine_backward(v(g), v(y), v(dest), v(w), M, H, topk, R, v(dy), v(dw),
                                         None)


def experts(lib, name, x=A[0], qw=A[1], s=A[2], off=A[3], R=8, K=64, N=64, E=8, g=32, y=A[4]):
    return getattr(lib, name)(v(x), v(qw), v(s), v(off), R, K, N, E, g, v(y), None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), SHAPE), (dict(H=0), SHAPE), (dict(H=-8), SHAPE), (dict(H=60), SHAPE),
    (dict(H=65536 + 8), SHAPE), (dict(topk=0), SHAPE), (dict(topk=65), SHAPE),
    (dict(E=0), SHAPE), (dict(E=1025), SHAPE), (dict(nb=2), SHAPE), (dict(nb=0), SHAPE),
    (dict(M=(1 << 23) // 2 + 1), SHAPE), (dict(M=1 << 62), SHAPE),
    (dict(x=0), NULL), (dict(ids=0), NULL), (dict(xs=0), NULL), (dict(off=0), NULL),
    (dict(dest=0), NULL), (dict(M=0, off=0), NULL),
    (dict(x=A[0] + 8), ALIGN), (dict(xs=A[2] + 2), ALIGN), (dict(ids=A[1] + 2), ALIGN),
    (dict(nb=8, ids=A[1] + 4), ALIGN), (dict(off=A[3] + 2), ALIGN), (dict(dest=A[4] + 1), ALIGN),
    (dict(xs=A[0]), ALIAS), (dict(off=A[0] + 16), ALIAS), (dict(dest=A[1]), ALIAS),
    (dict(dest=A[2]), ALIAS), (dict(off=A[4]), ALIAS),
])
def test_sort_argument_checks(lib, kw, status):
    assert sort(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), SHAPE), (dict(H=12), SHAPE), (dict(topk=0), SHAPE), (dict(topk=65), SHAPE),
    (dict(R=-1), SHAPE), (dict(R=(1 << 23) + 1), SHAPE),
    (dict(y=0), NULL), (dict(dest=0), NULL), (dict(out=0), NULL),
    (dict(y=A[0] + 4), ALIGN), (dict(out=A[3] + 8), ALIGN), (dict(w=A[2] + 1), ALIGN),
    (dict(dest=A[1] + 3), ALIGN),
    (dict(out=A[0]), ALIAS), (dict(out=A[1]), ALIAS), (dict(out=A[2]), ALIAS),
])
def test_combine_argument_checks(lib, kw, status):
    assert combine(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), SHAPE), (dict(H=4), SHAPE), (dict(topk=70), SHAPE), (dict(R=-2), SHAPE),
    (dict(g=0), NULL), (dict(y=0), NULL), (dict(dest=0), NULL), (dict(w=0), NULL),
    (dict(dy=0), NULL), (dict(dw=0), NULL),
    (dict(g=A[0] + 8), ALIGN), (dict(y=A[1] + 2), ALIGN), (dict(dy=A[4] + 4), ALIGN),
    (dict(w=A[3] + 2), ALIGN), (dict(dw=A[5] + 2), ALIGN),
    (dict(dy=A[0]), ALIAS), (dict(dy=A[1]), ALIAS), (dict(dw=A[2]), ALIAS), (dict(dw=A[3]), ALIAS),
    (dict(dw=A[4]), ALIAS),
])
def test_combine_backward_argument_checks(lib, kw, status):
    assert backward(lib, **kw) == status


@pytest.mark.parametrize("name", ["gptq_w4a16_gemm_experts", "gptq_w4a16_gemm_experts_dx"])
@pytest.mark.parametrize("kw,status", [
    (dict(R=-1), SHAPE), (dict(K=24), SHAPE), (dict(N=12), SHAPE), (dict(E=0), SHAPE),
    (dict(E=1025), SHAPE), (dict(R=(1 << 23) + 1), SHAPE), (dict(K=65536 + 16), SHAPE),
    (dict(g=8), GROUP), (dict(g=0), GROUP),
    (dict(x=0), NULL), (dict(qw=0), NULL), (dict(s=0), NULL), (dict(off=0), NULL),
    (dict(y=0), NULL),
    (dict(x=A[0] + 8), ALIGN), (dict(qw=A[1] + 4), ALIGN), (dict(s=A[2] + 2), ALIGN),
    (dict(off=A[3] + 2), ALIGN), (dict(y=A[4] + 8), ALIGN),
    (dict(y=A[0]), ALIAS), (dict(y=A[1] + 64), ALIAS), (dict(y=A[2]), ALIAS), (dict(y=A[3]), ALIAS),
])
def test_experts_argument_checks(lib, name, kw, status):
    assert experts(lib, name, **kw) == status


@pytest.mark.parametrize("kernel,tile", [(3, 0), (-1, 0), (1, 0), (1, 8), (2, 16), (0, 16)])
def test_experts_kernel_choice_checks(lib, kernel, tile):
    args = [v(a) for a in A[:4]] + [8, 64, 64, 8, 32, v(A[4]), None]
    assert lib.gptq_w4a16_gemm_experts_kernel(*args, kernel, tile) == 9


def test_empty_calls_are_no_ops(lib):
    assert combine(lib, M=0, y=0, dest=0, out=0) == 0
    assert backward(lib, M=0, g=0, y=0, dest=0, w=0, dy=0, dw=0) == 0
    for name in ("gptq_w4a16_gemm_experts", "gptq_w4a16_gemm_experts_dx"):
        assert experts(lib, name, R=0, x=0, y=0) == 0


def test_no_device_is_reported(lib):
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    assert sort(lib) == DEVICE
    assert sort(lib, M=0, x=0, ids=0, xs=0, dest=0) == DEVICE  # offsets would be written
    assert combine(lib) == DEVICE
    assert backward(lib) == DEVICE
    assert experts(lib, "gptq_w4a16_gemm_experts") == DEVICE
    assert experts(lib, "gptq_w4a16_gemm_experts_dx") == DEVICE


def test_binding_refuses_cpu_tensors(lib):
    x = torch.zeros(2, 64, dtype=torch.float16)
    ids = torch.zeros(2, 1, dtype=torch.int32)
    with pytest.raises(ValueError):
        B.moe_sort(x, ids, 4)
    with pytest.raises(ValueError):
        B.moe_combine(x, ids)
    with pytest.raises(ValueError):
        B.moe_combine_backward(x, x, ids, ids.float())
    qw = torch.zeros(4, 8, 64, dtype=torch.int32)
    s = torch.zeros(4, 2, 64, dtype=torch.float16)
    off = torch.zeros(5, dtype=torch.int32)
    with pytest.raises(ValueError):
        B.gemm_experts(x, qw, s, off, 32)
    with pytest.raises(ValueError):
        B.gemm_experts_dx(x, qw, s, off, 32)


def test_experts_shapes():
    t = lambda *s: torch.empty(s, device="meta")
    args = (t(4, 64, 40), t(4, 16, 40), t(5))
    assert B.experts_shapes(t(7, 512), *args, 32) == (7, 512, 40, 4)
    assert B.experts_shapes(t(7, 40), *args, 32, gradient=True) == (7, 512, 40, 4)
    for bad in [(t(7, 40), *args), (t(7, 512, 1), *args), (t(7, 512), t(64, 40), *args[1:]),
                (t(7, 512), args[0], t(4, 15, 40), args[2]),
                (t(7, 512), args[0], t(3, 16, 40), args[2]),
                (t(7, 512), args[0], t(4, 16, 48), args[2]),
                (t(7, 512), args[0], args[1], t(4)), (t(7, 512), args[0], args[1], t(5, 1))]:
        with pytest.raises(ValueError):
            B.experts_shapes(*bad, 32)
    with pytest.raises(ValueError):
        B.experts_shapes(t(7, 512), *args, 32, gradient=True)


def test_plain_forms_agree_with_a_worked_example():
    # three tokens, two choices, three experts; token 1's second choice dropped
    ids = np.array([[2, 0], [0, -1], [2, 2]], dtype=np.int32)
    offsets, dest = P.sort(ids, 3)
    assert offsets.tolist() == [0, 2, 2, 5]
    assert dest.tolist() == [[2, 0], [1, -1], [3, 4]]
    x = np.arange(6, dtype=np.float16).reshape(3, 2)
    xs = P.sorted_rows(x, dest, np.full((6, 2), 9, np.float16))
    assert xs.tolist() == [[0, 1], [2, 3], [0, 1], [4, 5], [4, 5], [9, 9]]
    out, _ = P.combine(xs, dest, np.array([[1, 2], [3, np.nan], [5, 6]], np.float32))
    assert out.tolist() == [[0, 3], [6, 9], [44, 55]]
    dw, _ = P.dweights(x, xs, dest)
    assert dw.tolist() == [[1, 1], [13, 0], [41, 41]]
    rng = np.random.default_rng(0)
    q, s = P.make_weights(rng, 3, 32, 16, 16)
    w = P.expert_weights(q, s, 16)
    k, n, e = 21, 5, 1
    code = (int(q[e, k // 8, n]) >> (4 * (k % 8))) & 15
    assert w[e, k, n] == np.float16(np.float64(code - 8) * np.float64(s[e, k // 16, n]))
    rows = P.make_rows(rng, 5, 32)
    y, _ = P.product(rows, w, offsets)
    assert np.array_equal(y[3], rows[3].astype(np.float64) @ w[2].astype(np.float64))
    g, _ = P.product(P.make_rows(rng, 5, 16), w, offsets, gradient=True)
    assert g.shape == (5, 32)


def test_experts_gradient_limits_the_length_of_its_sums(lib):
    assert experts(lib, "gptq_w4a16_gemm_experts_dx", N=65536 + 8, R=0) == SHAPE
    assert experts(lib, "gptq_w4a16_gemm_experts_dx", N=65536, R=0) == 0
    assert experts(lib, "gptq_w4a16_gemm_experts", N=65536 + 8, R=0) == 0
