"""Numbers wider than the library's types.  ctypes passes on their low bits: a
group of 2^32 + 128 would reach the library as 128 without the scales' shape
having been checked for it, and 2^64 + 8 experts as 8 with offsets allocated
for none.  No call here reaches the library."""
import contextlib
import ctypes
from types import SimpleNamespace

import pytest
import torch

from int4_weight_only_gptq_b200 import binding as B
from int4_weight_only_gptq_b200.build import build

WIDE = [2 ** 32 + 32, -2 ** 32 + 128, 2 ** 40 - 1, 2 ** 64 + 64, -2 ** 63 + 16]


@pytest.fixture
def sent(monkeypatch):
    """What the binding would hand to the library, in its types."""
    calls = []
    build()
    lib = B.load()

    def entry(name):
        def fn(*args):
            types = getattr(lib, name).argtypes
            assert len(args) == len(types)
            calls.append([t(a).value if t in (ctypes.c_int32, ctypes.c_int64) else a
                          for t, a in zip(types, args)])
            return 0
        return fn

    fake = SimpleNamespace(**{n: entry(n) for n in B.EXPORTS if n.startswith("gptq_")})
    monkeypatch.setattr(B, "load", lambda: fake)
    monkeypatch.setattr(B, "_lib", fake)
    monkeypatch.setattr(B, "_require", lambda *a: None)
    monkeypatch.setattr(B, "_fits", lambda *a: True)
    monkeypatch.setattr(B, "_device_index", lambda *a: 0)
    monkeypatch.setattr(B, "_current", lambda device: None)
    monkeypatch.setattr(B, "_call", lambda fn, index, *args: fn(*args, None))
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    return calls


half = lambda *s: torch.zeros(s, dtype=torch.float16)
word = lambda *s: torch.zeros(s, dtype=torch.int32)
x, q, sc = half(2, 64), word(8, 32), half(1, 32)  # scales for one group only
stacked = (x, word(3, 8, 32), half(3, 1, 32), word(4))
BY_GROUP = {
    "gemm": lambda g: B.gemm(x, q, sc, g),
    "gemm_kernel": lambda g: B.gemm(x, q, sc, g, kernel=B.KERNEL_DECODE),
    "gemm_splits": lambda g: B.gemm(x, q, sc, g, decode_splits=1),
    "gemm_grouped": lambda g: B.gemm_grouped(x, [q], [sc], g),
    "gemm_asym": lambda g: B.gemm_asym(x, q, sc, word(1, 4), g),
    "gemm_lora": lambda g: B.gemm_lora(x, q, sc, g, half(16, 64), half(32, 16)),
    "gemm_lora_noalloc": lambda g: B.gemm_lora_noalloc(x, q, sc, g, half(16, 64), half(32, 16)),
    "dequant": lambda g: B.dequant(q, sc, g),
    "gemm_experts": lambda g: B.gemm_experts(*stacked, g),
    "gemm_experts_dx": lambda g: B.gemm_experts_dx(half(2, 32), *stacked[1:], g),
}
GROUP_AT = {"gemm_grouped": 7, "gemm_asym": 7, "dequant": 4, "gemm_experts": 8,
            "gemm_experts_dx": 8}


@pytest.mark.parametrize("name", BY_GROUP)
@pytest.mark.parametrize("group", WIDE)
def test_a_wide_group_reaches_the_library_as_none(sent, name, group):
    BY_GROUP[name](group)
    assert sent[0][GROUP_AT.get(name, 6)] not in B.GROUP_SIZES
    BY_GROUP[name](64)
    assert sent[1][GROUP_AT.get(name, 6)] == 64


@pytest.mark.parametrize("n", WIDE + [2 ** 64 + 8, 2 ** 65 + 1024, 1025, 0, -1])
def test_a_wide_number_of_experts_reaches_the_library_as_none(sent, n):
    B.moe_sort(x, word(2, 1), n)
    assert not 1 <= sent[0][6] <= B.MOE_MAX_EXPERTS
    B.moe_sort(x, word(2, 1), 1024)
    assert sent[1][6] == 1024


@pytest.mark.parametrize("wide", [2 ** 32 + 1, 2 ** 32 + 16, 2 ** 33])
def test_wide_kernel_choices_reach_the_library_as_none(sent, wide):
    B.gemm(x, q, sc, 64, kernel=wide)
    B.gemm(x, q, sc, 64, decode_splits=wide)
    B.gemm_experts(*stacked, 64, kernel=wide)
    B.gemm_experts(*stacked, 64, kernel=B.KERNEL_DECODE, tile=wide)
    assert sent[0][9] < 0 and sent[1][9] < 0 and sent[2][11] < 0 and sent[3][12] < 0
