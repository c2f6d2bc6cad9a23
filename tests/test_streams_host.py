"""How the binding takes its stream= argument, without a device."""
import ctypes

import pytest
import torch

from int4_weight_only_gptq_b200 import binding as B

CALLS = {
    "moe_sort": ("x", "expert_ids", 4),
    "moe_combine": ("y_sorted", "dest"),
    "moe_combine_backward": ("dout", "y_sorted", "dest", "weights"),
    "gemm_experts": ("x_sorted", "qweight", "scales", "offsets", 32),
    "gemm_experts_dx": ("dy_sorted", "qweight", "scales", "offsets", 32),
    "gemm": ("x", "qweight", "scales", 32),
    "gemm_grouped": ("x", ["qweight"], ["scales"], 32),
    "gemm_asym": ("x", "qweight", "scales", "qzeros", 32),
    "gemm_gidx": ("x", "qweight", "scales", "g_idx"),
    "gemm_lora": ("x", "qweight", "scales", 32, "lora_a", "lora_b"),
    "gemm_lora_noalloc": ("x", "qweight", "scales", 32, "lora_a", "lora_b"),
    "dequant": ("qweight", "scales", 32),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("stream", [0, 12345, ctypes.c_void_p(64)])
def test_raw_handles_take_the_path_of_streams(name, stream, monkeypatch):
    """A handle, too, moves what a call allocates to its stream."""
    fn, seen = getattr(B, name), []
    monkeypatch.setattr(B, "_on_stream", lambda f, s, *args: seen.append((f, s, args)))
    fn(*CALLS[name], **{"outs" if name == "gemm_grouped" else "out": "out"}, stream=stream)
    (f, s, args), = seen
    assert f is fn and s is stream
    assert args[:len(CALLS[name])] == CALLS[name] and "out" in args


def test_handles_become_streams(monkeypatch):
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device: ("external", h, device))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: ("default", device))
    dev = torch.device("cuda", 0)
    # both names of the legacy default stream; a null handle must not become a
    # new stream
    for handle in (0, 1, ctypes.c_void_p(), ctypes.c_void_p(1)):
        assert B._torch_stream(handle, dev) == ("default", dev)
    assert B._torch_stream(2, dev) == ("external", 2, dev)
    assert B._torch_stream(ctypes.c_void_p(0x5500), dev) == ("external", 0x5500, dev)
    with pytest.raises(TypeError):
        B._torch_stream(object(), dev)


def test_a_stream_does_not_hide_a_refusal():
    x, ids = torch.zeros(2, 64, dtype=torch.float16), torch.zeros(2, 1, dtype=torch.int32)
    for stream in (0, 12345):
        with pytest.raises(ValueError):
            B.moe_sort(x, ids, 4, stream=stream)
        with pytest.raises(TypeError):
            B.moe_combine(None, ids, stream=stream)
