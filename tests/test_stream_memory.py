"""Memory that the binding makes for a call on a given stream (CPU only). It has to come from that stream's share of
torch's allocator: a block of the current stream may still be in use there by work that the given stream does not wait
for, such as the call before with the same workspace size. What goes back to the caller is also recorded on the
current stream. The library, the streams and the allocator are fakes; CPU tensors stand in for device tensors."""
import contextlib

import pytest
import torch

import hadamard_rotated_int8_b200 as sd
from hadamard_rotated_int8_b200 import _native

HERE, SIDE = "current", "side"


class _Library:
    def __getattr__(self, name):
        return lambda *a: 4096 if name.endswith("_workspace") else 0


@pytest.fixture
def made(monkeypatch):
    """[(tensor, stream it was made on)] of what the binding makes, the tensors of the caller, and {data pointer:
    streams it was recorded on}."""
    active, log, given, used = [HERE], [], [], {}

    @contextlib.contextmanager
    def on(stream):
        active.append(stream)
        yield
        active.pop()

    monkeypatch.setattr(_native, "lib", lambda: _Library())
    monkeypatch.setattr(_native, "_on_current_device", lambda t, name: None)
    monkeypatch.setattr(_native, "_paged_ws_bytes", {})
    monkeypatch.setattr(_native, "_SYNC_CACHE", {})
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: active[-1])
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, *a, **kw: {7: SIDE}[handle])
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: used.setdefault(t.data_ptr(), set()).add(s), raising=False)
    empty, zeros = torch.empty, torch.zeros

    def make_empty(*a, **kw):
        log.append((empty(*a, **kw), active[-1]))
        return log[-1][0]

    def make_zeros(shape, **kw):         # the callers below give no device
        t = zeros(shape, **kw)
        log.append((t, active[-1])) if "device" in kw else given.append(t)
        return t

    monkeypatch.setattr(torch, "empty", make_empty)
    monkeypatch.setattr(torch, "empty_like", lambda t: make_empty(t.shape, dtype=t.dtype))
    monkeypatch.setattr(torch, "zeros", make_zeros)
    return log, given, used


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def t8(*shape):
    return torch.zeros(shape, dtype=torch.int8)


def f32(*shape):
    return torch.zeros(shape, dtype=torch.float32)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


M, N, K, R = 8, 20, 64, 16
CODES, SCALES = t8(3, 2, 2, 16, 64), f32(3, 2, 2, 16)
SLOTS = torch.zeros(5, dtype=torch.int64)

CALLS = {
    "attention_paged": lambda: sd.sdnq_attention_paged(bf(3, 4, 64), CODES, SCALES, i32(3, 7), i32(3), stream=7),
    "attention_paged_given_ws": lambda: sd.sdnq_attention_paged(bf(3, 4, 64), CODES, SCALES, i32(3, 7), i32(3),
                                                                ws=u8(4096), stream=7),
    "attention_paged_given_out": lambda: sd.sdnq_attention_paged(bf(3, 4, 64), CODES, SCALES, i32(3, 7), i32(3),
                                                                 out=bf(3, 4, 64), stream=7),
    "kv_read": lambda: sd.sdnq_kv_read(SLOTS, CODES, SCALES, stream=7),
    "kv_read_given_k": lambda: sd.sdnq_kv_read(SLOTS, CODES, SCALES, k=bf(5, 2, 64), stream=7),
    "rotate_quant_weight": lambda: sd.sdnq_rotate_quant_weight(bf(N, K), stream=7),
    "rotquant_act": lambda: sd.sdnq_rotquant_act(bf(M, K), stream=7),
    "rotquant_fp8": lambda: sd.sdnq_rotquant_fp8(bf(M, K), 64, stream=7),
    "int8_linear": lambda: sd.sdnq_int8_linear(t8(M, K), f32(M), t8(N, K), f32(N), stream=7),
    "int8_linear_gelu": lambda: sd.sdnq_int8_linear_gelu(t8(M, K), f32(M), t8(N, K), f32(N), stream=7),
    "fp8_linear": lambda: sd.sdnq_fp8_linear(u8(M, K), f32(M), u8(N, K), f32(N), stream=7),
    "fused": lambda: sd.sdnq_int8_linear_fused(bf(M, K), 64, t8(N, K), f32(N), stream=7),
    "linear_lora": lambda: sd.linear(bf(M, K), t8(N, K), f32(N), 64, lora=(bf(K, R), bf(R, N), 1.0), stream=7),
    "lora_down": lambda: sd.sdnq_lora_down(bf(M, K), bf(K, R), stream=7),
    "lora_up": lambda: sd.sdnq_int8_linear_lora_up(t8(M, K), f32(M), t8(N, K), f32(N), None, bf(M, R), bf(R, N),
                                                   stream=7),
    "lora_noalloc": lambda: sd.sdnq_int8_linear_lora_noalloc(t8(M, K), f32(M), t8(N, K), f32(N), None, bf(M, K),
                                                             bf(K, R), bf(R, N), stream=7),
    "grad_input": lambda: sd.sdnq_int8_linear_grad_input(bf(M, N), t8(N, K), f32(N), 64, stream=7),
    "quant_grad_output": lambda: sd.sdnq_quant_grad_output(bf(M, N), f32(N), stream=7),
    "grad_input_gemm": lambda: sd.sdnq_int8_grad_input_gemm(t8(M, N), f32(M), t8(N, K), 64, stream=7),
    "gelu": lambda: sd.sdnq_gelu_bf16(bf(M, N), stream=7),
    "attention_int8qk": lambda: sd.sdnq_attention_int8qk(bf(1, 9, 2, 128), bf(1, 9, 2, 128), bf(1, 9, 2, 128),
                                                         stream=7),
    "attention_prep": lambda: _native.sdnq_attention_prep(bf(1, 9, 2, 128), bf(1, 9, 2, 128), stream=7),
    "attention_core": lambda: _native.sdnq_attention_core(bf(1, 9, 2, 128), 9, u8(4096), stream=7),
}


@pytest.mark.parametrize("name", CALLS)
def test_memory_comes_from_the_calls_stream(name, made):
    log, given, used = made
    result = CALLS[name]()
    assert log and all(stream == SIDE for _, stream in log)
    given = {t.data_ptr() for t in given}
    for t in result if isinstance(result, tuple) else (result,):
        if t.data_ptr() not in given:
            assert used.get(t.data_ptr()) == {HERE}


def test_the_default_stream_by_its_handles(monkeypatch):
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: "default")
    assert _native._torch_stream(0) == _native._torch_stream(1) == "default"
