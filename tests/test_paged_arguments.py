"""What the binding of the paged cache's calls hands to the library, and what it refuses (CPU only: the library is a
fake, CPU tensors stand in for device tensors)."""
import pytest
import torch

import hadamard_rotated_int8_b200 as sd
from hadamard_rotated_int8_b200 import _native


@pytest.fixture
def calls(monkeypatch):
    seen = []

    class Library:
        def __getattr__(self, name):
            if name.endswith("_workspace"):
                return lambda *a: 4096
            return lambda *a: seen.append((name, a)) or 0

    monkeypatch.setattr(_native, "lib", lambda: Library())
    monkeypatch.setattr(_native, "_on_current_device", lambda t, name: None)
    monkeypatch.setattr(_native, "_paged_ws_bytes", {})
    monkeypatch.setattr(_native, "_stream_on", lambda stream, dev: 0)
    return seen


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


CODES, SCALES = torch.zeros(3, 2, 2, 16, 64, dtype=torch.int8), torch.zeros(3, 2, 2, 16)
MAX_Q = 16   # its place among the library call's arguments


@pytest.mark.parametrize("T,cu,given,want", [(3, False, None, 1), (300, True, None, 300), (0, True, None, 1),
                                             (300, True, 7, 7), (300, True, 1, 1), (3, False, 5, 5),
                                             (3, True, None, 1), (2, True, None, 1), (4, True, None, 4)])
def test_the_bound_on_new_tokens(calls, T, cu, given, want):
    """A caller who gives offsets and no bound may have chunks of up to T tokens; one with no more rows than sequences
    has single ones."""
    sd.sdnq_attention_paged(bf(T, 4, 64), CODES, SCALES, i32(3, 7), i32(3), cu_q=i32(4) if cu else None,
                            **({} if given is None else {"max_q": given}))
    (name, args), = calls
    assert name == "sdnq_attention_paged" and args[MAX_Q] == want
    assert args[2] == T and args[6] == 3 and args[15] == 64   # T, B and D, to keep the place honest


def test_more_sequences_than_the_kernels_count_are_refused():
    """The kernels count sequences in groups of 32, in 32 bits. Fake addresses: validation comes first."""
    from hadamard_rotated_int8_b200 import _build
    _build.build()
    A = 0x10000

    def attn(B):
        return _native.ctypes.CDLL(_build.LIB).sdnq_attention_paged(
            *[t(v) for t, v in zip(_native.SIGNATURES["sdnq_attention_paged"],
                                   (A, 512, 4, 4, A, A, B, A, 1, 1, A, A, 9, 16, 2, 128, 1, 256, 0.1, 0, 0, A, 1 << 40,
                                    A, 512, 0))])

    for B in ((1 << 31) - 31, (1 << 31) - 2):
        assert attn(B) == _native.SDNQ_ERR_SHAPE


def test_a_cache_without_heads_is_refused(calls):
    with pytest.raises(ValueError):
        sd.sdnq_attention_paged(bf(3, 4, 64), CODES[:, :0], SCALES[:, :0], i32(3, 7), i32(3))
    assert not calls


def test_a_table_without_columns_reaches_the_library():
    """Sequences that have no page yet: an empty tensor has no address. (Refused here for its workspace, behind the
    check of the pointers.)"""
    from hadamard_rotated_int8_b200 import _build
    _build.build()
    A = 0x10000
    args = [A, 512, 4, 4, A, A, 3, 0, 0, 0, A, A, 9, 16, 2, 128, 1, 256, 0.1, 0, 0, A, 100, A, 512, 0]
    fn = _native.ctypes.CDLL(_build.LIB).sdnq_attention_paged
    types = _native.SIGNATURES["sdnq_attention_paged"]
    assert fn(*[t(v) for t, v in zip(types, args)]) == _native.SDNQ_ERR_SHAPE
    args[8] = args[9] = 1
    assert fn(*[t(v) for t, v in zip(types, args)]) == _native.SDNQ_ERR_NULL
