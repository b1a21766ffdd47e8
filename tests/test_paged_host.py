"""Host-only checks of the paged cache's calls: refusals of the C ABI (fake addresses that are never read, since
validation fails first) and of the Python binding (a library that fails the test if any call gets through)."""
import pytest
import torch

from hadamard_rotated_int8_b200 import _build, _native

A = 0x10000        # aligned fake address
MIS = 0x10002
NULL, SHAPE, ALIGN, UNSUP = (_native.SDNQ_ERR_NULL, _native.SDNQ_ERR_SHAPE, _native.SDNQ_ERR_ALIGN,
                             _native.SDNQ_ERR_UNSUPPORTED)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return _native.lib()


def write(lib, k=A, ldk=1024, v=A, ldv=1024, slots=A, T=4, Hkv=8, D=128, group=256, codes=A, scales=A, pages=9,
          page=16):
    return lib.sdnq_kv_write(k, ldk, v, ldv, slots, T, Hkv, D, group, codes, scales, pages, page, 0)


def read(lib, k=A, ldk=1024, v=A, ldv=1024, slots=A, T=4, Hkv=8, D=128, group=256, codes=A, scales=A, pages=9,
         page=16):
    return lib.sdnq_kv_read(slots, T, codes, scales, pages, page, Hkv, D, group, k, ldk, v, ldv, 0)


@pytest.mark.parametrize("over,want", [
    (dict(k=0), NULL), (dict(v=0), NULL), (dict(slots=0), NULL), (dict(codes=0), NULL), (dict(scales=0), NULL),
    (dict(T=-1), SHAPE), (dict(T=1 << 31), SHAPE), (dict(Hkv=0), SHAPE), (dict(Hkv=70000), SHAPE),
    (dict(pages=-1), SHAPE), (dict(pages=1 << 24), SHAPE), (dict(ldk=1016), SHAPE), (dict(ldv=0), SHAPE),
    (dict(D=96), UNSUP), (dict(D=256), UNSUP), (dict(page=8), UNSUP), (dict(page=48), UNSUP),
    (dict(page=512), UNSUP), (dict(group=4), UNSUP), (dict(group=512), UNSUP), (dict(group=24), UNSUP),
    (dict(ldk=1028), ALIGN), (dict(ldv=1028), ALIGN), (dict(k=MIS), ALIGN), (dict(v=A + 8), ALIGN),
    (dict(slots=A + 4), ALIGN), (dict(codes=A + 8), ALIGN), (dict(scales=A + 4), ALIGN),
])
def test_cache_calls_refuse(lib, over, want):
    assert write(lib, **over) == want
    assert read(lib, **over) == want


def attn(lib, q=A, ldq=4096, T=8, H=32, cu=A, lens=A, B=4, table=A, max_pages=10, ldt=10, codes=A, scales=A,
         pages=99, page=16, Hkv=8, D=128, max_q=8, group=256, scale=0.1, window=0, sinks=0, ws=A, ws_bytes=1 << 40,
         out=A, ldo=4096):
    return lib.sdnq_attention_paged(q, ldq, T, H, cu, lens, B, table, max_pages, ldt, codes, scales, pages, page,
                                    Hkv, D, max_q, group, scale, window, sinks, ws, ws_bytes, out, ldo, 0)


@pytest.mark.parametrize("over,want", [
    (dict(q=0), NULL), (dict(lens=0), NULL), (dict(table=0), NULL), (dict(codes=0), NULL), (dict(scales=0), NULL),
    (dict(out=0), NULL), (dict(ws=0), NULL),
    (dict(T=-1), SHAPE), (dict(B=-1), SHAPE), (dict(B=(1 << 31) - 1), SHAPE), (dict(H=0), SHAPE), (dict(H=30), SHAPE),
    (dict(H=70000), SHAPE), (dict(T=1 << 27, H=32), SHAPE), (dict(max_q=0), SHAPE), (dict(window=-1), SHAPE),
    (dict(sinks=-1), SHAPE), (dict(max_pages=-1, ldt=0), SHAPE), (dict(ldt=9), SHAPE),
    (dict(max_pages=1 << 27, ldt=1 << 27), SHAPE), (dict(cu=0, T=3), SHAPE), (dict(ldq=4088), SHAPE),
    (dict(ldo=4088), SHAPE), (dict(ws_bytes=100), SHAPE),
    (dict(scale=-1.0), UNSUP), (dict(scale=float("nan")), UNSUP), (dict(scale=float("inf")), UNSUP),
    (dict(D=80, ldq=1 << 20, ldo=1 << 20), UNSUP), (dict(page=24), UNSUP), (dict(group=2), UNSUP),
    (dict(q=A + 8), ALIGN), (dict(out=MIS), ALIGN), (dict(ldq=4100), ALIGN), (dict(ldo=4100), ALIGN),
    (dict(cu=MIS), ALIGN), (dict(lens=MIS), ALIGN), (dict(table=MIS), ALIGN), (dict(ws=A + 128), ALIGN),
    (dict(codes=MIS), ALIGN), (dict(scales=A + 4), ALIGN),
])
def test_attention_refuses(lib, over, want):
    assert attn(lib, **over) == want


def test_workspace(lib):
    assert lib.sdnq_attention_paged_workspace(32, 8, 128) > 0
    for bad in ((0, 1, 128), (4, 0, 128), (5, 2, 128), (4, 2, 96), (-4, -2, 64)):
        assert lib.sdnq_attention_paged_workspace(*bad) == -1


class _NoLibrary:
    def __getattr__(self, name):
        if name == "sdnq_attention_paged_workspace":
            return lambda *a: 4096
        raise AssertionError(f"{name} reached the library despite invalid arguments")


@pytest.fixture
def no_library(monkeypatch):
    monkeypatch.setattr(_native, "lib", lambda: _NoLibrary())
    monkeypatch.setattr(_native, "_on_current_device", lambda t, name: None)
    monkeypatch.setattr(_native, "_paged_ws_bytes", {})


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def i64(*shape):
    return torch.zeros(shape, dtype=torch.int64)


CODES, SCALES = torch.zeros(3, 2, 2, 16, 64, dtype=torch.int8), torch.zeros(3, 2, 2, 16)


@pytest.mark.parametrize("over,err", [
    (dict(k=bf(5, 2, 32)), ValueError), (dict(k=bf(5, 3, 64), v=bf(5, 3, 64)), ValueError),
    (dict(v=bf(4, 2, 64)), ValueError), (dict(k=bf(5, 2, 64).float()), TypeError),
    (dict(v=bf(5, 2, 64).half()), TypeError), (dict(k=bf(5, 128)), ValueError),
    (dict(k=bf(5, 64, 2).transpose(1, 2)), ValueError), (dict(k=bf(5, 4, 64)[:, ::2]), ValueError),
    (dict(slots=i32(5)), TypeError), (dict(slots=i64(4)), ValueError), (dict(slots=i64(6)), ValueError),
    (dict(slots=i64(5, 1)), ValueError), (dict(slots=i64(10)[::2]), ValueError), (dict(slots=None), ValueError),
    (dict(codes=CODES.to(torch.uint8)), TypeError), (dict(codes=CODES[:, :, :1]), ValueError),
    (dict(codes=CODES[:, :1]), ValueError), (dict(codes=CODES[0]), ValueError),
    (dict(scales=SCALES.double()), TypeError), (dict(scales=SCALES[:2]), ValueError),
    (dict(scales=SCALES[..., :8]), ValueError),
])
def test_write_binding_refuses(no_library, over, err):
    a = dict(k=bf(5, 2, 64), v=bf(5, 2, 64), slots=i64(5), codes=CODES, scales=SCALES)
    a.update(over)
    with pytest.raises(err):
        _native.sdnq_kv_write(**a)


@pytest.mark.parametrize("over,err", [
    (dict(slots=i32(5)), TypeError), (dict(slots=i64(5, 1)), ValueError), (dict(k=bf(4, 2, 64)), ValueError),
    (dict(v=bf(5, 1, 64)), ValueError), (dict(k=bf(5, 2, 64).float()), TypeError),
    (dict(codes=CODES.float()), TypeError), (dict(scales=SCALES[:, :1]), ValueError),
])
def test_read_binding_refuses(no_library, over, err):
    a = dict(slots=i64(5), codes=CODES, scales=SCALES, k=bf(5, 2, 64), v=bf(5, 2, 64))
    a.update(over)
    with pytest.raises(err):
        _native.sdnq_kv_read(**a)


@pytest.mark.parametrize("over,err", [
    (dict(q=bf(6, 4, 32)), ValueError), (dict(q=bf(6, 5, 64)), ValueError), (dict(q=bf(6, 4, 64).float()), TypeError),
    (dict(q=bf(6, 8, 64)[:, ::2]), ValueError), (dict(table=i64(3, 7)), TypeError), (dict(table=i32(21)), ValueError),
    (dict(table=i32(7, 3).t()), ValueError), (dict(table=i32(1, 7).expand(3, 7)), ValueError),
    (dict(lens=i32(2)), ValueError), (dict(lens=i32(4)), ValueError), (dict(lens=i64(3)), TypeError),
    (dict(cu_q=i32(3)), ValueError), (dict(cu_q=i32(5)), ValueError), (dict(cu_q=i64(4)), TypeError),
    (dict(cu_q=None), ValueError), (dict(ws=torch.zeros(4095, dtype=torch.uint8)), ValueError),
    (dict(ws=torch.zeros(4096, dtype=torch.int8)), TypeError), (dict(out=bf(5, 4, 64)), ValueError),
    (dict(out=bf(6, 4, 64).half()), TypeError), (dict(codes=CODES[:, :, :, :8]), ValueError),
    (dict(scales=SCALES.half()), TypeError),
])
def test_attention_binding_refuses(no_library, over, err):
    a = dict(q=bf(6, 4, 64), codes=CODES, scales=SCALES, table=i32(3, 7), lens=i32(3), cu_q=i32(4), max_q=2,
             ws=torch.zeros(4096, dtype=torch.uint8), out=bf(6, 4, 64))
    a.update(over)
    with pytest.raises(err):
        _native.sdnq_attention_paged(**a)
