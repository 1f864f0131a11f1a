"""Argument checks of the adapter calls: bad calls are refused on the host
before anything is enqueued (no GPU needed)."""
import ctypes

import pytest

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    import weight_only_quantization_b200 as m
    return m


def ptr(v):
    return P(v) if v else None


def struct(lib, A=256, B=256, s=None, sa=0, sb=0, count=2, rank=8, dtype=0):
    return lib._CAdapters(A or None, B or None, s, sa, sb, count, rank, dtype)


def forward(lib, ad, X=256, M=4, packed=256, scale=256, zero=256, zq=None, sq=None, rows=64,
            cols=128, nbits=4, group=64, index=256, Y=256, status=None, ws=256, wsb=1 << 20):
    r = lambda m: None if m is None else ctypes.byref(m)  # noqa: E731
    return lib._lib.hqq_linear_adapters(ptr(X), M, ptr(packed), ptr(scale), ptr(zero), r(zq),
                                        r(sq), rows, cols, nbits, group, r(ad), ptr(index),
                                        ptr(Y), ptr(status), ptr(ws), wsb, None)


def backward(lib, ad, dY=256, X=256, M=4, packed=256, scale=256, zero=256, zq=None, sq=None,
             rows=64, cols=128, nbits=4, group=64, index=256, dX=256, dA=256, dB=256, status=None,
             ws=256, wsb=1 << 20):
    r = lambda m: None if m is None else ctypes.byref(m)  # noqa: E731
    return lib._lib.hqq_linear_adapters_backward(
        ptr(dY), ptr(X), M, ptr(packed), ptr(scale), ptr(zero), r(zq), r(sq), rows, cols, nbits,
        group, r(ad), ptr(index), ptr(dX), ptr(dA), ptr(dB), ptr(status), ptr(ws), wsb, None)


SHARED = [
    (dict(M=-1), 2), (dict(M=1 << 31), 2), (dict(rows=-1), 2), (dict(cols=130), 2),
    (dict(rows=65535 * 128 + 1), 2), (dict(cols=65536 * 128), 2), (dict(nbits=5), 3),
    (dict(group=48), 3), (dict(packed=0), 1), (dict(scale=0), 1), (dict(zero=0), 1),
    (dict(ws=0), 1), (dict(packed=258), 5), (dict(scale=257), 5), (dict(zero=257), 5),
    (dict(X=264), 5), (dict(index=258), 5), (dict(status=258), 5), (dict(ws=384), 5),
    (dict(wsb=16), 4),
]
STRUCTS = [
    (dict(dtype=3), 3), (dict(dtype=-1), 3), (dict(rank=0), 4), (dict(rank=513), 4),
    (dict(count=0), 4), (dict(count=65536), 4), (dict(sa=-1), 2), (dict(sa=8 * 128 - 1), 2),
    (dict(sb=8 * 64 - 1), 2), (dict(A=0), 1), (dict(B=0), 1), (dict(A=257), 5),
    (dict(B=258, dtype=2), 5), (dict(s=258), 5),
]


@pytest.mark.parametrize("kw,want", SHARED + [(dict(X=0), 1), (dict(Y=0), 1), (dict(Y=257), 5)])
def test_forward_refusals(lib, kw, want):
    assert forward(lib, struct(lib), **kw) == want


@pytest.mark.parametrize("kw,want", SHARED + [
    (dict(X=0), 1), (dict(dY=0), 1), (dict(dY=264), 5), (dict(dX=257), 5), (dict(dA=258), 5),
    (dict(dB=258), 5), (dict(dX=0, dA=0, dB=0), 0)])
def test_backward_refusals(lib, kw, want):
    assert backward(lib, struct(lib), **kw) == want


@pytest.mark.parametrize("kw,want", STRUCTS)
def test_struct_refusals(lib, kw, want):
    assert forward(lib, struct(lib, **kw)) == want
    assert backward(lib, struct(lib, **kw)) == want


def test_other_refusals(lib):
    ad = struct(lib)
    good = lib._CMeta8(256, 256, 256, 0)
    bad = lib._CMeta8(256, 256, 256, 96)
    none = lib._CMeta8(None, 256, 256, 0)
    for call in (forward, backward):
        assert call(lib, ad, zq=good) == 4                   # both forms of a pair
        assert call(lib, ad, sq=good) == 4
        assert call(lib, ad, zero=0, zq=bad) == 3
        assert call(lib, ad, zero=0, zq=none) == 1
        assert call(lib, ad, M=0, X=0, packed=0, ws=0, **({"Y": 0} if call is forward else
                    {"dY": 0, "dX": 0, "dA": 0, "dB": 0})) == 0
    assert forward(lib, None) == 1
    # a backward call without adapters takes nothing that belongs to them
    for kw in (dict(index=0, X=0, dA=0), dict(index=0, X=0, dB=0), dict(index=0, dA=0, dB=0),
               dict(X=0, dA=0, dB=0)):
        assert backward(lib, None, **kw) == 4
    assert backward(lib, None, X=0, index=0, dA=0, dB=0, dY=0, ws=0) == 1


def test_workspace_bytes(lib):
    f = lib._lib.hqq_linear_adapters_workspace_bytes
    assert f(0, 64, 128, 8, 2, 0) == 0
    assert f(4, 64, 128, 8, 2, 0) == 256
    assert f(100, 64, 128, 17, 2, 0) == 100 * 32 * 4
    assert f(4, 64, 128, 8, 2, 1) == 2 * 256 + 2 * 256
    assert f(4, 65, 128, 8, 2, 1) == f(4, 64, 128, 8, 2, 1) + 768    # dY with padded rows
    assert f(4, 64, 128, 0, 0, 1) == 0
    for bad in ((-1, 64, 128, 8, 2, 0), (4, -1, 128, 8, 2, 0), (4, 64, -1, 8, 2, 1),
                (4, 64, 128, 0, 2, 0), (4, 64, 128, 513, 2, 0), (4, 64, 128, 8, 0, 0),
                (4, 64, 128, 8, 65536, 1), (4, 64, 128, -1, 1, 1)):
        assert f(*bad) == -1


def test_binding_refusals(lib):
    """No CPU path, and shapes and types are checked before the library is called."""
    torch = pytest.importorskip("torch")
    q = lib.QuantizedMatrix(torch.zeros(64 * 128 // 2, dtype=torch.uint8),
                            torch.zeros(64, 2, dtype=torch.float16),
                            torch.zeros(64, 2, dtype=torch.float16), 64, 128, 4, 64)
    ad = lib.Adapters(torch.zeros(2, 8, 128).half(), torch.zeros(2, 64, 8).half())
    X, dY = torch.zeros(3, 128).half(), torch.zeros(3, 64).half()
    index = torch.zeros(3, dtype=torch.int32)
    for bad in (dict(), dict(index=index), dict(index=index.long())):
        with pytest.raises(ValueError):
            lib.hqq_linear_adapters(X, q, ad, **bad)
        with pytest.raises(ValueError):
            lib.hqq_linear_adapters_backward(dY, X, q, ad, **bad)
    with pytest.raises(ValueError):
        lib.hqq_linear_adapters(X.float(), q, ad)
    with pytest.raises(ValueError):
        lib.hqq_linear_adapters_backward(dY, None, q, ad)
    with pytest.raises(ValueError):
        lib.hqq_linear_adapters_backward(dY, None, q, index=index)
