"""Host-side checks of the norm's, microscaled products' and sampling's entry points (no GPU needed)."""
import ctypes
import os

import pytest

from quantized_moe_decode_affine_amd import binding as B

A = [0x10000000 * i for i in range(1, 12)]   # fake, well-aligned device addresses: never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B._LIB_PATH):
        from quantized_moe_decode_affine_amd import build
        build.build()
    return B.load_library()


def test_rms_norm_rejects(lib):
    f = lib.rms_norm

    def call(x=A[0], r=A[1], w=A[2], rows=4, k=128, eps=1e-6, total=A[3], y=A[4], codes=A[5], scales=A[6]):
        return f(x, r, w, rows, k, eps, total, y, codes, scales, None)

    for bad in (dict(x=None), dict(w=None), dict(x=A[0] + 2), dict(w=A[2] + 8), dict(rows=-1), dict(k=0), dict(k=12),
                dict(r=None), dict(total=None), dict(codes=None), dict(scales=None),
                dict(y=None, codes=None, scales=None), dict(r=A[1] + 4), dict(total=A[3] + 4), dict(y=A[4] + 4),
                dict(codes=A[5] + 8), dict(scales=A[6] + 2), dict(eps=0.0), dict(eps=-1.0), dict(eps=1e-39),
                dict(eps=float("nan")), dict(eps=float("inf"))):
        assert call(**bad) == B.EINVAL, bad
    assert call(k=65544) == B.EUNSUPPORTED
    assert call(rows=1 << 31) == B.EUNSUPPORTED
    n = 4 * 128 * 2
    for bad in (dict(y=A[0]), dict(y=A[1]), dict(y=A[2]), dict(y=A[3]), dict(codes=A[4]), dict(scales=A[5]),
                dict(scales=A[0]), dict(codes=A[3] + n - 16), dict(total=A[0] + 16), dict(total=A[1] + 16),
                dict(total=A[2]), dict(total=A[0], r=A[0] + 512), dict(y=A[2] + 240)):
        assert call(**bad) == B.EINVAL, bad
    assert call(rows=0) == B.OK


def test_i8_gemm_rows_rejects(lib):
    f = lib.i8_gemm_rows
    W = lambda **o: ctypes.byref(B.q4moe_i8_matrix(*{**dict(c=A[0], s=A[1], count=1, n=64, k=128), **o}.values()))  # noqa: E731
    for W_, c, s, m, y, out in ((None, A[2], A[3], 4, A[4], 0), (W(k=100), A[2], A[3], 4, A[4], 0), (W(), None, A[3], 4, A[4], 0),
                                (W(), A[2] + 8, A[3], 4, A[4], 0), (W(), A[2], None, 4, A[4], 0), (W(), A[2], A[3] + 2, 4, A[4], 0),
                                (W(), A[2], A[3], -1, A[4], 0), (W(), A[2], A[3], 4, None, 0), (W(), A[2], A[3], 4, A[4], 2),
                                (W(), A[2], A[3], 4, A[2], 0), (W(), A[2], A[3], 4, A[3] - 16, 0)):
        assert f(W_, c, s, m, y, out, None) == B.EINVAL
    assert f(W(k=131072), A[2], A[3], 4, A[4], 0, None) == B.EUNSUPPORTED
    assert f(W(), A[2], A[3], 0, A[4], 0, None) == B.OK
