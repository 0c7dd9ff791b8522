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


def _mx(**o):
    return B.q4moe_mx4_matrix(*{**dict(c=A[0], s=A[1], count=1, n=64, k=128), **o}.values())


def test_mx4_rejects(lib):
    q, d, f = lib.mx4_quantize, lib.mx4_dequantize, lib.mx4_gemm
    for x, rows, k, c, s in ((None, 4, 128, A[1], A[2]), (A[0], 4, 128, None, A[2]), (A[0], 4, 128, A[1], None),
                             (A[0] + 8, 4, 128, A[1], A[2]), (A[0], 4, 128, A[1] + 8, A[2]), (A[0], 4, 128, A[1], A[2] + 1),
                             (A[0], -1, 128, A[1], A[2]), (A[0], 4, 96, A[1], A[2]), (A[0], 4, 0, A[1], A[2]),
                             (A[0], 4, 128, A[0] + 512, A[2]), (A[0], 4, 128, A[1], A[1] + 16), (A[0], 4, 128, A[1], A[0])):
        assert q(x, rows, k, c, s, None) == B.EINVAL
    assert q(A[0], 1, 65600, A[1], A[2], None) == q(A[0], 1 << 31, 64, A[1], A[2], None) == B.EUNSUPPORTED
    assert q(A[0], 0, 64, A[1], A[2], None) == B.OK
    bad = (dict(c=None), dict(s=None), dict(c=A[0] + 4), dict(s=A[1] + 1), dict(count=0), dict(n=0), dict(k=32), dict(k=0))
    for o in bad:
        assert d(ctypes.byref(_mx(**o)), A[2], None) == B.EINVAL, o
        assert f(ctypes.byref(_mx(**o)), A[2], 4, A[3], 0, A[4], 1 << 20, None) == B.EINVAL, o
        assert lib.mx4_gemm_workspace_bytes(ctypes.byref(_mx(**o)), 4) == 0
    assert d(ctypes.byref(_mx()), None, None) == d(ctypes.byref(_mx()), A[2] + 8, None) == B.EINVAL
    assert d(ctypes.byref(_mx()), A[0], None) == d(ctypes.byref(_mx()), A[1] - 64, None) == B.EINVAL
    assert d(ctypes.byref(_mx(k=131072)), A[2], None) == d(ctypes.byref(_mx(n=1 << 31)), A[2], None) == B.EUNSUPPORTED
    need = lib.mx4_gemm_workspace_bytes(ctypes.byref(_mx()), 40)
    assert need >= 40 * (64 + 4)
    W = ctypes.byref(_mx())
    for x, m, y, out, ws, n in ((None, 40, A[3], 0, A[4], need), (A[2] + 2, 40, A[3], 0, A[4], need), (A[2], -1, A[3], 0, A[4], need),
                                (A[2], 40, None, 0, A[4], need), (A[2], 40, A[3], 2, A[4], need), (A[2], 40, A[2] + 256, 0, A[4], need),
                                (A[2], 40, A[3], 0, A[3] + 256, need), (A[2], 40, A[3], 0, A[2], need)):
        assert f(W, x, m, y, out, ws, n, None) == B.EINVAL
    for ws, n in ((None, need), (A[4], need - 1), (A[4] + 128, need)):
        assert f(W, A[2], 40, A[3], 0, ws, n, None) == B.EWORKSPACE
    assert f(W, A[2], 0, A[3], 0, None, 0, None) == B.OK
    for o, m in ((dict(k=131072), 4), (dict(n=1 << 31), 4), (dict(count=1 << 20, n=1 << 20), 4), (dict(), 1 << 31),
                 (dict(n=1 << 30), 1 << 30)):
        assert f(ctypes.byref(_mx(**o)), A[2], m, A[3], 0, A[4], 1 << 60, None) == B.EUNSUPPORTED


def _experts(E=4, H=128, I=64, shared=True, **over):
    g, d = _mx(count=E, n=I, k=H), _mx(count=E, n=H, k=I)
    sh = (_mx(n=I, k=H), _mx(n=I, k=H), _mx(n=H, k=I)) if shared else (B.q4moe_mx4_matrix(),) * 3
    L = B.q4moe_mx4_experts(H, I, E, 0, g, g, d, *sh)
    for key, v in over.items():
        setattr(L, key, v)
    return L


def test_experts_mx4_rejects(lib):
    f, size = lib.moe_experts_mx4, lib.moe_experts_mx4_workspace_bytes
    need = size(ctypes.byref(_experts()), 10, 2)
    assert need > 0

    def call(L=None, x=A[2], T=10, ids=A[3], w=A[4], k=2, y=A[5], out=0, ws=A[6], n=need):
        return f(ctypes.byref(L if L is not None else _experts()), x, T, ids, w, k, y, out, ws, n, None)

    for L in (_experts(hidden=100), _experts(hidden=256), _experts(inter=0), _experts(n_experts=0), _experts(n_experts=5),
              _experts(gate=_mx()), _experts(down=_mx(count=4, n=64, k=128)), _experts(sh_up=_mx(n=32, k=128)),
              _experts(sh_down=B.q4moe_mx4_matrix())):
        assert call(L) == B.EINVAL and size(ctypes.byref(L), 10, 2) == 0
    for bad in (dict(x=None), dict(x=A[2] + 8), dict(T=-1), dict(ids=None), dict(ids=A[3] + 2), dict(w=None), dict(w=A[4] + 2),
                dict(k=0), dict(y=None), dict(out=2), dict(y=A[2]), dict(y=A[3] - 16), dict(y=A[4] - 16), dict(ws=A[5]),
                dict(ws=A[2]), dict(ws=A[3]), dict(ws=A[4])):
        assert call(**bad) == B.EINVAL, bad
    assert f(None, A[2], 10, A[3], A[4], 2, A[5], 0, A[6], need, None) == B.EINVAL
    for bad in (dict(ws=None), dict(n=need - 1), dict(ws=A[6] + 64)):
        assert call(**bad) == B.EWORKSPACE, bad
    assert call(k=33) == call(T=1 << 31) == call(T=1 << 30, k=32) == B.EUNSUPPORTED
    assert call(_experts(H=32768)) == call(_experts(E=2048)) == B.EUNSUPPORTED
    assert call(T=0, ws=None) == B.OK


def test_sample_rejects(lib):
    f, size = lib.sample_logits, lib.sample_logits_workspace_bytes
    need = size(4, 5000)
    assert need > 0 and size(0, 5000) == size(4, 0) == size(-1, 10) == size(4, 262145) == size(65537, 10) == 0

    def call(l=A[0], dt=0, b=4, v=5000, u=A[1], t=A[2], k=A[3], p=A[4], m=A[5], ids=A[6], probs=A[7], ws=A[8], n=need):
        return f(l, dt, b, v, u, t, k, p, m, ids, probs, ws, n, None)

    for bad in (dict(l=None), dict(l=A[0] + 2), dict(l=A[0] + 1, dt=1), dict(dt=2), dict(dt=-1), dict(b=-1), dict(v=0),
                dict(u=None), dict(u=A[1] + 2), dict(t=A[2] + 1), dict(k=A[3] + 2), dict(p=A[4] + 2), dict(m=A[5] + 2),
                dict(ids=None), dict(ids=A[6] + 2), dict(probs=A[7] + 1), dict(ids=A[1]), dict(ids=A[2]), dict(ids=A[3] + 12),
                dict(probs=A[4]), dict(probs=A[5]), dict(probs=A[6]), dict(ids=A[0]), dict(ids=A[8] + 256), dict(ws=A[0]),
                dict(ws=A[1])):
        assert call(**bad) == B.EINVAL, bad
    for bad in (dict(ws=None), dict(n=need - 1), dict(ws=A[8] + 128)):
        assert call(**bad) == B.EWORKSPACE, bad
    assert call(v=262145, n=1 << 60) == call(b=65537, n=1 << 60) == B.EUNSUPPORTED
    assert call(b=0, ws=None) == B.OK
