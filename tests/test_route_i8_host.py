"""Host-side checks of the routing rules' and 8-bit products' entry points (no GPU needed)."""
import ctypes
import os

import pytest

from quantized_moe_decode_affine_amd import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

A, A2 = 0x10000000, 0x20000000          # fake, well-aligned device addresses: never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B._LIB_PATH):
        from quantized_moe_decode_affine_amd import build
        build.build()
    return B.load_library()


def _rule(**over):
    r = B.q4moe_routing(64, 128, 4, 0, 8, 4, 2, 1, 1.0, 0, None, A, B.q4moe_matrix())
    for key, v in over.items():
        setattr(r, key, v)
    return ctypes.byref(r)


BAD_RULES = [dict(n_experts=0), dict(top_k=0), dict(top_k=33), dict(score=2), dict(score=-1), dict(n_groups=0),
             dict(n_groups=7), dict(top_groups=0), dict(top_groups=9), dict(top_groups=1, top_k=9), dict(group_terms=0),
             dict(group_terms=3), dict(renormalise=2), dict(scale=float("nan")), dict(scale=float("inf")),
             dict(bias=A + 2)]


def test_route_rejects(lib):
    need = lib.q4moe_workspace_bytes(B.OP_ROUTE_RULE, ctypes.byref(B.q4moe_layer(128, 0, 64, 4)), None, 10)
    f, g = lib.moe_route, lib.moe_route_logits
    for bad in BAD_RULES:
        assert f(_rule(**bad), A, 10, A2, A2, A, need, None) == B.EINVAL, bad
        assert g(_rule(**bad), A, 10, A2, A2, None) == B.EINVAL, bad
    big = dict(n_experts=2048)
    assert f(_rule(**big), A, 10, A2, A2, A, 1 << 30, None) == B.EUNSUPPORTED
    assert g(_rule(n_experts=1024, n_groups=128), A, 10, A2, A2, None) == B.EUNSUPPORTED
    assert g(_rule(n_groups=1, top_groups=1, top_k=33), A, 10, A2, A2, None) == B.EUNSUPPORTED
    assert g(_rule(), A, 1 << 31, A2, A2, None) == B.EUNSUPPORTED
    assert f(_rule(), A, (1 << 26) + 1, A2, A2, A, 1 << 60, None) == B.EUNSUPPORTED
    assert f(None, A, 10, A2, A2, A, need, None) == B.EINVAL
    for bad in (dict(hidden=100), dict(hidden=0), dict(router=None), dict(router=A + 8)):
        assert f(_rule(**bad), A, 10, A2, A2, A, need, None) == B.EINVAL, bad
    assert f(_rule(hidden=32768), A, 10, A2, A2, A, need, None) == B.EUNSUPPORTED
    q4 = B.q4moe_matrix(A, A2, A2, 1, 64, 128, 4)
    assert f(_rule(router_q8=q4), A, 10, A2, A2, A, need, None) == B.EINVAL          # 4-bit codes
    q8 = B.q4moe_matrix(A, A2, A2, 1, 63, 128, 8)
    assert f(_rule(router_q8=q8), A, 10, A2, A2, A, need, None) == B.EINVAL          # rows
    assert f(_rule(), A + 2, 10, A2, A2, A, need, None) == B.EINVAL
    assert f(_rule(), A, 10, None, A2, A, need, None) == B.EINVAL
    assert f(_rule(), A, 10, A2, None, A, need, None) == B.EINVAL
    assert f(_rule(), A, 10, A2 + 2, A2, A, need, None) == B.EINVAL
    assert f(_rule(), A, -1, A2, A2, A, need, None) == B.EINVAL
    assert f(_rule(), A, 10, A2, A2, A, need - 1, None) == B.EWORKSPACE
    assert f(_rule(), A, 10, A2, A2, A + 16, need, None) == B.EWORKSPACE
    assert f(_rule(), A, 0, A2, A2, None, 0, None) == B.OK
    assert g(_rule(router=None, hidden=0), None, 10, A2, A2, None) == B.EINVAL
    assert g(_rule(router=None, hidden=0), A, 0, A2, A2, None) == B.OK


def _mat(count=1, n=64, k=128, codes=A, scales=A2):
    return B.q4moe_i8_matrix(codes, scales, count, n, k)


def test_quantize_rejects(lib):
    f = lib.i8_quantize
    assert f(A, 4, 100, A2, A2 + 0x1000, None) == B.EINVAL                           # k % 64
    assert f(A, 4, 65536 + 64, A2, A2 + 0x100000, None) == B.EUNSUPPORTED
    assert f(A + 2, 4, 64, A2, A2 + 0x1000, None) == B.EINVAL
    assert f(A, 4, 64, A2 + 4, A2 + 0x1000, None) == B.EINVAL
    assert f(A, 4, 64, A2, A2 + 0x1002, None) == B.EINVAL
    assert f(A, 4, 64, A, A2, None) == B.EINVAL                                      # codes over X
    assert f(A, 4, 64, A2, A2 + 128, None) == B.EINVAL                               # scales over codes
    assert f(A, -1, 64, A2, A2 + 0x1000, None) == B.EINVAL
    assert f(A, 0, 64, A2, A2 + 0x1000, None) == B.OK


def test_i8_gemm_rejects(lib):
    W = ctypes.byref(_mat())
    need = lib.i8_gemm_workspace_bytes(W, 100)
    assert need >= 100 * 128
    Y = A + 0x1000000
    f = lib.i8_gemm
    for bad in (_mat(k=100), _mat(k=0), _mat(n=0), _mat(count=0), _mat(codes=A + 4), _mat(scales=A2 + 2), _mat(codes=None),
                _mat(scales=None)):
        assert f(ctypes.byref(bad), A, 100, Y, 0, A2, need, None) == B.EINVAL
        assert lib.i8_gemm_workspace_bytes(ctypes.byref(bad), 100) == 0
    for big in (_mat(k=65600), _mat(count=2, n=1 << 30), _mat(count=1 << 40, n=1 << 40), _mat(n=1 << 31)):
        assert f(ctypes.byref(big), A, 100, Y, 0, A2, 1 << 60, None) == B.EUNSUPPORTED
    assert f(None, A, 100, Y, 0, A2, need, None) == B.EINVAL
    assert f(W, A + 2, 100, Y, 0, A2, need, None) == B.EINVAL
    assert f(W, A, 100, Y + 4, 0, A2, need, None) == B.EINVAL
    assert f(W, A, 100, Y, B.OUT_BF16_RESIDUAL, A2, need, None) == B.EINVAL
    assert f(W, A, -1, Y, 0, A2, need, None) == B.EINVAL
    assert f(W, A, 100, A + 256, 0, A2, need, None) == B.EINVAL                      # Y over X
    assert f(W, A, 1 << 31, Y, 0, A2, 1 << 60, None) == B.EUNSUPPORTED
    # more tiles than a grid holds
    assert f(ctypes.byref(_mat(n=1 << 30)), A, 1 << 20, Y, 0, A2, 1 << 60, None) == B.EUNSUPPORTED
    assert f(W, A, 100, Y, 0, None, need, None) == B.EWORKSPACE
    assert f(W, A, 100, Y, 0, A2, need - 1, None) == B.EWORKSPACE
    assert f(W, A, 100, Y, 0, A2 + 16, need, None) == B.EWORKSPACE
    assert f(W, A, 0, Y, 0, None, 0, None) == B.OK


def _experts(E=4, H=128, I=64, shared=True, **over):
    L = B.q4moe_i8_experts(H, I, E, 0, _mat(E, I, H), _mat(E, I, H), _mat(E, H, I),
                           *([_mat(1, I, H), _mat(1, I, H), _mat(1, H, I)] if shared else [B.q4moe_i8_matrix()] * 3))
    for key, v in over.items():
        setattr(L, key, v)
    return L


def test_experts_rejects(lib):
    good = ctypes.byref(_experts())
    need = lib.moe_experts_i8_workspace_bytes(good, 10, 2)
    Y, I, Wt = A + 0x1000000, A + 0x2000000, A + 0x3000000
    f = lib.moe_experts_i8
    assert need > lib.moe_experts_i8_workspace_bytes(ctypes.byref(_experts(shared=False)), 10, 2) > 0
    for bad in (_experts(hidden=100), _experts(inter=0), _experts(n_experts=0), _experts(up=_mat(4, 64, 64)),
                _experts(down=_mat(4, 64, 128)), _experts(sh_up=_mat(2, 64, 128)), _experts(gate=_mat(4, 64, 128, codes=A + 8)),
                _experts(sh_down=_mat(1, 128, 64, scales=None))):
        assert f(ctypes.byref(bad), A, 10, I, Wt, 2, Y, 0, A2, need, None) == B.EINVAL
        assert lib.moe_experts_i8_workspace_bytes(ctypes.byref(bad), 10, 2) == 0
    assert f(ctypes.byref(_experts(E=1025)), A, 10, I, Wt, 2, Y, 0, A2, 1 << 40, None) == B.EUNSUPPORTED
    assert f(ctypes.byref(_experts(H=16384 + 64)), A, 10, I, Wt, 2, Y, 0, A2, 1 << 40, None) == B.EUNSUPPORTED
    # 2^18 tokens of 16,384 columns: the offsets of gathered rows
    assert f(ctypes.byref(_experts(H=16384)), A, 1 << 18, I, Wt, 2, Y, 0, A2, 1 << 60, None) == B.EUNSUPPORTED
    # and the tiles of a grid
    assert f(ctypes.byref(_experts(I=16384)), A, 1 << 22, I, Wt, 2, Y, 0, A2, 1 << 60, None) == B.EUNSUPPORTED
    assert f(good, A, 10, I, Wt, 33, Y, 0, A2, 1 << 40, None) == B.EUNSUPPORTED
    assert f(good, A, 1 << 30, I, Wt, 2, Y, 0, A2, 1 << 60, None) == B.EUNSUPPORTED
    assert f(good, A, 10, I, Wt, 0, Y, 0, A2, need, None) == B.EINVAL
    assert f(good, A, -1, I, Wt, 2, Y, 0, A2, need, None) == B.EINVAL
    assert f(good, A, 10, None, Wt, 2, Y, 0, A2, need, None) == B.EINVAL
    assert f(good, A, 10, I, Wt + 2, 2, Y, 0, A2, need, None) == B.EINVAL
    assert f(good, A, 10, I, Wt, 2, Y, B.OUT_BF16_RESIDUAL, A2, need, None) == B.EINVAL
    for over in (A, I, Wt):                                                          # Y over X, ids, weights
        assert f(good, A, 10, I, Wt, 2, over, 0, A2, need, None) == B.EINVAL
    assert f(good, A, 10, I, Wt, 2, Y, 0, A2, need - 1, None) == B.EWORKSPACE
    assert f(good, A, 10, I, Wt, 2, Y, 0, A2 + 16, need, None) == B.EWORKSPACE
    assert f(good, A, 0, I, Wt, 2, Y, 0, None, 0, None) == B.OK


def test_binding_refuses_host_tensors():
    import torch
    with pytest.raises(ValueError):
        B.DeviceI8(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4))
    with pytest.raises(ValueError):
        B.i8_quantize(torch.zeros(4, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        B.Routing(torch.zeros(4, 64, dtype=torch.bfloat16), 2)
    with pytest.raises(ValueError):
        B.Routing(4, 2, score="relu")
    with pytest.raises(ValueError):
        B.moe_route_logits(B.Routing(4, 2), torch.zeros(3, 4))


def test_structs_match_header(tmp_path):
    """The ctypes structures have the header's sizes and field offsets (gcc reads the header)."""
    import shutil
    import subprocess

    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    structs = (("q4moe_i8_matrix", B.q4moe_i8_matrix), ("q4moe_i8_experts", B.q4moe_i8_experts),
               ("q4moe_routing", B.q4moe_routing))
    checks = []
    for cname, cls in structs:
        checks.append(f'printf("{cname} size %zu\\n", sizeof({cname}));')
        checks += [f'printf("{cname} {field} %zu\\n", offsetof({cname}, {field}));' for field, _ in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "q4moe.h"\nint main(void) {\n'
                   + "\n".join(checks) + "\nreturn 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run([cc, "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n")
    got = {tuple(line.split()[:2]): int(line.split()[2]) for line in out if line}
    for cname, cls in structs:
        assert got[(cname, "size")] == ctypes.sizeof(cls), cname
        for field, _ in cls._fields_:
            assert got[(cname, field)] == getattr(cls, field).offset, (cname, field)


def test_outputs_over_inputs_are_refused(lib):
    """Outputs and workspaces that share bytes with each other or with an input."""
    r, f, g, T = _rule(), lib.moe_route, lib.moe_route_logits, 10
    need = lib.q4moe_workspace_bytes(B.OP_ROUTE_RULE, ctypes.byref(B.q4moe_layer(128, 0, 64, 4)), None, T)
    X, ids, w, ws = A, A + 0x100000, A + 0x200000, A + 0x300000
    x_bytes, s_bytes = T * 128 * 2, T * 4 * 4
    for bad in ((X, X, w, ws), (X, ids, X + x_bytes - 4, ws), (X, ids, ids, ws), (X, ids, ids + s_bytes - 4, ws),
                (X, ws + 512, w, ws), (X, ids, ws, ws), (ws + 256, ids, w, ws)):
        assert f(r, bad[0], T, bad[1], bad[2], bad[3], need, None) == B.EINVAL, bad
    l_bytes = T * 64 * 4
    for bad in ((X, X, w), (X, ids, X), (X, ids, X + l_bytes - 4), (X, X - s_bytes + 4, w), (X, ids, ids)):
        assert g(r, bad[0], T, bad[1], bad[2], None) == B.EINVAL, bad
    W = ctypes.byref(_mat())
    need = lib.i8_gemm_workspace_bytes(W, 100)
    Y = A + 0x100000
    for over in (A, A + 256 * 99, Y, Y + 256 * 99):
        assert lib.i8_gemm(W, A, 100, Y, 0, over, need, None) == B.EINVAL
    ex = ctypes.byref(_experts())
    need = lib.moe_experts_i8_workspace_bytes(ex, T, 2)
    Y, ids, w = A + 0x1000000, A + 0x2000000, A + 0x3000000
    for over in (A, Y, ids, w):
        assert lib.moe_experts_i8(ex, A, T, ids, w, 2, Y, 0, over, need, None) == B.EINVAL


def test_dense_tiles_of_the_tested_shapes(tmp_path):
    """Which tile the rule gives each shape of the GPU tests on 256 compute units: all three are met,
    the large ones by several shapes."""
    import shutil
    import subprocess

    import tests.test_gpu_i8 as gpu

    cc = shutil.which("g++") or shutil.which("c++")
    if cc is None:
        pytest.skip("no C++ compiler")

    def shapes(test):
        return [v for mark in test.pytestmark if mark.name == "parametrize" for v in mark.args[1]]

    large = shapes(gpu.test_gemm_large_tiles)
    asked = large + [(m, n, k) for m, n, k in shapes(gpu.test_gemm_parity) if m > 16] + [(8192, 8192, 4096), (512, 2048, 2048)]
    src = tmp_path / "tiles.cpp"
    src.write_text('#include <cstdio>\n#include "i8_tiles.h"\nint main() {\n'
                   + "\n".join(f'printf("%d\\n", q4moe::i8_dense_tile({m}, {n}, 256));' for m, n, _ in asked) + "\nreturn 0;\n}\n")
    exe = tmp_path / "tiles"
    subprocess.run([cc, "-std=c++17", "-I", os.path.join(ROOT, "quantized_moe_decode_affine_amd", "csrc"), str(src), "-o", str(exe)],
                   check=True)
    tiles = [int(line) for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert tiles[:len(large)] == [256, 256, 256, 128]
    assert set(tiles[len(large):-2]) == {64, 128} and tiles[-2:] == [256, 64]
