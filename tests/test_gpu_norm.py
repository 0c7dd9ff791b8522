"""rms_norm and i8_gemm_rows against their 64-bit forms."""
import numpy as np
import pytest
import torch

from oracle import q4moe_oracle as qorc
from oracle import route_i8_oracle as i8orc
from oracle import step_oracle as orc
from quantized_moe_decode_affine_amd import synth

pytestmark = pytest.mark.gpu

EPS = 1e-6
# y is rounded once to bf16 from fp32 that two products of 2^-24 and a factor's 2^-24 left
Y_REL = 2.0 ** -8 + 2.0 ** -22
Y_ABS = 2.0 ** -133  # the last bit of bf16's subnormals


@pytest.fixture(scope="module")
def B():
    from quantized_moe_decode_affine_amd import binding
    assert torch.cuda.is_available()
    binding.load_library()
    return binding


def _rows(seed, m, k, scale=1.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((m, k)) * np.exp(0.7 * rng.standard_normal((m, 1))) * scale
    return synth.to_bf16_bits(x.astype(np.float32))


def _bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


def _check_y(got, y):
    g = qorc.bf16_to_f64(_bits(got))
    assert (np.abs(g - y) <= Y_REL * np.abs(y) + Y_ABS).all(), np.abs(g - y).max()


def _check_codes(codes, scales, y):
    q, s = i8orc.quantize_rows(y)
    np.testing.assert_array_equal(scales.cpu().numpy(), s)
    np.testing.assert_array_equal(codes.cpu().numpy(), q)


SHAPES = [(1, 8), (3, 64), (5, 200), (1, 512), (7, 520), (600, 1024), (600, 1000), (1, 2048), (700, 2048), (513, 2040),
          (2, 4096), (515, 4104), (3, 8192), (2, 8200), (1, 16384), (2, 16392), (1, 65536), (2, 50000), (4097, 64),
          (1, 128), (3, 128), (65, 128), (40000, 128), (9, 136), (33, 256), (5, 264), (2, 32768), (3, 32776)]


@pytest.mark.parametrize("rows,k", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm(B, rows, k, residual):
    X, w = _rows(rows + k, rows, k), _rows(k, 1, k)[0]
    R = _rows(rows * 3 + k, rows, k, 3.0) if residual else None
    t, y = orc.rms_norm(X, w, EPS, R)
    x, wt = B.bf16_tensor(X), B.bf16_tensor(w)
    r = B.bf16_tensor(R) if residual else None
    got = B.rms_norm(x, wt, EPS, residual=r)
    codes, scales, *more = B.rms_norm_i8(x, wt, EPS, residual=r)
    both = torch.empty_like(x)
    codes2, scales2, *_ = B.rms_norm_i8(x, wt, EPS, residual=r, out=both)
    assert torch.equal(codes, codes2) and torch.equal(scales, scales2)
    if residual:
        got, total = got
        np.testing.assert_array_equal(qorc.bf16_to_f64(_bits(total)), t)
        assert torch.equal(total, more[0])
    _check_y(got, y)
    _check_y(both, y)
    _check_codes(codes, scales, y)


@pytest.mark.parametrize("rows,k", [(3, 2048), (1100, 2048), (2, 20000)])
def test_total_over_an_input(B, rows, k):
    """The stream's new state written over X or over the residual: the same bits."""
    X, R, w = _rows(1, rows, k), _rows(2, rows, k), B.bf16_tensor(_rows(3, 1, k)[0])
    x, r = B.bf16_tensor(X), B.bf16_tensor(R)
    y, total = B.rms_norm(x, w, EPS, residual=r)
    for over in (0, 1):
        ins = [x.clone(), r.clone()]
        y2, t2 = B.rms_norm(ins[0], w, EPS, residual=ins[1], total=ins[over])
        assert t2 is ins[over] and torch.equal(t2, total) and torch.equal(y2, y)
        assert torch.equal(ins[1 - over], (x, r)[1 - over])


@pytest.mark.parametrize("rows,k", [(5, 128), (3, 8), (65, 256), (2, 512), (2, 1000), (1, 16392), (2, 40000)])
def test_leaves_rows_behind(B, rows, k):
    """Rows behind the last one, in every buffer that is written, stay as they were; the stream's state in place."""
    X, R, w = _rows(1, rows, k), _rows(2, rows, k), B.bf16_tensor(_rows(3, 1, k)[0])
    want = B.rms_norm_i8(B.bf16_tensor(X), w, EPS, residual=B.bf16_tensor(R))
    codes, scales = torch.full((rows + 9, k), 77, dtype=torch.int8, device="cuda"), torch.full((rows + 9,), 7.0, device="cuda")
    y, x = (torch.full((rows + 9, k), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x[:rows] = B.bf16_tensor(X)
    got = B.rms_norm_i8(x[:rows], w, EPS, residual=B.bf16_tensor(R), total=x[:rows], codes=codes[:rows], scales=scales[:rows],
                        out=y[:rows])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert (codes[rows:] == 77).all() and all((t[rows:] == 7).all() for t in (scales, y, x))


def test_extremes(B):
    k = 256
    x = np.zeros((12, k))
    x[1] = 1.0                                    # every value the same
    x[2, 5] = -3.0                                # a lone value
    x[3] = 2.0 ** -130 * (np.arange(k) % 7)       # subnormal: eps rules
    x[4] = 3e38 * (1 - np.arange(k) / 128)        # squares beyond fp32
    x[5] = 1e-20 * np.arange(k)
    x[6] = np.where(np.arange(k) % 2, 1e30, 1e-30)
    x[7] = -1.0
    w = 1 + 0.5 * np.sin(np.arange(k))
    w[17] = 0.0
    X, W = synth.to_bf16_bits(x.astype(np.float32)), synth.to_bf16_bits(w.astype(np.float32))
    X[8, 9], X[9, 100], X[10, 17], X[11, 17] = 0x7F80, 0xFFC1, 0x7F80, 0x7FC0  # the last two under a zero weight
    for eps in (1e-6, 1e-30, 1.0):
        for rows in (slice(0, 8), slice(0, 12)):
            _, y = orc.rms_norm(X[rows], W, eps)
            xt, wt = B.bf16_tensor(X[rows]), B.bf16_tensor(W)
            got = qorc.bf16_to_f64(_bits(B.rms_norm(xt, wt, eps)))
            fine = np.isfinite(y)
            assert (np.isnan(got) == np.isnan(y)).all()
            # rounding to bf16 overflows from its largest value and half a step up
            want = orc.f64_to_bf16(y)
            big = fine & np.isinf(want)
            assert (got[big] == want[big]).all()
            fine &= ~big
            assert (np.abs(got - y)[fine] <= Y_REL * np.abs(y[fine]) + Y_ABS).all()
            codes, scales = B.rms_norm_i8(xt, wt, eps)
            _check_codes(codes[:8], scales[:8], y[:8])
            assert np.isnan(scales[8:].cpu().numpy()).all() and not codes[8:].any()
    # a weight that is not finite reaches every row
    W[3] = 0x7F80
    codes, scales = B.rms_norm_i8(B.bf16_tensor(X[:8]), B.bf16_tensor(W))
    assert torch.isnan(scales).all() and not codes.any()


def test_residual_rounding_and_overflow(B):
    """Ties of the addition go to even, a sum beyond the type becomes infinite, opposite infinities NaN."""
    k = 64
    a, r = np.zeros((4, k)), np.zeros((4, k))
    a[0], r[0] = 256.0 + 2 * np.arange(k), 1.0            # a half step: to the even one
    a[1], r[1] = -(256.0 + 2 * np.arange(k)), -1.0
    a[2], r[2] = 3e38, 1e38
    Xa, Xr = synth.to_bf16_bits(a.astype(np.float32)), synth.to_bf16_bits(r.astype(np.float32))
    Xa[3, 0], Xr[3, 0] = 0x7F80, 0xFF80
    w = synth.to_bf16_bits(np.ones(k, np.float32))
    _, total = B.rms_norm(B.bf16_tensor(Xa), B.bf16_tensor(w), residual=B.bf16_tensor(Xr))
    t, _ = orc.rms_norm(Xa, w, EPS, Xr)
    np.testing.assert_array_equal(qorc.bf16_to_f64(_bits(total)), t)
    codes, scales, _ = B.rms_norm_i8(B.bf16_tensor(Xa), B.bf16_tensor(w), residual=B.bf16_tensor(Xr))
    assert torch.isnan(scales[2:]).all() and not codes[2:].any() and not torch.isnan(scales[:2]).any()


def test_rows_alone_and_in_a_batch(B):
    """A row's sums depend on how many waves share it: results stay within the one rounding, codes are equal."""
    X, w = _rows(5, 1500, 2048), B.bf16_tensor(_rows(6, 1, 2048)[0])
    x = B.bf16_tensor(X)
    codes, scales = B.rms_norm_i8(x, w)
    for r in (0, 777, 1499):
        c1, s1 = B.rms_norm_i8(x[r:r + 1], w)
        assert torch.equal(c1[0], codes[r]) and torch.equal(s1[0], scales[r])


def test_offsets_past_32_bits(B):
    rows, k = 262200, 8192  # 2^31 columns and more
    x = torch.zeros((rows, k), dtype=torch.bfloat16, device="cuda")
    last = B.bf16_tensor(_rows(7, 1, k))
    x[-1:] = last
    w = B.bf16_tensor(_rows(8, 1, k)[0])
    codes, scales = B.rms_norm_i8(x, w)
    c1, s1 = B.rms_norm_i8(last, w)
    assert torch.equal(codes[-1], c1[0]) and torch.equal(scales[-1:], s1)
    assert not codes[:-1].any() and not scales[:-1].any()
    del codes
    y = B.rms_norm(x, w)
    assert torch.equal(y[-1], B.rms_norm(last, w)[0])


@pytest.mark.parametrize("m,n,k", [(1, 16, 64), (1, 1024, 2048), (3, 100, 192), (16, 4100, 2048), (17, 70, 320), (200, 513, 1088),
                                   (16, 64, 8192), (1500, 700, 512)])
def test_gemm_rows_is_gemm(B, m, n, k):
    """The product of rows that are codes: the bits of the product that makes them."""
    rng = np.random.default_rng(m + n + k)
    W = B.DeviceI8(torch.from_numpy(rng.integers(-127, 128, (n, k), dtype=np.int8)).cuda(),
                   torch.from_numpy((rng.random(n) * 0.01 + 1e-4).astype(np.float32)).cuda())
    X = B.bf16_tensor(_rows(m, m, k))
    for out in (B.OUT_F32, B.OUT_BF16):
        assert torch.equal(B.i8_gemm_rows(W, *B.i8_quantize(X), out), B.i8_gemm(W, X, out))


def test_norm_then_product(B):
    """A norm's codes through a product, against the 64-bit forms of both."""
    rows, k, n = 33, 1088, 515
    rng = np.random.default_rng(9)
    X, R, w = _rows(1, rows, k), _rows(2, rows, k), _rows(3, 1, k)[0]
    wc, ws = rng.integers(-127, 128, (n, k), dtype=np.int8), (rng.random(n) * 0.01 + 1e-4).astype(np.float32)
    codes, scales, _ = B.rms_norm_i8(B.bf16_tensor(X), B.bf16_tensor(w), EPS, residual=B.bf16_tensor(R))
    Y = B.i8_gemm_rows(B.DeviceI8(torch.from_numpy(wc).cuda(), torch.from_numpy(ws).cuda()), codes, scales)
    q, s = i8orc.quantize_rows(orc.rms_norm(X, w, EPS, R)[1])
    ref = (q.astype(np.float64) @ wc.astype(np.float64).T) * s[:, None] * ws.astype(np.float64)
    # the exact sum becomes fp32, then two scales: three roundings
    assert (np.abs(Y.double().cpu().numpy() - ref) <= 3.01 * 2.0 ** -24 * np.abs(ref)).all()


def test_norm_graph(B):
    X, R, w = (B.bf16_tensor(_rows(s, 40, 2048)) for s in (1, 2, 3))
    w = w[0].clone()
    y, total, codes, scales = torch.empty_like(X), torch.empty_like(X), torch.empty(40, 2048, dtype=torch.int8, device="cuda"), torch.empty(40, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        B.rms_norm_i8(X, w, residual=R, total=total, codes=codes, scales=scales, out=y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.rms_norm_i8(X, w, residual=R, total=total, codes=codes, scales=scales, out=y)
    for seed in range(3):
        X.copy_(B.bf16_tensor(_rows(10 + seed, 40, 2048)))
        g.replay()
        y2 = torch.empty_like(X)
        c2, s2, t2 = B.rms_norm_i8(X, w, residual=R, out=y2)
        assert torch.equal(y, y2) and torch.equal(total, t2) and torch.equal(codes, c2) and torch.equal(scales, s2)


def test_binding_refusals(B):
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(64, dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: B.rms_norm(x.float(), w), lambda: B.rms_norm(x, w[:32]), lambda: B.rms_norm(x.T, w),
                lambda: B.rms_norm(x.cpu(), w.cpu()), lambda: B.rms_norm(x, w, residual=x[:1]),
                lambda: B.rms_norm(x, w, total=x.clone()), lambda: B.rms_norm_i8(x, w, out=x.float()),
                lambda: B.rms_norm(x, w.cpu())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: B.rms_norm(x, w, eps=0.0), lambda: B.rms_norm(x, w, out=x),
                lambda: B.rms_norm(x, w, residual=x.clone(), total=x, out=x)):
        with pytest.raises(B.Q4Error) as err:
            bad()
        assert err.value.status == B.EINVAL
    assert B.rms_norm(x[:0], w).shape == (0, 64)


@pytest.mark.parametrize("rows,k", [(5, 64), (3, 200), (4, 512), (700, 1000), (2, 2048), (3, 4104), (2, 8200), (2, 20000), (1, 40000)])
def test_range_of_values_and_weights(B, rows, k):
    """Values and weights of every size that the type has: what underflows on the way to y, but not in y, is not lost."""
    rng = np.random.default_rng(k)
    x, w = (rng.choice([-1.0, 1.0], n) * np.exp2(rng.uniform(-130, 127, n)) for n in ((rows, k), k))
    x[0] = 2.0 ** -100
    x[0, 0] = 2.0 ** 60                     # a small value beside a large one, under a large weight: 2^-160 on the way
    w[:4] = 2.0 ** 60, 2.0 ** 60, 1.0, 2.0 ** 100
    x[-1] = 3e38 * rng.uniform(0.1, 1, k)   # the norm's factor itself is below 2^-126
    for most in (2.0 ** 127, 2.0 ** 14, 2.0 ** 13.9, 1.0):
        v = np.clip(w, -most, most)
        X, W = synth.to_bf16_bits(x.astype(np.float32)), synth.to_bf16_bits(v.astype(np.float32))
        _, y = orc.rms_norm(X, W, EPS)
        xt, wt = B.bf16_tensor(X), B.bf16_tensor(W)
        both = torch.empty_like(xt)
        B.rms_norm_i8(xt, wt, EPS, out=both)
        want = orc.f64_to_bf16(y)
        big = np.isinf(want)
        for got in (B.rms_norm(xt, wt, EPS), both):
            got = qorc.bf16_to_f64(_bits(got))
            assert (got[big] == want[big]).all()
            assert (np.abs(got - y)[~big] <= Y_REL * np.abs(y[~big]) + Y_ABS).all()


@pytest.mark.parametrize("rows,k,residual", [(2500, 4096, True), (2500, 4104, False), (2100, 8192, False), (1100, 16384, True),
                                             (600, 20000, False), (600, 32768, True), (530, 65536, False), (70000, 136, True)])
def test_rows_in_turn(B, rows, k, residual):
    """More rows than workgroups, several waves to each: what a row leaves (its sums, an infinity or a NaN in one of its
    waves) does not reach the next."""
    X, w = _rows(rows + k, rows, k), _rows(k, 1, k)[0]
    R = _rows(rows * 3 + k, rows, k, 3.0) if residual else None
    bad = np.random.default_rng(k).permutation(rows)[:rows // 8]
    X[bad, (np.arange(len(bad)) * 997) % k] = np.array([0x7F80, 0xFF80, 0x7FC0], np.uint16)[np.arange(len(bad)) % 3]
    fine = np.ones(rows, dtype=bool)
    fine[bad] = False
    t, y = orc.rms_norm(X, w, EPS, R)
    x, wt = B.bf16_tensor(X), B.bf16_tensor(w)
    r = B.bf16_tensor(R) if residual else None
    codes, scales, *total = B.rms_norm_i8(x, wt, EPS, residual=r)
    one = B.rms_norm(x, wt, EPS, residual=r)
    if residual:
        assert torch.equal(total[0].view(torch.int16), one[1].view(torch.int16))
        np.testing.assert_array_equal(qorc.bf16_to_f64(_bits(total[0])), t)
        one = one[0]
    keep = torch.from_numpy(fine).cuda()
    _check_codes(codes[keep], scales[keep], y[fine])
    _check_y(one[keep], y[fine])
    assert torch.isnan(scales[~keep]).all() and not codes[~keep].any()
    got = qorc.bf16_to_f64(_bits(one[~keep]))
    assert (np.isnan(got) == np.isnan(y[~fine])).all() and (got[~np.isnan(got)] == 0).all()


@pytest.mark.parametrize("k", [512, 2048, 4096, 8192, 16384, 40000])
def test_not_finite_in_any_wave(B, k):
    """An infinity or a NaN, alone in a row or in the weights, in each eighth of the columns; a large value crosses the waves too."""
    w = synth.to_bf16_bits(np.ones(k, np.float32))
    at = np.arange(8) * (k // 8) + 3
    X = _rows(k, 24, k)
    for i, bits in enumerate((0x7F80, 0xFFC1, 0x7F00)):
        X[np.arange(8) + 8 * i, at] = bits
    for rows in (slice(0, 24), slice(8, 9), slice(23, 24)):
        _, y = orc.rms_norm(X[rows], w, EPS)
        xt, wt = B.bf16_tensor(X[rows]), B.bf16_tensor(w)
        got = qorc.bf16_to_f64(_bits(B.rms_norm(xt, wt, EPS)))
        assert (np.isnan(got) == np.isnan(y)).all()
        there = ~np.isnan(y)
        assert (np.abs(got - y)[there] <= Y_REL * np.abs(y[there]) + Y_ABS).all()
        codes, scales = B.rms_norm_i8(xt, wt, EPS)
        large = np.arange(24)[rows] >= 16
        assert torch.isnan(scales[torch.from_numpy(~large).cuda()]).all() and not codes[torch.from_numpy(~large).cuda()].any()
        if large.any():
            _check_codes(codes[torch.from_numpy(large).cuda()], scales[torch.from_numpy(large).cuda()], y[large])
    for j in at:
        v = w.copy()
        v[j] = 0x7F80
        codes, scales = B.rms_norm_i8(B.bf16_tensor(X[16:18]), B.bf16_tensor(v))
        assert torch.isnan(scales).all() and not codes.any()


@pytest.mark.parametrize("k", [256, 1000, 4096, 20000])
@pytest.mark.parametrize("eps", [1.0, 1e-6, 1e-12])
def test_codes_of_exact_halves(B, k, eps):
    """Rows so small that eps alone is under the root, the largest 127 times a weight of 8 bits: scales are exact and a
    quotient is its value, halves among them, which go to the even code."""
    q = np.concatenate([[127.0], np.resize(np.arange(-127, 127) + 0.5, k - 1)])
    x = np.where(np.arange(64)[:, None] % 2 == 0, q, -q) * 2.0 ** -100
    X = synth.to_bf16_bits(x.astype(np.float32))
    xt = B.bf16_tensor(X)
    for s in range(129, 256, 14):
        W = synth.to_bf16_bits(np.full(k, s, np.float32))
        codes, scales = B.rms_norm_i8(xt, B.bf16_tensor(W), eps)
        assert (scales.double().cpu().numpy() == s * 2.0 ** -100 * round(1 / np.sqrt(eps))).all()
        np.testing.assert_array_equal(codes.cpu().numpy(), np.rint(x * 2.0 ** 100))
        R = torch.zeros_like(xt)
        more = B.rms_norm_i8(xt.clone(), B.bf16_tensor(W), eps, residual=R)
        assert torch.equal(more[0], codes) and torch.equal(more[1], scales) and torch.equal(more[2], xt)


@pytest.mark.parametrize("k", [64, 128, 256, 512])
def test_rows_beside_rows_beyond_fp32(B, k):
    """A row's bits do not hang on the rows that share its wave: rows of 1e38 between ordinary ones, which take fp64."""
    X, w = _rows(k, 2000000 // k, k), B.bf16_tensor(_rows(k + 1, 1, k)[0])  # some hundred values differ between fp32 and fp64
    alone = B.rms_norm(B.bf16_tensor(X), w, EPS)
    X[1::3] = synth.to_bf16_bits((3e38 * np.random.default_rng(k).uniform(0.1, 1, X[1::3].shape)).astype(np.float32))
    _, y = orc.rms_norm(X, _bits(w), EPS)
    got = B.rms_norm(B.bf16_tensor(X), w, EPS)
    _check_y(got, y)
    for first in (0, 2):
        assert torch.equal(got[first::3], alone[first::3])


@pytest.mark.parametrize("k", [256, 4096])
@pytest.mark.parametrize("every", [1, 4])
def test_codes_of_exact_halves_in_rows_of_one_magnitude(B, k, every):
    """Rows of +-t and zeros, beside which eps vanishes: y is +-w (or twice that), its quotients halves."""
    w = np.resize(np.concatenate([[127.0], np.arange(-127, 127) + 0.5, [1.0]]), k)
    W = synth.to_bf16_bits(w.astype(np.float32))
    t = np.arange(128.0, 256.0)[:, None]
    x = t * np.where(np.arange(k) % 3 == 0, -1, 1) * (np.arange(k) % every == 0)
    codes, scales = B.rms_norm_i8(B.bf16_tensor(synth.to_bf16_bits(x.astype(np.float32))), B.bf16_tensor(W), 1e-37)
    y = np.sign(x) * w * np.sqrt(every)
    assert (scales.double().cpu().numpy() == np.sqrt(every)).all()
    np.testing.assert_array_equal(codes.cpu().numpy(), np.rint(y / np.sqrt(every)))
