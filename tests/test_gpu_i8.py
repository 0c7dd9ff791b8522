"""i8_quantize, i8_gemm and moe_experts_i8 against their 64-bit forms."""
import numpy as np
import pytest
import torch

from oracle import q4moe_oracle as qorc
from oracle import route_i8_oracle as orc
from quantized_moe_decode_affine_amd import synth
from tests.parity_util import bf16_bits, bf16_bits_of_f32, to_f64

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -24       # half a step of fp32 at most, relative
HALF_F16 = 2.0 ** -11   # the same of fp16
HALF_BF16 = 2.0 ** -8   # and of bfloat16


@pytest.fixture(scope="module")
def B():
    from quantized_moe_decode_affine_amd import binding
    assert torch.cuda.is_available()
    binding.load_library()
    return binding


def _rows(seed, m, k):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((m, k)) * np.exp(0.7 * rng.standard_normal((m, 1)))
    return synth.to_bf16_bits(x.astype(np.float32))


def _weights(seed, *shape):
    rng = np.random.default_rng(seed)
    codes = rng.integers(-127, 128, shape, dtype=np.int8)
    scales = (rng.random(shape[:-1]) * 0.02 / 73 + 1e-5).astype(np.float32)
    return codes, scales


def _dev(B, w):
    return B.DeviceI8(torch.from_numpy(w[0]).cuda(), torch.from_numpy(w[1]).cuda())


# ------------------------------------------------------------------- quantize --

@pytest.mark.parametrize("rows,k", [(1, 64), (3, 128), (5, 192), (4, 2048), (1030, 320), (2, 16384), (1, 65536)])
def test_quantize_exact(B, rows, k):
    X = _rows(rows + k, rows, k)
    codes, scales = B.i8_quantize(B.bf16_tensor(X))
    q, s = orc.quantize_rows(qorc.bf16_to_f64(X))
    np.testing.assert_array_equal(codes.cpu().numpy(), q)
    np.testing.assert_array_equal(scales.cpu().numpy(), s)


def test_quantize_borders_and_extremes(B):
    k = 128
    x = np.zeros((12, k), np.float32)
    x[1] = np.arange(k) / 2 - 32                     # with 127 first: scale 1, halves are ties
    x[1, 0] = 127.0
    x[2] = (np.arange(k) / 2 - 32) * 2.0 ** -90
    x[2, 0] = 127.0 * 2.0 ** -90
    x[3] = np.arange(k) * 1.0                        # a scale of 127/127 and every integer
    x[4] = 2.0 ** -133 * (np.arange(k) % 5)          # subnormal bfloat16
    x[5] = 3.38e38 * (1 - np.arange(k) / 64)         # the type's largest
    x[6, 5] = np.inf
    x[7, 9] = np.nan
    x[8] = -0.0
    x[9] = 1.0                                       # every value the largest
    x[10, 3] = -5.5
    x[11] = np.linspace(-1, 1, k) * 2.0 ** -126
    X = synth.to_bf16_bits(np.nan_to_num(x, nan=0.0, posinf=0.0))
    X[6, 5], X[7, 9] = 0x7F80, 0xFFC1
    codes, scales = B.i8_quantize(B.bf16_tensor(X))
    v = qorc.bf16_to_f64(X)
    v[6, 5], v[7, 9] = np.inf, np.nan
    q, s = orc.quantize_rows(v)
    np.testing.assert_array_equal(codes.cpu().numpy(), q)
    np.testing.assert_array_equal(scales.cpu().numpy(), s)


# ----------------------------------------------------------------------- gemm --

def _check_gemm(B, W, X, y32, y16):
    some = slice(None) if X.shape[0] <= 1000 else slice(X.shape[0] % 17, None, 17)
    np.testing.assert_array_equal(bf16_bits(y16), bf16_bits_of_f32(y32))
    y32 = y32[some]
    ref = orc.i8_gemm(W[0].reshape(-1, W[0].shape[-1]), W[1].reshape(-1), X[some])
    # the sum becomes fp32, then one rounding at each scale
    assert (np.abs(to_f64(y32) - ref) <= 3 * HALF * (1 + 1e-6) * np.abs(ref) + 2.0 ** -149).all()


@pytest.mark.parametrize("m,n,k", [
    (1, 1, 64), (1, 16, 128), (1, 1024, 2048), (2, 17, 192), (3, 100, 64), (4, 1000, 320), (7, 257, 2048),
    (8, 4099, 256), (9, 64, 4096), (15, 33, 128), (16, 96, 704), (16, 40, 4096), (13, 20000, 1088), (5, 40000, 192), (16, 16, 16384), (17, 64, 128), (31, 300, 832),
    (33, 65, 64), (64, 64, 192), (65, 31, 2048), (100, 513, 320), (127, 128, 128), (129, 255, 576), (256, 1, 64),
    (381, 1027, 832), (513, 300, 256), (1000, 2048, 192),
    (2000, 2100, 320), (3900, 4100, 128), (4100, 3999, 64), (2049, 4095, 448)])
def test_gemm_parity(B, m, n, k):
    W, X = _weights(m + n, n, k), _rows(k + m, m, k)
    d, x = _dev(B, W), B.bf16_tensor(X)
    _check_gemm(B, W, X, B.i8_gemm(d, x), B.i8_gemm(d, x, B.OUT_BF16))


@pytest.mark.parametrize("m", [1, 5, 40, 200])
def test_gemm_stack(B, m):
    W, X = _weights(5, 3, 40, 128), _rows(m, m, 128)
    _check_gemm(B, W, X, B.i8_gemm(_dev(B, W), B.bf16_tensor(X)), B.i8_gemm(_dev(B, W), B.bf16_tensor(X), B.OUT_BF16))


@pytest.mark.parametrize("m", [1, 16, 150])
def test_gemm_largest_sums(B, m):
    """Every product 127 * -128 over the longest rows: the largest sum there is."""
    k = 65536
    W = np.full((3, k), -128, np.int8), np.array([1.0, 0.0, 2.0 ** -20], np.float32)
    W[0][1] = 127
    X = synth.to_bf16_bits(np.full((m, k), 3.0, np.float32))
    _check_gemm(B, W, X, B.i8_gemm(_dev(B, W), B.bf16_tensor(X)), B.i8_gemm(_dev(B, W), B.bf16_tensor(X), B.OUT_BF16))


@pytest.mark.parametrize("m", [3, 20])
def test_gemm_weights_past_4gb(B, m):
    """Code offsets and output rows beyond 32 bits: the last channels of a 4.4 GB matrix."""
    n, k = 2_100_000, 2112
    gen = torch.Generator(device="cuda").manual_seed(m)
    codes = torch.randint(-127, 128, (n, k), generator=gen, device="cuda", dtype=torch.int8)
    scales = torch.rand(n, generator=gen, device="cuda") * 1e-3
    X = _rows(m, m, k)
    y = B.i8_gemm(B.DeviceI8(codes, scales), B.bf16_tensor(X))
    for at in (slice(0, 70), slice(n // 2, n // 2 + 70), slice(n - 70, n)):
        ref = orc.i8_gemm(codes[at].cpu().numpy(), scales[at].cpu().numpy(), X)
        assert (np.abs(to_f64(y[:, at]) - ref) <= 3 * HALF * (1 + 1e-6) * np.abs(ref) + 2.0 ** -149).all()


@pytest.mark.parametrize("m", [3, 16, 70])
def test_gemm_rows_without_values(B, m):
    """A zero row gives zeros, a row with an infinity or a NaN gives NaN, and no other row notices."""
    W, X = _weights(1, 200, 192), _rows(m, m, 192)
    X[0] = 0
    X[1, 70], X[2, 3] = 0x7F80, 0x7FC1
    d = _dev(B, W)
    for out in (B.OUT_F32, B.OUT_BF16):
        y = B.i8_gemm(d, B.bf16_tensor(X), out)
        assert (y[0] == 0).all() and torch.isnan(y[1]).all() and torch.isnan(y[2]).all()
        if m > 3:
            assert torch.equal(y[3:], B.i8_gemm(d, B.bf16_tensor(X[3:]), out))


@pytest.mark.parametrize("m", [2, 33])
def test_gemm_writes_its_rows_only(B, m):
    W, X = _weights(2, 72, 128), _rows(m, m, 128)
    for out, t in ((B.OUT_F32, torch.float32), (B.OUT_BF16, torch.bfloat16)):
        buf = torch.full((m + 2, 72), 7.0, dtype=t, device="cuda")
        y = B.i8_gemm(_dev(B, W), B.bf16_tensor(X), out, out=buf[1:m + 1])
        assert torch.equal(y, B.i8_gemm(_dev(B, W), B.bf16_tensor(X), out))
        assert (buf[0] == 7).all() and (buf[-1] == 7).all()


def test_gemm_of_quantized_weights(B):
    """From bfloat16 weights on: the product approximates X W^T by the codes' resolution."""
    w, X = _rows(1, 96, 512), _rows(2, 20, 512)
    d = B.DeviceI8.quantize(B.bf16_tensor(w))
    q, s = orc.quantize_rows(qorc.bf16_to_f64(w))
    _check_gemm(B, (q.astype(np.int8), s.astype(np.float32)), X, B.i8_gemm(d, B.bf16_tensor(X)),
                B.i8_gemm(d, B.bf16_tensor(X), B.OUT_BF16))


def test_gemm_on_two_streams(B):
    """Calls in flight together, each with a workspace of its own."""
    W = _dev(B, _weights(3, 512, 1024))
    xs = [B.bf16_tensor(_rows(n, m, 1024)) for n, m in enumerate((1, 9, 64, 300))]
    want = [B.i8_gemm(W, x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                got.append(B.i8_gemm(W, x))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# -------------------------------------------------------------------- experts --

def _layer(seed, E, H, I, shared):
    g, u, d = _weights(seed, E, I, H), _weights(seed + 1, E, I, H), _weights(seed + 2, E, H, I)
    sh = (_weights(seed + 3, 1, I, H), _weights(seed + 4, 1, I, H), _weights(seed + 5, 1, H, I)) if shared else None
    return g, u, d, sh


def _experts(B, layer):
    g, u, d, sh = layer
    return B.DeviceI8Experts(*(_dev(B, w) for w in (g, u, d)), shared=None if sh is None else [_dev(B, w) for w in sh])


def _ids(seed, T, E, k, empty=0.0):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    ids[rng.random((T, k)) < empty] = -1
    return ids, rng.random((T, k)).astype(np.float32)


def _check_experts(B, layer, X, ids, w, ex=None):
    ex = ex or _experts(B, layer)
    x, i, wt = B.bf16_tensor(X), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()
    y, slack, parts = orc.experts_i8(*layer[:3], X, ids, w, layer[3])
    y32, y16 = B.moe_experts_i8(ex, x, i, wt), B.moe_experts_i8(ex, x, i, wt, B.OUT_BF16)
    assert (np.abs(to_f64(y32) - y) <= slack).all()
    # bfloat16: each summand may be rounded to fp16's 11 significant bits, then the output to 8.
    # Values in [2^e, 2^(e+1)) with 11 bits are 2^(e-10) apart, so half a step is up to 2^(e-11):
    # 2^-11 of the value (finfo(float16).eps / 2), not 2^-12.
    before = slack + HALF_F16 * parts
    assert (np.abs(to_f64(y16) - y) <= before + HALF_BF16 * (np.abs(y) + before)).all()


@pytest.mark.parametrize("T,E,H,I,k,shared", [
    (1, 8, 64, 64, 1, False), (1, 256, 256, 128, 8, True), (1, 16, 2048, 512, 8, True), (1, 8, 192, 1024, 3, True), (1, 8, 4160, 512, 2, False), (2, 4, 128, 192, 4, False),
    (3, 60, 1088, 704, 4, True), (5, 16, 192, 64, 2, True), (8, 32, 512, 256, 8, True), (16, 8, 256, 320, 2, False),
    (17, 16, 256, 128, 4, True), (40, 5, 320, 64, 3, False), (129, 3, 128, 128, 1, True), (300, 2, 192, 64, 2, True),
    (64, 1, 128, 256, 1, False), (33, 40, 64, 1088, 32, False)])
def test_experts_parity(B, T, E, H, I, k, shared):
    layer = _layer(T + E, E, H, I, shared)
    _check_experts(B, layer, _rows(T, T, H), *_ids(T, T, E, k, 0.1 if T > 2 else 0.0))


@pytest.mark.parametrize("T", [1, 6, 150])
@pytest.mark.parametrize("shared", [False, True])
def test_experts_empty_slots(B, T, shared):
    """Tokens whose every slot is empty get the shared expert alone, or zeros."""
    layer = _layer(9, 6, 128, 64, shared)
    X = _rows(1, T, 128)
    ids, w = _ids(2, T, 6, 3)
    ids[0] = [-1, 6, 2 ** 31 - 1]
    if T > 2:
        ids[2] = -2 ** 31
    w[0] = np.nan                                      # the weight of an empty slot is not read into the sum
    _check_experts(B, layer, X, ids, w)
    ids[:] = -1
    _check_experts(B, layer, X, ids, w)
    if not shared:
        y = B.moe_experts_i8(_experts(B, layer), B.bf16_tensor(X), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda())
        assert (y == 0).all()


@pytest.mark.parametrize("T", [1, 7, 90])
def test_experts_same_id_twice(B, T):
    layer = _layer(3, 5, 128, 128, True)
    ids, w = _ids(4, T, 5, 4)
    ids[:, 2] = ids[:, 0]
    ids[:, 3] = ids[:, 0]
    _check_experts(B, layer, _rows(5, T, 128), ids, w - 0.5)


def test_experts_all_to_one(B):
    """A full expert of several row tiles beside empty ones."""
    layer = _layer(6, 12, 192, 64, False)
    ids = np.full((401, 2), 11, np.int32)
    ids[:, 1] = np.where(np.arange(401) % 5 == 0, 3, -1)
    _check_experts(B, layer, _rows(7, 401, 192), ids, np.full((401, 2), 0.5, np.float32))


@pytest.mark.parametrize("T", [3, 16, 60])
def test_experts_rows_do_not_mix(B, T):
    """A token with a NaN, one with an infinity and one of zeros leave the others as they are."""
    layer = _layer(8, 4, 128, 64, True)
    ex = _experts(B, layer)
    X = _rows(9, T, 128)
    ids, w = _ids(10, T, 4, 2)
    clean = B.moe_experts_i8(ex, B.bf16_tensor(X), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda())
    X[0, 5], X[1, 100] = 0x7FC1, 0xFF80
    X[2] = 0
    y = B.moe_experts_i8(ex, B.bf16_tensor(X), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda())
    assert torch.isnan(y[:2]).all() and (y[2] == 0).all() and torch.equal(y[3:], clean[3:])


def test_experts_workspace_is_not_state(B):
    """A workspace full of anything, used for calls of several sizes."""
    layer = _layer(11, 8, 128, 64, True)
    ex = _experts(B, layer)
    ws = B.moe_experts_i8_workspace(ex, 200, 3)
    for n, T in enumerate((200, 1, 17, 4, 130)):
        X, (ids, w) = B.bf16_tensor(_rows(n, T, 128)), _ids(n, T, 8, 3, 0.3)
        args = ex, X, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()
        want = B.moe_experts_i8(*args)
        ws.fill_(255 - n)
        buf = torch.full((T + 2, 128), 3.0, device="cuda")
        B.moe_experts_i8(*args, out=buf[1:T + 1], ws=ws)
        assert torch.equal(buf[1:T + 1], want) and (buf[0] == 3).all() and (buf[-1] == 3).all()


@pytest.mark.parametrize("T", [1, 12, 100])
def test_route_then_experts(B, T):
    """The router's ids and weights, closed experts among them, into the experts' products; the
    same in a captured graph that is replayed on other tokens."""
    E, H, I, k = 24, 256, 128, 4
    rng = np.random.default_rng(T)
    R = synth.to_bf16_bits((np.clip(np.round(rng.standard_normal((E, H)) * 20), -255, 255) / 1024).astype(np.float32))
    tokens = [synth.to_bf16_bits((np.clip(np.round(rng.standard_normal((T, H)) * 8), -40, 40) / 8).astype(np.float32))
              for _ in range(3)]
    bias = rng.standard_normal(E).astype(np.float32) * 0.1
    bias[:4] = -np.inf
    rule = dict(top_k=k, score="sigmoid", n_groups=6, top_groups=2, scale=2.5)
    r = B.Routing(B.bf16_tensor(R), bias=torch.from_numpy(bias).cuda(), **rule)
    layer = _layer(12, E, H, I, True)
    ex = _experts(B, layer)
    X = B.bf16_tensor(tokens[0])
    ws, wr = B.moe_experts_i8_workspace(ex, T, k), B.moe_route_workspace(r, T)
    ids, w = B.moe_route(r, X, ws=wr)
    y = B.moe_experts_i8(ex, X, ids, w, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.moe_route(r, X, ids=ids, weights=w, ws=wr)
        B.moe_experts_i8(ex, X, ids, w, out=y, ws=ws)
    for bits in tokens:
        X.copy_(B.bf16_tensor(bits))
        y.zero_()
        graph.replay()
        ref_ids, ref_w = orc.route_rule(qorc.router_logits(R, bits), bias=bias, **rule)
        np.testing.assert_array_equal(ids.cpu().numpy(), ref_ids)
        ref, slack, parts = orc.experts_i8(*layer[:3], bits, ref_ids, ref_w, layer[3])
        assert (np.abs(to_f64(y) - ref) <= slack + 2 * HALF * parts).all()
        i2, w2 = B.moe_route(r, X)
        assert torch.equal(B.moe_experts_i8(ex, X, i2, w2), y)


def test_two_graphs_share_workspaces(B):
    """Two captured steps of different sizes on the same workspaces, replayed in turn between eager
    calls on them: each leaves them ready for the other."""
    E, H, I, k = 16, 256, 128, 4
    layer = _layer(21, E, H, I, True)
    ex = _experts(B, layer)
    r = B.Routing(B.bf16_tensor(_rows(22, E, H)), k, score="sigmoid")
    ws, wr = B.moe_experts_i8_workspace(ex, 90, k), B.moe_route_workspace(r, 90)

    def step(X, out):
        ids, w = B.moe_route(r, X, ws=wr)
        return B.moe_experts_i8(ex, X, ids, w, out=out, ws=ws)

    parts = []
    for T in (2, 90):
        X = B.bf16_tensor(_rows(T, T, H))
        Y = torch.empty(T, H, device="cuda")
        step(X, Y)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(X, Y)
        parts.append((X, Y, graph))
    for n in range(3):
        for X, Y, graph in parts:
            X.copy_(B.bf16_tensor(_rows(30 + n, X.shape[0], H)))
            Y.zero_()
            graph.replay()
            got = Y.clone()
            want = step(X, torch.empty_like(Y))
            torch.cuda.synchronize()
            assert torch.equal(got, want)


def test_experts_on_two_streams(B):
    """Calls in flight together on one set of weights, each with a workspace of its own."""
    layer = _layer(23, 12, 256, 192, True)
    ex = _experts(B, layer)
    args = []
    for T in (1, 6, 40, 200):
        ids, w = _ids(T, T, 12, 3, 0.1)
        args.append((B.bf16_tensor(_rows(T, T, 256)), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()))
    want = [B.moe_experts_i8(ex, *a) for a in args]
    streams = [torch.cuda.Stream() for _ in args]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for a, s in zip(args, streams):
            with torch.cuda.stream(s):
                got.append(B.moe_experts_i8(ex, *a))
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_refusals(B):
    W = _dev(B, _weights(1, 64, 128))
    X = torch.zeros(3, 128, dtype=torch.bfloat16, device="cuda")
    for bad in (X.float(), X.cpu(), X[:, :64], torch.zeros(128, 3, dtype=torch.bfloat16, device="cuda").T):
        with pytest.raises(ValueError):
            B.i8_gemm(W, bad)
    with pytest.raises(ValueError):
        B.i8_gemm(W, X, B.OUT_BF16_RESIDUAL)
    with pytest.raises(ValueError):
        B.i8_gemm(W, X, out=torch.empty(3, 65, device="cuda"))
    with pytest.raises(B.Q4Error) as e:
        B.i8_gemm(W, X, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == B.EWORKSPACE
    assert B.i8_gemm(W, X[:0]).shape == (0, 64)
    with pytest.raises(ValueError):
        B.DeviceI8(torch.zeros(4, 64, dtype=torch.int8, device="cuda"), torch.zeros(5, device="cuda"))
    ex = _experts(B, _layer(1, 4, 64, 128, False))
    x = torch.zeros(3, 64, dtype=torch.bfloat16, device="cuda")
    ids, w = torch.zeros(3, 2, dtype=torch.int32, device="cuda"), torch.zeros(3, 2, device="cuda")
    with pytest.raises(ValueError):
        B.moe_experts_i8(ex, x, ids.long(), w)
    with pytest.raises(ValueError):
        B.moe_experts_i8(ex, x, ids, w[:, :1])
    with pytest.raises(ValueError):
        B.DeviceI8Experts(ex.matrices[0], ex.matrices[1], ex.matrices[0])
    assert B.moe_experts_i8(ex, x[:0], ids[:0], w[:0]).shape == (0, 64)


# ------------------------------------------------------- one result in every form --

@pytest.mark.parametrize("T,E,H,I,k,shared", [(1, 16, 256, 512, 8, True), (9, 8, 192, 128, 4, False), (17, 16, 256, 128, 4, True),
                                              (129, 3, 128, 128, 1, True), (300, 2, 192, 64, 2, False),
                                              (70, 12, 1088, 320, 3, True)])
def test_experts_bf16_is_the_fp32_output_rounded(B, T, E, H, I, k, shared):
    """Nothing but the output's own rounding comes with a bfloat16 output, few slots or many."""
    ex = _experts(B, _layer(T + 40, E, H, I, shared))
    ids, w = _ids(T, T, E, k, 0.1 if T > 1 else 0.0)
    args = ex, B.bf16_tensor(_rows(T, T, H)), torch.from_numpy(ids).cuda(), torch.from_numpy(w - 0.4).cuda()
    np.testing.assert_array_equal(bf16_bits(B.moe_experts_i8(*args, B.OUT_BF16)), bf16_bits_of_f32(B.moe_experts_i8(*args)))


@pytest.mark.parametrize("E,H,I,k,shared", [(8, 256, 512, 4, True), (40, 1088, 320, 6, True), (5, 192, 64, 3, False),
                                            (300, 128, 1024, 8, True)])
def test_experts_token_does_not_depend_on_its_batch(B, E, H, I, k, shared):
    """The same bits alone, among few and among many tokens."""
    T = 90
    ex = _experts(B, _layer(E, E, H, I, shared))
    ids, w = _ids(E, T, E, k, 0.1)
    X, ids, w = B.bf16_tensor(_rows(E, T, H)), torch.from_numpy(ids).cuda(), torch.from_numpy(w - 0.4).cuda()
    for out in (B.OUT_F32, B.OUT_BF16):
        whole = B.moe_experts_i8(ex, X, ids, w, out)
        for part in (slice(0, 1), slice(7, 8), slice(3, 5), slice(20, 28), slice(40, 56), slice(50, 90)):
            assert torch.equal(B.moe_experts_i8(ex, X[part], ids[part], w[part], out), whole[part])


# ------------------------------------------------------------ loops and large tiles --

@pytest.mark.parametrize("m,n,k", [(4090, 4093, 448), (4096, 4096, 64), (3850, 4090, 1088), (3900, 4100, 1088)])
def test_gemm_large_tiles(B, m, n, k):
    """Tiles of 256 x 256 with whole and ragged edges, and the 128 x 128 ones (the last shape) over
    more steps of K than a tile has stages (tests/test_route_i8_host.py has each shape's tile)."""
    W, X = _weights(m + n, n, k), _rows(k + m, m, k)
    d, x = _dev(B, W), B.bf16_tensor(X)
    _check_gemm(B, W, X, B.i8_gemm(d, x), B.i8_gemm(d, x, B.OUT_BF16))


@pytest.mark.parametrize("T,E,H,I,k,shared", [(70, 12, 1088, 320, 3, True), (40, 16, 2048, 512, 4, True), (150, 6, 832, 192, 2, False),
                                              (300, 2, 1088, 1088, 2, True)])
def test_experts_grouped_long_rows(B, T, E, H, I, k, shared):
    """More slots than the few-slots form takes, over more steps of K than the tiles have stages."""
    assert T * k > 64
    _check_experts(B, _layer(T + E, E, H, I, shared), _rows(T, T, H), *_ids(T, T, E, k, 0.1))


@pytest.mark.parametrize("full", [16, 17, 33, 64])
def test_experts_many_slots_of_one(B, full):
    """16 tokens, `full` of their 64 slots on one expert: up to four passes of 16 over its rows."""
    layer = _layer(13, 6, 192, 128, True)
    ids, w = _ids(14, 16, 5, 4)
    flat = ids.reshape(-1)
    flat[np.random.default_rng(full).permutation(64)[:full]] = 5
    _check_experts(B, layer, _rows(15, 16, 192), ids, w - 0.5)


@pytest.mark.parametrize("T,E,H,I,k", [(1, 40, 256, 128, 32), (2, 40, 192, 320, 32), (1, 40, 128, 512, 32), (1, 10, 128, 8192, 9),
                                       (2, 8, 64, 16384, 8), (1, 8, 64, 16384, 8)])
def test_experts_more_slots_than_waves(B, T, E, H, I, k):
    """A wave of the down product takes several slots: more than 16 of them, or activations so long
    that fewer waves fit a workgroup."""
    _check_experts(B, _layer(T + I, E, H, I, True), _rows(T, T, H), *_ids(T, T, E, k))


def test_experts_gathered_rows_past_2gb(B):
    """Offsets of the tokens' codes between 2^31 and 2^32."""
    T, E, H, I = 135_001, 3, 16384, 64
    layer = _layer(17, E, H, I, False)
    gen = torch.Generator(device="cuda").manual_seed(1)
    X = torch.randn(T, H, generator=gen, device="cuda", dtype=torch.bfloat16)
    ids = torch.randint(-1, E, (T, 1), generator=gen, device="cuda", dtype=torch.int32)
    w = torch.rand(T, 1, generator=gen, device="cuda")
    y = B.moe_experts_i8(_experts(B, layer), X, ids, w)
    some = torch.cat([torch.arange(0, 9), torch.arange(131_067, 131_076), torch.arange(T - 9, T)]).cuda()
    ref, slack, _ = orc.experts_i8(*layer[:3], bf16_bits(X[some]), ids[some].cpu().numpy(), w[some].cpu().numpy())
    assert (np.abs(to_f64(y[some]) - ref) <= slack).all()


@pytest.mark.parametrize("T", [1, 10, 80])
def test_experts_gated_shared_as_a_stacked_one(B, T):
    """A shared expert stacked behind the routed ones and chosen in a last slot: with weight 1 the
    same bits as the shared form, with a gate's weights the definition's value."""
    E, H, I, k = 6, 192, 128, 3
    layer = _layer(31, E, H, I, True)
    stacked = tuple(tuple(np.concatenate([m[i], s[i]]) for i in (0, 1)) for m, s in zip(layer[:3], layer[3]))
    X, (ids, w) = _rows(32, T, H), _ids(33, T, E, k, 0.1 if T > 1 else 0.0)
    ids = np.concatenate([ids, np.full((T, 1), E, np.int32)], 1)
    ex = _experts(B, (*stacked, None))
    x, i = B.bf16_tensor(X), torch.from_numpy(ids).cuda()
    one = torch.from_numpy(np.concatenate([w, np.ones((T, 1), np.float32)], 1)).cuda()
    want = B.moe_experts_i8(_experts(B, layer), x, i[:, :k].contiguous(), one[:, :k].contiguous())
    assert torch.equal(B.moe_experts_i8(ex, x, i, one), want)
    gate = np.random.default_rng(34).random((T, 1)).astype(np.float32)
    _check_experts(B, (*stacked, None), X, ids, np.concatenate([w, gate], 1), ex)
