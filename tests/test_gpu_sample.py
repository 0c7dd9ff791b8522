"""sample_logits against its 64-bit form."""
import numpy as np
import pytest
import torch

from oracle import q4moe_oracle as qorc
from oracle import step_oracle as orc

pytestmark = pytest.mark.gpu

INF = np.inf
# a weight is off by half of 2^-45 of the largest at most, a total of n of them by n times that and by exp's
# own last bits, and the quotient is rounded to fp32
PROB = 2.0 ** -24 + 2.0 ** -40


@pytest.fixture(scope="module")
def B():
    from quantized_moe_decode_affine_amd import binding
    assert torch.cuda.is_available()
    binding.load_library()
    return binding


def _logits(rng, b, v, spread=2.0, dtype="f32"):
    x = (rng.standard_normal((b, v)) * spread).astype(np.float32)
    t = torch.from_numpy(x).cuda()
    return t.bfloat16() if dtype == "bf16" else t


def _gpu(v, dtype=torch.float32):
    return None if v is None else torch.tensor(np.asarray(v), dtype=dtype, device="cuda")


def _f32(v):
    return None if v is None else np.asarray(v, dtype=np.float32).astype(np.float64)


def _check(B, logits, u, t=None, k=None, p=None, m=None):
    got, probs = B.sample_logits(logits, _gpu(u), _gpu(t), _gpu(k, torch.int32), _gpu(p), _gpu(m))
    ids, want = orc.sample(logits.double().cpu().numpy(), _f32(u), _f32(t), k, _f32(p), _f32(m))
    np.testing.assert_array_equal(got.cpu().numpy(), ids)
    np.testing.assert_allclose(probs.double().cpu().numpy(), want, rtol=PROB, atol=2.0 ** -45 * logits.shape[1])
    return got, probs


SIZES = [1, 2, 63, 64, 65, 257, 1000, 2047, 2048, 2049, 4099, 32003, 151936, 262144]


@pytest.mark.parametrize("V", SIZES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_filters(B, V, dtype):
    """Every combination of the filters, each row with parameters of its own."""
    rng = np.random.default_rng(V)
    n = 10 if V < 100000 else 4
    for spread in (0.3, 2.5):
        logits = _logits(rng, n, V, spread, dtype)
        for on in range(16):
            u = rng.random(n)
            t = rng.choice([0.0, 0.5, 0.9, 1.0, 1.7], n) if on & 1 else None
            k = rng.choice([0, 1, 2, 5, 50, 300, 1000, 3000, V - 1, V, V + 5, -3], n) if on & 2 else None
            p = rng.choice([0.0, 1e-6, 0.1, 0.5, 0.9, 0.99, 0.9999, 1.0, 2.0], n) if on & 4 else None
            m = rng.choice([0.0, 1e-4, 0.02, 0.3, 1.0, 5.0], n) if on & 8 else None
            _check(B, logits, u, t, k, p, m)


@pytest.mark.parametrize("V", [50, 3001, 70001])
def test_draws_over_the_whole_range(B, V):
    """u from 0 to the last number below 1 and outside: the first and the last kept token among them."""
    rng = np.random.default_rng(V)
    u = np.array([0.0, 1e-30, 2.0 ** -24, 0.25, 0.5, 1 - 2.0 ** -24, 1.0, 7.0, -1.0, -0.0, np.nan, INF, -INF])
    row = _logits(rng, 1, V, 3.0)
    logits = row.expand(len(u), V).contiguous()
    for k, p, m in ((0, 1.0, 0.0), (7, 1.0, 0.0), (0, 0.8, 0.0), (40, 0.9, 0.01), (0, 1.0, 0.05)):
        got, _ = _check(B, logits, u, None, np.full(len(u), k), np.full(len(u), p), np.full(len(u), m))
        assert got[0] == got[8] == got[9] == got[10] == got[12] and got[6] == got[7] == got[11]


@pytest.mark.parametrize("V", [40, 2500, 151936])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_equal_logits(B, V, dtype):
    """Rows of one value, of two and of three: what a filter keeps of equals are the lower indices; lists overflow."""
    rng = np.random.default_rng(V)
    rows = [np.zeros(V), np.full(V, -7.25), rng.choice([0.0, 1.0], V), rng.choice([-1.0, 0.0, 0.5], V),
            np.where(np.arange(V) == V // 2, 5.0, -0.0), np.where(rng.random(V) < 0.5, 0.0, -0.0)]
    x = torch.from_numpy(np.array(rows, dtype=np.float32)).cuda()
    x = x.bfloat16() if dtype == "bf16" else x
    n = len(rows)
    for k, p, m in ((None, None, None), (5, None, None), (V // 3 + 1, None, None), (None, 0.4, None), (900, 0.37, None),
                    (V - 1, 0.77, None), (None, 0.9, 0.5), (3, 0.2, 0.1), (2000, None, None)):
        full = lambda v: None if v is None else np.full(n, v)  # noqa: E731
        _check(B, x, rng.random(n), None, full(k), full(p), full(m))
        _check(B, x, rng.random(n), np.full(n, 0.3), full(k), full(p), full(m))


@pytest.mark.parametrize("V", [64, 5000, 40000])
def test_closed_and_infinite_logits(B, V):
    """Masks by -infinity, by the type's lowest value and by NaN; a few open tokens, one, none; +infinity."""
    rng = np.random.default_rng(V)
    low = np.finfo(np.float32).min
    rows, n = [], 14
    for mask in (-INF, low, np.nan):
        for open_ in (1, 3, 20, V // 2):
            x = rng.standard_normal(V) * 2
            x[rng.permutation(V)[open_:]] = mask
            rows.append(x)
    rows.append(np.full(V, -INF))
    rows.append(np.full(V, np.nan))
    rows.append(np.full(V, low))
    x = rng.standard_normal(V)
    x[[3, V // 2, V - 1]] = INF
    rows.append(x)
    x = x.copy()
    x[5], x[7] = np.nan, -INF
    rows.append(x)
    rows.append(np.where(np.arange(V) % 2, INF, -INF))
    logits = torch.from_numpy(np.array(rows, dtype=np.float32)).cuda()
    n = len(rows)
    full = lambda v, dt=float: None if v is None else np.full(n, v, dtype=dt)  # noqa: E731
    for t, k, p, m in ((1.0, None, None, None), (0.8, 5, None, None), (1.0, None, 0.9, None), (1.0, 50, 0.5, 0.01), (0.0, 3, 0.5, None),
                       (1.3, None, None, 0.2), (1.0, V - 1, 0.95, None)):
        got, probs = _check(B, logits, rng.random(n), full(t), full(k, int), full(p), full(m))
        assert got[12] == got[13] == -1 and probs[12] == probs[13] == 0


def test_odd_parameters(B):
    """NaN, infinite and subnormal parameters."""
    rng = np.random.default_rng(5)
    for V in (300, 30000):
        t = np.array([np.nan, -1.0, INF, 1e-40, 1e-3, 1e30, 1.0, 1.0, 1.0, 1.0])
        p = np.array([0.9, 0.9, 0.9, 0.9, 0.9, 0.9, np.nan, -1.0, INF, 1e-45])
        m = np.array([0.0, 0.0, 0.0, 0.0, 0.0, 0.0, np.nan, -1.0, 0.0, 1e-40])
        _check(B, _logits(rng, len(t), V), rng.random(len(t)), t, None, p, m)
        _check(B, _logits(rng, len(t), V), rng.random(len(t)), t, np.full(len(t), 20), p, m)


def test_scales_of_logits(B):
    """Logits tiny, large, far from zero and of outliers: the bins' range and its ends."""
    rng = np.random.default_rng(6)
    V, n = 20000, 8
    base = rng.standard_normal((n, V))
    rows = np.stack([base[0] * 1e-6, base[1] * 1e-38, base[2] * 1e4, base[3] + 1e5, base[4] * 1e30, base[5] - 3e38,
                     np.where(np.arange(V) == 77, 60.0, base[6]), np.where(np.arange(V) == 99, -1e9, base[7])])
    logits = torch.from_numpy(rows.astype(np.float32)).cuda()
    for t in (1.0, 1e-5, 3e3):
        for k, p in ((None, 0.9), (30, None), (8000, 0.95), (None, None)):
            _check(B, logits, rng.random(n), np.full(n, t), None if k is None else np.full(n, k), None if p is None else np.full(n, p))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_lists_that_overflow(B, dtype):
    """Flat rows: more tokens than a list holds under min-p alone, under top-k by ties, and in top-p's band."""
    rng = np.random.default_rng(21)
    V, n = 60000, 6
    flat = _logits(rng, n, V, 0.4, dtype)
    u = rng.random(n)
    for m in (0.01, 0.2, 0.5, 0.9):
        _check(B, flat, u, None, None, None, np.full(n, m))
        _check(B, flat, u, rng.choice([0.3, 1.0, 2.0], n), None, None, np.full(n, m))
    steps = torch.round(flat.float() * 8) / 8   # some tens of values: thousands of tokens to each
    steps = steps.bfloat16() if dtype == "bf16" else steps
    for k, p, m in ((30, None, None), (300, 0.5, None), (None, 0.5, None), (None, 0.99, 0.3), (5000, 0.9, None), (None, None, 0.6)):
        full = lambda v: None if v is None else np.full(n, v)  # noqa: E731
        _check(B, steps, u, rng.choice([0.2, 1.0], n), full(k), full(p), full(m))


def test_frequencies(B):
    """Draws by evenly spaced numbers occur as often as their probability says, to within one."""
    rng = np.random.default_rng(8)
    V, n = 3001, 4096
    row = _logits(rng, 1, V, 1.0)
    logits = row.expand(n, V).contiguous()
    u = (np.arange(n) + 0.5) / n
    ids, _ = B.sample_logits(logits, _gpu(u), None, _gpu(np.full(n, 40), torch.int32))
    x = row.double().cpu().numpy()[0]
    top = np.argsort(-x, kind="stable")[:40]
    w = np.exp(x[top] - x[top].max())
    count = np.bincount(ids.cpu().numpy(), minlength=V)
    assert count.sum() == count[top].sum() == n
    assert (np.abs(count[top] - n * w / w.sum()) <= 1.0 + 1e-6).all()


def test_rows_alone_and_in_any_batch(B):
    rng = np.random.default_rng(9)
    V = 50001
    for n in (3, 70, 600):
        logits = _logits(rng, n, V, 2.0)
        u, t = _gpu(rng.random(n)), _gpu(rng.choice([0.0, 0.7, 1.0], n))
        k, p = _gpu(rng.choice([0, 40, 20000], n), torch.int32), _gpu(rng.choice([0.9, 0.99, 1.0], n))
        ids, probs = B.sample_logits(logits, u, t, k, p)
        for r in {0, n // 2, n - 1}:
            one, pr = B.sample_logits(logits[r:r + 1], u[r:r + 1], t[r:r + 1], k[r:r + 1], p[r:r + 1])
            assert one == ids[r] and pr == probs[r]


def test_unaligned_rows_and_what_is_behind(B):
    """Odd vocabularies and a start in the middle of a buffer: nothing outside the rows is drawn."""
    rng = np.random.default_rng(10)
    for dtype in (torch.float32, torch.bfloat16):
        for V in (33, 4097, 20001):
            for start in (1, 2, 3):
                buf = torch.full((start + 3 * V + 9,), 100.0, dtype=dtype, device="cuda")
                x = buf[start:start + 3 * V].view(3, V)
                x.copy_(torch.from_numpy(rng.standard_normal((3, V)).astype(np.float32)))
                for k, p in ((None, None), (9, 0.9), (None, 0.8)):
                    _check(B, x, rng.random(3), None, None if k is None else np.full(3, k), None if p is None else np.full(3, p))


def test_many_rows(B):
    """More rows than the chip holds workgroups; offsets of rows past 2^31."""
    rng = np.random.default_rng(11)
    n, V = 9000, 262144
    logits = torch.full((n, V), -1.0, dtype=torch.bfloat16, device="cuda")
    hot = torch.from_numpy(rng.integers(0, V, n)).cuda()
    logits.scatter_(1, hot[:, None], 40.0)
    u = torch.rand(n, device="cuda")
    for kw in (dict(), dict(top_k=torch.full((n,), 30, dtype=torch.int32, device="cuda"))):
        ids, probs = B.sample_logits(logits, u, **kw)
        assert torch.equal(ids.long(), hot) and (probs > 0.99).all()
    p = torch.full((n,), 0.5, device="cuda")
    ids, probs = B.sample_logits(logits, u, top_p=p)
    assert torch.equal(ids.long(), hot) and (probs == 1).all()


def test_workspace_reused_and_captured(B):
    """One workspace, dirty, for calls of every kind, and replayed in a graph with eager calls between."""
    rng = np.random.default_rng(12)
    n, V = 6, 40000
    ws = B.sample_logits_workspace(n, V)
    logits, u = _logits(rng, n, V), _gpu(rng.random(n))
    t, p = _gpu(np.full(n, 0.9)), _gpu([0.9, 1.0, 0.5, 0.99, 1.0, 0.3])
    k, m = _gpu([0, 50, 0, 30000, 0, 5], torch.int32), _gpu([0, 0, 0.1, 0, 0.02, 0])
    for fill in (0, 0xFF, 0xA5):
        ws.fill_(fill)
        for args in ((None, None, None, None), (t, k, p, m), (t, None, p, None), (t, k, None, None)):
            assert all(torch.equal(a, b) for a, b in zip(B.sample_logits(logits, u, *args, ws=ws), B.sample_logits(logits, u, *args)))
    ids, probs = torch.empty(n, dtype=torch.int32, device="cuda"), torch.empty(n, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        B.sample_logits(logits, u, t, k, p, m, ids=ids, probs=probs, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.sample_logits(logits, u, t, k, p, m, ids=ids, probs=probs, ws=ws)
    for seed in range(4):
        logits.copy_(_logits(np.random.default_rng(seed), n, V))
        u.copy_(_gpu(np.random.default_rng(seed).random(n)))
        g.replay()
        torch.cuda.synchronize()
        want = B.sample_logits(logits, u, t, k, p, m)
        assert torch.equal(ids, want[0]) and torch.equal(probs, want[1])


def test_head_then_sample(B):
    """A step's end as it is used: norm, its codes through the head's product, the draw from its logits."""
    rng = np.random.default_rng(13)
    n, H, V = 5, 256, 3000
    x = torch.from_numpy(rng.standard_normal((n, H)).astype(np.float32)).cuda().bfloat16()
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    head = B.DeviceI8.quantize(torch.from_numpy(rng.standard_normal((V, H)).astype(np.float32) * 0.2).cuda().bfloat16())
    codes, scales = B.rms_norm_i8(x, w)
    logits = B.i8_gemm_rows(head, codes, scales)
    _check(B, logits, rng.random(n), np.full(n, 0.8), np.full(n, 40), np.full(n, 0.9), np.full(n, 0.01))
    head4 = B.DeviceMx4.quantize(torch.from_numpy(rng.standard_normal((V, H)).astype(np.float32) * 0.2).cuda().bfloat16())
    for out in (B.OUT_F32, B.OUT_BF16):
        _check(B, B.mx4_gemm(head4, B.rms_norm(x, w), out), rng.random(n), np.full(n, 0.8), None, np.full(n, 0.95))
    greedy, _ = B.sample_logits(logits, _gpu(np.zeros(n)), _gpu(np.zeros(n)))
    assert torch.equal(greedy.long(), logits.argmax(1))


def test_binding_refusals(B):
    x, u = torch.zeros(3, 100, device="cuda"), torch.zeros(3, device="cuda")
    for bad in (lambda: B.sample_logits(x.half(), u), lambda: B.sample_logits(x, u.double()), lambda: B.sample_logits(x, u[:2]),
                lambda: B.sample_logits(x.T, u), lambda: B.sample_logits(x, u, top_k=u), lambda: B.sample_logits(x, u, u.cpu()),
                lambda: B.sample_logits(x, u, ids=torch.empty(3, dtype=torch.int64, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(B.Q4Error) as err:
        B.sample_logits(torch.zeros(3, 5000, device="cuda"), u, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert err.value.status == B.EWORKSPACE
    with pytest.raises(B.Q4Error) as err:
        B.sample_logits(x, u, probs=u)
    assert err.value.status == B.EINVAL
    assert B.sample_logits(x[:0], u[:0])[0].shape == (0,)


# Weights in units of 2^-45 of the largest, by hand at a temperature of 1: a logit of 0 weighs 2^45, one of -2^-45 (a
# 45th of a bit below it) 2^45 - 1, one of -45 ln 2 a single unit, one of -1000 nothing.
ONE_LESS, UNIT, NONE = -2.0 ** -45, -45 * np.log(2.0), -1000.0


def _draw(B, row, u, k=None, p=None):
    x = torch.from_numpy(np.asarray(row, dtype=np.float32)[None]).cuda()
    ids, _ = B.sample_logits(x, _gpu([u]), None, _gpu(k and [k], torch.int32), _gpu(p and [p]))
    return int(ids[0])


def _with(rng, V, values):
    """A row of V tokens without weight but those of `values`, at places in order, and these places."""
    at = np.sort(rng.permutation(V)[:len(values)])
    row = np.full(V, NONE)
    row[at] = values
    return row, at


@pytest.mark.parametrize("V,k,p", [(512, None, None), (2000, None, None), (8192, None, None), (2000, 512, None), (60000, 512, None),
                                   (2000, None, 1 - 2.0 ** -24), (8192, None, 1 - 2.0 ** -24), (60000, 3000, None)])
def test_draw_at_a_border(B, V, k, p):
    """512 tokens whose weights sum to 2^54 - 1, which fp64 does not hold: half of it is 2^53 - 1/2, and the running sum
    exceeds that with the 256th token, not with the one after."""
    row, at = _with(np.random.default_rng(V), V, [0.0] * 511 + [ONE_LESS])
    assert _draw(B, row, 0.5, k, p) == at[255]
    assert _draw(B, row, 0.5 + 2.0 ** -24, k, p) == at[256]


@pytest.mark.parametrize("V,k", [(513, None), (2000, None), (8192, None), (151936, None), (2000, 600), (60000, 600), (60000, 5000)])
def test_top_p_at_a_border(B, V, k):
    """513 tokens whose weights sum to 2^54 + 1: the fewest that reach half of it, 2^53 + 1/2, are 257."""
    row, at = _with(np.random.default_rng(V), V, [0.0] * 512 + [UNIT])
    assert _draw(B, row, 1.0, k, 0.5) == at[256]
    row[at[-1]] = NONE
    assert _draw(B, row, 1.0, k, 0.5) == at[255]
