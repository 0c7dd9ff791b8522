"""moe_route and moe_route_logits against the 64-bit routing rules.

Router inputs lie on a grid on which every fp32 sum of products is exact, so ids have to be
equal, ties included.  A weight is rounded once from 64 bits: half a step of fp32, 2^-24 of it.
"""
import numpy as np
import pytest
import torch

from oracle import q4moe_oracle as qorc
from oracle import route_i8_oracle as orc
from quantized_moe_decode_affine_amd import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from quantized_moe_decode_affine_amd import binding
    assert torch.cuda.is_available()
    binding.load_library()
    return binding


def _check(ids, w, ref_ids, ref_w):
    np.testing.assert_array_equal(ids.cpu().numpy(), ref_ids)
    got = w.double().cpu().numpy()
    # half a step, and the 64-bit sums' own order (under 2^-44 of the weight)
    assert (np.abs(got - ref_w) <= np.abs(ref_w) * 2.0 ** -24 * (1 + 2.0 ** -20) + 2.0 ** -150).all()


def _logits(seed, T, E, step=2.0 ** -6):
    """Random logits with many ties (multiples of step)."""
    rng = np.random.default_rng(seed)
    return (np.round(rng.standard_normal((T, E)) * 1.5 / step) * step).astype(np.float32)


RULES = [
    dict(top_k=1), dict(top_k=8), dict(top_k=4, renormalise=False, scale=2.5),
    dict(top_k=8, score="sigmoid"), dict(top_k=8, score="sigmoid", n_groups=4, top_groups=2, group_terms=2),
    dict(top_k=8, score="sigmoid", n_groups=4, top_groups=2, group_terms=1, renormalise=False, scale=-0.5),
    dict(top_k=3, score="softmax", n_groups=2, top_groups=1, group_terms=2),
    dict(top_k=3, score="softmax", n_groups=1, top_groups=1, group_terms=1, renormalise=False),
]


@pytest.mark.parametrize("E", [12, 60, 64, 68, 256, 260, 512, 1000, 1024])
@pytest.mark.parametrize("bias", [False, True])
def test_rules(B, E, bias):
    for n, rule in enumerate(RULES):
        for T in (1, 5):
            l = _logits(100 * E + n, T, E)
            b = None
            if bias:
                b = (np.random.default_rng(E).standard_normal(E) * 0.1).astype(np.float32)
                b[::7] = 0.0
            rule_ = dict(rule, top_k=min(rule["top_k"], E // 4))
            r = B.Routing(E, bias=None if b is None else torch.from_numpy(b).cuda(), **rule_)
            _check(*B.moe_route_logits(r, torch.from_numpy(l).cuda()), *orc.route_rule(l, bias=b, **rule_))


@pytest.mark.parametrize("E,G,keep", [(2, 2, 1), (15, 3, 2), (35, 5, 4), (64, 64, 9), (128, 64, 32), (126, 63, 63),
                                      (1024, 32, 3), (1023, 33, 20), (1024, 2, 1), (513, 1, 1)])
@pytest.mark.parametrize("terms", [1, 2])
def test_group_shapes(B, E, G, keep, terms):
    rule = dict(top_k=min(32, keep * (E // G)), score="sigmoid", n_groups=G, top_groups=keep, group_terms=terms)
    l = _logits(E + G, 9, E)
    b = (np.round(np.random.default_rng(G).standard_normal(E) * 8) / 64).astype(np.float32)
    r = B.Routing(E, bias=torch.from_numpy(b).cuda(), **rule)
    _check(*B.moe_route_logits(r, torch.from_numpy(l).cuda()), *orc.route_rule(l, bias=b, **rule))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [False, True])
def test_closed_and_extreme_logits(B, score, renormalise):
    low = np.float32(np.finfo(np.float32).min)
    E = 20
    l = _logits(5, 12, E)
    l[0] = -np.inf                       # nothing open
    l[1] = np.nan
    l[2, 3:] = -np.inf                   # fewer open than top_k
    l[3] = low                           # the type's lowest value: open, equal
    l[4, ::2] = low
    l[5, 4] = np.inf
    l[6, [4, 9]] = np.inf
    l[7, ::3] = np.nan
    l[8] = 90.0                          # a sigmoid of 1 in 64 bits too
    l[9, :10] = -90.0
    l[10] = 0.0
    l[10, ::2] = -0.0                    # equal to +0: lower id first
    l[11, :] = np.linspace(-110, 110, E, dtype=np.float32)
    for extra in (dict(), dict(n_groups=5, top_groups=2, group_terms=2), dict(n_groups=5, top_groups=5, group_terms=1)):
        for b in (None, np.where(np.arange(E) % 4 == 1, -np.inf, 0.25).astype(np.float32)):
            if b is not None:
                b[2], b[6], b[7] = np.nan, np.inf, np.inf
            rule = dict(top_k=6, score=score, renormalise=renormalise, **extra)
            r = B.Routing(E, bias=None if b is None else torch.from_numpy(b).cuda(), **rule)
            _check(*B.moe_route_logits(r, torch.from_numpy(l).cuda()), *orc.route_rule(l, bias=b, **rule))


def _grid(seed, shape, std, step, most):
    v = np.random.default_rng(seed).standard_normal(shape) * (std / step)
    return synth.to_bf16_bits((np.clip(np.round(v), -most, most) * step).astype(np.float32))


@pytest.mark.parametrize("T,E,H,k", [(1, 256, 2048, 8), (2, 16, 64, 4), (3, 60, 1088, 6), (4, 1000, 576, 9), (4, 257, 4096, 3), (15, 256, 128, 8), (16, 512, 320, 10),
                                     (17, 512, 2048, 10), (33, 1024, 192, 32),
                                     (64, 60, 2048, 6), (63, 81, 2112, 7), (5, 1024, 64, 3), (13, 250, 4160, 8), (64, 8, 256, 2), (130, 257, 448, 5),
                                     (2048, 256, 2048, 8)])
def test_route_bf16_router(B, T, E, H, k):
    R, X = _grid(E + H, (E, H), 0.02, 2.0 ** -10, 255), _grid(T, (T, H), 1.0, 2.0 ** -3, 40)
    b = (np.random.default_rng(E).standard_normal(E) * 0.05).astype(np.float32)
    rule = dict(top_k=k, score="sigmoid")
    r = B.Routing(B.bf16_tensor(R), bias=torch.from_numpy(b).cuda(), **rule)
    some = slice(None) if T <= 130 else slice(0, T, 61)
    ref = orc.route_rule(qorc.router_logits(R, X[some]), bias=b, **rule)
    ids, w = B.moe_route(r, B.bf16_tensor(X))
    _check(ids[some], w[some], *ref)


@pytest.mark.parametrize("T,E,H,k", [(1, 256, 2048, 8), (2, 7, 64, 3), (3, 600, 1088, 8), (4, 60, 192, 6), (5, 60, 192, 6), (64, 128, 320, 6), (63, 60, 2112, 6), (16, 100, 320, 4), (37, 512, 1088, 10),
                                     (1111, 509, 448, 7), (2100, 256, 128, 3)])
def test_route_q8_router(B, T, E, H, k):
    rng = np.random.default_rng(E + T)
    codes = rng.integers(0, 256, (E, H), dtype=np.uint8).view(np.uint32)
    sc = synth.to_bf16_bits(np.full((E, H // 64), 2.0 ** -12, np.float32))
    bi = synth.to_bf16_bits(np.full((E, H // 64), -128 * 2.0 ** -12, np.float32))
    X = _grid(T, (T, H), 1.0, 2.0 ** -3, 40)
    rule = dict(top_k=k, renormalise=False, scale=1.5)
    d = B.DeviceQ4(codes, sc, bi)
    same = B.DeviceQ4.from_device(d.codes[0], d.scales[0].view(torch.bfloat16), d.biases[0].view(torch.bfloat16))
    ref = orc.route_rule(qorc.q4_gemm(codes, sc, bi, X), **rule)
    for router in (d, same):
        _check(*B.moe_route(B.Routing(router, **rule), B.bf16_tensor(X)), *ref)


def test_softmax_rule_agrees_with_route_topk(B):
    R, X = _grid(1, (256, 512), 0.02, 2.0 ** -10, 255), _grid(2, (40, 512), 1.0, 2.0 ** -3, 40)
    ids, w = B.moe_route(B.Routing(B.bf16_tensor(R), 8), B.bf16_tensor(X))
    ids0, w0 = B.moe_route_topk(B.bf16_tensor(R), B.bf16_tensor(X), 8)
    assert torch.equal(ids, ids0)
    torch.testing.assert_close(w, w0, rtol=2e-6, atol=0)   # expf and an fp32 sum there


def test_outputs_beyond_the_rows_stay(B):
    r = B.Routing(12, 3)
    l = torch.from_numpy(_logits(3, 7, 12)).cuda()
    ids, w = torch.full((9, 3), 77, dtype=torch.int32, device="cuda"), torch.full((9, 3), 5.0, device="cuda")
    B.moe_route_logits(r, l, ids=ids[1:8], weights=w[1:8])
    _check(ids[1:8], w[1:8], *orc.route_rule(l.cpu().numpy(), 3))
    assert (ids[[0, 8]] == 77).all() and (w[[0, 8]] == 5.0).all()


@pytest.mark.parametrize("E,H,q8", [(256, 2048, False), (60, 192, True), (1024, 64, False)])
def test_one_workspace_for_many_calls(B, E, H, q8):
    """A workspace serves calls of few and of many rows in turn, on one stream after the other."""
    if q8:
        router = B.DeviceQ4(np.random.default_rng(1).integers(0, 256, (E, H), dtype=np.uint8).view(np.uint32),
                            synth.to_bf16_bits(np.full((E, H // 64), 2.0 ** -12, np.float32)),
                            synth.to_bf16_bits(np.full((E, H // 64), -2.0 ** -5, np.float32)))
    else:
        router = B.bf16_tensor(_grid(1, (E, H), 0.02, 2.0 ** -10, 255))
    r = B.Routing(router, 7, score="sigmoid")
    ws = B.moe_route_workspace(r, 50)
    side = torch.cuda.Stream()
    for n, T in enumerate((1, 4, 50, 2, 17, 5, 49, 3, 1, 1)):
        X = B.bf16_tensor(_grid(n, (T, H), 1.0, 2.0 ** -3, 40))
        want = B.moe_route(r, X)
        torch.cuda.synchronize()
        with torch.cuda.stream(side if n % 2 else torch.cuda.current_stream()):
            got = B.moe_route(r, X, ws=ws)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert not ws[:256].any()


def test_empty_batch_and_refusals(B):
    r = B.Routing(B.bf16_tensor(_grid(1, (16, 64), 0.02, 2.0 ** -10, 255)), 4)
    X = torch.zeros(3, 64, dtype=torch.bfloat16, device="cuda")
    ids, w = B.moe_route(r, X[:0])
    assert ids.shape == w.shape == (0, 4)
    for bad in (X.float(), X[:, ::2], X.cpu(), torch.zeros(3, 128, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(64, 3, dtype=torch.bfloat16, device="cuda").T):
        with pytest.raises(ValueError):
            B.moe_route(r, bad)
    with pytest.raises(ValueError):
        B.moe_route(r, X, ids=torch.empty(3, 4, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        B.Routing(16, 4, bias=torch.zeros(15, device="cuda"))
    with pytest.raises(B.Q4Error) as e:
        B.moe_route_logits(B.Routing(16, 4, n_groups=3), torch.zeros(3, 16, device="cuda"))
    assert e.value.status == B.EINVAL
    with pytest.raises(B.Q4Error) as e:
        B.moe_route(r, X, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == B.EWORKSPACE


@pytest.mark.parametrize("T", [1, 3, 40, 100])
def test_captured_route_replays(B, T):
    R = B.bf16_tensor(_grid(1, (64, 256), 0.02, 2.0 ** -10, 255))
    r = B.Routing(R, 6, score="sigmoid", bias=torch.linspace(-0.1, 0.1, 64, device="cuda"), n_groups=4, top_groups=2)
    X = B.bf16_tensor(_grid(2, (T, 256), 1.0, 2.0 ** -3, 40))
    ws = B.moe_route_workspace(r, T)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        ids, w = B.moe_route(r, X, ws=ws)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.moe_route(r, X, ids=ids, weights=w, ws=ws)
    for n in range(3):
        X.copy_(B.bf16_tensor(_grid(10 + n, (T, 256), 1.0, 2.0 ** -3, 40)))
        ids.zero_()
        graph.replay()
        got = ids.clone(), w.clone()
        want = B.moe_route(r, X)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("T", [1, 4, 10])
@pytest.mark.parametrize("fill", [1, 2, 15, -1, 2 ** 31 - 1, 0x3F800000])
def test_workspace_that_was_not_zeroed_shows(B, T, fill):
    """Arrival counts that do not start at zero give id -1 and weight NaN in every slot, call after
    call, and not the memory that was there; a zeroed head puts it right."""
    r = B.Routing(B.bf16_tensor(_grid(1, (64, 256), 0.02, 2.0 ** -10, 255)), 6, score="sigmoid")
    X = B.bf16_tensor(_grid(2, (T, 256), 1.0, 2.0 ** -3, 40))
    want = B.moe_route(r, X)
    ws = B.moe_route_workspace(r, T)
    ws.view(torch.int32).fill_(fill)
    ids, w = torch.full_like(want[0], 7), torch.full_like(want[1], 7.0)
    for _ in range(3):
        B.moe_route(r, X, ids=ids, weights=w, ws=ws)
        assert (ids == -1).all() and torch.isnan(w).all()
    ws[:256].zero_()
    B.moe_route(r, X, ids=ids, weights=w, ws=ws)
    assert torch.equal(ids, want[0]) and torch.equal(w, want[1])


def _check_near(ids, w, logits, delta, rule, bias=None):
    """Ids and weights of logits that are each within `delta` [T][E] of these: every id is chosen as
    the rule would for some such logits, and every weight is what it would give them."""
    T, E = logits.shape
    b = np.zeros(E) if bias is None else bias.astype(np.float64)
    if rule["score"] == "sigmoid":
        s, slope = 1.0 / (1.0 + np.exp(-logits)), 0.25
    else:
        s = np.exp(logits - logits.max(1, keepdims=True))
        s, slope = s / s.sum(1, keepdims=True), None
    for t in range(T):
        d = delta[t].max()
        # a sigmoid's slope is 1/4 at most; a softmax score moves by a factor of exp(2 d) at most
        eps = d * slope if slope else np.expm1(2 * d) * s[t].max()
        c, chosen = s[t] + b, ids[t]
        assert len(set(chosen)) == len(chosen) and chosen.min() >= 0 and chosen.max() < E
        left = np.delete(c, chosen)
        assert (c[chosen][:-1] >= c[chosen][1:] - 2 * eps).all()
        assert left.size == 0 or c[chosen].min() >= left.max() - 2 * eps
        want = s[t][chosen]
        if rule["renormalise"]:
            want = want / want.sum()
        # a score, or its share of the chosen ones' sum, moves by a factor of exp(2 d) at most; the
        # weight is rounded once
        bound = want * rule["scale"] * (np.expm1(2 * d) + 2.0 ** -24 * (1 + 2 * d))
        assert (np.abs(w[t] - want * rule["scale"]) <= bound * (1 + 1e-9)).all()


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("E,H,k", [(256, 2048, 8), (60, 1088, 6), (512, 320, 10)])
def test_route_of_ordinary_values(B, E, H, k, q8):
    """Values whose fp32 sums are rounded, through every form of the logits: a row's ids and weights
    belong to logits within the rounding of the exact ones, in whatever order they are summed."""
    X = synth.to_bf16_bits(np.random.default_rng(H).standard_normal((1500, H)).astype(np.float32))
    x = qorc.bf16_to_f64(X)
    if q8:
        mat = synth.q8_matrix(71, 0, synth.ROUTER_STREAM, 0, E, H, scale_std=0.02 / 74)
        router, logits = B.DeviceQ4(*mat), qorc.q4_gemm(*mat, X)
        s, b = (np.repeat(np.abs(qorc.bf16_to_f64(v)), 64, axis=1) for v in mat[1:])
        size = np.abs(x) @ (s * mat[0].view(np.uint8).reshape(E, H) + b).T   # of sum(x q) scale and of sum(x) bias
    else:
        R = synth.to_bf16_bits((np.random.default_rng(E).standard_normal((E, H)) * 0.02).astype(np.float32))
        router, logits = B.bf16_tensor(R), qorc.router_logits(R, X)
        size = np.abs(x) @ np.abs(qorc.bf16_to_f64(R)).T
    # products of two bfloat16 values (or of one and a code) are exact in fp32; a sum of H of them in any order
    # takes at most H roundings on a value's way, a folded group 2 more, each half a step, 2^-24, or a whole
    # one where a matrix core truncates
    delta = size * (H + 2 * (H // 64)) * 2.0 ** -23
    bias = (np.random.default_rng(k).standard_normal(E) * 0.05).astype(np.float32)
    for rule in (dict(top_k=k, score="sigmoid", renormalise=True, scale=2.5), dict(top_k=k, score="softmax", renormalise=True, scale=1.0),
                 dict(top_k=k, score="softmax", renormalise=False, scale=1.0)):
        for T in (1, 3, 20, 21, 64, 300, 1500):
            for b in (None, bias):
                r = B.Routing(router, bias=None if b is None else torch.from_numpy(b).cuda(), **rule)
                ids, w = B.moe_route(r, B.bf16_tensor(X[:T]))
                some = slice(None) if T <= 64 else slice(T % 29, None, 29)
                _check_near(ids[some].cpu().numpy(), w[some].double().cpu().numpy(), logits[:T][some], delta[:T][some], rule, b)


@pytest.mark.parametrize("T,E,H,k", [(1111, 512, 2048, 8), (1111, 512, 1088, 10), (1111, 512, 576, 7), (2080, 256, 2048, 8),
                                     (2080, 256, 768, 8)])
def test_q8_router_over_many_rounds(B, T, E, H, k):
    """The 8-bit router on a grid of more workgroups than compute units, over enough steps of K that
    its two stages are refilled: eight, five (of unequal quarters) and three."""
    rng = np.random.default_rng(E + T + H)
    codes = rng.integers(0, 256, (E, H), dtype=np.uint8).view(np.uint32)
    sc = synth.to_bf16_bits((2.0 ** -12 * rng.integers(1, 4, (E, H // 64))).astype(np.float32))
    bi = synth.to_bf16_bits((-(2.0 ** -5) * rng.integers(1, 4, (E, H // 64))).astype(np.float32))
    X = _grid(T, (T, H), 0.25, 2.0 ** -3, 4)
    rule = dict(top_k=k, score="sigmoid")
    d = B.DeviceQ4(codes, sc, bi)
    some = slice(T % 23, None, 23)
    logits = qorc.q4_gemm(codes, sc, bi, X[some])
    ids, w = B.moe_route(B.Routing(d, **rule), B.bf16_tensor(X))
    _check(ids[some], w[some], *orc.route_rule(logits, **rule))
    ids, w = B.moe_route_topk_q8(d, B.bf16_tensor(X), k)
    ref_ids, ref_w = orc.route_rule(logits, k)
    np.testing.assert_array_equal(ids[some].cpu().numpy(), ref_ids)
    np.testing.assert_allclose(w[some].cpu().numpy(), ref_w, rtol=1e-4, atol=1e-6)
