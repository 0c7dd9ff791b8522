"""The operators of a serving step one after another, as a program uses them: the residual's
addition and norm, routing, 4-bit experts, the next norm (to codes), a head in either form and
the draw of the next token.  Each is checked on the GPU's own input to it; replays of the
captured step, and steps on two streams at once, give the eager step's bits."""
import numpy as np
import pytest
import torch

from oracle import q4moe_oracle as qorc
from oracle import route_i8_oracle as i8orc
from oracle import step_oracle as orc
from tests.test_gpu_mx4 import HALF, HALF_BF16, _bits, _dev, _experts_ref, _rows, _values, _weights
from tests.test_gpu_norm import _check_codes, _check_y
from tests.test_gpu_sample import PROB

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def B():
    from quantized_moe_decode_affine_amd import binding
    assert torch.cuda.is_available()
    binding.load_library()
    return binding


class Step:
    """A block's weights and, for T tokens, every buffer of a step."""

    def __init__(self, B, seed, T, H=256, inter=128, E=12, k=4, V=5003):
        rng = np.random.default_rng(seed)
        shapes = ((inter, H), (inter, H), (H, inter))
        self.B, self.T, self.k = B, T, k
        self.norms = [_rows(seed + 20 + i, 1, H)[0] for i in range(2)]
        self.mats = [_weights(seed + i, E, *s, lo=119, hi=122) for i, s in enumerate(shapes)]
        self.shared = [_weights(seed + 9 + i, 1, *s, lo=119, hi=122) for i, s in enumerate(shapes)]
        self.head8 = (rng.integers(-127, 128, (V, H), dtype=np.int8), (rng.random(V) * 0.002 + 1e-4).astype(np.float32))
        self.head4 = _weights(seed + 30, V, H, lo=118, hi=121)
        self.w = [B.bf16_tensor(w) for w in self.norms]
        self.rule = B.Routing(B.bf16_tensor(_rows(seed + 40, E, H)), k)
        self.experts = B.DeviceMx4Experts(*(_dev(B, m) for m in self.mats), shared=tuple(_dev(B, m) for m in self.shared))
        self.W8 = B.DeviceI8(*(torch.from_numpy(v).cuda() for v in self.head8))
        self.W4 = _dev(B, self.head4)
        new = lambda *s, t=torch.bfloat16: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
        self.x, self.r, self.u = new(T, H), new(T, H), new(T, t=torch.float32)
        self.total, self.y, self.e, self.codes, self.scales, self.y2 = (new(T, H), new(T, H), new(T, H), new(T, H, t=torch.int8),
                                                                        new(T, t=torch.float32), new(T, H))
        self.ids, self.weights = new(T, k, t=torch.int32), new(T, k, t=torch.float32)
        self.l8, self.l4 = new(T, V, t=torch.float32), new(T, V)
        self.pick = [(new(T, t=torch.int32), new(T, t=torch.float32)) for _ in range(2)]
        self.params = (torch.full((T,), 0.8, device="cuda"), torch.tensor([0, 40, 700] * T, dtype=torch.int32, device="cuda")[:T],
                       torch.tensor([1.0, 0.9] * T, device="cuda")[:T], torch.tensor([0.0, 0.02] * T, device="cuda")[:T])
        self.ws = [B.moe_route_workspace(self.rule, T), B.moe_experts_mx4_workspace(self.experts, T, k),
                   B.mx4_gemm_workspace(self.W4, T), B.sample_logits_workspace(T, V)]

    def feed(self, seed):
        for t, s, scale in ((self.x, seed, 1), (self.r, seed + 1, 2)):
            t.copy_(self.B.bf16_tensor(_rows(s, self.T, t.shape[1])) * scale)
        self.u.copy_(torch.from_numpy(np.random.default_rng(seed).random(self.T, dtype=np.float32)))

    def run(self):
        B = self.B
        B.rms_norm(self.x, self.w[0], EPS, residual=self.r, total=self.total, out=self.y)
        B.moe_route(self.rule, self.y, ids=self.ids, weights=self.weights, ws=self.ws[0])
        B.moe_experts_mx4(self.experts, self.y, self.ids, self.weights, B.OUT_BF16, out=self.e, ws=self.ws[1])
        # the residual stream's new state replaces the old one
        B.rms_norm_i8(self.e, self.w[1], EPS, residual=self.total, total=self.r, codes=self.codes, scales=self.scales, out=self.y2)
        B.i8_gemm_rows(self.W8, self.codes, self.scales, out=self.l8)
        B.sample_logits(self.l8, self.u, *self.params, ids=self.pick[0][0], probs=self.pick[0][1], ws=self.ws[3])
        B.mx4_gemm(self.W4, self.y2, B.OUT_BF16, out=self.l4, ws=self.ws[2])
        B.sample_logits(self.l4, self.u, *self.params, ids=self.pick[1][0], probs=self.pick[1][1], ws=self.ws[3])

    def results(self):
        return [t.clone() for t in (self.total, self.y, self.ids, self.weights, self.e, self.r, self.codes, self.scales, self.y2,
                                    self.l8, self.l4, *self.pick[0], *self.pick[1])]


@pytest.mark.parametrize("T", [1, 5, 20, 45])
def test_step(B, T):
    s = Step(B, T, T)
    s.feed(100)
    x, r = _bits(s.x), _bits(s.r)
    s.run()
    f64 = lambda t: qorc.bf16_to_f64(_bits(t))  # noqa: E731
    t, y = orc.rms_norm(x, s.norms[0], EPS, r)
    np.testing.assert_array_equal(f64(s.total), t)
    _check_y(s.y, y)
    ids, w = s.ids.cpu().numpy(), s.weights.cpu().numpy()
    assert ((ids >= 0) & (ids < 12)).all() and (np.sort(ids, 1)[:, 1:] > np.sort(ids, 1)[:, :-1]).all()
    y, tol = _experts_ref(_bits(s.y), ids, w, _values(s.mats), [m[0] for m in _values(s.shared)])
    assert (np.abs(f64(s.e) - y) <= tol * (1 + HALF_BF16) + HALF_BF16 * np.abs(y)).all()
    t, y = orc.rms_norm(_bits(s.e), s.norms[1], EPS, _bits(s.total))
    np.testing.assert_array_equal(f64(s.r), t)
    _check_codes(s.codes, s.scales, y)
    _check_y(s.y2, y)
    q, scale = i8orc.quantize_rows(y)
    ref = (q.astype(np.float64) @ s.head8[0].astype(np.float64).T) * scale[:, None] * s.head8[1].astype(np.float64)
    assert (np.abs(s.l8.double().cpu().numpy() - ref) <= 3.01 * HALF * np.abs(ref)).all()
    q, m = orc.mx4_round(f64(s.y2)), orc.mx4_values(*s.head4)
    ref, size = q @ m.T, np.abs(q) @ np.abs(m).T
    # the sum's fp32 steps, then the rounding to bf16
    assert (np.abs(f64(s.l4) - ref) <= (q.shape[1] * HALF) * size * (1 + HALF_BF16) + HALF_BF16 * np.abs(ref)).all()
    host = [v.cpu().numpy() for v in s.params]
    u, temp, p, least = (np.asarray(v, dtype=np.float64) for v in (s.u.cpu().numpy(), host[0], host[2], host[3]))
    for logits, (got, probs) in ((s.l8, s.pick[0]), (s.l4, s.pick[1])):
        want, prob = orc.sample(logits.double().cpu().numpy(), u, temp, host[1], p, least)
        np.testing.assert_array_equal(got.cpu().numpy(), want)
        np.testing.assert_allclose(probs.double().cpu().numpy(), prob, rtol=PROB, atol=2.0 ** -45 * logits.shape[1])


@pytest.mark.parametrize("T", [3, 40])
def test_step_captured(B, T):
    """Replays with eager steps of other inputs between them; the residual's buffer is both read and written."""
    s, other = Step(B, 1, T), Step(B, 1, T)
    side = torch.cuda.Stream()
    s.feed(1)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.run()
    for seed in range(5):
        s.feed(seed)
        other.feed(seed)
        g.replay()
        other.run()
        assert all(torch.equal(a, b) for a, b in zip(s.results(), other.results())), seed


def test_steps_on_two_streams(B):
    """Two programs at once, each on a stream and workspaces of its own, launched and replayed."""
    steps = [Step(B, 7, 24), Step(B, 8, 33)]
    want = []
    for i, s in enumerate(steps):
        s.feed(50 + i)
        s.run()
        want.append(s.results())
    streams = [torch.cuda.Stream() for _ in steps]
    graphs = []
    torch.cuda.synchronize()
    for s, stream in zip(steps, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            s.run()
        graphs.append(g)
    for replay in (False, True):
        for turn in range(4):
            for i, s in enumerate(steps):
                s.feed(50 + i)
            torch.cuda.synchronize()
            for s, stream, g in zip(steps, streams, graphs):
                with torch.cuda.stream(stream):
                    if replay:
                        g.replay()
                    else:
                        s.run()
            torch.cuda.synchronize()
            for s, w in zip(steps, want):
                assert all(torch.equal(a, b) for a, b in zip(s.results(), w)), (replay, turn)
