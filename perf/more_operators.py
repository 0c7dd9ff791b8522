"""Cases that measure four operators of the library around its experts' products: the root-mean-square
norm with the residual's addition and an output in 8 bits (``rms_norm``, ``rms_norm_i8``), microscaled
4-bit floating point, its quantization and product (``mx4_quantize``, ``mx4_gemm``), the experts'
feed-forward on such products (``moe_experts_mx4``), and sampling of the next token with temperature,
top-k, top-p and min-p from given random numbers (``sample_logits``).

``own`` chooses what ``run`` computes with: the library's calls, or the operators' plain forms in
elementary torch operations.  Sizes are those of the benchmark's layer (hidden 2048, 256 routed
experts and one shared, intermediate 512, top-8, 2,048-token chunks, vocabulary 151,936), of the
tests' wider shapes and odd ones between.
"""
import math

import torch

own = False

VOCAB = 151936
EPS = 1e-6


def listed():
    return [
        # one decode step's hidden vector, residual added, codes for an 8-bit product: latency
        dict(name="norm_token_i8", op="norm", rows=1, k=2048, residual=True, i8=True),
        # a long prefill's rows between two layers, in bf16: bytes
        dict(name="norm_chunk", op="norm", rows=8191, k=4096, residual=True, i8=False),
        # a checkpoint's expert matrices on their way to 4 bits, and read back
        dict(name="mx4_pack", op="pack", rows=16384, k=2048),
        # one token through one expert's gate and up together: the smallest product
        dict(name="mx4_token", op="gemm", m=1, n=1024, k=2048, out="bf16"),
        # eight requests' logits: the LM head's weights streamed once
        dict(name="mx4_head_batch", op="gemm", m=8, n=VOCAB, k=2048, out="f32"),
        # a ragged batch on an odd number of channels, columns that no tile divides
        dict(name="mx4_ragged", op="gemm", m=381, n=1027, k=832, out="f32"),
        # a long prefill through a wide projection: compute-bound
        dict(name="mx4_chunk", op="gemm", m=8192, n=8192, k=4096, out="bf16"),
        # one decode step through the benchmark's layer
        dict(name="experts_mx4_token", op="experts", T=1, E=256, H=2048, I=512, k=8, shared=True, empty=0.0),
        # the prefill chunk through the benchmark's layer
        dict(name="experts_mx4_chunk", op="experts", T=2048, E=256, H=2048, I=512, k=8, shared=True, empty=0.0),
        # one request's next token, the usual filters: latency
        dict(name="sample_token", op="sample", B=1, V=VOCAB, dtype="f32", spread=2.5, top_k=True, top_p=True,
             min_p=False, banned=0.0),
        # a full batch of requests, each with parameters of its own, greedy ones among them
        dict(name="sample_batch", op="sample", B=256, V=VOCAB, dtype="f32", spread=2.5, top_k=True, top_p=True,
             min_p=True, banned=0.02),
        # requests with a temperature and top-p alone, bf16 logits (many equal ones) of an odd vocabulary
        dict(name="sample_bf16_odd", op="sample", B=37, V=32003, dtype="bf16", spread=1.5, top_k=False, top_p=True,
             min_p=False, banned=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "pack", "gemm", "experts", "sample", "sample"))
    if op == "norm":
        rows = _log(rng, 1, 8192)
        k = 64 * _log(rng, 1, min(256, 524288 // rows))
        return dict(op=op, rows=rows, k=k, residual=rng.random() < 0.7, i8=rng.random() < 0.5)
    if op == "pack":
        rows = _log(rng, 1, 65536)
        return dict(op=op, rows=rows, k=64 * _log(rng, 1, min(256, (1 << 19) // rows)))
    if op == "gemm":
        m, k = _log(rng, 1, 8192), 64 * _log(rng, 4, 64)
        n = _log(rng, 16, min(VOCAB, 8192 * 8192 * 4096 // (m * k), 2048 * VOCAB // k, (1 << 27) // m))
        return dict(op=op, m=m, n=n, k=k, out=rng.choice(("f32", "bf16")))
    if op == "experts":
        k = _log(rng, 1, 8)
        H, inter = 64 * _log(rng, 4, 32), 64 * _log(rng, 1, 8)
        return dict(op=op, T=_log(rng, 1, 2048), E=max(k, _log(rng, 8, 256)), H=H, I=inter, k=k,
                    shared=rng.random() < 0.5, empty=rng.choice((0.0, 0.1)))
    return dict(op=op, B=_log(rng, 1, 256), V=_log(rng, 500, VOCAB), dtype=rng.choice(("f32", "bf16")),
                spread=rng.choice((1.0, 2.0, 3.0)), top_k=rng.random() < 0.6, top_p=rng.random() < 0.6,
                min_p=rng.random() < 0.4, banned=rng.choice((0.0, 0.1)))


def _rows(gen, m, k):
    """Activations: normal, tokens of different size, some outlier channels."""
    x = torch.randn(m, k, generator=gen, device="cuda")
    x *= torch.exp(0.5 * torch.randn(m, 1, generator=gen, device="cuda"))
    x *= 1 + 7 * (torch.rand(1, k, generator=gen, device="cuda") < 0.01)
    return x.to(torch.bfloat16)


def _weights(gen, count, n, k):
    """Codes (two to a byte) and block scales (exponents) as normal weights of a channel's size have them."""
    codes = torch.empty(count, n, k // 2, dtype=torch.uint8, device="cuda")
    for c in codes.split(max(1, (1 << 28) // (n * k))):
        # how often each of the 16 codes occurs: magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6
        share = torch.tensor([0.08, 0.16, 0.16, 0.14, 0.2, 0.14, 0.09, 0.03], device="cuda").cumsum(0)
        pick = [torch.searchsorted(share, torch.rand(c.shape, generator=gen, device="cuda")).clamp_(max=7).to(torch.uint8)
                for _ in range(2)]
        sign = torch.randint(0, 4, c.shape, generator=gen, device="cuda", dtype=torch.uint8)
        c.copy_((pick[0] | (sign & 1) << 3) | (pick[1] | (sign >> 1) << 3) << 4)
    scales = torch.randint(120, 123, (count, n, k // 32), generator=gen, device="cuda", dtype=torch.uint8)
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    if case["op"] == "norm":
        s["X"] = _rows(gen, case["rows"], case["k"])
        s["R"] = (2 * torch.randn(case["rows"], case["k"], generator=gen, device="cuda")).bfloat16() if case["residual"] else None
        s["w"] = (1 + 0.2 * torch.randn(case["k"], generator=gen, device="cuda")).bfloat16()
    elif case["op"] == "pack":
        w = torch.randn(case["rows"], case["k"], generator=gen, device="cuda")
        w *= 0.02 * torch.exp(0.3 * torch.randn(case["rows"], 1, generator=gen, device="cuda"))
        s["X"] = w.bfloat16()
    elif case["op"] == "gemm":
        s["X"] = _rows(gen, case["m"], case["k"])
        s["W"] = _weights(gen, 1, case["n"], case["k"])
    elif case["op"] == "experts":
        T, E, H, inter, k = case["T"], case["E"], case["H"], case["I"], case["k"]
        s["X"] = _rows(gen, T, H)
        s["gate"], s["up"], s["down"] = _weights(gen, E, inter, H), _weights(gen, E, inter, H), _weights(gen, E, H, inter)
        if case["shared"]:
            s["sh"] = _weights(gen, 1, inter, H), _weights(gen, 1, inter, H), _weights(gen, 1, H, inter)
        logits = torch.randn(T, E, generator=gen, device="cuda") + 0.3 * torch.randn(1, E, generator=gen, device="cuda")
        top = torch.topk(logits, k)
        s["w"] = torch.softmax(top.values, 1)
        s["ids"] = top.indices.int()
        s["ids"][torch.rand(T, k, generator=gen, device="cuda") < case["empty"]] = -1
        # rows of the fullest expert: what a padded batch of products is sized by
        s["cap"] = int(torch.bincount(s["ids"].flatten().long() + 1, minlength=E + 1)[1:].max())
    else:
        B, V = case["B"], case["V"]
        x = torch.randn(B, V, generator=gen, device="cuda") * case["spread"]
        likely = torch.randint(0, V, (B, 12), generator=gen, device="cuda")  # what a context makes likely
        x.scatter_(1, likely, 2 + 4 * case["spread"] * torch.rand(B, 12, generator=gen, device="cuda"))
        x.masked_fill_(torch.rand(B, V, generator=gen, device="cuda") < case["banned"], -math.inf)
        s["logits"] = x.bfloat16() if case["dtype"] == "bf16" else x
        s["u"] = torch.rand(B, generator=gen, device="cuda")

        def choose(*values):
            of = torch.tensor(values, device="cuda")
            return of[torch.randint(0, len(values), (B,), generator=gen, device="cuda")]

        s["t"] = choose(0.7, 1.0, 1.0, 1.3) if B == 1 else choose(0.0, 0.7, 0.7, 1.0, 1.0, 1.0, 1.3)
        s["k"] = choose(20, 50, 200).int() if B == 1 else choose(0, 1, 20, 50, 50, 1000).int()
        s["p"] = choose(0.8, 0.9, 0.95) if B == 1 else choose(0.5, 0.8, 0.9, 0.95, 1.0)
        s["m"] = choose(0.02, 0.05) if B == 1 else choose(0.0, 0.02, 0.05, 0.1)
        for name, here in (("k", case["top_k"]), ("p", case["top_p"]), ("m", case["min_p"])):
            s[name] = s[name] if here else None
    if own:
        s["lib"] = _handles(s)
    return s


def _handles(s):
    """The descriptors, output buffers and workspace that a program keeps from call to call."""
    from quantized_moe_decode_affine_amd import binding as B
    if s["op"] in ("norm", "pack"):
        return (B,)
    if s["op"] == "sample":
        return B, B.sample_logits_workspace(s["B"], s["V"])
    if s["op"] == "gemm":
        W = B.DeviceMx4(*s["W"])
        return B, W, B.OUT_BF16 if s["out"] == "bf16" else B.OUT_F32, B.mx4_gemm_workspace(W, s["m"])
    ex = B.DeviceMx4Experts(*(B.DeviceMx4(*s[n]) for n in ("gate", "up", "down")),
                            shared=tuple(B.DeviceMx4(*w) for w in s["sh"]) if s["shared"] else None)
    return B, ex, B.moe_experts_mx4_workspace(ex, s["T"], s["k"])


def run(s):
    if own:
        B = s["lib"][0]
        if s["op"] == "norm":
            if s["i8"]:
                codes, scales, *total = B.rms_norm_i8(s["X"], s["w"], EPS, residual=s["R"])
                return (codes * scales[:, None], *total)  # the values that the codes stand for
            y = B.rms_norm(s["X"], s["w"], EPS, residual=s["R"])
            return y
        if s["op"] == "pack":
            return B.mx4_dequantize(*B.mx4_quantize(s["X"]))
        if s["op"] == "gemm":
            return B.mx4_gemm(s["lib"][1], s["X"], s["lib"][2], ws=s["lib"][3])
        if s["op"] == "experts":
            return B.moe_experts_mx4(s["lib"][1], s["X"], s["ids"], s["w"], B.OUT_BF16, ws=s["lib"][2])
        return B.sample_logits(s["logits"], s["u"], s["t"], s["k"], s["p"], s["m"], ws=s["lib"][1])
    return {"norm": _plain_norm, "pack": _plain_pack, "gemm": _plain_gemm, "experts": _plain_experts,
            "sample": _plain_sample}[s["op"]](s)


# ---- plain forms

def _plain_norm(s):
    total = s["X"] if s["R"] is None else (s["X"].float() + s["R"].float()).bfloat16()
    h = total.double()
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * s["w"].double()
    if s["i8"]:  # the borders between codes in 64 bits
        scale = (y.abs().amax(1, keepdim=True) / 127).float()
        q = torch.round(y / torch.where(scale > 0, scale, 1.0).double()).clamp(-127, 127)
        y = q.float() * scale
    else:
        y = y.bfloat16()
    return (y,) if s["R"] is None and s["i8"] else y if s["R"] is None else (y, total)


def _mx4_values(x):
    """float32 rows as the values that their microscaled 4-bit form stands for."""
    g = x.unflatten(-1, (-1, 32))
    # the block's scale: 2 to the exponent of its largest magnitude, less the 2 of 4-bit's own largest, 6
    e = torch.frexp(g.abs().amax(-1, keepdim=True)).exponent - 3
    a = torch.ldexp(g, -e)
    m = a.abs()
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    q = (torch.round(m / step) * step).clamp(max=6) * torch.sign(a)
    return torch.ldexp(q, e).flatten(-2)


def _plain_pack(s):
    return _mx4_values(s["X"].float()).bfloat16()


def _unpacked(codes, scales):
    """The float32 values of codes [.., k/2] (a byte's low four bits first) and block exponents [.., k/32]."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()
    m = (c & 7).float()
    m = torch.where(m < 4, 0.5 * m, torch.where(m < 6, m - 2, 2 * m - 8))
    v = torch.where(c > 7, -m, m).unflatten(-1, (-1, 32))
    return torch.ldexp(v, scales.int()[..., None] - 127).flatten(-2)


def _plain_gemm(s):
    y = _mx4_values(s["X"].float()) @ _unpacked(*(w[0] for w in s["W"])).T
    return y.bfloat16() if s["out"] == "bf16" else y


def _silu(x):
    return x / (1 + torch.exp(-x))


def _product(x, weight):
    """Batches of rows x [b, r, k] against weights [b, n, k]: [b, r, n]."""
    return torch.bmm(_unpacked(*weight), x.transpose(1, 2).contiguous()).transpose(1, 2)


def _expert(x, gate, up, down):
    return _product(_mx4_values((_silu(_product(x, gate)) * _product(x, up)).contiguous()), down)


def _plain_experts(s):
    T, k, E, H = s["T"], s["k"], s["E"], s["H"]
    x = _mx4_values(s["X"].float())
    ids = s["ids"].flatten().long()
    rows = torch.arange(T * k, device=ids.device)
    there = (ids >= 0)[:, None]
    if T * k <= E:  # few rows: each with its own copy of its expert's weights
        e = ids.clamp(min=0)
        y = _expert(x[rows // k][:, None], *(tuple(w[e] for w in s[n]) for n in ("gate", "up", "down")))[:, 0]
    else:  # a padded batch of each expert's rows
        first = ids.clamp(min=0)
        order = torch.where(ids >= 0, ids, E).sort(stable=True).indices
        starts = torch.bincount(ids + 1, minlength=E + 1).cumsum(0)[:-1] - torch.bincount(ids + 1, minlength=E + 1)[0]
        place = torch.empty_like(rows).scatter_(0, order, rows) - starts[first]
        at = torch.where(ids >= 0, first * s["cap"] + place, E * s["cap"])
        xp = torch.zeros(E * s["cap"] + 1, H, device=ids.device).index_copy_(0, at, x[rows // k] * there)
        y = _expert(xp[:-1].view(E, -1, H), s["gate"], s["up"], s["down"]).flatten(0, 1)[at.clamp(max=E * s["cap"] - 1)]
    y = (torch.where(there, y, 0.0).view(T, k, H) * s["w"][..., None]).sum(1)
    if s["shared"]:
        y = y + _expert(x[None], *s["sh"])[0]
    return y.bfloat16()


def _plain_sample(s):
    B, V = s["B"], s["V"]
    x = s["logits"].double()
    greedy = s["t"] <= 0
    x = (x - x.amax(1, keepdim=True)) / torch.where(greedy, 1.0, s["t"]).double()[:, None]
    order = x.sort(dim=1, descending=True, stable=True)
    w = torch.exp(order.values)
    place = torch.arange(V, device=x.device)
    keep = torch.ones_like(w, dtype=torch.bool)
    if s["k"] is not None:
        keep = place < torch.where(s["k"] > 0, s["k"], V)[:, None]
    if s["p"] is not None:  # a token stays while those before it do not reach the share
        kept = torch.where(keep, w, 0.0)
        before = kept.cumsum(1) - kept
        keep = keep & ((before < s["p"].double()[:, None] * kept.sum(1, keepdim=True)) | (s["p"] >= 1)[:, None])
    if s["m"] is not None:
        keep = keep & (w >= s["m"].double()[:, None])
    keep = keep & (~greedy[:, None] | (place == 0))
    w = torch.zeros_like(w).scatter_(1, order.indices, torch.where(keep, w, 0.0))  # in the vocabulary's order again
    total = w.cumsum(1)
    last = total[:, -1:]
    ids = (total <= s["u"].double()[:, None] * last).sum(1, keepdim=True)
    return ids[:, 0].int(), (w.gather(1, ids) / last)[:, 0].float()


# ---- the definitions in 64 bits

def _exact_norm(s):
    total = s["X"].double()
    if s["R"] is not None:
        total = (total + s["R"].double()).to(torch.bfloat16)
    h = total.double()
    rms = torch.linalg.vector_norm(h, dim=1).square() / s["k"] + EPS
    y = h * s["w"].double() * rms.pow(-0.5)[:, None]
    if s["i8"]:
        step = (torch.linalg.vector_norm(y, math.inf, dim=1) / 127).to(torch.float32).double()[:, None]
        y = (y / step.masked_fill(step == 0, 1.0)).round() * step
    if s["R"] is None:
        return (y,) if s["i8"] else y
    return y, total.double()


_LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # e2m1's magnitudes, by code


def _exact_mx4(x):
    """Rows as what their 4-bit form stands for: each magnitude goes to the nearest level, between two to the even code."""
    d = x.double().reshape(*x.shape[:-1], -1, 32)
    top = d.abs().max(dim=-1, keepdim=True).values
    unit = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -120))) - 2)
    level = torch.tensor(_LEVELS, dtype=torch.float64, device=x.device)
    a = d.abs() / unit
    code = torch.zeros_like(a, dtype=torch.long)
    for c in range(7):
        border = (level[c] + level[c + 1]) / 2
        code += (a > border) | ((a == border) & (c % 2 == 1))
    return (level[code] * unit * d.sign()).reshape(x.shape)


def _exact_unpack(codes, scales):
    level = torch.tensor(_LEVELS + tuple(-v for v in _LEVELS), dtype=torch.float64, device=codes.device)
    v = torch.empty(*codes.shape[:-1], codes.shape[-1] * 2, dtype=torch.float64, device=codes.device)
    v[..., 0::2] = level[(codes % 16).long()]
    v[..., 1::2] = level[(codes // 16).long()]
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def _exact_gemm(s):
    q = _exact_mx4(s["X"])
    codes, scales = s["W"]
    return torch.cat([q @ _exact_unpack(c, w).T for c, w in zip(codes[0].split(16384), scales[0].split(16384))], 1)


def _exact_expert(q, gate, up, down):
    g = q @ _exact_unpack(*gate).T
    h = g * torch.sigmoid(g) * (q @ _exact_unpack(*up).T)
    return _exact_mx4(h) @ _exact_unpack(*down).T


def _exact_experts(s):
    q = _exact_mx4(s["X"])
    y = torch.zeros(s["T"], s["H"], dtype=torch.float64, device=q.device)
    for e in range(s["E"]):
        t, slot = torch.nonzero(s["ids"] == e, as_tuple=True)
        if len(t):
            part = _exact_expert(q[t], *((s[n][0][e], s[n][1][e]) for n in ("gate", "up", "down")))
            y.index_add_(0, t, part * s["w"][t, slot].double()[:, None])
    if s["shared"]:
        y += _exact_expert(q, *((c[0], w[0]) for c, w in s["sh"]))
    return y


def _exact_sample(s):
    ids, probs = [], []
    for b in range(s["B"]):
        logits = s["logits"][b].double()
        rank = torch.argsort(-logits, stable=True)  # the best first, the lower index of equals
        t = float(s["t"][b])
        n = 1 if t <= 0 else s["V"]
        if s["k"] is not None and int(s["k"][b]) > 0:
            n = min(n, int(s["k"][b]))
        part = torch.softmax(logits[rank[:n]] / (t if t > 0 else 1.0), 0)
        if s["p"] is not None and float(s["p"][b]) < 1:
            reached = torch.nonzero(part.cumsum(0) >= float(s["p"][b]))
            n = int(reached[0]) + 1 if len(reached) else n
        part = part[:n]
        if s["m"] is not None:
            n = int((part / part[0] >= float(s["m"][b])).sum())
        chosen, back = rank[:n].sort()
        share = part[:n][back] / part[:n].sum()
        at = min(int((share.cumsum(0) <= float(s["u"][b])).sum()), n - 1)
        ids.append(int(chosen[at]))
        probs.append(float(share[at]))
    dev = s["logits"].device
    return torch.tensor(ids, dtype=torch.int32, device=dev), torch.tensor(probs, dtype=torch.float64, device=dev)


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "pack": lambda s: _exact_mx4(s["X"]), "gemm": _exact_gemm, "experts": _exact_experts,
            "sample": _exact_sample}[case["op"]](s)


def work(case):
    if case["op"] == "norm":
        n = case["rows"] * case["k"]
        moved = 2 + (4 if case["residual"] else 0) + (1 if case["i8"] else 2)  # in, the residual in and out, the result
        return {"bytes": n * moved + 2 * case["k"] + (4 * case["rows"] if case["i8"] else 0), "flops": 4 * n}
    if case["op"] == "pack":  # to codes and block scales, and back to bf16
        n = case["rows"] * case["k"]
        return {"bytes": n * (2 + 2 + 2 * (0.5 + 1 / 32)), "flops": 2 * n}
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": n * k * (0.5 + 1 / 32) + 2 * m * k + m * n * (2 if case["out"] == "bf16" else 4), "flops": 2 * m * n * k}
    if case["op"] == "experts":
        T, E, H, inter, k = case["T"], case["E"], case["H"], case["I"], case["k"]
        slots = T * k * (1 - case["empty"])
        distinct = E * (1 - (1 - 1 / E) ** slots) if T > 1 else slots  # experts that any token chose
        rows = slots + T * case["shared"]
        return {"bytes": (distinct + case["shared"]) * 3 * H * inter * (0.5 + 1 / 32) + 4 * T * H + 8 * T * k,
                "flops": 6 * H * inter * rows}
    B, V = case["B"], case["V"]
    return {"bytes": B * (V * (2 if case["dtype"] == "bf16" else 4) + 28), "flops": 4 * B * V}
