"""The 8-bit serving operators and the gradient clipping of the QLoRA NF4 layer, as measured cases.

Four operators: ``linear`` (matrix product of int8 codes with token and channel scales), ``rows`` (rows to int8 codes
and scales, and back), ``norm`` (root-mean-square norm with the residual's addition, to int8 codes and scales) and
``clip`` (the global norm of many gradients and their clipping). ``own`` selects the framework's kernels; otherwise the
plain form in elementary torch operations runs."""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6

# Layer sizes of the two models this repository measures: 7B (4096, 11008) and 65B (8192, 22016).
ATTN_7B, MLP_7B, ATTN_65B, MLP_65B = 4096, 11008, 8192, 22016


def listed():
    return [
        # one token through an attention projection: the decode step, latency and weight bytes
        {"name": "linear_1x4096x4096", "op": "linear", "m": 1, "n": ATTN_7B, "k": ATTN_7B, "type": "bf16"},
        # sixteen sequences decoding together through the gate projection
        {"name": "linear_16x11008x4096", "op": "linear", "m": 16, "n": MLP_7B, "k": ATTN_7B, "type": "bf16"},
        # a ragged batch on odd sizes (a projection that no tile divides), float32 out for what is summed outside
        {"name": "linear_333x5003x4100", "op": "linear", "m": 333, "n": 5003, "k": 4100, "type": "fp32"},
        # prefill of 2048 tokens through the 7B down projection
        {"name": "linear_2048x4096x11008", "op": "linear", "m": 2048, "n": ATTN_7B, "k": MLP_7B, "type": "fp16"},
        # prefill of 4096 tokens through a 65B up projection: the largest product
        {"name": "linear_4096x22016x8192", "op": "linear", "m": 4096, "n": MLP_65B, "k": ATTN_65B, "type": "bf16"},
        # a merged float32 weight quantized by channel, once for each deployed adapter
        {"name": "rows_11008x4096_fp32", "op": "rows", "m": MLP_7B, "k": ATTN_7B, "type": "fp32"},
        # a small odd batch of activations in front of the down projection, where no norm precedes
        {"name": "rows_37x11008_bf16", "op": "rows", "m": 37, "k": MLP_7B, "type": "bf16"},
        # the norm of one decoded token: latency
        {"name": "norm_1x4096_bf16", "op": "norm", "m": 1, "k": ATTN_7B, "type": "bf16", "residual": True},
        # the norm of a 65B prefill batch
        {"name": "norm_4096x8192_bf16", "op": "norm", "m": 4096, "k": ATTN_65B, "type": "bf16", "residual": True},
        # odd width, no residual (the first norm of a stack), half precision
        {"name": "norm_777x5001_fp16", "op": "norm", "m": 777, "k": 5001, "type": "fp16", "residual": False},
        # the adapters of one 7B decoder layer at rank 16: fourteen small gradients
        {"name": "clip_7b_layer_fp32", "op": "clip", "layers": 1, "rank": 16, "odd": 0, "type": "fp32"},
        # the adapters of the whole 7B model at rank 16: 448 gradients in one call
        {"name": "clip_7b_model_fp32", "op": "clip", "layers": 32, "rank": 16, "odd": 0, "type": "fp32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "rows", "norm", "clip"])
    kind = rng.choice(["bf16", "fp16", "fp32"])
    if op == "linear":
        return {"op": op, "m": _log(rng, 1, 4096), "n": _log(rng, 64, MLP_65B), "k": _log(rng, 64, MLP_7B), "type": kind}
    if op == "rows":
        return {"op": op, "m": _log(rng, 1, MLP_7B), "k": _log(rng, 16, ATTN_65B), "type": kind}
    if op == "norm":
        return {"op": op, "m": _log(rng, 1, 4096), "k": _log(rng, 16, ATTN_65B), "type": kind, "residual": rng.random() < 0.7}
    return {"op": op, "layers": _log(rng, 1, 32), "rank": rng.choice([4, 8, 15, 16]), "odd": rng.randint(0, 99), "type": kind}


def _sizes(case):
    """Elements of each adapter gradient: A (rank x inputs) and B (outputs x rank) of the seven projections of each layer;
    ``odd`` takes that many elements from every second one."""
    one = [(ATTN_7B, ATTN_7B)] * 4 + [(MLP_7B, ATTN_7B)] * 2 + [(ATTN_7B, MLP_7B)]
    return [s for n, k in one for s in (case["rank"] * k, case["rank"] * n - case["odd"])] * case["layers"]


def _padded(k):
    return -(-k // 64) * 64


def _codes(g, rows, k):
    """int8 codes as a quantizer leaves them: a normal's values on a grid of a third of its range, zeros up to the padded width."""
    codes = torch.zeros(rows, _padded(k), dtype=torch.int8, device="cuda")
    codes[:, :k] = (torch.randn(rows, k, generator=g, device="cuda") * 32).round().clamp_(-127, 127).to(torch.int8)
    return codes


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    t = TYPES.get(case["type"])
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        return {"case": case, "x": _codes(g, m, k), "w": _codes(g, n, k),
                "sx": (rand(m).abs() + 0.5) / 32, "sw": (rand(n).abs() + 0.5) / 1600}
    if case["op"] == "rows":
        return {"case": case, "x": (rand(case["m"], case["k"]) * (rand(case["m"], 1).abs() + 0.1)).to(t)}
    if case["op"] == "norm":
        m, k = case["m"], case["k"]
        return {"case": case, "x": rand(m, k).to(t), "gain": (1 + 0.2 * rand(k)).to(t),
                "residual": (rand(m, k) * 3).to(t) if case["residual"] else None}
    # one tensor for each gradient, as the backward passes leave them in buffers that the training loop keeps; the
    # clipped ones go packed to one buffer, which an optimizer or a reduction over ranks reads
    sizes = _sizes(case)
    grads = [v.to(t, copy=True) for v in (rand(sum(sizes)) * 2e-3).split(sizes)]
    state = {"case": case, "grads": grads, "max_norm": 0.3, "clipped": torch.empty(sum(sizes), dtype=t, device="cuda")}
    if own:  # the checked list of these buffers, which such a loop makes once
        import bit_nf4_quantized_18_amd as q

        state["list"] = q.GradList(grads)
    return state


def _plain_rows(v):
    """Values of the 8-bit codes of each row, and the rows' scales."""
    scale = v.abs().amax(dim=1, keepdim=True) / 127
    codes = torch.where(scale > 0, torch.round(v / scale), torch.zeros_like(v))
    return codes * scale, scale[:, 0]


def _plain(state):
    case = state["case"]
    t = TYPES[case["type"]]
    if case["op"] == "linear":
        y = state["x"].float() @ state["w"].float().t()
        return y.mul_(state["sx"][:, None]).mul_(state["sw"]).to(t)
    if case["op"] == "rows":
        values, scale = _plain_rows(state["x"].float())
        return values.to(torch.bfloat16), scale
    if case["op"] == "norm":
        h = state["x"].float()
        if state["residual"] is not None:
            h = h + state["residual"].float()
        r = torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS)
        values, scale = _plain_rows(h * r * state["gain"].float())
        return values.to(torch.bfloat16), scale, (h.to(t) if state["residual"] is not None else None)
    g = torch.cat(state["grads"]).float()
    norm = (g * g).sum().sqrt()
    return norm, (g * torch.clamp(state["max_norm"] / (norm + 1e-6), max=1.0)).to(t)


def run(state):
    if not own:
        return _plain(state)
    import bit_nf4_quantized_18_amd as q

    case = state["case"]
    if case["op"] == "linear":
        k = case["k"]
        w = q.PackedInt8(case["n"], k, state["w"], state["sw"])
        return q.int8_linear_fwd(w, q.PackedInt8(case["m"], k, state["x"], state["sx"]), TYPES[case["type"]])
    if case["op"] == "rows":
        p = q.quantize_int8(state["x"])
        return q.dequantize_int8(p, torch.bfloat16), p.scale
    if case["op"] == "norm":
        p, h = q.rmsnorm_int8(state["x"], state["gain"], EPS, residual=state["residual"])
        return q.dequantize_int8(p, torch.bfloat16), p.scale, h
    return q.grad_clip(state["list"], state["max_norm"], out=state["clipped"]), state["clipped"]


def work(case):
    s = SIZE[case["type"]]
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": (m + n) * (k + 4) + m * n * s, "flops": 2 * m * n * k}
    if case["op"] == "clip":
        total = sum(_sizes(case))
        return {"bytes": 2 * total * s, "flops": 3 * total}
    # the input once, the codes written and read back once, their values in 16 bits, the scales
    m, k = case["m"], case["k"]
    bytes_ = m * k * (s + 1 + 1 + 2) + 8 * m
    if case["op"] == "norm":
        bytes_ += k * s + (2 * m * k * s if case["residual"] else 0)
    return {"bytes": bytes_, "flops": (8 if case["op"] == "norm" else 4) * m * k}


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "linear":
        # whole numbers below 2^53: the product in float64 is exact
        acc = torch.mm(state["x"].double(), state["w"].double().t().contiguous())
        return acc * torch.outer(state["sx"].double(), state["sw"].double())
    if case["op"] == "clip":
        norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(v.double()) for v in state["grads"]]))
        factor = min(1.0, state["max_norm"] / (float(norm) + 1e-6))
        return norm, torch.cat([v.double() * factor for v in state["grads"]])
    v = state["x"].double()
    h = None
    if case["op"] == "norm":
        if state["residual"] is not None:
            v = h = v + state["residual"].double()
        v = v * state["gain"].double() / torch.sqrt(torch.sum(v ** 2, dim=1, keepdim=True) / case["k"] + EPS)
    top = torch.max(torch.abs(v), dim=1, keepdim=True).values
    codes = torch.round(v * 127 / torch.where(top == 0, torch.ones_like(top), top))
    values = codes * (top / 127)
    return (values, top[:, 0] / 127) if case["op"] == "rows" else (values, top[:, 0] / 127, h)
