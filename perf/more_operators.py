"""The gated feed-forward block of the QLoRA layer and the backward passes from 8-bit activation checkpoints, as measured
cases.

Four operators: ``block`` (gate and up projections of an NF4 weight with their adapters, activation and product in one
call), ``gated`` (the activation and product alone and their gradient, from pre-activations in 16 or 32 bits or in 8-bit
rows), ``int8_block`` (the block's projections in 8-bit integers, with activation and product) and ``backward`` (the NF4
linear's backward pass whose input was kept as 8-bit rows). ``own`` selects the framework's kernels; otherwise the plain
form in elementary torch operations runs."""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
BLOCK, GROUP = 64, 256  # weights of a scale, scales of a group

# Layer sizes of the two models this repository measures: 7B (4096, 11008) and 65B (8192, 22016).
ATTN_7B, MLP_7B, ATTN_65B, MLP_65B = 4096, 11008, 8192, 22016

NF4 = (-1.0, -0.69619292, -0.525073051, -0.394917488, -0.284441352, -0.18477343, -0.0910499915, 0.0, 0.0795803294,
       0.160930172, 0.246112287, 0.337915182, 0.4407098, 0.562616944, 0.722956717, 1.0)


def listed():
    return [
        # one token through the 7B block: the decode step, latency and weight bytes
        {"name": "block_1x11008x4096_bf16", "op": "block", "m": 1, "n": MLP_7B, "k": ATTN_7B, "r": 16, "type": "bf16", "act": "silu", "keep": False},
        # thirteen sequences decoding together, half precision
        {"name": "block_13x11008x4096_fp16", "op": "block", "m": 13, "n": MLP_7B, "k": ATTN_7B, "r": 16, "type": "fp16", "act": "silu", "keep": False},
        # a ragged prompt through a small block, the other activation
        {"name": "block_333x2560x1088_bf16", "op": "block", "m": 333, "n": 2560, "k": 1088, "r": 8, "type": "bf16", "act": "gelu", "keep": False},
        # the 7B training step's forward: the pre-activations are kept for the backward pass
        {"name": "block_2048x11008x4096_bf16", "op": "block", "m": 2048, "n": MLP_7B, "k": ATTN_7B, "r": 16, "type": "bf16", "act": "silu", "keep": True},
        # the down projection's input computed again from the 8-bit checkpoint of a 7B training step
        {"name": "fwd_2048x11008_int8_bf16", "op": "gated", "back": False, "m": 2048, "n": MLP_7B, "rows": True, "type": "bf16", "act": "silu"},
        # odd sizes: a few tokens of an odd width in float32
        {"name": "bwd_37x5001_fp32", "op": "gated", "back": True, "m": 37, "n": 5001, "rows": False, "type": "fp32", "act": "gelu"},
        # the gradient of a 65B training step from the 8-bit checkpoint: the largest pass over memory
        {"name": "bwd_4096x22016_int8_bf16", "op": "gated", "back": True, "m": 4096, "n": MLP_65B, "rows": True, "type": "bf16", "act": "silu"},
        # sixteen sequences decoding through the served 8-bit block
        {"name": "int8_block_16x11008x4096_bf16", "op": "int8_block", "m": 16, "n": MLP_7B, "k": ATTN_7B, "type": "bf16", "act": "silu"},
        # prefill of 4096 tokens through the 65B block in 8 bits: the largest product
        {"name": "int8_block_4096x22016x8192_fp16", "op": "int8_block", "m": 4096, "n": MLP_65B, "k": ATTN_65B, "type": "fp16", "act": "silu"},
        # a small ragged batch through an odd layer at an odd rank
        {"name": "backward_77x1040x1088_fp16", "op": "backward", "m": 77, "n": 1040, "k": 1088, "r": 5, "parts": 1, "type": "fp16"},
        # the 7B down projection of a training step, whose input is the widest one kept
        {"name": "backward_2048x4096x11008_bf16", "op": "backward", "m": 2048, "n": ATTN_7B, "k": MLP_7B, "r": 16, "parts": 1, "type": "bf16"},
        # gate and up of a training step in one grouped call
        {"name": "backward_2048x22016x4096_bf16", "op": "backward", "m": 2048, "n": 2 * MLP_7B, "k": ATTN_7B, "r": 16, "parts": 2, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["block", "block", "gated", "gated", "int8_block", "backward"])
    kind = rng.choice(["bf16", "fp16"])
    act = rng.choice(["silu", "silu", "gelu"])
    if op == "block":
        return {"op": op, "m": _log(rng, 1, 2048), "n": 256 * _log(rng, 1, MLP_7B // 256), "k": 64 * _log(rng, 1, ATTN_65B // 64),
                "r": rng.choice([4, 8, 15, 16, 32]), "type": kind, "act": act, "keep": rng.random() < 0.5}
    if op == "gated":
        rows = rng.random() < 0.5
        return {"op": op, "back": rng.random() < 0.5, "m": _log(rng, 1, 4096), "n": _log(rng, 16, MLP_65B), "rows": rows,
                "type": rng.choice(["bf16", "fp16", "fp32"]), "act": act}
    if op == "int8_block":
        return {"op": op, "m": _log(rng, 1, 4096), "n": _log(rng, 16, MLP_7B), "k": _log(rng, 64, ATTN_65B),
                "type": rng.choice(["bf16", "fp16", "fp32"]), "act": act}
    parts = rng.choice([1, 1, 2, 3])
    if parts == 1:
        n, r = 16 * _log(rng, 1, MLP_7B // 16), rng.choice([4, 8, 15, 16, 64])
    else:
        n, r = 256 * parts * _log(rng, 1, MLP_7B // 256 // parts), rng.choice([16, 32])
    return {"op": op, "m": _log(rng, 1, 2048), "n": n, "k": 64 * _log(rng, 1, MLP_7B // 64), "r": r, "parts": parts, "type": kind}


def _padded(k):
    return -(-k // 64) * 64


def _rows(g, rows, k):
    """int8 codes as a quantizer leaves them: a normal's values on a grid of a third of its range, zeros up to the padded width."""
    codes = torch.zeros(rows, _padded(k), dtype=torch.int8, device="cuda")
    codes[:, :k] = (torch.randn(rows, k, generator=g, device="cuda") * 32).round().clamp_(-127, 127).to(torch.int8)
    return codes


def _weight(g, n, k):
    """The packed buffers of an n x k NF4 weight with 8-bit scales: the levels are equally likely, as for normal weights."""
    groups = -(-n * k // (BLOCK * GROUP))
    return {"codes": torch.randint(0, 256, (n * k // 2,), generator=g, device="cuda", dtype=torch.uint8),
            "scale_codes": torch.randint(120, 256, (n * k // BLOCK,), generator=g, device="cuda", dtype=torch.uint8),
            "group_scale": 0.06 + 0.02 * torch.rand(groups, generator=g, device="cuda")}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    t, m, n, op = TYPES[case["type"]], case["m"], case["n"], case["op"]
    state = {"case": case}
    if op == "gated":
        # pre-activations of unit size, as a normalised input and the weights' scale give them
        if case["rows"]:
            state |= {"codes": _rows(g, 2 * m, n), "scale": (rand(2 * m).abs() + 0.5) / 32}
        else:
            state["y"] = (rand(m, 2 * n) * 1.3).to(t)
        if case["back"]:
            state["dp"] = rand(m, n).to(t)
    elif op == "int8_block":
        k = case["k"]
        state |= {"x": _rows(g, m, k), "w": _rows(g, 2 * n, k), "sx": (rand(m).abs() + 0.5) / 32, "sw": (rand(2 * n).abs() + 0.5) / 1600}
    else:
        k, r = case["k"], case["r"]
        parts = 2 if op == "block" else case["parts"]
        full = 2 * n if op == "block" else n
        state |= {"weight": _weight(g, full, k), "alpha": 2.0 * r, "a": (rand(parts * r, k) / r).to(t), "b": (0.01 * rand(full, r)).to(t)}
        if op == "block":
            state["x"] = rand(m, k).to(t)
        else:
            # the forward's H, its input as 8-bit rows, and the gradient of its output
            state |= {"h": rand(m, parts * r) * 4, "codes": _rows(g, m, k), "scale": (rand(m).abs() + 0.5) / 32, "dy": rand(m, n).to(t)}
        if own:
            import bit_nf4_quantized_18_amd as q

            w = state["weight"]
            state["packed"] = q.PackedNF4(full, k, w["codes"], True, w["scale_codes"], w["group_scale"])
    return state


def _restored(weight, n, k, t):
    """The layer's weight as it multiplies: level times scale, rounded to the compute type."""
    c = weight["codes"]
    codes = torch.stack([c & 15, c >> 4], dim=1).reshape(-1, BLOCK)
    scale = weight["scale_codes"].float() / 255 * weight["group_scale"].repeat_interleave(GROUP)[: codes.shape[0]]
    levels = torch.tensor(NF4, dtype=torch.float32, device="cuda")
    return (levels[codes.int()] * scale[:, None]).to(t).float().view(n, k)


def _sigma(z):
    return 1 / (1 + torch.exp(-z))


def _bent(g, act):
    """The argument of the activation g sigma(z), and dz / dg."""
    if act == "silu":
        return g, torch.ones_like(g)
    c = 2 * math.sqrt(2 / math.pi)
    return c * (g + 0.044715 * g * g * g), c * (1 + 3 * 0.044715 * g * g)


def _halves(state):
    """Gate and up in 32 bits, of the pre-activations or their 8-bit rows (row 2i the gate of token i, 2i + 1 its up)."""
    case = state["case"]
    m, n = case["m"], case["n"]
    if case["rows"]:
        y = (state["codes"][:, :n].float() * state["scale"][:, None]).view(m, 2 * n)
    else:
        y = state["y"].float()
    return y[:, :n], y[:, n:]


def _per_part(rows, parts, r):
    """1 where an output row (of `parts` equal runs) owns an adapter slot."""
    part = torch.arange(rows, device="cuda") * parts // rows
    return (part[:, None] == torch.arange(parts * r, device="cuda")[None, :] // r).float()


def _plain(state):
    case = state["case"]
    t, m, n, op = TYPES[case["type"]], case["m"], case["n"], case["op"]
    if op == "gated":
        gate, up = _halves(state)
        z, slope = _bent(gate, case["act"])
        s = _sigma(z)
        if not case["back"]:
            return (gate * s * up).to(t)
        dp = state["dp"].float()
        return torch.cat([dp * up * (s + gate * s * (1 - s) * slope), dp * gate * s], dim=1).to(t)
    if op == "int8_block":
        y = (state["x"].float() @ state["w"].float().t()).mul_(state["sx"][:, None]).mul_(state["sw"])
        gate, up = y[:, :n], y[:, n:]
        return (gate * _sigma(_bent(gate, case["act"])[0]) * up).to(t)
    k, r = case["k"], case["r"]
    s = state["alpha"] / r
    a = state["a"].float()
    if op == "block":
        x = state["x"].float()
        own_slots = state["b"].float().repeat(1, 2) * _per_part(2 * n, 2, r)
        h = x @ a.t()
        y = x @ _restored(state["weight"], 2 * n, k, t).t() + s * (h @ own_slots.t())
        gate, up = y[:, :n], y[:, n:]
        p = (gate * _sigma(_bent(gate, case["act"])[0]) * up).to(t)
        return (p, y.to(t), h) if case["keep"] else p
    mask = _per_part(n, case["parts"], r)
    own_slots = state["b"].float().repeat(1, case["parts"]) * mask
    dy = state["dy"].float()
    dh = s * (dy @ own_slots)
    dx = (dy @ _restored(state["weight"], n, k, t) + dh @ a).to(t)
    da = dh.t() @ (state["codes"][:, :k].float() * state["scale"][:, None])
    db = ((s * (dy.t() @ state["h"])) * mask).view(n, case["parts"], r).sum(dim=1)
    return dx, da, db


def run(state):
    if not own:
        return _plain(state)
    import bit_nf4_quantized_18_amd as q

    case = state["case"]
    m, n, op = case["m"], case["n"], case["op"]
    if op == "backward":
        x = q.PackedInt8(m, case["k"], state["codes"], state["scale"])
        if case["parts"] == 1:
            return q.linear_bwd(state["packed"], x, state["dy"], state["a"], state["b"], state["alpha"], h=state["h"])
        return q.linear_bwd_grouped(state["packed"], [n // case["parts"]] * case["parts"], x, state["dy"], state["a"], state["b"],
                                    state["alpha"], h=state["h"])
    act = q.ACT_SILU if case["act"] == "silu" else q.ACT_GELU
    if op == "gated":
        y = q.PackedInt8(2 * m, n, state["codes"], state["scale"]) if case["rows"] else state["y"]
        return q.gated_bwd(y, state["dp"], act) if case["back"] else q.gated_fwd(y, act, dtype=TYPES[case["type"]])
    if op == "int8_block":
        w = q.PackedInt8(2 * n, case["k"], state["w"], state["sw"])
        return q.int8_linear_fwd_gated(w, q.PackedInt8(m, case["k"], state["x"], state["sx"]), act, TYPES[case["type"]])
    p, y, h = q.linear_fwd_gated(state["packed"], state["x"], state["a"], state["b"], state["alpha"], act, want_y=case["keep"],
                                 want_h=case["keep"])
    return (p, y, h) if case["keep"] else p


def work(case):
    s, m, n = SIZE[case["type"]], case["m"], case["n"]
    if case["op"] == "gated":
        y = 2 * m * (n + 4) if case["rows"] else 2 * m * n * s
        return {"bytes": y + (3 if case["back"] else 1) * m * n * s, "flops": (24 if case["back"] else 12) * m * n}
    k = case["k"]
    if case["op"] == "int8_block":
        return {"bytes": (m + 2 * n) * (k + 4) + m * n * s, "flops": 4 * m * n * k}
    r = case["r"]
    if case["op"] == "block":
        full, slots = 2 * n, 2 * r
        extra = (m * full * s + 4 * m * slots if case["keep"] else 0) + m * n * s + m * k * s
        flops = 2 * m * full * k + 2 * m * slots * k + 2 * m * r * full
    else:
        full, slots = n, case["parts"] * r
        extra = m * full * s + m * (k + 4) + 4 * m * slots + m * k * s + 4 * (slots * k + full * r)
        flops = 2 * m * full * k + 4 * m * r * full + 4 * m * slots * k
    weight = full * k // 2 + full * k // BLOCK + full * k // (BLOCK * GROUP) * 4
    return {"bytes": weight + (slots * k + full * r) * s + extra, "flops": flops}


def exact(case, seed):
    state = prepare(case, seed)
    m, n, op = case["m"], case["n"], case["op"]

    def activated(v):  # the activation and its derivative
        if case["act"] == "silu":
            sig = torch.special.expit(v)
            return v * sig, sig + v * sig * torch.special.expit(-v)
        inner = math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
        th = torch.tanh(inner)
        return 0.5 * v * (1 + th), 0.5 * (1 + th) + 0.5 * v * (1 - th ** 2) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * v ** 2)

    if op == "gated":
        if case["rows"]:
            v = (state["codes"].double() * state["scale"].double().unsqueeze(1)).view(m, 2, -1)[:, :, :n]
        else:
            v = state["y"].double().view(m, 2, n)
        value, slope = activated(v[:, 0])
        if not case["back"]:
            return value * v[:, 1]
        dp = state["dp"].double()
        return torch.stack([dp * v[:, 1] * slope, dp * value], dim=1).view(m, 2 * n)
    if op == "int8_block":
        # whole numbers below 2^53: the products in float64 are exact
        v = torch.mm(state["x"].double(), state["w"].double().t().contiguous()) * torch.outer(state["sx"].double(), state["sw"].double())
        return activated(v[:, :n])[0] * v[:, n:]
    k, r = case["k"], case["r"]
    full = 2 * n if op == "block" else n
    parts = 2 if op == "block" else case["parts"]
    # the weight as its definition gives it: float32 steps, then the compute type
    c = state["weight"]["codes"].long()
    level = torch.tensor(NF4, dtype=torch.float32, device="cuda")[torch.stack([c % 16, c // 16], dim=-1).flatten()]
    unit = (state["weight"]["scale_codes"].double() / 255).float()
    at = torch.arange(unit.numel(), device="cuda")
    scale = (unit * state["weight"]["group_scale"][at // GROUP]).repeat_interleave(BLOCK)
    w = (level * scale).to(TYPES[case["type"]]).double().view(full, k)
    s = float(state["alpha"]) / r
    a = state["a"].double().view(parts, r, k)
    b = state["b"].double().view(parts, full // parts, r)
    if op == "block":
        x = state["x"].double()
        h = [torch.mm(x, a[l].t().contiguous()) for l in range(parts)]
        v = [torch.mm(x, w[l * n:(l + 1) * n].t().contiguous()) + s * torch.mm(h[l], b[l].t().contiguous()) for l in range(parts)]
        p = activated(v[0])[0] * v[1]
        return (p, torch.cat(v, dim=1), torch.cat(h, dim=1)) if case["keep"] else p
    dy = state["dy"].double()
    by_part = dy.view(m, parts, full // parts)
    x = state["codes"][:, :k].double() * state["scale"].double().unsqueeze(1)
    h = state["h"].double().view(m, parts, r)
    dh = [s * torch.mm(by_part[:, l].contiguous(), b[l].contiguous()) for l in range(parts)]
    dx = torch.mm(dy, w)
    for l in range(parts):
        dx += torch.mm(dh[l], a[l].contiguous())
    da = torch.cat([torch.mm(dh[l].t().contiguous(), x) for l in range(parts)])
    db = torch.cat([s * torch.mm(by_part[:, l].t().contiguous(), h[:, l].contiguous()) for l in range(parts)])
    return dx, da, db
