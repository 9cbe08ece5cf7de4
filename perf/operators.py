"""What is measured of the router's losses, the MXFP4 quantisation and the MXFP4 expert MLP, and their plain forms.

Three operators of a mixture-of-experts layer:

* "router": one training step of the router.  Logits -> the k experts of every token and their probabilities, how
  many tokens went to each expert, the load-balance loss and the z-loss; then, from the gradients of the
  probabilities and of the two losses, the gradient of the logits.  Masked tokens (padding) get probabilities and
  gradients of zero and count nowhere.
* "quant": bf16 or fp32 rows -> 4-bit codes with one power-of-two scale per 32 values (MXFP4), returned as the values
  that the codes and scales stand for.
* "mlp": the grouped expert MLP with MXFP4 weights and activations, from routed tokens to the combined output.

`run` computes them with elementary torch operations in 32 bits, or through the package where `own` is true;
`exact` computes them in 64 bits from their definitions, written apart from both.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 32
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # magnitudes of E2M1


# ----------------------------------------------------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------------------------------------------------
def listed():
    return [
        # router of the smallest layer: a handful of microseconds, latency only
        dict(name="router tiny", op="router", T=512, E=4, k=2, dtype="f32", masked=False),
        # a padded bf16 batch of the 32-expert layer: ties between bf16 logits, masked tokens
        dict(name="router 32 experts bf16", op="router", T=8192, E=32, k=4, dtype="bf16", masked=True),
        # a training batch of the 128-expert layer
        dict(name="router 128 experts", op="router", T=16384, E=128, k=8, dtype="f32", masked=False),
        # the largest router (256 experts) over a long batch, partly padded: bandwidth counts
        dict(name="router 256 experts long", op="router", T=262144, E=256, k=8, dtype="f32", masked=True),
        # activations of one small batch
        dict(name="quant tokens", op="quant", rows=512, K=256, dtype="bf16"),
        # activations whose width is no multiple of 128
        dict(name="quant width 2880", op="quant", rows=8191, K=2880, dtype="bf16"),
        # W_gate_up of all eight experts of the Mixtral layer
        dict(name="quant weights", op="quant", rows=229376, K=4096, dtype="bf16"),
        # one new token through the 128-expert layer
        dict(name="mlp one token", op="mlp", T=1, H=2048, I=768, E=128, k=8, skew=1.5),
        # a decoding batch through the 32-expert layer (2880 is no multiple of 128)
        dict(name="mlp decode batch", op="mlp", T=64, H=2880, I=2880, E=32, k=4, skew=0.0),
        # a prompt through the 128-expert layer with skewed routing: tiny, empty and very large groups
        dict(name="mlp ragged prompt", op="mlp", T=4096, H=2048, I=768, E=128, k=8, skew=1.5),
        # prompts through the 32-expert layer, an odd number of tokens
        dict(name="mlp odd prompt", op="mlp", T=8191, H=2880, I=2880, E=32, k=4, skew=0.0),
        # two full sequences through the Mixtral layer
        dict(name="mlp long prompts", op="mlp", T=8192, H=4096, I=14336, E=8, k=2, skew=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["router", "quant", "mlp", "mlp"])
    if op == "router":
        E = _log(rng, 2, 256)
        k = rng.randint(1, min(E, 16))
        T = max(1, min(_log(rng, 1, 262144), (262144 * 256) // E))
        return dict(op=op, T=T, E=E, k=k, dtype=rng.choice(["f32", "bf16"]), masked=rng.random() < 0.5)
    if op == "quant":
        K = BLOCK * _log(rng, 1, 512)
        rows = max(1, min(_log(rng, 1, 200000), (1 << 29) // K))
        return dict(op=op, rows=rows, K=K, dtype=rng.choice(["bf16", "bf16", "f32"]))
    T = _log(rng, 1, 8192)
    H = BLOCK * _log(rng, 8, 128)
    I = 64 * _log(rng, 8, 96)
    E = rng.choice([4, 8, 16, 32, 60, 64, 128])
    k = rng.randint(2, min(E, 8))
    while T * k * H * I > 8192 * 2 * 4096 * 7168:
        T = (T + 1) // 2
    while E * H * I > 8 * 4096 * 14336:
        E //= 2
    return dict(op=op, T=T, H=H, I=I, E=E, k=min(k, E), skew=rng.choice([0.0, 0.0, 1.0, 1.5]))


def work(case):
    op = case["op"]
    if op == "router":
        T, E, k = case["T"], case["E"], case["k"]
        size = 4 if case["dtype"] == "f32" else 2
        # logits in, their gradient out; ids and probabilities out, the probabilities' gradient in; counts
        return {"bytes": 2 * T * E * size + T * k * 12 + 4 * E, "flops": 12.0 * T * E}
    if op == "quant":
        n = case["rows"] * case["K"]
        return {"bytes": 2 * n * (4 if case["dtype"] == "f32" else 2), "flops": 4.0 * n}
    T, H, I, E, k = (case[f] for f in ("T", "H", "I", "E", "k"))
    # the weights of the experts that T tokens reach when all are equally likely
    reached = E * (1.0 - (1.0 - k / E) ** T)
    return {"bytes": reached * 3 * H * I * (0.5 + 1 / BLOCK) + 4 * T * H + 8 * T * k, "flops": 6.0 * T * k * H * I}


# ----------------------------------------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _plain_quant(x):
    """x [..., K] -> (magnitude-and-sign values on the E2M1 grid, exponents s of the scales 2^s): the smallest power of
    two that keeps a block's largest magnitude within 6; a block without a finite magnitude has the exponent NaN."""
    b = x.float().unflatten(-1, (-1, BLOCK))
    amax = b.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(amax)
    s = (e - 2 - (m <= 0.75).int()).clamp(-127, 127)
    s = torch.where(amax == 0, torch.full_like(s, -127), s).float()
    s = torch.where(amax.isfinite(), s, torch.full_like(s, float("nan")))
    a = (b.abs() * torch.exp2(-s)).clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign(torch.round(a / step) * step, b), s


def _pack(v, s):
    """Grid values and exponents -> bytes of two codes (the even element in the low half) and scale bytes s + 127."""
    a = v.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = code | (torch.signbit(v).to(torch.uint8) << 3)
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), (s.squeeze(-1) + 127).to(torch.uint8)


def _weights(E, rows, K, g):
    """[E, rows, K] ~ N(0, 1/K), as a checkpoint in 4 bits holds them: packed codes and scale bytes in row order."""
    codes = torch.empty(E, rows, K // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(E, rows, K // BLOCK, dtype=torch.uint8, device=DEV)
    for e in range(E):
        w = torch.randn(rows, K, generator=g, device=DEV) / math.sqrt(K)
        codes[e], scales[e] = _pack(*_plain_quant(w))
    return codes, scales


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "router":
        T, E, k = case["T"], case["E"], case["k"]
        logits = torch.randn(T, E, generator=g, device=DEV) * 2 + torch.randn(E, generator=g, device=DEV)
        state = dict(case=case,
                     # the gradients that a mean loss over the tokens and its usual coefficients send back
                     dprob=torch.randn(T, k, generator=g, device=DEV) * (0.05 / T),
                     dlosses=torch.tensor([1e-2, 1e-3], device=DEV),
                     mask=torch.rand(T, generator=g, device=DEV) < 0.8 if case["masked"] else None)
        if case["masked"]:  # what stands in padded rows is anything
            logits[~state["mask"]] = float("nan") if seed % 2 else 0.0
        state["logits"] = logits.to(torch.bfloat16) if case["dtype"] == "bf16" else logits
        if own:
            from mxfp8_grouped_gemm_x32_b200.layer import GroupedMLP
            state["layer"] = GroupedMLP(T, 32, 64, E, k, device=DEV, backward=False, mxfp8=False)
        return state
    if op == "quant":
        rows, K = case["rows"], case["K"]
        # rows of different magnitudes, one in sixteen blocks without a value
        x = torch.randn(rows, K, generator=g, device=DEV, dtype=torch.bfloat16)
        x *= torch.exp2(torch.randint(-8, 9, (rows, 1), generator=g, device=DEV).float()).to(torch.bfloat16)
        zero = torch.rand(rows, K // BLOCK, 1, generator=g, device=DEV) < 1 / 16
        x.view(rows, -1, BLOCK).masked_fill_(zero, 0.0)
        if case["dtype"] == "f32":
            x = x.float() * (1 + 1e-3 * torch.rand(rows, 1, generator=g, device=DEV))
        return dict(case=case, x=x)
    T, H, I, E, k = (case[f] for f in ("T", "H", "I", "E", "k"))
    logits = torch.randn(T, E, generator=g, device=DEV)
    logits += case["skew"] * torch.randn(E, generator=g, device=DEV)
    top = torch.sort(logits, dim=-1, descending=True, stable=True)
    idx = top.indices[:, :k].to(torch.int32).contiguous()
    prob = torch.softmax(top.values[:, :k], -1).contiguous()
    w1, s1 = _weights(E, 2 * I, H, g)  # gate rows first
    w2, s2 = _weights(E, H, I, g)
    x = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
    state = dict(case=case, x=x, idx=idx, prob=prob, w1=w1, s1=s1, w2=w2, s2=s2)
    # the plan of the plain loop over experts: how many rows each has
    state["sizes"] = torch.bincount(idx.flatten().long(), minlength=E).tolist()
    if own:
        from mxfp8_grouped_gemm_x32_b200.layer import GroupedMLP
        layer = state["layer"] = GroupedMLP(T, H, I, E, k, device=DEV, backward=False, mxfp8=False)
        layer.load_weights_mxfp4(w1, s1, w2, s2)
    return state


# ----------------------------------------------------------------------------------------------------------------------
# the operators
# ----------------------------------------------------------------------------------------------------------------------
def _unpack(codes, scales):
    """Packed codes [rows, K/2] and scale bytes [rows, K/32] -> fp32 values [rows, K]."""
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=codes.device)
    nib = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    v = grid[nib.int()].unflatten(-1, (-1, BLOCK))
    return (v * torch.exp2(scales.float() - 127).unsqueeze(-1)).flatten(-2)


def _round_trip(x):
    v, s = _plain_quant(x)
    return (v * torch.exp2(s)).flatten(-2)


def _router(st):
    case, k, E = st["case"], st["case"]["k"], st["case"]["E"]
    raw = st["logits"].float()
    mask = st["mask"]
    # NaN ranks last; equal logits go to the lower expert
    key = torch.where(raw.isnan(), torch.full_like(raw, -math.inf), raw)
    top = torch.sort(key, dim=-1, descending=True, stable=True)
    idx = top.indices[:, :k]
    kept = top.values[:, :k]
    ex = torch.exp(kept - kept[:, :1])
    valid = torch.ones(raw.shape[0], dtype=torch.bool, device=raw.device) if mask is None else mask
    prob = torch.where(valid.unsqueeze(-1), ex / ex.sum(-1, keepdim=True), 0.0)
    n = valid.sum().float().clamp(min=1)
    counts = torch.zeros(E, dtype=torch.int32, device=raw.device)
    counts.index_add_(0, idx.flatten(), valid.unsqueeze(-1).expand_as(idx).flatten().int())
    # softmax and its logarithm's normaliser over all experts; masked rows (padding) leave nothing
    top1 = raw.amax(-1, keepdim=True)
    e = torch.exp(raw - top1)
    total = e.sum(-1, keepdim=True)
    lse = torch.where(valid, (top1 + torch.log(total)).squeeze(-1), 0.0)
    s = torch.where(valid.unsqueeze(-1), e / total, 0.0)
    f = counts.float() / (n * k)
    losses = torch.stack((E * (f * (s.sum(0) / n)).sum(), (lse * lse).sum() / n))
    # backward
    gb, gz = st["dlosses"][0], st["dlosses"][1]
    d = s * (gb * E / n * (f - (s * f).sum(-1, keepdim=True)) + (gz * 2 / n) * lse.unsqueeze(-1))
    dp = st["dprob"]
    d.scatter_add_(1, idx, prob * (dp - (prob * dp).sum(-1, keepdim=True)))
    return {"idx": idx.int(), "prob": prob, "counts": counts, "losses": losses, "dlogits": d.to(st["logits"].dtype)}


def _mlp(st):
    case, x, E, k = st["case"], st["x"], st["case"]["E"], st["case"]["k"]
    H, I = case["H"], case["I"]
    order = torch.sort(st["idx"].flatten(), stable=True).indices
    xq = _round_trip(x)
    p = st["prob"].flatten()
    y = torch.empty(order.numel(), H, device=x.device)
    at = 0
    for e in range(E):
        n = st["sizes"][e]
        if n == 0:
            continue
        slots = order[at:at + n]
        at += n
        a = xq[slots // k] @ _unpack(st["w1"][e], st["s1"][e]).T
        gate, up = a[:, :I], a[:, I:]
        h = p[slots, None] * (gate / (1 + torch.exp(-gate))) * up
        y[slots] = _round_trip(h) @ _unpack(st["w2"][e], st["s2"][e]).T
    return {"out": y.view(-1, k, H).sum(1).to(torch.bfloat16)}


def run(state):
    case = state["case"]
    if own:
        if case["op"] == "router":
            layer = state["layer"]
            idx, prob, losses = layer.route_losses(state["logits"], state["mask"])
            dlogits = layer.route_backward(state["logits"], state["dprob"], state["dlosses"], state["mask"])
            return {"idx": idx, "prob": prob, "counts": layer.expert_counts, "losses": losses, "dlogits": dlogits}
        if case["op"] == "quant":
            from mxfp8_grouped_gemm_x32_b200 import mxfp4
            codes, scales = mxfp4.quantize(state["x"])
            return {"values": mxfp4.dequantize(codes, scales, state["x"].dtype)}
        layer = state["layer"]
        layer.permute_index(state["idx"], state["prob"])
        return {"out": layer.forward_mxfp4(state["x"])}
    if case["op"] == "router":
        return _router(state)
    if case["op"] == "quant":
        return {"values": _round_trip(state["x"]).to(state["x"].dtype)}
    return _mlp(state)


# ----------------------------------------------------------------------------------------------------------------------
# 64 bits
# ----------------------------------------------------------------------------------------------------------------------
def _exact_quant(x, step=1 << 26):
    """The values that the nearest codes and the scales stand for: the scale by comparison with 6 * 2^s, the code as
    the nearest grid value, the one with the even index where two are equally near."""
    rows = max(1, step // x.shape[-1])
    parts = []
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    middle = (grid[1:] + grid[:-1]) / 2
    for at in range(0, x.shape[0], rows):
        b = x[at:at + rows].double().unflatten(-1, (-1, BLOCK))
        top = b.abs().amax(-1, keepdim=True)
        s = torch.floor(torch.log2(torch.where((top > 0) & top.isfinite(), top, torch.ones_like(top)) / 6))
        s = s - 2
        for _ in range(5):  # the smallest s with top <= 6 * 2^s
            s = torch.where(top > 6 * torch.exp2(s), s + 1, s)
        s = torch.where(top > 0, s, torch.full_like(s, -127)).clamp(-127, 127)
        a = b.abs() / torch.exp2(s)
        below = torch.bucketize(a, middle)          # borders strictly below a
        upto = torch.bucketize(a, middle, right=True)  # borders below or at a
        code = torch.where(below % 2 == 0, below, upto)  # at a border: the even one of the two
        v = torch.copysign(grid[code], b) * torch.exp2(s)
        v = torch.where(top.isfinite(), v, torch.full_like(v, float("nan")))
        parts.append(v.flatten(-2))
    return torch.cat(parts)


def _exact_router(st):
    case = st["case"]
    T, E, k = case["T"], case["E"], case["k"]
    z = st["logits"].double()
    keep = torch.ones(T, dtype=torch.bool, device=z.device) if st["mask"] is None else st["mask"]
    ranked = torch.nan_to_num(z, nan=-math.inf, posinf=math.inf, neginf=-math.inf)
    val, pos = torch.sort(ranked, dim=1, descending=True, stable=True)
    val, pos = val[:, :k], pos[:, :k]
    prob = torch.where(keep[:, None], torch.softmax(val, 1), 0.0)
    n = int(keep.sum())
    hot = torch.zeros(T, E, dtype=torch.float64, device=z.device).scatter_(1, pos, 1.0)
    counts = hot[keep].sum(0)
    soft = torch.softmax(z[keep], 1)
    norm = torch.logsumexp(z[keep], 1)
    share = counts / max(1, n * k)
    balance = E * (share * soft.sum(0)).sum() / max(1, n)
    zloss = (norm ** 2).sum() / max(1, n)
    gb, gz = (float(v) for v in st["dlosses"].double())
    grad = torch.zeros(T, E, dtype=torch.float64, device=z.device)
    if n:
        grad[keep] = gb * E / n * (soft * share - soft * (soft @ share)[:, None]) + gz * 2 / n * norm[:, None] * soft
    dp = st["dprob"].double()
    inner = prob * dp - prob * (prob * dp).sum(1, keepdim=True)
    grad += torch.zeros_like(grad).scatter_add_(1, pos, inner)
    return {"idx": None, "prob": prob, "counts": None, "losses": torch.stack((balance, zloss)), "dlogits": grad}


def _exact_weights(codes, scales):
    grid = torch.tensor(GRID, dtype=torch.float64, device=codes.device)
    out = torch.empty(codes.shape[0], codes.shape[1] * 2, dtype=torch.float64, device=codes.device)
    for half in (0, 1):
        c = (codes >> (4 * half)).long() & 15
        out[:, half::2] = torch.where(c >= 8, -grid[c % 8], grid[c % 8])
    return out * torch.exp2(scales.double() - 127).repeat_interleave(BLOCK, 1)


def _exact_mlp(st):
    T, H, I, E, k = (st["case"][f] for f in ("T", "H", "I", "E", "k"))
    xq = _exact_quant(st["x"])
    out = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    for e in range(E):
        t, j = torch.nonzero(st["idx"] == e, as_tuple=True)
        if not len(t):
            continue
        a = xq[t] @ _exact_weights(st["w1"][e], st["s1"][e]).T
        h = st["prob"][t, j].double()[:, None] * torch.nn.functional.silu(a[:, :I]) * a[:, I:]
        out.index_add_(0, t, _exact_quant(h) @ _exact_weights(st["w2"][e], st["s2"][e]).T)
    return {"out": out}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "router":
        return _exact_router(st)
    if case["op"] == "quant":
        return {"values": _exact_quant(st["x"])}
    return _exact_mlp(st)
