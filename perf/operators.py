"""Operators of a routed expert layer, as a user's program calls them: choosing
experts for tokens (with its gradient), casting tensors to 4-bit block-scaled
floats, and the grouped product over 4-bit experts.

``run`` computes each in its plain form (elementary torch operations, fp32)
where ``own`` is false, and calls this repository's operators where it is true.

The 4-bit formats.  Codes are e2m1 (0, .5, 1, 1.5, 2, 3, 4, 6 and their
negatives), two to a byte, the even element in the low half.
  "mxfp4"  one e8m0 scale byte for 32 elements of a row: the power of two
           s = 2^floor(log2(6 / amax)) multiplies the elements before the cast
           and the byte holds 1 / s, biased by 127
  "nvfp4"  one e4m3 scale for 16 elements, and one power of two R for the row:
           R = 2^floor(log2(2688 / row amax)), b = e4m3(R amax16 / 6), the codes
           are e2m1(R x / b) and stand for code * b / R
Scales lie in tiles of 128 rows by one 4-byte word of a row (4 scales: 128
elements of mxfp4, 64 of nvfp4): [row tile][word][row % 32][row / 32 % 4][4].
"""

import math

import torch

own = False

BLOCK = {"mxfp4": 32, "nvfp4": 16}
MASKED = -3.3e38  # a logit at or below it masks its expert (-inf, and the lowest value of either type)


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # one token at decode: the smallest routing call, a wide sigmoid router with a balance bias and expert groups
        dict(name="route_token", op="route", T=1, E=256, k=8, scoring="sigmoid", bias=True, groups=8, keep=4, group_top=2,
             renorm=True, scale=2.5, dtype="float32", masked=0, train=False),
        # a prompt's routing: bf16 logits, softmax over 128 experts, a few of them switched off
        dict(name="route_prompt", op="route", T=4001, E=128, k=8, scoring="softmax", bias=False, groups=1, keep=1,
             group_top=1, renorm=True, scale=1.0, dtype="bfloat16", masked=3, train=False),
        # a training step's routing of the 64-expert, top-6 layer, with the gradient of the logits
        dict(name="route_step_softmax", op="route", T=16384, E=64, k=6, scoring="softmax", bias=False, groups=1, keep=1,
             group_top=1, renorm=False, scale=1.0, dtype="float32", masked=0, train=True),
        # the largest routing: a long training batch over many experts, groups and bias, with the gradient
        dict(name="route_step_groups", op="route", T=65536, E=256, k=8, scoring="sigmoid", bias=True, groups=8, keep=4,
             group_top=2, renorm=True, scale=2.5, dtype="float32", masked=0, train=True),
        # a decode batch's activations to 4 bits and back (what quantisation-aware evaluation calls)
        dict(name="quant_tokens", op="quant", fmt="nvfp4", E=1, N=16, K=5120),
        # an odd set of rows whose length ends inside a scale word
        dict(name="quant_ragged", op="quant", fmt="mxfp4", E=3, N=1001, K=1440),
        # the weights of an 8-expert layer, cast once at load and read back
        dict(name="quant_weights", op="quant", fmt="nvfp4", E=8, N=6400, K=4096),
        # one token against one of 128 experts: latency
        dict(name="gmm_token", op="gmm", fmt="nvfp4", M=1, E=128, active=1, K=5120, N=8192, skew=0.0),
        # a decode batch, every row at an expert of its own: the weights' stream
        dict(name="gmm_decode", op="gmm", fmt="mxfp4", M=16, E=128, active=16, K=5120, N=8192, skew=0.0),
        # a small ragged batch with empty experts and sizes that end inside every tile
        dict(name="gmm_ragged", op="gmm", fmt="mxfp4", M=777, E=12, active=9, K=1440, N=1000, skew=0.7),
        # the 8-expert layer at 1024 rows: the weights' stream against the product
        dict(name="gmm_layer", op="gmm", fmt="nvfp4", M=1024, E=8, active=8, K=4096, N=6400, skew=0.0),
        # the 64-expert layer over 16384 tokens, six experts each: the largest product
        dict(name="gmm_prompt", op="gmm", fmt="nvfp4", M=98304, E=64, active=60, K=2048, N=1408, skew=0.4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _odd(v):
    return v | 1


def draw(rng):
    op = rng.choice(["route", "route", "quant", "gmm", "gmm", "gmm"])
    if op == "route":
        train = rng.random() < 0.5
        scoring = rng.choice(["softmax", "sigmoid"])
        groups = rng.choice([1, 1, 4, 8])
        E = groups * rng.randint(3, 40) if groups > 1 else _odd(_log(rng, 8, 400))
        keep = rng.randint(1, groups)
        k = min(rng.randint(1, 10), keep * (E // groups))
        T = _odd(_log(rng, 1, min(65536, 16777216 // E)))
        return dict(op=op, T=T, E=E, k=k, scoring=scoring, bias=scoring == "sigmoid" and rng.random() < 0.7,
                    groups=groups, keep=keep, group_top=rng.choice([1, 2]) if groups > 1 else 1,
                    renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["float32", "bfloat16"]),
                    masked=rng.choice([0, 0, 1, 5]), train=train)
    fmt = rng.choice(["mxfp4", "nvfp4"])
    K = 32 * _odd(_log(rng, 2, 200)) if rng.random() < 0.5 else 512 * _odd(rng.randint(0, 8))
    if op == "quant":
        E = rng.choice([1, 1, 3, 8])
        return dict(op=op, fmt=fmt, E=E, N=_odd(_log(rng, 1, max(2, 200000000 // (E * K)))), K=K)
    E = _odd(_log(rng, 1, 64))
    N = 8 * _odd(_log(rng, 4, 800)) if rng.random() < 0.5 else 128 * _odd(rng.randint(0, 40))
    while E * N * K > 400000000:
        E = _odd(max(1, E // 2)) if E > 1 else 1
        N = max(8, N // 16 * 8) if E == 1 else N
    M = _odd(_log(rng, 1, min(60000, max(64, 250000000000 // (N * K)))))
    return dict(op=op, fmt=fmt, M=M, E=E, active=rng.randint(1, min(M, E)), K=K, N=N, skew=rng.choice([0.0, 0.5]))


def work(case):
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        size = 2 if case["dtype"] == "bfloat16" else 4
        nbytes = T * E * size + T * k * 8 + (4 * E if case["bias"] else 0)
        flops = 4 * T * E
        if case["train"]:  # and the weights' gradients in, the logits' gradients out
            nbytes += T * k * 4 + T * E * size
            flops += 2 * T * E
        return {"bytes": nbytes, "flops": flops}
    if case["op"] == "quant":
        n = case["E"] * case["N"] * case["K"]
        return {"bytes": 4 * n, "flops": 4 * n}
    M, N, K = case["M"], case["N"], case["K"]
    per = 0.5 + 1.0 / BLOCK[case["fmt"]]
    weights = case["active"] * N * (K * per + (4 if case["fmt"] == "nvfp4" else 0))
    return {"bytes": weights + 2 * M * K + 2 * M * N + 8 * case["E"], "flops": 2 * M * N * K}


# ------------------------------------------------------------------ the inputs
def _generator(seed, salt):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + salt)


def _logits(case, seed):
    g = _generator(seed, 1)
    T, E = case["T"], case["E"]
    popular = 0.5 * torch.randn(E, generator=g, device="cuda")
    logits = 1.5 * torch.randn(T, E, generator=g, device="cuda") + popular
    bias = 0.1 * torch.randn(E, generator=g, device="cuda") if case["bias"] else None
    grad = torch.randn(T, case["k"], generator=g, device="cuda") if case["train"] else None
    off = torch.randperm(E, generator=g, device="cuda")[: min(case["masked"], E - 1)]
    logits[:, off] = -math.inf
    return logits.to(getattr(torch, case["dtype"])), bias, grad


def _rows(shape, g, scale):
    """Rows with a few strong channels, as activations and weights have them."""
    channel = torch.exp(0.5 * torch.randn(shape[-1], generator=g, device="cuda"))
    v = torch.randn(shape, generator=g, device="cuda")
    return v.mul_(channel).mul_(scale).to(torch.bfloat16)


def _group_sizes(case, seed):
    """`active` of the E experts own rows, at least one each, the others by a popularity i^-skew."""
    g = torch.Generator().manual_seed(int(seed) * 1000003 + 2)
    M, E, A = case["M"], case["E"], case["active"]
    pop = torch.arange(1, A + 1, dtype=torch.float64) ** -case["skew"]
    picks = torch.multinomial(pop, M - A, replacement=True, generator=g) if M > A else torch.zeros(0, dtype=torch.int64)
    sizes = torch.zeros(E, dtype=torch.int64)
    sizes[torch.randperm(E, generator=g)[:A]] = 1 + torch.bincount(picks, minlength=A)
    return sizes


def _weights(case, seed, e):
    return _rows((case["N"], case["K"]), _generator(seed, 100 + e), 0.02)


def _tokens(case, seed):
    return _rows((case["M"], case["K"]), _generator(seed, 4), 1.0)


def prepare(case, seed):
    if case["op"] == "route":
        logits, bias, grad = _logits(case, seed)
        return dict(case=case, logits=logits, bias=bias, grad=grad)
    if case["op"] == "quant":
        return dict(case=case, x=_rows((case["E"], case["N"], case["K"]), _generator(seed, 5), 0.1))
    sizes = _group_sizes(case, seed)
    codes, scales, row_scale = [], [], []
    for e in range(case["E"]):  # an expert at a time: the fp32 steps of all of them would fill the card
        q, byte, r = _cast(_weights(case, seed, e)[None], case["fmt"])
        codes.append(_pack(q))
        scales.append(_tiles(byte))
        row_scale.append(r)
    return dict(case=case, x=_tokens(case, seed), sizes=sizes.cuda(), most=int(sizes.max()), codes=torch.cat(codes),
                scales=torch.cat(scales), row_scale=torch.cat(row_scale) if case["fmt"] == "nvfp4" else None)


# ------------------------------------------------------------- the plain forms
def _floor_pow2(v):
    return (v.view(torch.int32) & 0x7F800000).view(torch.float32)


def _to_e2m1(a):
    """Magnitudes to the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6, ties to the even code."""
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.clamp(torch.round(a / step) * step, max=6.0)


def _cast(x, fmt):
    """Codes as values (fp32), the blocks' scale bytes, and the rows' powers of two (nvfp4)."""
    x = x.float()
    b = BLOCK[fmt]
    row_scale = None
    if fmt == "nvfp4":
        row_scale = _floor_pow2(2688.0 / torch.clamp(x.abs().amax(-1), min=1e-12))
        x = x * row_scale[..., None]
    blocks = x.view(*x.shape[:-1], x.shape[-1] // b, b)
    amax = blocks.abs().amax(-1)
    if fmt == "nvfp4":
        scale = (amax / 6.0).to(torch.float8_e4m3fn)
        byte, s = scale.view(torch.uint8), scale.float()
        y = torch.where(s[..., None] > 0, blocks / torch.where(s > 0, s, 1.0)[..., None], 0.0)
    else:
        s = _floor_pow2(6.0 / torch.clamp(amax, min=1e-12))
        byte = (254 - (s.view(torch.int32) >> 23)).to(torch.uint8)
        y = blocks * s[..., None]
    q = torch.copysign(_to_e2m1(y.abs()), y)
    return q.view(x.shape), byte, row_scale


def _scale_values(byte, fmt):
    if fmt == "nvfp4":
        return byte.view(torch.float8_e4m3fn).float()
    return torch.exp2(byte.float() - 127.0)


def _pack(q):
    a = q.abs()
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = code | (torch.signbit(q).to(torch.uint8) << 3)
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _tiles(byte):
    """Scale bytes [E, N, blocks] in the tiled layout, zeros past the rows and blocks."""
    E, N, nb = byte.shape
    tiles, words = -(-N // 128), -(-nb // 4)
    full = torch.zeros(E, tiles * 128, words * 4, dtype=torch.uint8, device=byte.device)
    full[:, :N, :nb] = byte
    return full.view(E, tiles, 4, 32, words, 4).permute(0, 1, 4, 3, 2, 5).contiguous().view(-1)


def _untile(scales, E, N, nb):
    tiles, words = -(-N // 128), -(-nb // 4)
    return scales.view(E, tiles, words, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(E, tiles * 128, words * 4)[:, :N, :nb]


def _decode(codes, byte, row_scale, fmt):
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    q = table[torch.stack([codes & 15, codes >> 4], -1).int()].view(*codes.shape[:-1], -1)
    b = BLOCK[fmt]
    v = (q.view(*byte.shape, b) * _scale_values(byte, fmt)[..., None]).view(q.shape)
    return v if row_scale is None else v / row_scale[..., None]


def _gmm(state):
    case, fmt = state["case"], state["case"]["fmt"]
    M, E, K, N = case["M"], case["E"], case["K"], case["N"]
    q, byte, row_scale = _cast(state["x"], fmt)
    x = (q.view(*byte.shape, BLOCK[fmt]) * _scale_values(byte, fmt)[..., None]).view(M, K)
    x = x if row_scale is None else x / row_scale[:, None]
    ends = torch.cumsum(state["sizes"], 0)
    row = torch.arange(M, device=x.device)
    expert = torch.searchsorted(ends, row, right=True)
    byte_w, row_w = _untile(state["scales"], E, N, K // BLOCK[fmt]), state["row_scale"]
    if M <= E:  # few rows: the weights of each row's expert
        w = _decode(state["codes"][expert], byte_w[expert], None if row_w is None else row_w[expert], fmt)
        return torch.bmm(x[:, None], w.transpose(1, 2))[:, 0].to(torch.bfloat16)
    place = row - (ends - state["sizes"])[expert]
    padded = torch.zeros(E, state["most"], K, device=x.device)
    padded[expert, place] = x
    w = _decode(state["codes"], byte_w, row_w, fmt)
    return torch.bmm(padded, w.transpose(1, 2))[expert, place].to(torch.bfloat16)


def _route(state):
    case, bias = state["case"], state["bias"]
    T, E, k, G, scale = case["T"], case["E"], case["k"], case["groups"], case["scale"]
    lowest = torch.finfo(torch.float32).min
    logits = state["logits"].float()
    masked = logits <= MASKED
    if case["scoring"] == "sigmoid":
        s = torch.where(masked, 0.0, 1.0 / (1.0 + torch.exp(-logits)))
        key = gkey = s if bias is None else s + bias
    else:
        top = logits.amax(-1, keepdim=True)
        e = torch.where(masked, 0.0, torch.exp(logits - torch.where(top <= MASKED, 0.0, top)))
        total = e.sum(-1, keepdim=True)
        s = torch.where(total == 0, 0.0, e / total)
        key = logits if bias is None else s + bias
        gkey = key if bias is not None or case["group_top"] == 1 else e
    key, gkey = torch.where(masked, lowest, key), torch.where(masked, lowest, gkey)
    if G > 1:
        best = torch.sort(gkey.view(T, G, E // G), dim=-1, descending=True).values[..., : case["group_top"]]
        gscore = torch.where(best[..., 0] == lowest, lowest, torch.where(best == lowest, 0.0, best).sum(-1))
        kept = torch.sort(gscore, dim=-1, descending=True, stable=True).indices[:, : case["keep"]]
        keeps = torch.zeros(T, G, dtype=torch.bool, device=key.device).scatter(1, kept, True)
        key = torch.where(keeps[:, :, None].expand(T, G, E // G).reshape(T, E), key, -math.inf)
    ids = torch.sort(key, dim=-1, descending=True, stable=True).indices[:, :k]
    r = s.gather(1, ids)
    if case["renorm"]:
        total = r.sum(-1, keepdim=True)
        r = torch.where(total == 0, 0.0, r / total)
    w = r * scale
    out = {"weights": w, "ids": ids.to(torch.int32)}
    if not case["train"]:
        return out
    g = state["grad"]
    if case["renorm"]:
        d = w * (g - (g * (w / scale)).sum(-1, keepdim=True))
    else:
        d = w * g
    grad = torch.zeros(T, E, device=key.device)
    if case["scoring"] == "sigmoid":
        picked = logits.gather(1, ids)
        grad.scatter_(1, ids, d / (1.0 + torch.exp(torch.where(picked <= MASKED, 0.0, picked))))
    else:
        grad.scatter_(1, ids, d)
        if not case["renorm"]:
            grad = grad - s * d.sum(-1, keepdim=True)
    return {**out, "grad_logits": grad.to(state["logits"].dtype)}


# ------------------------------------------------------------------------- run
def run(state):
    case = state["case"]
    if not own:
        if case["op"] == "route":
            return _route(state)
        if case["op"] == "gmm":
            return _gmm(state)
        q, byte, row_scale = _cast(state["x"], case["fmt"])
        v = (q.view(*byte.shape, BLOCK[case["fmt"]]) * _scale_values(byte, case["fmt"])[..., None]).view(q.shape)
        return (v if row_scale is None else v / row_scale[..., None]).to(torch.bfloat16)

    import mixture_experts_grouped_gmm_gb300 as mg

    if case["op"] == "route":
        how = dict(scoring=case["scoring"], bias=state["bias"], n_group=case["groups"], topk_group=case["keep"],
                   group_top=case["group_top"], renormalize=case["renorm"], scale=case["scale"])
        w, ids = mg.moe.route_experts(state["logits"], case["k"], **how)
        out = {"weights": w, "ids": ids}
        if case["train"]:
            out["grad_logits"] = mg.moe.route_experts_backward(
                state["grad"], state["logits"], w, ids, scoring=case["scoring"], renormalize=case["renorm"],
                scale=case["scale"])
        return out
    if case["op"] == "quant":
        return mg.dequantize_fp4(mg.quantize_fp4(state["x"], case["fmt"]))
    w = mg.Fp4Tensor(state["codes"], state["scales"], state["row_scale"], case["fmt"])
    return mg.gmm_fp4(state["x"], w, state["sizes"])


# ---------------------------------------------------------- 64-bit definitions
def _exponent(v):
    """floor(log2 v) of positive v."""
    return torch.frexp(v).exponent.double() - 1.0


def _exact_cast(x, fmt):
    """Values that the cast rows stand for, from the definition: the codes by the midpoints between levels."""
    x = x.double()
    unit = torch.ones_like(x[..., :1])
    if fmt == "nvfp4":
        unit = torch.exp2(_exponent(2688.0 / torch.clamp(x.abs().amax(-1, keepdim=True), min=1e-12)))
    b = BLOCK[fmt]
    rows = (x * unit).unflatten(-1, (-1, b))
    most = rows.abs().amax(-1, keepdim=True)
    if fmt == "nvfp4":  # e4m3: 3 bits after the leading one, exponents from -6
        v = most / 6.0
        ulp = torch.exp2(torch.clamp(_exponent(torch.clamp(v, min=2.0 ** -40)), min=-6.0) - 3.0)
        s = torch.clamp(torch.round(v / ulp) * ulp, max=448.0)
    else:
        s = torch.exp2(-_exponent(6.0 / torch.clamp(most, min=1e-12)))
    mag = torch.where(s > 0, rows.abs() / torch.where(s > 0, s, 1.0), 0.0)
    v = 0.5 * (mag > 0.25) + 0.5 * (mag >= 0.75) + 0.5 * (mag > 1.25) + 0.5 * (mag >= 1.75)
    v = v + 1.0 * (mag > 2.5) + 1.0 * (mag >= 3.5) + 2.0 * (mag > 5.0)
    return (torch.sign(rows) * v * s).flatten(-2) / unit


def _exact_route(case, seed):
    logits, bias, grad = _logits(case, seed)
    l = logits.double()
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    dead = torch.isinf(l)
    if case["scoring"] == "sigmoid":
        s = torch.sigmoid(l)
    else:
        s = torch.softmax(l, -1)
    c = s + bias.double() if bias is not None else s
    c = c.masked_fill(dead, -1e9)
    if G > 1:
        best = torch.topk(c.view(T, G, E // G), case["group_top"], -1).values
        score = torch.where(best[..., 0] == -1e9, -1e9, best.masked_fill(best == -1e9, 0.0).sum(-1))
        order = torch.argsort(score, dim=-1, descending=True, stable=True)
        lost = torch.ones(T, G, dtype=torch.bool, device=l.device)
        lost.scatter_(1, order[:, : case["keep"]], False)
        c = c.masked_fill(lost.repeat_interleave(E // G, 1), -2e9)
    ids = torch.argsort(c, dim=-1, descending=True, stable=True)[:, :k]
    chosen = torch.zeros(T, E, dtype=torch.float64, device=l.device).scatter_(1, ids, 1.0)
    p = s * chosen
    total = p.sum(-1, keepdim=True) if case["renorm"] else torch.ones_like(p[:, :1])
    total = torch.where(total == 0, 1.0, total)
    w = case["scale"] * p / total
    out = {"weights": w.gather(1, ids), "ids": None}
    if case["train"]:
        up = torch.zeros(T, E, dtype=torch.float64, device=l.device).scatter_(1, ids, grad.double())
        ds = case["scale"] * up * chosen / total  # through the picked scores
        if case["renorm"]:
            ds = ds - chosen * (case["scale"] * up * p).sum(-1, keepdim=True) / total ** 2
        if case["scoring"] == "sigmoid":
            out["grad_logits"] = ds * s * (1 - s)
        else:
            out["grad_logits"] = s * (ds - (ds * s).sum(-1, keepdim=True))
    return out


def exact(case, seed):
    if case["op"] == "route":
        return _exact_route(case, seed)
    if case["op"] == "quant":
        return _exact_cast(_rows((case["E"], case["N"], case["K"]), _generator(seed, 5), 0.1), case["fmt"])
    x = _exact_cast(_tokens(case, seed), case["fmt"])
    out, first = torch.empty(case["M"], case["N"], dtype=torch.float64, device="cuda"), 0
    for e, size in enumerate(_group_sizes(case, seed).tolist()):
        if size:
            out[first : first + size] = x[first : first + size] @ _exact_cast(_weights(case, seed, e), case["fmt"]).t()
        first += size
    return out
