"""A decode, verify or prefill step's 8-bit floating-point products and the steps beside them, as calls to measure.

Each case is one pass through one operator: the products of e4m3 activations
with e4m3 weights that have a scale for each block of 128 (``dense``,
``gather``, ``swiglu`` and ``combine``), writing such blocks (``norm``,
``quantize`` and ``weights``: the norm's output, a row's blocks and a matrix's
square ones, each read back as values), the norms of queries and keys with the
position rotation (``qk``), and the log probabilities of given tokens with
entropy and top alternatives (``logprobs``).  ``run`` makes the pass with this
package's calls where ``own`` is true, and with elementary torch operations
where it is not.

    listed()            the cases
    draw(rng)           one more case of the same ranges
    prepare(case, seed) a case's inputs on the GPU
    run(state)          one pass; its outputs
    work(case)          bytes and operations one pass cannot do without
    exact(case, seed)   the outputs from the definitions, in 64 bits
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2, "none": 0}
F8 = torch.float8_e4m3fn
BLOCK = 128
LARGEST = 448.0                     # e4m3's
LEAST_SCALE = 2.0 ** -126
EPS = 1e-5


def listed():
    return [
        # one token through a dense projection
        dict(name="dense 1 token", op="dense", M=1, E=1, top_k=1, N=2048, K=7168, holes=False),
        # one token's gate and up projections in 8 of 256 experts
        dict(name="swiglu 1 token", op="swiglu", M=1, E=256, top_k=8, N=2048, K=7168, holes=False),
        # four tokens' down projections with the router's weights, one expert input per slot
        dict(name="combine 4 tokens", op="combine", M=4, E=256, top_k=8, N=7168, K=2048, holes=False),
        # a prefill chunk through 32 experts whose rows end inside a block of 128
        dict(name="swiglu 512 tokens", op="swiglu", M=512, E=32, top_k=4, N=2880, K=2880, holes=False),
        # a chunk of a model with 256 experts; the padding's ids are outside the range
        dict(name="gather 1024 tokens", op="gather", M=1024, E=256, top_k=8, N=2048, K=7168, holes=True),
        # a dense projection of a whole prefill
        dict(name="dense 8192x7168x7168", op="dense", M=8192, E=1, top_k=1, N=7168, K=7168, holes=False),
        # a prefill chunk's residual, sum and norm, written as 8-bit blocks
        dict(name="norm 2048x7168", op="norm", M=2048, K=7168, x="f32", res="bf16"),
        # one projection of 32 experts, quantised when a model is loaded; square blocks cut at both edges
        dict(name="weights 32x2880x2880", op="weights", E=32, N=2880, K=2880, x="bf16"),
        # one token's 64 query and 8 key heads out of the projection's fp32 row
        dict(name="qk 1 token", op="qk", M=1, Hq=64, Hk=8, D=64, R=64, style="half", x="f32", y="bf16", rest=512,
             P=131072, holes=False),
        # a prefill's heads of 128, as a bf16 projection leaves them
        dict(name="qk 8192 tokens", op="qk", M=8192, Hq=32, Hk=8, D=128, R=128, style="half", x="bf16", y="bf16",
             rest=1024, P=32768, holes=True),
        # the sampled token of one sequence and its 20 alternatives
        dict(name="logprobs 1 token", op="logprobs", M=1, V=201088, top_k=20, x="f32", masked=0.0, holes=False),
        # scoring a prompt; the vocabulary's odd width leaves every row at another alignment
        dict(name="logprobs 1024 tokens", op="logprobs", M=1024, V=131071, top_k=5, x="bf16", masked=0.1, holes=True),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], its logarithm spread evenly."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(("dense", "gather", "swiglu", "combine", "dense", "norm", "quantize", "weights", "qk", "qk",
                     "logprobs", "logprobs"))
    if op in ("norm", "quantize"):
        K = 32 * _log(rng, 1, 512)
        return dict(op=op, M=_log(rng, 1, min(16384, (1 << 26) // K)), K=K, x=rng.choice(("f32", "bf16", "f16")),
                    res=rng.choice(("none", "bf16", "f32")) if op == "norm" else "none")
    if op == "weights":
        E, N, K = _log(rng, 1, 64), _log(rng, 17, 8192), 32 * _log(rng, 1, 256)
        while E * N * K > 1 << 28:
            E, N = max(1, E // 2), max(17, N // 2)
        return dict(op=op, E=E, N=N, K=K, x=rng.choice(("f32", "bf16", "f16")))
    if op == "qk":
        D = rng.choice((32, 64, 80, 96, 128, 128, 192, 256))
        Hk = rng.choice((1, 2, 4, 8))
        Hq = Hk * rng.choice((1, 3, 4, 8))
        M = _log(rng, 1, max(1, min(16384, (1 << 25) // ((Hq + Hk) * D))))
        return dict(op=op, M=M, Hq=Hq, Hk=Hk, D=D, R=rng.choice((D, D, D // 2)), style=rng.choice(("half", "pairs")),
                    x=rng.choice(("f32", "bf16", "f16")), y=rng.choice(("bf16", "bf16", "f16", "f32")),
                    rest=rng.choice((0, Hk * D, 24)), P=_log(rng, 64, 131072), holes=rng.random() < 0.3)
    if op == "logprobs":
        V = _log(rng, 101, 262143)
        return dict(op=op, M=_log(rng, 1, max(1, min(4096, (1 << 27) // V))), V=V, top_k=rng.randint(1, 20),
                    x=rng.choice(("f32", "bf16", "f16")), masked=rng.choice((0.0, 0.0, 0.3)), holes=rng.random() < 0.3)
    K, N = 32 * _log(rng, 4, 256), _log(rng, 33, 8192)
    if op == "dense":
        return dict(op=op, M=_log(rng, 1, 8192), E=1, top_k=1, N=N, K=K, holes=False)
    E = _log(rng, 2, 256)
    while E * N * K > 256 * 2048 * 7168:
        E = max(2, E // 2)
        N = max(33, N // 2)
    top_k = rng.randint(1, min(8, E))
    return dict(op=op, M=_log(rng, 1, (8192 if op != "swiglu" else 2048) // top_k), E=E, top_k=top_k, N=N, K=K,
                holes=rng.random() < 0.3)


# ------------------------------------------------------------------ inputs

def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    def codes(*shape):
        # a normal value's largest of a block lies near four deviations
        out = torch.empty(shape, dtype=F8, device="cuda")
        flat = out.view(torch.uint8).reshape(-1).view(F8)
        step = 1 << 27
        for i in range(0, flat.numel(), step):
            n = min(step, flat.numel() - i)
            flat[i:i + n] = (110.0 * normal(n)).clamp_(-LARGEST, LARGEST).to(F8)
        return out

    def weights(lead, N, K):
        return codes(*lead, N, K), 2e-4 * torch.exp(0.3 * normal(*lead, _blocks(N), _blocks(K)))

    c, s = case, dict(case=dict(case))
    op = c["op"]
    if op in ("norm", "quantize"):
        # hidden values grow along the depth and a few channels stand far out
        spread = torch.exp(0.5 * normal(c["K"]))
        s["x"] = (normal(c["M"], c["K"]) * spread).to(TYPES[c["x"]])
        s["res"] = None if c["res"] == "none" else (4.0 * normal(c["M"], c["K"]) * spread).to(TYPES[c["res"]])
        s["weight"] = (1.0 + 0.2 * normal(c["K"])).to(torch.bfloat16)
    elif op == "weights":
        s["x"] = (0.02 * normal(c["E"], c["N"], c["K"]) * torch.exp(0.3 * normal(c["E"], c["N"], 1))).to(TYPES[c["x"]])
    elif op == "qk":
        width = (c["Hq"] + c["Hk"]) * c["D"] + c["rest"]
        s["x"] = (2.0 * normal(c["M"], width) * torch.exp(0.3 * normal(c["M"], 1))).to(TYPES[c["x"]])
        s["qw"] = (1.0 + 0.2 * normal(c["D"])).to(torch.bfloat16)
        s["kw"] = (1.0 + 0.2 * normal(c["D"])).to(torch.bfloat16)
        # the angles of far positions in 64 bits, once per model
        i = torch.arange(c["R"] // 2, device="cuda", dtype=torch.float64)
        angle = torch.arange(c["P"], device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-2.0 * i / c["R"])
        s["table"] = torch.cat((torch.cos(angle), torch.sin(angle)), dim=1).to(torch.float32)
        s["pos"] = torch.randint(0, c["P"], (c["M"],), device="cuda", generator=g, dtype=torch.int32)
        if c["holes"]:
            t = torch.arange(c["M"], device="cuda")
            s["pos"] = torch.where(t >= c["M"] - c["M"] // 8, torch.full_like(s["pos"], -1), s["pos"])
    elif op == "logprobs":
        x = 2.5 * normal(c["M"], c["V"]) + 1.5 * normal(c["V"])
        # words that may not be sampled
        masked = torch.rand(c["V"], device="cuda", generator=g) < c["masked"]
        s["x"] = torch.where(masked, torch.full_like(x, -math.inf), x).to(TYPES[c["x"]])
        live = torch.nonzero(~masked)[:, 0].to(torch.int32)
        s["t"] = live[torch.randint(0, live.numel(), (c["M"],), device="cuda", generator=g)]
        if c["holes"]:
            t = torch.arange(c["M"], device="cuda")
            s["t"] = torch.where(t % 16 == 7, torch.full_like(s["t"], -1), s["t"])
    else:
        lead = () if op == "dense" else (c["E"],)
        s["codes"], s["scales"] = weights(lead, c["N"], c["K"])
        if op == "swiglu":
            s["up_codes"], s["up_scales"] = weights(lead, c["N"], c["K"])
        if op != "dense":
            # popular and unpopular experts; a token's experts are distinct
            score = normal(c["M"], c["E"]) + 0.7 * normal(c["E"])
            ids = torch.argsort(score, dim=1, descending=True)[:, :c["top_k"]].to(torch.int32).contiguous()
            if c["holes"]:
                # the chunk's last eighth is padding, and one slot in 16 is unused
                t = torch.arange(c["M"], device="cuda")[:, None]
                hole = (t >= c["M"] - c["M"] // 8) | (torch.rand(c["M"], c["top_k"], device="cuda", generator=g) < 1 / 16)
                ids = torch.where(hole, torch.full_like(ids, -1), ids)
            s["ids"] = ids
        lead = (c["M"], c["top_k"]) if op == "combine" else (c["M"],)
        s["x"], s["xs"] = codes(*lead, c["K"]), 8e-3 * torch.exp(0.3 * normal(*lead, _blocks(c["K"])))
        if op == "combine":
            s["rw"] = torch.softmax(normal(c["M"], c["top_k"]), dim=1)
    return s


def prepare(case, seed):
    return _inputs(case, seed)


# ---------------------------------------------------------- the plain forms

def _to_e4m3(q):
    """64-bit q, |q| <= 448, rounded to e4m3's nearest value, ties to even: steps of 1/8 of q's power of two, at
    least 2^-9."""
    e = torch.clamp(torch.frexp(q).exponent - 1, min=-6)
    step = torch.ldexp(torch.ones_like(q), e - 3)
    return torch.round(q / step) * step


def _padded(x, rows):
    """x (..., N, K) with zeros up to whole blocks (of rows too, where rows is true)."""
    n, k = x.shape[-2:]
    return torch.nn.functional.pad(x, (0, -k % BLOCK, 0, -n % BLOCK if rows else 0))


def _round_trip(x, square):
    """What quantising the 32-bit values x (..., N, K) and reading them back as bf16 gives."""
    n, k = x.shape[-2:]
    p = _padded(x, square)
    h = BLOCK if square else 1
    b = p.reshape(p.shape[:-2] + (p.shape[-2] // h, h, p.shape[-1] // BLOCK, BLOCK))
    d = (b.abs().amax(dim=(-3, -1), keepdim=True) / LARGEST).clamp(min=LEAST_SCALE)
    # codes change where a quotient crosses a border, so it is formed in 64 bits
    v = _to_e4m3((b.to(torch.float64) / d.to(torch.float64)).clamp(-LARGEST, LARGEST)).to(torch.float32) * d
    return v.reshape(p.shape)[..., :n, :k].to(torch.bfloat16)


def _plain_norm(s):
    h = s["x"].to(torch.float32)
    if s["res"] is not None:
        h = h + s["res"].to(torch.float32)
    d = h.to(torch.float64)
    r = 1.0 / torch.sqrt((d * d).mean(dim=1, keepdim=True) + EPS)
    out = [_round_trip((d * r * s["weight"].to(torch.float64)).to(torch.float32), False)]
    if s["res"] is not None:
        out.append(h.to(s["res"].dtype))
    return out


def _plain_weights(s):
    # a matrix at a time, so that the 64-bit quotients of a stack do not fill the card
    return [torch.stack([_round_trip(s["x"][e].to(torch.float32), True) for e in range(s["x"].shape[0])])]


def _plain_qk(s):
    c = s["case"]
    M, D, R = c["M"], c["D"], c["R"]
    inside = (s["pos"] >= 0) & (s["pos"] < c["P"])
    row = s["table"][torch.where(inside, s["pos"], torch.zeros_like(s["pos"])).to(torch.int64)]
    cos, sin = row[:, None, :R // 2], row[:, None, R // 2:]
    out = []
    for h0, H, w in ((0, c["Hq"], s["qw"]), (c["Hq"], c["Hk"], s["kw"])):
        x = s["x"][:, h0 * D:(h0 + H) * D].to(torch.float32).reshape(M, H, D)
        x = x / torch.sqrt((x * x).mean(dim=2, keepdim=True) + EPS) * w.to(torch.float32)
        a, b = (x[..., :R // 2], x[..., R // 2:R]) if c["style"] == "half" else (x[..., 0:R:2], x[..., 1:R:2])
        u, v = a * cos - b * sin, b * cos + a * sin
        y = torch.cat((u, v), dim=2) if c["style"] == "half" else torch.stack((u, v), dim=3).reshape(M, H, R)
        y = torch.cat((y, x[..., R:]), dim=2)
        out.append(torch.where(inside[:, None, None], y, torch.zeros_like(y)).to(TYPES[c["y"]]))
    return out


def _plain_logprobs(s):
    c = s["case"]
    l = s["x"].to(torch.float32)
    live = l > -math.inf
    m = l.amax(dim=1, keepdim=True)
    z = torch.where(live, l - m, torch.zeros_like(l))
    e = torch.where(live, torch.exp(z), torch.zeros_like(l))
    # long sums, and the logarithm of one that is hardly above 1
    total = e.to(torch.float64).sum(dim=1)
    lse = torch.log(total)
    entropy = lse - (e * z).to(torch.float64).sum(dim=1) / total
    t = s["t"].to(torch.int64)
    inside = (t >= 0) & (t < c["V"])
    lt = torch.gather(l, 1, torch.where(inside, t, torch.zeros_like(t))[:, None])[:, 0]
    shift = (lse + m[:, 0].to(torch.float64))
    logp = torch.where(inside, lt.to(torch.float64) - shift, torch.zeros_like(lse)).to(torch.float32)
    order = torch.sort(l, dim=1, descending=True, stable=True)
    top = order.values[:, :c["top_k"]].to(torch.float64)
    ids = order.indices[:, :c["top_k"]].to(torch.int32)
    ids = torch.where(top > -math.inf, ids, torch.full_like(ids, -1))
    return [logp, entropy.to(torch.float32), ids, (top - shift[:, None]).to(torch.float32)]


def _values(codes, scales, square):
    """e4m3 codes (..., N, K) and the scales of their blocks -> the values, in 32 bits."""
    n, k = codes.shape[-2:]
    s = scales.repeat_interleave(BLOCK, dim=-1)[..., :k]
    if square:
        s = s.repeat_interleave(BLOCK, dim=-2)[..., :n, :]
    return codes.to(torch.float32) * s


def _plain_gather(ids, codes, scales, x, per_slot):
    """Every (token, slot) row's product with its expert's weights: (M, top_k, N)."""
    M, top_k = ids.shape
    E, N = codes.shape[:2]
    flat = ids.reshape(-1).to(torch.int64)
    inside = (flat >= 0) & (flat < E)
    if flat.numel() <= E:                                       # few pairs: their own weights
        e = torch.where(inside, flat, torch.zeros_like(flat))
        w = _values(codes.view(torch.uint8)[e].view(F8), scales[e], True)
        v = x.reshape(M * top_k, -1) if per_slot else x[:, None].expand(M, top_k, x.shape[-1]).reshape(M * top_k, -1)
        y = torch.bmm(w, v[:, :, None].contiguous())[:, :, 0]
        return torch.where(inside[:, None], y, torch.zeros_like(y)).reshape(M, top_k, N)
    # many pairs: sorted by expert, each expert's pairs padded to the longest list
    e = torch.where(inside, flat, torch.full_like(flat, E))
    order = torch.argsort(e, stable=True)
    se = e[order]
    counts = torch.bincount(e, minlength=E + 1)
    at = torch.arange(flat.numel(), device=flat.device) - (torch.cumsum(counts, 0) - counts)[se]
    kept = se < E
    se, at, order = se[kept], at[kept], order[kept]
    longest = max(1, int(counts[:E].max()))
    v = torch.zeros(E, x.shape[-1], longest, device=x.device)
    v[se, :, at] = x.reshape(M * top_k, -1)[order] if per_slot else x[order // top_k]
    out = torch.bmm(_values(codes, scales, True), v)            # (E, N, longest)
    y = torch.zeros(M * top_k, N, device=x.device)
    y[order] = out[se, :, at]
    return y.reshape(M, top_k, N)


def _plain_product(s):
    op = s["case"]["op"]
    x = _values(s["x"], s["xs"], False)
    if op == "dense":
        return [x @ _values(s["codes"], s["scales"], True).t()]
    g = _plain_gather(s["ids"], s["codes"], s["scales"], x, op == "combine")
    if op == "swiglu":
        u = _plain_gather(s["ids"], s["up_codes"], s["up_scales"], x, False)
        return [g / (1.0 + torch.exp(-g)) * u]
    if op == "combine":
        return [(s["rw"][:, :, None] * g).sum(dim=1)]
    return [g]


# --------------------------------------------------- the framework's calls

def _own(s):
    import bit_block_quantized_amd as q

    c = s["case"]
    op = c["op"]
    if op == "norm":
        y, ys, h = q.qmx_rmsnorm(s["x"], s["weight"], eps=EPS, residual=s["res"], fmt="f8")
        y = q.qmx_dequantize(y, ys, "f8")
        return [y] if h is None else [y, h]
    if op == "quantize":
        return [q.qmx_dequantize(*q.qmx_quantize(s["x"], "f8"), "f8")]
    if op == "weights":
        return [q.qmt_dequantize_weights(*q.qmt_quantize_weights(s["x"]))]
    if op == "qk":
        return list(q.qmt_qk_norm_rope(s["x"], c["Hq"], c["Hk"], c["D"], s["table"], s["pos"], s["qw"], s["kw"], eps=EPS,
                                       style=c["style"], dtype=TYPES[c["y"]]))
    if op == "logprobs":
        return list(q.qmt_logprobs(s["x"], s["t"], c["top_k"]))
    if op == "dense":
        return [q.qmv_dense("f8", s["codes"], s["scales"], s["x"], s["xs"])]
    if op == "gather":
        return [q.qmv_gather_moe("f8", s["codes"], s["scales"], s["ids"], s["x"], s["xs"])]
    if op == "swiglu":
        return [q.qmv_gather_moe_swiglu("f8", s["codes"], s["scales"], s["up_codes"], s["up_scales"], s["ids"], s["x"],
                                        s["xs"])]
    return [q.qmv_gather_moe_combine("f8", s["codes"], s["scales"], s["ids"], s["rw"], s["x"], s["xs"])]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "quantize":
        return [_round_trip(state["x"].to(torch.float32), False)]
    plain = {"norm": _plain_norm, "weights": _plain_weights, "qk": _plain_qk, "logprobs": _plain_logprobs}
    return plain.get(op, _plain_product)(state)


# ------------------------------------------------------------------- costs

def work(case):
    c = case
    op = c["op"]
    if op in ("norm", "quantize"):
        n = c["M"] * c["K"]
        # codes and scales are written and, for the values, read once; the values are bf16
        return dict(bytes=n * (BYTES[c["x"]] + 2 * BYTES[c["res"]] + 2 + 2) + 8 * c["M"] * _blocks(c["K"]) +
                    (2 * c["K"] if op == "norm" else 0), flops=(4 if op == "norm" else 2) * n)
    if op == "weights":
        n = c["E"] * c["N"] * c["K"]
        return dict(bytes=n * (BYTES[c["x"]] + 2 + 2) + 8 * c["E"] * _blocks(c["N"]) * _blocks(c["K"]), flops=2 * n)
    if op == "qk":
        n = c["M"] * (c["Hq"] + c["Hk"]) * c["D"]
        return dict(bytes=n * (BYTES[c["x"]] + BYTES[c["y"]]) + 4 * c["M"] * (c["R"] + 1) + 4 * c["D"], flops=7 * n)
    if op == "logprobs":
        n = c["M"] * c["V"]
        return dict(bytes=n * BYTES[c["x"]] + c["M"] * (12 + 8 * c["top_k"]), flops=6 * n)
    pairs = c["M"] * c["top_k"]
    # the experts that the pairs can select at most; each selected one's weights are read once
    selected = min(c["E"], pairs) * (2 if op == "swiglu" else 1)
    kb = _blocks(c["K"])
    vectors = pairs if op == "combine" else c["M"]
    out = (c["M"] if op == "combine" else pairs) * c["N"]
    return dict(bytes=selected * (c["N"] * c["K"] + 4 * _blocks(c["N"]) * kb) + vectors * (c["K"] + 4 * kb) + 4 * out +
                (0 if op == "dense" else 4 * pairs) + (4 * pairs if op == "combine" else 0),
                flops=2 * pairs * c["N"] * c["K"] * (2 if op == "swiglu" else 1))


# ------------------------------------------------- the definitions, 64 bits

def _e4m3_values():
    """The 127 values 0 .. 448 in order, from sign, exponent and mantissa."""
    return [m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:127]


def _exact_codes(codes, device):
    """Bytes -> the values that they stand for, in 64 bits (NaN at 127 and 255)."""
    up = _e4m3_values() + [math.nan]
    table = torch.tensor(up + [-v for v in up], dtype=torch.float64, device=device)
    return table[codes.view(torch.uint8).int()]


def _exact_values(codes, scales, square):
    v = _exact_codes(codes, codes.device)
    for b in range(scales.shape[-1]):
        part = v[..., b * BLOCK:(b + 1) * BLOCK]
        if square:
            for r in range(scales.shape[-2]):
                part[..., r * BLOCK:(r + 1) * BLOCK, :] *= scales[..., r, b].double()[..., None, None]
        else:
            part *= scales[..., b].double()[..., None]
    return v


def _exact_quantized(x, square):
    """The values x (N, K), 64 bits, as blocks hold them; the scale is held in 32 bits."""
    grid = torch.tensor(_e4m3_values(), dtype=torch.float64, device=x.device)
    middle = (grid[1:] + grid[:-1]) / 2
    out = torch.empty_like(x)
    for r in range(0, x.shape[0], BLOCK if square else x.shape[0]):
        rows = slice(r, r + (BLOCK if square else x.shape[0]))
        for k in range(0, x.shape[1], BLOCK):
            b = x[rows, k:k + BLOCK]
            amax = b.abs().max() if square else b.abs().amax(dim=1, keepdim=True)
            d = torch.clamp((amax / LARGEST).float().double(), min=LEAST_SCALE)
            a = (b / d).abs().clamp(max=LARGEST)
            i = torch.searchsorted(middle, a)                   # values at a middle stay below it ..
            at = (i < 126) & (a == middle[i.clamp(max=125)])
            i = i + (at & (i % 2 == 1))                         # .. unless the code above is the even one
            out[rows, k:k + BLOCK] = torch.sign(b) * grid[i] * d
    return out


def _exact_gather(ids, codes, scales, x, per_slot):
    M, top_k = ids.shape
    y = torch.zeros(M, top_k, codes.shape[1], dtype=torch.float64, device=x.device)
    for e in range(codes.shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel():
            y[t, j] = (x[t, j] if per_slot else x[t]) @ _exact_values(codes[e], scales[e], True).t()
    return y


def _exact_heads(x, w, cos, sin, R, style):
    x = x * torch.rsqrt(x.square().sum(dim=-1, keepdim=True) / x.shape[-1] + EPS) * w.double()
    i = torch.arange(R // 2, device=x.device)
    first, second = (i, i + R // 2) if style == "half" else (2 * i, 2 * i + 1)
    turned = x.clone()
    z = torch.complex(x[..., first], x[..., second]) * torch.complex(cos, sin)[:, None]
    turned[..., first], turned[..., second] = z.real, z.imag
    return turned


def exact(case, seed):
    s = _inputs(case, seed)
    c, op = case, case["op"]
    if op == "norm":
        h = s["x"].double() if s["res"] is None else s["x"].double() + s["res"].double()
        n = h / torch.sqrt(h.square().sum(dim=1, keepdim=True) / c["K"] + EPS) * s["weight"].double()
        y = _exact_quantized(n, False)
        return [y] if s["res"] is None else [y, h]
    if op == "quantize":
        return [_exact_quantized(s["x"].double(), False)]
    if op == "weights":
        if c["E"] * _blocks(c["N"]) * _blocks(c["K"]) > 40000:  # (a few launches for each block)
            return None
        return [torch.stack([_exact_quantized(s["x"][e].double(), True) for e in range(c["E"])])]
    if op == "qk":
        out = []
        inside = (s["pos"] >= 0) & (s["pos"] < c["P"])
        row = s["table"][s["pos"].long() % c["P"]].double()
        for lo, H, w in ((0, c["Hq"], s["qw"]), (c["Hq"] * c["D"], c["Hk"], s["kw"])):
            x = s["x"][:, lo:lo + H * c["D"]].double().reshape(c["M"], H, c["D"])
            y = _exact_heads(x, w, row[:, :c["R"] // 2], row[:, c["R"] // 2:], c["R"], c["style"])
            out.append(y * inside[:, None, None])
        return out
    if op == "logprobs":
        logp, entropy, ids, top = [], [], [], []
        for r0 in range(0, c["M"], 64):                         # (64 rows at a time in 64 bits)
            lp = torch.log_softmax(s["x"][r0:r0 + 64].double(), dim=1)
            t = s["t"][r0:r0 + 64].long()
            given = torch.gather(lp, 1, t.clamp(min=0)[:, None])[:, 0]
            logp.append(torch.where(t >= 0, given, torch.zeros_like(given)))
            entropy.append(torch.special.entr(torch.exp(lp)).sum(dim=1))
            # among equal logits the lower index comes first
            i = torch.argsort(-lp, dim=1, stable=True)[:, :c["top_k"]]
            v = torch.gather(lp, 1, i)
            ids.append(torch.where(v > -math.inf, i, torch.full_like(i, -1)).int())
            top.append(v)
        return [torch.cat(logp), torch.cat(entropy), torch.cat(ids), torch.cat(top)]
    x = _exact_values(s["x"], s["xs"], False)
    if op == "dense":
        return [x @ _exact_values(s["codes"], s["scales"], True).t()]
    g = _exact_gather(s["ids"], s["codes"], s["scales"], x, op == "combine")
    if op == "swiglu":
        return [g * torch.sigmoid(g) * _exact_gather(s["ids"], s["up_codes"], s["up_scales"], x, False)]
    if op == "combine":
        return [(s["rw"].double()[:, :, None] * g).sum(dim=1)]
    return [g]
