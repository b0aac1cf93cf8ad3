"""Cases and plain forms of the operators for sublayers in 8 bits.

A root-mean-square norm that adds the residual first and gives its output in 8
bits (and its backward), the matrix product of 8-bit numbers with a scale for
each block of 128 (forward, and the gradient of its rows with the cast in front
of it), and a whole mixture-of-experts layer for a few tokens.  ``run`` computes
a case with elementary torch operations where ``own`` is false and with this
repository's kernels where it is true; ``exact`` computes it in 64 bits.

8-bit numbers are E4M3 codes (uint8) with UE8M0 scale bytes or fp32 scales: one
for 128 values of a row, or for a block of 128 x 128 of a weight matrix.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZE = {"fp32": 4, "bf16": 2, "fp16": 2}
BLOCK = 128
EPS = 1e-6


def listed():
    return [
        # a decode step's sublayer input: 16 tokens at the model's width, in bf16 and in 8 bits; latency
        {"name": "norm_decode", "op": "norm", "n": 16, "d": 5120, "x": "bf16", "w": "fp32", "pitch": 5120, "residual": True,
         "out": "both"},
        # the long prefill: 65,536 tokens, 8 bits only (a product reads them)
        {"name": "norm_prefill", "op": "norm", "n": 65536, "d": 5120, "x": "bf16", "w": "fp32", "pitch": 5120,
         "residual": True, "out": "fp8"},
        # training: 8,192 tokens, bf16 activations, fp32 gradients, one of them past the norm
        {"name": "norm_backward", "op": "norm_backward", "n": 8192, "d": 5120, "x": "bf16", "g": "fp32", "w": "fp32",
         "pitch": 5120, "residual": True},
        # an odd width in fp32, rows cut out of a wider buffer
        {"name": "norm_backward_odd", "op": "norm_backward", "n": 1501, "d": 1031, "x": "fp32", "g": "fp32", "w": "fp32",
         "pitch": 1040, "residual": False},
        # one token through a small projection: the smallest call, latency
        {"name": "mm_token", "op": "mm", "M": 1, "N": 512, "K": 1024, "scales": "ue8m0", "y": "bf16"},
        # a decode batch through a wide projection: bound by the weights
        {"name": "mm_decode", "op": "mm", "M": 16, "N": 16384, "K": 5120, "scales": "ue8m0", "y": "bf16"},
        # a prefill's projection with scales as checkpoints have them, fp32: bound by the tensor cores
        {"name": "mm_prefill", "op": "mm", "M": 16384, "N": 10240, "K": 5120, "scales": "fp32", "y": "bf16"},
        # training: the gradient of the rows of a projection, with the cast of the output's gradient
        {"name": "mm_gradient", "op": "mm_gradient", "M": 8192, "N": 10240, "K": 5120, "scales": "ue8m0", "g": "bf16",
         "y": "bf16"},
        # the same at sizes that fill no tile and no block of scales
        {"name": "mm_gradient_ragged", "op": "mm_gradient", "M": 777, "N": 1040, "K": 720, "scales": "fp32", "g": "fp16",
         "y": "fp32"},
        # one sequence's token through 6 of 64 experts, 8-bit weights, routed in the call
        {"name": "moe_token", "op": "moe", "T": 1, "experts": 64, "k": 6, "d": 5120, "inner": 2048, "x": "bf16",
         "w": "ue8m0", "route": "softmax", "pad": 0},
        # a decode batch of 16 sequences
        {"name": "moe_decode", "op": "moe", "T": 16, "experts": 64, "k": 6, "d": 5120, "inner": 2048, "x": "bf16",
         "w": "ue8m0", "route": "sigmoid", "pad": 0},
        # 16-bit weights, odd sizes, routed by the user, a batch with padded tokens
        {"name": "moe_ragged", "op": "moe", "T": 37, "experts": 13, "k": 3, "d": 1072, "inner": 336, "x": "bf16",
         "w": "same", "route": "given", "pad": 4},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "mm", "mm", "mm_gradient", "moe", "moe"])
    if op in ("norm", "norm_backward"):
        d = _log(rng, 1, 16384)
        if rng.random() < 0.6:
            d = max(16, d // 16 * 16)
        n = _log(rng, 1, 65536)
        x = rng.choice(["bf16", "fp16", "fp32"])
        n = max(1, min(n, (65536 if op == "norm" else 8192) * 5120 * 2 // (d * 2 * SIZE[x])))
        c = {"op": op, "n": n, "d": d, "x": x, "w": rng.choice(["fp32", x]), "pitch": d + rng.choice([0, 0, 0, 1, 8, 64]),
             "residual": rng.random() < 0.7}
        if op == "norm":
            c["out"] = rng.choice(["y", "fp8", "both"])
        else:
            c["g"] = rng.choice(["fp32", x])
        return c
    if op in ("mm", "mm_gradient"):
        M = rng.choice([_log(rng, 1, 64), _log(rng, 1, 16384)])
        N, K = 16 * _log(rng, 1, 1024), 16 * _log(rng, 1, 640)
        most = 16384 * 10240 * 5120 // (1 if op == "mm" else 4)
        M = max(1, min(M, most // (N * K)))
        c = {"op": op, "M": M, "N": N, "K": K, "scales": rng.choice(["ue8m0", "fp32"]), "y": rng.choice(["bf16", "fp16", "fp32"])}
        if op == "mm_gradient":
            c["g"] = rng.choice(["bf16", "fp16", "fp32"])
        return c
    E = _log(rng, 1, 64)
    d, inner = 16 * _log(rng, 1, 400), 16 * _log(rng, 1, 256)
    w = rng.choice(["ue8m0", "fp32", "same"])
    inner = max(16, min(inner, 48 * 5120 * 2048 // (2 if w == "same" else 1) // (E * d) // 16 * 16))
    return {"op": op, "T": _log(rng, 1, 64), "experts": E, "k": rng.randint(1, min(8, E)), "d": d, "inner": inner,
            "x": rng.choice(["bf16", "fp16"]), "w": w,
            "route": rng.choice(["softmax", "sigmoid", "given"]), "pad": 0}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _blocks(n):
    return -(-n // BLOCK)


def _scales(shape, kind, typical, g):
    """Scales of weight blocks: within a factor of four of `typical`, as UE8M0 bytes or fp32."""
    if kind == "fp32":
        return typical * torch.exp2(2 * torch.rand(shape, generator=g, device=DEV) - 1)
    e = round(math.log2(typical)) + 127
    return torch.randint(e - 1, e + 2, shape, generator=g, device=DEV, dtype=torch.uint8)


def _codes(shape, g):
    """E4M3 codes of a matrix whose blocks were scaled to reach about 448."""
    v = torch.empty(shape, dtype=torch.float16, device=DEV).normal_(0, 110, generator=g).clamp_(-448, 448)
    return v.to(torch.float8_e4m3fn).view(torch.uint8)


def _activations(n, d, g):
    """Tokens of different scale, one channel in a hundred twenty times the others."""
    x = torch.randn((n, d), generator=g, device=DEV)
    x.mul_(torch.where(torch.rand((d,), generator=g, device=DEV) < 0.01, 20.0, 1.0))
    return x.mul_(0.3 + 1.5 * torch.rand((n, 1), generator=g, device=DEV))


def _pitched(x, pitch, t):
    buf = torch.zeros((x.shape[0], pitch), dtype=t, device=DEV)
    buf[:, :x.shape[1]] = x
    return buf[:, :x.shape[1]]


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] in ("norm", "norm_backward"):
        n, d, t = case["n"], case["d"], TYPES[case["x"]]
        s = {"case": case, "x": _pitched(_activations(n, d, g), case["pitch"], t),
             "w": (0.5 + torch.rand((d,), generator=g, device=DEV)).to(TYPES[case["w"]]), "residual": None, "g_r": None}
        if case["op"] == "norm":
            if case["residual"]:
                s["residual"] = torch.randn((n, d), generator=g, device=DEV).mul_(2).to(t)
            return s
        gt = TYPES[case["g"]]
        s["g_y"] = torch.randn((n, d), generator=g, device=DEV).to(gt)
        if case["residual"]:
            s["g_r"] = torch.randn((n, d), generator=g, device=DEV).mul_(0.5).to(gt)
        s["rstd"] = (s["x"].float().square().mean(1, dtype=torch.float64) + EPS).rsqrt().float()
        return s
    if case["op"] in ("mm", "mm_gradient"):
        M, N, K = case["M"], case["N"], case["K"]
        s = {"case": case, "w": _codes((N, K), g), "w_scales": _scales((_blocks(N), _blocks(K)), case["scales"], K ** -0.5 / 110, g)}
        if case["op"] == "mm":
            s["x"], e = _cast(_activations(M, K, g))
            s["x_scales"] = e if case["scales"] == "ue8m0" else _power(e)
        else:
            # an output's gradient: small, of different size from row to row
            s["g_y"] = _activations(M, N, g).mul_(1e-3 if case["g"] != "fp16" else 0.1).to(TYPES[case["g"]])
        return s
    T, E, k, d, inner, t = case["T"], case["experts"], case["k"], case["d"], case["inner"], TYPES[case["x"]]
    s = {"case": case, "x": torch.randn((T, d), generator=g, device=DEV).to(t), "up_scales": None, "down_scales": None}
    if case["w"] == "same":
        s["up"] = torch.empty((E, 2, inner, d), dtype=t, device=DEV).normal_(0, d ** -0.5, generator=g)
        s["down"] = torch.empty((E, d, inner), dtype=t, device=DEV).normal_(0, inner ** -0.5, generator=g)
    else:
        s["up"], s["down"] = _codes((E, 2, inner, d), g), _codes((E, d, inner), g)
        s["up_scales"] = _scales((E, 2, _blocks(inner), _blocks(d)), case["w"], d ** -0.5 / 110, g)
        s["down_scales"] = _scales((E, _blocks(d), _blocks(inner)), case["w"], inner ** -0.5 / 110, g)
    # (some experts are more in demand than others)
    logits = torch.randn((T, E), generator=g, device=DEV) + 0.5 * torch.randn((E,), generator=g, device=DEV)
    if case["route"] == "given":
        p, ids = torch.softmax(logits, 1).topk(k, 1)
        s["ids"], s["p"] = ids.int(), p / p.sum(1, keepdim=True)
        s["ids"][T - case["pad"]:] = -1
    else:
        s["logits"] = logits
    return s


# ------------------------------------------------------------------ 8-bit numbers
def _power(byte):
    """2^(byte - 127) of scale bytes from 1 on: the byte is the exponent field of the fp32 number."""
    return (byte.int() << 23).view(torch.float32)


def _value(scales):
    return scales if scales.dtype == torch.float32 else _power(scales)


def _grouped(x):
    """Rows as groups of 128, the last one filled up with zeros."""
    d = x.shape[1]
    if d % BLOCK:
        x = torch.nn.functional.pad(x, (0, BLOCK - d % BLOCK))
    return x.view(x.shape[0], -1, BLOCK)


def _cast(x):
    """fp32 rows -> E4M3 codes and UE8M0 scales of groups of 128 (bytes).  The scale is the smallest power of two at or
    above amax / 448, from 2^-126 on."""
    n, d = x.shape
    x = _grouped(x)
    mant, expo = torch.frexp(x.abs().amax(2))
    expo = (expo - 9 + (mant > 0.875).to(expo.dtype)).clamp(-126, 127)      # 448 is 0.875 * 2^9
    expo = torch.where(mant == 0, torch.full_like(expo, -126), expo)
    scales = (expo + 127).to(torch.uint8)
    codes = (x / _power(scales)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.reshape(n, -1)[:, :d].contiguous(), scales


def _rows(codes, scales):
    """The fp32 values of rows in groups of 128."""
    d = codes.shape[1]
    return codes.view(torch.float8_e4m3fn).float() * _value(scales).repeat_interleave(BLOCK, 1)[:, :d]


def _matrix(codes, scales):
    """The fp32 values of matrices [..., N, K] in blocks of 128 x 128."""
    N, K = codes.shape[-2:]
    s = _value(scales).repeat_interleave(BLOCK, -2)[..., :N, :].repeat_interleave(BLOCK, -1)[..., :K]
    return codes.view(torch.float8_e4m3fn).float().mul_(s)


def _as_numbers(codes, scales):
    """8-bit codes and scales as the numbers that their formats hold."""
    return {"codes": codes.view(torch.float8_e4m3fn), "scales": scales.view(torch.float8_e8m0fnu)}


# ------------------------------------------------------------------ one pass
def run(state):
    return {"norm": _norm, "norm_backward": _norm_backward, "mm": _mm, "mm_gradient": _mm_gradient,
            "moe": _moe}[state["case"]["op"]](state)


def _norm(s):
    out = s["case"]["out"]
    if own:
        import hyper_connection_residual_mixes_gb300 as hcg
        r = hcg.hc_rms_norm(s["x"], s["w"], s["residual"], norm_eps=EPS, out=out, return_rstd=True)
        return {**r, **_as_numbers(r["codes"], r["scales"])} if "codes" in r else r
    res = {}
    v = s["x"].float()
    if s["residual"] is not None:
        res["r"] = (v + s["residual"].float()).to(s["x"].dtype)
        v = res["r"].float()
    rstd = (v.square().mean(1, keepdim=True) + EPS).rsqrt()
    res["rstd"] = rstd[:, 0]
    y = v * rstd * s["w"].float()
    if out != "fp8":
        res["y"] = y.to(s["x"].dtype)
    return res if out == "y" else {**res, **_as_numbers(*_cast(y))}


def _norm_backward(s):
    if own:
        import hyper_connection_residual_mixes_gb300 as hcg
        return hcg.hc_rms_norm_backward(s["g_y"], s["x"], s["w"], s["rstd"], g_r=s["g_r"])
    g, rstd = s["g_y"].float(), s["rstd"][:, None]
    xh = s["x"].float() * rstd
    wg = g * s["w"].float()
    g_x = rstd * (wg - xh * (wg * xh).mean(1, keepdim=True))
    if s["g_r"] is not None:
        g_x = g_x + s["g_r"].float()
    return {"g_x": g_x.to(s["g_y"].dtype), "g_norm_w": (g * xh).sum(0)}


def _mm(s):
    t = TYPES[s["case"]["y"]]
    if own:
        import hyper_connection_residual_mixes_gb300 as hcg
        return hcg.hc_fp8_mm(s["x"], s["x_scales"], s["w"], s["w_scales"], out_dtype=t)
    return (_rows(s["x"], s["x_scales"]) @ _matrix(s["w"], s["w_scales"]).t()).to(t)


def _mm_gradient(s):
    t = TYPES[s["case"]["y"]]
    if own:
        import hyper_connection_residual_mixes_gb300 as hcg
        codes, scales = hcg.hc_fp8_cast(s["g_y"])
        g_x = hcg.hc_fp8_mm(codes, scales, s["w"], s["w_scales"], transposed=True, out_dtype=t)
        return {"g_x": g_x, **_as_numbers(codes, scales)}
    codes, scales = _cast(s["g_y"].float())
    return {"g_x": (_rows(codes, scales) @ _matrix(s["w"], s["w_scales"])).to(t), **_as_numbers(codes, scales)}


def _moe(s):
    c, x = s["case"], s["x"].float()
    if own:
        import hyper_connection_residual_mixes_gb300 as hcg
        if c["route"] == "given":
            return {"y": hcg.hc_moe_tokens(s["x"], s["up"], s["down"], s["ids"], s["p"], up_scales=s["up_scales"],
                                           down_scales=s["down_scales"])}
        y, ids, p = hcg.hc_moe_tokens(s["x"], s["up"], s["down"], logits=s["logits"], top_k=c["k"], score=c["route"],
                                      up_scales=s["up_scales"], down_scales=s["down_scales"])
        return {"y": y, "ids": ids, "p": p}
    if c["route"] == "given":
        ids, p = s["ids"], s["p"]
    else:
        top, ids = s["logits"].topk(c["k"], 1)
        p = torch.exp(top - top[:, :1]) if c["route"] == "softmax" else torch.sigmoid(top)
        p, ids = p / p.sum(1, keepdim=True), ids.int()
    p_in = torch.where(ids >= 0, p, 0.0)
    at = ids.long().clamp(min=0)
    if c["T"] * c["k"] <= c["experts"]:
        # few choices: the chosen experts' weights, one matrix after another for each choice
        chosen = at.reshape(-1)
        up, down = (_gathered(s[n], s[n + "_scales"], chosen) for n in ("up", "down"))
        h = torch.matmul(up, x.repeat_interleave(c["k"], 0)[:, None, :, None])[..., 0]
        a = torch.nn.functional.silu(h[:, 0]) * h[:, 1] * p_in.reshape(-1, 1)
        y = torch.matmul(down, a[..., None])[..., 0].view(c["T"], c["k"], -1).sum(1)
    else:
        # all tokens through all experts, those not chosen with weight zero
        up, down = (_gathered(s[n], s[n + "_scales"], slice(None)) for n in ("up", "down"))
        share = torch.zeros((c["T"], c["experts"]), device=DEV).scatter_add_(1, at, p_in)
        h = torch.matmul(up, x.t())
        a = torch.nn.functional.silu(h[:, 0]) * h[:, 1] * share.t()[:, None, :]
        y = torch.matmul(down, a).sum(0).t()
    y = y.to(s["x"].dtype)
    return {"y": y} if c["route"] == "given" else {"y": y, "ids": ids, "p": p}


def _gathered(w, scales, at):
    return w[at].float() if scales is None else _matrix(w[at], scales[at])


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "norm":
        n, d, b = case["n"], case["d"], SIZE[case["x"]]
        each = b + (2 * b if case["residual"] else 0) + (0 if case["out"] == "fp8" else b) + (0 if case["out"] == "y" else 1 + 1 / BLOCK)
        return {"bytes": n * d * each + d * SIZE[case["w"]] + 4 * n, "flops": 6 * n * d}
    if case["op"] == "norm_backward":
        n, d = case["n"], case["d"]
        each = SIZE[case["x"]] + SIZE[case["g"]] * (3 if case["residual"] else 2)
        return {"bytes": n * d * each + d * (SIZE[case["w"]] + 4) + 4 * n, "flops": 10 * n * d}
    if case["op"] in ("mm", "mm_gradient"):
        M, N, K = case["M"], case["N"], case["K"]
        b = 1 if case["scales"] == "ue8m0" else 4
        size = N * K + b * _blocks(N) * _blocks(K)
        if case["op"] == "mm":
            size += M * K + b * M * _blocks(K) + M * N * SIZE[case["y"]]
        else:
            # the cast's codes are an output
            size += M * N * (SIZE[case["g"]] + 1) + M * _blocks(N) + M * K * SIZE[case["y"]]
        return {"bytes": size, "flops": 2 * M * N * K}
    T, E, k, d, inner = case["T"], case["experts"], case["k"], case["d"], case["inner"]
    rows = (T - case["pad"]) * k
    # experts without a token need no weights: with choices spread evenly this many have one
    busy = E * (1 - (1 - k / E) ** (T - case["pad"]))
    each = 2 if case["w"] == "same" else 1
    return {"bytes": busy * 3 * inner * d * each + 4 * T * d, "flops": 6 * rows * inner * d}


# ------------------------------------------------------------------ 64 bits
def _two(e):
    """2^e for whole e, from the bits of a 64-bit number (pow() need not be exact)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _expo(top):
    """The exponent of the smallest power of two at or above top / 448, from -126 on."""
    e = torch.frexp(top)[1].long() - 10
    e = e + (448 * _two(e) < top)
    e = e + (448 * _two(e) < top)
    return torch.where(top > 0, e, -126).clamp(-126, 127)


def _nearest_code(q):
    """The nearest number of three mantissa bits (steps of 2^-9 below 2^-6), at most 448."""
    grain = _two(torch.frexp(q.abs().clamp(min=2.0 ** -6))[1] - 4)
    return (torch.round(q / grain) * grain).clamp(-448, 448)


def _cast64(x):
    n, d = x.shape
    x = torch.cat([x, x.new_zeros((n, -d % BLOCK))], 1).view(n, -1, BLOCK)
    s = _two(_expo(x.abs().amax(2)))
    return _nearest_code(x / s[..., None]).view(n, -1)[:, :d], s


def _scale64(scales):
    return scales.double() if scales.dtype == torch.float32 else _two(scales.long() - 127)


def _matrix64(codes, scales):
    N, K = codes.shape
    i, j = (torch.arange(size, device=DEV) // BLOCK for size in (N, K))
    return codes.view(torch.float8_e4m3fn).double() * _scale64(scales)[i][:, j]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        d, part = case["d"], max(1, (1 << 27) // case["d"])
        res = {}
        for a in range(0, case["n"], part):
            got = {}
            v = s["x"][a:a + part].double()
            if s["residual"] is not None:
                got["r"] = v + s["residual"][a:a + part].double()
                v = got["r"].to(s["x"].dtype).double()
            rstd = 1 / torch.sqrt((v * v).sum(1, keepdim=True) / d + EPS)
            got["rstd"] = rstd[:, 0]
            y = v * rstd * s["w"].double()
            if case["out"] != "fp8":
                got["y"] = y
            if case["out"] != "y":
                got["codes"], got["scales"] = _cast64(y)
            for k, t in got.items():
                res.setdefault(k, []).append(t)
        return {k: torch.cat(t) for k, t in res.items()}
    if case["op"] == "norm_backward":
        g, rstd = s["g_y"].double(), s["rstd"].double()[:, None]
        xh = s["x"].double() * rstd
        wg = g * s["w"].double()
        g_x = (wg - xh * ((wg * xh).sum(1, keepdim=True) / case["d"])) * rstd
        if s["g_r"] is not None:
            g_x = g_x + s["g_r"].double()
        return {"g_x": g_x, "g_norm_w": (g * xh).sum(0)}
    if case["op"] == "mm":
        w = _matrix64(s["w"], s["w_scales"])
        j = torch.arange(case["K"], device=DEV) // BLOCK
        return (s["x"].view(torch.float8_e4m3fn).double() * _scale64(s["x_scales"])[:, j]) @ w.t()
    if case["op"] == "mm_gradient":
        codes, scales = _cast64(s["g_y"].double())
        j = torch.arange(case["N"], device=DEV) // BLOCK
        return {"g_x": (codes * scales[:, j]) @ _matrix64(s["w"], s["w_scales"]), "codes": codes, "scales": scales}
    x, E, k = s["x"].double(), case["experts"], case["k"]
    if case["route"] == "given":
        ids, p = s["ids"], s["p"].double()
    else:
        order = torch.sort(s["logits"], dim=1, descending=True, stable=True)[1][:, :k]
        top = torch.gather(s["logits"].double(), 1, order)
        p = torch.softmax(top, 1) if case["route"] == "softmax" else 1 / (1 + torch.exp(-top))
        p, ids = p / p.sum(1, keepdim=True), order.int()
    y = torch.zeros(x.shape, dtype=torch.float64, device=DEV)
    for e in range(E):
        t, slot = (ids == e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        wide = lambda name, *at: (s[name][(e, *at)].double() if s[name + "_scales"] is None
                                  else _matrix64(s[name][(e, *at)], s[name + "_scales"][(e, *at)]))
        gate, up = x[t] @ wide("up", 0).t(), x[t] @ wide("up", 1).t()
        y.index_add_(0, t, ((gate / (1 + torch.exp(-gate)) * up) @ wide("down").t()) * p[t, slot][:, None])
    return {"y": y} if case["route"] == "given" else {"y": y, "ids": ids, "p": p}
