"""Cases and plain forms of the sublayer's training and serving operators.

Three operators stand between two steps of the hyper-connection path: the
layer norm of the sublayer input (forward and backward), the experts' matrix
products on rows sorted by expert (forward and both gradients), and the AdamW
step of the parameters.  ``run`` computes a case with elementary torch
operations where ``own`` is false and with this repository's kernels where it
is true; ``exact`` computes it in 64 bits.

The plain forms work on whole buffers: the experts' products on a copy of the
rows padded to the busiest expert, the AdamW step on the flat buffers whose
slices are the parameters.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZE = {"fp32": 4, "bf16": 2, "fp16": 2}

# one side's hyper-connection parameters: hc_fn [24, 4 * 5120], hc_base [24], hc_scale [3], norm_w [5120]
SIDE = (24 * 4 * 5120, 24, 3, 5120)
GROUP = 32       # values that share a scale in the 8-bit states
LN_EPS = 1e-5
ADAM = {"beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "weight_decay": 0.1, "lr": 3e-4, "step": 1200}


def listed():
    return [
        # a decode step's sublayer input: 16 tokens at the model's width; latency
        {"name": "norm_decode", "op": "norm", "n": 16, "d": 5120, "x": "bf16", "w": "fp32", "pitch": 5120},
        # the long prefill: 65,536 tokens
        {"name": "norm_prefill", "op": "norm", "n": 65536, "d": 5120, "x": "bf16", "w": "fp32", "pitch": 5120},
        # training: 8,192 tokens, bf16 activations with fp32 gradients as the side step's backward gives them
        {"name": "norm_backward", "op": "norm_backward", "n": 8192, "d": 5120, "x": "bf16", "g": "fp32", "w": "fp32",
         "pitch": 5120},
        # an odd width in fp32, rows cut out of a wider buffer
        {"name": "norm_backward_odd", "op": "norm_backward", "n": 1501, "d": 1031, "x": "fp32", "g": "fp32",
         "w": "fp32", "pitch": 1040},
        # one sequence's token through its 6 experts of 8: the smallest serving call, latency
        {"name": "experts_token", "op": "experts", "n": 6, "pad": 0, "experts": 8, "K": 1024, "N": 512, "x": "bf16",
         "kn": False, "skew": 0.3},
        # a decode batch: 128 tokens to 6 of 64 experts each; bound by the weights
        {"name": "experts_decode", "op": "experts", "n": 768, "pad": 0, "experts": 64, "K": 5120, "N": 2048, "x": "bf16",
         "kn": False, "skew": 0.5},
        # a prefill chunk: 8,192 tokens to 6 of 64 experts each; bound by the tensor cores
        {"name": "experts_prefill", "op": "experts", "n": 49152, "pad": 0, "experts": 64, "K": 5120, "N": 2048,
         "x": "bf16", "kn": False, "skew": 0.2},
        # training: both gradients of the products of 16 experts
        {"name": "experts_backward", "op": "experts_backward", "n": 16384, "pad": 0, "experts": 16, "K": 5120, "N": 2048,
         "x": "bf16", "kn": False, "skew": 0.2},
        # ragged: fp16, odd row counts, sizes that fill no tile, rows behind the last expert's, weights stored [K, N]
        {"name": "experts_backward_ragged", "op": "experts_backward", "n": 1777, "pad": 45, "experts": 13, "K": 1032,
         "N": 520, "x": "fp16", "kn": True, "skew": 0.9},
        # one side's four parameters: latency
        {"name": "adamw_side", "op": "adamw", "lay": "sides", "count": 1, "numel": 0, "align": 32, "p": "fp32", "g": "fp32",
         "states": "fp32", "copy": "", "scaled": False},
        # the hyper-connection parameters of 80 sides: 320 tensors in one step
        {"name": "adamw_sides", "op": "adamw", "lay": "sides", "count": 80, "numel": 0, "align": 32, "p": "fp32",
         "g": "fp32", "states": "fp32", "copy": "", "scaled": True},
        # experts' weights in bf16 with 8-bit states: 24 matrices of 2048 x 5120
        {"name": "adamw_experts_8bit", "op": "adamw", "lay": "even", "count": 24, "numel": 2048 * 5120, "align": 32,
         "p": "bf16", "g": "bf16", "states": "mxfp8", "copy": "", "scaled": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "experts", "experts", "experts_backward", "adamw", "adamw"])
    if op in ("norm", "norm_backward"):
        d = _log(rng, 1, 16384)
        if rng.random() < 0.5:
            d = max(64, d // 64 * 64)
        n = _log(rng, 1, 65536)
        n = max(1, min(n, (65536 if op == "norm" else 16384) * 5120 // d))
        x = rng.choice(["bf16", "fp16", "fp32"])
        c = {"op": op, "n": n, "d": d, "x": x, "w": rng.choice(["fp32", x]), "pitch": d + rng.choice([0, 0, 0, 1, 8, 64])}
        if op == "norm_backward":
            c["g"] = rng.choice(["fp32", x])
        return c
    if op in ("experts", "experts_backward"):
        E = _log(rng, 1, 64)
        K, N = 8 * _log(rng, 1, 1024), 8 * _log(rng, 1, 1024)
        most = 49152 * 5120 * 2048 // (1 if op == "experts" else 3)
        N = max(8, min(N, 64 * 5120 * 2048 // (E * K) // 8 * 8))
        n = max(1, min(_log(rng, 1, 49152), most // (K * N)))
        n = max(1, min(n, 65536 * 5120 // max(K, N)))
        return {"op": op, "n": n, "pad": rng.choice([0, 0, 1, n // 7]) if n > 1 else 0, "experts": E, "K": K, "N": N,
                "x": rng.choice(["bf16", "fp16"]), "kn": rng.random() < 0.5, "skew": rng.choice([0.0, 0.3, 0.9])}
    lay = rng.choice(["sides", "even", "ragged"])
    states = rng.choice(["fp32", "mxfp8"])
    p = rng.choice(["fp32", "fp32", "bf16", "fp16"])
    c = {"op": op, "lay": lay, "count": _log(rng, 1, 80 if lay == "sides" else 300), "numel": 0,
         "align": 32 if states == "mxfp8" else rng.choice([32, 32, 1]), "p": p, "g": rng.choice(["fp32", p]),
         "states": states, "copy": rng.choice(["", "bf16"]) if p == "fp32" else "", "scaled": rng.random() < 0.5}
    if lay != "sides":
        c["numel"] = _log(rng, 1, max(1, 100_000_000 // c["count"]))
    return c


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _sizes(case):
    if case["lay"] == "sides":
        return list(SIDE) * case["count"]
    if case["lay"] == "even":
        return [case["numel"]] * case["count"]
    r = random.Random(case["numel"])
    return [max(1, int(case["numel"] * r.uniform(0.1, 1.9))) for _ in range(case["count"])]


def _places(case):
    """(start, size) of each parameter in the flat buffers, and the buffers' length."""
    at, places = 0, []
    for s in _sizes(case):
        places.append((at, s))
        at += -(-s // case["align"]) * case["align"]
    return places, at


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] in ("norm", "norm_backward"):
        n, d, t = case["n"], case["d"], TYPES[case["x"]]
        # tokens of different scale and offset, one channel in a hundred twenty times the others
        x = torch.randn((n, d), generator=g, device=DEV)
        x.mul_(torch.where(torch.rand((d,), generator=g, device=DEV) < 0.01, 20.0, 1.0))
        x.mul_(0.3 + 1.5 * torch.rand((n, 1), generator=g, device=DEV)).add_(0.3 * torch.randn((n, 1), generator=g, device=DEV))
        buf = torch.zeros((n, case["pitch"]), dtype=t, device=DEV)
        buf[:, :d] = x
        s = {"case": case, "x": buf[:, :d],
             "w": (0.5 + torch.rand((d,), generator=g, device=DEV)).to(TYPES[case["w"]]),
             "b": (0.1 * torch.randn((d,), generator=g, device=DEV)).to(TYPES[case["w"]])}
        if case["op"] == "norm_backward":
            s["g_y"] = torch.randn((n, d), generator=g, device=DEV).to(TYPES[case["g"]])
            v = x.copy_(s["x"])
            mean = v.mean(1, dtype=torch.float64)
            var = torch.var_mean(v, 1, correction=0)[0].double()
            s["mean"], s["rstd"] = mean.float(), (var + LN_EPS).rsqrt().float()
        return s
    if case["op"] in ("experts", "experts_backward"):
        n, E, K, N, t = case["n"], case["experts"], case["K"], case["N"], TYPES[case["x"]]
        cpu = torch.Generator().manual_seed(seed)
        share = torch.softmax(case["skew"] * torch.randn((E,), generator=cpu), 0)
        counts = torch.bincount(torch.multinomial(share, n - case["pad"], True, generator=cpu), minlength=E)
        offsets = torch.zeros((E + 1,), dtype=torch.int32)
        offsets[1:] = counts.cumsum(0)
        s = {"case": case, "offsets": offsets.to(DEV), "most": max(1, int(counts.max())),
             "x": torch.randn((n, K), generator=g, device=DEV).to(t),
             "w": torch.empty((E, K, N) if case["kn"] else (E, N, K), dtype=t, device=DEV).normal_(0, K ** -0.5, generator=g)}
        if case["op"] == "experts_backward":
            s["g_y"] = torch.randn((n, N), generator=g, device=DEV).to(t)
        return s
    places, total = _places(case)
    real = torch.zeros((total,), device=DEV)
    real.scatter_(0, torch.tensor([a for a, _ in places], device=DEV), 1.0)
    ends = torch.tensor([a + k for a, k in places], device=DEV)
    real.scatter_add_(0, ends[ends < total], torch.full((int((ends < total).sum()),), -1.0, device=DEV))
    real = real.cumsum(0).clamp_(0, 1) if case["align"] > 1 else torch.ones_like(real)
    # gradients of a few magnitudes with a few large ones, moments of a run in its middle
    size = 1e-3 * torch.exp(torch.randn((total,), generator=g, device=DEV)) * real
    grad = torch.randn((total,), generator=g, device=DEV) * size
    m = 0.3 * torch.randn((total,), generator=g, device=DEV) * size
    r = (0.5 + torch.rand((total,), generator=g, device=DEV)) * size
    flat = {"p": (0.02 * torch.randn((total,), generator=g, device=DEV) * real).to(TYPES[case["p"]]),
            "g": grad.to(TYPES[case["g"]])}
    if case["states"] == "mxfp8":
        flat["m"], flat["m_scales"] = _encode(m, False)
        flat["v"], flat["v_scales"] = _encode(r, True)
    else:
        flat["m"], flat["v"] = m, r * r
    if case["copy"]:
        flat["copy"] = flat["p"].to(TYPES[case["copy"]])
    s = {"case": case, "flat": flat,
         "scale": torch.full((1,), 0.37, device=DEV) if case["scaled"] else None}
    if own:
        # the plan that a training program makes once, of the tensors that it keeps
        import hyper_connection_residual_mixes_gb300 as hcg
        cut = lambda k: [flat[k][a:a + c] for a, c in places]
        if case["states"] == "mxfp8":
            cut_s = lambda k: [flat[k][a // GROUP:-(-(a + c) // GROUP)] for a, c in places]
            m_states, v_states = list(zip(cut("m"), cut_s("m_scales"))), list(zip(cut("v"), cut_s("v_scales")))
        else:
            m_states, v_states = cut("m"), cut("v")
        s["plan"] = hcg.adamw_plan(cut("p"), cut("g"), m_states, v_states, copies=cut("copy") if case["copy"] else None)
    return s


# ------------------------------------------------------------------ 8-bit states
def _power(byte):
    """2^(byte - 127) of scale bytes from 1 on: the byte is the exponent field of the fp32 number."""
    return (byte.int() << 23).view(torch.float32)


def _encode(x, root):
    """fp32 values -> E4M3 codes and UE8M0 scales of groups of 32 (bytes).  The scale is the smallest power of two at or
    above amax / 448, from 2^-126 on; roots of second moments (root) never round to zero."""
    x = x.view(-1, GROUP)
    mant, expo = torch.frexp(x.abs().amax(1) / 448)
    expo = (expo - (mant == 0.5).to(expo.dtype)).clamp(-126, 127)
    expo = torch.where(mant == 0, torch.full_like(expo, -126), expo)
    scales = (expo + 127).to(torch.uint8)
    q = (x / _power(scales)[:, None]).clamp(-448, 448)
    codes = q.to(torch.float8_e4m3fn).view(torch.uint8)
    if root:
        codes = torch.where((codes == 0) & (x > 0), torch.ones_like(codes), codes)
    return codes.reshape(-1), scales


def _decode(codes, scales):
    v = codes.view(torch.float8_e4m3fn).float().view(-1, GROUP)
    return (v * _power(scales)[:, None]).reshape(-1)


# ------------------------------------------------------------------ one pass
def run(state):
    return {"norm": _norm, "norm_backward": _norm_backward, "experts": _experts, "experts_backward": _experts_backward,
            "adamw": _adamw}[state["case"]["op"]](state)


def _norm(s):
    if own:
        import hyper_connection_residual_mixes_gb300 as hcg
        y, mean, rstd = hcg.hc_layer_norm(s["x"], s["w"], s["b"], norm_eps=LN_EPS, return_stats=True)
        return {"y": y, "mean": mean, "rstd": rstd}
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    xc = x - mean
    rstd = (xc.square().mean(1, keepdim=True) + LN_EPS).rsqrt()
    y = (xc * rstd * s["w"].float() + s["b"].float()).to(s["x"].dtype)
    return {"y": y, "mean": mean[:, 0], "rstd": rstd[:, 0]}


def _norm_backward(s):
    if own:
        import hyper_connection_residual_mixes_gb300 as hcg
        return hcg.hc_layer_norm_backward(s["g_y"], s["x"], s["w"], s["mean"], s["rstd"])
    g = s["g_y"].float()
    rstd = s["rstd"][:, None]
    xh = (s["x"].float() - s["mean"][:, None]) * rstd
    wg = g * s["w"].float()
    g_x = rstd * (wg - wg.mean(1, keepdim=True) - xh * (wg * xh).mean(1, keepdim=True))
    return {"g_x": g_x.to(s["g_y"].dtype), "g_norm_w": (g * xh).sum(0), "g_norm_b": g.sum(0)}


def _slots(s):
    """For every row its place in the buffer of E x most rows, one more for the rows behind the last expert's."""
    n, E, most = s["x"].shape[0], s["case"]["experts"], s["most"]
    row = torch.arange(n, device=DEV, dtype=torch.int32)
    e = torch.searchsorted(s["offsets"][1:], row, right=True)
    inside = e < E
    at = e * most + (row - s["offsets"].long()[e.clamp(max=E - 1)])
    return torch.where(inside, at, E * most), inside[:, None]


def _padded(rows, slot, s):
    E, most = s["case"]["experts"], s["most"]
    buf = torch.zeros((E * most + 1, rows.shape[1]), device=DEV)
    buf[slot] = rows.float()
    return buf[:-1].view(E, most, -1)


def _rows(buf, slot, inside):
    buf = buf.reshape(-1, buf.shape[-1])
    return torch.where(inside, buf[slot.clamp(max=buf.shape[0] - 1)], 0.0)


def _experts(s):
    if own:
        import hyper_connection_residual_mixes_gb300 as hcg
        return hcg.hc_grouped_mm(s["x"], s["w"], s["offsets"], transposed=s["case"]["kn"])
    slot, inside = _slots(s)
    w = s["w"].float() if s["case"]["kn"] else s["w"].float().transpose(1, 2)
    return _rows(torch.bmm(_padded(s["x"], slot, s), w), slot, inside).to(s["x"].dtype)


def _experts_backward(s):
    if own:
        import hyper_connection_residual_mixes_gb300 as hcg
        return hcg.hc_grouped_mm_backward(s["g_y"], s["x"], s["w"], s["offsets"], transposed=s["case"]["kn"])
    slot, inside = _slots(s)
    x, g = _padded(s["x"], slot, s), _padded(s["g_y"], slot, s)
    w = s["w"].float().transpose(1, 2) if s["case"]["kn"] else s["w"].float()
    g_w = torch.bmm(x.transpose(1, 2), g) if s["case"]["kn"] else torch.bmm(g.transpose(1, 2), x)
    return {"g_x": _rows(torch.bmm(g, w), slot, inside).to(s["x"].dtype), "g_w": g_w.to(s["x"].dtype)}


def _adam_scalars():
    a = ADAM
    return (1 - a["lr"] * a["weight_decay"], a["lr"] / (1 - a["beta1"] ** a["step"]),
            1 / math.sqrt(1 - a["beta2"] ** a["step"]))


def _adamw(s):
    f = s["flat"]
    if own:
        import hyper_connection_residual_mixes_gb300 as hcg
        a = ADAM
        hcg.hc_adamw_step(s["plan"], lr=a["lr"], step=a["step"], betas=(a["beta1"], a["beta2"]), adam_eps=a["eps"],
                          weight_decay=a["weight_decay"], grad_scale=s["scale"])
        return _adam_outputs(f)
    decay, rate, root = _adam_scalars()
    g = f["g"].float()
    if s["scale"] is not None:
        g = g * s["scale"]
    packed = "m_scales" in f
    m = _decode(f["m"], f["m_scales"]) if packed else f["m"]
    v = _decode(f["v"], f["v_scales"]).square() if packed else f["v"]
    m = m * ADAM["beta1"] + g * (1 - ADAM["beta1"])
    v = v * ADAM["beta2"] + g * g * (1 - ADAM["beta2"])
    r = v.sqrt()
    p = f["p"].float() * decay - m / (r * root + ADAM["eps"]) * rate
    f["p"].copy_(p)
    if "copy" in f:
        f["copy"].copy_(p)
    if packed:
        codes, scales = _encode(m, False)
        f["m"].copy_(codes), f["m_scales"].copy_(scales)
        codes, scales = _encode(r, True)
        f["v"].copy_(codes), f["v_scales"].copy_(scales)
    else:
        f["m"].copy_(m), f["v"].copy_(v)
    return _adam_outputs(f)


def _adam_outputs(f):
    """The updated buffers; 8-bit codes and scales as the numbers that their formats hold."""
    out = {k: f[k] for k in ("p", "copy") if k in f}
    if "m_scales" not in f:
        return {**out, "m": f["m"], "v": f["v"]}
    return {**out, **{k: f[k].view(torch.float8_e4m3fn) for k in ("m", "v")},
            **{k: f[k].view(torch.float8_e8m0fnu) for k in ("m_scales", "v_scales")}}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "norm":
        n, d = case["n"], case["d"]
        return {"bytes": 2 * n * d * SIZE[case["x"]] + 2 * d * SIZE[case["w"]] + 8 * n, "flops": 8 * n * d}
    if case["op"] == "norm_backward":
        n, d = case["n"], case["d"]
        return {"bytes": n * d * (SIZE[case["x"]] + 2 * SIZE[case["g"]]) + d * (SIZE[case["w"]] + 8) + 8 * n, "flops": 14 * n * d}
    if case["op"] in ("experts", "experts_backward"):
        n, E, K, N = case["n"] - case["pad"], case["experts"], case["K"], case["N"]
        back = case["op"] == "experts_backward"
        # experts without a row need no weights: with n rows spread evenly this many have one
        busy = E * (1 - (1 - 1 / E) ** n)
        weights = busy * K * N + (E * K * N if back else 0)
        rows = n * (K + N) + (n * K if back else case["pad"] * N)
        return {"bytes": 2 * (weights + rows), "flops": (4 if back else 2) * n * K * N}
    total = sum(_sizes(case))
    states = 16 if case["states"] == "fp32" else 4 + 4 / GROUP
    each = 2 * SIZE[case["p"]] + SIZE[case["g"]] + states + (2 if case["copy"] else 0)
    return {"bytes": total * each, "flops": 16 * total}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        x = s["x"].double()
        var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
        rstd = 1 / torch.sqrt(var + LN_EPS)
        return {"y": x.sub_(mean).mul_(rstd).mul_(s["w"].double()).add_(s["b"].double()), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if case["op"] == "norm_backward":
        d = case["d"]
        g, rstd = s["g_y"].double(), s["rstd"].double()[:, None]
        xh = (s["x"].double() - s["mean"].double()[:, None]) * rstd
        wg = g * s["w"].double()
        a, c = wg.sum(1, keepdim=True) / d, (wg * xh).sum(1, keepdim=True) / d
        return {"g_x": (wg - a - xh * c) * rstd, "g_norm_w": (g * xh).sum(0), "g_norm_b": g.sum(0)}
    if case["op"] in ("experts", "experts_backward"):
        ends = s["offsets"].tolist()
        x, kn = s["x"], case["kn"]
        back = case["op"] == "experts_backward"
        y = torch.zeros((x.shape[0], case["K"] if back else case["N"]), dtype=torch.float64, device=DEV)
        g_w = torch.zeros(s["w"].shape, dtype=torch.float64, device=DEV) if back else None
        for e in range(case["experts"]):
            a, b = ends[e], ends[e + 1]
            w = s["w"][e].double()
            w = w.t() if kn else w          # [N, K]
            if back:
                ge, xe = s["g_y"][a:b].double(), x[a:b].double()
                y[a:b] = ge @ w
                g_w[e] = xe.t() @ ge if kn else ge.t() @ xe
            else:
                y[a:b] = x[a:b].double() @ w.t()
        return {"g_x": y, "g_w": g_w} if back else y
    f = {k: v for k, v in s["flat"].items()}
    b1, b2 = ADAM["beta1"], ADAM["beta2"]
    g = f["g"].double() * (s["scale"].double() if s["scale"] is not None else 1.0)
    if case["states"] == "mxfp8":
        step = lambda k: torch.pow(2.0, f[k].double() - 127).repeat_interleave(GROUP)
        m = f["m"].view(torch.float8_e4m3fn).double() * step("m_scales")
        v = (f["v"].view(torch.float8_e4m3fn).double() * step("v_scales")) ** 2
    else:
        m, v = f["m"].double(), f["v"].double()
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g ** 2
    mh, vh = m / (1 - b1 ** ADAM["step"]), v / (1 - b2 ** ADAM["step"])
    p = f["p"].double()
    p = p - ADAM["lr"] * (mh / (torch.sqrt(vh) + ADAM["eps"]) + ADAM["weight_decay"] * p)
    out = {"p": p}
    if case["copy"]:
        out["copy"] = p
    if case["states"] == "fp32":
        return {**out, "m": m, "v": v}
    for k, x in (("m", m), ("v", v.sqrt())):
        x = x.view(-1, GROUP)
        top = x.abs().amax(1)
        e = torch.where(top > 0, torch.ceil(torch.log2(top.clamp(min=1e-300) / 448)), -126.0).clamp(-126, 127)
        q = x / torch.pow(2.0, e)[:, None]
        # the nearest number of three mantissa bits (steps of 2^-9 below 2^-6), at most 448
        grain = torch.pow(2.0, torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
        q = (torch.round(q / grain) * grain).clamp(-448, 448)
        if k == "v":
            q = torch.where((q == 0) & (x > 0), 2.0 ** -9, q)
        out[k], out[k + "_scales"] = q.reshape(-1), torch.pow(2.0, e)
    return out
