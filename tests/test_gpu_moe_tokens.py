"""GPU: the experts' layer for a few tokens against its formulas in 64 bits.

Bounds.  With a = p silu(g) u, u = 2^-24 and h the half step of the type that a goes into
the second product with (2^-16 for the two bf16 numbers of bf16 weights, 2^-22 for two fp16 numbers, 2^-11 for one):
 - g and u' are sums of d products in fp32: a lane of the tensor cores adds them in
   some order and may cut off the last bit, then up to 16 warps' sums, each scaled:
   (d + 40) * 2^-23 of S, the sum of their terms' sizes (x is exact in fp16 to 2^-39 of its
   block's largest: below that),
 - silu's slope is at most 1.1: |d a| <= p (1.1 e(g) |u'| + |silu(g)| e(u')) + 4u |a|,
 - y: |d y| <= (half a step of its type) |y| + sum |D| (|d a| + h |a|)
                + (experts x inner + 40) * 2^-23 sum |D| |a|."""
import pytest
import torch

import hyper_connection_residual_mixes_gb300 as hcg
from hyper_connection_residual_mixes_gb300 import _lib
from hyper_connection_residual_mixes_gb300 import build as hc_build

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
T = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    hc_build.build()
    _lib.load()


def _blocks(n):
    return -(-n // 128)


def _value(s):
    return s.double() if s.dtype == torch.float32 else ((s.long() + 896) << 52).view(torch.float64)


def _wide(w, s):
    """A matrix in 64 bits."""
    if s is None:
        return w.double()
    s = _value(s).repeat_interleave(128, 0)[:w.shape[0]].repeat_interleave(128, 1)[:, :w.shape[1]]
    return w.view(torch.float8_e4m3fn).double() * s


def _weights(E, d, inner, x, w, g):
    """Weights of x's type, or codes with scales of kind w."""
    out = {}
    for name, shape, width in (("up", (E, 2, inner, d), d), ("down", (E, d, inner), inner)):
        v = torch.randn(shape, generator=g, device="cuda") * width ** -0.5
        if w == "same":
            out[name], out[name + "_scales"] = v.to(T[x]), None
            continue
        s_shape = (*shape[:-2], _blocks(shape[-2]), _blocks(shape[-1]))
        out[name] = (v * width ** 0.5 * 60).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        if w == "fp32":
            out[name + "_scales"] = torch.exp(torch.randn(s_shape, generator=g, device="cuda")) * width ** -0.5 / 60
        else:
            out[name + "_scales"] = torch.randint(114, 120, s_shape, generator=g, device="cuda", dtype=torch.uint8)
    return out


def _call(x, w, **kw):
    return hcg.hc_moe_tokens(x, w["up"], w["down"], up_scales=w["up_scales"], down_scales=w["down_scales"], **kw)


def _check(y, x, w, ids, p):
    E, _, inner, d = w["up"].shape
    xd = x.double()
    want, room = torch.zeros_like(xd), torch.zeros_like(xd)
    h = 2.0 ** -22 if x.dtype == torch.float16 else 2.0 ** -16 if w["up_scales"] is None else 2.0 ** -11
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        scale = lambda name, *at: None if w[name + "_scales"] is None else w[name + "_scales"][(e, *at)]
        G, V, D = _wide(w["up"][e, 0], scale("up", 0)), _wide(w["up"][e, 1], scale("up", 1)), _wide(w["down"][e], scale("down"))
        g, u = xd[t] @ G.t(), xd[t] @ V.t()
        eg, eu = ((d + 40) * 2.0 ** -23 * (xd[t].abs() @ m.abs().t()) for m in (G, V))
        pe = p[t, j].double()[:, None]
        silu = g / (1 + torch.exp(-g))
        a = pe * silu * u
        da = pe.abs() * (1.1 * eg * (u.abs() + eu) + silu.abs() * eu) + (4 * U + h) * a.abs()
        want.index_add_(0, t, a @ D.t())
        room.index_add_(0, t, (da + (ids.shape[1] * inner + 40) * 2.0 ** -23 * a.abs()) @ D.abs().t())
    assert y.dtype == x.dtype and y.shape == x.shape
    half = torch.finfo(y.dtype).eps / 2
    tiny = torch.finfo(y.dtype).smallest_normal * half
    bad = (y.double() - want).abs() > half * (want.abs() + room) + room + tiny
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())
    return room


def _choice(T_, E, k, g):
    ids = torch.stack([torch.randperm(E, generator=g, device="cuda")[:k] for _ in range(T_)]).int() if T_ else torch.empty((0, k), dtype=torch.int32, device="cuda")
    return ids, torch.rand((T_, k), generator=g, device="cuda")


SIZES = [(1, 1, 1, 16, 16), (1, 8, 2, 1024, 512), (2, 5, 3, 144, 80), (7, 13, 3, 272, 400), (8, 4, 4, 512, 128), (9, 4, 4, 528, 1040),
         (16, 16, 6, 2048, 256), (17, 3, 2, 320, 384), (32, 9, 1, 640, 144), (33, 2, 2, 1072, 336), (37, 13, 3, 1072, 336),
         (64, 1, 1, 256, 272), (64, 31, 8, 400, 208), (64, 300, 16, 48, 32), (3, 1024, 4, 32, 16), (5, 6, 2, 7680, 48), (40, 3, 2, 7696, 32),
         (2, 4, 2, 64, 4112)]


@pytest.mark.parametrize("T_,E,k,d,inner", SIZES)
@pytest.mark.parametrize("x,w", [("bf16", "ue8m0"), ("bf16", "same"), ("fp16", "fp32"), ("fp16", "same")])
def test_given_choice(T_, E, k, d, inner, x, w):
    g = torch.Generator(device="cuda").manual_seed(T_ + E + d)
    xv = torch.randn((T_, d), generator=g, device="cuda").to(T[x])
    wv = _weights(E, d, inner, x, w, g)
    ids, p = _choice(T_, E, k, g)
    y = _call(xv, wv, ids=ids, weights=p)
    _check(y, xv, wv, ids, p)
    assert torch.equal(y, _call(xv, wv, ids=ids, weights=p))


def test_offsets_past_32_bits():
    """Experts whose weights lie more than 2^32 bytes behind the first's."""
    E, d, inner = 66, 8192, 8192
    g = torch.Generator(device="cuda").manual_seed(5)
    codes = lambda *shape: torch.randint(0, 100, shape, generator=g, dtype=torch.uint8, device="cuda") | torch.randint(0, 2, (shape[-1],), generator=g, dtype=torch.uint8, device="cuda") << 7
    scales = lambda *shape: torch.randint(108, 112, shape, generator=g, dtype=torch.uint8, device="cuda")
    w = {"up": codes(E, 2, inner, d), "down": codes(E, d, inner),
         "up_scales": scales(E, 2, inner // 128, d // 128), "down_scales": scales(E, d // 128, inner // 128)}
    x = torch.randn((3, d), generator=g, device="cuda").bfloat16()
    ids = torch.tensor([[65, 0], [64, 65], [33, 1]], dtype=torch.int32, device="cuda")
    p = torch.rand((3, 2), generator=g, device="cuda")
    _check(_call(x, w, ids=ids, weights=p), x, w, ids, p)


def test_scales_that_are_no_tensors():
    g = torch.Generator(device="cuda").manual_seed(1)
    x, w = torch.randn((2, 64), generator=g, device="cuda").bfloat16(), _weights(4, 64, 32, "bf16", "fp32", g)
    lg = torch.randn((2, 4), generator=g, device="cuda")
    with pytest.raises(TypeError, match="up_scales must be"):
        hcg.hc_moe_tokens(x, w["up"], w["down"], logits=lg, top_k=2, up_scales=1.0, down_scales=w["down_scales"])
    with pytest.raises(TypeError, match="down_scales must be"):
        hcg.hc_moe_tokens(x, w["up"], w["down"], logits=lg, top_k=2, up_scales=w["up_scales"], down_scales=1.0)


@pytest.mark.parametrize("T_", list(range(1, 20)) + [31, 32, 33, 47, 48, 49, 63, 64])
def test_every_count_of_tokens(T_):
    """... all of them to one expert, and to the same two of four."""
    g = torch.Generator(device="cuda").manual_seed(T_)
    x = torch.randn((T_, 272), generator=g, device="cuda").bfloat16()
    for w in ("ue8m0", "same"):
        wv = _weights(4, 272, 144, "bf16", w, g)
        for chosen in ([2], [3, 1]):
            ids = torch.tensor(chosen, dtype=torch.int32, device="cuda").repeat(T_, 1)
            p = torch.rand(ids.shape, generator=g, device="cuda")
            _check(_call(x, wv, ids=ids, weights=p), x, wv, ids, p)


def _choose_ref(logits, k, score, normalise, scale):
    """The choice from its rules, in 64 bits, token by token."""
    ids, ps = [], []
    for row in logits.double().tolist():
        order = sorted((i for i, v in enumerate(row) if v > float("-inf")), key=lambda i: (-row[i], i))[:k]
        some = [row[i] for i in order]
        v = torch.tensor(some, dtype=torch.float64)
        if score == "sigmoid":
            p = torch.sigmoid(v)
        else:
            every = torch.tensor([q for q in row if q > float("-inf")], dtype=torch.float64)
            p = torch.exp(v - torch.logsumexp(every, 0)) if every.numel() else v
        if normalise and p.numel():
            p = p / p.sum()
        ids.append(order + [-1] * (k - len(order)))
        ps.append((p * scale).tolist() + [0.0] * (k - len(order)))
    return torch.tensor(ids, dtype=torch.int32).view(-1, k), torch.tensor(ps, dtype=torch.float64).view(-1, k)


@pytest.mark.parametrize("T_,E,k", [(1, 1, 1), (3, 8, 2), (16, 64, 6), (64, 256, 8), (5, 1000, 16), (33, 33, 16)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalise,scale", [(True, 1.0), (False, 2.5)])
def test_choice(T_, E, k, score, normalise, scale):
    g = torch.Generator(device="cuda").manual_seed(T_ * E)
    logits = torch.randn((T_, E), generator=g, device="cuda") * 2
    # equal ones, masked ones, a row with too few left and one with none, both zeros
    logits[0, ::3] = logits[0, 0].clone()
    if T_ > 2:
        logits[1, 1:] = -float("inf")
        logits[2, :] = float("nan")
        logits[T_ - 1, : E // 2] = float("-inf")
    if T_ > 4:
        logits[3, ::2], logits[3, 1::2] = 0.0, -0.0
    x = torch.randn((T_, 64), generator=g, device="cuda").bfloat16()
    w = _weights(E, 64, 32, "bf16", "ue8m0", g)
    y, ids, p = _call(x, w, logits=logits, top_k=k, score=score, normalise=normalise, scale=scale)
    want, weight = _choose_ref(logits.cpu(), k, score, normalise, scale)
    assert ids.dtype == torch.int32 and torch.equal(ids.cpu(), want)
    # (a sum of up to 1,000 exponentials in fp32, each of an argument rounded to 2^-24 of up to 30)
    assert ((p.cpu().double() - weight).abs() <= (64 + 48) * U * weight.abs()).all()
    _check(y, x, w, ids, p)
    assert torch.equal(y, _call(x, w, ids=ids, weights=p))
    if T_ > 2:
        assert (y[2] == 0).all()


def test_places_that_count_for_nothing():
    """Ids out of range, padded tokens, an expert named twice; experts that no token
    chooses may hold anything."""
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((6, 208), generator=g, device="cuda").bfloat16()
    for w in ("ue8m0", "same"):
        wv = _weights(5, 208, 176, "bf16", w, g)
        ids = torch.tensor([[0, 1, -1], [4, 4, 2], [-1, -1, -1], [7, 5, 2], [-2 ** 31, 2 ** 31 - 1, 0], [1, 1, 1]], dtype=torch.int32, device="cuda")
        p = torch.rand((6, 3), generator=g, device="cuda")
        p[2], p[3, 0] = float("nan"), float("inf")
        y = _call(x, wv, ids=ids, weights=p)
        q = torch.where((ids < 0) | (ids >= 5), 0.0, p)
        _check(y, x, wv, ids, q)
        assert (y[2] == 0).all()
        if w == "same":
            wv["up"][3], wv["down"][3] = float("nan"), float("inf")
        else:
            wv["up"][3], wv["down"][3] = 0x7f, 0xff
        assert torch.equal(_call(x, wv, ids=ids, weights=p), y)
    none = torch.full((6, 2), -1, dtype=torch.int32, device="cuda")
    assert (_call(x, wv, ids=none, weights=torch.ones((6, 2), device="cuda")) == 0).all()


@pytest.mark.parametrize("w", ["ue8m0", "same"])
@pytest.mark.parametrize("x", ["bf16", "fp16"])
def test_sizes_of_values(x, w):
    """Tokens and activations far from 1: what is large, small and zero in one batch, a
    block of a token a million times the others."""
    g = torch.Generator(device="cuda").manual_seed(6)
    big = 2.0 ** 20 if x == "bf16" else 2.0 ** 6
    xv = torch.randn((5, 400), generator=g, device="cuda") * torch.tensor([1.0, big, 1 / big, 0.0, 1.0], device="cuda")[:, None]
    xv[4, 128:256] *= 1 / big
    xv = xv.to(T[x])
    wv = _weights(3, 400, 320, x, w, g)
    if w == "same":
        wv["down"] = (wv["down"].float() * 2.0 ** -8).to(T[x])
    ids = torch.tensor([[0, 1], [1, 2], [2, 0], [0, 2], [1, 0]], dtype=torch.int32, device="cuda")
    p = torch.full((5, 2), 0.5 if x == "bf16" else 0.01, device="cuda")
    y = _call(xv, wv, ids=ids, weights=p)
    assert y.isfinite().all()
    _check(y, xv, wv, ids, p)
    assert (y[3] == 0).all()


def test_not_finite():
    """What is not finite in a token spoils that token alone."""
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn((4, 272), generator=g, device="cuda").bfloat16()
    ids = torch.tensor([[0, 1]] * 4, dtype=torch.int32, device="cuda")
    p = torch.rand((4, 2), generator=g, device="cuda")
    for w in ("ue8m0", "same"):
        wv = _weights(2, 272, 144, "bf16", w, g)
        clean = _call(x, wv, ids=ids, weights=p)
        for v in (float("nan"), float("inf")):
            bad = x.clone()
            bad[1, 200] = v
            y = _call(bad, wv, ids=ids, weights=p)
            assert not y[1].isfinite().any()
            for t in (0, 2, 3):
                assert torch.equal(y[t], clean[t])


@pytest.mark.parametrize("T_", [1, 5, 40])
def test_strided_rows(T_):
    g = torch.Generator(device="cuda").manual_seed(9)
    buf = torch.randn((T_, 400 + 48), generator=g, device="cuda").half()
    x = buf[:, 16:416]
    w = _weights(4, 400, 96, "fp16", "fp32", g)
    ids, p = _choice(T_, 4, 2, g)
    out = torch.full((T_, 400 + 7), 9.0, dtype=torch.float16, device="cuda")
    y = _call(x, w, ids=ids, weights=p, y=out[:, 3:403])
    assert y.data_ptr() == out[:, 3:403].data_ptr() and (out[:, :3] == 9).all() and (out[:, 403:] == 9).all()
    assert torch.equal(y, _call(x.contiguous(), w, ids=ids, weights=p))
    one = buf[:1, 16:416].expand(T_, 400)  # the same token for all
    _check(_call(one, w, ids=ids, weights=p), one, w, ids, p)


def test_no_tokens_and_binding():
    g = torch.Generator(device="cuda").manual_seed(9)
    w = _weights(4, 64, 32, "bf16", "same", g)
    x = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    y, ids, p = _call(x, w, logits=torch.zeros((0, 4), device="cuda"), top_k=2)
    assert y.shape == (0, 64) and ids.shape == p.shape == (0, 2)
    x = torch.zeros((2, 64), dtype=torch.bfloat16, device="cuda")
    ids, p = _choice(2, 4, 2, g)
    for kw, err in ((dict(), "either"), (dict(ids=ids, weights=p, logits=torch.zeros((2, 4), device="cuda")), "either"),
                    (dict(logits=torch.zeros((2, 4), device="cuda")), "top_k"),
                    (dict(logits=torch.zeros((2, 4), device="cuda"), top_k=2, score="tanh"), "score"),
                    (dict(logits=torch.zeros((2, 5), device="cuda"), top_k=2), "logits has shape"),
                    (dict(ids=ids, weights=p[:, :1].contiguous()), "weights has shape")):
        with pytest.raises(ValueError, match=err):
            _call(x, w, **kw)
    with pytest.raises(TypeError, match="weights must be"):
        _call(x, w, ids=ids)
    with pytest.raises(ValueError, match="w_down has shape"):
        hcg.hc_moe_tokens(x, w["up"], w["up"][:, 0].contiguous(), ids, p)
    with pytest.raises(ValueError, match="go together"):
        hcg.hc_moe_tokens(x, w["up"].view(torch.uint8)[..., :64].contiguous(), w["down"], ids, p, up_scales=torch.ones((4, 2, 1, 1), device="cuda"))
    with pytest.raises(hcg.HcError, match="UNSUPPORTED"):
        _call(torch.zeros((65, 64), dtype=torch.bfloat16, device="cuda"), w, ids=torch.zeros((65, 1), dtype=torch.int32, device="cuda"),
              weights=torch.ones((65, 1), device="cuda"))
    with pytest.raises(hcg.HcError, match="INVALID"):
        _call(x, w, logits=torch.zeros((2, 4), device="cuda"), top_k=5)


@pytest.mark.parametrize("T_", [2, 20, 50])
def test_streams_and_graph(T_):
    """On a stream of its own; captured, with a workspace that two graphs share, and
    replayed on new tokens and another choice."""
    g = torch.Generator(device="cuda").manual_seed(10)
    w = _weights(6, 528, 272, "bf16", "ue8m0", g)
    new = lambda: (torch.randn((T_, 528), generator=g, device="cuda").bfloat16(), torch.randn((T_, 6), generator=g, device="cuda"))
    inputs = [new() for _ in range(3)]
    want = [_call(x, w, logits=lg, top_k=2) for x, lg in inputs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, ids, p = _call(inputs[0][0], w, logits=inputs[0][1], top_k=2, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want[0][0])
    ws = torch.empty((_lib.load().hc_moe_tokens_workspace_bytes(T_, 2, 272),), dtype=torch.uint8, device="cuda")
    static = [[t.clone() for t in i] for i in inputs[:2]]
    graphs, outs = [], []
    for x, lg in static:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(_call(x, w, logits=lg, top_k=2, workspace=ws))
        graphs.append(graph)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    for o, r in zip(outs, want):
        for a, b in zip(o, r):
            assert torch.equal(a, b)
    for s, t in zip(static[0], inputs[2]):
        s.copy_(t)
    graphs[0].replay()
    graphs[1].replay()
    for a, b in zip(outs[0], want[2]):
        assert torch.equal(a, b)
