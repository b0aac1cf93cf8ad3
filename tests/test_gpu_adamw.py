"""GPU: the AdamW step against its formula in 64 bits, and, with fp32 states, bit
for bit against the same fp32 operations done one after the other in torch.

Bounds.  u = 2^-24.  m and v take two products and a sum of rounded
coefficients: off by at most 4 u (|m beta1| + |g (1 - beta1)|) and 6 u v.  The
step q = m rate / (r root + eps) is off by that over the denominator and by
some 16 u |q| more, p by 4 u |p| and half a step of its type.  An 8-bit code
stands for its value within half a step, 2^-4 of it or 2^-10 of the group's
scale."""
import pytest
import torch

import hyper_connection_residual_mixes_gb300 as hcg
from hyper_connection_residual_mixes_gb300 import _lib
from hyper_connection_residual_mixes_gb300 import build as hc_build

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
T = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
HYPER = dict(lr=2e-3, betas=(0.9, 0.95), adam_eps=1e-8, weight_decay=0.1)


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    hc_build.build()
    _lib.load()


def _power(byte):
    return torch.where(byte == 0, torch.tensor(2.0 ** -127, device="cuda"), (byte.int() << 23).view(torch.float32))


def _groups(x):
    x = x.reshape(-1)
    return torch.nn.functional.pad(x, (0, -x.numel() % 32)).view(-1, 32)


def _decode(state):
    codes, scales = state
    v = _groups(codes).view(torch.float8_e4m3fn).float() * _power(scales)[:, None]
    return v.reshape(-1)[:codes.numel()].view(codes.shape)


def _encode(x, root):
    """The documented rounding with torch operations."""
    g = _groups(x)
    t = g.abs().amax(1) / 448
    bits = t.view(torch.int32)
    byte = ((bits >> 23) + ((bits & 0x7FFFFF) != 0).int()).clamp(1, 254)
    codes = (g / _power(byte)[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    if root:
        codes = torch.where((codes == 0) & (g > 0), torch.ones_like(codes), codes)
    return codes.reshape(-1)[:x.numel()].view(x.shape), byte.to(torch.uint8)


class Case:
    def __init__(self, sizes, p, g, packed=False, copy=None, seed=0, offset=0, zero=False):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def cut(n, dtype, std):
            buf = torch.zeros((n + offset,), dtype=dtype, device="cuda")
            if std:
                size = std * torch.exp(1.5 * torch.randn((n,), generator=gen, device="cuda"))
                buf[offset:] = torch.randn((n,), generator=gen, device="cuda") * size
            return buf[offset:]
        self.p = [cut(n, T[p], 0.02) for n in sizes]
        self.g = [cut(n, T[g], 1e-2) for n in sizes]
        if packed:
            self.m = [_encode(cut(n, torch.float32, 0 if zero else 3e-3), False) for n in sizes]
            self.v = [_encode(cut(n, torch.float32, 0 if zero else 1e-2).abs(), True) for n in sizes]
            if offset:
                odd = lambda t: torch.cat([t.new_zeros(offset), t])[offset:]
                self.m = [(odd(a), odd(b)) for a, b in self.m]
                self.v = [(odd(a), odd(b)) for a, b in self.v]
        else:
            self.m = [cut(n, torch.float32, 0 if zero else 3e-3) for n in sizes]
            self.v = [cut(n, torch.float32, 0 if zero else 1e-2).square_() for n in sizes]
        self.copy = None if copy is None else [cut(n, T[copy], 0) for n in sizes]
        self.packed = packed
        self.plan = hcg.adamw_plan(self.p, self.g, self.m, self.v, self.copy)

    def tensors(self):
        flat = lambda s: [t for pair in s for t in pair] if self.packed else s
        return self.p + flat(self.m) + flat(self.v) + (self.copy or [])

    def expected(self, step, scale=None, lr=None):
        """fp32, op by op: the bits that the step must give; and 64 bits."""
        b1, b2 = HYPER["betas"]
        lr, eps, wd = lr or HYPER["lr"], HYPER["adam_eps"], HYPER["weight_decay"]
        out = []
        for i, (p, g) in enumerate(zip(self.p, self.g)):
            m = _decode(self.m[i]) if self.packed else self.m[i]
            r0 = _decode(self.v[i]) if self.packed else None
            v = r0 * r0 if self.packed else self.v[i]
            e = {}
            gf = g.float() * scale if scale is not None else g.float()
            m32 = m * b1 + gf * (1 - b1)
            v32 = v * b2 + (gf * gf) * (1 - b2)
            r32 = v32.sqrt()
            p32 = p.float() * (1 - lr * wd) - (m32 / (r32 * (1 / (1 - b2 ** step) ** 0.5) + eps)) * (lr / (1 - b1 ** step))
            e["m32"], e["v32"], e["r32"], e["p32"] = m32, v32, r32, p32
            gd = g.double() * (scale.double() if scale is not None else 1.0)
            md, vd = m.double() * b1 + gd * (1 - b1), v.double() * b2 + gd * gd * (1 - b2)
            den = (vd / (1 - b2 ** step)).sqrt() + eps
            q = lr * (md / (1 - b1 ** step)) / den
            pd = p.double() * (1 - lr * wd) - q
            am = m.double().abs() * b1 + gd.abs() * (1 - b1)
            e["m"], e["m_room"] = md, 4 * U * am + 2 ** -149
            e["v"], e["v_room"] = vd, 6 * U * vd + 2 ** -147
            e["p"], e["p_room"] = pd, 16 * U * q.abs() + 4 * U * p.double().abs() + lr / (1 - b1 ** step) / den * e["m_room"]
            out.append(e)
        return out

    def check(self, want, exact_bits=True):
        for i, e in enumerate(want):
            t = self.p[i].dtype
            half = torch.finfo(t).eps / 2
            tiny = torch.finfo(t).smallest_normal * half
            assert ((self.p[i].double() - e["p"]).abs() <= e["p_room"] + half * (e["p"].abs() + e["p_room"]) + tiny).all()
            if self.copy is not None:
                assert torch.equal(self.copy[i], self.p[i].to(self.copy[i].dtype))
            if exact_bits and not self.packed:
                assert torch.equal(self.p[i], e["p32"].to(t))
            if not self.packed:
                assert ((self.m[i].double() - e["m"]).abs() <= e["m_room"]).all()
                assert ((self.v[i].double() - e["v"]).abs() <= e["v_room"]).all()
                if exact_bits:
                    assert torch.equal(self.m[i], e["m32"]) and torch.equal(self.v[i], e["v32"])
                continue
            for state, key, x, room in ((self.m[i], "m32", e["m"], e["m_room"]),
                                        (self.v[i], "r32", e["v"].sqrt(), 4 * U * e["v"].sqrt())):
                scale = _power(state[1]).repeat_interleave(32)[:x.numel()].view(x.shape)
                got = _decode(state).double()
                if key == "r32":   # never rounded to zero
                    assert ((state[0] > 0) == (e["r32"] > 0)).all()
                    room = room + 2 ** -10 * scale.double()
                assert ((got - x).abs() <= room + 2 ** -4 * x.abs() + 2 ** -10 * scale.double()).all()
                top = _groups(x.abs()).amax(1) / 448
                s = _power(state[1]).double()
                assert (top <= s * (1 + 32 * U)).all() and ((top > s / 2 * (1 - 32 * U)) | (state[1] == 1)).all()
                # and the scale byte by the documented rule, but for an amax within the bound of a step
                codes, bytes_ = _encode(e[key], key == "r32")
                near = (torch.frexp(top).mantissa - 0.5).abs() <= 32 * U
                near |= (torch.frexp(top).mantissa - 1.0).abs() <= 32 * U
                assert ((state[1] == bytes_) | near).all()


SIZES = {"one": [1], "few": [3, 24, 1, 31, 32, 33], "blocks": [4096, 4097, 8191, 12288, 100], "many": [7 + 13 * k for k in range(500)],
         "with_empty": [0, 5, 0, 64, 0]}


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("p,g", [("fp32", "fp32"), ("bf16", "fp32"), ("bf16", "bf16"), ("fp16", "fp16"), ("fp16", "fp32")])
@pytest.mark.parametrize("packed", [False, True])
def test_step(sizes, p, g, packed):
    c = Case(SIZES[sizes], p, g, packed, seed=len(sizes))
    for step in (1, 2, 1000) if len(c.p) < 100 else (3,):
        want = c.expected(step)
        hcg.hc_adamw_step(c.plan, step=step, **HYPER)
        c.check(want)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("copy", [None, "bf16", "fp16"])
@pytest.mark.parametrize("offset", [0, 1, 2, 4])
def test_copies_scales_and_offsets(packed, copy, offset):
    """The rounded copy, a gradient scale, and tensors that begin anywhere."""
    c = Case([1000, 4100, 77, 3], "fp32", "fp32", packed, copy, seed=offset, offset=offset)
    scale = torch.tensor([0.37], device="cuda")
    want = c.expected(7, scale)
    hcg.hc_adamw_step(c.plan, step=7, grad_scale=scale, **HYPER)
    c.check(want)


def test_memory_around_the_tensors_stays():
    """Tensors cut out of one buffer at odd places: the gaps keep their values."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    flat = {k: torch.randn((4000,), generator=gen, device="cuda").abs() for k in "pgmv"}
    before = {k: t.clone() for k, t in flat.items()}
    places = [(1, 30), (37, 1), (40, 1000), (1041, 2), (1100, 2500)]
    cut = lambda k: [flat[k][a:a + n] for a, n in places]
    hcg.hc_adamw_step(hcg.adamw_plan(cut("p"), cut("g"), cut("m"), cut("v")), step=3, **HYPER)
    inside = torch.zeros((4000,), dtype=torch.bool, device="cuda")
    for a, n in places:
        inside[a:a + n] = True
    for k in "pmv":
        assert torch.equal(flat[k][~inside], before[k][~inside]) and not torch.equal(flat[k][inside], before[k][inside])
    assert torch.equal(flat["g"], before["g"])


def test_mixed_types_in_one_call():
    """One launch over parameters of several types and both kinds of states."""
    cs = [Case([513, 64], "fp32", "fp32", False, "bf16", 1), Case([700], "bf16", "bf16", True, None, 2), Case([9, 4200], "fp16", "fp32", False, None, 3),
          Case([4096], "fp32", "fp32", True, None, 4)]
    copies = [t for c in cs for t in (c.copy or [None] * len(c.p))]
    plan = hcg.adamw_plan(*[[t for c in cs for t in getattr(c, k)] for k in "pgmv"], copies)
    want = [c.expected(5) for c in cs]
    hcg.hc_adamw_step(plan, step=5, **HYPER)
    for c, w in zip(cs, want):
        c.check(w)


def test_hundreds_of_tensors_of_both_kinds():
    """More tensors than one launch describes, fp32 and 8-bit states in turn."""
    a, b = Case([17 * k + 1 for k in range(460)], "fp32", "fp32", False, None, 1), Case([5 * k + 40 for k in range(460)], "bf16", "bf16", True, None, 2)
    mix = lambda k: [t for two in zip(getattr(a, k), getattr(b, k)) for t in two]
    want = [c.expected(9) for c in (a, b)]
    hcg.hc_adamw_step(hcg.adamw_plan(mix("p"), mix("g"), mix("m"), mix("v")), step=9, **HYPER)
    a.check(want[0])
    b.check(want[1])


@pytest.mark.parametrize("packed", [False, True])
def test_zero_states_and_zero_gradients(packed):
    c = Case([100, 5000], "fp32", "fp32", packed, zero=True)
    for i, p in enumerate(c.p):
        zero = hcg.adamw_state(p, mxfp8=packed)
        for have, new in zip((c.m[i], c.v[i]), zero):
            for a, b in zip(have, new) if packed else ((have, new),):
                a.copy_(b)
    c.g[0].zero_()
    before = [p.clone() for p in c.p]
    want = c.expected(1)
    hcg.hc_adamw_step(c.plan, step=1, **HYPER)
    c.check(want)
    # no gradient: decay alone; the first step of the others is lr |g| / (|g| + eps), both moments' corrections
    # cancelling the rests: 32 u of it, and the roundings of two values of p's size
    assert torch.equal(c.p[0], before[0] * (1 - HYPER["lr"] * HYPER["weight_decay"]))
    move = (before[1].double() * (1 - HYPER["lr"] * HYPER["weight_decay"]) - c.p[1].double()).abs()
    g = c.g[1].double().abs()
    want = HYPER["lr"] * g / (g + HYPER["adam_eps"])
    assert ((move - want).abs() <= 32 * U * want + 4 * U * before[1].double().abs()).all()


def test_small_roots_do_not_become_zero():
    """A group with one huge second moment: the others' roots keep the smallest code, so their weights stay put."""
    c = Case([64], "fp32", "fp32", True, zero=True)
    c.g[0].fill_(1e-6)
    c.g[0][5] = 1e4
    hcg.hc_adamw_step(c.plan, step=1, **HYPER)
    assert (c.v[0][0] > 0).all()
    before = c.p[0].clone()
    c.g[0].zero_()
    hcg.hc_adamw_step(c.plan, step=2, **HYPER)
    assert ((c.p[0] - before).abs() <= 4 * HYPER["lr"]).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("packed", [False, True])
def test_non_finite_gradient_stays_in_its_place(packed, bad):
    c = Case([4200], "fp32", "fp32", packed, seed=3)
    c.g[0][70] = bad
    hcg.hc_adamw_step(c.plan, step=2, **HYPER)
    ok = torch.ones((4200,), dtype=torch.bool, device="cuda")
    ok[70] = False
    assert c.p[0][ok].isfinite().all() and c.p[0][70].isnan()


def test_coefficients_on_the_device_and_graph():
    """lr and step as tensors: a captured step follows them.  expm1 of fp32 puts
    some 4 u on each correction (its argument is rounded once, the function has
    an error of a few units)."""
    sizes = [300, 5000]
    a, b = Case(sizes, "fp32", "fp32", seed=6), Case(sizes, "fp32", "fp32", seed=6)
    lr, step = torch.tensor([1e-3], device="cuda"), torch.tensor([0], dtype=torch.int64, device="cuda")
    kw = {k: v for k, v in HYPER.items() if k != "lr"}
    warm = Case(sizes, "fp32", "fp32", seed=9)
    hcg.hc_adamw_step(warm.plan, lr=lr, step=torch.ones_like(step), **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.add_(1)
        hcg.hc_adamw_step(a.plan, lr=lr, step=step, **kw)
    for t in (1, 2, 3, 40):
        lr.fill_(1e-3 / t), step.fill_(t - 1)
        for x, y in zip(a.tensors(), b.tensors()):
            y.copy_(x)
        for x, y in zip(a.g, b.g):
            x.copy_(torch.randn(x.shape, generator=torch.Generator(device="cuda").manual_seed(t), device="cuda"))
            y.copy_(x)
        graph.replay()
        hcg.hc_adamw_step(b.plan, lr=float(lr), step=t, **kw)
        for x, y, z in zip(a.p, b.p, a.m):
            assert ((x.double() - y.double()).abs() <= 32 * U * (y.double().abs() + 1e-3)).all()
        for x, y in zip(a.m + a.v, b.m + b.v):
            assert torch.equal(x, y)


def test_other_stream_and_moved_storage():
    c, d = Case([5000, 3], "fp32", "fp32", seed=8), Case([5000, 3], "fp32", "fp32", seed=8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    hcg.hc_adamw_step(c.plan, step=1, stream=s, **HYPER)
    s.synchronize()
    hcg.hc_adamw_step(d.plan, step=1, **HYPER)
    assert all(torch.equal(x, y) for x, y in zip(c.tensors(), d.tensors()))
    old = c.p[0].clone()
    c.p[0].data = c.p[0].clone()          # new storage: the next step follows it
    c.g[1].data = c.g[1].clone()
    hcg.hc_adamw_step(c.plan, step=2, **HYPER)
    hcg.hc_adamw_step(d.plan, step=2, **HYPER)
    assert all(torch.equal(x, y) for x, y in zip(c.tensors(), d.tensors())) and not torch.equal(c.p[0], old)
    c.p[0].data = torch.zeros((7,), device="cuda")
    with pytest.raises(ValueError, match="changed"):
        hcg.hc_adamw_step(c.plan, step=3, **HYPER)


def test_same_tensor_twice_is_refused():
    c = Case([100], "fp32", "fp32")
    plan = hcg.adamw_plan(c.p * 2, c.g * 2, c.m * 2, c.v * 2)
    with pytest.raises(hcg.HcError, match="ALIAS"):
        hcg.hc_adamw_step(plan, step=1, **HYPER)
    shared = hcg.adamw_plan([c.p[0], torch.zeros_like(c.p[0])], c.g * 2, [c.m[0], torch.zeros_like(c.m[0])],
                            [c.v[0], torch.zeros_like(c.v[0])])
    hcg.hc_adamw_step(shared, step=1, **HYPER)   # one gradient for two parameters is fine


@pytest.mark.parametrize("packed", [False, True])
def test_tensors_changed_in_place_are_refused(packed):
    """A shorter, a transposed and another type's tensor at the same address; put
    back, the step gives what an untouched one gives."""
    c, d = Case([4096, 300], "fp32", "fp32", packed, seed=12), Case([4096, 300], "fp32", "fp32", packed, seed=12)
    hcg.hc_adamw_step(c.plan, step=1, **HYPER)
    hcg.hc_adamw_step(d.plan, step=1, **HYPER)
    before = [t.clone() for t in c.tensors()]
    m = c.m[0][0] if packed else c.m[0]
    for t in (c.p[0], c.g[0], m):
        old = t.data
        for change in (old[:10], old.view(64, 64), old.view(torch.int8 if t.dtype == torch.uint8 else torch.int32), old[::2]):
            t.data = change
            with pytest.raises(ValueError, match="changed"):
                hcg.hc_adamw_step(c.plan, step=2, **HYPER)
        t.data = old
    assert all(torch.equal(a, b) for a, b in zip(c.tensors(), before))
    hcg.hc_adamw_step(c.plan, step=2, **HYPER)
    hcg.hc_adamw_step(d.plan, step=2, **HYPER)
    assert all(torch.equal(a, b) for a, b in zip(c.tensors(), d.tensors()))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("p,g,offset", [("fp32", "fp32", 0), ("bf16", "bf16", 0), ("fp32", "fp32", 1)])
def test_non_finite_gradient_in_the_states(p, g, offset, packed, bad):
    """A NaN stays in both moments of its value and nowhere else; an infinite
    gradient spoils the 8-bit states of its group at the most."""
    c, d = Case([4200], p, g, packed, seed=3, offset=offset), Case([4200], p, g, packed, seed=3, offset=offset)
    c.g[0][70] = bad
    hcg.hc_adamw_step(c.plan, step=2, **HYPER)
    hcg.hc_adamw_step(d.plan, step=2, **HYPER)
    other = torch.ones((4200,), dtype=torch.bool, device="cuda")
    other[70] = False
    assert c.p[0][70].isnan() and torch.equal(c.p[0][other], d.p[0][other])
    group = other.clone()
    group[64:96] = False
    for x, y in ((c.m[0], d.m[0]), (c.v[0], d.v[0])):
        got, want = (_decode(x), _decode(y)) if packed else (x, y)
        assert torch.equal(got[group if packed else other], want[group if packed else other])
        if bad != bad:
            assert got[70].isnan() and got[other].isfinite().all()
        elif not packed:
            assert got[70].isinf()
    if packed and bad != bad:   # its group's scales are those of the other values
        for x, y in ((c.m[0], d.m[0]), (c.v[0], d.v[0])):
            top = _decode(y)[64:96][other[64:96]].abs().max()
            assert (_decode(x)[64:96][other[64:96]].abs().max() - top).abs() <= 2.0 ** -3 * top


def test_groups_of_nothing_but_nan():
    c = Case([128], "fp32", "fp32", True, seed=4)
    c.g[0][32:64] = float("nan")
    hcg.hc_adamw_step(c.plan, step=2, **HYPER)
    for s in (c.m[0], c.v[0]):
        v = _decode(s)
        assert v[32:64].isnan().all() and v[:32].isfinite().all() and v[64:].isfinite().all()


@pytest.mark.parametrize("eps", [0.0, 1e-30])
@pytest.mark.parametrize("p", ["fp32", "bf16"])
def test_roots_of_tiny_second_moments(p, eps):
    """8-bit states, gradients whose squares are subnormal in fp32: the step is lr
    g / (|g| + eps) like any first step.  A sum of subnormal terms is off by half a
    unit of 2^-149 for each of its (at most three) roundings: relative to v, and
    half of that in the root."""
    gen = torch.Generator(device="cuda").manual_seed(21)
    c = Case([2000], p, "fp32", True, seed=5, zero=True)
    size = torch.exp2(-66 + 3 * torch.rand((2000,), generator=gen, device="cuda"))
    c.g[0].copy_(torch.where(torch.rand((2000,), generator=gen, device="cuda") < 0.5, -size, size))
    b1, b2 = HYPER["betas"]
    for step in (1, 2, 3):
        m0, r0, p0, g = _decode(c.m[0]).double(), _decode(c.v[0]).double(), c.p[0].double(), c.g[0].double()
        hcg.hc_adamw_step(c.plan, step=step, **{**HYPER, "adam_eps": eps})
        m, v = m0 * b1 + g * (1 - b1), r0 * r0 * b2 + g * g * (1 - b2)
        am = m0.abs() * b1 + g.abs() * (1 - b1)
        rate = HYPER["lr"] / (1 - b1 ** step) / ((v / (1 - b2 ** step)).sqrt() + eps)
        want = p0 * (1 - HYPER["lr"] * HYPER["weight_decay"]) - rate * m
        room = rate * am * (16 * U + 4 * 2.0 ** -150 / v) + 4 * U * p0.abs()
        half = torch.finfo(c.p[0].dtype).eps / 2
        assert ((c.p[0].double() - want).abs() <= room + half * (want.abs() + room)).all()
        assert ((c.v[0][0] > 0) & (c.v[0][0] < 0x7F)).all()
        scale = _power(c.v[0][1]).double().repeat_interleave(32)[:2000]
        root = v.sqrt()
        assert ((_decode(c.v[0]).double() - root).abs() <= (2.0 ** -4 + 2.0 ** -150 / v) * root + 2.0 ** -9 * scale).all()
