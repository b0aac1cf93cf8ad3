"""The AdamW step on the host: refusals of the C entry point (before any CUDA
call; the pointers are not allocations) and of the binding."""
import pytest
import torch

import hyper_connection_residual_mixes_gb300 as hcg
from hyper_connection_residual_mixes_gb300 import _lib, sublayer
from hyper_connection_residual_mixes_gb300 import build as hc_build

F32, BF16, F16 = 0, 1, 2
A, STEP = 0x1000000, 0x1000000


@pytest.fixture(scope="module", autouse=True)
def _built():
    hc_build.build()


def _tensor(k=0, **kw):
    at = A + 16 * k * STEP
    a = dict(p=at, g=at + STEP, m=at + 2 * STEP, v=at + 3 * STEP, m_scales=None, v_scales=None, p_copy=None, numel=1000,
             p_type=F32, g_type=F32, copy_type=0)
    a.update(kw)
    return _lib.AdamwTensor(**a)


def _step(described, **kw):
    a = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, wd=0.1, step=1, lr_dev=None, step_dev=None, scale=None, stream=None)
    a.update(kw)
    arr = (_lib.AdamwTensor * max(1, len(described)))(*described)
    count = a.pop("count", len(described))
    return _lib.raw("hc_adamw_step", a.pop("tensors", arr), count, *a.values())


@pytest.mark.parametrize("kw,expect", [
    (dict(lr=-1.0), 1), (dict(lr=float("nan")), 1), (dict(beta1=1.0), 1), (dict(beta1=-0.1), 1), (dict(beta2=float("nan")), 1),
    (dict(eps=-1e-8), 1), (dict(wd=float("inf")), 1), (dict(step=0), 1), (dict(count=-1), 1), (dict(tensors=None, count=1), 1),
    (dict(count=0), 0), (dict(lr_dev=A + 2), 3), (dict(step_dev=A + 4), 3), (dict(scale=A + 1), 3),
    (dict(lr_dev=A), 4), (dict(scale=A + 2 * STEP + 8), 4),   # a coefficient inside what the step writes
])
def test_scalar_refusals(kw, expect):
    assert _step([_tensor()], **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(numel=-1), 1), (dict(p_type=3), 1), (dict(g_type=-1), 1), (dict(g_type=BF16), 2), (dict(p_type=BF16, g_type=F16), 2),
    (dict(p=None), 1), (dict(g=None), 1), (dict(m=None), 1), (dict(v=None), 1),
    (dict(m_scales=A + 5 * STEP), 1),                                            # scales come together
    (dict(p_copy=A + 6 * STEP, copy_type=F32), 2), (dict(p_copy=A + 6 * STEP, copy_type=BF16, p_type=BF16), 2),
    (dict(p=A + 2), 3), (dict(g=A + STEP + 2), 3), (dict(m=A + 2 * STEP + 1), 3), (dict(p_copy=A + 6 * STEP + 1, copy_type=BF16), 3),
    (dict(g=A), 4), (dict(m=A + 3996), 4), (dict(v=A + 2 * STEP), 4), (dict(p_copy=A + 100, copy_type=BF16), 4),
    (dict(m_scales=A + 5 * STEP, v_scales=A + 5 * STEP + 31), 4),
    (dict(numel=0, p=None, g=None), None),
])
def test_tensor_refusals(kw, expect):
    if expect is None:   # an empty tensor is described by its size alone; with no other there is nothing to launch
        assert _step([_tensor(**kw)]) == 0
    else:
        assert _step([_tensor(**kw)]) == expect
        assert _step([_tensor(1), _tensor(**kw), _tensor(2)]) == expect


def test_tensors_that_share_memory():
    assert _step([_tensor(), _tensor()]) == 4                                     # the same tensor twice
    assert _step([_tensor(), _tensor(1, p=A + 3999 - 3)]) == 4                    # its last value and another's first
    assert _step([_tensor(k) for k in range(40)] + [_tensor(50, g=A + 16 * 7 * STEP)]) == 4   # a gradient that is a parameter
    assert _step([_tensor(k) for k in range(40)] + [_tensor(17)]) == 4


def test_binding_refusals():
    p = torch.zeros(4)
    m, v = hcg.adamw_state(p)
    with pytest.raises(ValueError, match="empty"):
        hcg.adamw_plan([], [], [], [])
    with pytest.raises(ValueError, match="one entry"):
        hcg.adamw_plan([p], [], [m], [v])
    with pytest.raises(TypeError, match="params"):
        hcg.adamw_plan([p.double()], [p], [m], [v])
    with pytest.raises(TypeError, match="one kind"):
        hcg.adamw_plan([p], [p], [m], [hcg.adamw_state(p, mxfp8=True)[1]])
    with pytest.raises(TypeError, match="copies"):
        hcg.adamw_plan([p.bfloat16()], [p.bfloat16()], [m], [v], [p.bfloat16()])
    with pytest.raises(ValueError, match="CUDA"):
        hcg.adamw_plan([p], [p], [m], [v])
    with pytest.raises(TypeError, match="adamw_plan"):
        hcg.hc_adamw_step([p], 1e-3, 1)
    codes, scales = hcg.adamw_state(torch.zeros(5, 13), mxfp8=True)[0]
    assert codes.shape == (5, 13) and scales.shape == (3,) and codes.dtype == scales.dtype == torch.uint8


@pytest.fixture
def host_plans(monkeypatch):
    """adamw_plan on host tensors: its descriptions can be looked at without a device."""
    def plan(*lists):
        with monkeypatch.context() as m:
            m.setattr(sublayer, "_tensor", lambda t, *a, **kw: t)
            return hcg.adamw_plan(*lists)
    return plan


def _parameters(sizes=((8, 12), (64,), (3, 5, 7))):
    p, g = [torch.zeros(s) for s in sizes], [torch.ones(s) for s in sizes]
    states = [hcg.adamw_state(t) for t in p]
    return p, g, [s[0] for s in states], [s[1] for s in states]


def _described(plan, lists):
    plan._describe()
    return all(getattr(d, k) == t.data_ptr() for k, ts in zip("pgmv", lists) for d, t in zip(plan._array, ts)) and all(
        d.numel == t.numel() and d.p_type == d.g_type == F32 for d, t in zip(plan._array, lists[0]))


def test_refused_change_leaves_the_description_whole(host_plans):
    """One tensor moved, another no longer of its size: refused; with both put back
    the description holds the old places again, not the first one's for a while."""
    lists = _parameters()
    plan = host_plans(*lists)
    assert _described(plan, lists)
    old, other = lists[0][0].data, lists[0][1].data
    lists[0][0].data, lists[0][1].data = torch.zeros(8, 12), torch.zeros(7)
    with pytest.raises(ValueError, match="changed"):
        plan._describe()
    lists[0][0].data, lists[0][1].data = old, other
    assert _described(plan, lists)


CHANGES = {
    "shorter": lambda t: t[:3], "another order": lambda t: t.t(), "another type": lambda t: t.view(torch.int32),
    "another shape": lambda t: t.view(12, 8), "one value for all": lambda t: t[:1, :1].expand(8, 12),
    "another type of half the size": lambda t: t.view(torch.bfloat16)[:, :12],
    "rows over one another": lambda t: t.as_strided((8, 12), (8, 1)),
}


@pytest.mark.parametrize("which", range(4))
@pytest.mark.parametrize("change", CHANGES)
@pytest.mark.parametrize("moved", [False, True])
def test_changed_tensors_are_refused(host_plans, which, change, moved):
    """Also where the tensor still begins at the same place."""
    lists = _parameters()
    plan = host_plans(*lists)
    assert _described(plan, lists)
    t = lists[which][0]
    old = t.data
    t.data = CHANGES[change](old.clone() if moved else old)
    assert moved or t.data_ptr() == old.data_ptr()
    with pytest.raises(ValueError, match=r"%s of tensor 0 has changed" % "pgmv"[which]):
        plan._describe()
    t.data = old
    assert _described(plan, lists)
    t.data = old.clone()           # moved alone: followed
    assert _described(plan, lists)


@pytest.mark.parametrize("k", range(3))
def test_changed_copies_and_codes_are_refused(host_plans, k):
    p, g = [torch.zeros(8, 12)], [torch.ones(8, 12)]
    m, v = hcg.adamw_state(p[0], mxfp8=True)
    copy = torch.zeros(8, 12, dtype=torch.bfloat16)
    plan = host_plans(p, g, [m], [v], [copy])
    plan._describe()
    t = (m[0], v[1], copy)[k]
    old = t.data
    for change in (old[:1], old.view(torch.int16 if t is copy else torch.int8), old.view(*old.shape[::-1], 1)):
        t.data = change
        with pytest.raises(ValueError, match="changed"):
            plan._describe()
    t.data = old
    plan._describe()


def test_snapshots(monkeypatch):
    """Equal for the same tensors, different after any change; refused for what is no list of tensors."""
    f = _lib.snapshot()
    ts = [torch.zeros(6, 4), torch.tensor(1.0), torch.zeros(0, 3), torch.nn.Parameter(torch.zeros(5))]
    base = f(ts)
    assert f(ts) == base and f([t.detach() for t in ts]) == base and f([]) == b"" and f(ts[:3]) != base
    for change in (lambda t: t[:5], lambda t: t.view(4, 6), lambda t: t.t(), lambda t: t.view(torch.int32), lambda t: t[:, :3], lambda t: t.clone(),
                   lambda t: t.as_strided((6, 4), (2, 1)), lambda t: t.unsqueeze(0)):
        assert f([change(ts[0])] + ts[1:]) != base
    for bad in (None, 3, tuple(ts), [ts[0], 3], [ts]):
        with pytest.raises(TypeError, match="list of tensors"):
            f(bad)
    from hyper_connection_residual_mixes_gb300 import _tensors
    monkeypatch.setattr(_tensors, "torch_version", "0.0")
    with pytest.raises(RuntimeError, match="built for torch 0.0"):
        _lib.snapshot()
