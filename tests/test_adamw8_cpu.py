"""AdamW on 8-bit moments without a GPU: the reference's codes against closed
forms and its rounding against its mean, the planner's rows of that kind, and
every refusal of the entry points and of the binding."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import adamw8_ref as R

mo = pytest.importorskip("matrix_orthogonalizing_optimizer_amd")

E_ARG, E_SHAPE, E_DTYPE, E_METHOD, E_WORKSPACE = -1, -2, -3, -4, -5
P = 1 << 20  # an aligned address that is never followed: the calls are refused first


def _lib():
    try:
        return mo.lib()
    except RuntimeError as e:
        pytest.skip(str(e))


def test_codes_closed_forms():
    # 1.0 has bits 127 << 23: 1016 units of 2^20; a block whose largest is 1 has offset 1016 - K
    x = np.array([1.0, 0.5, -0.25, 0.0, -0.0], dtype=np.float32)
    for moment, top in ((0, 127), (1, 255)):
        c, o = R.encode(np.abs(x) if moment else x, 5, moment)
        assert o.tolist() == [1016 - top]
        assert c[:3].tolist() == [top, top - 8, top - 16 + (0 if moment else 128)]
        assert R.decode(c, o, moment).tolist() == ([1.0, 0.5, 0.25, 0, 0] if moment else [1.0, 0.5, -0.25, 0, 0])
    # the largest value is rounded up in the offset, so it fits whichever way it goes
    c, o = R.encode(np.array([1.01], dtype=np.float32), 0, 0)
    assert o.tolist() == [1017 - 127] and c[0] in (126, 127)
    # zeros, and values so small that the offset is held at 0
    c, o = R.encode(np.zeros(300, dtype=np.float32), 3, 0)
    assert not c.any() and o.tolist() == [0, 0]
    tiny = np.array([2.0 ** -129, 1e-45, 0.0], dtype=np.float32)
    c, o = R.encode(tiny, 3, 1)
    assert o.tolist() == [0] and c.tolist() == [1, 1, 0]  # 2^-129 is one unit
    assert R.decode(c, o, 1).tolist() == [2.0 ** -129, 2.0 ** -129, 0.0]
    # NaN and infinity are kept
    c, o = R.encode(np.array([np.inf, np.nan, -np.inf, 1.0], dtype=np.float32), 3, 0)
    d = R.decode(c, o, 0)
    assert d[0] == np.inf and np.isnan(d[1]) and d[2] == -np.inf and abs(d[3]) < 2.0 ** 113


@pytest.mark.parametrize("moment", [0, 1])
def test_rounding_keeps_the_mean(moment):
    """Over many steps the codes' mean is the value (m everywhere, v down to its
    smallest code): 4000 draws of a variable whose steps are at most 1/8 of
    the value leave a standard error of at most 1/8 / 2 / sqrt(4000) = 1e-3 of
    it (5 of them allowed); the 16-bit granularity adds 2^-16 of a step."""
    rng = np.random.default_rng(1)
    x = (np.exp(rng.uniform(-6, 0, 64)) * (1 if moment else rng.choice([-1, 1], 64))).astype(np.float32)
    x[0] = 1.0
    n = 4000
    rand = np.stack([R.random_bits(64, t, moment) for t in range(n)])
    got = np.mean([R.decode(*R.encode(x, 0, moment, rand=r), moment) for r in rand], axis=0)
    assert (np.abs(got - x) <= 5e-3 * np.abs(x)).all()
    # a value under the smallest code: lo with probability x / lo, or lo
    y = np.array([1.0, 2.0 ** -17 if moment == 0 else 2.0 ** -40], dtype=np.float32)
    c = np.array([R.encode(y, 0, moment, rand=r[:2])[0][1] for r in rand])
    if moment:
        assert (c == 1).all()
    else:
        lo = float(R.from_bits((1016 - 127 + 1) << 20))
        p = 2.0 ** -17 / lo
        assert set(c) <= {0, 1} and abs(c.mean() - p) <= 5 * np.sqrt(p * (1 - p) / n)


def test_random_bits_depend_on_step_and_index():
    a = R.random_bits(512, 1, 0)
    assert len(set(a.tolist())) > 480 and not np.array_equal(a, R.random_bits(512, 2, 0))
    assert np.array_equal(a[100:], R.random_bits(412, 1, 0, first=100))
    # far elements: the group's number passes 32 bits
    assert not np.array_equal(a[:8], R.random_bits(8, 1, 0, first=1 << 34))
    assert not np.array_equal(a, R.random_bits(512, 1 + (1 << 32), 0))


def test_a_step_of_the_reference_is_adamw():
    rng = np.random.default_rng(2)
    g, m = rng.standard_normal(50), rng.standard_normal(50)
    v = rng.random(50)
    m2, v2 = R.moments(g, m, v, 0.9, 0.95)
    assert np.allclose(m2, 0.9 * m + 0.1 * g, rtol=1e-5, atol=1e-6) and np.allclose(v2, 0.95 * v + 0.05 * g * g, rtol=1e-5)
    w = R.weights(np.ones(50), m2, v2, 1e-3, 0.9, 0.95, 1e-8, 0.1, 3)
    mh, vh = np.float64(m2) / (1 - 0.9 ** 3), np.float64(v2) / (1 - 0.95 ** 3)
    assert np.allclose(w, 1 - 1e-4 - 1e-3 * mh / np.sqrt(vh), rtol=1e-6)


def test_plan_takes_the_kind():
    _lib()
    table = [(3, 1, 5, 7, 0, 0), (0, 1, 64, 32, 0, 0), (3, 0, 0, 4, 0, 0), (1, 1, 1, 8, 0, 0)]
    plan = mo.muon_plan_create(table)
    assert len(mo.muon_plan_units(plan)) == 1
    # they need no workspace
    assert mo.muon_plan_workspace_bytes(mo.muon_plan_create([(3, 1, 5000, 700, 0, 0)])) == 0
    for row, status in (((3, 1, 4, 4, 2, 0), E_SHAPE), ((3, 2, 4, 4, 0, 0), E_DTYPE), ((3, 1, -4, 4, 0, 0), E_SHAPE),
                        ((3, 1, 1 << 21, 1 << 20, 0, 0), E_SHAPE), ((2, 1, 4, 4, 0, 0), E_ARG), ((4, 1, 4, 4, 0, 0), E_ARG)):
        with pytest.raises(mo.MuonError) as e:
            mo.muon_plan_create([row])
        assert e.value.status == status, row


def test_state_bytes():
    L = _lib()
    for n in (0, 1, 255, 256, 257, 2048, 2049, 10 ** 6 + 1, 1 << 40):
        assert mo.muon_adamw8_state_bytes(n) == R.state_bytes(n)
    b = ctypes.c_size_t()
    assert L.muon_adamw8_state_bytes(-1, ctypes.byref(b)) == E_SHAPE
    assert L.muon_adamw8_state_bytes((1 << 40) + 1, ctypes.byref(b)) == E_SHAPE
    assert L.muon_adamw8_state_bytes(5, None) == E_ARG


def test_step_refusals():
    """A step over one such parameter, each argument wrong in turn: refused before any launch."""
    L = _lib()
    from matrix_orthogonalizing_optimizer_amd import _lib as B
    plan = mo.muon_plan_create([(3, 1, 5, 7, 0, 0)])

    def step(hp=None, n=1, **kw):
        d = dict(param=P, grad=P, momentum=None, exp_avg=P, exp_avg_sq=P, update_out=None)
        d.update(kw)
        arr = (B.MuonParamPtrs * 1)(B.MuonParamPtrs(*d.values()))
        return L.muon_step(plan.handle, arr, n, ctypes.byref(mo.make_hparams(**(hp or {}))), None, 0, None)

    for kw in (dict(param=None), dict(grad=None), dict(exp_avg=None), dict(exp_avg_sq=None), dict(param=P + 1),
               dict(grad=P + 1), dict(exp_avg=P + 2), dict(exp_avg_sq=P + 1)):
        assert step(**kw) == E_ARG, kw
    for hp in (dict(adam_beta1=1.0), dict(adam_beta2=1.0), dict(adam_beta1=-0.1), dict(adam_beta2=-0.1),
               dict(adam_beta1=float("nan")), dict(adam_step=0), dict(adam_lr=float("inf")), dict(adam_eps=float("nan"))):
        assert step(hp) == E_ARG, hp
    assert step(n=0) == -7
    # an empty parameter needs no buffers
    empty = mo.muon_plan_create([(3, 1, 0, 7, 0, 0)])
    arr = (B.MuonParamPtrs * 1)()
    assert L.muon_step(empty.handle, arr, 1, ctypes.byref(mo.make_hparams()), None, 0, None) == 0


def test_conversion_refusals():
    L = _lib()
    for args, status in (((P, 5, 2, 0, P, None), E_METHOD), ((P, -1, 0, 0, P, None), E_SHAPE),
                         ((P, (1 << 40) + 1, 0, 0, P, None), E_SHAPE), ((None, 5, 0, 0, P, None), E_ARG),
                         ((P + 2, 5, 0, 0, P, None), E_ARG), ((P, 5, 0, 0, None, None), E_ARG),
                         ((P, 5, 1, 0, P + 1, None), E_ARG), ((None, 0, 0, 0, None, None), 0)):
        assert L.muon_adamw8_pack(*args) == status, args
    for args, status in (((P, 5, -1, P, None), E_METHOD), ((P, -1, 0, P, None), E_SHAPE), ((None, 5, 0, P, None), E_ARG),
                         ((P, 5, 0, None, None), E_ARG), ((P, 5, 0, P + 2, None), E_ARG), ((None, 0, 1, None, None), 0)):
        assert L.muon_adamw8_unpack(*args) == status, args


def test_binding_refusals():
    _lib()
    plan = mo.muon_plan_create([(3, 1, 5, 7, 0, 0)])
    w, g, hp = torch.zeros(5, 7, dtype=torch.bfloat16), torch.zeros(5, 7, dtype=torch.bfloat16), mo.make_hparams()
    s = torch.zeros(mo.muon_adamw8_state_bytes(35), dtype=torch.uint8)
    with pytest.raises(ValueError):  # host tensors
        mo.muon_step(plan, [w], [g], [None], [s], [s], hp, None)
    from matrix_orthogonalizing_optimizer_amd import _lib as B
    for bad in (s[:-1], s.view(torch.int8), torch.zeros(2 * s.numel(), dtype=torch.uint8)[::2],
                torch.zeros(s.numel() + 1, dtype=torch.uint8)[1:]):
        with pytest.raises(ValueError):
            B._check_moment8("m", bad, 35, None)
    for x in (torch.zeros(5, dtype=torch.float64), torch.zeros(5, 4)[:, :2], torch.zeros(5)):
        with pytest.raises(ValueError):
            mo.muon_adamw8_pack(x)
        with pytest.raises(ValueError):
            mo.muon_adamw8_unpack(s, x)
