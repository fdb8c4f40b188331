"""The products grouped by expert without a GPU: the reference's gradients
against differences, and every refusal of the C entry points and of the
binding (all of them come before any launch)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import experts_ref as R

mo = pytest.importorskip("matrix_orthogonalizing_optimizer_amd")

E_ARG, E_SHAPE, E_DTYPE, E_METHOD, E_WORKSPACE = -1, -2, -3, -4, -5
P = 1 << 20  # an aligned address that is never followed: the calls are refused first


def _lib():
    try:
        return mo.lib()
    except RuntimeError as e:
        pytest.skip(str(e))


def test_reference_gradients_match_differences():
    rng = np.random.default_rng(1)
    off = [1, 3, 3, 7]
    x, w, dy = rng.standard_normal((8, 5)), rng.standard_normal((3, 4, 5)), rng.standard_normal((8, 4))
    nobody = np.zeros((8, 4))
    loss = lambda x_, w_: (R.forward(x_, w_, off, nobody) * dy).sum()
    dx, dw = R.input_grad(dy, w, off, np.zeros((8, 5))), R.weight_grad(dy, x, off)
    assert not dw[1].any() and not dx[0].any() and not dx[7].any()
    h = 1e-6
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        assert math.isclose((loss(x + e, w) - loss(x - e, w)) / (2 * h), dx[i], rel_tol=1e-6, abs_tol=1e-8)
    for i in np.ndindex(w.shape):
        e = np.zeros_like(w)
        e[i] = h
        assert math.isclose((loss(x, w + e) - loss(x, w - e)) / (2 * h), dw[i], rel_tol=1e-6, abs_tol=1e-8)


F = dict(x=P, ldx=20, w=P, ldw=20, stride=120, offsets=P, rows=9, experts=3, out=6, in_=20, dtype=1, y=P, ldy=6, y_dtype=1,
         workspace=P, workspace_bytes=1 << 24, stream=None)
X = dict(dy=P, lddy=6, w=P, ldw=20, stride=120, offsets=P, rows=9, experts=3, out=6, in_=20, dtype=1, dx=P, lddx=20,
         dx_dtype=1, workspace=P, workspace_bytes=1 << 24, stream=None)
W = dict(dy=P, lddy=6, x=P, ldx=20, offsets=P, rows=9, experts=3, out=6, in_=20, dtype=1, dw=P, lddw=20, stride=120,
         dw_dtype=1, accumulate=0, workspace=P, workspace_bytes=1 << 24, stream=None)
COMMON_SHAPE = [dict(rows=-1), dict(experts=-1), dict(out=-1), dict(in_=-1), dict(rows=(1 << 30) + 1),
                dict(experts=(1 << 16) + 1, stride=1 << 20), dict(stride=119), dict(stride=0), dict(stride=-120),
                dict(stride=(1 << 42) + 8)]
REFUSED = [
    ("muon_experts_forward", F, E_DTYPE, [dict(dtype=2), dict(y_dtype=-1)]),
    ("muon_experts_forward", F, E_SHAPE, COMMON_SHAPE + [dict(ldx=19), dict(ldw=19), dict(ldy=5), dict(ldx=(1 << 21) + 8),
                                                         dict(ldw=(1 << 21) + 8, stride=1 << 30), dict(ldy=(1 << 21) + 1),
                                                         dict(rows=1 << 30, out=1 << 20, ldy=1 << 20, stride=1 << 40)]),
    ("muon_experts_forward", F, E_ARG, [dict(x=None), dict(w=None), dict(offsets=None), dict(y=None), dict(x=P + 1),
                                        dict(w=P + 1), dict(offsets=P + 2), dict(y=P + 1), dict(y=P + 2, y_dtype=0),
                                        dict(x=P + 2, dtype=0), dict(w=P + 2, dtype=0)]),
    ("muon_experts_input_grad", X, E_DTYPE, [dict(dtype=-1), dict(dx_dtype=3)]),
    ("muon_experts_input_grad", X, E_SHAPE, COMMON_SHAPE + [dict(lddy=5), dict(ldw=19), dict(lddx=19)]),
    ("muon_experts_input_grad", X, E_ARG, [dict(dy=None), dict(w=None), dict(offsets=None), dict(dx=None), dict(dy=P + 1),
                                           dict(w=P + 1), dict(offsets=P + 1), dict(dx=P + 1)]),
    ("muon_experts_weight_grad", W, E_DTYPE, [dict(dtype=9), dict(dw_dtype=2)]),
    ("muon_experts_weight_grad", W, E_SHAPE, COMMON_SHAPE + [dict(lddy=5), dict(ldx=19), dict(lddw=19),
                                                             dict(experts=1 << 16, out=16384, lddy=16384, stride=1 << 19)]),
    ("muon_experts_weight_grad", W, E_ARG, [dict(dy=None), dict(x=None), dict(offsets=None), dict(dw=None), dict(dy=P + 1),
                                            dict(x=P + 1), dict(offsets=P + 3), dict(dw=P + 1)]),
]


@pytest.mark.parametrize("fn,base,status,changes", REFUSED)
def test_refusals(fn, base, status, changes):
    f = getattr(_lib(), fn)
    for c in changes:
        assert f(*dict(base, **c).values()) == status, (fn, c)


def test_nothing_to_do_is_accepted_without_pointers():
    L = _lib()
    none = dict(x=None, w=None, offsets=None, y=None, dy=None, dx=None, dw=None, workspace=None, workspace_bytes=0)
    pick = lambda base: {k: none.get(k, v) for k, v in base.items()}
    for fn, base, empties in (("muon_experts_forward", F, ("rows", "experts", "out")),
                              ("muon_experts_input_grad", X, ("rows", "experts", "in_")),
                              ("muon_experts_weight_grad", W, ("experts", "out", "in_"))):
        for e in empties:
            assert getattr(L, fn)(*dict(pick(base), **{e: 0}).values()) == 0, (fn, e)
    # sums over nothing still write, so they need the offsets and the result
    for fn, base, e in (("muon_experts_forward", F, "in_"), ("muon_experts_input_grad", X, "out"),
                        ("muon_experts_weight_grad", W, "rows")):
        assert getattr(L, fn)(*dict(pick(base), **{e: 0}).values()) == E_ARG, fn


def test_workspace_is_asked_for_and_checked():
    L = _lib()
    b = ctypes.c_size_t()
    q = lambda *a: L.muon_experts_workspace_bytes(*a, ctypes.byref(b))
    assert q(3, 9, 3, 6, 20, 1) == E_METHOD and q(-1, 9, 3, 6, 20, 1) == E_METHOD
    assert q(0, 9, 3, 6, 20, 2) == E_DTYPE and q(0, -9, 3, 6, 20, 1) == E_SHAPE and q(0, 9, 1 << 17, 6, 20, 1) == E_SHAPE
    assert L.muon_experts_workspace_bytes(0, 9, 3, 6, 20, 1, None) == E_ARG
    for empty in ((0, 3, 6, 20), (9, 0, 6, 20), (9, 3, 0, 20), (9, 3, 6, 0)):
        assert q(1, *empty, 1) == 0 and b.value == 0
    # a long sum into few tiles is split; too small a workspace is refused
    big = dict(W, rows=30000, experts=1, stride=0)
    assert q(1, 30000, 1, 6, 20, 1) == 0 and b.value > 0
    assert L.muon_experts_weight_grad(*dict(big, workspace_bytes=b.value - 1).values()) == E_WORKSPACE
    assert L.muon_experts_weight_grad(*dict(big, workspace=None).values()) == E_WORKSPACE


def test_binding_refusals():
    _lib()
    off = torch.zeros(4, dtype=torch.int32)
    x, w, dy = torch.zeros(9, 20), torch.zeros(3, 6, 20), torch.zeros(9, 6)
    for bad in ((x.double(), w, off), (x, w.bfloat16(), off), (x, w[:, :, :19], off), (x, w[:2], off), (x[0], w, off),
                (x, w.transpose(1, 2), off), (x, w, off.long()), (x, w, off[:0]), (x, w, torch.zeros(8, dtype=torch.int32)[::2]),
                (x, torch.zeros(17, 20), off), (x, w[:1].expand(3, 6, 20), off), (x, w, off)):  # the last: host tensors
        with pytest.raises(ValueError):
            mo.muon_experts_forward(*bad)
    for bad in ((dy, x[:8], off), (dy, x.bfloat16(), off), (dy.t(), x, off), (dy, x, off)):
        with pytest.raises(ValueError):
            mo.muon_experts_weight_grad(*bad)
    for bad in ((dy[:, :5], w, off), (dy.bfloat16(), w, off), (dy, w, off)):
        with pytest.raises(ValueError):
            mo.muon_experts_input_grad(*bad)


def test_widths_past_a_leading_dimension():
    """2^21 is the most a row can be apart, so wider matrices are refused, by the
    query too (whose counts of tiles would not fit 64 bits)."""
    L = _lib()
    b = ctypes.c_size_t()
    for kind in range(3):
        for wide in ((1 << 30, 1 << 16, 1 << 30, 1 << 30), (1 << 30, 1, (1 << 21) + 1, 8), (9, 1, 8, (1 << 21) + 1)):
            for dtype in (0, 1):
                assert L.muon_experts_workspace_bytes(kind, *wide, dtype, ctypes.byref(b)) == E_SHAPE
        for dtype in (0, 1):
            assert L.muon_experts_workspace_bytes(kind, 1 << 30, 1 << 16, 1 << 21, 1 << 21, dtype, ctypes.byref(b)) == 0
    assert L.muon_experts_forward(*dict(F, out=(1 << 21) + 8, ldy=(1 << 21) + 8, stride=1 << 40).values()) == E_SHAPE
