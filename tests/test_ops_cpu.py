"""The operators around the step without a GPU: the fp64 reference against
closed forms and differences, and every refusal of the C entry points and of
the binding (all of them come before any launch)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import ops_ref as R

mo = pytest.importorskip("matrix_orthogonalizing_optimizer_amd")

E_ARG, E_SHAPE, E_DTYPE, E_METHOD, E_WORKSPACE = -1, -2, -3, -4, -5
P = 1 << 20  # an aligned address that is never followed: the calls are refused first


def _lib():
    try:
        return mo.lib()
    except RuntimeError as e:
        pytest.skip(str(e))


# ------------------------------------------------------------- the reference

def test_rows8_closed_forms():
    x = np.array([[127.0, -127.0, 0.5, 1.5],       # scale 1, ties to even
                  [127.00001, 0.0, 0.0, 2.0],      # just above: scale 2
                  [0.0, 0.0, 0.0, 0.0],
                  [1e-45, 0.0, 0.0, 0.0],
                  [254.0, 63.0, 1.0, 3.0],
                  [np.inf, 1.0, 0.0, 0.0],
                  [np.nan, 1.0, 0.0, 0.0],
                  [3.3895314e38, 0.0, 0.0, 0.0]])
    q, s = R.rows8(x)
    assert s[:5].tolist() == [1.0, 2.0, 2.0 ** -126, 2.0 ** -126, 2.0]
    assert np.isnan(s[5:7]).all() and not q[5:7].any()
    assert q[0].tolist() == [127, -127, 0, 2] and q[1].tolist() == [64, 0, 0, 1]
    assert q[4].tolist() == [127, 32, 0, 2]
    assert s[7] == 2.0 ** 122 and q[7, 0] == 63
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 33)) * np.exp(rng.uniform(-30, 30, (50, 1)))
    q, s = R.rows8(x)
    assert (np.abs(R.restore(q, s) - x) <= s[:, None] / 2).all()
    top = np.abs(x).max(axis=1)
    assert (top <= 127 * s).all() and (top > 127 * s / 2).all()


@pytest.mark.parametrize("layer", [True, False])
def test_norm_gradients_match_differences(layer):
    rng = np.random.default_rng(2)
    x, dy = rng.standard_normal((3, 7)), rng.standard_normal((3, 7))
    gamma, beta = rng.standard_normal(7), rng.standard_normal(7) if layer else None
    _, mean, rstd = R.norm_forward(x, gamma, beta, 1e-3, layer)
    dx, dg, db = R.norm_backward(dy, x, gamma, mean, rstd, layer)
    loss = lambda x_, g_, b_: float((R.norm_forward(x_, g_, b_, 1e-3, layer)[0] * dy).sum())
    h = 1e-6
    for i in range(3):
        for j in range(7):
            e = np.zeros_like(x)
            e[i, j] = h
            assert math.isclose((loss(x + e, gamma, beta) - loss(x - e, gamma, beta)) / (2 * h), dx[i, j],
                                rel_tol=1e-6, abs_tol=1e-7)
    for j in range(7):
        e = np.zeros(7)
        e[j] = h
        assert math.isclose((loss(x, gamma + e, beta) - loss(x, gamma - e, beta)) / (2 * h), dg[j], rel_tol=1e-6,
                            abs_tol=1e-7)
        if layer:
            assert math.isclose((loss(x, gamma, beta + e) - loss(x, gamma, beta - e)) / (2 * h), db[j],
                                rel_tol=1e-6, abs_tol=1e-7)


def test_linear8_gradients_match_differences():
    rng = np.random.default_rng(3)
    q, s = R.rows8(rng.standard_normal((4, 5)))
    wq, ws = R.rows8(rng.standard_normal((3, 5)))
    dy = rng.standard_normal((4, 3))
    x, w = R.restore(q, s), R.restore(wq, ws)
    assert np.allclose(R.linear8_forward(q, s, wq, ws), x @ w.T)
    dw, dx = R.linear8_weight_grad(dy, q, s), R.linear8_input_grad(dy, wq, ws)
    h = 1e-6
    for i in range(3):
        for j in range(5):
            e = np.zeros_like(w)
            e[i, j] = h
            assert math.isclose((((x @ (w + e).T) - (x @ (w - e).T)) * dy).sum() / (2 * h), dw[i, j], rel_tol=1e-6)
    for i in range(4):
        for j in range(5):
            e = np.zeros_like(x)
            e[i, j] = h
            assert math.isclose(((((x + e) @ w.T) - ((x - e) @ w.T)) * dy).sum() / (2 * h), dx[i, j], rel_tol=1e-6)


# ------------------------------------------------- refusals of the C entries

Q = dict(x=P, rows=4, cols=20, ldx=20, dtype=1, q=P, ldq=32, scale=P, stream=None)
D = dict(q=P, ldq=32, scale=P, rows=4, cols=20, y=P, ldy=20, dtype=1, stream=None)
NF = dict(kind=0, x=P, rows=4, cols=20, ldx=20, dtype=1, gamma=P, beta=P, vec_dtype=1, eps=1e-5, y=P, ldy=20, q=P,
          ldq=32, scale=P, mean=P, rstd=P, stream=None)
NB = dict(kind=0, dy=P, lddy=20, x=P, ldx=20, rows=4, cols=20, dtype=1, gamma=P, vec_dtype=1, mean=P, rstd=P, dx=P,
          lddx=20, dgamma=P, dbeta=P, accumulate=0, workspace=P, workspace_bytes=1 << 20, stream=None)
LF = dict(q=P, ldq=32, scale=P, wq=P, ldw=32, wscale=P, bias=P, bias_dtype=1, tokens=4, out=6, in_=20, y=P, ldy=6,
          dtype=1, workspace=P, workspace_bytes=1 << 24, stream=None)
LW = dict(dy=P, lddy=6, dy_dtype=1, q=P, ldq=32, scale=P, tokens=4, out=6, in_=20, dw=P, lddw=20, dw_dtype=1,
          accumulate=0, workspace=P, workspace_bytes=1 << 24, stream=None)
LX = dict(dy=P, lddy=6, dy_dtype=1, wq=P, ldw=32, wscale=P, tokens=4, out=6, in_=20, dx=P, lddx=20, dx_dtype=1,
          workspace=P, workspace_bytes=1 << 24, stream=None)

REFUSED = [
    ("muon_rows8_quantize", Q, E_DTYPE, [dict(dtype=2), dict(dtype=-1)]),
    ("muon_rows8_quantize", Q, E_SHAPE, [dict(rows=-1), dict(cols=-1), dict(ldx=19), dict(ldq=16), dict(ldq=24),
                                         dict(rows=1 << 31), dict(cols=1 << 31, ldx=1 << 31, ldq=1 << 31),
                                         dict(cols=(1 << 27) + 16, ldx=1 << 28, ldq=1 << 28), dict(ldx=1 << 41)]),
    ("muon_rows8_quantize", Q, E_ARG, [dict(x=None), dict(q=None), dict(scale=None), dict(x=P + 1), dict(q=P + 8),
                                       dict(scale=P + 2), dict(x=P + 2, dtype=0)]),
    ("muon_rows8_dequantize", D, E_DTYPE, [dict(dtype=7)]),
    ("muon_rows8_dequantize", D, E_SHAPE, [dict(rows=-1), dict(cols=-2), dict(ldy=19), dict(ldq=30)]),
    ("muon_rows8_dequantize", D, E_ARG, [dict(q=None), dict(y=None), dict(scale=None), dict(q=P + 4), dict(y=P + 1)]),
    ("muon_norm_forward", NF, E_METHOD, [dict(kind=2), dict(kind=-1)]),
    ("muon_norm_forward", NF, E_DTYPE, [dict(dtype=3), dict(vec_dtype=3)]),
    ("muon_norm_forward", NF, E_SHAPE, [dict(rows=-1), dict(cols=-1), dict(ldx=1), dict(ldy=19), dict(ldq=31),
                                        dict(ldq=16)]),
    ("muon_norm_forward", NF, E_ARG, [dict(x=None), dict(gamma=None), dict(eps=-1.0), dict(eps=math.inf),
                                      dict(eps=math.nan), dict(q=None), dict(scale=None), dict(kind=1),
                                      dict(y=None, q=None, scale=None, mean=None, rstd=None), dict(y=P + 1),
                                      dict(mean=P + 2), dict(rstd=P + 1), dict(beta=P + 1), dict(ldy=24)]),
    ("muon_norm_backward", NB, E_METHOD, [dict(kind=5)]),
    ("muon_norm_backward", NB, E_DTYPE, [dict(dtype=2), dict(vec_dtype=-1)]),
    ("muon_norm_backward", NB, E_SHAPE, [dict(rows=-1), dict(cols=-1), dict(lddy=3), dict(ldx=3), dict(lddx=3)]),
    ("muon_norm_backward", NB, E_ARG, [dict(dy=None), dict(x=None), dict(dx=None), dict(gamma=None), dict(mean=None),
                                       dict(rstd=None), dict(kind=1), dict(dgamma=P + 1), dict(dbeta=P + 1),
                                       dict(lddx=24)]),
    ("muon_norm_backward", NB, E_WORKSPACE, [dict(workspace=None), dict(workspace_bytes=100)]),
    ("muon_linear8_forward", LF, E_DTYPE, [dict(dtype=2), dict(bias_dtype=9)]),
    ("muon_linear8_forward", LF, E_SHAPE, [dict(tokens=-1), dict(out=-1), dict(in_=-1), dict(in_=131072, ldq=131072,
                                           ldw=131072), dict(ldq=16), dict(ldw=40), dict(ldy=5), dict(ldy=1 << 22)]),
    ("muon_linear8_forward", LF, E_ARG, [dict(q=None), dict(wq=None), dict(scale=None), dict(wscale=None),
                                         dict(y=None), dict(q=P + 1), dict(wq=P + 8), dict(bias=P + 1)]),
    ("muon_linear8_weight_grad", LW, E_DTYPE, [dict(dy_dtype=2), dict(dw_dtype=2)]),
    ("muon_linear8_weight_grad", LW, E_SHAPE, [dict(tokens=-1), dict(out=-1), dict(in_=-1), dict(lddy=5),
                                               dict(ldq=16), dict(ldq=33), dict(lddw=19),
                                           dict(out=1 << 20, in_=1 << 20, lddy=1 << 20, ldq=1 << 20, lddw=1 << 20,
                                                workspace_bytes=1 << 62)]),
    ("muon_linear8_weight_grad", LW, E_ARG, [dict(dy=None), dict(q=None), dict(scale=None), dict(dw=None),
                                             dict(dy=P + 1), dict(q=P + 2), dict(dw=P + 1)]),
    ("muon_linear8_input_grad", LX, E_DTYPE, [dict(dy_dtype=2), dict(dx_dtype=2)]),
    ("muon_linear8_input_grad", LX, E_SHAPE, [dict(tokens=-1), dict(out=-1), dict(in_=-1), dict(lddy=5),
                                              dict(ldw=16), dict(lddx=19)]),
    ("muon_linear8_input_grad", LX, E_ARG, [dict(dy=None), dict(wq=None), dict(wscale=None), dict(dx=None)]),
]


@pytest.mark.parametrize("fn,good,status,changes", REFUSED, ids=[f"{r[0]}{r[2]}" for r in REFUSED])
def test_c_entries_refuse(fn, good, status, changes):
    f = getattr(_lib(), fn)
    for ch in changes:
        args = dict(good, **ch)
        assert f(*args.values()) == status, (fn, ch)


def test_c_entries_accept_empty():
    """Sizes that leave nothing to do return without following a pointer."""
    L = _lib()
    call = lambda fn, good, **ch: getattr(L, fn)(*dict(good, **ch).values())
    assert call("muon_rows8_quantize", Q, rows=0, x=None, q=None, scale=None) == 0
    assert call("muon_rows8_dequantize", D, rows=0, q=None) == 0
    assert call("muon_rows8_dequantize", D, cols=0, q=None) == 0
    assert call("muon_norm_forward", NF, rows=0) == 0 and call("muon_norm_forward", NF, cols=0) == 0
    assert call("muon_norm_backward", NB, cols=0) == 0
    assert call("muon_norm_backward", NB, rows=0, dgamma=None, dbeta=None) == 0
    assert call("muon_linear8_forward", LF, tokens=0) == 0 and call("muon_linear8_forward", LF, out=0) == 0
    assert call("muon_linear8_weight_grad", LW, out=0) == 0 and call("muon_linear8_weight_grad", LW, in_=0) == 0
    assert call("muon_linear8_input_grad", LX, tokens=0) == 0


def test_workspace_queries():
    L = _lib()
    n = ctypes.c_size_t()
    assert L.muon_norm_backward_workspace_bytes(8, 8, None) == E_ARG
    assert L.muon_norm_backward_workspace_bytes(-1, 8, ctypes.byref(n)) == E_SHAPE
    assert L.muon_linear8_workspace_bytes(0, 8, 8, 8, None, 0, 0, None) == E_ARG
    assert L.muon_linear8_workspace_bytes(3, 8, 8, 8, None, 0, 0, ctypes.byref(n)) == E_METHOD
    assert L.muon_linear8_workspace_bytes(1, 8, 8, 8, None, 8, 2, ctypes.byref(n)) == E_DTYPE
    assert L.muon_linear8_workspace_bytes(1, 8, -8, 8, None, 0, 0, ctypes.byref(n)) == E_SHAPE
    assert L.muon_linear8_workspace_bytes(0, 8, 8, 1 << 20, None, 0, 0, ctypes.byref(n)) == E_SHAPE
    assert mo.muon_norm_backward_workspace_bytes(0, 8) == 0
    assert mo.muon_norm_backward_workspace_bytes(100, 8) >= 2 * 8 * 4


# --------------------------------------------------- refusals of the binding

def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def _q(rows, cols):
    return torch.zeros(rows, (cols + 15) // 16 * 16, dtype=torch.int8)[:, :cols]


F32 = torch.float32
BINDING = [
    (lambda: mo.muon_rows8_quantize(_t(4, 20)), "device memory"),
    (lambda: mo.muon_rows8_quantize(_t(20)), "2-D"),
    (lambda: mo.muon_rows8_quantize(_t(4, 20, dtype=torch.float16)), "float32 or bfloat16"),
    (lambda: mo.muon_rows8_quantize(_t(20, 4).t()), "contiguous"),
    (lambda: mo.muon_rows8_quantize(_t(1, 20).expand(4, 20)), "overlap"),
    (lambda: mo.muon_rows8_quantize(_t(4, 20), q=_q(4, 20)), "both or neither"),
    (lambda: mo.muon_rows8_dequantize(_t(4, 20), _t(4, dtype=F32)), "int8"),
    (lambda: mo.muon_rows8_dequantize(torch.zeros(4, 20, dtype=torch.int8), _t(4, dtype=F32)), "16"),
    (lambda: mo.muon_rows8_dequantize(torch.zeros(127, dtype=torch.int8).as_strided((4, 31), (32, 1)).narrow(1, 0, 20),
                                      _t(4, dtype=F32)), "storage"),
    (lambda: mo.muon_rows8_dequantize(_q(4, 20), _t(3, dtype=F32)), "vector of 4"),
    (lambda: mo.muon_rows8_dequantize(_q(4, 20), _t(4)), "float32"),
    (lambda: mo.muon_norm_forward(_t(4, 20), _t(19), y=_t(4, 20)), "vector of 20"),
    (lambda: mo.muon_norm_forward(_t(4, 20), _t(20), beta=_t(20, dtype=F32), y=_t(4, 20)), "bfloat16"),
    (lambda: mo.muon_norm_forward(_t(4, 20), _t(20), y=_t(4, 20, dtype=F32)), "y: expected"),
    (lambda: mo.muon_norm_forward(_t(4, 20), _t(20), y=_t(4, 20), mean=_t(4)), "mean"),
    (lambda: mo.muon_norm_forward(_t(4, 20), _t(20), y=_t(4, 20)), "device memory"),
    (lambda: mo.muon_norm_backward(_t(4, 20), _t(4, 21), _t(20), _t(4, dtype=F32), _t(4, dtype=F32)), "x: expected"),
    (lambda: mo.muon_norm_backward(_t(4, 20), _t(4, 20), _t(20), _t(4, dtype=F32), _t(4, dtype=F32),
                                   dgamma=_t(20, dtype=F32)), "dgamma"),
    (lambda: mo.muon_linear8_forward(_q(4, 20), _t(4, dtype=F32), _q(6, 21), _t(6, dtype=F32)), "20 columns"),
    (lambda: mo.muon_linear8_forward(_q(4, 20), _t(4, dtype=F32), _q(6, 20), _t(6, dtype=F32), bias=_t(5)), "bias"),
    (lambda: mo.muon_linear8_weight_grad(_t(5, 6), _q(4, 20), _t(4, dtype=F32)), "4 rows for 5"),
    (lambda: mo.muon_linear8_input_grad(_t(5, 6), _q(4, 20), _t(4, dtype=F32)), "4 rows for 6"),
    (lambda: mo.muon_linear8_input_grad(_t(5, 4), _q(4, 20), _t(4, dtype=F32)), "device memory"),
]


@pytest.mark.parametrize("i", range(len(BINDING)))
def test_binding_refuses(i):
    _lib()
    call, text = BINDING[i]
    with pytest.raises(ValueError, match=text):
        call()


def test_norm_into_empty_rows8_is_accepted():
    """An empty q has a null address; its scales may not."""
    L = _lib()
    for ch in (dict(cols=0, q=None), dict(rows=0, q=None), dict(cols=0, scale=None)):
        assert L.muon_norm_forward(*dict(NF, **ch).values()) == 0, ch
    assert L.muon_norm_forward(*dict(NF, cols=0, kind=1).values()) == E_ARG  # RMS norms have no mean


def test_workspace_has_to_be_contiguous():
    """The kernels write the workspace's bytes in a row: one whose elements lie
    apart, or upon each other, holds less than it has elements."""
    one = torch.zeros(1, dtype=torch.uint8)
    for ws in (one.expand(4096), torch.zeros(8192, dtype=torch.uint8)[::2], torch.zeros(64, 64)[:, :32]):
        with pytest.raises(ValueError, match="workspace"):
            mo._lib._scratch(0, None, ws, 16)
    ws = torch.zeros(64, 16)[8:24]
    assert mo._lib._scratch(0, None, ws, 16) == (ws, ws.data_ptr(), 16 * 16 * 4)
