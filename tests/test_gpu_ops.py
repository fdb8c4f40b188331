"""GPU tests of the operators around the step (8-bit rows, row norms and
their gradients, the linear layer on 8-bit rows) against the fp64 reference,
at the sizes, strides and values where each can go wrong.

Tolerances.  u = 2^-24 bounds one fp32 rounding, half(t) = eps(t) / 2 one
rounding to the output's type.  A sum whose terms pass through at most d
additions is off by at most d u sum|terms|.
"""
import math

import numpy as np
import pytest
import torch

from oracle import ops_ref as R
from tests.gpu_util import dev, f64

mo = pytest.importorskip("matrix_orthogonalizing_optimizer_amd")

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def half(t):
    return torch.finfo(t).eps / 2


def gen(seed):
    return torch.Generator().manual_seed(seed)


def matrix(rows, cols, dtype, seed, scale=1.0, pad=0, off=0):
    """A device matrix with rows cols + pad apart, starting off elements into
    its storage, and the storage itself."""
    base = torch.randn(rows * (cols + pad) + off + pad, generator=gen(seed)).mul_(scale).to(dtype).to(dev())
    return base[off:off + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]


def rows8(rows, cols, seed, scale=1.0):
    """(q, scale) in padded storage, and the fp64 values they stand for."""
    q, s = R.rows8(torch.randn(rows, cols, generator=gen(seed)).mul_(scale).numpy())
    store = torch.zeros(rows, (cols + 15) // 16 * 16, dtype=torch.int8)
    store[:, :cols] = torch.from_numpy(q)
    return store.to(dev())[:, :cols], torch.from_numpy(s).float().to(dev())


def check(got, ref, bound, what):
    """|got - ref| <= bound everywhere (NaN where the reference is NaN)."""
    got, bound = f64(got), np.broadcast_to(bound, ref.shape)
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(got), nan), what
    err = np.where(nan, 0.0, np.abs(got - np.where(nan, 0.0, ref)))
    over = np.where(nan, 0.0, err - bound)
    i = np.unravel_index(np.argmax(over), over.shape) if over.size else None
    assert i is None or over[i] <= 0, f"{what}: {got[i]} for {ref[i]} at {i}, bound {bound[i]}"


# ------------------------------------------------------------- 8-bit rows

WIDTHS = [1, 2, 7, 8, 15, 16, 17, 63, 64, 65, 300, 511, 512, 513, 768, 1001, 1024, 1025, 2047, 2049, 4096, 4104, 8191,
          8200, 14336, 16384, 16385, 20001]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cols", WIDTHS)
def test_rows8_are_exact(cols, dtype):
    print("rows8", cols, dtype, flush=True)
    rows = 9
    x = matrix(rows, cols, dtype, cols, 3.0, pad=3, off=1)
    x[1] = 0
    x[2] *= 1e-30
    x[3] *= 1e30
    x[4, cols - 1] = 127.0 if dtype == F32 else 128.0
    q, s = mo.muon_rows8_quantize(x)
    store = q.as_strided((rows, q.stride(0)), (q.stride(0), 1))
    rq, rs = R.rows8(f64(x))
    assert np.array_equal(f64(s), rs)
    assert np.array_equal(q.cpu().numpy(), rq)
    assert store[:, cols:].count_nonzero().item() == 0
    for t in (BF, F32):
        y = mo.muon_rows8_dequantize(q, s, dtype=t)
        ref = R.restore(rq, rs)
        # exact, but for values below the smallest bf16/fp32 number
        check(y, ref, np.where(np.abs(ref) < 2.0 ** -120, 2.0 ** -126, 0.0), t)


def test_rows8_special_values():
    d = dev()
    x = torch.tensor([[math.nan, 1.0, 2.0], [math.inf, 1.0, 0.0], [-math.inf, math.nan, 0.0], [0.0, 0.0, 0.0],
                      [3.3895314e38, -1.0, 0.0], [1e-45, 0.0, -1e-45], [127.0, 0.5, 1.5], [127.00001, 2.0, 0.0],
                      [1.1754944e-38, 0.0, 0.0]], dtype=F32, device=d)
    q, s = mo.muon_rows8_quantize(x)
    rq, rs = R.rows8(f64(x))
    assert np.array_equal(f64(s), rs, equal_nan=True) and np.array_equal(q.cpu().numpy(), rq)
    y = mo.muon_rows8_dequantize(q, s, dtype=F32)
    assert torch.isnan(y[:3]).all() and torch.isfinite(y[3:]).all()


def test_rows8_writes_only_its_rows():
    """Bytes behind the 16-byte padding, rows behind the last one and the
    columns between rows of the restored matrix keep their values."""
    d = dev()
    x = matrix(5, 20, BF, 1)
    store = torch.full((8, 64), 77, dtype=torch.int8, device=d)
    scale = torch.full((8,), 5.0, device=d)
    mo.muon_rows8_quantize(x, q=store[1:6, :20], scale=scale[1:6])
    assert (store[[0, 6, 7]] == 77).all() and (store[:, 32:] == 77).all() and (store[1:6, 20:32] == 0).all()
    assert (scale[[0, 6, 7]] == 5).all()
    out = torch.full((8, 40), 9.0, dtype=BF, device=d)
    mo.muon_rows8_dequantize(store[1:6, :20], scale[1:6], out=out[1:6, 3:23])
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[1:6, 3:23] = False
    assert (out[keep] == 9).all() and not (out[~keep] == 9).all()
    # no columns: scales only; no rows: nothing
    mo.muon_rows8_quantize(x[:, :0], q=store[1:6, :0], scale=scale[1:6])
    assert (scale[1:6] == 2.0 ** -126).all()
    mo.muon_rows8_quantize(x[:0])
    assert mo.muon_rows8_dequantize(store[:0, :20], scale[:0]).shape == (0, 20)


def test_rows8_past_32_bit_offsets():
    """A matrix of more than 2^32 elements: first and last rows."""
    d = dev()
    rows, cols = 270000, 16384
    x = torch.empty(rows, cols, dtype=BF, device=d)
    ends = [0, 1, rows - 2, rows - 1]
    x.zero_()
    x[ends] = matrix(4, cols, BF, 4)
    q, s = mo.muon_rows8_quantize(x)
    rq, rs = R.rows8(f64(x[ends]))
    assert np.array_equal(q[ends].cpu().numpy(), rq) and np.array_equal(f64(s[ends]), rs)
    mo.muon_rows8_dequantize(q, s, out=x)
    assert np.array_equal(f64(x[ends]), R.restore(rq, rs))
    assert x[rows // 2].count_nonzero().item() == 0


def test_rows8_more_rows_than_one_grid_dimension():
    """2^24 rows of 256 threads are 2^32 threads: the last rows of a longer
    matrix are reached all the same."""
    d = dev()
    rows, cols = (1 << 24) + 5, 1040
    x = torch.zeros(rows, cols, dtype=BF, device=d)
    ends = [0, (1 << 20) - 1, 1 << 20, (1 << 24) - 1, 1 << 24, rows - 1]
    x[ends] = matrix(len(ends), cols, BF, 4)
    q, s = mo.muon_rows8_quantize(x)
    rq, rs = R.rows8(f64(x[ends]))
    assert np.array_equal(q[ends].cpu().numpy(), rq) and np.array_equal(f64(s[ends]), rs)
    x.zero_()
    mo.muon_rows8_dequantize(q, s, out=x)
    assert np.array_equal(f64(x[ends]), R.restore(rq, rs))


# ------------------------------------------------------------------- norms

# additions on the way of a term into a row sum: at most 24 of a thread (rows
# up to 24576 columns), 6 of a wave, 16 across waves, and the roundings of
# the quotient, the square root and the products around it
ROW_DEPTH = 64


@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("dtype,vec", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("cols", WIDTHS)
def test_norm_forward(cols, dtype, vec, layer):
    print("norm_forward", cols, dtype, vec, layer, flush=True)
    d, rows, eps = dev(), 6, 1e-5
    x = matrix(rows, cols, dtype, cols + 1, 2.0, pad=1, off=3)
    x[1] += 3.0
    x[2] = 0
    gamma = (1 + 0.1 * torch.randn(cols, generator=gen(5))).to(vec).to(d)
    beta = torch.randn(cols, generator=gen(6)).to(vec).to(d) if layer else None
    y = torch.full((rows + 1, cols + 5), 9.0, dtype=dtype, device=d)
    mean = torch.full((rows,), 9.0, device=d) if layer else None
    rstd = torch.full((rows,), 9.0, device=d)
    kind = mo.MUON_NORM_LAYER if layer else mo.MUON_NORM_RMS
    mo.muon_norm_forward(x, gamma, beta, eps, kind, y=y[:rows, 2:cols + 2], mean=mean, rstd=rstd)
    ry, rm, rr = R.norm_forward(f64(x), f64(gamma), f64(beta) if layer else None, eps, layer)
    X = f64(x)
    ax = np.abs(X).mean(axis=1)
    dm = ROW_DEPTH * U * ax  # the mean's error
    if layer:
        check(mean, rm, dm, "mean")
    # the variance's relative error, halved by the square root, and the mean's
    # error in it (first order cancels: the sum of x - mu is zero up to dm)
    var = ((X - rm[:, None]) ** 2).mean(axis=1)
    dr = rr * (ROW_DEPTH * U + dm * dm / (var + eps))
    check(rstd, rr, dr, "rstd")
    dh = (rr * (dm + U * np.abs(X).max(axis=1)))[:, None] + np.abs(X - rm[:, None]) * (dr + 4 * U * rr)[:, None]
    G = np.abs(f64(gamma))
    bound = dh * G + 2 * U * (np.abs(ry) + (np.abs(f64(beta)) if layer else 0.0))
    check(y[:rows, 2:cols + 2], ry, bound + half(dtype) * (np.abs(ry) + bound), "y")
    assert (y[rows] == 9).all() and (y[:, :2] == 9).all() and (y[:, cols + 2:] == 9).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cols", [5, 64, 768, 1025, 4096, 14336, 20001])
def test_norm_forward_into_rows8(cols, dtype):
    """The 8-bit rows stand for y before its rounding: off by half a step of
    the row's scale, and by the norm's own error."""
    print("norm rows8", cols, dtype, flush=True)
    d, rows = dev(), 7
    x = matrix(rows, cols, dtype, cols, 2.0)
    x[3, 0] = math.nan
    x[4] = 0
    gamma = (1 + 0.1 * torch.randn(cols, generator=gen(5))).to(dtype).to(d)
    beta = torch.randn(cols, generator=gen(6)).to(dtype).to(d)
    q = torch.full((rows, (cols + 15) // 16 * 16 + 16), 77, dtype=torch.int8, device=d)
    s = torch.empty(rows, device=d)
    y = torch.empty_like(x)
    mo.muon_norm_forward(x, gamma, beta, q=q[:, :cols], scale=s, y=y)
    ry = R.norm_forward(f64(x), f64(gamma), f64(beta), 1e-5, True)[0]
    S = f64(s)
    err = 2 * ROW_DEPTH * U * (np.abs(ry) + 4)  # a loose form of the forward test's bound
    check(torch.from_numpy(R.restore(q[:, :cols].cpu().numpy(), S)), np.where(np.isnan(ry), np.nan, ry),
          S[:, None] / 2 + err, "rows8")
    ok = np.isfinite(S)
    assert not ok[3] and ok.sum() == rows - 1
    top = np.abs(ry[ok]).max(axis=1)
    assert (top <= 127 * S[ok] * (1 + 1e-4)).all() and (top > 63.4 * S[ok]).all()
    cpad = (cols + 15) // 16 * 16
    assert (q[:, cols:cpad] == 0).all() and (q[:, cpad:] == 77).all()
    # without y: the same rows
    q2, s2 = torch.empty_like(q), torch.empty_like(s)
    mo.muon_norm_forward(x, gamma, beta, q=q2[:, :cols], scale=s2)
    assert torch.equal(q2[:, :cpad], q[:, :cpad]) and np.array_equal(f64(s2), S, equal_nan=True)
    # in place
    z = x.clone()
    mo.muon_norm_forward(z, gamma, beta, y=z)
    assert np.array_equal(f64(z), f64(y), equal_nan=True)


@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("dtype,vec", [(BF, BF), (F32, F32), (BF, F32)])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (1, 4096), (5, 513), (130, 768), (2050, 65), (700, 1001),
                                       (5000, 64), (300, 2048), (600, 4097), (33, 8191), (9, 14336), (40, 20001)])
def test_norm_backward(rows, cols, dtype, vec, layer):
    print("norm_backward", rows, cols, dtype, vec, layer, flush=True)
    d = dev()
    x = matrix(rows, cols, dtype, rows + cols, 1.5, pad=2, off=1)
    dy = matrix(rows, cols, dtype, rows + cols + 1, 1e-3, pad=1)
    gamma = (1 + 0.1 * torch.randn(cols, generator=gen(5))).to(vec).to(d)
    _, rm, rr = R.norm_forward(f64(x), f64(gamma), None, 1e-5, layer)
    mean = torch.from_numpy(rm).float().to(d) if layer else None
    rstd = torch.from_numpy(rr).float().to(d)
    kind = mo.MUON_NORM_LAYER if layer else mo.MUON_NORM_RMS
    dg0 = torch.randn(cols, generator=gen(7)).to(vec).to(d)
    db0 = torch.randn(cols, generator=gen(8)).to(vec).to(d)
    dx = torch.full((rows + 1, cols + 3), 9.0, dtype=dtype, device=d)
    M = f64(mean) if layer else None
    rx, rg, rb = R.norm_backward(f64(dy), f64(x), f64(gamma), M, f64(rstd), layer)
    DY, r = np.abs(f64(dy)), f64(rstd)[:, None]
    h = np.abs((f64(x) - (M[:, None] if layer else 0.0)) * r)
    g = DY * np.abs(f64(gamma))
    # dx: two row sums of depth ROW_DEPTH, and a few roundings of each term
    bx = r * U * (ROW_DEPTH * (g.mean(axis=1, keepdims=True) + h * (g * h).mean(axis=1, keepdims=True)) + 8 * g)
    # vector gradients: rows in order inside a workgroup (at most 512 share
    # them), 4 of them joined, then the workgroups a quarter at a time
    depth = rows // 512 + 4 + 128 + 8
    bg, bb = depth * U * (DY * h).sum(axis=0), depth * U * DY.sum(axis=0)
    for acc in (False, True):
        dg, db = dg0.clone(), db0.clone()
        mo.muon_norm_backward(dy, x, gamma, mean, rstd, kind, dx=dx[:rows, 1:cols + 1], dgamma=dg,
                              dbeta=db if layer else None, accumulate=acc)
        check(dx[:rows, 1:cols + 1], rx, bx + half(dtype) * (np.abs(rx) + bx), "dx")
        assert (dx[rows] == 9).all() and (dx[:, :1] == 9).all() and (dx[:, cols + 1:] == 9).all()
        for got, ref, b, old in ((dg, rg, bg, dg0), (db, rb, bb, db0)):
            if got is db and not layer:
                assert torch.equal(db, db0)
                continue
            want = ref + (f64(old) if acc else 0.0)
            b2 = b + U * np.abs(want)
            check(got, want, b2 + half(vec) * (np.abs(want) + b2), "vector gradient")
    # dx alone, and in place of dy
    z = dy.clone()
    mo.muon_norm_backward(z, x, gamma, mean, rstd, kind, dx=z)
    assert torch.equal(z, dx[:rows, 1:cols + 1])


def test_norm_backward_empty_and_nan():
    d = dev()
    x = matrix(4, 64, F32, 1)
    dy = matrix(4, 64, F32, 2)
    gamma = torch.ones(64, device=d)
    mean, rstd = torch.zeros(4, device=d), torch.ones(4, device=d)
    dg = torch.full((64,), 3.0, device=d)
    db = torch.full((64,), 3.0, device=d)
    mo.muon_norm_backward(dy[:0], x[:0], gamma, mean[:0], rstd[:0], dgamma=dg, dbeta=db, accumulate=True)
    assert (dg == 3).all() and (db == 3).all()
    mo.muon_norm_backward(dy[:0], x[:0], gamma, mean[:0], rstd[:0], dgamma=dg, dbeta=db)
    assert (dg == 0).all() and (db == 0).all()
    dy[2, 5] = math.inf  # a bad row leaves the other rows and columns alone
    dx = mo.muon_norm_backward(dy, x, gamma, mean, rstd, dgamma=dg, dbeta=db)
    ok = [0, 1, 3]
    assert torch.isfinite(dx[ok]).all() and not torch.isfinite(dx[2]).any()
    cols = [c for c in range(64) if c != 5]
    assert torch.isfinite(dg[cols]).all() and torch.isfinite(db[cols]).all() and not torch.isfinite(db[5])


# ------------------------------------------------------------ linear layer

SIZES = [(1, 1, 1), (1, 16, 16), (1, 4096, 4096), (2, 70, 33), (3, 17, 129), (5, 300, 768), (16, 1000, 100),
         (17, 64, 1024), (33, 65, 47), (64, 256, 2304), (65, 129, 255), (100, 100, 100), (128, 128, 128),
         (129, 257, 64), (200, 513, 1001), (256, 256, 256), (300, 768, 512), (511, 300, 250), (1000, 264, 520),
         (1027, 333, 77), (2000, 48, 1040), (4100, 96, 40)]
# few tokens with short rows of many channels; between the ways for few tokens and for many
FEW_SIZES = [(1, 16384, 64), (9, 16390, 1000), (16, 16387, 1024), (16, 16385, 1040), (32, 100, 8192), (33, 100, 8000),
             (64, 40, 4112), (17, 8208, 50)]


@pytest.mark.parametrize("dtype,bias", [(BF, BF), (F32, None), (BF, None), (F32, F32), (BF, F32)])
@pytest.mark.parametrize("t,n,k", SIZES + FEW_SIZES)
def test_linear8_forward(t, n, k, dtype, bias):
    print("linear8_forward", t, n, k, dtype, bias, flush=True)
    d = dev()
    q, s = rows8(t, k, t + k)
    wq, ws = rows8(n, k, n + k + 1, 0.02)
    b = torch.randn(n, generator=gen(3)).to(bias).to(d) if bias else None
    y = torch.full((t + 1, n + 3), 9.0, dtype=dtype, device=d)
    out = mo.muon_linear8_forward(q, s, wq, ws, bias=b, y=y[:t, 1:n + 1])
    prod = R.linear8_forward(q.cpu().numpy(), f64(s), wq.cpu().numpy(), f64(ws))
    ref = prod + (f64(b) if bias else 0.0)
    # the integer sum is exact: its rounding to fp32, two scales, the bias
    bound = 3 * U * np.abs(prod) + U * np.abs(ref)
    check(out, ref, bound + half(dtype) * (np.abs(ref) + bound), "y")
    assert (y[t] == 9).all() and (y[:, :1] == 9).all() and (y[:, n + 1:] == 9).all()


def grad_bounds(dy, v, trans, dtype):
    """Worst case of a sum in fp32, and what a random walk of its roundings
    reaches in the 2-norm (three pieces of fp32 dy make three sums of it)."""
    A = np.abs(f64(dy))
    terms = (A.T if trans else A) @ np.abs(v)
    n = (dy.shape[0] if trans else dy.shape[1]) * (3 if dtype == F32 else 1) + 16
    return 2 * n * U * terms, U * math.sqrt(n) * 2


def check_grad(got, ref, bound, rms, out_dtype, what):
    check(got, ref, bound + half(out_dtype) * (np.abs(ref) + bound), what)
    norm = np.linalg.norm(ref)
    assert np.linalg.norm(f64(got) - ref) <= (rms + half(out_dtype)) * norm + 1e-300, what


@pytest.mark.parametrize("dtype,odt", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("t,n,k", SIZES)
def test_linear8_gradients(t, n, k, dtype, odt):
    print("linear8 gradients", t, n, k, dtype, odt, flush=True)
    d = dev()
    q, s = rows8(t, k, t + k)
    wq, ws = rows8(n, k, n + k + 1, 0.02)
    for pad, off in ((0, 0), (5, 1), (8, 0)):
        dy = matrix(t, n, dtype, t + n, 1e-3, pad=pad, off=off)
        dw = torch.full((n + 1, k + 3), 9.0, dtype=odt, device=d)
        out = mo.muon_linear8_weight_grad(dy, q, s, dw=dw[:n, 2:k + 2])
        v = R.restore(q.cpu().numpy(), f64(s))
        ref = R.linear8_weight_grad(f64(dy), q.cpu().numpy(), f64(s))
        bound, rms = grad_bounds(dy, v, True, dtype)
        check_grad(out, ref, bound, rms, odt, "dW")
        assert (dw[n] == 9).all() and (dw[:, :2] == 9).all() and (dw[:, k + 2:] == 9).all()
        old = f64(out)
        mo.muon_linear8_weight_grad(dy, q, s, dw=out, accumulate=True)
        want = ref + old
        check(out, want, bound + U * np.abs(want) + half(odt) * (np.abs(want) + bound), "dW added")

        dx = torch.full((t + 1, k + 3), 9.0, dtype=odt, device=d)
        out = mo.muon_linear8_input_grad(dy, wq, ws, dx=dx[:t, 1:k + 1])
        v = R.restore(wq.cpu().numpy(), f64(ws))
        ref = R.linear8_input_grad(f64(dy), wq.cpu().numpy(), f64(ws))
        bound, rms = grad_bounds(dy, v, False, dtype)
        check_grad(out, ref, bound, rms, odt, "dX")
        assert (dx[t] == 9).all() and (dx[:, :1] == 9).all() and (dx[:, k + 1:] == 9).all()


def test_linear8_empty():
    d = dev()
    q, s = rows8(5, 32, 1)
    wq, ws = rows8(7, 32, 2)
    dy = matrix(5, 7, BF, 3)
    bias = torch.randn(7, generator=gen(1)).to(BF).to(d)
    assert mo.muon_linear8_forward(q[:0], s[:0], wq, ws).shape == (0, 7)
    assert mo.muon_linear8_forward(q, s, wq[:0], ws[:0]).shape == (5, 0)
    y = mo.muon_linear8_forward(q[:, :0], s, wq[:, :0], ws, bias=bias)
    assert torch.equal(y, bias.expand(5, 7))
    dw = torch.full((7, 32), 2.0, device=d)
    mo.muon_linear8_weight_grad(dy[:0], q[:0], s[:0], dw=dw, accumulate=True)
    assert (dw == 2).all()
    mo.muon_linear8_weight_grad(dy[:0], q[:0], s[:0], dw=dw)
    assert (dw == 0).all()
    dx = torch.full((5, 32), 2.0, device=d)
    mo.muon_linear8_input_grad(dy[:, :0], wq[:0], ws[:0], dx=dx)
    assert (dx == 0).all()


def test_linear8_largest_integer_sums():
    """127 * 127 * 131071 stays exact; so does -128 * -128 * 131071, which
    only rows written by hand hold."""
    d = dev()
    k = 131071
    for t in (1, 3, 70):
        for v in (127, -128):
            q = torch.full((t, k + 1), v, dtype=torch.int8, device=d)
            q[:, k] = 0
            one = torch.ones(t, device=d)
            y = mo.muon_linear8_forward(q[:, :k], one, q[:, :k], one, dtype=F32)
            assert (y == float(np.float32(v * v * k))).all()


def test_linear8_nan_rows_and_other_scales():
    """A token whose scale is NaN spoils its own outputs and the whole weight
    gradient, not its neighbours; scales other than powers of two are taken
    as they are in y and rounded with q to bf16 in the gradients."""
    d = dev()
    t, n, k = 40, 50, 96
    q, s = rows8(t, k, 1)
    wq, ws = rows8(n, k, 2)
    dy = matrix(t, n, BF, 3)
    s2 = s.clone()
    s2[7] = math.nan
    y = mo.muon_linear8_forward(q, s2, wq, ws)
    assert torch.isnan(y[7]).all() and torch.isfinite(y[:7]).all() and torch.isfinite(y[8:]).all()
    assert torch.isnan(mo.muon_linear8_weight_grad(dy, q, s2)).all()
    dy2 = dy.clone()
    dy2[3, 4] = math.nan
    dw = mo.muon_linear8_weight_grad(dy2, q, s)
    assert torch.isnan(dw[4]).all() and torch.isfinite(dw[:4]).all() and torch.isfinite(dw[5:]).all()
    dx = mo.muon_linear8_input_grad(dy2, wq, ws)
    assert torch.isnan(dx[3]).all() and torch.isfinite(dx[:3]).all() and torch.isfinite(dx[4:]).all()
    s3 = s * 1.37
    Q = q.cpu().numpy()
    prod = R.linear8_forward(Q, f64(s3), wq.cpu().numpy(), f64(ws))
    check(mo.muon_linear8_forward(q, s3, wq, ws, dtype=F32), prod, 4 * U * np.abs(prod), "y")
    ref = R.linear8_weight_grad(f64(dy), Q, f64(s3))
    terms = np.abs(f64(dy)).T @ np.abs(R.restore(Q, f64(s3)))
    check(mo.muon_linear8_weight_grad(dy, q, s3, dtype=F32), ref, (half(BF) + 2 * (t + 16) * U) * terms, "dW")


def test_linear8_neighbours_of_dy_do_not_leak():
    """dy as a column range of a wider tensor that holds NaN elsewhere."""
    d = dev()
    t, n, k = 70, 37, 50
    q, s = rows8(t, k, 1)
    wq, ws = rows8(n, k, 2)
    for dtype in (BF, F32):
        for width, lo in ((64, 8), (64, 3), (48, 0)):
            wide = torch.full((t, width), math.nan, dtype=dtype, device=d)
            dy = wide[:, lo:lo + n]
            dy.copy_(matrix(t, n, dtype, 3))
            dw = mo.muon_linear8_weight_grad(dy, q, s)
            dx = mo.muon_linear8_input_grad(dy, wq, ws)
            c = dy.contiguous()
            assert torch.isfinite(dw).all() and torch.isfinite(dx).all()
            assert torch.equal(dw, mo.muon_linear8_weight_grad(c, q, s))
            assert torch.equal(dx, mo.muon_linear8_input_grad(c, wq, ws))


@pytest.mark.parametrize("t,n,k", [(70, 37, 50), (130, 300, 129), (300, 2100, 2300), (2100, 300, 2300)])
def test_linear8_fp32_dy_with_infinities(t, n, k):
    """fp32 dy in three pieces, cut in the product or laid out first: numbers of
    all sizes count fully; an infinity or a NaN (its payload in the low bits
    only) spoils its own row and column and nothing else."""
    d = dev()
    q, s = rows8(t, k, 1)
    wq, ws = rows8(n, k, 2)
    dy = matrix(t, n, F32, 3)
    dy[:, 2] *= 2.0 ** -60
    dy[5] *= 2.0 ** 40
    for name, pass_, args in (("dW", mo.muon_linear8_weight_grad, (q, s)),
                              ("dX", mo.muon_linear8_input_grad, (wq, ws))):
        left = f64(dy).T if name == "dW" else f64(dy)
        right = R.restore(args[0].cpu().numpy(), f64(args[1]))
        ref, terms = left @ right, np.abs(left) @ np.abs(right)
        # a sum of three pieces of each value, as in grad_bounds
        check(pass_(dy, *args, dtype=F32), ref, 2 * (3 * left.shape[1] + 16) * U * terms, name)
    dy[5] *= 2.0 ** -40
    bad = dy.clone()
    bad[3, 4] = math.inf
    bad.view(torch.int32)[6, 7] = 0x7f800001  # NaN
    bad[t - 1, n - 1] = -math.inf
    dw = mo.muon_linear8_weight_grad(bad, q, s)
    dx = mo.muon_linear8_input_grad(bad, wq, ws)
    cols, rows = [4, 7, n - 1], [3, 6, t - 1]
    assert not torch.isfinite(dw[cols]).any() and not torch.isfinite(dx[rows]).any()
    assert torch.isnan(dw[7]).all() and torch.isnan(dx[6]).all()
    ok = [i for i in range(n) if i not in cols]
    assert torch.equal(dw[ok], mo.muon_linear8_weight_grad(dy, q, s)[ok])
    ok = [i for i in range(t) if i not in rows]
    assert torch.equal(dx[ok], mo.muon_linear8_input_grad(dy, wq, ws)[ok])


def test_linear8_past_32_bit_offsets():
    """Kept rows and gradients of more than 2^31 bytes; only the last rows
    are not zero, so a wrong offset shows."""
    d = dev()
    t, k, n = 140000, 16384, 40
    store = torch.zeros(t, k, dtype=torch.int8, device=d)
    q, s = rows8(64, k, 1)
    store[t - 64:] = q
    scale = torch.ones(t, device=d)
    scale[t - 64:] = s
    dy = torch.zeros(t, n, dtype=BF, device=d)
    dy[t - 64:] = matrix(64, n, BF, 2)
    dw = mo.muon_linear8_weight_grad(dy, store, scale, dtype=F32)
    ref = mo.muon_linear8_weight_grad(dy[t - 64:], q, s, dtype=F32)
    assert float((dw - ref).norm() / ref.norm()) <= 1e-6  # the same 64 terms, another grouping: 64 u = 4e-6 at worst
    wq, ws = rows8(n, k, 3)
    y = mo.muon_linear8_forward(store, scale, wq, ws)
    assert torch.equal(y[t - 64:], mo.muon_linear8_forward(q, s, wq, ws)) and (y[:t - 64] == 0).all()
    dx = mo.muon_linear8_input_grad(dy, wq, ws)
    assert torch.equal(dx[t - 64:], mo.muon_linear8_input_grad(dy[t - 64:], wq, ws))
    assert dx[t - 65].count_nonzero().item() == 0


# ------------------------------------------- streams, graphs, repeated calls

def all_calls(d, t=600, n=300, k=500, dtype=BF):
    x = matrix(t, k, dtype, 1, 2.0)
    gamma = (1 + 0.1 * torch.randn(k, generator=gen(2))).to(dtype).to(d)
    beta = torch.randn(k, generator=gen(3)).to(dtype).to(d)
    wq, ws = rows8(n, k, 4, 0.02)
    bias = torch.randn(n, generator=gen(5)).to(dtype).to(d)
    dy = matrix(t, n, dtype, 6, 1e-3)
    store = torch.zeros(t, (k + 15) // 16 * 16, dtype=torch.int8, device=d)
    b = {"q": store[:, :k], "s": torch.zeros(t, device=d), "mean": torch.zeros(t, device=d),
         "rstd": torch.zeros(t, device=d), "y": torch.zeros(t, n, dtype=dtype, device=d),
         "dw": torch.zeros(n, k, dtype=dtype, device=d), "dh": torch.zeros(t, k, dtype=dtype, device=d),
         "dx": torch.zeros(t, k, dtype=dtype, device=d), "dg": torch.zeros(k, dtype=dtype, device=d),
         "db": torch.zeros(k, dtype=dtype, device=d), "back": torch.zeros(t, k, dtype=dtype, device=d)}

    def run(stream=None):
        mo.muon_norm_forward(x, gamma, beta, q=b["q"], scale=b["s"], mean=b["mean"], rstd=b["rstd"], stream=stream)
        mo.muon_rows8_dequantize(b["q"], b["s"], out=b["back"], stream=stream)
        mo.muon_linear8_forward(b["q"], b["s"], wq, ws, bias=bias, y=b["y"], stream=stream)
        mo.muon_linear8_weight_grad(dy, b["q"], b["s"], dw=b["dw"], stream=stream)
        mo.muon_linear8_input_grad(dy, wq, ws, dx=b["dh"], stream=stream)
        mo.muon_norm_backward(b["dh"], x, gamma, b["mean"], b["rstd"], dx=b["dx"], dgamma=b["dg"], dbeta=b["db"],
                              stream=stream)
    return run, b


@pytest.mark.parametrize("dtype", [BF, F32])
def test_calls_repeat_bit_for_bit_and_replay_from_a_graph(dtype):
    """Eager, on a side stream, on a raw stream handle, and captured in two
    graphs that share the buffers: always the same bits."""
    d = dev()
    run, b = all_calls(d, dtype=dtype)
    run()
    torch.cuda.synchronize()
    want = {k: v.clone() for k, v in b.items()}

    def same(what):
        torch.cuda.synchronize()
        for k, v in b.items():
            assert torch.equal(v, want[k]), (what, k)
            v.zero_()
        torch.cuda.synchronize()

    same("eager")
    run()
    same("again")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    run(st)
    same("stream")
    run(st.cuda_stream)
    same("raw stream")
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for g in graphs:
        with torch.cuda.graph(g):
            run()
    for v in b.values():
        v.zero_()
    for i in range(3):
        for g in graphs:
            torch.cuda.synchronize()
            g.replay()
            same(("replay", i))
        run()
        same(("eager between", i))


def test_two_streams_at_once():
    """Two sets of buffers on two streams, calls interleaved."""
    d = dev()
    sets = [all_calls(d, 900, 310, 520), all_calls(d, 520, 640, 300)]
    want = []
    for run, b in sets:
        run()
        torch.cuda.synchronize()
        want.append({k: v.clone() for k, v in b.items()})
        for v in b.values():
            v.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for (run, _b), st in zip(sets, streams):
            run(st)
    torch.cuda.synchronize()
    for (_, b), w in zip(sets, want):
        for k, v in b.items():
            assert torch.equal(v, w[k]), k


def test_workspaces_are_checked():
    d = dev()
    x, dy = matrix(300, 64, F32, 1), matrix(300, 64, F32, 2)
    one, z = torch.ones(64, device=d), torch.zeros(300, device=d)
    small = torch.empty(8, dtype=torch.uint8, device=d)
    with pytest.raises(mo.MuonError) as e:
        mo.muon_norm_backward(dy, x, one, z, z + 1, dgamma=torch.empty_like(one), workspace=small)
    assert e.value.status == -5
