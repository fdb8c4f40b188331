"""The tiled 8-bit linear products on sizes that take each of their kernels:
128 and 256 tiles, the 8-bit operand converted on its way or expanded first,
fp32 dy cut in the product, tiles whole, split and both at once, several
K-stages and ragged ends everywhere.  tests/test_linear8_plan.py asks the
planner whether the sizes still do.

The reference is the definition in 64 bits.  Tolerances: u = 2^-24 is one fp32
rounding.  A sum of n terms in fp32 is off by at most n u sum|terms|, and its
roundings, each at most u times a partial sum that itself grows like a random
walk, reach about u sqrt(n) / 2.4 of the result in the 2-norm over a whole
matrix; the test allows 2 u sqrt(n).  The three pieces of fp32 dy are three
sums' worth of terms.  That norm is held apart for every 64 rows, so that one
wrong tile cannot drown in the others."""
import math

import pytest
import torch

from tests.gpu_util import dev
from tests.linear8_cases import CASES, DW, DX, Y

mo = pytest.importorskip("matrix_orthogonalizing_optimizer_amd")

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def kept(rows, cols, g):
    """8-bit rows with scales 2^-9 to 2^-4, and the 64-bit values they stand for."""
    store = torch.zeros(rows, (cols + 15) // 16 * 16, dtype=torch.int8, device=dev())
    store[:, :cols] = torch.randint(-127, 128, (rows, cols), generator=g, device=dev(), dtype=torch.int8)
    s = torch.ldexp(torch.ones(rows, device=dev()), torch.randint(-9, -3, (rows,), generator=g, device=dev()))
    q = store[:, :cols]
    return q, s, q.double() * s.double()[:, None]


def framed(rows, cols, dtype):
    """An output inside a wider buffer of nines."""
    buf = torch.full((rows + 1, cols + 3), 9.0, dtype=dtype, device=dev())
    return buf, buf[:rows, 1:cols + 1]


def compare(buf, out, ref, terms, n, old=None):
    """out against ref (plus old, if the call added to it)."""
    half = torch.finfo(out.dtype).eps / 2
    want = ref if old is None else ref + old
    err = (out.double() - want).abs()
    # the sum, the addition of the old value, the output's rounding
    bound = n * U * terms + U * want.abs()
    bound = bound + half * (want.abs() + bound)
    assert bool((err <= bound).all())
    for lo in range(0, out.shape[0], 64):
        rms = 2 * U * math.sqrt(n) * ref[lo:lo + 64].norm() + (half + U) * want[lo:lo + 64].norm()
        assert bool(err[lo:lo + 64].norm() <= rms), lo
    rows, cols = out.shape
    assert (buf[rows] == 9).all() and (buf[:, 0] == 9).all() and (buf[:, cols + 1:] == 9).all()


@pytest.mark.parametrize("odt", [F32, BF])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:4])))
def test_tiles(case, odt):
    print("tiles", case, odt, flush=True)
    which, t, n, k, f32, whole, _ = case
    g = torch.Generator(device="cuda").manual_seed(t + n + k)
    d = dev()
    if which == Y:
        q, s, x = kept(t, k, g)
        wq, ws, w = kept(n, k, g)
        bias = torch.randn(n, generator=g, device=d)
        buf, y = framed(t, n, odt)
        mo.muon_linear8_forward(q, s, wq, ws, bias=bias, y=y)
        prod = torch.mm(x, w.t().contiguous())
        # an exact integer sum: one rounding to fp32 and one of the bias
        compare(buf, y, prod + bias.double(), prod.abs(), 1)
        return
    pad = 0 if whole else 3
    dy = torch.randn(t, n + pad, generator=g, device=d).to(F32 if f32 else BF)[:, :n]
    left = dy.double().t().contiguous() if which == DW else dy.double()
    q, s, v = kept(t if which == DW else n, k, g)
    ref, terms = torch.mm(left, v), torch.mm(left.abs(), v.abs())
    terms_n = left.shape[1] * (3 if f32 else 1)
    buf, out = framed(left.shape[0], k, odt)
    if which == DX:
        mo.muon_linear8_input_grad(dy, q, s, dx=out)
        compare(buf, out, ref, terms, terms_n)
        return
    mo.muon_linear8_weight_grad(dy, q, s, dw=out)
    compare(buf, out, ref, terms, terms_n)
    old = out.double()
    mo.muon_linear8_weight_grad(dy, q, s, dw=out, accumulate=True)
    compare(buf, out, ref, terms, terms_n, old)
