"""The forward product of the 8-bit linear layer over the whole range of the
scales that 8-bit rows may have (2^-126 to 2^122): what is finite comes out
finite, whatever the order of the factors, on every path of the product."""
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
# few-token kernels of 1, 2 and 4 tiles, and of 4 channel groups; 128 tiles whole
# and split; 256 tiles whole and split
PATHS = [(3, 50, 4096), (20, 70, 300), (50, 40, 1000), (5, 16390, 900), (200, 130, 600), (300, 200, 5000),
         (4100, 2100, 500), (1000, 4360, 6800)]


def kept(rows, cols, seed):
    store = torch.zeros(rows, (cols + 15) // 16 * 16, dtype=torch.int8)
    g = torch.Generator().manual_seed(seed)
    store[:, :cols] = torch.randint(-127, 128, (rows, cols), generator=g, dtype=torch.int8)
    store[0, :cols] = 127  # the largest sums
    return store.to(dev())[:, :cols]


def powers(n, lo, hi, seed):
    e = torch.randint(lo, hi + 1, (n,), generator=torch.Generator().manual_seed(seed))
    return torch.ldexp(torch.ones(n), e).to(dev())


@pytest.mark.parametrize("dtype,bias", [(F32, False), (BF, True)])
@pytest.mark.parametrize("tok,ch", [((90, 122), (-126, -90)), ((-126, -90), (90, 122)), ((-20, 20), (-20, 20))])
@pytest.mark.parametrize("t,n,k", PATHS)
def test_no_early_overflow(t, n, k, tok, ch, dtype, bias):
    print("scales", t, n, k, tok, ch, dtype, flush=True)
    q, wq = kept(t, k, 1), kept(n, k, 2)
    s, ws = powers(t, *tok, 3), powers(n, *ch, 4)
    b = torch.randn(n, generator=torch.Generator().manual_seed(5)).to(dev()) if bias else None
    y = mo.muon_linear8_forward(q, s, wq, ws, bias=b, dtype=dtype)
    assert torch.isfinite(y).all()
    prod = R.linear8_forward(q.cpu().numpy(), f64(s), wq.cpu().numpy(), f64(ws))
    ref = prod + (f64(b) if bias else 0.0)
    # the integer sum is rounded to fp32 once, powers of two round nothing (the
    # results are at least 2^-36), then the bias and the output's type
    bound = U * np.abs(prod) + U * np.abs(ref)
    bound = bound + torch.finfo(dtype).eps / 2 * (np.abs(ref) + bound)
    assert (np.abs(f64(y) - ref) <= bound).all()


@pytest.mark.parametrize("t,n,k", PATHS)
def test_true_overflow_and_nan(t, n, k):
    """Results past fp32's range are infinite, sums of zero are zero under the
    largest scales, and a NaN scale spoils its row or column only."""
    print("overflow", t, n, k, flush=True)
    q, wq = kept(t, k, 1), kept(n, k, 2)
    wq[1:] = wq[0]
    q[1] = 0
    s, ws = torch.full((t,), 2.0 ** 122, device=dev()), torch.full((n,), 2.0 ** 100, device=dev())
    s[2], ws[3] = math.nan, math.nan
    y = mo.muon_linear8_forward(q, s, wq, ws, dtype=F32)
    cols = [c for c in range(n) if c != 3]
    assert (y[0, cols] == math.inf).all() and (y[1, cols] == 0).all()
    assert torch.isnan(y[2]).all() and torch.isnan(y[:, 3]).all()
    assert not torch.isnan(y[[r for r in range(t) if r != 2]][:, cols]).any()


@pytest.mark.parametrize("t", [1, 5, 40, 200, 5000])
def test_no_channels_in_is_the_bias(t):
    """A sum of nothing is zero whatever the scales hold; the norm of rows
    without columns leaves them as they are."""
    n = 300
    x = torch.zeros(t, 16, dtype=BF, device=dev())[:, :0]
    q = torch.empty(t, 16, dtype=torch.int8, device=dev())[:, :0]
    s, ws = torch.full((t,), math.nan, device=dev()), torch.full((n,), math.inf, device=dev())
    rstd = torch.full((t,), 5.0, device=dev())
    mo.muon_norm_forward(x, torch.ones(0, dtype=BF, device=dev()), q=q, scale=s, rstd=rstd)
    assert torch.isnan(s).all() and (rstd == 5).all()
    wq = torch.empty(n, 16, dtype=torch.int8, device=dev())[:, :0]
    b = torch.randn(n, generator=torch.Generator().manual_seed(5)).to(dev())
    for dtype in (F32, BF):
        assert torch.equal(mo.muon_linear8_forward(q, s, wq, ws, bias=b, dtype=dtype), b.to(dtype).expand(t, n))
        assert (mo.muon_linear8_forward(q, s, wq, ws, dtype=dtype) == 0).all()
