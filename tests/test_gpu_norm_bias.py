"""The bias gradient of RMS norms: the forward pass takes a bias, so the
backward pass gives its gradient, written or added, at the widths of every
kernel, and leaves dx and the weight gradient as they are without it."""
import numpy as np
import pytest
import torch

from oracle import ops_ref as R
from tests.gpu_util import dev, f64

mo = pytest.importorskip("matrix_orthogonalizing_optimizer_amd")

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def rnd(seed, *shape, dtype):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(dev())


@pytest.mark.parametrize("dtype,vec", [(BF, BF), (F32, F32), (BF, F32)])
@pytest.mark.parametrize("rows,cols", [(1, 1), (2050, 57), (700, 200), (300, 510), (130, 768), (700, 1001), (300, 2048),
                                       (600, 4097), (33, 8191), (40, 8200), (9, 14336)])
def test_rms_norm_bias_gradient(rows, cols, dtype, vec):
    print("rms bias", rows, cols, dtype, vec, flush=True)
    x, dy = rnd(1, rows, cols, dtype=dtype), rnd(2, rows, cols, dtype=dtype)
    gamma, beta = rnd(3, cols, dtype=vec), rnd(4, cols, dtype=vec)
    rstd, y = torch.empty(rows, device=dev()), torch.empty_like(x)
    mo.muon_norm_forward(x, gamma, beta, kind=mo.MUON_NORM_RMS, y=y, rstd=rstd)
    rx, rg, rb = R.norm_backward(f64(dy), f64(x), f64(gamma), None, f64(rstd), layer=False)
    plain_g, dg = torch.empty_like(gamma), torch.empty_like(gamma)
    plain_x = mo.muon_norm_backward(dy, x, gamma, None, rstd, kind=mo.MUON_NORM_RMS, dgamma=plain_g)
    half = torch.finfo(vec).eps / 2
    # rows in order inside a workgroup, at most 32 of them joined, then at most
    # 512 workgroups in 16 groups
    bound = (rows // 256 + 1 + 32 + 32 + 16) * U * np.abs(f64(dy)).sum(axis=0)
    for acc in (False, True):
        db = beta.clone()
        dx = mo.muon_norm_backward(dy, x, gamma, None, rstd, kind=mo.MUON_NORM_RMS, dgamma=None if acc else dg,
                                   dbeta=db, accumulate=acc)
        assert torch.equal(dx, plain_x)
        want = rb + (f64(beta) if acc else 0.0)
        b = bound + U * np.abs(want)
        assert (np.abs(f64(db) - want) <= b + half * (np.abs(want) + b)).all()
        assert acc or torch.equal(dg, plain_g)
    # no rows: the sums are zero, or what was there
    db = beta.clone()
    empty = lambda **kw: mo.muon_norm_backward(dy[:0], x[:0], gamma, None, rstd[:0], kind=mo.MUON_NORM_RMS, **kw)
    empty(dbeta=db, accumulate=True)
    assert torch.equal(db, beta)
    empty(dbeta=db)
    assert not db.any()
