"""Rows that the row operators read again for every pass (norm forward above
16384 columns, backward above 8192), in place: a row's last piece reaches past
its end, and must not depend on what its neighbour's thread writes."""
import pytest
import torch

from oracle import ops_ref as R
from tests.gpu_util import dev, f64

mo = pytest.importorskip("matrix_orthogonalizing_optimizer_amd")

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def rnd(seed, *shape, dtype):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(dev())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("cols", [8193, 8199, 12300, 16385, 16390, 20007, 24576, 24577, 24585, 33001])
def test_in_place_is_what_it_is_out_of_place(cols, layer, dtype):
    print("long rows in place", cols, layer, dtype, flush=True)
    rows, kind = 300, mo.MUON_NORM_LAYER if layer else mo.MUON_NORM_RMS
    x, dy = rnd(1, rows, cols, dtype=dtype), rnd(2, rows, cols, dtype=dtype)
    gamma, beta = rnd(3, cols, dtype=dtype), rnd(4, cols, dtype=dtype)
    mean = torch.empty(rows, device=dev()) if layer else None
    rstd = torch.empty(rows, device=dev())
    y, z = torch.empty_like(x), x.clone()
    q = torch.full((rows, (cols + 15) // 16 * 16), 7, dtype=torch.int8, device=dev())
    s = torch.empty(rows, device=dev())
    mo.muon_norm_forward(x, gamma, beta, kind=kind, y=y, mean=mean, rstd=rstd)
    mo.muon_norm_forward(z, gamma, beta, kind=kind, y=z, q=q[:, :cols], scale=s)
    assert torch.equal(z, y)
    assert not q[:, cols:].any()
    # the 8-bit rows are of y before its rounding: within half a step and that rounding
    ry = f64(y[:5])
    half = torch.finfo(dtype).eps / 2
    err = abs(R.restore(q[:5, :cols].cpu().numpy(), f64(s[:5])) - ry)
    assert (err <= f64(s[:5])[:, None] / 2 * (1 + 2 ** -20) + 2 * half * abs(ry)).all()
    dx = mo.muon_norm_backward(dy, x, gamma, mean, rstd, kind=kind)
    d = dy.clone()
    mo.muon_norm_backward(d, x, gamma, mean, rstd, kind=kind, dx=d)
    assert torch.equal(d, dx)
