"""Gradients of the 8-bit linear layer for dy down to the smallest numbers of
its type: fp32 dy counts with every bit from 2^-110 up and with its bits from
2^-133 up below, bf16 dy with all of them; numbers below the normal range are
not taken for zero."""
import pytest
import torch

from tests.gpu_util import dev

mo = pytest.importorskip("matrix_orthogonalizing_optimizer_amd")

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def kept(rows, cols, g):
    store = torch.zeros(rows, (cols + 15) // 16 * 16, dtype=torch.int8, device=dev())
    store[:, :cols] = torch.randint(-127, 128, (rows, cols), generator=g, device=dev(), dtype=torch.int8)
    s = torch.ldexp(torch.ones(rows, device=dev()), torch.randint(-3, 3, (rows,), generator=g, device=dev()))
    return store[:, :cols], s, store[:, :cols].double() * s.double()[:, None]


# fp32 dy cut in the product; laid out as planes (128 and 256 tiles)
@pytest.mark.parametrize("t,n,k", [(70, 37, 50), (222, 8555, 195), (300, 2100, 2300), (1357, 399, 5614)])
@pytest.mark.parametrize("lo,hi", [(-110, -100), (-140, -111)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_small_dy(t, n, k, lo, hi, dtype):
    print("small dy", t, n, k, lo, hi, dtype, flush=True)
    g = torch.Generator(device="cuda").manual_seed(t + n + k)
    # magnitudes from 2^lo to 2^(hi + 1)
    e = torch.randint(lo, hi + 1, (t, n), generator=g, device=dev())
    m = 1 + torch.rand(t, n, generator=g, device=dev(), dtype=torch.float64)
    sign = torch.randint(0, 2, (t, n), generator=g, device=dev()) * 2 - 1
    dy = (torch.ldexp(m, e) * sign).to(dtype)
    d64 = dy.double()
    assert bool((d64 != 0).any())
    # what a value of fp32 may lose; bf16 and larger values lose nothing
    lost = (d64.abs() < 2.0 ** -110).double() * (2.0 ** -133 if dtype == F32 else 0.0)
    pieces = 3 if dtype == F32 else 1
    for name, call, rows in (("dW", mo.muon_linear8_weight_grad, t), ("dX", mo.muon_linear8_input_grad, n)):
        q, s, v = kept(rows, k, g)
        left, cut = (d64.t().contiguous(), lost.t().contiguous()) if name == "dW" else (d64, lost)
        ref, terms = torch.mm(left, v), torch.mm(left.abs(), v.abs())
        # 32-bit sums of all pieces' terms, each rounding relative or, below the
        # normal range, half of 2^-149; and what the pieces lack
        N = pieces * rows + 16
        bound = N * U * terms + N * 2.0 ** -150 + torch.mm(cut, v.abs())
        got = call(dy, q, s, dtype=F32).double()
        over = (got - ref).abs() - bound
        assert bool((over <= U * ref.abs()).all()), (name, float(over.max()))
