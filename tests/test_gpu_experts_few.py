"""GPU tests of every form of the few-row forward product grouped by expert
(tests/experts_cases.py, whose choice of kernels a CPU test holds), against the
fp64 reference with operands of small whole numbers: every partial sum is exact
in fp32, so results are equal to the reference rounded once."""
import numpy as np
import pytest
import torch

from oracle import experts_ref as R
from tests import experts_cases as C
from tests.gpu_util import dev, f64
from tests.test_gpu_experts import BF, F32, same, tensor

mo = pytest.importorskip("matrix_orthogonalizing_optimizer_amd")

pytestmark = pytest.mark.gpu


def offsets(counts, lead=0):
    """Offsets of groups of these sizes; the first and last `lead` rows are nobody's."""
    o = np.concatenate([[0], np.cumsum(counts)])
    return torch.from_numpy(np.clip(o, lead, o[-1] - lead).astype(np.int32)).to(dev())


@pytest.mark.parametrize("case", C.FEW, ids=lambda c: "-".join(map(str, c[:5])))
def test_few_rows(case):
    """Contiguous; rows apart, at any element of their storage; rows of nobody,
    whose results stay."""
    rows, experts, out, in_ = case[:4]
    dtype = BF if case[4] == C.BF16 else F32
    print("experts few", case, flush=True)
    for pads, shifts, lead in (((0, 0, 0), (0, 0, 0), 0), ((1, 3, 5), (1, 3, 1), 0), ((8, 8, 4), (8, 16, 4), 2)):
        off = offsets(C.counts(case), lead)
        x = tensor((rows, in_), dtype, 1, pads[0], shifts[0])
        w = tensor((experts, out, in_), dtype, 2, pads[1], shifts[1])
        for odt in (BF, F32):
            y = tensor((rows, out), odt, 3, pads[2], shifts[2])
            ref = R.forward(f64(x), f64(w), off.cpu().numpy(), f64(y))
            whole = torch.empty(0, dtype=odt, device=y.device).set_(y.untyped_storage())
            before = whole.clone()
            same(mo.muon_experts_forward(x, w, off, y=y), ref, odt, (case, pads, odt))
            # what lies around the rows and between them
            before.as_strided(y.size(), y.stride(), y.storage_offset()).copy_(y)
            assert torch.equal(before, whole), (case, pads, odt)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("in_", [128, 75])
def test_values_that_are_not_finite_stay_with_their_rows(in_, dtype):
    """NaN and infinities in a row of x, a row of w, in rows of nobody and in
    experts without rows: only the results that take them have them."""
    print("experts few not finite", in_, dtype, flush=True)
    case = next(c for c in C.FEW if c[:4] == (384, 64, 264, 128))
    n = C.counts(case)
    off = offsets(n) + 3
    x, w = tensor((390, in_), dtype, 1), tensor((64, 273, in_), dtype, 2)
    x[:3], x[387:] = float("nan"), float("inf")
    for e, k in enumerate(n):
        if k == 0:
            w[e] = float("nan")
    big, small = n.index(70), n.index(16)
    first = off.tolist()
    x[first[big] + 33, in_ - 1], x[first[small] + 15, 0] = float("nan"), float("-inf")
    w[big, 272, 5], w[small, 16, in_ - 1] = float("inf"), float("nan")
    y = torch.full((390, 273), 7.0, device=dev())
    mo.muon_experts_forward(x, w, off, y=y)
    with np.errstate(all="ignore"):
        ref = R.forward(f64(x), f64(w), off.cpu().numpy(), np.full((390, 273), 7.0))
    got = f64(y)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    ok = ~np.isnan(ref)
    assert np.array_equal(got[ok], ref[ok])
    assert (got[:3] == 7).all() and (got[387:] == 7).all()
    assert np.isfinite(ref[first[big]:first[big] + 33, :272]).all() and not np.isfinite(ref).all()


def test_graph_replays_with_other_offsets():
    """One capture of the two-tile kernel, replayed with offsets only the device
    sees: even, all rows to one expert, none, and to the last experts."""
    print("experts few graph", flush=True)
    rows, experts, out, in_ = 384, 64, 264, 136
    x, w = tensor((rows, in_), BF, 1), tensor((experts, out, in_), BF, 2)
    off = torch.zeros(experts + 1, dtype=torch.int32, device=dev())
    y = torch.zeros(rows, out, device=dev())
    mo.muon_experts_forward(x, w, off, y=y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mo.muon_experts_forward(x, w, off, y=y)
    last = [0] * 62 + [100, 200]
    for counts in ([6] * 64, [0] * 31 + [384] + [0] * 32, [0] * 64, last, C.counts(C.FEW[0])):
        off.copy_(offsets(counts))
        y.fill_(5)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        same(y, R.forward(f64(x), f64(w), off.cpu().numpy(), np.full((rows, out), 5.0)), F32, counts)
