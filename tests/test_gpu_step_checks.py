"""The binding's checks of a step's buffers: they are looked at once, in lists,
whatever form the workspace has and whichever parameters are empty, and what
is wrong is still refused by name."""
import pytest
import torch

from tests.gpu_util import dev

mo = pytest.importorskip("matrix_orthogonalizing_optimizer_amd")
binding = pytest.importorskip("matrix_orthogonalizing_optimizer_amd._lib")

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
TABLE = [(mo.MUON_KIND_MUON, mo.MUON_BF16, 40, 72, 0, 0), (mo.MUON_KIND_ADAMW, mo.MUON_F32, 1, 33, 0, 0),
         (mo.MUON_KIND_ADAMW8, mo.MUON_BF16, 7, 100, 0, 0)]
EMPTY = [(mo.MUON_KIND_MUON, mo.MUON_F32, 0, 8, 0, 0), (mo.MUON_KIND_ADAMW, mo.MUON_BF16, 3, 0, 0, 0),
         (mo.MUON_KIND_ADAMW8, mo.MUON_BF16, 0, 5, 0, 0)]


def buffers(table, seed, missing=False):
    """params, grads, moms, exp_avgs, exp_avg_sqs; missing: None for what belongs to
    a parameter without elements."""
    g = torch.Generator().manual_seed(seed)
    lists = [[], [], [], [], []]
    for kind, dt, r, c, _, _ in table:
        own = F32 if dt == mo.MUON_F32 else BF
        none = missing and r * c == 0
        for k in (0, 1):
            lists[k].append(None if none else torch.randn(r, c, generator=g).to(own).to(dev()))
        for k in (2, 3, 4):
            if none or (k == 2) != (kind == mo.MUON_KIND_MUON):
                lists[k].append(None)
            elif kind == mo.MUON_KIND_ADAMW8:
                lists[k].append(torch.zeros(mo.muon_adamw8_state_bytes(r * c), dtype=torch.uint8, device=dev()))
            else:
                lists[k].append(torch.zeros(r, c, device=dev()))
    return lists


@pytest.fixture
def looked_at(monkeypatch):
    """How many buffers the binding checked one by one."""
    seen = []
    for f in ("_check_buffer", "_check_moment8"):
        real = getattr(binding, f)
        monkeypatch.setattr(binding, f, lambda *a, real=real: (seen.append(a[0]), real(*a))[1])
    return seen


def workspace(plan):
    return torch.empty(max(1, mo.muon_plan_workspace_bytes(plan)), dtype=torch.uint8, device=dev())


def results(table, lists, form):
    plan = mo.muon_plan_create(table)
    ws = workspace(plan)
    mo.muon_step(plan, *lists, mo.make_hparams(), form(ws))
    torch.cuda.synchronize()
    return [t for k in (0, 2, 3, 4) for t, (_, _, r, c, _, _) in zip(lists[k], table) if t is not None and r * c]


FORMS = {"tensor": lambda ws: ws, "address": lambda ws: (ws.data_ptr(), ws.numel())}


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("empty", ["none", "missing", "there"])
def test_buffers_are_looked_at_once(form, empty, looked_at):
    print("step checks", form, empty, flush=True)
    want = results(TABLE, buffers(TABLE, 1), FORMS["tensor"])
    looked_at.clear()
    table = TABLE if empty == "none" else TABLE + EMPTY
    got = results(table, buffers(table, 1, empty == "missing"), FORMS[form])
    assert looked_at == []
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_step_without_a_workspace(looked_at):
    print("step checks, no workspace", flush=True)
    table = TABLE[2:] + EMPTY[2:]
    lists = buffers(table, 2, True)
    plan = mo.muon_plan_create(table)
    assert mo.muon_plan_workspace_bytes(plan) == 0
    mo.muon_step(plan, *lists, mo.make_hparams(), None)
    torch.cuda.synchronize()
    assert looked_at == [] and lists[3][0].any()


@pytest.mark.parametrize("where", range(len(TABLE + EMPTY)))
def test_wrong_buffers_are_refused_by_name(where):
    print("step checks, refusals", where, flush=True)
    table = TABLE + EMPTY
    plan = mo.muon_plan_create(table)
    ws, hp = workspace(plan), mo.make_hparams()
    kind, _, r, c, _, _ = table[where]
    names = ["params", "grads"] + (["moms"] if kind == mo.MUON_KIND_MUON else ["exp_avgs", "exp_avg_sqs"])
    for name in names:
        k = ["params", "grads", "moms", "exp_avgs", "exp_avg_sqs"].index(name)
        for change in (lambda t: t.to(torch.float16), lambda t: torch.zeros(t.numel() + 1, dtype=t.dtype, device=t.device),
                       lambda t: t.cpu()):
            lists = buffers(table, 3)
            lists[k][where] = change(lists[k][where])
            # on the host: refused before the names are looked at
            match = r"muon_step" if not lists[k][where].is_cuda else rf"{name}\[{where}\]"
            for form in FORMS.values():
                with pytest.raises(ValueError, match=match):
                    mo.muon_step(plan, *lists, hp, form(ws))
    lists = buffers(table, 3)
    if r * c:
        lists[0][where] = None
        with pytest.raises(mo.MuonError):
            mo.muon_step(plan, *lists, hp, ws)


def test_wrong_workspaces_are_refused():
    print("step checks, workspaces", flush=True)
    plan = mo.muon_plan_create(TABLE)
    lists, hp = buffers(TABLE, 4), mo.make_hparams()
    before = [t.clone() for k in lists for t in k if t is not None]
    ws = workspace(plan)
    need = mo.muon_plan_workspace_bytes(plan)
    with pytest.raises(ValueError):
        mo.muon_step(plan, *lists, hp, ws.cpu())
    for bad in (ws[:need - 1], (ws.data_ptr(), need - 1), (None, need), None):
        with pytest.raises(mo.MuonError):
            mo.muon_step(plan, *lists, hp, bad)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before, (t for k in lists for t in k if t is not None)))
