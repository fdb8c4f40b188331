"""Compiled-code checks of the products grouped by expert and of AdamW on 8-bit
moments (no GPU needed: hipcc cross-compiles for gfx950).

- No kernel uses scratch memory, none contains packed-fp32 arithmetic or FLAT
  accesses.
- No copy to LDS sits in a waterfall loop, and none is under way at a barrier.
- The tiles' fragments are read from LDS in inline assembly, which the compiler
  does not wait for.  On every path through each kernel, no instruction touches
  the destination of an LDS read before an s_waitcnt that covers it, counting
  LDS instructions in issue order.  (Scalar loads share the counter and complete
  in any order: with one under way a wait for n leaves at most n LDS instructions,
  or fewer.)
- The tiles' kernels wait for no copy to LDS but at their barriers.
"""
import os
import re
import shutil
import subprocess

import pytest

from matrix_orthogonalizing_optimizer_amd import build as B
from tests.test_ops_code import _vregs

TILED = ["experts_y.hip", "experts_dw.hip", "experts_dx.hip", "experts_big_y.hip", "experts_big_dw.hip",
         "experts_big_dx.hip"]
SOURCES = TILED + ["experts_few.hip", "adamw8.hip"]
KERNELS = r"^(_ZN4muon\d+experts(?:_big)?_kernel\w*):(.*?)^\.Lfunc_end"


@pytest.fixture(scope="module")
def compiled(tmp_path_factory):
    h = B._hipcc()
    if not (os.path.exists(h) or shutil.which(h)):
        pytest.skip("hipcc not available")
    d = tmp_path_factory.mktemp("experts")
    made = {}

    def get(src):
        if src not in made:
            out = d / (src + ".s")
            cmd = [h] + B.hip_flags() + ["--cuda-device-only", "-S", "-o", str(out),
                                         "-Rpass-analysis=kernel-resource-usage", os.path.join(B.CSRC, src)]
            r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)
            assert r.returncode == 0, r.stderr[-2000:]
            made[src] = (out.read_text(), r.stderr)
        return made[src]
    return get


@pytest.mark.parametrize("src", SOURCES)
def test_no_scratch_and_no_packed_fp32(src, compiled):
    text, notes = compiled(src)
    names = re.findall(r"Function Name: (\S+)", notes)
    scratch = [int(x) for x in re.findall(r"ScratchSize \[bytes/lane\]: (\d+)", notes)]
    assert names and len(names) == len(scratch)
    assert not [(n, s) for n, s in zip(names, scratch) if s]
    assert not re.findall(r"\bv_pk_(?:add|mul|fma)_f32\b", text)
    assert not re.findall(r"^\s*flat_", text, flags=re.M)


@pytest.mark.parametrize("src", TILED)
def test_copies_not_in_waterfall_loops(src, compiled):
    lines = [l.split(";")[0].strip() for l in compiled(src)[0].splitlines()]
    copies = [i for i, l in enumerate(lines) if l.startswith("buffer_load") and l.endswith(" lds")]
    assert copies, "no direct-to-LDS copies found"
    for i in copies:
        window = lines[max(0, i - 4):i]
        assert not any(w.startswith("s_and_saveexec") for w in window), window + [lines[i]]


def _copies_at_barriers(text, late):
    """(barriers that a path reaches with copies to LDS under way, copies).
    late: how many stores, issued after the copies, a wait may leave."""
    body = [l.split(";")[0].strip() for l in text.splitlines()]
    body = [l for l in body if l and (not l.startswith(".") or re.match(r"\.LBB\d+_\d+:", l))]
    labels = {l[:-1]: i for i, l in enumerate(body) if l.startswith(".LBB")}
    copies = sum(l.startswith("buffer_load") and l.endswith(" lds") for l in body)
    bad, seen, stack = set(), set(), [(0, False)]
    while stack:
        pc, open_ = stack.pop()
        while pc < len(body) and (pc, open_) not in seen:
            seen.add((pc, open_))
            l = body[pc]
            if l.startswith("buffer_load") and l.endswith(" lds"):
                open_ = True
            elif l.startswith("s_waitcnt") and "vmcnt" in l:
                open_ &= int(re.search(r"vmcnt\((\d+)\)", l).group(1)) not in {0, late}
            elif l.startswith("s_barrier") and open_:
                bad.add(pc)
            elif l.startswith("s_cbranch"):
                stack.append((labels[l.split()[-1]], open_))
            elif l.startswith("s_branch"):
                pc = labels[l.split()[-1]]
                continue
            elif l.startswith("s_endpgm"):
                break
            pc += 1
    return len(bad), copies


@pytest.mark.parametrize("src", TILED)
def test_copies_to_lds_are_waited_for_at_barriers(src, compiled):
    found = 0
    for m in re.finditer(KERNELS, compiled(src)[0], re.S | re.M):
        # the stores of half a tile's strips by a wave: 8 of bf16, 16 of fp32
        late = 0 if "big" not in src else 8 if "DF16bEE" in m.group(1) else 16
        bad, copies = _copies_at_barriers(m.group(2), late)
        assert bad == 0, m.group(1)
        if copies:
            found += 1
            assert _copies_at_barriers(m.group(2).replace("vmcnt(0)", "vmcnt(1)"), late)[0] > 0
            if late:
                assert _copies_at_barriers(m.group(2), 0)[0] > 0
    assert found >= 2


def _decode(text):
    body = [l.split(";")[0].strip() for l in text.splitlines()]
    body = [l for l in body if l and (not l.startswith(".") or re.match(r"\.LBB\d+_\d+:", l))]
    labels = {l[:-1]: i for i, l in enumerate(body) if l.startswith(".LBB")}
    ins = []
    for l in body:
        op = l.split()[0]
        if l.startswith(".LBB"):
            ins.append(("label", None, l))
        elif op.startswith("ds_read"):
            dst, addr = l[len(op):].split(",")[:2]
            ins.append(("read", (_vregs(dst), _vregs(addr)), l))
        elif op.startswith("ds_"):
            ins.append(("ds", _vregs(l[len(op):]), l))
        elif op == "s_waitcnt":
            w = re.search(r"lgkmcnt\((\d+)\)", l)
            ins.append(("wait", int(w.group(1)) if w else None, l))
        elif op.startswith("s_cbranch") or op == "s_branch":
            ins.append(("branch", labels[l.split()[-1]], l))
        elif op == "s_endpgm":
            ins.append(("end", None, l))
        else:
            ins.append(("other", _vregs(l[len(op):]), l))
    return ins


def _early_uses(text):
    """Instructions that touch an LDS read's destination before a wait covers it."""
    ins = _decode(text)
    bad, seen, stack = set(), set(), [(0, ())]
    while stack:
        pc, queue = stack.pop()
        while pc < len(ins):
            kind, arg, line = ins[pc]
            if kind == "label":
                if (pc, queue) in seen:
                    break
                seen.add((pc, queue))
            elif kind == "read":
                if any(q & (arg[0] | arg[1]) for q in queue):
                    bad.add(line)
                queue += (arg[0],)
            elif kind in ("ds", "other"):
                if any(q & arg for q in queue):
                    bad.add(line)
                if kind == "ds":
                    queue += (frozenset(),)
            elif kind == "wait" and arg is not None:
                queue = queue[len(queue) - arg:] if 0 < arg < len(queue) else (() if arg == 0 else queue)
                while queue and not queue[0]:
                    queue = queue[1:]
            elif kind == "branch":
                if line.startswith("s_branch"):
                    pc = arg
                    continue
                if (arg, queue) not in seen:
                    stack.append((arg, queue))
            elif kind == "end":
                break
            pc += 1
    return bad


@pytest.mark.parametrize("src", TILED)
def test_lds_reads_are_waited_for(src, compiled):
    found = 0
    for m in re.finditer(KERNELS, compiled(src)[0], re.S | re.M):
        found += 1
        assert not _early_uses(m.group(2)), m.group(1)
        # the check sees a missing wait: with every wait loosened it reports
        assert _early_uses(re.sub(r"lgkmcnt\(\d+\)", "lgkmcnt(15)", m.group(2)))
    assert found >= 2


@pytest.mark.parametrize("src", TILED)
def test_copies_run_on_between_barriers(src, compiled):
    """In the part of a stage that issues the copies of the one after next,
    nothing waits for them: from a barrier to the branch behind the copies."""
    for m in re.finditer(KERNELS, compiled(src)[0], re.S | re.M):
        lines = [l.split(";")[0].strip() for l in m.group(2).splitlines()]
        copies = [i for i, l in enumerate(lines) if l.startswith("buffer_load") and l.endswith(" lds")]
        barriers = [i for i, l in enumerate(lines) if l.startswith("s_barrier")]
        for b in barriers:
            mine = [c for c in copies if c > b and not any(b < x < c for x in barriers)]
            if mine:
                assert not [l for l in lines[mine[0]:mine[-1]] if "vmcnt" in l], m.group(1)
