"""Compiled-code checks of the operators around the step (no GPU needed:
hipcc cross-compiles for gfx950).

- No kernel uses scratch memory, none contains packed-fp32 arithmetic or FLAT
  accesses (those also count in lgkmcnt).
- No buffer access sits in a waterfall loop: a resource that the compiler takes
  for divergent costs a loop around every load.
- The transposed LDS reads of the gradient products are written in inline
  assembly, which the compiler does not wait for.  On every path through each
  kernel, no instruction touches the destination of such a read before an
  s_waitcnt that covers it, counting LDS instructions in issue order; and no
  scalar load, which shares the counter and completes out of order, is under
  way together with one.
- No copy to LDS is under way at a barrier: the waves behind it read what the
  others copied.
"""
import os
import re
import shutil
import subprocess

import pytest

from matrix_orthogonalizing_optimizer_amd import build as B

SOURCES = ["row_ops.hip", "linear8_y.hip", "linear8_dw.hip", "linear8_dx.hip"]


@pytest.fixture(scope="module")
def compiled(tmp_path_factory):
    h = B._hipcc()
    if not (os.path.exists(h) or shutil.which(h)):
        pytest.skip("hipcc not available")
    d = tmp_path_factory.mktemp("ops")
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


@pytest.mark.parametrize("src", SOURCES[1:])
def test_buffer_accesses_not_in_waterfall_loops(src, compiled):
    lines = [l.split(";")[0].strip() for l in compiled(src)[0].splitlines()]
    accesses = [i for i, l in enumerate(lines) if l.startswith(("buffer_load", "buffer_store"))]
    assert any(lines[i].endswith(" lds") for i in accesses), "no direct-to-LDS copies found"
    for i in accesses:
        window = lines[max(0, i - 4):i]
        assert not any(w.startswith("s_and_saveexec") for w in window), window + [lines[i]]


def _vregs(text):
    out = set()
    for a, b, c in re.findall(r"\bv\[(\d+):(\d+)\]|\bv(\d+)\b", text):
        out |= {int(c)} if c else set(range(int(a), int(b) + 1))
    return frozenset(out)


def _decode(text):
    body = [l.split(";")[0].strip() for l in text.splitlines()]
    body = [l for l in body if l and (not l.startswith(".") or re.match(r"\.LBB\d+_\d+:", l))]
    labels = {l[:-1]: i for i, l in enumerate(body) if l.startswith(".LBB")}
    ins = []
    for l in body:
        op = l.split()[0]
        if l.startswith(".LBB"):
            ins.append(("label", None, l))
        elif op.startswith("ds_read_b64_tr"):
            dst, addr = l[len(op):].split(",")[:2]
            ins.append(("tr", (_vregs(dst), _vregs(addr)), l))
        elif op.startswith("ds_"):
            ins.append(("ds", _vregs(l[len(op):]), l))
        elif op == "s_waitcnt":
            w = re.search(r"lgkmcnt\((\d+)\)", l)
            ins.append(("wait", int(w.group(1)) if w else None, l))
        elif op.startswith("s_cbranch") or op == "s_branch":
            ins.append(("branch", labels[l.split()[-1]], l))
        elif op == "s_endpgm":
            ins.append(("end", None, l))
        elif op.startswith(("s_load", "s_buffer_load")):
            ins.append(("scalar", None, l))
        else:
            ins.append(("other", _vregs(l[len(op):]), l))
    return ins


def _untracked_uses(text):
    """Instructions that touch a transposed read's destination too early."""
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
            elif kind == "tr":
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
            elif kind == "scalar":
                if any(queue):
                    bad.add(line)
            elif kind == "end":
                break
            pc += 1
    return bad


@pytest.mark.parametrize("src", ["linear8_dw.hip", "linear8_dx.hip"])
def test_transposed_reads_are_waited_for(src, compiled):
    found = 0
    for m in re.finditer(r"^(_ZN4muon14linear8_kernel\w*):(.*?)^\.Lfunc_end", compiled(src)[0], re.S | re.M):
        if "ds_read_b64_tr" not in m.group(2):
            continue
        found += 1
        assert not _untracked_uses(m.group(2)), m.group(1)
        # the check sees a missing wait: with every wait loosened it reports
        loose = re.sub(r"lgkmcnt\(\d+\)", "lgkmcnt(15)", m.group(2))
        assert _untracked_uses(loose)
    assert found >= 6


def _copies_at_barriers(text):
    """Barriers with copies to LDS under way, in the order of the text (which a
    loop of these kernels enters with its copies behind the barrier)."""
    open_, bad, copies = False, 0, 0
    for l in (l.split(";")[0].strip() for l in text.splitlines()):
        if l.startswith("buffer_load") and l.endswith(" lds"):
            open_, copies = True, copies + 1
        elif l.startswith("s_waitcnt") and "vmcnt(0)" in l:
            open_ = False
        elif l.startswith("s_barrier") and open_:
            bad += 1
    return bad, copies


@pytest.mark.parametrize("src", SOURCES[1:])
def test_copies_to_lds_are_waited_for_at_barriers(src, compiled):
    found = 0
    for m in re.finditer(r"^(_ZN4muon14linear8_kernel\w*):(.*?)^\.Lfunc_end", compiled(src)[0], re.S | re.M):
        bad, copies = _copies_at_barriers(m.group(2))
        assert bad == 0, m.group(1)
        if copies:
            found += 1
            assert _copies_at_barriers(m.group(2).replace("vmcnt(0)", "vmcnt(1)"))[0] > 0
    assert found >= 4
