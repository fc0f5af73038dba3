"""Writes to LDS are in before the other waves go on: in the linear layer's
kernels as compiled, every way from an LDS write to the next barrier passes a
wait for it (CPU only: the sources are compiled to assembly, which is read).

A barrier does not wait for LDS writes by itself.  The compiler sees to its own;
those written as inline assembly, or made where a wave then skips the reads that
would have waited, are the source's to wait for."""
import os
import re
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "half_precision_gemm_amd", "csrc")
# In hg_linear_outer.hip no other wave and no load touches what a wave writes: there is nothing to wait for.
SOURCES = sorted(f for f in os.listdir(CSRC) if re.fullmatch(r"hg_linear_(?!outer).*\.hip", f))


@pytest.fixture(scope="module")
def listings(hg, tmp_path_factory):
    """{source: its assembly}."""
    from half_precision_gemm_amd import build
    folder = tmp_path_factory.mktemp("asm")

    def compile(source):
        out = folder / (source + ".s")
        r = subprocess.run([build.HIPCC] + build.FLAGS + ["--offload-device-only", "-S", os.path.join(CSRC, source),
                                                          "-o", str(out)], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        return out.read_text()

    with ThreadPoolExecutor(4) as pool:
        return dict(zip(SOURCES, pool.map(compile, SOURCES)))


def kernels(asm):
    """{name: its instructions and labels} of an assembly listing."""
    out, name = {}, None
    for line in asm.splitlines():
        line = line.split(";")[0].rstrip()
        if re.match(r"_Z\w+:", line):
            name = line[:-1]
            out[name] = []
        elif re.match(r"\.Lfunc_end", line):
            name = None
        elif name and (line.startswith("\t") and not line.startswith("\t.") or re.match(r"\.LBB\w+:", line)):
            out[name] += [line.strip()]
    return out


def unwaited(code):
    """(write, barrier) line numbers of a way from an LDS write to a barrier without a wait for the write.

    LDS operations of a wave complete in order, so that a wait that leaves n of them outstanding covers a write that
    at least n others follow."""
    at = {line[:-1]: i for i, line in enumerate(code) if line.endswith(":")}
    for first, line in enumerate(code):
        if not line.startswith("ds_write"):
            continue
        seen, todo = set(), [(first + 1, 0)]
        while todo:
            i, after = todo.pop()
            while (i, after) not in seen:
                seen.add((i, after))
                op = code[i].split()
                if op[0] == "s_barrier":
                    return first, i
                if op[0] == "s_endpgm":
                    break
                if op[0] == "s_waitcnt":
                    n = re.search(r"lgkmcnt\((\d+)\)", code[i])
                    if n and int(n[1]) <= after:
                        break
                if op[0].startswith("ds_"):
                    after = min(after + 1, 15)
                if op[0] in ("s_setpc_b64", "s_swappc_b64"):
                    raise AssertionError(f"{op[0]}: a way this test does not follow")
                if op[0].startswith(("s_branch", "s_cbranch")):
                    todo.append((at[op[1]], after))
                    if op[0] == "s_branch":
                        break
                i += 1
    return None


def test_the_walk_itself():
    assert unwaited(["ds_write_b32 v0, v1", "s_barrier", "s_endpgm"]) == (0, 1)
    assert unwaited(["ds_write_b32 v0, v1", "s_waitcnt lgkmcnt(0)", "s_barrier", "s_endpgm"]) is None
    assert unwaited(["ds_write_b32 v0, v1", "s_waitcnt vmcnt(0)", "s_barrier", "s_endpgm"]) == (0, 2)
    assert unwaited(["ds_write_b32 v0, v1", "ds_read_b32 v2, v0", "s_waitcnt lgkmcnt(1)", "s_barrier", "s_endpgm"]) is None
    skip = ["ds_write_b32 v0, v1", "s_cbranch_scc1 .L1", "s_waitcnt lgkmcnt(0)", ".L1:", "s_barrier", "s_endpgm"]
    assert unwaited(skip) == (0, 4)
    loop = [".L0:", "s_barrier", "ds_write_b32 v0, v1", "s_cbranch_scc1 .L0", "s_endpgm"]
    assert unwaited(loop) == (2, 1)


@pytest.mark.parametrize("source", SOURCES)
def test_every_lds_write_is_waited_for(listings, source):
    found = kernels(listings[source])
    assert found
    bad = {name: (where, code[where[0]]) for name, code in found.items() if (where := unwaited(code))}
    assert not bad, bad
