"""Results of the matrix cores are waited for: in the linear layer's kernels as
compiled, no way from a matrix instruction reaches another use of its result's
registers, or one of its operands' own in a later one, before eight instructions
have gone by (CPU only: the sources are compiled to assembly, which is read).

The hardware does not wait by itself, and the compiler has been seen to leave the
waits out where a branch lies between the two."""
import re

import pytest

from test_linear_lds_order import SOURCES, kernels, listings  # noqa: F401

WAIT = 8                                 # of 16×16×32 products of 16 bits, as the compiler waits on straight ways


def registers(operand):
    m = re.match(r"-?\|?([va])\[(\d+):(\d+)\]", operand)
    if m:
        return {m[1] + str(i) for i in range(int(m[2]), int(m[3]) + 1)}
    m = re.match(r"-?\|?([va]\d+)\b", operand)
    return {m[1]} if m else set()


def early(code):
    """(matrix instruction, use, instructions between) of uses that come too early."""
    at = {line[:-1]: i for i, line in enumerate(code) if line.endswith(":")}
    split = [(line.split(None, 1) + [""])[:2] for line in code]
    split = [(op, [x.strip() for x in rest.split(",")]) for op, rest in split]
    bad = []
    for first, (op, operands) in enumerate(split):
        if not op.startswith("v_mfma"):
            continue
        out, seen, ways = registers(operands[0]), {}, [(first + 1, 0)]
        while ways:
            i, gone = ways.pop()
            if i >= len(code) or gone >= WAIT or seen.get(i, WAIT) <= gone:
                continue
            seen[i] = gone
            op, operands = split[i]
            if op.endswith(":"):
                ways.append((i + 1, gone))
                continue
            if op.startswith("v_mfma"):
                if (registers(operands[1]) | registers(operands[2])) & out:
                    bad.append((code[first], code[i], gone))
                if registers(operands[0]) != out:          # else it is that one's to be waited for
                    ways.append((i + 1, gone + 1))
                continue
            if out & set().union(*(registers(x) for x in operands)):
                bad.append((code[first], code[i], gone))
                continue
            if op == "s_endpgm":
                continue
            gone += int(operands[0], 0) + 1 if op == "s_nop" else 1
            if op.startswith(("s_branch", "s_cbranch")):
                ways.append((at[operands[0]], gone))
            if op != "s_branch":
                ways.append((i + 1, gone))
    return bad


def test_the_walk_itself():
    mfma, read = "v_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[4:7], a[0:3]", "v_accvgpr_read_b32 v9, a3"
    assert early([mfma, "s_nop 6", read]) and not early([mfma, "s_nop 7", read])
    assert early([mfma, "s_cbranch_scc1 .LBB0_1", "s_nop 7", ".LBB0_1:", read])
    assert not early([mfma, "s_cbranch_scc1 .LBB0_1", "s_endpgm", ".LBB0_1:", "s_nop 7", read])
    assert not early([mfma, mfma, "s_nop 7", read]) and not early([mfma, "v_mov_b32_e32 v9, v8"])
    assert early([mfma, "v_mfma_f32_16x16x32_bf16 v[8:11], a[0:3], v[4:7], v[8:11]"])
    assert early([".LBB0_0:", read, mfma, "s_branch .LBB0_0"])


@pytest.mark.parametrize("source", SOURCES)
def test_every_result_is_waited_for(listings, source):  # noqa: F811
    found = {name: early(code) for name, code in kernels(listings[source]).items()}
    assert not {name: bad for name, bad in found.items() if bad}
