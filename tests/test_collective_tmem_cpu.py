"""Tensor-memory loads, stores and their waits are instructions of a whole converged warp (`.sync.aligned`). A loop
that repeats one must bring its lanes together again after any branch that only some of them take (a partly
filled row slice), instead of leaving that to where the compiler happens to join them. Checked on the sources:
such a loop has no `continue`, `break` or `return`, and ends in `__syncwarp();` where it branches at all."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mla_decode_attention_14_b200", "csrc")
COLLECTIVE = re.compile(r"\btmem_(ld|st)\d+\(|\btmem_wait_(ld|st)\(")


def closing(text, at, pair):
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] == pair[0]) - (text[i] == pair[1])
        if depth == 0:
            return i
    raise ValueError("unbalanced %s" % pair)


def loops(text):
    """The braced bodies of the for loops that issue a collective access themselves (not through an inner loop)."""
    out = []
    for m in re.finditer(r"\bfor \(", text):
        end = closing(text, m.end() - 1, "()")
        start = re.compile(r"\s*\{").match(text, end + 1)
        if not start:
            continue
        body = text[start.end():closing(text, start.end() - 1, "{}")]
        if COLLECTIVE.search(body):
            out.append(body)
    return [b for b in out if not any(o is not b and o in b for o in out)]


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.cu"))), ids=os.path.basename)
def test_loops_around_collective_accesses_stay_converged(path):
    text = re.sub(r"//[^\n]*", "", open(path).read())
    for body in loops(text):
        inner = re.sub(r"\bif constexpr \(", "", body)
        assert not re.search(r"\b(continue|break|return)\b", inner), body
        if re.search(r"\bif \(", inner):
            assert body.rstrip().endswith("__syncwarp();"), body


def test_the_check_sees_the_loops():
    found = {os.path.basename(p): len(loops(re.sub(r"//[^\n]*", "", open(p).read()))) for p in glob.glob(os.path.join(CSRC, "*.cu"))}
    assert found["shared.cu"] == 2 and found["decode_sm100.cu"] >= 2 and found["head_gemm.cu"] == 1
    bad = "for (int c = 0; c < 8; ++c) { tmem_ld16(a, o); if (!row_ok) continue; store(o); }"
    assert len(loops(bad)) == 1 and "continue" in loops(bad)[0]
