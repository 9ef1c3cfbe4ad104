"""Block barriers of the kernels and the waits that may give up, read from the sources: a bounded wait may end
differently in two warps, so no barrier of the block may hang on its outcome, unless the block has voted on it
(__syncthreads_and / __syncthreads_or)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp4_compressed_sparse_gb300", "csrc")
WAITS = re.compile(r"\b(mbar_wait_bounded|mbar_try_wait|wait_all)\b")
VOTE = re.compile(r"__syncthreads_(and|or|count)\b")
BARRIER = re.compile(r"__syncthreads\w*\s*\(|\bcluster_sync\s*\(|\"bar\.sync")
ASSIGNED = re.compile(r"\b(\w+)\s*(?:&|\|)?=(?!=)\s*([^;]*);")


def _kernels(text):
    """(name, body) of every __global__ function, comments taken out."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"__global__[^;{]*?\b(k_\w+)\s*\(", text):
        at = text.index("{", m.end())
        end, depth = at, 0
        while True:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
            if depth == 0:
                break
        yield m.group(1), text[at:end]


def _conditions(body, at):
    """The conditions of the if statements that `at` stands under."""
    out, depth, pos = [], 0, at
    while pos > 0:
        pos -= 1
        depth += {"}": 1, "{": -1}.get(body[pos], 0)
        if depth >= 0:
            continue
        depth = 0  # the opening of a block around `at`
        head = body[:pos].rstrip()
        if head.endswith(")"):
            i, p = len(head) - 1, 0
            while True:
                p += {")": 1, "(": -1}.get(head[i], 0)
                if p == 0:
                    break
                i -= 1
            if re.search(r"\bif\s*(constexpr\s*)?$", head[:i]):
                out.append(head[i:])
    head = body[:at].rstrip()  # a statement without braces
    m = re.search(r"\bif\s*(\([^;{}]*\))$", head)
    return out + ([m.group(1)] if m else [])


def _unvoted(body, at):
    """Names whose last assignment before `at` is the outcome of a wait, or of such a name."""
    names = set()
    for m in ASSIGNED.finditer(body[:at]):
        name, value = m.groups()
        if VOTE.search(value):
            names.discard(name)
        elif WAITS.search(value) or names & set(re.findall(r"\w+", value)):
            names.add(name)
        # (another assignment may stand in another branch: it clears nothing)
    return names


def _hanging(text):
    found = []
    for name, body in _kernels(text):
        for m in BARRIER.finditer(body):
            bad = _unvoted(body, m.start())
            for cond in _conditions(body, m.start()):
                if not VOTE.search(cond) and (WAITS.search(cond) or bad & set(re.findall(r"\w+", cond))):
                    found.append((name, cond))
    return found


@pytest.mark.parametrize("src", sorted(os.path.basename(f) for f in glob.glob(os.path.join(CSRC, "*.cu"))))
def test_no_barrier_under_a_wait_that_may_give_up(src):
    assert not _hanging(open(os.path.join(CSRC, src)).read())


def test_the_reading_finds_such_a_barrier():
    kernel = """__global__ void k_x(int *p) { int ok = 1; if (lane == 0) ok = mbar_wait_bounded(&b, 0, 9);
      bool have = __shfl_sync(~0u, ok, 0) != 0; __syncthreads(); VOTE if (!have) { if (t == 0) f(); __syncthreads(); } }"""
    assert _hanging(kernel.replace("VOTE", "")) == [("k_x", "(!have)")]
    assert not _hanging(kernel.replace("VOTE", "have = __syncthreads_and(have);"))
    assert _hanging("__global__ void k_y() { bool ok = wait_all(b, 0); if (!ok) __syncthreads(); }")
