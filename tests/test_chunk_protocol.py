"""The hand-overs of k_chunk_attn, walked through on the host in every order that its waits allow."""
import os
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp4_compressed_sparse_gb300", "csrc",
                   "csa2_chunk.cu")


def _barriers(name):
    """How many mbarriers the kernel keeps under a name."""
    text = open(SRC).read()
    m = re.search(r"uint64_t[^;]*\b" + name + r"(\[(\d+)\])?\s*[,;]", text)
    assert m, name
    return int(m.group(2) or 1)


def _stuck(tiles, n_s, n_p):
    """Whether some order of the issuing warp's and the softmax's steps leaves both waiting.  A barrier is the
    number of its completed phases; a parity wait for phase k passes while that number has k + 1's parity."""
    passed = lambda done, k: (done - k) % 2 == 1
    todo, seen = [(0, 0, False, 0, (0,) * n_s, (0,) * n_p)], set()
    while todo:
        st = todo.pop()
        if st in seen:
            continue
        seen.add(st)
        i, stage, ahead, soft, s_full, p_full = st
        nxt = []
        bump = lambda t, at: tuple(v + (k == at) for k, v in enumerate(t))
        if i < tiles:
            if stage == 0:    # S of tile i, unless it is issued already
                nxt.append((i, 1, False, soft, s_full if ahead else bump(s_full, i % n_s), p_full))
            else:
                if not ahead and i + 1 < tiles:  # the next tile is filled: its S first
                    nxt.append((i, 1, True, soft, bump(s_full, (i + 1) % n_s), p_full))
                if passed(p_full[i % n_p], i // n_p):  # P of tile i: PV, on to the next tile
                    nxt.append((i + 1, 0, ahead, soft, s_full, p_full))
        if soft < tiles and passed(s_full[soft % n_s], soft // n_s):  # S of its tile: leave P
            nxt.append((i, stage, ahead, soft + 1, s_full, bump(p_full, soft % n_p)))
        if not nxt and (i < tiles or soft < tiles):
            return True
        todo += nxt
    return False


@pytest.mark.parametrize("tiles", [1, 2, 3, 8])
def test_every_order_of_s_and_p_ends(tiles):
    assert not _stuck(tiles, _barriers("s_full"), _barriers("p_full"))


def test_the_walk_finds_a_barrier_short():
    assert _stuck(3, 2, 1) and not _stuck(3, 2, 2)


def _function(name):
    """The body of a function of the kernel's source."""
    text = open(SRC).read()
    m = re.search(r"\b" + name + r"\([^;{]*\)\s*\{", text)
    depth, at = 1, m.end()
    while depth:
        depth += {"{": 1, "}": -1}.get(text[at], 0)
        at += 1
    return text[m.end():at]


@pytest.mark.parametrize("name", ["wait_warp", "mbar_test", "ring_base"])
def test_a_warp_agrees_how_a_bounded_wait_ended(name):
    """What follows a wait that gave up differs, and has warp-wide operations: the lanes must not decide for
    themselves.  (The ahead warp's wait is one lane's alone.)"""
    assert re.search(r"__(all|any|ballot|shfl)_sync\(0xffffffffu", _function(name))


def test_shared_arrays_read_in_16_bytes_are_aligned_to_them():
    """A shared array that is read through a 16-byte type is declared with that alignment."""
    text = open(SRC).read()
    wide = set(re.findall(r"reinterpret_cast<(?:const )?(?:float4|uint4) \*>\(&?(?:sm\.)?(\w+)\[", text))
    declared = {n: line for line in text.splitlines() for n in wide
                if re.match(r"\s*(__shared__ )?(__align__\(\d+\) )?(float|float2|uint8_t) .*\b" + n + r"\[\w+\](\[\w+\])*[,;]", line)}
    assert {"wt", "sg", "plain"} <= set(declared)
    for n, line in declared.items():
        assert "__align__(16)" in line, line.strip()
