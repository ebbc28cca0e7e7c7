"""The orders that the kernel of packed rows' attention relies on, on its rings as its
source has them: an entry of a ring is written again only behind its last read.

A key block k of a CTA is copied (keys, and the word that says which of them lie in
pages), multiplied with each block of rows that the tile has (S), read by that block's
softmax (the word too), and its values are copied and multiplied (P V). The waits
between these steps are the edges of a graph; a read that no path orders ahead of the
next write to its entry is a race.
"""

import os
import random
import re

import pytest

from quantized_moe_transformer_gb300 import build


def source():
    with open(os.path.join(build.CSRC, "paged_prefill.cu")) as f:
        return f.read()


def value(text, names):
    """A C expression of names, comparisons and conditions."""
    if "?" in text:
        condition, rest = text.split("?", 1)
        yes, no = rest.split(":", 1)
        return value(yes, names) if value(condition, names) else value(no, names)
    text = text.replace("&&", " and ").replace("||", " or ").replace("C::", "")
    return eval(text, {"__builtins__": {}}, dict(names))


def rings(hdp, f32):
    """(stages of keys, of values, words) of the kernel of ``hdp`` padded head dims."""
    s = source()
    names = {"HDP": hdp, "F32": f32}
    for text in re.findall(r"static constexpr int ([^;]*);", s):
        for part in text.split(","):
            name, _, v = part.partition("=")
            if name.strip() in ("KST", "VST", "RING"):
                names[name.strip()] = value(v, names)
    words = value(re.search(r"__shared__ uint32_t there\[([^\]]*)\]", s).group(1), names)
    return names["KST"], names["VST"], words


def unordered(kst, vst, words, second, free="PV0"):
    """Pairs (k, block of rows) whose word may be overwritten unread. ``second[k]``: the tile of
    key block k has a second block of rows; ``free``: the step that gives S's buffer back."""
    n = len(second)
    behind = {}  # event -> the events that it comes behind

    def event(name, k, *after):
        have = set()
        for e in after:
            if e in behind:
                have |= behind[e] | {e}
        behind[name, k] = have

    own = [k for k in range(n) if second[k]]
    before = {k: own[i - 1] if i else -1 for i, k in enumerate(own)}
    for k in range(n):
        event("K", k, ("K", k - 1), ("S0", k - kst), ("S1", k - kst))
        event("V", k, ("V", k - 1), ("PV0", k - vst), ("PV1", k - vst))
        event("S0", k, ("K", k), ("S0", k - 1), (free, k - 2))
        event("R0", k, ("S0", k), ("R0", k - 1))
        event("PV0", k, ("V", k), ("R0", k), ("PV0", k - 1))
        if second[k]:
            event("S1", k, ("K", k), ("S1", k - 1), ("PV1", before.get(before[k], -1)))
            event("R1", k, ("S1", k), ("R1", before[k]))
            event("PV1", k, ("V", k), ("R1", k), ("PV1", k - 1))
        else:  # the stages are given back, as far as these warps go
            event("S1", k, ("K", k), ("S1", k - 1))
            event("PV1", k, ("V", k), ("PV1", k - 1))
    return [(k, r) for k in range(n - words) for r in ("R0", "R1")
            if (r, k) in behind and (r, k) not in behind["K", k + words]]


@pytest.mark.parametrize("hdp", [64, 128])
def test_words_of_key_blocks_are_read_before_they_are_written_again(hdp):
    """bf16 rows: two blocks of rows, of which a tile may have the first alone."""
    kst, vst, words = rings(hdp, False)
    rng = random.Random(hdp)
    for second in [[True] * 8 + [False] * 40, [True] + [False] * 40, [True, False] * 20] + \
            [[rng.random() < share for _ in range(60)] for share in (0.1, 0.5, 0.9)]:
        assert not unordered(kst, vst, words, second)


def test_one_block_of_rows():
    """bf16 rows of more than 128 head dims, and fp32 rows, whose S waits for the softmax alone."""
    for hdp, f32 in ((256, False), (64, True), (128, True), (256, True)):
        kst, vst, words = rings(hdp, f32)
        assert not unordered(kst, vst, words, [False] * 60, "R0" if f32 else "PV0")


def test_a_ring_that_is_too_short_is_seen():
    assert unordered(4, 4, 9, [True] + [False] * 40) == [(0, "R1")] and not unordered(4, 4, 10, [True] + [False] * 40)
