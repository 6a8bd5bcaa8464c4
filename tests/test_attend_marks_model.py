"""CPU model of two row slots that share the key tiles of wide units (CPU only).

Slot 0's MMA warp takes the non-finite values out of a tile of values before either slot multiplies it, and marks the
segment; each slot's softmax warps read the mark when the segment's rows are complete, and add those values to the rows
that see them.  The waits of the two MMA and the two softmax warps are transcribed from the kernel (queries, turns on
the tensor core, scores, probabilities, ring stages, mended tiles), and every order that they allow is walked: a mark
must still be there when the slower slot reads it.  The number of marks is read from the kernel's source.
"""
import os
import re

import mxfp4_moe_expert_gb300 as pkg

SEGMENTS = 4                       # of one tile each: the shortest, where one slot gets furthest ahead
RING = 2                           # tiles of keys and values in the ring


def programs():
    """Per warp a list of (condition, effect): counters are how often a barrier was passed on."""
    def mma(x, k):
        o, turn = 1 - x, lambda c, n: c[f"turn{x}"] + (x == 0) > n       # (slot 0 has the first turn)
        take = [] if x else [(lambda c: min(c["pv0"], c["pv1"]) > k - RING, "mark")]
        wait = [(lambda c: c["mended"] > k, None)] if x else []
        return [(lambda c: c[f"q{x}"] > k, None), (lambda c: turn(c, 2 * k), f"s{x} turn{o}"), *take, *wait,
                (lambda c: c[f"p{x}"] > k, None), (lambda c: turn(c, 2 * k + 1), f"pv{x} turn{o}")]

    def softmax(x, k):
        return [(lambda c: True, f"q{x}"), (lambda c: c[f"s{x}"] > k, f"p{x}"), (lambda c: c[f"pv{x}"] > k, "read")]

    return [sum((part(x, k) for k in range(SEGMENTS)), []) for part in (mma, softmax) for x in (0, 1)]


NAMES = ["q0", "q1", "s0", "s1", "p0", "p1", "pv0", "pv1", "turn0", "turn1", "mended"]


def lost_marks(words):
    """Whether some order lets a softmax warp miss the mark of its segment; raises where an order cannot go on."""
    progs = programs()
    todo, seen, lost = [((0,) * 4, (0,) * words)], set(), False
    while todo:
        at = todo.pop()
        if at in seen:
            continue
        seen.add(at)
        pcs, marks = at
        count = dict.fromkeys(NAMES, 0)
        for prog, pc in zip(progs, pcs):
            for _, effect in prog[:pc]:
                for name in (effect or "").split():
                    if name != "read":
                        count["mended" if name == "mark" else name] += 1
        steps = 0
        for w, (prog, pc) in enumerate(zip(progs, pcs)):
            if pc == len(prog) or not prog[pc][0](count):
                continue
            steps += 1
            now = marks
            if prog[pc][1] == "mark":
                k = count["mended"]
                now = tuple(k + 1 if i == k % words else m for i, m in enumerate(marks))
            elif prog[pc][1] == "read":
                k = pc // 3
                lost |= marks[k % words] != k + 1
            todo.append((pcs[:w] + (pc + 1,) + pcs[w + 1:], now))
        assert steps or all(pc == len(prog) for prog, pc in zip(progs, pcs))
    return lost


def test_one_mark_would_be_overwritten():
    assert lost_marks(1)


def test_the_kernel_has_as_many_marks_as_it_needs():
    path = os.path.join(os.path.dirname(pkg.__file__), "csrc", "cache_attend.cu")
    found = re.search(r"constexpr int kWideMarks = (\d+);", open(path).read())
    assert not lost_marks(int(found.group(1)) if found else 1)
