"""The order of the two-sub-tile decode over the 16-bit paged cache (fa_paged_decode.cuh, NQ = 2), on the CPU:
its roles with what they wait for, run in random order.  Sub-tile 0's softmax warps leave in one of a few
slots that a segment's V held a value that is not finite; both sub-tiles read the slot at the end of the segment,
and neither may find a later segment's."""
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_tiled_attention_20_gb300",
                      "csrc", "fa_paged_decode.cuh")


def slots_of_the_kernel():
    with open(SOURCE, encoding="utf-8") as f:
        src = f.read()
    found = re.search(r"kOddSlots = (\d+);", src)
    uses = re.findall(r"odd_seg\[([^\]]*)\]", src)
    if found:
        assert uses and set(uses) <= {"tcount % kOddSlots", "i"}, uses
        return int(found.group(1))
    assert set(uses) <= {"tcount & 1u", "0", "1"}
    return 2


def run(segments, slots, ring, seed):
    """segments: the tiles of each; every tile hides a key.  Returns what each sub-tile read for each segment."""
    rng, done = random.Random(seed), set()  # done: events (name, index)
    flag, read = [0] * slots, {}
    first = [sum(segments[:t]) for t in range(len(segments))]

    def load(n):  # the ring's load n takes the buffer of load n - ring
        return n < ring or ("free", n - ring) in done

    def k_and_q():
        for t, n in enumerate(segments):
            for j in range(n):
                it = first[t] + j
                yield lambda it=it: load(2 * it)
                done.add(("full", 2 * it))
                if j == 0:
                    yield lambda t=t: t == 0 or ("q free", t - 1) in done
                    done.add(("q", t))

    def v():
        for it in range(sum(segments)):
            yield lambda it=it: load(2 * it + 1)
            done.add(("full", 2 * it + 1))

    def products():
        def s(t, j, q):
            done.add(("S", q, first[t] + j))
            if q == 1 and j + 1 == segments[t]:
                done.add(("q free", t))
            if q == 1:
                done.add(("free", 2 * (first[t] + j)))
        for t, n in enumerate(segments):
            yield lambda t=t: ("q", t) in done and ("full", 2 * first[t]) in done
            for q in (0, 1):
                s(t, 0, q)
            for j in range(n):
                it = first[t] + j
                yield lambda it=it: ("full", 2 * it + 1) in done
                for q in (0, 1):
                    yield lambda it=it, q=q, t=t, j=j: ("P", q, it) in done and (j or not t or ("O free", q, t - 1) in done)
                    if j + 1 == n:
                        done.add(("O", q, t))
                    if q == 1:
                        done.add(("free", 2 * it + 1))
                    if j + 1 < n:
                        if q == 0:
                            yield lambda it=it: ("full", 2 * it + 2) in done
                        s(t, j + 1, q)

    def softmax(q):
        for t, n in enumerate(segments):
            for j in range(n):
                it = first[t] + j
                if q == 0:
                    yield lambda it=it: ("full", 2 * it + 1) in done
                    flag[t % slots] = t + 1
                yield lambda it=it: ("S", q, it) in done
                done.add(("P", q, it))
            yield lambda t=t: ("O", q, t) in done
            yield lambda: True  # (it may take its time here)
            read[q, t] = flag[t % slots]
            done.add(("O free", q, t))

    roles = [k_and_q(), v(), products(), softmax(0), softmax(1)]
    waits = [next(r) for r in roles]
    while roles:
        ready = [i for i, w in enumerate(waits) if w()]
        assert ready, "the roles wait for one another"
        slow = rng.random() < 0.8  # sub-tile 1's softmax is often late
        i = rng.choice([r for r in ready if not slow or roles[r].__name__ != "softmax" or roles[r].gi_frame.f_locals["q"] == 0]
                       or ready)
        try:
            waits[i] = next(roles[i])
        except StopIteration:
            del roles[i], waits[i]
    return read


@pytest.mark.parametrize("ring", [4, 6])
def test_a_segment_finds_its_own_flag(ring):
    slots = slots_of_the_kernel()
    for seed in range(400):
        rng = random.Random(seed)
        segments = [rng.choice([1, 1, 1, 2, 3]) for _ in range(12)]
        read = run(segments, slots, ring, seed)
        assert all(read[q, t] == t + 1 for q in (0, 1) for t in range(len(segments))), (segments, seed)


def test_two_slots_are_too_few():
    """What the model is for: with a slot for every other segment it finds a later one's."""
    assert any(run([1] * 12, 2, 4, seed)[1, t] != t + 1 for seed in range(200) for t in range(12))
