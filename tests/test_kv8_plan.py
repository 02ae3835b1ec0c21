"""Invariants of the 8-bit decode's plan (tests/kv8_plan.py), on the CPU: every key is taken
once, a cut pair's pieces have slots of their own inside the workspace, and the merge looks
for exactly those."""
import random

import pytest

import kv8_plan


def _check(lens, Hkv, capacity, ns, resident, D):
    B = len(lens)
    slots = 0 if ns == 1 else B * Hkv * ns
    grid, whole, solo = kv8_plan.host(B, Hkv, capacity, slots, resident, D)
    assert 1 <= grid <= resident
    segs, merged = kv8_plan.segments(lens, Hkv, grid, whole, solo)
    taken = {(b, hk): [] for b in range(B) for hk in range(Hkv) if lens[b]}
    used = {}
    for r, b, hk, k0, k1, slot in segs:
        taken[(b, hk)].append((k0, k1, slot))
        if slot is not None:
            assert 0 <= slot < slots and slot not in used
            used[slot] = (b, hk)
    for (b, hk), parts in taken.items():
        parts.sort()
        assert parts[0][0] == 0 and parts[-1][1] == lens[b]
        assert all(x[1] == y[0] for x, y in zip(parts, parts[1:]))
        if len(parts) > 1:
            assert merged[(b, hk)] == [s for _, _, s in parts]
        else:
            assert (b, hk) not in merged and parts[0][2] is None


@pytest.mark.parametrize("seed", range(60))
def test_every_key_once_and_every_piece_found(seed):
    rng = random.Random(seed)
    B, Hkv = rng.choice([1, 2, 3, 9, 40]), rng.choice([1, 2, 3, 8])
    top = rng.choice([1, 40, 130, 320, 500, 2000, 9000])
    lens = [rng.choice([0, 1, top, rng.randint(0, top)]) for _ in range(B)]
    lens[rng.randrange(B)] = top
    capacity = max(16, -(-top // 16) * 16 * rng.choice([1, 1, 3]))
    # the default number of slots for a pair, none, and a few
    default = max(1, min(-(-8 * 152 // (B * Hkv)), -(-capacity // 256), 1024))
    for ns in (default, 1, 2, 7):
        for resident in (304, 456, 5):
            _check(lens, Hkv, capacity, ns, resident, rng.choice([64, 128, 256]))


def test_an_empty_batch_has_no_work():
    grid, whole, solo = kv8_plan.host(4, 2, 256, 8, 456)
    assert kv8_plan.segments([0] * 4, 2, grid, whole, solo) == ([], {})


def test_one_partial_result_a_pair_cuts_a_long_sequence_among_many():
    """The default's room for 160 sequences of 8 kv heads: no range holds more than its units."""
    lens = [1000] * 159 + [32768]
    grid, whole, solo = kv8_plan.host(160, 8, 32768, 160 * 8, 456)
    segs, _ = kv8_plan.segments(lens, 8, grid, whole, solo)
    held = {}
    for r, _, _, k0, k1, _ in segs:
        held[r] = held.get(r, 0) + k1 - k0
    width = -(-8 * sum(kv8_plan.units(n) for n in lens) // grid)
    assert max(held.values()) <= width * kv8_plan.UNIT < 32768 / 7
    grid, whole, solo = kv8_plan.host(160, 8, 32768, 0, 456)    # what a caller's 1 asks for
    held = {}
    for r, _, _, k0, k1, _ in kv8_plan.segments(lens, 8, grid, whole, solo)[0]:
        held[r] = held.get(r, 0) + k1 - k0
    assert max(held.values()) >= 32768
