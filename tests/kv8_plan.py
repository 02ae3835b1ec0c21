"""The plan of the 8-bit decode, written out in Python for the tests: which CTA or warp takes
which keys of which (sequence, kv head) pair, and where a cut pair's partial results go."""
UNIT, LEAD = 64, 4


def host(B, Hkv, capacity, slots, resident, D=128, in_registers=True):
    """What the launch decides: (ranges, whole, solo_keys)."""
    pairs = B * Hkv
    most = pairs * -(-capacity // UNIT)
    ranges = min(resident, most, max(slots // 2, slots - pairs))
    whole = slots == 0 or ranges < min(resident, 2 * pairs)
    grid = min(resident, pairs) if whole else ranges
    solo = 0
    if in_registers:
        solo = 128 if pairs > grid else 0
        if D != 256 and pairs >= 2 * grid:
            solo = 512 if pairs >= 4 * grid else 320
    return grid, whole, solo


def units(n):
    return -(-n // UNIT) + LEAD if n > 0 else 0


def segments(lens, Hkv, grid, whole, solo_keys):
    """[(range, b, hk, k0, k1, slot or None)] and {(b, hk): pieces as the merge counts them}."""
    u = [units(n) for n in lens]
    prefix = [0]
    for x in u:
        prefix.append(prefix[-1] + x)
    solo = solo_keys > 0 and max(u) <= solo_keys // UNIT + LEAD
    ranges = grid * 4 if solo else grid
    total = Hkv * prefix[-1]
    W = max(-(-total // ranges), 1)
    uncut = whole or solo
    out, merged = [], {}
    pairs = [(b, hk, Hkv * prefix[b] + hk * u[b]) for b in range(len(lens)) if u[b] for hk in range(Hkv)]
    for r in range(ranges):
        x0, x1 = min(r * W, total), min(r * W + W, total)
        for b, hk, start in pairs:
            if uncut:
                if x0 <= start < x1:
                    out.append((r, b, hk, 0, lens[b], None))
                continue
            lo, hi = max(start, x0), min(start + u[b], x1)
            k0 = max(lo - start - LEAD, 0) * UNIT
            k1 = min((hi - start - LEAD) * UNIT, lens[b])
            if lo >= hi or k1 <= k0:
                continue
            first = (start + LEAD) // W
            n = (start + u[b] - 1) // W - first + 1
            slot = None
            if n > 1:
                slot = r if r != first else grid + (r if grid <= len(lens) * Hkv else b * Hkv + hk)
            out.append((r, b, hk, k0, k1, slot))
    if not uncut:
        for b, hk, start in pairs:
            first = (start + LEAD) // W
            n = (start + u[b] - 1) // W - first + 1
            if n > 1:
                merged[(b, hk)] = [first + c if c else grid + (first if grid <= len(lens) * Hkv else b * Hkv + hk)
                                   for c in range(n)]
    return out, merged
