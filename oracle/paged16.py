"""The 16-bit paged cache in 64 bits: rotated append, attention under any mask.  Test
infrastructure; shares no code with the CUDA path.

A pool is [k_pages, v_pages], arrays [num_pages, page, Hkv, D]; key r of sequence b is row
r % page of page table[b][r // page]."""
import numpy as np


def rotate(x, cos, sin, interleaved):
    """Rows x [..., D] turned by angles of cosines and sines [..., rot / 2]; also the bound's
    magnitudes |x c| + |y s|, |y c| + |x s| in the same places (zeros where nothing turns)."""
    half = cos.shape[-1]
    d = np.arange(half)
    i, j = (2 * d, 2 * d + 1) if interleaved else (d, d + half)
    out, mag = x.copy(), np.zeros_like(x)
    a, b = x[..., i], x[..., j]
    out[..., i], out[..., j] = a * cos - b * sin, b * cos + a * sin
    mag[..., i], mag[..., j] = abs(a * cos) + abs(b * sin), abs(b * cos) + abs(a * sin)
    return out, mag


def new_keys(lens, cu, total, B):
    """(row, sequence, key) of each packed row that a sequence owns; cu None: total / B each."""
    out = []
    for b in range(B):
        lo, hi = (cu[b], cu[b + 1]) if cu is not None else (b * (total // B), (b + 1) * (total // B))
        out += [(t, b, int(lens[b]) - (hi - lo) + t - lo) for t in range(lo, hi)]
    return out


def place(pool, table, b, key):
    """(page, row) of a key, or None outside the table's capacity or the pool."""
    page = pool.shape[1]
    if key < 0 or key >= page * table.shape[1]:
        return None
    at = int(table[b][key // page])
    return (at, key % page) if 0 <= at < pool.shape[0] else None


def cached(pool, table, b, n):
    """Rows 0 .. n - 1 of sequence b, [n, Hkv, D]; zeros on pages outside the pool."""
    out = np.zeros((n,) + pool.shape[2:])
    for r in range(n):
        at = place(pool, table, b, r)
        if at:
            out[r] = pool[at]
    return out


def sees_window(n, Sq, left, sinks):
    """[Sq, n]: which of n keys each of the last Sq tokens sees."""
    p, j = n - Sq + np.arange(Sq)[:, None], np.arange(n)
    return (j <= p) & ((j >= p - left if left >= 0 else True) | (j < sinks))


def sees_tree(n, Sq, tree):
    """The same for drafts: tree [Sq, Sq] says which token (row) sees which draft."""
    j = np.arange(n)
    t = j - (n - Sq)
    return (t < 0) | ((t >= 0) & tree[:, np.clip(t, 0, Sq - 1)])


def pack_tree(tree):
    """Truth values [..., Sq, Sq] as int32 words [..., Sq, ceil(Sq / 32)], bit t % 32 of word t // 32."""
    Sq = tree.shape[-1]
    bits = np.zeros(tree.shape[:-1] + (-(-Sq // 32) * 32,), dtype=bool)
    bits[..., :Sq] = tree
    return np.packbits(bits, axis=-1, bitorder="little").view("<i4")


def random_trees(rng, B, Sq):
    """Trees whose parents come before their children; about one draft in seven is a root."""
    tree = np.zeros((B, Sq, Sq), dtype=bool)
    for b in range(B):
        for t in range(Sq):
            parent = int(rng.integers(max(0, t - 6) - 1, t)) if t else -1
            if parent >= 0:
                tree[b, t] = tree[b, parent]
            tree[b, t, t] = True
    return tree


def attend(q, k, v, sees, scale):
    """q [Sq, Hq, D], k and v [n, Hkv, D], sees [Sq, n] -> o [Sq, Hq, D], lse [Hq, Sq], and what
    error bounds are made of: A = sum p |v| and T = max p * sum |v| over the seen keys [Sq, Hq, D],
    E = max over them of scale * sum_d |q_d k_d| [Hq, Sq].  A hidden key takes no part at all."""
    Sq, Hq, D = q.shape
    g = Hq // k.shape[1]
    o, A, T = (np.zeros((Sq, Hq, D)) for _ in range(3))
    lse, E = np.full((Hq, Sq), -np.inf), np.zeros((Hq, Sq))
    for i in range(Sq):
        at = np.nonzero(sees[i])[0]
        if len(at) == 0:
            continue
        for h in range(Hq):
            ks, vs = k[at, h // g], v[at, h // g]
            x = ks @ q[i, h] * scale
            m = x.max()
            p = np.exp(x - m)
            l = p.sum()
            p /= l
            with np.errstate(invalid="ignore"):
                if np.isfinite(vs).all():
                    o[i, h], A[i, h], T[i, h] = p @ vs, p @ abs(vs), p.max() * abs(vs).sum(0)
                else:  # (a product with BLAS may not keep inf and NaN to their columns)
                    o[i, h] = (p[:, None] * vs).sum(0)
                    A[i, h], T[i, h] = (p[:, None] * abs(vs)).sum(0), p.max() * abs(vs).sum(0)
            lse[h, i] = m + np.log(l)
            E[h, i] = abs(scale) * (abs(ks) @ abs(q[i, h])).max()
    return o, lse, A, T, E
