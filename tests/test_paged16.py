"""The operators over the 16-bit paged cache on the GPU against their 64-bit reference
(oracle/paged16.py): the rotated append, the decodes under a draft tree and under a window with
sinks.  Pools start as garbage with NaNs and infinities in it: nothing outside the sequences may
matter.

Bounds, from the roundings (a rounding is off by at most half a step, u = eps / 2 of the type: 2^-8
for bf16, 2^-11 for fp16):

append:  y = x c - y s in fp32 (two products and a sum, each off by 2^-24 of what it holds, so by
    2^-22 M together with room, M = |x c| + |y s|), rounded once: |d| <= u |y| + 2^-22 M, and half
    of a subnormal step.
decode:  |dO| <= u |O| + c A + f T, with A = sum_j p_j |v_j|, T = max_j p_j sum_j |v_j|:
    c = u (P rounded for the product) + 2 e_s + 2^-21 + N 2^-23
    e_s  error of a score, in its exponent: (D + 8) 2^-22 max_j scale sum_d |q_d k_jd| (a sum of D
         products in 32 bits in any order, each step allowed a truncation, and the scale), twice
         because it enters the numerator and the denominator; 2^-21: exp2 and the division;
         N = n / 4 + 64: sums over the n keys (four partial sums run side by side at least)
    f    fp16 only: P is at least 1 for the row's largest weight, and below 2^-14 its steps are 2^-24,
         so a weight is off by 2^-25 of the largest there (bf16 has fp32's range)
    |dLSE| <= e_s + 2^-21 + N 2^-23 + 2^-22 |LSE|.
"""
import math

import numpy as np
import pytest
import torch

from oracle import paged16

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
TINY = {"bf16": 2.0 ** -133, "fp16": 2.0 ** -24}  # least subnormals
DEV = "cuda:0"


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import exact_tiled_attention_20_gb300 as fa_mod
    from exact_tiled_attention_20_gb300 import build

    build.build_library()
    fa_mod.load()
    return fa_mod


def garbage(gen, shape, dtype):
    """Random values, every eleventh or so an infinity or NaN."""
    x = torch.randn(shape, generator=gen)
    bad = torch.tensor([math.inf, -math.inf, math.nan])
    at = torch.randint(0, 33, shape, generator=gen)
    return torch.where(at < 3, bad[at.clamp(max=2)], x).to(DT[dtype])


class Pool:
    """A pool of garbage, a scattered table, and the sequences' own rows written into it."""

    def __init__(self, B, Hkv, D, page, lens, dtype, seed=0, max_pages=None):
        self.gen = torch.Generator().manual_seed(seed)
        self.dtype, self.page, self.lens = dtype, page, list(lens)
        max_pages = max_pages or max(1, -(-max(lens) // page))
        n = B * max_pages + 2
        self.cpu = [garbage(self.gen, (n, page, Hkv, D), dtype) for _ in range(2)]
        self.table = torch.randperm(n, generator=self.gen)[:B * max_pages].view(B, max_pages).to(torch.int32)

    def fill(self):
        """Finite rows for every key of the sequences."""
        t = self.table.numpy()
        for b, n in enumerate(self.lens):
            for pool in self.cpu:
                rows = torch.randn((n,) + pool.shape[2:], generator=self.gen).to(DT[self.dtype])
                for r0 in range(0, n, self.page):
                    take = min(self.page, n - r0)
                    pool[int(t[b][r0 // self.page]), :take] = rows[r0:r0 + take]
        return self

    def np(self):
        return [p.double().numpy() for p in self.cpu]

    def gpu(self):
        return [p.to(DEV) for p in self.cpu] + [self.table.to(DEV), torch.tensor(self.lens, dtype=torch.int32).to(DEV)]


def check(o, lse, q, pool, sees, scale, dtype):
    """o [B, Sq, Hq, D], lse [B, Hq, Sq] of the GPU against the reference; sees(b, n) -> [Sq, n]."""
    o, lse, qn = o.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
    kp, vp = pool.np()
    t, D = pool.table.numpy(), q.shape[-1]
    u = U[dtype]
    for b, n in enumerate(pool.lens):
        k, v = paged16.cached(kp, t, b, n), paged16.cached(vp, t, b, n)
        s = sees(b, n)
        k = np.where(s.any(0)[:, None, None], k, 0.0)  # keys that no token sees
        v = np.where(s.any(0)[:, None, None], v, 0.0)
        ro, rl, A, T, E = paged16.attend(qn[b], k, v, s, scale)
        e_s = (D + 8) * 2.0 ** -22 * E
        N = n / 4 + 64
        common = 2.0 ** -21 + N * 2.0 ** -23
        c = u + 2 * e_s.T[..., None] + common
        bound = u * abs(ro) + c * A + (2.0 ** -25 * T if dtype == "fp16" else 0) + TINY[dtype]
        fin = np.isfinite(ro)
        assert np.array_equal(np.isnan(o[b]), np.isnan(ro)), f"NaN pattern of sequence {b}"
        assert np.array_equal(o[b][~fin & ~np.isnan(ro)], ro[~fin & ~np.isnan(ro)]), f"infinities of sequence {b}"
        off = abs(o[b][fin] - ro[fin]) / bound[fin]
        assert off.size == 0 or off.max() <= 1, f"sequence {b}: |dO| is {off.max():.2f} of its bound"
        some = np.isfinite(rl)
        assert np.array_equal(some, np.isfinite(lse[b])) and (lse[b][~some] == -np.inf).all(), f"LSE of sequence {b}"
        lb = e_s + common + 2.0 ** -22 * abs(np.where(some, rl, 0))
        off = (abs(np.where(some, lse[b], 0) - np.where(some, rl, 0)) / lb)
        assert off.max() <= 1, f"sequence {b}: |dLSE| is {off.max():.2f} of its bound"


def queries(pool, B, Sq, Hq, D, dtype):
    return torch.randn((B, Sq, Hq, D), generator=pool.gen).to(DT[dtype])


# (Sq, Hq, Hkv, D, page, lens, dtype)
TREES = [
    (1, 2, 1, 64, 16, [1, 0, 2, 129], "bf16"),                  # one draft: itself and the cache
    (7, 8, 2, 64, 16, [333, 7, 3, 0, 8], "bf16"),               # trees longer than their sequence
    (33, 4, 4, 128, 48, [33, 160, 161, 300], "fp16"),           # a mask of two words, one head each
    (16, 16, 2, 128, 128, [1000, 16, 2500], "bf16"),            # 128 rows: one full sub-tile
    (17, 16, 2, 128, 64, [900, 17, 140], "fp16"),               # 136 rows: a second sub-tile of one token
    (64, 8, 2, 96, 32, [64, 700, 1], "bf16"),                   # 256 rows
    (100, 12, 3, 64, 80, [100, 431, 99], "fp16"),               # 400 rows: row blocks
    (5, 24, 2, 256, 16, [77, 5, 640], "bf16"),                  # D = 256, 60 rows
    (40, 8, 1, 256, 112, [41, 200], "fp16"),                    # D = 256, 320 rows
    (256, 2, 2, 64, 256, [256, 1111], "bf16"),                  # the longest mask
    (3, 128, 1, 64, 16, [50, 260], "bf16"),                     # 128 heads of one kv head: a sub-tile per token
    (11, 15, 3, 96, 16, [0, 0, 12], "fp16"),                    # an odd group, empty sequences
]


@pytest.mark.parametrize("case", TREES, ids=lambda c: f"sq{c[0]}_h{c[1]}_{c[2]}_d{c[3]}_p{c[4]}_{c[6]}")
def test_tree_matches_the_reference(fa, case):
    Sq, Hq, Hkv, D, page, lens, dtype = case
    B = len(lens)
    pool = Pool(B, Hkv, D, page, lens, dtype, seed=Sq + D).fill()
    q = queries(pool, B, Sq, Hq, D, dtype)
    tree = paged16.random_trees(np.random.default_rng(Sq), B, Sq)
    mask = torch.from_numpy(paged16.pack_tree(tree)).to(DEV)
    o, lse = fa.fa_decode_splitkv_paged_tree(q.to(DEV), *pool.gpu(), mask)
    torch.cuda.synchronize()
    check(o, lse, q, pool, lambda b, n: paged16.sees_tree(n, Sq, tree[b]), 1 / math.sqrt(D), dtype)


# (Sq, Hq, Hkv, D, page, lens, window, sinks, dtype)
WINDOWS = [
    (1, 8, 2, 64, 16, [1, 0, 500, 64, 65], 63, 4, "bf16"),
    (1, 4, 4, 128, 128, [5000, 127, 1025, 2, 0], 1023, 4, "bf16"),
    (3, 12, 12, 96, 48, [3, 1, 700, 1300], 600, 37, "fp16"),     # sinks that end inside a tile
    (4, 8, 2, 128, 256, [2000, 4, 300], -1, 0, "bf16"),          # no window: a causal decode
    (1, 8, 1, 256, 16, [900, 63, 64], 0, 0, "fp16"),             # itself alone
    (2, 6, 3, 64, 32, [1500, 30], 10, 200, "bf16"),              # more sinks than window
    (1, 16, 2, 256, 64, [3000, 513], 511, 129, "bf16"),
    (60, 16, 4, 128, 16, [60, 59, 800], 100, 1, "fp16"),         # 240 rows, windows that slide across tiles
    (5, 4, 2, 64, 16, [300, 10], 10 ** 9, 10 ** 9, "bf16"),      # past every length
    (1, 2, 2, 128, 16, [8000], -1, 0, "bf16"),                   # one long sequence, cut into pieces
]


@pytest.mark.parametrize("case", WINDOWS, ids=lambda c: f"sq{c[0]}_h{c[1]}_{c[2]}_d{c[3]}_w{c[6]}_s{c[7]}_{c[8]}")
def test_window_matches_the_reference(fa, case):
    Sq, Hq, Hkv, D, page, lens, left, sinks, dtype = case
    B = len(lens)
    pool = Pool(B, Hkv, D, page, lens, dtype, seed=Sq + D + left % 97).fill()
    q = queries(pool, B, Sq, Hq, D, dtype)
    o, lse = fa.fa_decode_splitkv_paged_window(q.to(DEV), *pool.gpu(), left, sinks=sinks)
    torch.cuda.synchronize()
    check(o, lse, q, pool, lambda b, n: paged16.sees_window(n, Sq, left, sinks), 1 / math.sqrt(D), dtype)


# The forms for few and for many rows of a kv head, each with several short sequences per CTA.
# (Sq, Hq, Hkv, D, page, window, sinks, dtype)
BATCHES = [
    (1, 4, 1, 128, 16, 600, 4, "bf16"),       # 4 rows
    (4, 8, 2, 128, 64, 1023, 33, "fp16"),     # 16 rows, the most of one form
    (17, 2, 2, 128, 32, 500, 1, "bf16"),      # 17, the least of the other
    (2, 16, 2, 64, 48, -1, 0, "fp16"),
    (3, 3, 1, 96, 16, 300, 200, "bf16"),
    (4, 8, 2, 256, 64, 700, 4, "bf16"),
]


@pytest.mark.parametrize("case", BATCHES, ids=lambda c: f"sq{c[0]}_h{c[1]}_{c[2]}_d{c[3]}_w{c[5]}_s{c[6]}_{c[7]}")
def test_many_short_sequences(fa, case):
    """More sequences than CTAs, of 0 to 1400 keys, under a window and under a tree, over and over:
    the buffers of one are handed to the next."""
    Sq, Hq, Hkv, D, page, left, sinks, dtype = case
    B = 230
    rng = np.random.default_rng(D + Sq)
    lens = [int(n) for n in rng.integers(0, 1400, B)]
    pool = Pool(B, Hkv, D, page, lens, dtype, seed=5).fill()
    q = queries(pool, B, Sq, Hq, D, dtype)
    tree = paged16.random_trees(rng, B, Sq)
    qd, gpu, mask = q.to(DEV), pool.gpu(), torch.from_numpy(paged16.pack_tree(tree)).to(DEV)
    first = fa.fa_decode_splitkv_paged_window(qd, *gpu, left, sinks=sinks)
    t_first = fa.fa_decode_splitkv_paged_tree(qd, *gpu, mask)
    torch.cuda.synchronize()
    for _ in range(5):
        again = fa.fa_decode_splitkv_paged_window(qd, *gpu, left, sinks=sinks)
        t_again = fa.fa_decode_splitkv_paged_tree(qd, *gpu, mask)
        torch.cuda.synchronize()
        for a, b in zip((*first, *t_first), (*again, *t_again)):
            assert torch.equal(a, b)
    check(*first, q, pool, lambda b, n: paged16.sees_window(n, Sq, left, sinks), 1 / math.sqrt(D), dtype)
    check(*t_first, q, pool, lambda b, n: paged16.sees_tree(n, Sq, tree[b]), 1 / math.sqrt(D), dtype)


@pytest.mark.parametrize("rising", [True, False])
@pytest.mark.parametrize("Sq,D", [(2, 64), (4, 128), (8, 128), (5, 96), (3, 256), (40, 128)])
def test_scores_that_rise_or_fall_along_the_sequence(fa, Sq, D, rising):
    """Keys that grow, or shrink, by a factor of 200 along the sequence: the references of the softmax
    are raised again and again, the early keys' weights going to zero, or never."""
    lens = [1900, 700, 64]
    pool = Pool(3, 2, D, 32, lens, "bf16", seed=D).fill()
    t = pool.table.numpy()
    for b, n in enumerate(lens):
        for j in range(n):
            at = j if rising else n - 1 - j
            pool.cpu[0][int(t[b][j // 32]), j % 32] *= 10.0 * 200.0 ** (at / n - 1)
    q = queries(pool, 3, Sq, 8, D, "bf16")
    o, lse = fa.fa_decode_splitkv_paged_window(q.to(DEV), *pool.gpu())
    torch.cuda.synchronize()
    check(o, lse, q, pool, lambda b, n: paged16.sees_window(n, Sq, -1, 0), 1 / math.sqrt(D), "bf16")


@pytest.mark.parametrize("Sq", [1, 9])
def test_lengths_outside_the_table_are_clamped(fa, Sq):
    pool = Pool(3, 2, 128, 16, [64, 0, 33], "bf16", seed=Sq, max_pages=4).fill()
    q = queries(pool, 3, Sq, 4, 128, "bf16")
    kp, vp, table, kl = pool.gpu()
    want = fa.fa_decode_splitkv_paged_window(q.to(DEV), kp, vp, table, kl, 50, sinks=3)
    wrong = torch.tensor([2 ** 31 - 1, -2 ** 31, 33], dtype=torch.int32, device=DEV)
    got = fa.fa_decode_splitkv_paged_window(q.to(DEV), kp, vp, table, wrong, 50, sinks=3)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_pages_past_two_to_the_32_values(fa):
    """Pools of more than 2^32 values each, the sequences' pages at their far ends."""
    D, Hkv, page, Sq, Hq = 128, 8, 256, 2, 16
    each = page * Hkv * D
    pages = 2 ** 32 // each + 8
    if torch.cuda.mem_get_info()[0] < 5 * pages * each:
        pytest.skip("not enough memory")
    small = Pool(2, Hkv, D, page, [700, 300], "bf16", seed=3).fill()
    kp, vp, table, kl = small.gpu()
    wide = [torch.empty((pages, page, Hkv, D), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    far = torch.where(table < 4, table, table + (pages - kp.shape[0]))   # most at the far end
    for big, p in zip(wide, (kp, vp)):
        big[:4], big[4 - p.shape[0]:] = p[:4], p[4:]
    new = torch.randn((2, 2, Sq, Hkv, D), generator=small.gen).to(torch.bfloat16).to(DEV)
    q = queries(small, 2, Sq, Hq, D, "bf16").to(DEV)
    kp, vp = kp.clone(), vp.clone()
    for k, v, t in ((kp, vp, table), (*wide, far)):
        fa.fa_kv_append_paged_rope(new[0], new[1], k, v, t, kl)
    want = fa.fa_decode_splitkv_paged_window(q, kp, vp, table, kl, 400, sinks=5)
    got = fa.fa_decode_splitkv_paged_window(q, *wide, far, kl, 400, sinks=5)
    torch.cuda.synchronize()
    for big, p in zip(wide, (kp, vp)):
        assert torch.equal(big[4 - p.shape[0]:].view(torch.int16), p[4:].view(torch.int16))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_pages_outside_the_window_may_be_anything(fa):
    """Table entries of pages with no visible key are out of the pool; a visible key on such a page
    counts as a zero row."""
    pool = Pool(2, 2, 64, 16, [2000, 1000], "bf16", seed=5).fill()
    pool.table[0, 4:100] = torch.tensor([-1, 1 << 30, -(1 << 31), 10 ** 6]).repeat(24).to(torch.int32)  # keys 64 .. 1599
    pool.table[1, 62] = -7                                                                              # keys 992 ..
    q = queries(pool, 2, 2, 4, 64, "bf16")
    o, lse = fa.fa_decode_splitkv_paged_window(q.to(DEV), *pool.gpu(), 200, sinks=64)
    torch.cuda.synchronize()
    check(o, lse, q, pool, lambda b, n: paged16.sees_window(n, 2, 200, 64), 1 / math.sqrt(64), "bf16")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", ["nan", "inf"])
def test_values_that_are_not_finite_reach_those_that_see_them(fa, D, kind):
    """An infinity or NaN in V of a draft, or of a key at a window's edge, is in the output of the
    tokens that see that key and in no other; in K it makes only those tokens' rows NaN."""
    Sq, Hq, Hkv, lens = 40, 8, 2, [41, 500]
    pool = Pool(2, Hkv, D, 16, lens, "bf16", seed=D).fill()
    t = pool.table
    for b, n in enumerate(lens):
        for draft, d in ((3, 5), (3, 40), (39, 0), (20, D - 1)):
            key = n - Sq + draft
            pool.cpu[1][int(t[b][key // 16]), key % 16, 1, d] = math.nan if kind == "nan" else math.inf
    tree = paged16.random_trees(np.random.default_rng(D), 2, Sq)
    q = queries(pool, 2, Sq, Hq, D, "bf16")
    mask = torch.from_numpy(paged16.pack_tree(tree)).to(DEV)
    o, lse = fa.fa_decode_splitkv_paged_tree(q.to(DEV), *pool.gpu(), mask)
    torch.cuda.synchronize()
    check(o, lse, q, pool, lambda b, n: paged16.sees_tree(n, Sq, tree[b]), 1 / math.sqrt(D), "bf16")
    o, lse = fa.fa_decode_splitkv_paged_window(q.to(DEV), *pool.gpu(), 12, sinks=3)
    torch.cuda.synchronize()
    check(o, lse, q, pool, lambda b, n: paged16.sees_window(n, Sq, 12, 3), 1 / math.sqrt(D), "bf16")
    key = lens[1] - Sq + 7
    pool.cpu[0][int(t[1][key // 16]), key % 16, 0, 2] = math.nan
    o, lse = fa.fa_decode_splitkv_paged_tree(q.to(DEV), *pool.gpu(), mask)
    torch.cuda.synchronize()
    hit = torch.from_numpy(tree[1][:, 7])
    assert torch.isnan(o[1, :, :4].cpu()[hit]).all() and torch.isnan(lse[1, :4].cpu()[:, hit]).all()
    assert torch.isfinite(lse[1, :4].cpu()[:, ~hit]).all() and torch.isfinite(lse[1, 4:]).all()


@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("kind", ["nan", "-inf"])
def test_values_that_are_not_finite_and_few_rows(fa, D, kind):
    """The same where a kv head has 16 rows, over several tiles and in outputs that are cut and joined."""
    Sq, Hq, Hkv, lens = 4, 8, 2, [4, 4000]
    pool = Pool(2, Hkv, D, 32, lens, "bf16", seed=D).fill()
    t = pool.table
    for b, n in enumerate(lens):
        for at, d in ((1, 5), (2, D - 1), (3, 33)):
            key = n - Sq + at
            pool.cpu[1][int(t[b][key // 32]), key % 32, 1, d] = float(kind)
    edge = lens[1] - 3 - 600                                 # the window's first key of token 1
    pool.cpu[1][int(t[1][edge // 32]), edge % 32, 0, 7] = float(kind)
    tree = paged16.random_trees(np.random.default_rng(D), 2, Sq)
    q = queries(pool, 2, Sq, Hq, D, "bf16")
    mask = torch.from_numpy(paged16.pack_tree(tree)).to(DEV)
    o, lse = fa.fa_decode_splitkv_paged_window(q.to(DEV), *pool.gpu(), 600, sinks=70)
    torch.cuda.synchronize()
    check(o, lse, q, pool, lambda b, n: paged16.sees_window(n, Sq, 600, 70), 1 / math.sqrt(D), "bf16")
    pool.cpu[1][int(t[1][edge // 32]), edge % 32, 0, 7] = 1.0
    o, lse = fa.fa_decode_splitkv_paged_tree(q.to(DEV), *pool.gpu(), mask)
    torch.cuda.synchronize()
    check(o, lse, q, pool, lambda b, n: paged16.sees_tree(n, Sq, tree[b]), 1 / math.sqrt(D), "bf16")
    key = lens[1] - Sq + 1
    pool.cpu[0][int(t[1][key // 32]), key % 32, 0, 2] = math.nan
    q[1, 0, 7] = math.nan                                    # a query head of the other kv head
    o, lse = fa.fa_decode_splitkv_paged_tree(q.to(DEV), *pool.gpu(), mask)
    torch.cuda.synchronize()
    hit = torch.from_numpy(tree[1][:, 1])
    o, lse = o[1].cpu(), lse[1].cpu()
    assert torch.isnan(o[:, :4][hit]).all() and torch.isnan(lse[:4][:, hit]).all()
    assert torch.isfinite(o[:, :4][~hit]).all() and torch.isfinite(lse[:4][:, ~hit]).all()
    assert torch.isnan(o[0, 7]).all() and torch.isnan(lse[7, 0])
    assert torch.isfinite(lse[4:7]).all() and torch.isfinite(lse[7, 1:]).all()


def test_two_streams_at_once_and_a_replay_with_few_rows(fa):
    """Calls on two streams with workspaces of their own do not disturb one another; a captured step
    follows lengths and a table that moved on."""
    B, Hq, Hkv, D = 20, 32, 8, 128
    rng = np.random.default_rng(4)
    pools = [Pool(B, Hkv, D, 64, [int(n) for n in rng.integers(0, 2500, B)], "bf16", seed=i).fill() for i in range(2)]
    qs = [queries(p, B, 1, Hq, D, "bf16").to(DEV) for p in pools]
    gpu = [p.gpu() for p in pools]
    want = [fa.fa_decode_splitkv_paged_window(q, *g, 500, sinks=4) for q, g in zip(qs, gpu)]
    torch.cuda.synchronize()
    n = fa.fa_decode_paged_workspace_bytes(B, 1, Hq, Hkv, D)
    ws = [torch.empty(n, dtype=torch.uint8, device=DEV) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[(torch.empty_like(q), torch.empty((B, Hq, 1), device=DEV)) for _ in range(8)] for q in qs]
    torch.cuda.synchronize()
    for k in range(8):
        for i in range(2):
            fa.fa_decode_splitkv_paged_window(qs[i], *gpu[i], 500, sinks=4, out=outs[i][k][0], lse=outs[i][k][1],
                                              workspace=ws[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        for o, lse in outs[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])
    check(*want[0], qs[0].cpu(), pools[0], lambda b, k: paged16.sees_window(k, 1, 500, 4), 1 / math.sqrt(D), "bf16")
    graph, o, lse = torch.cuda.CUDAGraph(), *outs[0][0]
    with torch.cuda.graph(graph):
        fa.fa_decode_splitkv_paged_window(qs[0], *gpu[0], 500, sinks=4, out=o, lse=lse, workspace=ws[0])
    for lens in (rng.permutation(pools[0].lens), np.minimum(pools[0].lens, 3), np.zeros(B)):
        lens = [int(min(a, b)) for a, b in zip(lens, pools[0].lens)]     # rows that hold keys
        gpu[0][3].copy_(torch.tensor(lens, dtype=torch.int32))
        o.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        part = Pool.__new__(Pool)
        part.__dict__.update(pools[0].__dict__, lens=lens)
        check(o, lse, qs[0].cpu(), part, lambda b, k: paged16.sees_window(k, 1, 500, 4), 1 / math.sqrt(D), "bf16")


def test_guards_repeats_and_graphs(fa):
    """Outputs inside larger buffers leave the rest alone; the same call gives the same bits, from
    a captured graph and on another stream too; a replay follows lengths that moved on."""
    B, Sq, Hq, Hkv, D = 3, 9, 8, 2, 128
    pool = Pool(B, Hkv, D, 64, [1500, 9, 700], "bf16", seed=3).fill()
    q = queries(pool, B, Sq, Hq, D, "bf16").to(DEV)
    g = pool.gpu()
    tree = paged16.random_trees(np.random.default_rng(1), B, Sq)
    mask = torch.from_numpy(paged16.pack_tree(tree)).to(DEV)
    big_o = torch.full((B + 2, Sq, Hq, D), 7.0, dtype=torch.bfloat16, device=DEV)
    big_l = torch.full((B + 2, Hq, Sq), 7.0, device=DEV)
    n = fa.fa_decode_paged_workspace_bytes(B, Sq, Hq, Hkv, D)
    ws = torch.full((n + 4096,), 0x7f, dtype=torch.uint8, device=DEV)
    o, lse = fa.fa_decode_splitkv_paged_tree(q, *g, mask, out=big_o[1:-1], lse=big_l[1:-1], workspace=ws[:n])
    torch.cuda.synchronize()
    assert (big_o[0] == 7).all() and (big_o[-1] == 7).all() and (big_l[0] == 7).all() and (big_l[-1] == 7).all()
    assert (ws[n:] == 0x7f).all()
    check(o, lse, q.cpu(), pool, lambda b, k: paged16.sees_tree(k, Sq, tree[b]), 1 / math.sqrt(D), "bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, lse2 = fa.fa_decode_splitkv_paged_tree(q, *g, mask, stream=side)
    side.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    graph = torch.cuda.CUDAGraph()
    o3, lse3, ws3 = torch.empty_like(q), torch.empty((B, Hq, Sq), device=DEV), torch.empty_like(ws)
    fa.fa_decode_splitkv_paged_window(q, *g, 100, sinks=2, out=o3, lse=lse3, workspace=ws3)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        fa.fa_decode_splitkv_paged_window(q, *g, 100, sinks=2, out=o3, lse=lse3, workspace=ws3)
    for lens in ([1500, 9, 700], [1499, 0, 64], [10, 9, 1]):
        g[3].copy_(torch.tensor(lens, dtype=torch.int32))
        pool.lens = lens
        o3.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        check(o3, lse3, q.cpu(), pool, lambda b, k: paged16.sees_window(k, Sq, 100, 2), 1 / math.sqrt(D), "bf16")


# ------------------------------------------------------------------------------ append
# (B, counts, pasts, Hq, Hkv, D, page, rot, interleaved, explicit positions, packed, dtype)
APPENDS = [
    (2, [1, 1], [0, 70], 8, 2, 64, 16, 64, False, False, False, "bf16"),
    (3, [0, 5, 33], [17, 0, 40], 4, 4, 128, 48, 128, False, True, True, "fp16"),
    (2, [3, 3], [5, 9], 6, 3, 96, 1, 48, True, False, False, "bf16"),       # pages of one row, half of the dims
    (1, [130], [3], 5, 1, 256, 100, 16, True, True, True, "fp16"),
    (2, [7, 2], [0, 0], 0, 2, 128, 16, 0, False, False, True, "bf16"),      # no queries, no rotation
    (4, [600, 0, 1100, 300], [5, 5, 0, 77], 32, 8, 128, 64, 96, False, False, True, "bf16"),  # several rows a lane
    (70, [1] * 70, list(range(70)), 3, 1, 64, 16, 32, False, True, False, "fp16"),
]


@pytest.mark.parametrize("case", APPENDS, ids=lambda c: f"b{c[0]}_h{c[3]}_{c[4]}_d{c[5]}_rot{c[7]}_{c[11]}")
def test_append_matches_the_reference(fa, case):
    B, counts, pasts, Hq, Hkv, D, page, rot, inter, explicit, packed, dtype = case
    lens = [a + b for a, b in zip(counts, pasts)]
    pool = Pool(B, Hkv, D, page, lens, dtype, seed=D + rot)
    total = sum(counts) + (3 if packed else 0)              # rows behind the last sequence
    # one projection's output, with a gap beside it
    wide = torch.randn((total, Hq + 2 * Hkv + 1, D), generator=pool.gen).to(DT[dtype])
    cu = [0] + list(np.cumsum(counts)) if packed else None
    max_pos = max(lens) + 4
    angle = torch.rand((max_pos, max(rot // 2, 1)), generator=pool.gen) * 6.3
    cos, sin = angle.cos(), angle.sin()
    pos = torch.randint(0, max_pos, (total,), generator=pool.gen, dtype=torch.int32) if explicit else None
    w = wide.to(DEV)
    if not packed:
        w = w.view(B, counts[0], *w.shape[1:])
    qd, kd, vd = w[..., :Hq, :], w[..., Hq:Hq + Hkv, :], w[..., Hq + Hkv:Hq + 2 * Hkv, :]
    kp, vp, table, kl = pool.gpu()
    out = torch.full(qd.shape, 3.0, dtype=DT[dtype], device=DEV) if Hq else None
    got = fa.fa_kv_append_paged_rope(
        kd, vd, kp, vp, table, kl, *((cos.to(DEV), sin.to(DEV)) if rot else (None, None)), q=qd if Hq else None,
        q_out=out, positions=None if pos is None else pos.to(DEV), interleaved=inter,
        cu_seqlens_new=None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert got is out
    x = wide.double().numpy()
    ref = pool.np()
    expect_q = np.full((total, Hq, D), 3.0)
    mag_q, mag_k = np.zeros_like(expect_q), np.zeros_like(ref[0])
    t = pool.table.numpy()
    for row, b, key in paged16.new_keys(lens, cu, total, B):
        at = int(pos[row]) if explicit else key
        c, s = cos[at].double().numpy()[None], sin[at].double().numpy()[None]
        turn = (lambda y: paged16.rotate(y, c, s, inter)) if rot else (lambda y: (y, np.zeros_like(y)))
        expect_q[row], mag_q[row] = turn(x[row, :Hq])
        where = paged16.place(ref[0], t, b, key)
        ref[0][where], mag_k[where] = turn(x[row, Hq:Hq + Hkv])
        ref[1][where] = x[row, Hq + Hkv:Hq + 2 * Hkv]

    def close(a, e, mag):
        a = a.double().cpu().numpy()
        same = mag == 0
        assert np.array_equal(a[same], e[same], equal_nan=True)
        a, e, mag = a[~same], e[~same], mag[~same]
        assert (abs(a - e) <= U[dtype] * abs(e) + 2.0 ** -22 * mag + TINY[dtype]).all()

    close(kp, ref[0], mag_k)
    assert np.array_equal(vp.double().cpu().numpy(), ref[1], equal_nan=True)
    if Hq:
        close(out.view(total, Hq, D), expect_q, mag_q)


def test_append_in_place_drops_and_clamps(fa):
    """q_out may be q; keys outside the table and pages outside the pool are dropped, their queries
    written all the same; positions outside the table of angles are clamped."""
    D, Hq, Hkv = 64, 4, 2
    pool = Pool(3, Hkv, D, 16, [40, 3, 33], "bf16", seed=1, max_pages=2)     # 32 keys fit: 0 loses its last row
    pool.table[2, 1] = -5                                                   # keys 16 .. 31 of 2
    x = torch.randn((3, 4, Hq + 2 * Hkv, D), generator=pool.gen).to(torch.bfloat16)
    q = x[:, :, :Hq].contiguous().to(DEV)
    before = q.double().cpu().numpy().reshape(12, Hq, D)
    kp, vp, table, kl = pool.gpu()
    cos, sin = torch.rand((50, D // 2), generator=pool.gen), torch.rand((50, D // 2), generator=pool.gen)
    pos = torch.tensor([0, 49, 50, -1] * 3, dtype=torch.int32)
    out = fa.fa_kv_append_paged_rope(x[:, :, Hq:Hq + Hkv].to(DEV), x[:, :, Hq + Hkv:].to(DEV), kp, vp, table, kl,
                                     cos.to(DEV), sin.to(DEV), q=q, q_out=q, positions=pos.view(3, 4).to(DEV))
    torch.cuda.synchronize()
    assert out is q
    ref = pool.np()
    at = pos.clamp(0, 49).long()
    c, s = cos[at].double().numpy()[:, None], sin[at].double().numpy()[:, None]
    e, mag = paged16.rotate(before, c, s, False)
    assert (abs(q.double().cpu().numpy().reshape(12, Hq, D) - e) <= 2.0 ** -8 * abs(e) + 2.0 ** -22 * mag).all()
    rows = x.double().numpy().reshape(12, Hq + 2 * Hkv, D)
    bound = np.zeros_like(ref[0])
    for row, b, key in paged16.new_keys(pool.lens, None, 12, 3):
        where = paged16.place(ref[0], pool.table.numpy(), b, key)
        if where:
            ref[0][where], m = paged16.rotate(rows[row, Hq:Hq + Hkv], c[row], s[row], False)
            bound[where] = 2.0 ** -8 * abs(ref[0][where]) + 2.0 ** -22 * m
            ref[1][where] = rows[row, Hq + Hkv:]
    got = kp.double().cpu().numpy()
    fin = np.isfinite(ref[0])
    assert np.array_equal(got[~fin], ref[0][~fin], equal_nan=True)
    assert (abs(got[fin] - ref[0][fin]) <= bound[fin]).all()
    assert np.array_equal(vp.double().cpu().numpy(), ref[1], equal_nan=True)


def test_prompt_then_drafts_then_steps(fa):
    """The operators as a serving loop uses them, one after the other on one stream without a wait:
    prompts appended, a tree of drafts appended at its depths and attended over, then steps with a
    window, each against the reference over the cache that the GPU holds at that point."""
    B, Hq, Hkv, D, page, Sq = 3, 8, 2, 128, 32, 6
    pool = Pool(B, Hkv, D, page, [0] * B, "bf16", seed=11, max_pages=9)
    kp, vp, table, kl = pool.gpu()
    freq = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
    angle = torch.arange(300, dtype=torch.float64)[:, None] * freq
    cos, sin = angle.cos().float().to(DEV), angle.sin().float().to(DEV)
    rnd = lambda *s: torch.randn(s, generator=pool.gen).to(torch.bfloat16).to(DEV)
    counts = [200, 0, 31]
    cu = torch.tensor([0, 200, 200, 231], dtype=torch.int32, device=DEV)
    kl.copy_(torch.tensor(counts, dtype=torch.int32))
    fa.fa_kv_append_paged_rope(rnd(231, Hkv, D), rnd(231, Hkv, D), kp, vp, table, kl, cos, sin, cu_seqlens_new=cu)
    tree = paged16.random_trees(np.random.default_rng(2), B, Sq)
    depth = torch.from_numpy(tree.sum(-1)).to(torch.int32).to(DEV) - 1
    positions = kl[:, None] + depth
    kl += Sq
    q = fa.fa_kv_append_paged_rope(rnd(B, Sq, Hkv, D), rnd(B, Sq, Hkv, D), kp, vp, table, kl, cos, sin,
                                   q=rnd(B, Sq, Hq, D), positions=positions)
    o, lse = fa.fa_decode_splitkv_paged_tree(q, kp, vp, table, kl,
                                             torch.from_numpy(paged16.pack_tree(tree)).to(DEV))
    pool.lens = [n + Sq for n in counts]
    pool.cpu = [kp.cpu(), vp.cpu()]
    check(o, lse, q.cpu(), pool, lambda b, n: paged16.sees_tree(n, Sq, tree[b]), 1 / math.sqrt(D), "bf16")
    kl -= 3                                                  # three drafts were accepted, the rest is overwritten
    for _ in range(3):
        kl += 1
        q = fa.fa_kv_append_paged_rope(rnd(B, 1, Hkv, D), rnd(B, 1, Hkv, D), kp, vp, table, kl, cos, sin,
                                       q=rnd(B, 1, Hq, D))
        o, lse = fa.fa_decode_splitkv_paged_window(q, kp, vp, table, kl, 63, sinks=4)
    pool.lens = kl.cpu().tolist()
    pool.cpu = [kp.cpu(), vp.cpu()]
    check(o, lse, q.cpu(), pool, lambda b, n: paged16.sees_window(n, 1, 63, 4), 1 / math.sqrt(D), "bf16")


def test_the_prompt_forward_and_the_decode_agree(fa):
    """Packed prompts of a fused projection: the append turns queries and keys and fills the cache, the
    forward with a window and sinks runs over what it turned, and the decode of the last tokens over
    the cache gives the same."""
    Hq, Hkv, D, page, left, sinks = 8, 2, 128, 16, 127, 4
    lens, cu = [300, 2, 77], [0, 300, 302, 379]
    pool = Pool(3, Hkv, D, page, lens, "bf16", seed=21)
    kp, vp, table, kl = pool.gpu()
    qkv = torch.randn((379, Hq + 2 * Hkv, D), generator=pool.gen).to(torch.bfloat16).to(DEV)
    angle = torch.arange(300, device=DEV)[:, None] * 1000.0 ** -torch.linspace(0, 1, D // 2, device=DEV)
    cud = torch.tensor(cu, dtype=torch.int32, device=DEV)
    k, v = qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    qk = fa.fa_kv_append_paged_rope(k, v, kp, vp, table, kl, angle.cos(), angle.sin(), q=qkv[:, :Hq + Hkv],
                                    cu_seqlens_new=cud)
    q, k = (x.contiguous() for x in qk.split((Hq, Hkv), 1))
    o, lse = fa.fa_fwd_varlen(q, k, v.contiguous(), cud, cud, causal=True, window=(left, 0), sinks=sinks)
    last = torch.stack([q[n - 2:n] for n in cu[1:]])
    od, lsed = fa.fa_decode_splitkv_paged_window(last, kp, vp, table, kl, left, sinks=sinks)
    torch.cuda.synchronize()
    pool.cpu = [kp.cpu(), vp.cpu()]
    t, kn, vn = pool.table.numpy(), k.double().cpu().numpy(), v.double().cpu().numpy()
    for b, n in enumerate(lens):
        rows = slice(cu[b], cu[b + 1])
        assert np.array_equal(paged16.cached(pool.np()[0], t, b, n), kn[rows])
        assert np.array_equal(paged16.cached(pool.np()[1], t, b, n), vn[rows])
        part = Pool.__new__(Pool)
        part.__dict__.update(lens=[n], cpu=pool.cpu, table=pool.table[b:b + 1])
        check(o[None, rows], lse[None, :, rows], q[None, rows].cpu(), part,
              lambda _, m: paged16.sees_window(m, m, left, sinks), 1 / math.sqrt(D), "bf16")
    check(od, lsed, last.cpu(), pool, lambda b, n: paged16.sees_window(n, 2, left, sinks), 1 / math.sqrt(D), "bf16")


@pytest.mark.parametrize("S", [77, 1500])
def test_append_and_forward_on_one_buffer_without_a_wait(fa, S):
    """The append turns queries into a buffer that the forward with sinks reads, over and over without a
    wait or another kernel between them: neither starts on what the other is not done with."""
    Hq, Hkv, D, n = 8, 2, 128, 12
    pool = Pool(1, Hkv, D, 16, [S], "bf16", seed=5)
    kp, vp, table, kl = pool.gpu()
    rnd = lambda *s: torch.randn(s, generator=pool.gen).to(torch.bfloat16).to(DEV)
    q, k, v = [rnd(1, S, Hq, D) for _ in range(n)], rnd(1, S, Hkv, D), rnd(1, S, Hkv, D)
    angle = torch.rand((S, D // 2), device=DEV)
    cos, sin = angle.cos(), angle.sin()
    turned, outs = torch.empty_like(q[0]), [torch.empty_like(q[0]) for _ in range(n)]
    lse = torch.empty((1, Hq, S), device=DEV)
    for wait in (True, False):
        want = [o.clone() for o in outs] if not wait else None
        for o in outs:
            o.fill_(7.0)
        torch.cuda.synchronize()
        for i in range(n):
            fa.fa_kv_append_paged_rope(k, v, kp, vp, table, kl, cos, sin, q=q[i], q_out=turned)
            if wait:
                torch.cuda.synchronize()
            fa.fa_fwd(turned, k, v, causal=True, window=(63, 0), sinks=4, out=outs[i], lse=lse)
            if wait:
                torch.cuda.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
