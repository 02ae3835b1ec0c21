"""Infinities and NaNs in V under the forward with sinks (fa_fwd_sinks, fa_fwd_varlen_sinks): they reach the
rows that see them and no others, whatever the lengths.  Against the 64-bit reference and the bounds of
test_sinks."""
import math

import numpy as np
import pytest
import torch

from test_sinks import DEV, check, fa, make, sees  # noqa: F401  (fa is a fixture)

pytestmark = pytest.mark.gpu
BAD = (math.nan, math.inf, -math.inf)


def call(fa, packed, q, k, v, causal, win, sinks):  # noqa: F811
    d = [t.to(DEV) for t in (q, k, v)]
    if packed:
        cu = [torch.tensor([0, t.shape[1]], dtype=torch.int32, device=DEV) for t in (q, k)]
        o, lse = fa.fa_fwd_varlen(*(t[0] for t in d), *cu, causal=causal, window=win, sinks=sinks)
        o, lse = o[None], lse[None]
    else:
        o, lse = fa.fa_fwd(*d, causal=causal, window=win, sinks=sinks)
    torch.cuda.synchronize()
    return o, lse


@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (96, "fp16"), (128, "bf16"), (128, "fp16"), (256, "fp16")])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("sinks", [5, 150])
def test_many_values_that_are_not_finite(fa, D, dtype, packed, sinks):  # noqa: F811
    """Sinks, single values, whole rows of V: rows that see one have it in those dims; the others have the
    bits of a call whose V is zero there."""
    Sq, Sk, left = 900, 1000, 130
    q, k, v = make(1, Sq, Sk, 4, 2, D, dtype, seed=D + sinks)
    g = np.random.default_rng(D)
    for key in (0, 3, 200, 201, 202, 640, 999):
        for d in g.integers(0, D, 3):
            v[0, key, key % 2, d] = BAD[int(g.integers(0, 3))]
    v[0, 400:420, 1] = math.nan
    v[0, 777, 0] = math.inf
    o, lse = call(fa, packed, q, k, v, True, (left, 0), sinks)
    seen = sees(Sq, Sk, True, left, 0, sinks)
    check(o[0], lse[0], q[0], k[0], v[0], seen, 1 / math.sqrt(D), dtype)
    clean = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
    o0, lse0 = call(fa, packed, q, k, clean, True, (left, 0), sinks)
    bad = ~torch.isfinite(v[0]).repeat_interleave(2, dim=1)                       # [Sk, Hq, D]
    hit = torch.einsum("ij,jhd->ihd", torch.from_numpy(seen).float(), bad.float()) > 0
    assert torch.equal(o.cpu()[0][~hit], o0.cpu()[0][~hit]) and torch.equal(lse, lse0)
    assert not torch.isfinite(o.cpu()[0][hit]).any()


def test_rows_that_see_very_many_keys(fa):  # noqa: F811
    """No right side: rows see up to 2^18 keys, and a NaN that 100 of them do not see stays out of these."""
    n, D = 1 << 18, 64
    q, k, v = make(1, n, n, 1, 1, D, "bf16", seed=1)
    v[0, 5, 0, 3], v[0, n - 300, 0, 60] = math.nan, math.inf
    o, lse = call(fa, False, q, k, v, False, (10, -1), 4)
    rows = np.array([0, 15, 16, 100, n - 291, n - 290, n - 289, n - 1])
    seen = np.zeros((n, 1), bool)  # only the rows that are checked are made
    at = rows[:, None] - 10
    seen = (np.arange(n)[None] >= at) | (np.arange(n)[None] < 4)
    full = {int(r): s for r, s in zip(rows, seen)}
    for r in rows:
        one = slice(int(r), int(r) + 1)
        check(o[0, one], lse[0, :, one], q[0, one], k[0], v[0], full[int(r)][None], 1 / math.sqrt(D), "bf16")


def test_early_rows_of_a_very_long_window(fa):  # noqa: F811
    """A window of over 2^20 keys: the first rows see few, and not the NaN behind them."""
    n, left, D = (1 << 20) + 2048, (1 << 20) + 1000, 64
    q, k, v = make(1, n, n, 1, 1, D, "bf16", seed=2)
    v[0, 310, 0, 7] = math.nan
    o, lse = call(fa, False, q, k, v, True, (left, 0), 4)
    m = 700
    check(o[0, :m], lse[0, :, :m], q[0, :m], k[0, :m], v[0, :m], sees(m, m, True, left, 0, 4), 1 / math.sqrt(D), "bf16")
    assert torch.isnan(o[0, 310:311 + left, 0, 7]).all() and torch.isfinite(o[0, 311 + left:, 0, 7]).all()
    assert torch.isfinite(o[0, :, 0, 8]).all()


def test_keys_past_the_packed_tensor_are_zeros(fa):  # noqa: F811
    """cu_seqlens_k that ends past total_k: the missing keys read as zeros, and a V that is not finite changes
    nothing about that."""
    nq, nk, total_k, D, left, sinks = [200, 350], [100, 400], 320, 128, 90, 6
    q, k, v = (t[0] for t in make(1, sum(nq), sum(nk), 2, 1, D, "bf16", seed=9))
    k[total_k:], v[total_k:] = 0, 0
    v[130, 0, 5], v[319, 0, 77], v[10, 0, 0] = math.nan, math.inf, -math.inf
    cu = [torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device=DEV) for n in (nq, nk)]
    o, lse = fa.fa_fwd_varlen(q.to(DEV), k[:total_k].to(DEV), v[:total_k].to(DEV), *cu, causal=True, window=(left, 0),
                              sinks=sinks)
    torch.cuda.synchronize()
    for b, (a, e, ka, ke) in enumerate(((0, 200, 0, 100), (200, 550, 100, 500))):
        check(o[a:e], lse[:, a:e], q[a:e], k[ka:ke], v[ka:ke], sees(nq[b], nk[b], True, left, 0, sinks),
              1 / math.sqrt(D), "bf16")


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_graph_replayed_with_finite_and_other_values(fa, D):  # noqa: F811
    """Many tiles a CTA: nothing of a call with values that are not finite is left for the next."""
    B, n, Hq, Hkv = 2, 2100, 16, 4
    q, k, v = (t.to(DEV) for t in make(B, n, n, Hq, Hkv, D, "bf16", seed=D))
    kw = dict(causal=True, window=(300, 0), sinks=4)
    o, lse = fa.fa_fwd(q, k, v, **kw)
    g, go, gl = torch.cuda.CUDAGraph(), torch.empty_like(o), torch.empty_like(lse)
    with torch.cuda.graph(g):
        fa.fa_fwd(q, k, v, out=go, lse=gl, **kw)
    keep = v.clone()
    for key, value in ((2, math.nan), (1000, math.inf), (None, 0)):
        v.copy_(keep)
        if key is not None:
            v[1, key, 2, D // 2] = value
        g.replay()
        torch.cuda.synchronize()
        i = torch.arange(n, device=DEV)
        hit = torch.zeros((B, n, Hq, D), dtype=torch.bool, device=DEV)
        if key is not None:
            hit[1, :, 8:12, D // 2] = ((i >= key) & ((i <= key + 300) | (key < 4)))[:, None]
        assert torch.equal(go[~hit], o[~hit]) and torch.equal(gl, lse), key
        assert not torch.isfinite(go[hit]).any(), key
