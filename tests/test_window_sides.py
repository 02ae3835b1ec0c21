"""Sides of a window that reach past every key, up to the largest number a call takes: a right side of at
least the queries and a left side of at least the keys leave that side open (fa_fwd_window, fa_fwd_varlen,
fa_fwd_sinks, fa_fwd_varlen_sinks).  Against the 64-bit reference and the bounds of test_sinks."""
import math

import numpy as np
import pytest
import torch

from test_sinks import DEV, check, fa, make, sees  # noqa: F401  (fa is a fixture)

MAX = 2 ** 31 - 1
# (Sq, Sk, Hq, Hkv, D, dtype)
SHAPES = [(400, 400, 2, 1, 128, "bf16"), (300, 700, 2, 2, 96, "fp16"), (700, 290, 2, 1, 64, "bf16"),
          (290, 130, 2, 2, 256, "fp16"), (500, 120, 2, 1, 128, "bf16")]
WINDOWS = [(100, MAX), (100, MAX - 1), (100, MAX - 400), (100, 10 ** 9), (MAX, 3), (MAX, MAX), (10 ** 9, 0),
           (MAX - 120, 200), (MAX, -1), (0, MAX)]


@pytest.mark.gpu
@pytest.mark.parametrize("sinks", [0, 4, 200])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda c: "_".join(map(str, c)))
def test_fixed_length_sides_past_every_key(fa, shape, sinks):  # noqa: F811
    Sq, Sk, Hq, Hkv, D, dtype = shape
    q, k, v = make(1, Sq, Sk, Hq, Hkv, D, dtype, seed=Sq + Sk)
    d = [t.to(DEV) for t in (q, k, v)]
    for left, right in WINDOWS:
        o, lse = fa.fa_fwd(*d, window=(left, right), sinks=sinks)
        torch.cuda.synchronize()
        check(o[0], lse[0], q[0], k[0], v[0], sees(Sq, Sk, False, left, right, sinks), 1 / math.sqrt(D), dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("sinks", [0, 5])
@pytest.mark.parametrize("D,dtype", [(128, "bf16"), (64, "fp16"), (256, "bf16")])
def test_packed_sides_past_every_key(fa, D, dtype, sinks):  # noqa: F811
    nq, nk, Hq, Hkv = [300, 1, 77, 413], [180, 90, 0, 500], 2, 1
    cq, ck = np.concatenate([[0], np.cumsum(nq)]), np.concatenate([[0], np.cumsum(nk)])
    q, k, v = (t[0] for t in make(1, cq[-1], ck[-1], Hq, Hkv, D, dtype, seed=D))
    d = [t.to(DEV) for t in (q, k, v)]
    cu = [torch.tensor(c, dtype=torch.int32, device=DEV) for c in (cq, ck)]
    for left, right in WINDOWS:
        o, lse = fa.fa_fwd_varlen(*d, *cu, window=(left, right), sinks=sinks)
        torch.cuda.synchronize()
        for b in range(len(nq)):
            a, e = cq[b], cq[b + 1]
            check(o[a:e], lse[:, a:e], q[a:e], k[ck[b]:ck[b + 1]], v[ck[b]:ck[b + 1]],
                  sees(nq[b], nk[b], False, left, right, sinks), 1 / math.sqrt(D), dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("sinks", [0, 4])
def test_numbers_past_32_bits(fa, sinks):  # noqa: F811
    """Python's integers do not wrap on their way into the library: a side past every key is one of
    2**31 - 1, and a number far below zero is refused."""
    q, k, v = (t.to(DEV) for t in make(1, 300, 300, 2, 1, 128, "bf16", seed=5))
    cu = torch.tensor([0, 300], dtype=torch.int32, device=DEV)

    def fixed(win, n=sinks):
        return fa.fa_fwd(q, k, v, window=win, sinks=n)

    def packed(win, n=sinks):
        return fa.fa_fwd_varlen(q[0], k[0], v[0], cu, cu, window=win, sinks=n)

    for call in (fixed, packed):
        for win, same in (((2 ** 32 + 9, 7), (MAX, 7)), ((50, 2 ** 32), (50, MAX)), ((2 ** 63, 2 ** 70), (MAX, MAX))):
            a, b = call(win), call(same)
            torch.cuda.synchronize()
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), win
        for win in ((-2 ** 32, 0), (5, -2 ** 32 - 1), (-2 ** 33 + 4, -1)):
            with pytest.raises(fa.FaError):
                call(win)
        with pytest.raises(fa.FaError):
            call((50, 0), -2 ** 32)
    pages = torch.zeros((3, 16, 1, 128), dtype=torch.bfloat16, device=DEV)
    table, lens = torch.arange(3, dtype=torch.int32, device=DEV)[None], torch.tensor([40], dtype=torch.int32, device=DEV)
    for left, n in ((-2 ** 32, 0), (-2 ** 32 - 1, 0), (3, -2 ** 32)):
        with pytest.raises(fa.FaError):
            fa.fa_decode_splitkv_paged_window(q[:, :1].contiguous(), pages, pages, table, lens, left, sinks=n)
