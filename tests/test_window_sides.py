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
