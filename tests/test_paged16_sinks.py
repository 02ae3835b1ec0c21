"""The window decode over the 16-bit paged cache with long stretches of sinks (fa_decode_splitkv_paged_window), on
the GPU against the reference and the bounds of test_paged16."""
import math

import pytest
import torch

from oracle import paged16
from test_paged16 import DEV, Pool, check, fa, queries  # noqa: F401  (fa is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,Sq,Hq,dtype", [(64, 1, 4, "bf16"), (128, 3, 4, "bf16"), (96, 40, 4, "fp16"),
                                           (128, 70, 8, "bf16"), (256, 2, 2, "fp16")])
@pytest.mark.parametrize("sinks", [31, 32, 33, 96, 500, 511, 10 ** 6])
def test_sinks_that_hold_values_that_are_not_finite(fa, D, Sq, Hq, dtype, sinks):  # noqa: F811
    """Among sinks that fill whole strips of 32 keys, and in the last one, which they share."""
    left = 40
    pool = Pool(3, 2, D, 48, [900, 130, 560], dtype, seed=D + sinks % 1000).fill()
    q = queries(pool, 3, Sq, Hq, D, dtype)
    v = pool.cpu[1]
    for b, key, h, d, x in ((0, 5, 0, 1, math.nan), (0, 31, 1, D - 1, math.inf), (0, 70, 1, 2, -math.inf),
                            (0, 510, 0, 40, math.inf), (1, 32, 0, 3, math.inf), (1, 95, 1, 9, math.nan),
                            (2, 499, 1, 5, math.nan), (2, 559, 0, 6, math.inf), (2, 530, 1, 7, math.nan)):
        v[int(pool.table[b, key // 48]), key % 48, h, d] = x
    o, lse = fa.fa_decode_splitkv_paged_window(q.to(DEV), *pool.gpu(), left, sinks=sinks)
    torch.cuda.synchronize()
    check(o, lse, q, pool, lambda b, n: paged16.sees_window(n, Sq, left, sinks), 1 / math.sqrt(D), dtype)


@pytest.mark.parametrize("D,Hq", [(128, 4), (128, 32), (256, 4)])
@pytest.mark.parametrize("bad", [0, 20380])
def test_one_bad_value_among_many_sinks_costs_little(fa, D, Hq, bad):  # noqa: F811
    """160 sequences of 20000 sinks (of the same pages), most worked on in one piece or two: a NaN in V, of a
    sink or in the strip where the window begins, is not looked for in all of the sinks, key by key, while
    other warps wait for 2 s at most."""
    n, B, page = 20480, 160, 256
    g = torch.Generator(device=DEV).manual_seed(3)
    k, v = (torch.randn((n // page, page, 1, D), generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    q = torch.randn((B, 1, Hq, D), generator=g, device=DEV).to(torch.bfloat16)
    table = torch.arange(n // page, dtype=torch.int32, device=DEV).repeat(B, 1)
    lens = torch.full((B,), n, dtype=torch.int32, device=DEV)
    v[bad // page, bad % page, 0, 3] = math.nan

    def call():
        return fa.fa_decode_splitkv_paged_window(q, k, v, table, lens, 100, sinks=20000)

    call()
    a, e = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    o, lse = call()
    e.record()
    torch.cuda.synchronize()
    assert torch.isnan(o[..., 3]).all() and torch.isfinite(o[..., 4:]).all() and torch.isfinite(lse).all()
    print(f"{a.elapsed_time(e):.2f} ms")
    assert a.elapsed_time(e) < 20
