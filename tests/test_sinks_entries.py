"""fa_fwd_sinks and fa_fwd_varlen_sinks called as C functions where the sinks do not matter (none, an open left
side, or one of at least the keys): they are fa_fwd_window and fa_fwd_varlen, bit for bit."""
import ctypes
import math

import pytest
import torch

from test_sinks import DEV, fa, make  # noqa: F401  (fa is a fixture)

P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float


@pytest.fixture(scope="module")
def lib(fa):  # noqa: F811
    from exact_tiled_attention_20_gb300 import build

    lib = ctypes.CDLL(build.build_library())
    fixed, packed = [P] * 5 + [I] * 6 + [F] + [I] * 3, [P] * 7 + [I] * 6 + [F] + [I] * 3
    lib.fa_fwd_window.argtypes, lib.fa_fwd_varlen.argtypes = fixed + [I, P], packed + [I, P]
    lib.fa_fwd_sinks.argtypes, lib.fa_fwd_varlen_sinks.argtypes = fixed + [I, I, P], packed + [I, I, P]
    return lib


WITHOUT = [((100, 0), 0), ((100, 30), 0), ((0, -1), 0), ((-1, -1), 7), ((-1, 25), 600), ("keys", 7), ("more", 7)]


def sides(win, keys):
    return {"keys": (keys, 5), "more": (keys + 900, 5)}.get(win, win)


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("D,dtype,Sq,Sk", [(64, "fp16", 300, 520), (96, "bf16", 520, 520), (128, "bf16", 700, 333),
                                           (256, "fp16", 270, 390)])
def test_fixed_length(lib, D, dtype, Sq, Sk, causal):
    q, k, v = (t.to(DEV) for t in make(2, Sq, Sk, 4, 2, D, dtype, seed=D))

    def call(entry, *more):
        o, lse = torch.full_like(q, 7), torch.full((2, 4, Sq), 7.0, device=DEV)
        st = entry(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), 2, Sq, Sk, 4, 2, D,
                   1 / math.sqrt(D), causal, *more, int(dtype == "fp16"), torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert st == 0
        return o, lse

    for win, sinks in WITHOUT:
        win = sides(win, Sk)
        a, b = call(lib.fa_fwd_sinks, *win, sinks), call(lib.fa_fwd_window, *win)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), (win, sinks)


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "fp16"), (256, "bf16")])
def test_packed(lib, D, dtype, causal):
    cu_q, cu_k = ([0, 200, 200, 531, 600], [0, 150, 190, 520, 520])
    q, k, v = (t[0].to(DEV) for t in make(1, 600, 520, 4, 2, D, dtype, seed=D))
    cq, ck = (torch.tensor(c, dtype=torch.int32, device=DEV) for c in (cu_q, cu_k))

    def call(entry, *more):
        o, lse = torch.full_like(q, 7), torch.full((4, 600), 7.0, device=DEV)
        st = entry(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), cq.data_ptr(), ck.data_ptr(), 4,
                   600, 520, 4, 2, D, 1 / math.sqrt(D), causal, *more, int(dtype == "fp16"),
                   torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert st == 0
        return o, lse

    for win, sinks in WITHOUT:
        win = sides(win, 520)
        a, b = call(lib.fa_fwd_varlen_sinks, *win, sinks), call(lib.fa_fwd_varlen, *win)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), (win, sinks)
