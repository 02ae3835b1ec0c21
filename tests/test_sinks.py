"""fa_fwd_sinks and fa_fwd_varlen_sinks, the windowed forward whose first keys stay visible, on the
GPU against a 64-bit reference (oracle/paged16.py's attention under the mask below).

Bounds per output value, from the roundings (u = eps / 2 of the type; half a step each):
    |dO| <= u |O| + c A + f T,  A = sum_j p_j |v_j|, T = max_j p_j sum_j |v_j| over the row's keys,
    c = u (P rounded for the product) + 2 e_s + 2^-21 + N 2^-23,
    e_s = (D + 8) 2^-22 max_j scale sum_d |q_d k_jd| (a score, a sum of D products in 32 bits in any
    order, each step allowed a truncation; twice, for numerator and denominator), 2^-21: exp2 and the
    division, N = n / 4 + 64 sums over the n keys, f = 2^-25 in fp16 (P below 2^-14 has steps of 2^-24,
    the largest weight being at least 1), 0 in bf16;
    |dLSE| <= e_s + 2^-21 + N 2^-23 + 2^-22 |LSE|.
"""
import math

import numpy as np
import pytest
import torch

from oracle import paged16

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
TINY = {"bf16": 2.0 ** -133, "fp16": 2.0 ** -24}
DEV = "cuda:0"
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import exact_tiled_attention_20_gb300 as fa_mod
    from exact_tiled_attention_20_gb300 import build

    build.build_library()
    fa_mod.load()
    return fa_mod


def sees(Sq, Sk, causal, left, right, sinks):
    """[Sq, Sk]"""
    p, j = np.arange(Sq)[:, None] + Sk - Sq, np.arange(Sk)[None]
    hi = p if causal else p + right if right >= 0 else np.full_like(p, Sk - 1)
    return (j <= hi) & ((j >= p - left if left >= 0 else np.full((Sq, Sk), True)) | (j < sinks))


def check(o, lse, q, k, v, seen, scale, dtype, rows=None):
    """One sequence: o, q [Sq, Hq, D], lse [Hq, Sq], k and v [Sk, Hkv, D]; rows: those that are checked."""
    rows = np.arange(q.shape[0]) if rows is None else rows
    o, lse, q, k, v = (t.double().cpu().numpy() for t in (o, lse, q, k, v))
    o, lse, q, seen, D = o[rows], lse[:, rows], q[rows], seen[rows], q.shape[-1]
    ro, rl, A, T, E = paged16.attend(q, k, v, seen, scale)
    e_s, u = (D + 8) * 2.0 ** -22 * E, U[dtype]
    common = 2.0 ** -21 + (seen.sum(1).max() / 4 + 64) * 2.0 ** -23
    bound = u * abs(ro) + (u + 2 * e_s.T[..., None] + common) * A + (2.0 ** -25 * T if dtype == "fp16" else 0) + TINY[dtype]
    fin = np.isfinite(ro)
    assert np.array_equal(np.isnan(o), np.isnan(ro)), "NaN pattern"
    assert np.array_equal(o[~fin & ~np.isnan(ro)], ro[~fin & ~np.isnan(ro)]), "infinities"
    off = abs(o[fin] - ro[fin]) / bound[fin]
    assert off.max() <= 1, f"|dO| is {off.max():.2f} of its bound"
    some = np.isfinite(rl)
    assert np.array_equal(some, np.isfinite(lse)) and (lse[~some] == -np.inf).all(), "LSE pattern"
    off = abs(lse[some] - rl[some]) / (e_s[some] + common + 2.0 ** -22 * abs(rl[some]))
    assert off.size == 0 or off.max() <= 1, f"|dLSE| is {off.max():.2f} of its bound"


def make(B, Sq, Sk, Hq, Hkv, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(s, generator=g).to(DT[dtype]) for s in ((B, Sq, Hq, D), (B, Sk, Hkv, D), (B, Sk, Hkv, D))]


CASES = [
    # (B, Sq, Sk, Hq, Hkv, D, left, right, causal, sinks, dtype)
    (1, 600, 600, 2, 1, 128, 100, 0, True, 4, "bf16"),
    (2, 1030, 1030, 2, 2, 128, 127, 0, True, 1, "fp16"),       # a window of one block: most dead for a sub-tile
    (1, 1100, 1100, 2, 1, 96, 200, 0, True, 300, "bf16"),      # sinks over three blocks, and inside windows
    (1, 700, 700, 4, 2, 64, 90, 0, True, 130, "bf16"),
    (1, 500, 500, 2, 1, 256, 64, 0, True, 65, "fp16"),
    (1, 300, 333, 2, 1, 256, 40, 10, False, 7, "bf16"),        # a right side
    (1, 400, 400, 2, 2, 128, 0, -1, False, 3, "bf16"),         # no right side
    (1, 200, 900, 2, 2, 128, 300, 0, True, 5, "bf16"),         # fewer queries than keys
    (1, 500, 120, 2, 1, 128, 30, 5, False, 9, "fp16"),         # more queries: leading rows see no key
    (1, 500, 120, 2, 1, 64, 30, 0, True, 9, "bf16"),
    (1, 1, 1000, 4, 1, 64, 17, 0, True, 2, "bf16"),            # one query
    (1, 1, 1, 1, 1, 128, 0, 0, True, 1, "bf16"),
    (1, 400, 400, 2, 1, 128, 0, 0, True, 1, "bf16"),           # itself and the first key
    (1, 260, 260, 2, 1, 96, 50, 0, True, 10 ** 9, "fp16"),     # every key a sink: causal
    (1, 50, 300, 6, 3, 128, 10 ** 9, 0, True, 4, "bf16"),      # a window past every key
]


@gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: "_".join(map(str, c)))
def test_sinks_match_the_reference(fa, case):
    B, Sq, Sk, Hq, Hkv, D, left, right, causal, sinks, dtype = case
    q, k, v = make(B, Sq, Sk, Hq, Hkv, D, dtype, seed=Sq + left % 1000)
    o, lse = fa.fa_fwd(q.to(DEV), k.to(DEV), v.to(DEV), causal=causal, window=(left, right), sinks=sinks)
    torch.cuda.synchronize()
    seen = sees(Sq, Sk, causal, left, right, sinks)
    for b in range(B):
        check(o[b], lse[b], q[b], k[b], v[b], seen, 1 / math.sqrt(D), dtype)


@gpu
@pytest.mark.parametrize("Hq,Hkv,D,left,sinks,dtype", [
    (4, 2, 128, 70, 4, "bf16"), (2, 2, 64, 129, 1, "fp16"), (3, 1, 96, 0, 200, "bf16"), (2, 1, 256, 100, 63, "fp16")])
def test_packed_sinks_match_the_reference(fa, Hq, Hkv, D, left, sinks, dtype):
    """Sequences without queries, without keys, longer and shorter than a tile; rows behind the last
    one are left as they were."""
    nq, nk = [300, 0, 1, 77, 513, 5], [300, 9, 400, 200, 513, 0]
    cq, ck = np.concatenate([[0], np.cumsum(nq)]), np.concatenate([[0], np.cumsum(nk)])
    q, k, v = make(1, cq[-1] + 5, ck[-1] + 3, Hq, Hkv, D, dtype, seed=D)
    q, k, v = q[0], k[0], v[0]
    k[ck[-1]:], v[ck[-1]:] = math.nan, math.nan
    o = torch.full(q.shape, 3.0, dtype=q.dtype, device=DEV)
    lse = torch.full((Hq, q.shape[0]), 3.0, device=DEV)
    cu = [torch.tensor(c, dtype=torch.int32, device=DEV) for c in (cq, ck)]
    fa.fa_fwd_varlen(q.to(DEV), k.to(DEV), v.to(DEV), *cu, causal=True, window=(left, 0), sinks=sinks, out=o, lse=lse)
    torch.cuda.synchronize()
    assert (o[cq[-1]:] == 3).all() and (lse[:, cq[-1]:] == 3).all()
    for b in range(len(nq)):
        if nq[b]:
            a, e = cq[b], cq[b + 1]
            check(o[a:e], lse[:, a:e], q[a:e], k[ck[b]:ck[b + 1]], v[ck[b]:ck[b + 1]],
                  sees(nq[b], nk[b], True, left, 0, sinks), 1 / math.sqrt(D), dtype)


@gpu
@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("packed", [False, True])
def test_values_that_are_not_finite_stay_behind_the_mask(fa, D, packed):
    """NaN and infinities in K and V of keys that some rows do not see reach those that do alone."""
    Sq, Sk, Hq, Hkv, left, sinks = 400, 420, 4, 2, 60, 5
    q, k, v = make(1, Sq, Sk, Hq, Hkv, D, "bf16", seed=D)
    v[0, 100, 0, 3], v[0, 250, 0, D - 1], v[0, 2, 1, 40], v[0, 419, 1, 0] = math.nan, math.inf, -math.inf, math.nan
    for n in (300, 305):
        v[0, n, 1] = math.nan
    dev = [t.to(DEV) for t in (q, k, v)]
    cu = [torch.tensor([0, n], dtype=torch.int32, device=DEV) for n in (Sq, Sk)]

    def call():
        if packed:
            o, lse = fa.fa_fwd_varlen(*(t[0] for t in dev), *cu, causal=True, window=(left, 0), sinks=sinks)
            return o[None], lse[None]
        return fa.fa_fwd(*dev, causal=True, window=(left, 0), sinks=sinks)

    seen = sees(Sq, Sk, True, left, 0, sinks)
    o, lse = call()
    torch.cuda.synchronize()
    check(o[0], lse[0], q[0], k[0], v[0], seen, 1 / math.sqrt(D), "bf16")
    dev[1][0, 200, 0, 1] = math.nan                       # in K: the rows that see it are NaN, the others as before
    o2, lse2 = call()
    torch.cuda.synchronize()
    hit = torch.from_numpy(seen[:, 200]).to(DEV)
    assert torch.isnan(o2[0, hit, :2]).all() and torch.isnan(lse2[0, :2][:, hit]).all()
    eq = (o2 == o) | (torch.isnan(o2) & torch.isnan(o))
    assert eq[0, ~hit].all() and eq[0, :, 2:].all() and torch.equal(lse2[0, :2][:, ~hit], lse[0, :2][:, ~hit])


@gpu
def test_no_sinks_or_no_window_is_the_forward_bit_for_bit(fa):
    q, k, v = (t.to(DEV) for t in make(2, 520, 520, 4, 2, 128, "bf16", seed=410))
    for win, sinks in (((100, 0), 0), ((-1, -1), 7), ((520, 0), 7)):
        a = fa.fa_fwd(q, k, v, causal=True, window=win, sinks=sinks)
        b = fa.fa_fwd(q, k, v, causal=True, window=win if sinks == 0 else None)
        torch.cuda.synchronize()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), (win, sinks)


@gpu
def test_long_prompt_guards_and_a_graph(fa):
    """[1, 8192, 4, 128] with a window of 1024 and four sinks: sampled rows against the reference; the
    same bits again from a captured graph, into the middle of a larger buffer."""
    q, k, v = make(1, 8192, 8192, 4, 2, 128, "bf16", seed=7)
    d = [t.to(DEV) for t in (q, k, v)]
    o, lse = fa.fa_fwd(*d, causal=True, window=(1023, 0), sinks=4)
    torch.cuda.synchronize()
    rows = np.unique(np.concatenate([[0, 3, 4, 1023, 1024, 1027, 1028, 8191], np.random.default_rng(5).integers(0, 8192, 40)]))
    check(o[0], lse[0], q[0], k[0], v[0], sees(8192, 8192, True, 1023, 0, 4), 1 / math.sqrt(128), "bf16", rows)
    big = torch.full((3, 8192, 4, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    bl = torch.full((3, 4, 8192), 7.0, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fa_fwd(*d, causal=True, window=(1023, 0), sinks=4, out=big[1:2], lse=bl[1:2])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(big[1], o[0]) and torch.equal(bl[1], lse[0])
    assert (big[0] == 7).all() and (big[2] == 7).all() and (bl[0] == 7).all() and (bl[2] == 7).all()


@gpu
def test_a_prompt_then_steps_agree_with_one_prompt(fa):
    """A prompt of n + 3 tokens with window and sinks, and a prompt of n followed by three steps over the
    paged cache: the last rows agree within both operators' bounds."""
    B, n, Hq, Hkv, D, page, left, sinks = 2, 700, 8, 2, 128, 64, 127, 4
    q, k, v = make(B, n + 3, n + 3, Hq, Hkv, D, "bf16", seed=3)
    d = [t.to(DEV) for t in (q, k, v)]
    whole, whole_lse = fa.fa_fwd(*d, causal=True, window=(left, 0), sinks=sinks)
    kp, vp = (torch.zeros((B * 11, page, Hkv, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    table = torch.arange(B * 11, dtype=torch.int32, device=DEV).flip(0).view(B, 11).contiguous()
    lens = torch.full((B,), n, dtype=torch.int32, device=DEV)
    fa.fa_kv_append_paged_rope(d[1][:, :n].contiguous(), d[2][:, :n].contiguous(), kp, vp, table, lens)
    seen = sees(n + 3, n + 3, True, left, 0, sinks)
    for i in range(3):
        lens += 1
        fa.fa_kv_append_paged_rope(*(t[:, n + i:n + i + 1].contiguous() for t in d[1:]), kp, vp, table, lens)
        o, lse = fa.fa_decode_splitkv_paged_window(d[0][:, n + i:n + i + 1].contiguous(), kp, vp, table, lens, left,
                                                   sinks=sinks)
        torch.cuda.synchronize()
        for b in range(B):
            row = slice(n + i, n + i + 1)
            check(o[b], lse[b], q[b, row], k[b], v[b], seen[row], 1 / math.sqrt(D), "bf16")
            check(whole[b, row], whole_lse[b, :, row], q[b, row], k[b], v[b], seen[row], 1 / math.sqrt(D), "bf16")


FAKE = 1 << 20


@pytest.mark.parametrize("change,code", [
    (dict(sinks=-1), 1), (dict(left=-2), 1), (dict(right=-2), 1), (dict(q=None), 1), (dict(k=FAKE + 8), 1),
    (dict(lse=FAKE + 2), 1), (dict(Sq=0), 1), (dict(Hq=3), 1), (dict(scale=float("nan")), 1), (dict(scale=0.0), 1),
    (dict(scale=-1.0), 1), (dict(D=80), 2),
    (dict(dtype=7), 2), (dict(B=1 << 16, Sq=1 << 16), 2)])
def test_sinks_refuse(change, code):
    from exact_tiled_attention_20_gb300 import _lib, build

    build.build_library()
    args = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, lse=None, B=1, Sq=8, Sk=8, Hq=2, Hkv=2, D=64, scale=0.1, causal=1, left=4,
                right=0, sinks=2, dtype=0, stream=None)
    assert _lib.load().fa_fwd_sinks(*{**args, **change}.values()) == code


@pytest.mark.parametrize("change,code", [
    (dict(sinks=-1), 1), (dict(left=-2), 1), (dict(cu_q=None), 1), (dict(cu_k=FAKE + 2), 1), (dict(total_q=0), 1),
    (dict(scale=0.0), 1),
    (dict(B=1025), 2), (dict(D=80), 2)])
def test_packed_sinks_refuse(change, code):
    import ctypes

    from exact_tiled_attention_20_gb300 import build

    P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib = ctypes.CDLL(build.build_library())
    lib.fa_fwd_varlen_sinks.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, F, I, I, I, I, I, P]
    args = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, lse=None, cu_q=FAKE, cu_k=FAKE, B=1, total_q=8, total_k=8, Hq=2, Hkv=2,
                D=64, scale=0.1, causal=1, left=4, right=0, sinks=2, dtype=0, stream=None)
    assert lib.fa_fwd_varlen_sinks(*{**args, **change}.values()) == code
