"""The 8-bit paged KV cache on the GPU against its 64-bit reference (oracle/kv8.py).

Writing and reading back are exact by definition (a power-of-two scale, one rounding), so
codes, scales and read values are compared bit for bit.

The decode's bound, per output value, from its roundings (a rounding is off by at most half
a step: 2^-9 ... here taken as eps / 2 of the type):
    |dO| <= u_o |O| + c A + 2^-36 T,   A = sum_j p_j |v_j|,   T = max_j (p_j vscale_j) sum_j |vcode_j|
    u_o  one rounding of the output: 2^-8 (bf16), 2^-11 (fp16); of a subnormal, half of its step
    c    2^-11 (P rounded to fp16) + 2 e_s + 2^-21 + N 2^-23
    e_s  error of a score, in its exponent: (D + 8) 2^-22 max_j scale sum_d |q_d k_jd| (a sum of
         D products in 32 bits in any order, each step allowed a truncation, and the scale
         factors), twice because it enters the numerator and the denominator; 2^-21 is
         exp2's and the division's; N = n / 4 + 64 sums over the n keys (at least four
         partial sums run side by side in any split)
    T    P_j is fp16(2^11 w_j / r), w_j = p_j vscale_j, with r at least 2^-4 of the largest w and at
         most it: below 2^-14 its steps are 2^-24, an error of at most 2^-25 r / 2^11 <= 2^-36 max w
         for each key, whose code it multiplies
and |dLSE| <= e_s + (2^-21 + N 2^-23) + 2^-22 |LSE|.
"""
import math

import numpy as np
import pytest
import torch

from oracle import kv8

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
U_O = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
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


class Pool:
    """A pool on the GPU filled with random bytes (NaN codes and scale byte 255 among them:
    nothing outside the sequences may matter), its copy in numpy and a scattered table."""

    def __init__(self, pages, Hkv, page, D, B, max_pages, seed=0):
        rng = np.random.default_rng(seed)
        self.np = [rng.integers(0, 256, (pages, Hkv, page, D), dtype=np.uint8) for _ in range(2)] + \
                  [rng.integers(0, 256, (pages, Hkv, page), dtype=np.uint8) for _ in range(2)]
        self.table_np = rng.permutation(pages)[:B * max_pages].reshape(B, max_pages).astype(np.int32)
        self.upload()

    def upload(self):
        t = [torch.from_numpy(a.copy()).to(DEV) for a in self.np]
        self.k, self.v = t[0].view(torch.float8_e4m3fn), t[1].view(torch.float8_e4m3fn)
        self.ks, self.vs = t[2], t[3]
        self.table = torch.from_numpy(self.table_np).to(DEV)

    @property
    def args(self):
        return self.k, self.v, self.ks, self.vs, self.table

    def host(self):
        return [t.view(torch.uint8).cpu().numpy() for t in (self.k, self.v, self.ks, self.vs)]

    def fill(self, rng, lens, spread=3):
        """Ordinary rows for the first lens[b] keys of every sequence, in numpy and on the GPU."""
        k, v, ks, vs = self.np
        page = k.shape[2]
        for b, n in enumerate(lens):
            for j in range(n):
                p = self.table_np[b, j // page]
                if not 0 <= p < k.shape[0]:
                    continue
                for codes, scales in ((k, ks), (v, vs)):
                    x = rng.standard_normal(codes.shape[1::2]) * 2.0 ** rng.uniform(-spread, spread, (codes.shape[1], 1))
                    codes[p, :, j % page], scales[p, :, j % page] = kv8.quantise(x)
        self.upload()


def _int(x):
    return torch.tensor([int(i) for i in x], dtype=torch.int32, device=DEV)


def _cu(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(int)


def _same(got, want):
    for g, w in zip(got, want):
        assert np.array_equal(g, w), f"{np.count_nonzero(g != w)} of {w.size} bytes differ"


def _rows(rng, n, Hkv, D, dtype):
    x = rng.standard_normal((n, Hkv, D)) * 2.0 ** rng.uniform(-6, 6, (n, Hkv, 1))
    return torch.from_numpy(x).to(DT[dtype])


# ------------------------------------------------------------------------ append ----
@pytest.mark.parametrize("D,Hkv,page,counts,pasts,dtype", [
    (64, 2, 16, [1], [0], "bf16"),
    (64, 1, 16, [16, 17], [15, 0], "fp16"),
    (96, 3, 48, [0, 33, 1, 0], [5, 40, 47, 0], "bf16"),
    (128, 8, 32, [7, 70], [60, 0], "bf16"),
    (128, 1, 64, [1, 0, 1, 1, 5], [63, 64, 65, 0, 127], "fp16"),
    (256, 4, 16, [31, 2], [1, 16], "bf16"),
    (96, 16, 16, [3, 3], [0, 29], "fp16"),
])
def test_append_packed(fa, D, Hkv, page, counts, pasts, dtype):
    rng = np.random.default_rng(D + Hkv)
    B, cu = len(counts), _cu(counts)
    lens = [c + p for c, p in zip(counts, pasts)]
    mp = -(-max(lens) // page) + 1
    pool = Pool(B * mp + 2, Hkv, page, D, B, mp, seed=7)
    extra = 3                                   # rows behind the last sequence: not written
    k, v = _rows(rng, cu[-1] + extra, Hkv, D, dtype), _rows(rng, cu[-1] + extra, Hkv, D, dtype)
    want = [a.copy() for a in pool.np]
    kv8.append(want, k.double().numpy(), v.double().numpy(), pool.table_np, lens, cu)
    fa.fa_kv_append_paged_fp8(k.to(DEV), v.to(DEV), *pool.args, _int(lens), cu_seqlens_new=_int(cu))
    _same(pool.host(), want)


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("n", [1, 3])
def test_append_equal_counts_from_a_fused_projection(fa, D, n):
    """[B, n, Hkv, D] slices of one [B, n, (Hq + 2 Hkv) D] buffer: strided tokens."""
    rng = np.random.default_rng(n)
    B, Hq, Hkv, page = 5, 4, 2, 16
    lens = [n, n + 1, 15 + n, 16 + n, 40 + n]
    pool = Pool(24, Hkv, page, D, B, 4, seed=8)
    qkv = torch.from_numpy(rng.standard_normal((B, n, Hq + 2 * Hkv, D))).to(torch.bfloat16)
    want = [a.copy() for a in pool.np]
    flat = qkv.view(B * n, Hq + 2 * Hkv, D).double().numpy()
    kv8.append(want, flat[:, Hq:Hq + Hkv], flat[:, Hq + Hkv:], pool.table_np, lens, _cu([n] * B))
    dev = qkv.to(DEV)
    fa.fa_kv_append_paged_fp8(dev[:, :, Hq:Hq + Hkv], dev[:, :, Hq + Hkv:], *pool.args, _int(lens))
    _same(pool.host(), want)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append_edge_values(fa, dtype):
    """Rows at the border of a scale (448 2^e and its neighbours), zeros, subnormals, the
    type's largest values, infinities and NaN among and instead of finite ones."""
    D, dt = 64, DT[dtype]
    big = torch.finfo(dt).max
    tops = [448.0, 7.0, 0.875 * 2.0 ** -10, 448 * 2.0 ** 4, 1.0, 1.75, 0.0, float(torch.finfo(dt).tiny), big]
    rows = []
    for top in tops:
        t = torch.tensor(top).to(dt)
        for a in (t, torch.nextafter(t, torch.tensor(0.0, dtype=dt)), torch.nextafter(t, torch.tensor(big, dtype=dt))):
            row = torch.linspace(-1, 1, D).to(dt) * a * 0.99
            row[7] = -a
            rows.append(row)
    sub = torch.tensor(float(torch.finfo(dt).smallest_normal)).to(dt) * torch.linspace(0, 1, D).to(dt)
    rows += [sub, torch.zeros(D, dtype=dt), -torch.zeros(D, dtype=dt)]
    for bad in (math.inf, -math.inf, math.nan):
        mixed = torch.linspace(-3, 3, D).to(dt)
        mixed[11] = bad
        rows += [mixed, torch.full((D,), bad, dtype=dt)]
    x = torch.stack(rows)[:, None]
    n = len(rows)
    mp = -(-n // 16)
    pool = Pool(mp + 1, 1, 16, D, 1, mp, seed=9)
    want = [a.copy() for a in pool.np]
    kv8.append(want, x.double().numpy(), -x.double().numpy(), pool.table_np, [n], [0, n])
    fa.fa_kv_append_paged_fp8(x.to(DEV), -x.to(DEV), *pool.args, _int([n]), cu_seqlens_new=_int([0, n]))
    _same(pool.host(), want)


def test_append_drops_rows_without_a_place(fa):
    """Keys before 0, behind the table's capacity, on pages outside the pool: nothing of the
    pool changes but the rows that have a place."""
    rng = np.random.default_rng(2)
    Hkv, page, D = 2, 16, 128
    pool = Pool(9, Hkv, page, D, 5, 1, seed=10)
    pool.table_np[2, 0], pool.table_np[3, 0] = -5, 9
    pool.upload()
    counts, lens = [4, 6, 5, 3, 2], [2, 20, 5, 3, -7]
    cu = _cu(counts)
    k, v = _rows(rng, cu[-1], Hkv, D, "bf16"), _rows(rng, cu[-1], Hkv, D, "bf16")
    want = [a.copy() for a in pool.np]
    kv8.append(want, k.double().numpy(), v.double().numpy(), pool.table_np, lens, cu)
    assert not np.array_equal(want[0], pool.np[0])
    fa.fa_kv_append_paged_fp8(k.to(DEV), v.to(DEV), *pool.args, _int(lens), cu_seqlens_new=_int(cu))
    _same(pool.host(), want)


def test_append_of_nothing(fa):
    pool = Pool(3, 2, 16, 64, 2, 1)
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    fa.fa_kv_append_paged_fp8(none, none, *pool.args, _int([5, 5]), cu_seqlens_new=_int([0, 0, 0]))
    none = torch.empty(2, 0, 2, 64, dtype=torch.bfloat16, device=DEV)
    fa.fa_kv_append_paged_fp8(none, none, *pool.args, _int([5, 5]))
    _same(pool.host(), pool.np)


def test_append_many_sequences(fa):
    """1024 sequences (the most), most of them with no new token."""
    rng = np.random.default_rng(4)
    B, Hkv, page, D = 1024, 1, 16, 64
    counts = rng.integers(0, 3, B) * (rng.random(B) < 0.3)
    lens = counts + rng.integers(0, 30, B)
    cu = _cu(counts)
    pool = Pool(2 * B, Hkv, page, D, B, 2, seed=11)
    k, v = _rows(rng, cu[-1], Hkv, D, "bf16"), _rows(rng, cu[-1], Hkv, D, "bf16")
    want = [a.copy() for a in pool.np]
    kv8.append(want, k.double().numpy(), v.double().numpy(), pool.table_np, lens, cu)
    fa.fa_kv_append_paged_fp8(k.to(DEV), v.to(DEV), *pool.args, _int(lens), cu_seqlens_new=_int(cu))
    _same(pool.host(), want)


# -------------------------------------------------------------------------- read ----
@pytest.mark.parametrize("D,Hkv,page,counts,starts,dtype", [
    (64, 2, 16, [1], None, "bf16"),
    (64, 1, 16, [0, 33, 16, 0], [3, 5, 16, 0], "fp16"),
    (96, 3, 48, [50, 1], [47, 0], "bf16"),
    (128, 8, 32, [7, 70], None, "bf16"),
    (256, 4, 16, [31, 2], [1, 16], "fp16"),
])
def test_read(fa, D, Hkv, page, counts, starts, dtype):
    rng = np.random.default_rng(D)
    B, cu = len(counts), _cu(counts)
    first = starts or [0] * B
    ends = [c + s for c, s in zip(counts, first)]
    mp = -(-max(ends) // page) + 1
    pool = Pool(B * mp + 1, Hkv, page, D, B, mp, seed=12)
    pool.fill(rng, ends, spread=20)             # past fp16's range at both ends
    extra = 2
    dt = DT[dtype]
    k, v = (torch.full((cu[-1] + extra, Hkv, D), 7.0, dtype=dt, device=DEV) for _ in range(2))
    out = fa.fa_kv_read_paged_fp8(*pool.args, _int(cu), kv_starts=None if starts is None else _int(starts), k_out=k,
                                  v_out=v)
    assert out[0] is k and out[1] is v
    for got, codes, scales in ((k, pool.np[0], pool.np[2]), (v, pool.np[1], pool.np[3])):
        want = np.concatenate([kv8.cached(codes, scales, pool.table_np, b, first[b], counts[b]) for b in range(B)])
        want = torch.from_numpy(want).float().to(dt)       # 4 significant bits: exact in fp32, rounded once
        assert torch.equal(got[:cu[-1]].cpu().view(torch.int16), want.view(torch.int16))
        assert (got[cu[-1]:] == 7).all()


def test_read_every_code_and_scale(fa):
    """All 256 codes at all 256 scale bytes, NaN codes, infinite results and byte 255 included."""
    pool = Pool(32, 1, 16, 256, 1, 32)
    pool.np[0][:] = pool.np[1][:] = np.arange(256, dtype=np.uint8)
    pool.table_np[0] = np.arange(32)
    pool.np[2][:, 0] = np.minimum(np.arange(512), 255).reshape(32, 16)
    pool.np[3][:] = pool.np[2]
    pool.upload()
    for dt in (torch.bfloat16, torch.float16):
        k, v = fa.fa_kv_read_paged_fp8(*pool.args, _int([0, 255]), total=255, dtype=dt)
        want = torch.from_numpy(kv8.values(pool.np[0], pool.np[2]).reshape(512, 1, 256)[:255]).float().to(dt)
        for got in (k, v):
            assert torch.equal(got.cpu().isnan(), want.isnan())
            assert torch.equal(got.cpu().nan_to_num(0).view(torch.int16), want.nan_to_num(0).view(torch.int16))


def test_read_zeros_where_there_is_no_page(fa):
    rng = np.random.default_rng(6)
    pool = Pool(7, 2, 16, 64, 3, 2, seed=13)
    pool.table_np[0, 1], pool.table_np[1, 0] = 7, -2147483648
    pool.fill(rng, [32, 32, 32])
    counts, starts = [32, 20, 30], [0, 4, 20]   # the last runs past the table's capacity
    cu = _cu(counts)
    k, v = fa.fa_kv_read_paged_fp8(*pool.args, _int(cu), kv_starts=_int(starts), total=int(cu[-1]))
    want = np.concatenate([kv8.cached(pool.np[0], pool.np[2], pool.table_np, b, starts[b], counts[b]) for b in range(3)])
    assert np.array_equal(k.double().cpu().numpy(), want)
    assert (want[16:32] == 0).all() and (want[32:44] == 0).all() and (want[-18:] == 0).all()
    k, _ = fa.fa_kv_read_paged_fp8(*pool.args, _int(cu), kv_starts=_int([-40, -2147483648, 2147483647]), total=int(cu[-1]))
    assert (k == 0).all()


# ------------------------------------------------------------------------ decode ----
def _check(o, lse, ref, n, D, dtype):
    o_ref, lse_ref, o_abs, s_abs, o_top = ref
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    e_s = (D + 8) * 2.0 ** -22 * s_abs                                     # [B, Hq, Sq]
    sums = 2.0 ** -21 + (n / 4 + 64) * 2.0 ** -23
    c = np.transpose(2.0 ** -11 + 2 * e_s + sums, (0, 2, 1))[..., None]
    step = float(torch.finfo(DT[dtype]).smallest_normal) * float(torch.finfo(DT[dtype]).eps)
    bound = U_O[dtype] * np.abs(o_ref) + c * o_abs + 2.0 ** -36 * o_top + step / 2
    assert np.isfinite(o).all()
    off = np.abs(o - o_ref)
    assert (off <= bound).all(), f"|dO| {off.max():.3e}, {np.max(off / bound):.2f} of its bound"
    fin = np.isfinite(lse_ref)
    assert np.array_equal(fin, np.isfinite(lse)) and (lse[~fin] == -np.inf).all()
    e_s, lse, lse_ref = e_s[fin], lse[fin], lse_ref[fin]
    assert (np.abs(lse - lse_ref) <= e_s + sums + 2.0 ** -22 * np.abs(lse_ref)).all()


def _decode_case(fa, D, Hq, Hkv, Sq, page, lens, dtype="bf16", causal=True, ns=0, seed=0, qscale=1.0, spread=3, table=None,
                 fill=None):
    rng = np.random.default_rng(seed + D + Hq)
    B = len(lens)
    mp = max(1, -(-max(lens) // page)) + 1
    pool = Pool(B * mp + 3, Hkv, page, D, B, mp, seed=seed)
    if table:
        table(pool.table_np)
    pool.fill(rng, lens, spread)
    if fill:
        fill(pool)
    q = torch.from_numpy(rng.standard_normal((B, Sq, Hq, D)) * qscale).to(DT[dtype])
    o, lse = fa.fa_decode_splitkv_paged_fp8(q.to(DEV), *pool.args, _int(lens), causal=causal, num_splits=ns)
    ref = kv8.decode(q.double().numpy(), pool.np, pool.table_np, lens, 1 / math.sqrt(D), causal)
    _check(o, lse, ref, max(lens), D, dtype)
    return pool, q, o, lse


HEAD_DIMS = [64, 96, 128, 256]


@pytest.mark.parametrize("D", HEAD_DIMS)
@pytest.mark.parametrize("ns", [0, 1, 3])
def test_decode_lengths(fa, D, ns):
    """Lengths around the pages, the 16-key runs and the 128-key tiles; empty and single keys;
    everything behind them is random bytes."""
    _decode_case(fa, D, 4, 2, 1, 16, [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 257, 300], ns=ns)


@pytest.mark.parametrize("D", HEAD_DIMS)
@pytest.mark.parametrize("group,Sq,Hkv", [(1, 1, 3), (8, 1, 2), (9, 1, 1), (16, 1, 2), (1, 16, 2), (4, 4, 2), (3, 5, 1),
                                          (2, 7, 5)])
def test_decode_columns(fa, D, group, Sq, Hkv):
    """1..16 query rows a kv head, of heads and of tokens; causal rows that see no key."""
    _decode_case(fa, D, group * Hkv, Hkv, Sq, 32, [200, 3, 77, 0, 1], seed=group)


@pytest.mark.parametrize("D", HEAD_DIMS)
def test_decode_without_the_mask(fa, D):
    _decode_case(fa, D, 4, 2, 4, 48, [2, 130, 0, 49], causal=False)


@pytest.mark.parametrize("D", HEAD_DIMS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("page", [16, 80, 512])
def test_decode_split_long(fa, D, dtype, page):
    """Pairs cut into many pieces beside short ones."""
    _decode_case(fa, D, 6, 2, 1, page, [2111, 40, 700], dtype=dtype, ns=64)


def test_decode_one_sequence_many_pieces(fa):
    _decode_case(fa, 128, 8, 1, 2, 16, [6001], ns=400)


@pytest.mark.parametrize("D", HEAD_DIMS)
def test_decode_wide_scales(fa, D):
    """Rows whose magnitudes are 2^-20 .. 2^20: a probability's weight is that of its value too."""
    _decode_case(fa, D, 4, 2, 1, 16, [150, 400], spread=20, qscale=2.0 ** -18)


def test_decode_large_scores(fa):
    """Scores in the hundreds: one key takes all; queries past fp16's range."""
    _decode_case(fa, 64, 4, 2, 1, 16, [333, 64], qscale=40.0)
    _decode_case(fa, 64, 4, 2, 1, 16, [333, 64], qscale=2.0 ** 20, spread=0)
    _decode_case(fa, 64, 4, 2, 1, 16, [333, 64], qscale=2.0 ** -100, spread=0)


def test_decode_rising_scores(fa):
    """Every key scores higher than the one before: the running maximum moves all the time."""
    def fill(pool):
        k = pool.np[0]
        page = k.shape[2]
        for j in range(500):
            p = pool.table_np[0, j // page]
            k[p, :, j % page], pool.np[2][p, :, j % page] = kv8.quantise(np.full((k.shape[1], k.shape[3]), 0.02 * (j + 1)))
        pool.upload()
    for q in (2.0, -2.0):
        _decode_case(fa, 128, 2, 1, 1, 16, [500], fill=fill, qscale=q)


def test_decode_pages_outside_the_pool_are_zero_rows(fa):
    def table(t):
        t[0, 1], t[0, 3], t[1, 0], t[2, :] = -1, 2147483647, 10 ** 6, -2147483648
    _decode_case(fa, 128, 4, 2, 1, 16, [100, 40, 30], table=table)


def test_decode_shared_pages(fa):
    """Two sequences with a common prefix on the same pages; a page twice in one sequence."""
    def table(t):
        t[1, :4] = t[0, :4]
        t[2, 1] = t[2, 0]
    _decode_case(fa, 64, 4, 2, 1, 16, [90, 77, 32], table=table)


@pytest.mark.parametrize("D", HEAD_DIMS)
def test_decode_nan_key_reaches_its_rows_only(fa, D):
    """A NaN code of a visible key makes that kv head's rows NaN and no others."""
    pool, q, o, lse = _decode_case(fa, D, 4, 2, 1, 16, [200, 150], seed=3)
    p = pool.table_np[0, 3]
    pool.np[0][p, 1, 5, 17] = 0x7F
    pool.upload()
    o2, lse2 = fa.fa_decode_splitkv_paged_fp8(q.to(DEV), *pool.args, _int([200, 150]))
    assert o2[0, 0, 2:].isnan().all() and lse2[0, 2:].isnan().all()
    assert torch.equal(o2[0, 0, :2], o[0, 0, :2]) and torch.equal(o2[1], o[1])
    pool.np[0][p, 1, 5, 17] = 0
    pool.np[1][p, 1, 5, 17] = 0xFF                # a NaN value: that dimension alone
    pool.upload()
    o3, lse3 = fa.fa_decode_splitkv_paged_fp8(q.to(DEV), *pool.args, _int([200, 150]))
    assert o3[0, 0, 2:, 17].isnan().all() and o3[0].isnan().sum() == 2 and lse3.isfinite().all()


@pytest.mark.parametrize("D", HEAD_DIMS)
@pytest.mark.parametrize("group,Sq,length,seqs", [(1, 2, 200, 1), (2, 4, 64, 1), (4, 4, 33, 1), (1, 16, 2050, 2),
                                                  (1, 16, 7, 1), (2, 3, 70, 240)])
def test_decode_nan_of_a_hidden_key(fa, D, group, Sq, length, seqs):
    """NaN codes among the last Sq keys, in K or in V, change nothing for the tokens that the mask
    hides them from (with one in K the seen rows' scores no longer move the references: other
    roundings within the bound).  240 sequences: warps take pairs alone."""
    Hkv, lens = 2, [length] * seqs
    pool, q, o, lse = _decode_case(fa, D, group * Hkv, Hkv, Sq, 16, lens, seed=9)
    ref = kv8.decode(q.double().numpy()[:1], pool.np, pool.table_np[:1], lens[:1], 1 / math.sqrt(D), True)
    for back in range(1, min(Sq, length)):        # the key `back` before the last: tokens from Sq - 1 - back on see it
        key, first = length - 1 - back, Sq - 1 - back
        page, slot = pool.table_np[0, key // 16], key % 16
        dim = (back * 37) % D
        for which in (0, 1):
            was = pool.np[which][page, 1, slot, dim]
            pool.np[which][page, 1, slot, dim] = 0x7F + 0x80 * (back % 2)
            pool.upload()
            o2, lse2 = fa.fa_decode_splitkv_paged_fp8(q.to(DEV), *pool.args, _int(lens))
            pool.np[which][page, 1, slot, dim] = was
            assert torch.equal(o2[1:], o[1:]) and torch.equal(o2[0, :, :group], o[0, :, :group])
            seen = o2[0, first:, group:]
            if which == 0:
                assert seen.isnan().all() and lse2[0, group:, first:].isnan().all()
                o2[0, first:, group:], lse2[0, group:, first:] = o[0, first:, group:], lse[0, group:, first:]
                _check(o2[:1], lse2[:1], ref, length, D, "bf16")
            else:
                assert seen[..., dim].isnan().all() and seen.isnan().sum() == seen[..., dim].numel()
                assert torch.equal(o2[0, :first], o[0, :first]) and torch.equal(lse2, lse)


def test_decode_clamps_lengths_and_takes_all_empty(fa):
    pool, q, o, lse = _decode_case(fa, 128, 4, 2, 1, 16, [64, 64], seed=4)
    # max_pages is one more than needed: fill it too, then ask for more keys than there are
    pool.fill(np.random.default_rng(1), [80, 80])
    o1, l1 = fa.fa_decode_splitkv_paged_fp8(q.to(DEV), *pool.args, _int([80, 80]))
    o2, l2 = fa.fa_decode_splitkv_paged_fp8(q.to(DEV), *pool.args, _int([2 ** 31 - 1, 81]))
    assert torch.equal(o1, o2) and torch.equal(l1, l2)
    o3, l3 = fa.fa_decode_splitkv_paged_fp8(q.to(DEV), *pool.args, _int([-5, 0]))
    assert (o3 == 0).all() and (l3 == -math.inf).all()


def test_decode_many_sequences(fa):
    """1024 sequences, many of them empty."""
    rng = np.random.default_rng(8)
    lens = (rng.integers(0, 40, 1024) * (rng.random(1024) < 0.5)).tolist()
    _decode_case(fa, 64, 2, 1, 1, 16, lens)


@pytest.mark.parametrize("D", HEAD_DIMS)
@pytest.mark.parametrize("group,Sq,longest,ns", [(1, 1, 320, 0), (4, 1, 321, 0), (3, 2, 128, 0), (5, 3, 129, 0),
                                                 (2, 1, 90, 1), (15, 1, 320, 0)])
def test_decode_many_short_pairs(fa, D, group, Sq, longest, ns):
    """960 pairs, all short: the kernel may give each warp pairs of its own. Empty sequences among
    them, lengths at and one past the longest that form takes."""
    rng = np.random.default_rng(D)
    lens = (rng.integers(0, 60, 80) * (rng.random(80) < 0.8)).tolist()
    lens[7], lens[-1] = longest, 33
    _decode_case(fa, D, group * 12, 12, Sq, 16, lens, ns=ns, seed=group)


@pytest.mark.parametrize("D", HEAD_DIMS)
@pytest.mark.parametrize("group,Sq,longest", [(1, 1, 512), (2, 4, 512), (4, 1, 513), (5, 3, 500)])
def test_decode_a_pair_for_each_warp(fa, D, group, Sq, longest):
    """1920 pairs, four for each CTA: lengths at and one past the longest that warps take alone."""
    rng = np.random.default_rng(D)
    lens = (rng.integers(0, 30, 160) * (rng.random(160) < 0.8)).tolist()
    lens[3], lens[90], lens[-1] = longest, 257, 33
    _decode_case(fa, D, group * 12, 12, Sq, 16, lens, seed=group)


def test_decode_without_a_workspace_cuts_as_with_one(fa):
    """More than eight pairs an SM, where the default is one partial result a pair, and a long
    sequence among short ones: the call that makes its workspace has the bits of one that is given
    it, so the long pairs are cut in both, and other bits than one that may not cut."""
    rng = np.random.default_rng(31)
    B, Hkv, D, page, mp = 160, 8, 64, 64, 96
    lens = rng.integers(1, 40, B)
    lens[77] = 6000
    pool = Pool(B * 1 + mp, Hkv, page, D, 1, 1, seed=31)
    pool.table_np = np.full((B, mp), -1, np.int32)
    pages = rng.permutation(B + mp)
    pool.table_np[:, 0] = pages[:B]
    pool.table_np[77] = pages[B:]
    pool.fill(rng, lens)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert B * Hkv >= 8 * sms and fa.fa_decode_default_splits(B, Hkv, mp * page) == 1
    q = torch.from_numpy(rng.standard_normal((B, 1, Hkv, D))).to(torch.bfloat16).to(DEV)
    ws = torch.empty(fa.fa_decode_workspace_bytes(B, Hkv, D, 1), dtype=torch.uint8, device=DEV)
    given = fa.fa_decode_splitkv_paged_fp8(q, *pool.args, _int(lens), workspace=ws)
    made = fa.fa_decode_splitkv_paged_fp8(q, *pool.args, _int(lens))
    uncut = fa.fa_decode_splitkv_paged_fp8(q, *pool.args, _int(lens), num_splits=1)
    assert torch.equal(made[0], given[0]) and torch.equal(made[1], given[1])
    assert not torch.equal(uncut[1][77], given[1][77])
    ref = kv8.decode(q.double().cpu().numpy(), pool.np, pool.table_np, lens, 1 / math.sqrt(D))
    for o, lse in (made, uncut):
        _check(o, lse, ref, 6000, D, "bf16")


def test_decode_contiguous_cache_is_one_page_each(fa):
    """page_size = the whole capacity and an identity table: the same bits as small pages."""
    pool, q, o, lse = _decode_case(fa, 96, 4, 2, 2, 16, [300, 222], ns=5)
    B, mp = pool.table_np.shape
    big = [np.ascontiguousarray(np.moveaxis(a[pool.table_np], 2, 1).reshape(B, a.shape[1], mp * 16, *a.shape[3:]))
           for a in pool.np]
    t = [torch.from_numpy(a).to(DEV) for a in big]
    table = _int(range(B)).view(B, 1)
    o2, lse2 = fa.fa_decode_splitkv_paged_fp8(q.to(DEV), t[0].view(torch.float8_e4m3fn), t[1].view(torch.float8_e4m3fn),
                                              t[2], t[3], table, _int([300, 222]), num_splits=5)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_decode_with_a_wide_table(fa):
    """A table for 2^30 + 2^20 keys a sequence, over 2^31 in the batch: the bits of one for 2^20."""
    B, Hq, Hkv, D, page = 2, 4, 1, 64, 1 << 20
    g = torch.Generator(DEV).manual_seed(17)
    pages = [torch.zeros(B, Hkv, page, D, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.zeros(B, Hkv, page, dtype=torch.uint8, device=DEV) for _ in range(2)]
    x = torch.randn(2, 700, Hkv, D, generator=g, device=DEV).to(torch.bfloat16)
    q = torch.randn(B, 1, Hq, D, generator=g, device=DEV).to(torch.bfloat16)
    kl, cu = _int([400, 300]), _int([0, 400, 700])
    outs = []
    for mp in (1, 1025):
        table = torch.full((B, mp), -1, dtype=torch.int32, device=DEV)
        table[:, 0] = torch.tensor([1, 0], dtype=torch.int32)
        pool = (*pages, *scales, table)
        fa.fa_kv_append_paged_fp8(x[0], x[1], *pool, kl, cu_seqlens_new=cu)
        outs.append((*fa.fa_decode_splitkv_paged_fp8(q, *pool, kl, num_splits=5),
                     *fa.fa_kv_read_paged_fp8(*pool, cu, total=700)))
    for a, b in zip(*outs):
        assert a.isfinite().all() and torch.equal(a, b)


def test_decode_guard_bands_and_no_lse(fa):
    """Writes stay inside O, LSE and the workspace; LSE may be absent at the C entry."""
    B, Hq, Hkv, D, Sq, ns, pad = 3, 8, 2, 96, 2, 7, 4096
    lens = [900, 0, 129]
    pool, q, o_ref, lse_ref = _decode_case(fa, D, Hq, Hkv, Sq, 16, lens, ns=ns)
    need = fa.fa_decode_workspace_bytes(B * Sq, Hq, D, ns)
    ob = torch.full((2 * pad + q.numel(),), 7.0, dtype=torch.bfloat16, device=DEV)
    lb = torch.full((2 * pad + B * Hq * Sq,), 7.0, device=DEV)
    wb = torch.full((2 * pad + need,), 0xA5, dtype=torch.uint8, device=DEV)
    o, lse = ob[pad:-pad].view(B, Sq, Hq, D), lb[pad:-pad].view(B, Hq, Sq)
    fa.fa_decode_splitkv_paged_fp8(q.to(DEV), *pool.args, _int(lens), num_splits=ns, workspace=wb[pad:-pad], out=o, lse=lse)
    assert torch.equal(o, o_ref) and torch.equal(lse, lse_ref)
    for buf, fill in ((ob, 7.0), (lb, 7.0), (wb, 0xA5)):
        assert (buf[:pad] == fill).all() and (buf[-pad:] == fill).all()
    from exact_tiled_attention_20_gb300 import _lib

    o.zero_()
    qd, kl = q.to(DEV), _int(lens)
    num_pages, _, page, _ = pool.k.shape
    st = _lib._load_fp8().fa_decode_splitkv_paged_fp8(
        qd.data_ptr(), pool.k.data_ptr(), pool.v.data_ptr(), pool.ks.data_ptr(), pool.vs.data_ptr(), pool.table.data_ptr(),
        kl.data_ptr(), o.data_ptr(), None, B, Sq, Hq, Hkv, D, num_pages, page, pool.table.shape[1], 1 / math.sqrt(D), 1,
        ns, wb[pad:].data_ptr(), need, 0, torch.cuda.current_stream().cuda_stream)
    assert st == 0 and torch.equal(o, o_ref)


def test_decode_uncut_needs_no_workspace(fa):
    """num_splits = 1 at the C entry without a workspace: the binding's bits, in every form that a CTA or
    a warp alone takes pairs in."""
    from exact_tiled_attention_20_gb300 import _lib

    for D, Hkv, lens in ((128, 2, [700, 0, 129]), (64, 12, [20, 0, 300, 64] * 40), (256, 3, [90])):
        pool, q, o, lse = _decode_case(fa, D, 4 * Hkv, Hkv, 1, 16, lens, ns=1)
        got = torch.full_like(o, 7.0), torch.full_like(lse, 7.0)
        qd, kl = q.to(DEV), _int(lens)
        num_pages, _, page, _ = pool.k.shape
        st = _lib._load_fp8().fa_decode_splitkv_paged_fp8(
            qd.data_ptr(), pool.k.data_ptr(), pool.v.data_ptr(), pool.ks.data_ptr(), pool.vs.data_ptr(),
            pool.table.data_ptr(), kl.data_ptr(), got[0].data_ptr(), got[1].data_ptr(), len(lens), 1, 4 * Hkv, Hkv, D,
            num_pages, page, pool.table.shape[1], 1 / math.sqrt(D), 1, 1, None, 0, 0, torch.cuda.current_stream().cuda_stream)
        assert st == 0 and torch.equal(got[0], o) and torch.equal(got[1], lse)


@pytest.mark.parametrize("D", HEAD_DIMS)
def test_decode_is_deterministic_and_independent_of_the_split(fa, D):
    pool, q, o, lse = _decode_case(fa, D, 8, 2, 1, 16, [1500, 200, 801], ns=1, seed=5)
    for ns in (2, 5, 64):
        a = fa.fa_decode_splitkv_paged_fp8(q.to(DEV), *pool.args, _int([1500, 200, 801]), num_splits=ns)
        b = fa.fa_decode_splitkv_paged_fp8(q.to(DEV), *pool.args, _int([1500, 200, 801]), num_splits=ns)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        # 2 u_o: both sides are rounded; 2^-10: P's roundings on both sides
        assert ((a[0] - o).float().abs() <= 2.0 ** -7 * o.float().abs() + 2.0 ** -6 * 1.0).all()
        assert ((a[1] - lse).abs() <= 1e-4).all()


@pytest.mark.parametrize("D", HEAD_DIMS)
@pytest.mark.parametrize("ns", [1, 2, 5, 64])
def test_decode_holds_its_bound_for_every_split(fa, D, ns):
    _decode_case(fa, D, 8, 2, 1, 16, [1500, 200, 801], ns=ns, seed=5)


# -------------------------------------------------------------- used as a program ----
def test_prompt_then_steps(fa):
    """A chunked prefill and decode steps as a serving loop runs them: each chunk is appended,
    the prefix is read back for fa_fwd_varlen, then single tokens are appended and decoded.
    The decode's last step agrees with fa_fwd_varlen over the rows read back."""
    rng = np.random.default_rng(9)
    B, Hq, Hkv, D, page, mp = 3, 8, 2, 128, 32, 8
    pool = Pool(B * mp, Hkv, page, D, B, mp, seed=14)
    ref = [a.copy() for a in pool.np]
    lens = np.zeros(B, int)
    for counts in ([50, 0, 129], [33, 7, 64], [1, 1, 1], [1, 1, 1]):
        cu = _cu(counts)
        lens = lens + counts
        k, v = _rows(rng, cu[-1], Hkv, D, "bf16") / 8, _rows(rng, cu[-1], Hkv, D, "bf16")
        kv8.append(ref, k.double().numpy(), v.double().numpy(), pool.table_np, lens, cu)
        step = counts[0] == 1
        if step:
            fa.fa_kv_append_paged_fp8(k.view(B, 1, Hkv, D).to(DEV), v.view(B, 1, Hkv, D).to(DEV), *pool.args, _int(lens))
        else:
            fa.fa_kv_append_paged_fp8(k.to(DEV), v.to(DEV), *pool.args, _int(lens), cu_seqlens_new=_int(cu))
        q = torch.from_numpy(rng.standard_normal((cu[-1], Hq, D))).to(torch.bfloat16).to(DEV)
        cu_k = _cu(lens)
        kr, vr = fa.fa_kv_read_paged_fp8(*pool.args, _int(cu_k), total=int(cu_k[-1]))
        o, lse = fa.fa_fwd_varlen(q, kr, vr, _int(cu), _int(cu_k), causal=True)
        if step:
            od, ld = fa.fa_decode_splitkv_paged_fp8(q.view(B, 1, Hq, D), *pool.args, _int(lens))
            want = kv8.decode(q.view(B, 1, Hq, D).double().cpu().numpy(), ref, pool.table_np, lens, 1 / math.sqrt(D))
            _check(od, ld, want, int(max(lens)), D, "bf16")
            # fa_fwd_varlen rounds P to bf16 as well: 2^-8 of A beside both outputs' roundings
            bound = 2.0 ** -7 * np.abs(want[0]) + 2.0 ** -7 * want[2]
            assert (np.abs(od.double().cpu().numpy()[:, 0] - o.double().cpu().numpy()) <= bound[:, 0]).all()
            assert ((ld[:, :, 0].T - lse).abs() <= 1e-3).all()
    _same(pool.host(), ref)


def test_step_of_a_padded_batch(fa):
    """Entries of a batch that hold no sequence (length 0, a table of -1): their rows are dropped by the
    append, their outputs are zeros, and the other sequences are as in a batch without them."""
    rng = np.random.default_rng(12)
    Hq, Hkv, D, page, mp = 8, 2, 96, 16, 6
    pool = Pool(4 * mp, Hkv, page, D, 4, mp, seed=17)
    pool.table_np[1], pool.table_np[3] = -1, -1
    lens = [60, 0, 33, 0]
    pool.fill(rng, lens)
    lens = [61, 0, 34, 0]
    k, v, q = (torch.from_numpy(rng.standard_normal((4, 1, h, D))).to(torch.bfloat16) for h in (Hkv, Hkv, Hq))
    real = [0, 2]
    want = [a.copy() for a in pool.np]
    kv8.append(want, k[real, 0].double().numpy(), v[real, 0].double().numpy(), pool.table_np[real], [61, 34], _cu([1, 1]))
    fa.fa_kv_append_paged_fp8(k.to(DEV), v.to(DEV), *pool.args, _int(lens))
    _same(pool.host(), want)
    o, lse = fa.fa_decode_splitkv_paged_fp8(q.to(DEV), *pool.args, _int(lens))
    assert (o[[1, 3]] == 0).all() and (lse[[1, 3]] == -math.inf).all()
    _check(o, lse, kv8.decode(q.double().numpy(), want, pool.table_np, lens, 1 / math.sqrt(D)), 61, D, "bf16")


def test_captured_step_replays_with_new_lengths(fa):
    """Append and decode captured into one graph; replays follow kv_lens and the new rows."""
    rng = np.random.default_rng(10)
    B, Hq, Hkv, D, page, mp = 4, 8, 2, 64, 16, 6
    pool = Pool(B * mp, Hkv, page, D, B, mp, seed=15)
    lens0 = [20, 0, 47, 80]
    pool.fill(rng, lens0)
    ref = [a.copy() for a in pool.np]
    k, v, q = (torch.zeros(B, 1, h, D, dtype=torch.bfloat16, device=DEV) for h in (Hkv, Hkv, Hq))
    kl = _int(lens0)
    ws = torch.empty(fa.fa_decode_workspace_bytes(B, Hq, D, 8), dtype=torch.uint8, device=DEV)
    o, lse = torch.empty_like(q), torch.empty(B, Hq, 1, device=DEV)

    def step():
        kl.add_(1)
        fa.fa_kv_append_paged_fp8(k, v, *pool.args, kl)
        fa.fa_decode_splitkv_paged_fp8(q, *pool.args, kl, num_splits=8, workspace=ws, out=o, lse=lse)

    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step()
    lens = np.array(lens0)
    for _ in range(5):
        for t, h in ((k, Hkv), (v, Hkv), (q, Hq)):
            t.copy_(torch.from_numpy(rng.standard_normal((B, 1, h, D))).to(torch.bfloat16))
        graph.replay()
        lens = lens + 1
        kv8.append(ref, k.view(B, Hkv, D).double().cpu().numpy(), v.view(B, Hkv, D).double().cpu().numpy(),
                   pool.table_np, lens, _cu([1] * B))
        _check(o, lse, kv8.decode(q.double().cpu().numpy(), ref, pool.table_np, lens, 1 / math.sqrt(D)), int(max(lens)), D,
               "bf16")
    _same(pool.host(), ref)


def test_captured_split_decode_follows_the_lengths(fa):
    """Sequences cut into many pieces, the lengths moved on inside the graph: each replay gives the
    bits of an eager call with its lengths (the merge plans from the new ones too)."""
    rng = np.random.default_rng(11)
    pool = Pool(2 * 40, 2, 32, 128, 2, 40, seed=16)
    pool.fill(rng, [1200, 1100])
    q = torch.from_numpy(rng.standard_normal((2, 1, 8, 128))).to(torch.bfloat16).to(DEV)
    q0, kl = q.clone(), _int([1000, 60])
    ws = torch.empty(fa.fa_decode_workspace_bytes(2, 8, 128, 16), dtype=torch.uint8, device=DEV)
    o, lse = torch.empty_like(q), torch.empty(2, 8, 1, device=DEV)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        kl.add_(33)
        q.copy_(q0)                              # a copy and not a kernel before the decode
        fa.fa_decode_splitkv_paged_fp8(q, *pool.args, kl, num_splits=16, workspace=ws, out=o, lse=lse)
    for i in range(1, 5):
        q.zero_()
        graph.replay()
        torch.cuda.synchronize()
        a, b = fa.fa_decode_splitkv_paged_fp8(q, *pool.args, _int([1000 + 33 * i, 60 + 33 * i]), num_splits=16)
        assert torch.equal(a, o) and torch.equal(b, lse)


def test_lengths_written_by_the_kernel_before(fa):
    """The decode starts, and guesses its plan, while the kernel before it may still be running; here
    that kernel (a read whose bf16 rows are the int32 lengths: 1.25 * 2^-125 is 288) writes
    other lengths.  Each decode has the bits of one whose lengths have long been there."""
    rng = np.random.default_rng(21)
    B, n = 32, 60000
    pool = Pool(B * 26, 2, 16, 64, B, 26, seed=22)
    pool.fill(rng, [400] * B)
    q = torch.from_numpy(rng.standard_normal((B, 1, 8, 64))).to(torch.bfloat16).to(DEV)
    sets, wants = [], []
    for i in range(3):
        # lengths 0, 256, 272, 288, 320, 352 and 384 (codes at scale 2^-127)
        codes = rng.choice([0.0, 4.0, 4.5, 5.0, 6.0, 7.0, 8.0], B)
        bits = torch.from_numpy(codes * 2.0 ** -127).to(torch.bfloat16).view(torch.int16)
        lens = bits.to(torch.int32).tolist()
        assert max(lens) <= 400 and sum(x > 0 for x in lens) > 10
        row = np.zeros(64)
        row[::2] = codes                          # low halves of the 32-bit lengths
        k = np.zeros((n // 16, 1, 16, 64), np.uint8)
        k[-1, 0, -1] = torch.from_numpy(row).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        k = torch.from_numpy(k).to(DEV).view(torch.float8_e4m3fn)
        zero = torch.zeros(k.shape[:3], dtype=torch.uint8, device=DEV)
        sets.append((k, k, zero, zero, torch.arange(n // 16, dtype=torch.int32, device=DEV).view(1, -1)))
        wants.append(fa.fa_decode_splitkv_paged_fp8(q, *pool.args, _int(lens), num_splits=8))
    out = [torch.empty(n, 1, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    kl = out[0][n - 1, 0].view(torch.int32)
    ws = torch.empty(fa.fa_decode_workspace_bytes(B, 8, 64, 8), dtype=torch.uint8, device=DEV)
    got = [[torch.empty_like(q), torch.empty(B, 8, 1, device=DEV)] for _ in range(12)]
    cu = _int([0, n])
    for i, (o, lse) in enumerate(got):
        fa.fa_kv_read_paged_fp8(*sets[i % 3], cu, k_out=out[0], v_out=out[1])
        fa.fa_decode_splitkv_paged_fp8(q, *pool.args, kl, num_splits=8, workspace=ws, out=o, lse=lse)
    for i, (o, lse) in enumerate(got):
        assert torch.equal(o, wants[i % 3][0]) and torch.equal(lse, wants[i % 3][1])


def test_two_streams_at_once(fa):
    """Two decodes with a workspace each on two streams give what each gives alone."""
    pool, q, o, lse = _decode_case(fa, 128, 8, 2, 1, 16, [1800, 900], ns=16, seed=6)
    qd, kl = q.to(DEV), _int([1800, 900])
    q2 = -qd
    alone = fa.fa_decode_splitkv_paged_fp8(q2, *pool.args, kl, num_splits=16)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for s, x in zip(streams, (qd, q2)):
            got.append(fa.fa_decode_splitkv_paged_fp8(x, *pool.args, kl, num_splits=16, stream=s))
    torch.cuda.synchronize()
    for i, (oo, ll) in enumerate(got):
        assert torch.equal(oo, (o, alone[0])[i % 2]) and torch.equal(ll, (lse, alone[1])[i % 2])


def test_another_stream_leaves_the_current_ones_memory_alone(fa):
    """Blocks of the sizes that a call makes, freed on the current stream while work queued there has
    yet to read or to write them: a call on another stream, which nothing orders behind that work,
    takes none of them.  And its outputs, freed while the current stream has yet to read them, are
    not handed to its next call."""
    pool, q, o_ref, lse_ref = _decode_case(fa, 128, 8, 2, 1, 16, [1800, 900], ns=16, seed=7)
    qd, kl, cu = q.to(DEV), _int([1800, 900]), _int([0, 1800, 2700])
    minus = -qd
    k_ref, v_ref = fa.fa_kv_read_paged_fp8(*pool.args, cu, total=2700)
    need = fa.fa_decode_workspace_bytes(2, 8, 128, 16)
    sizes = [q.numel() * 2, lse_ref.numel() * 4, need] + [k_ref.numel() * 2] * 2
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    for late in ("read", "written"):
        kept = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes]
        blocks = [torch.full((n,), 0x5A, dtype=torch.uint8, device=DEV) for n in sizes]
        torch.cuda.synchronize()
        torch.cuda._sleep(200_000_000)            # 0.1 s
        for a, b in zip(kept, blocks):
            if late == "read":
                a.copy_(b)
            else:
                b.fill_(0x77)
        del b, blocks
        got = [*fa.fa_decode_splitkv_paged_fp8(qd, *pool.args, kl, num_splits=16, stream=other),
               *fa.fa_kv_read_paged_fp8(*pool.args, cu, total=2700, stream=other)]
        torch.cuda.synchronize()
        assert late != "read" or all((a == 0x5A).all() for a in kept)
        for a, b in zip(got, (o_ref, lse_ref, k_ref, v_ref)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    del got, a
    for _ in range(3):
        o, lse = fa.fa_decode_splitkv_paged_fp8(qd, *pool.args, kl, num_splits=16, stream=other)
        torch.cuda.current_stream().wait_stream(other)
        torch.cuda._sleep(50_000_000)
        copies = o.clone(), lse.clone()
        del o, lse
        fa.fa_decode_splitkv_paged_fp8(minus, *pool.args, kl, num_splits=16, stream=other)
        torch.cuda.synchronize()
        assert torch.equal(copies[0], o_ref) and torch.equal(copies[1], lse_ref)


def test_streams_are_found_by_torchs_public_calls_too(fa, monkeypatch):
    from exact_tiled_attention_20_gb300 import _lib

    pool, q, o, lse = _decode_case(fa, 64, 4, 2, 1, 16, [300, 17], seed=8)
    qd, kl, side = q.to(DEV), _int([300, 17]), torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert _lib._raw_stream(0) == _lib._public_raw_stream(0) == side.cuda_stream
    monkeypatch.setattr(_lib, "_raw_stream", _lib._public_raw_stream)
    monkeypatch.setattr(_lib, "_current_device", torch.cuda.current_device)
    torch.cuda.synchronize()
    for stream in (None, side):
        a, b = fa.fa_decode_splitkv_paged_fp8(qd, *pool.args, kl, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(a, o) and torch.equal(b, lse)


def test_offsets_past_32_bits(fa):
    """A pool of more than 2^32 bytes of codes: the last pages are written, read and decoded."""
    Hkv, page, D, B = 8, 64, 128, 2
    pages = (1 << 32) // (Hkv * page * D) + 40
    k = torch.empty(pages, Hkv, page, D, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    v = torch.empty(pages, Hkv, page, D, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    ks, vs = (torch.empty(pages, Hkv, page, dtype=torch.uint8, device=DEV) for _ in range(2))
    high = torch.arange(pages - 6, pages, dtype=torch.int32, device=DEV).view(B, 3)
    low = torch.arange(6, dtype=torch.int32, device=DEV).view(B, 3)
    g = torch.Generator(DEV).manual_seed(3)
    kn, vn = (torch.randn(B, 150, Hkv, D, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(B, 1, 32, D, generator=g, device=DEV).to(torch.bfloat16)
    kl = _int([150, 150])
    outs = []
    for table in (low, high):
        fa.fa_kv_append_paged_fp8(kn, vn, k, v, ks, vs, table, kl)
        outs.append((*fa.fa_kv_read_paged_fp8(k, v, ks, vs, table, _int([0, 150, 300]), total=300),
                     *fa.fa_decode_splitkv_paged_fp8(q, k, v, ks, vs, table, kl, num_splits=3)))
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    off = (outs[1][0].view(B, 150, Hkv, D) - kn).float().abs()
    assert (off <= kn.float().abs() * 2.0 ** -4 + 2.0 ** -16).all()


# ---------------------------------------------------------------------- refusals ----
def test_binding_refuses(fa):
    pool = Pool(8, 2, 16, 64, 2, 2)
    kl, cu = _int([5, 5]), _int([0, 1, 2])
    x = torch.zeros(2, 1, 2, 64, dtype=torch.bfloat16, device=DEV)
    q = torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16, device=DEV)
    k, v, ks, vs, t = pool.args
    app, dec, rd = fa.fa_kv_append_paged_fp8, fa.fa_decode_splitkv_paged_fp8, fa.fa_kv_read_paged_fp8
    for bad in ((k.view(torch.uint8), v, ks, vs, t), (k, v[:7], ks, vs, t), (k, v, ks[:, :, :8], vs, t),
                (k, v, ks.int(), vs, t), (k, v, ks, vs, t.long()), (k, v, ks, vs, t[0]), (k.transpose(1, 2), v, ks, vs, t),
                (k[0], v[0], ks, vs, t), (k.cpu(), v, ks, vs, t), (k, v, ks, vs, t.cpu())):
        for call in (lambda: app(x, x, *bad, kl), lambda: dec(q, *bad, kl), lambda: rd(*bad, cu, total=2)):
            with pytest.raises((TypeError, ValueError)):
                call()
    for call in (lambda: app(x.float(), x.float(), *pool.args, kl), lambda: app(x, x.half(), *pool.args, kl),
                 lambda: app(x[:1], x[:1], *pool.args, kl), lambda: app(x[:, 0], x[:, 0], *pool.args, kl),
                 lambda: app(x, x, *pool.args, kl, cu_seqlens_new=cu), lambda: app(x, x, *pool.args, kl.long()),
                 lambda: app(x[:, 0], x[:, 0], *pool.args, kl, cu_seqlens_new=cu[:2]),
                 lambda: app(x[..., :32], x[..., :32], *pool.args, kl),
                 lambda: app(x.transpose(2, 3), x.transpose(2, 3), *pool.args, kl),
                 lambda: app(x, x, *pool.args, kl[:1]),
                 lambda: dec(q[:1], *pool.args, kl), lambda: dec(q[..., :32], *pool.args, kl),
                 lambda: dec(q.float(), *pool.args, kl), lambda: dec(q[:, 0], *pool.args, kl),
                 lambda: dec(q, *pool.args, kl, out=q[:, :, :2]), lambda: dec(q, *pool.args, kl, lse=torch.empty(2, 4, device=DEV)),
                 lambda: dec(q, *pool.args, kl, workspace=torch.empty(4, device=DEV)),
                 lambda: rd(*pool.args, cu), lambda: rd(*pool.args, cu, total=2, dtype=torch.float32),
                 lambda: rd(*pool.args, cu, k_out=x[:, 0], v_out=x[:, 0].half()),
                 lambda: rd(*pool.args, cu, total=3, k_out=x[:, 0], v_out=x[:, 0]),
                 lambda: rd(*pool.args, cu[:2], total=2), lambda: rd(*pool.args, cu, total=2, kv_starts=kl[:1])):
        with pytest.raises((TypeError, ValueError)):
            call()
    for call, status in ((lambda: dec(q, *pool.args, kl, num_splits=4, workspace=torch.empty(64, dtype=torch.uint8, device=DEV)), 3),
                         (lambda: dec(torch.zeros(2, 9, 4, 64, dtype=torch.bfloat16, device=DEV), *pool.args, kl), 2),
                         (lambda: dec(torch.zeros(2, 1, 3, 64, dtype=torch.bfloat16, device=DEV), *pool.args, kl), 1),
                         (lambda: dec(q, *pool.args, kl, scale=math.nan), 1)):
        with pytest.raises(fa.FaError) as e:
            call()
        assert e.value.status == status
    strided = torch.zeros(2, 1, 2 * 64 + 4, dtype=torch.bfloat16, device=DEV)[..., :128].unflatten(-1, (2, 64))
    with pytest.raises(fa.FaError) as e:          # a token stride that breaks the 16-byte alignment
        app(strided, strided, *pool.args, kl)
    assert e.value.status == 1
