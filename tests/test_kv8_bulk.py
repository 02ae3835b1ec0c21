"""The forms of the 8-bit cache's append and read that take several rows for each group of lanes, as
prompts do, and the decode's merge where pieces are many.  Values are compared bit for bit
over all rows, against a vectorised statement of the format that is itself held against
oracle/kv8.py."""
import math

import numpy as np
import pytest
import torch

import kv8_plan
from oracle import kv8
from test_kv8 import _check

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
DEV = "cuda:0"
CODES = torch.from_numpy(kv8.CODE_VALUES)


def quantise(x):
    """(codes uint8, scale bytes uint8) of finite rows, in 64 bits: every step but the last is exact."""
    x = x.double()
    amax = x.abs().amax(-1)
    e = torch.full(amax.shape, -127, dtype=torch.int64)
    if amax.numel() and amax.max() > 0:
        frac, two = torch.frexp(amax)             # amax = frac 2^two, frac in [0.5, 1)
        least = two.long() - 9                    # 448 = 0.875 2^9
        e = torch.where(amax > 0, least + (frac > 0.875).long(), e).clamp(min=-127)
    y = torch.ldexp(x, -e[..., None]).float()     # at most 11 bits: exact
    return y.to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)


def value(codes, scales):
    return torch.ldexp(CODES[codes.long()], scales.long()[..., None] - 127)


def place(table, counts, starts, num_pages, page):
    """(page, slot, whether it has one) of each packed row."""
    b = torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts))
    first = torch.tensor(np.concatenate([[0], np.cumsum(counts)[:-1]]))
    key = torch.tensor(starts)[b] + torch.arange(len(b)) - first[b]
    fits = (key >= 0) & (key < table.shape[1] * page)
    key = torch.where(fits, key, 0)
    at = torch.from_numpy(table).long()[b, key // page]
    return at, key % page, fits & (at >= 0) & (at < num_pages)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_the_vectorised_statement_is_the_oracles(dtype):
    g = torch.Generator().manual_seed(2)
    x = torch.randn(300, 2, 96, generator=g, dtype=torch.float64) * 2.0 ** torch.randint(-14, 12, (300, 2, 1), generator=g)
    x = x.to(DT[dtype])
    x[5], x[6, 0], x[7] = 0, x[6, 0] * 0 + 448, float(torch.finfo(DT[dtype]).tiny)
    codes, scales = quantise(x)
    want = kv8.quantise(x.double().numpy())
    assert np.array_equal(codes.numpy(), want[0]) and np.array_equal(scales.numpy(), want[1])
    assert np.array_equal(value(codes, scales).numpy(), kv8.values(*want))
    rng = np.random.default_rng(3)
    table = rng.permutation(12)[:9].reshape(3, 3).astype(np.int32)
    table[1, 1], table[2, 2] = 12, -3
    counts, starts = [20, 33, 0], [5, 20, 9]
    pages = [rng.integers(0, 127, (12, 2, 16, 64)).astype(np.uint8), rng.integers(100, 140, (12, 2, 16)).astype(np.uint8)]
    at, slot, ok = place(table, counts, starts, 12, 16)
    at = torch.where(ok, at, 0)
    got = torch.where(ok[:, None, None], value(torch.from_numpy(pages[0])[at, :, slot], torch.from_numpy(pages[1])[at, :, slot]), 0.0)
    want = np.concatenate([kv8.cached(*pages, table, b, starts[b], counts[b]) for b in range(3)])
    assert np.array_equal(got.numpy(), want)


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import exact_tiled_attention_20_gb300 as fa_mod
    from exact_tiled_attention_20_gb300 import build

    build.build_library()
    fa_mod.load()
    return fa_mod


def _int(x):
    return torch.tensor([int(i) for i in x], dtype=torch.int32, device=DEV)


def _cu(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(int)


def _batch(rng, tokens):
    """Ragged counts of `tokens` tokens, sequences without any among them."""
    cuts = np.sort(rng.integers(0, tokens + 1, 6))
    counts = np.diff(np.concatenate([[0], cuts, [tokens]])).tolist()
    return [0] + counts[:3] + [0, 0] + counts[3:] + [1, 0]


# Lane groups of a CTA (128 threads over the lanes of a row): rows a group takes 2 rows from 8 of
# them on for each SM and group, 4 from 64 on.
GROUPS = {"append": {64: 16, 96: 8, 128: 8, 256: 4}, "read": {64: 16, 96: 10, 128: 8, 256: 4}}


def _tokens(op, D, Hkv, u):
    """An odd number of tokens whose rows just reach the form with u rows a group."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rows = GROUPS[op][D] * sms * {2: 8, 4: 64}[u]
    return (-(-rows // Hkv) + 5) | 1


BULK = [(64, 1, 16, "bf16", 2), (64, 3, 48, "fp16", 4), (64, 24, 16, "bf16", 4), (96, 12, 32, "fp16", 2), (96, 1, 16, "bf16", 4),
        (96, 5, 48, "bf16", 2), (128, 3, 64, "fp16", 2), (128, 8, 16, "bf16", 4), (128, 12, 32, "bf16", 2),
        (128, 1, 16, "fp16", 4), (256, 1, 16, "bf16", 2), (256, 12, 32, "bf16", 4), (256, 3, 16, "fp16", 4), (256, 6, 48, "fp16", 2)]


@pytest.mark.gpu
@pytest.mark.parametrize("D,Hkv,page,dtype,u", BULK)
def test_append_of_prompts(fa, D, Hkv, page, dtype, u):
    """Every byte of the pool, with ragged sequences behind a prefix, pages outside the pool, keys
    outside the table, rows behind the last sequence and, for every other case, strided tokens."""
    rng = np.random.default_rng(D * 31 + Hkv)
    tokens = _tokens("append", D, Hkv, u)
    counts = _batch(rng, tokens)
    B, cu = len(counts), _cu(counts)
    starts = rng.integers(0, 70, B).tolist()
    mp = -(-(max(c + s for c, s in zip(counts, starts))) // page)
    used = B * mp
    table = rng.permutation(used + 2)[:used].reshape(B, mp).astype(np.int32)
    longest = int(np.argmax(counts))
    table[longest, mp // 2], table[longest, 0] = used + 2, -1
    starts[1] = -3                                                    # its first keys lie before 0
    starts[longest] += page                                           # its last ones behind the table
    pool = [torch.from_numpy(rng.integers(0, 256, (used + 2, Hkv, page) + last, dtype=np.uint8)) for last in ((D,), (D,), (), ())]
    rows, extra = int(cu[-1]), 7
    x = torch.from_numpy(rng.standard_normal((2, rows + extra, Hkv, D), dtype=np.float32))
    x *= torch.from_numpy(2.0 ** rng.integers(-6, 7, (2, rows + extra, Hkv, 1))).float()
    x = x.to(DT[dtype])
    want = [t.clone() for t in pool]
    at, slot, ok = place(table, counts, starts, used + 2, page)
    assert ok.any() and not ok.all()
    for i in range(2):
        codes, scales = quantise(x[i, :rows][ok])
        want[i][at[ok], :, slot[ok]] = codes
        want[2 + i][at[ok], :, slot[ok]] = scales
    dev = [t.to(DEV) for t in pool]
    args = (dev[0].view(torch.float8_e4m3fn), dev[1].view(torch.float8_e4m3fn), dev[2], dev[3], torch.from_numpy(table).to(DEV))
    if Hkv % 2:                                                       # K and V side by side, as a projection leaves them
        both = torch.cat([x[0], x[1]], 1).to(DEV)
        k, v = both[:, :Hkv], both[:, Hkv:]
    else:
        k, v = x[0].to(DEV), x[1].to(DEV)
    lens = [c + s for c, s in zip(counts, starts)]
    fa.fa_kv_append_paged_fp8(k, v, *args, _int(lens), cu_seqlens_new=_int(cu))
    for got, w in zip(dev, want):
        assert torch.equal(got.cpu(), w)


@pytest.mark.gpu
@pytest.mark.parametrize("D,u", [(64, 2), (64, 4), (96, 4), (128, 4), (256, 2)])
def test_append_of_prompts_with_equal_counts(fa, D, u):
    """[B, n, Hkv, D] without cu_seqlens: the same number of tokens for every sequence."""
    rng = np.random.default_rng(D)
    B, Hkv, page = 7, 3, 32
    n = -(-_tokens("append", D, Hkv, u) // B)
    starts = rng.integers(0, 40, B).tolist()
    mp = -(-(n + 40) // page)
    table = rng.permutation(B * mp).reshape(B, mp).astype(np.int32)
    pool = [torch.from_numpy(rng.integers(0, 256, (B * mp, Hkv, page) + last, dtype=np.uint8)) for last in ((D,), (D,), (), ())]
    x = torch.from_numpy(rng.standard_normal((2, B, n, Hkv, D), dtype=np.float32)).to(torch.bfloat16)
    at, slot, ok = place(table, [n] * B, starts, B * mp, page)
    assert ok.all()
    want = [t.clone() for t in pool]
    for i in range(2):
        codes, scales = quantise(x[i].view(B * n, Hkv, D))
        want[i][at, :, slot], want[2 + i][at, :, slot] = codes, scales
    dev = [t.to(DEV) for t in pool]
    fa.fa_kv_append_paged_fp8(x[0].to(DEV), x[1].to(DEV), dev[0].view(torch.float8_e4m3fn), dev[1].view(torch.float8_e4m3fn),
                              dev[2], dev[3], torch.from_numpy(table).to(DEV), _int([s + n for s in starts]))
    for got, w in zip(dev, want):
        assert torch.equal(got.cpu(), w)


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_append_of_prompts_with_values_that_are_not_finite(fa, bad):
    """A few of them among 40000 rows: their own codes are NaN, the rest of their rows is as if they were 0."""
    rng = np.random.default_rng(4)
    D, Hkv, page = 128, 2, 64
    tokens = _tokens("append", D, Hkv, 2)
    mp = -(-tokens // page)
    table = rng.permutation(mp).reshape(1, mp).astype(np.int32)
    x = torch.from_numpy(rng.standard_normal((2, tokens, Hkv, D), dtype=np.float32)).to(torch.bfloat16)
    hit = torch.from_numpy(rng.random((2, tokens, Hkv, D)) < 1e-5)
    assert 10 < hit.sum() < 1000
    at, slot, _ = place(table, [tokens], [0], mp, page)
    dev = [torch.zeros((mp, Hkv, page) + last, dtype=torch.uint8, device=DEV) for last in ((D,), (D,), (), ())]
    y = torch.where(hit, bad, x)
    fa.fa_kv_append_paged_fp8(y[0].to(DEV), y[1].to(DEV), dev[0].view(torch.float8_e4m3fn), dev[1].view(torch.float8_e4m3fn),
                              dev[2], dev[3], torch.from_numpy(table).to(DEV), _int([tokens]), cu_seqlens_new=_int([0, tokens]))
    for i in range(2):
        codes, scales = quantise(torch.where(hit[i], 0.0, x[i]))
        codes[hit[i]] = 0x7F
        assert torch.equal(dev[i].cpu()[at, :, slot], codes) and torch.equal(dev[2 + i].cpu()[at, :, slot], scales)


@pytest.mark.gpu
@pytest.mark.parametrize("D,Hkv,page,dtype,u", BULK)
def test_read_of_prefixes(fa, D, Hkv, page, dtype, u):
    """Every row, with ragged sequences from odd starts on, pages outside the pool, keys outside the
    table and rows that no sequence owns."""
    rng = np.random.default_rng(D * 7 + Hkv)
    tokens = _tokens("read", D, Hkv, u)
    counts = _batch(rng, tokens)
    B, cu = len(counts), _cu(counts)
    starts = rng.integers(0, 70, B).tolist()
    mp = -(-(max(c + s for c, s in zip(counts, starts))) // page)
    used = B * mp
    table = rng.permutation(used + 2)[:used].reshape(B, mp).astype(np.int32)
    longest = int(np.argmax(counts))
    table[longest, mp // 2], table[longest, 0] = used + 2, -1
    starts[1] = -3
    starts[longest] += page
    pool = [torch.from_numpy(rng.integers(0, 256, (used + 2, Hkv, page, D), dtype=np.uint8)) for _ in range(2)]
    pool += [torch.from_numpy(rng.integers(90, 165, (used + 2, Hkv, page), dtype=np.uint8)) for _ in range(2)]
    at, slot, ok = place(table, counts, starts, used + 2, page)
    assert ok.any() and not ok.all()
    at = torch.where(ok, at, 0)
    rows, extra, dt = int(cu[-1]), 7, DT[dtype]
    dev = [t.to(DEV) for t in pool]
    out = [torch.full((rows + extra, Hkv, D), 7.0, dtype=dt, device=DEV) for _ in range(2)]
    fa.fa_kv_read_paged_fp8(dev[0].view(torch.float8_e4m3fn), dev[1].view(torch.float8_e4m3fn), dev[2], dev[3],
                            torch.from_numpy(table).to(DEV), _int(cu), kv_starts=_int(starts), k_out=out[0], v_out=out[1])
    for i in range(2):
        want = value(pool[i][at, :, slot], pool[2 + i][at, :, slot])
        want = torch.where(ok[:, None, None], want, 0.0).float().to(dt)     # exact in 32 bits, then rounded once
        got = out[i].cpu()
        assert torch.equal(got[:rows].isnan(), want.isnan())
        fine = ~want.isnan()
        assert torch.equal(got[:rows].view(torch.int16)[fine], want.view(torch.int16)[fine])
        assert (got[rows:] == 7).all()


# ------------------------------------------------------------------------- merge ----
@pytest.mark.gpu
@pytest.mark.parametrize("D,Hq,Hkv,Sq,B,longest,ns,pieces", [
    # eight warps a row, each with 8 pieces in a batch (4 at D = 256)
    (64, 2, 1, 1, 1, 30011, 400, 65), (96, 3, 1, 2, 1, 30011, 400, 65), (128, 2, 1, 1, 1, 30011, 400, 65),
    (128, 8, 2, 1, 1, 30011, 300, 129), (256, 2, 1, 1, 1, 20011, 300, 33), (256, 1, 1, 3, 2, 9011, 150, 33),
    # one warp a row: more than eight rows an SM
    (64, 16, 4, 4, 20, 6011, 16, 9), (96, 16, 4, 4, 20, 6011, 16, 9), (128, 16, 4, 4, 20, 6011, 16, 9),
    (256, 16, 4, 4, 20, 6011, 16, 9)])
def test_decode_of_many_pieces(fa, D, Hq, Hkv, Sq, B, longest, ns, pieces):
    """Pairs cut into more pieces than a warp of the merge loads at once, so that it moves its running
    maximum from batch to batch; short and empty sequences beside them."""
    rng = np.random.default_rng(D + Hq)
    page, mp = 64, -(-longest // 64)
    lens = [longest] + rng.integers(0, 100, B - 1).tolist()
    if B > 2:
        lens[1], lens[2], lens[-1] = 0, 2, longest - 7
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert (B * Sq * Hq > 8 * sms) == (B > 2)
    plan = kv8_plan.host(B, Hkv, mp * page, B * Hkv * ns, (2 if D == 256 or Hq // Hkv * Sq > 8 else 3) * sms, D)
    assert max(map(len, kv8_plan.segments(lens, Hkv, *plan)[1].values())) >= pieces
    table = rng.permutation(B * mp).reshape(B, mp).astype(np.int32)
    pool = []
    for _ in range(2):
        x = rng.standard_normal((B * mp, Hkv, page, D), dtype=np.float32) * 2.0 ** rng.uniform(-3, 3, (B * mp, Hkv, page, 1))
        pool.append(quantise(torch.from_numpy(x).bfloat16()))
    pool = [pool[0][0], pool[1][0], pool[0][1], pool[1][1]]
    q = torch.from_numpy(rng.standard_normal((B, Sq, Hq, D))).bfloat16()
    dev = [t.to(DEV) for t in pool]
    o, lse = fa.fa_decode_splitkv_paged_fp8(q.to(DEV), dev[0].view(torch.float8_e4m3fn), dev[1].view(torch.float8_e4m3fn),
                                            dev[2], dev[3], torch.from_numpy(table).to(DEV), _int(lens), num_splits=ns)
    ref = kv8.decode(q.double().numpy(), [t.numpy() for t in pool], table, lens, 1 / math.sqrt(D))
    _check(o, lse, ref, longest, D, "bf16")
