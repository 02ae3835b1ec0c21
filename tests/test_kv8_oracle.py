"""The 64-bit reference of the 8-bit paged KV cache (oracle/kv8.py), held against other
statements of the same things. No GPU."""
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import kv8


def test_code_values_are_e4m3():
    codes = torch.arange(256, dtype=torch.uint8)
    assert np.array_equal(kv8.CODE_VALUES, codes.view(torch.float8_e4m3fn).double().numpy(), equal_nan=True)


def test_encode_rounds_to_nearest_even():
    g = torch.Generator().manual_seed(1)
    y = torch.cat([(torch.rand(4000, generator=g) * 2 - 1) * 448, torch.randn(4000, generator=g) * 0.02,
                   torch.tensor([0.0, -0.0, 448.0, -448.0, 2.0 ** -10, 3 * 2.0 ** -10, 17.0, 19.0, float("nan")])])
    want = y.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(kv8.encode(y.double().numpy()), want)


@pytest.mark.parametrize("amax,e", [(448.0, 0), (448.0 * 2 ** 5, 5), (449.0, 1), (1.0, -8), (0.875, -9), (0.876, -8),
                                    (0.0, -127), (448 * 2.0 ** -127, -127), (2.0 ** -133, -127),
                                    (1.75 * 2.0 ** 127, 119), (1.9 * 2.0 ** 127, 120)])
def test_scale_is_the_least_power_of_two(amax, e):
    row = np.zeros((1, 64))
    row[0, 5] = -amax
    codes, s = kv8.quantise(row)
    assert int(s[0]) == e + 127
    assert abs(kv8.values(codes, s)[0, 5] + amax) <= max(amax * 2.0 ** -4, 2.0 ** (e - 10))


def test_quantise_keeps_nonfinite_values_visible():
    row = np.ones((1, 64))
    row[0, 3], row[0, 4], row[0, 5] = np.inf, -np.inf, np.nan
    codes, s = kv8.quantise(row)
    assert int(s[0]) == 127 - 8
    assert (codes[0, 3:6] == 0x7F).all() and np.isnan(kv8.values(codes, s)[0, 3:6]).all()
    assert (kv8.values(codes, s)[0, 6:] == 1).all()


def test_decode_is_attention_over_the_values():
    """The same values in a 16-bit cache go through the paged reference of the C oracle; a
    page outside the pool is a page of zeros."""
    rng = np.random.default_rng(3)
    B, Hq, Hkv, D, page, mp, pages = 3, 4, 2, 64, 16, 3, 11
    codes = rng.integers(0, 127, (2, pages, Hkv, page, D)).astype(np.uint8)
    scales = rng.integers(117, 122, (2, pages, Hkv, page)).astype(np.uint8)
    table = rng.permutation(pages)[:B * mp].reshape(B, mp).astype(np.int32)
    table[1, 1] = pages
    table[2, 0] = -1
    lens = np.array([48, 40, 17], np.int32)
    q = rng.standard_normal((B, 1, Hq, D))
    o, lse, o_abs, _, o_top = kv8.decode(q, (codes[0], codes[1], scales[0], scales[1]), table, lens, 0.1)
    safe = np.where((table < 0) | (table >= pages), pages, table)
    vals = [np.concatenate([kv8.values(c, s).transpose(0, 2, 1, 3), np.zeros((1, page, Hkv, D))])
            for c, s in zip(codes, scales)]
    o_ref, lse_ref = oracle.decode_paged(q, vals[0], vals[1], safe, lens, scale=0.1)
    np.testing.assert_allclose(o[:, 0], o_ref, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(lse[:, :, 0], lse_ref, rtol=1e-12)
    assert (o_abs >= np.abs(o) - 1e-12).all() and (o_top >= o_abs - 1e-12).all()


def test_decode_masks_from_the_bottom_right():
    """Sq = 4 tokens over 2 keys: the first two see none; the last sees both."""
    pool = (np.full((1, 1, 16, 64), 0x38, np.uint8),) * 2 + (np.full((1, 1, 16), 127, np.uint8),) * 2
    q = np.ones((1, 4, 1, 64))
    o, lse, _, _, _ = kv8.decode(q, pool, np.zeros((1, 1), np.int32), [2], 0.5)
    assert (o[0, :2] == 0).all() and np.isneginf(lse[0, 0, :2]).all()
    assert lse[0, 0, 2] == 32.0 and abs(lse[0, 0, 3] - (32 + math.log(2))) < 1e-12
    assert (kv8.decode(q, pool, np.zeros((1, 1), np.int32), [2], 0.5, causal=False)[0] == 1).all()


def test_append_then_cached_round_trips():
    rng = np.random.default_rng(5)
    pages, Hkv, page, D = 6, 2, 16, 64
    pool = (np.zeros((pages, Hkv, page, D), np.uint8), np.zeros((pages, Hkv, page, D), np.uint8),
            np.zeros((pages, Hkv, page), np.uint8), np.zeros((pages, Hkv, page), np.uint8))
    table = np.array([[4, 1], [0, 9]], np.int32)                   # 9: outside the pool, dropped
    k, v = rng.standard_normal((2, 30, Hkv, D))
    kv8.append(pool, k, v, table, [20, 20], [0, 12, 30])
    back = kv8.cached(pool[0], pool[2], table, 0, 8, 12)
    assert (np.abs(back - k[:12]) <= np.abs(k[:12]) * 2.0 ** -4 + 2.0 ** -16).all()
    back = kv8.cached(pool[1], pool[3], table, 1, 0, 20)
    assert (back[:2] == 0).all() and (back[16:] == 0).all()        # before the new keys; no page
    assert (np.abs(back[2:16] - v[12:26]) <= np.abs(v[12:26]) * 2.0 ** -4 + 2.0 ** -16).all()
