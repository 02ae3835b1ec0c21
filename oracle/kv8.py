"""The 8-bit paged KV cache in plain numpy, 64 bits -- TEST INFRASTRUCTURE ONLY.

A row of D values is held as e4m3 codes and a byte s: code * 2^(s - 127), with 2^(s - 127)
the least power of two 2^e, e >= -127, for which max|x| <= 448 * 2^e.  Pools are
[num_pages, Hkv, page_size, D] (codes, uint8 here) and [num_pages, Hkv, page_size] (s).
"""
from __future__ import annotations

import numpy as np


def _code_values() -> np.ndarray:
    """The 256 values of e4m3: sign, 4 exponent bits (bias 7), 3 fraction bits; exponent 0 is
    subnormal; exponent 15 with fraction 7 is NaN; there is no infinity."""
    v = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        x = f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        if e == 15 and f == 7:
            x = np.nan
        v[c] = -x if c & 128 else x
    return v


CODE_VALUES = _code_values()
_POSITIVE = CODE_VALUES[:127]  # 0 .. 448, ascending


def encode(y) -> np.ndarray:
    """e4m3 codes of values with |y| <= 448: nearest, ties to the even code; NaN -> 0x7f."""
    y = np.asarray(y, np.float64)
    a = np.abs(np.where(np.isnan(y), 0.0, y))
    assert a.max(initial=0.0) <= 448
    hi = np.searchsorted(_POSITIVE, a, side="left").clip(0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = _POSITIVE[hi] - a, a - _POSITIVE[lo]
    pick = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    pick = np.where(_POSITIVE[hi] == a, hi, pick)
    return np.where(np.isnan(y), 0x7F, pick | (np.signbit(y) * 128)).astype(np.uint8)


def quantise(x):
    """(codes uint8 [..., D], scale bytes uint8 [...]) of rows x [..., D]."""
    x = np.asarray(x, np.float64)
    fine = np.isfinite(x)
    amax = np.abs(np.where(fine, x, 0.0)).max(-1)
    e = np.full(amax.shape, -127)
    for i in np.ndindex(amax.shape):
        while amax[i] > 448 * 2.0 ** e[i]:
            # jump close, then step: 448 2^e >= amax has a least solution above -127
            e[i] = max(e[i] + 1, int(np.floor(np.log2(amax[i]))) - 10)
    with np.errstate(invalid="ignore"):
        y = np.where(fine, x, np.nan) / (2.0 ** e.astype(np.float64))[..., None]
    return encode(y), (e + 127).astype(np.uint8)


def values(codes, scales):
    return CODE_VALUES[codes] * (2.0 ** (np.asarray(scales, np.float64) - 127))[..., None]


def _where(table, b, key, num_pages, page):
    """(page, slot) of a key, or None outside the table or the pool."""
    if key < 0 or key >= table.shape[1] * page:
        return None
    p = int(table[b, key // page])
    return (p, key % page) if 0 <= p < num_pages else None


def append(pool, k_new, v_new, table, kv_lens, cu):
    """Writes packed rows [total, Hkv, D] (float64) into pool = (k, v, ks, vs), in place."""
    k, v, ks, vs = pool
    num_pages, _, page, _ = k.shape
    for b in range(len(cu) - 1):
        n = cu[b + 1] - cu[b]
        for i in range(n):
            at = _where(table, b, int(kv_lens[b]) - n + i, num_pages, page)
            if at is None:
                continue
            k[at[0], :, at[1]], ks[at[0], :, at[1]] = quantise(k_new[cu[b] + i])
            v[at[0], :, at[1]], vs[at[0], :, at[1]] = quantise(v_new[cu[b] + i])


def cached(codes, scales, table, b, first, n):
    """Keys first .. first + n - 1 of sequence b as values [n, Hkv, D]; zeros where there is no page."""
    num_pages, Hkv, page, D = codes.shape
    out = np.zeros((n, Hkv, D))
    for i in range(n):
        at = _where(table, b, first + i, num_pages, page)
        if at is not None:
            out[i] = values(codes[at[0], :, at[1]], scales[at[0], :, at[1]])
    return out


def cached_scales(scales, table, b, n):
    """The scales of keys 0 .. n - 1 of sequence b, [n, Hkv]; of a key without a page the least."""
    num_pages, Hkv, page = scales.shape
    out = np.full((n, Hkv), 2.0 ** -127)
    for i in range(n):
        at = _where(table, b, i, num_pages, page)
        if at is not None:
            out[i] = 2.0 ** (scales[at[0], :, at[1]].astype(np.float64) - 127)
    return out


def decode(q, pool, table, kv_lens, scale, causal=True):
    """q [B, Sq, Hq, D] -> (o [B, Sq, Hq, D], lse [B, Hq, Sq], o_abs, s_abs, o_top), the last three
    what the error bounds of a computation in fewer bits go by: o_abs = sum_j p_j |v_j|; s_abs the
    largest scale * sum_d |q_d k_jd| of the row; o_top = max_j (p_j vscale_j) * sum_j |vcode_j|."""
    q = np.asarray(q, np.float64)
    B, Sq, Hq, D = q.shape
    k, v, ks, vs = pool
    capacity = table.shape[1] * k.shape[2]
    g = Hq // k.shape[1]
    o, o_abs, o_top = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape)
    lse, s_abs = np.full((B, Hq, Sq), -np.inf), np.zeros((B, Hq, Sq))
    for b in range(B):
        n = min(max(int(kv_lens[b]), 0), capacity)
        kb, vb = cached(k, ks, table, b, 0, n), cached(v, vs, table, b, 0, n)
        sb = cached_scales(vs, table, b, n)
        for i in range(Sq):
            m = min(n, n - Sq + i + 1) if causal else n
            if m <= 0:
                continue
            for h in range(Hq):
                s = kb[:m, h // g] @ q[b, i, h] * scale
                top = s.max()
                p = np.exp(s - top)
                l = p.sum()
                o[b, i, h] = p @ vb[:m, h // g] / l
                va, sv = np.abs(vb[:m, h // g]), sb[:m, h // g]
                o_abs[b, i, h] = p @ va / l
                o_top[b, i, h] = (p * sv).max() / l * (va / sv[:, None]).sum(0)
                lse[b, h, i] = top + np.log(l)
                s_abs[b, h, i] = (np.abs(kb[:m, h // g]) @ np.abs(q[b, i, h])).max() * scale
    return o, lse, o_abs, s_abs, o_top
