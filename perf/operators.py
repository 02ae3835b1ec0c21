"""Cases for measuring the 8-bit paged KV cache: writing it, attending over it, reading it back.

The cache of one layer is a pool of pages in e4m3 with one power-of-two scale per
(token, kv head) row:

    k_pages, v_pages    float8_e4m3fn [num_pages, Hkv, page, D]
    k_scales, v_scales  uint8 [num_pages, Hkv, page]: exponent byte s, the scale is 2^(s - 127)
    block_table         int32 [B, max_pages]: key r of sequence b is row r % page of page
                        block_table[b][r // page]

Three operators work on it:

* append: quantises new K/V rows as it writes them. A row's scale is the least power of two
  2^e, e >= -127, with max|x| <= 448 * 2^e; its codes are e4m3(x / 2^e), round to nearest even.
* decode: softmax(scale * q k^T) v of Sq query tokens per sequence over its cached keys,
  bottom-right causal, and the natural log-sum-exp.
* read: rows of the cache as bf16/fp16, packed along the sequences (what a prefill over an
  already cached prefix takes as K and V).

Where ``own`` is false ``run`` computes them with elementary torch operations in 32 bits,
else it calls the package's entry points. Lengths are spread evenly over [lo, hi] and handed
to the sequences in a seeded order, so a case's work does not depend on the seed.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # One short chat turn on a small model: launch latency is all there is.
        _dec("decode_small", B=1, sq=1, Hq=8, Hkv=2, D=64, page=16, lo=113, hi=113, dtype="bf16"),
        # One long conversation: few (sequence, head) pairs, split over the length.
        _dec("decode_one_long", B=1, sq=1, Hq=32, Hkv=8, D=128, page=64, lo=32768, hi=32768, dtype="bf16"),
        # The benchmark's decode workload, lengths 1024..32768, in 256-key pages.
        _dec("decode_ragged", B=8, sq=1, Hq=32, Hkv=8, D=128, page=256, lo=1024, hi=32768, dtype="bf16"),
        # A busy server: many sequences of all lengths, small pages, one of them new (length 1).
        _dec("decode_server", B=64, sq=1, Hq=32, Hkv=8, D=128, page=16, lo=1, hi=8192, dtype="fp16"),
        # Head dim 96, one query head per kv head, odd batch, an empty sequence, pages of 48.
        _dec("decode_d96_mha", B=13, sq=1, Hq=12, Hkv=12, D=96, page=48, lo=0, hi=5001, dtype="bf16"),
        # Speculative decoding: four draft tokens at the widest head dim, causal among them.
        _dec("decode_draft_d256", B=8, sq=4, Hq=32, Hkv=8, D=256, page=128, lo=700, hi=16384, dtype="bf16"),
        # The write of a decode step: one token per sequence.
        _app("append_step", B=8, lo=1, hi=1, Hkv=8, D=128, page=64, past=2000, dtype="bf16"),
        # The same for a large batch at head dim 64 in fp16.
        _app("append_step_batch", B=256, lo=1, hi=1, Hkv=8, D=64, page=16, past=500, dtype="fp16"),
        # A batch of prompts written at once, 256..8192 tokens each.
        _app("append_prompts", B=16, lo=256, hi=8192, Hkv=8, D=128, page=64, past=0, dtype="bf16"),
        # Chunks of odd sizes behind an odd prefix, head dim 96, some sequences with no new token.
        _app("append_chunks_d96", B=7, lo=0, hi=1023, Hkv=12, D=96, page=48, past=333, dtype="bf16"),
        # A short cached prefix read back for the next prompt chunk.
        _rd("read_prefix", B=2, lo=97, hi=611, Hkv=2, D=64, page=16, dtype="bf16"),
        # Long prefixes of a batch read back.
        _rd("read_batch", B=16, lo=256, hi=8192, Hkv=8, D=128, page=64, dtype="bf16"),
    ]


def _dec(name, **c):
    return {"name": name, "op": "decode", **c}


def _app(name, **c):
    return {"name": name, "op": "append", **c}


def _rd(name, **c):
    return {"name": name, "op": "read", **c}


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "append", "read"])
    D = rng.choice([64, 96, 128, 256])
    Hkv = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
    B = _log_int(rng, 1, 256)
    page = 16 * _log_int(rng, 1, 16)
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    # tokens of the whole batch, so that no drawn case costs more than the largest listed one
    most = {"decode": 4.0e8, "append": 6.0e7, "read": 6.0e7}[op] / (2 * Hkv * D)
    mean = _log_int(rng, 1, max(1, min(16384, int(most / B))))
    spread = rng.choice([0.0, 0.5, 1.0])
    lo, hi = int(mean * (1 - spread)), int(mean * (1 + spread))
    if op == "decode":
        sq = rng.choice([1, 1, 1, 2, 3, 4])
        g = rng.randint(1, 16 // sq)
        return {"op": op, "B": B, "sq": sq, "Hq": g * Hkv, "Hkv": Hkv, "D": D, "page": page, "lo": lo,
                "hi": hi, "dtype": dtype}
    if op == "append":
        return {"op": op, "B": B, "lo": lo, "hi": hi, "Hkv": Hkv, "D": D, "page": page,
                "past": rng.randint(0, 700), "dtype": dtype}
    return {"op": op, "B": B, "lo": lo, "hi": hi, "Hkv": Hkv, "D": D, "page": page, "dtype": dtype}


def _spread(c):
    """The case's lengths: spread evenly over [lo, hi], the last one hi."""
    B, lo, hi = c["B"], c["lo"], c["hi"]
    return [hi if B == 1 else lo + (hi - lo) * i // (B - 1) for i in range(B)]


def _rows(g, *shape):
    """Rows as projections give them: normal, each row with a magnitude of its own."""
    x = torch.randn(shape, generator=g, device="cuda")
    return x.mul_(torch.randn((*shape[:-1], 1), generator=g, device="cuda").mul_(0.5).exp_())


def _quantise(x):
    """(codes, exponent bytes) of rows of finite values."""
    x = x.float()
    frac, ex = torch.frexp(x.abs().amax(-1))           # amax = frac 2^ex, 0.5 <= frac < 1; 448 = 0.875 2^9
    e = ex - 9 + (frac > 0.875).int()
    e = torch.where(frac == 0, -127, e).clamp(min=-127)
    return torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _value(codes, scales):
    return torch.ldexp(codes.float(), scales.int()[..., None] - 127)


def prepare(case, seed):
    c = case
    B, Hkv, D, page, dt = c["B"], c["Hkv"], c["D"], c["page"], _DT[c["dtype"]]
    g = torch.Generator("cuda").manual_seed(seed)
    host = torch.Generator("cpu").manual_seed(seed)
    counts = torch.tensor(_spread(c))[torch.randperm(B, generator=host)]
    past = c.get("past", 0)
    pasts = torch.randint(past // 2, past + 1, (B,), generator=host)
    lens = counts + pasts                               # keys in the cache (after the write, for append)
    max_pages = max(1, -(-(c["hi"] + past) // page))
    used = B * max_pages
    num_pages = used + 3
    table = torch.randperm(num_pages, generator=host)[:used].view(B, max_pages).to(torch.int32)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).to(torch.int32)
    s = {"case": dict(c), "table": table.cuda(), "lens": lens.to(torch.int32).cuda(), "cu": cu.cuda(),
         "total": int(counts.sum())}
    for n in ("k", "v"):
        codes, scales = [], []
        step = max(1, (1 << 26) // (Hkv * page * D))
        for p in range(0, num_pages, step):             # in parts: the 32-bit rows need not fit beside the pool
            a, b = _quantise(_rows(g, min(step, num_pages - p), Hkv, page, D))
            codes.append(a)
            scales.append(b)
        s[n + "_pages"], s[n + "_scales"] = torch.cat(codes), torch.cat(scales)
    if c["op"] == "decode":
        Hq, sq = c["Hq"], c["sq"]
        s["q"] = torch.randn((B, sq, Hq, D), generator=g, device="cuda").to(dt)
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((B, Hq, sq), device="cuda")
        # at most one partial result per 256 keys of the capacity for each query row
        rows = B * sq * Hq * max(1, -(-max_pages * page // 256))
        s["workspace"] = torch.empty(rows * D * 4 + rows * 4 + 512, dtype=torch.uint8, device="cuda")
    elif c["op"] == "append":
        s["k_new"], s["v_new"] = (_rows(g, s["total"], Hkv, D).to(dt) for _ in range(2))
    else:
        s["k"], s["v"] = (torch.empty((s["total"], Hkv, D), dtype=dt, device="cuda") for _ in range(2))
    return s


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        import exact_tiled_attention_20_gb300 as fa

        pool = (s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["table"])
        if op == "decode":
            return fa.fa_decode_splitkv_paged_fp8(s["q"], *pool, s["lens"], causal=True, workspace=s["workspace"],
                                                  out=s["o"], lse=s["lse"])
        if op == "append":
            fa.fa_kv_append_paged_fp8(s["k_new"], s["v_new"], *pool, s["lens"], cu_seqlens_new=s["cu"])
            return pool[:4]
        return fa.fa_kv_read_paged_fp8(*pool, s["cu"], k_out=s["k"], v_out=s["v"])
    return {"decode": _decode, "append": _append, "read": _read}[op](s)


def _sequence_of(s):
    """(sequence, offset within its rows) of each packed row."""
    row = torch.arange(s["total"], device="cuda")
    b = torch.searchsorted(s["cu"][1:].long(), row, right=True)
    return b, row - s["cu"].long()[b]


def _write(s, n, at, slot):
    codes, scales = _quantise(s[n + "_new"])
    s[n + "_pages"].view(torch.uint8)[at, :, slot] = codes.view(torch.uint8)
    s[n + "_scales"][at, :, slot] = scales


def _append(s):
    page = s["case"]["page"]
    b, i = _sequence_of(s)
    cu = s["cu"].long()
    key = s["lens"].long()[b] - (cu[b + 1] - cu[b]) + i
    at, slot = s["table"].long()[b, key // page], key % page
    _write(s, "k", at, slot)
    _write(s, "v", at, slot)
    return s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"]


def _gather(s, n, at, slot):
    codes = s[n + "_pages"].view(torch.uint8)[at, :, slot].view(torch.float8_e4m3fn)
    return s[n].copy_(_value(codes, s[n + "_scales"][at, :, slot]))


def _read(s):
    page = s["case"]["page"]
    b, key = _sequence_of(s)
    at, slot = s["table"].long()[b, key // page], key % page
    return _gather(s, "k", at, slot), _gather(s, "v", at, slot)


def _decode(s):
    c = s["case"]
    B, sq, Hq, Hkv, D = c["B"], c["sq"], c["Hq"], c["Hkv"], c["D"]
    L = s["table"].shape[1] * c["page"]
    at = s["table"].long()

    def rows(n):                                        # [B, Hkv, L, D] in 32 bits
        codes = s[n + "_pages"].view(torch.uint8)[at].view(torch.float8_e4m3fn)
        x = _value(codes, s[n + "_scales"][at])         # [B, pages, Hkv, page, D]
        return x.transpose(1, 2).reshape(B, Hkv, L, D)

    q = s["q"].float().view(B, sq, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    x = torch.matmul(q, rows("k").transpose(-1, -2)) * (1 / math.sqrt(D))      # [B, Hkv, g sq, L]
    token = torch.arange(sq, device="cuda").repeat(Hq // Hkv)                  # column (head, token)
    last = s["lens"].long()[:, None] - sq + token                             # last visible key
    seen = torch.arange(L, device="cuda") <= last[:, None, :, None]
    x = torch.where(seen, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(x - m), 0.0)
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, rows("v")) / torch.where(l > 0, l, 1.0)
    lse = torch.where(l > 0, m + torch.log(l), -math.inf)
    back = (B, Hkv, Hq // Hkv, sq)
    s["o"].copy_(o.view(*back, D).permute(0, 3, 1, 2, 4).reshape(B, sq, Hq, D))
    s["lse"].copy_(lse.view(B, Hq, sq))
    return s["o"], s["lse"]


def exact(case, seed):
    """The definitions in 64 bits, sequence by sequence."""
    s = prepare(case, seed)
    c, f8 = case, torch.float8_e4m3fn
    B, Hkv, D, page = c["B"], c["Hkv"], c["D"], c["page"]
    table, lens, cu = s["table"].tolist(), s["lens"].tolist(), s["cu"].tolist()

    def cached(n, b, upto):                             # [upto, Hkv, D]
        ids = table[b][:-(-upto // page)]
        codes = torch.stack([s[n + "_pages"][i] for i in ids]).double()
        two = torch.stack([s[n + "_scales"][i] for i in ids]).double()
        x = codes * torch.exp2(two - 127)[..., None]
        return x.permute(0, 2, 1, 3).reshape(-1, Hkv, D)[:upto]

    if c["op"] == "read":
        parts = [[cached(n, b, cu[b + 1] - cu[b]) for b in range(B) if cu[b + 1] > cu[b]] for n in ("k", "v")]
        empty = torch.empty((0, Hkv, D), dtype=torch.float64, device="cuda")
        return tuple(torch.cat(p) if p else empty for p in parts)
    if c["op"] == "append":
        outs = []
        for n in ("k", "v"):
            pool = s[n + "_pages"].double()
            x = s[n + "_new"].double()
            big = x.abs().amax(-1, keepdim=True)
            e = torch.ceil(torch.log2(torch.where(big > 0, big, 1.0) / 448))
            e = e - (big <= 448 * torch.exp2(e - 1)).double()    # log2 of an exact power may come out above it
            e = (e + (big > 448 * torch.exp2(e)).double()).clamp(min=-127)
            y = x * torch.exp2(-torch.where(big > 0, e, -127.0))
            grid = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)   # spacing of e4m3 at y
            y = torch.round(y / grid) * grid
            for b in range(B):
                new = cu[b + 1] - cu[b]
                first, done = lens[b] - new, 0
                while done < new:
                    key = first + done
                    take = min(new - done, page - key % page)
                    rows = y[cu[b] + done:cu[b] + done + take]
                    pool[table[b][key // page], :, key % page:key % page + take] = rows.transpose(0, 1)
                    done += take
            outs.append(pool)
        return outs[0], outs[1], None, None
    Hq, sq = c["Hq"], c["sq"]
    o = torch.zeros((B, sq, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, sq), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        if lens[b] == 0:
            continue
        k, v = cached("k", b, lens[b]), cached("v", b, lens[b])
        for t in range(sq):
            n = lens[b] - sq + t + 1                    # keys that token t sees
            if n <= 0:
                continue
            q = s["q"][b, t].double().view(Hkv, Hq // Hkv, D)
            x = torch.einsum("hgd,nhd->hgn", q, k[:n]) / math.sqrt(D)
            z = torch.logsumexp(x, -1)
            o[b, t] = torch.einsum("hgn,nhd->hgd", torch.exp(x - z[..., None]), v[:n]).reshape(Hq, D)
            lse[b, :, t] = z.reshape(Hq)
    return o, lse


def work(case):
    c = case
    total, Hkv, D = sum(_spread(c)), c["Hkv"], c["D"]
    if c["op"] == "decode":
        rows = c["B"] * c["sq"] * c["Hq"]
        pages = sum(-(-n // c["page"]) for n in _spread(c))
        return {"bytes": total * Hkv * 2 * (D + 1) + rows * (4 * D + 4) + 4 * pages + 4 * c["B"],
                "flops": 4 * total * c["sq"] * c["Hq"] * D}
    # a row: two bytes a value on the 16-bit side, one and the scale on the other
    return {"bytes": total * Hkv * 2 * (2 * D + D + 1), "flops": 2 * total * Hkv * 2 * D}
