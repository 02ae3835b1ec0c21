"""Cases for measuring attention over a 16-bit paged KV cache under masks of its own, and what goes with it.

The cache of one layer is the pool of the paged decode:

    k_pages, v_pages    [num_pages, page, Hkv, D], bf16 or fp16
    block_table         int32 [B, max_pages]: key r of sequence b is row r % page of page
                        block_table[b][r // page]

Four operators:

* append: new K/V rows are written into the pool, keys and queries rotated by their positions on
  the way: with an angle's cosine c and sine s, (x, y) -> (x c - y s, y c + x s) for the pairs
  (d, d + rot / 2) or, interleaved, (2 d, 2 d + 1) of the first rot dims.
* tree: softmax(scale q k^T) v of Sq drafted tokens per sequence, the last Sq keys of its cache:
  every token sees all keys before the drafts, and of the drafts those its mask names.
* step: Sq tokens per sequence, the last ones of its cache, each seeing the last window + 1 keys
  up to its own and the first `sinks` ones (a sliding window with sinks).
* prompt: the forward over whole prompts under the same mask, [B, S, H, D] or packed.

Where ``own`` is false ``run`` computes them with elementary torch operations in 32 bits,
else it calls the package's entry points. Lengths are spread evenly over [lo, hi] and handed
to the sequences in a seeded order, so a case's work does not depend on the seed.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # One decode step's write for a batch of eight: launch latency is all there is.
        _case("append_step", "append", B=8, Hq=32, Hkv=8, D=128, lo=1, hi=1, past=2000, page=256, rot=128,
              interleaved=False, explicit=False, dtype="bf16"),
        # Drafted trees written for a batch: positions of their own, interleaved pairs, part of the dims.
        _case("append_tree_d64", "append", B=48, Hq=12, Hkv=4, D=64, lo=13, hi=13, past=500, page=16, rot=32,
              interleaved=True, explicit=True, dtype="fp16"),
        # A batch of prompts written at once, 256..8192 tokens each.
        _case("append_prompts", "append", B=16, Hq=32, Hkv=8, D=128, lo=256, hi=8192, past=0, page=128, rot=128,
              interleaved=False, explicit=False, dtype="bf16"),
        # A short chat on a small model, a tree of seven drafts, small pages.
        _case("tree_small", "tree", B=1, sq=7, Hq=8, Hkv=2, D=64, lo=333, hi=333, page=16, dtype="bf16"),
        # The benchmark's decode lengths with 26 drafts each: 104 query rows per kv head.
        _case("tree_ragged", "tree", B=8, sq=26, Hq=32, Hkv=8, D=128, lo=1024, hi=32768, page=256, dtype="bf16"),
        # A server with wide trees: 64 drafts of 4 heads, 256 query rows per kv head, lengths of all sizes.
        _case("tree_wide", "tree", B=16, sq=64, Hq=32, Hkv=8, D=128, lo=65, hi=8192, page=64, dtype="fp16"),
        # The widest head dim, few drafts.
        _case("tree_d256", "tree", B=5, sq=9, Hq=16, Hkv=4, D=256, lo=701, hi=9001, page=128, dtype="bf16"),
        # A decode step of a streaming server: long caches of which a window and four sinks are read.
        _case("step_stream", "step", B=64, sq=1, Hq=32, Hkv=8, D=128, lo=1, hi=16384, page=128, window=1023, sinks=4,
              dtype="bf16"),
        # Head dim 96, one query head per kv head, three tokens, a window of odd size, pages of 48.
        _case("step_d96_mha", "step", B=13, sq=3, Hq=12, Hkv=12, D=96, lo=3, hi=5001, page=48, window=600, sinks=37,
              dtype="fp16"),
        # A chunk of a prompt behind its cached part on a small model.
        _case("prompt_small", "prompt", B=1, Sq=77, Sk=500, Hq=8, Hkv=2, D=64, window=127, sinks=4, packed=False,
              dtype="bf16"),
        # The benchmark's sliding window shape (two of its sixteen sequences), with four sinks.
        _case("prompt_long", "prompt", B=2, Sq=8192, Sk=8192, Hq=32, Hkv=32, D=128, window=1023, sinks=4, packed=False,
              dtype="bf16"),
        # Packed prompts of all lengths, grouped heads.
        _case("prompt_packed", "prompt", B=8, Sq=4096, Sk=4096, Hq=32, Hkv=8, D=128, window=511, sinks=64, packed=True,
              dtype="bf16"),
    ]


def _case(name, op, **c):
    return {"name": name, "op": op, **c}


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "tree", "tree", "step", "prompt"])
    D = rng.choice([64, 96, 128, 256])
    Hkv = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
    g = rng.choice([1, 1, 2, 3, 4, 4, 5, 8, 16])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    page = 16 * _log_int(rng, 1, 16)
    c = {"op": op, "Hq": g * Hkv, "Hkv": Hkv, "D": D, "dtype": dtype}
    if op == "prompt":
        Sq = _log_int(rng, 1, 4096)
        Sk = Sq + rng.choice([0, 0, _log_int(rng, 1, 2048)])
        most = 2 * 32 * 8192 * 1024 * 128               # the longest listed one's products
        B = min(_log_int(rng, 1, 16), max(1, int(min(most / (g * Hkv * Sq * Sk * D), 4.0e9 / (g * Hkv * Sq * Sk)))))
        return {**c, "B": B, "Sq": Sq, "Sk": Sk, "window": _log_int(rng, 1, 4096), "sinks": _log_int(rng, 1, 200) - 1,
                "packed": rng.random() < 0.5}
    B = _log_int(rng, 1, 128)
    most = {"append": 1.0e8, "tree": 2.5e8, "step": 2.5e8}[op] / (Hkv * D * (1 + g if op == "append" else 2))
    mean = _log_int(rng, 1, max(1, min(16384, int(most / B))))
    spread = rng.choice([0.0, 0.5, 1.0])
    c |= {"B": B, "page": page, "lo": int(mean * (1 - spread)), "hi": int(mean * (1 + spread))}
    if op == "append":
        rot = rng.choice([D, D, D // 2])
        return {**c, "past": rng.randint(0, 700), "rot": rot, "interleaved": rng.random() < 0.3,
                "explicit": rng.random() < 0.3}
    if op == "tree":
        sq = _log_int(rng, 1, max(1, min(100, int(2.5e10 / (c["hi"] * B * g * Hkv * D)))))
        return {**c, "sq": sq, "lo": c["lo"] + sq, "hi": c["hi"] + sq}
    return {**c, "sq": rng.choice([1, 1, 1, 2, 4, 7]), "window": _log_int(rng, 1, 4096),
            "sinks": _log_int(rng, 1, 200) - 1}


def _spread(c):
    """The case's lengths: spread evenly over [lo, hi], the last one hi."""
    B, lo, hi = c["B"], c["lo"], c["hi"]
    return [hi if B == 1 else lo + (hi - lo) * i // (B - 1) for i in range(B)]


def _packed(c):
    """(queries, keys) of each sequence of a packed prompt: the last has all of Sq and Sk."""
    B = c["B"]
    return [(c["Sq"] * (i + 1) // B, c["Sk"] * (i + 1) // B) for i in range(B)]


def _trees(rng, B, sq):
    """Random trees, drafts in an order that puts parents first: bool [B, sq, sq], who sees whom."""
    sees = np.zeros((B, sq, sq), dtype=bool)
    at = np.arange(B)
    for t in range(sq):
        if t:
            parent = rng.integers(max(0, t - 6) - 1, t, B)          # -1: a root of its own
            sees[:, t] = sees[at, np.maximum(parent, 0)] & (parent >= 0)[:, None]
        sees[:, t, t] = True
    return sees


def _words(sees):
    """Rows of truth values as int32 words, bit t % 32 of word t // 32 being value t."""
    B, sq, n = sees.shape
    bits = np.zeros((B, sq, -(-n // 32) * 32), dtype=bool)
    bits[:, :, :n] = sees
    return np.packbits(bits, axis=-1, bitorder="little").view("<i4")


def prepare(case, seed):
    c, dt = case, _DT[case["dtype"]]
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    g = torch.Generator("cuda").manual_seed(seed)
    host = torch.Generator("cpu").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=dt)

    s = {"case": dict(c), "scale": 1 / math.sqrt(D)}
    if c["op"] == "prompt":
        if c["packed"]:
            nq, nk = (torch.tensor([x[i] for x in _packed(c)]) for i in (0, 1))
            order = torch.randperm(B, generator=host)
            nq, nk = nq[order], nk[order]
            zero = torch.zeros(1, dtype=torch.int64)
            s["cu_q"], s["cu_k"] = (torch.cat([zero, n.cumsum(0)]).to(torch.int32).cuda() for n in (nq, nk))
            tq, tk = int(nq.sum()), int(nk.sum())
            s["q"], s["k"], s["v"] = normal(tq, Hq, D), normal(tk, Hkv, D), normal(tk, Hkv, D)
            s["lse"] = torch.empty((Hq, tq), device="cuda")
        else:
            Sq, Sk = c["Sq"], c["Sk"]
            s["q"], s["k"], s["v"] = normal(B, Sq, Hq, D), normal(B, Sk, Hkv, D), normal(B, Sk, Hkv, D)
            s["lse"] = torch.empty((B, Hq, Sq), device="cuda")
        s["o"] = torch.empty_like(s["q"])
        return s
    page = c["page"]
    counts = torch.tensor(_spread(c))[torch.randperm(B, generator=host)]
    past = c.get("past", 0)
    pasts = torch.randint(past // 2, past + 1, (B,), generator=host)
    lens = counts + pasts                               # keys in the cache, the new ones among them
    max_pages = max(1, -(-(c["hi"] + past) // page))
    used = B * max_pages
    num_pages = used + 3
    table = torch.randperm(num_pages, generator=host)[:used].view(B, max_pages).to(torch.int32)
    s["table"], s["lens"] = table.cuda(), lens.to(torch.int32).cuda()
    s["k_pages"], s["v_pages"] = normal(num_pages, page, Hkv, D), normal(num_pages, page, Hkv, D)
    if c["op"] == "append":
        total = int(counts.sum())
        cu = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])
        s["total"], s["cu"] = total, cu.to(torch.int32).cuda()
        # one projection's output: queries, keys and values of a token side by side
        qkv = normal(total, Hq + 2 * Hkv, D)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["q_out"] = torch.empty((total, Hq, D), dtype=dt, device="cuda")
        most = c["hi"] + past
        freq = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64) / c["rot"])
        angle = torch.arange(most, dtype=torch.float64).cuda()[:, None] * freq.cuda()
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        s["positions"] = (torch.randint(0, most, (total,), generator=g, device="cuda", dtype=torch.int32)
                          if c["explicit"] else None)
        return s
    sq = c["sq"]
    s["q"] = normal(B, sq, Hq, D)
    s["o"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((B, Hq, sq), device="cuda")
    # two partial results for each SM, of at most 256 query rows
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    s["workspace"] = torch.empty(2 * sms * min(256, Hq // Hkv * sq) * (D + 1) * 4 + 512, dtype=torch.uint8, device="cuda")
    if c["op"] == "tree":
        s["mask"] = torch.from_numpy(_words(_trees(np.random.default_rng(seed), B, sq))).cuda()
    return s


def run(state):
    s = state
    c = s["case"]
    if own:
        import exact_tiled_attention_20_gb300 as fa

        if c["op"] == "append":
            fa.fa_kv_append_paged_rope(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["cos"],
                                       s["sin"], q=s["q"], q_out=s["q_out"], positions=s["positions"],
                                       cu_seqlens_new=s["cu"], interleaved=c["interleaved"])
            return s["q_out"], s["k_pages"], s["v_pages"]
        if c["op"] == "tree":
            return fa.fa_decode_splitkv_paged_tree(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["mask"],
                                                   workspace=s["workspace"], out=s["o"], lse=s["lse"])
        if c["op"] == "step":
            return fa.fa_decode_splitkv_paged_window(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"],
                                                     c["window"], sinks=c["sinks"], workspace=s["workspace"],
                                                     out=s["o"], lse=s["lse"])
        window = (c["window"], 0)
        if c["packed"]:
            return fa.fa_fwd_varlen(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=True, window=window,
                                    sinks=c["sinks"], out=s["o"], lse=s["lse"])
        return fa.fa_fwd(s["q"], s["k"], s["v"], causal=True, window=window, sinks=c["sinks"], out=s["o"], lse=s["lse"])
    return {"append": _append, "tree": _decode, "step": _decode, "prompt": _prompt}[c["op"]](s)


def _rotate(s, x, position):
    """x [total, H, D] in 32 bits, each row by the angles of its position."""
    c = s["case"]
    rot = c["rot"]
    co, si = s["cos"][position][:, None], s["sin"][position][:, None]
    y = x.float()
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if c["interleaved"] else (y[..., :rot // 2], y[..., rot // 2:rot])
    pair = (a * co - b * si, b * co + a * si)
    turned = torch.stack(pair, -1).flatten(-2) if c["interleaved"] else torch.cat(pair, -1)
    return torch.cat([turned, y[..., rot:]], -1)


def _append(s):
    c = s["case"]
    row = torch.arange(s["total"], device="cuda")
    cu = s["cu"].long()
    b = torch.searchsorted(cu[1:], row, right=True)
    key = s["lens"].long()[b] - (cu[b + 1] - cu[b]) + row - cu[b]
    at, slot = s["table"].long()[b, key // c["page"]], key % c["page"]
    position = key if s["positions"] is None else s["positions"].long()
    s["q_out"].copy_(_rotate(s, s["q"], position))
    s["k_pages"][at, slot] = _rotate(s, s["k"], position).to(s["k_pages"].dtype)
    s["v_pages"][at, slot] = s["v"]
    return s["q_out"], s["k_pages"], s["v_pages"]


def _attend(q, k, v, seen, scale):
    """q [..., R, D], k and v [..., L, D] in 32 bits, seen [..., R, L]: the output and the log-sum-exp."""
    x = torch.matmul(q, k.transpose(-1, -2)) * scale
    x = torch.where(seen, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, 0.0)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(l > 0, l, 1.0)
    return o, torch.where(l > 0, m + torch.log(l), -math.inf)[..., 0]


def _decode(s):
    c = s["case"]
    B, sq, Hq, Hkv, D = c["B"], c["sq"], c["Hq"], c["Hkv"], c["D"]
    g, L = Hq // Hkv, s["table"].shape[1] * c["page"]
    at = s["table"].long()

    def rows(n):                                        # [B, Hkv, L, D] in 32 bits
        return s[n][at].float().reshape(B, L, Hkv, D).transpose(1, 2)

    key = torch.arange(L, device="cuda")
    lens = s["lens"].long()[:, None, None]
    token = torch.arange(sq, device="cuda")[None, :, None]
    if c["op"] == "step":
        last = lens - sq + token
        seen = (key <= last) & ((key >= last - c["window"]) | (key < c["sinks"]))
    else:
        draft = (key - (lens - sq)).expand(B, 1, L)     # below 0: before the drafts
        t = draft.clamp(0, sq - 1)
        word = torch.gather(s["mask"].long(), 2, (t // 32).expand(B, sq, L))
        seen = (draft < 0) | ((word >> (t % 32)) % 2 == 1) & (draft < sq)
    q = s["q"].float().view(B, sq, Hkv, g, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, g * sq, D)
    seen = seen[:, None].repeat(1, 1, g, 1)             # [B, 1, g sq, L]
    o, lse = _attend(q, rows("k_pages"), rows("v_pages"), seen, s["scale"])
    s["o"].copy_(o.view(B, Hkv, g, sq, D).permute(0, 3, 1, 2, 4).reshape(B, sq, Hq, D))
    s["lse"].copy_(lse.view(B, Hq, sq))
    return s["o"], s["lse"]


def _prompt(s):
    c = s["case"]
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    Sq, Sk = c["Sq"], c["Sk"]
    i, j = torch.arange(Sq, device="cuda")[:, None], torch.arange(Sk, device="cuda")
    if c["packed"]:                                     # each sequence a row of a padded batch
        cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
        nq, nk = cu_q.diff()[:, None, None], cu_k.diff()[:, None, None]
        at_q = (cu_q[:-1, None] + i[:, 0]).clamp(max=s["q"].shape[0] - 1)
        at_k = (cu_k[:-1, None] + j).clamp(max=s["k"].shape[0] - 1)
        q, k, v = s["q"][at_q], s["k"][at_k], s["v"][at_k]
        last, there = i + nk - nq, j < nk
    else:
        q, k, v = s["q"], s["k"], s["v"]
        last, there = (i + Sk - Sq)[None], True
    seen = (j <= last) & ((j >= last - c["window"]) | (j < c["sinks"])) & there      # [B or 1, Sq, Sk]
    g = Hq // Hkv
    q = q.float().view(B, Sq, Hkv, g, D).permute(0, 2, 3, 1, 4)
    k, v = (x.float().transpose(1, 2)[:, :, None] for x in (k, v))
    o, lse = _attend(q, k, v, seen[:, None, None], s["scale"])
    o, lse = o.permute(0, 3, 1, 2, 4).reshape(B, Sq, Hq, D), lse.reshape(B, Hq, Sq)
    if c["packed"]:
        b = torch.searchsorted(cu_q[1:], torch.arange(s["q"].shape[0], device="cuda"), right=True)
        r = torch.arange(s["q"].shape[0], device="cuda") - cu_q[b]
        o, lse = o[b, r], lse[b, :, r].t()
    s["o"].copy_(o)
    s["lse"].copy_(lse)
    return s["o"], s["lse"]


def exact(case, seed):
    """The definitions in 64 bits, sequence by sequence."""
    s = prepare(case, seed)
    return {"append": _exact_append, "tree": _exact_decode, "step": _exact_decode, "prompt": _exact_prompt}[
        case["op"]](case, s)


def _exact_append(c, s):
    table, lens, cu = s["table"].tolist(), s["lens"].tolist(), s["cu"].tolist()
    page, rot = c["page"], c["rot"]
    kp, vp = s["k_pages"].double(), s["v_pages"].double()
    q_out = s["q"].double()
    first = torch.arange(rot // 2, device="cuda")
    i, j = (2 * first, 2 * first + 1) if c["interleaved"] else (first, first + rot // 2)

    def turn(x, pos):
        z = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), torch.zeros((), dtype=torch.float64,
                                                                                       device="cuda"))
        z = z * torch.complex(s["cos"][pos].double(), s["sin"][pos].double())[:, None]
        w = torch.complex(x[..., i], x[..., j]) * z
        y = x.clone()
        y[..., i], y[..., j] = w.real, w.imag
        return y

    for b in range(c["B"]):
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        rows = slice(cu[b], cu[b + 1])
        keys = range(lens[b] - n, lens[b])
        pos = (torch.tensor(list(keys), device="cuda") if s["positions"] is None else s["positions"][rows].long())
        q_out[rows] = turn(s["q"][rows].double(), pos)
        k, v = turn(s["k"][rows].double(), pos), s["v"][rows].double()
        done = 0
        while done < n:
            key = keys[done]
            take = min(n - done, page - key % page)
            where = (table[b][key // page], slice(key % page, key % page + take))
            kp[where], vp[where] = k[done:done + take], v[done:done + take]
            done += take
    return q_out, kp, vp


def _exact_rows(q, k, v, seen, scale):
    """q [R, Hkv, g, D], k and v [L, Hkv, D], seen [R, L]."""
    x = torch.einsum("rhgd,nhd->hgrn", q, k) * scale
    x.masked_fill_(~seen, -math.inf)
    z = torch.logsumexp(x, -1)
    p = torch.exp(x - torch.where(z > -math.inf, z, 0.0)[..., None])
    o = torch.einsum("hgrn,nhd->rhgd", p, v)
    return o.flatten(1, 2), z.flatten(0, 1)


def _exact_decode(c, s):
    B, sq, Hq, Hkv, D, page = c["B"], c["sq"], c["Hq"], c["Hkv"], c["D"], c["page"]
    lens = s["lens"].tolist()
    o = torch.zeros((B, sq, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, sq), -math.inf, dtype=torch.float64, device="cuda")
    words = s["mask"].cpu().numpy().view(np.uint32) if c["op"] == "tree" else None
    for b in range(B):
        n = lens[b]
        if n == 0:
            continue
        pages = s["table"][b, :-(-n // page)].long()
        k, v = (s[x][pages].double().flatten(0, 1)[:n] for x in ("k_pages", "v_pages"))
        seen = torch.zeros((sq, n), dtype=torch.bool, device="cuda")
        for t in range(sq):
            last = n - sq + t
            if c["op"] == "step":
                if last >= 0:
                    seen[t, :min(c["sinks"], last + 1)] = True
                    seen[t, max(0, last - c["window"]):last + 1] = True
            else:
                seen[t, :max(0, n - sq)] = True
                for u in range(sq):
                    if int(words[b, t, u // 32]) >> (u % 32) & 1 and n - sq + u >= 0:
                        seen[t, n - sq + u] = True
        q = s["q"][b].double().view(sq, Hkv, Hq // Hkv, D)
        some = seen.any(0)                              # keys that no token sees need no products
        o[b], lse[b] = _exact_rows(q, k[some], v[some], seen[:, some], s["scale"])
    return o, lse


def _exact_prompt(c, s):
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    o = torch.zeros(s["o"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        if c["packed"]:
            q0, q1 = s["cu_q"][b:b + 2].tolist()
            k0, k1 = s["cu_k"][b:b + 2].tolist()
            q, k, v, ob, lb = s["q"][q0:q1], s["k"][k0:k1], s["v"][k0:k1], o[q0:q1], lse[:, q0:q1]
        else:
            q, k, v, ob, lb = s["q"][b], s["k"][b], s["v"][b], o[b], lse[b]
        nq, nk = q.shape[0], k.shape[0]
        k, v = k.double(), v.double()
        for i in range(0, nq, 256):                     # rows i .. i + n - 1 and the keys that they see
            n = min(256, nq - i)
            last = torch.arange(i, i + n, device="cuda") + nk - nq
            j = torch.arange(nk, device="cuda")
            seen = (j <= last[:, None]) & ((last[:, None] - j <= c["window"]) | (j < c["sinks"]))
            some = seen.any(0)
            if not some.any():
                continue
            ob[i:i + n], lb[:, i:i + n] = _exact_rows(q[i:i + n].double().view(n, Hkv, Hq // Hkv, D), k[some], v[some],
                                                      seen[:, some], s["scale"])
    return o, lse


def _step_keys(c, n, tokens):
    """Of a sequence of n keys: (those that some token sees, the (token, key) pairs that see one another)."""
    first = max(0, n - tokens - c["window"])
    keys = n - first + min(c["sinks"], first)
    pairs = 0
    for last in {max(n - tokens, 0), max(n - 1, 0)} if n else ():
        lo = max(0, last - c["window"])
        pairs += last + 1 - lo + min(c["sinks"], lo)
    return keys, pairs * tokens // (2 if n and tokens > 1 and n > tokens else 1)


def work(case):
    c = case
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    if c["op"] == "append":
        total = sum(_spread(c))
        return {"bytes": total * (Hq + 2 * Hkv) * D * 4 + min(total, c["hi"] + c["past"]) * c["rot"] * 4
                + (4 * total if c["explicit"] else 0) + 4 * c["B"],
                "flops": total * (Hq + Hkv) * c["rot"] * 3}
    if c["op"] == "prompt":
        rows = _packed(c) if c["packed"] else [(c["Sq"], c["Sk"])] * c["B"]
        keys = pairs = 0
        for nq, nk in rows:
            first = max(0, nk - nq - c["window"])
            keys += nk - first + min(c["sinks"], first)
            i = np.arange(max(0, nk - nq), nk)
            lo = np.maximum(0, i - c["window"])
            pairs += int((i + 1 - lo + np.minimum(c["sinks"], lo)).sum())
        nq = sum(x for x, _ in rows)
        return {"bytes": nq * Hq * (4 * D + 4) + keys * Hkv * D * 4, "flops": 4 * pairs * Hq * D}
    B, sq = c["B"], c["sq"]
    keys = pairs = 0
    for n in _spread(c):
        if c["op"] == "step":
            k, p = _step_keys(c, n, sq)
        else:
            k, p = n, (n - sq) * sq + sq
        keys, pairs = keys + k, pairs + p
    return {"bytes": keys * Hkv * D * 4 + B * sq * Hq * (4 * D + 4) + 4 * (keys // c["page"] + B),
            "flops": 4 * pairs * Hq * D}
