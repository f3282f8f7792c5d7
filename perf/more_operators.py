"""What the operators around a growing cache are measured on, all of one attention layer with head dimension 128:

  grow     block tables extended and a slot map made on the GPU from the requests' lengths, and the new
           tokens' K and V written to bf16 pages through the slot map
  cache8   new tokens stored in an 8-bit cache with one scale for each block and KV head (INT8 or E4M3), and
           the requests' rows read back in bf16, as the attention of a prompt behind them takes them
  decode8  attention of one new token per request over such a cache
  window   attention that sees the last `window` tokens and the first `sinks` ones: prompts over packed rows
           or bf16 pages, decode steps over bf16 pages, the segment-quantised INT8 cache or an 8-bit block cache

`run` computes each in its plain form (elementary torch operations in 32 bits, rounded once) or, where
`own` is true, through the framework's calls.

The 8-bit block cache: a block of `block` tokens of one KV head has one scale s, the smallest bf16 number
not below amax / 127 (INT8) or amax / 448 (E4M3), amax being the largest |x| of the block's tokens (0 where
that is below 2^-80); a value is stored as x / s rounded to the nearest whole number (as the byte 128 + it)
or E4M3 number, ties to even.  A token that joins a partly filled block makes the scale grow where its
values need it, and the codes that are there are then rounded anew from the values that they stood for.
"""
import numpy as np
import torch

own = False

D = 128
DEV = "cuda"
TOP = {"int8": 127.0, "e4m3": 448.0}


# ---- cases ------------------------------------------------------------------------------------------

def listed():
    return [
        # the step of a small batch: one token each, latency of the smallest calls
        dict(name="grow-step-tiny", op="grow", batch=2, past_lo=37, past_hi=300, new_lo=1, new_hi=1, hkv=2, block=16),
        # chunks of a prefill batch behind earlier ones: 64 requests, up to 2048 new tokens each
        dict(name="grow-chunks-64", op="grow", batch=64, past_lo=0, past_hi=2048, new_lo=64, new_hi=2048, hkv=8,
             block=64),
        # two short requests, a few new tokens that join partly filled blocks
        dict(name="cache8-tiny-int8", op="cache8", fmt="int8", batch=2, past_lo=37, past_hi=300, new_lo=1, new_hi=40,
             hkv=2, block=16),
        # four chunks of 2048 tokens behind histories of up to 30720
        dict(name="cache8-chunks-e4m3", op="cache8", fmt="e4m3", batch=4, past_lo=100, past_hi=30720, new_lo=2048,
             new_hi=2048, hkv=8, block=64),
        # two short requests: latency of the smallest decode call
        dict(name="decode8-tiny-int8", op="decode8", fmt="int8", batch=2, lo=37, hi=300, hq=4, hkv=2, block=16),
        # 32 requests of 2048 tokens, blocks of 16
        dict(name="decode8-2048x32-int8", op="decode8", fmt="int8", batch=32, lo=2048, hi=2048, hq=32, hkv=8,
             block=16),
        # one request of 131072 tokens: the cache's length has to be split
        dict(name="decode8-131072-e4m3", op="decode8", fmt="e4m3", batch=1, lo=131072, hi=131072, hq=32, hkv=8,
             block=64),
        # two short prompts: latency of the smallest prompt call
        dict(name="window-prompt-tiny", op="window", source="packed", batch=2, q_lo=37, q_hi=300, past_lo=0,
             past_hi=0, window=64, sinks=4, hq=4, hkv=2, block=16),
        # one long prompt over bf16 pages of 64
        dict(name="window-prompt-16384-paged", op="window", source="paged", batch=1, q_lo=16384, q_hi=16384,
             past_lo=0, past_hi=0, window=4096, sinks=64, hq=32, hkv=8, block=64),
        # ragged prompts of a serving batch without shared KV heads, a short window
        dict(name="window-prompt-mha-ragged", op="window", source="packed", batch=16, q_lo=256, q_hi=2048, past_lo=0,
             past_hi=0, window=256, sinks=4, hq=32, hkv=32, block=16),
        # mixed serving over bf16 pages
        dict(name="window-decode-mixed-64", op="window", source="bf16", batch=64, lo=128, hi=32768, window=4096,
             sinks=16, hq=32, hkv=8, block=64),
        # long requests in the segment-quantised INT8 cache
        dict(name="window-decode-int8-32", op="window", source="dgq", batch=32, lo=32768, hi=32768, window=8192,
             sinks=128, hq=32, hkv=8, block=16),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["grow", "cache8", "decode8", "window", "window"])
    hkv = rng.choice([1, 2, 3, 4, 8, 16, 32])
    group = rng.choice([g for g in (1, 2, 4, 8) if g * hkv <= 64])
    block = rng.choice([16, 32, 64])
    if op in ("grow", "cache8"):
        new = _log(rng, 1, 4096)
        past = rng.choice([0, _log(rng, 1, 32768 if op == "cache8" else 2048)])
        c = dict(op=op, batch=_log(rng, 1, 256), past_lo=_log(rng, 1, past) if past else 0, past_hi=past,
                 new_lo=rng.choice([0, _log(rng, 1, new)]), new_hi=new, hkv=hkv, block=block)
        if op == "cache8":
            c["fmt"] = rng.choice(["int8", "e4m3"])
        while c["batch"] > 1 and work(c)["bytes"] > 3.0e8:
            c["batch"] = (c["batch"] + 1) // 2
        while work(c)["bytes"] > 3.0e8:
            c["new_hi"] = c["new_hi"] * 3 // 4
            c["past_hi"] = c["past_hi"] * 3 // 4
            c["new_lo"], c["past_lo"] = min(c["new_lo"], c["new_hi"]), min(c["past_lo"], c["past_hi"])
        return c
    if op == "window" and rng.random() < 0.5:
        top = _log(rng, 1, 16384)
        past = rng.choice([0, 0, _log(rng, 1, 32768)])
        c = dict(op=op, source=rng.choice(["packed", "paged"]), batch=_log(rng, 1, 32), q_lo=_log(rng, 1, top),
                 q_hi=top, past_lo=_log(rng, 1, past) if past else 0, past_hi=past, window=_log(rng, 1, 8192),
                 sinks=rng.choice([0, 1, 4, _log(rng, 1, 512)]), hq=group * hkv, hkv=hkv, block=block)
        while c["batch"] > 1 and (work(c)["flops"] > 8e11 or work(c)["bytes"] > 8e8):
            c["batch"] = (c["batch"] + 1) // 2
        while work(c)["flops"] > 9e11 or work(c)["bytes"] > 8e8:
            c["q_hi"] = c["q_hi"] * 3 // 4
            c["q_lo"] = min(c["q_lo"], c["q_hi"])
        return c
    top = _log(rng, 1, 131072)
    c = dict(op=op, batch=_log(rng, 1, 128), lo=_log(rng, 1, top), hi=top, hq=group * hkv, hkv=hkv, block=block)
    if op == "decode8":
        c["fmt"] = rng.choice(["int8", "e4m3"])
    else:
        c.update(source=rng.choice(["bf16", "dgq", "int8", "e4m3"]), window=_log(rng, 1, 16384),
                 sinks=rng.choice([0, 1, 4, _log(rng, 1, 512)]))
    # (what a windowed step does not see is there all the same)
    size = lambda: max(work(c)["bytes"], sum(_lens(c)) * c["hkv"] * 64)
    while c["batch"] > 1 and size() > 2.6e8:
        c["batch"] = (c["batch"] + 1) // 2
    while size() > 2.6e8:
        c["hi"] = c["hi"] * 3 // 4
        c["lo"] = min(c["lo"], c["hi"])
    return c


def _spread(lo, hi, n):
    """n whole numbers spread over the logarithm of [lo, hi], in an order that is not sorted."""
    if n == 1 or lo == hi:
        return [hi] * n
    lo1 = max(lo, 1)
    vals = [int(round(lo1 * (hi / lo1) ** (i / (n - 1)))) for i in range(n)]
    vals[0] = lo
    step = next(s for s in range(n // 2 + 1, 2 * n + 1) if np.gcd(s, n) == 1)
    return [vals[(i * step + n // 2) % n] for i in range(n)]


def _lens(c):
    return _spread(c["lo"], c["hi"], c["batch"])


def _grown(c):
    """Tokens there and new ones of every request."""
    return _spread(c["past_lo"], c["past_hi"], c["batch"])[::-1], _spread(c["new_lo"], c["new_hi"], c["batch"])


def _prompt_lens(c):
    q = _spread(c["q_lo"], c["q_hi"], c["batch"])
    past = _spread(c["past_lo"], c["past_hi"], c["batch"])[::-1]
    return q, [a + b for a, b in zip(q, past)]


def _seen_pairs(n, m, window, sinks):
    """(query, key) pairs of n queries at the end of m keys, and the keys that any of them sees."""
    p = np.arange(m - n, m, dtype=np.int64)
    first = np.maximum(p + 1 - window, 0)
    pairs = int((p + 1 - first + np.minimum(first, sinks)).sum())
    low = max(m - n + 1 - window, 0)
    return pairs, m - low + min(low, sinks)


def work(case):
    c, row = case, 2 * D
    if c["op"] == "grow":
        past, new = _grown(c)
        pages = sum(-(-(a + b) // c["block"]) - -(-a // c["block"]) for a, b in zip(past, new))
        # lengths read and written, ids read and named in the tables, slots; rows read and written
        return {"bytes": 4 * (4 * c["batch"] + 1 + 2 * pages + sum(new)) + 4 * row * sum(new) * c["hkv"], "flops": 0}
    if c["op"] == "cache8":
        past, new = _grown(c)
        blocks = sum(-(-(a + b) // c["block"]) for a, b in zip(past, new))
        # new rows read, their codes written; the old codes and the scales read; all rows written
        return {"bytes": 2 * c["hkv"] * (sum(new) * (row + D) + sum(past) * D + 4 * blocks + sum(past + new) * row),
                "flops": 0}
    if c["op"] == "decode8":
        lens = _lens(c)
        blocks = sum(-(-n // c["block"]) for n in lens)
        return {"bytes": 2 * D * sum(lens) * c["hkv"] + 8 * blocks * c["hkv"] + 2 * row * c["batch"] * (c["hq"] + c["hkv"]),
                "flops": 4 * D * c["hq"] * sum(n + 1 for n in lens)}
    if c["source"] in ("packed", "paged"):
        q, kv = _prompt_lens(c)
        seen = [_seen_pairs(n, m, c["window"], c["sinks"]) for n, m in zip(q, kv)]
        return {"bytes": 2 * row * (sum(q) * c["hq"] + sum(k for _, k in seen) * c["hkv"]),
                "flops": 4 * D * c["hq"] * sum(p for p, _ in seen)}
    keys = sum(_seen_pairs(1, n + 1, c["window"], c["sinks"])[0] - 1 for n in _lens(c))
    return {"bytes": (2 if c["source"] == "bf16" else 1) * 2 * D * keys * c["hkv"]
            + 2 * row * c["batch"] * (c["hq"] + c["hkv"]), "flops": 4 * D * c["hq"] * (keys + c["batch"])}


# ---- inputs -----------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _rows(g, n, heads):
    """bf16 rows [n, heads, 128] whose spread changes along the tokens (spans of 64) and heads, as the
    variance of a decoder's keys does."""
    sigma = torch.tensor([0.03, 0.15, 0.47, 1.5], device=DEV)
    spans = torch.randint(0, 4, ((n + 63) // 64, heads), generator=g, device=DEV)
    s = sigma[spans].repeat_interleave(64, dim=0)[:n]
    out = torch.empty(n, heads, D, dtype=torch.bfloat16, device=DEV)
    for i in range(0, n, 1 << 16):
        m = min(n, i + (1 << 16))
        out[i:m] = (torch.randn(m - i, heads, D, generator=g, device=DEV) * s[i:m, :, None]).to(torch.bfloat16)
    return out


def _new_rows(g, n, hkv):
    """K and V of n tokens as a fused projection leaves them: [n, K heads | V heads, 128]."""
    kv = _rows(g, n, 2 * hkv)
    return kv[:, :hkv], kv[:, hkv:]


def _tables(g, lens, block, spare):
    """A shuffled block table [batch, columns] of the requests' blocks, how many blocks there are, and the
    ids of the `spare` ones that no request has, in some order.  Unused entries are 0."""
    need = [(n + block - 1) // block for n in lens]
    total = sum(need) + spare
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    at = np.concatenate([[0], np.cumsum(need)])
    columns = max(1, max(need))
    i = torch.arange(columns, device=DEV)[None, :]
    first, count = torch.tensor(at[:-1], device=DEV)[:, None], torch.tensor(need, device=DEV)[:, None]
    table = torch.where(i < count, order[(first + i).clamp(max=total - 1)], 0).to(torch.int32)
    return table.contiguous(), total, order[int(at[-1]):].clone()


def _pages(g, total, hkv, block):
    return _rows(g, total * block, hkv).view(total, block, hkv, D).transpose(1, 2).contiguous()


def _codes(g, fmt, total, hkv, block):
    """Codes of normal values whose block scale is set by the largest of them, and the scales."""
    codes = torch.empty(total, hkv, block, D, dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 26) // (hkv * block * D))
    for i in range(0, total, step):
        n = min(total, i + step) - i
        x = torch.randn(n, hkv, block, D, generator=g, device=DEV)
        x = x * (TOP[fmt] / x.abs().amax(dim=(2, 3), keepdim=True))
        codes[i:i + n] = (x.round() + 128).to(torch.uint8) if fmt == "int8" else \
            x.to(torch.float8_e4m3fn).view(torch.uint8)
    sigma = torch.tensor([0.03, 0.15, 0.47, 1.5], device=DEV)
    s = sigma[torch.randint(0, 4, (total, hkv), generator=g, device=DEV)] * (4.0 / TOP[fmt])
    s = s * (1 + 0.3 * torch.rand(total, hkv, generator=g, device=DEV))
    return codes, s.to(torch.bfloat16).float()


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _cu(lens):
    return _ints([0] + [int(x) for x in np.cumsum(lens)])


def _segments(g, lens, hkv):
    """Segment records [batch, hkv, 32 words]: three segments that start at multiples of 16, each with the
    smallest value and the step of its codes."""
    words = torch.zeros(len(lens), hkv, 32, dtype=torch.int32, device=DEV)
    n = _ints(lens)[:, None].expand(len(lens), hkv)
    words[..., 0] = torch.where(n > 32, 3, torch.where(n > 16, 2, 1)) * (n > 0)
    words[..., 1] = n
    cuts = torch.rand(len(lens), hkv, 2, generator=g, device=DEV).sort(dim=-1).values
    a = (cuts[..., 0] * (n - 32).clamp(min=1)).int() // 16 * 16 + 16
    b = torch.maximum(a + 16, (cuts[..., 1] * n).int() // 16 * 16)
    words[..., 2:7] = n[..., None]
    words[..., 2] = 0
    words[..., 3] = torch.where(words[..., 0] > 1, a, n)
    words[..., 4] = torch.where(words[..., 0] > 2, b, n)
    sigma = torch.tensor([0.03, 0.15, 0.47, 1.5], device=DEV)
    f = words.view(torch.float32)
    live = torch.arange(5, device=DEV) < words[..., 0:1]
    for at in (7, 17):
        s = sigma[torch.randint(0, 4, (len(lens), hkv, 5), generator=g, device=DEV)]
        low = -s * (3.5 + torch.rand(len(lens), hkv, 5, generator=g, device=DEV))
        high = s * (3.5 + torch.rand(len(lens), hkv, 5, generator=g, device=DEV))
        f[..., at:at + 5] = torch.where(live, low, 0.0)
        f[..., at + 5:at + 10] = torch.where(live, (high - low) / 255, 0.0)
    return words


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c, "block": c["block"]}
    hkv, block = c["hkv"], c["block"]
    if c["op"] in ("grow", "cache8"):
        past, new = _grown(c)
        lens = [a + b for a, b in zip(past, new)]
        s.update(past=past, new=new, lens=lens, seq_lens=_ints(past), new_lens=_ints(new), cu_new=_cu(new))
        s["k"], s["v"] = _new_rows(g, sum(new), hkv)
        if c["op"] == "grow":
            need = sum(-(-n // block) for n in lens) - sum(-(-n // block) for n in past)
            s["table"], s["total"], s["free_ids"] = _tables(g, past, block, need + 5)
            columns = max(1, max(-(-n // block) for n in lens))
            s["table"] = torch.nn.functional.pad(s["table"], (0, columns - s["table"].shape[1])).contiguous()
            s["used"] = _ints([3])
            s["slots"] = torch.empty(sum(new), dtype=torch.int32, device=DEV)
            s["cu_out"], s["lens_out"], s["used_out"] = torch.empty_like(s["cu_new"]), _ints(past), _ints([0])
            s["k_pages"], s["v_pages"] = _pages(g, s["total"], hkv, block), _pages(g, s["total"], hkv, block)
        else:
            s["table"], s["total"], _ = _tables(g, lens, block, 3)
            s["k_codes"], s["k_scales"] = _codes(g, c["fmt"], s["total"], hkv, block)
            s["v_codes"], s["v_scales"] = _codes(g, c["fmt"], s["total"], hkv, block)
            s["cu"] = _cu(lens)
            # the slot map that the step's table update left: block and place of every new token
            t = torch.tensor([a + i for a, n in zip(past, new) for i in range(n)], device=DEV)
            b = torch.tensor([b for b, n in enumerate(new) for _ in range(n)], device=DEV)
            s["slots"] = (s["table"][b, t // block] * block + t % block).to(torch.int32)
            s["k_rows"] = torch.empty(sum(lens), hkv, D, dtype=torch.bfloat16, device=DEV)
            s["v_rows"] = torch.empty_like(s["k_rows"])
    elif c["op"] == "window" and c["source"] in ("packed", "paged"):
        q, kv = _prompt_lens(c)
        s.update(q_lens=q, kv_lens=kv, cu_q=_cu(q), cu_kv=_cu(kv))
        s["q"] = torch.randn(sum(q), c["hq"], D, generator=g, device=DEV).to(torch.bfloat16)
        if c["source"] == "packed":
            s["k"], s["v"] = _rows(g, sum(kv), hkv), _rows(g, sum(kv), hkv)
        else:
            s["table"], total, _ = _tables(g, kv, block, 3)
            s["k"], s["v"] = _pages(g, total, hkv, block), _pages(g, total, hkv, block)
            s["seq_lens"] = _ints(kv)
        s["out"] = torch.zeros_like(s["q"])
    else:
        lens = _lens(c)
        s.update(lens=lens, max_seqlen=max(lens), seq_lens=_ints(lens))
        s["table"], total, _ = _tables(g, lens, block, 3)
        source = c.get("fmt") or c["source"]
        if source == "bf16":
            s["k"], s["v"] = _pages(g, total, hkv, block), _pages(g, total, hkv, block)
        elif source == "dgq":
            shape = (total, hkv, block, D)
            s["k"] = torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8)
            s["v"] = torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8)
            s["records"] = _segments(g, lens, hkv)
        else:
            s["k"], s["k_scales"] = _codes(g, source, total, hkv, block)
            s["v"], s["v_scales"] = _codes(g, source, total, hkv, block)
        s["q"] = torch.randn(c["batch"], c["hq"], D, generator=g, device=DEV).to(torch.bfloat16)
        s["k_new"], s["v_new"] = _rows(g, c["batch"], hkv), _rows(g, c["batch"], hkv)
        s["out"] = torch.zeros_like(s["q"])
    if own:
        import int8_group_quantized_gb300 as dgq
        if c["op"] == "grow":
            size = dgq.dgq_extend_tables_workspace_size()
        elif c["op"] == "cache8":
            size = dgq.dgq_block8_workspace_size()
        elif "q_lens" in s:
            size = dgq.dgq_prompt_attn_workspace_size(c["batch"], c["hq"], hkv)
        else:
            size = dgq.dgq_attn_workspace_size(c["batch"], c["hq"], hkv, s["max_seqlen"])
        s["workspace"] = torch.zeros(size, dtype=torch.uint8, device=DEV)
    return s


# ---- one pass ---------------------------------------------------------------------------------------

def run(state):
    s, c = state, state["case"]
    op, source = c["op"], c.get("source")
    if not own:
        if op == "grow":
            return _plain_grow(s)
        if op == "cache8":
            return _plain_cache8(s)
        return _plain_prompt(s) if source in ("packed", "paged") else _plain_decode(s)
    import int8_group_quantized_gb300 as dgq
    if op == "grow":
        dgq.dgq_extend_tables(s["seq_lens"], s["new_lens"], s["block"], s["total"], s["free_ids"], s["used"], s["table"],
                              s["slots"], s["cu_out"], s["lens_out"], s["used_out"], s["workspace"])
        dgq.dgq_write_slots(s["k"], s["v"], s["slots"], s["k_pages"], s["v_pages"], s["workspace"])
        return [s["table"], s["slots"], s["cu_out"], s["lens_out"], s["used_out"], s["k_pages"], s["v_pages"]]
    if op == "cache8":
        dgq.dgq_store_block8(c["fmt"], s["k"], s["v"], s["slots"], s["k_codes"], s["v_codes"], s["k_scales"],
                             s["v_scales"], s["workspace"])
        dgq.dgq_load_block8(c["fmt"], s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"], s["table"], s["cu"],
                            s["k_rows"], s["v_rows"], s["workspace"])
        return [s["k_rows"], s["v_rows"], s["k_scales"], s["v_scales"]]
    limits = dict(window=c["window"], sinks=c["sinks"]) if op == "window" else {}
    if source == "packed":
        dgq.dgq_prompt_attn(s["q"], s["k"], s["v"], s["cu_q"], s["cu_kv"], s["out"], s["workspace"], **limits)
    elif source == "paged":
        dgq.dgq_prompt_attn_paged(s["q"], s["cu_q"], s["k"], s["v"], s["table"], s["seq_lens"], s["out"], s["workspace"],
                                  **limits)
    elif source == "bf16":
        dgq.dgq_paged_decode_attn_bf16(s["q"], s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["seq_lens"],
                                       s["max_seqlen"], s["out"], s["workspace"], **limits)
    elif source == "dgq":
        dgq.dgq_paged_decode_attn(s["q"], s["k_new"], s["v_new"], s["k"], s["v"], s["records"], s["table"],
                                  s["seq_lens"], s["max_seqlen"], s["out"], s["workspace"], **limits)
    else:
        dgq.dgq_paged_decode_attn_block8(c.get("fmt") or source, s["q"], s["k_new"], s["v_new"], s["k"], s["v"],
                                         s["k_scales"], s["v_scales"], s["table"], s["seq_lens"], s["max_seqlen"],
                                         s["out"], s["workspace"], **limits)
    return s["out"]


def _of(counts, total):
    """For `total` items, counts[b] of them of request b: the request of each, and its place among them."""
    b = torch.repeat_interleave(torch.arange(counts.numel(), device=DEV), counts, output_size=total)
    return b, torch.arange(total, device=DEV) - (counts.cumsum(0) - counts)[b]


def _plain_grow(s):
    block, table = s["block"], s["table"]
    past, new = s["seq_lens"].long(), s["new_lens"].long()
    had = (past + block - 1) // block
    need = (past + new + block - 1) // block - had
    b, i = _of(need, s["total"] - int(sum(-(-n // block) for n in s["past"])) - 5)
    at = s["used"].long() + (need.cumsum(0) - need)[b] + i
    table[b, had[b] + i] = s["free_ids"][at]
    b, i = _of(new, sum(s["new"]))
    position = past[b] + i
    page = table[b, position // block].long()
    slot = position % block
    s["slots"].copy_(page * block + slot)
    s["k_pages"][page, :, slot] = s["k"]
    s["v_pages"][page, :, slot] = s["v"]
    cu = torch.nn.functional.pad(new.cumsum(0), (1, 0)).to(torch.int32)
    return [table, s["slots"], cu, (past + new).to(torch.int32), s["used"] + need.sum().to(torch.int32), s["k_pages"],
            s["v_pages"]]


def _values(codes, scale, fmt):
    x = codes.float() - 128.0 if fmt == "int8" else codes.view(torch.float8_e4m3fn).float()
    return x * scale


def _needed_scale(amax, fmt):
    """The smallest bf16 number not below amax / 127 or amax / 448."""
    t = amax.double() / TOP[fmt]
    s = t.to(torch.bfloat16)
    above = (s.view(torch.int16) + 1).view(torch.bfloat16)
    return torch.where(amax < 2.0 ** -80, 0.0, torch.where(s.double() < t, above, s).float())


def _encoded(x, scale, fmt):
    y = torch.where(scale > 0, x / torch.where(scale > 0, scale, 1.0), 0.0)
    return (y.round() + 128.0).to(torch.uint8) if fmt == "int8" else y.to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_cache8(s):
    c, block, fmt = s["case"], s["block"], s["case"]["fmt"]
    past, new, cu = s["seq_lens"].long(), s["new_lens"].long(), s["cu_new"].long()
    count = torch.where(new > 0, (past + new + block - 1) // block - past // block, 0)
    b, i = _of(count, sum(-(-(a + n) // block) - a // block for a, n in zip(s["past"], s["new"]) if n))
    column = past[b] // block + i
    page = s["table"][b, column].long()
    t = column[:, None] * block + torch.arange(block, device=DEV)
    old, fresh = t < past[b][:, None], (t >= past[b][:, None]) & (t < (past + new)[b][:, None])
    row = (cu[b] - past[b])[:, None] + t
    for x, codes, scales in ((s["k"], s["k_codes"], s["k_scales"]), (s["v"], s["v_codes"], s["v_scales"])):
        if not b.numel():
            continue
        v = x[row.clamp(0, x.shape[0] - 1)].float().transpose(1, 2)              # [blocks, hkv, tokens, 128]
        fresh_, old_ = fresh[:, None, :, None], old[:, None, :, None]
        needed = _needed_scale(torch.where(fresh_, v.abs(), 0.0).amax(dim=(2, 3)), fmt)
        had = torch.where(old.any(dim=1)[:, None], scales[page], 0.0)
        scale = torch.maximum(needed, had)
        there = codes[page]
        again = _encoded(_values(there, had[..., None, None], fmt), scale[..., None, None], fmt)
        again = torch.where((scale > had)[..., None, None], again, there)
        codes[page] = torch.where(fresh_, _encoded(v, scale[..., None, None], fmt), torch.where(old_, again, there))
        scales[page] = scale
    b, t = _of(past + new, sum(s["lens"]))
    page = s["table"][b, t // block].long()
    out = [_values(codes[page, :, t % block], scales[page][..., None], fmt).to(torch.bfloat16)
           for codes, scales in ((s["k_codes"], s["k_scales"]), (s["v_codes"], s["v_scales"]))]
    return out + [s["k_scales"], s["v_scales"]]


def _softmax_mean(z, seen, v):
    """Weights of the scores z [..., rows, keys] over the keys that are seen, times v; zeros for a row that sees none."""
    z = z.masked_fill(~seen, float("-inf"))
    top = z.amax(dim=-1, keepdim=True)
    w = torch.exp(z - torch.where(torch.isinf(top), 0.0, top))
    total = w.sum(dim=-1, keepdim=True)
    return torch.matmul(w / torch.where(total > 0, total, 1.0), v)


def _plain_prompt(s):
    """Blocks of 128 query rows, each with the sinks and the window of keys that its rows can see."""
    c = s["case"]
    hq, hkv, group, rows = c["hq"], c["hkv"], c["hq"] // c["hkv"], 128
    window, sinks = min(c["window"], max(s["kv_lens"])), min(c["sinks"], max(s["kv_lens"]))
    n, m = _ints(s["q_lens"]).long(), _ints(s["kv_lens"]).long()
    b, i = _of((n + rows - 1) // rows, sum(-(-x // rows) for x in s["q_lens"]))
    out = torch.zeros_like(s["q"])
    keys = sinks + window + rows - 1
    step = max(1, (1 << 29) // (keys * (hq * rows + 4 * hkv * D)))
    for at in range(0, b.numel(), step):
        bb, first = b[at:at + step], i[at:at + step] * rows
        row = first[:, None] + torch.arange(rows, device=DEV)
        p = (m - n)[bb][:, None] + row                                           # positions of the rows
        t = torch.cat([torch.arange(sinks, device=DEV).expand(bb.numel(), sinks),
                       p[:, :1] + 1 - window + torch.arange(window + rows - 1, device=DEV)], dim=1)
        is_sink = torch.arange(keys, device=DEV) < sinks
        seen = (t[:, None, :] <= p[..., None]) & (is_sink | ((t[:, None, :] > p[..., None] - window) & (t[:, None, :] >= sinks)))
        at_key = torch.minimum(t.clamp(min=0), (m[bb] - 1).clamp(min=0)[:, None])
        k, v = (_prompt_keys(s, x, bb, at_key) for x in (s["k"], s["v"]))       # [blocks, hkv, keys, 128]
        live = row < n[bb][:, None]
        at_row = s["cu_q"].long()[bb][:, None] + torch.where(live, row, 0)
        q = s["q"][at_row].float().view(bb.numel(), rows, hkv, group, D) * D ** -0.5
        q = q.permute(0, 2, 3, 1, 4).reshape(bb.numel(), hkv, group * rows, D)
        z = torch.matmul(q, k.transpose(2, 3)).view(bb.numel(), hkv, group, rows, keys)
        y = _softmax_mean(z, seen[:, None, None], v[:, :, None]).permute(0, 3, 1, 2, 4).reshape(bb.numel(), rows, hq, D)
        out[at_row[live]] = y[live].to(torch.bfloat16)
    return out


def _prompt_keys(s, x, b, t):
    if s["case"]["source"] == "packed":
        return x[(s["cu_kv"].long()[b][:, None] + t).clamp(max=x.shape[0] - 1)].float().transpose(1, 2)
    return x[s["table"][b[:, None], t // s["block"]].long(), :, t % s["block"]].float().transpose(1, 2)


def _cached(s, source, b, t, which):
    """Rows of the tokens t [requests, keys] of the requests b in 32 bits, [requests, hkv, keys, 128]."""
    block = s["block"]
    page = s["table"][b[:, None], t // block].long()
    x = s[which][page, :, t % block]
    if source == "bf16":
        return x.float().transpose(1, 2)
    if source != "dgq":
        return _values(x, s[which + "_scales"][page][..., None], source).transpose(1, 2)
    words = s["records"][b]
    seg = (t[:, None, :, None] >= words[:, :, None, 3:7]).sum(dim=-1)             # [requests, hkv, keys]
    low, step = (words.view(torch.float32)[..., at:at + 5].gather(2, seg) for at in ((7, 12) if which == "k" else (17, 22)))
    return x.float().transpose(1, 2) * step[..., None] + low[..., None]


def _plain_decode(s):
    """The sinks and the window (or all tokens) of every request, padded to the longest, and its new token."""
    c = s["case"]
    hkv, group = c["hkv"], c["hq"] // c["hkv"]
    source = c.get("fmt") or c["source"]
    longest = max(s["lens"])
    window, sinks = (min(c["window"] - 1, longest), min(c["sinks"], longest)) if c["op"] == "window" else (longest, 0)
    out = torch.empty_like(s["q"])
    step = max(1, (1 << 31) // (hkv * D * (sinks + window + 1)))
    for at in range(0, c["batch"], step):
        b = torch.arange(at, min(c["batch"], at + step), device=DEV)
        n = s["seq_lens"][b].long()[:, None]
        t = torch.cat([torch.arange(sinks, device=DEV).expand(b.numel(), sinks),
                       n - window + torch.arange(window, device=DEV)], dim=1)
        seen = torch.where(torch.arange(sinks + window, device=DEV) < sinks, t < n, t >= sinks)
        t = torch.minimum(t.clamp(min=0), (n - 1).clamp(min=0))
        k = torch.cat([_cached(s, source, b, t, "k"), s["k_new"][b].float()[:, :, None]], dim=2)
        v = torch.cat([_cached(s, source, b, t, "v"), s["v_new"][b].float()[:, :, None]], dim=2)
        seen = torch.nn.functional.pad(seen, (0, 1), value=True)
        q = s["q"][b].float().view(b.numel(), hkv, group, D) * D ** -0.5
        y = _softmax_mean(torch.matmul(q, k.transpose(2, 3)), seen[:, None, None], v)
        out[b] = y.reshape(b.numel(), c["hq"], D).to(torch.bfloat16)
    return out


# ---- the definition in 64 bits ----------------------------------------------------------------------

def _exact_rows(x, scale, fmt):
    """Codes as the numbers that they stand for in float64: the bits of an E4M3 number read by hand."""
    c = x.long()
    if fmt == "int8":
        return (c - 128).double() * scale
    e, f = (c >> 3) & 15, (c & 7).double()
    y = torch.where(e > 0, (1 + f / 8) * torch.exp2((e - 7).double()), f / 8 * 2.0 ** -6)
    return torch.where(c > 127, -y, y) * scale


def _exact_rounded(x, s, fmt):
    """x / s (numpy, float64) rounded to the nearest whole or E4M3 number, ties to even, as a number."""
    y = x / s if s > 0 else np.zeros_like(x)
    if fmt == "int8":
        return np.rint(y)
    e = np.maximum(np.frexp(y)[1] - 1, -6)
    unit = np.ldexp(1.0, e - 3)
    return np.rint(y / unit) * unit


def _exact_scale(top, fmt):
    if top < 2.0 ** -80:
        return 0.0
    t = float(top) / TOP[fmt]
    unit = 2.0 ** (int(np.frexp(t)[1]) - 8)
    return float(np.ceil(t / unit) * unit)


def _exact_cache8(s):
    c, block, fmt = s["case"], s["block"], s["case"]["fmt"]
    scales = [s["k_scales"].double().cpu().numpy().copy(), s["v_scales"].double().cpu().numpy().copy()]
    table, rows = s["table"].cpu().numpy(), [[], []]
    at = 0
    for b, (a, n) in enumerate(zip(s["past"], s["new"])):
        t = torch.arange(a + n, device=DEV)
        page = s["table"][b].long()[t // block]
        for w, (x, codes) in enumerate(((s["k"], s["k_codes"]), (s["v"], s["v_codes"]))):
            sc = torch.from_numpy(scales[w]).to(DEV)[page][..., None]
            y = _exact_rows(codes[page, :, t % block], sc, fmt).cpu().numpy()
            fresh = x[at:at + n].double().cpu().numpy()
            for first in range(a // block * block, a + n, block) if n else ():
                lo, hi = max(first, a), min(first + block, a + n)
                for h in range(c["hkv"]):
                    new = fresh[lo - a:hi - a, h]
                    had = scales[w][table[b, first // block], h] if first < a else 0.0
                    scale = max(had, _exact_scale(np.abs(new).max(), fmt))
                    if scale > had and first < a:
                        y[first:a, h] = _exact_rounded(y[first:a, h], scale, fmt) * scale
                    y[lo:hi, h] = _exact_rounded(new, scale, fmt) * scale
                    scales[w][table[b, first // block], h] = scale
            rows[w].append(torch.from_numpy(y))
        at += n
    return [torch.cat(rows[0]).to(DEV), torch.cat(rows[1]).to(DEV)] + [torch.from_numpy(x).to(DEV) for x in scales]


def exact(case, seed):
    """out[i, h] = sum_t w_t v_t / sum_t w_t with w_t = exp(q_i . k_t / sqrt(128)) over the keys t <= p with
    t > p - window or t < sinks (p: the row's position), head by head in float64; cached rows as the numbers
    that their codes stand for.  Tables, slots and copied rows are whole numbers or copies: no such value."""
    c = case
    if c["op"] == "grow":
        return None
    if c["op"] == "cache8":
        past, new = _grown(c)
        blocks = sum(-(-(a + n) // c["block"]) - a // c["block"] for a, n in zip(past, new) if n)
        if blocks * c["hkv"] > 20000 or sum(past + new) * c["hkv"] * D > 1.5e8:
            return None
        return _exact_cache8(prepare(c, seed))
    if work(c)["flops"] > 2e12:
        return None
    s = prepare(c, seed)
    group, block = c["hq"] // c["hkv"], c["block"]
    source = c.get("fmt") or c["source"]
    window, sinks = (c["window"], c["sinks"]) if c["op"] == "window" else (1 << 40, 0)
    decode = "k_new" in s
    queries, keys = ([1] * c["batch"], s["lens"]) if decode else (s["q_lens"], s["kv_lens"])
    out = torch.zeros(sum(queries), c["hq"], D, dtype=torch.float64, device=DEV)
    row = base = 0
    for b in range(c["batch"]):
        n, m = queries[b], keys[b]
        total = m + 1 if decode else m
        # keys that a row of this request can see
        low = min(max(total - n + 1 - window, sinks), m)
        t = torch.cat([torch.arange(min(sinks, low), device=DEV), torch.arange(low, m, device=DEV)]) if low > sinks \
            else torch.arange(m, device=DEV)
        for h in range(c["hkv"]):
            kv = []
            for which in ("k", "v"):
                if source == "packed":
                    x = s[which][base + t, h].double()
                else:
                    page = s["table"][b].long()[t // block]
                    x = s[which][page, h, t % block]
                    if source in ("bf16", "paged"):
                        x = x.double()
                    elif source == "dgq":
                        f, w = s["records"].view(torch.float32)[b, h].double(), s["records"][b, h].tolist()
                        seg = torch.bucketize(t, torch.tensor(w[3:2 + max(w[0], 1)], device=DEV), right=True)
                        at = 7 if which == "k" else 17
                        x = f[at + seg][:, None] + x.double() * f[at + 5 + seg][:, None]
                    else:
                        x = _exact_rows(x, s[which + "_scales"][page, h].double()[:, None], source)
                kv.append(torch.cat([x, s[which + "_new"][b, h][None].double()]) if decode else x)
            k, v = kv
            at_key = torch.cat([t, torch.tensor([m], device=DEV)]) if decode else t
            for i in range(0, n, 1024):
                e = min(n, i + 1024)
                p = torch.arange(total - n + i, total - n + e, device=DEV)[:, None]
                lo = int(torch.searchsorted(at_key, max(total - n + i + 1 - window, sinks)))  # keys before: sinks, or unseen
                hi = int(torch.searchsorted(at_key, total - n + e))
                first = int(torch.searchsorted(at_key, sinks))
                part = torch.cat([torch.arange(min(first, lo, hi), device=DEV), torch.arange(min(lo, hi), hi, device=DEV)])
                tt = at_key[part][None, :]
                seen = (tt <= p) & ((tt > p - window) | (tt < sinks))
                for j in range(h * group, (h + 1) * group):
                    x = s["q"][row + i:row + e, j].double() @ k[part].T / np.sqrt(float(D))
                    x = torch.where(seen, x, -torch.inf)
                    if x.shape[1] == 0:
                        continue
                    top = x.max(dim=1, keepdim=True).values
                    w = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
                    l = w.sum(dim=1, keepdim=True)
                    out[row + i:row + e, j] = (w @ v[part]) / torch.where(l > 0, l, 1.0)
        row += n
        base += m
    return out
