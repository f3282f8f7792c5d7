"""What the operators around the bf16 side of the cache are measured on.

Three families, all of one attention layer with head dimension 128:

  prompt   causal grouped-query attention of a prompt (or of a chunk of it behind a history), K and V
           as packed rows or in a bf16 paged cache
  decode   attention of one new token per request over a bf16 paged cache, plus the token's own K and V
  pages    pages of a paged cache copied (a fork's last page with the segment records; a compaction with
           its block tables rewritten)

`run` computes each in its plain form (elementary torch operations in 32 bits, rounded once) or, where
`own` is true, through the framework's calls.
"""
import numpy as np
import torch

own = False

D = 128
DEV = "cuda"


# ---- cases ------------------------------------------------------------------------------------------

def listed():
    return [
        # two short requests, two query heads to a KV head: latency of the smallest prompt call
        dict(name="prompt-tiny", op="prompt", source="packed", batch=2, q_lo=37, q_hi=300, past_lo=0, past_hi=0,
             hq=4, hkv=2, block=16),
        # a prefill batch of equal prompts, 32 query and 8 KV heads
        dict(name="prompt-2048x8", op="prompt", source="packed", batch=8, q_lo=2048, q_hi=2048, past_lo=0,
             past_hi=0, hq=32, hkv=8, block=16),
        # ragged prompts of a serving batch without shared KV heads
        dict(name="prompt-mha-ragged", op="prompt", source="packed", batch=16, q_lo=256, q_hi=2048, past_lo=0,
             past_hi=0, hq=32, hkv=32, block=16),
        # one long prompt, its K and V already in bf16 pages of 64
        dict(name="prompt-16384-paged", op="prompt", source="paged", batch=1, q_lo=16384, q_hi=16384, past_lo=0,
             past_hi=0, hq=32, hkv=8, block=64),
        # short turns behind long histories (a follow-up question, a verified draft): few rows, long axis
        dict(name="prompt-turns-paged", op="prompt", source="paged", batch=16, q_lo=1, q_hi=64, past_lo=128,
             past_hi=32768, hq=32, hkv=8, block=64),
        # two short requests: latency of the smallest decode call
        dict(name="decode-tiny", op="decode", batch=2, lo=37, hi=300, hq=4, hkv=2, block=16),
        # 32 requests of 2048 tokens, pages of 16
        dict(name="decode-2048x32", op="decode", batch=32, lo=2048, hi=2048, hq=32, hkv=8, block=16),
        # one request of 131072 tokens: the cache's length has to be split
        dict(name="decode-131072", op="decode", batch=1, lo=131072, hi=131072, hq=32, hkv=8, block=64),
        # mixed serving: lengths spread over the whole range
        dict(name="decode-mixed-64", op="decode", batch=64, lo=128, hi=32768, hq=32, hkv=8, block=64),
        # one request of a small model forked: its last page and its records
        dict(name="pages-fork-tiny", op="pages", kind="fork", layers=1, pages=32, moves=1, hkv=2, block=16,
             rows=4, columns=8),
        # 32 forks (parallel samples) over 32 layers: 32 last pages of 64 pools, and the records
        dict(name="pages-fork-32", op="pages", kind="fork", layers=32, pages=256, moves=32, hkv=8, block=16,
             rows=64, columns=128),
        # a fragmented pool drawn together: 400 of 1024 pages of 64 tokens move, tables rewritten
        dict(name="pages-compact-1024", op="pages", kind="compact", layers=4, pages=1024, moves=400, hkv=8,
             block=64, rows=64, columns=512),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "decode", "decode", "pages"])
    hkv = rng.choice([1, 2, 3, 4, 8, 16, 32])
    group = rng.choice([g for g in (1, 2, 4, 8) if g * hkv <= 64])
    if op == "prompt":
        top = _log(rng, 1, 16384)
        past = rng.choice([0, 0, _log(rng, 1, 32768)])
        c = dict(op=op, source=rng.choice(["packed", "paged"]), batch=_log(rng, 1, 32), q_lo=_log(rng, 1, top),
                 q_hi=top, past_lo=_log(rng, 1, past) if past else 0, past_hi=past, hq=group * hkv, hkv=hkv,
                 block=rng.choice([16, 32, 64]))
        while c["batch"] > 1 and (work(c)["flops"] > 1.2e12 or work(c)["bytes"] > 1.5e9):
            c["batch"] = (c["batch"] + 1) // 2
        while work(c)["flops"] > 2.0e12 or work(c)["bytes"] > 1.5e9:
            c["q_hi"] = c["q_hi"] * 3 // 4
            c["q_lo"] = min(c["q_lo"], c["q_hi"])
        return c
    if op == "decode":
        top = _log(rng, 1, 131072)
        c = dict(op=op, batch=_log(rng, 1, 128), lo=_log(rng, 1, top), hi=top, hq=group * hkv, hkv=hkv,
                 block=rng.choice([16, 32, 64]))
        while c["batch"] > 1 and work(c)["bytes"] > 1.5e9:
            c["batch"] = (c["batch"] + 1) // 2
        while work(c)["bytes"] > 1.5e9:
            c["hi"] = c["hi"] * 3 // 4
            c["lo"] = min(c["lo"], c["hi"])
        return c
    pages = _log(rng, 8, 1024)
    c = dict(op=op, kind=rng.choice(["fork", "compact"]), layers=_log(rng, 1, 32), pages=pages,
             moves=_log(rng, 1, max(1, pages * 2 // 5)), hkv=hkv, block=rng.choice([16, 32, 64]),
             rows=_log(rng, 2, 128), columns=_log(rng, 1, 512))
    while c["layers"] > 1 and 2 * c["layers"] * pages * hkv * c["block"] * D > 5e8:
        c["layers"] = (c["layers"] + 1) // 2
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


def _prompt_lens(c):
    q = _spread(c["q_lo"], c["q_hi"], c["batch"])
    past = _spread(c["past_lo"], c["past_hi"], c["batch"])[::-1]
    return q, [a + b for a, b in zip(q, past)]


def work(case):
    c = case
    if c["op"] == "prompt":
        q, kv = _prompt_lens(c)
        pairs = sum(n * (m - n) + n * (n + 1) // 2 for n, m in zip(q, kv))
        return {"bytes": 4 * D * (sum(q) * c["hq"] + sum(kv) * c["hkv"]), "flops": 4 * D * c["hq"] * pairs}
    if c["op"] == "decode":
        lens = _spread(c["lo"], c["hi"], c["batch"])
        return {"bytes": 4 * D * (sum(lens) * c["hkv"] + c["batch"] * (c["hq"] + c["hkv"])),
                "flops": 4 * D * c["hq"] * sum(n + 1 for n in lens)}
    page = c["hkv"] * c["block"] * D
    total = 2 * 2 * c["layers"] * c["moves"] * page
    if c["kind"] == "fork":
        total += 2 * c["layers"] * _forked_rows(c) * c["hkv"] * 128
    else:
        total += 2 * 4 * c["rows"] * c["columns"]
    return {"bytes": total, "flops": 0}


def _forked_rows(c):
    return min(c["moves"], c["rows"] // 2)


# ---- inputs -----------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _kv_rows(g, n, hkv):
    """bf16 rows [n, hkv, 128] whose spread changes along the tokens (spans of 64) and heads, as the
    variance of a decoder's keys does."""
    sigma = torch.tensor([0.03, 0.15, 0.47, 1.5], device=DEV)
    spans = torch.randint(0, 4, ((n + 63) // 64, hkv), generator=g, device=DEV)
    s = sigma[spans].repeat_interleave(64, dim=0)[:n]
    out = torch.empty(n, hkv, D, dtype=torch.bfloat16, device=DEV)
    for i in range(0, n, 1 << 16):
        m = min(n, i + (1 << 16))
        out[i:m] = (torch.randn(m - i, hkv, D, generator=g, device=DEV) * s[i:m, :, None]).to(torch.bfloat16)
    return out


def _paged(g, lens, hkv, block):
    """K and V pages [n, hkv, block, 128] with a shuffled block table [batch, columns]; slots behind a
    request's end hold other values."""
    need = [(n + block - 1) // block for n in lens]
    total = sum(need) + 3
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32).cpu()
    table = torch.zeros(len(lens), max(1, max(need)), dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    k = _kv_rows(g, total * block, hkv).view(total, block, hkv, D).transpose(1, 2).contiguous()
    v = _kv_rows(g, total * block, hkv).view(total, block, hkv, D).transpose(1, 2).contiguous()
    return k, v, table.to(DEV)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _cu(lens):
    return _ints([0] + list(np.cumsum(lens)))


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["op"] == "prompt":
        q, kv = _prompt_lens(c)
        s.update(q_lens=q, kv_lens=kv, cu_q=_cu(q))
        s["q"] = torch.randn(sum(q), c["hq"], D, generator=g, device=DEV).to(torch.bfloat16)
        if c["source"] == "packed":
            s.update(k=_kv_rows(g, sum(kv), c["hkv"]), v=_kv_rows(g, sum(kv), c["hkv"]), cu_kv=_cu(kv))
        else:
            s["k"], s["v"], s["table"] = _paged(g, kv, c["hkv"], c["block"])
            s["seq_lens"] = _ints(kv)
        s["out"] = torch.zeros_like(s["q"])
    elif c["op"] == "decode":
        lens = _spread(c["lo"], c["hi"], c["batch"])
        s.update(lens=lens, max_seqlen=max(lens), seq_lens=_ints(lens))
        s["k"], s["v"], s["table"] = _paged(g, lens, c["hkv"], c["block"])
        s["q"] = torch.randn(c["batch"], c["hq"], D, generator=g, device=DEV).to(torch.bfloat16)
        s["k_new"] = _kv_rows(g, c["batch"], c["hkv"])
        s["v_new"] = _kv_rows(g, c["batch"], c["hkv"])
        s["out"] = torch.zeros_like(s["q"])
    else:
        # K and V pools of every layer, slices of one allocation as a serving engine reserves it
        shape = (2 * c["layers"], c["pages"], c["hkv"], c["block"], D)
        s["cache"] = torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8)
        s["pools"] = list(s["cache"].unbind(0))
        order = torch.randperm(c["pages"], generator=g, device=DEV).to(torch.int32)
        n = c["moves"]
        if c["kind"] == "fork":
            s["pairs"] = torch.stack([order[:n], order[n:2 * n]], dim=1).contiguous()
            r = _forked_rows(c)
            rows = torch.randperm(c["rows"], generator=g, device=DEV).to(torch.int32)
            s["row_pairs"] = torch.stack([rows[:r], rows[r:2 * r]], dim=1).contiguous()
            s["all_records"] = torch.randint(0, 256, (c["layers"], c["rows"], c["hkv"], 128), generator=g,
                                             device=DEV, dtype=torch.uint8)
            s["records"] = list(s["all_records"].unbind(0))
        else:
            # live pages scattered over the pool; those behind the live count move into the holes
            live_n = max(n, c["pages"] - n - c["pages"] // 8)
            dst = torch.randperm(live_n, generator=g, device=DEV)[:n].sort().values.to(torch.int32)
            src = (live_n + torch.randperm(c["pages"] - live_n, generator=g, device=DEV)[:n].sort().values)
            src = src.to(torch.int32)
            s["pairs"] = torch.stack([src, dst], dim=1).contiguous()
            s["remap"] = torch.arange(c["pages"], dtype=torch.int32, device=DEV)
            s["remap"][src.long()] = dst
            live = torch.ones(c["pages"], dtype=torch.bool, device=DEV)
            live[live_n:] = False
            live[dst.long()] = False
            live[src.long()] = True
            ids = live.nonzero().flatten().to(torch.int32)
            pick = torch.randint(0, ids.numel(), (c["rows"], c["columns"]), generator=g, device=DEV)
            s["table"] = ids[pick].contiguous()
            s["new_table"] = torch.empty_like(s["table"])
    if own:
        import int8_group_quantized_gb300 as dgq
        if c["op"] == "prompt":
            size = dgq.dgq_prompt_attn_workspace_size(c["batch"], c["hq"], c["hkv"])
        elif c["op"] == "decode":
            size = dgq.dgq_attn_workspace_size(c["batch"], c["hq"], c["hkv"], s["max_seqlen"])
        else:
            size = dgq.dgq_copy_pages_workspace_size()
        s["workspace"] = torch.zeros(size, dtype=torch.uint8, device=DEV)
    return s


# ---- one pass ---------------------------------------------------------------------------------------

def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"prompt": _plain_prompt, "decode": _plain_decode, "pages": _plain_pages}[op](s)
    import int8_group_quantized_gb300 as dgq
    if op == "prompt":
        if s["case"]["source"] == "packed":
            dgq.dgq_prompt_attn(s["q"], s["k"], s["v"], s["cu_q"], s["cu_kv"], s["out"], s["workspace"])
        else:
            dgq.dgq_prompt_attn_paged(s["q"], s["cu_q"], s["k"], s["v"], s["table"], s["seq_lens"], s["out"],
                                      s["workspace"])
        return s["out"]
    if op == "decode":
        dgq.dgq_paged_decode_attn_bf16(s["q"], s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["seq_lens"],
                                       s["max_seqlen"], s["out"], s["workspace"])
        return s["out"]
    dgq.dgq_copy_pages(s["pools"], s["pairs"], s["workspace"])
    if s["case"]["kind"] == "fork":
        dgq.dgq_copy_pages(s["records"], s["row_pairs"], s["workspace"])
        return [s["cache"], s["all_records"]]
    dgq.dgq_remap_tables(s["table"], s["remap"], s["new_table"], s["workspace"])
    return [s["cache"], s["new_table"]]


def _tokens(cache, row, n):
    """The first n tokens of a table row as fp32 [hkv, n, 128]."""
    block = cache.shape[2]
    ids = row[:(n + block - 1) // block].long()
    x = cache[ids].transpose(0, 1).reshape(cache.shape[1], -1, D)
    return x[:, :n].float()


def _plain_prompt(s):
    c = s["case"]
    hq, hkv = c["hq"], c["hkv"]
    group = hq // hkv
    outs, at_q, at_kv = [], 0, 0
    for b, (n, m) in enumerate(zip(s["q_lens"], s["kv_lens"])):
        if c["source"] == "packed":
            k = s["k"][at_kv:at_kv + m].float().transpose(0, 1)
            v = s["v"][at_kv:at_kv + m].float().transpose(0, 1)
        else:
            k, v = _tokens(s["k"], s["table"][b], m), _tokens(s["v"], s["table"][b], m)
        q = s["q"][at_q:at_q + n].float() * D ** -0.5
        step = max(1, min(n, (1 << 28) // max(1, hq * m)))
        for i in range(0, n, step):
            e = min(n, i + step)
            seen = m - n + e                                      # keys that the chunk's last row sees
            x = q[i:e].view(e - i, hkv, group, D).permute(1, 2, 0, 3).reshape(hkv, group * (e - i), D)
            z = torch.matmul(x, k[:, :seen].transpose(1, 2)).view(hkv, group, e - i, seen)
            at = torch.arange(m - n + i, seen, device=DEV)
            z = z.masked_fill(torch.arange(seen, device=DEV)[None, :] > at[:, None], float("-inf"))
            z = torch.exp(z - z.amax(dim=-1, keepdim=True))
            z = z / z.sum(dim=-1, keepdim=True)
            y = torch.matmul(z.view(hkv, group * (e - i), seen), v[:, :seen])
            outs.append(y.view(hkv, group, e - i, D).permute(2, 0, 1, 3).reshape(e - i, hq, D).to(torch.bfloat16))
        at_q += n
        at_kv += m
    return torch.cat(outs)


def _plain_decode(s):
    c = s["case"]
    hkv, group = c["hkv"], c["hq"] // c["hkv"]
    outs = []
    for b, n in enumerate(s["lens"]):
        k = torch.cat([_tokens(s["k"], s["table"][b], n), s["k_new"][b].float()[:, None]], dim=1)
        v = torch.cat([_tokens(s["v"], s["table"][b], n), s["v_new"][b].float()[:, None]], dim=1)
        q = s["q"][b].float().view(hkv, group, D) * D ** -0.5
        z = torch.matmul(q, k.transpose(1, 2))
        z = torch.exp(z - z.amax(dim=-1, keepdim=True))
        z = z / z.sum(dim=-1, keepdim=True)
        outs.append(torch.matmul(z, v).reshape(1, c["hq"], D).to(torch.bfloat16))
    return torch.cat(outs)


def _plain_pages(s):
    src, dst = s["pairs"][:, 0].long(), s["pairs"][:, 1].long()
    for p in s["pools"]:
        p[dst] = p[src]
    if s["case"]["kind"] == "fork":
        src, dst = s["row_pairs"][:, 0].long(), s["row_pairs"][:, 1].long()
        for r in s["records"]:
            r[dst] = r[src]
        return [s["cache"], s["all_records"]]
    return [s["cache"], s["remap"][s["table"].long()]]


# ---- the definition in 64 bits ----------------------------------------------------------------------

def exact(case, seed):
    """out[i, h] = sum_t w_t v_t / sum_t w_t with w_t = exp(q_i . k_t / sqrt(128)) over the keys that the
    row sees, head by head in float64.  Copies of pages are whole numbers: no such value."""
    c = case
    if c["op"] == "pages" or work(c)["flops"] > 3e12:
        return None
    s = prepare(c, seed)
    group = c["hq"] // c["hkv"]
    if c["op"] == "decode":
        queries, keys, extra = [1] * c["batch"], s["lens"], 1
    else:
        queries, keys, extra = s["q_lens"], s["kv_lens"], 0
    out = torch.zeros(sum(queries), c["hq"], D, dtype=torch.float64, device=DEV)
    row = base = 0
    for b in range(c["batch"]):
        n, m = queries[b], keys[b]
        t = torch.arange(m, device=DEV)
        for h in range(c["hkv"]):
            if c.get("source") == "packed":
                k, v = (s[x][base:base + m, h].double() for x in ("k", "v"))
            else:
                page = s["table"][b].long()[t // c["block"]]
                k, v = (s[x][page, h, t % c["block"]].double() for x in ("k", "v"))
            if extra:
                k = torch.cat([k, s["k_new"][b, h][None].double()])
                v = torch.cat([v, s["v_new"][b, h][None].double()])
            total = m + extra
            for i in range(0, n, 1024):
                e = min(n, i + 1024)
                upto = total - n + e
                seen = torch.arange(upto, device=DEV)[None, :] <= torch.arange(total - n + i, upto, device=DEV)[:, None]
                for j in range(h * group, (h + 1) * group):
                    x = s["q"][row + i:row + e, j].double() @ k[:upto].T / np.sqrt(float(D))
                    top = torch.where(seen, x, -torch.inf).max(dim=1, keepdim=True).values
                    w = torch.where(seen, torch.exp(x - top), 0.0)
                    out[row + i:row + e, j] = (w @ v[:upto]) / w.sum(dim=1, keepdim=True)
        row += n
        base += m
    return out
