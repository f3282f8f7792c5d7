"""The bf16 operators in one run with the INT8 cache, as a serving engine uses them: a prompt attended
in chunks over bf16 pages, decode over those pages, compression into INT8 pages, requests forked
(pages shared, the last page and the records copied), both sides appended to and decoded, a
re-segmented fork given pages of its own first, requests ended and the pools compacted.  Forks and
moves change no answer: the outputs are compared bit for bit."""
import numpy as np
import pytest
import torch

from attn_reference import Pages, check, prompt, rows

pytestmark = pytest.mark.gpu

HQ, HKV, BS = 8, 2, 16


def zeros(n):
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def test_prompt_decode_compress_fork_append_free_compact():
    import int8_group_quantized_gb300 as dgq
    lens = [300, 77, 160]
    B = len(lens)
    ks = [rows(n, HKV, 10 + b) for b, n in enumerate(lens)]
    vs = [rows(n, HKV, 20 + b) for b, n in enumerate(lens)]
    q = rows(sum(lens), HQ, 30, 1.0)
    src = Pages(ks, vs, HKV, BS, fill=0.0).cuda()

    # ---- the prompt, in two chunks per request, over bf16 pages; the same from packed rows
    ref, bound = prompt(q, ks, vs, lens, HQ, HKV)
    ws = zeros(dgq.dgq_prompt_attn_workspace_size(B, HQ, HKV))
    first = [n // 2 for n in lens]
    start = np.concatenate([[0], np.cumsum(lens)])
    got = torch.empty(sum(lens), HQ, 128, dtype=torch.bfloat16, device="cuda")
    for lo, hi in (([0] * B, first), (first, lens)):
        idx = torch.cat([torch.arange(start[b] + lo[b], start[b] + hi[b]) for b in range(B)])
        n = [h - l for l, h in zip(lo, hi)]
        out = torch.empty(sum(n), HQ, 128, dtype=torch.bfloat16, device="cuda")
        dgq.dgq_prompt_attn_paged(q[idx].cuda(), i32([0] + list(np.cumsum(n))), src.k, src.v, src.table, i32(hi), out, ws)
        got[idx.cuda()] = out
    check(got, ref, bound)
    cu = i32([0] + list(np.cumsum(lens)))
    whole = torch.empty_like(got)
    dgq.dgq_prompt_attn(q.cuda(), torch.cat(ks).cuda(), torch.cat(vs).cuda(), cu, cu, whole, ws)
    check(whole, ref, bound)

    # ---- a decode step over the bf16 pages (what the compressed cache below approximates)
    step = [x.cuda() for x in (rows(B, HQ, 40, 1.0), rows(B, HKV, 41, 0.15), rows(B, HKV, 42, 0.15))]
    max_len = 512
    aws = zeros(dgq.dgq_attn_workspace_size(2 * B, HQ, HKV, max_len))
    exact = torch.empty(B, HQ, 128, dtype=torch.bfloat16, device="cuda")
    dgq.dgq_paged_decode_attn_bf16(*step, src.k, src.v, src.table, src.lens, src.table.shape[1] * BS, exact, aws)

    # ---- compressed into INT8 pages of a pool with room for the forks
    pool = dgq.BlockPool(120)
    columns = max_len // BS
    table = np.zeros((2 * B, columns), dtype=np.int32)
    for b, n in enumerate(lens):
        pool.alloc_table_row(n, BS, table, b)
    kp = torch.full((120, HKV, BS, 128), 9, dtype=torch.uint8, device="cuda")
    vp = kp.clone()
    rec = torch.zeros(2 * B, HKV, 128, dtype=torch.uint8, device="cuda")
    cws = zeros(dgq.dgq_compress_workspace_size(B, max_len, HKV))
    bt = torch.from_numpy(table).cuda()
    dgq.dgq_compress_paged(src.k, src.v, src.table, cu, src.table.shape[1] * BS, BS, bt[:B].contiguous(), kp, vp,
                           rec[:B], cws)

    def decode(table, rows_, lens_):
        b = len(rows_)
        out = torch.empty(b, HQ, 128, dtype=torch.bfloat16, device="cuda")
        pick = [r % B for r in rows_]
        dgq.dgq_paged_decode_attn(*[x[pick].contiguous() for x in step], kp, vp, rec[rows_].contiguous(),
                                  torch.from_numpy(table[rows_]).cuda(), i32(lens_), max_len, out, aws)
        return out
    base = decode(table, list(range(B)), lens)
    assert (base.float() - exact.float()).abs().max() < 1e-2 and not torch.equal(base, exact)

    # ---- every request forked: whole pages shared, the last page and the records copied
    pws, used = zeros(dgq.dgq_copy_pages_workspace_size()), 120 - pool.num_free()
    pairs = [pool.fork_row(n, BS, table, b, B + b) for b, n in enumerate(lens)]
    pairs = np.concatenate(pairs)
    assert len(pairs) == sum(n % BS != 0 for n in lens) and 120 - pool.num_free() == used + len(pairs)
    dgq.dgq_copy_pages([kp, vp], torch.from_numpy(pairs).cuda(), pws)
    dgq.dgq_copy_pages([rec], i32([[b, B + b] for b in range(B)]), pws)
    forked = list(range(B, 2 * B))
    assert torch.equal(decode(table, forked, lens), base)

    # ---- the forks grow (a new page where the last one is full); the requests they came from do not change
    for b, n in enumerate(lens):
        if n % BS == 0:
            table[B + b, n // BS] = pool.alloc(1)[0]
    new = [rows(B, HKV, 50, 0.15).cuda(), rows(B, HKV, 51, 0.15).cuda()]
    dgq.dgq_append(*new, BS, torch.from_numpy(table[B:]).cuda(), kp, vp, rec[B:], pws)
    assert torch.equal(decode(table, list(range(B)), lens), base)
    grown = decode(table, forked, [n + 1 for n in lens])
    assert not torch.equal(grown, base)

    # ---- one fork gets pages of its own (as before it is re-encoded in place): its answer stays
    own = pool.own_row(table, B, 0, lens[0] // BS)
    assert len(own) == lens[0] // BS
    dgq.dgq_copy_pages([kp, vp], torch.from_numpy(own).cuda(), pws)
    kp[torch.from_numpy(table[0, :lens[0] // BS]).cuda().long()] ^= 255   # the first request's own pages overwritten
    vp[torch.from_numpy(table[0, :lens[0] // BS]).cuda().long()] ^= 255
    assert torch.equal(decode(table, forked, [n + 1 for n in lens]), grown)

    # ---- the first requests end; what is left moves together; every answer stays
    for b, n in enumerate(lens):
        pool.free_row(table, b, (n + BS - 1) // BS)
    remap, moves = pool.compact()
    assert len(moves) and moves[:, 1].max() < 120 - pool.num_free() <= moves[:, 0].min()
    dgq.dgq_copy_pages([kp, vp], torch.from_numpy(moves).cuda(), pws)
    bt = torch.from_numpy(table).cuda()
    dgq.dgq_remap_tables(bt, torch.from_numpy(remap).cuda(), bt, pws)
    live = 120 - pool.num_free()
    kp[live:], vp[live:] = 0, 0
    assert torch.equal(decode(bt.cpu().numpy(), forked, [n + 1 for n in lens]), grown)
    for w in (ws, aws, cws, pws):
        assert dgq.dgq_workspace_error(w) == 0


def test_workspace_outside_the_current_device_is_refused():
    """A workspace in host memory, or one with gaps, is refused by every call before anything is launched."""
    import int8_group_quantized_gb300 as dgq
    q, kv = rows(4, HQ, 1).cuda(), rows(4, HKV, 2).cuda()
    src = Pages([rows(4, HKV, 3)], [rows(4, HKV, 4)], HKV, BS).cuda()
    cu, one, ids = i32([0, 4]), i32([3]), i32([[0, 0]])
    out = torch.full_like(q, 7.0)
    size = max(dgq.dgq_prompt_attn_workspace_size(1, HQ, HKV), dgq.dgq_attn_workspace_size(4, HQ, HKV, 16))
    for bad in (torch.zeros(size, dtype=torch.uint8), zeros(2 * size)[::2]):
        for call in (lambda: dgq.dgq_prompt_attn(q, kv, kv, cu, cu, out, bad),
                     lambda: dgq.dgq_prompt_attn_paged(q, cu, src.k, src.v, src.table, src.lens, out, bad),
                     lambda: dgq.dgq_paged_decode_attn_bf16(q[:1], kv[:1], kv[:1], src.k, src.v, src.table, one, 16, out[:1], bad),
                     lambda: dgq.dgq_copy_pages([src.k], ids, bad),
                     lambda: dgq.dgq_remap_tables(src.table, one, src.table, bad)):
            with pytest.raises(dgq.DGQError):
                call()
    assert torch.all(out == 7.0)
