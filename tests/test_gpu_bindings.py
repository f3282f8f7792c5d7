"""The binding's checks in front of raw pointers, on CUDA operands that are shown to be accepted first: then
one property of one operand is changed at a time (type, shape, stride, host memory), and the call is
refused with nothing written."""
import pytest
import torch

from attn_reference import Pages, rows

pytestmark = pytest.mark.gpu

B, HQ, HKV, BS, INVALID = 2, 4, 2, 16, -1


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def zeros(n):
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def gap(x):
    """The same values with a gap between neighbours of the last dimension."""
    return x.repeat_interleave(2, dim=-1)[..., ::2]


def spoiled(x, dtypes):
    """x with one property changed: another type, a row more or less, gaps, host memory."""
    yield from (x.to(t) for t in dtypes)
    yield torch.cat([x, x[-1:]])
    yield x[:-1].clone()
    yield gap(x)
    yield x.cpu()


def calls():
    import int8_group_quantized_gb300 as dgq
    f, i, b = (torch.float16, torch.float32), (torch.int64,), (torch.int8,)
    q, kv = rows(9, HQ, 1, 1.0).cuda(), [rows(9, HKV, s).cuda() for s in (2, 3)]
    cu = i32([0, 4, 9])
    pages = Pages([rows(n, HKV, 4 + n) for n in (4, 20)], [rows(n, HKV, 40 + n) for n in (4, 20)], HKV, BS).cuda()
    ws = zeros(max(dgq.dgq_prompt_attn_workspace_size(B, HQ, HKV), dgq.dgq_attn_workspace_size(B, HQ, HKV, 32)))
    out = lambda x: torch.full_like(x, 7)
    yield "prompt", dgq.dgq_prompt_attn, "out", dict(
        q=(q, f), k=(kv[0], f), v=(kv[1], f), cu_q=(cu, i), cu_kv=(cu.clone(), i), out=(out(q), f), workspace=ws)
    yield "prompt_paged", dgq.dgq_prompt_attn_paged, "out", dict(
        q=(q, f), cu_q=(cu, i), k_src=(pages.k, f), v_src=(pages.v, f), src_block_tables=(pages.table, i),
        seq_lens=(pages.lens, i), out=(out(q), f), workspace=ws)
    yield "decode_bf16", dgq.dgq_paged_decode_attn_bf16, "out", dict(
        q=(q[:B].clone(), f), k_new=(kv[0][:B].clone(), f), v_new=(kv[1][:B].clone(), f), k_src=(pages.k, f),
        v_src=(pages.v, f), src_block_tables=(pages.table, i), seq_lens=(pages.lens, i), max_seqlen=20,
        out=(out(q[:B]), f), workspace=ws)
    yield "remap", dgq.dgq_remap_tables, "out", dict(
        tables=(i32([[1, 2], [0, 3]]), i), remap=(i32([3, 2, 1, 0]), i), out=(out(i32([[0, 0], [0, 0]])), i), workspace=ws)
    yield "fork_records", dgq.dgq_fork_records, "seg_table", dict(
        seg_table=(torch.full((3, HKV, 128), 1, dtype=torch.uint8, device="cuda"), b), forks=(i32([[0, 1, 0]]), i),
        workspace=ws)


# operands whose first dimension is the call's own measure: a longer or shorter one is another valid call
FREE = {("remap", "remap"), ("fork_records", "seg_table"), ("fork_records", "forks")}


@pytest.mark.parametrize("which", ["prompt", "prompt_paged", "decode_bf16", "remap", "fork_records"])
def test_one_changed_property_is_refused(which):
    import int8_group_quantized_gb300 as dgq
    name, call, written, args = next(c for c in calls() if c[0] == which)
    good = {k: v[0] if isinstance(v, tuple) else v for k, v in args.items()}
    before = good[written].clone()
    call(**good)                                       # the operands are accepted, and the call writes
    torch.cuda.synchronize()
    assert not torch.equal(good[written], before)
    good[written].copy_(before)
    tried = 0
    for arg, v in args.items():
        if not isinstance(v, tuple):
            continue
        for kind, bad in enumerate(spoiled(*v)):
            if (name, arg) in FREE and bad.shape != v[0].shape:
                continue
            if bad.shape == v[0].shape and bad.dtype is v[0].dtype and bad.is_cuda and bad.is_contiguous():
                continue                               # (one entry has no gaps)
            with pytest.raises(dgq.DGQError) as e:
                call(**{**good, arg: bad})
            assert e.value.status == INVALID, (arg, kind)
            tried += 1
    torch.cuda.synchronize()
    assert torch.equal(good[written], before) and tried >= 3 * (len(args) - 2)


def test_page_arrays_are_checked_one_by_one():
    import int8_group_quantized_gb300 as dgq
    ws = zeros(dgq.dgq_copy_pages_workspace_size())
    a, b = (torch.arange(4 * 64, device="cuda").to(torch.uint8).view(4, 64) + s for s in (0, 1))
    pairs = i32([[0, 1]])
    dgq.dgq_copy_pages([a, b], pairs, ws)
    assert torch.equal(a[1], a[0]) and torch.equal(b[1], b[0])
    a[1], b[1] = 9, 9
    keep = a.clone(), b.clone()
    wide = torch.zeros(4, 128, dtype=torch.uint8, device="cuda")
    for bad in (b[:3], wide, wide[:, ::2], wide[:, :64], b.to(torch.int16), b.view(torch.int8), b.cpu(),
                torch.zeros(8, 64, dtype=torch.uint8, device="cuda")[::2]):
        for arrays in ([a, bad], [bad, a]):
            with pytest.raises(dgq.DGQError) as e:
                dgq.dgq_copy_pages(arrays, pairs, ws)
            assert e.value.status == INVALID
    for bad in (pairs.long(), pairs.flatten(), i32([[0, 1, 2]]), pairs.cpu(), i32([[0, 0, 1, 1]])[:, ::2]):
        with pytest.raises(dgq.DGQError) as e:
            dgq.dgq_copy_pages([a, b], bad, ws)
        assert e.value.status == INVALID
    torch.cuda.synchronize()
    assert torch.equal(a, keep[0]) and torch.equal(b, keep[1])
