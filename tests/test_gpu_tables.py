"""Block tables grown and slot maps made on the GPU, and rows written through them, against the definition
in whole numbers: ragged batches, what a request is refused for, outputs over their inputs, replayed steps,
strided rows, tokens without a slot, slots that do not exist."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BAD_BLOCK, BAD_LENGTH, NO_BLOCK = 5, 6, 4


def i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")


def workspace():
    import int8_group_quantized_gb300 as dgq
    return torch.zeros(dgq.dgq_extend_tables_workspace_size(), dtype=torch.uint8, device="cuda")


def grown(lens, new, bs, num_blocks, ids, used, table, total):
    """The definition; returns the outputs and the error words that may be recorded."""
    table, slots, lens_out = table.copy(), np.full(total, -1, dtype=np.int64), list(lens)
    cu = np.concatenate([[0], np.cumsum(np.maximum(new, 0))])
    errors, need_sum, used_out = set(), 0, used
    for b, (L, n) in enumerate(zip(lens, new)):
        bad = L < 0 or n < 0 or L + max(n, 0) > table.shape[1] * bs
        need = 0 if bad else -(-(L + n) // bs) - -(-L // bs)
        first, need_sum = used + need_sum, need_sum + need
        if bad or cu[b + 1] > total:
            errors.add(BAD_LENGTH)
            continue
        if need and first + need > len(ids):
            errors.add(NO_BLOCK)
            continue
        if need:
            used_out = first + need
        lens_out[b] = L + n
        had = -(-L // bs)
        for i in range(n):
            c, r = divmod(L + i, bs)
            block = ids[first + c - had] if c >= had else table[b, c]
            if not 0 <= block < num_blocks:
                errors.add(BAD_BLOCK)
                continue
            slots[cu[b] + i] = block * bs + r
            if r == 0:
                table[b, c] = block
    return table, slots, np.minimum(cu, total), lens_out, used_out, errors


def run(lens, new, bs, num_blocks, ids, used, table, total, in_place=False):
    import int8_group_quantized_gb300 as dgq
    ws = workspace()
    d_lens, d_used, d_table = i32(lens), i32([used]), i32(table)
    slots, cu = i32(np.full(total, 77)), i32(np.full(len(lens) + 1, 77))
    lens_out, used_out = (d_lens, d_used) if in_place else (i32(np.full(len(lens), 77)), i32([77]))
    dgq.dgq_extend_tables(d_lens, i32(new), bs, num_blocks, i32(ids), d_used, d_table, slots, cu, lens_out, used_out, ws)
    torch.cuda.synchronize()
    want = grown(lens, new, bs, num_blocks, ids, used, np.asarray(table), total)
    for got, x in zip((d_table, slots, cu, lens_out, used_out), want):
        assert np.array_equal(got.cpu().numpy().ravel(), np.asarray(x).ravel())
    error = dgq.dgq_workspace_error(ws)
    assert error in want[5] if want[5] else error == 0
    assert ws[16:24].cpu().tolist() == [0] * 8            # the count of finished blocks is back at 0


def case(rng, batch, bs, past, new, spare=0, columns=0):
    lens, new = rng.integers(0, past + 1, batch), rng.integers(0, new + 1, batch)
    columns = columns or int(-(-(lens + new).max() // bs)) + 2
    had, need = -(-lens // bs), -(-(lens + new) // bs) - -(-lens // bs)
    order = rng.permutation(int(had.sum() + need.sum()) + spare + 3)
    table = np.full((batch, columns), -9, dtype=np.int32)
    at = 0
    for b in range(batch):
        table[b, :had[b]] = order[at:at + had[b]]
        at += had[b]
    return dict(lens=lens.tolist(), new=new.tolist(), bs=bs, num_blocks=len(order),
                ids=np.concatenate([[0, 0], order[at:]]), used=2, table=table, total=int(new.sum()))


@pytest.mark.parametrize("batch,past,new", [(1, 0, 1), (1, 40, 0), (3, 100, 1), (33, 500, 90), (257, 64, 3), (700, 9, 2),
                                            (8192, 40, 1), (5, 3000, 9000)])
@pytest.mark.parametrize("bs", [16, 64])
def test_definition(batch, past, new, bs):
    c = case(np.random.default_rng(batch + bs), batch, bs, past, new)
    run(**c)
    run(**c, in_place=True)
    run(**dict(c, total=c["total"] + 5))                   # a padded step


def test_block_of_32_and_empty_slots():
    run(**case(np.random.default_rng(1), 7, 32, 200, 70))
    run([3, 4], [0, 0], 16, 8, [1], 0, [[1], [2]], 0)


@pytest.mark.parametrize("short", [1, 3, 1000])
def test_list_that_is_too_short(short):
    c = case(np.random.default_rng(short), 40, 16, 100, 30)
    run(**dict(c, ids=c["ids"][:max(2, len(c["ids"]) - 3 - short)]), in_place=True)


def test_no_free_ids_at_all():
    run([5, 16, 20], [3, 0, 12], 16, 9, [], 0, [[1, 0], [2, 0], [3, 4]], 15)      # all of them fit
    run([5, 16, 20], [3, 1, 12], 16, 9, [], 0, [[1, 0], [2, 0], [3, 4]], 16)      # the second does not


@pytest.mark.parametrize("lens,new", [([-1, 4, 3], [2, 2, 2]), ([5, 4, 3], [2, -2, 2]), ([5, 30, 3], [2, 3, 2]),
                                      ([5, 4, 3], [2, 2, 2 ** 31 - 1]), ([2 ** 31 - 1, 4, 3], [2, 2, 1])])
def test_lengths_that_do_not_fit_leave_the_others_alone(lens, new):
    table = [[1, 2], [3, 4], [5, 6]]
    run(lens, new, 16, 20, [10, 11, 12, 13], 1, table, 6)


def test_slots_that_the_buffer_does_not_have():
    run([0, 0, 0, 0], [5, 9, 4, 1], 16, 20, [10, 11, 12, 13], 0, np.zeros((4, 2)), 15)


def test_ids_that_are_not_blocks():
    run([10, 16, 7], [3, 20, 1], 16, 20, [10, 99, -1, 13], 0, [[50, 0, 0], [3, 0, 0], [4, 0, 0]], 24)


@pytest.mark.parametrize("used", [-1, 5])
def test_bad_count_of_used_ids(used):
    import int8_group_quantized_gb300 as dgq
    ws, lens, count, table = workspace(), i32([3, 16]), i32([used]), i32([[1, 0], [2, 0]])
    slots, cu = i32([7] * 3), i32([7] * 3)
    dgq.dgq_extend_tables(lens, i32([2, 1]), 16, 9, i32([5, 6, 7, 8]), count, table, slots, cu, lens, count, ws)
    assert dgq.dgq_workspace_error(ws) != 0
    assert slots.tolist() == [19, 20, -1] and lens.tolist() == [5, 16] and count.tolist() == [used]
    assert table.tolist() == [[1, 0], [2, 0]]


def test_replayed_steps_grow_the_tables():
    import int8_group_quantized_gb300 as dgq
    lens0, bs, steps = [0, 15, 16, 40], 16, 37
    table = np.full((4, 6), -9)
    table[1, :1], table[2, :1], table[3, :3] = [5], [6], [7, 8, 9]
    ids = np.arange(10, 40)[::-1].copy()
    lens, used, d_table, ws = i32(lens0), i32([0]), i32(table), workspace()
    slots, cu, new, d_ids = i32([0] * 4), i32([0] * 5), i32([1, 1, 0, 1]), i32(ids)
    call = lambda: dgq.dgq_extend_tables(lens, new, bs, 64, d_ids, used, d_table, slots, cu, lens, used, ws)
    call()                                                 # the launcher's setup, and the first step
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    state = grown(lens0, [1, 1, 0, 1], bs, 64, ids, 0, table, 4)
    for _ in range(steps):
        graph.replay()
        state = grown(state[3], [1, 1, 0, 1], bs, 64, ids, state[4], state[0], 4)
    torch.cuda.synchronize()
    assert dgq.dgq_workspace_error(ws) == 0
    for got, x in zip((d_table, slots, cu, lens, used), state):
        assert np.array_equal(got.cpu().numpy().ravel(), np.asarray(x).ravel())


# ---- rows ---------------------------------------------------------------------------------------------

def fused(T, hkv, seed, pad=0):
    """K and V as slices of one buffer [T, pad + 2 hkv, 128] of arbitrary bits (NaN patterns too)."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(-32768, 32768, (T, pad + 2 * hkv, 128), generator=g, dtype=torch.int16).view(torch.bfloat16).cuda()
    return x[:, pad:pad + hkv], x[:, pad + hkv:]


@pytest.mark.parametrize("T,hkv,bs", [(1, 1, 16), (3, 3, 16), (50, 2, 32), (257, 8, 64), (100, 32, 16), (2000, 1, 64)])
def test_rows_go_to_their_slots(T, hkv, bs):
    import int8_group_quantized_gb300 as dgq
    k, v = fused(T, hkv, T + hkv, pad=hkv)
    blocks = T // bs + 4
    slots = torch.randperm(blocks * bs, generator=torch.Generator().manual_seed(T))[:T].to(torch.int32)
    slots[1::7] = -1
    pages = [torch.full((blocks, hkv, bs, 128), float(i), dtype=torch.bfloat16, device="cuda") for i in (3, 4)]
    want = [p.clone().view(torch.int16) for p in pages]
    live = (slots >= 0).nonzero().flatten().cuda()
    at = slots.cuda().long()[live]
    for w, x in zip(want, (k, v)):
        w[at // bs, :, at % bs] = x[live].view(torch.int16)
    ws = workspace()
    dgq.dgq_write_slots(k, v, slots.cuda(), *pages, ws)
    torch.cuda.synchronize()
    assert dgq.dgq_workspace_error(ws) == 0
    assert all(torch.equal(p.view(torch.int16), w) for p, w in zip(pages, want))
    dgq.dgq_write_slots(k.contiguous(), v.contiguous(), slots.cuda(), *pages, ws)
    assert all(torch.equal(p.view(torch.int16), w) for p, w in zip(pages, want))


@pytest.mark.parametrize("bad", [-2, 64, 2 ** 31 - 1, -2 ** 31])
def test_a_slot_that_does_not_exist_is_flagged_and_left_out(bad):
    import int8_group_quantized_gb300 as dgq
    k, v = fused(3, 2, 1)
    pages = [torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ws = workspace()
    dgq.dgq_write_slots(k, v, i32([0, bad, 63]), *pages, ws)
    assert dgq.dgq_workspace_error(ws) == BAD_BLOCK
    for p, x in zip(pages, (k, v)):
        p, x = p.view(torch.int16), x.view(torch.int16)
        assert torch.equal(p[0, :, 0], x[0]) and torch.equal(p[3, :, 15], x[2])
        p[0, :, 0], p[3, :, 15] = 0, 0
        assert not p.any()


def test_rows_behind_two_gigabytes():
    import int8_group_quantized_gb300 as dgq
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    blocks = (5 << 30) // (2 * 64 * 256)
    pages = [torch.zeros(blocks, 2, 64, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    k, v = fused(2, 2, 2)
    dgq.dgq_write_slots(k, v, i32([blocks * 64 - 1, 5]), *pages, workspace())
    for p, x in zip(pages, (k, v)):
        assert torch.equal(p[-1, :, 63].view(torch.int16), x[0].view(torch.int16))
        assert torch.equal(p[0, :, 5].view(torch.int16), x[1].view(torch.int16))


def test_binding_refuses_rows_it_would_misread():
    import int8_group_quantized_gb300 as dgq
    k, v = fused(4, 2, 3)
    pages = [torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    slots, ws = i32([0, 1, 2, 3]), workspace()
    dgq.dgq_write_slots(k, v, slots, *pages, ws)           # accepted
    wide = torch.zeros(4, 2, 256, dtype=torch.bfloat16, device="cuda")
    heads = torch.zeros(4, 4, 128, dtype=torch.bfloat16, device="cuda")[:, ::2]
    for bad in (k.float(), k.half(), k[:3], wide[..., ::2], wide[..., :128], heads, k.cpu(), k[:1].expand(4, 2, 128),
                k.transpose(0, 1).contiguous().transpose(0, 1)):
        for args in ((bad, v), (k, bad)):
            with pytest.raises(dgq.DGQError):
                dgq.dgq_write_slots(*args, slots, *pages, ws)
    for bad in (slots.long(), slots[:3], slots.cpu()):
        with pytest.raises(dgq.DGQError):
            dgq.dgq_write_slots(k, v, bad, *pages, ws)
    with pytest.raises(dgq.DGQError):
        dgq.dgq_write_slots(k, v, slots, pages[0], pages[1][:3], ws)
