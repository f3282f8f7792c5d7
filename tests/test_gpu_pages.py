"""dgq_copy_pages and dgq_remap_tables on the GPU: every byte of every array against indexed copies on
the CPU (whole numbers: equal), for page sizes from 16 bytes up, many arrays, repeated sources, ids
outside the pools, and captured."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def ws():
    import int8_group_quantized_gb300 as dgq
    return torch.zeros(dgq.dgq_copy_pages_workspace_size(), dtype=torch.uint8, device="cuda")


def arrays(n, pages, size, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randint(0, 256, (pages, size), generator=g, dtype=torch.uint8) for _ in range(n)]


def expected(arrs, pairs):
    out = [a.clone() for a in arrs]
    for s, d in pairs:
        for a, o in zip(arrs, out):
            o[d] = a[s]
    return out


@pytest.mark.parametrize("size", [16, 48, 256, 1024, 4080, 4096, 4112, 16384, 65536 + 16])
@pytest.mark.parametrize("count", [1, 3])
def test_page_sizes(size, count):
    import int8_group_quantized_gb300 as dgq
    arrs = arrays(count, 20, size, seed=size + count)
    pairs = [(3, 0), (3, 19), (7, 2), (18, 11)]
    dev, w = [a.cuda() for a in arrs], ws()
    dgq.dgq_copy_pages(dev, torch.tensor(pairs, dtype=torch.int32, device="cuda"), w)
    assert dgq.dgq_workspace_error(w) == 0
    for a, b in zip(dev, expected(arrs, pairs)):
        assert torch.equal(a.cpu(), b)


@pytest.mark.parametrize("count", [64, 256, 257, 600])
def test_many_arrays(count):
    import int8_group_quantized_gb300 as dgq
    g = torch.Generator().manual_seed(count)
    whole = torch.randint(0, 256, (count, 9, 2, 16, 128), generator=g, dtype=torch.uint8)
    pairs = torch.tensor([(8, 1), (4, 5), (8, 0)], dtype=torch.int32)
    dev, w = whole.cuda(), ws()
    dgq.dgq_copy_pages(dev.unbind(0), pairs.cuda(), w)
    assert dgq.dgq_workspace_error(w) == 0
    want = whole.clone()
    want[:, pairs[:, 1].long()] = whole[:, pairs[:, 0].long()]
    assert torch.equal(dev.cpu(), want)


def test_bf16_pools_and_records():
    import int8_group_quantized_gb300 as dgq
    pool = torch.randn(12, 2, 16, 128, device="cuda").to(torch.bfloat16)
    rec = torch.randint(0, 256, (6, 2, 128), dtype=torch.uint8, device="cuda")
    p0, r0, w = pool.clone(), rec.clone(), ws()
    dgq.dgq_copy_pages([pool], torch.tensor([(2, 9)], dtype=torch.int32, device="cuda"), w)
    dgq.dgq_copy_pages([rec], torch.tensor([(0, 5), (0, 3)], dtype=torch.int32, device="cuda"), w)
    p0[9], r0[5], r0[3] = p0[2], r0[0], r0[0]
    assert torch.equal(pool, p0) and torch.equal(rec, r0)


def test_nothing_to_copy():
    import int8_group_quantized_gb300 as dgq
    a, w = arrays(1, 4, 64, 0)[0].cuda(), ws()
    b = a.clone()
    dgq.dgq_copy_pages([a], torch.zeros(0, 2, dtype=torch.int32, device="cuda"), w)
    dgq.dgq_copy_pages([], torch.tensor([(0, 1)], dtype=torch.int32, device="cuda"), w)
    assert torch.equal(a, b)


@pytest.mark.parametrize("bad", [(20, 1), (1, 20), (-1, 4), (4, -1), (2 ** 31 - 1, 0)])
def test_ids_outside_are_flagged_and_skipped(bad):
    import int8_group_quantized_gb300 as dgq
    arrs, w = arrays(2, 20, 512, seed=5), ws()
    dev = [a.cuda() for a in arrs]
    dgq.dgq_copy_pages(dev, torch.tensor([(3, 7), bad, (6, 8)], dtype=torch.int32, device="cuda"), w)
    assert dgq.dgq_workspace_error(w) == 5
    for a, b in zip(dev, expected(arrs, [(3, 7), (6, 8)])):
        assert torch.equal(a.cpu(), b)


def test_pages_behind_four_gigabytes():
    import int8_group_quantized_gb300 as dgq
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    size = 1 << 20
    pool = torch.empty((5 << 30) // size, size, dtype=torch.uint8, device="cuda")
    n = pool.shape[0]
    pool[1].random_(0, 256), pool[n - 1].random_(0, 256)
    a, b, w = pool[1].clone(), pool[n - 1].clone(), ws()
    dgq.dgq_copy_pages([pool], torch.tensor([(1, n - 2), (n - 1, 0)], dtype=torch.int32, device="cuda"), w)
    assert torch.equal(pool[n - 2], a) and torch.equal(pool[0], b)


@pytest.mark.parametrize("shape", [(1, 1), (3, 7), (64, 512), (2000, 300)])
def test_remap(shape):
    import int8_group_quantized_gb300 as dgq
    g = torch.Generator().manual_seed(1)
    remap = torch.randperm(1000, generator=g).to(torch.int32)
    table = torch.randint(0, 1000, shape, generator=g, dtype=torch.int32)
    t, w = table.cuda(), ws()
    out = torch.empty_like(t)
    dgq.dgq_remap_tables(t, remap.cuda(), out, w)
    assert torch.equal(out.cpu(), remap[table.long()]) and torch.equal(t.cpu(), table)
    dgq.dgq_remap_tables(t, remap.cuda(), t, w)  # in place
    assert torch.equal(t, out) and dgq.dgq_workspace_error(w) == 0


def test_remap_keeps_and_flags_foreign_entries():
    import int8_group_quantized_gb300 as dgq
    t, w = torch.tensor([[0, 9, -1, 1 << 30]], dtype=torch.int32, device="cuda"), ws()
    remap = torch.arange(9, -1, -1, dtype=torch.int32, device="cuda")
    dgq.dgq_remap_tables(t, remap, t, w)
    assert t.tolist() == [[9, 0, -1, 1 << 30]] and dgq.dgq_workspace_error(w) == 5


def test_graph_replays_equal_calls():
    import int8_group_quantized_gb300 as dgq
    pool, w = arrays(1, 16, 4096, 3)[0].cuda(), ws()
    pairs = torch.tensor([(0, 8), (1, 9)], dtype=torch.int32, device="cuda")
    table = torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda")
    remap = torch.arange(16, dtype=torch.int32, device="cuda").flip(0).contiguous()
    out = torch.empty_like(table)

    def call():
        dgq.dgq_copy_pages([pool], pairs, w)
        dgq.dgq_remap_tables(table, remap, out, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for k in range(2):
        pool[8:10] = 0
        pairs[0, 0] = 3 + k  # a replay reads the pairs as they are then
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(pool[8], pool[3 + k]) and torch.equal(pool[9], pool[1])
        assert out.tolist() == [[15, 14, 13]]
