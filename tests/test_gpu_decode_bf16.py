"""Decode attention over a bf16 paged cache against plain attention in 64 bits, element by element within
the bound of the roundings: group sizes, block sizes, empty and ragged requests, long splits, slots
that hold anything, repeatability, graphs and device guards."""
import pytest
import torch

from attn_reference import Pages, attend, check, rows

pytestmark = pytest.mark.gpu


class Step:
    def __init__(self, lens, hq, hkv, block, seed, sigma=0.5, fill=float("nan")):
        self.lens, self.hq, self.hkv = lens, hq, hkv
        b = len(lens)
        self.q = rows(b, hq, seed, 1.0)
        self.kn, self.vn = rows(b, hkv, seed + 1), rows(b, hkv, seed + 2)
        self.ks = [rows(n, hkv, seed + 100 + i, sigma) for i, n in enumerate(lens)]
        self.vs = [rows(n, hkv, seed + 9000 + i) for i, n in enumerate(lens)]
        self.pages = Pages(self.ks, self.vs, hkv, block, fill=fill)
        self.ref = None

    def device(self):
        import int8_group_quantized_gb300 as dgq
        self.pages.cuda()
        self.d = [x.cuda() for x in (self.q, self.kn, self.vn)]
        self.max = max(1, max(self.lens))
        self.ws = torch.zeros(dgq.dgq_attn_workspace_size(len(self.lens), self.hq, self.hkv, self.max),
                              dtype=torch.uint8, device="cuda")
        return self

    def call(self, out):
        import int8_group_quantized_gb300 as dgq
        p = self.pages
        dgq.dgq_paged_decode_attn_bf16(*self.d, p.k, p.v, p.table, p.lens, self.max, out, self.ws)

    def run(self):
        import int8_group_quantized_gb300 as dgq
        out = torch.zeros_like(self.d[0])
        self.call(out)
        torch.cuda.synchronize()
        assert dgq.dgq_workspace_error(self.ws) == 0
        return out

    def reference(self):
        if self.ref is None:
            g = self.hq // self.hkv
            out = torch.zeros(len(self.lens), self.hq, 128, dtype=torch.float64)
            bound = torch.zeros_like(out)
            for b, n in enumerate(self.lens):
                for h in range(self.hkv):
                    k = torch.cat([self.ks[b][:, h], self.kn[b, h][None]]).double()
                    v = torch.cat([self.vs[b][:, h], self.vn[b, h][None]]).double()
                    s = slice(h * g, (h + 1) * g)
                    out[b, s], bound[b, s] = attend(self.q[b, s].double(), k, v, torch.full((g,), n + 1))
            self.ref = out, bound
        return self.ref

    def check(self, out):
        check(out, *self.reference())


def verify(*a, **kw):
    s = Step(*a, **kw).device()
    s.check(s.run())


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (8, 8), (8, 4), (6, 3), (16, 4), (16, 2), (8, 1)])
def test_group_sizes(hq, hkv):
    verify([5, 64, 65, 700, 3000], hq, hkv, 16, seed=hq + hkv)


@pytest.mark.parametrize("block", [16, 32, 64])
def test_block_sizes_and_ragged_tails(block):
    verify([0, 1, 15, 16, 17, 63, 64, 65, 129, 1000, 4097], 8, 2, block, seed=block)


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), 3e38])
def test_slots_behind_the_end_may_hold_anything(fill):
    verify([1, 3, 5, 9, 13, 18, 250], 8, 2, 64, seed=3, fill=fill)


def test_empty_cache_returns_the_new_value():
    s = Step([0, 7, 0], 4, 2, 16, seed=5).device()
    out = s.run().cpu()
    s.check(out)
    for b in (0, 2):
        assert torch.equal(out[b], s.vn[b].repeat_interleave(2, dim=0))


def test_long_requests_are_split():
    verify([40000, 100], 8, 2, 64, seed=7)
    verify([70001], 2, 1, 32, seed=8)


@pytest.mark.parametrize("lens", [[200] * 128, [300] * 8])  # warp merge, block merge
def test_merges(lens):
    verify(lens, 8, 2, 16, seed=9)


def test_running_maximum_that_keeps_climbing():
    s = Step([3000, 2000], 8, 2, 16, seed=10, fill=0.0)
    for i in range(2):
        f = torch.linspace(0.01, 6.0, s.lens[i])
        s.ks[i] = (s.ks[i].float() * f[:, None, None]).to(torch.bfloat16)
    s.pages = Pages(s.ks, s.vs, 2, 16, fill=0.0)
    s.device()
    s.check(s.run())


def test_runs_repeat_and_pages_may_move():
    s = Step([3000, 70, 9000], 8, 2, 32, seed=11).device()
    one = s.run()
    assert torch.equal(one, s.run())
    p = s.pages
    perm = torch.randperm(p.k.shape[0], generator=torch.Generator().manual_seed(1)).cuda()
    k, v = torch.empty_like(p.k), torch.empty_like(p.v)
    k[perm], v[perm] = p.k, p.v
    p.k, p.v, p.table = k, v, perm[p.table.long()].to(torch.int32)
    assert torch.equal(one, s.run())


def test_rows_behind_two_gigabytes():
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    s = Step([300, 40], 4, 2, 64, seed=12).device()
    p, blocks = s.pages, (5 << 30) // (2 * 64 * 256)
    k = torch.empty(blocks, 2, 64, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    n = p.k.shape[0]
    k[-n:], v[-n:] = p.k, p.v
    p.k, p.v, p.table = k, v, p.table + (blocks - n)
    s.check(s.run())


@pytest.mark.parametrize("lens", [[200] * 128, [3000] * 8])
def test_graph_replays_equal_calls(lens):
    s = Step(lens, 8, 2, 16, seed=13).device()
    want = s.run()
    out = torch.zeros_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.call(out)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.call(out)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_device_guards():
    import int8_group_quantized_gb300 as dgq
    s = Step([300, 37], 4, 2, 16, seed=14, fill=0.0).device()
    good, out = s.pages.table.clone(), torch.zeros_like(s.d[0])
    for value in (s.pages.k.shape[0], -5):
        s.pages.table = good.clone()
        s.pages.table[0, 3] = value
        s.call(out)
        assert dgq.dgq_workspace_error(s.ws) == 5
        ref, bound = s.reference()
        check(out[1:], ref[1:], bound[1:])
        dgq.dgq_workspace_init(s.ws)
    s.pages.table = good
    s.pages.lens[1] = good.shape[1] * 16 + 1
    s.call(out)
    assert dgq.dgq_workspace_error(s.ws) == 6
    dgq.dgq_workspace_init(s.ws)
    s.pages.lens[1] = 37
    s.check(s.run())
