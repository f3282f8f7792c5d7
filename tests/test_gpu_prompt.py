"""Causal attention of prompts on the GPU (packed rows and bf16 pages) against plain attention in 64
bits, element by element within a bound derived from the roundings; lengths from nothing to long
histories, every group size, rows that see no key, values outside the requests, repeatability,
graphs, streams and threads."""
import threading

import numpy as np
import pytest
import torch

from attn_reference import Pages, check, prompt, rows

pytestmark = pytest.mark.gpu


def cu(lens):
    return torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")


def workspace(b, hq, hkv):
    import int8_group_quantized_gb300 as dgq
    return torch.zeros(dgq.dgq_prompt_attn_workspace_size(b, hq, hkv), dtype=torch.uint8, device="cuda")


class Prompt:
    """One call's inputs: per request `n` query rows and `m` keys."""

    def __init__(self, shape, hq, hkv, seed, block=None, sigma=0.5, q_sigma=1.0):
        self.n, self.m = [s[0] for s in shape], [s[1] for s in shape]
        self.hq, self.hkv, self.block = hq, hkv, block
        self.q = rows(sum(self.n), hq, seed, q_sigma)
        self.ks = [rows(m, hkv, seed + 100 + i, sigma) for i, m in enumerate(self.m)]
        self.vs = [rows(m, hkv, seed + 5000 + i) for i, m in enumerate(self.m)]
        self.ref = None

    def device(self):
        self.dq, self.cu_q = self.q.cuda(), cu(self.n)
        self.ws = workspace(len(self.n), self.hq, self.hkv)
        if self.block is None:
            self.k = torch.cat(self.ks).cuda()
            self.v = torch.cat(self.vs).cuda()
            self.cu_kv = cu(self.m)
        else:
            self.pages = Pages(self.ks, self.vs, self.hkv, self.block).cuda()
        return self

    def call(self, out, ws=None, stream=None):
        import int8_group_quantized_gb300 as dgq
        ws = self.ws if ws is None else ws
        if self.block is None:
            dgq.dgq_prompt_attn(self.dq, self.k, self.v, self.cu_q, self.cu_kv, out, ws, stream)
        else:
            p = self.pages
            dgq.dgq_prompt_attn_paged(self.dq, self.cu_q, p.k, p.v, p.table, p.lens, out, ws, stream)

    def run(self):
        import int8_group_quantized_gb300 as dgq
        out = torch.full_like(self.dq, 7.0)
        self.call(out)
        torch.cuda.synchronize()
        assert dgq.dgq_workspace_error(self.ws) == 0
        return out

    def check(self, out):
        if self.ref is None:
            self.ref = prompt(self.q, self.ks, self.vs, self.n, self.hq, self.hkv)
        check(out, *self.ref)


def verify(shape, hq, hkv, seed, **kw):
    p = Prompt(shape, hq, hkv, seed, **kw).device()
    p.check(p.run())


WHOLE = [[1], [2, 1], [63, 64, 65], [127, 128, 129], [300, 37], [0, 5, 0, 1, 257, 0], [1000, 511, 513]]


@pytest.mark.parametrize("lens", WHOLE, ids=str)
@pytest.mark.parametrize("block", [None, 16])
def test_whole_prompts(lens, block):
    verify([(n, n) for n in lens], 8, 2, seed=sum(lens), block=block)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (2, 1), (6, 3), (4, 1), (8, 1), (16, 2), (32, 8)])
def test_head_layouts(hq, hkv):
    verify([(70, 70), (5, 200), (129, 140)], hq, hkv, seed=hq * 10 + hkv)
    verify([(70, 70), (5, 200), (129, 140)], hq, hkv, seed=hq * 10 + hkv, block=32)


@pytest.mark.parametrize("block", [None, 16, 32, 64])
def test_chunks_behind_a_history(block):
    verify([(1, 1), (1, 500), (3, 129), (64, 1064), (130, 4000), (17, 128), (128, 256)], 8, 2, seed=9, block=block)


@pytest.mark.parametrize("block", [None, 16])
def test_rows_that_see_no_key_are_zero(block):
    p = Prompt([(10, 3), (300, 1), (200, 0), (5, 0), (400, 129), (4, 4)], 4, 2, seed=3, block=block).device()
    out = p.run()
    p.check(out)
    at = 0
    for n, m in zip(p.n, p.m):
        assert (out[at:at + max(0, n - m)] == 0).all()
        at += n


@pytest.mark.parametrize("block", [None, 64])
def test_few_rows_long_axis(block):
    verify([(1, 20000), (3, 5000), (40, 9001)], 8, 2, seed=5, block=block)
    verify([(1, 33000)], 1, 1, seed=6, block=block)


@pytest.mark.parametrize("lens", [[2500], [1, 3000, 2]])
def test_long_prompts(lens):
    verify([(n, n) for n in lens], 4, 2, seed=8)


@pytest.mark.parametrize("block", [None, 16])
def test_running_maximum_that_keeps_climbing(block):
    # keys grow along the axis, so almost every tile raises the maximum; then shrink
    p = Prompt([(200, 1500), (64, 1400)], 4, 1, seed=12, block=block, q_sigma=2.0)
    for i, up in ((0, True), (1, False)):
        m = p.m[i]
        f = torch.linspace(0.01, 4.0, m) if up else torch.linspace(4.0, 0.01, m)
        p.ks[i] = (p.ks[i].float() * f[:, None, None]).to(torch.bfloat16)
    p.device()
    p.check(p.run())


def test_one_hot_rows_return_the_value_row():
    # a key that matches its query far above the others: the softmax is one weight
    p = Prompt([(256, 256)], 1, 1, seed=13)
    p.ks[0] = (p.q[:, :1].float() * 40).to(torch.bfloat16)
    p.device()
    out = p.run()
    p.check(out)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -3e38])
def test_other_requests_cannot_reach_a_row(bad):
    p = Prompt([(70, 70), (33, 40), (100, 333), (20, 20)], 4, 2, seed=21)
    p.device()
    a, b = p.m[0], p.m[0] + p.m[1]
    p.k[a:b], p.v[a:b] = bad, bad                     # request 1's keys and values
    last = sum(p.m[:3])
    p.k[last:], p.v[last:] = bad, bad                 # and the last request's
    out = p.run()
    ref, bound = prompt(p.q, p.ks, p.vs, p.n, p.hq, p.hkv)
    at = 0
    for i, n in enumerate(p.n):
        if i in (0, 2):
            check(out[at:at + n], ref[at:at + n], bound[at:at + n])
        at += n


@pytest.mark.parametrize("block", [None, 16])
def test_rows_behind_the_last_request_are_left(block):
    p = Prompt([(37, 37), (90, 120)], 4, 2, seed=23, block=block).device()
    tail = torch.full((50, 4, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    p.dq = torch.cat([p.dq, tail])
    if block is None:
        p.k = torch.cat([p.k, tail[:, :2]]).contiguous()
        p.v = torch.cat([p.v, tail[:, :2]]).contiguous()
    out = p.run()
    p.check(out[:127])
    assert (out[127:] == 7.0).all()


@pytest.mark.parametrize("block", [None, 32])
def test_runs_repeat_and_pages_may_move(block):
    p = Prompt([(300, 300), (7, 6000), (65, 2000)], 8, 2, seed=31, block=block).device()
    one = p.run()
    assert torch.equal(one, p.run())
    if block:
        perm = torch.randperm(p.pages.k.shape[0], generator=torch.Generator().manual_seed(1)).cuda()
        k, v = torch.empty_like(p.pages.k), torch.empty_like(p.pages.v)
        k[perm], v[perm] = p.pages.k, p.pages.v
        p.pages.k, p.pages.v, p.pages.table = k, v, perm[p.pages.table.long()].to(torch.int32)
        assert torch.equal(one, p.run())


def test_packed_and_paged_agree_bitwise():
    shape = [(300, 300), (7, 6000), (65, 2000), (1, 1)]
    a = Prompt(shape, 8, 2, seed=33).device().run()
    for block in (16, 32, 64):
        assert torch.equal(a, Prompt(shape, 8, 2, seed=33, block=block).device().run())


def test_many_requests():
    import random
    r = random.Random(4)
    shape = [(r.randint(0, 9), r.randint(0, 40)) for _ in range(700)]
    verify(shape, 2, 1, seed=41)
    verify(shape, 2, 1, seed=41, block=16)


@pytest.mark.parametrize("n", [40, 64, 128, 200])
def test_many_short_units_to_a_block(n):
    # every thread block goes through a dozen units of one to four key tiles, one after the other
    p = Prompt([(n, n)] * (12000 // n), 32, 8, seed=44).device()
    out = p.run()
    per = max(1, len(p.n) // 12)
    for b in list(range(0, len(p.n), per)) + [len(p.n) - 1]:     # a dozen requests are looked at
        ref, bound = prompt(p.q[b * n:(b + 1) * n], p.ks[b:b + 1], p.vs[b:b + 1], [n], 32, 8)
        check(out[b * n:(b + 1) * n], ref, bound)
    assert torch.equal(out, p.run())


def drawn(block, seed=0):
    """A batch whose units are drawn from the counter: 80 requests, some of them empty, the last ones too."""
    g = np.random.default_rng(seed)
    n = [0 if b % 7 == 3 or b >= 76 else int(g.integers(1, 201)) for b in range(80)]
    m = [x + int(g.integers(0, 3)) * 50 - (30 if b % 11 == 0 and x > 40 else 0) for b, x in enumerate(n)]
    return Prompt(list(zip(n, m)), 64, 8, seed=46, block=block)


@pytest.mark.parametrize("block", [None, 16])
def test_units_drawn_from_a_counter(block):
    p = drawn(block).device()
    out = p.run()
    start = np.concatenate([[0], np.cumsum(p.n)])
    for b in list(range(0, 80, 9)) + [33, 75]:
        if p.n[b]:
            lo, hi = int(start[b]), int(start[b + 1])
            ref, bound = prompt(p.q[lo:hi], p.ks[b:b + 1], p.vs[b:b + 1], [p.n[b]], 64, 8)
            check(out[lo:hi], ref, bound)
    for _ in range(3):      # whichever block draws a unit, and however often the counter was used
        assert torch.equal(out, p.run())


def test_drawn_and_sliced_calls_share_a_workspace_and_a_graph():
    a, b = drawn(None).device(), Prompt([(3, 9000), (40, 40)], 64, 8, seed=47).device()
    ra, rb = a.run(), b.run()
    b.check(rb)
    oa, ob = torch.zeros_like(a.dq), torch.zeros_like(b.dq)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for p, o in ((a, oa), (b, ob), (a, oa)):
            p.call(o, a.ws)
    for _ in range(3):
        oa.fill_(7.0)
        ob.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(oa, ra) and torch.equal(ob, rb)
    assert torch.equal(a.run(), ra)


@pytest.mark.parametrize("block", [None, 16])
@pytest.mark.parametrize("shape", [
    [(0, 0)] * 40 + [(5, 300)] + [(0, 7)] * 70 + [(130, 130)] + [(0, 0)] * 500,
    [(0, 0)] * 33 + [(3, 6000)] + [(0, 0)] * 31 + [(2, 5000)] + [(0, 0)] * 32 + [(1, 4000)],
    [(1, 200)] + [(0, 0)] * 63 + [(1, 100)],
], ids=["few", "cut", "ends"])
def test_padded_batches(shape, block):
    # empty requests before, between and behind the others, in runs of more than a warp's lanes
    verify(shape, 8, 2, seed=48, block=block)


def test_drawn_units_of_a_padded_batch():
    shape = [(0, 0)] * 50 + [(n, n) for n in range(150, 200)] + [(0, 0)] * 70 + [(n, n + 9) for n in range(100, 130)] + \
        [(0, 0)] * 900
    p = Prompt(shape, 64, 8, seed=49).device()
    out = p.run()
    start = np.concatenate([[0], np.cumsum(p.n)])
    for b in (50, 75, 99, 170, 199):
        lo, hi = int(start[b]), int(start[b + 1])
        ref, bound = prompt(p.q[lo:hi], p.ks[b:b + 1], p.vs[b:b + 1], [p.n[b]], 64, 8)
        check(out[lo:hi], ref, bound)
    assert not torch.any(torch.all(out == 7.0, dim=-1))  # every row is written


def test_chunks_of_a_prompt_equal_the_whole_within_the_bound():
    # the same prompt in three chunks against the pages written so far
    import int8_group_quantized_gb300 as dgq
    n = 700
    p = Prompt([(n, n)], 8, 2, seed=43, block=16).device()
    out = torch.empty_like(p.dq)
    for a, b in ((0, 256), (256, 257), (257, n)):
        part = torch.empty(b - a, 8, 128, dtype=torch.bfloat16, device="cuda")
        dgq.dgq_prompt_attn_paged(p.dq[a:b], cu([b - a]), p.pages.k, p.pages.v, p.pages.table,
                                  torch.tensor([b], dtype=torch.int32, device="cuda"), part, p.ws)
        out[a:b] = part
    p.check(out)


def test_rows_behind_two_gigabytes():
    # the last pages of pools larger than 2^32 bytes
    import int8_group_quantized_gb300 as dgq
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    p = Prompt([(40, 200)], 4, 2, seed=47, block=64).device()
    blocks = (5 << 30) // (2 * 64 * 256)
    k = torch.empty(blocks, 2, 64, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    n = p.pages.k.shape[0]
    k[-n:], v[-n:] = p.pages.k, p.pages.v
    p.pages.k, p.pages.v, p.pages.table = k, v, p.pages.table + (blocks - n)
    p.check(p.run())


def test_graph_replays_equal_calls():
    for block in (None, 16):
        p = Prompt([(130, 130), (3, 5000)], 8, 2, seed=51, block=block).device()
        want = p.run()
        out = torch.zeros_like(want)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            p.call(out)
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            p.call(out)
        for _ in range(3):
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)


def test_calls_in_a_row_share_a_workspace():
    # calls of different shapes back to back on one stream, no synchronisation between them
    a = Prompt([(3, 9000), (200, 200)], 8, 2, seed=53).device()
    b = Prompt([(64, 64), (1, 7000)], 8, 2, seed=54, block=16).device()
    oa, ob = torch.empty_like(a.dq), torch.empty_like(b.dq)
    ws = a.ws
    for _ in range(4):
        a.call(oa, ws)
        b.call(ob, ws)
    torch.cuda.synchronize()
    a.check(oa)
    b.check(ob)


def test_another_stream_and_threads():
    ps = [Prompt([(130, 130), (3, 5000)], 8, 2, seed=61), Prompt([(700, 900)], 4, 4, seed=62, block=16),
          Prompt([(1, 50)] * 40, 8, 1, seed=63, block=64)]
    for p in ps:
        p.device()
    torch.cuda.synchronize()
    res = [None] * len(ps)

    def work(i):
        try:
            torch.cuda.set_device(0)
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                out = torch.empty_like(ps[i].dq)
                for _ in range(4):
                    ps[i].call(out, stream=s)
            s.synchronize()
            res[i] = out
        except BaseException as e:
            res[i] = e
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(ps))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for p, r in zip(ps, res):
        assert not isinstance(r, BaseException), r
        p.check(r)


def test_device_guards():
    import int8_group_quantized_gb300 as dgq
    bad_block, bad_length = 5, 6
    p = Prompt([(40, 300), (20, 37)], 4, 2, seed=71, block=16).device()
    good = p.pages.table.clone()
    p.pages.k.nan_to_num_(0.0), p.pages.v.nan_to_num_(0.0)
    out = torch.empty_like(p.dq)
    ref, bound = prompt(p.q, p.ks, p.vs, p.n, p.hq, p.hkv)
    for value in (p.pages.k.shape[0] + 7, -1):
        p.pages.table = good.clone()
        p.pages.table[0, 3] = value
        p.call(out)
        assert dgq.dgq_workspace_error(p.ws) == bad_block
        check(out[40:], ref[40:], bound[40:])  # the other request's rows
        dgq.dgq_workspace_init(p.ws)
    p.pages.table = good
    p.pages.lens[1] = good.shape[1] * 16 + 100
    p.call(out)
    assert dgq.dgq_workspace_error(p.ws) == bad_length
    dgq.dgq_workspace_init(p.ws)
    p.pages.lens[1] = 37
    p.check(p.run())
    c = Prompt([(40, 60), (20, 37)], 4, 2, seed=72).device()
    for attr, value in (("cu_q", [0, 40, 75]), ("cu_q", [0, 61, 40]), ("cu_kv", [0, 60, 98]), ("cu_kv", [-1, 60, 97])):
        keep = getattr(c, attr)
        setattr(c, attr, torch.tensor(value, dtype=torch.int32, device="cuda"))
        c.call(torch.empty_like(c.dq))
        assert dgq.dgq_workspace_error(c.ws) == bad_length, (attr, value)
        dgq.dgq_workspace_init(c.ws)
        setattr(c, attr, keep)
    c.check(c.run())

