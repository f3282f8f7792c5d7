"""Attention with a sliding window and sinks against plain attention in 64 bits: prompts over packed rows and
pages, decode steps over bf16 pages and the INT8 cache; windows that end at every place of a tile, windows
larger than a request, rows that see nothing, blocks that were given back."""
import numpy as np
import pytest
import torch

from attn_reference import Pages, check, rows
from dgq_cases import Case, table_to_numpy
from test_gpu_decode_bf16 import Step
from test_gpu_prompt import Prompt
from window_reference import attend, visible

pytestmark = pytest.mark.gpu

# ---- prompts ----------------------------------------------------------------------------------------------


class WindowPrompt(Prompt):
    def __init__(self, shape, hq, hkv, seed, window, sinks, **kw):
        super().__init__(shape, hq, hkv, seed, **kw)
        self.limits = dict(window=window, sinks=sinks)

    def call(self, out, ws=None, stream=None):
        import int8_group_quantized_gb300 as dgq
        ws = self.ws if ws is None else ws
        if self.block is None:
            dgq.dgq_prompt_attn(self.dq, self.k, self.v, self.cu_q, self.cu_kv, out, ws, stream, **self.limits)
        else:
            p = self.pages
            dgq.dgq_prompt_attn_paged(self.dq, self.cu_q, p.k, p.v, p.table, p.lens, out, ws, stream, **self.limits)

    def check(self, out):
        g, at = self.hq // self.hkv, 0
        ref = torch.zeros(self.q.shape, dtype=torch.float64)
        bound = torch.zeros_like(ref)
        for n, m, k, v in zip(self.n, self.m, self.ks, self.vs):
            seen = visible(m - n + torch.arange(n), m, **self.limits)
            for h in range(self.hq):
                ref[at:at + n, h], bound[at:at + n, h] = attend(
                    self.q[at:at + n, h].double(), k[:, h // g].double(), v[:, h // g].double(), seen)
            at += n
        check(out, ref, bound)

    def forget(self):
        """Blocks that no row sees are given back: their entries name no block, their contents are NaN."""
        p, w, s = self.pages, self.limits["window"], self.limits["sinks"]
        table = p.table.clone()
        for b, (n, m) in enumerate(zip(self.n, self.m)):
            low = max(m - n + 1 - w, 0)
            for c in range(table.shape[1]):
                if c * self.block >= s and (c + 1) * self.block <= low or c * self.block >= m:
                    if c * self.block < m:
                        p.k[table[b, c].long()], p.v[table[b, c].long()] = float("nan"), float("nan")
                    table[b, c] = 10 ** 6 + c
        p.table = table
        return self


def verify(*a, **kw):
    p = WindowPrompt(*a, **kw).device()
    out = p.run()
    p.check(out)
    return p, out


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 0), (64, 4), (127, 0), (128, 128), (129, 1), (300, 130), (4000, 9)])
@pytest.mark.parametrize("block", [None, 16])
def test_whole_prompts(window, sinks, block):
    verify([(n, n) for n in (1, 2, 63, 129, 0, 600, 257)], 4, 2, window + sinks, window, sinks, block=block)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (4, 2), (8, 2), (8, 1)])
def test_group_sizes(hq, hkv):
    verify([(700, 700), (130, 900), (5, 1000)], hq, hkv, hq + hkv, 200, 10)


@pytest.mark.parametrize("window,sinks", [(1, 0), (40, 0), (100, 4), (256, 64), (257, 200), (3000, 0)])
@pytest.mark.parametrize("block", [None, 64])
def test_chunks_behind_a_history(window, sinks, block):
    verify([(1, 1500), (64, 64), (200, 1333), (3, 0), (300, 40), (129, 2000), (17, 1024)], 4, 2, window, window, sinks, block=block)


@pytest.mark.parametrize("window", range(120, 137))
def test_windows_that_end_at_every_place_of_a_tile(window):
    verify([(300, 700)], 8, 1, window, window, 3, block=16)


@pytest.mark.parametrize("block", [16, 32, 64])
@pytest.mark.parametrize("window,sinks", [(50, 0), (200, 20), (64, 64)])
def test_blocks_given_back_are_not_read(block, window, sinks):
    p = WindowPrompt([(40, 2000), (1, 700), (300, 1100)], 4, 2, block, window, sinks, block=block).device()
    out = p.run()
    p.check(out)
    p.forget()
    assert torch.equal(out, p.run())


def test_a_window_over_everything_gives_the_causal_result():
    for block in (None, 32):
        p = WindowPrompt([(500, 500), (100, 900)], 8, 2, 3, 1 << 30, 0, block=block).device()
        q = Prompt([(500, 500), (100, 900)], 8, 2, 3, block=block).device()
        assert torch.equal(p.run(), q.run())


def test_units_drawn_and_units_cut():
    """Many units (drawn one by one) and few behind a long window (cut between blocks of threads and merged)."""
    import int8_group_quantized_gb300 as dgq
    seen = set()
    for shape, hq, hkv, w, s in (([(700, 700)] * 16, 8, 8, 64, 4), ([(20, 9000), (3, 9000)], 8, 1, 7000, 300),
                                 ([(300, 300)] * 90, 8, 8, 64, 4)):
        p, out = verify(shape, hq, hkv, 11, w, s)
        seen.add(int(p.ws[4:8].view(torch.int32)[0]))
        assert torch.equal(out, p.run())
    assert seen == {5, 6}


def test_packed_and_paged_agree_and_replay():
    shape = [(300, 1000), (1, 77), (513, 513)]
    a, out = verify(shape, 8, 2, 12, 150, 20)
    b, paged = verify(shape, 8, 2, 12, 150, 20, block=16)
    assert torch.equal(out, paged)
    got = torch.zeros_like(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.call(got)
    for _ in range(2):
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, out)


def test_rows_that_see_nothing_are_zero():
    p, out = verify([(200, 30), (5, 0)], 4, 2, 13, 8, 2)
    assert not out[:170].any() and not out[200:].any()


# ---- decode over bf16 pages ---------------------------------------------------------------------------------

class WindowStep(Step):
    def __init__(self, lens, hq, hkv, block, seed, window, sinks, **kw):
        super().__init__(lens, hq, hkv, block, seed, **kw)
        self.limits = dict(window=window, sinks=sinks)

    def call(self, out):
        import int8_group_quantized_gb300 as dgq
        p = self.pages
        dgq.dgq_paged_decode_attn_bf16(*self.d, p.k, p.v, p.table, p.lens, self.max, out, self.ws, **self.limits)

    def check(self, out):
        g = self.hq // self.hkv
        ref = torch.zeros(len(self.lens), self.hq, 128, dtype=torch.float64)
        bound = torch.zeros_like(ref)
        for b, n in enumerate(self.lens):
            for h in range(self.hkv):
                s = slice(h * g, (h + 1) * g)
                k, v = (torch.cat([x[b][:, h], y[b, h][None]]).double() for x, y in ((self.ks, self.kn), (self.vs, self.vn)))
                ref[b, s], bound[b, s] = attend(self.q[b, s].double(), k, v, visible(torch.full((g,), n), n + 1, **self.limits))
        check(out, ref, bound)


LENS = [0, 1, 15, 16, 17, 64, 100, 127, 128, 129, 1000, 3001]


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (1, 40), (2, 0), (16, 0), (17, 16), (33, 5), (128, 100), (1000, 3), (9999, 0)])
@pytest.mark.parametrize("hq,hkv,block", [(8, 2, 16), (3, 3, 64)])
def test_decode(window, sinks, hq, hkv, block):
    s = WindowStep(LENS, hq, hkv, block, window, window, sinks).device()
    out = s.run()
    s.check(out)
    assert torch.equal(out, s.run())


def test_decode_windows_that_end_at_every_place_of_a_tile():
    for window in range(20, 38):
        s = WindowStep([200, 211], 8, 1, 32, window, window, 2).device()
        s.check(s.run())


def test_decode_window_over_everything_gives_the_whole_result():
    a = WindowStep([3000, 70, 0, 900], 8, 2, 32, 14, 1 << 30, 0).device()
    b = Step([3000, 70, 0, 900], 8, 2, 32, 14).device()
    assert torch.equal(a.run(), b.run())


def test_decode_of_the_new_token_alone():
    s = WindowStep([0, 7, 640], 4, 2, 16, 15, 1, 0).device()
    assert torch.equal(s.run().cpu(), s.vn.repeat_interleave(2, dim=1))


@pytest.mark.parametrize("window,sinks", [(40, 0), (200, 20), (16, 16)])
def test_decode_blocks_given_back_are_not_read(window, sinks):
    s = WindowStep([2000, 64, 700, 33], 8, 2, 16, 16, window, sinks).device()
    out = s.run()
    s.check(out)
    p = s.pages
    for b, n in enumerate(s.lens):
        low = max(n + 1 - window, 0)
        for c in range(p.table.shape[1]):
            if (c * 16 >= sinks and (c + 1) * 16 <= low) or c * 16 >= n:
                if c * 16 < n:
                    p.k[p.table[b, c].long()], p.v[p.table[b, c].long()] = float("nan"), float("nan")
                p.table[b, c] = -5 - c
    assert torch.equal(out, s.run())


def test_decode_long_windows_are_split():
    s = WindowStep([40000, 100, 9000], 8, 2, 64, 17, 30000, 70).device()
    s.check(s.run())


# ---- decode over the INT8 cache -------------------------------------------------------------------------------

@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 0), (64, 16), (700, 40), (1 << 30, 0)])
def test_decode_int8(window, sinks):
    import int8_group_quantized_gb300 as dgq
    case = Case([0, 37, 300, 2100, 640], hq=8, hkv=2, bs=16, seed=1, rule=1)
    case.gpu_compress()
    case.gpu_attn()
    out = torch.zeros(5, 8, 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(dgq.dgq_attn_workspace_size(5, 8, 2, 2100), dtype=torch.uint8, device="cuda")
    dgq.dgq_paged_decode_attn(case.d_q, case.d_knew, case.d_vnew, case.d_kp, case.d_vp, case.d_table, case.d_bt,
                              case.d_lens, 2100, out, ws, window=window, sinks=sinks)
    torch.cuda.synchronize()
    assert dgq.dgq_workspace_error(ws) == 0
    if window == 1 << 30:
        assert torch.equal(out, case.d_out)
        return
    table = table_to_numpy(case.d_table)
    kp, vp = case.d_kp.cpu().numpy(), case.d_vp.cpu().numpy()
    q, kn, vn = (x.cpu().double() for x in (case.d_q, case.d_knew, case.d_vnew))
    bt = case.d_bt.cpu().numpy()
    ref = torch.zeros(5, 8, 128, dtype=torch.float64)
    bound = torch.zeros_like(ref)
    for b, n in enumerate(case.lens):
        t = np.arange(n)
        for h in range(2):
            r = table[b, h]
            seg = np.searchsorted(r["start"][:max(int(r["n_seg"]), 1)], t, side="right") - 1
            k, v = (torch.from_numpy(r[x + "_min"][seg].astype(np.float64)[:, None] + p[bt[b][t // 16], h, t % 16].astype(np.float64)
                                     * r[x + "_scale"][seg].astype(np.float64)[:, None]) for x, p in (("k", kp), ("v", vp)))
            # (what accumulates: 1024 + code times the step, and the smallest value less 1024 steps)
            size = [torch.from_numpy(2048.0 * r[x + "_scale"][seg].astype(np.float64) + np.abs(r[x + "_min"][seg])) for x in "kv"]
            pad = lambda x: torch.cat([x, torch.zeros(1, dtype=torch.float64)])
            ref[b, 4 * h:4 * h + 4], bound[b, 4 * h:4 * h + 4] = attend(
                q[b, 4 * h:4 * h + 4], torch.cat([k, kn[b, h][None]]), torch.cat([v, vn[b, h][None]]),
                visible(torch.full((4,), n), n + 1, window, sinks), weight_unit=2.0 ** -11, k_size=pad(size[0]),
                v_size=pad(size[1]), v_scale=torch.full((n + 1,), float(r["v_scale"].max()), dtype=torch.float64), top=1280.0)
    check(out, ref, bound)
