"""Decode with windows and over 8-bit block caches for the batches in which the work is split in other ways than
for a few requests: more than 32 requests (starts searched for in shared memory), 64 and more pairs of a request
and a KV head with up to 40 tiles each (taken whole), more short pairs than there are blocks of threads
(several whole pairs to one), and long ones (cut and merged).  Against plain attention in 64 bits, and twice
for the same bits."""
import numpy as np
import pytest
import torch

from attn_reference import check
from dgq_cases import Case, table_to_numpy
from test_gpu_block8 import FMT
from test_gpu_block8 import Step as Block8Step
from test_gpu_window import WindowStep
from window_reference import attend, visible

pytestmark = pytest.mark.gpu


def ragged(batch, top, seed):
    """`batch` lengths up to `top`, 0 and 1 and `top` itself among them."""
    lens = np.random.default_rng(seed).integers(0, top + 1, batch)
    lens[[0, batch // 2, batch - 1]] = 1, top, 0
    return lens.tolist()


# (lengths, KV heads): cut and merged; whole pairs of 25 to 40 tiles; several whole pairs to a block of threads
BATCHES = {
    "32 cut": (ragged(32, 1500, 1), 2),
    "33 cut": (ragged(33, 1500, 2), 2),
    "130 cut": (ragged(130, 1000, 3), 1),
    "64 pairs whole": (ragged(32, 640, 4), 2),
    "66 pairs whole": (ragged(66, 630, 5), 1),
    "600 pairs whole": (ragged(200, 500, 6), 3),
    "one end long": ([16] * 150 + ragged(50, 500, 7), 3),
}
ALL = pytest.mark.parametrize("batch", list(BATCHES))


@FMT
@ALL
@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 20), (90, 3)])
def test_block_caches(fmt, batch, window, sinks):
    lens, hkv = BATCHES[batch]
    s = Block8Step(fmt, lens, 4 * hkv, hkv, 16, len(lens))
    out = s.run(window, sinks)
    s.check(out, window, sinks)
    assert torch.equal(out, s.run(window, sinks))


@ALL
@pytest.mark.parametrize("window,sinks", [(700, 20), (90, 3)])
def test_bf16_windows(batch, window, sinks):
    lens, hkv = BATCHES[batch]
    s = WindowStep(lens, 2 * hkv, hkv, 32, len(lens), window, sinks).device()
    out = s.run()
    s.check(out)
    assert torch.equal(out, s.run())


def check_int8(case, out, window, sinks):
    table = table_to_numpy(case.d_table)
    kp, vp = case.d_kp.cpu().numpy(), case.d_vp.cpu().numpy()
    q, kn, vn = (x.cpu().double() for x in (case.d_q, case.d_knew, case.d_vnew))
    bt, g = case.d_bt.cpu().numpy(), case.hq // case.hkv
    ref = torch.zeros(case.B, case.hq, 128, dtype=torch.float64)
    bound = torch.zeros_like(ref)
    for b, n in enumerate(case.lens.tolist()):
        t = np.arange(n)
        blk = bt[b][t // case.bs]
        for h in range(case.hkv):
            r, s = table[b, h], slice(h * g, (h + 1) * g)
            seg = np.searchsorted(r["start"][:max(int(r["n_seg"]), 1)], t, side="right") - 1
            of = lambda name: r[name][seg].astype(np.float64)
            k, v = (torch.from_numpy(of(x + "_min")[:, None] + p[blk, h, t % case.bs].astype(np.float64) * of(x + "_scale")[:, None])
                    for x, p in (("k", kp), ("v", vp)))
            # (what accumulates: 1024 + code times the step, and the smallest value less 1024 steps)
            size = [torch.from_numpy(2048.0 * of(x + "_scale") + np.abs(of(x + "_min"))) for x in "kv"]
            pad = lambda x: torch.cat([x, torch.zeros(1, dtype=torch.float64)])
            ref[b, s], bound[b, s] = attend(
                q[b, s], torch.cat([k, kn[b, h][None]]), torch.cat([v, vn[b, h][None]]),
                visible(torch.full((g,), n), n + 1, window, sinks), weight_unit=2.0 ** -11, k_size=pad(size[0]),
                v_size=pad(size[1]), v_scale=torch.full((n + 1,), float(r["v_scale"].max()), dtype=torch.float64), top=1280.0)
    check(out, ref, bound)


def int8_window(lens, hq, hkv, bs, window, sinks):
    import int8_group_quantized_gb300 as dgq
    case = Case(lens, hq=hq, hkv=hkv, bs=bs, seed=3, rule=1)
    case.gpu_compress()
    case.gpu_attn()
    ws = torch.zeros(dgq.dgq_attn_workspace_size(case.B, hq, hkv, case.max_seqlen), dtype=torch.uint8, device="cuda")
    outs = []
    for _ in range(2):
        outs.append(torch.zeros(case.B, hq, 128, dtype=torch.bfloat16, device="cuda"))
        dgq.dgq_paged_decode_attn(case.d_q, case.d_knew, case.d_vnew, case.d_kp, case.d_vp, case.d_table, case.d_bt,
                                  case.d_lens, case.max_seqlen, outs[-1], ws, window=window, sinks=sinks)
        torch.cuda.synchronize()
        assert dgq.dgq_workspace_error(ws) == 0
    check_int8(case, outs[0], window, sinks)
    assert torch.equal(*outs)


@ALL
@pytest.mark.parametrize("window,sinks", [(700, 20), (90, 3)])
def test_int8_windows(batch, window, sinks):
    lens, hkv = BATCHES[batch]
    int8_window(lens, 2 * hkv, hkv, 16, window, sinks)


@pytest.mark.parametrize("bs", [16, 32, 64])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (6, 3), (8, 4), (12, 3), (8, 1)])
def test_int8_windows_of_other_blocks_and_groups(bs, hq, hkv):
    for window, sinks in ((33, 17), (500, 64)):
        int8_window([0, 1, 37, 300, 2100, 640], hq, hkv, bs, window, sinks)
