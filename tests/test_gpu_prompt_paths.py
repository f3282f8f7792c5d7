"""Both ways prompt attention hands out its units, each shown to be the one that ran (the workspace header
says which): units drawn from a counter, and equal slices with blocks that finish several pieces and then
end inside another unit, whose parts are merged.  All rows against plain attention in 64 bits."""
import functools

import numpy as np
import pytest
import torch

from attn_reference import prompt
from test_gpu_prompt import Prompt, drawn

DRAWN, SLICED = 5, 6
UNIT_COST, LONE = 160, 104  # the kernel's cost of a unit in keys, and of 128 keys where a unit has one tile only


def units(shape, hq, hkv):
    """Costs of the units of one KV head and request after request, in the kernel's measure."""
    u = 256 // (hq // hkv)
    out = []
    for n, m in shape:
        for i in range(0, n, u):
            keys = max(0, m - n + min(n, i + u))
            out.append(UNIT_COST + (keys * LONE // 128 if n - i <= u // 2 else keys))
    return out


def mixed(ratio, seed, place, blocks, hq, hkv):
    """Requests whose units' cost is `ratio` of the longest unit a block: short prompts, turns of a few rows
    behind some hundred to some thousand keys, and one long turn at `place` of the list."""
    g = np.random.default_rng(seed)
    longest = (5, 6000)
    shape, total, goal = [], sum(units([longest], hq, hkv)), ratio * blocks * (longest[1] + UNIT_COST) / hkv
    while total < goal:
        kind = g.random()
        if kind < 0.5:
            n = int(g.integers(1, 130))
            s = (n, n)
        elif kind < 0.9:
            s = (int(g.integers(1, 70)), int(g.integers(500, 2500)))
        else:
            s = (0, int(g.integers(0, 50)))
        s = (s[0], max(s))
        shape.append(s)
        total += sum(units([s], hq, hkv))
    shape.insert(int(place * len(shape)), longest)
    return shape


@functools.lru_cache(maxsize=1)
def mixed_prompt(ratio, place, blocks):
    """Inputs and reference, the same for packed rows and pages of any size."""
    p = Prompt(mixed(ratio, 7, place, blocks, 8, 2), 8, 2, seed=77)
    p.ref = prompt(p.q, p.ks, p.vs, p.n, p.hq, p.hkv)
    return p


def path(p):
    return int(p.ws[4:8].view(torch.int32)[0])


def ends_inside(p, blocks):
    """Blocks that finish other pieces and then end inside a unit (their part goes to their second slot)."""
    return int((p.ws[256:256 + 16 * blocks].view(torch.int32).view(blocks, 4)[:, 0] == 2).sum())


@pytest.mark.parametrize("ratio", [1.0, 1.7, 2.5])
def test_mixed_batches_give_every_block_several_units(ratio):
    shape = mixed(ratio, 1, 0.5, 152, 8, 2)
    assert len(units(shape, 8, 2)) * 2 / 152 >= 5 * ratio
    assert 0.98 * ratio < sum(units(shape, 8, 2)) * 2 / 152 / 6160 < 1.05 * ratio


@pytest.mark.gpu
@pytest.mark.parametrize("block", [None, 16, 64])
@pytest.mark.parametrize("ratio,place", [(1.0, 0.5), (1.7, 0.0), (2.5, 1.0)])
def test_slices_of_many_pieces(ratio, place, block):
    blocks = torch.cuda.get_device_properties(0).multi_processor_count
    p = mixed_prompt(ratio, place, blocks)
    p.block = block
    p.device()
    out = p.run()
    assert path(p) == SLICED and ends_inside(p, blocks) >= blocks // 4
    p.check(out)
    for _ in range(2):
        assert torch.equal(out, p.run())


@pytest.mark.gpu
@pytest.mark.parametrize("block", [None, 16])
def test_drawn_batches_are_drawn(block):
    p = drawn(block).device()
    out = p.run()
    assert path(p) == DRAWN
    p.check(out)


@pytest.mark.gpu
@pytest.mark.parametrize("last", [False, True])
def test_drawn_batch_with_its_longest_request_last(last):
    # whichever request is handed out last, and however long its units are
    shape = [(200, 200)] * 130 + [(40, 1200)]
    p = Prompt(shape if last else shape[::-1], 32, 8, seed=78).device()
    out = p.run()
    assert path(p) == DRAWN
    p.check(out)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [[(1, 20000), (3, 5000), (40, 9001)], [(1, 33000)], [(2500, 2500)], [(1, 1)]], ids=str)
def test_few_requests_are_sliced(shape):
    p = Prompt(shape, 8, 2, seed=79).device()
    p.check(p.run())
    assert path(p) == SLICED
