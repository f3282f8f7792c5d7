"""Long key axes that are cut into slices and merged: inputs on which a lost or doubled key tile shows.

Over a long axis of zero-mean values the output shrinks below the bound of the roundings, so that a check
element by element would not notice a missing part.  Here a tile's values lie in one of the 128 columns
only (tile % 128), all positive, each tile at a level of its own, and head g of a group looks mostly at the
tiles of its own class (tile // 128 % G): an output element is then the mean of the few tiles that share its
column and class, and each of them moves it by far more than the bound.  The first test shows that on the CPU
for every whole tile of every case below: more than twice the bound, so that no rounding within it can hide
the loss.  (On zero-mean values and flat scores the same figure is 0.14 at 20000 keys.)"""
import pytest
import torch

from attn_reference import Pages, attend
from test_gpu_decode_bf16 import Step
from test_gpu_prompt import Prompt

BIAS = 6.0  # component of keys along their class's direction, and of queries along their head's


def marked(m, hkv, g, unit, seed):
    """K, V bf16 [m, hkv, 128] of m keys in tiles of `unit`."""
    gen = torch.Generator().manual_seed(seed)
    tile = torch.arange(m) // unit
    k = torch.randn(m, hkv, 128, generator=gen) * 0.3
    k[torch.arange(m), :, (tile // 128) % g] += BIAS
    v = torch.zeros(m, hkv, 128)
    level = 0.8 + 0.4 * torch.rand((m + unit - 1) // unit, hkv, generator=gen)
    v[torch.arange(m), :, tile % 128] = level[tile] * (1 + 0.1 * torch.randn(m, hkv, generator=gen))
    return k.to(torch.bfloat16), v.to(torch.bfloat16)


def queries(n, hq, hkv, seed):
    gen = torch.Generator().manual_seed(seed)
    q = torch.randn(n, hq, 128, generator=gen) * 0.5
    for h in range(hq):
        q[:, h, h % (hq // hkv)] += BIAS
    return q.to(torch.bfloat16)


# (query rows, keys) per request, query heads, KV heads; key tiles are cut at multiples of 128
PROMPTS = [([(1, 20000), (3, 5000), (40, 9001)], 8, 2), ([(1, 33000)], 1, 1), ([(2, 70001)], 8, 1),
           ([(33, 12345), (1, 129), (64, 40000)], 4, 1)]
# cached keys per request; tiles of 16
DECODES = [([40000, 100], 8, 2, 64), ([70001], 8, 1, 32), ([9000, 17, 3000], 8, 1, 16), ([2500] * 12, 16, 2, 16)]


def marked_prompt(shape, hq, hkv, block=None):
    p = Prompt([(1, 1)], hq, hkv, 0)
    p.n, p.m, p.block = [s[0] for s in shape], [s[1] for s in shape], block
    p.q = queries(sum(p.n), hq, hkv, 7)
    kv = [marked(m, hkv, hq // hkv, 128, 20 + i) for i, m in enumerate(p.m)]
    p.ks, p.vs = [x[0] for x in kv], [x[1] for x in kv]
    return p


def marked_step(lens, hq, hkv, block):
    s = Step([1], hq, hkv, block, 0)
    s.lens = lens
    s.q = queries(len(lens), hq, hkv, 8)
    kv = [marked(n, hkv, hq // hkv, 16, 40 + i) for i, n in enumerate(lens)]
    s.ks, s.vs = [x[0] for x in kv], [x[1] for x in kv]
    new = [marked(1, hkv, hq // hkv, 16, 80 + i) for i in range(len(lens))]
    s.kn, s.vn = torch.cat([x[0] for x in new]), torch.cat([x[1] for x in new])
    s.pages = Pages(s.ks, s.vs, hkv, block)
    return s


def least_trace(qs, k, v, unit):
    """How far a key tile left out, or counted twice, moves the most affected output of the group's heads
    qs [G, 128], in units of that output's bound: the least over all whole tiles."""
    n, tile = k.shape[0], torch.arange(k.shape[0]) // unit
    tiles = int(tile[-1]) + 1
    most = torch.zeros(tiles, dtype=torch.float64)
    out, bound = attend(qs, k, v, torch.full((qs.shape[0],), n))
    for o, e, w in zip(out, bound, torch.softmax(qs @ k.T / 128.0 ** 0.5, dim=1)):
        share = torch.zeros(tiles, dtype=torch.float64).index_add_(0, tile, w)[:, None]
        part = torch.zeros(tiles, 128, dtype=torch.float64).index_add_(0, tile, w[:, None] * v)
        for x in ((o - part) / (1 - share), (o + part) / (1 + share)):
            most = torch.maximum(most, ((x - o).abs() / e.clamp(min=1e-300)).max(dim=1).values)
    return float(most[torch.bincount(tile) == unit].min())


@pytest.mark.parametrize("case", range(len(PROMPTS)))
def test_every_key_tile_of_the_prompts_shows(case):
    p = marked_prompt(*PROMPTS[case])
    g, at = p.hq // p.hkv, 0
    for n, m, k, v in zip(p.n, p.m, p.ks, p.vs):
        for i in sorted({0, n - 1}):
            for h in range(p.hkv):
                seen = m - n + i + 1
                t = least_trace(p.q[at + i, h * g:(h + 1) * g].double(), k[:seen, h].double(), v[:seen, h].double(), 128)
                assert t > 2.0, (n, m, i, h, t)
        at += n


@pytest.mark.parametrize("case", range(len(DECODES)))
def test_every_key_tile_of_the_decode_steps_shows(case):
    s = marked_step(*DECODES[case])
    g = s.hq // s.hkv
    for b in range(len(s.lens)):
        for h in range(s.hkv):
            k, v = (torch.cat([x[b][:, h], y[b, h][None]]).double() for x, y in ((s.ks, s.kn), (s.vs, s.vn)))
            t = least_trace(s.q[b, h * g:(h + 1) * g].double(), k, v, 16)
            assert t > 2.0, (s.lens[b], h, t)


@pytest.mark.gpu
@pytest.mark.parametrize("block", [None, 16, 64])
@pytest.mark.parametrize("case", range(len(PROMPTS)))
def test_prompts(case, block):
    p = marked_prompt(*PROMPTS[case], block=block).device()
    p.check(p.run())


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(DECODES)))
def test_decode_steps(case):
    s = marked_step(*DECODES[case]).device()
    s.check(s.run())
