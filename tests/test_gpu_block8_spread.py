"""Decode over 8-bit block caches whose V scales lie as far apart as the cache allows: what a token weighs in the
softmax depends on its score alone, so blocks of zeros and blocks of small values keep their share of the
sum beside blocks of large ones -- in one warp (a warp takes every fourth tile of 16 tokens), in the merge of
warps, and in the merge of pieces."""
import pytest
import torch

from attn_reference import rows
from test_gpu_block8 import FMT, TOP, Step, slots_of

pytestmark = pytest.mark.gpu

# which of a request's tiles of 16 tokens hold the large values
PLACES = {
    "in a warp": lambda tile, tiles: tile // 4 % 2 == 1,
    "in a warp, large ones first": lambda tile, tiles: tile // 4 % 2 == 0,
    "across warps": lambda tile, tiles: tile % 2 == 1,
    "across pieces": lambda tile, tiles: 2 * tile >= tiles,
    "one tile of large ones": lambda tile, tiles: tile == tiles // 2,
    "one tile of small ones": lambda tile, tiles: tile != tiles // 2,
}


def step(fmt, n, place, small, large, scores):
    """Values of size `small` and `large`; all scores 0, or of ordinary size."""
    s = Step(fmt, [n], 4, 1, 16, 90)
    tile = torch.arange(n) // 16
    size = torch.where(PLACES[place](tile, (n + 15) // 16), large, small).float()
    k = rows(n, 1, 91, 1.0) if scores else torch.zeros(n, 1, 128, dtype=torch.bfloat16)
    v = (rows(n, 1, 92, 1.0).float() * size[:, None, None]).to(torch.bfloat16)
    s.c.store(k, v, slots_of(s.table[0], 16, 0, n))
    s.vn[:] = 0
    if not scores:
        s.kn[:] = 0
    return s


@FMT
@pytest.mark.parametrize("place", list(PLACES))
@pytest.mark.parametrize("small,large", [(0.0, 2.0 ** 27), (0.0, 2.0 ** 40), (0.0, 2.0 ** 97), (2.0 ** -76, 2.0 ** 60),
                                         (2.0 ** -70, 2.0 ** 97)])
@pytest.mark.parametrize("n", [128, 333, 20000])
def test_scales_far_apart(fmt, place, small, large, n):
    for scores in (False, True):
        s = step(fmt, n, place, small, large, scores)
        s.check(s.run())


@FMT
@pytest.mark.parametrize("place", ["in a warp", "across warps", "across pieces"])
def test_scales_far_apart_in_a_window(fmt, place):
    for n, window, sinks in ((300, 200, 20), (20000, 9000, 2000)):
        s = step(fmt, n, place, 0.0, 2.0 ** 60, True)
        s.check(s.run(window, sinks), window, sinks)


@FMT
def test_equal_scores_share_the_sum_equally(fmt):
    """Eight tiles of which half hold zeros, equal scores: half of the large value, less the new token's share."""
    for place in ("in a warp", "across warps"):
        s = step(fmt, 128, place, 0.0, 1.0, False)
        tile = torch.arange(128) // 16
        top = TOP[fmt] * 2.0 ** 33                              # (the largest code, its scale 2^33)
        v = torch.where(PLACES[place](tile, 8), top, 0.0).to(torch.bfloat16)[:, None, None].expand(128, 1, 128)
        s.c.store(torch.zeros(128, 1, 128, dtype=torch.bfloat16), v, slots_of(s.table[0], 16, 0, 128))
        want = 64 / 129 * top
        # weights and their sum 2^-11 each, the output 2^-8, INT8's offset of 1152 behind 144 sums 2^-12
        assert ((s.run().cpu().double() - want).abs() <= want * (2.0 ** -8 + 2.0 ** -9)).all()
