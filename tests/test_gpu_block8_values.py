"""Values that the 8-bit block cache cannot hold leave a trace: they are flagged, and an infinite or NaN one makes the
scale of its block and head NaN, so that rows and attention that read it are NaN, and nothing else is."""
import numpy as np
import pytest
import torch

from test_gpu_block8 import FMT, Cache, Step, i32, slots_of, tokens

pytestmark = pytest.mark.gpu
BAD_VALUE = 8
NAN, INF = float("nan"), float("inf")


def same(a, b):
    """Equal to the bit (NaN scales too)."""
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


@FMT
@pytest.mark.parametrize("bs", [16, 32, 64])
@pytest.mark.parametrize("value", [NAN, -NAN, INF, -INF])
@pytest.mark.parametrize("which", [0, 1])
def test_store_and_load(fmt, bs, value, which):
    import int8_group_quantized_gb300 as dgq
    hkv, n = 3, 300
    clean, c = (Cache(fmt, n // bs + 2, hkv, bs) for _ in range(2))
    order = np.random.default_rng(bs).permutation(n // bs + 2)
    slots = slots_of(order, bs, 0, n)
    x = [tokens(n, hkv, 1), tokens(n, hkv, 2)]
    clean.store(*x, slots)
    clean.verify()
    at, h = 7 * bs // 2 + 5, 1                              # in the fourth block, as its only bad value
    block = int(order[at // bs])
    x[which][at, h, 77] = value
    dgq.dgq_store_block8(fmt, x[0].cuda(), x[1].cuda(), i32(slots), *c.d_codes, *c.d_scales, c.ws)
    assert dgq.dgq_workspace_error(c.ws) == BAD_VALUE
    assert torch.isnan(c.d_scales[which][block, h])
    rows = [torch.zeros(n, hkv, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    table = i32(order[None, :-(-n // bs)])
    c.ws.zero_()
    dgq.dgq_load_block8(fmt, *c.d_codes, *c.d_scales, table, i32([0, n]), *rows, c.ws)
    nan = torch.isnan(rows[which]).cpu()
    first = at // bs * bs
    assert nan[first:first + bs, h].all() and int(nan.sum()) == bs * 128 and not torch.isnan(rows[1 - which]).any()

    # a token that joins the block does not hide it
    c.d_scales[which][block, h] = NAN
    one = tokens(1, hkv, 3)
    dgq.dgq_store_block8(fmt, one.cuda(), one.cuda(), i32([block * bs + bs - 1]), *c.d_codes, *c.d_scales, c.ws)
    assert dgq.dgq_workspace_error(c.ws) == 0 and torch.isnan(c.d_scales[which][block, h])
    # everything else is as without the value, and a run from the first place on starts the block anew
    again = [tokens(bs, hkv, 4), tokens(bs, hkv, 5)]
    for cache in (clean, c):
        dgq.dgq_store_block8(fmt, again[0].cuda(), again[1].cuda(), i32(block * bs + np.arange(bs)), *cache.d_codes,
                             *cache.d_scales, cache.ws)
        assert dgq.dgq_workspace_error(cache.ws) == 0
    assert same((*c.d_codes, *c.d_scales), (*clean.d_codes, *clean.d_scales))


@FMT
def test_values_of_2_to_the_100_are_stored_and_flagged(fmt):
    import int8_group_quantized_gb300 as dgq
    for size, error in ((1.9921875 * 2.0 ** 99, 0), (2.0 ** 100, BAD_VALUE), (2.0 ** 120, BAD_VALUE)):
        c = Cache(fmt, 4, 2, 16)
        x = tokens(40, 2, 6)
        x[20, 1, 5] = -size
        c.store(x, x, list(range(40)))
        assert dgq.dgq_workspace_error(c.ws) == error
        c.ws.zero_()
        c.verify()


@FMT
@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("lens", [[9, 33, 0], [700, 16, 120], [20000, 5, 64]])
def test_attention_shows_it(fmt, value, which, lens):
    """In the first tile, a tile inside, the last one: NaN for the heads that read the block, nothing else changed."""
    import int8_group_quantized_gb300 as dgq
    hkv, bs = 2, 16
    n = lens[0]
    for at in sorted({0, n // 2, n - 1}):
        s = Step(fmt, lens, 4, hkv, bs, 60)
        want = s.run()
        first = at // bs * bs
        x = [tokens(min(bs, n - first), hkv, 62), tokens(min(bs, n - first), hkv, 63)]   # (the block anew)
        x[which][at - first, 1, 3] = value
        t = i32(slots_of(s.table[0], bs, first, min(n, first + bs)))
        dgq.dgq_store_block8(fmt, x[0].cuda(), x[1].cuda(), t, *s.c.d_codes, *s.c.d_scales, s.c.ws)
        assert dgq.dgq_workspace_error(s.c.ws) == BAD_VALUE
        out = s.run()
        assert torch.isnan(out[0, 2:]).all() and not torch.isnan(out[0, :2]).any()
        assert torch.equal(out[1:], want[1:])
        if n > 500 and 64 <= at < n - 300:                  # outside the window: not read
            assert not torch.isnan(s.run(200, 16)).any()
        elif n > 500:
            assert torch.isnan(s.run(200, 16)[0, 2:]).all()
