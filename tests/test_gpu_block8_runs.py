"""A block of the 8-bit cache belongs to one run of tokens in a call.  What else comes for it within 64 tokens (a
slot named twice, a dropped token, interleaved requests) is flagged and left out; the rest of the call is
stored as if it had not been there."""
import numpy as np
import pytest
import torch

from test_gpu_block8 import FMT, Cache, i32, slots_of, tokens

pytestmark = pytest.mark.gpu
SPLIT = 7


def keep(slots, bs, back=64):
    """The slots with -1 for every run whose block one of the `back` tokens in front of it names."""
    out, t = list(slots), 0
    while t < len(slots):
        n = 1
        if slots[t] >= 0:
            while t + n < len(slots) and slots[t + n] == slots[t] + n and (slots[t] + n) % bs:
                n += 1
            if any(s >= 0 and s // bs == slots[t] // bs for s in slots[max(0, t - back):t]):
                out[t:t + n] = [-1] * n
        t += n
    return out


def verify(c, slots, hkv, seed):
    import int8_group_quantized_gb300 as dgq
    k, v = tokens(len(slots), hkv, seed), tokens(len(slots), hkv, seed + 1)
    kept = keep(slots, c.bs)
    dgq.dgq_store_block8(c.fmt, k.cuda(), v.cuda(), i32(slots), *c.d_codes, *c.d_scales, c.ws)
    torch.cuda.synchronize()
    assert dgq.dgq_workspace_error(c.ws) == (0 if kept == list(slots) else SPLIT)
    c.ws.zero_()
    host = [x.clone() for x in (*c.d_codes, *c.d_scales)]    # what the call left, against the kept tokens alone
    c.store(k, v, kept)
    c.verify()
    for a, b in zip(host, (*c.d_codes, *c.d_scales)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


CASES = {
    "dropped": [5, -1, 6],
    "dropped, more tokens behind": [3, 4, -1, -1, 7, 8, 9, 40, 41],
    "twice": [5, 5],
    "twice in a run": [5, 6, 6, 7],
    "first place twice": [0, 0],
    "first place again behind a run": [0, 1, 2, 0, 1],
    "interleaved": [0, 16, 32, 1, 17, 33, 2, 18, 34],
    "down": [9, 8, 7, 6],
    "64 apart": [5] + [64 + 16 * i for i in range(63)] + [6],
    "neighbours": [15, 16, 17, 31, 32, -1, -1, 48, 64],
    "other blocks between": [5, 64, 6, 80, 7, 81],
}


@FMT
@pytest.mark.parametrize("name", list(CASES))
@pytest.mark.parametrize("hkv", [1, 3, 8])
def test_runs(fmt, name, hkv):
    c = Cache(fmt, 80, hkv, 16)
    full = list(range(80 * 16))
    c.store(tokens(len(full), hkv, 1), tokens(len(full), hkv, 2), full)
    verify(c, CASES[name], hkv, 3)


@FMT
@pytest.mark.parametrize("bs", [16, 32, 64])
@pytest.mark.parametrize("hkv", [1, 8])
def test_tokens_dropped_from_long_calls(fmt, bs, hkv):
    """Prompts and steps large enough for every window of slots, tokens dropped at all places of it."""
    n = 6000
    blocks = n // bs + 2
    order = np.random.default_rng(bs).permutation(blocks)
    slots = slots_of(order, bs, 0, n)
    c = Cache(fmt, blocks, hkv, bs)
    c.store(tokens(n, hkv, 5), tokens(n, hkv, 6), slots)
    dropped = [-1 if t % 131 == 7 else s for t, s in enumerate(slots)]
    verify(c, dropped, hkv, 7)
    # a decode step (behind tokens that are there) that names every 50th block twice, 1 to 64 apart
    step = [int(b) * bs + 3 for b in order[:-(-n // bs)]]
    for i, t in enumerate(range(0, len(step) - 70, 50)):
        step[t + 1 + i * 7 % 64] = step[t] + 1
    verify(c, step, hkv, 9)


def test_what_is_left_out_is_the_same_in_every_run():
    import int8_group_quantized_gb300 as dgq
    slots = [16 * (t % 40) + t // 40 for t in range(400)]    # 40 requests, ten tokens each, interleaved
    k, v = tokens(400, 2, 1).cuda(), tokens(400, 2, 2).cuda()
    outs = []
    for _ in range(5):
        c = Cache("int8", 40, 2, 16)
        dgq.dgq_store_block8("int8", k, v, i32(slots), *c.d_codes, *c.d_scales, c.ws)
        assert dgq.dgq_workspace_error(c.ws) == SPLIT
        outs.append([x.cpu().view(torch.uint8) for x in (*c.d_codes, *c.d_scales)])
    assert all(torch.equal(a, b) for o in outs[1:] for a, b in zip(o, outs[0]))
