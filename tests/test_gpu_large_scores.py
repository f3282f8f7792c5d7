"""Finite inputs whose scores are so far apart that a row's softmax is the one key it matches best: the
output is that key's value, whatever the scores' size, in every tile, across cuts and merges.

One dimension of q and k is not zero, so a score is one exact product; the keys' values are distinct with at
least 2^-8 between neighbours relative to their size, so at scores of 2^20 and more the second best key has a
weight below 2^-500.  Tolerance: the weight rounded to bf16 before it meets V while the sum holds it in fp32
(a factor 1 + e, |e| <= 2^-8), the output rounded to bf16 (2^-8): 2^-7 (1 + 2^-8) and what the exponential
and the reciprocal add in the last places of fp32, together below 2^-7 (1 + 2^-7) of the value."""
import pytest
import torch

from attn_reference import Pages
from test_gpu_decode_bf16 import Step
from test_gpu_prompt import Prompt

TOL = 2.0 ** -7 * (1 + 2.0 ** -7)


def distinct(m, seed):
    """m <= 1280 different bf16 numbers in [1, 1024), shuffled."""
    e, f = torch.arange(10, dtype=torch.float64), 1 + torch.arange(128, dtype=torch.float64) / 128
    x = (2 ** e[:, None] * f[None, :]).flatten()
    return x[torch.randperm(len(x), generator=torch.Generator().manual_seed(seed))[:m]]


def one_column(n, heads, column):
    x = torch.zeros(n, heads, 128, dtype=torch.bfloat16)
    x[:, :, 5] = column[:, None].to(torch.bfloat16)
    assert torch.isfinite(x).all()
    return x


def close(got, want):
    got, want = got.cpu().double(), want.double()
    assert torch.isfinite(got).all()
    assert ((got - want).abs() <= TOL * want.abs()).all(), float(((got - want).abs() / want.abs().clamp(min=1e-30)).max())


EXPONENTS = [20, 26, 30, 31, 32, 34, 38, 50, 80, 110]


@pytest.mark.gpu
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("exponent", EXPONENTS)
@pytest.mark.parametrize("block", [None, 16])
def test_prompt_rows_take_their_best_key(exponent, sign, block):
    shape, hkv, g = [(200, 200), (3, 1280), (70, 700)], 2, 4
    p = Prompt(shape, g * hkv, hkv, seed=91, block=block)
    scale = 2.0 ** (exponent // 2)
    p.q = one_column(sum(p.n), g * hkv, torch.full((sum(p.n),), sign * scale))
    p.q[:, 1::2] *= -1                                     # every second head prefers the smallest product
    f = [distinct(m, 10 + i) for i, m in enumerate(p.m)]
    p.ks = [one_column(m, hkv, x * 2.0 ** (exponent - exponent // 2)) for m, x in zip(p.m, f)]
    out, at = p.device().run(), 0
    for n, m, x, v in zip(p.n, p.m, f, p.vs):
        for i in range(n):
            seen = x[:m - n + i + 1]
            for h in range(g * hkv):
                up = (sign > 0) == (h % 2 == 0)
                close(out[at + i, h], v[int(seen.argmax() if up else seen.argmin()), h // g])
        at += n


@pytest.mark.gpu
@pytest.mark.parametrize("exponent", EXPONENTS)
def test_decode_rows_take_their_best_key(exponent):
    lens, hkv, g = [1200, 300, 17], 2, 4
    s = Step(lens, g * hkv, hkv, 16, seed=92)
    s.q = one_column(3, g * hkv, torch.full((3,), 2.0 ** (exponent // 2)))
    s.q[:, 1::2] *= -1
    f = [distinct(n + 1, 20 + i) for i, n in enumerate(lens)]
    up = 2.0 ** (exponent - exponent // 2)
    s.ks = [one_column(n, hkv, x[:n] * up) for n, x in zip(lens, f)]
    s.kn = one_column(3, hkv, torch.stack([x[-1] for x in f]) * up)
    s.pages = Pages(s.ks, s.vs, hkv, 16)
    out = s.device().run()
    for b, x in enumerate(f):
        for h in range(g * hkv):
            v = torch.cat([s.vs[b][:, h // g], s.vn[b, h // g][None]])
            close(out[b, h], v[int(x.argmax() if h % 2 == 0 else x.argmin())])
