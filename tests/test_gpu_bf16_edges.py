"""Calls of the bf16 attention operators at the ends of what they accept: no key at all, rows before the first
request, the largest batch, many KV heads, packed rows behind 2^32 bytes."""
import pytest
import torch

from attn_reference import check, prompt, rows
from test_gpu_decode_bf16 import Step
from test_gpu_prompt import Prompt, cu, verify, workspace

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("block", [None, 16])
def test_no_key_at_all(block):
    p = Prompt([(70, 0), (0, 0), (300, 0)], 8, 2, seed=1, block=block)
    out = p.device().run()
    assert (out == 0).all()


def test_no_query_row():
    p = Prompt([(0, 5), (0, 0)], 8, 2, seed=2).device()
    assert p.run().shape == (0, 8, 128)


def test_rows_before_the_first_request_are_left():
    p = Prompt([(37, 40), (90, 120)], 4, 2, seed=3).device()
    nan = torch.full((21, 4, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    p.dq, p.cu_q = torch.cat([nan, p.dq]), p.cu_q + 21
    p.k, p.v = (torch.cat([nan[:, :2], x]).contiguous() for x in (p.k, p.v))
    p.cu_kv = p.cu_kv + 21
    out = p.run()
    assert (out[:21] == 7.0).all()
    p.check(out[21:])


@pytest.mark.parametrize("block", [None, 16])
def test_largest_batch_of_prompts(block):
    shape = [(b % 4, b % 4 + b % 3) for b in range(8192)]
    verify(shape, 8, 1, seed=4, block=block)


def test_largest_batch_of_decode():
    s = Step([b % 37 for b in range(8192)], 8, 1, 16, seed=5).device()
    s.check(s.run())


@pytest.mark.parametrize("hq,hkv", [(64, 64), (5, 5), (56, 7)])
def test_many_and_odd_kv_heads(hq, hkv):
    verify([(70, 90), (1, 700)], hq, hkv, seed=6)
    verify([(70, 90), (1, 700)], hq, hkv, seed=6, block=64)


def test_packed_rows_behind_four_gigabytes():
    import int8_group_quantized_gb300 as dgq
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    b, n, h = 8192, 36, 64
    q = torch.zeros(b * n, h, 128, dtype=torch.bfloat16, device="cuda")
    k, v, out = torch.zeros_like(q), torch.zeros_like(q), torch.full_like(q, 7)
    assert q.nbytes > 1 << 32
    some = [0, 1, 4000, 7500, b - 1]
    for i in some:
        for s, x in enumerate((q, k, v)):
            x[i * n:(i + 1) * n] = rows(n, h, 10 * i + s, 1.0).cuda()
    c, ws = cu([n] * b), workspace(b, h, h)
    dgq.dgq_prompt_attn(q, k, v, c, c, out, ws)
    assert dgq.dgq_workspace_error(ws) == 0
    for i in some:
        at = slice(i * n, (i + 1) * n)
        check(out[at], *prompt(q[at].cpu(), [k[at].cpu()], [v[at].cpu()], [n], h, h))
    for i in (2, 3999, 7501, b - 2):
        assert (out[i * n:(i + 1) * n] == 0).all()
