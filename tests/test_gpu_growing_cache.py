"""The operators of a growing cache in one run, as a serving loop uses them: prompts in chunks behind an 8-bit
history, then decode steps without the host in between (tables, bf16 pages and the 8-bit cache grown from
lengths on the GPU, attention over both with a window and sinks), eager and replayed as a graph."""
import numpy as np
import pytest
import torch

from attn_reference import check, rows
from test_gpu_block8 import TOP, decode
from window_reference import attend, visible

pytestmark = pytest.mark.gpu

HQ, HKV, BS, BLOCKS, COLUMNS, B = 8, 2, 16, 160, 40, 3
WINDOW, SINKS = 70, 5


def i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")


class Serving:
    def __init__(self, fmt):
        import int8_group_quantized_gb300 as dgq
        self.dgq, self.fmt = dgq, fmt
        pool = dgq.BlockPool(BLOCKS)
        self.ids, self.used = i32(pool.alloc(BLOCKS - 2)), i32([0])
        self.lens, self.before, self.table = i32([0] * B), i32([0] * B), i32(np.full((B, COLUMNS), -1))
        cache = (BLOCKS, HKV, BS, 128)
        self.pages = [torch.full(cache, float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        self.codes = [torch.full(cache, 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.scales = [torch.full(cache[:2], float("nan"), device="cuda") for _ in range(2)]
        self.ws = torch.zeros(1 << 27, dtype=torch.uint8, device="cuda")
        self.kept = [[[], []] for _ in range(B)]             # every token's rows, on the CPU

    def extend(self, new, total):
        slots, cu = i32([0] * total), i32([0] * (B + 1))
        self.before.copy_(self.lens)
        self.dgq.dgq_extend_tables(self.lens, new, BS, BLOCKS, self.ids, self.used, self.table, slots, cu, self.lens,
                                   self.used, self.ws)
        return slots, cu

    def write(self, k, v, slots):
        self.dgq.dgq_write_slots(k, v, slots, *self.pages, self.ws)
        self.dgq.dgq_store_block8(self.fmt, k, v, slots, *self.codes, *self.scales, self.ws)

    def keep(self, k, v, new):
        at = 0
        for b, n in enumerate(new):
            self.kept[b][0].append(k[at:at + n].cpu())
            self.kept[b][1].append(v[at:at + n].cpu())
            at += n

    def chunk(self, new, seed):
        """A prompt chunk of every request: its rows stored, the history read back, attention over it."""
        total = sum(new)
        kv = rows(total, 2 * HKV, seed, 0.7).cuda()           # a fused projection's output
        q = rows(total, HQ, seed + 1, 1.0).cuda()
        slots, cu_q = self.extend(i32(new), total)
        self.write(kv[:, :HKV], kv[:, HKV:], slots)
        self.keep(kv[:, :HKV], kv[:, HKV:], new)
        n = self.lens.tolist()
        cu_kv = i32(np.concatenate([[0], np.cumsum(n)]))
        k, v = (torch.zeros(sum(n), HKV, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.dgq.dgq_load_block8(self.fmt, *self.codes, *self.scales, self.table, cu_kv, k, v, self.ws)
        out = torch.zeros_like(q)
        self.dgq.dgq_prompt_attn(q, k, v, cu_q, cu_kv, out, self.ws, window=WINDOW, sinks=SINKS)
        paged = torch.zeros_like(q)
        self.dgq.dgq_prompt_attn_paged(q, cu_q, *self.pages, self.table, self.lens, paged, self.ws, window=WINDOW, sinks=SINKS)
        torch.cuda.synchronize()
        assert self.dgq.dgq_workspace_error(self.ws) == 0
        at = 0
        for b, (m, c) in enumerate(zip(new, n)):
            seen = visible(c - m + torch.arange(m), c, WINDOW, SINKS)
            first = int(cu_kv[b])
            own = [torch.cat(x) for x in self.kept[b]]
            for got, ks, vs in ((out, k[first:first + c].cpu(), v[first:first + c].cpu()), (paged, *own)):
                for h in range(HQ):
                    ref = attend(q[at:at + m, h].cpu().double(), ks[:, h // 4].double(), vs[:, h // 4].double(), seen)
                    check(got[at:at + m, h], *ref)
            at += m

    def step(self, q, k, v, new, slots, cu, out, whole, paged):
        """One token of every request; everything is enqueued, nothing read back."""
        args = (q, k, v, *self.codes, *self.scales, self.table, self.lens, COLUMNS * BS)
        self.dgq.dgq_paged_decode_attn_block8(self.fmt, *args, out, self.ws, window=WINDOW, sinks=SINKS)
        self.dgq.dgq_paged_decode_attn_block8(self.fmt, *args, whole, self.ws)
        self.dgq.dgq_paged_decode_attn_bf16(q, k, v, *self.pages, self.table, self.lens, COLUMNS * BS, paged, self.ws,
                                            window=WINDOW, sinks=SINKS)
        self.dgq.dgq_extend_tables(self.lens, new, BS, BLOCKS, self.ids, self.used, self.table, slots, cu, self.lens,
                                   self.used, self.ws)
        self.write(k, v, slots)

    def cached(self, b, n, which):
        t = torch.arange(n)
        block = self.table[b].cpu().long()[t // BS]
        s = self.scales[which].cpu()[block].double()
        return torch.from_numpy(decode(self.codes[which].cpu()[block, :, t % BS].numpy(), self.fmt)) * s[..., None], s

    def check_step(self, q, k, v, lens, out, whole, paged):
        for b, n in enumerate(lens):
            (kc, ks), (vc, vs) = self.cached(b, n, 0), self.cached(b, n, 1)
            own = [torch.cat(x)[:n] for x in self.kept[b]]
            for h in range(HKV):
                s = slice(4 * h, 4 * h + 4)
                cat = lambda x, y: torch.cat([x[:, h].double(), y[b, h][None].cpu().double()])
                pad = lambda x: torch.cat([x[:, h], torch.zeros(1, dtype=torch.float64)])
                off = 1152.0 if self.fmt == "int8" else 0.0
                at, qq = torch.full((4,), n), q[b, s].cpu().double()
                for got, w, sk in ((out, WINDOW, SINKS), (whole, 0, 0)):
                    check(got[b, s], *attend(qq, cat(kc, k), cat(vc, v), visible(at, n + 1, w, sk), 2.0 ** -11, off * pad(ks),
                                             off * pad(vs), pad(vs), TOP[self.fmt]))
                check(paged[b, s], *attend(qq, cat(own[0], k), cat(own[1], v), visible(at, n + 1, WINDOW, SINKS)))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_prompts_in_chunks_then_steps_eager_and_replayed(fmt):
    s = Serving(fmt)
    s.chunk([37, 200, 1], 1)
    s.chunk([64, 3, 129], 2)
    s.chunk([5, 120, 0], 3)
    q, k, v = (torch.zeros(B, h, 128, dtype=torch.bfloat16, device="cuda") for h in (HQ, HKV, HKV))
    outs = [torch.zeros_like(q) for _ in range(3)]
    new, slots, cu = i32([1, 1, 1]), i32([0] * B), i32([0] * (B + 1))

    def one(enqueue, seed):
        q.copy_(rows(B, HQ, seed, 1.0)), k.copy_(rows(B, HKV, seed + 1, 0.7)), v.copy_(rows(B, HKV, seed + 2, 2.0 ** (seed % 5)))
        lens = s.lens.tolist()
        cached = [s.codes[0].clone(), s.codes[1].clone(), s.scales[0].clone(), s.scales[1].clone()]
        enqueue()
        torch.cuda.synchronize()
        assert s.dgq.dgq_workspace_error(s.ws) == 0
        assert s.lens.tolist() == [n + 1 for n in lens]
        after, s.codes, s.scales = (s.codes, s.scales), cached[:2], cached[2:]  # the attention came before the store
        s.check_step(q, k, v, lens, *outs)
        s.codes, s.scales = after
        s.keep(k, v, [1] * B)

    enqueue = lambda: s.step(q, k, v, new, slots, cu, *outs)
    for i in range(2):
        one(enqueue, 10 + i)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        enqueue()
    for i in range(20):
        one(graph.replay, 20 + i)
    # the pages hold every token as it came
    for b, n in enumerate(s.lens.tolist()):
        t = torch.arange(n)
        block = s.table[b].cpu().long()[t // BS]
        for x, kept in zip(s.pages, s.kept[b]):
            assert torch.equal(x.cpu()[block, :, t % BS], torch.cat(kept))
    used = s.table[s.table >= 0].tolist()
    assert len(used) == len(set(used)) == int(s.used) == sum(-(-n // BS) for n in s.lens.tolist())
