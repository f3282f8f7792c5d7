"""The 8-bit cache with one scale per block and head: codes and scales against the definition in 64 bits, to
the bit, as tokens arrive in any portions; rows read back; decode attention over it within the bound of its
roundings."""
import numpy as np
import pytest
import torch

from attn_reference import check, rows
from window_reference import attend, visible

pytestmark = pytest.mark.gpu

TOP = {"int8": 127.0, "e4m3": 448.0}
FMT = pytest.mark.parametrize("fmt", ["int8", "e4m3"])


def i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")


def workspace(n=256):
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


# ---- the definition -----------------------------------------------------------------------------------

def decode(codes, fmt):
    """Codes (uint8 numpy) as numbers."""
    c = codes.astype(np.int64)
    if fmt == "int8":
        return (c - 128).astype(np.float64)
    e, f = (c >> 3) & 15, (c & 7).astype(np.float64)
    y = np.where(e > 0, (1 + f / 8) * 2.0 ** (e - 7), f / 8 * 2.0 ** -6)
    return np.where(c > 127, -y, y)


def scale_of(amax, fmt):
    if amax < 2.0 ** -80:
        return 0.0
    t = float(amax) / TOP[fmt]
    unit = 2.0 ** (int(np.frexp(t)[1]) - 8)
    return float(np.ceil(t / unit) * unit)


def encode(x, s, fmt):
    y = x / s if s > 0 else np.zeros_like(x)
    if fmt == "int8":
        return (np.rint(y) + 128).astype(np.uint8)
    e = np.maximum(np.frexp(y)[1] - 1, -6)
    q = np.rint(y / 2.0 ** (e - 3.0)) * 2.0 ** (e - 3.0)
    e = np.where(q != 0, np.maximum(np.frexp(q)[1] - 1, -6), -6)
    a = np.abs(q)
    normal = a >= 2.0 ** -6
    code = np.where(normal, (e + 7) * 8 + (a / 2.0 ** e.astype(float) - 1) * 8, a / 2.0 ** -9)
    return (code + np.where(np.signbit(q), 128, 0)).astype(np.uint8)


class Cache:
    """Pools and scales in both places; every slot that no token owns holds 0xFF (a NaN of E4M3), every scale
    that no block owns NaN."""

    def __init__(self, fmt, blocks, hkv, bs):
        self.fmt, self.bs, self.hkv, self.blocks = fmt, bs, hkv, blocks
        self.codes = [np.full((blocks, hkv, bs, 128), 0xFF, dtype=np.uint8) for _ in range(2)]
        self.scales = [np.full((blocks, hkv), np.nan, dtype=np.float32) for _ in range(2)]
        self.d_codes = [torch.from_numpy(c).cuda() for c in self.codes]
        self.d_scales = [torch.from_numpy(s).cuda() for s in self.scales]
        self.ws = workspace()

    def store(self, k, v, slots):
        """k, v bf16 [T, hkv, 128] on the CPU; both sides updated."""
        import int8_group_quantized_gb300 as dgq
        dgq.dgq_store_block8(self.fmt, k.cuda(), v.cuda(), i32(slots), *self.d_codes, *self.d_scales, self.ws)
        t = 0
        while t < len(slots):
            if slots[t] < 0:
                t += 1
                continue
            n, (block, r0) = 1, divmod(int(slots[t]), self.bs)
            while r0 + n < self.bs and t + n < len(slots) and slots[t + n] == slots[t] + n:
                n += 1
            for x, codes, scales in zip((k, v), self.codes, self.scales):
                x = x[t:t + n].double().numpy()
                for h in range(self.hkv):
                    had = float(scales[block, h]) if r0 else 0.0
                    s = max(had, scale_of(np.abs(x[:, h]).max(), self.fmt))
                    if r0 and s > had:
                        codes[block, h, :r0] = encode(decode(codes[block, h, :r0], self.fmt) * had, s, self.fmt)
                    codes[block, h, r0:r0 + n] = encode(x[:, h], s, self.fmt)
                    scales[block, h] = s
            t += n

    def verify(self):
        import int8_group_quantized_gb300 as dgq
        torch.cuda.synchronize()
        assert dgq.dgq_workspace_error(self.ws) == 0
        for a, b in zip(self.d_scales, self.scales):
            assert np.array_equal(a.cpu().numpy(), b, equal_nan=True)
        for a, b in zip(self.d_codes, self.codes):
            bad = a.cpu().numpy() != b
            assert not bad.any(), (int(bad.sum()), tuple(np.argwhere(bad)[0]))


def tokens(n, hkv, seed, spread=True):
    """Rows whose size changes from token to token and from head to head."""
    x = rows(n, hkv, seed, 1.0)
    if not spread:
        return x
    g = torch.Generator().manual_seed(seed + 1)
    return (x.float() * 2.0 ** (6 * torch.rand(n, hkv, 1, generator=g) - 3)).to(torch.bfloat16)


def slots_of(table, bs, begin, end):
    return [int(table[p // bs]) * bs + p % bs for p in range(begin, end)]


# ---- store ----------------------------------------------------------------------------------------------

@FMT
@pytest.mark.parametrize("bs", [16, 32, 64])
@pytest.mark.parametrize("hkv", [1, 3, 8])
def test_portions_of_any_size(fmt, bs, hkv):
    rng = np.random.default_rng(bs + hkv)
    c = Cache(fmt, 30, hkv, bs)
    order = rng.permutation(30)
    tables = [order[:9], order[9:18], order[18:27]]
    lens = [0, 0, 0]
    for step, new in enumerate([(1, 5, 16), (2, 0, 17), (bs, 1, 1), (3, bs + 7, 1), (1, 1, 2 * bs), (70, 1, 0), (1, 1, 1)]):
        slots, k, v = [], [], []
        for b, n in enumerate(new):
            n = min(n, 9 * bs - lens[b])
            slots += slots_of(tables[b], bs, lens[b], lens[b] + n)
            lens[b] += n
            slots += [-1] * (step % 3)                      # padding between requests
        k, v = tokens(len(slots), hkv, 100 * step), tokens(len(slots), hkv, 100 * step + 50)
        c.store(k, v, slots)
        c.verify()


@FMT
@pytest.mark.parametrize("T", [1, 31, 500, 4000])
def test_long_runs_and_many_single_tokens(fmt, T):
    blocks = T // 64 + 2
    c = Cache(fmt, blocks, 2, 64)
    order = np.random.default_rng(T).permutation(blocks)
    c.store(tokens(T, 2, T), tokens(T, 2, T + 1), slots_of(order, 64, 0, T))
    c.verify()
    c = Cache(fmt, T, 2, 16)                                # a decode step: each token in a block of its own
    c.store(tokens(T, 2, T + 2), tokens(T, 2, T + 3), (np.random.default_rng(T).permutation(T) * 16).tolist())
    c.verify()
    c.store(tokens(T, 2, T + 4), tokens(T, 2, T + 5), (np.random.default_rng(T + 1).permutation(T) * 16 + 1).tolist())
    c.verify()


@FMT
def test_every_pair_of_significands(fmt):
    """Blocks whose largest value has each significand, filled with values of all significands and sizes."""
    bits = np.arange(128, dtype=np.uint16)
    c = Cache(fmt, 128, 1, 16)
    x = np.zeros((128, 16, 128), dtype=np.uint16)
    for a in range(128):
        x[a] = ((127 - np.arange(16))[:, None] << 7) + bits[None, :]     # 2^0 .. 2^-15, sign alternating
        x[a, :, ::2] |= 0x8000
        x[a, 0] = np.where(bits <= a, x[a, 0], 0x3F80 + a)               # none larger than the block's
        x[a, 0, 0] = 0x3F80 + a
    t = torch.from_numpy(x.reshape(2048, 1, 128).view(np.int16)).view(torch.bfloat16)
    c.store(t, -t, list(range(2048)))
    c.verify()


@FMT
def test_scales_that_grow_by_every_amount(fmt):
    c = Cache(fmt, 200, 1, 16)
    first = tokens(200 * 7, 1, 5)
    c.store(first, first, [16 * b + r for b in range(200) for r in range(7)])
    for r in (7, 8):                                        # one more token each, 2^-3 to 2^13 times as large
        x = (rows(200, 1, 6 + r, 1.0).float() * 2.0 ** (torch.arange(200).float() / 200 * 16 - 3)[:, None, None]).to(torch.bfloat16)
        c.store(x, -x, [16 * b + r for b in range(200)])
        c.verify()


@FMT
def test_zeros_tiny_and_huge_values(fmt):
    x = torch.zeros(7 * 16, 1, 128, dtype=torch.bfloat16)
    for b, s in enumerate([0.0, 2.0 ** -81, 2.0 ** -80, 2.0 ** -70, 2.0 ** 90, 3e-5, 1.0]):
        x[16 * b:16 * b + 9] = s
    x[16 * 6 + 3] = float("-0.0")
    c = Cache(fmt, 7, 1, 16)
    slots = [16 * b + r for b in range(7) for r in range(9)]
    c.store(x[slots], x[slots], slots)
    c.verify()
    y = torch.ones(7, 1, 128, dtype=torch.bfloat16)          # behind a block of zeros, too
    c.store(y, 2 * y, [16 * b + 9 for b in range(7)])
    c.verify()


def test_a_slot_that_does_not_exist_is_flagged_and_left_out():
    import int8_group_quantized_gb300 as dgq
    for bad in (-2, 64, 2 ** 31 - 1):
        c = Cache("int8", 4, 2, 16)
        k = tokens(4, 2, 1)
        dgq.dgq_store_block8("int8", k.cuda(), k.cuda(), i32([16, 17, bad, 32]), *c.d_codes, *c.d_scales, c.ws)
        assert dgq.dgq_workspace_error(c.ws) == 5
        c.ws.zero_()
        c.store(k[[0, 1, 3]], k[[0, 1, 3]], [16, 17, 32])
        c.verify()


# ---- load -----------------------------------------------------------------------------------------------

def filled(fmt, lens, hkv, bs, seed):
    rng = np.random.default_rng(seed)
    need = [-(-n // bs) for n in lens]
    order = rng.permutation(sum(need) + 2)
    c = Cache(fmt, len(order), hkv, bs)
    table = np.full((len(lens), max(need) + 1), 10 ** 6, dtype=np.int32)   # (unused entries name no block)
    at, slots = 0, []
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        slots += slots_of(table[b], bs, 0, n)
    c.store(tokens(len(slots), hkv, seed), tokens(len(slots), hkv, seed + 1), slots)
    return c, table


def values(c, table, b, n, which):
    p = np.arange(n)
    block = table[b][p // c.bs]
    codes = c.codes[which][block, :, p % c.bs]
    return decode(codes, c.fmt) * c.scales[which][block][..., None].astype(np.float64), c.scales[which][block].astype(np.float64)


@FMT
@pytest.mark.parametrize("bs,hkv", [(16, 1), (32, 3), (64, 8)])
def test_rows_back_in_bf16(fmt, bs, hkv):
    import int8_group_quantized_gb300 as dgq
    lens = [0, 1, 15, 16, 17, 0, 64, 300, 0]
    c, table = filled(fmt, lens, hkv, bs, 3)
    gap = 2                                                  # rows in front of the first request and behind the last
    total = sum(lens) + 2 * gap
    out = [torch.full((total, hkv, 128), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    dgq.dgq_load_block8(fmt, *c.d_codes, *c.d_scales, i32(table), i32(gap + np.concatenate([[0], np.cumsum(lens)])), *out, c.ws)
    c.verify()
    for which, o in enumerate(out):
        want = [torch.from_numpy(values(c, table, b, n, which)[0]) for b, n in enumerate(lens)]
        want = torch.cat(want).to(torch.float32).to(torch.bfloat16)        # (exact in fp32: 15 bits)
        o = o.cpu()
        assert torch.equal(o[gap:-gap], want) and (o[:gap] == 9).all() and (o[-gap:] == 9).all()


def test_load_flags_what_it_cuts():
    import int8_group_quantized_gb300 as dgq
    c, table = filled("int8", [20, 20], 1, 16, 4)
    out = lambda: [torch.full((30, 1, 128), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    k, v = out()
    dgq.dgq_load_block8("int8", *c.d_codes, *c.d_scales, i32(table), i32([0, 20, 40]), k, v, c.ws)
    assert dgq.dgq_workspace_error(c.ws) == 6
    want = torch.from_numpy(values(c, table, 1, 10, 0)[0]).float().to(torch.bfloat16)
    assert torch.equal(k[20:].cpu(), want)
    c.ws.zero_()
    table[0, 1] = -1
    k, v = out()
    dgq.dgq_load_block8("int8", *c.d_codes, *c.d_scales, i32(table), i32([0, 20, 30]), k, v, c.ws)
    assert dgq.dgq_workspace_error(c.ws) == 5


# ---- decode ---------------------------------------------------------------------------------------------

class Step:
    def __init__(self, fmt, lens, hq, hkv, bs, seed):
        self.c, self.table = filled(fmt, lens, hkv, bs, seed)
        self.lens, self.hq, self.hkv, self.fmt = lens, hq, hkv, fmt
        self.q, self.kn, self.vn = rows(len(lens), hq, seed + 2, 1.0), rows(len(lens), hkv, seed + 3), rows(len(lens), hkv, seed + 4)

    def run(self, window=0, sinks=0, table=None):
        import int8_group_quantized_gb300 as dgq
        top = max(1, max(self.lens))
        ws = workspace(dgq.dgq_attn_workspace_size(len(self.lens), self.hq, self.hkv, top))
        out = torch.zeros(self.q.shape, dtype=torch.bfloat16, device="cuda")
        dgq.dgq_paged_decode_attn_block8(self.fmt, self.q.cuda(), self.kn.cuda(), self.vn.cuda(), *self.c.d_codes,
                                         *self.c.d_scales, i32(self.table if table is None else table), i32(self.lens),
                                         top, out, ws, window=window, sinks=sinks)
        torch.cuda.synchronize()
        assert dgq.dgq_workspace_error(ws) == 0
        return out

    def check(self, out, window=0, sinks=0):
        g = self.hq // self.hkv
        ref = torch.zeros(self.q.shape, dtype=torch.float64)
        bound = torch.zeros_like(ref)
        for b, n in enumerate(self.lens):
            (k, ks), (v, vs) = (values(self.c, self.table, b, n, w) for w in (0, 1))
            for h in range(self.hkv):
                s = slice(h * g, (h + 1) * g)
                one = lambda x, y: torch.cat([torch.from_numpy(x[:, h]), y[b, h][None].double()])
                pad = lambda x: torch.cat([torch.from_numpy(x[:, h]), torch.zeros(1, dtype=torch.float64)])
                off = 1152.0 if self.fmt == "int8" else 0.0
                ref[b, s], bound[b, s] = attend(
                    self.q[b, s].double(), one(k, self.kn), one(v, self.vn),
                    visible(torch.full((g,), n), n + 1, window, sinks), weight_unit=2.0 ** -11,
                    k_size=off * pad(ks), v_size=off * pad(vs), v_scale=pad(vs), top=TOP[self.fmt])
        check(out, ref, bound)


@FMT
@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (8, 4), (16, 4), (8, 1)])
def test_decode_group_sizes(fmt, hq, hkv):
    s = Step(fmt, [5, 64, 65, 700], hq, hkv, 16, hq + hkv)
    s.check(s.run())


@FMT
@pytest.mark.parametrize("bs", [16, 32, 64])
def test_decode_ragged_batches(fmt, bs):
    s = Step(fmt, [0, 1, 15, 16, 17, 63, 64, 65, 129, 1000, 4097], 8, 2, bs, bs)
    out = s.run()
    s.check(out)
    assert torch.equal(out, s.run())


@FMT
def test_decode_long_requests_find_every_block(fmt):
    """Each block of 16 tokens has a scale of its own, over 2^24; every 97th token is the only one that its
    query sees, all others far below, so a lost, doubled or wrongly scaled tile shows."""
    n, hkv = 20000, 1
    for at in (0, 1, 8191, 19999, 16 * 777 + 5):
        s = Step(fmt, [n], 4, hkv, 16, 5)
        c = s.c
        k = tokens(n, hkv, 6, spread=False)
        v = (rows(n, hkv, 7, 1.0).float() * 2.0 ** (torch.arange(n) // 16 % 25 - 12).float()[:, None, None]).to(torch.bfloat16)
        k[at] = 4 * s.q[0, 0]                               # about 4 sqrt(128) above the others for head 0
        c.store(k, v, slots_of(s.table[0], 16, 0, n))
        s.check(s.run())


@FMT
def test_blocks_of_zeros_keep_their_weight_in_the_sum(fmt):
    s = Step(fmt, [64], 4, 1, 16, 8)
    k = torch.zeros(64, 1, 128, dtype=torch.bfloat16)        # all scores 0: equal weights
    v = torch.zeros(64, 1, 128, dtype=torch.bfloat16)
    v[16:32], v[32:48] = 1.0, 2.0 ** -60
    s.c.store(k, v, slots_of(s.table[0], 16, 0, 64))
    s.kn.zero_()
    s.vn.zero_()
    out = s.run().cpu().double()
    assert (out - 16 / 65).abs().max() <= 16 / 65 * (2.0 ** -8 + 2.0 ** -11 * 2 + 1e-5)
    s.check(s.run())


@FMT
def test_decode_repeats_in_a_graph_and_on_a_stream(fmt):
    import int8_group_quantized_gb300 as dgq
    s = Step(fmt, [3000, 17, 0, 900], 8, 2, 32, 9)
    want = s.run()
    args = (s.q.cuda(), s.kn.cuda(), s.vn.cuda(), *s.c.d_codes, *s.c.d_scales, i32(s.table), i32(s.lens), 3000)
    out, ws = torch.zeros_like(want), workspace(dgq.dgq_attn_workspace_size(4, 8, 2, 3000))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dgq.dgq_paged_decode_attn_block8(fmt, *args, out, ws)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    stream = torch.cuda.Stream()
    out.zero_()
    stream.wait_stream(torch.cuda.current_stream())
    dgq.dgq_paged_decode_attn_block8(fmt, *args, out, ws, stream=stream)
    stream.synchronize()
    assert torch.equal(out, want)


@FMT
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (2, 0), (17, 0), (64, 16), (100, 5), (5000, 7)])
def test_decode_windows(fmt, window, sinks):
    s = Step(fmt, [0, 1, 2, 16, 17, 100, 116, 117, 1000, 2500], 8, 2, 16, window + sinks)
    s.check(s.run(window, sinks), window, sinks)


def test_binding_refuses_other_shapes_and_types():
    import int8_group_quantized_gb300 as dgq
    s = Step("int8", [40, 20], 4, 2, 16, 10)
    c, ws = s.c, workspace(1 << 26)
    k, slots = tokens(3, 2, 11).cuda(), i32([0, 1, 2])
    store = lambda **kw: dgq.dgq_store_block8(*{**dict(fmt="int8", k=k, v=k, slots=slots, kp=c.d_codes[0], vp=c.d_codes[1],
                                                       ks=c.d_scales[0], vs=c.d_scales[1], ws=c.ws), **kw}.values())
    store()
    for bad in (dict(fmt="fp8"), dict(fmt=7), dict(k=k.half()), dict(v=k[:2]), dict(slots=slots.long()), dict(kp=c.d_codes[0][1:]),
                dict(vp=c.d_codes[1].view(torch.int8)), dict(ks=c.d_scales[0].double()), dict(vs=c.d_scales[1][:, :1]),
                dict(ks=c.d_scales[0].cpu()), dict(ws=c.ws[:128])):
        with pytest.raises(dgq.DGQError):
            store(**bad)
    out = torch.zeros(s.q.shape, dtype=torch.bfloat16, device="cuda")
    good = dict(fmt="int8", q=s.q.cuda(), kn=s.kn.cuda(), vn=s.vn.cuda(), kp=c.d_codes[0], vp=c.d_codes[1], ks=c.d_scales[0],
                vs=c.d_scales[1], bt=i32(s.table), lens=i32(s.lens), top=40, out=out, ws=ws)
    dgq.dgq_paged_decode_attn_block8(*good.values())
    for bad in (dict(fmt="dgq"), dict(q=s.q), dict(kn=s.kn.cuda().float()), dict(ks=c.d_scales[0].t().contiguous()),
                dict(lens=i32([40])), dict(bt=i32(s.table).long()), dict(out=out[:1])):
        with pytest.raises(dgq.DGQError):
            dgq.dgq_paged_decode_attn_block8(*{**good, **bad}.values())
    for window, sinks in ((0, 1), (-1, 0), (4, -1)):
        with pytest.raises(dgq.DGQError):
            dgq.dgq_paged_decode_attn_block8(*good.values(), window=window, sinks=sinks)


@FMT
def test_windows_of_slots_with_many_runs_and_heads(fmt):
    """Calls large enough for the largest window of slots: whole blocks of a long prompt, and short runs."""
    blocks, hkv = 320, 32
    c = Cache(fmt, blocks, hkv, 64)
    x, y = tokens(20000, hkv, 21), tokens(20000, hkv, 22)
    order = np.random.default_rng(1).permutation(blocks)
    c.store(x, y, slots_of(order, 64, 0, 20000))
    c.verify()
    slots = [int(64 * b + b % 61 + r) for b in order[:312] for r in range(3)]  # (whole blocks, written again inside)
    k, v = tokens(len(slots), hkv, 23), tokens(len(slots), hkv, 24)
    c.store(k, v, slots)
    c.verify()


@pytest.mark.parametrize("batch", [300, 8192])
def test_load_of_many_requests(batch):
    import int8_group_quantized_gb300 as dgq
    lens = np.random.default_rng(batch).integers(0, 40, batch).tolist()
    c, table = filled("int8", lens, 1, 16, 31)
    out = [torch.zeros(sum(lens), 1, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    dgq.dgq_load_block8("int8", *c.d_codes, *c.d_scales, i32(table), i32(np.concatenate([[0], np.cumsum(lens)])), *out, c.ws)
    c.verify()
    for which, o in enumerate(out):
        want = torch.cat([torch.from_numpy(values(c, table, b, n, which)[0]) for b, n in enumerate(lens)])
        assert torch.equal(o.cpu(), want.float().to(torch.bfloat16))


@FMT
@pytest.mark.parametrize("window", [0, 300])
def test_decode_scores_of_any_size(fmt, window):
    """Scores of 10^4 to 10^9: one token's lies above all others by its own size, far more than fp32 loses
    (136 2^-24 of it), so its value is the result, rounded to bf16."""
    for size, big in ((30.0, 30.0), (3e4, 100.0), (6e4, 3e4)):
        s = Step(fmt, [1000], 4, 1, 16, 40)
        at = 900
        s.q[:] = (torch.sign(s.q.float()) * size).to(torch.bfloat16)
        sign = torch.sign(s.q[0, 0].float())
        s.q[:] = s.q[0, 0]
        k = (-big * sign).expand(1000, 1, 128).clone()
        k[at] = big * sign
        v = tokens(1000, 1, 41)
        s.kn[:] = (-big * sign).to(torch.bfloat16)
        s.c.store(k.to(torch.bfloat16), v, slots_of(s.table[0], 16, 0, 1000))
        out = s.run(window, 0).cpu()
        want = torch.from_numpy(values(s.c, s.table, 0, 1000, 1)[0][at, 0])
        assert ((out[0].double() - want).abs() <= 2.0 ** -8 * want.abs() * 1.01).all()


def test_threads_on_streams_of_their_own():
    import threading
    import int8_group_quantized_gb300 as dgq
    steps = [Step(fmt, [700, 33 + i, 0], 8, 2, 16, 50 + i) for i, fmt in enumerate(["int8", "e4m3"] * 3)]
    want = [s.run(100 if i % 3 else 0, 3 if i % 3 else 0) for i, s in enumerate(steps)]
    got, errors = [None] * 6, []

    def work(i, s):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    got[i] = s.run(100 if i % 3 else 0, 3 if i % 3 else 0)
        except Exception as e:  # (shown by the main thread)
            errors.append(e)
    threads = [threading.Thread(target=work, args=x) for x in enumerate(steps)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_load_stays_inside_its_buffers_when_lengths_overlap():
    """Cumulative lengths that go down are flagged; what overlaps holds values of either request."""
    import int8_group_quantized_gb300 as dgq
    c, table = filled("int8", [40] * 6, 1, 16, 60)
    out = [torch.full((44, 1, 128), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    dgq.dgq_load_block8("int8", *c.d_codes, *c.d_scales, i32(table), i32([2, 42, 2, 42, 2, 42, 2]), *out, c.ws)
    assert dgq.dgq_workspace_error(c.ws) == 6
    for which, o in enumerate(out):
        o = o.cpu()
        assert (o[:2] == 9).all() and (o[42:] == 9).all()
        rows_of = torch.stack([torch.from_numpy(values(c, table, b, 40, which)[0]).float().to(torch.bfloat16) for b in (0, 2, 4)])
        same = (rows_of == o[2:42]).view(3, 40, 16, 8).all(dim=-1)           # (written 16 bytes at a time)
        assert same.any(dim=0).all()


@FMT
def test_a_fork_goes_on_with_its_own_page_and_scale(fmt):
    """A request forked inside a block: the page and its scales copied, then different tokens to both sides."""
    import int8_group_quantized_gb300 as dgq
    hkv, bs = 4, 16
    c = Cache(fmt, 8, hkv, bs)
    pool, table = dgq.BlockPool(8), np.zeros((2, 3), dtype=np.int32)
    pool.alloc_table_row(20, bs, table, 0)
    c.store(tokens(20, hkv, 71), tokens(20, hkv, 72), slots_of(table[0], bs, 0, 20))
    pairs = pool.fork_row(20, bs, table, 0, 1)
    assert len(pairs) == 1
    ws, d_pairs = workspace(), i32(pairs)
    dgq.dgq_copy_pages(c.d_codes, d_pairs, ws)
    dgq.dgq_copy_pages(c.d_scales, d_pairs, ws)
    for host in (*c.codes, *c.scales):
        host[pairs[0][1]] = host[pairs[0][0]]
    c.verify()
    for step in range(3):
        x = (tokens(2, hkv, 73 + step).float() * torch.tensor([4.0 ** step, 1.0])[:, None, None]).to(torch.bfloat16)
        c.store(x, -x, [slots_of(table[b], bs, 20 + step, 21 + step)[0] for b in (0, 1)])
        c.verify()
    assert dgq.dgq_workspace_error(ws) == 0
    a, b = (c.scales[0][table[r, 1]] for r in (0, 1))
    assert (a > b).any()                                     # one side's scale grew, the other's did not
