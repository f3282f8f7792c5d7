"""Forks of INT8 requests at any length: pages by the pool's fork_row and dgq_copy_pages, records by
dgq_fork_records, then appends to all sides.  Every byte of the pools and every record is compared with
the oracle's appends over records that a plain model cuts, and decode with the oracle's."""
import numpy as np
import pytest

import oracle
import synth
from dgq_cases import Case, assert_attn_close, first_record_diff, table_to_numpy

BS = 16
INVALID, UNSUPPORTED, WORKSPACE, OK = -1, -2, -3, 0
FAKE = 0x10000  # a 16-byte aligned address that is never dereferenced: checks fail first


def cut(rec, length):
    """A record cut to its first `length` tokens, field by field from the layout's definition."""
    assert 0 <= length <= rec["seq_len"]
    out = np.zeros((), dtype=oracle.SEG_DTYPE)
    n = sum(int(rec["start"][i]) < length for i in range(rec["n_seg"]))
    out["n_seg"], out["seq_len"], out["start"] = n, length, length
    out["start"][:n] = rec["start"][:n]
    for f in ("k_min", "k_scale", "v_min", "v_scale"):
        out[f][:n] = rec[f][:n]
    for inv, scale in (("k_inv_last", "k_scale"), ("v_inv_last", "v_scale")):
        if n == rec["n_seg"]:
            out[inv] = rec[inv]
        elif n and rec[scale][n - 1] != 0:
            out[inv] = np.float32(1) / rec[scale][n - 1]
    return out


class Forked:
    """Requests compressed by the oracle into pages that a pool handed out, and forks of request 1 at
    lengths in its last page, earlier pages, earlier segments, at their edges and at nothing."""

    def __init__(self, steps, seed=5, lens=(16, 3000, 40), hkv=2, split=False):
        from int8_group_quantized_gb300 import BlockPool
        self.case = c = Case(lens, hq=4, hkv=hkv, bs=BS, seed=seed)
        self.steps, self.split = steps, split
        probe = oracle.compress(c.k, c.v, c.cu, hkv, BS, c.bt, c.num_blocks)[2]
        starts = sorted({int(x) for h in range(hkv) for x in probe[1, h]["start"][1:probe[1, h]["n_seg"]]})
        assert starts, "request 1 has to have several segments"
        n = lens[1]
        cuts = {n, n - 1, n - n % BS, n - n % BS - 1, n - 5 * BS, 20, 16, 1, 0}
        for s in starts:
            cuts |= {s - 1, s, s + 1}
        self.cuts = sorted(x for x in cuts if 0 <= x <= n)
        rows = len(lens) + len(self.cuts)
        columns = (max(lens) + steps + BS - 1) // BS
        self.blocks = sum((x + BS - 1) // BS for x in lens) + rows * (2 + steps // BS) + 4
        self.pool = BlockPool(self.blocks)
        self.table = np.zeros((rows, columns), dtype=np.int32)
        for b, x in enumerate(lens):
            self.pool.alloc_table_row(x, BS, self.table, b)
        assert self.table[0, 0] == 0        # block 0 belongs to another request than the one that is forked
        bt = self.table[:len(lens)].copy()
        if split:
            self.kp, self.vp, *self.first = oracle.compress_split(c.k, c.v, c.cu, hkv, BS, bt, self.blocks)
        else:
            self.kp, self.vp, *self.first = oracle.compress(c.k, c.v, c.cu, hkv, BS, bt, self.blocks)
        self.forks = [(1, len(lens) + i, x) for i, x in enumerate(self.cuts)] + [(2, 2, 33)]  # and one cut in place
        pairs = [self.pool.fork_row(x, BS, self.table, 1, dst) for _, dst, x in self.forks[:-1]]
        self.pairs = np.concatenate(pairs)
        self.lens = np.array([lens[0], lens[1], 33] + self.cuts, dtype=np.int32)
        for r, x in enumerate(self.lens):   # blocks for the tokens to come (the row cut in place keeps its own)
            have = (int(lens[r] if r < len(lens) else x) + BS - 1) // BS
            for col in range(have, (int(x) + steps + BS - 1) // BS):
                self.table[r, col] = self.pool.alloc(1)[0]
        self.hkv, self.rows = hkv, rows

    def records(self, i, cutting=True):
        """All rows' records of table i before the appends: the forks' cut from their source's, or copied."""
        out = np.zeros((self.rows, self.hkv), dtype=oracle.SEG_DTYPE)
        out[:len(self.first[i])] = self.first[i]
        for src, dst, x in self.forks:
            for h in range(self.hkv):
                out[dst, h] = cut(self.first[i][src, h], x) if cutting else self.first[i][src, h]
        return out

    def tokens(self, step):
        k = synth.fill_heads(3, synth.STREAM_KNEW, 100 + step, self.rows, self.hkv, 0.5)
        v = synth.fill_heads(3, synth.STREAM_VNEW, 100 + step, self.rows, self.hkv, 0.5)
        return k, v

    def grown(self, cutting=True):
        """The oracle's pools and records after the page copies and all appends."""
        kp, vp = self.kp.copy(), self.vp.copy()
        for p in (kp, vp):
            p[self.pairs[:, 1]] = p[self.pairs[:, 0]]
        recs = [self.records(i, cutting) for i in range(len(self.first))]
        for s in range(self.steps):
            append = oracle.append_split if self.split else oracle.append
            append(*self.tokens(s), BS, self.table, kp, vp, *recs)
        return kp, vp, recs


@pytest.mark.parametrize("split", [False, True])
def test_cut_records_keep_appends_inside_the_row(split):
    """The model: with cut records an append touches the blocks of its own row only; with copied ones the
    forks' appends reach block 0, another request's."""
    f = Forked(3, split=split)
    kp, vp, recs = f.grown()
    owned = np.zeros(f.blocks, dtype=bool)
    for r, x in enumerate(f.lens):
        owned[f.table[r, int(x) // BS:(int(x) + 2) // BS + 1]] = True
    base = f.kp.copy()
    base[f.pairs[:, 1]] = base[f.pairs[:, 0]]
    assert np.array_equal(kp[~owned], base[~owned])
    assert np.array_equal(kp[0], f.kp[0])
    assert all((r["seq_len"][:, 0] == f.lens + 3).all() for r in recs)
    copied, _, _ = f.grown(cutting=False)
    assert not np.array_equal(copied[0], f.kp[0])


def test_factor_of_an_earlier_segment_is_the_encoders():
    """1 / scale against 255 / (max - min) of the segment's own values: two roundings, 2^-24 each."""
    f = Forked(0)
    c, rec = f.case, f.first[0]
    k = (c.k.astype(np.uint32) << 16).view(np.float32)[c.cu[1]:c.cu[2]]
    seen = 0
    for h in range(f.hkv):
        r = rec[1, h]
        for s in range(r["n_seg"] - 1):
            x = k[r["start"][s]:r["start"][s + 1], h]
            want = 255.0 / np.float64(x.max() - x.min())
            got = np.float64(cut(r, int(r["start"][s]) + 1)["k_inv_last"])
            assert abs(got - want) <= want * 2.0 ** -23 * (1 + 2.0 ** -20)
            seen += 1
    assert seen


def test_refusals():
    import int8_group_quantized_gb300 as dgq
    L = dgq.lib()

    def call(table=FAKE, rows=4, hkv=2, forks=FAKE, n=3, ws=FAKE, wsb=256):
        return L.dgq_fork_records(table, rows, hkv, forks, n, ws, wsb, 0)
    for kw in (dict(table=0), dict(table=FAKE + 8), dict(rows=0), dict(hkv=0), dict(n=-1), dict(forks=0),
               dict(forks=FAKE + 4)):
        assert call(**kw) == INVALID, kw
    assert call(n=1 << 30) == UNSUPPORTED
    assert call(ws=0) == WORKSPACE and call(wsb=255) == WORKSPACE
    assert call(n=0, forks=0) == OK


@pytest.mark.gpu
@pytest.mark.parametrize("split", [False, True])
def test_forks_at_any_length_append_and_decode_as_the_oracle(split):
    import torch
    import int8_group_quantized_gb300 as dgq
    f = Forked(20, split=split)
    dev = torch.device("cuda:0")
    kp, vp = torch.from_numpy(f.kp).to(dev), torch.from_numpy(f.vp).to(dev)
    recs = []
    for t in f.first:
        raw = np.zeros((f.rows, f.hkv, 128), dtype=np.uint8)
        raw[:len(t)] = t.view(np.uint8).reshape(*t.shape, 128)
        recs.append(torch.from_numpy(raw).to(dev))
    ws = torch.zeros(dgq.dgq_append_workspace_size(), dtype=torch.uint8, device=dev)
    dgq.dgq_copy_pages([kp, vp], torch.from_numpy(f.pairs).to(dev), ws)
    forks = torch.tensor(f.forks, dtype=torch.int32, device=dev)
    for i, r in enumerate(recs):
        dgq.dgq_fork_records(r, forks, ws)
        want, got = f.records(i), table_to_numpy(r)
        assert got.tobytes() == want.tobytes(), first_record_diff(want, got)
    bt = torch.from_numpy(f.table).to(dev)
    for s in range(f.steps):
        k, v = (torch.from_numpy(x.view(np.int16)).to(dev).view(torch.bfloat16) for x in f.tokens(s))
        if split:
            dgq.dgq_append_split(k, v, BS, bt, kp, vp, *recs, ws)
        else:
            dgq.dgq_append(k, v, BS, bt, kp, vp, *recs, ws)
    assert dgq.dgq_workspace_error(ws) == 0
    want_k, want_v, want = f.grown()
    for w, r in zip(want, recs):
        got = table_to_numpy(r)
        assert got.tobytes() == w.tobytes(), first_record_diff(w, got)
    assert np.array_equal(kp.cpu().numpy(), want_k) and np.array_equal(vp.cpu().numpy(), want_v)
    if split:
        return
    hq, lens = 4, f.lens + f.steps
    q = synth.fill_heads(8, synth.STREAM_Q, 0, f.rows, hq, 1.0)
    kn, vn = (synth.fill_heads(9, s, 0, f.rows, f.hkv, 0.15) for s in (synth.STREAM_KNEW, synth.STREAM_VNEW))
    ref = oracle.paged_decode_attn(q, kn, vn, want_k, want_v, want[0], f.table, lens)
    aws = torch.zeros(dgq.dgq_attn_workspace_size(f.rows, hq, f.hkv, int(lens.max())), dtype=torch.uint8, device=dev)
    out = torch.zeros(f.rows, hq, 128, dtype=torch.bfloat16, device=dev)
    d = [torch.from_numpy(x.view(np.int16)).to(dev).view(torch.bfloat16) for x in (q, kn, vn)]
    dgq.dgq_paged_decode_attn(*d, kp, vp, recs[0], bt, torch.from_numpy(lens).to(dev), int(lens.max()), out, aws)
    assert dgq.dgq_workspace_error(aws) == 0
    assert_attn_close(ref, out.double().cpu().numpy())


@pytest.mark.gpu
@pytest.mark.parametrize("bad,code", [((3, 1, 4), 5), ((-1, 1, 4), 5), ((0, 3, 4), 5), ((0, -1, 4), 5), ((0, 1, 17), 6),
                                      ((0, 1, -1), 6), ((0, 1, 2 ** 31 - 1), 6)])
def test_bad_forks_are_flagged_and_leave_their_row(bad, code):
    import torch
    import int8_group_quantized_gb300 as dgq
    c = Case([16, 40, 40], hq=4, hkv=2, bs=BS, seed=2)
    _, _, table = c.oracle_compress()
    rec = torch.from_numpy(table.view(np.uint8).reshape(3, 2, 128).copy()).cuda()
    before = rec.clone()
    ws = torch.zeros(dgq.dgq_append_workspace_size(), dtype=torch.uint8, device="cuda")
    dgq.dgq_fork_records(rec, torch.tensor([bad, (0, 2, 7)], dtype=torch.int32, device="cuda"), ws)
    assert dgq.dgq_workspace_error(ws) == code
    assert torch.equal(rec[:2], before[:2])
    assert table_to_numpy(rec)[2, 1].tobytes() == cut(table[0, 1], 7).tobytes()


@pytest.mark.gpu
def test_forks_of_a_replayed_graph_read_the_list_as_it_is():
    import torch
    import int8_group_quantized_gb300 as dgq
    c = Case([16, 40], hq=4, hkv=2, bs=BS, seed=2)
    _, _, table = c.oracle_compress()
    rec = torch.from_numpy(table.view(np.uint8).reshape(2, 2, 128).copy()).cuda()
    rec = torch.cat([rec, torch.zeros_like(rec[:1])])
    ws = torch.zeros(dgq.dgq_append_workspace_size(), dtype=torch.uint8, device="cuda")
    forks = torch.tensor([[1, 2, 9]], dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dgq.dgq_fork_records(rec, forks, ws)
    for length in (9, 40, 0):
        forks[0, 2] = length
        graph.replay()
        assert dgq.dgq_workspace_error(ws) == 0
        assert table_to_numpy(rec)[2, 0].tobytes() == cut(table[1, 0], length).tobytes()
