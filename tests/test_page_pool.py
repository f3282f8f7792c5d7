"""The host block pool's references: sharing, forked rows, copy on write, freed rows and compaction,
against a plain model; refusals leave the pool and the table unchanged.  And the refusals of the bf16
attention and page calls before any launch.  CPU only."""
import random

import numpy as np
import pytest

from int8_group_quantized_gb300 import _build

OK, INVALID, UNSUPPORTED, WORKSPACE, EXHAUSTED = 0, -1, -2, -3, -5
FAKE = 0x10000  # a 16-byte aligned address that is never dereferenced: checks fail first


@pytest.fixture(scope="module")
def dgq():
    _build.build()
    import int8_group_quantized_gb300 as m
    m.lib()
    return m


def refs(pool):
    return [pool.references(i) for i in range(pool.num_blocks)]


def test_share_and_free(dgq):
    p = dgq.BlockPool(4)
    a = p.alloc(2)
    p.share(a)
    assert refs(p) == [2, 2, 0, 0] and p.num_free() == 2
    p.free(a)
    assert refs(p) == [1, 1, 0, 0] and p.num_free() == 2
    p.free([a[0]])
    assert refs(p) == [0, 1, 0, 0] and p.num_free() == 3
    for bad in ([a[0]], [9], [-1], [a[1], a[1]], [a[1], 3]):
        for call in (p.free, p.share):
            with pytest.raises(dgq.DGQError):
                call(bad)
        assert refs(p) == [0, 1, 0, 0]
    assert p.references(4) == -1 and p.references(-1) == -1
    assert p.alloc(3) == [0, 2, 3]


@pytest.mark.parametrize("length", [0, 1, 15, 16, 17, 32, 47, 48])
def test_fork_row(dgq, length):
    p = dgq.BlockPool(8)
    t = np.full((3, 4), 77, dtype=np.int32)
    p.alloc_table_row(48, 16, t, 1)
    pairs = p.fork_row(length, 16, t, 1, 0)
    whole, n = length // 16, (length + 15) // 16
    assert t[0, :whole].tolist() == t[1, :whole].tolist() and (t[0, n:] == 0).all() and (t[2] == 77).all()
    assert [p.references(int(b)) for b in t[1, :3]] == [2 if i < whole else 1 for i in range(3)]
    if n > whole:
        assert pairs.tolist() == [[t[1, whole], t[0, whole]]] and p.references(int(t[0, whole])) == 1
        assert t[0, whole] != t[1, whole]
    else:
        assert pairs.shape == (0, 2)


def test_fork_row_refusals_change_nothing(dgq):
    p = dgq.BlockPool(3)
    t = np.zeros((2, 4), dtype=np.int32)
    p.alloc_table_row(40, 16, t, 0)
    before, r = t.copy(), refs(p)
    for args in ((40, 16, t, 0, 1), ):                                    # a partial block, none free
        with pytest.raises(dgq.DGQError) as e:
            p.fork_row(*args)
        assert e.value.status == EXHAUSTED
    for args in ((32, 16, t, 0, 0), (65, 16, t, 0, 1), (-1, 16, t, 0, 1), (16, 0, t, 0, 1), (16, 16, t, 0, 2),
                 (16, 16, t, -1, 1), (64, 16, t, 0, 1)):                  # same row, too long, ..., unowned block
        with pytest.raises(dgq.DGQError) as e:
            p.fork_row(*args)
        assert e.value.status == INVALID
    with pytest.raises(dgq.DGQError):
        p.fork_row(16, 16, t.astype(np.int64), 0, 1)
    with pytest.raises(dgq.DGQError):
        p.fork_row(16, 16, np.zeros((2, 8), dtype=np.int32)[:, ::2], 0, 1)
    assert (t == before).all() and refs(p) == r
    assert p.fork_row(32, 16, t, 0, 1).shape == (0, 2)                    # whole blocks need no free one


def test_own_row_copies_only_what_is_shared(dgq):
    p = dgq.BlockPool(10)
    t = np.zeros((2, 4), dtype=np.int32)
    p.alloc_table_row(64, 16, t, 0)
    p.fork_row(48, 16, t, 0, 1)
    old = t.copy()
    pairs = p.own_row(t, 0, 1, 3)                                         # blocks 1, 2 shared, 3 its own
    assert pairs.tolist() == [[old[0, 1], t[0, 1]], [old[0, 2], t[0, 2]]]
    assert t[0, 0] == old[0, 0] and t[0, 3] == old[0, 3] and (t[1] == old[1]).all()
    assert len(set(t[0].tolist())) == 4 and not set(t[0, 1:3].tolist()) & set(old.flatten().tolist())
    assert [p.references(int(b)) for b in old[0]] == [2, 1, 1, 1]
    assert p.own_row(t, 0, 1, 3).shape == (0, 2)
    with pytest.raises(dgq.DGQError):
        p.own_row(t, 0, 2, 3)


def test_own_row_is_all_or_nothing(dgq):
    p = dgq.BlockPool(5)
    t = np.zeros((2, 4), dtype=np.int32)
    p.alloc_table_row(64, 16, t, 0)
    p.fork_row(64, 16, t, 0, 1)
    before, r = t.copy(), refs(p)
    with pytest.raises(dgq.DGQError) as e:
        p.own_row(t, 1, 0, 2)
    assert e.value.status == EXHAUSTED and (t == before).all() and refs(p) == r


def test_free_row(dgq):
    p = dgq.BlockPool(8)
    t = np.zeros((2, 4), dtype=np.int32)
    p.alloc_table_row(40, 16, t, 0)
    p.fork_row(40, 16, t, 0, 1)
    p.free_row(t, 0, 3)
    assert (t[0] == 0).all() and p.num_free() == 8 - 3
    with pytest.raises(dgq.DGQError):
        p.free_row(t, 1, 5)
    p.free_row(t, 1, 3)
    assert p.num_free() == 8 and refs(p) == [0] * 8


@pytest.mark.parametrize("blocks", [1, 2, 7, 64, 301])
def test_compact_against_a_model(dgq, blocks):
    r = random.Random(blocks)
    p = dgq.BlockPool(blocks)
    content, held = {}, []                     # block -> what it holds; one entry per reference
    for step in range(40):
        ids = p.alloc(r.randint(0, p.num_free()))
        for i in ids:
            content[i] = (step, i)
            held.append(i)
        shared = [i for i in set(held) if r.random() < 0.2]
        p.share(shared)
        held += shared
        r.shuffle(held)
        drop, keep, seen = [], [], set()
        for i in held:
            if r.random() < 0.5 and i not in seen:
                drop.append(i)
                seen.add(i)
            else:
                keep.append(i)
        p.free(drop)
        held = keep
        before = {i: p.references(i) for i in range(blocks)}
        remap, pairs = p.compact()
        live = sorted(set(held))
        n = len(live)
        assert sorted(int(remap[i]) for i in live) == list(range(n))
        src, dst = pairs[:, 0].tolist(), pairs[:, 1].tolist()
        assert not set(src) & set(dst) and len(set(dst)) == len(dst) and len(src) <= blocks // 2
        assert all(s >= n for s in src) and all(d < n and before[d] == 0 for d in dst)
        assert [int(remap[s]) for s in src] == dst
        assert all(remap[i] == i for i in range(blocks) if i not in src)
        assert all(p.references(int(remap[i])) == before[i] for i in live)
        assert p.num_free() == blocks - n and all(p.references(i) == 0 for i in range(n, blocks))
        content = {int(remap[i]): content[i] for i in live}
        held = [int(remap[i]) for i in held]
        assert len(content) == n
    if p.num_free():
        assert p.alloc(1) == [len(set(held))]


# ---- refusals before any launch -----------------------------------------------------------------------

def _prompt(L, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, tq=300, tkv=300, cuq=FAKE, cukv=FAKE, b=2, hq=4, hkv=2, d=128, out=FAKE, ws=FAKE,
             wsb=1 << 40)
    a.update(kw)
    return L.dgq_prompt_attn(*(a[n] for n in "q k v tq tkv cuq cukv b hq hkv d out ws wsb".split()), 0)


def _paged(L, **kw):
    a = dict(q=FAKE, tq=300, cuq=FAKE, k=FAKE, v=FAKE, nb=32, bt=FAKE, mb=19, lens=FAKE, b=2, hq=4, hkv=2, d=128, bs=16,
             out=FAKE, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return L.dgq_prompt_attn_paged(*(a[n] for n in "q tq cuq k v nb bt mb lens b hq hkv d bs out ws wsb".split()), 0)


def test_prompt_refusals(dgq):
    L = dgq.lib()
    for call in (_prompt, _paged):
        assert call(L, d=64) == UNSUPPORTED
        assert call(L, hq=48, hkv=3) == UNSUPPORTED                       # 16 query heads to a KV head
        assert call(L, hq=6, hkv=2) == UNSUPPORTED                        # 3
        for kw in (dict(hq=5), dict(b=0), dict(b=8193), dict(tq=-1), dict(hkv=0), dict(q=0), dict(k=0), dict(v=FAKE + 8),
                   dict(out=FAKE + 2), dict(cuq=0), dict(cuq=FAKE + 4), dict(out=0)):
            assert call(L, **kw) == INVALID, kw
        assert call(L, tq=1 << 30) == UNSUPPORTED                         # rows x heads past 32 bits
    assert _prompt(L, tkv=-1) == INVALID
    assert _prompt(L, cukv=0) == INVALID
    assert _paged(L, bs=48) == UNSUPPORTED
    assert _paged(L, nb=1 << 27) == UNSUPPORTED
    for kw in (dict(nb=0), dict(mb=0), dict(bt=0), dict(bt=FAKE + 4), dict(lens=0)):
        assert _paged(L, **kw) == INVALID, kw


def _decode(L, **kw):
    a = dict(q=FAKE, kn=FAKE, vn=FAKE, k=FAKE, v=FAKE, nb=32, bt=FAKE, mb=19, lens=FAKE, ms=300, b=2, hq=4, hkv=2, d=128,
             bs=16, out=FAKE, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return L.dgq_paged_decode_attn_bf16(
        *(a[n] for n in "q kn vn k v nb bt mb lens ms b hq hkv d bs out ws wsb".split()), 0)


def test_decode_bf16_refusals(dgq):
    L = dgq.lib()
    for kw in (dict(d=64), dict(bs=8), dict(hq=32, hkv=2), dict(nb=1 << 27)):
        assert _decode(L, **kw) == UNSUPPORTED, kw
    for kw in (dict(q=0), dict(kn=0), dict(k=FAKE + 8), dict(bt=0), dict(lens=0), dict(ms=305), dict(b=0), dict(hq=5),
               dict(nb=0), dict(out=0)):
        assert _decode(L, **kw) == INVALID, kw
    # the bf16 cache is not a dgq_format
    assert L.dgq_paged_decode_attn_format(16, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 300, 2, 4, 2,
                                          128, 16, 19, 32, FAKE, FAKE, 1 << 40, 0) == INVALID


def test_copy_pages_refusals(dgq):
    import ctypes
    L = dgq.lib()
    two = (ctypes.c_void_p * 2)(FAKE, FAKE)

    def copy(arr=two, n=2, size=64, pages=8, pairs=FAKE, np_=3, ws=FAKE, wsb=256):
        return L.dgq_copy_pages(arr, n, size, pages, pairs, np_, ws, wsb, 0)
    for kw in (dict(n=-1), dict(np_=-1), dict(size=0), dict(size=24), dict(pages=0), dict(arr=None), dict(pairs=0),
               dict(pairs=FAKE + 8), dict(arr=(ctypes.c_void_p * 2)(FAKE, 0)),
               dict(arr=(ctypes.c_void_p * 2)(FAKE, FAKE + 8))):
        assert copy(**kw) == INVALID, kw
    assert copy(ws=0) == WORKSPACE and copy(wsb=255) == WORKSPACE
    assert copy(size=1 << 41) == UNSUPPORTED
    assert copy(np_=0) == OK and copy(n=0) == OK                          # nothing to do: nothing launched

    def remap(t=FAKE, n=8, r=FAKE, pages=8, out=FAKE, ws=FAKE, wsb=256):
        return L.dgq_remap_tables(t, n, r, pages, out, ws, wsb, 0)
    for kw in (dict(n=-1), dict(pages=0), dict(t=0), dict(r=0), dict(out=0), dict(out=FAKE + 4)):
        assert remap(**kw) == INVALID, kw
    assert remap(wsb=10) == WORKSPACE and remap(n=0) == OK


def test_binding_refuses_what_pointers_would_misread(dgq):
    import torch
    bf, i32 = torch.bfloat16, torch.int32
    q, k = torch.zeros(8, 4, 128, dtype=bf), torch.zeros(8, 2, 128, dtype=bf)
    cu, ws = torch.zeros(2, dtype=i32), torch.zeros(256, dtype=torch.uint8)

    def prompt(q=q, k=k, v=k, cu_q=cu, cu_kv=cu, out=q):
        dgq.dgq_prompt_attn(q, k, v, cu_q, cu_kv, out, ws)
    for kw in (dict(q=q.half()), dict(k=k.float()), dict(v=k[:7]), dict(cu_kv=cu.long()), dict(out=q[:, :2]),
               dict(q=torch.zeros(8, 128, 4, dtype=bf).transpose(1, 2)), dict(cu_q=torch.zeros(3, dtype=i32)),
               dict(out=torch.zeros(9, 4, 128, dtype=bf))):
        with pytest.raises(dgq.DGQError) as e:
            prompt(**kw)
        assert e.value.status == INVALID
    pool = torch.zeros(4, 2, 16, 128, dtype=torch.uint8)
    pairs = torch.zeros(1, 2, dtype=i32)
    for arrs, pr in (([pool, pool[:3]], pairs), ([pool.transpose(0, 1)], pairs), ([pool], pairs.long()),
                     ([pool], pairs.flatten()), ([pool[:, :, ::2]], pairs)):
        with pytest.raises(dgq.DGQError):
            dgq.dgq_copy_pages(arrs, pr, ws)
    with pytest.raises(dgq.DGQError):
        dgq.dgq_remap_tables(pairs, pairs.flatten(), torch.zeros(2, dtype=i32), ws)
