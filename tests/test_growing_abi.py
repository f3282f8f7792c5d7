"""Refusals of the calls around a growing cache and of windowed attention: every check runs on the host before
any launch, so no GPU is needed."""
import pytest

from int8_group_quantized_gb300 import _build

FAKE = 0x10000
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3


@pytest.fixture(scope="module")
def L():
    import int8_group_quantized_gb300 as dgq
    _build.build()
    return dgq.lib()


def caller(f, names, defaults):
    def call(**kw):
        a = dict(defaults, **kw)
        assert set(kw) <= set(names)
        return f(*(a[n] for n in names))
    return call


def check_pointers(call, *names, status=INVALID):
    for n in names:
        assert call(**{n: 0}) == status, n
        assert call(**{n: FAKE + 4}) == status, n


def test_extend_tables(L):
    names = "lens new batch bs nb ids nf used bt mb slots ts cu lo uo ws wsb stream".split()
    call = caller(L.dgq_extend_tables, names, dict(
        {n: FAKE for n in names}, batch=2, bs=16, nb=64, nf=8, mb=19, ts=10, wsb=256, stream=0))
    assert L.dgq_extend_tables_workspace_size() == 256
    check_pointers(call, *"lens new ids used bt slots cu lo uo".split())
    check_pointers(call, "ws", status=WORKSPACE)
    assert call(wsb=255) == WORKSPACE
    for bad in (dict(batch=0), dict(batch=8193), dict(nb=0), dict(mb=0), dict(nf=-1), dict(ts=-1)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(bs=8), dict(bs=48), dict(nb=1 << 28), dict(mb=(1 << 26) + 1)):
        assert call(**bad) == UNSUPPORTED, bad


ROWS = "k v ks vs T hkv d slots kp vp nb bs ws wsb stream".split()


def rows_refusals(call):
    check_pointers(call, "k", "v", "slots", "kp", "vp")
    check_pointers(call, "ws", status=WORKSPACE)
    assert call(wsb=255) == WORKSPACE
    for bad in (dict(T=-1), dict(hkv=0), dict(nb=0), dict(ks=2 * 128 - 8), dict(vs=2 * 128 + 4), dict(ks=0), dict(vs=-256)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(d=64), dict(bs=24), dict(nb=1 << 27), dict(T=1 << 26)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(T=0, k=0, v=0, slots=0, ks=0, vs=0) == 0        # no tokens: nothing is launched


def test_write_slots(L):
    rows_refusals(caller(L.dgq_write_slots, ROWS, dict(
        {n: FAKE for n in ROWS}, ks=256, vs=256, T=5, hkv=2, d=128, nb=8, bs=16, wsb=256, stream=0)))


def test_store_block8(L):
    names = "fmt k v ks vs T hkv d slots kp vp ksc vsc nb bs ws wsb stream".split()
    call = caller(L.dgq_store_block8, names, dict(
        {n: FAKE for n in names}, fmt=0, ks=256, vs=256, T=5, hkv=2, d=128, nb=8, bs=16, wsb=256, stream=0))
    assert L.dgq_block8_workspace_size() == 256
    rows_refusals(call)
    check_pointers(call, "ksc", "vsc")
    assert call(fmt=2) == INVALID and call(fmt=-1) == INVALID


def test_load_block8(L):
    names = "fmt kp vp ksc vsc nb bs bt mb cu batch hkv d k v total ws wsb stream".split()
    call = caller(L.dgq_load_block8, names, dict(
        {n: FAKE for n in names}, fmt=1, nb=8, bs=32, mb=4, batch=2, hkv=2, d=128, total=50, wsb=256, stream=0))
    check_pointers(call, *"kp vp ksc vsc bt cu k v".split())
    check_pointers(call, "ws", status=WORKSPACE)
    for bad in (dict(fmt=3), dict(batch=0), dict(batch=8193), dict(hkv=0), dict(nb=0), dict(mb=0), dict(total=-1)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(d=64), dict(bs=8), dict(nb=1 << 27), dict(total=1 << 30)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(total=0, k=0, v=0) == 0


DECODE = ("lens max_seqlen batch hq hkv d bs mb nb win sinks out ws wsb stream").split()
SIZES = dict(max_seqlen=300, batch=2, hq=4, hkv=2, d=128, bs=16, mb=19, nb=32, win=64, sinks=4, wsb=1 << 30, stream=0)


def decode_refusals(call):
    for bad in (dict(win=0, sinks=1), dict(win=-1), dict(sinks=-1), dict(max_seqlen=305), dict(batch=0), dict(hq=5)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(d=64), dict(bs=48), dict(hq=32)):
        assert call(**bad) == UNSUPPORTED, bad
    check_pointers(call, "q", "kn", "vn", "kp", "vp", "bt", "lens", "out")


def test_decode_windows(L):
    names = "q kn vn kp vp table bt".split() + DECODE
    call = caller(L.dgq_paged_decode_attn_window, names, dict({n: FAKE for n in names}, **SIZES))
    decode_refusals(call)
    check_pointers(call, "table")
    assert call(win=0, sinks=0) == INVALID
    names = "q kn vn kp vp nb bt mb lens max_seqlen batch hq hkv d bs win sinks out ws wsb stream".split()
    call = caller(L.dgq_paged_decode_attn_bf16_window, names, dict({n: FAKE for n in names}, **SIZES))
    decode_refusals(call)
    assert call(win=0, sinks=0) == INVALID


def test_decode_block8(L):
    names = "fmt q kn vn kp vp ksc vsc bt".split() + DECODE
    call = caller(L.dgq_paged_decode_attn_block8, names, dict({n: FAKE for n in names}, fmt=0, **SIZES))
    decode_refusals(call)
    check_pointers(call, "ksc", "vsc")
    assert call(fmt=2) == INVALID and call(fmt=-1) == INVALID


def test_prompt_windows(L):
    packed = "q k v tq tkv cq ck batch hq hkv d win sinks out ws wsb stream".split()
    paged = "q tq cq k v nb bt mb lens batch hq hkv d bs win sinks out ws wsb stream".split()
    sizes = dict(tq=50, tkv=60, batch=2, hq=4, hkv=2, d=128, win=8, sinks=1, wsb=1 << 30, stream=0, nb=32, mb=19, bs=16)
    for f, names in ((L.dgq_prompt_attn_window, packed), (L.dgq_prompt_attn_paged_window, paged)):
        call = caller(f, names, dict({n: FAKE for n in names}, **{n: v for n, v in sizes.items() if n in names}))
        for bad in (dict(win=0), dict(win=0, sinks=0), dict(win=-5), dict(sinks=-1), dict(tq=-1), dict(hq=5)):
            assert call(**bad) == INVALID, bad
        for bad in (dict(d=64), dict(hq=32)):
            assert call(**bad) == UNSUPPORTED, bad
        check_pointers(call, "q", "k", "v", "out", "cq")


def test_binding_refuses_windows_that_say_nothing():
    import int8_group_quantized_gb300 as dgq
    assert dgq._windowed("x", 0, 0) is False and dgq._windowed("x", 1, 0) is True
    for window, sinks in ((0, 1), (-1, 0), (5, -1)):
        with pytest.raises(dgq.DGQError):
            dgq._windowed("x", window, sinks)
