"""The checks on tensors run natively where that module is built and in Python elsewhere: both give the same
answers to the same operands.  CPU only: the device is a stand-in where there is no GPU."""
import pytest
import torch


@pytest.fixture
def dgq(monkeypatch):
    import int8_group_quantized_gb300 as dgq
    return dgq


def test_native_module_is_built_and_found(dgq, monkeypatch):
    from int8_group_quantized_gb300 import _build
    _build.build()
    monkeypatch.setattr(dgq, "_native_module", False)       # (looked for before it was built)
    assert dgq._native() is not None
    assert dgq._native().__name__.endswith("_tensors")


def test_entry_points_without_ctypes(dgq, monkeypatch):
    """Same statuses; an argument that does not fit its C type is an error and not cut."""
    monkeypatch.setattr(dgq, "_native_module", False)
    native, fake = dgq._native(), 0x10000
    rows = [fake, fake, 256, 256, 5, 2, 128, fake, fake, fake, 8, 16, fake, 256, 0]
    for change, status in (({}, None), ({4: 0}, 0), ({4: -1}, -1), ({6: 64}, -2), ({13: 255}, -3), ({0: fake + 4}, -1)):
        args = [change.get(i, a) for i, a in enumerate(rows)]
        if status is not None:
            assert native.dgq_write_slots(*args) == status == dgq.lib().dgq_write_slots(*args)
    for bad in ({4: 1 << 32}, {13: -1}, {2: 1 << 70}):
        with pytest.raises(OverflowError):
            native.dgq_write_slots(*[bad.get(i, a) for i, a in enumerate(rows)])
    with pytest.raises(TypeError):
        native.dgq_write_slots(*rows[:-1])
    with pytest.raises(TypeError):
        native.dgq_write_slots(*[None] + rows[1:])


def test_host_tensors_are_refused_by_both(dgq, monkeypatch):
    x, ws = torch.zeros(3, dtype=torch.int32), torch.zeros(256, dtype=torch.uint8)
    for native in (dgq._native(), None):
        monkeypatch.setattr(dgq, "_native", lambda: native)
        with pytest.raises(dgq.DGQError):
            dgq._operands("x", ws, (x, torch.int32, (3,)))
        with pytest.raises(dgq.DGQError):
            dgq._token_rows("x", torch.zeros(2, 2, 128, dtype=torch.bfloat16))


def test_tensors_of_other_kinds_are_errors_and_not_the_end_of_the_process(dgq, monkeypatch):
    ws = torch.zeros(256, dtype=torch.uint8)
    sparse = torch.eye(3).to_sparse()
    others = [(ws, (sparse, torch.float32, (3, 3))), (sparse, (ws, torch.uint8, (256,))),
              (ws, (torch.empty(3, device="meta"), torch.float32, (3,))), (ws, (None, torch.float32, (3,))),
              (ws, ("x", torch.float32, (3,))), (None, (ws, torch.uint8, (256,)))]
    rows = [torch.eye(3).to_sparse(), torch.empty(2, 2, 128, dtype=torch.bfloat16, device="meta"),
            torch.zeros(2, 128, dtype=torch.bfloat16)]
    monkeypatch.setattr(dgq, "_native_module", False)
    for native in (dgq._native(), None):
        monkeypatch.setattr(dgq, "_native", lambda: native)
        for w, spec in others:
            with pytest.raises((RuntimeError, AttributeError)):
                dgq._operands("x", w, spec)
        for x in rows:
            with pytest.raises((RuntimeError, AttributeError, ValueError)):
                dgq._token_rows("x", x)


@pytest.mark.gpu
def test_both_give_the_same_answers(dgq, monkeypatch):
    d = "cuda"
    i, f = torch.arange(12, dtype=torch.int32, device=d), torch.zeros(3, 4, device=d)
    ws = torch.zeros(256, dtype=torch.uint8, device=d)
    empty = torch.zeros(0, dtype=torch.int32, device=d)
    fused = torch.zeros(5, 6, 128, dtype=torch.bfloat16, device=d)
    operands = [
        (ws, ((i, torch.int32, (12,)), (f, torch.float32, (3, 4)))), (ws, ((empty, torch.int32, (0,)),)), (ws, ()),
        (ws, ((i, torch.int64, (12,)),)), (ws, ((i, torch.int32, (11,)),)), (ws, ((i, torch.int32, (12, 1)),)),
        (ws, ((i, torch.int32, ()),)), (ws, ((f.t(), torch.float32, (4, 3)),)), (ws, ((f[:, :2], torch.float32, (3, 2)),)),
        (ws, ((i.cpu(), torch.int32, (12,)),)), (ws[::2], ((i, torch.int32, (12,)),)), (ws.cpu(), ((i, torch.int32, (12,)),)),
        (ws, ((torch.nn.Parameter(f), torch.float32, (3, 4)),)), (ws, ((i.view(3, 4), torch.int32, (3, torch.Size([4])[0])),)),
    ]
    token_rows = [(fused[:, :2], fused[:, 2:4]), (fused[:, :1],), (fused[:, ::2],), (fused[:, :2], fused[:, :3]), (fused[:0],),
                  (fused.half(),), (fused.cpu(),), (fused[..., :64],), (fused[:, :1, ::2],), (fused[:1].expand(5, 6, 128),),
                  (fused[:, 3:4].transpose(0, 1),)]

    def answers():
        for w, specs in operands:
            try:
                yield dgq._operands("x", w, *specs)
            except dgq.DGQError as e:
                yield e.status
        for xs in token_rows:
            try:
                yield dgq._token_rows("x", *xs)
            except dgq.DGQError as e:
                yield e.status
    native = list(answers())
    monkeypatch.setattr(dgq, "_native", lambda: None)
    assert native == list(answers())
    assert native[0] == [i.data_ptr(), f.data_ptr(), ws.data_ptr()] and native.count(-1) == 9 + 7  # refused operands, refused rows
