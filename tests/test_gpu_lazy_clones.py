"""Operands that share their storage until one of them is written (torch's lazy clones): a call that writes one
leaves the tensor that it was cloned from as it was, with the native checks and with those in Python."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("native", [True, False])
def test_what_is_written_is_the_clone(native, monkeypatch):
    import int8_group_quantized_gb300 as dgq
    assert dgq._native() is not None
    if not native:
        monkeypatch.setattr(dgq, "_native", lambda: None)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    kept = dict(table=torch.full((2, 4), -1, dtype=torch.int32, device="cuda"), slots=i32(7, 7), cu=i32(9, 9, 9), lens=i32(16, 3),
                used=i32(0), ws=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    before = {n: x.clone() for n, x in kept.items()}
    c = {n: torch._lazy_clone(x) for n, x in kept.items()}
    table = torch._lazy_clone(kept["table"])
    table[1, 0] = 5
    dgq.dgq_extend_tables(kept["lens"], i32(1, 1), 16, 8, i32(3, 2), kept["used"], table, c["slots"], c["cu"], c["lens"],
                          c["used"], c["ws"])
    torch.cuda.synchronize()
    assert dgq.dgq_workspace_error(c["ws"]) == 0
    assert c["slots"].tolist() == [48, 83] and c["cu"].tolist() == [0, 1, 2] and c["lens"].tolist() == [17, 4] and c["used"].tolist() == [1]
    for n, x in kept.items():
        assert torch.equal(x, before[n]), n

    q, kv = (torch.randn(2, h, 128, device="cuda").to(torch.bfloat16) for h in (4, 2))
    pages = torch.randn(8, 2, 16, 128, device="cuda").to(torch.bfloat16)
    pages_before, zeros = pages.clone(), torch.zeros_like(q)
    out, new = torch._lazy_clone(zeros), torch._lazy_clone(pages)
    dgq.dgq_write_slots(kv, kv, i32(0, 17), new, torch.zeros_like(pages), ws)
    aws = torch.zeros(dgq.dgq_attn_workspace_size(2, 4, 2, 16), dtype=torch.uint8, device="cuda")
    dgq.dgq_paged_decode_attn_bf16(q, kv, kv, pages, pages, torch.zeros(2, 1, dtype=torch.int32, device="cuda"), i32(16, 3), 16, out, aws)
    torch.cuda.synchronize()
    assert torch.equal(pages, pages_before) and not zeros.any() and out.any()
    assert torch.equal(new[0, :, 0], kv[0]) and torch.equal(new[1, :, 1], kv[1])
