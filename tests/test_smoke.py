"""smoke() runs both paths of the library: the W4Ax step and a routed step on E4M3 weights."""
import pytest


@pytest.mark.gpu
def test_smoke_runs_a_routed_step(capsys, monkeypatch):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__ as entry
    from bit_quantized_gemm_fmpq_gb300 import build, fmpq
    build.build()
    ran = []
    for name in ("fmpq_quantize", "w4ax_gemm", "fp8_pack_weights", "moe_route", "moe_experts"):
        call = getattr(fmpq, name)
        monkeypatch.setattr(fmpq, name, lambda *a, _call=call, _name=name, **kw: ran.append(_name) or _call(*a, **kw))
    entry.smoke()
    assert {"fmpq_quantize", "w4ax_gemm", "fp8_pack_weights", "moe_route", "moe_experts"} <= set(ran)
    assert "routed experts" in capsys.readouterr().out
