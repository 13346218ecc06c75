"""What one infinity or NaN of a row does to the rest of the row in block_norm: the formula's own values, in every channel.

RMS: the mean square is infinite, so the infinite channel is inf / inf = NaN and every other v / inf + bias = bias (0 without one). Layer: the mean is
infinite and the differences are NaN, so the row is. A norm before the residual leaves a NaN in r, which makes y's row NaN.
"""
import pytest

from tests.test_block_norm import draw, vectors
from tests.test_fp8_linear import fmpq_mod  # noqa: F401  (the fixture)

BLOCK = 128


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,pad", [(9, 256, 0), (9, 4096, 0), (9, 17000, 0), (400, 4096, 0), (400, 2003, 0), (330, 17003, 1), (1300, 300, 0), (700, 513, 5)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_whole_rows(fmpq_mod, M, K, pad, kind, value):  # noqa: F811
    import torch
    at = K // 3
    X, residual = draw(M, K, torch.bfloat16, 1, pad), draw(M, K, torch.bfloat16, 2, pad)
    weight, bias = vectors(K, torch.bfloat16, 3, 2)
    layer = fmpq_mod.Fp8Layer(K, 16)

    def run(X, residual, **kw):
        Y = torch.empty(M, K, dtype=X.dtype, device="cuda")
        return fmpq_mod.block_norm(X, residual, kind=kind, weight=weight, layer=layer, Y=Y, **kw)

    for kw in (dict(), dict(bias=bias)):
        bad = residual.clone()
        bad[4, at] = value
        clean, out = run(X, residual, **kw), run(X, bad, **kw)
        rest = [m for m in range(M) if m != 4]
        for got, want in ((out.Y, clean.Y), (out.R, clean.R), (out.a_scales[:, :M].t(), clean.a_scales[:, :M].t()),
                          (out.A_packed.transpose(0, 1), clean.A_packed.transpose(0, 1))):
            assert torch.equal(got[rest], want[rest])
        others = torch.arange(K, device="cuda") != at
        assert torch.equal(out.R[4, others], clean.R[4, others])
        assert bool(out.R[4, at].isnan()) if value != value else float(out.R[4, at]) == value
        scales = out.a_scales[:, 4]
        if kind == "layer" or value != value:
            assert bool(out.Y[4].isnan().all()) and bool(scales.isnan().all())
            continue
        want = bias if "bias" in kw else torch.zeros(K, dtype=X.dtype, device="cuda")
        assert bool(out.Y[4, at].isnan()) and bool((out.Y[4, others] == want[others]).all())
        top = torch.nn.functional.pad(want.float().abs(), (0, -K % BLOCK)).view(-1, BLOCK).amax(1)
        top = top / torch.full_like(top, 448)
        blocks = torch.arange(len(scales), device="cuda") != at // BLOCK
        assert bool(scales[at // BLOCK].isnan()) and torch.equal(scales[blocks], top[blocks])
    # an infinity before the norm of X
    bad = X.clone()
    bad[4, at] = value
    out = run(bad, residual, post_norm=True)
    assert bool(out.R[4, at].isnan()) and bool(out.Y[4].isnan().all()) and bool(out.a_scales[:, 4].isnan().all())
    if kind == "rms" and value == value:
        assert torch.equal(out.R[4, others], residual[4, others])
    else:
        assert bool(out.R[4].isnan().all())
