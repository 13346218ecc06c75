"""The operators around the products as a model runs them: a dense feed-forward and one of routed 16-bit experts between their norms,
on E4M3 codes and residuals that never leave the library's formats; eager, captured and replayed on new inputs, on two streams at once.

Tolerance of the whole against 64 bits on the same weights: every step rounds to 16 bits once (half a step eps / 2 of the
value), the activations to E4M3 (2^-4 of a value at most, over K values of either sign); in norm the E4M3 parts lead:
sqrt(2) * 2^-4 / sqrt(3) for two of them in a row, of the feed-forward's share of the stream, which is below a half.
"""
import pytest

from tests.test_fp8_linear import fmpq_mod  # noqa: F401  (the fixture)


class Block:
    """Stream r: r += down(gelu(up(norm(r)) + b) + b'), r += experts(norm(r)), in the library's steps."""

    def __init__(self, fmpq, H, F, E, k):
        import torch
        g = torch.Generator().manual_seed(H)
        w = lambda *s: (torch.randn(*s, generator=g) / s[-1] ** 0.5).bfloat16().cuda()      # noqa: E731
        self.f, self.k, self.E = fmpq, k, E
        self.up, self.down = fmpq.Fp8Layer(H, F), fmpq.Fp8Layer(F, H)
        self.router = fmpq.W16Layer(H, E, torch.bfloat16)
        self.e_up = fmpq.W16Layer(H, 2 * F, torch.bfloat16, experts=E, gated=True)
        self.e_down = fmpq.W16Layer(F, H, torch.bfloat16, experts=E)
        self.w = dict(up=w(F, H), down=w(H, F), router=w(E, H), e_up=w(E, 2 * F, H), e_down=w(E, H, F))
        self.p_up, self.p_down = fmpq.fp8_pack_weights(self.up, self.w["up"]), fmpq.fp8_pack_weights(self.down, self.w["down"])
        self.p_router = fmpq.w16_pack_weights(self.router, self.w["router"])
        self.p_e_up, self.p_e_down = (fmpq.w16_pack_weights(self.e_up, self.w["e_up"]),
                                      fmpq.w16_pack_weights(self.e_down, self.w["e_down"]))
        v = lambda n, c: (torch.randn(n, generator=g) * 0.2 + c).bfloat16().cuda()          # noqa: E731
        self.n1, self.n2, self.n3, self.gate = v(H, 1), v(H, 1), v(H, 1), v(H, 0.7)
        self.b1, self.b2 = v(F, 0), v(H, 0).float()

    def __call__(self, r):
        import torch
        f, M = self.f, r.shape[0]
        n = f.block_norm(r, weight=self.n1, layer=self.up)
        h = f.fp8_gemm(self.up, n.A_packed, n.a_scales, *self.p_up, M, dtype=r.dtype, bias=self.b1, activation="gelu_tanh")
        y = f.fp8_quantize_gemm(self.down, h, *self.p_down, bias=self.b2)
        n = f.block_norm(y, r, post_norm=True, post_weight=self.n2, gate=self.gate, weight=self.n3)
        logits = f.w16_gemm(self.router, n.Y, self.p_router, dtype=torch.float32)
        ids, w = f.moe_route(logits, self.k)
        plan = f.moe_plan(ids, self.E)
        hidden = f.w16_experts_gemm(self.e_up, plan, n.Y, self.p_e_up, activation="silu")
        D = f.w16_experts_gemm(self.e_down, plan, hidden, self.p_e_down, weights=w, dtype=torch.float32)
        out = f.block_norm(f.moe_combine(D, plan), n.R, pre_norm=False)
        return out.R, ids, w

    def exact(self, r, ids, w):
        import torch
        d = lambda t: t.cpu().double()                                                       # noqa: E731
        rms = lambda v, g: v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6) * d(g)       # noqa: E731
        r, W = d(r), {k: d(v) for k, v in self.w.items()}
        x = rms(r, self.n1) @ W["up"].t() + d(self.b1)
        x = x * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (x + 0.044715 * x ** 3))
        r = r + d(self.gate) * rms(x @ W["down"].t() + d(self.b2), self.n2)
        n = rms(r, self.n3)
        out = torch.zeros_like(r)
        for e in range(self.E):
            t, j = (ids.cpu() == e).nonzero(as_tuple=True)
            a = n[t] @ W["e_up"][e].t()
            F = a.shape[1] // 2
            out.index_add_(0, t, (a[:, :F] * torch.sigmoid(a[:, :F]) * a[:, F:]) @ W["e_down"][e].t() * d(w)[t, j, None])
        return r + out


@pytest.mark.gpu
@pytest.mark.parametrize("M,H,F,E,k", [(1, 512, 1024, 8, 2), (37, 500, 388, 5, 3), (300, 256, 512, 4, 2), (700, 768, 640, 16, 4)])
def test_block(fmpq_mod, M, H, F, E, k):  # noqa: F811
    import torch
    block = Block(fmpq_mod, H, F, E, k)
    g = torch.Generator().manual_seed(M)
    new = lambda: (torch.randn(M, H, generator=g) * 2).bfloat16().cuda()     # noqa: E731
    r = new()
    out, ids, w = block(r)
    ref = block.exact(r, ids, w)
    assert float((out.cpu().double() - ref).norm()) <= (0.5 * 2 ** 0.5 * 2.0 ** -4 / 3 ** 0.5 + 4 * 2.0 ** -9) * float(ref.norm())
    # captured, and replayed on other inputs
    held = r.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = block(held)
    for _ in range(3):
        held.copy_(new())
        graph.replay()
        want = block(held.clone())
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    # two streams at once
    inputs = [new() for _ in range(6)]
    want = [block(x)[0] for x in inputs]
    sides = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for side in sides:
        side.wait_stream(torch.cuda.current_stream())
    for i, x in enumerate(inputs):
        with torch.cuda.stream(sides[i % 2]):
            got.append(block(x)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for layer in (block.router, block.e_up, block.e_down):
        assert fmpq_mod.w16_device_status(layer) == 0
    assert fmpq_mod.fp8_device_status(block.up) == 0 and fmpq_mod.fp8_device_status(block.down) == 0
