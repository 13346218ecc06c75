"""A mixture-of-experts feed-forward step on E4M3 weights: router product, routing, experts.

    python examples/routed_experts.py [tokens]

Random weights stand in for a checkpoint. The router is an E4M3 layer itself (its logits are the
routing's input); the experts' weights are laid out once. The step is captured into a CUDA graph and
checked against the same arithmetic written with torch operations.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bit_quantized_gemm_fmpq_gb300 import build, fmpq  # noqa: E402

BLOCK = 128


class RoutedExperts:
    """experts x (gate, up [F, H]; down [H, F]), `k` of them a token, chosen by a router [experts, H]."""

    def __init__(self, H, F, experts, k, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weights(*shape):
            return (torch.randn(*shape, generator=g, device="cuda") / shape[-1] ** 0.5).to(dtype)

        self.k = k
        self.router = fmpq.Fp8Layer(H, experts)
        self.up = fmpq.Fp8Layer(H, 2 * F, experts=experts, gated=True)
        self.down = fmpq.Fp8Layer(F, H, experts=experts)
        self.bias = torch.randn(experts, generator=g, device="cuda") * 0.01     # load balance
        self.w_router = fmpq.fp8_pack_weights(self.router, weights(experts, H))
        self.w_up = fmpq.fp8_pack_weights(self.up, weights(experts, 2 * F, H))
        self.w_down = fmpq.fp8_pack_weights(self.down, weights(experts, H, F))

    def __call__(self, X):
        logits = fmpq.fp8_quantize_gemm(self.router, X, *self.w_router)
        ids, weights = fmpq.moe_route(logits, self.k, score="sigmoid", bias=self.bias)
        return fmpq.moe_experts(self.up, self.down, X, ids, weights, *self.w_up, *self.w_down), ids, weights

    def plain(self, X, ids, weights):
        """The experts' part in FP32 with torch operations, for the given routing."""
        def quantized(x):
            b = torch.nn.functional.pad(x.float(), (0, -x.shape[1] % BLOCK)).view(x.shape[0], -1, BLOCK)
            amax = b.abs().amax(2, keepdim=True)
            s = amax / torch.full_like(amax, 448.0)      # (by a number, torch multiplies by its reciprocal)
            q = (b / s.clamp_min(1e-30)).clamp(-448, 448).to(torch.float8_e4m3fn).float() * s
            return q.view(x.shape[0], -1)[:, :x.shape[1]]

        Y = torch.zeros(X.shape, device="cuda")
        xq, F = quantized(X), self.down.K
        for e in range(self.up.experts):
            t, j = (ids == e).nonzero(as_tuple=True)
            if t.numel():
                w = fmpq.fp8_unpack_weights(self.up, *self.w_up, expert=e)
                g, u = xq[t] @ w[:F].t(), xq[t] @ w[F:].t()
                h = quantized(g * torch.sigmoid(g) * u)
                Y.index_add_(0, t, (h @ fmpq.fp8_unpack_weights(self.down, *self.w_down, expert=e).t()) * weights[t, j, None])
        return Y


def main(tokens=256):
    build.build()
    layer = RoutedExperts(H=1024, F=512, experts=16, k=2)
    X = torch.randn(tokens, 1024, device="cuda").to(torch.bfloat16)
    layer(X)                                 # first use: library, workspaces
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Y, ids, weights = layer(X)
    graph.replay()
    torch.cuda.synchronize()
    ref = layer.plain(X, ids, weights)
    err = float((Y.float() - ref).norm() / ref.norm())
    load = torch.bincount(ids.flatten().long(), minlength=16)
    print(f"{tokens} tokens, 2 of 16 experts each, load {load.min().item()}-{load.max().item()}: "
          f"relative error {err:.2e} against FP32 on the same codes")
    return err


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 256)
