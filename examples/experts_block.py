"""A feed-forward block of routed experts with 4-bit weights, end to end.

    router logits = x @ wr^T                        (fp32 linear)
    weights, experts = route_experts(logits)        (softmax, best k of E)
    layout = experts_layout(experts)                (rows in expert order)
    h = relu(experts_linear_mxfp4(x, w1, layout))   (each row to its experts)
    y = experts_linear_mxfp4(h, w2, layout)
    out = experts_combine(y, weights)               (weighted sum per token)

Run it on a GB300: ``python examples/experts_block.py [tokens]`` prints the time of
a pass, replayed from a CUDA graph, and how far it is from the same block
computed with the weights and activations that MXFP4 holds, in plain torch.
"""
import math
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

from addmm_implicit_im2col_gb300 import binding  # noqa: E402


class ExpertsBlock:
    """Weights of the block: the router's in fp32, the experts' in MXFP4."""

    def __init__(self, width, hidden, experts, k, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def normal(*shape):
            return torch.randn(*shape, generator=g, device=device) / math.sqrt(shape[-1])

        self.k, self.experts = k, experts
        self.router = normal(experts, width)
        self.up = binding.quantize_mxfp4(normal(experts, hidden, width))
        self.down = binding.quantize_mxfp4(normal(experts, width, hidden))

    def __call__(self, x):
        """x [tokens, width] float32 -> [tokens, width]."""
        # few columns and long rows: the tensor cores, whatever the number of tokens
        logits = binding.linear(x, self.router, mode="force_tc3")
        weights, experts = binding.route_experts(logits, self.k)
        layout = binding.experts_layout(experts, self.experts)
        h = binding.experts_linear_mxfp4(x, self.up, layout, relu=True)
        y = binding.experts_linear_mxfp4(h, self.down, layout)
        return binding.experts_combine(y, weights)

    def plain(self, x):
        """The same with the dequantised operands, one expert at a time."""
        def held(v):  # what MXFP4 holds of v
            return binding.dequantize_mxfp4(binding.quantize_mxfp4(v))

        scores = torch.softmax(x @ self.router.t(), -1)
        weights, experts = scores.topk(self.k, -1)
        weights = weights / weights.sum(-1, keepdim=True)
        up, down = binding.dequantize_mxfp4(self.up), binding.dequantize_mxfp4(self.down)
        out = torch.zeros_like(x)
        for e in range(self.experts):
            token, place = (experts == e).nonzero(as_tuple=True)
            if len(token):
                h = torch.relu(held(x[token]) @ up[e].t())
                out.index_add_(0, token, weights[token, place, None] * (held(h) @ down[e].t()))
        return out


def main():
    tokens = int(sys.argv[1]) if len(sys.argv) > 1 else 512
    block = ExpertsBlock(width=1024, hidden=2048, experts=32, k=4)
    x = torch.randn(tokens, 1024, device="cuda")
    want = block.plain(x)
    out = block(x)  # sets the kernels up before the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block(x)
    graph.replay()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(20):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    off = ((out - want).norm() / want.norm()).item()
    print(f"{tokens} tokens, 32 experts, 4 per token: {begin.elapsed_time(end) / 20 * 1e3:.1f} us a pass, "
          f"relative difference from the plain block {off:.1e}")
    # a value of h at the edge of a rounding step may land on its other side (a
    # quarter of the value); such values are rare
    return 0 if off < 1e-2 and binding.check_device_error() == binding.IMC_OK else 1


if __name__ == "__main__":
    sys.exit(main())
