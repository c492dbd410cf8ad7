"""The feed-forward half of a mixture-of-experts block, served by gmmfr's operators.

A decoding step (up to 64 tokens) is one call of MoeLayer: gate, routed experts, shared expert and residual.
A prompt runs the same weights through the operators for many tokens: MoeGate, the routing step, the grouped
SwiGLU FFN, and the shared expert as two dense products, the second of which adds the residual.

    python examples/moe_block.py [--tokens 512] [--steps 16]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from moe_grouped_gemm_mxfp8_gb300 import binding as B  # noqa: E402


class MoeBlock:
    """y = residual + shared(x) + sum over the chosen experts of weight * expert(x)."""

    def __init__(self, gate_weight, w13, w2, shared_w13, shared_w2, **rule):
        self.E, self.H = gate_weight.shape
        self.I = w2.shape[1]
        self.layer = B.MoeLayer(gate_weight, w13, w2, shared_w13=shared_w13, shared_w2=shared_w2, **rule)
        self.gate = B.MoeGate(gate_weight, **rule)
        self.shared_up = B.Linear(shared_w13.t().contiguous(), activation="swiglu")
        self.shared_down = B.Linear(shared_w2.t().contiguous())

    def decode(self, x, residual):
        return self.layer(x, residual=residual)

    def prefill(self, x, residual):
        T, topk = x.shape[0], self.gate.topk
        ids, weights = self.gate(x)
        # the routing step moves bytes: a BF16 row is 2H of them, and there are no scales to go with it
        scales = torch.empty((T, (2 * self.H + 63) // 64, 2), dtype=torch.uint8, device=x.device)
        routed, _ = B.route(ids, weights, x.view(torch.uint8), scales, self.E, group_list_type=0)
        ends = torch.zeros(self.E + 1, dtype=torch.int32, device=x.device)
        ends[1:] = routed["group_list"]
        y, _ = B.ffn(routed["x1"].view(torch.bfloat16), self.layer.prepared, ends, self.H, self.I, self.E)
        place = torch.empty(T * topk, dtype=torch.int64, device=x.device)
        place[routed["perm"].long()] = torch.arange(T * topk, device=x.device)
        out = (y[place].view(T, topk, self.H).float() * weights[:, :, None]).sum(1)
        return out + self.shared_down(self.shared_up(x), residual=residual).float()


def random_block(E=64, H=2048, I=512, shared_I=512, topk=8, device="cuda", seed=0):
    g = torch.Generator(device=device).manual_seed(seed)

    def randn(*shape, scale=1.0):
        return (torch.randn(*shape, device=device, generator=g) * scale).to(torch.bfloat16)

    weights = dict(gate_weight=randn(E, H, scale=H ** -0.5), w13=randn(E, H, 2 * I, scale=H ** -0.5),
                   w2=randn(E, I, H, scale=I ** -0.5), shared_w13=randn(H, 2 * shared_I, scale=H ** -0.5),
                   shared_w2=randn(shared_I, H, scale=shared_I ** -0.5))
    bias = torch.randn(E, device=device, generator=g) * 0.1
    return weights, MoeBlock(**weights, topk=topk, scoring="sigmoid", select_bias=bias, n_group=8, topk_group=4, scale=2.5)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=512, help="tokens of the prompt")
    ap.add_argument("--steps", type=int, default=16, help="decoding steps")
    a = ap.parse_args()
    _, block = random_block()
    x = torch.randn(a.tokens, block.H, device="cuda").to(torch.bfloat16)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    block.prefill(x, x)
    start.record()
    h = block.prefill(x, x)
    end.record()
    torch.cuda.synchronize()
    print(f"prompt of {a.tokens} tokens: {start.elapsed_time(end) * 1e3:.0f} us")
    few = x[:48]
    far = (block.decode(few, few).float() - h[:48]).abs().max() / h[:48].abs().max()
    print(f"the same 48 tokens as a decoding step: {far:.1e} of the largest value away")
    for T in (1, 16, 64):
        h = x[:T].clone()
        step, out = torch.cuda.CUDAGraph(), torch.empty_like(h)
        block.layer(h, residual=h, out=out)
        with torch.cuda.graph(step):
            block.layer(h, residual=h, out=out)
        start.record()
        for _ in range(a.steps):
            step.replay()
        end.record()
        torch.cuda.synchronize()
        print(f"decoding step of {T:2d} tokens: {start.elapsed_time(end) * 1e3 / a.steps:.1f} us")


if __name__ == "__main__":
    main()
