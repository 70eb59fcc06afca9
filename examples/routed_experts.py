"""A routed-experts feed-forward layer on the package's operators.

  out[t] = x[t] + sum_j w[t,j] * (gelu(x[t] @ W1[e] + b1[e]) @ W2[e] + b2[e]),   e = experts[t,j]

The router is a linear layer without a bias; its k best experts of each token (softmax or
sigmoid scores, an optional balance bias and expert groups) are sorted into runs
of rows by moe_plan, the experts' products run over those runs, and moe_combine
brings the rows back.  forward() reads token rows through the plan, so that the
sorted copy of x is only made where the weight gradient needs it.

    python examples/routed_experts.py             # a few training steps, then single-token decoding
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import activation_epilogue_amd as fl  # noqa: E402


def every_row(x):
    """The offsets of one expert that has every row of x: [0, rows]."""
    T = x.shape[0]
    return (torch.arange(0, T + 1, T, dtype=torch.int32, device=x.device) if T
            else torch.zeros(2, dtype=torch.int32, device=x.device))


class RoutedExperts:
    """Weights of E experts (hidden -> ffn -> hidden) and of their router, and
    how tokens are routed (the options of moe_route)."""

    def __init__(self, hidden, ffn, E, k, dtype=torch.bfloat16, seed=0, score="softmax", renorm=True, scale=1.0, bias=None,
                 **groups):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)
        self.Wr = normal(hidden, E, std=hidden ** -0.5)
        self.W1, self.b1 = normal(E, hidden, ffn, std=hidden ** -0.5), normal(E, ffn, std=0.02)
        self.W2, self.b2 = normal(E, ffn, hidden, std=ffn ** -0.5), normal(E, hidden, std=0.02)
        self.E, self.k = E, k
        self.weighting = {"score": score, "renorm": renorm, "scale": scale}
        self.choice = {"bias": bias, **groups}

    def parameters(self):
        return {"Wr": self.Wr, "W1": self.W1, "b1": self.b1, "W2": self.W2, "b2": self.b2}

    def forward(self, x, keep=False):
        """out (T,hidden) for x (T,hidden); with keep=True also what backward needs."""
        # the router's product is one expert that has every token: few tokens
        # by a narrow weight are what the experts' low tiles are for
        logits = fl.grouped_linear(x, self.Wr[None], every_row(x), act="none")
        weights, experts = fl.moe_route(logits, self.k, **self.weighting, **self.choice)
        plan = fl.moe_plan(experts, self.E)
        h = fl.grouped_linear(x, self.W1, plan.offsets, self.b1, act="gelu_tanh", index=plan.token_of_row, pre=keep)
        h, pre = h if keep else (h, None)
        y = fl.grouped_linear(h, self.W2, plan.offsets, self.b2, act="none")
        out = fl.moe_combine(y, plan.row_of_slot, weights, R=x)
        return (out, (x, logits, weights, experts, plan, pre, h, y)) if keep else out

    def backward(self, dout, kept):
        """(dx, gradients of the parameters by name) from the gradient of out."""
        x, logits, weights, experts, plan, pre, h, y = kept
        o = plan.offsets
        dy, dweights = fl.moe_combine_bwd(dout, y, plan.row_of_slot, weights)
        dW2, db2 = fl.grouped_weight_grad(h, dy, o)
        dpre, _ = fl.grouped_linear_bwd(dy, self.W2, pre, o, act="gelu_tanh")
        dW1, db1 = fl.grouped_weight_grad(fl.moe_gather(x, plan.token_of_row), dpre, o)
        drows, _ = fl.grouped_linear_bwd(dpre, self.W1, None, o, act="none")
        dx = fl.moe_combine(drows, plan.row_of_slot, R=dout)
        dlogits = fl.moe_route_bwd(logits, experts, dweights, **self.weighting)
        dWr, _ = fl.grouped_weight_grad(x, dlogits, every_row(x), dbias=None)
        dx = fl.fused_linear(dlogits, self.Wr.t().contiguous(), R=dx, act="none")
        return dx, {"Wr": dWr[0], "W1": dW1, "b1": db1, "W2": dW2, "b2": db2}


def main():
    layer = RoutedExperts(hidden=1024, ffn=2048, E=16, k=2)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(4096, 1024, generator=g, device="cuda").bfloat16()
    target = torch.randn(4096, 1024, generator=g, device="cuda").bfloat16()
    for step in range(5):
        out, kept = layer.forward(x, keep=True)
        diff = out.float() - target.float()
        print(f"step {step}: loss {float(diff.square().mean()):.4f}", flush=True)
        _, grads = layer.backward((diff * (2.0 / diff.shape[0])).bfloat16(), kept)
        for name, p in layer.parameters().items():
            p -= (0.01 * grads[name].float()).to(p.dtype)
    token = x[:1].contiguous()
    for _ in range(3):  # one token at a time, each the next one's input
        token = layer.forward(token)
    print("decoded", float(token.float().norm()))


if __name__ == "__main__":
    main()
