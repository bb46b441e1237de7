"""One MoE layer, forward and backward, through the library: routing,
dispatch, the experts' FFN, a shared expert, combine, and the gradients back
to the tokens, the router logits and every weight.

    python examples/moe_layer.py [tokens]
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import combine_moe_gate_warp_gb300 as moe


class MoELayer:
    """E routed experts of inner size F (top-k) and one shared expert, hidden size H."""

    def __init__(self, T, H=2048, F=1024, E=32, k=8, P=8, device="cuda"):
        def weights(*shape):
            return (torch.randn(*shape, device=device) * shape[-1] ** -0.5).bfloat16()

        self.plan = moe.RoutePlan(moe.RouteShape(T=T, H=H, E=E, k=k, P=P, mode=moe.MOE_SOFTMAX_TOPK, Ks=1), device)
        self.router = torch.randn(E, H, device=device) * H ** -0.5
        self.experts = moe.ExpertFFN(moe.ExpertRows.of(self.plan), weights(E, 2 * F, H), weights(E, H, F))
        self.shared = moe.ExpertFFN(moe.ExpertRows(rows=T), weights(2 * F, H), weights(H, F))

    def forward(self, x):
        self.x, self.logits = x, x.float() @ self.router.T
        p = self.plan
        p.route(self.logits)
        p.dispatch(x)
        p.combine(self.experts.forward(p.packed), self.shared.forward(x)[None])
        return p.y

    def backward(self, dy):
        """(dx, d_router); the experts' gradients are in self.experts.grads and self.shared.grads."""
        p = self.plan
        p.combine_backward(dy, self.experts.y)
        p.dispatch_backward(self.experts.backward(p.d_expert_out, p.packed).dx)
        p.gate_backward(self.logits)
        dx = p.dx.float() + self.shared.backward(dy, self.x).dx.float() + p.d_logits @ self.router
        return dx.bfloat16(), p.d_logits.T @ self.x.float()


def main():
    T = int(sys.argv[1]) if len(sys.argv) > 1 else 8192
    torch.manual_seed(0)
    layer = MoELayer(T)
    x, dy = (torch.randn(T, 2048, device="cuda").bfloat16() for _ in range(2))
    for i in range(4):
        a, b, c = (torch.cuda.Event(enable_timing=True) for _ in range(3))
        a.record()
        y = layer.forward(x)
        b.record()
        dx, d_router = layer.backward(dy)
        c.record()
        torch.cuda.synchronize()
        if layer.plan.status() or layer.shared.rows.status():
            raise RuntimeError("a device-detected problem")
        print(f"pass {i}: forward {a.elapsed_time(b):.3f} ms, backward {b.elapsed_time(c):.3f} ms, "
              f"|y| {y.float().norm().item():.1f}, |dx| {dx.float().norm().item():.1f}, "
              f"|d_router| {d_router.norm().item():.1f}")


if __name__ == "__main__":
    main()
