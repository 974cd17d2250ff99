"""A mixture-of-experts block from end to end: training step and token-by-token decoding.

    python examples/moe_block.py

The block stands between two others of a residual stream r (bf16):

    r1, u   = norms around the previous block's output y0 (MoeBlockNorm)
    logits  = u . Wr^T                                     (the caller's own product)
    ids, scores, counts, losses = router(logits)           (MoeRouter)
    y1      = routed experts of u                          (MoePlan)
    r2, out = norms around y1                              (MoeBlockNorm)

train_step() runs it forward and backward with the balance and z losses of the
router; decode_step() runs it for a few new tokens on NVFP4 expert weights.
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import routed_mixture_experts_gb300 as moe  # noqa: E402


class MoeBlock:
    """The parameters of one block, and its handles for up to `tokens` tokens."""

    def __init__(self, tokens, d, I, E, k, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        n = lambda *s, scale=1.0: torch.randn(*s, generator=g, device=device) * scale
        bf16 = torch.bfloat16
        self.d, self.I, self.E, self.k = d, I, E, k
        self.w_router = n(E, d, scale=d ** -0.5)
        self.w13 = n(E, 2 * I, d, scale=d ** -0.5).to(bf16)
        self.w2 = n(E, d, I, scale=I ** -0.5).to(bf16)
        # before the experts: the previous block's output joins the stream; after them:
        # theirs does, scaled channel by channel
        ones = lambda: 1.0 + n(d, scale=0.05)
        self.before = dict(w_post=ones(), gate=0.5 + n(d, scale=0.1), w_pre=ones())
        self.after = dict(w_post=ones(), gate=0.5 + n(d, scale=0.1), w_pre=ones())
        norm = lambda: moe.MoeBlockNorm(tokens, d, gate=moe.MOE_GATE_CHANNEL)
        self.norm_before, self.norm_after = norm(), norm()
        self.router = moe.MoeRouter(tokens, E, k)
        self.plan = moe.MoePlan(tokens, d, I, E, k)
        self.prepared = self.decode_plan = None

    def prepare_decode(self, tokens):
        """NVFP4 expert weights (again after each change of w13, w2) and a plan for up
        to `tokens` tokens at a time."""
        self.prepared = moe.prepare_weights_nvfp4(self.w13, self.w2)
        self.decode_plan = moe.MoePlan(tokens, self.d, self.I, self.E, self.k,
                                       precision=moe.MOE_PREC_NVFP4, flags=0)

    def forward(self, r0, y0, experts, token_mask=None):
        """experts(u, route) -> y1.  -> every value that the backward reads."""
        r1, u = self.norm_before.forward(r0, y=y0, **self.before)
        logits = u.float() @ self.w_router.t()
        route = self.router.forward(logits, token_mask=token_mask)
        y1 = experts(u, route)
        r2, out = self.norm_after.forward(r1, y=y1, **self.after)
        return dict(y0=y0, r1=r1, u=u, logits=logits, route=route, y1=y1, r2=r2, out=out)

    def decode_step(self, r0, y0):
        """The block for a few new tokens, one row each -> (r2, out)."""
        v = self.forward(r0, y0, lambda u, route: self.decode_plan.decode_nvfp4(
            u, route.ids, route.scores, self.prepared))
        return v["r2"], v["out"]

    def train_step(self, r0, y0, d_out, balance=0.01, z=0.001, token_mask=None):
        """Forward and backward.  d_out: the gradient at `out`.  -> (values, gradients)"""
        v = self.forward(r0, y0, lambda u, route: self.plan.forward(
            u, route.ids, route.scores, self.w13, self.w2, save=True), token_mask)
        route = v["route"]
        dw13 = torch.zeros(self.w13.shape, device=r0.device)
        dw2 = torch.zeros(self.w2.shape, device=r0.device)
        after = self.norm_after.backward(v["r2"], None, d_out, y=v["y1"], **self.after)
        du, d_scores = self.plan.backward(after.dy, self.w13, self.w2, dw13, dw2)
        d_logits = self.router.backward(
            v["logits"], route.ids, route.counts, route.row_stat, d_scores=d_scores,
            d_losses=torch.tensor([balance, z], device=r0.device))
        dw_router = d_logits.t() @ v["u"].float()
        du = (du.float() + d_logits @ self.w_router).to(torch.bfloat16)
        before = self.norm_before.backward(v["r1"], after.d_residual, du, y=y0, **self.before)
        return v, dict(r0=before.d_residual, y0=before.dy, w_router=dw_router, w13=dw13, w2=dw2,
                       before=before, after=after)


def main():
    T, d, I, E, k = 2048, 1024, 512, 32, 4
    block = MoeBlock(T, d, I, E, k)
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    for step in range(3):
        v, grads = block.train_step(r(T, d), r(T, d), r(T, d) * 0.01)
        counts = v["route"].counts
        print("step %d: balance loss %.4f, z loss %.3f, busiest expert %d of %d tokens, "
              "|dWr| %.3e" % (step, v["route"].losses[0], v["route"].losses[1],
                              int(counts[:E].max()), int(counts[E]), grads["w_router"].norm()))
    assert block.plan.check()[0] == moe.MOE_OK
    block.prepare_decode(8)
    for tokens in (1, 5, 8):
        r2, out = block.decode_step(r(tokens, d), r(tokens, d))
        print("decoded %d token(s): |out| %.3f" % (tokens, out.float().norm()))
    assert block.decode_plan.check()[0] == moe.MOE_OK


if __name__ == "__main__":
    main()
