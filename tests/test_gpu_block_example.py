"""The example block: its gradients against automatic differentiation in 64 bits, and
its decoding against its own prompt path."""

import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


@pytest.fixture(scope="module")
def ex():
    from routed_mixture_experts_gb300 import build

    build.build()
    import moe_block

    return moe_block


def rms_norm(v, w):
    return v / (v.square().mean(1, keepdim=True) + 1e-6).sqrt() * w


def reference(block, r0, y0, ids, d_out, balance, z):
    """The block in 64 bits with the given choice, differentiated."""
    leaf = lambda t: t.detach().double().cpu().requires_grad_(True)
    p = {n: leaf(t) for n, t in dict(r0=r0, y0=y0, w_router=block.w_router, w13=block.w13,
                                     w2=block.w2).items()}
    for name, group in (("before", block.before), ("after", block.after)):
        for n, t in group.items():
            p[name + "." + n] = leaf(t)
    r1 = p["r0"] + p["before.gate"] * rms_norm(p["y0"], p["before.w_post"])
    u = rms_norm(r1, p["before.w_pre"])
    logits = u @ p["w_router"].t()
    ids = ids.cpu().long()
    T, E, k, I = r0.shape[0], block.E, block.k, block.I
    scores = torch.softmax(logits.gather(1, ids), 1)
    a = torch.einsum("td,tknd->tkn", u, p["w13"][ids])
    h = torch.nn.functional.silu(a[..., :I]) * a[..., I:]
    y1 = (torch.einsum("tki,tkdi->tkd", h, p["w2"][ids]) * scores[..., None]).sum(1)
    r2 = r1 + p["after.gate"] * rms_norm(y1, p["after.w_post"])
    out = rms_norm(r2, p["after.w_pre"])
    counts = torch.bincount(ids.reshape(-1), minlength=E).double()
    bal = E / (k * T * T) * (counts * torch.softmax(logits, 1).sum(0)).sum()
    lse = torch.logsumexp(logits, 1)
    total = (out * d_out.double().cpu()).sum() + balance * bal + z * lse.square().mean()
    grads = torch.autograd.grad(total, list(p.values()))
    return out, bal, lse.square().mean(), dict(zip(p, grads))


def far(got, want):
    return ((got.double().cpu() - want).norm() / want.norm()).item()


def test_training_step_against_autograd(ex):
    T, d, I, E, k = 96, 256, 256, 8, 2
    block = ex.MoeBlock(T, d, I, E, k, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    r = lambda: torch.randn(T, d, generator=g, device="cuda").to(torch.bfloat16)
    r0, y0, d_out = r(), r(), r()
    v, grads = block.train_step(r0, y0, d_out, balance=50.0, z=5.0)
    assert block.plan.check()[0] == 0
    out, bal, zl, want = reference(block, r0, y0, v["route"].ids, d_out, 50.0, 5.0)
    # values pass through about ten bf16 roundings (2^-8 each at most, independent), the
    # gradients through twice as many: 10 * 2^-8 and 20 * 2^-8 of the norm would be all
    # of them at their worst in one direction; a quarter of it bounds independent ones
    assert far(v["out"], out) < 2.5 * 2 ** -8
    assert abs(float(v["route"].losses[0]) / bal.item() - 1) < 2.5 * 2 ** -8
    assert abs(float(v["route"].losses[1]) / zl.item() - 1) < 2.5 * 2 ** -8
    for n in ("r0", "y0", "w_router", "w13", "w2"):
        assert far(grads[n], want[n]) < 5 * 2 ** -8, n
    for side in ("before", "after"):
        for n in ("w_post", "gate", "w_pre"):
            got = getattr(grads[side], "dgate" if n == "gate" else "d" + n)
            assert far(got, want[side + "." + n]) < 5 * 2 ** -8, (side, n)


def test_decoding_follows_the_prompt_path(ex):
    T, d, I, E, k = 40, 512, 256, 8, 2
    block = ex.MoeBlock(T, d, I, E, k, seed=5)
    g = torch.Generator(device="cuda").manual_seed(6)
    r = lambda: torch.randn(T, d, generator=g, device="cuda").to(torch.bfloat16)
    r0, y0 = r(), r()
    whole = block.forward(r0, y0, lambda u, route: block.plan.forward(
        u, route.ids, route.scores, block.w13, block.w2))
    block.prepare_decode(T)
    for n in (1, 3, T):
        r2, out = block.decode_step(r0[:n].contiguous(), y0[:n].contiguous())
        # E2M1 weights with a scale per 16: about a tenth of each weight's size
        assert far(out, whole["out"][:n].double().cpu()) < 0.15
        assert far(r2, whole["r2"][:n].double().cpu()) < 0.15
    assert block.decode_plan.check()[0] == 0


def test_it_runs_as_a_program(ex, capsys):
    ex.main()
    assert "decoded 8 token(s)" in capsys.readouterr().out
