"""The routed experts of a few tokens on NVFP4 weights against a 64-bit
implementation on the same prepared weights.

Bound: y is one bf16 rounding (2^-8 of the element) of fp32 sums.  h is rounded to
11 significant bits before the second product: each of the I terms of a y element
errs by at most 2^-11 of itself, and the fp32 sums by 64 * 2^-24 of their terms'
magnitudes, so `mag`, the sum of the magnitudes of all the products that make a y
element, carries both: 2^-11 is never reached by all terms at once with one sign,
but bounds them.  For h itself, fp32 sums of d terms: 64 * 2^-24 of the terms'
magnitudes through silu(G) * U (slope at most 1.1).
"""

import ctypes

import numpy as np
import pytest
import torch

import moe_inputs as mi
from gpu_case import to_dev
from parity import f32
from test_gpu_nvfp4 import untile16

pytestmark = pytest.mark.gpu

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


@pytest.fixture(scope="module")
def moe():
    from routed_mixture_experts_gb300 import build

    build.build()
    import routed_mixture_experts_gb300 as m

    return m


def dequantised(codes, sf, scale, rows, K, E, gu_I):
    """[E, rows, K] in 64 bits."""
    c = codes.reshape(E * rows, K // 2)
    v = np.empty((E * rows, K))
    v[:, 0::2], v[:, 1::2] = E2M1[c & 15], E2M1[c >> 4]
    s = torch.from_numpy(untile16(sf, E * rows, K, gu_I)).view(torch.float8_e4m3fn).double().numpy()
    return (v * np.repeat(s, 16, 1)).reshape(E, rows, K) * scale.astype(np.float64)[:, None, None]


def reference(x, ids, scores, w13, w2, clamp=0.0):
    """-> (y, mag)"""
    T, d = x.shape
    E, I = w13.shape[0], w2.shape[2]
    y, mag = np.zeros((T, d)), np.zeros((T, d))
    for t in range(T):
        seen = set()
        for j, e in enumerate(ids[t]):
            if not 0 <= e < E or e in seen:
                continue
            seen.add(e)
            a = w13[e] @ x[t]
            big = np.abs(w13[e]) @ np.abs(x[t])
            G, U = a[:I], a[I:]
            if clamp > 0:
                G, U = np.clip(G, -clamp, clamp), np.clip(U, -clamp, clamp)
            h = G / (1 + np.exp(-G)) * U
            # terms of h: an error of G's and U's terms, times the other factor
            bigh = np.abs(h) + 64 * 2.0 ** -13 * 1.1 * (big[:I] * np.abs(U) + big[I:] * np.abs(G))
            y[t] += scores[t, j] * (w2[e] @ h)
            mag[t] += abs(scores[t, j]) * (np.abs(w2[e]) @ bigh)
    return y, mag


def make(T, d, I, E, k, seed=7, **over):
    return mi.make_inputs(None, seed=seed, need=("x", "ids", "scores", "w13", "w2"), T=T, d=d, I=I,
                          E=E, k=k, **over)


class Weights:
    def __init__(self, moe, dev, E, I, d):
        self.prep = moe.prepare_weights_nvfp4(dev["w13"], dev["w2"])
        torch.cuda.synchronize()
        n = [t.cpu().numpy() for t in self.prep]
        self.w13 = dequantised(n[0], n[1], n[2], 2 * I, d, E, I)
        self.w2 = dequantised(n[3], n[4], n[5], d, I, E, 0)


def check(y, x, ids, scores, w, clamp=0.0):
    want, mag = reference(f32(x).astype(np.float64), ids, scores.astype(np.float64), w.w13, w.w2,
                          clamp)
    got = y.float().cpu().numpy().astype(np.float64)
    assert np.sqrt(np.mean(want ** 2)) > 1e-4
    over = np.abs(got - want) - 2.0 ** -8 * np.abs(want) - 2.0 ** -11 * mag
    assert over.max() <= 0, over.max()
    # and in norm: independent roundings of 2^-8 at most, 2^-11 of the terms
    rel = np.linalg.norm(got - want) / np.linalg.norm(want)
    assert rel <= 2.0 ** -8, rel


SIZES = [dict(T=1, d=256, I=256, E=4, k=2), dict(T=1, d=512, I=768, E=300 // 2, k=8),
         dict(T=3, d=768, I=256, E=5, k=5), dict(T=7, d=256, I=512, E=16, k=3),
         dict(T=16, d=256, I=256, E=32, k=2), dict(T=9, d=256, I=256, E=1, k=1),
         dict(T=33, d=512, I=256, E=8, k=4), dict(T=64, d=256, I=256, E=64, k=8),
         dict(T=256, d=256, I=256, E=7, k=2), dict(T=40, d=256, I=256, E=256, k=20),
         dict(T=5, d=256, I=1280, E=6, k=2, clamp=0.5),
         # enough units for a unit a warp, in the first or the second product, with the
         # shortest rows and several passes of one expert's tokens
         dict(T=60, d=512, I=768, E=80, k=4), dict(T=100, d=2048, I=256, E=48, k=3),
         dict(T=150, d=256, I=1280, E=40, k=5)]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: ",".join("%s%s" % kv for kv in s.items()))
def test_sizes(moe, sizes):
    inp = make(**sizes)
    c, dev = inp["cfg"], to_dev(inp)
    w = Weights(moe, dev, c["E"], c["I"], c["d"])
    plan = moe.MoePlan(c["T"], c["d"], c["I"], c["E"], c["k"], precision=moe.MOE_PREC_NVFP4,
                       flags=0, clamp=c.get("clamp", 0.0))
    y = plan.decode_nvfp4(dev["x"], dev["ids"], dev["scores"], w.prep)
    assert plan.check()[0] == moe.MOE_OK
    check(y, inp["x"], inp["ids"], inp["scores"], w, c.get("clamp", 0.0))
    again = plan.decode_nvfp4(dev["x"], dev["ids"], dev["scores"], w.prep)
    assert torch.equal(y, again)


def test_fewer_tokens_than_the_plan_and_no_tokens(moe):
    inp = make(T=50, d=256, I=256, E=8, k=3)
    dev = to_dev(inp)
    w = Weights(moe, dev, 8, 256, 256)
    plan = moe.MoePlan(50, 256, 256, 8, 3, precision=moe.MOE_PREC_NVFP4, flags=0)
    whole = plan.decode_nvfp4(dev["x"], dev["ids"], dev["scores"], w.prep)
    for n in (0, 1, 8, 9, 49):
        y = plan.decode_nvfp4(dev["x"][:n], dev["ids"][:n], dev["scores"][:n], w.prep)
        assert torch.equal(y, whole[:n])           # a token's result does not hang on the others
    assert plan.check()[0] == moe.MOE_OK


def test_range_of_activations(moe):
    """Rows of very large, very small and mixed values, zeros and outliers."""
    inp = make(T=6, d=512, I=256, E=4, k=2)
    x = inp["x"].copy()
    f = torch.from_numpy(f32(x).copy())
    f[0] *= 1e4
    f[1] *= 1e-3
    f[2] = 0
    f[3, ::7] *= 300
    f[4, 1:] = 0
    bf = f.to(torch.bfloat16)
    inp["x"] = bf.view(torch.int16).numpy().view(np.uint16)
    dev = to_dev(inp)
    w = Weights(moe, dev, 4, 256, 512)
    plan = moe.MoePlan(6, 512, 256, 4, 2, precision=moe.MOE_PREC_NVFP4, flags=0)
    y = plan.decode_nvfp4(dev["x"], dev["ids"], dev["scores"], w.prep)
    got = y.float().cpu().numpy().astype(np.float64)
    want, mag = reference(f32(inp["x"]).astype(np.float64), inp["ids"],
                          inp["scores"].astype(np.float64), w.w13, w.w2)
    assert (got[2] == 0).all()
    for t in range(6):
        over = np.abs(got[t] - want[t]) - 2.0 ** -8 * np.abs(want[t]) - 2.0 ** -11 * mag[t]
        assert over.max() <= 2.0 ** -133, (t, over.max())


def test_a_bad_token_leaves_the_others_alone(moe):
    inp = make(T=9, d=256, I=256, E=4, k=2)
    dev = to_dev(inp)
    w = Weights(moe, dev, 4, 256, 256)
    plan = moe.MoePlan(9, 256, 256, 4, 2, precision=moe.MOE_PREC_NVFP4, flags=0)
    clean = plan.decode_nvfp4(dev["x"], dev["ids"], dev["scores"], w.prep)
    x = dev["x"].clone()
    x[3, 17] = float("nan")
    x[5, 200] = float("inf")
    y = plan.decode_nvfp4(x, dev["ids"], dev["scores"], w.prep)
    keep = [0, 1, 2, 4, 6, 7, 8]
    assert torch.equal(y[keep], clean[keep])
    assert y[3].isnan().all() and not y[5].isfinite().all()


def test_bad_ids_are_dropped_and_reported(moe):
    inp = make(T=12, d=256, I=256, E=6, k=3)
    ids = inp["ids"].copy()
    ids[4, 1] = 6
    ids[7, 2] = ids[7, 0]
    ids[9, 0] = -1
    inp["ids"] = ids
    dev = to_dev(inp)
    w = Weights(moe, dev, 6, 256, 256)
    plan = moe.MoePlan(12, 256, 256, 6, 3, precision=moe.MOE_PREC_NVFP4, flags=0)
    y = plan.decode_nvfp4(dev["x"], dev["ids"], dev["scores"], w.prep)
    assert plan.check() == (moe.MOE_ERR_BAD_IDS, 13)
    check(y, inp["x"], ids, inp["scores"], w)
    one = plan.decode_nvfp4(dev["x"][4:5], dev["ids"][4:5], dev["scores"][4:5], w.prep)
    assert plan.check() == (moe.MOE_ERR_BAD_IDS, 1)
    assert torch.equal(one[0], y[4])


def test_every_token_on_one_expert_and_empty_experts(moe):
    inp = make(T=100, d=256, I=256, E=64, k=1)
    inp["ids"] = np.full((100, 1), 37, np.int32)
    dev = to_dev(inp)
    w = Weights(moe, dev, 64, 256, 256)
    plan = moe.MoePlan(100, 256, 256, 64, 1, precision=moe.MOE_PREC_NVFP4, flags=0)
    y = plan.decode_nvfp4(dev["x"], dev["ids"], dev["scores"], w.prep)
    check(y, inp["x"], inp["ids"], inp["scores"], w)


def test_in_a_graph_and_on_another_stream(moe):
    inp = make(T=5, d=256, I=256, E=8, k=2)
    dev = to_dev(inp)
    w = Weights(moe, dev, 8, 256, 256)
    plan = moe.MoePlan(5, 256, 256, 8, 2, precision=moe.MOE_PREC_NVFP4, flags=0)
    want = plan.decode_nvfp4(dev["x"], dev["ids"], dev["scores"], w.prep)
    x, y = torch.zeros_like(dev["x"]), torch.empty_like(want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        for _ in range(3):
            plan.decode_nvfp4(x, dev["ids"], dev["scores"], w.prep, y=y)
    x.copy_(dev["x"])
    for _ in range(4):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_beside_the_prompt_path_on_one_plan(moe):
    """Alternating with moe_forward_nvfp4 changes neither's results."""
    inp = make(T=64, d=256, I=256, E=8, k=2)
    dev = to_dev(inp)
    w = Weights(moe, dev, 8, 256, 256)
    plan = moe.MoePlan(64, 256, 256, 8, 2, precision=moe.MOE_PREC_NVFP4, flags=0)
    plan.set_activation_scales(0.002, 0.002)
    args = dev["x"], dev["ids"], dev["scores"], w.prep
    a, b = plan.forward_nvfp4(*args), plan.decode_nvfp4(*args)
    c, e = plan.forward_nvfp4(*args), plan.decode_nvfp4(*args)
    assert torch.equal(a, c) and torch.equal(b, e)
    # the prompt path quantises its activations to 4 bits; the two agree to that
    rel = ((a.float() - b.float()).norm() / b.float().norm()).item()
    assert rel < 0.3, rel


def test_outputs_belong_to_the_given_stream(moe):
    """Memory that the current stream has yet to write is not handed to another one."""
    inp = make(T=5, d=256, I=256, E=8, k=2)
    dev = to_dev(inp)
    w = Weights(moe, dev, 8, 256, 256)
    plan = moe.MoePlan(5, 256, 256, 8, 2, precision=moe.MOE_PREC_NVFP4, flags=0)
    want = [plan.decode_nvfp4(dev["x"], dev["ids"], dev["scores"], w.prep)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    busy = [torch.empty_like(t) for t in want for _ in range(2)]
    torch.cuda._sleep(100_000_000)                      # some 50 ms
    for t in busy:
        t.fill_(77)
    del t, busy
    got = [plan.decode_nvfp4(dev["x"], dev["ids"], dev["scores"], w.prep, stream=s)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_refusals(moe):
    L = moe.lib()
    inp = make(T=4, d=256, I=256, E=4, k=2)
    dev = to_dev(inp)
    prep = moe.prepare_weights_nvfp4(dev["w13"], dev["w2"])
    plan = moe.MoePlan(4, 256, 256, 4, 2, precision=moe.MOE_PREC_NVFP4, flags=0)
    args = (dev["x"], dev["ids"], dev["scores"])
    for bad in ((torch.cat([args[0]] * 2), torch.cat([args[1]] * 2), torch.cat([args[2]] * 2)),
                (args[0].float(), args[1], args[2]), (args[0][:, :128], args[1], args[2]),
                (args[0], args[1].long(), args[2]), (args[0], args[1][:, :1], args[2]),
                (args[0], args[1], args[2].half())):
        with pytest.raises(moe.MoeError) as e:
            plan.decode_nvfp4(*bad, prep)
        assert e.value.code == moe.MOE_ERR_INVALID_ARG
    wide = moe.MoePlan(300, 256, 256, 4, 2, precision=moe.MOE_PREC_NVFP4, flags=0)
    big = torch.zeros(257, 256, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(moe.MoeError):
        wide.decode_nvfp4(big, torch.zeros(257, 2, dtype=torch.int32, device="cuda"),
                          torch.zeros(257, 2, device="cuda"), prep)
    # 65536 pairs: their list does not fit in shared memory
    many = moe.MoePlan(256, 256, 256, 256, 256, precision=moe.MOE_PREC_NVFP4, flags=0)
    with pytest.raises(moe.MoeError) as e:
        many.decode_nvfp4(big[:256], torch.arange(256, dtype=torch.int32, device="cuda").expand(
            256, 256).contiguous(), torch.zeros(256, 256, device="cuda"),
            moe.prepare_weights_nvfp4(
                torch.zeros(256, 512, 256, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(256, 256, 256, dtype=torch.bfloat16, device="cuda")))
    assert e.value.code == moe.MOE_ERR_UNSUPPORTED
    p16 = moe.MoePlan(4, 256, 256, 4, 2, flags=0)
    with pytest.raises(moe.MoeError) as e:
        p16.decode_nvfp4(*args, prep)
    assert e.value.code == moe.MOE_ERR_UNSUPPORTED
    vp = ctypes.c_void_p
    p = lambda t: vp(t.data_ptr())
    call = lambda x, y, n=4: L.moe_decode_nvfp4(plan.ptr, x, p(args[1]), p(args[2]), n,
                                                *[p(t) for t in prep], y, None)
    y = torch.empty_like(args[0])
    assert call(None, p(y)) == moe.MOE_ERR_INVALID_ARG
    assert call(p(args[0]), None) == moe.MOE_ERR_INVALID_ARG
    assert call(vp(args[0].data_ptr() + 2), p(y)) == moe.MOE_ERR_INVALID_ARG
    assert call(p(args[0]), p(y), -1) == moe.MOE_ERR_INVALID_ARG
    assert call(None, None, 0) == moe.MOE_OK


def test_weights_of_another_plan_are_refused(moe):
    inp = make(T=5, d=256, I=256, E=8, k=2)
    dev = to_dev(inp)
    w = Weights(moe, dev, 8, 256, 256)
    plan = moe.MoePlan(5, 256, 256, 16, 2, precision=moe.MOE_PREC_NVFP4, flags=0)
    with pytest.raises(moe.MoeError):
        plan.decode_nvfp4(dev["x"], dev["ids"], dev["scores"], w.prep)
    plan = moe.MoePlan(5, 256, 256, 8, 2, precision=moe.MOE_PREC_NVFP4, flags=0)
    for i in range(6):
        wrong = list(w.prep)
        wrong[i] = wrong[i].reshape(-1)[:-1]
        with pytest.raises(moe.MoeError):
            plan.decode_nvfp4(dev["x"], dev["ids"], dev["scores"], wrong)
    plan.decode_nvfp4(dev["x"], dev["ids"], dev["scores"], w.prep)


@pytest.mark.parametrize("clamp", [0.0, 0.5])
@pytest.mark.parametrize("T,E,I", [(1, 4, 256), (9, 4, 256), (40, 64, 256)],
                         ids=["one token", "split", "stream"])
def test_nan_stays_in_its_row_with_a_clamp(moe, T, E, I, clamp):
    """Clipping a NaN gives a NaN."""
    inp = make(T=T, d=256, I=I, E=E, k=2)
    dev = to_dev(inp)
    w = Weights(moe, dev, E, I, 256)
    plan = moe.MoePlan(T, 256, I, E, 2, precision=moe.MOE_PREC_NVFP4, flags=0, clamp=clamp)
    clean = plan.decode_nvfp4(dev["x"], dev["ids"], dev["scores"], w.prep)
    x = dev["x"].clone()
    at = T // 2
    x[at, 17] = float("nan")
    y = plan.decode_nvfp4(x, dev["ids"], dev["scores"], w.prep)
    assert y[at].isnan().all()
    keep = [t for t in range(T) if t != at]
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("T", [1, 2])
@pytest.mark.parametrize("d,I", [(46080, 256), (256, 46080)])
def test_rows_that_leave_room_for_one_cta_an_sm(moe, d, I, T):
    """A row of fp16 that fits in 200 KB, but not twice."""
    inp = make(T=T, d=d, I=I, E=1, k=1)
    dev = to_dev(inp)
    w = Weights(moe, dev, 1, I, d)
    plan = moe.MoePlan(T, d, I, 1, 1, precision=moe.MOE_PREC_NVFP4, flags=0)
    y = plan.decode_nvfp4(dev["x"], dev["ids"], dev["scores"], w.prep)
    assert plan.check()[0] == moe.MOE_OK
    check(y, inp["x"], inp["ids"], inp["scores"], w)


def test_a_workspace_without_the_decode_scratch(moe):
    """Its size before there was decoding: the plan takes it and runs prompts, and only
    decoding is refused."""
    T, d, I, E, k = 40, 256, 512, 8, 2
    inp = make(T=T, d=d, I=I, E=E, k=k)
    dev = to_dev(inp)
    w = Weights(moe, dev, E, I, d)
    plan = moe.MoePlan(T, d, I, E, k, precision=moe.MOE_PREC_NVFP4, flags=0)
    plan.set_activation_scales(0.002, 0.002)
    args = dev["x"], dev["ids"], dev["scores"], w.prep
    want = plan.forward_nvfp4(*args)
    L = moe.lib()
    up = lambda n: (n + 255) // 256 * 256
    scratch = up(4 * T * k * I) + up(4 * T * k * d) + up(T * k)
    small = plan.workspace.numel() - scratch
    p = ctypes.c_void_p(plan.workspace.data_ptr())
    assert L.moe_plan_set_workspace(plan.ptr, p, small - 1, 0) == moe.MOE_ERR_WORKSPACE
    assert L.moe_plan_set_workspace(plan.ptr, p, small, 0) == moe.MOE_OK
    plan.workspace[small:] = 7
    assert torch.equal(plan.forward_nvfp4(*args), want)
    assert plan.check()[0] == moe.MOE_OK
    assert (plan.workspace[small:] == 7).all()
    with pytest.raises(moe.MoeError) as e:
        plan.decode_nvfp4(*args)
    assert e.value.code == moe.MOE_ERR_WORKSPACE
    assert L.moe_plan_set_workspace(plan.ptr, p, plan.workspace.numel(), 0) == moe.MOE_OK
    check(plan.decode_nvfp4(*args), inp["x"], inp["ids"], inp["scores"], w)


# Rows wider than 2048: eight tokens' rows no longer fit beside the stream's ring (4096:
# four do, in several passes of one expert) or in half an SM's shared memory (7168: six
# do); and one token that leaves the two-launch path: more than eight experts, or eight
# rows of h that do not fit together.
WIDE = [dict(T=20, d=4096, I=1280, E=8, k=2), dict(T=19, d=256, I=4096, E=3, k=2),
        dict(T=11, d=7168, I=256, E=2, k=1), dict(T=13, d=256, I=7168, E=2, k=1),
        dict(T=9, d=2560, I=2560, E=2, k=2), dict(T=1, d=256, I=256, E=12, k=9),
        dict(T=1, d=512, I=256, E=40, k=33), dict(T=1, d=256, I=12800, E=8, k=8),
        dict(T=1, d=7168, I=2048, E=3, k=2)]


@pytest.mark.parametrize("sizes", WIDE, ids=lambda s: ",".join("%s%s" % kv for kv in s.items()))
def test_wide_rows_and_many_experts_of_one_token(moe, sizes):
    inp = make(**sizes)
    c, dev = inp["cfg"], to_dev(inp)
    w = Weights(moe, dev, c["E"], c["I"], c["d"])
    plan = moe.MoePlan(c["T"], c["d"], c["I"], c["E"], c["k"], precision=moe.MOE_PREC_NVFP4,
                       flags=0)
    y = plan.decode_nvfp4(dev["x"], dev["ids"], dev["scores"], w.prep)
    assert plan.check()[0] == moe.MOE_OK
    check(y, inp["x"], inp["ids"], inp["scores"], w)
    assert torch.equal(y, plan.decode_nvfp4(dev["x"], dev["ids"], dev["scores"], w.prep))


def test_a_token_alone_and_among_others(moe):
    """Different kernels add K in different orders: both are within the bound."""
    T, d, I, E, k = 50, 2048, 768, 16, 4
    inp = make(T=T, d=d, I=I, E=E, k=k)
    dev = to_dev(inp)
    w = Weights(moe, dev, E, I, d)
    plan = moe.MoePlan(T, d, I, E, k, precision=moe.MOE_PREC_NVFP4, flags=0)
    for n in (1, 3, T):
        y = plan.decode_nvfp4(dev["x"][:n], dev["ids"][:n], dev["scores"][:n], w.prep)
        check(y, inp["x"][:n], inp["ids"][:n], inp["scores"][:n], w)
