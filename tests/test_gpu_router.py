"""The router (forward and gradient) against a 64-bit implementation."""

import numpy as np
import pytest
import torch

import operator_refs as ref

pytestmark = pytest.mark.gpu

INF = float("inf")
SCORINGS = ["softmax_topk", "softmax", "sigmoid"]
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def moe():
    from routed_mixture_experts_gb300 import build

    build.build()
    import routed_mixture_experts_gb300 as m

    return m


def npy(t):
    return None if t is None else (t.float() if t.dtype == torch.bfloat16 else t).cpu().numpy()


def make_router(moe, T, E, k, scoring, scale=1.0, dtype="fp32"):
    return moe.MoeRouter(max(T, 1), E, k, scale=scale, dtype=TYPES[dtype], scoring={
        "softmax_topk": moe.MOE_ROUTER_SOFTMAX_TOPK, "softmax": moe.MOE_ROUTER_SOFTMAX,
        "sigmoid": moe.MOE_ROUTER_SIGMOID}[scoring])


def check_forward(r, logits, k, scoring, scale=1.0, bias=None, mask=None):
    got = r.forward(logits, bias=bias, token_mask=mask)
    want = ref.router_forward(npy(logits), k, scoring, scale, npy(bias), npy(mask))
    assert np.array_equal(npy(got.ids), want["ids"])
    assert np.array_equal(npy(got.counts), want["counts"])
    for name in ("scores", "prob_sum", "row_stat", "losses"):
        ref.check(npy(getattr(got, name)), want[name], name)
    return got


def check_backward(r, logits, f, k, scoring, scale=1.0, seed=0):
    T = logits.shape[0]
    g = torch.Generator().manual_seed(seed)
    ds = torch.randn(T, k, generator=g).cuda()
    dl = torch.tensor([0.3 * T, 0.0 if scoring == "sigmoid" else 0.01 * T], device="cuda")
    for a, b in ((ds, dl), (None, dl), (ds, None)):
        got = r.backward(logits, f.ids, f.counts, f.row_stat, d_scores=a, d_losses=b)
        want, mag = ref.router_backward(npy(logits), npy(f.ids), npy(f.counts),
                                        npy(f.row_stat).astype(np.float64), k, scoring, scale,
                                        npy(a), npy(b))
        ref.check(npy(got), want, "d_logits", mag, bf16=got.dtype == torch.bfloat16)
    return got


SIZES = [(1, 128, 8), (1, 1, 1), (5, 3, 3), (64, 128, 8), (65, 128, 8), (300, 60, 6),
         (1000, 33, 4), (257, 256, 8), (40, 256, 256), (70, 100, 40), (3000, 64, 2), (8, 31, 31)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("scoring", SCORINGS)
@pytest.mark.parametrize("T,E,k", SIZES)
def test_sizes(moe, T, E, k, scoring, dtype):
    g = torch.Generator().manual_seed(T * 1000 + E)
    logits = (torch.randn(T, E, generator=g) * 2).to(TYPES[dtype]).cuda()
    r = make_router(moe, T, E, k, scoring, 1.5, dtype)
    f = check_forward(r, logits, k, scoring, 1.5)
    check_backward(r, logits, f, k, scoring, 1.5)


@pytest.mark.parametrize("scoring", SCORINGS)
def test_several_rows_to_a_warp(moe, scoring):
    """More rows than warps on the GPU, live and masked ones in turn."""
    T, E, k = 15001, 40, 3
    g = torch.Generator().manual_seed(11)
    logits = (torch.randn(T, E, generator=g) * 2).cuda()
    mask = (torch.rand(T, generator=g) < 0.7).to(torch.uint8).cuda()
    r = make_router(moe, T, E, k, scoring)
    f = check_forward(r, logits, k, scoring, mask=mask)
    check_backward(r, logits, f, k, scoring)


@pytest.mark.parametrize("scoring", SCORINGS)
@pytest.mark.parametrize("dtype", list(TYPES))
def test_bias_mask_strides_and_switched_off_experts(moe, scoring, dtype):
    T, E, k = 517, 90, 7
    g = torch.Generator().manual_seed(4)
    wide = torch.full((T, E + 5), float("nan"))
    wide[:, :E] = torch.randn(T, E, generator=g) * 2
    wide[:, [3, 50, 89]] = -INF
    bias = (torch.randn(E, generator=g)).cuda()
    mask = (torch.rand(T, generator=g) < 0.8).to(torch.uint8)
    mask[5], mask[6], mask[7] = 1, 0, 1
    wide[mask == 0] = float("nan")                       # what padding holds is not read
    wide[5, :E] = -INF                                   # nothing left in these rows
    wide[6, :E] = -INF
    wide[7, : E - 4] = -INF                              # fewer left than k
    logits = wide.to(TYPES[dtype]).cuda()[:, :E]
    r = make_router(moe, T, E, k, scoring, 1.0, dtype)
    f = check_forward(r, logits, k, scoring, 1.0, bias, mask.cuda())
    got = check_backward(r, logits, f, k, scoring)
    dead = npy(f.row_stat) == -np.inf
    assert dead[5] and dead[6] and not dead[7]
    assert (npy(got)[dead] == 0).all() and np.isfinite(npy(got)).all()
    for row in npy(f.ids):
        assert len(set(row.tolist())) == k and 0 <= row.min() and row.max() < E


def test_ties_go_to_the_lowest_index(moe):
    logits = torch.tensor([[0.0, -0.0, 0.0, 1.0], [2.0, 2.0, 2.0, 2.0], [-0.0, 0.0, -1.0, -0.0],
                           [-1.0, -1.0, 3.0, 3.0]]).cuda()
    r = make_router(moe, 4, 4, 3, "softmax_topk")
    f = check_forward(r, logits, 3, "softmax_topk")
    assert f.ids.tolist() == [[3, 0, 1], [0, 1, 2], [0, 1, 3], [2, 3, 0]]


@pytest.mark.parametrize("scoring", SCORINGS)
def test_extreme_logits(moe, scoring):
    """The type's lowest value as a mask, very large and very small logits."""
    low = torch.finfo(torch.float32).min
    rows = torch.randn(8, 40, generator=torch.Generator().manual_seed(2))
    rows[0, :30] = low
    rows[1] *= 1e4
    rows[2] = -88.0 + rows[2]
    rows[3] = 1e-30 * rows[3]
    rows[4, 7] = 80.0
    rows[5, 1:] = low
    logits = rows.cuda()
    r = make_router(moe, 8, 40, 6, scoring)
    f = check_forward(r, logits, 6, scoring)
    assert all(torch.isfinite(t).all() for t in (f.scores, f.prob_sum, f.losses))
    d = r.backward(logits, f.ids, f.counts, f.row_stat, d_scores=torch.randn(8, 6).cuda())
    assert torch.isfinite(d).all()


def test_nan_and_inf_logits(moe):
    """A NaN ranks below every number and makes its row's probabilities NaN; the ids
    stay distinct and valid, other rows keep their scores."""
    g = torch.Generator().manual_seed(9)
    logits = torch.randn(6, 50, generator=g).cuda()
    r = make_router(moe, 6, 50, 5, "softmax")
    clean = r.forward(logits)
    bad = logits.clone()
    bad[1, 10] = float("nan")
    bad[2] = float("nan")
    bad[4, 3] = INF
    f = r.forward(bad)
    want = ref.choose(bad.cpu().numpy(), 5)
    assert np.array_equal(npy(f.ids), want)
    assert f.ids[4, 0] == 3
    keep = [0, 3, 5]
    assert torch.equal(f.scores[keep], clean.scores[keep])
    assert f.scores[[1, 2]].isnan().all() and f.scores[4].isnan().any()
    assert f.prob_sum.isnan().all()


def test_repeats_bit_for_bit(moe):
    logits = torch.randn(5000, 128, generator=torch.Generator().manual_seed(1)).cuda()
    r = make_router(moe, 5000, 128, 8, "softmax")
    a, b = r.forward(logits), r.forward(logits)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_scratch_contents_do_not_matter(moe):
    logits = torch.randn(700, 70, generator=torch.Generator().manual_seed(1)).cuda()
    r = make_router(moe, 700, 70, 5, "softmax_topk")
    a = r.forward(logits)
    r.workspace.fill_(255)
    b = r.forward(logits)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_no_tokens(moe):
    r = make_router(moe, 0, 16, 2, "softmax")
    f = r.forward(torch.empty(0, 16, device="cuda"))
    assert f.ids.shape == (0, 2) and f.scores.shape == (0, 2)
    for t in (f.counts, f.prob_sum, f.losses):
        assert torch.equal(t, torch.zeros_like(t))
    d = r.backward(torch.empty(0, 16, device="cuda"), f.ids, f.counts, f.row_stat)
    assert d.shape == (0, 16)


@pytest.mark.parametrize("scoring", SCORINGS)
def test_gradient_against_differences(moe, scoring):
    T, E, k = 24, 20, 4
    g = torch.Generator().manual_seed(7)
    logits = torch.randn(T, E, generator=g).cuda()
    ds = torch.randn(T, k, generator=g)
    dl = torch.tensor([2.0, 0.0 if scoring == "sigmoid" else 0.5])
    r = make_router(moe, T, E, k, scoring, 1.25)
    f = r.forward(logits)
    got = npy(r.backward(logits, f.ids, f.counts, f.row_stat, d_scores=ds.cuda(),
                         d_losses=dl.cuda())).astype(np.float64)
    base = npy(logits).astype(np.float64)

    def loss(l):
        o = ref.router_forward(l, k, scoring, 1.25, ids=npy(f.ids))
        return np.sum(o["scores"] * ds.numpy()) + np.dot(o["losses"], dl.numpy())

    rng = np.random.default_rng(3)
    h = 1e-5
    for _ in range(4):
        v = rng.standard_normal(base.shape)
        slope = (loss(base + h * v) - loss(base - h * v)) / (2 * h)
        # differences: h^2 truncation, 2^-53/h rounding; the kernel: fp32
        assert abs(slope - np.sum(got * v)) <= 1e-6 * np.linalg.norm(got) * np.linalg.norm(v) + 1e-8


def test_in_place_gradient_and_reused_outputs(moe):
    logits = torch.randn(300, 128, generator=torch.Generator().manual_seed(1)).cuda()
    r = make_router(moe, 300, 128, 8, "softmax")
    f = r.forward(logits)
    again = r.forward(logits, out=r.outputs(300))
    for x, y in zip(f, again):
        assert torch.equal(x, y)
    ds = torch.randn(300, 8).cuda()
    want = r.backward(logits, f.ids, f.counts, f.row_stat, d_scores=ds)
    mine = logits.clone()
    r.backward(mine, f.ids, f.counts, f.row_stat, d_scores=ds, d_logits=mine)
    assert torch.equal(mine, want)


def test_rows_further_apart_than_32_bits_reach(moe):
    apart = 2 ** 30 + 8
    pool = torch.empty(2 * apart + 256, dtype=torch.bfloat16, device="cuda")
    logits = torch.randn(3, 90, generator=torch.Generator().manual_seed(1)).to(
        torch.bfloat16).cuda()
    wide, out = (pool.as_strided((3, 90), (apart, 1), at) for at in (0, 128))
    wide.copy_(logits)
    r = make_router(moe, 3, 90, 5, "softmax", dtype="bf16")
    f, g = r.forward(logits), r.forward(wide)
    for x, y in zip(f, g):
        assert torch.equal(x, y)
    ds = torch.ones(3, 5).cuda() * torch.arange(5).cuda()
    want = r.backward(logits, f.ids, f.counts, f.row_stat, d_scores=ds)
    r.backward(wide, f.ids, f.counts, f.row_stat, d_scores=ds, d_logits=out)
    assert torch.equal(out, want)


def test_ids_and_scores_feed_the_experts(moe):
    """What the router makes is what the dispatch takes (valid, distinct ids)."""
    T, d, I, E, k = 200, 128, 64, 16, 4
    g = torch.Generator().manual_seed(5)
    bf = lambda *s: (torch.randn(*s, generator=g) * 0.1).to(torch.bfloat16).cuda()
    r = make_router(moe, T, E, k, "softmax_topk")
    mask = (torch.arange(T) < 170).to(torch.uint8).cuda()
    f = r.forward(torch.randn(T, E, generator=g).cuda(), token_mask=mask)
    plan = moe.MoePlan(T, d, I, E, k, flags=0)
    y = plan.forward(bf(T, d), f.ids, f.scores, bf(E, 2 * I, d), bf(E, d, I))
    assert plan.check()[0] == moe.MOE_OK
    counts = torch.bincount(f.ids[:170].flatten().long(), minlength=E)
    assert torch.equal(counts, f.counts[:E].long()) and f.counts[E] == 170
    assert (y[170:] == 0).all() and not (y[:170] == 0).all()


def test_outputs_belong_to_the_given_stream(moe):
    """Memory that the current stream has yet to write is not handed to another one."""
    logits = torch.randn(500, 60, generator=torch.Generator().manual_seed(3)).cuda()
    r = make_router(moe, 500, 60, 4, "softmax_topk")
    want = r.forward(logits)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    busy = [torch.empty_like(t) for t in want for _ in range(2)]
    torch.cuda._sleep(100_000_000)                      # some 50 ms
    for t in busy:
        t.fill_(77)
    del t, busy
    got = r.forward(logits, stream=s)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_refusals(moe):
    for bad in (dict(E=257), dict(E=0), dict(k=0), dict(k=17), dict(scoring=9),
                dict(dtype=torch.float16), dict(scale=float("nan"))):
        a = dict(E=16, k=2, scoring=0, scale=1.0, dtype=torch.float32)
        with pytest.raises(moe.MoeError):
            moe.MoeRouter(8, **{**a, **bad})
    r = make_router(moe, 8, 16, 2, "softmax")
    l = torch.randn(8, 16).cuda()
    for call in (lambda: r.forward(l.to(torch.bfloat16)), lambda: r.forward(l[:, :15]),
                 lambda: r.forward(torch.randn(9, 16).cuda()), lambda: r.forward(l.cpu()),
                 lambda: r.forward(l.t().contiguous().t()),
                 lambda: r.forward(l, bias=torch.zeros(15).cuda()),
                 lambda: r.forward(l, token_mask=torch.ones(8).cuda())):
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.code == moe.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("scoring", SCORINGS)
def test_gradient_of_rows_far_from_zero(moe, scoring):
    """The gradient where row_stat is large, so that its rounding to fp32 is not small
    beside 1.  A logit d below the logarithm of the row's sum has a weight that errs by
    2^-24 d for each of: d itself, its product with log2(e), and half of that for the
    constant; 4 d 2^-24 holds them all, on top of the other roundings.  A weight below
    2^-126, fp32's smallest normal number, may be lost whole, times factors below 2^10."""
    low = torch.finfo(torch.float32).min
    T, E, k = 10, 40, 6
    rows = torch.randn(T, E, generator=torch.Generator().manual_seed(2))
    rows[0, :30] = low
    rows[1] *= 1e4
    rows[2] -= 88.0
    rows[3] *= 1e-30
    rows[4, 7] = 80.0
    rows[5, 1:] = low
    rows[6] += 1e4
    rows[7] -= 600.0
    rows[8] += 300.0
    logits = rows.cuda()
    r = make_router(moe, T, E, k, scoring)
    f = r.forward(logits)
    ds = torch.randn(T, k, generator=torch.Generator().manual_seed(3)).cuda()
    dl = torch.tensor([0.3 * T, 0.0 if scoring == "sigmoid" else 0.01 * T], device="cuda")
    l = npy(logits).astype(np.float64)
    exact = ref.router_forward(l, k, scoring, ids=npy(f.ids))["row_stat"]
    below = np.abs(l - exact[:, None])
    for a, b in ((ds, dl), (None, dl), (ds, None)):
        got = r.backward(logits, f.ids, f.counts, f.row_stat, d_scores=a, d_losses=b)
        want, mag = ref.router_backward(l, npy(f.ids), npy(f.counts),
                                        npy(f.row_stat).astype(np.float64), k, scoring, 1.0,
                                        npy(a), npy(b))
        ref.check(npy(got), want, "d_logits",
                  mag * (1.0 + below / 16.0) + 2.0 ** -116 / ref.FP32)


def test_as_many_rows_as_an_int_counts(moe):
    T = 2 ** 31 - 1
    logits = torch.zeros(T, 1, dtype=torch.bfloat16, device="cuda")
    r = make_router(moe, T, 1, 1, "softmax_topk", dtype="bf16")
    f = r.forward(logits)
    assert f.counts.tolist() == [T, T]
    for part in (slice(0, 1 << 20), slice(T - (1 << 20), T)):
        assert (f.scores[part] == 1).all() and (f.ids[part] == 0).all()
        assert (f.row_stat[part] == 0).all()
    del f
    logits[-3:] = 5.0
    n = moe.MoeBlockNorm(T, 1, eps=0.0)
    u = n.forward(logits, w_pre=torch.full((1,), 2.0, device="cuda"))[1]
    assert (u[-3:] == 2).all()
    del logits, u, r
    torch.cuda.empty_cache()
