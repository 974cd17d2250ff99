"""The router with groups against a 64-bit implementation."""

import numpy as np
import pytest
import torch

import fp8_refs
import operator_refs as ref

pytestmark = pytest.mark.gpu

INF = float("inf")
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def moe():
    from routed_mixture_experts_gb300 import build

    build.build()
    import routed_mixture_experts_gb300 as m

    return m


def npy(t):
    return None if t is None else (t.float() if t.dtype == torch.bfloat16 else t).cpu().numpy()


def make(moe, T, E, k, groups, top, scoring, pair, scale=1.0, dtype="fp32"):
    return moe.MoeGroupRouter(
        max(T, 1), E, k, groups, top, scale=scale, dtype=TYPES[dtype],
        group_score=moe.MOE_GROUP_TOP2 if pair else moe.MOE_GROUP_MAX,
        scoring={"softmax_topk": moe.MOE_ROUTER_SOFTMAX_TOPK, "softmax": moe.MOE_ROUTER_SOFTMAX,
                 "sigmoid": moe.MOE_ROUTER_SIGMOID}[scoring])


def check(r, logits, scoring, pair, scale=1.0, bias=None, mask=None):
    got = r.forward(logits, bias=bias, token_mask=mask)
    l, k = npy(logits), r.k
    ids = fp8_refs.group_choice(l, k, r.groups, r.top_groups, scoring, pair, npy(bias))
    if mask is not None:
        for t in np.nonzero(npy(mask) == 0)[0]:
            ids[t] = (t * k + np.arange(k)) % r.E
    assert np.array_equal(npy(got.ids), ids)
    want = ref.router_forward(l, k, scoring, scale, mask=npy(mask), ids=ids)
    assert np.array_equal(npy(got.counts), want["counts"])
    for name in ("scores", "prob_sum", "row_stat", "losses"):
        ref.check(npy(getattr(got, name)), want[name], name)
    return got


SIZES = [(1, 256, 8, 8, 4), (5, 8, 1, 8, 1), (33, 64, 6, 8, 3), (300, 160, 6, 20, 5),
         (1, 1, 1, 1, 1), (70, 96, 24, 3, 1), (40, 250, 16, 125, 8), (64, 256, 4, 256, 4),
         (9, 256, 256, 2, 2), (50, 60, 20, 4, 2), (200, 36, 5, 12, 12), (31, 200, 7, 5, 2)]


@pytest.mark.parametrize("T,E,k,groups,top", SIZES)
@pytest.mark.parametrize("scoring", ["softmax_topk", "softmax", "sigmoid"])
@pytest.mark.parametrize("pair", [False, True])
def test_forward(moe, T, E, k, groups, top, scoring, pair):
    g = torch.Generator().manual_seed(T + E)
    for dtype in ("fp32", "bf16"):
        logits = (torch.randn(T, E, generator=g) * 1.5).to(TYPES[dtype]).cuda()
        bias = (torch.randn(E, generator=g) * 0.1).cuda()
        r = make(moe, T, E, k, groups, top, scoring, pair, 1.75, dtype)
        check(r, logits, scoring, pair, 1.75)
        check(r, logits, scoring, pair, 1.75, bias)
        check(r, logits, scoring, pair, 1.75, torch.zeros_like(bias))


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("pair", [False, True])
def test_keys_closer_than_fp32_tells(moe, scoring, pair):
    """Biases that make the keys of neighbours, and the values of groups, agree to a few
    2^-26: the order is that of 64-bit keys."""
    T, E, k, groups, top = 64, 64, 6, 8, 4
    g = torch.Generator().manual_seed(3)
    logits = torch.randn(1, E, generator=g).repeat(T, 1)
    s = (torch.sigmoid(logits.double()) if scoring == "sigmoid"
         else torch.softmax(logits.double(), 1))[0]
    near = (0.75 - s).float()                                # keys of 0.75, off by a rounding
    bias = near + torch.randint(-2, 3, (E,), generator=g).float() * 2.0 ** -26
    # the rows differ in their last bits
    logits = logits + torch.randint(-3, 4, (T, E), generator=g).float() * 2.0 ** -23
    check(make(moe, T, E, k, groups, top, scoring, pair), logits.cuda(), scoring, pair,
          bias=bias.cuda())


@pytest.mark.parametrize("scoring", ["softmax_topk", "softmax", "sigmoid"])
@pytest.mark.parametrize("pair", [False, True])
def test_ties_infinities_nan(moe, scoring, pair):
    T, E, k, groups, top = 12, 48, 8, 6, 2
    g = torch.Generator().manual_seed(5)
    logits = torch.randn(T, E, generator=g)
    logits[0] = 0.25                                         # all equal
    logits[1] = -INF                                         # nothing to choose
    logits[2, 5:] = -INF                                     # fewer than k left
    logits[3, ::8] = 3.0                                     # groups tie
    logits[4, 8:40] = -INF                                   # whole groups switched off
    logits[5] = 60.0                                         # sigmoids of 1
    logits[6] = -120.0                                       # sigmoids below 2^-149
    logits[7, 9] = -0.0
    logits[7, 10] = 0.0
    logits[8, 17] = INF
    for bias in (None, torch.zeros(E), torch.randn(E, generator=g) * 0.2):
        dev = None if bias is None else bias.cuda()
        r = make(moe, T, E, k, groups, top, scoring, pair)
        if scoring == "sigmoid":
            check(r, logits.cuda(), scoring, pair, bias=dev)
        else:
            check(r, logits[:8].contiguous().cuda(), scoring, pair, bias=dev)
        nan = logits.clone()
        nan[9, 11] = float("nan")
        nan[10] = float("nan")
        got = r.forward(nan.cuda(), bias=dev)
        ids = npy(got.ids)
        assert ids.min() >= 0 and ids.max() < E
        assert all(len(set(row)) == k for row in ids)
        if scoring == "sigmoid" or (bias is None and not pair):
            want = fp8_refs.group_choice(npy(nan), k, groups, top, scoring, pair, npy(bias))
            assert np.array_equal(ids, want)


def test_mask_strides_empty(moe):
    T, E, k, groups, top = 77, 40, 4, 5, 3
    g = torch.Generator().manual_seed(6)
    wide = torch.randn(T, E + 9, generator=g).cuda()
    mask = (torch.rand(T, generator=g) < 0.7).to(torch.uint8).cuda()
    r = make(moe, T, E, k, groups, top, "sigmoid", True)
    check(r, wide[:, 3:3 + E], "sigmoid", True, bias=torch.zeros(E).cuda(), mask=mask)
    got = r.forward(wide[:0, :E])
    assert got.ids.shape == (0, k) and int(got.counts.sum()) == 0


@pytest.mark.parametrize("scoring", ["softmax_topk", "softmax", "sigmoid"])
def test_gradient_is_the_routers(moe, scoring):
    """Against differences of sum(d_scores * scores) + sum(d_losses * losses) in 64 bits, the
    choice held."""
    T, E, k, groups, top = 40, 24, 4, 6, 3
    g = torch.Generator().manual_seed(8)
    logits = torch.randn(T, E, generator=g)
    r = make(moe, T, E, k, groups, top, scoring, True, 2.5)
    f = r.forward(logits.cuda(), bias=(torch.randn(E, generator=g) * 0.1).cuda())
    ds = torch.randn(T, k, generator=g)
    dl = torch.tensor([2.0, 0.0 if scoring == "sigmoid" else 0.5])
    got = npy(r.backward(logits.cuda(), f.ids, f.counts, f.row_stat, d_scores=ds.cuda(),
                         d_losses=dl.cuda())).astype(np.float64)
    want, mag = ref.router_backward(npy(logits), npy(f.ids), npy(f.counts),
                                    npy(f.row_stat).astype(np.float64), k, scoring, 2.5, npy(ds),
                                    npy(dl))
    ref.check(got, want, "d_logits", mag)
    along = np.random.RandomState(1).randn(T, E)

    def total(h):
        w = ref.router_forward(npy(logits).astype(np.float64) + h * along, k, scoring, 2.5,
                               ids=npy(f.ids))
        return (w["scores"] * npy(ds)).sum() + (w["losses"] * npy(dl)).sum()

    h = 1e-5
    slope = (total(h) - total(-h)) / (2 * h)
    # differences: h^2 of the third derivative, and 2^-52 / h of the sums
    assert abs((got * along).sum() - slope) <= 1e-4 * (np.abs(got * along).sum() + 1)


def test_bias_update(moe):
    E = 70
    g = torch.Generator().manual_seed(9)
    counts = torch.randint(0, 50, (E + 1,), generator=g, dtype=torch.int32)
    counts[:3] = 2 ** 30
    counts[3] = 0
    bias = torch.randn(E, generator=g)
    r = make(moe, 8, E, 2, 7, 2, "sigmoid", True)
    got = r.update_bias(bias.clone().cuda(), counts.cuda(), 0.001).cpu()
    n = counts[:E].double()
    want = bias + torch.sign(n.mean() - n).float() * 0.001
    assert torch.equal(got, want)
    even = torch.full((E + 1,), 7, dtype=torch.int32)
    assert torch.equal(r.update_bias(bias.clone().cuda(), even.cuda(), 0.1).cpu(), bias)


def test_many_rows_repeat_and_replay(moe):
    """Two runs and a captured one give the same bits; experts are those of 64-bit keys."""
    T, E, k, groups, top = 3000, 256, 8, 8, 4
    g = torch.Generator().manual_seed(10)
    logits = torch.randn(T, E, generator=g).cuda()
    bias = (torch.randn(E, generator=g) * 0.05).cuda()
    r = make(moe, T, E, k, groups, top, "sigmoid", True)
    a = check(r, logits, "sigmoid", True, bias=bias)
    b = r.forward(logits, bias=bias)
    out = r.outputs(T)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r.forward(logits, bias=bias, out=out)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        r.forward(logits, bias=bias, out=out)
    for t in out:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for x, y, z in zip(a, b, out):
        assert torch.equal(x, y) and torch.equal(x, z)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("T,E,k,groups,top", [(40, 64, 6, 8, 3), (9, 8, 1, 8, 1), (30, 48, 4, 12, 2),
                                              (50, 256, 8, 8, 4)])
def test_biases_of_any_size(moe, T, E, k, groups, top, scoring, pair):
    """Experts switched off or forced by their bias, and keys whose sums pass fp32's range."""
    g = torch.Generator().manual_seed(T + E)
    logits = (torch.randn(T, E, generator=g) * 1.5).cuda()
    for off in (-1e9, -INF, 1e9, INF, 3e38, -3e38):
        for n in (1, 2, E // 2):
            bias = torch.randn(E, generator=g) * 0.1
            bias[torch.randperm(E, generator=g)[:n]] = off
            check(make(moe, T, E, k, groups, top, scoring, pair), logits, scoring, pair,
                  bias=bias.cuda())
    # two groups whose sums fp32 holds for infinite: the second is larger
    if pair and E > groups:
        size = E // groups
        bias = torch.zeros(E)
        bias[0], bias[1] = 2e38, 2e38
        bias[size], bias[size + 1] = 3e38, 1.5e38
        check(make(moe, T, E, 1, groups, 1, scoring, pair), logits, scoring, pair,
              bias=bias.cuda())
