"""The 8-bit block operators where offsets, buffers and magnitudes reach their limits."""

import numpy as np
import pytest
import torch

import fp8_refs as ref
from test_gpu_fp8 import F8, TYPES, bytes_of, f32, gen, moe, offsets_of, wide_rows  # noqa: F401

pytestmark = pytest.mark.gpu


def i32(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


def codes_of(codes, scales, offsets):
    """64-bit values of the columns that the segments take."""
    n, _ = ref.columns(offsets, offsets[-1])
    return n, ref.values(bytes_of(codes)[:, :n[-1]], f32(scales)[:n[-1] // 128])


@pytest.mark.parametrize("accumulate", [False, True])
def test_weight_gradient_of_more_rows_than_its_codes(moe, accumulate):
    """Offsets that need a block more than the codes have are refused as a whole, and recorded."""
    N, K, E = 70, 300, 3
    fits, longer = [0, 128, 200, 328], [0, 129, 201, 329]         # 3 and 5 blocks
    g = gen(61)
    both = dict(offsets=i32(fits), by_row=False, by_column=True)
    _, dy = moe.quantize_fp8(torch.randn(328, N, generator=g).cuda(), **both)
    _, x = moe.quantize_fp8(torch.randn(328, K, generator=g).cuda(), **both)
    cut = lambda m: moe.Fp8Matrix(m.codes[:, :384], m.scales[:3])
    dy, x = cut(dy), cut(x)
    lin = moe.MoeFp8Linear(N, K, E)
    for bad in (longer, [0, 0, 0, 385], [0, 128, 128, 385]):
        dw = torch.full((E, N, K), 7.0).cuda()
        lin.grad_weight(dy, x, offsets=i32(bad), dw=dw, accumulate=accumulate)
        assert (dw == 7).all(), bad
        assert lin.check()[0] == moe.MOE_ERR_INVALID_ARG and lin.check()[0] == moe.MOE_OK
    dw = torch.zeros(E, N, K).cuda()
    lin.grad_weight(dy, x, offsets=i32(fits), dw=dw, accumulate=accumulate)
    (n, a), (_, b) = codes_of(*dy, fits), codes_of(*x, fits)
    for e in range(E):
        cols = slice(n[e], n[e + 1])
        ref.check_product(f32(dw)[e], a[:, cols], b[:, cols], "dw %d" % e)
    assert lin.check() == (moe.MOE_OK, 0)


@pytest.mark.parametrize("accumulate", [False, True])
def test_weight_gradient_of_no_columns(moe, accumulate):
    """Codes without columns: 0 where no expert has rows, refused where one has."""
    N, K, E = 33, 1100, 3
    none = lambda n: (torch.zeros(n, 0, dtype=torch.uint8).cuda().view(F8),
                      torch.zeros(0, n).cuda())
    lin = moe.MoeFp8Linear(N, K, E)
    for offsets, ok in (([0, 0, 0, 0], True), ([9, 9, 9, 9], True), ([0, 0, 1, 1], False),
                        ([0, 4, 2, 4], False), ([-1, -1, -1, -1], False)):
        dw = torch.full((E, N, K), 7.0).cuda()
        lin.grad_weight(none(N), none(K), offsets=i32(offsets), dw=dw, accumulate=accumulate)
        assert (dw == (0.0 if ok and not accumulate else 7.0)).all(), offsets
        assert lin.check()[0] == (moe.MOE_OK if ok else moe.MOE_ERR_INVALID_ARG)
    dense = moe.MoeFp8Linear(N, K)
    dw = torch.full((1, N, K), 7.0).cuda()
    dense.grad_weight(none(N), none(K), dw=dw, accumulate=accumulate)
    assert (dw == (7.0 if accumulate else 0.0)).all() and dense.check() == (moe.MOE_OK, 0)


@pytest.mark.parametrize("C", [128, 100, 130, 384])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_swiglu_gradient_at_large_gates(moe, C, dtype):
    """Gates of either sign up to 2^30, where the sigmoid is 0 or 1 and dsilu with it.  (One
    row has one gate, so that the blocks at the gate have magnitudes of their own.)"""
    gates = [s * 2.0 ** e * m for e in range(0, 31) for m in (1.0, 1.25) for s in (1.0, -1.0)]
    M = len(gates)
    a = torch.ones(M, 2 * C)
    a[:, :C] = torch.tensor(gates)[:, None]
    a[:, C:] = torch.randn(M, C, generator=gen(62))
    dh = torch.randn(M, C, generator=gen(63))
    a, dh = a.to(TYPES[dtype]), dh.to(TYPES[dtype])
    q, _ = moe.swiglu_grad_fp8(dh.cuda(), a.cuda())
    want, _ = ref.swiglu_grad(f32(dh), f32(a))
    # fp32: a dozen roundings, and the sigmoid's exponent |g| 2^-24 off where it is not 0 or 1
    g = np.array(gates)[:, None]
    mag = np.abs(want) + np.where(np.abs(g) < 110, np.concatenate(
        [np.abs(f32(dh) * f32(a)[:, C:]) * ref.ref.sigmoid(g) * (1 + np.abs(g)) ** 2,
         np.abs(want[:, C:]) * (1 + np.abs(g))], 1), 0.0)
    # (sigmoids below 2^-126 count as 0)
    mag = mag + 2.0 ** -126 / ref.FP32 * np.abs(g) ** 2 * (1 + np.abs(np.concatenate(
        [f32(dh) * f32(a)[:, C:], f32(dh)], 1)))
    ref.check_codes(bytes_of(q.codes), f32(q.scales), want, mag, "rows")


def test_no_rows(moe):
    """Every quantiser of no rows, either way, and what the products make of them."""
    C, N, E = 64, 48, 3
    none = torch.zeros(0, 2 * C).cuda()
    for offsets in (None, i32([0, 0, 0, 0])):
        for both in (dict(), dict(by_column=True), dict(by_row=False, by_column=True)):
            for q, t in (moe.quantize_fp8(none[:, :C], offsets=offsets, **both),
                         moe.quantize_fp8(torch.ones(5, C).cuda(), rows=i32([]), offsets=offsets,
                                          **both),
                         moe.swiglu_fp8(none, offsets=offsets, **both),
                         moe.swiglu_grad_fp8(none[:, :C], none, offsets=offsets, **both)):
                if both.get("by_row", True):
                    assert q.codes.shape[0] == 0
                if both:
                    assert t.codes.shape[1] == moe.fp8_columns(0, E if offsets is not None else 1,
                                                               offsets is not None)
    lin = moe.MoeFp8Linear(N, C)
    q, t = moe.quantize_fp8(none[:, :C], by_column=True)
    w, wt = moe.quantize_fp8_weights(torch.randn(N, C).cuda(), transposed=True)
    assert lin.forward(q, w).shape == (0, N)
    dy, dyt = moe.quantize_fp8(torch.zeros(0, N).cuda(), by_column=True)
    assert lin.grad_input(dy, wt).shape == (0, C)
    assert (lin.grad_weight(dyt, t) == 0).all()
    assert lin.check() == (moe.MOE_OK, 0)


@pytest.mark.parametrize("M", [0, 1, 128, 200])
@pytest.mark.parametrize("source", ["rows", "swiglu", "swiglu_grad"])
@pytest.mark.parametrize("C", [128, 90])
def test_columns_beyond_the_rows_without_offsets(moe, M, source, C):
    """A buffer kept for more rows than there are: its last columns are 0, and the weight
    gradient over all of them is that of the rows."""
    R, g = 512, gen(64)
    width = 2 * C if source == "swiglu_grad" else C
    a, dh = torch.randn(M, 2 * C, generator=g).cuda(), torch.randn(M, C, generator=g).cuda()

    def run(**kw):
        if source == "rows":
            return moe.quantize_fp8(dh, by_column=True, **kw)
        if source == "swiglu":
            return moe.swiglu_fp8(a, by_column=True, **kw)
        return moe.swiglu_grad_fp8(dh, a, by_column=True, **kw)

    kept = moe.Fp8Matrix(torch.full((width, R), 0x7F, dtype=torch.uint8).cuda().view(F8),
                         torch.full((R // 128, width), float("nan")).cuda())
    q, t = run(out_t=kept)
    alone, own = run()
    n = own.codes.shape[1]
    assert np.array_equal(bytes_of(q.codes), bytes_of(alone.codes))
    assert np.array_equal(bytes_of(t.codes)[:, :n], bytes_of(own.codes))
    assert torch.equal(t.scales[:n // 128], own.scales)
    assert (bytes_of(t.codes)[:, n:] == 0).all() and torch.isfinite(t.scales).all()
    lin = moe.MoeFp8Linear(width, width)
    assert torch.equal(lin.grad_weight(t, t), lin.grad_weight(own, own))


@pytest.mark.parametrize("source", ["rows", "swiglu_grad"])
@pytest.mark.parametrize("dtype,C", [("bf16", 256), ("bf16", 70), ("fp32", 130)])
@pytest.mark.parametrize("blocks", [0, 1, 3])
def test_columns_that_do_not_fit(moe, source, dtype, C, blocks):
    """Codes by columns as far as there is room, within a larger buffer of which nothing else
    is written; codes by rows whole all the same."""
    counts = [5, 0, 130, 1, 0, 64]                                 # five blocks
    M, g, offsets = sum(counts), gen(65), offsets_of(counts).cuda()
    width = 2 * C if source == "swiglu_grad" else C
    a = torch.randn(M, 2 * C, generator=g).to(TYPES[dtype]).cuda()
    dh = torch.randn(M, C, generator=g).to(TYPES[dtype]).cuda()

    def run(**kw):
        if source == "rows":
            return moe.quantize_fp8(dh, offsets=offsets, **kw)
        return moe.swiglu_grad_fp8(dh, a, offsets=offsets, **kw)

    whole, columns = run(by_column=True)
    room = torch.full((width + 3, 1024), 0x55, dtype=torch.uint8).cuda()
    room_s = torch.full((blocks + 3, width + 5), -1.0).cuda()
    n = 128 * blocks
    for by_row in (True, False) if blocks else (True,):
        room.fill_(0x55)
        room_s.fill_(-1.0)
        out_t = (room.view(F8)[1:width + 1, 128:128 + n], room_s[1:blocks + 1, 2:width + 2])
        q, t = run(by_row=by_row, by_column=True, out_t=out_t)
        if by_row:
            assert np.array_equal(bytes_of(q.codes), bytes_of(whole.codes))
            assert torch.equal(q.scales, whole.scales)
        want, want_s = np.full(room.shape, 0x55, np.uint8), np.full(room_s.shape, -1.0, np.float32)
        want[1:width + 1, 128:128 + n] = bytes_of(columns.codes)[:, :n]
        want_s[1:blocks + 1, 2:width + 2] = f32(columns.scales)[:blocks]
        assert np.array_equal(bytes_of(room), want) and np.array_equal(f32(room_s), want_s)


BAD = [[0, 20, 10, 30], [-1, 10, 20, 30], [0, 10, 20, 33], [5, 2 ** 31 - 1, 7, 9], [2, 1, 0, 0]]


@pytest.mark.parametrize("bad", BAD)
def test_bad_offsets_of_few_rows(moe, bad):
    """Nothing is written, and it is recorded; good offsets of the same call work after that."""
    M, N, K = 32, 40, 300
    g = gen(66)
    q, _ = moe.quantize_fp8(torch.randn(M, K, generator=g).cuda())
    w = moe.quantize_fp8_weights(torch.randn(3, N, K, generator=g).cuda())
    lin = moe.MoeFp8Linear(N, K, 3, dtype=torch.float32)
    y = torch.full((M, N), 7.0).cuda()
    lin.forward(q, w, offsets=i32(bad), out=y)
    assert (y == 7).all()
    assert lin.check()[0] == moe.MOE_ERR_INVALID_ARG and lin.check()[0] == moe.MOE_OK
    lin.forward(q, w, offsets=i32([0, 20, 20, 30]), out=y)
    x, t = ref.values(bytes_of(q.codes), f32(q.scales)), ref.tile_values(bytes_of(w.codes),
                                                                         f32(w.scales))
    ref.check_product(f32(y)[:20], x[:20], t[0], "first")
    ref.check_product(f32(y)[20:30], x[20:30], t[2], "last")
    assert (y[30:] == 7).all() and lin.check() == (moe.MOE_OK, 0)


@pytest.mark.parametrize("M,E", [(1, 1), (1, 256), (9, 9), (31, 256), (32, 2), (32, 200)])
@pytest.mark.parametrize("N,K", [(16, 4000), (1, 1), (17, 1025), (300, 130)])
def test_few_rows_anywhere(moe, M, E, N, K):
    """Rows of any experts, one of them with most, on a CTA for each that may have some."""
    g = np.random.default_rng(M * E + N)
    counts = np.bincount(np.append(g.integers(0, E, M // 2), [E // 3] * (M - M // 2)), minlength=E)
    offsets = offsets_of(counts.tolist())
    q, _ = moe.quantize_fp8(torch.randn(M, K, generator=gen(67)).cuda())
    w = moe.quantize_fp8_weights(torch.randn(E, N, K, generator=gen(68)).cuda())
    lin = moe.MoeFp8Linear(N, K, E, dtype=torch.float32)
    got, at = f32(lin.forward(q, w, offsets=offsets.cuda())), offsets.tolist()
    x, t = ref.values(bytes_of(q.codes), f32(q.scales)), ref.tile_values(bytes_of(w.codes),
                                                                         f32(w.scales))
    for e in range(E):
        rows = slice(at[e], at[e + 1])
        ref.check_product(got[rows], x[rows], t[e], "expert %d" % e)
    assert lin.check() == (moe.MOE_OK, 0)


def layer(moe, M, N, K, E, seed):
    """A step of one layer of experts as a closure over its offsets, outputs kept."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, dy = (torch.randn(M, w, generator=g, device="cuda") for w in (K, N))
    w, wt = moe.quantize_fp8_weights(torch.randn(E, N, K, generator=g, device="cuda"),
                                     transposed=True)
    lin = moe.MoeFp8Linear(N, K, E, dtype=torch.float32)
    out = [torch.zeros(M, N, device="cuda"), torch.zeros(M, K, device="cuda"),
           torch.zeros(E, N, K, device="cuda")]

    def step(offsets):
        for t in out:
            t.zero_()
        xq, xc = moe.quantize_fp8(x, offsets=offsets, by_column=True)
        yq, yc = moe.quantize_fp8(dy, offsets=offsets, by_column=True)
        lin.forward(xq, w, offsets=offsets, out=out[0])
        lin.grad_input(yq, wt, offsets=offsets, out=out[1])
        lin.grad_weight(yc, xc, offsets=offsets, dw=out[2], accumulate=True)
        return out

    return lin, step


@pytest.mark.parametrize("M,N,K", [(700, 384, 520), (30, 40, 300)])
def test_replays_follow_the_offsets(moe, M, N, K):
    """One captured step, replayed on other offsets than it was captured with, bad ones among
    them: the same bits as without capture."""
    E = 4
    lin, step = layer(moe, M, N, K, E, 81)
    offsets = i32([0, M // 2, M // 2, M - 5, M])
    step(offsets)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(offsets)
    for at in ([0, 0, 0, 0, M], [3, 10, M // 3, M // 3 + 1, M - 1], [0, 0, 0, 0, 0],
               [0, 9, 8, M, M], [0, 1, 2, 3, M + 1], [0, M // 4, M // 2, M - 7, M]):
        offsets.copy_(i32(at))
        graph.replay()
        got = [t.clone() for t in out]
        code = lin.check()[0]
        want = step(offsets)
        assert lin.check()[0] == code, at
        assert code == (moe.MOE_ERR_INVALID_ARG if at[1] > at[2] or at[-1] > M else moe.MOE_OK)
        # (beyond M nothing was quantised, and the weight gradient, which has the codes' columns
        # to go by and not M, added what the codes held)
        known = 3 if at[-1] <= M else 2
        for a, b in zip(got[:known], want):
            assert torch.equal(a, b), at


def test_steps_on_two_streams_at_once(moe):
    """Two layers' steps, of few rows and of many, at the same time on streams of their own."""
    sizes = ((3000, 1030, 700, 8, 82), (24, 48, 900, 8, 83))
    steps, offsets, want = [], [], []
    for M, N, K, E, seed in sizes:
        lin, step = layer(moe, M, N, K, E, seed)
        off = i32(np.linspace(0, M, E + 1).astype(int).tolist())
        steps.append((lin, step))
        offsets.append(off)
        want.append([t.clone() for t in step(off)])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sizes]
    got = [[], []]
    for _ in range(20):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got[i].append([t.clone() for t in steps[i][1](offsets[i])])
    torch.cuda.synchronize()
    for i in range(2):
        for out in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(out, want[i]))
        assert steps[i][0].check() == (moe.MOE_OK, 0)
