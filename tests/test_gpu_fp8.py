"""The 8-bit block quantisers and products against plain implementations."""

import numpy as np
import pytest
import torch

import fp8_refs as ref

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def moe():
    from routed_mixture_experts_gb300 import build

    build.build()
    import routed_mixture_experts_gb300 as m

    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


def f32(t):
    return t.detach().float().cpu().numpy()


def bytes_of(t):
    return t.cpu().contiguous().view(torch.uint8).numpy()


def offsets_of(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32)


def wide_rows(M, C, dtype, g, scale=1.0):
    """Rows apart, with blocks of very different magnitudes."""
    x = torch.randn(M, C, generator=g) * torch.exp2(
        torch.randint(-12, 12, (M, (C + 63) // 64), generator=g).float()).repeat_interleave(
            64, 1)[:, :C] * scale
    return x.to(TYPES[dtype])


# ---- quantisers ------------------------------------------------------------------


@pytest.mark.parametrize("M,C", [(1, 1), (1, 128), (3, 2048), (127, 129), (128, 256), (129, 100),
                                 (300, 516), (640, 130), (1000, 31), (5, 4100)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("pow2", [False, True])
def test_rows(moe, M, C, dtype, pow2):
    x = wide_rows(M, C, dtype, gen(M + C))
    q, t = moe.quantize_fp8(x.cuda(), pow2=pow2, by_column=True)
    codes, scales = ref.by_row(f32(x), pow2)
    assert np.array_equal(bytes_of(q.codes), codes)
    assert np.array_equal(f32(q.scales), scales)
    codes, scales = ref.by_column(f32(x), [0, M], pow2)
    assert t.codes.shape == (C, (M + 127) // 128 * 128)
    assert np.array_equal(bytes_of(t.codes), codes)
    assert np.array_equal(f32(t.scales), scales)
    only, none = moe.quantize_fp8(x.cuda(), pow2=pow2)
    assert none is None and np.array_equal(bytes_of(only.codes), bytes_of(q.codes))
    none, only = moe.quantize_fp8(x.cuda(), pow2=pow2, by_row=False, by_column=True)
    assert none is None and np.array_equal(bytes_of(only.codes), bytes_of(t.codes))


@pytest.mark.parametrize("counts", [[0, 0, 0], [1], [128, 128], [5, 0, 130, 1, 0, 64],
                                    [0, 300, 0], [1] * 40])
def test_segments_gathered(moe, counts):
    """Rows of experts through an index, rows outside all segments and columns beyond the
    last block left as they were."""
    E, used = len(counts), sum(counts)
    M, C, n_src = used + 37, 200, 50
    g = gen(7)
    x = wide_rows(n_src, C, "bf16", g)
    rows = torch.randint(-3, n_src + 3, (M,), generator=g, dtype=torch.int32)
    offsets = offsets_of(counts)
    R = moe.fp8_columns(M, E) + 128
    out = (torch.full((M, 208), 0x55, dtype=torch.uint8).cuda().view(F8)[:, :C],
           torch.full((2, M + 5), -1.0).cuda()[:, :M])
    out_t = (torch.full((C, R), 0x55, dtype=torch.uint8).cuda().view(F8),
             torch.full((R // 128, C), -1.0).cuda())
    q, t = moe.quantize_fp8(x.cuda(), rows=rows.cuda(), offsets=offsets.cuda(), by_column=True,
                            out=out, out_t=out_t)
    inside = (rows >= 0) & (rows < n_src)
    v = np.where(inside[:, None].numpy(), f32(x)[rows.clamp(0, n_src - 1).numpy()],
                 np.float32(0))
    codes, scales = ref.by_row(v)
    codes[used:], scales = 0x55, scales.copy()
    scales[:, used:] = -1
    assert np.array_equal(bytes_of(q.codes), codes)
    assert np.array_equal(f32(q.scales), scales)
    codes, scales = ref.by_column(v, offsets.tolist())
    n = codes.shape[1]
    assert np.array_equal(bytes_of(t.codes)[:, :n], codes)
    assert np.array_equal(f32(t.scales)[:n // 128], scales)
    assert (bytes_of(t.codes)[:, n:] == 0x55).all() and (f32(t.scales)[n // 128:] == -1).all()
    # only as many columns as fit, no further
    if n > 128:
        short = (torch.full((C, 128), 0x55, dtype=torch.uint8).cuda().view(F8),
                 torch.full((1, C), -1.0).cuda())
        guard = torch.full((4096,), 0x55, dtype=torch.uint8).cuda()
        _, t = moe.quantize_fp8(x.cuda(), rows=rows.cuda(), offsets=offsets.cuda(), by_row=False,
                                by_column=True, out_t=short)
        assert np.array_equal(bytes_of(t.codes), codes[:, :128])
        assert (guard == 0x55).all()


def test_bad_offsets_write_nothing(moe):
    M, C = 300, 64
    x = wide_rows(M, C, "bf16", gen(1)).cuda()
    for bad in ([0, 200, 100, 300], [-1, 10, 20, 30], [0, 10, 20, 301], [5, 2 ** 31 - 1, 7, 9]):
        out = (torch.full((M, C), 0x55, dtype=torch.uint8).cuda().view(F8),
               torch.full((1, M), -1.0).cuda())
        moe.quantize_fp8(x, offsets=torch.tensor(bad, dtype=torch.int32).cuda(), out=out)
        assert (out[0].view(torch.uint8) == 0x55).all() and (out[1] == -1).all()
        lin = moe.MoeFp8Linear(32, C, 3)
        w = moe.quantize_fp8_weights(torch.randn(3, 32, C).cuda())
        q, _ = moe.quantize_fp8(x)
        y = torch.full((M, 32), 7.0, dtype=torch.bfloat16).cuda()
        lin.forward(q, w, offsets=torch.tensor(bad, dtype=torch.int32).cuda(), out=y)
        assert (y == 7).all()
        assert lin.check()[0] == moe.MOE_ERR_INVALID_ARG and lin.check()[0] == moe.MOE_OK


def test_extremes(moe):
    """Zeros, the smallest and largest numbers, infinities and NaN."""
    x = torch.randn(8, 384, generator=gen(2))
    x[0] = 0
    x[1, :128] = 2.0 ** -140
    x[2, :128] = 2.0 ** -101
    x[3] = 3e38
    x[4, 5] = float("inf")
    x[5, 200] = float("nan")
    x[6, :128] = 2.0 ** -30
    x[6, 0] = 448.0
    x[7, 0] = -0.0
    for pow2 in (False, True):
        q, t = moe.quantize_fp8(x.cuda(), pow2=pow2, by_column=True)
        codes, scales = ref.by_row(x.numpy(), pow2)
        same = lambda a, b: np.array_equal(a, b, equal_nan=True)
        assert same(ref.values(bytes_of(q.codes), f32(q.scales)), ref.values(codes, scales))
        assert np.isnan(ref.values(codes, scales)[4, :128]).all()
        codes, scales = ref.by_column(x.numpy(), [0, 8], pow2)
        assert same(ref.values(bytes_of(t.codes), f32(t.scales)), ref.values(codes, scales))


@pytest.mark.parametrize("M,C", [(1, 1), (2, 64), (130, 128), (257, 300), (100, 77), (384, 768)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("clamp", [0.0, 1.25])
def test_swiglu(moe, M, C, dtype, clamp):
    g = gen(M + C)
    a = (torch.randn(M, 2 * C, generator=g) * 2).to(TYPES[dtype])
    dh = (torch.randn(M, C, generator=g) * 0.01).to(TYPES[dtype])
    if C > 1:
        a[0, :2] = torch.tensor([-90.0, 90.0])
    offsets = offsets_of([M // 3, M - M // 3])
    n, place = ref.columns(offsets.tolist(), M)
    for got, (want, mag) in (
            (moe.swiglu_fp8(a.cuda(), clamp, offsets.cuda(), by_column=True),
             ref.swiglu(f32(a), clamp)),
            (moe.swiglu_grad_fp8(dh.cuda(), a.cuda(), clamp, offsets.cuda(), by_column=True),
             ref.swiglu_grad(f32(dh), f32(a), clamp))):
        q, t = got
        ref.check_codes(bytes_of(q.codes), f32(q.scales), want, mag, "rows")
        tall, tall_mag = np.zeros((want.shape[1], n[-1])), np.zeros((want.shape[1], n[-1]))
        tall[:, place], tall_mag[:, place] = want.T, mag.T
        ref.check_codes(bytes_of(t.codes)[:, :n[-1]], f32(t.scales)[:n[-1] // 128], tall,
                        tall_mag, "columns")


def test_swiglu_nan_under_a_clamp(moe):
    a = torch.zeros(2, 256)
    a[0, 3] = float("nan")
    a[1, 128 + 4] = float("nan")
    q, _ = moe.swiglu_fp8(a.cuda(), 1.0)
    v = ref.values(bytes_of(q.codes), f32(q.scales))
    assert np.isnan(v).all()


@pytest.mark.parametrize("E,N,K", [(1, 1, 1), (1, 128, 128), (3, 130, 200), (2, 64, 1000),
                                   (5, 300, 48)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_weights(moe, E, N, K, dtype):
    w = wide_rows(E * N, K, dtype, gen(E + N)).view(E, N, K)
    for pow2 in (False, True):
        q, t = moe.quantize_fp8_weights(w.cuda(), transposed=True, pow2=pow2)
        codes, scales = ref.by_tile(f32(w), pow2)
        assert np.array_equal(bytes_of(q.codes), codes)
        assert np.array_equal(f32(q.scales), scales)
        assert np.array_equal(bytes_of(t.codes), codes.transpose(0, 2, 1))
        assert np.array_equal(f32(t.scales), scales.transpose(0, 2, 1))
        only = moe.quantize_fp8_weights(w.cuda(), pow2=pow2)
        assert np.array_equal(bytes_of(only.codes), codes)


# ---- products ----------------------------------------------------------------------


def operands(moe, M, N, K, E, seed, pow2=False):
    g = gen(seed)
    x, w = torch.randn(M, K, generator=g), torch.randn(E, N, K, generator=g) * K ** -0.5
    q, _ = moe.quantize_fp8(x.cuda(), pow2=pow2)
    wq, wt = moe.quantize_fp8_weights(w.cuda(), transposed=True, pow2=pow2)
    return q, wq, wt, ref.values(bytes_of(q.codes), f32(q.scales)), ref.tile_values(
        bytes_of(wq.codes), f32(wq.scales))


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 128, 128), (1, 1536, 2048), (2, 257, 129),
                                   (7, 64, 96), (16, 300, 500), (17, 512, 640), (64, 130, 4096),
                                   (65, 128, 33), (127, 129, 127), (128, 256, 256),
                                   (129, 300, 1000), (300, 1000, 260), (1003, 37, 513),
                                   (500, 640, 384)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_dense(moe, M, N, K, dtype):
    q, wq, wt, x, w = operands(moe, M, N, K, 1, M + N + K)
    lin = moe.MoeFp8Linear(N, K, dtype=TYPES[dtype])
    y = lin.forward(q, wq)
    ref.check_product(f32(y), x, w[0], "y", bf16=dtype == "bf16")
    # the gradient at the input: the transposed weights
    dy, _ = moe.quantize_fp8(torch.randn(M, N, generator=gen(1)).cuda())
    dx = lin.grad_input(dy, wt)
    ref.check_product(f32(dx), ref.values(bytes_of(dy.codes), f32(dy.scales)), w[0].T, "dx",
                      bf16=dtype == "bf16")
    assert lin.check() == (moe.MOE_OK, 0)


COUNTS = [[0, 3, 0, 1, 130, 0, 128, 64], [1] * 8, [0] * 7 + [5], [300] + [0] * 7,
          [1, 2, 3, 4, 5, 6, 7, 8], [17, 33, 65, 0, 1, 16, 32, 64], [0] * 8]


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("N,K", [(256, 512), (130, 200)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_experts(moe, counts, N, K, dtype):
    """Rows of experts; rows before, behind and between stay as they were."""
    E, used = len(counts), sum(counts)
    first, M = 9, 9 + used + 21
    q, wq, _, x, w = operands(moe, M, N, K, E, N + used)
    offsets = offsets_of(counts) + first
    lin = moe.MoeFp8Linear(N, K, E, dtype=TYPES[dtype])
    out = torch.full((M, N + 3), 7.0, dtype=TYPES[dtype]).cuda()
    y = lin.forward(q, wq, offsets=offsets.cuda(), out=out[:, :N])
    got, at = f32(out), offsets.tolist()
    for e in range(E):
        rows = slice(at[e], at[e + 1])
        ref.check_product(got[rows, :N], x[rows], w[e], "expert %d" % e, bf16=dtype == "bf16")
    assert (got[:first] == 7).all() and (got[first + used:] == 7).all() and (got[:, N:] == 7).all()
    dense = lin.forward(q, wq, offsets=offsets.cuda())
    assert torch.equal(dense[first:first + used], y[first:first + used])
    assert lin.check() == (moe.MOE_OK, 0)


@pytest.mark.parametrize("counts", [[1], [8], [9], [0, 1, 0, 20, 3], [32], [0, 0, 17, 8, 1, 5],
                                    [1] * 31, [0] * 6])
@pytest.mark.parametrize("N,K", [(16, 128), (40, 3001), (33, 17), (8, 20000)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_few_rows_of_experts(moe, counts, N, K, dtype):
    """Up to 32 rows, 32 of one expert among them, and more blocks than are on their way."""
    E, used = len(counts), sum(counts)
    first = min(1, 32 - used)
    M = max(used + first, 1)
    q, wq, _, x, w = operands(moe, M, N, K, E, N + used)
    offsets = offsets_of(counts) + first
    lin = moe.MoeFp8Linear(N, K, E, dtype=TYPES[dtype])
    out = torch.full((M, N + 1), 7.0, dtype=TYPES[dtype]).cuda()
    lin.forward(q, wq, offsets=offsets.cuda(), out=out[:, :N])
    got, at = f32(out), offsets.tolist()
    for e in range(E):
        rows = slice(at[e], at[e + 1])
        ref.check_product(got[rows, :N], x[rows], w[e], "expert %d" % e, bf16=dtype == "bf16")
    assert (got[:first] == 7).all() and (got[at[-1]:] == 7).all() and (got[:, N:] == 7).all()
    assert lin.check() == (moe.MOE_OK, 0)


@pytest.mark.parametrize("N,K", [(1500, 1300), (1501, 257)])
def test_more_tiles_than_processors(moe, N, K):
    """Every CTA takes several tiles, with all of its rings going round."""
    M = 7000
    q, wq, _, x, w = operands(moe, M, N, K, 1, 31)
    y = moe.MoeFp8Linear(N, K, dtype=torch.float32).forward(q, wq)
    ref.check_product(f32(y), x, w[0], "y")
    E, counts = 6, [700, 0, 130, 1, 900, 300]
    offsets = offsets_of(counts)
    both = dict(offsets=offsets.cuda(), by_row=False, by_column=True)
    g = gen(32)
    _, dy = moe.quantize_fp8(torch.randn(sum(counts), N, generator=g).cuda(), **both)
    _, xt = moe.quantize_fp8(torch.randn(sum(counts), K, generator=g).cuda(), **both)
    dw = f32(moe.MoeFp8Linear(N, K, E).grad_weight(dy, xt, offsets=offsets.cuda()))
    n, _ = ref.columns(offsets.tolist(), sum(counts))
    a, b = (ref.values(bytes_of(m.codes)[:, :n[-1]], f32(m.scales)[:n[-1] // 128])
            for m in (dy, xt))
    for e in range(E):
        cols = slice(n[e], n[e + 1])
        ref.check_product(dw[e], a[:, cols], b[:, cols], "dw %d" % e)


@pytest.mark.parametrize("E,N,K", [(256, 300, 520), (97, 129, 1300), (256, 100, 60)])
def test_weight_gradient_of_many_experts(moe, E, N, K):
    """Experts of every depth, none and the same as another's among them, whose tiles are
    dealt to the CTAs several times round."""
    counts = np.random.default_rng(E + N).integers(0, 520, E)
    counts[::7], counts[3::11] = 0, 256
    offsets = offsets_of(counts.tolist())
    R = int(counts.sum())
    both = dict(offsets=offsets.cuda(), by_row=False, by_column=True)
    g = gen(41)
    _, dy = moe.quantize_fp8(torch.randn(R, N, generator=g).cuda(), **both)
    _, xt = moe.quantize_fp8(torch.randn(R, K, generator=g).cuda(), **both)
    linear = moe.MoeFp8Linear(N, K, E)
    dw = linear.grad_weight(dy, xt, offsets=offsets.cuda())
    n, _ = ref.columns(offsets.tolist(), R)
    a, b = (ref.values(bytes_of(m.codes)[:, :n[-1]], f32(m.scales)[:n[-1] // 128])
            for m in (dy, xt))
    got = f32(dw)
    for e in range(E):
        cols = slice(n[e], n[e + 1])
        ref.check_product(got[e], a[:, cols], b[:, cols], "dw %d" % e)
    assert torch.equal(dw, linear.grad_weight(dy, xt, offsets=offsets.cuda()))


@pytest.mark.parametrize("shift", [0, 1, 2, 4])
@pytest.mark.parametrize("N,K", [(130, 260), (33, 36), (200, 1028)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_weight_gradient_in_place(moe, shift, N, K, accumulate):
    """Weights at 16-byte boundaries and between them, alike to the bit, and nothing written
    beside them."""
    E, offsets = 3, offsets_of([140, 0, 300])
    both = dict(offsets=offsets.cuda(), by_row=False, by_column=True)
    g = gen(51)
    _, dy = moe.quantize_fp8(torch.randn(440, N, generator=g).cuda(), **both)
    _, xt = moe.quantize_fp8(torch.randn(440, K, generator=g).cuda(), **both)
    linear = moe.MoeFp8Linear(N, K, E)
    want = linear.grad_weight(dy, xt, offsets=offsets.cuda())
    room = torch.randn(shift + E * N * K + 64, generator=g).cuda()
    before = room.clone()
    dw = room[shift:shift + E * N * K].view(E, N, K)
    linear.grad_weight(dy, xt, offsets=offsets.cuda(), dw=dw, accumulate=accumulate)
    old = before[shift:shift + E * N * K].view(E, N, K)
    assert torch.equal(dw, old + want if accumulate else want)
    assert torch.equal(room[:shift], before[:shift])
    assert torch.equal(room[shift + E * N * K:], before[shift + E * N * K:])


def test_every_significand(moe):
    """Scales of all 2^23 significands are the rounded quotients."""
    top = (np.arange(1 << 23, dtype=np.uint32) | np.uint32(0x3F800000)).view(np.float32)
    q, _ = moe.quantize_fp8(torch.from_numpy(top)[:, None].cuda())
    assert np.array_equal(f32(q.scales)[0], top / np.float32(448))
    # and the factors: 300 / x times x / 300 of a second element lands on a code's border or
    # on one side of it as the rounded product says
    x = np.stack([top, top * np.float32(0.0390625)], 1)       # codes of 17.5, between 17 and 18
    q, _ = moe.quantize_fp8(torch.from_numpy(x).cuda())
    want = ref.e4m3(x * (np.float32(448) / top)[:, None])
    assert np.array_equal(bytes_of(q.codes), want)


def test_many_experts(moe):
    g = gen(11)
    E, N, K = 256, 192, 384
    counts = torch.randint(0, 9, (E,), generator=g).tolist()
    M = sum(counts)
    q, wq, _, x, w = operands(moe, M, N, K, E, 12)
    offsets = offsets_of(counts)
    lin = moe.MoeFp8Linear(N, K, E)
    got, at = f32(lin.forward(q, wq, offsets=offsets.cuda())), offsets.tolist()
    for e in range(E):
        rows = slice(at[e], at[e + 1])
        ref.check_product(got[rows], x[rows], w[e], "expert %d" % e, bf16=True)


@pytest.mark.parametrize("R,N,K", [(1, 1, 1), (5, 40, 300), (128, 128, 256), (130, 129, 100),
                                   (1000, 257, 515), (2000, 300, 64)])
def test_weight_gradient_dense(moe, R, N, K):
    g = gen(R + N)
    _, dy = moe.quantize_fp8(torch.randn(R, N, generator=g).cuda(), by_row=False, by_column=True)
    _, x = moe.quantize_fp8(torch.randn(R, K, generator=g).cuda(), by_row=False, by_column=True)
    lin = moe.MoeFp8Linear(N, K)
    a, b = (ref.values(bytes_of(m.codes), f32(m.scales)) for m in (dy, x))
    dw = lin.grad_weight(dy, x)
    ref.check_product(f32(dw)[0], a, b, "dw")
    base = torch.randn(1, N, K, generator=g)
    more = lin.grad_weight(dy, x, dw=base.clone().cuda(), accumulate=True)
    ref.check_product(f32(more)[0], a, b, "dw added", base=base[0].double().numpy())
    assert torch.equal(lin.grad_weight(dy, x), dw)
    assert lin.check() == (moe.MOE_OK, 0)


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("N,K", [(256, 264), (65, 131)])
def test_weight_gradient_experts(moe, counts, N, K):
    g = gen(N + sum(counts))
    E, M = len(counts), sum(counts)
    offsets = offsets_of(counts)
    if M == 0:
        M = 3
    both = dict(offsets=offsets.cuda(), by_row=False, by_column=True)
    _, dy = moe.quantize_fp8(torch.randn(M, N, generator=g).cuda(), **both)
    _, x = moe.quantize_fp8(torch.randn(M, K, generator=g).cuda(), **both)
    lin = moe.MoeFp8Linear(N, K, E)
    n, _ = ref.columns(offsets.tolist(), M)
    a, b = (ref.values(bytes_of(m.codes)[:, :n[-1]], f32(m.scales)[:n[-1] // 128])
            for m in (dy, x))
    base = torch.randn(E, N, K, generator=g)
    dw = f32(lin.grad_weight(dy, x, offsets=offsets.cuda(),
                             dw=torch.full((E, N, K), float("nan")).cuda()))
    more = f32(lin.grad_weight(dy, x, offsets=offsets.cuda(), dw=base.clone().cuda(),
                               accumulate=True))
    for e in range(E):
        cols = slice(n[e], n[e + 1])
        ref.check_product(dw[e], a[:, cols], b[:, cols], "dw %d" % e)
        ref.check_product(more[e], a[:, cols], b[:, cols], "dw added %d" % e,
                          base=base[e].double().numpy())
    assert lin.check() == (moe.MOE_OK, 0)


def test_scales_of_any_size(moe):
    """Block scales 2^60 apart, in both operands."""
    M, N, K = 40, 60, 1024
    g = gen(13)
    q, wq, _, _, _ = operands(moe, M, N, K, 1, 14)
    q = moe.Fp8Matrix(q.codes, torch.exp2(torch.randint(-30, 30, (8, M), generator=g).float())
                      .cuda())
    wq = moe.Fp8Matrix(wq.codes, torch.exp2(torch.randint(-30, 30, (1, 1, 8), generator=g)
                                            .float()).cuda())
    y = moe.MoeFp8Linear(N, K, dtype=torch.float32).forward(q, wq)
    x = ref.values(bytes_of(q.codes), f32(q.scales))
    w = ref.tile_values(bytes_of(wq.codes), f32(wq.scales))
    ref.check_product(f32(y), x, w[0], "y")


def test_nan_stays_in_its_rows(moe):
    M, N, K = 150, 70, 300
    x = torch.randn(M, K, generator=gen(15))
    x[3, 5] = float("nan")
    x[140, 299] = float("inf")
    q, _ = moe.quantize_fp8(x.cuda())
    w = moe.quantize_fp8_weights(torch.randn(N, K, generator=gen(16)).cuda())
    y = f32(moe.MoeFp8Linear(N, K).forward(q, w))
    bad = np.zeros(M, bool)
    bad[[3, 140]] = True
    assert np.isnan(y[bad]).all() and np.isfinite(y[~bad]).all()


def test_no_rows(moe):
    lin = moe.MoeFp8Linear(64, 128, 2)
    w = moe.quantize_fp8_weights(torch.randn(2, 64, 128).cuda())
    offsets = torch.zeros(3, dtype=torch.int32).cuda()
    q, t = moe.quantize_fp8(torch.zeros(0, 128).cuda(), offsets=offsets, by_column=True)
    assert q.codes.shape == (0, 128)
    assert lin.forward(q, w, offsets=offsets).shape == (0, 64)
    empty = lambda n: (torch.zeros(n, 0, dtype=torch.uint8).cuda().view(F8),
                       torch.zeros(0, n).cuda())
    dw = lin.grad_weight(empty(64), empty(128), offsets=offsets)
    assert (dw == 0).all()
    dw.fill_(2)
    lin.grad_weight(empty(64), empty(128), offsets=offsets, dw=dw, accumulate=True)
    assert (dw == 2).all()


def test_replay_and_streams(moe):
    """A captured step on another stream gives the bits of the eager one."""
    M, N, K, E = 200, 320, 384, 4
    g = gen(17)
    x = torch.randn(M, K, generator=g).cuda()
    offsets = offsets_of([50, 0, 120, 30]).cuda()
    wq = moe.quantize_fp8_weights(torch.randn(E, N, K, generator=g).cuda())
    lin = moe.MoeFp8Linear(N, K, E)
    q, t = moe.quantize_fp8(x, offsets=offsets, by_column=True)
    y = lin.forward(q, wq, offsets=offsets)
    _, dy = moe.quantize_fp8(y, offsets=offsets, by_row=False, by_column=True)
    dw = lin.grad_weight(dy, t, offsets=offsets)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2 = lin.forward(q, wq, offsets=offsets, stream=side)
    side.synchronize()
    assert torch.equal(y, y2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q3, t3 = moe.quantize_fp8(x, offsets=offsets, by_column=True)
        y3 = lin.forward(q3, wq, offsets=offsets)
        _, dy3 = moe.quantize_fp8(y3, offsets=offsets, by_row=False, by_column=True)
        dw3 = lin.grad_weight(dy3, t3, offsets=offsets)
    for _ in range(2):
        y3.zero_()
        dw3.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y3) and torch.equal(dw, dw3)


def test_rows_beyond_32_bits(moe):
    """Codes, scales and outputs more than 2^32 bytes from their tensors' starts."""
    N, K = 128, 16384
    M = (1 << 32) // K + 300
    codes = torch.zeros(M, K, dtype=torch.uint8, device="cuda")
    scales = torch.ones(K // 128, M, device="cuda")
    q, _ = moe.quantize_fp8(torch.randn(200, K, generator=gen(18)).cuda())
    codes[-200:], scales[:, -200:] = q.codes.view(torch.uint8), q.scales
    w = moe.quantize_fp8_weights(torch.randn(N, K, generator=gen(19)).cuda())
    y = moe.MoeFp8Linear(N, K, dtype=torch.float32).forward((codes.view(F8), scales), w)
    x = ref.values(bytes_of(q.codes), f32(q.scales))
    ref.check_product(f32(y[-200:]), x, ref.tile_values(bytes_of(w.codes), f32(w.scales))[0], "y")
    assert (y[:-200] == 0).all()
    del codes, scales, y
    x = torch.zeros(M // 2 + 100, K, dtype=torch.bfloat16, device="cuda")
    x[-7] = torch.randn(K, generator=gen(20)).cuda()
    far, _ = moe.quantize_fp8(x)
    near, _ = moe.quantize_fp8(x[-7:-6])
    assert torch.equal(far.codes[-7].view(torch.uint8), near.codes[0].view(torch.uint8))
    assert torch.equal(far.scales[:, -7], near.scales[:, 0])


# ---- together ------------------------------------------------------------------------


def test_experts_layer_forward_and_backward(moe):
    """Router with groups, dispatch, the experts' two products with SwiGLU between, combined;
    then every gradient, all on the codes, against 64-bit products of the same codes."""
    T, d, I, E, k = 150, 256, 192, 16, 4
    g = gen(21)
    x = torch.randn(T, d, generator=g).to(torch.bfloat16).cuda()
    w13 = (torch.randn(E, 2 * I, d, generator=g) * d ** -0.5).cuda()
    w2 = (torch.randn(E, d, I, generator=g) * I ** -0.5).cuda()
    logits = torch.randn(T, E, generator=g).cuda()
    router = moe.MoeGroupRouter(T, E, k, 4, 2)
    route = router.forward(logits, bias=torch.zeros(E).cuda())
    # rows in their experts' order, as a dispatch lays them out
    flat = route.ids.long().view(-1)
    order = flat.sort(stable=True)[1]
    token = (order // k).to(torch.int32)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64).cuda(),
                         torch.bincount(flat, minlength=E).cumsum(0)]).to(torch.int32)
    at = offsets.tolist()
    up, down = moe.MoeFp8Linear(2 * I, d, E), moe.MoeFp8Linear(d, I, E, dtype=torch.float32)
    w13q, w13t = moe.quantize_fp8_weights(w13, transposed=True)
    w2q, w2t = moe.quantize_fp8_weights(w2, transposed=True)
    xq, xt = moe.quantize_fp8(x, rows=token, offsets=offsets, by_column=True)
    a = up.forward(xq, w13q, offsets=offsets)
    hq, ht = moe.swiglu_fp8(a, offsets=offsets, by_column=True)
    rows = down.forward(hq, w2q, offsets=offsets)
    weight = route.scores.view(-1)[order]
    y = torch.zeros(T, d, device="cuda").index_add_(0, token.long(), rows * weight[:, None])

    def val(m):
        return ref.values(bytes_of(m.codes), f32(m.scales))

    def tiles(m):
        return ref.tile_values(bytes_of(m.codes), f32(m.scales))

    X, H, W13, W2 = val(xq), val(hq), tiles(w13q), tiles(w2q)
    for e in range(E):
        s = slice(at[e], at[e + 1])
        ref.check_product(f32(a)[s], X[s], W13[e], "a", bf16=True)
        ref.check_product(f32(rows)[s], H[s], W2[e], "rows")
    ref.check_codes(bytes_of(hq.codes), f32(hq.scales), *ref.swiglu(f32(a)), "h")
    # the layer itself, without codes: every operand is off by up to 2^-4 of an element,
    # three of them one after another, independently
    full = np.zeros((T, d))
    for i, f in enumerate(order.tolist()):
        e, t = int(flat[f]), f // k
        h, _ = ref.swiglu((f32(w13[e]).astype(np.float64) @ f32(x)[t])[None])
        full[t] += float(weight[i]) * (f32(w2[e]).astype(np.float64) @ h[0])
    assert np.linalg.norm(f32(y) - full) <= 0.1 * np.linalg.norm(full)

    # backward
    dy = (torch.randn(T, d, generator=g) * 0.01).cuda()
    drows = dy[token.long()] * weight[:, None]
    gq, gt = moe.quantize_fp8(drows, offsets=offsets, by_column=True)
    dh = down.grad_input(gq, w2t, offsets=offsets)
    dw2 = down.grad_weight(gt, ht, offsets=offsets)
    a32 = a.float()
    aq, at_ = moe.swiglu_grad_fp8(dh, a32, offsets=offsets, by_column=True)
    dxe = up.grad_input(aq, w13t, offsets=offsets)
    dw13 = up.grad_weight(at_, xt, offsets=offsets)
    n, place = ref.columns(at, len(order))

    def cols(m):
        return ref.values(bytes_of(m.codes)[:, :n[-1]], f32(m.scales)[:n[-1] // 128])

    G, A, Gt, Ht, At, Xt = val(gq), val(aq), cols(gt), cols(ht), cols(at_), cols(xt)
    ref.check_codes(bytes_of(aq.codes), f32(aq.scales), *ref.swiglu_grad(f32(dh), f32(a)), "da")
    for e in range(E):
        s, c = slice(at[e], at[e + 1]), slice(n[e], n[e + 1])
        ref.check_product(f32(dh)[s], G[s], W2[e].T, "dh")
        ref.check_product(f32(dxe)[s], A[s], W13[e].T, "dx", bf16=True)
        ref.check_product(f32(dw2)[e], Gt[:, c], Ht[:, c], "dw2")
        ref.check_product(f32(dw13)[e], At[:, c], Xt[:, c], "dw13")
    for lin in (up, down):
        assert lin.check() == (moe.MOE_OK, 0)
    # the whole against 64-bit autograd of the layer without codes
    w13_, w2_ = (t.double().cpu().requires_grad_(True) for t in (w13, w2))
    X64 = x.double().cpu()[token.long().cpu()]
    total = 0
    for e in range(E):
        s = slice(at[e], at[e + 1])
        u = X64[s] @ w13_[e].t()
        h = torch.nn.functional.silu(u[:, :I]) * u[:, I:]
        total = total + ((h @ w2_[e].t()) * drows[s].double().cpu()).sum()
    total.backward()
    for got, want in ((dw13, w13_.grad), (dw2, w2_.grad)):
        assert (got.double().cpu() - want).norm() <= 0.12 * want.norm()
