"""The 8-bit block operators and the router with groups where every CTA takes many tiles (or
every warp many rows): against calls so small that none takes a second one, against the block
rule in torch, and against 64-bit products."""

import ctypes

import numpy as np
import pytest
import torch

import fp8_refs as ref
from test_gpu_fp8 import F8, TYPES, bytes_of, f32, gen, moe, offsets_of  # noqa: F401

pytestmark = pytest.mark.gpu


def i32(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


def raw(t):
    return t.contiguous().view(torch.uint8)


def cuda_gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rule(blocks):
    """Codes and scales of [..., 128] fp32: each quotient of two tensors, so rounded to nearest."""
    top = blocks.abs().amax(-1).clamp(min=2.0 ** -100)
    limit = torch.full_like(top, 448.0)
    return ((blocks * torch.div(limit, top)[..., None]).to(F8).view(torch.uint8),
            torch.div(top, limit))


def inputs(source, M, C, dtype, seed):
    g = cuda_gen(seed)
    n = lambda w: torch.randn(M, w, generator=g, device="cuda").mul_(
        torch.exp2(torch.randint(-8, 8, (M, 1), generator=g, device="cuda").float())).to(
            TYPES[dtype])
    return (n(C),) if source == "rows" else (n(2 * C),) if source == "swiglu" else (n(C), n(2 * C))


def quantise(moe, source, x, **kw):
    return {"rows": moe.quantize_fp8, "swiglu": moe.swiglu_fp8,
            "swiglu_grad": moe.swiglu_grad_fp8}[source](*x, **kw)


# of some 300 CTAs (the gradient's 152) each has 2 to 30 tiles, alone or in runs of neighbours
@pytest.mark.parametrize("source,M,C", [("rows", 128 * 300, 300), ("rows", 128 * 70, 2048 + 8),
                                        ("rows", 128 * 600, 2048), ("rows", 128 * 200, 515),
                                        ("swiglu", 128 * 300, 384), ("swiglu", 128 * 200, 130),
                                        ("swiglu", 128 * 900, 1000),
                                        ("swiglu_grad", 128 * 300, 256),
                                        ("swiglu_grad", 128 * 900, 768),
                                        ("swiglu_grad", 128 * 200, 388),
                                        ("swiglu_grad", 128 * 150, 133)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_quantisers_of_many_tiles(moe, source, M, C, dtype):
    x = inputs(source, M, C, dtype, M + C)
    q, t = quantise(moe, source, x, by_column=True)
    only, _ = quantise(moe, source, x)
    _, only_t = quantise(moe, source, x, by_row=False, by_column=True)
    assert torch.equal(raw(only.codes), raw(q.codes)) and torch.equal(only.scales, q.scales)
    assert torch.equal(raw(only_t.codes), raw(t.codes)) and torch.equal(only_t.scales, t.scales)
    width = q.codes.shape[1]
    step = 128 * max(1, 120 // ((width + 127) // 128))         # at most 120 tiles a call
    for lo in range(0, M, step):
        hi = min(lo + step, M)
        a, b = quantise(moe, source, [v[lo:hi] for v in x], by_column=True)
        assert torch.equal(raw(a.codes), raw(q.codes[lo:hi])), lo
        assert torch.equal(a.scales, q.scales[:, lo:hi]), lo
        assert torch.equal(raw(b.codes), raw(t.codes[:, lo:hi])), lo
        assert torch.equal(b.scales, t.scales[lo // 128:hi // 128]), lo
    if source == "rows":
        v = torch.zeros(M, (C + 127) // 128 * 128, device="cuda")
        v[:, :C] = x[0]
        codes, scales = rule(v.view(M, -1, 128))
        assert torch.equal(raw(q.codes), codes.view(M, -1)[:, :C].contiguous())
        assert torch.equal(q.scales, scales.t())
        codes, scales = rule(x[0].float().t().reshape(C, -1, 128))
        assert torch.equal(raw(t.codes), codes.view(C, -1))
        assert torch.equal(t.scales, scales.t())


@pytest.mark.parametrize("source,C", [("rows", 1024), ("rows", 1030), ("swiglu", 512),
                                      ("swiglu_grad", 512), ("swiglu_grad", 300)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_segments_of_many_tiles(moe, source, C, dtype):
    """Gathered where rows can be; every segment as by itself."""
    rng = np.random.default_rng(C)
    counts = rng.integers(0, 900, 60)
    counts[::9], counts[1::9], counts[2::9] = 0, 128, 1
    M, E, offsets = int(counts.sum()), len(counts), offsets_of(counts.tolist())
    x, kw = inputs(source, M, C, dtype, C), {}
    if source == "rows":
        kw["rows"] = torch.randint(-2, M + 2, (M,), generator=cuda_gen(1), device="cuda",
                                   dtype=torch.int32)
    q, t = quantise(moe, source, x, offsets=offsets.cuda(), by_column=True, **kw)
    n, _ = ref.columns(offsets.tolist(), M)
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if lo == hi:
            continue
        if source == "rows":
            a, b = quantise(moe, source, x, by_column=True, rows=kw["rows"][lo:hi])
        else:
            a, b = quantise(moe, source, [v[lo:hi] for v in x], by_column=True)
        assert torch.equal(raw(a.codes), raw(q.codes[lo:hi])), e
        assert torch.equal(a.scales, q.scales[:, lo:hi]), e
        assert torch.equal(raw(b.codes), raw(t.codes[:, n[e]:n[e + 1]])), e
        assert torch.equal(b.scales, t.scales[n[e] // 128:n[e + 1] // 128]), e


@pytest.mark.parametrize("E,N,K", [(40, 640, 1280), (9, 1000, 1300), (3, 2049, 3001)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_weights_of_many_tiles(moe, E, N, K, dtype):
    w = torch.randn(E, N, K, generator=cuda_gen(E), device="cuda").mul_(
        torch.exp2(torch.randint(-8, 8, (E, N, 1), generator=cuda_gen(2), device="cuda").float()))
    w = w.to(TYPES[dtype])
    q, t = moe.quantize_fp8_weights(w, transposed=True)
    only = moe.quantize_fp8_weights(w)
    nb, kb = (N + 127) // 128, (K + 127) // 128
    v = torch.zeros(E, nb * 128, kb * 128, device="cuda")
    v[:, :N, :K] = w
    v = v.view(E, nb, 128, kb, 128)
    top = v.abs().amax((2, 4)).clamp(min=2.0 ** -100)
    limit = torch.full_like(top, 448.0)
    codes = (v * torch.div(limit, top)[:, :, None, :, None]).to(F8).view(torch.uint8).view(
        E, nb * 128, kb * 128)[:, :N, :K]
    assert torch.equal(raw(q.codes), codes.contiguous())
    assert torch.equal(q.scales, torch.div(top, limit))
    assert torch.equal(raw(t.codes), codes.transpose(1, 2).contiguous())
    assert torch.equal(t.scales, q.scales.transpose(1, 2))
    assert torch.equal(raw(only.codes), raw(q.codes)) and torch.equal(only.scales, q.scales)


def values(m, lo=None, hi=None):
    """64-bit values of codes by rows (or of some columns of codes by columns)."""
    v = m.codes[:, lo:hi].double()
    s = m.scales.double().t().repeat_interleave(128, 1)
    return v * s[:, lo:hi][:, :v.shape[1]]


def near(got, a, b, what):
    """got against a b^T, as fp8_refs.check_product has it."""
    want, mag = a @ b.t(), a.abs() @ b.abs().t()
    tol = (256 + 3 * ((a.shape[1] + 127) // 128)) * 2.0 ** -24 * mag
    assert bool(((got.double() - want).abs() <= tol).all()), what


@pytest.mark.parametrize("N,K", [(1000, 520), (1536, 260), (129, 2047)])
def test_products_over_experts_of_many_tiles(moe, N, K):
    """Forward, the gradient at the inputs and the weights' gradient of experts with ragged
    ends."""
    rng = np.random.default_rng(N)
    counts = rng.integers(0, 700, 50)
    counts[::9], counts[1::9], counts[2::9] = 0, 128, 1
    M, E, offsets = int(counts.sum()), len(counts), offsets_of(counts.tolist())
    g, off = cuda_gen(N), offsets.cuda()
    x, dy = (torch.randn(M, w, generator=g, device="cuda") for w in (K, N))
    w, wt = moe.quantize_fp8_weights(torch.randn(E, N, K, generator=g, device="cuda"),
                                     transposed=True)
    (xq, xc), (yq, yc) = (moe.quantize_fp8(v, offsets=off, by_column=True) for v in (x, dy))
    lin = moe.MoeFp8Linear(N, K, E, dtype=torch.float32)
    y, dx = lin.forward(xq, w, offsets=off), lin.grad_input(yq, wt, offsets=off)
    dw = lin.grad_weight(yc, xc, offsets=off)
    n, _ = ref.columns(offsets.tolist(), M)
    X, DY = values(xq), values(yq)
    for e in range(E):
        rows = slice(int(offsets[e]), int(offsets[e + 1]))
        W = w.codes[e].double() * w.scales[e].double().repeat_interleave(128, 0)[
            :N].repeat_interleave(128, 1)[:, :K]
        near(y[rows], X[rows], W, "y %d" % e)
        near(dx[rows], DY[rows], W.t(), "dx %d" % e)
        near(dw[e], values(yc, n[e], n[e + 1]), values(xc, n[e], n[e + 1]), "dw %d" % e)
    assert lin.check() == (moe.MOE_OK, 0)


BAD = [[0, 200, 100, 300], [-1, 10, 20, 30], [0, 10, 20, 301], [5, 2 ** 31 - 1, 7, 9]]


@pytest.mark.parametrize("bad", BAD)
def test_bad_offsets_by_columns(moe, bad):
    """Neither codes along columns nor a weight gradient are written; the gradient records it."""
    M, N, K, E = 300, 70, 260, 3
    g = gen(71)
    dy, x = torch.randn(M, N, generator=g).cuda(), torch.randn(M, K, generator=g).cuda()
    R = moe.fp8_columns(M, E)
    for source in ("rows", "swiglu", "swiglu_grad"):
        width = {"rows": K, "swiglu": K // 2, "swiglu_grad": 2 * K}[source]
        out = (torch.full((M, (width + 15) // 16 * 16), 0x55, dtype=torch.uint8).cuda().view(F8)[
            :, :width], torch.full(((width + 127) // 128, M), -1.0).cuda())
        out_t = (torch.full((width, R), 0x55, dtype=torch.uint8).cuda().view(F8),
                 torch.full((R // 128, width), -1.0).cuda())
        a = (x, torch.cat([x, x], 1)) if source == "swiglu_grad" else (x,)
        quantise(moe, source, a, offsets=i32(bad), by_column=True, out=out, out_t=out_t)
        for codes, scales in (out, out_t):
            assert (raw(codes) == 0x55).all() and (scales == -1).all()
    good = dict(offsets=i32([0, 100, 250, 300]), by_row=False, by_column=True)
    (_, dyq), (_, xq) = moe.quantize_fp8(dy, **good), moe.quantize_fp8(x, **good)
    lin = moe.MoeFp8Linear(N, K, E)
    for accumulate in (False, True):
        if bad == [0, 10, 20, 301]:          # (whose blocks fit into the columns)
            continue
        dw = torch.full((E, N, K), 7.0).cuda()
        lin.grad_weight(dyq, xq, offsets=i32(bad), dw=dw, accumulate=accumulate)
        assert (dw == 7).all()
        assert lin.check()[0] == moe.MOE_ERR_INVALID_ARG and lin.check()[0] == moe.MOE_OK


# ---- beyond 32 bits --------------------------------------------------------------


def test_outputs_and_scales_beyond_32_bits(moe):
    """An output of more than 2^32 elements, scales of more than 2^32 bytes, from first to last."""
    M, N, K, apart = 300, 200, 520, (1 << 24) + 4
    g = gen(72)
    out = torch.zeros(M * apart, dtype=torch.float32, device="cuda")      # 2^32 elements and more
    assert out.numel() > 1 << 32
    y = out.view(M, apart)[:, 3:3 + N]
    q, _ = moe.quantize_fp8(torch.randn(M, K, generator=g).cuda())
    w = moe.quantize_fp8_weights(torch.randn(N, K, generator=g).cuda())
    lin = moe.MoeFp8Linear(N, K, dtype=torch.float32)
    want = lin.forward(q, w)
    lin.forward(q, w, out=y)
    assert torch.equal(y, want)
    y.zero_()
    lin.forward((q.codes[:20], q.scales[:, :20].contiguous()), w, out=y[-20:])
    assert torch.equal(y[-20:, :], lin.forward((q.codes[:20], q.scales[:, :20].contiguous()), w))
    y.zero_()
    assert int(torch.count_nonzero(out)) == 0                # nothing beside the rows' columns
    # the scales [blocks, M] of both quantisers and operands, rows as far apart
    far = out[:6 * (1 << 29)].view(6, 1 << 29)
    scales = far[:5, 5:5 + M]
    p, _ = moe.quantize_fp8(torch.randn(M, K, generator=gen(73)).cuda(),
                            out=(torch.empty(M, 528, dtype=torch.uint8).cuda().view(F8)[:, :K],
                                 scales))
    near_p = moe.Fp8Matrix(p.codes, scales.contiguous())
    assert torch.equal(lin.forward(p, w), lin.forward(near_p, w))
    few = lambda m: (m.codes[:9], m.scales[:, :9])
    assert torch.equal(lin.forward(few(p), w), lin.forward(few(near_p), w))


def test_weight_gradients_beyond_32_bits(moe):
    """More than 2^32 elements of dw, of which the last experts' are looked at."""
    E, N, K = 132, 8192, 4096
    counts = [0] * (E - 2) + [130, 3]
    offsets = i32([0] * (E - 1) + [130, 133])
    assert E * N * K > 1 << 32 and len(counts) == E
    both = dict(offsets=offsets, by_row=False, by_column=True)
    g = cuda_gen(74)
    _, dy = moe.quantize_fp8(torch.randn(133, N, generator=g, device="cuda"), **both)
    _, x = moe.quantize_fp8(torch.randn(133, K, generator=g, device="cuda"), **both)
    dw = torch.full((E, N, K), 5.0, device="cuda")
    lin = moe.MoeFp8Linear(N, K, E)
    lin.grad_weight(dy, x, offsets=offsets, dw=dw)
    assert int(torch.count_nonzero(dw[:-2])) == 0
    near(dw[-2], values(dy, 0, 256), values(x, 0, 256), "first")
    near(dw[-1], values(dy, 256, 384), values(x, 256, 384), "last")
    more = dw[-2:].clone()
    lin.grad_weight(dy, x, offsets=offsets, dw=dw, accumulate=True)
    assert torch.equal(dw[-2:], more * 2) and int(torch.count_nonzero(dw[0])) == 0


def test_codes_by_columns_beyond_32_bits(moe):
    """More than 2^32 codes, and 2^32 bytes between the first and the last rows of x."""
    M, C = (1 << 20) + 200, 4160
    x = torch.zeros(M, C, dtype=torch.bfloat16, device="cuda")
    x[-300:] = torch.randn(300, C, generator=cuda_gen(75), device="cuda")
    q, t = moe.quantize_fp8(x, by_column=True)
    lo = (M - 300) // 128 * 128
    a, b = moe.quantize_fp8(x[lo:], by_column=True)
    assert t.codes.numel() > 1 << 32
    assert torch.equal(raw(q.codes[lo:]), raw(a.codes)) and torch.equal(q.scales[:, lo:], a.scales)
    assert torch.equal(raw(t.codes[:, lo:]), raw(b.codes))
    assert torch.equal(t.scales[lo // 128:], b.scales)
    assert int(torch.count_nonzero(raw(t.codes[-1])[:lo])) == 0


# ---- the dispatch's own tables ------------------------------------------------------


def test_on_the_tables_of_a_dispatch(moe):
    """moe_dispatch_static's padded offsets and token_of, whose padding is -1, as the header
    names them: forward and backward of one product, against the sum over each token's experts."""
    T, k, E, N, K = 333, 4, 24, 200, 260
    L = moe.lib()
    g = gen(76)
    like = torch.rand(T, E, generator=g)
    like[:, 3], like[:, 7] = -1.0, 2.0                     # every token's expert, and nobody's
    ids = like.argsort(1)[:, :k].to(torch.int32).cuda()
    scores = torch.rand(T, k, generator=g).cuda()
    cap = (T * k + E * 127) // 128 * 128
    e32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")
    m_indptr, off_pad, row_of, token_of = e32(E + 1), e32(E + 1), e32(T * k), e32(cap)
    status = e32(2)
    score_of = torch.empty(cap, device="cuda")
    vp, n = ctypes.c_void_p, ctypes.c_int
    L.moe_dispatch_static.argtypes = [vp, vp, n, n, n] + [vp] * 5 + [ctypes.c_longlong, vp, vp]
    L.moe_dispatch_static.restype = n
    p = lambda t: t.data_ptr()
    assert L.moe_dispatch_static(p(ids), p(scores), T, k, E, p(m_indptr), p(off_pad), p(row_of),
                                 p(token_of), p(score_of), cap, p(status),
                                 torch.cuda.current_stream().cuda_stream) == moe.MOE_OK
    assert status.tolist()[0] == moe.MOE_OK
    x = torch.randn(T, K, generator=g).to(torch.bfloat16).cuda()
    w, wt = moe.quantize_fp8_weights(torch.randn(E, N, K, generator=g).cuda(), transposed=True)
    lin = moe.MoeFp8Linear(N, K, E, dtype=torch.float32)
    used = int(off_pad[-1])
    xq, xc = moe.quantize_fp8(x, rows=token_of, offsets=off_pad, by_column=True)
    y = lin.forward(xq, w, offsets=off_pad)
    token = token_of[:used].long()
    assert (token == -1).any() and (y[:used][token == -1] == 0).all()
    dense, _ = moe.quantize_fp8(x)
    X, W = values(dense), torch.stack([w.codes[e].double() * w.scales[e].double().repeat_interleave(
        128, 0)[:N].repeat_interleave(128, 1)[:, :K] for e in range(E)])
    for j in range(k):
        rows = row_of.view(T, k)[:, j].long()
        e = ids[:, j].long()
        want = torch.bmm(W[e], X[:, :, None])[:, :, 0]
        mag = torch.bmm(W[e].abs(), X.abs()[:, :, None])[:, :, 0]
        assert bool(((y[rows].double() - want).abs() <= (256 + 9) * 2.0 ** -24 * mag).all())
    dy = torch.randn(T, N, generator=g).cuda()
    dyq, dyc = moe.quantize_fp8(dy, rows=token_of, offsets=off_pad, by_column=True)
    dx, dw = lin.grad_input(dyq, wt, offsets=off_pad), lin.grad_weight(dyc, xc, offsets=off_pad)
    for e in range(E):
        rows = slice(int(off_pad[e]), int(off_pad[e + 1]))     # whole blocks: the columns too
        near(dx[rows], values(dyq)[rows], W[e].t(), "dx %d" % e)
        near(dw[e], values(dyc, rows.start, rows.stop), values(xc, rows.start, rows.stop), "dw")
    assert lin.check() == (moe.MOE_OK, 0)


# ---- router -------------------------------------------------------------------------


@pytest.mark.parametrize("E,k,groups,top", [(256, 8, 8, 4), (160, 6, 20, 5), (96, 24, 3, 1),
                                            (33, 2, 11, 4)])
@pytest.mark.parametrize("scoring", ["softmax_topk", "softmax", "sigmoid"])
@pytest.mark.parametrize("pair", [False, True])
def test_router_of_many_rows(moe, E, k, groups, top, scoring, pair):
    """Rows as in calls of which each warp has one, masked ones among them."""
    T, g = 20011, cuda_gen(E)
    logits = torch.randn(T, E, generator=g, device="cuda") * 1.5
    logits[5::97, :E // 2] = -float("inf")
    bias = torch.randn(E, generator=g, device="cuda") * 0.05
    mask = (torch.rand(T, generator=g, device="cuda") < 0.9).to(torch.uint8)
    r = moe.MoeGroupRouter(
        T, E, k, groups, top, group_score=moe.MOE_GROUP_TOP2 if pair else moe.MOE_GROUP_MAX,
        scoring={"softmax_topk": moe.MOE_ROUTER_SOFTMAX_TOPK, "softmax": moe.MOE_ROUTER_SOFTMAX,
                 "sigmoid": moe.MOE_ROUTER_SIGMOID}[scoring])
    a = r.forward(logits, bias=bias, token_mask=mask)
    counts, total, live = torch.zeros(E + 1, dtype=torch.int64, device="cuda"), 0.0, mask != 0
    for lo in range(0, T, 2000):
        s = slice(lo, min(lo + 2000, T))
        b = r.forward(logits[s], bias=bias, token_mask=mask[s])
        assert torch.equal(a.ids[s][live[s]], b.ids[live[s]]), lo
        assert torch.equal(a.scores[s], b.scores) and torch.equal(a.row_stat[s], b.row_stat), lo
        counts += b.counts
        total = total + b.prob_sum.double()
    assert torch.equal(a.counts.long(), counts)
    # one order of adding some 20000 probabilities against another, each within a rounding a term
    assert bool(((a.prob_sum.double() - total).abs() <= T * 2.0 ** -24 * total).all())
    ids = ref.group_choice(f32(logits[-300:]), k, groups, top, scoring, pair, f32(bias))
    on = live[-300:].cpu().numpy()
    assert np.array_equal(a.ids[-300:].cpu().numpy()[on], ids[on])
