"""The block norms (forward and gradient) against a 64-bit implementation, at the
widths, lengths, types, strides and gates where they can go wrong."""

import numpy as np
import pytest
import torch

import operator_refs as ref

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
TYPES = {"bf16": (BF, BF), "mixed": (BF, F), "fp32": (F, F)}


@pytest.fixture(scope="module")
def moe():
    from routed_mixture_experts_gb300 import build

    build.build()
    import routed_mixture_experts_gb300 as m

    return m


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def check(got, want, what, mag=None):
    ref.check(np64(got), want, what, mag, bf16=got.dtype == BF)


def strided(t, extra):
    """The same values with rows `extra` elements further apart."""
    if not extra:
        return t
    wide = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), dtype=t.dtype,
                      device=t.device)
    wide[:, : t.shape[1]] = t
    return wide[:, : t.shape[1]]


class Case:
    def __init__(self, moe, T, d, types="bf16", gate="channel", post=True, pre=True, y=True,
                 alpha=0.5, params=F, extra=0, seed=3):
        act, res = TYPES[types]
        g = torch.Generator().manual_seed(seed)
        n = lambda *s: torch.randn(*s, generator=g)
        self.kind = gate
        big = 1.0 + 20.0 * (torch.rand(d, generator=g) < 0.01)
        cu = lambda t, dt: None if t is None else t.to(dt).cuda()
        self.res = strided(cu(n(T, d) * big, res), extra)
        self.y = strided(cu(n(T, d) * 0.3, act), extra) if y else None
        self.w_post = cu(1 + 0.1 * n(d), params) if post and y else None
        self.w_pre = cu(1 + 0.1 * n(d), params) if pre else None
        self.gate = None
        if y and gate == "channel":
            self.gate = cu(0.5 + 0.2 * n(d), params)
        elif y and gate == "token":
            self.gate = cu(torch.rand(T, generator=g), params)
        self.d_out = strided(cu(n(T, d), res), extra)
        self.d_u = strided(cu(n(T, d), act), extra) if pre else None
        self.alpha = alpha
        self.h = moe.MoeBlockNorm(
            max(T, 1), d, dtype=act, residual_dtype=res, param_dtype=params, alpha=alpha,
            gate={"none": moe.MOE_GATE_NONE, "channel": moe.MOE_GATE_CHANNEL,
                  "token": moe.MOE_GATE_TOKEN}[gate])

    def np_gate(self):
        g = np64(self.gate)
        return g[:, None] if g is not None and self.kind == "token" else g

    def params(self):
        return dict(y=self.y, w_post=self.w_post, gate=self.gate, w_pre=self.w_pre)

    def np_params(self):
        return dict(y=np64(self.y), w_post=np64(self.w_post), gate=self.np_gate(),
                    w_pre=np64(self.w_pre), alpha=self.alpha)

    def check_forward(self):
        out, u = self.h.forward(self.res, **self.params())
        wo, wu = ref.block_norm_forward(np64(self.res), **self.np_params())
        check(out, wo, "out")
        if wu is None:
            assert u is None
        else:
            check(u, wu, "u")

    def check_backward(self):
        got = self.h.backward(self.res, self.d_out, self.d_u, **self.params())
        want, mag = ref.block_norm_backward(np64(self.res), d_out=np64(self.d_out),
                                            d_u=np64(self.d_u), **self.np_params())
        check(got.d_residual, want["d_residual"], "d_residual", mag["d_residual"])
        for name in ("dy", "dw_post", "dw_pre"):
            assert (getattr(got, name) is not None) == (name in want), name
            if name in want:
                check(getattr(got, name), want[name], name, mag[name])
        if self.gate is not None:
            over = 1 if self.kind == "token" else 0
            check(got.dgate, want["dgate_full"].sum(over), "dgate", mag["dgate_full"].sum(over))
        return got


SHAPES = [(1, 2048), (3, 1), (5, 7), (2, 8), (33, 64), (17, 100), (300, 1537), (7, 2056),
          (640, 2048), (1300, 256), (4, 8192), (9, 8200), (3, 16384), (2, 16383)]


@pytest.mark.parametrize("types", list(TYPES))
@pytest.mark.parametrize("T,d", SHAPES)
def test_forward_and_gradient(moe, T, d, types):
    c = Case(moe, T, d, types, gate="token" if d % 2 else "channel")
    c.check_forward()
    c.check_backward()


@pytest.mark.parametrize("types", list(TYPES))
@pytest.mark.parametrize("T,d,extra", [(700, 1537, 0), (1300, 77, 0), (5000, 9, 2), (650, 4095, 0),
                                       (700, 2048, 3), (620, 5001, 1), (700, 250, 0)])
def test_many_unaligned_rows(moe, T, d, extra, types):
    c = Case(moe, T, d, types, gate="token" if d % 2 else "channel", extra=extra)
    c.check_forward()
    c.check_backward()


@pytest.mark.parametrize("types", list(TYPES))
@pytest.mark.parametrize("T,d", [(700, 1537), (700, 2048), (3, 513), (640, 4097), (620, 8191)])
def test_tensors_that_begin_between_16_byte_boundaries(moe, T, d, types):
    c = Case(moe, T, d, types)

    def moved(t):
        wide = torch.full((t.numel() + 1,), float("nan"), dtype=t.dtype, device=t.device)
        wide[1:] = t.reshape(-1)
        return wide[1:].view(t.shape)

    for name in ("res", "y", "d_out", "d_u", "w_post", "w_pre", "gate"):
        whole = getattr(c, name)
        setattr(c, name, moved(whole))
        c.check_forward()
        c.check_backward()
        setattr(c, name, whole)
    c.res, c.y, c.d_out, c.d_u = moved(c.res), moved(c.y), moved(c.d_out), moved(c.d_u)
    c.check_forward()
    c.check_backward()


@pytest.mark.parametrize("parts", [
    dict(y=False, gate="none"), dict(pre=False), dict(post=False), dict(post=False, pre=False),
    dict(gate="none"), dict(gate="token"), dict(post=False, gate="token"),
    dict(gate="token", pre=False), dict(params=BF), dict(params=BF, gate="token"),
    dict(alpha=0.0), dict(extra=8), dict(extra=3), dict(extra=1, types="mixed")],
    ids=lambda p: ",".join("%s=%s" % kv for kv in p.items()))
@pytest.mark.parametrize("d", [2048, 513])
def test_parts_types_and_strides(moe, d, parts):
    c = Case(moe, 77, d, **parts)
    if c.y is not None or c.w_pre is not None:
        c.check_forward()
        c.check_backward()


def test_rows_of_zeros_and_of_one_value(moe):
    c = Case(moe, 4, 512, "fp32")
    c.res[0] = 0
    c.y[0] = 0
    c.y[1] = 0
    c.res[2] = 5.0
    c.y[2] = -2.0
    c.check_forward()
    c.check_backward()


def test_a_row_of_nan_stays_in_its_row(moe):
    c = Case(moe, 6, 256, "bf16")
    clean = c.h.forward(c.res, **c.params())
    c.y[3] = float("nan")
    out, u = c.h.forward(c.res, **c.params())
    keep = [0, 1, 2, 4, 5]
    assert torch.equal(out[keep], clean[0][keep]) and torch.equal(u[keep], clean[1][keep])
    assert out[3].isnan().all() and u[3].isnan().all()


@pytest.mark.parametrize("types", list(TYPES))
def test_in_place(moe, types):
    c = Case(moe, 50, 1024, types)
    out, u = c.h.forward(c.res, **c.params())
    g = c.h.backward(c.res, c.d_out, c.d_u, **c.params())
    res, y = c.res.clone(), c.y.clone()
    o2, u2 = c.h.forward(res, y=y, w_post=c.w_post, gate=c.gate, w_pre=c.w_pre, residual_out=res,
                         u=y)
    assert o2.data_ptr() == res.data_ptr() and torch.equal(res, out) and torch.equal(y, u)
    d_out, d_u = c.d_out.clone(), c.d_u.clone()
    c.h.backward(c.res, d_out, d_u, **c.params(), d_residual=d_out, dy=d_u)
    assert torch.equal(d_out, g.d_residual) and torch.equal(d_u, g.dy)


def test_no_upstream_gradient(moe):
    c = Case(moe, 40, 256)
    c.d_out = None
    got = c.h.backward(c.res, None, c.d_u, **c.params())
    want, mag = ref.block_norm_backward(np64(c.res), d_u=np64(c.d_u), **c.np_params())
    for name in ("d_residual", "dy"):
        check(getattr(got, name), want[name], name, mag[name])


def test_accumulate_and_repeat(moe):
    c = Case(moe, 700, 1000, "mixed")
    a = c.check_backward()
    b = c.check_backward()
    for x, y in zip(a, b):
        assert torch.equal(x, y)                       # the same bits
    before = {n: torch.randn_like(getattr(a, n)) for n in ("dw_post", "dw_pre", "dgate")}
    mine = {n: t.clone() for n, t in before.items()}
    c.h.backward(c.res, c.d_out, c.d_u, **c.params(), accumulate=True, **mine)
    for n in mine:
        assert torch.equal(mine[n], before[n] + getattr(a, n)), n


def test_no_rows(moe):
    c = Case(moe, 0, 256)
    out, u = c.h.forward(c.res, **c.params())
    assert out.shape == (0, 256) and u.shape == (0, 256)
    g = c.h.backward(c.res, c.d_out, c.d_u, **c.params())
    for t in (g.dw_post, g.dw_pre, g.dgate):
        assert torch.equal(t, torch.zeros_like(t))
    ones = torch.ones(256, device="cuda")
    c.h.backward(c.res, c.d_out, c.d_u, **c.params(), dw_post=ones, accumulate=True)
    assert torch.equal(ones, torch.ones_like(ones))


def test_gradient_against_differences(moe):
    """Central differences of the 64-bit forward along random directions."""
    c = Case(moe, 12, 96, "fp32", gate="token")
    p = c.np_params()
    base = np64(c.res)                                  # the stream before the block here
    out, _ = ref.block_norm_forward(base, **p)
    x = torch.tensor(out, dtype=F, device="cuda")
    got = c.h.backward(x, c.d_out, c.d_u, **c.params())
    do, du = np64(c.d_out), np64(c.d_u)

    def loss(res=base, **change):
        o, u = ref.block_norm_forward(res, **{**p, **change})
        return np.sum(o * do) + np.sum(u * du)

    rng = np.random.default_rng(5)
    h = 1e-5
    for name, grad, at in [("res", got.d_residual, base), ("y", got.dy, p["y"]),
                           ("w_post", got.dw_post, p["w_post"]), ("w_pre", got.dw_pre, p["w_pre"]),
                           ("gate", got.dgate, p["gate"])]:
        v = rng.standard_normal(at.shape)
        slope = (loss(**{name: at + h * v}) - loss(**{name: at - h * v})) / (2 * h)
        mine = np.sum(np64(grad).reshape(at.shape) * v)
        # differences: h^2 truncation and 2^-53/h rounding of a sum of ~1e3 terms of
        # size ~10; the kernel: fp32 (x rounded, and its own arithmetic)
        size = np.linalg.norm(np64(grad)) * np.linalg.norm(v)
        assert abs(slope - mine) <= 1e-6 * size + 1e-6, name


def test_rows_further_apart_than_32_bits_reach(moe):
    """Three rows of every tensor 2^30 + 8 elements apart: offsets beyond 2^31."""
    c = Case(moe, 3, 256, "bf16")
    want = c.h.forward(c.res, **c.params())
    g = c.h.backward(c.res, c.d_out, c.d_u, **c.params())
    apart = 2 ** 30 + 8
    pool = torch.empty(2 * apart + 4096, dtype=BF, device="cuda")
    at = 0

    def spread(t=None):
        nonlocal at
        v = pool.as_strided((3, 256), (apart, 1), at)
        at += 256
        if t is not None:
            v.copy_(t)
        return v

    res, y, d_out, d_u = (spread(t) for t in (c.res, c.y, c.d_out, c.d_u))
    p = dict(y=y, w_post=c.w_post, gate=c.gate, w_pre=c.w_pre)
    out, u = c.h.forward(res, **p, residual_out=spread(), u=spread())
    assert torch.equal(out, want[0]) and torch.equal(u, want[1])
    b = c.h.backward(res, d_out, d_u, **p, d_residual=spread(), dy=spread())
    for x, z in zip(b, g):
        assert torch.equal(x, z)


def test_another_stream(moe):
    c = Case(moe, 512, 2048)
    want = c.h.forward(c.res, **c.params())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = c.y * 1.0                                   # made on the side stream
        got = c.h.forward(c.res, y=y, w_post=c.w_post, gate=c.gate, w_pre=c.w_pre)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_outputs_belong_to_the_given_stream(moe):
    """Memory that the current stream has yet to write is not handed to another one."""
    c = Case(moe, 64, 2048)
    want = c.h.forward(c.res, **c.params())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    busy = [torch.empty_like(t) for t in want for _ in range(2)]
    torch.cuda._sleep(100_000_000)                      # some 50 ms
    for t in busy:
        t.fill_(77)
    del t, busy
    got = c.h.forward(c.res, stream=s, **c.params())
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_refusals(moe):
    with pytest.raises(moe.MoeError):
        moe.MoeBlockNorm(4, 16385)
    with pytest.raises(moe.MoeError):
        moe.MoeBlockNorm(4, 64, dtype=torch.float16)
    with pytest.raises(moe.MoeError):
        moe.MoeBlockNorm(4, 64, dtype=F, residual_dtype=BF)
    c = Case(moe, 8, 64)
    for bad in (dict(y=c.y.float()), dict(y=c.y[:7]), dict(y=c.y.t().contiguous().t()),
                dict(w_post=c.w_post.to(BF)), dict(gate=c.gate[:5]), dict(gate=None),
                dict(w_pre=c.w_pre.cpu()), dict(y=None)):
        with pytest.raises(moe.MoeError) as e:
            c.h.forward(c.res, **{**c.params(), **bad})
        assert e.value.code == moe.MOE_ERR_INVALID_ARG
    with pytest.raises(moe.MoeError):
        c.h.backward(torch.cat([c.res, c.res]), None, None, y=torch.cat([c.y, c.y]),
                     gate=c.gate)                       # more rows than it was made for


@pytest.mark.parametrize("d", [512, 777, 5120, 9216])
def test_gradient_of_very_large_rows(moe, d):
    """rms(x)^-3 is below fp32's range, the gradient is not."""
    c = Case(moe, 6, d, "fp32")
    c.res[2:4] *= 1e15
    c.d_out[2:4] *= 1e-15                # else it hides what comes through the norm
    c.y[3:5] *= 1e15
    c.check_forward()
    c.check_backward()


@pytest.mark.parametrize("d", [512, 777, 5120, 9216])
def test_gradient_of_rows_of_zeros_with_a_tiny_eps(moe, d):
    """rms^-3 of a row of zeros is above fp32's range, the gradient is not."""
    c = Case(moe, 5, d, "fp32")
    c.res[1] = 0
    c.y[1:3] = 0
    h = moe.MoeBlockNorm(5, d, dtype=F, gate=moe.MOE_GATE_CHANNEL, alpha=c.alpha, eps=1e-30)
    got = h.backward(c.res, c.d_out, c.d_u, **c.params())
    want, mag = ref.block_norm_backward(np64(c.res), d_out=np64(c.d_out), d_u=np64(c.d_u),
                                        eps=1e-30, **c.np_params())
    for name in ("d_residual", "dy", "dw_post", "dw_pre"):
        check(getattr(got, name), want[name], name, mag[name])
    check(got.dgate, want["dgate_full"].sum(0), "dgate", mag["dgate_full"].sum(0))


def test_outputs_without_their_inputs_are_refused(moe):
    """A tensor that the call would leave unwritten."""
    c = Case(moe, 8, 64)
    buf = torch.empty_like(c.res)
    for call in (lambda: c.h.forward(c.res, w_pre=c.w_pre, residual_out=buf),
                 lambda: c.h.forward(c.res, y=c.y, gate=c.gate, w_post=c.w_post, u=buf)):
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.code == moe.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("types", list(TYPES))
@pytest.mark.parametrize("T,d,extra", [(700, 2048, 0), (700, 1537, 0), (640, 4095, 0),
                                       (620, 5001, 1), (300, 8192, 0), (200, 9216, 0),
                                       (200, 9001, 0), (200, 16384, 0), (700, 250, 3)])
def test_in_place_at_every_layout(moe, T, d, extra, types):
    """Aligned and unaligned rows of every kernel, each read before it is overwritten."""
    c = Case(moe, T, d, types, gate="token" if d % 2 else "channel", extra=extra)
    p = c.params()
    out, u = c.h.forward(c.res, **p)
    g = c.h.backward(c.res, c.d_out, c.d_u, **p)
    copy = lambda t: strided(t.clone(), extra)
    for _ in range(3):
        res, y = copy(c.res), copy(c.y)
        c.h.forward(res, **{**p, "y": y}, residual_out=res, u=y)
        assert torch.equal(res, out) and torch.equal(y, u)
        d_out, d_u = copy(c.d_out), copy(c.d_u)
        b = c.h.backward(c.res, d_out, d_u, **p, d_residual=d_out, dy=d_u)
        for got, want in zip(b, g):
            assert torch.equal(got, want)
