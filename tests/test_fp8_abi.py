"""Host-side argument checks of the 8-bit block operators and the router with groups (CPU
only)."""

import ctypes

import pytest

OK, INVALID, WORKSPACE = 0, 1, 2
A, ODD = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 1)
SHIFTED = ctypes.c_void_p((1 << 20) + 8)


@pytest.fixture(scope="module")
def B():
    from routed_mixture_experts_gb300 import build as b

    b.build()
    from routed_mixture_experts_gb300 import binding

    binding.lib()
    return binding


def test_group_router_checks(B):
    L = B.lib()

    def desc(E=128, k=8, dtype=1, scoring=2, scale=1.0, groups=8, top=4, score=1):
        return B.GroupRouterDesc(B.RouterDesc(E, k, dtype, scoring, scale), groups, top, score)

    good = desc()
    p = ctypes.addressof(good)
    assert L.moe_group_router_workspace_bytes(p, 8192) > 0
    for bad in (dict(E=0), dict(E=257, groups=1, top=1), dict(k=0), dict(scoring=3),
                dict(groups=0), dict(groups=7), dict(groups=256), dict(top=0), dict(top=9),
                dict(score=2), dict(score=-1), dict(k=65), dict(k=33, top=2),
                dict(scale=float("nan"))):
        s = desc(**bad)
        at = ctypes.addressof(s)
        assert L.moe_group_router_workspace_bytes(at, 64) == 0, bad
        assert L.moe_group_router_forward(at, 64, A, 128, None, None, A, A, A, A, A, A, A, 1 << 30,
                                          None) == INVALID, bad
    assert L.moe_group_router_workspace_bytes(None, 64) == 0
    assert L.moe_group_router_workspace_bytes(p, -1) == 0
    assert L.moe_group_router_workspace_bytes(p, 1 << 28) == 0            # T*k = 2^31

    def forward(T=4096, logits=A, ld=128, bias=None, ids=A, scores=A, counts=A, prob=A, losses=A,
                stat=A, ws=A, nbytes=1 << 30, at=p):
        return L.moe_group_router_forward(at, T, logits, ld, bias, None, ids, scores, counts, prob,
                                          losses, stat, ws, nbytes, None)

    for bad in (dict(at=None), dict(T=-1), dict(logits=None), dict(ld=127), dict(ids=None),
                dict(scores=None), dict(counts=None), dict(prob=None), dict(losses=None),
                dict(stat=None), dict(logits=ODD), dict(bias=ODD), dict(ws=ODD)):
        assert forward(**bad) == INVALID, bad
    assert forward(ws=None) == WORKSPACE
    assert forward(nbytes=16) == WORKSPACE
    for bad in ((None, A, 8, 0.1), (A, None, 8, 0.1), (A, A, 0, 0.1), (A, A, 257, 0.1),
                (A, A, 8, float("inf")), (ODD, A, 8, 0.1), (A, ODD, 8, 0.1)):
        assert L.moe_router_update_bias(*bad, None) == INVALID, bad


def test_quantiser_checks(B):
    L = B.lib()

    def call(source=0, C=256, dtype=0, E=1, clamp=0.0, flags=0, M=300, x=A, ld=None, n_src=300,
             dh=None, ld_dh=0, rows=None, offsets=None, codes=A, ld_c=512, scales=A, ld_s=300,
             codes_t=A, ld_t=384, cols=384, scales_t=A, ld_st=512, desc=True):
        d = B.Fp8QuantDesc(source, C, dtype, E, clamp, flags)
        if ld is None:
            ld = C if source == 0 else 2 * C
        return L.moe_fp8_quantize(ctypes.addressof(d) if desc else None, M, x, ld, n_src, dh, ld_dh,
                                  rows, offsets, codes, ld_c, scales, ld_s, codes_t, ld_t, cols,
                                  scales_t, ld_st, None)

    assert call(M=0) == OK
    grad = dict(source=2, dh=A, ld_dh=256)
    assert call(M=0, **grad) == OK
    for bad in (dict(desc=False), dict(source=3), dict(source=-1), dict(C=0), dict(C=(1 << 19) + 1),
                dict(dtype=2), dict(E=0), dict(E=257, offsets=A), dict(E=2), dict(clamp=-1.0),
                dict(clamp=float("nan")), dict(clamp=1.0), dict(flags=2), dict(M=-1),
                dict(x=None), dict(x=ODD), dict(ld=255), dict(rows=ODD), dict(offsets=ODD),
                dict(source=1, rows=A), dict(source=1, ld=511), dict(source=2), dict(dh=A),
                dict(grad, ld_dh=255), dict(grad, dh=ODD), dict(rows=A, n_src=-1),
                dict(codes=None, codes_t=None), dict(codes=SHIFTED), dict(ld_c=255),
                dict(ld_c=520), dict(scales=None), dict(scales=ODD), dict(ld_s=299),
                dict(codes_t=SHIFTED), dict(cols=256), dict(cols=300), dict(ld_t=383),
                dict(ld_t=392), dict(scales_t=None), dict(scales_t=ODD), dict(ld_st=255),
                dict(grad, ld_st=511), dict(grad, ld_c=496), dict(ld=1 << 31)):
        assert call(**bad) == INVALID, bad


def test_weight_quantiser_checks(B):
    L = B.lib()

    def call(w=A, dtype=0, E=2, N=100, K=200, flags=0, codes=A, ld=208, scales=A, codes_t=A,
             ld_t=112, scales_t=A):
        return L.moe_fp8_quantize_weights(w, dtype, E, N, K, flags, codes, ld, scales, codes_t, ld_t,
                                          scales_t, None)

    for bad in (dict(w=None), dict(w=ODD), dict(dtype=2), dict(E=0), dict(E=257), dict(N=0),
                dict(K=0), dict(N=(1 << 20) + 1), dict(K=(1 << 20) + 1), dict(flags=4),
                dict(codes=None, codes_t=None), dict(codes=SHIFTED), dict(ld=199), dict(ld=200),
                dict(scales=None), dict(codes_t=SHIFTED), dict(ld_t=99), dict(ld_t=104),
                dict(scales_t=None), dict(scales=ODD), dict(scales_t=ODD)):
        assert call(**bad) == INVALID, bad


def test_product_checks(B):
    L = B.lib()

    def call(N=100, K=200, E=1, dtype=0, M=50, a=A, ld_a=208, sa=A, ld_sa=50, b=A, ld_b=208, sb=A,
             offsets=None, c=A, ld_c=100, status=A, desc=True):
        d = B.Fp8GemmDesc(N, K, E, dtype)
        return L.moe_fp8_gemm(ctypes.addressof(d) if desc else None, M, a, ld_a, sa, ld_sa, b, ld_b,
                              sb, offsets, c, ld_c, status, None)

    assert call(M=0) == OK
    for bad in (dict(desc=False), dict(N=0), dict(K=0), dict(N=(1 << 20) + 1), dict(E=0),
                dict(E=257, offsets=A), dict(E=2), dict(dtype=2), dict(M=-1), dict(a=None),
                dict(a=SHIFTED), dict(ld_a=199), dict(ld_a=200), dict(sa=None), dict(sa=ODD),
                dict(ld_sa=49), dict(b=None), dict(b=SHIFTED), dict(ld_b=192), dict(ld_b=204),
                dict(sb=None), dict(sb=ODD), dict(offsets=ODD), dict(c=None), dict(c=ODD),
                dict(ld_c=99), dict(status=None), dict(status=SHIFTED),
                dict(N=1 << 20, K=1 << 20, ld_a=1 << 20, ld_b=1 << 20, ld_c=1 << 20)):
        assert call(**bad) == INVALID, bad

    def wgrad(N=100, K=200, E=1, dtype=1, R=256, dy=A, ld_y=256, sy=A, ld_sy=100, x=A, ld_x=256,
              sx=A, ld_sx=200, offsets=None, dw=A, acc=0, status=A, desc=True):
        d = B.Fp8GemmDesc(N, K, E, dtype)
        return L.moe_fp8_gemm_wgrad(ctypes.addressof(d) if desc else None, R, dy, ld_y, sy, ld_sy, x,
                                    ld_x, sx, ld_sx, offsets, dw, acc, status, None)

    assert wgrad(R=0, acc=1) == OK
    for bad in (dict(desc=False), dict(N=0), dict(E=0), dict(E=2), dict(dtype=-1), dict(R=-128),
                dict(R=200), dict(R=1 << 31), dict(dy=None), dict(dy=SHIFTED), dict(ld_y=240),
                dict(ld_y=264), dict(sy=None), dict(sy=ODD), dict(ld_sy=99), dict(x=None),
                dict(x=SHIFTED), dict(ld_x=128), dict(sx=None), dict(sx=ODD), dict(ld_sx=199),
                dict(offsets=ODD), dict(dw=None), dict(dw=ODD), dict(status=None),
                dict(status=SHIFTED)):
        assert wgrad(**bad) == INVALID, bad
    assert L.moe_fp8_check(None, None) == INVALID


# ---- the Python calls, without a GPU -------------------------------------------------


class OnGpu:
    """What the binding looks at of a tensor on GPU `dev` (no GPU needed)."""

    def __init__(self, dtype, shape, dev=0, strides=None):
        self.dtype, self.shape, self.dev = dtype, tuple(shape), dev
        self.device = "cuda:%d" % dev
        dense = []
        for n in reversed(self.shape):
            dense.insert(0, dense[0] * self.shape[len(self.shape) - len(dense)] if dense else 1)
        self.dense = tuple(dense)
        self.strides = strides or self.dense

    def get_device(self):
        return self.dev

    def is_contiguous(self):
        return self.strides == self.dense

    def stride(self):
        return self.strides

    def dim(self):
        return len(self.shape)

    def data_ptr(self):
        return 1 << 20


@pytest.fixture
def on_gpu_0(B, monkeypatch):
    """The binding with GPU 0 current and a library that only counts its calls."""
    import torch

    class Library:
        calls = 0

        def moe_status_string(self, code):
            return b"status"

        def __getattr__(self, name):
            def call(*args):
                self.calls += 1
                return OK

            return call

    library = Library()
    monkeypatch.setattr(B, "_lib", library)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    return library


def refused(B, library, call, tensors, bad):
    """`call` is made with `tensors`, and refused with any of `bad` in the place of one."""
    call({n: OnGpu(*t) for n, t in tensors.items()})
    before = library.calls
    assert before > 0
    for name, t in bad:
        with pytest.raises(B.MoeError) as e:
            call({**{n: OnGpu(*v) for n, v in tensors.items()}, name: t})
        assert e.value.code == INVALID, (name, t.shape, t.strides)
    assert library.calls == before


def test_python_calls_refuse(B, on_gpu_0):
    import torch

    f8, f32, bf16, i32 = torch.float8_e4m3fn, torch.float32, torch.bfloat16, torch.int32
    M, N, K, E = 40, 48, 256, 3
    tensors = dict(x=(bf16, (M, K)), offsets=(i32, (E + 1,)), codes=(f8, (M, K)),
                   scales=(f32, (2, M)), codes_t=(f8, (K, 512)), scales_t=(f32, (4, K)))
    bad = [(n, OnGpu(t, s, dev=1)) for n, (t, s) in tensors.items()]
    bad += [("x", OnGpu(torch.float16, (M, K))), ("x", OnGpu(bf16, (M, K), strides=(K - 1, 1))),
            ("x", OnGpu(bf16, (M, K, 1))), ("codes", OnGpu(torch.uint8, (M, K))),
            ("codes", OnGpu(f8, (M, K), strides=(K + 8, 1))),
            ("codes", OnGpu(f8, (M, K), strides=(2 * K, 2))), ("codes", OnGpu(f8, (M, K - 1))),
            ("scales", OnGpu(f32, (M, 2))), ("scales", OnGpu(f32, (1, M))),
            ("codes_t", OnGpu(f8, (K - 1, 512))), ("scales_t", OnGpu(f32, (3, K))),
            ("offsets", OnGpu(torch.int64, (E + 1,)))]
    refused(B, on_gpu_0, lambda t: B.quantize_fp8(
        t["x"], offsets=t["offsets"], by_column=True, out=(t["codes"], t["scales"]),
        out_t=(t["codes_t"], t["scales_t"])), tensors, bad)
    for by_row, by_column, out, out_t in ((False, False, None, None), (False, True, 1, None),
                                          (True, False, None, 1)):
        with pytest.raises(B.MoeError):
            B.quantize_fp8(OnGpu(bf16, (M, K)), by_row=by_row, by_column=by_column, out=out,
                           out_t=out_t)
    refused(B, on_gpu_0, lambda t: B.quantize_fp8(
        OnGpu(bf16, (M, K)), rows=t["rows"], out=(OnGpu(f8, (9, K)), OnGpu(f32, (2, 9)))),
        dict(rows=(i32, (9,))), [("rows", OnGpu(i32, (9,), dev=1)),
                                 ("rows", OnGpu(torch.int64, (9,)))])

    h = object.__new__(B.MoeFp8Linear)
    h.N, h.K, h.E, h.dtype = N, K, E, bf16
    h._ahead, h._back = h._side(N, K, E, 0), h._side(K, N, E, 0)

    def forward(t):
        h.status = t["status"]
        h.forward((t["codes"], t["scales"]), (t["w"], t["ws"]), offsets=t["offsets"], out=t["out"])

    tensors = dict(status=(i32, (4,)), codes=(f8, (M, K)), scales=(f32, (2, M)),
                   w=(f8, (E, N, K)), ws=(f32, (E, 1, 2)), offsets=(i32, (E + 1,)),
                   out=(bf16, (M, N)))
    bad = [(n, OnGpu(t, s, dev=1)) for n, (t, s) in tensors.items()]
    bad += [("codes", OnGpu(f8, (M, K + 16))), ("scales", OnGpu(f32, (3, M))),
            ("w", OnGpu(f8, (E, K, N))), ("w", OnGpu(f8, (E, N, K), strides=(N * K + 16, K, 1))),
            ("ws", OnGpu(f32, (E, 2, 1))), ("offsets", OnGpu(i32, (E,))),
            ("out", OnGpu(f32, (M, N))), ("out", OnGpu(bf16, (M, N + 1)))]
    refused(B, on_gpu_0, forward, tensors, bad)
    with pytest.raises(B.MoeError):            # experts without offsets
        forward({**{n: OnGpu(*t) for n, t in tensors.items()}, "offsets": None})

    def weight(t):
        h.status = t["status"]
        h.grad_weight((t["dy"], t["sy"]), (t["x"], t["sx"]), offsets=t["offsets"], dw=t["dw"])

    tensors = dict(status=(i32, (4,)), dy=(f8, (N, 512)), sy=(f32, (4, N)), x=(f8, (K, 512)),
                   sx=(f32, (4, K)), offsets=(i32, (E + 1,)), dw=(f32, (E, N, K)))
    bad = [(n, OnGpu(t, s, dev=1)) for n, (t, s) in tensors.items()]
    bad += [("dy", OnGpu(f8, (N, 384))), ("sy", OnGpu(f32, (3, N))), ("dw", OnGpu(bf16, (E, N, K))),
            ("dw", OnGpu(f32, (E, K, N)))]
    refused(B, on_gpu_0, weight, tensors, bad)
    for bad in ((0, 8, 1), (8, 0, 1), (8, 8, 0), (8, 8, 257), ((1 << 20) + 1, 8, 1)):
        with pytest.raises(B.MoeError):
            B.MoeFp8Linear(*bad, device="meta")


def test_group_router_is_refused(B):
    for bad in ((64, 128, 8, 7, 2), (64, 128, 8, 8, 9), (64, 128, 8, 8, 0), (64, 128, 33, 8, 2)):
        with pytest.raises(B.MoeError):
            B.MoeGroupRouter(*bad, device="meta")


def test_columns_hold_any_segments(B):
    for M, E in ((1, 1), (300, 4), (0, 3), (129, 256)):
        R = B.fp8_columns(M, E)
        worst = min(M, E)                      # every expert's last block with one row
        rows = M - (worst - 1) if worst else 0
        used = (worst - 1) * 128 + (rows + 127) // 128 * 128 if worst else 0
        assert R % 128 == 0 and R >= used
    assert B.fp8_columns(129, 1, offsets=False) == 256


def test_product_of_rows_that_32_bits_cannot_round_up(B):
    """The last 127 row counts below 2^31, whose blocks of 128 would be counted beyond it."""
    L = B.lib()
    d = B.Fp8GemmDesc(16, 16, 1, 0)
    for M in (0x7FFFFF81, 0x7FFFFFFF):
        assert L.moe_fp8_gemm(ctypes.addressof(d), M, A, 16, A, M, A, 16, A, None, A, 16, A,
                              None) == INVALID


def test_descriptions_outlive_their_calls(B, on_gpu_0, monkeypatch):
    """A call's description stays while the library has its address, whatever other threads'
    calls bring into the table of descriptions meanwhile."""
    import gc
    import weakref

    import torch

    made = []

    class Desc(B.Fp8QuantDesc):
        def __init__(self, *values):
            super().__init__(*values)
            made.append(weakref.ref(self))

    monkeypatch.setattr(B, "Fp8QuantDesc", Desc)
    B._quant_desc.cache_clear()

    def quantize(at, *rest):
        (desc,) = [d for d in (r() for r in made) if d is not None and ctypes.addressof(d) == at]
        del desc
        for C in range(1000, 1400):                # as many as the table holds, and more
            B._quant_desc(0, C, 0, 1, 0.0, 0)
        gc.collect()
        assert any(d is not None and ctypes.addressof(d) == at for d in (r() for r in made[:1]))
        seen.append(at)
        return OK

    seen = []
    on_gpu_0.moe_fp8_quantize = quantize
    bf16, f8, f32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32
    B.quantize_fp8(OnGpu(bf16, (8, 256)), out=(OnGpu(f8, (8, 256)), OnGpu(f32, (2, 8))))
    assert seen
    B._quant_desc.cache_clear()


def test_no_rows_are_no_mistake(B):
    """Codes of no rows have no address; the other checks hold for them too."""
    L = B.lib()

    def call(source, M=0, E=1, C=64, offsets=None):
        d = B.Fp8QuantDesc(source, C, 0, E, 0.0, 0)
        return L.moe_fp8_quantize(ctypes.addressof(d), M, None, 2 * C, 0, None, C, None, offsets,
                                  None, 2 * C, None, M, None, 0, 0, None, 0, None)

    for source in (0, 1, 2):
        assert call(source) == OK and call(source, E=3, offsets=A) == OK
        assert call(source, M=1) == INVALID
        assert call(source, E=3) == INVALID and call(source, C=0) == INVALID


def test_shapes_are_refused_as_such(B, on_gpu_0):
    """Tensors of too few dimensions, offsets of no expert, a status of another GPU: errors of
    this library, before anything is called."""
    import torch

    f8, f32, bf16, i32 = torch.float8_e4m3fn, torch.float32, torch.bfloat16, torch.int32
    x, codes, scales = OnGpu(bf16, (8, 256)), OnGpu(f8, (8, 256)), OnGpu(f32, (2, 8))
    wide, out_t = OnGpu(bf16, (8, 512)), (OnGpu(f8, (256, 128)), OnGpu(f32, (1, 256)))
    bad = [lambda: B.quantize_fp8(OnGpu(bf16, (256,)), out=(codes, scales)),
           lambda: B.quantize_fp8(OnGpu(bf16, ()), out=(codes, scales)),
           lambda: B.quantize_fp8(x, rows=OnGpu(i32, ()), out=(codes, scales)),
           lambda: B.quantize_fp8(x, offsets=OnGpu(i32, (0,)), out=(codes, scales)),
           lambda: B.quantize_fp8(x, offsets=OnGpu(i32, (1,)), by_column=True, out=(codes, scales),
                                  out_t=out_t),
           lambda: B.quantize_fp8(x, by_row=False, by_column=True, out_t=(OnGpu(f8, ()), scales)),
           lambda: B.swiglu_fp8(OnGpu(bf16, (512,)), out=(codes, scales)),
           lambda: B.swiglu_grad_fp8(x, OnGpu(bf16, (512,)), out=(codes, scales)),
           lambda: B.swiglu_grad_fp8(OnGpu(bf16, ()), wide, out=(codes, scales)),
           lambda: B.quantize_fp8_weights(OnGpu(bf16, (256,))),
           lambda: B.quantize_fp8_weights(OnGpu(bf16, (2, 3, 4, 5)))]
    h = object.__new__(B.MoeFp8Linear)
    h.N, h.K, h.E, h.dtype, h.status = 48, 256, 1, bf16, OnGpu(i32, (4,))
    h._ahead, h._back = h._side(48, 256, 1, 0), h._side(256, 48, 1, 0)
    w = (OnGpu(f8, (1, 48, 256)), OnGpu(f32, (1, 1, 2)))
    y = OnGpu(bf16, (8, 48))
    bad += [lambda: h.forward((OnGpu(f8, ()), scales), w, out=y),
            lambda: h.forward((codes, scales), (OnGpu(f8, (48,)), w[1]), out=y),
            lambda: h.forward((codes, scales), w, offsets=OnGpu(i32, ()), out=y),
            lambda: h.grad_weight((OnGpu(f8, ()), scales), (OnGpu(f8, ()), scales))]
    before = on_gpu_0.calls
    for i, call in enumerate(bad):
        with pytest.raises(B.MoeError) as e:
            call()
        assert e.value.code == INVALID, i
    h.status = OnGpu(i32, (4,), dev=1)
    with pytest.raises(B.MoeError):
        h.check()
    assert on_gpu_0.calls == before
