"""Host-side argument checks of the router and block-norm entry points (CPU only)."""

import ctypes

import pytest

OK, INVALID, WORKSPACE = 0, 1, 2
A, ODD = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 1)


@pytest.fixture(scope="module")
def B():
    from routed_mixture_experts_gb300 import build as b

    b.build()
    from routed_mixture_experts_gb300 import binding

    binding.lib()
    return binding


def test_router_checks(B):
    L = B.lib()
    good = B.RouterDesc(128, 8, 1, 0, 1.0)
    p = ctypes.addressof(good)
    assert L.moe_router_workspace_bytes(p, 8192) > 0
    for bad in [(0, 1, 1, 0, 1.0), (257, 1, 1, 0, 1.0), (8, 9, 1, 0, 1.0), (8, 0, 1, 0, 1.0),
                (8, 2, 2, 0, 1.0), (8, 2, 1, 3, 1.0), (8, 2, 1, 0, float("inf"))]:
        s = B.RouterDesc(*bad)
        assert L.moe_router_workspace_bytes(ctypes.addressof(s), 64) == 0, bad
    assert L.moe_router_workspace_bytes(None, 64) == 0
    assert L.moe_router_workspace_bytes(p, -1) == 0
    assert L.moe_router_workspace_bytes(p, 1 << 28) == 0                   # T*k = 2^31

    def forward(T=4096, logits=A, ld=128, ids=A, scores=A, counts=A, prob=A, losses=A, stat=A,
                ws=A, nbytes=1 << 30, desc=p):
        return L.moe_router_forward(desc, T, logits, ld, None, None, ids, scores, counts, prob,
                                    losses, stat, ws, nbytes, None)

    for bad in (dict(desc=None), dict(T=-1), dict(logits=None), dict(ld=127), dict(ids=None),
                dict(scores=None), dict(counts=None), dict(prob=None), dict(losses=None),
                dict(stat=None), dict(logits=ODD), dict(ids=ODD), dict(ws=ODD)):
        assert forward(**bad) == INVALID, bad
    assert forward(ws=None) == WORKSPACE
    assert forward(nbytes=16) == WORKSPACE

    def backward(T=64, logits=A, ld=128, ids=A, counts=A, stat=A, ds=A, dl=A, out=A, ld_d=128):
        return L.moe_router_backward(p, T, logits, ld, ids, counts, stat, ds, dl, out, ld_d, None)

    for bad in (dict(T=-1), dict(logits=None), dict(ld=1), dict(ids=None), dict(counts=None),
                dict(stat=None), dict(out=None), dict(ld_d=127), dict(out=ODD), dict(ds=ODD)):
        assert backward(**bad) == INVALID, bad
    assert backward(T=0) == OK


def test_block_norm_checks(B):
    L = B.lib()

    def desc(d=2048, dtype=0, res=0, param=1, gate=1, alpha=1.0, eps=1e-6):
        return B.BlockNormDesc(d, dtype, res, param, gate, alpha, eps)

    for bad in (dict(d=0), dict(d=16385), dict(dtype=2), dict(res=-1), dict(param=2),
                dict(gate=3), dict(eps=-1.0), dict(eps=float("nan")), dict(dtype=1, res=0)):
        s = desc(**bad)
        assert L.moe_block_norm_workspace_bytes(ctypes.addressof(s), 64) == 0, bad
    s = desc()
    p = ctypes.addressof(s)
    assert L.moe_block_norm_workspace_bytes(p, 64) > 0
    assert L.moe_block_norm_workspace_bytes(p, -1) == 0

    def forward(T=64, res=A, ldr=2048, y=A, ldy=2048, wp=A, gate=A, wq=A, out=A, ldo=2048, u=A,
                ldu=2048):
        return L.moe_block_norm_forward(p, T, res, ldr, y, ldy, wp, gate, wq, out, ldo, u, ldu,
                                        None)

    for bad in (dict(T=-1), dict(res=None), dict(ldr=2047), dict(y=None), dict(ldy=1),
                dict(gate=None), dict(wq=None), dict(out=None), dict(u=None), dict(ldu=7),
                dict(res=ODD), dict(y=ODD), dict(u=ODD), dict(wp=ODD), dict(gate=ODD)):
        assert forward(**bad) == INVALID, bad
    assert forward(T=0) == OK

    def backward(T=640, x=A, ldx=2048, y=A, ldy=2048, do=A, lddo=2048, du=A, lddu=2048, wp=A,
                 gate=A, wq=A, dr=A, lddr=2048, dy=A, lddy=2048, dwp=A, dg=A, dwq=A, acc=0, ws=A,
                 nbytes=1 << 30):
        return L.moe_block_norm_backward(p, T, x, ldx, y, ldy, do, lddo, du, lddu, wp, gate, wq,
                                         dr, lddr, dy, lddy, dwp, dg, dwq, acc, ws, nbytes, None)

    for bad in (dict(T=-1), dict(x=None), dict(y=None), dict(gate=None), dict(wq=None),
                dict(wp=None), dict(dr=None), dict(du=None), dict(ldx=1), dict(lddo=1),
                dict(lddu=1), dict(lddr=1), dict(lddy=1), dict(dwp=ODD), dict(dg=ODD),
                dict(dwq=ODD), dict(do=ODD), dict(ws=ODD)):
        assert backward(**bad) == INVALID, bad
    assert backward(ws=None) == WORKSPACE
    assert backward(nbytes=64) == WORKSPACE
    assert backward(T=0, acc=1) == OK


def test_row_counts_near_the_limit_of_an_int(B):
    """The largest accepted T: a full grid's scratch, as from a few thousand rows on."""
    L = B.lib()
    most = 2 ** 31 - 1
    r = B.RouterDesc(16, 1, 1, 0, 1.0)
    p = ctypes.addressof(r)
    full = L.moe_router_workspace_bytes(p, 1 << 20)
    for T in (most, most - 30, most - 31):
        assert L.moe_router_workspace_bytes(p, T) == full, T
    for d in (1, 2048, 16384):
        s = B.BlockNormDesc(d, 0, 0, 1, 1, 1.0, 1e-6)
        p = ctypes.addressof(s)
        full = L.moe_block_norm_workspace_bytes(p, 1 << 20)
        for T in (most, most - 15):
            assert L.moe_block_norm_workspace_bytes(p, T) == full, (d, T)


class OnGpu:
    """What the binding looks at of a tensor on GPU `dev` (no GPU needed)."""

    is_cuda = True

    def __init__(self, dtype, shape, dev=0):
        self.dtype, self.shape, self.dev = dtype, shape, dev
        self.device = "cuda:%d" % dev

    def get_device(self):
        return self.dev

    def is_contiguous(self):
        return True

    def stride(self):
        return (self.shape[-1], 1)

    def data_ptr(self):
        return 1 << 20

    @property
    def nbytes(self):
        n = self.dtype.itemsize
        for s in self.shape:
            n *= s
        return n


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


def only_one_elsewhere(B, library, call, tensors):
    """`call` is made with all tensors on GPU 0, and refused with any of them on GPU 1."""
    made = {n: OnGpu(*t) for n, t in tensors.items()}
    call(made)
    before = library.calls
    assert before > 0
    for n, t in tensors.items():
        with pytest.raises(B.MoeError) as e:
            call({**made, n: OnGpu(*t, dev=1)})
        assert e.value.code == INVALID, n
    assert library.calls == before


def test_tensors_on_another_gpu_are_refused_by_the_router(B, on_gpu_0):
    import torch

    T, E, k = 40, 16, 2
    r = object.__new__(B.MoeRouter)
    r.max_tokens, r.E, r.k, r.dtype, r._desc, r._ws = T, E, k, torch.float32, 0, (0, 0)
    f32, i32 = torch.float32, torch.int32
    out = dict(ids=(i32, (T, k)), scores=(f32, (T, k)), counts=(i32, (E + 1,)),
               prob_sum=(f32, (E,)), losses=(f32, (2,)), row_stat=(f32, (T,)))

    def forward(t):
        r.workspace = t["workspace"]
        r.forward(t["logits"], t["bias"], t["mask"], out=B.RouterResult(*(t[n] for n in out)))

    only_one_elsewhere(B, on_gpu_0, forward, dict(
        out, workspace=(torch.uint8, (64,)), logits=(f32, (T, E)), bias=(f32, (E,)),
        mask=(torch.uint8, (T,))))
    only_one_elsewhere(B, on_gpu_0, lambda t: r.backward(
        t["logits"], t["ids"], t["counts"], t["row_stat"], t["d_scores"], t["d_losses"],
        t["d_logits"]), dict(
            logits=(f32, (T, E)), ids=out["ids"], counts=out["counts"], row_stat=out["row_stat"],
            d_scores=(f32, (T, k)), d_losses=(f32, (2,)), d_logits=(f32, (T, E))))


def test_tensors_on_another_gpu_are_refused_by_the_block_norm(B, on_gpu_0):
    import torch

    T, d, f32 = 10, 64, torch.float32
    h = object.__new__(B.MoeBlockNorm)
    h.max_tokens, h.d, h.gate, h._desc, h._ws_bytes = T, d, B.MOE_GATE_CHANNEL, 0, 0
    h.dtype = h.residual_dtype = h.param_dtype = f32
    rows, column = (f32, (T, d)), (f32, (d,))
    params = dict(w_post=column, gate=column, w_pre=column)
    only_one_elsewhere(B, on_gpu_0, lambda t: h.forward(
        t["residual"], **{n: v for n, v in t.items() if n != "residual"}), dict(
            params, residual=rows, y=rows, residual_out=rows, u=rows))

    def backward(t):
        h.workspace = t["workspace"]
        h.backward(t["x"], **{n: v for n, v in t.items() if n not in ("x", "workspace")})

    only_one_elsewhere(B, on_gpu_0, backward, dict(
        params, workspace=(torch.uint8, (64,)), x=rows, d_residual_out=rows, d_u=rows, y=rows,
        d_residual=rows, dy=rows, dw_post=column, dgate=column, dw_pre=column))


def test_tensors_on_another_gpu_are_refused_by_the_decode(B, on_gpu_0):
    import torch

    n, d, E, k = 3, 256, 4, 2
    p = object.__new__(B.MoePlan)
    p.ptr, p.d, p.k, p.precision, p._prepared_bytes = None, d, k, B.MOE_PREC_NVFP4, [64] * 6
    bf16 = torch.bfloat16
    weights = {"w%d" % i: (torch.uint8, (64,)) for i in range(6)}

    def call(t):
        p.workspace = t["workspace"]
        p.decode_nvfp4(t["x"], t["ids"], t["scores"], [t[n] for n in weights], t["y"])

    only_one_elsewhere(B, on_gpu_0, call, dict(
        weights, workspace=(torch.uint8, (64,)), x=(bf16, (n, d)), y=(bf16, (n, d)),
        ids=(torch.int32, (n, k)), scores=(torch.float32, (n, k))))


def test_decode_checks_without_a_workspace(B):
    """Argument checks come first: a plan without a workspace refuses a good call for that."""
    L = B.lib()
    plan = L.moe_plan_create(8, 256, 256, 4, 2, 2)
    assert plan
    names = ("x", "ids", "scores", "w13", "w13_sf", "w13_scale", "w2", "w2_sf", "w2_scale", "y")

    def call(n=8, **change):
        a = [change.get(name, A) for name in names]
        return L.moe_decode_nvfp4(plan, *a[:3], n, *a[3:], None)

    assert call() == WORKSPACE
    for name in ("w13", "w13_sf", "w13_scale", "w2", "w2_sf", "w2_scale"):
        assert call(**{name: ODD}) == INVALID, name
        assert call(**{name: None}) == INVALID, name
    assert call(n=9) == INVALID and call(n=-1) == INVALID
    L.moe_plan_destroy(plan)


def test_decode_refuses_weights_that_are_not_whole(B, on_gpu_0):
    """An expanded tensor counts bytes that it does not have."""
    import torch

    n, d, E, k = 3, 256, 4, 2
    p = object.__new__(B.MoePlan)
    p.ptr, p.d, p.k, p.precision, p._prepared_bytes = None, d, k, B.MOE_PREC_NVFP4, [64] * 6
    p.workspace = OnGpu(torch.uint8, (64,))
    x = OnGpu(torch.bfloat16, (n, d))
    args = x, OnGpu(torch.int32, (n, k)), OnGpu(torch.float32, (n, k))
    good = [OnGpu(torch.uint8, (64,)) for _ in range(6)]
    p.decode_nvfp4(*args, good, x)
    assert on_gpu_0.calls == 1
    for i in range(6):
        bad = list(good)
        bad[i] = OnGpu(torch.uint8, (64,))
        bad[i].is_contiguous = lambda: False
        with pytest.raises(B.MoeError):
            p.decode_nvfp4(*args, bad, x)
    assert on_gpu_0.calls == 1


def test_more_rows_than_an_int_counts_are_refused(B, on_gpu_0):
    """2^32 + 5 rows are not five rows."""
    import torch

    many, f32, bf16 = 2 ** 32 + 5, torch.float32, torch.bfloat16
    r = object.__new__(B.MoeRouter)
    r.max_tokens, r.E, r.k, r.dtype, r._desc = 8, 1, 1, f32, 0
    n = object.__new__(B.MoeBlockNorm)
    n.max_tokens, n.d, n.gate, n._desc = 8, 1, B.MOE_GATE_NONE, 0
    n.dtype = n.residual_dtype = n.param_dtype = f32
    p = object.__new__(B.MoePlan)
    p.ptr, p.d, p.k, p.precision, p._prepared_bytes = None, 256, 1, B.MOE_PREC_NVFP4, [64] * 6
    p.workspace = OnGpu(torch.uint8, (64,))
    rows, one = OnGpu(f32, (many, 1)), OnGpu(f32, (1,))
    x = OnGpu(bf16, (many, 256))
    for call in (lambda: r.backward(rows, OnGpu(torch.int32, (many, 1)), OnGpu(torch.int32, (2,)),
                                    OnGpu(f32, (many,)), d_logits=rows),
                 lambda: n.forward(rows, w_pre=one, u=rows),
                 lambda: p.decode_nvfp4(x, OnGpu(torch.int32, (many, 1)), rows,
                                        [OnGpu(torch.uint8, (64,))] * 6, x)):
        with pytest.raises(B.MoeError) as e:
            call()
        assert e.value.code == INVALID
    assert on_gpu_0.calls == 0


def test_handles_for_more_rows_than_an_int_counts_are_refused(B):
    for make in (lambda: B.MoeRouter(2 ** 32 + 5, 1, 1), lambda: B.MoeBlockNorm(2 ** 32 + 5, 1)):
        with pytest.raises(B.MoeError) as e:
            make()
        assert e.value.code == INVALID
