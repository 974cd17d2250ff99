"""ctypes binding of include/moe.h (argument marshalling only)."""

import collections
import ctypes
import os
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe_gb300.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_WORKSPACE = 2
MOE_ERR_STATE = 3
MOE_ERR_BAD_IDS = 4
MOE_ERR_TIMEOUT = 5
MOE_ERR_CUDA = 6
MOE_ERR_UNSUPPORTED = 7
MOE_PREC_BF16 = 0
MOE_PREC_MXFP8 = 1
MOE_PREC_NVFP4 = 2
MOE_WS_TRAINING = 1
MOE_WS_HOST_STAGING = 2
MOE_BUF = dict(m_indptr=0, off_pad=1, row_of=2, token_of=3, score_of=4, xe=5, a=6, h=7, ys=8,
               dye=9, dA=10, hs=11, dxe=12, xq=13, xsf=14, hq=15, hsf=16, xqT=17, xqTsf=18,
               dAq=19, dAsf=20, dAqT=21, dAqTsf=22, hsqT=23, hsqTsf=24)

MOE_DTYPE_BF16 = 0
MOE_DTYPE_FP32 = 1
MOE_ROUTER_SOFTMAX_TOPK = 0
MOE_ROUTER_SOFTMAX = 1
MOE_ROUTER_SIGMOID = 2
MOE_GATE_NONE = 0
MOE_GATE_CHANNEL = 1
MOE_GATE_TOKEN = 2
MOE_DECODE_MAX_TOKENS = 256

_lock = threading.Lock()
_lib = None


class RouterDesc(ctypes.Structure):
    """moe_router_desc"""
    _fields_ = [("E", ctypes.c_int), ("k", ctypes.c_int), ("dtype", ctypes.c_int),
                ("scoring", ctypes.c_int), ("scale", ctypes.c_float)]


class BlockNormDesc(ctypes.Structure):
    """moe_block_norm_desc"""
    _fields_ = [("d", ctypes.c_int), ("dtype", ctypes.c_int), ("residual_dtype", ctypes.c_int),
                ("param_dtype", ctypes.c_int), ("gate", ctypes.c_int), ("alpha", ctypes.c_float),
                ("eps", ctypes.c_float)]


class MoeError(RuntimeError):
    def __init__(self, code, what=""):
        self.code = code
        name = _lib.moe_status_string(code).decode() if _lib is not None else str(code)
        super().__init__("%s%s" % (name, (": " + what) if what else ""))


def _declare(L):
    vp, i32, f32, sz, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_long
    L.moe_plan_create.argtypes = [i32] * 6
    L.moe_plan_create.restype = vp
    L.moe_plan_destroy.argtypes = [vp]
    L.moe_plan_destroy.restype = None
    L.moe_plan_set_swiglu_clamp.argtypes = [vp, f32]
    L.moe_plan_workspace_bytes.argtypes = [vp, i32]
    L.moe_plan_workspace_bytes.restype = sz
    L.moe_plan_set_workspace.argtypes = [vp, vp, sz, i32]
    L.moe_forward.argtypes = [vp] * 9 + [i32, vp]
    L.moe_backward.argtypes = [vp] * 9
    L.moe_forward_routed.argtypes = [vp, vp, ctypes.c_longlong] + [vp] * 9
    L.moe_step_host.argtypes = [vp] * 13
    L.moe_quantize_mxfp8.argtypes = [vp, i64, i32, vp, vp, vp]
    L.moe_plan_check.argtypes = [vp, ctypes.POINTER(ctypes.c_longlong)]
    L.moe_status_string.argtypes = [i32]
    L.moe_status_string.restype = ctypes.c_char_p
    L.moe_plan_buffer.argtypes = [vp, i32, ctypes.POINTER(vp), ctypes.POINTER(sz)]
    L.moe_tile_rows.restype = i32
    L.moe_plan_set_cta_pairs.argtypes = [vp, i32]
    L.moe_plan_row_granule.argtypes = [vp]
    L.moe_plan_row_granule.restype = i32
    L.moe_gemm_scratch_bytes.argtypes = [i32, i32]
    L.moe_gemm_scratch_bytes.restype = sz
    L.moe_gemm_bf16.argtypes = [i32, vp, vp, vp, i32, i32, i32, vp, vp]
    L.moe_plan_set_timing_events.argtypes = [vp, i32, ctypes.POINTER(vp), i32]
    L.moe_plan_set_debug.argtypes = [vp, ctypes.c_longlong, i32]
    L.moe_mxfp8_weight_scale_bytes.argtypes = [i32, i32, i32, i32]
    L.moe_mxfp8_weight_scale_bytes.restype = sz
    L.moe_prepare_weights_mxfp8.argtypes = [vp, vp, i32, i32, i32, vp, vp, vp, vp, vp]
    L.moe_prepare_weights_mxfp8_backward.argtypes = [vp, vp, i32, i32, i32, vp, vp, vp, vp, vp]
    L.moe_backward_mxfp8.argtypes = [vp] * 11
    L.moe_plan_set_activation_scales.argtypes = [vp, f32, f32]
    L.moe_nvfp4_weight_bytes.argtypes = [i32, i32, i32, i32]
    L.moe_nvfp4_weight_bytes.restype = sz
    L.moe_prepare_weights_nvfp4.argtypes = [vp, vp, i32, i32, i32] + [vp] * 7
    L.moe_forward_nvfp4.argtypes = [vp] * 12
    L.moe_decode_nvfp4.argtypes = [vp] * 4 + [i32] + [vp] * 8
    L.moe_decode_nvfp4.restype = i32
    L.moe_amax_bf16.argtypes = [vp, ctypes.c_longlong, vp, vp]
    L.moe_plan_set_backward_split.argtypes = [vp, i32]
    L.moe_plan_set_wgrad_interleave.argtypes = [vp, ctypes.c_longlong]
    L.moe_plan_num_sms.argtypes = [vp]
    L.moe_plan_num_sms.restype = i32
    L.moe_plan_launch_count.argtypes = [vp]
    L.moe_plan_launch_count.restype = ctypes.c_longlong
    i64x = ctypes.c_longlong
    L.moe_router_workspace_bytes.argtypes = [vp, i32]
    L.moe_router_workspace_bytes.restype = sz
    L.moe_router_forward.argtypes = [vp, i32, vp, i64x] + [vp] * 9 + [sz, vp]
    L.moe_router_backward.argtypes = [vp, i32, vp, i64x] + [vp] * 6 + [i64x, vp]
    L.moe_block_norm_workspace_bytes.argtypes = [vp, i32]
    L.moe_block_norm_workspace_bytes.restype = sz
    L.moe_block_norm_forward.argtypes = [vp, i32] + [vp, i64x] * 2 + [vp] * 3 + [vp, i64x] * 2 + [vp]
    L.moe_block_norm_backward.argtypes = ([vp, i32] + [vp, i64x] * 4 + [vp] * 3 + [vp, i64x] * 2 +
                                          [vp] * 3 + [i32, vp, sz, vp])
    for name in ("moe_router_forward", "moe_router_backward", "moe_block_norm_forward",
                 "moe_block_norm_backward"):
        getattr(L, name).restype = i32
    for name in ("moe_plan_set_swiglu_clamp", "moe_plan_set_workspace", "moe_forward",
                 "moe_forward_routed",
                 "moe_backward", "moe_step_host", "moe_quantize_mxfp8", "moe_plan_check",
                 "moe_plan_buffer", "moe_gemm_bf16", "moe_plan_set_timing_events",
                 "moe_prepare_weights_mxfp8", "moe_plan_set_debug", "moe_plan_set_cta_pairs",
                 "moe_prepare_weights_mxfp8_backward", "moe_backward_mxfp8",
                 "moe_plan_set_activation_scales", "moe_prepare_weights_nvfp4",
                 "moe_forward_nvfp4", "moe_amax_bf16", "moe_plan_set_backward_split",
                 "moe_plan_set_wgrad_interleave"):
        getattr(L, name).restype = i32
    return L


def lib():
    """The loaded C library.  Raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    "libmoe_gb300.so is not built; run `python -m routed_mixture_experts_gb300.build` "
                    "(there is no CPU fallback)")
            _lib = _declare(ctypes.CDLL(LIB_PATH))
        return _lib


def _check(rc, what=""):
    if rc != MOE_OK:
        raise MoeError(rc, what)


def _stream(stream):
    import torch

    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


class MoePlan:
    """A routed-expert layer plan with its workspace (a torch uint8 device tensor)."""

    def __init__(self, T, d, I, E, k, precision=MOE_PREC_BF16, clamp=0.0,
                 flags=MOE_WS_TRAINING, device="cuda", cta_pairs=False):
        import torch

        L = lib()
        self.T, self.d, self.I, self.E, self.k = T, d, I, E, k
        self.precision = precision
        self.flags = flags
        self.ptr = L.moe_plan_create(T, d, I, E, k, precision)
        if not self.ptr:
            raise MoeError(MOE_ERR_INVALID_ARG, "moe_plan_create(%d,%d,%d,%d,%d)" % (T, d, I, E, k))
        _check(L.moe_plan_set_swiglu_clamp(self.ptr, float(clamp)), "clamp")
        if cta_pairs:
            _check(L.moe_plan_set_cta_pairs(self.ptr, 1), "cta_pairs")
        if precision == MOE_PREC_NVFP4:       # of codes, scales and fp32 scales of W13 and W2
            size = [L.moe_nvfp4_weight_bytes(d, I, E, which) for which in range(4)]
            self._prepared_bytes = [size[0], size[1], 4 * E, size[2], size[3], 4 * E]
        nbytes = L.moe_plan_workspace_bytes(self.ptr, flags)
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        _check(L.moe_plan_set_workspace(self.ptr, _p(self.workspace), nbytes, flags), "workspace")

    def __del__(self):
        if getattr(self, "ptr", None) and _lib is not None:
            _lib.moe_plan_destroy(self.ptr)
            self.ptr = None

    def forward(self, x, ids, scores, w13, w2, y=None, save=False, w13_sf=None, w2_sf=None,
                stream=None):
        import torch

        if y is None:
            y = torch.empty(self.T, self.d, dtype=torch.bfloat16, device=x.device)
        _check(lib().moe_forward(self.ptr, _p(x), _p(ids), _p(scores), _p(w13), _p(w2), _p(w13_sf),
                                 _p(w2_sf), _p(y), 1 if save else 0, _stream(stream)), "forward")
        return y

    def forward_routed(self, x_e, m_indptr, off_pad, w13, w2, score_of=None, ys=None,
                       row_of=None, y=None, stream=None):
        """Forward over caller-laid-out expert-major rows x_e [rows, d] (see
        moe_forward_routed in moe.h).  Returns (ys, y); y only with row_of."""
        import torch

        rows = x_e.shape[0]
        if ys is None:
            ys = torch.empty(rows, self.d, dtype=torch.bfloat16, device=x_e.device)
        if row_of is not None and y is None:
            y = torch.empty(self.T, self.d, dtype=torch.bfloat16, device=x_e.device)
        _check(lib().moe_forward_routed(self.ptr, _p(x_e), rows, _p(m_indptr), _p(off_pad),
                                        _p(score_of), _p(w13), _p(w2), _p(ys), _p(row_of), _p(y),
                                        _stream(stream)), "forward_routed")
        return ys, y

    def set_activation_scales(self, x_scale, h_scale):
        """Static NVFP4 activation dequantisation scales (see moe.h)."""
        _check(lib().moe_plan_set_activation_scales(self.ptr, float(x_scale), float(h_scale)),
               "set_activation_scales")

    def forward_nvfp4(self, x, ids, scores, prepared, y=None, stream=None):
        """NVFP4 inference forward; prepared = prepare_weights_nvfp4(w13, w2)."""
        import torch

        if y is None:
            y = torch.empty(self.T, self.d, dtype=torch.bfloat16, device=x.device)
        w13q, w13s, w13c, w2q, w2s, w2c = prepared
        _check(lib().moe_forward_nvfp4(self.ptr, _p(x), _p(ids), _p(scores), _p(w13q), _p(w13s),
                                       _p(w13c), _p(w2q), _p(w2s), _p(w2c), _p(y),
                                       _stream(stream)), "forward_nvfp4")
        return y

    def decode_nvfp4(self, x, ids, scores, prepared, y=None, stream=None):
        """The routed experts of x [tokens, d], tokens <= min(T, MOE_DECODE_MAX_TOKENS);
        prepared = prepare_weights_nvfp4(w13, w2) (see moe_decode_nvfp4 in moe.h)."""
        import torch

        if stream is not None:               # y then belongs to that stream too
            with torch.cuda.stream(stream):
                return self.decode_nvfp4(x, ids, scores, prepared, y)
        n, k = x.shape[0], self.k
        _rows_fit(n, "decode_nvfp4")
        bf16 = torch.bfloat16
        dev = _device()
        _scratch_on(self.workspace, dev)
        xp = _want(x, "x", bf16, (n, self.d), dev)
        if y is None:
            y = torch.empty((n, self.d), dtype=bf16, device=x.device)
            yp = y.data_ptr()
        else:
            yp = _want(y, "y", bf16, (n, self.d), dev)
        if (self.precision == MOE_PREC_NVFP4 and
                [t.nbytes if t.get_device() == dev and t.is_contiguous() else 0 for t in prepared]
                != self._prepared_bytes):
            raise MoeError(MOE_ERR_INVALID_ARG, "decode_nvfp4: the weights are not those of "
                           "prepare_weights_nvfp4 for this plan's d, I and E")
        w13q, w13s, w13c, w2q, w2s, w2c = prepared
        _check(_lib.moe_decode_nvfp4(
            self.ptr, xp, _want(ids, "ids", torch.int32, (n, k), dev),
            _want(scores, "scores", torch.float32, (n, k), dev), n,
            w13q.data_ptr(), w13s.data_ptr(), w13c.data_ptr(), w2q.data_ptr(), w2s.data_ptr(),
            w2c.data_ptr(), yp, _raw_stream(dev)), "decode_nvfp4")
        return y

    def backward(self, dy, w13, w2, dw13, dw2, dx=None, dscores=None, stream=None):
        import torch

        if dx is None:
            dx = torch.empty(self.T, self.d, dtype=torch.bfloat16, device=dy.device)
        if dscores is None:
            dscores = torch.empty(self.T, self.k, dtype=torch.float32, device=dy.device)
        _check(lib().moe_backward(self.ptr, _p(dy), _p(w13), _p(w2), _p(dx), _p(dw13), _p(dw2),
                                  _p(dscores), _stream(stream)), "backward")
        return dx, dscores

    def backward_mxfp8(self, dy, w13t, w13t_sf, w2t, w2t_sf, dw13, dw2, dx=None, dscores=None,
                       stream=None):
        """Backward of an MXFP8 plan; w13t.. from prepare_weights_mxfp8_backward."""
        import torch

        if dx is None:
            dx = torch.empty(self.T, self.d, dtype=torch.bfloat16, device=dy.device)
        if dscores is None:
            dscores = torch.empty(self.T, self.k, dtype=torch.float32, device=dy.device)
        _check(lib().moe_backward_mxfp8(self.ptr, _p(dy), _p(w13t), _p(w13t_sf), _p(w2t),
                                        _p(w2t_sf), _p(dx), _p(dw13), _p(dw2), _p(dscores),
                                        _stream(stream)), "backward_mxfp8")
        return dx, dscores

    def step_host(self, x_h, ids_h, scores_h, w13, w2, y_h, dy_h=None, dw13=None, dw2=None,
                  dx_h=None, dscores_h=None, stream=None):
        _check(lib().moe_step_host(self.ptr, _p(x_h), _p(ids_h), _p(scores_h), _p(dy_h), _p(w13),
                                   _p(w2), _p(dw13), _p(dw2), _p(y_h), _p(dx_h), _p(dscores_h),
                                   _stream(stream)), "step_host")

    def set_timing_events(self, which, events):
        """Record `events` (torch.cuda.Event list, None entries skipped; or None) at the
        stage boundaries of every following forward (which=0) or backward (which=1) call."""
        if not events:
            self._ev = getattr(self, "_ev", {})
            self._ev.pop(which, None)
            _check(lib().moe_plan_set_timing_events(self.ptr, which, None, 0), "timing")
            return
        handles = [None if e is None else e.cuda_event for e in events]
        arr = (ctypes.c_void_p * len(events))(*handles)
        self._ev = getattr(self, "_ev", {})
        self._ev[which] = (arr, events)          # keep the handles alive while set
        _check(lib().moe_plan_set_timing_events(self.ptr, which, arr, len(events)), "timing")

    def set_backward_split(self, wgrad_sms):
        """Weight-gradient GEMMs on wgrad_sms SMs beside DGRAD-W13 (0: off); see moe.h."""
        _check(lib().moe_plan_set_backward_split(self.ptr, int(wgrad_sms)), "backward_split")

    def set_wgrad_interleave(self, min_rows):
        """Weight-gradient tiles of experts with more than min_rows rows run
        interleaved with the lighter ones (0: plain order); see moe.h."""
        _check(lib().moe_plan_set_wgrad_interleave(self.ptr, int(min_rows)), "wgrad_interleave")

    def num_sms(self):
        return lib().moe_plan_num_sms(self.ptr)

    def set_debug(self, wait_limit_ns=0, stall_w13=False):
        """Failure-path testing knobs (see moe_plan_set_debug in moe.h)."""
        _check(lib().moe_plan_set_debug(self.ptr, int(wait_limit_ns), 1 if stall_w13 else 0),
               "set_debug")

    def row_granule(self):
        """Padding granule of the expert segments (128, or 256 with CTA-pair GEMMs)."""
        return lib().moe_plan_row_granule(self.ptr)

    def launch_count(self):
        return lib().moe_plan_launch_count(self.ptr)

    def check(self):
        """Synchronise and return (status, detail) of the device error word."""
        det = ctypes.c_longlong(0)
        rc = lib().moe_plan_check(self.ptr, ctypes.byref(det))
        return rc, det.value

    def buffer(self, name, dtype, shape=None):
        """A torch view of one internal workspace tensor (see MOE_BUF_* in moe.h)."""
        import torch

        ptr = ctypes.c_void_p()
        nb = ctypes.c_size_t()
        _check(lib().moe_plan_buffer(self.ptr, MOE_BUF[name], ctypes.byref(ptr), ctypes.byref(nb)),
               name)
        off = ptr.value - self.workspace.data_ptr()
        t = self.workspace[off:off + nb.value].view(dtype)
        return t if shape is None else t[: int(torch.tensor(shape).prod())].view(*shape)


def quantize_mxfp8(w, stream=None):
    """bf16 [..., K] -> (E4M3 codes uint8 [..., K], E8M0 scales uint8 [..., K/32])."""
    import torch

    K = w.shape[-1]
    rows = w.numel() // K
    codes = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
    scales = torch.empty(w.shape[:-1] + (K // 32,), dtype=torch.uint8, device=w.device)
    _check(lib().moe_quantize_mxfp8(_p(w), rows, K, _p(codes), _p(scales), _stream(stream)),
           "quantize_mxfp8")
    return codes, scales


def prepare_weights_mxfp8(w13, w2, stream=None):
    """bf16 W13 [E,2I,d], W2 [E,d,I] -> (w13 codes, w13 tiled scales, w2 codes,
    w2 tiled scales), the prepared MXFP8 weights of moe_forward."""
    import torch

    E, I2, d = w13.shape
    I = I2 // 2
    L = lib()
    w13q = torch.empty(w13.shape, dtype=torch.uint8, device=w13.device)
    w2q = torch.empty(w2.shape, dtype=torch.uint8, device=w2.device)
    w13s = torch.empty(L.moe_mxfp8_weight_scale_bytes(d, I, E, 0), dtype=torch.uint8,
                       device=w13.device)
    w2s = torch.empty(L.moe_mxfp8_weight_scale_bytes(d, I, E, 1), dtype=torch.uint8,
                      device=w2.device)
    _check(L.moe_prepare_weights_mxfp8(_p(w13), _p(w2), d, I, E, _p(w13q), _p(w13s), _p(w2q),
                                       _p(w2s), _stream(stream)), "prepare_weights_mxfp8")
    return w13q, w13s, w2q, w2s


def prepare_weights_nvfp4(w13, w2, stream=None):
    """bf16 W13 [E,2I,d], W2 [E,d,I] -> (w13 codes, w13 tiled scales, w13 per-expert
    scales, w2 codes, w2 tiled scales, w2 per-expert scales), the prepared NVFP4
    weights of moe_forward_nvfp4."""
    import torch

    E, I2, d = w13.shape
    I = I2 // 2
    L = lib()
    dev = w13.device
    nb = lambda which: L.moe_nvfp4_weight_bytes(d, I, E, which)
    w13q = torch.empty(E, I2, d // 2, dtype=torch.uint8, device=dev)
    w13s = torch.empty(nb(1), dtype=torch.uint8, device=dev)
    w2q = torch.empty(E, d, I // 2, dtype=torch.uint8, device=dev)
    w2s = torch.empty(nb(3), dtype=torch.uint8, device=dev)
    w13c = torch.empty(E, dtype=torch.float32, device=dev)
    w2c = torch.empty(E, dtype=torch.float32, device=dev)
    _check(L.moe_prepare_weights_nvfp4(_p(w13), _p(w2), d, I, E, _p(w13q), _p(w13s), _p(w13c),
                                       _p(w2q), _p(w2s), _p(w2c), _stream(stream)),
           "prepare_weights_nvfp4")
    return w13q, w13s, w13c, w2q, w2s, w2c


def amax_bf16(t, stream=None):
    """max |t| of a bf16 device tensor, as a one-element fp32 device tensor."""
    import torch

    out = torch.empty(1, dtype=torch.float32, device=t.device)
    _check(lib().moe_amax_bf16(_p(t), t.numel(), _p(out), _stream(stream)), "amax_bf16")
    return out


def prepare_weights_mxfp8_backward(w13, w2, stream=None):
    """bf16 W13 [E,2I,d], W2 [E,d,I] -> (W13^T codes [E,d,2I], their tiled scales,
    W2^T codes [E,I,d], their tiled scales), the prepared weights of
    moe_backward_mxfp8 (quantised along 2I and along d)."""
    import torch

    E, I2, d = w13.shape
    I = I2 // 2
    L = lib()
    w13t = torch.empty(E, d, I2, dtype=torch.uint8, device=w13.device)
    w2t = torch.empty(E, I, d, dtype=torch.uint8, device=w2.device)
    w13ts = torch.empty(L.moe_mxfp8_weight_scale_bytes(d, I, E, 2), dtype=torch.uint8,
                        device=w13.device)
    w2ts = torch.empty(L.moe_mxfp8_weight_scale_bytes(d, I, E, 3), dtype=torch.uint8,
                       device=w2.device)
    _check(L.moe_prepare_weights_mxfp8_backward(_p(w13), _p(w2), d, I, E, _p(w13t), _p(w13ts),
                                                _p(w2t), _p(w2ts), _stream(stream)),
           "prepare_weights_mxfp8_backward")
    return w13t, w13ts, w2t, w2ts


def gemm_bf16(mode, A, B, C, M, N, K, stream=None):
    """Dense GEMM through the grouped tcgen05 kernels (modes as in moe.h)."""
    import torch

    L = lib()
    scratch = torch.empty(L.moe_gemm_scratch_bytes(M, K), dtype=torch.uint8, device=A.device)
    _check(L.moe_gemm_bf16(mode, _p(A), _p(B), _p(C), M, N, K, _p(scratch), _stream(stream)),
           "gemm_bf16")
    return C


# ---- the operators around the experts -----------------------------------------


def _device():
    """The index of the current device, whose stream a call takes."""
    import torch

    return torch._C._cuda_getDevice()


def _raw_stream(dev):
    """The handle of device dev's current stream.  (The public
    torch.cuda.current_stream() builds a Stream object for it, a third of the host
    time of a small call.)"""
    import torch

    return torch._C._cuda_getCurrentRawStream(dev)


def _dtype_code(dtype, what):
    import torch

    if dtype == torch.bfloat16:
        return MOE_DTYPE_BF16
    if dtype == torch.float32:
        return MOE_DTYPE_FP32
    raise MoeError(MOE_ERR_INVALID_ARG, "%s: dtype %s (bfloat16 or float32)" % (what, dtype))


def _rows_fit(T, what):
    """ctypes would cut a row count to 32 bits without a word."""
    if T > 0x7FFFFFFF:
        raise MoeError(MOE_ERR_INVALID_ARG, "%s: %d rows (2^31 - 1 at most)" % (what, T))


def _want(t, what, dtype, shape, dev):
    """t: a contiguous tensor of this dtype and shape on CUDA device dev (its address)."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    raise MoeError(MOE_ERR_INVALID_ARG, "%s: want contiguous %s %s on the current GPU (%d), got "
                   "%s %s on %s" % (what, dtype, tuple(shape), dev, t.dtype, tuple(t.shape),
                                    t.device))


def _maybe(t, what, dtype, shape, dev):
    return None if t is None else _want(t, what, dtype, shape, dev)


def _rows(t, what, dtype, shape, dev):
    """t: a [T, n] tensor on CUDA device dev whose rows may lie further apart (address, row
    distance)."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev:
        if t.is_contiguous():
            return t.data_ptr(), shape[1]
        apart, inner = t.stride()
        if shape[0] <= 1:
            apart = shape[1]
        if (inner == 1 or shape[1] == 1) and apart >= shape[1]:
            return t.data_ptr(), apart
    raise MoeError(MOE_ERR_INVALID_ARG, "%s: want %s %s on the current GPU (%d), rows dense and "
                   "apart; got %s %s on %s, strides %s" % (what, dtype, tuple(shape), dev, t.dtype,
                                                           tuple(t.shape), t.device, t.stride()))


def _scratch_on(workspace, dev):
    if workspace.get_device() != dev:
        raise MoeError(MOE_ERR_INVALID_ARG, "the handle's scratch is on %s, the current GPU is %d"
                       % (workspace.device, dev))


RouterResult = collections.namedtuple(
    "RouterResult", "ids scores counts prob_sum losses row_stat")


class MoeRouter:
    """Top-k routing with the balance and z losses (moe_router_* in moe.h).

    max_tokens sizes the scratch; a call takes any T up to it.  One MoeRouter per
    concurrent stream."""

    def __init__(self, max_tokens, E, k, scoring=MOE_ROUTER_SOFTMAX_TOPK, scale=1.0, dtype=None,
                 device="cuda"):
        import torch

        L = lib()
        _rows_fit(max_tokens, "MoeRouter")
        self.max_tokens, self.E, self.k = max_tokens, E, k
        self.dtype = dtype if dtype is not None else torch.float32
        self.desc = RouterDesc(E, k, _dtype_code(self.dtype, "MoeRouter"), scoring, scale)
        self._desc = ctypes.addressof(self.desc)
        nbytes = L.moe_router_workspace_bytes(self._desc, max_tokens)
        if not nbytes:
            raise MoeError(MOE_ERR_INVALID_ARG, "MoeRouter(%d,%d,%d)" % (max_tokens, E, k))
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self._ws = (self.workspace.data_ptr(), nbytes)

    def outputs(self, T):
        """Fresh output tensors of a forward over T tokens."""
        from torch import empty, float32, int32

        dev, E, k = self.workspace.device, self.E, self.k
        return RouterResult(empty((T, k), dtype=int32, device=dev),
                            empty((T, k), dtype=float32, device=dev),
                            empty((E + 1,), dtype=int32, device=dev),
                            empty((E,), dtype=float32, device=dev),
                            empty((2,), dtype=float32, device=dev),
                            empty((T,), dtype=float32, device=dev))

    def forward(self, logits, bias=None, token_mask=None, out=None, stream=None):
        """logits [T, E] -> RouterResult(ids, scores, counts, prob_sum, losses, row_stat);
        `out`: an earlier result (or outputs(T)) to overwrite."""
        import torch

        if stream is not None:               # the outputs then belong to that stream too
            with torch.cuda.stream(stream):
                return self.forward(logits, bias, token_mask, out)
        f32, i32 = torch.float32, torch.int32
        T, E, k = logits.shape[0], self.E, self.k
        if T > self.max_tokens:
            raise MoeError(MOE_ERR_INVALID_ARG, "router: %d tokens, made for %d" % (
                T, self.max_tokens))
        dev = _device()
        _scratch_on(self.workspace, dev)
        lp, ld = _rows(logits, "logits", self.dtype, (T, E), dev)
        bp = _maybe(bias, "bias", f32, (E,), dev)
        mp = _maybe(token_mask, "token_mask", torch.uint8, (T,), dev)
        if out is None:
            out = self.outputs(T)
            at = [t.data_ptr() for t in out]
        else:
            at = (_want(out.ids, "ids", i32, (T, k), dev),
                  _want(out.scores, "scores", f32, (T, k), dev),
                  _want(out.counts, "counts", i32, (E + 1,), dev),
                  _want(out.prob_sum, "prob_sum", f32, (E,), dev),
                  _want(out.losses, "losses", f32, (2,), dev),
                  _want(out.row_stat, "row_stat", f32, (T,), dev))
        _check(_lib.moe_router_forward(self._desc, T, lp, ld, bp, mp, *at, *self._ws,
                                       _raw_stream(dev)), "router forward")
        return out

    def backward(self, logits, ids, counts, row_stat, d_scores=None, d_losses=None,
                 d_logits=None, stream=None):
        """Gradient at the logits of sum(d_scores * scores) + sum(d_losses * losses)."""
        import torch

        if stream is not None:
            with torch.cuda.stream(stream):
                return self.backward(logits, ids, counts, row_stat, d_scores, d_losses, d_logits)
        T, E, k = logits.shape[0], self.E, self.k
        _rows_fit(T, "router backward")
        f32 = torch.float32
        dev = _device()
        lp, ld = _rows(logits, "logits", self.dtype, (T, E), dev)
        if d_logits is None:
            d_logits = torch.empty((T, E), dtype=self.dtype, device=logits.device)
            dp, ld_d = d_logits.data_ptr(), E
        else:
            dp, ld_d = _rows(d_logits, "d_logits", self.dtype, (T, E), dev)
        _check(_lib.moe_router_backward(
            self._desc, T, lp, ld, _maybe(ids, "ids", torch.int32, (T, k), dev),
            _want(counts, "counts", torch.int32, (E + 1,), dev),
            _want(row_stat, "row_stat", f32, (T,), dev),
            _maybe(d_scores, "d_scores", f32, (T, k), dev),
            _maybe(d_losses, "d_losses", f32, (2,), dev), dp, ld_d, _raw_stream(dev)),
            "router backward")
        return d_logits


BlockNormGrads = collections.namedtuple("BlockNormGrads", "d_residual dy dw_post dgate dw_pre")


class MoeBlockNorm:
    """The norms around a block with its gate and residual scale (moe_block_norm_*
    in moe.h).  max_tokens sizes the backward's scratch; one MoeBlockNorm per
    concurrent stream.

    dtype: of y, u; residual_dtype: of the residual stream; param_dtype: of w_post,
    w_pre and gate ([d] with MOE_GATE_CHANNEL, [T] with MOE_GATE_TOKEN)."""

    def __init__(self, max_tokens, d, dtype=None, residual_dtype=None, param_dtype=None,
                 gate=MOE_GATE_NONE, alpha=1.0, eps=1e-6, device="cuda"):
        import torch

        _rows_fit(max_tokens, "MoeBlockNorm")
        self.max_tokens, self.d, self.gate = max_tokens, d, gate
        self.dtype = dtype if dtype is not None else torch.bfloat16
        self.residual_dtype = residual_dtype if residual_dtype is not None else self.dtype
        self.param_dtype = param_dtype if param_dtype is not None else torch.float32
        self.desc = BlockNormDesc(d, _dtype_code(self.dtype, "dtype"),
                                  _dtype_code(self.residual_dtype, "residual_dtype"),
                                  _dtype_code(self.param_dtype, "param_dtype"), gate, alpha, eps)
        self._desc = ctypes.addressof(self.desc)
        self._ws_bytes = lib().moe_block_norm_workspace_bytes(self._desc, max_tokens)
        if not self._ws_bytes:
            raise MoeError(MOE_ERR_INVALID_ARG, "MoeBlockNorm(%d,%d)" % (max_tokens, d))
        self.device, self.workspace = device, None     # scratch: from the first backward on

    def _params(self, T, w_post, gate, w_pre, dev):
        """Addresses of w_post, gate and w_pre, and the gate's shape."""
        pt, d = self.param_dtype, (self.d,)
        shape = (T,) if self.gate == MOE_GATE_TOKEN else d
        return (_maybe(w_post, "w_post", pt, d, dev), _maybe(gate, "gate", pt, shape, dev),
                _maybe(w_pre, "w_pre", pt, d, dev), shape)

    def forward(self, residual, y=None, w_post=None, gate=None, w_pre=None, residual_out=None,
                u=None, stream=None):
        """-> (residual_out, u); without y the first is residual, without w_pre u is None
        (and a tensor given for it is refused)."""
        import torch

        if stream is not None:               # the outputs then belong to that stream too
            with torch.cuda.stream(stream):
                return self.forward(residual, y, w_post, gate, w_pre, residual_out, u)
        T = residual.shape[0]
        _rows_fit(T, "block norm forward")
        shape, dev = (T, self.d), _device()
        rp, ld_r = _rows(residual, "residual", self.residual_dtype, shape, dev)
        wp, gp, wq, _ = self._params(T, w_post, gate, w_pre, dev)
        if (y is None and residual_out is not None) or (w_pre is None and u is not None):
            raise MoeError(MOE_ERR_INVALID_ARG, "block norm: residual_out goes with y, u with w_pre")
        yp = op = up = None
        ld_y = ld_o = ld_u = 0
        if y is not None:
            yp, ld_y = _rows(y, "y", self.dtype, shape, dev)
            if residual_out is None:
                residual_out = torch.empty(shape, dtype=self.residual_dtype,
                                           device=residual.device)
                op, ld_o = residual_out.data_ptr(), self.d
            else:
                op, ld_o = _rows(residual_out, "residual_out", self.residual_dtype, shape, dev)
        if w_pre is not None:
            if u is None:
                u = torch.empty(shape, dtype=self.dtype, device=residual.device)
                up, ld_u = u.data_ptr(), self.d
            else:
                up, ld_u = _rows(u, "u", self.dtype, shape, dev)
        _check(_lib.moe_block_norm_forward(self._desc, T, rp, ld_r, yp, ld_y, wp, gp, wq, op, ld_o,
                                            up, ld_u, _raw_stream(dev)), "block norm forward")
        return (residual if y is None else residual_out), (None if w_pre is None else u)

    def backward(self, residual_out, d_residual_out=None, d_u=None, y=None, w_post=None, gate=None,
                 w_pre=None, d_residual=None, dy=None, dw_post=None, dgate=None, dw_pre=None,
                 accumulate=False, stream=None):
        """-> BlockNormGrads(d_residual, dy, dw_post, dgate, dw_pre); entries of absent
        inputs are None.  accumulate adds to the given dw_post, dgate and dw_pre."""
        import torch

        if stream is not None:
            with torch.cuda.stream(stream):
                return self.backward(residual_out, d_residual_out, d_u, y, w_post, gate, w_pre,
                                     d_residual, dy, dw_post, dgate, dw_pre, accumulate)
        T, at, f32 = residual_out.shape[0], residual_out.device, torch.float32
        if T > self.max_tokens:
            raise MoeError(MOE_ERR_INVALID_ARG, "block norm: %d rows, made for %d" % (
                T, self.max_tokens))
        d, dev = self.d, _device()
        shape = (T, d)
        act, res = self.dtype, self.residual_dtype
        rp, ld_r = _rows(residual_out, "residual_out", res, shape, dev)
        wp, gp, wq, gshape = self._params(T, w_post, gate, w_pre, dev)
        yp = gr = gu = op = dp = wpp = ggp = wqp = None
        ld_y = ld_gr = ld_gu = ld_d = 0
        if y is not None:
            yp, ld_y = _rows(y, "y", act, shape, dev)
        if d_residual_out is not None:
            gr, ld_gr = _rows(d_residual_out, "d_residual_out", res, shape, dev)
        if d_u is not None:
            gu, ld_gu = _rows(d_u, "d_u", act, shape, dev)
        # outputs: the caller's are checked, fresh ones are what they have to be
        new = torch.zeros if accumulate else torch.empty
        if d_residual is not None:
            op, ld_o = _rows(d_residual, "d_residual", res, shape, dev)
        else:
            d_residual = torch.empty(shape, dtype=res, device=at)
            op, ld_o = d_residual.data_ptr(), d
        if dy is not None:
            dp, ld_d = _rows(dy, "dy", act, shape, dev)
        elif y is not None:
            dy = torch.empty(shape, dtype=act, device=at)
            dp, ld_d = dy.data_ptr(), d
        if dw_post is not None:
            wpp = _want(dw_post, "dw_post", f32, (d,), dev)
        elif w_post is not None:
            dw_post = new((d,), dtype=f32, device=at)
            wpp = dw_post.data_ptr()
        if dgate is not None:
            ggp = _want(dgate, "dgate", f32, gshape, dev)
        elif gate is not None:
            dgate = new(gshape, dtype=f32, device=at)
            ggp = dgate.data_ptr()
        if dw_pre is not None:
            wqp = _want(dw_pre, "dw_pre", f32, (d,), dev)
        elif w_pre is not None:
            dw_pre = new((d,), dtype=f32, device=at)
            wqp = dw_pre.data_ptr()
        if self.workspace is None:
            self.workspace = torch.empty(self._ws_bytes, dtype=torch.uint8, device=self.device)
        _scratch_on(self.workspace, dev)
        _check(_lib.moe_block_norm_backward(
            self._desc, T, rp, ld_r, yp, ld_y, gr, ld_gr, gu, ld_gu, wp, gp, wq, op, ld_o, dp, ld_d,
            wpp, ggp, wqp, 1 if accumulate else 0, self.workspace.data_ptr(), self._ws_bytes,
            _raw_stream(dev)), "block norm backward")
        return BlockNormGrads(d_residual, dy, dw_post, dgate, dw_pre)
