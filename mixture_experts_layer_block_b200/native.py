"""ctypes binding of libmoe_b200.so (the C ABI in include/moe_b200.h).

Argument marshalling only: every step of the layer runs in the library's CUDA kernels. The
functions keep the C names; ``MoELayer`` is a convenience owner of a handle that takes torch
tensors (device memory and streams come from PyTorch). torch is imported by the first call that needs it,
so that the C functions can be had without it. There is no fallback: if the library
is missing this module raises on import.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
# MOE_B200_LIBRARY may name another build of the same library (for A/B timing of builds)
LIB_PATH = os.environ.get("MOE_B200_LIBRARY") or os.path.join(_PKG, "libmoe_b200.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = -1
MOE_ERR_UNSUPPORTED = -2
MOE_ERR_CUDA = -3
MOE_ERR_OUT_OF_MEMORY = -4
MOE_ERR_MISALIGNED = -5
MOE_ERR_DEVICE_TIMEOUT = -6
MOE_ERR_NOT_READY = -7

MOE_FLAG_STAGE_TIMING = 1
MOE_FLAG_HOST_STAGING = 2
MOE_FLAG_PAIR_TILES = 8
MOE_FLAG_SINGLE_TILES = 16
MOE_FLAG_OUT_BF16 = 32
MOE_FLAG_TAIL_TILES = 64
MOE_FLAG_NO_TAIL_TILES = 128
MOE_FLAG_STATIC_QUOTA = 256
MOE_FLAG_MXFP8 = 512
MOE_FLAG_UNFUSED_SMALL = 1024
MOE_FLAG_TWO_TILES = 2048
MOE_FLAG_TRACE = 4

MOE_FFN_GRAD_F32 = 1
MOE_FFN_GRAD_ADD = 2


class moe_config(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("inter_shared", ctypes.c_int32), ("num_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("block_m", ctypes.c_int32),
                ("capacity_factor", ctypes.c_float), ("max_tokens", ctypes.c_int32),
                ("flags", ctypes.c_uint32), ("device", ctypes.c_int32),
                ("timeout_ns", ctypes.c_int64), ("claim_batch", ctypes.c_int32)]


class moe_shared_w(ctypes.Structure):
    _fields_ = [("up", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("down", ctypes.c_void_p)]


class moe_mxfp8_mat(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class moe_mxfp8_experts(ctypes.Structure):
    _fields_ = [(n, moe_mxfp8_mat) for n in ("up", "gate", "down", "shared_up", "shared_gate", "shared_down")]


class moe_ffn_grads(ctypes.Structure):
    _fields_ = [("up", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("down", ctypes.c_void_p)]


class moe_int4_mat(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


_INT4_FIELDS = ("up", "gate", "down", "shared_up", "shared_gate", "shared_down")


class moe_int4_experts(ctypes.Structure):
    _fields_ = [(n, moe_int4_mat) for n in _INT4_FIELDS] + [("group", ctypes.c_int32), ("zeros", ctypes.c_int32)]


# every symbol the header declares, with its C signature
_P, _I32, _I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
SIGNATURES = {
    "moe_init": (ctypes.c_int, [ctypes.POINTER(moe_config), ctypes.POINTER(ctypes.c_void_p)]),
    "moe_destroy": (None, [_P]),
    "moe_forward": (ctypes.c_int, [_P, _P, _I32, _P, _P, _P, _P, _P, ctypes.POINTER(moe_shared_w),
                                   _I32, _P, _P]),
    "moe_forward_host": (ctypes.c_int, [_P, _P, _I32, _P, _P, _P, _P, _P,
                                        ctypes.POINTER(moe_shared_w), _I32, _P, _P]),
    "moe_forward_host_async": (ctypes.c_int, [_P, _P, _I32, _P, _P, _P, _P, _P,
                                              ctypes.POINTER(moe_shared_w), _I32, _P, _P]),
    "moe_forward_host_join": (ctypes.c_int, [_P, _P, _I32]),
    "moe_get_status": (ctypes.c_int, [_P, ctypes.POINTER(ctypes.c_int32)]),
    "moe_mxfp8_scale_bytes": (_I64, [_I64, _I64]),
    "moe_quantize_mxfp8": (ctypes.c_int, [_P, _P, _I64, _I64, _P, _P, _P]),
    "moe_forward_mxfp8": (ctypes.c_int, [_P, _P, _I32, _P, _P, ctypes.POINTER(moe_mxfp8_experts), _I32, _P, _P]),
    "moe_int4_code_bytes": (_I64, [_I64, _I64]),
    "moe_int4_scale_bytes": (_I64, [_I64, _I64, _I32, _I32]),
    "moe_quantize_int4": (ctypes.c_int, [_P, _P, _I64, _I64, _I32, _I32, _P, _P, _P]),
    "moe_pack_int4": (ctypes.c_int, [_P, _P, _P, _P, _I64, _I64, _I32, _P, _P, _P]),
    "moe_matvec_int4": (ctypes.c_int, [_P, _P, _I64, ctypes.POINTER(moe_int4_mat), _I64, _I64, _I32, _I32, _P, _I32,
                                       _P]),
    "moe_experts_int4": (ctypes.c_int, [_P, _P, _I32, _P, _P, _I32, ctypes.POINTER(moe_int4_experts), _P, _I32, _P]),
    "moe_forward_int4": (ctypes.c_int, [_P, _P, _I32, _P, _P, ctypes.POINTER(moe_int4_experts), _I32, _P, _P]),
    "moe_ffn_workspace_bytes": (_I64, [_I64, _I32, _I32, _I32]),
    "moe_ffn_forward": (ctypes.c_int, [_P, _P, _I64, _I32, _I32, ctypes.POINTER(moe_shared_w), _P, _I32, _P, _P,
                                       _P, _I64, _P]),
    "moe_ffn_backward": (ctypes.c_int, [_P, _P, _P, _P, _P, _I64, _I32, _I32, ctypes.POINTER(moe_shared_w), _P,
                                        ctypes.POINTER(moe_ffn_grads), ctypes.c_uint32, _P, _I64, _P]),
    "moe_router_logits": (ctypes.c_int, [_P, _P, _I32, _P, _P, _P, _P]),
    "moe_gate_topk": (ctypes.c_int, [_P, _P, _I32, _I32, _P, _P, _P]),
    "moe_align_block_size": (ctypes.c_int, [_P, _P, _I32, _I32, _P, _P, _P, _P]),
    "moe_sorted_len": (_I64, [_P, _I32, _I32]),
    "moe_blocks_len": (_I64, [_P, _I32, _I32]),
    "moe_debug_outputs": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P]),
    "moe_debug_expert_rows": (ctypes.c_int, [_P, _P, _P, _P, _P, _P]),
    "moe_stage_times": (ctypes.c_int, [_P, ctypes.POINTER(ctypes.c_float), _I32]),
    "moe_query": (ctypes.c_int, [_P, _I32, ctypes.POINTER(ctypes.c_int64)]),
    "moe_trace_read": (ctypes.c_int, [_P, _P, _I64, ctypes.POINTER(ctypes.c_int64)]),
    "moe_debug_inject_stall": (ctypes.c_int, [_P, _I32]),
    "moe_trace_waits": (ctypes.c_int, [_P, _P, _I32, ctypes.POINTER(ctypes.c_int32)]),
    "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "moe_align_block_size_noalloc": (ctypes.c_int, [_P, _I32, _I32, _I32, _I32, ctypes.c_float, _P, _P, _P,
                                                    _P]),
}


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m mixture_experts_layer_block_b200.build` "
            "(there is no CPU fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


lib = _load()


def align_block_size_noalloc(topk_ids, num_experts, block_m, capacity_factor, sorted_ids, expert_ids,
                             num_post_padded, stream=None):
    """moe_align_block_size_noalloc on torch CUDA tensors (no handle, no allocation)."""
    T, k = topk_ids.shape
    check(lib.moe_align_block_size_noalloc(_ptr(topk_ids), T, k, num_experts, block_m, float(capacity_factor),
                                           _ptr(sorted_ids), _ptr(expert_ids), _ptr(num_post_padded),
                                           _stream(stream)), "moe_align_block_size_noalloc")


class MoEError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {lib.moe_status_string(code).decode()} ({code})")
        self.code = code


def check(code: int, where: str) -> int:
    if code != MOE_OK:
        raise MoEError(code, where)
    return code


# ------------------------------------------------------------------------------------------
# torch-facing convenience (marshalling only)
# ------------------------------------------------------------------------------------------

def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


# the dtypes that a tensor may have; filled when the first tensor is looked at, which is when torch is there
_BF16, _F32, _U8, _I32S, _BF16_F32 = [], [], [], [], []


def _fill_dtypes():
    import torch
    _BF16[:], _F32[:], _U8[:], _I32S[:] = [torch.bfloat16], [torch.float32], [torch.uint8], [torch.int32]
    _BF16_F32[:] = [torch.bfloat16, torch.float32]


def _is_tensor(t, name, shape, dtypes, device):
    """Raises unless t is a contiguous CUDA tensor of this shape and one of these dtypes on this
    device: the library sees only its address."""
    try:  # the common case in as few reads as it takes: a small call is as long as its checks
        if t.dtype in dtypes and t.shape == shape and t.is_contiguous() and t.get_device() == device:
            return
    except AttributeError:
        pass
    if not dtypes:
        _fill_dtypes()
        return _is_tensor(t, name, shape, dtypes, device)
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor, got {type(t).__name__}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d).split('.')[-1] for d in dtypes)}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must be on cuda:{device}, got {t.device}")


def _addr(t):
    return None if t is None else t.data_ptr()


def _current_raw_stream(device):
    """The handle of the device's current stream. The first call puts torch's own function in this one's place,
    which makes no Stream object (1 us less a call), where torch has it."""
    global _current_raw_stream
    import torch
    _current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
        (lambda device: torch.cuda.current_stream(device).cuda_stream)
    return _current_raw_stream(device)


def _raw_stream(stream, device):
    """The cudaStream_t of `stream`, or of the device's current stream."""
    return _current_raw_stream(device) if stream is None else stream.cuda_stream


class Int4Matrix:
    """A matrix [rows, cols] in 4 bits, in the library's layout (include/moe_b200.h): its codes and
    scales as uint8 CUDA tensors. Made by MoELayer.quantize_int4 or MoELayer.pack_int4."""
    __slots__ = ("codes", "scales", "rows", "cols", "group", "zeros", "device", "c")

    def __init__(self, rows, cols, group, zeros, device):
        nc, ns = lib.moe_int4_code_bytes(rows, cols), lib.moe_int4_scale_bytes(rows, cols, group, 1 if zeros else 0)
        if nc < 0 or ns < 0:
            raise ValueError("4-bit matrices have columns in a multiple of 8 and groups of 32, 64 or 128 columns: "
                             f"got {rows}x{cols} with groups of {group}")
        import torch
        self.codes = torch.empty(nc, dtype=torch.uint8, device=device)
        self.scales = torch.empty(ns, dtype=torch.uint8, device=device)
        self.rows, self.cols, self.group, self.zeros = rows, cols, group, 1 if zeros else 0
        self.device = self.codes.get_device()
        self.c = moe_int4_mat(self.codes.data_ptr(), self.scales.data_ptr())


class MoELayer:
    """Owns one moe_handle. Tensors are torch CUDA tensors laid out as include/moe_b200.h
    states (x [T,H] bf16, W_router [E,H], W_up/W_gate [E,D,H], W_down [E,H,D] bf16, bias [E]
    fp32, out [T,H] fp32, or bf16 with MOE_FLAG_OUT_BF16)."""

    def __init__(self, hidden, inter, num_experts, top_k, block_m, max_tokens, inter_shared=0,
                 capacity_factor=0.0, flags=0, device=-1, timeout_ns=0, claim_batch=0):
        self.cfg = moe_config(hidden, inter, inter_shared, num_experts, top_k, block_m,
                              float(capacity_factor), max_tokens, flags, device, timeout_ns,
                              claim_batch)
        h = ctypes.c_void_p()
        check(lib.moe_init(ctypes.byref(self.cfg), ctypes.byref(h)), "moe_init")
        self.h = h
        self.device = self.query(13)
        self.out_dtype = "bfloat16" if flags & MOE_FLAG_OUT_BF16 else "float32"

    def _check_out(self, out):
        # the library writes out in the dtype the handle was configured for
        dt = getattr(out, "dtype", None)
        if dt is not None and str(dt).split(".")[-1] != self.out_dtype:
            raise TypeError(f"out must be {self.out_dtype} for this handle, got {dt}")

    @classmethod
    def for_workload(cls, w, max_tokens=None, **kw):
        return cls(w.H, w.D, w.E, w.top_k, w.block_m, max_tokens or w.T, inter_shared=w.D_shared,
                   capacity_factor=w.capacity_factor, **kw)

    def close(self):
        if getattr(self, "h", None):
            lib.moe_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _shared(self, wts):
        if wts.get("Ws_up") is None:
            return None
        s = moe_shared_w(wts["Ws_up"].data_ptr(), wts["Ws_gate"].data_ptr(), wts["Ws_down"].data_ptr())
        return ctypes.byref(s), s

    def forward(self, x, wts, out, top_k=None, stream=None):
        self._check_out(out)
        sh = self._shared(wts)
        check(lib.moe_forward(self.h, _ptr(x), x.shape[0], _ptr(wts["W_router"]), _ptr(wts.get("bias")),
                              _ptr(wts["W_up"]), _ptr(wts["W_gate"]), _ptr(wts["W_down"]),
                              sh[0] if sh else None, top_k or self.cfg.top_k, _ptr(out),
                              _stream(stream)), "moe_forward")
        return out

    def forward_host(self, x_host, wts, out_host, top_k=None, stream=None):
        self._check_out(out_host)
        sh = self._shared(wts)
        check(lib.moe_forward_host(self.h, _ptr(x_host), x_host.shape[0], _ptr(wts["W_router"]),
                                   _ptr(wts.get("bias")), _ptr(wts["W_up"]), _ptr(wts["W_gate"]),
                                   _ptr(wts["W_down"]), sh[0] if sh else None, top_k or self.cfg.top_k,
                                   _ptr(out_host), _stream(stream)), "moe_forward_host")
        return out_host

    def forward_host_async(self, x_host, wts, out_host, top_k=None, stream=None):
        """Queue a host-buffer forward; consecutive calls overlap their copies with the
        previous forward. x_host / out_host must stay alive until forward_host_join."""
        self._check_out(out_host)
        sh = self._shared(wts)
        check(lib.moe_forward_host_async(self.h, _ptr(x_host), x_host.shape[0], _ptr(wts["W_router"]),
                                         _ptr(wts.get("bias")), _ptr(wts["W_up"]), _ptr(wts["W_gate"]),
                                         _ptr(wts["W_down"]), sh[0] if sh else None,
                                         top_k or self.cfg.top_k, _ptr(out_host), _stream(stream)),
              "moe_forward_host_async")
        return out_host

    # ---- 4-bit weights ----
    def quantize_int4(self, src, group=128, zeros=False, stream=None):
        """moe_quantize_int4 of a bf16 CUDA matrix [R, K] (a 3-D tensor is viewed as [-1, K])."""
        shape = getattr(src, "shape", ())
        if len(shape) < 2:
            raise ValueError("src must be a matrix or a stack of them")
        # no copy is made of a strided tensor: nothing would order it with `stream`
        _is_tensor(src, "src", shape, _BF16, self.device)
        out = self._int4_matrix(math.prod(shape[:-1]), shape[-1], group, zeros, stream)
        check(lib.moe_quantize_int4(self.h, src.data_ptr(), out.rows, out.cols, group, 1 if zeros else 0, out.c.codes,
                                    out.c.scales, _raw_stream(stream, self.device)), "moe_quantize_int4")
        return out

    def pack_int4(self, q, scales, zeros=None, group=128, stream=None):
        """moe_pack_int4: the library's layout of a matrix quantised elsewhere. q uint8 [R, K/2] (the
        even column in a byte's low half), scales bf16 [R, ceil(K/group)], zeros uint8 like scales
        or None."""
        if getattr(q, "ndim", 0) != 2:
            raise ValueError("q must be [R, K / 2]")
        rows, cols = q.shape[0], 2 * q.shape[1]
        out = self._int4_matrix(rows, cols, group, zeros is not None, stream)
        _is_tensor(q, "q", (rows, cols // 2), _U8, self.device)
        _is_tensor(scales, "scales", (rows, -(-cols // group)), _BF16, self.device)
        if zeros is not None:
            _is_tensor(zeros, "zeros", (rows, -(-cols // group)), _U8, self.device)
        check(lib.moe_pack_int4(self.h, q.data_ptr(), scales.data_ptr(), _addr(zeros), rows, cols, group, out.c.codes,
                                out.c.scales, _raw_stream(stream, self.device)), "moe_pack_int4")
        return out

    def _int4_matrix(self, rows, cols, group, zeros, stream):
        device = f"cuda:{self.device}"
        if stream is None:
            return Int4Matrix(rows, cols, group, zeros, device)
        import torch
        with torch.cuda.stream(stream):
            return Int4Matrix(rows, cols, group, zeros, device)

    def quantize_experts_int4(self, wts, group=128, zeros=False, stream=None):
        """The experts of a weight dict (W_up, W_gate, W_down and, with a shared expert, Ws_up, Ws_gate,
        Ws_down) as {name: Int4Matrix}."""
        names = ["W_up", "W_gate", "W_down"] + (["Ws_up", "Ws_gate", "Ws_down"] if wts.get("Ws_up") is not None else [])
        return {n: self.quantize_int4(wts[n], group, zeros, stream) for n in names}

    def matvec_int4(self, x, w, out, stream=None):
        """moe_matvec_int4: out [T, rows] (bf16 or fp32) = x [T, cols] (bf16) times the Int4Matrix w."""
        if not isinstance(w, Int4Matrix):
            raise TypeError(f"w must be an Int4Matrix, got {type(w).__name__}")
        if getattr(x, "ndim", 0) != 2:
            raise ValueError("x must be [T, cols]")
        T = x.shape[0]
        _is_tensor(x, "x", (T, w.cols), _BF16, self.device)
        _is_tensor(out, "out", (T, w.rows), _BF16_F32, self.device)
        if w.device != self.device:
            raise ValueError(f"w must be on cuda:{self.device}, got cuda:{w.device}")
        check(lib.moe_matvec_int4(self.h, x.data_ptr(), T, w.c, w.rows, w.cols, w.group, w.zeros, out.data_ptr(),
                                  1 if out.element_size() == 2 else 0, _raw_stream(stream, self.device)), "moe_matvec_int4")
        return out

    _EXPERT_NAMES = ("W_up", "W_gate", "W_down", "Ws_up", "Ws_gate", "Ws_down")

    def _int4_experts(self, wq):
        """The C struct of {name: Int4Matrix}, each checked against the layer's sizes."""
        cfg, dev = self.cfg, self.device
        H, D, E, Ds = cfg.hidden, cfg.inter, cfg.num_experts, cfg.inter_shared
        sizes = ((E * D, H), (E * D, H), (E * H, D), (Ds, H), (Ds, H), (H, Ds))
        out = moe_int4_experts()
        group = zeros = None
        for n, field, (rows, cols) in zip(self._EXPERT_NAMES, _INT4_FIELDS, sizes if Ds > 0 else sizes[:3]):
            w = wq.get(n)
            if not isinstance(w, Int4Matrix):
                raise TypeError(f"{n} must be an Int4Matrix, got {type(w).__name__}")
            if w.rows != rows or w.cols != cols:
                raise ValueError(f"{n} must be {rows}x{cols}, got {w.rows}x{w.cols}")
            if group is None:
                group, zeros = w.group, w.zeros
            elif w.group != group or w.zeros != zeros:
                raise ValueError("the experts' matrices must share their group size, and have zero points or none")
            if w.device != dev:
                raise ValueError(f"{n} must be on cuda:{dev}, got cuda:{w.device}")
            setattr(out, field, w.c)
        out.group, out.zeros = group, zeros
        return out

    def experts_int4(self, x, topk_ids, topk_w, wq, out, stream=None):
        """moe_experts_int4: the layer behind its gating. x [T, H] bf16 (T <= 16), topk_ids [T, k]
        int32, topk_w [T, k] fp32, wq {name: Int4Matrix} as quantize_experts_int4 returns, out [T, H]
        bf16 or fp32."""
        w = self._int4_experts(wq)
        if getattr(x, "ndim", 0) != 2 or getattr(topk_ids, "ndim", 0) != 2:
            raise ValueError("x must be [T, H] and topk_ids [T, k]")
        T, k = topk_ids.shape
        _is_tensor(x, "x", (T, self.cfg.hidden), _BF16, self.device)
        _is_tensor(topk_ids, "topk_ids", (T, k), _I32S, self.device)
        _is_tensor(topk_w, "topk_w", (T, k), _F32, self.device)
        _is_tensor(out, "out", (T, self.cfg.hidden), _BF16_F32, self.device)
        check(lib.moe_experts_int4(self.h, x.data_ptr(), T, topk_ids.data_ptr(), topk_w.data_ptr(), k, w,
                                   out.data_ptr(), 1 if out.element_size() == 2 else 0,
                                   _raw_stream(stream, self.device)), "moe_experts_int4")
        return out

    def forward_int4(self, x, w_router, bias, wq, out, top_k=None, stream=None):
        """moe_forward_int4: wq as quantize_experts_int4 returns; out in the handle's dtype."""
        w = self._int4_experts(wq)
        E, H = self.cfg.num_experts, self.cfg.hidden
        if getattr(x, "ndim", 0) != 2:
            raise ValueError("x must be [T, H]")
        T = x.shape[0]
        _is_tensor(x, "x", (T, H), _BF16, self.device)
        _is_tensor(w_router, "w_router", (E, H), _BF16, self.device)
        if bias is not None:
            _is_tensor(bias, "bias", (E,), _F32, self.device)
        _is_tensor(out, "out", (T, H), _BF16 if self.out_dtype == "bfloat16" else _F32, self.device)
        check(lib.moe_forward_int4(self.h, x.data_ptr(), T, w_router.data_ptr(), _addr(bias), w,
                                   top_k or self.cfg.top_k, out.data_ptr(), _raw_stream(stream, self.device)),
              "moe_forward_int4")
        return out

    # ---- the gated feed-forward block ----
    def _ffn_call(self, x, wts):
        """(T, H, D, the C struct of the weights) of a block's call, its input and weights checked."""
        up, gate, down = wts.get("Ws_up"), wts.get("Ws_gate"), wts.get("Ws_down")
        if up is None or gate is None or down is None:
            raise ValueError("the block needs Ws_up, Ws_gate and Ws_down")
        if getattr(up, "ndim", 0) != 2 or getattr(x, "ndim", 0) != 2:
            raise ValueError("x must be [T, H] and Ws_up [D, H]")
        (T, H), D, dev = x.shape, up.shape[0], self.device
        _is_tensor(x, "x", (T, H), _BF16, dev)
        _is_tensor(up, "Ws_up", (D, H), _BF16, dev)
        _is_tensor(gate, "Ws_gate", (D, H), _BF16, dev)
        _is_tensor(down, "Ws_down", (H, D), _BF16, dev)
        return T, H, D, moe_shared_w(up.data_ptr(), gate.data_ptr(), down.data_ptr())

    def _ffn_workspace(self, workspace, need, x, stream):
        """Address and bytes of the caller's workspace, or of one for this call alone (allocated in the
        order of the call's stream, so that its memory is reused only behind the call); and its owner."""
        if workspace is not None:
            _is_tensor(workspace, "workspace", getattr(workspace, "shape", None), _U8, self.device)
            if workspace.numel() < need:
                raise ValueError(f"the workspace needs {need} bytes, got {workspace.numel()}")
        elif stream is None:
            workspace = x.new_empty(need >> 1)  # of x's 2-byte type: the cheapest allocation there is
        else:
            import torch
            with torch.cuda.stream(stream):
                workspace = x.new_empty(need >> 1)
        return workspace.data_ptr(), workspace.nbytes, workspace

    @staticmethod
    @functools.lru_cache(maxsize=4096)
    def ffn_workspace_bytes(T, hidden, inter, backward=False):
        """Bytes of the workspace of ffn_forward or ffn_backward (a uint8 tensor)."""
        n = lib.moe_ffn_workspace_bytes(T, hidden, inter, 1 if backward else 0)
        if n < 0:
            raise ValueError("the block's hidden and inner sizes are multiples of 8 up to 2^20, its tokens at most "
                             f"2^24: got {hidden}, {inter} and {T}")
        return n

    def ffn_forward(self, x, wts, out, u=None, g=None, workspace=None, stream=None):
        """moe_ffn_forward: out = W_down (SiLU(W_up x) * (W_gate x)) with wts["Ws_up"] and
        wts["Ws_gate"] [D, H] and wts["Ws_down"] [H, D]; x [T, H] bf16, out [T, H] bf16 or fp32.
        u and g ([T, D] bf16, both or neither) receive the pre-activations for ffn_backward."""
        T, H, D, w = self._ffn_call(x, wts)
        _is_tensor(out, "out", (T, H), _BF16_F32, self.device)
        if u is not None or g is not None:
            if u is None or g is None:
                raise ValueError("u and g go together")
            _is_tensor(u, "u", (T, D), _BF16, self.device)
            _is_tensor(g, "g", (T, D), _BF16, self.device)
        ws, nbytes, owner = self._ffn_workspace(workspace, self.ffn_workspace_bytes(T, H, D), x, stream)
        check(lib.moe_ffn_forward(self.h, x.data_ptr(), T, H, D, w, out.data_ptr(), 1 if out.element_size() == 2 else 0,
                                  _addr(u), _addr(g), ws, nbytes, _raw_stream(stream, self.device)),
              "moe_ffn_forward")
        return out

    _GRADS = frozenset(("x", "Ws_up", "Ws_gate", "Ws_down"))
    _WEIGHT_GRADS = tuple((n, f"grads[{n!r}]") for n in ("Ws_up", "Ws_gate", "Ws_down"))

    def ffn_backward(self, dout, x, u, g, wts, grads, accumulate=False, workspace=None, stream=None):
        """moe_ffn_backward: fills grads["x"] ([T, H] bf16) and grads["Ws_up"], grads["Ws_gate"],
        grads["Ws_down"] (shaped as the weights, all bf16 or all fp32; with accumulate, fp32 and
        added to). A gradient that grads lacks, or has as None, is not computed."""
        T, H, D, w = self._ffn_call(x, wts)
        dev = self.device
        _is_tensor(dout, "dout", (T, H), _BF16, dev)
        _is_tensor(u, "u", (T, D), _BF16, dev)
        _is_tensor(g, "g", (T, D), _BF16, dev)
        if not grads.keys() <= self._GRADS:
            raise ValueError(f"gradients are named x, Ws_up, Ws_gate and Ws_down, got {sorted(grads)}")
        dx = grads.get("x")
        if dx is not None:
            _is_tensor(dx, "grads['x']", (T, H), _BF16, dev)
        first, addr = None, []
        for n, name in self._WEIGHT_GRADS:
            t = grads.get(n)
            if t is not None:
                _is_tensor(t, name, wts[n].shape, _F32 if accumulate else _BF16_F32, dev)
                first = t if first is None else first
                if t.dtype != first.dtype:
                    raise TypeError("the weight gradients must all be bfloat16 or all float32")
            addr.append(_addr(t))
        flags = 0 if first is None or first.element_size() == 2 else MOE_FFN_GRAD_F32 | (MOE_FFN_GRAD_ADD if accumulate else 0)
        ws, nbytes, owner = self._ffn_workspace(workspace, self.ffn_workspace_bytes(T, H, D, True), x, stream)
        check(lib.moe_ffn_backward(self.h, dout.data_ptr(), x.data_ptr(), u.data_ptr(), g.data_ptr(), T, H, D, w,
                                   _addr(dx), moe_ffn_grads(*addr), flags, ws, nbytes, _raw_stream(stream, dev)), "moe_ffn_backward")
        return grads

    # ---- MXFP8 experts ----
    def quantize_mxfp8(self, src, stream=None):
        """MXFP8 of a bf16 CUDA matrix [R, K] (a 3-D tensor is viewed as [-1, K]): returns
        (codes uint8 [R, K], scales uint8 [R*K/32] in the header's atom layout)."""
        import torch
        m = src.reshape(-1, src.shape[-1])
        R, K = m.shape
        nb = lib.moe_mxfp8_scale_bytes(R, K)
        if nb < 0:
            raise ValueError(f"MXFP8 needs both dimensions multiples of 128, got {R}x{K}")
        q = torch.empty(R, K, dtype=torch.uint8, device=src.device)
        sf = torch.empty(nb, dtype=torch.uint8, device=src.device)
        check(lib.moe_quantize_mxfp8(self.h, _ptr(m), R, K, _ptr(q), _ptr(sf), _stream(stream)),
              "moe_quantize_mxfp8")
        return q, sf

    def quantize_experts_mxfp8(self, wts, stream=None):
        """The quantised experts of a weight dict (keys W_up, W_gate, W_down and, with a
        shared expert, Ws_up, Ws_gate, Ws_down) as {name: (codes, scales)}."""
        names = ["W_up", "W_gate", "W_down"] + (["Ws_up", "Ws_gate", "Ws_down"] if wts.get("Ws_up") is not None else [])
        return {n: self.quantize_mxfp8(wts[n], stream) for n in names}

    def forward_mxfp8(self, x, w_router, bias, wq, out, top_k=None, stream=None):
        """moe_forward_mxfp8: wq as returned by quantize_experts_mxfp8 (needs MOE_FLAG_MXFP8)."""
        self._check_out(out)
        mats = []
        for n in ("W_up", "W_gate", "W_down", "Ws_up", "Ws_gate", "Ws_down"):
            q, sf = wq.get(n, (None, None))
            mats.append(moe_mxfp8_mat(None if q is None else q.data_ptr(), None if sf is None else sf.data_ptr()))
        ex = moe_mxfp8_experts(*mats)
        check(lib.moe_forward_mxfp8(self.h, _ptr(x), x.shape[0], _ptr(w_router), _ptr(bias), ctypes.byref(ex),
                                    top_k or self.cfg.top_k, _ptr(out), _stream(stream)), "moe_forward_mxfp8")
        return out

    def forward_host_join(self, stream=None, block=True):
        check(lib.moe_forward_host_join(self.h, _stream(stream), 1 if block else 0), "moe_forward_host_join")

    def router_logits(self, x, w_router, bias, logits, stream=None):
        check(lib.moe_router_logits(self.h, _ptr(x), x.shape[0], _ptr(w_router), _ptr(bias), _ptr(logits),
                                    _stream(stream)), "moe_router_logits")
        return logits

    def gate_topk(self, logits, top_k, ids, w, stream=None):
        check(lib.moe_gate_topk(self.h, _ptr(logits), logits.shape[0], top_k, _ptr(ids), _ptr(w),
                                _stream(stream)), "moe_gate_topk")
        return ids, w

    def align(self, topk_ids, sorted_ids, expert_ids, npp, stream=None):
        T, k = topk_ids.shape
        check(lib.moe_align_block_size(self.h, _ptr(topk_ids), T, k, _ptr(sorted_ids), _ptr(expert_ids),
                                       _ptr(npp), _stream(stream)), "moe_align_block_size")

    def sorted_len(self, T, k):
        return int(lib.moe_sorted_len(self.h, T, k))

    def blocks_len(self, T, k):
        return int(lib.moe_blocks_len(self.h, T, k))

    def debug_outputs(self, T, k, device, stream=None):
        import torch
        E = self.cfg.num_experts
        d = {"logits": torch.empty((T, E), dtype=torch.float32, device=device),
             "topk_ids": torch.empty((T, k), dtype=torch.int32, device=device),
             "topk_w": torch.empty((T, k), dtype=torch.float32, device=device),
             "sorted_ids": torch.empty((self.sorted_len(T, k),), dtype=torch.int32, device=device),
             "expert_ids": torch.empty((self.blocks_len(T, k),), dtype=torch.int32, device=device),
             "num_post_padded": torch.empty((1,), dtype=torch.int32, device=device)}
        check(lib.moe_debug_outputs(self.h, *(_ptr(d[n]) for n in ("logits", "topk_ids", "topk_w",
                                                                    "sorted_ids", "expert_ids",
                                                                    "num_post_padded")),
                                    _stream(stream)), "moe_debug_outputs")
        return d

    def debug_expert_rows(self, T, k, device, with_h=True, stream=None):
        """moe_debug_expert_rows: the GEMM rows of the last forward, as torch tensors (h and y
        bf16 [rows, ...], row_of_slot int32 [T*k], num_routed_tiles int)."""
        import torch
        rows, ldh = self.query(9), self.query(10)
        d = {"h": torch.empty((rows, ldh), dtype=torch.bfloat16, device=device) if with_h else None,
             "y": torch.empty((rows, self.cfg.hidden), dtype=torch.bfloat16, device=device),
             "row_of_slot": torch.empty((T * k,), dtype=torch.int32, device=device),
             "num_routed_tiles": torch.empty((1,), dtype=torch.int32, device=device)}
        check(lib.moe_debug_expert_rows(self.h, _ptr(d["h"]), _ptr(d["y"]), _ptr(d["row_of_slot"]),
                                        _ptr(d["num_routed_tiles"]), _stream(stream)), "moe_debug_expert_rows")
        return d

    def status(self):
        st = ctypes.c_int32(0)
        rc = lib.moe_get_status(self.h, ctypes.byref(st))
        return rc, st.value

    STAGES = ("router", "gating", "align_scatter", "row_gather", "expert_gemm", "combine")

    def stage_times(self):
        ms = (ctypes.c_float * 6)()
        check(lib.moe_stage_times(self.h, ms, 6), "moe_stage_times")
        return list(ms)

    def query(self, which):
        v = ctypes.c_int64(0)
        check(lib.moe_query(self.h, which, ctypes.byref(v)), "moe_query")
        return v.value

    def trace(self, cap):
        import numpy as np
        buf = np.zeros((cap, 4), dtype=np.int64)
        n = ctypes.c_int64(0)
        check(lib.moe_trace_read(self.h, buf.ctypes.data_as(ctypes.c_void_p), cap, ctypes.byref(n)),
              "moe_trace_read")
        return buf[: n.value]

    WAITS = ("prod_empty", "prod_dep", "prod_ring", "prod_claim", "mma_full", "mma_acc", "mma_task",
             "epi_task", "epi_acc", "prod_loop", "mma_loop", "epi_loop", "front_router", "front_schedule",
             "front_gather", "front_last", "front_to_end", "sched_arrive", "sched_logits", "sched_gating",
             "sched_tables", "sched_writes", "sched_publish", "combine_count", "combine_run")

    def trace_waits(self):
        """moe_trace_waits: [CTAs, 25] int64 ns (columns named by WAITS)."""
        import numpy as np
        buf = np.zeros((1024, len(self.WAITS)), dtype=np.int64)
        n = ctypes.c_int32(0)
        check(lib.moe_trace_waits(self.h, buf.ctypes.data_as(ctypes.c_void_p), 1024, ctypes.byref(n)),
              "moe_trace_waits")
        return buf[: n.value]

    def inject_stall(self, extra):
        check(lib.moe_debug_inject_stall(self.h, extra), "moe_debug_inject_stall")
