"""Python binding of the B200 MoE-layer library (include/moe.h).

Argument marshalling only: every function here forwards to the C ABI entry
point of the same name in libmoe_b200.so, passing torch tensors' device
addresses.  There is no fallback: if the library is missing or a call fails,
an exception is raised.  PyTorch supplies device memory and streams.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_b200.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = -1
MOE_ERR_UNSUPPORTED = -2
MOE_ERR_WORKSPACE = -3
MOE_ERR_CUDA = -4
MOE_ERR_DEVICE = -5

MOE_W_BF16 = 0
MOE_W_FP8_E4M3_B128 = 1

MOE_DEV_WAIT_TIMEOUT_GATE_UP = 0x1
MOE_DEV_WAIT_TIMEOUT_DOWN = 0x2
MOE_DEV_BAD_EXPERT_ID = 0x4
MOE_DEV_WAIT_TIMEOUT_ROUTER = 0x8
MOE_DEV_WAIT_TIMEOUT_SEND = 0x10
MOE_DEV_WAIT_TIMEOUT_FEW = 0x20
MOE_DEV_WAIT_TIMEOUT_PRODUCT = 0x40

MOE_T_BF16 = 0
MOE_T_FP32 = 1

MOE_FEW_TOKENS_MAX = 16

MOE_NUM_STAGES = 7
STAGE_NAMES = ("router", "topk", "permute", "gather", "gate_up_gemm", "down_gemm", "combine")

EXPORTED = ("moe_plan_create", "moe_plan_destroy", "moe_plan_set_wait_limit", "moe_forward",
            "moe_forward_scatter", "moe_forward_scatter_experts", "moe_reduce_partials",
            "moe_route_from_logits", "moe_route_from_logits_noalloc", "moe_check_device_status",
            "moe_get_workspace_views", "moe_status_string", "moe_last_cuda_error_string",
            "moe_pipeline_slot_bytes", "moe_pipeline_create", "moe_pipeline_submit",
            "moe_pipeline_synchronize", "moe_pipeline_streams", "moe_pipeline_destroy",
            "moe_router_split_bytes", "moe_split_router_weights", "moe_forward_scatter_pairs",
            "moe_reduce_pairs", "moe_forward_few", "moe_quantize_groups", "moe_product_create",
            "moe_product_destroy", "moe_product_set_wait_limit", "moe_block_scaled_product",
            "moe_product_device_status")
MAX_TP_RANKS = 8

MOE_STATIC_SCRATCH_BYTES = 4 << 20

_c_int = ctypes.c_int
_vp = ctypes.c_void_p


class moe_config(ctypes.Structure):
    _fields_ = [("max_tokens", _c_int), ("hidden", _c_int), ("num_experts", _c_int),
                ("top_k_max", _c_int), ("inter", _c_int), ("num_shared", _c_int),
                ("shared_inter", _c_int), ("renormalize", _c_int), ("wtype", _c_int)]


class moe_weights(ctypes.Structure):
    _fields_ = [("router_w", _vp), ("router_b", _vp), ("w_gate_up", _vp), ("w_down", _vp),
                ("s_gate_up", _vp), ("s_down", _vp), ("ws_gate_up", _vp), ("ws_down", _vp),
                ("ss_gate_up", _vp), ("ss_down", _vp), ("router_split", _vp)]


class moe_debug(ctypes.Structure):
    _fields_ = [("logits", _vp), ("topk_ids", _vp), ("topk_w", _vp), ("perm", _vp),
                ("offsets", _vp), ("events", _vp * (MOE_NUM_STAGES + 1))]


class moe_workspace_views(ctypes.Structure):
    _fields_ = [("row_token", _vp), ("x_perm", _vp), ("h", _vp), ("y", _vp),
                ("group_offsets", _vp), ("h_stride", _c_int), ("x_scale", _vp),
                ("h_scale", _vp)]


class moe_product_config(ctypes.Structure):
    _fields_ = [("max_rows", _c_int), ("n", _c_int), ("k", _c_int), ("out_type", _c_int)]


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        detail = f": {moe_last_cuda_error_string()}" if status == MOE_ERR_CUDA else ""
        super().__init__(f"{where}: {moe_status_string(status)} ({status}){detail}")


_lib = None


def load():
    """Loads libmoe_b200.so; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: run mixture_experts_fp32_b200.build.build()")
    L = ctypes.CDLL(LIB_PATH)
    L.moe_plan_create.argtypes = [ctypes.POINTER(moe_config), ctypes.POINTER(_vp),
                                  ctypes.POINTER(ctypes.c_size_t)]
    L.moe_plan_create.restype = _c_int
    L.moe_plan_destroy.argtypes = [_vp]
    L.moe_plan_destroy.restype = None
    L.moe_plan_set_wait_limit.argtypes = [_vp, ctypes.c_uint64]
    L.moe_plan_set_wait_limit.restype = _c_int
    L.moe_forward.argtypes = [_vp, ctypes.POINTER(moe_weights), _vp, _vp, _c_int, _c_int, _vp, _vp,
                              ctypes.c_size_t, _vp, ctypes.POINTER(moe_debug)]
    L.moe_forward.restype = _c_int
    L.moe_forward_scatter.argtypes = [_vp, ctypes.POINTER(moe_weights), _vp, _vp, _c_int, _c_int,
                                      ctypes.POINTER(_vp), _c_int, _c_int, _c_int, _vp,
                                      ctypes.c_size_t, _vp, ctypes.POINTER(moe_debug)]
    L.moe_forward_scatter.restype = _c_int
    L.moe_forward_scatter_experts.argtypes = [_vp, ctypes.POINTER(moe_weights), _vp, _vp, _c_int,
                                              _c_int, ctypes.POINTER(_vp), _c_int, _c_int, _c_int,
                                              _c_int, _c_int, _vp, ctypes.c_size_t, _vp,
                                              ctypes.POINTER(moe_debug)]
    L.moe_forward_scatter_experts.restype = _c_int
    L.moe_reduce_partials.argtypes = [_vp, _c_int, _c_int, _c_int, _vp, _vp, _vp]
    L.moe_reduce_partials.restype = _c_int
    L.moe_route_from_logits.argtypes = [_vp, _vp, _vp, _c_int, _c_int, _vp, _vp, _vp, _vp, _vp,
                                        ctypes.c_size_t, _vp]
    L.moe_route_from_logits.restype = _c_int
    L.moe_route_from_logits_noalloc.argtypes = [_vp, _vp, _vp, _c_int, _c_int, _vp, _vp, _vp,
                                                _vp, _vp]
    L.moe_route_from_logits_noalloc.restype = _c_int
    L.moe_check_device_status.argtypes = [_vp, _vp, _vp, ctypes.POINTER(ctypes.c_uint32)]
    L.moe_check_device_status.restype = _c_int
    L.moe_get_workspace_views.argtypes = [_vp, _vp, ctypes.POINTER(moe_workspace_views)]
    L.moe_get_workspace_views.restype = _c_int
    L.moe_status_string.argtypes = [_c_int]
    L.moe_status_string.restype = ctypes.c_char_p
    L.moe_last_cuda_error_string.argtypes = []
    L.moe_last_cuda_error_string.restype = ctypes.c_char_p
    L.moe_pipeline_slot_bytes.argtypes = [_vp, _c_int, _c_int, ctypes.POINTER(ctypes.c_size_t)]
    L.moe_pipeline_slot_bytes.restype = _c_int
    L.moe_pipeline_create.argtypes = [_vp, ctypes.POINTER(moe_weights), _c_int, _c_int, _c_int,
                                      _c_int, _vp, ctypes.c_size_t, _vp, ctypes.c_size_t,
                                      ctypes.POINTER(_vp)]
    L.moe_pipeline_create.restype = _c_int
    L.moe_pipeline_submit.argtypes = [_vp, _vp, _vp, _vp]
    L.moe_pipeline_submit.restype = _c_int
    L.moe_pipeline_synchronize.argtypes = [_vp]
    L.moe_pipeline_synchronize.restype = _c_int
    L.moe_pipeline_streams.argtypes = [_vp, ctypes.POINTER(_vp), ctypes.POINTER(_vp),
                                       ctypes.POINTER(_vp)]
    L.moe_pipeline_streams.restype = _c_int
    L.moe_forward_scatter_pairs.argtypes = [_vp, ctypes.POINTER(moe_weights), _vp, _vp, _c_int,
                                            _c_int, _vp, _c_int, _c_int, _c_int, _c_int,
                                            _c_int, _c_int, _vp, ctypes.c_size_t, _vp, _vp]
    L.moe_forward_scatter_pairs.restype = _c_int
    L.moe_reduce_pairs.argtypes = [_vp, _c_int, _c_int, _c_int, _c_int, _vp, _vp, _vp, _vp]
    L.moe_reduce_pairs.restype = _c_int
    L.moe_router_split_bytes.argtypes = [_vp]
    L.moe_router_split_bytes.restype = ctypes.c_size_t
    L.moe_split_router_weights.argtypes = [_vp, _vp, _vp, ctypes.c_size_t, _vp]
    L.moe_split_router_weights.restype = _c_int
    L.moe_forward_few.argtypes = [_vp, ctypes.POINTER(moe_weights), _vp, _vp, _c_int, _c_int, _vp,
                                  _vp, ctypes.c_size_t, _vp, ctypes.POINTER(moe_debug)]
    L.moe_forward_few.restype = _c_int
    L.moe_quantize_groups.argtypes = [_vp, _c_int, _c_int, _c_int, ctypes.c_int64, _c_int, _vp,
                                      _vp, _vp, _vp]
    L.moe_quantize_groups.restype = _c_int
    L.moe_product_create.argtypes = [ctypes.POINTER(moe_product_config), ctypes.POINTER(_vp),
                                     ctypes.POINTER(ctypes.c_size_t)]
    L.moe_product_create.restype = _c_int
    L.moe_product_destroy.argtypes = [_vp]
    L.moe_product_destroy.restype = None
    L.moe_product_set_wait_limit.argtypes = [_vp, ctypes.c_uint64]
    L.moe_product_set_wait_limit.restype = _c_int
    L.moe_block_scaled_product.argtypes = [_vp, _vp, _vp, _vp, _vp, _c_int, _vp, ctypes.c_int64,
                                           _vp, ctypes.c_size_t, _vp]
    L.moe_block_scaled_product.restype = _c_int
    L.moe_product_device_status.argtypes = [_vp, _vp, _vp, ctypes.POINTER(ctypes.c_uint32)]
    L.moe_product_device_status.restype = _c_int
    L.moe_pipeline_destroy.argtypes = [_vp]
    L.moe_pipeline_destroy.restype = None
    _lib = L
    return L


# element types accepted for each kind of tensor argument (torch dtype names)
_F32 = ("float32",)
_I32 = ("int32",)
_BF16 = ("bfloat16",)
_MASK = ("uint8", "bool")
_WEIGHT = ("bfloat16", "uint8", "float8_e4m3fn")
_CODES = ("uint8", "float8_e4m3fn")


_dtype_names: dict = {}          # torch dtype -> its name without "torch."


def _dtype_name(dtype) -> str:
    name = _dtype_names.get(dtype)
    if name is None:
        name = _dtype_names[dtype] = str(dtype).rsplit(".", 1)[-1]
    return name


def _addr(t, name: str = "argument", dtypes=None) -> int | None:
    """Address of a tensor argument, or an int taken as a raw address, or None.

    A tensor must be a contiguous CUDA tensor (of one of ``dtypes`` when given):
    the kernels read and write it as a dense row-major array in device memory, so a
    host tensor, a strided view or a wrong element type is refused here, before
    anything is enqueued, instead of being read out of bounds on the device."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError(f"{name}: a CUDA tensor is required, got one on {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous tensor is required")
    if dtypes is not None and _dtype_name(t.dtype) not in dtypes:
        raise ValueError(f"{name}: element type {t.dtype} is not one of {', '.join(dtypes)}")
    return t.data_ptr()


def _stream(s, device: int | None = None) -> int | None:
    """The handle of a stream, by default the current one of ``device`` (None: the current)."""
    if s is None:
        import torch
        # the current stream's handle without a Stream object around it, 3.5 us less a call (a
        # small quantisation takes 7.5); torch's name for it is private, so only where it exists
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is None:
            return torch.cuda.current_stream().cuda_stream
        return raw(torch.cuda.current_device() if device is None else device)
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(status: int, where: str):
    if status != MOE_OK:
        raise MoeError(status, where)


def moe_status_string(status: int) -> str:
    return load().moe_status_string(status).decode()


def moe_last_cuda_error_string() -> str:
    return load().moe_last_cuda_error_string().decode()


def moe_plan_create(cfg: moe_config):
    """Returns (plan handle, workspace bytes)."""
    plan = _vp()
    ws = ctypes.c_size_t()
    _check(load().moe_plan_create(ctypes.byref(cfg), ctypes.byref(plan), ctypes.byref(ws)),
           "moe_plan_create")
    return plan.value, ws.value


def moe_plan_destroy(plan) -> None:
    load().moe_plan_destroy(plan)


def moe_plan_set_wait_limit(plan, limit_ns: int) -> None:
    _check(load().moe_plan_set_wait_limit(plan, limit_ns), "moe_plan_set_wait_limit")


def make_weights(router_w, router_b=None, w_gate_up=None, w_down=None, s_gate_up=None,
                 s_down=None, ws_gate_up=None, ws_down=None, ss_gate_up=None,
                 ss_down=None, router_split=None) -> moe_weights:
    return moe_weights(_addr(router_w, "router_w", _F32), _addr(router_b, "router_b", _F32),
                       _addr(w_gate_up, "w_gate_up", _WEIGHT), _addr(w_down, "w_down", _WEIGHT),
                       _addr(s_gate_up, "s_gate_up", _F32), _addr(s_down, "s_down", _F32),
                       _addr(ws_gate_up, "ws_gate_up", _WEIGHT), _addr(ws_down, "ws_down", _WEIGHT),
                       _addr(ss_gate_up, "ss_gate_up", _F32), _addr(ss_down, "ss_down", _F32),
                       _addr(router_split, "router_split", _BF16))


def moe_router_split_bytes(plan) -> int:
    return int(load().moe_router_split_bytes(plan))


def moe_split_router_weights(plan, router_w, split, split_bytes: int, stream=None) -> None:
    _check(load().moe_split_router_weights(plan, _addr(router_w, "router_w", _F32),
                                           _addr(split, "split", _BF16), split_bytes,
                                           _stream(stream)), "moe_split_router_weights")


def make_debug(logits=None, topk_ids=None, topk_w=None, perm=None, offsets=None,
               events=None) -> moe_debug:
    d = moe_debug(_addr(logits, "logits", _F32), _addr(topk_ids, "topk_ids", _I32),
                  _addr(topk_w, "topk_w", _F32), _addr(perm, "perm", _I32),
                  _addr(offsets, "offsets", _I32))
    if events is not None:
        for i, ev in enumerate(events):
            d.events[i] = None if ev is None else ev.cuda_event
    return d


def moe_forward(plan, weights: moe_weights, hidden, valid, T: int, k: int, out, workspace,
                ws_bytes: int, stream=None, dbg: moe_debug | None = None) -> None:
    st = load().moe_forward(plan, ctypes.byref(weights), _addr(hidden, "hidden", _BF16),
                            _addr(valid, "valid", _MASK), T, k, _addr(out, "out", _BF16),
                            _addr(workspace, "workspace"), ws_bytes, _stream(stream),
                            None if dbg is None else ctypes.byref(dbg))
    _check(st, "moe_forward")


def moe_forward_scatter(plan, weights: moe_weights, hidden, valid, T: int, k: int, dst,
                        rows_per_rank: int, slot: int, workspace, ws_bytes: int, stream=None,
                        dbg: moe_debug | None = None) -> None:
    """dst: a sequence of device addresses (or tensors) of the owners' receive slabs."""
    arr = (_vp * len(dst))(*[_addr(d, "dst", _F32) for d in dst])
    st = load().moe_forward_scatter(plan, ctypes.byref(weights), _addr(hidden, "hidden", _BF16),
                                    _addr(valid, "valid", _MASK), T, k,
                                    arr, len(dst), rows_per_rank, slot, _addr(workspace, "workspace"),
                                    ws_bytes, _stream(stream),
                                    None if dbg is None else ctypes.byref(dbg))
    _check(st, "moe_forward_scatter")


def moe_forward_scatter_experts(plan, weights: moe_weights, hidden, valid, T: int, k: int, dst,
                                rows_per_rank: int, slot: int, expert_begin: int, expert_end: int,
                                workspace, ws_bytes: int, stream=None,
                                dbg: moe_debug | None = None) -> None:
    arr = (_vp * len(dst))(*[_addr(d, "dst", _F32) for d in dst])
    st = load().moe_forward_scatter_experts(plan, ctypes.byref(weights),
                                            _addr(hidden, "hidden", _BF16),
                                            _addr(valid, "valid", _MASK), T, k, arr, len(dst),
                                            rows_per_rank, slot, expert_begin, expert_end,
                                            _addr(workspace, "workspace"),
                                            ws_bytes, _stream(stream),
                                            None if dbg is None else ctypes.byref(dbg))
    _check(st, "moe_forward_scatter_experts")


def moe_forward_scatter_pairs(plan, weights: moe_weights, hidden, valid, T: int, k: int, dst,
                              rows_per_rank: int, shared_slot: int, expert_begin: int,
                              expert_end: int, send_ctas: int, workspace, ws_bytes: int,
                              stream=None, dbg: moe_debug | None = None) -> None:
    """dst: the owners' per-pair receive slabs (device addresses or tensors)."""
    arr = (_vp * len(dst))(*[_addr(d, "dst", _F32) for d in dst])
    st = load().moe_forward_scatter_pairs(plan, ctypes.byref(weights),
                                          _addr(hidden, "hidden", _BF16),
                                          _addr(valid, "valid", _MASK), T, k, arr, len(dst),
                                          rows_per_rank, shared_slot, expert_begin, expert_end,
                                          send_ctas, _addr(workspace, "workspace"), ws_bytes,
                                          _stream(stream),
                                          None if dbg is None else ctypes.byref(dbg))
    _check(st, "moe_forward_scatter_pairs")


def moe_reduce_pairs(slab, k: int, n_extra: int, rows: int, H: int, w, valid, out,
                     stream=None) -> None:
    st = load().moe_reduce_pairs(_addr(slab, "slab", _F32), k, n_extra, rows, H,
                                 _addr(w, "w", _F32), _addr(valid, "valid", _MASK),
                                 _addr(out, "out", _BF16), _stream(stream))
    _check(st, "moe_reduce_pairs")


def moe_forward_few(plan, weights: moe_weights, hidden, valid, T: int, k: int, out, workspace,
                    ws_bytes: int, stream=None, dbg: moe_debug | None = None) -> None:
    """moe_forward for T <= MOE_FEW_TOKENS_MAX tokens in one kernel."""
    st = load().moe_forward_few(plan, ctypes.byref(weights), _addr(hidden, "hidden", _BF16),
                                _addr(valid, "valid", _MASK), T, k, _addr(out, "out", _BF16),
                                _addr(workspace, "workspace"), ws_bytes, _stream(stream),
                                None if dbg is None else ctypes.byref(dbg))
    _check(st, "moe_forward_few")


def _on_current_device(tensors) -> int:
    """Every tensor on the current device, whose index is returned: the library launches there."""
    import torch
    cur = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != cur and t.is_cuda:
            raise ValueError(f"a tensor on {t.device}, while the current device is cuda:{cur}")
    return cur


def _rows_of(t, name: str, dtypes) -> tuple[int, int]:
    """(address, row stride in elements) of a 2-D CUDA tensor whose rows are contiguous;
    the rows themselves may lie further apart, as in a slice of a wider tensor."""
    if not t.is_cuda:
        raise ValueError(f"{name}: a CUDA tensor is required, got one on {t.device}")
    if _dtype_name(t.dtype) not in dtypes:
        raise ValueError(f"{name}: element type {t.dtype} is not one of {', '.join(dtypes)}")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: rows of consecutive elements are required")
    ld = t.stride(0) if rows > 1 else cols
    if ld < cols:
        raise ValueError(f"{name}: rows overlap (row stride {ld}, {cols} columns)")
    return t.data_ptr(), ld


def _groups(n: int) -> int:
    return (n + 127) // 128


def moe_quantize_groups(x, codes, scales, valid=None, gated: bool = False, stream=None) -> None:
    """e4m3 codes [rows, cols] (uint8 or float8_e4m3fn) and fp32 scales [rows,
    ceil(cols / 128)] of x [rows, cols] or, with ``gated``, of silu(g) * u for x = [g | u]
    [rows, 2 cols].  x: bf16 or fp32, rows may be strided; valid: uint8 or bool [rows],
    0 for padding rows, which get codes 0 and scales 1."""
    if x.dim() != 2 or codes.dim() != 2:
        raise ValueError("x and codes: two dimensions are required")
    rows, cols = codes.shape
    if x.shape != (rows, cols * (2 if gated else 1)):
        raise ValueError(f"x: shape {tuple(x.shape)} does not match codes {tuple(codes.shape)}"
                         f"{' and gated' if gated else ''}")
    if scales.shape != (rows, _groups(cols)):
        raise ValueError(f"scales: shape {tuple(scales.shape)}, needs {(rows, _groups(cols))}")
    if valid is not None and valid.shape != (rows,):
        raise ValueError(f"valid: shape {tuple(valid.shape)}, needs ({rows},)")
    addr, ld = _rows_of(x, "x", _BF16 + _F32)
    c, s, v = (_addr(codes, "codes", _CODES), _addr(scales, "scales", _F32),
               _addr(valid, "valid", _MASK))
    device = _on_current_device((x, codes, scales, valid))
    _check(load().moe_quantize_groups(addr, MOE_T_FP32 if x.element_size() == 4 else MOE_T_BF16,
                                      rows, cols, ld, int(bool(gated)), v, c, s,
                                      _stream(stream, device)),
           "moe_quantize_groups")


def moe_product_create(cfg: moe_product_config):
    """Returns (product handle, workspace bytes)."""
    h, n = _vp(), ctypes.c_size_t()
    _check(load().moe_product_create(ctypes.byref(cfg), ctypes.byref(h), ctypes.byref(n)),
           "moe_product_create")
    return h.value, n.value


def moe_product_destroy(product) -> None:
    load().moe_product_destroy(product)


def moe_product_set_wait_limit(product, limit_ns: int) -> None:
    _check(load().moe_product_set_wait_limit(product, limit_ns), "moe_product_set_wait_limit")


def moe_block_scaled_product(product, a, a_scales, w, w_scales, rows: int, out, ldo: int,
                             workspace, ws_bytes: int, stream=None) -> None:
    """out: a device address or tensor whose rows start ldo elements apart."""
    st = load().moe_block_scaled_product(
        product, _addr(a, "a", _CODES), _addr(a_scales, "a_scales", _F32), _addr(w, "w", _CODES),
        _addr(w_scales, "w_scales", _F32), rows,
        out if isinstance(out, int) else _rows_of(out, "out", _BF16 + _F32)[0], ldo,
        _addr(workspace, "workspace"), ws_bytes, _stream(stream))
    _check(st, "moe_block_scaled_product")


def moe_product_device_status(product, workspace, stream=None) -> int:
    """The device status bits of a product's workspace (0 = none); synchronises the stream."""
    bits = ctypes.c_uint32()
    st = load().moe_product_device_status(product, _addr(workspace, "workspace"), _stream(stream),
                                          ctypes.byref(bits))
    if st not in (MOE_OK, MOE_ERR_DEVICE):
        raise MoeError(st, "moe_product_device_status")
    return bits.value


def moe_reduce_partials(slots, n_slots: int, rows: int, H: int, valid, out, stream=None) -> None:
    st = load().moe_reduce_partials(_addr(slots, "slots", _F32), n_slots, rows, H,
                                    _addr(valid, "valid", _MASK), _addr(out, "out", _BF16),
                                    _stream(stream))
    _check(st, "moe_reduce_partials")


def moe_route_from_logits(plan, logits, valid, T: int, k: int, topk_ids, topk_w, perm, offsets,
                          workspace, ws_bytes: int, stream=None) -> None:
    st = load().moe_route_from_logits(plan, _addr(logits, "logits", _F32),
                                      _addr(valid, "valid", _MASK), T, k,
                                      _addr(topk_ids, "topk_ids", _I32),
                                      _addr(topk_w, "topk_w", _F32), _addr(perm, "perm", _I32),
                                      _addr(offsets, "offsets", _I32),
                                      _addr(workspace, "workspace"), ws_bytes, _stream(stream))
    _check(st, "moe_route_from_logits")


def moe_route_from_logits_noalloc(plan, logits, valid, T: int, k: int, topk_ids, topk_w, perm,
                                  offsets, stream=None) -> None:
    """Routing from logits with the library's own static device scratch: for
    callers that cannot allocate device memory (no workspace argument)."""
    st = load().moe_route_from_logits_noalloc(plan, _addr(logits, "logits", _F32),
                                              _addr(valid, "valid", _MASK), T, k,
                                              _addr(topk_ids, "topk_ids", _I32),
                                              _addr(topk_w, "topk_w", _F32),
                                              _addr(perm, "perm", _I32),
                                              _addr(offsets, "offsets", _I32), _stream(stream))
    _check(st, "moe_route_from_logits_noalloc")


def moe_check_device_status(plan, workspace, stream=None) -> int:
    """Returns the device status bits (0 = none); synchronises the stream."""
    bits = ctypes.c_uint32()
    st = load().moe_check_device_status(plan, _addr(workspace, "workspace"), _stream(stream),
                                        ctypes.byref(bits))
    if st not in (MOE_OK, MOE_ERR_DEVICE):
        raise MoeError(st, "moe_check_device_status")
    return bits.value


def _host_addr(t, name: str, dtypes=None) -> int | None:
    """Address of a host (CPU) tensor argument: contiguous, of one of ``dtypes``."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if t.is_cuda:
        raise ValueError(f"{name}: a host tensor is required, got one on {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous tensor is required")
    if dtypes is not None and _dtype_name(t.dtype) not in dtypes:
        raise ValueError(f"{name}: element type {t.dtype} is not one of {', '.join(dtypes)}")
    return t.data_ptr()


def moe_pipeline_slot_bytes(plan, rows: int, depth: int) -> int:
    n = ctypes.c_size_t()
    _check(load().moe_pipeline_slot_bytes(plan, rows, depth, ctypes.byref(n)),
           "moe_pipeline_slot_bytes")
    return n.value


def moe_pipeline_create(plan, weights: moe_weights, k: int, rows: int, depth: int,
                        use_graph: bool, slots, slots_bytes: int, workspace, ws_bytes: int):
    h = _vp()
    _check(load().moe_pipeline_create(plan, ctypes.byref(weights), k, rows, depth,
                                      int(bool(use_graph)), _addr(slots, "slots"), slots_bytes,
                                      _addr(workspace, "workspace"), ws_bytes, ctypes.byref(h)),
           "moe_pipeline_create")
    return h.value


def moe_pipeline_submit(pipeline, hidden_host, valid_host, out_host) -> None:
    _check(load().moe_pipeline_submit(pipeline, _host_addr(hidden_host, "hidden_host", _BF16),
                                      _host_addr(valid_host, "valid_host", _MASK),
                                      _host_addr(out_host, "out_host", _BF16)),
           "moe_pipeline_submit")


def moe_pipeline_synchronize(pipeline) -> None:
    _check(load().moe_pipeline_synchronize(pipeline), "moe_pipeline_synchronize")


def moe_pipeline_streams(pipeline):
    """(upload, compute, download) cudaStream_t handles as ints."""
    u, c, d = _vp(), _vp(), _vp()
    _check(load().moe_pipeline_streams(pipeline, ctypes.byref(u), ctypes.byref(c),
                                       ctypes.byref(d)), "moe_pipeline_streams")
    return u.value or 0, c.value or 0, d.value or 0


def moe_pipeline_destroy(pipeline) -> None:
    load().moe_pipeline_destroy(pipeline)


def moe_get_workspace_views(plan, workspace) -> moe_workspace_views:
    v = moe_workspace_views()
    _check(load().moe_get_workspace_views(plan, _addr(workspace, "workspace"), ctypes.byref(v)),
           "moe_get_workspace_views")
    return v


class Plan:
    """A plan plus a torch-allocated workspace on the current device."""

    def __init__(self, *, max_tokens: int, hidden: int, num_experts: int, top_k_max: int,
                 inter: int, num_shared: int = 0, shared_inter: int = 0, renormalize: int = 1,
                 wtype: int = MOE_W_BF16, device=None):
        import torch
        self.cfg = moe_config(max_tokens, hidden, num_experts, top_k_max, inter, num_shared,
                              shared_inter, renormalize, wtype)
        self.handle, self.ws_bytes = moe_plan_create(self.cfg)
        self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8,
                                     device=device if device is not None else "cuda")

    def weights(self, router_w, router_b=None, w_gate_up=None, w_down=None, s_gate_up=None,
                s_down=None, ws_gate_up=None, ws_down=None, ss_gate_up=None,
                ss_down=None, split_router=True, stream=None) -> moe_weights:
        """``make_weights`` with every tensor's shape checked against the plan: router
        [E, H] (+ bias [E]), gate/up [E, 2I, H], down [E, H, I], FP8 block scales
        [E, 2I/128, H/128] and [E, H/128, I/128], shared expert [2Is, H] / [H, Is] with
        scales [2Is/128, H/128] / [H/128, Is/128] (a mis-shaped tensor would be read
        past its end on the device).  Raw int addresses are taken as they are.
        With split_router, the router weights' bf16 split is made here once
        (moe_split_router_weights, on ``stream``) into a tensor the returned
        structure keeps alive, and forwards read it; make the weights again after
        changing router_w."""
        c = self.cfg
        E, H, I, Is = c.num_experts, c.hidden, c.inter, c.shared_inter
        fp8 = c.wtype == MOE_W_FP8_E4M3_B128
        want = {"router_w": (E, H), "w_gate_up": (E, 2 * I, H), "w_down": (E, H, I)}
        optional = {"router_b": (E,)}
        if fp8:
            want.update(s_gate_up=(E, 2 * I // 128, H // 128), s_down=(E, H // 128, I // 128))
        if c.num_shared:
            want.update(ws_gate_up=(2 * Is, H), ws_down=(H, Is))
            if fp8:
                want.update(ss_gate_up=(2 * Is // 128, H // 128), ss_down=(H // 128, Is // 128))
        given = dict(router_w=router_w, router_b=router_b, w_gate_up=w_gate_up, w_down=w_down,
                     s_gate_up=s_gate_up, s_down=s_down, ws_gate_up=ws_gate_up,
                     ws_down=ws_down, ss_gate_up=ss_gate_up, ss_down=ss_down)
        for name, shape in {**want, **optional}.items():
            t = given[name]
            if t is None:
                if name in want:
                    raise ValueError(f"{name} is required by this plan")
                continue
            if not isinstance(t, int) and tuple(t.shape) != shape:
                raise ValueError(f"{name}: shape {tuple(t.shape)}, the plan needs {shape}")
        if not split_router:
            return make_weights(**given)
        import torch
        nbytes = moe_router_split_bytes(self.handle)
        split = torch.empty(nbytes // 2, dtype=torch.bfloat16, device=self.workspace.device)
        moe_split_router_weights(self.handle, router_w, split, nbytes, stream)
        w = make_weights(**given, router_split=split)
        w._router_split = split          # the structure holds only its address
        return w

    def _rows(self, hidden, valid, out=None) -> int:
        """T of a call, after checking hidden [T, H], valid [T] and out [T, H]."""
        H = self.cfg.hidden
        if hidden.dim() != 2 or hidden.shape[1] != H:
            raise ValueError(f"hidden: shape {tuple(hidden.shape)}, the plan needs [T, {H}]")
        T = hidden.shape[0]
        if valid is not None and tuple(valid.shape) != (T,):
            raise ValueError(f"valid: shape {tuple(valid.shape)}, needs ({T},)")
        if out is not None and tuple(out.shape) != (T, H):
            raise ValueError(f"out: shape {tuple(out.shape)}, needs ({T}, {H})")
        return T

    def _slabs(self, dst, rows: int):
        """Each receive slab tensor must hold len(dst) row blocks of ``rows`` rows."""
        need = len(dst) * rows * self.cfg.hidden
        for d in dst:
            if not isinstance(d, int) and d.numel() < need:
                raise ValueError(f"dst: a slab of {d.numel()} values, needs {need}")

    def forward(self, weights: moe_weights, hidden, valid, k: int, out, stream=None, dbg=None):
        moe_forward(self.handle, weights, hidden, valid, self._rows(hidden, valid, out), k, out,
                    self.workspace, self.ws_bytes, stream, dbg)

    def forward_few(self, weights: moe_weights, hidden, valid, k: int, out, stream=None, dbg=None):
        """``forward`` for at most MOE_FEW_TOKENS_MAX tokens, in one kernel."""
        T = self._rows(hidden, valid, out)
        _on_current_device((hidden, valid, out, self.workspace))
        moe_forward_few(self.handle, weights, hidden, valid, T, k, out, self.workspace,
                        self.ws_bytes, stream, dbg)

    def forward_scatter(self, weights: moe_weights, hidden, valid, k: int, dst,
                        rows_per_rank: int, slot: int, stream=None, dbg=None):
        T = self._rows(hidden, valid)
        self._slabs(dst, rows_per_rank)
        moe_forward_scatter(self.handle, weights, hidden, valid, T, k, dst,
                            rows_per_rank, slot, self.workspace, self.ws_bytes, stream, dbg)

    def forward_scatter_experts(self, weights: moe_weights, hidden, valid, k: int, dst,
                                rows_per_rank: int, slot: int, expert_begin: int,
                                expert_end: int, stream=None, dbg=None):
        T = self._rows(hidden, valid)
        self._slabs(dst, rows_per_rank)
        moe_forward_scatter_experts(self.handle, weights, hidden, valid, T, k, dst,
                                    rows_per_rank, slot, expert_begin, expert_end,
                                    self.workspace, self.ws_bytes, stream, dbg)

    def forward_scatter_pairs(self, weights: moe_weights, hidden, valid, k: int, dst,
                              rows_per_rank: int, shared_slot: int, expert_begin: int,
                              expert_end: int, send_ctas: int, stream=None, dbg=None):
        T = self._rows(hidden, valid)
        need = (k + 1) * rows_per_rank * self.cfg.hidden
        for d in dst:
            if not isinstance(d, int) and d.numel() < need:
                raise ValueError(f"dst: a slab of {d.numel()} values, needs at least {need}")
        moe_forward_scatter_pairs(self.handle, weights, hidden, valid, T, k, dst, rows_per_rank,
                                  shared_slot, expert_begin, expert_end, send_ctas,
                                  self.workspace, self.ws_bytes, stream, dbg)

    def route_from_logits(self, logits, valid, k: int, topk_ids, topk_w, perm, offsets,
                          stream=None):
        moe_route_from_logits(self.handle, logits, valid, logits.shape[0], k, topk_ids, topk_w,
                              perm, offsets, self.workspace, self.ws_bytes, stream)

    def device_status(self, stream=None) -> int:
        return moe_check_device_status(self.handle, self.workspace, stream)

    def views(self) -> moe_workspace_views:
        return moe_get_workspace_views(self.handle, self.workspace)

    def set_wait_limit(self, ns: int):
        moe_plan_set_wait_limit(self.handle, ns)

    def close(self):
        if self.handle:
            moe_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Product:
    """A block-scaled product's shape plus a torch-allocated workspace on the current device."""

    def __init__(self, *, max_rows: int, n: int, k: int, out_dtype=None, device=None):
        import torch
        types = {None: MOE_T_BF16, torch.bfloat16: MOE_T_BF16, torch.float32: MOE_T_FP32}
        self.handle = None
        if out_dtype not in types:
            raise ValueError(f"out_dtype: {out_dtype} is neither bfloat16 nor float32")
        self._set_shape(moe_product_config(max_rows, n, k, types[out_dtype]),
                        out_dtype or torch.bfloat16)
        self.handle, self.ws_bytes = moe_product_create(self.cfg)
        self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8,
                                     device=device if device is not None else "cuda")

    def _set_shape(self, cfg: moe_product_config, out_dtype):
        self.cfg, self.out_dtype = cfg, out_dtype
        self._n, self._k, self._kb = cfg.n, cfg.k, _groups(cfg.k)
        self._w_shape, self._ws_shape = (cfg.n, cfg.k), (_groups(cfg.n), _groups(cfg.k))

    def forward(self, a, a_scales, w, w_scales, out, stream=None):
        """out [rows, n] = (a scaled by a_scales) (w scaled by w_scales)^T: a e4m3 [rows, k],
        a_scales fp32 [rows, ceil(k/128)], w e4m3 [n, k], w_scales fp32 [ceil(n/128),
        ceil(k/128)].  Rows of out may be strided (a slice of a wider tensor)."""
        rows = a.shape[0]
        for name, t, shape in (("a", a, (rows, self._k)), ("a_scales", a_scales, (rows, self._kb)),
                               ("w", w, self._w_shape), ("w_scales", w_scales, self._ws_shape),
                               ("out", out, (rows, self._n))):
            if t.shape != shape:
                raise ValueError(f"{name}: shape {tuple(t.shape)}, the product needs {shape}")
        if out.dtype != self.out_dtype:
            raise ValueError(f"out: element type {out.dtype}, the product needs {self.out_dtype}")
        addr, ldo = _rows_of(out, "out", _BF16 + _F32)
        _on_current_device((a, a_scales, w, w_scales, out, self.workspace))
        moe_block_scaled_product(self.handle, a, a_scales, w, w_scales, rows, addr, ldo,
                                 self.workspace, self.ws_bytes, stream)

    def device_status(self, stream=None) -> int:
        return moe_product_device_status(self.handle, self.workspace, stream)

    def set_wait_limit(self, ns: int):
        moe_product_set_wait_limit(self.handle, ns)

    def close(self):
        if self.handle:
            moe_product_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
