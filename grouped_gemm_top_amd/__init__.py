"""MI355X-native dropless MoE expert-MLP layer: thin Python binding over libmoe.so.

Every function here only marshals arguments (torch device tensors -> raw pointers and
sizes) into the C ABI declared in ``include/moe.h``; all computation runs in the HIP
kernels of ``libmoe.so``.  There is no fallback: if the library is missing or a call fails,
an exception is raised.  PyTorch supplies device memory and the current stream only.
"""
from __future__ import annotations

import ctypes
import functools
import os

__all__ = [
    "MoEError", "lib", "lib_path", "load_library", "Plan", "route_topk", "permute", "permute_noalloc",
    "route_token_rounding", "quantize_mxfp8", "grouped_gemm_fwd_mxfp8", "mx_scale_cols", "OP_GEMM_FWD_MXFP8",
    "quantize_dx_weights_mxfp8", "layer_bwd_mxfp8", "OP_LAYER_BWD_MXFP8",
    "route_capacity", "grouped_gemm_fwd", "unpermute_combine", "layer_bwd", "router_logits", "router_bwd",
    "workspace_bytes", "plan_rows_cap", "MOE_OK", "MOE_EINVAL", "MOE_EUNSUPPORTED", "MOE_EWORKSPACE",
    "MOE_EHIP", "OP_PERMUTE", "OP_ROUTE_TR", "OP_GEMM_FWD", "OP_LAYER_BWD", "OP_ROUTER_BWD",
    "OP_ROUTER_LOGITS", "PLAN_TOPK", "PLAN_TR", "PLAN_CAP", "CAP_POSITION", "CAP_PROBS",
    "EXPORTED_SYMBOLS", "KERNEL_IDS", "set_kernel_events", "add_rmsnorm", "add_rmsnorm_bwd", "OP_ADD_RMSNORM_BWD",
    "balance_loss", "balance_loss_bwd", "OP_BALANCE_LOSS", "linear_fwd", "linear_bwd", "OP_LINEAR_FWD", "OP_LINEAR_BWD",
    "ACTIVATIONS", "linear_ce_fwd", "linear_ce_bwd", "OP_LINEAR_CE_FWD", "OP_LINEAR_CE_BWD",
    "dequantize_mxfp8", "grouped_gemm_fwd_ckpt8", "layer_bwd_ckpt8", "OP_LAYER_BWD_CKPT8",
    "layer_few", "OP_LAYER_FEW", "FEW_MAX_TOKENS", "FEW_MAX_K",
]

MOE_OK, MOE_EINVAL, MOE_EUNSUPPORTED, MOE_EWORKSPACE, MOE_EHIP = 0, 1, 2, 3, 4
MOE_F32, MOE_BF16 = 0, 1
PLAN_TOPK, PLAN_TR, PLAN_CAP = 0, 1, 2
CAP_POSITION, CAP_PROBS = 0, 1
OP_PERMUTE, OP_ROUTE_TR, OP_GEMM_FWD, OP_LAYER_BWD, OP_ROUTER_BWD, OP_ROUTER_LOGITS = 0, 1, 2, 3, 4, 5
OP_GEMM_FWD_MXFP8 = 6
OP_LAYER_BWD_MXFP8 = 7
OP_ADD_RMSNORM_BWD = 8
OP_BALANCE_LOSS = 9
OP_LINEAR_FWD, OP_LINEAR_BWD = 10, 11
OP_LINEAR_CE_FWD, OP_LINEAR_CE_BWD = 12, 13
OP_LAYER_BWD_CKPT8 = 14
OP_LAYER_FEW = 15
FEW_MAX_TOKENS, FEW_MAX_K = 64, 32  # limits of layer_few
# activations of linear_fwd (moe_act in include/moe.h)
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}

EXPORTED_SYMBOLS = (
    "moe_plan_rows_cap", "moe_workspace_bytes", "moe_last_error", "moe_route_topk", "moe_permute",
    "moe_permute_noalloc",
    "moe_route_token_rounding", "moe_route_capacity", "moe_grouped_gemm_fwd", "moe_unpermute_combine",
    "moe_layer_bwd",
    "moe_router_logits", "moe_router_bwd", "moe_set_kernel_events", "moe_quantize_mxfp8",
    "moe_grouped_gemm_fwd_mxfp8", "moe_quantize_dx_weights_mxfp8", "moe_layer_bwd_mxfp8",
    "moe_add_rmsnorm", "moe_add_rmsnorm_bwd", "moe_balance_loss", "moe_balance_loss_bwd", "moe_router_bwd_acc",
    "moe_linear_fwd", "moe_linear_bwd", "moe_linear_ce_fwd", "moe_linear_ce_bwd",
    "moe_grouped_gemm_fwd_ckpt8", "moe_layer_bwd_ckpt8", "moe_dequantize_mxfp8",
    "moe_layer_few", "moe_layer_few_mxfp8",
)

# kernel ids of the measurement hook (moe_kernel_id in include/moe.h)
KERNEL_IDS = {"gateup": 0, "down": 1, "dh": 2, "dx": 3, "dwd": 4, "dw1": 5, "combine": 6, "dx_combine": 7,
              "route": 8, "permute": 9, "route_tr_plan": 10, "dswiglu": 11, "router_logits": 12,
              "router_dz": 13, "router_dx": 14, "router_dw": 15, "gateup_fp8": 16, "down_fp8": 17, "quant": 18,
              "dx_fp8": 19, "add_rmsnorm": 20, "add_rmsnorm_bwd": 21, "balance": 22,
              "balance_bwd": 23, "linear": 24, "linear_bwd": 25, "linear_ce": 26, "linear_ce_bwd": 27,
              "gateup_ckpt": 28, "dh_ckpt": 29, "dequant": 30, "layer_few": 31}

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = None


def lib_path() -> str:
    """The in-tree libmoe.so (built by ``grouped_gemm_top_amd.build``)."""
    return os.path.join(_HERE, "libmoe.so")


class MoEError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"moe status {status}: {msg}")
        self.status = status


class CPlan(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("N", ctypes.c_int32), ("E", ctypes.c_int32),
                ("k", ctypes.c_int32), ("M_cap", ctypes.c_int32), ("mtile", ctypes.c_int32),
                ("counts", ctypes.c_void_p), ("offsets", ctypes.c_void_p),
                ("row_token", ctypes.c_void_p), ("row_w", ctypes.c_void_p),
                ("row_pair", ctypes.c_void_p), ("tok_ptr", ctypes.c_void_p),
                ("tok_rows", ctypes.c_void_p)]


def lib():
    """Load libmoe.so (built by ``grouped_gemm_top_amd.build``); raise if it is missing."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = lib_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m grouped_gemm_top_amd.build` "
                           "(there is no fallback path)")
    _LIB = load_library(path)
    return _LIB


def load_library(path: str):
    """ctypes handle of a build of libmoe.so at `path` with every entry point's signature set
    (lib() uses it for the in-tree library; the host-sanitizer tests for their own build)."""
    L = ctypes.CDLL(path)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    pp = ctypes.POINTER(CPlan)
    L.moe_plan_rows_cap.argtypes = [i32, i32, i32, i32, i32]
    L.moe_plan_rows_cap.restype = ctypes.c_int64
    L.moe_workspace_bytes.argtypes = [ctypes.c_int, ctypes.c_int, i32, i32, i32, i32, i32, i32]
    L.moe_workspace_bytes.restype = sz
    L.moe_last_error.argtypes = []
    L.moe_last_error.restype = ctypes.c_char_p
    L.moe_route_topk.argtypes = [vp, vp, i32, i32, i32, vp, vp, vp, vp]
    L.moe_permute.argtypes = [vp, vp, i32, i32, i32, pp, vp, sz, vp]
    L.moe_permute_noalloc.argtypes = [vp, vp, i32, i32, i32, pp, vp]
    L.moe_route_token_rounding.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, vp, pp, vp, sz, vp]
    L.moe_route_capacity.argtypes = [vp, vp, i32, i32, i32, i32, i32, vp, vp, vp, pp, vp, sz, vp]
    L.moe_grouped_gemm_fwd.argtypes = [ctypes.c_int, vp, vp, vp, vp, i32, i32, pp, vp, vp, vp, sz, vp]
    L.moe_unpermute_combine.argtypes = [ctypes.c_int, vp, i32, pp, vp, vp, vp]
    L.moe_layer_bwd.argtypes = [ctypes.c_int, vp, vp, vp, vp, vp, i32, i32, pp, vp, vp, vp, vp, vp, vp,
                                vp, sz, vp]
    L.moe_router_logits.argtypes = [ctypes.c_int, vp, vp, vp, i32, i32, i32, vp, vp, sz, vp]
    L.moe_router_bwd.argtypes = [ctypes.c_int, vp, vp, vp, pp, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_set_kernel_events.argtypes = [i32, vp, vp]
    L.moe_quantize_mxfp8.argtypes = [ctypes.c_int, vp, ctypes.c_int64, i32, vp, vp, vp]
    L.moe_grouped_gemm_fwd_mxfp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, pp, vp, vp, vp, sz, vp]
    L.moe_quantize_dx_weights_mxfp8.argtypes = [ctypes.c_int, vp, vp, i32, i32, i32, vp, vp, vp]
    L.moe_layer_bwd_mxfp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, pp, vp, vp, vp, vp, vp, vp, vp, sz,
                                      vp]
    f32 = ctypes.c_float
    L.moe_add_rmsnorm.argtypes = [ctypes.c_int, ctypes.c_int, vp, vp, vp, f32, i32, i32, vp, vp, vp, vp, vp]
    L.moe_add_rmsnorm_bwd.argtypes = [ctypes.c_int, ctypes.c_int, vp, vp, vp, vp, f32, i32, i32, vp, vp, vp, vp, sz, vp]
    L.moe_balance_loss.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, f32, f32, vp, vp, vp, vp, sz, vp]
    L.moe_balance_loss_bwd.argtypes = [vp, vp, vp, vp, i32, i32, i32, vp, vp, vp, vp, vp]
    L.moe_router_bwd_acc.argtypes = [ctypes.c_int, vp, vp, vp, pp, vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_linear_fwd.argtypes = [ctypes.c_int, vp, vp, vp, i32, vp, i32, i32, i32, vp, vp, vp, sz, vp]
    L.moe_linear_bwd.argtypes = [ctypes.c_int, vp, vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, sz, vp]
    L.moe_linear_ce_fwd.argtypes = [ctypes.c_int, vp, vp, vp, i32, i32, i32, f32, vp, vp, vp, sz, vp]
    L.moe_linear_ce_bwd.argtypes = [ctypes.c_int, vp, vp, vp, vp, vp, i32, i32, i32, f32, vp, vp, vp, sz, vp]
    L.moe_grouped_gemm_fwd_ckpt8.argtypes = [vp, vp, vp, vp, i32, i32, pp, vp, vp, vp, vp, sz, vp]
    L.moe_layer_bwd_ckpt8.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, pp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_dequantize_mxfp8.argtypes = [ctypes.c_int, vp, vp, ctypes.c_int64, i32, vp, vp]
    L.moe_layer_few.argtypes = [ctypes.c_int, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp, vp, vp, sz, vp]
    L.moe_layer_few_mxfp8.argtypes = [vp] * 9 + [i32] * 5 + [vp, vp, vp, vp, sz, vp]
    for fn in ("moe_route_topk", "moe_permute", "moe_permute_noalloc", "moe_route_token_rounding",
               "moe_route_capacity",
               "moe_grouped_gemm_fwd",
               "moe_unpermute_combine", "moe_layer_bwd", "moe_router_logits", "moe_router_bwd",
               "moe_set_kernel_events", "moe_quantize_mxfp8", "moe_grouped_gemm_fwd_mxfp8",
               "moe_quantize_dx_weights_mxfp8", "moe_layer_bwd_mxfp8", "moe_add_rmsnorm", "moe_add_rmsnorm_bwd",
               "moe_balance_loss", "moe_balance_loss_bwd", "moe_router_bwd_acc",
               "moe_linear_fwd", "moe_linear_bwd", "moe_linear_ce_fwd", "moe_linear_ce_bwd",
               "moe_grouped_gemm_fwd_ckpt8", "moe_layer_bwd_ckpt8", "moe_dequantize_mxfp8",
               "moe_layer_few", "moe_layer_few_mxfp8"):
        getattr(L, fn).restype = ctypes.c_int
    return L


def _check(st: int):
    if st:
        raise MoEError(st, lib().moe_last_error().decode(errors="replace"))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return MOE_BF16
    if t.dtype == torch.float32:
        return MOE_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def set_kernel_events(name: str, start=None, stop=None):
    """Register torch.cuda.Event objects (enable_timing=True) to be recorded around every
    later launch of the named kernel on its launch stream; None switches it off."""
    h = (lambda ev: None if ev is None else ctypes.c_void_p(ev.cuda_event))
    _check(lib().moe_set_kernel_events(KERNEL_IDS[name], h(start), h(stop)))


def plan_rows_cap(kind: int, N: int, E: int, k: int, mtile: int = 0) -> int:
    v = lib().moe_plan_rows_cap(kind, N, E, k, mtile)
    if v < 0:
        raise MoEError(MOE_EINVAL, "invalid plan dimensions")
    return int(v)


def workspace_bytes(op: int, dtype_code: int, N: int, E: int, k: int, H: int = 8, I: int = 8,
                    M_cap: int = 0) -> int:
    v = lib().moe_workspace_bytes(op, dtype_code, N, E, k, H, I, M_cap)
    if v == 0:
        raise MoEError(MOE_EINVAL, "invalid workspace query")
    return int(v)


class Plan:
    """Device arrays of a routing plan (see moe_plan in include/moe.h), allocated with torch."""

    def __init__(self, N: int, E: int, k: int, kind: int = PLAN_TOPK, mtile: int = 0, device="cuda",
                 alloc=None):
        """alloc(name, numel, dtype) -> 1-D device tensor, if given, supplies the arrays
        (default: torch.empty on `device`)."""
        import torch
        self.N, self.E, self.k, self.kind = N, E, k, kind
        self.mtile = mtile if kind in (PLAN_TR, PLAN_CAP) else 0  # capacity plans: the capacity
        self.M_cap = plan_rows_cap(kind, N, E, k, self.mtile)
        if alloc is None:
            alloc = lambda name, n, dt: torch.empty(n, dtype=dt, device=device)  # noqa: E731
        i32 = torch.int32
        mc = max(self.M_cap, 1)
        self.counts = alloc("counts", E, i32)
        self.offsets = alloc("offsets", E + 1, i32)
        self.row_token = alloc("row_token", mc, i32)
        self.row_w = alloc("row_w", mc, torch.float32)
        self.row_pair = alloc("row_pair", mc, i32)
        self.tok_ptr = alloc("tok_ptr", N + 1, i32)
        self.tok_rows = alloc("tok_rows", mc, i32)
        self._c = CPlan(kind, N, E, k, self.M_cap, self.mtile, *(t.data_ptr() for t in (
            self.counts, self.offsets, self.row_token, self.row_w, self.row_pair, self.tok_ptr,
            self.tok_rows)))

    @property
    def c(self):
        return ctypes.byref(self._c)

    def host(self) -> dict:
        """Copy the plan to host numpy arrays, trimmed to the rows in use."""
        off = self.offsets.cpu().numpy()
        m = int(off[-1])
        return dict(counts=self.counts.cpu().numpy(), offsets=off,
                    row_token=self.row_token[:m].cpu().numpy(), row_w=self.row_w[:m].cpu().numpy(),
                    row_pair=self.row_pair[:m].cpu().numpy(), tok_ptr=self.tok_ptr.cpu().numpy(),
                    tok_rows=self.tok_rows[:m].cpu().numpy())


def _ws(nbytes: int, device, ws=None):
    import torch
    if ws is not None:
        if ws.numel() * ws.element_size() < nbytes:
            raise MoEError(MOE_EWORKSPACE, f"workspace holds {ws.numel() * ws.element_size()} < {nbytes} bytes")
        return ws
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def route_topk(logits, k: int, bias=None, want_probs: bool = False, idx=None, w=None, probs=None,
               stream=None):
    """-> (topk_idx int32 [N,k], topk_w fp32 [N,k], probs fp32 [N,E] or None)."""
    import torch
    N, E = logits.shape
    idx = idx if idx is not None else torch.empty((N, k), dtype=torch.int32, device=logits.device)
    w = w if w is not None else torch.empty((N, k), dtype=torch.float32, device=logits.device)
    if probs is None and want_probs:
        probs = torch.empty((N, E), dtype=torch.float32, device=logits.device)
    _check(lib().moe_route_topk(_ptr(logits), _ptr(bias), N, E, k, _ptr(idx), _ptr(w), _ptr(probs),
                                _stream(stream)))
    return idx, w, probs


def permute(topk_idx, topk_w, E: int, plan: Plan | None = None, ws=None, stream=None) -> Plan:
    N, k = topk_idx.shape
    plan = plan or Plan(N, E, k, device=topk_idx.device)
    nb = workspace_bytes(OP_PERMUTE, MOE_BF16, N, E, k)
    ws = _ws(nb, topk_idx.device, ws)
    _check(lib().moe_permute(_ptr(topk_idx), _ptr(topk_w), N, E, k, plan.c, _ptr(ws), nb, _stream(stream)))
    return plan


def permute_noalloc(topk_idx, topk_w, E: int, plan: Plan, stream=None) -> Plan:
    """moe_permute_noalloc: the permute with the library's fixed scratch instead of a
    workspace; `plan` (caller-allocated) is required, so this call allocates nothing."""
    N, k = topk_idx.shape
    _check(lib().moe_permute_noalloc(_ptr(topk_idx), _ptr(topk_w), N, E, k, plan.c, _stream(stream)))
    return plan


def route_token_rounding(logits, k: int, mtile: int, bias=None, plan: Plan | None = None, ws=None,
                         idx=None, w=None, probs=None, stream=None):
    """-> (plan, topk_idx, topk_w, probs)."""
    import torch
    N, E = logits.shape
    dev = logits.device
    plan = plan or Plan(N, E, k, kind=PLAN_TR, mtile=mtile, device=dev)
    idx = idx if idx is not None else torch.empty((N, k), dtype=torch.int32, device=dev)
    w = w if w is not None else torch.empty((N, k), dtype=torch.float32, device=dev)
    probs = probs if probs is not None else torch.empty((N, E), dtype=torch.float32, device=dev)
    nb = workspace_bytes(OP_ROUTE_TR, MOE_BF16, N, E, k)
    ws = _ws(nb, dev, ws)
    _check(lib().moe_route_token_rounding(_ptr(logits), _ptr(bias), N, E, k, mtile, _ptr(idx), _ptr(w),
                                          _ptr(probs), plan.c, _ptr(ws), nb, _stream(stream)))
    return plan, idx, w, probs


def route_capacity(logits, k: int, capacity: int, policy: int = CAP_POSITION, bias=None, plan: Plan | None = None,
                   ws=None, idx=None, w=None, probs=None, stream=None):
    """-> (plan, topk_idx, topk_w, probs): top-k routing, then each expert keeps at most
    `capacity` of its tokens (policy CAP_POSITION: token order; CAP_PROBS: largest P first)."""
    import torch
    N, E = logits.shape
    dev = logits.device
    plan = plan or Plan(N, E, k, kind=PLAN_CAP, mtile=capacity, device=dev)
    idx = idx if idx is not None else torch.empty((N, k), dtype=torch.int32, device=dev)
    w = w if w is not None else torch.empty((N, k), dtype=torch.float32, device=dev)
    probs = probs if probs is not None else torch.empty((N, E), dtype=torch.float32, device=dev)
    nb = workspace_bytes(OP_ROUTE_TR, MOE_BF16, N, E, k)
    ws = _ws(nb, dev, ws)
    _check(lib().moe_route_capacity(_ptr(logits), _ptr(bias), N, E, k, capacity, policy, _ptr(idx), _ptr(w),
                                    _ptr(probs), plan.c, _ptr(ws), nb, _stream(stream)))
    return plan, idx, w, probs


def grouped_gemm_fwd(x, w_gate, w_up, w_down, plan: Plan, hcache=None, y=None, ws=None, stream=None):
    """-> (hcache [M_cap, 2I], y [M_cap, H])."""
    import torch
    N, H = x.shape
    E, I, _ = w_gate.shape
    dt = _dtype_code(x)
    mc = max(plan.M_cap, 1)
    hcache = hcache if hcache is not None else torch.empty((mc, 2 * I), dtype=x.dtype, device=x.device)
    y = y if y is not None else torch.empty((mc, H), dtype=x.dtype, device=x.device)
    nb = workspace_bytes(OP_GEMM_FWD, dt, plan.N, plan.E, plan.k, H, I, plan.M_cap)
    ws = _ws(nb, x.device, ws)
    _check(lib().moe_grouped_gemm_fwd(dt, _ptr(x), _ptr(w_gate), _ptr(w_up), _ptr(w_down), H, I, plan.c,
                                      _ptr(hcache), _ptr(y), _ptr(ws), nb, _stream(stream)))
    return hcache, y


def mx_scale_cols(K: int) -> int:
    """Scale codes per row of an MX-FP8 matrix with K columns: 4 * ceil(K / 128)."""
    return 4 * ((K + 127) // 128)


def quantize_mxfp8(src, q=None, scales=None, stream=None):
    """MX-FP8 quantization of src [..., K] (bf16 or fp32, K a multiple of 32) along its last
    dimension -> (codes uint8 [..., K], scale codes uint8 [..., 4 ceil(K/128)])."""
    import torch
    K = src.shape[-1]
    rows = src.numel() // K if K else 0
    q = q if q is not None else torch.empty(src.shape, dtype=torch.uint8, device=src.device)
    scales = scales if scales is not None else torch.empty(src.shape[:-1] + (mx_scale_cols(K),), dtype=torch.uint8,
                                                           device=src.device)
    _check(lib().moe_quantize_mxfp8(_dtype_code(src), _ptr(src), rows, K, _ptr(q), _ptr(scales), _stream(stream)))
    return q, scales


def grouped_gemm_fwd_mxfp8(x, w_gate, w_up, w_down, plan: Plan, hcache=None, y=None, ws=None, stream=None):
    """Forward on MX-FP8 operands; x, w_gate, w_up, w_down are (codes, scale codes) pairs from
    quantize_mxfp8 of x [N,H], W_gate / W_up [E,I,H] and W_down [E,H,I].  -> (hcache [M_cap, 2I],
    y [M_cap, H]), both bf16."""
    import torch
    (xq, xs), (gq, gs), (uq, us), (dq, dsc) = x, w_gate, w_up, w_down
    N, H = xq.shape
    E, I, _ = gq.shape
    mc = max(plan.M_cap, 1)
    hcache = hcache if hcache is not None else torch.empty((mc, 2 * I), dtype=torch.bfloat16, device=xq.device)
    y = y if y is not None else torch.empty((mc, H), dtype=torch.bfloat16, device=xq.device)
    nb = workspace_bytes(OP_GEMM_FWD_MXFP8, MOE_BF16, plan.N, plan.E, plan.k, H, I, plan.M_cap)
    ws = _ws(nb, xq.device, ws)
    _check(lib().moe_grouped_gemm_fwd_mxfp8(_ptr(xq), _ptr(xs), _ptr(gq), _ptr(gs), _ptr(uq), _ptr(us), _ptr(dq),
                                            _ptr(dsc), H, I, plan.c, _ptr(hcache), _ptr(y), _ptr(ws), nb,
                                            _stream(stream)))
    return hcache, y


def unpermute_combine(y, plan: Plan, row_w="plan", out=None, stream=None):  # noqa: D401
    """out [N,H] = per-token sum of row_w[r] * y[r] (row_w: 'plan' for the plan's weights,
    None for weights 1, or an fp32 tensor [M_cap])."""
    import torch
    H = y.shape[1]
    dt = _dtype_code(y)
    out = out if out is not None else torch.empty((plan.N, H), dtype=y.dtype, device=y.device)
    rw = plan.row_w if isinstance(row_w, str) else row_w
    _check(lib().moe_unpermute_combine(dt, _ptr(y), H, plan.c, _ptr(rw), _ptr(out), _stream(stream)))
    return out


def layer_bwd(dout, x, w_gate, w_up, w_down, plan: Plan, hcache, dx=None, dw_gate=None, dw_up=None,
              dw_down=None, ds=None, ws=None, stream=None):
    """-> dict(dx, dw_gate, dw_up, dw_down, ds).  ds is [N,k] for top-k plans, [M_cap] for
    token-rounding plans."""
    import torch
    N, H = x.shape
    E, I, _ = w_gate.shape
    dt = _dtype_code(x)
    dev = x.device
    dx = dx if dx is not None else torch.empty_like(x)
    dw_gate = dw_gate if dw_gate is not None else torch.empty_like(w_gate)
    dw_up = dw_up if dw_up is not None else torch.empty_like(w_up)
    dw_down = dw_down if dw_down is not None else torch.empty_like(w_down)
    if ds is None:
        shape = (N, plan.k) if plan.kind == PLAN_TOPK else (max(plan.M_cap, 1),)
        ds = torch.empty(shape, dtype=torch.float32, device=dev)
    nb = workspace_bytes(OP_LAYER_BWD, dt, plan.N, plan.E, plan.k, H, I, plan.M_cap)
    ws = _ws(nb, dev, ws)
    _check(lib().moe_layer_bwd(dt, _ptr(dout), _ptr(x), _ptr(w_gate), _ptr(w_up), _ptr(w_down), H, I, plan.c,
                               _ptr(hcache), _ptr(dx), _ptr(dw_gate), _ptr(dw_up), _ptr(dw_down), _ptr(ds),
                               _ptr(ws), nb, _stream(stream)))
    return dict(dx=dx, dw_gate=dw_gate, dw_up=dw_up, dw_down=dw_down, ds=ds)


def quantize_dx_weights_mxfp8(w_gate, w_up, q=None, scales=None, stream=None):
    """The dX product's MX-FP8 weight operand: each expert's [W_gate^T | W_up^T] ([H, 2I])
    quantized along 2I -> (codes uint8 [E, H, 2I], scale codes uint8 [E, H, 4 ceil(2I/128)])."""
    import torch
    E, I, H = w_gate.shape
    q = q if q is not None else torch.empty((E, H, 2 * I), dtype=torch.uint8, device=w_gate.device)
    scales = scales if scales is not None else torch.empty((E, H, mx_scale_cols(2 * I)), dtype=torch.uint8,
                                                           device=w_gate.device)
    _check(lib().moe_quantize_dx_weights_mxfp8(_dtype_code(w_gate), _ptr(w_gate), _ptr(w_up), E, H, I, _ptr(q),
                                               _ptr(scales), _stream(stream)))
    return q, scales


def layer_bwd_mxfp8(dout, x, w_gate, w_up, w_down, wt, plan: Plan, hcache, dx=None, dw_gate=None, dw_up=None,
                    dw_down=None, ds=None, ws=None, stream=None):
    """layer_bwd for bf16 layers with the dX product on MX-FP8 operands; wt = (codes, scale
    codes) from quantize_dx_weights_mxfp8.  -> dict(dx, dw_gate, dw_up, dw_down, ds)."""
    import torch
    N, H = x.shape
    E, I, _ = w_gate.shape
    wq, wsc = wt
    dev = x.device
    dx = dx if dx is not None else torch.empty_like(x)
    dw_gate = dw_gate if dw_gate is not None else torch.empty_like(w_gate)
    dw_up = dw_up if dw_up is not None else torch.empty_like(w_up)
    dw_down = dw_down if dw_down is not None else torch.empty_like(w_down)
    if ds is None:
        shape = (N, plan.k) if plan.kind == PLAN_TOPK else (max(plan.M_cap, 1),)
        ds = torch.empty(shape, dtype=torch.float32, device=dev)
    nb = workspace_bytes(OP_LAYER_BWD_MXFP8, MOE_BF16, plan.N, plan.E, plan.k, H, I, plan.M_cap)
    ws = _ws(nb, dev, ws)
    _check(lib().moe_layer_bwd_mxfp8(_ptr(dout), _ptr(x), _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(wq),
                                     _ptr(wsc), H, I, plan.c, _ptr(hcache), _ptr(dx), _ptr(dw_gate), _ptr(dw_up),
                                     _ptr(dw_down), _ptr(ds), _ptr(ws), nb, _stream(stream)))
    return dict(dx=dx, dw_gate=dw_gate, dw_up=dw_up, dw_down=dw_down, ds=ds)


def router_logits(x, w_r, bias=None, logits=None, ws=None, stream=None):
    """logits [N,E] fp32 = x @ w_r (+ bias); x [N,H] (bf16 or fp32), w_r fp32 [H,E]."""
    import torch
    N, H = x.shape
    E = w_r.shape[1]
    dt = _dtype_code(x)
    logits = logits if logits is not None else torch.empty((N, E), dtype=torch.float32, device=x.device)
    nb = workspace_bytes(OP_ROUTER_LOGITS, dt, N, E, 1, H, 8, 0)
    ws = _ws(nb, x.device, ws)
    _check(lib().moe_router_logits(dt, _ptr(x), _ptr(w_r), _ptr(bias), N, H, E, _ptr(logits), _ptr(ws), nb,
                                   _stream(stream)))
    return logits


def router_bwd(logits, topk_idx, plan: Plan, ds, x, w_r, bias=None, dx_in=None, dx_out=None, dlogits=None,
               dw_r=None, dbias=None, want_dx=True, want_dw=True, want_dbias=True, ws=None, stream=None,
               dlogits_in=None):
    """Router backward from dS (moe_layer_bwd's ds) -> dict(dlogits, dx, dw_r, dbias).
    dx = dx_in + the router's share (dx_in defaults to zeros; dx_out may be dx_in).  dlogits_in
    fp32 [N,E]: a further gradient of the logits (balance_loss_bwd's), included in all four."""
    import torch
    N, H = x.shape
    E = logits.shape[1]
    dt = _dtype_code(x)
    dev = x.device
    dlogits = dlogits if dlogits is not None else torch.empty((N, E), dtype=torch.float32, device=dev)
    if want_dx:
        dx_in = dx_in if dx_in is not None else torch.zeros_like(x)
        dx_out = dx_out if dx_out is not None else torch.empty_like(x)
    else:
        dx_in = dx_out = None
    if want_dw:
        dw_r = dw_r if dw_r is not None else torch.empty((H, E), dtype=torch.float32, device=dev)
    else:
        dw_r = None
    if want_dbias:
        dbias = dbias if dbias is not None else torch.empty((E,), dtype=torch.float32, device=dev)
    else:
        dbias = None
    nb = workspace_bytes(OP_ROUTER_BWD, dt, plan.N, plan.E, plan.k, H, 8, 0) if (want_dx or want_dw or want_dbias) \
        else 0
    ws = _ws(nb, dev, ws) if nb else None
    if dlogits_in is not None:
        _want("dlogits_in", dlogits_in, (N, E), torch.float32, logits.get_device())
    _check(lib().moe_router_bwd_acc(dt, _ptr(logits), _ptr(bias), _ptr(topk_idx), plan.c, _ptr(ds), _ptr(dlogits_in),
                                    _ptr(x), _ptr(w_r), H, _ptr(dx_in), _ptr(dx_out), _ptr(dlogits), _ptr(dw_r),
                                    _ptr(dbias), _ptr(ws), nb, _stream(stream)))
    return dict(dlogits=dlogits, dx=dx_out, dw_r=dw_r, dbias=dbias)


# ---- the operators around the layer: these bindings check every tensor they are given ----
def _want(name, t, shape, dtype, dev):
    """Refuse a tensor whose type, shape, layout (contiguous, row-major) or device (index dev, -1: the
    host, which the call itself refuses) is not the one asked for."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == dev:
        return t
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (strides {t.stride()})")
    raise ValueError(f"tensors on different devices: {name} is on {t.device}")


def _out(name, t, shape, dtype, like, dev):
    """The caller's output tensor, checked, or a new one."""
    if t is None:
        return like.new_empty(shape, dtype=dtype)
    return _want(name, t, shape, dtype, dev)


def _on_gpu(t):
    if not t.is_cuda:
        raise ValueError(f"tensors must be on a GPU (got {t.device})")


@functools.lru_cache(maxsize=1024)
def _op_bytes(*query) -> int:
    return workspace_bytes(*query)


def _op_ws(nbytes, like, ws, dev):
    """The caller's workspace, checked, or a new one."""
    if ws is None:
        return like.new_empty((nbytes,), dtype=_torch.uint8)
    if ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError(f"the workspace must be contiguous and on the tensors' device (is on {ws.device})")
    return _ws(nbytes, None, ws)


def _addr(t):
    return None if t is None else t.data_ptr()


_torch = None  # the torch module, from the first call on


def _first_use():
    global _torch
    import torch
    _torch = torch
    return torch


def _on_stream(fn, at=0):
    """Run a binding on the device of its argument number `at` (a tensor) and, if `stream` (a torch stream, or any object
    whose cuda_stream is the handle of one of that device) is given, with that stream as the current
    one: what the call allocates then belongs to the stream that uses it."""
    name = fn.__code__.co_varnames[at]

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        torch = _torch or _first_use()
        first = args[at] if len(args) > at else kw.get(name)
        if first is None:
            raise TypeError(f"{fn.__name__}() needs {name}")
        # (a host tensor is refused by the binding)
        if stream is None and (first.get_device() == torch._C._cuda_getDevice() if first.is_cuda else True):
            return fn(*args, **kw)
        _on_gpu(first)
        if stream is not None:
            if getattr(stream, "device", first.device) != first.device:
                raise ValueError(f"the stream is on {stream.device}, the tensors on {first.device}")
            if not isinstance(stream, torch.cuda.Stream):  # a handle of a stream made elsewhere
                stream = torch.cuda.ExternalStream(stream.cuda_stream, device=first.device)
        with torch.cuda.device(first.device):
            if stream is None:
                return fn(*args, **kw)
            with torch.cuda.stream(stream):
                return fn(*args, **kw)
    return call


def _cur(dev):
    """The current stream's handle on device dev."""
    return _torch._C._cuda_getCurrentRawStream(dev)


@_on_stream
def add_rmsnorm(x, w=None, residual=None, eps: float = 1e-6, want_h=True, want_y=True, quantize=False, h=None, y=None,
                q=None, scales=None):
    """Residual addition with RMS norm: s = x + residual, y = s / rms(s) * w, optionally quantized.

    x [N,H] bf16 or fp32; residual [N,H] of x's type or fp32 (None: none); w fp32 [H] (None: ones).
    -> dict(h [N,H] (the sum, in residual's type), y [N,H] (x's type), q uint8 [N,H], scales uint8
    [N, 4 ceil(H/128)]: y as MX-FP8, as quantize_mxfp8 lays it out); what is not wanted is None.
    h may be residual (in place).  stream: a torch stream to run on (default: the current one)."""
    torch = _torch
    if x.dim() != 2:
        raise ValueError(f"x must be [N, H] (got {tuple(x.shape)})")
    N, H = x.shape
    dt = _dtype_code(x)
    rtype = x.dtype if residual is None else residual.dtype
    dev = x.get_device()
    _want("x", x, (N, H), x.dtype, dev)
    if residual is not None:
        _want("residual", residual, (N, H), rtype, dev)
        rdt = _dtype_code(residual)
    else:
        if h is not None and h.dtype == torch.float32:
            rtype = torch.float32
        rdt = MOE_F32 if rtype == torch.float32 else dt
    if w is not None:
        _want("w", w, (H,), torch.float32, dev)
    _on_gpu(x)
    if want_h or h is not None:
        h = _out("h", h, (N, H), rtype, x, dev)
    if want_y or y is not None:
        y = _out("y", y, (N, H), x.dtype, x, dev)
    if quantize or q is not None or scales is not None:
        q = _out("q", q, (N, H), torch.uint8, x, dev)
        scales = _out("scales", scales, (N, mx_scale_cols(H)), torch.uint8, x, dev)
    if N:
        _check(lib().moe_add_rmsnorm(dt, rdt, x.data_ptr(), _addr(residual), _addr(w), eps, N, H, _addr(h), _addr(y),
                                     _addr(q), _addr(scales), _cur(dev)))
    return dict(h=h, y=y, q=q, scales=scales)


@_on_stream
def add_rmsnorm_bwd(dy, h, w=None, dh_in=None, eps: float = 1e-6, want_dx=False, want_dw=True, dh=None, dx=None,
                    dw=None, ws=None):
    """Backward of add_rmsnorm at the stored sum h: dy [N,H] is the gradient of y, dh_in (h's type, or
    None) the one that reaches h itself.  -> dict(dh [N,H] in h's type (the gradient of x and of
    residual), dx: dh in dy's type if wanted, dw fp32 [H] or None).  dh may be dh_in (in place)."""
    torch = _torch
    if dy.dim() != 2:
        raise ValueError(f"dy must be [N, H] (got {tuple(dy.shape)})")
    N, H = dy.shape
    dt, rdt = _dtype_code(dy), _dtype_code(h)
    dev = dy.get_device()
    _want("dy", dy, (N, H), dy.dtype, dev)
    _want("h", h, (N, H), h.dtype, dev)
    if dh_in is not None:
        _want("dh_in", dh_in, (N, H), h.dtype, dev)
    if w is not None:
        _want("w", w, (H,), torch.float32, dev)
    _on_gpu(dy)
    dh = _out("dh", dh, (N, H), h.dtype, dy, dev)
    if want_dx or dx is not None:
        dx = _out("dx", dx, (N, H), dy.dtype, dy, dev)
    nb = 0
    if want_dw or dw is not None:
        dw = _out("dw", dw, (H,), torch.float32, dy, dev)
        nb = _op_bytes(OP_ADD_RMSNORM_BWD, dt, N, 1, 1, H, 0, 0)
        ws = _op_ws(nb, dy, ws, dev)
    _check(lib().moe_add_rmsnorm_bwd(dt, rdt, dy.data_ptr(), h.data_ptr(), _addr(dh_in), _addr(w), eps, N, H,
                                     dh.data_ptr(), _addr(dx), _addr(dw), _addr(ws) if nb else None, nb, _cur(dev)))
    return dict(dh=dh, dx=dx, dw=dw)


def _seqs(N, mask, seq_ptr, dev):
    """The sequences' checks shared by balance_loss and its backward -> B."""
    torch = _torch
    if mask is not None:
        if mask.dtype not in (torch.uint8, torch.bool):
            raise TypeError(f"mask must be uint8 or bool (got {mask.dtype})")
        _want("mask", mask, (N,), mask.dtype, dev)
    if seq_ptr is None:
        return 1
    if seq_ptr.dim() != 1 or seq_ptr.shape[0] < 2:
        raise ValueError(f"seq_ptr must be [B + 1], B >= 1 (got {tuple(seq_ptr.shape)})")
    _want("seq_ptr", seq_ptr, seq_ptr.shape, torch.int32, dev)
    return seq_ptr.shape[0] - 1


@_on_stream
def balance_loss(logits, topk_idx, alpha: float, beta: float = 0.0, bias=None, mask=None, seq_ptr=None, loss=None,
                 counts=None, saved=None, ws=None):
    """Balance loss and z-loss of the router over B sequences of tokens, with per-expert counts.

    logits fp32 [N,E] and topk_idx int32 [N,k] as route_topk takes and gives them; seq_ptr int32
    [B+1] (None: one sequence), mask uint8 or bool [N] (0: padding; None: no padding).
    -> dict(loss fp32 [2] (alpha's balance loss, beta's z-loss), counts int32 [B,E], saved fp32
    [B*E + 1] for balance_loss_bwd).  stream: a torch stream to run on (default: the current one)."""
    torch = _torch
    if logits.dim() != 2 or topk_idx.dim() != 2:
        raise ValueError("logits must be [N, E] and topk_idx [N, k]")
    N, E = logits.shape
    k = topk_idx.shape[1]
    dev = logits.get_device()
    _want("logits", logits, (N, E), torch.float32, dev)
    _want("topk_idx", topk_idx, (N, k), torch.int32, dev)
    if bias is not None:
        _want("bias", bias, (E,), torch.float32, dev)
    B = _seqs(N, mask, seq_ptr, dev)
    _on_gpu(logits)
    loss = _out("loss", loss, (2,), torch.float32, logits, dev)
    counts = _out("counts", counts, (B, E), torch.int32, logits, dev)
    saved = _out("saved", saved, (B * E + 1,), torch.float32, logits, dev)
    nb = _op_bytes(OP_BALANCE_LOSS, MOE_F32, N, E, k, 0, B, 0)
    ws = _op_ws(nb, logits, ws, dev)
    _check(lib().moe_balance_loss(_addr(logits), _addr(bias), _addr(topk_idx), _addr(mask), _addr(seq_ptr), B, N, E, k,
                                  alpha, beta, _addr(loss), _addr(counts), _addr(saved), _addr(ws), nb, _cur(dev)))
    return dict(loss=loss, counts=counts, saved=saved)


@_on_stream
def balance_loss_bwd(logits, saved, bias=None, mask=None, seq_ptr=None, dloss=None, dlogits_in=None, dlogits=None):
    """Gradient of balance_loss with respect to the logits, from its `saved` and the same logits,
    bias, mask and seq_ptr -> dlogits fp32 [N,E].  dloss fp32 [2]: the two losses' gradients (None:
    ones); dlogits_in is added (dlogits may be dlogits_in)."""
    torch = _torch
    if logits.dim() != 2:
        raise ValueError(f"logits must be [N, E] (got {tuple(logits.shape)})")
    N, E = logits.shape
    dev = logits.get_device()
    _want("logits", logits, (N, E), torch.float32, dev)
    if bias is not None:
        _want("bias", bias, (E,), torch.float32, dev)
    B = _seqs(N, mask, seq_ptr, dev)
    _want("saved", saved, (B * E + 1,), torch.float32, dev)
    if dloss is not None:
        _want("dloss", dloss, (2,), torch.float32, dev)
    if dlogits_in is not None:
        _want("dlogits_in", dlogits_in, (N, E), torch.float32, dev)
    _on_gpu(logits)
    dlogits = _out("dlogits", dlogits, (N, E), torch.float32, logits, dev)
    _check(lib().moe_balance_loss_bwd(_addr(logits), _addr(bias), _addr(mask), _addr(seq_ptr), B, N, E, _addr(saved),
                                      _addr(dloss), _addr(dlogits_in), _addr(dlogits), _cur(dev)))
    return dlogits


def _act(act):
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(ACTIVATIONS)} (got {act!r})")
    return ACTIVATIONS[act]


@_on_stream
def linear_fwd(x, w, bias=None, act="none", residual=None, want_z=False, out=None, z=None, ws=None):
    """out = act(x w^T + bias) + residual: x [N,K], w [O,K], residual [N,O] bf16 or fp32, bias fp32 [O];
    act: a key of ACTIVATIONS.  -> (out [N,O], z [N,O] (the product with its bias, for linear_bwd)
    or None).  out may be residual (in place).  stream: a torch stream to run on."""
    torch = _torch
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError("x must be [N, K] and w [O, K]")
    N, K = x.shape
    O = w.shape[0]
    dt, ty = _dtype_code(x), x.dtype
    dev = x.get_device()
    _want("x", x, (N, K), ty, dev)
    _want("w", w, (O, K), ty, dev)
    if bias is not None:
        _want("bias", bias, (O,), torch.float32, dev)
    if residual is not None:
        _want("residual", residual, (N, O), ty, dev)
    code = _act(act)
    _on_gpu(x)
    out = _out("out", out, (N, O), ty, x, dev)
    if want_z or z is not None:
        z = _out("z", z, (N, O), ty, x, dev)
    nb = _op_bytes(OP_LINEAR_FWD, dt, N, 1, 1, K, O, 0)
    ws = _op_ws(nb, x, ws, dev)
    _check(lib().moe_linear_fwd(dt, _addr(x), _addr(w), _addr(bias), code, _addr(residual), N, K, O, _addr(out), _addr(z),
                                _addr(ws), nb, _cur(dev)))
    return out, z


@_on_stream
def linear_bwd(dout, x, w, z=None, act="none", want_dx=True, want_dw=True, want_dbias=True, dx=None, dw=None,
               dbias=None, ws=None):
    """Backward of linear_fwd from dout [N,O] and the z it stored (None for act "none") -> dict(dx
    [N,K], dw [O,K], dbias fp32 [O]); what is not wanted is None.  residual's gradient is dout."""
    torch = _torch
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError("x must be [N, K] and w [O, K]")
    N, K = x.shape
    O = w.shape[0]
    dt, ty = _dtype_code(dout), dout.dtype
    dev = dout.get_device()
    _want("dout", dout, (N, O), ty, dev)
    _want("x", x, (N, K), ty, dev)
    _want("w", w, (O, K), ty, dev)
    code = _act(act)
    if z is not None:
        _want("z", z, (N, O), ty, dev)
    elif code:
        raise ValueError(f"the backward of {act} needs z")
    _on_gpu(dout)
    if want_dx or dx is not None:
        dx = _out("dx", dx, (N, K), ty, dout, dev)
    if want_dw or dw is not None:
        dw = _out("dw", dw, (O, K), ty, dout, dev)
    if want_dbias or dbias is not None:
        dbias = _out("dbias", dbias, (O,), torch.float32, dout, dev)
    nb = _op_bytes(OP_LINEAR_BWD, dt, N, 1, 1, K, O, 0)
    ws = _op_ws(nb, dout, ws, dev)
    if N or dw is not None or dbias is not None:
        _check(lib().moe_linear_bwd(dt, _addr(dout), _addr(x), _addr(w), _addr(z), code, N, K, O, _addr(dx), _addr(dw),
                                    _addr(dbias), _addr(ws), nb, _cur(dev)))
    return dict(dx=dx, dw=dw, dbias=dbias)


@_on_stream
def layer_few(x, w_r, w_gate, w_up, w_down, k: int, bias=None, out=None, topk_idx=None, topk_w=None, ws=None):
    """The whole expert layer for at most FEW_MAX_TOKENS tokens: router product, top-k, gate/up with
    SwiGLU, down and weighted sum.

    x [N,H] bf16 or fp32; w_r fp32 [H,E], bias fp32 [E] or None (-inf leaves an expert out); w_gate, w_up [E,I,H]
    and w_down [E,H,I] of x's type, or all three (codes, scale codes) from quantize_mxfp8 under bf16 x.
    -> dict(out [N,H], topk_idx int32 [N,k], topk_w fp32 [N,k]).  stream: a torch stream to run on."""
    torch = _torch
    quant = isinstance(w_gate, (tuple, list))
    mats = [("w_gate", w_gate), ("w_up", w_up), ("w_down", w_down)]
    if any(isinstance(m, (tuple, list)) != quant or (quant and len(m) != 2) for _, m in mats):
        raise ValueError("w_gate, w_up and w_down must all be tensors or all (codes, scale codes)")
    gate = w_gate[0] if quant else w_gate
    if x.dim() != 2 or w_r.dim() != 2 or gate.dim() != 3:
        raise ValueError("x must be [N, H], w_r [H, E], w_gate and w_up [E, I, H], w_down [E, H, I]")
    N, H = x.shape
    E, I = gate.shape[:2]
    dt, ty = _dtype_code(x), x.dtype
    if quant and dt != MOE_BF16:
        raise TypeError(f"MX-FP8 weights need x in bfloat16 (got {ty})")
    dev = x.get_device()
    _want("x", x, (N, H), ty, dev)
    _want("w_r", w_r, (H, E), torch.float32, dev)
    if bias is not None:
        _want("bias", bias, (E,), torch.float32, dev)
    for name, m in mats:
        shape = (E, H, I) if name == "w_down" else (E, I, H)
        if quant:
            _want(name + "'s codes", m[0], shape, torch.uint8, dev)
            _want(name + "'s scale codes", m[1], shape[:2] + (mx_scale_cols(shape[2]),), torch.uint8, dev)
        else:
            _want(name, m, shape, ty, dev)
    _on_gpu(x)
    out = _out("out", out, (N, H), ty, x, dev)
    topk_idx = _out("topk_idx", topk_idx, (N, k), torch.int32, x, dev)
    topk_w = _out("topk_w", topk_w, (N, k), torch.float32, x, dev)
    nb = _op_bytes(OP_LAYER_FEW, dt, N, E, k, H, I, 0)
    ws = _op_ws(nb, x, ws, dev)
    tail = (N, H, I, E, k, _addr(out), _addr(topk_idx), _addr(topk_w), _addr(ws), nb, _cur(dev))
    if quant:
        w = [_addr(t) for _, m in mats for t in m]
        _check(lib().moe_layer_few_mxfp8(_addr(x), _addr(w_r), _addr(bias), *w, *tail))
    else:
        _check(lib().moe_layer_few(dt, _addr(x), _addr(w_r), _addr(bias), _addr(w_gate), _addr(w_up), _addr(w_down), *tail))
    return dict(out=out, topk_idx=topk_idx, topk_w=topk_w)


def _ckpt_layer(H, w_gate, w_up, w_down, plan, dev):
    """The checks that the layer's 8-bit checkpoint calls share -> (E, I, rows of the row arrays)."""
    bf = _torch.bfloat16
    if w_gate.dim() != 3:
        raise ValueError("w_gate and w_up must be [E, I, H], w_down [E, H, I]")
    E, I = w_gate.shape[:2]
    if E != plan.E:
        raise ValueError(f"the plan is for {plan.E} experts, w_gate holds {E}")
    _want("w_gate", w_gate, (E, I, H), bf, dev)
    _want("w_up", w_up, (E, I, H), bf, dev)
    _want("w_down", w_down, (E, H, I), bf, dev)
    if plan.counts.get_device() != dev:
        raise ValueError(f"tensors on different devices: the plan is on {plan.counts.device}")
    return E, I, max(plan.M_cap, 1)


@_on_stream
def dequantize_mxfp8(q, scales, dtype=None, out=None):
    """The values that MX-FP8 codes q uint8 [..., K] and their scale codes (quantize_mxfp8's) stand for
    -> [..., K] in dtype (torch.bfloat16, the default, or torch.float32).  stream: a torch stream to run on."""
    torch = _torch
    K = q.shape[-1]
    rows = q.numel() // K if K else 0
    dev = q.get_device()
    if dtype is None:
        dtype = torch.bfloat16 if out is None else out.dtype
    _want("q", q, q.shape, torch.uint8, dev)
    _want("scales", scales, q.shape[:-1] + (mx_scale_cols(K),), torch.uint8, dev)
    _on_gpu(q)
    out = _out("out", out, q.shape, dtype, q, dev)
    _check(lib().moe_dequantize_mxfp8(_dtype_code(out), _addr(q), _addr(scales), rows, K, _addr(out), _cur(dev)))
    return out


@_on_stream
def grouped_gemm_fwd_ckpt8(x, w_gate, w_up, w_down, plan: Plan, hq=None, hs=None, y=None, ws=None):
    """grouped_gemm_fwd for bf16 layers that keeps [G | U] for the backward as MX-FP8 codes
    -> ((hq uint8 [M_cap, 2I], hs uint8 [M_cap, 2 mx_scale_cols(I)]), y [M_cap, H]); each half of a row is
    laid out as quantize_mxfp8 lays out a row of I values.  y is bit for bit grouped_gemm_fwd's.
    I a multiple of 32.  stream: a torch stream to run on (default: the current one)."""
    torch = _torch
    if x.dim() != 2:
        raise ValueError(f"x must be [N, H] (got {tuple(x.shape)})")
    H = x.shape[1]
    dev = x.get_device()
    _want("x", x, (plan.N, H), torch.bfloat16, dev)
    _, I, mc = _ckpt_layer(H, w_gate, w_up, w_down, plan, dev)
    _on_gpu(x)
    hq = _out("hq", hq, (mc, 2 * I), torch.uint8, x, dev)
    hs = _out("hs", hs, (mc, 2 * mx_scale_cols(I)), torch.uint8, x, dev)
    y = _out("y", y, (mc, H), torch.bfloat16, x, dev)
    nb = _op_bytes(OP_GEMM_FWD, MOE_BF16, plan.N, plan.E, plan.k, H, I, plan.M_cap)
    ws = _op_ws(nb, x, ws, dev)
    _check(lib().moe_grouped_gemm_fwd_ckpt8(_addr(x), _addr(w_gate), _addr(w_up), _addr(w_down), H, I, plan.c, _addr(hq),
                                            _addr(hs), _addr(y), _addr(ws), nb, _cur(dev)))
    return (hq, hs), y


@_on_stream
def layer_bwd_ckpt8(dout, x, w_gate, w_up, w_down, plan: Plan, hcache, dx=None, dw_gate=None, dw_up=None, dw_down=None,
                    ds=None, ws=None):
    """layer_bwd for bf16 layers at the [G | U] that hcache = (hq, hs) of grouped_gemm_fwd_ckpt8 stands for; x is
    bf16 [N,H], or (codes, scale codes) as add_rmsnorm and quantize_mxfp8 make them (dw_gate and dw_up are then taken
    at the values these stand for).  -> dict(dx, dw_gate, dw_up, dw_down, ds), as layer_bwd."""
    torch = _torch
    bf, u8 = torch.bfloat16, torch.uint8
    if dout.dim() != 2:
        raise ValueError(f"dout must be [N, H] (got {tuple(dout.shape)})")
    N, H = dout.shape
    dev = dout.get_device()
    _want("dout", dout, (plan.N, H), bf, dev)
    x, xs = x if isinstance(x, (tuple, list)) else (x, None)
    _want("x", x, (N, H), bf if xs is None else u8, dev)
    if xs is not None:
        _want("x's scale codes", xs, (N, mx_scale_cols(H)), u8, dev)
    _, I, mc = _ckpt_layer(H, w_gate, w_up, w_down, plan, dev)
    hq, hs = hcache
    _want("hq", hq, (mc, 2 * I), u8, dev)
    _want("hs", hs, (mc, 2 * mx_scale_cols(I)), u8, dev)
    _on_gpu(dout)
    dx = _out("dx", dx, (N, H), bf, dout, dev)
    dw_gate = _out("dw_gate", dw_gate, w_gate.shape, bf, dout, dev)
    dw_up = _out("dw_up", dw_up, w_up.shape, bf, dout, dev)
    dw_down = _out("dw_down", dw_down, w_down.shape, bf, dout, dev)
    ds = _out("ds", ds, (N, plan.k) if plan.kind == PLAN_TOPK else (mc,), torch.float32, dout, dev)
    nb = _op_bytes(OP_LAYER_BWD_CKPT8, MOE_BF16, plan.N, plan.E, plan.k, H, I, plan.M_cap)
    ws = _op_ws(nb, dout, ws, dev)
    _check(lib().moe_layer_bwd_ckpt8(_addr(dout), _addr(x), _addr(xs), _addr(w_gate), _addr(w_up), _addr(w_down), H, I,
                                     plan.c, _addr(hq), _addr(hs), _addr(dx), _addr(dw_gate), _addr(dw_up),
                                     _addr(dw_down), _addr(ds), _addr(ws), nb, _cur(dev)))
    return dict(dx=dx, dw_gate=dw_gate, dw_up=dw_up, dw_down=dw_down, ds=ds)


def _ce_args(x, w, targets):
    """The checks that linear_ce_fwd and its backward share -> (N, H, V, dtype code, device)."""
    torch = _torch
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError("x must be [N, H] and w [V, H]")
    N, H = x.shape
    V = w.shape[0]
    dev = x.get_device()
    _want("x", x, (N, H), x.dtype, dev)
    _want("w", w, (V, H), x.dtype, dev)
    _want("targets", targets, (N,), torch.int32, dev)
    return N, H, V, _dtype_code(x), dev


@_on_stream
def linear_ce_fwd(x, w, targets, z_coef: float = 0.0, loss=None, lse=None, ws=None):
    """Softmax cross entropy of the logits x w^T, which are never kept, with a z-loss: x [N,H] and w [V,H]
    bf16 or fp32, targets int32 [N] (outside [0, V), -100 say: the token takes no part).
    -> dict(loss fp32 [N]: lse - z_target + z_coef lse^2, lse fp32 [N]: log sum exp of the logits, for
    linear_ce_bwd); both 0 for tokens that take no part.  stream: a torch stream to run on."""
    torch = _torch
    N, H, V, dt, dev = _ce_args(x, w, targets)
    _on_gpu(x)
    loss = _out("loss", loss, (N,), torch.float32, x, dev)
    lse = _out("lse", lse, (N,), torch.float32, x, dev)
    nb = _op_bytes(OP_LINEAR_CE_FWD, dt, N, 1, 1, H, V, 0)
    ws = _op_ws(nb, x, ws, dev)
    _check(lib().moe_linear_ce_fwd(dt, _addr(x), _addr(w), _addr(targets), N, H, V, z_coef, _addr(loss), _addr(lse),
                                   _addr(ws), nb, _cur(dev)))
    return dict(loss=loss, lse=lse)


@functools.partial(_on_stream, at=1)
def linear_ce_bwd(dloss, x, w, targets, lse, z_coef: float = 0.0, want_dx=True, want_dw=True, dx=None, dw=None, ws=None):
    """Backward of linear_ce_fwd at the same x, w, targets and z_coef, from its lse and dloss fp32 [N], the
    gradients of the losses (None: ones) -> dict(dx [N,H] (zero for tokens that take no part), dw [V,H]); what is not
    wanted is None."""
    torch = _torch
    N, H, V, dt, dev = _ce_args(x, w, targets)
    if dloss is not None:
        _want("dloss", dloss, (N,), torch.float32, dev)
    _want("lse", lse, (N,), torch.float32, dev)
    _on_gpu(x)
    if want_dx or dx is not None:
        dx = _out("dx", dx, (N, H), x.dtype, x, dev)
    if want_dw or dw is not None:
        dw = _out("dw", dw, (V, H), x.dtype, x, dev)
    nb = _op_bytes(OP_LINEAR_CE_BWD, dt, N, 1, 1, H, V, 0)
    ws = _op_ws(nb, x, ws, dev)
    if N or dw is not None:
        _check(lib().moe_linear_ce_bwd(dt, _addr(dloss), _addr(x), _addr(w), _addr(targets), _addr(lse), N, H, V, z_coef,
                                       _addr(dx), _addr(dw), _addr(ws), nb, _cur(dev)))
    return dict(dx=dx, dw=dw)
