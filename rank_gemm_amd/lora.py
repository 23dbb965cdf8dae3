"""Python binding of liblora (include/lora.h): argument marshalling only.

Every step of the layer runs in the library: the planner in its host C++,
the GEMM, shrink, expand and pool writes in its gfx950 kernels. PyTorch is
used for device memory and streams (``torch.cuda.current_stream()``); the
library must be built (``python -m rank_gemm_amd.build``) and there is no
fallback of any kind: if it is missing, or no GPU is present, calls raise.

Names follow the C ABI: ``Pool.install`` -> lora_pool_install, ``plan`` ->
lora_plan, ``linear`` -> lora_linear, ``shrink`` -> lora_shrink,
``mx4_quantize`` -> lora_mx4_quantize, ``linear_mx4`` -> lora_linear_mx4,
``moe_route`` -> lora_moe_route, ``moe_experts`` -> lora_moe_experts.
"""
from __future__ import annotations

import ctypes
import os
import threading

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblora.so")

LORA_OK, LORA_EINVAL, LORA_ESLOT, LORA_ERANK, LORA_ENONFINITE, LORA_EHIP, LORA_ESPACE = 0, -1, -2, -3, -4, -5, -6
LORA_F32, LORA_BF16, LORA_MX4 = 0, 1, 2
LORA_PLAN_ROWS = 16

EXPORTS = (
    "lora_pool_create", "lora_pool_destroy", "lora_pool_install", "lora_pool_clear", "lora_pool_rank",
    "lora_plan", "lora_plan_max_items", "lora_workspace_bytes", "lora_linear", "lora_shrink",
    "lora_status_string", "lora_profile_begin", "lora_profile_end", "lora_workspace_bytes_multi",
    "lora_linear_multi", "lora_plan_device_words", "lora_plan_device", "lora_linear_device_plan",
    "lora_shrink_bgmv", "lora_linear_multi_device_plan", "lora_plan_chunked", "lora_delta", "lora_delta_bgmv",
    "lora_linear_noalloc", "lora_plan_upload", "lora_mx4_row_bytes", "lora_mx4_scale_bytes", "lora_mx4_quantize",
    "lora_mx4_dequantize", "lora_mx4_pack_scales", "lora_workspace_bytes_mx4", "lora_linear_mx4",
    "lora_linear_mx4_device_plan", "lora_moe_route_workspace_bytes", "lora_moe_route",
    "lora_moe_experts_workspace_bytes", "lora_moe_experts",
)
LORA_DEVICE_PLAN_MAX_SLOTS = 4096
LORA_NOALLOC_MAX_WORKSPACE = 32 << 20
LORA_MAX_SLICES = 4
LORA_MOE_MAX_EXPERTS, LORA_MOE_MAX_K, LORA_MOE_MAX_PAIRS = 512, 16, 512

_TORCH_DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
_CODE = {"bf16": LORA_BF16, "f32": LORA_F32}
_ACT = {"bf16": LORA_BF16, "mx4": LORA_MX4}


class LoraError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


class PlanInfo(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("S", ctypes.c_int32), ("T_a", ctypes.c_int32), ("k", ctypes.c_int32),
                ("n_items", ctypes.c_int32), ("max_seg", ctypes.c_int32), ("chunk", ctypes.c_int32)]


class SliceDesc(ctypes.Structure):
    """lora_slice: one projection of a multi-slice call."""
    _fields_ = [("pool", ctypes.c_void_p), ("W", ctypes.c_void_p), ("y", ctypes.c_void_p)]


class MoeWeightsDesc(ctypes.Structure):
    """lora_moe_weights: the experts' matrices of one layer."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("gate", "up", "down", "gate_scales", "up_scales", "down_scales")]


class KernelStat(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 48), ("count", ctypes.c_int32), ("mean_ms", ctypes.c_double),
                ("min_ms", ctypes.c_double), ("max_ms", ctypes.c_double), ("median_ms", ctypes.c_double)]


_lib = None
_lock = threading.Lock()
_P, _I, _F, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t


def lib():
    """Load liblora.so (raises if it was not built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m rank_gemm_amd.build`")
            L = ctypes.CDLL(LIB_PATH)
            L.lora_pool_create.argtypes = [ctypes.POINTER(_P), _I, _I, _I, _I, _I, _P, _P, _P, _P, _P]
            L.lora_pool_destroy.argtypes = [_P]
            L.lora_pool_destroy.restype = None
            L.lora_pool_install.argtypes = [_P, _I, _P, _P, _I, _F, _P]
            L.lora_pool_clear.argtypes = [_P, _I, _P]
            L.lora_pool_rank.argtypes = [_P, _I]
            L.lora_plan.argtypes = [_I, _P, _I, _P, _P, _P, _I, ctypes.POINTER(PlanInfo)]
            L.lora_plan_max_items.argtypes = [_I, _I]
            L.lora_plan_chunked.argtypes = [_I, _P, _I, _I, _P, _P, _P, _I, ctypes.POINTER(PlanInfo)]
            L.lora_delta.argtypes = [_P, _P, _P, _P, _P, ctypes.POINTER(PlanInfo), _P, _P, _SZ, _P]
            L.lora_delta_bgmv.argtypes = [_P, _P, _P, _I, _P, _P, _SZ, _P]
            L.lora_linear_noalloc.argtypes = [_P, _P, _P, _P, _P, _P, ctypes.POINTER(PlanInfo), _P, _P]
            L.lora_workspace_bytes.argtypes = [_P, _I]
            L.lora_workspace_bytes.restype = _SZ
            L.lora_linear.argtypes = [_P, _P, _P, _P, _P, _P, ctypes.POINTER(PlanInfo), _P, _P, _SZ, _P]
            L.lora_workspace_bytes_multi.argtypes = [ctypes.POINTER(SliceDesc), _I, _I]
            L.lora_workspace_bytes_multi.restype = _SZ
            L.lora_linear_multi.argtypes = [ctypes.POINTER(SliceDesc), _I, _P, _P, _P, _P, ctypes.POINTER(PlanInfo),
                                            _P, _SZ, _P]
            L.lora_plan_device_words.argtypes = [_I, _I]
            L.lora_plan_device_words.restype = _SZ
            L.lora_plan_device.argtypes = [_I, _P, _I, _P, _P]
            L.lora_plan_upload.argtypes = [_P, _P, _SZ, _P]
            L.lora_linear_device_plan.argtypes = [_P, _P, _P, _P, _I, _P, _P, _SZ, _P]
            L.lora_linear_multi_device_plan.argtypes = [ctypes.POINTER(SliceDesc), _I, _P, _P, _I, _P, _SZ, _P]
            L.lora_shrink_bgmv.argtypes = [_P, _P, _P, _I, _P, _P, _SZ, _P]
            L.lora_shrink.argtypes = [_P, _P, _P, _P, _P, ctypes.POINTER(PlanInfo), _P, _P, _SZ, _P]
            for name in ("lora_mx4_row_bytes", "lora_mx4_scale_bytes", "lora_workspace_bytes_mx4",
                         "lora_moe_route_workspace_bytes", "lora_moe_experts_workspace_bytes"):
                getattr(L, name).restype = _SZ
            L.lora_mx4_row_bytes.argtypes = [_I]
            L.lora_mx4_scale_bytes.argtypes = [_I, _I]
            L.lora_mx4_quantize.argtypes = [_I, _P, _I, _I, _I, _P, _P, _P]
            L.lora_mx4_dequantize.argtypes = [_P, _P, _I, _I, _I, _I, _P, _P]
            L.lora_mx4_pack_scales.argtypes = [_P, _I, _I, _I, _P, _P]
            L.lora_workspace_bytes_mx4.argtypes = [_P, _I, _I]
            L.lora_linear_mx4.argtypes = [_P, _P, _P, _P, _I, _P, _P, _P, ctypes.POINTER(PlanInfo), _P, _P, _SZ, _P]
            L.lora_linear_mx4_device_plan.argtypes = [_P, _P, _P, _P, _I, _P, _I, _P, _P, _SZ, _P]
            L.lora_moe_route_workspace_bytes.argtypes = [_I, _I, _I]
            L.lora_moe_route.argtypes = [_P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _SZ, _P]
            L.lora_moe_experts_workspace_bytes.argtypes = [_I, _I, _I, _I]
            L.lora_moe_experts.argtypes = [_I, _P, _P, _P, ctypes.POINTER(MoeWeightsDesc), _I, _I, _I, _I, _I, _P, _P,
                                           _SZ, _P]
            L.lora_profile_begin.argtypes = [_I]
            L.lora_profile_end.argtypes = [ctypes.POINTER(KernelStat), _I, ctypes.POINTER(_I)]
            L.lora_status_string.argtypes = [_I]
            L.lora_status_string.restype = ctypes.c_char_p
            _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().lora_status_string(int(status)).decode()


def _check(rc: int, what: str):
    if rc != LORA_OK:
        raise LoraError(rc, what)


def _require_gpu():
    if not torch.cuda.is_available():
        raise RuntimeError("liblora needs a HIP GPU; none is visible")


def _stream(device=None) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _dev_tensor(t: torch.Tensor, dtype, name: str, shape=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


def to_device(arr: np.ndarray, dtype: str, device="cuda") -> torch.Tensor:
    """Host array from rank_gemm_amd.inputs (uint16 bf16 bits or float32) ->
    device tensor of the pool's element type (bits unchanged)."""
    if dtype == "bf16":
        t = torch.from_numpy(np.ascontiguousarray(arr, np.uint16).view(np.int16)).view(torch.bfloat16)
    else:
        t = torch.from_numpy(np.ascontiguousarray(arr, np.float32))
    return t.to(device)


class Pool:
    """Device slot pool: A [S, r_max, d_in], B [S, d_out, r_max], rank [S],
    scale [S]; slot 0 is the zero adapter."""

    def __init__(self, S: int, r_max: int, d_in: int, d_out: int, dtype: str = "bf16", device="cuda"):
        _require_gpu()
        self.S, self.r_max, self.d_in, self.d_out, self.dtype = S, r_max, d_in, d_out, dtype
        self.device = torch.device(device)
        tdt = _TORCH_DTYPE[dtype]
        with torch.cuda.device(self.device):
            self.A = torch.empty((S, r_max, d_in), dtype=tdt, device=self.device)
            self.B = torch.empty((S, d_out, r_max), dtype=tdt, device=self.device)
            self.rank_dev = torch.empty(S, dtype=torch.int32, device=self.device)
            self.scale_dev = torch.empty(S, dtype=torch.float32, device=self.device)
            h = _P()
            _check(lib().lora_pool_create(ctypes.byref(h), S, r_max, d_in, d_out, _CODE[dtype], self.A.data_ptr(),
                                          self.B.data_ptr(), self.rank_dev.data_ptr(), self.scale_dev.data_ptr(),
                                          _stream(self.device)), "lora_pool_create")
        self._h = h
        self._ws = {}  # stream handle -> workspace
        self._ws_retired = []

    @property
    def handle(self):
        return self._h

    def install(self, slot: int, A: torch.Tensor, B: torch.Tensor, alpha: float):
        """lora_pool_install: A [r, d_in], B [d_out, r] device tensors."""
        tdt = _TORCH_DTYPE[self.dtype]
        if A.dim() != 2 or B.dim() != 2:
            raise ValueError("A and B must be 2-D")
        r = A.shape[0]
        _dev_tensor(A, tdt, "A", (r, self.d_in))
        _dev_tensor(B, tdt, "B", (self.d_out, r))
        with torch.cuda.device(self.device):
            _check(lib().lora_pool_install(self._h, int(slot), A.data_ptr(), B.data_ptr(), int(r), float(alpha),
                                           _stream(self.device)), "lora_pool_install")

    def clear(self, slot: int):
        with torch.cuda.device(self.device):
            _check(lib().lora_pool_clear(self._h, int(slot), _stream(self.device)), "lora_pool_clear")

    def rank(self, slot: int) -> int:
        return lib().lora_pool_rank(self._h, int(slot))

    def workspace_bytes(self, T: int) -> int:
        return int(lib().lora_workspace_bytes(self._h, int(T)))

    def workspace(self, T: int) -> torch.Tensor:
        """A device workspace of at least workspace_bytes(T) for calls on the
        current stream. One buffer per stream, so calls on two streams never
        share one; calls on one stream reuse it in stream order. A buffer
        that grows is replaced, but the old one is kept until the pool is
        released (a captured graph or a call still in flight may use it)."""
        n = self.workspace_bytes(T)
        key = torch.cuda.current_stream(self.device).cuda_stream
        ws = self._ws.get(key)
        if ws is None or ws.numel() < n:
            if ws is not None:
                self._ws_retired.append(ws)
            ws = torch.empty(max(n, 256), dtype=torch.uint8, device=self.device)
            self._ws[key] = ws
        return ws

    def __del__(self):
        h = getattr(self, "_h", None)
        if h and _lib is not None:
            _lib.lora_pool_destroy(h)
            self._h = None


class Plan:
    """Host result of lora_plan plus its device copy."""

    def __init__(self, S, T, info, host, dev, n_work, chunk=LORA_PLAN_ROWS):
        self.S, self.T, self.info, self.chunk = S, T, info, chunk
        self.host = host  # pinned int32: [work 4*n_work][token_order T][slot_indptr S+1]
        self.dev = dev
        self._n_work = n_work
        self._ptrs = None  # addresses in dev, which stays for the plan's lifetime
        # plan_into staging: two pinned buffers used in turn, the copy that
        # last read each (None: not read yet), the one to write next
        self._stage, self._ev, self._turn = [None, None], [None, None], 0

    def _off(self, which):
        if which == "work":
            return 0
        if which == "token_order":
            return 4 * self._n_work
        return 4 * self._n_work + self.T

    @property
    def token_order(self) -> np.ndarray:
        o = self._off("token_order")
        return self.host[o:o + self.T].numpy()

    @property
    def slot_indptr(self) -> np.ndarray:
        o = self._off("slot_indptr")
        return self.host[o:o + self.S + 1].numpy()

    @property
    def work(self) -> np.ndarray:
        return self.host[: 4 * self.info.n_items].numpy().reshape(-1, 4)

    def dev_ptrs(self):
        if self._ptrs is None:
            base = self.dev.data_ptr() if self.dev is not None else 0
            self._ptrs = tuple(base + 4 * self._off(n) for n in ("token_order", "slot_indptr", "work"))
        return self._ptrs


def plan(slot_ids, S: int, device="cuda", upload: bool = True, chunk: int = LORA_PLAN_ROWS) -> Plan:
    """lora_plan (or lora_plan_chunked for ``chunk`` of 32, 64 or 128 rows
    per work item) over host slot ids; with ``upload`` the result is copied
    to ``device`` on the current stream (non-blocking, from pinned memory).
    lora_linear, lora_linear_multi and lora_shrink take 16-row plans only;
    lora_delta takes any chunk."""
    ids = np.ascontiguousarray(np.asarray(slot_ids), dtype=np.int32)
    if ids.ndim != 1:
        raise ValueError("slot_ids must be 1-D")
    T = int(ids.shape[0])
    n_work = max(int(lib().lora_plan_max_items(T, int(S))), 1)
    total = 4 * n_work + T + S + 1
    pin = upload and torch.cuda.is_available()
    host = torch.empty(total, dtype=torch.int32, pin_memory=pin)
    base = host.data_ptr()
    info = PlanInfo()
    _check(lib().lora_plan_chunked(int(S), ids.ctypes.data, T, int(chunk), base + 16 * n_work,
                                   base + 4 * (4 * n_work + T), base, n_work, ctypes.byref(info)),
           "lora_plan_chunked")
    dev = None
    if upload:
        _require_gpu()
        dev = torch.empty(total, dtype=torch.int32, device=device)
        with torch.cuda.device(dev.device):
            _check(lib().lora_plan_upload(base, dev.data_ptr(), total, _stream(dev.device)), "lora_plan_upload")
    p = Plan(int(S), T, info, host, dev, n_work, int(chunk))
    if upload:
        # the staging buffers of plan_into, allocated now rather than on
        # first use: pinning host memory stalls the kernels running then
        ev = torch.cuda.Event()
        ev.record()
        p._stage = [host, torch.empty(total, dtype=torch.int32, pin_memory=True)]
        p._ev = [ev, None]
        p._turn = 1
    return p


def plan_into(p: Plan, slot_ids) -> Plan:
    """Re-plan ``slot_ids`` into the device buffer of an existing plan (same
    T and S, same chunk), so work captured against that buffer sees the new
    plan. The summary (p.info) is refreshed; kernels captured with an older
    summary stay valid only while it is unchanged, which the caller checks.

    The plan is written into one of two pinned staging buffers that the plan
    owns for its lifetime (the first is the buffer lora_plan filled), in
    turn, and copied from there on the current stream by lora_plan_upload
    (a kernel reading the pinned buffer in place). Before a staging
    buffer is written again, the host waits for the copy that last read it
    (two plans back). No pinned memory is allocated here: registering new
    host memory with the GPU stalls the kernels running at that moment."""
    ids = np.ascontiguousarray(np.asarray(slot_ids), dtype=np.int32)
    if ids.ndim != 1 or ids.shape[0] != p.T:
        raise ValueError("plan_into needs the same T and S")
    if p.dev is None:
        raise ValueError("plan was not uploaded")
    k = p._turn
    p._turn ^= 1
    if p._ev[k] is None:
        p._ev[k] = torch.cuda.Event()
    else:
        p._ev[k].synchronize()
    host = p._stage[k]
    base = host.data_ptr()
    info = PlanInfo()
    _check(lib().lora_plan_chunked(int(p.S), ids.ctypes.data, p.T, p.chunk, base + 16 * p._n_work,
                                   base + 4 * (4 * p._n_work + p.T), base, p._n_work, ctypes.byref(info)),
           "lora_plan_chunked")
    with torch.cuda.device(p.dev.device):
        _check(lib().lora_plan_upload(base, p.dev.data_ptr(), int(p.dev.numel()), _stream(p.dev.device)),
               "lora_plan_upload")
    p._ev[k].record()
    p.host, p.info = host, info
    return p


class DevicePlan:
    """A plan built on the device by lora_plan_device: one int32 buffer
    [work 4 W][token_order T][slot_indptr S + 1][info 8]."""

    def __init__(self, S: int, T: int, buf: torch.Tensor):
        self.S, self.T, self.buf = S, T, buf
        self.cap = max(int(lib().lora_plan_max_items(T, S)), 1)

    def read(self) -> dict:
        """Copy the plan to the host (synchronises): work (live items only),
        token_order, slot_indptr and the info words."""
        h = self.buf.cpu().numpy()
        o = 4 * self.cap
        info = h[o + self.T + self.S + 1:]
        keys = ("T", "S", "T_a", "k", "n_items", "max_seg", "status")
        d = {k: int(v) for k, v in zip(keys, info)}
        d["work"] = h[:4 * d["n_items"]].reshape(-1, 4)
        d["pad"] = h[4 * d["n_items"]:o].reshape(-1, 4)
        d["token_order"] = h[o:o + self.T]
        d["slot_indptr"] = h[o + self.T:o + self.T + self.S + 1]
        return d


def plan_device(slot_ids: torch.Tensor, S: int, out: DevicePlan | None = None) -> DevicePlan:
    """lora_plan_device: plan device-resident int32 slot ids on the current
    stream (no host work; graph-capturable). ``out`` reuses a buffer of the
    same T and S."""
    _dev_tensor(slot_ids, torch.int32, "slot_ids")
    if slot_ids.dim() != 1:
        raise ValueError("slot_ids must be 1-D")
    T = int(slot_ids.shape[0])
    words = int(lib().lora_plan_device_words(T, int(S)))
    if words == 0:
        raise ValueError(f"no device plan for T={T}, S={S} (1 <= S <= {LORA_DEVICE_PLAN_MAX_SLOTS})")
    if out is None:
        out = DevicePlan(int(S), T, torch.empty(words, dtype=torch.int32, device=slot_ids.device))
    elif out.T != T or out.S != S:
        raise ValueError("plan buffer has another T or S")
    _check(lib().lora_plan_device(int(S), slot_ids.data_ptr(), T, out.buf.data_ptr(), _stream(slot_ids.device)),
           "lora_plan_device")
    return out


def linear(x: torch.Tensor, W: torch.Tensor, pool: Pool, p, y: torch.Tensor | None = None,
           workspace: torch.Tensor | None = None) -> torch.Tensor:
    """lora_linear (host plan) or lora_linear_device_plan (DevicePlan):
    y = x W^T + per-row adapter correction."""
    tdt = _TORCH_DTYPE[pool.dtype]
    T = p.T
    _dev_tensor(x, tdt, "x", (T, pool.d_in))
    _dev_tensor(W, tdt, "W", (pool.d_out, pool.d_in))
    if y is None:
        y = torch.empty((T, pool.d_out), dtype=tdt, device=x.device)
    _dev_tensor(y, tdt, "y", (T, pool.d_out))
    ws = workspace if workspace is not None else pool.workspace(T)
    if isinstance(p, DevicePlan):
        if p.S != pool.S:
            raise ValueError("plan and pool have different S")
        _check(lib().lora_linear_device_plan(pool.handle, x.data_ptr(), W.data_ptr(), p.buf.data_ptr(), T,
                                             y.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size(),
                                             _stream(x.device)), "lora_linear_device_plan")
        return y
    if p.dev is None:
        raise ValueError("plan was not uploaded")
    to, ip, wk = p.dev_ptrs()
    _check(lib().lora_linear(pool.handle, x.data_ptr(), W.data_ptr(), to, ip, wk, ctypes.byref(p.info), y.data_ptr(),
                             ws.data_ptr(), ws.numel() * ws.element_size(), _stream(x.device)), "lora_linear")
    return y


def _slice_array(pools, Ws=None, ys=None):
    n = len(pools)
    arr = (SliceDesc * max(n, 1))()
    for i, pool in enumerate(pools):
        arr[i].pool = pool.handle
        arr[i].W = Ws[i].data_ptr() if Ws is not None else None
        arr[i].y = ys[i].data_ptr() if ys is not None else None
    return arr


def workspace_bytes_multi(pools, T: int) -> int:
    """lora_workspace_bytes_multi (0 when the pools cannot share a call)."""
    return int(lib().lora_workspace_bytes_multi(_slice_array(pools, None, None), len(pools), int(T)))


def linear_multi(x: torch.Tensor, Ws, pools, p: Plan, ys=None, workspace: torch.Tensor | None = None):
    """lora_linear_multi: y_i = x W_i^T + per-row correction from pools[i],
    for slices that share x and the plan (a merged q/k/v or gate/up)."""
    n = len(pools)
    if not 1 <= n <= LORA_MAX_SLICES or len(Ws) != n:
        raise ValueError(f"need 1..{LORA_MAX_SLICES} pools and as many weights")
    tdt = _TORCH_DTYPE[pools[0].dtype]
    T = p.T
    _dev_tensor(x, tdt, "x", (T, pools[0].d_in))
    if not isinstance(p, DevicePlan) and p.dev is None:
        raise ValueError("plan was not uploaded")
    if ys is None:
        ys = [torch.empty((T, pl.d_out), dtype=tdt, device=x.device) for pl in pools]
    for i, pl in enumerate(pools):
        _dev_tensor(Ws[i], tdt, f"W[{i}]", (pl.d_out, pl.d_in))
        _dev_tensor(ys[i], tdt, f"y[{i}]", (T, pl.d_out))
    arr = _slice_array(pools, Ws, ys)
    if workspace is None:
        need = int(lib().lora_workspace_bytes_multi(arr, n, T))
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    if isinstance(p, DevicePlan):
        if p.S != pools[0].S:
            raise ValueError("plan and pools have different S")
        _check(lib().lora_linear_multi_device_plan(arr, n, x.data_ptr(), p.buf.data_ptr(), T, workspace.data_ptr(),
                                                   workspace.numel() * workspace.element_size(), _stream(x.device)),
               "lora_linear_multi_device_plan")
        return ys
    to, ip, wk = p.dev_ptrs()
    _check(lib().lora_linear_multi(arr, n, x.data_ptr(), to, ip, wk, ctypes.byref(p.info), workspace.data_ptr(),
                                   workspace.numel() * workspace.element_size(), _stream(x.device)),
           "lora_linear_multi")
    return ys


def shrink(x: torch.Tensor, pool: Pool, p: Plan, h: torch.Tensor | None = None) -> torch.Tensor:
    """lora_shrink: h [T, r_max] fp32 (zeros past each row's rank)."""
    tdt = _TORCH_DTYPE[pool.dtype]
    _dev_tensor(x, tdt, "x", (p.T, pool.d_in))
    if h is None:
        h = torch.empty((p.T, pool.r_max), dtype=torch.float32, device=x.device)
    _dev_tensor(h, torch.float32, "h", (p.T, pool.r_max))
    ws = pool.workspace(p.T)
    to, ip, wk = p.dev_ptrs()
    _check(lib().lora_shrink(pool.handle, x.data_ptr(), to, ip, wk, ctypes.byref(p.info), h.data_ptr(), ws.data_ptr(),
                             ws.numel(), _stream(x.device)), "lora_shrink")
    return h


def shrink_bgmv(x: torch.Tensor, pool: Pool, slot_ids: torch.Tensor, h: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None) -> torch.Tensor:
    """lora_shrink_bgmv: h [T, r_max] fp32 in token order from device slot ids (no plan)."""
    tdt = _TORCH_DTYPE[pool.dtype]
    _dev_tensor(slot_ids, torch.int32, "slot_ids")
    T = int(slot_ids.shape[0])
    _dev_tensor(x, tdt, "x", (T, pool.d_in))
    if h is None:
        h = torch.empty((T, pool.r_max), dtype=torch.float32, device=x.device)
    _dev_tensor(h, torch.float32, "h", (T, pool.r_max))
    ws = workspace if workspace is not None else pool.workspace(T)
    _check(lib().lora_shrink_bgmv(pool.handle, x.data_ptr(), slot_ids.data_ptr(), T, h.data_ptr(), ws.data_ptr(),
                                  ws.numel() * ws.element_size(), _stream(x.device)), "lora_shrink_bgmv")
    return h


def correction(x: torch.Tensor, pool: Pool, p: Plan, y: torch.Tensor,
               workspace: torch.Tensor | None = None) -> torch.Tensor:
    """lora_delta: y += per-row adapter correction (SGMV over a plan of any
    chunk); rows on slot 0 are not touched."""
    tdt = _TORCH_DTYPE[pool.dtype]
    _dev_tensor(x, tdt, "x", (p.T, pool.d_in))
    _dev_tensor(y, tdt, "y", (p.T, pool.d_out))
    if p.dev is None:
        raise ValueError("plan was not uploaded")
    ws = workspace if workspace is not None else pool.workspace(p.T)
    to, ip, wk = p.dev_ptrs()
    _check(lib().lora_delta(pool.handle, x.data_ptr(), to, ip, wk, ctypes.byref(p.info), y.data_ptr(), ws.data_ptr(),
                            ws.numel() * ws.element_size(), _stream(x.device)), "lora_delta")
    return y


def correction_bgmv(x: torch.Tensor, pool: Pool, slot_ids: torch.Tensor, y: torch.Tensor,
                    workspace: torch.Tensor | None = None) -> torch.Tensor:
    """lora_delta_bgmv: y += per-row adapter correction, token by token from
    device slot ids (no plan)."""
    tdt = _TORCH_DTYPE[pool.dtype]
    _dev_tensor(slot_ids, torch.int32, "slot_ids")
    T = int(slot_ids.shape[0])
    _dev_tensor(x, tdt, "x", (T, pool.d_in))
    _dev_tensor(y, tdt, "y", (T, pool.d_out))
    ws = workspace if workspace is not None else pool.workspace(T)
    _check(lib().lora_delta_bgmv(pool.handle, x.data_ptr(), slot_ids.data_ptr(), T, y.data_ptr(), ws.data_ptr(),
                                 ws.numel() * ws.element_size(), _stream(x.device)), "lora_delta_bgmv")
    return y


class Mx4:
    """A matrix, or a batch of matrices, held as MXFP4 rows: ``codes`` uint8
    [..., rows, lora_mx4_row_bytes(K)] and ``scales`` uint8 [...,
    lora_mx4_scale_bytes(rows, K)] in the order the products read them.
    ``shape`` is that of the values. Checked here once; the buffers stay."""

    __slots__ = ("_codes", "_scales", "K", "rows", "batch", "shape", "device")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, K: int):
        K = int(K)
        if codes.dim() not in (2, 3) or K < 1:
            raise ValueError("MXFP4 rows need codes [rows, bytes] or [batch, rows, bytes] and K of at least 1")
        lead, rows = codes.shape[:-2], int(codes.shape[-2])
        for name, t, shape in (("codes", codes, (*lead, rows, int(lib().lora_mx4_row_bytes(K)))),
                               ("scales", scales, (*lead, int(lib().lora_mx4_scale_bytes(rows, K))))):
            if t.dtype != torch.uint8 or not t.is_contiguous() or tuple(t.shape) != shape:
                raise ValueError(f"{name} must be contiguous uint8 of shape {shape}, got {t.dtype} {tuple(t.shape)}")
        if codes.device != scales.device:
            raise ValueError(f"codes are on {codes.device}, scales on {scales.device}")
        self._codes, self._scales, self.K, self.rows = codes, scales, K, rows
        self.batch = int(lead[0]) if lead else 1
        self.shape, self.device = (*lead, rows, K), codes.device

    @property
    def codes(self) -> torch.Tensor:
        return self._codes

    @property
    def scales(self) -> torch.Tensor:
        return self._scales

    @staticmethod
    def empty(shape, device="cuda") -> "Mx4":
        """Buffers for values of ``shape`` ([rows, K] or [batch, rows, K])."""
        if len(shape) not in (2, 3) or shape[-1] < 1:
            raise ValueError(f"MXFP4 rows need a shape [rows, K] or [batch, rows, K], got {tuple(shape)}")
        *lead, rows, K = (int(n) for n in shape)
        rb, sb = int(lib().lora_mx4_row_bytes(K)), int(lib().lora_mx4_scale_bytes(rows, K))
        return Mx4(torch.empty((*lead, rows, rb), dtype=torch.uint8, device=device),
                   torch.empty((*lead, sb), dtype=torch.uint8, device=device), K)


def _mx4(q, name: str, shape=None) -> Mx4:
    if not isinstance(q, Mx4) or q.device.type != "cuda":
        raise ValueError(f"{name} must be an Mx4 on a GPU")
    if shape is not None and q.shape != tuple(shape):
        raise ValueError(f"{name} has shape {q.shape}, expected {tuple(shape)}")
    return q


def _same_device(*named):
    dev = named[0][1].device
    for name, t in named:
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, {named[0][0]} on {dev}")
    return dev


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _call(dev, fn, what: str, *args):
    """One call of the library on ``dev``'s current stream, with ``dev`` the
    current device (a decode step makes many such calls: the stream's handle
    is fetched without building a Stream object where torch offers it)."""
    if torch.cuda.current_device() != dev.index:
        with torch.cuda.device(dev):
            rc = fn(*args, _stream(dev))
    else:
        rc = fn(*args, _raw_stream(dev.index) if _raw_stream is not None else _stream(dev))
    if rc != LORA_OK:
        raise LoraError(rc, what)


_DTYPE_NAME = {t: n for n, t in _TORCH_DTYPE.items()}


def mx4_quantize(src: torch.Tensor, out: Mx4 | None = None) -> Mx4:
    """lora_mx4_quantize: bf16 or fp32 rows ([rows, K] or [batch, rows, K]) to
    MXFP4. ``out`` reuses buffers of the same shape."""
    dt = _DTYPE_NAME.get(getattr(src, "dtype", None))
    if dt is None:
        raise ValueError("src must be a bf16 or fp32 device tensor")
    _dev_tensor(src, src.dtype, "src")
    if out is None:
        out = Mx4.empty(src.shape, src.device)
    _mx4(out, "out", src.shape)
    _call(_same_device(("src", src), ("out", out)), lib().lora_mx4_quantize, "lora_mx4_quantize", _CODE[dt],
          src.data_ptr(), out.batch, out.rows, out.K, out._codes.data_ptr(), out._scales.data_ptr())
    return out


def mx4_dequantize(q: Mx4, dtype: str = "bf16", out: torch.Tensor | None = None) -> torch.Tensor:
    """lora_mx4_dequantize: the values MXFP4 codes stand for, in "bf16" or "f32"."""
    _mx4(q, "q")
    if out is None:
        out = torch.empty(q.shape, dtype=_TORCH_DTYPE[dtype], device=q.device)
    _dev_tensor(out, _TORCH_DTYPE[dtype], "out", q.shape)
    _call(_same_device(("q", q), ("out", out)), lib().lora_mx4_dequantize, "lora_mx4_dequantize",
          q._codes.data_ptr(), q._scales.data_ptr(), q.batch, q.rows, q.K, _CODE[dtype], out.data_ptr())
    return out


def mx4_pack(codes: torch.Tensor, e8m0: torch.Tensor, K: int) -> Mx4:
    """MXFP4 rows as a checkpoint holds them (codes uint8 [..., rows, 16
    ceil(K / 32)], one scale byte per block, [..., rows, ceil(K / 32)]) as an
    Mx4: the codes stay, the scales are laid out by lora_mx4_pack_scales."""
    _dev_tensor(codes, torch.uint8, "codes")
    if codes.dim() not in (2, 3) or int(K) < 1:
        raise ValueError("codes must be [rows, bytes] or [batch, rows, bytes], K at least 1")
    lead, rows = codes.shape[:-2], int(codes.shape[-2])
    _dev_tensor(e8m0, torch.uint8, "e8m0", (*lead, rows, (int(K) + 31) // 32))
    q = Mx4(codes, torch.empty((*lead, int(lib().lora_mx4_scale_bytes(rows, int(K)))), dtype=torch.uint8,
                               device=codes.device), K)
    _call(_same_device(("codes", codes), ("e8m0", e8m0)), lib().lora_mx4_pack_scales, "lora_mx4_pack_scales",
          e8m0.data_ptr(), q.batch, rows, q.K, q._scales.data_ptr())
    return q


def _space(workspace, n: int, dev):
    """(address, bytes) of the caller's workspace, or of a new one of n bytes.
    One per call: torch hands its memory on in stream order, and a captured
    graph keeps its own, so no two calls that may overlap share one."""
    if workspace is None:
        workspace = torch.empty(max(int(n), 256), dtype=torch.uint8, device=dev)
        return workspace, workspace.data_ptr(), workspace.numel()
    if workspace.device != dev:
        raise ValueError(f"workspace is on {workspace.device}, the inputs on {dev}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def linear_mx4(x: torch.Tensor, W: Mx4, pool: Pool, p, act: str = "bf16", y: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None) -> torch.Tensor:
    """lora_linear_mx4 (host plan) or lora_linear_mx4_device_plan (DevicePlan):
    y = act(x) What^T + per-row adapter correction over a base weight in
    MXFP4. ``act``: "bf16" (x as it is) or "mx4" (x rounded to MXFP4 for the
    base product; the correction reads x itself)."""
    code = _ACT.get(act)
    if code is None:
        raise ValueError(f"act must be one of {sorted(_ACT)}, got {act!r}")
    if pool.dtype != "bf16":
        raise ValueError("linear_mx4 needs a bf16 pool")
    T = p.T
    _dev_tensor(x, torch.bfloat16, "x", (T, pool.d_in))
    _mx4(W, "W", (pool.d_out, pool.d_in))
    if y is None:
        y = torch.empty((T, pool.d_out), dtype=torch.bfloat16, device=x.device)
    _dev_tensor(y, torch.bfloat16, "y", (T, pool.d_out))
    device_plan = isinstance(p, DevicePlan)
    if not device_plan and p.dev is None:
        raise ValueError("plan was not uploaded")
    if device_plan and p.S != pool.S:
        raise ValueError("plan and pool have different S")
    dev, pd = x.device, p.buf if device_plan else p.dev
    if W.device != dev or pool.A.device != dev or y.device != dev or pd.device != dev:
        _same_device(("x", x), ("W", W), ("pool", pool.A), ("y", y), ("plan", pd))
    L = lib()
    n = L.lora_workspace_bytes_mx4(pool.handle, T, code) if workspace is None else 0
    keep, ws, nb = _space(workspace, n, dev)
    base = (pool.handle, x.data_ptr(), W._codes.data_ptr(), W._scales.data_ptr(), code)
    if device_plan:
        _call(dev, L.lora_linear_mx4_device_plan, "lora_linear_mx4_device_plan", *base, p.buf.data_ptr(), T,
              y.data_ptr(), ws, nb)
    else:
        _call(dev, L.lora_linear_mx4, "lora_linear_mx4", *base, *p.dev_ptrs(), ctypes.byref(p.info), y.data_ptr(),
              ws, nb)
    return y


def moe_route(x: torch.Tensor, router: torch.Tensor, k: int, renorm: bool = True):
    """lora_moe_route: (ids int32 [T, k], weights fp32 [T, k]) of the k experts
    with the largest logits x router^T, their softmax taken over the chosen
    (``renorm``) or over all experts. x [T, H], router [E, H], bf16."""
    _dev_tensor(x, torch.bfloat16, "x")
    _dev_tensor(router, torch.bfloat16, "router")
    if x.dim() != 2 or router.dim() != 2 or router.shape[1] != x.shape[1]:
        raise ValueError(f"x {tuple(x.shape)} and router {tuple(router.shape)} must be [T, H] and [E, H]")
    (T, H), E, k = x.shape, router.shape[0], int(k)
    dev = _same_device(("x", x), ("router", router))
    ids = torch.empty((T, max(k, 0)), dtype=torch.int32, device=dev)
    weights = torch.empty((T, max(k, 0)), dtype=torch.float32, device=dev)
    L = lib()
    n = L.lora_moe_route_workspace_bytes(T, H, E)
    keep, ws, nb = _space(None, n, dev) if n else (None, None, 0)
    _call(dev, L.lora_moe_route, "lora_moe_route", x.data_ptr(), router.data_ptr(), T, H, E, k, int(bool(renorm)),
          ids.data_ptr(), weights.data_ptr(), ws, nb)
    return ids, weights


def moe_experts(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, gate, up, down,
                y: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """lora_moe_experts: y[t] = sum_j weights[t, j] down_e(silu(gate_e x_t) *
    up_e x_t), e = ids[t, j]. gate, up [E, I, H] and down [E, H, I], all bf16
    tensors or all Mx4 batches."""
    _dev_tensor(x, torch.bfloat16, "x")
    _dev_tensor(ids, torch.int32, "ids")
    if x.dim() != 2 or ids.dim() != 2 or ids.shape[0] != x.shape[0]:
        raise ValueError(f"x {tuple(x.shape)} and ids {tuple(ids.shape)} must be [T, H] and [T, k]")
    (T, H), k = x.shape, ids.shape[1]
    _dev_tensor(weights, torch.float32, "weights", (T, k))
    mx4 = isinstance(gate, Mx4)
    if len(gate.shape) != 3:
        raise ValueError(f"gate must be [E, I, H], got {tuple(gate.shape)}")
    E, I = gate.shape[:2]
    if mx4:
        _mx4(gate, "gate", (E, I, H)), _mx4(up, "up", (E, I, H)), _mx4(down, "down", (E, H, I))
        d = MoeWeightsDesc(*(w._codes.data_ptr() for w in (gate, up, down)),
                           *(w._scales.data_ptr() for w in (gate, up, down)))
    else:
        for name, w, shape in (("gate", gate, (E, I, H)), ("up", up, (E, I, H)), ("down", down, (E, H, I))):
            _dev_tensor(w, torch.bfloat16, name, shape)
        d = MoeWeightsDesc(gate.data_ptr(), up.data_ptr(), down.data_ptr())
    if y is None:
        y = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
    _dev_tensor(y, torch.bfloat16, "y", (T, H))
    dev = _same_device(("x", x), ("ids", ids), ("weights", weights), ("gate", gate), ("up", up), ("down", down),
                       ("y", y))
    L = lib()
    n = L.lora_moe_experts_workspace_bytes(T, H, I, k) if workspace is None else 0
    keep, ws, nb = _space(workspace, n, dev)
    _call(dev, L.lora_moe_experts, "lora_moe_experts", LORA_MX4 if mx4 else LORA_BF16, x.data_ptr(), ids.data_ptr(),
          weights.data_ptr(), ctypes.byref(d), T, H, I, E, k, y.data_ptr(), ws, nb)
    return y


def profile_begin(max_records: int = 100000):
    """lora_profile_begin: start recording per-kernel HIP event pairs."""
    _check(lib().lora_profile_begin(int(max_records)), "lora_profile_begin")


def profile_end() -> dict:
    """lora_profile_end: {kernel name: {count, mean_ms, min_ms, max_ms, median_ms}}."""
    cap = 32
    out = (KernelStat * cap)()
    n = _I()
    _check(lib().lora_profile_end(out, cap, ctypes.byref(n)), "lora_profile_end")
    return {out[i].name.decode(): {"count": out[i].count, "mean_ms": out[i].mean_ms, "min_ms": out[i].min_ms,
                                   "max_ms": out[i].max_ms, "median_ms": out[i].median_ms}
            for i in range(min(n.value, cap))}
