"""ctypes binding of libnvfp4moe.so (argument marshalling only).

Every function here has the name of the C entry point it calls (see
``include/nvfp4_moe.h``, ``include/mxfp4.h`` and ``include/moe_balance.h``)
and does nothing but check tensor placement, dtypes and shapes, allocate
outputs and workspace with torch, pass raw device pointers and torch's current
CUDA stream, and turn a non-OK status into an exception.  All arithmetic of the layer runs in the library's CUDA kernels;
there is no CPU path.  Importing this module loads the library and fails
loudly when it has not been built.
"""
from __future__ import annotations

import ctypes
import dataclasses
import os
from dataclasses import dataclass

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libnvfp4moe.so")

LAYOUT_CANONICAL = 0
LAYOUT_TILED = 1
LAYOUT_STAGED = 2          # weight codes in K-stage tiles, scales tiled
_LAYOUTS = {"canonical": LAYOUT_CANONICAL, "tiled": LAYOUT_TILED, "staged": LAYOUT_STAGED}

STATUS_NAMES = {0: "OK", 1: "INVALID_ARG", 2: "UNSUPPORTED_SHAPE", 3: "CUDA", 4: "TIMEOUT", 5: "WORKSPACE",
                6: "DEVICE"}


class Nvfp4Error(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -m nvfp4_w4a4_quantized_moe_b200.build` "
                      "(the layer has no other implementation)")

lib = ctypes.CDLL(LIB_PATH)

_vp, _i, _f, _sz, _ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_longlong


class MoeWeightsStruct(ctypes.Structure):
    _fields_ = [("E", _i), ("H", _i), ("I", _i), ("k", _i), ("routed_scaling_factor", _f),
                ("router_weight", _vp), ("bias", _vp),
                ("gate_codes", _vp), ("gate_scales", _vp), ("gate_gscale", _vp),
                ("up_codes", _vp), ("up_scales", _vp), ("up_gscale", _vp),
                ("down_codes", _vp), ("down_scales", _vp), ("down_gscale", _vp),
                ("shared_gate", _vp), ("shared_up", _vp), ("shared_down", _vp), ("I_shared", _i),
                ("codes_layout", _i)]


DEBUG_FIELDS = ("logits", "topk_idx", "topk_w", "expert_offsets", "perm", "inv_perm", "a_codes", "a_scales", "h",
                "h_amax", "h_codes", "h_scales", "y")
N_STAGE_EVENTS = 6


class MoeDebugStruct(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in DEBUG_FIELDS] + [("stage_events", _vp * N_STAGE_EVENTS)] +
                [("saliency_sum", _vp), ("saliency_count", _vp), ("shared_event", _vp)])


def _declare(name, restype, *argtypes):
    fn = getattr(lib, name)
    fn.restype = restype
    fn.argtypes = list(argtypes)
    return fn


_declare("nvfp4_last_error", ctypes.c_char_p)
_declare("nvfp4_abi_version", _i)
_declare("nvfp4_workspace_status", _i, _vp, _vp)
_declare("nvfp4_quantize_weights_workspace_size", _sz, _i)
_declare("nvfp4_quantize_weights", _i, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _sz, _vp)
_declare("nvfp4_quantize_weights_noalloc", _i, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp)
_declare("nvfp4_quantize_weights_noalloc_status", _i, _vp)
_declare("nvfp4_quantize_act", _i, _vp, _i, _i, _vp, _i, _vp, _vp, _vp)
_declare("moe_route_rows_capacity", _i, _i, _i, _i)
_declare("moe_route_workspace_size", _sz, _i, _i, _i)
_declare("moe_route", _i, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz,
         _vp)
_declare("moe_nvfp4_workspace_size", _sz, _i, _i, _i, _i, _i)
_declare("moe_nvfp4_workspace_size_shared", _sz, _i, _i, _i, _i, _i, _i)
_declare("moe_nvfp4_forward_launches", _i, _i, _i, _i, _i, _i, _i, _i)
_declare("moe_nvfp4_forward", _i, ctypes.POINTER(MoeWeightsStruct), _vp, _i, _vp, _vp, _vp, _vp,
         ctypes.POINTER(MoeDebugStruct), _vp, _sz, _vp)
_declare("moe_nvfp4_forward_scaled", _i, ctypes.POINTER(MoeWeightsStruct), _vp, _i, _i, _vp, _vp, _vp, _vp,
         ctypes.POINTER(MoeDebugStruct), _vp, _sz, _vp)
_declare("moe_nvfp4_workspace_size_host", _sz, _i, _i, _i, _i, _i, _i)
_declare("moe_nvfp4_forward_host", _i, ctypes.POINTER(MoeWeightsStruct), _vp, _i, _vp, _vp, _vp, _vp, _vp, _sz, _vp)
_declare("moe_nvfp4_host_join", _i, _vp, _vp)
_declare("moe_nvfp4_host_release", _i, _vp)
_declare("moe_nvfp4_gemm_workspace_size", _sz, _i)
_declare("moe_reap_keep", _i, _vp, _vp, _i, _i, _vp, _vp)
_declare("moe_nvfp4_gate_up", _i, ctypes.POINTER(MoeWeightsStruct), _vp, _vp, _vp, _vp, _i, _vp, _vp, _vp, _vp,
         _vp, _vp, _vp, _sz, _vp)
_declare("moe_nvfp4_down", _i, ctypes.POINTER(MoeWeightsStruct), _vp, _vp, _vp, _vp, _i, _vp, _vp, _vp, _vp,
         _vp, _sz, _vp)

_declare("nvfp4_block_stats_compute", _i, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _vp, _vp)
_declare("mxfp4_scale_bytes", _sz, _i, _i, _i)
_declare("mxfp4_quantize", _i, _vp, _i, _i, _i, _ll, _vp, _i, _i, _vp, _vp, _vp)
_declare("mxfp4_quantize_transposed", _i, _vp, _i, _i, _i, _ll, _i, _vp, _vp, _vp)
_declare("mxfp4_dequantize", _i, _vp, _vp, _i, _i, _i, _i, _vp, _ll, _vp)
_declare("mxfp4_matmul_workspace_size", _sz)
_declare("mxfp4_matmul", _i, _vp, _vp, _i, _vp, _vp, _i, _i, _i, _vp, _vp, _vp, _vp, _i, _vp, _ll, _vp, _sz, _vp)
_declare("mxfp4_linear_workspace_size", _sz, _i, _i)
_declare("mxfp4_linear", _i, _vp, _i, _i, _ll, _vp, _i, _vp, _vp, _i, _i, _i, _vp, _vp, _vp, _vp, _i, _vp, _ll, _vp,
         _sz, _vp)
_declare("moe_balance_loss_workspace_size", _sz, _i, _i, _i)
_declare("moe_balance_loss", _i, _vp, _i, _i, _i, _ll, _vp, _i, _i, _vp, _vp, _i, _f, _vp, _vp, _vp, _vp, _vp, _sz,
         _vp)
_declare("moe_balance_loss_backward", _i, _vp, _i, _i, _i, _ll, _i, _i, _vp, _vp, _i, _f, _vp, _vp, _vp, _vp, _ll,
         _vp)
_declare("nvfp4_test_e2m1", _i, _vp, _i, _vp, _vp, _vp)
_declare("nvfp4_test_e2m1_sweep", _i, ctypes.c_uint32, ctypes.c_uint64, _vp, _vp, _vp)
_declare("nvfp4_test_e4m3", _i, _vp, _i, _vp, _vp, _vp)
_declare("nvfp4_test_sigmoid", _i, _vp, _i, _vp, _vp)
_declare("nvfp4_test_mma_peak", _i, _i, _i, _i, _i, _vp, _vp, _vp)
_declare("nvfp4_test_wait_timeout", _i, _vp, ctypes.c_uint64, _vp, _sz, _vp, _vp, _vp)
_declare("nvfp4_test_block_scale_div", _i, _vp, _vp, _i, _vp, _vp, _vp, _vp, _vp)
_declare("nvfp4_test_router_splits", _i, _i, _i, ctypes.POINTER(ctypes.c_int))
_declare("nvfp4_test_mxfp4_plan", _i, _i, _i, _i, _i, ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int),
         ctypes.POINTER(ctypes.c_int))
_declare("nvfp4_test_mxfp4_residency", _i, _i, _i, _i, _i, ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int))
_declare("nvfp4_test_mxfp4_segments", _i, _vp, _vp, _i, _i, _vp, _vp)
_declare("nvfp4_test_mxfp4_fuses", _i, _i, _i, _i, _i, _i, ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int))

# Every symbol the public headers declare (checked by the CPU test suite).
EXPORTS = ("nvfp4_last_error", "nvfp4_abi_version", "nvfp4_workspace_status",
           "nvfp4_quantize_weights_workspace_size", "nvfp4_quantize_weights", "nvfp4_quantize_weights_noalloc",
           "nvfp4_quantize_weights_noalloc_status", "nvfp4_quantize_act",
           "moe_route_rows_capacity", "moe_route_workspace_size", "moe_route", "moe_nvfp4_workspace_size",
           "moe_nvfp4_forward", "moe_nvfp4_forward_scaled", "moe_nvfp4_workspace_size_shared",
           "moe_nvfp4_forward_launches", "moe_nvfp4_workspace_size_host", "moe_nvfp4_forward_host",
           "moe_nvfp4_host_join", "moe_nvfp4_host_release",
           "moe_nvfp4_gemm_workspace_size", "moe_nvfp4_gate_up",
           "moe_nvfp4_down", "moe_reap_keep",
           "nvfp4_block_stats_compute",
           "mxfp4_scale_bytes", "mxfp4_quantize", "mxfp4_quantize_transposed", "mxfp4_dequantize",
           "mxfp4_matmul_workspace_size", "mxfp4_matmul", "mxfp4_linear_workspace_size", "mxfp4_linear",
           "moe_balance_loss_workspace_size", "moe_balance_loss", "moe_balance_loss_backward",
           "nvfp4_test_e2m1", "nvfp4_test_e2m1_sweep", "nvfp4_test_e4m3", "nvfp4_test_sigmoid",
           "nvfp4_test_mma_peak", "nvfp4_test_wait_timeout", "nvfp4_test_block_scale_div",
           "nvfp4_test_router_splits", "nvfp4_test_mxfp4_plan", "nvfp4_test_mxfp4_segments",
           "nvfp4_test_mxfp4_residency", "nvfp4_test_mxfp4_fuses")


def _check(status: int):
    if status != 0:
        raise Nvfp4Error(status, lib.nvfp4_last_error().decode(errors="replace"))


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _cuda(t, dtype, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def tiled_scale_bytes(rows: int, cols: int) -> int:
    return (rows + 127) // 128 * 128 * (cols // 16)


def abi_version() -> int:
    return lib.nvfp4_abi_version()


def nvfp4_workspace_status(ws: torch.Tensor):
    """Raises Nvfp4Error(TIMEOUT) if a device-side wait of the call that used
    ``ws`` gave up; synchronises the current stream."""
    _check(lib.nvfp4_workspace_status(_p(ws), _stream()))


def moe_route_rows_capacity(T: int, E: int, k: int) -> int:
    return lib.moe_route_rows_capacity(T, E, k)


# ---------------------------------------------------------------------------
# quantisers
# ---------------------------------------------------------------------------

def _weight_outputs(w: torch.Tensor, lay: int, out):
    """(codes, scales, gscale) for n_mats [rows, cols] matrices: allocated
    with torch, or the caller's ``out``, checked for device, dtype and size."""
    n, rows, cols = w.shape
    need_scales = tiled_scale_bytes(n * rows, cols) if lay != LAYOUT_CANONICAL else n * rows * (cols // 16)
    if out is None:
        codes = torch.empty((n, rows, cols // 2), dtype=torch.uint8, device=w.device)
        scales = (torch.empty(need_scales, dtype=torch.uint8, device=w.device) if lay != LAYOUT_CANONICAL
                  else torch.empty((n, rows, cols // 16), dtype=torch.uint8, device=w.device))
        return codes, scales, torch.empty(n, dtype=torch.float32, device=w.device)
    codes, scales, gscale = out
    _cuda(codes, torch.uint8, "codes")
    _cuda(scales, torch.uint8, "scales")
    _cuda(gscale, torch.float32, "gscale")
    for t, name, need in ((codes, "codes", n * rows * (cols // 2)), (scales, "scales", need_scales),
                          (gscale, "gscale", n)):
        if t.device != w.device:
            raise ValueError(f"{name} must be on {w.device}, got {t.device}")
        if t.numel() < need:
            raise ValueError(f"{name} holds {t.numel()} elements; this call writes {need}")
    return codes, scales, gscale


def nvfp4_quantize_weights(w: torch.Tensor, layout: str = "tiled", workspace: torch.Tensor | None = None,
                           out=None):
    """w [n_mats, rows, cols] bf16 -> (codes [n, rows, cols/2] u8, scales u8, gscale [n] f32).
    ``out`` = (codes, scales, gscale) to write into instead of new tensors."""
    _cuda(w, torch.bfloat16, "w")
    if w.dim() == 2:
        w = w.unsqueeze(0)
    n, rows, cols = w.shape
    lay = _LAYOUTS[layout]
    codes, scales, gscale = _weight_outputs(w, lay, out)
    need = lib.nvfp4_quantize_weights_workspace_size(n)
    ws = workspace if workspace is not None else _workspace(need, w.device)
    _check(lib.nvfp4_quantize_weights(_p(w), n, rows, cols, lay, _p(codes), _p(scales), _p(gscale), _p(ws),
                                      ws.numel(), _stream()))
    return codes, scales, gscale


def nvfp4_quantize_weights_noalloc(w: torch.Tensor, layout: str = "tiled", out=None):
    """The weight quantiser without a workspace (its scratch is built into the
    library).  ``out`` = (codes, scales, gscale) to write into; allocated here
    with torch when None (the library itself allocates nothing)."""
    _cuda(w, torch.bfloat16, "w")
    if w.dim() == 2:
        w = w.unsqueeze(0)
    n, rows, cols = w.shape
    lay = _LAYOUTS[layout]
    codes, scales, gscale = _weight_outputs(w, lay, out)
    _check(lib.nvfp4_quantize_weights_noalloc(_p(w), n, rows, cols, lay, _p(codes), _p(scales), _p(gscale),
                                              _stream()))
    return codes, scales, gscale


def nvfp4_quantize_weights_noalloc_status():
    """Raises Nvfp4Error(TIMEOUT) if a device-side wait of the last
    nvfp4_quantize_weights_noalloc call on this device gave up; synchronises
    the current stream."""
    _check(lib.nvfp4_quantize_weights_noalloc_status(_stream()))


def nvfp4_quantize_act(x: torch.Tensor, gscale: torch.Tensor, layout: str = "canonical"):
    """x [rows, cols] bf16 under gscale (one f32 on the device) -> (codes, scales)."""
    _cuda(x, torch.bfloat16, "x")
    _cuda(gscale, torch.float32, "gscale")
    rows, cols = x.shape
    lay = _LAYOUTS[layout]
    codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=x.device)
    if lay == LAYOUT_TILED:
        scales = torch.empty(tiled_scale_bytes(rows, cols), dtype=torch.uint8, device=x.device)
    else:
        scales = torch.empty((rows, cols // 16), dtype=torch.uint8, device=x.device)
    _check(lib.nvfp4_quantize_act(_p(x), rows, cols, _p(gscale), lay, _p(codes), _p(scales), _stream()))
    return codes, scales


#: Fields of nvfp4_block_stats, in declaration order (9 uint64 counts, 6 fp64 sums).
BLOCK_STATS_FIELDS = ("elements", "outliers", "blocks", "outlier_blocks", "zero_scale_blocks",
                      "subnormal_scale_blocks", "saturated_elements", "neighbours", "clean", "sum_sq", "sse",
                      "sum_sq_neighbours", "sse_neighbours", "sum_sq_clean", "sse_clean")


def nvfp4_block_stats_compute(w: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, gscale: torch.Tensor,
                              layout: str = "tiled", threshold: float = 0.1, stats: torch.Tensor | None = None):
    """Block-scale distortion statistics of n_mats NVFP4 tensors.  Returns the
    device buffer ([n_mats, 15] int64 words: 9 counts, then 6 fp64 sums bit-cast);
    ``block_stats_to_dicts`` turns it into one dict per matrix."""
    _cuda(w, torch.bfloat16, "w")
    if w.dim() == 2:
        w = w.unsqueeze(0)
    n, rows, cols = w.shape
    _cuda(gscale, torch.float32, "gscale")
    if stats is None:
        stats = torch.empty((n, len(BLOCK_STATS_FIELDS)), dtype=torch.int64, device=w.device)
    _check(lib.nvfp4_block_stats_compute(_p(w), _p(codes), _p(scales), _p(gscale), n, rows, cols,
                                         _LAYOUTS[layout], float(threshold), _p(stats), _stream()))
    return stats


def block_stats_to_dicts(stats: torch.Tensor) -> list[dict]:
    h = stats.cpu()
    counts = h[:, :9].tolist()
    sums = h[:, 9:].contiguous().view(torch.float64).tolist()
    return [dict(zip(BLOCK_STATS_FIELDS, c + s)) for c, s in zip(counts, sums)]


# ---------------------------------------------------------------------------
# router
# ---------------------------------------------------------------------------

def moe_route(x, router_weight, bias, k: int, rsf: float, logit_offset=None, logits_in=None):
    """Router + permutation.  Pass either (x, router_weight) or logits_in."""
    _cuda(bias, torch.float32, "bias")
    E = bias.numel()
    if logits_in is not None:
        _cuda(logits_in, torch.float32, "logits_in")
        T, H = logits_in.shape[0], 64
        dev = logits_in.device
    else:
        _cuda(x, torch.bfloat16, "x")
        _cuda(router_weight, torch.bfloat16, "router_weight")
        T, H = x.shape
        dev = x.device
        if logit_offset is not None:
            _cuda(logit_offset, torch.float32, "logit_offset")
    cap = moe_route_rows_capacity(T, E, k)
    out = {
        "logits": torch.empty((T, E), dtype=torch.float32, device=dev),
        "topk_idx": torch.empty((T, k), dtype=torch.int32, device=dev),
        "topk_w": torch.empty((T, k), dtype=torch.float32, device=dev),
        "expert_offsets": torch.empty(E + 1, dtype=torch.int32, device=dev),
        "perm": torch.empty(cap, dtype=torch.int32, device=dev),
        "inv_perm": torch.empty((T, k), dtype=torch.int32, device=dev),
    }
    ws = _workspace(lib.moe_route_workspace_size(T, E, k), dev)
    _check(lib.moe_route(_p(x) if logits_in is None else None, _p(router_weight) if logits_in is None else None,
                         _p(logits_in), _p(bias), _p(logit_offset) if logits_in is None else None, T, H, E, k,
                         float(rsf), _p(out["logits"]), _p(out["topk_idx"]), _p(out["topk_w"]),
                         _p(out["expert_offsets"]), _p(out["perm"]), _p(out["inv_perm"]), _p(ws), ws.numel(),
                         _stream()))
    out["workspace"] = ws
    return out


# ---------------------------------------------------------------------------
# the layer
# ---------------------------------------------------------------------------

@dataclass
class MoeWeights:
    """Device tensors of one NVFP4 MoE layer (scales in the tiled layout; codes
    row-major or, with ``codes_layout`` = LAYOUT_STAGED, in K-stage tiles)."""
    E: int
    H: int
    I: int
    k: int
    rsf: float
    router_weight: torch.Tensor      # bf16 [E, H]
    bias: torch.Tensor               # f32 [E]
    gate_codes: torch.Tensor         # u8 [E, I, H/2]
    gate_scales: torch.Tensor
    gate_gscale: torch.Tensor        # f32 [E]
    up_codes: torch.Tensor
    up_scales: torch.Tensor
    up_gscale: torch.Tensor
    down_codes: torch.Tensor         # u8 [E, H, I/2]
    down_scales: torch.Tensor
    down_gscale: torch.Tensor
    # the shared expert, bf16 (None: none): gate, up [I_s, H], down [H, I_s]
    shared_gate: torch.Tensor | None = None
    shared_up: torch.Tensor | None = None
    shared_down: torch.Tensor | None = None
    codes_layout: int = LAYOUT_CANONICAL

    @property
    def I_shared(self) -> int:
        return 0 if self.shared_gate is None else int(self.shared_gate.shape[0])

    def with_shared(self, gate: torch.Tensor, up: torch.Tensor, down: torch.Tensor) -> "MoeWeights":
        """This layer plus a shared bf16 expert."""
        for n, t in (("shared gate", gate), ("shared up", up), ("shared down", down)):
            _cuda(t, torch.bfloat16, n)
        return dataclasses.replace(self, shared_gate=gate, shared_up=up, shared_down=down)

    def struct(self) -> MoeWeightsStruct:
        return MoeWeightsStruct(self.E, self.H, self.I, self.k, float(self.rsf), _p(self.router_weight),
                                _p(self.bias), _p(self.gate_codes), _p(self.gate_scales), _p(self.gate_gscale),
                                _p(self.up_codes), _p(self.up_scales), _p(self.up_gscale), _p(self.down_codes),
                                _p(self.down_scales), _p(self.down_gscale), _p(self.shared_gate),
                                _p(self.shared_up), _p(self.shared_down), self.I_shared, int(self.codes_layout))

    @classmethod
    def quantize(cls, gate, up, down, router_weight, bias, k: int, rsf: float,
                 codes_layout: str | None = None) -> "MoeWeights":
        """RTN-quantise bf16 expert weights (gate/up [E, I, H], down [E, H, I])
        with the library's weight quantiser, tiled scales.  The codes are
        staged when H and I are multiples of 256 (``codes_layout`` None), else
        row-major; "staged" or "canonical" forces one."""
        E, I, H = gate.shape
        if codes_layout is None:
            codes_layout = "staged" if H % 256 == 0 and I % 256 == 0 else "canonical"
        lay = "staged" if codes_layout == "staged" else "tiled"
        gc, gs, gg = nvfp4_quantize_weights(gate, lay)
        uc, us, ug = nvfp4_quantize_weights(up, lay)
        dc, ds, dg = nvfp4_quantize_weights(down, lay)
        return cls(E, H, I, k, rsf, _cuda(router_weight, torch.bfloat16, "router_weight"),
                   _cuda(bias, torch.float32, "bias"), gc, gs, gg, uc, us, ug, dc, ds, dg,
                   codes_layout=LAYOUT_STAGED if lay == "staged" else LAYOUT_CANONICAL)


def reap_keep(saliency_sum: torch.Tensor, saliency_count: torch.Tensor, keep: int) -> torch.Tensor:
    """Experts retained by REAP pruning (moe_reap_keep): the ``keep`` highest
    mean saliencies, ties to the lower index, in expert order.  Returns their
    indices as int64 on the host."""
    _cuda(saliency_sum, torch.float64, "saliency sum")
    _cuda(saliency_count, torch.int64, "saliency count")
    E = saliency_sum.numel()
    if saliency_count.numel() != E:
        raise ValueError("saliency sum and count must have one entry per expert")
    idx = torch.empty(max(int(keep), 1), dtype=torch.int32, device=saliency_sum.device)
    _check(lib.moe_reap_keep(_p(saliency_sum), _p(saliency_count), E, int(keep), _p(idx), _stream()))
    return idx[:keep].cpu().long()


def select_experts(W: "MoeWeights", keep: torch.Tensor) -> "MoeWeights":
    """The layer restricted to the experts ``keep`` (in that order), by byte
    slicing only (no arithmetic): gate.weight
    rows and e_score_correction_bias sliced as the pruned checkpoint does, and
    each retained expert's codes, tiled scales and global scales copied over
    (an expert's I or H rows are whole 128-row tiles, so its scales and its
    codes, row-major or staged, are contiguous ranges)."""
    idx = keep.to(W.router_weight.device)
    E2 = int(idx.numel())

    def rows(t, per):
        return t.reshape(W.E, per).index_select(0, idx).reshape(-1).contiguous()

    def codes(t):
        return t.reshape(W.E, -1).index_select(0, idx).reshape(E2, *t.shape[1:]).contiguous()

    return MoeWeights(E2, W.H, W.I, W.k, W.rsf, W.router_weight.index_select(0, idx).contiguous(),
                      W.bias.index_select(0, idx).contiguous(),
                      codes(W.gate_codes), rows(W.gate_scales, W.I * W.H // 16), W.gate_gscale.index_select(0, idx),
                      codes(W.up_codes), rows(W.up_scales, W.I * W.H // 16), W.up_gscale.index_select(0, idx),
                      codes(W.down_codes), rows(W.down_scales, W.H * W.I // 16), W.down_gscale.index_select(0, idx),
                      W.shared_gate, W.shared_up, W.shared_down, W.codes_layout)


def moe_nvfp4_forward_launches(T: int, E: int, H: int, I: int, k: int, I_shared: int = 0,
                               act_scale_mode: str = "tensor") -> int:
    """Kernels one forward call queues for this shape (host arithmetic only)."""
    n = lib.moe_nvfp4_forward_launches(T, E, H, I, k, I_shared, ACT_SCALE_MODES[act_scale_mode])
    if n < 0:
        raise ValueError(f"unsupported forward shape T={T} E={E} H={H} I={I} k={k} I_shared={I_shared}")
    return n


def moe_nvfp4_workspace_size(T: int, E: int, H: int, I: int, k: int, I_shared: int = 0) -> int:
    return lib.moe_nvfp4_workspace_size_shared(T, E, H, I, k, I_shared)


#: Activation global-scale modes of moe_nvfp4_forward_scaled (NVFP4_ACT_SCALE_*).
ACT_SCALE_MODES = {"tensor": 0, "expert": 1, "dynamic": 2, "dynamic_expert": 3}


def moe_nvfp4_forward(W: MoeWeights, x: torch.Tensor, act_gscale: torch.Tensor, h_gscale: torch.Tensor,
                      logit_offset: torch.Tensor | None = None, debug: bool = False,
                      out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                      stage_events=None, act_scale_mode: str = "tensor", saliency=None, shared_event=None):
    """out [T, H] bf16; with debug=True also a dict of intermediate results.
    ``act_scale_mode`` is one of ACT_SCALE_MODES: in "tensor" act_gscale and
    h_gscale hold one fp32 each, in "expert" E each; in "dynamic" and
    "dynamic_expert" the library writes g1 into act_gscale ([1] or [E]).
    ``stage_events``: optional list of 6 torch.cuda.Event(enable_timing=True),
    each already recorded once (torch creates the CUDA event lazily), which
    the library records again between the stages of the layer.
    ``saliency``: optional (sum float64 [E], count int64 [E]) REAP saliency
    accumulators on the device that the call adds this batch to.
    ``shared_event``: optional torch.cuda.Event (recorded once already) that
    the library records after the shared expert's GEMMs."""
    mode = ACT_SCALE_MODES[act_scale_mode]
    if saliency is not None:
        _cuda(saliency[0], torch.float64, "saliency sum")
        _cuda(saliency[1], torch.int64, "saliency count")
    _cuda(x, torch.bfloat16, "x")
    _cuda(act_gscale, torch.float32, "act_gscale")
    _cuda(h_gscale, torch.float32, "h_gscale")
    n_scales = W.E if mode & 1 else 1
    if act_gscale.numel() != n_scales or h_gscale.numel() != n_scales:
        raise ValueError(f"act_scale_mode {act_scale_mode!r} needs {n_scales} value(s) in act_gscale and h_gscale")
    T, H = x.shape
    dev = x.device
    out = torch.empty((T, H), dtype=torch.bfloat16, device=dev) if out is None else _cuda(out, torch.bfloat16, "out")
    if workspace is None:
        workspace = _workspace(moe_nvfp4_workspace_size(T, W.E, W.H, W.I, W.k, W.I_shared), dev)
    dbg_tensors = None
    dbg_ptr = None
    if debug:
        cap = moe_route_rows_capacity(T, W.E, W.k)
        z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device=dev)  # noqa: E731
        dbg_tensors = {
            "logits": z(T, W.E), "topk_idx": z(T, W.k, dt=torch.int32), "topk_w": z(T, W.k),
            "expert_offsets": z(W.E + 1, dt=torch.int32), "perm": z(cap, dt=torch.int32),
            "inv_perm": z(T, W.k, dt=torch.int32), "a_codes": z(cap, W.H // 2, dt=torch.uint8),
            "a_scales": z(tiled_scale_bytes(cap, W.H), dt=torch.uint8), "h": z(cap, W.I), "h_amax": z(n_scales),
            "h_codes": z(cap, W.I // 2, dt=torch.uint8), "h_scales": z(tiled_scale_bytes(cap, W.I), dt=torch.uint8),
            "y": z(cap, W.H),
        }
    if debug or stage_events is not None or saliency is not None or shared_event is not None:
        dbg = MoeDebugStruct()
        if saliency is not None:
            dbg.saliency_sum = saliency[0].data_ptr()
            dbg.saliency_count = saliency[1].data_ptr()
        if debug:
            for n in DEBUG_FIELDS:
                setattr(dbg, n, dbg_tensors[n].data_ptr())
        if stage_events is not None:
            for i, ev in enumerate(stage_events):
                if not ev.cuda_event:
                    raise ValueError("stage_events must have been recorded once (so that the CUDA event exists)")
                dbg.stage_events[i] = ev.cuda_event
        if shared_event is not None:
            if not shared_event.cuda_event:
                raise ValueError("shared_event must have been recorded once (so that the CUDA event exists)")
            dbg.shared_event = shared_event.cuda_event
        dbg_ptr = ctypes.pointer(dbg)
    ws_struct = W.struct()
    if mode == 0:
        _check(lib.moe_nvfp4_forward(ctypes.byref(ws_struct), _p(x), T, _p(act_gscale), _p(h_gscale),
                                     _p(logit_offset), _p(out), dbg_ptr, _p(workspace), workspace.numel(), _stream()))
    else:
        _check(lib.moe_nvfp4_forward_scaled(ctypes.byref(ws_struct), _p(x), T, mode, _p(act_gscale), _p(h_gscale),
                                            _p(logit_offset), _p(out), dbg_ptr, _p(workspace), workspace.numel(),
                                            _stream()))
    if debug:
        dbg_tensors["workspace"] = workspace
        return out, dbg_tensors
    return out


def moe_nvfp4_workspace_size_host(T: int, E: int, H: int, I: int, k: int, I_shared: int = 0) -> int:
    return lib.moe_nvfp4_workspace_size_host(T, E, H, I, k, I_shared)


def _host(t, dtype, name):
    if not isinstance(t, torch.Tensor) or t.is_cuda:
        raise ValueError(f"{name} must be a host (CPU) tensor")
    if t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor")
    return t


def moe_nvfp4_forward_host(W: MoeWeights, x_host: torch.Tensor, act_gscale: torch.Tensor, h_gscale: torch.Tensor,
                           out_host: torch.Tensor, workspace: torch.Tensor, logit_offset: torch.Tensor | None = None):
    """The forward on host buffers (per-tensor scales): enqueues x in, the
    layer on the current stream and out back, and returns without waiting.
    x_host and out_host are [T, H] bf16 CPU tensors (pinned for the copies to
    overlap); the workspace is a CUDA uint8 tensor of at least
    moe_nvfp4_workspace_size_host bytes.  out_host is complete after
    moe_nvfp4_host_join(workspace) and a synchronize of the current stream."""
    _host(x_host, torch.bfloat16, "x_host")
    _host(out_host, torch.bfloat16, "out_host")
    _cuda(act_gscale, torch.float32, "act_gscale")
    _cuda(h_gscale, torch.float32, "h_gscale")
    _cuda(workspace, torch.uint8, "workspace")
    T, H = x_host.shape
    if tuple(out_host.shape) != (T, H):
        raise ValueError("out_host must have the shape of x_host")
    ws_struct = W.struct()
    _check(lib.moe_nvfp4_forward_host(ctypes.byref(ws_struct), ctypes.c_void_p(x_host.data_ptr()), T,
                                      _p(act_gscale), _p(h_gscale), _p(logit_offset),
                                      ctypes.c_void_p(out_host.data_ptr()), _p(workspace), workspace.numel(),
                                      _stream()))
    return out_host


def moe_nvfp4_host_join(workspace: torch.Tensor):
    """Makes the current stream wait for the last host-buffer call on this
    workspace to have copied its out back."""
    _check(lib.moe_nvfp4_host_join(_p(workspace), _stream()))


def moe_nvfp4_host_release(workspace: torch.Tensor):
    """Waits for the workspace's last host-buffer call and frees the
    library's events for it."""
    _check(lib.moe_nvfp4_host_release(_p(workspace)))


def moe_nvfp4_gate_up(W: MoeWeights, a_codes, a_scales, expert_offsets, expert_counts, act_gscale, h_gscale,
                      want_h: bool = True, want_amax: bool = False):
    """Grouped gate/up GEMM on caller-supplied quantised rows."""
    rows = a_codes.shape[0]
    dev = a_codes.device
    h_codes = torch.empty((rows, W.I // 2), dtype=torch.uint8, device=dev)
    h_scales = torch.empty(tiled_scale_bytes(rows, W.I), dtype=torch.uint8, device=dev)
    h = torch.empty((rows, W.I), dtype=torch.float32, device=dev) if want_h else None
    amax = torch.zeros(1, dtype=torch.float32, device=dev) if want_amax else None
    ws = _workspace(lib.moe_nvfp4_gemm_workspace_size(rows), dev)
    st = W.struct()
    _check(lib.moe_nvfp4_gate_up(ctypes.byref(st), _p(a_codes), _p(a_scales), _p(expert_offsets), _p(expert_counts),
                                 rows, _p(act_gscale), _p(h_gscale), _p(h_codes), _p(h_scales), _p(h), _p(amax),
                                 _p(ws), ws.numel(), _stream()))
    return {"h_codes": h_codes, "h_scales": h_scales, "h": h, "h_amax": amax, "workspace": ws}


def moe_nvfp4_down(W: MoeWeights, h_codes, h_scales, expert_offsets, expert_counts, h_gscale, row_weight=None,
                   out_dtype=torch.float32):
    """Grouped down GEMM on caller-supplied quantised rows; y [rows, H]."""
    rows = h_codes.shape[0]
    dev = h_codes.device
    y = torch.zeros((rows, W.H), dtype=out_dtype, device=dev)
    ws = _workspace(lib.moe_nvfp4_gemm_workspace_size(rows), dev)
    st = W.struct()
    yb = y if out_dtype == torch.bfloat16 else None
    yf = y if out_dtype == torch.float32 else None
    _check(lib.moe_nvfp4_down(ctypes.byref(st), _p(h_codes), _p(h_scales), _p(expert_offsets), _p(expert_counts),
                              rows, _p(h_gscale), _p(row_weight), _p(yb), _p(yf), _p(ws), ws.numel(), _stream()))
    return {"y": y, "workspace": ws}


# ---------------------------------------------------------------------------
# MXFP4 matrices (include/mxfp4.h)
# ---------------------------------------------------------------------------

#: Element types of unquantised matrices (MXFP4_DTYPE_*).
_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}

# A small call is bound by its host side (14 us for mxfp4_linear of one token,
# of which the GPU works 8), so the functions below read each property of a
# tensor once, take the current stream as the raw handle and give
# torch.empty its sizes one by one (a tuple costs 0.7 us more).
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _launch(dev: int, fn, *args):
    """fn(*args, stream) on device ``dev`` and its current stream."""
    if _current_device() == dev:
        status = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(dev))
    if status:
        _check(status)


def _same_device(dev: int, *tensors):
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"all tensors of a call must be on one device: got {t.device} and cuda:{dev}")


_INT_MAX = 2 ** 31 - 1


def _int32(n: int, name: str) -> int:
    """n, if the library's int holds it (ctypes would pass its low 32 bits)."""
    if n > _INT_MAX:
        raise ValueError(f"{name} is {n}; the library takes sizes below 2^31")
    return n


def _matrix(t, name: str, dtypes=_DTYPES):
    """(rows, cols, row stride) of a CUDA matrix whose rows are contiguous."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be one of {', '.join(map(str, dtypes))}, got {t.dtype}")
    shape, strides = t.shape, t.stride()
    if len(shape) != 2 or shape[1] < 1:
        raise ValueError(f"{name} must be a matrix with at least one column, got shape {tuple(shape)}")
    rows, cols = shape
    if rows > _INT_MAX or cols > _INT_MAX:
        raise ValueError(f"{name} is {rows} x {cols}; the library takes sizes below 2^31")
    if cols > 1 and strides[1] != 1:
        raise ValueError(f"{name} must have contiguous rows (stride {strides})")
    if rows > 1 and strides[0] < cols:
        raise ValueError(f"{name} must not have overlapping rows (stride {strides})")
    return rows, cols, strides[0]


def _vector(t, dtype, name: str, n: int):
    _cuda(t, dtype, name)
    if t.numel() != n:
        raise ValueError(f"{name} must hold {n} values, got {t.numel()}")
    return t


def _ptr(t):
    return None if t is None else t.data_ptr()


def _mx_sizes(rows: int, cols: int, layout: str):
    """Bytes of (a row's codes, the scales) of an MXFP4 matrix."""
    blocks = (cols + 31) // 32
    if layout == "canonical":
        return blocks * 16, rows * blocks
    if layout == "tiled":
        return blocks * 16, (rows + 127) // 128 * ((blocks + 3) // 4) * 512
    raise ValueError(f"MXFP4 layout must be 'tiled' or 'canonical', got {layout!r}")


@dataclass
class Mxfp4:
    """A rows x cols matrix in MXFP4: packed codes [rows, 16 ceil(cols / 32)]
    (u8) and E8M0 scales (u8), "tiled" (what the products take) or
    "canonical" ([rows, ceil(cols / 32)])."""
    codes: torch.Tensor
    scales: torch.Tensor
    rows: int
    cols: int
    layout: str = "tiled"

    def __post_init__(self):
        _cuda(self.codes, torch.uint8, "codes")
        _cuda(self.scales, torch.uint8, "scales")
        if self.rows < 0 or self.cols < 1:
            raise ValueError(f"no MXFP4 matrix has shape {self.rows} x {self.cols}")
        _int32(max(self.rows, self.cols), "the matrix's larger side")
        row_bytes, scale_bytes = _mx_sizes(self.rows, self.cols, self.layout)
        if self.codes.numel() < self.rows * row_bytes:
            raise ValueError(f"codes hold {self.codes.numel()} bytes; a {self.rows} x {self.cols} matrix has "
                             f"{self.rows * row_bytes}")
        if self.scales.numel() < scale_bytes:
            raise ValueError(f"scales hold {self.scales.numel()} bytes; a {self.rows} x {self.cols} matrix has "
                             f"{scale_bytes} ({self.layout})")
        _same_device(self.codes.get_device(), self.scales)


def _mx_out(out, rows: int, cols: int, layout: str, device) -> Mxfp4:
    """The matrix a quantiser writes: ``out``, or a new one."""
    row_bytes, scale_bytes = _mx_sizes(rows, cols, layout)
    if out is not None:
        if (out.rows, out.cols, out.layout) != (rows, cols, layout):
            raise ValueError(f"out is {out.rows} x {out.cols} ({out.layout}); "
                             f"this call writes {rows} x {cols} ({layout})")
        return out
    q = Mxfp4.__new__(Mxfp4)                       # sizes and devices are right by construction
    q.codes = torch.empty(rows, row_bytes, dtype=torch.uint8, device=device)
    q.scales = torch.empty(scale_bytes, dtype=torch.uint8, device=device)
    if layout == "canonical":
        q.scales = q.scales.view(rows, row_bytes // 16)
    q.rows, q.cols, q.layout = rows, cols, layout
    return q


def mxfp4_quantize(x: torch.Tensor, layout: str = "tiled", perm: torch.Tensor | None = None,
                   out: Mxfp4 | None = None) -> Mxfp4:
    """x [rows, cols] (bf16, fp16 or fp32, any row stride; or a stack
    [n, rows, cols], contiguous, as n * rows rows) -> MXFP4.  With ``perm``
    (int32) row r of the result is x[perm[r]], zeros where perm[r] names no
    row."""
    if isinstance(x, torch.Tensor) and x.dim() == 3:
        if not x.is_contiguous():
            raise ValueError("a stack of matrices must be contiguous")
        x = x.flatten(0, 1)
    rows, cols, stride = _matrix(x, "x")
    n = rows if perm is None else _int32(_cuda(perm, torch.int32, "perm").numel(), "perm's length")
    q = _mx_out(out, n, cols, layout, x.device)
    dev = x.get_device()
    _same_device(dev, perm, q.codes)
    if n:
        _launch(dev, lib.mxfp4_quantize, x.data_ptr(), _DTYPES[x.dtype], rows, cols, stride, _ptr(perm), n,
                _LAYOUTS[layout], q.codes.data_ptr(), q.scales.data_ptr())
    return q


def mxfp4_quantize_transposed(x: torch.Tensor, layout: str = "tiled", out: Mxfp4 | None = None) -> Mxfp4:
    """x [rows, cols] -> the MXFP4 matrix of its transpose (cols x rows, the
    blocks along x's columns): the operand of a product that sums over rows."""
    rows, cols, stride = _matrix(x, "x")
    if rows < 1:
        raise ValueError("x must have at least one row")
    q = _mx_out(out, cols, rows, layout, x.device)
    dev = x.get_device()
    _same_device(dev, q.codes)
    _launch(dev, lib.mxfp4_quantize_transposed, x.data_ptr(), _DTYPES[x.dtype], rows, cols, stride, _LAYOUTS[layout],
            q.codes.data_ptr(), q.scales.data_ptr())
    return q


def mxfp4_dequantize(q: Mxfp4, dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """The values of an MXFP4 matrix, [rows, cols] (exact in bf16 and fp32),
    in ``dtype``, or in ``out``'s."""
    codes = q.codes
    if out is None:
        out = torch.empty(q.rows, q.cols, dtype=dtype, device=codes.device)
    rows, cols, stride = _matrix(out, "out")
    if rows != q.rows or cols != q.cols:
        raise ValueError(f"out must be {q.rows} x {q.cols}, got {rows} x {cols}")
    dev = codes.get_device()
    _same_device(dev, out)
    if rows:
        _launch(dev, lib.mxfp4_dequantize, codes.data_ptr(), q.scales.data_ptr(), _LAYOUTS[q.layout], rows, cols,
                _DTYPES[out.dtype], out.data_ptr(), stride)
    return out


def _product_args(M: int, b: Mxfp4, out_dtype, out, bias, row_weight, expert_offsets, expert_counts):
    """Checks a product's tensors; returns (E, N, out, its row stride)."""
    if b.layout != "tiled":
        raise ValueError("a product takes tiled scales; quantise with layout='tiled'")
    E, N = 0, b.rows
    if expert_offsets is not None:
        E = _int32(_cuda(expert_offsets, torch.int32, "expert_offsets").numel() - 1, "the number of experts")
        if E < 1 or N % E:
            raise ValueError(f"expert_offsets of {E + 1} entries do not divide b's {N} rows into experts")
        N //= E
        if expert_counts is not None:
            _vector(expert_counts, torch.int32, "expert_counts", E)
    elif expert_counts is not None:
        raise ValueError("expert_counts go with expert_offsets")
    if N < 1:
        raise ValueError("b has no rows")
    if row_weight is not None:
        _vector(row_weight, torch.float32, "row_weight", M)
    if bias is not None:
        _vector(bias, torch.float32, "bias", b.rows)
    if out is None:
        if out_dtype not in _DTYPES:
            raise ValueError(f"out_dtype must be one of {', '.join(map(str, _DTYPES))}, got {out_dtype}")
        # grouped: the rows of no expert are not written
        out = (torch.zeros if E else torch.empty)(M, N, dtype=out_dtype, device=b.codes.device)
        return E, N, out, N
    rows, cols, stride = _matrix(out, "out")
    if rows != M or cols != N:
        raise ValueError(f"out must be {M} x {N}, got {rows} x {cols}")
    return E, N, out, stride


def mxfp4_matmul_workspace_size() -> int:
    return lib.mxfp4_matmul_workspace_size()


def mxfp4_matmul(a: Mxfp4, b: Mxfp4, out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
                 bias: torch.Tensor | None = None, row_weight: torch.Tensor | None = None,
                 expert_offsets: torch.Tensor | None = None, expert_counts: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None) -> torch.Tensor:
    """a (M x K) times the transpose of b (N x K): y[m] = row_weight[m] *
    (sum_k a[m, k] b[n, k] + bias[n]), [M, N].  With ``expert_offsets`` (int32
    [E + 1], multiples of 128 as moe_route gives them) b holds E matrices of
    N rows and rows [offsets[e], offsets[e] + counts[e]) meet matrix e; the
    other rows of ``out`` are left as they were (0 in a new one).
    ``expert_counts`` count every token that was routed: moe_balance_loss's
    counts are fewer where it left tokens out."""
    if a.layout != "tiled":
        raise ValueError("a product takes tiled scales; quantise with layout='tiled'")
    if a.cols != b.cols:
        raise ValueError(f"a has {a.cols} columns and b {b.cols}")
    E, N, out, stride = _product_args(a.rows, b, out_dtype, out, bias, row_weight, expert_offsets, expert_counts)
    if workspace is None:
        workspace = _workspace(256, a.codes.device)
    else:
        _cuda(workspace, torch.uint8, "workspace")
    dev = a.codes.get_device()
    _same_device(dev, b.codes, out, bias, row_weight, expert_offsets, expert_counts, workspace)
    _launch(dev, lib.mxfp4_matmul, a.codes.data_ptr(), a.scales.data_ptr(), a.rows, b.codes.data_ptr(),
            b.scales.data_ptr(), N, a.cols, E, _ptr(expert_offsets), _ptr(expert_counts), _ptr(row_weight),
            _ptr(bias), _DTYPES[out.dtype], out.data_ptr(), stride, workspace.data_ptr(), workspace.numel())
    return out


def mxfp4_linear_workspace_size(M: int, K: int) -> int:
    return lib.mxfp4_linear_workspace_size(_int32(M, "M"), _int32(K, "K"))


def mxfp4_linear(x: torch.Tensor, w: Mxfp4, out_dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
                 bias: torch.Tensor | None = None, row_weight: torch.Tensor | None = None,
                 perm: torch.Tensor | None = None, expert_offsets: torch.Tensor | None = None,
                 expert_counts: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """mxfp4_matmul with a = x (or, with ``perm``, its rows x[perm[r]])
    quantised in the call.  x is [rows, K], any row stride; the result has
    x's dtype unless ``out_dtype`` or ``out`` says otherwise."""
    rows, K, x_stride = _matrix(x, "x")
    if K != w.cols:
        raise ValueError(f"x has {K} columns and w {w.cols}")
    M = rows if perm is None else _int32(_cuda(perm, torch.int32, "perm").numel(), "perm's length")
    dtype = x.dtype
    E, N, out, stride = _product_args(M, w, out_dtype or dtype, out, bias, row_weight, expert_offsets, expert_counts)
    if workspace is None:
        workspace = _workspace(lib.mxfp4_linear_workspace_size(M, K), x.device)
    else:
        _cuda(workspace, torch.uint8, "workspace")
    dev = x.get_device()
    _same_device(dev, w.codes, out, bias, row_weight, perm, expert_offsets, expert_counts, workspace)
    if M:
        _launch(dev, lib.mxfp4_linear, x.data_ptr(), _DTYPES[dtype], rows, x_stride, _ptr(perm), M,
                w.codes.data_ptr(), w.scales.data_ptr(), N, K, E, _ptr(expert_offsets), _ptr(expert_counts),
                _ptr(row_weight), _ptr(bias), _DTYPES[out.dtype], out.data_ptr(), stride, workspace.data_ptr(),
                workspace.numel())
    return out


# ---------------------------------------------------------------------------
# the router's balance loss (include/moe_balance.h)
# ---------------------------------------------------------------------------

BALANCE_SCORES = {"sigmoid": 0, "softmax": 1}


@dataclass
class BalanceLoss:
    """Outputs of moe_balance_loss and what its backward needs of the call."""
    loss: torch.Tensor               # f32 [1]
    counts: torch.Tensor             # i32 [S, E] choices per expert
    tokens: torch.Tensor             # i32 [S + 1] tokens per sequence, then the sequences that have any
    probs: torch.Tensor              # f32 [S, E] mean shares
    k: int
    score: str
    coeff: float
    token_mask: torch.Tensor | None
    seq_offsets: torch.Tensor | None
    n_tokens: int | None = None      # rows of the logits, where the object comes from moe_balance_loss


def moe_balance_loss_workspace_size(T: int, E: int, S: int = 1) -> int:
    return lib.moe_balance_loss_workspace_size(_int32(T, "T"), _int32(E, "E"), _int32(S, "S"))


def moe_balance_loss(logits: torch.Tensor, topk_idx: torch.Tensor, coeff: float, score: str = "sigmoid",
                     token_mask: torch.Tensor | None = None, seq_offsets: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None) -> BalanceLoss:
    """Load-balance loss of a router from its logits [T, E] (fp32, bf16 or
    fp16, any row stride) and choices topk_idx [T, k] (int32, as moe_route
    gives them).  ``token_mask`` (bool or uint8 [T]): tokens to count.
    ``seq_offsets`` (int32 [S + 1]): the loss per sequence, averaged over the
    sequences that have tokens.  The loss is no node of an autograd graph: its
    gradient is moe_balance_loss_backward's."""
    T, E, stride = _matrix(logits, "logits")
    idx_shape = _cuda(topk_idx, torch.int32, "topk_idx").shape
    if len(idx_shape) != 2 or idx_shape[0] != T:
        raise ValueError(f"topk_idx must be [{T}, k], got {tuple(idx_shape)}")
    k = _int32(idx_shape[1], "k")
    if score not in BALANCE_SCORES:
        raise ValueError(f"score must be one of {', '.join(BALANCE_SCORES)}, got {score!r}")
    if token_mask is not None:
        if isinstance(token_mask, torch.Tensor) and token_mask.dtype == torch.bool:
            token_mask = token_mask.view(torch.uint8)
        _vector(token_mask, torch.uint8, "token_mask", T)
    S = 1
    if seq_offsets is not None:
        S = _int32(_cuda(seq_offsets, torch.int32, "seq_offsets").numel() - 1, "the number of sequences")
        if S < 1:
            raise ValueError("seq_offsets must hold at least two values")
    device = logits.device
    loss = torch.empty(1, dtype=torch.float32, device=device)
    counts = torch.empty(S, E, dtype=torch.int32, device=device)
    tokens = torch.empty(S + 1, dtype=torch.int32, device=device)
    probs = torch.empty(S, E, dtype=torch.float32, device=device)
    if workspace is None:
        workspace = _workspace(lib.moe_balance_loss_workspace_size(T, E, S), device)
    else:
        _cuda(workspace, torch.uint8, "workspace")
    dev = logits.get_device()
    _same_device(dev, topk_idx, token_mask, seq_offsets, workspace)
    _launch(dev, lib.moe_balance_loss, logits.data_ptr(), _DTYPES[logits.dtype], T, E, stride, topk_idx.data_ptr(),
            k, BALANCE_SCORES[score], _ptr(token_mask), _ptr(seq_offsets), S, coeff, loss.data_ptr(),
            counts.data_ptr(), tokens.data_ptr(), probs.data_ptr(), workspace.data_ptr(), workspace.numel())
    return BalanceLoss(loss, counts, tokens, probs, k, score, coeff, token_mask, seq_offsets, T)


def moe_balance_loss_backward(logits: torch.Tensor, fwd: BalanceLoss, grad_loss: torch.Tensor,
                              out: torch.Tensor | None = None) -> torch.Tensor:
    """grad_loss (f32 [1] on the device) times the gradient of fwd.loss with
    respect to logits, in logits' dtype; ``fwd`` is the forward call's result
    for the same logits."""
    T, E, stride = _matrix(logits, "logits")
    counts, mask = fwd.counts, fwd.token_mask
    S, E_fwd = counts.shape
    if E_fwd != E:
        raise ValueError(f"logits have {E} experts and the forward call had {E_fwd}")
    if fwd.n_tokens is not None and fwd.n_tokens != T:
        raise ValueError(f"logits have {T} tokens and the forward call had {fwd.n_tokens}")
    if mask is not None and mask.numel() != T:
        raise ValueError(f"logits have {T} tokens and the forward call's mask {mask.numel()}")
    _vector(grad_loss, torch.float32, "grad_loss", 1)
    dtype = logits.dtype
    if out is None:
        out = torch.empty(T, E, dtype=dtype, device=logits.device)
        out_stride = E
    else:
        rows, cols, out_stride = _matrix(out, "out", (dtype,))
        if rows != T or cols != E:
            raise ValueError(f"out must be {T} x {E}, got {rows} x {cols}")
    dev = logits.get_device()
    _same_device(dev, counts, grad_loss, out)
    if T:
        _launch(dev, lib.moe_balance_loss_backward, logits.data_ptr(), _DTYPES[dtype], T, E, stride, fwd.k,
                BALANCE_SCORES[fwd.score], _ptr(mask), _ptr(fwd.seq_offsets), S, fwd.coeff, counts.data_ptr(),
                fwd.tokens.data_ptr(), grad_loss.data_ptr(), out.data_ptr(), out_stride)
    return out


# ---------------------------------------------------------------------------
# test hooks (include/nvfp4_moe_testing.h)
# ---------------------------------------------------------------------------

def nvfp4_test_e2m1(y: torch.Tensor):
    """(hardware codes, comparison codes) of fp32 values, one code per byte."""
    _cuda(y, torch.float32, "y")
    hw = torch.empty(y.numel(), dtype=torch.uint8, device=y.device)
    sw = torch.empty_like(hw)
    _check(lib.nvfp4_test_e2m1(_p(y), y.numel(), _p(hw), _p(sw), _stream()))
    return hw, sw


def nvfp4_test_e2m1_sweep(first: int, count: int, device="cuda"):
    """(number of disagreeing non-NaN fp32 patterns in [first, first+count), one example or None)."""
    mism = torch.zeros(1, dtype=torch.int64, device=device)
    ex = torch.full((1,), 0xFFFFFFFF, dtype=torch.int64, device=device)
    ex32 = torch.zeros(1, dtype=torch.int32, device=device)
    _check(lib.nvfp4_test_e2m1_sweep(first, count, _p(mism), _p(ex32), _stream()))
    n = int(mism.item())
    return n, (int(ex32.item()) & 0xFFFFFFFF) if n else None


def nvfp4_test_e4m3(s: torch.Tensor):
    _cuda(s, torch.float32, "s")
    codes = torch.empty(s.numel(), dtype=torch.uint8, device=s.device)
    val = torch.empty(s.numel(), dtype=torch.float32, device=s.device)
    _check(lib.nvfp4_test_e4m3(_p(s), s.numel(), _p(codes), _p(val), _stream()))
    return codes, val


def nvfp4_test_router_splits(T: int, H: int):
    """(splits, K stages per split) of the router GEMM for T tokens, hidden H."""
    per = ctypes.c_int(0)
    n = lib.nvfp4_test_router_splits(T, H, ctypes.byref(per))
    if n < 0:
        raise ValueError(f"no router split for T={T} H={H}")
    return n, per.value


def nvfp4_test_mxfp4_plan(M: int, N: int, K: int, E: int = 0):
    """(tokens per tile, K splits, on CTA pairs, pipeline stages) of an MXFP4 product."""
    v = [ctypes.c_int(0) for _ in range(3)]
    nt = lib.nvfp4_test_mxfp4_plan(M, N, K, E, *(ctypes.byref(x) for x in v))
    if nt < 0:
        raise ValueError(f"no MXFP4 product has M={M} N={N} K={K} E={E}")
    return nt, v[0].value, bool(v[1].value), v[2].value


def nvfp4_test_mxfp4_residency(M: int, N: int, K: int, E: int = 0):
    """(CTAs an SM is to hold, dynamic shared memory bytes, tensor memory columns of each) of an MXFP4 product."""
    v = [ctypes.c_int(0) for _ in range(2)]
    ctas = lib.nvfp4_test_mxfp4_residency(M, N, K, E, *(ctypes.byref(x) for x in v))
    if ctas < 0:
        raise ValueError(f"no MXFP4 product has M={M} N={N} K={K} E={E}")
    return ctas, v[0].value, v[1].value


def nvfp4_test_mxfp4_segments(offsets, counts, M: int):
    """[(first row, rows)] of each expert in a grouped product of M rows, from
    lists of E + 1 offsets and E counts (or None)."""
    E = len(offsets) - 1
    ints = ctypes.c_int32 * E
    row0, rows = ints(), ints()
    if lib.nvfp4_test_mxfp4_segments((ctypes.c_int32 * (E + 1))(*offsets), ints(*counts) if counts else None, M, E,
                                     row0, rows) < 0:
        raise ValueError(f"no MXFP4 product has M={M} and {E} experts")
    return list(zip(row0, rows))


def nvfp4_test_mxfp4_fuses(M: int, N: int, K: int, dtype: torch.dtype, wide: bool = True):
    """(pipeline stages, CTAs per SM) of a dense mxfp4_linear that quantises x
    inside the product, None where a kernel before it does."""
    v = [ctypes.c_int(0) for _ in range(2)]
    r = lib.nvfp4_test_mxfp4_fuses(M, N, K, _DTYPES[dtype], int(wide), *(ctypes.byref(x) for x in v))
    if r < 0:
        raise ValueError(f"no MXFP4 product has M={M} N={N} K={K}")
    return (v[0].value, v[1].value) if r else None


def nvfp4_test_sigmoid(l: torch.Tensor):
    _cuda(l, torch.float32, "l")
    out = torch.empty_like(l)
    _check(lib.nvfp4_test_sigmoid(_p(l), l.numel(), _p(out), _stream()))
    return out


def nvfp4_test_mma_peak(iters: int, n: int = 256, with_cp: int = 0, ctas: int | None = None):
    """(FLOP per SM clock per CTA, cycles per CTA) of back-to-back FP4 MMAs."""
    ctas = ctas or torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    cycles = torch.zeros(ctas, dtype=torch.int64, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _check(lib.nvfp4_test_mma_peak(iters, n, int(with_cp), ctas, _p(cycles), _p(status), _stream()))
    torch.cuda.synchronize()
    if int(status.item()) != 0:
        raise Nvfp4Error(4, "mma peak kernel: the completion wait gave up")
    cyc = cycles.cpu().double()
    flops = iters * 4 * 2.0 * 128 * n * 64
    return flops / cyc, cyc


def nvfp4_test_wait_timeout(src: torch.Tensor, limit_ns: int, workspace: torch.Tensor):
    """Queues the kernel whose bounded wait runs out after limit_ns; returns
    (elapsed_ns int64 [2], copied int32 [1]) device tensors.  The status word
    at the start of ``workspace`` is set when the wait gives up."""
    _cuda(src, torch.uint8, "src")
    if src.numel() < 4096:
        raise ValueError("src must hold at least 4096 bytes")
    elapsed = torch.zeros(2, dtype=torch.int64, device=src.device)
    copied = torch.zeros(1, dtype=torch.int32, device=src.device)
    _check(lib.nvfp4_test_wait_timeout(_p(src), int(limit_ns), _p(workspace), workspace.numel(), _p(elapsed),
                                       _p(copied), _stream()))
    return elapsed, copied


def nvfp4_test_block_scale_div(amax: torch.Tensor, g: torch.Tensor):
    """(q_lib, q_ieee, code_lib, code_ieee) for fp32 amax and g of equal size."""
    _cuda(amax, torch.float32, "amax")
    _cuda(g, torch.float32, "g")
    if amax.numel() != g.numel():
        raise ValueError("amax and g must have the same size")
    n = amax.numel()
    ql, qi = torch.empty_like(amax), torch.empty_like(amax)
    cl = torch.empty(n, dtype=torch.uint8, device=amax.device)
    ci = torch.empty_like(cl)
    _check(lib.nvfp4_test_block_scale_div(_p(amax), _p(g), n, _p(ql), _p(qi), _p(cl), _p(ci), _stream()))
    return ql, qi, cl, ci
