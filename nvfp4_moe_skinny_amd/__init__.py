"""nvfp4_moe_skinny_amd: Python binding of libnvfp4moe.so.

Argument marshalling only. Every computation runs in the library's HIP
kernels on the GPU; PyTorch supplies device memory and the current stream.
There is no CPU fallback: if the library is missing, importing the binding
raises.

The functions carry the C names (see include/nvfp4moe.h for the contract)
and take torch tensors on the GPU in the documented dtypes and layouts.
"""
import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnvfp4moe.so")

NVFP4MOE_OK = 0
NVFP4MOE_ERR_NULL_ARG = -1
NVFP4MOE_ERR_BAD_SHAPE = -2
NVFP4MOE_ERR_UNSUPPORTED = -3
NVFP4MOE_ERR_WORKSPACE = -4
NVFP4MOE_ERR_HIP = -5

_vp, _i64, _i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32


class NVFP4MoEError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        super().__init__(f"{where}: {strerror(status)} ({detail})")
        self.status = status


class MoeArgs(ctypes.Structure):
    """Mirror of struct moe_nvfp4_args."""
    _fields_ = [
        ("x", _vp), ("ids", _vp), ("w", _vp), ("offsets", _vp), ("pairs", _vp),
        ("active", _vp), ("active_offsets", _vp), ("n_active", _vp), ("w_gate_up", _vp),
        ("w_down", _vp),
        ("shared_gate_up", _vp), ("shared_down", _vp), ("residual", _vp), ("out", _vp),
        ("workspace", _vp), ("workspace_bytes", _i64),
        ("M", _i64), ("E", _i64), ("k", _i64), ("H", _i64), ("I", _i64),
        ("dense_min_rows", _i64), ("schedule", _i32),
        ("proj_w", _vp), ("proj_n", _i64), ("proj_out", _vp),
    ]

class GroupedArgs(ctypes.Structure):
    """Mirror of struct moe_grouped_args."""
    _fields_ = [
        ("x", _vp), ("x_scales", _vp), ("w", _vp), ("w_scales", _vp), ("pairs", _vp),
        ("active", _vp), ("active_offsets", _vp), ("n_active", _vp), ("y", _vp), ("ldy", _i64),
        ("R", _i64), ("x_rows", _i64), ("pairs_per_row", _i64), ("E", _i64), ("N", _i64),
        ("K", _i64), ("type", _i32), ("y_type", _i32),
    ]


# element types of the block-scaled and grouped calls
NVFP4MOE_BF16, NVFP4MOE_F32, NVFP4MOE_FP8 = 0, 1, 2
_FLOAT_TYPES = {torch.bfloat16: NVFP4MOE_BF16, torch.float32: NVFP4MOE_F32}

# moe_nvfp4_args.schedule
SCHEDULE_AUTO, SCHEDULE_THREE_LAUNCHES, SCHEDULE_TWO_LAUNCHES = 0, 2, 3


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() or "
                          "python nvfp4_moe_skinny_amd/build.py")
    L = ctypes.CDLL(LIB_PATH)
    L.nvfp4moe_strerror.restype = ctypes.c_char_p
    L.nvfp4moe_strerror.argtypes = [_i32]
    L.nvfp4moe_last_error_detail.restype = ctypes.c_char_p
    L.nvfp4moe_last_error_detail.argtypes = []
    L.nvfp4moe_version.restype = ctypes.c_char_p
    L.nvfp4moe_version.argtypes = []
    L.nvfp4_packed_bytes.restype = _i64
    L.nvfp4_packed_bytes.argtypes = [_i64, _i64, _i64]
    L.nvfp4_pack.restype = _i32
    L.nvfp4_pack.argtypes = [_vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp]
    L.nvfp4_quantize.restype = _i32
    L.nvfp4_quantize.argtypes = [_vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp]
    L.nvfp4_dequant_f32.restype = _i32
    L.nvfp4_dequant_f32.argtypes = [_vp, _i64, _i64, _i64, _i32, _i32, _vp, _vp]
    L.nvfp4_skinny_gemm.restype = _i32
    L.nvfp4_skinny_gemm.argtypes = [_vp, _i64, _i64, _vp, _i64, _vp, _vp]
    L.fp8_skinny_gemm.restype = _i32
    L.fp8_skinny_gemm.argtypes = [_vp, _i64, _i64, _vp, _vp, _i64, _vp, _vp]
    L.moe_route_topk.restype = _i32
    L.moe_route_topk.argtypes = [_vp, _vp, _i64, _i64, _i64] + [_vp] * 9
    L.moe_route_project_topk.restype = _i32
    L.moe_route_project_topk.argtypes = [_vp, _vp, _vp, _i64, _i64, _i64, _i64] + [_vp] * 10
    L.moe_nvfp4_workspace_bytes.restype = _i64
    L.moe_nvfp4_workspace_bytes.argtypes = [_i64, _i64, _i64, _i64, _i64, _i32]
    L.moe_nvfp4_decode.restype = _i32
    L.moe_nvfp4_decode.argtypes = [ctypes.POINTER(MoeArgs), _vp]
    L.moe_nvfp4_route_decode.restype = _i32
    L.moe_nvfp4_route_decode.argtypes = [ctypes.POINTER(MoeArgs), _vp, _vp, _vp]
    L.moe_nvfp4_route_decode_static.restype = _i32
    L.moe_nvfp4_route_decode_static.argtypes = [ctypes.POINTER(MoeArgs), _vp, _vp, _vp]
    L.fp8_quantize_rows.restype = _i32
    L.fp8_quantize_rows.argtypes = [_vp, _i32, _i64, _i64, _i64, _i32, _vp, _vp, _vp]
    L.fp8_quantize_blocks.restype = _i32
    L.fp8_quantize_blocks.argtypes = [_vp, _i32, _i64, _i64, _i64, _vp, _vp, _vp]
    L.fp8_block_gemm.restype = _i32
    L.fp8_block_gemm.argtypes = [_vp, _vp, _i64, _i64, _vp, _vp, _i64, _vp, _i32, _i64, _vp]
    L.moe_grouped_gemm.restype = _i32
    L.moe_grouped_gemm.argtypes = [ctypes.POINTER(GroupedArgs), _vp]
    L.moe_combine.restype = _i32
    L.moe_combine.argtypes = [_vp, _i32, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp]
    L.nvfp4moe_stream_blocks.restype = _i64
    L.nvfp4moe_stream_blocks.argtypes = [_i64]
    L.nvfp4moe_stream_read.restype = _i32
    L.nvfp4moe_stream_read.argtypes = [_vp, _i64, _vp, _i64, _vp]
    return L


lib = _load()

EXPORTS = ["nvfp4moe_strerror", "nvfp4moe_last_error_detail", "nvfp4moe_version",
           "fp8_skinny_gemm",
           "nvfp4_packed_bytes", "nvfp4_pack", "nvfp4_quantize", "nvfp4_dequant_f32", "nvfp4_skinny_gemm",
           "moe_route_topk", "moe_route_project_topk", "moe_nvfp4_workspace_bytes", "moe_nvfp4_decode",
           "moe_nvfp4_route_decode", "moe_nvfp4_route_decode_static", "nvfp4moe_stream_blocks",
           "nvfp4moe_stream_read",
           "fp8_quantize_rows", "fp8_quantize_blocks", "fp8_block_gemm", "moe_grouped_gemm",
           "moe_combine"]


def strerror(status: int) -> str:
    return lib.nvfp4moe_strerror(status).decode()


def last_error_detail() -> str:
    return lib.nvfp4moe_last_error_detail().decode()


def version() -> str:
    return lib.nvfp4moe_version().decode()


def _check(status: int, where: str):
    if status != NVFP4MOE_OK:
        raise NVFP4MoEError(status, where, last_error_detail())


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a GPU tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _want(t: Optional[torch.Tensor], name: str, shape, dtype, device):
    """Raises ValueError unless t is None or a contiguous tensor of this
    shape and dtype on `device` (the kernels index it by these sizes)."""
    if t is None:
        return
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, x on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


# ---- weights ------------------------------------------------------------------------

@dataclass
class PackedNVFP4:
    """G packed matrices of N x K in the library layout (device bytes)."""
    data: torch.Tensor  # uint8, nvfp4_packed_bytes(G, N, K)
    G: int
    N: int
    K: int


def nvfp4_packed_bytes(G: int, N: int, K: int) -> int:
    n = lib.nvfp4_packed_bytes(G, N, K)
    if n < 0:
        raise NVFP4MoEError(int(n), "nvfp4_packed_bytes", last_error_detail())
    return int(n)


def nvfp4_pack(codes: torch.Tensor, scales: torch.Tensor, g: torch.Tensor, stream=None,
               out: Optional[torch.Tensor] = None) -> PackedNVFP4:
    """codes uint8 [G][N][K/2], scales uint8 [G][N][K/16], g float32 [G] (GPU)."""
    G, N, kh = codes.shape
    K = kh * 2
    if tuple(scales.shape) != (G, N, K // 16) or tuple(g.shape) != (G,):
        raise ValueError("scales must be [G][N][K/16] and g [G]")
    nbytes = nvfp4_packed_bytes(G, N, K)
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=codes.device)
    _check(lib.nvfp4_pack(_ptr(codes), _ptr(scales), _ptr(g), G, N, K, _ptr(out),
                          _stream(stream)), "nvfp4_pack")
    return PackedNVFP4(out, G, N, K)


def nvfp4_quantize(x: torch.Tensor, stream=None):
    """x bfloat16 [G][N][K] (or [N][K]) -> canonical NVFP4 (codes uint8
    [G][N][K/2], scales uint8 [G][N][K/16], g float32 [G]) on x's device."""
    if x.dtype != torch.bfloat16:
        raise ValueError("x must be bfloat16")
    if x.dim() == 2:
        x = x.unsqueeze(0)
    x = x.contiguous()
    G, N, K = x.shape
    codes = torch.empty((G, N, K // 2), dtype=torch.uint8, device=x.device)
    scales = torch.empty((G, N, K // 16), dtype=torch.uint8, device=x.device)
    g = torch.empty(G, dtype=torch.float32, device=x.device)
    _check(lib.nvfp4_quantize(_ptr(x), G, N, K, _ptr(codes), _ptr(scales), _ptr(g),
                              _stream(stream)), "nvfp4_quantize")
    return codes, scales, g


def nvfp4_dequant_f32(w: PackedNVFP4, apply_g: bool = True, path: int = 0,
                      stream=None) -> torch.Tensor:
    out = torch.empty((w.G, w.N, w.K), dtype=torch.float32, device=w.data.device)
    _check(lib.nvfp4_dequant_f32(_ptr(w.data), w.G, w.N, w.K, int(apply_g), int(path),
                                 _ptr(out), _stream(stream)), "nvfp4_dequant_f32")
    return out


def nvfp4moe_stream_blocks(nbytes: int) -> int:
    n = lib.nvfp4moe_stream_blocks(nbytes)
    if n < 0:
        raise NVFP4MoEError(int(n), "nvfp4moe_stream_blocks", last_error_detail())
    return int(n)


def nvfp4moe_stream_read(src: torch.Tensor, stream=None,
                         sink: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Reads src (any dtype, contiguous, a multiple of 16 bytes) once; returns
    the sink, int32 [blocks], whose XOR is the XOR of src's 32-bit words."""
    nbytes = src.numel() * src.element_size()
    blocks = nvfp4moe_stream_blocks(nbytes)
    if sink is None:
        sink = torch.empty(blocks, dtype=torch.int32, device=src.device)
    _check(lib.nvfp4moe_stream_read(_ptr(src), nbytes, _ptr(sink), sink.numel(), _stream(stream)),
           "nvfp4moe_stream_read")
    return sink


def nvfp4_skinny_gemm(x: torch.Tensor, w: PackedNVFP4, stream=None,
                      out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x bfloat16 [M][K] -> bfloat16 [M][N] = x W^T."""
    if x.dtype != torch.bfloat16:
        raise ValueError("x must be bfloat16")
    M, K = x.shape
    if K != w.K or w.G != 1:
        raise ValueError("shape mismatch")
    if out is None:
        out = torch.empty((M, w.N), dtype=torch.bfloat16, device=x.device)
    _want(out, "out", (M, w.N), torch.bfloat16, x.device)
    _check(lib.nvfp4_skinny_gemm(_ptr(x), M, K, _ptr(w.data), w.N, _ptr(out), _stream(stream)),
           "nvfp4_skinny_gemm")
    return out


def fp8_skinny_gemm(x: torch.Tensor, w_fp8: torch.Tensor, scale: torch.Tensor, stream=None,
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x bfloat16 [M][K], w_fp8 uint8 [N][K] (E4M3 codes), scale float32 [1]
    -> bfloat16 [M][N] = (x W^T) * scale."""
    if x.dtype != torch.bfloat16 or w_fp8.dtype != torch.uint8 or scale.dtype != torch.float32:
        raise ValueError("need bfloat16 x, uint8 w_fp8, float32 scale")
    M, K = x.shape
    N = w_fp8.shape[0]
    if w_fp8.shape[1] != K:
        raise ValueError("shape mismatch")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _want(out, "out", (M, N), torch.bfloat16, x.device)
    _check(lib.fp8_skinny_gemm(_ptr(x), M, K, _ptr(w_fp8), _ptr(scale), N, _ptr(out),
                               _stream(stream)), "fp8_skinny_gemm")
    return out


# ---- routing -------------------------------------------------------------------------

@dataclass
class Routing:
    ids: torch.Tensor       # int32 [M][k]
    w: torch.Tensor         # float32 [M][k]
    counts: torch.Tensor    # int32 [E]
    offsets: torch.Tensor   # int32 [E+1]
    pairs: torch.Tensor     # int32 [M*k]
    active: torch.Tensor    # int32 [E]
    active_offsets: torch.Tensor  # int32 [E+1]
    n_active: torch.Tensor  # int32 [1]


def routing_buffers(M: int, E: int, k: int, device) -> Routing:
    i32 = dict(dtype=torch.int32, device=device)
    return Routing(torch.empty((M, k), **i32), torch.empty((M, k), dtype=torch.float32,
                                                           device=device),
                   torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(M * k, **i32),
                   torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(1, **i32))


def moe_route_topk(logits: torch.Tensor, k: int, bias: Optional[torch.Tensor] = None,
                   stream=None, out: Optional[Routing] = None) -> Routing:
    """logits float32 [M][E] (+ bias float32 [E])."""
    if logits.dtype != torch.float32 or (bias is not None and bias.dtype != torch.float32):
        raise ValueError("logits and bias must be float32")
    M, E = logits.shape
    r = routing_buffers(M, E, k, logits.device) if out is None else out
    _check(lib.moe_route_topk(_ptr(logits), _ptr(bias), M, E, k, _ptr(r.ids), _ptr(r.w),
                              _ptr(r.counts), _ptr(r.offsets), _ptr(r.pairs), _ptr(r.active),
                              _ptr(r.active_offsets), _ptr(r.n_active), _stream(stream)),
           "moe_route_topk")
    return r


def moe_route_project_topk(x: torch.Tensor, w_router: torch.Tensor, k: int,
                           bias: Optional[torch.Tensor] = None, stream=None,
                           out: Optional[Routing] = None,
                           logits: Optional[torch.Tensor] = None):
    """x bfloat16 [M][H], w_router bfloat16 [E][H] (+ bias float32 [E]) ->
    (logits float32 [M][E], Routing): the router projection, then top-k."""
    if x.dtype != torch.bfloat16 or w_router.dtype != torch.bfloat16:
        raise ValueError("x and w_router must be bfloat16")
    if bias is not None and bias.dtype != torch.float32:
        raise ValueError("bias must be float32")
    M, H = x.shape
    E = w_router.shape[0]
    if w_router.shape[1] != H:
        raise ValueError("shape mismatch")
    r = routing_buffers(M, E, k, x.device) if out is None else out
    if logits is None:
        logits = torch.empty((M, E), dtype=torch.float32, device=x.device)
    _check(lib.moe_route_project_topk(_ptr(x), _ptr(w_router), _ptr(bias), M, E, k, H,
                                      _ptr(logits), _ptr(r.ids), _ptr(r.w), _ptr(r.counts),
                                      _ptr(r.offsets), _ptr(r.pairs), _ptr(r.active),
                                      _ptr(r.active_offsets), _ptr(r.n_active), _stream(stream)),
           "moe_route_project_topk")
    return logits, r


# ---- MoE block ---------------------------------------------------------------------------

def moe_nvfp4_workspace_bytes(M: int, E: int, k: int, H: int, I: int, has_shared: bool) -> int:
    n = lib.moe_nvfp4_workspace_bytes(M, E, k, H, I, int(has_shared))
    if n < 0:
        raise NVFP4MoEError(int(n), "moe_nvfp4_workspace_bytes", last_error_detail())
    return int(n)


def moe_workspace(M: int, E: int, k: int, H: int, I: int, has_shared: bool,
                  device) -> torch.Tensor:
    """A workspace for these sizes (needs no initialisation)."""
    return torch.empty(moe_nvfp4_workspace_bytes(M, E, k, H, I, has_shared), dtype=torch.uint8,
                       device=device)


def _check_block_args(x, E, k, H, I, residual, out, ids, w, workspace, shared_gate_up,
                      shared_down):
    M = x.shape[0]
    dev = x.device
    _want(residual, "residual", (M, H), torch.bfloat16, dev)
    _want(out, "out", (M, H), torch.bfloat16, dev)
    _want(ids, "ids", (M, k), torch.int32, dev)
    _want(w, "w", (M, k), torch.float32, dev)
    if workspace is not None and (workspace.dtype != torch.uint8 or workspace.device != dev
                                  or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous uint8 tensor on x's device")
    if (shared_gate_up is None) != (shared_down is None):
        raise ValueError("shared_gate_up and shared_down go together")
    if shared_gate_up is not None:
        if (shared_gate_up.G, shared_gate_up.N, shared_gate_up.K) != (1, 2 * I, H) or \
                (shared_down.G, shared_down.N, shared_down.K) != (1, H, I):
            raise ValueError("shared expert shapes do not match the routed experts")


def moe_nvfp4_decode(x: torch.Tensor, routing: Routing, w_gate_up: PackedNVFP4,
                     w_down: PackedNVFP4, shared_gate_up: Optional[PackedNVFP4] = None,
                     shared_down: Optional[PackedNVFP4] = None,
                     residual: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None,
                     out: Optional[torch.Tensor] = None, schedule: int = SCHEDULE_AUTO,
                     dense_min_rows: int = 0) -> torch.Tensor:
    """x bfloat16 [M][H] -> bfloat16 [M][H] (routed experts + shared + residual).
    schedule: SCHEDULE_AUTO / SCHEDULE_THREE_LAUNCHES / SCHEDULE_TWO_LAUNCHES;
    dense_min_rows: rows from which a slot uses MFMA (0 = library default)."""
    if x.dtype != torch.bfloat16:
        raise ValueError("x must be bfloat16")
    M, H = x.shape
    E, I = w_gate_up.G, w_down.K
    k = routing.ids.shape[1]
    if w_gate_up.N != 2 * I or w_gate_up.K != H or w_down.N != H or w_down.G != E:
        raise ValueError("expert weight shapes do not match x")
    _check_block_args(x, E, k, H, I, residual, out, routing.ids, routing.w, workspace,
                      shared_gate_up, shared_down)
    dev = x.device
    for name, t, n in (("offsets", routing.offsets, E + 1), ("pairs", routing.pairs, M * k),
                       ("active", routing.active, E),
                       ("active_offsets", routing.active_offsets, E + 1),
                       ("n_active", routing.n_active, 1)):
        _want(t, name, (n,), torch.int32, dev)
    has_shared = shared_gate_up is not None
    if workspace is None:
        workspace = moe_workspace(M, E, k, H, I, has_shared, x.device)
    if out is None:
        out = torch.empty_like(x)
    a = MoeArgs()
    a.x, a.ids, a.w = _ptr(x), _ptr(routing.ids), _ptr(routing.w)
    a.offsets, a.pairs = _ptr(routing.offsets), _ptr(routing.pairs)
    a.active, a.n_active = _ptr(routing.active), _ptr(routing.n_active)
    a.active_offsets = _ptr(routing.active_offsets)
    a.w_gate_up, a.w_down = _ptr(w_gate_up.data), _ptr(w_down.data)
    a.shared_gate_up = _ptr(shared_gate_up.data) if has_shared else None
    a.shared_down = _ptr(shared_down.data) if has_shared else None
    a.residual = _ptr(residual)
    a.out = _ptr(out)
    a.workspace, a.workspace_bytes = _ptr(workspace), workspace.numel()
    a.M, a.E, a.k, a.H, a.I = M, E, k, H, I
    a.dense_min_rows, a.schedule = dense_min_rows, schedule
    _check(lib.moe_nvfp4_decode(ctypes.byref(a), _stream(stream)), "moe_nvfp4_decode")
    return out


def moe_nvfp4_route_decode(x: torch.Tensor, logits: torch.Tensor, k: int,
                           w_gate_up: PackedNVFP4, w_down: PackedNVFP4,
                           bias: Optional[torch.Tensor] = None,
                           shared_gate_up: Optional[PackedNVFP4] = None,
                           shared_down: Optional[PackedNVFP4] = None,
                           residual: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None, stream=None,
                           out: Optional[torch.Tensor] = None,
                           ids: Optional[torch.Tensor] = None, w: Optional[torch.Tensor] = None,
                           dense_min_rows: int = 0, proj: Optional[PackedNVFP4] = None,
                           proj_out: Optional[torch.Tensor] = None,
                           static_scratch: bool = False):
    """Routing (top-k + weights) and the MoE block in two launches, for few
    rows: x bfloat16 [M][H], logits float32 [M][E] (+ bias float32 [E]) ->
    (out bfloat16 [M][H], ids int32 [M][k], w float32 [M][k]). With proj
    (packed [N][H]), proj_out bfloat16 [M][N] = x proj^T is written too, by
    blocks of the down launch (allocated if not given).
    static_scratch: call moe_nvfp4_route_decode_static, whose h rows live in
    the library's own device array (no workspace; pass out, ids and w to
    allocate nothing here either)."""
    if x.dtype != torch.bfloat16 or logits.dtype != torch.float32:
        raise ValueError("x must be bfloat16 and logits float32")
    if bias is not None and bias.dtype != torch.float32:
        raise ValueError("bias must be float32")
    M, H = x.shape
    E, I = w_gate_up.G, w_down.K
    if w_gate_up.N != 2 * I or w_gate_up.K != H or w_down.N != H or w_down.G != E:
        raise ValueError("expert weight shapes do not match x")
    if tuple(logits.shape) != (M, E):
        raise ValueError("logits must be [M][E]")
    _want(logits, "logits", (M, E), torch.float32, x.device)
    _want(bias, "bias", (E,), torch.float32, x.device)
    _check_block_args(x, E, k, H, I, residual, out, ids, w, workspace, shared_gate_up,
                      shared_down)
    has_shared = shared_gate_up is not None
    if workspace is None and not static_scratch:
        workspace = moe_workspace(M, E, k, H, I, has_shared, x.device)
    if out is None:
        out = torch.empty_like(x)
    if ids is None:
        ids = torch.empty((M, k), dtype=torch.int32, device=x.device)
    if w is None:
        w = torch.empty((M, k), dtype=torch.float32, device=x.device)
    a = MoeArgs()
    a.x, a.ids, a.w = _ptr(x), _ptr(ids), _ptr(w)
    a.w_gate_up, a.w_down = _ptr(w_gate_up.data), _ptr(w_down.data)
    a.shared_gate_up = _ptr(shared_gate_up.data) if has_shared else None
    a.shared_down = _ptr(shared_down.data) if has_shared else None
    a.residual = _ptr(residual)
    a.out = _ptr(out)
    if not static_scratch:
        a.workspace, a.workspace_bytes = _ptr(workspace), workspace.numel()
    a.M, a.E, a.k, a.H, a.I = M, E, k, H, I
    a.dense_min_rows, a.schedule = dense_min_rows, SCHEDULE_AUTO
    if proj is not None:
        if proj.G != 1 or proj.K != H:
            raise ValueError("proj must be one packed [N][H] matrix")
        if proj_out is None:
            proj_out = torch.empty((M, proj.N), dtype=torch.bfloat16, device=x.device)
        _want(proj_out, "proj_out", (M, proj.N), torch.bfloat16, x.device)
        a.proj_w, a.proj_n, a.proj_out = _ptr(proj.data), proj.N, _ptr(proj_out)
    if static_scratch:
        _check(lib.moe_nvfp4_route_decode_static(ctypes.byref(a), _ptr(logits), _ptr(bias),
                                                 _stream(stream)), "moe_nvfp4_route_decode_static")
    else:
        _check(lib.moe_nvfp4_route_decode(ctypes.byref(a), _ptr(logits), _ptr(bias),
                                          _stream(stream)), "moe_nvfp4_route_decode")
    return out, ids, w


# ---- FP8 with a scale per block of 128, products grouped by expert -----------------------

@dataclass
class Fp8Rows:
    """Rows of E4M3 codes with a scale per 128 columns, block-major."""
    codes: torch.Tensor   # uint8 [M][K]
    scales: torch.Tensor  # float32 [ceil(K/128)][M]


@dataclass
class Fp8Blocks:
    """G weights of E4M3 codes with a scale per 128 x 128 block."""
    codes: torch.Tensor   # uint8 [G][N][K]
    scales: torch.Tensor  # float32 [G][ceil(N/128)][ceil(K/128)]


def _blocks128(n: int) -> int:
    return (n + 127) // 128


# The raw handle of a device's current stream (the plain accessor builds a
# Stream object for it, 2.8 us against 0.1 where a small call takes 8 in all).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _elsewhere(t: torch.Tensor, stream) -> bool:
    """Whether a call on t has to enter another device or stream first (_on)."""
    if not t.is_cuda:
        raise ValueError("expected a GPU tensor")
    return stream is not None or t.get_device() != _current_device()


def _on(t: torch.Tensor, stream):
    """Makes t's device current and the given stream, or the device's current
    one: outputs are then allocated for the stream that writes them."""
    if stream is None:
        stream = torch.cuda.current_stream(t.device)
    elif stream.device != t.device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {t.device}")
    return torch.cuda.stream(stream)


def _want_rows(t: torch.Tensor, name: str, shape, dtype, device):
    """As _want, for a matrix whose rows may be further apart than their length."""
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, x on {device}")
    _check_rows(t, name)


def _check_rows(t: torch.Tensor, name: str):
    if not t.is_contiguous() and (t.shape[1] > 1 and t.stride(1) != 1
                                  or t.shape[0] > 1 and t.stride(0) < t.shape[1]):
        raise ValueError(f"the columns of {name} must be contiguous and its rows apart")


def _row_stride(t: torch.Tensor) -> int:
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _float_type(dtype, name: str) -> int:
    t = _FLOAT_TYPES.get(dtype)
    if t is None:
        raise ValueError(f"{name} must be bfloat16 or float32, got {dtype}")
    return t


def _want_fp8_rows(x: Fp8Rows):
    if x.codes.dim() != 2:
        raise ValueError("row codes must be [M][K]")
    M, K = x.codes.shape
    _want(x.codes, "row codes", (M, K), torch.uint8, x.codes.device)
    _want(x.scales, "row scales", (_blocks128(K), M), torch.float32, x.codes.device)
    return M, K


def _want_fp8_blocks(w: Fp8Blocks, K: int, device):
    if w.codes.dim() != 3 or w.codes.shape[2] != K:
        raise ValueError(f"weight codes must be [G][N][{K}], got {list(w.codes.shape)}")
    G, N, _ = w.codes.shape
    _want(w.codes, "weight codes", (G, N, K), torch.uint8, device)
    _want(w.scales, "weight scales", (G, _blocks128(N), _blocks128(K)), torch.float32, device)
    return G, N


def fp8_quantize_rows(x: torch.Tensor, swiglu: bool = False, stream=None,
                      out: Optional[Fp8Rows] = None) -> Fp8Rows:
    """x bfloat16 or float32 [M][K] -> E4M3 rows; swiglu: x [M][2K], of
    silu(x[:, :K]) * x[:, K:]. Rows of x may be strided."""
    if _elsewhere(x, stream):
        with _on(x, stream):
            return fp8_quantize_rows(x, swiglu, None, out)
    if x.dim() != 2 or (swiglu and x.shape[1] % 2):
        raise ValueError("x must be [M][K], or [M][2K] with swiglu")
    xt = _float_type(x.dtype, "x")
    _check_rows(x, "x")
    M, K = x.shape
    ldx = x.stride(0) if M > 1 else K
    if swiglu:
        K //= 2
    if out is None:
        dev = x.device
        out = Fp8Rows(torch.empty(M, K, dtype=torch.uint8, device=dev),
                      torch.empty(_blocks128(K), M, dtype=torch.float32, device=dev))
    else:
        _want(out.codes, "out.codes", (M, K), torch.uint8, x.device)
        _want(out.scales, "out.scales", (_blocks128(K), M), torch.float32, x.device)
    _check(lib.fp8_quantize_rows(x.data_ptr(), xt, M, K, ldx, swiglu, out.codes.data_ptr(),
                                 out.scales.data_ptr(), _raw_stream(x.get_device())),
           "fp8_quantize_rows")
    return out


def fp8_quantize_blocks(w: torch.Tensor, stream=None,
                        out: Optional[Fp8Blocks] = None) -> Fp8Blocks:
    """w bfloat16 or float32 [G][N][K] (or [N][K]: G = 1) -> E4M3 weights."""
    if _elsewhere(w, stream):
        with _on(w, stream):
            return fp8_quantize_blocks(w, None, out)
    wt = _float_type(w.dtype, "w")
    if w.dim() == 2:
        w = w.unsqueeze(0)
    if w.dim() != 3:
        raise ValueError("w must be [G][N][K] or [N][K]")
    G, N, K = w.shape
    dev = w.device
    if out is None:
        out = Fp8Blocks(torch.empty(G, N, K, dtype=torch.uint8, device=dev),
                        torch.empty(G, _blocks128(N), _blocks128(K), dtype=torch.float32,
                                    device=dev))
    else:
        _want(out.codes, "out.codes", (G, N, K), torch.uint8, dev)
        _want(out.scales, "out.scales", (G, _blocks128(N), _blocks128(K)), torch.float32, dev)
    _check(lib.fp8_quantize_blocks(_ptr(w), wt, G, N, K, out.codes.data_ptr(),
                                   out.scales.data_ptr(), _raw_stream(w.get_device())),
           "fp8_quantize_blocks")
    return out


def fp8_block_gemm(x: Fp8Rows, w: Fp8Blocks, out_dtype: torch.dtype = torch.bfloat16,
                   stream=None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x [M][K], w G = 1 [N][K] -> out_dtype [M][N] = x w^T. Rows of out may be strided."""
    if _elsewhere(x.codes, stream):
        with _on(x.codes, stream):
            return fp8_block_gemm(x, w, out_dtype, None, out)
    M, K = _want_fp8_rows(x)
    dev = x.codes.device
    G, N = _want_fp8_blocks(w, K, dev)
    if G != 1:
        raise ValueError("w must hold one matrix")
    yt = _float_type(out_dtype, "out_dtype")
    if out is None:
        out = torch.empty(M, N, dtype=out_dtype, device=dev)
        ldy = N
    else:
        _want_rows(out, "out", (M, N), out_dtype, dev)
        ldy = _row_stride(out)
    _check(lib.fp8_block_gemm(x.codes.data_ptr(), x.scales.data_ptr(), M, K, w.codes.data_ptr(),
                              w.scales.data_ptr(), N, out.data_ptr(), yt, ldy,
                              _raw_stream(x.codes.get_device())), "fp8_block_gemm")
    return out


def moe_grouped_gemm(x, routing: Routing, w, out_dtype: torch.dtype = torch.bfloat16,
                     stream=None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Products grouped by expert: x bfloat16 [rows][K] with w bfloat16 [E][N][K],
    or x Fp8Rows with w Fp8Blocks -> out_dtype [M k][N] in pair order. rows is M
    (token rows: pair p reads row p // k) or M k (pair p reads row p). Rows of
    out may be strided; those of pairs in no active slot are left as they were."""
    fp8 = isinstance(x, Fp8Rows)
    if fp8 != isinstance(w, Fp8Blocks):
        raise ValueError("x and w must both be FP8 (Fp8Rows, Fp8Blocks) or both bfloat16")
    xc = x.codes if fp8 else x
    if _elsewhere(xc, stream):
        with _on(xc, stream):
            return moe_grouped_gemm(x, routing, w, out_dtype, None, out)
    M, k = routing.ids.shape
    R = M * k
    dev = xc.device
    a = GroupedArgs()
    if fp8:
        rows, K = _want_fp8_rows(x)
        E, N = _want_fp8_blocks(w, K, dev)
        a.x_scales, a.w_scales = x.scales.data_ptr(), w.scales.data_ptr()
        a.w, a.type = w.codes.data_ptr(), NVFP4MOE_FP8
    else:
        if x.dim() != 2 or w.dim() != 3 or x.shape[1] != w.shape[2]:
            raise ValueError("need x [rows][K] and w [E][N][K]")
        rows, K = x.shape
        E, N = w.shape[:2]
        _want(x, "x", (rows, K), torch.bfloat16, dev)
        _want(w, "w", (E, N, K), torch.bfloat16, dev)
        a.w, a.type = w.data_ptr(), NVFP4MOE_BF16
    if rows != M and rows != R:
        raise ValueError(f"x has {rows} rows: need {M} (token rows) or {R} (a row per pair)")
    for name, t, n in (("pairs", routing.pairs, R), ("active", routing.active, E),
                       ("active_offsets", routing.active_offsets, E + 1),
                       ("n_active", routing.n_active, 1)):
        _want(t, name, (n,), torch.int32, dev)
    a.x = xc.data_ptr()
    a.pairs, a.active = routing.pairs.data_ptr(), routing.active.data_ptr()
    a.active_offsets, a.n_active = routing.active_offsets.data_ptr(), routing.n_active.data_ptr()
    a.R, a.x_rows, a.pairs_per_row = R, rows, 1 if rows == R else k
    a.E, a.N, a.K = E, N, K
    a.y_type = _float_type(out_dtype, "out_dtype")
    if out is None:
        out = torch.empty(R, N, dtype=out_dtype, device=dev)
        a.ldy = N
    else:
        _want_rows(out, "out", (R, N), out_dtype, dev)
        a.ldy = _row_stride(out)
    a.y = out.data_ptr()
    _check(lib.moe_grouped_gemm(ctypes.byref(a), _raw_stream(xc.get_device())),
           "moe_grouped_gemm")
    return out


def moe_combine(y: torch.Tensor, w: torch.Tensor, shared: Optional[torch.Tensor] = None,
                residual: Optional[torch.Tensor] = None, stream=None,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y bfloat16 or float32 [M k][H], w float32 [M][k] (+ shared [M][H] of y's
    type, residual bfloat16 [M][H]) -> bfloat16 [M][H]."""
    if _elsewhere(y, stream):
        with _on(y, stream):
            return moe_combine(y, w, shared, residual, None, out)
    if y.dim() != 2 or w.dim() != 2:
        raise ValueError("need y [M k][H] and w [M][k]")
    yt = _float_type(y.dtype, "y")
    M, k = w.shape
    H = y.shape[1]
    dev = y.device
    _want(y, "y", (M * k, H), y.dtype, dev)
    _want(w, "w", (M, k), torch.float32, dev)
    _want(shared, "shared", (M, H), y.dtype, dev)
    _want(residual, "residual", (M, H), torch.bfloat16, dev)
    if out is None:
        out = torch.empty(M, H, dtype=torch.bfloat16, device=dev)
    else:
        _want(out, "out", (M, H), torch.bfloat16, dev)
    _check(lib.moe_combine(y.data_ptr(), yt, w.data_ptr(),
                           None if shared is None else shared.data_ptr(),
                           None if residual is None else residual.data_ptr(), M, k, H,
                           out.data_ptr(), _raw_stream(y.get_device())), "moe_combine")
    return out
