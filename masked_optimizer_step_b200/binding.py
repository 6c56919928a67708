"""Python binding of the C ABI in include/sf.h -- argument marshalling only.

Every function here has the name of the C entry point it calls and does nothing but turn torch
tensors into pointers and sizes; all work runs in the CUDA kernels of libsf.so. There is no
fallback: if the library is missing or no B200 is present, calls raise.

State holders (`Mask`, `Matrix`) allocate their device arrays with torch (PyTorch serves as the
device-memory and stream provider) and expose the C structs the ABI takes.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsf.so")

SF_OK = 0
SF_STATUS_SLOT_OVERFLOW = 0x1
SF_STATUS_NONFINITE = 0x2
SF_STATUS_BAD_TOKEN = 0x4
SF_STATUS_WAIT_TIMEOUT = 0x8
SF_STATUS_BAD_OFFSET = 0x10

SF_SRC_TOKENS = 0
SF_SRC_OUTPUT_BF16 = 1
SF_SRC_HITS_U32 = 2
SF_SRC_WORDS = 3

SF_PHASE_ALL = 0
SF_PHASE_FIRST = 1
SF_PHASE_SECOND = 2

SF_TYPE_F32 = 0
SF_TYPE_BF16 = 1
SF_TYPE_F16 = 2
SF_TYPE_E4M3 = 3
SF_DENSE_BLOCK = 256
SF_DENSE_PER_LAUNCH = 384
SF_GROUPED_MAX_EXPERTS = 1024
SF_GROUPED_FORWARD, SF_GROUPED_DX, SF_GROUPED_DW = 0, 1, 2
SF_GROUPED_NONE = 0
SF_GROUPED_SINGLE = 1
SF_GROUPED_ROUNDS = 2
SF_GROUPED_SLICES = 3
SF_GROUPED_CLUSTERS = 4
SF_GROUPED_PAIRS = 5
SF_GROUPED_PAIRS_FEW = 6
SF_GROUPED_PAIRS_ADD = 7

SF_DW_MAX_PER_LAUNCH = 96
SF_MASKS_PER_LAUNCH = 240
SF_MASK_SPLIT_ROWS = 16384
SF_MATS_PER_LAUNCH = 256

_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_F = ctypes.c_float


class sf_mask(ctypes.Structure):
    _fields_ = [("R", _I32), ("slot_cap", _I32), ("charge", _P), ("accum", _P), ("words", _P),
                ("active_rows", _P), ("active_tiles", _P), ("tile_rows", _P), ("row_slot", _P), ("free_slots", _P),
                ("slot_step", _P), ("counts", _P)]


class sf_mask_src(ctypes.Structure):
    _fields_ = [("kind", _I32), ("n", _I32), ("ld", _I64), ("ptr", _P)]


class sf_dw_problem(ctypes.Structure):
    _fields_ = [("dX", _P), ("ld_dx", _I64), ("A", _P), ("ld_a", _I64), ("T", _I32), ("C", _I32),
                ("mask", sf_mask), ("dW", _P), ("ld_dw", _I64)]


class sf_fwd_problem(ctypes.Structure):
    _fields_ = [("A", _P), ("ld_a", _I64), ("W", _P), ("ld_w", _I64), ("Y", _P), ("ld_y", _I64),
                ("T", _I32), ("C", _I32), ("mask", sf_mask)]


class sf_matrix(ctypes.Structure):
    _fields_ = [("C", _I32), ("partner", _I32), ("c_self", _F), ("c_partner", _F),
                ("mask", sf_mask), ("q", _P), ("s", _P), ("delta", _P), ("m", _P), ("v", _P),
                ("grad", _P), ("live", _P)]


class sf_checkpoint(ctypes.Structure):
    _fields_ = [("cap", _I32), ("count", _P), ("rows", _P), ("q", _P), ("s", _P), ("delta", _P),
                ("m", _P), ("v", _P), ("step", _P)]


class sf_adam(ctypes.Structure):
    _fields_ = [("lr", _F), ("beta1", _F), ("beta2", _F), ("eps", _F), ("one_minus_b1", _F),
                ("one_minus_b2", _F), ("wd", _F), ("clip", _F), ("bc1", _P), ("bc2", _P),
                ("t_max", _I32)]


class sf_dense(ctypes.Structure):
    _fields_ = [("n", _I64), ("p", _P), ("g", _P), ("m", _P), ("v", _P), ("m_scale", _P), ("v_scale", _P),
                ("live", _P), ("decay", _F), ("p_type", _I32), ("g_type", _I32), ("state_type", _I32)]


class sf_grouped(ctypes.Structure):
    _fields_ = [("A", _P), ("ld_a", _I64), ("W", _P), ("ld_w", _I64), ("stride_w", _I64), ("Y", _P), ("ld_y", _I64),
                ("offsets", _P), ("E", _I32), ("T", _I32), ("R", _I32), ("C", _I32), ("type", _I32), ("w_type", _I32)]


_lib = None


def load():
    """Load libsf.so (built in-tree by build.py). Raises if it is absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: run `python -m masked_optimizer_step_b200.build`;"
                           " there is no CPU fallback")
    L = ctypes.CDLL(LIB_PATH)
    L.sf_status_string.restype = ctypes.c_char_p
    L.sf_status_string.argtypes = [ctypes.c_int]
    L.sf_version.restype = ctypes.c_int
    L.sf_mask_init.argtypes = [ctypes.POINTER(sf_mask), _P]
    L.sf_mask_update.argtypes = [ctypes.POINTER(sf_mask), ctypes.POINTER(sf_mask_src), ctypes.c_int,
                                 _F, _P, _P]
    L.sf_masked_dw.argtypes = [ctypes.POINTER(sf_dw_problem), ctypes.c_int, _P, ctypes.c_size_t, _P, _P]
    L.sf_forward_tracked.argtypes = [ctypes.POINTER(sf_fwd_problem), ctypes.c_int, _P, _P]
    L.sf_mask_update_phase.argtypes = [ctypes.POINTER(sf_mask), ctypes.POINTER(sf_mask_src), ctypes.c_int,
                                       _F, ctypes.c_int, _P, _P]
    L.sf_masked_dw_phase.argtypes = [ctypes.POINTER(sf_dw_problem), ctypes.c_int, _P, ctypes.c_size_t,
                                     ctypes.c_int, _P, _P]
    L.sf_masked_dw_unit_rows.restype = ctypes.c_int
    L.sf_masked_dw_unit_rows.argtypes = []
    L.sf_masked_dw_ws_bytes.restype = ctypes.c_size_t
    L.sf_masked_dw_ws_bytes.argtypes = [ctypes.POINTER(sf_dw_problem), ctypes.c_int]
    L.sf_embed_grad_ws_bytes.restype = ctypes.c_size_t
    L.sf_embed_grad_ws_bytes.argtypes = [ctypes.c_int, ctypes.c_int]
    L.sf_embed_grad.argtypes = [_P, ctypes.c_int, _P, ctypes.c_int, _I64, ctypes.POINTER(sf_mask), _P,
                                _I64, _P, ctypes.c_size_t, _P, _P]
    L.sf_embed_grad_noalloc.argtypes = [_P, ctypes.c_int, _P, ctypes.c_int, _I64, ctypes.POINTER(sf_mask),
                                        _P, _I64, _P, _P]
    L.sf_embed_grad_noalloc.restype = ctypes.c_int
    L.sf_adam_tables.argtypes = [_F, _F, ctypes.c_int, _P, _P, _P]
    L.sf_sparse_update.argtypes = [ctypes.POINTER(sf_matrix), ctypes.c_int, ctypes.POINTER(sf_adam),
                                   _P, _P]
    L.sf_quantize_init.argtypes = [_P, ctypes.c_int, ctypes.c_int, _P, _P, _P, _P, _P]
    for name in ("sf_checkpoint_save", "sf_checkpoint_restore"):
        getattr(L, name).argtypes = [ctypes.POINTER(sf_matrix), ctypes.POINTER(sf_checkpoint), ctypes.c_int, _P, _P]
        getattr(L, name).restype = ctypes.c_int
    L.sf_grad_norm_ws_bytes.restype = ctypes.c_size_t
    L.sf_grad_norm_ws_bytes.argtypes = [ctypes.POINTER(sf_dense), ctypes.c_int]
    L.sf_grad_norm.argtypes = [ctypes.POINTER(sf_dense), ctypes.c_int, _F, _F, _P, _P, ctypes.c_size_t, _P, _P]
    L.sf_adamw_step.argtypes = [ctypes.POINTER(sf_dense), ctypes.c_int, ctypes.POINTER(sf_adam), _P, _P, _P, _P]
    L.sf_grouped_forward.argtypes = [ctypes.POINTER(sf_grouped), _P, _P]
    L.sf_grouped_dx.argtypes = [ctypes.POINTER(sf_grouped), _P, _P]
    L.sf_grouped_dw.argtypes = [ctypes.POINTER(sf_grouped), ctypes.c_int, _P, _P]
    L.sf_grouped_kernel.argtypes = [ctypes.POINTER(sf_grouped), ctypes.c_int, ctypes.c_int]
    for name in ("sf_grad_norm", "sf_adamw_step", "sf_grouped_forward", "sf_grouped_dx", "sf_grouped_dw", "sf_grouped_kernel"):
        getattr(L, name).restype = ctypes.c_int
    for name in ("sf_mask_init", "sf_mask_update", "sf_masked_dw", "sf_embed_grad", "sf_adam_tables",
                 "sf_sparse_update", "sf_quantize_init", "sf_mask_update_phase", "sf_masked_dw_phase",
                 "sf_forward_tracked"):
        getattr(L, name).restype = ctypes.c_int
    _lib = L
    return L


def _check(rc: int, what: str):
    if rc != SF_OK:
        msg = load().sf_status_string(rc).decode()
        raise RuntimeError(f"{what} failed: {msg} ({rc})")


def _ptr(t) -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("device tensor expected")
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream or None


def status_word(device=None) -> torch.Tensor:
    """A zeroed device status word (uint32 bits, held in an int32 tensor)."""
    return torch.zeros(1, dtype=torch.int32, device=device or "cuda")


# ---------------------------------------------------------------------------------------------
# State holders
# ---------------------------------------------------------------------------------------------

class Mask:
    """Device arrays of one sf_mask (section 2.1 state: charges, mask, lists, slots)."""

    def __init__(self, R: int, slot_cap: int, device="cuda"):
        if R % 32:
            raise ValueError("R must be a multiple of 32")
        i32 = dict(dtype=torch.int32, device=device)
        self.R, self.slot_cap = R, slot_cap
        self.charge = torch.zeros(R, dtype=torch.float32, device=device)
        self.accum = torch.zeros(R, **i32)
        self.words = torch.zeros(R // 32, **i32)
        self.active_rows = torch.zeros(R, **i32)
        self.active_tiles = torch.zeros(R // 32, **i32)
        self.tile_rows = torch.zeros(R // 32, **i32)
        self.row_slot = torch.full((R,), -1, **i32)
        self.free_slots = torch.zeros(max(slot_cap, 1), **i32)
        self.slot_step = torch.zeros(max(slot_cap, 1), **i32)
        self.counts = torch.zeros(8, **i32)

    def struct(self) -> sf_mask:
        return sf_mask(self.R, self.slot_cap, _ptr(self.charge), _ptr(self.accum), _ptr(self.words),
                       _ptr(self.active_rows), _ptr(self.active_tiles), _ptr(self.tile_rows), _ptr(self.row_slot),
                       _ptr(self.free_slots), _ptr(self.slot_step), _ptr(self.counts))


class Matrix:
    """int8 + scale + residual weights of one matrix with its moments, gradient and live copy."""

    def __init__(self, R: int, C: int, slot_cap: int, device="cuda", live=True):
        self.R, self.C = R, C
        self.mask = Mask(R, slot_cap, device)
        self.q = torch.zeros((R, C), dtype=torch.int8, device=device)
        self.s = torch.zeros(R, dtype=torch.float32, device=device)
        self.delta = torch.zeros((R, C), dtype=torch.float32, device=device)
        n = max(slot_cap, 1)
        self.m = torch.zeros((n, C), dtype=torch.int16, device=device)
        self.v = torch.zeros((n, C), dtype=torch.int16, device=device)
        self.grad = torch.zeros((n, C), dtype=torch.float32, device=device)
        self.live = torch.zeros((R, C), dtype=torch.int16, device=device) if live else None


# ---------------------------------------------------------------------------------------------
# Entry points (same names as the C ABI)
# ---------------------------------------------------------------------------------------------

def sf_mask_init(mask: Mask, stream=None):
    m = mask.struct()
    _check(load().sf_mask_init(ctypes.byref(m), _stream(stream)), "sf_mask_init")


class Desc:
    """A C descriptor together with the tensors its pointers refer to.

    The tensors stay referenced for as long as the descriptor lives, so that a temporary cannot
    be freed (and its memory handed to the next allocation) before the kernel that reads it has
    been enqueued.
    """

    __slots__ = ("c", "refs")

    def __init__(self, c, *refs):
        self.c = c
        self.refs = refs


def make_src(kind: int, tensor=None, n: int = 0, ld: int = 0) -> Desc:
    return Desc(sf_mask_src(kind, n, ld, _ptr(tensor) if tensor is not None else None), tensor)


def sf_mask_update(masks, srcs, threshold: float = 0.01, status=None, stream=None):
    """masks: list of Mask; srcs: list of make_src() descriptors."""
    n = len(masks)
    arr_m = (sf_mask * n)(*[m.struct() for m in masks])
    arr_s = (sf_mask_src * n)(*[s.c for s in srcs])
    _check(load().sf_mask_update(arr_m, arr_s, n, threshold, _ptr(status), _stream(stream)),
           "sf_mask_update")


def sf_mask_update_phase(masks, srcs, phase: int, threshold: float = 0.01, status=None, stream=None):
    """One pass of sf_mask_update (SF_PHASE_FIRST: activity, SF_PHASE_SECOND: finalize)."""
    n = len(masks)
    arr_m = (sf_mask * n)(*[m.struct() for m in masks])
    arr_s = (sf_mask_src * n)(*[s.c for s in srcs])
    _check(load().sf_mask_update_phase(arr_m, arr_s, n, threshold, phase, _ptr(status), _stream(stream)),
           "sf_mask_update_phase")


def dw_problem(dX, A, mask: Mask, dW) -> Desc:
    """dX [T x R] bf16, A [T x C] bf16, dW [slot_cap x C] fp32 (row = slot)."""
    T, R = dX.shape
    C = A.shape[1]
    assert A.shape[0] == T and R == mask.R and dX.dtype == torch.bfloat16 and A.dtype == torch.bfloat16
    c = sf_dw_problem(_ptr(dX), dX.stride(0), _ptr(A), A.stride(0), T, C, mask.struct(), _ptr(dW),
                      dW.stride(0))
    return Desc(c, dX, A, dW)


def sf_masked_dw_unit_rows() -> int:
    return load().sf_masked_dw_unit_rows()


def sf_masked_dw_ws_bytes(problems) -> int:
    n = len(problems)
    arr = (sf_dw_problem * n)(*[p.c for p in problems])
    return load().sf_masked_dw_ws_bytes(arr, n)


def dw_workspace(problems, device="cuda") -> torch.Tensor:
    """Scratch for sf_masked_dw's row mode (a byte tensor of sf_masked_dw_ws_bytes bytes)."""
    return torch.empty(max(sf_masked_dw_ws_bytes(problems), 1), dtype=torch.uint8, device=device)


def sf_masked_dw(problems, status=None, stream=None, ws=None):
    """problems: list of dw_problem() descriptors; ws: dw_workspace() scratch, or None for the
    mask-tile mode only."""
    n = len(problems)
    arr = (sf_dw_problem * n)(*[p.c for p in problems])
    nbytes = ws.numel() * ws.element_size() if ws is not None else 0
    _check(load().sf_masked_dw(arr, n, _ptr(ws), nbytes, _ptr(status), _stream(stream)), "sf_masked_dw")


def sf_masked_dw_phase(problems, phase: int, status=None, stream=None, ws=None):
    """One pass of sf_masked_dw (SF_PHASE_FIRST: row gather, SF_PHASE_SECOND: main launches)."""
    n = len(problems)
    arr = (sf_dw_problem * n)(*[p.c for p in problems])
    nbytes = ws.numel() * ws.element_size() if ws is not None else 0
    _check(load().sf_masked_dw_phase(arr, n, _ptr(ws), nbytes, phase, _ptr(status), _stream(stream)),
           "sf_masked_dw_phase")


def fwd_problem(A, W, Y, mask: Mask) -> Desc:
    """A [T x C] bf16 inputs, W [R x C] bf16 weights, Y [T x R] bf16 outputs (written)."""
    T, C = A.shape
    R = W.shape[0]
    assert W.shape[1] == C and Y.shape == (T, R) and R == mask.R
    assert A.dtype == W.dtype == Y.dtype == torch.bfloat16
    c = sf_fwd_problem(_ptr(A), A.stride(0), _ptr(W), W.stride(0), _ptr(Y), Y.stride(0), T, C, mask.struct())
    return Desc(c, A, W, Y)


def sf_forward_tracked(problems, status=None, stream=None):
    """Forward projections Y = A W^T with each projection's row magnitudes folded into its mask's
    accumulator; close the window with sf_mask_update_phase(..., SF_PHASE_SECOND)."""
    n = len(problems)
    arr = (sf_fwd_problem * max(n, 1))(*[p.c for p in problems])
    _check(load().sf_forward_tracked(arr, n, _ptr(status), _stream(stream)), "sf_forward_tracked")


def sf_embed_grad_ws_bytes(n_tok: int, slot_cap: int) -> int:
    return load().sf_embed_grad_ws_bytes(n_tok, slot_cap)


def sf_embed_grad(tokens, dY, mask: Mask, G, ws, status=None, stream=None):
    n_tok, H = dY.shape
    m = mask.struct()
    _check(load().sf_embed_grad(_ptr(tokens), n_tok, _ptr(dY), H, dY.stride(0), ctypes.byref(m), _ptr(G),
                                G.stride(0), _ptr(ws), ws.numel() * ws.element_size(), _ptr(status),
                                _stream(stream)), "sf_embed_grad")


def sf_embed_grad_noalloc(tokens, dY, mask: Mask, G, status=None, stream=None):
    """sf_embed_grad without a scratch buffer: the library's fixed per-GPU scratch is used, for
    callers that must not allocate device memory. Calls on one GPU must not overlap."""
    n_tok, H = dY.shape
    m = mask.struct()
    _check(load().sf_embed_grad_noalloc(_ptr(tokens), n_tok, _ptr(dY), H, dY.stride(0), ctypes.byref(m),
                                        _ptr(G), G.stride(0), _ptr(status), _stream(stream)),
           "sf_embed_grad_noalloc")


def sf_adam_tables(beta1: float, beta2: float, t_max: int, bc1, bc2, stream=None):
    _check(load().sf_adam_tables(beta1, beta2, t_max, _ptr(bc1), _ptr(bc2), _stream(stream)),
           "sf_adam_tables")


class AdamParams:
    """Adam hyper-parameters plus the device bias-correction tables."""

    def __init__(self, lr=1e-4, beta1=0.9, beta2=0.999, eps=1e-8, wd=0.0, clip=0.0, t_max=20000,
                 device="cuda", stream=None):
        import numpy as np
        self.lr, self.beta1, self.beta2, self.eps, self.wd, self.clip = lr, beta1, beta2, eps, wd, clip
        self.one_minus_b1 = float(np.float32(1.0) - np.float32(beta1))
        self.one_minus_b2 = float(np.float32(1.0) - np.float32(beta2))
        self.t_max = t_max
        self.bc1 = torch.empty(t_max + 1, dtype=torch.float32, device=device)
        self.bc2 = torch.empty(t_max + 1, dtype=torch.float32, device=device)
        sf_adam_tables(beta1, beta2, t_max, self.bc1, self.bc2, stream)

    def struct(self) -> sf_adam:
        return sf_adam(self.lr, self.beta1, self.beta2, self.eps, self.one_minus_b1, self.one_minus_b2,
                       self.wd, self.clip, _ptr(self.bc1), _ptr(self.bc2), self.t_max)


def matrix_struct(mat: Matrix, partner: int = -1, c_self: float = 1.0, c_partner: float = 0.0) -> sf_matrix:
    return sf_matrix(mat.C, partner, c_self, c_partner, mat.mask.struct(), _ptr(mat.q), _ptr(mat.s),
                     _ptr(mat.delta), _ptr(mat.m), _ptr(mat.v), _ptr(mat.grad), _ptr(mat.live))


def sf_sparse_update(mats, hp: AdamParams, status=None, stream=None):
    """mats: list of sf_matrix (see matrix_struct); partner indices refer to this list."""
    n = len(mats)
    arr = (sf_matrix * n)(*mats)
    h = hp.struct()
    _check(load().sf_sparse_update(arr, n, ctypes.byref(h), _ptr(status), _stream(stream)),
           "sf_sparse_update")


def sf_quantize_init(W, mat: Matrix, stream=None):
    R, C = W.shape
    assert W.dtype == torch.float32 and W.is_contiguous() and (R, C) == (mat.R, mat.C)
    _check(load().sf_quantize_init(_ptr(W), R, C, _ptr(mat.q), _ptr(mat.s), _ptr(mat.delta),
                                   _ptr(mat.live), _stream(stream)), "sf_quantize_init")


def sf_version() -> int:
    return load().sf_version()


class Checkpoint:
    """Device buffers of an active-row checkpoint of one matrix (section 2.6)."""

    def __init__(self, cap: int, C: int, device="cuda"):
        self.cap, self.C = cap, C
        n = max(cap, 1)
        self.count = torch.zeros(1, dtype=torch.int32, device=device)
        self.rows = torch.zeros(n, dtype=torch.int32, device=device)
        self.q = torch.zeros((n, C), dtype=torch.int8, device=device)
        self.s = torch.zeros(n, dtype=torch.float32, device=device)
        self.delta = torch.zeros((n, C), dtype=torch.float32, device=device)
        self.m = torch.zeros((n, C), dtype=torch.int16, device=device)
        self.v = torch.zeros((n, C), dtype=torch.int16, device=device)
        self.step = torch.zeros(n, dtype=torch.int32, device=device)

    def struct(self) -> sf_checkpoint:
        return sf_checkpoint(self.cap, _ptr(self.count), _ptr(self.rows), _ptr(self.q), _ptr(self.s),
                             _ptr(self.delta), _ptr(self.m), _ptr(self.v), _ptr(self.step))


def _ckpt_call(name, mats, ckpts, status, stream):
    n = len(mats)
    arr = (sf_matrix * n)(*mats)
    carr = (sf_checkpoint * n)(*[c.struct() for c in ckpts])
    _check(getattr(load(), name)(arr, carr, n, _ptr(status), _stream(stream)), name)


def sf_checkpoint_save(mats, ckpts, status=None, stream=None):
    """mats: list of sf_matrix (matrix_struct); ckpts: list of Checkpoint, same order."""
    _ckpt_call("sf_checkpoint_save", mats, ckpts, status, stream)


def sf_checkpoint_restore(mats, ckpts, status=None, stream=None):
    _ckpt_call("sf_checkpoint_restore", mats, ckpts, status, stream)


# ---------------------------------------------------------------------------------------------
# Dense tensors: AdamW and the global gradient norm
# ---------------------------------------------------------------------------------------------

_TYPE_OF = {torch.float32: SF_TYPE_F32, torch.bfloat16: SF_TYPE_BF16, torch.float16: SF_TYPE_F16,
            torch.float8_e4m3fn: SF_TYPE_E4M3, torch.uint8: SF_TYPE_E4M3}


def _type(t, allowed, what) -> int:
    k = _TYPE_OF.get(t.dtype)
    if k not in allowed:
        raise ValueError(f"{what}: {t.dtype} is not supported")
    return k


def _one_device(*tensors) -> int:
    """The index of the GPU that all the given tensors (None and addresses among them) are on."""
    index = -1
    for t in tensors:
        if t is None or isinstance(t, int):
            continue
        d = t.get_device()
        if d < 0 or (index >= 0 and d != index):
            raise ValueError("device tensors on one GPU expected")
        index = d
    if index < 0:
        raise ValueError("device tensors on one GPU expected")
    return index


def _status_ptr(status) -> int | None:
    """A status word's address: a device tensor's, or the address itself, as Pipeline and Trainer pass it on."""
    return status if isinstance(status, int) else _ptr(status)


def _on_current(index: int):
    if torch.cuda.current_device() != index:
        raise ValueError(f"the tensors are on cuda:{index}, which is not the current device")


_raw_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_on(index: int, stream) -> int | None:
    """_stream() for GPU `index`; looking up the current stream's handle without its Python object takes 0.1 us, not 3."""
    if stream is None and _raw_current_stream is not None:
        return _raw_current_stream(index) or None
    return _stream(stream)


def dense_tensor(p, g, m, v, live=None, decay: float = 1.0, m_scale=None, v_scale=None) -> Desc:
    """One tensor of an AdamW step. p fp32 or bf16; g fp32, bf16 or fp16; m, v fp32, or e4m3 codes
    (float8_e4m3fn or uint8) with one fp32 scale per SF_DENSE_BLOCK elements; live (optional) bf16,
    written with the stepped weights (bf16 weights may be their own); decay multiplies the step's
    weight decay (0: none). All contiguous, of one length."""
    n = p.numel()
    for t in (p, g, m, v, live):
        if t is not None and (t.numel() != n or not t.is_contiguous()):
            raise ValueError("p, g, m, v and live must be contiguous and of one length")
    pt = _type(p, (SF_TYPE_F32, SF_TYPE_BF16), "p")
    gt = _type(g, (SF_TYPE_F32, SF_TYPE_BF16, SF_TYPE_F16), "g")
    st = _type(m, (SF_TYPE_F32, SF_TYPE_E4M3), "m")
    if m.dtype != v.dtype:
        raise ValueError("m and v must have one type")
    if live is not None and live.dtype not in (torch.bfloat16, torch.int16):
        raise ValueError("live must hold bf16")
    if live is not None and pt == SF_TYPE_BF16 and live.data_ptr() == p.data_ptr():
        live = None                                      # bf16 weights are their own live copy
    if st == SF_TYPE_E4M3:
        blocks = -(-n // SF_DENSE_BLOCK)
        for s in (m_scale, v_scale):
            if s is None or s.dtype != torch.float32 or s.numel() != blocks or not s.is_contiguous():
                raise ValueError(f"8-bit moments need {blocks} fp32 scales each")
    elif m_scale is not None or v_scale is not None:
        raise ValueError("fp32 moments take no scales")
    refs = (p, g, m, v, live, m_scale, v_scale)
    _one_device(*refs)
    return Desc(sf_dense(n, _ptr(p), _ptr(g), _ptr(m), _ptr(v), _ptr(m_scale), _ptr(v_scale), _ptr(live), decay,
                         pt, gt, st), *refs)


class Dense:
    """A dense tensor's AdamW state: zero moments (fp32, or 8 bits with their scales) for weights p
    and gradient g, and optionally a bf16 live copy of p."""

    def __init__(self, p, g, state: int = SF_TYPE_F32, live: bool = False, decay: float = 1.0):
        if state not in (SF_TYPE_F32, SF_TYPE_E4M3):
            raise ValueError("moments are SF_TYPE_F32 or SF_TYPE_E4M3")
        self.p, self.g, self.decay = p, g, decay
        self.m_scale = self.v_scale = None
        if state == SF_TYPE_E4M3:
            blocks = -(-p.numel() // SF_DENSE_BLOCK)
            self.m_scale = torch.zeros(blocks, dtype=torch.float32, device=p.device)
            self.v_scale = torch.zeros(blocks, dtype=torch.float32, device=p.device)
        dt = torch.float32 if state == SF_TYPE_F32 else torch.float8_e4m3fn
        self.m = torch.zeros(p.shape, dtype=dt, device=p.device)
        self.v = torch.zeros(p.shape, dtype=dt, device=p.device)
        self.live = p.to(torch.bfloat16) if live else None

    def desc(self) -> Desc:
        return dense_tensor(self.p, self.g, self.m, self.v, self.live, self.decay, self.m_scale, self.v_scale)


class DenseTensors:
    """The argument array of a list of dense_tensor() descriptors, built once for many steps. It holds the tensors' addresses:
    gradients are to be written in place (zeroed, not dropped and made anew) from step to step."""

    def __init__(self, tensors):
        self.descs = [t.desc() if isinstance(t, Dense) else t for t in tensors]
        self.n = len(self.descs)
        self.arr = (sf_dense * max(self.n, 1))(*[d.c for d in self.descs])
        self.anchor = self.descs[0].refs[0] if self.n else None
        if self.n:
            _one_device(*[t for d in self.descs for t in d.refs])
        spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), k != 1)
                       for d in self.descs for k, t in enumerate(d.refs) if t is not None and t.numel())
        written_to = read_to = 0                         # ends of what the step writes and reads, from the lowest address up
        for start, end, written in spans:
            if start < written_to or (written and start < read_to):
                raise ValueError("a tensor is in the list twice, or shares its weights or state with another, or with a gradient")
            if written:
                written_to = max(written_to, end)
            else:
                read_to = max(read_to, end)


def step_words(device=None) -> torch.Tensor:
    """The device step count of sf_adamw_step: [steps taken, 0]."""
    return torch.zeros(2, dtype=torch.int32, device=device or "cuda")


def grad_norm_workspace(tensors: DenseTensors, device="cuda") -> torch.Tensor:
    """Zeroed scratch for sf_grad_norm over these tensors."""
    return torch.zeros(load().sf_grad_norm_ws_bytes(tensors.arr, tensors.n), dtype=torch.uint8, device=device)


def _check_words(name, t, dtype):
    if t.dtype != dtype or t.numel() < 2 or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous tensor of two {dtype} expected")


def sf_grad_norm(tensors: DenseTensors, out, ws, max_norm: float = 0.0, inv_scale: float = 1.0, status=None,
                 stream=None):
    """out (two floats): the gradients' global norm and the factor that clips it, for sf_adamw_step."""
    _check_words("out", out, torch.float32)
    index = _one_device(tensors.anchor, out, ws, status)
    _on_current(index)
    _check(load().sf_grad_norm(tensors.arr, tensors.n, inv_scale, max_norm, _ptr(out), _ptr(ws),
                               ws.numel() * ws.element_size(), _status_ptr(status), _stream_on(index, stream)), "sf_grad_norm")


def sf_adamw_step(tensors: DenseTensors, hp: AdamParams, step, factor=None, status=None, stream=None):
    """One AdamW step of every tensor; step: step_words(), factor: sf_grad_norm's output or None."""
    _check_words("step", step, torch.int32)
    if factor is not None:
        _check_words("factor", factor, torch.float32)
    index = _one_device(tensors.anchor, step, factor, status, hp.bc1)
    _on_current(index)
    h = hp.struct()
    _check(load().sf_adamw_step(tensors.arr, tensors.n, ctypes.byref(h), _ptr(step), _ptr(factor), _status_ptr(status),
                                _stream_on(index, stream)), "sf_adamw_step")


# ---------------------------------------------------------------------------------------------
# Products grouped by expert
# ---------------------------------------------------------------------------------------------

def grouped_problem(A, W, Y, offsets) -> Desc:
    """The operands of sf_grouped_forward (writes Y), sf_grouped_dx (writes A) or sf_grouped_dw (writes W).

    A [T x C] and Y [T x R] bf16 or fp16, rows sorted by expert; W [E x R x C] of the same type (fp32 or
    that type for the weight gradient); offsets int32 [E + 1] on the device: expert e owns rows
    offsets[e] .. offsets[e+1]-1. Rows may be strided, columns not."""
    if A.dim() != 2 or Y.dim() != 2 or W.dim() != 3:
        raise ValueError("A [T x C], W [E x R x C] and Y [T x R] expected")
    (T, C), (E, R) = A.shape, W.shape[:2]
    if W.shape[2] != C or tuple(Y.shape) != (T, R):
        raise ValueError(f"shapes do not match: A {tuple(A.shape)}, W {tuple(W.shape)}, Y {tuple(Y.shape)}")
    if E >= 2 ** 31 or max(T, R, C) > 2 ** 30:
        raise ValueError("sizes are 32-bit: at most 2^30 tokens, rows and columns")
    for name, t in (("A", A), ("W", W), ("Y", Y)):
        if t.numel() and t.stride(-1) != 1:
            raise ValueError(f"{name}: columns must be contiguous")
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or offsets.numel() != E + 1 or not offsets.is_contiguous():
        raise ValueError(f"offsets: {E + 1} contiguous int32 expected")
    ty = _type(A, (SF_TYPE_BF16, SF_TYPE_F16), "A")
    wt = _type(W, (ty, SF_TYPE_F32), "W")
    _type(Y, (ty,), "Y")
    _one_device(A, W, Y, offsets)
    # a single row's or matrix's stride says nothing: give the dense one
    ld_a = A.stride(0) if T > 1 else C
    ld_y = Y.stride(0) if T > 1 else R
    ld_w = W.stride(1) if R > 1 else C
    stride_w = W.stride(0) if E > 1 else R * ld_w
    c = sf_grouped(_ptr(A) or None, ld_a, _ptr(W), ld_w, stride_w, _ptr(Y) or None, ld_y, _ptr(offsets), E, T, R, C,
                   ty, wt)
    return Desc(c, A, W, Y, offsets)


def _grouped(name, p: Desc, status, stream, *extra):
    index = _one_device(p.refs[1], status)
    _on_current(index)
    _check(getattr(load(), name)(ctypes.byref(p.c), *extra, _status_ptr(status), _stream_on(index, stream)), name)


def sf_grouped_forward(p: Desc, status=None, stream=None):
    """Y[t] = W[e(t)] A[t] for every expert's rows."""
    _grouped("sf_grouped_forward", p, status, stream)


def sf_grouped_dx(p: Desc, status=None, stream=None):
    """A[t] = W[e(t)]^T Y[t]: the input gradient, with Y the gradient of the outputs."""
    _grouped("sf_grouped_dx", p, status, stream)


def sf_grouped_dw(p: Desc, status=None, stream=None, accumulate: bool = False):
    """W[e] = sum over e's tokens of Y[t] A[t]^T: the weight gradient, with Y the gradient of the outputs;
    accumulate adds it to what W (fp32) holds."""
    _grouped("sf_grouped_dw", p, status, stream, int(accumulate))


def sf_grouped_kernel(p: Desc, product: int, accumulate: bool = False) -> int:
    """Which kernel (SF_GROUPED_SINGLE ..) the call takes on the current device: for tests and measurements."""
    _on_current(_one_device(p.refs[1]))
    k = load().sf_grouped_kernel(ctypes.byref(p.c), product, int(accumulate))
    if k < 0:
        _check(k, "sf_grouped_kernel")
    return k
