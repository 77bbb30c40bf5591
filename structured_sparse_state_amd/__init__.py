"""Flash PD-SSM recurrence scan for AMD MI355X (gfx950).

The compute path is the C-ABI library ``libpdssm.so`` (hand-written HIP
kernels, declared in ``include/pdssm.h``).  This module is a thin ctypes
binding with the same function names: it only turns torch tensors into
device pointers and the current HIP stream into a ``hipStream_t``.  Every
step runs in the library's kernels; there is no fallback, and a missing
library raises.

Higher-level helpers allocate outputs (and workspaces) with torch and call
the C entry points: ``scan`` and ``scan_save`` (forward), ``scan_bwd``
(gradients), ``router_select`` (router scores and their argmax) with
``router_pack_weights`` (the weights in the faster kernel's layout),
``dict_hardmax`` (index maps from dense matrices), ``decode_step`` (one
recurrent step), ``select`` and ``compose`` (test exports).

Beside the scan (``include/pdssm_layers.h``): the gated delta rule,
``delta_rule`` (whole sequences), ``delta_rule_bwd`` (gradients) and
``delta_step`` (one step), and the norm of queries and keys with the rotation
by position, ``qk_norm_rope`` and ``qk_norm_rope_bwd``.

For a layer's block (``include/pdssm_block.h``): linear attention with decays,
``linear_attention``, ``linear_attention_bwd`` and ``linear_attention_step``;
the layer norm of a residual and a dropped-out branch, ``layer_norm`` and
``layer_norm_bwd``; and ``dropout``.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import re
from typing import NamedTuple, Optional

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(HERE, "libpdssm.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "pdssm.h")
LAYERS_HEADER = os.path.join(os.path.dirname(HERE), "include", "pdssm_layers.h")
BLOCK_HEADER = os.path.join(os.path.dirname(HERE), "include", "pdssm_block.h")

# Flag and status values of include/pdssm.h (tests check they agree).
PDSSM_SEL_I32 = 0x0
PDSSM_SEL_I16 = 0x1
PDSSM_LOGITS_F32 = 0x2
PDSSM_LOGITS_BF16 = 0x3
PDSSM_SEL_MASK = 0x3
PDSSM_COMPLEX = 0x4
PDSSM_BC_BF16 = 0x8
PDSSM_Y_BF16 = 0x10
PDSSM_DETERMINISTIC = 0x20
PDSSM_FLAGS_ALL = 0x3F
PDSSM_ROUTER_W_PACKED = 0x1

# Flags of include/pdssm_layers.h.
PDSSM_DATA_BF16 = 0x1
PDSSM_NORM_L2 = 0x2
PDSSM_ROPE_PAIRS = 0x4

# Flags of include/pdssm_block.h.
PDSSM_NO_DG = 0x2
PDSSM_DG_HEADS = 0x4

PDSSM_OK = 0
PDSSM_ERR_NULL = -1
PDSSM_ERR_DIM = -2
PDSSM_ERR_FLAGS = -3
PDSSM_ERR_ALIGN = -4
PDSSM_ERR_WORKSPACE = -5
PDSSM_ERR_HIP = -6
PDSSM_ERR_SCRATCH = -7

SEL_FLAG = {"sel_i32": PDSSM_SEL_I32, "sel_i16": PDSSM_SEL_I16,
            "logits_f32": PDSSM_LOGITS_F32, "logits_bf16": PDSSM_LOGITS_BF16}

_LIB = None


class PdssmError(RuntimeError):
    def __init__(self, status: int, text: str):
        super().__init__(f"pdssm status {status}: {text}")
        self.status = status


def _load(path: str) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with __graft_entry__.build() "
                           "(hipcc --offload-arch=gfx950); there is no fallback path")
    lib = ctypes.CDLL(path)
    P, I64, I32, U32, SZ = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32,
                            ctypes.c_size_t)
    lib.pdssm_scan_fwd.argtypes = [P, P, P, P, P, P, P, I64, I64, I64, I32, I32, U32, P, P, SZ, P]
    lib.pdssm_scan_fwd.restype = ctypes.c_int
    lib.pdssm_scan_fwd_noalloc.argtypes = [P, P, P, P, P, P, P, I64, I64, I64, I32, I32, U32, P, P]
    lib.pdssm_scan_fwd_noalloc.restype = ctypes.c_int
    lib.pdssm_scan_workspace_bytes.argtypes = [I64, I64, I64, I32, I32, U32]
    lib.pdssm_scan_workspace_bytes.restype = SZ
    lib.pdssm_select.argtypes = [P, P, I64, I64, I64, I32, U32, P]
    lib.pdssm_select.restype = ctypes.c_int
    lib.pdssm_compose.argtypes = [P, P, P, P, P, I64, I64, I64, I32, I32, U32, P, SZ, P]
    lib.pdssm_compose.restype = ctypes.c_int
    lib.pdssm_scan_fwd_save.argtypes = [P, P, P, P, P, P, P, P, P, I64, I64, I64, I32, I32, U32, P,
                                        P, SZ, P]
    lib.pdssm_scan_fwd_save.restype = ctypes.c_int
    lib.pdssm_scan_bwd.argtypes = [P, P, P, P, P, P, P, P, P, P, P, P, I64, I64, I64, I32, I32, U32,
                                   P, SZ, P]
    lib.pdssm_scan_bwd.restype = ctypes.c_int
    lib.pdssm_scan_bwd_workspace_bytes.argtypes = [I64, I64, I64, I32, I32, U32]
    lib.pdssm_scan_bwd_workspace_bytes.restype = SZ
    lib.pdssm_strerror.argtypes = [ctypes.c_int]
    lib.pdssm_strerror.restype = ctypes.c_char_p
    lib.pdssm_dict_hardmax.argtypes = [P, P, I64, I32, I32, U32, P]
    lib.pdssm_dict_hardmax.restype = ctypes.c_int
    lib.pdssm_decode_step.argtypes = [P, P, P, P, P, P, P, I64, I64, I32, I32, U32, P]
    lib.pdssm_decode_step.restype = ctypes.c_int
    lib.pdssm_router_select.argtypes = [P, P, P, I64, I64, I64, I32, I32, U32, P]
    lib.pdssm_router_select.restype = ctypes.c_int
    lib.pdssm_router_pack_weights.argtypes = [P, P, I64, I32, I32, P]
    lib.pdssm_router_pack_weights.restype = ctypes.c_int
    if path == LIBRARY:   # the test builds hold the scan alone
        F = ctypes.c_float
        lib.pdssm_delta_fwd.argtypes = [P] * 8 + [I64] * 4 + [I32, I32, F, U32, P, P, SZ, P]
        lib.pdssm_delta_fwd.restype = ctypes.c_int
        lib.pdssm_delta_bwd.argtypes = [P] * 14 + [I64] * 4 + [I32, I32, F, U32, P, P, SZ, P]
        lib.pdssm_delta_bwd.restype = ctypes.c_int
        lib.pdssm_delta_step.argtypes = [P] * 8 + [I64] * 3 + [I32, I32, F, U32, P, P]
        lib.pdssm_delta_step.restype = ctypes.c_int
        for size in (lib.pdssm_delta_workspace_bytes, lib.pdssm_delta_bwd_workspace_bytes):
            size.argtypes = [I64] * 4 + [I32, I32, U32]
            size.restype = SZ
        lib.pdssm_qk_norm_rope_fwd.argtypes = [P] * 9 + [I64] * 4 + [I32, I32, I64, F, U32, P, P]
        lib.pdssm_qk_norm_rope_fwd.restype = ctypes.c_int
        lib.pdssm_qk_norm_rope_bwd.argtypes = [P] * 13 + [I64] * 4 + [I32, I32, I64, F, U32, P, P, SZ, P]
        lib.pdssm_qk_norm_rope_bwd.restype = ctypes.c_int
        lib.pdssm_qk_norm_rope_bwd_workspace_bytes.argtypes = [I64] * 4 + [I32]
        lib.pdssm_qk_norm_rope_bwd_workspace_bytes.restype = SZ
        lib.pdssm_linear_fwd.argtypes = [P] * 7 + [I64] * 4 + [I32, I32, F, U32, P, P, SZ, P]
        lib.pdssm_linear_fwd.restype = ctypes.c_int
        lib.pdssm_linear_bwd.argtypes = [P] * 12 + [I64] * 4 + [I32, I32, F, U32, P, P, SZ, P]
        lib.pdssm_linear_bwd.restype = ctypes.c_int
        lib.pdssm_linear_step.argtypes = [P] * 7 + [I64] * 3 + [I32, I32, F, U32, P, P]
        lib.pdssm_linear_step.restype = ctypes.c_int
        for size in (lib.pdssm_linear_workspace_bytes, lib.pdssm_linear_bwd_workspace_bytes):
            size.argtypes = [I64] * 4 + [I32, I32, U32]
            size.restype = SZ
        U64, DB = ctypes.c_uint64, ctypes.c_double
        lib.pdssm_layer_norm_fwd.argtypes = [P] * 6 + [I64] * 3 + [I32, F, DB, U64, U64, P, U32, P, P]
        lib.pdssm_layer_norm_fwd.restype = ctypes.c_int
        lib.pdssm_layer_norm_bwd.argtypes = [P] * 8 + [I64] * 3 + [I32, F, DB, U64, U64, P, U32, P, P, SZ, P]
        lib.pdssm_layer_norm_bwd.restype = ctypes.c_int
        lib.pdssm_layer_norm_bwd_workspace_bytes.argtypes = [I64] * 3 + [I32]
        lib.pdssm_layer_norm_bwd_workspace_bytes.restype = SZ
        lib.pdssm_dropout.argtypes = [P] * 3 + [I64] * 3 + [I32, DB, U64, U64, P, U32, P, P]
        lib.pdssm_dropout.restype = ctypes.c_int
    return lib


def library() -> ctypes.CDLL:
    """The loaded HIP library (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        _LIB = _load(LIBRARY)
    return _LIB


_VARIANTS = {}


@contextlib.contextmanager
def variant(name: str):
    """Route every call in the block through the test build ``name`` of the
    library (``libpdssm_<name>.so``, see build_lib.VARIANTS)."""
    global _LIB
    if name not in _VARIANTS:
        _VARIANTS[name] = _load(os.path.join(HERE, f"libpdssm_{name}.so"))
    saved = library()
    _LIB = _VARIANTS[name]
    try:
        yield _LIB
    finally:
        _LIB = saved


def header_functions(header: str = HEADER) -> list:
    """Names of the functions a header (include/pdssm.h by default) declares."""
    text = open(header).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.findall(r"\b(pdssm_[a-z_]+)\s*\(", text)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ---------------------------------------------------------------------------
# The C entry points, same names and argument order.  Tensors (or raw
# addresses) in, status code out.
# ---------------------------------------------------------------------------

def pdssm_scan_fwd(sel_or_logits, dict_idx, diag, b, c, y, x_final, B, H, L, N, K, flags, x0,
                   workspace, workspace_bytes, stream=None) -> int:
    return library().pdssm_scan_fwd(_ptr(sel_or_logits), _ptr(dict_idx), _ptr(diag), _ptr(b),
                                    _ptr(c), _ptr(y), _ptr(x_final), B, H, L, N, K, flags,
                                    _ptr(x0), _ptr(workspace), workspace_bytes, _stream(stream))


def pdssm_scan_fwd_noalloc(sel_or_logits, dict_idx, diag, b, c, y, x_final, B, H, L, N, K, flags,
                           x0, stream=None) -> int:
    return library().pdssm_scan_fwd_noalloc(_ptr(sel_or_logits), _ptr(dict_idx), _ptr(diag), _ptr(b),
                                            _ptr(c), _ptr(y), _ptr(x_final), B, H, L, N, K, flags,
                                            _ptr(x0), _stream(stream))


def pdssm_scan_workspace_bytes(B, H, L, N, K, flags) -> int:
    return library().pdssm_scan_workspace_bytes(B, H, L, N, K, flags)


def pdssm_scan_fwd_save(sel_or_logits, dict_idx, diag, b, c, y, x_final, x_chunks, sel_out, B, H,
                        L, N, K, flags, x0, workspace, workspace_bytes, stream=None) -> int:
    return library().pdssm_scan_fwd_save(_ptr(sel_or_logits), _ptr(dict_idx), _ptr(diag), _ptr(b),
                                         _ptr(c), _ptr(y), _ptr(x_final), _ptr(x_chunks),
                                         _ptr(sel_out), B, H, L, N, K, flags, _ptr(x0),
                                         _ptr(workspace), workspace_bytes, _stream(stream))


def pdssm_scan_bwd(sel_or_logits, dict_idx, diag, b, c, x_chunks, gy, gx_final, gb, gc, gd, gx0, B,
                   H, L, N, K, flags, workspace, workspace_bytes, stream=None) -> int:
    return library().pdssm_scan_bwd(_ptr(sel_or_logits), _ptr(dict_idx), _ptr(diag), _ptr(b),
                                    _ptr(c), _ptr(x_chunks), _ptr(gy), _ptr(gx_final), _ptr(gb),
                                    _ptr(gc), _ptr(gd), _ptr(gx0), B, H, L, N, K, flags,
                                    _ptr(workspace), workspace_bytes, _stream(stream))


def pdssm_scan_bwd_workspace_bytes(B, H, L, N, K, flags) -> int:
    return library().pdssm_scan_bwd_workspace_bytes(B, H, L, N, K, flags)


def pdssm_select(sel_or_logits, sel_out, B, H, L, K, flags, stream=None) -> int:
    return library().pdssm_select(_ptr(sel_or_logits), _ptr(sel_out), B, H, L, K, flags,
                                  _stream(stream))


def pdssm_compose(sel_or_logits, dict_idx, diag, pi_out, d_out, B, H, L, N, K, flags, workspace,
                  workspace_bytes, stream=None) -> int:
    return library().pdssm_compose(_ptr(sel_or_logits), _ptr(dict_idx), _ptr(diag), _ptr(pi_out),
                                   _ptr(d_out), B, H, L, N, K, flags, _ptr(workspace),
                                   workspace_bytes, _stream(stream))


def pdssm_dict_hardmax(m, dict_idx, H, K, N, flags, stream=None) -> int:
    return library().pdssm_dict_hardmax(_ptr(m), _ptr(dict_idx), H, K, N, flags, _stream(stream))


def pdssm_decode_step(sel_or_logits, dict_idx, diag, b, c, y, x, B, H, N, K, flags,
                      stream=None) -> int:
    return library().pdssm_decode_step(_ptr(sel_or_logits), _ptr(dict_idx), _ptr(diag), _ptr(b),
                                       _ptr(c), _ptr(y), _ptr(x), B, H, N, K, flags,
                                       _stream(stream))


def pdssm_router_select(u, w, sel_out, B, L, H, K, D, flags, stream=None) -> int:
    return library().pdssm_router_select(_ptr(u), _ptr(w), _ptr(sel_out), B, L, H, K, D, flags,
                                         _stream(stream))


def pdssm_router_pack_weights(w, w_packed, H, K, D, stream=None) -> int:
    return library().pdssm_router_pack_weights(_ptr(w), _ptr(w_packed), H, K, D, _stream(stream))


def pdssm_strerror(status: int) -> str:
    return library().pdssm_strerror(status).decode()


def check(status: int) -> None:
    if status != PDSSM_OK:
        raise PdssmError(status, pdssm_strerror(status))


# ---------------------------------------------------------------------------
# Convenience layer over ScanInputs-like objects (fields: sel_mode,
# sel_or_logits, dict_idx, diag, b, c, x0, complex, bc_bf16, y_bf16, B, H,
# L, N, K), all tensors on the GPU.
# ---------------------------------------------------------------------------

def flags_of(inp, deterministic: bool = False) -> int:
    f = SEL_FLAG[inp.sel_mode]
    if deterministic:
        f |= PDSSM_DETERMINISTIC
    if inp.complex:
        f |= PDSSM_COMPLEX
    if inp.bc_bf16:
        f |= PDSSM_BC_BF16
    if inp.y_bf16:
        f |= PDSSM_Y_BF16
    return f


def workspace_for(inp, device=None) -> torch.Tensor:
    n = pdssm_scan_workspace_bytes(inp.B, inp.H, inp.L, inp.N, inp.K, flags_of(inp))
    if n == 0:
        raise PdssmError(PDSSM_ERR_DIM, "invalid sizes")
    return torch.empty(n, dtype=torch.uint8, device=device or inp.diag.device)


def scan(inp, *, workspace: Optional[torch.Tensor] = None, want_x_final: bool = True,
         y: Optional[torch.Tensor] = None, x_final: Optional[torch.Tensor] = None, stream=None,
         x0="from_inputs", deterministic: bool = False):
    """Run pdssm_scan_fwd on a batch; returns (y, x_final or None).
    ``deterministic`` sets PDSSM_DETERMINISTIC (bitwise reproducible)."""
    dev = inp.diag.device
    if y is None:
        y = torch.empty((inp.B, inp.H, inp.L), device=dev,
                        dtype=torch.bfloat16 if inp.y_bf16 else torch.float32)
    if want_x_final and x_final is None:
        shape = (inp.B, inp.H, inp.N, 2) if inp.complex else (inp.B, inp.H, inp.N)
        x_final = torch.empty(shape, device=dev, dtype=torch.float32)
    if workspace is None:
        workspace = workspace_for(inp)
    x0t = inp.x0 if isinstance(x0, str) else x0
    check(pdssm_scan_fwd(inp.sel_or_logits, inp.dict_idx, inp.diag, inp.b, inp.c, y,
                         x_final if want_x_final else None, inp.B, inp.H, inp.L, inp.N, inp.K,
                         flags_of(inp, deterministic), x0t, workspace, workspace.numel(), stream))
    return y, (x_final if want_x_final else None)


def scan_noalloc(inp, *, y: Optional[torch.Tensor] = None, x_final: Optional[torch.Tensor] = None,
                 stream=None, deterministic: bool = False):
    """pdssm_scan_fwd_noalloc on a batch (the library's own device scratch in
    place of a workspace); returns (y, x_final).  Output tensors passed in are
    written in place, so the call itself allocates nothing."""
    dev = inp.diag.device
    if y is None:
        y = torch.empty((inp.B, inp.H, inp.L), device=dev,
                        dtype=torch.bfloat16 if inp.y_bf16 else torch.float32)
    if x_final is None:
        shape = (inp.B, inp.H, inp.N, 2) if inp.complex else (inp.B, inp.H, inp.N)
        x_final = torch.empty(shape, device=dev, dtype=torch.float32)
    check(pdssm_scan_fwd_noalloc(inp.sel_or_logits, inp.dict_idx, inp.diag, inp.b, inp.c, y, x_final,
                                 inp.B, inp.H, inp.L, inp.N, inp.K, flags_of(inp, deterministic), inp.x0,
                                 stream))
    return y, x_final


CARRY_STRIDE = 16   # steps per saved chunk carry (include/pdssm.h)


def scan_save(inp, *, workspace: Optional[torch.Tensor] = None, stream=None, want_sel: bool = False,
              deterministic: bool = False):
    """pdssm_scan_fwd_save on a batch: (y, x_final, x_chunks), plus the int16
    selections [B,H,L] when want_sel."""
    dev = inp.diag.device
    y = torch.empty((inp.B, inp.H, inp.L), device=dev,
                    dtype=torch.bfloat16 if inp.y_bf16 else torch.float32)
    tail = (inp.N, 2) if inp.complex else (inp.N,)
    x_final = torch.empty((inp.B, inp.H) + tail, device=dev, dtype=torch.float32)
    nch = (inp.L + CARRY_STRIDE - 1) // CARRY_STRIDE
    x_chunks = torch.empty((inp.B, inp.H, nch) + tail, device=dev, dtype=torch.float32)
    if workspace is None:
        workspace = workspace_for(inp)
    sel = torch.empty((inp.B, inp.H, inp.L), device=dev, dtype=torch.int16) if want_sel else None
    check(pdssm_scan_fwd_save(inp.sel_or_logits, inp.dict_idx, inp.diag, inp.b, inp.c, y, x_final,
                              x_chunks, sel, inp.B, inp.H, inp.L, inp.N, inp.K,
                              flags_of(inp, deterministic), inp.x0,
                              workspace, workspace.numel(), stream))
    if want_sel:
        return y, x_final, x_chunks, sel
    return y, x_final, x_chunks


def bwd_workspace_for(inp, device=None) -> torch.Tensor:
    n = pdssm_scan_bwd_workspace_bytes(inp.B, inp.H, inp.L, inp.N, inp.K, flags_of(inp))
    if n == 0:
        raise PdssmError(PDSSM_ERR_DIM, "invalid sizes")
    return torch.empty(n, dtype=torch.uint8, device=device or inp.diag.device)


def scan_bwd(inp, x_chunks, gy, gx_final=None, *, want_gx0: bool = True,
             workspace: Optional[torch.Tensor] = None, stream=None, out=None, sel=None,
             deterministic: bool = False):
    """pdssm_scan_bwd on a batch: (gb, gc, gd, gx0 or None), in the storage
    of b, c, diag and x0.  ``sel``: the forward's saved int16 selections
    (scan_save(want_sel=True)), used in place of the inputs' scores.  ``out``
    may hold a previous call's result tuple to write into instead of
    allocating."""
    dev = inp.diag.device
    if out is not None:
        gb, gc, gd, gx0 = out
    else:
        gb = torch.empty_like(inp.b)
        gc = torch.empty_like(inp.c)
        gd = torch.empty_like(inp.diag)
        tail = (inp.N, 2) if inp.complex else (inp.N,)
        gx0 = torch.empty((inp.B, inp.H) + tail, device=dev, dtype=torch.float32) if want_gx0 else None
    if workspace is None:
        workspace = bwd_workspace_for(inp)
    flags = flags_of(inp, deterministic)
    if sel is not None:
        flags = (flags & ~PDSSM_SEL_MASK) | PDSSM_SEL_I16
    check(pdssm_scan_bwd(inp.sel_or_logits if sel is None else sel, inp.dict_idx, inp.diag, inp.b,
                         inp.c, x_chunks, gy, gx_final, gb, gc, gd, gx0, inp.B, inp.H, inp.L, inp.N,
                         inp.K, flags,
                         workspace, workspace.numel(), stream))
    return gb, gc, gd, gx0


def select(sel_or_logits, sel_mode: str, K: int, stream=None) -> torch.Tensor:
    shape = sel_or_logits.shape if sel_mode.startswith("sel") else sel_or_logits.shape[:-1]
    B, H, L = shape
    out = torch.empty((B, H, L), dtype=torch.int32, device=sel_or_logits.device)
    check(pdssm_select(sel_or_logits, out, B, H, L, K, SEL_FLAG[sel_mode], stream))
    return out


def compose(inp, workspace: Optional[torch.Tensor] = None, stream=None):
    """Total operator of every sequence: (pi int32 [B,H,N], d fp32 [B,H,N(,2)])."""
    dev = inp.diag.device
    flags = SEL_FLAG[inp.sel_mode] | (PDSSM_COMPLEX if inp.complex else 0)
    pi = torch.empty((inp.B, inp.H, inp.N), dtype=torch.int32, device=dev)
    d = torch.empty((inp.B, inp.H, inp.N, 2) if inp.complex else (inp.B, inp.H, inp.N),
                    dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = workspace_for(inp)
    check(pdssm_compose(inp.sel_or_logits, inp.dict_idx, inp.diag, pi, d, inp.B, inp.H, inp.L,
                        inp.N, inp.K, flags, workspace, workspace.numel(), stream))
    return pi, d


def dict_hardmax(m: torch.Tensor, stream=None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dict_idx int32 [H,K,N] from dense matrices m [H,K,N,N] (fp32 or bf16):
    the column-wise hardmax of every matrix."""
    H, K, N, N2 = m.shape
    if N != N2:
        raise ValueError("m must be [H,K,N,N]")
    flags = PDSSM_LOGITS_BF16 if m.dtype == torch.bfloat16 else PDSSM_LOGITS_F32
    if out is None:
        out = torch.empty((H, K, N), dtype=torch.int32, device=m.device)
    check(pdssm_dict_hardmax(m, out, H, K, N, flags, stream))
    return out


def decode_step(sel_or_logits, dict_idx, diag, b, c, x, *, sel_mode: str, complex: bool,
                bc_bf16: bool, y_bf16: bool, y: Optional[torch.Tensor] = None, stream=None):
    """One recurrent step for every (b, h): updates the state x [B,H,N(,2)]
    in place and returns y [B,H]."""
    B, H = diag.shape[:2]
    K, N = dict_idx.shape[1], dict_idx.shape[2]
    flags = SEL_FLAG[sel_mode] | (PDSSM_COMPLEX if complex else 0) | \
        (PDSSM_BC_BF16 if bc_bf16 else 0) | (PDSSM_Y_BF16 if y_bf16 else 0)
    if y is None:
        y = torch.empty((B, H), device=diag.device,
                        dtype=torch.bfloat16 if y_bf16 else torch.float32)
    check(pdssm_decode_step(sel_or_logits, dict_idx, diag, b, c, y, x, B, H, N, K, flags, stream))
    return y


class PackedRouterWeights(NamedTuple):
    """Router weights in the packed layout (bf16 [H, D/8, P, 8]) with the
    dictionary size K they were packed for."""
    data: torch.Tensor
    K: int


def router_pack_weights(w: torch.Tensor, *, stream=None) -> PackedRouterWeights:
    """The packed layout of router weights w [H,K,D] bf16 (pack once per
    weight update; router_select then runs its faster kernel)."""
    H, K, D = w.shape
    if w.dtype != torch.bfloat16:
        raise ValueError("w [H,K,D] must be bf16")
    P = 64 if K <= 64 else 128
    out = torch.empty((H, D // 8, P, 8), dtype=torch.bfloat16, device=w.device)
    check(pdssm_router_pack_weights(w, out, H, K, D, stream))
    return PackedRouterWeights(out, K)


def router_select(u: torch.Tensor, w, *, out: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """sel int16 [B,H,L] from bf16 step inputs u [B,L,D] and router weights
    w (bf16 [H,K,D], or PackedRouterWeights from router_pack_weights): the
    argmax of each head's K scores, computed on the matrix cores without
    writing the scores."""
    B, L, D = u.shape
    if isinstance(w, PackedRouterWeights):
        H, D8, P, _ = w.data.shape
        K, D2, wt, flags = w.K, D8 * 8, w.data, PDSSM_ROUTER_W_PACKED
    else:
        H, K, D2 = w.shape
        wt, flags = w, 0
    if D != D2 or u.dtype != torch.bfloat16 or wt.dtype != torch.bfloat16:
        raise ValueError("u [B,L,D] and the weights must be bf16 with the same D")
    if out is None:
        out = torch.empty((B, H, L), dtype=torch.int16, device=u.device)
    check(pdssm_router_select(u, wt, out, B, L, H, K, D, flags, stream))
    return out


# ---------------------------------------------------------------------------
# Operators beside the scan (include/pdssm_layers.h)
# ---------------------------------------------------------------------------

class _Strides(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int64), ("h", ctypes.c_int64), ("l", ctypes.c_int64)]


def _strides(strides):
    """The pdssm_strides list of (b, h, l) triples, or None (contiguous)."""
    if strides is None:
        return None
    return (_Strides * len(strides))(*strides)


def pdssm_delta_fwd(q, k, v, g, beta, s0, o, s_final, B, Hk, Hv, L, Dk, Dv, scale, flags, strides,
                    workspace, workspace_bytes, stream=None) -> int:
    return library().pdssm_delta_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(s0), _ptr(o),
                                     _ptr(s_final), B, Hk, Hv, L, Dk, Dv, scale, flags,
                                     _strides(strides), _ptr(workspace), workspace_bytes,
                                     _stream(stream))


def pdssm_delta_workspace_bytes(B, Hk, Hv, L, Dk, Dv, flags) -> int:
    return library().pdssm_delta_workspace_bytes(B, Hk, Hv, L, Dk, Dv, flags)


def pdssm_delta_bwd(q, k, v, g, beta, s0, d_o, ds_final, dq, dk, dv, dg, dbeta, ds0, B, Hk, Hv, L,
                    Dk, Dv, scale, flags, strides, workspace, workspace_bytes, stream=None) -> int:
    return library().pdssm_delta_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(s0),
                                     _ptr(d_o), _ptr(ds_final), _ptr(dq), _ptr(dk), _ptr(dv),
                                     _ptr(dg), _ptr(dbeta), _ptr(ds0), B, Hk, Hv, L, Dk, Dv, scale,
                                     flags, _strides(strides), _ptr(workspace), workspace_bytes,
                                     _stream(stream))


def pdssm_delta_bwd_workspace_bytes(B, Hk, Hv, L, Dk, Dv, flags) -> int:
    return library().pdssm_delta_bwd_workspace_bytes(B, Hk, Hv, L, Dk, Dv, flags)


def pdssm_delta_step(q, k, v, g, beta, s, o, s_out, B, Hk, Hv, Dk, Dv, scale, flags, strides,
                     stream=None) -> int:
    return library().pdssm_delta_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(s),
                                      _ptr(o), _ptr(s_out), B, Hk, Hv, Dk, Dv, scale, flags,
                                      _strides(strides), _stream(stream))


def pdssm_qk_norm_rope_fwd(q, k, wq, wk, cos, sin, pos, q_out, k_out, B, Hq, Hk, L, D, R, P, eps,
                           flags, strides, stream=None) -> int:
    return library().pdssm_qk_norm_rope_fwd(_ptr(q), _ptr(k), _ptr(wq), _ptr(wk), _ptr(cos),
                                            _ptr(sin), _ptr(pos), _ptr(q_out), _ptr(k_out), B, Hq,
                                            Hk, L, D, R, P, eps, flags, _strides(strides),
                                            _stream(stream))


def pdssm_qk_norm_rope_bwd(q, k, wq, wk, cos, sin, pos, dq_out, dk_out, dq, dk, dwq, dwk, B, Hq, Hk,
                           L, D, R, P, eps, flags, strides, workspace, workspace_bytes,
                           stream=None) -> int:
    return library().pdssm_qk_norm_rope_bwd(_ptr(q), _ptr(k), _ptr(wq), _ptr(wk), _ptr(cos),
                                            _ptr(sin), _ptr(pos), _ptr(dq_out), _ptr(dk_out),
                                            _ptr(dq), _ptr(dk), _ptr(dwq), _ptr(dwk), B, Hq, Hk, L,
                                            D, R, P, eps, flags, _strides(strides),
                                            _ptr(workspace), workspace_bytes, _stream(stream))


def pdssm_qk_norm_rope_bwd_workspace_bytes(B, Hq, Hk, L, D) -> int:
    return library().pdssm_qk_norm_rope_bwd_workspace_bytes(B, Hq, Hk, L, D)


# What a call's tensors must be, worked out once for every set of shapes,
# strides and types (the plans below) and not again for every call: a decode
# step's kernel takes about as long as these checks.

def _data_flag(name: str, *dtypes) -> int:
    """The storage flag of tensors that must share one type, bf16 or fp32."""
    if dtypes[0] not in (torch.bfloat16, torch.float32) or any(t != dtypes[0] for t in dtypes):
        raise ValueError(f"{name} must share one type, bf16 or fp32")
    return PDSSM_DATA_BF16 if dtypes[0] == torch.bfloat16 else 0


def _form(t):
    """Shape, strides, type and device (-1: not a GPU) of a tensor, or None."""
    return None if t is None else (t.shape, t.stride(), t.dtype, t.get_device())


def _one_device(*forms) -> None:
    """The kernels take addresses: a tensor elsewhere would be a fault there."""
    devices = {form[3] for form in forms if form is not None}
    if len(devices) > 1 or -1 in devices:
        raise ValueError("all tensors must be on one GPU")


def _want(name: str, form, shape, dtype, contiguous: bool = False) -> None:
    if form is None:
        return
    if tuple(form[0]) != tuple(shape) or form[2] != dtype:
        raise ValueError(f"{name} must be {dtype} {list(shape)}, not {form[2]} {list(form[0])}")
    if contiguous and 0 not in form[0]:
        step = 1
        for n, st in zip(reversed(form[0]), reversed(form[1])):
            if n > 1 and st != step:
                raise ValueError(f"{name} must be contiguous")
            step *= n


def _rows(dims: int, *forms):
    """The pdssm_strides list of [B,H,L(,D)] tensors (dims 3), or of [B,H(,D)]
    ones (dims 2); D must be contiguous."""
    out = []
    for shape, st, *_ in forms:
        if len(st) > dims and st[dims] != 1 and shape[dims] > 1:
            raise ValueError("the last dimension must be contiguous")
        out.append((*st[:dims], *(0,) * (3 - dims)))
    return _strides(out)


def _delta_form(q, k, v, g, beta, dims):
    """Flag and sizes (B, Hk, Hv, L, Dk, Dv) of a call; L is 1 for a step."""
    flag = _data_flag("q, k and v", q[2], k[2], v[2])
    if len(q[0]) != dims + 1 or len(v[0]) != dims + 1:
        raise ValueError("q, k and v must be [B,H,L,D] (a step: [B,H,D])")
    B, Hk, *L, Dk = q[0]
    Hv, Dv = v[0][1], v[0][-1]
    _want("k", k, q[0], q[2])
    _want("v", v, (B, Hv, *L, Dv), q[2])
    _want("g", g, (B, Hv, *L), torch.float32)
    _want("beta", beta, (B, Hv, *L), torch.float32)
    return flag, B, Hk, Hv, (L[0] if L else 1), Dk, Dv


def _workspace(need: int, workspace, device):
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError("the workspace must be contiguous and on the tensors' GPU")
    if workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"the workspace needs {need} bytes")
    return workspace


def _need(n: int) -> int:
    if n == 0:
        raise PdssmError(PDSSM_ERR_DIM, "invalid sizes")
    return n


def _on_stream(stream, call, *args, **kw):
    """The call as under torch.cuda.stream(stream): the results and the
    workspace that it allocates belong to that stream, so memory freed on
    return is not given to another stream's work while the kernels still run.
    (A call that is given all its buffers only takes the stream's handle,
    which is a few microseconds less.)"""
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, args[0].device)
    with torch.cuda.stream(stream):
        return call(*args, **kw)


# The current stream's handle without building a Stream object, where this
# torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda device: torch.cuda.current_stream(device).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _run(entry, t, stream, *args) -> None:
    """The call on `stream`, or the current stream of the tensor's device, with
    that device the current one: a default stream is the current device's."""
    device = t.get_device()
    if device != _current_device():
        with torch.cuda.device(device):
            return _run(entry, t, stream, *args)
    status = entry(*args, _raw_stream(device) if stream is None else _stream(stream))
    if status != PDSSM_OK:
        check(status)


@functools.lru_cache(maxsize=1024)
def _delta_plan(q, k, v, g, beta, o, s0, s_final):
    flag, B, Hk, Hv, L, Dk, Dv = sizes = _delta_form(q, k, v, g, beta, 3)
    _want("o", o, v[0], v[2])
    _want("s0", s0, (B, Hv, Dk, Dv), torch.float32, True)
    _want("s_final", s_final, (B, Hv, Dk, Dv), torch.float32, True)
    need = _need(pdssm_delta_workspace_bytes(B, Hk, Hv, L, Dk, Dv, flag))
    _one_device(q, k, v, g, beta, o, s0, s_final)
    return sizes, _rows(3, q, k, v, g, beta, o), need


def delta_rule(q, k, v, g, beta, s0=None, *, scale: Optional[float] = None, want_state: bool = True,
               o: Optional[torch.Tensor] = None, s_final: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, stream=None):
    """The gated delta rule over whole sequences: (o [B,Hv,L,Dv], s_final
    [B,Hv,Dk,Dv] or None).  q, k [B,Hk,L,Dk] and v [B,Hv,L,Dv] bf16 or fp32
    with any strides of the first three dimensions, g (log decay) and beta
    fp32 [B,Hv,L], s0 fp32 [B,Hv,Dk,Dv] or None; scale 1/sqrt(Dk) by default.
    o has the memory order of v; s_final may be s0.  ``stream`` (here and in
    the functions below): the call as under torch.cuda.stream(stream)."""
    if stream is not None and (o is None or workspace is None or (s_final is None and want_state)):
        return _on_stream(stream, delta_rule, q, k, v, g, beta, s0, scale=scale, want_state=want_state, o=o,
                          s_final=s_final, workspace=workspace)
    if o is None:
        o = torch.empty_like(v)
    if s_final is None and want_state:
        s_final = torch.empty((v.shape[0], v.shape[1], q.shape[-1], v.shape[-1]), dtype=torch.float32,
                              device=v.device)
    (flag, B, Hk, Hv, L, Dk, Dv), rows, need = _delta_plan(
        _form(q), _form(k), _form(v), _form(g), _form(beta), _form(o), _form(s0), _form(s_final))
    workspace = _workspace(need, workspace, v.device)
    _run(library().pdssm_delta_fwd, v, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
         _ptr(s0), o.data_ptr(), _ptr(s_final), B, Hk, Hv, L, Dk, Dv, Dk ** -0.5 if scale is None else scale, flag,
         rows, workspace.data_ptr(), need)
    return o, s_final


@functools.lru_cache(maxsize=1024)
def _delta_bwd_plan(q, k, v, g, beta, s0, do, ds_final, dq, dk, dv, dg, dbeta, ds0):
    flag, B, Hk, Hv, L, Dk, Dv = sizes = _delta_form(q, k, v, g, beta, 3)
    for name, form, like in (("do", do, v), ("dq", dq, q), ("dk", dk, k), ("dv", dv, v), ("dg", dg, g),
                             ("dbeta", dbeta, g)):
        _want(name, form, like[0], like[2])
    for name, form in (("s0", s0), ("ds_final", ds_final), ("ds0", ds0)):
        _want(name, form, (B, Hv, Dk, Dv), torch.float32, True)
    need = _need(pdssm_delta_bwd_workspace_bytes(B, Hk, Hv, L, Dk, Dv, flag))
    _one_device(q, k, v, g, beta, s0, do, ds_final, dq, dk, dv, dg, dbeta, ds0)
    return sizes, _rows(3, q, k, v, g, beta, do, dq, dk, dv, dg, dbeta), need


def delta_rule_bwd(q, k, v, g, beta, do, s0=None, ds_final=None, *, scale: Optional[float] = None,
                   want_ds0: bool = True, out=None, workspace: Optional[torch.Tensor] = None,
                   stream=None):
    """Gradients of delta_rule from its inputs, the gradient ``do`` of o and
    that of s_final (None: zero): (dq, dk, dv, dg, dbeta, ds0 or None), each
    in the memory order of its input.  ``out`` may hold a previous call's
    result to write into."""
    if stream is not None and (out is None or workspace is None):
        return _on_stream(stream, delta_rule_bwd, q, k, v, g, beta, do, s0, ds_final, scale=scale,
                          want_ds0=want_ds0, out=out, workspace=workspace)
    if out is not None:
        dq, dk, dv, dg, dbeta, ds0 = out
    else:
        dq, dk, dv, dg, dbeta = (torch.empty_like(t) for t in (q, k, v, g, beta))
        ds0 = torch.empty((v.shape[0], v.shape[1], q.shape[-1], v.shape[-1]), dtype=torch.float32,
                          device=v.device) if want_ds0 else None
    (flag, B, Hk, Hv, L, Dk, Dv), rows, need = _delta_bwd_plan(
        _form(q), _form(k), _form(v), _form(g), _form(beta), _form(s0), _form(do), _form(ds_final),
        _form(dq), _form(dk), _form(dv), _form(dg), _form(dbeta), _form(ds0))
    workspace = _workspace(need, workspace, v.device)
    _run(library().pdssm_delta_bwd, v, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
         _ptr(s0), do.data_ptr(), _ptr(ds_final), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dg.data_ptr(),
         dbeta.data_ptr(), _ptr(ds0), B, Hk, Hv, L, Dk, Dv, Dk ** -0.5 if scale is None else scale, flag, rows,
         workspace.data_ptr(), need)
    return dq, dk, dv, dg, dbeta, ds0


@functools.lru_cache(maxsize=1024)
def _step_plan(q, k, v, g, beta, o, s, s_out):
    flag, B, Hk, Hv, _, Dk, Dv = _delta_form(q, k, v, g, beta, 2)
    _want("o", o, v[0], v[2])
    _want("s", s, (B, Hv, Dk, Dv), torch.float32, True)
    _want("s_out", s_out, (B, Hv, Dk, Dv), torch.float32, True)
    _one_device(q, k, v, g, beta, o, s, s_out)
    return flag, B, Hk, Hv, Dk, Dv, _rows(2, q, k, v, g, beta, o)


def delta_step(q, k, v, g, beta, s, *, s_out: Optional[torch.Tensor] = None,
               scale: Optional[float] = None, o: Optional[torch.Tensor] = None, stream=None):
    """One step of the gated delta rule: o [B,Hv,Dv] from q, k [B,Hk,Dk],
    v [B,Hv,Dv], g, beta fp32 [B,Hv] and the state s fp32 [B,Hv,Dk,Dv], which
    is updated in place, or into s_out."""
    if stream is not None and o is None:
        return _on_stream(stream, delta_step, q, k, v, g, beta, s, s_out=s_out, scale=scale, o=o)
    if s_out is None:
        s_out = s
    if o is None:
        o = torch.empty_like(v)
    flag, B, Hk, Hv, Dk, Dv, rows = _step_plan(_form(q), _form(k), _form(v), _form(g), _form(beta),
                                               _form(o), _form(s), _form(s_out))
    _run(library().pdssm_delta_step, v, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(),
         beta.data_ptr(), s.data_ptr(), o.data_ptr(), s_out.data_ptr(), B, Hk, Hv, Dk, Dv,
         Dk ** -0.5 if scale is None else scale, flag, rows)
    return o


_NORM_KIND = {"rms": 0, "l2": PDSSM_NORM_L2}
_ROPE_PAIRS = {"half": 0, "adjacent": PDSSM_ROPE_PAIRS}


class UnknownWord(ValueError, KeyError):
    """A word that an argument does not have (a KeyError too, as callers may
    have caught it by that name)."""
    __str__ = Exception.__str__


def _word(name: str, words: dict, word) -> int:
    if word not in words:
        raise UnknownWord(f"{name} must be one of {', '.join(words)}, not {word!r}")
    return words[word]


def _norm_form(q, k, wq, wk, cos, sin, pos, kind, pairs):
    """Flags and sizes (B, Hq, Hk, L, D, R, P) of a call."""
    flags = _data_flag("q and k", q[2], k[2]) | _word("kind", _NORM_KIND, kind) | _word("pairs", _ROPE_PAIRS, pairs)
    if len(q[0]) != 4 or len(k[0]) != 4:
        raise ValueError("q and k must be [B,H,L,D]")
    B, Hq, L, D = q[0]
    Hk = k[0][1]
    _want("k", k, (B, Hk, L, D), q[2])
    _want("wq", wq, (D,), torch.float32, True)
    _want("wk", wk, (D,), torch.float32, True)
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin go together")
    if cos is not None and len(cos[0]) != 2:
        raise ValueError("cos and sin must be [P,R/2]")
    P, R = (0, 0) if cos is None else (cos[0][0], 2 * cos[0][1])
    _want("cos", cos, (P, R // 2), torch.float32, True)
    _want("sin", sin, (P, R // 2), torch.float32, True)
    _want("pos", pos, (B, L), torch.int32, True)
    return flags, B, Hq, Hk, L, D, R, P


@functools.lru_cache(maxsize=1024)
def _norm_plan(q, k, wq, wk, cos, sin, pos, kind, pairs, q_out, k_out):
    sizes = _norm_form(q, k, wq, wk, cos, sin, pos, kind, pairs)
    _want("q_out", q_out, q[0], q[2])
    _want("k_out", k_out, k[0], k[2])
    _one_device(q, k, wq, wk, cos, sin, pos, q_out, k_out)
    return sizes, _rows(3, q, k, q_out, k_out)


def qk_norm_rope(q, k, wq=None, wk=None, cos=None, sin=None, pos=None, *, kind: str = "rms",
                 pairs: str = "half", eps: float = 1e-6, out=None, stream=None):
    """The norm of every query and key head and the rotation of its first R
    dimensions: (q_out [B,Hq,L,D], k_out [B,Hk,L,D]).  q [B,Hq,L,D] and k
    [B,Hk,L,D] bf16 or fp32 with any strides of the first three dimensions;
    weights fp32 [D] or None; cos, sin fp32 [P,R/2] or None (no rotation); pos
    int32 [B,L] or None (the place in the sequence).  ``kind``: "rms" or "l2"
    (unit length); ``pairs``: "half" (i, i + R/2) or "adjacent" (2i, 2i + 1).
    The results have the memory order of q and k; ``out``: two tensors to
    write into instead (the inputs, to work in place)."""
    if stream is not None and out is None:
        return _on_stream(stream, qk_norm_rope, q, k, wq, wk, cos, sin, pos, kind=kind, pairs=pairs, eps=eps, out=out)
    q_out, k_out = (torch.empty_like(q), torch.empty_like(k)) if out is None else out
    (flags, B, Hq, Hk, L, D, R, P), rows = _norm_plan(
        _form(q), _form(k), _form(wq), _form(wk), _form(cos), _form(sin), _form(pos), kind, pairs,
        _form(q_out), _form(k_out))
    _run(library().pdssm_qk_norm_rope_fwd, q, stream, q.data_ptr(), k.data_ptr(), _ptr(wq), _ptr(wk), _ptr(cos),
         _ptr(sin), _ptr(pos), q_out.data_ptr(), k_out.data_ptr(), B, Hq, Hk, L, D, R, P, eps, flags, rows)
    return q_out, k_out


@functools.lru_cache(maxsize=1024)
def _norm_bwd_plan(q, k, wq, wk, cos, sin, pos, kind, pairs, dq_out, dk_out, dq, dk):
    flags, B, Hq, Hk, L, D, R, P = sizes = _norm_form(q, k, wq, wk, cos, sin, pos, kind, pairs)
    for name, form, like in (("dq_out", dq_out, q), ("dk_out", dk_out, k), ("dq", dq, q), ("dk", dk, k)):
        _want(name, form, like[0], like[2])
    need = 0
    if wq is not None or wk is not None:
        need = _need(pdssm_qk_norm_rope_bwd_workspace_bytes(B, Hq, Hk, L, D))
    _one_device(q, k, wq, wk, cos, sin, pos, dq_out, dk_out, dq, dk)
    return sizes, _rows(3, q, k, dq_out, dk_out, dq, dk), need


def qk_norm_rope_bwd(q, k, dq_out, dk_out, wq=None, wk=None, cos=None, sin=None, pos=None, *,
                     kind: str = "rms", pairs: str = "half", eps: float = 1e-6, out=None,
                     workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients of qk_norm_rope from its inputs and the gradients of its
    outputs: (dq, dk, dwq, dwk), the first two in the memory order of q and k,
    the last two None where the weight is.  ``out``: dq and dk to write into
    instead (dq_out and dk_out, to work in place)."""
    if stream is not None and (out is None or wq is not None or wk is not None):
        return _on_stream(stream, qk_norm_rope_bwd, q, k, dq_out, dk_out, wq, wk, cos, sin, pos, kind=kind,
                          pairs=pairs, eps=eps, out=out, workspace=workspace)
    dq, dk = (torch.empty_like(q), torch.empty_like(k)) if out is None else out
    (flags, B, Hq, Hk, L, D, R, P), rows, need = _norm_bwd_plan(
        _form(q), _form(k), _form(wq), _form(wk), _form(cos), _form(sin), _form(pos), kind, pairs,
        _form(dq_out), _form(dk_out), _form(dq), _form(dk))
    dwq, dwk = (None if w is None else torch.empty_like(w) for w in (wq, wk))
    if need:
        workspace = _workspace(need, workspace, q.device)
    _run(library().pdssm_qk_norm_rope_bwd, q, stream, q.data_ptr(), k.data_ptr(), _ptr(wq), _ptr(wk), _ptr(cos),
         _ptr(sin), _ptr(pos), dq_out.data_ptr(), dk_out.data_ptr(), dq.data_ptr(), dk.data_ptr(), _ptr(dwq),
         _ptr(dwk), B, Hq, Hk, L, D, R, P, eps, flags, rows, workspace.data_ptr() if need else None, need)
    return dq, dk, dwq, dwk


# ---------------------------------------------------------------------------
# Operators of a layer's block (include/pdssm_block.h)
# ---------------------------------------------------------------------------

def pdssm_linear_fwd(q, k, v, g, s0, o, s_final, B, Hk, Hv, L, Dk, Dv, scale, flags, strides, workspace,
                     workspace_bytes, stream=None) -> int:
    return library().pdssm_linear_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(s0), _ptr(o), _ptr(s_final), B,
                                      Hk, Hv, L, Dk, Dv, scale, flags, _strides(strides), _ptr(workspace),
                                      workspace_bytes, _stream(stream))


def pdssm_linear_workspace_bytes(B, Hk, Hv, L, Dk, Dv, flags) -> int:
    return library().pdssm_linear_workspace_bytes(B, Hk, Hv, L, Dk, Dv, flags)


def pdssm_linear_bwd(q, k, v, g, s0, d_o, ds_final, dq, dk, dv, dg, ds0, B, Hk, Hv, L, Dk, Dv, scale, flags,
                     strides, workspace, workspace_bytes, stream=None) -> int:
    return library().pdssm_linear_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(s0), _ptr(d_o), _ptr(ds_final),
                                      _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg), _ptr(ds0), B, Hk, Hv, L, Dk, Dv,
                                      scale, flags, _strides(strides), _ptr(workspace), workspace_bytes,
                                      _stream(stream))


def pdssm_linear_bwd_workspace_bytes(B, Hk, Hv, L, Dk, Dv, flags) -> int:
    return library().pdssm_linear_bwd_workspace_bytes(B, Hk, Hv, L, Dk, Dv, flags)


def pdssm_linear_step(q, k, v, g, s, o, s_out, B, Hk, Hv, Dk, Dv, scale, flags, strides, stream=None) -> int:
    return library().pdssm_linear_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(s), _ptr(o), _ptr(s_out), B, Hk,
                                       Hv, Dk, Dv, scale, flags, _strides(strides), _stream(stream))


def _linear_form(q, k, v, g, dims):
    """Flag, sizes (B, Hk, Hv, L, Dk, Dv) and the gates' strides of a call; L is
    1 for a step."""
    flag = _data_flag("q, k and v", q[2], k[2], v[2])
    if len(q[0]) != dims + 1 or len(v[0]) != dims + 1:
        raise ValueError("q, k and v must be [B,H,L,D] (a step: [B,H,D])")
    B, Hk, *L, Dk = q[0]
    Hv, Dv = v[0][1], v[0][-1]
    _want("k", k, q[0], q[2])
    _want("v", v, (B, Hv, *L, Dv), q[2])
    gates = (0, 0, 0)
    if g is not None and len(g[0]) == 1:
        _want("g", g, (Hv,), torch.float32)
        gates = (0, g[1][0], 0)
    elif g is not None:
        _want("g", g, (B, Hv, *L), torch.float32)
        gates = (*g[1], *(0,) * (3 - dims))
    return (flag, B, Hk, Hv, (L[0] if L else 1), Dk, Dv), gates


def _row_strides(dims, *forms):
    """The triples of _rows, as a list."""
    out = []
    for shape, st, *_ in forms:
        if st[dims] != 1 and shape[dims] > 1:
            raise ValueError("the last dimension must be contiguous")
        out.append((*st[:dims], *(0,) * (3 - dims)))
    return out


@functools.lru_cache(maxsize=1024)
def _linear_plan(q, k, v, g, o, s0, s_final):
    sizes, gates = _linear_form(q, k, v, g, 3)
    flag, B, Hk, Hv, L, Dk, Dv = sizes
    _want("o", o, v[0], v[2])
    _want("s0", s0, (B, Hv, Dk, Dv), torch.float32, True)
    _want("s_final", s_final, (B, Hv, Dk, Dv), torch.float32, True)
    need = _need(pdssm_linear_workspace_bytes(B, Hk, Hv, L, Dk, Dv, flag))
    _one_device(q, k, v, g, o, s0, s_final)
    rows = _row_strides(3, q, k, v, o)
    return sizes, _strides(rows[:3] + [gates] + rows[3:]), need


def linear_attention(q, k, v, g=None, s0=None, *, scale: Optional[float] = None, want_state: bool = True,
                     o: Optional[torch.Tensor] = None, s_final: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None):
    """Linear attention with decays over whole sequences: (o [B,Hv,L,Dv],
    s_final [B,Hv,Dk,Dv] or None).  q, k [B,Hk,L,Dk] and v [B,Hv,L,Dv] bf16 or
    fp32 with any strides of the first three dimensions; g the log decays, fp32
    [B,Hv,L], or [Hv] for a fixed one of each head, or None; s0 fp32
    [B,Hv,Dk,Dv] or None; scale 1/sqrt(Dk) by default.  o has the memory order
    of v; s_final may be s0.  ``stream`` (here and in the functions below): the
    call as under torch.cuda.stream(stream)."""
    if stream is not None and (o is None or workspace is None or (s_final is None and want_state)):
        return _on_stream(stream, linear_attention, q, k, v, g, s0, scale=scale, want_state=want_state, o=o,
                          s_final=s_final, workspace=workspace)
    if o is None:
        o = torch.empty_like(v)
    if s_final is None and want_state:
        s_final = torch.empty((v.shape[0], v.shape[1], q.shape[-1], v.shape[-1]), dtype=torch.float32,
                              device=v.device)
    (flag, B, Hk, Hv, L, Dk, Dv), rows, need = _linear_plan(
        _form(q), _form(k), _form(v), _form(g), _form(o), _form(s0), _form(s_final))
    workspace = _workspace(need, workspace, v.device)
    _run(library().pdssm_linear_fwd, v, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(g), _ptr(s0),
         o.data_ptr(), _ptr(s_final), B, Hk, Hv, L, Dk, Dv, Dk ** -0.5 if scale is None else scale, flag, rows,
         workspace.data_ptr(), need)
    return o, s_final


@functools.lru_cache(maxsize=1024)
def _linear_bwd_plan(q, k, v, g, s0, do, ds_final, dq, dk, dv, dg, ds0):
    sizes, gates = _linear_form(q, k, v, g, 3)
    flag, B, Hk, Hv, L, Dk, Dv = sizes
    for name, form, like in (("do", do, v), ("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        _want(name, form, like[0], like[2])
    if dg is not None:
        _want("dg", dg, g[0], torch.float32)
    for name, form in (("s0", s0), ("ds_final", ds_final), ("ds0", ds0)):
        _want(name, form, (B, Hv, Dk, Dv), torch.float32, True)
    dgates = (0, 0, 0)
    if dg is None:
        flag |= PDSSM_NO_DG
    elif len(dg[0]) == 1:
        flag |= PDSSM_DG_HEADS
        dgates = (0, dg[1][0], 0)
    else:
        dgates = tuple(dg[1])
    need = _need(pdssm_linear_bwd_workspace_bytes(B, Hk, Hv, L, Dk, Dv, flag))
    _one_device(q, k, v, g, s0, do, ds_final, dq, dk, dv, dg, ds0)
    rows = _row_strides(3, q, k, v, do, dq, dk, dv)
    return (flag, *sizes[1:]), _strides(rows[:3] + [gates] + rows[3:] + [dgates]), need


def linear_attention_bwd(q, k, v, g, do, s0=None, ds_final=None, *, scale: Optional[float] = None,
                         want_dg: bool = True, want_ds0: bool = True, out=None,
                         workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients of linear_attention from its inputs, the gradient ``do`` of o
    and that of s_final (None: zero): (dq, dk, dv, dg, ds0), the first four in
    the memory order of their inputs; dg has the shape of g (for [Hv] the sum
    over sequences and steps) and is None without g or with want_dg=False, ds0
    None with want_ds0=False.  ``out`` may hold a previous call's result to
    write into."""
    if stream is not None and (out is None or workspace is None):
        return _on_stream(stream, linear_attention_bwd, q, k, v, g, do, s0, ds_final, scale=scale,
                          want_dg=want_dg, want_ds0=want_ds0, out=out, workspace=workspace)
    if out is not None:
        dq, dk, dv, dg, ds0 = out
    else:
        dq, dk, dv = (torch.empty_like(t) for t in (q, k, v))
        dg = torch.empty_like(g) if g is not None and want_dg else None
        ds0 = torch.empty((v.shape[0], v.shape[1], q.shape[-1], v.shape[-1]), dtype=torch.float32,
                          device=v.device) if want_ds0 else None
    if g is None and dg is not None:
        raise ValueError("dg without g")
    (flag, B, Hk, Hv, L, Dk, Dv), rows, need = _linear_bwd_plan(
        _form(q), _form(k), _form(v), _form(g), _form(s0), _form(do), _form(ds_final), _form(dq), _form(dk),
        _form(dv), _form(dg), _form(ds0))
    workspace = _workspace(need, workspace, v.device)
    _run(library().pdssm_linear_bwd, v, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(g), _ptr(s0),
         do.data_ptr(), _ptr(ds_final), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), _ptr(dg), _ptr(ds0), B, Hk, Hv, L,
         Dk, Dv, Dk ** -0.5 if scale is None else scale, flag, rows, workspace.data_ptr(), need)
    return dq, dk, dv, dg, ds0


@functools.lru_cache(maxsize=1024)
def _linear_step_plan(q, k, v, g, o, s, s_out):
    (flag, B, Hk, Hv, _, Dk, Dv), gates = _linear_form(q, k, v, g, 2)
    _want("o", o, v[0], v[2])
    _want("s", s, (B, Hv, Dk, Dv), torch.float32, True)
    _want("s_out", s_out, (B, Hv, Dk, Dv), torch.float32, True)
    _one_device(q, k, v, g, o, s, s_out)
    rows = _row_strides(2, q, k, v, o)
    return flag, B, Hk, Hv, Dk, Dv, _strides(rows[:3] + [gates] + rows[3:])


def linear_attention_step(q, k, v, g, s, *, s_out: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                          o: Optional[torch.Tensor] = None, stream=None):
    """One step of linear attention: o [B,Hv,Dv] from q, k [B,Hk,Dk], v
    [B,Hv,Dv], g fp32 [B,Hv], [Hv] or None, and the state s fp32 [B,Hv,Dk,Dv],
    which is updated in place, or into s_out."""
    if stream is not None and o is None:
        return _on_stream(stream, linear_attention_step, q, k, v, g, s, s_out=s_out, scale=scale, o=o)
    if s_out is None:
        s_out = s
    if o is None:
        o = torch.empty_like(v)
    flag, B, Hk, Hv, Dk, Dv, rows = _linear_step_plan(_form(q), _form(k), _form(v), _form(g), _form(o), _form(s),
                                                      _form(s_out))
    _run(library().pdssm_linear_step, v, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(g), s.data_ptr(),
         o.data_ptr(), s_out.data_ptr(), B, Hk, Hv, Dk, Dv, Dk ** -0.5 if scale is None else scale, flag, rows)
    return o


def pdssm_layer_norm_fwd(x, residual, w, b, y, h, B, H, L, D, eps, p, seed, offset, rng, flags, strides,
                         stream=None) -> int:
    return library().pdssm_layer_norm_fwd(_ptr(x), _ptr(residual), _ptr(w), _ptr(b), _ptr(y), _ptr(h), B, H, L, D,
                                          eps, p, seed, offset, _ptr(rng), flags, _strides(strides),
                                          _stream(stream))


def pdssm_layer_norm_bwd(h, dy, dh, w, dr, dx, dw, db, B, H, L, D, eps, p, seed, offset, rng, flags, strides,
                         workspace, workspace_bytes, stream=None) -> int:
    return library().pdssm_layer_norm_bwd(_ptr(h), _ptr(dy), _ptr(dh), _ptr(w), _ptr(dr), _ptr(dx), _ptr(dw),
                                          _ptr(db), B, H, L, D, eps, p, seed, offset, _ptr(rng), flags,
                                          _strides(strides), _ptr(workspace), workspace_bytes, _stream(stream))


def pdssm_layer_norm_bwd_workspace_bytes(B, H, L, D) -> int:
    return library().pdssm_layer_norm_bwd_workspace_bytes(B, H, L, D)


def pdssm_dropout(x, residual, y, B, H, L, D, p, seed, offset, rng, flags, strides, stream=None) -> int:
    return library().pdssm_dropout(_ptr(x), _ptr(residual), _ptr(y), B, H, L, D, p, seed, offset, _ptr(rng), flags,
                                   _strides(strides), _stream(stream))


def _block_rows(*forms):
    """The (b, h, l) triples of row tensors [D] to [B,H,L,D] (None: zeros)."""
    out = []
    for form in forms:
        if form is None:
            out.append((0, 0, 0))
            continue
        shape, st = form[:2]
        if st[-1] != 1 and shape[-1] > 1:
            raise ValueError("the last dimension must be contiguous")
        out.append((*(0,) * (4 - len(shape)), *st[:-1]))
    return _strides(out)


def _block_form(name, x, rng, w, b, others):
    """Flag and sizes (B, H, L, D) of a call on rows like x."""
    if not 1 <= len(x[0]) <= 4:
        raise ValueError(f"{name} must have one to four dimensions")
    flag = _data_flag("row tensors", *(f[2] for f in (x, *others.values()) if f is not None))
    for other, form in others.items():
        _want(other, form, x[0], x[2])
    D = x[0][-1]
    _want("w", w, (D,), torch.float32, True)
    _want("b", b, (D,), torch.float32, True)
    _want("seed", rng, (2,), torch.int64, True)
    _one_device(x, rng, w, b, *others.values())
    return (flag, *(1,) * (4 - len(x[0])), *x[0])


def _seed(seed, offset):
    """(seed, offset, the tensor that holds both or None) of a call."""
    if isinstance(seed, torch.Tensor):
        if offset:
            raise ValueError("a seed tensor holds the offset too")
        return 0, 0, seed
    return seed & 0xFFFFFFFFFFFFFFFF, offset & 0xFFFFFFFFFFFFFFFF, None


def _drops(p: float) -> bool:
    """Whether dropout with p drops anything (its 16-bit threshold is above 0)."""
    return p * 65536 + 0.5 >= 1


def _same_place(a, b) -> bool:
    return a is not None and b is not None and (a is b or a.data_ptr() == b.data_ptr() != 0)


@functools.lru_cache(maxsize=1024)
def _layer_norm_plan(x, w, b, residual, y, h, rng):
    sizes = _block_form("x", x, rng, w, b, {"residual": residual, "y": y, "h": h})
    return sizes, _block_rows(x, residual, y, h)


def layer_norm(x, w=None, b=None, *, residual=None, eps: float = 1e-5, p: float = 0.0, seed=0, offset: int = 0,
               out: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None, stream=None):
    """The layer norm over the last dimension of h = residual + dropout(x):
    (y, h).  x and residual bf16 or fp32 of one to four dimensions, any strides
    but the last; w, b fp32 [D] or None (1 and 0).  Without residual and dropout
    h is x itself, unless y takes its place or a place for h is given.  ``p``: the
    part of x that is dropped; ``seed`` and ``offset`` pick the mask, or an int64
    GPU tensor [2] in place of seed holds both.  The results have the memory order
    of x; ``out`` and ``h``: two tensors to write into instead (x or residual among
    them)."""
    if _same_place(out, h):
        raise ValueError("y and h are two tensors")
    new = h is None and (residual is not None or _drops(p) or _same_place(out, x))
    if stream is not None and (out is None or new):
        return _on_stream(stream, layer_norm, x, w, b, residual=residual, eps=eps, p=p, seed=seed, offset=offset,
                          out=out, h=h)
    y = torch.empty_like(x) if out is None else out
    to = h
    if new:
        h = to = torch.empty_like(x)
    seed, offset, rng = _seed(seed, offset)
    (flag, B, H, L, D), rows = _layer_norm_plan(_form(x), _form(w), _form(b), _form(residual), _form(y), _form(to),
                                                _form(rng))
    _run(library().pdssm_layer_norm_fwd, x, stream, x.data_ptr(), _ptr(residual), _ptr(w), _ptr(b), y.data_ptr(),
         _ptr(to), B, H, L, D, eps, p, seed, offset, _ptr(rng), flag, rows)
    return y, x if h is None else h


@functools.lru_cache(maxsize=1024)
def _layer_norm_bwd_plan(h, w, dy, dh, dr, dx, rng, sums):
    sizes = _block_form("h", h, rng, w, None, {"dy": dy, "dh": dh, "dr": dr, "dx": dx})
    need = _need(pdssm_layer_norm_bwd_workspace_bytes(*sizes[1:])) if sums else 0
    return sizes, _block_rows(h, dy, dh, dr, dx), need


def layer_norm_bwd(h, dy, w=None, *, dh=None, want_db: bool = False, eps: float = 1e-5, p: float = 0.0, seed=0,
                   offset: int = 0, out=None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients of layer_norm from h, the gradient dy of y and the one dh that h
    has from elsewhere (None: zero): (dr, dx, dw, db), of h (and the residual), of
    x (without dropout dr itself), of w (None without it) and of b (with
    want_db).  p, seed and offset as in the forward.  ``out``: dr and dx to write
    into instead (of dy, dh and h; one tensor twice without dropout)."""
    if stream is not None and (out is None or w is not None or want_db):
        return _on_stream(stream, layer_norm_bwd, h, dy, w, dh=dh, want_db=want_db, eps=eps, p=p, seed=seed,
                          offset=offset, out=out, workspace=workspace)
    drops = _drops(p)
    dr, dx = (torch.empty_like(h), torch.empty_like(h) if drops else None) if out is None else out
    if dx is None:
        dx = dr
    if drops and _same_place(dr, dx):
        raise ValueError("with dropout dr and dx are two tensors")
    seed, offset, rng = _seed(seed, offset)
    sums = w is not None or want_db
    to = None if dx is dr else dx
    (flag, B, H, L, D), rows, need = _layer_norm_bwd_plan(_form(h), _form(w), _form(dy), _form(dh), _form(dr),
                                                          _form(to), _form(rng), sums)
    dw = None if w is None else torch.empty_like(w)
    db = torch.empty(D, dtype=torch.float32, device=h.device) if want_db else None
    if need:
        workspace = _workspace(need, workspace, h.device)
    _run(library().pdssm_layer_norm_bwd, h, stream, h.data_ptr(), dy.data_ptr(), _ptr(dh), _ptr(w), dr.data_ptr(),
         _ptr(to), _ptr(dw), _ptr(db), B, H, L, D, eps, p, seed, offset, _ptr(rng), flag, rows,
         workspace.data_ptr() if need else None, need)
    return dr, dx, dw, db


@functools.lru_cache(maxsize=1024)
def _dropout_plan(x, residual, y, rng):
    sizes = _block_form("x", x, rng, None, None, {"residual": residual, "y": y})
    return sizes, _block_rows(x, residual, y)


def dropout(x, p: float, seed, offset: int = 0, *, residual=None, out: Optional[torch.Tensor] = None, stream=None):
    """residual + dropout(x), the mask from ``seed`` and ``offset`` (or an int64
    GPU tensor [2] of both as seed) by value and place, never stored.  The
    gradient of x is dropout of the result's with the same seed and offset.  x
    bf16 or fp32 of one to four dimensions, any strides but the last; ``out``: a
    tensor to write into (x or residual among them)."""
    if stream is not None and out is None:
        return _on_stream(stream, dropout, x, p, seed, offset, residual=residual)
    y = torch.empty_like(x) if out is None else out
    seed, offset, rng = _seed(seed, offset)
    (flag, B, H, L, D), rows = _dropout_plan(_form(x), _form(residual), _form(y), _form(rng))
    _run(library().pdssm_dropout, x, stream, x.data_ptr(), _ptr(residual), y.data_ptr(), B, H, L, D, p, seed, offset,
         _ptr(rng), flag, rows)
    return y
