"""LB-ADMM low-rank binary factorisation on MI355X (gfx950).

Thin Python binding of the C ABI in include/nq.h. Every step of the
per-layer path runs in the HIP kernels of libnq.so; this module only checks
and marshals arguments (torch tensors supply device memory and the current
stream). Importing works without a GPU; calls that need the device fail
loudly when libnq.so or the GPU is missing. There is no CPU fallback.

Functions mirror the C names without the ``nq_`` prefix:
    lbadmm_create / lbadmm_run / lbadmm_query / lbadmm_get_state /
    lbadmm_destroy / lbadmm_workspace_bytes / pack_signs /
    transpose_signs / binary_matmul / binary_matmul_noalloc / lw_* (LedoitWolf) /
    ste_* (STERefiner) / act8_quantize / act8_dequantize / act8_steps (Act8) /
    binary_matmul_backward / vocab_loss / vocab_loss_backward /
    vocab_logprobs (VocabLogprobs) / vocab_distill / vocab_distill_backward (VocabDistill) /
    op_precondition / op_gram / op_gemm_rhs / op_cholesky_inverse / op_svid
plus the conveniences ``LBADMM`` (a handle object) and ``lbadmm`` (one call).
"""
from __future__ import annotations

import ctypes as C
from dataclasses import dataclass
from typing import Optional

from . import _lib
from ._lib import (NQ_FLAG_COMPUTE_ERROR, NQ_FLAG_INIT_DRAWS, NQ_FLAG_NO_BALANCE,  # noqa: F401
                   NQ_FLAG_PROFILE, NQ_FLAG_PROFILE_RHS_ONLY, NQ_FLAG_SINGLE_STREAM,
                   NQ_FLAG_SOLVE_CG, NQ_FLAG_SOLVE_GD, NQ_OK, PHASES, Desc, Stats)

__all__ = [
    "NQError", "lbadmm_create", "lbadmm_run", "lbadmm_query", "lbadmm_get_state",
    "lbadmm_destroy", "lbadmm_profile", "lbadmm_workspace_bytes", "pack_signs", "transpose_signs",
    "binary_matmul", "binary_matmul_noalloc", "binary_matmul_work_floats", "LedoitWolf", "ledoit_wolf_diag",
    "Act8", "ACT8_GROUP", "act8_quantize", "act8_dequantize", "act8_steps",
    "binary_matmul_backward", "binary_matmul_backward_work_bytes",
    "vocab_loss", "vocab_loss_backward", "vocab_loss_work_bytes",
    "VocabLogprobs", "vocab_logprobs", "vocab_logprobs_work_bytes",
    "VocabDistill", "vocab_distill", "vocab_distill_backward", "vocab_distill_work_bytes",
    "preconditioners", "STERefiner", "cosine_lr", "op_precondition", "op_gram",
    "op_gemm_rhs", "op_sign_gemm", "op_cholesky_inverse", "op_svid", "LBADMM", "lbadmm", "Result",
    "status_string", "version",
]


class NQError(RuntimeError):
    def __init__(self, status: int, where: str):
        lib = _lib.load()
        name = lib.nq_status_string(status).decode()
        msg = lib.nq_last_error_message().decode()
        super().__init__(f"{where}: {name}: {msg}")
        self.status = status


def _check(status: int, where: str):
    if status != NQ_OK:
        raise NQError(status, where)


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _ptr(t, name, dtype=None, ndim=None, allow_none=False, need_contig=True):
    if t is None:
        if allow_none:
            return None
        raise ValueError(f"{name} is required")
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims")
    if need_contig and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return C.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is not None:
        return C.c_void_p(int(stream))
    # the current stream's handle without a Stream object (2.7 us of every call)
    torch = _torch()
    return C.c_void_p(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))


def status_string(status: int) -> str:
    return _lib.load().nq_status_string(status).decode()


def version() -> int:
    return int(_lib.load().nq_version())


def _desc(m, n, r, rho, iters, svid_steps, seed, flags, solve_steps=0) -> Desc:
    return Desc(int(m), int(n), int(r), float(rho), int(iters), int(svid_steps), int(seed),
                int(flags), int(solve_steps))


def lbadmm_workspace_bytes(m, n, r, rho=1.0, iters=50, svid_steps=5, seed=0, flags=0,
                           solve_steps=0) -> int:
    out = C.c_size_t(0)
    d = _desc(m, n, r, rho, iters, svid_steps, seed, flags, solve_steps)
    _check(_lib.load().nq_lbadmm_workspace_bytes(C.byref(d), C.byref(out)),
           "nq_lbadmm_workspace_bytes")
    return int(out.value)


def lbadmm_create(m, n, r, rho=1.0, iters=50, svid_steps=5, seed=0,
                  flags=NQ_FLAG_COMPUTE_ERROR, solve_steps=0) -> int:
    h = C.c_void_p(0)
    d = _desc(m, n, r, rho, iters, svid_steps, seed, flags, solve_steps)
    _check(_lib.load().nq_lbadmm_create(C.byref(d), C.byref(h)), "nq_lbadmm_create")
    return h.value


def _stats_dict(s: Stats) -> dict:
    return {f: getattr(s, f) for f, _ in Stats._fields_ if f != "reserved"}


def lbadmm_run(h, W, d_out, d_in, U0=None, V0=None, U=None, V=None, s1=None, s2=None,
               U_bits=None, V_bits=None, want_stats=True, stream=None):
    """Enqueue one full per-layer run. Returns the stats dict when want_stats
    (the call then waits for the stream), else None."""
    torch = _torch()
    f32 = torch.float32
    if W is None or W.dim() != 2 or W.stride(1) != 1:
        raise ValueError("W must be a 2-D tensor with unit column stride")
    pW = _ptr(W, "W", f32, 2, need_contig=False)
    st = Stats()
    status = _lib.load().nq_lbadmm_run(
        C.c_void_p(h), pW, W.stride(0), _ptr(d_out, "d_out", f32, 1), _ptr(d_in, "d_in", f32, 1),
        _ptr(U0, "U0", f32, 2, True), _ptr(V0, "V0", f32, 2, True),
        _ptr(U, "U", f32, 2, True), _ptr(V, "V", f32, 2, True),
        _ptr(s1, "s1", f32, 1, True), _ptr(s2, "s2", f32, 1, True),
        _ptr(U_bits, "U_bits", torch.int32, 2, True), _ptr(V_bits, "V_bits", torch.int32, 2, True),
        C.byref(st) if want_stats else None, _stream(stream))
    _check(status, "nq_lbadmm_run")
    return _stats_dict(st) if want_stats else None


def lbadmm_query(h):
    st = Stats()
    status = _lib.load().nq_lbadmm_query(C.c_void_p(h), C.byref(st))
    return status, _stats_dict(st)


def lbadmm_get_state(h, U=None, V=None, Z_U=None, Lam_U=None, Z_V=None, Lam_V=None, stream=None):
    f32 = _torch().float32
    _check(_lib.load().nq_lbadmm_get_state(
        C.c_void_p(h), _ptr(U, "U", f32, 2, True), _ptr(V, "V", f32, 2, True),
        _ptr(Z_U, "Z_U", f32, 2, True), _ptr(Lam_U, "Lam_U", f32, 2, True),
        _ptr(Z_V, "Z_V", f32, 2, True), _ptr(Lam_V, "Lam_V", f32, 2, True), _stream(stream)),
        "nq_lbadmm_get_state")


def lbadmm_profile(h, reset=False) -> dict:
    """Per-phase device time under NQ_FLAG_PROFILE: {phase: (total_ms, intervals)}."""
    n = len(PHASES)
    ms = (C.c_double * n)()
    cnt = (C.c_int64 * n)()
    _check(_lib.load().nq_lbadmm_profile(C.c_void_p(h), ms, cnt, 1 if reset else 0),
           "nq_lbadmm_profile")
    return {p: (float(ms[i]), int(cnt[i])) for i, p in enumerate(PHASES)}


def lbadmm_time_svid(h, factor, reps=10, stream=None) -> float:
    """Average device ms of one SVID + dual update of factor 0 (U) or 1 (V),
    `reps` back to back on the handle's state after a run."""
    ms = C.c_double()
    _check(_lib.load().nq_lbadmm_time_svid(C.c_void_p(h), int(factor), int(reps), _stream(stream),
                                           C.byref(ms)), "nq_lbadmm_time_svid")
    return float(ms.value)


def lbadmm_destroy(h):
    if h:
        _lib.load().nq_lbadmm_destroy(C.c_void_p(h))


def pack_signs(X, bits=None, stream=None):
    """Sign bits of a 2-D float32 tensor (unit column stride): int32 words,
    bit k of word w of row i = [X[i, 32 w + k] >= 0]."""
    torch = _torch()
    if X.dim() != 2 or X.stride(1) != 1:
        raise ValueError("X must be 2-D with unit column stride")
    rows, cols = X.shape
    nw = (cols + 31) // 32
    if bits is None:
        bits = torch.empty((rows, nw), dtype=torch.int32, device=X.device)
    _check(_lib.load().nq_pack_signs(
        _ptr(X, "X", torch.float32, 2, need_contig=False), rows, cols, X.stride(0),
        _ptr(bits, "bits", torch.int32, 2, need_contig=False), bits.stride(0), _stream(stream)),
        "nq_pack_signs")
    return bits


def transpose_signs(bits, rows, cols, out=None, stream=None):
    """Sign bits of the transpose: bits holds rows x cols signs (int32 words,
    rows x ceil(cols/32) or wider, unit column stride); returns (or fills) the
    cols x ceil(rows/32) words of the cols x rows transpose."""
    torch = _torch()
    if bits.dim() != 2 or bits.stride(1) != 1 or bits.shape[0] != rows:
        raise ValueError("bits must be 2-D, rows x words, unit column stride")
    if bits.shape[1] < (cols + 31) // 32:
        raise ValueError(f"bits has {bits.shape[1]} words per row, needs ceil(cols/32)")
    if out is None:
        out = torch.empty((cols, (rows + 31) // 32), dtype=torch.int32, device=bits.device)
    elif (out.dim() != 2 or out.stride(1) != 1 or out.shape[0] < cols
          or out.shape[1] < (rows + 31) // 32):
        raise ValueError(f"out must be 2-D with unit column stride and at least {cols} x "
                         f"{(rows + 31) // 32} words, got {tuple(out.shape)}")
    _check(_lib.load().nq_transpose_signs(
        _ptr(bits, "bits", torch.int32, 2, need_contig=False), rows, cols, bits.stride(0),
        _ptr(out, "out", torch.int32, 2, need_contig=False), out.stride(0), _stream(stream)),
        "nq_transpose_signs")
    return out


def binary_matmul_work_floats(B, n, r):
    """Floats of workspace binary_matmul needs for B inputs of width n and
    rank r: the formula of nq_binary_matmul_work_floats (8 partial sums per
    input and rank, rounded up to 64 floats, then the inputs' bf16 terms,
    3072 floats per 16 inputs and 128 columns of the wider product),
    computed here so that buffer checks need no library call."""
    B, n, r = int(B), int(n), int(r)
    if B < 0 or n < 0 or r < 0:
        return -1
    return -(-8 * B * r // 64) * 64 + 3072 * (-(-B // 16)) * (-(-max(n, r) // 128))


def binary_matmul(U_bits, Vt_bits, s1, s2, X, r, Y=None, work=None, stream=None):
    """Y = X W^T for the factorised layer W = diag(s1) S_U S_V^T diag(s2):
    U_bits (m x ceil(r/32) int32), Vt_bits (r x ceil(n/32) int32, from
    transpose_signs of the run's V_bits), s1 (m), s2 (n), X (B x n float32,
    or a vector of length n); work, if given, holds
    binary_matmul_work_floats(B, n, r) float32 (16-byte aligned). Returns Y
    (B x m, or length m)."""
    torch = _torch()
    vec = X.dim() == 1
    X2 = X.unsqueeze(0) if vec else X
    if X2.dim() != 2 or X2.stride(1) != 1:
        raise ValueError("X must be 1-D or 2-D with unit column stride")
    B, n = X2.shape
    m = _check_binmm_shapes(U_bits, Vt_bits, s1, s2, n, r)
    Y2 = _binmm_out(Y, B, m, vec, X.device)
    need = binary_matmul_work_floats(B, n, r)
    if work is None:
        work = torch.empty((max(need, 1),), dtype=torch.float32, device=X.device)
    elif work.numel() < need:
        raise ValueError(f"work holds {work.numel()} floats, needs {need}")
    elif work.data_ptr() % 16:
        raise ValueError("work must be 16-byte aligned")
    _check(_lib.load().nq_binary_matmul(
        _ptr(U_bits, "U_bits", torch.int32, 2, need_contig=False), U_bits.stride(0),
        _ptr(Vt_bits, "Vt_bits", torch.int32, 2, need_contig=False), Vt_bits.stride(0),
        m, n, r, _ptr(s1, "s1", torch.float32), _ptr(s2, "s2", torch.float32),
        _ptr(X2, "X", torch.float32, 2, need_contig=False), B, X2.stride(0),
        _ptr(Y2, "Y", torch.float32, 2, need_contig=False), Y2.stride(0),
        _ptr(work, "work", torch.float32), _stream(stream)), "nq_binary_matmul")
    return Y2[0] if vec else Y2


# Workspace limit of binary_matmul_noalloc: its fixed scratch holds 2^23
# floats, so binary_matmul_work_floats(B, n, r) must not exceed that
NOALLOC_MAX_FLOATS = 1 << 23


def binary_matmul_noalloc(U_bits, Vt_bits, s1, s2, X, r, Y, stream=None):
    """binary_matmul into a caller-given Y with no device allocation: the
    library's fixed per-GPU scratch is the workspace, so
    binary_matmul_work_floats(B, n, r) must not exceed NOALLOC_MAX_FLOATS.
    Calls that overlap on one GPU race; calls ordered on one stream do not.
    Returns Y."""
    torch = _torch()
    vec = X.dim() == 1
    X2 = X.unsqueeze(0) if vec else X
    if X2.dim() != 2 or X2.stride(1) != 1:
        raise ValueError("X must be 1-D or 2-D with unit column stride")
    B, n = X2.shape
    m = _check_binmm_shapes(U_bits, Vt_bits, s1, s2, n, r)
    if Y is None:
        raise ValueError("Y is required: this entry point allocates nothing")
    Y2 = _binmm_out(Y, B, m, vec, X.device)
    need = binary_matmul_work_floats(B, n, r)
    if need > NOALLOC_MAX_FLOATS:
        raise ValueError(f"the call needs {need} floats of workspace, more than the fixed "
                         f"scratch ({NOALLOC_MAX_FLOATS})")
    _check(_lib.load().nq_binary_matmul_noalloc(
        _ptr(U_bits, "U_bits", torch.int32, 2, need_contig=False), U_bits.stride(0),
        _ptr(Vt_bits, "Vt_bits", torch.int32, 2, need_contig=False), Vt_bits.stride(0),
        m, n, r, _ptr(s1, "s1", torch.float32), _ptr(s2, "s2", torch.float32),
        _ptr(X2, "X", torch.float32, 2, need_contig=False), B, X2.stride(0),
        _ptr(Y2, "Y", torch.float32, 2, need_contig=False), Y2.stride(0), _stream(stream)),
        "nq_binary_matmul_noalloc")
    return Y


def _check_binmm_shapes(U_bits, Vt_bits, s1, s2, n, r):
    """Checks the factor operands of the binary-layer product against n and r
    (the C ABI cannot see buffer sizes); returns m."""
    for t, name in ((U_bits, "U_bits"), (Vt_bits, "Vt_bits")):
        if t.dim() != 2 or t.stride(1) != 1:
            raise ValueError(f"{name} must be 2-D with unit column stride")
    m = U_bits.shape[0]
    if U_bits.shape[1] < (r + 31) // 32:
        raise ValueError(f"U_bits has {U_bits.shape[1]} words per row, needs ceil(r/32)")
    if Vt_bits.shape[0] != r or Vt_bits.shape[1] < (n + 31) // 32:
        raise ValueError(f"Vt_bits must be r x (>= ceil(n/32)) words, got {tuple(Vt_bits.shape)}")
    if s1.numel() != m or s2.numel() != n:
        raise ValueError("s1 must hold m and s2 n values")
    return m


def _binmm_out(Y, B, m, vec, device):
    """Y as a B x m view with unit column stride (a vector when X is one),
    allocated when None."""
    torch = _torch()
    if Y is None:
        return torch.empty((B, m), dtype=torch.float32, device=device)
    Y2 = Y.unsqueeze(0) if (vec and Y.dim() == 1) else Y
    if Y2.dim() != 2 or Y2.stride(1) != 1 or Y2.shape[0] < B or Y2.shape[1] < m:
        raise ValueError(f"Y must be 2-D with unit column stride and at least {B} x {m}, "
                         f"got {tuple(Y.shape)}")
    return Y2


# ---------------------------------------------------------------- tuning a packed model

# consecutive columns of a row that share one exponent of an 8-bit checkpoint
ACT8_GROUP = 32


@dataclass
class Act8:
    """8-bit checkpoint of a rows x cols activation matrix: codes (rows x cols
    int8) and exps (rows x ceil(cols/32) uint8); the value of a code is
    code * 2^(exps - 127), NaN in a group whose exps is 255. dtype is the type
    of the activations it was made from (what act8_dequantize returns)."""
    codes: "object"
    exps: "object"
    dtype: "object" = None

    @property
    def shape(self):
        return tuple(self.codes.shape)


_DTYPES = {}   # torch type -> nq_dtype, filled on first use


def _dtype_code(dtype, name):
    if not _DTYPES:
        torch = _torch()
        _DTYPES.update({torch.float32: _lib.NQ_F32, torch.bfloat16: _lib.NQ_BF16,
                        torch.float16: _lib.NQ_F16})
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {dtype}")
    return code


def _matrix(t, name, rows=None, cols=None, dtype=None):
    """Checks that t is a 2-D tensor with unit column stride and rows that do
    not overlap (of the given size and type where given); returns its rows,
    columns and row stride (a single row's is not what it says)."""
    if not isinstance(t, _torch().Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    nr, nc = t.shape
    if (rows is not None and nr != rows) or (cols is not None and nc != cols):
        raise ValueError(f"{name} must be {'any' if rows is None else rows} x "
                         f"{'any' if cols is None else cols}, got {nr} x {nc}")
    ld, step = t.stride()
    if nr == 0 or nc == 0:
        return nr, nc, max(nc, 1)
    if nc > 1 and step != 1:
        raise ValueError(f"{name} must have unit column stride")
    if nr == 1:
        return nr, nc, nc
    if ld < nc:
        raise ValueError(f"{name}'s rows overlap (row stride {ld})")
    return nr, nc, ld


def _vector(t, name, n, dtype):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of {n} values")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


class _OnDevice:
    """The GPU `index`, and calls on it."""

    def __init__(self, index):
        self.index = index

    def call(self, stream, f):
        """f(handle) with this GPU the current one, and with `stream`, if one
        is given, the current stream: what f allocates belongs to the stream
        that uses it."""
        torch = _torch()
        cuda = torch.cuda
        if stream is None and cuda.current_device() == self.index:
            return f(torch._C._cuda_getCurrentRawStream(self.index))
        with cuda.device(self.index):
            if stream is None:
                return f(torch._C._cuda_getCurrentRawStream(self.index))
            stream = int(stream)
            with cuda.stream(cuda.ExternalStream(stream, self.index) if stream
                             else cuda.default_stream(self.index)):
                return f(stream)


def _on_device(names, *tensors):
    """Checks that every tensor (or None) lies on one GPU and returns it as an
    _OnDevice; names: the tensors', separated by spaces."""
    dev = None
    for i, t in enumerate(tensors):
        if t is None:
            continue
        d = t.device
        if dev is None:
            dev = d
            if d.type != "cuda":
                raise TypeError(f"{names.split()[i]} must be a CUDA (HIP) tensor")
        elif d != dev:
            raise ValueError(f"{names.split()[i]} is on {d}, the others on {dev}")
    return _OnDevice(dev.index)


def _p(t):
    return None if t is None else t.data_ptr()


def _workspace(work, need, device):
    """The workspace of a call: a new one, or the caller's after a check."""
    torch = _torch()
    if work is None:
        return torch.empty((max(need, 1),), dtype=torch.uint8, device=device)
    if not isinstance(work, torch.Tensor) or not work.is_contiguous():
        raise ValueError("work must be a contiguous tensor")
    if work.numel() * work.element_size() < need:
        raise ValueError(f"work holds {work.numel() * work.element_size()} bytes, needs {need}")
    if work.data_ptr() % 16:
        raise ValueError("work must be 16-byte aligned")
    return work


def _act8(q, name, rows=None, cols=None):
    """Checks a checkpoint; returns its rows, columns and the row strides of
    its codes and exponents."""
    torch = _torch()
    if not isinstance(q, Act8):
        raise TypeError(f"{name} must be an Act8")
    rows, cols, ldc = _matrix(q.codes, f"{name}.codes", rows, cols, torch.int8)
    _, _, lde = _matrix(q.exps, f"{name}.exps", rows, -(-cols // ACT8_GROUP), torch.uint8)
    return rows, cols, ldc, lde


def act8_quantize(X, q=None, stream=None):
    """8-bit checkpoint of X (rows x cols float32, bfloat16 or float16, unit
    column stride): 32 consecutive columns of a row share a power-of-two step,
    the least with max|x| <= 127 steps. q, if given, is an Act8 of that shape
    to fill. A group with a NaN or an infinity reads back as NaN."""
    torch = _torch()
    rows, cols, ldx = _matrix(X, "X")
    code = _dtype_code(X.dtype, "X")
    groups = -(-cols // ACT8_GROUP)
    ldc, lde = max(cols, 1), max(groups, 1)
    if q is not None:
        _, _, ldc, lde = _act8(q, "q", rows, cols)
        on = _on_device("X codes exps", X, q.codes, q.exps)
    else:
        on = _on_device("X", X)

    def run(handle):
        o = q
        if o is None:
            o = Act8(torch.empty((rows, cols), dtype=torch.int8, device=X.device),
                     torch.empty((rows, groups), dtype=torch.uint8, device=X.device))
        o.dtype = X.dtype
        _check(_lib.load().nq_act8_quantize(_p(X), code, rows, cols, ldx, _p(o.codes), ldc,
                                            _p(o.exps), lde, handle), "nq_act8_quantize")
        return o
    return on.call(stream, run)


def act8_dequantize(q, out=None, dtype=None, stream=None):
    """The activations of a checkpoint, in dtype (default: the type they had,
    float32 when q does not say), or into out."""
    torch = _torch()
    rows, cols, ldc, lde = _act8(q, "q")
    if out is not None:
        _, _, ldo = _matrix(out, "out", rows, cols, dtype)
        dtype = out.dtype
    else:
        dtype, ldo = dtype or q.dtype or torch.float32, max(cols, 1)
    code = _dtype_code(dtype, "out")
    on = _on_device("codes exps out", q.codes, q.exps, out)

    def run(handle):
        o = out
        if o is None:
            o = torch.empty((rows, cols), dtype=dtype, device=q.codes.device)
        _check(_lib.load().nq_act8_dequantize(_p(q.codes), ldc, _p(q.exps), lde, rows, cols,
                                              _p(o), code, ldo, handle), "nq_act8_dequantize")
        return o
    return on.call(stream, run)


def act8_steps(q, stream=None):
    """The step of each group of a checkpoint (rows x ceil(cols/32) float32,
    powers of two, NaN for a group that was not finite)."""
    torch = _torch()
    _, _, _, lde = _act8(q, "q")
    rows, groups = q.exps.shape

    def run(handle):
        steps = torch.empty((rows, groups), dtype=torch.float32, device=q.exps.device)
        _check(_lib.load().nq_act8_steps(_p(q.exps), lde, rows, groups, _p(steps),
                                         max(groups, 1), handle), "nq_act8_steps")
        return steps
    return _on_device("exps", q.exps).call(stream, run)


def binary_matmul_backward_work_bytes(T, m, n, r):
    """Bytes of workspace binary_matmul_backward needs for T tokens."""
    return int(_lib.load().nq_binary_matmul_backward_work_bytes(int(T), int(m), int(n), int(r)))


def binary_matmul_backward(U_bits, Ut_bits, V_bits, Vt_bits, s1, s2, X, dY, r, want_dX=True,
                           dX=None, ds1=None, ds2=None, work=None, stream=None):
    """Gradient of binary_matmul's layer Y = X W^T, W = diag(s1) S_U S_V^T
    diag(s2), with the signs held: returns (dX, ds1, ds2) for dY = dL/dY
    (T x m float32, bfloat16 or float16) from the 8-bit checkpoint X (an Act8,
    T x n) of the layer's input. U_bits (m x ceil(r/32) int32 words) and V_bits
    (n x ceil(r/32)) as lbadmm_run returns them, Ut_bits (r x ceil(m/32)) and
    Vt_bits (r x ceil(n/32)) their transposes (transpose_signs). dX (T x n) has
    dY's type (None with want_dX=False); ds1 (m) and ds2 (n) are float32 sums
    over the tokens. Outputs must not share memory with inputs. work, if given,
    holds binary_matmul_backward_work_bytes(T, m, n, r) bytes, 16-byte
    aligned."""
    torch = _torch()
    f32, i32 = torch.float32, torch.int32
    T, n, ldc, lde = _act8(X, "X")
    r = int(r)
    m, words, ldu = _matrix(U_bits, "U_bits", dtype=i32)
    got = [(m, words), None, None, None]
    lds = [ldu, 0, 0, 0]
    for k, (t, name) in enumerate(((Ut_bits, "Ut_bits"), (V_bits, "V_bits"), (Vt_bits, "Vt_bits"))):
        nr, nc, lds[k + 1] = _matrix(t, name, dtype=i32)
        got[k + 1] = (nr, nc)
    for (nr, nc), name, rows, cols in zip(got, ("U_bits", "Ut_bits", "V_bits", "Vt_bits"),
                                          (m, r, n, r), (r, m, r, n)):
        if nr != rows or nc < (cols + 31) // 32:
            raise ValueError(f"{name} must be {rows} x (>= {(cols + 31) // 32}) words, "
                             f"got {nr} x {nc}")
    _vector(s1, "s1", m, f32)
    _vector(s2, "s2", n, f32)
    _, _, lddy = _matrix(dY, "dY", T, m)
    code = _dtype_code(dY.dtype, "dY")
    if dX is not None:
        _, _, lddx = _matrix(dX, "dX", T, n, dY.dtype)
    else:
        lddx = max(n, 1)
    if ds1 is not None:
        _vector(ds1, "ds1", m, f32)
    if ds2 is not None:
        _vector(ds2, "ds2", n, f32)
    if min(m, n, r) < 1:
        raise ValueError("m, n and r must be >= 1")
    on = _on_device("U_bits Ut_bits V_bits Vt_bits s1 s2 codes exps dY dX ds1 ds2 work", U_bits,
                    Ut_bits, V_bits, Vt_bits, s1, s2, X.codes, X.exps, dY, dX, ds1, ds2, work)

    def run(handle):
        def out(t, shape, dtype):
            return torch.empty(shape, dtype=dtype, device=dY.device) if t is None else t
        x = out(dX, (T, n), dY.dtype) if want_dX or dX is not None else None
        g1, g2 = out(ds1, m, f32), out(ds2, n, f32)
        lib = _lib.load()
        w = _workspace(work, lib.nq_binary_matmul_backward_work_bytes(T, m, n, r), dY.device)
        _check(lib.nq_binary_matmul_backward(
            _p(U_bits), lds[0], _p(Ut_bits), lds[1], _p(V_bits), lds[2], _p(Vt_bits), lds[3], m, n,
            r, _p(s1), _p(s2), _p(X.codes), ldc, _p(X.exps), lde, T, _p(dY), code, lddy, _p(x),
            lddx, _p(g1), _p(g2), _p(w), handle), "nq_binary_matmul_backward")
        return x, g1, g2
    return on.call(stream, run)


def vocab_loss_work_bytes(T, V, d, dtype, grad=False):
    """Bytes of workspace vocab_loss (or, with grad, vocab_loss_backward)
    needs for T tokens, V words, hidden size d and H, W of dtype."""
    return int(_lib.load().nq_vocab_loss_work_bytes(int(T), int(V), int(d),
                                                    _dtype_code(dtype, "dtype"), int(bool(grad))))


def _head_args(H, W):
    T, d, ldh = _matrix(H, "H")
    V, _, ldw = _matrix(W, "W", None, d, H.dtype)
    code = _dtype_code(H.dtype, "H")
    if V < 1 or d < 1:
        raise ValueError("the vocabulary and the hidden size must be >= 1")
    return T, V, d, code, ldh, ldw


def _vocab_args(H, W, labels):
    args = _head_args(H, W)
    _vector(labels, "labels", args[0], _torch().int32)
    return args


def vocab_loss(H, W, labels, scale=1.0, loss=None, lse=None, work=None, stream=None):
    """Softmax cross entropy of logits z = scale H W^T, which are never kept:
    H (T x d) and W (V x d) float32, bfloat16 or float16 with unit column
    stride, labels (T) int32. Returns (loss, lse), T float32 each:
    lse = log sum exp z, loss = lse - z[label]. A negative label is ignored
    (loss and lse 0, its row of H is not used); a label >= V gives NaN. work,
    if given, holds vocab_loss_work_bytes(T, V, d, H.dtype) bytes."""
    torch = _torch()
    f32 = torch.float32
    T, V, d, code, ldh, ldw = _vocab_args(H, W, labels)
    if loss is not None:
        _vector(loss, "loss", T, f32)
    if lse is not None:
        _vector(lse, "lse", T, f32)
    on = _on_device("H W labels loss lse work", H, W, labels, loss, lse, work)

    def run(handle):
        a = torch.empty(T, dtype=f32, device=H.device) if loss is None else loss
        b = torch.empty(T, dtype=f32, device=H.device) if lse is None else lse
        lib = _lib.load()
        w = _workspace(work, lib.nq_vocab_loss_work_bytes(T, V, d, code, 0), H.device)
        _check(lib.nq_vocab_loss(_p(H), ldh, _p(W), ldw, code, T, V, d, _p(labels), float(scale),
                                 _p(a), _p(b), _p(w), handle), "nq_vocab_loss")
        return a, b
    return on.call(stream, run)


def vocab_loss_backward(H, W, labels, lse, dloss, scale=1.0, want_dH=True, want_dW=True, dH=None,
                        dW=None, work=None, stream=None):
    """Gradient of sum(dloss * loss) for vocab_loss(H, W, labels, scale), from
    its lse (of one call with these tokens): returns (dH, dW) in H's type (None where not wanted). lse and
    dloss are T float32. The logits are computed again in pieces of the
    vocabulary. Ignored tokens (negative labels) get zero rows of dH and add
    nothing to dW. Outputs must not share memory with inputs. work, if given,
    holds vocab_loss_work_bytes(T, V, d, H.dtype, grad=True) bytes."""
    torch = _torch()
    T, V, d, code, ldh, ldw = _vocab_args(H, W, labels)
    _vector(lse, "lse", T, torch.float32)
    _vector(dloss, "dloss", T, torch.float32)
    lddh = lddw = d
    if dH is not None:
        _, _, lddh = _matrix(dH, "dH", T, d, H.dtype)
    if dW is not None:
        _, _, lddw = _matrix(dW, "dW", V, d, H.dtype)
    want_dH, want_dW = want_dH or dH is not None, want_dW or dW is not None
    if not (want_dH or want_dW):
        raise ValueError("neither dH nor dW is wanted")
    on = _on_device("H W labels lse dloss dH dW work", H, W, labels, lse, dloss, dH, dW, work)

    def run(handle):
        gH, gW = dH, dW
        if want_dH and gH is None:
            gH = torch.empty((T, d), dtype=H.dtype, device=H.device)
        if want_dW and gW is None:
            gW = torch.empty((V, d), dtype=H.dtype, device=H.device)
        if T == 0:
            if gW is not None:
                gW.zero_()
            return gH, gW
        lib = _lib.load()
        w = _workspace(work, lib.nq_vocab_loss_work_bytes(T, V, d, code, 1), H.device)
        _check(lib.nq_vocab_loss_backward(
            _p(H), ldh, _p(W), ldw, code, T, V, d, _p(labels), float(scale), _p(lse), _p(dloss),
            _p(gH), lddh, _p(gW), lddw, _p(w), handle), "nq_vocab_loss_backward")
        return gH, gW
    return on.call(stream, run)


# words that a token can list or be given, and its best words at most
VOCAB_MAX_LISTED = 128


@dataclass
class VocabLogprobs:
    """What vocab_logprobs finds for T rows: logprobs (the shape of tokens; None
    without), entropy and lse (T), top_ids (T x k int32) and top_logprobs (T x k);
    float32 unless said otherwise."""
    logprobs: "object"
    entropy: "object"
    lse: "object"
    top_ids: "object"
    top_logprobs: "object"


def vocab_logprobs_work_bytes(T, V, d, dtype, given=0, k=0):
    """Bytes of workspace vocab_logprobs needs for T rows, V words, hidden size d,
    H and W of dtype, `given` tokens per row and k best words."""
    return int(_lib.load().nq_vocab_logprobs_work_bytes(
        int(T), int(V), int(d), _dtype_code(dtype, "dtype"), int(given), int(k)))


def vocab_logprobs(H, W, tokens=None, k=0, scale=1.0, out=None, work=None, stream=None):
    """Log probabilities under softmax of z = scale H W^T, which never leaves the call: H
    (T x d) and W (V x d) float32, bfloat16 or float16 with unit column stride.
    tokens (T, or T x G with G <= 128; int32): the words whose log probability is
    wanted, a negative one gives 0, one >= V NaN. Returns a VocabLogprobs with those,
    each row's entropy and lse = log sum exp z, and its k best words (k <= 128) with
    their log probabilities, best first, the lower word first among equals. out, if
    given, is a VocabLogprobs of contiguous tensors to fill; work holds
    vocab_logprobs_work_bytes(T, V, d, H.dtype, G, k) bytes. A row with a logit that
    is not finite has NaN and the words -1."""
    torch = _torch()
    f32, i32 = torch.float32, torch.int32
    T, V, d, code, ldh, ldw = _head_args(H, W)
    k, given, ldt = int(k), 0, 1
    if not 0 <= k <= min(VOCAB_MAX_LISTED, V):
        raise ValueError(f"k must be in 0 .. {min(VOCAB_MAX_LISTED, V)}")
    if tokens is not None:
        flat = isinstance(tokens, torch.Tensor) and tokens.dim() == 1
        if flat:
            _vector(tokens, "tokens", T, i32)
            given = 1
        else:
            _, given, ldt = _matrix(tokens, "tokens", T, None, i32)
        if given > VOCAB_MAX_LISTED:
            raise ValueError(f"a row has at most {VOCAB_MAX_LISTED} tokens")
    if out is not None:
        if not isinstance(out, VocabLogprobs):
            raise TypeError("out must be a VocabLogprobs")
        if tokens is not None:
            _vector(out.logprobs, "out.logprobs", T * given, f32)
        _vector(out.entropy, "out.entropy", T, f32)
        _vector(out.lse, "out.lse", T, f32)
        if k:
            _vector(out.top_ids, "out.top_ids", T * k, i32)
            _vector(out.top_logprobs, "out.top_logprobs", T * k, f32)
        on = _on_device("H W tokens logprobs entropy lse top_ids top_logprobs work", H, W, tokens,
                        out.logprobs, out.entropy, out.lse, out.top_ids, out.top_logprobs, work)
    else:
        on = _on_device("H W tokens work", H, W, tokens, work)

    def run(handle):
        o = out
        if o is None:
            def new(shape, dtype=f32):
                return torch.empty(shape, dtype=dtype, device=H.device)
            o = VocabLogprobs(None if tokens is None else new(tokens.shape), new(T), new(T),
                              new((T, k), i32), new((T, k)))
        lib = _lib.load()
        w = _workspace(work, lib.nq_vocab_logprobs_work_bytes(T, V, d, code, given, k), H.device)
        _check(lib.nq_vocab_logprobs(
            _p(H), ldh, _p(W), ldw, code, T, V, d, _p(tokens), ldt, given, k, float(scale),
            _p(o.logprobs), _p(o.entropy), _p(o.lse), _p(o.top_ids), _p(o.top_logprobs), _p(w),
            handle), "nq_vocab_logprobs")
        return o
    return on.call(stream, run)


@dataclass
class VocabDistill:
    """What vocab_distill hands to its gradient for T tokens with K entries each: lse
    and rest (T) and hit (T x K), float32; and, where it pays (up to 4 GiB), the
    logits (T x V to the next multiple of 128), which the gradient then need not
    compute again. They can be left out (None)."""
    lse: "object"
    rest: "object"
    hit: "object"
    logits: "object" = None


def vocab_distill_work_bytes(T, V, d, dtype, K, grad=False):
    """Bytes of workspace vocab_distill (or, with grad, vocab_distill_backward) needs
    for T tokens of K entries, V words, hidden size d and H, W of dtype."""
    return int(_lib.load().nq_vocab_distill_work_bytes(
        int(T), int(V), int(d), _dtype_code(dtype, "dtype"), int(K), int(bool(grad))))


def _distill_args(H, W, ids, logq):
    torch = _torch()
    T, V, d, code, ldh, ldw = _head_args(H, W)
    _, K, ldi = _matrix(ids, "ids", T, None, torch.int32)
    _, _, ldq = _matrix(logq, "logq", T, K, torch.float32)
    if not 1 <= K <= VOCAB_MAX_LISTED:
        raise ValueError(f"a token lists 1 .. {VOCAB_MAX_LISTED} words")
    return T, V, d, code, ldh, ldw, K, ldi, ldq


def _distill_state(q, T, V, K):
    f32 = _torch().float32
    if not isinstance(q, VocabDistill):
        raise TypeError("the loss's state must be a VocabDistill")
    _vector(q.lse, "lse", T, f32)
    _vector(q.rest, "rest", T, f32)
    _vector(q.hit, "hit", T * K, f32)
    if q.logits is not None:
        _vector(q.logits, "logits", T * -(-V // 128) * 128, f32)
        if q.logits.data_ptr() % 16:
            raise ValueError("logits must be 16-byte aligned")


def vocab_distill(H, W, ids, logq, scale=1.0, tail=True, keep=True, loss=None, state=None, work=None,
                  stream=None):
    """KL divergence of softmax(z), z = scale H W^T, from a teacher's K <= 128
    words per token: ids (T x K int32; a negative one is no entry, a token without
    any is ignored) and their log probabilities logq (T x K float32), as
    vocab_logprobs gives them for the teacher (at its own scale: one over the
    temperature). tail: the rest of the teacher's mass, 1 - sum exp logq, is one
    outcome more, "another word"; without it logq is normalised over a token's
    entries (and may be logits). Returns (loss, state): T float32, 0 for an ignored
    token, and the VocabDistill that vocab_distill_backward takes (keep: with the
    logits, up to 4 GiB, where that saves the gradient more time than their store costs;
    keep=False for a loss without a gradient); both can be given to be filled. A word
    >= V gives NaN; one listed twice counts with both entries; without tail, a row of
    nothing but -infinity has no softmax and gives NaN. work, if given, holds vocab_distill_work_bytes(T, V, d, H.dtype, K) bytes."""
    torch = _torch()
    f32 = torch.float32
    T, V, d, code, ldh, ldw, K, ldi, ldq = _distill_args(H, W, ids, logq)
    if loss is not None:
        _vector(loss, "loss", T, f32)
    if state is not None:
        _distill_state(state, T, V, K)
        given = (state.lse, state.rest, state.hit, state.logits)
    else:
        given = (None, None, None, None)
    on = _on_device("H W ids logq loss lse rest hit logits work", H, W, ids, logq, loss, *given, work)

    def run(handle):
        def new(*shape):
            return torch.empty(shape, dtype=f32, device=H.device)
        a = new(T) if loss is None else loss
        lib = _lib.load()
        q = state
        if q is None:
            kept = lib.nq_vocab_distill_logits(T, V, d, code) if keep else 0
            q = VocabDistill(new(T), new(T), new(T, K), new(T, kept // T) if kept > 0 else None)
        w = _workspace(work, lib.nq_vocab_distill_work_bytes(T, V, d, code, K, 0), H.device)
        _check(lib.nq_vocab_distill(
            _p(H), ldh, _p(W), ldw, code, T, V, d, _p(ids), ldi, _p(logq), ldq, K, float(scale),
            int(bool(tail)), _p(a), _p(q.lse), _p(q.rest), _p(q.hit), _p(q.logits), _p(w), handle),
            "nq_vocab_distill")
        return a, q
    return on.call(stream, run)


def vocab_distill_backward(H, W, ids, logq, state, dloss, scale=1.0, tail=True, want_dH=True,
                           want_dW=True, dH=None, dW=None, work=None, stream=None):
    """Gradient of sum(dloss * loss) for (loss, state) = vocab_distill(H, W, ids,
    logq, scale, tail) of one call with these tokens: returns (dH, dW) in H's type
    (None where not wanted). dloss is T float32. Where state has no logits they are
    computed again, in pieces of the vocabulary, with the same roundings. Ignored tokens get zero rows of dH and add nothing to
    dW. Outputs must not share memory with inputs. work, if given, holds
    vocab_distill_work_bytes(T, V, d, H.dtype, K, grad=True) bytes."""
    torch = _torch()
    T, V, d, code, ldh, ldw, K, ldi, ldq = _distill_args(H, W, ids, logq)
    _distill_state(state, T, V, K)
    _vector(dloss, "dloss", T, torch.float32)
    lddh = lddw = d
    if dH is not None:
        _, _, lddh = _matrix(dH, "dH", T, d, H.dtype)
    if dW is not None:
        _, _, lddw = _matrix(dW, "dW", V, d, H.dtype)
    want_dH, want_dW = want_dH or dH is not None, want_dW or dW is not None
    if not (want_dH or want_dW):
        raise ValueError("neither dH nor dW is wanted")
    on = _on_device("H W ids logq lse rest hit logits dloss dH dW work", H, W, ids, logq, state.lse,
                    state.rest, state.hit, state.logits, dloss, dH, dW, work)

    def run(handle):
        gH, gW = dH, dW
        if want_dH and gH is None:
            gH = torch.empty((T, d), dtype=H.dtype, device=H.device)
        if want_dW and gW is None:
            gW = torch.empty((V, d), dtype=H.dtype, device=H.device)
        if T == 0:
            if gW is not None:
                gW.zero_()
            return gH, gW
        lib = _lib.load()
        w = _workspace(work, lib.nq_vocab_distill_work_bytes(T, V, d, code, K, 1), H.device)
        _check(lib.nq_vocab_distill_backward(
            _p(H), ldh, _p(W), ldw, code, T, V, d, _p(ids), ldi, _p(logq), ldq, K, float(scale),
            int(bool(tail)), _p(state.lse), _p(state.rest), _p(state.hit), _p(state.logits), _p(dloss),
            _p(gH), lddh, _p(gW), lddw, _p(w), handle), "nq_vocab_distill_backward")
        return gH, gW
    return on.call(stream, run)


class LedoitWolf:
    """Running Ledoit-Wolf statistics of activation samples with p features
    (nq_lw_*): accumulate() chunks of tokens x p float32 samples, then
    finalize() -> (d, shrinkage), d the diagonal of the preconditioner
    sqrt(diag(shrunk second moment)) as a float32 device vector."""

    def __init__(self, p, max_rows=16384):
        h = C.c_void_p(0)
        _check(_lib.load().nq_lw_create(int(p), int(max_rows), C.byref(h)), "nq_lw_create")
        self.handle, self.p = h.value, int(p)

    def accumulate(self, Z, stream=None):
        torch = _torch()
        if Z.dim() != 2 or Z.shape[1] != self.p or Z.stride(1) != 1:
            raise ValueError(f"Z must be rows x {self.p} with unit column stride")
        _check(_lib.load().nq_lw_accumulate(
            C.c_void_p(self.handle), _ptr(Z, "Z", torch.float32, 2, need_contig=False),
            Z.shape[0], Z.stride(0), _stream(stream)), "nq_lw_accumulate")

    def finalize(self, d=None, stream=None):
        torch = _torch()
        if d is None:
            dev = torch.device("cuda", torch.cuda.current_device())
            d = torch.empty(self.p, dtype=torch.float32, device=dev)
        elif d.numel() != self.p:
            raise ValueError(f"d must hold {self.p} values")
        shrink = C.c_double(0.0)
        _check(_lib.load().nq_lw_finalize(C.c_void_p(self.handle), _ptr(d, "d", torch.float32),
                                          C.byref(shrink), _stream(stream)), "nq_lw_finalize")
        return d, shrink.value

    def reset(self):
        _check(_lib.load().nq_lw_reset(C.c_void_p(self.handle)), "nq_lw_reset")

    def close(self):
        if getattr(self, "handle", None):
            _lib.load().nq_lw_destroy(C.c_void_p(self.handle))
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def ledoit_wolf_diag(Z, max_rows=16384, stream=None):
    """(d, shrinkage) for one sample matrix Z (device, tokens x p float32)."""
    with LedoitWolf(Z.shape[1], min(max_rows, max(1, Z.shape[0]))) as lw:
        lw.accumulate(Z, stream)
        return lw.finalize(stream=stream)


def preconditioners(X_in, Z_out, max_rows=16384, stream=None):
    """(d_out, d_in) of a layer from its input-side sample X_in (N x n) and
    output-side sample Z_out (N x m), ready for nq_lbadmm_run."""
    d_in, _ = ledoit_wolf_diag(X_in, max_rows, stream)
    d_out, _ = ledoit_wolf_diag(Z_out, max_rows, stream)
    return d_out, d_in


def cosine_lr(t, K, lr_max=1e-4, lr_min=1e-6):
    """Learning rate of step t (0-based) of K on the cosine schedule."""
    import math
    return lr_min + (lr_max - lr_min) * (1.0 + math.cos(math.pi * t / K)) / 2.0


class STERefiner:
    """STE refinement of one factorised layer (nq_ste_*): set_params() from
    a run's U, V, s1, s2, then step() per batch (X, Y = X W^T device float32,
    X also as its 8-bit checkpoint, an Act8;
    rows: an int32 device index vector or None), or refine() over a list of
    batches with the cosine schedule."""

    def __init__(self, m, n, r, max_tokens):
        h = C.c_void_p(0)
        _check(_lib.load().nq_ste_create(int(m), int(n), int(r), int(max_tokens), C.byref(h)),
               "nq_ste_create")
        self.handle, self.m, self.n, self.r = h.value, int(m), int(n), int(r)
        self.max_tokens = int(max_tokens)

    def set_params(self, U, V, s1, s2, stream=None):
        torch = _torch()
        f32 = torch.float32
        if (tuple(U.shape) != (self.m, self.r) or tuple(V.shape) != (self.n, self.r)
                or s1.numel() != self.m or s2.numel() != self.n):
            raise ValueError("U, V, s1, s2 must be m x r, n x r, m and n")
        _check(_lib.load().nq_ste_set_params(
            C.c_void_p(self.handle), _ptr(U, "U", f32, 2), _ptr(V, "V", f32, 2),
            _ptr(s1, "s1", f32), _ptr(s2, "s2", f32), _stream(stream)), "nq_ste_set_params")

    def step(self, X, Y, lr, rows=None, stream=None, check_rows=True):
        """check_rows: verify on the host that every index is a row of X
        (a device read and a wait; the library cannot see X's length)."""
        torch = _torch()
        f32 = torch.float32
        if isinstance(X, Act8):
            _, _, ldc, lde = _act8(X, "X", None, self.n)
        elif X.dim() != 2 or X.shape[1] != self.n or X.stride(1) != 1:
            raise ValueError(f"X must be tokens x {self.n} with unit column stride")
        if Y.dim() != 2 or Y.shape[1] != self.m or Y.stride(1) != 1 or Y.shape[0] != X.shape[0]:
            raise ValueError(f"Y must be tokens x {self.m}, as many rows as X")
        if rows is None:
            T = X.shape[0]
            rp = None
        else:
            if rows.dtype != torch.int32 or rows.dim() != 1:
                raise ValueError("rows must be a 1-D int32 tensor")
            T = rows.numel()
            rp = _ptr(rows, "rows", torch.int32)
            if check_rows and T and (int(rows.min()) < 0 or int(rows.max()) >= X.shape[0]):
                raise ValueError("rows holds an index outside X")
        if not 1 <= T <= self.max_tokens:
            raise ValueError(f"a batch holds 1 .. {self.max_tokens} tokens")
        if isinstance(X, Act8):
            _on_device("codes exps Y rows", X.codes, X.exps, Y, rows).call(
                stream, lambda handle: _check(_lib.load().nq_ste_step_act8(
                    C.c_void_p(self.handle), _p(X.codes), ldc, _p(X.exps), lde,
                    _ptr(Y, "Y", f32, 2, need_contig=False), _matrix(Y, "Y")[2], rp, T, float(lr),
                    handle), "nq_ste_step_act8"))
            return
        _check(_lib.load().nq_ste_step(
            C.c_void_p(self.handle), _ptr(X, "X", f32, 2, need_contig=False), X.stride(0),
            _ptr(Y, "Y", f32, 2, need_contig=False), Y.stride(0), rp, T, float(lr),
            _stream(stream)), "nq_ste_step")

    def last_loss(self, stream=None):
        out = C.c_double(0.0)
        _check(_lib.load().nq_ste_last_loss(C.c_void_p(self.handle), C.byref(out),
                                            _stream(stream)), "nq_ste_last_loss")
        return out.value

    def params(self, stream=None):
        torch = _torch()
        dev = torch.device("cuda", torch.cuda.current_device())
        f32 = torch.float32
        U = torch.empty((self.m, self.r), dtype=f32, device=dev)
        V = torch.empty((self.n, self.r), dtype=f32, device=dev)
        s1 = torch.empty(self.m, dtype=f32, device=dev)
        s2 = torch.empty(self.n, dtype=f32, device=dev)
        _check(_lib.load().nq_ste_get_params(
            C.c_void_p(self.handle), _ptr(U, "U", f32), _ptr(V, "V", f32), _ptr(s1, "s1", f32),
            _ptr(s2, "s2", f32), _stream(stream)), "nq_ste_get_params")
        return U, V, s1, s2

    def refine(self, X, Y, batches, lr_max=1e-4, lr_min=1e-6, losses=True, stream=None,
               check_rows=True):
        """One step per batch (int32 device index vectors) on the cosine
        schedule from lr_max to lr_min; returns the per-step losses (each
        read back, which waits for the stream) or None."""
        out = [] if losses else None
        K = len(batches)
        for t, rows in enumerate(batches):
            self.step(X, Y, cosine_lr(t, K, lr_max, lr_min), rows, stream, check_rows)
            if losses:
                out.append(self.last_loss(stream))
        return out

    def close(self):
        if getattr(self, "handle", None):
            _lib.load().nq_ste_destroy(C.c_void_p(self.handle))
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def op_precondition(W, d_out, d_in, stream=None):
    torch = _torch()
    m, n = W.shape
    out = torch.empty((m, n), dtype=torch.float32, device=W.device)
    f32 = torch.float32
    _check(_lib.load().nq_op_precondition(
        _ptr(W, "W", f32, 2), n, m, n, _ptr(d_out, "d_out", f32, 1), _ptr(d_in, "d_in", f32, 1),
        _ptr(out, "Wt", f32, 2), n, _stream(stream)), "nq_op_precondition")
    return out


def op_gram(A, rho, stream=None):
    torch = _torch()
    rows, cols = A.shape
    G = torch.empty((cols, cols), dtype=torch.float32, device=A.device)
    _check(_lib.load().nq_op_gram(_ptr(A, "A", torch.float32, 2), rows, cols, cols, float(rho),
                                  _ptr(G, "G", torch.float32, 2), cols, _stream(stream)),
           "nq_op_gram")
    return G


def op_gemm_rhs(A, B, P=None, rho=0.0, stream=None):
    torch = _torch()
    rows, k = A.shape
    k2, cols = B.shape
    if k2 != k:
        raise ValueError("inner dimensions differ")
    Cm = torch.empty((rows, cols), dtype=torch.float32, device=A.device)
    f32 = torch.float32
    _check(_lib.load().nq_op_gemm_rhs(
        _ptr(A, "A", f32, 2), k, _ptr(B, "B", f32, 2), cols, _ptr(P, "P", f32, 2, True), cols,
        float(rho), _ptr(Cm, "C", f32, 2), cols, rows, cols, k, _stream(stream)), "nq_op_gemm_rhs")
    return Cm


def op_sign_gemm(A, S, transposed=False, stream=None):
    """C = A S^T for A (rows x k) and a +-1 matrix S (cols x k), on the bf16
    matrix cores; with transposed=True returns (C, C^T from the kernel)."""
    torch = _torch()
    rows, k = A.shape
    cols, k2 = S.shape
    if k2 != k:
        raise ValueError("A and S must have the same number of columns")
    f32 = torch.float32
    Cm = torch.empty((rows, cols), dtype=f32, device=A.device)
    Ct = torch.empty((cols, rows), dtype=f32, device=A.device) if transposed else None
    _check(_lib.load().nq_op_sign_gemm(
        _ptr(A, "A", f32, 2), k, _ptr(S, "S", f32, 2), k, _ptr(Cm, "C", f32, 2), cols,
        _ptr(Ct, "Ct", f32, 2, True), rows, rows, cols, k, _stream(stream)), "nq_op_sign_gemm")
    return (Cm, Ct) if transposed else Cm


def op_cholesky_inverse(G, stream=None):
    """Returns (L, Ginv, info); raises NQError on a non-positive pivot."""
    torch = _torch()
    r = G.shape[0]
    L = torch.empty((r, r), dtype=torch.float32, device=G.device)
    Gi = torch.empty((r, r), dtype=torch.float32, device=G.device)
    info = C.c_int64(0)
    f32 = torch.float32
    status = _lib.load().nq_op_cholesky_inverse(
        _ptr(G, "G", f32, 2), r, r, _ptr(L, "L", f32, 2), r, _ptr(Gi, "Ginv", f32, 2), r,
        C.byref(info), _stream(stream))
    if status not in (NQ_OK, _lib.NQ_ERR_NOT_POSITIVE_DEFINITE):
        _check(status, "nq_op_cholesky_inverse")
    return L, Gi, int(info.value)


def op_svid(X, T, stream=None):
    torch = _torch()
    rows, cols = X.shape
    f32 = torch.float32
    Z = torch.empty((rows, cols), dtype=f32, device=X.device)
    a = torch.empty((rows,), dtype=f32, device=X.device)
    b = torch.empty((cols,), dtype=f32, device=X.device)
    _check(_lib.load().nq_op_svid(_ptr(X, "X", f32, 2), rows, cols, cols, int(T),
                                  _ptr(Z, "Z", f32, 2), cols, _ptr(a, "a", f32, 1),
                                  _ptr(b, "b", f32, 1), _stream(stream)), "nq_op_svid")
    return Z, a, b


def op_svid_dual(U, Lam, T, stream=None):
    """X = U + Lam, Z = SVID_T(X), Lam_out = X - Z: returns (Z, Lam_out, a, b)."""
    torch = _torch()
    rows, cols = U.shape
    if tuple(Lam.shape) != (rows, cols):
        raise ValueError("U and Lam must have the same shape")
    f32 = torch.float32
    Z = torch.empty((rows, cols), dtype=f32, device=U.device)
    Lo = torch.empty((rows, cols), dtype=f32, device=U.device)
    a = torch.empty((rows,), dtype=f32, device=U.device)
    b = torch.empty((cols,), dtype=f32, device=U.device)
    _check(_lib.load().nq_op_svid_dual(_ptr(U, "U", f32, 2), _ptr(Lam, "Lam", f32, 2), rows, cols,
                                       cols, int(T), _ptr(Z, "Z", f32, 2), _ptr(Lo, "Lam_out", f32, 2),
                                       cols, _ptr(a, "a", f32, 1), _ptr(b, "b", f32, 1),
                                       _stream(stream)), "nq_op_svid_dual")
    return Z, Lo, a, b


@dataclass
class Result:
    U: "object"
    V: "object"
    s1: "object"
    s2: "object"
    U_bits: "object"
    V_bits: "object"
    stats: Optional[dict]


class LBADMM:
    """One handle for one layer shape; reusable across runs of that shape."""

    def __init__(self, m, n, r, rho=1.0, iters=50, svid_steps=5, seed=0, compute_error=True,
                 init_draws=False, balance=True, single_stream=False, profile=False,
                 solver=None):
        """init_draws: U0/V0 passed to run() are standard-normal draws that
        the run scales by sigma0 (default: they are the starting latents).
        profile: False, True (every phase) or "rhs" (only the RHS GEMM).
        solver: None (the Cholesky solve) or (method, steps) with method "cg"
        (conjugate gradients) or "gd" (steepest descent): an iterative solve
        of each half's system, warm-started from the factor's previous value."""
        flags, steps = 0, 0
        if solver is not None:
            method, steps = solver
            if method not in ("cg", "gd"):
                raise ValueError("solver method is 'cg' or 'gd'")
            flags |= NQ_FLAG_SOLVE_CG if method == "cg" else NQ_FLAG_SOLVE_GD
        flags |= NQ_FLAG_PROFILE if profile else 0
        flags |= NQ_FLAG_PROFILE_RHS_ONLY if profile == "rhs" else 0
        flags |= NQ_FLAG_COMPUTE_ERROR if compute_error else 0
        flags |= NQ_FLAG_INIT_DRAWS if init_draws else 0
        flags |= 0 if balance else NQ_FLAG_NO_BALANCE
        flags |= NQ_FLAG_SINGLE_STREAM if single_stream else 0
        self.m, self.n, self.r = int(m), int(n), int(r)
        self.handle = lbadmm_create(m, n, r, rho, iters, svid_steps, seed, flags, steps)

    def alloc_outputs(self, device):
        torch = _torch()
        nw = (self.r + 31) // 32
        f32 = torch.float32
        return dict(U=torch.empty((self.m, self.r), dtype=f32, device=device),
                    V=torch.empty((self.n, self.r), dtype=f32, device=device),
                    s1=torch.empty((self.m,), dtype=f32, device=device),
                    s2=torch.empty((self.n,), dtype=f32, device=device),
                    U_bits=torch.empty((self.m, nw), dtype=torch.int32, device=device),
                    V_bits=torch.empty((self.n, nw), dtype=torch.int32, device=device))

    def run(self, W, d_out, d_in, U0=None, V0=None, out=None, want_stats=True, stream=None):
        if out is None:
            out = self.alloc_outputs(W.device)
        st = lbadmm_run(self.handle, W, d_out, d_in, U0, V0, out["U"], out["V"], out["s1"],
                        out["s2"], out["U_bits"], out["V_bits"], want_stats, stream)
        return Result(out["U"], out["V"], out["s1"], out["s2"], out["U_bits"], out["V_bits"], st)

    def profile(self, reset=False):
        return lbadmm_profile(self.handle, reset)

    def time_svid(self, factor, reps=10, stream=None):
        return lbadmm_time_svid(self.handle, factor, reps, stream)

    def state(self, stream=None):
        torch = _torch()
        f32 = torch.float32
        dev = torch.device("cuda", torch.cuda.current_device())
        s = {k: torch.empty((self.m if k in ("U", "Z_U", "Lam_U") else self.n, self.r),
                            dtype=f32, device=dev)
             for k in ("U", "V", "Z_U", "Lam_U", "Z_V", "Lam_V")}
        lbadmm_get_state(self.handle, stream=stream, **s)
        return s

    def close(self):
        if getattr(self, "handle", None):
            lbadmm_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *a):
        self.close()


def lbadmm(W, d_out, d_in, r, rho=1.0, iters=50, svid_steps=5, U0=None, V0=None, seed=0,
           compute_error=True, init_draws=False, balance=True, single_stream=False,
           solver=None) -> Result:
    """Factorise one layer: W ~ diag(s1) sign(U) sign(V)^T diag(s2)."""
    m, n = W.shape
    with LBADMM(m, n, r, rho, iters, svid_steps, seed, compute_error, init_draws, balance,
                single_stream, solver=solver) as h:
        return h.run(W, d_out, d_in, U0, V0)
