"""Thin ctypes binding of librrq.so with the C ABI's names (argument marshalling only).

Every function checks that its tensors are contiguous CUDA tensors of the
right type, passes raw device pointers, sizes and torch's current CUDA stream
to the C entry point of the same name, and raises ``RRQError`` on a non-zero
status.  All arithmetic runs in the library's CUDA kernels; there is no CPU
path.  If ``librrq.so`` is missing the first call raises immediately.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import os

import numpy as np
import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "librrq.so")

RRQ_OK, RRQ_ERR_INVALID, RRQ_ERR_CUDA, RRQ_ERR_UNSUPPORTED, RRQ_ERR_SCRATCH = 0, 1, 2, 3, 4
RRQ_F32, RRQ_F16, RRQ_BF16 = 0, 1, 2
DTYPE_CODE = {torch.float32: RRQ_F32, torch.float16: RRQ_F16, torch.bfloat16: RRQ_BF16}
ROPE_SCHEDULES = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}
# GGML block types (ggml's own type numbers), as in include/rrq.h
GGML_TYPES = {"q4_0": 2, "q4_1": 3, "q5_0": 6, "q5_1": 7, "q8_0": 8}

_c_i64 = ctypes.c_int64
_c_u64 = ctypes.c_uint64
_vp = ctypes.c_void_p
_int = ctypes.c_int
_dbl = ctypes.c_double
_fp = ctypes.POINTER(ctypes.c_float)

# name -> (restype, argtypes), mirroring include/rrq.h
SIGNATURES = {
    "rrq_format_version": (_int, []),
    "rrq_strerror": (ctypes.c_char_p, [_int]),
    "rrq_codebook": (_int, [_int, _vp]),
    "rrq_rotate": (_int, [_vp, _int, _c_i64, _int, _c_u64, _int, _vp, _vp]),
    "rrq_encode": (_int, [_vp, _int, _c_i64, _int, _int, _c_u64, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "rrq_decode": (_int, [_vp, _vp, _c_i64, _int, _int, _c_u64, _vp, _vp, _int, _vp]),
    "rrq_drive_encode": (_int, [_vp, _int, _c_i64, _int, _c_u64, _int, _vp, _vp, _vp]),
    "rrq_qk_scores": (_int, [_vp, _int, _vp, _vp, _c_i64, _int, _int, _int, _c_u64, _vp,
                             ctypes.c_float, _vp, _vp]),
    "rrq_qk_scores_qjl": (_int, [_vp, _int, _vp, _vp, _vp, _vp, _vp, _c_i64, _int, _int, _int,
                                 _c_u64, _vp, ctypes.c_float, _vp, _vp]),
    "rrq_attention_decode": (_int, [_vp, _int, _vp, _vp, _vp, _vp, _c_i64, _int, _int, _int,
                                    _c_u64, _vp, _int, _c_u64, _vp, ctypes.c_float, _vp,
                                    ctypes.c_size_t, _vp, _vp]),
    "rrq_attention_workspace_bytes": (ctypes.c_size_t, [_int, _int, _int, _int, _int, _c_i64]),
    "rrq_attention_decode_noalloc": (_int, [_vp, _int, _vp, _vp, _vp, _vp, _c_i64, _int, _int,
                                            _int, _c_u64, _vp, _int, _c_u64, _vp, ctypes.c_float,
                                            _vp, _vp]),
    "rrq_q4_0_rot": (_int, [_vp, _int, _c_i64, _int, _c_u64, _int, _vp, _vp]),
    "rrq_q4_0_rot_decode": (_int, [_vp, _c_i64, _int, _c_u64, _int, _vp, _int, _vp]),
    "rrq_ggml_block_bytes": (_int, [_int]),
    "rrq_ggml_rot": (_int, [_vp, _int, _c_i64, _int, _c_u64, _int, _int, _vp, _vp]),
    "rrq_ggml_rot_decode": (_int, [_vp, _int, _c_i64, _int, _c_u64, _int, _vp, _int, _vp]),
    "rrq_qjl_matrix": (_int, [_c_u64, _int, _vp]),
    "rrq_attention_shared": (_int, [_vp, _int, _c_i64, _int, _vp, _vp, _vp, _vp, _c_i64, _vp, _vp, _vp,
                                    _vp, _c_i64, _vp, _int, _int, _int, _c_u64, _vp, _int, _c_u64, _vp,
                                    ctypes.c_float, _vp, ctypes.c_size_t, _vp, _vp]),
    "rrq_attention_shared_workspace_bytes": (ctypes.c_size_t, [_c_i64, _int, _int, _int, _c_i64, _c_i64]),
    "rrq_attention_mass": (_int, [_vp, _c_i64, _int, _int, _c_i64, _vp, ctypes.c_float, _vp, _vp, _vp]),
    "rrq_evict": (_int, [_vp, _c_i64, _int, _c_i64, _vp, _c_i64, _c_i64, _c_i64, _int, _int, _int, _vp, _vp,
                         _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "rrq_rope_frequencies": (_int, [_int, _int, _dbl, _dbl, _dbl, _dbl, _dbl, _vp, _vp]),
    "rrq_rope": (_int, [_vp, _int, _c_i64, _int, _int, _int, _int, _vp, _vp, _dbl, _int, _vp, _vp]),
}


class RRQError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {strerror(status)} (status {status})")


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library (loaded on first use; raises if it was never built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -m random_rotation_kv_b200.build` "
                "(there is no CPU fallback)")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype, fn.argtypes = res, args
        _lib = handle
    return _lib


def strerror(status: int) -> str:
    return lib().rrq_strerror(status).decode()


def _check(status: int, what: str) -> None:
    if status != RRQ_OK:
        raise RRQError(status, what)


def _dev_tensor(t: torch.Tensor, name: str, dtypes=None) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")


def _stream(t: torch.Tensor) -> _vp:
    return _vp(torch.cuda.current_stream(t.device).cuda_stream)


def _ptr(t) -> _vp:
    return _vp(None) if t is None else _vp(t.data_ptr())


class _HostFloats:
    """Keeps a host float32 copy of a codebook alive for the duration of a call."""

    def __init__(self, codebook):
        self.arr = None if codebook is None else np.ascontiguousarray(
            np.asarray(codebook, dtype=np.float32))

    @property
    def ptr(self) -> _vp:
        return _vp(None) if self.arr is None else _vp(self.arr.ctypes.data)


def rrq_format_version() -> int:
    return lib().rrq_format_version()


def rrq_codebook(bits: int) -> np.ndarray:
    """Default codebook: ascending Lloyd–Max levels for N(0,1), float32[2^bits]."""
    out = np.zeros(1 << bits if 1 <= bits <= 8 else 1, dtype=np.float32)
    _check(lib().rrq_codebook(bits, _vp(out.ctypes.data)), "rrq_codebook")
    return out


def rrq_rotate(x: torch.Tensor, seed: int, inverse: bool = False, out: torch.Tensor | None = None):
    """Πx (or Πᵀx) of every row of x [..., d]; float32 result of x's shape."""
    _dev_tensor(x, "x", DTYPE_CODE)
    d = x.shape[-1]
    n = x.numel() // d if d else 0
    if out is None:
        out = torch.empty(x.shape, dtype=torch.float32, device=x.device)
    _dev_tensor(out, "out", (torch.float32,))
    _check(lib().rrq_rotate(_ptr(x), DTYPE_CODE[x.dtype], n, d, seed, int(bool(inverse)),
                            _ptr(out), _stream(x)), "rrq_rotate")
    return out


def rrq_encode(x: torch.Tensor, bits: int, seed: int, codebook=None, codes=None, norms=None,
               qjl_S=None, qjl_bits=None, qjl_rnorm=None):
    """Encode rows of x [..., d].

    Returns (codes uint8 [..., d*bits/8], norms float32 [...]) and, with
    ``qjl_S`` (bf16 [d, d] on the device), also (qjl_bits uint8 [..., d/8],
    qjl_rnorm float32 [...]).
    """
    _dev_tensor(x, "x", DTYPE_CODE)
    d = x.shape[-1]
    n = x.numel() // d if d else 0
    lead = x.shape[:-1]
    if codes is None:
        codes = torch.empty(*lead, d * bits // 8, dtype=torch.uint8, device=x.device)
    if norms is None:
        norms = torch.empty(lead, dtype=torch.float32, device=x.device)
    _dev_tensor(codes, "codes", (torch.uint8,))
    _dev_tensor(norms, "norms", (torch.float32,))
    if codes.numel() != n * (d * bits // 8) or norms.numel() != n:
        raise ValueError("codes / norms have the wrong size")
    if qjl_S is not None:
        _dev_tensor(qjl_S, "qjl_S", (torch.bfloat16,))
        if qjl_S.shape != (d, d):
            raise ValueError("qjl_S must be [d, d]")
        if qjl_bits is None:
            qjl_bits = torch.empty(*lead, d // 8, dtype=torch.uint8, device=x.device)
        if qjl_rnorm is None:
            qjl_rnorm = torch.empty(lead, dtype=torch.float32, device=x.device)
        _dev_tensor(qjl_bits, "qjl_bits", (torch.uint8,))
        _dev_tensor(qjl_rnorm, "qjl_rnorm", (torch.float32,))
    cb = _HostFloats(codebook)
    _check(lib().rrq_encode(_ptr(x), DTYPE_CODE[x.dtype], n, d, bits, seed, cb.ptr, _ptr(codes),
                            _ptr(norms), _ptr(qjl_S), _ptr(qjl_bits), _ptr(qjl_rnorm),
                            _stream(x)), "rrq_encode")
    if qjl_S is not None:
        return codes, norms, qjl_bits, qjl_rnorm
    return codes, norms


def rrq_drive_encode(x: torch.Tensor, seed: int, unbiased: bool, codes=None, scales=None):
    """DRIVE one-bit encode of rows of x [..., d].

    Returns (codes uint8 [..., d/8], scales float32 [...]); scales hold S·√d,
    which rrq_decode / rrq_qk_scores with bits=1 and codebook [-1, 1] read as
    the norm.
    """
    _dev_tensor(x, "x", DTYPE_CODE)
    d = x.shape[-1]
    n = x.numel() // d if d else 0
    lead = x.shape[:-1]
    if codes is None:
        codes = torch.empty(*lead, d // 8, dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(lead, dtype=torch.float32, device=x.device)
    _dev_tensor(codes, "codes", (torch.uint8,))
    _dev_tensor(scales, "scales", (torch.float32,))
    if codes.numel() != n * (d // 8) or scales.numel() != n:
        raise ValueError("codes / scales have the wrong size")
    _check(lib().rrq_drive_encode(_ptr(x), DTYPE_CODE[x.dtype], n, d, seed, int(bool(unbiased)),
                                  _ptr(codes), _ptr(scales), _stream(x)), "rrq_drive_encode")
    return codes, scales


def rrq_decode(codes: torch.Tensor, norms: torch.Tensor, d: int, bits: int, seed: int,
               codebook=None, out_dtype=torch.float16, out=None):
    """Reconstruct vectors [..., d] of ``out_dtype`` from codes [..., d*bits/8] and norms [...]."""
    _dev_tensor(codes, "codes", (torch.uint8,))
    _dev_tensor(norms, "norms", (torch.float32,))
    n = norms.numel()
    if codes.numel() != n * (d * bits // 8):
        raise ValueError("codes / norms sizes disagree")
    if out is None:
        out = torch.empty(*norms.shape, d, dtype=out_dtype, device=codes.device)
    _dev_tensor(out, "out", DTYPE_CODE)
    if out.numel() != n * d:
        raise ValueError("out has the wrong size")
    cb = _HostFloats(codebook)
    _check(lib().rrq_decode(_ptr(codes), _ptr(norms), n, d, bits, seed, cb.ptr, _ptr(out),
                            DTYPE_CODE[out.dtype], _stream(codes)), "rrq_decode")
    return out


def rrq_qk_scores(q: torch.Tensor, codes: torch.Tensor, norms: torch.Tensor, hkv: int, d: int,
                  bits: int, seed: int, codebook=None, scale: float = 1.0, out=None):
    """Scores [hq, T] of unrotated fp16 queries q [hq, d] against a quantised K cache.

    codes: [T*hkv, d*bits/8] (row t*hkv + g) or [T, hkv, d*bits/8]; norms: T*hkv floats.
    """
    _dev_tensor(q, "q", (torch.float16,))
    _dev_tensor(codes, "codes", (torch.uint8,))
    _dev_tensor(norms, "norms", (torch.float32,))
    hq = q.shape[0]
    if q.shape != (hq, d):
        raise ValueError("q must be [hq, d]")
    rows = norms.numel()
    if rows % hkv:
        raise ValueError("norms must hold T*hkv values")
    t_len = rows // hkv
    if codes.numel() != rows * (d * bits // 8):
        raise ValueError("codes / norms sizes disagree")
    if out is None:
        out = torch.empty(hq, t_len, dtype=torch.float32, device=q.device)
    _dev_tensor(out, "out", (torch.float32,))
    cb = _HostFloats(codebook)
    _check(lib().rrq_qk_scores(_ptr(q), hq, _ptr(codes), _ptr(norms), t_len, hkv, d, bits, seed,
                               cb.ptr, float(scale), _ptr(out), _stream(q)), "rrq_qk_scores")
    return out


def rrq_qk_scores_qjl(q: torch.Tensor, codes: torch.Tensor, norms: torch.Tensor,
                      qjl_bits: torch.Tensor, qjl_rnorm: torch.Tensor, qjl_S: torch.Tensor, hkv: int,
                      d: int, bits: int, seed: int, codebook=None, scale: float = 1.0, out=None):
    """Unbiased scores [hq, T] of unrotated fp16 queries q [hq, d] against keys stored as
    b-bit codes + norms plus the QJL sign bits and residual norms (rows t*hkv + g), with
    the projection qjl_S (bf16 [d, d]) they were encoded with."""
    _dev_tensor(q, "q", (torch.float16,))
    _dev_tensor(codes, "codes", (torch.uint8,))
    _dev_tensor(norms, "norms", (torch.float32,))
    _dev_tensor(qjl_bits, "qjl_bits", (torch.uint8,))
    _dev_tensor(qjl_rnorm, "qjl_rnorm", (torch.float32,))
    _dev_tensor(qjl_S, "qjl_S", (torch.bfloat16,))
    hq = q.shape[0]
    if q.shape != (hq, d) or qjl_S.shape != (d, d):
        raise ValueError("q must be [hq, d] and qjl_S [d, d]")
    rows = norms.numel()
    if rows % hkv:
        raise ValueError("norms must hold T*hkv values")
    t_len = rows // hkv
    if (codes.numel() != rows * (d * bits // 8) or qjl_bits.numel() != rows * (d // 8)
            or qjl_rnorm.numel() != rows):
        raise ValueError("codes / norms / qjl sizes disagree")
    if out is None:
        out = torch.empty(hq, t_len, dtype=torch.float32, device=q.device)
    _dev_tensor(out, "out", (torch.float32,))
    cb = _HostFloats(codebook)
    _check(lib().rrq_qk_scores_qjl(_ptr(q), hq, _ptr(codes), _ptr(norms), _ptr(qjl_bits),
                                   _ptr(qjl_rnorm), _ptr(qjl_S), t_len, hkv, d, bits, seed, cb.ptr,
                                   float(scale), _ptr(out), _stream(q)), "rrq_qk_scores_qjl")
    return out


def rrq_attention_decode(q: torch.Tensor, k_codes: torch.Tensor, k_norms: torch.Tensor,
                         v_codes: torch.Tensor, v_norms: torch.Tensor, hkv: int, d: int,
                         k_seed: int, v_seed: int, k_bits: int = 4, v_bits: int = 4,
                         k_codebook=None, v_codebook=None, scale: float = 1.0, out=None,
                         workspace=None):
    """One decode step of attention, out [hq, d] float32, of unrotated fp16 queries q [hq, d]
    over a K/V cache of k_bits / v_bits codes + norms (rows t*hkv + g).

    ``workspace``: a uint8 device tensor of at least rrq_attention_workspace_bytes(...)
    bytes, zero before its first use (each call leaves it ready for the next); a zeroed
    one is allocated when none is given."""
    _dev_tensor(q, "q", (torch.float16,))
    for t_, nm in ((k_codes, "k_codes"), (v_codes, "v_codes")):
        _dev_tensor(t_, nm, (torch.uint8,))
    for t_, nm in ((k_norms, "k_norms"), (v_norms, "v_norms")):
        _dev_tensor(t_, nm, (torch.float32,))
    hq = q.shape[0]
    if q.shape != (hq, d):
        raise ValueError("q must be [hq, d]")
    rows = k_norms.numel()
    if rows % hkv or v_norms.numel() != rows:
        raise ValueError("norms must hold T*hkv values")
    t_len = rows // hkv
    if k_codes.numel() != rows * (d * k_bits // 8) or v_codes.numel() != rows * (d * v_bits // 8):
        raise ValueError("codes / norms sizes disagree")
    if out is None:
        out = torch.empty(hq, d, dtype=torch.float32, device=q.device)
    _dev_tensor(out, "out", (torch.float32,))
    need = rrq_attention_workspace_bytes(hq, hkv, d, t_len, k_bits, v_bits)
    if workspace is None:
        workspace = torch.zeros(need, dtype=torch.uint8, device=q.device)
    _dev_tensor(workspace, "workspace", (torch.uint8,))
    kc, vc = _HostFloats(k_codebook), _HostFloats(v_codebook)
    _check(lib().rrq_attention_decode(_ptr(q), hq, _ptr(k_codes), _ptr(k_norms), _ptr(v_codes),
                                      _ptr(v_norms), t_len, hkv, d, k_bits, k_seed, kc.ptr, v_bits,
                                      v_seed, vc.ptr, float(scale), _ptr(workspace),
                                      workspace.numel(), _ptr(out), _stream(q)),
           "rrq_attention_decode")
    return out


def rrq_attention_workspace_bytes(hq: int, hkv: int, d: int, t_len: int, k_bits: int = 4,
                                  v_bits: int = 4) -> int:
    """Workspace bytes rrq_attention_decode needs on the current device."""
    return int(lib().rrq_attention_workspace_bytes(hq, hkv, d, k_bits, v_bits, t_len))


def rrq_q4_0_rot(x: torch.Tensor, seed: int, rotate: bool = True, out=None):
    """Rotate (optionally) and q4_0-quantise rows of x [..., d] -> uint8 [..., d/32*18]."""
    _dev_tensor(x, "x", DTYPE_CODE)
    d = x.shape[-1]
    n = x.numel() // d if d else 0
    if out is None:
        out = torch.empty(*x.shape[:-1], d // 32 * 18, dtype=torch.uint8, device=x.device)
    _dev_tensor(out, "out", (torch.uint8,))
    if out.numel() != n * (d // 32 * 18):
        raise ValueError("out has the wrong size")
    _check(lib().rrq_q4_0_rot(_ptr(x), DTYPE_CODE[x.dtype], n, d, seed, int(bool(rotate)),
                              _ptr(out), _stream(x)), "rrq_q4_0_rot")
    return out


def rrq_q4_0_rot_decode(blocks: torch.Tensor, d: int, seed: int, rotate: bool = True,
                        out_dtype=torch.float16, out=None):
    _dev_tensor(blocks, "blocks", (torch.uint8,))
    per = d // 32 * 18
    if blocks.shape[-1] != per:
        raise ValueError("blocks must be [..., d/32*18]")
    n = blocks.numel() // per
    if out is None:
        out = torch.empty(*blocks.shape[:-1], d, dtype=out_dtype, device=blocks.device)
    _dev_tensor(out, "out", DTYPE_CODE)
    _check(lib().rrq_q4_0_rot_decode(_ptr(blocks), n, d, seed, int(bool(rotate)), _ptr(out),
                                     DTYPE_CODE[out.dtype], _stream(blocks)),
           "rrq_q4_0_rot_decode")
    return out


def rrq_ggml_block_bytes(fmt: str) -> int:
    """Bytes of one block of 32 values of a GGML block type ('q4_0', 'q4_1', 'q5_0', 'q5_1', 'q8_0')."""
    return lib().rrq_ggml_block_bytes(GGML_TYPES[fmt])


def rrq_ggml_rot(x: torch.Tensor, seed: int, fmt: str, rotate: bool = True, out=None):
    """Rotate (optionally) then quantise rows of x [..., d] into GGML blocks of type `fmt`:
    uint8 [..., d/32*block_bytes]."""
    _dev_tensor(x, "x", DTYPE_CODE)
    d = x.shape[-1]
    n = x.numel() // d if d else 0
    per = d // 32 * rrq_ggml_block_bytes(fmt)
    if out is None:
        out = torch.empty(*x.shape[:-1], per, dtype=torch.uint8, device=x.device)
    _dev_tensor(out, "out", (torch.uint8,))
    if out.numel() != n * per:
        raise ValueError("out has the wrong size")
    _check(lib().rrq_ggml_rot(_ptr(x), DTYPE_CODE[x.dtype], n, d, seed, int(bool(rotate)),
                              GGML_TYPES[fmt], _ptr(out), _stream(x)), "rrq_ggml_rot")
    return out


def rrq_ggml_rot_decode(blocks: torch.Tensor, d: int, seed: int, fmt: str, rotate: bool = True,
                        out_dtype=torch.float16, out=None):
    _dev_tensor(blocks, "blocks", (torch.uint8,))
    per = d // 32 * rrq_ggml_block_bytes(fmt)
    if blocks.shape[-1] != per:
        raise ValueError(f"blocks must be [..., d/32*{per // (d // 32)}]")
    n = blocks.numel() // per
    if out is None:
        out = torch.empty(*blocks.shape[:-1], d, dtype=out_dtype, device=blocks.device)
    _dev_tensor(out, "out", DTYPE_CODE)
    _check(lib().rrq_ggml_rot_decode(_ptr(blocks), GGML_TYPES[fmt], n, d, seed, int(bool(rotate)),
                                     _ptr(out), DTYPE_CODE[out.dtype], _stream(blocks)),
           "rrq_ggml_rot_decode")
    return out


def rrq_qjl_matrix(seed: int, d: int, device=None) -> torch.Tensor:
    """The QJL projection S (bf16 [d, d]); generated on the host by the library, then copied."""
    host = np.zeros(d * d if d > 0 else 1, dtype=np.uint16)
    _check(lib().rrq_qjl_matrix(seed, d, _vp(host.ctypes.data)), "rrq_qjl_matrix")
    t = torch.from_numpy(host.view(np.int16).copy()).view(torch.bfloat16).reshape(d, d)
    return t if device is None else t.to(device)


# ---- serving calls.  A decode step issues these every few microseconds, so they hand
# plain integers to ctypes and ask torch for the raw stream.  Only rrq_rope records a graph.
_raw_stream = torch._C._cuda_getCurrentRawStream
_F32, _U8, _I32, _I64 = torch.float32, torch.uint8, torch.int32, torch.int64
_HALVES = (torch.float16, torch.bfloat16)


def _need(t, name: str, dtype, numel: int, dev: int) -> int:
    """Address of a contiguous CUDA tensor of `numel` elements on device `dev`."""
    try:
        if t.dtype is dtype and t.numel() == numel and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _dev_tensor(t, name, (dtype,))  # raises what is wrong with the tensor itself
    if t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")
    raise ValueError(f"{name} is on another device than the first argument")


def _first(t, name: str, dtypes) -> int:
    """Device of a call's first tensor, which must be a contiguous CUDA tensor of one of `dtypes`."""
    try:
        dev = t.get_device()
        if dev >= 0 and t.dtype in dtypes and t.is_contiguous():
            return dev
    except AttributeError:
        pass
    _dev_tensor(t, name, dtypes)
    raise TypeError(f"{name} must be a CUDA tensor")


def _call(name: str, dev: int, *args) -> None:
    """The C entry point `name` on device `dev` (the current one for its duration)."""
    fn = getattr(_lib or lib(), name)
    if dev == torch.cuda.current_device():
        status = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(dev))
    if status:
        raise RRQError(status, name)


@functools.lru_cache(maxsize=256)
def _shared_workspace(dev: int, *shape) -> int:
    with torch.cuda.device(dev):
        return rrq_attention_shared_workspace_bytes(*shape)


def rrq_attention_shared(q: torch.Tensor, pk_codes, pk_norms, pv_codes, pv_norms, tk_codes, tk_norms,
                         tv_codes, tv_norms, tail_lens, hkv: int, d: int, k_seed: int, v_seed: int,
                         k_bits: int = 4, v_bits: int = 4, k_codebook=None, v_codebook=None,
                         scale: float = 1.0, out=None, workspace=None):
    """One decode step of attention for a batch: out [batch, hq, d] of q's dtype (fp16 or
    bf16) for unrotated queries q [batch, hq, d] over a shared quantised prefix
    (pk_*, pv_*: rows t*hkv + g, or None without a prefix) followed by the first
    tail_lens[b] rows of each sequence's own tail (tk_*, tv_*: [batch, cap, hkv, ...],
    or None without tails; tail_lens int32 [batch] on the device).  A sequence without
    any token gets zeros.

    ``workspace``: a uint8 device tensor of at least
    rrq_attention_shared_workspace_bytes(...) bytes, of any content; allocated when none
    is given."""
    dev = _first(q, "q", _HALVES)
    shape = q.shape
    if len(shape) != 3 or shape[2] != d:
        raise ValueError("q must be [batch, hq, d]")
    if hkv < 1:
        raise ValueError("hkv must be at least 1")
    batch, hq, _ = shape
    prefix = cap = 0
    pk = pkn = pv = pvn = tk = tkn = tv = tvn = tl = None
    k_row, v_row = d * k_bits // 8, d * v_bits // 8
    if pk_codes is not None:
        rows = pk_norms.numel()
        prefix = rows // hkv
        if prefix * hkv != rows:
            raise ValueError("pk_norms must hold prefix*hkv values")
        pk, pkn = _need(pk_codes, "pk_codes", _U8, rows * k_row, dev), _need(pk_norms, "pk_norms", _F32, rows, dev)
        pv, pvn = _need(pv_codes, "pv_codes", _U8, rows * v_row, dev), _need(pv_norms, "pv_norms", _F32, rows, dev)
    if tk_codes is not None:
        rows = tk_norms.numel()
        cap = rows // (batch * hkv) if batch else 0
        if cap * batch * hkv != rows:
            raise ValueError("tk_norms must hold batch*cap*hkv values")
        tk, tkn = _need(tk_codes, "tk_codes", _U8, rows * k_row, dev), _need(tk_norms, "tk_norms", _F32, rows, dev)
        tv, tvn = _need(tv_codes, "tv_codes", _U8, rows * v_row, dev), _need(tv_norms, "tv_norms", _F32, rows, dev)
        tl = _need(tail_lens, "tail_lens", _I32, batch, dev)
    if out is None:
        out = torch.empty_like(q)
    to = _need(out, "out", q.dtype, batch * hq * d, dev)
    if workspace is None:
        workspace = torch.empty(_shared_workspace(dev, batch, hq, hkv, d, prefix, cap), dtype=_U8, device=q.device)
    size = workspace.numel()
    ws = _need(workspace, "workspace", _U8, size, dev)
    kc = vc = None  # codebooks: host arrays that live until the call returns
    if k_codebook is not None:
        k_host = _HostFloats(k_codebook)
        kc = k_host.ptr
    if v_codebook is not None:
        v_host = _HostFloats(v_codebook)
        vc = v_host.ptr
    _call("rrq_attention_shared", dev, q.data_ptr(), DTYPE_CODE[q.dtype], batch, hq, pk, pkn, pv, pvn, prefix, tk,
          tkn, tv, tvn, cap, tl, hkv, d, k_bits, k_seed, kc, v_bits, v_seed, vc, scale, ws, size, to)
    return out


def rrq_attention_shared_workspace_bytes(batch: int, hq: int, hkv: int, d: int, prefix: int,
                                         tail_cap: int) -> int:
    """Workspace bytes rrq_attention_shared needs on the current device."""
    return (_lib or lib()).rrq_attention_shared_workspace_bytes(batch, hq, hkv, d, prefix, tail_cap)


def rrq_attention_mass(scores: torch.Tensor, hkv: int, mass=None, lens=None, decay: float = 1.0, out=None):
    """Softmax weights of scores [batch, hq, T] (or [hq, T], as rrq_qk_scores returns them)
    summed over the query heads of each kv head and added to decay * mass: float32
    [batch, hkv, T] (or [hkv, T]).

    ``lens``: int32 [batch] on the device; tokens behind a sequence's length keep their
    mass.  ``mass``: the sums so far, zeros when not given.  ``out`` may be ``mass``."""
    dev = _first(scores, "scores", (_F32,))
    shape = scores.shape
    if len(shape) not in (2, 3):
        raise ValueError("scores must be [batch, hq, T] or [hq, T]")
    if hkv < 1:
        raise ValueError("hkv must be at least 1")
    batch = shape[0] if len(shape) == 3 else 1
    hq, t_len = shape[-2], shape[-1]
    if out is None:
        out = torch.empty((batch, hkv, t_len) if len(shape) == 3 else (hkv, t_len), dtype=_F32, device=scores.device)
    n = batch * hkv * t_len
    to = _need(out, "out", _F32, n, dev)
    frm = None if mass is None else _need(mass, "mass", _F32, n, dev)
    ln = None if lens is None else _need(lens, "lens", _I32, batch, dev)
    _call("rrq_attention_mass", dev, scores.data_ptr(), batch, hq, hkv, t_len, ln, decay, frm, to)
    return out


@functools.lru_cache(maxsize=None)
def _row_widths(k_row: int, v_row: int):
    """(d, k_bits, v_bits) of a cache with code rows of these sizes (the move depends on the
    sizes alone, so any d that both fit will do)."""
    for d in (64, 128, 256, 512):
        if k_row * 8 % d == 0 and v_row * 8 % d == 0 and 1 <= k_row * 8 // d <= 4 and 1 <= v_row * 8 // d <= 4:
            return d, k_row * 8 // d, v_row * 8 // d
    raise ValueError(f"no d and bit widths give code rows of {k_row} and {v_row} bytes")


def rrq_evict(mass: torch.Tensor, lens, keep: int, k_codes: torch.Tensor, k_norms: torch.Tensor,
              v_codes: torch.Tensor, v_norms: torch.Tensor, sink: int = 0, recent: int = 0, index=None,
              out_lens=None, out_mass=None, out=None):
    """Cut a quantised cache back to `keep` tokens per kv head: the first `sink`, the last
    `recent`, and the largest mass [batch, hkv, cap] (ties to the lower token).

    k_codes [batch, cap, hkv, d*k_bits/8], k_norms [batch, cap, hkv], v_* alike; lens int32
    [batch] on the device or None.  Returns (index int32 [batch, hkv, keep], out_lens int32
    [batch], out_mass [batch, hkv, keep], k_codes, k_norms, v_codes, v_norms of capacity
    `keep`).  ``out``: the four arrays of the new cache; entries behind a sequence's new
    length are left as they were (zeros, and -1 in index, where this call allocates)."""
    dev = _first(mass, "mass", (_F32,))
    shape = mass.shape
    if len(shape) != 3:
        raise ValueError("mass must be [batch, hkv, cap]")
    batch, hkv, cap = shape
    if keep < 1:
        raise ValueError("keep must be at least 1")
    lead, k_shape, v_shape = (batch, cap, hkv), k_codes.shape, v_codes.shape
    if len(k_shape) != 4 or len(v_shape) != 4 or k_shape[:3] != lead or v_shape[:3] != lead:
        raise ValueError("k_codes and v_codes must be [batch, cap, hkv, row bytes]")
    if k_norms.shape != lead or v_norms.shape != lead:
        raise ValueError("k_norms and v_norms must be [batch, cap, hkv]")
    device = mass.device
    k_row, v_row = k_shape[3], v_shape[3]
    d, k_bits, v_bits = _row_widths(k_row, v_row)
    if index is None:
        index = torch.full((batch, hkv, keep), -1, dtype=_I32, device=device)
    if out_lens is None:
        out_lens = torch.empty(batch, dtype=_I32, device=device)
    if out_mass is None:
        out_mass = torch.zeros(batch, hkv, keep, dtype=_F32, device=device)
    if out is None:
        out = [torch.zeros(batch, keep, *t_.shape[2:], dtype=t_.dtype, device=device)
               for t_ in (k_codes, k_norms, v_codes, v_norms)]
    rows, new, slots = batch * cap * hkv, batch * keep * hkv, batch * hkv * keep
    ln = None if lens is None else _need(lens, "lens", _I32, batch, dev)
    _call("rrq_evict", dev, mass.data_ptr(), batch, hkv, cap, ln, keep, sink, recent, d, k_bits, v_bits,
          _need(k_codes, "k_codes", _U8, rows * k_row, dev), _need(k_norms, "k_norms", _F32, rows, dev),
          _need(v_codes, "v_codes", _U8, rows * v_row, dev), _need(v_norms, "v_norms", _F32, rows, dev),
          _need(index, "index", _I32, slots, dev), _need(out_lens, "out_lens", _I32, batch, dev),
          _need(out_mass, "out_mass", _F32, slots, dev), _need(out[0], "out[0]", _U8, new * k_row, dev),
          _need(out[1], "out[1]", _F32, new, dev), _need(out[2], "out[2]", _U8, new * v_row, dev),
          _need(out[3], "out[3]", _F32, new, dev))
    return (index, out_lens, out_mass, *out)


def rrq_rope_frequencies(rot: int, base: float = 10000.0, schedule: str = "none", stretch: float = 1.0,
                         original: float = 8192.0, fast: float = 32.0, slow: float = 1.0):
    """(frequencies float64 [rot/2] in radians per position, factor on cos and sin) of a
    rotary schedule: 'none', 'linear', 'ntk' or 'yarn'.  Host only."""
    out = np.zeros(max(rot // 2, 1), dtype=np.float64)
    factor = ctypes.c_double(0.0)
    _check(lib().rrq_rope_frequencies(ROPE_SCHEDULES[schedule], rot, base, stretch, original, fast, slow,
                                      _vp(out.ctypes.data), _vp(ctypes.addressof(factor))),
           "rrq_rope_frequencies")
    return out, factor.value


class _Rope(torch.autograd.Function):
    """The rotation and, as its gradient, the transposed map."""

    @staticmethod
    def forward(ctx, x, positions, freqs, interleaved, factor, inverse):
        ctx.save_for_backward(positions)
        ctx.how = freqs, interleaved, factor, inverse
        return rrq_rope(x, positions, freqs, interleaved, factor, inverse)

    @staticmethod
    def backward(ctx, grad):
        freqs, interleaved, factor, inverse = ctx.how
        (positions,) = ctx.saved_tensors
        return rrq_rope(grad.contiguous(), positions, freqs, interleaved, factor, not inverse), None, None, None, None, None


def rrq_rope(x: torch.Tensor, positions: torch.Tensor, freqs, interleaved: bool = False,
             factor: float = 1.0, inverse: bool = False, out=None):
    """Rotary positions of x [n, heads, d] at int64 positions [n]: the first 2*len(freqs)
    coordinates of every vector turned, the rest copied; ``inverse`` applies the transposed
    map (the gradient with respect to x).  ``freqs``: radians per position on the host
    (float64, as rrq_rope_frequencies returns them).  ``out`` may be ``x``.

    Differentiable in x (positions must then stay as they are until the backward pass); a call
    with ``out`` records no graph.  As for any torch operation, a backward pass is captured
    into a CUDA graph only while no graph of the same leaf from another stream is alive."""
    dev = _first(x, "x", DTYPE_CODE)
    shape, dtype = x.shape, x.dtype
    if len(shape) != 3:
        raise ValueError("x must be [n, heads, d]")
    if out is None and x.requires_grad and torch.is_grad_enabled():
        return _Rope.apply(x, positions, np.array(freqs, dtype=np.float64), interleaved, factor, inverse)
    n, heads, d = shape
    fr = np.ascontiguousarray(freqs, dtype=np.float64)
    if out is None:
        out = torch.empty_like(x)
    _call("rrq_rope", dev, x.data_ptr(), DTYPE_CODE[dtype], n, heads, d, 2 * fr.size, int(bool(interleaved)),
          _need(positions, "positions", _I64, n, dev), fr.__array_interface__["data"][0], factor, int(bool(inverse)),
          _need(out, "out", dtype, n * heads * d, dev))
    return out
