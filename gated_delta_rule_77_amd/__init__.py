"""MI355X (gfx950) gated delta-rule library: Python binding of libpdn.so.

This layer only marshals arguments: it checks tensor placement, dtypes and
shapes, passes raw device pointers and the current HIP stream to the C ABI
(include/pdn.h, include/pdn_layer.h, include/pdn_block.h), and raises on a non-zero return code.  Every step of the
computation runs in the HIP kernels of libpdn.so; there is no fallback, and
loading fails loudly when the library is missing.

PyTorch is used for device memory and streams only.

Entry points (same names as the C ABI):
    pdn_chunk_fwd(...)                 prefill over [B,H,T,d]
    pdn_chunk_fwd_noalloc(...)         the same with the library's static scratch
    pdn_chunk_fwd_workspace_size(...)  scratch bytes the prefill needs
    pdn_decode_step(...)               one token against a resident state
    pdn_chunk_bwd(...)                 gradients of the prefill
    pdn_chunk_bwd_workspace_size(...)  scratch bytes the backward needs
    pdn_abi_version(), pdn_strerror(code)
and the operators around the recurrence:
    pdn_qk_norm_fwd / _bwd(...)        norm and rotation of q and k, [B,T,Hx,d] -> [B,H,T,d]
    pdn_out_norm_fwd / _bwd(...)       gated norm of o, [B,H,T,dv] -> [B,T,H,dv]
    pdn_scan_fwd / _bwd / _step(...)   the gated recurrence with a vector state, [B,T,D]
    pdn_scan_marks(T)                  kept states of a scan over T tokens
    pdn_rope_freqs(...)                inverse frequencies, scaled for long contexts
and what a stack with attention layers needs besides:
    pdn_add_norm_fwd / _bwd(...)       dropout, residual and norm between two sublayers, y in 8 bits too
    pdn_attn_fwd / _bwd(...)           causal softmax attention over [B,H,T,d]
    pdn_cache_append(...)              new tokens' keys and values into a paged cache
    pdn_attn_paged(...)                attention of new tokens over that cache
with pdn_*_workspace_size(...) for those that take scratch.
"""
from __future__ import annotations

import ctypes
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpdn.so")

# The argument structs below mirror this version of include/pdn.h.
PDN_ABI_VERSION = 5
PDN_LAYER_VERSION = 1   # and this one of include/pdn_layer.h
PDN_BLOCK_VERSION = 1   # and of include/pdn_block.h

PDN_OK, PDN_EINVAL, PDN_EUNSUPPORTED, PDN_EWORKSPACE, PDN_EHIP, PDN_ESCRATCH = 0, -1, -2, -3, -4, -5
PDN_NOALLOC_SCRATCH_BYTES = 256 << 20   # static scratch of pdn_chunk_fwd_noalloc
PDN_F32, PDN_BF16, PDN_E4M3 = 0, 1, 2
PDN_ALPHA_NONE, PDN_ALPHA_SCALAR, PDN_ALPHA_VEC = 0, 1, 2
PDN_GATE_SCALAR, PDN_GATE_VEC, PDN_GAMMA_SAME_AS_BETA = 1, 2, 3
PDN_KEY_SYMMETRIC, PDN_KEY_ERASE_GATE, PDN_KEY_WRITE_GATE = 0, 1, 2
PDN_PRECOND_INVERSE, PDN_PRECOND_STABILISED = 0, 1
PDN_NORM_NONE, PDN_NORM_RMS, PDN_NORM_L2 = 0, 1, 2
PDN_ROPE_HALF, PDN_ROPE_INTERLEAVED = 0, 1
PDN_ROPE_PLAIN, PDN_ROPE_LINEAR, PDN_ROPE_BASE, PDN_ROPE_BY_PARTS = 0, 1, 2, 3
PDN_ACT_NONE, PDN_ACT_SILU, PDN_ACT_SIGMOID = 0, 1, 2
PDN_GAIN_NONE, PDN_GAIN_COMPLEMENT, PDN_GAIN_NORM = 0, 1, 2
PDN_SCAN_MARK = 96

_P = ctypes.c_void_p
_I = ctypes.c_int32
_L = ctypes.c_int64
_F = ctypes.c_float


class ChunkFwdArgs(ctypes.Structure):
    """Mirror of ``pdn_chunk_fwd_args``."""
    _fields_ = [("B", _I), ("H", _I), ("T", _I), ("dk", _I), ("dv", _I),
                ("qkv_dtype", _I), ("o_dtype", _I),
                ("q", _P), ("k", _P), ("v", _P),
                ("alpha_mode", _I), ("log_alpha", _P),
                ("beta_mode", _I), ("beta", _P),
                ("gamma_mode", _I), ("gamma", _P),
                ("key_mode", _I),
                ("precond_eps", ctypes.c_float), ("precond_mode", _I), ("precond_x", ctypes.c_float),
                ("precond_A0", _P), ("precond_AT", _P),
                ("S0", _P), ("ST", _P), ("o", _P),
                ("workspace", _P), ("workspace_bytes", ctypes.c_size_t)]


class ChunkBwdArgs(ctypes.Structure):
    """Mirror of ``pdn_chunk_bwd_args``."""
    _fields_ = [("fwd", ChunkFwdArgs), ("dO", _P), ("dST", _P),
                ("dq", _P), ("dk", _P), ("dv", _P),
                ("dlog_alpha", _P), ("dbeta", _P), ("dgamma", _P),
                ("dS0", _P), ("dA0", _P),
                ("workspace", _P), ("workspace_bytes", ctypes.c_size_t)]


class DecodeArgs(ctypes.Structure):
    """Mirror of ``pdn_decode_args``."""
    _fields_ = [("B", _I), ("H", _I), ("dk", _I), ("dv", _I),
                ("qkv_dtype", _I), ("o_dtype", _I),
                ("q", _P), ("k", _P), ("v", _P),
                ("alpha_mode", _I), ("log_alpha", _P),
                ("beta_mode", _I), ("beta", _P),
                ("gamma_mode", _I), ("gamma", _P),
                ("key_mode", _I),
                ("precond_eps", ctypes.c_float), ("precond_mode", _I), ("precond_x", ctypes.c_float),
                ("precond_A", _P),
                ("S", _P), ("o", _P)]


class QkNormArgs(ctypes.Structure):
    """Mirror of ``pdn_qk_norm_args``."""
    _fields_ = [("B", _I), ("T", _I), ("H", _I), ("Hq", _I), ("Hk", _I), ("d", _I),
                ("dtype", _I), ("norm", _I), ("eps", _F), ("q_scale", _F), ("k_scale", _F),
                ("rot_dim", _I), ("rope_layout", _I), ("rope_scale", _F),
                ("inv_freq", _P), ("positions", _P), ("wq", _P), ("wk", _P),
                ("xq", _P), ("xk", _P),
                ("xq_sb", _L), ("xq_st", _L), ("xq_sh", _L),
                ("xk_sb", _L), ("xk_st", _L), ("xk_sh", _L),
                ("q", _P), ("k", _P)]


class QkNormBwdArgs(ctypes.Structure):
    """Mirror of ``pdn_qk_norm_bwd_args``."""
    _fields_ = [("fwd", QkNormArgs), ("dq", _P), ("dk", _P), ("dxq", _P), ("dxk", _P),
                ("dxq_sb", _L), ("dxq_st", _L), ("dxq_sh", _L),
                ("dxk_sb", _L), ("dxk_st", _L), ("dxk_sh", _L),
                ("dwq", _P), ("dwk", _P),
                ("workspace", _P), ("workspace_bytes", ctypes.c_size_t)]


class OutNormArgs(ctypes.Structure):
    """Mirror of ``pdn_out_norm_args``."""
    _fields_ = [("B", _I), ("H", _I), ("T", _I), ("dv", _I), ("o_dtype", _I), ("dtype", _I),
                ("act", _I), ("eps", _F), ("o", _P), ("w", _P),
                ("z", _P), ("z_sb", _L), ("z_st", _L), ("z_sh", _L),
                ("y", _P), ("y_sb", _L), ("y_st", _L), ("y_sh", _L)]


class OutNormBwdArgs(ctypes.Structure):
    """Mirror of ``pdn_out_norm_bwd_args``."""
    _fields_ = [("fwd", OutNormArgs),
                ("dy", _P), ("dy_sb", _L), ("dy_st", _L), ("dy_sh", _L), ("d_o", _P),
                ("dz", _P), ("dz_sb", _L), ("dz_st", _L), ("dz_sh", _L), ("dw", _P),
                ("workspace", _P), ("workspace_bytes", ctypes.c_size_t)]


class ScanArgs(ctypes.Structure):
    """Mirror of ``pdn_scan_args``."""
    _fields_ = [("B", _I), ("T", _I), ("D", _I), ("dtype", _I), ("log_dtype", _I), ("gain", _I),
                ("x", _P), ("x_sb", _L), ("x_st", _L),
                ("log_a", _P), ("log_a_sb", _L), ("log_a_st", _L),
                ("h0", _P), ("hT", _P), ("h", _P), ("h_sb", _L), ("h_st", _L), ("marks", _P),
                ("workspace", _P), ("workspace_bytes", ctypes.c_size_t)]


class ScanBwdArgs(ctypes.Structure):
    """Mirror of ``pdn_scan_bwd_args``."""
    _fields_ = [("fwd", ScanArgs), ("dh", _P), ("dh_sb", _L), ("dh_st", _L), ("dhT", _P),
                ("dx", _P), ("dx_sb", _L), ("dx_st", _L),
                ("dlog_a", _P), ("dlog_a_sb", _L), ("dlog_a_st", _L), ("dh0", _P),
                ("workspace", _P), ("workspace_bytes", ctypes.c_size_t)]


class ScanStepArgs(ctypes.Structure):
    """Mirror of ``pdn_scan_step_args``."""
    _fields_ = [("B", _I), ("D", _I), ("dtype", _I), ("log_dtype", _I), ("gain", _I),
                ("x", _P), ("x_sb", _L), ("log_a", _P), ("log_a_sb", _L),
                ("h_prev", _P), ("h_next", _P), ("h", _P), ("h_sb", _L)]


class AddNormArgs(ctypes.Structure):
    """Mirror of ``pdn_add_norm_args``."""
    _fields_ = [("B", _I), ("T", _I), ("D", _I), ("dtype", _I), ("s_dtype", _I), ("y_dtype", _I), ("group", _I),
                ("eps", _F), ("drop_p", _F), ("seed", _P), ("w", _P),
                ("x", _P), ("x_sb", _L), ("x_st", _L), ("res", _P), ("res_sb", _L), ("res_st", _L),
                ("s", _P), ("s_sb", _L), ("s_st", _L), ("y", _P), ("y_sb", _L), ("y_st", _L), ("y_scale", _P)]


class AddNormBwdArgs(ctypes.Structure):
    """Mirror of ``pdn_add_norm_bwd_args``."""
    _fields_ = [("B", _I), ("T", _I), ("D", _I), ("dtype", _I), ("s_dtype", _I), ("y_dtype", _I),
                ("eps", _F), ("drop_p", _F), ("seed", _P), ("w", _P),
                ("s", _P), ("s_sb", _L), ("s_st", _L), ("dy", _P), ("dy_sb", _L), ("dy_st", _L),
                ("ds", _P), ("ds_sb", _L), ("ds_st", _L), ("dres", _P), ("dres_sb", _L), ("dres_st", _L),
                ("dx", _P), ("dx_sb", _L), ("dx_st", _L), ("dw", _P),
                ("workspace", _P), ("workspace_bytes", ctypes.c_size_t)]


class AttnArgs(ctypes.Structure):
    """Mirror of ``pdn_attn_args``."""
    _fields_ = [("B", _I), ("H", _I), ("Hk", _I), ("Tq", _I), ("Tk", _I), ("d", _I), ("dtype", _I), ("o_dtype", _I),
                ("window", _I), ("scale", _F), ("first", _P),
                ("q", _P), ("q_sb", _L), ("q_sh", _L), ("q_st", _L), ("k", _P), ("k_sb", _L), ("k_sh", _L), ("k_st", _L),
                ("v", _P), ("v_sb", _L), ("v_sh", _L), ("v_st", _L), ("o", _P), ("o_sb", _L), ("o_sh", _L), ("o_st", _L),
                ("lse", _P), ("workspace", _P), ("workspace_bytes", ctypes.c_size_t)]


class AttnBwdArgs(ctypes.Structure):
    """Mirror of ``pdn_attn_bwd_args``."""
    _fields_ = [("fwd", AttnArgs), ("g_dtype", _I), ("d_o", _P), ("do_sb", _L), ("do_sh", _L), ("do_st", _L),
                ("dq", _P), ("dq_sb", _L), ("dq_sh", _L), ("dq_st", _L), ("dk", _P), ("dk_sb", _L), ("dk_sh", _L), ("dk_st", _L),
                ("dv", _P), ("dv_sb", _L), ("dv_sh", _L), ("dv_st", _L),
                ("workspace", _P), ("workspace_bytes", ctypes.c_size_t)]


class Cache(ctypes.Structure):
    """Mirror of ``pdn_cache``."""
    _fields_ = [("B", _I), ("N", _I), ("max_new", _I), ("Hk", _I), ("d", _I), ("dtype", _I),
                ("pages", _I), ("page_size", _I), ("table_width", _I),
                ("k_pages", _P), ("k_sp", _L), ("k_st", _L), ("k_sh", _L),
                ("v_pages", _P), ("v_sp", _L), ("v_st", _L), ("v_sh", _L),
                ("table", _P), ("lens", _P), ("starts", _P)]


class CacheAppendArgs(ctypes.Structure):
    """Mirror of ``pdn_cache_append_args``."""
    _fields_ = [("cache", Cache), ("k", _P), ("k_sn", _L), ("k_sh", _L), ("v", _P), ("v_sn", _L), ("v_sh", _L)]


class AttnPagedArgs(ctypes.Structure):
    """Mirror of ``pdn_attn_paged_args``."""
    _fields_ = [("cache", Cache), ("H", _I), ("o_dtype", _I), ("window", _I), ("scale", _F),
                ("q", _P), ("q_sn", _L), ("q_sh", _L), ("o", _P), ("o_sn", _L), ("o_sh", _L), ("lse", _P),
                ("workspace", _P), ("workspace_bytes", ctypes.c_size_t)]


# the operators around the recurrence: their argument structs, and which of
# them have a workspace size to ask for
_AROUND = {"pdn_qk_norm_fwd": (QkNormArgs, "pdn_qk_norm_check", None),
           "pdn_qk_norm_bwd": (QkNormBwdArgs, "pdn_qk_norm_bwd_check", "pdn_qk_norm_bwd_workspace_size"),
           "pdn_out_norm_fwd": (OutNormArgs, "pdn_out_norm_check", None),
           "pdn_out_norm_bwd": (OutNormBwdArgs, "pdn_out_norm_bwd_check", "pdn_out_norm_bwd_workspace_size"),
           "pdn_scan_fwd": (ScanArgs, "pdn_scan_check", "pdn_scan_fwd_workspace_size"),
           "pdn_scan_bwd": (ScanBwdArgs, "pdn_scan_bwd_check", "pdn_scan_bwd_workspace_size"),
           "pdn_scan_step": (ScanStepArgs, "pdn_scan_step_check", None)}

# and those of include/pdn_block.h
_BLOCK = {"pdn_add_norm_fwd": (AddNormArgs, "pdn_add_norm_check", None),
          "pdn_add_norm_bwd": (AddNormBwdArgs, "pdn_add_norm_bwd_check", "pdn_add_norm_bwd_workspace_size"),
          "pdn_attn_fwd": (AttnArgs, "pdn_attn_check", "pdn_attn_fwd_workspace_size"),
          "pdn_attn_bwd": (AttnBwdArgs, "pdn_attn_bwd_check", "pdn_attn_bwd_workspace_size"),
          "pdn_cache_append": (CacheAppendArgs, "pdn_cache_append_check", None),
          "pdn_attn_paged": (AttnPagedArgs, "pdn_attn_paged_check", "pdn_attn_paged_workspace_size")}
_SIZES = {name: size for calls in (_AROUND, _BLOCK) for name, (_, _, size) in calls.items()}

EXPORTED = ("pdn_abi_version", "pdn_strerror", "pdn_chunk_fwd_workspace_size",
            "pdn_chunk_fwd_check", "pdn_chunk_fwd", "pdn_chunk_fwd_noalloc", "pdn_decode_check",
            "pdn_decode_step", "pdn_chunk_bwd_workspace_size", "pdn_chunk_bwd_check",
            "pdn_chunk_bwd")
# include/pdn_layer.h
EXPORTED_LAYER = ("pdn_layer_version", "pdn_rope_freqs", "pdn_scan_marks",
                  *(n for call, (_, check, size) in _AROUND.items() for n in (call, check, size) if n))

# include/pdn_block.h
EXPORTED_BLOCK = ("pdn_block_version", *(n for call, (_, check, size) in _BLOCK.items() for n in (call, check, size) if n))

_lib = None
_lock = threading.Lock()


class PdnError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__("%s failed: %s (code %d)" % (where, pdn_strerror(code), code))


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Load libpdn.so (built by ``gated_delta_rule_77_amd.build``); raise if absent."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError("libpdn.so not found at %s: build it with "
                               "`python -m gated_delta_rule_77_amd.build` (there is no "
                               "fallback implementation)" % p)
        lib = ctypes.CDLL(p)
        lib.pdn_abi_version.argtypes = []
        lib.pdn_abi_version.restype = ctypes.c_int
        lib.pdn_strerror.argtypes = [ctypes.c_int]
        lib.pdn_strerror.restype = ctypes.c_char_p
        lib.pdn_chunk_fwd_workspace_size.argtypes = [ctypes.POINTER(ChunkFwdArgs),
                                                     ctypes.POINTER(ctypes.c_size_t)]
        lib.pdn_chunk_fwd_workspace_size.restype = ctypes.c_int
        lib.pdn_chunk_fwd_check.argtypes = [ctypes.POINTER(ChunkFwdArgs)]
        lib.pdn_chunk_fwd_check.restype = ctypes.c_int
        lib.pdn_chunk_fwd.argtypes = [ctypes.POINTER(ChunkFwdArgs), _P]
        lib.pdn_chunk_fwd.restype = ctypes.c_int
        lib.pdn_chunk_fwd_noalloc.argtypes = [ctypes.POINTER(ChunkFwdArgs), _P]
        lib.pdn_chunk_fwd_noalloc.restype = ctypes.c_int
        lib.pdn_chunk_bwd_workspace_size.argtypes = [ctypes.POINTER(ChunkBwdArgs),
                                                     ctypes.POINTER(ctypes.c_size_t)]
        lib.pdn_chunk_bwd_workspace_size.restype = ctypes.c_int
        lib.pdn_chunk_bwd_check.argtypes = [ctypes.POINTER(ChunkBwdArgs)]
        lib.pdn_chunk_bwd_check.restype = ctypes.c_int
        lib.pdn_chunk_bwd.argtypes = [ctypes.POINTER(ChunkBwdArgs), _P]
        lib.pdn_chunk_bwd.restype = ctypes.c_int
        lib.pdn_decode_check.argtypes = [ctypes.POINTER(DecodeArgs)]
        lib.pdn_decode_check.restype = ctypes.c_int
        lib.pdn_decode_step.argtypes = [ctypes.POINTER(DecodeArgs), _P]
        lib.pdn_decode_step.restype = ctypes.c_int
        # a library built from another header version would read the
        # argument structs at other offsets (device pointers included)
        ver = int(lib.pdn_abi_version())
        if ver != PDN_ABI_VERSION:
            raise RuntimeError("%s has ABI version %d, this binding mirrors version %d: "
                               "rebuild it with `python -m gated_delta_rule_77_amd.build`"
                               % (p, ver, PDN_ABI_VERSION))
        if not hasattr(lib, "pdn_layer_version") or lib.pdn_layer_version() != PDN_LAYER_VERSION:
            raise RuntimeError("%s is of another version of include/pdn_layer.h than this binding (%d): "
                               "rebuild it with `python -m gated_delta_rule_77_amd.build`" % (p, PDN_LAYER_VERSION))
        if not hasattr(lib, "pdn_block_version") or lib.pdn_block_version() != PDN_BLOCK_VERSION:
            raise RuntimeError("%s is of another version of include/pdn_block.h than this binding (%d): "
                               "rebuild it with `python -m gated_delta_rule_77_amd.build`" % (p, PDN_BLOCK_VERSION))
        for name, (struct, check, size) in (*_AROUND.items(), *_BLOCK.items()):
            getattr(lib, name).argtypes = [ctypes.POINTER(struct), _P]
            getattr(lib, check).argtypes = [ctypes.POINTER(struct)]
            if size:
                getattr(lib, size).argtypes = [ctypes.POINTER(struct), ctypes.POINTER(ctypes.c_size_t)]
            for n in (name, check, size):
                if n:
                    getattr(lib, n).restype = ctypes.c_int
        lib.pdn_scan_marks.argtypes = [_I]
        lib.pdn_scan_marks.restype = ctypes.c_int
        lib.pdn_rope_freqs.argtypes = [_I, ctypes.c_double, _I, ctypes.c_double, _L,
                                       ctypes.POINTER(ctypes.c_double), ctypes.POINTER(_F)]
        lib.pdn_rope_freqs.restype = ctypes.c_int
        if path is None:
            _lib = lib
        return lib


def pdn_abi_version() -> int:
    return int(load_library().pdn_abi_version())


def pdn_strerror(code: int) -> str:
    return load_library().pdn_strerror(int(code)).decode()


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------

def _ptr(t):
    """Device pointer of a contiguous torch tensor (or None / raw int)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("tensor must live in device memory")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _qkv_dtype(t):
    import torch
    if t.dtype == torch.bfloat16:
        return PDN_BF16
    if t.dtype == torch.float32:
        return PDN_F32
    raise ValueError("q/k/v/o must be float32 or bfloat16, got %s" % t.dtype)


def _f32(t, name):
    import torch
    if t is None:
        return
    if t.dtype != torch.float32:
        raise ValueError("%s must be float32" % name)


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _shape(t, name, *allowed):
    """Raise unless tensor t (None allowed only when None is listed) has one
    of the allowed shapes.  The C ABI receives bare pointers and cannot know
    a tensor's extent, so a wrongly shaped tensor would be read (or written)
    past its end: every tensor is checked here before a pointer is taken."""
    if t is None:
        if None in allowed:
            return
        raise ValueError("%s is required" % name)
    shapes = [a for a in allowed if a is not None]
    if tuple(t.shape) not in shapes:
        raise ValueError("%s must have shape %s, got %s" % (
            name, " or ".join("[%s]" % ",".join(str(x) for x in a) for a in shapes),
            list(t.shape)))


def _same_device(ref, named):
    """Every tensor must live on the device of `ref` (q)."""
    for name, t in named:
        if t is not None and not isinstance(t, int) and t.device != ref.device:
            raise ValueError("%s is on %s, q on %s: every tensor must share q's device"
                             % (name, t.device, ref.device))


def _alpha_mode(log_alpha, lead):
    if log_alpha is None:
        return PDN_ALPHA_NONE
    return PDN_ALPHA_SCALAR if log_alpha.dim() == lead else PDN_ALPHA_VEC


def _gate_mode(g, lead):
    return PDN_GATE_SCALAR if g.dim() == lead else PDN_GATE_VEC


def _precond_fields(a, precond_eps, precond_mode, precond_x):
    a.precond_eps = -1.0 if precond_eps is None else float(precond_eps)
    a.precond_mode = int(precond_mode)
    a.precond_x = float(precond_x)


def _chunk_args(q, k, v, o, log_alpha, beta, gamma, precond_eps, precond_A0,
                precond_AT, S0, ST, workspace, key_mode, precond_mode=PDN_PRECOND_INVERSE,
                precond_x=1.5):
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k must be [B,H,T,dk] and v [B,H,T,dv]")
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    if tuple(k.shape) != (B, H, T, dk) or tuple(v.shape[:3]) != (B, H, T):
        raise ValueError("q, k must be [B,H,T,dk] and v [B,H,T,dv]")
    _shape(o, "o", (B, H, T, dv))
    if q.dtype != k.dtype or q.dtype != v.dtype:
        raise ValueError("q, k, v must share one dtype")
    _shape(log_alpha, "log_alpha", None, (B, H, T), (B, H, T, dk))
    _shape(beta, "beta", (B, H, T), (B, H, T, dk))
    _shape(gamma, "gamma", None, (B, H, T), (B, H, T, dv))
    _shape(precond_A0, "precond_A0", None, (B, H, dk))
    _shape(precond_AT, "precond_AT", None, (B, H, dk))
    _shape(S0, "S0", None, (B, H, dk, dv))
    _shape(ST, "ST", None, (B, H, dk, dv))
    _same_device(q, (("k", k), ("v", v), ("o", o), ("log_alpha", log_alpha), ("beta", beta),
                     ("gamma", gamma), ("precond_A0", precond_A0),
                     ("precond_AT", precond_AT), ("S0", S0), ("ST", ST),
                     ("workspace", workspace)))
    for name, t in (("log_alpha", log_alpha), ("beta", beta), ("gamma", gamma),
                    ("precond_A0", precond_A0), ("precond_AT", precond_AT),
                    ("S0", S0), ("ST", ST)):
        _f32(t, name)
    a = ChunkFwdArgs()
    a.B, a.H, a.T, a.dk, a.dv = B, H, T, dk, dv
    a.qkv_dtype, a.o_dtype = _qkv_dtype(q), _qkv_dtype(o)
    a.q, a.k, a.v, a.o = _ptr(q), _ptr(k), _ptr(v), _ptr(o)
    a.alpha_mode = _alpha_mode(log_alpha, 3)
    a.log_alpha = _ptr(log_alpha)
    a.beta_mode = _gate_mode(beta, 3)
    a.beta = _ptr(beta)
    a.gamma_mode = PDN_GAMMA_SAME_AS_BETA if gamma is None else _gate_mode(gamma, 3)
    a.gamma = _ptr(gamma)
    a.key_mode = int(key_mode)
    _precond_fields(a, precond_eps, precond_mode, precond_x)
    a.precond_A0, a.precond_AT = _ptr(precond_A0), _ptr(precond_AT)
    a.S0, a.ST = _ptr(S0), _ptr(ST)
    if workspace is not None:
        a.workspace = _ptr(workspace)
        a.workspace_bytes = workspace.numel() * workspace.element_size()
    return a


def pdn_chunk_fwd_workspace_size(q, k, v, o, log_alpha=None, beta=None, gamma=None,
                                 precond_eps=None, precond_A0=None, precond_AT=None,
                                 S0=None, ST=None, key_mode=PDN_KEY_SYMMETRIC,
                                 precond_mode=PDN_PRECOND_INVERSE, precond_x=1.5) -> int:
    a = _chunk_args(q, k, v, o, log_alpha, beta, gamma, precond_eps, precond_A0,
                    precond_AT, S0, ST, None, key_mode, precond_mode, precond_x)
    n = ctypes.c_size_t(0)
    rc = load_library().pdn_chunk_fwd_workspace_size(ctypes.byref(a), ctypes.byref(n))
    if rc != PDN_OK:
        raise PdnError(rc, "pdn_chunk_fwd_workspace_size")
    return int(n.value)


def pdn_chunk_fwd(q, k, v, o, log_alpha=None, beta=None, gamma=None, precond_eps=None,
                  precond_A0=None, precond_AT=None, S0=None, ST=None, workspace=None,
                  stream=None, key_mode=PDN_KEY_SYMMETRIC, precond_mode=PDN_PRECOND_INVERSE,
                  precond_x=1.5) -> None:
    """Prefill.  Tensors are device tensors in the layouts of include/pdn.h.

    The gate modes follow from the tensors' ranks: log_alpha None / [B,H,T] /
    [B,H,T,dk]; beta [B,H,T] / [B,H,T,dk]; gamma None (same as beta) / [B,H,T]
    / [B,H,T,dv].  key_mode is one of PDN_KEY_*; precond_mode one of
    PDN_PRECOND_* (precond_x is the stabilised mode's bound).  o (float32 or
    bfloat16) receives the output; ST and
    precond_AT, when given, receive the final state and running k(.)k sum.
    workspace: a device tensor of at least pdn_chunk_fwd_workspace_size() bytes.
    When None and the call needs one, it is allocated here with torch's caching
    allocator, whose stream-ordered reuse makes that safe on torch's current
    stream; pass one explicitly when launching on another stream.
    """
    a = _chunk_args(q, k, v, o, log_alpha, beta, gamma, precond_eps, precond_A0,
                    precond_AT, S0, ST, workspace, key_mode, precond_mode, precond_x)
    lib = load_library()
    if workspace is None:
        n = ctypes.c_size_t(0)
        rc = lib.pdn_chunk_fwd_workspace_size(ctypes.byref(a), ctypes.byref(n))
        if rc != PDN_OK:
            raise PdnError(rc, "pdn_chunk_fwd_workspace_size")
        if n.value:
            import torch
            workspace = torch.empty(int(n.value), dtype=torch.uint8, device=q.device)
            a.workspace = _ptr(workspace)
            a.workspace_bytes = int(n.value)
    rc = lib.pdn_chunk_fwd(ctypes.byref(a), _stream(stream))
    if rc != PDN_OK:
        raise PdnError(rc, "pdn_chunk_fwd")


def pdn_chunk_fwd_noalloc(q, k, v, o, log_alpha=None, beta=None, gamma=None, precond_eps=None,
                          precond_A0=None, precond_AT=None, S0=None, ST=None, stream=None,
                          key_mode=PDN_KEY_SYMMETRIC, precond_mode=PDN_PRECOND_INVERSE,
                          precond_x=1.5) -> None:
    """pdn_chunk_fwd without a workspace argument and without any allocation:
    the scratch comes from the library's static per-GPU array of
    PDN_NOALLOC_SCRATCH_BYTES (PdnError with PDN_ESCRATCH when the call needs
    more).  For callers that cannot allocate, e.g. under HIP graph capture.
    Calls on one GPU share that array: they must not overlap."""
    a = _chunk_args(q, k, v, o, log_alpha, beta, gamma, precond_eps, precond_A0,
                    precond_AT, S0, ST, None, key_mode, precond_mode, precond_x)
    rc = load_library().pdn_chunk_fwd_noalloc(ctypes.byref(a), _stream(stream))
    if rc != PDN_OK:
        raise PdnError(rc, "pdn_chunk_fwd_noalloc")


def _bwd_args(q, k, v, dO, dq, dk, dv, dlog_alpha, dbeta, dgamma, dS0, dA0, log_alpha, beta,
              gamma, precond_eps, precond_A0, S0, dST, workspace, key_mode, precond_mode,
              precond_x):
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k must be [B,H,T,dk] and v [B,H,T,dv]")
    B, H, T, dkk = q.shape
    dvv = v.shape[-1]
    if tuple(dq.shape) != (B, H, T, dkk) or tuple(dk.shape) != (B, H, T, dkk):
        raise ValueError("dq, dk must be [B,H,T,dk]")
    if tuple(dv.shape) != (B, H, T, dvv):
        raise ValueError("dv must be [B,H,T,dv]")
    _shape(dST, "dST", None, (B, H, dkk, dvv))
    _shape(dS0, "dS0", None, (B, H, dkk, dvv))
    _shape(dA0, "dA0", None, (B, H, dkk))
    _same_device(q, (("dO", dO), ("dST", dST), ("dq", dq), ("dk", dk), ("dv", dv),
                     ("dlog_alpha", dlog_alpha), ("dbeta", dbeta), ("dgamma", dgamma),
                     ("dS0", dS0), ("dA0", dA0), ("workspace", workspace)))
    for name, t, like in (("dlog_alpha", dlog_alpha, log_alpha), ("dbeta", dbeta, beta),
                          ("dgamma", dgamma, gamma)):
        if (t is None) != (like is None):
            raise ValueError("%s must be given exactly when its gate is" % name)
        if t is not None and tuple(t.shape) != tuple(like.shape):
            raise ValueError("%s must have the shape of its gate" % name)
    f = _chunk_args(q, k, v, dO, log_alpha, beta, gamma, precond_eps, precond_A0, None, S0,
                    None, None, key_mode, precond_mode, precond_x)
    f.o = None
    for name, t in (("dO", dO), ("dST", dST), ("dq", dq), ("dk", dk), ("dv", dv),
                    ("dlog_alpha", dlog_alpha), ("dbeta", dbeta), ("dgamma", dgamma),
                    ("dS0", dS0), ("dA0", dA0)):
        _f32(t, name)
    a = ChunkBwdArgs()
    a.fwd = f
    a.dO, a.dST = _ptr(dO), _ptr(dST)
    a.dq, a.dk, a.dv = _ptr(dq), _ptr(dk), _ptr(dv)
    a.dlog_alpha, a.dbeta, a.dgamma = _ptr(dlog_alpha), _ptr(dbeta), _ptr(dgamma)
    a.dS0, a.dA0 = _ptr(dS0), _ptr(dA0)
    if workspace is not None:
        a.workspace = _ptr(workspace)
        a.workspace_bytes = workspace.numel() * workspace.element_size()
    return a


def pdn_chunk_bwd_workspace_size(q, k, v, dO, dq, dk, dv, dlog_alpha=None, dbeta=None,
                                 dgamma=None, dS0=None, dA0=None, log_alpha=None, beta=None,
                                 gamma=None, precond_eps=None, precond_A0=None, S0=None,
                                 dST=None, key_mode=PDN_KEY_SYMMETRIC,
                                 precond_mode=PDN_PRECOND_INVERSE, precond_x=1.5) -> int:
    a = _bwd_args(q, k, v, dO, dq, dk, dv, dlog_alpha, dbeta, dgamma, dS0, dA0, log_alpha,
                  beta, gamma, precond_eps, precond_A0, S0, dST, None, key_mode, precond_mode,
                  precond_x)
    n = ctypes.c_size_t(0)
    rc = load_library().pdn_chunk_bwd_workspace_size(ctypes.byref(a), ctypes.byref(n))
    if rc != PDN_OK:
        raise PdnError(rc, "pdn_chunk_bwd_workspace_size")
    return int(n.value)


def pdn_chunk_bwd(q, k, v, dO, dq, dk, dv, dlog_alpha=None, dbeta=None, dgamma=None,
                  dS0=None, dA0=None, log_alpha=None, beta=None, gamma=None, precond_eps=None,
                  precond_A0=None, S0=None, dST=None, workspace=None, stream=None,
                  key_mode=PDN_KEY_SYMMETRIC, precond_mode=PDN_PRECOND_INVERSE,
                  precond_x=1.5) -> None:
    """Backward of the prefill: writes the gradients of
    sum <dO, o> + <dST, S_T> into the caller's fp32 tensors dq, dk [B,H,T,dk],
    dv [B,H,T,dv], dlog_alpha / dbeta / dgamma (shapes of their gates; given
    exactly when the gate is), dS0 [B,H,dk,dv] and dA0 [B,H,dk] (optional).
    The forward inputs are passed as to pdn_chunk_fwd.  workspace as for
    pdn_chunk_fwd (allocated here from torch's caching allocator when None).
    """
    a = _bwd_args(q, k, v, dO, dq, dk, dv, dlog_alpha, dbeta, dgamma, dS0, dA0, log_alpha,
                  beta, gamma, precond_eps, precond_A0, S0, dST, workspace, key_mode,
                  precond_mode, precond_x)
    lib = load_library()
    if workspace is None:
        n = ctypes.c_size_t(0)
        rc = lib.pdn_chunk_bwd_workspace_size(ctypes.byref(a), ctypes.byref(n))
        if rc != PDN_OK:
            raise PdnError(rc, "pdn_chunk_bwd_workspace_size")
        if n.value:
            import torch
            workspace = torch.empty(int(n.value), dtype=torch.uint8, device=q.device)
            a.workspace = _ptr(workspace)
            a.workspace_bytes = int(n.value)
    rc = lib.pdn_chunk_bwd(ctypes.byref(a), _stream(stream))
    if rc != PDN_OK:
        raise PdnError(rc, "pdn_chunk_bwd")


def _decode_args(q, k, v, o, S, log_alpha, beta, gamma, precond_eps, precond_A, key_mode,
                 precond_mode=PDN_PRECOND_INVERSE, precond_x=1.5):
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k must be [B,H,dk] and v [B,H,dv]")
    B, H, dk = q.shape
    dv = v.shape[-1]
    if tuple(k.shape) != (B, H, dk) or tuple(v.shape[:2]) != (B, H):
        raise ValueError("q, k must be [B,H,dk] and v [B,H,dv]")
    if tuple(o.shape) != (B, H, dv) or tuple(S.shape) != (B, H, dk, dv):
        raise ValueError("o must be [B,H,dv] and S [B,H,dk,dv]")
    if q.dtype != k.dtype or q.dtype != v.dtype:
        raise ValueError("q, k, v must share one dtype")
    _shape(log_alpha, "log_alpha", None, (B, H), (B, H, dk))
    _shape(beta, "beta", (B, H), (B, H, dk))
    _shape(gamma, "gamma", None, (B, H), (B, H, dv))
    _shape(precond_A, "precond_A", None, (B, H, dk))
    _same_device(q, (("k", k), ("v", v), ("o", o), ("S", S), ("log_alpha", log_alpha),
                     ("beta", beta), ("gamma", gamma), ("precond_A", precond_A)))
    for name, t in (("log_alpha", log_alpha), ("beta", beta), ("gamma", gamma),
                    ("precond_A", precond_A), ("S", S)):
        _f32(t, name)
    a = DecodeArgs()
    a.B, a.H, a.dk, a.dv = B, H, dk, dv
    a.qkv_dtype, a.o_dtype = _qkv_dtype(q), _qkv_dtype(o)
    a.q, a.k, a.v, a.o, a.S = _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(S)
    a.alpha_mode = _alpha_mode(log_alpha, 2)
    a.log_alpha = _ptr(log_alpha)
    a.beta_mode = _gate_mode(beta, 2)
    a.beta = _ptr(beta)
    a.gamma_mode = PDN_GAMMA_SAME_AS_BETA if gamma is None else _gate_mode(gamma, 2)
    a.gamma = _ptr(gamma)
    a.key_mode = int(key_mode)
    _precond_fields(a, precond_eps, precond_mode, precond_x)
    a.precond_A = _ptr(precond_A)
    return a


def pdn_decode_step(q, k, v, o, S, log_alpha=None, beta=None, gamma=None,
                    precond_eps=None, precond_A=None, stream=None,
                    key_mode=PDN_KEY_SYMMETRIC, precond_mode=PDN_PRECOND_INVERSE,
                    precond_x=1.5) -> None:
    """One decode token for all (b,h); S (and precond_A) updated in place."""
    a = _decode_args(q, k, v, o, S, log_alpha, beta, gamma, precond_eps, precond_A,
                     key_mode, precond_mode, precond_x)
    rc = load_library().pdn_decode_step(ctypes.byref(a), _stream(stream))
    if rc != PDN_OK:
        raise PdnError(rc, "pdn_decode_step")


# ---------------------------------------------------------------------------
# the operators around the recurrence
# ---------------------------------------------------------------------------

_torch = None   # torch and its types' codes, from the first call on: a single-token call is
_CODES = {}     # mostly host time, and an import statement in each of its functions is part of it


def _use_torch():
    global _torch, _current_stream
    import torch
    # the stream's handle without an object around it (3 us less), where torch has that
    _current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda index: torch.cuda.current_stream(index).cuda_stream)
    _CODES.update({torch.float32: PDN_F32, torch.bfloat16: PDN_BF16})
    _torch = torch


def _dtype_of(t, name):
    code = _CODES.get(t.dtype)
    if code is None:
        raise ValueError("%s must be float32 or bfloat16, got %s" % (name, t.dtype))
    return code


class _Call:
    """One call's argument struct, with the device that its first tensor sets.

    The checks below are most of what a single-token call costs on the host, so
    each is one comparison on the way through; the message is put together only
    when one fails."""

    __slots__ = ("a", "index", "moved")

    def __init__(self, struct, first):
        if _torch is None:
            _use_torch()
        index = first.get_device() if hasattr(first, "get_device") else -1
        if index < 0:
            raise ValueError("the first argument must be a tensor in device memory")
        self.a, self.index, self.moved = struct(), index, None

    def plain(self, t, name, shape, dtype):
        """Pointer of a contiguous tensor (None stays None)."""
        if t is None:
            return None
        if t.shape != shape or t.dtype != dtype or t.get_device() != self.index or not t.is_contiguous():
            self._refuse(t, name, shape, dtype)
            raise ValueError("%s must be contiguous" % name)
        return t.data_ptr()

    def table(self, a, t, name, shape, dtype):
        """Sets a.<name> to a contiguous tensor of 8-byte numbers, which may be a
        slice of a longer one and so begin 8 bytes off the library's alignment.
        Such a slice is copied on the launch's stream, into memory that begins
        where it has to; until then the field holds an address that only the
        checks see."""
        p = self.plain(t, name, shape, dtype)
        if p and p % 16:
            self.moved = (self.moved or []) + [(a, name, t)]
            p -= p % 16
        setattr(a, name, p)

    def rows(self, t, name, shape, dtype):
        """Pointer of a strided tensor; its last dimension must be contiguous."""
        if t is None:
            return None
        if t.shape != shape or t.dtype != dtype or t.get_device() != self.index or (t.stride(-1) != 1 and shape[-1] != 1):
            self._refuse(t, name, shape, dtype)
            raise ValueError("the last dimension of %s must be contiguous" % name)
        return t.data_ptr()

    def _refuse(self, t, name, shape, dtype):
        if t.shape != shape:
            raise ValueError("%s must have shape %s, got %s" % (name, list(shape), list(t.shape)))
        if not t.is_cuda:
            raise ValueError("%s must live in device memory" % name)
        if t.get_device() != self.index:
            raise ValueError("%s is on %s, the first argument on cuda:%d: every tensor must share its device"
                             % (name, t.device, self.index))
        if t.dtype != dtype:
            raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))

    def size(self, name):
        n = ctypes.c_size_t(0)
        rc = getattr(_lib or load_library(), name)(ctypes.byref(self.a), ctypes.byref(n))
        if rc != PDN_OK:
            raise PdnError(rc, name)
        return n.value

    def launch(self, name, stream, workspace=None):
        """Makes the call on `stream`, or torch's current stream of the tensors'
        device, with that device current.  A workspace that the caller does not
        give comes from torch's caching allocator, allocated on the launch's own
        stream, whose order then protects its reuse."""
        if self.index != _torch.cuda.current_device():
            with _torch.cuda.device(self.index):
                return self.launch(name, stream, workspace)
        a, size = self.a, _SIZES[name]
        lib = _lib or load_library()
        if self.moved:
            # a kernel (a sum with zero), as all that a captured call records
            if stream is None:
                copies = [t + 0 for _, _, t in self.moved]
            else:
                with _torch.cuda.stream(self._stream(stream)):
                    copies = [t + 0 for _, _, t in self.moved]
            for (struct, field, _), t in zip(self.moved, copies):
                setattr(struct, field, t.data_ptr())
        if size:
            if workspace is None:
                n = self.size(size)
                if n and stream is not None:
                    with _torch.cuda.stream(self._stream(stream)):
                        workspace = _torch.empty(n, dtype=_torch.uint8, device="cuda")
                elif n:
                    workspace = _torch.empty(n, dtype=_torch.uint8, device="cuda")
            elif workspace.get_device() != self.index:
                raise ValueError("workspace must be on cuda:%d" % self.index)
            if workspace is not None:
                a.workspace, a.workspace_bytes = _ptr(workspace), workspace.numel() * workspace.element_size()
        if stream is None:
            stream = _current_stream(self.index)
        elif not isinstance(stream, int):
            stream = stream.cuda_stream
        rc = getattr(lib, name)(ctypes.byref(a), stream)
        if rc != PDN_OK:
            raise PdnError(rc, name)

    def _stream(self, stream):
        """torch's object for a stream that the caller gave."""
        if not isinstance(stream, int):
            return stream
        # a handle; 0 is the default stream's
        return _torch.cuda.ExternalStream(stream, device=self.index) if stream else _torch.cuda.default_stream(self.index)


def _qk_norm(c, a, xq, xk, H, norm, eps, wq, wk, q_scale, k_scale, inv_freq, positions, rope_layout, rope_scale):
    if xq.dim() != 4 or xk.dim() != 4:
        raise ValueError("xq and xk must be [B,T,heads,d]")
    B, T, Hq, d = xq.shape
    Hk, dtype = xk.shape[2], xq.dtype
    a.B, a.T, a.H, a.Hq, a.Hk, a.d = B, T, H, Hq, Hk, d
    a.dtype, a.norm, a.eps, a.q_scale, a.k_scale = _dtype_of(xq, "xq"), norm, eps, q_scale, k_scale
    a.xq, a.xk = c.rows(xq, "xq", (B, T, Hq, d), dtype), c.rows(xk, "xk", (B, T, Hk, d), dtype)
    a.xq_sb, a.xq_st, a.xq_sh, _ = xq.stride()
    a.xk_sb, a.xk_st, a.xk_sh, _ = xk.stride()
    a.wq, a.wk = c.plain(wq, "wq", (d,), _torch.float32), c.plain(wk, "wk", (d,), _torch.float32)
    if inv_freq is not None:
        half = inv_freq.shape[0]
        a.rot_dim, a.rope_layout, a.rope_scale = 2 * half, rope_layout, rope_scale
        c.table(a, inv_freq, "inv_freq", (half,), _torch.float64)
        c.table(a, positions, "positions", (B, T), _torch.int64)
    elif positions is not None:
        raise ValueError("positions need inv_freq")
    return B, T, d


def pdn_qk_norm_fwd(xq, xk, q, k, norm=PDN_NORM_L2, eps=1e-6, wq=None, wk=None, q_scale=1.0, k_scale=1.0,
                    inv_freq=None, positions=None, rope_layout=PDN_ROPE_HALF, rope_scale=1.0, stream=None) -> None:
    """Norm of each head's queries and keys, and their rotation, into the
    recurrence's layout: xq [B,T,Hq,d], xk [B,T,Hk,d] (views into a
    projection's rows are fine) to q, k [B,H,T,d], which hold what the
    recurrence takes; an input head serves H / Hq (H / Hk) output heads.

    norm is one of PDN_NORM_*, wq / wk its fp32 weights [d].  inv_freq
    (float64 [rot_dim / 2], see pdn_rope_freqs) turns the rotation on, at
    positions (int64 [B,T]; None = 0, 1, .. in each sequence).  Both may be
    slices of longer tensors, as a generation loop's positions[:, t:t + 1] is: one
    that begins off 16 bytes is copied first, a kernel more."""
    c = _Call(QkNormArgs, xq)
    if q.dim() != 4:
        raise ValueError("q and k must be [B,H,T,d]")
    H = q.shape[1]
    B, T, d = _qk_norm(c, c.a, xq, xk, H, norm, eps, wq, wk, q_scale, k_scale, inv_freq, positions, rope_layout, rope_scale)
    c.a.q, c.a.k = c.plain(q, "q", (B, H, T, d), xq.dtype), c.plain(k, "k", (B, H, T, d), xq.dtype)
    c.launch("pdn_qk_norm_fwd", stream)


def _qk_norm_bwd(xq, xk, dq, dk, dxq, dxk, dwq, dwk, norm, eps, wq, wk, q_scale, k_scale, inv_freq, positions,
                 rope_layout, rope_scale):
    c = _Call(QkNormBwdArgs, xq)
    if dq.dim() != 4:
        raise ValueError("dq and dk must be [B,H,T,d]")
    a, H = c.a, dq.shape[1]
    B, T, d = _qk_norm(c, a.fwd, xq, xk, H, norm, eps, wq, wk, q_scale, k_scale, inv_freq, positions, rope_layout, rope_scale)
    f32 = _torch.float32
    a.dq, a.dk = c.plain(dq, "dq", (B, H, T, d), f32), c.plain(dk, "dk", (B, H, T, d), f32)
    a.dxq, a.dxk = c.rows(dxq, "dxq", xq.shape, xq.dtype), c.rows(dxk, "dxk", xk.shape, xq.dtype)
    a.dxq_sb, a.dxq_st, a.dxq_sh, _ = dxq.stride()
    a.dxk_sb, a.dxk_st, a.dxk_sh, _ = dxk.stride()
    a.dwq, a.dwk = c.plain(dwq, "dwq", (d,), f32), c.plain(dwk, "dwk", (d,), f32)
    return c


def pdn_qk_norm_bwd_workspace_size(xq, xk, dq, dk, dxq, dxk, dwq=None, dwk=None, norm=PDN_NORM_L2, eps=1e-6, wq=None,
                                   wk=None, q_scale=1.0, k_scale=1.0, inv_freq=None, positions=None,
                                   rope_layout=PDN_ROPE_HALF, rope_scale=1.0) -> int:
    return _qk_norm_bwd(xq, xk, dq, dk, dxq, dxk, dwq, dwk, norm, eps, wq, wk, q_scale, k_scale, inv_freq, positions,
                        rope_layout, rope_scale).size("pdn_qk_norm_bwd_workspace_size")


def pdn_qk_norm_bwd(xq, xk, dq, dk, dxq, dxk, dwq=None, dwk=None, norm=PDN_NORM_L2, eps=1e-6, wq=None, wk=None,
                    q_scale=1.0, k_scale=1.0, inv_freq=None, positions=None, rope_layout=PDN_ROPE_HALF, rope_scale=1.0,
                    workspace=None, stream=None) -> None:
    """Backward of pdn_qk_norm_fwd: from dq, dk (fp32 [B,H,T,d], as
    pdn_chunk_bwd writes them) to dxq, dxk (shapes and type of xq, xk; views
    are fine) and, where the norm has weights, dwq, dwk (fp32 [d])."""
    _qk_norm_bwd(xq, xk, dq, dk, dxq, dxk, dwq, dwk, norm, eps, wq, wk, q_scale, k_scale, inv_freq, positions,
                 rope_layout, rope_scale).launch("pdn_qk_norm_bwd", stream, workspace)


def _strides(a, field, t):
    """The strides of a [B,T,heads,d] tensor (None: all zero, as they are)."""
    if t is not None:
        sb, st, sh, _ = t.stride()
        setattr(a, field + "_sb", sb)
        setattr(a, field + "_st", st)
        setattr(a, field + "_sh", sh)


def _out_norm(c, a, o, z, w, like, act, eps):
    if o.dim() != 4:
        raise ValueError("o must be [B,H,T,dv]")
    B, H, T, dv = o.shape
    a.B, a.H, a.T, a.dv = B, H, T, dv
    a.o_dtype, a.dtype, a.eps = _dtype_of(o, "o"), _dtype_of(like, "y and dy"), eps
    a.act = (PDN_ACT_NONE if z is None else PDN_ACT_SILU) if act is None else act
    a.o = c.plain(o, "o", (B, H, T, dv), o.dtype)
    a.z = c.rows(z, "z", (B, T, H, dv), like.dtype)
    _strides(a, "z", z)
    a.w = c.plain(w, "w", (dv,), _torch.float32)
    return B, T, H, dv


def pdn_out_norm_fwd(o, y, z=None, w=None, act=None, eps=1e-6, stream=None) -> None:
    """Gated norm of the recurrence's output, back to the projection's layout:
    o [B,H,T,dv] to y [B,T,H,dv] (a view is fine), times the weights w (fp32
    [dv]) and the gate act(z), z [B,T,H,dv].  act is one of PDN_ACT_*; None
    means PDN_ACT_SILU where z is given."""
    c = _Call(OutNormArgs, o)
    shape = _out_norm(c, c.a, o, z, w, y, act, eps)
    c.a.y = c.rows(y, "y", shape, y.dtype)
    _strides(c.a, "y", y)
    c.launch("pdn_out_norm_fwd", stream)


def _out_norm_bwd(o, dy, do, z, dz, w, dw, act, eps):
    c = _Call(OutNormBwdArgs, o)
    a = c.a
    shape = _out_norm(c, a.fwd, o, z, w, dy, act, eps)
    a.dy, a.dz = c.rows(dy, "dy", shape, dy.dtype), c.rows(dz, "dz", shape, dy.dtype)
    _strides(a, "dy", dy)
    _strides(a, "dz", dz)
    a.d_o = c.plain(do, "do", o.shape, _torch.float32)
    a.dw = c.plain(dw, "dw", shape[-1:], _torch.float32)
    return c


def pdn_out_norm_bwd_workspace_size(o, dy, do, z=None, dz=None, w=None, dw=None, act=None, eps=1e-6) -> int:
    return _out_norm_bwd(o, dy, do, z, dz, w, dw, act, eps).size("pdn_out_norm_bwd_workspace_size")


def pdn_out_norm_bwd(o, dy, do, z=None, dz=None, w=None, dw=None, act=None, eps=1e-6, workspace=None,
                     stream=None) -> None:
    """Backward of pdn_out_norm_fwd: from dy [B,T,H,dv] to do (fp32
    [B,H,T,dv], the dO of pdn_chunk_bwd), dz (given exactly when z is) and dw
    (fp32 [dv], given exactly when w is)."""
    _out_norm_bwd(o, dy, do, z, dz, w, dw, act, eps).launch("pdn_out_norm_bwd", stream, workspace)


def pdn_scan_marks(T: int) -> int:
    """How many states a scan over T tokens keeps in `marks`."""
    n = load_library().pdn_scan_marks(int(T))
    if n < 0:
        raise PdnError(n, "pdn_scan_marks")
    return n


def _scan(c, a, x, log_a, h0, marks, gain):
    if x.dim() != 3:
        raise ValueError("x must be [B,T,D]")
    B, T, D = x.shape
    a.B, a.T, a.D = B, T, D
    a.dtype, a.log_dtype, a.gain = _dtype_of(x, "x"), _dtype_of(log_a, "log_a"), gain
    a.x, a.log_a = c.rows(x, "x", (B, T, D), x.dtype), c.rows(log_a, "log_a", (B, T, D), log_a.dtype)
    a.x_sb, a.x_st, _ = x.stride()
    a.log_a_sb, a.log_a_st, _ = log_a.stride()
    a.h0 = c.plain(h0, "h0", (B, D), _torch.float32)
    a.marks = c.plain(marks, "marks", (B, pdn_scan_marks(T), D), _torch.float32)
    return B, T, D


def _scan_fwd(x, log_a, h, h0, hT, marks, gain):
    c = _Call(ScanArgs, x)
    a = c.a
    B, T, D = _scan(c, a, x, log_a, h0, marks, gain)
    a.h = c.rows(h, "h", (B, T, D), x.dtype)
    a.h_sb, a.h_st, _ = h.stride()
    a.hT = c.plain(hT, "hT", (B, D), _torch.float32)
    return c


def pdn_scan_fwd_workspace_size(x, log_a, h, h0=None, hT=None, marks=None, gain=PDN_GAIN_NONE) -> int:
    return _scan_fwd(x, log_a, h, h0, hT, marks, gain).size("pdn_scan_fwd_workspace_size")


def pdn_scan_fwd(x, log_a, h, h0=None, hT=None, marks=None, gain=PDN_GAIN_NONE, workspace=None, stream=None) -> None:
    """The gated recurrence with a vector state: h_t = exp(log_a_t) h_{t-1} +
    g x_t over x, log_a, h [B,T,D] (views are fine), from h0 to hT (fp32
    [B,D]).  log_a = -inf starts a sequence within a row.  gain is one of
    PDN_GAIN_*.  marks (fp32 [B, pdn_scan_marks(T), D]), when given, receives
    the states that pdn_scan_bwd starts from."""
    _scan_fwd(x, log_a, h, h0, hT, marks, gain).launch("pdn_scan_fwd", stream, workspace)


def _scan_bwd(x, log_a, dh, dx, dlog_a, h0, dhT, dh0, marks, gain):
    c = _Call(ScanBwdArgs, x)
    a = c.a
    B, T, D = _scan(c, a.fwd, x, log_a, h0, marks, gain)
    a.dh, a.dx = c.rows(dh, "dh", (B, T, D), x.dtype), c.rows(dx, "dx", (B, T, D), x.dtype)
    a.dlog_a = c.rows(dlog_a, "dlog_a", (B, T, D), log_a.dtype)
    a.dh_sb, a.dh_st, _ = dh.stride()
    a.dx_sb, a.dx_st, _ = dx.stride()
    a.dlog_a_sb, a.dlog_a_st, _ = dlog_a.stride()
    a.dhT, a.dh0 = c.plain(dhT, "dhT", (B, D), _torch.float32), c.plain(dh0, "dh0", (B, D), _torch.float32)
    return c


def pdn_scan_bwd_workspace_size(x, log_a, dh, dx, dlog_a, h0=None, dhT=None, dh0=None, marks=None,
                                gain=PDN_GAIN_NONE) -> int:
    return _scan_bwd(x, log_a, dh, dx, dlog_a, h0, dhT, dh0, marks, gain).size("pdn_scan_bwd_workspace_size")


def pdn_scan_bwd(x, log_a, dh, dx, dlog_a, h0=None, dhT=None, dh0=None, marks=None, gain=PDN_GAIN_NONE,
                 workspace=None, stream=None) -> None:
    """Backward of pdn_scan_fwd: from dh [B,T,D] and dhT to dx, dlog_a and dh0.
    marks: as the forward wrote them, or None (they are formed here)."""
    _scan_bwd(x, log_a, dh, dx, dlog_a, h0, dhT, dh0, marks, gain).launch("pdn_scan_bwd", stream, workspace)


def pdn_scan_step(x, log_a, h, h_prev, h_next, gain=PDN_GAIN_NONE, stream=None) -> None:
    """One token of the recurrence for every sequence: x, log_a, h [B,D]
    (views are fine), h_prev and h_next fp32 [B,D], which may be one tensor."""
    c = _Call(ScanStepArgs, x)
    if x.dim() != 2:
        raise ValueError("x must be [B,D]")
    a = c.a
    B, D = x.shape
    a.B, a.D = B, D
    a.dtype, a.log_dtype, a.gain = _dtype_of(x, "x"), _dtype_of(log_a, "log_a"), gain
    a.x, a.log_a, a.h = c.rows(x, "x", (B, D), x.dtype), c.rows(log_a, "log_a", (B, D), log_a.dtype), c.rows(h, "h", (B, D), x.dtype)
    a.x_sb, a.log_a_sb, a.h_sb = x.stride(0), log_a.stride(0), h.stride(0)
    a.h_prev, a.h_next = c.plain(h_prev, "h_prev", (B, D), _torch.float32), c.plain(h_next, "h_next", (B, D), _torch.float32)
    c.launch("pdn_scan_step", stream)


def pdn_rope_freqs(rot_dim, base=10000.0, scaling=PDN_ROPE_PLAIN, factor=1.0, original_context=1):
    """(inverse frequencies, a list of rot_dim / 2 floats; rope_scale) for a
    rotation of rot_dim elements, changed for contexts `factor` times as long
    as original_context by one of PDN_ROPE_*."""
    n = int(rot_dim)
    freqs, scale = (ctypes.c_double * max(n // 2, 1))(), _F(1.0)
    rc = load_library().pdn_rope_freqs(n, float(base), int(scaling), float(factor), int(original_context), freqs,
                                       ctypes.byref(scale))
    if rc != PDN_OK:
        raise PdnError(rc, "pdn_rope_freqs")
    return list(freqs), float(scale.value)


# ---------------------------------------------------------------------------
# what a stack with attention layers needs besides the recurrence
# ---------------------------------------------------------------------------

def _in_32_bits(joined):
    """Of numbers joined by |: the structs' fields would take one past 32 bits for another."""
    if joined >> 31:
        raise ValueError("sizes, windows and bounds must lie between 0 and 2^31 - 1")


def _rows3(c, t, name, shape, dtype):
    """Pointer and strides of a [B,T,D] tensor."""
    if t is None:
        return None, 0, 0
    sb, st, _ = t.stride() if t.dim() == 3 else (0, 0, 0)
    return c.rows(t, name, shape, dtype), sb, st


def _seam(c, x, w, eps, drop_p, seed):
    if x.dim() != 3:
        raise ValueError("the rows must be [B,T,D]")
    a, (B, T, D) = c.a, x.shape
    _in_32_bits(B | T | D)
    a.B, a.T, a.D, a.eps, a.drop_p = B, T, D, eps, drop_p
    a.w = c.plain(w, "w", (D,), _torch.float32)
    a.seed = c.plain(seed, "seed", (2,), _torch.int64)
    return B, T, D


def pdn_add_norm_fwd(x, y, res=None, s=None, w=None, eps=1e-6, drop_p=0.0, seed=None, y_scale=None, stream=None) -> None:
    """The seam between two sublayers: s = res + dropout(x), y = its RMS norm times
    w (fp32 [D]), over x, res, s, y [B,T,D] (views are fine; s may be res).

    s, in res's type, is what the norm and the backward read; without res and
    dropout there is none: y is the norm of x.  y is fp32, bf16 or float8_e4m3fn,
    which takes y_scale (fp32 [B,T], a scale a row, or [B,T,D / 32, 64 or 128], one
    for each group of channels): y * y_scale is the value.  drop_p drops elements of x by
    seed (int64 [2] in device memory: a key and a number of the call, such as the
    layer's and step's), the same in pdn_add_norm_bwd; no mask is kept."""
    c = _Call(AddNormArgs, x)
    a = c.a
    B, T, D = shape = _seam(c, x, w, eps, drop_p, seed)
    s_dtype = x.dtype if res is None and s is None else (res if res is not None else s).dtype
    a.dtype, a.s_dtype = _dtype_of(x, "x"), _CODES.get(s_dtype, -1)
    a.x, a.x_sb, a.x_st = _rows3(c, x, "x", shape, x.dtype)
    a.res, a.res_sb, a.res_st = _rows3(c, res, "res", shape, s_dtype)
    a.s, a.s_sb, a.s_st = _rows3(c, s, "s", shape, s_dtype)
    a.y, a.y_sb, a.y_st = _rows3(c, y, "y", shape, y.dtype)
    if y.dtype == _torch.float8_e4m3fn:
        a.y_dtype = PDN_E4M3
        if y_scale is None:
            raise ValueError("y_scale is required for y in 8 bits")
        groups = y_scale.shape[2] if y_scale.dim() == 3 else 1
        if groups < 1 or D % groups:
            raise ValueError("y_scale must be [B,T] or [B,T,groups], groups a divisor of D")
        a.group = D // groups if groups > 1 else 0
        a.y_scale = c.plain(y_scale, "y_scale", (B, T) if y_scale.dim() == 2 else (B, T, groups), _torch.float32)
    else:
        a.y_dtype = _dtype_of(y, "y")
        if y_scale is not None:
            raise ValueError("y_scale goes with y in 8 bits")
    c.launch("pdn_add_norm_fwd", stream)


def _add_norm_bwd(s, dy, dres, ds, dx, w, dw, eps, drop_p, seed):
    c = _Call(AddNormBwdArgs, s)
    a, shape = c.a, _seam(c, s, w, eps, drop_p, seed)
    a.dtype = a.s_dtype = _dtype_of(s, "s")
    a.y_dtype = _dtype_of(dy, "dy")
    if dx is not None:
        a.dtype = _dtype_of(dx, "dx")
        a.dx, a.dx_sb, a.dx_st = _rows3(c, dx, "dx", shape, dx.dtype)
    a.s, a.s_sb, a.s_st = _rows3(c, s, "s", shape, s.dtype)
    a.dy, a.dy_sb, a.dy_st = _rows3(c, dy, "dy", shape, dy.dtype)
    a.ds, a.ds_sb, a.ds_st = _rows3(c, ds, "ds", shape, s.dtype)
    a.dres, a.dres_sb, a.dres_st = _rows3(c, dres, "dres", shape, s.dtype)
    a.dw = c.plain(dw, "dw", shape[-1:], _torch.float32)
    return c


def pdn_add_norm_bwd_workspace_size(s, dy, dres, ds=None, dx=None, w=None, dw=None, eps=1e-6, drop_p=0.0, seed=None) -> int:
    return _add_norm_bwd(s, dy, dres, ds, dx, w, dw, eps, drop_p, seed).size("pdn_add_norm_bwd_workspace_size")


def pdn_add_norm_bwd(s, dy, dres, ds=None, dx=None, w=None, dw=None, eps=1e-6, drop_p=0.0, seed=None, workspace=None,
                     stream=None) -> None:
    """Backward of pdn_add_norm_fwd: from dy and ds (what reaches s otherwise; None =
    zeros), with s as the forward left it (x where it had none), to dres (s's type;
    may be ds), dx (dropped as x was; None = not written) and dw (fp32 [D], given
    exactly when w is)."""
    _add_norm_bwd(s, dy, dres, ds, dx, w, dw, eps, drop_p, seed).launch("pdn_add_norm_bwd", stream, workspace)


def _rows4(c, t, name, shape, dtype):
    """Pointer and strides of a [B,heads,T,d] tensor."""
    p = c.rows(t, name, shape, dtype)
    sb, sh, st, _ = t.stride()
    return p, sb, sh, st


def _attn(c, a, q, k, v, o, lse, scale, window, first):
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q must be [B,H,Tq,d], k and v [B,Hk,Tk,d]")
    (B, H, Tq, d), (_, Hk, Tk, _) = q.shape, k.shape
    _in_32_bits(B | H | Tq | d | Hk | Tk | window)
    a.B, a.H, a.Hk, a.Tq, a.Tk, a.d = B, H, Hk, Tq, Tk, d
    a.dtype, a.o_dtype, a.window = _dtype_of(q, "q"), _dtype_of(o, "o"), window
    a.scale = d ** -0.5 if scale is None else scale
    queries, keys = (B, H, Tq, d), (B, Hk, Tk, d)
    a.q, a.q_sb, a.q_sh, a.q_st = _rows4(c, q, "q", queries, q.dtype)
    a.k, a.k_sb, a.k_sh, a.k_st = _rows4(c, k, "k", keys, q.dtype)
    a.v, a.v_sb, a.v_sh, a.v_st = _rows4(c, v, "v", keys, q.dtype)
    a.o, a.o_sb, a.o_sh, a.o_st = _rows4(c, o, "o", queries, o.dtype)
    a.lse = c.plain(lse, "lse", (B, H, Tq), _torch.float32)
    a.first = c.plain(first, "first", (B, Tq), _torch.int32)


def _attn_fwd(q, k, v, o, lse, scale, window, first):
    c = _Call(AttnArgs, q)
    _attn(c, c.a, q, k, v, o, lse, scale, window, first)
    return c


def pdn_attn_fwd_workspace_size(q, k, v, o, lse=None, scale=None, window=0, first=None) -> int:
    return _attn_fwd(q, k, v, o, lse, scale, window, first).size("pdn_attn_fwd_workspace_size")


def pdn_attn_fwd(q, k, v, o, lse=None, scale=None, window=0, first=None, workspace=None, stream=None) -> None:
    """Causal softmax attention: q, o [B,H,Tq,d], k, v [B,Hk,Tk,d] (views are fine:
    a projection's rows transposed, every n-th of pdn_qk_norm_fwd's heads), the
    queries being the last Tq of Tk tokens and head h reading key head h / (H / Hk).

    scale: None = d^-0.5 (1.0 where q carries it already).  window: the keys that a
    query sees at most, its own the last (0 = all).  first: int32 [B,Tq], the first
    key that each query may see (its sequence's start in a packed row; Tk or more:
    nothing).  lse: fp32 [B,H,Tq], which the backward needs."""
    _attn_fwd(q, k, v, o, lse, scale, window, first).launch("pdn_attn_fwd", stream, workspace)


def _attn_bwd(q, k, v, o, do, lse, dq, dk, dv, scale, window, first):
    c = _Call(AttnBwdArgs, q)
    a = c.a
    if lse is None:
        raise ValueError("lse is required")
    _attn(c, a.fwd, q, k, v, o, lse, scale, window, first)
    a.g_dtype = _dtype_of(dq, "dq")
    a.d_o, a.do_sb, a.do_sh, a.do_st = _rows4(c, do, "do", o.shape, o.dtype)
    a.dq, a.dq_sb, a.dq_sh, a.dq_st = _rows4(c, dq, "dq", q.shape, dq.dtype)
    a.dk, a.dk_sb, a.dk_sh, a.dk_st = _rows4(c, dk, "dk", k.shape, dq.dtype)
    a.dv, a.dv_sb, a.dv_sh, a.dv_st = _rows4(c, dv, "dv", v.shape, dq.dtype)
    return c


def pdn_attn_bwd_workspace_size(q, k, v, o, do, lse, dq, dk, dv, scale=None, window=0, first=None) -> int:
    return _attn_bwd(q, k, v, o, do, lse, dq, dk, dv, scale, window, first).size("pdn_attn_bwd_workspace_size")


def pdn_attn_bwd(q, k, v, o, do, lse, dq, dk, dv, scale=None, window=0, first=None, workspace=None, stream=None) -> None:
    """Backward of pdn_attn_fwd: from do (o's type) to dq, dk, dv (shapes of q, k, v;
    bf16 or fp32, views are fine), with o and lse as the forward wrote them."""
    _attn_bwd(q, k, v, o, do, lse, dq, dk, dv, scale, window, first).launch("pdn_attn_bwd", stream, workspace)


def _cache(c, m, N, k_pages, v_pages, table, lens, starts, max_new):
    if k_pages.dim() != 4 or table.dim() != 2:
        raise ValueError("k_pages and v_pages must be [pages,page_size,Hk,d], table [B,pages of a sequence]")
    shape, B = k_pages.shape, table.shape[0]
    m.pages, m.page_size, m.Hk, m.d = pages, page_size, Hk, d = shape
    m.B, m.N, m.table_width, m.dtype = B, N, table.shape[1], _dtype_of(k_pages, "k_pages")
    m.k_pages, m.v_pages = c.rows(k_pages, "k_pages", shape, k_pages.dtype), c.rows(v_pages, "v_pages", shape, k_pages.dtype)
    m.k_sp, m.k_st, m.k_sh, _ = k_pages.stride()
    m.v_sp, m.v_st, m.v_sh, _ = v_pages.stride()
    m.table = c.plain(table, "table", (B, m.table_width), _torch.int32)
    m.lens = c.plain(lens, "lens", (B,), _torch.int32)
    m.starts = c.plain(starts, "starts", (B + 1,), _torch.int32)
    if starts is None and B > 0 and N % B:
        raise ValueError("without starts every sequence has the same number of new tokens: %d rows, %d sequences" % (N, B))
    if max_new is None:
        max_new = N if starts is not None or B == 0 else N // B
    _in_32_bits(pages | page_size | Hk | d | B | N | max_new)
    m.max_new = max_new


def pdn_cache_append(k, v, k_pages, v_pages, table, lens, starts=None, max_new=None, stream=None) -> None:
    """New tokens' keys and values into a paged cache: k, v [N,Hk,d] (views are fine)
    to k_pages, v_pages [pages,page_size,Hk,d], sequence b's rows starts[b] ..
    starts[b + 1] - 1 (int32 [B + 1]; None: N / B each) to its last tokens of lens[b]
    (int32 [B], the new ones included) by table (int32 [B,width], its pages in
    order).  max_new: at least the most new tokens of any sequence (None: N / B, or N
    with starts: what it says of them sizes the launch, here and in pdn_attn_paged,
    which takes a sequence for a chunk of that many where it is left out)."""
    c = _Call(CacheAppendArgs, k)
    if k.dim() != 3:
        raise ValueError("k and v must be [N,Hk,d]")
    a, N = c.a, k.shape[0]
    _cache(c, a.cache, N, k_pages, v_pages, table, lens, starts, max_new)
    shape = (N, a.cache.Hk, a.cache.d)
    a.k, a.v = c.rows(k, "k", shape, k_pages.dtype), c.rows(v, "v", shape, k_pages.dtype)
    a.k_sn, a.k_sh, _ = k.stride()
    a.v_sn, a.v_sh, _ = v.stride()
    c.launch("pdn_cache_append", stream)


def _attn_paged(q, o, k_pages, v_pages, table, lens, starts, max_new, scale, window, lse):
    c = _Call(AttnPagedArgs, q)
    if q.dim() != 3:
        raise ValueError("q and o must be [N,H,d]")
    a, (N, H, d) = c.a, q.shape
    _cache(c, a.cache, N, k_pages, v_pages, table, lens, starts, max_new)
    if d != a.cache.d:
        raise ValueError("q's heads hold %d channels, the cache's %d" % (d, a.cache.d))
    _in_32_bits(H | window)
    a.H, a.o_dtype, a.window = H, _dtype_of(o, "o"), window
    a.scale = d ** -0.5 if scale is None else scale
    a.q, a.o = c.rows(q, "q", (N, H, d), k_pages.dtype), c.rows(o, "o", (N, H, d), o.dtype)
    a.q_sn, a.q_sh, _ = q.stride()
    a.o_sn, a.o_sh, _ = o.stride()
    a.lse = c.plain(lse, "lse", (N, H), _torch.float32)
    return c


def pdn_attn_paged_workspace_size(q, o, k_pages, v_pages, table, lens, starts=None, max_new=None, scale=None, window=0,
                                  lse=None) -> int:
    return _attn_paged(q, o, k_pages, v_pages, table, lens, starts, max_new, scale, window, lse).size("pdn_attn_paged_workspace_size")


def pdn_attn_paged(q, o, k_pages, v_pages, table, lens, starts=None, max_new=None, scale=None, window=0, lse=None,
                   workspace=None, stream=None) -> None:
    """Attention of new tokens over their sequences' paged caches, which hold their
    own keys and values already: q, o [N,H,d] (views are fine), the rest as in
    pdn_cache_append, scale and window as in pdn_attn_fwd; lse fp32 [N,H] or None.
    Rows that belong to no sequence are left as they were."""
    _attn_paged(q, o, k_pages, v_pages, table, lens, starts, max_new, scale, window, lse).launch("pdn_attn_paged", stream, workspace)
