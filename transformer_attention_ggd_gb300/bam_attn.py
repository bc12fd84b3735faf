"""Thin ctypes binding of the C ABI in include/bam_attn.h.

Argument marshalling only: torch tensors supply device pointers and the
current CUDA stream; every step of the computation runs in the CUDA kernels
of libbam_attn.so.  There is no fallback: if the library is missing or no
GPU is present, calls raise.

The entry points check every tensor argument (CUDA, current device,
contiguous, the dtype and shape the call implies) before the call and raise
ValueError; ``check=False`` skips that for buffers a caller has already
passed through a checked call (a loop over preallocated tensors).

With BAM_ATTN_DEBUG=1 in the environment the debug build
libbam_attn_debug.so is loaded instead (same ABI; every plain bulk copy and
tiled store is bounds-checked on the device, a failed check is reported by
bam_attn_check_status as BAM_ERR_BOUNDS).

The functions carry the C names (bam_attn_fwd, bam_attn_bwd, ...).  The
helpers at the bottom (``attention_forward`` and friends) allocate outputs
and workspace with torch and then call the same entry points.
"""

from __future__ import annotations

import contextlib
import ctypes
import os
import struct
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
DEBUG = os.environ.get("BAM_ATTN_DEBUG", "0") == "1"
LIB_PATH = os.path.join(PKG, "_build", "libbam_attn_debug.so" if DEBUG else "libbam_attn.so")

BAM_OK = 0
BAM_ERR_INVALID_ARG = 1
BAM_ERR_UNSUPPORTED = 2
BAM_ERR_CUDA = 3
BAM_ERR_TIMEOUT = 4
BAM_ERR_WORKSPACE = 5
BAM_ERR_BOUNDS = 6

BAM_OP_FWD, BAM_OP_BWD, BAM_OP_DECODE = 0, 1, 2
BAM_PRIOR_ALPHA, BAM_PRIOR_THETA = 0, 1

BAM_KERNEL_TABLE = 0
BAM_KERNEL_FWD = 1
BAM_KERNEL_BWD_PREP = 2
BAM_KERNEL_BWD = 3
BAM_KERNEL_BWD_FINAL = 4
BAM_KERNEL_DECODE = 5
BAM_KERNEL_DECODE_COMBINE = 6
BAM_KERNEL_KV_APPEND = 7
BAM_KERNEL_TREE_PREP = 8
BAM_KERNEL_TREE = 9
BAM_KERNEL_TREE_COMBINE = 10
BAM_KERNEL_KV_KEEP = 11
BAM_KERNEL_COUNT = 12

# Every symbol that include/bam_attn.h declares.
EXPORTED = (
    "bam_attn_workspace_size",
    "bam_attn_fwd",
    "bam_attn_bwd",
    "bam_attn_decode",
    "bam_attn_decode_varlen",
    "bam_attn_decode_paged",
    "bam_attn_check_status",
    "bam_status_string",
    "bam_attn_profile_events",
    "bam_attn_launch_count",
    "bam_attn_decode_noalloc",
    "bam_attn_decode_noalloc_check_status",
    "bam_attn_selftest_wait",
    "bam_attn_debug_build",
    "bam_attn_debug_arm_giveup",
    "bam_attn_debug_arm_giveup_noalloc",
    "bam_attn_bwd_schedule",
    "bam_kv_append_paged",
    "bam_attn_decode_tree_paged",
    "bam_attn_tree_workspace_size",
    "bam_kv_keep_paged",
    "bam_paged_call",
)

# Size of the fixed device scratch of bam_attn_decode_noalloc.
BAM_DECODE_NOALLOC_SCRATCH_BYTES = 4 << 20
# Workspace of bam_kv_append_paged and bam_kv_keep_paged (status words only).
BAM_CACHE_WORKSPACE_BYTES = 256
# Most nodes of a draft with parents (tree attention, keep).
BAM_TREE_MAX_NODES = 128


class BamError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {bam_status_string(status)} (status {status})")


class BamParams(ctypes.Structure):
    _fields_ = [
        ("alpha", ctypes.c_void_p),
        ("beta", ctypes.c_void_p),
        ("mu", ctypes.c_void_p),
        ("s", ctypes.c_void_p),
        ("eps", ctypes.c_float),
        ("causal", ctypes.c_int),
        ("ssmax", ctypes.c_int),
        ("prior", ctypes.c_int),
    ]


class BamRope(ctypes.Structure):
    _fields_ = [
        ("base", ctypes.c_double),
        ("dims", ctypes.c_int),
        ("interleaved", ctypes.c_int),
    ]


_lib = None
_lock = threading.Lock()


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libbam_attn.so and declare its signatures (no GPU needed)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
        lib = ctypes.CDLL(path)
        vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        pp = ctypes.POINTER(BamParams)
        lib.bam_attn_workspace_size.restype = sz
        lib.bam_attn_workspace_size.argtypes = [i, i, i, i, i]
        lib.bam_attn_fwd.restype = i
        lib.bam_attn_fwd.argtypes = [vp, vp, vp, vp, i, vp, i, i, i, i, pp, vp, sz, vp]
        lib.bam_attn_bwd.restype = i
        lib.bam_attn_bwd.argtypes = [vp, vp, vp, vp, i, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                     i, i, i, i, pp, vp, sz, vp]
        lib.bam_attn_decode.restype = i
        lib.bam_attn_decode.argtypes = [vp, vp, vp, vp, i, vp, i, i, i, i, pp, vp, sz, vp]
        lib.bam_attn_decode_paged.restype = i
        lib.bam_attn_decode_paged.argtypes = [vp, vp, vp, vp, vp, vp, i, vp, i, i, i, i, i, i, pp,
                                              vp, sz, vp]
        lib.bam_attn_decode_varlen.restype = i
        lib.bam_attn_decode_varlen.argtypes = [vp, vp, vp, vp, vp, i, vp, i, i, i, i, pp, vp, sz,
                                               vp]
        lib.bam_attn_check_status.restype = i
        lib.bam_attn_check_status.argtypes = [vp, vp]
        lib.bam_status_string.restype = ctypes.c_char_p
        lib.bam_status_string.argtypes = [i]
        lib.bam_attn_profile_events.restype = i
        lib.bam_attn_profile_events.argtypes = [i, vp, vp]
        lib.bam_attn_launch_count.restype = ctypes.c_uint64
        lib.bam_attn_launch_count.argtypes = []
        lib.bam_attn_decode_noalloc.restype = i
        lib.bam_attn_decode_noalloc.argtypes = [vp, vp, vp, vp, i, vp, i, i, i, i, pp, vp]
        lib.bam_attn_selftest_wait.restype = i
        lib.bam_attn_selftest_wait.argtypes = [vp, sz, vp]
        lib.bam_attn_debug_build.restype = i
        lib.bam_attn_debug_build.argtypes = []
        lib.bam_attn_decode_noalloc_check_status.restype = i
        lib.bam_attn_decode_noalloc_check_status.argtypes = [vp]
        lib.bam_attn_debug_arm_giveup.restype = i
        lib.bam_attn_debug_arm_giveup.argtypes = [vp, i]
        lib.bam_attn_debug_arm_giveup_noalloc.restype = i
        lib.bam_attn_debug_arm_giveup_noalloc.argtypes = [i]
        ip = ctypes.POINTER(ctypes.c_int)
        lib.bam_attn_bwd_schedule.restype = i
        lib.bam_attn_bwd_schedule.argtypes = [i, i, i, i, i, ip, ip, i]
        lp = ctypes.POINTER(ctypes.c_int64)
        lib.bam_kv_append_paged.restype = i
        lib.bam_kv_append_paged.argtypes = [vp] * 4 + [lp] + [vp] * 6 + [i] * 8 + [
            ctypes.POINTER(BamRope), vp, sz, vp]
        lib.bam_attn_decode_tree_paged.restype = i
        lib.bam_attn_decode_tree_paged.argtypes = [vp] * 8 + [i, vp] + [i] * 8 + [pp, vp, sz, vp]
        lib.bam_attn_tree_workspace_size.restype = sz
        lib.bam_attn_tree_workspace_size.argtypes = [i] * 6
        lib.bam_kv_keep_paged.restype = i
        lib.bam_kv_keep_paged.argtypes = [vp] * 8 + [i] * 7 + [vp, sz, vp]
        lib.bam_paged_call.restype = i
        lib.bam_paged_call.argtypes = [i, ctypes.c_char_p]
        _lib = lib
        return lib


# ---------------------------------------------------------------- raw entry points

def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def make_params(alpha, beta, mu, s=None, eps=1e-5, causal=True, ssmax=False,
                prior=BAM_PRIOR_ALPHA) -> BamParams:
    """alpha, beta, mu, s: contiguous float32 CUDA tensors of length H, which
    the returned struct keeps alive.  prior: BAM_PRIOR_ALPHA, or
    BAM_PRIOR_THETA when alpha, beta, mu hold the thetas."""
    import torch
    if not isinstance(alpha, torch.Tensor) or alpha.dim() != 1:
        raise ValueError("alpha must be a 1-D tensor of length H")
    H = alpha.shape[0]
    for name, t in (("alpha", alpha), ("beta", beta), ("mu", mu), ("s", s)):
        _require(t, name, (H,), (torch.float32,), alpha.device, optional=name == "s")
    if ssmax and s is None:
        raise ValueError("ssmax needs the per-head scale s")
    prm = BamParams(alpha.data_ptr(), beta.data_ptr(), mu.data_ptr(),
                    s.data_ptr() if s is not None else None, float(eps), int(bool(causal)),
                    int(bool(ssmax)), int(prior))
    prm.tensors = (alpha, beta, mu, s)
    return prm


# ---------------------------------------------------------------- argument checks
# The C ABI sees raw pointers and sizes only; these checks keep a tensor of
# the wrong shape, dtype, device or layout from reaching the kernels, which
# would read or write outside its storage.

def _require(t, name, shape, dtypes, device, optional=False):
    import torch
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if (t.dtype in dtypes and t.shape == shape and t.is_contiguous()
            and t.device == device):
        return
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _device(q, name="q"):
    """The CUDA device of q (called `name` in errors), which must be the current device (the library
    launches there, on that device's stream)."""
    import torch
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if q.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {q.device}, but cuda:{torch.cuda.current_device()} is "
                         "the current device")
    return q.device


_DTYPES = None


def _dt():
    """The dtype tuples the entry points accept: bf16, fp32, an output (fp32
    or bf16) and int32."""
    global _DTYPES
    if _DTYPES is None:
        import torch
        _DTYPES = ((torch.bfloat16,), (torch.float32,), (torch.float32, torch.bfloat16),
                   (torch.int32,))
    return _DTYPES


def _check_tensors(specs, device):
    """specs: (name, tensor, shape, dtypes, optional) per argument.  One quick
    pass over all of them; only when one fails does the detailed pass run,
    which raises for the first bad argument."""
    for name, t, shape, dtypes, optional in specs:
        if t is None:
            if optional:
                continue
            break
        try:
            if not (t.dtype in dtypes and t.shape == shape and t.is_contiguous()
                    and t.device == device):
                break
        except AttributeError:
            break
    else:
        return
    for name, t, shape, dtypes, optional in specs:
        _require(t, name, shape, dtypes, device, optional)
    raise ValueError("argument check failed")


def _param_specs(params: BamParams, H: int):
    tensors = getattr(params, "tensors", None)
    if tensors is None:
        return ()  # built by hand from raw pointers: the caller vouches for them
    f32 = _dt()[1]
    return tuple((n, t, (H,), f32, n == "s")
                 for n, t in zip(("alpha", "beta", "mu", "s"), tensors))


def _check_ws(ws, device):
    import torch
    if not isinstance(ws, torch.Tensor) or ws.dtype != torch.uint8 or ws.dim() != 1:
        raise ValueError("ws must be a 1-D uint8 tensor (see workspace())")
    if ws.device != device or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous tensor on {device}")


def _check(status: int, where: str):
    if status != BAM_OK:
        raise BamError(status, where)


def bam_status_string(status: int) -> str:
    return load_library().bam_status_string(int(status)).decode()


def bam_attn_tree_workspace_size(B: int, H: int, Hkv: int, N: int, Tmax: int, D: int = 64) -> int:
    return int(load_library().bam_attn_tree_workspace_size(B, H, Hkv, N, Tmax, D))


def bam_attn_workspace_size(op: int, B: int, H: int, T: int, D: int = 64) -> int:
    return int(load_library().bam_attn_workspace_size(op, B, H, T, D))


def bam_attn_fwd(q, k, v, o, lse, params: BamParams, ws, stream=None, check=True) -> None:
    import torch
    B, H, T, D = q.shape
    if check:
        dev = _device(q)
        bf, f32, out, _ = _dt()
        x4 = (B, H, T, D)
        _check_tensors((("q", q, x4, bf, False), ("k", k, x4, bf, False), ("v", v, x4, bf, False),
                        ("o", o, x4, out, False), ("lse", lse, (B, H, T), f32, True))
                       + _param_specs(params, H), dev)
        _check_ws(ws, dev)
    o_fp32 = 1 if o.dtype == torch.float32 else 0
    st = load_library().bam_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), o_fp32, _ptr(lse), B, H,
                                     T, D, ctypes.byref(params), _ptr(ws), ws.numel(),
                                     _stream(stream))
    _check(st, "bam_attn_fwd")


def bam_attn_bwd(q, k, v, o, lse, dO, dq, dk, dv, dalpha, dbeta, dmu, ds, params: BamParams,
                 ws, stream=None, check=True) -> None:
    import torch
    B, H, T, D = q.shape
    if check:
        dev = _device(q)
        bf, f32, out, _ = _dt()
        x4 = (B, H, T, D)
        _check_tensors(tuple((n, t, x4, bf, False) for n, t in (
                           ("q", q), ("k", k), ("v", v), ("dO", dO), ("dq", dq), ("dk", dk),
                           ("dv", dv)))
                       + (("o", o, x4, out, False), ("lse", lse, (B, H, T), f32, False))
                       + tuple((n, t, (H,), f32, False) for n, t in (
                           ("dalpha", dalpha), ("dbeta", dbeta), ("dmu", dmu), ("ds", ds)))
                       + _param_specs(params, H), dev)
        _check_ws(ws, dev)
    o_fp32 = 1 if o.dtype == torch.float32 else 0
    st = load_library().bam_attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), o_fp32, _ptr(lse),
                                     _ptr(dO), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dalpha),
                                     _ptr(dbeta), _ptr(dmu), _ptr(ds), B, H, T, D,
                                     ctypes.byref(params), _ptr(ws), ws.numel(),
                                     _stream(stream))
    _check(st, "bam_attn_bwd")


def _decode_specs(q, o, lse, B, H, D):
    bf, f32, out, _ = _dt()
    return (("q", q, (B, H, D), bf, False), ("o", o, (B, H, D), out, False),
            ("lse", lse, (B, H), f32, True))


def bam_attn_decode(q, kc, vc, o, lse, params: BamParams, ws, stream=None, check=True) -> None:
    import torch
    B, H, Tkv, D = kc.shape
    if check:
        dev = _device(q)
        bf = _dt()[0]
        kv = (B, H, Tkv, D)
        _check_tensors((("kc", kc, kv, bf, False), ("vc", vc, kv, bf, False))
                       + _decode_specs(q, o, lse, B, H, D) + _param_specs(params, H), dev)
        _check_ws(ws, dev)
    o_fp32 = 1 if o.dtype == torch.float32 else 0
    st = load_library().bam_attn_decode(_ptr(q), _ptr(kc), _ptr(vc), _ptr(o), o_fp32, _ptr(lse),
                                        B, H, Tkv, D, ctypes.byref(params), _ptr(ws), ws.numel(),
                                        _stream(stream))
    _check(st, "bam_attn_decode")


def bam_attn_decode_varlen(q, kc, vc, cache_lens, o, lse, params: BamParams, ws,
                           stream=None, check=True) -> None:
    """cache_lens: int32 CUDA tensor [B] (each in [1, Tmax]); kc, vc: [B,H,Tmax,64]."""
    import torch
    B, H, Tmax, D = kc.shape
    if check:
        dev = _device(q)
        bf, _, _, i32 = _dt()
        _check_tensors((("kc", kc, (B, H, Tmax, D), bf, False),
                        ("vc", vc, (B, H, Tmax, D), bf, False),
                        ("cache_lens", cache_lens, (B,), i32, False))
                       + _decode_specs(q, o, lse, B, H, D) + _param_specs(params, H), dev)
        _check_ws(ws, dev)
    o_fp32 = 1 if o.dtype == torch.float32 else 0
    st = load_library().bam_attn_decode_varlen(_ptr(q), _ptr(kc), _ptr(vc), _ptr(cache_lens),
                                               _ptr(o), o_fp32, _ptr(lse), B, H, Tmax, D,
                                               ctypes.byref(params), _ptr(ws), ws.numel(),
                                               _stream(stream))
    _check(st, "bam_attn_decode_varlen")


def bam_attn_decode_paged(q, k_pages, v_pages, block_table, cache_lens, o, lse,
                          params: BamParams, ws, stream=None, check=True) -> None:
    """k_pages, v_pages: [num_pages, H, page, 64]; block_table int32 [B, max_blocks];
    cache_lens int32 [B]."""
    import torch
    num_pages, H, page, D = k_pages.shape
    B, max_blocks = block_table.shape
    if check:
        dev = _device(q)
        bf, _, _, i32 = _dt()
        pages = (num_pages, H, page, D)
        _check_tensors((("k_pages", k_pages, pages, bf, False),
                        ("v_pages", v_pages, pages, bf, False),
                        ("block_table", block_table, (B, max_blocks), i32, False),
                        ("cache_lens", cache_lens, (B,), i32, False))
                       + _decode_specs(q, o, lse, B, H, D) + _param_specs(params, H), dev)
        _check_ws(ws, dev)
    o_fp32 = 1 if o.dtype == torch.float32 else 0
    st = load_library().bam_attn_decode_paged(_ptr(q), _ptr(k_pages), _ptr(v_pages),
                                              _ptr(block_table), _ptr(cache_lens), _ptr(o),
                                              o_fp32, _ptr(lse), B, H, page, max_blocks,
                                              num_pages, D, ctypes.byref(params), _ptr(ws),
                                              ws.numel(), _stream(stream))
    _check(st, "bam_attn_decode_paged")


def bam_attn_decode_noalloc(q, kc, vc, o, lse, params: BamParams, stream=None,
                            check=True) -> None:
    """Decode for callers that cannot allocate device memory (plugin-style
    hosts that only pass input/output pointers; loops that cannot afford
    cudaMalloc's possible synchronisation): no workspace argument, scratch
    from the library's fixed device array.  Overlapping calls race."""
    import torch
    B, H, Tkv, D = kc.shape
    if check:
        dev = _device(q)
        bf = _dt()[0]
        kv = (B, H, Tkv, D)
        _check_tensors((("kc", kc, kv, bf, False), ("vc", vc, kv, bf, False))
                       + _decode_specs(q, o, lse, B, H, D) + _param_specs(params, H), dev)
    o_fp32 = 1 if o.dtype == torch.float32 else 0
    st = load_library().bam_attn_decode_noalloc(_ptr(q), _ptr(kc), _ptr(vc), _ptr(o), o_fp32,
                                                _ptr(lse), B, H, Tkv, D, ctypes.byref(params),
                                                _stream(stream))
    _check(st, "bam_attn_decode_noalloc")


# ---------------------------------------------------------------- drafted tokens, paged cache

def make_rope(base=10000.0, dims=64, interleaved=False) -> BamRope:
    """Rotation by position of the first `dims` dimensions (a multiple of 16
    up to 64; 0: none).  interleaved: pairs (2f, 2f+1) instead of
    (f, f + dims/2)."""
    if not 0 <= int(dims) <= 64 or int(dims) % 16:
        raise ValueError("dims must be a multiple of 16 from 0 to 64")
    if not 1.0 <= float(base) < float("inf"):
        raise ValueError("base must be at least 1 and finite")
    return BamRope(float(base), int(dims), int(bool(interleaved)))


def _cache_specs(k_pages, v_pages, block_table, cache_lens, draft_lens, parents, B, N):
    """Specs of a paged cache and the drafts behind its committed keys."""
    if k_pages.dim() != 4 or block_table.dim() != 2:
        raise ValueError("k_pages must be [num_pages, Hkv, page, 64] and block_table "
                         "[B, max_blocks]")
    bf, _, _, i32 = _dt()
    pages = tuple(k_pages.shape[:3]) + (64,)
    return (("k_pages", k_pages, pages, bf, False), ("v_pages", v_pages, pages, bf, False),
            ("block_table", block_table, (B, block_table.shape[1]), i32, False),
            ("cache_lens", cache_lens, (B,), i32, False),
            ("draft_lens", draft_lens, (B,), i32, True),
            ("parents", parents, (B, N), i32, True))


def _check_rows(t, name, shape, device):
    """A bf16 input whose rows of 64 are contiguous and 16-byte aligned; the
    other strides are free."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} has dtype {t.dtype}, expected torch.bfloat16")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.stride(3) != 1 or any(x % 8 for x in t.stride()[:3]) or t.data_ptr() % 16:
        raise ValueError(f"{name} must have contiguous, 16-byte aligned rows")


# A decoding step calls these operators once per layer and token, and a call of
# theirs lasts a few microseconds on the GPU: the checks of a call in order are
# a handful of attribute reads per tensor, and only a call that fails them goes
# through the detailed ones above, which say what is wrong.

def _raw_stream(stream, index):
    import torch
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _address(t):
    return 0 if t is None else t.data_ptr()


def _struct_address(x, kind):
    if x is None:
        return 0
    if not isinstance(x, kind):
        raise TypeError(f"expected {kind.__name__}, got {type(x).__name__}")
    return ctypes.addressof(x)


# The words of bam_paged_call: a foreign call with 22 arguments takes 5 us, one
# with its words packed 1 us.
_append_words = struct.Struct("32q").pack
_tree_words = struct.Struct("22q").pack
_keep_words = struct.Struct("18q").pack


def _all_ok(index, pool, k_pages, v_pages, table, block_table, cache_lens, draft_lens, parents, ws,
            B, N, specs):
    """The cache's tensors and those of specs (tensor, dtype, shape) are contiguous, on CUDA
    device `index`, of their dtypes and shapes.  pool, table: the shapes of k_pages and
    block_table."""
    import torch
    bf, i32, lens = torch.bfloat16, torch.int32, (B,)
    specs += ((k_pages, bf, pool), (v_pages, bf, pool), (block_table, i32, table),
              (cache_lens, i32, lens))
    if draft_lens is not None:
        specs += ((draft_lens, i32, lens),)
    if parents is not None:
        specs += ((parents, i32, (B, N)),)
    for t, dtype, shape in specs:
        if (t.dtype is not dtype or t.get_device() != index or t.shape != shape
                or not t.is_contiguous()):
            return False
    return (pool[3] == 64 and len(table) == 2 and table[0] == B and ws.dtype is torch.uint8
            and ws.get_device() == index and ws.dim() == 1 and ws.is_contiguous())


def _rows_ok(index, shape, t):
    import torch
    if t.dtype is not torch.bfloat16 or t.get_device() != index or t.shape != shape:
        return False
    a, b, c, d = t.stride()
    return d == 1 and not (a | b | c) & 7 and not t.data_ptr() & 15


def _current_device():
    import torch
    return torch._C._cuda_getDevice()


def bam_kv_append_paged(k, v, k_pages, v_pages, block_table, cache_lens, new_lens, parents, q,
                        q_out, rope, ws, stream=None, check=True) -> None:
    """Append k, v [B, Hkv, N, 64] (any batch, head and token strides) to the
    pages [num_pages, Hkv, page, 64] behind cache_lens [B] committed keys, the
    keys rotated by their positions.  new_lens int32 [B] or None: tokens of
    each sequence; parents int32 [B, N] or None: the tree that positions
    follow; q [B, H, N, 64] -> q_out (contiguous) or both None: queries rotated
    on the way; rope: make_rope(...) or None."""
    B, Hkv, N, D = shape = k.shape
    num_pages, pool_heads, page, _ = pool = k_pages.shape
    table = block_table.shape
    index = k.get_device()
    H = Hkv
    strides = k.stride()[:3] + v.stride()[:3]
    if q is not None:
        H = q.shape[1]
        strides += q.stride()[:3]
    if check:
        import torch
        try:
            ok = (index >= 0 and index == _current_device() and D == 64 and pool_heads == Hkv
                  and _rows_ok(index, shape, k) and _rows_ok(index, shape, v)
                  and (q is None) == (q_out is None)
                  and (q is None or _rows_ok(index, (B, H, N, 64), q))
                  and _all_ok(index, pool, k_pages, v_pages, table, block_table, cache_lens,
                              new_lens, parents, ws, B, N,
                              () if q is None else ((q_out, torch.bfloat16, (B, H, N, 64)),)))
        except AttributeError:
            ok = False
        if not ok:
            dev = _device(k, "k")
            _check_rows(k, "k", (B, pool_heads, N, 64), dev)
            _check_rows(v, "v", shape, dev)
            if (q is None) != (q_out is None):
                raise ValueError("q and q_out go together")
            if q is not None:
                _check_rows(q, "q", (B, H, N, 64), dev)
            _check_tensors(_cache_specs(k_pages, v_pages, block_table, cache_lens, new_lens,
                                        parents, B, N)
                           + (("q_out", q_out, (B, H, N, 64), _dt()[0], True),), dev)
            _check_ws(ws, dev)
            raise ValueError("argument check failed")
    if q is None:
        strides += (0, 0, 0)
    st = load_library().bam_paged_call(0, _append_words(
        k.data_ptr(), v.data_ptr(), _address(q), _address(q_out),
        1, k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(),
        cache_lens.data_ptr(), _address(new_lens), _address(parents), B, H, Hkv, N, page,
        table[1], num_pages, D, _struct_address(rope, BamRope), ws.data_ptr(),
        ws.numel(), _raw_stream(stream, index), *strides))
    if st:
        _check(st, "bam_kv_append_paged")


def bam_attn_decode_tree_paged(q, k_pages, v_pages, block_table, cache_lens, draft_lens, parents,
                               o, lse, params: BamParams, ws, stream=None, check=True) -> None:
    """q, o: [B, H, N, 64]; pages [num_pages, Hkv, page, 64] that hold each
    sequence's committed keys and, behind them, its draft's; cache_lens int32
    [B] (committed keys); draft_lens int32 [B] or None (N each); parents int32
    [B, N] or None (a chain); lse [B, H, N] or None."""
    import torch
    B, H, N, D = shape = q.shape
    num_pages, Hkv, page, _ = pool = k_pages.shape
    table = block_table.shape
    index = q.get_device()
    out = o.dtype
    if check:
        f32 = torch.float32
        try:
            prm = getattr(params, "tensors", None)
            specs = ((q, torch.bfloat16, shape), (o, out, shape))
            if lse is not None:
                specs += ((lse, f32, (B, H, N)),)
            if prm is not None:
                specs += ((prm[0], f32, (H,)), (prm[1], f32, (H,)), (prm[2], f32, (H,)))
                if prm[3] is not None:
                    specs += ((prm[3], f32, (H,)),)
            ok = (index >= 0 and index == _current_device() and D == 64
                  and (out is torch.bfloat16 or out is f32)
                  and _all_ok(index, pool, k_pages, v_pages, table, block_table, cache_lens,
                              draft_lens, parents, ws, B, N, specs))
        except AttributeError:
            ok = False
        if not ok:
            dev = _device(q)
            bf, f32s, outs, _ = _dt()
            _check_tensors((("q", q, (B, H, N, 64), bf, False),
                            ("o", o, (B, H, N, 64), outs, False),
                            ("lse", lse, (B, H, N), f32s, True))
                           + _cache_specs(k_pages, v_pages, block_table, cache_lens, draft_lens,
                                          parents, B, N) + _param_specs(params, H), dev)
            _check_ws(ws, dev)
            raise ValueError("argument check failed")
    st = load_library().bam_paged_call(1, _tree_words(
        q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(),
        cache_lens.data_ptr(), _address(draft_lens), _address(parents), o.data_ptr(),
        1 if out is torch.float32 else 0, _address(lse), B, H, Hkv, N, page,
        table[1], num_pages, D, _struct_address(params, BamParams), ws.data_ptr(),
        ws.numel(), _raw_stream(stream, index)))
    if st:
        _check(st, "bam_attn_decode_tree_paged")


def bam_kv_keep_paged(k_pages, v_pages, block_table, cache_lens, draft_lens, parents, accepted,
                      new_lens, ws, stream=None, check=True) -> None:
    """Keep the path from the root to node accepted[b] (int32 [B], -1: none)
    of each draft; new_lens int32 [B] (may be cache_lens) gets the lengths."""
    num_pages, Hkv, page, D = pool = k_pages.shape
    table = block_table.shape
    B = table[0]
    N = parents.shape[1] if parents is not None else BAM_TREE_MAX_NODES
    index = k_pages.get_device()
    if parents is None and draft_lens is None:
        raise ValueError("draft_lens is required without parents")
    if check:
        import torch
        try:
            ok = (index >= 0 and index == _current_device()
                  and _all_ok(index, pool, k_pages, v_pages, table, block_table, cache_lens,
                              draft_lens, parents, ws, B, N,
                              ((accepted, torch.int32, (B,)), (new_lens, torch.int32, (B,)))))
        except AttributeError:
            ok = False
        if not ok:
            dev = _device(k_pages, "k_pages")
            i32 = _dt()[3]
            _check_tensors(_cache_specs(k_pages, v_pages, block_table, cache_lens, draft_lens,
                                        parents, B, N)
                           + (("accepted", accepted, (B,), i32, False),
                              ("new_lens", new_lens, (B,), i32, False)), dev)
            _check_ws(ws, dev)
            raise ValueError("argument check failed")
    st = load_library().bam_paged_call(2, _keep_words(
        k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(), cache_lens.data_ptr(),
        _address(draft_lens), _address(parents), accepted.data_ptr(), new_lens.data_ptr(), B, Hkv,
        N, page, table[1], num_pages, D, ws.data_ptr(), ws.numel(),
        _raw_stream(stream, index)))
    if st:
        _check(st, "bam_kv_keep_paged")


def bam_attn_selftest_wait(ws, stream=None) -> None:
    """Launch the failure-detection self-test: a bounded wait that runs out
    and records BAM_ERR_TIMEOUT in the status word of `ws` (about 2 s)."""
    _check(load_library().bam_attn_selftest_wait(_ptr(ws), ws.numel(), _stream(stream)),
           "bam_attn_selftest_wait")


def bam_attn_check_status(ws, stream=None) -> int:
    return int(load_library().bam_attn_check_status(_ptr(ws), _stream(stream)))


def bam_attn_decode_noalloc_check_status(stream=None) -> int:
    """Status of the no-alloc decode calls on the current device since the
    previous check (synchronises the stream; reads and clears)."""
    return int(load_library().bam_attn_decode_noalloc_check_status(_stream(stream)))


def bam_attn_debug_build() -> bool:
    """True when the loaded library is the bounds-checking debug build."""
    return bool(load_library().bam_attn_debug_build())


def bam_attn_debug_arm_giveup(ws, n: int) -> int:
    """Debug build: the n-th bounded device wait of the next calls on `ws`
    gives up (0 disarms).  Returns the status (BAM_ERR_UNSUPPORTED in the
    release build)."""
    return int(load_library().bam_attn_debug_arm_giveup(_ptr(ws), int(n)))


def bam_attn_debug_arm_giveup_noalloc(n: int) -> int:
    """As bam_attn_debug_arm_giveup, for the no-alloc decode's scratch."""
    return int(load_library().bam_attn_debug_arm_giveup_noalloc(int(n)))


def bam_attn_profile_events(which: int, before=None, after=None) -> None:
    b = ctypes.c_void_p(before.cuda_event) if before is not None else None
    a = ctypes.c_void_p(after.cuda_event) if after is not None else None
    _check(load_library().bam_attn_profile_events(which, b, a), "bam_attn_profile_events")


def bam_attn_launch_count() -> int:
    return int(load_library().bam_attn_launch_count())


def bam_attn_bwd_schedule(B: int, H: int, T: int, causal: bool, grid: int):
    """The causal backward's per-CTA item lists for `grid` CTAs (host only):
    a list of item-index lists, CTA by CTA, or None when the kernel deals
    items out round-robin itself.  Item w is key tile w // (B*H) of
    (b, h) = w % (B*H)."""
    nkb = (T + 127) // 128
    total = nkb * B * H
    g = min(grid, total)
    start = (ctypes.c_int * (g + 1))()
    item = (ctypes.c_int * max(total, 1))()
    n = int(load_library().bam_attn_bwd_schedule(int(B), int(H), int(T), int(bool(causal)),
                                                 int(grid), start, item, total))
    if n < 0:
        raise BamError(BAM_ERR_INVALID_ARG, "bam_attn_bwd_schedule")
    if n == 0:
        return None
    return [list(item[start[c]:start[c + 1]]) for c in range(g)]


# ---------------------------------------------------------------- allocating helpers

def workspace(op: int, B: int, H: int, T: int, device="cuda"):
    import torch
    n = bam_attn_workspace_size(op, B, H, T, 64)
    if n == 0:
        raise BamError(BAM_ERR_INVALID_ARG, "bam_attn_workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def tree_workspace(B: int, H: int, Hkv: int, N: int, Tmax: int, device="cuda"):
    """Workspace of bam_attn_decode_tree_paged (Tmax = max_blocks * page)."""
    import torch
    n = bam_attn_tree_workspace_size(B, H, Hkv, N, Tmax, 64)
    if n == 0:
        raise BamError(BAM_ERR_INVALID_ARG, "bam_attn_tree_workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def cache_workspace(device="cuda"):
    """Workspace of bam_kv_append_paged and bam_kv_keep_paged."""
    import torch
    return torch.zeros(BAM_CACHE_WORKSPACE_BYTES, dtype=torch.uint8, device=device)


def attention_forward(q, k, v, alpha, beta, mu, s=None, eps=1e-5, causal=True, ssmax=False,
                      o_dtype=None, ws=None, stream=None, prior=BAM_PRIOR_ALPHA):
    """q, k, v: bf16 [B,H,T,64] CUDA tensors -> (o, lse).  With
    prior=BAM_PRIOR_THETA, alpha, beta, mu are theta_alpha, theta_beta, theta_mu."""
    import torch
    B, H, T, D = q.shape
    o = torch.empty((B, H, T, D), dtype=o_dtype or torch.float32, device=q.device)
    lse = torch.empty((B, H, T), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(BAM_OP_FWD, B, H, T, q.device)
    prm = make_params(alpha, beta, mu, s, eps, causal, ssmax, prior)
    bam_attn_fwd(q, k, v, o, lse, prm, ws, stream)
    return o, lse


def attention_backward(q, k, v, o, lse, dO, alpha, beta, mu, s=None, eps=1e-5, causal=True,
                       ssmax=False, ws=None, stream=None, prior=BAM_PRIOR_ALPHA):
    """Returns dq, dk, dv (bf16) and dalpha, dbeta, dmu, ds (fp32 [H]); with
    prior=BAM_PRIOR_THETA the three prior gradients are the thetas'."""
    import torch
    B, H, T, D = q.shape
    dq, dk, dv = (torch.empty_like(q) for _ in range(3))
    g = [torch.empty(H, dtype=torch.float32, device=q.device) for _ in range(4)]
    if ws is None:
        ws = workspace(BAM_OP_BWD, B, H, T, q.device)
    prm = make_params(alpha, beta, mu, s, eps, causal, ssmax, prior)
    bam_attn_bwd(q, k, v, o, lse, dO, dq, dk, dv, g[0], g[1], g[2], g[3], prm, ws, stream)
    return dq, dk, dv, g[0], g[1], g[2], g[3]


def attention_decode(q, kc, vc, alpha, beta, mu, s=None, eps=1e-5, ssmax=False, o_dtype=None,
                     ws=None, stream=None, prior=BAM_PRIOR_ALPHA):
    """q: bf16 [B,H,64]; kc, vc: bf16 [B,H,Tkv,64] -> (o [B,H,64], lse [B,H])."""
    import torch
    B, H, Tkv, D = kc.shape
    o = torch.empty((B, H, D), dtype=o_dtype or torch.float32, device=q.device)
    lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(BAM_OP_DECODE, B, H, Tkv, q.device)
    prm = make_params(alpha, beta, mu, s, eps, True, ssmax, prior)
    bam_attn_decode(q, kc, vc, o, lse, prm, ws, stream)
    return o, lse


def attention_decode_varlen(q, kc, vc, cache_lens, alpha, beta, mu, s=None, eps=1e-5,
                            ssmax=False, o_dtype=None, ws=None, stream=None,
                            prior=BAM_PRIOR_ALPHA):
    """Ragged decode: q bf16 [B,H,64]; kc, vc bf16 [B,H,Tmax,64]; cache_lens
    int32 [B] -> (o [B,H,64], lse [B,H])."""
    import torch
    B, H, Tmax, D = kc.shape
    o = torch.empty((B, H, D), dtype=o_dtype or torch.float32, device=q.device)
    lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(BAM_OP_DECODE, B, H, Tmax, q.device)
    prm = make_params(alpha, beta, mu, s, eps, True, ssmax, prior)
    bam_attn_decode_varlen(q, kc, vc, cache_lens, o, lse, prm, ws, stream)
    return o, lse


def attention_decode_paged(q, k_pages, v_pages, block_table, cache_lens, alpha, beta, mu,
                           s=None, eps=1e-5, ssmax=False, o_dtype=None, ws=None, stream=None,
                           prior=BAM_PRIOR_ALPHA):
    """Paged decode: q bf16 [B,H,64]; k_pages, v_pages bf16 [num_pages,H,page,64];
    block_table int32 [B, max_blocks]; cache_lens int32 [B] -> (o, lse)."""
    import torch
    B, H, D = q.shape
    page, max_blocks = k_pages.shape[2], block_table.shape[1]
    o = torch.empty((B, H, D), dtype=o_dtype or torch.float32, device=q.device)
    lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(BAM_OP_DECODE, B, H, page * max_blocks, q.device)
    prm = make_params(alpha, beta, mu, s, eps, True, ssmax, prior)
    bam_attn_decode_paged(q, k_pages, v_pages, block_table, cache_lens, o, lse, prm, ws, stream)
    return o, lse


def _on(stream):
    """Makes `stream` (a torch stream, a raw handle or None) the current one: what
    is allocated and cleared for a call is then ready when its kernels run, and
    is not given to another stream before they are done."""
    import torch
    if stream is None:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream))
    return torch.cuda.stream(stream)


def kv_append_paged(k, v, k_pages, v_pages, block_table, cache_lens, new_lens=None, parents=None,
                    q=None, rope=None, ws=None, stream=None):
    """Append k, v [B, Hkv, N, 64] to the pages behind cache_lens committed
    keys, rotated by position when rope is given; returns the rotated q (None
    without q).  cache_lens is not changed.  Without ws, tokens that had no
    slot go unreported (bam_attn_check_status(ws))."""
    import torch
    q_out = None
    if q is not None:
        # rows behind new_lens are not written: no uninitialised memory in them
        make = torch.empty if new_lens is None else torch.zeros
        with _on(stream):
            q_out = make(q.shape, dtype=q.dtype, device=q.device)
    if ws is None:
        with _on(stream):
            ws = cache_workspace(k_pages.device)
    bam_kv_append_paged(k, v, k_pages, v_pages, block_table, cache_lens, new_lens, parents, q,
                        q_out, rope, ws, stream)
    return q_out


def attention_decode_tree_paged(q, k_pages, v_pages, block_table, cache_lens, alpha, beta, mu,
                                s=None, draft_lens=None, parents=None, eps=1e-5, ssmax=False,
                                o_dtype=None, ws=None, stream=None, prior=BAM_PRIOR_ALPHA):
    """Attention of drafted tokens q bf16 [B,H,N,64] over a paged cache that
    already holds their keys and values behind cache_lens committed ones ->
    (o [B,H,N,64], lse [B,H,N]); rows behind draft_lens are zero.  o_dtype:
    fp32 by default; bf16 is faster.  Without ws (tree_workspace(...)) each call
    clears one of its own, and what it would report is lost with it."""
    import torch
    B, H, N, D = q.shape
    make = torch.empty if draft_lens is None else torch.zeros
    with _on(stream):
        o = make((B, H, N, D), dtype=o_dtype or torch.float32, device=q.device)
        lse = make((B, H, N), dtype=torch.float32, device=q.device)
        if ws is None:
            ws = tree_workspace(B, H, k_pages.shape[1], N, k_pages.shape[2] * block_table.shape[1],
                                q.device)
    prm = make_params(alpha, beta, mu, s, eps, True, ssmax, prior)
    bam_attn_decode_tree_paged(q, k_pages, v_pages, block_table, cache_lens, draft_lens, parents,
                               o, lse, prm, ws, stream)
    return o, lse


def kv_keep_paged(k_pages, v_pages, block_table, cache_lens, accepted, parents, draft_lens=None,
                  new_lens=None, ws=None, stream=None):
    """Keep the accepted path of each draft; returns the new lengths (written
    to new_lens, which may be cache_lens, if given).  Without ws, paths that
    could not be kept go unreported."""
    import torch
    with _on(stream):
        if new_lens is None:
            new_lens = torch.empty_like(cache_lens)
        if ws is None:
            ws = cache_workspace(k_pages.device)
    bam_kv_keep_paged(k_pages, v_pages, block_table, cache_lens, draft_lens, parents, accepted,
                      new_lens, ws, stream)
    return new_lens
