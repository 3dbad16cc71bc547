"""ctypes binding of libllama_attn.so: the same entry points, torch tensors in.

Argument marshalling only: tensors become device pointers, the current torch
CUDA stream becomes ``cuda_stream``, outputs and workspaces are allocated by
torch when the caller does not pass them, and a non-zero status raises.  Every
step of the computation runs in the library's kernels.  There is no CPU
fallback: without the built library, or on a tensor that is not on a CUDA
device, the call raises.

cos/sin arguments are LLaMA RoPE tables as ``rope_table`` returns them: the
second half of every row repeats the first (the frequencies concatenated with
themselves).  The kernels may read either copy; a table whose halves differ
is not supported (include/llama_attn.h states the same for the C ABI).

``stream``: the work goes to that stream, which the caller has let wait for
whatever the inputs still wait for, and the inputs stay alive until it is done.
What the call allocates is made as under ``torch.cuda.stream(stream)``: a block
of the current stream's pool may still be in use by work queued there.  The
caller waits for ``stream`` before the current stream reads the outputs.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os
from typing import Optional, Tuple

import torch

from . import build as _build

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libllama_attn.so")

LLAMA_DT_F32 = 0
LLAMA_DT_BF16 = 1
LLAMA_OK = 0
LLAMA_ERR_INVALID_ARG = 1
LLAMA_ERR_UNSUPPORTED = 2
LLAMA_ERR_CUDA = 3
LLAMA_ERR_DEVICE_TIMEOUT = 4

# Every symbol include/llama_attn.h declares.
EXPORTED = (
    "llama_rope_table",
    "llama_rope_table_ntk",
    "llama_rope_table_banded",
    "llama_rope_table_yarn",
    "llama_rope_apply",
    "llama_attn_qkv_rope",
    "llama_attn_out_proj",
    "llama_attn_prefill_workspace_bytes",
    "llama_attn_prefill",
    "llama_attn_prefill_window",
    "llama_attn_prefill_varlen",
    "llama_attn_prefill_packed",
    "llama_attn_decode_workspace_bytes",
    "llama_attn_decode",
    "llama_attn_decode_append",
    "llama_attn_decode_noalloc",
    "llama_attn_decode_prefix_workspace_bytes",
    "llama_attn_decode_prefix",
    "llama_attn_device_status",
    "llama_attn_selftest_wait_timeout",
    "llama_attn_selftest_launch_error",
    "llama_attn_status_string",
    "llama_attn_abi_version",
)

_lib = None


class LlamaAttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


def load() -> ctypes.CDLL:
    """Load the in-tree library.

    Raises if it has not been built, or if it was built from sources other
    than the ones now in the tree (a stale library would silently run old
    kernels).
    """
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it with `python -m llama_gqa_causal_b200.build`")
    if os.path.abspath(LIB_PATH) == os.path.abspath(_build.LIB) and \
            _build.built_hash() != _build.source_hash():
        raise RuntimeError(
            f"{LIB_PATH} was built from other sources than the ones in the tree: "
            "rebuild it with `python -m llama_gqa_causal_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, D, Z, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_double, ctypes.c_size_t, ctypes.c_float
    lib.llama_rope_table.argtypes = [P, I, I, I, D, D, P, P, P]
    lib.llama_rope_table.restype = I
    lib.llama_rope_table_ntk.argtypes = [P, I, I, I, D, D, P, P, P]
    lib.llama_rope_table_ntk.restype = I
    lib.llama_rope_table_banded.argtypes = [P, I, I, I, D, D, D, D, D, P, P, P]
    lib.llama_rope_table_banded.restype = I
    lib.llama_rope_table_yarn.argtypes = [P, I, I, I, D, D, D, D, D, D, P, P, P]
    lib.llama_rope_table_yarn.restype = I
    lib.llama_rope_apply.argtypes = [P, P, P, P, I, I, I, I, I, I, I, I, P, P, P, P, P, P, I, P]
    lib.llama_rope_apply.restype = I
    lib.llama_attn_qkv_rope.argtypes = [P, P, P, P, I, I, I, I, I, P, P, P, I, P]
    lib.llama_attn_qkv_rope.restype = I
    lib.llama_attn_out_proj.argtypes = [P, P, I, I, I, P, I, P]
    lib.llama_attn_out_proj.restype = I
    lib.llama_attn_prefill_workspace_bytes.argtypes = [I, I, I, I, I, I, I]
    lib.llama_attn_prefill_workspace_bytes.restype = Z
    lib.llama_attn_prefill.argtypes = [P, P, P, P, P, I, I, I, I, I, F, I, P, P, I, P, Z, P]
    lib.llama_attn_prefill.restype = I
    lib.llama_attn_prefill_window.argtypes = [P, P, P, P, P, I, I, I, I, I, F, I, P, I, P, Z, P]
    lib.llama_attn_prefill_window.restype = I
    lib.llama_attn_prefill_varlen.argtypes = [P, P, P, P, P, P, I, I, I, I, I, F, I, P, I, P, Z, P]
    lib.llama_attn_prefill_varlen.restype = I
    lib.llama_attn_prefill_packed.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, F, I, P, I, P, Z, P]
    lib.llama_attn_prefill_packed.restype = I
    lib.llama_attn_decode_workspace_bytes.argtypes = [I, I, I, I]
    lib.llama_attn_decode_workspace_bytes.restype = Z
    lib.llama_attn_decode.argtypes = [P, P, P, P, P, P, I, I, I, I, I, F, P, P, Z, I, P]
    lib.llama_attn_decode.restype = I
    lib.llama_attn_decode_append.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, F, P, P, Z, I, P]
    lib.llama_attn_decode_append.restype = I
    lib.llama_attn_decode_noalloc.argtypes = [P, P, P, P, P, P, I, I, I, I, I, F, P, I, P]
    lib.llama_attn_decode_noalloc.restype = I
    lib.llama_attn_decode_prefix_workspace_bytes.argtypes = [I, I, I, I, I]
    lib.llama_attn_decode_prefix_workspace_bytes.restype = Z
    lib.llama_attn_decode_prefix.argtypes = [P, P, P, P, P, I, P, P, P, P, P, I, I, I, I, I, F, P, P, Z,
                                             I, P]
    lib.llama_attn_decode_prefix.restype = I
    lib.llama_attn_device_status.argtypes = [P]
    lib.llama_attn_device_status.restype = I
    lib.llama_attn_selftest_wait_timeout.argtypes = [ctypes.c_uint, P]
    lib.llama_attn_selftest_wait_timeout.restype = I
    lib.llama_attn_selftest_launch_error.argtypes = [P]
    lib.llama_attn_selftest_launch_error.restype = I
    lib.llama_attn_status_string.argtypes = [I]
    lib.llama_attn_status_string.restype = ctypes.c_char_p
    lib.llama_attn_abi_version.argtypes = []
    lib.llama_attn_abi_version.restype = I
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().llama_attn_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != LLAMA_OK:
        raise LlamaAttnError(status, where)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("llama_attn: tensors must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("llama_attn: tensors must be contiguous")
    return t.data_ptr()


def _need(t: Optional[torch.Tensor], where: str, name: str, dtype: torch.dtype,
          device: torch.device, shape=None, numel: Optional[int] = None) -> None:
    """Reject a tensor whose dtype, device or size disagrees with the sizes the
    entry point is given (the C ABI sees only pointers: a short buffer would be
    read or written past its end)."""
    if t is None:
        return
    if t.dtype != dtype:
        raise ValueError(f"{where}: {name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{where}: {name} is on {t.device}, expected {device}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{where}: {name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{where}: {name} must hold {numel} elements, got {t.numel()}")


def _tables(cos, sin, where, device, rows, D) -> None:
    if (cos is None) != (sin is None):
        raise ValueError(f"{where}: pass both cos and sin, or neither")
    _need(cos, where, "cos", torch.float32, device, numel=rows * D)
    _need(sin, where, "sin", torch.float32, device, numel=rows * D)


def _stream(stream=None) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _scratch(like: torch.Tensor, nbytes: int, stream) -> torch.Tensor:
    """Scratch memory of the stream that will use it: once freed it may only be handed
    to work that follows there."""
    if stream is None:
        return like.new_empty(nbytes, dtype=torch.uint8)
    with torch.cuda.stream(stream):
        return like.new_empty(nbytes, dtype=torch.uint8)


def _output(like: torch.Tensor, shape, dtype: torch.dtype, stream) -> torch.Tensor:
    """An output, from the pool of the stream that writes it as scratch is, and noted as
    used by the caller's stream, which reads it.  (Of torch's ways to make a tensor these
    take the host least: 1.7 us with the sizes as arguments, 2.6 as a tuple.)"""
    if stream is None:
        return torch.empty(*shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        t = torch.empty(*shape, dtype=dtype, device=like.device)
    t.record_stream(torch.cuda.current_stream(like.device))
    return t


def _output_like(like: torch.Tensor, stream) -> torch.Tensor:
    """_output of like's shape and type, contiguous."""
    if stream is None:
        return torch.empty_like(like, memory_format=torch.contiguous_format)
    return _output(like, like.shape, like.dtype, stream)


def _positions(pos: torch.Tensor, stream) -> torch.Tensor:
    """pos as contiguous int64, converted on the stream whose kernel reads it."""
    if pos.dtype is torch.int64 and pos.is_contiguous():
        return pos
    with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
        return pos.to(torch.int64).contiguous()


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.bfloat16:
        return LLAMA_DT_BF16
    if dt == torch.float32:
        return LLAMA_DT_F32
    raise ValueError(f"llama_attn: unsupported dtype {dt}")


def rope_table(pos: torch.Tensor, head_dim: int, theta: float = 10000.0,
               factor: float = 1.0, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """cos, sin [*pos.shape, head_dim] fp32 from int64 positions (llama_rope_table)."""
    lib = load()
    pos = _positions(pos, stream)
    n = pos.numel()
    cos = _output(pos, (*pos.shape, head_dim), torch.float32, stream)
    sin = _output_like(cos, stream)
    bsz = pos.shape[0] if pos.dim() > 1 else 1
    seq = n // bsz
    _check(lib.llama_rope_table(_ptr(pos), bsz, seq, head_dim, float(theta), float(factor),
                                _ptr(cos), _ptr(sin), _stream(stream)), "llama_rope_table")
    return cos, sin


def rope_table_ntk(pos: torch.Tensor, head_dim: int, theta: float = 10000.0, alpha: float = 1.0,
                   stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """cos, sin of the NTK-aware scaled table (llama_rope_table_ntk)."""
    lib = load()
    pos = _positions(pos, stream)
    n = pos.numel()
    cos = _output(pos, (*pos.shape, head_dim), torch.float32, stream)
    sin = _output_like(cos, stream)
    bsz = pos.shape[0] if pos.dim() > 1 else 1
    seq = n // bsz
    _check(lib.llama_rope_table_ntk(_ptr(pos), bsz, seq, head_dim, float(theta), float(alpha),
                                    _ptr(cos), _ptr(sin), _stream(stream)), "llama_rope_table_ntk")
    return cos, sin


def _on(device: torch.device, where: str, fn, args, stream):
    """Call a library function on the tensors' own device: a launch goes to the
    current device, which need not be theirs.  (The raw-stream and current-device
    calls are what torch.cuda's own wrappers end in; the wrappers take longer than
    a decode step's kernel.)"""
    index = device.index
    s = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if index == torch._C._cuda_getDevice():
        status = fn(*args, s)
    else:
        with torch.cuda.device(device):
            status = fn(*args, s)
    if status != LLAMA_OK:
        raise LlamaAttnError(status, where)


def _table_scaled(where: str, pos: torch.Tensor, head_dim: int, args, stream):
    fn = getattr(_lib or load(), where)
    pos = _positions(pos, stream)
    p = _ptr(pos)
    shape, dev = pos.shape, pos.device
    cos = _output(pos, (*shape, head_dim), torch.float32, stream)
    sin = _output_like(cos, stream)
    bsz = shape[0] if len(shape) > 1 else 1
    _on(dev, where, fn, (p, bsz, pos.numel() // max(bsz, 1), head_dim, *args, cos.data_ptr(),
                         sin.data_ptr()), stream)
    return cos, sin


def rope_table_banded(pos: torch.Tensor, head_dim: int, theta: float = 10000.0, *, factor: float,
                      original_len: float, low_freq_factor: float = 1.0,
                      high_freq_factor: float = 4.0, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """cos, sin [*pos.shape, head_dim] fp32 of the table scaled by wavelength band
    (llama_rope_table_banded): frequencies that turn more than high_freq_factor times
    over original_len are kept, those below low_freq_factor divided by factor."""
    return _table_scaled("llama_rope_table_banded", pos, head_dim,
                         (theta, factor, low_freq_factor, high_freq_factor, original_len), stream)


def rope_table_yarn(pos: torch.Tensor, head_dim: int, theta: float = 10000.0, *, factor: float,
                    original_len: float, beta_fast: float = 32.0, beta_slow: float = 1.0,
                    attn_factor: Optional[float] = None,
                    stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """cos, sin of the YaRN table (llama_rope_table_yarn); attn_factor, which multiplies
    both, is 0.1 ln(factor) + 1 unless given."""
    if attn_factor is None:
        attn_factor = 0.1 * math.log(factor) + 1.0 if factor > 0.0 else 1.0
    return _table_scaled("llama_rope_table_yarn", pos, head_dim,
                         (theta, factor, beta_fast, beta_slow, original_len, attn_factor), stream)


_Strides = ctypes.c_longlong * 3
_PrefixStrides = ctypes.c_longlong * 2


def _rope_view(t: torch.Tensor, where: str, name: str, dtype, device, shape):
    """(pointer, strides of batch entry, token and head) of [b, s, heads, D] or [s, heads, D]."""
    if not t.is_cuda:
        raise ValueError("llama_attn: tensors must live on a CUDA device")
    if t.dtype != dtype or t.device != device:
        raise ValueError(f"{where}: {name} must be {dtype} on {device}, got {t.dtype} on {t.device}")
    if t.shape != shape:
        raise ValueError(f"{where}: {name} must be {list(shape)}, got {list(t.shape)}")
    st = t.stride()
    if st[-1] != 1:
        raise ValueError(f"{where}: the dimensions of a head of {name} must be adjacent")
    return t.data_ptr(), _Strides(st[0] if len(st) == 4 else 0, st[-3], st[-2])


def rope_apply(q: torch.Tensor, k: Optional[torch.Tensor], cos: torch.Tensor, sin: torch.Tensor, *,
               interleaved: bool = False, transpose: bool = False, out=None,
               stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """llama_rope_apply.  q [b, s, H, D] or [s, H, D], k likewise with its own heads (or
    None), rotated by the rows of cos, sin [.., R], R <= D.  Both may be strided views
    (parts of a fused projection), and so may out, a pair of tensors (q and k themselves:
    in place; k's: rows of a cache).  transpose: the gradient of the rotation."""
    w = "llama_rope_apply"
    fn = (_lib or load()).llama_rope_apply
    shape, dev, dt = q.shape, q.device, q.dtype
    if len(shape) == 4:
        b, s, H, D = shape
    elif len(shape) == 3:
        b, (s, H, D) = 1, shape
    else:
        raise ValueError(f"{w}: q must be [b, s, heads, head_dim] or [s, heads, head_dim]")
    if cos is None or sin is None:
        raise ValueError(f"{w}: pass both cos and sin")
    R = cos.shape[-1]
    if not (cos.dtype is sin.dtype is torch.float32 and cos.device == sin.device == dev
            and cos.shape == sin.shape and cos.numel() == b * s * R):
        _tables(cos, sin, w, dev, b * s, R)
        raise ValueError(f"{w}: cos and sin must have one shape")
    qp, qs = _rope_view(q, w, "q", dt, dev, shape)
    q_out, k_out = out if out is not None else (None, None)
    qos = kp = ks = kop = kos = None  # (strides of an output made here: dense)
    Hkv = 0
    if q_out is None:
        q_out = _output_like(q, stream)
        qop = q_out.data_ptr()
    else:
        qop, qos = _rope_view(q_out, w, "out", dt, dev, shape)
    if k is not None:
        k_shape = k.shape
        if k_shape[:-2] != shape[:-2] or k_shape[-1] != D:
            raise ValueError(f"{w}: k must have q's tokens and head_dim")
        Hkv = k_shape[-2]
        kp, ks = _rope_view(k, w, "k", dt, dev, k_shape)
        if k_out is None:
            k_out = _output_like(k, stream)
            kop = k_out.data_ptr()
        else:
            kop, kos = _rope_view(k_out, w, "out", dt, dev, k_shape)
    elif k_out is not None:
        raise ValueError(f"{w}: an output for k needs k")
    _on(dev, w, fn, (qp, kp, _ptr(cos), _ptr(sin), b, s, H, Hkv, D, R, 1 if interleaved else 0,
                     1 if transpose else 0, qs, ks, qop, kop, qos, kos, _dtype_code(dt)), stream)
    return q_out, k_out


def qkv_rope(x: torch.Tensor, w_qkv: torch.Tensor, n_heads: int, n_kv_heads: int, head_dim: int,
             cos: Optional[torch.Tensor] = None, sin: Optional[torch.Tensor] = None, *,
             out: Optional[Tuple[torch.Tensor, torch.Tensor, torch.Tensor]] = None,
             stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """llama_attn_qkv_rope.  x [T, hidden], w_qkv [(H+2Hkv)D, hidden] -> q [T,H,D], k, v [T,Hkv,D]."""
    lib = load()
    T, hidden = x.shape
    w = "llama_attn_qkv_rope"
    _need(w_qkv, w, "w_qkv", x.dtype, x.device, shape=((n_heads + 2 * n_kv_heads) * head_dim, hidden))
    _tables(cos, sin, w, x.device, T, head_dim)
    if out is None:
        q = _output(x, (T, n_heads, head_dim), x.dtype, stream)
        k = _output(x, (T, n_kv_heads, head_dim), x.dtype, stream)
        v = _output_like(k, stream)
    else:
        q, k, v = out
        _need(q, w, "q", x.dtype, x.device, numel=T * n_heads * head_dim)
        _need(k, w, "k", x.dtype, x.device, numel=T * n_kv_heads * head_dim)
        _need(v, w, "v", x.dtype, x.device, numel=T * n_kv_heads * head_dim)
    _check(lib.llama_attn_qkv_rope(_ptr(x), _ptr(w_qkv), _ptr(cos), _ptr(sin), T, hidden, n_heads,
                                   n_kv_heads, head_dim, _ptr(q), _ptr(k), _ptr(v),
                                   _dtype_code(x.dtype), _stream(stream)), "llama_attn_qkv_rope")
    return q, k, v


def out_proj(attn: torch.Tensor, w_o: torch.Tensor, *, out: Optional[torch.Tensor] = None,
             stream=None) -> torch.Tensor:
    """llama_attn_out_proj.  attn [T, in], w_o [out, in] -> y [T, out]."""
    lib = load()
    with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
        attn2 = attn.reshape(attn.shape[0], -1)  # (a copy, if it takes one, is read there)
    T, d_in = attn2.shape
    d_out = w_o.shape[0]
    _need(w_o, "llama_attn_out_proj", "w_o", attn.dtype, attn.device, shape=(d_out, d_in))
    if out is None:
        out = _output(attn, (T, d_out), attn.dtype, stream)
    _need(out, "llama_attn_out_proj", "out", attn.dtype, attn.device, numel=T * d_out)
    _check(lib.llama_attn_out_proj(_ptr(attn2), _ptr(w_o), T, d_in, d_out, _ptr(out),
                                   _dtype_code(attn.dtype), _stream(stream)), "llama_attn_out_proj")
    return out


def prefill_workspace_bytes(bsz, n_heads, n_kv_heads, seq, head_dim, dtype, has_rope) -> int:
    return int(load().llama_attn_prefill_workspace_bytes(
        bsz, n_heads, n_kv_heads, seq, head_dim, _dtype_code(dtype), int(bool(has_rope))))


def decode_workspace_bytes(bsz, n_heads, max_cache_len, head_dim) -> int:
    return int(load().llama_attn_decode_workspace_bytes(bsz, n_heads, max_cache_len, head_dim))


def prefill(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
            cos: Optional[torch.Tensor] = None, sin: Optional[torch.Tensor] = None, *,
            causal: bool = True, scale: Optional[float] = None,
            mask: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
            workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """llama_attn_prefill.  q [b,S,H,D], k/v [b,S,Hkv,D] -> out [b, S, H*D]."""
    lib = load()
    b, S, H, D = q.shape
    Hkv = k.shape[2]
    _need(k, "llama_attn_prefill", "k", q.dtype, q.device, shape=(b, S, Hkv, D))
    _need(v, "llama_attn_prefill", "v", q.dtype, q.device, shape=(b, S, Hkv, D))
    _tables(cos, sin, "llama_attn_prefill", q.device, b * S, D)
    _need(out, "llama_attn_prefill", "out", q.dtype, q.device, numel=b * S * H * D)
    _need(mask, "llama_attn_prefill", "mask", torch.float32, q.device, numel=b * S * S)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = _output(q, (b, S, H * D), q.dtype, stream)
    need = prefill_workspace_bytes(b, H, Hkv, S, D, q.dtype, cos is not None)
    if workspace is None and need > 0:
        workspace = _scratch(q, need, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.llama_attn_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(cos), _ptr(sin), b, H, Hkv, S,
                                  D, float(scale), int(bool(causal)), _ptr(out), _ptr(mask),
                                  _dtype_code(q.dtype), _ptr(workspace), ws_bytes,
                                  _stream(stream)), "llama_attn_prefill")
    return out


def prefill_window(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                   cos: Optional[torch.Tensor] = None, sin: Optional[torch.Tensor] = None, *,
                   window: int, scale: Optional[float] = None,
                   out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """llama_attn_prefill_window.  Causal; query i sees keys i - window < j <= i."""
    lib = load()
    b, S, H, D = q.shape
    Hkv = k.shape[2]
    _need(k, "llama_attn_prefill_window", "k", q.dtype, q.device, shape=(b, S, Hkv, D))
    _need(v, "llama_attn_prefill_window", "v", q.dtype, q.device, shape=(b, S, Hkv, D))
    _tables(cos, sin, "llama_attn_prefill_window", q.device, b * S, D)
    _need(out, "llama_attn_prefill_window", "out", q.dtype, q.device, numel=b * S * H * D)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = _output(q, (b, S, H * D), q.dtype, stream)
    need = prefill_workspace_bytes(b, H, Hkv, S, D, q.dtype, cos is not None)
    if workspace is None and need > 0:
        workspace = _scratch(q, need, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.llama_attn_prefill_window(_ptr(q), _ptr(k), _ptr(v), _ptr(cos), _ptr(sin), b, H,
                                         Hkv, S, D, float(scale), int(window), _ptr(out),
                                         _dtype_code(q.dtype), _ptr(workspace), ws_bytes,
                                         _stream(stream)), "llama_attn_prefill_window")
    return out


def prefill_varlen(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, seq_lens: torch.Tensor,
                   cos: Optional[torch.Tensor] = None, sin: Optional[torch.Tensor] = None, *,
                   causal: bool = True, scale: Optional[float] = None,
                   out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """llama_attn_prefill_varlen.  Right-padded batch; seq_lens int32 [b] valid rows."""
    lib = load()
    b, S, H, D = q.shape
    Hkv = k.shape[2]
    _need(k, "llama_attn_prefill_varlen", "k", q.dtype, q.device, shape=(b, S, Hkv, D))
    _need(v, "llama_attn_prefill_varlen", "v", q.dtype, q.device, shape=(b, S, Hkv, D))
    _tables(cos, sin, "llama_attn_prefill_varlen", q.device, b * S, D)
    _need(out, "llama_attn_prefill_varlen", "out", q.dtype, q.device, numel=b * S * H * D)
    _need(seq_lens, "llama_attn_prefill_varlen", "seq_lens", torch.int32, q.device, numel=b)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if seq_lens.dtype != torch.int32:
        raise ValueError("llama_attn_prefill_varlen: seq_lens must be int32")
    if out is None:
        out = _output(q, (b, S, H * D), q.dtype, stream)
    need = prefill_workspace_bytes(b, H, Hkv, S, D, q.dtype, cos is not None)
    if workspace is None and need > 0:
        workspace = _scratch(q, need, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.llama_attn_prefill_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(cos), _ptr(sin),
                                         _ptr(seq_lens), b, H, Hkv, S, D, float(scale),
                                         int(bool(causal)), _ptr(out), _dtype_code(q.dtype),
                                         _ptr(workspace), ws_bytes, _stream(stream)),
           "llama_attn_prefill_varlen")
    return out


def prefill_packed(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                   max_seqlen: int, cos: Optional[torch.Tensor] = None,
                   sin: Optional[torch.Tensor] = None, *, causal: bool = True,
                   scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """llama_attn_prefill_packed.  q [T,H,D], k/v [T,Hkv,D], cu_seqlens int32 [n+1] -> out [T, H*D]."""
    lib = load()
    T, H, D = q.shape
    Hkv = k.shape[1]
    n = cu_seqlens.numel() - 1
    w = "llama_attn_prefill_packed"
    _need(k, w, "k", q.dtype, q.device, shape=(T, Hkv, D))
    _need(v, w, "v", q.dtype, q.device, shape=(T, Hkv, D))
    _tables(cos, sin, w, q.device, T, D)
    _need(out, w, "out", q.dtype, q.device, numel=T * H * D)
    _need(cu_seqlens, w, "cu_seqlens", torch.int32, q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if cu_seqlens.dtype != torch.int32:
        raise ValueError("llama_attn_prefill_packed: cu_seqlens must be int32")
    if out is None:
        out = _output(q, (T, H * D), q.dtype, stream)
    need = prefill_workspace_bytes(1, H, Hkv, T, D, q.dtype, cos is not None)
    if workspace is None and need > 0:
        workspace = _scratch(q, need, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.llama_attn_prefill_packed(_ptr(q), _ptr(k), _ptr(v), _ptr(cos), _ptr(sin),
                                         _ptr(cu_seqlens), n, T, int(max_seqlen), H, Hkv, D,
                                         float(scale), int(bool(causal)), _ptr(out),
                                         _dtype_code(q.dtype), _ptr(workspace), ws_bytes,
                                         _stream(stream)), "llama_attn_prefill_packed")
    return out


def decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
           cache_lens: torch.Tensor, cos: Optional[torch.Tensor] = None,
           sin: Optional[torch.Tensor] = None, *, scale: Optional[float] = None,
           out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
           stream=None) -> torch.Tensor:
    """llama_attn_decode.  q [b,H,D], caches [b,Hkv,L,D], cache_lens int32 [b] -> out [b, H*D]."""
    lib = load()
    b, H, D = q.shape
    Hkv, L = k_cache.shape[1], k_cache.shape[2]
    _need(k_cache, "llama_attn_decode", "k_cache", q.dtype, q.device, shape=(b, Hkv, L, D))
    _need(v_cache, "llama_attn_decode", "v_cache", q.dtype, q.device, shape=(b, Hkv, L, D))
    _need(cache_lens, "llama_attn_decode", "cache_lens", torch.int32, q.device, numel=b)
    _tables(cos, sin, "llama_attn_decode", q.device, b, D)
    _need(out, "llama_attn_decode", "out", q.dtype, q.device, numel=b * H * D)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = _output(q, (b, H * D), q.dtype, stream)
    if workspace is None:
        workspace = _scratch(q, decode_workspace_bytes(b, H, L, D), stream)
    ws_bytes = workspace.numel() * workspace.element_size()
    if cache_lens.dtype != torch.int32:
        raise ValueError("llama_attn_decode: cache_lens must be int32")
    _check(lib.llama_attn_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(cache_lens),
                                 _ptr(cos), _ptr(sin), b, H, Hkv, L, D, float(scale), _ptr(out),
                                 _ptr(workspace), ws_bytes, _dtype_code(q.dtype),
                                 _stream(stream)), "llama_attn_decode")
    return out


def decode_append(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                  k_cache: torch.Tensor, v_cache: torch.Tensor, cache_lens: torch.Tensor,
                  cos: Optional[torch.Tensor] = None, sin: Optional[torch.Tensor] = None, *,
                  scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """llama_attn_decode_append.  q [b,H,D], k_new/v_new [b,Hkv,D] (k_new not rotated),
    caches [b,Hkv,L,D] (written at row min(cache_lens[b], L-1)), cache_lens int32 [b]
    (read only) -> out [b, H*D]."""
    lib = load()
    b, H, D = q.shape
    Hkv, L = k_cache.shape[1], k_cache.shape[2]
    _need(k_cache, "llama_attn_decode_append", "k_cache", q.dtype, q.device, shape=(b, Hkv, L, D))
    _need(v_cache, "llama_attn_decode_append", "v_cache", q.dtype, q.device, shape=(b, Hkv, L, D))
    _need(cache_lens, "llama_attn_decode_append", "cache_lens", torch.int32, q.device, numel=b)
    _tables(cos, sin, "llama_attn_decode_append", q.device, b, D)
    _need(out, "llama_attn_decode_append", "out", q.dtype, q.device, numel=b * H * D)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = _output(q, (b, H * D), q.dtype, stream)
    if workspace is None:
        workspace = _scratch(q, decode_workspace_bytes(b, H, L, D), stream)
    ws_bytes = workspace.numel() * workspace.element_size()
    if cache_lens.dtype != torch.int32:
        raise ValueError("llama_attn_decode_append: cache_lens must be int32")
    for name, t in (("k_new", k_new), ("v_new", v_new)):
        if tuple(t.shape) != (b, Hkv, D) or not t.is_contiguous():
            raise ValueError(f"llama_attn_decode_append: {name} must be contiguous [b, Hkv, D]")
    _check(lib.llama_attn_decode_append(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache),
                                        _ptr(v_cache), _ptr(cache_lens), _ptr(cos), _ptr(sin), b, H,
                                        Hkv, L, D, float(scale), _ptr(out), _ptr(workspace),
                                        ws_bytes, _dtype_code(q.dtype), _stream(stream)),
           "llama_attn_decode_append")
    return out


def decode_noalloc(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   cache_lens: torch.Tensor, cos: Optional[torch.Tensor] = None,
                   sin: Optional[torch.Tensor] = None, *, scale: Optional[float] = None,
                   out: torch.Tensor, stream=None) -> torch.Tensor:
    """llama_attn_decode_noalloc: decode with the library's static scratch.

    For callers that must not allocate device memory: ``out`` is required
    (shape [b, H*D], same dtype as q) and nothing is allocated here either.
    """
    lib = load()
    b, H, D = q.shape
    Hkv, L = k_cache.shape[1], k_cache.shape[2]
    _need(k_cache, "llama_attn_decode_noalloc", "k_cache", q.dtype, q.device, shape=(b, Hkv, L, D))
    _need(v_cache, "llama_attn_decode_noalloc", "v_cache", q.dtype, q.device, shape=(b, Hkv, L, D))
    _need(cache_lens, "llama_attn_decode_noalloc", "cache_lens", torch.int32, q.device, numel=b)
    _tables(cos, sin, "llama_attn_decode_noalloc", q.device, b, D)
    _need(out, "llama_attn_decode_noalloc", "out", q.dtype, q.device, numel=b * H * D)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if cache_lens.dtype != torch.int32:
        raise ValueError("llama_attn_decode_noalloc: cache_lens must be int32")
    _check(lib.llama_attn_decode_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(cache_lens),
                                         _ptr(cos), _ptr(sin), b, H, Hkv, L, D, float(scale),
                                         _ptr(out), _dtype_code(q.dtype), _stream(stream)),
           "llama_attn_decode_noalloc")
    return out


@functools.lru_cache(maxsize=256)
def decode_prefix_workspace_bytes(bsz, n_heads, n_kv_heads, prefix_len, head_dim) -> int:
    return int(load().llama_attn_decode_prefix_workspace_bytes(bsz, n_heads, n_kv_heads, prefix_len,
                                                               head_dim))


def _prefix_view(t: torch.Tensor, name: str, P: int, D: int):
    """(pointer, strides of K/V head and row) of a prefix tensor [Hkv, P, D]."""
    if not t.is_cuda:
        raise ValueError("llama_attn: tensors must live on a CUDA device")
    head, row, one = t.stride()
    if one != 1:
        raise ValueError("llama_attn_decode_prefix: the dimensions of a row of "
                         f"{name} must be adjacent")
    # the stride of an extent of one is never used; torch leaves it arbitrary
    row = row if P > 1 else D
    return t.data_ptr(), _PrefixStrides(head if t.shape[0] > 1 else P * row, row)


def decode_prefix(q: torch.Tensor, k_prefix: torch.Tensor, v_prefix: torch.Tensor,
                  k_cache: torch.Tensor, v_cache: torch.Tensor, cache_lens: torch.Tensor, *,
                  k_new: Optional[torch.Tensor] = None, v_new: Optional[torch.Tensor] = None,
                  scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """llama_attn_decode_prefix.  q [b,H,D] (rotated), the shared prefix [Hkv,P,D] (keys
    rotated; a strided view is taken as it is), caches [b,Hkv,L,D] of the rows after it,
    cache_lens int32 [b] -> out [b, H*D].  With k_new, v_new [b,Hkv,D] (k_new rotated)
    the step's own row is appended to the caches first."""
    w = "llama_attn_decode_prefix"
    fn = (_lib or load()).llama_attn_decode_prefix
    b, H, D = q.shape
    _, Hkv, L, _ = k_cache.shape
    P = k_prefix.shape[1]
    dev, dt = q.device, q.dtype
    cache, prefix, new = (b, Hkv, L, D), (Hkv, P, D), (b, Hkv, D)
    # (one test of what fits; what does not is named by the checks that raise)
    if not (k_cache.shape == v_cache.shape == cache and k_prefix.shape == v_prefix.shape == prefix
            and k_cache.dtype is v_cache.dtype is k_prefix.dtype is v_prefix.dtype is dt
            and k_cache.device == v_cache.device == k_prefix.device == v_prefix.device == dev):
        for t, name, shape in ((k_cache, "k_cache", cache), (v_cache, "v_cache", cache),
                               (k_prefix, "k_prefix", prefix), (v_prefix, "v_prefix", prefix)):
            _need(t, w, name, dt, dev, shape)
    _need(k_new, w, "k_new", dt, dev, new)
    _need(v_new, w, "v_new", dt, dev, new)
    _need(out, w, "out", dt, dev, None, b * H * D)
    if cache_lens.dtype is not torch.int32 or cache_lens.device != dev or cache_lens.numel() != b:
        _need(cache_lens, w, "cache_lens", torch.int32, dev, None, b)
    if not (q.is_cuda and q.is_contiguous() and k_cache.is_contiguous() and v_cache.is_contiguous()
            and cache_lens.is_contiguous()):
        for t in (q, k_cache, v_cache, cache_lens):
            _ptr(t)
    kp, ks = _prefix_view(k_prefix, "k_prefix", P, D)
    vp, vs = _prefix_view(v_prefix, "v_prefix", P, D)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = _output(q, (b, H * D), dt, stream)
        op = out.data_ptr()
    else:
        op = _ptr(out)
    if workspace is None:
        need = decode_prefix_workspace_bytes(b, H, Hkv, P, D)
        workspace = _scratch(q, need, stream)
        ws, ws_bytes = workspace.data_ptr(), need
    else:
        ws, ws_bytes = _ptr(workspace), workspace.numel() * workspace.element_size()
    _on(dev, w, fn, (q.data_ptr(), _ptr(k_new), _ptr(v_new), kp, vp, P, ks, vs, k_cache.data_ptr(),
                     v_cache.data_ptr(), cache_lens.data_ptr(), b, H, Hkv, L, D, scale, op, ws,
                     ws_bytes, _dtype_code(dt)), stream)
    return out


def device_status(stream=None) -> int:
    """llama_attn_device_status: sync the stream, read and clear the device status word."""
    return int(load().llama_attn_device_status(_stream(stream)))


def selftest_wait_timeout(limit_us: int, stream=None) -> int:
    """llama_attn_selftest_wait_timeout: a bounded device wait that runs out (status code)."""
    return int(load().llama_attn_selftest_wait_timeout(int(limit_us), _stream(stream)))


def selftest_launch_error(stream=None) -> int:
    """llama_attn_selftest_launch_error: a launch the runtime refuses (status code)."""
    return int(load().llama_attn_selftest_launch_error(_stream(stream)))
