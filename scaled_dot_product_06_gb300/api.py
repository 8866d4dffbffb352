"""PyTorch-facing binding of the C ABI (same names as include/sdpa.h).

PyTorch provides device memory and the stream; every step of the attention
computation runs in libsdpa.so's kernels. The functions here only check
tensor properties, allocate outputs with torch and pass raw pointers.

Every call runs on ``stream``, by default the current one. What it allocates
(outputs and workspace that are not given) is then that stream's, as within
``torch.cuda.stream(stream)``; ordering it behind the work that makes the inputs,
and the readers of the outputs behind it, is the caller's part, and so is
keeping the inputs until it has run.
"""
from __future__ import annotations

import ctypes
import functools
import math

import torch

from . import _native

_DTYPE_CODE = {torch.bfloat16: _native.SDPA_BF16, torch.float16: _native.SDPA_FP16}


# The current stream's handle without building a torch.cuda.Stream object
# (which costs a few microseconds a call); the public route where the private
# accessor is missing.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_ptr(stream, t: torch.Tensor) -> int:
    if stream is not None:
        if getattr(stream, "device", t.device) != t.device:
            raise ValueError("stream must be one of the tensors' device")
        return int(stream.cuda_stream)
    if _raw_stream is not None:
        return int(_raw_stream(t.get_device()))
    return int(torch.cuda.current_stream(t.device).cuda_stream)


def _run(t: torch.Tensor, name: str, *args) -> None:
    """Calls the C entry point `name` with t's device current."""
    if t.get_device() == torch.cuda.current_device():
        st = getattr(_native.lib(), name)(*args)
    else:
        with torch.cuda.device(t.device):
            st = getattr(_native.lib(), name)(*args)
    if st:
        _native.check(st, name)


def new_tensor(shape, dtype, device, stream, scratch=False) -> torch.Tensor:
    """Memory for a call on ``stream`` (None: the current one).

    The allocator hands memory out in the order of the stream it is asked on:
    memory of the current stream's could still be in use there when ``stream``
    writes it, and a dropped workspace would be given to the next call while
    ``stream`` works in it. So it is asked on ``stream``. Outputs are noted as used
    by the caller's stream too: dropped, they wait for its work."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream.cuda_stream), device=device)
    caller = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if not scratch and stream != caller:
        t.record_stream(caller)
    return t


def _check_io(name: str, t: torch.Tensor, shape, dtype, device=None) -> None:
    """A contiguous CUDA tensor of this shape and type (and device)."""
    if (t.is_cuda if device is None else t.device == device) and t.shape == shape and t.dtype == dtype \
            and t.is_contiguous():
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on the device of q")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    raise ValueError(f"{name} must be contiguous (BHSD)")


def _check_device(device, **tensors) -> None:
    """The smaller operands, whose form is checked elsewhere, are on q's device."""
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} must be on the device of q")


def check_workspace(t: torch.Tensor, device):
    """(pointer, bytes) of a workspace that is one block of memory of this device."""
    if t.device != device or not t.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the device of q")
    return t.data_ptr(), t.numel() * t.element_size()


def _grad(name, t, shape, dtype, device, stream, written=True) -> torch.Tensor:
    """A gradient: the given tensor, checked where it is written, or a new one."""
    if t is None:
        return new_tensor(shape, dtype, device, stream)
    if written:
        _check_io(name, t, shape, dtype, device)
    return t


def _ptr(t):
    # an int converts to void* through the functions' argtypes
    return None if t is None else t.data_ptr()


def _window(is_causal, window, bottom_right, alibi_slopes, n_batch, h, dropout_mask=None,
            force=False, words=0):
    """(left, right, bottom_right, slopes pointer, slope stride, keep-bits
    pointer) for the *_ex entry points, or None for the plain causal / unmasked
    calls (unless force). alibi_slopes: fp32 CUDA [h] (every batch entry) or
    [n_batch, h]; dropout_mask: the int32 words of sdpa_dropout_mask (or of a
    forward's dropout_mask_out) for the same problem, `words` of them."""
    if (window is None and not bottom_right and alibi_slopes is None and dropout_mask is None
            and not force):
        return None
    if dropout_mask is not None and (not dropout_mask.is_cuda or dropout_mask.dtype != torch.int32
                                     or not dropout_mask.is_contiguous() or dropout_mask.numel() < words):
        raise ValueError(f"dropout_mask must be the contiguous int32 CUDA words of sdpa_dropout_mask, "
                         f"{words} of them")
    left, right = window if window is not None else (-1, 0 if is_causal else -1)
    stride = 0
    if alibi_slopes is not None:
        a = alibi_slopes
        if not a.is_cuda or a.dtype != torch.float32 or not a.is_contiguous():
            raise ValueError("alibi_slopes must be a contiguous fp32 CUDA tensor")
        if tuple(a.shape) == (h,):
            stride = 0
        elif tuple(a.shape) == (n_batch, h):
            stride = h
        else:
            raise ValueError(f"alibi_slopes has shape {tuple(a.shape)}, expected ({h},) or "
                             f"({n_batch}, {h})")
    return int(left), int(right), int(bool(bottom_right)), _ptr(alibi_slopes), stride, _ptr(dropout_mask)


def _capped(softcap, is_causal, window, bottom_right, bias, alibi_slopes, n_batch, h, dropout_mask, words):
    """(softcap, left, right, bottom_right, keep-bits pointer) for the *_capped
    entry points, or None for uncapped scores (softcap None or 0)."""
    if softcap is None or softcap == 0:
        return None
    if bias is not None or alibi_slopes is not None:
        raise ValueError("softcap takes no bias and no alibi_slopes")
    left, right, br, _, _, keep = _window(is_causal, window, bottom_right, None, n_batch, h,
                                          dropout_mask, force=True, words=words)
    return float(softcap), left, right, br, keep


def _words(dropout_p, b, h, s_q, s_kv) -> int:
    """Words of a problem's keep bits (0 without dropout, when none are read or written)."""
    return (b * h * s_q * s_kv + 31) // 32 if dropout_p > 0 else 0


def _mask_out(t, words):
    """A forward's keep-bit record buffer: contiguous int32 CUDA words."""
    if t is None:
        return None
    if not t.is_cuda or t.dtype != torch.int32 or not t.is_contiguous() or t.numel() < words:
        raise ValueError(f"dropout_mask_out must be a contiguous int32 CUDA tensor of at least "
                         f"{words} words")
    return _ptr(t)


def sdpa_fwd(q, k, v, *, scale=None, is_causal=False, dropout_p=0.0, seed=0, offset=0,
             bias=None, out=None, lse=None, stream=None, window=None, bottom_right=False,
             alibi_slopes=None, dropout_mask=None, dropout_mask_out=None, softcap=None):
    """Forward pass. Returns (o [b,h,s_q,d_v], lse fp32 [b,h,s_q]).

    k and v may have fewer heads than q (grouped-query attention): h_kv =
    k.shape[1] must divide h, and query head i reads K/V head i // (h // h_kv).
    window=(left, right) keeps key j visible to query i iff
    i + off - left <= j <= i + off + right (a negative size unbounded), with
    off = s_kv - s_q when bottom_right, else 0; is_causal is window (-1, 0).
    alibi_slopes (fp32 CUDA [h] or [b, h]) adds -slope * |j - i - off_a| to the
    scaled scores, off_a = 0 under a top-left window, else s_kv - s_q.
    dropout_mask_out (int32 CUDA, ceil(b*h*s_q*s_kv/32) words): the forward
    records the dropout keep bits it draws there, for sdpa_bwd's
    dropout_mask (needs s_kv % 32 == 0).
    softcap (in (0, 4096]; None or 0: none) replaces each scaled score s by
    softcap * tanh(s / softcap) before the mask; not with a bias or ALiBi."""
    b, h, s_q, d_qk = q.shape
    h_kv, s_kv, d_v = k.shape[1], k.shape[2], v.shape[3]
    dt, dev = q.dtype, q.device
    if dt not in _DTYPE_CODE:
        raise ValueError("q, k, v must be bf16 or fp16")
    _check_io("q", q, (b, h, s_q, d_qk), dt)
    _check_io("k", k, (b, h_kv, s_kv, d_qk), dt, dev)
    _check_io("v", v, (b, h_kv, s_kv, d_v), dt, dev)
    if bias is not None:
        _check_io("bias", bias, (1, h, s_q, s_kv), torch.float32, dev)
    scale = 1.0 / math.sqrt(d_qk) if scale is None else float(scale)
    if out is None:
        out = new_tensor((b, h, s_q, d_v), dt, dev, stream)
    else:
        _check_io("out", out, (b, h, s_q, d_v), dt, dev)
    if lse is None:
        lse = new_tensor((b, h, s_q), torch.float32, dev, stream)
    else:
        _check_io("lse", lse, (b, h, s_q), torch.float32, dev)
    if alibi_slopes is not None or dropout_p > 0:
        _check_device(dev, alibi_slopes=alibi_slopes, dropout_mask=dropout_mask,
                      dropout_mask_out=dropout_mask_out)
    words = _words(dropout_p, b, h, s_q, s_kv)
    cap = _capped(softcap, is_causal, window, bottom_right, bias, alibi_slopes, b, h, dropout_mask,
                  words)
    if cap is not None:
        rec = _mask_out(dropout_mask_out, (b * h * s_q * s_kv + 31) // 32)
        _run(q, "sdpa_fwd_capped", b, h, h_kv, s_q, s_kv, d_qk, d_v, scale, *cap, rec,
             float(dropout_p), int(seed), int(offset), _DTYPE_CODE[dt], _ptr(q), _ptr(k), _ptr(v),
             _ptr(out), _ptr(lse), _stream_ptr(stream, q))
        return out, lse
    w = _window(is_causal, window, bottom_right, alibi_slopes, b, h, dropout_mask,
                force=dropout_mask_out is not None, words=words)
    if w is None:
        _run(q, "sdpa_fwd_gqa", b, h, h_kv, s_q, s_kv, d_qk, d_v, scale, int(bool(is_causal)),
             float(dropout_p), int(seed), int(offset), _DTYPE_CODE[dt], _ptr(q), _ptr(k), _ptr(v),
             _ptr(bias), _ptr(out), _ptr(lse), _stream_ptr(stream, q))
    else:
        rec = _mask_out(dropout_mask_out, (b * h * s_q * s_kv + 31) // 32)
        _run(q, "sdpa_fwd_ex", b, h, h_kv, s_q, s_kv, d_qk, d_v, scale, *w, rec, float(dropout_p),
             int(seed), int(offset), _DTYPE_CODE[dt], _ptr(q), _ptr(k), _ptr(v), _ptr(bias),
             _ptr(out), _ptr(lse), _stream_ptr(stream, q))
    return out, lse


def sdpa_bwd_workspace_size(b, h, s_q, s_kv, d_qk, d_v, h_kv=None, deterministic=False) -> int:
    """Backward workspace bytes: the row statistics, plus the fp32 dQ
    accumulator of the default backward at d_qk <= 128 (not with
    deterministic=True); with h_kv (grouped K/V heads) the room for splitting
    large groups over several CTAs per key tile is included."""
    return _workspace_size(int(b), int(h), int(h if h_kv is None else h_kv), int(s_q), int(s_kv),
                           int(d_qk), int(d_v), int(bool(deterministic)))


@functools.lru_cache(maxsize=256)
def _workspace_size(b, h, h_kv, s_q, s_kv, d_qk, d_v, deterministic) -> int:
    return int(_native.lib().sdpa_bwd_workspace_size_ex(b, h, h_kv, s_q, s_kv, d_qk, d_v, deterministic))


def sdpa_bwd(q, k, v, o, dout, lse, *, scale=None, is_causal=False, dropout_p=0.0, seed=0,
             offset=0, bias=None, workspace=None, dq=None, dk=None, dv=None, dbias=None,
             stream=None, window=None, bottom_right=False, alibi_slopes=None,
             dropout_mask=None, deterministic=False, softcap=None):
    """Backward pass. Returns (dq, dk, dv, dbias or None); dk and dv have k's
    and v's shapes (with grouped K/V heads, sums over each group).
    deterministic=True runs the deterministic backward (dQ from the
    query-stationary kernel, bitwise reproducible) instead of accumulating dQ
    with fp32 reductions."""
    return sdpa_bwd_phases(_native.SDPA_BWD_ALL, q, k, v, o, dout, lse, scale=scale,
                           is_causal=is_causal, dropout_p=dropout_p, seed=seed, offset=offset,
                           bias=bias, workspace=workspace, dq=dq, dk=dk, dv=dv, dbias=dbias,
                           stream=stream, window=window, bottom_right=bottom_right,
                           alibi_slopes=alibi_slopes, dropout_mask=dropout_mask,
                           deterministic=deterministic, softcap=softcap)


def sdpa_bwd_phases(phases, q, k, v, o, dout, lse, *, scale=None, is_causal=False, dropout_p=0.0,
                    seed=0, offset=0, bias=None, workspace=None, dq=None, dk=None, dv=None,
                    dbias=None, stream=None, window=None, bottom_right=False, alibi_slopes=None,
                    dropout_mask=None, deterministic=False, softcap=None):
    """The backward phases selected by ``phases`` (SDPA_BWD_* bit mask; the
    SDPA_BWD_DETERMINISTIC bit, or deterministic=True, selects the
    deterministic backward)."""
    deterministic = bool(deterministic) or bool(int(phases) & _native.SDPA_BWD_DETERMINISTIC)
    phases = int(phases) | (_native.SDPA_BWD_DETERMINISTIC if deterministic else 0)
    b, h, s_q, d_qk = q.shape
    h_kv, s_kv, d_v = k.shape[1], k.shape[2], v.shape[3]
    dt, dev = q.dtype, q.device
    if dt not in _DTYPE_CODE:
        raise ValueError("q, k, v must be bf16 or fp16")
    for name, t, shp in (("q", q, (b, h, s_q, d_qk)), ("k", k, (b, h_kv, s_kv, d_qk)),
                         ("v", v, (b, h_kv, s_kv, d_v)), ("o", o, (b, h, s_q, d_v)),
                         ("dout", dout, (b, h, s_q, d_v))):
        _check_io(name, t, shp, dt, dev if t is not q else None)
    _check_io("lse", lse, (b, h, s_q), torch.float32, dev)
    if bias is not None:
        _check_io("bias", bias, (1, h, s_q, s_kv), torch.float32, dev)
    scale = 1.0 / math.sqrt(d_qk) if scale is None else float(scale)
    # (a phase may be given stand-ins for what it does not write)
    kv = phases & _native.SDPA_BWD_DKDV
    dq = _grad("dq", dq, q.shape, dt, dev, stream, phases & (_native.SDPA_BWD_DKDV | _native.SDPA_BWD_DQ))
    dk = _grad("dk", dk, k.shape, dt, dev, stream, kv)
    dv = _grad("dv", dv, v.shape, dt, dev, stream, kv)
    if bias is not None or dbias is not None:
        dbias = _grad("dbias", dbias, (1, h, s_q, s_kv), torch.float32, dev, stream)
    need = sdpa_bwd_workspace_size(b, h, s_q, s_kv, d_qk, d_v, h_kv, deterministic)
    if workspace is None:
        workspace = new_tensor(max(need, 1), torch.uint8, dev, stream, scratch=True)
        ws = workspace.data_ptr(), need
    else:
        ws = check_workspace(workspace, dev)
    if alibi_slopes is not None or dropout_p > 0:
        _check_device(dev, alibi_slopes=alibi_slopes, dropout_mask=dropout_mask)
    words = _words(dropout_p, b, h, s_q, s_kv)
    cap = _capped(softcap, is_causal, window, bottom_right, bias, alibi_slopes, b, h, dropout_mask,
                  words)
    if cap is not None:
        _run(q, "sdpa_bwd_phases_capped", int(phases), b, h, h_kv, s_q, s_kv, d_qk, d_v, scale,
             *cap, float(dropout_p), int(seed), int(offset), _DTYPE_CODE[dt], _ptr(q), _ptr(k),
             _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv), *ws,
             _stream_ptr(stream, q))
        return dq, dk, dv, None
    w = _window(is_causal, window, bottom_right, alibi_slopes, b, h, dropout_mask, words=words)
    if w is None:
        _run(q, "sdpa_bwd_phases_gqa", int(phases), b, h, h_kv, s_q, s_kv, d_qk, d_v, scale,
             int(bool(is_causal)), float(dropout_p), int(seed), int(offset), _DTYPE_CODE[dt],
             _ptr(q), _ptr(k), _ptr(v), _ptr(bias), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq),
             _ptr(dk), _ptr(dv), _ptr(dbias), *ws, _stream_ptr(stream, q))
    else:
        _run(q, "sdpa_bwd_phases_ex", int(phases), b, h, h_kv, s_q, s_kv, d_qk, d_v, scale, *w,
             float(dropout_p), int(seed), int(offset), _DTYPE_CODE[dt], _ptr(q), _ptr(k), _ptr(v),
             _ptr(bias), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dbias),
             *ws, _stream_ptr(stream, q))
    return dq, dk, dv, dbias


def _check_seqstart(name: str, t: torch.Tensor) -> int:
    if not t.is_cuda or t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 1-D int32 CUDA tensor")
    if t.numel() < 1:
        raise ValueError(f"{name} needs b + 1 entries")
    return t.numel() - 1


def sdpa_fwd_varlen(q, k, v, seqstart_q, seqstart_k, max_seqlen_q, max_seqlen_k, *, scale=None,
                    is_causal=False, dropout_p=0.0, seed=0, offset=0, out=None, lse=None,
                    stream=None, window=None, bottom_right=False, alibi_slopes=None,
                    dropout_mask=None, dropout_mask_out=None, softcap=None):
    """Forward pass over packed variable-length sequences. q [h, total_q, d_qk],
    k [h_kv, total_k, d_qk], v [h_kv, total_k, d_v]; seqstart_q / seqstart_k
    int32 CUDA tensors of b + 1 row offsets (sequence i owns query rows
    seqstart_q[i] .. seqstart_q[i+1] - 1 and the matching key rows).
    Returns (o [h, total_q, d_v], lse fp32 [h, total_q])."""
    h, total_q, d_qk = q.shape
    h_kv, total_k, d_v = k.shape[0], k.shape[1], v.shape[2]
    dt, dev = q.dtype, q.device
    if dt not in _DTYPE_CODE:
        raise ValueError("q, k, v must be bf16 or fp16")
    b = _check_seqstart("seqstart_q", seqstart_q)
    if _check_seqstart("seqstart_k", seqstart_k) != b:
        raise ValueError("seqstart_q and seqstart_k must have the same length")
    _check_io("q", q, (h, total_q, d_qk), dt)
    _check_io("k", k, (h_kv, total_k, d_qk), dt, dev)
    _check_io("v", v, (h_kv, total_k, d_v), dt, dev)
    scale = 1.0 / math.sqrt(d_qk) if scale is None else float(scale)
    if out is None:
        out = new_tensor((h, total_q, d_v), dt, dev, stream)
    else:
        _check_io("out", out, (h, total_q, d_v), dt, dev)
    if lse is None:
        lse = new_tensor((h, total_q), torch.float32, dev, stream)
    else:
        _check_io("lse", lse, (h, total_q), torch.float32, dev)
    _check_device(dev, seqstart_q=seqstart_q, seqstart_k=seqstart_k, alibi_slopes=alibi_slopes,
                  dropout_mask=dropout_mask, dropout_mask_out=dropout_mask_out)
    words = _words(dropout_p, b, h, int(max_seqlen_q), int(max_seqlen_k))
    cap = _capped(softcap, is_causal, window, bottom_right, None, alibi_slopes, b, h, dropout_mask,
                  words)
    if cap is not None:
        rec = _mask_out(dropout_mask_out, (b * h * int(max_seqlen_q) * int(max_seqlen_k) + 31) // 32)
        _run(q, "sdpa_fwd_varlen_capped", b, h, h_kv, total_q, total_k, int(max_seqlen_q),
             int(max_seqlen_k), d_qk, d_v, scale, *cap, rec, float(dropout_p), int(seed),
             int(offset), _DTYPE_CODE[dt], _ptr(seqstart_q), _ptr(seqstart_k), _ptr(q), _ptr(k),
             _ptr(v), _ptr(out), _ptr(lse), _stream_ptr(stream, q))
        return out, lse
    w = _window(is_causal, window, bottom_right, alibi_slopes, b, h, dropout_mask,
                force=dropout_mask_out is not None, words=words)
    if w is None:
        _run(q, "sdpa_fwd_varlen", b, h, h_kv, total_q, total_k, int(max_seqlen_q),
             int(max_seqlen_k), d_qk, d_v, scale, int(bool(is_causal)), float(dropout_p), int(seed),
             int(offset), _DTYPE_CODE[dt], _ptr(seqstart_q), _ptr(seqstart_k), _ptr(q), _ptr(k),
             _ptr(v), _ptr(out), _ptr(lse), _stream_ptr(stream, q))
    else:
        rec = _mask_out(dropout_mask_out, (b * h * int(max_seqlen_q) * int(max_seqlen_k) + 31) // 32)
        _run(q, "sdpa_fwd_varlen_ex", b, h, h_kv, total_q, total_k, int(max_seqlen_q),
             int(max_seqlen_k), d_qk, d_v, scale, *w, rec, float(dropout_p), int(seed), int(offset),
             _DTYPE_CODE[dt], _ptr(seqstart_q), _ptr(seqstart_k), _ptr(q), _ptr(k), _ptr(v),
             _ptr(out), _ptr(lse), _stream_ptr(stream, q))
    return out, lse


def sdpa_bwd_varlen_workspace_size(b, h, total_q, d_qk=None, deterministic=False) -> int:
    """Workspace bytes of the packed backward. Without d_qk: the row
    statistics alone, which run the deterministic backward; with d_qk: the
    bytes of the backward ``deterministic`` selects (the default one at
    d_qk <= 128 adds its fp32 dQ accumulator)."""
    if d_qk is None:
        return int(_native.lib().sdpa_bwd_varlen_workspace_size(b, h, total_q))
    return int(_native.lib().sdpa_bwd_varlen_workspace_size_ex(b, h, total_q, int(d_qk),
                                                               int(bool(deterministic))))


def sdpa_bwd_varlen(q, k, v, o, dout, lse, seqstart_q, seqstart_k, max_seqlen_q, max_seqlen_k, *,
                    scale=None, is_causal=False, dropout_p=0.0, seed=0, offset=0, workspace=None,
                    dq=None, dk=None, dv=None, stream=None, window=None, bottom_right=False,
                    alibi_slopes=None, dropout_mask=None, deterministic=False, softcap=None):
    """Backward pass over packed sequences (layouts as sdpa_fwd_varlen).
    Returns (dq, dk, dv) shaped like q, k, v. deterministic=True runs the
    deterministic backward, as sdpa_bwd."""
    return sdpa_bwd_phases_varlen(_native.SDPA_BWD_ALL, q, k, v, o, dout, lse, seqstart_q,
                                  seqstart_k, max_seqlen_q, max_seqlen_k, scale=scale,
                                  is_causal=is_causal, dropout_p=dropout_p, seed=seed,
                                  offset=offset, workspace=workspace, dq=dq, dk=dk, dv=dv,
                                  stream=stream, window=window, bottom_right=bottom_right,
                                  alibi_slopes=alibi_slopes, dropout_mask=dropout_mask,
                                  deterministic=deterministic, softcap=softcap)


def sdpa_bwd_phases_varlen(phases, q, k, v, o, dout, lse, seqstart_q, seqstart_k, max_seqlen_q,
                           max_seqlen_k, *, scale=None, is_causal=False, dropout_p=0.0, seed=0,
                           offset=0, workspace=None, dq=None, dk=None, dv=None, stream=None,
                           window=None, bottom_right=False, alibi_slopes=None,
                           dropout_mask=None, deterministic=False, softcap=None):
    """The packed-sequence backward phases selected by ``phases`` (the
    SDPA_BWD_DETERMINISTIC bit, or deterministic=True, selects the
    deterministic backward). A caller-given workspace smaller than the
    default backward's size runs the deterministic one."""
    deterministic = bool(deterministic) or bool(int(phases) & _native.SDPA_BWD_DETERMINISTIC)
    phases = int(phases) | (_native.SDPA_BWD_DETERMINISTIC if deterministic else 0)
    h, total_q, d_qk = q.shape
    h_kv, total_k, d_v = k.shape[0], k.shape[1], v.shape[2]
    dt, dev = q.dtype, q.device
    if dt not in _DTYPE_CODE:
        raise ValueError("q, k, v must be bf16 or fp16")
    b = _check_seqstart("seqstart_q", seqstart_q)
    if _check_seqstart("seqstart_k", seqstart_k) != b:
        raise ValueError("seqstart_q and seqstart_k must have the same length")
    for name, t, shp in (("q", q, (h, total_q, d_qk)), ("k", k, (h_kv, total_k, d_qk)),
                         ("v", v, (h_kv, total_k, d_v)), ("o", o, (h, total_q, d_v)),
                         ("dout", dout, (h, total_q, d_v))):
        _check_io(name, t, shp, dt, dev if t is not q else None)
    _check_io("lse", lse, (h, total_q), torch.float32, dev)
    scale = 1.0 / math.sqrt(d_qk) if scale is None else float(scale)
    # (a phase may be given stand-ins for what it does not write)
    kv = phases & _native.SDPA_BWD_DKDV
    dq = _grad("dq", dq, q.shape, dt, dev, stream, phases & (_native.SDPA_BWD_DKDV | _native.SDPA_BWD_DQ))
    dk = _grad("dk", dk, k.shape, dt, dev, stream, kv)
    dv = _grad("dv", dv, v.shape, dt, dev, stream, kv)
    need = sdpa_bwd_varlen_workspace_size(b, h, total_q, d_qk, deterministic)
    if workspace is None:
        workspace = new_tensor(max(need, 1), torch.uint8, dev, stream, scratch=True)
        ws = workspace.data_ptr(), need
    else:
        ws = check_workspace(workspace, dev)
    _check_device(dev, seqstart_q=seqstart_q, seqstart_k=seqstart_k, alibi_slopes=alibi_slopes,
                  dropout_mask=dropout_mask)
    words = _words(dropout_p, b, h, int(max_seqlen_q), int(max_seqlen_k))
    cap = _capped(softcap, is_causal, window, bottom_right, None, alibi_slopes, b, h, dropout_mask,
                  words)
    if cap is not None:
        _run(q, "sdpa_bwd_phases_varlen_capped", int(phases), b, h, h_kv, total_q, total_k,
             int(max_seqlen_q), int(max_seqlen_k), d_qk, d_v, scale, *cap, float(dropout_p),
             int(seed), int(offset), _DTYPE_CODE[dt], _ptr(seqstart_q), _ptr(seqstart_k), _ptr(q),
             _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv), *ws,
             _stream_ptr(stream, q))
        return dq, dk, dv
    w = _window(is_causal, window, bottom_right, alibi_slopes, b, h, dropout_mask, words=words)
    if w is None:
        _run(q, "sdpa_bwd_phases_varlen", int(phases), b, h, h_kv, total_q, total_k,
             int(max_seqlen_q), int(max_seqlen_k), d_qk, d_v, scale, int(bool(is_causal)),
             float(dropout_p), int(seed), int(offset), _DTYPE_CODE[dt], _ptr(seqstart_q),
             _ptr(seqstart_k), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq),
             _ptr(dk), _ptr(dv), *ws, _stream_ptr(stream, q))
    else:
        _run(q, "sdpa_bwd_phases_varlen_ex", int(phases), b, h, h_kv, total_q, total_k,
             int(max_seqlen_q), int(max_seqlen_k), d_qk, d_v, scale, *w, float(dropout_p),
             int(seed), int(offset), _DTYPE_CODE[dt], _ptr(seqstart_q), _ptr(seqstart_k), _ptr(q),
             _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv), *ws,
             _stream_ptr(stream, q))
    return dq, dk, dv


def sdpa_dropout_mask(b, h, s_q, s_kv, dropout_p, seed, offset, device="cuda", stream=None,
                      out=None):
    """Packed keep bits as an int32 tensor of ceil(b*h*s_q*s_kv/32) words (into
    ``out`` when given). Passed back as ``dropout_mask``, the attention calls
    read these bits instead of drawing them."""
    words = (b * h * s_q * s_kv + 31) // 32
    bits = new_tensor(max(words, 1), torch.int32, device, stream) if out is None else out
    if out is not None and (out.dtype != torch.int32 or out.numel() < words or not out.is_cuda
                            or not out.is_contiguous()):
        raise ValueError(f"out must be a contiguous int32 CUDA tensor of at least {words} words")
    _run(bits, "sdpa_dropout_mask", b, h, s_q, s_kv, float(dropout_p), int(seed), int(offset), _ptr(bits),
         _stream_ptr(stream, bits))
    return bits[:words]


def sdpa_device_error(clear: bool = True) -> int:
    """The device error word (synchronises); 0 when every kernel completed."""
    w = ctypes.c_uint32(0)
    st = _native.lib().sdpa_device_error(ctypes.byref(w), int(bool(clear)))
    if st not in (_native.SDPA_OK, _native.SDPA_ERR_DEVICE_TIMEOUT):
        _native.check(st, "sdpa_device_error")
    return int(w.value)


def sdpa_debug_fault(fault: int = 0, wait_limit_ns: int = 0) -> None:
    """Test hook of the C ABI (see include/sdpa.h): fault 1 makes later forward
    launches time out in a bounded wait; sdpa_debug_fault() restores normal operation."""
    _native.check(_native.lib().sdpa_debug_fault(int(fault), int(wait_limit_ns)), "sdpa_debug_fault")


def sdpa_status_string(status: int) -> str:
    return _native.status_string(status)
