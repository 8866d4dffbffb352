"""Binding of the shared-prefix attention (rules as in include/sdpa.h)."""
from __future__ import annotations

import functools
import math

import torch

from . import _native
from .api import _DTYPE_CODE, _run, _stream_ptr, check_workspace, new_tensor
from .rows import check_flat


@functools.lru_cache(maxsize=256)
def _bytes(b, h, h_kv, s_q, s_prefix, s_max, d_qk, d_v) -> int:
    return int(_native.lib().sdpa_fwd_prefix_workspace_size(b, h, h_kv, s_q, s_prefix, s_max, d_qk, d_v))


def sdpa_fwd_prefix_workspace_size(b, h, h_kv, s_q, s_prefix, s_max, d_qk, d_v) -> int:
    """Workspace bytes of sdpa_fwd_prefix."""
    return _bytes(int(b), int(h), int(h_kv), int(s_q), int(s_prefix), int(s_max), int(d_qk), int(d_v))


def sdpa_fwd_prefix(q, k_prefix, v_prefix, k, v, seqlens_k, *, scale=None, softcap=None, out=None,
                    lse=None, workspace=None, stream=None):
    """Attention of a batch's new tokens over a prefix that all its sequences
    share and each sequence's own keys behind it. Returns (o [b, h, s_q, d_v],
    lse fp32 [b, h, s_q]).

    q [b, h, s_q, d_qk]; k_prefix, v_prefix [h_kv, s_prefix, d], read once for
    the batch; k, v [b, h_kv, s_max, d], of which sequence i has its first
    seqlens_k[i] rows (int32 [b], the new tokens' rows among them; what lies
    behind them is not looked at). New token t sees the prefix and own keys
    j <= seqlens_k[i] - s_q + t. s_prefix and s_max may be 0. softcap as in
    sdpa_fwd. The workspace (sdpa_fwd_prefix_workspace_size bytes) is allocated
    when not given."""
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4 or k_prefix.dim() != 3 or v_prefix.dim() != 3:
        raise ValueError("q, k, v must have 4 dimensions, k_prefix and v_prefix 3")
    dt, dev = q.dtype, q.device
    if dt not in _DTYPE_CODE:
        raise ValueError("q, k, v must be bf16 or fp16")
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    b, h, s_q, d_qk = q.shape
    h_kv, s_max, d_v = k.shape[1], k.shape[2], v.shape[3]
    s_prefix = k_prefix.shape[1]
    q_p = check_flat("q", q, (b, h, s_q, d_qk), dt, dev)
    kp_p = check_flat("k_prefix", k_prefix, (h_kv, s_prefix, d_qk), dt, dev)
    vp_p = check_flat("v_prefix", v_prefix, (h_kv, s_prefix, d_v), dt, dev)
    k_p = check_flat("k", k, (b, h_kv, s_max, d_qk), dt, dev)
    v_p = check_flat("v", v, (b, h_kv, s_max, d_v), dt, dev)
    n_p = check_flat("seqlens_k", seqlens_k, (b,), torch.int32, dev)
    if out is None:
        out = new_tensor((b, h, s_q, d_v), dt, dev, stream)
        o_p = out.data_ptr()
    else:
        o_p = check_flat("out", out, (b, h, s_q, d_v), dt, dev)
    if lse is None:
        lse = new_tensor((b, h, s_q), torch.float32, dev, stream)
        l_p = lse.data_ptr()
    else:
        l_p = check_flat("lse", lse, (b, h, s_q), torch.float32, dev)
    if workspace is None:
        need = _bytes(b, h, h_kv, s_q, s_prefix, s_max, d_qk, d_v)
        workspace = new_tensor(max(need, 1), torch.uint8, dev, stream, scratch=True)
        ws = workspace.data_ptr(), need
    else:
        ws = check_workspace(workspace, dev)
    _run(q, "sdpa_fwd_prefix", b, h, h_kv, s_q, s_prefix, s_max, d_qk, d_v,
         1.0 / math.sqrt(d_qk) if scale is None else scale, softcap or 0.0, _DTYPE_CODE[dt], q_p, kp_p, vp_p,
         k_p, v_p, n_p, o_p, l_p, *ws, _stream_ptr(stream, q))
    return out, lse
