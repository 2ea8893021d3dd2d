"""Thin torch-facing binding over the C ABI (include/qws.h).

Argument marshalling only: every function passes device pointers, sizes and
the current CUDA stream to libqws.so; all arithmetic runs in its kernels.
Outputs are allocated with torch when ``out`` is not given (PyTorch is the
allocator, the library allocates nothing).  With ``stream`` a call runs on
that stream in place of the current one: its fresh outputs and workspaces
belong to it, and the caller makes it wait for the inputs, and the current
stream for the outputs.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import _lib
from ._lib import (OP_DECODE_CHAIN, OP_FFN, OP_KV_ATTENTION, OP_MATVEC, OP_PREFILL, Q4_0,
                   Q4_K, Q6_K, Q8_0,
                   QwsError, check, lib)

__all__ = [
    "Q4_0", "Q4_K", "Q6_K", "Q8_0", "QwsError", "q4k_matvec", "q6k_matvec", "q4_0_matvec",
    "matvec", "quantize_q8_0", "q8_matvec", "q8_qkv_proj", "q4k_prefill_matmul",
    "rope_at_pos", "kv_append", "kv_attention", "rms_norm_q8", "residual_rms_norm_q8",
    "q4k_qkv_proj", "q4k_ffn_gate_up_geglu", "q4k_ffn_gate_up_geglu_down", "rms_norm",
    "residual_add", "decode_chain", "decode_kv", "decode_kv_workspace_bytes", "workspace_bytes",
    "embed_tokens", "qk_norm_rope", "prompt_attention", "prefix_attention",
    "paged_kv_head_bytes", "paged_kv_append", "paged_kv_gather", "paged_kv_attention",
    "sample_tokens", "device_error", "Layer", "Dims",
    "stream_handle",
]


def stream_handle(stream: torch.cuda.Stream | None = None) -> int:
    if stream is not None:
        return stream.cuda_stream
    # the handle itself: building a Stream object around it takes 3 us
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _dev(t: torch.Tensor, name: str, dtype: torch.dtype | None = None) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _empty(shape, dtype: torch.dtype, device, stream, returned: bool = True) -> torch.Tensor:
    """A fresh tensor for a call's kernels: an output, or (not returned) a workspace.

    It comes from the pool of the stream that the kernels run on.  A block of another
    stream's pool may have belonged to a tensor that the other stream's queued work still
    reads or writes, and nothing orders these kernels behind that work.  An output is the
    current stream's too, so that it may be used there (behind a wait) and freed."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if returned and t.is_cuda:
        t.record_stream(torch.cuda.current_stream())
    return t


def _out(out, shape, like: torch.Tensor, stream) -> torch.Tensor:
    if out is None:
        return _empty(shape, torch.float32, like.device, stream)
    return out


def workspace_bytes(op: int, rows: int = 0, hidden: int = 0, inter: int = 0, batch: int = 1,
                    split_k: int = 0) -> int:
    return int(lib().qws_workspace_bytes(op, rows, hidden, inter, batch, split_k))


def _mv(name: str, W, x, rows: int, hidden: int, batch: int, out, stream):
    y = _out(out, (batch, rows) if batch > 1 else (rows,), x, stream)
    fn = getattr(lib(), name)
    check(fn(_dev(W, "W", torch.uint8), _dev(x, "x", torch.float32),
             _dev(y, "y", torch.float32), rows, hidden, batch, stream_handle(stream)))
    return y


def q4k_matvec(W, x, rows: int, hidden: int, batch: int = 1, out=None, stream=None):
    """y = dequant_Q4_K(W) @ x; x [batch, hidden] (or [hidden]), y [batch, rows]."""
    return _mv("qws_q4k_matvec", W, x, rows, hidden, batch, out, stream)


def q6k_matvec(W, x, rows: int, hidden: int, batch: int = 1, out=None, stream=None):
    return _mv("qws_q6k_matvec", W, x, rows, hidden, batch, out, stream)


def matvec(fmt: int, W, x, rows: int, hidden: int, batch: int = 1, split_k: int = 1,
           workspace=None, out=None, stream=None):
    y = _out(out, (batch, rows) if batch > 1 else (rows,), x, stream)
    ws_ptr, ws_bytes = (0, 0) if workspace is None else (_dev(workspace, "workspace"),
                                                          workspace.numel() * workspace.element_size())
    check(lib().qws_matvec(fmt, _dev(W, "W", torch.uint8), _dev(x, "x", torch.float32),
                           _dev(y, "y", torch.float32), rows, hidden, batch, split_k,
                           ws_ptr or None, ws_bytes, stream_handle(stream)))
    return y


def q4_0_matvec(W, x, rows: int, hidden: int, batch: int = 1, split_k: int = 1, workspace=None,
                out=None, stream=None):
    y = _out(out, (batch, rows) if batch > 1 else (rows,), x, stream)
    ws_ptr, ws_bytes = (0, 0) if workspace is None else (_dev(workspace, "workspace"),
                                                          workspace.numel() * workspace.element_size())
    check(lib().qws_q4_0_matvec(_dev(W, "W", torch.uint8), _dev(x, "x", torch.float32),
                                _dev(y, "y", torch.float32), rows, hidden, batch, split_k,
                                ws_ptr or None, ws_bytes, stream_handle(stream)))
    return y


def q4k_qkv_proj(Wq, Wk, Wv, x, hidden: int, q_dim: int, kv_dim: int, out=None, stream=None):
    if out is None:
        q = _empty(q_dim, torch.float32, x.device, stream)
        k = _empty(kv_dim, torch.float32, x.device, stream)
        v = _empty(kv_dim, torch.float32, x.device, stream)
    else:
        q, k, v = out
    check(lib().qws_q4k_qkv_proj(_dev(Wq, "Wq", torch.uint8), _dev(Wk, "Wk", torch.uint8),
                                 _dev(Wv, "Wv", torch.uint8), _dev(x, "x", torch.float32),
                                 _dev(q, "q", torch.float32), _dev(k, "k", torch.float32),
                                 _dev(v, "v", torch.float32), hidden, q_dim, kv_dim,
                                 stream_handle(stream)))
    return q, k, v


def quantize_q8_0(x, n: int, batch: int = 1, out=None, stream=None):
    """x [batch, n] (or [n]) f32 -> Q8_0 blocks, uint8 [batch, n / 32 * 34] (or flat)."""
    nbytes = n // 32 * 34
    if out is None:
        out = _empty((batch, nbytes) if batch > 1 else (nbytes,), torch.uint8, x.device, stream)
    check(lib().qws_quantize_q8_0(_dev(x, "x", torch.float32), _dev(out, "xq", torch.uint8), n,
                                  batch, stream_handle(stream)))
    return out


def _xq_out(out, n: int, batch: int, like, stream):
    if out is not None:
        return out
    nbytes = n // 32 * 34
    return _empty((batch, nbytes) if batch > 1 else (nbytes,), torch.uint8, like.device, stream)


def rms_norm_q8(x, w, eps: float, n: int, batch: int = 1, out=None, stream=None):
    """Q8_0 blocks of rms_norm(x, w) ([batch, n] or [n] f32 -> uint8 [.., n / 32 * 34])."""
    xq = _xq_out(out, n, batch, x, stream)
    check(lib().qws_rms_norm_q8(_dev(x, "x", torch.float32), _dev(w, "w", torch.float32),
                                _dev(xq, "xq", torch.uint8), n, eps, batch,
                                stream_handle(stream)))
    return xq


def residual_rms_norm_q8(h, y, w, eps: float, n: int, batch: int = 1, out=None, stream=None):
    """h += y (in place), then the Q8_0 blocks of rms_norm(h, w)."""
    xq = _xq_out(out, n, batch, h, stream)
    check(lib().qws_residual_rms_norm_q8(_dev(h, "h", torch.float32), _dev(y, "y", torch.float32),
                                         _dev(w, "w", torch.float32), _dev(xq, "xq", torch.uint8),
                                         n, eps, batch, stream_handle(stream)))
    return xq


def q8_matvec(wfmt: int, W, xq, rows: int, hidden: int, batch: int = 1, out=None, stream=None):
    """y = W @ xq for Q4_0 / Q8_0 weights and Q8_0 activations xq."""
    y = _out(out, (batch, rows) if batch > 1 else (rows,), xq, stream)
    check(lib().qws_q8_matvec(wfmt, _dev(W, "W", torch.uint8), _dev(xq, "xq", torch.uint8),
                              _dev(y, "y", torch.float32), rows, hidden, batch,
                              stream_handle(stream)))
    return y


def q8_qkv_proj(wfmt: int, Wq, Wk, Wv, xq, hidden: int, q_dim: int, kv_dim: int, out=None,
                stream=None):
    if out is None:
        q = _empty(q_dim, torch.float32, xq.device, stream)
        k = _empty(kv_dim, torch.float32, xq.device, stream)
        v = _empty(kv_dim, torch.float32, xq.device, stream)
    else:
        q, k, v = out
    check(lib().qws_q8_qkv_proj(wfmt, _dev(Wq, "Wq", torch.uint8), _dev(Wk, "Wk", torch.uint8),
                                _dev(Wv, "Wv", torch.uint8), _dev(xq, "xq", torch.uint8),
                                _dev(q, "q", torch.float32), _dev(k, "k", torch.float32),
                                _dev(v, "v", torch.float32), hidden, q_dim, kv_dim,
                                stream_handle(stream)))
    return q, k, v


def q4k_prefill_matmul(W, X, rows: int, hidden: int, n_tokens: int, workspace=None, out=None,
                       stream=None):
    """Y [n_tokens, rows] = X [n_tokens, hidden] @ dequant_Q4_K(W)^T on the tensor cores
    (f16 operands, f32 accumulation)."""
    Y = _out(out, (n_tokens, rows), X, stream)
    need = workspace_bytes(OP_PREFILL, 0, hidden, 0, n_tokens, 0)
    if workspace is None:
        workspace = _empty(max(need, 16), torch.uint8, X.device, stream, returned=False)
    check(lib().qws_q4k_prefill_matmul(
        _dev(W, "W", torch.uint8), _dev(X, "X", torch.float32), _dev(Y, "Y", torch.float32),
        rows, hidden, n_tokens, _dev(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), stream_handle(stream)))
    return Y


def rope_at_pos(x, n_heads: int, head_dim: int, rot_dim: int, pos: int, base: float,
                stream=None):
    """Rotates x [n_heads, head_dim] in place at position pos; returns x."""
    check(lib().qws_rope_at_pos(_dev(x, "x", torch.float32), n_heads, head_dim, rot_dim, pos,
                                float(base), stream_handle(stream)))
    return x


def kv_append(k_cache, v_cache, k, v, n_kv_heads: int, head_dim: int, max_seq: int, pos: int,
              stream=None):
    check(lib().qws_kv_append(_dev(k_cache, "k_cache", torch.float32),
                              _dev(v_cache, "v_cache", torch.float32),
                              _dev(k, "k", torch.float32), _dev(v, "v", torch.float32),
                              n_kv_heads, head_dim, max_seq, pos, stream_handle(stream)))


def kv_attention(q, k_cache, v_cache, n_q_heads: int, n_kv_heads: int, head_dim: int,
                 max_seq: int, n_ctx: int, scale: float, softcap: float = 0.0, workspace=None,
                 out=None, stream=None):
    """One query token q [n_q_heads, head_dim] over cache positions 0 .. n_ctx-1."""
    y = _out(out, (n_q_heads, head_dim), q, stream)
    need = workspace_bytes(OP_KV_ATTENTION, n_ctx, head_dim, n_q_heads, n_kv_heads)
    if workspace is None:
        workspace = _empty(max(need, 16), torch.uint8, q.device, stream, returned=False)
    check(lib().qws_kv_attention(
        _dev(q, "q", torch.float32), _dev(k_cache, "k_cache", torch.float32),
        _dev(v_cache, "v_cache", torch.float32), _dev(y, "out", torch.float32), n_q_heads,
        n_kv_heads, head_dim, max_seq, n_ctx, float(scale), float(softcap),
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        stream_handle(stream)))
    return y


# ------------------------------------------------------------ prompts and batches
def _here(t: torch.Tensor, name: str, dev: int) -> None:
    """Refuses a tensor of another device than the one the call launches on."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")


def _heads(t: torch.Tensor, name: str, dev: int, heads: int | None = None,
           head_dim: int | None = None):
    """qws_heads of a [tokens, heads, head_dim] f32 view; its last dimension is dense."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        _here(t, name, dev)
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be torch.float32, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or (heads is not None and (shape[1] != heads or shape[2] != head_dim)):
        raise ValueError(f"{name} must be [tokens, {heads or 'heads'}, {head_dim or 'head_dim'}], "
                         f"got {tuple(shape)}")
    a, b, c = t.stride()
    if c != 1:
        raise ValueError(f"{name}: the values of a head must be contiguous")
    return _lib.QwsHeads(t.data_ptr(), a if shape[0] > 1 else 0, b if shape[1] > 1 else 0)


def _vec(t, name: str, dev: int, dtype: torch.dtype, n: int) -> int:
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        _here(t, name, dev)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be {n} contiguous values, got {tuple(t.shape)}")
    return t.data_ptr()


def _cache(t, name: str, dev: int) -> int:
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        _here(t, name, dev)
    return _dev(t, name, torch.float32)


def _host_ints(v, name: str):
    """A ctypes int64 array of a list, tuple or CPU tensor of whole numbers."""
    if isinstance(v, torch.Tensor):
        if v.is_cuda or v.dim() != 1 or v.is_floating_point():
            raise TypeError(f"{name} must be a list or a 1-d CPU integer tensor: the lengths are "
                            "read on the host")
        v = v.tolist()
    return (C.c_int64 * len(v))(*v)


def _workspace(need: int, workspace, dev: int, stream):
    """(tensor, bytes) of the caller's workspace, or of a fresh one."""
    if workspace is None:
        if need == 0:
            return None, 0
        workspace = _empty(need, torch.uint8, dev, stream, returned=False)
    else:
        _here(workspace, "workspace", dev)
        _dev(workspace, "workspace")
    return workspace, workspace.numel() * workspace.element_size()


def embed_tokens(fmt: int, W, tokens, vocab: int, hidden: int, scale: float = 1.0, out=None,
                 stream=None):
    """out [n, hidden] = scale * rows `tokens` (int64, [n]) of the quantised table W (uint8,
    vocab rows).  A token outside the table gives zeros and sets device_error() bit 512."""
    dev = torch.cuda.current_device()
    _here(W, "W", dev)
    n = tokens.numel()
    block, size = {Q4_0: (32, 18), Q8_0: (32, 34), Q4_K: (256, 144), Q6_K: (256, 210)}.get(
        fmt, (1, 0))
    if W.numel() < vocab * (hidden // block) * size:
        raise ValueError(f"W has {W.numel()} bytes, {vocab} rows of {hidden} need "
                         f"{vocab * (hidden // block) * size}")
    out = _empty((n, hidden), torch.float32, dev, stream) if out is None else out
    check(lib().qws_embed_tokens(fmt, _dev(W, "W", torch.uint8),
                                 _vec(tokens, "tokens", dev, torch.int64, n),
                                 _vec(out, "out", dev, torch.float32, n * hidden), vocab, hidden,
                                 n, scale, stream_handle(stream)) if n else 0)
    return out


def qk_norm_rope(q, k, positions, rot_dim: int, base: float, w_q=None, w_k=None,
                 eps: float = 1e-6, q_out=None, k_out=None, stream=None):
    """RMS norm of every head of q [T, n_q, hd] and k [T, n_kv, hd] (w_q, w_k [hd]; None: no
    norm) and its rotation at positions [T] (int64).  Strided views welcome; q_out / k_out may
    be q / k themselves, or for k a view of a cache.  Returns (q_out, k_out)."""
    dev = torch.cuda.current_device()
    qh, kh = _heads(q, "q", dev), _heads(k, "k", dev)
    n, n_q, hd = q.shape
    n_kv = k.shape[1]
    if k.shape[0] != n or k.shape[2] != hd:
        raise ValueError(f"q {tuple(q.shape)} and k {tuple(k.shape)} do not match")
    q_out = _empty((n, n_q, hd), torch.float32, dev, stream) if q_out is None else q_out
    k_out = _empty((n, n_kv, hd), torch.float32, dev, stream) if k_out is None else k_out
    qo, ko = _heads(q_out, "q_out", dev, n_q, hd), _heads(k_out, "k_out", dev, n_kv, hd)
    if q_out.shape[0] != n or k_out.shape[0] != n:
        raise ValueError(f"q_out and k_out must have {n} tokens")
    if n:
        check(lib().qws_qk_norm_rope(
            C.byref(qh), C.byref(kh), C.byref(qo), C.byref(ko),
            None if w_q is None else _vec(w_q, "w_q", dev, torch.float32, hd),
            None if w_k is None else _vec(w_k, "w_k", dev, torch.float32, hd),
            _vec(positions, "positions", dev, torch.int64, n), n, n_q, n_kv, hd, rot_dim, base,
            eps, stream_handle(stream)))
    return q_out, k_out


def prompt_attention(q, k, v, cu_seqlens, scale: float, softcap: float = 0.0, cu_seqlens_k=None,
                     workspace=None, out=None, stream=None):
    """Causal attention of packed sequences: q [T, n_q, hd], k and v [Tk, n_kv, hd], sequence s
    at rows cu_seqlens[s] .. cu_seqlens[s + 1] - 1 (host integers) of q, and of k and v, or at
    cu_seqlens_k there; its last query sees all of its keys.  Rows of out that belong to no
    sequence are left as they were (in a fresh out: whatever the memory held)."""
    dev = torch.cuda.current_device()
    qh = _heads(q, "q", dev)
    _, n_q, hd = q.shape
    n_kv = k.shape[1]
    kh, vh = _heads(k, "k", dev, n_kv, hd), _heads(v, "v", dev, n_kv, hd)
    cu = _host_ints(cu_seqlens, "cu_seqlens")
    ck = cu if cu_seqlens_k is None else _host_ints(cu_seqlens_k, "cu_seqlens_k")
    n = len(cu) - 1
    if n < 0 or len(ck) != n + 1:
        raise ValueError("cu_seqlens (and cu_seqlens_k) hold one offset more than sequences")
    if max(cu) > q.shape[0] or max(ck) > min(k.shape[0], v.shape[0]):
        raise ValueError("the offsets pass the end of q, k or v")
    out = _empty(q.shape, torch.float32, dev, stream) if out is None else out
    oh = _heads(out, "out", dev, n_q, hd)
    if max(cu) > out.shape[0]:
        raise ValueError("the offsets pass the end of out")
    L = lib()
    ws, nbytes = _workspace(
        L.qws_prompt_attention_workspace_bytes(cu, ck, n, n_q, n_kv, hd), workspace, dev, stream)
    check(L.qws_prompt_attention(
        C.byref(qh), C.byref(kh), C.byref(vh), C.byref(oh), cu, ck, n, n_q, n_kv, hd,
        scale, softcap, None if ws is None else ws.data_ptr(), nbytes, stream_handle(stream)))
    return out


def prefix_attention(q, k_prefix, v_prefix, n_prefix: int, k_caches, v_caches, n_ctx,
                     scale: float, softcap: float = 0.0, workspace=None, out=None, stream=None):
    """One decode step of a batch, q [B, n_q, hd]: row b attends to positions 0 .. n_prefix - 1
    of the shared caches [n_kv, max_prefix, hd] and then to 0 .. n_ctx[b] - 1 (host integers)
    of its own, k_caches and v_caches [B, n_kv, max_seq, hd]."""
    dev = torch.cuda.current_device()
    qh = _heads(q, "q", dev)
    B, n_q, hd = q.shape
    shape_p, shape_c = k_prefix.shape, k_caches.shape
    n_kv = shape_p[0]
    if len(shape_p) != 3 or shape_p[2] != hd or v_prefix.shape != shape_p:
        raise ValueError(f"k_prefix {tuple(shape_p)} and v_prefix {tuple(v_prefix.shape)} must be "
                         f"[n_kv, max_prefix, {hd}]")
    if (len(shape_c) != 4 or shape_c[0] != B or shape_c[1] != n_kv or shape_c[3] != hd
            or v_caches.shape != shape_c):
        raise ValueError(f"k_caches {tuple(shape_c)} and v_caches {tuple(v_caches.shape)} must be "
                         f"[{B}, {n_kv}, max_seq, {hd}]")
    kp, vp = _cache(k_prefix, "k_prefix", dev), _cache(v_prefix, "v_prefix", dev)
    kc, vc = _cache(k_caches, "k_caches", dev), _cache(v_caches, "v_caches", dev)
    lens = _host_ints(n_ctx, "n_ctx")
    if len(lens) != B:
        raise ValueError(f"q has {B} rows, n_ctx {len(lens)}")
    out = _empty(q.shape, torch.float32, dev, stream) if out is None else out
    oh = _heads(out, "out", dev, n_q, hd)
    if out.shape[0] != B:
        raise ValueError(f"out must have {B} rows")
    if B == 0:
        return out
    L = lib()
    ws, nbytes = _workspace(
        L.qws_prefix_attention_workspace_bytes(n_prefix, lens, B, n_q, n_kv, hd), workspace, dev,
        stream)
    check(L.qws_prefix_attention(
        C.byref(qh), kp, vp, shape_p[1], n_prefix, kc, vc, shape_c[2], lens, C.byref(oh), B, n_q,
        n_kv, hd, scale, softcap,
        None if ws is None else ws.data_ptr(), nbytes, stream_handle(stream)))
    return out


# ------------------------------------------------------------ a paged cache, sampling
def paged_kv_head_bytes(fmt: int, head_dim: int, page_size: int) -> int:
    """Bytes of one kv head's part of a page; pages are uint8 [n_pages, n_kv, these bytes]."""
    n = int(lib().qws_paged_kv_head_bytes(fmt, head_dim, page_size))
    if n == 0:
        raise ValueError(f"no paged cache in format {fmt} with head_dim {head_dim} and page_size "
                         f"{page_size}: Q4_0 or Q8_0, 32 to 256, a multiple of 16")
    return n


def _out_heads(t, shape, name: str, dev: int, stream):
    """An output of that shape, the given one or a fresh one, and its qws_heads."""
    if t is None:
        t = _empty(shape, torch.float32, dev, stream)
        return t, _lib.QwsHeads(t.data_ptr(), shape[1] * shape[2], shape[2])
    h = _heads(t, name, dev, shape[1], shape[2])
    if t.shape[0] != shape[0]:
        raise ValueError(f"{name} must have {shape[0]} tokens")
    return t, h


def _paged(fmt: int, pages, table, head_dim: int, dev: int):
    """qws_paged_kv of pages uint8 [n_pages, n_kv, bytes] and table int32 [n_seqs, max_pages]."""
    if not isinstance(pages, torch.Tensor) or pages.get_device() != dev:
        _here(pages, "pages", dev)
    if not isinstance(table, torch.Tensor) or table.get_device() != dev:
        _here(table, "table", dev)
    if pages.dtype != torch.uint8 or table.dtype != torch.int32:
        raise TypeError(f"pages must be torch.uint8 and table torch.int32, got {pages.dtype} and "
                        f"{table.dtype}")
    shape, rows = pages.shape, table.shape
    if len(shape) != 3 or len(rows) != 2 or not pages.is_contiguous() or not table.is_contiguous():
        raise ValueError("pages must be [n_pages, n_kv, bytes] and table [n_seqs, max_pages], "
                         "contiguous")
    # the library refuses other formats and head sizes itself, but sees 32 bits of them
    if fmt not in (Q4_0, Q8_0):
        fmt = 0
    slab = {Q4_0: 18 * head_dim, Q8_0: 34 * head_dim}.get(fmt, 0) or shape[2] or 1
    if shape[2] == 0 or shape[2] % slab:
        raise ValueError(f"a kv head's part of a page has {shape[2]} bytes, not a multiple of "
                         f"{slab}, those of 16 positions")
    if shape[2] // slab > 4096:
        raise ValueError(f"a page has {shape[2] // slab * 16} positions, at most 65536 are taken")
    return _lib.QwsPagedKv(fmt, shape[2] // slab * 16, shape[1], head_dim, pages.data_ptr(),
                           shape[0], table.data_ptr(), rows[0], rows[1])


def paged_kv_append(fmt: int, pages, table, k, v, seqs, positions, rot_dim: int = 0,
                    base: float = 10000.0, w_k=None, eps: float = 1e-6, q=None, w_q=None,
                    q_out=None, stream=None):
    """Norm (w_k, w_q [hd]; None: no norm) and rotation (rot_dim 0: none) of every head of k and
    q at positions [T], then k and v [T, n_kv, hd] quantised into the pages of sequences seqs [T]
    (int64 both; negative: padding, not stored).  Returns q_out [T, n_q, hd], None without q."""
    dev = torch.cuda.current_device()
    kh = _heads(k, "k", dev)
    n, n_kv, hd = k.shape
    kv = _paged(fmt, pages, table, hd, dev)
    if kv.n_kv_heads != n_kv:
        raise ValueError(f"pages hold {kv.n_kv_heads} kv heads, k {n_kv}")
    vh = _heads(v, "v", dev, n_kv, hd)
    if v.shape[0] != n:
        raise ValueError(f"v must have {n} tokens")
    qh = oh = None
    n_q = 0
    if q is not None:
        qh = _heads(q, "q", dev)
        n_tok, n_q, hd_q = q.shape
        if n_tok != n or hd_q != hd:
            raise ValueError(f"q {tuple(q.shape)} and k {tuple(k.shape)} do not match")
        q_out, oh = _out_heads(q_out, (n, n_q, hd), "q_out", dev, stream)
        qh, oh = C.byref(qh), C.byref(oh)
    elif q_out is not None or w_q is not None:
        raise ValueError("q_out and w_q go with q")
    if n:
        check(lib().qws_paged_kv_append(
            C.byref(kv), qh, C.byref(kh), C.byref(vh), oh,
            None if w_q is None else _vec(w_q, "w_q", dev, torch.float32, hd),
            None if w_k is None else _vec(w_k, "w_k", dev, torch.float32, hd),
            _vec(seqs, "seqs", dev, torch.int64, n),
            _vec(positions, "positions", dev, torch.int64, n), n, n_q,
            max(-1, min(rot_dim, hd + 1)), base, eps,       # (the library sees 32 bits of it)
            stream_handle(stream)))
    return q_out


def paged_kv_gather(fmt: int, pages, table, seqs, positions, head_dim: int, k_out=None,
                    v_out=None, stream=None):
    """The f32 keys and values [T, n_kv, hd] that the cache holds for sequences seqs [T] at
    positions [T]; zeros for padding (negative ones)."""
    dev = torch.cuda.current_device()
    kv = _paged(fmt, pages, table, head_dim, dev)
    n = seqs.numel()
    shape = (n, kv.n_kv_heads, head_dim)
    k_out, kh = _out_heads(k_out, shape, "k_out", dev, stream)
    v_out, vh = _out_heads(v_out, shape, "v_out", dev, stream)
    if n:
        check(lib().qws_paged_kv_gather(
            C.byref(kv), _vec(seqs, "seqs", dev, torch.int64, n),
            _vec(positions, "positions", dev, torch.int64, n), n, C.byref(kh), C.byref(vh),
            stream_handle(stream)))
    return k_out, v_out


def paged_kv_attention(fmt: int, pages, table, q, seqs, positions, scale: float,
                       softcap: float = 0.0, workspace=None, out=None, stream=None,
                       tokens_per_seq: int = 0):
    """q [T, n_q, hd]: row t attends to positions 0 .. positions[t] of sequence seqs[t] in the
    pages (int64 both, on the device; negative: padding, a row of zeros).  tokens_per_seq: how
    many neighbouring rows a sequence has, about, for the form that is fastest for them; 0: more
    than one if there are more rows than the table has."""
    dev = torch.cuda.current_device()
    qh = _heads(q, "q", dev)
    n, n_q, hd = q.shape
    kv = _paged(fmt, pages, table, hd, dev)
    if tokens_per_seq < 0:
        raise ValueError(f"tokens_per_seq = {tokens_per_seq} < 0")
    kv.tokens_per_seq = min(tokens_per_seq, n)
    out, oh = _out_heads(out, (n, n_q, hd), "out", dev, stream)
    if n == 0:
        return out
    L = lib()
    ws, nbytes = _workspace(
        L.qws_paged_kv_attention_workspace_bytes(n, n_q, kv.n_kv_heads, hd), workspace, dev,
        stream)
    check(L.qws_paged_kv_attention(
        C.byref(kv), C.byref(qh), C.byref(oh), _vec(seqs, "seqs", dev, torch.int64, n),
        _vec(positions, "positions", dev, torch.int64, n), n, n_q, scale, softcap,
        None if ws is None else ws.data_ptr(), nbytes, stream_handle(stream)))
    return out


def sample_tokens(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, out=None,
                  stream=None):
    """The next token (int64 [n]) of every row of logits [n, vocab] (f32; rows may be strided)
    from the random numbers u [n] in [0, 1): the first top_k, then as few as reach top_p of
    them, those with at least min_p of the largest probability, at the temperature (0: the
    largest logit).  The parameters are tensors [n] (top_k int64, the others f32) or None."""
    dev = torch.cuda.current_device()
    if not isinstance(logits, torch.Tensor) or logits.get_device() != dev:
        _here(logits, "logits", dev)
    if logits.dtype != torch.float32:
        raise TypeError(f"logits must be torch.float32, got {logits.dtype}")
    shape = logits.shape
    if len(shape) != 2 or (logits.stride(1) != 1 and shape[1] > 1):
        raise ValueError(f"logits must be [rows, vocab] with contiguous rows, got {tuple(shape)}")
    n, vocab = shape
    f32, i64 = torch.float32, torch.int64
    out = _empty((n,), i64, dev, stream) if out is None else out
    if n:
        check(lib().qws_sample_tokens(
            logits.data_ptr(), logits.stride(0), vocab, n, _vec(u, "u", dev, f32, n),
            None if temperature is None else _vec(temperature, "temperature", dev, f32, n),
            None if top_k is None else _vec(top_k, "top_k", dev, i64, n),
            None if top_p is None else _vec(top_p, "top_p", dev, f32, n),
            None if min_p is None else _vec(min_p, "min_p", dev, f32, n),
            _vec(out, "out", dev, i64, n), stream_handle(stream)))
    return out


def q4k_ffn_gate_up_geglu(Wg, Wu, x, hidden: int, inter: int, out=None, stream=None):
    m = _out(out, (inter,), x, stream)
    check(lib().qws_q4k_ffn_gate_up_geglu(_dev(Wg, "Wg", torch.uint8), _dev(Wu, "Wu", torch.uint8),
                                          _dev(x, "x", torch.float32), _dev(m, "m", torch.float32),
                                          hidden, inter, stream_handle(stream)))
    return m


def q4k_ffn_gate_up_geglu_down(Wg, Wu, Wd, wd_fmt: int, x, hidden: int, inter: int,
                               workspace=None, out=None, stream=None):
    y = _out(out, (hidden,), x, stream)
    need = workspace_bytes(OP_FFN, 0, hidden, inter, 1, 0)
    if workspace is None:
        workspace = _empty(need, torch.uint8, x.device, stream, returned=False)
    check(lib().qws_q4k_ffn_gate_up_geglu_down(
        _dev(Wg, "Wg", torch.uint8), _dev(Wu, "Wu", torch.uint8), _dev(Wd, "Wd", torch.uint8),
        wd_fmt, _dev(x, "x", torch.float32), _dev(y, "y", torch.float32), hidden, inter,
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        stream_handle(stream)))
    return y


def q4k_ffn_gate_up_silu(Wg, Wu, x, hidden: int, inter: int, out=None, stream=None):
    m = _out(out, (inter,), x, stream)
    check(lib().qws_q4k_ffn_gate_up_silu(_dev(Wg, "Wg", torch.uint8), _dev(Wu, "Wu", torch.uint8),
                                         _dev(x, "x", torch.float32), _dev(m, "m", torch.float32),
                                         hidden, inter, stream_handle(stream)))
    return m


def q4k_ffn_gate_up_silu_down(Wg, Wu, Wd, wd_fmt: int, x, hidden: int, inter: int,
                              workspace=None, out=None, stream=None):
    y = _out(out, (hidden,), x, stream)
    need = workspace_bytes(OP_FFN, 0, hidden, inter, 1, 0)
    if workspace is None:
        workspace = _empty(need, torch.uint8, x.device, stream, returned=False)
    check(lib().qws_q4k_ffn_gate_up_silu_down(
        _dev(Wg, "Wg", torch.uint8), _dev(Wu, "Wu", torch.uint8), _dev(Wd, "Wd", torch.uint8),
        wd_fmt, _dev(x, "x", torch.float32), _dev(y, "y", torch.float32), hidden, inter,
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        stream_handle(stream)))
    return y


def residual_rms_norm(h, y, w, eps: float, batch: int = 1, out=None, stream=None):
    """h += y (in place), returns x = rms_norm(h, w)."""
    n = h.numel() // batch
    x = _out(out, tuple(h.shape), h, stream)
    check(lib().qws_residual_rms_norm(_dev(h, "h", torch.float32), _dev(y, "y", torch.float32),
                                      _dev(w, "w", torch.float32), _dev(x, "x", torch.float32), n,
                                      float(eps), batch, stream_handle(stream)))
    return x


def rms_norm(x, w, eps: float, batch: int = 1, out=None, stream=None):
    y = _out(out, tuple(x.shape), x, stream)
    n = x.numel() // batch
    check(lib().qws_rms_norm(_dev(x, "x", torch.float32), _dev(w, "w", torch.float32),
                             _dev(y, "y", torch.float32), n, float(eps), batch,
                             stream_handle(stream)))
    return y


def residual_add(h, y, batch: int = 1, stream=None):
    n = h.numel() // batch
    check(lib().qws_residual_add(_dev(h, "h", torch.float32), _dev(y, "y", torch.float32), n,
                                 batch, stream_handle(stream)))
    return h


Layer = _lib.QwsLayer
Dims = _lib.QwsDims


def make_layer(t: dict) -> Layer:
    """qws_layer from a dict of device tensors (Wq..Wd uint8, w_* float32) and formats."""
    return Layer(
        _dev(t["Wq"], "Wq", torch.uint8), _dev(t["Wk"], "Wk", torch.uint8),
        _dev(t["Wv"], "Wv", torch.uint8), _dev(t["Wo"], "Wo", torch.uint8),
        _dev(t["Wg"], "Wg", torch.uint8), _dev(t["Wu"], "Wu", torch.uint8),
        _dev(t["Wd"], "Wd", torch.uint8),
        int(t["fmt_qkv"]), int(t["fmt_o"]), int(t["fmt_gu"]), int(t["fmt_down"]),
        _dev(t["w_in"], "w_in", torch.float32), _dev(t["w_post_attn"], "w_post_attn", torch.float32),
        _dev(t["w_pre_ffn"], "w_pre_ffn", torch.float32),
        _dev(t["w_post_ffn"], "w_post_ffn", torch.float32))


def make_dims(d: dict) -> Dims:
    return Dims(int(d["hidden"]), int(d["inter"]), int(d["n_q_heads"]), int(d["n_kv_heads"]),
                int(d["head_dim"]), float(d["eps"]), int(d["post_norms"]))


def decode_chain(layers, h, dims: dict, workspace=None, stream=None, w_final=None, hn=None):
    """Runs len(layers) decoder layers on h (in place).  layers: list of dicts
    of device tensors (see make_layer) or prepared Layer structs.  With
    w_final and hn (qws_decode_chain_final_norm) the same launch also writes
    hn = rms_norm(h, w_final) after the last layer."""
    n = len(layers)
    arr = (Layer * n)(*[L if isinstance(L, Layer) else make_layer(L) for L in layers])
    D = make_dims(dims)
    # the kernel reads / writes `hidden` values of each: a shorter tensor
    # would be overrun on the device, so refuse it here
    for name, t in (("h", h), ("w_final", w_final), ("hn", hn)):
        if isinstance(t, torch.Tensor) and t.numel() < int(dims["hidden"]):
            raise ValueError(f"{name} has {t.numel()} elements, hidden is {dims['hidden']}")
    need = workspace_bytes(OP_DECODE_CHAIN, 0, dims["hidden"], dims["inter"], 1, 0)
    if workspace is None:
        workspace = _empty(max(need, 1), torch.uint8, h.device, stream, returned=False)
    nbytes = workspace.numel() * workspace.element_size()
    if w_final is None and hn is None:
        check(lib().qws_decode_chain(arr, n, _dev(h, "h", torch.float32), C.byref(D),
                                     _dev(workspace, "workspace"), nbytes,
                                     stream_handle(stream)))
        return h
    check(lib().qws_decode_chain_final_norm(
        arr, n, _dev(h, "h", torch.float32), _dev(w_final, "w_final", torch.float32),
        _dev(hn, "hn", torch.float32), C.byref(D), _dev(workspace, "workspace"), nbytes,
        stream_handle(stream)))
    return h


def decode_kv_workspace_bytes(dims: dict, max_seq: int) -> int:
    D = make_dims(dims)
    return int(lib().qws_decode_kv_workspace_bytes(C.byref(D), int(max_seq)))


def decode_kv(layers, h, dims: dict, k_caches, v_caches, max_seq: int, pos: int, rot_dim: int,
              rope_base: float, attn_scale: float, softcap: float = 0.0, workspace=None,
              stream=None):
    """One decode step at position pos over len(layers) layers with KV caches
    (qws_decode_kv): h in place; k_caches[l] / v_caches[l] are f32 device
    tensors [n_kv_heads, max_seq, head_dim], position pos is written."""
    n = len(layers)
    if len(k_caches) != n or len(v_caches) != n:
        raise ValueError("one k and one v cache per layer")
    # the kernels read / write these extents: refuse shorter tensors here
    if h.numel() < int(dims["hidden"]):
        raise ValueError(f"h has {h.numel()} elements, hidden is {dims['hidden']}")
    cache = int(dims["n_kv_heads"]) * int(max_seq) * int(dims["head_dim"])
    for t in list(k_caches) + list(v_caches):
        if isinstance(t, torch.Tensor) and t.numel() < cache:
            raise ValueError(f"a cache has {t.numel()} elements, needs {cache}")
    arr = (Layer * n)(*[L if isinstance(L, Layer) else make_layer(L) for L in layers])
    D = make_dims(dims)
    kp = (C.c_void_p * n)(*[_dev(t, "k_cache", torch.float32) for t in k_caches])
    vp = (C.c_void_p * n)(*[_dev(t, "v_cache", torch.float32) for t in v_caches])
    kv = _lib.QwsKv(C.cast(kp, C.c_void_p), C.cast(vp, C.c_void_p), int(max_seq), int(pos),
                    int(rot_dim), float(rope_base), float(attn_scale), float(softcap))
    need = decode_kv_workspace_bytes(dims, max_seq)
    if workspace is None:
        workspace = _empty(max(need, 1), torch.uint8, h.device, stream, returned=False)
    check(lib().qws_decode_kv(arr, n, _dev(h, "h", torch.float32), C.byref(D), C.byref(kv),
                              _dev(workspace, "workspace"),
                              workspace.numel() * workspace.element_size(),
                              stream_handle(stream)))
    return h


def device_error() -> int:
    """Waits for the device; returns (and clears) the kernels' error code (0 = none)."""
    code = C.c_uint(0)
    lib().qws_device_error(C.byref(code))
    return int(code.value)
