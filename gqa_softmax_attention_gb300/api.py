"""Python entry points with the C ABI's names; torch supplies memory and streams.

Every step of the computation runs in libgqa_attn.so.  These functions check
dtypes and devices, make inputs contiguous (TileOPs GQADenseFwdOp, forward:
non-contiguous inputs are copied first), resolve ``scale=None`` to 1/sqrt(D)
(RL-Kernel Tensor Contract), allocate outputs with torch and pass raw pointers
plus the current CUDA stream.  A non-OK status raises: ``ValueError`` for
argument problems (naming the refused limit), ``RuntimeError`` for CUDA errors.
"""
import ctypes
import math

import torch

from . import _lib

_ARG_ERRORS = {1, 2, 3, 4}


def _raise(status: int, what: str):
    name = _lib.status_name(status)
    msg = "%s: %s (%s)" % (what, _lib.load().gqa_status_string(status).decode(), name)
    if status in _ARG_ERRORS:
        raise ValueError(msg)
    raise RuntimeError(msg)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


_DTYPES = {torch.bfloat16: 0, torch.float16: 1}      # gqa_dtype


def _check_16_cuda(name, t, ndim, dtypes=(torch.bfloat16, torch.float16)):
    """A CUDA tensor of ndim dimensions and one of the given dtypes."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype not in dtypes:
        raise ValueError("%s must be %s, got %s" % (name, " or ".join(str(d) for d in dtypes), t.dtype))
    if t.dim() != ndim:
        raise ValueError("%s must have %d dimensions, got %d" % (name, ndim, t.dim()))


def resolve_scale(scale, D):
    """None -> 1/sqrt(D); an explicit value (0.0 included) is used verbatim."""
    return 1.0 / math.sqrt(D) if scale is None else float(scale)


def _options(window_left, window_right, softcap, sinks, Hq, device, dtype=0):
    """gqa_options for the optional terms and the element type, or None when
    none is set (the sinks tensor is returned too, to keep it alive for the
    call)."""
    if window_left == -1 and window_right == -1 and not softcap and sinks is None and dtype == 0:
        return None, None
    for n, w in (("window_left", window_left), ("window_right", window_right)):
        if int(w) < -1:
            raise ValueError("%s must be -1 (unlimited) or >= 0, got %d" % (n, int(w)))
    cap = 0.0 if softcap is None else float(softcap)
    if not math.isfinite(cap) or cap < 0.0:
        raise ValueError("softcap must be finite and >= 0, got %r" % (softcap,))
    sk = None
    if sinks is not None:
        sk = torch.as_tensor(sinks).to(device=device, dtype=torch.float32).contiguous()
        if tuple(sk.shape) != (Hq,):
            raise ValueError("sinks must be [Hq] = [%d]" % Hq)
    opt = _lib.Options(int(window_left), int(window_right), cap, sk.data_ptr() if sk is not None else None,
                       int(dtype))
    return opt, sk


def attn_fwd_dense(q, k, v, key_padding_mask=None, causal=True, scale=None, out=None, lse=None,
                   window_left=-1, window_right=-1, softcap=None, sinks=None):
    """Dense / chunked-prefill GQA attention.

    q [B,Sq,Hq,D], k/v [B,Skv,Hkv,D] CUDA tensors (BSHD), all bfloat16 or all
    float16 (the output takes the same type);
    key_padding_mask [B,Skv] bool (True = keep) or None.
    window_left / window_right: keys admitted left / right of each query's key
    position (-1 unlimited); softcap: c > 0 caps each scaled score to
    c*tanh(z/c) (None or 0 off); sinks: [Hq] float32 logits joining the
    softmax denominator only, or None.
    Returns (o [B,Sq,Hq,D] bf16, lse [B,Sq,Hq] float32, natural log).
    """
    _check_16_cuda("q", q, 4)
    for n, t in (("k", k), ("v", v)):
        _check_16_cuda(n, t, 4, (q.dtype,))
    B, Sq, Hq, D = q.shape
    Bk, Skv, Hkv, Dk = k.shape
    if Bk != B or Dk != D or tuple(v.shape) != tuple(k.shape):
        raise ValueError("shape mismatch: q %s, k %s, v %s" % (tuple(q.shape), tuple(k.shape), tuple(v.shape)))
    if Hq % Hkv != 0:
        raise ValueError("Hq (%d) must be divisible by Hkv (%d)" % (Hq, Hkv))
    q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    m = None
    if key_padding_mask is not None:
        if tuple(key_padding_mask.shape) != (B, Skv):
            raise ValueError("key_padding_mask must be [B, Skv] = [%d, %d]" % (B, Skv))
        m = key_padding_mask.to(device=q.device, dtype=torch.bool).contiguous().view(torch.uint8)
    if out is None:
        out = torch.empty((B, Sq, Hq, D), dtype=q.dtype, device=q.device)
    if lse is None:
        lse = torch.empty((B, Sq, Hq), dtype=torch.float32, device=q.device)
    opt, _keep = _options(window_left, window_right, softcap, sinks, Hq, q.device, _DTYPES[q.dtype])
    lib = _lib.load()
    if opt is None:
        st = lib.attn_fwd_dense(_ptr(q), _ptr(k), _ptr(v), _ptr(m), _ptr(out), _ptr(lse), B, Hq, Hkv, Sq, Skv, D,
                                int(bool(causal)), resolve_scale(scale, D), _stream(q.device))
    else:
        st = lib.attn_fwd_dense_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(m), _ptr(out), _ptr(lse), B, Hq, Hkv, Sq, Skv,
                                   D, int(bool(causal)), resolve_scale(scale, D), ctypes.byref(opt),
                                   _stream(q.device))
    if st != 0:
        _raise(st, "attn_fwd_dense")
    return out, lse


def _check_paged(q, k_cache, v_cache, real_seqlen_kv, block_table, dtypes=(torch.bfloat16, torch.float16)):
    """Checks shared by the paged decode entry points: q [B,Sq,Hq,D] and the
    caches [num_pages,page_size,Hkv,D] CUDA tensors of one 16-bit type, Hq a
    multiple of Hkv, real_seqlen_kv [B] and block_table [B,max_pages] int32 CUDA
    tensors.  Returns the five tensors made contiguous."""
    _check_16_cuda("q", q, 4, dtypes)
    _check_16_cuda("k_cache", k_cache, 4, (q.dtype,))
    _check_16_cuda("v_cache", v_cache, 4, (q.dtype,))
    B, Sq, Hq, D = q.shape
    num_pages, page_size, Hkv, Dk = k_cache.shape
    if Dk != D or tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError("cache shape mismatch: k %s, v %s, D %d" % (tuple(k_cache.shape), tuple(v_cache.shape), D))
    if Hq % Hkv != 0:
        raise ValueError("Hq (%d) must be divisible by Hkv (%d)" % (Hq, Hkv))
    for n, t in (("real_seqlen_kv", real_seqlen_kv), ("block_table", block_table)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.int32:
            raise ValueError("%s must be an int32 CUDA tensor" % n)
        if t.device != q.device:
            raise ValueError("%s must be on q's device %s, got %s" % (n, q.device, t.device))
    if tuple(real_seqlen_kv.shape) != (B,) or block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("real_seqlen_kv must be [B] and block_table [B, max_pages]")
    return (q.contiguous(), k_cache.contiguous(), v_cache.contiguous(), real_seqlen_kv.contiguous(),
            block_table.contiguous())


def attn_decode_paged_workspace_size(B, Sq, Hq, Hkv, D, page_size, max_pages):
    """Workspace bytes attn_decode_paged needs on the current device."""
    return int(_lib.load().attn_decode_paged_workspace_size(B, Sq, Hq, Hkv, D, page_size, max_pages))


def attn_decode_paged(q, k_cache, v_cache, real_seqlen_kv, block_table, causal=True, scale=None,
                      workspace=None, out=None, lse=None, window_left=-1, window_right=-1, softcap=None,
                      sinks=None):
    """Paged decode.

    q [B,Sq,Hq,D]; k_cache/v_cache [num_pages,page_size,Hkv,D], all bfloat16 or all float16;
    real_seqlen_kv [B] int32 (query tokens included); block_table [B,max_pages] int32.
    workspace: optional uint8 CUDA tensor of at least attn_decode_paged_workspace_size bytes.
    window_left / window_right / softcap / sinks as in attn_fwd_dense.
    Returns (o [B,Sq,Hq,D] bf16, lse [B,Sq,Hq] float32).
    """
    q, k_cache, v_cache, sl, bt = _check_paged(q, k_cache, v_cache, real_seqlen_kv, block_table)
    B, Sq, Hq, D = q.shape
    num_pages, page_size, Hkv, _ = k_cache.shape
    max_pages = bt.shape[1]
    need = attn_decode_paged_workspace_size(B, Sq, Hq, Hkv, D, page_size, max_pages)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty((B, Sq, Hq, D), dtype=q.dtype, device=q.device)
    if lse is None:
        lse = torch.empty((B, Sq, Hq), dtype=torch.float32, device=q.device)
    opt, _keep = _options(window_left, window_right, softcap, sinks, Hq, q.device, _DTYPES[q.dtype])
    lib = _lib.load()
    wsb = workspace.numel() * workspace.element_size()
    if opt is None:
        st = lib.attn_decode_paged(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(sl), _ptr(bt), page_size,
                                   _ptr(out), _ptr(lse), B, Sq, Hq, Hkv, D, num_pages, max_pages,
                                   int(bool(causal)), resolve_scale(scale, D), _ptr(workspace), wsb,
                                   _stream(q.device))
    else:
        st = lib.attn_decode_paged_ex(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(sl), _ptr(bt), page_size,
                                      _ptr(out), _ptr(lse), B, Sq, Hq, Hkv, D, num_pages, max_pages,
                                      int(bool(causal)), resolve_scale(scale, D), ctypes.byref(opt),
                                      _ptr(workspace), wsb, _stream(q.device))
    if st != 0:
        _raise(st, "attn_decode_paged")
    return out, lse


def attn_decode_paged_fp8kv(q, k_cache, v_cache, k_scale, v_scale, real_seqlen_kv, block_table, causal=True,
                            scale=None, workspace=None, out=None, lse=None, window_left=-1, window_right=-1,
                            softcap=None, sinks=None):
    """Paged decode over float8_e4m3fn key/value caches.

    q [B,Sq,Hq,D] bfloat16 or float16; k_cache/v_cache [num_pages,page_size,Hkv,D]
    torch.float8_e4m3fn (or uint8 holding e4m3fn codes); k_scale/v_scale [B,Hkv]
    float32 CUDA tensors or None (ones): key t of KV head r in request b is
    K * k_scale[b, r] and its value V * v_scale[b, r].  Every scale must be finite
    and positive; they stay on the GPU and are not checked.  D is 128 or 256.  Other
    arguments as attn_decode_paged.  Returns (o like q, lse [B,Sq,Hq] float32).
    """
    _check_16_cuda("q", q, 4)
    for n, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 4 or \
                t.dtype not in (torch.float8_e4m3fn, torch.uint8):
            raise ValueError("%s must be a 4-D float8_e4m3fn (or uint8) CUDA tensor" % n)
    B, Sq, Hq, D = q.shape
    num_pages, page_size, Hkv, Dk = k_cache.shape
    if Dk != D or tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError("cache shape mismatch: k %s, v %s, D %d" % (tuple(k_cache.shape), tuple(v_cache.shape), D))
    if Hq % Hkv != 0:
        raise ValueError("Hq (%d) must be divisible by Hkv (%d)" % (Hq, Hkv))
    for n, t in (("real_seqlen_kv", real_seqlen_kv), ("block_table", block_table)):
        if not t.is_cuda or t.dtype != torch.int32:
            raise ValueError("%s must be an int32 CUDA tensor" % n)
    if tuple(real_seqlen_kv.shape) != (B,) or block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("real_seqlen_kv must be [B] and block_table [B, max_pages]")
    scales = []
    for n, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        if t is not None:
            if not t.is_cuda or t.dtype != torch.float32 or t.numel() != B * Hkv:
                raise ValueError("%s must be a float32 CUDA tensor of B * Hkv values" % n)
            t = t.contiguous()
        scales.append(t)
    max_pages = block_table.shape[1]
    q, k_cache, v_cache = q.contiguous(), k_cache.contiguous(), v_cache.contiguous()
    sl, bt = real_seqlen_kv.contiguous(), block_table.contiguous()
    need = attn_decode_paged_workspace_size(B, Sq, Hq, Hkv, D, page_size, max_pages)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty((B, Sq, Hq, D), dtype=q.dtype, device=q.device)
    if lse is None:
        lse = torch.empty((B, Sq, Hq), dtype=torch.float32, device=q.device)
    opt, _keep = _options(window_left, window_right, softcap, sinks, Hq, q.device, _DTYPES[q.dtype])
    st = _lib.load().attn_decode_paged_fp8kv(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(scales[0]), _ptr(scales[1]), _ptr(sl), _ptr(bt), page_size,
        _ptr(out), _ptr(lse), B, Sq, Hq, Hkv, D, num_pages, max_pages, int(bool(causal)), resolve_scale(scale, D),
        ctypes.byref(opt) if opt is not None else None, _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(q.device))
    if st != 0:
        _raise(st, "attn_decode_paged_fp8kv")
    return out, lse


def attn_decode_paged_noalloc(q, k_cache, v_cache, real_seqlen_kv, block_table, causal=True, scale=None, out=None,
                              lse=None):
    """Paged decode through the entry point that allocates nothing in the library.

    For callers that cannot allocate device memory or supply a workspace: the
    split partials go to a fixed 32 MiB array inside the library, shared by all
    calls (calls overlapping on the GPU race).  Sizes whose partials do not fit
    raise ValueError.  Outputs are allocated here only when not passed in.
    """
    q, k_cache, v_cache, real_seqlen_kv, block_table = _check_paged(q, k_cache, v_cache, real_seqlen_kv,
                                                                    block_table, (torch.bfloat16,))
    B, Sq, Hq, D = q.shape
    num_pages, page_size, Hkv, _ = k_cache.shape
    max_pages = block_table.shape[1]
    if out is None:
        out = torch.empty((B, Sq, Hq, D), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((B, Sq, Hq), dtype=torch.float32, device=q.device)
    st = _lib.load().attn_decode_paged_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(real_seqlen_kv),
                                               _ptr(block_table), page_size, _ptr(out), _ptr(lse), B, Sq, Hq, Hkv,
                                               D, num_pages, max_pages, int(bool(causal)),
                                               resolve_scale(scale, D), _stream(q.device))
    if st != 0:
        _raise(st, "attn_decode_paged_noalloc (static scratch %d bytes)"
               % _lib.load().attn_decode_paged_noalloc_max_workspace())
    return out, lse


def attn_varlen_workspace_size(B, total_q, Hq, Hkv):
    """Workspace bytes of attn_fwd_varlen / attn_fwd_paged."""
    return int(_lib.load().attn_varlen_workspace_size(B, total_q, Hq, Hkv))


def attn_paged_workspace_size(B, total_q, Hq, Hkv, D, page_size, max_pages):
    """Workspace bytes of attn_fwd_paged with its single-query requests on the
    split-KV decode kernel (equal to attn_varlen_workspace_size when the sizes
    keep every request on the packed kernel)."""
    return int(_lib.load().attn_paged_workspace_size(B, total_q, Hq, Hkv, D, page_size, max_pages))


def _check_offsets(name, t, n):
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.int32 or tuple(t.shape) != (n,):
        raise ValueError("%s must be an int32 CUDA tensor of shape [%d]" % (name, n))
    return t.contiguous()


def _varlen_outputs(q, out, lse, workspace, B):
    total_q, Hq, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((total_q, Hq), dtype=torch.float32, device=q.device)
    return out, lse


def attn_fwd_varlen(q, k, v, cu_seqlens_q, cu_seqlens_kv, causal=True, scale=None, out=None, lse=None,
                    window_left=-1, window_right=-1, softcap=None, sinks=None, workspace=None):
    """Packed variable-length GQA attention (TileOPs GQAVarlenFwdOp).

    q [total_q, Hq, D], k / v [total_kv, Hkv, D] CUDA tensors (THD), all
    bfloat16 or all float16; cu_seqlens_q / cu_seqlens_kv [B + 1] int32 CUDA
    offsets (request b owns rows cu[b]:cu[b+1]; they stay on the device).
    Options as in attn_fwd_dense.  Returns (o [total_q, Hq, D], lse [total_q, Hq]).
    """
    _check_16_cuda("q", q, 3)
    for n, t in (("k", k), ("v", v)):
        _check_16_cuda(n, t, 3, (q.dtype,))
    total_q, Hq, D = q.shape
    total_kv, Hkv, Dk = k.shape
    if Dk != D or tuple(v.shape) != tuple(k.shape):
        raise ValueError("shape mismatch: q %s, k %s, v %s" % (tuple(q.shape), tuple(k.shape), tuple(v.shape)))
    if Hq % Hkv != 0:
        raise ValueError("Hq (%d) must be divisible by Hkv (%d)" % (Hq, Hkv))
    if cu_seqlens_q.dim() != 1 or cu_seqlens_q.shape[0] < 2:
        raise ValueError("cu_seqlens_q must hold B + 1 >= 2 offsets")
    B = cu_seqlens_q.shape[0] - 1
    cq = _check_offsets("cu_seqlens_q", cu_seqlens_q, B + 1)
    ck = _check_offsets("cu_seqlens_kv", cu_seqlens_kv, B + 1)
    q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    out, lse = _varlen_outputs(q, out, lse, workspace, B)
    need = attn_varlen_workspace_size(B, total_q, Hq, Hkv)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    opt, _keep = _options(window_left, window_right, softcap, sinks, Hq, q.device, _DTYPES[q.dtype])
    st = _lib.load().attn_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(cq), _ptr(ck), _ptr(out), _ptr(lse), B, total_q,
                                     total_kv, Hq, Hkv, D, int(bool(causal)), resolve_scale(scale, D),
                                     ctypes.byref(opt) if opt is not None else None, _ptr(workspace),
                                     workspace.numel() * workspace.element_size(), _stream(q.device))
    if st != 0:
        _raise(st, "attn_fwd_varlen")
    return out, lse


def attn_fwd_paged(q, k_cache, v_cache, cu_seqlens_q, cache_seqlens, block_table, causal=True, scale=None,
                   out=None, lse=None, window_left=-1, window_right=-1, softcap=None, sinks=None, workspace=None,
                   split_decode=True):
    """Packed queries over a paged cache: prefill chunks and decode steps in one
    call (TileOPs GQAPagedFwdOp).

    q [total_q, Hq, D]; k_cache / v_cache [num_pages, page_size, Hkv, D], all
    bfloat16 or all float16; cu_seqlens_q [B + 1], cache_seqlens [B] (query
    tokens included) and block_table [B, max_pages] int32 CUDA tensors.
    Any page size (multiples of 8 move by TMA, others are gathered row by
    row).  Options as in attn_fwd_dense.
    split_decode: give the call the workspace that sends requests with one
    query to the split-KV decode kernel (False: every request on the packed
    kernel).  A caller's workspace decides by its size instead.  With the
    split, the packed kernel runs beside the decode kernel on a library-owned
    high-priority stream, forked from and joined back into the current stream
    inside the call.
    Returns (o [total_q, Hq, D], lse [total_q, Hq]).
    """
    _check_16_cuda("q", q, 3)
    _check_16_cuda("k_cache", k_cache, 4, (q.dtype,))
    _check_16_cuda("v_cache", v_cache, 4, (q.dtype,))
    total_q, Hq, D = q.shape
    num_pages, page_size, Hkv, Dk = k_cache.shape
    if Dk != D or tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError("cache shape mismatch: k %s, v %s, D %d" % (tuple(k_cache.shape), tuple(v_cache.shape), D))
    if Hq % Hkv != 0:
        raise ValueError("Hq (%d) must be divisible by Hkv (%d)" % (Hq, Hkv))
    if cache_seqlens.dim() != 1:
        raise ValueError("cache_seqlens must be [B]")
    B = cache_seqlens.shape[0]
    cq = _check_offsets("cu_seqlens_q", cu_seqlens_q, B + 1)
    sl = _check_offsets("cache_seqlens", cache_seqlens, B)
    if not block_table.is_cuda or block_table.dtype != torch.int32 or block_table.dim() != 2 \
            or block_table.shape[0] != B:
        raise ValueError("block_table must be an int32 CUDA tensor [B, max_pages]")
    bt = block_table.contiguous()
    q, k_cache, v_cache = q.contiguous(), k_cache.contiguous(), v_cache.contiguous()
    out, lse = _varlen_outputs(q, out, lse, workspace, B)
    if split_decode:
        need = attn_paged_workspace_size(B, total_q, Hq, Hkv, D, page_size, bt.shape[1])
    else:
        need = attn_varlen_workspace_size(B, total_q, Hq, Hkv)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    opt, _keep = _options(window_left, window_right, softcap, sinks, Hq, q.device, _DTYPES[q.dtype])
    st = _lib.load().attn_fwd_paged(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(cq), _ptr(sl), _ptr(bt), page_size,
                                    _ptr(out), _ptr(lse), B, total_q, Hq, Hkv, D, num_pages, bt.shape[1],
                                    int(bool(causal)), resolve_scale(scale, D),
                                    ctypes.byref(opt) if opt is not None else None, _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), _stream(q.device))
    if st != 0:
        _raise(st, "attn_fwd_paged")
    return out, lse


def _on(device, fn, *args):
    """fn(*args) with `device` current (the library works on the current device)."""
    if device.index == torch._C._cuda_getDevice():
        return fn(*args)
    with torch.cuda.device(device):
        return fn(*args)


def _raw_stream(device):
    """Handle of the current stream of `device`."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _data(name, t, dtype, shape, device):
    """Address of a contiguous CUDA tensor of this dtype and shape on `device`.
    The test that every good argument passes comes first: these calls are
    launched for a few microseconds of work."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == device.index and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != dtype:
        raise ValueError("%s must be a %s CUDA tensor" % (name, dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.device != device:
        raise ValueError("%s must be on %s, got %s" % (name, device, t.device))
    raise ValueError("%s must be contiguous" % name)


def _size(name, t, ndim, axis):
    """Size of an axis of a tensor of ndim dimensions."""
    if not isinstance(t, torch.Tensor) or t.dim() != ndim:
        raise ValueError("%s must be a CUDA tensor of %d dimensions" % (name, ndim))
    return t.shape[axis]


def attn_fwd_paged_fp8kv(q, k_cache, v_cache, k_scale, v_scale, cu_seqlens_q, cache_seqlens, block_table, causal=True,
                         scale=None, out=None, lse=None, window_left=-1, window_right=-1, softcap=None, sinks=None,
                         workspace=None, split_decode=True):
    """attn_fwd_paged over float8_e4m3fn key/value caches: prefill chunks and
    decode steps in one call.

    q [total_q, Hq, D] bfloat16 or float16, D 128 or 256; k_cache / v_cache
    [num_pages, page_size, Hkv, D] torch.float8_e4m3fn (or uint8 holding e4m3fn
    codes), contiguous; k_scale / v_scale [B, Hkv] float32 CUDA tensors or None (ones):
    key t of KV head r in request b is K * k_scale[b, r], its value V *
    v_scale[b, r].  Every scale must be finite and positive; they stay on the
    GPU and are not checked.  Other arguments as attn_fwd_paged; the default
    workspace (attn_paged_fp8kv_workspace_size bytes) also lets the call cut the
    keys of few rows over long caches into parts for the idle SMs.
    Returns (o [total_q, Hq, D] like q, lse [total_q, Hq] float32).
    """
    _check_16_cuda("q", q, 3)
    dev, i32, f32 = q.device, torch.int32, torch.float32
    total_q, Hq, D = q.shape
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4 or not isinstance(v_cache, torch.Tensor):
        raise ValueError("k_cache and v_cache must be 4-D float8_e4m3fn (or uint8) CUDA tensors")
    num_pages, page_size, Hkv, Dk = shape = k_cache.shape
    if Dk != D or v_cache.shape != shape:
        raise ValueError("cache shape mismatch: k %s, v %s, D %d" % (tuple(shape), tuple(v_cache.shape), D))
    if Hkv == 0 or Hq % Hkv != 0:
        raise ValueError("Hq (%d) must be divisible by Hkv (%d)" % (Hq, Hkv))
    ct = torch.uint8 if k_cache.dtype == torch.uint8 else torch.float8_e4m3fn
    B = _size("cache_seqlens", cache_seqlens, 1, 0)
    max_pages = _size("block_table", block_table, 2, 1)
    kc = _data("k_cache", k_cache, ct, shape, dev)
    vc = _data("v_cache", v_cache, torch.uint8 if v_cache.dtype == torch.uint8 else torch.float8_e4m3fn, shape, dev)
    cq = _data("cu_seqlens_q", cu_seqlens_q, i32, (B + 1,), dev)
    sl = _data("cache_seqlens", cache_seqlens, i32, (B,), dev)
    bt = _data("block_table", block_table, i32, (B, max_pages), dev)
    ks = _data("k_scale", k_scale, f32, (B, Hkv), dev) if k_scale is not None else None
    vs = _data("v_scale", v_scale, f32, (B, Hkv), dev) if v_scale is not None else None
    q = q.contiguous()
    if out is None:
        out = torch.empty_like(q)
        po = out.data_ptr()
    else:
        po = _data("out", out, q.dtype, q.shape, dev)
    if lse is None:
        lse = torch.empty((total_q, Hq), dtype=f32, device=dev)
        pl = lse.data_ptr()
    else:
        pl = _data("lse", lse, f32, (total_q, Hq), dev)
    lib = _lib.load()
    if workspace is None:
        if split_decode:
            need = _on(dev, lib.attn_paged_fp8kv_workspace_size, B, total_q, Hq, Hkv, D, page_size, max_pages)
        else:
            need = lib.attn_varlen_workspace_size(B, total_q, Hq, Hkv)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    elif not isinstance(workspace, torch.Tensor) or not workspace.is_contiguous() or workspace.device != dev:
        raise ValueError("workspace must be a contiguous tensor on %s" % dev)
    opt, _keep = _options(window_left, window_right, softcap, sinks, Hq, dev, _DTYPES[q.dtype])
    st = _on(dev, lib.attn_fwd_paged_fp8kv, q.data_ptr(), kc, vc, ks, vs, cq, sl, bt, page_size, po, pl, B, total_q,
             Hq, Hkv, D, num_pages, max_pages, 1 if causal else 0, resolve_scale(scale, D),
             ctypes.byref(opt) if opt is not None else None, workspace.data_ptr(),
             workspace.numel() * workspace.element_size(), _raw_stream(dev))
    if st != 0:
        _raise(st, "attn_fwd_paged_fp8kv")
    return out, lse


def attn_paged_fp8kv_workspace_size(B, total_q, Hq, Hkv, D, page_size, max_pages):
    """Workspace bytes of attn_fwd_paged_fp8kv with everything split that may be
    (at least attn_paged_workspace_size)."""
    return int(_lib.load().attn_paged_fp8kv_workspace_size(B, total_q, Hq, Hkv, D, page_size, max_pages))


def attn_paged_slots(past_lens, new_lens, block_table, free_pages, page_size, num_pages, max_tokens, free_start=None,
                     out=None):
    """Metadata of one serving step, built on the GPU from the requests' lengths.

    past_lens / new_lens [B] int32: tokens each request holds and brings;
    block_table [B, max_pages] int32, updated in place: the pages the new tokens
    need are entered behind the past ones; free_pages [n] int32 ids handed out
    in request order, from index free_start (an int32 CUDA tensor of one value)
    on; max_tokens: rows of the packed batch, padding included.
    Returns (cu_seqlens_q [B + 1], cache_seqlens [B], slots [max_tokens],
    positions [max_tokens], requests [max_tokens], counts [3]) int32: slots are
    cache rows page * page_size + offset (-1 for padding and for tokens without
    a page), counts the tokens and pages asked for and the next free_start.
    out: the six tensors of an earlier call, written again (the buffers of a
    captured graph).  Nothing is read back: counts[0] > max_tokens, or
    counts[2] > n, tells the caller later that rows or pages ran out.
    The attention calls place query i of a request at cache_seqlens - nq + i, so a
    request whose tokens were cut (by max_tokens, or past the table's capacity of
    max_pages * page_size tokens: cache_seqlens < past + new, which counts does not
    show) has its queries, the valid ones too, at wrong positions: do not use their
    attention; repeat the step with new_lens cut to what fits.  Cache rows and
    other requests are not affected.
    """
    B = _size("past_lens", past_lens, 1, 0)
    dev, i32, T = past_lens.device, torch.int32, int(max_tokens)
    max_pages, n_free = _size("block_table", block_table, 2, 1), _size("free_pages", free_pages, 1, 0)
    pp = _data("past_lens", past_lens, i32, (B,), dev)
    pn = _data("new_lens", new_lens, i32, (B,), dev)
    pt = _data("block_table", block_table, i32, (B, max_pages), dev)
    pf = _data("free_pages", free_pages, i32, (n_free,), dev)
    fs = _data("free_start", free_start, i32, (1,), dev) if free_start is not None else None
    ps, pool = int(page_size), int(num_pages)
    if not 0 <= T < 1 << 30:
        raise ValueError("max_tokens must lie in [0, 2^30), got %d" % T)
    if not (0 < ps < 1 << 30 and 0 <= pool < 1 << 31):           # a C int would take their low 32 bits
        raise ValueError("page_size must lie in [1, 2^30), num_pages in [0, 2^31), got %d, %d" % (ps, pool))
    if out is None:
        buf = torch.empty(2 * B + 3 * T + 4, dtype=i32, device=dev)
        out, p = buf.split((B + 1, B, T, T, T, 3)), buf.data_ptr()
        at = p, p + 4 * (B + 1), p + 4 * (2 * B + 1), p + 4 * (2 * B + T + 1), p + 4 * (2 * B + 2 * T + 1), \
            p + 4 * (2 * B + 3 * T + 1)
    elif len(out) != 6:
        raise ValueError("out must hold six tensors")
    else:
        cu, lens, slots, positions, requests, counts = out
        at = (_data("out cu_seqlens_q", cu, i32, (B + 1,), dev), _data("out cache_seqlens", lens, i32, (B,), dev),
              _data("out slots", slots, i32, (T,), dev), _data("out positions", positions, i32, (T,), dev),
              _data("out requests", requests, i32, (T,), dev), _data("out counts", counts, i32, (3,), dev))
    st = _on(dev, _lib.load().attn_paged_slots, pp, pn, pt, pf, fs, B, max_pages, ps, pool, n_free, T, *at,
             _raw_stream(dev))
    if st != 0:
        _raise(st, "attn_paged_slots")
    return tuple(out)


def _head_rows(t, T):
    """gqa_head_rows of t [..., H, D] with T rows: strides as they are where the
    kernels take them, else of a copy (returned to keep it alive)."""
    if t.dim() == 4:
        t = t.reshape(T, t.shape[2], t.shape[3])      # a view where the rows have one stride
    _, H, D = t.shape
    ts, hs, ds = t.stride()
    # the stride of an axis of one element says nothing
    if T <= 1:
        ts = 0
    if H <= 1:
        hs = 0
    p = t.data_ptr()
    if ds != 1 or ts % 8 or hs % 8 or p % 16:
        t = t.clone(memory_format=torch.contiguous_format)
        p, ts, hs = t.data_ptr(), H * D, D
    return _lib.HeadRows(p, ts, hs), t


def _rope_args(q, k, v, cos_sin, positions, q_weight, k_weight, interleaved, axes):
    """Checks and C arguments shared by attn_qk_norm_rope and its paged form."""
    nd = q.dim() if isinstance(q, torch.Tensor) else 0
    if nd not in (3, 4):
        raise ValueError("q must be a CUDA tensor [T, Hq, D] or [B, S, Hq, D]")
    _check_16_cuda("q", q, nd)
    dev, dt, lead, D = q.device, q.dtype, q.shape[:-2], q.shape[-1]
    T = lead.numel()
    shape = k.shape
    if not (len(shape) == nd and shape[:-2] == lead and shape[-1] == D and k.dtype is dt and k.device == dev and
            (v is None or v.shape == shape and v.dtype is dt and v.device == dev)):
        raise ValueError("q, k and v must have one dtype, device, leading shape and head dim, k and v as many heads: "
                         + ", ".join("%s %s" % (tuple(t.shape), t.dtype) for t in (q, k, v) if t is not None))
    f32 = torch.float32
    wt = f32 if (q_weight is not None and q_weight.dtype is f32 or
                 k_weight is not None and k_weight.dtype is f32) else dt
    pqw = _data("q_weight", q_weight, wt, (D,), dev) if q_weight is not None else None
    pkw = _data("k_weight", k_weight, wt, (D,), dev) if k_weight is not None else None
    rope = None
    if cos_sin is not None:
        max_pos, rot = _size("cos_sin", cos_sin, 2, 0), cos_sin.shape[1]
        pc = _data("cos_sin", cos_sin, f32, (max_pos, rot), dev)
        if rot > D or rot % 16:
            raise ValueError("cos_sin must be [max_pos, rot] with rot <= D and a multiple of 16, got %s"
                             % (tuple(cos_sin.shape),))
        if axes is None:
            n_axes, pa, pshape = 1, None, lead
        else:
            try:                       # value by value: bytes(array) would take an array's memory
                pa = bytes(list(axes))
            except (TypeError, ValueError) as e:
                raise ValueError("axes must be integers in [0, 4)") from e
            if len(pa) != rot // 2 or not isinstance(positions, torch.Tensor) or positions.dim() < 2:
                raise ValueError("axes must name the axis of each of the rot / 2 = %d pairs, positions be "
                                 "[n_axes, ...]" % (rot // 2))
            n_axes = positions.shape[0]
            if n_axes > 4 or (rot > 0 and max(pa) >= n_axes):
                raise ValueError("axes must lie in [0, n_axes = %d), at most four axes" % n_axes)
            pshape = (n_axes, *lead)
        pp = _data("positions", positions, torch.int32, pshape, dev)
        rope = _lib.Rope(pc, pp, max_pos, rot, 1 if interleaved else 0, n_axes, pa)
    elif positions is not None or axes is not None:
        raise ValueError("positions and axes need cos_sin")
    return dev, T, D, (pqw, pkw), 1 if wt is f32 else 0, ctypes.byref(rope) if rope is not None else None


def _rope_out(name, out, like):
    """`out` (checked) or a new contiguous tensor like `like`, and its address."""
    if out is None:
        out = torch.empty(like.shape, dtype=like.dtype, device=like.device)
        return out, out.data_ptr()
    return out, _data(name, out, like.dtype, like.shape, like.device)


def attn_qk_norm_rope(q, k, cos_sin, positions, q_weight=None, k_weight=None, eps=1e-6, interleaved=False, axes=None,
                      out=None):
    """RMS norm of each query and key head and rotation by position, in one pass.

    q [T, Hq, D] or [B, S, Hq, D], k likewise with Hkv heads: bfloat16 or
    float16 CUDA tensors, D 64, 128 or 256; slices of a fused projection are
    read in place (strides of multiples of 8), other layouts are copied first.
    cos_sin [max_pos, rot] float32: cosines of the rot / 2 pairs, then their
    sines (rope_table), or None for no rotation; positions int32 of q's leading
    shape.  A pair is dims (j, j + rot / 2), or (2j, 2j + 1) with interleaved; dims
    past rot pass through.  axes: the position axis of each pair (rot / 2 integers),
    positions then [n_axes, *leading] with up to four axes.
    q_weight / k_weight [D] (q's dtype, or both float32) or None for no norm of
    that side.  FP32 throughout, rounded once.
    out: (q_out, k_out), contiguous; q_out may be q and k_out k.
    Returns (q_out, k_out).
    """
    if not isinstance(k, torch.Tensor):
        raise ValueError("k must be a CUDA tensor")
    dev, T, D, (pqw, pkw), wf, rope = _rope_args(q, k, None, cos_sin, positions, q_weight, k_weight, interleaved,
                                                 axes)
    oq, pq = _rope_out("out q", out[0] if out is not None else None, q)
    ok, pk = _rope_out("out k", out[1] if out is not None else None, k)
    rq, _kq = _head_rows(q, T)
    rk, _kk = _head_rows(k, T)
    st = _on(dev, _lib.load().attn_qk_norm_rope, ctypes.byref(rq), ctypes.byref(rk), pqw, pkw, wf, eps, rope, pq, pk,
             T, q.shape[-2], k.shape[-2], D, _DTYPES[q.dtype], _raw_stream(dev))
    if st != 0:
        _raise(st, "attn_qk_norm_rope")
    return oq, ok


def attn_qk_norm_rope_paged(q, k, v, cos_sin, positions, slots, k_cache, v_cache, q_weight=None, k_weight=None,
                            eps=1e-6, interleaved=False, axes=None, k_scale=None, v_scale=None, requests=None,
                            out=None):
    """attn_qk_norm_rope with the keys, and the values as they are, written into
    paged caches.

    v like k; slots int32 of q's leading shape (attn_paged_slots): the cache row
    page * page_size + offset of each token; a token with a slot outside the
    pool is padding: its rows of the result and the caches stay as they were.
    k_cache / v_cache [num_pages, page_size, Hkv, D], contiguous, written in
    place: q's dtype, or torch.float8_e4m3fn (or uint8 codes).  For e4m3 caches,
    k_scale / v_scale [B, Hkv] float32 (or None: ones) divide what is stored,
    with requests (int32 like slots) naming each token's row of them.
    Other arguments as attn_qk_norm_rope.  Returns q_out.
    """
    if not isinstance(k, torch.Tensor) or not isinstance(v, torch.Tensor):
        raise ValueError("k and v must be CUDA tensors")
    dev, T, D, (pqw, pkw), wf, rope = _rope_args(q, k, v, cos_sin, positions, q_weight, k_weight, interleaved, axes)
    i32, f32, Hkv, lead = torch.int32, torch.float32, k.shape[-2], q.shape[:-2]
    num_pages, page_size = _size("k_cache", k_cache, 4, 0), k_cache.shape[1]
    ct = k_cache.dtype
    e4m3 = ct is torch.float8_e4m3fn or ct is torch.uint8
    shape = (num_pages, page_size, Hkv, D)
    pkc = _data("k_cache", k_cache, ct if e4m3 else q.dtype, shape, dev)
    pvc = _data("v_cache", v_cache, ct if e4m3 else q.dtype, shape, dev)
    ps = _data("slots", slots, i32, lead, dev)
    B, pks, pvs, pr = 0, None, None, None
    if k_scale is not None or v_scale is not None:
        if not e4m3:
            raise ValueError("k_scale and v_scale need float8_e4m3fn caches")
        B = _size("k_scale" if k_scale is not None else "v_scale", k_scale if k_scale is not None else v_scale, 2, 0)
        pks = _data("k_scale", k_scale, f32, (B, Hkv), dev) if k_scale is not None else None
        pvs = _data("v_scale", v_scale, f32, (B, Hkv), dev) if v_scale is not None else None
        pr = _data("requests", requests, i32, lead, dev)
    elif requests is not None:
        raise ValueError("requests needs k_scale or v_scale")
    oq, pq = _rope_out("out", out, q)
    rq, _kq = _head_rows(q, T)
    rk, _kk = _head_rows(k, T)
    rv, _kv = _head_rows(v, T)
    st = _on(dev, _lib.load().attn_qk_norm_rope_paged, ctypes.byref(rq), ctypes.byref(rk), ctypes.byref(rv), pqw, pkw,
             wf, eps, rope, pq, ps, pkc, pvc, 1 if e4m3 else 0, pks, pvs, pr, B, T, q.shape[-2], Hkv, D, num_pages,
             page_size, _DTYPES[q.dtype], _raw_stream(dev))
    if st != 0:
        _raise(st, "attn_qk_norm_rope_paged")
    return oq


def rope_table(max_pos, rot, base=10000.0, device="cuda"):
    """cos_sin [max_pos, rot] float32 of attn_qk_norm_rope with the angles
    p * base^(-2j / rot), formed in 64 bits."""
    if rot <= 0 or rot % 2:
        raise ValueError("rot must be positive and even, got %r" % (rot,))
    freq = float(base) ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))
    angle = torch.arange(max_pos, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float().to(device)


def attn_validate_paged(real_seqlen_kv, block_table, Sq, page_size, num_pages, causal=True):
    """Host-side range check of paged metadata (synchronises the stream)."""
    B, max_pages = block_table.shape
    st = _lib.load().attn_validate_paged(_ptr(real_seqlen_kv.contiguous()), _ptr(block_table.contiguous()), B, Sq,
                                         page_size, num_pages, max_pages, int(bool(causal)),
                                         _stream(block_table.device))
    if st != 0:
        _raise(st, "attn_validate_paged")


def gqa_device_error():
    """Raise if a kernel recorded a timed-out wait since the last check (synchronises)."""
    st = _lib.load().gqa_device_error()
    if st != 0:
        _raise(st, "gqa_device_error")


# Short aliases in the style of the pages' op APIs.
attention = attn_fwd_dense
decode_paged = attn_decode_paged
varlen = attn_fwd_varlen
paged = attn_fwd_paged
