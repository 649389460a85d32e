"""Operators over several tokens of each sequence, on the cache that the decode step reads.

They are what a program needs around the decode step to verify drafted tokens or to run
prompt chunks: append the new nodes' keys and values to the paged cache
(`qk_norm_rope`), attend over the cache and the draft tree (`tree_attention`), multiply by
the routed experts' matrices (`expert_product`), keep the accepted path
(`commit_nodes`) and copy pages for a fork (`copy_pages`).  A *node* is a new token; node i
of sequence b owns cache position seq_lens[b] + i whatever its depth in the tree.

The functions check and marshal torch tensors for the entry points of include/mk.h, where
the operators are defined; a wrong tensor raises ValueError, a call that the library
refuses raises `binding.MkError`.  Like the library's calls they are asynchronous, on the
current stream of the tensors' device or on `stream` (a torch stream or a raw pointer), and
can be captured into a CUDA graph.  What a kernel finds wrong in device data (a page id, an
offset) goes to `status`, an int32[4] CUDA tensor from `new_status`, if one is given;
`check_status` reads it.  None of them has a backward pass.

Shapes: k_cache, v_cache bf16 [n_pages, n_kv_heads, 16, head_dim] (one layer) or
[n_layers, n_pages, n_kv_heads, 16, head_dim] (whole pools); page_table int32
[batch, max_pages]; seq_lens, counts int32 [batch]; positions int32 [batch, n].
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import inspect

import numpy as np

from . import binding as B

PAGE = 16


def _torch():
    import torch
    return torch


def _dtype(name):
    return getattr(_torch(), name)


def _need(t, name, dtype, shape, device=None, contiguous=True):
    """t is a CUDA tensor of this dtype and shape (None: any size), on `device` if given."""
    if not isinstance(t, _torch().Tensor):
        raise ValueError(f"{name} must be a tensor, not {type(t).__name__}")
    if not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name} must be a CUDA tensor" + (f" on {device}" if device is not None else ""))
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.dim() != len(shape) or any(w is not None and w != n for w, n in zip(shape, t.shape)):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, needs {tuple('any' if w is None else w for w in shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.requires_grad and _torch().is_grad_enabled():
        raise ValueError(f"{name} requires a gradient, and this operator has no backward pass")
    return t


def _optional(t, name, dtype, shape, device):
    return None if t is None else _need(t, name, dtype, shape, device).data_ptr()


def _operator(fn):
    """Run fn with its first tensor's device current and, where `stream` is given, on that
    stream: what it allocates belongs to the stream, and the tensors that it is given are
    kept for it."""
    lead = next(iter(inspect.signature(fn).parameters))

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        torch = _torch()
        first = args[0] if args else kw.get(lead)
        if not isinstance(first, torch.Tensor) or not first.is_cuda:
            raise ValueError(f"{lead} must be a CUDA tensor")
        dev = first.device
        with contextlib.ExitStack() as ctx:
            if dev.index != torch.cuda.current_device():
                ctx.enter_context(torch.cuda.device(dev))
            if stream is None:
                return fn(*args, **kw)
            s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), device=dev)
            ctx.enter_context(torch.cuda.stream(s))
            out = fn(*args, **kw)
            for t in (*args, *kw.values()):
                if isinstance(t, torch.Tensor) and t.is_cuda:
                    t.record_stream(s)
            return out
    return call


def _stream(device):
    return _torch().cuda.current_stream(device).cuda_stream


def _kv(k_cache, v_cache, page_table, seq_lens, device, pools=False):
    """(mk_paged_kv, batch, n_kv_heads, head_dim)."""
    lead = (None,) if pools else ()
    bf16, i32 = _dtype("bfloat16"), _dtype("int32")
    _need(k_cache, "k_cache", bf16, (*lead, None, None, PAGE, None), device)
    _need(v_cache, "v_cache", bf16, k_cache.shape, device)
    _need(page_table, "page_table", i32, (None, None), device)
    b, pages = page_table.shape
    _need(seq_lens, "seq_lens", i32, (b,), device)
    n_pages, hkv, _, hd = k_cache.shape[-4:]
    return B.mk_paged_kv(k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(), seq_lens.data_ptr(),
                         n_pages, hkv, hd, b, pages), b, hkv, hd


def _rows(t, name, shape, device):
    """(pointer, strides) of a [batch, n, heads, head_dim] operand."""
    _need(t, name, _dtype("bfloat16"), shape, device, contiguous=False)
    st = t.stride()
    if st[3] != 1 and shape[3] != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return t.data_ptr(), B._S3(*st[:3])


def new_status(device="cuda"):
    """An error record for `status` arguments: int32[4] zeros."""
    torch = _torch()
    return torch.zeros(4, dtype=torch.int32, device=device)


def check_status(status):
    """Read and clear an error record (synchronising); raises MkError for a recorded error."""
    code, where, index, value = status.tolist()
    if code:
        status.zero_()
        raise B.MkError(code, f"recorded by a kernel: sequence, expert or CTA {where}, index {index}, value {value}")


def tree_mask(parents):
    """(mask, depths) of draft trees: parents int32 [batch, n] holds each node's parent node,
    -1 for a root.  mask int32 [batch, n, ceil(n / 32)] shows every node its ancestors and
    itself (the argument of `tree_attention`); depths int32 [batch, n] is the number of its
    ancestors, so seq_lens[:, None] + depths are the positions.  Plain torch, any device."""
    torch = _torch()
    if parents.dim() != 2 or parents.dtype != torch.int32:
        raise ValueError("parents must be int32 [batch, n]")
    b, n = parents.shape
    node = torch.arange(n, device=parents.device)
    up = (parents[:, :, None] == node) | torch.eye(n, dtype=torch.bool, device=parents.device)
    for _ in range(max(1, (n - 1).bit_length())):  # ancestors at distance up to 2, 4, 8, ..
        up = (up.float() @ up.float()) > 0
    depths = (up.sum(-1) - 1).to(torch.int32)
    words = -(-n // 32)
    bits = torch.zeros(b, n, words * 32, dtype=torch.int64, device=parents.device)
    bits[:, :, :n] = up
    w = (bits.view(b, n, words, 32) << torch.arange(32, device=parents.device)).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32), depths


@_operator
def qk_norm_rope(q, k, v, k_cache, v_cache, page_table, seq_lens, *, theta, q_gain=None, k_gain=None, eps=1e-6,
                 positions=None, counts=None, out=None, status=None):
    """Norm every head of q and k (RMS over the head times its gain; no norm without a gain),
    rotate them to their positions (default seq_lens[b] + i) and append k and v to the
    cache.  q [batch, n, n_q_heads, head_dim], k and v [batch, n, n_kv_heads, head_dim] bf16
    may be strided views of one projection's result.  Returns the rotated q (`out`, which
    may be q).  Nodes from counts[b] on are left as they are."""
    dev = q.device
    kv, b, hkv, hd = _kv(k_cache, v_cache, page_table, seq_lens, dev)
    bf16, i32 = _dtype("bfloat16"), _dtype("int32")
    shape = (b, None, None, hd)
    qp, qs = _rows(q, "q", shape, dev)
    n, hq = q.shape[1:3]
    kp, ks = _rows(k, "k", (b, n, hkv, hd), dev)
    vp, vs = _rows(v, "v", (b, n, hkv, hd), dev)
    if out is None:
        # rows that the kernel leaves alone would be uninitialised memory
        out = _torch().empty(b, n, hq, hd, dtype=bf16, device=dev) if counts is None else \
            _torch().zeros(b, n, hq, hd, dtype=bf16, device=dev)
    op, os_ = _rows(out, "out", (b, n, hq, hd), dev)
    if n == 0 or b == 0:
        return out
    a = B.mk_rope_args(qp, kp, vp, op, qs, ks, vs, os_, _optional(q_gain, "q_gain", bf16, (hd,), dev),
                       _optional(k_gain, "k_gain", bf16, (hd,), dev), _optional(positions, "positions", i32, (b, n), dev),
                       _optional(counts, "counts", i32, (b,), dev), _optional(status, "status", i32, (4,), dev), n, hq,
                       float(eps), float(theta))
    B._check(B.load_library().mk_qk_norm_rope(ctypes.byref(kv), ctypes.byref(a), _stream(dev)))
    return out


@_operator
def tree_attention(q, k_cache, v_cache, page_table, seq_lens, *, mask=None, positions=None, counts=None, window=0,
                   scale=None, out=None, status=None):
    """Attention of the nodes q [batch, n, n_q_heads, head_dim] (bf16, may be strided) over
    the cached positions and the nodes that `mask` shows them (int32 words, see `tree_mask`;
    None: node i sees the nodes 0..i), whose K/V `qk_norm_rope` has appended.  window > 0:
    only positions greater than positions[b, i] - window (default positions: seq_lens[b] +
    i).  scale defaults to head_dim ** -0.5.  A node that sees nothing gets zeros.  Returns
    `out` (not q); nodes from counts[b] on are left as they are."""
    dev = q.device
    kv, b, _, hd = _kv(k_cache, v_cache, page_table, seq_lens, dev)
    i32 = _dtype("int32")
    qp, qs = _rows(q, "q", (b, None, None, hd), dev)
    n, hq = q.shape[1:3]
    if out is None:
        out = _torch().empty(b, n, hq, hd, dtype=q.dtype, device=dev) if counts is None else \
            _torch().zeros(b, n, hq, hd, dtype=q.dtype, device=dev)
    op, os_ = _rows(out, "out", (b, n, hq, hd), dev)
    if n == 0 or b == 0:
        return out
    a = B.mk_tree_args(qp, op, qs, os_, _optional(mask, "mask", i32, (b, n, -(-n // 32)), dev),
                       _optional(positions, "positions", i32, (b, n), dev), _optional(counts, "counts", i32, (b,), dev),
                       _optional(status, "status", i32, (4,), dev), n, hq, int(window), hd ** -0.5 if scale is None else float(scale))
    lib = B.load_library()
    need = ctypes.c_size_t()
    B._check(lib.mk_tree_attention_workspace(ctypes.byref(kv), ctypes.byref(a), ctypes.byref(need)))
    work = _torch().empty(need.value, dtype=_dtype("uint8"), device=dev)
    a.workspace, a.workspace_bytes = work.data_ptr(), need.value
    B._check(lib.mk_tree_attention(ctypes.byref(kv), ctypes.byref(a), _stream(dev)))
    return out


def _page_ids(ids, name):
    if isinstance(ids, _torch().Tensor):
        if ids.is_cuda:
            raise ValueError(f"{name} must be on the host")
        ids = ids.numpy()
    a = np.asarray(ids)
    if a.size == 0:
        a = a.astype(np.int32)
    if a.ndim != 1 or a.dtype.kind not in "iu":
        raise ValueError(f"{name} must be a list of page numbers")
    a32 = np.ascontiguousarray(a, dtype=np.int32)
    if a32 is not a and not np.array_equal(a32, a):
        raise ValueError(f"{name}: a page number does not fit 32 bits")
    return a32


@_operator
def copy_pages(k_cache, v_cache, src, dst):
    """Copy pages src[i] -> dst[i] in every layer of the pools [n_layers, n_pages,
    n_kv_heads, 16, head_dim].  src and dst are host lists (or CPU arrays); no page is
    written twice, and none is both read and written."""
    dev = k_cache.device
    bf16 = _dtype("bfloat16")
    _need(k_cache, "k_cache", bf16, (None, None, None, PAGE, None), dev)
    _need(v_cache, "v_cache", bf16, k_cache.shape, dev)
    s, d = _page_ids(src, "src"), _page_ids(dst, "dst")
    if s.size != d.size:
        raise ValueError(f"{s.size} source pages, {d.size} destination pages")
    n_layers, n_pages, hkv, _, hd = k_cache.shape
    B._check(B.load_library().mk_copy_pages(k_cache.data_ptr(), v_cache.data_ptr(), n_layers, n_pages, hkv, hd,
                                            s.ctypes.data, d.ctypes.data, s.size, _stream(dev)))


@_operator
def commit_nodes(k_cache, v_cache, page_table, seq_lens, accepted, *, out=None, status=None):
    """Keep the accepted path of a draft: in every layer of the pools [n_layers, ..] the K/V
    of node accepted[b, i] (int32 [batch, max_accept], ended by a negative entry) moves to
    position seq_lens[b] + i.  Returns the new lengths, int32 [batch] (`out`, not
    seq_lens)."""
    dev = k_cache.device
    i32 = _dtype("int32")
    kv, b, _, _ = _kv(k_cache, v_cache, page_table, seq_lens, dev, pools=True)
    _need(accepted, "accepted", i32, (b, None), dev)
    if out is None:
        out = _torch().empty(b, dtype=i32, device=dev)
    _need(out, "out", i32, (b,), dev)
    B._check(B.load_library().mk_commit_nodes(ctypes.byref(kv), k_cache.shape[0], accepted.data_ptr(), accepted.shape[1],
                                              out.data_ptr(), _optional(status, "status", i32, (4,), dev), _stream(dev)))
    return out


@_operator
def expert_product(x, w, offsets, *, w_up=None, rows=None, out=None, status=None):
    """Products grouped by expert: rows offsets[e] .. offsets[e + 1] - 1 of the result are
    x[rows] @ w[e].T, or silu(x[rows] @ w[e].T) * (x[rows] @ w_up[e].T) with w_up.  x bf16
    [n_x, k] (rows may be strided), w and w_up bf16 [n_experts, n, k], offsets int32
    [n_experts + 1] ascending, rows int32 [n_rows] or None (row r of x).  Returns bf16
    [n_rows, n]; rows that belong to no expert are left as they are (uninitialised in a new
    result)."""
    dev = x.device
    torch = _torch()
    bf16, i32 = _dtype("bfloat16"), _dtype("int32")
    _need(w, "w", bf16, (None, None, None), dev)
    e, n, k = w.shape
    _need(x, "x", bf16, (None, k), dev, contiguous=False)
    if x.stride(1) != 1 and k != 1:
        raise ValueError("x: the last dimension must be contiguous")
    _need(offsets, "offsets", i32, (e + 1,), dev)
    n_x = x.shape[0]
    n_rows = n_x
    if rows is not None:
        n_rows = _need(rows, "rows", i32, (None,), dev).shape[0]
    if out is None:
        out = torch.empty(n_rows, n, dtype=bf16, device=dev)
    _need(out, "out", bf16, (n_rows, n), dev, contiguous=False)
    if out.stride(1) != 1 and n != 1:
        raise ValueError("out: the last dimension must be contiguous")
    if n_rows == 0:
        return out
    a = B.mk_expert_args(x.data_ptr(), w.data_ptr(), _optional(w_up, "w_up", bf16, (e, n, k), dev), offsets.data_ptr(),
                         None if rows is None else rows.data_ptr(), out.data_ptr(), _optional(status, "status", i32, (4,), dev),
                         x.stride(0) if n_x > 1 else k, out.stride(0) if n_rows > 1 else n, n_x, n_rows, e, n, k)
    B._check(B.load_library().mk_expert_product(ctypes.byref(a), _stream(dev)))
    return out
