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

import ctypes
import functools
import inspect
import struct

import numpy as np
import torch

from . import binding as B

PAGE = 16
_BF16, _I32 = torch.bfloat16, torch.int32

# The argument structs of include/mk.h as packed bytes: a call at batch 1 runs for a few
# microseconds, and filling a ctypes.Structure field by field takes about as long.
_KV = struct.Struct("@4P5i4x")
_ROPE = struct.Struct("@4P12q5P2ifd")
_TREE = struct.Struct("@2P6q4P3if1P1N")
_EXPERT = struct.Struct("@7P2q5i4x")


def _need(t, name, dtype, shape, dev):
    """The address of t, a contiguous CUDA tensor of this dtype and shape on device `dev`."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev and t.shape == shape
            and t.is_contiguous() and not t.requires_grad):
        return t.data_ptr()
    return _refuse(t, name, dtype, shape, dev, True)


def _rows(t, name, shape, dev):
    """(address, strides) of a bf16 operand whose last dimension is contiguous."""
    if isinstance(t, torch.Tensor) and t.dtype is _BF16 and t.get_device() == dev and t.shape == shape and not t.requires_grad:
        st = t.stride()
        if st[-1] == 1 or shape[-1] == 1:
            return t.data_ptr(), st
    _refuse(t, name, _BF16, shape, dev, False)
    return t.data_ptr(), t.stride()


def _refuse(t, name, dtype, shape, dev, contiguous):
    """Say what is wrong with t (or return its address: it may require a gradient where none
    is recorded)."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor, not {type(t).__name__}")
    if t.get_device() != dev or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor on device {dev}, not on {t.device}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, needs {tuple(shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not contiguous and t.stride(-1) != 1 and shape[-1] != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires a gradient, and this operator has no backward pass")
    return t.data_ptr()


def _shape(t, name, dims):
    """The shape of t, a tensor of `dims` dimensions."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor, not {type(t).__name__}")
    if t.dim() != dims:
        raise ValueError(f"{name} has {t.dim()} dimensions, needs {dims}")
    return t.shape


def _operator(fn):
    """Run fn with its first tensor's device current and, where `stream` is given, on that
    stream: what it allocates belongs to the stream, and the tensors that it is given are
    kept for it."""
    lead = next(iter(inspect.signature(fn).parameters))

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        first = args[0] if args else kw.get(lead)
        if not isinstance(first, torch.Tensor) or not first.is_cuda:
            raise ValueError(f"{lead} must be a CUDA tensor")
        dev = first.get_device()
        if dev != torch.cuda.current_device():
            with torch.cuda.device(dev):
                return call(*args, stream=stream, **kw)
        if stream is None:
            return fn(*args, **kw)
        s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), device=first.device)
        with torch.cuda.stream(s):
            out = fn(*args, **kw)
        for t in (*args, *kw.values()):
            if isinstance(t, torch.Tensor) and t.is_cuda:
                t.record_stream(s)
        return out
    return call


def _stream(dev):
    # (a Stream object takes longer than the rest of a call's checks)
    return torch._C._cuda_getCurrentRawStream(dev)


def _kv(k_cache, v_cache, page_table, seq_lens, dev, dims):
    """(mk_paged_kv as bytes, batch, n_kv_heads, head_dim, max_pages); the pools have `dims`
    dimensions."""
    shape = _shape(k_cache, "k_cache", dims)
    n_pages, hkv, page, hd = shape[-4:]
    if page != PAGE:
        raise ValueError(f"k_cache has pages of {page} tokens, needs {PAGE}")
    b, pages = _shape(page_table, "page_table", 2)
    return _KV.pack(_need(k_cache, "k_cache", _BF16, shape, dev), _need(v_cache, "v_cache", _BF16, shape, dev),
                    _need(page_table, "page_table", _I32, (b, pages), dev), _need(seq_lens, "seq_lens", _I32, (b,), dev),
                    n_pages, hkv, hd, b, pages), b, hkv, hd, pages


def new_status(device="cuda"):
    """An error record for `status` arguments: int32[4] zeros."""
    return torch.zeros(4, dtype=_I32, device=device)


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
    dev = q.get_device()
    kv, b, hkv, hd, _ = _kv(k_cache, v_cache, page_table, seq_lens, dev, 4)
    _, n, hq, _ = _shape(q, "q", 4)
    shape, kshape = (b, n, hq, hd), (b, n, hkv, hd)
    qp, qs = _rows(q, "q", shape, dev)
    kp, ks = _rows(k, "k", kshape, dev)
    vp, vs = _rows(v, "v", kshape, dev)
    if out is None:
        # (nodes that the kernel leaves alone would be uninitialised memory)
        out = (torch.empty if counts is None else torch.zeros)(shape, dtype=_BF16, device=q.device)
    op, os_ = _rows(out, "out", shape, dev)
    if n == 0 or b == 0:
        return out
    args = _ROPE.pack(qp, kp, vp, op, *qs[:3], *ks[:3], *vs[:3], *os_[:3],
                      0 if q_gain is None else _need(q_gain, "q_gain", _BF16, (hd,), dev),
                      0 if k_gain is None else _need(k_gain, "k_gain", _BF16, (hd,), dev),
                      0 if positions is None else _need(positions, "positions", _I32, (b, n), dev),
                      0 if counts is None else _need(counts, "counts", _I32, (b,), dev),
                      0 if status is None else _need(status, "status", _I32, (4,), dev), n, hq, float(eps), float(theta))
    B._check(B.load_library().mk_qk_norm_rope(kv, args, _stream(dev)))
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
    dev = q.get_device()
    kv, b, hkv, hd, pages = _kv(k_cache, v_cache, page_table, seq_lens, dev, 4)
    _, n, hq, _ = _shape(q, "q", 4)
    shape = (b, n, hq, hd)
    qp, qs = _rows(q, "q", shape, dev)
    if out is None:
        out = (torch.empty if counts is None else torch.zeros)(shape, dtype=_BF16, device=q.device)
    op, os_ = _rows(out, "out", shape, dev)
    if n == 0 or b == 0:
        return out
    if not 0 <= window < 1 << 31:
        raise ValueError(f"window {window} is not in [0, 2^31)")
    need = _tree_workspace(dev, hkv, hd, b, pages, n, hq)
    work = torch.empty(need, dtype=torch.uint8, device=q.device)
    args = _TREE.pack(qp, op, *qs[:3], *os_[:3], 0 if mask is None else _need(mask, "mask", _I32, (b, n, -(-n // 32)), dev),
                      0 if positions is None else _need(positions, "positions", _I32, (b, n), dev),
                      0 if counts is None else _need(counts, "counts", _I32, (b,), dev),
                      0 if status is None else _need(status, "status", _I32, (4,), dev), n, hq, int(window),
                      hd ** -0.5 if scale is None else float(scale), work.data_ptr(), need)
    B._check(B.load_library().mk_tree_attention(kv, args, _stream(dev)))
    return out


@functools.lru_cache(maxsize=256)
def _tree_workspace(dev, hkv, hd, b, pages, n, hq):
    """Bytes of workspace for these sizes on device `dev` (the current one)."""
    need = ctypes.c_size_t()
    B._check(B.load_library().mk_tree_attention_workspace(_KV.pack(0, 0, 0, 0, 1, hkv, hd, b, pages),
                                                          _TREE.pack(*[0] * 12, n, hq, 0, 1.0, 0, 0), ctypes.byref(need)))
    return need.value


def _page_ids(ids, name):
    if isinstance(ids, torch.Tensor):
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
    dev = k_cache.get_device()
    shape = _shape(k_cache, "k_cache", 5)
    n_layers, n_pages, hkv, page, hd = shape
    if page != PAGE:
        raise ValueError(f"k_cache has pages of {page} tokens, needs {PAGE}")
    kp, vp = _need(k_cache, "k_cache", _BF16, shape, dev), _need(v_cache, "v_cache", _BF16, shape, dev)
    s, d = _page_ids(src, "src"), _page_ids(dst, "dst")
    if s.size != d.size:
        raise ValueError(f"{s.size} source pages, {d.size} destination pages")
    B._check(B.load_library().mk_copy_pages(kp, vp, n_layers, n_pages, hkv, hd, s.ctypes.data, d.ctypes.data, s.size, _stream(dev)))


@_operator
def commit_nodes(k_cache, v_cache, page_table, seq_lens, accepted, *, out=None, status=None):
    """Keep the accepted path of a draft: in every layer of the pools [n_layers, ..] the K/V
    of node accepted[b, i] (int32 [batch, max_accept], ended by a negative entry) moves to
    position seq_lens[b] + i.  Returns the new lengths, int32 [batch] (`out`, not
    seq_lens)."""
    dev = k_cache.get_device()
    kv, b, *_ = _kv(k_cache, v_cache, page_table, seq_lens, dev, 5)
    accept = _shape(accepted, "accepted", 2)[1]
    if out is None:
        out = torch.empty(b, dtype=_I32, device=k_cache.device)
    B._check(B.load_library().mk_commit_nodes(kv, k_cache.shape[0], _need(accepted, "accepted", _I32, (b, accept), dev), accept,
                                              _need(out, "out", _I32, (b,), dev),
                                              0 if status is None else _need(status, "status", _I32, (4,), dev), _stream(dev)))
    return out


@_operator
def expert_product(x, w, offsets, *, w_up=None, rows=None, out=None, status=None):
    """Products grouped by expert: rows offsets[e] .. offsets[e + 1] - 1 of the result are
    x[rows] @ w[e].T, or silu(x[rows] @ w[e].T) * (x[rows] @ w_up[e].T) with w_up.  x bf16
    [n_x, k] (rows may be strided), w and w_up bf16 [n_experts, n, k], offsets int32
    [n_experts + 1] ascending, rows int32 [n_rows] or None (row r of x).  Returns bf16
    [n_rows, n]; rows that belong to no expert are left as they are (uninitialised in a new
    result)."""
    dev = x.get_device()
    e, n, k = _shape(w, "w", 3)
    n_x = n_rows = _shape(x, "x", 2)[0]
    xp, xs = _rows(x, "x", (n_x, k), dev)
    if rows is not None:
        n_rows = _shape(rows, "rows", 1)[0]
    if out is None:
        out = torch.empty(n_rows, n, dtype=_BF16, device=x.device)
    op, os_ = _rows(out, "out", (n_rows, n), dev)
    if n_rows == 0:
        return out
    args = _EXPERT.pack(xp, _need(w, "w", _BF16, (e, n, k), dev), 0 if w_up is None else _need(w_up, "w_up", _BF16, (e, n, k), dev),
                        _need(offsets, "offsets", _I32, (e + 1,), dev), 0 if rows is None else _need(rows, "rows", _I32, (n_rows,), dev),
                        op, 0 if status is None else _need(status, "status", _I32, (4,), dev),
                        xs[0] if n_x > 1 else k, os_[0] if n_rows > 1 else n, n_x, n_rows, e, n, k)
    B._check(B.load_library().mk_expert_product(args, _stream(dev)))
    return out
