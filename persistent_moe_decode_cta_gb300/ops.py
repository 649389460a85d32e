"""Operators over several tokens of each sequence, on the cache that the decode step reads.

They are what a program needs around the decode step to verify drafted tokens or to run
prompt chunks: append the new nodes' keys and values to the paged cache
(`qk_norm_rope`), attend over the cache and the draft tree (`tree_attention`), multiply by
the routed experts' matrices (`expert_product`), keep the accepted path
(`commit_nodes`) and copy pages for a fork (`copy_pages`); the projections and the LM head
(`linear`), the routed layer of a few tokens as a whole (`moe_layer`), and the decision which
drafted tokens are accepted (`verify_nodes`).  A *node* is a new token; node i
of sequence b owns cache position seq_lens[b] + i whatever its depth in the tree.

The functions check and marshal torch tensors for the entry points of include/mk.h, where
the operators are defined; a wrong tensor raises ValueError, a call that the library
refuses raises `binding.MkError`.  Like the library's calls they are asynchronous, on the
current stream of the tensors' device or on `stream` (a torch stream or a raw pointer), and
can be captured into a CUDA graph.  What a kernel finds wrong in device data (a page id, an
offset, or a wait of its own that ran out) goes to `status`, an int32[4] CUDA tensor from
`new_status`, or without one to the device's own record; `check_status` reads either.  None of
them has a backward pass.

Shapes: k_cache, v_cache bf16 [n_pages, n_kv_heads, 16, head_dim] (one layer) or
[n_layers, n_pages, n_kv_heads, 16, head_dim] (whole pools); page_table int32
[batch, max_pages]; seq_lens, counts int32 [batch]; positions int32 [batch, n].
"""
from __future__ import annotations

import ctypes
import functools
import inspect

import numpy as np
import torch

from . import binding as B

PAGE = 16
_I32 = torch.int32

_module = None


def _native():
    """The native half (csrc/ops_module.cpp), loaded on first use; its absence is an error."""
    global _module
    if _module is None:
        B.load_library()
        try:
            from . import _ops
        except ImportError as e:
            raise ImportError("_ops is missing: build it with `python -m persistent_moe_decode_cta_gb300.build`") from e
        _ops.setup(B._check)
        _module = _ops
    return _module


def _operator(fn):
    """Run fn with its first tensor's device current and, where `stream` is given, on that
    stream: what it allocates belongs to the stream, and the tensors that it is given are
    kept for it."""
    lead = next(iter(inspect.signature(fn).parameters))

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        first = args[0] if args else kw.get(lead)
        here = (_module or _native()).is_here(first)
        if here is None:
            raise ValueError(f"{lead} must be a CUDA tensor")
        if not here:
            with torch.cuda.device(first.get_device()):
                return call(*args, stream=stream, **kw)
        if stream is None:
            return fn(*args, **kw)
        s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), device=first.device)
        if s.device != first.device:
            raise ValueError(f"{lead} is on {first.device}, the stream on {s.device}")
        with torch.cuda.stream(s):
            out = fn(*args, **kw)
        for t in (*args, *kw.values()):
            if isinstance(t, torch.Tensor) and t.is_cuda:
                t.record_stream(s)
        return out
    return call


def new_status(device="cuda"):
    """An error record for `status` arguments: int32[4] zeros."""
    return torch.zeros(4, dtype=_I32, device=device)


def check_status(status=None):
    """Read and clear an error record (synchronising); raises MkError for a recorded error.
    None: the current device's own record, of all calls so far that were given no `status`."""
    if status is None:
        torch.cuda.synchronize()
        found = (ctypes.c_int32 * 4)()
        B._check(B.load_library().mk_op_status(found, torch.cuda.current_stream().cuda_stream))
        code, where, index, value = found
    else:
        code, where, index, value = status.tolist()
    if code:
        if status is not None:
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
    return _native().qk_norm_rope(q, k, v, k_cache, v_cache, page_table, seq_lens, theta, q_gain, k_gain, eps, positions,
                                  counts, out, status)


@_operator
def tree_attention(q, k_cache, v_cache, page_table, seq_lens, *, mask=None, positions=None, counts=None, window=0,
                   scale=None, out=None, status=None):
    """Attention of the nodes q [batch, n, n_q_heads, head_dim] (bf16, may be strided) over
    the cached positions and the nodes that `mask` shows them (int32 words, see `tree_mask`;
    None: node i sees the nodes 0..i), whose K/V `qk_norm_rope` has appended.  window > 0:
    only positions greater than positions[b, i] - window (default positions: seq_lens[b] +
    i).  scale defaults to head_dim ** -0.5.  A node that sees nothing gets zeros.  Returns
    `out` (not q); nodes from counts[b] on are left as they are."""
    return _native().tree_attention(q, k_cache, v_cache, page_table, seq_lens, mask, positions, counts, window, scale, out,
                                    status)


def _page_ids(ids, name):
    """A list of ints from what else names pages (a CPU tensor, an array)."""
    if type(ids) in (list, tuple):
        return ids
    if isinstance(ids, torch.Tensor):
        if ids.is_cuda:
            raise ValueError(f"{name} must be on the host")
        ids = ids.numpy()
    a = np.asarray(ids)
    if a.ndim != 1 or (a.size and a.dtype.kind not in "iu"):
        raise ValueError(f"{name} must be a list of page numbers")
    return a.tolist()


@_operator
def copy_pages(k_cache, v_cache, src, dst):
    """Copy pages src[i] -> dst[i] in every layer of the pools [n_layers, n_pages,
    n_kv_heads, 16, head_dim].  src and dst are host lists (or CPU arrays); no page is
    written twice, and none is both read and written."""
    _native().copy_pages(k_cache, v_cache, _page_ids(src, "src"), _page_ids(dst, "dst"))


@_operator
def commit_nodes(k_cache, v_cache, page_table, seq_lens, accepted, *, out=None, status=None):
    """Keep the accepted path of a draft: in every layer of the pools [n_layers, ..] the K/V
    of node accepted[b, i] (int32 [batch, max_accept], ended by a negative entry) moves to
    position seq_lens[b] + i.  Returns the new lengths, int32 [batch] (`out`, not
    seq_lens)."""
    return _native().commit_nodes(k_cache, v_cache, page_table, seq_lens, accepted, out, status)


@_operator
def expert_product(x, w, offsets, *, w_up=None, rows=None, out=None, status=None):
    """Products grouped by expert: rows offsets[e] .. offsets[e + 1] - 1 of the result are
    x[rows] @ w[e].T, or silu(x[rows] @ w[e].T) * (x[rows] @ w_up[e].T) with w_up.  x bf16
    [n_x, k] (rows may be strided), w and w_up bf16 [n_experts, n, k], offsets int32
    [n_experts + 1] ascending, rows int32 [n_rows] or None (row r of x).  Returns bf16
    [n_rows, n]; rows that belong to no expert are left as they are (uninitialised in a new
    result)."""
    return _native().expert_product(x, w, offsets, w_up, rows, out, status)


_ACTIVATIONS = {None: B.MK_ACT_NONE, "relu": B.MK_ACT_RELU, "silu": B.MK_ACT_SILU, "gelu": B.MK_ACT_GELU, "gelu_tanh": B.MK_ACT_GELU_TANH}
_WIDE = {None: None, torch.bfloat16: False, torch.float32: True}


@_operator
def linear(x, w, *, bias=None, activation=None, residual=None, dtype=None, out=None, status=None):
    """act(x @ w.T + bias) + residual.  x bf16 [m, k] and residual bf16 [m, n] (rows may be strided), w bf16 [n, k],
    bias bf16 [n]; activation None, "relu", "silu", "gelu" (erf) or "gelu_tanh".  Returns [m, n] of `dtype`, bf16
    (default) or float32 (an LM head's logits); `out` may be strided, and the residual itself."""
    if not isinstance(activation, (str, type(None))) or activation not in _ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(a for a in _ACTIVATIONS if a)} or None, not {activation!r}")
    if dtype not in _WIDE:
        raise ValueError(f"dtype must be torch.bfloat16 or torch.float32, not {dtype!r}")
    return _native().linear(x, w, bias, _ACTIVATIONS[activation], residual, out, _WIDE[dtype], status)


@_operator
def moe_layer(x, router, w_gate, w_up, w_down, top_k, *, residual=None, ids=None, weights=None, out=None, status=None):
    """The routed layer of up to 256 tokens as a whole: residual + sum over a token's top_k experts of its softmax weight
    times w_down[e] @ (silu(w_gate[e] @ x) * (w_up[e] @ x)).  x, residual bf16 [n, d_model] (rows may be strided), router bf16
    [n_experts, d_model], w_gate and w_up bf16 [n_experts, d_ff, d_model], w_down bf16 [n_experts, d_model, d_ff].  The
    selection goes to `ids` and `weights` (int32, float32 [n, top_k], largest score first) where given.  Returns bf16
    [n, d_model]; `out` may be the residual itself."""
    return _native().moe_layer(x, router, w_gate, w_up, w_down, top_k, residual, ids, weights, out, status)


@_operator
def verify_nodes(logits, tokens, uniforms, *, parents=None, draft_probs=None, temperature=None, counts=None, accepted=None,
                 next_tokens=None, status=None):
    """Which drafted nodes the target model accepts, and its next token: (accepted, next_tokens).  Node 0 of a sequence is its
    last sampled token, the others a tree of drafted tokens (parents[b, i] < i; None: a chain).  logits [batch, n, vocab] (bf16
    or float32, last dimension contiguous) are the target's for the token after each node, draft_probs float32 [batch, n, vocab]
    what each node's children were drawn from (None: they were not drawn, but proposed), uniforms float32 [batch, n] random
    numbers in [0, 1): entry i decides on node i, entry 0 draws the next token.  temperature float32 [batch] (None: 1; 0: the
    largest logit).  accepted int32 [batch, n] holds the path from node 0, ended by -1, as `commit_nodes` takes it;
    next_tokens int32 [batch]."""
    return _native().verify_nodes(logits, tokens, uniforms, parents, draft_probs, temperature, counts, accepted, next_tokens, status)
