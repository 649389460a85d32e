"""Calls that the multi-token operators refuse before anything is launched: the C entry
points look at sizes, strides, alignment and host arrays first, so this needs no GPU (the
device pointers are made up and never followed)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from persistent_moe_decode_cta_gb300 import binding as B
from persistent_moe_decode_cta_gb300 import ops

P = 1 << 20          # a made-up, aligned device address
INV, UNS, BAD = B.MK_ERR_INVALID, B.MK_ERR_UNSUPPORTED, B.MK_ERR_BAD_PAGE


def kv(**over):
    a = dict(k=P, v=P, page_table=P, seq_lens=P, n_pages=10, n_kv_heads=2, head_dim=64, batch=2, max_pages=4)
    a.update(over)
    return B.mk_paged_kv(**a)


def rope(**over):
    s = B._S3
    a = dict(q=P, k=P, v=P, q_out=P, q_stride=s(1024, 512, 64), k_stride=s(512, 128, 64), v_stride=s(512, 128, 64),
             out_stride=s(1024, 512, 64), n_nodes=2, n_q_heads=8, eps=1e-6, theta=1e4)
    a.update(over)
    return B.mk_rope_args(**a)


def tree(**over):
    s = B._S3
    a = dict(q=P, out=2 * P, q_stride=s(1024, 512, 64), out_stride=s(1024, 512, 64), n_nodes=2, n_q_heads=8, window=0, scale=0.125,
             workspace=P, workspace_bytes=1 << 40)
    a.update(over)
    return B.mk_tree_args(**a)


def experts(**over):
    a = dict(x=P, w=P, offsets=P, out=2 * P, x_stride=64, out_stride=32, n_x=8, n_rows=8, n_experts=4, n=32, k=64)
    a.update(over)
    return B.mk_expert_args(**a)


CACHE = [(dict(head_dim=48), UNS), (dict(head_dim=256), UNS), (dict(batch=0), INV), (dict(batch=65536), INV), (dict(n_kv_heads=0), INV),
         (dict(max_pages=0), INV), (dict(n_pages=0), INV), (dict(n_pages=1 << 27), INV), (dict(k=None), INV), (dict(v=P + 8), INV),
         (dict(page_table=None), INV), (dict(seq_lens=None), INV)]


@pytest.mark.parametrize("over,code", CACHE)
def test_cache_arguments(over, code):
    lib = B.load_library()
    c = kv(**over)
    assert lib.mk_qk_norm_rope(ctypes.byref(c), ctypes.byref(rope()), None) == code
    assert lib.mk_tree_attention(ctypes.byref(c), ctypes.byref(tree()), None) == code
    assert lib.mk_commit_nodes(ctypes.byref(c), 2, P, 4, 2 * P, None, None) == code
    assert lib.mk_last_error(None)


@pytest.mark.parametrize("over,code", [
    (dict(q=None), INV), (dict(k=P + 2), INV), (dict(v=None), INV), (dict(q_out=P + 8), INV), (dict(n_nodes=0), INV),
    (dict(n_q_heads=7), INV), (dict(n_q_heads=0), INV), (dict(q_stride=B._S3(1024, 508, 64)), INV),
    (dict(k_stride=B._S3(512, 0, 64)), INV), (dict(out_stride=B._S3(-1024, 512, 64)), INV), (dict(q_gain=P + 2), INV),
    (dict(k_gain=P + 4), INV), (dict(theta=0.5), INV), (dict(theta=math.nan), INV), (dict(theta=math.inf), INV),
    (dict(eps=-1e-6), INV), (dict(eps=math.nan), INV), (dict(eps=math.inf), INV)])
def test_rope_arguments(over, code):
    assert B.load_library().mk_qk_norm_rope(ctypes.byref(kv()), ctypes.byref(rope(**over)), None) == code


@pytest.mark.parametrize("over,code", [
    (dict(q=None), INV), (dict(out=None), INV), (dict(out=P), INV), (dict(q=P + 2), INV), (dict(n_nodes=0), INV),
    (dict(n_nodes=1 << 30), INV), (dict(n_q_heads=9), INV), (dict(n_q_heads=2 * 129), UNS), (dict(window=-1), INV),
    (dict(scale=-0.1), INV), (dict(scale=3e38), INV), (dict(scale=math.nan), INV), (dict(scale=math.inf), INV), (dict(workspace=None), INV),
    (dict(workspace=P + 8), INV), (dict(q_stride=B._S3(1024, 512, 60)), INV), (dict(out_stride=B._S3(1024, 0, 64)), INV)])
def test_tree_arguments(over, code):
    a = tree(**over)
    assert B.load_library().mk_tree_attention(ctypes.byref(kv()), ctypes.byref(a), None) == code


def test_tree_work_is_bounded():
    c, a = kv(batch=128, max_pages=1 << 26, n_kv_heads=2), tree(n_nodes=1 << 20)
    n = ctypes.c_size_t()
    assert B.load_library().mk_tree_attention_workspace(ctypes.byref(c), ctypes.byref(a), ctypes.byref(n)) == UNS
    assert B.load_library().mk_tree_attention_workspace(ctypes.byref(c), ctypes.byref(a), None) == INV
    c, a = kv(batch=100), tree(n_nodes=1 << 16)                 # 102400 groups of 64 nodes
    assert B.load_library().mk_tree_attention_workspace(ctypes.byref(c), ctypes.byref(a), ctypes.byref(n)) == UNS


@pytest.mark.parametrize("over,code", [
    (dict(x=None), INV), (dict(w=None), INV), (dict(offsets=None), INV), (dict(out=None), INV), (dict(out=P), INV), (dict(x=P + 8), INV),
    (dict(w=P + 8), INV), (dict(w_up=P + 8), INV), (dict(n_experts=0), INV), (dict(n_experts=257), INV), (dict(n=0), INV),
    (dict(k=0), UNS), (dict(k=60), UNS), (dict(n_rows=-1), INV), (dict(n_x=7), INV), (dict(n_x=0, rows=P), INV),
    (dict(x_stride=56), INV), (dict(x_stride=68), INV), (dict(out_stride=31), INV)])
def test_expert_arguments(over, code):
    assert B.load_library().mk_expert_product(ctypes.byref(experts(**over)), None) == code


def test_no_rows_is_no_work():
    assert B.load_library().mk_expert_product(ctypes.byref(experts(n_rows=0)), None) == B.MK_OK


@pytest.mark.parametrize("src,dst,code", [([0, 1], [2, 2], INV), ([0, 1], [1, 2], INV), ([3], [3], INV), ([8], [0], BAD),
                                          ([0], [-1], BAD), ([-1], [0], BAD), ([0] * 9, list(range(1, 10)), INV)])
def test_page_lists(src, dst, code):
    s, d = np.array(src, np.int32), np.array(dst, np.int32)
    lib = B.load_library()
    assert lib.mk_copy_pages(P, P, 2, 8, 2, 32, s.ctypes.data, d.ctypes.data, len(s), None) == code
    assert lib.mk_copy_pages(P, P, 2, 8, 2, 32, None, None, 0, None) == B.MK_OK
    assert lib.mk_copy_pages(P, P, 2, 8, 2, 32, None, None, 1, None) == INV
    assert lib.mk_copy_pages(P, P, 0, 8, 2, 32, None, None, 1, None) == INV
    assert lib.mk_copy_pages(P + 8, P, 1, 8, 2, 32, None, None, 1, None) == INV
    assert lib.mk_copy_pages(P, None, 1, 8, 2, 32, None, None, 1, None) == INV


@pytest.mark.parametrize("n_layers,max_accept,new_lens,accepted", [(0, 4, 2 * P, P), (2, 0, 2 * P, P), (2, 513, 2 * P, P), (2, 4, P, P),
                                                                   (2, 4, None, P), (2, 4, 2 * P, None)])
def test_commit_arguments(n_layers, max_accept, new_lens, accepted):
    assert B.load_library().mk_commit_nodes(ctypes.byref(kv()), n_layers, accepted, max_accept, new_lens, None, None) == INV


def test_null_structs():
    lib = B.load_library()
    assert lib.mk_qk_norm_rope(None, ctypes.byref(rope()), None) == INV
    assert lib.mk_qk_norm_rope(ctypes.byref(kv()), None, None) == INV
    assert lib.mk_tree_attention(None, ctypes.byref(tree()), None) == INV
    assert lib.mk_tree_attention(ctypes.byref(kv()), None, None) == INV
    assert lib.mk_commit_nodes(None, 1, P, 1, 2 * P, None, None) == INV
    assert lib.mk_expert_product(None, None) == INV


def test_tensors_on_the_host_are_refused():
    x = torch.zeros(1, 1, 2, 32, dtype=torch.bfloat16)
    for call in (lambda: ops.tree_attention(x, x, x, x, x), lambda: ops.qk_norm_rope(x, x, x, x, x, x, x, theta=1e4),
                 lambda: ops.copy_pages(x, x, [0], [1]), lambda: ops.commit_nodes(x, x, x, x, x),
                 lambda: ops.expert_product(x, x, x), lambda: ops.expert_product(x=None, w=x, offsets=x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_native_module_loads_and_checks():
    m = ops._native()
    x = torch.zeros(1, 1, 2, 32, dtype=torch.bfloat16)
    for call, n in ((m.qk_norm_rope, 15), (m.tree_attention, 12), (m.copy_pages, 4), (m.commit_nodes, 7), (m.expert_product, 7)):
        with pytest.raises(TypeError, match="arguments"):
            call(x)
        with pytest.raises(ValueError, match="must be a tensor"):
            call(*[None] * n)
        with pytest.raises(ValueError, match="dimensions|CUDA"):
            call(*[x] * n)
    for ids in ([0.5], ["1"], [2 ** 31], [True, None]):
        with pytest.raises(ValueError):
            m.copy_pages(torch.zeros(1, 1, 1, 16, 32, dtype=torch.bfloat16), x, ids, ids)
    with pytest.raises(ValueError):
        ops._page_ids(np.zeros((2, 2), np.int32), "src")
    with pytest.raises(ValueError):
        ops._page_ids(np.zeros(2, np.float32), "src")
    assert ops._page_ids(torch.tensor([3, 4], dtype=torch.int32), "src") == [3, 4] and ops._page_ids(np.zeros(0), "src") == []


def test_tree_mask():
    parents = torch.tensor([[-1, 0, 0, 1, 3, 2] + [5] * 30 + [35], [-1] * 37], dtype=torch.int32)
    mask, depth = ops.tree_mask(parents)
    assert mask.shape == (2, 37, 2) and mask.dtype == torch.int32
    for b in range(2):
        for i in range(37):
            want, j, d = {i}, int(parents[b, i]), 0
            while j >= 0:
                want.add(j)
                j, d = int(parents[b, j]), d + 1
            got = {a for a in range(64) if (int(mask[b, i, a // 32]) >> (a % 32)) & 1}
            assert got == want and int(depth[b, i]) == d
    with pytest.raises(ValueError):
        ops.tree_mask(parents.long())
