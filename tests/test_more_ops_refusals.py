"""Calls of the projections, the routed layer and the verification that are refused before anything is launched: the C entry
points look at sizes, strides, alignment and overlaps first, so this needs no GPU (the device pointers are made up and never
followed)."""
import ctypes

import pytest
import torch

from persistent_moe_decode_cta_gb300 import binding as B
from persistent_moe_decode_cta_gb300 import ops

INV, UNS = B.MK_ERR_INVALID, B.MK_ERR_UNSUPPORTED
M = 1 << 24          # made-up, aligned device addresses, this far apart


def at(i):
    return (i + 1) * M


def linear(**over):
    a = dict(x=at(0), w=at(1), bias=at(2), residual=at(3), out=at(4), x_stride=64, residual_stride=32, out_stride=32, m=8, n=32, k=64)
    a.update(over)
    return B.mk_linear_args(**a)


def moe(**over):
    a = dict(x=at(0), router=at(1), w_gate=at(2), w_up=at(3), w_down=at(4), residual=at(5), out=at(6), ids=at(7), weights=at(8), x_stride=64,
             residual_stride=64, out_stride=64, n_tokens=4, d_model=64, d_ff=32, n_experts=8, top_k=2, workspace=at(9), workspace_bytes=1 << 20)
    a.update(over)
    return B.mk_moe_args(**a)


def verify(**over):
    s = B._S2
    a = dict(logits=at(0), draft_probs=at(1), tokens=at(2), parents=at(3), uniforms=at(4), temperature=at(5), counts=at(6), accepted=at(7),
             next_tokens=at(8), logits_stride=s(400, 100), draft_stride=s(400, 100), batch=3, n_nodes=4, vocab=100, logits_float=1,
             workspace=at(9), workspace_bytes=1 << 20)
    a.update(over)
    return B.mk_verify_args(**a)


@pytest.mark.parametrize("over,code", [
    (dict(x=None), INV), (dict(w=None), INV), (dict(out=None), INV), (dict(x=at(0) + 8), INV), (dict(w=at(1) + 2), INV), (dict(m=-1), INV),
    (dict(n=0), INV), (dict(k=0), UNS), (dict(k=60), UNS), (dict(activation=-1), INV), (dict(activation=5), INV), (dict(x_stride=56), INV),
    (dict(x_stride=68), INV), (dict(out_stride=31), INV), (dict(residual_stride=31), INV), (dict(out=at(4) + 1), INV), (dict(bias=at(2) + 1), INV),
    (dict(residual=at(3) + 1), INV), (dict(out=at(4) + 2, out_float=1), INV), (dict(m=1 << 28, n=1 << 24, out_stride=1 << 24, residual_stride=1 << 24), UNS),
    # overlaps: x, w, bias; the residual other than as itself
    (dict(out=at(0)), INV), (dict(out=at(1) + 32), INV), (dict(out=at(2) - 16), INV), (dict(out=at(3) + 16), INV), (dict(out=at(3), out_stride=40), INV),
    (dict(out=at(3), out_float=1), INV)])
def test_linear_arguments(over, code):
    lib = B.load_library()
    assert lib.mk_linear(ctypes.byref(linear(**over)), None) == code
    assert lib.mk_last_error(None)


def test_linear_columns_side_by_side():
    """Two halves of one tensor do not overlap, columns that cross do."""
    lib = B.load_library()

    def overlap(delta):
        a = linear(residual=at(3), out=at(3) + delta, residual_stride=64, out_stride=64)
        return lib.mk_linear(ctypes.byref(a), None) == INV and b"overlaps" in lib.mk_last_error(None)
    assert overlap(62) and overlap(66) and overlap(2) and overlap(-62)
    if not torch.cuda.is_available():       # (what is not refused would follow the made-up addresses)
        assert not overlap(64) and not overlap(-64)


@pytest.mark.parametrize("over,code", [
    (dict(x=None), INV), (dict(router=None), INV), (dict(w_gate=None), INV), (dict(w_up=None), INV), (dict(w_down=None), INV), (dict(out=None), INV),
    (dict(x=at(0) + 8), INV), (dict(router=at(1) + 2), INV), (dict(w_gate=at(2) + 8), INV), (dict(w_up=at(3) + 8), INV), (dict(w_down=at(4) + 8), INV),
    (dict(n_tokens=-1), INV), (dict(n_tokens=257), UNS), (dict(n_experts=0), INV), (dict(n_experts=257), INV), (dict(top_k=0), INV), (dict(top_k=9), INV),
    (dict(n_experts=32, top_k=17), INV), (dict(d_model=60), UNS), (dict(d_model=0), UNS), (dict(d_ff=30), UNS), (dict(d_ff=0), UNS),
    (dict(x_stride=56), INV), (dict(x_stride=68), INV), (dict(out_stride=63), INV), (dict(residual_stride=63), INV), (dict(out=at(6) + 1), INV),
    (dict(ids=at(7) + 2), INV), (dict(weights=at(8) + 1), INV), (dict(workspace=None), INV), (dict(workspace=at(9) + 8), INV), (dict(workspace_bytes=100), INV),
    (dict(out=at(0)), INV), (dict(out=at(2) + 64), INV), (dict(out=at(5) + 2), INV), (dict(ids=at(0)), INV), (dict(weights=at(7)), INV),
    (dict(workspace=at(1)), INV), (dict(workspace=at(6)), INV), (dict(ids=at(9) + 16), INV)])
def test_moe_arguments(over, code):
    lib = B.load_library()
    assert lib.mk_moe_layer(ctypes.byref(moe(**over)), None) == code
    assert lib.mk_last_error(None)


def test_moe_workspace():
    lib, n = B.load_library(), ctypes.c_size_t()
    assert lib.mk_moe_layer_workspace(ctypes.byref(moe()), ctypes.byref(n)) == B.MK_OK and n.value >= 8 * (8 + 64)
    need = n.value
    assert lib.mk_moe_layer(ctypes.byref(moe(workspace_bytes=need - 1)), None) == INV
    assert lib.mk_moe_layer_workspace(ctypes.byref(moe(n_tokens=300)), ctypes.byref(n)) == UNS
    assert lib.mk_moe_layer_workspace(ctypes.byref(moe()), None) == INV
    assert lib.mk_moe_layer_workspace(None, ctypes.byref(n)) == INV


@pytest.mark.parametrize("over", [
    dict(logits=None), dict(tokens=None), dict(uniforms=None), dict(accepted=None), dict(next_tokens=None), dict(logits=at(0) + 2),
    dict(logits=at(0) + 1, logits_float=0), dict(draft_probs=at(1) + 2), dict(batch=-1), dict(batch=65536), dict(n_nodes=0), dict(n_nodes=513),
    dict(vocab=0), dict(vocab=262145), dict(logits_stride=B._S2(400, 99)), dict(logits_stride=B._S2(0, 100)), dict(draft_stride=B._S2(400, 50)),
    dict(draft_stride=B._S2(-400, 100)), dict(workspace=None), dict(workspace=at(9) + 4), dict(workspace_bytes=16), dict(accepted=at(2)),
    dict(accepted=at(0) + 400), dict(next_tokens=at(7) + 44), dict(next_tokens=at(5)), dict(next_tokens=at(6) + 8), dict(accepted=at(3)),
    dict(accepted=at(4)), dict(workspace=at(1)), dict(workspace=at(7))])
def test_verify_arguments(over):
    lib = B.load_library()
    assert lib.mk_verify_nodes(ctypes.byref(verify(**over)), None) == INV
    assert lib.mk_last_error(None)


def test_verify_workspace():
    lib, n = B.load_library(), ctypes.c_size_t()
    assert lib.mk_verify_nodes_workspace(ctypes.byref(verify()), ctypes.byref(n)) == B.MK_OK
    assert lib.mk_verify_nodes(ctypes.byref(verify(workspace_bytes=n.value - 1)), None) == INV
    assert lib.mk_verify_nodes_workspace(ctypes.byref(verify(vocab=0)), ctypes.byref(n)) == INV
    assert lib.mk_verify_nodes_workspace(ctypes.byref(verify()), None) == INV
    assert lib.mk_verify_nodes_workspace(None, ctypes.byref(n)) == INV


def test_no_work():
    lib = B.load_library()
    assert lib.mk_linear(ctypes.byref(linear(m=0, x=None)), None) == B.MK_OK
    assert lib.mk_moe_layer(ctypes.byref(moe(n_tokens=0, x=None)), None) == B.MK_OK
    assert lib.mk_verify_nodes(ctypes.byref(verify(batch=0, logits=None)), None) == B.MK_OK
    assert lib.mk_linear(None, None) == lib.mk_moe_layer(None, None) == lib.mk_verify_nodes(None, None) == INV


def test_tensors_on_the_host_and_wrong_choices_are_refused():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    for call in (lambda: ops.linear(x, x), lambda: ops.moe_layer(x, x, x[None], x[None], x[None], 1), lambda: ops.verify_nodes(x[None], x, x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_native_module_checks():
    m = ops._native()
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    for call, n in ((m.linear, 8), (m.moe_layer, 11), (m.verify_nodes, 10)):
        with pytest.raises(TypeError, match="arguments"):
            call(x)
        with pytest.raises(ValueError, match="must be a tensor"):
            call(*[None] * n)
        with pytest.raises(ValueError, match="dimensions|CUDA"):
            call(*[x] * n)
    with pytest.raises(ValueError, match="x requires a gradient"):
        m.linear(x.clone().requires_grad_(), x, None, 0, None, None, None, None)
    with pytest.raises(ValueError, match="logits must be"):
        m.verify_nodes(torch.zeros(1, 2, 3, dtype=torch.float16), *[None] * 9)


@pytest.mark.parametrize("bad", [dict(activation="swish"), dict(activation=1), dict(activation=[]), dict(dtype=torch.float16), dict(dtype="bf16")])
def test_choices(bad, monkeypatch):
    class Here:
        def is_here(self, t):
            return True
    monkeypatch.setattr(ops, "_module", Here())
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="activation|dtype"):
        ops.linear(x, x, **bad)
