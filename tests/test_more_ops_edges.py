"""Calls at the edge of the newer operators' entry points that need no GPU."""
import pytest
import torch

import test_ops_edges as E
from persistent_moe_decode_cta_gb300 import ops


class Devices(E.Devices):
    def linear(self, x, *_):
        self.ran.append((self.now, [s.raw or s for s in self.streams]))

    moe_layer = verify_nodes = linear


@pytest.mark.parametrize("call", [lambda t, **k: ops.linear(t, t, **k), lambda t, **k: ops.moe_layer(t, t, t, t, t, 2, residual=t, **k),
                                  lambda t, **k: ops.verify_nodes(t, t, t, draft_probs=t, **k)])
def test_calls_run_on_the_device_of_their_tensors(monkeypatch, call):
    d = Devices(monkeypatch)
    x = d.tensor(1)
    call(x)
    assert d.ran == [(1, [])] and d.now == 0 and not d.kept
    s = d.Stream("cuda:1")
    call(x, stream=s)
    assert d.ran[1:] == [(1, [s])] and set(d.kept) == {s} and len(d.kept) >= 2 and d.now == 0
    with pytest.raises(ValueError, match="is on cuda:1, the stream on cuda:0"):
        call(x, stream=d.Stream("cuda:0"))
    assert len(d.ran) == 2


def test_native_arguments_of_the_wrong_kind():
    m = ops._native()
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        m.linear(x, x, None, "silu", None, None, None, None)
    with pytest.raises(ValueError, match="CUDA"):
        m.moe_layer(x, x, x[None], x[None], x[None], None, None, None, None, None, None)
