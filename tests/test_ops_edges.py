"""Calls at the edge of the multi-token operators' entry points that need no GPU."""
import contextlib
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch
import torch.autograd.forward_ad as forward

from persistent_moe_decode_cta_gb300 import binding as B
from persistent_moe_decode_cta_gb300 import ops
import test_ops_refusals as R

P = R.P
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_op_status_needs_somewhere_to_write():
    assert B.load_library().mk_op_status(None, None) == B.MK_ERR_INVALID


def run(code, **env):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, env={**os.environ, **env})
    assert r.returncode == 0, r.stderr[-2000:]
    return r.stdout


def test_the_package_alone_imports_no_torch():
    """`binding` and `sol` serve programs without torch; `ops` comes with its first use."""
    out = run("import sys, persistent_moe_decode_cta_gb300 as p\n"
              "p.binding.load_library()\n"
              "p.sol\n"
              "assert 'torch' not in sys.modules\n"
              "assert p.ops.PAGE == 16 and 'torch' in sys.modules\n"
              "from persistent_moe_decode_cta_gb300 import *\n"
              "print(ops.__name__)")
    assert out.split() == ["persistent_moe_decode_cta_gb300.ops"]


COMPILER = """#!{python}
import sys

import pytest
import torch
import torch.autograd.forward_ad as forward
open(sys.argv[sys.argv.index("-o") + 1], "w").write("built")
"""

BUILD = """
import os, sys
if {block}:
    class NoTorch:
        def find_spec(self, name, path=None, target=None):
            if name.split(".")[0] == "torch":
                raise ModuleNotFoundError(name)
    import importlib.util
    found = importlib.util.find_spec
    importlib.util.find_spec = lambda name, *a: None if name == "torch" else found(name, *a)
    sys.meta_path.insert(0, NoTorch())
from persistent_moe_decode_cta_gb300 import build as b
b.OUT_DIR, b.LIB, b.MODULE = (os.path.join({out!r}, x) for x in ("_build", "libmk.so", "_ops.so"))
b.build()
print(*sorted(x for x in os.listdir({out!r}) if x.endswith(".so")))
"""


@pytest.mark.parametrize("block", [True, False])
def test_the_library_is_built_without_torch(tmp_path, block):
    """(With a compiler that only writes its output: which files are asked for.)"""
    fake = tmp_path / "compiler"
    fake.write_text(COMPILER.format(python=sys.executable))
    fake.chmod(0o755)
    out = run(BUILD.format(block=block, out=str(tmp_path)), NVCC=str(fake), CXX=str(fake))
    assert out.split() == (["libmk.so"] if block else ["_ops.so", "libmk.so"])


def test_tensors_that_carry_derivatives_are_refused():
    """A gradient that would be wanted, and a forward-mode tangent that would be dropped."""
    m = ops._native()
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with forward.dual_level():
        dual = forward.make_dual(x, torch.ones_like(x))
        with pytest.raises(ValueError, match="x carries a forward-mode tangent"):
            m.expert_product(dual, x[None], x, None, None, None, None)
    with pytest.raises(ValueError, match="x requires a gradient"):
        m.expert_product(x.clone().requires_grad_(), x[None], x, None, None, None, None)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"), torch.no_grad():
        m.expert_product(x.clone().requires_grad_(), x[None], x, None, None, None, None)


@pytest.mark.parametrize("shift", [0, 16, 40959, 40960])
def test_pools_that_overlap_are_not_written(shift):
    """K and V of one layer are 40960 bytes here, of three 122880."""
    lib = B.load_library()
    pages = np.array([0, 1], np.int32)

    def refused(rc):
        return rc == B.MK_ERR_INVALID and b"overlap" in lib.mk_last_error(None)

    for k, v in ((P, P + shift // 16 * 16), (P + shift // 16 * 16, P)):
        one = R.kv(k=k, v=v)
        if shift < 40960:    # (what is not refused would follow the made-up addresses where there is a GPU)
            assert refused(lib.mk_qk_norm_rope(ctypes.byref(one), ctypes.byref(R.rope()), None))
        assert refused(lib.mk_commit_nodes(ctypes.byref(one), 3, P, 4, 1 << 40, None, None))
        if shift:    # (the same pool twice: the same copies twice)
            assert refused(lib.mk_copy_pages(k, v, 3, 10, 2, 64, pages[:1].ctypes.data, pages[1:].ctypes.data, 1, None))


@pytest.mark.parametrize("lens,table,accepted,new", [
    (0, 4096, 8192, 0), (0, 4096, 8192, 4), (4, 4096, 8192, 0), (0, 4096, 8192, 4096), (0, 4096, 8192, 4096 + 28), (0, 4096, 8192, 4092),
    (0, 4096, 8192, 8192), (0, 4096, 8192, 8192 + 20), (0, 4096, 8192, 8188)])
def test_new_lengths_are_no_part_of_what_is_read(lens, table, accepted, new):
    """Two sequences, tables of 4 pages, paths of 3 nodes; offsets in bytes."""
    c = R.kv(k=P, v=1 << 40, seq_lens=P + lens, page_table=P + table)
    lib = B.load_library()
    assert lib.mk_commit_nodes(ctypes.byref(c), 1, P + accepted, 3, P + new, None, None) == B.MK_ERR_INVALID
    assert b"new_lens" in lib.mk_last_error(None)


class Devices:
    """Two devices that are not there: which one is current, where calls run, what they keep."""

    def __init__(self, monkeypatch):
        self.now, self.streams, self.ran, self.kept = 0, [], [], []
        monkeypatch.setattr(ops, "_module", self)
        monkeypatch.setattr(torch.cuda, "device", lambda d: self.entered("now", d))
        monkeypatch.setattr(torch.cuda, "stream", lambda s: self.entered("streams", self.streams + [s]))
        monkeypatch.setattr(torch.cuda, "Stream", self.Stream)
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda raw, device: self.Stream(device, raw))

    class Stream:
        def __init__(self, device, raw=None):
            self.device, self.raw = torch.device(device), raw

    @contextlib.contextmanager
    def entered(self, name, value):
        before = getattr(self, name)
        setattr(self, name, value)
        try:
            yield
        finally:
            setattr(self, name, before)

    def is_here(self, t):
        return t.get_device() == self.now

    def copy_pages(self, k, *_):
        self.ran.append((self.now, [s.raw or s for s in self.streams]))

    def tensor(self, index):
        kept = self.kept

        class Tensor(torch.Tensor):
            device = torch.device("cuda", index)
            is_cuda = True

            def get_device(self):
                return index

            def record_stream(self, s):
                kept.append(s.raw or s)
        return torch.zeros(1).as_subclass(Tensor)


def test_calls_run_on_the_device_of_their_tensors(monkeypatch):
    d = Devices(monkeypatch)
    k = d.tensor(1)
    ops.copy_pages(k, k, [0], [1])
    assert d.ran == [(1, [])] and d.now == 0 and not d.kept
    s = d.Stream("cuda:1")
    ops.copy_pages(k, k, [0], [1], stream=s)
    ops.copy_pages(k, k, [0], [1], stream=77)            # a raw pointer: a stream of the tensors' device
    assert d.ran[1:] == [(1, [s]), (1, [77])] and d.kept == [s, s, 77, 77] and d.now == 0
    with pytest.raises(ValueError, match="k_cache is on cuda:1, the stream on cuda:0"):
        ops.copy_pages(k, k, [0], [1], stream=d.Stream("cuda:0"))
    assert len(d.ran) == 3 and d.now == 0
