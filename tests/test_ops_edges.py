"""Calls at the edge of the multi-token operators' entry points that need no GPU."""
import os
import subprocess
import sys

from persistent_moe_decode_cta_gb300 import binding as B

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
