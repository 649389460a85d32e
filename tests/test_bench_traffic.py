"""The DRAM traffic that bench.py reports beside the step belongs to the sources it runs."""
import os
import re

import pytest

import bench

CSRC = os.path.join(bench.ROOT, "persistent_moe_decode_cta_gb300", "csrc")


@pytest.mark.parametrize("workload", ["pages_b1_8k", "pages_fp8w_b1_8k"])
def test_traffic_is_of_the_current_step(workload):
    assert bench.profiled_traffic(workload)


def test_the_key_is_the_steps_sources(monkeypatch, tmp_path):
    """All that the step's files include, and nothing of the operators' (but the header that the host shares with them)."""
    names = set(bench.STEP_SOURCES)
    for n in names:
        text = open(os.path.join(CSRC, n)).read()
        assert set(re.findall(r'#include "([^"]+)"', text)) <= names | {"mk.h", "mk_ops.h"}, n
    key = bench.kernel_source_hash()
    here = tmp_path / "persistent_moe_decode_cta_gb300" / "csrc"
    here.mkdir(parents=True)
    for n in names:
        (here / n).write_bytes(open(os.path.join(CSRC, n), "rb").read())
    (here / "mk_other_operator.cu").write_text("// another one")
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    assert bench.kernel_source_hash() == key
    (here / "mk_kernel.cu").write_text("// changed")
    assert bench.kernel_source_hash() != key
