"""Orders in memory that the multi-token operators rely on, looked up in their sources: an
access that comes too early shows no wrong result on most runs, so no call can test for it."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "persistent_moe_decode_cta_gb300", "csrc")
KERNELS = ["mk_tree_attention.cu", "mk_experts.cu", "mk_qk_rope.cu", "mk_cache_pages.cu"]


def source(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def body(text, at):
    """From the first opening brace behind `at` to the one that closes it."""
    start = text.index("{", at)
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start:i + 1]
    raise AssertionError("unbalanced braces")


def kernels(name):
    """(name, body) of the __global__ functions of a file."""
    text = source(name)
    out = []
    for m in re.finditer(r"__global__", text):
        head = re.compile(r"(\w+)\s*\((?:[^()]|\([^()]*\))*\)\s*\{").search(text, re.compile(r"__launch_bounds__\([^()]*\)").search(text, m.end()).end())
        out.append((head.group(1), body(text, head.end() - 1)))
    return out


def readers(name):
    """Device functions of a file that read global memory, by themselves or through another one."""
    text = source(name)
    bodies = {m.group(1): body(text, m.end() - 1)
              for m in re.finditer(r"__device__[^;{}()]*?\b(\w+)\s*\((?:[^()]|\([^()]*\))*\)\s*(?:const\s*)?\{", text)}
    found = {"op_ld", "op_ld16", "op_ld16_once", "op_cp16", "op_error"}
    while True:
        more = {f for f, b in bodies.items() if f not in found and any(re.search(rf"\b{g}\s*\(", b) for g in found)}
        if not more:
            return found
        found |= more


def test_the_readers_are_found():
    assert {"seq_shape", "make_entry", "scan_units", "make_row"} <= readers("mk_tree_attention.cu")
    assert {"expert_rows", "scan_experts"} <= readers("mk_experts.cu")
    assert [[k for k, _ in kernels(f)] for f in KERNELS] == [["tree_kernel", "join_kernel"], ["expert_kernel"], ["rope_kernel"],
                                                             ["copy_pages_kernel", "commit_kernel"]]


@pytest.mark.parametrize("name", KERNELS)
def test_kernels_wait_for_earlier_ones_before_they_read(name):
    """A kernel that is launched early sees what earlier kernels wrote behind its own wait, not before."""
    reads = re.compile(r"\b(" + "|".join(sorted(readers(name))) + r")\s*\(|->\s*\w+\s*\[")
    for kernel, text in kernels(name):
        wait = text.index("pdl_wait()")
        early = reads.search(text[:wait])
        assert early is None, f"{kernel}: {early.group(0)} before the wait"
        assert "pdl_trigger()" not in text[:wait], kernel


def test_the_pair_meets_at_cluster_scope():
    """Arrivals on the other CTA's barriers, and waits for barriers that it arrives on, order at the
    scope of the cluster (at that of the CTA they would order nothing between the two)."""
    text = source("mk_experts.cu")
    arrivals = re.findall(r"mbarrier\.arrive\.[\w.:]*shared::cluster\S*", text)
    assert len(arrivals) >= 2 and all(".cluster.shared::cluster" in a for a in arrivals), arrivals
    assert set(re.findall(r"\bop_wait1?\(\s*(\w+)", text)) == {"gathered"}   # the CTA's own
    waits = re.findall(r"mbarrier\.try_wait\.parity\.[\w.:]+", text)
    assert waits and all(".cluster." in w for w in waits), waits
    assert len(re.findall(r"fence\.acquire\.sync_restrict::shared::cluster\.cluster", text)) == sum(".relaxed." in w for w in waits)
    for m in re.finditer(r"mbarrier\.arrive\.relaxed\.cluster", text):   # a release in front of it
        assert re.search(r"fence\.release\.\S*cluster;[^}]*$", text[:m.start()])


@pytest.mark.parametrize("name", KERNELS + ["mk_ops.cpp", "mk_ops.h"])
def test_launches_ask_the_device_for_its_sms(name):
    assert not re.search(r"\b(148|152)(u|l|ll)?\b", source(name)), "a number of SMs, written down"
