"""Orders in memory that the projections, the routed layer and the verification rely on, looked up in their sources."""
import re

import pytest

import test_ops_sources as T

NAMES = ["mk_moe.cu", "mk_verify.cu", "mk_linear.cu"]


def test_the_kernels_and_readers_are_found():
    assert [[k for k, _ in T.kernels(f)] for f in NAMES] == [["router_kernel", "layer_kernel", "sort_kernel", "sum_kernel"], ["row_kernel", "walk_kernel"],
                                                          ["split_kernel"]]
    assert {"gather_nodes"} <= readers("mk_verify.cu")


def readers(name):
    """Device functions that read global memory, by themselves or through another one, the small loads among them."""
    text = T.source(name)
    bodies = {m.group(1): T.body(text, m.end() - 1)
              for m in re.finditer(r"__device__[^;{}()]*?\b(\w+)\s*\((?:[^()]|\([^()]*\))*\)\s*(?:const\s*)?\{", text)}
    found = {"op_ld", "op_ld2", "op_ld8", "op_ldf", "op_ld16", "op_ld16_once", "op_cp16", "op_cp8", "cp16", "op_error"}
    while True:
        more = {f for f, b in bodies.items() if f not in found and any(re.search(rf"\b{g}\s*\(", b) for g in found)}
        if not more:
            return found
        found |= more


@pytest.mark.parametrize("name", NAMES)
def test_kernels_wait_for_earlier_ones_before_they_read(name):
    reads = re.compile(r"\b(" + "|".join(sorted(readers(name))) + r"|atomicAdd)\s*\(|->\s*\w+\s*\[")
    for kernel, text in T.kernels(name):
        wait = text.index("pdl_wait()")
        early = reads.search(text[:wait])
        assert early is None, f"{kernel}: {early.group(0)} before the wait"
        assert "pdl_trigger()" not in text[:wait], kernel


@pytest.mark.parametrize("name", NAMES + ["mk_linear.cuh"])
def test_launches_ask_the_device_for_its_sms(name):
    assert not re.search(r"\b(148|152)(u|l|ll)?\b", T.source(name)), "a number of SMs, written down"


@pytest.mark.parametrize("name", NAMES + ["mk_linear.cuh"])
def test_global_memory_is_not_read_through_the_read_only_path(name):
    assert not re.search(r"__ldg|ld\.global\.nc|__restrict__", T.source(name))


def test_a_cta_that_gave_up_a_wait_sends_no_more():
    """The other CTAs of a walk leave once they have had all that was sent for their own passes: one whose sums are wrong may walk longer than
    they do, and must not write to where they were."""
    text = T.source("mk_verify.cu")
    exchange = T.body(text, text.index("exchange(WalkShared& sh"))
    sends = [exchange[:m.start()] for m in re.finditer(r"\bput_async\s*\(", exchange)]
    assert len(sends) == 1 and len(re.findall(r"\bput_async\s*\(", text)) == 2      # (the function and its one call)
    assert re.search(r"if\s*\([^{;]*!\s*[^{;]*\bsh\.abort[^{;]*\)\s*\{[^}]*$", sends[0]), "sent whether a wait was given up or not"
