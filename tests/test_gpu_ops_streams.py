"""The multi-token operators side by side on several streams, and captured on their first use."""
import os
import subprocess
import sys

import pytest
import torch

import ops_ref as R
from persistent_moe_decode_cta_gb300 import ops

pytestmark = pytest.mark.gpu


def calls(seed):
    """One call of every operator that returns a tensor, on inputs of its own."""
    g = R.gen(seed)
    lens = [50, 300, 1900]
    k, v, table, sl = R.cache(g, lens, 40, 4, 64, layers=2)
    q, kn, vn = R.bf16(g, 3, 40, 16, 64), R.bf16(g, 3, 40, 4, 64), R.bf16(g, 3, 40, 4, 64)
    kc, vc, tc, _ = R.cache(g, lens, 40, 4, 64)
    ks, vs, ts, _ = R.cache(g, lens, 40, 1, 32)
    q1 = R.bf16(g, 3, 40, 4, 32)
    acc = torch.tensor([[1, 3, 4], [0, -1, 7], [39, 2, 39]], dtype=torch.int32, device="cuda")
    x, w, u = R.bf16(g, 900, 256), R.bf16(g, 5, 192, 256, std=0.05), R.bf16(g, 5, 192, 256, std=0.05)
    offsets = torch.tensor([0, 3, 300, 300, 870, 900], dtype=torch.int32, device="cuda")
    named = torch.randint(0, 900, (900,), generator=g, device="cuda").to(torch.int32)
    return [lambda **s: ops.tree_attention(q, kc, vc, tc, sl, **s),
            lambda **s: ops.tree_attention(q1, ks, vs, ts, sl, **s),
            lambda **s: ops.expert_product(x, w, offsets, **s),
            lambda **s: ops.expert_product(x, w, offsets, w_up=u, rows=named, **s),
            lambda **s: ops.qk_norm_rope(q, kn, vn, k[0], v[0], table, sl, theta=1e4, **s),
            lambda **s: ops.commit_nodes(k, v, table, sl, acc, **s)]


def test_streams_side_by_side():
    """Every operator on a stream of its own, all at once, several times: the results of calls one by one."""
    many = [c for seed in range(3) for c in calls(seed)]
    want = [c() for c in many]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in many]
    for _ in range(5):
        # (the fifth and the sixth write the same pools, and return nothing that they read there)
        got = [c(stream=s) for c, s in zip(many, streams)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)


FIRST = """
import sys
sys.path[:0] = [{tests!r}, {root!r}]
import torch
import test_gpu_ops_streams as T
graphs, outs = [], []
for call in T.calls(0):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs.append(call())
    graphs.append(graph)
for graph in graphs:
    graph.replay()
torch.cuda.synchronize()
for call, out in zip(T.calls(0), outs):
    assert torch.equal(call(), out)
print("equal")
"""


def test_captured_on_first_use():
    """In a process of its own, each operator's first call is a captured one."""
    here = os.path.dirname(os.path.abspath(__file__))
    run = subprocess.run([sys.executable, "-c", FIRST.format(tests=here, root=os.path.dirname(here))], capture_output=True,
                         text=True, timeout=300)
    assert run.returncode == 0 and run.stdout.split()[-1] == "equal", run.stderr[-2000:]


@pytest.mark.parametrize("heads,d,lens", [((8, 2, 32), 256, [5, 60, 700]), ((32, 4, 128), 512, [0, 3000])])
def test_chain_of_dependent_calls(heads, d, lens):
    """Each call reads what the one before it wrote, while their launches overlap: step by step with a
    synchronisation behind every call, back to back, and captured, the bits are the same."""
    hq, hkv, hd = heads
    g = R.gen(11)
    b, n = len(lens), 12
    k, v, table, sl = R.cache(g, lens, 4 * n, hkv, hd, layers=2)
    q, kn, vn = R.bf16(g, b, n, hq, hd), R.bf16(g, b, n, hkv, hd), R.bf16(g, b, n, hkv, hd)
    w = R.bf16(g, 3, d, hq * hd, std=0.05)
    back = R.bf16(g, 3, hq * hd, d, std=0.05)
    offsets = torch.tensor([0, 7, 7, b * n], dtype=torch.int32, device="cuda")
    acc = torch.tensor([[1, 3, 6, 7, -1]] * b, dtype=torch.int32, device="cuda")
    k0, v0 = k.clone(), v.clone()
    torch.cuda.synchronize()

    def run(pause):
        x, lengths = q, sl
        for _ in range(3):
            for layer in range(2):
                x = ops.qk_norm_rope(x, kn, vn, k[layer], v[layer], table, lengths, theta=1e4)
                pause()
                x = ops.tree_attention(x, k[layer], v[layer], table, lengths)
                pause()
                h = ops.expert_product(x.view(b * n, hq * hd), w, offsets)
                pause()
                x = ops.expert_product(h, back, offsets).view(b, n, hq, hd)
                pause()
            lengths = ops.commit_nodes(k, v, table, lengths, acc)
            pause()
        return x, lengths

    def reset():
        k.copy_(k0), v.copy_(v0)

    x, lengths = run(torch.cuda.synchronize)
    want = [t.clone() for t in (x, lengths, k, v)]
    assert torch.isfinite(x).all() and (lengths == sl + 12).all()
    for _ in range(10):
        reset()
        x, lengths = run(lambda: None)
        assert all(torch.equal(a, c) for a, c in zip(want, (x, lengths, k, v)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x, lengths = run(lambda: None)
    for _ in range(10):
        reset()
        graph.replay()
        assert all(torch.equal(a, c) for a, c in zip(want, (x, lengths, k, v)))
