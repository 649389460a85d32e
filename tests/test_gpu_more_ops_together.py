"""A whole verification step of drafted tokens out of the operators (projections, head rotation and append, tree attention,
routed layers, LM head, verification, commit), then further steps of the megakernel on the same cache; and the projections, the
routed layer and the verification side by side on streams, captured on first use, and in chains of dependent calls."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import more_ops_ref as M
import ops_ref as R
import parity_util as PU
import synth
import test_gpu_verify as V
from persistent_moe_decode_cta_gb300 import binding as B
from persistent_moe_decode_cta_gb300 import ops

pytestmark = pytest.mark.gpu


def norm(x, gain, eps):
    return V.rms(x.float(), gain, eps).to(torch.bfloat16)


def whole_pass(cfg, W, tokens, k, v, table, lens, mask, positions):
    """Logits [batch, n, vocab] in float32 of all nodes, and the experts chosen, [layer][batch, n, top_k]."""
    b, n = tokens.shape
    hq, hkv, hd, top = (cfg[x] for x in ("n_q_heads", "n_kv_heads", "head_dim", "top_k"))
    x = W["embed"][tokens.long()].view(b * n, -1)
    chosen = []
    for l in range(cfg["n_layers"]):
        h = norm(x, W["attn_norm"][l], cfg["rms_eps"])
        w = torch.cat([W["wq"][l], W["wk"][l], W["wv"][l]])
        qkv = ops.linear(h, w).view(b, n, hq + 2 * hkv, hd)
        q = ops.qk_norm_rope(qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:], k[l], v[l], table, lens,
                             theta=cfg["rope_theta"], positions=positions)
        o = ops.tree_attention(q, k[l], v[l], table, lens, mask=mask, positions=positions)
        x = ops.linear(o.view(b * n, hq * hd), W["wo"][l], residual=x)
        ids = torch.empty(b * n, top, dtype=torch.int32, device="cuda")
        x = ops.moe_layer(h, W["router"][l], W["w_gate"][l], W["w_up"][l], W["w_down"][l], top, residual=x, ids=ids)
        chosen.append(ids.view(b, n, top))
    h = norm(x, W["final_norm"], cfg["rms_eps"])
    return ops.linear(h, W["lm_head"], dtype=torch.float32).view(b, n, -1), chosen


@pytest.mark.parametrize("model,lens", [("tiny", [61, 14]), ("small", [130])])
def test_a_whole_verification_step(model, lens):
    cfg = dict(synth.MODELS[model], page_size=16)
    if model == "small":
        cfg["n_layers"] = 2
    parents = [-1, 0, 0, 1, 1, 2, 3, 6, 5, 8]
    n, b = len(parents), len(lens)
    W = synth.make_weights(cfg, seed=3, device="cuda", gain_jitter=0.1)
    pt, npages = synth.make_page_table(lens, steps=n + 4, seed=1, spare=8)
    k, v = synth.make_kv(cfg, npages, seed=1, device="cuda")
    table = torch.as_tensor(pt, device="cuda")
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    g = R.gen(5)
    up = torch.tensor([parents] * b, dtype=torch.int32, device="cuda")
    mask, depth = ops.tree_mask(up)
    tokens = torch.randint(0, cfg["vocab"], (b, n), generator=g, device="cuda").to(torch.int32)
    k0, v0 = k.clone(), v.clone()
    logits, chosen = whole_pass(cfg, W, tokens, k, v, table, sl, mask, sl[:, None] + depth)
    ops.check_status()
    experts = [c.cpu().numpy() for c in chosen]
    for s in range(b):
        for path in V.paths_of(parents):
            want, _, _ = V.oracle_path(cfg, W, path, tokens, k0, v0, pt, s, lens[s], experts)
            for node, ref in zip(path, want):
                off = float(np.abs(logits[s, node].cpu().numpy() - ref).max())
                assert off <= PU.LOGIT_ABS, (s, node, off)

    # which of the nodes are kept, the commit, and a step of the megakernel from there on.  (The drafting model is one that knows
    # the drafted tokens to be likely, so that some are kept.)
    heat = torch.full((b,), 0.5, device="cuda")
    draft = (logits / heat[:, None, None]).softmax(-1)
    uniforms = torch.rand(b, n, generator=g, device="cuda")
    for s in range(b):
        uniforms[s, 1 + s] = 0.0
    accepted, nxt = ops.verify_nodes(logits, tokens, uniforms, parents=up, draft_probs=draft, temperature=heat)
    path, drawn = M.verify(logits, tokens, uniforms, up, draft, heat)
    assert accepted.tolist() == path and nxt.tolist() == drawn
    assert max(sum(i >= 0 for i in p) for p in path) >= 2
    new = ops.commit_nodes(k, v, table, sl, accepted)
    ops.check_status()
    assert new.tolist() == [m + sum(i >= 0 for i in p) for m, p in zip(lens, path)]
    mk = B.Megakernel(cfg, W, max_batch=8)
    try:
        seq = new.tolist()
        mk.plan(seq, table, npages)
        before = (k.clone(), v.clone())
        out = torch.empty(b, cfg["vocab"], device="cuda")
        mk.step(nxt, k, v, out)
        assert mk.status()["code"] == 0
        PU.check_step(cfg, mk, W, seq, pt, before, nxt.cpu().numpy(), out, k, v)
    finally:
        mk.close()


def calls(seed):
    """Calls of every form of the three operators, on inputs of their own."""
    g = R.gen(seed)
    x, w, res = R.bf16(g, 700, 256), R.bf16(g, 320, 256, std=0.05), R.bf16(g, 700, 320)
    wide = R.bf16(g, 20000, 256, std=0.05)
    router, gate, up, down = R.bf16(g, 16, 256, std=0.05), R.bf16(g, 16, 128, 256, std=0.05), R.bf16(g, 16, 128, 256, std=0.05), R.bf16(g, 16, 256, 128, std=0.05)
    a = M.tree_inputs(g, 3, 6, 5000, True, True)
    c = M.tree_inputs(g, 2, 4, 1000, False, False, half=True)
    return [lambda **s: ops.linear(x[:7], w, residual=res[:7], **s),
            lambda **s: ops.linear(x[:90], w, activation="silu", **s),
            lambda **s: ops.linear(x, wide, activation="gelu", **s),
            lambda **s: ops.linear(x[:70], wide, dtype=torch.float32, **s),
            lambda **s: ops.moe_layer(x[:3], router, gate, up, down, 4, residual=x[:3], **s),
            lambda **s: ops.moe_layer(x[:14], router, gate, up, down, 4, **s),
            lambda **s: ops.moe_layer(x[:100], router, gate, up, down, 4, residual=x[:100], **s),
            lambda **s: torch.cat([t.view(-1) for t in ops.verify_nodes(a[0], a[1], a[2], parents=a[3], draft_probs=a[4], **s)]),
            lambda **s: ops.verify_nodes(c[0], c[1], c[2], **s)[1]]


def test_streams_side_by_side():
    many = [c for seed in range(2) for c in calls(seed)]
    want = [c() for c in many]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in many]
    for _ in range(5):
        got = [c(stream=s) for c, s in zip(many, streams)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)


FIRST = """
import sys
sys.path[:0] = [{tests!r}, {root!r}]
import torch
import test_gpu_more_ops_together as T
graphs, outs = [], []
for call in T.calls(0):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs.append(call())
    graphs.append(graph)
for _ in range(2):
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


@pytest.mark.parametrize("m", [1, 6, 12, 90, 256])
def test_chain_of_dependent_calls(m):
    """Each call reads what the one before it wrote, while their launches overlap: step by step with a synchronisation behind every
    call, back to back, and captured, the bits are the same."""
    g = R.gen(11)
    d, f, e, vocab = 256, 128, 12, 3000
    x0 = R.bf16(g, m, d)
    w, back, head = R.bf16(g, 2 * d, d, std=0.05), R.bf16(g, d, 2 * d, std=0.05), R.bf16(g, vocab, d, std=0.1)
    router, gate, up, down = R.bf16(g, e, d, std=0.05), R.bf16(g, e, f, d, std=0.05), R.bf16(g, e, f, d, std=0.05), R.bf16(g, e, d, f, std=0.05)
    tokens = torch.randint(0, vocab, (1, m), generator=g, device="cuda").to(torch.int32)
    uniforms = torch.rand(1, m, generator=g, device="cuda") * 0.02
    torch.cuda.synchronize()

    def run(pause):
        x = x0
        for _ in range(3):
            h = ops.linear(x, w, activation="gelu_tanh")
            pause()
            x = ops.linear(h, back, residual=x)
            pause()
            x = ops.moe_layer(x, router, gate, up, down, 3, residual=x)
            pause()
        logits = ops.linear(x, head, dtype=torch.float32)
        pause()
        accepted, drawn = ops.verify_nodes(logits.view(1, m, vocab), tokens, uniforms)
        pause()
        return x, logits, accepted, drawn

    want = [t.clone() for t in run(torch.cuda.synchronize)]
    assert torch.isfinite(want[0]).all() and want[2][0, 0] == 0
    for _ in range(10):
        assert all(torch.equal(a, c) for a, c in zip(want, run(lambda: None)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(lambda: None)
    for _ in range(10):
        graph.replay()
        assert all(torch.equal(a, c) for a, c in zip(want, got))


def test_two_graphs_of_one_pool():
    """Two captured calls whose workspaces may lie in the same memory, replayed in turn."""
    g = R.gen(12)
    w = (R.bf16(g, 16, 256, std=0.05), R.bf16(g, 16, 128, 256, std=0.05), R.bf16(g, 16, 128, 256, std=0.05), R.bf16(g, 16, 256, 128, std=0.05))
    xs = [R.bf16(g, t, 256) for t in (5, 30)]
    want = [ops.moe_layer(x, *w, 4) for x in xs]
    pool = torch.cuda.graph_pool_handle()
    graphs, outs = [], []
    for x in xs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=pool):
            outs.append(ops.moe_layer(x, *w, 4).clone())
        graphs.append(graph)
    for _ in range(3):
        for graph, out, ref in zip(graphs, outs, want):
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, ref)
