"""The multi-token operators together, as a program that drafts tokens uses them around the
decode step: a verification pass over draft trees (append, attention, experts), the commit
of an accepted path, a fork, and further steps of the megakernel on the same cache."""
import numpy as np
import pytest
import torch

import oracle
import parity_util as PU
import synth
from persistent_moe_decode_cta_gb300 import binding as B
from persistent_moe_decode_cta_gb300 import ops

pytestmark = pytest.mark.gpu


def rms(x, gain, eps):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * gain.float()


def verify_pass(cfg, W, tokens, k, v, table, lens, mask, positions):
    """Logits [batch, n, vocab] of all nodes and the experts chosen, [layer][batch, n, top_k].
    The nodes' K/V end up in their slots of every layer."""
    b, n = tokens.shape
    hq, hkv, hd, top, e = (cfg[x] for x in ("n_q_heads", "n_kv_heads", "head_dim", "top_k", "n_experts"))
    x = W["embed"][tokens.long()].float()                                  # fp32 residual
    chosen = []
    for l in range(cfg["n_layers"]):
        hf = rms(x, W["attn_norm"][l], cfg["rms_eps"])
        h = hf.to(torch.bfloat16)
        w = torch.cat([W["wq"][l], W["wk"][l], W["wv"][l]])
        qkv = (h @ w.T).view(b, n, hq + 2 * hkv, hd)
        q = ops.qk_norm_rope(qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:], k[l], v[l], table, lens,
                             theta=cfg["rope_theta"], positions=positions)
        window = cfg["sliding_window"] if l in cfg["swa_layers"] else 0
        o = ops.tree_attention(q, k[l], v[l], table, lens, mask=mask, positions=positions, window=window)
        attn = (o.view(b, n, hq * hd) @ W["wo"][l].T).float()
        weight, idx = (hf @ W["router"][l].float().T).topk(top, -1)
        weight = weight.softmax(-1)
        chosen.append(idx)
        flat = idx.reshape(-1)
        order = flat.argsort(stable=True)
        offsets = torch.cat([flat.new_zeros(1), torch.bincount(flat, minlength=e).cumsum(0)]).to(torch.int32)
        rows = (order // top).to(torch.int32)
        up = ops.expert_product(h.view(b * n, -1), W["w_gate"][l], offsets, w_up=W["w_up"][l], rows=rows)
        down = ops.expert_product(up, W["w_down"][l], offsets)
        moe = torch.zeros(b * n * top, x.shape[-1], device="cuda")
        moe[order] = down.float() * weight.reshape(-1)[order][:, None]
        x = x + attn + moe.view(b, n, top, -1).sum(2)
    return rms(x, W["final_norm"], cfg["rms_eps"]).to(torch.bfloat16).float() @ W["lm_head"].float().T, chosen


def oracle_path(cfg, W, path, tokens, k, v, pt, b, length, chosen):
    """Logits of the path's nodes, and the pools after them, by one oracle step per node (with
    the experts of the pass: near-ties of the router are no matter here)."""
    k, v = k.clone(), v.clone()
    out = []
    for i, node in enumerate(path):
        forced = {(l, 0): [int(e) for e in chosen[l][b, node]] for l in range(cfg["n_layers"])}
        ref = oracle.decode_step(cfg, synth.HostWeights(W), synth.HostKV(k, v), np.array([int(tokens[b, node])]), [length + i],
                                 pt[b:b + 1], forced=forced)
        for l, info in enumerate(ref["layers"]):
            rec = info["kv"][0]
            for pool, x in ((k, rec["k"]), (v, rec["v"])):
                pool[l, rec["page"], :, rec["slot"]] = torch.as_tensor(oracle.bf16_to_f64(x), device="cuda").to(torch.bfloat16)
        out.append(ref["logits"][0])
    return out, k, v


def paths_of(parents):
    """Root-to-leaf paths of a tree given as a list of parents."""
    leaves = [i for i in range(len(parents)) if i not in parents]
    out = []
    for leaf in leaves:
        path = [leaf]
        while parents[path[0]] >= 0:
            path.insert(0, parents[path[0]])
        out.append(path)
    return out


@pytest.mark.parametrize("model,lens,window", [("tiny", [61, 14], 0), ("tiny", [61, 14], 20), ("small", [130], 0)])
def test_verify_commit_and_decode_on(model, lens, window):
    cfg = dict(synth.MODELS[model], sliding_window=window, swa_layers=(1,) if window else (), page_size=16)
    if model == "small":
        cfg["n_layers"] = 2
    parents = [-1, 0, 0, 1, 1, 2, 3, 6, 5, 8]
    n, b = len(parents), len(lens)
    W = synth.make_weights(cfg, seed=3, device="cuda", gain_jitter=0.1)
    pt, npages = synth.make_page_table(lens, steps=n + 4, seed=1, spare=8)
    k, v = synth.make_kv(cfg, npages, seed=1, device="cuda")
    table = torch.as_tensor(pt, device="cuda")
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(5)
    tokens = torch.randint(0, cfg["vocab"], (b, n), generator=g, dtype=torch.int32).cuda()
    mask, depth = ops.tree_mask(torch.tensor([parents] * b, dtype=torch.int32, device="cuda"))
    k0, v0 = k.clone(), v.clone()
    logits, chosen = verify_pass(cfg, W, tokens, k, v, table, sl, mask, sl[:, None] + depth)
    chosen_np = [c.cpu().numpy() for c in chosen]
    pools = {}
    for s in range(b):
        for path in paths_of(parents):
            want, *pools[s, tuple(path)] = oracle_path(cfg, W, path, tokens, k0, v0, pt, s, lens[s], chosen_np)
            for node, ref in zip(path, want):
                off = float(np.abs(logits[s, node].cpu().numpy() - ref).max())
                assert off <= PU.LOGIT_ABS, (s, node, off)

    # a fork of sequence 0 first: its pages, copied to spare ones, keep the draft as it is
    used = set(pt[pt >= 0].tolist())
    spare = [p for p in range(npages) if p not in used]
    tail = [int(p) for p in pt[0, lens[0] // 16:] if p >= 0][:len(spare)]
    ops.copy_pages(k, v, tail, spare[:len(tail)])
    before = k[:, tail].clone()

    # accept another path in every sequence (node by node in path order) and decode on
    accept = [paths_of(parents)[s % len(paths_of(parents))] for s in range(b)]
    acc = torch.full((b, n), -1, dtype=torch.int32)
    for s, path in enumerate(accept):
        acc[s, :len(path)] = torch.tensor(path, dtype=torch.int32)
    status = ops.new_status()
    new = ops.commit_nodes(k, v, table, sl, acc.cuda(), status=status)
    ops.check_status(status)
    assert new.tolist() == [m + len(path) for m, path in zip(lens, accept)]
    for s, path in enumerate(accept):
        rk, rv = pools[s, tuple(path)]
        j = torch.arange(lens[s] + len(path), device="cuda")
        at = table[s].long()[j // 16], j % 16
        for mine, ref in ((k, rk), (v, rv)):
            assert torch.equal(mine[:, at[0], :, at[1]][:lens[s]], ref[:, at[0], :, at[1]][:lens[s]])
            assert PU.rel_l2(mine[:, at[0], :, at[1]].float().cpu().numpy(), ref[:, at[0], :, at[1]].float().cpu().numpy()) < PU.REL_L2
    assert torch.equal(k[:, spare[:len(tail)]], before)   # the fork did not move
    mk = B.Megakernel(cfg, W, max_batch=8)
    try:
        seq = new.tolist()
        mk.plan(seq, table, npages)
        nxt = torch.tensor([int(logits[s, path[-1]].argmax()) for s, path in enumerate(accept)], dtype=torch.int32, device="cuda")
        kv_before = (k.clone(), v.clone())
        out = torch.empty(b, cfg["vocab"], device="cuda")
        mk.step(nxt, k, v, out)
        assert mk.status()["code"] == 0
        PU.check_step(cfg, mk, W, seq, pt, kv_before, nxt.cpu().numpy(), out, k, v)
    finally:
        mk.close()


def test_prompt_chunks_equal_token_by_token():
    """A prompt of 37 tokens from an empty cache, in chunks of 20 and 17: every node's logits."""
    cfg = dict(synth.MODELS["tiny"], page_size=16)
    W = synth.make_weights(cfg, seed=4, device="cuda", gain_jitter=0.1)
    n, cut = 37, 20
    pt, npages = synth.make_page_table([0], steps=n, seed=2)
    k, v = synth.make_kv(cfg, npages, seed=2, device="cuda")
    k.fill_(float("nan")), v.fill_(float("nan"))
    table = torch.as_tensor(pt, device="cuda")
    tokens = synth.make_tokens(n, cfg["vocab"], seed=6, device="cuda")[None]
    got, chosen = [], []
    for a, b in ((0, cut), (cut, n)):
        lg, ch = verify_pass(cfg, W, tokens[:, a:b], k, v, table, torch.tensor([a], dtype=torch.int32, device="cuda"), None, None)
        got.append(lg), chosen.append(ch)
    got = torch.cat(got, 1)
    chosen = [torch.cat([c[l] for c in chosen], 1).cpu().numpy() for l in range(cfg["n_layers"])]
    want, _, _ = oracle_path(cfg, W, list(range(n)), tokens, torch.zeros_like(k), torch.zeros_like(v), pt, 0, 0, chosen)
    for i in range(n):
        off = float(np.abs(got[0, i].cpu().numpy() - want[i]).max())
        assert off <= PU.LOGIT_ABS, (i, off)
