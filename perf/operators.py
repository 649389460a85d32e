"""Workloads of the operators that run several tokens of a sequence at once: appending
normalised and rotated keys to the paged cache, attention of a draft tree (or of a
prompt chunk) over it, committing the accepted path, copying pages, and the products
grouped by expert.

`run(state)` computes an operator in its plain form (elementary torch operations in
float32) or, with `own` set, through the package's entry points; `exact` computes the
same from the definition in float64.  The shapes are those of the model shapes in
synth/: "tiny" (8 query heads, 2 KV heads of 32), "small" (16, 4 of 64) and "pages"
(32, 4 of 128; 48 layers; 128 experts of width 768, top-8, d_model 2048).
"""
import math

import torch

own = False

PAGE = 16
HEADS = {"tiny": (8, 2, 32), "small": (16, 4, 64), "pages": (32, 4, 128)}
THETA = {"tiny": 1e4, "small": 1e4, "pages": 1e6}
LAYERS = {"tiny": 2, "small": 8, "pages": 48}
# experts, experts per token, d_model, d_ff
EXPERTS = {"tiny": (8, 2, 256, 128), "small": (32, 4, 1024, 512), "pages": (128, 8, 2048, 768)}


def listed():
    return [
        # one sequence of the small model verifies a draft of 8 nodes: latency counts
        dict(name="tree_small_b1", op="tree", model="small", batch=1, nodes=8, lo=2048, hi=2048, window=0, tree=True, ragged=False),
        # a ragged batch of the pages-scale model verifies 16 nodes each, some sequences fewer
        dict(name="tree_pages_b8", op="tree", model="pages", batch=8, nodes=16, lo=1024, hi=32768, window=0, tree=True, ragged=True),
        # a prompt chunk of odd length after 8K cached tokens: the tensor cores are the bound
        dict(name="chunk_pages_b1", op="tree", model="pages", batch=1, nodes=2001, lo=8192, hi=8192, window=0, tree=False, ragged=False),
        # the keys of a verification step of 8 sequences, and of a prompt chunk
        dict(name="rope_pages_b8", op="rope", model="pages", batch=8, nodes=16, lo=1024, hi=32768, norm=True, ragged=True),
        dict(name="rope_chunk_b2", op="rope", model="pages", batch=2, nodes=4001, lo=0, hi=90000, norm=True, ragged=False),
        # forks of 8 sequences copy one tail page each; a whole 8K sequence is moved
        dict(name="copy_pages_8", op="copy", model="pages", pages=8, pool=64),
        dict(name="copy_pages_512", op="copy", model="pages", pages=512, pool=1100),
        # the accepted path of a draft, one small sequence and a batch of the pages-scale model
        dict(name="commit_small_b1", op="commit", model="small", batch=1, nodes=8, accept=4, lo=200, hi=300),
        dict(name="commit_pages_b8", op="commit", model="pages", batch=8, nodes=64, accept=16, lo=100, hi=400),
        # the down product of 2 sequences' single tokens; the gate/up products of a
        # verification step (128 tokens, top-8) and of a prompt chunk
        dict(name="down_pages_t2", op="experts", model="pages", tokens=2, glu=False),
        dict(name="glu_pages_t128", op="experts", model="pages", tokens=128, glu=True),
        dict(name="glu_pages_t4096", op="experts", model="pages", tokens=4096, glu=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "rope", "copy", "commit", "experts", "experts"])
    model = rng.choice(["tiny", "small", "pages", "pages"])
    if op == "tree":
        hi = _log(rng, 1, 33000)
        lo = rng.randint(0, hi)
        tree = rng.random() < 0.7
        batch = rng.randint(1, 8)
        nodes = _log(rng, 1, 64) if tree else _log(rng, 1, 1500)
        if nodes > 64:
            batch, lo, hi = 1, min(lo, 8000), min(hi, 8000)
        return dict(op=op, model=model, batch=batch, nodes=nodes, lo=lo, hi=hi, window=rng.choice([0, 0, _log(rng, 1, 5000)]),
                    tree=tree, ragged=rng.random() < 0.5)
    if op == "rope":
        hi = _log(rng, 1, 100000)
        return dict(op=op, model=model, batch=rng.randint(1, 8 if hi < 25000 else 2), nodes=_log(rng, 1, 900), lo=rng.randint(0, hi), hi=hi,
                    norm=rng.random() < 0.7, ragged=rng.random() < 0.5)
    if op == "copy":
        pages = _log(rng, 1, 400)
        return dict(op=op, model=model, pages=pages, pool=2 * pages + rng.randint(0, 50))
    if op == "commit":
        nodes = _log(rng, 1, 100)
        return dict(op=op, model=model, batch=rng.randint(1, 8), nodes=nodes, accept=rng.randint(1, min(nodes, 40)),
                    lo=rng.randint(0, 100), hi=rng.randint(100, 500))
    return dict(op=op, model=model, tokens=_log(rng, 1, 3000), glu=rng.random() < 0.5)


# ------------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _ints(g, lo, hi, shape):
    """int64 uniform in [lo, hi]."""
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda")


def _bf16(g, *shape, std=1.0):
    return torch.empty(*shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=g)


def _paged(g, case, layers):
    """Pools, page table and lengths of a batch whose lengths lie in [lo, hi], with room for the nodes."""
    _, hkv, hd = HEADS[case["model"]]
    b, cap = case["batch"], case["hi"] + case["nodes"]
    per = -(-cap // PAGE)
    lens = _ints(g, case["lo"], case["hi"], (b,))
    table = torch.randperm(b * per, generator=g, device="cuda").view(b, per).to(torch.int32)
    k = _bf16(g, layers, b * per, hkv, PAGE, hd)
    v = _bf16(g, layers, b * per, hkv, PAGE, hd)
    return dict(k=k, v=v, table=table, lens=lens.to(torch.int32))


def _counts(g, case):
    if not case["ragged"]:
        return None
    return _ints(g, max(1, case["nodes"] // 2), case["nodes"], (case["batch"],)).to(torch.int32)


def _tree(g, batch, nodes):
    """A random tree per sequence: (visibility words, depth of each node).  Every node's parent comes before it,
    near it, so that the trees are neither chains nor stars."""
    back = _ints(g, 1, 4, (batch, nodes))
    parent = torch.arange(nodes, device="cuda") - back
    sees = torch.eye(nodes, dtype=torch.bool, device="cuda").repeat(batch, 1, 1)
    up = sees | (parent.clamp(min=0)[:, :, None] == torch.arange(nodes, device="cuda")) & (parent >= 0)[:, :, None]
    for _ in range(max(1, (nodes - 1).bit_length())):
        sees = up
        up = (sees.float() @ sees.float()) > 0
    depth = up.sum(-1) - 1
    words = -(-nodes // 32)
    bits = torch.zeros(batch, nodes, words * 32, dtype=torch.int64, device="cuda")
    bits[:, :, :nodes] = up
    w = (bits.view(batch, nodes, words, 32) << torch.arange(32, device="cuda")).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32), depth.to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    op, model = case["op"], case["model"]
    if op in ("tree", "rope"):
        hq, hkv, hd = HEADS[model]
        b, n = case["batch"], case["nodes"]
        s.update(_paged(g, case, 1))
        s["counts"] = _counts(g, case)
        s["positions"] = s["mask"] = None
        if op == "tree":
            if case["tree"]:
                s["mask"], depth = _tree(g, b, n)
                s["positions"] = s["lens"][:, None] + depth
            s["q"] = _bf16(g, b, n, hq, hd, std=1.5)
        else:
            qkv = _bf16(g, b, n, hq + 2 * hkv, hd)  # the packed result of one projection
            s["q"], s["kn"], s["vn"] = qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:]
            _, depth = _tree(g, b, n) if n <= 64 else (None, torch.arange(n, dtype=torch.int32, device="cuda").repeat(b, 1))
            s["positions"] = s["lens"][:, None] + depth
            s["gq"] = s["gk"] = None
            if case["norm"]:
                s["gq"], s["gk"] = (1 + _bf16(g, hd, std=0.1) for _ in range(2))
        s["out"] = torch.zeros(b, n, hq, hd, dtype=torch.bfloat16, device="cuda")
    elif op == "copy":
        _, hkv, hd = HEADS[model]
        s["k"], s["v"] = (_bf16(g, LAYERS[model], case["pool"], hkv, PAGE, hd) for _ in range(2))
        ids = torch.randperm(case["pool"], generator=g, device="cuda").cpu().tolist()
        s["src"], s["dst"] = ids[:case["pages"]], ids[case["pages"]:2 * case["pages"]]
    elif op == "commit":
        b, n, a = case["batch"], case["nodes"], case["accept"]
        s.update(_paged(g, case, LAYERS[model]))
        order = torch.rand(b, n, generator=g, device="cuda").argsort(-1)[:, :a].sort(-1).values
        keep = torch.arange(a, device="cuda") < _ints(g, (a + 1) // 2, a, (b, 1))
        s["accepted"] = torch.where(keep, order, -1).to(torch.int32)
    else:
        e, k, d, f = EXPERTS[model]
        t = case["tokens"]
        logits = torch.randn(t, e, generator=g, device="cuda") + 0.3 * torch.randn(e, generator=g, device="cuda")
        chosen = logits.topk(k, -1).indices.reshape(-1)
        order = chosen.argsort(stable=True)
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), torch.bincount(chosen, minlength=e).cumsum(0)]).to(torch.int32)
        s["most"] = int(torch.bincount(chosen, minlength=e).max())
        if case["glu"]:
            s["x"] = _bf16(g, t, d)
            s["rows"] = (order // k).to(torch.int32)
            s["w"], s["w_up"] = (_bf16(g, e, f, d, std=0.02) for _ in range(2))
        else:
            s["x"] = _bf16(g, t * k, f)
            s["rows"] = s["w_up"] = None
            s["w"] = _bf16(g, e, d, f, std=0.02)
    return s


# ------------------------------------------------------------------ the operators

def run(s):
    op = s["case"]["op"]
    if own:
        from persistent_moe_decode_cta_gb300 import ops
        if op == "tree":
            return ops.tree_attention(s["q"], s["k"][0], s["v"][0], s["table"], s["lens"], mask=s["mask"], positions=s["positions"],
                                      counts=s["counts"], window=s["case"]["window"], out=s["out"])
        if op == "rope":
            out = ops.qk_norm_rope(s["q"], s["kn"], s["vn"], s["k"][0], s["v"][0], s["table"], s["lens"], theta=THETA[s["case"]["model"]],
                                   q_gain=s["gq"], k_gain=s["gk"], positions=s["positions"], counts=s["counts"], out=s["out"])
            return [out, s["k"], s["v"]]
        if op == "copy":
            ops.copy_pages(s["k"], s["v"], s["src"], s["dst"])
            return [s["k"], s["v"]]
        if op == "commit":
            return [ops.commit_nodes(s["k"], s["v"], s["table"], s["lens"], s["accepted"]), s["k"], s["v"]]
        return ops.expert_product(s["x"], s["w"], s["offsets"], w_up=s["w_up"], rows=s["rows"])
    return {"tree": _plain_tree, "rope": _plain_rope, "copy": _plain_copy, "commit": _plain_commit, "experts": _plain_experts}[op](s)


def _plain_tree(s):
    q, table, lens = s["q"], s["table"].long(), s["lens"].long()
    b, n, hq, hd = q.shape
    hkv = s["k"].shape[2]
    keys = table.shape[1] * PAGE
    # [B, Hkv, keys, hd]
    k, v = (x[0][table].permute(0, 2, 1, 3, 4).reshape(b, hkv, keys, hd).float() for x in (s["k"], s["v"]))
    node = torch.arange(n, device="cuda")
    j = torch.arange(keys, device="cuda")
    counts = s["counts"].long() if s["counts"] is not None else torch.full((b,), n, device="cuda")
    pos = s["positions"].long() if s["positions"] is not None else lens[:, None] + node
    a = j[None] - lens[:, None]                                        # node index of a key, negative for cached ones
    at = a.clamp(0, n - 1)
    if s["mask"] is not None:
        word = s["mask"].long().gather(2, (at // 32)[:, None].expand(b, n, keys))
        seen = (word >> (at % 32)[:, None]) & 1 == 1
    else:
        seen = at[:, None] <= node[:, None]
    key_pos = torch.where(a < 0, j[None], pos.gather(1, at))
    seen = ((a < 0)[:, None] | seen) & (a < counts[:, None])[:, None]
    if s["case"]["window"]:
        seen = seen & (key_pos[:, None] > pos[:, :, None] - s["case"]["window"])
    grp = hq // hkv
    x = q.float().view(b, n, hkv, grp, hd).permute(0, 2, 3, 1, 4).reshape(b, hkv, grp * n, hd)
    score = (x @ k.transpose(2, 3)).view(b, hkv, grp, n, keys).mul_(hd ** -0.5)
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(b, hkv, grp * n, keys) @ v).view(b, hkv, grp, n, hd) / torch.where(total == 0, 1.0, total)
    o = o.permute(0, 3, 1, 2, 4).reshape(b, n, hq, hd).to(torch.bfloat16)
    s["out"].copy_(torch.where((node < counts[:, None])[:, :, None, None], o, s["out"]))
    return s["out"]


def _slots(s, n):
    """(page, slot) of node i of every sequence, [B, n]."""
    at = s["lens"].long()[:, None] + torch.arange(n, device="cuda")
    return s["table"].long().gather(1, at // PAGE), at % PAGE


def _plain_rope(s):
    b, n, _, hd = s["q"].shape
    turn = s["positions"].double()[:, :, None] * THETA[s["case"]["model"]] ** (-2 * torch.arange(hd // 2, device="cuda", dtype=torch.float64) / hd)
    cos, sin = turn.cos().float()[:, :, None], turn.sin().float()[:, :, None]

    def turned(x, gain):
        x = x.float()
        if gain is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * gain.float()
        lo, hi = x[..., :hd // 2], x[..., hd // 2:]
        return torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], -1).to(torch.bfloat16)

    real = torch.arange(n, device="cuda") < (s["counts"].long()[:, None] if s["counts"] is not None else n)
    real = real.expand(b, n)
    page, slot = _slots(s, n)
    kept = real[:, :, None, None]
    s["out"].copy_(torch.where(kept, turned(s["q"], s["gq"]), s["out"]))
    for pool, new in ((s["k"][0], turned(s["kn"], s["gk"])), (s["v"][0], s["vn"])):
        pool[page, :, slot] = torch.where(kept, new, pool[page, :, slot])
    return [s["out"], s["k"], s["v"]]


def _plain_copy(s):
    src, dst = (torch.tensor(x, device="cuda") for x in (s["src"], s["dst"]))
    for pool in (s["k"], s["v"]):
        pool[:, dst] = pool[:, src]
    return [s["k"], s["v"]]


def _plain_commit(s):
    acc = s["accepted"].long()
    keep = acc >= 0
    at = s["lens"].long()[:, None] + acc.clamp(min=0)
    page, slot = s["table"].long().gather(1, at // PAGE), at % PAGE
    to_page, to_slot = _slots(s, acc.shape[1])
    for pool in (s["k"], s["v"]):
        old = pool[:, to_page, :, to_slot]
        pool[:, to_page, :, to_slot] = torch.where(keep[:, :, None, None, None], pool[:, page, :, slot], old)
    return [s["lens"] + keep.sum(1).to(torch.int32), s["k"], s["v"]]


def _plain_experts(s):
    x = s["x"] if s["rows"] is None else s["x"][s["rows"].long()]
    first = s["offsets"].long()
    col = torch.arange(s["most"], device="cuda")
    at = first[:-1, None] + col                                        # [E, most]
    real = at < first[1:, None]
    xs = x[at.clamp(max=x.shape[0] - 1)].float()
    y = xs @ s["w"].float().transpose(1, 2)
    if s["w_up"] is not None:
        y = y / (1 + (-y).exp()) * (xs @ s["w_up"].float().transpose(1, 2))
    return y[real].to(torch.bfloat16)                                  # rows in order of expert


# ------------------------------------------------------------------------- sizes

def _expected_keys(case):
    """Keys that one node of an average sequence attends to."""
    mean = (case["lo"] + case["hi"]) / 2
    return min(mean, case["window"]) if case["window"] else mean


def work(case):
    op, model = case["op"], case["model"]
    hq, hkv, hd = HEADS[model]
    if op == "tree":
        b = case["batch"]
        n = case["nodes"] * (0.75 if case["ragged"] else 1.0)
        cached, own_keys = _expected_keys(case), n / 2
        span = cached + n
        return {"bytes": b * (2 * span * hkv * hd + 2 * n * hq * hd) * 2, "flops": 4.0 * b * n * hq * hd * (cached + own_keys)}
    if op == "rope":
        n = case["batch"] * case["nodes"] * (0.75 if case["ragged"] else 1.0)
        return {"bytes": n * (2 * hq + 4 * hkv) * hd * 2, "flops": n * (hq + hkv) * hd * 8.0}
    if op == "copy":
        return {"bytes": 2.0 * 2 * LAYERS[model] * case["pages"] * hkv * PAGE * hd * 2, "flops": 0.0}
    if op == "commit":
        return {"bytes": 2.0 * 2 * LAYERS[model] * case["batch"] * 0.75 * case["accept"] * hkv * hd * 2, "flops": 0.0}
    e, k, d, f = EXPERTS[model]
    rows = case["tokens"] * k
    active = e * (1 - (1 - k / e) ** case["tokens"])
    if case["glu"]:
        return {"bytes": (active * 2 * d * f + case["tokens"] * d + rows * f) * 2, "flops": 4.0 * rows * d * f}
    return {"bytes": (active * d * f + rows * (d + f)) * 2, "flops": 2.0 * rows * d * f}


# -------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "tree":
        return _exact_tree(s)
    if op == "rope":
        return _exact_rope(s)
    if op == "copy":
        for a, b in zip(s["src"], s["dst"]):
            s["k"][:, b].copy_(s["k"][:, a])
            s["v"][:, b].copy_(s["v"][:, a])
        return [s["k"], s["v"]]
    if op == "commit":
        return _exact_commit(s)
    return _exact_experts(s)


def _sequence(s, b, total):
    """K and V of sequence b, [total, Hkv, hd] float64."""
    pages = s["table"][b, :-(-total // PAGE)].long()
    return (x[0].index_select(0, pages).transpose(1, 2).flatten(0, 1)[:total].double() for x in (s["k"], s["v"]))


def _exact_tree(s):
    q, out = s["q"].double(), s["out"].double()
    b, n, hq, hd = q.shape
    w = s["case"]["window"]
    for i in range(b):
        length = int(s["lens"][i])
        m = int(s["counts"][i]) if s["counts"] is not None else n
        k, v = _sequence(s, i, length + m)
        pos = s["positions"][i, :m].long() if s["positions"] is not None else torch.arange(length, length + m, device="cuda")
        sees = torch.ones(m, length + m, dtype=torch.bool, device="cuda")
        if s["mask"] is not None:
            bit = torch.arange(m, device="cuda")
            sees[:, length:] = (s["mask"][i, :m].long()[:, bit // 32] >> (bit % 32)) % 2 != 0
        else:
            sees = sees.tril(length)
        if w:
            at = torch.cat([torch.arange(length, device="cuda"), pos])
            sees &= pos[:, None] - at[None] < w
        for h in range(hq):
            kv = h * k.shape[1] // hq
            z = q[i, :m, h] @ k[:, kv].T / math.sqrt(hd)
            out[i, :m, h] = z.masked_fill(~sees, -math.inf).softmax(-1) @ v[:, kv]
    return out


def _exact_rope(s):
    b, n, hq, hd = s["q"].shape
    freq = torch.tensor([THETA[s["case"]["model"]] ** (-2.0 * i / hd) for i in range(hd // 2)], dtype=torch.float64, device="cuda")
    spin = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), s["positions"].double()[..., None] * freq)[:, :, None]

    def turned(x, gain):
        x = x.double()
        if gain is not None:
            x = x / (x.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * gain.double()
        z = torch.complex(x[..., :hd // 2], x[..., hd // 2:]) * spin
        return torch.cat([z.real, z.imag], -1)

    q, kn, vn = turned(s["q"], s["gq"]), turned(s["kn"], s["gk"]), s["vn"].double()
    out, k, v = s["out"].double(), s["k"].double(), s["v"].double()
    for i in range(b):
        m = int(s["counts"][i]) if s["counts"] is not None else n
        out[i, :m] = q[i, :m]
        at = torch.arange(m, device="cuda") + int(s["lens"][i])
        page = s["table"][i].long()[at // PAGE]
        k[0, page, :, at % PAGE] = kn[i, :m]
        v[0, page, :, at % PAGE] = vn[i, :m]
    return [out, k, v]


def _exact_commit(s):
    lens = s["lens"].clone()
    acc, first, table = s["accepted"].tolist(), s["lens"].tolist(), s["table"].tolist()
    for b, path in enumerate(acc):
        path = [a for a in path if a >= 0]
        lens[b] += len(path)
        for pool in (s["k"], s["v"]):
            kept = [pool[:, table[b][(first[b] + a) // PAGE], :, (first[b] + a) % PAGE].clone() for a in path]
            for i, row in enumerate(kept):
                at = first[b] + i
                pool[:, table[b][at // PAGE], :, at % PAGE] = row
    return [lens, s["k"], s["v"]]


def _exact_experts(s):
    x = s["x"].double()
    ends = s["offsets"].tolist()
    parts = []
    for e in range(len(ends) - 1):
        mine = x[ends[e]:ends[e + 1]] if s["rows"] is None else x[s["rows"][ends[e]:ends[e + 1]].long()]
        y = mine @ s["w"][e].double().T
        if s["w_up"] is not None:
            y = y * torch.sigmoid(y) * (mine @ s["w_up"][e].double().T)
        parts.append(y)
    return torch.cat(parts)
