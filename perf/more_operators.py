"""Workloads of the operators that complete a verification step of drafted tokens: the
projections with bias, activation and residual in one product, the whole mixture-of-experts
layer of a few tokens, and the verification of the drafted tokens against the target's
probabilities from given random numbers.

`run(state)` computes an operator in its plain form (elementary torch operations) or, with
`own` set, through the package's entry points; `exact` computes the same from the definition
in float64.  The shapes are those of the model shapes in synth/: "tiny" (d_model 256, 8
experts of width 128, top-2, 1024 tokens of vocabulary), "small" (1024, 32 of 512, top-4,
32000) and "pages" (2048, 128 of 768, top-8, 151936; dense layers of width 4096).
"""
import math

import torch

own = False

# experts, experts per token, d_model, d_ff
EXPERTS = {"tiny": (8, 2, 256, 128), "small": (32, 4, 1024, 512), "pages": (128, 8, 2048, 768)}
VOCAB = {"tiny": 1024, "small": 32000, "pages": 151936}
# (n, k) of the projections: queries, keys and values together; attention output; a dense layer's first and second
# product; the LM head
SHAPES = {"tiny": dict(qkv=(384, 256), o=(256, 256), up=(256, 256), down=(256, 256), lm=(1024, 256)),
          "small": dict(qkv=(1536, 1024), o=(1024, 1024), up=(1024, 1024), down=(1024, 1024), lm=(32000, 1024)),
          "pages": dict(qkv=(5120, 2048), o=(2048, 4096), up=(4096, 2048), down=(2048, 4096), lm=(151936, 2048))}


def listed():
    return [
        # one token of the small model, and of the pages-scale model: a chain of dependent products where latency counts
        dict(name="moe_small_t1", op="moe", model="small", tokens=1, lean=0.5, residual=True),
        dict(name="moe_pages_t1", op="moe", model="pages", tokens=1, lean=0.5, residual=True),
        # two sequences verify 8 nodes each; eight sequences 16 nodes each, which select every expert
        dict(name="moe_pages_t16", op="moe", model="pages", tokens=16, lean=0.5, residual=True),
        dict(name="moe_pages_t128", op="moe", model="pages", tokens=128, lean=0.5, residual=False),
        # five nodes of the small model through its first projection: latency
        dict(name="linear_small_m5", op="linear", m=5, n=1536, k=1024, bias=True, act=None, residual=False, wide=False),
        # the attention output of a verification step of 128 nodes, added to the residual
        dict(name="linear_pages_o_m128", op="linear", m=128, n=2048, k=4096, bias=False, act=None, residual=True, wide=False),
        # the LM head of eight sequences of nine nodes, logits in float32
        dict(name="linear_pages_lm_m72", op="linear", m=72, n=151936, k=2048, bias=False, act=None, residual=False, wide=True),
        # a dense layer's first product for a prompt chunk of odd length
        dict(name="linear_pages_up_m2001", op="linear", m=2001, n=4096, k=2048, bias=True, act="gelu_tanh", residual=False, wide=False),
        # one sequence of the small model with four drafted tokens in a chain
        dict(name="verify_small_b1", op="verify", vocab=32000, batch=1, nodes=5, tree=False, probs=True, half=False, ragged=False, greedy=0.0),
        # eight sequences with eight drafted tokens each, drawn from the drafting model's probabilities
        dict(name="verify_pages_b8", op="verify", vocab=151936, batch=8, nodes=9, tree=False, probs=True, half=False, ragged=False, greedy=0.0),
        # trees of drafted tokens without probabilities (a lookup proposed them), some sequences greedy, bfloat16 logits
        dict(name="verify_pages_tree_b8", op="verify", vocab=151936, batch=8, nodes=16, tree=True, probs=False, half=True, ragged=True, greedy=0.25),
        # the largest: sixteen trees of 32 nodes drawn from probabilities
        dict(name="verify_pages_tree_b16", op="verify", vocab=151936, batch=16, nodes=32, tree=True, probs=True, half=False, ragged=True, greedy=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["moe", "linear", "verify"])
    model = rng.choice(["tiny", "small", "pages", "pages"])
    if op == "moe":
        return dict(op=op, model=model, tokens=_log(rng, 1, 256), lean=round(rng.random(), 3), residual=rng.random() < 0.7)
    if op == "linear":
        if rng.random() < 0.6:
            what = rng.choice(sorted(SHAPES[model]))
            n, k = SHAPES[model][what]
            m = _log(rng, 1, 72 if what == "lm" else 2500)
        else:
            n, k, m = _log(rng, 1, 6000), 8 * _log(rng, 1, 700), _log(rng, 1, 1500)
        return dict(op=op, m=m, n=n, k=k, bias=rng.random() < 0.5, act=rng.choice([None, "relu", "silu", "gelu", "gelu_tanh"]),
                    residual=rng.random() < 0.5, wide=rng.random() < 0.3)
    nodes = _log(rng, 1, 32)
    vocab = VOCAB[model] if rng.random() < 0.7 else _log(rng, 2, 150000)
    return dict(op=op, vocab=vocab, batch=rng.randint(1, max(1, min(16, 256 // nodes))), nodes=nodes, tree=rng.random() < 0.5,
                probs=rng.random() < 0.6, half=rng.random() < 0.3, ragged=rng.random() < 0.5, greedy=rng.choice([0.0, 0.3]))


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


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    if case["op"] == "moe":
        e, _, d, f = EXPERTS[case["model"]]
        t = case["tokens"]
        s["x"] = _bf16(g, t, d)
        # rows of different size: the more the routing leans, the more often some experts are chosen
        size = 0.02 * (1 + case["lean"] * (torch.rand(e, 1, generator=g, device="cuda") - 0.5))
        s["router"] = (torch.randn(e, d, generator=g, device="cuda") * size).to(torch.bfloat16)
        s["gate"], s["up"] = (_bf16(g, e, f, d, std=0.02) for _ in range(2))
        s["down"] = _bf16(g, e, d, f, std=0.02)
        s["residual"] = _bf16(g, t, d) if case["residual"] else None
    elif case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        s["x"], s["w"] = _bf16(g, m, k), _bf16(g, n, k, std=0.02)
        s["bias"] = _bf16(g, n, std=0.1) if case["bias"] else None
        s["residual"] = _bf16(g, m, n) if case["residual"] else None
    else:
        b, n, v = case["batch"], case["nodes"], case["vocab"]
        # a few likely tokens over a long tail
        logits = torch.randn(b, n, v, generator=g, device="cuda").mul_(2.5)
        at = _ints(g, 0, v - 1, (b, n, 8))
        logits.scatter_add_(2, at, 5 + 5 * torch.rand(b, n, 8, generator=g, device="cuda"))
        back = _ints(g, 1, 3 if case["tree"] else 1, (b, n))
        s["parents"] = (torch.arange(n, device="cuda") - back).clamp(min=0).to(torch.int32)
        s["parents"][:, 0] = -1
        # the drafting model's opinion of every node's next token, and the tokens drawn from it
        draft = torch.empty_like(logits).normal_(generator=g).mul_(0.5).add_(logits).softmax(-1)
        parent = s["parents"].long().clamp(min=0)
        s["tokens"] = _ints(g, 0, v - 1, (b, n)).to(torch.int32)
        for i in range(1, n):
            race = torch.empty(b, v, device="cuda").exponential_(generator=g)
            s["tokens"][:, i] = (draft[torch.arange(b, device="cuda"), parent[:, i]] / race).argmax(-1).to(torch.int32)
        s["logits"] = logits.to(torch.bfloat16) if case["half"] else logits
        s["probs"] = draft if case["probs"] else None
        s["uniforms"] = torch.rand(b, n, generator=g, device="cuda")
        temperature = 0.7 + 0.6 * torch.rand(b, generator=g, device="cuda")
        s["temperature"] = torch.where(torch.rand(b, generator=g, device="cuda") < case["greedy"], 0.0, temperature)
        s["counts"] = _ints(g, (n + 1) // 2, n, (b,)).to(torch.int32) if case["ragged"] else None
    return s


# ------------------------------------------------------------------ the operators

def run(s):
    case = s["case"]
    if own:
        from persistent_moe_decode_cta_gb300 import ops
        if case["op"] == "moe":
            return ops.moe_layer(s["x"], s["router"], s["gate"], s["up"], s["down"], EXPERTS[case["model"]][1], residual=s["residual"])
        if case["op"] == "linear":
            return ops.linear(s["x"], s["w"], bias=s["bias"], activation=case["act"], residual=s["residual"],
                              dtype=torch.float32 if case["wide"] else torch.bfloat16)
        return list(ops.verify_nodes(s["logits"], s["tokens"], s["uniforms"], parents=s["parents"], draft_probs=s["probs"],
                                     temperature=s["temperature"], counts=s["counts"]))
    return {"moe": _plain_moe, "linear": _plain_linear, "verify": _plain_verify}[case["op"]](s)


def _plain_moe(s):
    e, k, _, _ = EXPERTS[s["case"]["model"]]
    t = s["x"].shape[0]
    scores = s["x"].double() @ s["router"].double().T      # (a selection can hang on the last bits)
    top, ids = torch.sort(scores, dim=-1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    share = (top - top[:, :1]).exp()
    share = (share / share.sum(-1, keepdim=True)).float()
    x = s["x"].float()
    if t * k <= e:     # the chosen experts' matrices, a product per token and expert
        chosen = ids.reshape(-1)
        xs = x.repeat_interleave(k, 0)[:, :, None]
        g, u = s["gate"][chosen].float() @ xs, s["up"][chosen].float() @ xs
        y = s["down"][chosen].float() @ (g / (1 + (-g).exp()) * u)
        y = (y.view(t, k, -1) * share[:, :, None]).sum(1)
    else:              # every expert for every token, unchosen ones with weight 0
        weight = torch.zeros(t, e, device="cuda").scatter_(1, ids, share)
        g, u = x @ s["gate"].float().transpose(1, 2), x @ s["up"].float().transpose(1, 2)
        h = g / (1 + (-g).exp()) * u * weight.T[:, :, None]
        y = (h @ s["down"].float().transpose(1, 2)).sum(0)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(torch.bfloat16)


def _plain_linear(s):
    y = s["x"].float() @ s["w"].float().T
    if s["bias"] is not None:
        y = y + s["bias"].float()
    act = s["case"]["act"]
    if act == "relu":
        y = y.clamp(min=0)
    elif act == "silu":
        y = y / (1 + (-y).exp())
    elif act == "gelu":
        y = 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    elif act == "gelu_tanh":
        y = 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y if s["case"]["wide"] else y.to(torch.bfloat16)


def _plain_verify(s):
    """Every node's distribution, cut by its drafted children one after another; then the walk from the root.
    In 64 bits: a token is drawn where a sum of up to 150000 terms passes a number."""
    logits, tokens, parents = s["logits"].double(), s["tokens"].long(), s["parents"].long()
    b, n, v = logits.shape
    row = torch.arange(b, device="cuda")
    heat = s["temperature"].double()[:, None, None]
    top = logits.amax(-1, keepdim=True)
    place = torch.arange(v, device="cuda")
    first = torch.where(logits == top, place, v).amin(-1, keepdim=True)      # (of equal ones the lowest)
    left = ((logits - top) / torch.where(heat == 0, 1.0, heat)).exp()
    left = torch.where(heat == 0, (place == first).double(), left / left.sum(-1, keepdim=True))
    counts = s["counts"].long() if s["counts"] is not None else torch.full((b,), n, device="cuda")
    child = torch.full((b, n), -1, device="cuda")                            # the child that is accepted
    for i in range(1, n):
        up = parents[:, i]
        p = left[row, up]
        if s["probs"] is not None:
            q = s["probs"][row, up].double()
        else:
            q = (place == tokens[:, i, None]).double()
        mine = tokens[:, i, None]
        live = (i < counts) & (child[row, up] < 0)
        taken = live & (s["uniforms"][:, i].double() * q.gather(1, mine)[:, 0] < p.gather(1, mine)[:, 0])
        child[row, up] = torch.where(taken, i, child[row, up])
        rest = (p - q).clamp(min=0)
        total = rest.sum(-1, keepdim=True)
        rest = torch.where(total > 0, rest / total, p)
        left[row, up] = torch.where((live & ~taken)[:, None], rest, p)
    at = torch.zeros(b, dtype=torch.int64, device="cuda")
    going = torch.ones(b, dtype=torch.bool, device="cuda")
    accepted = torch.full((b, n), -1, device="cuda")
    for j in range(n):
        accepted[:, j] = torch.where(going, at, -1)
        nxt = child[row, at]
        going = going & (nxt >= 0)
        at = torch.where(going, nxt, at)
    total = left[row, at].cumsum(-1)
    drawn = torch.where(total > s["uniforms"][:, :1].double() * total[:, -1:], place, v).amin(-1)
    return [accepted.to(torch.int32), drawn.to(torch.int32)]


# ------------------------------------------------------------------------- sizes

def work(case):
    if case["op"] == "moe":
        e, k, d, f = EXPERTS[case["model"]]
        t = case["tokens"]
        active = e * (1 - (1 - k / e) ** t)
        return {"bytes": 2.0 * (active * 3 * d * f + e * d + t * d * (3 if case["residual"] else 2)), "flops": 2.0 * t * (k * 3 * d * f + e * d)}
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": 2.0 * (m * k + n * k + (n if case["bias"] else 0) + (m * n if case["residual"] else 0)) + (4.0 if case["wide"] else 2.0) * m * n,
                "flops": 2.0 * m * n * k}
    b, n, v = case["batch"], case["nodes"], case["vocab"]
    rows = b * n * (0.75 if case["ragged"] else 1.0)
    # the target's row of every node; the drafting model's of every node that has children (a chain: all but the last)
    inner = (rows - b) * (0.65 if case["tree"] else 1.0) if n > 1 else 0.0
    return {"bytes": rows * v * (2 if case["half"] else 4) + (inner * v * 4 if case["probs"] else 0.0), "flops": 10.0 * rows * v}


# -------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"moe": _exact_moe, "linear": _exact_linear, "verify": _exact_verify}[case["op"]](s)


def _exact_moe(s):
    e, k, _, _ = EXPERTS[s["case"]["model"]]
    x = s["x"].double()
    scores = torch.einsum("td,ed->te", x, s["router"].double()).cpu()
    y = torch.zeros_like(x) if s["residual"] is None else s["residual"].double()
    mine = [([], []) for _ in range(e)]
    for t, line in enumerate(scores.tolist()):
        chosen = sorted(range(e), key=lambda i: (-line[i], i))[:k]
        part = [math.exp(line[i] - line[chosen[0]]) for i in chosen]
        for i, w in zip(chosen, part):
            mine[i][0].append(t)
            mine[i][1].append(w / math.fsum(part))
    for i, (rows, parts) in enumerate(mine):
        if rows:
            xs = x[rows]
            g = xs @ s["gate"][i].double().T
            h = g * torch.sigmoid(g) * (xs @ s["up"][i].double().T)
            y[rows] += torch.tensor(parts, dtype=torch.float64, device="cuda")[:, None] * (h @ s["down"][i].double().T)
    return y


def _exact_linear(s):
    y = torch.nn.functional.linear(s["x"].double(), s["w"].double(), None if s["bias"] is None else s["bias"].double())
    f = torch.nn.functional
    act = {None: lambda z: z, "relu": f.relu, "silu": f.silu, "gelu": f.gelu, "gelu_tanh": lambda z: f.gelu(z, approximate="tanh")}
    y = act[s["case"]["act"]](y)
    return y if s["residual"] is None else y + s["residual"].double()


def _exact_verify(s):
    """One sequence after another, from its root on."""
    b, n, v = s["logits"].shape
    path = torch.full((b, n), -1, dtype=torch.int32)
    drawn = torch.zeros(b, dtype=torch.int32)
    parents, tokens, us = s["parents"].tolist(), s["tokens"].tolist(), s["uniforms"].double().tolist()
    for i in range(b):
        m = int(s["counts"][i]) if s["counts"] is not None else n
        heat = float(s["temperature"][i])
        node, length = 0, 0
        while True:
            path[i, length] = node
            length += 1
            line = s["logits"][i, node].double()
            if heat == 0:
                p = torch.zeros_like(line)
                p[int((line == line.max()).nonzero()[0, 0])] = 1.0
            else:
                p = torch.softmax(line / heat, -1)
            step = None
            for c in range(1, m):
                if parents[i][c] != node:
                    continue
                x = tokens[i][c]
                if s["probs"] is not None:
                    q = s["probs"][i, node].double()
                else:
                    q = torch.zeros_like(p)
                    q[x] = 1.0
                if us[i][c] * float(q[x]) < float(p[x]):
                    step = c
                    break
                r = torch.relu(p - q)
                if float(r.sum()) > 0:
                    p = r / r.sum()
            if step is None:
                break
            node = step
        c = torch.cumsum(p, 0)
        drawn[i] = int((c > us[i][0] * float(c[-1])).nonzero()[0, 0])
    return [path, drawn]
