"""Plain float64 forms of the projections, the routed layer and the verification of drafted tokens, with bounds of how far
results may be off."""
import math

import torch

import ops_ref as R

ACTS = [None, "relu", "silu", "gelu", "gelu_tanh"]


def activation(y, act):
    """(act(y), bound of its error in fp32 relative to itself, a bound of its slope)."""
    if act is None:
        return y, torch.zeros_like(y), 1.0
    if act == "relu":
        return y.clamp(min=0), torch.zeros_like(y), 1.0
    if act == "silu":
        z = y
        out = y * torch.sigmoid(y)
    elif act == "gelu":
        z = y * y           # erfc(t) changes by 2 t^2 = y^2 times a relative change of t
        out = 0.5 * y * torch.special.erfc(-y * math.sqrt(0.5))
    else:
        z = math.sqrt(8 / math.pi) * (y + 0.044715 * y ** 3)
        out = y * torch.sigmoid(z)
    # exp(-z) changes by |z| times a relative change of z, which is below 2^-22 (three roundings); exponential, error function
    # and division are good to 2^-20 each
    return out, 2.0 ** -18 + 2.0 ** -22 * z.abs(), 1.13


def linear(x, w, bias=None, act=None, residual=None, wide=False):
    """(result, bound).  Products of bf16 values are exact in fp32 and k of them are summed with a rounding or truncation each,
    at most 2^-23 of sum |x||w|; bias and residual are one addition each; the result is rounded once (bf16 2^-8, fp32 2^-24 of
    itself)."""
    x, w = x.double(), w.double()
    y = x @ w.T
    off = x.abs() @ w.abs().T * x.shape[1] * 2.0 ** -23
    if bias is not None:
        y = y + bias.double()
        off = off + 2.0 ** -23 * y.abs()
    out, rel, slope = activation(y, act)
    off = slope * off + rel * out.abs()
    if residual is not None:
        out = out + residual.double()
        off = off + 2.0 ** -23 * out.abs()
    return out, off + (2.0 ** -24 if wide else R.HALF_BF16) * (out.abs() + off) + 1e-30


def scores(x, router):
    return x.double() @ router.double().T


def select(s, k):
    """The top k of every row, ties to the lower index, NaN first; (ids, softmax weights of the selected)."""
    s = s.cpu()
    ids = []
    for line in s.tolist():
        order = sorted(range(len(line)), key=lambda e: (0 if line[e] != line[e] else 1, -line[e] if line[e] == line[e] else 0.0, e))
        ids.append(order[:k])
    ids = torch.tensor(ids, dtype=torch.int64).view(s.shape[0], k)
    top = s.gather(1, ids)
    c = (top - top[:, :1]).exp()
    return ids.cuda(), (c / c.sum(-1, keepdim=True)).cuda()


def moe(x, router, gate, up, down, k, residual=None):
    """(out, bound, ids, weights).  Gate and up as sums of k exact products (2^-23 of sum |x||w| each); their product with the
    weight is rounded to bf16 (2^-8); the second sums likewise, and one rounding of the result.  A weight comes from fp32 scores,
    off by (d / 64 + 12) 2^-24 |w| |x| at most, which changes it by twice that, and an fp32 softmax: 2^-20."""
    ids, c = select(scores(x, router), k)
    off_c = 2 * (x.shape[1] / 64 + 12) * 2.0 ** -24 * float(x.double().norm(dim=1).max() * router.double().norm(dim=1).max())
    off_c = off_c if math.isfinite(off_c) else 0.0
    x = x.double()
    t, d = x.shape
    f = gate.shape[1]
    out = torch.zeros(t, d, dtype=torch.float64, device="cuda")
    size, off = torch.zeros_like(out), torch.zeros_like(out)
    for e in range(gate.shape[0]):
        rows, slot = (ids == e).nonzero(as_tuple=True)
        if not rows.numel():
            continue
        xs, ge, ue, de = x[rows], gate[e].double(), up[e].double(), down[e].double()
        g, u = xs @ ge.T, xs @ ue.T
        dg, du = (xs.abs() @ m.abs().T * d * 2.0 ** -23 for m in (ge, ue))
        s = g * torch.sigmoid(g)
        w = c[rows, slot][:, None]
        h = w * s * u
        dh = w * (1.1 * dg * u.abs() + s.abs() * du + dg * du) + (off_c + 2.0 ** -17 + R.HALF_BF16) * h.abs()
        out[rows] += h @ de.T
        off[rows] += dh @ de.abs().T
        size[rows] += h.abs() @ de.abs().T
    off += size * (f * 2.0 ** -23 + k * 2.0 ** -23)
    if residual is not None:
        out = out + residual.double()
    return out, off * 1.01 + R.HALF_BF16 * (out.abs() + off) + 1e-30, ids, c


def verify(logits, tokens, uniforms, parents=None, draft=None, temperature=None, counts=None):
    """(accepted, next_tokens) from the definition, sequence by sequence, in float64; lists of lists and a list."""
    b, n, v = logits.shape
    path, drawn = [], []
    for i in range(b):
        m = n if counts is None else int(counts[i])
        heat = 1.0 if temperature is None else float(temperature[i])
        up = list(range(-1, n - 1)) if parents is None else parents[i].tolist()
        us, xs = uniforms[i].double().tolist(), tokens[i].tolist()
        node, walk = 0, []
        while node is not None:
            walk.append(node)
            line = logits[i, node].double()
            if heat == 0:
                p = torch.zeros_like(line)
                p[int((line == line.max()).nonzero()[0, 0])] = 1.0
            else:
                p = torch.softmax(line / heat, -1)
            step = None
            for c in range(1, m):
                if up[c] != node:
                    continue
                if draft is None:
                    q = torch.zeros_like(p)
                    q[xs[c]] = 1.0
                else:
                    q = draft[i, node].double()
                if us[c] * float(q[xs[c]]) < float(p[xs[c]]):
                    step = c
                    break
                rest = (p - q).clamp(min=0)
                if float(rest.sum()) > 0:
                    p = rest / rest.sum()
            node, last = step, p
        total = last.cumsum(0)
        drawn.append(int((total > us[0] * float(total[-1])).nonzero()[0, 0]))
        path.append(walk + [-1] * (n - len(walk)))
    return path, drawn


def tree_inputs(g, b, n, v, tree=True, probs=True, sharp=6.0, half=False):
    """Logits with a few likely tokens, parents, drafted tokens (drawn where `probs`), the drafting model's rows, uniforms."""
    logits = torch.randn(b, n, v, generator=g, device="cuda") * 2
    hot = torch.randint(0, v, (b, n, 6), generator=g, device="cuda")
    logits.scatter_add_(2, hot, sharp * torch.rand(b, n, 6, generator=g, device="cuda"))
    back = torch.randint(1, (4 if tree else 1) + 1, (b, n), generator=g, device="cuda")
    parents = (torch.arange(n, device="cuda") - back).clamp(min=0).to(torch.int32)
    parents[:, 0] = -1
    draft = (logits + 0.7 * torch.randn(b, n, v, generator=g, device="cuda")).softmax(-1)
    tokens = torch.zeros(b, n, dtype=torch.int32, device="cuda")
    rows = torch.arange(b, device="cuda")
    for i in range(1, n):
        q = draft[rows, parents[:, i].long()]
        race = torch.empty(b, v, device="cuda").exponential_(generator=g)
        tokens[:, i] = (q / race).argmax(-1).to(torch.int32)
    uniforms = torch.rand(b, n, generator=g, device="cuda")
    return (logits.to(torch.bfloat16) if half else logits), tokens, uniforms, parents, (draft if probs else None)
