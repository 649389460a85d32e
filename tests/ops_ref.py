"""Plain float64 forms of the multi-token operators, and inputs for their tests."""
import math

import torch

PAGE = 16
HALF_BF16 = 2.0 ** -8   # a rounding to bf16 is off by at most this, relative to the value


def bf16(g, *shape, std=1.0):
    return torch.empty(*shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=g)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def cache(g, lens, room, hkv, hd, layers=None, spare=3, fill=None):
    """Pools, page table and lengths: `room` slots behind every sequence.  Pages in random
    order; unused table entries are -1.  fill: the value of every slot that holds no cached
    token (None: random, like the rest)."""
    need = [-(-(n + room) // PAGE) for n in lens]
    total = sum(need) + spare
    ids = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    lead = () if layers is None else (layers,)
    k, v = (bf16(g, *lead, total, hkv, PAGE, hd) for _ in range(2))
    if fill is not None:
        live = torch.zeros(total, PAGE, dtype=torch.bool, device="cuda")
        for b, n in enumerate(lens):
            j = torch.arange(n, device="cuda")
            live[table[b].long()[j // PAGE], j % PAGE] = True
        for x in (k, v):
            x.movedim(-3, -2)[..., ~live, :, :] = fill
    return k, v, table, torch.tensor(lens, dtype=torch.int32, device="cuda")


def put(pool, table, b, pos, rows):
    """Write rows [m, hkv, hd] at positions pos [m] of sequence b (one layer's pool)."""
    pool[table[b].long()[pos // PAGE], :, pos % PAGE] = rows


def take(pool, table, b, n):
    """The first n positions of sequence b, [n, hkv, hd]."""
    j = torch.arange(n, device=pool.device)
    return pool[table[b].long()[j // PAGE], :, j % PAGE]


def visible(lens, n, count, b, mask, positions, window):
    """bool [count, len + count]: what the nodes of sequence b see."""
    length = int(lens[b])
    node = torch.arange(count, device="cuda")
    if mask is None:
        nodes = node[None] <= node[:, None]
    else:
        nodes = (mask[b, :count].long()[:, node // 32] >> (node % 32)) & 1 == 1
    sees = torch.cat([torch.ones(count, length, dtype=torch.bool, device="cuda"), nodes], 1)
    if window:
        pos = length + node if positions is None else positions[b, :count].long().clamp(length, length + max(count, 1) - 1)
        at = torch.cat([torch.arange(length, device="cuda"), pos])
        sees &= at[None] > pos[:, None] - window
    return sees


def attention(q, k, v, table, lens, mask=None, positions=None, counts=None, window=0, scale=None):
    """(out, bound): float64 results [batch, n, hq, hd] (rows of no node are NaN) and how far
    a bf16 result of the kernel may be from them.

    The bound: one rounding of the result (2^-8 of its size); the softmax weights are
    rounded to bf16 (2^-8 of every weight), and a score computed in fp32 from exact bf16
    products is off by at most hd * 2^-23 of sum |q||k| * scale, which changes a weight by
    twice that at most (numerator and sum), as do 2^-21 from exponential and argument and
    keys * 2^-23 from the sums; each relative to sum p |v|."""
    b_, n, hq, hd = q.shape
    hkv = k.shape[1]
    scale = hd ** -0.5 if scale is None else scale
    out = torch.full(q.shape, math.nan, dtype=torch.float64, device="cuda")
    bound = torch.full(q.shape, math.nan, dtype=torch.float64, device="cuda")
    for b in range(b_):
        count = n if counts is None else int(counts[b])
        if count == 0:
            continue
        keys = int(lens[b]) + count
        sees = visible(lens, n, count, b, mask, positions, window)
        kk, vv = take(k, table, b, keys).double(), take(v, table, b, keys).double()
        for h in range(hq):
            kh, vh, qh = kk[:, h * hkv // hq], vv[:, h * hkv // hq], q[b, :count, h].double()
            s = torch.where(sees, qh @ kh.T * scale, -math.inf)
            top = s.amax(1, keepdim=True)
            p = torch.where(sees, torch.exp(s - torch.where(top == -math.inf, 0.0, top)), 0.0)
            p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
            some = sees.any(0)                       # keys that no row sees may hold anything
            p, vs = p[:, some], vh[some]
            o = torch.zeros(count, hd, dtype=torch.float64, device="cuda")
            # zero weights times NaN or infinity are no part of the sum
            o += torch.where(p[:, :, None] == 0, 0.0, p[:, :, None] * vs).sum(1) if not torch.isfinite(vs).all() else p @ vs
            out[b, :count, h] = o
            off = torch.where(sees, qh.abs() @ torch.nan_to_num(kh.abs()).T, 0.0).amax(1) * scale * hd * 2.0 ** -23
            w = HALF_BF16 + 2 * off + 2.0 ** -20 + keys * 2.0 ** -23
            bound[b, :count, h] = HALF_BF16 * o.abs() + w[:, None] * (p @ torch.nan_to_num(vs, nan=0.0, posinf=0.0, neginf=0.0).abs()) + 1e-30
    return out, bound


def assert_close(got, want, bound, what=""):
    got = got.double()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), f"{what}: infinities"
    off = (got - want).abs()[fine]
    worst = (off / bound[fine].clamp(min=1e-300)).max() if off.numel() else torch.tensor(0.0)
    assert float(worst) <= 1.0, f"{what}: {float(worst):.3g} times the bound, {float(off.max()):.3g} off"


def random_tree(g, batch, n, back=4):
    """parents int32 [batch, n]: every node's parent is one of the `back` before it (or none)."""
    p = torch.arange(n, device="cuda") - torch.randint(1, back + 1, (batch, n), generator=g, device="cuda")
    return p.clamp(min=-1).to(torch.int32)


def rope(x, gain, positions, theta, eps=1e-6):
    """(rotated and normalised x in float64, bound of a bf16 result): the bound is one
    rounding (2^-8) plus fp32 arithmetic on the pair: norm (hd + 4 operations), angle
    (2^-23 turns) and rotation, together below 2^-18 of |lo| + |hi|."""
    hd = x.shape[-1]
    x = x.double()
    if gain is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * gain.double()
    f = theta ** (-2 * torch.arange(hd // 2, dtype=torch.float64, device="cuda") / hd)
    a = positions.double()[..., None, None] * f
    lo, hi = x[..., :hd // 2], x[..., hd // 2:]
    y = torch.cat([lo * a.cos() - hi * a.sin(), hi * a.cos() + lo * a.sin()], -1)
    size = (lo.abs() + hi.abs()).repeat_interleave(1, -1)
    return y, HALF_BF16 * y.abs() + 2.0 ** -18 * torch.cat([size, size], -1) + 1e-30
