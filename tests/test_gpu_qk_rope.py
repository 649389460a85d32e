"""mk_qk_norm_rope against float64: norms, rotation, and the append to the paged cache."""
import pytest
import torch

import ops_ref as R
from persistent_moe_decode_cta_gb300 import ops

pytestmark = pytest.mark.gpu
HEADS = [(8, 2, 32), (16, 4, 64), (32, 4, 128), (3, 3, 128), (5, 1, 32), (7, 7, 64)]


def check(heads, lens, n, norm=True, counts=None, positions=None, theta=1e6, packed=True, in_place=False, seed=0):
    hq, hkv, hd = heads
    g = R.gen(seed)
    k, v, table, sl = R.cache(g, lens, n, hkv, hd)
    b = len(lens)
    if packed:  # views of one projection's result
        x = R.bf16(g, b, n, hq + 2 * hkv, hd)
        q, kn, vn = x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:]
    else:
        q, kn, vn = R.bf16(g, b, n, hq, hd), R.bf16(g, b, n, hkv, hd), R.bf16(g, b, n, hkv, hd)
    gq, gk = ((1 + R.bf16(g, hd, std=0.1)) for _ in range(2)) if norm else (None, None)
    cnt = None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda")
    pos = None if positions is None else torch.tensor(positions, dtype=torch.int32, device="cuda").expand(b, n).contiguous()
    at = sl[:, None] + torch.arange(n, device="cuda") if pos is None else pos
    want_q, bound_q = R.rope(q, gq, at, theta)
    want_k, bound_k = R.rope(kn, gk, at, theta)
    k0, v0 = k.clone(), v.clone()
    status = ops.new_status()
    out = q if in_place else torch.full((b, n, hq, hd), 7.0, dtype=torch.bfloat16, device="cuda")
    before = out.clone()
    got = ops.qk_norm_rope(q, kn, vn, k, v, table, sl, theta=theta, q_gain=gq, k_gain=gk, positions=pos, counts=cnt,
                           out=out, status=status)
    assert got is out
    ops.check_status(status)
    ek, ev = k0.clone(), v0.clone()
    for i in range(b):
        m = n if counts is None else counts[i]
        R.assert_close(out[i, :m], want_q[i, :m], bound_q[i, :m], "q")
        assert torch.equal(out[i, m:], before[i, m:])
        if not m:
            continue
        slot = torch.arange(lens[i], lens[i] + m, device="cuda")
        kk = k[table[i].long()[slot // 16], :, slot % 16]
        R.assert_close(kk, want_k[i, :m], bound_k[i, :m], "k")
        R.put(ek, table, i, slot, kk)
        R.put(ev, table, i, slot, vn[i, :m])
    assert torch.equal(k, ek) and torch.equal(v, ev)   # nothing but the nodes' slots


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("n", [1, 5])
def test_head_layouts(heads, n):
    check(heads, [0, 15, 33], n)


@pytest.mark.parametrize("n", [1, 2, 17, 300])
def test_lengths(n):
    check((32, 4, 128), [0, 1, 16, 4097], n)


@pytest.mark.parametrize("heads,lens,n", [((32, 4, 128), [3, 40], 1001), ((16, 4, 64), [0], 6000), ((8, 2, 32), [5] * 1300, 5),
                                          ((3, 3, 128), [1] * 2500, 1)])
def test_many_tokens_behind_one_another(heads, lens, n):
    counts = [n - (i % 3 if n > 1 else 0) for i in range(len(lens))]
    check(heads, lens, n, counts=counts if n < 100 else None, in_place=n > 2000, packed=n <= 2000)


def test_no_norm_unpacked_in_place():
    check((16, 4, 64), [3, 40], 9, norm=False, packed=False, in_place=True)
    check((32, 4, 128), [3, 40], 9, in_place=True)


def test_counts_leave_the_rest():
    check((32, 4, 128), [5, 0, 31, 7], 6, counts=[6, 0, 1, 3])


@pytest.mark.parametrize("theta", [1.0, 1e4, 1e6])
def test_far_and_equal_positions(theta):
    # siblings of a tree share a position; angles of far positions keep their accuracy
    check((8, 2, 32), [4, 9], 7, positions=[0, 1, 1, 131071, 16777217, 2147483647, -5], theta=theta)
    check((8, 2, 128), [4], 7, positions=[0, 1, 1, 131071, 16777217, 2147483647, -5], theta=theta)


def test_zero_head_and_large_values():
    g = R.gen(1)
    k, v, table, sl = R.cache(g, [0], 2, 1, 64)
    x = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16, device="cuda")
    x[0, 1] = 1e15
    one = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    out = ops.qk_norm_rope(x, x, x, k, v, table, sl, theta=1e4, q_gain=one, k_gain=one)
    want, bound = R.rope(x, one, sl[:, None] + torch.arange(2, device="cuda"), 1e4)
    assert torch.equal(out[0, 0], torch.zeros_like(out[0, 0]))
    R.assert_close(out, want, bound)


def test_bad_pages_and_lengths_are_reported_and_skipped():
    g = R.gen(2)
    k, v, table, sl = R.cache(g, [0, 16], 4, 2, 32)
    x = R.bf16(g, 2, 4, 2, 32)
    table[1, 1] = k.shape[0]
    k0, v0 = k.clone(), v.clone()
    status = ops.new_status()
    ops.qk_norm_rope(x, x, x, k, v, table, sl, theta=1e4, status=status)
    with pytest.raises(Exception, match="MK_ERR_BAD_PAGE"):
        ops.check_status(status)
    ops.check_status(status)  # cleared
    at = int(table[0, 0])
    changed = (k != k0).any(-1).any(-1).any(-1)
    assert changed[at] and int(changed.sum()) == 1
    for bad in (-1, 16 * table.shape[1] - 3):   # four nodes would pass the table's end
        sl2 = torch.tensor([bad, 0], dtype=torch.int32, device="cuda")
        k.copy_(k0), v.copy_(v0)
        ops.qk_norm_rope(x, x, x, k, v, table, sl2, theta=1e4, status=status)
        with pytest.raises(Exception, match="MK_ERR_INVALID"):
            ops.check_status(status)
        changed = (k != k0).any(-1).any(-1).any(-1)
        assert int(changed.sum()) == 1 and changed[int(table[1, 0])]


def test_captured_and_replayed():
    g = R.gen(3)
    heads = (16, 4, 64)
    k, v, table, sl = R.cache(g, [7, 30], 3, 4, 64)
    q, kn, vn = R.bf16(g, 2, 3, 16, 64), R.bf16(g, 2, 3, 4, 64), R.bf16(g, 2, 3, 4, 64)
    out = torch.zeros_like(q)
    run = lambda: ops.qk_norm_rope(q, kn, vn, k, v, table, sl, theta=1e4, out=out)
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    q.copy_(R.bf16(g, *q.shape)), kn.copy_(R.bf16(g, *kn.shape))
    sl.add_(1)
    graph.replay()
    a = (out.clone(), k.clone(), v.clone())
    run()
    assert all(torch.equal(x, y) for x, y in zip(a, (out, k, v))) and heads
