"""Calls of the multi-token operators that the documentation allows and that lie at the edge of
what a program makes: inputs written just before the call, positions of siblings in a prompt
chunk, long lists of sequences, many heads."""
import pytest
import torch

import ops_ref as R
from persistent_moe_decode_cta_gb300 import binding as B
from persistent_moe_decode_cta_gb300 import ops
from test_gpu_tree_attention import LAYOUTS, check, setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,n", [((8, 2, 32), 3), ((32, 4, 128), 40)])
def test_lengths_written_just_before_the_call(heads, n):
    """The kernels of a call, launched before the copies of its lengths and counts have ended, all work with the
    new ones: other lengths every time split the items elsewhere."""
    a = setup(heads, [3000, 700, 1], n, counts=[n, n, n])
    sets = [([3000, 700, 1], [n, n, n]), ([5, 690, 0], [n - 1, n, 1]), ([1700, 0, 1], [1, n, n]), ([2999, 128, 1], [n, 0, 2])]
    sets = [tuple(torch.tensor(x, dtype=torch.int32, device="cuda") for x in s) for s in sets]
    out = torch.zeros_like(a["q"])

    def call(i):
        a["seq_lens"].copy_(sets[i][0])
        a["counts"].copy_(sets[i][1])
        return ops.tree_attention(**a, out=out)

    want = []
    for i in range(4):
        call(i)
        torch.cuda.synchronize()
        want.append(out.clone())
    got = [call(i % 4).clone() for i in range(40)]
    # (rows of no node keep what the call before has left there: compared where a node is)
    for i, x in enumerate(got):
        for b, m in enumerate(sets[i % 4][1].tolist()):
            assert torch.equal(x[b, :m], want[i % 4][b, :m]), (i, b)


@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("sizes,n,k", [([300, 0, 129, 5, 256, 1000], 384, 1024), ([700] * 16, 768, 256), ([3, 9, 1, 0, 30] * 8, 512, 2048)])
def test_named_rows_equal_rows_in_order(sizes, n, k, glu):
    """Both CTAs of a pair fetch named rows themselves; the bits are those of rows that lie in order."""
    g = R.gen(len(sizes))
    e, total = len(sizes), sum(sizes)
    offsets = torch.tensor([0] + sizes, device="cuda").cumsum(0).to(torch.int32)
    x = R.bf16(g, 611, k)
    w, u = R.bf16(g, e, n, k, std=0.05), R.bf16(g, e, n, k, std=0.05) if glu else None
    for _ in range(8):
        rows = torch.randint(0, 611, (total,), generator=g, device="cuda").to(torch.int32)
        want = ops.expert_product(x[rows.long()], w, offsets, w_up=u)
        for _ in range(4):
            assert torch.equal(ops.expert_product(x, w, offsets, w_up=u, rows=rows), want)


@pytest.mark.parametrize("heads", LAYOUTS + [(6, 6, 64), (128, 1, 32)])
@pytest.mark.parametrize("window", [1, 40, 300])
def test_window_and_positions_of_a_chain(heads, window):
    """Without a mask, positions of the nodes that do not ascend one by one: a node's key leaves the window by its
    position, whatever its slot is."""
    for n, lens, counts in ((500, [70, 0], [500, 431]), (131, [300], None)):
        a = setup(heads, lens, n, tree=False, counts=counts)
        g = R.gen(window)
        start = a["seq_lens"][:, None]
        node = torch.arange(n, device="cuda")
        for depth in (torch.zeros_like(node), node // 2, node.flip(0), torch.randint(0, n, (n,), generator=g, device="cuda"),
                      torch.where(node < n // 2, 0, n - 1)):
            a["positions"] = (start + depth).to(torch.int32)
            check(a, window)


def test_what_is_found_without_a_status_is_recorded():
    """A call that is given no record leaves what it finds in the device's own."""
    g = R.gen(8)
    k, v, table, sl = R.cache(g, [20, 3], 4, 2, 32, layers=1)
    q = R.bf16(g, 2, 4, 4, 32)
    kn = R.bf16(g, 2, 4, 2, 32)
    x, w = R.bf16(g, 8, 64), R.bf16(g, 2, 40, 64)
    keep = table.clone()
    bad = keep.clone()
    bad[1, 0] = k.shape[1]
    table.copy_(bad)
    calls = [(B.MK_ERR_BAD_PAGE, 1, lambda **s: ops.qk_norm_rope(q, kn, kn, k[0], v[0], table, sl, theta=1e4, **s)),
             (B.MK_ERR_BAD_PAGE, 1, lambda **s: ops.tree_attention(q, k[0], v[0], table, sl, **s)),
             (B.MK_ERR_BAD_PAGE, 1, lambda **s: ops.commit_nodes(k, v, table, sl, torch.ones_like(sl)[:, None], **s)),
             (B.MK_ERR_INVALID, 0, lambda **s: ops.expert_product(x, w, torch.tensor([-1, 2, 8], dtype=torch.int32, device="cuda"), **s))]
    ops.check_status()
    for code, where, call in calls:
        call()
        with pytest.raises(B.MkError, match=f"expert or CTA {where},") as e:
            ops.check_status()
        assert e.value.code == code
        ops.check_status()      # cleared
        status = ops.new_status()
        call(status=status)
        ops.check_status()      # the caller's record, not the device's
        with pytest.raises(B.MkError):
            ops.check_status(status)
    graph = torch.cuda.CUDAGraph()
    table.copy_(keep)
    with torch.cuda.graph(graph):
        calls[1][2]()
    graph.replay()
    ops.check_status()
    table.copy_(bad)
    graph.replay()
    with pytest.raises(B.MkError):
        ops.check_status()


def test_an_empty_batch_is_no_work():
    """No sequence: every operator on the cache returns without one."""
    g = R.gen(2)
    k, v = R.bf16(g, 2, 4, 2, 16, 32), R.bf16(g, 2, 4, 2, 16, 32)
    k0, v0 = k.clone(), v.clone()
    table = torch.zeros(0, 3, dtype=torch.int32, device="cuda")
    lens = torch.zeros(0, dtype=torch.int32, device="cuda")
    q, kn = R.bf16(g, 0, 5, 4, 32), R.bf16(g, 0, 5, 2, 32)
    assert ops.qk_norm_rope(q, kn, kn, k[0], v[0], table, lens, theta=1e4).shape == q.shape
    assert ops.tree_attention(q, k[0], v[0], table, lens).shape == q.shape
    new = ops.commit_nodes(k, v, table, lens, torch.zeros(0, 4, dtype=torch.int32, device="cuda"))
    assert new.shape == (0,) and new.dtype == torch.int32
    ops.copy_pages(k, v, [], [])
    assert torch.equal(k, k0) and torch.equal(v, v0)
    ops.check_status()
