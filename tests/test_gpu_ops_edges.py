"""Calls of the multi-token operators that the documentation allows and that lie at the edge of
what a program makes: inputs written just before the call, positions of siblings in a prompt
chunk, long lists of sequences, many heads."""
import pytest
import torch

import ops_ref as R
from persistent_moe_decode_cta_gb300 import binding as B
from persistent_moe_decode_cta_gb300 import ops
import test_gpu_qk_rope as Rope
from test_gpu_experts import reference
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


@pytest.mark.parametrize("heads,n", [((64, 8, 128), 3), ((64, 8, 128), 700), ((256, 128, 32), 5), ((96, 96, 64), 40), ((400, 4, 128), 9)])
def test_rotation_of_many_heads(heads, n):
    """More heads than the threads of a block: several blocks share a token."""
    Rope.check(heads, [3, 40], n, counts=[n, n - 1])
    Rope.check(heads, [0], n, norm=False, packed=False, in_place=True)


@pytest.mark.parametrize("layers,pages,hkv,hd,n", [(2, 40, 8, 128, 15), (3, 20, 9, 128, 7), (1, 10, 33, 128, 5), (2, 90, 40, 64, 41)])
def test_copies_of_large_pages(layers, pages, hkv, hd, n):
    """Pages above 16 KB: several blocks a page, the last of them with less than the others."""
    g = R.gen(pages)
    k, v = (R.bf16(g, layers, pages, hkv, 16, hd) for _ in range(2))
    ids = torch.randperm(pages, generator=g, device="cuda").tolist()
    src, dst = ids[:n], ids[n:2 * n]
    ek, ev = k.clone(), v.clone()
    ek[:, dst] = k[:, src]
    ev[:, dst] = v[:, src]
    ops.copy_pages(k, v, src, dst)
    assert torch.equal(k, ek) and torch.equal(v, ev)


def ragged(batch, far):
    """Short lengths, some of them zero, and `far` sequences of several thousand keys, the last among them."""
    lens = [(53 * i * i) % 190 * (i % 5 != 0) for i in range(batch)]
    for i in range(far):
        lens[batch - 1 - i * (batch // far)] = 2500 + 1300 * i
    return lens


@pytest.mark.parametrize("window", [0, 150])
@pytest.mark.parametrize("heads,n,batch", [((4, 1, 32), 2, 128), ((4, 1, 32), 2, 129), ((4, 2, 64), 3, 256), ((4, 2, 64), 3, 257),
                                           ((4, 1, 32), 70, 300), ((2, 1, 128), 1, 1000), ((8, 2, 32), 2, 1000)])
def test_long_lists_of_sequences(heads, n, batch, window):
    """Work lists of more than one entry a thread, and of more than the join adds up itself."""
    counts = [0 if i % 7 == 3 else 1 + i % n for i in range(batch)]
    check(setup(heads, ragged(batch, 4), n, counts=counts), window)
    check(setup(heads, ragged(batch, 1), n, tree=False, counts=counts), window)


@pytest.mark.parametrize("window", [0, 1000])
def test_long_chunks(window):
    """A chunk whose groups of nodes are more than 256 entries, beside a short one."""
    check(setup((8, 1, 32), [100], 8300, tree=False), window)
    check(setup((16, 1, 32), [40, 3], 2100, tree=False, counts=[2099, 1300]), window)


@pytest.mark.parametrize("named", [False, True])
@pytest.mark.parametrize("offsets,rows,owner", [
    ([0, 9, 12], None, [0] * 8), ([-3, 2, 8], None, [0] * 2 + [1] * 6), ([4, 2, 8], None, [None] * 2 + [1] * 6),
    ([2 ** 31 - 1, -2 ** 31, 5], None, [1] * 5 + [None] * 3), ([0, 4, 8], [0, 1, 2, 3, 4, 5, 6, 8], [0] * 4 + [1] * 4),
    ([0, 4, 8], [0, 1, -2 ** 31, 3, 4, 2 ** 31 - 1, 6, 7], [0] * 4 + [1] * 4)])
def test_bad_offsets_and_rows_stay_inside(offsets, rows, owner, named):
    """Beyond the error: rows that belong to an expert are those of the clamped numbers, all others as they were."""
    g = R.gen(5)
    x, w = R.bf16(g, 8, 64), R.bf16(g, 2, 40, 64)
    base = torch.full((24, 40), 3.0, dtype=torch.bfloat16, device="cuda")
    out = base[8:16]
    if rows is None and named:
        rows = list(range(8))
    r = None if rows is None else torch.tensor(rows, dtype=torch.int32, device="cuda")
    status = ops.new_status()
    ops.expert_product(x, w, torch.tensor(offsets, dtype=torch.int32, device="cuda"), rows=r, out=out, status=status)
    with pytest.raises(B.MkError) as e:
        ops.check_status(status)
    assert e.value.code == B.MK_ERR_INVALID
    ends = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    at = torch.arange(8, device="cuda") if rows is None else torch.tensor(rows, device="cuda").clamp(0, 7)
    want, bound = zip(*(reference(x[at], w[i:i + 1], ends, None, None) for i in range(2)))
    for i, e in enumerate(owner):
        if e is None:
            assert bool((out[i] == 3.0).all())
        else:
            R.assert_close(out[i], want[e][i], bound[e][i], f"row {i}")
    assert bool((base[:8] == 3.0).all() and (base[16:] == 3.0).all())


@pytest.mark.parametrize("n", [3, 70])
@pytest.mark.parametrize("heads", LAYOUTS)
def test_bad_pages_and_lengths_of_one_sequence(heads, n):
    """A bad page is read as page 0, a sequence of a bad length left out; the other sequence has its bits."""
    a = setup(heads, [900, 433], n)
    a["k_cache"].nan_to_num_(nan=0.5), a["v_cache"].nan_to_num_(nan=0.5)
    fine = ops.tree_attention(**a)
    table, status = a["page_table"], ops.new_status()
    keep = table.clone()
    table[0, 1] = 0
    zero = ops.tree_attention(**a)
    for bad in (-1, a["k_cache"].shape[0], 2 ** 31 - 1, -2 ** 31):
        table[0, 1] = bad
        got = ops.tree_attention(**a, status=status)
        assert torch.equal(got, zero) and torch.equal(got[1], fine[1])
        with pytest.raises(B.MkError, match="MK_ERR_BAD_PAGE"):
            ops.check_status(status)
    table.copy_(keep)
    for length, count in ((-1, n), (16 * table.shape[1] - n + 1, n), (900, n + 1), (2 ** 31 - 1, n), (0, 2 ** 31 - 1)):
        bad = dict(a, seq_lens=torch.tensor([length, 433], dtype=torch.int32, device="cuda"),
                   counts=torch.tensor([count, n], dtype=torch.int32, device="cuda"))
        out = torch.full_like(a["q"], 5.0)
        ops.tree_attention(**bad, out=out, status=status)
        assert bool((out[0] == 5.0).all())
        want, bound = R.attention(a["q"], a["k_cache"], a["v_cache"], table, a["seq_lens"], a["mask"], a["positions"])
        R.assert_close(out[1], want[1], bound[1])
        with pytest.raises(B.MkError, match="MK_ERR_INVALID"):
            ops.check_status(status)


def test_pages_whose_offsets_pass_32_bits():
    """The same tokens in a pool of 40 pages and in the last pages of pools of 10 GB a layer: equal bits."""
    g = R.gen(12)
    far, pages, hkv, hd, n, lens = 600_000, 40, 4, 128, 9, [300, 77]
    small = [R.bf16(g, 2, pages, hkv, 16, hd) for _ in range(2)]
    large = [torch.empty(2, far, hkv, 16, hd, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for a, b in zip(small, large):
        b[:, far - pages:] = a
    table = torch.randperm(pages, generator=g, device="cuda")[:pages // 2 * 2].view(2, -1).to(torch.int32)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q, kn, vn = R.bf16(g, 2, n, 32, hd), R.bf16(g, 2, n, hkv, hd), R.bf16(g, 2, n, hkv, hd)
    acc = torch.tensor([[1, 4, 8], [0, 2, -1]], dtype=torch.int32, device="cuda")
    src, dst = table[0, :5].tolist(), table[1, -5:].tolist()
    got = []
    for (k, v), first in ((small, 0), (large, far - pages)):
        t = table + first
        r = [ops.qk_norm_rope(q, kn, vn, k[l], v[l], t, sl, theta=1e6) for l in range(2)]
        r += [ops.tree_attention(r[l], k[l], v[l], t, sl) for l in range(2)]
        r.append(ops.commit_nodes(k, v, t, sl, acc))
        ops.copy_pages(k, v, [first + p for p in src], [first + p for p in dst])
        got.append(r + [k[:, first:first + pages].clone(), v[:, first:first + pages].clone()])
    ops.check_status()
    assert all(torch.equal(a, b) for a, b in zip(*got))
