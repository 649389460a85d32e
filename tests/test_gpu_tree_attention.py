"""mk_tree_attention against float64: draft trees, prompt chunks, windows, ragged batches."""
import math

import pytest
import torch

import ops_ref as R
from persistent_moe_decode_cta_gb300 import binding as B
from persistent_moe_decode_cta_gb300 import ops

pytestmark = pytest.mark.gpu
NAN = float("nan")


def setup(heads, lens, n, tree=True, counts=None, seed=0, fill=NAN, std=1.5):
    """Inputs whose unused cache slots hold `fill`; the nodes' K/V are in their slots."""
    hq, hkv, hd = heads
    g = R.gen(seed)
    k, v, table, sl = R.cache(g, lens, n, hkv, hd, fill=fill)
    b = len(lens)
    cnt = [n] * b if counts is None else counts
    for i in range(b):
        at = torch.arange(lens[i], lens[i] + cnt[i], device="cuda")
        for pool in (k, v):
            R.put(pool, table, i, at, R.bf16(g, cnt[i], hkv, hd))
    a = dict(q=R.bf16(g, b, n, hq, hd, std=std), k_cache=k, v_cache=v, page_table=table, seq_lens=sl)
    mask = pos = None
    if tree:
        mask, depth = ops.tree_mask(R.random_tree(g, b, n))
        pos = sl[:, None] + depth
    a.update(mask=mask, positions=pos, counts=None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda"))
    return a


def check(a, window=0, scale=None):
    q, counts = a["q"], a["counts"]
    out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    status = ops.new_status()
    got = ops.tree_attention(**a, window=window, scale=scale, out=out, status=status)
    ops.check_status(status)
    assert got is out
    want, bound = R.attention(q, a["k_cache"], a["v_cache"], a["page_table"], a["seq_lens"], a["mask"], a["positions"],
                              counts, window, scale)
    for b in range(q.shape[0]):
        m = q.shape[1] if counts is None else int(counts[b])
        R.assert_close(out[b, :m], want[b, :m], bound[b, :m], f"sequence {b}")
        assert bool((out[b, m:] == 5.0).all())
    return out


LAYOUTS = [(8, 2, 32), (16, 4, 64), (32, 4, 128)]


@pytest.mark.parametrize("heads", LAYOUTS)
@pytest.mark.parametrize("n", [1, 3])
def test_one_short_sequence(heads, n):
    check(setup(heads, [5], n))


@pytest.mark.parametrize("heads", LAYOUTS)
@pytest.mark.parametrize("lens", [[0], [1], [15], [16], [127], [128], [129], [300]])
def test_lengths(heads, lens):
    check(setup(heads, lens, 4))


@pytest.mark.parametrize("heads", LAYOUTS)
@pytest.mark.parametrize("n", [16, 17, 31, 32, 33, 40, 64, 65, 100])
def test_nodes(heads, n):
    check(setup(heads, [70, 0], n))


@pytest.mark.parametrize("heads", LAYOUTS)
@pytest.mark.parametrize("n", [1, 2, 16, 33, 130, 300])
def test_chain(heads, n):
    check(setup(heads, [0, 133], n, tree=False))


@pytest.mark.parametrize("heads", [(1, 1, 128), (3, 3, 64), (6, 2, 128), (5, 1, 32), (7, 1, 64), (48, 1, 64), (128, 1, 32), (64, 8, 128)])
@pytest.mark.parametrize("n", [1, 7, 50])
def test_head_groups(heads, n):
    check(setup(heads, [40, 200], n))


@pytest.mark.parametrize("heads", LAYOUTS)
@pytest.mark.parametrize("tree", [False, True])
def test_ragged_batch(heads, tree):
    check(setup(heads, [3000, 0, 17, 640, 1, 1500, 15, 129], 20, tree, counts=[20, 20, 1, 7, 0, 19, 20, 3]))
    check(setup(heads, [3000, 0, 17, 640, 1, 1500, 15, 129], 70, tree, counts=[70, 64, 1, 7, 0, 33, 70, 3]))


@pytest.mark.parametrize("heads", LAYOUTS)
@pytest.mark.parametrize("window", [1, 2, 15, 64, 300, 100000])
@pytest.mark.parametrize("tree", [False, True])
def test_windows(heads, window, tree):
    check(setup(heads, [0, 40, 700], 12, tree), window)
    check(setup(heads, [0, 40, 700], 75, tree, counts=[75, 20, 75]), window)


@pytest.mark.parametrize("window", [0, 100])
def test_more_items_than_runs(window):
    """Work lists with several items a run: many sequences, many groups of nodes."""
    lens = [(37 * i * i) % 400 for i in range(60)]
    check(setup((8, 4, 64), lens, 3, counts=[i % 4 for i in range(60)]), window)
    check(setup((8, 4, 32), lens, 40, tree=False, counts=[(7 * i) % 41 for i in range(60)]), window)
    check(setup((32, 8, 128), lens[:40], 45), window)
    check(setup((16, 4, 64), [0, 777], 1500, tree=False, counts=[1500, 1301]), window)
    check(setup((8, 1, 128), [40], 3001, tree=False), window)


def test_long_context_is_split_and_joined():
    check(setup((32, 4, 128), [20011], 3))
    check(setup((32, 4, 128), [9000], 64))
    check(setup((16, 4, 64), [33333, 5], 9))


def test_needles():
    """One key with a dominating score, at every border of pages, blocks and tree: the
    result is its value."""
    heads, n, length = (8, 2, 128), 40, 517
    a = setup(heads, [length], n, tree=False, std=0.0)
    k = a["k_cache"]
    g = R.gen(9)
    for node in (0, 1, 15, 16, 31, 39):
        for key in (0, 15, 16, 127, 128, 255, 256, 511, 512, 516, 517, 517 + node):
            a["q"].zero_()
            d = R.bf16(g, 128).sign()
            a["q"][0, node] = d
            old = R.take(k, a["page_table"], 0, length + n)[key].clone()
            at = torch.tensor([key], device="cuda")
            R.put(k, a["page_table"], 0, at, (4 * d).expand(1, 2, 128))
            out = ops.tree_attention(**a)
            want = R.take(a["v_cache"], a["page_table"], 0, length + n)[key].repeat_interleave(4, 0).double()
            # the others' weight is below 600 * exp(-(512 - 6 * 11.4) / 11.4) < 1e-13
            R.assert_close(out[0, node], want, R.HALF_BF16 * want.abs() + 1e-9, f"node {node} key {key}")
            R.put(k, a["page_table"], 0, at, old[None])


def test_rising_scores_rescale():
    """Scores that grow along the keys by far more than the allowed lag of the maximum."""
    for heads in LAYOUTS:
        a = setup(heads, [1500], 9, std=1.0)
        pos = torch.arange(1500, device="cuda")
        rows = R.take(a["k_cache"], a["page_table"], 0, 1500) * (1 + pos[:, None, None] / 100)
        R.put(a["k_cache"], a["page_table"], 0, pos, rows.to(torch.bfloat16))
        check(a)
        R.put(a["k_cache"], a["page_table"], 0, pos, rows.flip(0).to(torch.bfloat16))
        check(a)


def test_rows_that_see_nothing_are_zero():
    for n in (5, 60):
        a = setup((16, 4, 64), [0, 200], n)
        a["mask"][:, 1] = 0
        a["mask"][0, 3] = 0
        out = check(a)
        assert bool((out[0, 1] == 0).all()) and bool((out[0, 3] == 0).all())
        a = setup((16, 4, 64), [0, 200], n)
        a["mask"][:] = 0
        out = check(a, window=1)     # no cached key is inside a window of one
        assert bool((out[:, :] == 0).all())


def test_masked_values_do_not_leak():
    """NaN and infinities in K and V of nodes and cached keys that a row does not see."""
    for heads in LAYOUTS:
        for n in (6, 60):
            hkv, hd = heads[1], heads[2]
            a = setup(heads, [90, 300], n)
            mask = torch.zeros_like(a["mask"])
            i = torch.arange(n, device="cuda")
            mask[:, i, i // 32] = torch.where(i % 32 == 31, -2 ** 31, 1 << (i % 32)).to(torch.int32)   # every node sees itself only
            a["mask"] = mask
            for b, length in enumerate((90, 300)):
                at = torch.tensor([length + 2, length + 4], device="cuda")
                R.put(a["v_cache"], a["page_table"], b, at[:1], torch.full((1, hkv, hd), NAN, dtype=torch.bfloat16, device="cuda"))
                R.put(a["v_cache"], a["page_table"], b, at[1:], torch.full((1, hkv, hd), math.inf, dtype=torch.bfloat16, device="cuda"))
                R.put(a["k_cache"], a["page_table"], b, at[:1], torch.full((1, hkv, hd), NAN, dtype=torch.bfloat16, device="cuda"))
            out = check(a)
            assert torch.isnan(out[:, 2]).all() and torch.isfinite(out[:, 3]).all()
            assert torch.isinf(out[:, 4]).all()
            # cached keys behind the window
            a = setup(heads, [300], n, tree=False)
            at = torch.arange(0, 300 - 50, device="cuda")
            for pool in (a["k_cache"], a["v_cache"]):
                R.put(pool, a["page_table"], 0, at, torch.full((250, hkv, hd), NAN, dtype=torch.bfloat16, device="cuda"))
            check(a, window=50)


@pytest.mark.parametrize("heads", LAYOUTS)
@pytest.mark.parametrize("n,length", [(6, 300), (60, 300), (6, 3000), (60, 3000)])
def test_infinities_of_masked_and_unmasked_blocks_add(heads, n, length):
    """Infinities of a cached key (in a block that every row sees) and of nodes that some rows see."""
    hkv, hd = heads[1], heads[2]
    a = setup(heads, [length], n)
    i = torch.arange(n, device="cuda")
    seen = (i[:, None] == i) | (i == 0) | ((i == 2) & (i[:, None] % 2 == 0)) | ((i == 4) & (i[:, None] % 3 == 0))
    words = torch.zeros(n, a["mask"].shape[2], dtype=torch.int64, device="cuda")
    for x in range(n):
        words[:, x // 32] += seen[:, x].long() << (x % 32)
    a["mask"][0] = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)
    for at, values in ((10, (-math.inf, NAN, math.inf)), (length + 2, (math.inf, math.inf, 1.0, -math.inf)),
                       (length + 4, (1.0, 1.0, -math.inf, 1.0, math.inf))):
        row = torch.zeros(1, hkv, hd, dtype=torch.bfloat16, device="cuda")
        row[:, :, :len(values)] = torch.tensor(values, dtype=torch.bfloat16)
        R.put(a["v_cache"], a["page_table"], 0, torch.tensor([at], device="cuda"), row)
    out = check(a)
    assert torch.isnan(out[0, 2, :, 0]).all() and (out[0, 1, :, 0] == -math.inf).all() and torch.isnan(out[0, :, :, 1]).all()


def test_positions_are_clamped_to_the_sequence():
    a = setup((8, 2, 32), [100], 6)
    for lo in (-1000, 2 ** 31 - 1):
        a["positions"] = torch.full((1, 6), lo, dtype=torch.int32, device="cuda")
        check(a, window=30)


def test_strided_operands():
    a = setup((16, 4, 64), [50, 9], 11)
    g = R.gen(3)
    packed = R.bf16(g, 11, 2, 24, 80)            # [node, sequence, heads, ..]: views in another order
    a["q"] = packed.transpose(0, 1)[:, :, 4:20, 8:72]
    want, bound = R.attention(a["q"], a["k_cache"], a["v_cache"], a["page_table"], a["seq_lens"], a["mask"])
    base = torch.zeros(2, 11, 40, 72, dtype=torch.bfloat16, device="cuda")
    out = base[:, :, 3:19, :64]
    ops.tree_attention(**a, out=out)
    R.assert_close(out, want, bound)
    out.zero_()
    assert not base.any()


def test_scale():
    a = setup((8, 2, 32), [70], 5)
    check(a, scale=0.0)
    check(a, scale=1.0)


def test_bad_pages_and_lengths_are_reported():
    a = setup((8, 2, 32), [40, 33], 3)
    status = ops.new_status()
    table = a["page_table"]
    keep = int(table[0, 1])
    for bad in (-1, a["k_cache"].shape[0], 2 ** 31 - 1):
        table[0, 1] = bad
        ops.tree_attention(**a, status=status)
        with pytest.raises(B.MkError, match="MK_ERR_BAD_PAGE"):
            ops.check_status(status)
    table[0, 1] = keep
    for lens in ([-1, 33], [40, 16 * table.shape[1] - 2]):
        sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        ops.tree_attention(**dict(a, seq_lens=sl), status=status)
        with pytest.raises(B.MkError, match="MK_ERR_INVALID"):
            ops.check_status(status)
    for cnt in ([4, 3], [3, 2 ** 31 - 1]):
        ops.tree_attention(**dict(a, counts=torch.tensor(cnt, dtype=torch.int32, device="cuda")), status=status)
        with pytest.raises(B.MkError, match="MK_ERR_INVALID"):
            ops.check_status(status)
    check(a)


def test_equal_calls_give_equal_bits():
    a = setup((32, 4, 128), [5000, 100, 777], 20)
    first = ops.tree_attention(**a)
    for _ in range(3):
        assert torch.equal(ops.tree_attention(**a), first)


def test_captured_graphs_on_two_streams():
    """Two graphs with workspaces of their own, replayed side by side, after the lengths and
    the queries have changed."""
    calls = [setup((32, 4, 128), [2000, 31], 12, seed=1), setup((32, 4, 128), [700, 900], 40, seed=2)]
    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for a in calls:
        ops.tree_attention(**a)
    torch.cuda.synchronize()
    for a, s in zip(calls, streams):
        graph, out = torch.cuda.CUDAGraph(), torch.zeros_like(a["q"])
        with torch.cuda.graph(graph, stream=s):
            ops.tree_attention(**a, out=out)
        graphs.append(graph), outs.append(out)
    g = R.gen(4)
    for a in calls:
        a["q"].copy_(R.bf16(g, *a["q"].shape))
        a["seq_lens"].sub_(5)
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for a, out in zip(calls, outs):
        assert torch.equal(out, ops.tree_attention(**a))


def test_on_another_stream():
    a = setup((16, 4, 64), [300], 8)
    want = ops.tree_attention(**a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ops.tree_attention(**a, stream=side)
    raw = ops.tree_attention(**a, stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want) and torch.equal(raw, want)


@pytest.mark.parametrize("lens,n", [([130], 3), ([5000], 3), ([300, 0, 2500], 70)])
def test_workspace_contents_do_not_matter(lens, n):
    """The C entry point with a workspace full of NaN and exactly of the size asked for."""
    import ctypes
    a = setup((8, 2, 64), lens, n, tree=False)
    want = ops.tree_attention(**a)
    kv = B.mk_paged_kv(a["k_cache"].data_ptr(), a["v_cache"].data_ptr(), a["page_table"].data_ptr(), a["seq_lens"].data_ptr(),
                       a["k_cache"].shape[0], 2, 64, len(lens), a["page_table"].shape[1])
    out = torch.zeros_like(a["q"])
    s = B._S3(*a["q"].stride()[:3])
    args = B.mk_tree_args(a["q"].data_ptr(), out.data_ptr(), s, s, None, None, None, None, n, 8, 0, 64 ** -0.5)
    need = ctypes.c_size_t()
    lib = B.load_library()
    assert lib.mk_tree_attention_workspace(ctypes.byref(kv), ctypes.byref(args), ctypes.byref(need)) == B.MK_OK
    work = torch.full((need.value + 1024,), 255, dtype=torch.uint8, device="cuda")   # NaN in every float
    args.workspace, args.workspace_bytes = work.data_ptr(), need.value - 1
    stream = torch.cuda.current_stream().cuda_stream
    assert lib.mk_tree_attention(ctypes.byref(kv), ctypes.byref(args), stream) == B.MK_ERR_INVALID
    args.workspace_bytes = need.value
    assert lib.mk_tree_attention(ctypes.byref(kv), ctypes.byref(args), stream) == B.MK_OK
    torch.cuda.synchronize()
    assert torch.equal(out, want) and bool((work[need.value:] == 255).all())
