"""mk_copy_pages and mk_commit_nodes: bytes move exactly, and nothing else changes."""
import pytest
import torch

import ops_ref as R
from persistent_moe_decode_cta_gb300 import binding as B
from persistent_moe_decode_cta_gb300 import ops

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layers,pages,hkv,hd,n", [(1, 5, 1, 32, 1), (2, 40, 2, 32, 17), (8, 200, 4, 64, 65), (3, 300, 3, 128, 100),
                                                   (1, 9000, 1, 32, 4321), (48, 20, 4, 128, 7)])
def test_copy_pages(layers, pages, hkv, hd, n):
    g = R.gen(n)
    k, v = (R.bf16(g, layers, pages, hkv, 16, hd) for _ in range(2))
    k[0, 0, 0, 0, 0] = float("nan")
    ids = torch.randperm(pages, generator=g, device="cuda").tolist()
    half = pages // 2
    dst = ids[:n]
    src = [ids[half + i % (pages - half)] for i in range(n)]   # some pages are copied to several places
    ek, ev = k.clone(), v.clone()
    ek[:, dst] = k[:, src]
    ev[:, dst] = v[:, src]
    ops.copy_pages(k, v, src, torch.tensor(dst, dtype=torch.int32))
    for got, want in ((k, ek), (v, ev)):
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))


def test_copy_pages_refusals():
    g = R.gen(0)
    k, v = (R.bf16(g, 2, 8, 2, 16, 32) for _ in range(2))
    k0 = k.clone()
    for src, dst, code in (([0, 1], [2, 2], B.MK_ERR_INVALID), ([0, 1], [1, 2], B.MK_ERR_INVALID), ([3], [3], B.MK_ERR_INVALID),
                           ([8], [0], B.MK_ERR_BAD_PAGE), ([0], [-1], B.MK_ERR_BAD_PAGE)):
        with pytest.raises(B.MkError) as e:
            ops.copy_pages(k, v, src, dst)
        assert e.value.code == code
    for src, dst in (([0], [1, 2]), (torch.tensor([0], device="cuda"), [1]), ([0.5], [1]), ([2 ** 40], [1])):
        with pytest.raises(ValueError):
            ops.copy_pages(k, v, src, dst)
    ops.copy_pages(k, v, [], [])
    assert torch.equal(k, k0)


def commit_ref(k, v, table, lens, accepted):
    new = lens.clone()
    for b, path in enumerate(accepted.tolist()):
        m = next((i for i, a in enumerate(path) if a < 0), len(path))
        new[b] += m
        at = [int(lens[b]) + a for a in path[:m]]
        for pool in (k, v):
            rows = [pool[:, int(table[b, p // 16]), :, p % 16].clone() for p in at]
            for i, r in enumerate(rows):
                p = int(lens[b]) + i
                pool[:, int(table[b, p // 16]), :, p % 16] = r
    return new


@pytest.mark.parametrize("layers,hkv,hd,lens,paths", [
    (2, 2, 32, [0], [[0]]),
    (2, 2, 32, [15, 16, 0], [[0, 2, 5], [1, -1, 4], [-1, 0, 0]]),           # ends at the first negative entry
    (3, 3, 64, [30, 1], [[5, 3, 4, 0], [2, 2, 2, 2]]),                      # any order, the same node twice
    (48, 4, 128, [100, 7, 3, 0, 1, 2, 5, 9], [[0, 3, 7, 12, 40]] * 8),
    (38, 6, 32, [100, 7, 3, 0, 1, 2, 5, 9], [[0, 3, 7, 12, 40]] * 8),       # blocks of 4 heads and of 2
    (48, 5, 64, [100, 7, 3, 0, 1, 2, 5, 9], [[9, -1, 2]] * 8),
    (1, 1, 128, [9], [list(range(1, 513))]),                                # the longest path, a shift by one
    (1, 1, 32, [9], [list(range(511, -1, -1))]),
])
def test_commit_nodes(layers, hkv, hd, lens, paths):
    g = R.gen(len(lens))
    room = max(max(p) for p in paths) + 1
    k, v, table, sl = R.cache(g, lens, max(room, len(paths[0])), hkv, hd, layers=layers)
    acc = torch.tensor(paths, dtype=torch.int32, device="cuda")
    ek, ev = k.clone(), v.clone()
    want = commit_ref(ek, ev, table, sl, acc)
    status = ops.new_status()
    got = ops.commit_nodes(k, v, table, sl, acc, status=status)
    ops.check_status(status)
    assert torch.equal(got, want) and sl.tolist() == lens
    assert torch.equal(k, ek) and torch.equal(v, ev)


def test_commit_reports_and_skips_bad_sequences():
    g = R.gen(5)
    k, v, table, sl = R.cache(g, [0, 0, 4], 16, 2, 32, layers=2)
    table[1, 0] = -7
    acc = torch.tensor([[3, 16 * table.shape[1]], [1, 2], [2, 3]], dtype=torch.int32, device="cuda")
    ek, ev = k.clone(), v.clone()
    only = acc.clone()
    only[:2] = -1
    want = commit_ref(ek, ev, table, sl, only)
    status = ops.new_status()
    got = ops.commit_nodes(k, v, table, sl, acc, status=status)
    with pytest.raises(B.MkError):
        ops.check_status(status)
    assert torch.equal(got, want) and torch.equal(k, ek) and torch.equal(v, ev)


def test_commit_refusals():
    g = R.gen(6)
    k, v, table, sl = R.cache(g, [0], 16, 2, 32, layers=2)
    acc = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    with pytest.raises(B.MkError):
        ops.commit_nodes(k, v, table, sl, acc, out=sl)
    with pytest.raises(B.MkError):
        ops.commit_nodes(k, v, table, sl, torch.zeros(1, 513, dtype=torch.int32, device="cuda"))
    with pytest.raises(B.MkError):
        ops.commit_nodes(k, v, table, sl, torch.zeros(1, 0, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        ops.commit_nodes(k[0], v[0], table, sl, acc)
    with pytest.raises(ValueError):
        ops.commit_nodes(k, v, table, sl, acc.long())


def test_captured_on_another_stream():
    g = R.gen(7)
    k, v, table, sl = R.cache(g, [9, 20], 8, 2, 64, layers=3)
    acc = torch.tensor([[2, 5], [1, -1]], dtype=torch.int32, device="cuda")
    ek, ev = k.clone(), v.clone()
    want = commit_ref(ek, ev, table, sl, acc)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    spare_k, spare_v, lens = k.clone(), v.clone(), torch.zeros_like(sl)
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ops.commit_nodes(k, v, table, sl, acc, out=lens)
    graph.replay()
    got = ops.commit_nodes(spare_k, spare_v, table, sl, acc, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(k, ek) and torch.equal(spare_k, ek) and torch.equal(spare_v, ev)
    assert torch.equal(lens, want) and torch.equal(got, want)
