"""mk_expert_product against float64: ragged groups, gathered rows, SwiGLU."""
import pytest
import torch

import ops_ref as R
from persistent_moe_decode_cta_gb300 import binding as B
from persistent_moe_decode_cta_gb300 import ops

pytestmark = pytest.mark.gpu


def reference(x, w, offsets, w_up, rows):
    """(result, bound).  Products of bf16 values are exact in fp32 and k of them are summed
    with a rounding or truncation each, at most 2^-23 of sum |x||w|: k * 2^-23 of that sum.
    silu' is at most 1.1; the result is rounded once (2^-8)."""
    first = int(offsets[0])
    n_rows, k = int(offsets[-1]), x.shape[1]
    y = torch.zeros(n_rows, w.shape[1], dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(y)
    for e in range(w.shape[0]):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if a == b:
            continue
        xs = (x[a:b] if rows is None else x[rows[a:b].long()]).double()
        g = xs @ w[e].double().T
        dg = xs.abs() @ w[e].double().abs().T * k * 2.0 ** -23
        if w_up is None:
            y[a:b], bound[a:b] = g, dg
        else:
            u = xs @ w_up[e].double().T
            du = xs.abs() @ w_up[e].double().abs().T * k * 2.0 ** -23
            s = g * torch.sigmoid(g)
            y[a:b] = s * u
            bound[a:b] = 1.1 * dg * u.abs() + s.abs() * du + dg * du + 2.0 ** -19 * (s * u).abs()
    return y[first:], (bound + R.HALF_BF16 * y.abs() + 1e-30)[first:]


def check(sizes, n, k, glu=False, gather=None, first=0, pad=0, x_extra=0, out_extra=0, seed=0):
    g = R.gen(seed)
    e = len(sizes)
    ends = torch.tensor([0] + sizes, device="cuda").cumsum(0) + first
    offsets = ends.to(torch.int32)
    total = int(offsets[-1]) + pad
    n_x = total if gather is None else gather
    x = R.bf16(g, n_x, k + x_extra)[:, :k]
    rows = None if gather is None else torch.randint(0, gather, (total,), generator=g, device="cuda").to(torch.int32)
    w = R.bf16(g, e, n, k, std=0.05)
    w_up = R.bf16(g, e, n, k, std=0.05) if glu else None
    out = torch.full((total, n + out_extra), 3.0, dtype=torch.bfloat16, device="cuda")
    status = ops.new_status()
    ops.expert_product(x, w, offsets, w_up=w_up, rows=rows, out=out[:, :n], status=status)
    ops.check_status(status)
    want, bound = reference(x, w, offsets, w_up, rows)
    live = out[first:int(offsets[-1]), :n]
    R.assert_close(live, want, bound)
    keep = torch.full_like(out, 3.0)
    keep[first:int(offsets[-1]), :n] = live
    assert torch.equal(out, keep)   # rows of no expert and columns behind the result


@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("sizes", [[1], [0, 0, 3], [2, 0, 130, 17, 0], [128, 128], [1] * 40, [129, 1, 255, 300]])
def test_ragged_groups(sizes, glu):
    check(sizes, 256, 192, glu)


@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("n,k", [(128, 256), (256, 128), (8, 8), (1, 64), (130, 72), (257, 200), (768, 1024), (383, 40)])
def test_sizes(n, k, glu):
    check([5, 0, 33, 140], n, k, glu)


@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("n_x", [1, 7, 500])
def test_gathered_rows(n_x, glu):
    check([3, 0, 130, 64, 1], 384, 256, glu, gather=n_x)


def test_strides_first_row_and_padding():
    check([3, 40, 0, 9], 264, 128, first=5, pad=11, x_extra=24, out_extra=3)
    check([3, 40, 0, 9], 264, 128, True, first=5, pad=11, x_extra=8, out_extra=8, gather=20)


def test_all_rows_to_one_expert_and_none():
    check([0] * 100 + [700] + [0] * 155, 128, 128)
    check([0, 0], 128, 128, pad=4)


@pytest.mark.parametrize("glu,gather,rows", [(False, None, 150), (True, 77, 150), (False, 500, 6)])
def test_many_tiles_of_few_columns(glu, gather, rows):
    """A cluster has more tiles under way than the ring has stages (64 columns: one stage a tile)."""
    check([rows + i % 7 for i in range(64)], 4096 + 40, 64, glu=glu, gather=gather)


def test_pages_scale_shapes():
    g = torch.Generator().manual_seed(3)
    sizes = torch.bincount(torch.randint(0, 128, (1024,), generator=g), minlength=128).tolist()
    check(sizes, 768, 2048, True, gather=128)
    check(sizes, 2048, 768)


def test_values_that_are_not_finite_stay_in_their_rows():
    g = R.gen(4)
    x = R.bf16(g, 6, 64)
    x[2, 5] = float("nan")
    x[3, 0] = float("inf")
    w = R.bf16(g, 2, 40, 64, std=0.1)
    off = torch.tensor([0, 3, 6], dtype=torch.int32, device="cuda")
    y = ops.expert_product(x, w, off)
    assert torch.isnan(y[2]).all() and not torch.isfinite(y[3]).any()
    fine = [0, 1, 4, 5]
    want, bound = reference(torch.nan_to_num(x, nan=0.0, posinf=0.0), w, off, None, None)
    R.assert_close(y[fine], want[fine], bound[fine])


def test_bad_offsets_and_rows_are_reported_and_clamped():
    g = R.gen(5)
    x, w = R.bf16(g, 8, 64), R.bf16(g, 2, 40, 64)
    for offsets, rows in (([0, 9, 12], None), ([-3, 2, 8], None), ([4, 2, 8], None), ([0, 4, 8], [0, 1, 2, 3, 4, 5, 6, 8]),
                          ([0, 4, 8], [0, 1, -1, 3, 4, 5, 6, 7])):
        status = ops.new_status()
        r = None if rows is None else torch.tensor(rows, dtype=torch.int32, device="cuda")
        ops.expert_product(x, w, torch.tensor(offsets, dtype=torch.int32, device="cuda"), rows=r, status=status)
        with pytest.raises(B.MkError) as e:
            ops.check_status(status)
        assert e.value.code == B.MK_ERR_INVALID


def test_captured_replay_follows_the_offsets():
    g = R.gen(6)
    x, w, u = R.bf16(g, 50, 128), R.bf16(g, 4, 128, 128, std=0.1), R.bf16(g, 4, 128, 128, std=0.1)
    offsets = torch.tensor([0, 10, 10, 30, 50], dtype=torch.int32, device="cuda")
    out = torch.zeros(50, 128, dtype=torch.bfloat16, device="cuda")
    run = lambda: ops.expert_product(x, w, offsets, w_up=u, out=out)
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    offsets.copy_(torch.tensor([0, 0, 41, 41, 50], dtype=torch.int32))
    x.copy_(R.bf16(g, 50, 128))
    graph.replay()
    want, bound = reference(x, w, offsets, u, None)
    R.assert_close(out, want, bound)
