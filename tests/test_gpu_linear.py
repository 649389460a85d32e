"""mk_linear against float64: sizes, strides, activations, both result types, every split of the work."""
import pytest
import torch

import more_ops_ref as M
import ops_ref as R
from persistent_moe_decode_cta_gb300 import ops

pytestmark = pytest.mark.gpu


def check(m, n, k, bias=True, act=None, residual=True, wide=False, x_extra=0, r_extra=0, out_extra=0, in_place=False, seed=0):
    g = R.gen(seed)
    x = R.bf16(g, m, k + x_extra)[:, :k]
    w = R.bf16(g, n, k, std=k ** -0.5)
    b = R.bf16(g, n, std=0.5) if bias else None
    r = R.bf16(g, m, n + r_extra) if residual else None
    want, bound = M.linear(x, w, b, act, None if r is None else r[:, :n], wide)
    dtype = torch.float32 if wide else torch.bfloat16
    whole = r if in_place else torch.full((m, n + out_extra), 3.0, dtype=dtype, device="cuda")
    before = whole.clone()
    status = ops.new_status()
    got = ops.linear(x, w, bias=b, activation=act, residual=None if r is None else r[:, :n], out=whole[:, :n], dtype=dtype, status=status)
    ops.check_status(status)
    assert got.data_ptr() == whole.data_ptr() and got.dtype == dtype
    R.assert_close(whole[:, :n], want, bound, f"{m} {n} {k}")
    assert torch.equal(whole[:, n:], before[:, n:])
    # equal calls, equal bits
    if not in_place:
        again = ops.linear(x, w, bias=b, activation=act, residual=None if r is None else r[:, :n], dtype=dtype)
        assert torch.equal(again, whole[:, :n])


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("m", [1, 2, 7, 8, 9, 16, 17, 31, 33, 64, 65, 100, 128, 129, 200, 255, 256, 257, 513])
def test_rows(m, wide):
    check(m, 384, 256, wide=wide)


@pytest.mark.parametrize("m", [1, 8, 24, 100, 300])
@pytest.mark.parametrize("n,k", [(1, 8), (8, 8), (3, 64), (130, 72), (257, 200), (1000, 1032), (15, 2048), (2048, 16), (5121, 136), (700, 4096)])
def test_sizes(m, n, k):
    check(m, n, k)


@pytest.mark.parametrize("act", M.ACTS)
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("m", [3, 40, 300])
def test_activations(m, act, wide):
    check(m, 264, 128, act=act, wide=wide, residual=m != 40)


@pytest.mark.parametrize("m", [5, 70, 400])
@pytest.mark.parametrize("x_extra,r_extra,out_extra", [(8, 0, 0), (0, 3, 0), (0, 0, 1), (24, 8, 4), (64, 5, 7)])
def test_strides(m, x_extra, r_extra, out_extra):
    check(m, 200, 136, x_extra=x_extra, r_extra=r_extra, out_extra=out_extra)
    check(m, 200, 136, x_extra=x_extra, r_extra=r_extra, out_extra=out_extra, wide=True, act="silu")


@pytest.mark.parametrize("m", [1, 12, 90, 300])
def test_the_residual_in_place(m):
    check(m, 256, 192, in_place=True)
    check(m, 256, 192, in_place=True, r_extra=9, act="gelu")


@pytest.mark.parametrize("m", [1, 6, 30, 128, 500])
def test_without_anything(m):
    check(m, 320, 256, bias=False, residual=False)


def test_odd_addresses():
    """Bias, residual and result at addresses that are no multiple of four values."""
    g = R.gen(3)
    for m in (3, 50, 290):
        x, w = R.bf16(g, m, 128), R.bf16(g, 96, 128, std=0.1)
        b, r, out = R.bf16(g, 97)[1:], R.bf16(g, m * 96 + 1)[1:].view(m, 96), torch.zeros(m * 96 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(m, 96)
        ops.linear(x, w, bias=b, residual=r, out=out)
        R.assert_close(out, *M.linear(x, w, b, None, r))


def test_columns_of_one_tensor():
    """Result and residual as columns of the same rows."""
    g = R.gen(4)
    for m in (4, 60, 300):
        both = R.bf16(g, m, 256)
        r = both[:, 128:].clone()
        x, w = R.bf16(g, m, 64), R.bf16(g, 128, 64, std=0.1)
        ops.linear(x, w, residual=both[:, 128:], out=both[:, :128])
        R.assert_close(both[:, :128], *M.linear(x, w, None, None, r))
        assert torch.equal(both[:, 128:], r)


@pytest.mark.parametrize("m", [2, 20, 130, 300])
def test_values_that_are_not_finite_stay_in_their_rows_and_columns(m):
    g = R.gen(5)
    x, w = R.bf16(g, m, 64), R.bf16(g, 40, 64, std=0.1)
    x[1, 5] = float("nan")
    w[7, 3] = float("inf")
    y = ops.linear(x, w, activation="silu")
    keep = torch.ones(m, 40, dtype=torch.bool, device="cuda")
    keep[1] = keep[:, 7] = False
    assert torch.isnan(y[1]).all() and ((y[:, 7] == 0) | ~torch.isfinite(y[:, 7])).all()   # (silu of -infinity is no number, or zero)
    want, bound = M.linear(torch.nan_to_num(x), torch.nan_to_num(w, posinf=0.0), None, "silu")
    R.assert_close(y[keep], want[keep], bound[keep])


def test_activations_far_out():
    """Both tails, where a form with 1 + tanh or 1 + erf cancels, and infinity."""
    x = torch.zeros(33, 8, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = torch.linspace(-40, 40, 33, device="cuda")
    x[32, 0] = float("inf")
    w = torch.zeros(1, 8, dtype=torch.bfloat16, device="cuda")
    w[0, 0] = 1
    for act in ("relu", "silu", "gelu", "gelu_tanh"):
        for rows in (x, x[-8:]):
            y = ops.linear(rows, w, activation=act, dtype=torch.float32)
            want, bound = M.linear(torch.nan_to_num(rows, posinf=100.0), w, None, act, None, True)
            R.assert_close(y[:-1], want[:-1], bound[:-1] + 2e-38, act)   # (denormal results may be zero)
            assert y[-1, 0] == float("inf")


def test_no_rows():
    w = torch.zeros(16, 64, dtype=torch.bfloat16, device="cuda")
    assert ops.linear(w[:0], w).shape == (0, 16)


@pytest.mark.parametrize("m,n,k", [(128, 2048, 4096), (16, 5120, 2048), (2001, 4096, 2048), (9, 151936, 2048)])
def test_model_shapes(m, n, k):
    check(m, n, k, bias=False, wide=n > 100000, residual=n < 100000)


def test_captured_replay():
    g = R.gen(6)
    for m in (4, 48, 300):
        x, w, r = R.bf16(g, m, 128), R.bf16(g, 192, 128, std=0.1), R.bf16(g, m, 192)
        out = torch.zeros(m, 192, dtype=torch.bfloat16, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ops.linear(x, w, residual=r, activation="gelu_tanh", out=out)
        x.copy_(R.bf16(g, m, 128))
        for _ in range(2):
            graph.replay()
            R.assert_close(out, *M.linear(x, w, None, "gelu_tanh", r))


def test_offsets_beyond_32_bits():
    """Rows whose elements lie further than 2^32 bytes apart."""
    g = R.gen(7)
    stride = (1 << 31) // 2 + 64
    big = torch.empty(2 * stride + 256, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(big, (3, 128), (stride, 1))
    x.copy_(R.bf16(g, 3, 128))
    w = R.bf16(g, 64, 128, std=0.1)
    R.assert_close(ops.linear(x, w), *M.linear(x, w))
    # ... of the result and the residual, in both forms of the product
    for n in (64, 20000):
        stride = (1 << 31) // 2 + 20000
        big = torch.empty(2 * stride + 20000, dtype=torch.bfloat16, device="cuda")
        both = torch.as_strided(big, (3, n), (stride, 1))
        both.copy_(R.bf16(g, 3, n))
        x, w, before = R.bf16(g, 3, 64), R.bf16(g, n, 64, std=0.1), both.clone()
        ops.linear(x, w, residual=both, out=both)
        R.assert_close(both, *M.linear(x, w, None, None, before))


@pytest.mark.parametrize("act", M.ACTS)
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("m", [2, 300])
def test_activations_at_the_ends_of_the_range(m, act, wide):
    """What the formula gives for infinite, NaN and huge sums: an infinite sum stays, a product of zero and infinity is a NaN."""
    ends = [float("inf"), -float("inf"), float("nan"), 3e38, -3e38, 1e30, -1e30, 1e13, -1e13, 40.0, -40.0, 0.0, -0.0, 1e-38, -1e-38]
    n = 8 * len(ends)
    b = torch.tensor(ends, device="cuda").repeat(8).to(torch.bfloat16)
    x = torch.zeros(m, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(n, 64, dtype=torch.bfloat16, device="cuda")
    got = ops.linear(x, w, bias=b, activation=act, dtype=torch.float32 if wide else torch.bfloat16).double()
    y = b.double().expand(m, n)
    want, rel, _ = M.activation(y, act)
    assert torch.equal(got.isnan(), want.isnan())
    some = want.isinf()
    assert torch.equal(got[some], want[some])
    rest = ~want.isnan() & ~some
    rel = torch.as_tensor(rel, device="cuda").expand_as(want)[rest]
    step = 2.0 ** -24 if wide else 2.0 ** -8
    # (a value below the smallest normal one may be zero)
    assert ((got[rest] - want[rest]).abs() <= want[rest].abs() * (step + rel) + 2.0 ** -126).all()


@pytest.mark.parametrize("m,n,k", [(1024, 2048, 4096), (512, 2048, 4096), (1000, 1500, 4104), (1024, 2048, 16384), (130, 250, 16384), (1, 700, 16384),
                                   (9, 2048, 24576), (40, 100, 1024), (72, 30000, 4096)])
def test_long_sums_of_float32_results(m, n, k):
    """In the 2-norm, whatever the length and whichever kernel has the product: the products' accumulator drops what lies below its last
    bit, half a step (2^-24) of the sum so far in the mean, at every 16 columns.  Segments of 512 columns (32 additions, of sums that are
    two thirds of the last one in the mean, mantissas 0.7 of a step) make that 9e-7 at most; joining them adds 2^-25 each, at random."""
    g = R.gen(k + m)
    x, w = R.bf16(g, m, k), R.bf16(g, n, k, std=k ** -0.5)
    got = ops.linear(x, w, dtype=torch.float32).double()
    want = x.double() @ w.double().T
    assert float((got - want).norm() / want.norm()) <= 1e-6
