"""mk_moe_layer against float64: selection, weights, both products and their sum."""
import pytest
import torch

import more_ops_ref as M
import ops_ref as R
from persistent_moe_decode_cta_gb300 import binding as B
from persistent_moe_decode_cta_gb300 import ops

pytestmark = pytest.mark.gpu


def weights(g, e, d, f):
    return (R.bf16(g, e, d, std=0.05), R.bf16(g, e, f, d, std=d ** -0.5), R.bf16(g, e, f, d, std=d ** -0.5), R.bf16(g, e, d, f, std=f ** -0.5))


def check(t, e, k, d, f, residual=True, x_extra=0, r_extra=0, out_extra=0, seed=0, spoil=None, in_place=False):
    g = R.gen(seed)
    x = R.bf16(g, t, d + x_extra)[:, :d]
    router, gate, up, down = weights(g, e, d, f)
    if spoil:
        spoil(x, router)
    r = R.bf16(g, t, d + r_extra) if residual else None
    res = None if r is None else r[:, :d]
    want, bound, ids, c = M.moe(x, router, gate, up, down, k, res)
    got_ids = torch.full((t, k), -7, dtype=torch.int32, device="cuda")
    got_c = torch.zeros(t, k, device="cuda")
    whole = r if in_place else torch.full((t, d + out_extra), 3.0, dtype=torch.bfloat16, device="cuda")
    before = whole.clone()
    status = ops.new_status()
    ops.moe_layer(x, router, gate, up, down, k, residual=res, ids=got_ids, weights=got_c, out=whole[:, :d], status=status)
    ops.check_status(status)
    assert torch.equal(got_ids.long(), ids)
    # an fp32 score is off by (d / 64 + 12) 2^-24 |w| |x| at most (a sum of d terms in 64 parts), a weight by twice that of itself,
    # and by 2^-20 from the exponentials and their sum
    off = (d / 64 + 12) * 2.0 ** -24 * float(x.double().norm(dim=1).max() * router.double().norm(dim=1).max())
    assert float((got_c.double() - c).abs().max()) <= 2 * off + 2.0 ** -20
    R.assert_close(whole[:, :d], want, bound, f"{t} tokens")
    assert torch.equal(whole[:, d:], before[:, d:])
    if not in_place:
        again = ops.moe_layer(x, router, gate, up, down, k, residual=res)
        assert torch.equal(again, whole[:, :d])


@pytest.mark.parametrize("t", [1, 2, 3, 7, 8, 9, 16, 31, 33, 64, 65, 100, 128, 129, 255, 256])
def test_tokens(t):
    check(t, 8, 2, 256, 128, residual=t % 2 == 0)


@pytest.mark.parametrize("t", [1, 5, 20, 100])
@pytest.mark.parametrize("e,k,d,f", [(1, 1, 8, 8), (3, 3, 64, 72), (5, 2, 136, 40), (33, 4, 1024, 512), (256, 16, 128, 64), (40, 16, 72, 200),
                                     (16, 1, 2568, 24), (7, 5, 520, 1032)])
def test_sizes(t, e, k, d, f):
    check(t, e, k, d, f)


@pytest.mark.parametrize("t", [1, 16, 128, 250])
def test_pages_scale(t):
    check(t, 128, 8, 2048, 768)


@pytest.mark.parametrize("t", [3, 30, 200])
@pytest.mark.parametrize("x_extra,r_extra,out_extra", [(8, 0, 0), (0, 3, 0), (0, 0, 5), (16, 7, 9)])
def test_strides(t, x_extra, r_extra, out_extra):
    check(t, 12, 3, 192, 64, x_extra=x_extra, r_extra=r_extra, out_extra=out_extra)


@pytest.mark.parametrize("t", [1, 8, 40, 256])
def test_the_residual_in_place(t):
    check(t, 8, 2, 256, 128, in_place=True)
    check(t, 8, 2, 256, 128, in_place=True, r_extra=11)


@pytest.mark.parametrize("t", [1, 8, 64, 256])
def test_every_token_to_the_same_experts(t):
    """One expert's rows fill several tiles, others have none."""
    def same(x, router):
        x[:] = x[:1]
    check(t, 24, 3, 256, 128, spoil=same)


@pytest.mark.parametrize("t", [1, 6, 50])
def test_equal_scores_go_to_the_lower_expert(t):
    def equal(x, router):
        router[3:] = router[3]
    check(t, 40, 4, 128, 64, spoil=equal)

    def nothing(x, router):
        router[:] = 0
    check(t, 40, 4, 128, 64, spoil=nothing)


def test_scores_that_differ_in_their_last_bits():
    """Two experts' scores differ by 2^-30 of the sum of their terms' sizes: an fp32 sum cannot tell them apart."""
    d = 512
    x = torch.ones(4, d, dtype=torch.bfloat16, device="cuda")
    x[:, 1::2] = -1
    router = torch.zeros(6, d, dtype=torch.bfloat16, device="cuda")
    router[:, :] = torch.linspace(100, 200, d // 2, device="cuda").repeat_interleave(2).to(torch.bfloat16)   # (pairs cancel)
    for e in range(6):
        router[e, 2 * e] = router[e, 2 * e]
        router[e, -1] = 0
        x[:, -1] = 0
        router[e, -2] = 2.0 ** -14 * (1 + (5 * e) % 6)
    x[:, -2] = 1
    g = R.gen(8)
    _, gate, up, down = weights(g, 6, d, 64)
    ids = torch.zeros(4, 3, dtype=torch.int32, device="cuda")
    ops.moe_layer(x, router, gate, up, down, 3, ids=ids)
    want, _ = M.select(M.scores(x, router), 3)
    assert torch.equal(ids.long(), want) and len(set(want[0].tolist())) == 3 and want[0].tolist() != [0, 1, 2]


def test_scores_that_are_not_finite():
    """A NaN score is the largest; the outputs of such a token are NaN, those of others are as ever."""
    g = R.gen(9)
    x, (router, gate, up, down) = R.bf16(g, 5, 64), weights(g, 8, 64, 32)
    x[1, 3] = float("nan")
    x[2, 4] = float("inf")
    ids = torch.zeros(5, 2, dtype=torch.int32, device="cuda")
    y = ops.moe_layer(x, router, gate, up, down, 2, ids=ids)
    assert ids.min() >= 0 and ids.max() < 8 and (ids[:, 0] != ids[:, 1]).all()
    assert torch.isnan(y[1:3]).all()
    fine = [0, 3, 4]
    want, bound, want_ids, _ = M.moe(x[fine], router, gate, up, down, 2)
    assert torch.equal(ids[fine].long(), want_ids)
    R.assert_close(y[fine], want, bound)


def test_no_tokens():
    g = R.gen(10)
    router, gate, up, down = weights(g, 4, 64, 32)
    assert ops.moe_layer(router[:0], router, gate, up, down, 2).shape == (0, 64)


def test_one_row_more_than_the_layer_takes():
    g = R.gen(11)
    router, gate, up, down = weights(g, 4, 64, 32)
    with pytest.raises(B.MkError) as e:
        ops.moe_layer(R.bf16(g, 257, 64), router, gate, up, down, 2)
    assert e.value.code == B.MK_ERR_UNSUPPORTED


@pytest.mark.parametrize("t", [1, 20, 200])
def test_captured_replay(t):
    g = R.gen(12)
    x, (router, gate, up, down) = R.bf16(g, t, 128), weights(g, 16, 128, 64)
    out = torch.zeros(t, 128, dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.moe_layer(x, router, gate, up, down, 4, residual=x, out=out)
    x.copy_(R.bf16(g, t, 128))
    for _ in range(3):
        graph.replay()
        want, bound, _, _ = M.moe(x, router, gate, up, down, 4, x)
        R.assert_close(out, want, bound)


def test_many_calls_side_by_side():
    """Calls that share the GPU: a wait for the first product never waits for a CTA that cannot start."""
    g = R.gen(13)
    jobs = []
    for i, t in enumerate((1, 8, 30, 128, 256, 2)):
        w = weights(g, 32, 512, 256)
        jobs.append((R.bf16(g, t, 512), w))
    want = [ops.moe_layer(x, *w, 4) for x, w in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(30):
        got = [ops.moe_layer(x, *w, 4, stream=s) for (x, w), s in zip(jobs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    ops.check_status()


@pytest.mark.parametrize("t", [2, 18])
def test_weights_beyond_32_bits(t):
    """More than 2^32 bytes in each of the experts' tensors."""
    check(t, 40, 2, 8192, 8192)


@pytest.mark.parametrize("t,d", [(1, 2048), (4, 2048), (6, 256), (50, 256), (200, 72)])
@pytest.mark.parametrize("e,k", [(65, 4), (128, 8), (256, 16)])
def test_equal_scores_among_many_experts(t, d, e, k):
    """Ties inside the selection, at its border and behind it, and nothing but ties."""
    def inside(x, router):
        router[40] = router[3]
        router[e - 1] = router[10]
    check(t, e, k, d, 16, spoil=inside)

    def border(x, router):
        router[k // 2:] = router[k // 2]
    check(t, e, k, d, 16, spoil=border)

    def nothing(x, router):
        router[:] = 0
    check(t, e, k, d, 16, spoil=nothing)


def test_many_scores_that_differ_in_their_last_bits():
    """As above with 100 experts: the selected five lie within 2^-30 of the terms' sizes of one another, the others far below."""
    d = 512
    x = torch.ones(3, d, dtype=torch.bfloat16, device="cuda")
    x[:, 1::2] = -1
    x[:, -1] = 0
    router = torch.zeros(100, d, dtype=torch.bfloat16, device="cuda")
    router[:] = torch.linspace(100, 200, d // 2, device="cuda").repeat_interleave(2).to(torch.bfloat16)   # (pairs cancel)
    router[:, -1] = 0
    router[:, -2] = -5
    for i, e in enumerate([7, 31, 64, 65, 99]):
        router[e, -2] = 2.0 ** -14 * (1 + (2 * i) % 5)
    g = R.gen(18)
    _, gate, up, down = weights(g, 100, d, 64)
    ids = torch.zeros(3, 4, dtype=torch.int32, device="cuda")
    ops.moe_layer(x, router, gate, up, down, 4, ids=ids)
    want, _ = M.select(M.scores(x, router), 4)
    assert torch.equal(ids.long(), want) and want[0].tolist() == [64, 99, 31, 65]   # (5, 4, 3 and 2 of 1, 3, 5, 2, 4)


def test_many_scores_that_are_not_finite():
    g = R.gen(19)
    x, (router, gate, up, down) = R.bf16(g, 5, 64), weights(g, 90, 64, 32)
    x[1, 3] = float("nan")
    x[2, 4] = float("inf")
    router[80, 5] = float("inf")           # (one expert's scores, of any sign, for every token)
    ids = torch.zeros(5, 3, dtype=torch.int32, device="cuda")
    ops.moe_layer(x, router, gate, up, down, 3, ids=ids)
    assert ids.min() >= 0 and ids.max() < 90 and all(len(set(r)) == 3 for r in ids.tolist())
    fine = [0, 3, 4]
    want, _ = M.select(M.scores(x, router)[fine], 3)
    assert torch.equal(ids[fine].long(), want)


@pytest.mark.parametrize("t", [1, 4, 5, 8, 9, 40, 200])
@pytest.mark.parametrize("e,k,d,f", [(8, 2, 256, 128), (32, 4, 1024, 512)])
def test_one_rounding_of_the_result(t, e, k, d, f):
    """In the 2-norm the result is off by its own rounding: what the products add (the inner results, kept to 2^-17, the weights to
    2^-20, sums of up to 1024 terms in fp32) is below 2^-12.  An inner result in one bf16 value would be as much as the rounding."""
    g = R.gen(20 + t)
    x, (router, gate, up, down) = R.bf16(g, t, d), weights(g, e, d, f)
    got = ops.moe_layer(x, router, gate, up, down, k).double()
    want = M.moe(x, router, gate, up, down, k)[0]
    rounding = (want.to(torch.bfloat16).double() - want).norm()
    assert float((got - want).norm()) <= float(rounding + 2.0 ** -12 * want.norm())


@pytest.mark.parametrize("t", [1, 2, 4, 5, 8, 9, 40, 200])
@pytest.mark.parametrize("e,k,d,f", [(8, 2, 256, 128), (20, 3, 72, 200)])
def test_weights_that_are_not_finite_stay_with_the_tokens_that_chose_them(t, e, k, d, f):
    """Infinities and a NaN in the second matrix of some experts: the outputs of tokens that have not selected those are as ever, those of
    the others what the formula gives."""
    g = R.gen(30 + t)
    x, (router, gate, up, down) = R.bf16(g, t, d), weights(g, e, d, f)
    router[2], router[1] = 0.5 * router[2], 0.0
    down[1, 3, 5], down[1, 60, 9] = float("inf"), float("nan")
    down[2, 7, f - 1], down[2, 8] = -float("inf"), float("inf")
    down[4, 7, 0] = float("inf")
    r = R.bf16(g, t, d)
    got_ids = torch.zeros(t, k, dtype=torch.int32, device="cuda")
    for res in (None, r):
        want, bound, ids, _ = M.moe(x, router, gate, up, down, k, res)
        y = ops.moe_layer(x, router, gate, up, down, k, residual=res, ids=got_ids)
        assert torch.equal(got_ids.long(), ids)
        R.assert_close(y, want, bound, f"{t} tokens")
        assert torch.equal(y.view(torch.int16), ops.moe_layer(x, router, gate, up, down, k, residual=res).view(torch.int16))


@pytest.mark.parametrize("e,k,d", [(8, 2, 512), (60, 4, 1024), (100, 8, 2048), (256, 16, 512)])
@pytest.mark.parametrize("x_size,router_size", [(0, 0), (-76, 0), (-76, 13), (-100, 10), (0, -76), (13, -90), (-60, -50)])
def test_equal_scores_of_any_size(e, k, d, x_size, router_size):
    """Rows of the router that are one another's permutations and tokens of equal values: all scores are equal, sums in fp32 are not, however
    small the squares of what they are sums of.  Ties go to the lowest experts."""
    g = R.gen(40)
    line = torch.randn(d, generator=g, device="cuda") * 2.0 ** torch.randint(-10, 11, (d,), generator=g, device="cuda")
    line = torch.where(line.abs() < 2.0 ** -10, 1.0, line)            # (sums of 32 bits or so, no term below 2^-120)
    order = torch.rand(e, d, generator=g, device="cuda").argsort(-1)
    router = (line.to(torch.bfloat16).float()[order] * 2.0 ** router_size).to(torch.bfloat16)
    x = torch.full((5, d), 2.0 ** x_size, dtype=torch.bfloat16, device="cuda")
    x[1] *= -1.5
    x[3] = 0
    _, gate, up, down = weights(g, e, d, 16)
    ids = torch.full((5, k), -1, dtype=torch.int32, device="cuda")
    share = torch.zeros(5, k, device="cuda")
    ops.moe_layer(x, router, gate, up, down, k, ids=ids, weights=share)
    assert torch.equal(ids, torch.arange(k, dtype=torch.int32, device="cuda").expand(5, k))
    assert float((share - 1 / k).abs().max()) <= 2.0 ** -20 / k      # (exponentials of 0, a sum of k and a quotient)
