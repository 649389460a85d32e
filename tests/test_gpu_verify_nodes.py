"""mk_verify_nodes against float64: paths and drawn tokens, exactly."""
import pytest
import torch

import more_ops_ref as M
import ops_ref as R
from persistent_moe_decode_cta_gb300 import binding as B
from persistent_moe_decode_cta_gb300 import ops

pytestmark = pytest.mark.gpu


def check(logits, tokens, uniforms, parents=None, draft=None, temperature=None, counts=None):
    status = ops.new_status()
    accepted, drawn = ops.verify_nodes(logits, tokens, uniforms, parents=parents, draft_probs=draft, temperature=temperature, counts=counts,
                                       status=status)
    ops.check_status(status)
    path, nxt = M.verify(logits, tokens, uniforms, parents, draft, temperature, counts)
    assert accepted.tolist() == path
    assert drawn.tolist() == nxt
    return path


@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("b,n,v", [(1, 1, 1), (1, 1, 2), (2, 2, 5), (3, 5, 17), (4, 9, 127), (2, 8, 128), (2, 8, 129), (5, 3, 1000), (8, 12, 1024),
                                   (2, 6, 4099), (3, 33, 2050), (2, 5, 32000), (1, 4, 151936), (1, 3, 200001), (1, 2, 262144)])
def test_sizes(b, n, v, half, probs):
    for seed in range(3):
        g = R.gen(seed)
        check(*M.tree_inputs(g, b, n, v, True, probs, half=half))


@pytest.mark.parametrize("probs", [True, False])
def test_chains(probs):
    """Drafts that are mostly accepted and mostly rejected; no parents given: a chain."""
    lengths = set()
    for seed in range(8):
        g = R.gen(20 + seed)
        logits, tokens, uniforms, parents, draft = M.tree_inputs(g, 6, 7, 500, False, probs, sharp=3.0 * seed)
        path = check(logits, tokens, uniforms, None, draft)
        assert path == check(logits, tokens, uniforms, parents, draft)
        lengths |= {sum(x >= 0 for x in p) for p in path}
    assert len(lengths) >= 4


@pytest.mark.parametrize("probs", [True, False])
def test_temperatures_and_counts(probs):
    for seed in range(4):
        g = R.gen(40 + seed)
        logits, tokens, uniforms, parents, draft = M.tree_inputs(g, 8, 10, 3001, True, probs)
        temperature = torch.tensor([0.0, 1.0, 0.3, 5.0, 0.0, 0.01, 1e-30, 100.0], device="cuda")
        # greedy sequences whose drafts are the largest logits for a while
        for b in (0, 4, 6):
            best = logits.argmax(-1).to(torch.int32)
            tokens[b, 1:6] = best[b, parents[b, 1:6].long()]
        counts = torch.tensor([10, 1, 10, 5, 7, 2, 9, 3], dtype=torch.int32, device="cuda")
        check(logits, tokens, uniforms, parents, draft, temperature, counts)
        check(logits, tokens, uniforms, parents, draft, temperature)


def test_many_rejected_children():
    """A star: one child after another is cut out of the distribution, drawn again or not."""
    for seed in range(6):
        g = R.gen(60 + seed)
        for probs in (True, False):
            logits, tokens, uniforms, parents, draft = M.tree_inputs(g, 4, 40, 300, True, probs)
            parents[:, 1:] = 0
            uniforms[:, 1:] = 0.5 + 0.5 * uniforms[:, 1:]
            if not probs:
                tokens[:, 5:9] = tokens[:, 1:5]        # the same tokens proposed twice
            check(logits, tokens, uniforms, parents, draft)


def test_draft_equal_to_the_target():
    """Nothing is left of p - q: p stays, and drawn tokens are accepted."""
    g = R.gen(70)
    logits = torch.zeros(3, 4, 64, device="cuda")
    draft = torch.full((3, 4, 64), 1 / 64, device="cuda")
    tokens = torch.randint(0, 64, (3, 4), generator=g, device="cuda").to(torch.int32)
    uniforms = torch.rand(3, 4, generator=g, device="cuda")
    assert check(logits, tokens, uniforms, None, draft) == [[0, 1, 2, 3]] * 3
    # (tokens that the target excludes are rejected; q covers the rest exactly)
    logits[:, :, 32:] = -float("inf")
    draft[:] = 0
    draft[:, :, :32] = 1 / 32
    tokens[:, 1:] = 40
    check(logits, tokens, uniforms, None, draft)


def test_excluded_tokens_and_equal_logits():
    g = R.gen(71)
    logits, tokens, uniforms, parents, draft = M.tree_inputs(g, 4, 6, 777, True, True)
    logits[:, :, ::2] = -float("inf")
    check(logits, tokens, uniforms, parents, draft)
    flat = torch.zeros_like(logits)
    check(flat, tokens, uniforms, parents, draft)
    check(flat, tokens, uniforms, parents, draft, torch.zeros(4, device="cuda"))
    check(flat, tokens, uniforms, parents, None, torch.zeros(4, device="cuda"))


def test_draws_at_both_ends():
    """Uniforms of zero and of the largest value below one, and a running sum that needs all its bits: the drawn token's border
    is met to 2^-40."""
    v = 151936
    logits = torch.full((4, 1, v), -3.0, device="cuda")
    logits[:, :, 7] = 4.0
    logits[1, 0, :5] = -float("inf")
    u = torch.tensor([[0.0], [0.0], [1 - 2.0 ** -24], [0.5]], device="cuda")
    tokens = torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    check(logits, tokens, u)
    g = R.gen(72)
    for seed in range(4):
        logits = torch.randn(8, 1, v, generator=g, device="cuda")
        check(logits, torch.zeros(8, 1, dtype=torch.int32, device="cuda"), torch.rand(8, 1, generator=g, device="cuda"))


def test_strided_rows():
    g = R.gen(73)
    for half in (False, True):
        logits, tokens, uniforms, parents, draft = M.tree_inputs(g, 3, 5, 501, True, True, half=half)
        wide = torch.full((3, 7, 511), float("nan"), dtype=logits.dtype, device="cuda")
        wide[:, 1:6, 3:504] = logits
        q = torch.full((4, 5, 503), float("nan"), device="cuda")
        q[1:, :, 1:502] = draft
        check(wide[:, 1:6, 3:504], tokens, uniforms, parents, q[1:, :, 1:502])


def test_the_distribution_is_the_targets():
    """First tokens of many sequences with one distribution: drafted or not, as often as p says (chi-squared of 7 degrees of
    freedom, the bound is passed by chance once in 10^9 runs; the draws are fixed by the seed)."""
    g = R.gen(74)
    n, v = 40000, 8
    line = torch.randn(v, generator=g, device="cuda")
    p = line.softmax(0)
    q = (torch.randn(v, generator=g, device="cuda") * 1.5).softmax(0)
    logits = line.repeat(n, 4, 1)
    draft = q.repeat(n, 4, 1)
    parents = torch.tensor([-1, 0, 0, 0], dtype=torch.int32, device="cuda").repeat(n, 1)
    tokens = torch.multinomial(q, n * 4, replacement=True, generator=g).view(n, 4).to(torch.int32)
    uniforms = torch.rand(n, 4, generator=g, device="cuda")
    accepted, drawn = ops.verify_nodes(logits, tokens, uniforms, parents=parents, draft_probs=draft)
    second = accepted[:, 1].long()
    first = torch.where(second >= 0, tokens.gather(1, second.clamp(min=0)[:, None])[:, 0], drawn)
    count = torch.bincount(first.long(), minlength=v).double()
    assert float(((count - n * p.double()) ** 2 / (n * p.double())).sum()) < 60
    assert 0.2 < float((second >= 0).float().mean()) < 0.999


@pytest.mark.parametrize("case", ["count", "count0", "temperature", "nan_temperature", "row", "empty_row", "inf_row", "parent", "token", "uniform", "nan_uniform"])
def test_bad_values_are_recorded(case):
    g = R.gen(75)
    logits, tokens, uniforms, parents, draft = M.tree_inputs(g, 3, 6, 100, False, True)
    temperature, counts = torch.ones(3, device="cuda"), torch.full((3,), 6, dtype=torch.int32, device="cuda")
    uniforms[:, 1:] = 0.0                                     # (everything that is looked at is accepted)
    want, _ = M.verify(logits, tokens, uniforms, parents, draft)
    assert want[1] == list(range(6))
    ends = True
    if case == "count":
        counts[1] = 7
    elif case == "count0":
        counts[1] = 0
    elif case == "temperature":
        temperature[1] = -0.5
    elif case == "nan_temperature":
        temperature[1] = float("nan")
    elif case == "row":
        logits[1, 2, 50] = float("nan")
    elif case == "empty_row":
        logits[1, 2] = -float("inf")
    elif case == "inf_row":
        logits[1, 2, 50] = float("inf")
    else:
        ends = False
        if case == "parent":
            parents[1, 3] = 3
        elif case == "token":
            tokens[1, 3] = 100
        elif case == "uniform":
            uniforms[1, 3] = 1.0
        else:
            uniforms[1, 3] = float("nan")
    status = ops.new_status()
    accepted, drawn = ops.verify_nodes(logits, tokens, uniforms, parents=parents, draft_probs=draft, temperature=temperature, counts=counts,
                                       status=status)
    assert status[0] == B.MK_ERR_INVALID and status[1] == 1
    with pytest.raises(B.MkError):
        ops.check_status(status)
    for b in (0, 2):
        assert accepted[b].tolist() == want[b]
    if ends:
        length = 3 if "row" in case else 0
        assert accepted[1].tolist() == list(range(length)) + [-1] * (6 - length) and int(drawn[1]) == -1
    else:
        assert accepted[1].tolist() == [0, 1, 2, -1, -1, -1] and 0 <= int(drawn[1]) < 100


def test_no_sequences():
    z = torch.zeros(0, 3, 10, device="cuda")
    i = torch.zeros(0, 3, dtype=torch.int32, device="cuda")
    accepted, drawn = ops.verify_nodes(z, i, torch.zeros(0, 3, device="cuda"))
    assert accepted.shape == (0, 3) and drawn.shape == (0,)


def test_captured_replay():
    g = R.gen(76)
    a = M.tree_inputs(g, 4, 8, 3000, True, True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        accepted, drawn = ops.verify_nodes(a[0], a[1], a[2], parents=a[3], draft_probs=a[4])
    for seed in range(3):
        for old, new in zip(a, M.tree_inputs(R.gen(80 + seed), 4, 8, 3000, True, True)):
            old.copy_(new)
        graph.replay()
        path, nxt = M.verify(a[0], a[1], a[2], a[3], a[4])
        assert accepted.tolist() == path and drawn.tolist() == nxt


def test_many_sequences():
    """More clusters than fit the GPU at once."""
    g = R.gen(77)
    logits, tokens, uniforms, parents, draft = M.tree_inputs(g, 70, 4, 20000, True, True)
    check(logits, tokens, uniforms, parents, draft)


def test_offsets_beyond_32_bits():
    """Sequences whose rows lie further than 2^32 bytes apart."""
    g = R.gen(78)
    for half in (True, False):
        logits, tokens, uniforms, parents, draft = M.tree_inputs(g, 3, 4, 900, True, True, half=half)
        stride = (1 << 31) // logits.element_size() + 4096
        far = torch.as_strided(torch.empty(2 * stride + 4 * 900, dtype=logits.dtype, device="cuda"), logits.shape, (stride, 900, 1))
        far.copy_(logits)
        apart = (1 << 30) // 2 + 1024
        q = torch.as_strided(torch.empty(2 * apart + 4 * 900, device="cuda"), draft.shape, (apart, 900, 1))
        q.copy_(draft)
        check(far, tokens, uniforms, parents, q)


def test_a_long_chain_and_deep_tree():
    """As many nodes as a call takes."""
    g = R.gen(79)
    for tree in (False, True):
        logits, tokens, uniforms, parents, draft = M.tree_inputs(g, 2, 512, 257, tree, True, sharp=30.0)
        uniforms[:, 1:] *= 0.3
        check(logits, tokens, uniforms, parents, draft)
        # whatever may be drafted at all is accepted.  (The draw keeps its number: 0 would be the border in front of the first token of
        # all, which the integers of 2^-44 of the largest probability leave at 0 where it is below 2^-45 of that.)
        sure = uniforms * 0
        sure[:, 0] = uniforms[:, 0]
        path = check(logits, tokens, sure, parents, draft)
        assert tree or path == [list(range(512))] * 2


@pytest.mark.parametrize("bad", ["nan", "inf", "empty"])
def test_bad_rows_where_the_walk_ends(bad):
    """The row of a node without children."""
    g = R.gen(90)
    logits, tokens, uniforms, parents, draft = M.tree_inputs(g, 3, 6, 300, False, True)
    uniforms[:, 1:] = 0.0
    want, drawn = M.verify(logits, tokens, uniforms, parents, draft)
    if bad == "empty":
        logits[1, 5] = -float("inf")
    else:
        logits[1, 5, 299] = float(bad)
    for temperature in (None, torch.tensor([1.0, 0.0, 1.0], device="cuda")):
        status = ops.new_status()
        if temperature is not None:
            tokens[1, 1:] = logits[1, :5].argmax(-1).to(torch.int32)
        accepted, nxt = ops.verify_nodes(logits, tokens, uniforms, parents=parents, draft_probs=draft, temperature=temperature, status=status)
        assert status[:3].tolist() == [B.MK_ERR_INVALID, 1, 5]
        assert accepted.tolist() == want and want[1] == list(range(6))
        assert int(nxt[1]) == -1 and [int(nxt[0]), int(nxt[2])] == [drawn[0], drawn[2]]


def test_little_left_behind_a_rejection():
    """Drafts from all but the target's own distribution: what a rejection leaves is small beside what it takes away."""
    for seed in range(6):
        g = R.gen(91 + seed)
        logits, tokens, uniforms, parents, _ = M.tree_inputs(g, 4, 12, 700, True, False)
        draft = (logits + 1e-4 * torch.randn(logits.shape, generator=g, device="cuda")).softmax(-1)
        parents[:, 1:] = parents[:, 1:] // 2
        tokens[:, 1::3] = logits.argmin(-1)[:, :1].to(torch.int32)      # (some that are hardly ever accepted)
        uniforms[:, 1:] = 1 - 2.0 ** -24
        check(logits, tokens, uniforms, parents, draft)


def test_excluded_drafts_with_siblings():
    """The target excludes what was drafted first: every sibling is tested against what is left."""
    for half in (False, True):
        g = R.gen(98)
        logits, tokens, uniforms, parents, draft = M.tree_inputs(g, 6, 14, 2500, True, True, half=half)
        parents[:, 1:] = (torch.arange(1, 14, device="cuda") - 1) // 4
        for b in range(6):
            for i in range(1, 14, 2):
                logits[b, int(parents[b, i]), int(tokens[b, i])] = -float("inf")
        check(logits, tokens, uniforms, parents, draft)


@pytest.mark.parametrize("v,spread,heat,n", [(262144, 0.0, 1.0, 24), (151936, 2.5, 20.0, 32), (100003, 2.5, 100.0, 32)])
def test_many_rejections_on_a_flat_row(v, spread, heat, n):
    """One child after another is cut out of a row of hundreds of thousands of tokens of about the same size: what is cut adds up to
    many times the whole, and what an earlier rejection has taken stays away, however many there were."""
    b = 16
    g = R.gen(110)
    line = spread * torch.randn(b, v, generator=g, device="cuda")
    # what was drafted lies in one half of the tokens, with more than the target gives them there
    half = torch.rand(b, v, generator=g, device="cuda") < 0.5
    q = torch.where(half, torch.rand(b, v, generator=g, device="cuda") + 0.5, 0.0)
    q = q / q.sum(-1, keepdim=True)
    row = torch.arange(b, device="cuda")
    counts = n - row.to(torch.int32)
    parents = torch.zeros(b, n, dtype=torch.int32, device="cuda")
    tokens = q.argmax(-1, keepdim=True).to(torch.int32).repeat(1, n)
    uniforms = torch.rand(b, n, generator=g, device="cuda")
    uniforms[:, 1:] = 1 - 2.0 ** -24
    # (the last child of every fourth sequence is a token of the other half with little of the draft)
    other = (~half).float().argmax(-1)
    tokens[row[::4], counts[::4].long() - 1] = other[::4].to(torch.int32)
    q[row[::4], other[::4]] = 1e-12
    logits, draft = (torch.zeros(b, n, v, device="cuda") for _ in range(2))
    logits[:] = line[:, None]
    draft[:] = q[:, None]
    path = check(logits, tokens, uniforms, parents, draft, torch.full((b,), heat, device="cuda"), counts)
    assert [p[1] for p in path] == [int(counts[i]) - 1 if i % 4 == 0 else -1 for i in range(b)]


@pytest.mark.parametrize("some", [2, 3, 4])
def test_proposed_tokens_that_are_all_there_is(some):
    """Logits masked to a few tokens, all of them proposed, and uniforms that reject one after another: the last one is all that is left,
    and accepted.  Whatever happens, the next token is written."""
    b, v, n = 400, 37, some + 2
    g = R.gen(120 + some)
    place = torch.rand(b, v, generator=g, device="cuda").argsort(-1)[:, :some]
    logits = torch.full((b, n, v), -float("inf"), device="cuda")
    size = torch.cumsum(0.5 + 6 * torch.rand(b, some, generator=g, device="cuda"), -1).neg()
    logits.scatter_(2, place[:, None].expand(b, n, some), size[:, None].expand(b, n, some))
    tokens = torch.zeros(b, n, dtype=torch.int32, device="cuda")
    tokens[:, 1:some + 1] = place
    tokens[:, some + 1] = place[:, 0]
    parents = torch.zeros(b, n, dtype=torch.int32, device="cuda")
    uniforms = 1 - 2.0 ** -24 * torch.randint(1, 5, (b, n), generator=g, device="cuda")
    uniforms[:, 0] = torch.rand(b, generator=g, device="cuda")
    uniforms = uniforms.float()
    status = ops.new_status()
    drawn = torch.full((b,), -5, dtype=torch.int32, device="cuda")
    accepted, _ = ops.verify_nodes(logits, tokens, uniforms, parents=parents, next_tokens=drawn, status=status)
    ops.check_status(status)
    path, nxt = M.verify(logits, tokens, uniforms, parents)
    assert accepted.tolist() == path and drawn.tolist() == nxt
    assert sum(p[1] == some for p in path) > b // 4      # (rejections up to the last)


def test_two_tokens_of_which_one_is_left():
    """Two tokens, the likely one rejected: the other one's probability is 1."""
    logits = torch.tensor([0.0, -5.0625], device="cuda").expand(1, 3, 2).contiguous()
    tokens = torch.tensor([[0, 0, 1]], dtype=torch.int32, device="cuda")
    parents = torch.zeros(1, 3, dtype=torch.int32, device="cuda")
    uniforms = torch.tensor([[0.3, 0.9995, 0.999997]], device="cuda")
    assert check(logits, tokens, uniforms, parents) == [[0, 2, -1]]


@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("half,v", [(False, 151936), (True, 151936), (False, 900)])
def test_verdicts_at_their_border(half, v, probs):
    """Uniforms next to p / q on either side, 2^-26 of it away at least (probabilities are right to 2^-32), of a first child and of a
    sibling behind a rejection."""
    b, n = 64, 3
    g = R.gen(130)
    logits, tokens, uniforms, parents, draft = M.tree_inputs(g, b, n, v, True, True, sharp=8.0, half=half)
    parents[:, 1:] = 0
    heat = 0.6 + torch.rand(b, generator=g, device="cuda")
    heat[::4] = 1.0
    p = torch.softmax(logits[:, 0].double() / heat.double()[:, None], -1)
    likely = p.topk(3, -1).indices
    row = torch.arange(b, device="cuda")
    tokens[:, 1], tokens[:, 2] = likely[:, 1], likely[:, 2]
    # (probabilities of the draft that leave the border inside (0, 1))
    at = p[row, likely[:, 1]] * (1 + 2 * torch.rand(b, generator=g, device="cuda"))
    draft[row, 0, likely[:, 1]] = at.clamp(max=1).float()
    # (... and some of the target's left at the sibling)
    draft[row, 0, likely[:, 2]] = (p[row, likely[:, 2]] * (0.1 + 0.7 * torch.rand(b, generator=g, device="cuda"))).float()
    q = draft[:, 0].double() if probs else torch.nn.functional.one_hot(likely[:, 1], v).double()

    def beside(border, below):
        u = (border * (1 - 2.0 ** -26 if below else 1 + 2.0 ** -26)).float()
        off = torch.nextafter(u, torch.full_like(u, 0.0 if below else 1.0))
        right = u.double() <= border * (1 - 2.0 ** -26) if below else u.double() >= border * (1 + 2.0 ** -26)
        return torch.where(right, u, off).clamp(max=1 - 2.0 ** -24)

    first = p[row, likely[:, 1]] / q[row, likely[:, 1]]
    rest = (p - q).clamp(min=0)
    rest = rest / rest.sum(-1, keepdim=True)
    second = rest[row, likely[:, 2]] / (draft[row, 0, likely[:, 2]].double() if probs else 1.0)
    for below in (True, False):
        uniforms[:, 1] = beside(first, below)
        path = check(logits, tokens, uniforms, parents, draft if probs else None, heat)
        assert (sum(x[1] == 1 for x in path) > b // 2) == below
        uniforms[:, 1] = 1 - 2.0 ** -24            # (rejected, where it can be)
        uniforms[:, 2] = beside(second, below)
        check(logits, tokens, uniforms, parents, draft if probs else None, heat)
