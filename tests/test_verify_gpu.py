"""Verification of drafts against the definition in fp64.

Results are whole numbers and must be equal.  Both sides take the same fp32 (or
bf16) values; the kernel's sums are in units of 2^-43, an error of 2^-44 for each
of V entries, so a test or draw within V 2^-43 of its border could go either way:
`ref.verify` gives the nearest one, which the seeds keep beyond that."""
import pytest

torch = pytest.importorskip("torch")

import io_aware_exact_06_gb300 as fa
from tests import sample_ref as ref
from tests.test_cache_gpu import cu_of
from tests.test_tree_gpu import signed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import __graft_entry__
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    __graft_entry__.build()
    return torch.device("cuda:0")


def trees(seed, ns, wide):
    """Mask words: each token's parent is one of the `wide` before it; now and then none."""
    import random
    rng, words = random.Random(seed), []
    for n in ns:
        mine = []
        for i in range(n):
            up = mine[rng.randrange(max(0, i - wide), i)] if i and rng.random() > 0.05 else 0
            mine.append(up | 1 << i)
        words += mine
    return torch.tensor([signed(w) for w in words], dtype=torch.int64)


def parents(mask, cu):
    out = []
    for b in range(len(cu) - 1):
        for i in range(cu[b + 1] - cu[b]):
            seen = [j for j in range(i) if (j == i - 1 if mask is None else int(mask[cu[b] + i]) >> j & 1)]
            out.append(cu[b] + (seen[-1] if seen else 0))
    return torch.tensor(out)


def make(seed, ns, V, kind, draft, tree, std=2.5, off=1.0):
    g = torch.Generator().manual_seed(seed)
    cu = [sum(ns[:i]) for i in range(len(ns) + 1)]
    total = cu[-1]
    t = torch.randn(total, V, generator=g) * std
    q = (t + off * torch.randn(total, V, generator=g)).softmax(-1).to(kind)
    p = t.softmax(-1).to(kind)
    mask = trees(seed, ns, 4) if tree else None
    up = parents(mask, cu)
    tokens = torch.multinomial(q[up].float(), 1, generator=g)[:, 0].to(torch.int32) if total else torch.zeros(0, dtype=torch.int32)
    return dict(tokens=tokens, probs=p, cu=cu, u=torch.rand(total, generator=g), u_next=torch.rand(len(ns), generator=g),
                draft=q if draft else None, mask=mask)


def call(dev, s, seqlens=None, **over):
    to = lambda x: None if x is None else x.to(dev)
    a = {n: to(s[n]) if n != "cu" else torch.tensor(s["cu"], dtype=torch.int32, device=dev) for n in s}
    a.update(over)
    return fa.verify_drafts(a["tokens"], a["probs"], a["cu"], a["u"], a["u_next"], draft_probs=a["draft"], mask=a["mask"],
                            seqlens=seqlens)


def check(dev, s, got=None):
    got = got or call(dev, s)
    assert fa.attn_last_device_error() == 0
    path, kept, nxt, near = ref.verify(s["tokens"], s["probs"], s["cu"], s["u"], s["u_next"], s["draft"], s["mask"])
    assert near > s["probs"].shape[1] * 2.0 ** -43, "a case next to a border says nothing"
    assert got[1].tolist() == kept and got[0].tolist()[:s["cu"][-1]] == path and got[2].tolist() == nxt
    return path, kept, nxt


CASES = [  # new tokens, V, type, draft's probabilities, tree
    ([1], 1, torch.float32, False, False),
    ([2, 3], 1, torch.float32, True, False),
    ([1, 1, 1], 2, torch.bfloat16, True, False),
    ([5, 0, 3, 1], 31, torch.float32, True, False),
    ([5, 0, 3, 1], 1000, torch.bfloat16, False, True),
    ([16, 9, 12], 1025, torch.float32, True, True),
    ([64, 64, 2], 4096, torch.float32, True, True),
    ([64, 64, 2], 4096, torch.bfloat16, False, True),
    ([9] * 5, 50021, torch.bfloat16, True, True),
    ([9] * 5, 50021, torch.float32, False, True),
    ([4] * 3, 131072, torch.float32, True, False),
    ([3] * 2, 262144, torch.bfloat16, True, True),
    ([6] * 100, 8192 + 4, torch.float32, True, True),
    ([3] * 300, 16384, torch.bfloat16, True, True),
    ([2] * 700, 999, torch.float32, False, False),
]


@pytest.mark.parametrize("ns,V,kind,draft,tree", CASES)
def test_against_the_definition(dev, ns, V, kind, draft, tree):
    for off in (0.5, 2.0):  # drafts that are often right, and seldom
        check(dev, make(500 + len(ns) + V % 97, ns, V, kind, draft, tree, off=off))


@pytest.mark.parametrize("draft", [False, True])
def test_many_rejections_at_a_node(dev, draft):
    """63 children of the first token, some the same token, none likely to be taken."""
    g = torch.Generator().manual_seed(9)
    V, n = 3000, 64
    q = torch.rand(1, V, generator=g).repeat(n, 1)
    q = (q / q.sum(-1, keepdim=True))
    p = torch.rand(n, V, generator=g) ** 4
    p = p / p.sum(-1, keepdim=True)
    low = p[0].argsort()[:40].to(torch.int32)
    s = dict(tokens=torch.cat([low[:1], low, low[:23]]), probs=p, cu=[0, n], u=torch.full((n,), 0.9), u_next=torch.rand(1, generator=g),
             draft=q if draft else None, mask=torch.tensor([1] + [signed(1 | 1 << i) for i in range(1, n)]))
    _, kept, _ = check(dev, s)
    assert kept == [1]


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_rows_any_distance_apart(dev, kind):
    """Odd strides and starts that are no multiple of 16 bytes."""
    s = make(520, [5, 4], 1003, kind, True, True)
    for pad, start in ((0, 0), (5, 0), (8, 3), (13, 1)):
        wide = torch.full((2, 9, 1003 + pad + start), 9.0, dtype=kind, device=dev)
        views = [wide[k, :, start:start + 1003] for k in range(2)]
        views[0].copy_(s["probs"])
        views[1].copy_(s["draft"])
        check(dev, s, call(dev, s, probs=views[0], draft=views[1]))


@pytest.mark.parametrize("draft", [False, True])
def test_random_numbers_at_their_ends(dev, draft):
    s = make(530, [4, 4, 4], 500, torch.float32, draft, True)
    for u in (0.0, 1.0 - 2.0 ** -24, 1.0, float("nan"), -1.0, 7.0):
        got = call(dev, s, u_next=torch.full((3,), u, device=dev))
        kept, nxt = got[1].tolist(), got[2].tolist()
        assert all(0 <= x < 500 for x in nxt)
        _, want, _, _ = ref.verify(s["tokens"], s["probs"], s["cu"], s["u"], [0.5] * 3, s["draft"], s["mask"])
        assert kept == want  # the draw at the end does not touch the walk
    s["u"] = torch.zeros(12)
    assert call(dev, s)[1].tolist() == check(dev, s)[1]
    assert fa.attn_last_device_error() == 0


def test_equal_and_disjoint_distributions(dev):
    g = torch.Generator().manual_seed(3)
    p = torch.rand(4, 400, generator=g).softmax(-1)
    s = dict(tokens=torch.tensor([0, 5, 6, 7], dtype=torch.int32), probs=p, cu=[0, 4], u=torch.full((4,), 0.999999),
             u_next=torch.tensor([0.3]), draft=p.clone(), mask=None)
    assert call(dev, s)[1].tolist() == [4]  # the same: every draft is accepted
    p = p.clone()
    q = p.clone()
    p[:, :200], q[:, 200:] = 0, 0
    s = dict(s, probs=p, draft=q, u=torch.full((4,), 0.5))
    _, kept, nxt = check(dev, s)  # nothing in common: the first is rejected
    assert kept == [1] and nxt[0] >= 200
    # the draft has all that the target has, and more: nothing is left, and the target's row is drawn from
    q = (p * 2).clamp_max(1.0)
    s = dict(s, probs=p, draft=q, tokens=torch.tensor([0, 300, 301, 302], dtype=torch.int32), u=torch.full((4,), 0.9))
    got = call(dev, s)
    c = p[0].double().cumsum(0)
    assert got[1].tolist() == [1] and got[2].tolist() == [int((c > float(s["u_next"][0]) * c[-1]).nonzero()[0])]


def test_entries_that_are_no_probabilities(dev):
    """NaN counts as 0, and so does what is below it; what is above 1 counts as 1; a row of zeros draws nothing."""
    p = torch.zeros(3, 64)
    p[0, 3], p[0, 10], p[0, 20] = float("nan"), -5.0, 0.25
    p[1] = float("nan")
    p[2, 7], p[2, 9] = float("inf"), 0.5
    s = dict(tokens=torch.zeros(3, dtype=torch.int32), probs=p, cu=[0, 1, 2, 3], u=torch.zeros(3), u_next=torch.tensor([0.5, 0.5, 0.9]),
             draft=None, mask=None)
    got = call(dev, s)
    assert fa.attn_last_device_error() == 0
    assert got[2].tolist() == [20, -1, 9] and got[1].tolist() == [1, 1, 1]


def test_the_next_token_is_distributed_as_the_target(dev):
    """One draft for each of 40000 sequences: what comes out first (the draft or the token behind a
    rejection) has the target's frequencies, within six standard deviations of a count."""
    B, V = 40000, 8
    g = torch.Generator().manual_seed(12)
    p, q = torch.rand(V, generator=g), torch.rand(V, generator=g)
    p, q = p / p.sum(), q / q.sum()
    draft = torch.multinomial(q, B, replacement=True, generator=g).to(torch.int32)
    tokens = torch.stack([torch.zeros_like(draft), draft], 1).flatten().to(dev)
    rows = lambda x: x.repeat(2 * B, 1).to(dev)
    for dp in (rows(q), None):
        if dp is None:  # certain drafts: any fixed token may be offered
            tokens[1::2] = 5
        path, kept, nxt, lens = fa.verify_drafts(tokens, rows(p), cu_of(dev, [2] * 100).new_tensor(range(0, 2 * B + 1, 2)),
                                                 torch.rand(2 * B, generator=g).to(dev), torch.rand(B, generator=g).to(dev),
                                                 draft_probs=dp)
        assert lens is None
        first = torch.where(kept == 2, tokens[1::2], nxt).cpu().long()
        count = torch.bincount(first, minlength=V).double()
        want = p.double() * B
        assert ((count - want).abs() <= 6 * (want * (1 - p.double())).sqrt()).all()
    assert fa.attn_last_device_error() == 0


def test_lengths_and_padding(dev):
    s = make(540, [4, 0, 3], 300, torch.float32, True, True)
    wide = {n: torch.cat([s[n], s[n][:2]]) if n in ("tokens", "probs", "u", "draft", "mask") else s[n] for n in s}
    got = call(dev, wide, seqlens=torch.tensor([50, 20, 3], dtype=torch.int32, device=dev))
    _, kept, _ = check(dev, s, got)
    assert got[3].tolist() == [50 - 4 + kept[0], 20, kept[2]]


@pytest.mark.parametrize("what", ["token", "negative token", "long", "short", "total", "first", "falls"])
@pytest.mark.parametrize("V", [300, 40000])
def test_bad_batches_are_reported(dev, what, V):
    s = make(550, [4, 5, 3], V, torch.float32, True, False, off=0.2)
    lens = torch.tensor([50, 20, 30], dtype=torch.int32, device=dev)
    cu = torch.tensor(s["cu"], dtype=torch.int32, device=dev)
    tokens, status, refused = s["tokens"].clone(), -8, [1]
    good = call(dev, s, seqlens=lens)
    over = {}
    if what.endswith("token"):
        tokens[5], status, refused = V if what == "token" else -1, -11, []
    elif what == "long":
        s = make(551, [4, 65, 3], V, torch.float32, False, False)
        cu, tokens = torch.tensor(s["cu"], dtype=torch.int32, device=dev), s["tokens"]
        good = None
    elif what == "short":
        lens[1] = 4
    elif what == "total":
        cu[3], refused = 13, [2]
    elif what == "first":
        cu[0], refused = 1, [0]
    else:
        cu[1], refused = 10, [0, 1, 2]
    got = call(dev, s, seqlens=lens, cu=cu, tokens=tokens.to(dev), **over)
    assert fa.attn_last_device_error() == status
    for b in range(3):
        if b in refused:
            assert got[1][b] == 0 and got[2][b] == -1 and got[3][b] == lens[b]
        elif good is not None and not (what.endswith("token") and b == 1):
            assert got[1][b] == good[1][b] and got[2][b] == good[2][b]
    if what.endswith("token"):  # rejected: the token behind it is drawn from the target's rest
        assert got[1][1] == 1 and got[0][4:9].tolist() == [0, -1, -1, -1, -1]
    assert fa.attn_last_device_error() == 0


def test_rows_behind_the_batch_stay(dev):
    """The C call, on the caller's buffers: what belongs to no sequence is left as it was."""
    s = make(560, [4, 3], 300, torch.float32, True, False)
    tokens, probs, u = (torch.cat([s[n], s[n][:3]]).to(dev) for n in ("tokens", "probs", "u"))
    path, kept, nxt = torch.full((10,), 99, dtype=torch.int32, device=dev), *torch.full((2, 3), 99, dtype=torch.int32, device=dev)
    cu, un = torch.tensor([0, 4, 7], dtype=torch.int32, device=dev), s["u_next"].to(dev)
    fa.attn_verify_drafts(tokens, probs, 300, None, 0, False, cu, None, u, un, None, path, kept, nxt, None, 2, 10, 300,
                          torch.cuda.current_stream())
    assert fa.attn_last_device_error() == 0
    assert (path[7:] == 99).all() and kept[2] == 99 and nxt[2] == 99 and (path[:7] != 99).all()


def test_lengths_in_place(dev):
    s = make(570, [5, 4], 900, torch.bfloat16, True, True)
    lens = torch.tensor([80, 70], dtype=torch.int32, device=dev)
    want = call(dev, s, seqlens=lens.clone())
    path, (kept, nxt) = torch.empty(9, dtype=torch.int32, device=dev), torch.empty((2, 2), dtype=torch.int32, device=dev)
    a = {n: s[n].to(dev) for n in ("tokens", "probs", "draft", "mask", "u", "u_next")}
    fa.attn_verify_drafts(a["tokens"], a["probs"], 900, a["draft"], 900, True, torch.tensor(s["cu"], dtype=torch.int32, device=dev),
                          a["mask"], a["u"], a["u_next"], lens, path, kept, nxt, lens, 2, 9, 900, torch.cuda.current_stream())
    assert fa.attn_last_device_error() == 0
    assert torch.equal(lens, want[3]) and torch.equal(path, want[0]) and torch.equal(nxt, want[2])


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [300, 40000])
def test_entries_next_to_the_unit_of_sums(dev, kind, V):
    """An entry counts as the nearest multiple of 2^-43, one of 2^-44 as 0: in the draw, where a row draws
    nothing, and where a residual has nothing left and the target's row is drawn from."""
    above = 2.0 ** -44 * (1 + 2 * torch.finfo(kind).eps)
    p = torch.zeros(9, V, dtype=torch.float64)
    q = torch.zeros(9, V, dtype=torch.float64)
    p[0] = 2.0 ** -44                       # nothing to draw
    p[1, 5:], p[1, 250], p[1, 290] = 2.0 ** -44, above, above  # two entries, a unit each
    p[2, 7], p[2, 200], p[2, 299] = 0.75 * 2.0 ** -43, 1.25 * 2.0 ** -43, 1.75 * 2.0 ** -43  # 1, 1 and 2 units
    for b, left in ((3, 2.0 ** -44), (5, above), (7, 2.0 ** -42)):  # a rejected draft: what the target has beside it
        p[b, 3], p[b, 260], q[b, 3] = 0.25, left, 0.5
    s = dict(tokens=torch.full((9,), 3, dtype=torch.int32), probs=p.to(kind), cu=[0, 1, 2, 3, 5, 7, 9], u=torch.full((9,), 0.9),
             u_next=torch.zeros(6), draft=q.to(kind), mask=None)
    want = {0.0: [-1, 250, 7, 3, 260, 260],
            0.5: [-1, 290, 299, 3, 260, 260],    # the first behind half of the units
            0.26: [-1, 250, 200, 3, 260, 260]}
    for u, tokens in want.items():
        got = call(dev, dict(s, u_next=torch.full((6,), u)))
        assert got[2].tolist() == tokens and got[1].tolist() == [1] * 6
    assert fa.attn_last_device_error() == 0
