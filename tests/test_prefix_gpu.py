"""Attention of new tokens over shared prefixes against fp64: every sequence over
its own page table.  The kernels and their roundings are those of attention over
one sequence's pages, and so are the tolerances (tests/test_tree_gpu.py counts
them); the join of pieces is fp32, inside the 2^-17 A counted for sums there."""
import math
import random

import pytest

torch = pytest.importorskip("torch")

import io_aware_exact_06_gb300 as fa
from tests import serve_ref as ref
from tests.test_cache_gpu import cu_of, normal
from tests.test_tree_gpu import check, fill, random_masks, rows_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import __graft_entry__
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    __graft_entry__.build()
    return torch.device("cuda:0")


def ints(dev, values):
    return torch.tensor(values, dtype=torch.int32, device=dev)


def share(c, groups, prefix):
    """The tables of a group's sequences name the first one's pages for the whole pages of the prefix."""
    for g, p in enumerate(prefix):
        n = p // c["page"]
        if groups[g + 1] > groups[g]:
            c["page_table"][groups[g]:groups[g + 1], :n] = c["page_table"][groups[g], :n].clone()
    return c


def call(dev, c, q, lens, ns, mask, groups, prefix, **kw):
    cu = [sum(ns[:i]) for i in range(len(ns) + 1)]
    kw.setdefault("max_new", max(ns))
    kw.setdefault("max_len", max(lens))
    kw.setdefault("max_group", max([cu[groups[g + 1]] - cu[groups[g]] for g in range(len(prefix))] + [0]))
    kw.setdefault("max_prefix", max(prefix + [0]))
    return fa.prefix_decode(q, c["k_cache"], c["v_cache"], c["page_table"], ints(dev, lens), cu_of(dev, ns),
                            cu_groups=ints(dev, groups), prefix_lens=ints(dev, prefix),
                            mask=None if mask is None else mask.to(dev), k_scale=c["k_scale"], v_scale=c["v_scale"], **kw)


CASES = [  # lengths, new tokens, groups' offsets, prefixes, Hq, H, d, page, codes, tree, splits
    ([50, 60], [1, 1], [0, 2], [48], 1, 1, 64, 16, False, False, 0),
    ([300, 320, 301, 300], [1, 1, 1, 1], [0, 4], [299], 8, 2, 128, 16, False, False, 0),
    ([300, 320, 301, 300], [1, 1, 1, 1], [0, 4], [299], 16, 4, 128, 64, True, False, 3),
    ([40, 700, 720, 40, 520, 530], [1, 1, 1, 1, 1, 1], [1, 3, 3, 4, 6], [650, 9, 0, 512], 12, 4, 64, 32, True, False, 0),
    ([40, 700, 720, 40, 520, 530], [2, 3, 0, 1, 4, 1], [0, 0, 1, 3, 6], [0, 33, 640, 15], 6, 2, 128, 32, False, True, 2),
    ([1100, 1090, 1030], [5, 31, 3], [0, 3], [1027], 8, 1, 128, 16, False, True, 0),
    ([1100, 1090, 1030], [5, 31, 3], [0, 3], [1027], 8, 1, 128, 16, True, True, 5),
    ([900] * 9, [33] * 9, [0, 9], [777], 4, 2, 64, 256, False, True, 0),
    ([900] * 9, [33] * 9, [0, 9], [777], 4, 2, 128, 128, True, True, 1),
    ([900] * 9, [33] * 9, [0, 9], [777], 2, 1, 128, 64, False, True, 0),
    ([600 + b for b in range(70)], [1] * 70, [0, 35, 70], [599, 500], 4, 1, 128, 16, False, False, 0),
    ([600 + b for b in range(70)], [1] * 70, [0, 35, 70], [599, 500], 4, 1, 64, 16, True, False, 0),
    ([130] * 40, [2] * 40, [0, 40], [128], 2, 2, 64, 16, False, True, 1),
    ([2000, 2001], [64, 64], [0, 2], [1900], 5, 1, 128, 16, False, True, 256),
    ([16 * 9] * 200, [1] * 200, list(range(0, 201, 2)), [16 * (g % 9) for g in range(100)], 3, 1, 128, 16, True, False, 0),
]


@pytest.mark.parametrize("lens,ns,groups,prefix,Hq,H,d,page,codes,tree,splits", CASES)
def test_against_fp64(dev, lens, ns, groups, prefix, Hq, H, d, page, codes, tree, splits):
    seed = 300 + len(lens) * 7 + Hq + d
    c = share(fill(dev, seed, lens, H, d, page, codes), groups, prefix)
    total = sum(ns)
    q = normal(dev, seed + 2, total, Hq + 2, d, std=1.5)[:, :Hq]  # a token stride
    mask = random_masks(seed, ns) if tree else None
    got = call(dev, c, q, lens, ns, mask, groups, prefix, num_splits=splits)
    assert fa.attn_last_device_error() == 0
    check(c, q, lens, ns, mask, got)
    again = call(dev, c, q, lens, ns, mask, groups, prefix, num_splits=splits)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("B", [2, 40, 90])  # few rows of a group, one tile, several
def test_peaky_and_flat_scores(dev, codes, B):
    lens, ns, groups, prefix = [400 + b % 5 for b in range(B)], [1] * B, [0, B], [390]
    for std in (0.0, 6.0):
        c = share(fill(dev, 310, lens, 1, 128, 16, codes, std=max(std, 1.0)), groups, prefix)
        q = normal(dev, 311, B, 4, 128, std=std)
        check(c, q, lens, ns, None, call(dev, c, q, lens, ns, None, groups, prefix))
        check(c, q, lens, ns, None, call(dev, c, q, lens, ns, None, groups, prefix, scale=0.0), scale=0.0)
    assert fa.attn_last_device_error() == 0


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("B", [3, 60])
def test_value_scales_of_all_sizes(dev, codes, B):
    """A prefix whose values differ by many powers of two, from token to token."""
    from tests.test_cache_gpu import make, put
    lens, ns, groups, prefix = [310] * B, [1] * B, [0, B], [304]
    c = make(dev, 320, lens, 1, 128, 16, codes)
    kv = normal(dev, 321, sum(lens), 2, 128)
    kv[:, 1] *= torch.exp2(torch.arange(sum(lens), device=dev) % 41 - 20.0)[:, None].to(torch.bfloat16)
    put(dev, c, kv[:, :1], kv[:, 1:], lens, lens)
    share(c, groups, prefix)
    q = normal(dev, 322, B, 4, 128)
    check(c, q, lens, ns, None, call(dev, c, q, lens, ns, None, groups, prefix))
    assert fa.attn_last_device_error() == 0


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("G", [1, 8])
def test_what_rows_do_not_see_does_not_matter(dev, codes, G):
    """Drafts hidden from others hold NaN; rows behind a sequence, and pages behind a prefix's last
    whole one in the first sequence's table, are other sequences' business."""
    lens, ns, groups, prefix, d = [200 + b for b in range(20)], [6] * 20, [0, 20], [150], 128
    c = share(fill(dev, 330, lens, 1, d, 16, codes), groups, prefix)
    table = c["page_table"].cpu()
    for b in range(20):
        row = int(ref.row_index(table, 16, b, torch.tensor(lens[b] - 6 + 2)))
        if codes:
            c["v_cache"].view(torch.uint8)[row // 16, row % 16] = 0x7f
        else:
            c["v_cache"][row // 16, row % 16] = float("nan")
    mask = torch.tensor([1 | 1 << i for _ in ns for i in range(6)], dtype=torch.int64)
    q = normal(dev, 331, 120, G, d)
    got = call(dev, c, q, lens, ns, mask, groups, prefix)
    assert fa.attn_last_device_error() == 0
    o, lse = (x.view(20, 6, *x.shape[1:]) for x in got)
    assert o[:, 2].isnan().all() and o[:, [0, 1, 3, 4, 5]].isfinite().all() and lse.isfinite().all()
    k, v = rows_of(c)
    wo, wl, A, S = ref.tree(q.cpu(), k, v, table, 16, lens, [6 * b for b in range(21)], mask, d ** -0.5)
    keep = [0, 1, 3, 4, 5]
    off = (o.cpu().double() - wo.view_as(o)).abs()[:, keep]
    # bf16 of O and of the probabilities, as in test_tree_gpu; scores below 20 in magnitude
    assert (off <= (2.0 ** -7 * A.view_as(o) + 2.0 ** -12)[:, keep]).all()


@pytest.mark.parametrize("codes", [False, True])
def test_rows_that_see_the_prefix_alone_or_nothing(dev, codes):
    lens, ns, groups, prefix = [70, 75, 12], [6, 6, 12], [0, 2, 3], [64, 0]
    c = share(fill(dev, 340, lens, 2, 64, 16, codes), groups, prefix)
    # lengths end right behind the prefix: a token without bits sees the prefix alone
    q = normal(dev, 341, 24, 4, 64)
    mask = torch.tensor([0, 3] * 6 + [0, 2] * 6, dtype=torch.int64)
    got = call(dev, c, q, lens, ns, mask, groups, prefix)
    assert fa.attn_last_device_error() == 0
    check(c, q, lens, ns, mask, got)
    assert (got[0][12::2] == 0).all() and (got[1][12::2] == -math.inf).all()


def test_without_groups_it_is_tree_decode(dev):
    lens, ns = [333, 40, 512], [1, 3, 2]
    for codes in (False, True):
        c = fill(dev, 350, lens, 2, 128, 16, codes)
        q = normal(dev, 351, 6, 8, 128)
        want = fa.tree_decode(q, c["k_cache"], c["v_cache"], c["page_table"], ints(dev, lens), cu_of(dev, ns), 3, 512,
                              k_scale=c["k_scale"], v_scale=c["v_scale"])
        for groups, prefix in (([0], []), ([0, 1, 3], [0, 15])):
            got = call(dev, c, q, lens, ns, None, groups, prefix)
            # keys are cut into other pieces: each is within its own rounding of fp64 (check), so the two
            # differ by twice that at most, and not bit for bit
            check(c, q, lens, ns, None, got)
            check(c, q, lens, ns, None, want)
    assert fa.attn_last_device_error() == 0


def test_padded_batch_and_bounds(dev):
    lens, ns, groups, prefix = [90, 95, 33, 0], [3, 2, 1, 0], [0, 2], [80]
    c = share(fill(dev, 360, lens, 2, 128, 32, True), groups, prefix)
    q = normal(dev, 361, 12, 4, 128)
    for bounds in (dict(), dict(max_new=64, max_len=5000, max_group=12, max_prefix=4000), dict(max_group=1 << 30)):
        out = torch.full((12, 4, 128), 7.0, dtype=torch.bfloat16, device=dev)
        lse = torch.full((12, 4), 7.0, device=dev)
        call(dev, c, q, lens, ns, None, groups, prefix, out=out, lse=lse, **bounds)
        assert fa.attn_last_device_error() == 0
        check(c, q, lens, ns, None, (out, lse))
        assert (out[6:] == 7).all() and (lse[6:] == 7).all()


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("G", [2, 40])
def test_finished_sequences_in_a_group(dev, codes, G):
    """Places of a batch that hold nothing, a group's first among them: no length, no pages, no new tokens."""
    lens, ns, groups, prefix = [300, 300, 300, 310, 300, 90], [0, 1, 0, 2, 0, 1], [0, 5, 6], [299, 64]
    c = share(fill(dev, 335, lens, 1, 128, 16, codes), groups, prefix)
    for b in (0, 2, 4):
        lens[b] = 0
        c["page_table"][b] = -1
    q = normal(dev, 336, sum(ns), G, 128)
    check(c, q, lens, ns, None, call(dev, c, q, lens, ns, None, groups, prefix))
    assert fa.attn_last_device_error() == 0


def test_groups_without_new_tokens_have_any_prefix(dev):
    """An empty group, and one whose sequences have all finished: behind the table, below 0."""
    lens, ns, groups, prefix = [300, 0, 0, 310], [1, 0, 0, 2], [0, 1, 1, 3, 4], [299, 5000, -7, 304]
    c = share(fill(dev, 337, [300, 300, 300, 310], 2, 64, 16, False), groups, [299, 0, 0, 304])
    q = normal(dev, 338, sum(ns), 6, 64)
    check(c, q, lens, ns, None, call(dev, c, q, lens, ns, None, groups, prefix, max_prefix=304))
    assert fa.attn_last_device_error() == 0


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("B", [4, 100])
def test_a_nan_in_a_prefix_stays_in_its_group(dev, codes, B):
    lens, ns, groups, prefix = [300] * B, [1] * B, [0, B // 2, B], [256, 128]
    c = share(fill(dev, 370, lens, 1, 128, 16, codes), groups, prefix)
    page = int(c["page_table"][0, 3])
    if codes:
        c["k_scale"][page, :, 5] = float("nan")
    else:
        c["k_cache"][page, 5, :, 7] = float("nan")
    q = normal(dev, 371, B, 4, 128)
    o, lse = call(dev, c, q, lens, ns, None, groups, prefix)
    assert fa.attn_last_device_error() == 0
    assert o[:B // 2].isnan().all() and lse[:B // 2].isnan().all()
    assert o[B // 2:].isfinite().all() and lse[B // 2:].isfinite().all()


def test_offsets_past_32_bits(dev):
    pages = 17000
    for codes in (True, False):
        lens, ns, groups, prefix, H, d, page = [600, 610], [40, 3], [0, 2], [512], 8, 128, 256
        c = fill(dev, 380, lens, H, d, page, codes)
        big = {**c}
        for n in "kv":
            for x in ("_cache", "_scale"):
                if c[n + x] is None:
                    continue
                t = c[n + x].view(torch.uint8) if codes and x == "_cache" else c[n + x]
                wide = torch.empty((pages + t.shape[0], *t.shape[1:]), dtype=t.dtype, device=dev)
                wide[pages:] = t
                big[n + x] = wide.view(c[n + x].dtype)
        big["page_table"] = c["page_table"] + pages
        share(c, groups, prefix), share(big, groups, prefix)
        q = normal(dev, 381, 43, 16, d)
        want, got = (call(dev, x, q, lens, ns, None, groups, prefix) for x in (c, big))
        assert fa.attn_last_device_error() == 0
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        del big, got
        torch.cuda.empty_cache()


BAD = ["falling groups", "group below", "group beyond", "long prefix", "negative prefix", "large group", "prefix in drafts",
       "prefix page", "short sequence", "falling offsets", "first offset"]


@pytest.mark.parametrize("what", BAD)
@pytest.mark.parametrize("G", [2, 40])
def test_bad_plans_are_reported(dev, what, G):
    """Sequences that are not concerned are right; the others are not written, or NaN where a page is wrong."""
    lens, ns, groups, prefix, d = [120, 130, 200, 210, 50], [2, 1, 3, 1, 1], [0, 2, 4], [96, 160], 64
    c = share(fill(dev, 390, lens, 1, d, 16, True), groups, prefix)
    q = normal(dev, 391, 8, G, d)
    good = call(dev, c, q, lens, ns, None, groups, prefix)
    lens_d, cu, cg, pl, table = ints(dev, lens), cu_of(dev, ns), ints(dev, groups), ints(dev, prefix), c["page_table"].clone()
    bounds = dict(max_new=3, max_len=210, max_group=4, max_prefix=160)
    status, ruined = -8, [3, 4, 5, 6]  # the second group's rows
    if what == "falling groups":
        cg[1], ruined = 5, list(range(8))
    elif what == "group below":
        cg[0], ruined = -1, [0, 1, 2]
    elif what == "group beyond":
        cg[2], ruined = 6, [3, 4, 5, 6, 7]
    elif what == "long prefix":
        bounds["max_prefix"] = 159
    elif what == "negative prefix":
        pl[1] = -1
    elif what == "large group":
        bounds["max_group"] = 3
    elif what == "prefix in drafts":
        pl[0], ruined = 128, [0, 1, 2]  # beyond the first sequence's 118, and the second's only new token
    elif what == "prefix page":
        table[2, 4], status = 1 << 28, -11
    elif what == "short sequence":
        lens_d[3], ruined = 150, [6]
    elif what == "falling offsets":
        cu[2], ruined = 7, list(range(8))
    else:
        cu[0], ruined = 1, [0, 1]
    out = torch.full((8, G, d), 7.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((8, G), 7.0, device=dev)
    if what == "prefix in drafts":
        lens_d[1] = 128
    fa.prefix_decode(q, c["k_cache"], c["v_cache"], table, lens_d, cu, cu_groups=cg, prefix_lens=pl, k_scale=c["k_scale"],
                     v_scale=c["v_scale"], out=out, lse=lse, **bounds)
    assert fa.attn_last_device_error() == status
    if status == -11:
        assert out[ruined].isnan().all() and lse[ruined].isnan().all()
    else:
        assert (out[ruined] == 7).all() and (lse[ruined] == 7).all()
    others = [t for t in range(8) if t not in ruined]
    assert ((out[others].float() - good[0][others].float()).abs() <= 2.0 ** -7).all()
    assert ((lse[others] - good[1][others]).abs() <= 2.0 ** -14).all()
    assert fa.attn_last_device_error() == 0


@pytest.mark.parametrize("codes", [False, True])
def test_more_groups_and_sequences_than_threads_plan(dev, codes):
    """700 sequences in groups of two, with empty groups between them and sequences in none."""
    B, d, page = 700, 64, 16
    lens = [40 + (7 * b) % 33 for b in range(B)]
    ns = [b % 3 for b in range(B)]
    groups, prefix = [5], []
    for g in range(340):
        prefix += [16 * (g % 3) + g % 2, 31]
        groups += [min(5 + 2 * (g + 1), B - 3)] * 2  # the second one is empty
    c = share(fill(dev, 400, lens, 1, d, page, codes), groups, prefix)
    q = normal(dev, 401, sum(ns), 3, d)
    got = call(dev, c, q, lens, ns, None, groups, prefix)
    assert fa.attn_last_device_error() == 0
    check(c, q, lens, ns, None, got)


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("B,G,d", [(44, 1, 128), (36, 1, 64), (10, 5, 128)])
def test_many_row_tiles(dev, codes, B, G, d):
    """9 to 13 row tiles of a group: CTAs beside each other over the same keys, some without a tile."""
    lens, ns, groups, prefix = [300 + b for b in range(B)], [64] * B, [0, B], [230]
    c = share(fill(dev, 410, lens, 1, d, 16, codes), groups, prefix)
    q = normal(dev, 411, 64 * B, G, d)
    got = call(dev, c, q, lens, ns, None, groups, prefix)
    assert fa.attn_last_device_error() == 0
    check(c, q, lens, ns, None, got)


def test_infinite_values_in_a_prefix(dev):
    """An infinite value makes its channel infinite (or NaN, where a probability is the sum of two parts and
    the second is 0 or negative, as over one sequence's own pages), and no other, also where a tile ends behind
    the prefix."""
    for B in (2, 60):
        lens, ns, groups, prefix, d = [180 + b % 4 for b in range(B)], [1] * B, [0, B], [176], 128
        c = share(fill(dev, 420, lens, 1, d, 16, False), groups, prefix)
        c["v_cache"][int(c["page_table"][0, 10]), 15, 0, 9] = float("inf")  # the prefix's last position
        q = normal(dev, 421, B, 4, d)
        o, lse = call(dev, c, q, lens, ns, None, groups, prefix)
        assert fa.attn_last_device_error() == 0
        assert not o[..., 9].isfinite().any() and lse.isfinite().all()
        o[..., 9] = 0
        assert o.isfinite().all()


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("graph", [False, True])
def test_other_batches_one_behind_the_other(dev, codes, graph):
    """The same buffers with other offsets, lengths and groups from call to call, nothing waited for between."""
    rng, B, T, P, S, page, pages = random.Random(7), 30, 3, 500, 70, 16, 1500
    kind = torch.float8_e4m3fn if codes else torch.bfloat16
    kc, vc = (normal(dev, 370 + i, pages * page, 2, 128).view(pages, page, 2, 128).to(kind) for i in range(2))
    scales = {n: torch.full((pages, 2, page), 1.5, device=dev) if codes else None for n in ("k_scale", "v_scale")}
    batches = []
    for i in range(12):
        groups = sorted([0, B] + [rng.randint(0, B) for _ in range(2)])
        prefix, ns = [rng.randint(0, P) for _ in range(3)], [rng.randint(0, T) for _ in range(B - 1)] + [T]
        lens, table = [], torch.randint(0, pages, (B, (P + S + T) // page + 2), generator=torch.Generator().manual_seed(i))
        for k in range(3):
            for b in range(groups[k], groups[k + 1]):
                lens.append(prefix[k] + ns[b] + rng.randint(0, S))
                table[b, :prefix[k] // page] = table[groups[k], :prefix[k] // page]
        batches.append((normal(dev, 380 + i, B * T, 8, 128), table.to(dev, torch.int32), ints(dev, lens), cu_of(dev, ns),
                        ints(dev, groups), ints(dev, prefix), sum(ns)))
    q, table, lens, cu, groups, prefix = bufs = [x.clone() for x in batches[0][:6]]
    run = lambda: fa.prefix_decode(q, kc, vc, table, lens, cu, T, P + S + T, groups, prefix, B * T, P, **scales)

    def put(batch):
        for x, y in zip(bufs, batch):
            x.copy_(y)

    want = []
    for batch in batches:
        put(batch)
        torch.cuda.synchronize()
        want.append([x[:batch[6]].clone() for x in run()])
        torch.cuda.synchronize()
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run()
    got = []
    for batch in batches * 3:
        put(batch)
        if graph:
            g.replay()
        else:
            run()
            out = run()
        got.append([x[:batch[6]].clone() for x in out])
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for a, b in zip(got, want * 3) for x, y in zip(a, b))
    assert fa.attn_last_device_error() == 0


@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("H,G,n,codes", [(1825, 1, 300, False), (2001, 8, 70, True), (3001, 1, 20, False)])
def test_more_heads_than_units(dev, H, G, n, codes, grouped):
    """Odd head counts above the units of a line: each head is a segment of its own, and every one is computed."""
    lens, ns, groups, prefix = [n], [1], [0, 1] if grouped else [0], [n - 2] if grouped else []
    c = fill(dev, 430, lens, H, 64, 16, codes)
    q = normal(dev, 431, 1, H * G, 64)
    out = torch.full((1, H * G, 64), 7.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((1, H * G), -77.0, device=dev)  # no row's: scores are below 30, and keys above one
    call(dev, c, q, lens, ns, None, groups, prefix, out=out, lse=lse)
    assert fa.attn_last_device_error() == 0
    assert not (lse == -77.0).any()
    check(c, q, lens, ns, None, (out, lse))


@pytest.mark.parametrize("B", [12, 60, 150])  # one row tile of a group, a pair, several CTAs beside each other
@pytest.mark.parametrize("d,G", [(64, 16), (128, 5), (128, 8)])
def test_one_token_rows_lose_nothing_of_their_weights(dev, B, d, G):
    """A row that attention over its own pages takes with probabilities as the sum of two bf16 (up to 8 rows
    a key head, 16 at d = 64) has them over a shared prefix too: 2^-8 of 2^-8 of each is lost, so O is good to
    its own rounding (2^-8) and what scores and sums add, as in tests/test_tree_gpu.py."""
    lens, ns, groups, prefix = [700 + b % 7 for b in range(B)], [1] * B, [0, B], [696]
    c = share(fill(dev, 440, lens, 1, d, 16, False), groups, prefix)
    q = normal(dev, 441, B, G, d, std=1.5)
    o, lse = (t.cpu().double() for t in call(dev, c, q, lens, ns, None, groups, prefix))
    assert fa.attn_last_device_error() == 0
    k, v = rows_of(c)
    wo, wl, A, S = ref.tree(q.cpu(), k, v, c["page_table"].cpu(), 16, lens, list(range(B + 1)), None, d ** -0.5)
    tol = 2.0 ** -8 * wo.abs() + A * (2.0 ** -16 + 2.0 ** -19 * S[..., None] + 2.0 ** -17)
    assert ((o - wo).abs() <= tol).all(), ((o - wo).abs() / tol).max()
    assert ((lse - wl).abs() <= 2.0 ** -19 * S + 2.0 ** -20 * wl.abs() + 2.0 ** -18).all()
