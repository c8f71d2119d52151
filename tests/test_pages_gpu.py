"""Pages between steps: the next batch's page table, copies, accepted rows moved
together.  Whole numbers and bytes: results must be equal."""
import random

import pytest

torch = pytest.importorskip("torch")

import io_aware_exact_06_gb300 as fa
from tests import sample_ref as ref
from tests import serve_ref
from tests.test_cache_gpu import cu_of, make, normal, put

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


# ----------------------------------------------------------------------- fork --
def plan(seed, B, page, top, spare, share=0.5):
    """A batch in which some rows share the beginning of the row before them, at times all of it."""
    rng = random.Random(seed)
    lens = [rng.randrange(0, top + 1) for _ in range(B)]
    order, at, table = list(range(2 * B * (top // page + 2) + spare)), 0, []
    rng.shuffle(order)
    width = top // page + 3
    for b in range(B):
        if b and rng.random() < 0.3:
            lens[b] = lens[b - 1]
        n, take = -(-lens[b] // page), 0
        if b and rng.random() < share:
            both = min(lens[b], lens[b - 1])
            take = n if lens[b] == lens[b - 1] and rng.random() < 0.7 else rng.randrange(0, both // page + 1)
        row = table[-1][:take] if take else []
        row = row + order[at:at + n - take] + [-9] * (width - n)
        at += n - take
        table.append(row)
    pages = at + spare
    names = sorted(p for row in table for p in set(row) if p >= 0)
    number = {p: i for i, p in enumerate(sorted(set(names), key=lambda p: (p * 7919) % 1000003))}
    spread = sorted(rng.sample(range(pages), len(number)))
    rng.shuffle(spread)
    table = [[spread[number[p]] if p >= 0 else -9 for p in row] for row in table]
    refs = [0] * pages
    for b, row in enumerate(table):
        for p in row[:-(-lens[b] // page)]:
            refs[p] += 1
    return table, lens, refs, width * page


def call(dev, table, lens, parents, new, refs, page, **kw):
    t = ints(dev, table) if table else torch.zeros((0, kw.pop("width")), dtype=torch.int32, device=dev)
    return fa.cache_fork(t, ints(dev, lens), ints(dev, parents), ints(dev, new), ints(dev, refs), page, **kw)


@pytest.mark.parametrize("B,N,page,top,seed", [(1, 1, 16, 40, 1), (3, 8, 16, 100, 2), (8, 3, 32, 500, 3), (20, 20, 64, 900, 4),
                                               (40, 90, 16, 300, 5), (90, 40, 128, 2000, 6), (300, 700, 16, 200, 7),
                                               (1500, 1400, 16, 60, 8)])
def test_against_the_definition(dev, B, N, page, top, seed):
    rng = random.Random(seed)
    table, lens, refs, room = plan(seed, B, page, top, 40 + N * (top // page + 4))
    parents, new = [], []
    for i in range(N):
        r = rng.choice([i % B, rng.randrange(B), rng.randrange(B), -1])
        old = lens[r] if r >= 0 else 0
        kind = rng.randrange(4)
        parents.append(r)
        new.append(min(room, [old, old + rng.randrange(1, 40), max(0, old - rng.randrange(0, 40)), rng.randrange(0, top + 1)][kind]))
    got = call(dev, table, lens, parents, new, refs, page)
    assert fa.attn_last_device_error() == 0
    want = ref.fork(table, lens, parents, new, refs, page)
    for x, y in zip(got, want):
        assert x.tolist() == y
    again = ints(dev, refs)
    out = torch.empty_like(got[0])
    got = fa.cache_fork(ints(dev, table), ints(dev, lens), ints(dev, parents), ints(dev, new), again, page, out=out, refs_out=again)
    assert again.tolist() == want[1] and out.tolist() == want[0] and got[2].tolist() == want[2]
    assert fa.attn_last_device_error() == 0


def test_steps_one_after_the_other(dev):
    """Twenty steps of forks, growth and ends: counts are those of the tables, and no page is lost."""
    rng, page, pages, width = random.Random(3), 16, 4000, 40
    table, lens, refs = [], [], [0] * pages
    for step in range(20):
        B = len(lens)
        parents = [rng.randrange(-1, B) for _ in range(rng.randrange(1, 40))]
        new = [min(width * page, (lens[r] if r >= 0 else 0) + rng.randrange(-10, 60)) for r in parents]
        new = [max(0, n) for n in new]
        got = call(dev, table, lens, parents, new, refs, page, **({} if table else {"width": width}))
        assert fa.attn_last_device_error() == 0
        want = ref.fork(table, lens, parents, new, refs, page) if table else None
        table, refs = got[0].tolist(), got[1].tolist()
        if want:
            assert (table, refs, got[2].tolist(), got[3].tolist()) == want
        lens = new
        counted = [0] * pages
        for row, n in zip(table, lens):
            for p in row[:-(-n // page)]:
                counted[p] += 1
            assert all(p == -1 for p in row[-(-n // page):])
        assert counted == refs
    got = call(dev, table, lens, [], [], refs, page)
    assert not any(got[1].tolist()) and got[0].shape == (0, width)


def test_many_pages(dev):
    """A pool of a million pages, few of them free and far apart; the last one among them."""
    page, pages = 16, 1 << 20
    refs = torch.ones(pages, dtype=torch.int32)
    free = torch.randperm(pages, generator=torch.Generator().manual_seed(1))[:3000].sort().values
    free[-1] = pages - 1
    refs[free] = 0
    got = fa.cache_fork(torch.zeros((0, 50), dtype=torch.int32, device=dev), ints(dev, []), ints(dev, [-1] * 60),
                        ints(dev, [800] * 60), refs.to(dev), page)
    assert fa.attn_last_device_error() == 0
    assert torch.equal(got[0].flatten().cpu(), free.int())
    assert (got[1] == 1).all() and (got[2] == -1).all() and (got[3] == -1).all()


@pytest.mark.parametrize("what", ["pages", "parent", "low parent", "length", "new length", "negative", "page", "count"])
def test_plans_that_are_not_possible(dev, what):
    """Nothing changes hands, and the reason is reported."""
    page, table, lens, parents, new = 16, [[3, 5, -1], [3, 7, 8]], [20, 40], [0, 0, 1], [40, 20, 41]
    refs = [0, 0, 0, 2, 0, 1, 0, 1, 1, 0]
    status = -11
    if what == "pages":
        refs = [1 if n == 0 and p != 4 else n for p, n in enumerate(refs)]
        status = -12
    elif what == "parent":
        parents[2] = 2
    elif what == "low parent":
        parents[0] = -2
    elif what == "length":
        lens[1], status = 49, -8
    elif what == "negative":
        lens[0], status = -1, -8
    elif what == "new length":
        new[1], status = 49, -8
    elif what == "page":
        table[1][1] = 10
    else:
        refs[5] = 0
    got = call(dev, table, lens, parents, new, refs, page)
    assert fa.attn_last_device_error() == status
    assert got[1].tolist() == refs
    for x in (got[0], got[2], got[3]):
        assert (x == -1).all()
    refs = [0, 0, 0, 2, 0, 1, 0, 1, 1, 0]
    good = call(dev, [[3, 5, -1], [3, 7, 8]], [20, 40], [0, 0, 1], [40, 20, 41], refs, page)
    assert fa.attn_last_device_error() == 0
    # row 0 grows into page 5, which row 1 still reads; pages 0, 1 and 2 are the lowest free ones
    assert good[0].tolist() == [[3, 0, 1], [3, 5, -1], [3, 7, 8]] and good[2].tolist() == [5, -1, -1] and good[3].tolist() == [0, -1, -1]
    assert good[1].tolist() == [1, 1, 0, 3, 0, 1, 0, 1, 1, 0]


def test_counts_that_are_too_low(dev):
    """A page named twice and counted once: reported; memory stays sound."""
    got = call(dev, [[1], [1]], [10, 10], [], [], [0, 1, 0], 16)
    assert fa.attn_last_device_error() == -11
    assert got[1].tolist() == [0, -1, 0]


def test_tables_that_overlap_are_refused(dev):
    t = torch.zeros((2, 3), dtype=torch.int32, device=dev)
    a = ints(dev, [0, 0])
    with pytest.raises(fa.AttnError):
        fa.cache_fork(t, a, a, a, ints(dev, [0] * 5), 16, out=t)


# ----------------------------------------------------------------------- copy --
def bytes_of(c):
    return [t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)
            for t in (c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"]) if t is not None]


def noise(dev, seed, pages, H, d, page, codes):
    g = torch.Generator(device=dev).manual_seed(seed)
    c = {"page": page}
    for n in "kv":
        if codes:
            c[n + "_cache"] = torch.randint(0, 256, (pages, page, H, d), generator=g, device=dev, dtype=torch.uint8).view(torch.float8_e4m3fn)
            c[n + "_scale"] = torch.rand(pages, H, page, generator=g, device=dev)
        else:
            c[n + "_cache"] = torch.randint(-32768, 32768, (pages, page, H, d), generator=g, device=dev, dtype=torch.int16).view(torch.bfloat16)
            c[n + "_scale"] = None
    return c


@pytest.mark.parametrize("pages,n,H,d,page,codes", [(5, 1, 1, 64, 16, False), (40, 13, 3, 64, 16, True), (40, 20, 8, 128, 64, True),
                                                   (300, 150, 5, 128, 256, False), (3000, 1400, 1, 64, 16, True)])
def test_copies(dev, pages, n, H, d, page, codes):
    c = noise(dev, 600, pages, H, d, page, codes)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(5)).tolist()
    src, dst = order[:n], order[n:2 * n]
    src[n // 2:] = [src[0]] * (n - n // 2)  # one page into many
    for i in range(3, n, 4):
        src[i], dst[i] = -1, (-1 if i % 8 == 3 else 1 << 30)  # left out, whatever the target
    want = [t.clone() for t in bytes_of(c)]
    for a, b in zip(src, dst):
        if a >= 0:
            for t, w in zip(bytes_of(c), want):
                w[b] = t[a]
    fa.cache_copy(c["k_cache"], c["v_cache"], ints(dev, src), ints(dev, dst), k_scale=c["k_scale"], v_scale=c["v_scale"])
    assert fa.attn_last_device_error() == 0
    for t, w in zip(bytes_of(c), want):
        assert torch.equal(t, w)


@pytest.mark.parametrize("src,dst", [(-2, 3), (9, 3), (1, -1), (1, 9), (1 << 30, 1)])
def test_copies_outside_the_cache(dev, src, dst):
    c = noise(dev, 601, 9, 2, 64, 16, True)
    want = [t.clone() for t in bytes_of(c)]
    for w in want:
        w[4] = w[0]
    fa.cache_copy(c["k_cache"], c["v_cache"], ints(dev, [src, 0]), ints(dev, [dst, 4]), k_scale=c["k_scale"], v_scale=c["v_scale"])
    assert fa.attn_last_device_error() == -11
    for t, w in zip(bytes_of(c), want):
        assert torch.equal(t, w)


@pytest.mark.parametrize("codes", [False, True])
def test_copies_past_32_bits(dev, codes):
    pages = 17000 if codes else 9000
    c = noise(dev, 602, pages, 8, 128, 256, codes)
    want = [t[pages - 1].clone() for t in bytes_of(c)], [t[0].clone() for t in bytes_of(c)]
    fa.cache_copy(c["k_cache"], c["v_cache"], ints(dev, [pages - 1, 0]), ints(dev, [1, pages - 2]), k_scale=c["k_scale"],
                  v_scale=c["v_scale"])
    assert fa.attn_last_device_error() == 0
    for t, a, b in zip(bytes_of(c), *want):
        assert torch.equal(t[1], a) and torch.equal(t[pages - 2], b)


# -------------------------------------------------------------------- compact --
def walks(seed, ns):
    rng, path, kept = random.Random(seed), [], []
    for n in ns:
        mine = sorted(rng.sample(range(n), rng.randrange(0, n + 1)))
        path += mine + [-1] * (n - len(mine))
        kept.append(len(mine))
    return path, kept


COMPACT = [  # lengths, new tokens, H, d, page, codes
    ([1], [1], 1, 64, 16, False), ([40, 0, 33], [9, 0, 33], 3, 64, 16, True), ([300, 64, 65, 200], [64, 64, 1, 33], 8, 128, 16, True),
    ([300, 64, 65, 200], [64, 64, 1, 33], 5, 128, 64, False), ([500, 450], [300, 129], 40, 64, 256, True), ([30] * 300, [5, 6] * 150, 2, 64, 32, False)]


def compact(dev, c, lens, ns, path, kept, **kw):
    fa.cache_compact(c["k_cache"], c["v_cache"], c["page_table"], ints(dev, lens), kw.pop("cu", cu_of(dev, ns)), ints(dev, path),
                     ints(dev, kept), k_scale=c["k_scale"], v_scale=c["v_scale"])


def moved(c, lens, ns, path, kept, sequences=None):
    """The cache's bytes with the accepted rows in their places."""
    table, page, at, want = c["page_table"].cpu(), c["page"], 0, []
    flat = [t.transpose(1, 2).flatten(0, 1) if t.dim() == 3 else t.flatten(0, 1) for t in bytes_of(c)]
    out = [t.clone() for t in flat]
    for b, (L, n) in enumerate(zip(lens, ns)):
        if sequences is None or b in sequences:
            for j in range(kept[b]):
                to, come = (int(serve_ref.row_index(table, page, b, torch.tensor(L - n + x))) for x in (j, path[at + j]))
                for t, o in zip(flat, out):
                    o[to] = t[come]
        at += n
    for t, o in zip(bytes_of(c), out):
        o = o.unflatten(0, (-1, page))
        want.append(o.transpose(1, 2) if t.dim() == 3 else o)
    return want


@pytest.mark.parametrize("lens,ns,H,d,page,codes", COMPACT)
def test_accepted_rows_move_together(dev, lens, ns, H, d, page, codes):
    for seed in range(3):
        c = make(dev, 610 + seed, lens, H, d, page, codes)
        c.update({n: t for n, t in noise(dev, 611, c["k_cache"].shape[0], H, d, page, codes).items() if n != "page"})
        path, kept = walks(seed, ns)
        want = moved(c, lens, ns, path, kept)
        compact(dev, c, lens, ns, path, kept)
        assert fa.attn_last_device_error() == 0
        for t, w in zip(bytes_of(c), want):
            assert torch.equal(t, w)


@pytest.mark.parametrize("what", ["order", "twice", "beyond", "below", "many", "negative", "short", "falls", "total", "page"])
def test_walks_that_are_none(dev, what):
    """Reported; the sequence concerned stays as it is, the others are moved."""
    lens, ns = [50, 60, 70], [6, 6, 6]
    c = make(dev, 620, lens, 2, 64, 16, True)
    c.update({n: t for n, t in noise(dev, 621, c["k_cache"].shape[0], 2, 64, 16, True).items() if n != "page"})
    path, kept = [0, 2, 5, -1, -1, -1] * 3, [3, 3, 3]
    cu, lens_now, status, fine = cu_of(dev, ns), list(lens), -11, {0, 2}
    if what == "order":
        path[6:9] = [0, 5, 2]
    elif what == "twice":
        path[6:9] = [0, 2, 2]
    elif what == "beyond":
        path[8] = 6
    elif what == "below":
        path[6] = -1
    elif what == "many":
        kept[1] = 7
    elif what == "negative":
        kept[1] = -1
    elif what == "short":
        lens_now[1], status = 5, -8
    elif what == "falls":
        cu[2], status, fine = 3, -8, set()
    elif what == "total":
        cu[3], status, fine = 19, -8, {0, 1}
    else:
        c["page_table"][1, 3] = 1 << 28  # positions 48 .. : all the new tokens after the place 54
        fine = {0, 2}
    safe = dict(c, page_table=c["page_table"].clamp_max(0x7fff)) if what == "page" else c
    want = moved(safe, lens, ns, path, kept, fine)
    compact(dev, c, lens_now, ns, path, kept, cu=cu)
    assert fa.attn_last_device_error() == status
    for t, w in zip(bytes_of(c), want):
        assert torch.equal(t, w)
