"""Attention of new tokens over the paged cache against fp64.

The reference takes the cache's own values (codes times scales), so the
tolerance counts the kernel's arithmetic alone.  With A = sum_j p_j |v_j| and S
the largest scale * sum |q k| of a row:
  - O is rounded to bf16 once: 2^-8 |O|;
  - probabilities are rounded to bf16 (2^-8 of each, so 2^-8 A), or with codes,
    times the value scale, to fp16 (2^-11 A, and 2^-25 of the largest weight for
    each key below fp16's normal range: 2^-25 L max|v|); where many rows share a
    key, probabilities and scaled values are, each (2^-11 A twice, so 2^-10 A);
  - scores are fp32 sums of d products (below 2^-19 S), a probability errs by
    its score's error and that of exp2 and the sums (2^-18): (2^-19 S + 2^-17) A;
  - LSE: 2^-19 S + 2^-20 |LSE| + 2^-18.
"""
import math
import random

import pytest

torch = pytest.importorskip("torch")

import io_aware_exact_06_gb300 as fa
from tests import serve_ref as ref
from tests.test_cache_gpu import cu_of, make, normal, put

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import __graft_entry__
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    __graft_entry__.build()
    return torch.device("cuda:0")


def signed(word):
    return word - (1 << 64) if word >> 63 else word


def random_masks(seed, ns):
    """Trees, full rows, rows that see one token, and empty ones."""
    rng, words = random.Random(seed), []
    for n in ns:
        mine = []
        for i in range(n):
            kind = rng.randrange(6)
            up = mine[rng.randrange(i)] if i else 0
            w = up | 1 << i if kind < 3 else 0 if kind == 3 else 1 << rng.randrange(n) if kind == 4 else (1 << 64) - 1
            mine.append(w)
        words += mine
    return torch.tensor([signed(w) for w in words], dtype=torch.int64)


def rows_of(c):
    """fp64 rows [rows, H, d] of the cache's keys and values."""
    out = []
    for n in "kv":
        x = c[n + "_cache"].cpu().double().flatten(0, 1)
        if c[n + "_scale"] is not None:
            x = x * c[n + "_scale"].cpu().double().transpose(1, 2).flatten(0, 1)[..., None]
        out.append(x)
    return out


def fill(dev, seed, lens, H, d, page, codes, std=1.0):
    c = make(dev, seed, lens, H, d, page, codes)
    total = sum(lens)
    kv = normal(dev, seed + 1, total, 2 * H, d, std=std)
    put(dev, c, kv[:, :H], kv[:, H:], lens, lens)
    assert fa.attn_last_device_error() == 0
    return c


def call(dev, c, q, lens, ns, mask, **kw):
    kw.setdefault("max_new", max(ns))
    kw.setdefault("max_len", max(lens))
    return fa.tree_decode(q, c["k_cache"], c["v_cache"], c["page_table"],
                          torch.tensor(lens, dtype=torch.int32, device=dev), cu_of(dev, ns),
                          mask=None if mask is None else mask.to(dev), k_scale=c["k_scale"], v_scale=c["v_scale"], **kw)


def check(c, q, lens, ns, mask, got, scale=None, rows=None):
    o, lse = (t.cpu().double() for t in got)
    cu = [sum(ns[:i]) for i in range(len(ns) + 1)]
    total = cu[-1]
    k, v = rows or rows_of(c)
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    wo, wl, A, S = ref.tree(q[:total].cpu(), k, v, c["page_table"].cpu(), c["page"], lens, cu, mask, scale)
    o, lse = o[:total], lse[:total]
    codes = c["k_scale"] is not None
    empty = wl == -math.inf
    assert (o[empty] == 0).all() and (lse[empty] == -math.inf).all()
    fine = ~empty
    vmax = v[torch.isfinite(v)].abs().max()
    step = 2.0 ** -10 if codes else 2.0 ** -8
    tol = 2.0 ** -8 * wo.abs() + A * (step + 2.0 ** -19 * S[..., None] + 2.0 ** -17)
    if codes:
        tol = tol + 2.0 ** -25 * max(lens) * vmax
    off = (o - wo).abs()
    assert (off[fine] <= tol[fine]).all(), (off[fine] / tol[fine]).max()
    off, tol = (lse - wl).abs()[fine], (2.0 ** -19 * S + 2.0 ** -20 * wl.abs() + 2.0 ** -18)[fine]
    assert (off <= tol).all(), (off / tol).max()


CASES = [  # lengths, new tokens, Hq, H, d, page, codes, tree, splits
    ([1], [1], 1, 1, 64, 16, False, False, 0),
    ([1, 7, 64, 65, 129], [1, 1, 1, 1, 1], 4, 4, 128, 16, False, False, 0),
    ([300, 1, 63], [1, 1, 1], 16, 2, 64, 32, True, False, 3),
    ([513, 16, 200], [1, 0, 1], 24, 3, 128, 64, True, False, 7),
    ([257, 31, 64], [5, 31, 3], 6, 2, 128, 16, False, True, 0),
    ([257, 31, 64], [5, 31, 3], 6, 2, 128, 16, True, True, 2),
    ([400, 64, 65], [64, 64, 1], 8, 1, 64, 128, True, True, 0),
    ([400, 64, 65], [64, 64, 1], 8, 1, 64, 128, False, True, 4),
    ([1000, 700], [33, 64], 8, 4, 128, 256, True, True, 1),
    ([1000, 700], [33, 64], 6, 2, 128, 256, False, True, 5),
    ([150, 90, 10], [17, 9, 10], 5, 5, 64, 16, False, False, 0),
    ([90, 130], [20, 2], 14, 2, 128, 16, True, False, 0),
    ([2000], [2], 40, 2, 128, 64, True, True, 256),
    ([130] * 40, [2] * 40, 2, 1, 64, 16, True, True, 2),
    ([900, 500], [64, 50], 16, 2, 128, 16, True, True, 2),
    ([900, 500], [64, 50], 16, 2, 64, 32, False, True, 0),
]


@pytest.mark.parametrize("lens,ns,Hq,H,d,page,codes,tree,splits", CASES)
def test_against_fp64(dev, lens, ns, Hq, H, d, page, codes, tree, splits):
    seed = 100 + len(lens) * 7 + Hq + d
    c = fill(dev, seed, lens, H, d, page, codes)
    total = sum(ns)
    base = normal(dev, seed + 2, total, Hq + 2, d, std=1.5)  # a token stride
    q = base[:, :Hq]
    mask = random_masks(seed, ns) if tree else None
    got = call(dev, c, q, lens, ns, mask, num_splits=splits)
    assert fa.attn_last_device_error() == 0
    check(c, q, lens, ns, mask, got)
    again = call(dev, c, q, lens, ns, mask, num_splits=splits)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("std", [0.0, 6.0])
def test_peaky_and_flat_scores(dev, codes, std):
    """A running maximum that moves often, and one that never does."""
    lens, ns = [800, 333], [9, 4]
    c = fill(dev, 200, lens, 2, 128, 16, codes, std=max(std, 1.0))
    q = normal(dev, 203, 13, 8, 128, std=std)
    for splits in (0, 4):
        got = call(dev, c, q, lens, ns, None, num_splits=splits)
        check(c, q, lens, ns, None, got)
    got = call(dev, c, q, lens, ns, None, scale=0.0)
    check(c, q, lens, ns, None, got, scale=0.0)
    assert fa.attn_last_device_error() == 0


@pytest.mark.parametrize("codes", [False, True])
def test_value_scales_of_all_sizes(dev, codes):
    """Tokens whose keys and values differ by many powers of two, and queries that do."""
    lens, ns, H, d = [300], [5], 1, 128
    c = make(dev, 210, lens, H, d, 16, codes)
    kv = normal(dev, 211, 300, 2, d)
    kv[:, 1] *= torch.exp2(torch.arange(300, device=dev) % 41 - 20.0)[:, None].to(torch.bfloat16)
    put(dev, c, kv[:, :1], kv[:, 1:], lens, lens)
    q = normal(dev, 212, 5, 2, d)
    q[1] *= 2.0 ** -30
    q[2] *= 2.0 ** 5
    q[3, 0] = 0
    q[4, 1, ::2] *= 2.0 ** -20
    check(c, q, lens, ns, None, call(dev, c, q, lens, ns, None))
    q[0] *= 2.0 ** 20  # one key takes all
    got = call(dev, c, q, lens, ns, None)
    assert got[0].isfinite().all() and got[1].isfinite().all()


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("splits", [1, 3])
def test_what_hidden_keys_hold_does_not_matter(dev, codes, d, splits):
    """Drafted tokens with NaN and infinite keys, values and scales reach only the
    rows that see them; rows behind a sequence (NaN in every fresh page) reach none."""
    lens, ns, H, Hq = [200, 70], [6, 6], 2, 4
    c = fill(dev, 220, lens, H, d, 16, codes)
    table = c["page_table"].cpu()
    bad = {}
    for b, j, n in ((0, 1, "k"), (0, 2, "v"), (1, 3, "v"), (1, 5, "k")):
        row = int(ref.row_index(table, 16, b, torch.tensor(lens[b] - ns[b] + j)))
        page, at = row // 16, row % 16
        if codes:
            c[n + "_cache"].view(torch.uint8)[page, at, :, 5] = 0x7f
            c[n + "_scale"][page, :, at] = float("nan") if j % 2 else float("inf")
        else:
            c[n + "_cache"][page, at, :, 5] = float("nan") if j % 2 else float("inf")
        bad[(b, j)] = n
    q = normal(dev, 223, 12, Hq, d)
    # row i sees itself and token 0; the bad tokens are seen by themselves alone
    mask = torch.tensor([1 | 1 << i for _ in ns for i in range(6)], dtype=torch.int64)
    got = call(dev, c, q, lens, ns, mask, num_splits=splits)
    assert fa.attn_last_device_error() == 0
    k, v = rows_of(c)
    cu = [0, 6, 12]
    clean = [t for b in range(2) for t in range(cu[b], cu[b + 1]) if (b, t - cu[b]) not in bad]
    wo, wl, A, S = ref.tree(q.cpu(), k, v, table, 16, lens, cu, mask, d ** -0.5)
    assert wo[clean].isfinite().all()
    o, lse = got[0].cpu().double(), got[1].cpu().double()
    assert ((o[clean] - wo[clean]).abs() <= 2.0 ** -7 * (A[clean] + 0.01)).all()
    assert ((lse[clean] - wl[clean]).abs() <= 1e-4).all()
    for (b, j), n in bad.items():
        t = cu[b] + j
        if n == "k":
            assert o[t].isnan().all()
        else:
            assert not o[t, :, 5].isfinite().any()
            if not codes:  # an infinite value is what the sum holds; the other columns stay sound
                assert o[t, :, 6:].isfinite().all() and (o[t, :, 5].isnan().all() if j % 2 else o[t, :, 5].isinf().all())


@pytest.mark.parametrize("codes", [False, True])
def test_rows_that_see_nothing(dev, codes):
    lens, ns = [4, 70], [4, 6]
    c = fill(dev, 230, lens, 1, 64, 16, codes)
    q = normal(dev, 233, 10, 3, 64)
    mask = torch.tensor([0, 2, 0, 9] + [0] * 6, dtype=torch.int64)
    for splits in (1, 2):
        got = call(dev, c, q, lens, ns, mask, num_splits=splits)
        assert fa.attn_last_device_error() == 0
        check(c, q, lens, ns, mask, got)
        assert (got[0][[0, 2]] == 0).all() and (got[1][[0, 2]] == -math.inf).all()


def test_padded_batch_and_bounds(dev):
    """Rows behind the last sequence stay as they were; larger bounds than needed change nothing but the split."""
    lens, ns = [90, 0, 33], [3, 0, 2]
    c = fill(dev, 240, lens, 2, 128, 32, True)
    q = normal(dev, 243, 12, 4, 128)
    out = torch.full((12, 4, 128), 7.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((12, 4), 7.0, device=dev)
    call(dev, c, q, lens, ns, None, out=out, lse=lse, max_new=64, max_len=5000)
    assert fa.attn_last_device_error() == 0
    check(c, q, lens, ns, None, (out, lse))
    assert (out[5:] == 7).all() and (lse[5:] == 7).all()


def test_equals_decode_on_a_dense_cache(dev):
    """One token, one query head per key head, pages in order: attn_fwd_decode's
    answer, to both kernels' rounding (2^-8 of probabilities, 2^-8 of O)."""
    B, H, d, L = 3, 4, 128, 512
    k, v = normal(dev, 250, B * L, H, d), normal(dev, 251, B * L, H, d)
    q = normal(dev, 252, B, H, d)
    table = torch.arange(B * L // 64, dtype=torch.int32, device=dev).view(B, -1)
    o, lse = fa.tree_decode(q, k.view(-1, 64, H, d), v.view(-1, 64, H, d), table,
                            torch.full((B,), L, dtype=torch.int32, device=dev), cu_of(dev, [1] * B), 1, L)
    o2, lse2 = fa.decode(q, k, v, cu_of(dev, [L] * B), L)
    assert fa.attn_last_device_error() == 0
    assert (o.float() - o2.float()).abs().max() <= 2.0 ** -7
    assert (lse - lse2).abs().max() <= 2.0 ** -14


def test_offsets_past_32_bits(dev):
    pages = 17000
    for codes in (True, False):
        lens, ns, H, d, page = [300], [4], 8, 128, 256
        c = make(dev, 260, lens, H, d, page, codes, spare=pages)
        c["page_table"] = torch.tensor([[pages, pages - 1]], dtype=torch.int32, device=dev)
        kv = normal(dev, 261, 300, 2 * H, d)
        put(dev, c, kv[:, :H], kv[:, H:], lens, lens)
        q = normal(dev, 262, 4, 16, d)
        got = call(dev, c, q, lens, ns, None)
        assert fa.attn_last_device_error() == 0
        small = {**c, "page_table": torch.tensor([[1, 0]], dtype=torch.int32, device=dev)}
        for n in "kv":
            small[n + "_cache"] = c[n + "_cache"][pages - 1:pages + 1].clone()
            if codes:
                small[n + "_scale"] = c[n + "_scale"][pages - 1:pages + 1].clone()
        want = call(dev, small, q, lens, ns, None)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        del c, got
        torch.cuda.empty_cache()


@pytest.mark.parametrize("what", ["page", "negative page", "draft page", "short", "long", "too many", "past total"])
def test_bad_plans_are_reported(dev, what):
    """Other sequences are right; rows that read a page outside the cache are NaN,
    rows of a sequence with impossible lengths are not written."""
    lens, ns, H, d = [200, 300, 50], [2, 3, 4], 2, 64
    c = fill(dev, 270, lens, H, d, 16, True)
    q = normal(dev, 273, 9, 4, d)
    good = call(dev, c, q, lens, ns, None, num_splits=3)
    lens_d, cu, table = torch.tensor(lens, dtype=torch.int32, device=dev), cu_of(dev, ns), c["page_table"].clone()
    max_new, total, status, ruined = 4, 9, -8, slice(2, 5)
    if what == "page":
        table[1, 2], status = table.new_tensor(c["k_cache"].shape[0]), -11
    elif what == "negative page":
        table[1, 0], status = -3, -11
    elif what == "draft page":
        table[1, 18], status = 1 << 30, -11
    elif what == "short":
        lens_d[1] = 2
    elif what == "long":
        lens_d[1] = 301
    elif what == "too many":
        max_new, ruined = 3, slice(5, 9)
    else:
        total, ruined = 8, slice(5, 8)
    for splits in (1, 3):
        out = torch.full((total, 4, d), 7.0, dtype=torch.bfloat16, device=dev)
        lse = torch.full((total, 4), 7.0, device=dev)
        fa.tree_decode(q[:total], c["k_cache"], c["v_cache"], table, lens_d, cu, max_new, 300, k_scale=c["k_scale"],
                       v_scale=c["v_scale"], num_splits=splits, out=out, lse=lse)
        assert fa.attn_last_device_error() == status
        if status == -11:
            assert out[ruined].isnan().all() and lse[ruined].isnan().all()
        else:
            assert (out[ruined] == 7).all() and (lse[ruined] == 7).all()
        others = [t for t in range(total) if not ruined.start <= t < ruined.stop]
        assert ((out[others].float() - good[0][others].float()).abs() <= 2.0 ** -7).all()
        assert ((lse[others] - good[1][others]).abs() <= 2.0 ** -14).all()
    assert fa.attn_last_device_error() == 0
