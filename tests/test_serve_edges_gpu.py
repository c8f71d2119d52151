"""What the norm, the paged cache and attention over it do at their edges: values
that are not finite where a kernel could lose or spread them, value scales far
apart, plans whose offsets are no batch, kinds without heads.

Tolerances as in test_tree_gpu.py, where nothing else is said.
"""
import math

import pytest

torch = pytest.importorskip("torch")

import io_aware_exact_06_gb300 as fa
from tests import serve_ref as ref
from tests.test_cache_gpu import make, normal, put
from tests.test_norm_gpu import inputs, to
from tests.test_tree_gpu import call, fill, rows_of

pytestmark = pytest.mark.gpu

ROWS = [1, 2, 3, 24, 40]  # query heads to a key head: 6, 12, 18, 144 and 240 rows with six new tokens
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def dev():
    import __graft_entry__
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    __graft_entry__.build()
    return torch.device("cuda:0")


def want_of(c, q, lens, ns, mask):
    cu = [sum(ns[:i]) for i in range(len(ns) + 1)]
    return ref.tree(q.cpu(), *rows_of(c), c["page_table"].cpu(), c["page"], lens, cu, mask, q.shape[-1] ** -0.5)


def near(got, want, codes, which, heaviest=None):
    """O and LSE of the rows `which` [total, Hq] to the tolerances of test_tree_gpu.py.  heaviest: a row's
    largest p_j max|v_j|, of which a key may lose 2^-20 where its weight (over codes an fp16) is below
    fp16's normal range; given per row, times the keys."""
    o, lse = (t.cpu().double() for t in got)
    wo, wl, A, S = want
    step = 2.0 ** -10 if codes else 2.0 ** -8
    tol = 2.0 ** -8 * wo.abs() + A * (step + 2.0 ** -19 * S[..., None] + 2.0 ** -17)
    if codes and heaviest is not None:
        tol = tol + 2.0 ** -20 * heaviest[..., None]
    off = (o - wo).abs()
    assert (off[which] <= tol[which]).all(), (off[which] / tol[which]).max()
    off, tol = (lse - wl).abs(), 2.0 ** -19 * S + 2.0 ** -20 * wl.abs() + 2.0 ** -18
    assert (off[which] <= tol[which]).all(), (off[which] / tol[which]).max()


def heaviest_of(c, q, lens, ns, mask):
    """[total, Hq]: the keys of a row's sequence times its largest p_j max_c |v_jc|, in fp64."""
    k, v = rows_of(c)
    G, out, at = q.shape[1] // k.shape[1], [], 0
    for b, (L, n) in enumerate(zip(lens, ns)):
        r = ref.row_index(c["page_table"].cpu(), c["page"], b, torch.arange(L))
        x = torch.einsum("thd,lhd->thl", q[at:at + n].cpu().double(), k[r].repeat_interleave(G, 1)) * q.shape[-1] ** -0.5
        j = torch.arange(n)
        word = (mask[at:at + n, None] >> j) & 1 if mask is not None else (j <= j[:, None]).long()
        x[:, :, L - n:] = x[:, :, L - n:].masked_fill(word[:, None] == 0, -math.inf)
        p = torch.softmax(x, -1).nan_to_num(0.0)
        out.append(L * (p * v[r].abs().amax(-1).t().repeat_interleave(G, 0)).amax(-1))
        at += n
    return torch.cat(out)


@pytest.mark.parametrize("G", ROWS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("spot,large", [(5, 200), (200, 5), (5, 300), (300, 130)])
def test_nan_keys_beside_large_scores(dev, codes, d, G, spot, large):
    """A NaN key that every row sees makes every row NaN, however far the scores of
    other key tiles lie above it (here more than 2^126 in weight) and whichever tile
    holds it.  One piece a segment, so that tiles meet inside the launch."""
    L, ns, H = 400, [6], 1
    c = make(dev, 600, [L], H, d, 16, codes)
    kv = normal(dev, 601, L, 2, d)
    kv[large, 0] = 160.0 / d ** 0.5  # score about 160 against a query of ones
    put(dev, c, kv[:, :1], kv[:, 1:], [L], [L])
    row = int(ref.row_index(c["page_table"].cpu(), 16, 0, torch.tensor(spot)))
    if codes:
        c["k_cache"].view(torch.uint8)[row // 16, row % 16, :, 3] = 0x7f
    else:
        c["k_cache"][row // 16, row % 16, :, 3] = NAN
    q = torch.ones(6, H * G, d, dtype=torch.bfloat16, device=dev)
    o, lse = call(dev, c, q, [L], ns, None, num_splits=1)
    assert fa.attn_last_device_error() == 0
    assert o.isnan().all() and lse.isnan().all()


@pytest.mark.parametrize("G", ROWS)
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("spot,large", [(5, 200), (200, 5)])
def test_infinite_values_beside_large_scores(dev, codes, G, spot, large):
    """An infinite or NaN value of the context with next to no weight: its channel is not finite."""
    L, ns, H, d = 400, [6], 1, 128
    c = make(dev, 605, [L], H, d, 16, codes)
    kv = normal(dev, 606, L, 2, d)
    kv[large, 0] = 160.0 / d ** 0.5
    put(dev, c, kv[:, :1], kv[:, 1:], [L], [L])
    row = int(ref.row_index(c["page_table"].cpu(), 16, 0, torch.tensor(spot)))
    if codes:
        c["v_cache"].view(torch.uint8)[row // 16, row % 16, :, 3] = 0x7f
    else:
        c["v_cache"][row // 16, row % 16, :, 3] = INF
    q = torch.ones(6, H * G, d, dtype=torch.bfloat16, device=dev)
    o, lse = call(dev, c, q, [L], ns, None, num_splits=1)
    assert fa.attn_last_device_error() == 0
    assert not o[..., 3].isfinite().any() and lse.isfinite().all()
    assert o[..., :3].isfinite().all() and o[..., 4:].isfinite().all()


@pytest.mark.parametrize("G", ROWS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("splits", [0, 1])
def test_queries_that_are_not_finite(dev, codes, d, G, splits):
    """A query row with an infinity or a NaN is NaN wherever it sees a key, and no
    other row is touched: whatever the kernel, also where its one key's score is -inf
    (the third sequence).  Rows that see nothing stay 0 and -inf."""
    lens, ns, H = [300, 6, 1, 1], [6, 6, 1, 1], 2
    Hq = H * G
    c = fill(dev, 610, lens, H, d, 16, codes)
    q = normal(dev, 611, sum(ns), Hq, d)
    mask = torch.tensor([(1 << i + 1) - 1 for i in range(6)] + [0, 1, 0, 8, 0, 63, 1, 1], dtype=torch.int64)
    want, most = want_of(c, q, lens, ns, mask), heaviest_of(c, q, lens, ns, mask)
    bad = torch.zeros(sum(ns), Hq, dtype=torch.bool)
    q = q.clone()
    for t, h, ch, x in ((0, 0, 3, INF), (2, Hq - 1, d - 1, -INF), (3, Hq // 2, 17, NAN), (8, 0, 0, INF), (9, Hq - 1, 8, NAN),
                        (11, 0, 31, -INF), (12, 0, 5, INF), (13, 0, 5, -INF)):
        q[t, h, ch] = x
        bad[t, h] = True
    got = call(dev, c, q, lens, ns, mask, num_splits=splits)
    assert fa.attn_last_device_error() == 0
    empty = (mask == 0)[:, None].expand(-1, Hq)
    assert (got[0][empty.to(dev)] == 0).all() and (got[1][empty.to(dev)] == -math.inf).all()
    hit = (bad & ~empty).to(dev)
    assert got[0][hit].isnan().all() and got[1][hit].isnan().all()
    near(got, want, codes, ~bad & ~empty, most)


def same_finiteness(got, want, what):
    got = got.cpu().double()
    assert torch.equal(got.isfinite(), want.isfinite()), what
    fine = want.isfinite()
    assert ((got - want)[fine].abs() <= 2 ** -7 * want[fine].abs() + 2 ** -16).all(), what


@pytest.mark.parametrize("d,rot,inter", [(64, 0, False), (128, 0, True), (64, 32, False), (128, 48, True), (128, 16, False)])
def test_channels_that_do_not_rotate_stand_alone(dev, d, rot, inter):
    """An infinity or NaN in a channel from rot on reaches what the formula says: its own
    output and the row's norm, the gradient's row and its own weight, not a neighbour."""
    x = inputs(620, 9, 3, 2, d, rot, 1, None)
    x["wq"][d - 3] = INF                    # one weight: its channel of every query row
    x["k"] = x["k"].clone()
    x["k"][2, 1, d - 6] = NAN               # one input: its row, by the norm
    x["k"][4, 0, d - 1] = INF
    y = to(dev, {**x, "q": x["q"].clone()})
    got = fa.qk_norm_rope(y["q"], y["k"], y["wq"], y["wk"], y["cos"], y["sin"], y["positions"], interleaved=inter)
    assert fa.attn_last_device_error() == 0
    c, s = ref.angles(x["cos"], x["sin"], x["positions"], (rot // 2,)) if rot else (None, None)
    for n, o in zip("qk", got):
        same_finiteness(o, ref.norm_rope(x[n], x["w" + n], c, s, rot, inter, 1e-6)[0], n)
    # the gradient: one output gradient that is not finite
    x = inputs(621, 9, 3, 2, d, rot, 1, None)
    c, s = ref.angles(x["cos"], x["sin"], x["positions"], (rot // 2,)) if rot else (None, None)
    x["gq"][5, 2, d - 4] = INF
    x["gk"][1, 0, d - 7] = NAN
    y = to(dev, x)
    got = fa.qk_norm_rope_backward(y["q"], y["k"], y["wq"], y["wk"], y["cos"], y["sin"], y["positions"], y["gq"], y["gk"],
                                   interleaved=inter)
    assert fa.attn_last_device_error() == 0
    for i, n in enumerate("qk"):
        dx, dw, _, _ = ref.norm_rope_backward(x[n], x["w" + n], x["g" + n], c, s, rot, inter, 1e-6)
        same_finiteness(got[i], dx, n)
        same_finiteness(got[2 + i], dw, n)
        assert (~dw.isfinite()).sum() == 1


PLANS = {  # offsets of three sequences with 3, 2 and 4 new tokens (9 packed rows): the sequences that stay sound
    "start": ([1, 3, 5, 9], [1, 2]),
    "negative start": ([-2, 3, 5, 9], [1, 2]),
    "past total": ([0, 3, 5, 10], [0, 1]),
    "far past total": ([0, 3, 5, 2**31 - 1], [0, 1]),
    "two past total": ([0, 3, 10, 12], [0]),
    "decreasing": ([0, 3, 2, 9], []),
    "decreasing over a sequence": ([0, 7, 2, 9], []),
    "falling back to the start": ([0, 3, 5, 0], []),
    "past total and back": ([0, 3, 40, 9], []),
}


@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("what", PLANS)
def test_offsets_that_are_no_batch(dev, what, codes):
    """Offsets that decrease place no token: nothing is written.  A first sequence that does not
    begin at 0 or one that ends past the packed rows is refused by itself."""
    lens, ns, H, d, page = [40, 50, 60], [3, 2, 4], 2, 64, 16
    offsets, sound = PLANS[what]
    start = [0, 3, 5]
    c = make(dev, 630, lens, H, d, page, codes)
    kv = normal(dev, 631, 9, 2 * H, d)
    table, cu = c["page_table"], torch.tensor(offsets, dtype=torch.int32, device=dev)
    fa.cache_write(kv[:, :H], kv[:, H:], c["k_cache"], c["v_cache"], table, torch.tensor(lens, dtype=torch.int32, device=dev),
                   cu, k_scale=c["k_scale"], v_scale=c["v_scale"])
    assert fa.attn_last_device_error() == -8
    k, v = rows_of(c)
    mine = torch.zeros(k.shape[0], dtype=torch.bool)
    for b in sound:
        at = ref.row_index(table.cpu(), page, b, torch.arange(lens[b] - ns[b], lens[b]))
        mine[at] = True
        for x, got in ((kv[:, :H], k), (kv[:, H:], v)):
            x = x[start[b]:start[b] + ns[b]].cpu()
            if codes:
                values, scale = ref.quantise(x)
                x = values * scale.double()[..., None]
            assert torch.equal(got[at], x.double()), b
    assert k[~mine].isnan().all() and v[~mine].isnan().all()
    # reading back: the same sequences, each from its first position on
    full = fill(dev, 632, lens, H, d, page, codes)
    out = [torch.full((9, H, d), 3.0, dtype=torch.bfloat16, device=dev) for _ in "kv"]
    ptr = lambda t: None if t is None else t.data_ptr()
    cache = fa.AttnPagedCache(*(ptr(full[n]) for n in ("k_cache", "v_cache", "k_scale", "v_scale", "page_table")),
                              full["page_table"].shape[1], full["k_cache"].shape[0], page, H, d)
    fa.attn_cache_read(cache, *out, cu, 3, 9)
    assert fa.attn_last_device_error() == -8
    for got, rows in zip(out, rows_of(full)):
        left = torch.ones(9, dtype=torch.bool)
        for b in sound:
            at = ref.row_index(full["page_table"].cpu(), page, b, torch.arange(ns[b]))
            assert torch.equal(got[start[b]:start[b] + ns[b]].cpu(), rows[at].to(torch.bfloat16))
            left[start[b]:start[b] + ns[b]] = False
        assert (got.cpu()[left] == 3).all()


@pytest.mark.parametrize("fall", [1, 700, 1299])
def test_offsets_that_fall_in_a_large_batch(dev, fall):
    """One decrease among 1300 sequences (more than a CTA looks at in one go), at either end or inside."""
    B, H, d, page = 1300, 1, 64, 16
    c = make(dev, 635, [3] * B, H, d, page, True)
    kv = normal(dev, 636, B, 2 * H, d)
    cu = torch.arange(B + 1, dtype=torch.int32, device=dev)
    lens = torch.full((B,), 3, dtype=torch.int32, device=dev)
    write = lambda: fa.cache_write(kv[:, :H], kv[:, H:], c["k_cache"], c["v_cache"], c["page_table"], lens, cu,
                                   k_scale=c["k_scale"], v_scale=c["v_scale"])
    cu[fall] += 2
    write()
    assert fa.attn_last_device_error() == -8
    assert rows_of(c)[0].isnan().all()
    cu[fall] -= 2
    write()
    assert fa.attn_last_device_error() == 0


@pytest.mark.parametrize("G", ROWS)
@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("what", PLANS)
def test_attention_of_offsets_that_are_no_batch(dev, what, codes, G):
    """As for the cache: reported, no row written of a sequence that does not begin at 0 or ends past
    the packed rows, none at all where the offsets decrease."""
    lens, ns, H, d = [200, 300, 50], [3, 2, 4], 2, 64
    offsets, sound = PLANS[what]
    start = [0, 3, 5]
    c = fill(dev, 640, lens, H, d, 16, codes)
    q = normal(dev, 641, 9, H * G, d)
    want, most = want_of(c, q, lens, ns, None), heaviest_of(c, q, lens, ns, None)
    lens_d, cu = torch.tensor(lens, dtype=torch.int32, device=dev), torch.tensor(offsets, dtype=torch.int32, device=dev)
    which = torch.zeros(9, H * G, dtype=torch.bool)
    for b in sound:
        which[start[b]:start[b] + ns[b]] = True
    for splits in (0, 1):
        out = torch.full((9, H * G, d), 7.0, dtype=torch.bfloat16, device=dev)
        lse = torch.full((9, H * G), 7.0, device=dev)
        fa.tree_decode(q, c["k_cache"], c["v_cache"], c["page_table"], lens_d, cu, 8, 300, k_scale=c["k_scale"],
                       v_scale=c["v_scale"], num_splits=splits, out=out, lse=lse)
        assert fa.attn_last_device_error() == -8
        near((out, lse), want, codes, which, most)
        assert (out.cpu()[~which] == 7).all() and (lse.cpu()[~which] == 7).all()


def test_attention_of_offsets_that_fall_in_a_large_batch(dev):
    B, H, d, page = 1300, 1, 64, 16
    c = fill(dev, 645, [3] * B, H, d, page, True)
    q = normal(dev, 646, B, 2, d)
    lens = torch.full((B,), 3, dtype=torch.int32, device=dev)
    for fall in (1, 700, 1299):
        cu = torch.arange(B + 1, dtype=torch.int32, device=dev)
        cu[fall] += 2
        out = torch.full((B, 2, d), 7.0, dtype=torch.bfloat16, device=dev)
        fa.tree_decode(q, c["k_cache"], c["v_cache"], c["page_table"], lens, cu, 3, 3, k_scale=c["k_scale"],
                       v_scale=c["v_scale"], out=out)
        assert fa.attn_last_device_error() == -8
        assert (out == 7).all()


@pytest.mark.parametrize("T", [0, 5])
@pytest.mark.parametrize("Hq,Hk", [(0, 3), (3, 0), (0, 0)])
def test_gradient_of_a_kind_without_heads(dev, T, Hq, Hk):
    """No rows, so the sum over them is 0: its weight gradient is written, not left as it was."""
    d = 64
    x = inputs(650, T, Hq, Hk, d, d, 1, None)
    y = to(dev, {**x, "q": x["q"].clone(), "k": x["k"].clone()})
    dq, dk, dwq, dwk = fa.qk_norm_rope_backward(y["q"], y["k"], y["wq"], y["wk"], y["cos"], y["sin"], y["positions"],
                                                y["gq"], y["gk"])
    assert dq.shape == (T, Hq, d) and dk.shape == (T, Hk, d)
    dws = [torch.full((d,), 7.0, device=dev) for _ in "qk"]
    rot = fa.AttnRotary(y["cos"].data_ptr(), y["sin"].data_ptr(), y["positions"].data_ptr(), y["cos"].shape[0], d, 1)
    ws = torch.empty(max(1, fa.attn_qk_norm_rope_bwd_workspace(T, Hq, Hk, d)), dtype=torch.uint8, device=dev)
    p = lambda t: t.data_ptr() or None
    fa.attn_qk_norm_rope_bwd(p(y["q"]), Hq * d, p(y["k"]), Hk * d, y["wq"], y["wk"], p(y["gq"]), Hq * d, p(y["gk"]), Hk * d,
                             p(dq), Hq * d, p(dk), Hk * d, *dws, T, Hq, Hk, d, 1e-6, rot, ws, ws.numel())
    assert fa.attn_last_device_error() == 0
    for H, w, got in ((Hq, dws[0], dwq), (Hk, dws[1], dwk)):
        assert torch.equal(w, got)
        assert (w == 0).all() if H * T == 0 else (w != 7).all()


@pytest.mark.parametrize("G", ROWS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("up", [40, 90])
def test_large_values_of_hidden_tokens(dev, codes, d, G, up):
    """A drafted token whose values are 2^40 or 2^90 times the others' does not cost the rows that do
    not see it a bit, nor do they cost the row that does."""
    lens, ns, H = [200, 131, 64], [6, 6, 6], 2
    c = make(dev, 660, lens, H, d, 16, codes)
    kv = normal(dev, 661, sum(lens), 2 * H, d)
    ends = [sum(lens[:i + 1]) for i in range(3)]
    for end, j in zip(ends, (1, 3, 5)):
        kv[end - 6 + j, H:] *= 2.0 ** up
    put(dev, c, kv[:, :H], kv[:, H:], lens, lens)
    q = normal(dev, 662, 18, H * G, d)
    mask = torch.tensor([1 | 1 << i for _ in ns for i in range(6)], dtype=torch.int64)
    want, most = want_of(c, q, lens, ns, mask), heaviest_of(c, q, lens, ns, mask)
    for splits in (0, 1, 2):
        got = call(dev, c, q, lens, ns, mask, num_splits=splits)
        assert fa.attn_last_device_error() == 0
        near(got, want, codes, torch.ones(18, H * G, dtype=torch.bool), most)


@pytest.mark.parametrize("G", ROWS)
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("sink", [0, 130, 290, 399])
@pytest.mark.parametrize("splits", [0, 1])
def test_small_values_that_take_the_weight(dev, codes, G, sink, splits):
    """One token takes the weight (the others e^-80 and less) and its values are 2^-45 of the others':
    O is those values, to their own size."""
    L, ns, H, d = 400, [6], 1, 128
    c = make(dev, 670, [L], H, d, 16, codes)
    kv = normal(dev, 671, L, 2, d)
    kv[:, 0] *= 0.25
    kv[sink, 0] = 100.0 / d ** 0.5
    kv[sink, 1] *= 2.0 ** -45
    put(dev, c, kv[:, :1], kv[:, 1:], [L], [L])
    q = torch.ones(6, H * G, d, dtype=torch.bfloat16, device=dev)
    mask = torch.full((6,), 63, dtype=torch.int64)
    got = call(dev, c, q, [L], ns, mask, num_splits=splits)
    assert fa.attn_last_device_error() == 0
    near(got, want_of(c, q, [L], ns, mask), codes, torch.ones(6, H * G, dtype=torch.bool),
         heaviest_of(c, q, [L], ns, mask))


@pytest.mark.parametrize("G", [3, 24, 40])
@pytest.mark.parametrize("d", [64, 128])
def test_value_scales_without_order(dev, d, G):
    """Value scales drawn from 2^-50 .. 2^50, scores that move the maximum often, tiles of one size
    between them: a row's frame moves both ways."""
    lens, ns, H = [1500, 700], [6, 6], 2
    c = make(dev, 680, lens, H, d, 32, True)
    g = torch.Generator().manual_seed(681)
    kv = normal(dev, 682, sum(lens), 2 * H, d)
    e = torch.randint(-50, 51, (sum(lens), 1, 1), generator=g).double()
    at = torch.arange(sum(lens)) // 128
    e[(at % 3 == 0)[:, None, None]] = 0.0  # every third stretch is of one size
    kv[:, H:] = (kv[:, H:].double() * torch.exp2(e).to(dev)).to(torch.bfloat16)
    put(dev, c, kv[:, :H], kv[:, H:], lens, lens)
    q = normal(dev, 683, 12, H * G, d, std=4.0)
    mask = torch.tensor([1 | 1 << i for _ in ns for i in range(6)], dtype=torch.int64)
    want, most = want_of(c, q, lens, ns, mask), heaviest_of(c, q, lens, ns, mask)
    for splits in (0, 1, 3):
        got = call(dev, c, q, lens, ns, mask, num_splits=splits)
        assert fa.attn_last_device_error() == 0
        near(got, want, True, torch.ones(12, H * G, dtype=torch.bool), most)


def test_streams_by_address(dev):
    """`stream` may be a torch stream or its address, the default stream's 0 among them."""
    x = inputs(690, 33, 4, 2, 64, 64, 1, None)
    y = to(dev, x)
    call_ = lambda **kw: fa.qk_norm_rope(y["q"], y["k"], y["wq"], y["wk"], y["cos"], y["sin"], y["positions"], **kw)
    want = call_()
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    for stream in (0, torch.cuda.current_stream(), torch.cuda.current_stream().cuda_stream, other, other.cuda_stream):
        got = call_(stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert fa.attn_last_device_error() == 0


def test_interleaved_without_a_truth_value(dev):
    """Its own error, not a result with an error behind it."""
    x = inputs(695, 3, 2, 1, 64, 64, 1, None)
    y = to(dev, x)
    with pytest.raises(RuntimeError, match="ambiguous"):
        fa.qk_norm_rope(y["q"], y["k"], y["wq"], y["wk"], y["cos"], y["sin"], y["positions"],
                        interleaved=torch.tensor([True, False]))
    assert fa.attn_last_device_error() == 0


@pytest.mark.parametrize("G", ROWS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("splits", [0, 1])
def test_weights_that_are_rounded_add_up_to_one(dev, d, G, splits):
    """Keys that all hold the same values give back those values: the bf16 probabilities of a bf16 cache
    are divided by their own sum (few rows: are two bf16 each).  One key takes 0.98 of a row, against a running maximum that an earlier
    one has set (its weight is no power of two); the rounding of the others, 2^-8 of 0.02, stays under half
    a step of the result (2^-9 of it at least), so it is exact."""
    lens, ns, H = [700, 333], [6, 6], 2
    c = make(dev, 700, lens, H, d, 16, False)
    kv = normal(dev, 701, sum(lens), 2 * H, d, std=0.05)
    for first in (0, lens[0]):
        kv[first + 3, :H], kv[first + 300, :H] = 40.0 / d ** 0.5, 45.0 / d ** 0.5  # scores f 40 and f 45
    value = (1.99 * torch.exp2(torch.arange(d, device=dev) % 9 - 4.0)).to(torch.bfloat16)
    kv[:, H:] = value
    put(dev, c, kv[:, :H], kv[:, H:], lens, lens)
    g = torch.Generator().manual_seed(702)
    f = 0.82 + 0.18 * torch.rand(12, H * G, 1, generator=g)  # e^(-5 f) < 0.02, e^(-38 f) next to nothing
    q = f.expand(-1, -1, d).to(torch.bfloat16).to(dev).contiguous()
    o, lse = call(dev, c, q, lens, ns, None, num_splits=splits)
    assert fa.attn_last_device_error() == 0
    assert (o == value).all()


@pytest.mark.parametrize("d,G", [(64, 1), (64, 2), (128, 1)])
@pytest.mark.parametrize("splits", [0, 1])
def test_few_rows_lose_nothing_of_their_weights(dev, d, G, splits):
    """Up to 8 rows (16 at d = 64) over a bf16 cache take a probability as the sum of two bf16: 2^-8 of 2^-8
    of it is lost, so O is good to its own rounding and what scores and sums add."""
    lens, ns, H = [3000, 700, 65], [6, 6, 6], 2
    c = fill(dev, 710, lens, H, d, 32, False)
    q = normal(dev, 711, 18, H * G, d, std=1.5)
    o, lse = (t.cpu().double() for t in call(dev, c, q, lens, ns, None, num_splits=splits))
    assert fa.attn_last_device_error() == 0
    wo, wl, A, S = want_of(c, q, lens, ns, None)
    tol = 2.0 ** -8 * wo.abs() + A * (2.0 ** -16 + 2.0 ** -19 * S[..., None] + 2.0 ** -17)
    assert ((o - wo).abs() <= tol).all(), ((o - wo).abs() / tol).max()
