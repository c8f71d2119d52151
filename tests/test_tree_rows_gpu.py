"""Attention over the paged cache where its kernels differ: few query rows of a key
head, up to 128 of them, and more.  Six new tokens with 1, 2, 3, 24 or 40 query
heads to a key head are 6, 12, 18, 144 or 240 rows.

Tolerances as in test_tree_gpu.py.
"""
import math

import pytest

torch = pytest.importorskip("torch")

import io_aware_exact_06_gb300 as fa
from tests import serve_ref as ref
from tests.test_cache_gpu import cu_of, make, normal, put
from tests.test_tree_gpu import call, check, fill, random_masks, rows_of

pytestmark = pytest.mark.gpu

ROWS = [1, 2, 3, 24, 40]  # query heads to a key head


@pytest.fixture(scope="module")
def dev():
    import __graft_entry__
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    __graft_entry__.build()
    return torch.device("cuda:0")


@pytest.mark.parametrize("G", ROWS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("codes", [False, True])
def test_long_ragged_batches(dev, codes, d, G):
    """Many segments to a CTA, segments in many pieces, sequences of one key tile and less."""
    lens, ns, H = [3000, 1, 257, 128, 1500, 100], [2, 1, 6, 3, 2, 6], 2
    c = fill(dev, 400, lens, H, d, 32, codes)
    q = normal(dev, 402, sum(ns), H * G, d, std=1.5)
    mask = random_masks(403, ns)
    got = call(dev, c, q, lens, ns, mask, num_splits=0 if d == 128 else 1)
    assert fa.attn_last_device_error() == 0
    check(c, q, lens, ns, mask, got)


@pytest.mark.parametrize("G", ROWS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("codes", [False, True])
def test_hidden_keys(dev, codes, d, G):
    """Drafted tokens with NaN and infinite keys, values and scales reach only the rows that see them."""
    lens, ns, H = [200, 131], [6, 6], 2
    c = fill(dev, 410, lens, H, d, 16, codes)
    table = c["page_table"].cpu()
    bad = {(0, 1): "k", (0, 2): "v", (1, 3): "v", (1, 5): "k"}
    for (b, j), n in bad.items():
        row = int(ref.row_index(table, 16, b, torch.tensor(lens[b] - ns[b] + j)))
        page, at = row // 16, row % 16
        if codes:
            c[n + "_cache"].view(torch.uint8)[page, at, :, 5] = 0x7f
            c[n + "_scale"][page, :, at] = float("nan") if j % 2 else float("inf")
        else:
            c[n + "_cache"][page, at, :, 5] = float("nan") if j % 2 else float("inf")
    q = normal(dev, 413, 12, H * G, d)
    mask = torch.tensor([1 | 1 << i for _ in ns for i in range(6)], dtype=torch.int64)
    clean = [t for t in range(12) if (t // 6, t % 6) not in bad]
    for splits in (1, 3):
        o, lse = (t.cpu().double() for t in call(dev, c, q, lens, ns, mask, num_splits=splits))
        assert fa.attn_last_device_error() == 0
        k, v = rows_of(c)
        wo, wl, A, S = ref.tree(q.cpu(), k, v, table, 16, lens, [0, 6, 12], mask, d ** -0.5)
        assert wo[clean].isfinite().all()
        assert ((o[clean] - wo[clean]).abs() <= 2.0 ** -7 * (A[clean] + 0.01)).all()
        assert ((lse[clean] - wl[clean]).abs() <= 1e-4).all()
        for (b, j), n in bad.items():
            t = 6 * b + j
            if n == "k":
                assert o[t].isnan().all()
            else:
                assert not o[t, :, 5].isfinite().any()
                if not codes:
                    assert o[t, :, 6:].isfinite().all()


@pytest.mark.parametrize("G", ROWS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("up", [True, False])
def test_values_that_grow_and_shrink_along_a_sequence(dev, up, d, G):
    """Value scales that double every 16 tokens (2^40 in all), scores that grow along the way too."""
    L, ns, H = 640, [6], 1
    c = make(dev, 420, [L], H, d, 64, True)
    kv = normal(dev, 421, L, 2, d)
    e = torch.arange(L, device=dev) // 16
    e = (e if up else 39 - e).to(torch.float32) - 20
    kv[:, 1] = (kv[:, 1].float() * torch.exp2(e)[:, None]).to(torch.bfloat16)
    q = normal(dev, 422, 6, H * G, d)
    kv[:, 0] = (kv[:, 0].float() * (0.1 + torch.arange(L, device=dev)[:, None] / 300)).to(torch.bfloat16)
    put(dev, c, kv[:, :1], kv[:, 1:], [L], [L])
    for splits in (1, 4):
        got = call(dev, c, q, [L], ns, None, num_splits=splits)
        assert fa.attn_last_device_error() == 0
        check(c, q, [L], ns, None, got)


@pytest.mark.parametrize("G", ROWS)
@pytest.mark.parametrize("codes", [False, True])
def test_rows_without_keys_and_padding(dev, codes, G):
    """Rows that see nothing, a sequence without new tokens, rows behind the last sequence."""
    lens, ns, H, d = [6, 90, 140], [6, 0, 6], 2, 128
    c = fill(dev, 430, lens, H, d, 16, codes)
    q = normal(dev, 431, 20, H * G, d)
    mask = torch.tensor([0, 2, 0, 9, 0, 63] + [1, 0, 4, 0, 0, 32], dtype=torch.int64)
    empty = [0, 2, 4, 7, 9, 10]
    mask = torch.cat([mask, torch.full((8,), -1, dtype=torch.int64)])
    out = torch.full((20, H * G, d), 7.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((20, H * G), 7.0, device=dev)
    for splits in (0, 2):
        call(dev, c, q, lens, ns, mask, out=out, lse=lse, max_new=7, max_len=200, num_splits=splits)
        assert fa.attn_last_device_error() == 0
        check(c, q, lens, ns, mask[:12], (out, lse))
        assert (lse[[0, 2, 4]] == -math.inf).all() and (out[[0, 2, 4]] == 0).all()  # no context: no key at all
        assert lse[[t for t in empty if t >= 6]].isfinite().all()                   # the context is seen
        assert (out[12:] == 7).all() and (lse[12:] == 7).all()


@pytest.mark.parametrize("G", ROWS)
@pytest.mark.parametrize("what", ["page", "draft page", "short", "too many"])
def test_bad_plans(dev, what, G):
    lens, ns, H, d = [200, 300, 50], [2, 3, 6], 2, 128
    c = fill(dev, 440, lens, H, d, 16, True)
    q = normal(dev, 443, 11, H * G, d)
    good = call(dev, c, q, lens, ns, None)
    lens_d, table = torch.tensor(lens, dtype=torch.int32, device=dev), c["page_table"].clone()
    max_new, status, ruined = 6, -8, slice(2, 5)
    if what == "page":
        table[1, 2], status = table.new_tensor(c["k_cache"].shape[0]), -11
    elif what == "draft page":
        table[1, 18], status = 1 << 30, -11
    elif what == "short":
        lens_d[1] = 2
    else:
        max_new, ruined = 5, slice(5, 11)
    for splits in (1, 3):
        out = torch.full((11, H * G, d), 7.0, dtype=torch.bfloat16, device=dev)
        lse = torch.full((11, H * G), 7.0, device=dev)
        fa.tree_decode(q, c["k_cache"], c["v_cache"], table, lens_d, cu_of(dev, ns), max_new, 300,
                       k_scale=c["k_scale"], v_scale=c["v_scale"], num_splits=splits, out=out, lse=lse)
        assert fa.attn_last_device_error() == status
        if status == -11:
            assert out[ruined].isnan().all() and lse[ruined].isnan().all()
        else:
            assert (out[ruined] == 7).all() and (lse[ruined] == 7).all()
        others = [t for t in range(11) if not ruined.start <= t < ruined.stop]
        assert ((out[others].float() - good[0][others].float()).abs() <= 2.0 ** -7).all()
        assert ((lse[others] - good[1][others]).abs() <= 2.0 ** -14).all()
    assert fa.attn_last_device_error() == 0


@pytest.mark.parametrize("G", [3, 40])
def test_two_at_once_and_replayed(dev, G):
    """Two calls on two streams, and a captured one replayed beside them, give what each gives alone."""
    lens, ns, H, d = [3000, 700], [6, 6], 2, 128
    cs = [fill(dev, 450 + i, lens, H, d, 64, bool(i)) for i in range(2)]
    qs = [normal(dev, 452 + i, 12, H * G, d) for i in range(2)]
    want = [[t.clone() for t in call(dev, c, q, lens, ns, None)] for c, q in zip(cs, qs)]
    lens_d, cu = torch.tensor(lens, dtype=torch.int32, device=dev), cu_of(dev, ns)

    def run(i, out, lse):
        c = cs[i]
        fa.tree_decode(qs[i], c["k_cache"], c["v_cache"], c["page_table"], lens_d, cu, 6, 3000, k_scale=c["k_scale"],
                       v_scale=c["v_scale"], out=out, lse=lse)

    outs = [[(torch.empty_like(w[0]), torch.empty_like(w[1])) for _ in range(20)] for w in want]
    streams = [torch.cuda.Stream() for _ in range(3)]
    held = torch.empty_like(want[0][0]), torch.empty_like(want[0][1])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        run(0, *held)
    for n in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                run(i, *outs[i][n])
        with torch.cuda.stream(streams[2]):
            graph.replay()
    torch.cuda.synchronize()
    assert fa.attn_last_device_error() == 0
    for i in range(2):
        for o, lse in outs[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])
    assert torch.equal(held[0], want[0][0]) and torch.equal(held[1], want[0][1])
