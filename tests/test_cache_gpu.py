"""Writing and reading the paged cache against its formula.

Codes and scales are whole: the formula's fp32 steps (one division, one
reciprocal, one product, one rounding to e4m3) are IEEE operations, so they must
match bit for bit; a read code is one product and one rounding to bf16."""
import pytest

torch = pytest.importorskip("torch")

import io_aware_exact_06_gb300 as fa
from tests import serve_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import __graft_entry__
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    __graft_entry__.build()
    return torch.device("cuda:0")


def make(dev, seed, lens, H, d, page, codes, spare=3, width=None):
    """An empty cache whose memory holds NaN patterns, and a shuffled page table."""
    g = torch.Generator().manual_seed(seed)
    per = [-(-n // page) for n in lens]
    pages = sum(per) + spare
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), width or max(per + [1])), -7, dtype=torch.int32)  # unused entries are never read
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    c = {"page_table": table.to(dev), "page": page}
    for n in "kv":
        if codes:
            c[n + "_cache"] = torch.full((pages, page, H, d), 0x7f, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)
            c[n + "_scale"] = torch.full((pages, H, page), float("nan"), device=dev)
        else:
            c[n + "_cache"] = torch.full((pages, page, H, d), float("nan"), dtype=torch.bfloat16, device=dev)
            c[n + "_scale"] = None
    return c


def cu_of(dev, ns):
    return torch.tensor([sum(ns[:i]) for i in range(len(ns) + 1)], dtype=torch.int32, device=dev)


def put(dev, c, k, v, lens, ns, **kw):
    fa.cache_write(k, v, c["k_cache"], c["v_cache"], c["page_table"], torch.tensor(lens, dtype=torch.int32, device=dev),
                   cu_of(dev, ns), k_scale=c["k_scale"], v_scale=c["v_scale"], **kw)


def get(dev, c, lens, total=None):
    return fa.cache_read(c["k_cache"], c["v_cache"], c["page_table"], cu_of(dev, lens), total or sum(lens),
                         k_scale=c["k_scale"], v_scale=c["v_scale"])


def normal(dev, seed, *shape, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16).to(dev)


CASES = [  # lengths, new tokens, H, d, page, codes
    ([1], [1], 1, 64, 16, True),
    ([5, 0, 33, 17], [1, 0, 1, 1], 8, 128, 16, True),
    ([100, 64, 1, 257], [37, 64, 1, 0], 3, 128, 32, True),
    ([300, 129], [300, 129], 5, 64, 64, True),
    ([513, 256, 255], [9, 256, 1], 2, 128, 256, False),
    ([77, 16, 15], [77, 16, 14], 4, 64, 16, False),
    ([40] * 70, [1] * 70, 1, 128, 128, True),          # more sequences than one probe
    ([3] * 1100, [1, 0] * 550, 1, 64, 16, True),       # more than two
]


@pytest.mark.parametrize("lens,ns,H,d,page,codes", CASES)
def test_write_then_read(dev, lens, ns, H, d, page, codes):
    c = make(dev, 40 + len(lens), lens, H, d, page, codes)
    before = {n: t.clone() for n, t in c.items() if torch.is_tensor(t)}
    total = sum(ns)
    fused = normal(dev, 41, total + 2, 2 * H + 1, d)  # slices with a token stride, and two rows of padding
    put(dev, c, fused[:, :H], fused[:, H:2 * H], lens, ns)
    assert fa.attn_last_device_error() == 0
    # where each token belongs, by the table
    table, at = c["page_table"].cpu(), []
    for b, (L, n) in enumerate(zip(lens, ns)):
        at.append(ref.row_index(table, page, b, torch.arange(L - n, L)))
    at = torch.cat(at)
    rest = torch.ones(c["k_cache"].shape[0] * page, dtype=torch.bool)
    rest[at] = False
    for n, x in (("k", fused[:total, :H]), ("v", fused[:total, H:2 * H])):
        rows = lambda t: t.view(torch.uint8).cpu().flatten(0, 1) if codes else t.view(torch.int16).cpu().flatten(0, 1)
        got, old = rows(c[n + "_cache"]), rows(before[n + "_cache"])
        assert torch.equal(got[rest], old[rest]), "rows of no new token"
        if not codes:
            assert torch.equal(got[at], x.contiguous().view(torch.int16).cpu())
            continue
        values, scale = ref.quantise(x.cpu())
        assert torch.equal(got[at].view(torch.float8_e4m3fn).double(), values)
        sc = c[n + "_scale"].cpu().transpose(1, 2).flatten(0, 1)
        assert torch.equal(sc[at], scale)
        assert sc[rest].isnan().all()
    if lens == ns:
        k, v = get(dev, c, lens)
        assert fa.attn_last_device_error() == 0
        for n, got, x in (("k", k, fused[:total, :H]), ("v", v, fused[:total, H:2 * H])):
            if codes:
                values, scale = ref.quantise(x.cpu())
                x = (values.float() * scale[..., None]).to(torch.bfloat16)
            assert torch.equal(got.cpu(), x.cpu())


@pytest.mark.parametrize("codes", [True, False])
def test_read_ragged_and_padded(dev, codes):
    """Lengths that end inside pages, an empty sequence, rows behind the last sequence untouched."""
    lens, H, d, page = [31, 0, 16, 100, 1], 3, 64, 16
    c = make(dev, 50, lens, H, d, page, codes)
    total = sum(lens)
    kv = normal(dev, 51, total, 2 * H, d)
    put(dev, c, kv[:, :H], kv[:, H:], lens, lens)
    k = torch.full((total + 9, H, d), 3.0, dtype=torch.bfloat16, device=dev)
    v = torch.full_like(k, 3.0)
    ptr = lambda t: None if t is None else t.data_ptr()
    cache = fa.AttnPagedCache(ptr(c["k_cache"]), ptr(c["v_cache"]), ptr(c["k_scale"]), ptr(c["v_scale"]),
                              ptr(c["page_table"]), c["page_table"].shape[1], c["k_cache"].shape[0], page, H, d)
    fa.attn_cache_read(cache, k, v, cu_of(dev, lens), len(lens), total + 9)
    assert fa.attn_last_device_error() == 0
    assert (k[total:] == 3).all() and (v[total:] == 3).all()
    a, b = get(dev, c, lens)
    assert torch.equal(k[:total], a) and torch.equal(v[:total], b)
    assert torch.equal(a, kv[:, :H]) if not codes else ((a - kv[:, :H]).abs() <= kv[:, :H].abs() / 16 + 0.02).all()


def test_special_rows(dev):
    """A zero row, tiny and huge rows, a NaN and an infinity."""
    H, d = 1, 64
    x = normal(dev, 60, 6, 1, 64)
    x[0] = 0
    x[1] = 2.0 ** -100
    x[2] *= 2.0 ** 100
    x[3, 0, 7] = float("nan")
    x[4, 0, 3] = float("inf")
    c = make(dev, 61, [6], H, d, 16, True)
    put(dev, c, x, x, [6], [6])
    k, _ = get(dev, c, [6])
    assert fa.attn_last_device_error() == 0
    assert (k[0] == 0).all() and (k[1] == 0).all()  # 2^-100 is below half a step of the scale floor
    values, scale = ref.quantise(x[[2, 5]].cpu())
    assert torch.equal(k[[2, 5]].cpu(), (values.float() * scale[..., None]).to(torch.bfloat16))
    assert k[3].isnan().any() and k[4].isnan().any()


def test_offsets_past_32_bits(dev):
    """Pages whose codes and bf16 rows lie more than 4 GB into the cache."""
    for codes, H, d, page, pages in ((True, 8, 128, 256, 17000), (False, 8, 128, 256, 9000)):
        c = make(dev, 70, [300], H, d, page, codes, spare=pages)
        c["page_table"] = torch.tensor([[pages - 1, pages]], dtype=torch.int32, device=dev)
        kv = normal(dev, 71, 300, 2 * H, d)
        put(dev, c, kv[:, :H], kv[:, H:], [300], [300])
        k, v = get(dev, c, [300])
        assert fa.attn_last_device_error() == 0
        assert c["k_cache"].numel() * c["k_cache"].element_size() > 1 << 32
        for got, x in ((k, kv[:, :H]), (v, kv[:, H:])):
            if codes:
                values, scale = ref.quantise(x.cpu())
                x = (values.float() * scale[..., None]).to(torch.bfloat16)
            assert torch.equal(got.cpu(), x.cpu())
        del c, k, v
        torch.cuda.empty_cache()


@pytest.mark.parametrize("what", ["page", "negative page", "short", "long", "decreasing", "start", "past total"])
def test_bad_plans_are_reported(dev, what):
    """Reported in the error word; the tokens of sound sequences are written, nothing else."""
    lens, ns, H, d, page = [40, 50, 60], [3, 2, 4], 2, 64, 16
    c = make(dev, 80, lens, H, d, page, True)
    kv = normal(dev, 81, 9, 2 * H, d)
    lens_d, cu = torch.tensor(lens, dtype=torch.int32, device=dev), cu_of(dev, ns)
    table = c["page_table"]
    status, sound = -8, [0, 2]
    if what == "page":
        table[1, 3], status = table.new_tensor(c["k_cache"].shape[0]), -11
    elif what == "negative page":
        table[1, 3], status = -1, -11
    elif what == "short":
        lens_d[1] = 1
    elif what == "long":
        lens_d[1] = 16 * table.shape[1] + 1
    elif what == "decreasing":
        cu[2], sound = 2, []
    elif what == "start":
        cu[0], sound = 1, [1, 2]
    else:
        cu[3], sound = 10, [0, 1]
    write = lambda: fa.cache_write(kv[:, :H], kv[:, H:], c["k_cache"], c["v_cache"], table, lens_d, cu,
                                   k_scale=c["k_scale"], v_scale=c["v_scale"])
    write()
    assert fa.attn_last_device_error() == status
    start = [0, 3, 5]
    values, _ = ref.quantise(kv[:, :H].cpu())
    flat = c["k_cache"].cpu().double().flatten(0, 1)
    mine = torch.zeros(flat.shape[0], dtype=torch.bool)
    for b in sound:
        at = ref.row_index(table.cpu(), page, b, torch.arange(lens[b] - ns[b], lens[b]))
        mine[at] = True
        assert torch.equal(flat[at], values[start[b]:start[b] + ns[b]]), b
    if what in ("page", "negative page", "short", "long"):
        assert flat[~mine].isnan().all()
    if what in ("page", "negative page"):
        k, _ = fa.cache_read(c["k_cache"], c["v_cache"], table, cu_of(dev, lens), sum(lens),
                             k_scale=c["k_scale"], v_scale=c["v_scale"])
        assert fa.attn_last_device_error() == -11
