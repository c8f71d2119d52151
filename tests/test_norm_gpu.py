"""The per-head norm with rotation and its gradient against fp64.

Tolerances, from the arithmetic (fp32 inside, one rounding to bf16, off by at
most 2^-8 of the value):
  - an output is two products of normed channels a, b: the mean of squares adds
    at most 2^-24 (7 + 4) relative (seven adds a lane, four shuffles), halved by
    the square root, rsqrt 2^-22, five products and sums 2^-24 each: below
    2^-20 (|a| + |b|);
  - dx likewise, with the row sum of g w x (2^-20 of its magnitudes);
  - dw adds fp32 terms good to 2^-20 of their magnitude through a chain of at
    most n + 80 additions (n a lane's rows; then shuffles, 8 warps, up to 10
    partial rows, 32 slices): 2^-24 (n + 80) of the sum of magnitudes.
"""
import pytest

torch = pytest.importorskip("torch")

import io_aware_exact_06_gb300 as fa
from tests import serve_ref as ref

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def dev():
    import __graft_entry__
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    __graft_entry__.build()
    return torch.device("cuda:0")


def tables(P, rot):
    half = rot // 2
    a = torch.arange(P, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))
    return a.cos().float(), a.sin().float()


def inputs(seed, T, Hq, Hk, d, rot, axes, sections, P=977, gap=0, std=1.3):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: (torch.randn(*s, generator=g) * std).to(torch.bfloat16)
    fused = n(T, Hq + Hk + gap, d)
    x = {"q": fused[:, :Hq], "k": fused[:, Hq:Hq + Hk], "wq": n(d), "wk": n(d),
         "gq": n(T, Hq, d), "gk": n(T, Hk, d),
         "positions": torch.randint(0, P, (axes, T), generator=g, dtype=torch.int32)}
    x["cos"], x["sin"] = tables(P, rot)
    x["sections"] = sections or (rot // 2,)
    return x


def to(dev, x):
    """On the device; q and k stay slices of one tensor (token stride > heads * d)."""
    y = {n: v.to(dev) if torch.is_tensor(v) and n not in "qk" else v for n, v in x.items()}
    base = x["q"]._base.to(dev) if x["q"]._base is not None else None
    if base is None:
        y["q"], y["k"] = x["q"].to(dev), x["k"].to(dev)
    else:
        Hq, Hk = x["q"].shape[1], x["k"].shape[1]
        y["q"], y["k"] = base[:, :Hq], base[:, Hq:Hq + Hk]
    return y


def forward(y, inter, **kw):
    return fa.qk_norm_rope(y["q"], y["k"], y["wq"], y["wk"], y["cos"], y["sin"], y["positions"], eps=EPS,
                           sections=y["sections"], interleaved=inter, **kw)


def check_forward(x, got, rot, inter):
    c, s = ref.angles(x["cos"], x["sin"], x["positions"], x["sections"]) if rot else (None, None)
    for n, o in zip("qk", got):
        want, mag = ref.norm_rope(x[n], x["w" + n], c, s, rot, inter, EPS)
        off = (o.cpu().double() - want).abs()
        assert (off <= 2 ** -8 * want.abs() + 2 ** -20 * mag).all(), (n, (off - 2 ** -8 * want.abs()).max())


CASES = [  # T, Hq, Hk, d, rot, axes, sections, interleaved, gap
    (1, 1, 1, 64, 64, 1, None, False, 0),
    (1, 32, 8, 128, 128, 1, None, False, 8),
    (3, 5, 3, 128, 128, 1, None, True, 1),
    (257, 7, 1, 64, 32, 1, None, False, 3),
    (33, 9, 2, 64, 48, 1, None, True, 0),
    (65, 16, 16, 128, 16, 1, None, False, 0),
    (40, 3, 17, 128, 112, 1, None, False, 2),
    (129, 4, 4, 128, 128, 3, (16, 24, 24), False, 4),
    (50, 4, 2, 128, 128, 3, (5, 30, 29), False, 0),   # axes that end inside a lane's pairs
    (50, 4, 2, 64, 64, 3, (3, 0, 29), True, 0),
    (21, 6, 2, 64, 64, 2, (13, 19), False, 0),
    (5, 2, 2, 64, 0, 1, None, False, 0),              # the norm alone
    (700, 12, 4, 64, 64, 1, None, False, 4),
]


@pytest.mark.parametrize("T,Hq,Hk,d,rot,axes,sections,inter,gap", CASES)
def test_forward(dev, T, Hq, Hk, d, rot, axes, sections, inter, gap):
    x = inputs(T * 131 + d, T, Hq, Hk, d, rot, axes, sections, gap=gap)
    got = forward(to(dev, x), inter)
    assert fa.attn_last_device_error() == 0
    check_forward(x, got, rot, inter)


@pytest.mark.parametrize("T,Hq,Hk,d,rot,axes,sections,inter,gap", CASES)
def test_gradient(dev, T, Hq, Hk, d, rot, axes, sections, inter, gap):
    x = inputs(T * 37 + d, T, Hq, Hk, d, rot, axes, sections, gap=gap)
    y = to(dev, x)
    call = lambda: fa.qk_norm_rope_backward(y["q"], y["k"], y["wq"], y["wk"], y["cos"], y["sin"], y["positions"],
                                            y["gq"], y["gk"], eps=EPS, sections=y["sections"], interleaved=inter)
    got = call()
    assert fa.attn_last_device_error() == 0
    c, s = ref.angles(x["cos"], x["sin"], x["positions"], x["sections"]) if rot else (None, None)
    for i, n in enumerate("qk"):
        dx, dw, dx_mag, dw_mag = ref.norm_rope_backward(x[n], x["w" + n], x["g" + n], c, s, rot, inter, EPS)
        off = (got[i].cpu().double() - dx).abs()
        assert (off <= 2 ** -8 * dx.abs() + 2 ** -19 * dx_mag).all(), n
        off = (got[2 + i].cpu().double() - dw).abs()
        rows = T * x[n].shape[1]
        assert (off <= (2 ** -20 + 2 ** -24 * (min(rows, 4 * (1 + rows // 2432)) + 80)) * dw_mag).all(), n
    again = call()  # fixed order of sums: the same bits
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_gradient_against_differences(dev):
    """The fp64 forward's central differences of sum(out * g), at every channel of
    one row and of the weights: step h = 2^-10, so the cubic term adds about
    h^2 = 2^-20 relative to the gradient's magnitudes."""
    T, Hq, Hk, d, rot, inter = 3, 2, 1, 64, 48, False
    x = inputs(5, T, Hq, Hk, d, rot, 1, None)
    y = to(dev, x)
    got = fa.qk_norm_rope_backward(y["q"], y["k"], y["wq"], y["wk"], y["cos"], y["sin"], y["positions"], y["gq"],
                                   y["gk"], eps=EPS, sections=y["sections"], interleaved=inter)
    c, s = ref.angles(x["cos"], x["sin"], x["positions"], x["sections"])
    loss = lambda q, w: (ref.norm_rope(q, w, c, s, rot, inter, EPS)[0] * x["gq"].double()).sum()
    q, w, h = x["q"].double().clone(), x["wq"].double().clone(), 2.0 ** -10
    _, _, dx_mag, dw_mag = ref.norm_rope_backward(x["q"], x["wq"], x["gq"], c, s, rot, inter, EPS)
    for ch in range(d):
        e = torch.zeros_like(q)
        e[1, 1, ch] = h
        diff = (loss(q + e, w) - loss(q - e, w)) / (2 * h)
        assert abs(got[0][1, 1, ch].item() - diff) <= 2 ** -8 * abs(diff) + 2 ** -16 * dx_mag[1, 1].max()
        e = torch.zeros_like(w)
        e[ch] = h
        diff = (loss(q, w + e) - loss(q, w - e)) / (2 * h)
        assert abs(got[2][ch].item() - diff) <= 2 ** -17 * dw_mag[ch]


def test_in_place_and_given_outputs(dev):
    x = inputs(9, 77, 6, 3, 128, 128, 1, None, gap=3)
    y = to(dev, x)
    want = forward(y, False)
    room = torch.full((77, 20, 128), 9.0, dtype=torch.bfloat16, device=dev)
    got = forward(y, False, q_out=room[:, 2:8], k_out=room[:, 10:13])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert (room[:, :2] == 9).all() and (room[:, 8:10] == 9).all() and (room[:, 13:] == 9).all()
    rest = y["q"]._base[:, 9:].clone()
    got = forward(y, False, q_out=y["q"], k_out=y["k"])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(y["q"]._base[:, 9:], rest)


def test_no_tokens_and_no_heads(dev):
    x = inputs(10, 4, 3, 2, 64, 64, 1, None)
    y = to(dev, x)
    none = {**y, "q": y["q"][:0], "k": y["k"][:0], "positions": y["positions"][:, :0].contiguous()}
    assert forward(none, False)[0].shape == (0, 3, 64)
    dq, dk, dwq, dwk = fa.qk_norm_rope_backward(none["q"], none["k"], y["wq"], y["wk"], y["cos"], y["sin"],
                                                none["positions"], y["gq"][:0], y["gk"][:0])
    assert (dwq == 0).all() and (dwk == 0).all() and dq.numel() == dk.numel() == 0
    got = forward({**y, "k": y["k"][:, :0]}, False)  # queries alone
    assert torch.equal(got[0], forward(y, False)[0]) and got[1].shape == (4, 0, 64)
    assert fa.attn_last_device_error() == 0


def test_extreme_rows(dev):
    """Zero rows, the smallest and large channels, one infinity and one NaN: each stays in its row."""
    x = inputs(11, 6, 2, 2, 64, 64, 1, None)
    q = x["q"].clone()
    q[0] = 0
    q[1] *= 2.0 ** -60
    q[2] *= 2.0 ** 40
    q[3, 0, 5] = float("nan")
    q[4, 1, 9] = float("inf")
    x = {**x, "q": q, "k": x["k"].clone()}
    got = forward(to(dev, x), False)
    assert (got[0][0] == 0).all()
    assert got[0][3, 0].isnan().all() and got[0][3, 1].isfinite().all()
    assert got[0][4, 1].isnan().any() and got[0][4, 0].isfinite().all()
    keep = [0, 1, 2, 5]
    sub = {**x, "q": q[keep], "k": x["k"][keep], "positions": x["positions"][:, keep]}
    check_forward(sub, (got[0][keep], got[1][keep]), 64, False)


@pytest.mark.parametrize("bad", [-1, 977, 2**31 - 1, -2**31])
@pytest.mark.parametrize("axis", [0, 2])
def test_positions_outside_the_table(dev, bad, axis):
    """The token is reported and left alone, the others are right; it adds nothing to the weight gradients."""
    x = inputs(12, 30, 2, 1, 128, 128, 3, (20, 20, 24))
    y = to(dev, x)
    good = forward(y, False)
    y["positions"] = y["positions"].clone()
    y["positions"][axis, 7] = bad
    out = torch.full((30, 2, 128), 5.0, dtype=torch.bfloat16, device=dev)
    ko = torch.full((30, 1, 128), 5.0, dtype=torch.bfloat16, device=dev)
    forward(y, False, q_out=out, k_out=ko)
    assert fa.attn_last_device_error() == -11
    assert "position" in fa.attn_status_string(-11)
    others = [t for t in range(30) if t != 7]
    assert (out[7] == 5).all() and (ko[7] == 5).all()
    assert torch.equal(out[others], good[0][others]) and torch.equal(ko[others], good[1][others])
    args = (y["q"], y["k"], y["wq"], y["wk"], y["cos"], y["sin"])
    got = fa.qk_norm_rope_backward(*args, y["positions"], y["gq"], y["gk"], sections=y["sections"])
    assert fa.attn_last_device_error() == -11
    sub = {n: y[n][others] for n in ("q", "k", "gq", "gk")}
    c, s = ref.angles(x["cos"], x["sin"], x["positions"][:, others], x["sections"])
    for i, n in enumerate("qk"):
        _, dw, _, mag = ref.norm_rope_backward(sub[n].cpu(), x["w" + n], sub["g" + n].cpu(), c, s, 128, False, EPS)
        assert ((got[2 + i].cpu().double() - dw).abs() <= 2 ** -16 * mag).all()


@pytest.mark.parametrize("d", [64, 128])
def test_gradient_without_eps(dev, d):
    """eps = 0 and head counts that leave rows of a warp without a head: those are not rows of zeros."""
    T, Hq, Hk = 19, 5, 3
    x = inputs(77, T, Hq, Hk, d, d, 1, None)
    y = to(dev, x)
    got = fa.qk_norm_rope_backward(y["q"], y["k"], y["wq"], y["wk"], y["cos"], y["sin"], y["positions"], y["gq"],
                                   y["gk"], eps=0.0, sections=y["sections"], interleaved=False)
    assert fa.attn_last_device_error() == 0
    c, s = ref.angles(x["cos"], x["sin"], x["positions"], x["sections"])
    for i, n in enumerate("qk"):
        dx, dw, dx_mag, dw_mag = ref.norm_rope_backward(x[n], x["w" + n], x["g" + n], c, s, d, False, 0.0)
        assert ((got[i].cpu().double() - dx).abs() <= 2 ** -8 * dx.abs() + 2 ** -19 * dx_mag).all(), n
        rows = T * x[n].shape[1]
        assert ((got[2 + i].cpu().double() - dw).abs() <= (2 ** -20 + 2 ** -24 * (rows + 80)) * dw_mag).all(), n
