"""The operators run together, as a serving step and a training step use them:
in one stream, on two streams at once, captured into graphs that replay at the
same time, and as the process's first call inside a capture."""
import os
import subprocess
import sys
import textwrap

import pytest

torch = pytest.importorskip("torch")

import io_aware_exact_06_gb300 as fa
from tests import serve_ref as ref
from tests.test_cache_gpu import cu_of, make, normal, put
from tests.test_norm_gpu import EPS, tables
from tests.test_tree_gpu import check, random_masks

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def dev():
    import __graft_entry__
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    __graft_entry__.build()
    return torch.device("cuda:0")


FIRST = """
    import sys, torch
    sys.path.insert(0, "@ROOT@")
    import io_aware_exact_06_gb300 as fa
    dev = torch.device("cuda:0")
    x = torch.randn(9, 4, 64, device=dev).bfloat16()
    w = torch.ones(64, device=dev).bfloat16()
    cos, sin = torch.ones(16, 32, device=dev), torch.zeros(16, 32, device=dev)
    pos = torch.zeros(9, dtype=torch.int32, device=dev)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a, b = fa.qk_norm_rope(x, x, w, w, cos, sin, pos)
    g.replay()
    torch.cuda.synchronize()
    assert fa.attn_last_device_error() == 0
    want = x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)
    assert (a.float() - want).abs().max() < 0.02 and torch.equal(a, b)
    print("ok")
"""


class Step:
    """One serving step: norm and rotation of the new tokens' queries and keys,
    their keys and values written, attention over the cache."""

    def __init__(self, dev, seed, codes=True, d=128, lens=(300, 77, 1030), ns=(7, 1, 12), Hq=8, H=2):
        self.lens, self.ns, self.Hq, self.H, self.d = list(lens), list(ns), Hq, H, d
        total = sum(ns)
        self.c = make(dev, seed, self.lens, H, d, 32, codes)
        old = [L - n for L, n in zip(lens, ns)]
        kv = normal(dev, seed + 1, sum(old), 2 * H, d)
        put(dev, self.c, kv[:, :H], kv[:, H:], old, old)
        self.qkv = normal(dev, seed + 2, total, Hq + 2 * H, d)
        self.w = normal(dev, seed + 3, 2, d)
        cos, sin = tables(2048, d)
        self.cos, self.sin = cos.to(dev), sin.to(dev)
        self.pos = torch.cat([torch.arange(L - n, L) for L, n in zip(lens, ns)]).to(torch.int32).to(dev)
        self.lens_d, self.cu = torch.tensor(self.lens, dtype=torch.int32, device=dev), cu_of(dev, self.ns)
        self.mask = random_masks(seed, self.ns).to(dev)

    def run(self, stream=None):
        q, k, v = self.qkv.split([self.Hq, self.H, self.H], 1)
        q, k = fa.qk_norm_rope(q, k, self.w[0], self.w[1], self.cos, self.sin, self.pos, eps=EPS, stream=stream)
        c = self.c
        s = dict(k_scale=c["k_scale"], v_scale=c["v_scale"], stream=stream)
        fa.cache_write(k, v, c["k_cache"], c["v_cache"], c["page_table"], self.lens_d, self.cu, **s)
        o, lse = fa.tree_decode(q, c["k_cache"], c["v_cache"], c["page_table"], self.lens_d, self.cu, max(self.ns),
                                max(self.lens), mask=self.mask, **s)
        return q, o, lse


@pytest.mark.parametrize("codes,d", [(True, 128), (False, 64)])
def test_serving_step(dev, codes, d):
    st = Step(dev, 300, codes, d)
    q, o, lse = st.run()
    assert fa.attn_last_device_error() == 0
    check(st.c, q, st.lens, st.ns, st.mask.cpu(), (o, lse))
    # the prompt path over the same cache: read back, the last position's attention agrees with decode()
    k, v = fa.cache_read(st.c["k_cache"], st.c["v_cache"], st.c["page_table"], cu_of(dev, st.lens), sum(st.lens),
                         k_scale=st.c["k_scale"], v_scale=st.c["v_scale"])
    ends = torch.tensor(st.ns).cumsum(0) - 1
    full = torch.full((sum(st.ns),), -1, dtype=torch.int64, device=dev)
    c = st.c
    o2, _ = fa.tree_decode(q, c["k_cache"], c["v_cache"], c["page_table"], st.lens_d, st.cu, max(st.ns), max(st.lens),
                           mask=full, k_scale=c["k_scale"], v_scale=c["v_scale"])
    G = st.Hq // st.H
    last = q[ends.to(dev)].contiguous()
    o3, _ = fa.decode(last, k.repeat_interleave(G, 1), v.repeat_interleave(G, 1), cu_of(dev, st.lens), max(st.lens))
    assert fa.attn_last_device_error() == 0
    # read back values are rounded to bf16 (2^-8 of each v, 2^-8 of k in the score: |score| up to about 4)
    assert (o2[ends.to(dev)].float() - o3.float()).abs().max() <= 6 * 2.0 ** -8

def test_training_step(dev):
    """norm + rotation -> attention -> its gradient -> the norm's gradient, against fp64 through
    the same bf16 intermediate values; query heads share nothing here (the forward takes equal heads)."""
    T, H, d = 200, 3, 64
    x = normal(dev, 310, T, 3 * H, d)
    w = normal(dev, 311, 2, d)
    cos, sin = (t.to(dev) for t in tables(T, d))
    pos = torch.arange(T, dtype=torch.int32, device=dev)
    q0, k0, v = x.split(H, 1)
    q, k = fa.qk_norm_rope(q0, k0, w[0], w[1], cos, sin, pos)
    q4, k4, v4 = (t.reshape(1, T, H, d).contiguous() for t in (q, k, v))
    o, lse = fa.forward(q4, k4, v4, True)
    do = normal(dev, 312, 1, T, H, d)
    dq, dk, dv = fa.backward(q4, k4, v4, o, do, lse, True)
    got = fa.qk_norm_rope_backward(q0, k0, w[0], w[1], cos, sin, pos, dq[0], dk[0])
    assert fa.attn_last_device_error() == 0
    c, s = ref.angles(cos.cpu(), sin.cpu(), pos.cpu()[None], (d // 2,))
    for i, (a, wi, g) in enumerate(((q0, w[0], dq[0]), (k0, w[1], dk[0]))):
        dx, dw, mx, mw = ref.norm_rope_backward(a.cpu(), wi.cpu(), g.cpu(), c, s, d, False, 1e-6)
        assert ((got[i].cpu().double() - dx).abs() <= 2 ** -8 * dx.abs() + 2 ** -19 * mx).all()
        assert ((got[2 + i].cpu().double() - dw).abs() <= 2 ** -16 * mw).all()


def test_two_streams_at_once(dev):
    steps = [Step(dev, 320 + 10 * i, codes=bool(i % 2)) for i in range(2)]
    want = [[t.clone() for t in st.run()] for st in steps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    got = [[] for _ in steps]
    for _ in range(20):
        for i, st in enumerate(steps):
            got[i].append(st.run(streams[i]))  # named, not current: outputs belong to that stream
    torch.cuda.synchronize()
    assert all(fa.attn_last_device_error(s) == 0 for s in streams)
    for i in range(2):
        for out in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(out, want[i]))


def test_graphs_that_replay_at_the_same_time(dev):
    """Two graphs captured on one stream and replayed on two: nothing is shared."""
    steps = [Step(dev, 340 + 10 * i) for i in range(2)]
    want = [[t.clone() for t in st.run()] for st in steps]
    graphs, outs = [], []
    cap = torch.cuda.Stream()
    for st in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=cap):
            outs.append(st.run())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(10):
        for o in outs:
            for t in o:
                t.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(o, w))
    # other lengths through the same graph: the plan is read on the device
    st = steps[0]
    st.lens_d -= 2
    graphs[0].replay()
    torch.cuda.synchronize()
    again = st.run()
    assert all(torch.equal(a, b) for a, b in zip(outs[0], again))
    assert fa.attn_last_device_error() == 0


def test_gradient_captured(dev):
    T, H, d = 300, 4, 128
    q, k, gq, gk = (normal(dev, 360 + i, T, H, d) for i in range(4))
    w = normal(dev, 365, 2, d)
    cos, sin = (t.to(dev) for t in tables(T, d))
    pos = torch.arange(T, dtype=torch.int32, device=dev)
    run = lambda: fa.qk_norm_rope_backward(q, k, w[0], w[1], cos, sin, pos, gq, gk)
    want = run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    for _ in range(3):
        for t in out:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_first_call_of_a_process_inside_a_capture(dev):
    script = textwrap.dedent(FIRST).replace("@ROOT@", ROOT)
    out = subprocess.run([sys.executable, "-c", script], capture_output=True, text=True, timeout=600)
    assert out.returncode == 0 and "ok" in out.stdout, out.stderr[-2000:]
