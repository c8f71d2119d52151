"""The operators run together, as sampling with drafts uses them: prompts forked
into samples, their half-filled pages copied, drafts written and attended to over
the shared prefixes, verified, and the accepted ones moved together; on one
stream, on two at once, and captured into graphs."""
import pytest

torch = pytest.importorskip("torch")

import io_aware_exact_06_gb300 as fa
from tests import sample_ref
from tests.test_cache_gpu import cu_of, get, make, normal, put
from tests.test_tree_gpu import check, rows_of
from tests.test_verify_gpu import trees

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import __graft_entry__
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    __graft_entry__.build()
    return torch.device("cuda:0")


class Round:
    """Prompts of given lengths, samples of each, drafts of each sample."""

    def __init__(self, dev, seed, codes=True, d=128, prompts=(200, 77), samples=(5, 3), drafts=(7, 1, 12), Hq=8, H=2, page=16,
                 V=600):
        self.dev, self.codes, self.page, self.Hq, self.H = dev, codes, page, Hq, H
        self.prompts = list(prompts)
        B, N = len(prompts), sum(samples)
        self.ns = [drafts[i % len(drafts)] for i in range(N)]
        self.parents = [b for b, n in enumerate(samples) for _ in range(n)]
        self.lens = [prompts[b] + n for b, n in zip(self.parents, self.ns)]
        self.groups = [sum(samples[:b]) for b in range(B + 1)]
        spare = 3 + sum(-(-n // page) + 1 for n in self.lens)
        self.c = make(dev, seed, self.prompts, H, d, page, codes, spare=spare, width=max(self.lens) // page + 2)
        self.kv = normal(dev, seed + 1, sum(prompts), 2 * H, d)
        put(dev, self.c, self.kv[:, :H], self.kv[:, H:], self.prompts, self.prompts)
        pages = self.c["k_cache"].shape[0]
        refs = torch.zeros(pages, dtype=torch.int32)
        for b, n in enumerate(prompts):
            refs[self.c["page_table"][b, :-(-n // page)].cpu().long()] += 1
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
        self.refs, self.prompts_d, self.parents_d, self.lens_d = refs.to(dev), i32(self.prompts), i32(self.parents), i32(self.lens)
        self.groups_d, self.cu = i32(self.groups), cu_of(dev, self.ns)
        total = sum(self.ns)
        self.qkv = normal(dev, seed + 2, total, Hq + 2 * H, d)
        self.mask_cpu = trees(seed, self.ns, 3)
        self.mask = self.mask_cpu.to(dev)
        # a channel of the attention for each token of the vocabulary, in place of the rest of a model (a library's
        # product would share its workspace between graphs that are captured on one stream)
        self.channel = torch.arange(V, device=dev) % (Hq * d)
        self.bias = normal(dev, seed + 3, V).float()
        g = torch.Generator().manual_seed(seed)
        self.draft = (2.0 * torch.randn(total, V, generator=g)).softmax(-1).to(dev)
        self.tokens = torch.randint(0, V, (total,), generator=g, dtype=torch.int32).to(dev)
        self.u, self.u_next = torch.rand(total, generator=g).to(dev) ** 4, torch.rand(N, generator=g).to(dev)

    def run(self, stream=None):
        c, page = self.c, self.page
        s = dict(k_scale=c["k_scale"], v_scale=c["v_scale"], stream=stream)
        q, k, v = self.qkv.split([self.Hq, self.H, self.H], 1)
        table, refs, src, dst = fa.cache_fork(c["page_table"], self.prompts_d, self.parents_d, self.lens_d, self.refs, page, stream=stream)
        fa.cache_copy(c["k_cache"], c["v_cache"], src, dst, **s)
        fa.cache_write(k, v, c["k_cache"], c["v_cache"], table, self.lens_d, self.cu, **s)
        bounds = dict(max_new=max(self.ns), max_len=max(self.lens), max_prefix=max(self.prompts),
                      max_group=max(sum(self.ns[a:b]) for a, b in zip(self.groups, self.groups[1:])))
        o, lse = fa.prefix_decode(q, c["k_cache"], c["v_cache"], table, self.lens_d, self.cu, cu_groups=self.groups_d,
                                  prefix_lens=self.prompts_d, mask=self.mask, **bounds, **s)
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            probs = (4.0 * o.float().flatten(1)[:, self.channel] + self.bias).softmax(-1)
            k0, v0 = (t.clone() for t in fa.cache_read(c["k_cache"], c["v_cache"], table, self.all_cu(), sum(self.lens),
                                                       k_scale=c["k_scale"], v_scale=c["v_scale"]))
        path, kept, nxt, lens = fa.verify_drafts(self.tokens, probs, self.cu, self.u, self.u_next, draft_probs=self.draft,
                                                 mask=self.mask, seqlens=self.lens_d, stream=stream)
        fa.cache_compact(c["k_cache"], c["v_cache"], table, self.lens_d, self.cu, path, kept, **s)
        return q, o, lse, probs, table, refs, path, kept, nxt, lens, k0, v0

    def all_cu(self):
        if not hasattr(self, "_cu"):
            self._cu = cu_of(self.dev, self.lens)
        return self._cu


@pytest.mark.parametrize("codes,d,Hq", [(True, 128, 8), (False, 64, 2), (False, 128, 16)])
def test_a_round(dev, codes, d, Hq):
    r = Round(dev, 700, codes, d, Hq=Hq)
    q, o, lse, probs, table, refs, path, kept, nxt, lens, k0, v0 = r.run()
    assert fa.attn_last_device_error() == 0
    want = sample_ref.fork(r.c["page_table"].tolist(), r.prompts, r.parents, r.lens, r.refs.tolist(), r.page)
    assert table.tolist() == want[0] and refs.tolist() == want[1]
    # what the attention read: the forked prompt and the new tokens' own rows, before any of them moved
    total = sum(r.lens)
    at = 0
    prompt = torch.tensor(r.prompts).cumsum(0).tolist()
    back = get(dev, r.c, r.prompts)
    for i, (b, n) in enumerate(zip(r.parents, r.ns)):
        rows = slice(prompt[b] - r.prompts[b], prompt[b])
        if not codes:
            assert torch.equal(k0[at:at + r.prompts[b]], r.kv[rows, :r.H])
        else:
            assert torch.equal(k0[at:at + r.prompts[b]], back[0][rows])
        at += r.lens[i]
    # verification by the definition, on the probabilities that came out
    ns_cu = r.cu.tolist()
    wp, wk, wn, near = sample_ref.verify(r.tokens.cpu(), probs.cpu(), ns_cu, r.u.cpu(), r.u_next.cpu(), r.draft.cpu(), r.mask_cpu)
    assert near > 600 * 2.0 ** -43
    assert path.tolist() == wp and kept.tolist() == wk and nxt.tolist() == wn
    assert lens.tolist() == [L - n + a for L, n, a in zip(r.lens, r.ns, wk)] and max(wk) > 1
    # the cache as the sequences go on with it
    c = dict(r.c, page_table=table)
    k, v = get(dev, c, lens.tolist())
    at, to = 0, 0
    for i, n in enumerate(r.ns):
        base = r.lens[i] - n
        rows = list(range(base)) + [base + x for x in wp[ns_cu[i]:ns_cu[i] + wk[i]]]
        assert torch.equal(k[to:to + len(rows)], k0[at:at + r.lens[i]][rows]) and torch.equal(v[to:to + len(rows)], v0[at:at + r.lens[i]][rows])
        at, to = at + r.lens[i], to + len(rows)
    assert fa.attn_last_device_error() == 0


@pytest.mark.parametrize("codes,d,Hq", [(True, 128, 8), (False, 64, 2), (False, 128, 16)])
def test_the_attention_of_a_round(dev, codes, d, Hq):
    r = Round(dev, 710, codes, d, Hq=Hq)
    r.u.fill_(0.999999)  # nothing moves but what cannot be refused
    q, o, lse, probs, table, refs, path, kept, *_ = r.run()
    assert fa.attn_last_device_error() == 0
    if kept.max() > 1:  # put the rows back that the walk has moved
        qkv = r.qkv.split([r.Hq, r.H, r.H], 1)
        fa.cache_write(qkv[1], qkv[2], r.c["k_cache"], r.c["v_cache"], table, r.lens_d, r.cu, k_scale=r.c["k_scale"], v_scale=r.c["v_scale"])
    check(dict(r.c, page_table=table), q, r.lens, r.ns, r.mask_cpu, (o, lse))


def test_two_streams_at_once(dev):
    rounds = [Round(dev, 720 + 10 * i, codes=bool(i % 2), Hq=16) for i in range(2)]
    want = [[t.clone() for t in r.run()] for r in rounds]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in rounds]
    got = [[] for _ in rounds]
    for _ in range(20):
        for i, r in enumerate(rounds):
            got[i].append(r.run(streams[i]))
    torch.cuda.synchronize()
    assert all(fa.attn_last_device_error(s) == 0 for s in streams)
    for i in range(2):
        for out in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(out, want[i]))


def test_graphs_that_replay_at_the_same_time(dev):
    rounds = [Round(dev, 740 + 10 * i, Hq=16 * (i + 1)) for i in range(2)]
    want = [[t.clone() for t in r.run()] for r in rounds]
    graphs, outs = [], []
    cap = torch.cuda.Stream()
    for r in rounds:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=cap):
            outs.append(r.run())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in rounds]
    for _ in range(10):
        for o in outs:
            for t in o[1:]:
                t.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(o, w))
    # another plan through the same graph: it is read on the device
    r = rounds[0]
    r.prompts_d -= 3
    r.lens_d -= 3
    r.all_cu().copy_(torch.tensor([sum(x - 3 for x in r.lens[:i]) for i in range(len(r.lens) + 1)], dtype=torch.int32))
    graphs[0].replay()
    torch.cuda.synchronize()
    again = r.run()
    # (cache_read leaves the rows behind the last sequence as they were)
    rows = sum(r.lens) - 3 * len(r.lens)
    assert all(torch.equal(a[:rows] if i >= 10 else a, b[:rows] if i >= 10 else b) for i, (a, b) in enumerate(zip(outs[0], again)))
    assert fa.attn_last_device_error() == 0


def test_streams_by_address(dev):
    r = Round(dev, 760)
    want = r.run()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = fa.prefix_decode(want[0], r.c["k_cache"], r.c["v_cache"], want[4], r.lens_d, r.cu, max(r.ns), max(r.lens), r.groups_d,
                           r.prompts_d, 64, 200, mask=r.mask, k_scale=r.c["k_scale"], v_scale=r.c["v_scale"], stream=s.cuda_stream)
    fork = fa.cache_fork(r.c["page_table"], r.prompts_d, r.parents_d, r.lens_d, r.refs, r.page, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(fork[0], want[4]) and got[0].shape == want[1].shape
    assert fa.attn_last_device_error(s) == 0


FIRST = """
    import sys, torch
    sys.path.insert(0, "@ROOT@")
    import io_aware_exact_06_gb300 as fa
    dev = torch.device("cuda:0")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)
    table, lens, parents, new, refs = i32(0, 1, 2, -1).view(1, 4), i32(40), i32(0, 0), i32(41, 42), i32(1, 1, 1, 0, 0)
    kc, vc = torch.randn(2, 5, 16, 1, 64, device=dev).bfloat16()
    q = torch.randn(2, 4, 64, device=dev).bfloat16()
    probs = torch.full((2, 50), 0.02, device=dev)
    cu, groups, prefix, u = i32(0, 1, 2), i32(0, 2), i32(40), torch.rand(2, device=dev)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        t, r, src, dst = fa.cache_fork(table, lens, parents, new, refs, 16)
        fa.cache_copy(kc, vc, src, dst)
        o, lse = fa.prefix_decode(q, kc, vc, t, new, cu, 1, 42, groups, prefix, 2, 40)
        path, kept, nxt, left = fa.verify_drafts(torch.zeros(2, dtype=torch.int32, device=dev), probs, cu, u, u, seqlens=new)
        fa.cache_compact(kc, vc, t, new, cu, path, kept)
    g.replay()
    torch.cuda.synchronize()
    assert fa.attn_last_device_error() == 0
    assert t.tolist() == [[0, 1, 2, -1], [0, 1, 3, -1]] and r.tolist() == [2, 2, 1, 1, 0] and kept.tolist() == [1, 1]
    for b, n in enumerate((41, 42)):
        rows = t[b].long()[torch.arange(n, device=dev) // 16], torch.arange(n, device=dev) % 16
        k, v = kc[rows][:, 0].double(), vc[rows][:, 0].double()
        p = (q[b].double() @ k.T / 8).softmax(-1)
        assert (o[b].double() - p @ v).abs().max() < 0.03
    print("ok")
"""


def test_first_calls_of_a_process_inside_a_capture(dev):
    import os
    import subprocess
    import sys
    import textwrap
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    script = textwrap.dedent(FIRST).replace("@ROOT@", root)
    out = subprocess.run([sys.executable, "-c", script], capture_output=True, text=True, timeout=600)
    assert out.returncode == 0 and "ok" in out.stdout, out.stderr[-2000:]


@pytest.mark.parametrize("codes,d,Hq", [(True, 128, 8), (False, 64, 2), (False, 128, 16)])
def test_attention_on_a_stream_by_address_is_the_same(dev, codes, d, Hq):
    r = Round(dev, 770, codes, d, Hq=Hq)
    q, table = (r.run()[i] for i in (0, 4))  # accepted rows have moved since: the cache as it is now
    s = torch.cuda.Stream()
    run = lambda **kw: fa.prefix_decode(q, r.c["k_cache"], r.c["v_cache"], table, r.lens_d, r.cu, max(r.ns), max(r.lens), r.groups_d,
                                        r.prompts_d, 64, 200, mask=r.mask, k_scale=r.c["k_scale"], v_scale=r.c["v_scale"], **kw)
    want = run()
    torch.cuda.synchronize()
    out, lse = torch.full_like(want[0], 7.0), torch.full_like(want[1], 7.0)
    torch.cuda.synchronize()
    got = run(out=out, lse=lse, stream=s.cuda_stream)
    s.synchronize()
    assert got[0].data_ptr() == out.data_ptr() and torch.equal(out, want[0]) and torch.equal(lse, want[1])
    check(r.c | {"page_table": table}, q, r.lens, r.ns, r.mask_cpu, (out, lse))
    assert fa.attn_last_device_error(s) == 0
