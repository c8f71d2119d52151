"""Refusals of the norm, cache and tree calls that need no device: bad
arguments are turned down before anything touches the GPU, and the torch
conveniences check what the C calls cannot see."""
import ctypes

import pytest

import io_aware_exact_06_gb300 as fa
from io_aware_exact_06_gb300 import build

BUF = 1 << 20  # fake aligned addresses: validation fails before any use


@pytest.fixture(scope="module")
def lib():
    build.build()
    return fa.lib()


def rotary(**kw):
    a = dict(cos=BUF, sin=BUF, positions=BUF, table_len=128, rot=64, axes=1, section=(0, 0, 0), interleaved=0)
    a.update(kw)
    a["section"] = (ctypes.c_int * 3)(*a["section"])
    return fa.AttnRotary(*(a[n] for n, _ in fa.AttnRotary._fields_))


ROT = [(dict(rot=72), -2), (dict(rot=-16), -2), (dict(rot=256), -2), (dict(axes=0), -2), (dict(axes=4), -2),
       (dict(table_len=0), -2), (dict(axes=2, section=(16, 15, 0)), -2), (dict(axes=2, section=(-1, 33, 0)), -2),
       (dict(axes=3, section=(16, 16, 16)), -2), (dict(cos=None), -1), (dict(positions=None), -1),
       (dict(sin=BUF + 8), -4), (dict(positions=BUF + 2), -4)]
ARGS = [(dict(T=-1), -2), (dict(Hq=-1), -2), (dict(Hk=-2), -2), (dict(d=96), -3), (dict(eps=-1e-6), -5),
        (dict(eps=float("nan")), -5), (dict(q=None), -1), (dict(k=None), -1), (dict(q=BUF + 8), -4),
        (dict(k_stride=4 * 128 + 4), -4), (dict(q_stride=8 * 128 - 8), -2), (dict(wq=None), -1),
        (dict(wk=BUF + 8), -4), (dict(qo=None), -1), (dict(ko_stride=8), -2), (dict(Hq=9000), -2)]


def norm(lib, r, **kw):
    a = dict(q=BUF, q_stride=8 * 128, k=BUF, k_stride=4 * 128, wq=BUF, wk=BUF, qo=BUF, qo_stride=8 * 128, ko=BUF,
             ko_stride=4 * 128, T=5, Hq=8, Hk=4, d=128, eps=1e-6)
    a.update(kw)
    return lib.attn_qk_norm_rope(*a.values(), ctypes.addressof(r) if r else None, None)


@pytest.mark.parametrize("rot,status", ROT)
def test_rotary_refusals(lib, rot, status):
    assert norm(lib, rotary(**rot)) == status
    assert bwd(lib, rotary(**rot)) == status


@pytest.mark.parametrize("args,status", ARGS)
def test_norm_refusals(lib, args, status):
    assert norm(lib, rotary(), **args) == status


def test_norm_without_a_rotary_or_work(lib):
    assert norm(lib, None) == -1
    assert norm(lib, rotary(), T=0, q=None, k=None) == 0
    assert norm(lib, rotary(), Hq=0, Hk=0) == 0


def bwd(lib, r, **kw):
    a = dict(q=BUF, q_stride=8 * 128, k=BUF, k_stride=4 * 128, wq=BUF, wk=BUF, gq=BUF, gq_stride=8 * 128, gk=BUF,
             gk_stride=4 * 128, dq=BUF, dq_stride=8 * 128, dk=BUF, dk_stride=4 * 128, dwq=BUF, dwk=BUF, T=5, Hq=8,
             Hk=4, d=128, eps=1e-6)
    ws = dict(ws=BUF, bytes=1 << 20)
    ws.update({n: kw.pop(n) for n in list(kw) if n in ws})
    a.update(kw)
    return lib.attn_qk_norm_rope_bwd(*a.values(), ctypes.addressof(r), ws["ws"], ws["bytes"], None)


@pytest.mark.parametrize("args,status", [
    (dict(T=-1), -2), (dict(d=32), -3), (dict(eps=-1.0), -5), (dict(gq=None), -1), (dict(dk=None), -1),
    (dict(dwq=None), -1), (dict(dwk=BUF + 2), -4), (dict(dq=BUF + 8), -4), (dict(gk_stride=8), -2),
    (dict(dq_stride=8 * 128 + 4), -4), (dict(ws=None), -10), (dict(bytes=16), -10), (dict(ws=BUF + 8), -4),
])
def test_gradient_refusals(lib, args, status):
    assert bwd(lib, rotary(), **args) == status


def test_gradient_workspace_size():
    assert fa.attn_qk_norm_rope_bwd_workspace(1, 1, 1, 64) == 2 * 64 * 4
    big = fa.attn_qk_norm_rope_bwd_workspace(1 << 20, 64, 64, 128)
    assert big == fa.attn_qk_norm_rope_bwd_workspace(1 << 21, 64, 64, 128) <= 1 << 20
    assert fa.attn_qk_norm_rope_bwd_workspace(-1, 1, 1, 64) == 0


def cache(**kw):
    a = dict(k=BUF, v=BUF, k_scale=None, v_scale=None, page_table=BUF, page_table_stride=8, num_pages=100,
             page_size=16, H=4, d=128)
    a.update(kw)
    return fa.AttnPagedCache(*a.values())


CACHE = [(dict(d=80), -3), (dict(H=0), -2), (dict(num_pages=0), -2), (dict(page_size=8), -2), (dict(page_size=48), -2),
         (dict(page_size=512), -2), (dict(page_table_stride=0), -2), (dict(num_pages=1 << 28), -2),
         (dict(page_table_stride=1 << 28), -2), (dict(k=None), -1), (dict(page_table=None), -1),
         (dict(k_scale=BUF), -1), (dict(v_scale=BUF), -1), (dict(v=BUF + 8), -4), (dict(page_table=BUF + 2), -4),
         (dict(k_scale=BUF + 4, v_scale=BUF), -4)]


def write(lib, c, **kw):
    a = dict(k=BUF, ks=512, v=BUF, vs=512, lens=BUF, cu=BUF, B=2, total=10)
    a.update(kw)
    return lib.attn_cache_write(ctypes.addressof(c) if c else None, *a.values(), None)


def read(lib, c, **kw):
    a = dict(k=BUF, v=BUF, cu=BUF, B=2, total=10)
    a.update(kw)
    return lib.attn_cache_read(ctypes.addressof(c) if c else None, *a.values(), None)


def tree(lib, c, **kw):
    a = dict(q=BUF, qs=1024, lens=BUF, cu=BUF, mask=None, o=BUF, lse=BUF, B=2, total=10, Hq=8, max_new=8,
             max_len=128, scale=0.1, splits=0, ws=BUF, bytes=1 << 24)
    a.update(kw)
    return lib.attn_fwd_tree(a["q"], a["qs"], ctypes.addressof(c) if c else None,
                             *[a[n] for n in list(a)[2:]], None)


@pytest.mark.parametrize("args,status", CACHE)
def test_cache_refusals(lib, args, status):
    assert write(lib, cache(**args)) == status
    assert read(lib, cache(**args)) == status
    assert tree(lib, cache(**args)) == status


@pytest.mark.parametrize("args,status", [
    (dict(B=-1), -2), (dict(total=-1), -2), (dict(k=None), -1), (dict(ks=504), -2), (dict(vs=516), -4),
    (dict(lens=None), -1), (dict(cu=None), -1), (dict(cu=BUF + 2), -4), (dict(k=BUF + 8), -4)])
def test_write_refusals(lib, args, status):
    assert write(lib, cache(), **args) == status


@pytest.mark.parametrize("args,status", [
    (dict(B=-1), -2), (dict(total=-1), -2), (dict(v=None), -1), (dict(k=BUF + 8), -4), (dict(cu=None), -1)])
def test_read_refusals(lib, args, status):
    assert read(lib, cache(), **args) == status


@pytest.mark.parametrize("args,status", [
    (dict(B=-1), -2), (dict(Hq=6), -2), (dict(Hq=0), -2), (dict(max_new=65), -2), (dict(max_new=-1), -2),
    (dict(max_len=7), -2), (dict(max_len=2**31 - 1), -2), (dict(splits=257), -2), (dict(splits=-1), -2),
    (dict(scale=-0.1), -5), (dict(scale=float("inf")), -5), (dict(q=None), -1), (dict(o=None), -1),
    (dict(lens=None), -1), (dict(q=BUF + 8), -4), (dict(mask=BUF + 4), -4), (dict(lse=BUF + 2), -4),
    (dict(qs=1016), -2), (dict(qs=1028), -4), (dict(max_len=4096, splits=8, ws=None), -10),
    (dict(max_len=4096, splits=8, bytes=1024), -10)])
def test_tree_refusals(lib, args, status):
    assert tree(lib, cache(), **args) == status


def test_null_cache_and_empty_calls(lib):
    assert write(lib, None) == read(lib, None) == tree(lib, None) == -1
    assert write(lib, cache(), B=0) == read(lib, cache(), total=0, k=None) == 0
    assert tree(lib, cache(), B=0) == tree(lib, cache(), max_new=0) == tree(lib, cache(), total=0) == 0


def test_tree_workspace_size():
    """Bounded by the launch, not by the lengths; nothing for a call that is refused or has no work."""
    size = lambda *a: fa.attn_fwd_tree_workspace(*a)
    assert 0 < size(2, 10, 8, 4, 128, 8, 4096, 8) <= 64 << 20
    assert size(64, 64, 32, 8, 128, 1, 1 << 20, 0) == size(64, 64, 32, 8, 128, 1, 1 << 24, 0) <= 64 << 20
    assert size(2, 10, 7, 4, 128, 8, 4096, 8) == 0  # refused by the call itself
    assert size(0, 10, 8, 4, 128, 8, 4096, 0) == size(2, 10, 8, 4, 128, 0, 4096, 0) == 0


def test_convenience_refusals():
    """Types, shapes, strides and devices, on CPU tensors (refused before the library is called)."""
    torch = pytest.importorskip("torch")
    q, k = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    w, c, pos = torch.zeros(64, dtype=torch.bfloat16), torch.zeros(8, 32), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError):
        fa.qk_norm_rope(q.float(), k, w, w, c, c, pos)
    with pytest.raises(ValueError):  # not on a GPU
        fa.qk_norm_rope(q, k, w, w, c, c, pos)
    with pytest.raises(ValueError):
        fa.qk_norm_rope_backward(q, k, w, w, c, c, pos, q, k)
    kc = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    lens, cu, table = torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32)
    for call in (lambda **s: fa.cache_write(k, k, kc, kc, table, lens, cu, **s),
                 lambda **s: fa.cache_read(kc, kc, table, cu, 3, **s),
                 lambda **s: fa.tree_decode(q, kc, kc, table, lens, cu, 3, 16, **s)):
        with pytest.raises(ValueError):  # not on a GPU
            call()
        with pytest.raises(ValueError):  # one scale without the other
            call(k_scale=torch.zeros(2, 2, 16))
        with pytest.raises(TypeError):  # scales with a bf16 cache
            call(k_scale=torch.zeros(2, 2, 16), v_scale=torch.zeros(2, 2, 16))


def test_a_stream_of_another_device_is_refused():
    """The call would run on the tensors' device, on whatever stream is current there."""
    torch = pytest.importorskip("torch")
    from types import SimpleNamespace
    stream = SimpleNamespace(device=torch.device("cuda:1"), cuda_stream=0)
    k, kc = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    lens, cu, table = torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32)
    w, c, pos = torch.zeros(64, dtype=torch.bfloat16), torch.zeros(8, 32), torch.zeros(3, dtype=torch.int32)
    for call in (lambda: fa.qk_norm_rope(k, k, w, w, c, c, pos, stream=stream),
                 lambda: fa.qk_norm_rope_backward(k, k, w, w, c, c, pos, k, k, stream=stream),
                 lambda: fa.cache_write(k, k, kc, kc, table, lens, cu, stream=stream),
                 lambda: fa.cache_read(kc, kc, table, cu, 3, stream=stream),
                 lambda: fa.tree_decode(k, kc, kc, table, lens, cu, 3, 16, stream=stream)):
        with pytest.raises(ValueError, match="stream must be on"):
            call()
