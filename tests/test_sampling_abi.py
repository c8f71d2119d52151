"""Refusals of the shared-prefix, verification and page calls that need no device."""
import ctypes
from types import SimpleNamespace

import pytest

import io_aware_exact_06_gb300 as fa
from io_aware_exact_06_gb300 import build
from tests.test_serve_abi import BUF, CACHE, cache


@pytest.fixture(scope="module")
def lib():
    build.build()
    return fa.lib()


def at(c):
    return ctypes.addressof(c) if c else None


def prefix(lib, c, **kw):
    a = dict(q=BUF, qs=1024, cache=at(c), lens=BUF, cu=BUF, mask=None, cg=BUF, pl=BUF, o=BUF, lse=BUF, B=2, total=10, Hq=8,
             max_new=8, max_len=128, groups=1, max_group=10, max_prefix=100, scale=0.1, splits=0, ws=BUF, bytes=1 << 26)
    a.update(kw)
    return lib.attn_fwd_prefix(*a.values(), None)


def copy(lib, c, **kw):
    a = dict(src=BUF, dst=BUF, n=3)
    a.update(kw)
    return lib.attn_cache_copy(at(c), *a.values(), None)


def compact(lib, c, **kw):
    a = dict(lens=BUF, cu=BUF, path=BUF, kept=BUF, B=2, total=10)
    a.update(kw)
    return lib.attn_cache_compact(at(c), *a.values(), None)


def fork(lib, **kw):
    a = dict(table=BUF, W=8, lens=BUF, B=4, parents=BUF, new=BUF, N=6, refs=BUF, refs_out=BUF, pages=100, page=16, out=2 * BUF,
             src=BUF, dst=BUF, ws=BUF, bytes=1 << 20)
    a.update(kw)
    return lib.attn_cache_fork(*a.values(), None)


def verify(lib, **kw):
    a = dict(tokens=BUF, p=BUF, ps=1000, q=BUF, qs=1000, bf16=0, cu=BUF, mask=None, u=BUF, un=BUF, lens=BUF, path=BUF, kept=BUF,
             next=BUF, out=BUF, B=2, total=10, V=1000)
    a.update(kw)
    return lib.attn_verify_drafts(*a.values(), None)


@pytest.mark.parametrize("args,status", CACHE)
def test_cache_refusals(lib, args, status):
    assert prefix(lib, cache(**args)) == status
    assert compact(lib, cache(**args)) == status
    if not set(args) & {"page_table", "page_table_stride"}:
        assert copy(lib, cache(**args)) == status


@pytest.mark.parametrize("args,status", [
    (dict(B=-1), -2), (dict(Hq=6), -2), (dict(max_new=65), -2), (dict(max_len=7), -2), (dict(splits=257), -2),
    (dict(groups=-1), -2), (dict(max_group=-1), -2), (dict(max_prefix=-1), -2), (dict(max_prefix=129), -2),
    (dict(scale=-0.1), -5), (dict(scale=float("nan")), -5), (dict(q=None), -1), (dict(lse=None), -1), (dict(cu=None), -1),
    (dict(cg=None), -1), (dict(pl=None), -1), (dict(cg=BUF + 2), -4), (dict(pl=BUF + 1), -4), (dict(o=BUF + 8), -4),
    (dict(mask=BUF + 4), -4), (dict(qs=1016), -2), (dict(qs=1028), -4), (dict(ws=None), -10), (dict(bytes=4096), -10)])
def test_prefix_refusals(lib, args, status):
    assert prefix(lib, cache(), **args) == status


def test_prefix_workspace_size():
    size = lambda *a: fa.attn_fwd_prefix_workspace(*a)
    rows = 2 * 64 * 32 * 129 * 4  # of both lines, besides the pieces
    small = size(64, 64, 32, 8, 128, 1, 1 << 20, 1, 64, 1 << 18, 0)
    assert rows < small == size(64, 64, 32, 8, 128, 1, 1 << 24, 1, 64, 1 << 22, 0) <= rows + (96 << 20)
    assert size(2, 10, 7, 4, 128, 8, 4096, 1, 10, 100, 0) == size(0, 10, 8, 4, 128, 8, 4096, 1, 10, 100, 0) == 0
    assert size(2, 10, 8, 4, 128, 8, 4096, 0, 0, 0, 0) > 0


@pytest.mark.parametrize("args,status", [(dict(n=-1), -2), (dict(src=None), -1), (dict(dst=None), -1), (dict(src=BUF + 2), -4)])
def test_copy_refusals(lib, args, status):
    assert copy(lib, cache(), **args) == status


@pytest.mark.parametrize("args,status", [
    (dict(B=-1), -2), (dict(total=-1), -2), (dict(lens=None), -1), (dict(cu=None), -1), (dict(path=None), -1),
    (dict(kept=None), -1), (dict(path=BUF + 2), -4)])
def test_compact_refusals(lib, args, status):
    assert compact(lib, cache(), **args) == status


@pytest.mark.parametrize("args,status", [
    (dict(B=-1), -2), (dict(N=-1), -2), (dict(W=0), -2), (dict(pages=0), -2), (dict(page=24), -2), (dict(W=1 << 28), -2),
    (dict(pages=1 << 28), -2), (dict(N=1 << 28), -2), (dict(table=None), -1), (dict(lens=None), -1), (dict(parents=None), -1),
    (dict(new=None), -1), (dict(refs=None), -1), (dict(refs_out=None), -1), (dict(out=None), -1), (dict(src=None), -1),
    (dict(dst=None), -1), (dict(out=2 * BUF + 2), -4), (dict(refs=BUF + 1), -4), (dict(out=BUF), -2), (dict(out=BUF + 64), -2),
    (dict(out=BUF - 64), -2), (dict(ws=None), -10), (dict(bytes=100), -10)])
def test_fork_refusals(lib, args, status):
    assert fork(lib, **args) == status


@pytest.mark.parametrize("shift", [4, -4, 396, -396])
def test_fork_counts_that_overlap_are_refused(lib, shift):
    assert fork(lib, refs_out=BUF + shift) == -2


def test_fork_workspace_size():
    assert fa.attn_cache_fork_workspace(4, 6, 8, 100, 16) == 4 * (4 * 10 + 48)
    assert fa.attn_cache_fork_workspace(4, 6, 8, 10, 16) == 4 * (4 * 10 + 10)
    assert fa.attn_cache_fork_workspace(4, 6, 8, 100, 15) == 0


@pytest.mark.parametrize("args,status", [
    (dict(B=-1), -2), (dict(total=-1), -2), (dict(V=0), -2), (dict(V=262145, ps=262145, qs=262145), -2), (dict(ps=999), -2),
    (dict(qs=999), -2), (dict(tokens=None), -1), (dict(p=None), -1), (dict(cu=None), -1), (dict(u=None), -1), (dict(un=None), -1),
    (dict(path=None), -1), (dict(kept=None), -1), (dict(next=None), -1), (dict(lens=None), -1), (dict(out=None), -1),
    (dict(p=BUF + 2), -4), (dict(bf16=1, q=BUF + 1), -4), (dict(mask=BUF + 4), -4), (dict(tokens=BUF + 1), -4)])
def test_verify_refusals(lib, args, status):
    assert verify(lib, **args) == status


def test_null_cache_and_empty_calls(lib):
    assert prefix(lib, None) == copy(lib, None) == compact(lib, None) == -1
    assert prefix(lib, cache(), B=0) == prefix(lib, cache(), total=0, q=None) == prefix(lib, cache(), max_new=0) == 0
    assert copy(lib, cache(), n=0, src=None) == compact(lib, cache(), B=0) == compact(lib, cache(), total=0, path=None) == 0
    assert verify(lib, B=0, tokens=None) == 0


def test_status_string(lib):
    assert "free pages" in fa.attn_status_string(-12)


def tensors():
    torch = pytest.importorskip("torch")
    i = lambda *n: torch.zeros(*n, dtype=torch.int32)
    q, kc = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    calls = {
        "prefix": lambda **s: fa.prefix_decode(q, kc, kc, i(1, 1), i(1), i(2), 3, 16, i(2), i(1), 3, 16, **s),
        "copy": lambda **s: fa.cache_copy(kc, kc, i(2), i(2), **s),
        "compact": lambda **s: fa.cache_compact(kc, kc, i(1, 1), i(1), i(2), i(3), i(1), **s),
        "fork": lambda **s: fa.cache_fork(i(1, 1), i(1), i(2), i(2), i(5), 16, **s),
        "verify": lambda **s: fa.verify_drafts(i(3), torch.zeros(3, 8), i(2), torch.zeros(3), torch.zeros(1), **s)}
    return torch, calls


@pytest.mark.parametrize("name", ["prefix", "copy", "compact", "fork", "verify"])
def test_convenience_refusals(name):
    """Types, shapes and devices, on CPU tensors (refused before the library is called)."""
    torch, calls = tensors()
    call = calls[name]
    with pytest.raises(ValueError):  # not on a GPU
        call()
    with pytest.raises(ValueError, match="stream must be on"):  # a stream of another device
        call(stream=SimpleNamespace(device=torch.device("cuda:1"), cuda_stream=0))
    if name in ("prefix", "copy", "compact"):
        scale = torch.zeros(2, 2, 16)
        with pytest.raises(ValueError):  # one scale without the other
            call(k_scale=scale)
        with pytest.raises(TypeError):  # scales with a bf16 cache
            call(k_scale=scale, v_scale=scale)
    with pytest.raises(TypeError):
        if name == "verify":
            fa.verify_drafts(torch.zeros(3), torch.zeros(3, 8), None, None, None)
        elif name == "fork":
            fa.cache_fork(torch.zeros(1, 1), None, None, None, None, 16)
        else:
            fa.cache_copy(torch.zeros(2, 16, 2, 64), torch.zeros(2, 16, 2, 64), None, None)
