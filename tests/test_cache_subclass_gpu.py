"""The paged-cache calls on tensor subclasses, which the extension leaves to the Python wrappers:
the same results, in the same places, and the same errors."""
import pytest
import torch

from cache_common import DEV, make_cache, make_table
from gpu_common import load_fa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    return load_fa()


def _sub(*ts):
    return [torch.nn.Parameter(t, requires_grad=False) for t in ts]


def _cache(seed=1, num=60):
    """Codes, scales, a table with pages of their own for 30 more tokens each, lengths."""
    (kc, ks), (vc, vs) = (make_cache(num, 2, 16, 128, 8, seed + i, pow2=True) for i in range(2))
    lens = [300, 0, 37, 16]
    return [t.to(DEV) for t in (kc, vc, ks, vs, make_table([n + 30 for n in lens], 16, 24, num, seed),
                                torch.tensor(lens, dtype=torch.int32))]


def _rand(*shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(7)).to(torch.bfloat16).to(DEV)


@pytest.mark.parametrize("causal,Nq", [(False, 1), (True, 5)])
def test_decode(fa, causal, Nq):
    c, q = _cache(), _rand(4, 6, Nq, 128)
    expect = fa.decode_paged_fp8(q, *c, causal=causal, scale=0.1)
    got = fa.decode_paged_fp8(*_sub(q), *_sub(*c), causal=causal, scale=0.1)
    assert all(torch.equal(a, b) for a, b in zip(expect, got))
    out, lse = torch.empty_like(expect[0]), torch.empty_like(expect[1])
    ws = torch.empty(fa.fa_decode_paged_fp8_workspace_bytes(4, 6, 2, Nq, 128, 16, 24), dtype=torch.uint8,
                     device=DEV)
    o, _ = fa.decode_paged_fp8(*_sub(q), *c, causal=causal, scale=0.1, out=out, lse=lse, workspace=ws)
    assert o is out and torch.equal(out, expect[0]) and torch.equal(lse, expect[1])
    assert fa.fa_device_status(None) == 0


@pytest.mark.parametrize("offsets", [[0, 9, 9, 10, 30], None])
def test_append(fa, offsets):
    a, b = _cache(), _cache()
    T = 4 if offsets is None else 30
    kv = _rand(T, 5, 128)
    cu = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device=DEV)
    fa.append_paged_fp8(kv[:, :2], kv[:, 2:4], *a, cu_seqlens=cu)
    (sub,) = _sub(kv)
    fa.append_paged_fp8(sub[:, :2], sub[:, 2:4], *_sub(*b), cu_seqlens=None if cu is None else _sub(cu)[0])
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert fa.fa_device_status(None) == 0


def test_pages(fa):
    c = _cache()
    table, lens = c[4:]
    parents, fresh = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([2, 0, 2], [57, 58, 59]))
    for call, args in ((fa.free_pages, ()), (fa.fork_pages, (parents, fresh)), (fa.compact_pages, ())):
        expect = call(table, lens, *args, 16, 60)
        got = call(*_sub(table, lens), *_sub(*args), 16, 60)
        assert all(torch.equal(x, y) and x.shape == y.shape for x, y in zip(expect, got))
    _, _, src, dst = fa.fork_pages(table, lens, parents, fresh, 16, 60)
    a, b = _cache()[:4], _cache()[:4]
    fa.copy_pages(a, src, dst)
    fa.copy_pages(tuple(_sub(*b)), *_sub(src, dst))
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert fa.fa_device_status(None) == 0


def test_errors(fa):
    """Statuses of the C calls and refusals of the wrappers, from both paths."""
    c, q = _cache(), _rand(4, 6, 1, 128)
    small = torch.empty(16, dtype=torch.uint8, device=DEV)
    for f in (lambda *ts: list(ts), _sub):
        with pytest.raises(fa.FaError) as e:
            fa.decode_paged_fp8(*f(q), *f(*c), workspace=small)
        assert e.value.status == 6
        with pytest.raises(fa.FaError) as e:
            fa.decode_paged_fp8(*f(q), *f(*c), scale=-1.0)
        assert e.value.status == 1
        with pytest.raises(fa.FaError) as e:
            fa.free_pages(*f(*c[4:]), 16, (1 << 22) + 1)
        assert e.value.status == 2
        with pytest.raises(ValueError, match="dividing H"):
            fa.decode_paged_fp8(*f(_rand(4, 3, 1, 128)), *f(*c))
        with pytest.raises(ValueError, match="one row per sequence"):
            fa.append_paged_fp8(*f(_rand(3, 2, 128), _rand(3, 2, 128)), *f(*c))
