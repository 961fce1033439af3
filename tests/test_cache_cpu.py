"""The paged e4m3 cache without a GPU: its oracle's pins, and every refusal of the entry
points (all of which return before anything touches CUDA)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import cache as oc
from oracle.fp8 import e4m3_value
from test_boundary_cpu import _on, fa  # noqa: F401

P = 0x10000  # aligned, never dereferenced


# ------------------------------------------------------------------------ pins

def test_least_scale():
    assert oc.least_scale(0.0) == 2.0 ** -126
    assert oc.least_scale(448.0) == 1.0 and oc.least_scale(448.1) == 2.0
    assert oc.least_scale(1.75) == 2.0 ** -8 and oc.least_scale(1.76) == 2.0 ** -7
    assert oc.least_scale(3.0e38) == 2.0 ** 120


def _small_cache():
    codes = np.full((6, 2, 8, 4), 0x55, dtype=np.uint8)
    return codes, np.full((6, 2, 2), 3.0, dtype=np.float32)


def test_append_places_tokens_and_keeps_other_rows():
    codes, scale = _small_cache()
    x = np.arange(1, 1 + 5 * 2 * 4, dtype=np.float64).reshape(5, 2, 4)
    table, lens, cu = np.array([[5, 0], [2, 3]]), np.array([6, 0]), np.array([0, 4, 5])
    c, s = oc.append(x, codes, np.ones_like(scale), table, lens, cu)
    value = e4m3_value(c) * np.repeat(s.astype(np.float64), 4, axis=2)[..., None]
    for h in range(2):  # tokens 6, 7 of sequence 0 end page 5; 8, 9 begin page 0
        for i, (p, r) in enumerate(((5, 6), (5, 7), (0, 0), (0, 1), (2, 0))):
            assert np.all(np.abs(value[p, h, r] - x[i, h]) <= 2.0 ** -4 * x[i, h])
    rest = np.ones_like(c, dtype=bool)
    for p, r in ((5, 6), (5, 7), (0, 0), (0, 1), (2, 0)):
        rest[p, :, r] = False
    rest[5, :, 4:6] = False  # the group's older tokens may have been rounded again
    assert np.all(c[rest] == 0x55)


def test_append_growing_scale_moves_old_codes_exactly():
    codes, scale = _small_cache()
    codes[5, :, 4:6] = 0x48  # 4.0 under scale 1
    x = np.full((1, 2, 4), 448.0 * 4)
    c, s = oc.append(x, codes, np.ones_like(scale), np.array([[5]]), np.array([6]), np.array([0, 1]))
    assert np.all(s[5, :, 1] == 4.0) and np.all(e4m3_value(c[5, :, 4:6]) == 1.0)
    assert np.all(e4m3_value(c[5, :, 6]) == 448.0)


def test_append_keeps_nonfinite_apart():
    codes, scale = _small_cache()
    x = np.array([[[np.inf, 1.0, np.nan, -1.75]] * 2])
    c, s = oc.append(x, codes, scale, np.array([[1]]), np.array([0]), np.array([0, 1]))
    assert s[1, 0, 0] == 2.0 ** -8
    assert list(np.isnan(e4m3_value(c[1, 0, 0]))) == [True, False, True, False]
    assert e4m3_value(c[1, 0, 0, 3]) == -448.0


def test_decode_oracle_against_softmax():
    scipy_special = pytest.importorskip("scipy.special")
    rng = np.random.default_rng(0)
    codes = rng.integers(0, 0x78, (5, 1, 4, 8)).astype(np.uint8)
    scale = rng.uniform(0.01, 0.02, (5, 1, 2)).astype(np.float32)
    q = rng.standard_normal((1, 2, 3, 8))
    table = np.array([[4, 1, 3]])
    o, lse, _ = oc.decode(q, codes, codes, scale, scale, table, np.array([10]), True, 0.5)
    x = np.concatenate([e4m3_value(codes[p, 0]) * np.repeat(scale[p, 0], 2)[:, None].astype(float)
                        for p in (4, 1, 3)])[:10]
    for h in range(2):
        for i in range(3):
            s = 0.5 * (x[:8 + i] @ q[0, h, i])
            assert np.allclose(o[0, h, i], scipy_special.softmax(s) @ x[:8 + i], atol=1e-13)
            assert np.isclose(lse[0, h, i], scipy_special.logsumexp(s))
    o, lse, _ = oc.decode(q, codes, codes, scale, scale, table, np.array([2]), True, 0.5)
    assert np.all(np.isneginf(lse[:, :, 0])) and np.all(o[:, :, 0] == 0) and np.isfinite(lse[0, 0, 1])


def test_page_plans():
    table = np.array([[7, 2, -1], [7, 5, 0], [1, 1, 1]])
    lens = np.array([8, 9, 0])
    pages, n = oc.free(table, lens, 4, 8)
    assert pages == [1, 3, 4, 6, -1, -1, -1, -1] and n == 4
    new, src, dst, live, moves = oc.compact(table, lens, 4, 8)
    assert (live, moves) == (4, 2) and src == [5, 7, -1, -1] and dst == [1, 3, -1, -1]
    assert new.tolist() == [[3, 2, -1], [3, 1, 0], [1, 1, 1]]
    rows, out, src, dst = oc.fork(table, lens, [1, 0, 2], [6, 4, 3], 4)
    assert rows.tolist() == [[7, 5, 6], [7, 2, -1], [-1, -1, -1]] and out.tolist() == [9, 8, 0]
    assert src.tolist() == [0, -1, -1] and dst.tolist() == [6, -1, -1]


# -------------------------------------------------------------------- refusals

APPEND = dict(k=P, v=P, k_cache=P, v_cache=P, k_scale=P, v_scale=P, block_table=P, seq_lens=P,
              cu=P, B=2, T=5, Hkv=2, d=64, ps=16, mp=4, num=9, group=8, kst=128, vst=128, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), 1), (dict(v_cache=None), 1), (dict(k_scale=None), 1), (dict(block_table=None), 1),
    (dict(seq_lens=None), 1), (dict(B=0), 1), (dict(T=0), 1), (dict(Hkv=0), 1), (dict(mp=0), 1),
    (dict(num=0), 1), (dict(group=0), 1), (dict(group=5), 1), (dict(ps=256, group=256), 1),
    (dict(cu=None), 1), (dict(kst=120), 1), (dict(vst=0), 1), (dict(ps=1 << 20, mp=1 << 11), 1),
    (dict(num=1 << 30), 1), (dict(d=80), 2), (dict(d=0), 2), (dict(kst=132), 3), (dict(vst=129), 3),
    (dict(k=P + 8), 3), (dict(k_cache=P + 1), 3), (dict(v_scale=P + 2), 3), (dict(cu=P + 2), 3),
])
def test_append_rejects_bad_arguments(fa, kw, code):  # noqa: F811
    assert fa.fa_append_paged_fp8(*{**APPEND, **kw}.values()) == code


DECODE = dict(q=P, k_cache=P, v_cache=P, k_scale=P, v_scale=P, block_table=P, seq_lens=P, o=P, lse=P,
              B=2, H=4, Hkv=2, Nq=1, d=128, ps=16, mp=4, num=9, group=16, causal=0, scale=0.1,
              ws=None, ws_bytes=0, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(v_cache=None), 1), (dict(k_scale=None), 1), (dict(lse=None), 1),
    (dict(B=0), 1), (dict(H=0), 1), (dict(H=3), 1), (dict(Hkv=8), 1), (dict(Nq=0), 1),
    (dict(Nq=40000), 1), (dict(ps=0), 1), (dict(mp=0), 1), (dict(num=0), 1), (dict(group=3), 1),
    (dict(num=1 << 30), 1), (dict(B=1 << 20, mp=1 << 11), 1), (dict(d=80), 2), (dict(d=192), 2),
    (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
])
def test_decode_rejects_bad_arguments(fa, kw, code):  # noqa: F811
    assert fa.fa_decode_paged_fp8(*{**DECODE, **kw}.values()) == code


def test_decode_workspace_of_invalid_sizes(fa):  # noqa: F811
    assert fa.fa_decode_paged_fp8_workspace_bytes(1, 4, 3, 1, 128, 16, 4) == 0
    assert fa.fa_decode_paged_fp8_workspace_bytes(1, 4, 4, 1, 80, 16, 4) == 0
    assert fa.fa_decode_paged_fp8_workspace_bytes(1, 4, 4, 0, 128, 16, 4) == 0


def test_page_calls_reject_bad_arguments(fa):  # noqa: F811
    assert fa.fa_free_pages(None, P, P, P, 1, 1, 1, 1, None) == 1
    assert fa.fa_free_pages(P, P, P, P, 0, 1, 1, 1, None) == 1
    assert fa.fa_free_pages(P, P, P, P, 1, 1, 0, 1, None) == 1
    assert fa.fa_free_pages(P, P, P, P, 1, 1, 1, (1 << 22) + 1, None) == 2
    assert fa.fa_free_pages(P + 2, P, P, P, 1, 1, 1, 1, None) == 3
    assert fa.fa_compact_pages(P, P, P, P, P, None, 1, 1, 1, 1, None) == 1
    assert fa.fa_compact_pages(P, P, P, P, P, P, 1 << 16, 1 << 15, 1, 1, None) == 1
    assert fa.fa_compact_pages(P, P, P, P + 1, P, P, 1, 1, 1, 1, None) == 3
    assert fa.fa_fork_pages(P, P, P, P, P, P, P, None, 1, 1, 1, 1, 1, None) == 1
    assert fa.fa_fork_pages(P, P, P, P, P, P, P, P, 1, 0, 1, 1, 1, None) == 1
    assert fa.fa_fork_pages(P, P, P, P + 2, P, P, P, P, 1, 1, 1, 1, 1, None) == 3


def test_copy_rejects_bad_arguments(fa):  # noqa: F811
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    one, size = (vp * 1)(P), (sz * 1)(64)
    assert fa.fa_copy_pages(None, size, 1, 4, P, P, 1, None, None) == 1
    assert fa.fa_copy_pages(one, size, 0, 4, P, P, 1, None, None) == 1
    assert fa.fa_copy_pages(one, size, 129, 4, P, P, 1, None, None) == 1
    assert fa.fa_copy_pages(one, size, 1, 0, P, P, 1, None, None) == 1
    assert fa.fa_copy_pages(one, size, 1, 4, P, P, 0, None, None) == 1
    assert fa.fa_copy_pages(one, size, 1, 4, P, P + 2, 1, None, None) == 3
    assert fa.fa_copy_pages((vp * 1)(None), size, 1, 4, P, P, 1, None, None) == 1
    assert fa.fa_copy_pages(one, (sz * 1)(0), 1, 4, P, P, 1, None, None) == 1


def _cache_args(index=0):
    x = lambda shape, dt: _on(torch.zeros(shape, dtype=dt), index)
    return dict(k_cache=x((9, 2, 16, 64), torch.uint8), v_cache=x((9, 2, 16, 64), torch.uint8),
                k_scale=x((9, 2, 2), torch.float32), v_scale=x((9, 2, 2), torch.float32),
                block_table=x((3, 4), torch.int32), seq_lens=x((3,), torch.int32))


@pytest.mark.parametrize("change,match", [
    (dict(k_cache=((9, 2, 16, 64), torch.float32)), "k_cache must be"),
    (dict(v_cache=((9, 2, 8, 64), torch.uint8)), "v_cache must have shape"),
    (dict(k_scale=((9, 2, 3), torch.float32)), "page_size / group"),
    (dict(k_scale=((9, 2, 0), torch.float32)), "page_size / group"),
    (dict(v_scale=((9, 2, 1), torch.float32)), "v_scale must have shape"),
    (dict(block_table=((12,), torch.int32)), "block_table must be"),
    (dict(block_table=((3, 4), torch.int64)), "block_table must be"),
    (dict(seq_lens=((4,), torch.int32)), "seq_lens must have shape"),
    (dict(k=((3, 3, 64), torch.bfloat16)), "k must be"),
    (dict(k=((3, 2, 64), torch.float16)), "k must be"),
    (dict(v=((4, 2, 64), torch.bfloat16)), "same number of rows"),
    (dict(k=((4, 2, 64), torch.bfloat16), v=((4, 2, 64), torch.bfloat16)), "one row per sequence"),
    (dict(cu_seqlens=((3,), torch.int32)), "cu_seqlens must have shape"),
])
def test_append_wrapper_rejects(fa, change, match):  # noqa: F811
    a = _cache_args()
    a["k"] = a["v"] = _on(torch.zeros((3, 2, 64), dtype=torch.bfloat16), 0)
    for name, (shape, dt) in change.items():
        a[name] = _on(torch.zeros(shape, dtype=dt), 0)
    with pytest.raises(ValueError, match=match):
        fa.append_paged_fp8(**a)


def test_append_wrapper_rejects_strided_heads_and_other_devices(fa):  # noqa: F811
    a = _cache_args()
    rows = torch.zeros((3, 64, 2), dtype=torch.bfloat16).transpose(1, 2)
    ok = _on(torch.zeros((3, 2, 64), dtype=torch.bfloat16), 0)
    with pytest.raises(ValueError, match="contiguous"):
        fa.append_paged_fp8(_on(rows, 0), ok, **a)
    with pytest.raises(ValueError, match="v is on cuda:1"):
        fa.append_paged_fp8(ok, _on(torch.zeros((3, 2, 64), dtype=torch.bfloat16), 1), **a)
    with pytest.raises(ValueError, match="CUDA tensor"):
        fa.append_paged_fp8(torch.zeros((3, 2, 64), dtype=torch.bfloat16), ok, **a)


def test_decode_wrapper_rejects(fa):  # noqa: F811
    q = _on(torch.zeros((3, 4, 1, 64), dtype=torch.bfloat16), 0)
    a = _cache_args()
    for bad, match in ((dict(q=torch.zeros((3, 4, 1, 64), dtype=torch.bfloat16)), "CUDA tensor"),
                       (dict(q=_on(torch.zeros((3, 4, 64), dtype=torch.bfloat16), 0)), r"q must be \[B"),
                       (dict(q=_on(torch.zeros((2, 4, 1, 64), dtype=torch.bfloat16), 0)), "block_table"),
                       (dict(q=_on(torch.zeros((3, 3, 1, 64), dtype=torch.bfloat16), 0)), "dividing H"),
                       (dict(q=_on(torch.zeros((3, 4, 1, 128), dtype=torch.bfloat16), 0)), "dividing H"),
                       (dict(out=_on(torch.zeros((3, 4, 1, 64)), 0)), "out must be"),
                       (dict(lse=_on(torch.zeros((3, 4, 2)), 0)), "lse must have shape"),
                       (dict(k_scale=_on(torch.zeros((9, 2, 2)), 1)), "k_scale is on cuda:1")):
        with pytest.raises(ValueError, match=match):
            fa.decode_paged_fp8(**{**a, "q": q, **bad})


def test_page_wrappers_reject(fa):  # noqa: F811
    x = lambda shape, dt=torch.int32, i=0: _on(torch.zeros(shape, dtype=dt), i)
    with pytest.raises(ValueError, match="block_table"):
        fa.free_pages(x((3,)), x((3,)), 16, 8)
    with pytest.raises(ValueError, match="seq_lens"):
        fa.compact_pages(x((3, 2)), x((2,)), 16, 8)
    with pytest.raises(ValueError, match="fresh"):
        fa.fork_pages(x((3, 2)), x((3,)), x((2,)), x((3,)), 16, 8)
    with pytest.raises(ValueError, match="parents"):
        fa.fork_pages(x((3, 2)), x((3,)), x((2, 1)), x((2, 1)), 16, 8)
    cache = x((8, 2, 16), torch.uint8)
    with pytest.raises(ValueError, match="caches must be"):
        fa.copy_pages([], x((2,)), x((2,)))
    with pytest.raises(ValueError, match="like the first"):
        fa.copy_pages([cache, x((7, 2), torch.float32)], x((2,)), x((2,)))
    with pytest.raises(ValueError, match="dst must have shape"):
        fa.copy_pages([cache], x((2,)), x((3,)))
    with pytest.raises(ValueError, match="count must have shape"):
        fa.copy_pages([cache], x((2,)), x((2,)), count=x((2,)))
    with pytest.raises(ValueError, match=r"caches\[1\] is on cuda:1"):
        fa.copy_pages([cache, x((8, 2, 16), torch.uint8, 1)], x((2,)), x((2,)))
    with pytest.raises(ValueError, match="contiguous"):
        fa.copy_pages([_on(torch.zeros((8, 4, 2)).transpose(1, 2), 0)], x((2,)), x((2,)))


class _OtherStream:
    """Stands for a torch stream of GPU 1."""
    device_index, cuda_stream = 1, 0x1000


def test_streams_of_another_device_are_refused(fa, monkeypatch):  # noqa: F811
    monkeypatch.setattr(torch.cuda, "Stream", _OtherStream)
    q = _on(torch.zeros((3, 4, 1, 64), dtype=torch.bfloat16), 0)
    a, i32 = _cache_args(), _on(torch.zeros(2, dtype=torch.int32), 0)
    kv = _on(torch.zeros((3, 2, 64), dtype=torch.bfloat16), 0)
    s = _OtherStream()
    calls = [lambda: fa.decode_paged_fp8(q, **a, stream=s), lambda: fa.append_paged_fp8(kv, kv, **a, stream=s),
             lambda: fa.free_pages(a["block_table"], a["seq_lens"], 16, 9, stream=s),
             lambda: fa.compact_pages(a["block_table"], a["seq_lens"], 16, 9, stream=s),
             lambda: fa.fork_pages(a["block_table"], a["seq_lens"], i32, i32, 16, 9, stream=s),
             lambda: fa.copy_pages([a["k_cache"]], i32, i32, stream=s),
             lambda: fa.forward(q, q, q, stream=s), lambda: fa.backward(q, q, q, q, q, q, stream=s),
             lambda: fa.decode(q, q, q, stream=s), lambda: fa.quantize_fp8(q, stream=s)]
    for call in calls:
        with pytest.raises(ValueError, match="stream is on cuda:1"):
            call()
