"""Calls with `stream=` another stream than the current one: what a call allocates belongs to the
stream its kernels run on, and neither side's later work can take it away."""
import pytest
import torch

from cache_common import DEV, make_cache, make_table
from gpu_common import load_fa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    return load_fa()


def _paged(fa):
    """name -> a call of the paged e4m3 cache, taking the stream."""
    lens = torch.tensor([9000, 700, 0, 4100], dtype=torch.int32, device=DEV)
    num = 900
    table = make_table(lens.tolist(), 16, 600, num, 3).to(DEV)
    (kc, ks), (vc, vs) = ([t.to(DEV) for t in make_cache(num, 2, 16, 128, 16, s)] for s in (1, 2))
    q = torch.randn((4, 8, 1, 128), generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).to(DEV)
    parents = torch.tensor([0, 3, 1], dtype=torch.int32, device=DEV)
    fresh = torch.tensor([880, 881, 882], dtype=torch.int32, device=DEV)
    return {
        "decode_paged_fp8": lambda s: fa.decode_paged_fp8(q, kc, vc, ks, vs, table, lens, stream=s),
        "decode_paged_fp8 of a tensor subclass": lambda s: fa.decode_paged_fp8(
            torch.nn.Parameter(q, requires_grad=False), kc, vc, ks, vs, table, lens, stream=s),
        "free_pages": lambda s: fa.free_pages(table, lens, 16, num, stream=s),
        "fork_pages": lambda s: fa.fork_pages(table, lens, parents, fresh, 16, num, stream=s),
        "compact_pages": lambda s: fa.compact_pages(table, lens, 16, num, stream=s),
    }


def _dense(fa):
    """name -> a call on tensors that are not a paged e4m3 cache, taking the stream."""
    g = torch.Generator().manual_seed(5)

    def rand(*shape):
        return torch.randn(shape, generator=g).to(torch.bfloat16).to(DEV)

    q, k, v, do = (rand(1, 2, 2048, 128) for _ in range(4))
    o, lse = fa.forward(q, k, v, causal=True)
    q1, kc, vc = rand(2, 4, 1, 128), rand(2, 4, 6000, 128), rand(2, 4, 6000, 128)
    pages = (rand(400, 2, 16, 128), rand(400, 2, 16, 128))
    table = torch.randperm(400, generator=g).to(torch.int32).reshape(2, 200).to(DEV)
    lens = torch.tensor([3100, 77], dtype=torch.int32, device=DEV)
    tq, tk, tv, tdo = (rand(700, 4, 64) for _ in range(4))
    cu = torch.tensor([0, 300, 700], dtype=torch.int32, device=DEV)
    to, tl = fa.forward_varlen(tq, tk, tv, cu, 400, causal=True)
    x8 = [fa.quantize_fp8(t) for t in (q, k)] + [fa.quantize_fp8(v, 0, transpose=True)]
    torch.cuda.synchronize()
    return {
        "forward": lambda s: fa.forward(q, k, v, causal=True, stream=s),
        "forward with cut key ranges": lambda s: fa.forward(q, k, v, causal=True, stream=s, kv_chunk=512),
        "backward": lambda s: fa.backward(q, k, v, o, lse, do, causal=True, stream=s)[1:],  # dQ: atomic sums
        "decode": lambda s: fa.decode(q1, kc, vc, num_splits=8, stream=s),
        "decode_paged": lambda s: fa.decode_paged(q1, *pages, table, lens, num_splits=8, stream=s),
        "forward_varlen": lambda s: fa.forward_varlen(tq, tk, tv, cu, 400, causal=True, stream=s),
        "backward_varlen": lambda s: fa.backward_varlen(tq, tk, tv, to, tl, tdo, cu, 400, causal=True,
                                                        stream=s)[1:],
        "quantize_fp8": lambda s: fa.quantize_fp8(q, stream=s),
        "forward_fp8": lambda s: fa.forward_fp8(*(t[0] for t in x8), *(t[1] for t in x8), causal=True,
                                                stream=s),
    }


DENSE = ["forward", "forward with cut key ranges", "backward", "decode", "decode_paged", "forward_varlen",
         "backward_varlen", "quantize_fp8", "forward_fp8"]
PAGED = ["decode_paged_fp8", "decode_paged_fp8 of a tensor subclass", "free_pages", "fork_pages",
         "compact_pages"]


@pytest.fixture(scope="module")
def calls(fa):
    return {**_paged(fa), **_dense(fa)}


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", PAGED + DENSE)
def test_allocations_belong_to_the_given_stream(fa, calls, name, handle):
    s = torch.cuda.Stream()
    call = calls[name]
    expect = call(None)
    torch.cuda.synchronize()
    torch.cuda.memory._record_memory_history(context=None)
    try:
        got = call(s.cuda_stream if handle else s)
        trace = torch.cuda.memory._snapshot()["device_traces"][0]
    finally:
        torch.cuda.memory._record_memory_history(enabled=None)
    torch.cuda.synchronize()
    streams = [e["stream"] for e in trace if e["action"] == "alloc"]
    assert streams and set(streams) == {s.cuda_stream}
    assert all(torch.equal(a, b) for a, b in zip(expect, got))


@pytest.mark.parametrize("name", PAGED + DENSE)
def test_the_current_stream_goes_on_meanwhile(fa, calls, name):
    """Calls on one stream while the current one allocates and writes memory of all sizes."""
    s = torch.cuda.Stream()
    call = calls[name]
    expect = call(None)
    torch.cuda.synchronize()
    got = []
    for i in range(30):
        got.append(call(s))
        for size in (64, 4096, 40000, 700000, 5000000):
            torch.empty(size, dtype=torch.uint8, device=DEV).fill_(i)
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(expect, g))


@pytest.mark.parametrize("name", PAGED + DENSE)
def test_results_outlive_their_release_while_the_caller_reads_them(fa, calls, name):
    """Results released while the current stream has not read them yet: the next calls on the
    other stream must not be given their memory."""
    s = torch.cuda.Stream()
    call = calls[name]
    expect = call(None)
    torch.cuda.synchronize()
    junk = []
    for _ in range(5):
        got = call(s)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda._sleep(20_000_000)  # about 10 ms
        copies = [t.clone() for t in got]
        sizes = [t.numel() * t.element_size() for t in got]
        del got
        with torch.cuda.stream(s):
            junk += [torch.full((n,), 77, dtype=torch.uint8, device=DEV) for n in sizes]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(expect, copies))


def test_given_the_current_stream_or_the_default_one(fa, calls):
    """The current stream by name, by handle, and the default stream's handle 0 from another."""
    call = calls["decode_paged_fp8"]
    expect = call(None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = [call(s), call(s.cuda_stream), call(0)]
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(expect, g))
    assert fa.fa_device_status(None) == 0


@pytest.mark.parametrize("name", PAGED + ["forward with cut key ranges", "decode", "backward_varlen"])
def test_captured_on_a_side_stream(fa, calls, name):
    """A capture whose calls run on a stream that forks from the capturing one and joins it."""
    call = calls[name]
    expect = call(None)
    side = torch.cuda.Stream()
    call(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        got = call(side)
        torch.cuda.current_stream().wait_stream(side)
        copies = [t.clone() for t in got]
        del got
    for _ in range(3):
        for c in copies:
            c.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(expect, copies))
    assert fa.fa_device_status(None) == 0
