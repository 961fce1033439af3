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


PAGED = ["decode_paged_fp8", "decode_paged_fp8 of a tensor subclass", "free_pages", "fork_pages",
         "compact_pages"]


@pytest.fixture(scope="module")
def calls(fa):
    return _paged(fa)


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", PAGED)
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


@pytest.mark.parametrize("name", PAGED)
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


@pytest.mark.parametrize("name", PAGED)
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
