"""Page upkeep of a paged cache (free, fork, compact, copy) against the oracle: whole numbers
and copied bytes, equal throughout."""
import numpy as np
import pytest
import torch

from cache_common import DEV, make_cache, make_table
from gpu_common import load_fa
from oracle import cache as oc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    return load_fa()


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def _random(B, ps, num_pages, seed, share=0.0, fill=0.6):
    """Lengths (zeros among them) and a table of random pages, some shared."""
    r = np.random.default_rng(seed)
    width = max(1, int(2 * num_pages * fill / B) + 1)
    left, lens = int(num_pages * fill), []
    for _ in range(B):
        n = int(r.integers(0, min(left, width) * ps + 1)) if r.random() > 0.15 else 0
        left -= -(-n // ps)
        lens.append(n)
    table = make_table(lens, ps, width, num_pages, seed).numpy()
    for b in range(1, B):
        if r.random() < share:  # shares its first pages with the sequence before it
            k = min(-(-lens[b] // ps), -(-lens[b - 1] // ps))
            table[b, :k] = table[b - 1, :k]
    return table, np.array(lens)


SIZES = [(1, 1, 1, 0), (3, 16, 31, 0), (2, 8, 32, 1), (7, 16, 33, 2), (40, 24, 1000, 3), (5, 1, 257, 4),
         (300, 64, 9000, 5), (1, 16, 70000, 6), (64, 128, 262144, 7)]


@pytest.mark.parametrize("B,ps,num,seed", SIZES)
def test_free_and_compact_match_oracle(fa, B, ps, num, seed):
    table, lens = _random(B, ps, num, seed, share=0.4)
    pages, count = fa.free_pages(_i32(table), _i32(lens), ps, num)
    ref, n = oc.free(table, lens, ps, num)
    assert count.item() == n and pages.tolist() == ref
    new, src, dst, counts = fa.compact_pages(_i32(table), _i32(lens), ps, num)
    rn, rs, rd, live, moves = oc.compact(table, lens, ps, num)
    assert counts.tolist() == [live, moves]
    assert src.tolist() == rs and dst.tolist() == rd and np.array_equal(new.cpu().numpy(), rn)
    assert fa.fa_device_status(None) == 0


def test_free_and_compact_of_empty_and_full_caches(fa):
    t = _i32([[3, 1], [0, 2]])
    pages, count = fa.free_pages(t, _i32([0, 0]), 4, 4)
    assert count.item() == 4 and pages.tolist() == [0, 1, 2, 3]
    new, src, dst, counts = fa.compact_pages(t, _i32([0, 0]), 4, 4)
    assert counts.tolist() == [0, 0] and torch.equal(new, t) and src.tolist() == [-1, -1]
    pages, count = fa.free_pages(t, _i32([8, 5]), 4, 4)
    assert count.item() == 0 and pages.tolist() == [-1] * 4
    new, src, dst, counts = fa.compact_pages(t, _i32([8, 5]), 4, 4)
    assert counts.tolist() == [4, 0] and torch.equal(new, t)
    assert fa.fa_device_status(None) == 0


def test_plans_record_bad_lengths_and_pages(fa):
    t = _i32([[3, 9], [0, -5], [1, 2]])
    pages, count = fa.free_pages(t, _i32([8, 8, -1]), 4, 5)
    assert fa.fa_device_status(None) == 7
    assert count.item() == 3 and pages.tolist() == [1, 2, 4, -1, -1]
    _, count = fa.free_pages(_i32([[3, 1]]), _i32([100]), 4, 5)  # as long as its row
    assert fa.fa_device_status(None) == 7 and count.item() == 3
    new, src, dst, counts = fa.compact_pages(t, _i32([8, 8, -1]), 4, 5)
    assert fa.fa_device_status(None) == 7
    assert counts.tolist() == [2, 1] and new.tolist() == [[1, 9], [0, -5], [1, 2]]


@pytest.mark.parametrize("B,ps,n,seed", [(1, 16, 1, 0), (5, 8, 12, 1), (60, 24, 33, 2), (9, 1, 9, 3)])
def test_fork_matches_oracle(fa, B, ps, n, seed):
    table, lens = _random(B, ps, 900, seed)
    r = np.random.default_rng(seed)
    parents = r.integers(0, B, n)
    fresh = r.permutation(np.arange(600, 900))[:n]
    out = fa.fork_pages(_i32(table), _i32(lens), _i32(parents), _i32(fresh), ps, 900)
    for got, ref in zip(out, oc.fork(table, lens, parents, fresh, ps)):
        assert np.array_equal(got.cpu().numpy(), ref)
    assert fa.fa_device_status(None) == 0


def test_fork_records_bad_arguments(fa):
    t, lens = _i32([[3, 1], [0, 7]]), _i32([6, 7])
    rows, out, src, dst = fa.fork_pages(t, lens, _i32([0, 2, -1]), _i32([-1, 4, 4]), 4, 5)
    assert fa.fa_device_status(None) == 7
    assert rows.tolist() == [[3, -1], [-1, -1], [-1, -1]] and out.tolist() == [6, 0, 0]
    assert src.tolist() == [-1] * 3 and dst.tolist()[1:] == [-1] * 2
    rows, _, src, dst = fa.fork_pages(t, lens, _i32([1]), _i32([4]), 4, 5)  # the parent's page is bad
    assert fa.fa_device_status(None) == 7 and src.tolist() == [-1] and dst.tolist() == [-1]


@pytest.mark.parametrize("Hkv,ps,d,group,layers", [(8, 16, 128, 16, 1), (2, 24, 96, 8, 3), (1, 5, 64, 5, 1),
                                                   (3, 64, 256, 32, 2), (1, 1, 64, 1, 32)])
def test_copy_pages(fa, Hkv, ps, d, group, layers):
    num, r = 41, np.random.default_rng(layers)
    caches = [t.to(DEV) for i in range(2 * layers) for t in make_cache(num, Hkv, ps, d, group, i)]
    before = [t.cpu().numpy() for t in caches]
    perm = r.permutation(num)
    src, dst = perm[:15].copy(), perm[15:30].copy()
    src[3:5] = src[0]  # a page may be a source more than once
    src[7] = -1
    fa.copy_pages(caches, _i32(src), _i32(dst))
    for t, ref in zip(caches, before):
        keep = src >= 0
        ref[dst[keep]] = ref[src[keep]]
        assert np.array_equal(t.cpu().numpy(), ref)
    assert fa.fa_device_status(None) == 0


@pytest.mark.parametrize("dtype,row", [(torch.bfloat16, (2, 16, 64)), (torch.uint8, (13,)), (torch.float32, (3,)),
                                       (torch.int64, (5, 7)), (torch.uint8, (4097,)), (torch.bfloat16, (70000,))])
def test_copy_pages_of_any_size_and_type(fa, dtype, row):
    t = torch.randint(0, 100, (9, *row), device=DEV).to(dtype)
    ref = t.clone()
    fa.copy_pages([t], _i32([8, 1, 5]), _i32([0, 2, 7]))
    ref[[0, 2, 7]] = ref[[8, 1, 5]]
    assert torch.equal(t, ref)


def test_copy_pages_counts_and_bad_pages(fa):
    t = torch.arange(8 * 6, device=DEV, dtype=torch.int32).reshape(8, 6)
    for count, moved in ((0, 0), (2, 2), (9, 3), (-4, 0)):
        u, ref = t.clone(), t.clone()
        fa.copy_pages([u], _i32([1, 2, 3]), _i32([5, 6, 7]), count=_i32([count]))
        ref[5:5 + moved] = ref[1:1 + moved]
        assert torch.equal(u, ref)
    assert fa.fa_device_status(None) == 0
    for src, dst in ((8, 0), (-2, 0), (0, 8), (0, -1)):
        u = t.clone()
        fa.copy_pages([u], _i32([src]), _i32([dst]))
        assert fa.fa_device_status(None) == 7 and torch.equal(u, t)


def test_plan_and_copy_in_a_captured_graph(fa):
    """Lengths and tables change between replays; nothing is read back to the host."""
    ps, num = 16, 64
    cache = torch.arange(num, device=DEV, dtype=torch.int32)[:, None].repeat(1, 40)
    table, lens = _i32(np.zeros((6, 12))), _i32([0] * 6)
    work = cache.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        new, src, dst, counts = fa.compact_pages(table, lens, ps, num)
        fa.copy_pages([work], src, dst, count=counts[1:])
    for seed in range(4):
        r = np.random.default_rng(seed)
        n = r.integers(0, 12 * ps // 2, 6)
        ref = make_table(list(n), ps, 12, num, seed).numpy()
        table.copy_(_i32(ref))
        lens.copy_(_i32(n))
        work.copy_(cache)
        g.replay()
        torch.cuda.synchronize()
        got = work.cpu().numpy()[:, 0]
        rn, _, _, live, _ = oc.compact(ref, n, ps, num)
        assert counts[0].item() == live and np.array_equal(new.cpu().numpy(), rn)
        for b in range(6):
            need = -(-n[b] // ps)
            assert np.array_equal(got[rn[b, :need]], ref[b, :need])
    assert fa.fa_device_status(None) == 0


def test_copy_beyond_four_gigabytes(fa):
    big = torch.empty((70, 1 << 26), dtype=torch.uint8, device=DEV)  # 4.4 GB
    big[69], big[1], big[2] = 5, 7, 9
    fa.copy_pages([big], _i32([69, 1]), _i32([0, 68]))
    assert bool((big[0] == 5).all()) and bool((big[68] == 7).all()) and bool((big[2] == 9).all())
