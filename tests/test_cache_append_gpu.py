"""Storing tokens in the paged e4m3 cache (fa_append_paged_fp8) against the oracle: codes and
scales are equal bit for bit, and every other byte of the cache stays as it was."""
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


def _rows(T, Hkv, d, seed, extra=0):
    """k and v as slices of one fused tensor (row stride larger than Hkv * d)."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, 2 * Hkv + extra, d), generator=g)
    x = x * torch.exp(2 * torch.randn((T, 2 * Hkv + extra, 1), generator=g))
    return x.to(torch.bfloat16)


def _run(fa, x, Hkv, d, ps, group, old, new, seed=0, cu=None, num_extra=3, stream=None, edit=None):
    B = len(old)
    lens_after = [a + n for a, n in zip(old, new)]
    width = max(1, max(-(-n // ps) for n in lens_after)) + 1
    num_pages = sum(-(-n // ps) for n in lens_after) + num_extra
    table = make_table(lens_after, ps, width, num_pages, seed + 1)
    kc, ks = make_cache(num_pages, Hkv, ps, d, group, seed + 2, pow2=True)
    vc, vs = make_cache(num_pages, Hkv, ps, d, group, seed + 3, pow2=True)
    if edit:
        edit(kc, vc, ks, vs, table)
    offs = np.concatenate(([0], np.cumsum(new))) if cu is None else np.asarray(cu)
    t = [y.to(DEV) for y in (kc, vc, ks, vs, table, torch.tensor(old, dtype=torch.int32),
                             torch.tensor(offs, dtype=torch.int32))]
    xd = x.to(DEV)
    fa.append_paged_fp8(xd[:, :Hkv], xd[:, Hkv:2 * Hkv], *t[:6], cu_seqlens=t[6], stream=stream)
    torch.cuda.synchronize()
    for i, (codes, scale) in enumerate(((kc, ks), (vc, vs))):
        rc, rs = oc.append(x[:, i * Hkv:(i + 1) * Hkv].double().numpy(), codes.numpy(), scale.numpy(),
                           table.numpy(), old, offs)
        got_c, got_s = t[i].cpu().numpy(), t[i + 2].cpu().numpy()
        assert np.array_equal(got_s, rs), f"scales of {'kv'[i]} at {np.argwhere(got_s != rs)[:4]}"
        assert np.array_equal(got_c, rc), f"codes of {'kv'[i]} at {np.argwhere(got_c != rc)[:4]}"
    return t


@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("ps,group", [(16, 16), (24, 8), (64, 32), (128, 128), (6, 3), (96, 48), (5, 1)])
def test_append_matches_oracle(fa, d, ps, group):
    old, new = [0, 5, ps, 3 * ps - 1, 2 * ps + 3, 0, 7], [ps + 3, 1, 0, 2, 4 * ps + 1, 0, 70]
    _run(fa, _rows(sum(new), 2, d, d + ps, extra=1), 2, d, ps, group, old, new, seed=ps)
    assert fa.fa_device_status(None) == 0


@pytest.mark.parametrize("B,Hkv", [(1, 1), (3, 5), (70, 8), (200, 1)])
def test_append_one_token_each(fa, B, Hkv):
    old = [(7 * b) % 50 for b in range(B)]
    x = _rows(B, Hkv, 128, B)
    t = _run(fa, x, Hkv, 128, 16, 16, old, [1] * B, seed=B)
    u = [y.to(DEV) for y in make_cache(t[0].shape[0], Hkv, 16, 128, 16, B + 2, pow2=True)]
    w = [y.to(DEV) for y in make_cache(t[0].shape[0], Hkv, 16, 128, 16, B + 3, pow2=True)]
    xd = x.to(DEV)  # without offsets: the same result
    fa.append_paged_fp8(xd[:, :Hkv], xd[:, Hkv:], u[0], w[0], u[1], w[1], t[4], t[5])
    assert all(torch.equal(a, b) for a, b in zip((u[0], w[0], u[1], w[1]), t[:4]))
    assert fa.fa_device_status(None) == 0


def test_append_many_sequences_and_long_ones(fa):
    old, new = [b % 33 for b in range(300)], [(b * 37) % 11 for b in range(300)]
    new[17], new[200] = 500, 333
    _run(fa, _rows(sum(new), 1, 64, 9), 1, 64, 32, 16, old, new, seed=5)
    assert fa.fa_device_status(None) == 0


def test_append_special_values(fa):
    x = _rows(40, 2, 128, 3)
    x[0] = 0.0
    x[16:32, 0] = 0.0                                   # a whole group of zeros
    x[3, 1, 5], x[4, 1, 6], x[5, 2, 0] = float("inf"), float("-inf"), float("nan")
    x[33:, 3] = float("nan")                            # a group with no finite element
    x[6, 0, 0], x[7, 2, 1] = 3.0e38, -2.0 ** -133       # bf16's ends
    _run(fa, x, 2, 128, 16, 16, [0], [40])
    _run(fa, x, 2, 128, 16, 16, [9], [40])
    assert fa.fa_device_status(None) == 0


def test_append_rounds_ties_to_even(fa):
    x = torch.zeros((16, 2, 64), dtype=torch.bfloat16)
    x[:, :, 0] = 256.0
    x[:, :, 1:] = torch.arange(1, 64) * 0.5 + 8         # halves of the step 1 between 8 and 16
    _run(fa, x, 1, 64, 16, 16, [0], [16])


def test_append_rows_outside_every_sequence(fa):
    x = _rows(30, 1, 64, 8)
    _run(fa, x, 1, 64, 8, 8, [3, 0], [9, 6], cu=[5, 14, 20])
    assert fa.fa_device_status(None) == 0


def test_append_grown_scale_of_foreign_groups(fa):
    """A group whose scale is no power of two gets one, its older codes rounded again."""
    def edit(kc, vc, ks, vs, table):
        ks[:], vs[:] = 0.3, 1e-3
    _run(fa, _rows(20, 2, 128, 4), 2, 128, 16, 16, [5, 3], [10, 10], edit=edit)


def test_append_in_steps_equals_tokens_seen_so_far(fa):
    """Token by token: after each step the group's codes are its tokens at its scale."""
    x = _rows(16, 1, 128, 12)
    xd = x.to(DEV)
    kc, ks = make_cache(2, 1, 16, 128, 16, 1, pow2=True)
    ref_c, ref_s = kc.numpy(), ks.numpy()
    dev = [kc.to(DEV), kc.to(DEV), ks.to(DEV), ks.to(DEV)]
    table = torch.ones((1, 1), dtype=torch.int32, device=DEV)
    for j in range(16):
        lens = torch.tensor([j], dtype=torch.int32, device=DEV)
        fa.append_paged_fp8(xd[j:j + 1, :1], xd[j:j + 1, 1:], *dev, table, lens)
        ref_c, ref_s = oc.append(x[j:j + 1, :1].double().numpy(), ref_c, ref_s, np.array([[1]]), [j], [0, 1])
        assert np.array_equal(dev[0].cpu().numpy(), ref_c) and np.array_equal(dev[2].cpu().numpy(), ref_s)


def test_append_bad_indices_touch_nothing(fa):
    x = _rows(12, 1, 64, 2)
    xd = x.to(DEV)
    kc, ks = make_cache(4, 1, 8, 64, 8, 1, pow2=True)

    def call(table, lens, cu):
        t = [y.to(DEV) for y in (kc, kc, ks, ks)]
        fa.append_paged_fp8(xd[:, :1], xd[:, 1:], *t, torch.tensor(table, dtype=torch.int32, device=DEV),
                            torch.tensor(lens, dtype=torch.int32, device=DEV),
                            cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV))
        status = fa.fa_device_status(None)
        return status, torch.equal(t[0].cpu(), kc) and torch.equal(t[2].cpu(), ks)

    for table, lens, cu in (([[4, 1]], [0], [0, 8]), ([[-1, 1]], [0], [0, 8]), ([[0, 1]], [-1], [0, 8]),
                            ([[0, 1]], [9], [0, 8]), ([[0, 1]], [0], [-3, 8]), ([[0, 1]], [0], [0, 13]),
                            ([[0, 1]], [0], [9, 3])):
        assert call(table, lens, cu) == (7, True), (table, lens, cu)
    status, same = call([[7, 1], [2, 3]], [0, 0], [0, 4, 8])  # the other sequence is stored
    assert status == 7 and not same


def test_append_on_another_stream_and_captured(fa):
    old, new = [3, 20], [9, 4]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    _run(fa, _rows(13, 2, 128, 6), 2, 128, 16, 16, old, new, stream=s)
    x = _rows(2, 2, 128, 7)
    xd = x.to(DEV)
    kc, ks = make_cache(6, 2, 16, 128, 16, 5, pow2=True)
    t = [y.to(DEV) for y in (kc, kc, ks, ks)]
    table = torch.tensor([[0, 4], [2, 5]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([3, 15], dtype=torch.int32, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fa.append_paged_fp8(xd[:, :2], xd[:, 2:], *t, table, lens)
        lens += 1
    rc, rs = kc.numpy(), ks.numpy()
    for step in range(3):  # replays follow the lengths and rows of the moment
        xd.copy_(_rows(2, 2, 128, 70 + step))
        g.replay()
        torch.cuda.synchronize()
        rc, rs = oc.append(_rows(2, 2, 128, 70 + step)[:, :2].double().numpy(), rc, rs, table.cpu().numpy(),
                           [3 + step, 15 + step], [0, 1, 2])
        assert np.array_equal(t[0].cpu().numpy(), rc) and np.array_equal(t[2].cpu().numpy(), rs)
    assert fa.fa_device_status(None) == 0


def _bad_offset_cases():
    """(offsets, sequences stored, rows): offsets outside 0 .. T among good ones."""
    yield [-3, 4, 8], [1], 12
    yield [0, 4, 99, 8, 12], [0, 3], 12
    yield [2, -1, 5, 12], [2], 12
    yield [0, 13, 4, 12], [2], 12
    yield [0, 3, 7, 13], [0, 1], 12
    cu = list(range(0, 303, 3))
    for at in (0, 1, 31, 32, 50, 64, 96, 99, 100):  # the search for a row's sequence meets it or not
        for wild in (-1, 1 << 30):
            yield cu[:at] + [wild] + cu[at + 1:], [b for b in range(100) if b not in (at - 1, at)], 300


@pytest.mark.parametrize("cu,good,T", list(_bad_offset_cases()))
@pytest.mark.parametrize("ps,group,old", [(8, 4, 0), (16, 16, 5), (6, 1, 3)])
def test_append_bad_offsets_skip_their_sequences_only(fa, cu, good, T, ps, group, old):
    B, Hkv, d = len(cu) - 1, 2, 64
    x = _rows(T, Hkv, d, 31)
    table = make_table([old + 20] * B, ps, -(-(old + 20) // ps), B * (-(-(old + 20) // ps)) + 2, 32)
    caches = [make_cache(int(table.max()) + 2, Hkv, ps, d, group, seed, pow2=True) for seed in (33, 34)]
    (kc, ks), (vc, vs) = caches
    dev = [t.to(DEV) for t in (kc, vc, ks, vs)]
    xd = x.to(DEV)
    fa.append_paged_fp8(xd[:, :Hkv], xd[:, Hkv:], *dev, table.to(DEV),
                        torch.full((B,), old, dtype=torch.int32, device=DEV),
                        cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV))
    assert fa.fa_device_status(None) == 7
    for i, (codes, scale) in enumerate(caches):
        rc, rs = codes.numpy(), scale.numpy()
        for b in good:
            rc, rs = oc.append(x[cu[b]:cu[b + 1], i * Hkv:(i + 1) * Hkv].double().numpy(), rc, rs,
                               table[b:b + 1].numpy(), [old], [0, cu[b + 1] - cu[b]])
        assert np.array_equal(dev[i].cpu().numpy(), rc) and np.array_equal(dev[i + 2].cpu().numpy(), rs)
