"""Decode against the paged e4m3 cache (fa_decode_paged_fp8) against the float64 oracle, at
every head dimension, head grouping, page and scale-group size, and at the lengths and masks
where it can go wrong; what lies behind a sequence's last token is NaN in every test."""
import math

import numpy as np
import pytest
import torch

from cache_common import DEV, check_decode, make_cache, make_table, oracle_decode
from gpu_common import load_fa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    return load_fa()


def _problem(B, H, Hkv, Nq, d, ps, group, lens, seed=0, spread=1.0, extra=2, qmul=1.0,
             room=1):
    """(q, kc, vc, ks, vs, table, lens) on the CPU; rows behind the last token and whole unused
    pages hold NaN codes, their scales are NaN too, unused table entries point nowhere.  The table
    has room for at least `room` tokens per sequence (longer sequences may be cut differently)."""
    num = sum(-(-n // ps) for n in lens) + extra
    width = max(-(-room // ps), max(-(-n // ps) for n in lens)) + 1
    table = make_table(lens, ps, width, num, seed, unused=1 << 30)
    kc, ks = make_cache(num, Hkv, ps, d, group, seed + 1, spread)
    vc, vs = make_cache(num, Hkv, ps, d, group, seed + 2, spread)
    unused = torch.ones((num, ps), dtype=torch.bool)
    for b, n in enumerate(lens):
        for j in range(-(-n // ps)):
            unused[table[b, j], :max(0, n - j * ps)] = False
    for codes, scale in ((kc, ks), (vc, vs)):
        codes.permute(0, 2, 1, 3)[unused] = 0x7F
        whole = unused.reshape(num, ps // group, group).all(-1)
        scale.permute(0, 2, 1)[whole] = float("nan")
    g = torch.Generator().manual_seed(seed + 3)
    q = (qmul * torch.randn((B, H, Nq, d), generator=g)).to(torch.bfloat16)
    return q, kc, vc, ks, vs, table, torch.tensor(lens, dtype=torch.int32)


def _check(fa, prob, causal=False, scale=None, what="", **kw):
    dev = [t.to(DEV) for t in prob]
    o, lse = fa.decode_paged_fp8(*dev, causal=causal, scale=scale, **kw)
    torch.cuda.synchronize()
    assert fa.fa_device_status(None) == 0
    ref = oracle_decode(*prob, causal, scale or 1 / math.sqrt(prob[0].shape[3]))
    check_decode(o.float().cpu().numpy(), lse.cpu().numpy(), ref, what)
    return o, lse


LENS = [0, 1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 300, 500]


@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 3), (8, 2), (7, 1)])
def test_lengths_and_heads(fa, d, H, Hkv):
    _check(fa, _problem(len(LENS), H, Hkv, 1, d, 16, 16, LENS, seed=d + H))


@pytest.mark.parametrize("ps,group", [(1, 1), (2, 1), (5, 5), (8, 4), (24, 8), (48, 16), (64, 64), (100, 25),
                                      (128, 32), (192, 64), (256, 128), (512, 512)])
def test_page_and_group_sizes(fa, ps, group):
    _check(fa, _problem(5, 4, 2, 1, 128, ps, group, [1, 130, 257, 700, 1025], seed=ps))
    _check(fa, _problem(3, 4, 1, 2, 64, ps, group, [0, 97, 600], seed=ps + 1), causal=True)


@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("H,Hkv,Nq", [(2, 2, 2), (4, 1, 2), (8, 1, 1), (9, 1, 1), (4, 2, 4), (8, 2, 4),
                                      (17, 1, 1), (16, 1, 2), (33, 1, 1), (8, 1, 8), (5, 1, 13), (16, 2, 16),
                                      (64, 1, 3), (2, 1, 70)])
@pytest.mark.parametrize("causal", [False, True])
def test_rows_per_head(fa, d, H, Hkv, Nq, causal):
    _check(fa, _problem(4, H, Hkv, Nq, d, 32, 16, [0, Nq - 1, 150, 411], seed=d + H + Nq), causal=causal,
           what=f"{d} {H} {Hkv} {Nq}")


def test_causal_rows_before_the_first_token(fa):
    prob = _problem(5, 4, 2, 6, 128, 16, 16, [0, 1, 4, 6, 131], seed=3)
    o, lse = _check(fa, prob, causal=True)
    assert np.isneginf(lse[1, :, :5].cpu().numpy()).all() and bool(torch.isfinite(lse[1, :, 5]).all())


@pytest.mark.parametrize("B,H,Hkv,Nq,d,lens", [
    (1, 8, 8, 1, 128, [20000]), (1, 4, 1, 1, 64, [33333]), (2, 16, 2, 2, 128, [9000, 12345]),
    (3, 4, 4, 1, 256, [7000, 1, 5000]), (1, 2, 2, 3, 96, [15001])])
def test_long_sequences_are_cut_and_merged(fa, B, H, Hkv, Nq, d, lens):
    _check(fa, _problem(B, H, Hkv, Nq, d, 64, 32, lens, seed=d), causal=Nq > 1)


@pytest.mark.parametrize("ps,group", [(2, 1), (2, 2), (6, 3), (7, 7), (16, 8), (64, 32), (512, 128)])
@pytest.mark.parametrize("H,Hkv,Nq", [(2, 2, 1), (4, 2, 4), (4, 1, 4)])
def test_keys_of_half_a_row(fa, ps, group, H, Hkv, Nq):
    """d = 64, where two keys share a row of a tile: sequences that end in either half of one, on
    both sides of a tile of 128 and of 256 keys."""
    lens = [1, 2, 127, 128, 129, 255, 256, 257, 258, 511, 512, 513, 1000, 0, 3001]
    for room in (1, 150000):
        _check(fa, _problem(len(lens), H, Hkv, Nq, 64, ps, group, lens, seed=ps, room=room), causal=Nq > 1)


def test_a_chunk_of_many_queries(fa):
    """A causal chunk of 300 new tokens behind, and as all of, a sequence."""
    for d in (64, 128, 256):
        _check(fa, _problem(3, 4, 2, 300, d, 16, 16, [300, 1111, 299], seed=d), causal=True)


def test_many_sequences(fa):
    lens = [(b * 131) % 300 for b in range(400)]
    _check(fa, _problem(400, 2, 1, 1, 64, 16, 16, lens, seed=1))


@pytest.mark.parametrize("H,Hkv,Nq,d", [(8, 2, 1, 128), (8, 1, 2, 64), (32, 1, 1, 256)])
def test_a_long_sequence_among_many_short_ones(fa, H, Hkv, Nq, d):
    """Hundreds of CTAs share the long sequence, and its partial results meet; then a bad page of
    it, which leaves it alone and no other."""
    lens = [(b * 17) % 40 for b in range(110)]
    lens[40], lens[77] = 50000, 3000
    prob = _problem(len(lens), H, Hkv, Nq, d, 64, 32, lens, seed=d)
    _check(fa, prob, causal=Nq > 1)
    dev = [t.to(DEV) for t in prob]
    dev[5][40, 300] = -1
    out = torch.full(prob[0].shape, 3.0, dtype=torch.bfloat16, device=DEV)
    again, _ = fa.decode_paged_fp8(*dev, causal=Nq > 1)
    assert fa.fa_device_status(None) == 7
    fa.decode_paged_fp8(*dev, causal=Nq > 1, out=out)
    assert fa.fa_device_status(None) == 7
    keep = torch.ones(len(lens), dtype=torch.bool)
    keep[40] = False
    assert torch.equal(out[keep.to(DEV)], again[keep.to(DEV)]) and bool((out[40] == 3.0).all())


def test_all_sequences_empty(fa):
    o, lse = _check(fa, _problem(3, 4, 2, 1, 128, 16, 16, [0, 0, 0]))
    assert bool((o == 0).all()) and bool(torch.isneginf(lse).all())


@pytest.mark.parametrize("scale,qmul", [(1.5, 1.0), (1e-4, 1.0), (0.088, 30.0), (0.088, 1e-3)])
def test_scales_of_the_scores(fa, scale, qmul):
    _check(fa, _problem(2, 4, 2, 1, 128, 16, 16, [700, 300], seed=5, qmul=qmul), scale=scale)


def test_queries_over_many_binades(fa):
    """q elements far below the row's largest keep their place in the scores."""
    prob = list(_problem(2, 4, 2, 2, 128, 16, 16, [400, 129], seed=6))
    prob[0] = prob[0] * torch.exp2(-torch.arange(128) / 8).to(torch.bfloat16)
    _check(fa, prob, scale=0.3)


@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("exponent", [-2, -6, -7, -8, -9, -12, -16])
def test_small_elements_beside_a_large_one_of_a_query(fa, d, exponent):
    """The row's largest element, 2^7, meets keys of zero, and the rest, all near 2^exponent and of
    one sign with its keys, make up the score, which is L for a single key.  q is kept exactly down
    to 2^-14 of the largest element; below, an element x is off by at most 2^-15 where the largest
    is 2^7, and by f16's half step below 2^-14, 2^-25, with it: 2^-22 (1 + 2^-10) of the largest."""
    H = 8
    g = torch.Generator().manual_seed(d - exponent)
    mantissa = 1 + torch.randint(0, 128, (1, H, 1, d), generator=g) / 128
    mantissa[0, 0], mantissa[0, 1] = 1 + 1 / 128, 1 + 127 / 128
    sign = torch.where(torch.rand(d, generator=g) < 0.5, -1.0, 1.0)
    q = (mantissa * 2.0 ** exponent * sign).to(torch.bfloat16)
    assert torch.equal(q.float(), mantissa * 2.0 ** exponent * sign)
    q[..., d // 2] = 128.0
    kc = torch.where(sign > 0, 0x38, 0xB8).to(torch.uint8).expand(1, 1, 16, d).contiguous()  # 1.0
    kc[..., d // 2] = 0
    vc, vs = make_cache(1, 1, 16, d, 16, 5)
    ks = torch.full((1, 1, 1), 2.0 ** (-exponent - 6))
    prob = [q, kc, vc, ks, vs, torch.zeros((1, 1), dtype=torch.int32), torch.ones(1, dtype=torch.int32)]
    _, lse = fa.decode_paged_fp8(*[t.to(DEV) for t in prob], scale=1.0)
    ref = oracle_decode(*prob, False, 1.0)
    off = 0.0 if exponent >= -7 else 2.0 ** -22 * (1 + 2.0 ** -10) * 128 * (d - 1) * float(ks)
    bound = off + 2.0 ** -20 * ref[2][2] + 2.0 ** -20 * (1 + np.abs(ref[1]))
    err = np.abs(lse.cpu().double().numpy() - ref[1])
    assert np.all(err <= bound), f"L off by {err.max():.3e}, bound {bound[err > bound].min():.3e}"


def test_a_sink_token_and_many_small_weights(fa):
    """One key takes nearly all of the weight and has a small value; thousands of weights near
    2^-12 of the largest make up the rest of the output."""
    prob = list(_problem(1, 2, 1, 1, 128, 16, 16, [6000], seed=7, spread=0.0))
    q, kc, vc, ks, vs, table, lens = prob
    page = int(table[0, 0])
    kc[page, 0, 0] = torch.where(q[0, 0, 0].float() > 0, 0x70, 0xF0).to(torch.uint8)
    q[0, 1] = q[0, 0]
    vs[page] *= 2.0 ** -8
    _check(fa, prob, scale=0.02)
    _check(fa, prob, scale=0.05)


def test_value_scales_over_many_binades(fa):
    _check(fa, _problem(2, 4, 2, 1, 128, 16, 8, [900, 333], seed=8, spread=3.0))


@pytest.mark.parametrize("exponent", [120, 100, -100, -126])
def test_extreme_value_scales(fa, exponent):
    prob = list(_problem(2, 4, 2, 1, 128, 16, 16, [700, 140], seed=19))
    prob[2] &= 0xBF  # codes below 2, so that the outputs fit
    prob[4] = torch.full_like(prob[4], 2.0 ** exponent)
    _check(fa, prob)
    prob[4][:, :, 0] *= torch.exp2(-torch.randint(0, 40, prob[4].shape[:2]).float())
    _check(fa, prob)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H,Hkv,Nq,room", [(2, 2, 4, 1), (4, 2, 7, 1), (2, 2, 7, 150000), (4, 1, 8, 1), (8, 1, 8, 1)])
@pytest.mark.parametrize("grow", [-40, 12, 25, 45])
def test_value_scales_of_later_tokens_stay_out_of_a_row(fa, d, H, Hkv, Nq, room, grow):
    """Value scales that grow from one new token to the next, to 2^grow and more times the cached
    ones': every row is as exact as if the tokens behind it were not there."""
    lens = [300, 2, Nq, 127 + Nq, 128, 0, 512 + Nq // 2]
    prob = list(_problem(len(lens), H, Hkv, Nq, d, 16, 1, lens, seed=d + Nq, room=room))
    for b, n in enumerate(lens):
        for j in range(max(0, n - Nq), n):
            prob[4][int(prob[5][b, j // 16]), :, j % 16] *= 2.0 ** (grow * (j - n + Nq) / (Nq - 1))
    o, lse = fa.decode_paged_fp8(*[t.to(DEV) for t in prob], causal=True)
    rows = [oracle_decode(prob[0][:, :, i:i + 1], *prob[1:6], (prob[6] - Nq + 1 + i).clamp(min=0), False,
                          d ** -0.5) for i in range(Nq)]
    ref = [np.concatenate([r[k] for r in rows], 2) for k in (0, 1)]
    terms = tuple(np.concatenate([r[2][k] for r in rows], 2) for k in range(3))
    check_decode(o.float().cpu().numpy(), lse.cpu().numpy(), (*ref, terms))
    assert fa.fa_device_status(None) == 0


@pytest.mark.parametrize("exponent", [-126, -100, 90, 120])
def test_last_tokens_of_an_extreme_value_scale(fa, exponent):
    prob = list(_problem(2, 4, 2, 4, 128, 16, 16, [145, 40], seed=22))
    prob[2] &= 0xBF  # codes below 2, so that the outputs fit
    prob[4][int(prob[5][0, 9])] = 2.0 ** exponent  # token 144, alone in its group
    _check(fa, prob, causal=True)
    prob = list(_problem(3, 4, 2, 4, 128, 16, 16, [4, 3, 1], seed=23))  # no key that all rows see
    prob[2] &= 0xBF
    prob[4] = torch.full_like(prob[4], 2.0 ** exponent)
    o, lse = _check(fa, prob, causal=True)
    assert float(o[0, :, 3].float().abs().max()) > 0
    if exponent == -100:  # normal in bf16: as outputs near 1, to which the bound's last term is nothing
        ro, rl, (pv, vmax, qk) = oracle_decode(*prob, True, 128 ** -0.5)
        f = 2.0 ** 100
        check_decode(o.double().cpu().numpy() * f, lse.cpu().numpy(), (ro * f, rl, (pv * f, vmax * f, qk)))


@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("H,Hkv,Nq,causal", [(4, 1, 5, True), (24, 1, 1, False), (32, 2, 2, True), (16, 1, 4, False),
                                             (33, 1, 2, True)])
def test_many_items_of_many_rows(fa, d, H, Hkv, Nq, causal):
    """17 to 66 rows per head and several items per CTA, some of them cut: two and four row
    warpgroups, two row blocks, the queries of the next item prepared ahead."""
    lens = [(b * 37) % 280 for b in range(260)]
    lens[9], lens[100], lens[101], lens[259] = 5000, 12000, 0, 900
    prob = _problem(len(lens), H, Hkv, Nq, d, 32, 16, lens, seed=d + H)
    o, lse = fa.decode_paged_fp8(*[t.to(DEV) for t in prob], causal=causal)
    assert fa.fa_device_status(None) == 0
    some = [9, 100, 101, 259, *range(0, 260, 7)]
    ref = oracle_decode(prob[0][some], *prob[1:5], prob[5][some], prob[6][some], causal, d ** -0.5)
    check_decode(o[some].float().cpu().numpy(), lse[some].cpu().numpy(), ref)


def test_groups_of_zero_scale(fa):
    prob = _problem(2, 4, 2, 1, 128, 16, 16, [300, 140], seed=9)
    for b, n in ((0, 300), (1, 140)):
        prob[3][prob[5][b, 1].long()] = 0.0
        prob[4][prob[5][b, 2].long()] = 0.0
        prob[4][prob[5][b, 0].long()] = 2.0 ** -126
    _check(fa, prob)
    prob[4][:] = 0.0  # every value is zero
    o, _ = _check(fa, prob)
    assert bool((o == 0).all())


def test_nan_and_infinities_stay_in_their_rows(fa):
    prob = list(_problem(3, 4, 2, 1, 128, 16, 16, [200, 300, 20], seed=10))
    prob[0][0, 1, 0, 5] = float("nan")
    prob[0][1, 2, 0, 7] = float("inf")
    prob[1][int(prob[5][2, 0]), 1, 3, 9] = 0x7F  # a NaN key: heads 2 and 3 of sequence 2
    prob[2][int(prob[5][1, 3]), 0, 2, 11] = 0xFF  # a NaN value: column 11, heads 0 and 1 of sequence 1
    o, lse = fa.decode_paged_fp8(*[t.to(DEV) for t in prob])
    o, lse = o.float().cpu(), lse.cpu()
    nan = torch.zeros((3, 4), dtype=torch.bool)
    nan[0, 1] = nan[1, 2] = nan[2, 2] = nan[2, 3] = True
    assert torch.equal(torch.isnan(lse[:, :, 0]), nan)
    expect = nan[:, :, None, None].expand_as(o).clone()
    expect[1, :2, 0, 11] = True
    assert torch.equal(torch.isnan(o), expect)
    assert fa.fa_device_status(None) == 0


@pytest.mark.parametrize("d,room", [(64, 1), (64, 150000), (96, 1), (128, 1), (256, 1)])
@pytest.mark.parametrize("H,Hkv,Nq", [(2, 2, 3), (4, 1, 4), (8, 2, 7), (8, 1, 8)])
def test_causal_rows_are_free_of_later_tokens_nans(fa, d, room, H, Hkv, Nq):
    """NaN codes in K and V of the last Nq tokens: rows before them stay finite."""
    for n in (Nq, 127, 128, 130, 255, 256, 300):
        prob = list(_problem(2, H, Hkv, Nq, d, 16, 16, [n, 40], seed=n + d, room=room))
        table = prob[5]
        hits = [(n - 1, 0, 3), (n - 2, Hkv - 1, d - 1), (n - 2, 0, 0), (n - Nq, 0, d // 2)]
        for key, h, col in hits[:3] if n % 2 else hits:
            prob[2][int(table[0, key // 16]), h, key % 16, col] = 0x7F if col % 2 else 0xFF
        prob[1][int(table[1, 39 // 16]), 0, 39 % 16, 1] = 0x7F  # the last key of sequence 1
        o, lse = fa.decode_paged_fp8(*[t.to(DEV) for t in prob], causal=True)
        ref = oracle_decode(*prob, True, d ** -0.5)
        o, lse = o.float().cpu().numpy(), lse.cpu().numpy()
        assert np.array_equal(np.isnan(o), np.isnan(ref[0])), n
        assert np.array_equal(np.isnan(lse), np.isnan(ref[1])), n
        clean = [np.where(np.isnan(x), 0, x) for x in (o, ref[0], *ref[2][:2])]
        rows = ~np.isnan(ref[1])
        check_decode(clean[0][rows], lse[rows], (clean[1][rows], ref[1][rows],
                                                 (clean[2][rows], clean[3][rows], ref[2][2][rows])))
    assert fa.fa_device_status(None) == 0


@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("H,Hkv,Nq", [(4, 1, 5), (7, 1, 7), (2, 1, 3)])
def test_nan_values_of_many_items_stay_in_their_rows(fa, d, H, Hkv, Nq):
    """20, 49 and 6 rows per head and several items per CTA, whose row warpgroups may be an item
    apart: NaN codes of V among the last Nq tokens of every third sequence and of no other."""
    g = torch.Generator().manual_seed(d + H)
    lens = torch.randint(Nq, 300, (1500,), generator=g).tolist()
    prob = list(_problem(len(lens), H, Hkv, Nq, d, 16, 16, lens, seed=d))
    expect = np.zeros((len(lens), H, Nq, d), dtype=bool)
    for b in range(0, len(lens), 3):
        for back, col in ((1, b % d), (2, (7 * b + 3) % d), (Nq, (5 * b) % d)):
            key = lens[b] - back
            prob[2][int(prob[5][b, key // 16]), 0, key % 16, col] = 0x7F if col % 2 else 0xFF
            expect[b, :, Nq - back:, col] = True
    dev = [t.to(DEV) for t in prob]
    first = None
    for _ in range(20):
        o, lse = fa.decode_paged_fp8(*dev, causal=True)
        if first is None:
            first = (o, lse)
            assert np.array_equal(torch.isnan(o).cpu().numpy(), expect)
            assert not bool(torch.isnan(lse).any())
        assert torch.equal(torch.nan_to_num(o), torch.nan_to_num(first[0])) and torch.equal(lse, first[1])
        assert torch.equal(torch.isnan(o), torch.isnan(first[0]))
    assert fa.fa_device_status(None) == 0
    some = list(range(0, 60)) + list(range(len(lens) - 30, len(lens)))
    ref = oracle_decode(prob[0][some], *prob[1:5], prob[5][some], prob[6][some], True, d ** -0.5)
    o, lse = first[0][some].float().cpu().numpy(), first[1][some].cpu().numpy()
    clean = [np.where(expect[some], 0, x) for x in (o, ref[0], *ref[2][:2])]
    check_decode(clean[0], lse, (clean[1], ref[1], (clean[2], clean[3], ref[2][2])))


@pytest.mark.parametrize("room", [1, 150000])
def test_captured_calls_of_half_rows_follow_the_lengths(fa, room):
    prob = _problem(4, 8, 2, 2, 64, 16, 8, [3000, 1000, 500, 64], seed=21, room=room)
    dev = [t.to(DEV) for t in prob]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = fa.decode_paged_fp8(*dev, causal=True)
    for lens in ([3000, 1000, 500, 64], [1, 0, 500, 63], [0, 0, 0, 0], [257, 998, 129, 1]):
        dev[6].copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        ref = oracle_decode(*prob[:6], torch.tensor(lens), True, 0.125)
        check_decode(o.float().cpu().numpy(), lse.cpu().numpy(), ref, str(lens))
    dev[5][1, 30] = -5
    dev[6].copy_(torch.tensor([3000, 1000, 500, 64], dtype=torch.int32))
    o.fill_(3.0)
    g.replay()
    assert fa.fa_device_status(None) == 7
    assert bool((o[1] == 3.0).all()) and not bool((o[[0, 2, 3]] == 3.0).all())


def test_shared_pages_and_repeated_entries(fa):
    prob = list(_problem(4, 4, 2, 1, 128, 16, 16, [100, 160, 33, 64], seed=11))
    prob[5][1, :6] = prob[5][0, :6]
    prob[5][3, :4] = prob[5][3, 0]
    _check(fa, prob)


def test_outputs_workspace_and_stream_given(fa):
    prob = _problem(3, 8, 2, 1, 128, 16, 16, [4000, 100, 0], seed=12)
    need = fa.fa_decode_paged_fp8_workspace_bytes(3, 8, 2, 1, 128, 16, prob[5].shape[1])
    out = torch.full((3, 8, 1, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.full((3, 8, 1), float("nan"), device=DEV)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o, _ = _check(fa, prob, out=out, lse=lse, workspace=ws[:need], stream=s)
    assert o is out and bool((ws[need:] == 0xFF).all())
    again, _ = fa.decode_paged_fp8(*[t.to(DEV) for t in prob])
    assert torch.equal(again, out)  # the same bits each time
    with pytest.raises(fa.FaError):
        fa.decode_paged_fp8(*[t.to(DEV) for t in prob], workspace=ws[:need - 1])


def test_two_calls_at_once(fa):
    probs = [_problem(2, 8, 8, 1, 128, 16, 16, [5000, 3000], seed=s) for s in (13, 14)]
    dev = [[t.to(DEV) for t in p] for p in probs]
    alone = [fa.decode_paged_fp8(*d) for d in dev]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in dev]
    for _ in range(20):
        both = []
        for d, s in zip(dev, streams):
            with torch.cuda.stream(s):
                both.append(fa.decode_paged_fp8(*d))
        torch.cuda.synchronize()
        for a, b in zip(alone, both):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_captured_calls_follow_the_lengths(fa):
    prob = _problem(4, 8, 2, 2, 128, 16, 16, [3000, 1000, 500, 64], seed=15)
    dev = [t.to(DEV) for t in prob]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = fa.decode_paged_fp8(*dev, causal=True)
    for lens in ([3000, 1000, 500, 64], [1, 0, 500, 63], [2999, 1, 2, 1], [0, 0, 0, 0], [7, 998, 129, 64]):
        dev[6].copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        ref = oracle_decode(*prob[:6], torch.tensor(lens), True, 128 ** -0.5)
        check_decode(o.float().cpu().numpy(), lse.cpu().numpy(), ref, str(lens))
    assert fa.fa_device_status(None) == 0


@pytest.mark.parametrize("entry,length", [(-1, None), (1 << 30, None), (None, -1), (None, 100000)])
def test_bad_index_is_reported_and_writes_nothing(fa, entry, length):
    prob = _problem(3, 4, 2, 1, 128, 16, 16, [2000, 2500, 700], seed=16)
    dev = [t.to(DEV) for t in prob]
    if entry is not None:
        dev[5][1, 100] = entry
    else:
        dev[6][1] = length
    out = torch.full((3, 4, 1, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((3, 4, 1), 3.0, device=DEV)
    fa.decode_paged_fp8(*dev, out=out, lse=lse)
    assert fa.fa_device_status(None) == 7
    assert bool((out[1] == 3.0).all()) and bool((lse[1] == 3.0).all())
    ref = oracle_decode(*prob, False, 128 ** -0.5)
    ok = [0, 2]
    check_decode(out[ok].float().cpu().numpy(), lse[ok].cpu().numpy(),
                 (ref[0][ok], ref[1][ok], tuple(x[ok] for x in ref[2])))


def test_pages_beyond_four_gigabytes(fa):
    """Pages whose bytes lie past 2^32 of the cache."""
    Hkv, ps, d, group = 8, 128, 128, 128
    num = (1 << 32) // (Hkv * ps * d) + 50
    prob = list(_problem(2, 8, 8, 1, d, ps, group, [700, 1000], seed=17))
    used = prob[1].shape[0]
    big = []
    for codes, scale in ((prob[1], prob[3]), (prob[2], prob[4])):
        c = torch.empty((num, Hkv, ps, d), dtype=torch.uint8, device=DEV)
        s = torch.zeros((num, Hkv, 1), device=DEV)
        c[num - used:], s[num - used:] = codes.to(DEV), scale.to(DEV)
        big.append((c, s))
    table = torch.where(prob[5] < used, prob[5] + (num - used), prob[5])
    o, lse = fa.decode_paged_fp8(prob[0].to(DEV), big[0][0], big[1][0], big[0][1], big[1][1],
                                 table.to(DEV), prob[6].to(DEV))
    assert fa.fa_device_status(None) == 0
    check_decode(o.float().cpu().numpy(), lse.cpu().numpy(), oracle_decode(*prob, False, d ** -0.5))


@pytest.mark.parametrize("B,Hkv,group", [(3, 1, 2), (64, 2, 4)])
def test_calls_that_follow_one_another_at_once(fa, B, Hkv, group):
    """Store, attention, page copy and attention with no other kernel between them, so that each
    may start while the one before it ends: the bits of calls that wait for one another, eager and
    replayed.  Magnitudes grow, so that scales beside each other change from step to step."""
    H, d, ps, num, steps = 4 * Hkv, 128, 16, 8 * B, 60
    g = torch.Generator().manual_seed(24)
    table = torch.randperm(4 * B, generator=g).to(torch.int32).reshape(B, 4).to(DEV)
    lens = [torch.full((B,), n, dtype=torch.int32, device=DEV) + (torch.arange(B, device=DEV) % 3).int()
            for n in range(steps + 1)]
    x = torch.randn((steps, B, 2 * Hkv, d), generator=g) * torch.exp2(torch.arange(steps) // 3 % 7)[:, None, None, None]
    x, q = x.to(torch.bfloat16).to(DEV), torch.randn((B, H, 1, d), generator=g).to(torch.bfloat16).to(DEV)
    src, dst = (torch.arange(4 * B, dtype=torch.int32, device=DEV) + k * 4 * B for k in (0, 1))
    later = table + 4 * B

    def caches():
        return [torch.zeros((num, Hkv, ps, d), dtype=torch.uint8, device=DEV) for _ in "kv"] + \
               [torch.zeros((num, Hkv, ps // group), device=DEV) for _ in "kv"]

    def run(c, wait):
        out = []
        for i in range(steps):
            fa.append_paged_fp8(x[i, :, :Hkv], x[i, :, Hkv:], *c, table, lens[i])
            wait()
            out += fa.decode_paged_fp8(q, *c, table, lens[i + 1])
            wait()
            fa.copy_pages(c, src, dst)
            wait()
            out += fa.decode_paged_fp8(q, *c, later, lens[i + 1])
            wait()
        return out

    expect = run(caches(), torch.cuda.synchronize)
    for a, b in zip(expect[0::4] + expect[1::4], expect[2::4] + expect[3::4]):
        assert torch.equal(a, b)  # the copies
    for _ in range(3):
        got = run(caches(), lambda: None)
        assert all(torch.equal(a, b) for a, b in zip(expect, got))
    c = caches()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(c, lambda: None)
    for _ in range(3):
        for t in c:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(expect, got))
    assert fa.fa_device_status(None) == 0


def test_a_serving_loop(fa):
    """Prefill, decode steps, a fork, more steps, a release with compaction, more steps: the
    cache as the oracle keeps it, and attention over it, at every step."""
    from oracle import cache as oc
    H, Hkv, d, ps, group, num, width, layers = 4, 2, 128, 16, 8, 60, 12, 1
    g = torch.Generator().manual_seed(20)
    kc, ks = (t.to(DEV) for t in make_cache(num, Hkv, ps, d, group, 1, pow2=True))
    vc, vs = (t.to(DEV) for t in make_cache(num, Hkv, ps, d, group, 2, pow2=True))
    ref = [t.cpu().numpy() for t in (kc, ks, vc, vs)]
    B = 4  # rows 2 and 3 begin empty
    lens = np.array([37, 16, 0, 0])
    table = np.full((B, width), -1)
    table[0, :5], table[1, :5] = [50, 3, 44, 7, 30], [1, 59, 20, 21, 22]
    dlens = torch.zeros(B, dtype=torch.int32, device=DEV)
    dtable = torch.as_tensor(table, dtype=torch.int32, device=DEV)

    def step(counts):
        cu = np.concatenate(([0], np.cumsum(counts)))
        x = torch.randn((max(1, int(cu[-1])), 2 * Hkv, d), generator=g).to(torch.bfloat16)
        xd = x.to(DEV)
        fa.append_paged_fp8(xd[:, :Hkv], xd[:, Hkv:], kc, vc, ks, vs, dtable, dlens,
                            cu_seqlens=torch.as_tensor(cu, dtype=torch.int32, device=DEV))
        old = dlens.cpu().numpy()
        for i in range(2):
            ref[2 * i], ref[2 * i + 1] = oc.append(x[:, i * Hkv:(i + 1) * Hkv].double().numpy(), ref[2 * i],
                                                   ref[2 * i + 1], dtable.cpu().numpy(), old, cu)
        dlens.add_(torch.as_tensor(counts, dtype=torch.int32, device=DEV))
        for t, r in zip((kc, ks, vc, vs), ref):
            assert np.array_equal(t.cpu().numpy(), r)
        q = torch.randn((B, H, 1, d), generator=g).to(torch.bfloat16)
        o, lse = fa.decode_paged_fp8(q.to(DEV), kc, vc, ks, vs, dtable, dlens)
        check_decode(o.float().cpu().numpy(), lse.cpu().numpy(),
                     oc.decode(q.double().numpy(), ref[0], ref[2], ref[1], ref[3], dtable.cpu().numpy(),
                               dlens.cpu().numpy(), False, d ** -0.5))

    step(lens)
    for _ in range(3):
        step(np.array([1, 1, 0, 0]))
    free, count = fa.free_pages(dtable, dlens, ps, num)
    parents = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    rows, clens, src, dst = fa.fork_pages(dtable, dlens, parents, free[30:32], ps, num)
    fa.copy_pages([kc, ks, vc, vs], src, dst)
    dtable[2:], dlens[2:] = rows, clens
    dtable[2, 3:5], dtable[3, 2:5] = free[32:34], free[34:37]  # room to grow
    for s_, d_ in zip(src.tolist(), dst.tolist()):
        if s_ >= 0:
            for r in ref:
                r[d_] = r[s_]
    for n in ([1, 1, 1, 1], [3, 0, 2, 9], [1, 1, 1, 1]):
        step(np.array(n))
    dlens[1] = 0  # released
    table2, src, dst, counts = fa.compact_pages(dtable, dlens, ps, num)
    fa.copy_pages([kc, ks, vc, vs], src, dst, count=counts[1:])
    for s_, d_ in zip(src.tolist(), dst.tolist()):
        if s_ >= 0:
            for r in ref:
                r[d_] = r[s_]
    dtable.copy_(table2)
    free, _ = fa.free_pages(dtable, dlens, ps, num)
    assert free[0].item() == counts[0].item()
    for b in (0, 2, 3):  # the pages after the last one in use: fresh ones
        need = -(-int(dlens[b]) // ps)
        dtable[b, need:need + 2] = free[2 * b:2 * b + 2]
    for n in ([1, 0, 1, 1], [20, 0, 1, 15], [1, 0, 1, 1]):
        step(np.array(n))
    assert fa.fa_device_status(None) == 0
