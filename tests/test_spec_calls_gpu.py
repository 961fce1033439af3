"""The calls of speculative decoding as a program makes them: refusals, streams, graphs, tensor
subclasses, buffers beyond 2^31 elements, and whole steps of several rounds."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from gpu_common import load_fa
from oracle import spec
from spec_common import DEV, check_tree, make_paged, oracle_tree, random_trees

pytestmark = pytest.mark.gpu

BAD_INDEX = 7


@pytest.fixture(scope="module")
def fa():
    return load_fa()


def tree_inputs(lens=(100, 17, 300, 0), H=4, Hkv=2, Nt=9, Nq=9, d=128, page=16, seed=3):
    k, v, table = make_paged(list(lens), Nt, page, Hkv, d, seed)
    q = torch.randn((len(lens), H, Nq, d), generator=torch.Generator().manual_seed(seed)).bfloat16()
    return [q, k, v, table, torch.tensor(lens, dtype=torch.int32), random_trees(len(lens), Nt, seed)]


def dev(ts):
    return [t.to(DEV) if t is not None else None for t in ts]


# -------------------------------------------------------------------- refusals

def test_bad_sequences_write_nothing_and_the_others_all(fa):
    """A bad length, page or parent is recorded and leaves its sequence's rows; also in an item that is
    cut over many CTAs."""
    lens = [100, 5000, 300, 40, 64, 7000]
    q, k, v, table, n, par = tree_inputs(lens)
    good = dev((q, k, v, table, n, par))
    ro, rl = fa.decode_paged_tree(*good)
    assert fa.fa_device_status() == fa.FA_OK

    def bad_call(change, which):
        t2, n2, p2 = table.clone(), n.clone(), par.clone()
        change(t2, n2, p2)
        out, lse = torch.full_like(ro, 7.0), torch.full_like(rl, 7.0)
        fa.decode_paged_tree(*good[:3], t2.to(DEV), n2.to(DEV), p2.to(DEV), out=out, lse=lse)
        assert fa.fa_device_status() == BAD_INDEX and fa.fa_device_status() == fa.FA_OK
        for b in range(len(lens)):
            if b in which:
                assert (out[b] == 7).all() and (lse[b] == 7).all(), b
            else:
                # another cut of the work may round otherwise
                assert torch.allclose(out[b].float(), ro[b].float(), atol=0.05)
                assert torch.allclose(lse[b], rl[b], atol=1e-4)

    def lengths(t, n2, p):
        n2[0], n2[2] = -1, t.shape[1] * 16 + 1

    def pages(t, n2, p):
        t[1, 100], t[3, 1], t[5, 3] = -1, k.shape[0], 1 << 30

    def parents(t, n2, p):
        p[2, 4], p[5, 8], p[4, 0] = 4, 100, 0

    def hidden_parent(t, n2, p):
        p[0, 3], p[0, 5] = -2, 3
    bad_call(lengths, (0, 2))
    bad_call(pages, (1, 3, 5))
    bad_call(parents, (2, 4, 5))
    bad_call(hidden_parent, (0,))


def test_pages_of_places_without_a_node_are_not_looked_at(fa):
    lens = [30, 16]
    q, k, v, table, n, par = tree_inputs(lens, Nt=20, Nq=20)
    par[0, 2:], par[1, 16:] = -2, -2
    ref = oracle_tree(q, k, v, table, lens, par)
    table[0, 2:], table[1, 2:] = -1, 1 << 20
    o, lse = fa.decode_paged_tree(*dev((q, k, v, table[:, :3].contiguous(), n, par)))
    assert fa.fa_device_status() == fa.FA_OK
    check_tree(o, lse, ref)


def test_a_full_table_and_nodes_behind_it(fa):
    """A sequence that fills its table's row exactly; one more node is one too many."""
    lens = [28]
    q, k, v, table, n, par = tree_inputs(lens, Nt=4, Nq=4, page=16)
    o, lse = fa.decode_paged_tree(*dev((q, k, v, table, n, par)))
    check_tree(o, lse, oracle_tree(q, k, v, table, lens, par))
    n += 1
    out = torch.full_like(o, 7.0)
    fa.decode_paged_tree(*dev((q, k, v, table, n, par)), out=out)
    assert fa.fa_device_status() == BAD_INDEX and (out == 7).all()


def test_arguments_that_do_not_fit_are_named(fa):
    q, k, v, table, n, par = dev(tree_inputs())
    call = fa.decode_paged_tree
    for args, match in [
        ((q.float(), k, v, table, n, par), "q must be torch.bfloat16"),
        ((q, k.float(), v, table, n, par), "k_cache must be torch.bfloat16"),
        ((q, k, v[:-1], table, n, par), "v_cache must have shape"),
        ((q, k, v, table.long(), n, par), "block_table must be torch.int32"),
        ((q, k, v, table[:2], n[:2], par), "block_table must be"),
        ((q, k, v, table, n[:2], par), "seq_lens must have shape"),
        ((q, k, v, table, n, par[:, :5].contiguous()), "parents must be"),
        ((q, k, v, table, n, par.T), "parents must be"),
        ((q.transpose(1, 2), k, v, table, n, par), "q must be contiguous"),
        ((q[:, :3].contiguous(), k, v, table, n, par), "Hkv dividing H"),
    ]:
        with pytest.raises(ValueError, match=match):
            call(*args)
    with pytest.raises(fa.FaError):
        call(q, k, v, table, n, par, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(fa.FaError):
        call(q, k, v, table, n, torch.full((4, 300), -1, dtype=torch.int32, device=DEV))
    tok, u = torch.zeros((2, 3), dtype=torch.int32, device=DEV), torch.zeros((2, 3), device=DEV)
    p = torch.rand((2, 3, 10), device=DEV)
    for args, match in [
        ((tok.long(), tok, p, p, u), "tokens must be torch.int32"), ((tok, tok, p.half(), None, u), "target_probs"),
        ((tok, tok[:, :2], p, p, u), "parents must"), ((tok, tok, p, p.bfloat16(), u), "draft_probs must be torch.float32"),
        ((tok, tok, p, p, u[:1]), "uniform must have shape"), ((tok, tok, p[:, :2], None, u), "target_probs must be"),
        ((tok, tok, p.transpose(1, 2), None, u), "target_probs must be contiguous"),
    ]:
        with pytest.raises(ValueError, match=match):
            fa.verify_tree(*args)
    path, count = torch.zeros((4, 9), dtype=torch.int32, device=DEV), torch.ones(4, dtype=torch.int32, device=DEV)
    for args, match in [
        (([k, v[:-1]], table, n, path, count), r"caches\[1\] must have shape"),
        (([k.float()], table, n, path, count), r"caches\[0\] must be torch.bfloat16"),
        (([k], table, n, path[:2], count), "path must be"), (([k], table, n, path, count[:2]), "count must have shape"),
    ]:
        with pytest.raises(ValueError, match=match):
            fa.keep_path(*args)
    with pytest.raises(fa.FaError):
        fa.keep_path([k, k], table, n, path, count)


# --------------------------------------------------------- streams, graphs, subclasses

def verify_inputs(B=3, Nt=7, V=5000, seed=1):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = 2 * torch.randn((B, Nt, V), generator=g, device=DEV)
    p = torch.softmax(x, -1)
    q = torch.softmax(x + 0.5 * torch.randn((B, Nt, V), generator=g, device=DEV), -1)
    par = random_trees(B, Nt, seed).to(DEV)
    rows = q.gather(1, par.clamp(min=0).long()[..., None].expand(B, Nt, V))
    tok = torch.multinomial(rows.reshape(-1, V), 1, generator=g).reshape(B, Nt).int()
    return tok, par, p, q, torch.rand((B, Nt), generator=g, device=DEV)


@pytest.fixture(scope="module")
def calls(fa):
    t, w = dev(tree_inputs()), verify_inputs()
    long = dev(tree_inputs((9000, 3), seed=4))
    path = torch.tensor([[0, 2, 3, -1, -1, -1, -1, -1, -1]] * 4, dtype=torch.int32, device=DEV)
    count = torch.tensor([3, 2, 0, 3], dtype=torch.int32, device=DEV)

    def keep(s):
        c = [t[1].clone(), t[2].clone()]
        torch.cuda.synchronize()
        lens = fa.keep_path(c, t[3], t[4], path, count, stream=s)
        if s is not None:
            torch.cuda.synchronize()
        return lens, *c
    return {"decode_paged_tree": lambda s: fa.decode_paged_tree(*t, stream=s),
            "decode_paged_tree of cut items": lambda s: fa.decode_paged_tree(*long, stream=s),
            "decode_paged_tree of a tensor subclass": lambda s: fa.decode_paged_tree(
                torch.nn.Parameter(t[0], requires_grad=False), *t[1:], stream=s),
            "verify_tree": lambda s: fa.verify_tree(*w, stream=s),
            "verify_tree of a tensor subclass": lambda s: fa.verify_tree(
                torch.nn.Parameter(w[0], requires_grad=False), *w[1:], stream=s),
            "keep_path": keep}


NAMES = ["decode_paged_tree", "decode_paged_tree of cut items", "decode_paged_tree of a tensor subclass",
         "verify_tree", "verify_tree of a tensor subclass", "keep_path"]


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_allocations_belong_to_the_given_stream(fa, calls, name, handle):
    s = torch.cuda.Stream()
    expect = calls[name](None)
    torch.cuda.synchronize()
    torch.cuda.memory._record_memory_history(context=None)
    try:
        got = calls[name](s.cuda_stream if handle else s)
        trace = torch.cuda.memory._snapshot()["device_traces"][0]
    finally:
        torch.cuda.memory._record_memory_history(enabled=None)
    torch.cuda.synchronize()
    streams = [e["stream"] for e in trace if e["action"] == "alloc"]
    if name != "keep_path":  # whose caches this test itself copies
        assert streams and set(streams) == {s.cuda_stream}
    else:
        assert s.cuda_stream in streams
    assert all(torch.equal(a, b) for a, b in zip(expect, got))


@pytest.mark.parametrize("name", NAMES[:5])
def test_two_streams_at_once(fa, calls, name):
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    expect = calls[name](None)
    torch.cuda.synchronize()
    got = [calls[name](s) for _ in range(20) for s in (a, b)]
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(x, y) for x, y in zip(expect, g))


def test_subclasses_give_the_same(fa):
    t, w = dev(tree_inputs()), verify_inputs()
    sub = [torch.nn.Parameter(x, requires_grad=False) for x in t]
    out, lse = torch.empty_like(t[0]), torch.empty(t[0].shape[:3], device=DEV)
    ws = torch.empty(fa.fa_decode_paged_tree_workspace_bytes(4, 4, 2, 9, 9, 128, 16, t[3].shape[1]),
                     dtype=torch.uint8, device=DEV)
    expect = fa.decode_paged_tree(*t, scale=0.1)
    o, _ = fa.decode_paged_tree(*sub, scale=0.1, out=out, lse=lse, workspace=ws)
    assert o is out and torch.equal(out, expect[0]) and torch.equal(lse, expect[1])
    o, _ = fa.decode_paged_tree(*t, scale=0.1, out=out, lse=lse, workspace=ws)
    assert o is out and torch.equal(out, expect[0])
    a = fa.verify_tree(*w, replacement=False)
    b = fa.verify_tree(*(torch.nn.Parameter(x, requires_grad=False) for x in w), replacement=False)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    path, count = a[0][:, :9], a[2]
    lens = torch.tensor([100, 17, 300], dtype=torch.int32, device=DEV)
    c, e = [t[1].clone()], [torch.nn.Parameter(t[1].clone(), requires_grad=False)]
    n = fa.keep_path(c, t[3][:3], lens, path.contiguous(), count)
    m = fa.keep_path(e, t[3][:3], torch.nn.Parameter(lens, requires_grad=False), path.contiguous(), count)
    assert torch.equal(n, m) and torch.equal(c[0], e[0])


def test_outputs_at_any_16_bytes(fa):
    t = dev(tree_inputs())
    expect = fa.decode_paged_tree(*t)
    big = torch.full((t[0].numel() + 24,), 7.0, dtype=torch.bfloat16, device=DEV)
    out = big[8:8 + t[0].numel()].view(t[0].shape)
    need = fa.fa_decode_paged_tree_workspace_bytes(4, 4, 2, 9, 9, 128, 16, t[3].shape[1])
    ws = torch.empty(need + 16, dtype=torch.uint8, device=DEV)[16:]
    fa.decode_paged_tree(*t, out=out, workspace=ws)
    assert torch.equal(out, expect[0]) and (big[:8] == 7).all() and (big[-16:] == 7).all()


def test_a_graph_follows_lengths_and_trees(fa):
    lens, Nt = [100, 17, 300, 0, 4000], 12
    q, k, v, table, n, par = dev(tree_inputs(lens, Nt=Nt, Nq=Nt, H=8))
    fa.decode_paged_tree(q, k, v, table, n, par)
    graphs = []
    for _ in range(2):  # two of them, replayed in turn
        s = torch.cuda.Stream()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            got = fa.decode_paged_tree(q, k, v, table, n, par)
        graphs.append((g, got))
    for step in range(4):
        n.copy_(torch.tensor([[1, 2000, 0, 64, 3][(b + step) % 5] if b != 4 else 3900 - 999 * step
                              for b in range(5)]).int().clamp(max=torch.tensor(lens).int()))
        par.copy_(random_trees(5, Nt, 50 + step, ragged=True))
        expect = fa.decode_paged_tree(q, k, v, table, n, par)
        for g, got in graphs:
            g.replay()
            assert torch.equal(got[0], expect[0]) and torch.equal(got[1], expect[1])
    assert fa.fa_device_status() == fa.FA_OK


# ------------------------------------------------------------------ large buffers

def test_caches_beyond_32_bit_offsets(fa):
    """Pages whose elements lie behind 2^31; the others are never written, nor read."""
    pages, Hkv, page, d, Nt = 40000, 8, 64, 128, 5
    lens = [130, 63]
    k, v = (torch.empty((pages, Hkv, page, d), dtype=torch.bfloat16, device=DEV) for _ in "kv")
    table = torch.tensor([[39999, 5, 36000], [34001, 39998, 0]], dtype=torch.int32)
    g = torch.Generator().manual_seed(1)
    used = table.reshape(-1).long()
    small = [torch.randn((6, Hkv, page, d), generator=g).bfloat16() for _ in "kv"]
    for c, x in zip((k, v), small):
        c[used.to(DEV)] = x.to(DEV)
    q = torch.randn((2, 16, Nt, d), generator=g).bfloat16()
    par = random_trees(2, Nt, 2)
    local = torch.arange(6, dtype=torch.int32).reshape(2, 3)
    n = torch.tensor(lens, dtype=torch.int32)
    o, lse = fa.decode_paged_tree(*dev((q,)), k, v, *dev((table, n, par)))
    check_tree(o, lse, oracle_tree(q, *small, local, lens, par))
    path, count = torch.tensor([[0, 2, 4, -1, -1], [1, 3, -1, -1, -1]], dtype=torch.int32), torch.tensor([3, 2]).int()
    fa.keep_path([k, v], *dev((table, n, path, count)))
    for c, x in zip((k, v), small):
        want = spec.keep(x.view(torch.int16).numpy(), local.numpy(), lens, path.numpy(), count.numpy())
        assert np.array_equal(c[used.to(DEV)].cpu().view(torch.int16).numpy(), want)
    assert fa.fa_device_status() == fa.FA_OK


def test_probabilities_beyond_32_bit_offsets(fa):
    B, Nt, V = 5, 256, 2_000_003  # 2.56e9 elements; the last sequence's rows are the ones in use
    target = torch.zeros((B, Nt, V), dtype=torch.bfloat16, device=DEV)
    tokens = torch.zeros((B, Nt), dtype=torch.int32, device=DEV)
    target[4, 0, 1_999_999], target[4, 255, 2_000_002], target[4, 255, 17] = 1.0, 0.5, 0.5
    target[:4, 0, 5] = 1.0
    parents = torch.full((B, Nt), -2, dtype=torch.int32, device=DEV)
    parents[:, 0], parents[4, 255], tokens[4, 255] = -1, 0, 1_999_999
    u = torch.full((B, Nt), 0.75, device=DEV)
    path, new, count = fa.verify_tree(tokens, parents, target, None, u)
    assert count.tolist() == [1, 1, 1, 1, 2] and path[4, :2].tolist() == [0, 255]
    assert new[4, :2].tolist() == [1_999_999, 2_000_002] and new[:4, 0].tolist() == [5] * 4


# -------------------------------------------------------------------- whole steps

class Model:
    """A toy decoder of two layers without a residual: tokens have fixed keys, values and queries per
    layer, and the last layer's output is turned into probabilities."""

    def __init__(self, V, H, Hkv, d, layers, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.kv = [tuple(torch.randn((V, Hkv, d), generator=g, device=DEV).bfloat16() for _ in "kv")
                   for _ in range(layers)]
        self.q = [torch.randn((V, H, d), generator=g, device=DEV).bfloat16() for _ in range(layers)]
        self.w = torch.randn((H * d, V), generator=g, device=DEV) * 0.2

    def probs(self, o):  # [B, H, n, d] -> [B, n, V]
        return torch.softmax(o.float().transpose(1, 2).flatten(2) @ self.w, -1)


def step(fa, m, caches, table, lens, tokens, parents, uniform, draft):
    """One step of speculative decoding: store the tree's keys and values, attend, verify, keep."""
    B, Nt = tokens.shape
    page = caches[0].shape[2]
    pos = lens[:, None].long() + torch.arange(Nt, device=DEV)[None]
    at, row = table.long().gather(1, pos // page), pos % page
    for i, (k, v) in enumerate(m.kv):
        for c, x in zip(caches[2 * i:2 * i + 2], (k, v)):
            c[at.reshape(-1), :, row.reshape(-1)] = x[tokens.long()].reshape(B * Nt, *x.shape[1:])
        q = m.q[i][tokens.long()].transpose(1, 2).contiguous()
        o, _ = fa.decode_paged_tree(q, *caches[2 * i:2 * i + 2], table, lens, parents)
    path, new, count = fa.verify_tree(tokens, parents, m.probs(o), draft, uniform)
    return path, new, count, fa.keep_path(caches, table, lens, path, count)


def test_steps_of_speculative_decoding(fa):
    """Several rounds, eager and from a graph: the cache always holds the accepted tokens' rows in
    order, as if they had been decoded one by one, and attention over it says the same."""
    V, H, Hkv, d, layers, B, Nt, page, rounds = 50, 4, 2, 64, 2, 3, 8, 16, 5
    m = Model(V, H, Hkv, d, layers, 1)
    width = -(-(rounds * Nt + Nt + 40) // page)
    g = torch.Generator(device=DEV).manual_seed(2)
    perm = torch.randperm(B * width, generator=g, device=DEV).int().reshape(B, width)
    texts = [torch.randint(V, (n,), generator=torch.Generator().manual_seed(n)).tolist() for n in (0, 5, 33)]

    def fresh():
        caches = [torch.zeros((B * width, Hkv, page, d), dtype=torch.bfloat16, device=DEV) for _ in range(2 * layers)]
        for b, text in enumerate(texts):
            for j, t in enumerate(text):
                for i, (k, v) in enumerate(m.kv):
                    caches[2 * i][perm[b, j // page].long(), :, j % page] = k[t]
                    caches[2 * i + 1][perm[b, j // page].long(), :, j % page] = v[t]
        return caches, torch.tensor([len(t) for t in texts], dtype=torch.int32, device=DEV)

    draft = torch.softmax(torch.randn((B, Nt, V), generator=g, device=DEV), -1)
    results = []
    for graphed in (False, True):
        caches, lens = fresh()
        last = torch.tensor([7, 8, 9], dtype=torch.int32, device=DEV)
        tokens, parents = torch.zeros((B, Nt), dtype=torch.int32, device=DEV), torch.zeros((B, Nt), dtype=torch.int32, device=DEV)
        parents.copy_(random_trees(B, Nt, 0))
        uniform = torch.zeros((B, Nt), device=DEV)
        graph = None
        if graphed:
            step(fa, m, caches, perm, lens, tokens, parents, uniform, draft)
            caches, lens = fresh()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                got = step(fa, m, caches, perm, lens, tokens, parents, uniform, draft)
        seqs, log = [list(t) for t in texts], []
        for r in range(rounds):
            gr = torch.Generator(device=DEV).manual_seed(100 + r)
            parents.copy_(random_trees(B, Nt, r, ragged=r == 3).clamp(min=-1 if r != 3 else -2))
            parents[:, 0] = -1
            rows = draft.gather(1, parents.clamp(min=0).long()[..., None].expand(B, Nt, V)).reshape(-1, V)
            tokens.copy_(torch.multinomial(rows, 1, generator=gr).reshape(B, Nt))
            tokens[:, 0] = last
            uniform.copy_(torch.rand((B, Nt), generator=gr, device=DEV))
            if graphed:
                graph.replay()
                path, new, count, n = got
            else:
                path, new, count, n = step(fa, m, caches, perm, lens, tokens, parents, uniform, draft)
            for b in range(B):
                c = int(count[b])
                seqs[b] += [int(tokens[b, j]) for j in path[b, :c].tolist()]
                assert new[b, :c - 1].tolist() == [int(tokens[b, j]) for j in path[b, 1:c].tolist()]
                assert int(n[b]) == len(seqs[b])
                last[b] = new[b, c - 1]
            lens.copy_(n)
            log.append((path.clone(), new.clone(), count.clone()))
            for b, seq in enumerate(seqs):  # the cache is that of the accepted tokens
                j = torch.arange(len(seq), device=DEV)
                for i, kv in enumerate(m.kv):
                    for c, x in zip(caches[2 * i:2 * i + 2], kv):
                        assert torch.equal(c[perm[b].long()[j // page], :, j % page], x[torch.tensor(seq, device=DEV)])
        assert sum(int((x[2] > 1).sum()) for x in log) > 0, "no draft was ever accepted"
        # attention of the next tokens over what was kept, a chain of three
        nxt = torch.randint(V, (B, 3), generator=torch.Generator().manual_seed(9)).to(DEV)
        pos = lens[:, None].long() + torch.arange(3, device=DEV)
        for c, x in zip(caches[:2], m.kv[0]):
            c[perm.long().gather(1, pos // page).reshape(-1), :, (pos % page).reshape(-1)] = x[nxt].reshape(B * 3, Hkv, d)
        q = m.q[0][nxt].transpose(1, 2).contiguous()
        o, lse = fa.decode_paged_tree(q, caches[0], caches[1], perm, lens)
        check_tree(o, lse, oracle_tree(q, caches[0], caches[1], perm, lens.tolist(), None))
        results.append(log)
    for a, b in zip(*results):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert fa.fa_device_status() == fa.FA_OK
