"""Pages of a paged cache and the compaction of an accepted path, against
plain statements of the transaction and of the moves."""
import random

import pytest
import torch

import rope_period_truncated_b200 as wp
import serving_ref as ref

pytestmark = pytest.mark.gpu


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _bf16(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def _update(refs, table, lens, parent, keep, new, P):
    out = wp.wp_pages_update(_i32(refs), _i32(table), _i32(lens), _i32(parent), _i32(keep), _i32(new), P)
    return tuple(t.tolist() for t in out)


def _state(rng, B, MP, P, pool, share):
    """Rows over random pages; some pages have a holder elsewhere."""
    order = list(range(pool))
    rng.shuffle(order)
    table, lens, refs, at = [], [], [0] * pool, 0
    for b in range(B):
        n = min(rng.randint(0, MP * P), (pool - at) * P)
        h = -(-n // P)
        table.append(order[at:at + h] + [-1] * (MP - h))
        lens.append(n)
        for p in order[at:at + h]:
            refs[p] = 1 + (rng.random() < share)
        at += h
    return refs, table, lens


@pytest.mark.parametrize("seed", range(12))
@pytest.mark.parametrize("B,MP,P,pool", [(1, 1, 16, 3), (5, 7, 16, 60), (33, 9, 48, 400), (300, 5, 32, 3000), (1100, 2, 16, 9000)])
def test_pages_update_random(B, MP, P, pool, seed):
    rng = random.Random(seed * 1000 + B)
    refs, table, lens = _state(rng, B, MP, P, pool, 0.2 if seed % 2 else 0.0)
    for _ in range(3):
        parent, keep, new = [], [], []
        few = [rng.randrange(B) for _ in range(3)]
        for b in range(B):
            p = rng.choice(few) if rng.random() < 0.4 else b
            k = 0 if rng.random() < 0.1 else rng.choice([lens[p], rng.randint(0, lens[p]), lens[p] // P * P])
            parent.append(p if k or rng.random() < 0.5 else rng.choice([-1, B + 5]))  # not read where nothing is kept
            keep.append(k)
            new.append(min(MP * P, k + rng.choice([0, 1, P, rng.randint(0, 2 * P)])))
        want = ref.pages_update(refs, table, lens, parent, keep, new, P)
        got = _update(refs, table, lens, parent, keep, new, P)
        assert got == want
        refs, table, lens = got[:3]


def test_pages_update_copy_on_write():
    """One partly filled page, held by three rows: the last holder keeps it, also when nobody else is left."""
    P, MP = 16, 3
    refs, table, lens = [3, 0, 0, 0, 0, 0], [[0, -1, -1]] * 3, [10, 10, 10]
    r, t, ln, copies, info = _update(refs, table, lens, [0, 1, 2], [10, 10, 10], [12, 10, 20], P)
    # row 1 does not write, so it is the one that keeps the shared page; rows 0 and 2 copy
    assert copies == [[0, 1, 10], [-1, -1, 0], [0, 2, 10]] and t == [[1, -1, -1], [0, -1, -1], [2, 3, -1]]
    assert r == [1, 1, 1, 1, 0, 0] and ln == [12, 10, 20] and info == [0, 3, 5, 2]
    r, t, ln, copies, info = _update(refs, table, lens, [0, 1, 2], [10, 10, 10], [11, 11, 11], P)
    assert copies == [[-1, -1, 0], [0, 1, 10], [0, 2, 10]] and t[0] == [0, -1, -1] and r == [1, 1, 1, 0, 0, 0]
    # a holder outside the batch: nobody may write into it
    r, t, ln, copies, info = _update([4, 0, 0, 0, 0, 0], table, lens, [0, 1, 2], [10, 10, 10], [11, 11, 11], P)
    assert [c[0] for c in copies] == [0, 0, 0] and r == [1, 1, 1, 1, 0, 0]


def test_pages_update_refuses_as_a_whole():
    P = 16
    refs, table, lens = [1, 1, 0, 0], [[0, -1, -1], [1, -1, -1]], [16, 9]
    short = _update(refs, table, lens, [0, 1], [16, 9], [48, 30], P)
    assert short == (refs, table, lens, [[-1, -1, 0]] * 2, [1, 3, 2, 0])
    for parent, keep, new, rf, tb, ln in [
        ([0, 2], [16, 9], [16, 9], refs, table, lens), ([0, -1], [16, 9], [16, 9], refs, table, lens), ([0, 1], [17, 9], [17, 9], refs, table, lens),
        ([0, 1], [16, -1], [16, 9], refs, table, lens), ([0, 1], [16, 9], [16, 8], refs, table, lens), ([0, 1], [16, 9], [16, 49], refs, table, lens),
        ([0, 1], [16, 9], [16, 9], [1, 1, -1, 0], table, lens), ([0, 1], [16, 9], [16, 9], [1, 0, 0, 0], table, lens),
        ([0, 1], [16, 9], [16, 9], refs, [[4, -1, -1], [1, -1, -1]], lens), ([0, 1], [16, 9], [16, 9], refs, table, [16, 49]),
        ([0, 1], [16, 9], [16, 9], refs, table, [-1, 9]), ([0, 1], [16, 9], [16, 9], refs, [[-1, -1, -1], [1, -1, -1]], lens)]:
        assert _update(rf, tb, ln, parent, keep, new, P) == (rf, tb, ln, [[-1, -1, 0]] * 2, [2, 0, 0, 0])


def test_pages_update_large_pool_and_captured():
    """More pages than one block sees at a time; a captured call replayed on changed inputs."""
    rng = random.Random(3)
    B, MP, P, pool = 40, 60, 16, 70001
    refs, table, lens = _state(rng, B, MP, P, pool, 0.1)
    args = [refs, table, lens, list(range(B)), lens, [min(MP * P, n + 100) for n in lens]]
    dev = [_i32(a) for a in args]
    graph = torch.cuda.CUDAGraph()
    wp.wp_pages_update(*dev, P)
    with torch.cuda.graph(graph):
        out = wp.wp_pages_update(*dev, P)
    graph.replay()
    assert tuple(t.tolist() for t in out) == ref.pages_update(*args, P)
    args[5] = list(lens)
    dev[5].copy_(_i32(lens))
    graph.replay()
    assert tuple(t.tolist() for t in out) == ref.pages_update(*args, P)


@pytest.mark.parametrize("gm", [False, True])
@pytest.mark.parametrize("P,Hkv,d", [(16, 1, 64), (48, 3, 128), (128, 2, 128)])
def test_pages_copy(gm, P, Hkv, d):
    n = 12
    v = _bf16(1, n, Hkv, P, d)
    k = _bf16(2, n, Hkv, d // 16, P, 16) if gm else _bf16(2, n, Hkv, P, d)
    copies = [[0, 5, 1], [3, 7, P], [0, 8, P - 1], [-1, -1, 0], [2, 2, 4], [1, n, 3], [n, 1, 3], [1, 9, P + 1], [1, 10, 0], [4, -2, 5]]
    rows = lambda x: x.permute(0, 1, 3, 2, 4).flatten(3) if x.dim() == 5 else x  # noqa: E731
    k0, v0 = rows(k).clone(), v.clone()
    wp.wp_pages_copy(k, v, _i32(copies))
    for a, b, r in copies[:3]:
        k0[b, :, :r], v0[b, :, :r] = k0[a, :, :r].clone(), v0[a, :, :r].clone()
    assert torch.equal(rows(k), k0) and torch.equal(v, v0)


@pytest.mark.parametrize("gm", [False, True])
@pytest.mark.parametrize("P", [0, 16, 48])
@pytest.mark.parametrize("d,Hkv", [(64, 1), (128, 3)])
def test_kv_compact(gm, P, d, Hkv):
    """Paths of every kind, next to sequences whose length, count, path or page is bad: those stay as they were."""
    cap = 96
    lens = [0, 5, 95, 30, 47, 10, 10, 10, 96, 10, 10, -1]
    paths = [[0, 1, 2, 3], [0, 2, 5, 60], [0], [], list(range(1, 40)), [2, 2], [3, 1], [-1, 2], [0], [0, 86], [0, 1], [0]]
    bad = {5, 6, 7, 8, 9, 10, 11}
    B, A = len(lens), 40
    table = None
    n = B
    if P:
        n = B * cap // P + 1
        table = torch.randperm(n, generator=torch.Generator().manual_seed(2))[:B * cap // P].reshape(B, cap // P).to(torch.int32)
        table[10, 0] = n
    else:
        bad.discard(10)
    v = _bf16(1, n, Hkv, P or cap, d)
    k = _bf16(2, n, Hkv, d // 16, P or cap, 16) if gm else _bf16(2, n, Hkv, P or cap, d)
    rows = lambda x: x.permute(0, 1, 3, 2, 4).flatten(3) if x.dim() == 5 else x  # noqa: E731
    k0, v0 = rows(k).clone(), v.clone()
    at = lambda b, s: (b, s) if table is None else (int(table[b, s // P]), s % P)  # noqa: E731
    for b in range(B):
        if b not in bad:
            for i, t in enumerate(paths[b]):
                (fp, fr), (tp, tr) = at(b, lens[b] + t), at(b, lens[b] + i)
                k0[tp, :, tr], v0[tp, :, tr] = k0[fp, :, fr].clone(), v0[fp, :, fr].clone()
    want = [-1 if b in bad else lens[b] + len(paths[b]) for b in range(B)]
    dev = _i32(lens)
    args = (k, v, dev, _i32([p + [-7] * (A - len(p)) for p in paths]), _i32([len(p) for p in paths]))
    out = wp.wp_kv_compact(*args, block_table=None if table is None else table.cuda(), out=dev)  # the lengths in place
    assert out is dev and out.tolist() == want
    assert torch.equal(rows(k), k0) and torch.equal(v, v0)
    out = wp.wp_kv_compact(k, v, _i32(lens), args[3], _i32([-1] * 6 + [41] * 6), block_table=None if table is None else table.cuda())
    assert out.tolist() == [-1] * B and torch.equal(v, v0)
