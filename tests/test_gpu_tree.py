"""Attention of a tree of drafted tokens over a cache, against the definition
in 64 bits: shapes, layouts, trees, cutoffs, empty rows, garbage where nothing
may be read, bad arguments, streams, graphs, and the operators run together."""
import math
import random

import numpy as np
import pytest
import torch

import rope_period_truncated_b200 as wp
import serving_ref as ref
from serving_ref import assert_tree, f64

pytestmark = pytest.mark.gpu

ODD_CUT = [5, 40, 300, 1100, 2 ** 31 - 1, 0, 63, 130]


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _tree(rng, T, kind):
    if kind == "chain":
        return [t - 1 for t in range(T)]
    if kind == "star":
        return [-1] * T
    return [rng.randint(max(-1, t - 5), t - 1) for t in range(T)]


class Case:
    """Inputs on the GPU, and the rows of every sequence for the reference."""

    def __init__(self, seed, d, Hq, Hkv, T, lens, nodes, P=0, gm=False, kind="random", scale=1.0, ramp=0.0, garbage=float("nan")):
        rng = random.Random(seed)
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)  # noqa: E731
        B = len(lens)
        self.d, self.T, self.B, self.lens, self.nodes = d, T, B, lens, nodes
        self.q = (scale * torch.randn(B, T, Hq, d, generator=g)).to(torch.bfloat16)
        self.parents = [_tree(rng, T, kind) for _ in range(B)]
        for b in range(B):
            self.q[b, nodes[b]:] = garbage
            for t in range(nodes[b], T):
                self.parents[b][t] = rng.choice([-9, 1000, t])  # not used
        total = [a + n for a, n in zip(lens, nodes)]
        self.keys = [(scale * (1 + ramp * torch.arange(n, 0, -1)[None, :, None] / max(n, 1)) * torch.randn(Hkv, n, d, generator=g)).to(torch.bfloat16) for n in total]
        self.vals = [rnd(Hkv, n, d) for n in total]
        cap = max(max(total), 1)
        if P:
            held = [-(-n // P) for n in total]
            n_pages = sum(held) + 2
            order = torch.randperm(n_pages, generator=g).tolist()
            table, at = [], 0
            for h in held:
                table.append(order[at:at + h] + [n_pages + 99] * (max(held + [1]) - h))  # entries behind the end are not read
                at += h
            self.table = _i32(table)
            k, v = (torch.full((n_pages, Hkv, P, d), garbage, dtype=torch.bfloat16) for _ in range(2))
            for b in range(B):
                for j in range(held[b]):
                    m = min(P, total[b] - j * P)
                    k[table[b][j], :, :m], v[table[b][j], :, :m] = self.keys[b][:, j * P:j * P + m], self.vals[b][:, j * P:j * P + m]
        else:
            self.table = None
            k, v = (torch.full((B, Hkv, cap + 3, d), garbage, dtype=torch.bfloat16) for _ in range(2))
            for b in range(B):
                k[b, :, :total[b]], v[b, :, :total[b]] = self.keys[b], self.vals[b]
        self.k = (k.unflatten(-1, (-1, 16)).permute(0, 1, 3, 2, 4).contiguous() if gm else k).cuda()
        self.v = v.cuda()

    def args(self):
        return (self.q.cuda(), self.k, self.v, _i32(self.lens), _i32(self.parents))

    def run(self, cut, **more):
        return wp.wp_decode_tree(*self.args(), n_nodes=_i32(self.nodes), block_table=self.table, group_cut=cut, **more)

    def ref(self, cut, scale=None):
        q = np.nan_to_num(f64(self.q))
        return ref.tree(q, [f64(k) for k in self.keys], [f64(v) for v in self.vals], self.lens, self.nodes, self.parents, cut, scale)


def check(c, cut, tag=""):
    o, lse = c.run(cut)
    assert_tree(o, lse, c.ref(cut), tag)
    assert wp.wp_device_status() == 0


@pytest.mark.parametrize("gm", [False, True])
@pytest.mark.parametrize("P", [0, 16, 48, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_tree_layouts(d, P, gm):
    c = Case(d + P, d, 8, 2, 9, [300, 0, 63, 64, 129], [9, 3, 0, 1, 9], P, gm)
    check(c, ODD_CUT[:d // 16])


@pytest.mark.parametrize("Hq,Hkv,T", [(1, 1, 1), (2, 2, 64), (3, 1, 43), (16, 1, 7), (16, 1, 64), (8, 1, 16), (8, 1, 17), (10, 2, 33), (32, 8, 31)])
def test_tree_heads_and_sizes(Hq, Hkv, T):
    """Rows per KV head from 1 to 1024, on both sides of every tile border."""
    lens = [200, 77]
    c = Case(Hq * 100 + T, 128, Hq, Hkv, T, lens, [T, max(1, T - 5)], 32, Hq % 2 == 0)
    check(c, [160, 5063, 2 ** 31 - 1, 2 ** 31 - 1] * 2)


@pytest.mark.parametrize("length", [1, 15, 16, 62, 63, 64, 65, 127, 128, 191, 255, 256, 257, 511, 1023, 1024, 1025])
def test_tree_lengths(length):
    c = Case(length, 64, 4, 2, 6, [length, length + 58, max(0, length - 3)], [6, 6, 2], 16 if length % 2 else 0, length % 3 == 0)
    check(c, [6, 64, 1000, 2 ** 31 - 1])


@pytest.mark.parametrize("kind", ["chain", "star", "random"])
@pytest.mark.parametrize("cut", [None, [0] * 8, [6, 6, 31, 31, 2 ** 31 - 1, 2, 700, 64], [2 ** 31 - 1] * 8, ODD_CUT])
def test_tree_kinds_and_cutoffs(kind, cut):
    """Chains deeper than the cutoffs: distances between drafted nodes mask groups as well."""
    c = Case(5, 128, 4, 1, 64, [700, 31, 0], [64, 64, 50], 64, True, kind)
    check(c, cut)


@pytest.mark.parametrize("gm", [False, True])
def test_tree_long(gm):
    """Many splits, ragged lengths, a sequence of one node beside long ones; half-split cutoffs at theta 1e6."""
    cut = wp.wp_cutoffs(128, 1e6, wp.ROPE_HALF_SPLIT)[1]
    c = Case(9, 128, 8, 2, 5, [9000, 4097, 12, 6500], [5, 4, 5, 1], 64, gm)
    check(c, [int(w) for w in cut])
    cut = wp.wp_cutoffs(128, 1e6, wp.ROPE_INTERLEAVED)[1]
    check(c, [int(w) for w in cut])


def test_tree_large_logits():
    """Logits over hundreds of base-2 units, growing along the row and against it: the running maximum moves often."""
    for ramp in (0.0, 2.0, -0.9):
        c = Case(11, 128, 4, 2, 7, [1500, 300], [7, 7], 0, False, scale=8.0, ramp=ramp)
        check(c, ODD_CUT)


def test_tree_scale():
    c = Case(12, 64, 4, 4, 3, [100], [3])
    o, lse = c.run(None, softmax_scale=0.5)
    assert_tree(o, lse, c.ref(None, 0.5))


def test_tree_of_one_is_decode():
    """One node after the context is the package's decode at length + 1."""
    B, Hq, Hkv, d, cap = 3, 8, 2, 128, 3000
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(*s, generator=g).to(torch.bfloat16).cuda() for s in ((B, Hq, d), (B, Hkv, cap, d), (B, Hkv, cap, d)))
    lens = _i32([2999, 1, 1500])
    cut = wp.wp_cutoffs(d, 1e4, wp.ROPE_HALF_SPLIT)[1]
    o, lse = wp.wp_decode_tree(q[:, None].contiguous(), k, v, lens, _i32([[-1]] * B), group_cut=cut)
    o2, lse2 = wp.wp_decode(q, k, v, lens + 1, cut)
    # two kernels of the same definition, each within its own tolerance
    assert (o[:, 0].float() - o2.float()).abs().max() <= 2e-2 and (lse[:, :, 0] - lse2).abs().max() <= 2e-3


def test_tree_garbage_is_not_read():
    """What lies behind the last node and in unused q rows may be anything; NaN and infinite keys that a row does not see
    (siblings, groups out of window) do not reach it."""
    c = Case(21, 128, 4, 2, 8, [333, 64], [8, 5], 16, True, "star", garbage=float("inf"))
    check(c, ODD_CUT)
    sib = Case(22, 64, 2, 1, 4, [40], [4], 0, False, "star")
    want = sib.ref([10, 2 ** 31 - 1, 20, 30])
    sib.k[0, :, 42] = float("nan")  # node 2's key: only node 2 sees it
    sib.k[0, :, 3, :16] = float("inf")  # group 0 of a key further away than its cutoff
    o, lse = sib.run([10, 2 ** 31 - 1, 20, 30])
    keep = [0, 1, 3]
    assert_tree(o[:, keep], lse[:, :, keep], (want[0][:, keep], want[1][:, :, keep], want[2][:, keep], want[3][:, :, keep]))
    assert torch.isnan(o[:, 2].float()).all()


def test_tree_bad_sequences_get_nan_rows():
    """A bad length, node count, parent or page: NaN rows for that sequence, the others as without it."""
    c = Case(31, 64, 4, 2, 5, [100, 90, 80, 70, 60, 50, 40], [5] * 7, 16, False)
    good, glse = c.run(None)
    q, k, v, lens, parents = c.args()
    nodes, table = _i32(c.nodes), c.table.clone()
    lens[0], lens[1] = -1, 16 * table.shape[1] - 4
    nodes[2] = 6
    nodes[3] = -1
    parents[4, 3] = 3
    table[5, 2] = table.max() + 1000
    o, lse = wp.wp_decode_tree(q, k, v, lens, parents, n_nodes=nodes, block_table=table)
    assert torch.isnan(o[:6].float()).all() and torch.isnan(lse[:6]).all()
    assert torch.equal(o[6], good[6]) and torch.equal(lse[6], glse[6])
    parents[4, 3], parents[4, 2] = 2, -2
    o, _ = wp.wp_decode_tree(q, k, v, lens, parents, n_nodes=nodes, block_table=table)
    assert torch.isnan(o[4].float()).all()
    assert wp.wp_device_status() == 0


def test_tree_optional_arguments():
    """No node counts (all T), no LSE, given outputs and workspace; a workspace that is too small is refused."""
    c = Case(41, 128, 4, 2, 6, [1500, 20], [6, 6], 0, False)
    want, lse = c.run(ODD_CUT)
    o, none = wp.wp_decode_tree(*c.args(), group_cut=ODD_CUT, want_lse=False)
    assert none is None and torch.equal(o, want)
    need = wp.wp_decode_tree_workspace_bytes(2, 6, 4, 2, 128, c.v.shape[2])
    out, l2, ws = torch.empty_like(want), torch.empty_like(lse), torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    assert need > 0
    o, l = wp.wp_decode_tree(*c.args(), group_cut=ODD_CUT, out=out, lse=l2, workspace=ws)
    assert o is out and l is l2 and torch.equal(out, want) and torch.equal(l2, lse)
    with pytest.raises(wp.WavePruneError):
        wp.wp_decode_tree(*c.args(), workspace=ws[:need - 1])
    with pytest.raises(ValueError):
        wp.wp_decode_tree(*c.args(), group_cut=[1] * 7)
    q, k, v, lens, parents = c.args()
    with pytest.raises(ValueError):
        wp.wp_decode_tree(q, k, v, lens, parents[:, :5].contiguous())
    with pytest.raises(TypeError):
        wp.wp_decode_tree(q.float(), k, v, lens, parents)


def test_tree_repeats_to_the_bit_on_two_streams_and_in_graphs():
    """Two calls at once, two captured graphs replayed in turn with other calls between: the same bits each time."""
    a, b = Case(51, 128, 8, 2, 8, [3000, 900], [8, 6], 64, True), Case(52, 64, 4, 2, 16, [2500], [16], 16, False)
    wa, wb = a.run(ODD_CUT), b.run(None)
    ia, ib = (a.args(), _i32(a.nodes)), (b.args(), _i32(b.nodes))  # held, and in place before the other streams read them
    run = lambda c, i, cut, **more: wp.wp_decode_tree(*i[0], n_nodes=i[1], block_table=c.table, group_cut=cut, **more)  # noqa: E731
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(5):
        got.append((run(a, ia, ODD_CUT, stream=s1), run(b, ib, None, stream=s2)))
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x[0], wa[0]) and torch.equal(x[1], wa[1]) and torch.equal(y[0], wb[0]) and torch.equal(y[1], wb[1])
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga):
        oa = run(a, ia, ODD_CUT)
    with torch.cuda.graph(gb):
        ob = run(b, ib, None)
    for _ in range(3):
        ga.replay()
        gb.replay()
        a.run(None)
    assert torch.equal(oa[0], wa[0]) and torch.equal(ob[0], wb[0]) and torch.equal(ob[1], wb[1])
    ia[0][3].copy_(_i32([100, 600]))  # other lengths in the captured call
    ga.replay()
    assert torch.equal(oa[0], run(a, ia, ODD_CUT)[0])


def test_offsets_beyond_32_bits():
    """A pool whose last pages lie more than 2^32 elements in."""
    n, Hkv, P, d = 131100, 4, 64, 128  # 4.3e9 elements, 8.6 GB a tensor
    c = Case(61, d, 8, Hkv, 4, [150], [4], P, False)
    k, v = (torch.empty(n, Hkv, P, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = _i32([[n - 1, n - 3, n - 2]])
    for j, p in enumerate(table[0].tolist()):
        k[p], v[p] = c.k[int(c.table[0, j])], c.v[int(c.table[0, j])]
    q, _, _, lens, parents = c.args()
    o, lse = wp.wp_decode_tree(q, k, v, lens, parents, block_table=table, group_cut=ODD_CUT)
    assert_tree(o, lse, c.ref(ODD_CUT))
    new = torch.randn(1, Hkv, d, device="cuda").to(torch.bfloat16)
    wp.wp_rope_append(None, new, new, k, v, _i32([0]), _i32([0]), _i32([2 * P + 40]), 1e4, 0, block_table=table)
    assert torch.equal(v[n - 2, :, 40], new[0]) and torch.equal(k[n - 2, :, 40], new[0])
    wp.wp_kv_compact(k, v, _i32([2 * P]), _i32([[40]]), _i32([1]), block_table=table)
    assert torch.equal(v[n - 2, :, 0], new[0])
    wp.wp_pages_copy(k, v, _i32([[n - 2, n - 5, 1]]))
    assert torch.equal(k[n - 5, :, 0], new[0])


def test_speculative_steps_together():
    """Pages, append, tree attention and compaction as a server runs them: three steps of a batch, with a fork and an end on
    the way. After each step every sequence's cache holds exactly the rows it would have had token by token, and the
    attention of each step agrees with the definition."""
    rng, g = random.Random(5), torch.Generator().manual_seed(5)
    B, T, Hq, Hkv, d, P, pool, MP, theta = 4, 6, 4, 2, 64, 16, 64, 8, 1e4
    cut = [int(w) for w in wp.wp_cutoffs(d, theta, wp.ROPE_HALF_SPLIT)[1]]
    kc, vc = torch.full((pool, Hkv, d // 16, P, 16), float("nan"), dtype=torch.bfloat16, device="cuda"), torch.full((pool, Hkv, P, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    refs, table, alloc = _i32([0] * pool), torch.full((B, MP), -1, dtype=torch.int32, device="cuda"), _i32([0] * B)
    content = [0] * B
    model = [(np.zeros((Hkv, 0, d)), np.zeros((Hkv, 0, d))) for _ in range(B)]  # rows per sequence, as appended
    rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)  # noqa: E731

    def rows_of(b, n):
        t = table[b].tolist()
        k = torch.stack([kc[t[j // P], :, :, j % P].flatten(1) for j in range(n)], 1) if n else torch.zeros(Hkv, 0, d)
        v = torch.stack([vc[t[j // P], :, j % P] for j in range(n)], 1) if n else torch.zeros(Hkv, 0, d)
        return f64(k), f64(v)

    parent = list(range(B))
    for step in range(4):
        if step == 0:  # prompts
            nodes, parents, grow = [37, 16, 5, 1], None, [37, 16, 5, 1]
        else:
            nodes = [rng.randint(1, T) for _ in range(B)]
            parents = [_tree(rng, n, "random") + [-1] * (T - n) for n in nodes]
            grow = nodes
        parent = [0, 1, 0, 3] if step == 2 else list(range(B))  # row 2 ends and becomes a fork of row 0
        model = [tuple(x.copy() for x in model[p]) for p in parent]
        content = [content[p] for p in parent]
        new = [n + m for n, m in zip(content, grow)]
        refs, table, alloc, copies, info = wp.wp_pages_update(refs, table, alloc, _i32(parent), _i32(content), _i32(new), P)
        assert info.tolist()[0] == wp.PAGES_OK
        wp.wp_pages_copy(kc, vc, copies)
        depth = [[i for i in range(n)] if parents is None else [len(x) - 1 for x in ref.chains(parents[b], n)] for b, n in enumerate(nodes)]
        seq = [b for b in range(B) for _ in range(nodes[b])]
        slot = [content[b] + t for b in range(B) for t in range(nodes[b])]
        pos = [content[b] + e for b in range(B) for e in depth[b]]
        n = sum(nodes)
        q, k, v = rnd(n, Hq, d).cuda(), rnd(n, Hkv, d).cuda(), rnd(n, Hkv, d).cuda()
        qr = wp.wp_rope_append(q, k, v, kc, vc, _i32(pos), _i32(seq), _i32(slot), theta, wp.ROPE_HALF_SPLIT, block_table=table)
        kr, _ = wp.wp_rope_qk(k[None], None, theta, wp.ROPE_HALF_SPLIT, pos=_i32([pos]))
        kr, vr = f64(kr[0]), f64(v)
        if parents is None:
            at = 0
            for b in range(B):
                model[b] = (kr[at:at + nodes[b]].transpose(1, 0, 2), vr[at:at + nodes[b]].transpose(1, 0, 2))
                at += nodes[b]
            content = new
        else:
            qt = torch.zeros(B, T, Hq, d, dtype=torch.bfloat16, device="cuda")
            at = 0
            full, accepted = [], []
            for b in range(B):
                m = nodes[b]
                qt[b, :m] = qr[at:at + m]
                full.append(tuple(np.concatenate((old, x[at:at + m].transpose(1, 0, 2)), 1) for old, x in zip(model[b], (kr, vr))))
                accepted.append(sorted(rng.choice(ref.chains(parents[b], m))))
                at += m
            o, lse = wp.wp_decode_tree(qt, kc, vc, _i32(content), _i32(parents), n_nodes=_i32(nodes), block_table=table, group_cut=cut)
            assert_tree(o, lse, ref.tree(f64(qt), [x[0] for x in full], [x[1] for x in full], content, nodes, parents, cut), f"step {step}")
            width = max(len(a) for a in accepted)
            got = wp.wp_kv_compact(kc, vc, _i32(content), _i32([a + [-1] * (width - len(a)) for a in accepted]), _i32([len(a) for a in accepted]), block_table=table)
            model = [tuple(np.concatenate((old, x[:, [content[b] + t for t in accepted[b]]]), 1) for old, x in zip(model[b], full[b])) for b in range(B)]
            content = [c + len(a) for c, a in zip(content, accepted)]
            assert got.tolist() == content
        for b in range(B):
            k_now, v_now = rows_of(b, content[b])
            assert np.array_equal(k_now, model[b][0]) and np.array_equal(v_now, model[b][1]), f"step {step} sequence {b}"
        assert sum(refs.tolist()) == int((table >= 0).sum())
    # and everything given back
    refs, table, alloc, copies, info = wp.wp_pages_update(refs, table, alloc, _i32([0] * B), _i32([0] * B), _i32([0] * B), P)
    assert refs.tolist() == [0] * pool and table.unique().tolist() == [-1] and info.tolist() == [0, 0, pool, 0]
