"""The serving calls where they could go wrong beside each other: many ragged
sequences on one line of tiles, row counts on both sides of the choice of
kernel, sequences with nothing to attend, waits that give up, other streams,
and what the binding refuses."""
import random

import pytest
import torch

import rope_period_truncated_b200 as wp
import serving_ref as ref
from serving_ref import assert_tree
from test_gpu_tree import ODD_CUT, Case, _i32, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,T", [(8, 1, 4), (4, 4, 32), (11, 1, 3), (3, 3, 33), (16, 1, 2), (32, 2, 1), (5, 1, 6)])
@pytest.mark.parametrize("lens", [[700, 0, 2100, 64], [1, 60, 350]])
def test_tree_rows_around_the_choice_of_kernel(Hq, Hkv, T, lens):
    """30 to 33 rows per KV head, long and short capacities (a CTA per unit, or tiles dealt out)."""
    c = Case(Hq + T, 64, Hq, Hkv, T, lens, [T, T, max(T - 2, 0), 1][:len(lens)], 16, T % 2 == 0)
    check(c, [20, 500, 2 ** 31 - 1, 90])


@pytest.mark.parametrize("P", [0, 16])
def test_tree_many_sequences(P):
    """More sequences than threads in a CTA and more units than CTAs: several segments per CTA, empty ones between them."""
    rng = random.Random(P)
    B, T = 401, 3
    lens = [rng.choice([0, 0, 1, 5, 127, 128, 129, 700, rng.randint(0, 900)]) for _ in range(B)]
    nodes = [0 if rng.random() < 0.2 else rng.randint(1, T) for _ in range(B)]
    nodes[0] = nodes[B - 1] = 0
    c = Case(71 + P, 64, 4, 2, T, lens, nodes, P, P == 16)
    check(c, [9, 200, 2 ** 31 - 1, 64])


@pytest.mark.parametrize("T,Hq", [(4, 4), (20, 4)])
@pytest.mark.parametrize("cap", [300, 3000])
def test_tree_all_sequences_empty(T, Hq, cap):
    """No sequence has a node: zeros and -inf, whatever lies in the cache."""
    nan = float("nan")
    q, k, v = (torch.full(s, nan, dtype=torch.bfloat16, device="cuda") for s in ((3, T, Hq, 64), (3, 2, cap, 64), (3, 2, cap, 64)))
    parents = torch.full((3, T), 9999, dtype=torch.int32, device="cuda")
    o, lse = wp.wp_decode_tree(q, k, v, _i32([0, 0, 0]), parents, n_nodes=_i32([0, 0, 0]))
    assert (o == 0).all() and (lse == float("-inf")).all()
    o, lse = wp.wp_decode_tree(q, k, v, _i32([0, -1, cap + 1]), parents, n_nodes=_i32([0, 0, 0]))
    assert (o[0] == 0).all() and torch.isnan(o[1:].float()).all() and torch.isnan(lse[1:]).all()
    assert wp.wp_device_status() == 0


@pytest.mark.parametrize("T,Hq,Hkv,lens", [(4, 4, 2, [200, 130]), (4, 4, 2, [2500, 900]), (20, 4, 2, [200, 130]), (20, 4, 2, [2500, 900])])
def test_tree_waits_that_give_up(T, Hq, Hkv, lens):
    """A wait limit that no load can keep: the call ends, the status says so, every row is NaN or right, and the next call is right."""
    c = Case(T, 128, Hq, Hkv, T, lens, [T, T], 16, True)
    want = c.ref(ODD_CUT)
    assert wp.wp_device_status() == 0
    prev = wp.wp_set_wait_limit(1)
    try:
        o, lse = c.run(ODD_CUT)
        assert wp.wp_device_status() == wp.WP_ERR_TIMEOUT
    finally:
        wp.wp_set_wait_limit(prev)
    lost = torch.isnan(lse)
    assert lost.any()
    assert torch.isnan(o.float()).all(-1).transpose(1, 2)[lost].all()
    good, glse = c.run(ODD_CUT)
    assert_tree(good, glse, want)
    assert torch.equal(lse[~lost], glse[~lost]) and torch.equal(o.transpose(1, 2)[~lost], good.transpose(1, 2)[~lost])
    assert wp.wp_device_status() == 0


def test_pages_and_compaction_on_another_stream_and_captured():
    rng = random.Random(8)
    B, MP, P, pool = 6, 9, 16, 90
    refs, lens = [0] * pool, [rng.randint(1, MP * P - 20) for _ in range(B)]
    table, at = [], 0
    for n in lens:
        h = -(-n // P)
        table.append(list(range(at, at + h)) + [-1] * (MP - h))
        for p in range(at, at + h):
            refs[p] = 1
        at += h
    parent = [0, 0, 2, 3, 3, 5]
    keep = [lens[p] for p in parent]
    args = [refs, table, lens, parent, keep, [k + 20 for k in keep]]
    want = ref.pages_update(*args, P)
    dev = [_i32(a) for a in args]
    k, v = (torch.randn(pool, 2, P, 64, device="cuda").to(torch.bfloat16) for _ in range(2))
    k0, v0 = k.clone(), v.clone()
    path, n_keep = _i32([[0, 2, 5]] * B), _i32([3] * B)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = wp.wp_pages_update(*dev, P, stream=side)
    wp.wp_pages_copy(k, v, out[3], stream=side)
    new = wp.wp_kv_compact(k, v, dev[4], path, n_keep, block_table=out[1], stream=side)
    side.synchronize()
    assert tuple(t.tolist() for t in out) == want and new.tolist() == [n + 3 for n in keep]
    k1, v1 = k.clone(), v.clone()
    k.copy_(k0), v.copy_(v0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o2 = wp.wp_pages_update(*dev, P)
        wp.wp_pages_copy(k, v, o2[3])
        n2 = wp.wp_kv_compact(k, v, dev[4], path, n_keep, block_table=o2[1])
    graph.replay()
    assert tuple(t.tolist() for t in o2) == want and torch.equal(n2, new)
    assert torch.equal(k, k1) and torch.equal(v, v1)


def test_compaction_of_a_length_beyond_the_cache():
    k, v = (torch.randn(2, 1, 32, 64, device="cuda").to(torch.bfloat16) for _ in range(2))
    out = wp.wp_kv_compact(k, v, _i32([33, 32]), _i32([[0], [0]]), _i32([0, 0]))
    assert out.tolist() == [-1, 32]


def test_binding_refusals():
    q, kv = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 2, 40, 64, dtype=torch.bfloat16, device="cuda")
    lens, par = _i32([5, 6]), _i32([[-1, 0, 1]] * 2)
    tree = lambda **m: wp.wp_decode_tree(**{**dict(q=q, kcache=kv, vcache=kv.clone(), lens=lens, parents=par), **m})  # noqa: E731
    tree()
    for more, error in [(dict(q=q.half()), TypeError), (dict(q=q[:, :, ::2]), ValueError), (dict(q=q[0]), ValueError), (dict(lens=lens.long()), TypeError),
                        (dict(lens=lens.cpu()), TypeError), (dict(lens=_i32([1])), ValueError), (dict(n_nodes=_i32([1])), ValueError),
                        (dict(kcache=kv[:1]), ValueError), (dict(vcache=kv[:, :, :, :32].contiguous()), ValueError), (dict(block_table=lens), ValueError),
                        (dict(group_cut=[1, 2, 3]), ValueError), (dict(group_cut=[1, 2, 3, 1 << 40]), ValueError), (dict(group_cut=[1, 2, 3, 0.5]), TypeError),
                        (dict(group_cut=[1, 2, 3, -1]), wp.WavePruneError), (dict(softmax_scale="x"), TypeError), (dict(out=q[:1]), ValueError),
                        (dict(out=q), wp.WavePruneError), (dict(lse=torch.zeros(2, 4, 3, device="cuda").half()), TypeError), (dict(workspace=5), TypeError),
                        (dict(kcache=None), TypeError), (dict(stream=7), AttributeError)]:
        with pytest.raises(error):
            tree(**more)
    rope = lambda *a, **m: wp.wp_rope_qk(*a, 1e4, 0, **m)  # noqa: E731
    for a, more, error in [((q, q.float()), {}, TypeError), ((q, q[:1]), {}, ValueError), ((q, None), dict(out_k=q), ValueError),
                           ((q, None), dict(pos=_i32([0, 1])), ValueError), ((q, None), dict(freq_scale=[1.0] * 31), ValueError),
                           ((q, None), dict(rot_dim=24), wp.WavePruneError), ((q, None), dict(freq_scale=["a"] * 32), TypeError),
                           ((q.transpose(2, 3), None), {}, ValueError), ((q, None), dict(pos0=1 << 40), ValueError)]:
        with pytest.raises(error):
            rope(*a, **more)
    with pytest.raises(wp.WavePruneError) as e:
        rope(q, None, rot_dim=8)
    assert e.value.code == wp.WP_ERR_ARG and "wp_rope_qk" in str(e.value)
    with pytest.raises(ValueError):
        wp.wp_pages_copy(kv, kv.clone(), lens[:, None])
    with pytest.raises(ValueError):
        wp.wp_pages_update(lens, par, lens, lens, lens, _i32([1]), 16)
    assert wp.wp_device_status() == 0


@pytest.mark.parametrize("T,Hq", [(3, 4), (20, 4)])
def test_steps_without_waiting_between_them(T, Hq):
    """Each kernel is set up while the one before it ends: thirty steps enqueued at once give what they give one by one."""
    B, Hkv, d, P, MP, pool = 5, 2, 64, 16, 40, 260

    def steps(wait):
        g = torch.Generator(device="cuda").manual_seed(4)
        pause = torch.cuda.synchronize if wait else (lambda: None)
        k, v = (torch.zeros(pool, Hkv, P, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        refs, table = torch.zeros(pool, dtype=torch.int32, device="cuda"), torch.full((B, MP), -1, dtype=torch.int32, device="cuda")
        held, lens = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
        rows, node = torch.arange(B, dtype=torch.int32, device="cuda"), torch.arange(T, dtype=torch.int32, device="cuda")
        seq, parents = rows.repeat_interleave(T), (node - 1).repeat(B, 1)
        path = torch.arange(0, T, 2, dtype=torch.int32, device="cuda").repeat(B, 1)
        outs = []
        for i in range(30):
            q, kn, vn = (torch.randn(B * T, h, d, generator=g, device="cuda").to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
            pause()
            parent = rows if i % 7 else rows.flip(0)
            keep = lens[parent.long()]
            pause()
            refs, table, held, copies, info = wp.wp_pages_update(refs, table, held, parent, keep, keep + T, P)
            pause()
            wp.wp_pages_copy(k, v, copies)
            pause()
            slot = (keep[:, None] + node).flatten()
            qr = wp.wp_rope_append(q, kn, vn, k, v, slot, seq, slot, 1e4, wp.ROPE_HALF_SPLIT, block_table=table)
            pause()
            o, lse = wp.wp_decode_tree(qr.view(B, T, Hq, d), k, v, keep, parents, block_table=table, group_cut=[50, 7, 2 ** 31 - 1, 200])
            pause()
            n_keep = 1 + (rows + i) % path.shape[1]
            lens = wp.wp_kv_compact(k, v, keep, path, n_keep, block_table=table)
            pause()
            back, _ = wp.wp_rope_qk(qr.view(B, T, Hq, d), None, 1e4, wp.ROPE_HALF_SPLIT, pos=slot.view(B, T), inverse=True)
            outs += [o, lse, lens, info, back]
        torch.cuda.synchronize()
        return outs + [k, v, refs, table]

    one, many = steps(True), steps(False)
    assert all(int(i[0]) == wp.PAGES_OK for i in one[3:-4:5])
    for x, y in zip(one, many):
        assert torch.equal(x, y)
    assert torch.isfinite(one[0].float()).all() and wp.wp_device_status() == 0
