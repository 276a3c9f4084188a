"""Rotation of Q and K in one call, both directions, and rotation with
placing in a cache, against the definition in 64 bits."""
import numpy as np
import pytest
import torch

import rope_period_truncated_b200 as wp
from serving_ref import assert_rotation, f64, rotate

pytestmark = pytest.mark.gpu

INTER, HALF, PAIRED = wp.ROPE_INTERLEAVED, wp.ROPE_HALF_SPLIT, wp.ROPE_HALF_SPLIT_PAIRED


def _bf16(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("layout", [INTER, HALF, PAIRED])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("d,rot,B,N,Hq,Hk", [(64, 64, 1, 1, 1, 1), (64, 16, 2, 5, 3, 1), (128, 128, 1, 33, 8, 2), (128, 48, 3, 7, 4, 4),
                                             (128, 112, 1, 2100, 2, 1), (64, 32, 1, 8195, 1, 1)])
def test_rope_qk(layout, inverse, d, rot, B, N, Hq, Hk):
    q, k = _bf16(d + N, B, N, Hq, d), _bf16(d + N + 1, B, N, Hk, d)
    scale, amp = wp.wp_rope_scaling(rot, 1e4, 4.0, 4096)
    pos = torch.randint(0, 200000, (B, N), generator=torch.Generator().manual_seed(N), dtype=torch.int32)
    oq, ok = wp.wp_rope_qk(q, k, 1e4, layout, pos=pos.cuda(), rot_dim=rot, freq_scale=scale, scale_all=0.5, amplitude=amp, inverse=inverse)
    for x, y in ((q, oq), (k, ok)):
        ref, mag = rotate(f64(x), pos.numpy(), 1e4, rot, layout, scale, 0.5, amp, inverse)
        assert_rotation(y, ref, mag)


def test_rope_qk_is_rope_apply_where_both_apply():
    """Whole heads, amplitude 1: the same bits as the package's single-tensor rotation."""
    q, k = _bf16(1, 2, 100, 4, 128), _bf16(2, 2, 100, 2, 128)
    for layout in (INTER, HALF, PAIRED):
        oq, ok = wp.wp_rope_qk(q, k, 1e6, layout, pos0=1000)
        assert torch.equal(oq, wp.wp_rope_apply(q, 1e6, layout, pos0=1000))
        assert torch.equal(ok, wp.wp_rope_apply(k, 1e6, layout, pos0=1000))


def test_rope_qk_views_in_place_and_one_side():
    """Slices of one projection, in place: what lies between is not touched. Heads before tokens in memory. q or k alone."""
    B, N, Hq, Hk, d = 2, 37, 4, 2, 64
    buf = _bf16(5, B, N, Hq + 2 * Hk, d)
    before = buf.clone()
    q, k = buf[:, :, :Hq], buf[:, :, Hq:Hq + Hk]
    oq, ok = wp.wp_rope_qk(q, k, 1e4, HALF, out_q=q, out_k=k, rot_dim=32)
    assert oq.data_ptr() == q.data_ptr() and ok.data_ptr() == k.data_ptr()
    pos = np.broadcast_to(np.arange(N), (B, N))
    ref, mag = rotate(f64(before), pos, 1e4, 32, HALF)
    assert_rotation(buf[:, :, :Hq + Hk], ref[:, :, :Hq + Hk], mag[:, :, :Hq + Hk])
    assert torch.equal(buf[:, :, Hq + Hk:], before[:, :, Hq + Hk:])
    assert torch.equal(buf[..., 32:], before[..., 32:])
    t = before[:, :, :Hq].permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    one, none = wp.wp_rope_qk(t, None, 1e4, HALF, rot_dim=32)
    assert none is None and torch.equal(one, buf[:, :, :Hq])
    none, one = wp.wp_rope_qk(None, before[:, :, Hq:Hq + Hk], 1e4, HALF, rot_dim=32)
    assert none is None and torch.equal(one, buf[:, :, Hq:Hq + Hk])
    wide = before[:, :, :1].expand(B, N, 3, d)  # a broadcast input
    many, _ = wp.wp_rope_qk(wide, None, 1e4, INTER)
    assert torch.equal(many, wp.wp_rope_qk(wide.contiguous(), None, 1e4, INTER)[0])


def test_rope_qk_refuses():
    q = _bf16(1, 1, 4, 2, 64)
    with pytest.raises(wp.WavePruneError):
        wp.wp_rope_qk(q, None, 1e4, PAIRED, out_q=q)
    with pytest.raises(wp.WavePruneError):
        wp.wp_rope_qk(q, q, 1e4, HALF, out_q=q)  # k would read what q writes
    with pytest.raises(ValueError):
        wp.wp_rope_qk(q, None, 1e4, HALF, freq_scale=[1.0] * 31)
    with pytest.raises(ValueError):
        wp.wp_rope_qk(q[..., ::2], None, 1e4, HALF)
    with pytest.raises(TypeError):
        wp.wp_rope_qk(q.float(), None, 1e4, HALF)
    with pytest.raises(ValueError):
        wp.wp_rope_qk(q, None, 1e4, HALF, pos=_i32([[0, 1, 2]]))


@pytest.mark.parametrize("layout", [INTER, HALF, PAIRED])
def test_rope_gradient(layout):
    """The inverse is the gradient: <g, R x> = <R^T g, x> for the rounded outputs, and a central difference of the 64-bit
    rotation along x agrees with it. Rounding: each side's output elements are off by 2^-8 of their size at most."""
    d, rot, amp = 128, 96, 1.25
    x, g, w = _bf16(7, 1, 50, 2, d), _bf16(8, 1, 50, 2, d), _bf16(9, 1, 50, 2, d)
    dx, _ = wp.wp_rope_qk(g, None, 1e6, layout, pos0=900, rot_dim=rot, amplitude=amp, inverse=True)
    pos = 900 + np.arange(50)[None]
    turn = lambda v: rotate(v, pos, 1e6, rot, layout, amp=amp)[0]  # noqa: E731
    X, G, W = f64(x), f64(g), f64(w)
    slope = ((turn(X + 1e-3 * W) - turn(X - 1e-3 * W)) / 2e-3 * G).sum()
    assert abs((f64(dx) * W).sum() - slope) <= 2.0 ** -7 * (np.abs(f64(dx)) * np.abs(W)).sum()
    y, _ = wp.wp_rope_qk(x, None, 1e6, layout, pos0=900, rot_dim=rot, amplitude=amp)
    assert abs((f64(y) * G).sum() - (f64(dx) * X).sum()) <= 2.0 ** -7 * ((np.abs(f64(y)) * np.abs(G)).sum() + (np.abs(f64(dx)) * np.abs(X)).sum())


# ---------------------------------------------------------------------- append


def _cache(seed, n, Hkv, P, d, gm):
    v = _bf16(seed, n, Hkv, P, d)
    k = _bf16(seed + 1, n, Hkv, d // 16, P, 16) if gm else _bf16(seed + 1, n, Hkv, P, d)
    return k, v


def _k_rows(k):
    """[n, Hkv, P, d] whatever the layout."""
    return k.permute(0, 1, 3, 2, 4).flatten(3) if k.dim() == 5 else k


@pytest.mark.parametrize("layout", [INTER, HALF, PAIRED])
@pytest.mark.parametrize("gm", [False, True])
@pytest.mark.parametrize("paged", [0, 16, 48])
@pytest.mark.parametrize("d,rot,Hq,Hkv,T", [(128, 128, 4, 2, 9), (64, 16, 3, 3, 70), (128, 48, 2, 1, 2111)])
def test_rope_append(layout, gm, paged, d, rot, Hq, Hkv, T):
    """Ragged tokens of three sequences, some of them padding or out of range: their slots and everything between stay as
    they were, to the bit."""
    B, cap = 3, 96 * ((T + 95) // 96)
    P = paged or cap
    n_pages = B if not paged else B * cap // P + 2
    k_c, v_c = _cache(T, n_pages, Hkv, P, d, gm)
    table = None
    if paged:
        order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(T))[:B * cap // P]
        table = order.to(torch.int32).reshape(B, cap // P)
        table[1, 0] = -1  # sequence 1 has lost its first page
    g = torch.Generator().manual_seed(T + 3)
    qkv = _bf16(T + 9, T, Hq + 2 * Hkv, d)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    seq = torch.randint(-1, B + 1, (T,), generator=g)
    slot = torch.randperm(cap, generator=g)[:T]
    slot[0], seq[0] = cap, 0        # just outside
    slot[1], seq[1] = -1, 0
    slot[2], seq[2] = cap - 1, 0    # the last one
    slot[3:][slot[3:] == cap - 1] = -1
    pos = torch.randint(0, 1 << 20, (T,), generator=g)
    k0, v0 = _k_rows(k_c).clone(), v_c.clone()
    i32 = lambda t: t.to(torch.int32).cuda()  # noqa: E731
    oq = wp.wp_rope_append(q, k, v, k_c, v_c, i32(pos), i32(seq), i32(slot), 1e6, layout, block_table=None if table is None else table.cuda(),
                           rot_dim=rot, amplitude=1.5)
    refq, magq = rotate(f64(q), pos.numpy(), 1e6, rot, layout, amp=1.5)
    assert_rotation(oq, refq, magq, "q")
    refk, magk = rotate(f64(k), pos.numpy(), 1e6, rot, layout, amp=1.5)
    page, row, tok = [], [], []
    for i in range(T):
        s, t = int(seq[i]), int(slot[i])
        if 0 <= s < B and 0 <= t < cap:
            p = s if table is None else int(table[s, t // P])
            if p >= 0:
                page.append(p), row.append(t % P), tok.append(i)
    assert tok
    got = _k_rows(k_c)
    assert_rotation(got[page, :, row], refk[tok], magk[tok], "k")
    assert torch.equal(v_c[page, :, row], v[tok])
    k0[page, :, row] = got[page, :, row]
    v0[page, :, row] = v_c[page, :, row]
    assert torch.equal(got, k0) and torch.equal(v_c, v0)


def test_rope_append_without_q_and_in_place():
    k_c, v_c = _cache(1, 2, 2, 40, 64, True)
    q, k, v = _bf16(2, 4, 6, 64), _bf16(3, 4, 2, 64), _bf16(4, 4, 2, 64)
    seq, slot, pos = _i32([0, 0, 1, 1]), _i32([5, 6, 0, 39]), _i32([5, 6, 0, 39])
    assert wp.wp_rope_append(None, k, v, k_c, v_c, pos, seq, slot, 1e4, HALF) is None
    ka, va = k_c.clone(), v_c.clone()
    q0 = q.clone()
    assert wp.wp_rope_append(q, k, v, k_c, v_c, pos, seq, slot, 1e4, HALF, out_q=q) is q
    assert torch.equal(k_c, ka) and torch.equal(v_c, va)
    assert torch.equal(q, wp.wp_rope_append(q0, k, v, k_c, v_c, pos, seq, slot, 1e4, HALF))
    with pytest.raises(wp.WavePruneError):
        wp.wp_rope_append(q, k, v, k_c, v_c, pos, seq, slot, 1e4, PAIRED, out_q=q)
    with pytest.raises(ValueError):
        wp.wp_rope_append(q, k, v, k_c, v_c, pos, seq[:3], slot, 1e4, HALF)


def test_rotary_on_another_stream_and_captured():
    q, k = _bf16(11, 1, 300, 4, 128), _bf16(12, 1, 300, 2, 128)
    want = wp.wp_rope_qk(q, k, 1e4, HALF)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = wp.wp_rope_qk(q, k, 1e4, HALF, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = wp.wp_rope_qk(q, k, 1e4, HALF)
    q.copy_(_bf16(13, 1, 300, 4, 128))
    graph.replay()
    assert torch.equal(out[0], wp.wp_rope_qk(q, k, 1e4, HALF)[0])
