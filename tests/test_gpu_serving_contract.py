"""What the serving calls' contracts say of rows, paths, memory and sizes that
no ordinary step reaches: nodes that are not there, whatever stands in their q;
indices that point outside; streams of the caller's; sizes beyond 32 bits."""
import pytest
import torch

import rope_period_truncated_b200 as wp
from test_gpu_tree import Case, _i32

pytestmark = pytest.mark.gpu

INF = float("inf")


def _unused(c, kind):
    """Writes into the q rows of nodes that are not there."""
    for b, n in enumerate(c.nodes):
        q = c.q[b, n:]
        q.zero_()
        if kind == "one":
            q[..., 5] = 3e38
        elif kind == "all":
            q[:] = 3e38
        elif kind == "inf":
            q[..., 0] = INF
        elif kind == "minus":
            q[..., 17] = -INF
        elif kind == "large":
            q.copy_(torch.linspace(-40, 40, q.numel()).reshape(q.shape))
        elif kind == "nan":
            q[:, ::2] = float("nan")


# few rows: a CTA per unit; whole units of a line of tiles; parts of units. Many rows: one split; several.
ABSENT = [(64, 4, 2, 5, [40, 0, 333, 128], [3, 1, 5, 2], 0),
          (128, 8, 2, 6, [100, 64, 5] * 40 + [700], [6, 2, 1] * 40 + [4], 16),
          (128, 8, 2, 8, [2500, 900, 1300], [7, 8, 1], 64),
          (64, 4, 1, 20, [120, 200], [11, 19], 0),
          (128, 8, 2, 21, [1500, 2300], [20, 3], 16)]


@pytest.mark.parametrize("kind", ["one", "all", "inf", "minus", "nan"])
@pytest.mark.parametrize("d,Hq,Hkv,T,lens,nodes,P", ABSENT)
def test_absent_nodes_are_zero(d, Hq, Hkv, T, lens, nodes, P, kind):
    """Whatever their q holds: a finite value whose products overflow, infinities, NaN."""
    c = Case(d + T, d, Hq, Hkv, T, lens, nodes, P, False)
    _unused(c, kind)
    o, lse = c.run([40, 2 ** 31 - 1, 300, 70] * (d // 64))
    for b, n in enumerate(nodes):
        assert (o[b, n:] == 0).all() and (lse[b, :, n:] == -INF).all(), f"sequence {b}"
        assert torch.isfinite(o[b, :n].float()).all() and torch.isfinite(lse[b, :, :n]).all(), f"sequence {b}"
    assert wp.wp_device_status() == 0


@pytest.mark.parametrize("kind", ["one", "all", "large", "nan"])
@pytest.mark.parametrize("d,Hq,Hkv,T,lens,nodes,P", ABSENT)
def test_absent_nodes_change_nothing(d, Hq, Hkv, T, lens, nodes, P, kind):
    """The rows that are there come out to the bit as with zeros in the unused q."""
    c = Case(d + T, d, Hq, Hkv, T, lens, nodes, P, False)
    cut = [40, 2 ** 31 - 1, 300, 70] * (d // 64)
    _unused(c, "zeros")
    want, wlse = c.run(cut)
    _unused(c, kind)
    o, lse = c.run(cut)
    assert torch.equal(o, want) and torch.equal(lse, wlse)


@pytest.mark.parametrize("d,Hq,Hkv,T", [(128, 8, 2, 21), (64, 4, 1, 10), (128, 8, 2, 9), (64, 3, 1, 43), (128, 8, 2, 5), (64, 3, 1, 7)])
def test_tree_whatever_shared_memory_held(d, Hq, Hkv, T):
    """Row counts that do not fill a warp: the lanes without a row have no say, so a call repeats to the bit whatever the
    calls before it left in shared memory."""
    c = Case(d + T, d, Hq, Hkv, T, [1500, 2300], [T, T], 16, False)
    wide = wp.TREE_MAX_NODES // (Hq // Hkv)  # another row count: its q, k and v lie elsewhere
    before = [Case(7, d, Hq, Hkv, n, [2048, 2048], [n, n], 0, gm, scale=scale)
              for scale in (0.0, 30.0) for n, gm in ((T, False), (T, True), (wide, False))]
    got = []
    for x in before:
        x.run(None)
        got.append(c.run(None))
    for o, lse in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(lse, got[0][1])


@pytest.mark.parametrize("gm", [False, True])
@pytest.mark.parametrize("P", [0, 16])
def test_compaction_of_paths_that_leave_the_cache(P, gm):
    """Paths that increase from entry to entry in places, and lead below key 0 or behind the capacity there: refused whole,
    also in the last row of the block table, whose neighbours are other memory."""
    cap, B = 64, 4
    low = -2 ** 31
    paths = [[0, -1000000, -999999, -999998, 5, 6], [0, low, low + 1, 0, 1, 2], [3, 4, 0, 1, 2, 3], [0, -5, -4, -3, -2, -1]]
    lens = [10, 40, 60, 59]  # with 60 + 4 and 59 + 5 at the capacity
    n = B * cap // P if P else B
    v = torch.randn(n, 2, P or cap, 64, device="cuda").to(torch.bfloat16)
    k = torch.randn(*((n, 2, 4, P or cap, 16) if gm else (n, 2, P or cap, 64)), device="cuda").to(torch.bfloat16)
    k0, v0 = k.clone(), v.clone()
    table = torch.arange(n, dtype=torch.int32, device="cuda").view(B, -1) if P else None
    out = wp.wp_kv_compact(k, v, _i32(lens), _i32(paths), _i32([6] * B), block_table=table)
    assert out.tolist() == [-1] * B and torch.equal(k, k0) and torch.equal(v, v0)
    out = wp.wp_kv_compact(k, v, _i32([58] * B), _i32([[0, 1, 2, 3, 4, 5]] * B), _i32([6] * B), block_table=table)  # up to the last key
    assert out.tolist() == [64] * B and torch.equal(k, k0) and torch.equal(v, v0)


def _bf16(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def test_results_on_another_stream_take_no_memory_still_in_use():
    """A call on a stream of its own, while the current stream has yet to read memory that it has given back; and the other
    way round, a call's result given back while the current stream has yet to read it."""
    shape = (1, 4096, 8, 128)
    x, q, r = _bf16(1, *shape), _bf16(2, *shape), _bf16(3, *shape)
    want_x, want_q = x.clone(), wp.wp_rope_qk(q, None, 1e4, wp.ROPE_HALF_SPLIT)[0]
    y, z, side = torch.empty_like(x), torch.empty_like(x), torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    y.copy_(x)
    del x
    o, _ = wp.wp_rope_qk(q, None, 1e4, wp.ROPE_HALF_SPLIT, stream=side)  # does not wait for the current stream
    torch.cuda.synchronize()
    assert torch.equal(y, want_x) and torch.equal(o, want_q)
    torch.cuda._sleep(200_000_000)
    z.copy_(o)
    del o
    o, _ = wp.wp_rope_qk(r, None, 1e4, wp.ROPE_HALF_SPLIT, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(z, want_q) and torch.equal(o, wp.wp_rope_qk(r, None, 1e4, wp.ROPE_HALF_SPLIT)[0])


def test_given_stream_of_a_captured_fork():
    """Inside a capture, calls on a stream that was forked into it: outputs and workspace are the graph's own."""
    c = Case(3, 128, 8, 2, 8, [3000, 900], [8, 6], 64, True)
    args, nodes = c.args(), _i32(c.nodes)
    want = wp.wp_decode_tree(*args, n_nodes=nodes, block_table=c.table)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        o, lse = wp.wp_decode_tree(*args, n_nodes=nodes, block_table=c.table, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        o.zero_()
        graph.replay()
        other = wp.wp_decode_tree(*args, n_nodes=nodes, block_table=c.table)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1]) and torch.equal(other[0], want[0])


@pytest.mark.parametrize("pool", [6, 9000])
def test_pages_with_counts_near_32_bits(pool):
    """A page that the caller has pinned by the largest count can be kept and given up; one more holder is refused whole."""
    top, P = 2 ** 31 - 1, 16
    refs, table, lens = [0] * pool, [[0, -1], [1, -1]], [16, 16]
    refs[0], refs[1] = top, 1

    def update(refs, parent, keep, new):
        return [t.tolist() for t in wp.wp_pages_update(*(_i32(x) for x in (refs, table, lens, parent, keep, new)), P)]

    one = update(refs, [0, 1], [16, 16], [20, 16])
    assert one[0][:3] == [top, 1, 1] and one[1] == [[0, 2], [1, -1]] and one[4][0] == wp.PAGES_OK
    gone = update(refs, [0, 1], [0, 16], [0, 16])
    assert gone[0][:2] == [top - 1, 1] and gone[4][0] == wp.PAGES_OK
    fork = update(refs, [0, 0], [16, 16], [16, 16])
    assert fork == [refs, table, lens, [[-1, -1, 0]] * 2, [wp.PAGES_BAD_ARGUMENT, 0, 0, 0]]
    less = [top - 1] + refs[1:]
    fork = update(less, [0, 0], [16, 16], [16, 16])
    assert fork[0][:2] == [top, 0] and fork[1] == [[0, -1], [0, -1]] and fork[4][0] == wp.PAGES_OK


def test_sizes_that_do_not_fit_32_bits():
    """A head of 2^32 + 128 dims is no head of 128, nor a block table of 2^32 + 1 rows one of a single row."""
    x = torch.empty(1, 1, 1, 2 ** 32 + 128, dtype=torch.bfloat16, device="cuda")
    for more in ({}, {"out_q": x}):
        with pytest.raises(ValueError, match="32 bits"):
            wp.wp_rope_qk(x, None, 1e4, wp.ROPE_INTERLEAVED, **more)
    with pytest.raises(ValueError, match="32 bits"):
        wp.wp_rope_append(None, x[0], x[0], x, x, _i32([0]), _i32([0]), _i32([0]), 1e4, wp.ROPE_INTERLEAVED)
    del x
    kv, rows = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.empty(2 ** 32 + 1, 1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="32 bits"):
        wp.wp_rope_append(None, rows, rows, kv, kv.clone(), _i32([0]), _i32([0]), _i32([0]), 1e4, wp.ROPE_INTERLEAVED, block_table=table)
    del table
    torch.cuda.empty_cache()
