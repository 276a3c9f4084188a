"""What the serving and rotary operators are measured on: the cases, their plain torch forms and their definitions in 64 bits.

Five operators, next to the prefill and decode that the package has:
  rope     rotation of Q and K in one call: part of the head, scaled frequencies, both directions (the inverse is the gradient)
  append   rotation of new Q/K rows and their placing, with V, in a contiguous or paged cache
  tree     attention of a tree of drafted tokens over a cache that holds their rows behind the context
  commit   drafted rows appended, then the accepted path moved to the front (compaction)
  pages    one transaction on the pages of many sequences (fork, grow, copy on write, free), then the copies it asks for
"""
import math
import random

import torch

own = False

LAYOUTS = {"interleaved": 0, "half": 1, "paired": 2}
INF = 2 ** 31 - 1


def listed():
    return [
        # one packed training sequence of 32K tokens, rotated in place of the fused projection's Q and K columns
        {"name": "rope_train_32k", "op": "rope", "B": 1, "N": 32768, "Hq": 32, "Hkv": 8, "d": 128, "rot": 128, "theta": 1e6,
         "layout": "half", "factor": 1.0, "orig": 0, "fused": True, "inverse": False, "pos0": 0},
        # the gradient of a small batch whose model rotates half of each head, scaled to four times its context
        {"name": "rope_grad_tiny", "op": "rope", "B": 1, "N": 256, "Hq": 2, "Hkv": 2, "d": 64, "rot": 32, "theta": 1e4,
         "layout": "interleaved", "factor": 4.0, "orig": 4096, "fused": False, "inverse": True, "pos0": 7},
        # a draft step of 16 sequences: 8 new tokens each into a paged, group-major cache
        {"name": "append_draft", "op": "append", "plan": 1, "B": 16, "T": 8, "lo": 1024, "hi": 2048, "Hq": 32, "Hkv": 8, "d": 128,
         "rot": 128, "theta": 1e6, "layout": "half", "factor": 1.0, "orig": 0, "page": 64, "gm": True},
        # five prompts of up to 4K tokens go into an empty paged cache in rows; half of the head rotates, scaled frequencies
        {"name": "append_prompt", "op": "append", "plan": 2, "B": 5, "T": 4001, "lo": 0, "hi": 0, "Hq": 32, "Hkv": 8, "d": 128,
         "rot": 64, "theta": 1e6, "layout": "half", "factor": 4.0, "orig": 8192, "page": 16, "gm": False},
        # the smallest call: one short sequence, four drafted tokens, a contiguous cache
        {"name": "tree_tiny", "op": "tree", "plan": 3, "B": 1, "T": 4, "lo": 201, "hi": 201, "Hq": 2, "Hkv": 2, "d": 64,
         "theta": 1e4, "layout": "interleaved", "scale": 1.0, "page": 0, "gm": False},
        # a few sequences of ordinary length, 16 nodes each, small pages in rows
        {"name": "tree_4k", "op": "tree", "plan": 4, "B": 4, "T": 16, "lo": 2500, "hi": 4096, "Hq": 32, "Hkv": 8, "d": 128,
         "theta": 1e6, "layout": "interleaved", "scale": 1.0, "page": 16, "gm": False},
        # the decode workload's batch (16 sequences of 16K to 32K) with 8 drafted nodes each
        {"name": "tree_32k", "op": "tree", "plan": 5, "B": 16, "T": 8, "lo": 16384, "hi": 32768, "Hq": 32, "Hkv": 8, "d": 128,
         "theta": 1e6, "layout": "half", "scale": 1.0, "page": 64, "gm": True},
        # one long document under position interpolation by 4, a wide tree of 63 nodes
        {"name": "tree_wide_128k", "op": "tree", "plan": 6, "B": 1, "T": 63, "lo": 131001, "hi": 131001, "Hq": 32, "Hkv": 8, "d": 128,
         "theta": 1e6, "layout": "half", "scale": 0.25, "page": 0, "gm": True},
        # the end of a speculative step for 16 sequences
        {"name": "commit_16", "op": "commit", "plan": 7, "B": 16, "T": 16, "lo": 1000, "hi": 2000, "Hq": 32, "Hkv": 8, "d": 128,
         "rot": 128, "theta": 1e6, "layout": "half", "factor": 1.0, "orig": 0, "page": 64, "gm": True},
        # the same for a large batch of short sequences
        {"name": "commit_256", "op": "commit", "plan": 8, "B": 256, "T": 31, "lo": 100, "hi": 500, "Hq": 32, "Hkv": 8, "d": 128,
         "rot": 128, "theta": 1e6, "layout": "interleaved", "factor": 1.0, "orig": 0, "page": 32, "gm": False},
        # a serving step's pages: 16 sequences, a few forks and ends
        {"name": "pages_step", "op": "pages", "plan": 9, "B": 16, "lo": 300, "hi": 2000, "room": 9, "page": 64, "Hkv": 8, "d": 128,
         "pool": 640, "gm": True},
        # a large batch of samples that share their prompts: 256 rows over 40000 small pages
        {"name": "pages_fork_256", "op": "pages", "plan": 10, "B": 256, "lo": 500, "hi": 2000, "room": 33, "page": 16, "Hkv": 2, "d": 64,
         "pool": 40000, "gm": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "tree", "tree", "commit", "pages"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    R = rng.choice([1, 2, 3, 4, 8])
    rotary = {"d": d, "rot": rng.choice([16, 32, 48, d // 2, d, d]), "theta": rng.choice([1e4, 1e6]),
              "layout": rng.choice(["interleaved", "half", "paired"])}
    rotary["factor"], rotary["orig"] = rng.choice([(1.0, 0), (1.0, 0), (2.0, 4096), (8.0, 8192)])
    page, gm = rng.choice([16, 32, 48, 64, 128]), rng.random() < 0.5
    if op == "rope":
        B = rng.choice([1, 2, 3])
        N = _log(rng, 1, 32768 * 40 // (B * Hkv * (R + 1)) if B * Hkv * (R + 1) > 40 else 32768)
        return {"op": op, "B": B, "N": N, "Hq": Hkv * R, "Hkv": Hkv, "fused": rng.random() < 0.5, "inverse": rng.random() < 0.5,
                "pos0": rng.choice([0, 1, 100003]), **rotary}
    if op == "append":
        return {"op": op, "plan": rng.randrange(1 << 20), "B": _log(rng, 1, 32), "T": _log(rng, 1, 500), "lo": rng.randrange(500),
                "hi": 500 + rng.randrange(1000), "Hq": Hkv * R, "Hkv": Hkv, "page": page, "gm": gm, **rotary}
    if op == "commit":
        return {"op": op, "plan": rng.randrange(1 << 20), "B": _log(rng, 1, 128), "T": rng.randint(1, 64), "lo": rng.randrange(300),
                "hi": 300 + rng.randrange(700), "Hq": Hkv * R, "Hkv": Hkv, "page": page, "gm": gm, **rotary}
    if op == "pages":
        B, hi = _log(rng, 1, 200), _log(rng, 17, 2000)
        page = rng.choice([16, 32, 64])
        return {"op": op, "plan": rng.randrange(1 << 20), "B": B, "lo": rng.randint(0, hi), "hi": hi, "room": rng.randint(0, 70),
                "page": page, "Hkv": rng.choice([1, 2]), "d": 64, "pool": 2 * B * ((hi + 70) // page + 3) + rng.randrange(500), "gm": gm}
    B, T = _log(rng, 1, 16), rng.choice([1, rng.randint(1, 16), rng.randint(1, 64)])
    hi = _log(rng, 1, 32768)
    most = max(1, 24_000_000 // (B * Hkv * max(R * T, 8)))
    hi = min(hi, most)
    return {"op": op, "plan": rng.randrange(1 << 20), "B": B, "T": T, "lo": rng.randint(0, hi), "hi": hi, "Hq": Hkv * R, "Hkv": Hkv, "d": d,
            "theta": rotary["theta"], "layout": rng.choice(["interleaved", "half"]), "scale": rng.choice([1.0, 0.25]),
            "page": rng.choice([0, page]), "gm": gm}


# ------------------------------------------------------------- what a case fixes


def _spread(c):
    """Context lengths of the B sequences: from lo to hi, in an order of their own."""
    rng = random.Random(c["plan"])
    B = c["B"]
    lens = [c["lo"] + (c["hi"] - c["lo"]) * b // max(1, B - 1) for b in range(B)]
    rng.shuffle(lens)
    return lens, rng


def _tree_plan(c):
    """lens, n_nodes, parents: random trees, every fourth one a chain; one in three sequences has fewer than T nodes."""
    lens, rng = _spread(c)
    nodes, parents = [], []
    for b in range(c["B"]):
        n = c["T"] if rng.random() < 0.67 else rng.randint(1, c["T"])
        chain = b % 4 == 3
        nodes.append(n)
        parents.append([(t - 1 if chain else rng.randint(max(-1, t - 4), t - 1)) if t < n else -1 for t in range(c["T"])])
    return lens, nodes, parents


def _path_plan(c):
    """A root-to-leaf path of each tree: the accepted nodes."""
    lens, nodes, parents = _tree_plan(c)
    rng = random.Random(c["plan"] + 1)
    paths = []
    for b in range(c["B"]):
        t, path = rng.randrange(nodes[b]), []
        while t >= 0:
            path.append(t)
            t = parents[b][t]
        paths.append(path[::-1])
    return lens, nodes, parents, paths


def _append_plan(c):
    """Context lengths and how many new tokens each sequence has (at most T, ragged)."""
    lens, rng = _spread(c)
    return lens, [c["T"] if c["T"] <= 8 else rng.randint(max(1, c["T"] // 2), c["T"]) for _ in range(c["B"])]


def _pages_plan(c):
    """lens, parent, keep, new_lens: most rows go on, one in six is forked from another row, one in eight ends."""
    lens, rng = _spread(c)
    B = c["B"]
    parent, keep, new = [], [], []
    for b in range(B):
        x = rng.random()
        p = rng.randrange(B) if x < 0.17 else b
        k = max(0, lens[p] - rng.choice([0, 0, 3]))
        parent.append(p)
        keep.append(0 if x > 0.88 else k)
        new.append(0 if x > 0.88 else k + rng.randint(0, c["room"]))
    return lens, parent, keep, new


def _freqs(c):
    """Frequency scale of each channel and the amplitude of a long-context ramp: full rotations over the original length below 1 are
    slowed by `factor`, above 32 kept, a linear ramp between."""
    n = c["rot"] // 2
    if c["factor"] == 1.0:
        return [1.0] * n, 1.0
    out = []
    for i in range(n):
        turns = c["orig"] * c["theta"] ** (-2.0 * i / c["rot"]) / (2 * math.pi)
        keep = min(1.0, max(0.0, (turns - 1.0) / (32.0 - 1.0)))
        out.append((1 - keep) / c["factor"] + keep)
    return out, 0.1 * math.log(c["factor"]) + 1.0


def _cutoffs(c):
    """Group cutoffs: the largest period, rounded down, of the channels that own one of the group's 16 dims."""
    n = c["d"] // 2
    w = [min(INF, math.floor(2 * math.pi / (c["scale"] * c["theta"] ** (-2.0 * i / c["d"])))) for i in range(n)]
    own_of = (lambda k: k // 2) if c["layout"] == "interleaved" else (lambda k: k % n)
    return [max(w[own_of(k)] for k in range(16 * g, 16 * g + 16)) for g in range(c["d"] // 16)]


def _ceil(a, b):
    return -(-a // b)


# ------------------------------------------------------------------------ inputs


def _bf16(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda").to(torch.bfloat16)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cache(c, gen, tokens):
    """K and V storage for sequences of `tokens` tokens, and a block table of shuffled pages (None: contiguous)."""
    B, H, d, G = c["B"], c["Hkv"], c["d"], c["d"] // 16
    if not c["page"]:
        n, P, table = B, max(tokens), None
    else:
        P = c["page"]
        held = [_ceil(t, P) for t in tokens]
        n = sum(held) + 3
        order = torch.randperm(n, generator=gen, device="cuda").tolist()
        rows, at = [], 0
        for h in held:
            rows.append(order[at:at + h] + [-1] * (max(held) - h))
            at += h
        table = _i32(rows)
    k = _bf16(gen, n, H, G, P, 16) if c["gm"] else _bf16(gen, n, H, P, d)
    return k, _bf16(gen, n, H, P, d), table


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": c, "op": c["op"]}
    if c["op"] in ("rope", "append", "commit"):
        s["fscale"], s["amp"] = _freqs(c)
        s["freq"] = torch.tensor([f * c["theta"] ** (-2.0 * i / c["rot"]) for i, f in enumerate(s["fscale"])], dtype=torch.float64, device="cuda")
    if c["op"] == "rope":
        B, N, Hq, Hkv, d = c["B"], c["N"], c["Hq"], c["Hkv"], c["d"]
        if c["fused"]:
            qkv = _bf16(gen, B, N, Hq + 2 * Hkv, d)
            s["q"], s["k"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv]
        else:
            s["q"], s["k"] = _bf16(gen, B, N, Hq, d), _bf16(gen, B, N, Hkv, d)
        s["pos"] = (c["pos0"] + torch.arange(N, device="cuda", dtype=torch.int32)).expand(B, N).contiguous()
    elif c["op"] in ("append", "commit"):
        if c["op"] == "append":
            lens, new = _append_plan(c)
            depth = [range(n) for n in new]
        else:
            lens, new, parents, paths = _path_plan(c)
            depth = []
            for n, par in zip(new, parents):
                dep = []
                for t in range(n):
                    dep.append(0 if par[t] < 0 else dep[par[t]] + 1)
                depth.append(dep)
            s["lens"], s["nodes"], s["n_keep"] = _i32(lens), _i32(new), _i32([len(p) for p in paths])
            s["path"] = _i32([p + [-1] * (c["T"] - len(p)) for p in paths])
        s["kc"], s["vc"], s["table"] = _cache(c, gen, [a + n for a, n in zip(lens, new)])
        s["seq"] = _i32([b for b, n in enumerate(new) for _ in range(n)])
        s["slot"] = _i32([a + t for a, n in zip(lens, new) for t in range(n)])
        s["pos"] = _i32([a + t for a, dep in zip(lens, depth) for t in dep])
        T = sum(new)
        qkv = _bf16(gen, T, c["Hq"] + 2 * c["Hkv"], c["d"])
        s["q"], s["k"], s["v"] = qkv[:, :c["Hq"]], qkv[:, c["Hq"]:c["Hq"] + c["Hkv"]], qkv[:, c["Hq"] + c["Hkv"]:]
    elif c["op"] == "tree":
        lens, nodes, parents = _tree_plan(c)
        s["kc"], s["vc"], s["table"] = _cache(c, gen, [a + n for a, n in zip(lens, nodes)])
        s["q"] = _bf16(gen, c["B"], c["T"], c["Hq"], c["d"])
        s["lens"], s["nodes"], s["parents"], s["cut"] = _i32(lens), _i32(nodes), _i32(parents), _cutoffs(c)
    else:
        lens, parent, keep, new = _pages_plan(c)
        P = c["page"]
        most = max(1, max(_ceil(x, P) for x in lens + new))
        order = torch.randperm(c["pool"], generator=gen, device="cuda")
        held = [_ceil(x, P) for x in lens]
        at = 0
        table = torch.full((c["B"], most), -1, dtype=torch.int32, device="cuda")
        for b, h in enumerate(held):
            table[b, :h] = order[at:at + h].to(torch.int32)
            at += h
        refs = torch.zeros(c["pool"], dtype=torch.int32, device="cuda")
        refs[order[:at]] = 1
        refs[order[:at:7]] += 1  # a prefix cache holds some of them as well
        s.update(refs=refs, table=table, lens=_i32(lens), parent=_i32(parent), keep=_i32(keep), new=_i32(new))
        s["vc"] = _bf16(gen, c["pool"], c["Hkv"], P, c["d"])
        s["kc"] = _bf16(gen, c["pool"], c["Hkv"], c["d"] // 16, P, 16) if c["gm"] else _bf16(gen, c["pool"], c["Hkv"], P, c["d"])
    return s


# --------------------------------------------------------------------- plain form


def _rotate(x, pos, freq, amp, rot, layout, inverse):
    """x [..., tokens, H, d] in 32 bits, pos [..., tokens]: angles in 64 bits, the rotation in 32."""
    ang = pos[..., None].double() * freq
    cos, sin = (torch.cos(ang) * amp).float()[..., None, :], (torch.sin(ang) * amp).float()[..., None, :]
    if inverse:
        sin = -sin
    r, n = x[..., :rot], rot // 2
    pairs_in = layout == "interleaved" or (layout == "paired" and inverse)
    pairs_out = layout == "interleaved" or (layout == "paired" and not inverse)
    a, b = (r[..., 0::2], r[..., 1::2]) if pairs_in else (r[..., :n], r[..., n:])
    u, v = a * cos - b * sin, a * sin + b * cos
    r = torch.stack((u, v), -1).flatten(-2) if pairs_out else torch.cat((u, v), -1)
    return torch.cat((r, x[..., rot:]), -1)


def _place(s, seq, slot):
    """Page and row within the page of each token."""
    P = s["vc"].shape[2]
    seq, slot = seq.long(), slot.long()
    return (seq, slot) if s["table"] is None else (s["table"][seq, slot // P].long(), slot % P)


def _put(s, page, row, k, v):
    """Rows k, v [n, Hkv, d] into the caches."""
    if s["case"]["gm"]:
        s["kc"][page, :, :, row] = k.reshape(k.shape[0], k.shape[1], -1, 16)
    else:
        s["kc"][page, :, row] = k
    s["vc"][page, :, row] = v


def _plain_append(s):
    c = s["case"]
    turn = lambda x: _rotate(x.float(), s["pos"], s["freq"], s["amp"], c["rot"], c["layout"], False).to(torch.bfloat16)  # noqa: E731
    page, row = _place(s, s["seq"], s["slot"])
    _put(s, page, row, turn(s["k"]), s["v"])
    return turn(s["q"])


def _plain_commit(s):
    _plain_append(s)
    B, A = s["path"].shape
    i = torch.arange(A, device="cuda")
    ok = i < s["n_keep"][:, None]
    rows = torch.arange(B, device="cuda")[:, None].expand(B, A).reshape(-1)
    # behind the path: the last node's row onto itself (that slot is a target only where the path holds every node, in place)
    still = s["nodes"][:, None] - 1
    fp, fr = _place(s, rows, (s["lens"][:, None] + torch.where(ok, s["path"], still)).reshape(-1))
    tp, tr = _place(s, rows, (s["lens"][:, None] + torch.where(ok, i, still)).reshape(-1))
    k = s["kc"][fp, :, :, fr].flatten(2) if s["case"]["gm"] else s["kc"][fp, :, fr]
    _put(s, tp, tr, k, s["vc"][fp, :, fr])
    return s["lens"] + s["n_keep"]


def _ancestors(parents, nodes):
    """[B, T, T]: is u the node t or above it? Doubling of the one-step relation."""
    B, T = parents.shape
    t = torch.arange(T, device=parents.device)
    step = (parents[:, :, None] == t).float()
    up = torch.eye(T, device=parents.device) + step
    reach = 1
    while reach < T:
        up = ((up @ up) > 0).float()
        reach *= 2
    return (up > 0) & (t < nodes[:, None])[:, :, None] & (t < nodes[:, None])[:, None, :]


def _rows_of(s, L):
    """The first L keys of every sequence as [B, Hkv, L, d]."""
    k, v, c = s["kc"], s["vc"], s["case"]
    if s["table"] is not None:
        page = s["table"].clamp(min=0).long()
        k, v = k[page].transpose(1, 2), v[page].transpose(1, 2)  # [B, Hkv, pages, ...]
        k = k.transpose(3, 4).flatten(4) if c["gm"] else k
        return k.flatten(2, 3)[:, :, :L], v.flatten(2, 3)[:, :, :L]
    k = k.transpose(2, 3).flatten(3) if c["gm"] else k
    return k[:, :, :L], v[:, :, :L]


def _plain_tree(s):
    c = s["case"]
    B, T, Hq, d = s["q"].shape
    H = c["Hkv"]
    P = s["vc"].shape[2]
    L = P if s["table"] is None else P * s["table"].shape[1]
    k, v = _rows_of(s, L)
    lens, nodes = s["lens"].long()[:, None], s["nodes"].long()[:, None]
    j = torch.arange(L, device="cuda")[None]
    used = j < lens + nodes
    v = torch.where(used[:, None, :, None], v.float(), 0.0)
    up = _ancestors(s["parents"], s["nodes"])
    depth = (up.sum(-1) - 1).clamp(min=0)
    node = (j - lens).clamp(0, T - 1)
    kpos = torch.where(j < lens, j, lens + depth.gather(1, node))
    see = (j < lens)[:, None] | (up.gather(2, node[:, None].expand(B, T, L)) & (used & (j >= lens))[:, None])
    live = torch.arange(T, device="cuda") < nodes
    see = see & live[:, :, None]
    dist = (lens + depth)[:, :, None] - kpos[:, None]
    q = s["q"].float().reshape(B, T, H, Hq // H, d).permute(0, 2, 3, 1, 4).reshape(B, H, -1, d)
    logit = None
    for g, w in enumerate(s["cut"]):
        part = (q[..., 16 * g:16 * g + 16] @ k[..., 16 * g:16 * g + 16].float().transpose(2, 3)).reshape(B, H, Hq // H, T, L)
        part = torch.where((dist <= w)[:, None, None], part, 0.0)
        logit = part if logit is None else logit + part
    logit = torch.where(see[:, None, None], logit / math.sqrt(d), -math.inf)
    top = logit.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(logit - top)
    total = p.sum(-1, keepdim=True)
    o = (p.reshape(B, H, -1, L) @ v).reshape(B, H, Hq // H, T, d) / torch.where(total == 0, 1.0, total)
    lse = (top + torch.log(total))[..., 0].reshape(B, Hq, T)
    return o.permute(0, 3, 1, 2, 4).reshape(B, T, Hq, d).to(torch.bfloat16), lse


def _plain_pages(s):
    refs, table, lens, parent, keep, new = (s[n] for n in ("refs", "table", "lens", "parent", "keep", "new"))
    P = s["case"]["page"]
    B, most = table.shape
    pool = refs.numel()
    cols, rows = torch.arange(most, device="cuda"), torch.arange(B, device="cuda")
    up = lambda x: (x + P - 1) // P  # noqa: E731
    r = refs.clone()
    r.scatter_add_(0, table.clamp(min=0).long().reshape(-1), -(cols < up(lens)[:, None]).int().reshape(-1))
    src = table[parent.long()]
    kept, wanted = up(keep), up(new)
    r.scatter_add_(0, src.clamp(min=0).long().reshape(-1), (cols < kept[:, None]).int().reshape(-1))
    # the last kept page, where it is partly filled and will be written: its own, or a copy while somebody else holds it
    last = src.gather(1, (kept - 1).clamp(min=0).long()[:, None])[:, 0].clamp(min=0).long()
    writes = (new > keep) & (keep % P != 0)
    writers = torch.zeros_like(r).scatter_add_(0, last, writes.int())
    first = torch.full_like(r, B).scatter_reduce_(0, last, torch.where(writes, rows, B).int(), "amin")
    copy = writes & (r[last] > 1) & ~((writers[last] == r[last]) & (first[last] == rows))
    r.scatter_add_(0, last, -copy.int())
    need = wanted - kept + copy.int()
    off = torch.cumsum(need, 0) - need
    total = need.sum()
    free = r == 0
    rank = torch.cumsum(free, 0) - 1
    order = torch.zeros(pool + 1, dtype=torch.int64, device="cuda").scatter_(0, torch.where(free, rank, pool), torch.arange(pool, device="cuda"))
    r = torch.where(free & (rank < total), 1, r)
    base = kept - copy.int()
    fresh = order[(off[:, None] + cols - base[:, None]).clamp(0, pool)].int()
    out = torch.where(cols < base[:, None], src, torch.where(cols < wanted[:, None], fresh, -1))
    dst = order[off.clamp(max=pool).long()].int()
    copies = torch.stack((torch.where(copy, last.int(), -1), torch.where(copy, dst, -1), torch.where(copy, keep % P, 0)), 1).int()
    info = torch.stack((torch.zeros_like(total), total, free.sum(), copy.sum())).int()
    # the copies: the kept rows of each copied page, in the K and the V pool
    at = torch.arange(P, device="cuda").expand(B, P)
    take = copy[:, None] & (at < (keep % P)[:, None])
    held = torch.argmin(free.int())  # a page that nobody takes: onto itself where nothing is copied
    a, b = (torch.where(take, x[:, None].long(), held).reshape(-1) for x in (copies[:, 0], copies[:, 1]))
    row = at.reshape(-1)
    if s["case"]["gm"]:
        s["kc"][b, :, :, row] = s["kc"][a, :, :, row]
    else:
        s["kc"][b, :, row] = s["kc"][a, :, row]
    s["vc"][b, :, row] = s["vc"][a, :, row]
    return r, out, new.clone(), copies, info


# ---------------------------------------------------------------------------- run


def _own_append(s, wp):
    c = s["case"]
    return wp.wp_rope_append(s["q"], s["k"], s["v"], s["kc"], s["vc"], s["pos"], s["seq"], s["slot"], c["theta"], LAYOUTS[c["layout"]],
                             block_table=s["table"], rot_dim=c["rot"], freq_scale=s["fscale"], amplitude=s["amp"])


def run(state):
    s, c = state, state["case"]
    if own:
        import rope_period_truncated_b200 as wp
        if s["op"] == "rope":
            return wp.wp_rope_qk(s["q"], s["k"], c["theta"], LAYOUTS[c["layout"]], pos=s["pos"], rot_dim=c["rot"], freq_scale=s["fscale"],
                                 amplitude=s["amp"], inverse=c["inverse"])
        if s["op"] == "append":
            return _own_append(s, wp), s["kc"], s["vc"]
        if s["op"] == "tree":
            return wp.wp_decode_tree(s["q"], s["kc"], s["vc"], s["lens"], s["parents"], n_nodes=s["nodes"], block_table=s["table"],
                                     group_cut=s["cut"])
        if s["op"] == "commit":
            _own_append(s, wp)
            return wp.wp_kv_compact(s["kc"], s["vc"], s["lens"], s["path"], s["n_keep"], block_table=s["table"]), s["kc"], s["vc"]
        out = wp.wp_pages_update(s["refs"], s["table"], s["lens"], s["parent"], s["keep"], s["new"], c["page"])
        wp.wp_pages_copy(s["kc"], s["vc"], out[3])
        return (*out, s["kc"], s["vc"])
    if s["op"] == "rope":
        return tuple(_rotate(x.float(), s["pos"], s["freq"], s["amp"], c["rot"], c["layout"], c["inverse"]).to(torch.bfloat16)
                     for x in (s["q"], s["k"]))
    if s["op"] == "append":
        return _plain_append(s), s["kc"], s["vc"]
    if s["op"] == "tree":
        return _plain_tree(s)
    if s["op"] == "commit":
        return _plain_commit(s), s["kc"], s["vc"]
    return (*_plain_pages(s), s["kc"], s["vc"])


# --------------------------------------------------------------------------- work


def _attended(c):
    """Per sequence: total keys, and the keys of each group that some node's window holds (the bytes and products that count)."""
    lens, nodes, parents = _tree_plan(c)
    cut = _cutoffs(c)
    for L, n, par in zip(lens, nodes, parents):
        dep = []
        for t in range(n):
            dep.append(0 if par[t] < 0 else dep[par[t]] + 1)
        # context keys in the window of a node at depth e: those at distance L + e - j <= w
        inside = [[min(L, max(0, w - e)) for e in dep] for w in cut]
        pairs = n * L + sum(e + 1 for e in dep)
        yield L, n, [max(x) for x in inside], [sum(x) + sum(min(e + 1, w + 1) for e in dep) for x, w in zip(inside, cut)], pairs


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["B"] * c["N"] * (c["Hq"] + c["Hkv"]) * c["d"]
        return {"bytes": 4 * n + 4 * c["B"] * c["N"], "flops": 3 * n * c["rot"] / c["d"]}
    if c["op"] in ("append", "commit"):
        T = sum(_append_plan(c)[1] if c["op"] == "append" else _tree_plan(c)[1])
        n = T * (c["Hq"] + 2 * c["Hkv"]) * c["d"]
        moved = 0 if c["op"] == "append" else sum(sum(i != t for i, t in enumerate(p)) for p in _path_plan(c)[3])
        return {"bytes": 4 * n + 12 * T + 8 * moved * c["Hkv"] * c["d"], "flops": 3 * T * (c["Hq"] + c["Hkv"]) * c["rot"]}
    if c["op"] == "tree":
        bytes_, flops = 4 * c["B"] * c["T"] * c["Hq"] * c["d"] + 4 * c["B"] * c["T"] * c["Hq"], 0
        for L, n, keys, products, pairs in _attended(c):
            bytes_ += c["Hkv"] * (sum(32 * (x + n) for x in keys) + 2 * c["d"] * (L + n))
            flops += c["Hq"] * (32 * sum(products) + 2 * c["d"] * pairs)
        return {"bytes": bytes_, "flops": flops}
    lens, parent, keep, new = _pages_plan(c)
    P = c["page"]
    most = max(1, max(_ceil(x, P) for x in lens + new))
    # at most: every forked row that goes on in a partly filled page copies its rows there
    copied = sum(k % P for b, (p, k, n) in enumerate(zip(parent, keep, new)) if p != b and n > k)
    return {"bytes": 8 * c["pool"] + 8 * c["B"] * most + 36 * c["B"] + 8 * copied * c["Hkv"] * c["d"], "flops": 0}


# -------------------------------------------------------------------------- exact


def _exact_rotation(x, pos, c, fscale, amp, inverse):
    """Each pair of a head as a complex number, times exp(i angle) and the amplitude, one channel at a time."""
    x, out = x.double(), x.double().clone()
    n = c["rot"] // 2
    for i in range(n):
        f = fscale[i] * math.exp(-2.0 * i / c["rot"] * math.log(c["theta"]))
        ang = (-1.0 if inverse else 1.0) * pos.double() * f
        w = torch.polar(torch.full_like(ang, amp), ang)[..., None]
        split, pair = (i, n + i), (2 * i, 2 * i + 1)
        src = pair if c["layout"] == "interleaved" or (c["layout"] == "paired" and inverse) else split
        dst = pair if c["layout"] == "interleaved" or (c["layout"] == "paired" and not inverse) else split
        z = torch.complex(x[..., src[0]], x[..., src[1]]) * w
        out[..., dst[0]], out[..., dst[1]] = z.real, z.imag
    return out


def _exact_put(s, kc, vc, b, slot, k, v):
    P = vc.shape[2]
    page, row = (b, slot) if s["table"] is None else (s["host_table"][b][slot // P], slot % P)
    if s["case"]["gm"]:
        kc[page, :, :, row] = k.reshape(k.shape[0], -1, 16)
    else:
        kc[page, :, row] = k
    vc[page, :, row] = v


def _exact_get(s, kc, vc, b, slot):
    P = vc.shape[2]
    page, row = (b, slot) if s["table"] is None else (s["host_table"][b][slot // P], slot % P)
    return (kc[page, :, :, row].reshape(kc.shape[1], -1) if s["case"]["gm"] else kc[page, :, row]).clone(), vc[page, :, row].clone()


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "rope":
        return tuple(_exact_rotation(x, s["pos"], c, s["fscale"], s["amp"], c["inverse"]) for x in (s["q"], s["k"]))
    if c["op"] in ("append", "commit"):
        T = s["q"].shape[0]
        q, k = (_exact_rotation(x, s["pos"], c, s["fscale"], s["amp"], False) for x in (s["q"], s["k"]))
        kc, vc = s["kc"].double(), s["vc"].double()
        s["host_table"] = None if s["table"] is None else s["table"].tolist()
        if T > 4096:  # one index per token instead of a loop
            P = vc.shape[2]
            slot = s["slot"].long()
            page, row = s["table"][s["seq"].long(), torch.div(slot, P, rounding_mode="floor")].long(), slot.remainder(P)
            if c["gm"]:
                kc[page, :, :, row] = k.unflatten(-1, (-1, 16))
            else:
                kc[page, :, row] = k
            vc[page, :, row] = s["v"].double()
        else:
            for i, (b, slot) in enumerate(zip(s["seq"].tolist(), s["slot"].tolist())):
                _exact_put(s, kc, vc, b, slot, k[i], s["v"][i].double())
        if c["op"] == "append":
            return q, kc, vc
        lens, _, _, paths = _path_plan(c)
        for b, path in enumerate(paths):
            for i, t in enumerate(path):
                if i != t:
                    _exact_put(s, kc, vc, b, lens[b] + i, *_exact_get(s, kc, vc, b, lens[b] + t))
        return None, kc, vc
    if c["op"] == "tree":
        return _exact_tree(c, s)
    return _exact_pages(c, s)


def _exact_tree(c, s):
    """One sequence and KV head at a time: every node's own list of visible keys, its groups masked key by key."""
    lens, nodes, parents = _tree_plan(c)
    B, T, Hq, d = s["q"].shape
    H, R = c["Hkv"], Hq // c["Hkv"]
    P = s["vc"].shape[2]
    o = torch.zeros(B, T, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        n, L = nodes[b], lens[b]
        total = L + n
        chain = []
        for t in range(n):
            chain.append([t] + (chain[parents[b][t]] if parents[b][t] >= 0 else []))
        at = torch.tensor([L + len(x) - 1 for x in chain], device="cuda")
        where = torch.cat((torch.arange(L, device="cuda"), at))
        visible = torch.zeros(n, total, dtype=torch.bool, device="cuda")
        visible[:, :L] = True
        for t in range(n):
            visible[t, [L + u for u in chain[t]]] = True
        away = at[:, None] - where[None]
        for h in range(H):
            if s["table"] is None:
                k, v = s["kc"][b, h], s["vc"][b, h, :total].double()
                k = (k.permute(1, 0, 2).reshape(P, d) if c["gm"] else k)[:total].double()
            else:
                page = s["table"][b, :_ceil(total, P)].long()
                k, v = s["kc"][page, h], s["vc"][page, h].reshape(-1, d)[:total].double()
                k = (k.permute(0, 2, 1, 3) if c["gm"] else k).reshape(-1, d)[:total].double()
            for r in range(R):
                q = s["q"][b, :n, h * R + r].double()
                x = torch.zeros(n, total, dtype=torch.float64, device="cuda")
                for g, w in enumerate(s["cut"]):
                    x += torch.einsum("td,kd->tk", q[:, 16 * g:16 * g + 16], k[:, 16 * g:16 * g + 16]).masked_fill(away > w, 0.0)
                x = (x * d ** -0.5).masked_fill(~visible, -math.inf)
                lse[b, h * R + r, :n] = torch.logsumexp(x, -1)
                o[b, :n, h * R + r] = torch.softmax(x, -1) @ v
    return o, lse


def _exact_pages(c, s):
    """The transaction as a program on lists: drop every row's pages, take up the kept ones, then hand out free pages in order."""
    refs, table = s["refs"].tolist(), s["table"].tolist()
    lens, parent, keep, new = _pages_plan(c)
    P, B = c["page"], c["B"]
    for b in range(B):
        for p in table[b][:_ceil(lens[b], P)]:
            refs[p] -= 1
    rows = [table[parent[b]][:_ceil(keep[b], P)] for b in range(B)]
    for r in rows:
        for p in r:
            refs[p] += 1
    writers = {}
    for b in range(B):
        if new[b] > keep[b] and keep[b] % P:
            writers.setdefault(rows[b][-1], []).append(b)
    copying = set()
    for p, who in writers.items():
        if refs[p] > 1:
            copying.update(who[1:] if len(who) == refs[p] else who)
    for b in copying:
        refs[rows[b][-1]] -= 1
    free = [p for p in range(c["pool"]) if refs[p] == 0]
    n_free, taken = len(free), 0
    kc, vc = s["kc"].double(), s["vc"].double()
    copies = []
    for b in range(B):
        if b in copying:
            a, k = rows[b].pop(), keep[b] % P
            copies.append([a, free[taken], k])
            vc[free[taken], :, :k] = vc[a, :, :k]
            if c["gm"]:
                kc[free[taken], :, :, :k] = kc[a, :, :, :k]
            else:
                kc[free[taken], :, :k] = kc[a, :, :k]
        else:
            copies.append([-1, -1, 0])
        while len(rows[b]) < _ceil(new[b], P):
            rows[b].append(free[taken])
            refs[free[taken]] = 1
            taken += 1
    most = len(table[0])
    ints = [refs, [r + [-1] * (most - len(r)) for r in rows], new, copies, [0, taken, n_free, len(copying)]]
    return (*(_i32(x) for x in ints), kc, vc)
