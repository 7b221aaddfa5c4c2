"""Drafted trees and cross attention over the paged cache, as a user's
program calls them, next to their plain forms in elementary torch.

  plan   the trees of a step, given as each node's parent: packed ancestor
         masks and rotary positions (once a step, before the layers)
  tree   attention of every drafted node to its sequence's cached context, to
         its ancestors and to itself (once a layer)
  cross  attention of a decoder's rows to all of an encoder's cached states
         (single tokens, beams, whole prompts)
  keep   the accepted nodes' rows of every layer's cache moved to the
         positions that follow the context (once a step, after the layers)

``own`` selects what run() does: False, the plain forms; True, the calls of
kv_cache_decode_gqa_gb300.
"""
import math

import torch

own = False

GROUP = 16       # channels per E4M3 scale of an MXFP4 row
MAX_NODES = 256  # of a tree


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one sequence's tree: latency
        dict(name="plan-one", kind="plan", batch=1, rows=16, nodes=16,
             window=0),
        # the trees of a large batch
        dict(name="plan-batch", kind="plan", batch=256, rows=30011,
             nodes=MAX_NODES, window=0),
        # one sequence's drafted tree (Llama-3.1-70B heads)
        dict(name="tree-one", kind="tree", batch=1, rows=16, nodes=16,
             context=4000, n_h=64, n_kv=8, d=128, dtype="bf16", block=64,
             window=0),
        # ragged trees of a batch over long contexts
        dict(name="tree-batch", kind="tree", batch=16, rows=500, nodes=64,
             context=16384, n_h=64, n_kv=8, d=128, dtype="bf16", block=64,
             window=0),
        # small trees over an E4M3 cache
        dict(name="tree-fp8", kind="tree", batch=32, rows=250, nodes=12,
             context=8192, n_h=64, n_kv=8, d=128, dtype="fp8", block=64,
             window=0),
        # large trees over a 4-bit cache
        dict(name="tree-mxfp4", kind="tree", batch=8, rows=480, nodes=64,
             context=32768, n_h=64, n_kv=8, d=128, dtype="mxfp4", block=64,
             window=0),
        # a decoding step against encoded audio: one token a sequence,
        # one query head a key head
        dict(name="cross-step", kind="cross", batch=16, rows=16, listed=False,
             context=1500, n_h=16, n_kv=16, d=64, dtype="bf16", block=64,
             starts=False),
        # five beams a sequence against the same states
        dict(name="cross-beams", kind="cross", batch=16, rows=80, listed=True,
             context=1500, n_h=16, n_kv=16, d=64, dtype="bf16", block=64,
             starts=False),
        # prompts of a decoder over E4M3 states of left-padded inputs
        dict(name="cross-prompt-fp8", kind="cross", batch=6, rows=2003,
             listed=True, context=5000, n_h=32, n_kv=8, d=128, dtype="fp8",
             block=32, starts=True),
        # one long decoder sequence over one long input
        dict(name="cross-long", kind="cross", batch=1, rows=2011, listed=True,
             context=20011, n_h=64, n_kv=8, d=128, dtype="bf16", block=64,
             starts=False),
        # one sequence's accepted nodes in all layers
        dict(name="keep-one", kind="keep", batch=1, layers=32, n_kv=8, d=128,
             dtype="bf16", block=64, nodes=16, width=6, base=60),
        # a batch's, in 80 layers
        dict(name="keep-batch", kind="keep", batch=16, layers=80, n_kv=8,
             d=128, dtype="fp8", block=64, nodes=64, width=9, base=60),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["plan", "tree", "tree", "cross", "cross", "keep"])
    n_kv = rng.choice([1, 2, 4, 8])
    dtype = rng.choice(["bf16", "bf16", "fp8", "mxfp4"])
    d = 128 if dtype == "mxfp4" else rng.choice([64, 128])
    block = rng.choice([8, 16, 32, 48, 64, 128])
    if kind == "plan":
        nodes = _log(rng, 1, MAX_NODES)
        batch = _log(rng, 1, 256)
        return dict(kind=kind, batch=batch, nodes=nodes,
                    rows=rng.randint(batch, min(batch * nodes, 30000)
                                     if nodes > 1 else batch),
                    window=rng.choice([0, 0, rng.randint(1, 12)]))
    if kind == "tree":
        batch, nodes = _log(rng, 1, 16), _log(rng, 1, 100)
        return dict(kind=kind, batch=batch, nodes=nodes,
                    rows=rng.randint(batch, max(batch * nodes * 3 // 4,
                                                batch)),
                    context=_log(rng, 1, 9000),
                    n_h=n_kv * rng.choice([1, 2, 3, 4, 7, 8, 16]), n_kv=n_kv,
                    d=d, dtype=dtype, block=block,
                    window=rng.choice([0, 0, _log(rng, 2, 4000)]))
    if kind == "cross":
        batch = _log(rng, 1, 16)
        one = rng.random() < 0.25
        return dict(kind=kind, batch=batch,
                    rows=batch if one else max(batch, _log(rng, 2, 1500)),
                    listed=not one, context=_log(rng, 1, 9000),
                    n_h=n_kv * rng.choice([1, 2, 3, 4, 7, 8, 16]), n_kv=n_kv,
                    d=d, dtype=dtype, block=block,
                    starts=rng.random() < 0.3)
    return dict(kind=kind, batch=_log(rng, 1, 16), layers=_log(rng, 1, 80),
                n_kv=n_kv, d=d, dtype=dtype, block=block,
                nodes=rng.randint(20, 64), width=rng.randint(1, 9),
                base=_log(rng, 1, 100))


def _split(total, parts, most, g):
    """Ragged sizes in [1, most] that sum to total (parts <= total <= parts
    * most)."""
    w = torch.rand(parts, generator=g, dtype=torch.float64) + 0.25
    n = (w / w.sum() * (total - parts)).floor().long() + 1
    n.clamp_(max=most)
    left, i = total - int(n.sum()), 0
    while left > 0:
        add = min(left, most - int(n[i]))
        n[i] += add
        left -= add
        i += 1
    return n.tolist()


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _starts(n):
    out = [0]
    for x in n:
        out.append(out[-1] + x)
    return _i32(out)


def _row_bytes(dtype, d):
    return d // 2 + d // GROUP if dtype == "mxfp4" else d


def _cached(shape, dtype, d, g):
    """Random rows [*shape] of a cache of this type."""
    if dtype == "bf16":
        return _randn(g, *shape, d).bfloat16()
    if dtype == "fp8":
        return (_randn(g, *shape, d) * 40).to(torch.float8_e4m3fn).view(
            torch.uint8)
    codes = torch.randint(0, 256, (*shape, d // 2), generator=g,
                          device="cuda", dtype=torch.uint8)
    scale = (0.1 + 0.4 * torch.rand((*shape, d // GROUP), generator=g,
                                    device="cuda")).to(torch.float8_e4m3fn)
    return torch.cat([codes, scale.view(torch.uint8)], -1)


def _tables(block, last, g):
    """A block table over a shuffled pool that holds `last` positions."""
    per = [(x + block - 1) // block for x in last]
    width, total = max(max(per), 1), sum(per) + 2
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    j = torch.arange(width, device="cuda")[None, :]
    n = torch.tensor(per, device="cuda")[:, None]
    first = torch.cumsum(n, 0) - n
    table = torch.where(j < n, perm[(first + j).clamp(max=total - 1)], 0)
    return table.to(torch.int32).contiguous(), total


def _trees(n, g):
    """Parents of every sequence's nodes: node 0 is the root, a node hangs
    below one of those before it, more often a late one; now and then below
    the context itself."""
    parts = []
    for k in n:
        i = torch.arange(k, dtype=torch.float64)
        u = torch.rand(2, k, generator=g, dtype=torch.float64)
        p = (i * u[0].sqrt()).floor().long()
        p[u[1] < 0.03] = -1
        p[0] = -1
        parts.append(p)
    return torch.cat(parts).to(torch.int32).cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.Generator().manual_seed(977 + 31 * seed)
    s, kind, B = dict(case=case), case["kind"], case["batch"]
    if kind == "keep":
        return _prepare_keep(s, case, g, h)
    if kind == "cross":
        n = _split(case["rows"], B, case["rows"], h)
        if case["rows"] % B == 0:       # beams are equally many
            n = [case["rows"] // B] * B
        c = case["context"]
        last = (torch.randint((c + 1) // 2, c + 1, (B,), generator=h).tolist()
                if B > 1 else [c])
        past = None
    else:
        n = _split(case["rows"], B, case["nodes"], h)
        c = case.get("context", 4096)
        past = (torch.randint(c // 8, c + 1, (B,), generator=h).tolist()
                if B > 1 else [c])
        last = [a + b for a, b in zip(n, past)]
        s["parents"] = _trees(n, h)
        s["start"] = _i32(past)
    s["n"], s["row_start"] = n, _starts(n)
    # a program's trees have a budget of nodes
    s["max_rows"] = case["nodes"] if kind != "cross" else max(n)
    if kind == "plan":
        return s
    s["table"], blocks = _tables(case["block"], last, g)
    s["seq_lens"], s["max_seq_len"] = _i32(last), max(last)
    shape = (blocks, case["n_kv"], case["block"])
    s["k"] = _cached(shape, case["dtype"], case["d"], g)
    s["v"] = _cached(shape, case["dtype"], case["d"], g)
    s["scales"] = (None, None)
    if case["dtype"] == "fp8":
        sc = 0.01 + 0.02 * torch.rand(2, case["n_kv"], generator=g,
                                      device="cuda")
        s["scales"] = (sc[0].contiguous(), sc[1].contiguous())
    s["q"] = _randn(g, sum(n), case["n_h"], case["d"]).bfloat16()
    s["first"] = None
    if kind == "tree":                  # the step's plan, kept by its layers
        s["masks"], s["positions"] = _plain_plan(s)
    elif case["starts"]:
        s["first"] = _i32([int(x * u) for x, u in
                           zip(last, torch.rand(B, generator=h).tolist())])
    return s


def _prepare_keep(s, case, g, h):
    B, w = case["batch"], case["width"]
    start = torch.randint(0, case["base"] + 1, (B,), generator=h).tolist()
    s["start"] = _i32(start)
    # (a pool of one size, whatever the lengths)
    s["table"], blocks = _tables(case["block"],
                                 [case["base"] + case["nodes"]] * B, g)
    shape = (case["layers"], blocks, case["n_kv"], case["block"])
    s["k"] = _cached(shape, case["dtype"], case["d"], g)
    s["v"] = _cached(shape, case["dtype"], case["d"], g)
    # the root and, level by level, one node behind the first levels
    # (a pass can be repeated: no node is moved onto another accepted one)
    paths, keep = [], []
    for _ in range(B):
        rest = torch.randperm(case["nodes"] - w, generator=h)[:w - 1] + w
        paths.append([0] + sorted(rest.tolist()))
        keep.append(int(torch.randint(1, w + 1, (1,), generator=h)))
    s["path"], s["n_keep"] = _i32(paths), _i32(keep)
    if own:
        import kv_cache_decode_gqa_gb300 as K
        s["caches"] = K.CacheList(
            K.PagedCache(s["k"][i], s["v"][i], case["block"], case["n_kv"],
                         case["d"], case["dtype"])
            for i in range(case["layers"]))
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _owner(s):
    """Sequence of every row, and its index there."""
    rs = s["row_start"].long()
    row = torch.arange(s["case"]["rows"], device="cuda")
    b = torch.bucketize(row, rs[1:], right=True)
    return b, row - rs[b]


def _plain_plan(s):
    """Ancestors by doubling: after step k a node's mask holds its 2^k
    nearest, and `up` is the one behind them."""
    b, i = _owner(s)
    R, rows = s["max_rows"], i.numel()
    first = s["row_start"].long()[b]
    p = s["parents"].long()
    none = rows                                   # a row with no bits
    up = torch.cat([torch.where(p >= 0, first + p, none),
                    torch.tensor([none], device="cuda")])
    m = torch.zeros(rows + 1, R, dtype=torch.bool, device="cuda")
    m[torch.arange(rows, device="cuda"), i] = True
    depth = torch.zeros(rows + 1, dtype=torch.long, device="cuda")
    depth[:rows] = 1
    for _ in range(max(R - 1, 1).bit_length()):
        m = m | m[up]
        depth = depth + depth[up]
        up = up[up]
    m, depth = m[:rows], depth[:rows] - 1
    w = s["case"]["window"]
    if w:
        d = torch.zeros(rows, R, dtype=torch.long, device="cuda")
        padded = (first[:, None] + torch.arange(R, device="cuda")).clamp(
            max=rows - 1)
        d = depth[padded]
        m = m & (depth[:, None] - d < w)
    words = (R + 31) // 32
    bits = torch.zeros(rows, words * 32, dtype=torch.long, device="cuda")
    bits[:, :R] = m
    packed = (bits.view(rows, words, 32) <<
              torch.arange(32, device="cuda")).sum(-1)
    packed = torch.where(packed >= 2 ** 31, packed - 2 ** 32, packed)
    return (packed.to(torch.int32),
            (s["start"].long()[b] + depth).to(torch.int32))


def _values(t, s, i):
    """fp32 values of cached rows t [..][heads][positions][bytes]."""
    dtype, d = s["case"]["dtype"], s["case"]["d"]
    if dtype == "bf16":
        return t.float()
    if dtype == "fp8":
        return (t.view(torch.float8_e4m3fn).float() *
                s["scales"][i][:, None, None])
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3,
                         -4, -6], device=t.device)
    codes = t[..., :d // 2]
    scale = t[..., d // 2:].contiguous().view(torch.float8_e4m3fn).float()
    v = torch.stack([grid[(codes & 15).int()], grid[(codes >> 4).int()]], -1)
    v = v.flatten(-2).unflatten(-1, (d // GROUP, GROUP))
    return (v * scale[..., None]).flatten(-2)


def _seen(s):
    """Which positions [B][R][L] the rows of every sequence attend to."""
    case = s["case"]
    lens, rs = s["seq_lens"].long(), s["row_start"].long()
    L, R = s["max_seq_len"], s["max_rows"]
    pos = torch.arange(L, device="cuda")
    if case["kind"] == "cross":
        ok = pos < lens[:, None]
        if s["first"] is not None:
            ok &= pos >= s["first"].long()[:, None]
        return ok[:, None].expand(-1, R, -1)
    n = rs[1:] - rs[:-1]
    past = lens - n
    row = (rs[:-1, None] + torch.arange(R, device="cuda")).clamp(
        max=case["rows"] - 1)                                 # [B][R]
    ok = (pos < past[:, None])[:, None].expand(-1, R, -1)
    if case["window"]:
        at = s["positions"].long()[row]
        ok = ok & (pos > (at - case["window"])[..., None])
    node = pos[None, :] - past[:, None]                       # [B][L]
    inside = (node >= 0) & (node < n[:, None])
    node = node.clamp(0, R - 1)
    words = s["masks"][row].long()                            # [B][R][W]
    word = words.gather(2, (node // 32)[:, None].expand(-1, R, -1))
    bit = (word >> (node % 32)[:, None]) & 1
    return ok | ((bit == 1) & inside[:, None])


def _plain_attend(s):
    """softmax(q K^T / sqrt(d)) V of every row over the positions it sees:
    ragged rows padded to the longest."""
    case, bs = s["case"], s["case"]["block"]
    hk, d = case["n_kv"], case["d"]
    grp = case["n_h"] // hk
    rs = s["row_start"].long()
    L, R, B = s["max_seq_len"], s["max_rows"], case["batch"]
    pos = torch.arange(L, device="cuda")
    blk = s["table"].long()[:, pos // bs]
    k = _values(s["k"][blk, :, pos % bs].transpose(1, 2), s, 0)
    row = (rs[:-1, None] + torch.arange(R, device="cuda")).clamp(
        max=case["rows"] - 1)
    q = s["q"].float()[row].view(B, R, hk, grp, d).permute(0, 2, 3, 1, 4)
    x = torch.matmul(q.reshape(B, hk, grp * R, d), k.transpose(2, 3))
    del k
    x = x.view(B, hk, grp, R, L).mul_(d ** -0.5)
    x.masked_fill_(~_seen(s)[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(m.clamp(min=-3e38)).exp_()
    l = x.sum(-1, keepdim=True)
    v = _values(s["v"][blk, :, pos % bs].transpose(1, 2), s, 1)
    o = torch.matmul(x.view(B, hk, grp * R, L), v).view(B, hk, grp, R, d)
    o = torch.where(l > 0, o / l, 0)
    lse = (m + l.log())[..., 0]
    b, i = _owner(s)
    out = o.permute(0, 3, 1, 2, 4)[b, i].reshape(-1, case["n_h"], d)
    return (out.bfloat16(),
            lse.permute(0, 3, 1, 2)[b, i].reshape(-1, case["n_h"]))


def _plain_keep(s):
    w, bs = s["case"]["width"], s["case"]["block"]
    j = torch.arange(w, device="cuda")
    b, j = torch.nonzero(j < s["n_keep"][:, None], as_tuple=True)
    src = s["start"].long()[b] + s["path"].long()[b, j]
    dst = s["start"].long()[b] + j
    table = s["table"].long()
    for t in (s["k"], s["v"]):
        t[:, table[b, dst // bs], :, dst % bs] = (
            t[:, table[b, src // bs], :, src % bs])
    return s["k"], s["v"]


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    kind = s["case"]["kind"]
    if own:
        return _own(s, kind)
    if kind == "plan":
        return _plain_plan(s)
    if kind == "keep":
        return _plain_keep(s)
    return _plain_attend(s)


def _own(s, kind):
    import kv_cache_decode_gqa_gb300 as K
    case = s["case"]
    if kind == "plan":
        return K.tree_plan(s["parents"], s["start"], s["row_start"],
                           s["max_rows"], window=case["window"])
    if kind == "keep":
        K.kv_keep(s["caches"], s["table"], s["start"], s["path"],
                  s["n_keep"])
        return s["k"], s["v"]
    cache = K.PagedCache(s["k"], s["v"], case["block"], case["n_kv"],
                         case["d"], case["dtype"], *s["scales"])
    if kind == "tree":
        return K.gqa_tree(cache, s["table"], s["seq_lens"], s["max_seq_len"],
                          s["q"], s["row_start"], s["max_rows"], s["masks"],
                          positions=s["positions"], window=case["window"])
    if not case["listed"]:              # row b belongs to sequence b
        return K.gqa_cross(cache, s["table"], s["seq_lens"],
                           s["max_seq_len"], s["q"], first=s["first"])
    return K.gqa_cross(cache, s["table"], s["seq_lens"], s["max_seq_len"],
                       s["q"], s["row_start"], s["max_rows"],
                       first=s["first"])


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _reach(case):
    """Expected positions a sequence's rows attend to."""
    B, c = case["batch"], case["context"]
    if case["kind"] == "cross":
        reach = c if B == 1 else 0.75 * c
        return reach / 2 if case["starts"] else reach
    past = c if B == 1 else 9 * c / 16
    return min(past, case["window"]) if case["window"] else past


def work(case):
    kind, B = case["kind"], case["batch"]
    if kind == "plan":
        words = (case["nodes"] + 31) // 32
        return {"bytes": case["rows"] * (8 + 4 * words),
                "flops": 2 * case["rows"] * words}
    if kind == "keep":
        # about half of the longest path is accepted; its root stays
        row = _row_bytes(case["dtype"], case["d"]) * (
            2 if case["dtype"] == "bf16" else 1)
        moved = B * (case["width"] - 1) / 2
        return {"bytes": int(4 * moved * case["layers"] * case["n_kv"] * row +
                             4 * B * case["width"] + 8),
                "flops": 1}
    row = _row_bytes(case["dtype"], case["d"]) * (
        2 if case["dtype"] == "bf16" else 1)
    reach = _reach(case)
    own_rows = case["rows"] / B if kind == "tree" else 0
    heads = case["rows"] * case["n_h"]
    return {"bytes": int(B * (reach + own_rows) * case["n_kv"] * 2 * row +
                         heads * (4 * case["d"] + 4)),
            "flops": int(heads * (reach + 1) * 4 * case["d"])}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _value64(t, s, i, head):
    """fp64 values of one head's cached rows [positions][bytes]."""
    dtype, d = s["case"]["dtype"], s["case"]["d"]
    if dtype == "bf16":
        return t.double()
    if dtype == "fp8":
        return t.view(torch.float8_e4m3fn).double() * s["scales"][i][
            head].double()
    pair = torch.stack([t[:, :d // 2] % 16, t[:, :d // 2] // 16],
                       -1).flatten(-2)
    m = (pair % 8).double()
    mag = torch.where(m < 4, m / 2, torch.where(m < 6, m - 2, 2 * m - 8))
    sc = t[:, d // 2:].double()
    e, f = sc // 8, sc % 8
    sv = torch.where(e > 0, (1 + f / 8) * torch.pow(2.0, e - 7),
                     f * 2.0 ** -9)
    return (torch.where(pair >= 8, -mag, mag) *
            sv.repeat_interleave(GROUP, -1))


def _chains(s):
    """Of every row: its ancestors and itself, by walking up."""
    parents, out, at = s["parents"].tolist(), [], 0
    for n in s["n"]:
        own_chains = []
        for i in range(n):
            p = parents[at + i]
            own_chains.append((own_chains[p] if p >= 0 else []) + [i])
        out += own_chains
        at += n
    w = s["case"]["window"]
    depth = [len(c) - 1 for c in out]
    return [c[-w:] if w else c for c in out], depth


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "plan":
        chains, depth = _chains(s)
        words = (s["max_rows"] + 31) // 32
        start = s["start"].tolist()
        masks, positions, r = [], [], 0
        for b, n in enumerate(s["n"]):
            for _ in range(n):
                bits = sum(1 << j for j in chains[r])
                row = [(bits >> (32 * k)) & 0xffffffff for k in range(words)]
                masks.append([x - 2 ** 32 if x >= 2 ** 31 else x
                              for x in row])
                positions.append(start[b] + depth[r])
                r += 1
        return _i32(masks), _i32(positions)
    if kind == "keep":
        table, start = s["table"].tolist(), s["start"].tolist()
        path, bs = s["path"].tolist(), case["block"]
        for b, keep in enumerate(s["n_keep"].tolist()):
            for j in range(keep):
                a, z = start[b] + path[b][j], start[b] + j
                for t in (s["k"], s["v"]):
                    t[:, table[b][z // bs], :, z % bs] = t[
                        :, table[b][a // bs], :, a % bs].clone()
        return s["k"], s["v"]
    bs, d, at = case["block"], case["d"], 0
    grp = case["n_h"] // case["n_kv"]
    if kind == "tree":
        chains, depth = _chains(s)
        start = s["start"].tolist()
    outs, lses = [], []
    for b, (n, T) in enumerate(zip(s["n"], s["seq_lens"].tolist())):
        pos = torch.arange(T, device="cuda")
        blk = s["table"][b].long()[pos // bs]
        hide = torch.zeros(n, T, dtype=torch.bool)
        if kind == "tree":
            hide[:, T - n:] = True
            for i in range(n):
                if case["window"]:
                    low = start[b] + depth[at + i] + 1 - case["window"]
                    hide[i, :min(max(low, 0), T - n)] = True
                hide[i, [T - n + j for j in chains[at + i]]] = False
        elif s["first"] is not None:
            hide[:, :int(s["first"][b])] = True
        hide = hide.cuda()
        q = s["q"][at:at + n].double()
        oh, lh = [], []
        for h in range(case["n_h"]):
            if h % grp == 0:
                kk = _value64(s["k"][blk, h // grp, pos % bs], s, 0, h // grp)
                vv = _value64(s["v"][blk, h // grp, pos % bs], s, 1, h // grp)
            x = (q[:, h] @ kk.t() / math.sqrt(d)).masked_fill(hide, -math.inf)
            lse = torch.logsumexp(x, -1)
            w = torch.exp(x - lse[:, None])
            oh.append(torch.nan_to_num(w, nan=0.0) @ vv)
            lh.append(lse)
        outs.append(torch.stack(oh, 1))
        lses.append(torch.stack(lh, 1))
        at += n
    return torch.cat(outs), torch.cat(lses)
