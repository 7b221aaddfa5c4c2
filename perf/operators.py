"""The operators of the prompt path and of the 4-bit cache, as a user's
program calls them, next to their plain forms in elementary torch.

  rope    rotary positions of one to four axes (time, height, width) applied
          to the query and key heads of a step or a prompt
  write   a ragged batch of new key and value rows quantised into the paged
          cache (the keys rotated on the way where the case says so) and read
          back as the bf16 values the cache now stands for
  read    whole cached contexts read back as bf16
  extend  attention of several new tokens a sequence (a prompt, a chunk of
          one, a few speculated tokens) over an MXFP4 cache that holds them
  decode  attention of one new token a sequence over an MXFP4 cache, query
          groups beyond 4 heads

``own`` selects what run() does: False, the plain forms; True, the calls of
kv_cache_decode_gqa_gb300.
"""
import math

import torch

own = False

D = 128          # head width of an MXFP4 cache
GROUP = 16       # channels per E4M3 scale of an MXFP4 row
ROW4 = D // 2 + D // GROUP


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decode step of 32 sequences: launch latency
        dict(name="rope-step", kind="rope", rows=32, n_h=64, n_kv=8, d=128,
             d_rot=128, axes=1, spread=False, pairing="half", inverse=False,
             fused_qkv=False, base=8192),
        # a video prompt: three axes, heads inside a fused qkv projection
        dict(name="rope-video-prompt", kind="rope", rows=16384, n_h=64,
             n_kv=8, d=128, d_rot=128, axes=3, spread=False, pairing="half",
             inverse=False, fused_qkv=True, base=500000),
        # one token of each of 64 sequences into 4 bits
        dict(name="write-step-mxfp4", kind="write", batch=64, rows=64,
             n_h=0, n_kv=8, dtype="mxfp4", block=64, axes=0, base=4000),
        # ragged prompts into 4 bits
        dict(name="write-prompt-mxfp4", kind="write", batch=8, rows=30011,
             n_h=0, n_kv=8, dtype="mxfp4", block=64, axes=0, base=0),
        # image prompts: queries and keys rotated and the keys and values
        # quantised to E4M3 in the same call
        dict(name="write-image-prompt-fp8", kind="write", batch=4,
             rows=12007, n_h=64, n_kv=8, dtype="fp8", block=64, axes=3,
             base=100),
        # whole 4-bit contexts back to bf16 (to move or re-encode them)
        dict(name="read-context-mxfp4", kind="read", batch=4, rows=110003,
             n_kv=8, dtype="mxfp4", block=64, base=0),
        # four speculated tokens of 16 sequences verified at once
        dict(name="extend-verify", kind="extend", batch=16, rows=64,
             context=16384, n_h=64, n_kv=8, block=64, window=0),
        # whole ragged prompts (Llama-3.1-70B heads)
        dict(name="extend-prompt", kind="extend", batch=2, rows=7001,
             context=0, n_h=64, n_kv=8, block=64, window=0),
        # a prompt chunk over a long context, seven query heads a group
        dict(name="extend-chunk", kind="extend", batch=1, rows=1021,
             context=32000, n_h=56, n_kv=8, block=64, window=0),
        # one sequence's decode step: latency
        dict(name="decode-one", kind="decode", batch=1, context=4096,
             n_h=64, n_kv=8, block=64, window=0),
        # the Llama-3.1-70B batch over a 4-bit cache
        dict(name="decode-batch", kind="decode", batch=32, context=8192,
             n_h=64, n_kv=8, block=64, window=0),
        # long contexts, sixteen query heads a group
        dict(name="decode-long", kind="decode", batch=32, context=32768,
             n_h=64, n_kv=4, block=64, window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope", "write", "read", "extend", "decode"])
    n_kv = rng.choice([1, 2, 4, 8])
    block = rng.choice([16, 32, 64, 128])
    if kind == "rope":
        d = rng.choice([64, 128])
        return dict(kind=kind, rows=_log(rng, 1, 12000),
                    n_h=n_kv * rng.choice([1, 4, 5, 7, 8]), n_kv=n_kv, d=d,
                    d_rot=rng.choice([d, d // 2]), axes=rng.choice([1, 2, 3]),
                    spread=rng.random() < 0.4,
                    pairing=rng.choice(["half", "adjacent"]),
                    inverse=rng.random() < 0.3,
                    fused_qkv=rng.random() < 0.5,
                    base=_log(rng, 1, 1000000))
    if kind == "write":
        batch = _log(rng, 1, 64)
        dtype = rng.choice(["bf16", "fp8", "mxfp4"])
        # a rotation of fp32 products lies next to a border of the 4-bit
        # grid now and then, where the last bit of a cosine decides: the
        # rotating draws go to the wider types
        axes = rng.choice([0, 1, 3]) if dtype != "mxfp4" else 0
        return dict(kind=kind, batch=batch,
                    rows=max(batch, _log(rng, 1, 9000)),
                    n_h=n_kv * rng.choice([4, 8]) if axes else 0, n_kv=n_kv,
                    dtype=dtype, block=block, axes=axes,
                    base=_log(rng, 1, 5000))
    if kind == "read":
        batch = _log(rng, 1, 32)
        return dict(kind=kind, batch=batch,
                    rows=max(batch, _log(rng, 1, 50000)), n_kv=n_kv,
                    dtype=rng.choice(["bf16", "fp8", "mxfp4"]), block=block,
                    base=_log(rng, 1, 2000))
    if kind == "extend":
        batch = _log(rng, 1, 8)
        return dict(kind=kind, batch=batch,
                    rows=max(batch, _log(rng, 2, 1500)),
                    context=_log(rng, 1, 8000),
                    n_h=n_kv * rng.choice([1, 3, 4, 5, 7, 8, 16]), n_kv=n_kv,
                    block=block,
                    window=rng.choice([0, 0, _log(rng, 16, 2000)]))
    return dict(kind=kind, batch=_log(rng, 1, 32), context=_log(rng, 8, 12000),
                n_h=n_kv * rng.choice([8, 16]), n_kv=n_kv, block=block,
                window=rng.choice([0, 0, _log(rng, 16, 2000)]))


def _split(total, parts, g):
    """Ragged sizes >= 1 that sum to total, drawn from generator g."""
    w = torch.rand(parts, generator=g, dtype=torch.float64) + 0.25
    n = (w / w.sum() * (total - parts)).floor().long() + 1
    n[0] += total - int(n.sum())
    return n.tolist()


def _lengths(case, seed):
    """New rows and cached positions before them, per sequence."""
    g = torch.Generator().manual_seed(977 + 31 * seed)
    B, kind = case["batch"], case["kind"]
    if kind in ("write", "read"):
        n = _split(case["rows"], B, g)
        base = torch.randint(0, case["base"] + 1, (B,), generator=g).tolist()
        return n, base
    n = _split(case["rows"], B, g) if kind == "extend" else [1] * B
    if kind == "extend" and case["rows"] == 4 * B:
        n = [4] * B                       # a verified draft is equally long
    c = case["context"]
    past = (torch.randint(c // 8, c + 1, (B,), generator=g) if B > 1
            else torch.tensor([c])).tolist()
    if kind == "decode":
        past = [max(p - 1, 0) for p in past]
    return n, past


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _starts(n):
    out = [0]
    for x in n:
        out.append(out[-1] + x)
    return torch.tensor(out, dtype=torch.int32, device="cuda")


def _frequencies(d_rot, axes, spread):
    """Radians per position of each pair (fp64), and the pair's axis."""
    half = d_rot // 2
    f = 10000.0 ** (-2.0 * torch.arange(half, dtype=torch.float64) / d_rot)
    sections = _sections(half, axes)
    if spread:                 # axes in turn while their sections last
        left, ax = list(sections), []
        while len(ax) < half:
            for a in range(axes):
                if left[a]:
                    left[a] -= 1
                    ax.append(a)
    else:
        ax = [a for a in range(axes) for _ in range(sections[a])]
    return f.cuda(), torch.tensor(ax, device="cuda")


def _sections(half, axes):
    if axes == 3:
        a = half // 4
        return [a, (half - a) // 2, half - a - (half - a) // 2]
    return [half // axes] * (axes - 1) + [half - half // axes * (axes - 1)]


def _positions(rows, axes, base, g):
    """Frames of a grid of patches: time, height and width of each row."""
    i = torch.arange(rows, device="cuda")
    gh, gw = 24, 36
    cols = [i // (gh * gw), (i // gw) % gh, i % gw][:axes]
    if axes < 3:
        cols = [i // (1 + 7 * a) for a in range(axes)]
    off = torch.randint(0, base + 1, (axes, 1), generator=g, device="cuda")
    return (torch.stack(cols) + off).to(torch.int32).contiguous()


def _tables(case, last, g):
    """A block table over a shuffled pool that holds `last` positions."""
    bs = case["block"]
    per = [(x + bs - 1) // bs for x in last]
    width, total = max(max(per), 1), sum(per) + 2
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    j = torch.arange(width, device="cuda")[None, :]
    n = torch.tensor(per, device="cuda")[:, None]
    first = torch.cumsum(n, 0) - n
    table = torch.where(j < n, perm[(first + j).clamp(max=total - 1)], 0)
    return table.to(torch.int32).contiguous(), total


def _row_bytes(dtype):
    return ROW4 if dtype == "mxfp4" else D


def _cache_of(case, blocks, dtype, g, filled):
    """K and V storage; filled: values of N(0,1) in every row."""
    out = []
    for _ in range(2):
        shape = (blocks, case["n_kv"], case["block"])
        if dtype == "bf16":
            t = (_randn(g, *shape, D).bfloat16() if filled else
                 torch.zeros(*shape, D, dtype=torch.bfloat16, device="cuda"))
        elif not filled:
            t = torch.zeros(*shape, _row_bytes(dtype), dtype=torch.uint8,
                            device="cuda")
        elif dtype == "fp8":
            t = (_randn(g, *shape, D) * 40).to(torch.float8_e4m3fn).view(
                torch.uint8)
        else:
            t = _encode4(_randn(g, *shape, D).bfloat16())
        out.append(t)
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=case)
    kind = case["kind"]
    if kind == "rope":
        h, hk, d = case["n_h"], case["n_kv"], case["d"]
        if case["fused_qkv"]:
            qkv = _randn(g, case["rows"], h + 2 * hk, d).bfloat16()
            s["q"], s["k"] = qkv[:, :h], qkv[:, h:h + hk]
        else:
            s["q"] = _randn(g, case["rows"], h, d).bfloat16()
            s["k"] = _randn(g, case["rows"], hk, d).bfloat16()
        _rope_state(s, case["d_rot"], case["axes"], case["spread"],
                    case["pairing"], case["rows"], case["base"], g)
        return s
    n, past = _lengths(case, seed)
    last = [a + b for a, b in zip(n, past)]
    s["table"], blocks = _tables(case, last, g)
    s["row_start"] = _starts(n)
    s["start"] = torch.tensor(past, dtype=torch.int32, device="cuda")
    dtype = case.get("dtype", "mxfp4")
    s["dtype"] = dtype
    s["k"], s["v"] = _cache_of(case, blocks, dtype, g, kind != "write")
    s["scales"] = None
    if dtype == "fp8":   # one scale a head, its inverse for the writes
        sc = 0.01 + 0.02 * torch.rand(2, case["n_kv"], generator=g,
                                      device="cuda")
        s["scales"] = (sc[0].contiguous(), sc[1].contiguous(),
                       (1 / sc[0]).contiguous(), (1 / sc[1]).contiguous())
    rows = sum(n)
    if kind == "write":
        s["k_new"] = _randn(g, rows, case["n_kv"], D).bfloat16()
        s["v_new"] = _randn(g, rows, case["n_kv"], D).bfloat16()
        if case["axes"]:
            s["q"] = _randn(g, rows, case["n_h"], D).bfloat16()
            _rope_state(s, D, case["axes"], False, "half", rows,
                        case["base"], g)
        return s
    if kind == "read":
        s["rows"] = rows
        return s
    s["q"] = _randn(g, rows, case["n_h"], D).bfloat16()
    s["seq_lens"] = torch.tensor(last, dtype=torch.int32, device="cuda")
    s["max_seq_len"], s["max_rows"] = max(last), max(n)
    return s


def _rope_state(s, d_rot, axes, spread, pairing, rows, base, g):
    s["freq"], s["axis"] = _frequencies(d_rot, axes, spread)
    s["positions"] = _positions(rows, axes, base, g)
    if own:
        import kv_cache_decode_gqa_gb300 as K
        s["plan"] = K.rope_plan(d_rot, theta=10000.0,
                                sections=_sections(d_rot // 2, axes),
                                interleave=spread, pairing=pairing,
                                device="cuda")


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _rotate(x, s, d_rot, pairing, inverse):
    """Pairs of x [rows][heads][d] turned by position * frequency."""
    ang = s["positions"][s["axis"]].double().t() * s["freq"]
    c, n = ang.cos().float()[:, None], ang.sin().float()[:, None]
    if inverse:
        n = -n
    x = x.float()
    out = x.clone()
    if pairing == "half":
        a, b = x[..., :d_rot // 2], x[..., d_rot // 2:d_rot]
        out[..., :d_rot // 2] = a * c - b * n
        out[..., d_rot // 2:d_rot] = b * c + a * n
    else:
        a, b = x[..., 0:d_rot:2], x[..., 1:d_rot:2]
        out[..., 0:d_rot:2] = a * c - b * n
        out[..., 1:d_rot:2] = b * c + a * n
    return out.bfloat16()


def _encode4(x):
    """MXFP4 rows of x [..., D] bf16: codes, then group scales."""
    x = x.float().unflatten(-1, (D // GROUP, GROUP))
    scale = (x.abs().amax(-1) / 6).clamp(max=448).to(torch.float8_e4m3fn)
    sv = scale.float()[..., None]
    q = torch.where(sv > 0, x / sv, 0)
    a = q.abs()
    code = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() +
            (a >= 1.75).byte() + (a > 2.5).byte() + (a >= 3.5).byte() +
            (a > 5).byte())
    code = code + 8 * ((x < 0) & (sv > 0)).byte()
    code = code.flatten(-2)
    packed = code[..., 0::2] | (code[..., 1::2] << 4)
    return torch.cat([packed, scale.view(torch.uint8)], -1)


def _decode4(rows):
    """The fp32 values of MXFP4 rows [..., ROW4]."""
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3,
                         -4, -6], device=rows.device)
    codes = rows[..., :D // 2]
    scale = rows[..., D // 2:].contiguous().view(torch.float8_e4m3fn).float()
    v = torch.stack([grid[(codes & 15).int()], grid[(codes >> 4).int()]], -1)
    v = v.flatten(-2).unflatten(-1, (D // GROUP, GROUP))
    return (v * scale[..., None]).flatten(-2)


def _slots(s):
    """Physical block and slot of every ragged row."""
    rs, bs = s["row_start"].long(), s["case"]["block"]
    row = torch.arange(s["case"]["rows"], device="cuda")
    b = torch.bucketize(row, rs[1:], right=True)
    pos = s["start"].long()[b] + row - rs[b]
    return s["table"].long()[b, pos // bs], pos % bs


def _stored(x, s, i):
    """New rows x [rows][n_kv][D] bf16 as the cache's bytes."""
    if s["dtype"] == "bf16":
        return x
    if s["dtype"] == "fp8":
        y = x.float() * s["scales"][2 + i][:, None]
        return y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return _encode4(x)


def _value(rows, s, i):
    if s["dtype"] == "bf16":
        return rows
    if s["dtype"] == "fp8":
        return (rows.view(torch.float8_e4m3fn).float() *
                s["scales"][i][:, None]).bfloat16()
    return _decode4(rows).bfloat16()


def _plain_write(s):
    blk, slot = _slots(s)
    k, out = s["k_new"], ()
    if s["case"]["axes"]:
        k = _rotate(k, s, D, "half", False)
        out = (_rotate(s["q"], s, D, "half", False),)
    s["k"][blk, :, slot] = _stored(k, s, 0)
    s["v"][blk, :, slot] = _stored(s["v_new"], s, 1)
    return out + _plain_read(s)


def _plain_read(s):
    blk, slot = _slots(s)
    return (_value(s["k"][blk, :, slot], s, 0),
            _value(s["v"][blk, :, slot], s, 1))


def _plain_attend(s):
    """softmax(q K^T / sqrt(D)) V of every new row over the positions up to
    its own (within the window): ragged rows padded to the longest."""
    case, bs = s["case"], s["case"]["block"]
    hk = case["n_kv"]
    grp = case["n_h"] // hk
    lens, rs = s["seq_lens"].long(), s["row_start"].long()
    L, R = s["max_seq_len"], s["max_rows"]
    n = rs[1:] - rs[:-1]
    pos = torch.arange(L, device="cuda")
    blk = s["table"].long()[:, pos // bs]
    k = _decode4(s["k"][blk, :, pos % bs]).transpose(1, 2)
    r = torch.arange(R, device="cuda")
    row = (rs[:-1, None] + r).clamp(max=s["q"].shape[0] - 1)
    B = lens.numel()
    q = s["q"].float()[row].view(B, R, hk, grp, D).permute(0, 2, 3, 1, 4)
    x = torch.matmul(q.reshape(B, hk, grp * R, D), k.transpose(2, 3))
    del k
    x = x.view(B, hk, grp, R, L).mul_(D ** -0.5)
    at = lens[:, None] - n[:, None] + r                     # [B][R]
    seen = pos <= at[..., None]
    if case["window"]:
        seen &= pos > at[..., None] - case["window"]
    x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(m.clamp(min=-3e38)).exp_()
    l = x.sum(-1, keepdim=True)
    v = _decode4(s["v"][blk, :, pos % bs]).transpose(1, 2)
    o = torch.matmul(x.view(B, hk, grp * R, L), v).view(B, hk, grp, R, D)
    o = torch.where(l > 0, o / l, 0)
    lse = (m + l.log())[..., 0]
    b = torch.repeat_interleave(torch.arange(B, device="cuda"), n,
                                output_size=s["q"].shape[0])
    i = torch.arange(s["q"].shape[0], device="cuda") - rs[b]
    out = o.permute(0, 3, 1, 2, 4)[b, i].reshape(-1, case["n_h"], D)
    return (out.bfloat16(),
            lse.permute(0, 3, 1, 2)[b, i].reshape(-1, case["n_h"]))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    kind = s["case"]["kind"]
    if own:
        return _own(s, kind)
    if kind == "rope":
        c = s["case"]
        return (_rotate(s["q"], s, c["d_rot"], c["pairing"], c["inverse"]),
                _rotate(s["k"], s, c["d_rot"], c["pairing"], c["inverse"]))
    if kind == "write":
        return _plain_write(s)
    if kind == "read":
        return _plain_read(s)
    return _plain_attend(s)


def _own(s, kind):
    import kv_cache_decode_gqa_gb300 as K
    case = s["case"]
    if kind == "rope":
        return K.rope(s["plan"], s["positions"], s["q"], s["k"],
                      inverse=case["inverse"])
    sc = s["scales"] or (None,) * 4
    cache = K.PagedCache(s["k"], s["v"], case["block"], case["n_kv"], D,
                         s["dtype"], *sc)
    if kind == "write":
        rope = {}
        if case["axes"]:
            rope = dict(rope=s["plan"], positions=s["positions"], q=s["q"])
        q = K.kv_write(cache, s["table"], s["start"], s["row_start"],
                       s["k_new"], s["v_new"], **rope)
        kv = K.kv_read(cache, s["table"], s["start"], s["row_start"],
                       case["rows"])
        return ((q,) if case["axes"] else ()) + tuple(kv)
    if kind == "read":
        return K.kv_read(cache, s["table"], s["start"], s["row_start"],
                         s["rows"])
    if kind == "extend":
        return K.gqa_extend(cache, s["table"], s["seq_lens"],
                            s["max_seq_len"], s["q"], s["row_start"],
                            s["max_rows"], window=case["window"])
    # one new token a sequence: row b belongs to sequence b
    return K.gqa_extend(cache, s["table"], s["seq_lens"], s["max_seq_len"],
                        s["q"], window=case["window"])


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _seen(case):
    """Expected positions read per sequence, and (row, position) pairs."""
    B, c, w = case["batch"], case["context"], case["window"]
    n = case["rows"] / B if case["kind"] == "extend" else 1
    past = c if B == 1 else 9 * c / 16
    if case["kind"] == "decode":
        past = max(past - 1, 0)
    total = past + n
    reach = min(total, w + n - 1) if w else total
    per_row = past + (n + 1) / 2
    return reach, n * (min(per_row, w) if w else per_row)


def work(case):
    kind = case["kind"]
    if kind == "rope":
        heads = case["n_h"] + case["n_kv"]
        return {"bytes": case["rows"] * (heads * case["d"] * 4 +
                                         4 * case["axes"]),
                "flops": 3 * case["rows"] * heads * case["d_rot"]}
    store = {"bf16": 2 * D, "fp8": D, "mxfp4": ROW4}
    if kind in ("write", "read"):
        kv = 2 * case["rows"] * case["n_kv"]
        b = kv * (store[case["dtype"]] + 2 * D)
        if kind == "write":
            b *= 2
            b += case["rows"] * (case["n_h"] * D * 4 + 4 * case["axes"])
        return {"bytes": b, "flops": kv * D}
    reach, pairs = _seen(case)
    B = case["batch"]
    rows = case["rows"] if kind == "extend" else B
    return {"bytes": int(B * reach * case["n_kv"] * 2 * ROW4 +
                         rows * case["n_h"] * (4 * D + 4)),
            "flops": int(B * pairs * case["n_h"] * 4 * D)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _near(y, grid):
    """Values of y >= 0 on `grid`, nearest, ties to the even index."""
    hi = torch.bucketize(y, grid).clamp(1, grid.numel() - 1)
    lo = hi - 1
    up = (y - grid[lo]) - (grid[hi] - y)
    return grid[torch.where((up > 0) | ((up == 0) & (hi % 2 == 0)), hi, lo)]


def _e4m3_grid():
    e = [m * 2.0 ** -9 for m in range(8)]
    e += [(1 + m / 8) * 2.0 ** x for x in range(-6, 9) for m in range(8)]
    return torch.tensor(e[:-1], dtype=torch.float64, device="cuda")  # <= 448


def _e4m3(y):
    return y.sign() * _near(y.abs(), _e4m3_grid())


def _mxfp4_value(x):
    x = x.double().reshape(*x.shape[:-1], -1, GROUP)
    sc = _e4m3(x.abs().amax(-1) / 6)[..., None]
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64,
                        device="cuda")
    y = torch.where(sc > 0, x / sc.clamp(min=1e-30), 0)
    return (y.sign() * _near(y.abs(), grid) * sc).flatten(-2)


def _turned(x, s, d_rot, pairing, inverse):
    x = x.double()
    half = d_rot // 2
    i = torch.arange(half, device="cuda")
    lo, hi = (i, i + half) if pairing == "half" else (2 * i, 2 * i + 1)
    ang = s["positions"].double()[s["axis"]] * s["freq"][:, None]
    turn = torch.polar(torch.ones_like(ang), -ang if inverse else ang).t()
    z = torch.complex(x[..., lo], x[..., hi]) * turn[:, None]
    out = x.clone()
    out[..., lo], out[..., hi] = z.real, z.imag
    return out


def _read_exact(s, i):
    """fp64 values [block][head][slot][D] of the whole cache tensor."""
    t = s["kv"[i]]
    if s["dtype"] == "bf16":
        return t.double()
    if s["dtype"] == "fp8":
        return (t.view(torch.float8_e4m3fn).double() *
                s["scales"][i].double()[None, :, None, None])
    pair = torch.stack([t[..., :64] % 16, t[..., :64] // 16], -1).flatten(-2)
    m = (pair % 8).double()
    mag = torch.where(m < 4, m / 2, torch.where(m < 6, m - 2, 2 * m - 8))
    sc = t[..., 64:].double()
    e, f = (sc // 8), sc % 8
    sv = torch.where(e > 0, (1 + f / 8) * 2.0 ** (e - 7), f * 2.0 ** -9)
    val = torch.where(pair >= 8, -mag, mag)
    return val * sv.repeat_interleave(GROUP, -1)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "rope":
        a = (s, case["d_rot"], case["pairing"], case["inverse"])
        return _turned(s["q"], *a), _turned(s["k"], *a)
    if kind == "write":
        k, v, out = s["k_new"], s["v_new"], ()
        if case["axes"]:
            out = (_turned(s["q"], s, D, "half", False),)
            # the cache takes the rotated key as bf16
            k = _turned(k, s, D, "half", False).float().bfloat16()
        kv = []
        for i, x in enumerate((k, v)):
            if s["dtype"] == "bf16":
                kv.append(x.double())
            elif s["dtype"] == "fp8":
                y = x.double() * s["scales"][2 + i].double()[:, None]
                kv.append(_e4m3(y) * s["scales"][i].double()[:, None])
            else:
                kv.append(_mxfp4_value(x))
        return out + tuple(kv)
    bs, rs = case["block"], s["row_start"].tolist()
    if kind == "read":
        start = s["start"].tolist()
        both = ([], [])
        for b in range(case["batch"]):
            pos = start[b] + torch.arange(rs[b + 1] - rs[b], device="cuda")
            blk = s["table"][b].long()[pos // bs]
            for i in range(2):
                sub = dict(s, **{"kv"[i]: s["kv"[i]][blk, :, pos % bs][
                    :, :, None]})
                both[i].append(_read_exact(sub, i)[:, :, 0])
        return torch.cat(both[0]), torch.cat(both[1])
    outs, lses = [], []
    grp = case["n_h"] // case["n_kv"]
    for b, T in enumerate(s["seq_lens"].tolist()):
        n = rs[b + 1] - rs[b]
        pos = torch.arange(T, device="cuda")
        blk = s["table"][b].long()[pos // bs]
        sub = dict(s, k=s["k"][blk, :, pos % bs][:, :, None],
                   v=s["v"][blk, :, pos % bs][:, :, None])
        kk = _read_exact(sub, 0)[:, :, 0]
        vv = _read_exact(sub, 1)[:, :, 0]
        at = T - n + torch.arange(n, device="cuda")
        hide = pos > at[:, None]
        if case["window"]:
            hide |= pos <= at[:, None] - case["window"]
        q = s["q"][rs[b]:rs[b + 1]].double()
        oh, lh = [], []
        for h in range(case["n_h"]):
            x = q[:, h] @ kk[:, h // grp].t() / math.sqrt(D)
            x = x.masked_fill(hide, -math.inf)
            lse = torch.logsumexp(x, -1)
            oh.append(torch.exp(x - lse[:, None]) @ vv[:, h // grp])
            lh.append(lse)
        outs.append(torch.stack(oh, 1))
        lses.append(torch.stack(lh, 1))
    return torch.cat(outs), torch.cat(lses)
