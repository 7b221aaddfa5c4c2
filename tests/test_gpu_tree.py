"""Drafted trees and cross attention on the GPU (include/kvd_tree.h) against
fp64 formulas. Tolerances are sums of the roundings each result goes
through."""
import dataclasses
import gc
import math
import os
import subprocess
import sys
import weakref

import numpy as np
import pytest
import torch

import kv_cache_decode_gqa_gb300 as K

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
HALF_BF16 = torch.finfo(BF).eps / 2


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(BF)


def _starts(n):
    return _i32([0] + [int(x) for x in np.cumsum(n)])


@pytest.fixture(autouse=True)
def _no_device_error():
    K.device_error()
    yield
    torch.cuda.synchronize()


# ---------------------------------------------------------------------------
# plans
# ---------------------------------------------------------------------------
def _random_tree(rng, n, roots=0.05):
    p = [-1] * n
    for i in range(1, n):
        p[i] = -1 if rng.random() < roots else int(rng.integers(0, i))
    return p


def _plan_ref(parents, start, n, words, window):
    masks, positions = [], []
    at = 0
    for b, k in enumerate(n):
        chains = []
        for i in range(k):
            p = parents[at + i]
            chains.append((chains[p] if p >= 0 else []) + [i])
            seen = chains[i][-window:] if window else chains[i]
            bits = sum(1 << j for j in seen)
            masks.append([(bits >> (32 * w)) & 0xffffffff
                          for w in range(words)])
            positions.append(start[b] + len(chains[i]) - 1)
        at += k
    m = np.array(masks, dtype=np.uint32).reshape(-1, words)
    return (torch.from_numpy(m.view(np.int32)).cuda(), _i32(positions))


PLANS = [
    # nodes of each sequence, bound, window
    ([1], 1, 0),
    ([0], 1, 0),
    ([5, 0, 1, 33, 0], 33, 0),
    ([256], 256, 0),
    ([64, 63, 65, 256, 31, 32], 256, 0),
    ([100, 7], 120, 3),
    ([40], 40, 1),
    ([3] * 300, 3, 0),
]


@pytest.mark.parametrize("case", PLANS)
def test_tree_plan(case):
    n, bound, window = case
    rng = np.random.default_rng(sum(n))
    parents = [p for k in n for p in _random_tree(rng, k)]
    start = rng.integers(0, 10 ** 6, len(n)).tolist()
    if not parents:
        parents = [-1]           # a row that no sequence owns
    masks, pos = K.tree_plan(_i32(parents), _i32(start), _starts(n), bound,
                             window=window)
    words = (bound + 31) // 32
    assert masks.shape == (len(parents), words)
    want, wpos = _plan_ref(parents, start, n, words, window)
    assert torch.equal(masks[:sum(n)], want[:sum(n)])
    assert torch.equal(pos[:sum(n)], wpos[:sum(n)])
    assert K.device_error() == 0


def test_tree_plan_chain_of_all_nodes_and_positions_near_the_end():
    n = K.TREE_NODES
    masks, pos = K.tree_plan(_i32(range(-1, n - 1)), _i32([2 ** 31 - n]),
                             _starts([n]), n)
    bits = masks.cpu().numpy().view(np.uint32)
    for i in (0, 1, 31, 32, 100, 255):
        value = sum(int(w) << (32 * k) for k, w in enumerate(bits[i]))
        assert value == (1 << (i + 1)) - 1
    assert pos[-1].item() == 2 ** 31 - 1
    assert K.device_error() == 0


def test_tree_plan_bad_parents_and_lists():
    n = [4, 3]
    good = [-1, 0, 1, 0, -1, 0, 0]
    bad = list(good)
    bad[2], bad[5] = 2, -5           # itself; below -1
    masks, pos = K.tree_plan(_i32(bad), _i32([10, 20]), _starts(n), 4)
    assert K.device_error() == K.DEVERR_INDEX
    fixed = list(good)
    fixed[2] = fixed[5] = -1
    want, wpos = _plan_ref(fixed, [10, 20], n, 1, 0)
    assert torch.equal(masks, want) and torch.equal(pos, wpos)
    # a sequence longer than the bound, and lists that descend or end past
    # the rows: those sequences' rows stay, the ones before are done
    for rows, first_kept in (([0, 2, 7], 2), ([0, 4, 2], 4), ([0, 4, 9], 4),
                             ([-1, 3, 7], 0)):
        masks = torch.full((7, 1), 77, dtype=torch.int32, device="cuda")
        pos = torch.full((7,), 77, dtype=torch.int32, device="cuda")
        K.tree_plan(_i32(good), _i32([10, 20]), _i32(rows), 4, masks=masks,
                    positions=pos)
        assert K.device_error() & K.DEVERR_LEN
        if first_kept:
            assert bool((pos[:first_kept] != 77).all())
            assert bool((pos[first_kept:] == 77).all())
            assert bool((masks[first_kept:] == 77).all())


# ---------------------------------------------------------------------------
# caches and their fp64 values
# ---------------------------------------------------------------------------
def _cache(g, blocks, n_kv, bs, dtype, d):
    kw, out = {}, []
    for _ in range(2):
        shape = (blocks, n_kv, bs)
        if dtype == "bf16":
            out.append(_randn(g, *shape, d))
        elif dtype == "fp8":
            x = torch.randn((*shape, d), generator=g, device="cuda") * 20
            out.append(x.to(torch.float8_e4m3fn).view(torch.uint8))
        else:
            codes = torch.randint(0, 256, (*shape, d // 2), generator=g,
                                  device="cuda", dtype=torch.uint8)
            sc = torch.rand((*shape, d // 16), generator=g, device="cuda")
            out.append(torch.cat([codes, (0.05 + 0.5 * sc).to(
                torch.float8_e4m3fn).view(torch.uint8)], -1))
    if dtype == "fp8":
        s = 0.02 + 0.05 * torch.rand(2, n_kv, generator=g, device="cuda")
        kw = dict(k_scale=s[0].contiguous(), v_scale=s[1].contiguous(),
                  k_inv_scale=(1 / s[0]).contiguous(),
                  v_inv_scale=(1 / s[1]).contiguous())
    return K.PagedCache(out[0], out[1], bs, n_kv, d, dtype, **kw)


E2M1 = [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]


def _rows64(c, which, blk, slot):
    """fp64 [n][n_kv][d] of the cached rows at these blocks and slots."""
    t = (c.k if which == 0 else c.v)[blk, :, slot]
    if c.dtype == "bf16":
        return t.double()
    if c.dtype == "fp8":
        s = c.k_scale if which == 0 else c.v_scale
        return t.view(torch.float8_e4m3fn).double() * s.double()[:, None]
    grid = torch.tensor(E2M1, dtype=torch.float64, device=t.device)
    d = c.head_dim
    codes = t[..., :d // 2]
    v = torch.stack([grid[(codes % 16).long()], grid[(codes // 16).long()]],
                    -1).flatten(-2)
    s = t[..., d // 2:].contiguous().view(torch.float8_e4m3fn).double()
    return v * s.repeat_interleave(16, -1)


def _table(g, lens, bs, width=None):
    per = [max((n + bs - 1) // bs, 1) for n in lens]
    total = sum(per) + 2
    perm = torch.randperm(total, generator=g, device="cuda").tolist()
    width = width or max(per)
    rows, at = [], 0
    for n in per:
        # entries past a sequence's length are never followed
        rows.append(perm[at:at + n] + [-7] * (width - n))
        at += n
    return _i32(rows), total


def _reference(c, bt, lens, q, n, sees, scale=None):
    """fp64 (out, lse, what the roundings may add to either) of rows whose
    visible positions are sees(b) -> bool [n_b][T_b]."""
    d = c.head_dim
    scale = scale or d ** -0.5
    n_h = q.shape[1]
    grp = n_h // c.n_kv
    outs, lses, otol, ltol = [], [], [], []
    at = 0
    for b, (k, T) in enumerate(zip(n, lens)):
        x = q[at:at + k].double().view(k, c.n_kv, grp, d)
        at += k
        if k == 0:
            continue
        if T == 0:
            z = torch.zeros(k, n_h, d, dtype=torch.float64, device="cuda")
            outs.append(z)
            lses.append(z[..., 0] - math.inf)
            otol.append(z)
            ltol.append(z[..., 0])
            continue
        pos = torch.arange(T, device="cuda")
        blk, slot = bt[b].long()[pos // c.block_size], pos % c.block_size
        kk, vv = _rows64(c, 0, blk, slot), _rows64(c, 1, blk, slot)
        ok = sees(b)[:, None, None]                       # [k][1][1][T]
        s = torch.einsum("rhgd,phd->rhgp", x, kk) * scale
        mag = torch.einsum("rhgd,phd->rhgp", x.abs(), kk.abs()) * scale
        mag = torch.where(ok, mag, 0.0).amax(-1)
        s = s.masked_fill(~ok, -math.inf)
        lse = torch.logsumexp(s, -1)
        p = torch.nan_to_num(torch.exp(s - lse[..., None]), nan=0.0)
        o = torch.einsum("rhgp,phd->rhgd", p, vv)
        ov = torch.einsum("rhgp,phd->rhgd", p, vv.abs())
        # scores: d + 8 fp32 additions and products of terms up to mag (a
        # step of 2^-23 each), the exponential's 2^-22
        ds = (d + 8) * 2.0 ** -23 * mag + 2.0 ** -22
        acc = (T + 64) * 2.0 ** -24                # fp32 sums over positions
        # probabilities to 16 bits (bf16 at the least), the output to bf16
        otol.append((HALF_BF16 * o.abs() + ov * (
            HALF_BF16 + 2 * ds + 2 * acc)[..., None]).reshape(k, n_h, d))
        ltol.append((ds + acc + 2.0 ** -21 * (
            1 + torch.nan_to_num(lse, neginf=0.0).abs())).reshape(k, n_h))
        outs.append(o.reshape(k, n_h, d))
        lses.append(lse.reshape(k, n_h))
    return tuple(torch.cat(x) for x in (outs, lses, otol, ltol))


def _check(got, ref):
    out, lse = got
    o, l, otol, ltol = ref
    m = o.shape[0]
    out, lse = out[:m].double(), lse[:m].double()
    assert bool(torch.isfinite(out).all())
    assert bool(((out - o).abs() <= otol + 1e-38).all()), (
        ((out - o).abs() / (otol + 1e-38)).max().item())
    empty = torch.isneginf(l)
    assert torch.equal(torch.isneginf(lse), empty)
    assert bool((out[empty] == 0).all())
    assert bool(((lse - l).abs()[~empty] <= ltol[~empty]).all())


def _bits(masks, n, words):
    """bool [n][32 words] of packed rows."""
    m = masks.cpu().numpy().view(np.uint32).reshape(n, words)
    b = (m[:, :, None] >> np.arange(32, dtype=np.uint32)) & 1
    return torch.from_numpy(b.astype(bool).reshape(n, words * 32)).cuda()


def _tree_sees(n, past, masks, words, lo=None):
    at = [0] + list(np.cumsum(n))

    def sees(b):
        k = n[b]
        bits = _bits(masks[at[b]:at[b + 1]], k, words)[:, :k]
        ctx = torch.ones(k, past[b], dtype=torch.bool, device="cuda")
        if lo is not None:
            first = torch.tensor(lo[at[b]:at[b + 1]], device="cuda")
            ctx &= torch.arange(past[b], device="cuda") >= first[:, None]
        return torch.cat([ctx, bits], 1)
    return sees


# ---------------------------------------------------------------------------
# attention of trees
# ---------------------------------------------------------------------------
TREES = [
    # dtype, d, n_h, n_kv, block, nodes, context, bound
    ("bf16", 128, 8, 2, 64, [1], [0], 1),
    ("bf16", 128, 8, 2, 64, [1], [1], 1),
    ("bf16", 128, 8, 1, 16, [7, 16, 1], [100, 0, 1999], 16),
    ("bf16", 128, 64, 8, 64, [16], [4000], 16),
    ("bf16", 128, 16, 2, 64, [64, 33, 0, 5], [300, 127, 9, 1025], 64),
    ("bf16", 128, 12, 4, 8, [40, 3], [130, 77], 40),
    ("bf16", 128, 7, 1, 48, [50, 9], [511, 63], 60),
    ("bf16", 128, 32, 1, 32, [17, 256], [640, 384], 256),
    ("bf16", 128, 128, 1, 64, [5], [700], 5),
    ("bf16", 64, 16, 16, 64, [12, 12], [500, 60], 12),
    ("bf16", 64, 6, 2, 16, [100, 1, 29], [33, 2000, 128], 128),
    ("bf16", 64, 4, 1, 1, [9], [21], 9),
    ("bf16", 128, 4, 1, 3, [9], [200], 9),
    ("bf16", 128, 8, 8, 20, [3, 30], [130, 45], 30),
    ("fp8", 128, 8, 1, 64, [1, 12, 30], [0, 4000, 129], 30),
    ("fp8", 128, 64, 8, 16, [64, 12], [200, 1000], 64),
    ("fp8", 64, 12, 4, 32, [77, 1], [300, 64], 80),
    ("fp8", 64, 8, 2, 5, [20], [99], 20),
    ("mxfp4", 128, 8, 1, 64, [1, 12, 60], [0, 3000, 129], 60),
    ("mxfp4", 128, 64, 8, 16, [64, 5], [250, 1000], 64),
    ("mxfp4", 128, 6, 2, 2, [33], [70], 33),
    ("mxfp4", 128, 3, 3, 128, [256, 2], [1000, 130], 256),
]


def _setup(case, seed, width=None):
    dtype, d, n_h, n_kv, bs, n, past, bound = case
    g = _gen(seed)
    lens = [a + b for a, b in zip(n, past)]
    bt, blocks = _table(g, lens, bs, width)
    c = _cache(g, blocks, n_kv, bs, dtype, d)
    rng = np.random.default_rng(seed)
    parents = [p for k in n for p in _random_tree(rng, k)]
    masks, pos = K.tree_plan(_i32(parents), _i32(past), _starts(n), bound)
    q = _randn(g, sum(n), n_h, d)
    return c, bt, lens, masks, pos, q


@pytest.mark.parametrize("case", TREES)
def test_gqa_tree(case):
    dtype, d, n_h, n_kv, bs, n, past, bound = case
    c, bt, lens, masks, pos, q = _setup(case, 7 * sum(n) + d)
    got = K.gqa_tree(c, bt, _i32(lens), max(lens), q, _starts(n), bound,
                     masks)
    words = (bound + 31) // 32
    _check(got, _reference(c, bt, lens, q, n,
                           _tree_sees(n, past, masks, words)))
    assert K.device_error() == 0


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64),
                                     ("fp8", 128), ("mxfp4", 128)])
def test_gqa_tree_window_and_starts(dtype, d):
    n, past, bound = [20, 7, 60, 3], [500, 40, 1300, 0], 64
    case = (dtype, d, 12, 2, 16, n, past, bound)
    c, bt, lens, masks, pos, q = _setup(case, 5)
    starts = [0, 10, 1299, 5]
    for window in (1, 64, 300, 2 ** 31 - 1):
        owner = np.repeat(np.arange(4), n)
        lo = [max(starts[b], int(p) + 1 - window)
              for b, p in zip(owner, pos.tolist())]
        got = K.gqa_tree(c, bt, _i32(lens), max(lens), q, _starts(n), bound,
                         masks, positions=pos, window=window,
                         window_start=_i32(starts))
        _check(got, _reference(c, bt, lens, q, n,
                               _tree_sees(n, past, masks, 2, lo)))
    assert K.device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "mxfp4"])
def test_gqa_tree_any_masks_empty_rows_and_bits_past_the_tree(dtype):
    n, past, bound = [33, 5, 70], [0, 129, 0], 96
    case = (dtype, 128, 8, 1, 64, n, past, bound)
    c, bt, lens, _, _, q = _setup(case, 11)
    g = _gen(3)
    masks = torch.randint(-2 ** 31, 2 ** 31, (sum(n), 3), generator=g,
                          device="cuda").to(torch.int32)
    masks[::5] = 0               # rows without context see nothing then
    masks[7] = -1
    got = K.gqa_tree(c, bt, _i32(lens), max(lens), q, _starts(n), bound,
                     masks)
    _check(got, _reference(c, bt, lens, q, n, _tree_sees(n, past, masks, 3)))
    assert bool(torch.isneginf(got[1][0]).all())
    assert K.device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "mxfp4"])
def test_what_lies_past_the_lengths_is_not_used(dtype):
    """Slots behind a sequence (of its own last block too) and before its
    start hold NaN and infinities; no result changes."""
    d, bs, n, past = 128, 64, [9, 40], [200, 117]
    case = (dtype, d, 16, 2, bs, n, past, 40)
    c, bt, lens, masks, pos, q = _setup(case, 13)
    starts = [70, 3]
    args = (bt, _i32(lens), max(lens), q, _starts(n), 40, masks)
    want = K.gqa_tree(c, *args, window_start=_i32(starts))
    dirty = dataclasses.replace(c, k=c.k.clone(), v=c.v.clone())
    keep = torch.zeros(c.num_blocks, bs, dtype=torch.bool, device="cuda")
    for b, T in enumerate(lens):
        p = torch.arange(starts[b], T, device="cuda")
        keep[bt[b].long()[p // bs], p % bs] = True
    gone = ~keep[:, None, :].expand(-1, 2, -1)
    for t in (dirty.k, dirty.v):
        t[gone] = float("nan") if dtype == "bf16" else 0x7f
    got = K.gqa_tree(dirty, *args, window_start=_i32(starts))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    first = _i32(starts)
    want = K.gqa_cross(c, *args[:-3], args[4], 40, first=first)
    got = K.gqa_cross(dirty, *args[:-3], args[4], 40, first=first)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert K.device_error() == 0


@pytest.mark.parametrize("dtype,d", [("fp8", 128), ("fp8", 64),
                                     ("mxfp4", 128)])
def test_probabilities_beside_f16_values_are_f16(dtype, d):
    """Few positions, so that their roundings show: over fp8 and MXFP4 caches
    the probabilities are off by half a step of f16, which bf16's would
    exceed."""
    lens, n, n_h, n_kv, bs = [2, 3, 4, 2, 5], [40] * 5, 32, 4, 16
    g = _gen(79 + d)
    bt, blocks = _table(g, lens, bs)
    c = _cache(g, blocks, n_kv, bs, dtype, d)
    q = _randn(g, sum(n), n_h, d) * 0.2
    out, lse = K.gqa_cross(c, bt, _i32(lens), max(lens), q, _starts(n), 40)
    o, l, _, ltol = _reference(c, bt, lens, q, n, _cross_sees(n, lens, None))
    worst, at = 0.0, 0
    for b, (k, T) in enumerate(zip(n, lens)):
        pos = torch.arange(T, device="cuda")
        blk, slot = bt[b].long()[pos // bs], pos % bs
        kk, vv = _rows64(c, 0, blk, slot), _rows64(c, 1, blk, slot)
        x = q[at:at + k].double().view(k, n_kv, n_h // n_kv, d)
        s = torch.einsum("rhgd,phd->rhgp", x, kk) * d ** -0.5
        mag = torch.einsum("rhgd,phd->rhgp", x.abs(), kk.abs()).amax(
            -1) * d ** -0.5
        p = torch.softmax(s, -1)
        ov = torch.einsum("rhgp,phd->rhgd", p, vv.abs())
        # as in _reference, with a probability off by 2^-11, or by 2^-25
        # below f16's normal range where the largest is 2^7 or more
        ds = (d + 8) * 2.0 ** -23 * mag + 2.0 ** -22
        acc = (T + 64) * 2.0 ** -24
        tol = HALF_BF16 * o[at:at + k].abs() + (
            (2.0 ** -11 + 2 * ds + 2 * acc)[..., None] * ov +
            2.0 ** -32 * vv.abs().sum(0)[None, :, None]).reshape(k, n_h, d)
        err = (out[at:at + k].double() - o[at:at + k]).abs()
        assert bool((err <= tol).all()), (err / tol).max().item()
        # the same with the weights relative to the largest in bf16
        w = p / p.amax(-1, keepdim=True)
        w = w.to(BF).double() / w.sum(-1, keepdim=True)
        bad = torch.einsum("rhgp,phd->rhgd", w, vv).reshape(k, n_h, d)
        worst = max(worst, ((bad - o[at:at + k]).abs() / tol).max().item())
        at += k
    assert bool(((lse.double() - l).abs() <= ltol).all())
    assert worst > 1.5
    assert K.device_error() == 0


def test_masked_nodes_with_infinite_keys():
    """A node's key may be anything where a row's mask leaves it out."""
    case = ("bf16", 128, 8, 1, 64, [6], [130], 6)
    c, bt, lens, masks, pos, q = _setup(case, 17)
    masks = _i32([[1 << i] for i in range(6)])   # every node alone
    args = (bt, _i32(lens), lens[0], q, _starts([6]), 6, masks)
    want = K.gqa_tree(c, *args)
    p = 130 + 4
    c.k[bt[0, p // 64].item(), 0, p % 64] = float("inf")
    got = K.gqa_tree(c, *args)
    rows = torch.tensor([0, 1, 2, 3, 5], device="cuda")
    assert torch.equal(got[0][rows], want[0][rows])
    assert torch.equal(got[1][rows], want[1][rows])


# ---------------------------------------------------------------------------
# what no row sees
# ---------------------------------------------------------------------------
def _spoil(c, bt, b, positions):
    """NaN (infinities beside them) in K and V at these positions."""
    for i, p in enumerate(positions):
        blk, slot = bt[b, p // c.block_size].item(), p % c.block_size
        for t in (c.k, c.v):
            t[blk, :, slot] = (0x7f if c.dtype != "bf16" else
                               math.inf if i % 2 else math.nan)


UNSEEN = [("bf16", 128, 8, 2, 64), ("bf16", 128, 12, 1, 16),
          ("bf16", 64, 6, 2, 5), ("fp8", 128, 8, 2, 64), ("fp8", 64, 4, 1, 16),
          ("mxfp4", 128, 12, 1, 16), ("mxfp4", 128, 4, 2, 64)]


@pytest.mark.parametrize("shape", UNSEEN)
def test_nodes_that_no_row_sees_may_hold_anything(shape):
    """Spare nodes of a fixed budget, whose bits are clear in every mask: their
    rows of K and V change nothing, and rows that see nothing stay empty."""
    dtype, d, n_h, n_kv, bs = shape
    n, past, bound = [40, 6, 200, 33, 1], [100, 0, 5000, 127, 0], 200
    case = (dtype, d, n_h, n_kv, bs, n, past, bound)
    c, bt, lens, masks, pos, q = _setup(case, 61)
    spare = [[3, 31, 32, 39], [0, 2, 3, 4, 5], list(range(150, 200)) + [7, 64],
             [32], [0]]
    rs = _starts(n)
    for b, nodes in enumerate(spare):
        for j in nodes:
            masks[rs[b]:rs[b + 1], j // 32] &= ~(1 << (j % 32)) if (
                j % 32 != 31) else 0x7fffffff
    masks[45] = 0                # (no context either: this row sees nothing)
    args = (bt, _i32(lens), max(lens), q, rs, bound, masks)
    want = K.gqa_tree(c, *args)
    _check(want, _reference(c, bt, lens, q, n,
                            _tree_sees(n, past, masks, 7)))
    for b, nodes in enumerate(spare):
        _spoil(c, bt, b, [past[b] + j for j in nodes])
    got = K.gqa_tree(c, *args)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for row in (45, sum(n) - 1):
        assert bool((got[0][row] == 0).all())
        assert bool(torch.isneginf(got[1][row]).all())
    assert K.device_error() == 0


@pytest.mark.parametrize("shape", UNSEEN)
@pytest.mark.parametrize("window", [1, 30, 200])
def test_context_before_every_window_may_hold_anything(shape, window):
    """No node at the tree's first position: the context before the lowest
    window of a sequence is in no row's, and may hold anything."""
    dtype, d, n_h, n_kv, bs = shape
    n, past, bound = [20, 50, 3, 70], [500, 140, 1000, 64], 70
    case = (dtype, d, n_h, n_kv, bs, n, past, bound)
    c, bt, lens, masks, _, q = _setup(case, 67)
    rng = np.random.default_rng(window)
    up = [[past[b] + int(x) for x in rng.integers(3, 40, k)]
          for b, k in enumerate(n)]
    up[2] = [past[2] + 5000] * 3          # past all of the context
    pos = [x for u in up for x in u]
    starts = [0, 0, 0, 50]
    owner = np.repeat(np.arange(4), n)
    lo = [max(starts[b], p + 1 - window) for b, p in zip(owner, pos)]
    args = (bt, _i32(lens), max(lens), q, _starts(n), bound, masks)
    kw = dict(positions=_i32(pos), window=window, window_start=_i32(starts))
    want = K.gqa_tree(c, *args, **kw)
    _check(want, _reference(c, bt, lens, q, n,
                            _tree_sees(n, past, masks, 3, lo)))
    for b, u in enumerate(up):
        first = max(starts[b], min(u) + 1 - window)
        _spoil(c, bt, b, range(max(0, past[b] - window - 3),
                               min(first, past[b])))
    got = K.gqa_tree(c, *args, **kw)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert K.device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "mxfp4"])
def test_rows_that_see_nothing_beside_values_that_are_not_finite(dtype):
    """A row that sees nothing gives 0 whatever its neighbours see, in units of
    one tile and of two."""
    for n_h, n, past in ((8, 6, 0), (64, 9, 0), (8, 200, 0)):
        case = (dtype, 128, n_h, 1, 64, [n], [past], n)
        c, bt, lens, masks, _, q = _setup(case, 71)
        masks[:] = -1
        masks[::3] = 0
        _spoil(c, bt, 0, [1, n - 1])
        out, lse = K.gqa_tree(c, bt, _i32(lens), max(lens), q, _starts([n]),
                              n, masks)
        assert bool((out[::3] == 0).all())
        assert bool(torch.isneginf(lse[::3]).all())
        assert bool(out[1].isnan().any())
        assert K.device_error() == 0


# ---------------------------------------------------------------------------
# cross attention
# ---------------------------------------------------------------------------
CROSS = [
    # dtype, d, n_h, n_kv, block, rows, states, first
    ("bf16", 128, 8, 2, 64, [1], [1], None),
    ("bf16", 128, 8, 2, 64, [3], [0], None),
    ("bf16", 128, 64, 8, 64, [300], [1500], None),
    ("bf16", 128, 64, 8, 16, [5, 0, 2000, 17], [700, 5, 129, 0], None),
    ("bf16", 64, 16, 16, 64, [5] * 8, [1500, 3, 64, 65, 1, 127, 128, 1000],
     None),
    ("bf16", 64, 20, 4, 32, [448, 200], [1500, 1499],
     [0, 700]),
    ("bf16", 128, 5, 5, 128, [129, 1], [257, 3000], [256, 3000]),
    ("bf16", 128, 24, 2, 7, [30], [100], None),
    ("fp8", 128, 32, 8, 32, [333, 100, 1], [900, 33, 2000], [100, 0, 1999]),
    ("fp8", 64, 8, 8, 64, [70, 300], [1000, 130], None),
    ("mxfp4", 128, 32, 8, 16, [333, 100, 1], [900, 33, 2000],
     [101, 1, 1999]),
    ("mxfp4", 128, 4, 4, 64, [60, 300], [1000, 130], None),
]


def _cross_sees(n, lens, first):
    def sees(b):
        ok = torch.arange(lens[b], device="cuda") >= (first[b] if first
                                                       else 0)
        return ok[None].expand(n[b], -1)
    return sees


@pytest.mark.parametrize("case", CROSS)
def test_gqa_cross(case):
    dtype, d, n_h, n_kv, bs, n, lens, first = case
    g = _gen(sum(n) + d)
    bt, blocks = _table(g, lens, bs)
    c = _cache(g, blocks, n_kv, bs, dtype, d)
    q = _randn(g, sum(n), n_h, d)
    for bound in (max(n), None):
        got = K.gqa_cross(c, bt, _i32(lens), max(lens), q, _starts(n), bound,
                          first=None if first is None else _i32(first))
        _check(got, _reference(c, bt, lens, q, n,
                               _cross_sees(n, lens, first)))
    assert K.device_error() == 0


@pytest.mark.parametrize("grp", [1, 2, 3, 4, 8, 16, 20])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64),
                                     ("fp8", 128), ("fp8", 64),
                                     ("mxfp4", 128)])
def test_gqa_cross_single_rows(dtype, d, grp):
    lens = [700, 1, 0, 64, 129]
    g = _gen(grp + d)
    bt, blocks = _table(g, lens, 64)
    c = _cache(g, blocks, 2, 64, dtype, d)
    q = _randn(g, 5, 2 * grp, d)
    for first in (None, [3, 0, 0, 64, 100]):
        got = K.gqa_cross(c, bt, _i32(lens), 700, q,
                          first=None if first is None else _i32(first))
        _check(got, _reference(c, bt, lens, q, [1] * 5,
                               _cross_sees([1] * 5, lens, first)))
    assert K.device_error() == 0


# ---------------------------------------------------------------------------
# how the attention is called
# ---------------------------------------------------------------------------
def test_scales_strides_outputs_and_large_scores():
    case = ("bf16", 128, 12, 4, 32, [21, 40], [300, 64], 40)
    dtype, d, n_h, n_kv, bs, n, past, bound = case
    c, bt, lens, masks, pos, _ = _setup(case, 19)
    g = _gen(2)
    # the query part of a fused projection, heads apart
    qkv = _randn(g, sum(n) + 3, n_h + 2 * n_kv, d) * 6
    q = qkv[:, :n_h]
    extra = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    m = torch.cat([masks, extra])
    out = torch.full((sum(n) + 3, n_h, d), 7.0, dtype=BF, device="cuda")
    lse = torch.full((sum(n) + 3, n_h), 7.0, device="cuda")
    got = K.gqa_tree(c, bt, _i32(lens), max(lens), q, _starts(n), bound, m,
                     scale=0.5, out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    _check((out, lse), _reference(c, bt, lens, q[:sum(n)], n,
                                  _tree_sees(n, past, masks, 2), 0.5))
    # rows behind the last sequence stay
    assert bool((out[-3:] == 7).all()) and bool((lse[-3:] == 7).all())
    again = K.gqa_tree(c, bt, _i32(lens), max(lens), q.contiguous(),
                       _starts(n), bound, m, scale=0.5, want_lse=False)
    assert again[1] is None
    assert torch.equal(again[0][:sum(n)], out[:sum(n)])
    assert K.device_error() == 0


def test_row_lists_that_do_not_fit():
    case = ("bf16", 128, 8, 2, 16, [6, 9, 5], [40, 50, 60], 9)
    c, bt, lens, masks, pos, q = _setup(case, 23)
    base = K.gqa_tree(c, bt, _i32(lens), max(lens), q, _starts([6, 9, 5]), 9,
                      masks)[0]
    # (list, rows that are done)
    for rows, done in (([0, 6, 3, 20], 6), ([0, 6, 15, 21], 15),
                       ([0, 6, 5, 3], 6), ([0, 6, 20, 20], 6)):
        out = torch.full_like(q, 7)
        K.gqa_tree(c, bt, _i32(lens), max(lens), q, _i32(rows), 9, masks,
                   out=out)
        assert K.device_error() & K.DEVERR_LEN
        assert torch.equal(out[:done], base[:done])
        assert bool((out[done:] == 7).all())
    # a sequence shorter than its tree
    short = list(lens)
    short[1] = 8
    out = torch.full_like(q, 7)
    K.gqa_tree(c, bt, _i32(short), max(lens), q, _starts([6, 9, 5]), 9, masks,
               out=out)
    assert K.device_error() & K.DEVERR_LEN
    assert torch.equal(out[:6], base[:6]) and torch.equal(out[15:], base[15:])
    assert bool((out[6:15] == 7).all())


def test_bad_blocks_are_flagged():
    for dtype in ("bf16", "fp8", "mxfp4"):
        case = (dtype, 128, 8, 2, 16, [6], [40], 6)
        c, bt, lens, masks, pos, q = _setup(case, 29)
        for bad in (-1, c.num_blocks, 2 ** 31 - 1):
            t = bt.clone()
            t[0, 1] = bad
            K.gqa_tree(c, t, _i32(lens), max(lens), q, _starts([6]), 6, masks)
            assert K.device_error() == K.DEVERR_BLOCK
            K.gqa_cross(c, t, _i32(lens), max(lens), q, _starts([6]), 6)
            assert K.device_error() == K.DEVERR_BLOCK


@pytest.mark.parametrize("dtype,d,batch", [("bf16", 128, 1000),
                                           ("fp8", 128, 1024),
                                           ("mxfp4", 128, 300),
                                           ("bf16", 64, 1024)])
def test_many_sequences(dtype, d, batch):
    """More sequences than a CTA has threads or keeps at hand: short ones, empty
    ones and a few long ones."""
    rng = np.random.default_rng(batch + d)
    n = rng.integers(0, 4, batch).tolist()
    lens = rng.integers(0, 60, batch).tolist()
    for b in (3, batch // 2, batch - 1):
        n[b], lens[b] = 9, 700
    n[7], lens[8] = 0, 0
    g = _gen(batch)
    bt, blocks = _table(g, lens, 16)
    c = _cache(g, blocks, 2, 16, dtype, d)
    q = _randn(g, sum(n), 6, d)
    got = K.gqa_cross(c, bt, _i32(lens), 700, q, _starts(n), 9)
    _check(got, _reference(c, bt, lens, q, n, _cross_sees(n, lens, None)))
    past = [max(x - k, 0) for x, k in zip(lens, n)]
    lens = [p + k for p, k in zip(past, n)]
    if max(lens) > 700:
        return
    bt, blocks = _table(g, lens, 16)
    c = _cache(g, blocks, 2, 16, dtype, d)
    masks, _ = K.tree_plan(_i32([-1] * sum(n)), _i32(past), _starts(n), 9)
    got = K.gqa_tree(c, bt, _i32(lens), 700, q, _starts(n), 9, masks)
    _check(got, _reference(c, bt, lens, q, n,
                           _tree_sees(n, past, masks, 1)))
    assert K.device_error() == 0


def test_keys_and_values_in_one_tensor():
    """K and V may be the same storage, or V may lie first."""
    n, lens = [5, 30], [200, 77]
    g = _gen(59)
    bt, blocks = _table(g, lens, 64)
    both = _randn(g, 2, blocks, 2, 64, 128)
    q = _randn(g, sum(n), 8, 128)
    for k, v in ((0, 0), (0, 1), (1, 0)):
        c = K.PagedCache(both[k], both[v], 64, 2, 128)
        got = K.gqa_cross(c, bt, _i32(lens), 200, q, _starts(n), 30)
        _check(got, _reference(c, bt, lens, q, n,
                               _cross_sees(n, lens, None)))
    assert K.device_error() == 0


def _far_apart():
    """Whether K and V could be placed 2^40 bytes and more apart, and then gave
    what they give side by side."""
    some = [torch.empty(mb << 19, dtype=BF, device="cuda")
            for mb in [*range(21, 121, 3), 200, 400, 1000, 2000]]
    at = [t.data_ptr() for t in some]
    ends = [some[at.index(f(at))] for f in (min, max)]
    if max(at) - min(at) < 2 ** 40:
        return False
    n, past, bound = [20, 40], [3000, 64], 40
    for d in (64, 128):
        case = ("bf16", d, 8, 2, 16, n, past, bound)
        c, bt, lens, masks, _, q = _setup(case, 83)
        args = (bt, _i32(lens), max(lens), q, _starts(n), bound)
        want = K.gqa_tree(c, *args, masks), K.gqa_cross(c, *args)
        low, high = (t[:c.k.numel()].view(c.k.shape) for t in ends)
        for k, v in ((low, high), (high, low)):
            k.copy_(c.k), v.copy_(c.v)
            x = dataclasses.replace(c, k=k, v=v)
            got = K.gqa_tree(x, *args, masks), K.gqa_cross(x, *args)
            for a, b in zip(got, want):
                assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert K.device_error() == 0
    return True


def test_keys_and_values_far_apart():
    """Allocations may lie anywhere: in a process that has made few, those of
    some tens of MB lie 2^48 bytes below the others here."""
    r = subprocess.run(
        [sys.executable, "-c", "import tests.test_gpu_tree as t; "
         "print('far' if t._far_apart() else 'near')"],
        cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
        capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    if r.stdout.split()[-1] == "near":
        pytest.skip("no two allocations that far apart")


def test_cache_beyond_32_bit_offsets():
    """Blocks at byte offsets past 2^32 and element offsets past 2^31."""
    bs, n_kv, d, n, past = 64, 8, 128, [5, 12], [200, 70]
    blocks = 2 ** 32 // (bs * n_kv * d * 2) * 2 + 40
    k = torch.empty(blocks, n_kv, bs, d, dtype=BF, device="cuda")
    v = torch.empty_like(k)
    c = K.PagedCache(k, v, bs, n_kv, d)
    lens = [a + b for a, b in zip(n, past)]
    bt = _i32([[blocks - 1, blocks - 3, 0, blocks - 9, 0],
               [5, blocks - 2, 0, 0, 0]])
    g = _gen(31)
    for b in set(bt.flatten().tolist()):
        k[b] = _randn(g, n_kv, bs, d)
        v[b] = _randn(g, n_kv, bs, d)
    rng = np.random.default_rng(1)
    parents = [p for x in n for p in _random_tree(rng, x)]
    masks, _ = K.tree_plan(_i32(parents), _i32(past), _starts(n), 12)
    q = _randn(g, sum(n), 64, d)
    got = K.gqa_tree(c, bt, _i32(lens), max(lens), q, _starts(n), 12, masks)
    _check(got, _reference(c, bt, lens, q, n, _tree_sees(n, past, masks, 1)))
    before = c.k[blocks - 1].clone(), c.k[blocks - 3].clone()
    # sequence 0: node rows 200 .. 204 lie in block blocks - 9
    K.kv_keep([c], bt, _i32(past), _i32([[1, 3], [0, 5]]), _i32([2, 2]))
    assert torch.equal(c.k[blocks - 1], before[0])
    assert torch.equal(c.k[blocks - 3], before[1])
    assert K.device_error() == 0


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("fp8", 64), ("fp8", 128),
                                     ("mxfp4", 128)])
@pytest.mark.parametrize("bs", [6, 100, 512, 10 ** 6])
def test_the_longest_lengths(dtype, d, bs):
    """2^31 - 256 positions, through a table that repeats three blocks, whose
    last block ends past 2^31; rows see the last few hundred."""
    T = 2 ** 31 - 256
    g = _gen(bs + d)
    c = _cache(g, 3, 1, bs, dtype, d)
    bt = (torch.arange(-(-T // bs), device="cuda", dtype=torch.int32) % 3)[None]
    # the same rows as a short sequence, in blocks that divide the long ones
    u = math.gcd(bs, 64)
    small = dataclasses.replace(
        c, block_size=u, **{x: getattr(c, x).view(3 * bs // u, 1, u, -1)
                            for x in ("k", "v")})
    first = T - 300
    base = first // u * u
    p = torch.arange(base, T, u, device="cuda")
    st = ((bt[0].long()[p // bs] * bs + p % bs) // u).to(torch.int32)[None]
    q = _randn(g, 7, 4, d)
    got = K.gqa_cross(c, bt, _i32([T]), T, q, _starts([7]), 7,
                      first=_i32([first]))
    assert K.device_error() == 0
    _check(got, _reference(small, st, [T - base], q, [7], _cross_sees(
        [7], [T - base], [first - base])))
    masks, pos = K.tree_plan(_i32([-1, 0, 0, 1, 2, 2, 4]), _i32([T - 7]),
                             _starts([7]), 7)
    for window in (0, 150):
        got = K.gqa_tree(c, bt, _i32([T]), T, q, _starts([7]), 7, masks,
                         positions=pos, window=window,
                         window_start=_i32([first]))
        assert K.device_error() == 0
        lo = [max(first, x + 1 - window) if window else first
              for x in pos.tolist()]
        _check(got, _reference(small, st, [T - base], q, [7], _tree_sees(
            [7], [T - base - 7], masks, 1, [x - base for x in lo])))


def test_streams_graphs_and_repeats():
    case = ("bf16", 128, 16, 2, 64, [20, 33], [3000, 900], 33)
    c, bt, lens, masks, pos, q = _setup(case, 37)
    args = (c, bt, _i32(lens), max(lens), q, _starts(case[5]), 33, masks)
    want = K.gqa_tree(*args)
    again = K.gqa_tree(*args)
    assert torch.equal(want[0], again[0]) and torch.equal(want[1], again[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = K.gqa_tree(*args, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other[0], want[0])
    # two graphs, each with a workspace of its own, replayed on two streams
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append((K.gqa_tree(*args), K.gqa_cross(*args[:-1])))
        graphs.append(gr)
    for _ in range(3):
        for o in outs:
            for t in o:
                t[0].zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        for o in outs:
            assert torch.equal(o[0][0], want[0])
            assert torch.equal(o[0][1], want[1])
    assert torch.equal(outs[0][1][0], outs[1][1][0])
    assert K.device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "mxfp4"])
def test_many_calls_give_the_same_bits(dtype):
    """Short units among long ones, call after call: what one call still
    reads, the next copy or call must not overwrite."""
    n, lens, first = [333, 100, 1], [900, 33, 2000], [100, 0, 1999]
    g = _gen(53)
    bt, blocks = _table(g, lens, 32)
    c = _cache(g, blocks, 8, 32, dtype, 128)
    q = _randn(g, sum(n), 32, 128)
    args = (c, bt, _i32(lens), 2000, q, _starts(n))
    fi = _i32(first)
    want = K.gqa_cross(*args, max(n), first=fi)
    _check(want, _reference(c, bt, lens, q, n, _cross_sees(n, lens, first)))
    outs = [K.gqa_cross(*args, max(n), first=fi) for _ in range(600)]
    assert all(torch.equal(o[0], want[0]) and torch.equal(o[1], want[1])
               for o in outs)


def test_workspace_of_the_stated_size():
    case = ("bf16", 128, 16, 2, 64, [20, 33], [3000, 900], 33)
    c, bt, lens, masks, pos, q = _setup(case, 41)
    a = (c, bt, _i32(lens), max(lens))
    size = K.attend_workspace_size(*a, q.shape[0], 16, 33)
    ws = torch.full((max(size, 256) + 256,), 0xff, dtype=torch.uint8,
                    device="cuda")
    want = K.gqa_tree(*a, q, _starts(case[5]), 33, masks)
    got = K.gqa_tree(*a, q, _starts(case[5]), 33, masks,
                     workspace=ws[:max(size, 256)])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bool((ws[max(size, 256):] == 0xff).all())
    if size:
        with pytest.raises(K.KvdError, match="workspace"):
            K.gqa_tree(*a, q, _starts(case[5]), 33, masks,
                       workspace=ws[:size - 256])


# ---------------------------------------------------------------------------
# accepted rows
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64),
                                     ("fp8", 128), ("mxfp4", 128),
                                     ("bf16", 576)])
@pytest.mark.parametrize("layers", [1, 3, 100])
def test_kv_keep(dtype, d, layers):
    g = _gen(layers)
    bs, n_kv = 16, 3 if d < 576 else 1
    start, width = [0, 13, 100, 40], 12
    bt, blocks = _table(g, [s + 64 for s in start], bs)
    rng = np.random.default_rng(layers)
    path = [sorted(rng.choice(40, width, replace=False).tolist()),
            list(range(width)), [0, 1] + list(range(5, width + 3)),
            list(range(50, 50 + width))]
    keep = [width, width, 5, 0]
    caches = [_cache(g, blocks, n_kv, bs, dtype, d) for _ in range(layers)]
    if d == 576:
        caches = [dataclasses.replace(c, v=None) for c in caches]
    want = [[None if t is None else t.clone() for t in (c.k, c.v)]
            for c in caches]
    for w in want:
        for t in w:
            if t is None:
                continue
            old = t.clone()
            for b in range(4):
                for j in range(keep[b]):
                    x, y = start[b] + path[b][j], start[b] + j
                    t[bt[b, y // bs].item(), :, y % bs] = old[
                        bt[b, x // bs].item(), :, x % bs]
    K.kv_keep(caches, bt, _i32(start), _i32(path), _i32(keep))
    for c, w in zip(caches, want):
        assert torch.equal(c.k, w[0])
        assert c.v is None or torch.equal(c.v, w[1])
    assert K.device_error() == 0


def test_kv_keep_of_keys_and_values_in_one_tensor():
    """A row is moved once: with two passes over one tensor the second could
    take rows that the first has replaced."""
    g = _gen(5)
    bt, blocks = _table(g, [64, 64], 16)
    layers = []
    for _ in range(40):
        c = _cache(g, blocks, 2, 16, "bf16", 128)
        layers.append(dataclasses.replace(c, v=c.k))
    path = [[0] + list(range(2, 40)), list(range(1, 40))]
    want = [c.k.clone() for c in layers]
    for t in want:
        old = t.clone()
        for b in range(2):
            for j, x in enumerate(path[b]):
                x, y = 7 + x, 7 + j
                t[bt[b, y // 16].item(), :, y % 16] = old[
                    bt[b, x // 16].item(), :, x % 16]
    K.kv_keep(layers, bt, _i32([7, 7]), _i32(path), _i32([39, 39]))
    for c, w in zip(layers, want):
        assert torch.equal(c.k, w)
    assert K.device_error() == 0


def test_a_tensor_listed_twice_is_refused():
    g = _gen(6)
    t = [_cache(g, 2, 2, 16, "bf16", 64) for _ in range(2)]
    a, b, c, d = t[0].k, t[0].v, t[1].k, t[1].v

    def cache(k, v):
        return dataclasses.replace(t[0], k=k, v=v)
    for x, y in ((cache(a, b), cache(a, c)), (cache(a, b), cache(c, b)),
                 (cache(a, b), cache(c, a)), (cache(a, a), cache(b, a)),
                 (cache(a, b), cache(a, b)), (cache(a, None), cache(a, None))):
        with pytest.raises(ValueError, match="twice"):
            K.CacheList([x, y])
    assert len(K.CacheList([cache(a, a), cache(b, b)]).caches) == 2
    assert len(K.CacheList([cache(a, b), cache(c, d)]).caches) == 2


def test_a_cache_list_keeps_the_tensors_it_points_to():
    """A layer that is given other tensors leaves the list the old ones: their
    memory is not handed out while the list's calls may write it."""
    g = _gen(8)
    bt, blocks = _table(g, [64], 16)
    c = _cache(g, blocks, 2, 16, "bf16", 64)
    old = [weakref.ref(c.k), weakref.ref(c.v)]
    want = [t.clone() for t in (c.k, c.v)]
    for t in want:
        t[bt[0, 0].item(), :, 3] = t[bt[0, 1].item(), :, 4]
    layers = K.CacheList([c])
    new = [torch.zeros_like(c.k), torch.zeros_like(c.v)]
    c.k, c.v = new
    gc.collect()
    assert all(r() is not None for r in old)
    K.kv_keep(layers, bt, _i32([3]), _i32([[17]]), _i32([1]))
    assert all(torch.equal(r(), w) for r, w in zip(old, want))
    assert not any(bool(t.any()) for t in new)
    assert K.device_error() == 0


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("mxfp4", 128)])
def test_kv_keep_beyond_32_bit_offsets(dtype, d):
    """Rows move between blocks at byte offsets past 2^32 (and element offsets
    past 2^31), and nothing else changes in either tensor."""
    bs, n_kv = 64, 8
    g = _gen(47)
    row = 72 if dtype == "mxfp4" else 2 * d
    blocks = 2 ** 32 // (bs * n_kv * row) * 2 + 40
    bt = [[blocks - 1, blocks - 3, 7], [blocks - 9, 5, blocks - 2],
          [3, blocks - 20, 1]]
    some = _cache(g, 9, n_kv, bs, dtype, d)
    kv = []
    for t in (some.k, some.v):
        x = torch.zeros((blocks, *t.shape[1:]), dtype=t.dtype, device="cuda")
        for i, b in enumerate(sum(bt, [])):
            x[b] = t[i]
        kv.append(x)
    c = K.PagedCache(*kv, bs, n_kv, d, dtype)
    start, path = [60, 20, 0], [[1, 6, 70], [0, 90, 120], [64, 65, 127]]
    want = [x.clone() for x in kv]
    for w, x in zip(want, kv):
        for b in range(3):
            for j, i in enumerate(path[b]):
                p, t = start[b] + i, start[b] + j
                w[bt[b][t // bs], :, t % bs] = x[bt[b][p // bs], :, p % bs]
    K.kv_keep([c], _i32(bt), _i32(start), _i32(path), _i32([3, 3, 3]))
    for x, w, t in zip(kv, want, (some.k, some.v)):
        assert torch.equal(x, w)
        assert not torch.equal(x[blocks - 1], t[0])
    assert K.device_error() == 0


def test_kv_keep_long_paths():
    g = _gen(3)
    n = K.TREE_NODES
    bt, blocks = _table(g, [2 * n], 32)
    c = _cache(g, blocks, 2, 32, "bf16", 128)
    pos = torch.arange(2 * n, device="cuda")
    rows = c.k[bt[0].long()[pos // 32], :, pos % 32]
    path = [0] + list(range(2, n + 1))
    K.kv_keep([c], bt, _i32([5]), _i32([path]), _i32([n]))
    got = c.k[bt[0].long()[pos // 32], :, pos % 32]
    want = rows.clone()
    want[5:5 + n] = rows[torch.tensor(path, device="cuda") + 5]
    assert torch.equal(got, want)
    assert K.device_error() == 0


def test_kv_keep_bad_values_leave_the_sequence():
    g = _gen(4)
    bt, blocks = _table(g, [64, 64, 64], 16)
    good = [0, 2, 5]
    for path, keep, start, code in (
            ([0, 2, 2], 3, 10, K.DEVERR_INDEX),
            ([0, 5, 3], 3, 10, K.DEVERR_INDEX),
            ([-1, 2, 3], 3, 10, K.DEVERR_INDEX),
            (good, 4, 10, K.DEVERR_LEN),
            (good, -1, 10, K.DEVERR_LEN),
            (good, 3, 60, K.DEVERR_POS),
            (good, 3, -1, K.DEVERR_POS),
            (good, 3, 2 ** 31 - 1, K.DEVERR_POS)):
        c = _cache(g, blocks, 2, 16, "bf16", 64)
        want = dataclasses.replace(c, k=c.k.clone(), v=c.v.clone())
        K.kv_keep([want], bt, _i32([3, 0, 7]), _i32([good] * 3),
                  _i32([3, 0, 3]))
        assert K.device_error() == 0
        K.kv_keep([c], bt, _i32([3, start, 7]), _i32([good, path, good]),
                  _i32([3, keep, 3]))
        assert K.device_error() == code
        assert torch.equal(c.k, want.k) and torch.equal(c.v, want.v)
    t = bt.clone()
    t[1, 0] = -1
    c = _cache(g, blocks, 2, 16, "bf16", 64)
    before = c.k.clone()
    K.kv_keep([c], t, _i32([3, 3, 7]), _i32([good] * 3), _i32([0, 3, 0]))
    assert K.device_error() == K.DEVERR_BLOCK and torch.equal(c.k, before)


# ---------------------------------------------------------------------------
# a step and the next
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "fp8", "mxfp4"])
def test_a_tree_step_leaves_the_cache_of_the_accepted_tokens(dtype):
    """Plan, write, attend and keep: the cache then equals one into which the
    accepted tokens were written one after the other, an accepted node's
    output is that of the same token as a chain, and the next tree attends to
    the kept rows."""
    d, n_h, n_kv, bs = 128, 16, 2, 16
    past, n, bound = [37, 90], [12, 9], 12
    parents = [-1, 0, 0, 1, 2, 2, 4, 5, 5, 7, 8, 9,
               -1, 0, 1, 1, 2, 3, 5, 6, 6]
    path, keep = [[0, 2, 5, 8, 10], [0, 1, 3, 5, 6]], [5, 4]
    g = _gen(43)
    bt, blocks = _table(g, [p + 2 * bound for p in past], bs)
    c = _cache(g, blocks, n_kv, bs, dtype, d)
    flat = dataclasses.replace(c, k=c.k.clone(), v=c.v.clone())
    plan = K.rope_plan(d)
    start, rs = _i32(past), _starts(n)
    k, v = _randn(g, sum(n), n_kv, d), _randn(g, sum(n), n_kv, d)
    q = _randn(g, sum(n), n_h, d)
    masks, pos = K.tree_plan(_i32(parents), start, rs, bound)
    qr = K.kv_write(c, bt, start, rs, k, v, rope=plan, positions=pos, q=q)
    lens = [a + b for a, b in zip(past, n)]
    out, lse = K.gqa_tree(c, bt, _i32(lens), max(lens), qr, rs, bound, masks)
    K.kv_keep([c], bt, start, _i32(path), _i32(keep))
    # the accepted tokens as a chain
    rows = [path[0][j] for j in range(5)] + [12 + path[1][j]
                                             for j in range(4)]
    sel = torch.tensor(rows, device="cuda")
    crs = _starts(keep)
    cpos = _i32([past[b] + j for b in range(2) for j in range(keep[b])])
    assert torch.equal(pos[sel], cpos)
    qc = K.kv_write(flat, bt, start, crs, k[sel].contiguous(),
                    v[sel].contiguous(), rope=plan, positions=cpos,
                    q=q[sel].contiguous())
    zero = _i32([0, 0])
    new = [a + b for a, b in zip(past, keep)]
    for x, y in zip(K.kv_read(c, bt, zero, _starts(new), sum(new)),
                    K.kv_read(flat, bt, zero, _starts(new), sum(new))):
        assert torch.equal(x, y)
    chain, _ = K.tree_plan(_i32([-1, 0, 1, 2, 3, -1, 0, 1, 2]), start, crs, 5)
    oc, lc = K.gqa_tree(flat, bt, _i32(new), max(new), qc, crs, 5, chain)
    ref = _reference(flat, bt, new, qc, keep,
                     _tree_sees(keep, past, chain, 1))
    _check((oc, lc), ref)
    _check((out[sel], lse[sel]), ref)
    # the next step's tree over the kept rows
    n2 = [3, 3]
    m2, p2 = K.tree_plan(_i32([-1, 0, 0] * 2), _i32(new), _starts(n2), 3)
    last = [a + 3 for a in new]
    k2, v2 = _randn(g, 6, n_kv, d), _randn(g, 6, n_kv, d)
    q2 = _randn(g, 6, n_h, d)
    got = []
    for cache in (c, flat):
        qw = K.kv_write(cache, bt, _i32(new), _starts(n2), k2, v2, rope=plan,
                        positions=p2, q=q2)
        got.append(K.gqa_tree(cache, bt, _i32(last), max(last), qw,
                              _starts(n2), 3, m2))
    assert torch.equal(got[0][0], got[1][0])
    assert torch.equal(got[0][1], got[1][1])
    assert K.device_error() == 0
