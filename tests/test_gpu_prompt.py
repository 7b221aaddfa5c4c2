"""The prompt path on the GPU (include/kvd_prompt.h): rotary positions,
ragged writes and reads, and attention over MXFP4 caches, against fp64
formulas. Tolerances are sums of the roundings each result goes through."""
import math

import numpy as np
import pytest
import torch

import kv_cache_decode_gqa_gb300 as K
import oracle

pytestmark = pytest.mark.gpu
D = 128
BF = torch.bfloat16
HALF_BF16 = torch.finfo(BF).eps / 2


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(BF)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _starts(n):
    return _i32([0] + list(np.cumsum(n)))


@pytest.fixture(autouse=True)
def _no_device_error():
    K.device_error()
    yield
    torch.cuda.synchronize()


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
def _rope_ref(x, freqs, axes, pos, pairing, d_rot, inverse):
    """fp64 rotation (angles reduced in fp64: positions times frequencies
    below 2^53 of a 2^-30 radian)."""
    x = x.double().cpu()
    half = d_rot // 2
    i = torch.arange(half)
    a, b = (i, i + half) if pairing == "half" else (2 * i, 2 * i + 1)
    f = torch.tensor(freqs, dtype=torch.float64)
    ang = pos.cpu().double()[torch.tensor(axes)].t() * f
    if inverse:
        ang = -ang
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    out = x.clone()
    out[..., a] = x[..., a] * c - x[..., b] * s
    out[..., b] = x[..., b] * c + x[..., a] * s
    mag = torch.zeros_like(x)
    mag[..., a] = mag[..., b] = x[..., a].abs() + x[..., b].abs()
    return out, mag


ROPE_CASES = [
    # rows, n_h, n_kv, d, d_rot, sections, interleave, pairing, far
    (1, 1, 1, 128, 128, None, False, "half", 10),
    (5, 8, 2, 128, 128, [16, 24, 24], False, "half", 4000),
    (37, 64, 8, 128, 128, [16, 24, 24], True, "half", 1000000),
    (700, 6, 3, 64, 32, [8, 4, 4], False, "half", 100000),
    (9, 3, 3, 128, 64, [32], False, "adjacent", 5000),
    (2500, 4, 1, 64, 64, [10, 11, 11], True, "adjacent", 3000),
    (13, 5, 1, 22, 20, [3, 7], False, "half", 999),      # no 16-byte pieces
    (13, 5, 1, 22, 20, [3, 7], True, "adjacent", 999),
    (3, 2, 2, 2, 2, None, False, "half", 7),
    (4, 3, 1, 1024, 1024, [128, 128, 128, 128], True, "half", 50),
    (1, 200, 1, 128, 128, None, False, "half", 31),
]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("case", ROPE_CASES)
def test_rope(case, inverse):
    rows, n_h, n_kv, d, d_rot, sections, inter, pairing, far = case
    g = _gen(rows)
    plan = K.rope_plan(d_rot, sections=sections, interleave=inter,
                       pairing=pairing)
    axes = K.rope_axes(d_rot, sections or [d_rot // 2], inter)
    pos = torch.randint(-far, far, (plan.n_axes, rows), generator=g,
                        device="cuda").to(torch.int32)
    q, k = _randn(g, rows, n_h, d), _randn(g, rows, n_kv, d)
    qo, ko = K.rope(plan, pos, q, k, inverse=inverse)
    freqs = [10000.0 ** (-2.0 * i / d_rot) for i in range(d_rot // 2)]
    for x, y in ((q, qo), (k, ko)):
        ref, mag = _rope_ref(x, freqs, axes, pos, pairing, d_rot, inverse)
        # bf16 rounding; cosines off by < 2^-20 (angle 2^-24 of a half turn,
        # 2 ulp of sincospi) and three fp32 operations
        tol = HALF_BF16 * ref.abs() + 2.0 ** -19 * mag
        assert bool(((y.cpu().double() - ref).abs() <= tol).all())
    assert K.device_error() == 0


def test_rope_strided_in_place_and_untouched_neighbours():
    """q and k inside a fused projection, rotated where they lie; the values
    between them stay."""
    g = _gen(3)
    rows, h, hk, d = 45, 8, 2, 128
    qkv = _randn(g, rows, h + 2 * hk, d)
    plan = K.rope_plan(96, sections=[16, 16, 16])
    pos = torch.randint(0, 500, (3, rows), generator=g,
                        device="cuda").to(torch.int32)
    want_q, want_k = K.rope(plan, pos, qkv[:, :h].contiguous(),
                            qkv[:, h:h + hk].contiguous())
    v = qkv[:, h + hk:].clone()
    q, k = qkv[:, :h], qkv[:, h:h + hk]
    K.rope(plan, pos, q, k, q_out=q, k_out=k)
    assert torch.equal(q, want_q) and torch.equal(k, want_k)
    assert torch.equal(qkv[:, h + hk:], v)
    # heads outermost, and an odd offset that no 16-byte access fits
    flat = torch.zeros(3 + rows * h * d, dtype=BF, device="cuda")
    odd = flat[3:].view(h, rows, d).transpose(0, 1)
    odd.copy_(want_q)
    back, _ = K.rope(plan, pos, odd, inverse=True)
    again, _ = K.rope(plan, pos, want_q, inverse=True)
    assert torch.equal(back, again)


def test_rope_far_positions_are_exact():
    """At 2^31 - 1 the angle still has 2^-32 of a turn: the rotation by p is
    the composition of those by 2^30 and p - 2^30 in exact arithmetic."""
    plan = K.rope_plan(64, freqs=[2 * math.pi * (i + 1) / 64.0
                                  for i in range(32)])
    # frequencies of whole 64ths of a turn: angles repeat every 64 positions
    p = [2 ** 31 - 1, 2 ** 30 + 17, -2 ** 31, 64 * 12345 + 5]
    near = [x % 64 for x in p]
    x = _randn(_gen(9), 4, 2, 64)
    far, _ = K.rope(plan, _i32([p]), x)
    ref, _ = K.rope(plan, _i32([near]), x)
    # the frequency's own rounding, 2^-53 relative times 2^31, is 2^-22 turn
    d = (far.double() - ref.double()).abs()
    assert float(d.max()) <= 2 * HALF_BF16 * float(x.double().abs().max()) * 2


def test_rope_axis_out_of_range_is_flagged():
    plan = K.rope_plan(64, sections=[16, 16])
    plan.axis[3] = 2
    x = _randn(_gen(1), 3, 1, 64)
    K.rope(plan, _i32([[1, 2, 3], [4, 5, 6]]), x)
    assert K.device_error() == K.DEVERR_INDEX


# ---------------------------------------------------------------------------
# caches
# ---------------------------------------------------------------------------
def _cache(g, blocks, n_kv, bs, dtype, d=D, fill=True):
    shape = (blocks, n_kv, bs, d)
    out = []
    for _ in range(2):
        x = torch.randn(shape, generator=g, device="cuda").to(BF)
        if not fill:
            x.zero_()
        if dtype == "bf16":
            out.append(x)
        elif dtype == "fp8":
            out.append(x.float().mul(20).to(torch.float8_e4m3fn).view(
                torch.uint8))
        else:
            bits = x.view(torch.int16).cpu().numpy().view(np.uint16)
            out.append(torch.from_numpy(oracle.mxfp4_encode_rows(bits)).cuda())
    kw = {}
    if dtype == "fp8":
        s = 0.02 + 0.05 * torch.rand(2, n_kv, generator=g, device="cuda")
        kw = dict(k_scale=s[0].contiguous(), v_scale=s[1].contiguous(),
                  k_inv_scale=(1 / s[0]).contiguous(),
                  v_inv_scale=(1 / s[1]).contiguous())
    return K.PagedCache(out[0], out[1], bs, n_kv, d, dtype, **kw)


def _clone(c):
    import dataclasses
    return dataclasses.replace(c, k=c.k.clone(),
                               v=None if c.v is None else c.v.clone())


def _table(g, lens, bs, width=None):
    """A shuffled block table for sequences of these lengths, and the size
    of its pool (two blocks of it unused)."""
    per = [max((n + bs - 1) // bs, 1) for n in lens]
    total = sum(per) + 2
    perm = torch.randperm(total, generator=g, device="cuda").tolist()
    width = width or max(per)
    rows, at = [], 0
    for n in per:
        rows.append(perm[at:at + n] + [0] * (width - n))
        at += n
    return _i32(rows), total


def _append_one_by_one(c, bt, start, counts, k, v):
    """kv_append of the same rows, a token of every sequence at a time."""
    first = np.cumsum([0] + list(counts))
    for i in range(max(counts)):
        for b, n in enumerate(counts):
            if i < n:
                r = int(first[b]) + i
                K.kv_append(c, bt[b:b + 1].contiguous(), _i32([start[b] + i]),
                            k[r:r + 1].contiguous(), v[r:r + 1].contiguous())


WRITE_CASES = [
    # counts, starts, n_kv, block size
    ([1], [0], 1, 64),
    ([3, 0, 5, 1], [0, 7, 62, 13], 2, 16),
    ([70, 1], [5, 0], 8, 64),
    ([0, 0, 2], [1, 2, 3], 5, 2),
    ([19], [1], 33, 32),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "mxfp4"])
@pytest.mark.parametrize("case", WRITE_CASES)
def test_write_equals_append_and_reads_back(case, dtype):
    counts, starts, n_kv, bs = case
    g = _gen(sum(counts))
    last = [a + b for a, b in zip(counts, starts)]
    bt, blocks = _table(g, last, bs)
    a = _cache(g, blocks, n_kv, bs, dtype)
    b = _clone(a)
    rows, pad = sum(counts), 4
    k, v = _randn(g, rows + pad, n_kv, D), _randn(g, rows + pad, n_kv, D)
    K.kv_write(a, bt, _i32(starts), _starts(counts), k, v)
    _append_one_by_one(b, bt, starts, counts, k, v)
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
    # read back: the fp64 values of the codes, rounded once
    ko, vo = (torch.full((rows + pad, n_kv, D), 7.0, dtype=BF, device="cuda")
              for _ in range(2))
    K.kv_read(a, bt, _i32(starts), _starts(counts), rows + pad, ko, vo)
    for t, o, sc in ((a.k, ko, a.k_scale), (a.v, vo, a.v_scale)):
        r = 0
        for s, n in enumerate(counts):
            for i in range(n):
                p = starts[s] + i
                row = t[int(bt[s, p // bs]), :, p % bs].cpu()
                if dtype == "bf16":
                    want = row
                elif dtype == "fp8":
                    want = (row.view(torch.float8_e4m3fn).float() *
                            sc.cpu()[:, None]).to(BF)
                else:
                    want = torch.from_numpy(oracle.mxfp4_rows_to_f64(
                        row.numpy(), D)).to(BF)
                assert torch.equal(o[r].cpu(), want)
                r += 1
        assert bool((o[rows:] == 7).all())        # padding left as it was
    assert K.device_error() == 0


def test_write_mxfp4_every_bf16_pattern():
    """Every bf16 value (infinities, NaN, subnormals, both zeros) beside
    group maxima of every exponent: the bytes of kv_append."""
    g = _gen(5)
    bits = torch.arange(65536, device="cuda").to(torch.int32)
    top = torch.randint(0, 65536, (65536,), generator=g, device="cuda")
    x = torch.stack([bits, top.to(torch.int32)], 1)
    x = x.repeat_interleave(4, 1).reshape(-1)            # 8 per value
    x = torch.cat([x, torch.randint(0, 65536, (65536 * 8,), generator=g,
                                    device="cuda").to(torch.int32)])
    # ties: multiples of scale midpoints
    m = torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6.0] * 2,
                     device="cuda")
    sc = 2.0 ** torch.randint(-8, 6, (4096, 1), generator=g, device="cuda")
    sc = sc * (1 + torch.randint(0, 8, (4096, 1), generator=g,
                                 device="cuda") / 8)
    sign = torch.where(torch.rand(4096, 16, generator=g, device="cuda") < .5,
                       -1.0, 1.0)
    ties = (m * sc * sign).to(BF).view(torch.int16).to(torch.int32).reshape(-1)
    x = torch.cat([x, ties]).to(torch.int16).view(BF).reshape(-1, 1, D)
    n = x.shape[0]
    bs = 64
    bt = torch.arange((n + bs - 1) // bs, device="cuda",
                      dtype=torch.int32)[None].contiguous()
    a = K.PagedCache(torch.zeros((bt.shape[1], 1, bs, 72), dtype=torch.uint8,
                                 device="cuda"), None, bs, 1, D, "mxfp4")
    b = _clone(a)
    K.kv_write(a, bt, _i32([0]), _i32([0, n]), x)
    seq = bt.expand(n, -1).contiguous()
    for r in range(0, n, 4096):
        m = min(4096, n - r)
        K.kv_append(b, seq[:m], torch.arange(r, r + m, device="cuda",
                                             dtype=torch.int32),
                    x[r:r + m].contiguous())
    assert torch.equal(a.k, b.k)


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "mxfp4"])
@pytest.mark.parametrize("counts,n_kv,n_h,d_rot,pairing", [
    ([1, 1, 1], 8, 64, 128, "half"),
    ([33, 0, 4], 2, 14, 128, "adjacent"),
    ([300], 4, 4, 64, "half"),
    ([6], 40, 40, 36, "half"),           # pairs without 16-byte pieces
])
def test_write_with_rotation_equals_rope_then_write(dtype, counts, n_kv, n_h,
                                                    d_rot, pairing):
    g = _gen(n_h)
    bs = 32
    starts = [11 * i for i in range(len(counts))]
    bt, blocks = _table(g, [a + b for a, b in zip(counts, starts)], bs)
    a = _cache(g, blocks, n_kv, bs, dtype)
    b = _clone(a)
    rows = sum(counts) + 3
    qkv = _randn(g, rows, n_h + 2 * n_kv, D)
    q, k, v = qkv[:, :n_h], qkv[:, n_h:n_h + n_kv], qkv[:, n_h + n_kv:]
    sections = [d_rot // 2 - 2 * (d_rot // 6), d_rot // 6, d_rot // 6]
    plan = K.rope_plan(d_rot, sections=sections, pairing=pairing)
    pos = torch.randint(0, 9000, (3, rows), generator=g,
                        device="cuda").to(torch.int32)
    wq, wk = K.rope(plan, pos, q, k)
    K.kv_write(b, bt, _i32(starts), _starts(counts), wk, v)
    keep = q[-3:].clone()
    out = K.kv_write(a, bt, _i32(starts), _starts(counts), k, v, rope=plan,
                     positions=pos, q=q, q_out=q)
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
    assert torch.equal(out[:-3], wq[:-3]) and torch.equal(out[-3:], keep)
    assert K.device_error() == 0


def test_write_and_read_flag_bad_slots():
    g = _gen(2)
    bt, blocks = _table(g, [40, 40], 16)
    c = _cache(g, blocks, 2, 16, "mxfp4")
    before = c.k.clone()
    k = _randn(g, 4, 2, D)
    K.kv_write(c, bt, _i32([-1, 47]), _i32([0, 1, 4]), k, k)
    # rows 0 (position -1) and 2, 3 (positions 48, 49 of 48) are skipped
    assert K.device_error() == K.DEVERR_POS
    assert not torch.equal(c.k, before)
    changed = (c.k != before).any(-1).any(1).nonzero().tolist()
    assert changed == [[int(bt[1, 2]), 15]]
    bad = bt.clone()
    bad[0, 0], bad[1, 0] = -1, blocks
    ko, _ = K.kv_read(c, bad, _i32([0, 0]), _i32([0, 2, 4]), 4,
                      k_out=torch.full((4, 2, D), 3.0, dtype=BF,
                                       device="cuda"))
    assert K.device_error() == K.DEVERR_BLOCK
    assert bool((ko == 3).all())


def test_read_into_strided_outputs():
    """K into [n_kv][rows][d], V into a slice of a wider tensor."""
    g = _gen(8)
    bt, blocks = _table(g, [100, 7], 64)
    c = _cache(g, blocks, 4, 64, "mxfp4")
    args = (c, bt, _i32([3, 0]), _i32([0, 97, 104]), 104)
    k, v = K.kv_read(*args)
    kt = torch.zeros((4, 104, D), dtype=BF, device="cuda")
    wide = torch.zeros((104, 9, D), dtype=BF, device="cuda")
    K.kv_read(*args, k_out=kt.transpose(0, 1), v_out=wide[:, 2:6])
    assert torch.equal(kt.transpose(0, 1), k)
    assert torch.equal(wide[:, 2:6], v)
    assert not wide[:, :2].any() and not wide[:, 6:].any()


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def _attend_ref(c, bt, lens, counts, q, window=0, starts=None, scale=None):
    """(out, lse, tolerance of out, tolerance of lse) in fp64, by rows."""
    bs, n_kv = c.block_size, c.n_kv
    n_h = q.shape[1]
    grp = n_h // n_kv
    scale = scale or D ** -0.5
    q = q.double().cpu()
    outs, lses, tols, ltols = [], [], [], []
    r0 = 0
    for b, (T, n) in enumerate(zip(lens, counts)):
        if n == 0:
            continue
        pos = torch.arange(T)
        blk = bt[b].cpu().long()[pos // bs]
        kk, vv = (torch.from_numpy(oracle.mxfp4_rows_to_f64(
            t.cpu()[blk, :, pos % bs].numpy(), D)).reshape(T, n_kv, D)
            for t in (c.k, c.v))
        at = T - n + torch.arange(n)
        s0 = starts[b] if starts is not None else 0
        seen = (pos <= at[:, None]) & (pos >= s0)
        if window:
            seen &= pos > at[:, None] - window
        qq = q[r0:r0 + n].reshape(n, n_kv, grp, D)
        x = torch.einsum("ncgd,tcd->ncgt", qq, kk) * scale
        size = torch.einsum("ncgd,tcd->ncgt", qq.abs(), kk.abs()) * scale
        x = x.masked_fill(~seen[:, None, None], -math.inf)
        m = x.amax(-1, keepdim=True) if T else x.new_full((n, n_kv, grp, 1),
                                                         -math.inf)
        p = torch.exp(x - m.clamp(min=-1e300))
        l = p.sum(-1, keepdim=True)
        w = torch.where(l > 0, p / l, 0)
        o = torch.einsum("ncgt,tcd->ncgd", w, vv)
        av = torch.einsum("ncgt,tcd->ncgd", w, vv.abs())
        # a score is a sum of 128 fp32 products, then scaled in fp32 (q's
        # f16 form is off by 2^-40 of its largest element at most)
        es = (size.amax(-1, keepdim=True) if T else l) * 2.0 ** -15
        # bf16 rounding of the output; f16 rounding of p (2^-11, or 2^-25
        # below its normal range); p off by the scores' error and ex2's
        tol = (HALF_BF16 * o.abs() + (2.0 ** -11 + 2 * es + 2.0 ** -20) * av +
               2.0 ** -25 * (vv.abs().sum(0)[None, :, None] if T else 0))
        lse = (m + torch.log(l))[..., 0]
        ltol = es[..., 0] + 2.0 ** -20 * (1 + lse.abs().nan_to_num(
            0, posinf=0, neginf=0))
        outs.append(o.reshape(n, n_h, D))
        tols.append(tol.reshape(n, n_h, D))
        lses.append(lse.reshape(n, n_h))
        ltols.append(ltol.reshape(n, n_h))
        r0 += n
    return tuple(torch.cat(t) for t in (outs, lses, tols, ltols))


def _check(out, lse, ref):
    o, l, tol, ltol = ref
    n = o.shape[0]
    err = (out[:n].cpu().double() - o).abs()
    assert bool((err <= tol).all()), float((err - tol).max())
    g = lse[:n].cpu().double()
    dead = torch.isinf(l)
    assert torch.equal(torch.isneginf(g), dead)
    assert bool(((g - l).abs() <= ltol)[~dead].all())


EXTEND_CASES = [
    # counts, lengths after them, n_h, n_kv, block size, window
    # -- at most 16 (row, head) pairs a kv head
    ([1], [1], 8, 8, 64, 0),
    ([1, 1], [1, 300], 64, 8, 64, 0),
    ([1] * 5, [64, 65, 1, 0, 129], 16, 1, 16, 0),
    ([1] * 3, [700, 5000, 33], 56, 8, 64, 0),
    ([2, 0, 1], [900, 4, 1], 10, 2, 32, 0),
    ([4, 4], [1000, 4], 12, 4, 2, 0),
    ([1] * 40, [37 * i + 1 for i in range(40)], 32, 4, 64, 0),
    ([1] * 3, [500, 20, 4000], 64, 8, 64, 100),
    ([3, 2], [500, 2], 4, 1, 6, 7),
    ([2], [6000], 16, 2, 128, 0),
    ([1] * 2, [150, 100], 16, 2, 64, 1),
    # -- up to 32
    ([4] * 9, [4, 70, 1000, 333, 64, 65, 2000, 5, 128], 64, 8, 64, 0),
    ([3, 1, 2], [700, 1, 3000], 18, 2, 32, 0),
    ([4] * 40, [100 * i + 4 for i in range(40)], 64, 8, 64, 0),
    ([5, 4], [4, 900], 24, 4, 16, 50),
    ([2] * 50, [50 * i + 2 for i in range(50)], 32, 4, 64, 0),
    ([1] * 64, [60 * i + 1 for i in range(64)], 64, 8, 64, 0),
    ([1] * 64, [60 * i + 1 for i in range(64)], 32, 8, 16, 300),
    ([1] * 64, [97 * i + 1 for i in range(64)], 12, 1, 6, 0),
    # -- one tile of pairs
    ([5], [5], 8, 1, 64, 0),
    ([4, 4, 4], [1000, 4, 2333], 64, 8, 64, 0),
    ([17], [4100], 7, 1, 16, 0),
    ([16], [128], 8, 1, 64, 0),
    ([3], [129], 24, 2, 2, 0),
    ([9, 0, 1], [300, 50, 257], 96, 1, 6, 0),
    ([20], [700], 5, 1, 64, 33),
    # -- two tiles
    ([40], [40], 8, 1, 64, 0),
    ([33, 200, 1], [33, 777, 1], 16, 2, 32, 0),
    ([257], [257], 1, 1, 64, 0),
    ([300, 5], [2000, 5], 3, 1, 64, 0),
    ([129], [3000], 128, 1, 64, 0),
    ([150], [1500], 10, 2, 128, 200),
    ([64, 64], [64, 1000], 12, 2, 10, 1),
    ([6], [4], 64, 1, 16, 0),            # two rows before position 0
    ([40], [38], 8, 1, 16, 5),
]


@pytest.mark.parametrize("case", EXTEND_CASES)
def test_extend(case):
    counts, lens, n_h, n_kv, bs, window = case
    g = _gen(len(counts) * 1000 + n_h)
    bt, blocks = _table(g, lens, bs)
    c = _cache(g, blocks, n_kv, bs, "mxfp4")
    rows, pad = sum(counts), 3
    q = _randn(g, rows + pad, n_h, D)
    out = torch.full((rows + pad, n_h, D), 9.0, dtype=BF, device="cuda")
    lse = torch.full((rows + pad, n_h), 9.0, device="cuda")
    K.gqa_extend(c, bt, _i32(lens), max(lens), q, _starts(counts),
                 max(counts), out=out, lse=lse, window=window)
    _check(out, lse, _attend_ref(c, bt, lens, counts, q, window))
    assert bool((out[rows:] == 9).all()) and bool((lse[rows:] == 9).all())
    assert K.device_error() == 0
