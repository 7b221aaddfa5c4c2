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


@pytest.mark.parametrize("counts,lens,window,starts", [
    ([1, 1, 1], [200, 90, 10], 0, [50, 89, 40]),       # the last sees nothing
    ([4, 4], [300, 64], 20, [290, 62]),
    ([60, 3], [900, 70], 0, [500, 69]),
    ([90, 80], [700, 600], 128, [640, 599]),
])
def test_extend_from_replay_starts(counts, lens, window, starts):
    g = _gen(7)
    bt, blocks = _table(g, lens, 64)
    c = _cache(g, blocks, 2, 64, "mxfp4")
    q = _randn(g, sum(counts), 16, D)
    out, lse = K.gqa_extend(c, bt, _i32(lens), max(lens), q, _starts(counts),
                            max(counts), window=window,
                            window_start=_i32(starts))
    _check(out, lse, _attend_ref(c, bt, lens, counts, q, window, starts))
    assert K.device_error() == 0


@pytest.mark.parametrize("counts", [[1, 2], [20, 10], [70, 40]])
def test_extend_strided_queries_scales_and_no_lse(counts):
    """Queries inside a fused projection, a scale of the caller's, and
    queries of very different magnitudes: 2^-100 and 2^100 side by side."""
    g = _gen(31)
    lens = [n + 130 for n in counts]
    bt, blocks = _table(g, lens, 64)
    c = _cache(g, blocks, 2, 64, "mxfp4")
    qkv = _randn(g, sum(counts), 12, D)
    q = qkv[:, 2:10]
    big = torch.tensor([2.0 ** -100, 2.0 ** -130, 1, 2.0 ** -8] * 2,
                       device="cuda")
    q.copy_((q.float() * big[:, None]).to(BF))
    args = (c, bt, _i32(lens), max(lens), q, _starts(counts), max(counts))
    out, lse = K.gqa_extend(*args, scale=0.25)
    _check(out, lse, _attend_ref(c, bt, lens, counts, q, scale=0.25))
    out2, none = K.gqa_extend(*args, scale=0.25, want_lse=False)
    assert none is None and torch.equal(out, out2)


@pytest.mark.parametrize("n_h", [64, 128])
def test_extend_shares_of_very_unequal_sequences(n_h):
    """One long sequence among empty and short ones: some CTAs' shares hold
    several units, some none of their chunks."""
    g = _gen(43)
    lens = [0, 1, 9000, 64, 63, 0, 130, 2, 65] + [1] * 15
    counts = [1] * len(lens)
    bt, blocks = _table(g, lens, 64)
    c = _cache(g, blocks, 8, 64, "mxfp4")
    q = _randn(g, len(lens), n_h, D)
    out, lse = K.gqa_extend(c, bt, _i32(lens), 9000, q)
    _check(out, lse, _attend_ref(c, bt, lens, counts, q))
    assert K.device_error() == 0


@pytest.mark.parametrize("counts,n_h", [([3], 8), ([30], 8), ([120], 8)])
def test_extend_nan_and_infinite_queries_stay_in_their_rows(counts, n_h):
    g = _gen(41)
    lens = [counts[0] + 300]
    bt, blocks = _table(g, lens, 64)
    c = _cache(g, blocks, 2, 64, "mxfp4")
    q = _randn(g, counts[0], n_h, D)
    args = (c, bt, _i32(lens), lens[0])
    want, wl = K.gqa_extend(*args, q, _starts(counts), counts[0])
    q[1, 2, 5] = float("nan")
    q[2, 0, 0] = float("inf")
    out, lse = K.gqa_extend(*args, q, _starts(counts), counts[0])
    bad = torch.zeros((counts[0], n_h), dtype=torch.bool, device="cuda")
    bad[1, 2] = bad[2, 0] = True
    assert torch.equal(out[~bad], want[~bad])
    assert torch.equal(lse[~bad], wl[~bad])
    assert bool(torch.isnan(out[1, 2]).all()) and bool(torch.isnan(lse[1, 2]))


@pytest.mark.parametrize("max_rows", [1, 4, 40])
def test_extend_flags_bad_lists_lengths_and_blocks(max_rows):
    g = _gen(51)
    lens = [200, 120, 300]
    bt, blocks = _table(g, lens, 64)
    c = _cache(g, blocks, 1, 64, "mxfp4")
    n = max_rows
    q = _randn(g, 3 * n, 8, D)
    good = [0, n, 2 * n, 3 * n]

    def run(rs=good, lens=lens, table=bt, top=300):
        out = torch.full((3 * n, 8, D), 9.0, dtype=BF, device="cuda")
        K.gqa_extend(c, table, _i32(lens), top, q, _i32(rs), n, out=out)
        return out
    want = run()
    assert K.device_error() == 0
    # a list that descends, passes the rows or jumps too far: that sequence
    # is skipped, the others are right
    for bad in ([0, n, 0, n], [0, n, 2 * n, 3 * n + 1], [0, n, n, 3 * n + 9]):
        out = run(bad)
        assert K.device_error() == K.DEVERR_LEN
        assert torch.equal(out[:n], want[:n])
    # a length above the bound is clamped to it
    out = run(lens=[200, 500, 300])
    assert K.device_error() == K.DEVERR_LEN
    assert torch.equal(out[:n], want[:n])
    bad = bt.clone()
    bad[1, 0] = blocks + 5
    out = run(table=bad)
    assert K.device_error() == K.DEVERR_BLOCK
    assert torch.equal(out[:n], want[:n]) and torch.equal(out[2 * n:],
                                                          want[2 * n:])


def test_extend_single_tokens_match_gqa_decode():
    """Query groups that gqa_decode takes: the same values within the two
    calls' roundings."""
    g = _gen(61)
    lens = [1, 64, 1000, 4097]
    bt, blocks = _table(g, lens, 64)
    c = _cache(g, blocks, 8, 64, "mxfp4")
    q = _randn(g, 4, 32, D)
    a, la = K.gqa_extend(c, bt, _i32(lens), 4097, q)
    b, lb = K.gqa_decode(c, bt, _i32(lens), 4097, q)
    assert float((la - lb).abs().max()) <= 1e-4
    ref = _attend_ref(c, bt, lens, [1] * 4, q)
    _check(a, la, ref)
    # gqa_decode's own probabilities are rounded more coarsely (2^-8)
    assert float((a.float() - b.float()).abs().max()) <= 0.02


def test_prompt_then_tokens_run_together():
    """A model's use: two prompts written with rotated keys and attended in
    two chunks, then single tokens; every step against the fp64 formula over
    everything written so far."""
    g = _gen(71)
    n_kv, n_h, bs = 2, 16, 16
    plan = K.rope_plan(D, sections=[16, 24, 24])
    total = [150, 40]
    bt, blocks = _table(g, [t + 8 for t in total], bs)
    c = _cache(g, blocks, n_kv, bs, "mxfp4", fill=False)
    past = [0, 0]
    for counts in ([100, 33], [50, 7], [1, 1], [1, 1], [3, 0]):
        rows = sum(counts)
        qkv = _randn(g, rows, n_h + 2 * n_kv, D)
        q, k, v = qkv[:, :n_h], qkv[:, n_h:n_h + n_kv], qkv[:, n_h + n_kv:]
        pos = torch.randint(0, 300, (3, rows), generator=g,
                            device="cuda").to(torch.int32)
        rs = _starts(counts)
        wq, wk = K.rope(plan, pos, q, k)
        qr = K.kv_write(c, bt, _i32(past), rs, k, v, rope=plan, positions=pos,
                        q=q)
        assert torch.equal(qr, wq)
        kb, vb = K.kv_read(c, bt, _i32(past), rs, rows)
        bits = wk.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
        want = oracle.mxfp4_rows_to_f64(oracle.mxfp4_encode_rows(bits), D)
        assert torch.equal(kb.cpu().double(), torch.from_numpy(want))
        past = [a + b for a, b in zip(past, counts)]
        out, lse = K.gqa_extend(c, bt, _i32(past), max(past), qr, rs,
                                max(counts))
        _check(out, lse, _attend_ref(c, bt, past, counts, qr))
    assert K.device_error() == 0


# ---------------------------------------------------------------------------
# graphs, streams, repetition
# ---------------------------------------------------------------------------
def _step(c, bt, past, lens, rs, max_rows, qkv, n_h, n_kv, plan, pos):
    q, k, v = qkv[:, :n_h], qkv[:, n_h:n_h + n_kv], qkv[:, n_h + n_kv:]
    qr = K.kv_write(c, bt, past, rs, k, v, rope=plan, positions=pos, q=q)
    out, lse = K.gqa_extend(c, bt, lens, bt.shape[1] * c.block_size, qr, rs,
                            max_rows)
    kb, vb = K.kv_read(c, bt, past, rs, qkv.shape[0])
    return qr, out, lse, kb, vb


@pytest.mark.parametrize("counts,n_kv", [([1, 1], 8), ([5, 6], 8),
                                         ([200, 90], 2)])
def test_captured_and_replayed(counts, n_kv):
    """Two graphs of the same step share no workspace; replays with other
    inputs, other lengths and interleaved with eager calls."""
    g = _gen(81)
    n_h = 8 * n_kv
    rows = sum(counts)
    bt, blocks = _table(g, [2000, 1200], 64)
    plan = K.rope_plan(D)
    rs = _starts(counts)
    state = []
    for i in range(2):
        c = _cache(g, blocks, n_kv, 64, "mxfp4")
        state.append(dict(
            c=c, past=_i32([1500, 700]), qkv=_randn(g, rows, n_h + 2 * n_kv,
                                                    D),
            pos=torch.randint(0, 999, (1, rows), generator=g,
                              device="cuda").to(torch.int32)))
    for s in state:
        s["lens"] = s["past"] + _i32(counts)

    def run(s):
        return _step(s["c"], bt, s["past"], s["lens"], rs, max(counts),
                     s["qkv"], n_h, n_kv, plan, s["pos"])
    for s in state:
        run(s)
    torch.cuda.synchronize()
    for s in state:
        s["graph"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(s["graph"]):
            s["out"] = run(s)
    for past in ([1500, 700], [3, 0], [1799, 64]):
        for s in state:
            s["past"].copy_(_i32(past))
            s["lens"].copy_(_i32([a + b for a, b in zip(past, counts)]))
            s["qkv"].copy_(_randn(g, *s["qkv"].shape))
        for s in state:
            s["graph"].replay()
        torch.cuda.synchronize()
        got = [[t.clone() for t in s["out"]] for s in state]
        for s, o in zip(state, got):
            for a, b in zip(o, run(s)):
                assert torch.equal(a, b)
    assert K.device_error() == 0


@pytest.mark.parametrize("counts,n_kv", [([1] * 8, 8), ([200, 90], 2)])
def test_on_another_stream_and_repeated(counts, n_kv):
    """A stream of the caller's, both ways of naming it, and the same bits
    from every repetition."""
    g = _gen(91)
    n_h = 8 * n_kv
    lens = [700 + 100 * i for i in range(len(counts))]
    bt, blocks = _table(g, lens, 64)
    c = _cache(g, blocks, n_kv, 64, "mxfp4")
    q = _randn(g, sum(counts), n_h, D)
    args = (c, bt, _i32(lens), max(lens), q, _starts(counts), max(counts))
    want, wl = K.gqa_extend(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        a, la = K.gqa_extend(*args, stream=side)
        with torch.cuda.stream(side):
            b, lb = K.gqa_extend(*args)
        side.synchronize()
        assert torch.equal(a, want) and torch.equal(b, want)
        assert torch.equal(la, wl) and torch.equal(lb, wl)


def test_workspace_of_the_caller():
    g = _gen(101)
    lens = [3000]
    bt, blocks = _table(g, lens, 64)
    c = _cache(g, blocks, 1, 64, "mxfp4")
    q = _randn(g, 40, 8, D)
    rs = _starts([40])
    n = K.extend_workspace_size(c, bt, _i32(lens), 3000, 40, 8, 40)
    assert n > 0
    args = (c, bt, _i32(lens), 3000, q, rs, 40)
    want, _ = K.gqa_extend(*args)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # NaN
    out, _ = K.gqa_extend(*args, workspace=ws)
    assert torch.equal(out, want)
    with pytest.raises(K.KvdError, match="workspace"):
        K.gqa_extend(*args, workspace=ws[:n - 256])
    # no launch of few CTAs or many changes the values beyond the merge's
    # rounding
    for ctas in (1, 7, 1000):
        K.set_tuning(decode_ctas=ctas)
        try:
            out, lse = K.gqa_extend(*args)
            one, l1 = K.gqa_extend(c, bt, _i32(lens), 3000, q[:1])
        finally:
            K.set_tuning()
        _check(out, lse, _attend_ref(c, bt, lens, [40], q))
        _check(one, l1, _attend_ref(c, bt, lens, [1], q[:1]))


def test_empty_calls():
    g = _gen(111)
    bt, blocks = _table(g, [10], 16)
    c = _cache(g, blocks, 2, 16, "mxfp4")
    none = _randn(g, 0, 2, D)
    rs = _i32([0, 0])
    K.kv_write(c, bt, _i32([0]), rs, none, none)
    k, v = K.kv_read(c, bt, _i32([0]), rs, 0)
    out, lse = K.gqa_extend(c, bt, _i32([10]), 10, _randn(g, 0, 4, D), rs, 0)
    plan = K.rope_plan(D)
    q, _ = K.rope(plan, _i32([[]]).reshape(1, 0), none)
    assert k.shape == v.shape == q.shape == (0, 2, D)
    assert out.shape == (0, 4, D) and lse.shape == (0, 4)
    # rows that no sequence owns: nothing is written, nothing attended
    rows = _randn(g, 3, 2, D)
    before = c.k.clone()
    K.kv_write(c, bt, _i32([0]), rs, rows, rows)
    o = torch.full((3, 4, D), 5.0, dtype=BF, device="cuda")
    K.gqa_extend(c, bt, _i32([10]), 10, _randn(g, 3, 4, D), rs, 3, out=o)
    assert torch.equal(c.k, before) and bool((o == 5).all())
    assert K.device_error() == 0


def test_tensors_of_two_devices_are_refused():
    g = _gen(121)
    bt, blocks = _table(g, [10], 16)
    c = _cache(g, blocks, 2, 16, "mxfp4")

    class Elsewhere(torch.Tensor):
        @property
        def device(self):
            return torch.device("cuda", 7)
    q = _randn(g, 1, 4, D).as_subclass(Elsewhere)
    with pytest.raises(ValueError, match="in one call"):
        K.gqa_extend(c, bt, _i32([10]), 10, q)


def test_offsets_past_32_bits():
    """Blocks and rows whose byte (and element) offsets pass 2^32: written,
    read back, attended by every kernel, rotated."""
    g = _gen(131)
    n_kv, bs = 8, 64
    blocks = 2 ** 32 // (n_kv * bs * 72) + 100
    cache = [torch.empty((blocks, n_kv, bs, 72), dtype=torch.uint8,
                         device="cuda") for _ in range(2)]
    c = K.PagedCache(*cache, bs, n_kv, D, "mxfp4")
    counts = [200, 150]
    bt = _i32([[blocks - 1 - i for i in range(4)],
               [1, blocks - 9, 0, blocks - 8]])
    k, v = (_randn(g, 350, n_kv, D) for _ in range(2))
    rs, start = _starts(counts), _i32([0, 0])
    K.kv_write(c, bt, start, rs, k, v)
    small = K.PagedCache(*(t[[blocks - 1 - i for i in range(4)] +
                             [1, blocks - 9, 0]].contiguous() for t in cache),
                         bs, n_kv, D, "mxfp4")
    st = _i32([[0, 1, 2, 3], [4, 5, 6, 0]])
    for a, b in zip(K.kv_read(c, bt, start, rs, 350),
                    K.kv_read(small, st, start, rs, 350)):
        assert torch.equal(a, b)
    for n in (1, 3, 20, 70):
        q = _randn(g, 2 * n, 64, D)
        args = (_i32(counts), 200, q, _starts([n, n]), n)
        a, la = K.gqa_extend(c, bt, *args)
        b, lb = K.gqa_extend(small, st, *args)
        assert torch.equal(a, b) and torch.equal(la, lb)
    assert K.device_error() == 0
    del c, cache
    far = torch.empty(2 ** 32 + 4096, dtype=BF, device="cuda")
    rows = far.as_strided((5, 2, D), (2 ** 30, 512, 1))
    x = _randn(g, 5, 2, D)
    rows.copy_(x)
    plan = K.rope_plan(D)
    pos = _i32([[1, 2, 3, 4, 5]])
    want, _ = K.rope(plan, pos, x)
    K.rope(plan, pos, rows, q_out=rows)
    assert torch.equal(rows, want)


# ---------------------------------------------------------------------------
# row lists that are none
# ---------------------------------------------------------------------------
# lists in units of n rows for four sequences, of 4 n rows in all, and the
# sequences that are attended: those before the first descent whose own
# entries fit
BAD_LISTS = [
    ([0, 1, 0, 0, 1], [0]),          # the last would take the first's rows
    ([0, 1, 2, 1, 2], [0, 1]),
    ([1, 0, 1, 2, 3], []),
    ([0, 1, 9, 3, 4], [0]),          # past the rows, then a descent
    ([-1, 1, 2, 3, 4], [1, 2, 3]),
    ([0, 1, 2, 3, 5], [0, 1, 2]),
    ([0, 2, 3, 3, 4], [1, 3]),       # two units where one is the bound
]


@pytest.mark.parametrize("units,good", BAD_LISTS)
@pytest.mark.parametrize("n,lens", [
    (1, [200, 90, 300, 70]), (2, [7000, 900, 5000, 64]),
    (4, [200, 90, 300, 70]), (5, [9000, 1000, 2500, 300]),
    (40, [9000, 1000, 2500, 300]), (70, [900, 80, 200, 300])])
def test_extend_follows_a_list_to_its_first_descent(units, good, n, lens):
    g = _gen(53)
    bt, blocks = _table(g, lens, 64)
    c = _cache(g, blocks, 1, 64, "mxfp4")
    q = _randn(g, 4 * n, 8, D)
    out = torch.full((4 * n, 8, D), 9.0, dtype=BF, device="cuda")
    lse = torch.full((4 * n, 8), 9.0, device="cuda")
    K.gqa_extend(c, bt, _i32(lens), max(lens), q, _i32([u * n for u in units]),
                 n, out=out, lse=lse)
    assert K.device_error() == K.DEVERR_LEN
    rest = torch.ones(4 * n, dtype=torch.bool, device="cuda")
    for b in good:
        r = slice(units[b] * n, units[b + 1] * n)
        if r.stop > r.start:
            _check(out[r], lse[r], _attend_ref(
                c, bt[b:b + 1], lens[b:b + 1], [r.stop - r.start], q[r]))
        rest[r] = False
    assert bool((out[rest] == 9).all()) and bool((lse[rest] == 9).all())


def test_extend_finds_the_rows_of_many_sequences():
    """A merge launch over more than 32 sequences, empty ones and padding
    among them."""
    g = _gen(57)
    counts = [0, 3] * 20 + [0] * 30 + [5, 0, 4]
    lens = [90 * i % 1700 + 5 for i in range(len(counts))]
    bt, blocks = _table(g, lens, 64)
    c = _cache(g, blocks, 1, 64, "mxfp4")
    rows = sum(counts)
    q = _randn(g, rows + 2, 8, D)
    out = torch.full((rows + 2, 8, D), 9.0, dtype=BF, device="cuda")
    _, lse = K.gqa_extend(c, bt, _i32(lens), max(lens), q, _starts(counts), 5,
                          out=out)
    _check(out, lse, _attend_ref(c, bt, lens, counts, q))
    assert bool((out[rows:] == 9).all())
    assert K.device_error() == 0


# the same for writes and reads, which do nothing where a list descends
WRITE_LISTS = [(u, [] if any(b < a for a, b in zip(u, u[1:])) else good)
               for u, good in BAD_LISTS[:6]] + [([0, 5, 5, 5, 5], []),
                                                ([-3, -1, 1, 2, 4], [2, 3])]


@pytest.mark.parametrize("units,good", WRITE_LISTS)
@pytest.mark.parametrize("dtype,n,rotate", [
    ("mxfp4", 1, False), ("bf16", 7, True), ("fp8", 33, False),
    ("mxfp4", 200, True)])
def test_write_and_read_flag_bad_lists(units, good, dtype, n, rotate):
    g = _gen(59)
    n_kv, bs, starts = 2, 16, [3, 0, 40, 16]
    bt, blocks = _table(g, [s + 9 * n for s in starts], bs)
    a = _cache(g, blocks, n_kv, bs, dtype)
    b = _clone(a)
    k, v = _randn(g, 4 * n, n_kv, D), _randn(g, 4 * n, n_kv, D)
    rs = _i32([u * n for u in units])
    rope, kw = K.rope_plan(D), {}
    if rotate:
        pos = torch.arange(4 * n, dtype=torch.int32, device="cuda")
        q = _randn(g, 4 * n, 4, D)
        turned, _ = K.rope(rope, pos, q)
        kw = dict(rope=rope, positions=pos)
        got = dict(kw, q=q, q_out=torch.full_like(q, 9.0))
    out = K.kv_write(a, bt, _i32(starts), rs, k, v,
                     **(got if rotate else {}))
    assert K.device_error() == K.DEVERR_LEN
    ko, vo = K.kv_read(a, bt, _i32(starts), rs, 4 * n,
                       *(torch.full_like(k, 9.0) for _ in range(2)))
    assert K.device_error() == K.DEVERR_LEN
    # each good sequence by itself
    rest = torch.ones(4 * n, dtype=torch.bool, device="cuda")
    for s in good:
        r = slice(units[s] * n, units[s + 1] * n)
        one = (b, bt[s:s + 1].contiguous(), _i32([starts[s]]),
               _starts([r.stop - r.start]))
        if rotate:
            kw["positions"] = pos[r].contiguous()
            assert torch.equal(out[r], turned[r])
        K.kv_write(*one, k[r], v[r], **kw)
        for x, y in zip(K.kv_read(*one, r.stop - r.start), (ko, vo)):
            assert torch.equal(x, y[r])
        rest[r] = False
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
    for x in (ko, vo) + ((out,) if rotate else ()):
        assert bool((x[rest] == 9).all())
    assert K.device_error() == 0


@pytest.mark.parametrize("batch", [257, 2048, 2049, 5000])
def test_write_and_read_of_many_sequences(batch):
    """Lists that every CTA checks as a whole and lists that it checks a share
    of: one token of most sequences, three or none of some."""
    g = _gen(batch)
    n_kv, bs = 1, 4
    counts = [3 if i % 7 == 2 else 0 if i % 11 == 5 else 1
              for i in range(batch)]
    rows = sum(counts)
    bt = torch.randperm(batch, generator=g, device="cuda").to(
        torch.int32)[:, None].contiguous()
    c = _cache(g, batch, n_kv, bs, "bf16")
    want = c.k.clone(), c.v.clone()
    start = torch.randint(0, 2, (batch,), generator=g, device="cuda")
    k, v = _randn(g, rows + 1, n_kv, D), _randn(g, rows + 1, n_kv, D)
    rs = _starts(counts)
    seq = torch.repeat_interleave(torch.arange(batch, device="cuda"),
                                  torch.tensor(counts, device="cuda"))
    at = start[seq] + torch.arange(rows, device="cuda") - rs.long()[seq]
    for t, x in zip(want, (k, v)):
        t[bt[seq, 0].long(), :, at] = x[:rows]
    args = (c, bt, start.to(torch.int32))
    K.kv_write(*args, rs, k, v)
    assert torch.equal(c.k, want[0]) and torch.equal(c.v, want[1])
    ko, vo = K.kv_read(*args, rs, rows)
    assert torch.equal(ko, k[:rows]) and torch.equal(vo, v[:rows])
    assert K.device_error() == 0
    # a descent or an end past the rows, anywhere, is flagged
    for i, x in ((batch - 1, 0), (batch // 2, rows), (batch, rows + 2),
                 (1, -1)):
        bad = rs.clone()
        bad[i] = x
        K.kv_write(*args, bad, k, v)
        assert K.device_error() & K.DEVERR_LEN
        ko = torch.full_like(k, 9.0)
        K.kv_read(*args, bad, rows + 1, k_out=ko)
        assert K.device_error() & K.DEVERR_LEN
        if batch <= 2048 and i != batch:
            assert bool((ko == 9).all())
            assert torch.equal(c.k, want[0]) and torch.equal(c.v, want[1])


# ---------------------------------------------------------------------------
# a flat tail behind one dominant key
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("rows,n_h", [(1, 8), (1, 16), (2, 8), (5, 8), (20, 8),
                                      (40, 8), (60, 12)])
def test_extend_keeps_a_flat_tail(rows, n_h):
    """Position 0 scores 18.7 above every other one (2^-27 of its weight each)
    and its value is 0, so the outputs are the tail alone: 4,095 positions of
    one value. With one CTA for all no part has a reference of its own.
    f16 rounds a probability below its normal range by 2^-25, and the largest
    is 2^7 or more, so the tail's error is 2^-32 a position, not 2^-25."""
    g = _gen(141)
    T = 4096
    bt, blocks = _table(g, [T], 64)
    c = _cache(g, blocks, 1, 64, "mxfp4")

    def row(x):
        bits = np.array([[x] * D], dtype=np.float32).view(np.uint32) >> 16
        return torch.from_numpy(oracle.mxfp4_encode_rows(
            bits.astype(np.uint16))).cuda()
    c.k[:], c.v[:] = row(0.0), row(1.0)
    c.k[int(bt[0, 0]), :, 0] = row(1.0)
    c.v[int(bt[0, 0]), :, 0] = row(0.0)
    q = torch.full((rows, n_h, D), 1.6, device="cuda").to(BF)
    K.set_tuning(decode_ctas=1)
    try:
        out, lse = K.gqa_extend(c, bt, _i32([T]), T, q, _starts([rows]), rows)
    finally:
        K.set_tuning()
    o, l, tol, ltol = _attend_ref(c, bt, [T], [rows], q)
    v = oracle.mxfp4_rows_to_f64(c.v[int(bt[0, 0]), 0, 1:2].cpu().numpy(), D)
    tol = tol - (2.0 ** -25 - 2.0 ** -32) * (T - 1) * float(v[0, 0])
    assert float(tol.max()) < 0.05 * float(o.min())
    _check(out, lse, (o, l, tol, ltol))
    assert K.device_error() == 0


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 8, 1])
@pytest.mark.parametrize("counts,lens,n_h", [
    ([6, 1], [2, 3], 2), ([20, 5], [10, 0], 8), ([60, 9], [50, 70], 8),
    ([300, 40], [30, 40], 4)])
def test_extend_windows_of_any_size_with_rows_before_position_0(counts, lens,
                                                                n_h, window):
    g = _gen(151)
    bt, blocks = _table(g, lens, 16)
    c = _cache(g, blocks, 1, 16, "mxfp4")
    q = _randn(g, sum(counts), n_h, D)
    out, lse = K.gqa_extend(c, bt, _i32(lens), max(lens), q, _starts(counts),
                            max(counts), window=window)
    _check(out, lse, _attend_ref(c, bt, lens, counts, q, window))
    assert K.device_error() == 0


@pytest.mark.parametrize("d,d_rot,n_kv", [(2056, 1024, 3), (32768, 1024, 2),
                                          (100344, 1024, 1), (4104, 64, 9)])
def test_write_rotates_wide_heads(d, d_rot, n_kv):
    """Heads that take one key head's shared memory past 40 and 48 KB, up to
    the limit."""
    g = _gen(161)
    rows, bs = 5, 4
    bt, blocks = _table(g, [rows], bs)
    a = _cache(g, blocks, n_kv, bs, "bf16", d=d)
    b = _clone(a)
    k, v = _randn(g, rows, n_kv, d), _randn(g, rows, n_kv, d)
    plan = K.rope_plan(d_rot)
    pos = torch.arange(7, 7 + rows, dtype=torch.int32, device="cuda")
    wk, _ = K.rope(plan, pos, k)
    K.kv_write(b, bt, _i32([0]), _starts([rows]), wk, v)
    K.kv_write(a, bt, _i32([0]), _starts([rows]), k, v, rope=plan,
               positions=pos)
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
    freqs = [10000.0 ** (-2.0 * i / d_rot) for i in range(d_rot // 2)]
    ref, mag = _rope_ref(k, freqs, [0] * (d_rot // 2), pos[None], "half",
                         d_rot, False)
    tol = HALF_BF16 * ref.abs() + 2.0 ** -19 * mag
    assert bool(((wk.cpu().double() - ref).abs() <= tol).all())
    assert K.device_error() == 0


@pytest.mark.parametrize("counts", [[1, 1, 1], [2, 1, 0], [4, 9, 1],
                                    [60, 1, 30]])
def test_extend_without_a_bound_on_the_rows(counts):
    """A row list without max_rows: every row is attended, in the workspace
    that extend_workspace_size gives without it."""
    g = _gen(171)
    lens = [900, 64, 3000]
    bt, blocks = _table(g, lens, 64)
    c = _cache(g, blocks, 1, 64, "mxfp4")
    rows = sum(counts)
    q = _randn(g, rows, 8, D)
    ref = _attend_ref(c, bt, lens, counts, q)
    args = (c, bt, _i32(lens), max(lens))
    ws = torch.empty(K.extend_workspace_size(*args, rows, 8),
                     dtype=torch.uint8, device="cuda")
    for kw in ({}, dict(workspace=ws)):
        out = torch.full((rows, 8, D), 9.0, dtype=BF, device="cuda")
        _, lse = K.gqa_extend(*args, q, _starts(counts), out=out, **kw)
        assert K.device_error() == 0
        _check(out, lse, ref)
    if rows == 3 and max(counts) == 1:      # and without a list
        out, lse = K.gqa_extend(*args, q, workspace=ws)
        _check(out, lse, ref)


def test_extend_outputs_beside_the_queries():
    """Outputs in the gaps of strided queries are no overlap; in place is
    refused and leaves the queries alone."""
    g = _gen(181)
    lens, n_h = [70, 40], 8
    bt, blocks = _table(g, lens, 64)
    c = _cache(g, blocks, 1, 64, "mxfp4")
    arena = _randn(g, 9, n_h, D)
    args = (c, bt, _i32(lens), max(lens))
    q = arena[1:9:6]                                    # rows 1 and 7
    want, wl = K.gqa_extend(*args, q.contiguous())
    for at in (2, 5):
        out, lse = K.gqa_extend(*args, q, out=arena[at:at + 2])
        assert torch.equal(arena[at:at + 2], want) and torch.equal(lse, wl)
    before = arena.clone()
    for at in (0, 1, 6, 7):
        with pytest.raises(K.KvdError, match="overlaps"):
            K.gqa_extend(*args, q, out=arena[at:at + 2])
    apart = arena[:2].transpose(0, 1).contiguous().transpose(0, 1)
    with pytest.raises(K.KvdError, match="overlaps"):
        K.gqa_extend(*args, apart, out=apart.transpose(0, 1).view(
            2, n_h, D))
    assert torch.equal(arena, before)


@pytest.mark.parametrize("rows", [1, 20, 60])
def test_extend_with_the_largest_length_bound(rows):
    """max_seq_len of 2^31 - 1 plans like one a few chunks below it, and the
    call is right."""
    g = _gen(191)
    bs, T = 2 ** 20, 5000
    k, v = (torch.zeros((1, 1, bs, 72), dtype=torch.uint8, device="cuda")
            for _ in range(2))
    small = _cache(g, 1, 1, 8192, "mxfp4")
    k[:, :, :8192], v[:, :, :8192] = small.k, small.v
    c = K.PagedCache(k, v, bs, 1, D, "mxfp4")
    bt = torch.zeros((1, 2048), dtype=torch.int32, device="cuda")
    top = 2 ** 31 - 1
    assert K.extend_workspace_size(c, bt, _i32([T]), top, rows, 8, rows) == \
        K.extend_workspace_size(c, bt, _i32([T]), top - 4096, rows, 8, rows) > 0
    q = _randn(g, rows, 8, D)
    out, lse = K.gqa_extend(c, bt, _i32([T]), top, q, _starts([rows]), rows)
    _check(out, lse, _attend_ref(small, _i32([[0]]), [T], [rows], q))
    assert K.device_error() == 0


@pytest.mark.parametrize("pairing", ["half", "adjacent"])
def test_rope_angles_at_any_position(pairing):
    """At positions over the whole int32 range the rotation is the one by
    position times the plan's 64-bit fraction of a turn, formed in exact
    integers here; tolerance as in test_rope, whatever the position."""
    d = 128
    plan = K.rope_plan(d, theta=500000.0, pairing=pairing)
    turns = [int(x) % 2 ** 64 for x in plan.turns.tolist()]
    g = _gen(201)
    p = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, -2 ** 29 - 7,
         123456789, 16777217, -99999999]
    x = _randn(g, len(p), 3, d)
    y, _ = K.rope(plan, _i32([p]), x)
    frac = np.array([[(t * a % 2 ** 64) / 2.0 ** 64 for t in turns]
                     for a in p])[:, None]
    c, s = (torch.from_numpy(f(2 * np.pi * frac)) for f in (np.cos, np.sin))
    i = torch.arange(d // 2)
    a, b = (i, i + d // 2) if pairing == "half" else (2 * i, 2 * i + 1)
    v = x.double().cpu()
    ref, mag = v.clone(), v.clone()
    ref[..., a] = v[..., a] * c - v[..., b] * s
    ref[..., b] = v[..., b] * c + v[..., a] * s
    mag[..., a] = mag[..., b] = v[..., a].abs() + v[..., b].abs()
    tol = HALF_BF16 * ref.abs() + 2.0 ** -19 * mag
    assert bool(((y.cpu().double() - ref).abs() <= tol).all())
    assert K.device_error() == 0


# ---------------------------------------------------------------------------
# many sequences, wide groups of single tokens, two calls at once
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("batch,n_h,n_kv,counts,window", [
    (65, 8, 1, 1, 0), (300, 16, 2, 1, 0), (1024, 16, 1, 1, 0),
    (1024, 3, 1, 2, 40), (200, 8, 1, 4, 0), (1024, 16, 1, 2, 0),
    (1000, 40, 1, 1, 0)])
def test_extend_many_sequences(batch, n_h, n_kv, counts, window):
    """Up to 1,024 sequences by either kernel, a tenth of them empty, one of
    them long."""
    g = _gen(batch + n_h)
    lens = [0 if i % 10 == 3 else 7 * i % 90 + 1 for i in range(batch)]
    lens[batch // 2] = 6000
    n = [0 if i % 9 == 4 else counts for i in range(batch)]
    if counts == 1:
        n = [1] * batch
    bt, blocks = _table(g, lens, 32)
    c = _cache(g, blocks, n_kv, 32, "mxfp4")
    q = _randn(g, sum(n), n_h, D)
    args = (c, bt, _i32(lens), 6000, q)
    ref = _attend_ref(c, bt, lens, n, q, window)
    out, lse = K.gqa_extend(*args, _starts(n), counts, window=window)
    _check(out, lse, ref)
    if counts == 1:
        a, b = K.gqa_extend(*args, window=window)
        assert torch.equal(a, out) and torch.equal(b, lse)
    assert K.device_error() == 0


@pytest.mark.parametrize("group", [17, 24, 100, 128])
def test_extend_single_tokens_of_wide_groups(group):
    """One token a sequence without a row list on tcgen05."""
    g = _gen(211 + group)
    lens = [5000, 1, 0, 129, 700]
    bt, blocks = _table(g, lens, 64)
    c = _cache(g, blocks, 2, 64, "mxfp4")
    q = _randn(g, 5, 2 * group, D)
    for window in (0, 60):
        out, lse = K.gqa_extend(c, bt, _i32(lens), 5000, q, window=window)
        _check(out, lse, _attend_ref(c, bt, lens, [1] * 5, q, window))
    assert K.device_error() == 0


def test_calls_on_two_streams_at_once():
    """Prompts, drafts and single tokens of two models, interleaved on two
    streams with nothing between them, give each call's own result."""
    g = _gen(221)
    jobs = []
    for counts, n_kv in (([300, 200], 2), ([4, 4], 8), ([1, 1], 8)):
        for _ in range(2):
            lens = [9000, 5000]
            bt, blocks = _table(g, lens, 64)
            c = _cache(g, blocks, n_kv, 64, "mxfp4")
            q = _randn(g, sum(counts), 8 * n_kv, D)
            args = (c, bt, _i32(lens), 9000, q, _starts(counts), max(counts))
            jobs.append((args, K.gqa_extend(*args)))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for i, (args, _) in enumerate(jobs):
            got.append((i, K.gqa_extend(*args, stream=streams[i & 1])))
    torch.cuda.synchronize()
    for i, (out, lse) in got:
        assert torch.equal(out, jobs[i][1][0])
        assert torch.equal(lse, jobs[i][1][1])
    assert K.device_error() == 0
