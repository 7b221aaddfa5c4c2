"""The prompt path without a GPU: include/kvd_prompt.h's functions are
exported and refuse bad arguments on the host before any CUDA call (fake
aligned pointers stand in for device buffers; every call here fails
validation or has nothing to do), the frequencies of rotary positions, and
the binding's refusals."""
import ctypes
import os
from fractions import Fraction

import numpy as np
import pytest
import torch

import kv_cache_decode_gqa_gb300 as K
from kv_cache_decode_gqa_gb300 import _native as N

FAKE = 0x10000          # 16-byte aligned, never dereferenced
# 1 / (2 pi) to 60 digits
INV_2PI = Fraction(
    159154943091895335768883763372514362034459645740456448747667,
    10 ** 60)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(N.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return N.lib()


def _with(obj, kw):
    for k, v in kw.items():
        setattr(obj, k, v)
    return obj


def _cache(**kw):
    return _with(N.KvdCache(FAKE, FAKE + 0x100000, 10, 64, 8, 128, 2, 0, None,
                            None, None, None), kw)


def _seqs(**kw):
    return _with(N.KvdSeqs(FAKE + 0x200000, FAKE + 0x300000, 4, 16, 1000, 0),
                 kw)


def _rows(heads=8, **kw):
    return _with(N.KvdRows(FAKE + 0x400000, 6, heads, heads * 128, 128), kw)


def _plan(**kw):
    return _with(N.KvdRopePlan(FAKE, None, 128, 1, 0, 0), kw)


def _says(lib, text):
    return text.encode() in lib.kvd_last_error()


def test_exports_every_declared_function(lib):
    names = N.header_functions(N.PROMPT_HEADER)
    assert names == sorted(["kvd_rope_turns", "kvd_rope", "kvd_kv_write",
                            "kvd_kv_read", "kvd_gqa_extend",
                            "kvd_extend_workspace_size"])
    for name in names:
        assert hasattr(lib, name) and name in N._SIGS


# ---------------------------------------------------------------------------
# frequencies
# ---------------------------------------------------------------------------
def _turns(lib, freqs):
    f = np.array(freqs, dtype=np.float64)
    t = np.empty(f.size, dtype=np.uint64)
    assert lib.kvd_rope_turns(f.ctypes.data, f.size, t.ctypes.data) == 0
    return [int(x) for x in t]


def test_turns_are_the_fractions_of_a_turn(lib):
    freqs = [1.0, 0.5, 1e-4, 10000.0 ** -0.9, 3.25, 6.5, 123.456, 2.0 ** 30,
             1e-12, 0.0, -1.0, -1e-4, -77.7]
    for f, t in zip(freqs, _turns(lib, freqs)):
        want = (Fraction(f) * INV_2PI) % 1 * 2 ** 64
        d = (t - want) % 2 ** 64
        d = min(d, 2 ** 64 - d)
        # half a unit of 2^-64, and 2^-104 of the product's size
        assert d <= Fraction(1, 2) + abs(Fraction(f)) * Fraction(1, 2 ** 38)


def test_turns_refusals(lib):
    t = np.empty(2, dtype=np.uint64)
    for bad in (np.nan, np.inf, 2.0 ** 31, -2.0 ** 31):
        f = np.array([1.0, bad])
        assert lib.kvd_rope_turns(f.ctypes.data, 2, t.ctypes.data) == 2
    assert lib.kvd_rope_turns(None, 2, t.ctypes.data) == 1
    assert lib.kvd_rope_turns(None, -1, None) == 2
    assert lib.kvd_rope_turns(None, 0, None) == 0


def test_rope_axes():
    assert K.rope_axes(8, [1, 2, 1]) == [0, 1, 1, 2]
    assert K.rope_axes(12, [1, 2, 3], interleave=True) == [0, 1, 2, 1, 2, 2]
    assert K.rope_axes(4, [2]) == [0, 0]
    for bad in ([1, 1], [], [1, 1, 1, 1, 0], [5, -1]):
        with pytest.raises(ValueError):
            K.rope_axes(8, bad)
    with pytest.raises(ValueError):
        K.rope_plan(7, device="cpu")
    with pytest.raises(ValueError):
        K.rope_plan(8, pairing="quarter", device="cpu")
    with pytest.raises(ValueError):
        K.rope_plan(8, freqs=[1.0], device="cpu")


# ---------------------------------------------------------------------------
# refusals of the C ABI
# ---------------------------------------------------------------------------
def _rope(lib, plan=None, pos=FAKE, stride=6, d=128, q=None, qo=None, k=None,
          ko=None):
    q = _rows() if q is None else q
    qo = _rows(data=FAKE + 0x800000) if qo is None else qo
    return lib.kvd_rope(plan or _plan(), pos, stride, d, q, qo, k, ko, None)


def test_rope_refusals(lib):
    assert lib.kvd_rope(None, FAKE, 6, 128, _rows(), _rows(), None, None,
                        None) == 1
    assert lib.kvd_rope(_plan(), FAKE, 6, 128, None, None, None, None,
                        None) == 1
    assert _rope(lib, _plan(d_rot=7)) == 2
    assert _rope(lib, _plan(d_rot=130)) == 2          # wider than the head
    wide = _rows(head_stride=4096, row_stride=8 * 4096)
    assert _rope(lib, _plan(d_rot=2048), d=4096, q=wide, qo=wide) == 3
    assert _rope(lib, _plan(n_axes=5), stride=6) == 3
    assert _rope(lib, _plan(n_axes=3), stride=5) == 2  # axes overlap
    assert _rope(lib, _plan(pairing=2)) == 3
    assert _rope(lib, _plan(inverse=2)) == 2
    assert _rope(lib, _plan(turns=None)) == 1
    assert _rope(lib, pos=None) == 1
    assert _rope(lib, q=_rows(data=None)) == 1
    assert _rope(lib, q=_rows(rows=-1)) == 2
    assert _rope(lib, q=_rows(row_stride=-8)) == 2
    assert _rope(lib, qo=_rows(rows=5)) == 2 and _says(lib, "shapes")
    # output rows that overlap, and in place with other strides
    assert _rope(lib, qo=_rows(row_stride=128)) == 2
    assert _says(lib, "overlap")
    assert _rope(lib, qo=_rows(head_stride=0)) == 2
    assert _rope(lib, q=_rows(row_stride=2048), qo=_rows()) == 2
    assert _says(lib, "in place")
    assert _rope(lib, k=_rows(rows=5), ko=_rows(rows=5)) == 2
    assert _rope(lib, k=_rows()) == 1                  # k without k_out
    e = _rows(rows=0)
    assert _rope(lib, q=e, qo=e) == 0                  # nothing to do


def _write(lib, c=None, bt=FAKE, nb=16, start=FAKE, rs=FAKE, B=4, k=None,
           v=None, plan=None, pos=None, stride=6, q=None, qo=None):
    return lib.kvd_kv_write(c or _cache(), bt, nb, start, rs, B,
                            k or _rows(), v or _rows(), plan, pos, stride, q,
                            qo, None)


def test_write_refusals(lib):
    assert _write(lib, _cache(k=None)) == 1
    assert _write(lib, _cache(block_size=63)) == 2
    assert _write(lib, bt=None) == 1
    assert _write(lib, start=None) == 1
    assert _write(lib, rs=None) == 1
    assert _write(lib, nb=0) == 2
    assert _write(lib, B=-1) == 2
    assert _write(lib, B=65536) == 2
    assert _write(lib, k=_rows(heads=7)) == 2
    assert _write(lib, v=_rows(rows=5)) == 2
    assert _write(lib, k=_rows(data=FAKE + 2)) == 2 and _says(lib, "aligned")
    assert _write(lib, k=_rows(row_stride=1028)) == 2
    assert _write(lib, _cache(dtype=1)) == 1           # inverse scales
    assert lib.kvd_kv_write(_cache(), FAKE, 16, FAKE, FAKE, 4, _rows(), None,
                            None, None, 0, None, None, None) == 1
    assert lib.kvd_kv_write(_cache(), FAKE, 16, FAKE, FAKE, 4, None, _rows(),
                            None, None, 0, None, None, None) == 1
    assert _write(lib, q=_rows(), qo=_rows()) == 1     # q without rope
    assert _write(lib, plan=_plan(), pos=FAKE, q=_rows()) == 1
    assert _write(lib, plan=_plan(), pos=FAKE, q=_rows(rows=5),
                  qo=_rows(rows=5)) == 2
    assert _write(lib, plan=_plan()) == 1              # no positions
    assert _write(lib, plan=_plan(d_rot=256), pos=FAKE) == 2
    assert _write(lib, B=0) == 0
    e = _rows(rows=0)
    assert _write(lib, k=e, v=e) == 0


def test_read_refusals(lib):
    def read(c=None, k=None, v=None, **kw):
        a = dict(bt=FAKE, nb=16, start=FAKE, rs=FAKE, B=4)
        a.update(kw)
        return lib.kvd_kv_read(c or _cache(), a["bt"], a["nb"], a["start"],
                               a["rs"], a["B"], k, v, None)
    assert read() == 1                                  # no output at all
    assert read(_cache(v=None), v=_rows()) == 1
    assert read(k=_rows(heads=4)) == 2
    assert read(k=_rows(), v=_rows(rows=3)) == 2
    assert read(k=_rows(row_stride=128)) == 2           # rows overlap
    assert read(_cache(dtype=1), k=_rows()) == 1        # scales
    assert read(k=_rows(), rs=None) == 1
    assert read(k=_rows(data=FAKE + 8)) == 2
    assert read(k=_rows(), B=0) == 0


def _extend(lib, c=None, s=None, rs=FAKE, max_rows=6, q=None, out=FAKE,
            lse=None, ws=None, n=0):
    return lib.kvd_gqa_extend(c or _cache(), s or _seqs(), rs, max_rows,
                              q or _rows(64), 0.0, out, lse, ws, n, None)


def test_extend_refusals(lib):
    assert lib.kvd_gqa_extend(_cache(), _seqs(), FAKE, 6, None, 0.0, FAKE,
                              None, None, 0, None) == 1
    assert _extend(lib, _cache(v=None)) == 1
    assert _extend(lib, _cache(dtype=0)) == 3 and _says(lib, "MXFP4")
    assert _extend(lib, _cache(dtype=1)) == 3
    assert _extend(lib, _cache(head_dim=64)) == 3
    assert _extend(lib, q=_rows(60)) == 2              # not a multiple
    assert _extend(lib, q=_rows(8 * 129)) == 3         # group 129
    assert _extend(lib, s=_seqs(batch=1025)) == 3
    assert _extend(lib, s=_seqs(flags=4)) == 2
    assert _extend(lib, s=_seqs(window=-1)) == 2
    assert _extend(lib, s=_seqs(max_seq_len=16 * 64 + 1)) == 4
    assert _extend(lib, max_rows=-1) == 2
    assert _extend(lib, rs=None) == 2                  # 6 rows, 4 sequences
    assert _extend(lib, rs=None, max_rows=2, q=_rows(64, rows=4)) == 2
    assert _extend(lib, q=_rows(64, rows=1 << 26)) == 2
    assert _extend(lib, q=_rows(64, data=FAKE + 8)) == 2
    assert _extend(lib, q=_rows(64, head_stride=132)) == 2
    assert _extend(lib, out=FAKE + 2) == 2
    assert _extend(lib, out=None) == 1
    assert _extend(lib, s=_seqs(batch=0)) == 0
    assert _extend(lib, q=_rows(64, rows=0), max_rows=0) == 0
    size = ctypes.c_size_t(0)
    assert lib.kvd_extend_workspace_size(_cache(), _seqs(), 6, 6, 64,
                                         None) == 1
    assert lib.kvd_extend_workspace_size(_cache(dtype=0), _seqs(), 6, 6, 64,
                                         size) == 3


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------
def _host():
    i32 = dict(dtype=torch.int32)
    bf = dict(dtype=torch.bfloat16)
    cache = K.PagedCache(torch.zeros((2, 2, 16, 72), dtype=torch.uint8),
                         torch.zeros((2, 2, 16, 72), dtype=torch.uint8), 16,
                         2, 128, "mxfp4")
    return dict(cache=cache, bt=torch.zeros((1, 2), **i32),
                one=torch.zeros(1, **i32), rs=torch.zeros(2, **i32),
                kv=torch.zeros((3, 2, 128), **bf),
                q=torch.zeros((3, 4, 128), **bf))


CALLS = {
    "rope": lambda a: K.rope(None, None, a["q"]),
    "kv_write": lambda a: K.kv_write(a["cache"], a["bt"], a["one"], a["rs"],
                                     a["kv"], a["kv"]),
    "kv_read": lambda a: K.kv_read(a["cache"], a["bt"], a["one"], a["rs"], 3),
    "gqa_extend": lambda a: K.gqa_extend(a["cache"], a["bt"], a["one"], 32,
                                         a["q"], a["rs"], 3),
    "extend_workspace_size": lambda a: K.extend_workspace_size(
        a["cache"], a["bt"], a["one"], 32, 3, 4, 3),
    "rope_plan": lambda a: K.RopePlan(torch.zeros(4, dtype=torch.int64), None,
                                      8, 1, "half"),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_host_tensors_are_refused(name, monkeypatch):
    def no_library():
        raise AssertionError("the library was called with host tensors")
    monkeypatch.setattr(K, "lib", no_library)
    with pytest.raises(ValueError, match="CUDA tensor"):
        CALLS[name](_host())


def test_calls_take_a_stream_keyword():
    import inspect
    for f in (K.rope, K.kv_write, K.kv_read, K.gqa_extend):
        assert "stream" in inspect.signature(f).parameters
        assert f.__doc__


def test_write_rotates_heads_that_fit_in_shared_memory(lib):
    """2 head_dim + 4 d_rot bytes up to 204,784 (nothing to do: no rows)."""
    for d_rot, most in ((128, 102136), (1024, 100344)):
        assert 2 * most + 4 * d_rot == 204784
        for d, want in ((most, 0), (most + 8, 3)):
            e = _rows(rows=0, head_stride=d, row_stride=8 * d)
            assert _write(lib, _cache(dtype=0, head_dim=d), k=e, v=e,
                          plan=_plan(d_rot=d_rot), pos=FAKE) == want


def test_extend_refuses_outputs_over_the_queries(lib):
    """Six rows of 64 heads: in place, and a few bytes shared at either end;
    strided queries of which one vector is met."""
    n = 6 * 64 * 128 * 2
    at = FAKE + 0x400000                                # where _rows() lie
    row = 64 * 128
    wide = _rows(64, rows=2, row_stride=8 * row)
    apart = _rows(64, rows=1, head_stride=128 * 65)
    for q, out in ((_rows(64), at), (_rows(64), at + n - 16),
                   (_rows(64), at - n + 16), (wide, at + 2 * 7 * row),
                   (wide, at + 2 * 8 * row), (apart, at + 2 * 128 + 16),
                   (apart, at + 2 * 128 * 65 * 63)):
        assert _extend(lib, q=q, out=out) == 2 and _says(lib, "overlaps")
