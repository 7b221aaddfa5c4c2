"""Drafted trees and cross attention without a GPU: include/kvd_tree.h's
functions are exported and refuse bad arguments on the host before any CUDA
call (fake aligned pointers stand in for device buffers; every call here fails
validation or has nothing to do), and the binding's refusals."""
import ctypes
import os

import pytest
import torch

import kv_cache_decode_gqa_gb300 as K
from kv_cache_decode_gqa_gb300 import _native as N

FAKE = 0x10000          # 16-byte aligned, never dereferenced


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
    return _with(N.KvdCache(FAKE, FAKE + 0x100000, 10, 64, 8, 128, 0, 0, None,
                            None, None, None), kw)


def _seqs(**kw):
    return _with(N.KvdSeqs(FAKE + 0x200000, FAKE + 0x300000, 4, 16, 1000, 0),
                 kw)


def _rows(heads=64, **kw):
    return _with(N.KvdRows(FAKE + 0x400000, 6, heads, heads * 128, 128), kw)


def _says(lib, text):
    return text.encode() in lib.kvd_last_error()


def test_exports_every_declared_function(lib):
    names = N.header_functions(N.TREE_HEADER)
    assert names == sorted(["kvd_tree_plan", "kvd_gqa_tree", "kvd_gqa_cross",
                            "kvd_attend_workspace_size", "kvd_kv_keep"])
    for name in names:
        assert hasattr(lib, name) and name in N._SIGS


def _plan(lib, parents=FAKE, start=FAKE, row_start=FAKE, batch=4, rows=6,
          max_rows=6, window=0, masks=FAKE, positions=None):
    return lib.kvd_tree_plan(parents, start, row_start, batch, rows, max_rows,
                             window, masks, positions, None)


def test_tree_plan_validation(lib):
    for name in ("parents", "start", "row_start", "masks"):
        assert _plan(lib, **{name: None}) == 1
    for name in ("batch", "rows", "max_rows", "window"):
        assert _plan(lib, **{name: -1}) == 2
    assert _plan(lib, max_rows=257) == 3 and _says(lib, "256")
    assert _plan(lib, batch=1025) == 3
    for name in ("batch", "rows", "max_rows"):
        assert _plan(lib, parents=None, **{name: 0}) == 0   # nothing to do


def _tree(lib, c=None, s=None, row_start=FAKE, max_rows=6, q=None, masks=FAKE,
          positions=None, out=FAKE + 0x800000):
    return lib.kvd_gqa_tree(c or _cache(), s or _seqs(), row_start, max_rows,
                            q or _rows(), masks, positions, 0.0, out, None,
                            None, 0, None)


def _cross(lib, c=None, s=None, row_start=FAKE, max_rows=6, q=None,
           out=FAKE + 0x800000):
    return lib.kvd_gqa_cross(c or _cache(), s or _seqs(), row_start, max_rows,
                             q or _rows(), 0.0, out, None, None, 0, None)


@pytest.mark.parametrize("call", [_tree, _cross])
def test_attention_validation(lib, call):
    assert call(lib, _cache(k=None)) == 1
    assert call(lib, _cache(v=None)) == 1
    assert call(lib, _cache(head_dim=96)) == 3
    assert call(lib, _cache(dtype=1)) == 1 and _says(lib, "k_scale")
    assert call(lib, _cache(dtype=2, head_dim=64)) == 3
    assert call(lib, _cache(dtype=2, block_size=3)) == 2
    assert call(lib, _cache(dtype=9)) == 3
    assert call(lib, _cache(), _seqs(batch=1025)) == 3
    assert call(lib, _cache(), _seqs(batch=-1)) == 2
    assert call(lib, _cache(), _seqs(max_seq_len=1025)) == 4
    assert call(lib, _cache(), _seqs(max_blocks_per_seq=2 ** 26,
                                     max_seq_len=2 ** 31 - 1)) == 3
    assert call(lib, _cache(num_blocks=2 ** 22)) == 3  # 2^31 rows
    assert call(lib, _cache(), _seqs(flags=4)) == 2
    assert call(lib, _cache(), _seqs(window=-1)) == 2
    assert call(lib, q=_rows(60)) == 2                 # not a multiple
    assert call(lib, q=_rows(129 * 8)) == 3            # groups of 129
    assert call(lib, q=_rows(data=FAKE + 8)) == 2
    assert call(lib, q=_rows(row_stride=8193)) == 2
    assert call(lib, q=_rows(row_stride=-8)) == 2
    assert call(lib, q=_rows(rows=-1)) == 2
    assert call(lib, q=_rows(data=None)) == 1
    assert call(lib, q=_rows(rows=1 << 25)) == 2       # rows x n_h over 2^31
    assert call(lib, max_rows=-1) == 2
    assert call(lib, out=None) == 1
    assert call(lib, out=FAKE + 8) == 2
    assert call(lib, out=FAKE + 0x400000) == 2 and _says(lib, "overlaps")
    assert call(lib, _cache(), _seqs(batch=0)) == 0    # nothing to do
    assert call(lib, q=_rows(rows=0)) == 0
    assert call(lib, max_rows=0) == 0


def test_tree_and_cross_refusals_of_their_own(lib):
    assert _tree(lib, masks=None) == 1
    assert _tree(lib, row_start=None) == 1
    assert _tree(lib, s=_seqs(batch=6), row_start=None, max_rows=1) == 1
    assert _tree(lib, max_rows=257) == 3 and _says(lib, "256")
    assert _tree(lib, s=_seqs(window=5)) == 1 and _says(lib, "positions")
    assert _cross(lib, s=_seqs(window=5)) == 3
    assert _cross(lib, row_start=None) == 2 and _says(lib, "one row")
    assert _cross(lib, s=_seqs(batch=6), row_start=None, max_rows=2) == 2


@pytest.mark.parametrize("call", [_tree, _cross])
def test_keys_and_values_far_apart_are_refused(lib, call):
    for k, v in ((FAKE, FAKE + 2 ** 40), (FAKE + 2 ** 41, FAKE)):
        assert call(lib, _cache(k=k, v=v)) == 3 and _says(lib, "apart")
    # (rows = 0: over before anything is read)
    near = _cache(k=FAKE, v=FAKE + 2 ** 40 - 16)
    assert call(lib, near, q=_rows(rows=0)) == 0
    assert call(lib, _cache(v=FAKE + 2 ** 40, dtype=1, k_scale=FAKE,
                            v_scale=FAKE), q=_rows(rows=0)) == 0


def test_workspace_size_validation(lib):
    size = ctypes.c_size_t(0)
    f = lib.kvd_attend_workspace_size
    assert f(_cache(), _seqs(), 6, 6, 64, 1, None) == 1
    assert f(_cache(), _seqs(), 6, 6, 60, 1, ctypes.byref(size)) == 2
    assert f(_cache(), _seqs(), 6, 1, 64, 0, ctypes.byref(size)) == 2
    assert f(_cache(head_dim=32), _seqs(), 6, 6, 64, 1,
             ctypes.byref(size)) == 3


def _keep(lib, caches=None, n=None, table=FAKE, blocks=4, start=FAKE,
          path=FAKE, width=5, n_keep=FAKE, batch=3):
    caches = caches or [_cache(), _cache()]
    arr = (N.KvdCache * len(caches))(*caches)
    return lib.kvd_kv_keep(arr, len(caches) if n is None else n, table, blocks,
                           start, path, width, n_keep, batch, None)


def test_kv_keep_validation(lib):
    for name in ("table", "start", "path", "n_keep"):
        assert _keep(lib, **{name: None}) == 1
    assert _keep(lib, [_cache(k=None)]) == 1
    assert lib.kvd_kv_keep(None, 1, FAKE, 4, FAKE, FAKE, 5, FAKE, 3, None) == 1
    for name in ("n", "width", "batch"):
        assert _keep(lib, **{name: -1}) == 2
    assert _keep(lib, blocks=0) == 2
    assert _keep(lib, width=257) == 3
    assert _keep(lib, batch=1025) == 3
    for field, value in (("num_blocks", 11), ("block_size", 32), ("n_kv", 4),
                         ("head_dim", 64), ("dtype", 1), ("v", None)):
        assert _keep(lib, [_cache(), _cache(**{field: value})]) == 2
        assert _says(lib, "cache 1")
    assert _keep(lib, [_cache(k=FAKE + 4)]) == 2
    for name in ("n", "width", "batch"):
        assert _keep(lib, table=None, **{name: 0}) == 0


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------
def _i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_host_tensors_are_refused(monkeypatch):
    def no_library():
        raise AssertionError("the library was called with host tensors")
    monkeypatch.setattr(K, "lib", no_library)
    bf = dict(dtype=torch.bfloat16)
    c = K.PagedCache(torch.zeros(2, 2, 16, 64, **bf),
                     torch.zeros(2, 2, 16, 64, **bf), 16, 2, 64)
    q = torch.zeros(3, 4, 64, **bf)
    for call in (
            lambda: K.tree_plan(_i32(3), _i32(1), _i32(2), 3),
            lambda: K.gqa_tree(c, _i32(1, 2), _i32(1), 32, q, _i32(2), 3,
                               _i32(3, 1)),
            lambda: K.gqa_cross(c, _i32(1, 2), _i32(1), 32, q, _i32(2)),
            lambda: K.kv_keep([c], _i32(1, 2), _i32(1), _i32(1, 2), _i32(1)),
            lambda: K.attend_workspace_size(c, _i32(1, 2), _i32(1), 32, 3,
                                            4)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


def test_empty_cache_list_is_refused():
    with pytest.raises(ValueError, match="needs a cache"):
        K.CacheList([])
