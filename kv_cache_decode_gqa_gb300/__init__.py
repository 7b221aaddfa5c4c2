"""kv_cache_decode_gqa_gb300: Python binding of libkvd.so.

The functions here only marshal arguments: they take torch CUDA tensors,
pass their device pointers and the current CUDA stream to the C ABI
(include/kvd.h), and allocate outputs / workspace with torch when the caller
does not pass them. Every step of the computation runs in the library's
CUDA kernels; there is no other path.

Cache layout (per layer): K and V tensors [num_blocks][n_kv][block_size]
[head_dim] of bf16 (torch.bfloat16) or fp8-e4m3 codes (torch.uint8), or
[num_blocks][n_kv][block_size][head_dim/2 + head_dim/16] bytes of MXFP4 rows
(torch.uint8; include/kvd.h gives the row format).
"""
import contextlib
import ctypes
import functools
import inspect
from dataclasses import dataclass
from typing import Optional

from . import _native
from ._native import KvdError, check, lib

__all__ = ["PagedCache", "kv_append", "gqa_decode", "mla_decode",
           "indexer_topk", "indexer_pool", "indexer_topk_pool",
           "BlockPool", "copy_blocks",
           "sparse_decode", "workspace_size",
           "RopePlan", "rope_plan", "rope", "kv_write", "kv_read",
           "gqa_extend", "extend_workspace_size",
           "bytes_per_token", "device_error", "launch_count", "set_tuning",
           "KvdError",
           "OP_GQA_DECODE", "OP_MLA_DECODE", "OP_INDEXER_TOPK",
           "OP_SPARSE_DECODE"]

BF16 = 0
FP8_E4M3 = 1
MXFP4 = 2
_DTYPES = {"bf16": BF16, "fp8": FP8_E4M3, "mxfp4": MXFP4}
OP_GQA_DECODE = 0
OP_MLA_DECODE = 1
OP_INDEXER_TOPK = 2
OP_SPARSE_DECODE = 3
OP_INDEXER_TOPK_POOL = 4
POOL_BLOCKS = 2048   # KVD_POOL_BLOCKS
POOL_BLOCK = 8       # KVD_POOL_BLOCK


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t, name, dtype=None, numel=None):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must have {numel} elements, got {t.numel()}")
    return t


@dataclass
class PagedCache:
    """One layer's paged cache. ``v`` is None for a K-only cache."""
    k: "torch.Tensor"
    v: Optional["torch.Tensor"]
    block_size: int
    n_kv: int
    head_dim: int
    dtype: str = "bf16"          # "bf16" | "fp8" | "mxfp4"
    k_scale: Optional["torch.Tensor"] = None      # fp32 [n_kv]
    v_scale: Optional["torch.Tensor"] = None
    k_inv_scale: Optional["torch.Tensor"] = None
    v_inv_scale: Optional["torch.Tensor"] = None

    @property
    def num_blocks(self):
        return self.k.shape[0]

    def struct(self):
        import torch
        want = torch.bfloat16 if self.dtype == "bf16" else torch.uint8
        _need(self.k, "cache.k", want)
        if self.v is not None:
            _need(self.v, "cache.v", want, self.k.numel())
        row = (self.head_dim // 2 + self.head_dim // 16
               if self.dtype == "mxfp4" else self.head_dim)
        shape = (self.num_blocks, self.n_kv, self.block_size, row)
        if tuple(self.k.shape) != shape:
            raise ValueError(f"cache.k shape {tuple(self.k.shape)} != {shape}")
        for n in ("k_scale", "v_scale", "k_inv_scale", "v_inv_scale"):
            t = getattr(self, n)
            if t is not None:
                _need(t, n, torch.float32, self.n_kv)
        return _native.KvdCache(
            _ptr(self.k), _ptr(self.v), self.num_blocks, self.block_size,
            self.n_kv, self.head_dim, _DTYPES[self.dtype],
            0, _ptr(self.k_scale), _ptr(self.v_scale), _ptr(self.k_inv_scale),
            _ptr(self.v_inv_scale))


SEQS_STABLE = 1  # KVD_SEQS_STABLE
SEQS_PREFIX_READY = 2  # KVD_SEQS_PREFIX_READY (with SEQS_STABLE)


def _seqs(block_table, seq_lens, max_seq_len, flags=0, window=0,
          window_start=None):
    import torch
    _need(block_table, "block_table", torch.int32)
    _need(seq_lens, "seq_lens", torch.int32)
    if block_table.dim() != 2 or block_table.shape[0] != seq_lens.numel():
        raise ValueError("block_table must be [batch][max_blocks_per_seq]")
    if window_start is not None:
        _need(window_start, "window_start", torch.int32, seq_lens.numel())
    return _native.KvdSeqs(_ptr(block_table), _ptr(seq_lens),
                           block_table.shape[0], block_table.shape[1],
                           int(max_seq_len), int(flags), int(window),
                           _ptr(window_start))


def workspace_size(op, cache, block_table, seq_lens, max_seq_len, n_h, k=0,
                   window=0):
    """Workspace bytes of a call (kvd_workspace_size); a GQA decode's window
    is part of its plan (short windows need none)."""
    c = cache.struct()
    s = _seqs(block_table, seq_lens, max_seq_len, window=window)
    out = ctypes.c_size_t(0)
    check(lib().kvd_workspace_size(op, ctypes.byref(c), ctypes.byref(s), n_h,
                                   k, ctypes.byref(out)))
    return out.value


def _workspace(op, cache, block_table, seq_lens, max_seq_len, n_h, k,
               workspace, window=0):
    import torch
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8)
        return workspace
    n = workspace_size(op, cache, block_table, seq_lens, max_seq_len, n_h, k,
                       window)
    # every partial a call keeps here is written before it is read
    return torch.empty(max(n, 256), dtype=torch.uint8,
                       device=block_table.device)


def kv_append(cache, block_table, pos, k_new, v_new=None, stream=None):
    """Write k_new (and v_new) [batch][n_kv][head_dim] bf16 at slot pos[b]."""
    import torch
    c = cache.struct()
    _need(block_table, "block_table", torch.int32)
    _need(pos, "pos", torch.int32)
    _need(k_new, "k_new", torch.bfloat16)
    if v_new is not None:
        _need(v_new, "v_new", torch.bfloat16, k_new.numel())
    check(lib().kvd_kv_append(ctypes.byref(c), _ptr(block_table),
                              block_table.shape[1], _ptr(pos), pos.numel(),
                              _ptr(k_new), _ptr(v_new), _stream(stream)))


def _outputs(q, n_h, dv, out, lse, want_lse):
    import torch
    B = q.shape[0]
    if out is None:
        out = torch.empty((B, n_h, dv), dtype=torch.bfloat16, device=q.device)
    _need(out, "out", torch.bfloat16, B * n_h * dv)
    if lse is None and want_lse:
        lse = torch.empty((B, n_h), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", torch.float32, B * n_h)
    return out, lse


def gqa_decode(cache, block_table, seq_lens, max_seq_len, q, scale=None,
               out=None, lse=None, workspace=None, want_lse=True,
               stream=None, seqs_flags=0, window=0, window_start=None):
    """GQA/MHA decode: q [batch][n_h][head_dim] bf16 -> (out, lse).
    seqs_flags: 0 or SEQS_STABLE (see KVD_SEQS_STABLE in kvd.h). window W >
    0: sliding-window decode over positions [max(s_b, len_b - W), len_b),
    s_b = window_start[b] (int32 device tensor) or 0."""
    import torch
    _need(q, "q", torch.bfloat16)
    n_h = q.shape[1]
    c = cache.struct()
    s = _seqs(block_table, seq_lens, max_seq_len, seqs_flags, window,
              window_start)
    out, lse = _outputs(q, n_h, cache.head_dim, out, lse, want_lse)
    ws = _workspace(OP_GQA_DECODE, cache, block_table, seq_lens, max_seq_len,
                    n_h, 0, workspace, window)
    check(lib().kvd_gqa_decode(ctypes.byref(c), ctypes.byref(s), _ptr(q), n_h,
                               float(scale or 0.0), _ptr(out), _ptr(lse),
                               _ptr(ws), ws.numel(), _stream(stream)))
    return out, lse


def gqa_append_decode(cache, block_table, seq_lens, max_seq_len, pos, k_new,
                      v_new, q, scale=None, out=None, lse=None,
                      workspace=None, want_lse=True, stream=None,
                      seqs_flags=0, window=0, window_start=None):
    """kv_append then gqa_decode in one pass (kvd_gqa_append_decode);
    window / window_start as for gqa_decode."""
    import torch
    _need(q, "q", torch.bfloat16)
    _need(pos, "pos", torch.int32)
    _need(k_new, "k_new", torch.bfloat16)
    _need(v_new, "v_new", torch.bfloat16)
    n_h = q.shape[1]
    c = cache.struct()
    s = _seqs(block_table, seq_lens, max_seq_len, seqs_flags, window,
              window_start)
    out, lse = _outputs(q, n_h, cache.head_dim, out, lse, want_lse)
    ws = _workspace(OP_GQA_DECODE, cache, block_table, seq_lens, max_seq_len,
                    n_h, 0, workspace, window)
    check(lib().kvd_gqa_append_decode(
        ctypes.byref(c), ctypes.byref(s), _ptr(pos), _ptr(k_new), _ptr(v_new),
        _ptr(q), n_h, float(scale or 0.0), _ptr(out), _ptr(lse), _ptr(ws),
        ws.numel(), _stream(stream)))
    return out, lse


def mla_decode(cache, block_table, seq_lens, max_seq_len, q, d_c=512,
               scale=None, out=None, lse=None, workspace=None, want_lse=True,
               stream=None):
    """Latent-cache decode: q [batch][n_h][d_c + d_rope] -> out [..][d_c]."""
    import torch
    _need(q, "q", torch.bfloat16)
    n_h = q.shape[1]
    c = cache.struct()
    s = _seqs(block_table, seq_lens, max_seq_len)
    out, lse = _outputs(q, n_h, d_c, out, lse, want_lse)
    ws = _workspace(OP_MLA_DECODE, cache, block_table, seq_lens, max_seq_len,
                    n_h, 0, workspace)
    check(lib().kvd_mla_decode(ctypes.byref(c), d_c, ctypes.byref(s), _ptr(q),
                               n_h, float(scale or 0.0), _ptr(out), _ptr(lse),
                               _ptr(ws), ws.numel(), _stream(stream)))
    return out, lse


def indexer_topk(cache, block_table, seq_lens, max_seq_len, q_idx, w, k,
                 indices=None, scores=None, workspace=None, stream=None,
                 seqs_flags=0):
    """Indexer scores + top-k: returns (indices [batch][k] int32, scores).
    seqs_flags: SEQS_STABLE [| SEQS_PREFIX_READY] (see kvd_seqs)."""
    import torch
    _need(q_idx, "q_idx", torch.bfloat16)
    _need(w, "w", torch.float32, q_idx.shape[0] * q_idx.shape[1])
    c = cache.struct()
    s = _seqs(block_table, seq_lens, max_seq_len, seqs_flags)
    B = q_idx.shape[0]
    if indices is None:
        indices = torch.empty((B, k), dtype=torch.int32, device=q_idx.device)
    _need(indices, "indices", torch.int32, B * k)
    if scores is not None:
        _need(scores, "scores", torch.float32, B * max(max_seq_len, 1))
        ws = None
    else:
        ws = _workspace(OP_INDEXER_TOPK, cache, block_table, seq_lens,
                        max_seq_len, q_idx.shape[1], k, workspace)
    check(lib().kvd_indexer_topk(ctypes.byref(c), ctypes.byref(s),
                                 _ptr(q_idx), q_idx.shape[1], _ptr(w), k,
                                 _ptr(indices), _ptr(scores), _ptr(ws),
                                 0 if ws is None else ws.numel(),
                                 _stream(stream)))
    return indices, scores


def indexer_pool(block_table, seq_lens, max_seq_len, indices, pool=None,
                 pool_n=None, stream=None):
    """The hierarchical indexer's pool of a selection indices [batch][k]:
    returns (pool [batch][POOL_BLOCKS] ascending 8-position block ids,
    pool_n [batch] their counts)."""
    import torch
    _need(indices, "indices", torch.int32)
    B, k = indices.shape
    s = _seqs(block_table, seq_lens, max_seq_len)
    if pool is None:
        pool = torch.empty((B, POOL_BLOCKS), dtype=torch.int32,
                           device=indices.device)
    if pool_n is None:
        pool_n = torch.empty((B,), dtype=torch.int32, device=indices.device)
    _need(pool, "pool", torch.int32, B * POOL_BLOCKS)
    _need(pool_n, "pool_n", torch.int32, B)
    check(lib().kvd_indexer_pool(ctypes.byref(s), _ptr(indices), k,
                                 _ptr(pool), _ptr(pool_n), _stream(stream)))
    return pool, pool_n


def indexer_topk_pool(cache, block_table, seq_lens, max_seq_len, q_idx, w,
                      pool, pool_n, k, indices=None, scores=None,
                      workspace=None, stream=None):
    """A Reindex layer over a pool: indexer scores of the pool's candidates
    and their top k. Returns (indices [batch][k] int32, scores)."""
    import torch
    _need(q_idx, "q_idx", torch.bfloat16)
    _need(w, "w", torch.float32, q_idx.shape[0] * q_idx.shape[1])
    c = cache.struct()
    s = _seqs(block_table, seq_lens, max_seq_len)
    B = q_idx.shape[0]
    _need(pool, "pool", torch.int32, B * POOL_BLOCKS)
    _need(pool_n, "pool_n", torch.int32, B)
    if indices is None:
        indices = torch.empty((B, k), dtype=torch.int32, device=q_idx.device)
    _need(indices, "indices", torch.int32, B * k)
    if scores is not None:
        _need(scores, "scores", torch.float32, B * POOL_BLOCKS * POOL_BLOCK)
        ws = None
    else:
        ws = _workspace(OP_INDEXER_TOPK_POOL, cache, block_table, seq_lens,
                        max_seq_len, q_idx.shape[1], k, workspace)
    check(lib().kvd_indexer_topk_pool(ctypes.byref(c), ctypes.byref(s),
                                      _ptr(q_idx), q_idx.shape[1], _ptr(w),
                                      _ptr(pool), _ptr(pool_n), k,
                                      _ptr(indices), _ptr(scores), _ptr(ws),
                                      0 if ws is None else ws.numel(),
                                      _stream(stream)))
    return indices, scores


def sparse_decode(cache, block_table, seq_lens, max_seq_len, indices, q,
                  scale=None, out=None, lse=None, workspace=None,
                  want_lse=True, stream=None):
    """Decode over the positions in indices [batch][k] (-1 = skip)."""
    import torch
    _need(q, "q", torch.bfloat16)
    _need(indices, "indices", torch.int32)
    n_h = q.shape[1]
    k = indices.shape[1]
    c = cache.struct()
    s = _seqs(block_table, seq_lens, max_seq_len)
    out, lse = _outputs(q, n_h, cache.head_dim, out, lse, want_lse)
    ws = _workspace(OP_SPARSE_DECODE, cache, block_table, seq_lens,
                    max_seq_len, n_h, k, workspace)
    check(lib().kvd_sparse_decode(ctypes.byref(c), ctypes.byref(s),
                                  _ptr(indices), k, _ptr(q), n_h,
                                  float(scale or 0.0), _ptr(out), _ptr(lse),
                                  _ptr(ws), ws.numel(), _stream(stream)))
    return out, lse


# ---------------------------------------------------------------------------
# the prompt path (include/kvd_prompt.h)
# ---------------------------------------------------------------------------
def _one_device(first, *tensors):
    """The device of a call, all of whose tensors must lie on it."""
    dev = first.device
    for t in tensors:
        if t is not None and t.device != dev:
            raise ValueError(f"tensors on {dev} and {t.device} in one call")
    return dev


def _launching(device, stream):
    """A context in which `device` and the call's stream are current (so that
    what the call allocates belongs to that stream), or None where they are:
    small calls are over sooner than two context managers."""
    import torch
    if stream is None and device.index == torch.cuda.current_device():
        return None
    if stream is not None and stream.device != device:
        raise ValueError(f"a stream of {stream.device} for tensors on "
                         f"{device}")
    stack = contextlib.ExitStack()
    stack.enter_context(torch.cuda.device(device))
    if stream is not None:
        stack.enter_context(torch.cuda.stream(stream))
    return stack


def _current(device):
    """The current stream of `device`, which is current."""
    import torch
    try:
        return torch._C._cuda_getCurrentRawStream(device.index)
    except AttributeError:
        return torch.cuda.current_stream().cuda_stream


def _in_context(call):
    """A call of this module from a function that checks its arguments and
    returns (device, launch): launch(stream handle) runs with the device and
    the keyword `stream` (default: the device's current stream) current."""
    @functools.wraps(call)
    def run(*args, stream=None, **kw):
        device, launch = call(*args, **kw)
        context = _launching(device, stream)
        if context is None:
            return launch(_current(device))
        with context:
            return launch(_current(device))
    sig = inspect.signature(call)
    run.__signature__ = sig.replace(parameters=[
        *sig.parameters.values(),
        inspect.Parameter("stream", inspect.Parameter.KEYWORD_ONLY,
                          default=None)])
    return run


def _rows3(t, name, heads=None, width=None):
    """bf16 [rows][heads][width] with any strides but a unit innermost one."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be torch.bfloat16, got {t.dtype}")
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or (stride[2] != 1 and shape[2] > 1):
        raise ValueError(f"{name} must be [rows][heads][width] with "
                         "contiguous vectors")
    if heads is not None and shape[1] != heads:
        raise ValueError(f"{name} must have {heads} heads, got {shape[1]}")
    if width is not None and shape[2] != width:
        raise ValueError(f"{name} must be {width} wide, got {shape[2]}")
    return _native.KvdRows(t.data_ptr(), shape[0], shape[1], stride[0],
                           stride[1])


def _out_rows(out, like, rows, name):
    """The output of a call that returns rows shaped as `like` (whose KvdRows
    is `rows`): `out`, or a new contiguous tensor; and its KvdRows."""
    import torch
    h, d = rows.heads, like.shape[2]
    if out is not None:
        return out, _rows3(out, name, h, d)
    out = torch.empty_like(like, memory_format=torch.contiguous_format)
    return out, _native.KvdRows(out.data_ptr(), rows.rows, h, h * d, d)


@dataclass(frozen=True)
class RopePlan:
    """Frequencies and axes of rotary positions, on the device (rope_plan
    makes one; a model keeps it)."""
    turns: "torch.Tensor"            # int64 [d_rot / 2]: 64-bit turn fractions
    axis: Optional["torch.Tensor"]   # uint8 [d_rot / 2], or None: one axis
    d_rot: int
    n_axes: int
    pairing: str                     # "half" | "adjacent"

    def __post_init__(self):
        import torch
        _need(self.turns, "plan.turns", torch.int64, self.d_rot // 2)
        if self.axis is not None:
            _need(self.axis, "plan.axis", torch.uint8, self.d_rot // 2)
        if self.pairing not in _PAIRINGS:
            raise ValueError(f"pairing must be one of {sorted(_PAIRINGS)}")

    def struct(self, inverse=False):
        return _native.KvdRopePlan(
            self.turns.data_ptr(),
            None if self.axis is None else self.axis.data_ptr(), self.d_rot,
            self.n_axes, _PAIRINGS[self.pairing], 1 if inverse else 0)


_PAIRINGS = {"half": 0, "adjacent": 1}


def rope_axes(d_rot, sections, interleave=False):
    """Axis of each of the d_rot / 2 pairs. ``sections``: pairs per axis,
    summing to d_rot / 2. In order of the axes, or (interleave) the axes in
    turn, each while pairs of its section are left."""
    sections = [int(n) for n in sections]
    if not 1 <= len(sections) <= 4 or min(sections) < 0:
        raise ValueError("sections: 1 to 4 counts of pairs")
    if sum(sections) * 2 != d_rot:
        raise ValueError(f"sections {sections} do not sum to d_rot / 2 = "
                         f"{d_rot / 2}")
    if not interleave:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, axes = list(sections), []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                axes.append(a)
    return axes


def rope_plan(d_rot, theta=10000.0, sections=None, interleave=False,
              pairing="half", freqs=None, device=None):
    """A RopePlan: pair i turns by theta^(-2 i / d_rot) radians a position,
    or by ``freqs[i]`` (d_rot / 2 Python floats or a float64 tensor; scaled
    frequencies for long contexts go in here). ``sections`` and
    ``interleave`` give the pairs' axes (rope_axes); None: one axis.
    ``pairing``: "half" (channels i and i + d_rot / 2) or "adjacent"
    (channels 2 i and 2 i + 1)."""
    import numpy as np
    import torch
    d_rot = int(d_rot)
    if d_rot < 2 or d_rot % 2:
        raise ValueError(f"d_rot must be even and positive, got {d_rot}")
    if pairing not in _PAIRINGS:
        raise ValueError(f"pairing must be one of {sorted(_PAIRINGS)}")
    if freqs is None:
        f = [float(theta) ** (-2.0 * i / d_rot) for i in range(d_rot // 2)]
    else:
        f = [float(x) for x in freqs]
        if len(f) != d_rot // 2:
            raise ValueError(f"freqs must have {d_rot // 2} entries")
    f = np.array(f, dtype=np.float64)
    turns = np.empty(d_rot // 2, dtype=np.uint64)
    check(lib().kvd_rope_turns(f.ctypes.data, f.size, turns.ctypes.data))
    device = torch.device("cuda" if device is None else device)
    axis = None
    n_axes = 1
    if sections is not None:
        axes = rope_axes(d_rot, sections, interleave)
        n_axes = len(sections)
        axis = torch.tensor(axes, dtype=torch.uint8, device=device)
    return RopePlan(torch.from_numpy(turns.view(np.int64)).to(device), axis,
                    d_rot, n_axes, pairing)


def _positions(plan, positions, rows):
    """positions int32 [n_axes][rows] ([rows] for one axis), contiguous."""
    import torch
    _need(positions, "positions", torch.int32, plan.n_axes * rows)
    if positions.dim() > 2 or positions.shape[-1] != rows:
        raise ValueError(f"positions must be [{plan.n_axes}][{rows}]")
    return positions


@_in_context
def rope(plan, positions, q, k=None, q_out=None, k_out=None, inverse=False):
    """Rotate q [rows][n_h][d] (and k [rows][n_kv][d]) bf16 to positions
    int32 [n_axes][rows]: returns (q_out, k_out). Any strides with
    contiguous vectors; q_out=q rotates in place. ``inverse`` turns back
    (also the gradient of a rotation). ``stream``: as for the other calls."""
    qs = _rows3(q, "q")
    ks = None if k is None else _rows3(k, "k", width=q.shape[2])
    if k_out is not None and k is None:
        raise ValueError("k_out without k")
    r = plan.struct(inverse)
    rows = qs.rows
    _positions(plan, positions, rows)
    dev = _one_device(q, k, q_out, k_out, positions, plan.turns, plan.axis)

    def launch(s, q_out=q_out, k_out=k_out):
        q_out, qo = _out_rows(q_out, q, qs, "q_out")
        ko = None
        if ks is not None:
            k_out, ko = _out_rows(k_out, k, ks, "k_out")
        check(lib().kvd_rope(r, positions.data_ptr(), rows, q.shape[2], qs,
                             qo, ks, ko, s))
        return q_out, k_out
    return dev, launch


def _ragged(cache, block_table, start, row_start):
    import torch
    _need(block_table, "block_table", torch.int32)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [batch][max_blocks_per_seq]")
    B = block_table.shape[0]
    _need(start, "start", torch.int32, B)
    _need(row_start, "row_start", torch.int32, B + 1)
    return B


@_in_context
def kv_write(cache, block_table, start, row_start, k_new, v_new=None,
             rope=None, positions=None, q=None, q_out=None):
    """Write ragged new rows k_new (and v_new) [rows][n_kv][head_dim] bf16
    into the cache: rows row_start[b] .. row_start[b + 1] - 1 go to positions
    start[b] .. of sequence b. With ``rope`` (a RopePlan) and ``positions``
    the keys are rotated on the way, and so is q [rows][n_h][head_dim] if
    given: returns q_out (None without q; q_out=q rotates in place). Rows of
    a new q_out that no sequence owns are not initialised. With a row_start
    that descends nothing is done; it is flagged, as is a sequence that the
    rows do not hold (device_error(): DEVERR_LEN; so for the other calls)."""
    c = cache.struct()
    B = _ragged(cache, block_table, start, row_start)
    ks = _rows3(k_new, "k_new", cache.n_kv, cache.head_dim)
    vs = None
    if v_new is not None:
        vs = _rows3(v_new, "v_new", cache.n_kv, cache.head_dim)
    qs = r = None
    if rope is not None:
        r = rope.struct()
        _positions(rope, positions, ks.rows)
    elif q is not None or q_out is not None or positions is not None:
        raise ValueError("q and positions need rope")
    if q is not None:
        qs = _rows3(q, "q", width=cache.head_dim)
    elif q_out is not None:
        raise ValueError("q_out without q")
    dev = _one_device(cache.k, cache.v, block_table, start, row_start, k_new,
                      v_new, positions, q, q_out,
                      rope and rope.turns, rope and rope.axis,
                      cache.k_inv_scale, cache.v_inv_scale)

    def launch(s, q_out=q_out):
        qo = None
        if qs is not None:
            q_out, qo = _out_rows(q_out, q, qs, "q_out")
        check(lib().kvd_kv_write(
            c, block_table.data_ptr(), block_table.shape[1], start.data_ptr(),
            row_start.data_ptr(), B, ks, vs, r,
            None if positions is None else positions.data_ptr(), ks.rows, qs,
            qo, s))
        return q_out
    return dev, launch


@_in_context
def kv_read(cache, block_table, start, row_start, rows, k_out=None,
            v_out=None):
    """Read positions start[b] .. of every sequence back as bf16 rows
    row_start[b] .. row_start[b + 1] - 1: returns (k, v) [rows][n_kv]
    [head_dim] (v None for a K-only cache). ``rows``: rows of the outputs;
    outputs passed in may have any strides with contiguous vectors. Rows of
    new outputs that no sequence owns are not initialised."""
    import torch
    c = cache.struct()
    B = _ragged(cache, block_table, start, row_start)
    if cache.v is None and v_out is not None:
        raise ValueError("v_out for a K-only cache")
    dev = _one_device(cache.k, cache.v, block_table, start, row_start, k_out,
                      v_out, cache.k_scale, cache.v_scale)
    shape = (int(rows), cache.n_kv, cache.head_dim)

    def launch(s, k_out=k_out, v_out=v_out):
        if k_out is None:
            k_out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
        if v_out is None and cache.v is not None:
            v_out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
        ks = _rows3(k_out, "k_out", shape[1], shape[2])
        vs = None if v_out is None else _rows3(v_out, "v_out", shape[1],
                                               shape[2])
        if ks.rows != shape[0] or (vs is not None and vs.rows != shape[0]):
            raise ValueError(f"outputs must have {shape[0]} rows")
        check(lib().kvd_kv_read(
            c, block_table.data_ptr(), block_table.shape[1], start.data_ptr(),
            row_start.data_ptr(), B, ks, vs, s))
        return k_out, v_out
    return dev, launch


def extend_workspace_size(cache, block_table, seq_lens, max_seq_len, rows,
                          n_h, max_rows=None, window=0):
    """Workspace bytes of a gqa_extend call (kvd_extend_workspace_size) with
    these arguments; without ``max_rows``, enough for a call without it, with
    row_start or not."""
    import torch
    c = cache.struct()
    s = _seqs(block_table, seq_lens, max_seq_len, window=window)
    rows = int(rows)
    bounds = [int(max_rows)] if max_rows is not None else [rows]
    if max_rows is None and rows == s.batch:
        bounds.append(1)
    most = 0
    with torch.cuda.device(block_table.device):
        for bound in bounds:
            out = ctypes.c_size_t(0)
            check(lib().kvd_extend_workspace_size(
                ctypes.byref(c), ctypes.byref(s), rows, bound, n_h,
                ctypes.byref(out)))
            most = max(most, out.value)
    return most


@_in_context
def gqa_extend(cache, block_table, seq_lens, max_seq_len, q, row_start=None,
               max_rows=None, scale=None, out=None, lse=None, workspace=None,
               want_lse=True, window=0, window_start=None):
    """Attention of new tokens over an MXFP4 cache that holds them: q
    [rows][n_h][head_dim] bf16 (contiguous vectors) -> (out [rows][n_h]
    [head_dim] bf16, lse [rows][n_h] fp32). Rows row_start[b] ..
    row_start[b + 1] - 1 (int32 [batch + 1]) are the last positions of
    sequence b, at most ``max_rows`` of them (it chooses the kernel: the
    smallest bound is the fastest; None: all rows, which fits any list);
    without row_start row b is sequence b's one new token. Each row attends to the positions up to its
    own, within ``window`` and from ``window_start`` if given. ``out`` must not
    overlap q. Rows of new outputs that no sequence owns are not
    initialised."""
    import torch
    d = cache.head_dim
    qs = _rows3(q, "q", width=d)
    c = cache.struct()
    seqs = _seqs(block_table, seq_lens, max_seq_len, 0, window, window_start)
    rows, n_h = qs.rows, qs.heads
    if max_rows is None:
        max_rows = 1 if row_start is None else rows
    max_rows = int(max_rows)
    if row_start is not None:
        _need(row_start, "row_start", torch.int32, seqs.batch + 1)
    if out is not None:
        _need(out, "out", torch.bfloat16, rows * n_h * d)
    if lse is not None:
        _need(lse, "lse", torch.float32, rows * n_h)
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8)
    dev = _one_device(q, cache.k, cache.v, block_table, seq_lens, row_start,
                      window_start, out, lse, workspace)

    def launch(s, out=out, lse=lse, workspace=workspace):
        L = lib()
        if out is None:
            out = torch.empty((rows, n_h, d), dtype=torch.bfloat16,
                              device=dev)
        if lse is None and want_lse:
            lse = torch.empty((rows, n_h), dtype=torch.float32, device=dev)
        if workspace is not None:
            nbytes = workspace.numel()
        else:
            need = ctypes.c_size_t(0)
            check(L.kvd_extend_workspace_size(c, seqs, rows, max_rows, n_h,
                                              need))
            nbytes = need.value
            if nbytes:
                # every partial a call keeps here is written before it is read
                workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        check(L.kvd_gqa_extend(
            c, seqs, None if row_start is None else row_start.data_ptr(),
            max_rows, qs, float(scale or 0.0), out.data_ptr(),
            None if lse is None else lse.data_ptr(),
            None if workspace is None else workspace.data_ptr(), nbytes, s))
        return out, lse
    return dev, launch


class BlockPool:
    """The library's copy-on-write block pool (kvd_block_pool_*): host
    reference counts of num_blocks physical blocks. Block tables and id
    lists are host numpy int32 arrays."""

    def __init__(self, num_blocks):
        h = ctypes.c_void_p()
        check(lib().kvd_block_pool_create(int(num_blocks), ctypes.byref(h)))
        self._h = h

    def close(self):
        if self._h:
            lib().kvd_block_pool_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @staticmethod
    def _ids(blocks):
        import numpy as np
        a = np.ascontiguousarray(blocks, dtype=np.int32)
        return a, a.ctypes.data

    def free_count(self):
        return int(lib().kvd_block_pool_free_count(self._h))

    def refcount(self, block):
        return int(lib().kvd_block_pool_refcount(self._h, int(block)))

    def alloc(self, n):
        import numpy as np
        out = np.empty(int(n), dtype=np.int32)
        check(lib().kvd_block_pool_alloc(self._h, int(n), out.ctypes.data))
        return out

    def share(self, blocks):
        a, p = self._ids(blocks)
        check(lib().kvd_block_pool_share(self._h, p, a.size))

    def release(self, blocks):
        a, p = self._ids(blocks)
        check(lib().kvd_block_pool_release(self._h, p, a.size))

    def prepare_append(self, block_table, pos, block_size):
        """block_table: host int32 [batch][max_blocks], updated in place;
        pos: host int32 [batch]. Returns (src, dst) block ids of the copies
        to make before appending."""
        import numpy as np
        assert block_table.dtype == np.int32 and block_table.flags.c_contiguous
        pos = np.ascontiguousarray(pos, dtype=np.int32)
        B, M = block_table.shape
        src = np.empty(max(B, 1), dtype=np.int32)
        dst = np.empty(max(B, 1), dtype=np.int32)
        n = ctypes.c_int32(0)
        check(lib().kvd_block_pool_prepare_append(
            self._h, block_table.ctypes.data, B, M, pos.ctypes.data,
            int(block_size), src.ctypes.data, dst.ctypes.data,
            ctypes.byref(n)))
        return src[:n.value].copy(), dst[:n.value].copy()


def copy_blocks(cache, src, dst, stream=None):
    """Whole blocks dst[i] := src[i] of the cache's K and V (device int32
    tensors)."""
    import torch
    _need(src, "src", torch.int32)
    _need(dst, "dst", torch.int32, src.numel())
    c = cache.struct()
    check(lib().kvd_copy_blocks(ctypes.byref(c), _ptr(src), _ptr(dst),
                                src.numel(), _stream(stream)))


def bytes_per_token(n_l, n_kv, d_h, elem_bytes):
    return int(lib().kvd_bytes_per_token(n_l, n_kv, d_h, elem_bytes))


# device error bits (KVD_DEVERR_* in kvd.h)
DEVERR_BLOCK, DEVERR_POS, DEVERR_TIMEOUT, DEVERR_INDEX, DEVERR_LEN = (
    1, 2, 4, 8, 16)


def set_tuning(decode_ctas=0, mla_cuda_cores=False):
    """Process-wide launch overrides (kvd_set_tuning): decode_ctas > 0
    forces the CTAs of every decode launch; mla_cuda_cores runs the latent
    decode on its CUDA-core kernel."""
    check(lib().kvd_set_tuning(int(decode_ctas), int(bool(mla_cuda_cores))))


def launch_count():
    """Kernels the library has launched in this process (a launch captured
    into a CUDA graph counts once, when captured)."""
    return int(lib().kvd_launch_count())


def device_error():
    """Synchronise, then read and clear the device error word."""
    code = ctypes.c_int32(0)
    check(lib().kvd_device_error(ctypes.byref(code)))
    return code.value
