"""PyTorch-facing wrappers of libspava's answering side (include/spava.h): norm
and rotation of queries and keys, the paged key-value cache, attention of one
new token.

Argument marshalling only, as in ``api``: shapes, dtypes and devices are
checked, pointers and the current CUDA stream of the tensors' device are handed
to the library.  Nothing here synchronises (but ``device_status``), and every
call can be captured into a CUDA graph.  Inference only: no gradients.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import native
from .native import SpavaCacheBatch, SpavaCacheConfig, SpavaCachePools, SpavaRopeConfig

_CACHE_TYPES = {torch.bfloat16: 0, torch.float8_e4m3fn: 1}


@dataclass
class RopeLayout:
    """Heads and rotation of one layer's queries and keys.  ``rope_dim``
    elements of each head turn (None: all); ``sections`` deals their pairs out
    to the position axes ((): one axis)."""
    Hq: int
    Hkv: int
    d: int
    rope_dim: int | None = None
    interleaved: bool = False
    sections: tuple = ()
    norm: bool = True
    eps: float = 1e-6

    def c(self) -> SpavaRopeConfig:
        rope = self.d if self.rope_dim is None else self.rope_dim
        sections = tuple(self.sections) or (rope // 2,)
        if len(sections) > 4:
            raise ValueError("at most 4 position axes")
        return SpavaRopeConfig(self.Hq, self.Hkv, self.d, rope, int(self.interleaved), len(sections),
                               (ctypes.c_int32 * 4)(*sections), int(self.norm), float(self.eps))


@dataclass
class CacheLayout:
    """A paged cache of one layer: pools [n_pages, Hkv, page_size, d] in
    ``dtype``, torch.bfloat16 or torch.float8_e4m3fn (which has an int8
    exponent for every row besides).  ``scale`` is the softmax scale (0: 1/sqrt(d))."""
    Hq: int
    Hkv: int
    d: int
    page_size: int = 64
    n_pages: int = 1
    dtype: torch.dtype = torch.bfloat16
    scale: float = 0.0

    def c(self) -> SpavaCacheConfig:
        if self.dtype not in _CACHE_TYPES:
            raise ValueError(f"cache dtype {self.dtype}: expected torch.bfloat16 or torch.float8_e4m3fn")
        return SpavaCacheConfig(self.Hq, self.Hkv, self.d, self.page_size, self.n_pages,
                                _CACHE_TYPES[self.dtype], float(self.scale))


def cache_workspace_size(lay: CacheLayout) -> int:
    n = ctypes.c_size_t()
    cfg = lay.c()
    native.call("spava_cache_workspace_size", ctypes.byref(cfg), ctypes.byref(n))
    return n.value


# A decode step makes these calls many thousand times a second on tensors of a
# few KiB, so a call's host time is most of its cost: the checks below look at
# each property once, and outputs come from empty_like, the cheapest allocation.
_bf16, _f32, _i32 = torch.bfloat16, torch.float32, torch.int32
_empty_like = torch.empty_like


def _check(t, shape, dtype, index, name):
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != index:
        raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)} on cuda:{index}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device} contiguous={t.is_contiguous()}")


def _token_stride(t, rows, heads, d, index, name):
    """Elements between the tokens of a bf16 [rows, heads, d] tensor or view."""
    if t.dtype != _bf16 or t.shape != (rows, heads, d) or t.get_device() != index:
        raise ValueError(f"{name}: expected torch.bfloat16 ({rows}, {heads}, {d}) on cuda:{index}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    token, head, one = t.stride()
    if one != 1 or (head != d and heads > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous, got strides {t.stride()}")
    return token if rows > 1 else heads * d


def _rows(t, name):
    if t.dim() != 3:
        raise ValueError(f"{name}: expected (rows, heads, d), got {tuple(t.shape)}")
    return t.shape[0]


# The raw stream handle without a Stream object (1 us less a call), where torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


class _OnDevice:
    """Calls into the library with the tensors' device current, on its current stream."""

    def _bind(self, device):
        device = torch.device(device)
        if device.type != "cuda":
            raise ValueError(f"expected a CUDA device, got {device}")
        index = torch.cuda.current_device() if device.index is None else device.index
        self.device, self._index = torch.device("cuda", index), index
        self._lib = native.load()

    def _call(self, name, *args):
        index = self._index
        if torch.cuda.current_device() == index:
            rc = getattr(self._lib, name)(*args, _raw_stream(index))
        else:
            with torch.cuda.device(index):
                rc = getattr(self._lib, name)(*args, _raw_stream(index))
        if rc:
            raise native.SpavaError(name, rc, self._lib.spava_last_cuda_error() if rc == 5 else 0)


class QKNormRope(_OnDevice):
    """RMS norm of every query and key head and their rotation, in one launch.
    ``inv_freq``: float32 [rope_dim / 2], radians per position; ``q_weight``,
    ``k_weight``: bf16 [d] (None: ones)."""

    def __init__(self, lay: RopeLayout, inv_freq=None, q_weight=None, k_weight=None, device=None):
        given = next((t for t in (inv_freq, q_weight, k_weight) if t is not None), None)
        self._bind(device if device is not None else "cuda" if given is None else given.device)
        self.lay, self.cfg = lay, lay.c()
        half = self.cfg.rope_dim // 2
        if half:
            if inv_freq is None:
                raise ValueError("inv_freq: a rotation needs it")
            _check(inv_freq, (half,), _f32, self._index, "inv_freq")
        for t, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
            if t is not None:
                _check(t, (lay.d,), _bf16, self._index, name)
        self.inv_freq, self.q_weight, self.k_weight = inv_freq, q_weight, k_weight
        self._cfg = ctypes.byref(self.cfg)
        self._axes = self.cfg.n_axes if half else 0
        self._tables = tuple(None if t is None else t.data_ptr() for t in (q_weight, k_weight, inv_freq))

    def _positions(self, positions, rows):
        axes = self._axes
        if not axes:
            return None
        if positions is None:
            raise ValueError("positions: a rotation needs them")
        if positions.dtype != _i32 or not positions.is_contiguous() or positions.get_device() != self._index or \
                (positions.shape != (axes, rows) and (axes > 1 or positions.shape != (rows,))):
            raise ValueError(f"positions: expected contiguous torch.int32 ({axes}, {rows}) on "
                             f"{self.device}, got {positions.dtype} {tuple(positions.shape)} on {positions.device}")
        return positions.data_ptr()

    def apply(self, q, k, positions=None, q_out=None, k_out=None):
        """q [rows, Hq, d], k [rows, Hkv, d] (views of one projection are fine),
        positions int32 [axes, rows] -> contiguous q_out, k_out; in place with
        ``q_out=q`` and ``k_out=k`` where those are contiguous."""
        lay, index, rows = self.lay, self._index, _rows(q, "q")
        qs = _token_stride(q, rows, lay.Hq, lay.d, index, "q")
        ks = _token_stride(k, rows, lay.Hkv, lay.d, index, "k")
        if q_out is None:
            q_out = _empty_like(q, memory_format=torch.contiguous_format)
        else:
            _check(q_out, q.shape, _bf16, index, "q_out")
        if k_out is None:
            k_out = _empty_like(k, memory_format=torch.contiguous_format)
        else:
            _check(k_out, k.shape, _bf16, index, "k_out")
        self._call("spava_qk_norm_rope", self._cfg, rows, q.data_ptr(), qs, k.data_ptr(), ks, *self._tables,
                   self._positions(positions, rows), q_out.data_ptr(), k_out.data_ptr())
        return q_out, k_out


class PagedCache(_OnDevice):
    """Pools and workspace of one layer's paged cache.  Position t of a sequence
    lies in row t % page_size of page ``table[sequence, t // page_size]``;
    ``lens`` counts a sequence's tokens, new ones included.  ``table`` (int32
    [sequences, max_pages]) and ``lens`` (int32 [sequences]) stay on the device.

    Calls that may run at the same time (other streams, graphs replayed side by
    side) need workspaces of their own: ``new_workspace()`` and ``workspace=``."""

    def __init__(self, lay: CacheLayout, device="cuda", k_pages=None, v_pages=None, k_exp=None, v_exp=None,
                 workspace=None):
        self._bind(device if k_pages is None else k_pages.device)
        self.lay, self.cfg = lay, lay.c()
        self._ws_bytes = cache_workspace_size(lay)
        shape = (lay.n_pages, lay.Hkv, lay.page_size, lay.d)

        def pool(t, shape, dtype, name):
            if t is None:
                return torch.zeros(shape, dtype=torch.uint8 if dtype.itemsize == 1 else dtype,
                                   device=self.device).view(dtype)
            _check(t, shape, dtype, self._index, name)
            return t

        self.k_pages = pool(k_pages, shape, lay.dtype, "k_pages")
        self.v_pages = pool(v_pages, shape, lay.dtype, "v_pages")
        self.k_exp = self.v_exp = None
        if self.cfg.type == 1:
            self.k_exp = pool(k_exp, shape[:3], torch.int8, "k_exp")
            self.v_exp = pool(v_exp, shape[:3], torch.int8, "v_exp")
        elif k_exp is not None or v_exp is not None:
            raise ValueError("k_exp, v_exp: only a torch.float8_e4m3fn cache has them")
        self.workspace = self.new_workspace() if workspace is None else workspace
        self._pools = SpavaCachePools(*(None if t is None else t.data_ptr()
                                        for t in (self.k_pages, self.v_pages, self.k_exp, self.v_exp)))
        self._head = (ctypes.byref(self.cfg), ctypes.byref(self._pools))
        self._own_ws = self._check_ws(self.workspace)
        self._lse_of = torch.empty((lay.Hq, 1), dtype=_f32, device=self.device)

    @property
    def tensors(self):
        """The pools: (k_pages, v_pages), and (k_exp, v_exp) of a quantised cache."""
        return (self.k_pages, self.v_pages) if self.k_exp is None else \
            (self.k_pages, self.v_pages, self.k_exp, self.v_exp)

    def new_workspace(self):
        return torch.zeros(self._ws_bytes, dtype=torch.uint8, device=self.device)

    def _check_ws(self, ws):
        if ws.dtype != torch.uint8 or ws.get_device() != self._index or not ws.is_contiguous():
            raise ValueError(f"workspace: expected contiguous torch.uint8 on {self.device}")
        return ws.data_ptr(), ws.numel()

    def _ws(self, workspace):
        return self._own_ws if workspace is None else self._check_ws(workspace)

    def _batch(self, table, lens):
        if lens.dtype == _i32 and table.dtype == _i32 and lens.dim() == 1 and table.dim() == 2 and \
                lens.is_contiguous() and table.is_contiguous() and \
                lens.get_device() == self._index == table.get_device():
            n, pages = table.shape
            if lens.shape[0] == n:
                return n, ctypes.byref(SpavaCacheBatch(n, pages, table.data_ptr(), lens.data_ptr()))
        raise ValueError(f"table, lens: expected contiguous torch.int32 (sequences, max_pages) and (sequences,) "
                         f"on {self.device}, got {table.dtype} {tuple(table.shape)} on {table.device} and "
                         f"{lens.dtype} {tuple(lens.shape)} on {lens.device}")

    @staticmethod
    def _new_rows(rows, n, name):
        if n == 0 and rows == 0:
            return 0
        if n == 0 or rows % n:
            raise ValueError(f"{name}: {rows} rows for {n} sequences: expected as many for each")
        return rows // n

    def write(self, k, v, table, lens, workspace=None):
        """k, v [sequences * new, Hkv, d] (views fine): the last ``new`` positions of every sequence."""
        lay, index, (n, batch), rows = self.lay, self._index, self._batch(table, lens), _rows(k, "k")
        ks = _token_stride(k, rows, lay.Hkv, lay.d, index, "k")
        vs = _token_stride(v, rows, lay.Hkv, lay.d, index, "v")
        self._call("spava_cache_write", *self._head, batch, self._new_rows(rows, n, "k"), k.data_ptr(), ks,
                   v.data_ptr(), vs, *self._ws(workspace))

    def append(self, rope: QKNormRope, q, k, v, positions, table, lens, q_out=None, workspace=None):
        """``rope.apply(q, k, positions)`` and ``write`` of its keys and of v, in one
        launch; returns the queries.  ``positions`` are the rotation's, [axes, sequences * new]."""
        lay, index, (n, batch), rows = self.lay, self._index, self._batch(table, lens), _rows(q, "q")
        if rope._index != index:
            raise ValueError(f"rope: expected on {self.device}, is on {rope.device}")
        qs = _token_stride(q, rows, lay.Hq, lay.d, index, "q")
        ks = _token_stride(k, rows, lay.Hkv, lay.d, index, "k")
        vs = _token_stride(v, rows, lay.Hkv, lay.d, index, "v")
        if q_out is None:
            q_out = _empty_like(q, memory_format=torch.contiguous_format)
        else:
            _check(q_out, q.shape, _bf16, index, "q_out")
        self._call("spava_cache_append", rope._cfg, *self._head, batch, self._new_rows(rows, n, "q"),
                   q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, *rope._tables,
                   rope._positions(positions, rows), q_out.data_ptr(), *self._ws(workspace))
        return q_out

    def read(self, table, lens, rows, first=0, k_out=None, v_out=None, workspace=None):
        """Positions [first, first + rows) of every sequence as bf16 [sequences, rows,
        Hkv, d], keys and values; zeros from position lens[b] on."""
        lay, (n, batch) = self.lay, self._batch(table, lens)
        shape = (n, rows, lay.Hkv, lay.d)
        if k_out is None:
            k_out = torch.empty(shape, dtype=_bf16, device=self.device)
        else:
            _check(k_out, shape, _bf16, self._index, "k_out")
        if v_out is None:
            v_out = _empty_like(k_out)
        else:
            _check(v_out, shape, _bf16, self._index, "v_out")
        self._call("spava_cache_read", *self._head, batch, first, rows, k_out.data_ptr(), v_out.data_ptr(),
                   *self._ws(workspace))
        return k_out, v_out

    def attn(self, q, table, lens, o=None, lse=None, want_lse=True, workspace=None):
        """One query token per sequence, q [sequences, Hq, d], over positions [0,
        lens[b]): o like q, and lse float32 [Hq, sequences] (natural log; -inf and
        o = 0 for a sequence without positions)."""
        lay, (n, batch) = self.lay, self._batch(table, lens)
        _check(q, (n, lay.Hq, lay.d), _bf16, self._index, "q")
        if o is None:
            o = _empty_like(q)
        else:
            _check(o, q.shape, _bf16, self._index, "o")
        if lse is not None:
            _check(lse, (lay.Hq, n), _f32, self._index, "lse")
        elif want_lse:
            like = self._lse_of  # of the last batch size; a local, as other threads may change it
            if like.shape[1] != n:
                self._lse_of = like = torch.empty((lay.Hq, n), dtype=_f32, device=self.device)
            lse = _empty_like(like)
        self._call("spava_cache_attn", *self._head, batch, q.data_ptr(), o.data_ptr(),
                   None if lse is None else lse.data_ptr(), *self._ws(workspace))
        return o, lse

    def device_status(self, workspace=None) -> int:
        """Synchronises, returns and clears the status word: bit 1 is a length
        beyond its table or a page outside the pool (0 = clean)."""
        flags = ctypes.c_int32()
        ptr, size = self._ws(workspace)
        with torch.cuda.device(self._index):
            native.load().spava_device_status(ptr, size, torch.cuda.current_stream(self._index).cuda_stream,
                                              ctypes.byref(flags))
        return flags.value
