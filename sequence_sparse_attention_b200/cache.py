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


def _check(t, shape, dtype, device, name):
    if t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name}: expected contiguous {dtype} {shape} on {device}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device} contiguous={t.is_contiguous()}")


def _token_stride(t, heads, d, device, name):
    """Elements between the tokens of a bf16 [rows, heads, d] tensor or view."""
    shape = t.shape
    if t.dtype != torch.bfloat16 or len(shape) != 3 or shape[1] != heads or shape[2] != d or t.device != device:
        raise ValueError(f"{name}: expected torch.bfloat16 (rows, {heads}, {d}) on {device}, got "
                         f"{t.dtype} {tuple(shape)} on {t.device}")
    stride = t.stride()
    if stride[2] != 1 or (heads > 1 and stride[1] != d):
        raise ValueError(f"{name}: the heads of a token must be contiguous, got strides {stride}")
    return stride[0] if shape[0] > 1 else heads * d


class _OnDevice:
    """Calls into the library with the tensors' device current, on its current stream."""

    def _bind(self, device):
        device = torch.device(device)
        if device.type != "cuda":
            raise ValueError(f"expected a CUDA device, got {device}")
        index = torch.cuda.current_device() if device.index is None else device.index
        self.device, self._index = torch.device("cuda", index), index

    def _call(self, name, *args):
        if torch.cuda.current_device() == self._index:
            native.call(name, *args, torch.cuda.current_stream(self._index).cuda_stream)
        else:
            with torch.cuda.device(self._index):
                native.call(name, *args, torch.cuda.current_stream(self._index).cuda_stream)


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
            _check(inv_freq, (half,), torch.float32, self.device, "inv_freq")
        for t, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
            if t is not None:
                _check(t, (lay.d,), torch.bfloat16, self.device, name)
        self.inv_freq, self.q_weight, self.k_weight = inv_freq, q_weight, k_weight
        self._cfg = ctypes.byref(self.cfg)
        self._tables = tuple(None if t is None else t.data_ptr() for t in (q_weight, k_weight, inv_freq))

    def _positions(self, positions, rows):
        if not self.cfg.rope_dim:
            return None
        if positions.dtype != torch.int32 or not positions.is_contiguous() or positions.device != self.device or \
                positions.numel() != self.cfg.n_axes * rows or positions.shape[-1:] != (rows,):
            raise ValueError(f"positions: expected contiguous torch.int32 ({self.cfg.n_axes}, {rows}) on "
                             f"{self.device}, got {positions.dtype} {tuple(positions.shape)} on {positions.device}")
        return positions.data_ptr()

    def apply(self, q, k, positions=None, q_out=None, k_out=None):
        """q [rows, Hq, d], k [rows, Hkv, d] (views of one projection are fine),
        positions int32 [axes, rows] -> contiguous q_out, k_out; in place with
        ``q_out=q`` and ``k_out=k`` where those are contiguous."""
        lay, rows = self.lay, q.shape[0]
        qs = _token_stride(q, lay.Hq, lay.d, self.device, "q")
        ks = _token_stride(k, lay.Hkv, lay.d, self.device, "k")
        if k.shape[0] != rows:
            raise ValueError(f"k: expected {rows} rows, got {k.shape[0]}")
        if q_out is None:
            q_out = torch.empty((rows, lay.Hq, lay.d), dtype=torch.bfloat16, device=self.device)
        else:
            _check(q_out, (rows, lay.Hq, lay.d), torch.bfloat16, self.device, "q_out")
        if k_out is None:
            k_out = torch.empty((rows, lay.Hkv, lay.d), dtype=torch.bfloat16, device=self.device)
        else:
            _check(k_out, (rows, lay.Hkv, lay.d), torch.bfloat16, self.device, "k_out")
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
            _check(t, shape, dtype, self.device, name)
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

    @property
    def tensors(self):
        """The pools: (k_pages, v_pages), and (k_exp, v_exp) of a quantised cache."""
        return (self.k_pages, self.v_pages) if self.k_exp is None else \
            (self.k_pages, self.v_pages, self.k_exp, self.v_exp)

    def new_workspace(self):
        return torch.zeros(self._ws_bytes, dtype=torch.uint8, device=self.device)

    def _ws(self, workspace):
        ws = self.workspace if workspace is None else workspace
        if ws.dtype != torch.uint8 or ws.device != self.device or not ws.is_contiguous():
            raise ValueError(f"workspace: expected contiguous torch.uint8 on {self.device}")
        return ws.data_ptr(), ws.numel()

    def _batch(self, table, lens):
        n = lens.shape[0] if lens.dim() == 1 else -1
        if table.dtype != torch.int32 or lens.dtype != torch.int32 or n < 0 or table.dim() != 2 or \
                table.shape[0] != n or not table.is_contiguous() or not lens.is_contiguous() or \
                table.device != self.device or lens.device != self.device:
            raise ValueError(f"table, lens: expected contiguous torch.int32 (sequences, max_pages) and (sequences,) "
                             f"on {self.device}, got {table.dtype} {tuple(table.shape)} on {table.device} and "
                             f"{lens.dtype} {tuple(lens.shape)} on {lens.device}")
        return n, ctypes.byref(SpavaCacheBatch(n, table.shape[1], table.data_ptr(), lens.data_ptr()))

    @staticmethod
    def _new_rows(rows, n, name):
        if n == 0 and rows == 0:
            return 0
        if n == 0 or rows % n:
            raise ValueError(f"{name}: {rows} rows for {n} sequences: expected as many for each")
        return rows // n

    def write(self, k, v, table, lens, workspace=None):
        """k, v [sequences * new, Hkv, d] (views fine): the last ``new`` positions of every sequence."""
        lay, (n, batch) = self.lay, self._batch(table, lens)
        ks = _token_stride(k, lay.Hkv, lay.d, self.device, "k")
        vs = _token_stride(v, lay.Hkv, lay.d, self.device, "v")
        if v.shape[0] != k.shape[0]:
            raise ValueError(f"v: expected {k.shape[0]} rows, got {v.shape[0]}")
        self._call("spava_cache_write", *self._head, batch, self._new_rows(k.shape[0], n, "k"), k.data_ptr(), ks,
                   v.data_ptr(), vs, *self._ws(workspace))

    def append(self, rope: QKNormRope, q, k, v, positions, table, lens, q_out=None, workspace=None):
        """``rope.apply(q, k, positions)`` and ``write`` of its keys and of v, in one
        launch; returns the queries.  ``positions`` are the rotation's, [axes, sequences * new]."""
        lay, (n, batch) = self.lay, self._batch(table, lens)
        rows = q.shape[0]
        if rope.device != self.device:
            raise ValueError(f"rope: expected on {self.device}, is on {rope.device}")
        qs = _token_stride(q, lay.Hq, lay.d, self.device, "q")
        ks = _token_stride(k, lay.Hkv, lay.d, self.device, "k")
        vs = _token_stride(v, lay.Hkv, lay.d, self.device, "v")
        if k.shape[0] != rows or v.shape[0] != rows:
            raise ValueError(f"k, v: expected {rows} rows, got {k.shape[0]} and {v.shape[0]}")
        if q_out is None:
            q_out = torch.empty((rows, lay.Hq, lay.d), dtype=torch.bfloat16, device=self.device)
        else:
            _check(q_out, (rows, lay.Hq, lay.d), torch.bfloat16, self.device, "q_out")
        self._call("spava_cache_append", rope._cfg, *self._head, batch, self._new_rows(rows, n, "q"),
                   q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, *rope._tables,
                   rope._positions(positions, rows), q_out.data_ptr(), *self._ws(workspace))
        return q_out

    def read(self, table, lens, rows, first=0, k_out=None, v_out=None, workspace=None):
        """Positions [first, first + rows) of every sequence as bf16 [sequences, rows,
        Hkv, d], keys and values; zeros from position lens[b] on."""
        lay, (n, batch) = self.lay, self._batch(table, lens)
        shape, out = (n, rows, lay.Hkv, lay.d), []
        for t, name in ((k_out, "k_out"), (v_out, "v_out")):
            if t is None:
                t = torch.empty(shape, dtype=torch.bfloat16, device=self.device)
            else:
                _check(t, shape, torch.bfloat16, self.device, name)
            out.append(t)
        self._call("spava_cache_read", *self._head, batch, first, rows, out[0].data_ptr(), out[1].data_ptr(),
                   *self._ws(workspace))
        return tuple(out)

    def attn(self, q, table, lens, o=None, lse=None, want_lse=True, workspace=None):
        """One query token per sequence, q [sequences, Hq, d], over positions [0,
        lens[b]): o like q, and lse float32 [Hq, sequences] (natural log; -inf and
        o = 0 for a sequence without positions)."""
        lay, (n, batch) = self.lay, self._batch(table, lens)
        _check(q, (n, lay.Hq, lay.d), torch.bfloat16, self.device, "q")
        if o is None:
            o = torch.empty_like(q)
        else:
            _check(o, (n, lay.Hq, lay.d), torch.bfloat16, self.device, "o")
        if lse is not None:
            _check(lse, (lay.Hq, n), torch.float32, self.device, "lse")
        elif want_lse:
            lse = torch.empty((lay.Hq, n), dtype=torch.float32, device=self.device)
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
