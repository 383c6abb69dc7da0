"""PyTorch-facing wrappers of libspava's answering side (include/spava.h): norm
and rotation of queries and keys, the paged key-value cache, attention of one
new token.

Argument marshalling only, as in ``api``: shapes, dtypes and devices are
checked, pointers and the current CUDA stream of the tensors' device are handed
to the library.  The calls of a decode step do this in compiled code
(csrc/calls.cpp), as their host time is most of their cost.  Nothing here
synchronises (but ``device_status``), and every call can be captured into a CUDA
graph.  Inference only: no gradients.
"""
from __future__ import annotations

import ctypes
import functools
from dataclasses import dataclass

import torch

from . import native
from .native import SpavaCacheConfig, SpavaRopeConfig

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


def _check(t, shape, dtype, index, name):
    if t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous() or t.get_device() != index:
        raise ValueError(f"{name}: expected contiguous {dtype} {shape} on cuda:{index}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device} contiguous={t.is_contiguous()}")


def _bind(device):
    device = torch.device(device)
    if device.type != "cuda":
        raise ValueError(f"expected a CUDA device, got {device}")
    return torch.device("cuda", torch.cuda.current_device() if device.index is None else device.index)


def _failed(name, status):
    raise native.SpavaError(name, status, native.load().spava_last_cuda_error() if status == 5 else 0)


@functools.cache
def _load_calls():
    """The compiled calls; loaded at first use, as the package that builds them must import without."""
    try:
        from . import _calls
    except ImportError as e:
        raise ImportError("_calls.so is missing or does not load: build it with "
                          "`python -m sequence_sparse_attention_b200.build`") from e
    _calls.on_failure(_failed)
    return _calls


def _kept(name):
    """A tensor that the compiled calls keep.  Its contents and memory (``.data``) may
    be replaced; another tensor takes another object."""
    return property(lambda self: getattr(self._calls, name), doc=f"``{name}``, read-only.")


class QKNormRope:
    """RMS norm of every query and key head and their rotation, in one launch.
    ``inv_freq``: float32 [rope_dim / 2], radians per position; ``q_weight``,
    ``k_weight``: bf16 [d] (None: ones)."""

    def __init__(self, lay: RopeLayout, inv_freq=None, q_weight=None, k_weight=None, device=None):
        given = next((t for t in (inv_freq, q_weight, k_weight) if t is not None), None)
        self.device = _bind(device if device is not None else "cuda" if given is None else given.device)
        self.lay, self.cfg = lay, lay.c()
        index, half = self.device.index, self.cfg.rope_dim // 2
        if half:
            if inv_freq is None:
                raise ValueError("inv_freq: a rotation needs it")
            _check(inv_freq, (half,), torch.float32, index, "inv_freq")
        for t, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
            if t is not None:
                _check(t, (lay.d,), torch.bfloat16, index, name)
        self._calls = _load_calls().Rope(ctypes.addressof(self.cfg), q_weight, k_weight, inv_freq, index)

    q_weight, k_weight, inv_freq = _kept("q_weight"), _kept("k_weight"), _kept("inv_freq")

    def apply(self, q, k, positions=None, q_out=None, k_out=None):
        """q [rows, Hq, d], k [rows, Hkv, d] (views of one projection are fine),
        positions int32 [axes, rows] -> contiguous q_out, k_out; in place with
        ``q_out=q`` and ``k_out=k`` where those are contiguous."""
        return self._calls.apply(q, k, positions, q_out, k_out)


class PagedCache:
    """Pools and workspace of one layer's paged cache.  Position t of a sequence
    lies in row t % page_size of page ``table[sequence, t // page_size]``;
    ``lens`` counts a sequence's tokens, new ones included.  ``table`` (int32
    [sequences, max_pages]) and ``lens`` (int32 [sequences]) stay on the device.

    Calls that may run at the same time (other streams, graphs replayed side by
    side) need workspaces of their own: ``new_workspace()`` and ``workspace=``.
    Caches of the same heads whose calls follow each other, as those of a model's
    layers do, can share one."""

    def __init__(self, lay: CacheLayout, device="cuda", k_pages=None, v_pages=None, k_exp=None, v_exp=None,
                 workspace=None):
        self.device = _bind(device if k_pages is None else k_pages.device)
        self.lay, self.cfg = lay, lay.c()
        self._ws_bytes = cache_workspace_size(lay)
        index, shape = self.device.index, (lay.n_pages, lay.Hkv, lay.page_size, lay.d)

        def pool(t, shape, dtype, name):
            if t is None:
                return torch.zeros(shape, dtype=torch.uint8 if dtype.itemsize == 1 else dtype,
                                   device=self.device).view(dtype)
            _check(t, shape, dtype, index, name)
            return t

        k_pages = pool(k_pages, shape, lay.dtype, "k_pages")
        v_pages = pool(v_pages, shape, lay.dtype, "v_pages")
        if self.cfg.type == 1:
            k_exp = pool(k_exp, shape[:3], torch.int8, "k_exp")
            v_exp = pool(v_exp, shape[:3], torch.int8, "v_exp")
        elif k_exp is not None or v_exp is not None:
            raise ValueError("k_exp, v_exp: only a torch.float8_e4m3fn cache has them")
        workspace = self.new_workspace() if workspace is None else workspace
        _check(workspace, (workspace.numel(),), torch.uint8, index, "workspace")
        self._calls = _load_calls().Cache(ctypes.addressof(self.cfg), (k_pages, v_pages), (k_exp, v_exp), workspace, index)

    k_pages, v_pages, k_exp, v_exp, workspace = map(_kept, ("k_pages", "v_pages", "k_exp", "v_exp", "workspace"))

    @property
    def tensors(self):
        """The pools: (k_pages, v_pages), and (k_exp, v_exp) of a quantised cache."""
        return (self.k_pages, self.v_pages) if self.k_exp is None else \
            (self.k_pages, self.v_pages, self.k_exp, self.v_exp)

    def new_workspace(self):
        return torch.zeros(self._ws_bytes, dtype=torch.uint8, device=self.device)

    def write(self, k, v, table, lens, workspace=None):
        """k, v [sequences * new, Hkv, d] (views fine): the last ``new`` positions of every sequence."""
        self._calls.write(k, v, table, lens, workspace)

    def append(self, rope: QKNormRope, q, k, v, positions, table, lens, q_out=None, workspace=None):
        """``rope.apply(q, k, positions)`` and ``write`` of its keys and of v, in one
        launch; returns the queries.  ``positions`` are the rotation's, [axes, sequences * new]."""
        return self._calls.append(getattr(rope, "_calls", None), q, k, v, positions, table, lens, q_out, workspace)

    def read(self, table, lens, rows, first=0, k_out=None, v_out=None, workspace=None):
        """Positions [first, first + rows) of every sequence as bf16 [sequences, rows,
        Hkv, d], keys and values; zeros from position lens[b] on."""
        return self._calls.read(table, lens, rows, first, k_out, v_out, workspace)

    def attn(self, q, table, lens, o=None, lse=None, want_lse=True, workspace=None):
        """One query token per sequence, q [sequences, Hq, d], over positions [0,
        lens[b]): o like q, and lse float32 [Hq, sequences] (natural log; -inf and
        o = 0 for a sequence without positions)."""
        return self._calls.attn(q, table, lens, o, lse, want_lse, workspace)

    def device_status(self, workspace=None) -> int:
        """Synchronises, returns and clears the status word: bit 1 is a length
        beyond its table or a page outside the pool (0 = clean).  Raises where
        the word cannot be read."""
        ws = self.workspace if workspace is None else workspace
        _check(ws, (ws.numel(),), torch.uint8, self.device.index, "workspace")
        with torch.cuda.device(self.device):
            return native.device_status(ws, torch.cuda.current_stream(self.device).cuda_stream)
