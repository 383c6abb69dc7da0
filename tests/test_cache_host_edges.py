"""The answering side's Python calls on the host: what they refuse before any
work, and what they must not do to the process."""
import ctypes

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from sequence_sparse_attention_b200 import CacheLayout, PagedCache, QKNormRope, RopeLayout, Spava, native
from sequence_sparse_attention_b200.cache import _load_calls


# ------------------------------------------------------------------ tensors without memory
@pytest.mark.parametrize("transform", ["vmap", "grad", "none"])
def test_tensors_without_memory_are_refused(transform):
    """Inside torch.func's transforms a tensor has no address to take, nor has one
    of a FakeTensorMode: the call raises (and does not end the process), before it
    looks for a device."""
    cfg = RopeLayout(4, 2, 64).c()
    rope = _load_calls().Rope(ctypes.addressof(cfg), 0, 0, 0, 0)
    with FakeTensorMode():
        q, k, qo, ko = (torch.empty(2, h, 64, dtype=torch.bfloat16, device="cuda:0") for h in (4, 2, 4, 2))
        pos = torch.empty(1, 2, dtype=torch.int32, device="cuda:0")
        with pytest.raises((RuntimeError, ValueError), match="data pointer|storage|memory"):
            if transform == "vmap":
                torch.vmap(lambda x: rope.apply(x, k, pos, qo, ko))(torch.stack([q] * 3))
            elif transform == "grad":
                torch.func.grad(lambda x: rope.apply(x, k, pos, qo, ko)[0].float().sum())(q)
            else:
                rope.apply(q, k, pos, qo, ko)


# ------------------------------------------------------------------ kept tensors
def test_kept_tensors_are_read_only():
    """Another tensor in an attribute would not reach the calls: it is refused."""
    for cls, names in ((QKNormRope, ("q_weight", "k_weight", "inv_freq")),
                       (PagedCache, ("k_pages", "v_pages", "k_exp", "v_exp", "workspace"))):
        for name in names:
            assert isinstance(getattr(cls, name, None), property) and getattr(cls, name).fset is None


def test_compiled_calls_keep_tensors_not_addresses():
    """What a call uses is the tensor as it is then: one whose memory was replaced
    by another type, shape or device is refused, before any device is looked for."""
    calls = _load_calls()
    cfg = RopeLayout(4, 2, 64).c()
    with FakeTensorMode():
        def cuda(*shape, dtype=torch.bfloat16):
            return torch.empty(shape, dtype=dtype, device="cuda:0")

        w, f = cuda(64), cuda(32, dtype=torch.float32)
        rope = calls.Rope(ctypes.addressof(cfg), w, None, f, 0)
        assert rope.q_weight is w and rope.k_weight is None and rope.inv_freq is f
        with pytest.raises(AttributeError):
            rope.q_weight = w
    for bad in (1, "x"):
        with pytest.raises(ValueError):
            calls.Rope(ctypes.addressof(cfg), bad, None, None, 0)
    lay = CacheLayout(4, 2, 64, page_size=16, n_pages=8).c()
    k = torch.zeros(8, 2, 16, 64)
    with pytest.raises(ValueError):
        calls.Cache(ctypes.addressof(lay), (k,), (None, None), k, 0)
    cache = calls.Cache(ctypes.addressof(lay), (k, k), (None, None), None, 0)
    assert cache.k_pages is k and cache.k_exp is None and cache.workspace is None
    # the objects give their references back, also in a circle
    import gc
    import sys
    import weakref
    held = sys.getrefcount(k)
    k.owner = cache
    del cache, k.owner
    gc.collect()
    assert sys.getrefcount(k) == held - 2
    cache = calls.Cache(ctypes.addressof(lay), (k, k), (None, None), None, 0)
    k.owner = cache
    ref = weakref.ref(k)
    del k, cache
    gc.collect()
    assert ref() is None


# ------------------------------------------------------------------ empty batches
def test_an_empty_batch_needs_no_addresses():
    """Tensors without elements have none."""
    lib = native.load()
    buf = ctypes.create_string_buffer(4096)
    at = (ctypes.addressof(buf) + 255) // 256 * 256      # never dereferenced on these paths
    lay = CacheLayout(4, 2, 64, page_size=16, n_pages=8).c()
    rope = RopeLayout(4, 2, 64).c()
    pools = native.SpavaCachePools(at, at, None, None)
    end = (at, 1 << 40, None)

    def calls(batch, rows=1):
        h = ctypes.byref(lay), ctypes.byref(pools), ctypes.byref(batch)
        return [lib.spava_cache_write(*h, rows, None, 128, None, 128, *end),
                lib.spava_cache_append(ctypes.byref(rope), *h, rows, None, 256, None, 128, None, 128, None, None, None, None,
                                       None, *end),
                lib.spava_cache_read(*h, 0, rows, None, None, *end), lib.spava_cache_attn(*h, None, None, None, *end)]

    assert calls(native.SpavaCacheBatch(0, 3, None, None)) == [0] * 4
    assert calls(native.SpavaCacheBatch(0, 3, None, None), rows=0) == [0] * 4
    # the rest of the arguments are looked at all the same
    assert calls(native.SpavaCacheBatch(0, 0, None, None)) == [1] * 4
    assert calls(native.SpavaCacheBatch(2, 3, None, at)) == [1] * 4
    assert calls(native.SpavaCacheBatch(2, 3, at, None)) == [1] * 4


# ------------------------------------------------------------------ the status word
@pytest.mark.parametrize("status,flags,want", [(0, 0, 0), (1, 2, 2), (6, 1, 1), (6, 3, 3), (5, 0, None), (1, 0, None)])
def test_a_status_that_cannot_be_read_raises(monkeypatch, status, flags, want):
    """A workspace that is too short or a CUDA error is not a clean status word."""
    import contextlib
    import types

    class Lib:
        def spava_device_status(self, ws, size, stream, to):
            to._obj.value = flags
            return status

        def spava_last_cuda_error(self):
            return 700

        def spava_status_string(self, s):
            return b"a status"

    monkeypatch.setattr(native, "load", lambda: Lib())
    stream = types.SimpleNamespace(cuda_stream=0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: stream)
    monkeypatch.setattr(torch.cuda, "device", lambda *a: contextlib.nullcontext())
    ws = torch.zeros(256, dtype=torch.uint8)
    device = types.SimpleNamespace(index=-1)
    for read in (lambda: PagedCache.device_status(types.SimpleNamespace(workspace=ws, device=device)),
                 lambda: PagedCache.device_status(types.SimpleNamespace(workspace=None, device=device), workspace=ws),
                 lambda: Spava.device_status(types.SimpleNamespace(ws=ws, device=device))):
        if want is not None:
            assert read() == want
            continue
        with pytest.raises(native.SpavaError) as e:
            read()
        assert e.value.status == status and e.value.cuda_error == (700 if status == 5 else 0)


# ------------------------------------------------------------------ errors of the runtime
def test_a_refused_call_leaves_no_error_behind(tmp_path):
    """The runtime remembers a call's error until it is asked: left there, the next
    launch that is checked by asking would report it as its own.  The helpers are
    compiled with a runtime of four lines."""
    import os
    import subprocess

    from sequence_sparse_attention_b200 import build
    (tmp_path / "t.cpp").write_text(r'''
#include "status.cuh"
static cudaError_t pending = cudaSuccess;
extern "C" cudaError_t cudaGetLastError() { cudaError_t e = pending; pending = cudaSuccess; return e; }
static cudaError_t refused() { return pending = cudaErrorLaunchOutOfResources; }
static spava_status macro() { SPAVA_CUDA(refused()); return SPAVA_OK; }
int main() {
    using namespace spava;
    if (cuda_ok(refused()) != SPAVA_ERR_CUDA || g_last_cuda_error != cudaErrorLaunchOutOfResources) return 1;
    if (launched() != SPAVA_OK) return 2;   // a launch that was fine
    if (macro() != SPAVA_ERR_CUDA) return 3;
    if (launched() != SPAVA_OK) return 4;
    refused();                              // one that was not
    if (launched() != SPAVA_ERR_CUDA || g_last_cuda_error != cudaErrorLaunchOutOfResources) return 5;
    return launched() == SPAVA_OK ? 0 : 6;
}
''')
    cuda = os.path.dirname(os.path.dirname(build.nvcc()))
    subprocess.check_call(["g++", "-std=c++17", "-I" + os.path.join(cuda, "include"), "-I" + build.CSRC,
                           str(tmp_path / "t.cpp"), "-o", str(tmp_path / "t")])
    assert subprocess.run([str(tmp_path / "t")]).returncode == 0
