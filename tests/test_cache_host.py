"""The answering side's C ABI on the host: bad arguments are refused before any
CUDA call (so the statuses come back without a GPU), and workspace sizes hold.
Also the 64-bit row quantiser that the GPU tests compare with, against brute
force."""
import ctypes

import pytest
import torch

from cache_util import E4M3, quantise
from sequence_sparse_attention_b200 import CacheLayout, RopeLayout, native
from sequence_sparse_attention_b200.cache import cache_workspace_size
from sequence_sparse_attention_b200.native import (SpavaCacheBatch, SpavaCachePools, SpavaError)

BUF = ctypes.create_string_buffer(4096)
FAKE = (ctypes.addressof(BUF) + 255) // 256 * 256     # aligned, never dereferenced on these paths
WS = 1 << 40                                          # a workspace size that is always enough


def rope(**kw):
    base = dict(Hq=4, Hkv=2, d=64)
    post = {k: kw.pop(k) for k in list(kw) if k in ("section", "n_axes", "rope_dim", "norm", "interleaved")}
    c = RopeLayout(**{**base, **kw}).c()
    for k, v in post.items():
        setattr(c, k, (ctypes.c_int32 * 4)(*v) if k == "section" else v)
    return c


def call_rope(c, rows=1, q=FAKE, qs=256, k=FAKE, ks=128, qw=FAKE, kw=FAKE, freq=FAKE, pos=FAKE, qo=FAKE, ko=FAKE):
    return native.load().spava_qk_norm_rope(ctypes.byref(c), rows, q, qs, k, ks, qw, kw, freq, pos, qo, ko, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(Hq=3), 1), (dict(Hq=0), 1), (dict(d=96), 2), (dict(d=0), 1), (dict(Hq=8192, Hkv=1), 2),
    (dict(rope_dim=-16), 1), (dict(rope_dim=80), 1), (dict(rope_dim=7), 1), (dict(rope_dim=24), 2),
    (dict(interleaved=2), 1), (dict(norm=2), 1), (dict(n_axes=0), 1), (dict(n_axes=5), 2),
    (dict(section=(31, 0, 0, 0)), 1), (dict(n_axes=2, section=(40, -8, 0, 0)), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
])
def test_rope_config_refused(kw, expect):
    assert call_rope(rope(**kw)) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(rows=-1), 1), (dict(q=None), 1), (dict(k=None), 1), (dict(qo=None), 1), (dict(ko=None), 1),
    (dict(q=FAKE + 2), 3), (dict(ko=FAKE + 8), 3), (dict(qw=FAKE + 4), 3), (dict(freq=None), 1),
    (dict(pos=None), 1), (dict(pos=FAKE + 2), 3), (dict(freq=FAKE + 1), 3), (dict(qs=255), 1),
    (dict(ks=132), 3), (dict(ks=120), 1), (dict(rows=1 << 40), 2), (dict(rows=(1 << 31) // 6 + 1), 2),
])
def test_rope_arguments_refused(kw, expect):
    assert call_rope(rope(), **kw) == expect


def test_rope_no_rows_is_nothing():
    assert call_rope(rope(), rows=0, q=None, k=None, qo=None, ko=None) == 0


def cache(**kw):
    return CacheLayout(**{**dict(Hq=4, Hkv=2, d=64, page_size=16, n_pages=8), **kw})


def batch(n=2, pages=3, table=FAKE, lens=FAKE):
    return SpavaCacheBatch(n, pages, table, lens)


def pools(k=FAKE, v=FAKE, ke=None, ve=None):
    return SpavaCachePools(k, v, ke, ve)


def refs(c, p, b):
    return ctypes.byref(c), ctypes.byref(p), ctypes.byref(b)


def status_of_all(c, p, b, ws=FAKE, ws_bytes=WS):
    """The same refusal by each of the four calls."""
    lib, r = native.load(), None
    h = refs(c, p, b)
    ro = ctypes.byref(rope(Hq=c.n_q_heads if c.n_q_heads > 0 and c.n_kv_heads > 0 and
                           c.n_q_heads % c.n_kv_heads == 0 and c.n_q_heads <= 4096 else 4,
                           Hkv=c.n_kv_heads if c.n_q_heads > 0 and c.n_kv_heads > 0 and
                           c.n_q_heads % c.n_kv_heads == 0 and c.n_q_heads <= 4096 else 2,
                           d=c.head_dim if c.head_dim in (64, 128) else 64))
    got = {
        lib.spava_cache_write(*h, 1, FAKE, 1 << 20, FAKE, 1 << 20, ws, ws_bytes, None),
        lib.spava_cache_append(ro, *h, 1, FAKE, 1 << 20, FAKE, 1 << 20, FAKE, 1 << 20, None, None, FAKE, FAKE, FAKE,
                               ws, ws_bytes, None),
        lib.spava_cache_read(*h, 0, 1, FAKE, FAKE, ws, ws_bytes, None),
        lib.spava_cache_attn(*h, FAKE, FAKE, None, ws, ws_bytes, None),
    }
    assert len(got) == 1, got
    return got.pop()


@pytest.mark.parametrize("kw,expect", [
    (dict(Hq=5), 1), (dict(Hkv=0), 1), (dict(d=80), 2), (dict(page_size=0), 1), (dict(page_size=65537), 2),
    (dict(n_pages=0), 1), (dict(n_pages=1 << 28), 2), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
])
def test_cache_config_refused(kw, expect):
    assert status_of_all(cache(**kw).c(), pools(), batch()) == expect
    with pytest.raises(SpavaError) as e:
        cache_workspace_size(cache(**kw))
    assert e.value.status == expect


def test_cache_type_refused():
    c = cache().c()
    c.type = 7
    assert status_of_all(c, pools(), batch()) == 1
    with pytest.raises(ValueError):
        cache(dtype=torch.float16).c()


@pytest.mark.parametrize("b,expect", [
    (batch(n=-1), 1), (batch(n=1 << 20), 2), (batch(pages=0), 1), (batch(pages=(1 << 31) // 16 + 1), 2),
    (batch(pages=((1 << 31) - (1 << 16)) // 16 + 1), 2),
    (batch(table=None), 1), (batch(lens=None), 1), (batch(table=FAKE + 2), 3), (batch(lens=FAKE + 1), 3),
])
def test_cache_batch_refused(b, expect):
    assert status_of_all(cache().c(), pools(), b) == expect


@pytest.mark.parametrize("p,kw,expect", [
    (pools(k=None), {}, 1), (pools(v=FAKE + 8), {}, 3), (pools(), dict(dtype=E4M3), 1),
    (pools(ke=FAKE), dict(dtype=E4M3), 1), (pools(ke=FAKE, ve=FAKE + 8), dict(dtype=E4M3), 3),
])
def test_cache_pools_refused(p, kw, expect):
    assert status_of_all(cache(**kw).c(), p, batch()) == expect


def test_cache_workspace_refused():
    for kw in ({}, dict(dtype=E4M3), dict(Hq=32)):
        lay = cache(**kw)
        need = cache_workspace_size(lay)
        p = pools(ke=FAKE, ve=FAKE)
        assert status_of_all(lay.c(), p, batch(), ws=None) == 4
        assert status_of_all(lay.c(), p, batch(), ws_bytes=need - 1) == 4
        assert status_of_all(lay.c(), p, batch(), ws=FAKE + 16) == 3


def test_call_arguments_refused():
    lib, h = native.load(), refs(cache().c(), pools(), batch())
    w = (FAKE, WS, None)
    assert lib.spava_cache_write(*h, -1, FAKE, 128, FAKE, 128, *w) == 1
    assert lib.spava_cache_write(*h, 1 << 31, FAKE, 128, FAKE, 128, *w) == 2
    assert lib.spava_cache_write(*h, (1 << 31) // 8 + 1, FAKE, 128, FAKE, 128, *w) == 2
    assert lib.spava_cache_write(*h, 1, None, 128, FAKE, 128, *w) == 1
    assert lib.spava_cache_write(*h, 1, FAKE, 127, FAKE, 128, *w) == 1
    assert lib.spava_cache_write(*h, 1, FAKE, 128, FAKE, 132, *w) == 3
    assert lib.spava_cache_read(*h, -1, 1, FAKE, FAKE, *w) == 1
    assert lib.spava_cache_read(*h, 0, -1, FAKE, FAKE, *w) == 1
    assert lib.spava_cache_read(*h, (1 << 31) - 1, 1, FAKE, FAKE, *w) == 2
    assert lib.spava_cache_read(*h, 0, 1 << 29, FAKE, FAKE, *w) == 2
    assert lib.spava_cache_read(*h, 0, 1, None, FAKE, *w) == 1
    assert lib.spava_cache_read(*h, 0, 1, FAKE, FAKE + 4, *w) == 3
    # more work units than 32 bits count
    wide = refs(cache(Hq=32, Hkv=32).c(), pools(), batch(n=1 << 10, pages=1 << 26))
    assert lib.spava_cache_attn(*wide, FAKE, FAKE, None, *w) == 2
    assert lib.spava_cache_attn(*h, None, FAKE, None, *w) == 1
    assert lib.spava_cache_attn(*h, FAKE, FAKE + 8, None, *w) == 3
    assert lib.spava_cache_attn(*h, FAKE, FAKE, FAKE + 2, *w) == 3
    # the rotation's heads must be the cache's
    ro = ctypes.byref(rope(Hq=8, Hkv=2))
    assert lib.spava_cache_append(ro, *h, 1, FAKE, 1024, FAKE, 1024, FAKE, 1024, None, None, FAKE, FAKE, FAKE, *w) == 1
    ro = ctypes.byref(rope())
    assert lib.spava_cache_append(ro, *h, 1, FAKE, 1024, FAKE, 1024, FAKE, 1024, None, None, FAKE, FAKE, None, *w) == 1
    assert lib.spava_cache_append(ro, *h, 1, FAKE, 1024, FAKE, 1024, FAKE, 1024, None, None, None, FAKE, FAKE, *w) == 1


def test_nothing_to_do_is_ok():
    lib, h = native.load(), refs(cache().c(), pools(), batch(n=0))
    w = (FAKE, WS, None)
    assert lib.spava_cache_write(*h, 1, None, 128, None, 128, *w) == 0
    assert lib.spava_cache_read(*h, 0, 1, None, None, *w) == 0
    assert lib.spava_cache_attn(*h, None, None, None, *w) == 0
    h = refs(cache().c(), pools(), batch())
    assert lib.spava_cache_write(*h, 0, None, 128, None, 128, *w) == 0
    assert lib.spava_cache_read(*h, 5, 0, None, None, *w) == 0


def test_sections_default_and_limit():
    assert list(RopeLayout(4, 2, 64).c().section) == [32, 0, 0, 0]
    assert list(RopeLayout(4, 2, 128, rope_dim=64, sections=(8, 12, 12)).c().section) == [8, 12, 12, 0]
    with pytest.raises(ValueError):
        RopeLayout(4, 2, 64, sections=(8, 8, 8, 4, 4)).c()


def test_quantiser_against_every_e4m3_value():
    """Nearest of all finite e4m3 values (ties to the even code), smallest exponent."""
    codes = torch.arange(256, dtype=torch.uint8).view(E4M3).double()
    fine = codes[codes.isfinite()]
    vals = fine.unique()                       # ascending, one zero
    half = torch.arange(len(vals)) - (vals == 0).nonzero().item()      # signed code number
    x = torch.randn(50, 64, generator=torch.Generator().manual_seed(0), dtype=torch.float64) * 3
    x[0] = 0
    x[1, 0] = 448 * 8.0
    x[2] = torch.linspace(-448, 448, 64)
    x[3, :4] = torch.tensor([448.0, 1.0625, 1.1875, 2.0 ** -10])        # ties
    x = x.to(torch.bfloat16)
    z, e = quantise(x)
    for i in range(50):
        top = float(x[i].abs().max())
        assert top <= 448 * 2.0 ** float(e[i])
        assert e[i] == -120 or top > 448 * 2.0 ** (float(e[i]) - 1)
        y = x[i].double() * 2.0 ** -float(e[i])
        dist = (y[:, None] - vals).abs()
        best = dist.min(1).values
        near = dist == best[:, None]
        even = near & ((half % 2 == 0)[None] | (near.sum(1) == 1)[:, None])
        assert torch.equal(vals[even.double().argmax(1)], z[i])


def test_package_imports_before_its_extensions_are_built(tmp_path):
    """A fresh checkout can import the package, and so build it."""
    import os
    import shutil
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    shutil.copytree(os.path.join(root, "sequence_sparse_attention_b200"), tmp_path / "sequence_sparse_attention_b200",
                    ignore=shutil.ignore_patterns("*.so", "__pycache__"))
    shutil.copytree(os.path.join(root, "include"), tmp_path / "include")
    code = ("import sequence_sparse_attention_b200 as s, sequence_sparse_attention_b200.build, sys\n"
            "try:\n    s.cache._load_calls()\nexcept ImportError as e:\n    sys.exit(0 if 'build it with' in str(e) else 1)\n"
            "sys.exit(2)")
    assert subprocess.run([sys.executable, "-c", code], cwd=tmp_path).returncode == 0


def test_compiled_calls_load_without_a_gpu():
    from sequence_sparse_attention_b200.cache import _load_calls
    calls = _load_calls()
    with pytest.raises(ValueError):
        calls.Rope(0, 0, 0, 0, 0)
    with pytest.raises(ValueError):
        calls.Cache(0, 0, 0, 0, 0)
    c = rope()
    r = calls.Rope(ctypes.addressof(c), 0, 0, 0, 0)
    with pytest.raises(TypeError):
        r.apply(1)
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    for bad in ((x, x, None, None, None), (1, x, None, None, None), (x[0], x, None, None, None)):
        with pytest.raises(ValueError):      # host tensors, no tensor, no rows
            r.apply(*bad)
