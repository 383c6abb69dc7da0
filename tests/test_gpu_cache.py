"""The answering side on the GPU against 64-bit formulas (cache_util): norm with
rotation, paged writes and reads, attention of one new token, and a run of them
around a prefill layer."""
import math

import pytest
import torch

import cache_util as cu
from cache_util import E4M3
from sequence_sparse_attention_b200 import (CacheLayout, Layout, PagedCache, QKNormRope, RopeLayout, Spava,
                                            SpavaError)
from sequence_sparse_attention_b200.synth import Workload, make_inputs

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(*shape, g, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(BF16)


def freqs(rope, theta=1e6):
    j = torch.arange(rope // 2, dtype=torch.float64, device="cuda")
    return (theta ** (-2 * j / max(rope, 1))).float()


def split(rope, axes):
    half, out = rope // 2, []
    for a in range(axes - 1):
        out.append(half // (axes + 1) + a)
    return tuple(out) + (half - sum(out),)


# ------------------------------------------------------------------ norm and rotation
ROPE_CASES = [
    # rows, Hq, Hkv, d, rope, interleaved, axes, norm, weights, far
    (1, 28, 4, 128, 128, False, 3, True, True, 1 << 17),
    (1, 1, 1, 64, 64, False, 1, True, True, 100),
    (2, 1, 1, 128, 128, False, 1, True, False, 100),
    (7, 4, 2, 64, 64, False, 1, True, True, 1 << 20),
    (33, 28, 4, 128, 64, False, 2, True, True, 1 << 18),
    (129, 3, 3, 128, 16, False, 1, True, True, 5000),
    (64, 32, 8, 128, 128, True, 1, True, True, 1 << 17),
    (65, 14, 2, 64, 32, True, 4, True, True, 1 << 17),
    (31, 16, 1, 128, 112, False, 1, True, True, 1 << 17),
    (17, 5, 5, 64, 0, False, 1, True, True, 10),
    (19, 6, 2, 128, 128, False, 1, False, False, 1 << 31),
    (1000, 28, 4, 128, 128, False, 3, True, True, 1 << 31),
]


@pytest.mark.parametrize("rows,Hq,Hkv,d,rope,inter,axes,norm,weights,far", ROPE_CASES)
def test_norm_rope(rows, Hq, Hkv, d, rope, inter, axes, norm, weights, far):
    g = gen(rows)
    qkv = randn(rows, (Hq + 2 * Hkv) * d + 8, g=g, scale=3.0)       # tokens not packed
    q = qkv[:, :Hq * d].unflatten(1, (Hq, d))
    k = qkv[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d))
    qw, kw = (1 + 0.3 * randn(d, g=g).float()).to(BF16), randn(d, g=g)
    if not weights:
        qw = kw = None
    pos = torch.randint(0, far, (axes, rows), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    pos[:, 0] = far - 1
    sections, freq = split(rope, axes), freqs(rope)
    op = QKNormRope(RopeLayout(Hq, Hkv, d, rope_dim=rope, interleaved=inter, sections=sections, norm=norm, eps=1e-5),
                    freq if rope else None, qw, kw, device="cuda")
    keep = qkv.clone()
    qo, ko = op.apply(q, k, pos if rope else None)
    assert torch.equal(keep, qkv)
    for got, x, w in ((qo, q, qw), (ko, k, kw)):
        cu.check_norm_rope(got, cu.norm_rope(x, w, pos, freq, rope, inter, sections, norm, 1e-5))
    if rope == 0 and not norm:
        assert torch.equal(qo, q) and torch.equal(ko, k)
    # the rows that pass through keep their bits without the norm
    if not norm and rope < d:
        assert torch.equal(qo[..., rope:], q[..., rope:])
    # in place, on packed tensors: the same bytes
    q2, k2 = q.contiguous(), k.contiguous()
    r = op.apply(q2, k2, pos if rope else None, q_out=q2, k_out=k2)
    assert r[0] is q2 and torch.equal(q2, qo) and torch.equal(k2, ko)


def test_norm_rope_pass_through_and_zero_rows():
    g = gen(1)
    q, k = randn(5, 4, 64, g=g), randn(5, 2, 64, g=g)
    op = QKNormRope(RopeLayout(4, 2, 64, rope_dim=0, norm=False), device="cuda")
    qo, ko = op.apply(q, k)
    assert torch.equal(qo, q) and torch.equal(ko, k)
    qo, ko = op.apply(q[:0], k[:0])
    assert qo.shape == (0, 4, 64) and ko.shape == (0, 2, 64)
    # a head of zeros stays zero with eps, is NaN (0 / 0) without
    q.zero_()
    f, p = freqs(64), torch.arange(5, dtype=torch.int32, device="cuda")
    for eps in (1e-6, 0.0):
        qo, _ = QKNormRope(RopeLayout(4, 2, 64, eps=eps), f).apply(q, k, p)
        assert (qo == 0).all() if eps else qo.isnan().all()


def test_norm_rope_refusals():
    g = gen(2)
    q, k = randn(4, 4, 64, g=g), randn(4, 2, 64, g=g)
    p = torch.arange(4, dtype=torch.int32, device="cuda")
    op = QKNormRope(RopeLayout(4, 2, 64), freqs(64))
    for bad in ((q.float(), k, p), (q, k[:3], p), (q.transpose(0, 1), k, p), (q, k, p.long()),
                (q, k, p[:3]), (q, k, p.cpu()), (q[..., :32], k, p), (q.transpose(1, 2).contiguous().transpose(1, 2), k, p),
                (q.cpu(), k, p)):
        with pytest.raises(ValueError):
            op.apply(*bad)
    with pytest.raises(ValueError):
        op.apply(q, k, p, q_out=torch.empty_like(q, dtype=torch.float32))
    with pytest.raises(ValueError):
        QKNormRope(RopeLayout(4, 2, 64), freqs(32))
    with pytest.raises(ValueError):
        QKNormRope(RopeLayout(4, 2, 64), None, torch.ones(64, dtype=BF16, device="cuda"))
    odd = torch.empty(4 * 4 * 64 + 1, dtype=BF16, device="cuda")[1:].view(4, 4, 64)
    with pytest.raises(SpavaError) as e:
        op.apply(odd, k, p)
    assert e.value.status == 3


# ------------------------------------------------------------------ cache rows
WRITE_CASES = [
    # lens, new, Hkv, d, page
    ([1], 1, 1, 64, 1),
    ([5, 0, 9], 3, 2, 64, 4),          # an empty sequence: all its rows skipped
    ([2, 7], 5, 3, 128, 5),            # the first sequence is shorter than the new rows
    ([333], 333, 4, 128, 24),
    ([100, 131, 64], 31, 8, 128, 16),
    ([1000], 17, 2, 64, 64),
]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,new,Hkv,d,page", WRITE_CASES)
def test_write_and_read(lens, new, Hkv, d, page, kind):
    g = gen(new)
    n, e4m3 = len(lens), kind == "e4m3"
    per = max(1, -(-max(lens) // page)) + 1
    n_pages = n * per + 3
    pools = cu.make_pools(n_pages, Hkv, page, d, e4m3, g)
    table = cu.make_table(n, per, n_pages, g)
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cache = PagedCache(CacheLayout(Hkv, Hkv, d, page_size=page, n_pages=n_pages, dtype=pools[0].dtype),
                       k_pages=pools[0], v_pages=pools[1], k_exp=pools[2], v_exp=pools[3])
    kv = randn(n * new, 2 * Hkv * d + 16, g=g)
    kv *= torch.exp2(torch.randint(-20, 20, (n * new, 1), generator=g, device="cuda").float()).to(BF16)
    k, v = kv[:, :Hkv * d].unflatten(1, (Hkv, d)), kv[:, Hkv * d:2 * Hkv * d].unflatten(1, (Hkv, d))
    v[0, 0] = 0.0
    want = cu.written(pools, k, v, table, lt, page, new)
    cache.write(k, v, table, lt)
    for got, ref in zip(pools, want):
        if got is not None:
            assert torch.equal(got.cpu().to(ref.dtype), ref)
    assert cache.device_status() == 0
    # read back: windows that start inside, end behind and lie past the sequences
    for first, rows in ((0, max(lens)), (0, max(lens) + 3), (3, 9), (max(lens) + 1, 4)):
        rows = min(rows, per * page * 2)
        kr, vr = cache.read(table, lt, rows, first=first)
        assert kr.shape == (n, rows, Hkv, d)
        for b, m in enumerate(lens):
            ks, vs = cu.rows_of(pools, table, b, m, page)
            end = max(0, min(rows, m - first))
            for got, ref in ((kr, ks), (vr, vs)):
                assert torch.equal(got[b, :end].double(), ref[first:first + end])
                assert (got[b, end:] == 0).all()
    assert cache.device_status() == 0


def test_quantised_rows_at_the_edges():
    """Zeros, the smallest and largest bf16 rows, ties, NaN and infinities."""
    g = gen(5)
    d, n = 64, 12
    x = randn(n, 1, d, g=g)
    tiny, big = 2.0 ** -133, float(torch.finfo(BF16).max)
    x[0] = 0
    x[1] = tiny
    x[2, 0, :3] = torch.tensor([big, -big, 1.0], device="cuda")
    x[3] = torch.linspace(-448, 448, d, device="cuda").to(BF16)
    x[4, 0, :5] = torch.tensor([448.0, 1.0625, 1.1875, 2.0 ** -10, 3 * 2.0 ** -10], device="cuda")
    x[5, 0, 1] = math.nan
    x[6, 0, 2] = math.inf
    x[7, 0, 3] = -math.inf
    x[8] = math.inf
    x[9] = math.nan
    x[10, 0, :2] = torch.tensor([449.0, 1.0], device="cuda")
    x[11] = 2.0 ** -126
    cache = PagedCache(CacheLayout(1, 1, d, page_size=n, n_pages=1, dtype=E4M3))
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    cache.write(x, x, table, lens)
    z, e = cu.quantise(x)
    for pool, exps in ((cache.k_pages, cache.k_exp), (cache.v_pages, cache.v_exp)):
        assert torch.equal(exps[0, 0].double(), e[:, 0])
        got = pool[0, 0].double()
        assert torch.equal(got.isnan(), z[:, 0].isnan())
        assert torch.equal(got.nan_to_num(0.0), z[:, 0].nan_to_num(0.0))
    k, v = cache.read(table, lens, n)
    want = (z * torch.exp2(e)[..., None]).to(BF16)
    assert torch.equal(k[0].nan_to_num(7.0), want.nan_to_num(7.0)) and torch.equal(v[0].nan_to_num(7.0), want.nan_to_num(7.0))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,d,rope,inter,axes,n,new,page", [
    (28, 4, 128, 128, False, 3, 1, 1, 64), (4, 2, 64, 32, True, 1, 5, 3, 7), (16, 1, 128, 64, False, 2, 3, 1, 16),
    (12, 12, 64, 64, False, 1, 40, 1, 1)])
def test_append_is_norm_rope_and_write(Hq, Hkv, d, rope, inter, axes, n, new, page, kind):
    g = gen(n + page)
    dtype = BF16 if kind == "bf16" else E4M3
    per, rows = 9, n * new
    lens = torch.randint(new, per * page + 1, (n,), generator=g, device="cuda", dtype=torch.int32).clamp(max=per * page)
    lens[-1] = 0 if n > 1 else lens[-1]
    lay = CacheLayout(Hq, Hkv, d, page_size=page, n_pages=n * per, dtype=dtype)
    table = cu.make_table(n, per, n * per, g)
    qkv = randn(rows, (Hq + 2 * Hkv) * d, g=g)
    q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([Hq * d, Hkv * d, Hkv * d], 1))
    op = QKNormRope(RopeLayout(Hq, Hkv, d, rope_dim=rope, interleaved=inter, sections=split(rope, axes)), freqs(rope),
                    randn(d, g=g), randn(d, g=g))
    pos = torch.randint(0, 100000, (axes, rows), generator=g, device="cuda", dtype=torch.int32)
    one, two = PagedCache(lay), PagedCache(lay)
    qo, ko = op.apply(q, k, pos)
    one.write(ko, v, table, lens)
    qa = two.append(op, q, k, v, pos, table, lens)
    assert torch.equal(qa, qo)
    for a, b in zip(one.tensors, two.tensors):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert two.k_pages.view(torch.uint8).any()
    assert one.device_status() == 0 and two.device_status() == 0


# ------------------------------------------------------------------ attention
def attn_case(lens, Hq, Hkv, d, page, e4m3, seed=0, extra=1, q_scale=1.0, poison=True):
    """A cache whose rows behind the sequences' ends (and free pages) are NaN."""
    g = gen(seed)
    n = len(lens)
    per = max(1, -(-max(lens) // page)) + extra
    n_pages = n * per + 2
    pools = cu.make_pools(n_pages, Hkv, page, d, e4m3, g)
    table = cu.make_table(n, per, n_pages, g)
    if poison:
        used = torch.zeros((n_pages, page), dtype=torch.bool, device="cuda")
        for b, m in enumerate(lens):
            pos = torch.arange(m, device="cuda")
            used[table[b][pos // page].long(), pos % page] = True
        for pool in pools[:2]:
            bytes_ = pool.view(torch.uint8).view(n_pages, Hkv, page, -1)
            bytes_.copy_(torch.where(used[:, None, :, None], bytes_, 0x7f if e4m3 else 0xff))
            assert pool.double().isnan().any() or used.all()
    cache = PagedCache(CacheLayout(Hq, Hkv, d, page_size=page, n_pages=n_pages, dtype=pools[0].dtype),
                       k_pages=pools[0], v_pages=pools[1], k_exp=pools[2], v_exp=pools[3])
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    return cache, pools, randn(n, Hq, d, g=g, scale=q_scale), table, lt


ATTN_CASES = [
    ([1], 1, 1, 64, 1), ([1], 28, 4, 128, 64), ([0, 3, 0, 0, 17], 4, 2, 64, 16), ([2], 8, 1, 128, 5),
    ([15, 16, 17, 31, 32, 33], 14, 2, 64, 8), ([63, 64, 65, 127, 128, 129], 28, 4, 128, 24),
    ([255, 256, 257], 9, 1, 64, 48), ([1000, 1, 700], 16, 1, 128, 1), ([511], 40, 2, 128, 100),
    ([5000], 28, 4, 128, 64), ([4097, 0, 2048, 33], 32, 8, 128, 16), ([20011], 24, 2, 64, 256),
    ([300] * 200, 4, 4, 64, 64), (list(range(0, 400)), 6, 3, 128, 7), ([65536], 17, 1, 128, 64),    # 64, 128 and 204 items: clusters of 4, 2 and 1 blocks where the tables are short
    ([50, 130, 0, 700] * 4, 28, 4, 128, 16), ([33, 90] * 16, 12, 4, 64, 24), ([20, 400, 61] * 17, 40, 4, 128, 64),
]


def widen(table, page, tokens=1 << 17):
    """The same table with room for more tokens (entries that are not read):
    short contexts then run as long ones may."""
    wide = torch.full((table.shape[0], -(-tokens // page)), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table[:, :wide.shape[1]]
    return wide


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,Hq,Hkv,d,page", ATTN_CASES)
def test_attn(lens, Hq, Hkv, d, page, kind, wide):
    cache, pools, q, table, lt = attn_case(lens, Hq, Hkv, d, page, kind == "e4m3", seed=len(lens) + Hq)
    if wide:
        table = widen(table, page)
    o, lse = cache.attn(q, table, lt)
    assert cache.device_status() == 0
    cu.check_attn(o, lse, q, pools, table, lens, page)
    # the same bytes again, with outputs given and without lse
    o2 = torch.full_like(o, math.nan)
    cache.attn(q, table, lt, o=o2, want_lse=False)
    assert torch.equal(o, o2)
    # whatever the workspace holds behind its status block
    cache.workspace[256:] = 0xff
    o3, lse3 = cache.attn(q, table, lt)
    assert torch.equal(o, o3) and torch.equal(lse, lse3)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_attn_sharp_and_ordered_scores(kind):
    """Scores that grow along the context (the reference moves all the time),
    that fall, one dominant key, all keys equal, and a scale of the caller's."""
    lens, Hq, Hkv, d, page = [3000], 7, 1, 128, 64
    for mode in ("rising", "falling", "spike", "equal", "scale"):
        cache, pools, q, table, lt = attn_case(lens, Hq, Hkv, d, page, False, seed=3, q_scale=1.0, poison=False)
        g = gen(11)
        k = randn(lens[0], Hkv, d, g=g, scale=0.05)
        v = randn(lens[0], Hkv, d, g=g)
        ramp = torch.arange(lens[0], device="cuda").float() / 100
        if mode in ("rising", "falling"):
            q[..., 0] = 8.0
            k[:, 0, 0] = (ramp if mode == "rising" else 30 - ramp).to(BF16)
        elif mode == "spike":
            q[..., 1] = 16.0
            k[1777, 0, 1] = 100.0
        elif mode == "equal":
            k[:] = k[0]
        lay = CacheLayout(Hq, Hkv, d, page_size=page, n_pages=cache.lay.n_pages,
                          dtype=E4M3 if kind == "e4m3" else BF16, scale=0.31 if mode == "scale" else 0.0)
        cache = PagedCache(lay)
        cache.write(k, v, table, lt)
        pools = list(cache.tensors) + ([] if kind == "e4m3" else [None, None])
        o, lse = cache.attn(q, table, lt)
        cu.check_attn(o, lse, q, pools, table, lens, page, scale=0.31 if mode == "scale" else None)


def test_attn_wide_scales_of_a_quantised_cache():
    """Value rows of zeros, of 2^-100 and 2^100, keys of 2^-30 and 2^6 beside each
    other: sums and outputs keep their own references."""
    Hq, Hkv, d, page = 4, 2, 64, 16
    for case in range(4):
        g = gen(case)
        lens = [700]
        k, v = randn(700, Hkv, d, g=g), randn(700, Hkv, d, g=g)
        if case == 0:
            v.zero_()
        elif case == 1:
            v *= 2.0 ** -100
        elif case == 2:
            v *= 2.0 ** 100
            v[::3] = 0
        else:
            v *= torch.exp2(torch.randint(-40, 40, (700, 1, 1), generator=g, device="cuda").float()).to(BF16)
            k *= torch.exp2(torch.randint(-30, 3, (700, 1, 1), generator=g, device="cuda").float()).to(BF16)
        cache = PagedCache(CacheLayout(Hq, Hkv, d, page_size=page, n_pages=44, dtype=E4M3))
        table = cu.make_table(1, 44, 44, g)
        lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
        cache.write(k, v, table, lt)
        for q_scale in (1.0, 2.0 ** -60, 2.0 ** 3):
            q = randn(1, Hq, d, g=g, scale=q_scale)
            o, lse = cache.attn(q, table, lt)
            cu.check_attn(o, lse, q, cache.tensors, table, lens, page)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_attn_non_finite_rows(kind):
    """NaN in a key or value that counts reaches the output of the heads that
    read it and no other; keys whose scores are all -inf leave an empty row."""
    Hq, Hkv, d, page, lens = 8, 2, 64, 16, [200]
    cache, pools, q, table, lt = attn_case(lens, Hq, Hkv, d, page, kind == "e4m3", seed=9)
    clean, _ = cache.attn(q, table, lt)
    p, r = cu.place(table, page, 0, 123)
    if kind == "bf16":
        pools[1][p, 1, r, 5] = math.nan
    else:
        pools[1].view(torch.uint8)[p, 1, r, 5] = 0x7f
    o, _ = cache.attn(q, table, lt)
    assert torch.equal(o[0, :4], clean[0, :4])                 # KV head 0's query heads
    assert o[0, 4:, 5].isnan().all()
    rest = [i for i in range(d) if i != 5]
    assert torch.equal(o[0, 4:][:, rest], clean[0, 4:][:, rest])
    if kind == "bf16":
        q2 = q.abs() + 0.5
        pools[0][:, 0] = -math.inf
        o, lse = cache.attn(q2, table, lt)
        assert (o[0, :4] == 0).all() and (lse[:4] == -math.inf).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_bad_lengths_and_pages_are_reported_and_skipped(kind):
    Hq, Hkv, d, page = 6, 2, 64, 8
    lens = [100, 77, 50]
    cache, pools, q, table, lt = attn_case(lens, Hq, Hkv, d, page, kind == "e4m3", seed=4, extra=0)
    bad = table.clone()
    bad[0, 3], bad[0, 12], bad[1, 0] = -1, cache.lay.n_pages, 2 ** 31 - 1

    def keep(b):
        m = torch.ones(lens[b], dtype=torch.bool, device="cuda")
        if b == 0:
            m[24:32] = False
            m[96:104] = False
        elif b == 1:
            m[0:8] = False
        return m

    o, lse = cache.attn(q, bad, lt)
    assert cache.device_status() == 2 and cache.device_status() == 0
    cu.check_attn(o, lse, q, pools, torch.where(bad == table, bad, 0), lens, page, keep=keep)
    kr, _ = cache.read(bad, lt, 100)
    assert cache.device_status() == 2
    assert (kr[0, 24:32] == 0).all() and (kr[1, :8] == 0).all() and kr[0, :24].any()
    before = [x.view(torch.uint8).clone() for x in cache.tensors]
    new = randn(3 * 100, Hkv, d, g=gen(1))
    cache.write(new, new, torch.full_like(bad, -5), lt)
    assert cache.device_status() == 2
    assert all(torch.equal(a, x.view(torch.uint8)) for a, x in zip(before, cache.tensors))
    # lengths: below zero is empty, beyond the table is the table's end
    odd = torch.tensor([-3, 2 ** 31 - 1, 50], dtype=torch.int32, device="cuda")
    o, lse = cache.attn(q, table, odd)
    assert cache.device_status() == 2
    assert (o[0] == 0).all() and (lse[:, 0] == -math.inf).all()
    o2, _ = cache.attn(q, table, torch.tensor([0, table.shape[1] * page, 50], dtype=torch.int32, device="cuda"))
    assert cache.device_status() == 0
    assert torch.equal(o.nan_to_num(9.0), o2.nan_to_num(9.0))
    cu.check_attn(o[2:], lse[:, 2:], q[2:], pools, table[2:], [50], page)


def test_attn_shared_pages_and_growing_lengths():
    """Several new tokens of one sequence: rows of the batch that share its pages."""
    Hq, Hkv, d, page = 28, 4, 128, 16
    cache, pools, q, table, lt = attn_case([900] + [1] * 5, Hq, Hkv, d, page, False, seed=6, extra=0, poison=False)
    table = table[:1].expand(6, -1).contiguous()
    lens = [895, 896, 897, 898, 899, 900]
    o, lse = cache.attn(q, table, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    cu.check_attn(o, lse, q, pools, table, lens, page)


def test_attn_partials_of_a_split_context_merge():
    """lse joins what two caches hold of one context."""
    Hq, Hkv, d, page = 14, 2, 128, 32
    cache, pools, q, table, lt = attn_case([2500], Hq, Hkv, d, page, False, seed=8, extra=0)
    o, lse = cache.attn(q, table, lt)
    cut = 40
    parts = [cache.attn(q, t.contiguous(), torch.tensor([m], dtype=torch.int32, device="cuda"))
             for t, m in ((table[:, :cut], cut * page), (table[:, cut:], 2500 - cut * page))]
    top = torch.logaddexp(parts[0][1], parts[1][1])
    assert torch.allclose(top, lse, rtol=0, atol=2e-5)
    merged = sum(torch.exp(l - top).t()[..., None] * x.float() for x, l in parts)
    assert (merged - o.float()).abs().max() <= 3 * 2.0 ** -8 * o.float().abs().max()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_offsets_past_32_bits(kind):
    """Rows more than 4 GiB (and 2^31 elements) into the pools."""
    Hkv, d, page = 8, 128, 64
    e4m3 = kind == "e4m3"
    n_pages = 80000 if e4m3 else 40000          # 5.2 GB a pool: 5.2e9 or 2.6e9 elements
    dtype = E4M3 if e4m3 else BF16
    lay = CacheLayout(32, Hkv, d, page_size=page, n_pages=n_pages, dtype=dtype)
    shape = (n_pages, Hkv, page, d)
    kp, vp = (torch.empty(shape, dtype=dtype, device="cuda") for _ in range(2))
    ke, ve = (torch.empty(shape[:3], dtype=torch.int8, device="cuda") if e4m3 else None for _ in range(2))
    cache = PagedCache(lay, k_pages=kp, v_pages=vp, k_exp=ke, v_exp=ve)
    table = torch.tensor([[n_pages - 1, 0, n_pages - 2, n_pages // 2 + 1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([250], dtype=torch.int32, device="cuda")
    g = gen(1)
    k, v = randn(250, Hkv, d, g=g), randn(250, Hkv, d, g=g)
    cache.write(k, v, table, lens)
    kr, vr = cache.read(table, lens, 250)
    for got, x in ((kr, k), (vr, v)):
        z, e = cu.quantise(x)
        assert torch.equal(got[0].double(), z * torch.exp2(e)[..., None] if e4m3 else x.double())
    q = randn(1, 32, d, g=g)
    o, lse = cache.attn(q, table, lens)
    cu.check_attn(o, lse, q, (kp, vp, ke, ve), table, [250], page)


# ------------------------------------------------------------------ streams, graphs, workspaces
def test_attn_in_a_graph_follows_lengths_and_tables():
    """Two graphs share a workspace, replayed in turn with other contents."""
    Hq, Hkv, d, page = 28, 4, 128, 16
    cache, pools, q, table, lt = attn_case([900, 300, 1200], Hq, Hkv, d, page, False, seed=12, extra=0)
    outs, graphs = [], []
    side = torch.cuda.Stream()
    for _ in range(2):
        o, lse = torch.empty_like(q), torch.empty((Hq, 3), device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side):
            cache.attn(q, table, lt, o=o, lse=lse)
        outs.append((o, lse))
        graphs.append(gr)
    for lens in ([900, 300, 1200], [1, 0, 1200], [900, 299, 17]):
        lt.copy_(torch.tensor(lens, dtype=torch.int32))
        want = cache.attn(q, table, lt)
        for gr, (o, lse) in zip(graphs, outs):
            o.fill_(math.nan)
            gr.replay()
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        cu.check_attn(outs[0][0], outs[0][1], q, pools, table, lens, page)


def test_a_captured_step_among_copies_and_forks():
    """A graph of a whole decode step -- copies, a length counted up, append on
    one stream, attention on another -- replayed token by token, gives what the
    calls give one by one."""
    Hq, Hkv, d, page, n = 8, 2, 64, 16, 3
    g = gen(31)
    for cap in (64, 1 << 16):                     # short and long tables
        lay = CacheLayout(Hq, Hkv, d, page_size=page, n_pages=n * 4)
        table = cu.make_table(n, 4, n * 4, g)
        wide = widen(table, page, cap) if cap > 64 else table
        op = QKNormRope(RopeLayout(Hq, Hkv, d), freqs(d), randn(d, g=g), randn(d, g=g))
        steps = [randn(n, (Hq + 2 * Hkv) * d, g=g) for _ in range(20)]
        results = []
        for captured in (False, True):
            cache = PagedCache(lay)
            lens = torch.zeros(n, dtype=torch.int32, device="cuda")
            pos = torch.zeros((1, n), dtype=torch.int32, device="cuda")
            x = torch.zeros_like(steps[0])
            src = torch.zeros_like(x)
            o, lse = torch.empty((n, Hq, d), dtype=BF16, device="cuda"), torch.empty((Hq, n), device="cuda")
            qa = torch.empty_like(o)
            other = torch.cuda.Stream()

            def step():
                x.copy_(src)
                pos.copy_(lens[None])
                lens.add_(1)
                q, k, v = (y.unflatten(1, (-1, d)) for y in x.split([Hq * d, Hkv * d, Hkv * d], 1))
                cache.append(op, q, k, v, pos, wide, lens, q_out=qa)
                if captured:
                    other.wait_stream(torch.cuda.current_stream())
                    with torch.cuda.stream(other):
                        cache.attn(qa, wide, lens, o=o, lse=lse)
                    torch.cuda.current_stream().wait_stream(other)
                else:
                    torch.cuda.synchronize()
                    cache.attn(qa, wide, lens, o=o, lse=lse)
                    torch.cuda.synchronize()

            if captured:
                side, gr = torch.cuda.Stream(), torch.cuda.CUDAGraph()
                side.wait_stream(torch.cuda.current_stream())
                with torch.cuda.graph(gr, stream=side):
                    step()
            out = []
            for s in steps:
                src.copy_(s)
                gr.replay() if captured else step()
                out.append((o.clone(), lse.clone()))
            results.append(out + [(cache.k_pages, cache.v_pages)])
            assert cache.device_status() == 0
        for a, b in zip(*results):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_a_chain_of_calls_without_waiting():
    """Hundreds of dependent launches back to back: every call sees what the one
    before wrote (a cache that is rewritten, read and attended in turn)."""
    Hq, Hkv, d, page, rows = 28, 4, 128, 16, 300
    g = gen(32)
    table = cu.make_table(1, 20, 20, g)
    lens = torch.tensor([rows], dtype=torch.int32, device="cuda")
    data = [(randn(rows, Hkv, d, g=g), randn(rows, Hkv, d, g=g), randn(1, Hq, d, g=g)) for _ in range(4)]
    cache = PagedCache(CacheLayout(Hq, Hkv, d, page_size=page, n_pages=20))
    want = []
    for k, v, q in data:
        cache.write(k, v, table, lens)
        torch.cuda.synchronize()
        want.append(cache.attn(q, table, lens))
        torch.cuda.synchronize()
    for wide in (False, True):
        tb = widen(table, page) if wide else table
        got = []
        for i in range(200):
            k, v, q = data[i % 4]
            cache.write(k, v, tb, lens)
            got.append((*cache.read(tb, lens, rows), cache.attn(q, tb, lens)[0]))
        first = got[:4]
        for i, (k, v, o) in enumerate(got):
            assert torch.equal(k[0], data[i % 4][0]) and torch.equal(v[0], data[i % 4][1])
            assert torch.equal(o, first[i % 4][2])
            if not wide:
                assert torch.equal(o, want[i % 4][0])


def test_calls_wait_for_events_of_other_streams():
    """Between two calls on one stream, an event of another stream on which what
    the second call reads is still being made: the dependent launch waits for both."""
    Hq, Hkv, d, page = 28, 4, 128, 16
    for tokens in (16, 900, 1 << 16):             # tables for a warp, a cluster, the line
        lens = [min(900, tokens)]
        cache, pools, q, table, lt = attn_case(lens, Hq, Hkv, d, page, False, seed=41, extra=0, poison=False)
        tb = widen(table, page, tokens) if tokens > 900 else table
        q2 = q.flip(1).contiguous()
        rows = randn(lens[0], Hkv, d, g=gen(2))
        want = cache.attn(q2, tb, lt)
        torch.cuda.synchronize()
        a, b = torch.cuda.Stream(), torch.cuda.Stream()
        qb = q.clone()
        for _ in range(3):
            qb.copy_(q)
            torch.cuda.synchronize()
            with torch.cuda.stream(a):
                torch.cuda._sleep(5_000_000)      # a few ms
                qb.copy_(q2)
                made = a.record_event()
            with torch.cuda.stream(b):
                cache.read(tb, lt, lens[0])
                cache.attn(q, tb, lt)
                b.wait_event(made)
                got = cache.attn(qb, tb, lt)
            b.synchronize()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        # and the other way: a later kernel of another stream waits for the last call
        other = PagedCache(cache.lay, k_pages=pools[0].clone(), v_pages=pools[1].clone())
        with torch.cuda.stream(a):
            torch.cuda._sleep(5_000_000)
            other.write(rows, rows, tb, lt)
            k, v = other.read(tb, lt, lens[0])
            done = a.record_event()
        b.wait_event(done)
        with torch.cuda.stream(b):
            copy = k.clone()
        b.synchronize()
        assert torch.equal(copy[0], rows)


def test_threads_share_a_cache():
    """Calls from several host threads, each on its own stream with its own workspace."""
    import threading
    Hq, Hkv, d, page = 28, 4, 128, 16
    cache, pools, q, table, lt = attn_case([700, 1, 90, 2000], Hq, Hkv, d, page, True, seed=33, extra=0)
    want = {m: cache.attn(q[:m].contiguous(), table[:m], lt[:m]) for m in (1, 2, 3, 4)}
    torch.cuda.synchronize()
    bad = []

    def work(m):
        try:
            ws, s = cache.new_workspace(), torch.cuda.Stream()
            s.wait_stream(torch.cuda.default_stream())
            with torch.cuda.stream(s):
                qm, tm, lm = q[:m].contiguous(), table[:m], lt[:m]
                got = [cache.attn(qm, tm, lm, workspace=ws) for _ in range(100)]
            s.synchronize()
            for o, lse in got:
                if not (torch.equal(o, want[m][0]) and torch.equal(lse, want[m][1])):
                    bad.append(m)
        except Exception as e:  # noqa: BLE001
            bad.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(m,)) for m in (1, 2, 3, 4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad


def test_two_streams_with_their_own_workspaces():
    Hq, Hkv, d, page = 32, 8, 128, 64
    cache, pools, q, table, lt = attn_case([20000, 3000], Hq, Hkv, d, page, True, seed=13, extra=0)
    want = cache.attn(q, table, lt)
    streams = [torch.cuda.Stream() for _ in range(3)]
    spaces = [cache.new_workspace() for _ in streams]
    got = []
    torch.cuda.synchronize()
    for _ in range(5):
        for s, ws in zip(streams, spaces):
            with torch.cuda.stream(s):
                got.append(cache.attn(q, table, lt, workspace=ws))
    torch.cuda.synchronize()
    for o, lse in got:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_cache_refusals():
    cache, pools, q, table, lt = attn_case([50, 60], 4, 2, 64, 16, False, seed=14)
    k = randn(2, 2, 64, g=gen(0))
    for bad in (lambda: cache.attn(None, table, lt), lambda: cache.attn(q, [[0]], lt),
                lambda: cache.append(None, q, k, k, None, table, lt), lambda: cache.read(table, lt, -1),
                lambda: cache.attn(q.float(), table, lt), lambda: cache.attn(q[:1], table, lt),
                lambda: cache.attn(q, table.long(), lt), lambda: cache.attn(q, table[:1], lt),
                lambda: cache.attn(q, table, lt.cpu()), lambda: cache.attn(q, table.t().contiguous().t(), lt),
                lambda: cache.attn(q, table, lt, o=torch.empty_like(q[:1])),
                lambda: cache.attn(q, table, lt, lse=torch.empty((2, 4), device="cuda")),
                lambda: cache.attn(q, table, lt, workspace=torch.zeros(10, device="cuda")),
                lambda: cache.write(k[:1], k, table, lt), lambda: cache.write(k[:1], k[:1], table, lt),
                lambda: cache.write(k.double(), k, table, lt), lambda: cache.write(k, k[:, :1], table, lt),
                lambda: cache.read(table, lt, 4, k_out=torch.empty(3, device="cuda")),
                lambda: PagedCache(cache.lay, k_pages=pools[0][:1], v_pages=pools[1]),
                lambda: PagedCache(cache.lay, k_exp=torch.zeros(1, dtype=torch.int8, device="cuda")),
                lambda: PagedCache(cache.lay, device="cpu")):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(SpavaError) as e:
        cache.attn(q, table, lt, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 4


# ------------------------------------------------------------------ a run of them
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_prefill_then_answer(kind):
    """Norm and rotation, the prefill layer, its keys and values into a cache,
    then answer tokens one by one, against dense 64-bit attention."""
    w = Workload("answer", H=2, Hq=14, Hkv=2, d=128, N=1100, a=60, q=40, l=64, frame=32, seed=5)
    Hq, Hkv, d, N, steps, page = w.Hq, w.Hkv, w.d, w.N, 5, 24
    g = gen(21)
    x = randn(N + steps, (Hq + 2 * Hkv) * d, g=g)
    q, k, v = (y.unflatten(1, (-1, d)) for y in x.split([Hq * d, Hkv * d, Hkv * d], 1))
    t = torch.arange(N + steps, device="cuda", dtype=torch.int32)
    pos = torch.stack([t // 32, t // 8 % 4, t % 8]).contiguous()
    lay = RopeLayout(Hq, Hkv, d, sections=(16, 24, 24))
    qw, kw, f = randn(d, g=g), randn(d, g=g), freqs(d)
    op = QKNormRope(lay, f, qw, kw)
    n_pages = -(-(N + steps) // page)
    cache = PagedCache(CacheLayout(Hq, Hkv, d, page_size=page, n_pages=n_pages, dtype=E4M3 if kind == "e4m3" else BF16))
    table = cu.make_table(1, n_pages, n_pages, g)
    lens = torch.tensor([N], dtype=torch.int32, device="cuda")

    qn, kn = op.apply(q[:N], k[:N], pos[:, :N].contiguous())
    sp = Spava(Layout.from_workload(w))
    o, lse, _ = sp.prefill_attention(qn, kn, v[:N].contiguous())
    cache.write(kn, v[:N], table, lens)
    pools = list(cache.tensors) + ([] if kind == "e4m3" else [None, None])
    if kind == "bf16":
        # the question's last row attends everything before it exactly, in both
        oa, la = cache.attn(qn[-1:], table, lens)
        assert (oa[0].float() - o[-1].float()).abs().max() <= 2e-2
        assert (la[:, 0] - lse[:, -1]).abs().max() <= 2e-3
    for i in range(steps):
        at = N + i
        lens += 1
        qa = cache.append(op, q[at:at + 1], k[at:at + 1], v[at:at + 1], pos[:, at:at + 1].contiguous(), table, lens)
        cu.check_norm_rope(qa, cu.norm_rope(q[at:at + 1], qw, pos[:, at:at + 1], f, d, False, lay.sections, True, lay.eps))
        oa, la = cache.attn(qa, table, lens)
        cu.check_attn(oa, la, qa, pools, table, [at + 1], page)
    # what the cache holds is what was written, token by token
    want = cu.norm_rope(k, kw, pos, f, d, False, lay.sections, True, lay.eps)
    kr, vr = cache.read(table, lens, N + steps)
    if kind == "bf16":
        cu.check_norm_rope(kr[0], want)
        assert torch.equal(vr[0], v)
    else:
        z, e = cu.quantise(v)
        assert torch.equal(vr[0].double(), z * torch.exp2(e)[..., None])
    assert sp.device_status() == 0 and cache.device_status() == 0
