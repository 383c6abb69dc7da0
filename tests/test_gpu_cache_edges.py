"""The answering side at the edges of its ranges: small softmax weights of a
quantised cache, lengths beyond the table, tensors without an address or with
another one, empty batches, exponents at the ends of bf16, blocks full of tokens."""
import math

import pytest
import torch

import cache_util as cu
from cache_util import E4M3
from sequence_sparse_attention_b200 import CacheLayout, PagedCache, QKNormRope, RopeLayout, SpavaError

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(*shape, g, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(BF16)


def lengths(*lens):
    return torch.tensor(lens, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ weights of a quantised cache
def check_weights(o, q, pools, table, lens, page):
    """One-token attention over an e4m3 cache, whose weights enter as two fp16.

    Bound, with A = sum_t p_t |v_t| and one element's half step of bf16, 2^(floor
    log2 |o| - 8), for the output's rounding:
      * the score: d products and additions in fp32, each off by at most 2^-23 of
        the partial sums' bound sum |q_i k_i|, four scalings of 2^-24, and q's
        fp16 below 2^-24 of the head's largest (half a step of it, 2^-25); a
        weight is off by twice that, numerator and sum;
      * the exponential: 2^-21 of it, and its fp32 argument by 2^-24 of |s| / ln 2,
        taken twice (sum and weight): in ds as 2 * 2^-24 |s|;
      * the weight as hi + lo: 2^-22, and below fp16's normal range half a step,
        2^-25, of a unit that is 2^18 times smaller than the reference, which is
        no larger than the largest p_t 2^e_t: with |v| <= 448 2^e and max|v_t| >
        224 2^e_t, 2^-43 * 2 of the largest p_t max|v_t| a token;
      * two MMAs of 16 tokens each and the joins: (2 m / 16 + 64) * 2^-23 of A,
        the sum of the weights as much."""
    n, Hq, d = q.shape
    Hkv = pools[0].shape[1]
    scale = 1 / math.sqrt(d)
    for b, m in enumerate(lens):
        k, v = cu.rows_of(pools, table, b, m, page)
        for h in range(Hq):
            kk, vv, qb = k[:, h * Hkv // Hq], v[:, h * Hkv // Hq], q[b, h].double()
            s = scale * (kk @ qb)
            mag = scale * (kk.abs() @ qb.abs())
            ds = (d + 4) * 2.0 ** -23 * mag + 2.0 ** -25 * scale * qb.abs().max() * kk.abs().sum(-1) + 2 * 2.0 ** -24 * s.abs()
            p = torch.softmax(s, 0)
            want, A = p @ vv, p @ vv.abs()
            # keys that carry no weight do not move the result: their ds counts with their weight
            rel = 2.0 ** -20 + 2.0 ** -22 + 2 * (2 * m / 16 + 64) * 2.0 ** -23
            err = rel * A + 2 * (p * ds) @ vv.abs() + (p @ ds) * 2 * want.abs()
            err = err + 2.0 ** -43 * (p * vv.abs().amax(-1)).max() * 2 * m
            half = torch.exp2(torch.floor(torch.log2(want.abs() + err)) - 8)
            off = (o[b, h].double() - want).abs()
            worst = float((off / (half + err)).max())
            assert worst <= 1, (b, h, m, worst)


@pytest.mark.parametrize("tokens,at,rows", [(600, 3, 1), (4000, 3999, 1), (131072, 70000, 1), (30000, 5, 300)])
def test_small_weights_of_a_quantised_cache(tokens, at, rows):
    """One key 18 nats above the rest, whose value is zero in every other column:
    there the output is what the others leave, each with a weight of 2^-26.  Many
    rows of the batch (over the same pages): each is one block's, with one reference."""
    Hq, Hkv, d, page = 2, 1, 64, 64
    g = gen(tokens + at)
    k, v = randn(tokens, Hkv, d, g=g, scale=0.05), randn(tokens, Hkv, d, g=g).abs()
    q = randn(rows, Hq, d, g=g)
    q[..., 0] = 8.0
    k[:, 0, 0] = 0
    k[at, 0] = 0
    k[at, 0, 0] = 18.0
    v[at, :, ::2] = 0
    pages = -(-tokens // page)
    cache = PagedCache(CacheLayout(Hq, Hkv, d, page_size=page, n_pages=pages, dtype=E4M3))
    table = cu.make_table(1, pages, pages, g)
    cache.write(k, v, table, lengths(tokens))
    o, _ = cache.attn(q, table.expand(rows, -1).contiguous(), lengths(*[tokens] * rows))
    assert cache.device_status() == 0
    some = sorted({0, rows // 2, rows - 1})
    check_weights(o[some], q[some], cache.tensors, table.expand(len(some), -1), [tokens] * len(some), page)


@pytest.mark.parametrize("Hq,Hkv,d", [(32, 8, 128), (4, 2, 64), (24, 2, 128), (16, 1, 64)])
@pytest.mark.parametrize("tokens", [2, 40, 300])
def test_weights_of_a_quantised_cache_keep_their_bits(Hq, Hkv, d, tokens):
    """Ordinary contexts: the output is the 64-bit one, rounded once."""
    page, n = 16, 24
    g = gen(tokens)
    pages = -(-tokens // page)
    pools = cu.make_pools(n * pages, Hkv, page, d, True, g)
    cache = PagedCache(CacheLayout(Hq, Hkv, d, page_size=page, n_pages=n * pages, dtype=E4M3),
                       k_pages=pools[0], v_pages=pools[1], k_exp=pools[2], v_exp=pools[3])
    table, q = cu.make_table(n, pages, n * pages, g), randn(n, Hq, d, g=g)
    o, _ = cache.attn(q, table, lengths(*[tokens] * n))
    check_weights(o, q, pools, table, [tokens] * n, page)


# ------------------------------------------------------------------ lengths beyond the table
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("over,new", [(1, 1), (3, 1), (3, 5), (1, 40), (2 ** 31 - 1, 5), (-7, 2)])
def test_rows_beyond_the_table_are_skipped(over, new, kind):
    """A sequence that grows past its table keeps what it holds: rows whose
    position is behind the table go nowhere, those before it to their place."""
    Hq, Hkv, d, page, per = 4, 2, 64, 8, 4
    cap, n = page * per, 3
    g = gen(new)
    pools = cu.make_pools(n * per, Hkv, page, d, kind == "e4m3", g)
    cache = PagedCache(CacheLayout(Hq, Hkv, d, page_size=page, n_pages=n * per, dtype=pools[0].dtype),
                       k_pages=pools[0], v_pages=pools[1], k_exp=pools[2], v_exp=pools[3])
    table = cu.make_table(n, per, n * per, g)
    raw = [20, min(cap + over, 2 ** 31 - 1) if over > 0 else over, cap]
    q, k, v = randn(n * new, Hq, d, g=g), randn(n * new, Hkv, d, g=g), randn(n * new, Hkv, d, g=g)
    want = [x if x is None else x.double() for x in pools]
    for i, x in enumerate((k, v)):
        vals, exps = cu.quantise(x) if kind == "e4m3" else (x.double(), None)
        for b in range(n):
            for r in range(new):
                pos = raw[b] - new + r
                if not 0 <= pos < cap:
                    continue
                p, at = cu.place(table, page, b, pos)
                want[i][p, :, at] = vals[b * new + r]
                if exps is not None:
                    want[2 + i][p, :, at] = exps[b * new + r]
    rope = QKNormRope(RopeLayout(Hq, Hkv, d, rope_dim=0, norm=False), device="cuda")
    before = [x if x is None else x.view(torch.uint8).clone() for x in pools]
    for call in ("write", "append"):
        for x, was in zip(pools, before):
            if x is not None:
                x.view(torch.uint8).copy_(was)
        if call == "write":
            cache.write(k, v, table, lengths(*raw))
        else:
            assert torch.equal(cache.append(rope, q, k, v, None, table, lengths(*raw)), q)
        for got, ref in zip(pools, want):
            assert got is None or torch.equal(got.double(), ref)
        assert cache.device_status() == 2 and cache.device_status() == 0


# ------------------------------------------------------------------ tensors without an address
def test_transforms_raise_and_leave_the_process_and_the_calls_alone():
    Hq, Hkv, d, page = 4, 2, 64, 16
    g = gen(7)
    q, k = randn(3, 2, Hq, d, g=g), randn(3, 2, Hkv, d, g=g)
    cache = PagedCache(CacheLayout(Hq, Hkv, d, page_size=page, n_pages=4))
    rope = QKNormRope(RopeLayout(Hq, Hkv, d, rope_dim=0), device="cuda")
    table, lens = cu.make_table(2, 2, 4, g), lengths(20, 30)
    cache.write(k[0], k[1], table, lens)
    want = cache.attn(q[0], table, lens)
    for call in (lambda x, y: rope.apply(x, y), lambda x, y: cache.write(y, y, table, lens),
                 lambda x, y: cache.append(rope, x, y, y, None, table, lens), lambda x, y: cache.attn(x, table, lens)):
        with pytest.raises(RuntimeError):
            torch.vmap(call)(q, k)
        with pytest.raises(RuntimeError):
            torch.func.jvp(lambda x: call(x, x[:, :Hkv]), (q[0],), (q[1],))
    with pytest.raises(RuntimeError):
        torch.vmap(lambda t: cache.read(t, lens, 4))(torch.stack([table] * 3))
    cache.write(k[0], k[1], table, lens)
    got = cache.attn(q[0], table, lens)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------ kept tensors
def test_replaced_memory_of_kept_tensors_is_followed():
    """``.data`` of a weight, a table of frequencies, a pool or a workspace may be
    replaced; the next call takes what is there then."""
    Hq, Hkv, d, page, n = 4, 2, 64, 16, 3
    g = gen(8)
    w1, w2 = randn(d, g=g), randn(d, g=g)
    f1, f2 = (torch.rand(d // 2, generator=g, device="cuda") for _ in range(2))
    q, k = randn(n, Hq, d, g=g), randn(n, Hkv, d, g=g)
    pos = torch.arange(5, 5 + n, dtype=torch.int32, device="cuda")
    lay = RopeLayout(Hq, Hkv, d)
    want = [QKNormRope(lay, f, w, w).apply(q, k, pos) for f, w in ((f1, w1), (f2, w2))]
    w, f = torch.nn.Parameter(w1.clone(), requires_grad=False), f1.clone()
    rope = QKNormRope(lay, f, w, w)
    assert rope.q_weight is w
    old = [w.data, f.data]
    for i in (0, 1):
        assert all(torch.equal(a, b) for a, b in zip(rope.apply(q, k, pos), want[i]))
        w.data, f.data = w2.clone(), f2.clone()
        del old[:]
    w.data = w2.float()
    with pytest.raises(ValueError):
        rope.apply(q, k, pos)
    w.data = w2.cpu()
    with pytest.raises(ValueError):
        rope.apply(q, k, pos)
    w.data, f.data = w2, f2[:5]
    with pytest.raises(ValueError):
        rope.apply(q, k, pos)

    for dtype in (BF16, E4M3):
        lay = CacheLayout(Hq, Hkv, d, page_size=page, n_pages=4, dtype=dtype)
        cache, other = PagedCache(lay), PagedCache(lay)
        table, lens = torch.tensor([[1, 3]], dtype=torch.int32, device="cuda"), lengths(n)
        cache.write(k, k, table, lens)
        other.write(-k, -k, table, lens)
        for t, x in zip((*cache.tensors, cache.workspace), (*other.tensors, other.workspace)):
            t.data = x.clone()
        got = cache.read(table, lens, n)
        assert all(torch.equal(a, b) for a, b in zip(got, other.read(table, lens, n)))
        assert torch.equal(cache.attn(q[:1], table, lens)[0], other.attn(q[:1], table, lens)[0])
        cache.attn(q[:1], table, lengths(-1))
        assert cache.device_status() == 2 and other.device_status() == 0
        cache.k_pages.data = cache.k_pages[:2]
        with pytest.raises(ValueError):
            cache.write(k, k, table, lens)
        cache.k_pages.data = other.k_pages
        cache.workspace.data = cache.workspace[:256]
        with pytest.raises(SpavaError):
            cache.attn(q[:1], table, lens)


# ------------------------------------------------------------------ empty batches
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_an_empty_batch_does_nothing(kind):
    Hq, Hkv, d = 4, 2, 64
    cache = PagedCache(CacheLayout(Hq, Hkv, d, page_size=16, n_pages=4, dtype=BF16 if kind == "bf16" else E4M3))
    rope = QKNormRope(RopeLayout(Hq, Hkv, d), torch.ones(d // 2, device="cuda"))
    table, lens = torch.zeros((2, 3), dtype=torch.int32, device="cuda")[:0], lengths(1, 2)[:0]
    q, k = randn(2, Hq, d, g=gen())[:0], randn(2, Hkv, d, g=gen())[:0]
    pos = torch.empty((1, 0), dtype=torch.int32, device="cuda")
    assert [x.shape for x in rope.apply(q, k, pos)] == [(0, Hq, d), (0, Hkv, d)]
    cache.write(k, k, table, lens)
    assert cache.append(rope, q, k, k, pos, table, lens).shape == (0, Hq, d)
    assert [x.shape for x in cache.read(table, lens, 7)] == [(0, 7, Hkv, d)] * 2
    o, lse = cache.attn(q, table, lens)
    assert o.shape == (0, Hq, d) and lse.shape == (Hq, 0)
    assert not any(x.view(torch.uint8).any() for x in cache.tensors) and cache.device_status() == 0
    with pytest.raises(ValueError):      # rows without a sequence
        cache.write(randn(1, Hkv, d, g=gen()), randn(1, Hkv, d, g=gen()), table, lens)


# ------------------------------------------------------------------ the status word
def test_a_short_workspace_has_no_clean_status():
    cache = PagedCache(CacheLayout(4, 2, 64, page_size=16, n_pages=4))
    assert cache.device_status() == 0 == cache.device_status(workspace=cache.new_workspace())
    with pytest.raises(SpavaError) as e:
        cache.device_status(workspace=torch.zeros(255, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 1


# ------------------------------------------------------------------ extreme exponents
@pytest.mark.parametrize("k_exp,q_exp", [(124, -124), (124, -130), (100, -108), (-124, 124), (-133, 126), (60, -60)])
@pytest.mark.parametrize("tokens", [20, 900, 20000])
def test_scores_of_opposite_exponents(k_exp, q_exp, tokens):
    """Keys and queries next to the ends of bf16, products of ordinary size: the
    scores are those of the products."""
    Hq, Hkv, d, page = 4, 2, 64, 16
    g = gen(tokens)
    k, v = randn(tokens, Hkv, d, g=g), randn(tokens, Hkv, d, g=g)
    k = torch.ldexp(k.float(), torch.tensor(k_exp, device="cuda")).to(BF16)
    q = torch.ldexp(randn(1, Hq, d, g=g).float(), torch.tensor(q_exp, device="cuda")).to(BF16)
    assert k.isfinite().all() and k.any() and q.any()
    pages = -(-tokens // page)
    cache = PagedCache(CacheLayout(Hq, Hkv, d, page_size=page, n_pages=pages, dtype=E4M3))
    table, lens = cu.make_table(1, pages, pages, g), lengths(tokens)
    cache.write(k, v, table, lens)
    o, lse = cache.attn(q, table, lens)
    cu.check_attn(o, lse, q, cache.tensors, table, [tokens], page)


@pytest.mark.parametrize("tokens", [20, 900, 131072])
def test_outputs_next_to_the_smallest(tokens):
    """Values of 2^-117: the average of many keeps its bits."""
    Hq, Hkv, d, page = 4, 2, 64, 16
    g = gen(tokens)
    k, v = randn(tokens, Hkv, d, g=g, scale=0.1), randn(tokens, Hkv, d, g=g).abs()
    v = torch.ldexp(v.float(), torch.tensor(-117, device="cuda")).to(BF16)
    q = randn(1, Hq, d, g=g)
    pages = -(-tokens // page)
    cache = PagedCache(CacheLayout(Hq, Hkv, d, page_size=page, n_pages=pages, dtype=E4M3))
    table, lens = cu.make_table(1, pages, pages, g), lengths(tokens)
    cache.write(k, v, table, lens)
    o, lse = cache.attn(q, table, lens)
    cu.check_attn(o, lse, q, cache.tensors, table, [tokens], page)


# ------------------------------------------------------------------ blocks of many tokens
def full_pools(e4m3, *shape):
    out = [torch.zeros(shape, dtype=torch.uint8 if e4m3 else BF16, device="cuda") for _ in range(2)]
    if e4m3:
        return [x.view(E4M3) for x in out] + [torch.zeros(shape[:3], dtype=torch.int8, device="cuda") for _ in range(2)]
    return out + [None, None]


def check_pools(pools, k, v, table, lens, page, new):
    """Pools that held zeros, after a write of k and v [sequences * new, Hkv, d]."""
    n = len(lens)
    pos = torch.tensor(lens, device="cuda")[:, None] - new + torch.arange(new, device="cuda")
    p, r = table.long().gather(1, pos // page).flatten(), (pos % page).flatten()
    for i, x in enumerate((k, v)):
        vals, exps = (x.double(), None) if pools[2] is None else cu.quantise(x)
        assert torch.equal(pools[i][p, :, r].double(), vals)
        if exps is not None:
            assert torch.equal(pools[2 + i][p, :, r].double(), exps)
        rest = pools[i].view(torch.uint8).clone()
        rest[p, :, r] = 0
        assert not rest.any()
    assert len({*zip(p.tolist(), r.tolist())}) == n * new


# Rows around the thresholds from which a block takes twice the tokens (2368, 4736,
# ... rows), up to 32 of them, with a remainder in the last block.
MANY = [(2369, 28, 4, 128), (4737, 28, 4, 128), (38001, 28, 4, 128), (18945, 2, 1, 64), (75777, 2, 1, 64), (9473, 4, 2, 128),
        (5001, 40, 8, 64), (35, 1, 1, 64)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows,Hq,Hkv,d", MANY)
def test_blocks_of_many_tokens(rows, Hq, Hkv, d, kind):
    """Norm with rotation, append, write and read of as many rows as a prefill has."""
    e4m3, page = kind == "e4m3", 48
    g = gen(rows)
    qkv = randn(rows, (Hq + 2 * Hkv) * d, g=g)
    q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([Hq * d, Hkv * d, Hkv * d], 1))
    pos = torch.randint(0, 1 << 20, (2, rows), generator=g, device="cuda", dtype=torch.int32)
    sections, freq = (d // 8, d // 2 - d // 8), (1e6 ** (-torch.arange(d // 2, device="cuda") / (d // 2))).float()
    qw, kw = randn(d, g=g), randn(d, g=g)
    rope = QKNormRope(RopeLayout(Hq, Hkv, d, sections=sections), freq, qw, kw)
    qo, ko = rope.apply(q, k, pos)
    for got, x, w in ((qo, q, qw), (ko, k, kw)):
        cu.check_norm_rope(got, cu.norm_rope(x, w, pos, freq, d, False, sections, True, 1e-6))
    # the rows as those of one sequence, or of as many as divide them
    n = next(n for n in (7, 5, 3, 1) if rows % n == 0)
    new = rows // n
    per = -(-(new + 11) // page)
    table = cu.make_table(n, per, n * per + 2, g)
    lens = [new + 11 - b for b in range(n)]
    for call in ("write", "append"):
        pools = full_pools(e4m3, n * per + 2, Hkv, page, d)
        cache = PagedCache(CacheLayout(Hq, Hkv, d, page_size=page, n_pages=n * per + 2, dtype=pools[0].dtype),
                           k_pages=pools[0], v_pages=pools[1], k_exp=pools[2], v_exp=pools[3])
        if call == "write":
            cache.write(ko, v, table, lengths(*lens))
        else:
            assert torch.equal(cache.append(rope, q, k, v, pos, table, lengths(*lens)), qo)
        check_pools(pools, ko, v, table, lens, page, new)
    kr, vr = cache.read(table, lengths(*lens), new + 13, first=1)
    for b, m in enumerate(lens):
        ks, vs = cu.rows_of(pools, table, b, m, page)
        for got, ref in ((kr, ks), (vr, vs)):
            assert torch.equal(got[b, :m - 1].double(), ref[1:]) and not got[b, m - 1:].any()
    assert cache.device_status() == 0


def test_tensors_whose_memory_was_given_back_are_refused():
    """A weight without its storage is not a missing weight, whose place ones take."""
    g = gen(9)
    q, k, w = randn(3, 4, 64, g=g), randn(3, 2, 64, g=g), randn(64, g=g)
    rope = QKNormRope(RopeLayout(4, 2, 64, rope_dim=0), None, w, w)
    rope.apply(q, k)
    w.untyped_storage().resize_(0)
    with pytest.raises(ValueError):
        rope.apply(q, k)
    cache = PagedCache(CacheLayout(4, 2, 64, page_size=16, n_pages=4))
    table, lens = cu.make_table(1, 2, 4, g), lengths(3)
    cache.write(k, k, table, lens)
    cache.v_pages.untyped_storage().resize_(0)
    with pytest.raises(ValueError):
        cache.read(table, lens, 3)
