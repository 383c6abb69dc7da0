"""Plain 64-bit implementations of the answering side's operators, written from
their formulas, and the error bounds that the kernels are held to.

Bounds.  One rounding to bf16 is off by at most 2^-8 of the value, to fp16 by
2^-11, to e4m3 by 2^-4 (half a step), one fp32 operation by 2^-24."""
import math

import torch

E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------ norm and rotation
def norm_rope(x, w, positions, freq, rope, interleaved, sections, norm, eps):
    """x [rows, heads, d], positions [axes, rows]; 64 bits, unrounded."""
    y = x.double()
    if norm:
        y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt()
        if w is not None:
            y = y * w.double()
    if rope:
        axis = [a for a, n in enumerate(sections) for _ in range(n)]
        angle = positions.double()[axis].t() * freq.double()          # [rows, rope / 2]
        cos, sin = angle.cos()[:, None], angle.sin()[:, None]
        lo = slice(0, rope, 2) if interleaved else slice(0, rope // 2)
        hi = slice(1, rope, 2) if interleaved else slice(rope // 2, rope)
        a, b = y[..., lo].clone(), y[..., hi].clone()
        y[..., lo], y[..., hi] = a * cos - b * sin, b * cos + a * sin
    return y


def check_norm_rope(got, want):
    """bf16 output: half a step of the value, and the fp32 work before it: the
    norm's sum of at most 128 squares (rounding 128 * 2^-24 relative, halved by
    the root), half a dozen more roundings, and a cosine off by at most 2^-20
    (its angle, under 1e-6, and its own error), all relative to the pair's
    larger element, which the head's largest bounds."""
    top = want.abs().amax(-1, keepdim=True)
    off = (got.double() - want).abs()
    bound = 2.0 ** -8 * want.abs() + (64 + 8) * 2.0 ** -24 * 2 * top + 2 * 2.0 ** -20 * top
    assert (off <= bound).all(), float((off - bound).max())


# ------------------------------------------------------------------ cache rows
def quantise(x):
    """(values, exponents) of rows of x, in 64 bits: the smallest e >= -120 with
    max|x| <= 448 * 2^e over the finite elements, values rounded to four
    significant bits, to multiples of 2^-9 below 2^-6, ties to even."""
    y = x.double()
    fine = y.isfinite()
    top = torch.where(fine, y, 0.0).abs().amax(-1)
    e = torch.full_like(top, -120.0)
    for step in range(-119, 121):
        e = torch.where(top > 448 * 2.0 ** (step - 1), float(step), e)
    z = y * torch.exp2(-e)[..., None]
    mag = z.abs().clamp(min=2.0 ** -6)
    unit = torch.exp2(torch.floor(torch.log2(mag)) - 3)
    z = torch.where(fine, torch.round(z / unit) * unit, math.nan)
    return z, e


def place(table, page, b, pos):
    return int(table[b, pos // page]), pos % page


def written(pools, k, v, table, lens, page, new):
    """64-bit copies of the pools after a write (exponents None for bf16)."""
    kp, vp, ke, ve = pools
    out = [kp.double().cpu().clone(), vp.double().cpu().clone(),
           None if ke is None else ke.cpu().clone(), None if ve is None else ve.cpu().clone()]
    table, lens, k, v = table.cpu(), lens.tolist(), k.cpu(), v.cpu()
    for i, x in enumerate((k, v)):
        vals, exps = (x.double(), None) if ke is None else quantise(x)
        for b, n in enumerate(lens):
            for r in range(new):
                pos = n - new + r
                if pos < 0:
                    continue
                p, o = place(table, page, b, pos)
                out[i][p, :, o] = vals[b * new + r]
                if exps is not None:
                    out[2 + i][p, :, o] = exps[b * new + r].to(torch.int8)
    return out


def rows_of(pools, table, b, n, page):
    """Keys and values [n, Hkv, d] of positions [0, n) of sequence b in 64 bits."""
    pos = torch.arange(n, device=table.device)
    p, o = table[b][pos // page].long(), pos % page
    got = []
    for pool, exps in ((pools[0], pools[2]), (pools[1], pools[3])):
        if exps is None:
            got.append(pool[p, :, o].double())
        else:
            x = pool.view(torch.uint8)[p, :, o].view(E4M3).double()
            got.append(x * torch.exp2(exps[p, :, o].double())[..., None])
    return got


# ------------------------------------------------------------------ attention
def check_attn(o, lse, q, pools, table, lens, page, scale=None, keep=None):
    """o [n, Hq, d], lse [Hq, n] of one-token attention against 64 bits.

    ``keep(b)``: mask of the positions that count (all of them if None).

    Bound.  With A = sum_t p_t |v_t| (p the softmax, in 64 bits):
      * a score is a sum of d products in fp32, each addition off by at most
        2^-23 of a partial sum (the tensor core may truncate), scaled by three
        roundings: ds = (d + 4) * 2^-23 * scale * sum_i |q_i k_i|; fp16 q of the
        e4m3 path: 2^-25 of the head's largest |q| per element, and where q is
        that small only;  p is then off by 2 ds relative (numerator and sum),
        2^-21 for the exponential and its fp32 argument of magnitude up to
        |s| / ln 2 (2^-24 of it, twice);
      * P is rounded to two bf16 (2^-16) or one fp16 (2^-11, and 2^-25 of the
        largest product of weight and value scale below fp16's normal range);
      * n additions in fp32 of O and of the sum, and the joins: (n / 16 + 64) *
        2^-23 of A each;
      * the output: 2^-8 of the value."""
    n, Hq, d = q.shape
    e4m3 = pools[2] is not None
    scale = 1 / math.sqrt(d) if scale is None else scale
    Hkv = pools[0].shape[1]
    per = Hq // Hkv
    for b, m in enumerate(lens):
        if m > 0:
            k, v = rows_of(pools, table, b, m, page)
            if keep is not None:
                mask = keep(b)
                k, v = k[mask], v[mask]
        if m <= 0 or k.shape[0] == 0:
            assert (o[b] == 0).all() and (lse is None or (lse[:, b] == -math.inf).all())
            continue
        m = k.shape[0]
        kk, vv = (x.repeat_interleave(per, 1) for x in (k, v))     # [m, Hq, d]
        qb = q[b].double()
        s = scale * (qb * kk).sum(-1).t()                         # [Hq, m]
        mag = scale * (qb.abs() * kk.abs()).sum(-1).t()
        ds = (d + 4) * 2.0 ** -23 * mag
        if e4m3:
            ds = ds + 2.0 ** -25 * scale * qb.abs().amax(-1)[:, None] * kk.abs().sum(-1).t()
        ds = (ds + 2 * 2.0 ** -24 * s.abs()).amax(-1)             # [Hq]
        want_lse = torch.logsumexp(s, -1)
        p = torch.exp(s - want_lse[:, None])
        want = torch.einsum("hm,mhd->hd", p, vv)
        A = torch.einsum("hm,mhd->hd", p, vv.abs())
        rel = 2 * ds + 2.0 ** -20 + (2.0 ** -11 if e4m3 else 2.0 ** -16) + 2 * (m / 16 + 64) * 2.0 ** -23
        bound = 2.0 ** -8 * want.abs() + rel[:, None] * A
        if e4m3:
            # weights below fp16's normal range: an absolute 2^-25 of the reference's
            bound = bound + 2.0 ** -25 * (p[..., None] * vv.abs().amax(-1).t()[..., None]).amax(1) * 2 * m
        off = (o[b].double() - want).abs()
        assert o[b].isfinite().all()
        assert (off <= bound).all(), (b, m, float((off / bound).max()))
        if lse is not None:
            off = (lse[:, b].double() - want_lse).abs()
            lb = ds + 2.0 ** -20 + (m / 16 + 64) * 2.0 ** -23 + 2.0 ** -22 * want_lse.abs()
            assert (off <= lb).all(), (b, m, float((off / lb).max()))


# ------------------------------------------------------------------ inputs
def make_pools(n_pages, Hkv, page, d, e4m3, g, fill="rows", device="cuda"):
    """Pools of random rows (keys ~ N(0,1) with a page's own offset, values ~ N(0,1))."""
    shape = (n_pages, Hkv, page, d)
    out = []
    for i in range(2):
        x = torch.randn(shape, generator=g, device=device)
        if i == 0:
            x = x + 0.5 * torch.randn((n_pages, Hkv, 1, d), generator=g, device=device)
        out.append(x)
    if not e4m3:
        return [x.to(torch.bfloat16) for x in out] + [None, None]
    vals, exps = [], []
    for x in out:
        z, e = quantise(x)
        vals.append(z.float().to(E4M3))
        exps.append(e.to(torch.int8))
    return vals + exps


def make_table(n, max_pages, n_pages, g, device="cuda"):
    return torch.randperm(n_pages, generator=g, device=device)[:n * max_pages].to(torch.int32).view(n, max_pages)
