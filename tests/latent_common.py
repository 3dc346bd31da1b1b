"""Plain 64-bit forms of the operators around the latent cache, written from their formulas (torch float64)."""

from __future__ import annotations

import math

import torch


def freqs64(R, base=10000.0, scaling="none", factor=1.0, original_len=4096, beta_fast=32.0, beta_slow=1.0):
    f = [base ** (-2.0 * i / R) for i in range(R // 2)]
    if scaling == "none":
        return f, 1.0
    if scaling == "linear":
        return [v / factor for v in f], 1.0
    d = lambda beta: R * math.log(original_len / (2 * math.pi * beta)) / (2 * math.log(base))
    low, high = max(math.floor(d(beta_fast)), 0), min(math.ceil(d(beta_slow)), R - 1)
    out = []
    for i, v in enumerate(f):
        r = min(max((i - low) / max(high - low, 0.001), 0.0), 1.0)
        out.append((1 - r) * v + r * v / factor)
    return out, 0.1 * math.log(factor) + 1.0


def norm64(x, kind, weight, bias, eps):
    x = x.double()
    if kind == "none":
        return x
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if weight is not None:
        y = y * weight.double()
    return y if bias is None else y + bias.double()


def rotate64(y, pos, freqs, off, layout, mul):
    """y [T, ..., D] float64; freqs float64 [R / 2]."""
    n = freqs.numel()
    a = pos.double().view(-1, *[1] * (y.dim() - 1)) * freqs
    c, s = mul * torch.cos(a), mul * torch.sin(a)
    y = y.clone()
    if layout == "half":
        iu = off + torch.arange(n, device=y.device)
        iv = iu + n
    else:
        iu = off + 2 * torch.arange(n, device=y.device)
        iv = iu + 1
    u, v = y[..., iu], y[..., iv]
    y[..., iu], y[..., iv] = u * c - v * s, v * c + u * s
    return y


def rows_tol(y, mul=1.0):
    """What a result may be off by: half a bf16 step (2^-8 of it) and the 32-bit arithmetic.  The latter, for D <= 1024:
    sums of at most 32 terms in sequence and 5 levels of shuffles are off by 37 * 2^-24 of the sum of magnitudes, a norm
    by about half that and five roundings, a centred value of a row whose mean is below its spread by twice that, and a
    rotation by four roundings of |u| + |v| (sin and cos 2 ulp, the reduced angle half an ulp of pi): below 128 * 2^-24
    of the row's largest magnitude in all (times mul).  2^-134: half the smallest bf16 step."""
    return y.abs() * 2.0 ** -8 + 2.0 ** -134 + 2.0 ** -17 * max(mul, 1.0) * y.abs().amax(-1, keepdim=True)


def check_rows(got, y, mul=1.0):
    bad = (got.double() - y).abs() > rows_tol(y, mul)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"


def check_codes(codes, scale, y, mul=1.0):
    """e4m3 codes and scales against y: half a step (2^-4 of the value, 2^-10 among the subnormals), the quotient's
    32-bit error 448 * 2^-17 mul."""
    amax = y.abs().amax(-1)
    want = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
    assert ((scale.double() - want).abs() <= want * 2.0 ** -16 * max(mul, 1.0)).all()
    q = y / want.unsqueeze(-1)
    v = codes.view(torch.float8_e4m3fn).double()
    tol = torch.maximum(q.abs() * 2.0 ** -4, torch.full_like(q, 2.0 ** -10)) + 448 * 2.0 ** -16 * max(mul, 1.0)
    bad = (v - q).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} codes off, first at {bad.nonzero()[0].tolist()}"


def prefix64(q, prefix, scale, pages, table, own_len, b):
    """Query b: out [H, 512], lse [H], the mean magnitude of its values [H, 512], the largest error of a logit."""
    keys = [] if prefix is None else [prefix]
    if own_len is not None:
        page = pages.shape[1]
        i = torch.arange(int(own_len[b]), device=q.device)
        keys.append(pages.reshape(-1, 576)[table[b].long()[i // page] * page + i % page])
    k = torch.cat(keys).double() if keys else q.new_zeros(0, 576).double()
    qb = q[b].double()
    if k.shape[0] == 0:
        z = qb.new_zeros(qb.shape[0], 512)
        return z, torch.full_like(z[:, 0], -math.inf), z, 0.0
    z = scale * (qb @ k.T)
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    # fp32 accumulation of 576 exact products in any order, truncated adds included: 576 * 2^-23 of the magnitudes
    dz = abs(scale) * float((qb.abs() @ k.abs().T).max()) * 576 * 2.0 ** -23
    return p @ k[:, :512], lse, p @ k[:, :512].abs(), dz


def check_prefix(out, lse, q, prefix, scale, pages=None, table=None, own_len=None, rows=None):
    """out: half a bf16 step of the result; each probability half a bf16 step, off by e^dz - 1 <= 1.02 dz with its sum
    the same again, and 2^-12 for the exponentials (2^-21 each) and the 32-bit sums; lse: dz and 32-bit roundings."""
    for b in rows if rows is not None else range(q.shape[0]):
        o, l, mag, dz = prefix64(q, prefix, scale, pages, table, own_len, b)
        tol = 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2.1 * dz + 2.0 ** -12) * mag * (1 + 2.0 ** -8)
        bad = ~((out[b].double() - o).abs() <= tol)
        assert not bad.any(), f"query {b}: {int(bad.sum())} off, first at {bad.nonzero()[0].tolist()}"
        if lse is not None:
            fin = torch.isfinite(l)
            assert torch.equal(torch.isfinite(lse[b]), fin) and bool((lse[b][~fin] == -math.inf).all())
            if fin.any():
                err = (lse[b].double() - l)[fin].abs()
                assert (err <= dz + 2.0 ** -18 * (1 + l[fin].abs())).all(), f"query {b}: lse off by {float(err.max())}"
