"""The operators around the latent cache against their formulas in 64 bits, and a run of them together."""

import math

import numpy as np
import pytest
import torch

import sparse_long_context_lightning_b200 as lsa
from latent_common import check_codes, check_prefix, check_rows, norm64, prefix64, rotate64
from oracle import lsa_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _status_ok():
    lsa.lsa_device_status()


# ------------------------------------------------------------------------------------------------ norm_rope


def _weights(g, norm, D, bias=True):
    w = 1 + 0.2 * _randn(g, D) if norm != "none" else None
    return w, (0.1 * _randn(g, D) if norm == "layer" and bias else None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H,D,norm,off,R,layout", [
    (1, 1, 8, "none", 0, 0, "half"), (3, 2, 16, "rms", 0, 16, "half"), (5, 3, 24, "layer", 8, 16, "interleaved"),
    (17, 64, 128, "rms", 0, 64, "half"), (9, 64, 128, "layer", 64, 64, "half"), (4, 33, 128, "rms", 0, 128, "interleaved"),
    (33, 5, 64, "none", 0, 64, "half"), (7, 16, 32, "rms", 0, 32, "interleaved"), (2, 128, 576, "none", 512, 64, "interleaved"),
    (3, 7, 576, "rms", 512, 64, "half"), (6, 4, 192, "layer", 128, 64, "half"), (2, 3, 96, "rms", 32, 64, "half"),
    (2, 3, 40, "layer", 8, 32, "half"), (1, 2, 1024, "layer", 0, 1024, "half"), (2, 1, 1024, "rms", 8, 992, "interleaved"),
    (1, 300, 128, "rms", 0, 64, "half"), (301, 1, 128, "layer", 0, 64, "half"), (70, 1, 32, "none", 0, 32, "half"),
    (2000, 64, 128, "rms", 0, 64, "half"), (1500, 128, 64, "layer", 0, 64, "interleaved")])
def test_norm_rope(T, H, D, norm, off, R, layout, fp8):
    g = _gen(T + 7 * H + D)
    x = (1.5 * _randn(g, T, H, D) + 0.25).bfloat16()
    w, b = _weights(g, norm, D)
    pos = torch.randint(0, 10 ** 7, (T,), generator=g, device=DEV)
    freqs, mul = lsa.lsa_rope_freqs(R, scaling="yarn", factor=32.0) if R else (None, 1.0)
    y = torch.empty(T, H, D, dtype=torch.uint8 if fp8 else torch.bfloat16, device=DEV)
    sc = torch.empty(T, H, device=DEV) if fp8 else None
    lsa.lsa_norm_rope(x, y, pos if R else None, freqs, norm=norm, weight=w, bias=b, eps=1e-5, rope_off=off, layout=layout,
                      mul=mul, y_scale=sc)
    want = norm64(x, norm, w, b, 1e-5)
    if R:
        want = rotate64(want, pos, freqs, off, layout, mul)
    check_codes(y, sc, want, mul) if fp8 else check_rows(y, want, mul)


@pytest.mark.parametrize("norm", ["none", "rms", "layer"])
def test_norm_rope_special_rows(norm):
    """Rows of zeros, constant rows, rows of the type's largest and smallest values, without weights too."""
    T, D = 6, 128
    x = torch.zeros(T, 1, D, dtype=torch.bfloat16, device=DEV)
    x[1], x[2], x[3, 0, 5], x[4] = 3.0, -1e-30, 1.0, torch.finfo(torch.bfloat16).tiny
    x[5] = _randn(_gen(1), 1, D).bfloat16() * 1e15
    pos = torch.arange(T, device=DEV) - 2  # negative positions too
    freqs, mul = lsa.lsa_rope_freqs(64)
    for weighted in (False, True):
        w, b = _weights(_gen(2), norm, D) if weighted else (None, None)
        want = rotate64(norm64(x, norm, w, b, 1e-6), pos, freqs, 0, "half", mul)
        y = torch.empty_like(x)
        lsa.lsa_norm_rope(x, y, pos, freqs, norm=norm, weight=w, bias=b, eps=1e-6, layout="half")
        check_rows(y, want)
        c, sc = torch.empty(T, 1, D, dtype=torch.uint8, device=DEV), torch.empty(T, 1, device=DEV)
        lsa.lsa_norm_rope(x[:4], c[:4], pos[:4], freqs, norm=norm, weight=w, bias=b, eps=1e-6, layout="half",
                          y_scale=sc[:4])
        if norm != "none":  # 1e-30 / 448 and its quotients are ordinary numbers, but only as far as the norm keeps them
            check_codes(c[:4], sc[:4], want[:4])
        else:
            check_codes(c[[0, 1, 3]], sc[[0, 1, 3]], want[[0, 1, 3]])
        assert float(sc[0]) == 1.0 or (norm == "layer" and weighted)


def test_codes_of_rows_whose_scale_has_no_reciprocal():
    """Rows so small that 1 / scale overflows: zeros stay zero and the others are the scale's multiples all the same."""
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=DEV)
    x[0, 0, ::3] = 1e-37
    x[0, 1] = torch.finfo(torch.bfloat16).tiny * (1 + torch.arange(64, device=DEV) / 64)
    x[1, 0] = -3e-34 * (1 + torch.arange(64, device=DEV) / 64)
    x[2, 1, 7] = 2e-36
    y, sc = torch.empty(3, 2, 64, dtype=torch.uint8, device=DEV), torch.empty(3, 2, device=DEV)
    lsa.lsa_norm_rope(x, y, y_scale=sc)
    v = y.view(torch.float8_e4m3fn).double()
    # a scale near 2^-133 has 16 bits (2^-149 is the smallest step), so quotients are off by 2^-16 more
    q = x.double() / sc.double()[..., None]
    assert ((v - q).abs() <= torch.maximum(q.abs() * (2.0 ** -4 + 2.0 ** -15), torch.tensor(2.0 ** -10, device=DEV))).all()
    want = x.double().abs().amax(-1) / 448
    assert ((sc.double() - want)[want > 0].abs() <= 2.0 ** -149 + 2.0 ** -22 * want[want > 0]).all()
    assert not v[x == 0].any() and bool((sc[want == 0] == 1).all())


def test_norm_rope_strides_and_in_place():
    """A head slice of a wider projection, transposed heads, a broadcast input, and the result over the input."""
    g, T, H, D = _gen(3), 37, 6, 64
    freqs, mul = lsa.lsa_rope_freqs(64)
    pos = torch.randint(0, 100000, (T,), generator=g, device=DEV)
    wide = _randn(g, T, H, 640).bfloat16()
    heads_first = _randn(g, H, T, D).bfloat16().transpose(0, 1)
    one = _randn(g, T, 1, D).bfloat16().expand(T, H, D)
    every = _randn(g, 1, H, D).bfloat16().expand(T, H, D)
    for x in (wide[:, :, 512:576], heads_first, one, every):
        y = torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV)
        lsa.lsa_norm_rope(x, y, pos, freqs, norm="rms")
        check_rows(y, rotate64(norm64(x, "rms", None, None, 1e-6), pos, freqs, 0, "interleaved", mul))
    # the rotary part written between other columns, which stay
    full = _randn(g, T, H, 576).bfloat16()
    before = full.clone()
    lsa.lsa_norm_rope(wide[:, :, :64], full[:, :, 512:], pos, freqs)
    check_rows(full[:, :, 512:], rotate64(wide[:, :, :64].double(), pos, freqs, 0, "interleaved", mul))
    assert torch.equal(full[:, :, :512], before[:, :, :512])
    for layout in ("half", "interleaved"):
        for norm in ("none", "layer"):
            x = before.clone()
            want = rotate64(norm64(x, norm, None, None, 1e-6), pos, freqs, 512, layout, mul)
            lsa.lsa_norm_rope(x, x, pos, freqs, norm=norm, rope_off=512, layout=layout)
            check_rows(x, want)
            if norm == "none":
                assert torch.equal(x[..., :512], before[..., :512])


@pytest.mark.parametrize("T,H,t,h", [(3, 2, 2 * 64, 3 * 64), (5, 4, 64, 5 * 64), (4, 5, 5 * 64, 64), (2, 3, 64, 200),
                                     (7, 2, 208, 72), (1, 6, 0, 64), (6, 1, 64, 0)])
def test_norm_rope_interleaved_outputs(T, H, t, h):
    """Rows of y that lie between each other without sharing an element are written; what lies between them stays."""
    g, D = _gen(T + h), 64
    at = torch.tensor(sorted(i * t + j * h for i in range(T) for j in range(H)))
    assert T * H == 1 or int((at[1:] - at[:-1]).min()) >= D
    flat = _randn(g, int(at.max()) + D + 40).bfloat16()
    before, x = flat.clone(), _randn(g, T, H, D).bfloat16()
    y = flat.as_strided((T, H, D), (t, h, 1))
    freqs, mul = lsa.lsa_rope_freqs(64)
    pos = torch.arange(T, device=DEV)
    lsa.lsa_norm_rope(x, y, pos, freqs, norm="rms")
    check_rows(y, rotate64(norm64(x, "rms", None, None, 1e-6), pos, freqs, 0, "interleaved", mul))
    rest = torch.ones_like(flat, dtype=torch.bool)
    rest.as_strided((T, H, D), (t, h, 1)).fill_(False)
    assert torch.equal(flat[rest], before[rest])
    with pytest.raises(lsa.LsaError):
        lsa.lsa_norm_rope(x.expand(T, H, D).repeat(1, 2, 1), flat.as_strided((T, 2 * H, D), (t or 8, 32, 1)), pos, freqs)


def test_norm_rope_refusals():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device=DEV)
    y, freqs = torch.empty_like(x), lsa.lsa_rope_freqs(64)[0]
    pos = torch.arange(4, device=DEV)
    for kw in (dict(pos=pos), dict(freqs=freqs), dict(pos=pos.int(), freqs=freqs), dict(pos=pos[:3], freqs=freqs),
               dict(pos=pos, freqs=freqs.float()), dict(norm="rms", weight=torch.ones(32, device=DEV)), dict(norm="l2"),
               dict(norm="rms", weight=torch.ones(64)), dict(layout="both"), dict(y_scale=torch.ones(4, 2, device=DEV)),
               dict(norm="rms", bias=torch.ones(64, device=DEV))):
        with pytest.raises(lsa.LsaError):
            lsa.lsa_norm_rope(x, y, **kw)
    for bad in (torch.empty(4, 2, 32, dtype=torch.bfloat16, device=DEV), y.float(), y[:, :1].expand(4, 2, 64),
                torch.empty(4, 64, 2, dtype=torch.bfloat16, device=DEV).transpose(1, 2)):
        with pytest.raises(lsa.LsaError):
            lsa.lsa_norm_rope(x, bad)


# ------------------------------------------------------------------------------------------------ cache_append


@pytest.mark.parametrize("keys", ["none", "bf16", "e4m3"])
@pytest.mark.parametrize("T,d_I,k_norm,k_off,k_layout,skip", [
    (1, 128, "layer", 0, "half", 0), (2, 64, "rms", 0, "interleaved", 2), (16, 128, "rms", 64, "half", 0),
    (513, 128, "layer", 8, "interleaved", 3), (1021, 64, "none", 0, "half", 5), (5, 32, "layer", -1, "half", 0),
    (3, 128, "none", -1, "half", 1)])
def test_cache_append(T, d_I, k_norm, k_off, k_layout, skip, keys):
    g, n = _gen(T + d_I), T + 77
    a = _randn(g, T, 576).bfloat16()
    wa = 1 + 0.2 * _randn(g, 512)
    pos = torch.randint(0, 10 ** 7, (T,), generator=g, device=DEV)
    slot = torch.randperm(n, generator=g, device=DEV)[:T].contiguous()
    if skip:
        slot[torch.arange(T, device=DEV) % skip == skip - 1] = -1
    kv = _randn(g, n, 576).bfloat16()
    freqs, mul = lsa.lsa_rope_freqs(64, scaling="yarn", factor=4.0)
    kv0 = kv.clone()
    kw = {}
    if keys != "none":
        k = _randn(g, T, d_I).bfloat16()
        wk, bk = _weights(g, k_norm, d_I)
        kc = _randn(g, n, d_I).bfloat16() if keys == "bf16" else torch.randint(0, 120, (n, d_I), generator=g, device=DEV,
                                                                              dtype=torch.uint8)
        ks = 0.5 + _randn(g, n).abs() if keys == "e4m3" else None
        kc0, ks0 = kc.clone(), None if ks is None else ks.clone()
        kw = dict(k=k, k_cache=kc, k_scale=ks, k_norm=k_norm, k_weight=wk, k_bias=bk, k_eps=1e-5, k_rope_off=k_off,
                  k_layout=k_layout)
    lsa.lsa_cache_append(a, kv, slot, pos, freqs, kv_weight=wa, kv_eps=1e-6, layout="half", mul=mul, **kw)
    live, at = slot >= 0, slot[slot >= 0]
    rest = torch.ones(n, dtype=torch.bool, device=DEV)
    rest[at] = False
    want = torch.cat([norm64(a[:, :512], "rms", wa, None, 1e-6),
                      rotate64(a[:, 512:].double(), pos, freqs, 0, "half", mul)], 1)[live]
    if at.numel():
        check_rows(kv[at][:, :512], want[:, :512])
        check_rows(kv[at][:, 512:], want[:, 512:], mul)
    assert torch.equal(kv[rest], kv0[rest])
    if keys != "none":
        want = norm64(k, k_norm, wk, bk, 1e-5)
        if k_off >= 0:
            want = rotate64(want, pos, freqs, k_off, k_layout, mul)
        if at.numel():
            if keys == "bf16":
                check_rows(kc[at], want[live], mul)
            else:
                check_codes(kc[at], ks[at], want[live], mul)
        assert torch.equal(kc[rest], kc0[rest])
        if ks is not None:
            assert torch.equal(ks[rest], ks0[rest])
    _status_ok()


def test_cache_append_plain_copy_and_strides():
    """No norm, no rotation: the rows' bytes; rows taken out of a wider projection."""
    g = _gen(5)
    proj = _randn(g, 21, 2304).bfloat16()
    a, k = proj[:, 1152:1728], proj[:, 64:192]
    kv, kc = torch.zeros(30, 576, dtype=torch.bfloat16, device=DEV), torch.zeros(30, 128, dtype=torch.bfloat16, device=DEV)
    slot = torch.arange(29, 8, -1, device=DEV)
    lsa.lsa_cache_append(a, kv, slot, k=k, k_cache=kc)
    assert torch.equal(kv[slot], a) and torch.equal(kc[slot], k) and not kv[:9].any() and not kc[:9].any()


def test_cache_append_codes_as_float8_and_unaligned_weights():
    """A cache of the codes' own type; weights that begin four bytes off a 16-byte boundary."""
    g, n = _gen(8), 12
    a, k = _randn(g, 3, 576).bfloat16(), _randn(g, 3, 128).bfloat16()
    wa, wk = (1 + 0.2 * _randn(g, 513))[1:], (1 + 0.2 * _randn(g, 129))[1:]
    kv = torch.zeros(n, 576, dtype=torch.bfloat16, device=DEV)
    kc, ks = torch.zeros(n, 128, device=DEV).to(torch.float8_e4m3fn), torch.zeros(n, device=DEV)
    slot = torch.tensor([11, 0, 5], device=DEV)
    lsa.lsa_cache_append(a, kv, slot, kv_weight=wa, k=k, k_cache=kc, k_scale=ks, k_norm="rms", k_weight=wk)
    check_rows(kv[slot][:, :512], norm64(a[:, :512], "rms", wa, None, 1e-6))
    check_codes(kc.view(torch.uint8)[slot], ks[slot], norm64(k, "rms", wk, None, 1e-6))


def test_cache_append_refusals():
    a, kv = torch.zeros(3, 576, dtype=torch.bfloat16, device=DEV), torch.zeros(8, 576, dtype=torch.bfloat16, device=DEV)
    k, kc, ks = a[:, :128].contiguous(), kv[:, :128].contiguous(), torch.zeros(8, device=DEV)
    slot, pos, freqs = torch.arange(3, device=DEV), torch.arange(3, device=DEV), lsa.lsa_rope_freqs(64)[0]
    for args, kw in (((a, kv, slot.int()), {}), ((a[:2], kv, slot), {}), ((a.float(), kv, slot), {}), ((a, kv.t(), slot), {}),
                     ((a, kv, slot), dict(pos=pos)), ((a, kv, slot), dict(freqs=freqs)),
                     ((a, kv, slot), dict(pos=pos, freqs=lsa.lsa_rope_freqs(32)[0])), ((a, kv, slot), dict(k=k)),
                     ((a, kv, slot), dict(k=k, k_cache=kc[:4])), ((a, kv, slot), dict(k=k, k_cache=kc, k_scale=ks)),
                     ((a, kv, slot), dict(k=k, k_cache=kc, k_norm="layer", k_weight=torch.ones(64, device=DEV))),
                     ((a, kv, slot), dict(k=k, k_cache=kc, k_rope_off=0)),
                     ((a, kv, slot), dict(kv_weight=torch.ones(576, device=DEV)))):
        with pytest.raises(lsa.LsaError):
            lsa.lsa_cache_append(*args, **kw)
    assert not kv.any() and not kc.any()


def test_cache_append_slots_outside_are_skipped_and_reported():
    g, n = _gen(6), 20
    a, kv = _randn(g, 5, 576).bfloat16(), _randn(g, n, 576).bfloat16()
    kv0 = kv.clone()
    lsa.lsa_cache_append(a, kv, torch.tensor([3, n, -2, -1, 1 << 40], device=DEV))
    with pytest.raises(lsa.LsaError) as e:
        lsa.lsa_device_status()
    assert e.value.status == -5 and "k_cache_append" in str(e.value)
    assert torch.equal(kv[3], a[0])
    kv0[3] = a[0]
    assert torch.equal(kv, kv0)
    _status_ok()


def test_cache_append_past_32_bit_offsets():
    """A cache of more than 2^32 bytes and 2^31 elements: the last rows are reached, the first stay."""
    n = (1 << 31) // 576 + 100
    kv = torch.empty(n, 576, dtype=torch.bfloat16, device=DEV)
    kv[:4], kv[-4:] = 0, 0
    a = _randn(_gen(7), 2, 576).bfloat16()
    lsa.lsa_cache_append(a, kv, torch.tensor([n - 1, n - 3], device=DEV))
    assert torch.equal(kv[[n - 1, n - 3]], a) and not kv[:4].any() and not kv[[n - 2, n - 4]].any()


# ------------------------------------------------------------------------------------------------ values that are not finite


def _with_bad_rows(g, T, H, D):
    """Rows 0, 3, 6 .. hold one NaN, rows 1, 4 .. one infinity of either sign, the others are ordinary."""
    x = _randn(g, T, H, D).bfloat16()
    x[0::3, :, 5] = math.nan
    x[1::3, :, D - 1] = math.inf
    x[4::6, :, D - 1] = -math.inf
    return x


@pytest.mark.parametrize("norm", ["none", "rms", "layer"])
@pytest.mark.parametrize("D,H,R", [(128, 64, 64), (24, 3, 16), (1024, 1, 0)])
def test_norm_rope_values_that_are_not_finite(norm, D, H, R):
    """A NaN reaches its whole row's codes and their scale, an infinity the scale; in bf16 every element is what the
    formula gives; other rows are as always."""
    T = 13
    x = _with_bad_rows(_gen(D), T, H, D)
    pos = torch.arange(T, device=DEV) * 1000
    freqs, mul = lsa.lsa_rope_freqs(R) if R else (None, 1.0)
    want = norm64(x, norm, None, None, 1e-6)
    if R:
        want = rotate64(want, pos, freqs, 0, "half", mul)
    kw = dict(norm=norm, layout="half") if R == 0 else dict(pos=pos, freqs=freqs, norm=norm, layout="half", mul=mul)
    y = torch.empty_like(x)
    lsa.lsa_norm_rope(x, y, **kw)
    assert torch.equal(y.isnan(), want.isnan()) and torch.equal(y.isinf(), want.isinf())
    fine = torch.isfinite(x.float()).all(-1).all(-1)
    check_rows(y[fine], want[fine], mul)
    c, sc = torch.empty(T, H, D, dtype=torch.uint8, device=DEV), torch.empty(T, H, device=DEV)
    lsa.lsa_norm_rope(x, c, y_scale=sc, **kw)
    v = c.view(torch.float8_e4m3fn).float()
    check_codes(c[fine], sc[fine], want[fine], mul)
    top = want.abs().amax(-1)  # NaN where the row has one
    assert torch.equal(sc.isnan(), top.isnan()) and torch.equal(sc.isinf(), top.isinf())
    assert bool(v[top.isnan()].isnan().all())
    inf = top.isinf()
    assert torch.equal(v[inf].isnan(), want[inf].isinf()) and not v[inf][~want[inf].isinf()].any()


def test_norm_rope_sums_of_squares_that_overflow():
    """128 elements of 1e20: their squares' sum is past 32 bits, so the normed values are 0, ahead of weight and bias; of
    1e18 it is 1.28e38 and the rows are the formula's."""
    D = 128
    sign = torch.ones(D, device=DEV)
    sign[1::2] = -1
    x = torch.stack([1e20 * sign, 1e18 * sign]).bfloat16().view(2, 1, D)
    w, b = _weights(_gen(9), "layer", D)
    for norm, bias in (("rms", None), ("layer", b)):
        y = torch.empty_like(x)
        lsa.lsa_norm_rope(x, y, norm=norm, weight=w, bias=bias)
        assert torch.equal(y[0, 0], bias.bfloat16() if bias is not None else torch.zeros_like(y[0, 0]))
        check_rows(y[1:], norm64(x[1:], norm, w, bias, 1e-6))


@pytest.mark.parametrize("k_norm", ["none", "rms", "layer"])
@pytest.mark.parametrize("d_I", [32, 128])
def test_cache_append_values_that_are_not_finite(k_norm, d_I):
    """The same for the rows of both caches."""
    g, T = _gen(d_I + 1), 13
    a, k = _with_bad_rows(g, T, 1, 576)[:, 0], _with_bad_rows(g, T, 1, d_I)[:, 0].contiguous()
    k_off = 0 if d_I >= 64 else -1
    pos, slot = torch.arange(T, device=DEV) * 1000, torch.randperm(T, generator=g, device=DEV)
    freqs, mul = lsa.lsa_rope_freqs(64)
    wa = 1 + 0.2 * _randn(g, 512)
    want_a = torch.cat([norm64(a[:, :512], "rms", wa, None, 1e-6), rotate64(a[:, 512:].double(), pos, freqs, 0, "half", mul)], 1)
    want = norm64(k, k_norm, None, None, 1e-6)
    if k_off >= 0:
        want = rotate64(want, pos, freqs, k_off, "half", mul)
    fine = torch.isfinite(a.float()).all(-1) & torch.isfinite(k.float()).all(-1)
    for fp8 in (False, True):
        kv = torch.zeros(T, 576, dtype=torch.bfloat16, device=DEV)
        kc = torch.zeros(T, d_I, dtype=torch.uint8 if fp8 else torch.bfloat16, device=DEV)
        ks = torch.zeros(T, device=DEV) if fp8 else None
        lsa.lsa_cache_append(a, kv, slot, pos, freqs, kv_weight=wa, layout="half", mul=mul, k=k, k_cache=kc, k_scale=ks,
                             k_norm=k_norm, k_rope_off=k_off)
        got = kv[slot]
        assert torch.equal(got.isnan(), want_a.isnan()) and torch.equal(got.isinf(), want_a.isinf())
        check_rows(got[fine], want_a[fine], mul)
        if not fp8:
            got = kc[slot]
            assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.isinf(), want.isinf())
            check_rows(got[fine], want[fine], mul)
            continue
        sc, v = ks[slot], kc[slot].view(torch.float8_e4m3fn).float()
        check_codes(kc[slot][fine], sc[fine], want[fine], mul)
        top = want.abs().amax(-1)
        assert torch.equal(sc.isnan(), top.isnan()) and torch.equal(sc.isinf(), top.isinf())
        assert bool(v[top.isnan()].isnan().all())
        inf = top.isinf()
        assert torch.equal(v[inf].isnan(), want[inf].isinf()) and not v[inf][~want[inf].isinf()].any()


def test_index_scores_of_codes_that_are_not_finite():
    """A NaN or infinite index key, or query, gives NaN scores and not a finite one that could pass for an unrelated key."""
    g, L, H = _gen(81), 300, 16
    k, qi = _randn(g, L, 128).bfloat16(), _randn(g, 3, H, 128).bfloat16()
    k[7, 3], k[200, 90], qi[1, 5, 64] = math.nan, math.inf, math.nan
    for norm in ("none", "layer"):
        kc, ks = torch.zeros(L, 128, dtype=torch.uint8, device=DEV), torch.zeros(L, device=DEV)
        at = torch.arange(L, device=DEV)
        a, kv = torch.zeros(L, 576, dtype=torch.bfloat16, device=DEV), torch.zeros(L, 576, dtype=torch.bfloat16, device=DEV)
        lsa.lsa_cache_append(a, kv, at, k=k, k_cache=kc, k_scale=ks, k_norm=norm)
        qc, qs = torch.empty(3, H, 128, dtype=torch.uint8, device=DEV), torch.empty(3, H, device=DEV)
        lsa.lsa_norm_rope(qi, qc, norm="rms", y_scale=qs)
        scores = torch.empty(3, L, device=DEV)
        lsa.lsa_index_score(qc, _randn(g, 3, H), kc, torch.full((3,), L - 1, device=DEV), scores, q_scale=qs, k_scale=ks)
        assert bool(scores[1].isnan().all())
        ok = torch.ones(L, dtype=torch.bool, device=DEV)
        ok[[7, 200]] = False
        assert bool(scores[[0, 2]][:, ~ok].isnan().all()) and bool(torch.isfinite(scores[[0, 2]][:, ok]).all())


# ------------------------------------------------------------------------------------------------ prefix_attn


def _prefix_case(seed, B, H, Lp, lens, page, spread=2.0, spare=3, cols=None):
    """Pages in random order; every row behind a sequence's end, spare pages and unused table entries hold garbage."""
    g = _gen(seed)
    q = (spread * _randn(g, B, H, 576)).bfloat16()
    prefix = _randn(g, Lp, 576).bfloat16() if Lp else None
    if lens is None:
        return q, prefix, None, None, None
    need = [-(-n // page) for n in lens]
    total = sum(need) + spare
    pages = torch.full((total, page, 576), math.nan, dtype=torch.bfloat16, device=DEV)
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    table = torch.full((B, cols or max(max(need), 1)), 0x7FFFFFFF, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(lens):
        for j in range(need[b]):
            r = min(page, n - j * page)
            pages[order[at].long(), :r] = _randn(g, r, 576).bfloat16()
            table[b, j] = order[at]
            at += 1
    return q, prefix, pages, table, torch.tensor(lens, dtype=torch.int32, device=DEV)


def _run_prefix(q, prefix, pages, table, own, scale, lse=True):
    B, H = q.shape[:2]
    out = torch.full((B, H, 512), math.nan, dtype=torch.bfloat16, device=DEV)
    l = torch.full((B, H), math.nan, device=DEV) if lse else None
    ws = lsa.workspace(lsa.lsa_prefix_attn_workspace_size(B, H), DEV).fill_(0xFF)
    lsa.lsa_prefix_attn(q, prefix, scale, out, l, pages=pages, table=table, own_len=own, ws=ws)
    return out, l


@pytest.mark.parametrize("B,H,Lp,lens,page", [
    (1, 1, 1, None, 0), (1, 128, 64, None, 0), (1, 5, 0, [1], 16), (2, 128, 1000, [0, 77], 16), (2, 128, 63, [64, 65], 64),
    (3, 16, 130, [0, 1, 65], 8), (5, 48, 257, [64, 63, 128, 0, 200], 32), (4, 200, 0, [0, 5, 64, 129], 64),
    (2, 256, 4097, [300, 0], 128), (7, 33, 513, [1, 2, 3, 0, 31, 32, 33], 16), (1, 128, 20000, [31], 1024),
    (130, 8, 300, [(37 * b) % 90 for b in range(130)], 8), (3, 128, 0, [0, 0, 0], 16), (9, 100, 700, None, 0),
    (40, 128, 2049, [(53 * b) % 140 for b in range(40)], 64), (1, 300, 129, [200], 32), (300, 1, 65, [b % 5 for b in range(300)], 8)])
def test_prefix_attn(B, H, Lp, lens, page):
    q, prefix, pages, table, own = _prefix_case(B * 31 + H, B, H, Lp, lens, page)
    out, lse = _run_prefix(q, prefix, pages, table, own, 576 ** -0.5)
    check_prefix(out, lse, q, prefix, 576 ** -0.5, pages, table, own, rows=range(0, B, 1 if B <= 40 else 7))
    _status_ok()


@pytest.mark.parametrize("B,H,Lp,lens,page", [
    (400, 128, 130, [b % 3 for b in range(400)], 16),          # more tiles than threads that count them
    (300, 33, 70, [(7 * b) % 40 for b in range(300)], 8),      # many tiles of several queries
    (150, 48, 0, [(29 * b) % 300 for b in range(150)], 128),   # own tokens alone, items over several pairs
    (6, 64, 3000, [1500, 0, 0, 700, 1, 129], 64), (2, 130, 777, [260, 3], 16), (80, 128, 127, None, 0)])
def test_prefix_attn_many_tiles(B, H, Lp, lens, page):
    q, prefix, pages, table, own = _prefix_case(B + H, B, H, Lp, lens, page)
    out, lse = _run_prefix(q, prefix, pages, table, own, 0.04)
    check_prefix(out, lse, q, prefix, 0.04, pages, table, own, rows=sorted({0, 1, B // 3, B // 2, B - 2, B - 1} & set(range(B))))
    assert torch.isfinite(out.float()).all() or lens is not None
    again, lse2 = _run_prefix(q, prefix, pages, table, own, 0.04)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    _status_ok()


@pytest.mark.parametrize("B,H,Lp,lens,page", [
    (400, 128, 130, [b % 3 for b in range(400)], 16), (300, 33, 70, [(7 * b) % 40 for b in range(300)], 8),
    (150, 48, 0, [(29 * b) % 300 for b in range(150)], 128), (6, 64, 3000, [1500, 0, 0, 700, 1, 129], 64),
    (2, 130, 777, [260, 3], 16), (80, 128, 127, None, 0), (70, 8, 0, [0] * 70, 8)])
def test_prefix_attn_every_row_is_written_and_finite(B, H, Lp, lens, page):
    """Outputs that held NaN, beside pages that hold NaN behind each sequence's end: every element of every row is finite,
    and a row without keys is zeros with lse -inf."""
    q, prefix, pages, table, own = _prefix_case(B * 3 + H, B, H, Lp, lens, page)
    out, lse = _run_prefix(q, prefix, pages, table, own, 0.04)
    assert bool(torch.isfinite(out.float()).all())
    none = torch.zeros(B, dtype=torch.bool, device=DEV) if Lp or lens is None else own == 0
    assert not out[none].any() and bool((lse[none] == -math.inf).all()) and bool(torch.isfinite(lse[~none]).all())
    assert bool(out[~none].abs().amax(-1).gt(0).all())
    _status_ok()


def test_prefix_attn_past_32_bit_offsets():
    """A prefix of more than 2^32 bytes and 2^31 elements: rows of zeros (logit 0, value 0) but for the last 300."""
    g, B, H, L, n = _gen(51), 2, 16, (1 << 31) // 576 + 1001, 300
    prefix = torch.zeros(L, 576, dtype=torch.bfloat16, device=DEV)
    prefix[-n:] = _randn(g, n, 576).bfloat16()
    q = (8 * _randn(g, B, H, 576)).bfloat16()
    out, lse = _run_prefix(q, prefix, None, None, None, 0.04)
    k = prefix[-n:].double()
    z = 0.04 * q.double() @ k.T
    l = torch.logaddexp(torch.logsumexp(z, -1), torch.full((B, H), math.log(L - n), dtype=torch.float64, device=DEV))
    p = torch.exp(z - l[..., None])
    o, mag = p @ k[:, :512], p @ k[:, :512].abs()
    dz = 0.04 * float((q.double().abs() @ k.abs().T).max()) * 576 * 2.0 ** -23
    assert ((out.double() - o).abs() <= 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2.1 * dz + 2.0 ** -12) * mag * (1 + 2.0 ** -8)).all()
    # 32-bit sums of 2^22 equal terms, four at a time and then joined: 2^-18 of the sum
    assert ((lse.double() - l).abs() <= dz + 2.0 ** -16 * (1 + l.abs())).all()
    assert out.any()


def test_prefix_attn_empty_tables_and_slices():
    """A table without columns, a cache without pages, an empty prefix, a prefix that is a slice of a longer cache."""
    q, cache, pages, table, own = _prefix_case(50, 3, 16, 500, [0, 0, 0], 16)
    prefix = cache[100:357]
    want = _run_prefix(q, prefix, None, None, None, 0.04)
    check_prefix(*want, q, prefix, 0.04)
    for pg, tb in ((pages, table[:, :0].contiguous()), (pages[:0], table)):
        got = _run_prefix(q, prefix, pg, tb, own, 0.04)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out, lse = _run_prefix(q, cache[:0], pages, table, own, 0.04)
    assert not out.any() and bool((lse == -math.inf).all())
    _status_ok()


@pytest.mark.parametrize("scale", [0.0, -0.05, 0.04, 0.5])
def test_prefix_attn_scales(scale):
    """Uniform weights, negative scales, ordinary and peaked rows."""
    q, prefix, pages, table, own = _prefix_case(11, 3, 64, 777, [100, 0, 41], 16)
    out, lse = _run_prefix(q, prefix, pages, table, own, scale)
    check_prefix(out, lse, q, prefix, scale, pages, table, own)


@pytest.mark.parametrize("H", [32, 128])
def test_prefix_attn_rising_maxima(H):
    """Logits that grow along the prefix by more than any block before (every block changes its reference), and that fall."""
    q, prefix, pages, table, own = _prefix_case(12, 2, H, 2000, [90, 10], 32, spread=1.0)
    d = _randn(_gen(13), 576)
    d = d / d.norm() * 24
    q = (0.1 * q.float() + d).bfloat16()
    for order in (1, -1):
        ramp = torch.linspace(0, 12, 2000, device=DEV)
        ramp = ramp if order > 0 else ramp.flip(0)
        p = (0.1 * prefix.float() + ramp[:, None] * d / 24).bfloat16()
        out, lse = _run_prefix(q, p, pages, table, own, 1.0)
        check_prefix(out, lse, q, p, 1.0, pages, table, own)


def test_prefix_attn_without_lse_and_without_keys():
    q, prefix, pages, table, own = _prefix_case(14, 3, 16, 0, [0, 3, 0], 8)
    out, _ = _run_prefix(q, None, pages, table, own, 0.04, lse=False)
    check_prefix(out, None, q, None, 0.04, pages, table, own)
    out, lse = _run_prefix(q, None, None, None, None, 0.04)
    assert not out.any() and bool((lse == -math.inf).all())


def test_prefix_attn_a_non_finite_sequence_stays_its_own():
    """Infinities and NaN in one sequence's tokens reach no other sequence's rows, in the same tile either."""
    q, prefix, pages, table, own = _prefix_case(15, 4, 32, 200, [40, 50, 0, 60], 16)
    pages[table[1, 0].long(), 3] = math.inf
    pages[table[1, 2].long(), 5] = math.nan
    out, lse = _run_prefix(q, prefix, pages, table, own, 0.04)
    check_prefix(out, lse, q, prefix, 0.04, pages, table, own, rows=[0, 2, 3])
    assert not torch.isfinite(out[1].float()).all()


@pytest.mark.parametrize("B,H,L", [(1, 16, 20000), (1, 128, 20000), (1, 300, 3000), (3, 128, 9000), (40, 128, 9000), (3, 48, 9000)])
def test_prefix_attn_infinite_values_of_keys_that_weigh_nothing(B, H, L):
    """A key with an infinite element and a logit of -inf, among keys whose weights underflow: the column is NaN (0 times
    infinity) in every row, wherever the work was cut, and the other columns and the sums are ordinary."""
    g = _gen(90 + B)
    q = (0.2 * _randn(g, B, H, 576)).bfloat16()
    q[:, :, 5], q[:, :, 7] = 1.0, 8.0
    prefix = _randn(g, L, 576).bfloat16()
    prefix[:, 7] = 0
    prefix[: L // 3, 7] = -60.0  # logits 480 below the others
    prefix[3, 5] = -math.inf
    out, lse = _run_prefix(q, prefix, None, None, None, 1.0)
    assert bool(out[:, :, 5].isnan().all())
    other = [d for d in range(512) if d != 5]
    clean = prefix[torch.arange(L, device=DEV) != 3]
    # Column 7 is -60 times weights of e^-480: in 32 bits a weight below 2^-126 may be 0, so up to 2^15 keys of magnitude
    # up to 2^6 lose up to 2^-126 * 2^15 * 2^6 = 2^-105 of a sum whose largest weight is 1 (it is divided by 1 or more).
    lost = 2.0 ** -105
    for b in range(0, B, 13):
        o, l, mag, dz = prefix64(q, clean, 1.0, None, None, None, b)
        tol = 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2.1 * dz + 2.0 ** -12) * mag * (1 + 2.0 ** -8) + lost
        assert ((out[b].double() - o).abs() <= tol)[:, other].all()
        assert ((lse[b].double() - l).abs() <= dz + 2.0 ** -18 * (1 + l.abs())).all()
    _status_ok()


def test_prefix_attn_shared_pages_and_speculative_tokens():
    """Queries of one sequence: the same table row, growing lengths."""
    q, prefix, pages, table, own = _prefix_case(16, 1, 64, 300, [70], 16)
    q = torch.cat([q * (1 + 0.1 * i) for i in range(4)])
    table, own = table.expand(4, -1).contiguous(), torch.tensor([67, 68, 69, 70], dtype=torch.int32, device=DEV)
    out, lse = _run_prefix(q, prefix, pages, table, own, 0.04)
    check_prefix(out, lse, q, prefix, 0.04, pages, table, own)


def test_prefix_attn_bad_tables_are_reported():
    q, prefix, pages, table, own = _prefix_case(17, 3, 16, 100, [40, 20, 16], 16)
    good = table.clone()
    for change in ("page", "negative page", "long", "negative"):
        t, o = good.clone(), own.clone()
        if change == "page":
            t[0, 1] = pages.shape[0]
        elif change == "negative page":
            t[0, 0] = -1
        elif change == "long":
            o[1] = 16 * t.shape[1] + 1
            t[1] = good[0]
        else:
            o[1] = -1
        out, lse = _run_prefix(q, prefix, pages, t, o, 0.04)
        with pytest.raises(lsa.LsaError) as e:
            lsa.lsa_device_status()
        assert e.value.status == -5 and "k_prefix_attn" in str(e.value), change
        check_prefix(out, lse, q, prefix, 0.04, pages, good, own, rows=[2])
        if change == "negative":
            check_prefix(out, lse, q, prefix, 0.04, rows=[1])
    _status_ok()


def test_prefix_attn_agrees_with_sparse_attention_over_every_row():
    """The framework's selected attention with every row selected reads the same keys."""
    g, B, H, L = _gen(18), 2, 128, 600
    q, kv = (2 * _randn(g, B, H, 576)).bfloat16(), _randn(g, L, 576).bfloat16()
    idx = torch.arange(L, dtype=torch.int32, device=DEV).expand(B, L).contiguous()
    cnt = torch.full((B,), L, dtype=torch.int32, device=DEV)
    o1, l1 = torch.empty(B, H, 512, dtype=torch.bfloat16, device=DEV), torch.empty(B, H, device=DEV)
    ws = lsa.workspace(lsa.lsa_workspace_size(lsa.LSA_OP_ATTN, B, L, L, H), DEV)
    lsa.lsa_sparse_attn(q, kv, idx, cnt, 576 ** -0.5, o1, l1, ws)
    o2, l2 = _run_prefix(q, kv, None, None, None, 576 ** -0.5)
    check_prefix(o2, l2, q, kv, 576 ** -0.5)
    assert (l1 - l2).abs().max() <= 1e-2


def test_prefix_attn_refusals():
    q, prefix, pages, table, own = _prefix_case(19, 2, 16, 32, [3, 4], 8)
    out, ws = torch.empty(2, 16, 512, dtype=torch.bfloat16, device=DEV), lsa.workspace(1 << 27, DEV)
    full = dict(pages=pages, table=table, own_len=own, ws=ws)
    for kw in (dict(full, table=None), dict(full, own_len=own.long()), dict(full, own_len=own[:1].clone()),
               dict(full, table=table[:, :0].t()), dict(full, pages=pages[:, ::2]), dict(full, pages=pages.half()),
               dict(full, lse=torch.empty(2, 8, device=DEV)), dict(full, ws=None), dict(full, ws=ws[:128])):
        with pytest.raises(lsa.LsaError):
            lsa.lsa_prefix_attn(q, prefix, 0.04, out, **kw)
    for bad_q in (q.float(), q[:, ::2], q.transpose(0, 1)):
        with pytest.raises(lsa.LsaError):
            lsa.lsa_prefix_attn(bad_q, prefix, 0.04, out, ws=ws)


# ------------------------------------------------------------------------------------------------ together


def test_queries_rotated_right_before_the_sparse_attention():
    """The decode attention loads its query before it waits for the kernel ahead of it: a rotation that writes the query
    has to be over by then (new queries each time, more than one wave of blocks)."""
    g, B, H, L, n = _gen(40), 16, 128, 4096, 24
    kv = _randn(g, L, 576).bfloat16()
    raw = [(2 * _randn(g, B, H, 576)).bfloat16() for _ in range(n)]
    pos = torch.randint(0, 100000, (B,), generator=g, device=DEV)
    freqs, _ = lsa.lsa_rope_freqs(64)
    idx = torch.stack([torch.randperm(L, generator=g, device=DEV)[:256].sort().values for _ in range(B)]).int().contiguous()
    cnt = torch.full((B,), 256, dtype=torch.int32, device=DEV)
    ws = lsa.workspace(lsa.lsa_workspace_size(lsa.LSA_OP_ATTN, B, L, 256, H), DEV)
    q, outs = torch.zeros_like(raw[0]), [torch.empty(B, H, 512, dtype=torch.bfloat16, device=DEV) for _ in range(n)]
    for i in range(n):
        lsa.lsa_norm_rope(raw[i], q, pos, freqs, norm="rms", rope_off=512)
        lsa.lsa_sparse_attn(q, kv, idx, cnt, 0.04, outs[i], None, ws)
    torch.cuda.synchronize()
    for i in range(n):
        lsa.lsa_norm_rope(raw[i], q, pos, freqs, norm="rms", rope_off=512)
        torch.cuda.synchronize()
        want = torch.empty_like(outs[i])
        lsa.lsa_sparse_attn(q, kv, idx, cnt, 0.04, want, None, ws)
        assert torch.equal(outs[i], want), i


def test_streams_graphs_and_repeats():
    """Each operator on a side stream, captured and replayed on new inputs, two graphs in flight with their own
    workspaces; the same inputs give the same bytes."""
    cases = [_prefix_case(20 + i, 5, 48, 900, [70, 0, 33, 64, 5], 16) for i in range(3)]
    want = [_run_prefix(*c, 0.04) for c in cases]
    again = _run_prefix(*cases[0], 0.04)
    assert torch.equal(again[0], want[0][0]) and torch.equal(again[1], want[0][1])
    freqs, _ = lsa.lsa_rope_freqs(64)
    bufs, graphs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for i in range(2):
        q, prefix, pages, table, own = [t.clone() for t in cases[i]]
        raw, pos = q.clone(), torch.zeros(5, dtype=torch.int64, device=DEV)
        slot = torch.tensor([-1, -1, -1, -1, -1], device=DEV)
        a = torch.zeros(5, 576, dtype=torch.bfloat16, device=DEV)
        out, lse = torch.empty(5, 48, 512, dtype=torch.bfloat16, device=DEV), torch.empty(5, 48, device=DEV)
        ws = lsa.workspace(lsa.lsa_prefix_attn_workspace_size(5, 48), DEV)
        bufs.append((q, raw, prefix, pages, table, own, pos, slot, a, out, lse, ws))

        def step():
            lsa.lsa_norm_rope(raw, q, pos, freqs, rope_off=512)
            lsa.lsa_cache_append(a, pages.view(-1, 576), slot, pos, freqs)
            lsa.lsa_prefix_attn(q, prefix, 0.04, out, lse, pages=pages, table=table, own_len=own, ws=ws)

        streams[i].wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(streams[i]):
            step()
        streams[i].synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=streams[i]):
            step()
        graphs.append(graph)
    for rnd in range(2):
        src = (1, 2) if rnd == 0 else (2, 0)
        for i in range(2):
            for dst, s in zip((bufs[i][1], *bufs[i][2:6]), cases[src[i]]):
                if dst.shape == s.shape:
                    dst.copy_(s)
                else:
                    raise AssertionError("cases of one shape wanted")
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            # position 0: the rotation is the identity
            assert torch.equal(bufs[i][9], want[src[i]][0]) and torch.equal(bufs[i][10], want[src[i]][1])
    _status_ok()


def test_many_streams_at_once():
    """Calls of different shapes, the sparse attention and the indexer on four streams at a time, each call with its own
    workspace: the same bytes as alone."""
    shapes = [(5, 48, 900, [70, 0, 33, 64, 5], 16), (16, 128, 1200, [10 * b for b in range(16)], 64), (1, 128, 7000, [31], 32),
              (40, 128, 200, None, 16), (3, 16, 100, [1, 0, 200], 8)]
    cases = [_prefix_case(70 + i, *s) for i, s in enumerate(shapes)]
    g, B, H, L = _gen(71), 16, 128, 4096
    kv, q = _randn(g, L, 576).bfloat16(), (2 * _randn(g, B, H, 576)).bfloat16()
    idx = torch.stack([torch.randperm(L, generator=g, device=DEV)[:256].sort().values for _ in range(B)]).int().contiguous()
    cnt = torch.full((B,), 256, dtype=torch.int32, device=DEV)
    qi, w, ki = _randn(g, B, 64, 128).bfloat16(), _randn(g, B, 64), _randn(g, 20000, 128).bfloat16()
    q_pos = torch.full((B,), 19999, device=DEV)

    def sparse():
        out = torch.empty(B, H, 512, dtype=torch.bfloat16, device=DEV)
        lsa.lsa_sparse_attn(q, kv, idx, cnt, 0.04, out, None, lsa.workspace(lsa.lsa_workspace_size(lsa.LSA_OP_ATTN, B, L, 256, H)))
        return (out,)

    def index():
        scores = torch.empty(B, 20000, device=DEV)
        lsa.lsa_index_score(qi, w, ki, q_pos, scores)
        return (scores,)

    calls = [lambda c=c: _run_prefix(*c, 0.04) for c in cases] + [sparse, index]
    want = [f() for f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    for rnd in range(6):
        got = []
        for k in range(28):
            j = (5 * k + rnd) % 7
            with torch.cuda.stream(streams[(k + rnd) % 4]):
                got.append((j, calls[j]()))
        torch.cuda.synchronize()
        for j, o in got:
            assert all(torch.equal(x, y) for x, y in zip(o, want[j])), j
    _status_ok()


def test_explicit_stream_and_another_current_device(monkeypatch):
    """A stream given to the call; and a current device that is not the tensors' (as far as one GPU can show it: the calls
    make the tensors' device current and give the same)."""
    q, prefix, pages, table, own = _prefix_case(60, 3, 32, 400, [20, 0, 50], 16)
    want = _run_prefix(q, prefix, pages, table, own, 0.04)
    freqs, _ = lsa.lsa_rope_freqs(64)
    pos = torch.arange(3, device=DEV)
    a = q[:, 0].contiguous()

    def run(**kw):
        out, lse = torch.empty(3, 32, 512, dtype=torch.bfloat16, device=DEV), torch.empty(3, 32, device=DEV)
        ws = lsa.workspace(lsa.lsa_prefix_attn_workspace_size(3, 32), DEV)
        y, kv = torch.empty_like(q), torch.zeros(4, 576, dtype=torch.bfloat16, device=DEV)
        torch.cuda.synchronize()
        lsa.lsa_norm_rope(q, y, pos, freqs, rope_off=512, **kw)
        lsa.lsa_cache_append(a, kv, pos, pos, freqs, **kw)
        lsa.lsa_prefix_attn(q, prefix, 0.04, out, lse, pages=pages, table=table, own_len=own, ws=ws, **kw)
        torch.cuda.synchronize()
        return out, lse, y, kv

    plain, side = run(), run(stream=torch.cuda.Stream())
    answers = []

    def first_yes(dev):  # another device is current, until the call has made the tensors' own the current one
        answers.append(len(answers) % 2 == 0)
        return answers[-1]

    monkeypatch.setattr(lsa, "_off_device", first_yes)
    moved = run()
    monkeypatch.undo()
    assert len(answers) == 6  # each call asked twice
    for got in (plain, side, moved):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(got[2], plain[2]) and torch.equal(got[3], plain[3])


def test_decode_steps_together():
    """A few decode steps of a layer as a server runs them: queries normed and rotated, rows appended to pages, the index
    scored over them and its top-K attended to, and dense attention over prefix and own pages; against 64 bits."""
    g, B, H, HI, Lp, page, steps = _gen(30), 3, 128, 16, 384, 16, 3
    scale = 576 ** -0.5
    freqs, mul = lsa.lsa_rope_freqs(64, scaling="yarn", factor=4.0)
    n_pages = 12
    prefix = torch.empty(Lp, 576, dtype=torch.bfloat16, device=DEV)
    pages = torch.zeros(n_pages, page, 576, dtype=torch.bfloat16, device=DEV)
    kcodes, kscale = torch.empty(Lp, 128, dtype=torch.uint8, device=DEV), torch.empty(Lp, device=DEV)
    wa, wk, bk = 1 + 0.1 * _randn(g, 512), 1 + 0.1 * _randn(g, 128), 0.1 * _randn(g, 128)
    wq = 1 + 0.1 * _randn(g, 128)
    # the prefix's prefill: latent rows and e4m3 index keys
    a, k = _randn(g, Lp, 576).bfloat16(), _randn(g, Lp, 128).bfloat16()
    pos = torch.arange(Lp, device=DEV)
    lsa.lsa_cache_append(a, prefix, pos, pos, freqs, kv_weight=wa, mul=mul, k=k, k_cache=kcodes, k_scale=kscale,
                         k_norm="layer", k_weight=wk, k_bias=bk, k_rope_off=0)
    lat = lambda x, p: torch.cat([norm64(x[:, :512], "rms", wa, None, 1e-6),
                                  rotate64(x[:, 512:].double(), p, freqs, 0, "interleaved", mul)], 1)
    check_rows(prefix[:, :512], lat(a, pos)[:, :512])
    check_rows(prefix[:, 512:], lat(a, pos)[:, 512:], mul)
    check_codes(kcodes, kscale, rotate64(norm64(k, "layer", wk, bk, 1e-6), pos, freqs, 0, "half", mul), mul)
    table = torch.randperm(n_pages, generator=g, device=DEV)[: 3 * B].view(B, 3).to(torch.int32).contiguous()
    own = torch.tensor([15, 0, 31], dtype=torch.int32, device=DEV)
    pages.view(-1, 576)[:] = _randn(g, n_pages * page, 576).bfloat16()
    ws = lsa.workspace(lsa.lsa_prefix_attn_workspace_size(B, H), DEV)
    for _ in range(steps):
        p = Lp + own.long()
        slot = table[torch.arange(B, device=DEV), (own // page).long()].long() * page + own.long() % page
        new = _randn(g, B, 576).bfloat16()
        lsa.lsa_cache_append(new, pages.view(-1, 576), slot, p, freqs, kv_weight=wa, mul=mul)
        own += 1
        qi = _randn(g, B, HI, 128).bfloat16()
        qc, qs = torch.empty(B, HI, 128, dtype=torch.uint8, device=DEV), torch.empty(B, HI, device=DEV)
        lsa.lsa_norm_rope(qi, qc, p, freqs, norm="rms", weight=wq, layout="half", mul=mul, y_scale=qs)
        check_codes(qc, qs, rotate64(norm64(qi, "rms", wq, None, 1e-6), p, freqs, 0, "half", mul), mul)
        # the prefix's index scores from those codes
        w, scores = _randn(g, B, HI), torch.empty(B, Lp, device=DEV)
        q_pos = torch.full((B,), Lp - 1, device=DEV)
        lsa.lsa_index_score(qc, w, kcodes, q_pos, scores, q_scale=qs, k_scale=kscale)
        dq = lambda c, s: (c.view(torch.float8_e4m3fn).double() * s.double()[..., None]).cpu().numpy()
        ref = O.index_score(dq(qc, qs), w.double().cpu().numpy(), dq(kcodes, kscale), np.full(B, Lp - 1))
        assert np.abs(scores.cpu().numpy() - ref).max() <= 1e-3 * np.abs(ref).max()
        q = (2 * _randn(g, B, H, 576)).bfloat16()
        raw = q.clone()
        lsa.lsa_norm_rope(q, q, p, freqs, rope_off=512, mul=mul)
        check_rows(q, rotate64(raw.double(), p, freqs, 512, "interleaved", mul), mul)
        out, lse = torch.empty(B, H, 512, dtype=torch.bfloat16, device=DEV), torch.empty(B, H, device=DEV)
        lsa.lsa_prefix_attn(q, prefix, scale, out, lse, pages=pages, table=table, own_len=own, ws=ws)
        check_prefix(out, lse, q, prefix, scale, pages, table, own)
        at = slot
        check_rows(pages.view(-1, 576)[at][:, :512], lat(new, p)[:, :512])
    _status_ok()
