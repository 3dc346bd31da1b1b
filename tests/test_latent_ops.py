"""The operators around the latent cache, without a GPU: frequencies, sizes and refusals (nothing is launched)."""

import ctypes
import math

import pytest
import torch

import sparse_long_context_lightning_b200 as lsa
from latent_common import freqs64

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
FAKE = 0x1000  # 256-byte aligned, never dereferenced: every call below fails its checks first


@pytest.fixture(scope="module")
def lib():
    return lsa.load_library()


@pytest.mark.parametrize("R,kw", [(64, {}), (128, dict(scaling="linear", factor=8.0)), (2, {}), (64, dict(base=500000.0)),
                                  (64, dict(scaling="yarn", factor=32.0)), (16, dict(scaling="yarn", factor=1.0)),
                                  (128, dict(scaling="yarn", factor=40.0, original_len=8192, beta_fast=16.0))])
def test_rope_freqs(R, kw):
    f, mul = lsa.lsa_rope_freqs(R, device="cpu", **kw)
    want, want_mul = freqs64(R, **kw)
    assert f.dtype == torch.float64 and f.shape == (R // 2,)
    # the ramp's (1 - r) f + r f / s, pow and a division: a few roundings of 64 bits
    assert torch.allclose(f, torch.tensor(want, dtype=torch.float64), rtol=1e-14, atol=0)
    assert abs(mul - want_mul) <= 2.0 ** -24 * want_mul


@pytest.mark.parametrize("kw", [dict(R=63), dict(R=0), dict(R=2048), dict(R=64, base=1.0), dict(R=64, base=math.nan),
                                dict(R=64, scaling="linear", factor=0.5), dict(R=64, scaling="yarn", factor=math.nan),
                                dict(R=64, scaling="yarn", factor=4.0, original_len=0),
                                dict(R=64, scaling="yarn", factor=4.0, beta_fast=1.0, beta_slow=2.0),
                                dict(R=64, scaling="ntk")])
def test_rope_freqs_refusals(kw):
    with pytest.raises(lsa.LsaError) as e:
        lsa.lsa_rope_freqs(device="cpu", **kw)
    assert e.value.status == INVALID


def _norm_rope(lib, **kw):
    a = dict(x=FAKE, x_ldt=8192, x_ldh=128, T=4, H=64, D=128, norm=1, weight=FAKE, bias=None, eps=1e-6, freqs=FAKE, off=0,
             R=64, layout=0, mul=1.0, pos=FAKE, y=FAKE, y_ldt=8192, y_ldh=128, dtype=0, y_scale=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.lsa_norm_rope(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(H=65536), INVALID), (dict(D=0), INVALID), (dict(norm=3), INVALID),
    (dict(norm=0), INVALID), (dict(bias=FAKE), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID),
    (dict(dtype=2), INVALID), (dict(dtype=1), INVALID), (dict(y_scale=FAKE), INVALID), (dict(D=100), UNSUPPORTED),
    (dict(D=1032), UNSUPPORTED), (dict(T=1 << 62), UNSUPPORTED), (dict(layout=2), INVALID), (dict(off=-8), INVALID), (dict(off=72), INVALID),
    (dict(off=4), UNSUPPORTED), (dict(R=24), UNSUPPORTED), (dict(R=0), INVALID), (dict(R=136), INVALID),
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(pos=None), INVALID), (dict(x=FAKE + 8), INVALID),
    (dict(y=FAKE + 8), INVALID), (dict(x_ldt=8191), INVALID), (dict(y_ldh=132), INVALID), (dict(T=0, x=None), 0)])
def test_norm_rope_refusals(lib, kw, want):
    assert _norm_rope(lib, **kw) == want


@pytest.mark.parametrize("kw", [
    dict(y_ldh=64), dict(y_ldh=-120), dict(y_ldh=0), dict(y_ldt=0), dict(y_ldt=120), dict(y_ldt=128), dict(y_ldt=8064),
    dict(y_ldt=-256, y_ldh=128), dict(T=4, H=3, y_ldt=256, y_ldh=384), dict(T=8, H=8, y_ldt=136, y_ldh=1000),
    dict(T=1, y_ldh=64), dict(H=1, y_ldt=64), dict(T=1 << 40, y_ldt=1 << 30, y_ldh=1 << 30)])
def test_norm_rope_refuses_outputs_that_overlap_themselves(lib, kw):
    """Two rows of y that share elements: which row's results stay would depend on the order of the blocks."""
    a = dict(dict(T=4, H=64, y_ldt=8192, y_ldh=128), **kw)
    if a["T"] < 100:  # by the definition: some two begin less than a row apart (the call would be launched otherwise)
        at = sorted(i * a["y_ldt"] + j * a["y_ldh"] for i in range(a["T"]) for j in range(a["H"]))
        assert min(v - u for u, v in zip(at, at[1:])) < 128
    assert _norm_rope(lib, **kw) == INVALID


def _append(lib, **kw):
    a = dict(a=FAKE, a_ld=576, T=4, d_qk=576, d_v=512, kv_weight=FAKE, kv_eps=1e-6, freqs=FAKE, layout=0, mul=1.0,
             pos=FAKE, slot=FAKE, kv=FAKE, n_slots=64, k=FAKE, k_ld=128, d_I=128, k_norm=2, k_weight=FAKE, k_bias=FAKE,
             k_eps=1e-5, k_rope_off=0, k_layout=1, k_cache=FAKE, k_dtype=0, k_scale=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.lsa_cache_append(*a.values())


NO_KEYS = dict(k=None, k_cache=None, k_weight=None, k_bias=None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(n_slots=-1), INVALID), (dict(d_qk=512), UNSUPPORTED), (dict(d_v=576), UNSUPPORTED),
    (dict(kv_eps=-1.0), INVALID), (dict(layout=5), INVALID), (dict(d_I=96), UNSUPPORTED), (dict(k_norm=7), INVALID),
    (dict(k_norm=0), INVALID), (dict(k_norm=1), INVALID), (dict(k_eps=math.nan), INVALID), (dict(k_dtype=3), INVALID),
    (dict(k_dtype=1), INVALID), (dict(k_scale=FAKE), INVALID), (dict(k_rope_off=72), INVALID),
    (dict(d_I=32, k_rope_off=0), INVALID), (dict(k_rope_off=4), UNSUPPORTED), (dict(freqs=None), INVALID),
    (dict(k_layout=2), INVALID), (dict(k=None), INVALID), (dict(NO_KEYS, k_scale=FAKE), INVALID), (dict(a=None), INVALID),
    (dict(slot=None), INVALID), (dict(kv=None), INVALID), (dict(pos=None), INVALID), (dict(k_cache=None), INVALID),
    (dict(a=FAKE + 2), INVALID), (dict(kv=FAKE + 8), INVALID), (dict(a_ld=580), INVALID), (dict(k_ld=4), INVALID),
    (dict(k=FAKE + 8), INVALID), (dict(T=0, a=None), 0), (dict(NO_KEYS, T=0), 0)])
def test_cache_append_refusals(lib, kw, want):
    assert _append(lib, **kw) == want


def _prefix(lib, **kw):
    a = dict(q=FAKE, B=2, H=128, d_qk=576, d_v=512, prefix=FAKE, Lp=64, pages=FAKE, n_pages=8, page=64, table=FAKE,
             table_ld=4, own_len=FAKE, scale=0.1, out=FAKE, lse=None, ws=FAKE, ws_bytes=1 << 40, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.lsa_prefix_attn(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), INVALID), (dict(B=65536), INVALID), (dict(B=1 << 62), INVALID), (dict(H=0), INVALID), (dict(H=65536), INVALID), (dict(Lp=-1), INVALID),
    (dict(n_pages=-1), INVALID), (dict(table_ld=-1), INVALID), (dict(scale=math.nan), INVALID),
    (dict(scale=math.inf), INVALID), (dict(d_qk=512), UNSUPPORTED), (dict(d_v=576), UNSUPPORTED), (dict(page=0), INVALID),
    (dict(page=4), UNSUPPORTED), (dict(page=48), UNSUPPORTED), (dict(page=1 << 17), UNSUPPORTED),
    (dict(n_pages=1 << 26), UNSUPPORTED), (dict(Lp=1 << 31), UNSUPPORTED), (dict(q=None), INVALID),
    (dict(out=None), INVALID), (dict(prefix=None), INVALID), (dict(table=None), INVALID), (dict(pages=None), INVALID),
    (dict(q=FAKE + 8), INVALID), (dict(prefix=FAKE + 2), INVALID), (dict(pages=FAKE + 8), INVALID),
    (dict(out=FAKE + 4), INVALID), (dict(ws=None), WORKSPACE), (dict(ws=FAKE + 128), WORKSPACE),
    (dict(ws_bytes=0), WORKSPACE), (dict(B=0, q=None), 0)])
def test_prefix_attn_refusals(lib, kw, want):
    assert _prefix(lib, **kw) == want


def test_prefix_attn_workspace_size(lib):
    bad = ctypes.c_size_t(-1).value
    assert lib.lsa_prefix_attn_workspace_size(0, 128) == 0
    for B, H in [(1, 1), (16, 128), (33, 32), (64, 128), (4, 200)]:
        assert lib.lsa_prefix_attn_workspace_size(B, H) > 0
    for B, H in [(-1, 128), (1, 0), (65536, 128), (1, 65536)]:
        assert lib.lsa_prefix_attn_workspace_size(B, H) == bad


@pytest.mark.parametrize("B,H", [(1, 128), (1, 5), (16, 128), (33, 32), (256, 8), (4096, 8), (1024, 16), (65535, 1), (3, 65535)])
def test_prefix_attn_workspace_follows_the_query_rows(lib, B, H):
    """A row of the queries costs one fp32 row of 512 with its maximum and sum, or two, whatever share of a tile its query
    fills; beside them the pairs' 74 x 128 rows and 8 bytes for each item."""
    rows = 74 * 128 + (2 if H % 128 and B > 1 else 1) * B * H
    tiles = -(-B * H // 128)
    assert rows * 2056 <= lib.lsa_prefix_attn_workspace_size(B, H) <= rows * 2056 + 8 * (B + 2 * tiles) + 1024


def test_packed_forms(lib):
    """The structs that the binding packs are the library's: their sizes are taken, every field lands where the plain call
    has it (each refusal of one field), and another size is refused."""
    z = dict(size=lsa._NORM_ROPE.size, x=FAKE, x_ldt=64, x_ldh=64, T=0, weight=0, bias=0, freqs=0, pos=0, y=FAKE, y_ldt=64,
             y_ldh=64, y_scale=0, stream=0, H=1, D=64, norm=0, rope_off=0, rope_dims=0, layout=0, dtype=0, eps=1.0, mul=1.0)
    call = lambda **kw: lib.lsa_norm_rope_packed(lsa._NORM_ROPE.pack(*dict(z, **kw).values()))
    assert call() == 0 and call(size=8) == INVALID and lib.lsa_norm_rope_packed(None) == INVALID
    for kw, want in ((dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(D=12), UNSUPPORTED), (dict(norm=5), INVALID),
                     (dict(weight=FAKE), INVALID), (dict(bias=FAKE), INVALID), (dict(norm=1, eps=-1.0), INVALID),
                     (dict(dtype=1), INVALID), (dict(y_scale=FAKE), INVALID), (dict(freqs=FAKE), INVALID),
                     (dict(freqs=FAKE, rope_dims=16, rope_off=4), UNSUPPORTED), (dict(freqs=FAKE, rope_dims=16, layout=2), INVALID),
                     (dict(T=1, x=0), INVALID), (dict(T=1, y=0), INVALID), (dict(T=1, x_ldt=1), INVALID),
                     (dict(T=1, x_ldh=1), INVALID), (dict(T=1, y_ldt=1), INVALID), (dict(T=1, y_ldh=1), INVALID),
                     (dict(T=1, freqs=FAKE, rope_dims=16), INVALID)):
        assert call(**kw) == want, kw
    z = dict(size=lsa._CACHE_APPEND.size, a=FAKE, a_ld=576, T=0, kv_weight=0, freqs=0, pos=0, slot=FAKE, kv=FAKE, n_slots=4,
             k=0, k_ld=0, k_weight=0, k_bias=0, k_cache=0, k_scale=0, stream=0, d_qk=576, d_v=512, layout=0, d_I=0, k_norm=0,
             k_rope_off=-1, k_layout=0, k_dtype=0, kv_eps=0.0, mul=1.0, k_eps=0.0)
    call = lambda **kw: lib.lsa_cache_append_packed(lsa._CACHE_APPEND.pack(*dict(z, **kw).values()))
    keys = dict(k=FAKE, k_ld=128, d_I=128, k_cache=FAKE)
    assert call() == 0 and call(**keys) == 0 and call(size=0) == INVALID and lib.lsa_cache_append_packed(None) == INVALID
    for kw, want in ((dict(T=-1), INVALID), (dict(n_slots=-1), INVALID), (dict(d_qk=1), UNSUPPORTED), (dict(d_v=1), UNSUPPORTED),
                     (dict(kv_weight=FAKE, kv_eps=-1.0), INVALID), (dict(freqs=FAKE, layout=3), INVALID),
                     (dict(k_cache=FAKE), INVALID), (dict(k_scale=FAKE), INVALID), (dict(k_weight=FAKE), INVALID),
                     (dict(k_bias=FAKE), INVALID), (dict(keys, d_I=7), UNSUPPORTED), (dict(keys, k_norm=9), INVALID),
                     (dict(keys, k_norm=1, k_eps=-1.0), INVALID), (dict(keys, k_rope_off=0), INVALID),
                     (dict(keys, k_rope_off=0, freqs=FAKE, k_layout=4), INVALID), (dict(keys, k_dtype=1), INVALID),
                     (dict(T=1, a=0), INVALID), (dict(T=1, slot=0), INVALID), (dict(T=1, kv=0), INVALID),
                     (dict(T=1, a_ld=4), INVALID), (dict(keys, T=1, k_ld=4), INVALID), (dict(T=1, freqs=FAKE), INVALID)):
        assert call(**kw) == want, kw
    z = dict(size=lsa._PREFIX_ATTN.size, q=FAKE, B=0, prefix=FAKE, Lp=8, pages=FAKE, n_pages=4, table=FAKE, table_ld=2,
             own_len=FAKE, out=FAKE, lse=0, ws=FAKE, ws_bytes=1 << 40, stream=0, H=8, d_qk=576, d_v=512, page=16, scale=1.0)
    call = lambda **kw: lib.lsa_prefix_attn_packed(lsa._PREFIX_ATTN.pack(*dict(z, **kw).values()))
    assert call() == 0 and call(size=1) == INVALID and lib.lsa_prefix_attn_packed(None) == INVALID
    for kw, want in ((dict(B=-1), INVALID), (dict(H=0), INVALID), (dict(Lp=-1), INVALID), (dict(n_pages=-1), INVALID),
                     (dict(table_ld=-1), INVALID), (dict(d_qk=1), UNSUPPORTED), (dict(d_v=1), UNSUPPORTED),
                     (dict(page=3), UNSUPPORTED), (dict(scale=math.nan), INVALID), (dict(B=1, q=0), INVALID),
                     (dict(B=1, out=0), INVALID), (dict(B=1, prefix=0), INVALID), (dict(B=1, pages=0), INVALID),
                     (dict(B=1, table=0), INVALID), (dict(B=1, ws=0), WORKSPACE), (dict(B=1, ws_bytes=0), WORKSPACE)):
        assert call(**kw) == want, kw


def _cpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("call", [
    lambda: lsa.lsa_norm_rope(_cpu(2, 4, 64), _cpu(2, 4, 64)),
    lambda: lsa.lsa_norm_rope(_cpu(2, 4, 64, dtype=torch.float32), _cpu(2, 4, 64)),
    lambda: lsa.lsa_cache_append(_cpu(2, 576), _cpu(8, 576), _cpu(2, dtype=torch.int64)),
    lambda: lsa.lsa_prefix_attn(_cpu(1, 4, 576), _cpu(8, 576), 1.0, _cpu(1, 4, 512))])
def test_host_tensors_are_refused(call):
    with pytest.raises(lsa.LsaError) as e:
        call()
    assert e.value.status == INVALID
