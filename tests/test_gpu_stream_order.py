"""Attention kernels beside the kernels around them on their stream: queries that have no rows to attend to, whose own
copies are still under way when the output is formed, and queries written by the kernel right ahead."""

import math

import pytest
import torch

import sparse_long_context_lightning_b200 as lsa

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _sparse(q, kv, idx, cnt, ws):
    B, H = q.shape[:2]
    out = torch.full((B, H, 512), math.nan, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((B, H), math.nan, device=DEV)
    lsa.lsa_sparse_attn(q, kv, idx, cnt, 0.04, out, lse, ws)
    return out, lse


@pytest.mark.parametrize("H", [16, 128])
@pytest.mark.parametrize("B,ld", [(4, 64), (5, 512), (140, 32)])  # one unit a query; several; a whole wave of one-tile units
def test_empty_rows_of_the_sparse_attention(B, ld, H):
    """A query without rows gives zeros, whatever its query holds and however late its copy lands."""
    g, L = _gen(B + H), 2000
    kv = _randn(g, L, 576).bfloat16()
    idx = torch.stack([torch.randperm(L, generator=g, device=DEV)[:ld] for _ in range(B)]).int().contiguous()
    cnt = torch.full((B,), ld, dtype=torch.int32, device=DEV)
    cnt[::2] = 0
    ws = lsa.workspace(lsa.lsa_workspace_size(lsa.LSA_OP_ATTN, B, L, ld, H), DEV)
    got = []
    for i in range(20):
        got.append(_sparse((1 + i) * torch.ones(B, H, 576, device=DEV).bfloat16(), kv, idx, cnt, ws))
    torch.cuda.synchronize()
    for out, lse in got:
        assert not out[::2].any() and bool((lse[::2] == -math.inf).all())
        assert bool(torch.isfinite(out[1::2].float()).all()) and bool(torch.isfinite(lse[1::2]).all())
    lsa.lsa_device_status()


@pytest.mark.parametrize("G", [2, 4, 8])
def test_empty_groups_of_the_msa_attention(G):
    """A group that kept no block gives zeros, and what runs behind it on its SM is not disturbed: the same call again and
    again, each with the bytes of the first."""
    g, B, L = _gen(G), 40, 1024
    kv, q = _randn(g, L, 576).bfloat16(), (2 * _randn(g, B, 128, 576)).bfloat16()
    idx = torch.arange(256, dtype=torch.int32, device=DEV).expand(B, 256).contiguous()
    cnt = torch.full((B,), 256, dtype=torch.int32, device=DEV)
    cnt[3::5] = 0
    gmask = torch.full((B, 256), 1, dtype=torch.uint8, device=DEV)  # group 0 alone
    gmask[1::2] = (1 << G) - 1
    outs = []
    for _ in range(20):
        out, lse = torch.full((B, 128, 512), math.nan, dtype=torch.bfloat16, device=DEV), torch.full((B, 128), math.nan, device=DEV)
        lsa.lsa_msa_attn(q, kv, idx, gmask, cnt, G, 0.04, out, lse)
        outs.append((out, lse))
    torch.cuda.synchronize()
    has = torch.ones(B, 128, dtype=torch.bool, device=DEV)
    has[::2, 128 // G:] = False
    has[3::5] = False
    for out, lse in outs:
        assert not out[~has].any() and bool((lse[~has] == -math.inf).all()) and bool(torch.isfinite(lse[has]).all())
        assert torch.equal(out, outs[0][0]) and torch.equal(lse, outs[0][1])
    lsa.lsa_device_status()


# ------------------------------------------------------------------------------------------------ queries written right ahead


def _check_ahead(calls, n=24):
    """`calls(i)`: write query i and attend.  Back to back, then each alone with the device idle ahead of the attention."""
    write, attend = calls
    outs = []
    for i in range(n):
        write(i)
        outs.append(attend())
    torch.cuda.synchronize()
    for i in range(n):
        write(i)
        torch.cuda.synchronize()
        want = attend()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], want), i


@pytest.mark.parametrize("B,H,ld", [(16, 32, 256), (16, 128, 2048), (2, 128, 64), (300, 128, 256)])
def test_queries_rotated_right_before_the_sparse_attention(B, H, ld):
    """The rotation writes the query and the attention follows at once: padded heads, many units a query, one unit, and a
    batch that runs the value-half kernel."""
    g, L, n = _gen(B + ld), 4096, 24
    kv = _randn(g, L, 576).bfloat16()
    raw = [(2 * _randn(g, B, H, 576)).bfloat16() for _ in range(n)]
    pos = torch.randint(0, 100000, (B,), generator=g, device=DEV)
    freqs, _ = lsa.lsa_rope_freqs(64)
    idx = torch.stack([torch.randperm(L, generator=g, device=DEV)[:ld].sort().values for _ in range(B)]).int().contiguous()
    cnt = torch.full((B,), ld, dtype=torch.int32, device=DEV)
    ws = lsa.workspace(lsa.lsa_workspace_size(lsa.LSA_OP_ATTN, B, L, ld, H), DEV)
    q = torch.zeros_like(raw[0])

    def write(i):
        lsa.lsa_norm_rope(raw[i], q, pos, freqs, norm="rms", rope_off=512)

    def attend():
        out = torch.empty(B, H, 512, dtype=torch.bfloat16, device=DEV)
        lsa.lsa_sparse_attn(q, kv, idx, cnt, 0.04, out, None, ws)
        return out

    _check_ahead((write, attend))


def test_queries_rotated_right_before_the_msa_attention():
    g, B, L, G, n = _gen(3), 16, 1024, 4, 24
    kv = _randn(g, L, 576).bfloat16()
    raw = [(2 * _randn(g, B, 128, 576)).bfloat16() for _ in range(n)]
    pos = torch.randint(0, 100000, (B,), generator=g, device=DEV)
    freqs, _ = lsa.lsa_rope_freqs(64)
    idx = torch.arange(512, dtype=torch.int32, device=DEV).expand(B, 512).contiguous()
    cnt = torch.full((B,), 512, dtype=torch.int32, device=DEV)
    gmask = torch.full((B, 512), (1 << G) - 1, dtype=torch.uint8, device=DEV)
    q = torch.zeros_like(raw[0])

    def write(i):
        lsa.lsa_norm_rope(raw[i], q, pos, freqs, norm="rms", rope_off=512)

    def attend():
        out = torch.empty(B, 128, 512, dtype=torch.bfloat16, device=DEV)
        lsa.lsa_msa_attn(q, kv, idx, gmask, cnt, G, 0.04, out)
        return out

    _check_ahead((write, attend))


def test_queries_written_by_any_kernel_right_before_the_attention():
    """The same with a kernel ahead that is not this library's."""
    g, B, H, L, ld, n = _gen(4), 16, 128, 4096, 256, 24
    kv = _randn(g, L, 576).bfloat16()
    raw = [(2 * _randn(g, B, H, 576)).bfloat16() for _ in range(n)]
    idx = torch.stack([torch.randperm(L, generator=g, device=DEV)[:ld].sort().values for _ in range(B)]).int().contiguous()
    cnt = torch.full((B,), ld, dtype=torch.int32, device=DEV)
    ws = lsa.workspace(lsa.lsa_workspace_size(lsa.LSA_OP_ATTN, B, L, ld, H), DEV)
    q = torch.zeros_like(raw[0])

    def attend():
        out = torch.empty(B, H, 512, dtype=torch.bfloat16, device=DEV)
        lsa.lsa_sparse_attn(q, kv, idx, cnt, 0.04, out, None, ws)
        return out

    _check_ahead((lambda i: torch.mul(raw[i], 0.5, out=q), attend))
