"""The operators around the latent cache: the cases they are measured at, and their plain forms.

norm_rope     norms of index queries, queries and keys for each head, with the position rotation in the same pass
cache_append  a step's latent rows (and index keys) normed, rotated and written to their slots of the cache
prefix_attn   attention of a batch that shares one long prefix, each sequence with its own tokens in pages behind it
"""

import math

import torch

own = False

LATENT, VALUE, ROPE = 576, 512, 64  # a latent row: 512 compressed dims (the value) and 64 rotary dims


def listed():
    return [
        # index queries of one decode step (16 sequences, 64 index heads of 128 dims), to the FP8 indexer's codes
        dict(name="norm_rope_decode", op="norm_rope", T=16, H=64, D=128, norm="rms", off=0, R=64, layout="half",
             yarn=1.0, out="e4m3", far=131072, eps=1e-6),
        # index queries of a prefill chunk of 8192 tokens, bf16, whole heads rotated
        dict(name="norm_rope_prefill", op="norm_rope", T=8192, H=64, D=128, norm="rms", off=0, R=128,
             layout="interleaved", yarn=1.0, out="bf16", far=131072, eps=1e-6),
        # an odd chunk at far positions: layer norm with bias, half of each head rotated, long-context scaling, codes
        dict(name="norm_rope_codes_odd", op="norm_rope", T=4099, H=64, D=128, norm="layer", off=64, R=64,
             layout="half", yarn=32.0, out="e4m3", far=10000000, eps=1e-5),
        # the rotary part of absorbed queries into its place in [T, 128, 576], without a norm
        dict(name="rope_queries", op="norm_rope", T=2047, H=128, D=64, norm="none", off=0, R=64,
             layout="interleaved", yarn=32.0, out="part", far=131072, eps=0.0),
        # one token of each of 16 sequences into pages of 64, bf16 index keys
        dict(name="append_decode", op="append", T=16, slots=16384, keys="bf16", d_I=128, skip=0, far=131072),
        # a prefill chunk of 8192 tokens, index keys as e4m3 codes with a scale for each row
        dict(name="append_prefill", op="append", T=8192, slots=16384, keys="e4m3", d_I=128, skip=0, far=131072),
        # a ragged batch of several chunks padded to a multiple, its padding skipped; latent rows alone
        dict(name="append_ragged", op="append", T=1021, slots=4099, keys="none", d_I=128, skip=5, far=1048576),
        # a small batch of few heads behind a short prefix: latency
        dict(name="prefix_small", op="prefix", B=4, H=16, Lp=1024, tail=40, page=16),
        # one sequence behind a long prefix: the prefix's bytes
        dict(name="prefix_one", op="prefix", B=1, H=128, Lp=131072, tail=300, page=64),
        # the decode batch of the benchmark's sizes
        dict(name="prefix_decode", op="prefix", B=16, H=128, Lp=131072, tail=512, page=64),
        # a wide batch behind a shorter prefix of odd length
        dict(name="prefix_wide", op="prefix", B=64, H=128, Lp=32749, tail=1024, page=64),
        # fewer heads, odd numbers, tails longer than usual
        dict(name="prefix_heads32", op="prefix", B=33, H=32, Lp=10007, tail=2000, page=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "prefix"])
    if op == "norm_rope":
        D, off, R = rng.choice([(128, 0, 64), (128, 64, 64), (128, 0, 128), (64, 0, 64), (32, 0, 32), (576, 512, 64),
                                (192, 128, 64)])
        H = rng.choice([1, 4, 16, 33, 64, 128])
        T = min(_log(rng, 1, 8192), 8192 * 64 * 128 // (H * D))
        norm = rng.choice(["none", "rms", "layer"])
        out = rng.choice(["bf16", "e4m3"] + (["part"] if D == 64 else []))
        return dict(op=op, T=T, H=H, D=D, norm=norm, off=off, R=R, layout=rng.choice(["half", "interleaved"]),
                    yarn=rng.choice([1.0, 4.0, 32.0]), out=out, far=_log(rng, 4096, 10000000),
                    eps=rng.choice([1e-6, 1e-5]))
    if op == "append":
        T = _log(rng, 1, 8192)
        return dict(op=op, T=T, slots=T + _log(rng, 1, 8192), keys=rng.choice(["none", "bf16", "e4m3"]),
                    d_I=rng.choice([64, 128]), skip=rng.choice([0, 0, 3, 7]), far=_log(rng, 4096, 10000000))
    B, H = _log(rng, 1, 64), rng.choice([8, 16, 32, 64, 128])
    Lp = min(_log(rng, 256, 131072), 130000 * 2048 // (B * H))
    return dict(op=op, B=B, H=H, Lp=Lp, tail=_log(rng, 1, 1024), page=rng.choice([16, 32, 64, 128]))


# ------------------------------------------------------------------------------------------------ inputs


def _freqs(R, s):
    """Angular frequencies (64 bits) and the factor of cos and sin: base 10000, scaled for long contexts by YaRN."""
    f = [10000.0 ** (-2.0 * i / R) for i in range(R // 2)]
    if s == 1.0:
        return f, 1.0
    def dim(beta):
        return R * math.log(4096 / (beta * 2 * math.pi)) / (2 * math.log(10000.0))

    low, high = max(math.floor(dim(32)), 0), min(math.ceil(dim(1)), R - 1)
    ramp = [min(max((i - low) / max(high - low, 0.001), 0.0), 1.0) for i in range(R // 2)]
    return [(1 - r) * a + r * a / s for a, r in zip(f, ramp)], 0.1 * math.log(s) + 1.0


def _tails(c):
    """The own tokens of each sequence: spread over [1, tail], every seventh sequence has none yet."""
    return [0 if b % 7 == 3 else 1 + int((c["tail"] - 1) * (((b + 1) * 0.6180339887) % 1.0) + 0.5) for b in range(c["B"])]


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    c = dict(case)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    if c["op"] == "norm_rope":
        T, H, D = c["T"], c["H"], c["D"]
        f, mul = _freqs(c["R"], c["yarn"])
        st = dict(case=c, mul=mul, freqs=torch.tensor(f, dtype=torch.float64, device=dev))
        st["x"] = (normal(T, H, D) * 1.5 + 0.25).bfloat16()
        st["pos"] = torch.randint(0, c["far"], (T,), generator=g, device=dev)
        st["weight"] = 1 + 0.2 * normal(D) if c["norm"] != "none" else None
        st["bias"] = 0.1 * normal(D) if c["norm"] == "layer" else None
        st["scale"] = torch.empty(T, H, device=dev) if c["out"] == "e4m3" else None
        if c["out"] == "part":
            st["y"] = normal(T, H, LATENT).bfloat16()[:, :, VALUE:]
        else:
            st["y"] = torch.empty(T, H, D, dtype=torch.uint8 if c["out"] == "e4m3" else torch.bfloat16, device=dev)
        return st
    if c["op"] == "append":
        T, n, d = c["T"], c["slots"], c["d_I"]
        f, mul = _freqs(ROPE, 1.0)
        st = dict(case=c, mul=mul, freqs=torch.tensor(f, dtype=torch.float64, device=dev))
        st["a"] = normal(T, LATENT).bfloat16()
        st["a_weight"] = 1 + 0.2 * normal(VALUE)
        st["pos"] = torch.randint(0, c["far"], (T,), generator=g, device=dev)
        st["slot"] = torch.randperm(n, generator=g, device=dev)[:T].contiguous()
        if c["skip"]:
            st["slot"][torch.arange(T, device=dev) % c["skip"] == c["skip"] - 1] = -1
        st["kv"] = normal(n, LATENT).bfloat16()
        st["k"] = st["k_cache"] = st["k_scale"] = None
        if c["keys"] != "none":
            st["k"] = normal(T, d).bfloat16()
            st["k_weight"], st["k_bias"] = 1 + 0.2 * normal(d), 0.1 * normal(d)
            st["k_cache"] = normal(n, d).bfloat16()
            if c["keys"] == "e4m3":
                st["k_cache"] = (40 * normal(n, d)).to(torch.float8_e4m3fn).view(torch.uint8)
                st["k_scale"] = 0.01 + 0.001 * normal(n).abs()
        return st
    B, H, page = c["B"], c["H"], c["page"]
    lens = _tails(c)
    cols = max(1, -(-c["tail"] // page))
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 5
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((B, cols), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at : at + n]
        at += n
    st = dict(case=c, scale=LATENT ** -0.5, table=table, own_len=torch.tensor(lens, dtype=torch.int32, device=dev))
    # queries whose logits have a spread of about 2, latents of unit variance
    st["q"] = (2 * normal(B, H, LATENT)).bfloat16()
    st["prefix"] = normal(c["Lp"], LATENT).bfloat16()
    st["pages"] = normal(pages, page, LATENT).bfloat16()
    st["out"] = torch.empty(B, H, VALUE, dtype=torch.bfloat16, device=dev)
    st["lse"] = torch.empty(B, H, device=dev)
    return st


# ------------------------------------------------------------------------------------------------ plain forms


def _rotate(y, pos, freqs, off, layout, mul):
    """y [..., D] fp32 with its first axis the token's: dims [off, off + R) rotated by pos * freqs."""
    R = 2 * freqs.numel()
    a = pos.double().unsqueeze(-1) * freqs  # 64 bits: an fp32 angle at position 1e7 is off by half a radian
    shape = [a.shape[0]] + [1] * (y.dim() - 2) + [R // 2]
    cos, sin = (torch.cos(a) * mul).float().view(shape), (torch.sin(a) * mul).float().view(shape)
    r = y[..., off : off + R]
    if layout == "half":
        u, v = r[..., : R // 2], r[..., R // 2 :]
        r = torch.cat([u * cos - v * sin, v * cos + u * sin], -1)
    else:
        u, v = r[..., 0::2], r[..., 1::2]
        r = torch.stack([u * cos - v * sin, v * cos + u * sin], -1).flatten(-2)
    return torch.cat([y[..., :off], r, y[..., off + R :]], -1)


def _norm(y, kind, weight, bias, eps):
    if kind == "rms":
        return y * torch.rsqrt((y * y).mean(-1, keepdim=True) + eps) * weight
    if kind == "layer":
        y = y - y.mean(-1, keepdim=True)
        return y * torch.rsqrt((y * y).mean(-1, keepdim=True) + eps) * weight + bias
    return y


def _codes(y):
    """e4m3 codes with one scale for each row: amax / 448, 1 for a row of zeros."""
    amax = y.abs().amax(-1)
    scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    return (y / scale.unsqueeze(-1)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale


def _plain_norm_rope(s):
    c = s["case"]
    y = _norm(s["x"].float(), c["norm"], s["weight"], s["bias"], c["eps"])
    y = _rotate(y, s["pos"], s["freqs"], c["off"], c["layout"], s["mul"])
    if c["out"] == "e4m3":
        codes, scale = _codes(y)
        return {"codes": codes, "scale": scale}
    if c["out"] == "part":
        s["y"].copy_(y)
        return {"y": s["y"]}
    return {"y": y.bfloat16()}


def _plain_append(s):
    c = s["case"]
    keep = s["slot"] >= 0
    slot = s["slot"][keep]
    a = s["a"].float()
    row = torch.cat([_norm(a[:, :VALUE], "rms", s["a_weight"], None, 1e-6), a[:, VALUE:]], -1)
    row = _rotate(row, s["pos"], s["freqs"], VALUE, "interleaved", s["mul"])
    s["kv"][slot] = row.bfloat16()[keep]
    r = {"kv": s["kv"]}
    if c["keys"] != "none":
        k = _norm(s["k"].float(), "layer", s["k_weight"], s["k_bias"], 1e-5)
        k = _rotate(k, s["pos"], s["freqs"], 0, "half", s["mul"])
        if c["keys"] == "e4m3":
            codes, scale = _codes(k)
            s["k_cache"][slot] = codes.view(torch.uint8)[keep]
            s["k_scale"][slot] = scale[keep]
            r["k_cache"], r["k_scale"] = s["k_cache"].view(torch.float8_e4m3fn), s["k_scale"]
        else:
            s["k_cache"][slot] = k.bfloat16()[keep]
            r["k_cache"] = s["k_cache"]
    return r


def _plain_prefix(s):
    c = s["case"]
    B, H, page = c["B"], c["H"], c["page"]
    q, prefix = s["q"].float(), s["prefix"].float()
    at = torch.arange(s["table"].shape[1] * page, device=q.device)
    rows = s["pages"][s["table"].clamp(min=0).long()].float().view(B, -1, LATENT)
    s_own = torch.matmul(q, rows.transpose(1, 2)) * s["scale"]
    s_own = s_own.masked_fill((at >= s["own_len"].unsqueeze(1)).unsqueeze(1), -math.inf)
    s_pre = (q.view(B * H, LATENT) @ prefix.T).view(B, H, -1) * s["scale"]
    m = torch.maximum(s_pre.amax(-1), s_own.amax(-1)).unsqueeze(-1)
    p_pre, p_own = torch.exp(s_pre - m), torch.exp(s_own - m)
    total = p_pre.sum(-1) + p_own.sum(-1)
    o = (p_pre.view(B * H, -1) @ prefix[:, :VALUE]).view(B, H, VALUE) + torch.matmul(p_own, rows[:, :, :VALUE])
    return {"out": (o / total.unsqueeze(-1)).bfloat16(), "lse": m.squeeze(-1) + torch.log(total)}


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"norm_rope": _plain_norm_rope, "append": _plain_append, "prefix": _plain_prefix}[c["op"]](s)
    import sparse_long_context_lightning_b200 as lsa

    if c["op"] == "norm_rope":
        lsa.lsa_norm_rope(s["x"], s["y"], s["pos"], s["freqs"], norm=c["norm"], weight=s["weight"], bias=s["bias"],
                          eps=c["eps"], rope_off=c["off"], layout=c["layout"], mul=s["mul"], y_scale=s["scale"])
        if c["out"] == "e4m3":
            return {"codes": s["y"].view(torch.float8_e4m3fn), "scale": s["scale"]}
        return {"y": s["y"]}
    if c["op"] == "append":
        if c["keys"] == "none":
            lsa.lsa_cache_append(s["a"], s["kv"], s["slot"], s["pos"], s["freqs"], kv_weight=s["a_weight"],
                                 kv_eps=1e-6, layout="interleaved", mul=s["mul"])
            return {"kv": s["kv"]}
        lsa.lsa_cache_append(s["a"], s["kv"], s["slot"], s["pos"], s["freqs"], kv_weight=s["a_weight"], kv_eps=1e-6,
                             layout="interleaved", mul=s["mul"], k=s["k"], k_cache=s["k_cache"],
                             k_scale=s["k_scale"], k_norm="layer", k_weight=s["k_weight"], k_bias=s["k_bias"],
                             k_eps=1e-5, k_rope_off=0, k_layout="half")
        if c["keys"] == "e4m3":
            return {"kv": s["kv"], "k_cache": s["k_cache"].view(torch.float8_e4m3fn), "k_scale": s["k_scale"]}
        return {"kv": s["kv"], "k_cache": s["k_cache"]}
    if "ws" not in s:  # a program keeps its workspace from step to step
        s["ws"] = lsa.workspace(lsa.lsa_prefix_attn_workspace_size(c["B"], c["H"]), s["q"].device)
    lsa.lsa_prefix_attn(s["q"], s["prefix"], s["scale"], s["out"], s["lse"], pages=s["pages"], table=s["table"],
                        own_len=s["own_len"], ws=s["ws"])
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------------------------------------ work


def work(case):
    c = case
    if c["op"] == "norm_rope":
        n = c["T"] * c["H"] * c["D"]
        out = n + 4 * c["T"] * c["H"] if c["out"] == "e4m3" else 2 * n
        return {"bytes": 2 * n + out + 8 * c["T"], "flops": 8 * n}
    if c["op"] == "append":
        live = c["T"] - (c["T"] // c["skip"] if c["skip"] else 0)
        row = 2 * 2 * LATENT + {"none": 0, "bf16": 4 * c["d_I"], "e4m3": 3 * c["d_I"] + 4}[c["keys"]]
        return {"bytes": live * row + 16 * c["T"], "flops": 8 * live * (LATENT + (c["d_I"] if c["keys"] != "none" else 0))}
    lens = _tails(c)
    B, H = c["B"], c["H"]
    nbytes = 2 * LATENT * (c["Lp"] + sum(lens)) + B * H * (2 * LATENT + 2 * VALUE + 4)
    return {"bytes": nbytes, "flops": 2 * H * (LATENT + VALUE) * (B * c["Lp"] + sum(lens))}


# ------------------------------------------------------------------------------------------------ 64 bits


def _exact_turn(v, pos, freqs, layout, mul):
    """Complex form of the rotation: v [N, ..., R] in 64 bits, the angle of pair i is pos * freqs[i]."""
    R = v.shape[-1]
    z = torch.complex(v[..., : R // 2], v[..., R // 2 :]) if layout == "half" else torch.view_as_complex(
        v.reshape(*v.shape[:-1], R // 2, 2).contiguous())
    a = torch.outer(pos.double(), freqs)
    z = z * torch.polar(torch.full_like(a, mul), a).view([a.shape[0]] + [1] * (z.dim() - 2) + [R // 2])
    return torch.cat([z.real, z.imag], -1) if layout == "half" else torch.view_as_real(z).flatten(-2)


def _exact_norm(v, kind, weight, bias, eps):
    if kind == "none":
        return v
    mean = v.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(v[..., :1])
    second = ((v - mean) ** 2).sum(-1, keepdim=True) / v.shape[-1]
    v = (v - mean) / torch.sqrt(second + eps) * weight.double()
    return v + bias.double() if bias is not None else v


def _exact_scale(v):
    top = v.abs().max(-1).values / 448
    return torch.where(top > 0, top, torch.ones_like(top))


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "norm_rope":
        y = _exact_norm(s["x"].double(), c["norm"], s["weight"], s["bias"], c["eps"])
        end = c["off"] + c["R"]
        y[..., c["off"] : end] = _exact_turn(y[..., c["off"] : end].clone(), s["pos"], s["freqs"], c["layout"], s["mul"])
        if c["out"] == "e4m3":
            k = _exact_scale(y)
            return {"codes": y / k[..., None], "scale": k}
        return {"y": y}
    if c["op"] == "append":
        a = s["a"].double()
        low = _exact_norm(a[:, :VALUE], "rms", s["a_weight"], None, 1e-6)
        rows = torch.cat([low, _exact_turn(a[:, VALUE:], s["pos"], s["freqs"], "interleaved", s["mul"])], 1)
        live = torch.nonzero(s["slot"] >= 0).flatten()
        at = s["slot"][live]
        r = {"kv": s["kv"].double().index_copy(0, at, rows[live])}
        if c["keys"] != "none":
            k = _exact_norm(s["k"].double(), "layer", s["k_weight"], s["k_bias"], 1e-5)
            k[:, :ROPE] = _exact_turn(k[:, :ROPE].clone(), s["pos"], s["freqs"], "half", s["mul"])
            if c["keys"] == "e4m3":
                top = _exact_scale(k)
                old = s["k_cache"].view(torch.float8_e4m3fn).double()
                r["k_cache"] = old.index_copy(0, at, (k / top[:, None])[live])
                r["k_scale"] = s["k_scale"].double().index_copy(0, at, top[live])
            else:
                r["k_cache"] = s["k_cache"].double().index_copy(0, at, k[live])
        return r
    # one query at a time: softmax over the prefix rows and the query's own rows, joined
    prefix = s["prefix"].double()
    flat = s["pages"].double().view(-1, LATENT)
    page = c["page"]
    outs, lses = [], []
    for b, n in enumerate(_tails(c)):
        i = torch.arange(n, device=prefix.device)
        mine = flat[s["table"][b].long()[i // page] * page + i % page]
        logits = [s["q"][b].double() @ prefix.T * s["scale"], s["q"][b].double() @ mine.T * s["scale"]]
        lse = torch.logsumexp(torch.cat([torch.logsumexp(x, 1, keepdim=True) for x in logits], 1), 1, keepdim=True)
        outs.append(torch.exp(logits[0] - lse) @ prefix[:, :VALUE] + torch.exp(logits[1] - lse) @ mine[:, :VALUE])
        lses.append(lse.squeeze(1))
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}
