"""Cases of the attention-side operators: per-head norm with rotation of queries
and keys, the append to the paged MXFP8 cache, and the attention of a chunk of
new tokens over that cache.

``prepare`` makes what a serving program holds before the call, ``run`` makes
one pass (the plain torch form, or the library's calls where ``own`` is true),
``exact`` gives the same outputs from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

EPS = 1e-6
THETA = 1e6
_fs = None


def _lib():
    global _fs
    if _fs is None:
        import mxfp8_swiglu_mlp_gb300 as fs

        _fs = fs
    return _fs


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one request decoding alone: the q and k rows of a single token, latency only
        dict(name="norm_rope_one", op="norm_rope", T=1, Hq=32, Hkv=8, D=128, R=128, interleaved=False, norm=True,
             far=4096, prompt=False),
        # a decode step of 64 sequences, each at its own position
        dict(name="norm_rope_step", op="norm_rope", T=64, Hq=32, Hkv=8, D=128, R=128, interleaved=False, norm=True,
             far=6144, prompt=False),
        # odd row count, small heads, half of each head rotated in adjacent pairs, far positions, no norm
        dict(name="norm_rope_odd", op="norm_rope", T=1777, Hq=14, Hkv=2, D=64, R=32, interleaved=True, norm=False,
             far=1000000, prompt=False),
        # long prompts: bandwidth
        dict(name="norm_rope_prompt", op="norm_rope", T=16384, Hq=32, Hkv=8, D=128, R=128, interleaved=False, norm=True,
             far=131072, prompt=True),
        # one token of one request into the cache
        dict(name="append_one", op="append", B=1, n_lo=1, n_hi=1, ctx_lo=4000, ctx_hi=4000, mixed=False, Hkv=8, P=16,
             R=128, interleaved=False, norm=True, pad=0, mix=1),
        # a decode step of 64 sequences into pages of 16
        dict(name="append_step", op="append", B=64, n_lo=1, n_hi=1, ctx_lo=255, ctx_hi=1100, mixed=False, Hkv=8, P=16,
             R=128, interleaved=False, norm=True, pad=0, mix=2),
        # three ragged prompts in a padded buffer, pages of 64
        dict(name="append_prompt", op="append", B=3, n_lo=1501, n_hi=6007, ctx_lo=0, ctx_hi=333, mixed=False, Hkv=8,
             P=64, R=128, interleaved=False, norm=True, pad=100, mix=3),
        # one token of one request against a short cache: latency only
        dict(name="chunk_one", op="chunk", B=1, n_lo=1, n_hi=1, ctx_lo=516, ctx_hi=516, mixed=False, Hq=32, Hkv=8, P=16,
             window=0, pad=0, mix=4),
        # five drafted tokens a sequence, 64 sequences of 2k-6k tokens: bound by the cache's bytes
        dict(name="chunk_verify", op="chunk", B=64, n_lo=5, n_hi=5, ctx_lo=2043, ctx_hi=6139, mixed=False, Hq=32, Hkv=8,
             P=16, window=0, pad=0, mix=5),
        # a mixed batch: three prompt chunks among decoding sequences, seven query heads a KV head, padded buffer
        dict(name="chunk_mixed", op="chunk", B=24, n_lo=1, n_hi=512, ctx_lo=100, ctx_hi=4096, mixed=True, Hq=28, Hkv=4,
             P=32, window=0, pad=7, mix=6),
        # sliding window over long contexts, two query heads a KV head
        dict(name="chunk_window", op="chunk", B=2, n_lo=1024, n_hi=1024, ctx_lo=8001, ctx_hi=12001, mixed=False, Hq=16,
             Hkv=8, P=128, window=4096, pad=0, mix=7),
        # the last chunk of a 16k-token prompt: bound by the products
        dict(name="chunk_prompt", op="chunk", B=1, n_lo=2048, n_hi=2048, ctx_lo=14336, ctx_hi=14336, mixed=False, Hq=32,
             Hkv=8, P=64, window=0, pad=0, mix=8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "chunk", "chunk"])
    if op == "norm_rope":
        D = rng.choice([64, 96, 128, 128, 192, 256])
        Hkv = rng.randint(1, 8)
        return dict(op=op, T=_log_int(rng, 1, 8192), Hq=Hkv * rng.randint(1, 5), Hkv=Hkv, D=D,
                    R=rng.choice([r for r in (32, 64, 96, 128, 192, 256) if r <= D]), interleaved=rng.random() < 0.4,
                    norm=rng.random() < 0.7, far=_log_int(rng, 1000, 1000000), prompt=rng.random() < 0.5)
    mixed = rng.random() < 0.3
    if op == "append":
        B = _log_int(rng, 1, 96)
        n_hi = max(1, _log_int(rng, 1, 8192) // B)
        return dict(op=op, B=B, n_lo=rng.randint(1, n_hi), n_hi=n_hi, ctx_lo=0, ctx_hi=_log_int(rng, 1, 1500),
                    mixed=mixed, Hkv=rng.randint(1, 12), P=rng.choice([16, 32, 64, 128]),
                    R=rng.choice([0, 32, 64, 96, 128, 128]), interleaved=rng.random() < 0.4, norm=rng.random() < 0.6,
                    pad=rng.choice([0, 0, rng.randint(1, 50)]), mix=rng.randrange(1 << 30))
    B = _log_int(rng, 1, 64)
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    ctx_hi = _log_int(rng, 16, 12000)
    # the plain form holds B * Hq * n_hi * (ctx_hi + n_hi) scores: at most 1.5e9
    n_hi = max(1, min(_log_int(rng, 1, 3000), int(1.5e9 / (B * Hkv * G * (ctx_hi + 3000)))))
    return dict(op=op, B=B, n_lo=rng.randint(1, n_hi), n_hi=n_hi, ctx_lo=rng.randint(0, ctx_hi), ctx_hi=ctx_hi,
                mixed=mixed, Hq=Hkv * G, Hkv=Hkv, P=rng.choice([16, 32, 64, 128]),
                window=rng.choice([0, 0, _log_int(rng, 16, 8000)]), pad=rng.choice([0, 0, rng.randint(1, 50)]),
                mix=rng.randrange(1 << 30))


def _lengths(case):
    """New tokens and tokens held before, of each sequence: from the case alone."""
    r = random.Random(case["mix"])
    new, ctx = [], []
    for b in range(case["B"]):
        if case["mixed"]:
            new.append(case["n_hi"] if b % 8 == 3 or case["B"] == 1 else case["n_lo"])
        else:
            new.append(r.randint(case["n_lo"], case["n_hi"]))
        ctx.append(r.randint(case["ctx_lo"], case["ctx_hi"]))
    return new, ctx


def work(case):
    if case["op"] == "norm_rope":
        n = case["T"] * (case["Hq"] + case["Hkv"]) * case["D"]
        return {"bytes": 4 * n + 4 * case["T"], "flops": 8 * n}
    new, ctx = _lengths(case)
    rows, D = sum(new), 128
    if case["op"] == "append":
        n = rows * case["Hkv"] * D
        return {"bytes": 2 * (2 * n + n + n // 32), "flops": 16 * n}
    W, keys, pairs = case["window"], 0, 0
    for n, c in zip(new, ctx):
        keys += c + n - (max(0, c + 1 - W) if W else 0)
        if W:
            k = max(0, min(n, W - 1 - c))  # rows that see everything before them
            pairs += k * c + k * (k + 1) // 2 + (n - k) * W
        else:
            pairs += n * c + n * (n + 1) // 2
    return {"bytes": 4 * rows * case["Hq"] * D + keys * case["Hkv"] * 2 * (D + D // 32),
            "flops": 4 * D * case["Hq"] * pairs}


# ---------------------------------------------------------------- inputs
def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _mxfp8(x):
    """fp32 [..., D] -> E4M3 codes [..., D] and UE8M0 scales [..., D / 32], as bytes (OCP MX rule)."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    e = torch.frexp(b.abs().amax(-1, keepdim=True))[1] - 9
    e = torch.where((b != 0).any(-1, keepdim=True), e.clamp(-127, 127), -127)
    c = torch.ldexp(b, -e).clamp(-448, 448).to(torch.float8_e4m3fn)
    return c.view(torch.uint8).reshape(x.shape), (e + 127).to(torch.uint8).squeeze(-1)


def _value(codes, scales):
    """MXFP8 bytes -> the fp32 values they stand for."""
    s = (scales.to(torch.int32) << 23).view(torch.float32)
    c = codes.view(torch.float8_e4m3fn).float()
    return (c.reshape(*scales.shape, 32) * s.unsqueeze(-1)).reshape(c.shape)


def _paged(case, g):
    """The cache with its page tables, filled with quantised keys and values, and the batch's offsets and lengths."""
    new, ctx = _lengths(case)
    B, P, Hkv, D = case["B"], case["P"], case["Hkv"], 128
    npg = [-(-(n + c) // P) for n, c in zip(new, ctx)]
    total, widest = sum(npg), max(npg)
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, widest), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(npg):
        table[b, :n] = perm[at:at + n]
        at += n
    cu = torch.tensor([sum(new[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda")
    lens = torch.tensor([n + c for n, c in zip(new, ctx)], dtype=torch.int32, device="cuda")
    s = dict(case=case, table=table, cu=cu, lens=lens, pages=total, max_pages=widest, rows=sum(new), n_max=max(new),
             len_max=max(n + c for n, c in zip(new, ctx)))
    for name in ("k", "v"):
        s[name + "_codes"], s[name + "_scales"] = _mxfp8(_normal(g, total, Hkv, P, D))
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    if op == "chunk":
        s = _paged(case, g)
        T = s["rows"] + case["pad"]
        s.update(T=T, q=_normal(g, T, case["Hq"], 128).to(torch.bfloat16),
                 out=torch.zeros(T, case["Hq"], 128, dtype=torch.bfloat16, device="cuda"))
        return s
    if op == "append":
        s = _paged(case, g)
        T, D, Hq = s["rows"] + case["pad"], 128, 4 * case["Hkv"]
    else:
        s, T, D, Hq = dict(case=case), case["T"], case["D"], case["Hq"]
    Hkv, R = case["Hkv"], case["R"]
    # the projection's output: q, k and v of a token in one row
    qkv = (_normal(g, T, (Hq + 2 * Hkv) * D) * torch.exp(0.5 * _normal(g, T, 1))).to(torch.bfloat16)
    s.update(T=T, ld=qkv.shape[1], q=qkv[:, :Hq * D], k=qkv[:, Hq * D:(Hq + Hkv) * D], v=qkv[:, (Hq + Hkv) * D:],
             inv_freq=(THETA ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / max(R, 1))).float())
    for name in ("gamma_q", "gamma_k"):
        s[name] = (1 + 0.1 * _normal(g, D)).to(torch.bfloat16) if case["norm"] else None
    if op == "append":
        s["status"] = torch.zeros(64, dtype=torch.int32, device="cuda")
        return s
    at = torch.randint(0, case["far"], (T,), generator=g, device="cuda")
    s["positions"] = (at[0] + torch.arange(T, device="cuda") if case["prompt"] else at).to(torch.int32)
    s["q_out"] = torch.empty(T, Hq * D, dtype=torch.bfloat16, device="cuda")
    s["k_out"] = torch.empty(T, Hkv * D, dtype=torch.bfloat16, device="cuda")
    return s


# ---------------------------------------------------------------- the plain forms
def _norm_rotate(x, heads, gamma, s, pos):
    """fp32 [T, heads, D]: the per-head norm and the rotation; angles in 64 bits."""
    c = s["case"]
    R, T = c["R"], x.shape[0]
    x = x.float().reshape(T, heads, -1)
    if gamma is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gamma.float()
    if not R:
        return x
    a = pos.double()[:, None] * s["inv_freq"].double()
    cos, sin = torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]
    r = x[..., :R]
    if c["interleaved"]:
        u, w = r[..., 0::2], r[..., 1::2]
        r = torch.stack([u * cos - w * sin, w * cos + u * sin], -1).reshape(T, heads, R)
    else:
        u, w = r[..., :R // 2], r[..., R // 2:]
        r = torch.cat([u * cos - w * sin, w * cos + u * sin], -1)
    return torch.cat([r, x[..., R:]], -1)


def _rows(s):
    """Sequence, place in its chunk and position of every row in use."""
    t = torch.arange(s["rows"], device="cuda")
    b = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    i = t - s["cu"][b]
    return b, i, s["lens"][b] - (s["cu"][b + 1] - s["cu"][b]) + i


def _plain_append(s):
    c = s["case"]
    n, Hkv, P = s["rows"], c["Hkv"], c["P"]
    b, _, pos = _rows(s)
    k = _norm_rotate(s["k"][:n], Hkv, s["gamma_k"], s, pos)
    page, slot = s["table"][b, pos // P].long(), (pos % P).long()
    for name, x in (("k", k), ("v", s["v"][:n].float().reshape(n, Hkv, 128))):
        codes, scales = _mxfp8(x)
        s[name + "_codes"][page, :, slot] = codes
        s[name + "_scales"][page, :, slot] = scales


def _plain_chunk(s):
    c = s["case"]
    B, Hq, Hkv, L, n = c["B"], c["Hq"], c["Hkv"], s["len_max"], s["n_max"]
    G = Hq // Hkv
    pages = s["table"].clamp(min=0).long()
    kv = []
    for name in ("k", "v"):
        x = _value(s[name + "_codes"][pages], s[name + "_scales"][pages])  # [B, pages, Hkv, P, D]
        kv.append(x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, 128)[:, :, :L])
    i = torch.arange(n, device="cuda")
    rows = (s["cu"][:-1, None] + i).clamp(max=s["T"] - 1).long()
    q = s["q"][rows].float().reshape(B, n, Hkv, G, 128).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, 128)
    x = torch.matmul(q, kv[0].transpose(-1, -2))
    x = x.mul_(1 / math.sqrt(128)).reshape(B, Hkv, n, G, L)
    t = torch.arange(L, device="cuda")
    pos = (s["lens"] - (s["cu"][1:] - s["cu"][:-1]))[:, None] + i  # [B, n]
    hidden = t > pos[..., None]
    if c["window"]:
        hidden |= t <= pos[..., None] - c["window"]
    x.masked_fill_(hidden[:, None, :, None, :], -math.inf)
    x = x.sub_(x.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
    o = torch.matmul(x.reshape(B, Hkv, n * G, L), kv[1]) / x.sum(-1).reshape(B, Hkv, n * G, 1)
    o = o.reshape(B, Hkv, n, G, 128).permute(0, 2, 1, 3, 4).reshape(B, n, Hq, 128)
    b, i, _ = _rows(s)
    s["out"][:s["rows"]] = o[b, i].to(torch.bfloat16)


# ---------------------------------------------------------------- one pass
def _cache(s):
    """The cache as it stands after the pass: codes and scales by their values."""
    return {name + kind: s[name + kind].view(t) for name in ("k", "v")
            for kind, t in (("_codes", torch.float8_e4m3fn), ("_scales", torch.float8_e8m0fnu))}


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        fs = _lib()
    if op == "norm_rope":
        Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
        if own:
            fs.fsops_qk_norm_rope(s["q"], s["ld"], s["k"], s["ld"], s["gamma_q"], s["gamma_k"], EPS, s["positions"],
                                  (s["inv_freq"], c["R"], c["interleaved"]), s["q_out"], Hq * D, s["k_out"], Hkv * D,
                                  s["T"], Hq, Hkv, D)
            return {"q": s["q_out"], "k": s["k_out"]}
        q = _norm_rotate(s["q"], Hq, s["gamma_q"], s, s["positions"])
        k = _norm_rotate(s["k"], Hkv, s["gamma_k"], s, s["positions"])
        return {"q": q.to(torch.bfloat16).reshape(-1, Hq * D), "k": k.to(torch.bfloat16).reshape(-1, Hkv * D)}
    if op == "append":
        if own:
            fs.fsops_mxfp8_kv_append(s["k"], s["ld"], s["v"], s["ld"], s["gamma_k"], EPS, None,
                                     (s["inv_freq"], c["R"], c["interleaved"]) if c["R"] else None, s["k_codes"],
                                     s["k_scales"], s["v_codes"], s["v_scales"], s["pages"], s["table"],
                                     s["max_pages"], s["cu"], s["lens"], s["T"], c["B"], c["Hkv"], 128, c["P"],
                                     s["status"])
        else:
            _plain_append(s)
        return _cache(s)
    if own:
        if "ws" not in s:  # kept beside the cache, as a serving program keeps it
            s["ws_bytes"] = fs.fsops_paged_chunk_attention_workspace_bytes(s["T"], c["B"], c["Hq"], c["Hkv"], 128,
                                                                           c["P"], s["max_pages"])
            s["ws"] = torch.zeros(s["ws_bytes"], dtype=torch.uint8, device="cuda")
        fs.fsops_mxfp8_paged_chunk_attention(s["q"], c["Hq"] * 128, s["k_codes"], s["k_scales"], s["v_codes"],
                                             s["v_scales"], s["pages"], s["table"], s["max_pages"], s["cu"], s["lens"],
                                             s["out"], c["Hq"] * 128, s["T"], c["B"], c["Hq"], c["Hkv"], 128, c["P"],
                                             c["window"], 1 / math.sqrt(128), s["ws"], s["ws_bytes"])
    else:
        _plain_chunk(s)
    return s["out"]


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_heads(x, heads, gamma, s, pos):
    c = s["case"]
    R = c["R"]
    x = x.double().unflatten(-1, (heads, -1))
    if gamma is not None:
        x = x / ((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * gamma.double()
    if R:
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                           pos.double().outer(s["inv_freq"].double()))[:, None]
        pairs = x[..., :R].unflatten(-1, (-1, 2)) if c["interleaved"] else x[..., :R].unflatten(-1, (2, -1)).mT
        pairs = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        x[..., :R] = (pairs if c["interleaved"] else pairs.mT).flatten(-2)
    return x


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm_rope":
        return {n: _exact_heads(s[n], h, s["gamma_" + n], s, s["positions"]).flatten(1)
                for n, h in (("q", case["Hq"]), ("k", case["Hkv"]))}
    new, ctx = _lengths(case)
    Hkv, P, D = case["Hkv"], case["P"], 128
    table = s["table"].long()
    if op == "append":
        # codes before their rounding to E4M3, scales by the MX rule: 2^(floor(log2 amax) - 8)
        held = {n: s[n].view(t).double() for t, ns in ((torch.float8_e4m3fn, ("k_codes", "v_codes")),
                                                       (torch.float8_e8m0fnu, ("k_scales", "v_scales"))) for n in ns}
        r = 0
        for b in range(case["B"]):
            pos = torch.arange(ctx[b], ctx[b] + new[b], device="cuda")
            rows = slice(r, r + new[b])
            r += new[b]
            for n in ("k", "v"):
                x = (_exact_heads(s["k"][rows], Hkv, s["gamma_k"], s, pos) if n == "k"
                     else s["v"][rows].double().unflatten(-1, (Hkv, -1)))
                x = x.unflatten(-1, (-1, 32))
                e = (torch.frexp(x.abs().amax(-1))[1] - 9).clamp(-127, 127).double()
                page, slot = table[b, pos // P], pos % P
                held[n + "_codes"][page, :, slot] = (x * torch.exp2(-e)[..., None]).clamp(-448, 448).flatten(-2)
                held[n + "_scales"][page, :, slot] = torch.exp2(e)
        return held
    G, W, r = case["Hq"] // Hkv, case["window"], 0
    out = torch.zeros(s["T"], case["Hq"], D, dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        n, L = new[b], new[b] + ctx[b]
        at = torch.arange(L, device="cuda")
        page, slot = table[b, at // P], at % P
        pos = torch.arange(ctx[b], L, device="cuda")[:, None]
        seen = at <= pos
        if W:
            seen &= at > pos - W
        for h in range(Hkv):
            k, v = ((s[x + "_codes"][page, h, slot].view(torch.float8_e4m3fn).double().unflatten(-1, (-1, 32))
                     * torch.exp2(s[x + "_scales"][page, h, slot].double() - 127)[..., None]).flatten(-2)
                    for x in ("k", "v"))
            for j in range(h * G, h * G + G):
                x = s["q"][r:r + n, j].double() @ k.T / math.sqrt(D)
                out[r:r + n, j] = torch.softmax(x.masked_fill(~seen, -math.inf), -1) @ v
        r += n
    return out
