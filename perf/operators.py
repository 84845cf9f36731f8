"""The serving operators around a MosaicQuant layer, as cases to be measured.

Four operators, each in a plain form (elementary torch operations) and as the call a
program makes of this package:

* ``gemv``  Y = g_w X (Q(W) + R)^T for up to 16 tokens of 16-bit activations on the packed
  NVFP4 base and residual blocks that ``mq_gemm`` reads.
* ``rope``  RMS norm of every query and key head with the position rotation.
* ``append``  keys and values into the paged 4-bit cache, and the same slots read back.
* ``attn``  attention of query tokens over that cache (pages, ragged lengths, causal).

The cache is a byte tensor [pages][kv heads][page/16][18 D]: one record holds 16 tokens of
one head. ``record_maps`` states where each of its bytes lies.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------- the cases
def listed():
    return [
        # one token through LLaMA3-8B's q_proj with its 10 % residual: a call's latency
        {"name": "gemv_q_proj_1", "op": "gemv", "M": 1, "N": 4096, "K": 4096, "frac": 0.10, "dtype": "bf16"},
        # four sequences through the LLaMA3-8B MLP up layer
        {"name": "gemv_mlp_up_4", "op": "gemv", "M": 4, "N": 14336, "K": 4096, "frac": 0.10, "dtype": "bf16"},
        # the decode batch of 16 through the Qwen3-32B down layer, fp16, base alone
        {"name": "gemv_down_16", "op": "gemv", "M": 16, "N": 5120, "K": 25600, "frac": 0.0, "dtype": "f16"},
        # a decode step of 16 sequences, Qwen3-32B heads (norms, 64 query and 8 key heads)
        {"name": "rope_decode_16", "op": "rope", "T": 16, "Hq": 64, "Hk": 8, "D": 128, "rot": 128, "norm": True,
         "inter": False, "theta": 1e6, "far": 131072, "dtype": "bf16"},
        # a prompt of 8191 tokens, LLaMA3-8B heads (rotation without norms)
        {"name": "rope_prompt_8191", "op": "rope", "T": 8191, "Hq": 32, "Hk": 8, "D": 128, "rot": 128, "norm": False,
         "inter": False, "theta": 5e5, "far": 8192, "dtype": "bf16"},
        # the keys and values of one decode step
        {"name": "append_decode_16", "op": "append", "T": 16, "H": 8, "D": 128, "P": 64, "pages": 2048, "dtype": "bf16"},
        # those of a prompt
        {"name": "append_prompt_8191", "op": "append", "T": 8191, "H": 8, "D": 128, "P": 64, "pages": 256,
         "dtype": "bf16"},
        # one short conversation: latency
        {"name": "attn_1x509", "op": "attn", "B": 1, "len": 509, "ragged": False, "nq": 1, "Hq": 32, "Hk": 8, "D": 128,
         "P": 64, "window": 0, "dtype": "bf16"},
        # the decode batch of 16, ragged lengths
        {"name": "attn_16x8192_ragged", "op": "attn", "B": 16, "len": 8192, "ragged": True, "nq": 1, "Hq": 64, "Hk": 8,
         "D": 128, "P": 64, "window": 0, "dtype": "bf16"},
        # few long documents
        {"name": "attn_4x131072", "op": "attn", "B": 4, "len": 131072, "ragged": False, "nq": 1, "Hq": 64, "Hk": 8,
         "D": 128, "P": 128, "window": 0, "dtype": "bf16"},
        # five drafted tokens a sequence, checked at once
        {"name": "attn_verify_8x5", "op": "attn", "B": 8, "len": 4001, "ragged": True, "nq": 5, "Hq": 32, "Hk": 8,
         "D": 128, "P": 32, "window": 0, "dtype": "f16"},
        # a chunk of 512 prompt tokens behind a cached prefix
        {"name": "attn_chunk_2x512", "op": "attn", "B": 2, "len": 8192, "ragged": False, "nq": 512, "Hq": 32, "Hk": 8,
         "D": 128, "P": 64, "window": 0, "dtype": "bf16"},
    ]


def draw(rng):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    op = rng.choice(("gemv", "gemv", "rope", "append", "attn", "attn", "attn"))
    dt = rng.choice(("bf16", "f16"))
    if op == "gemv":
        n, k = 64 * log(4, 448), 64 * log(4, 448)
        while n * k > 5120 * 25600:
            n, k = 64 * max(4, n // 128), 64 * max(4, k // 128)
        return {"op": op, "M": rng.randint(1, 16), "N": n, "K": k, "frac": rng.choice((0.0, 0.05, 0.1, 0.2)), "dtype": dt}
    if op == "rope":
        d = rng.choice((64, 128))
        hk = rng.choice((1, 2, 4, 8))
        return {"op": op, "T": log(1, 8191), "Hq": hk * rng.randint(1, 8), "Hk": hk, "D": d,
                "rot": rng.choice((d, d // 2)), "norm": rng.random() < 0.6, "inter": rng.random() < 0.4,
                "theta": rng.choice((1e4, 5e5, 1e6)), "far": log(64, 131072), "dtype": dt}
    if op == "append":
        p, t = rng.choice((16, 32, 64, 128)), log(1, 8191)
        return {"op": op, "T": t, "H": rng.randint(1, 8), "D": rng.choice((64, 128)), "P": p,
                "pages": t // p + rng.randint(1, 64), "dtype": dt}
    b, ln, hk = log(1, 64), log(1, 16384), rng.choice((1, 2, 4, 8))
    nq = rng.choice((1, 1, 1, rng.randint(2, 8), log(9, 300)))
    if nq > 8:
        b = min(b, 3)
    return {"op": op, "B": b, "len": ln, "ragged": rng.random() < 0.7, "nq": nq, "Hq": hk * rng.randint(1, 8), "Hk": hk,
            "D": rng.choice((64, 128)), "P": rng.choice((16, 32, 64, 128)),
            "window": rng.choice((0, 0, log(1, 4096))), "dtype": dt}


def lengths(case):
    """Cached tokens of every sequence, the call's own query tokens among them."""
    b, ln = case["B"], case["len"]
    if not case["ragged"]:
        return [ln] * b
    return [max(1, ln * ((37 * i + 11) % 64 + 1) // 64) for i in range(b)]


def seen(n, nq, window):
    """(pairs, tokens): what the nq last positions of n tokens attend to, and how many tokens are read."""
    pairs, first = 0, n
    for i in range(nq):
        p = n - nq + i
        if p >= 0:
            lo = max(0, p - window + 1) if window else 0
            pairs, first = pairs + p - lo + 1, min(first, lo)
    return pairs, n - first


def work(case):
    if case["op"] == "gemv":
        m, n, k = case["M"], case["N"], case["K"]
        nb = int(case["frac"] * (n // 64) * (k // 64))
        return {"bytes": n * k * 9 // 16 + nb * (2304 + 4) + 2 * m * (n + k), "flops": 2.0 * m * (n * k + 4096 * nb)}
    if case["op"] == "rope":
        t, h, d = case["T"], case["Hq"] + case["Hk"], case["D"]
        return {"bytes": 4 * t * h * d + 8 * t + 4 * d, "flops": 8.0 * t * h * d}
    if case["op"] == "append":
        n = case["T"] * case["H"] * case["D"]
        return {"bytes": 8 * n + 4 * (n * 9 // 16) + 8 * case["T"], "flops": 10.0 * n}
    pairs = tokens = 0
    for n in lengths(case):
        p, t = seen(n, case["nq"], case["window"])
        pairs, tokens = pairs + p, tokens + t
    q = case["B"] * case["nq"] * case["Hq"]
    return {"bytes": tokens * case["Hk"] * case["D"] * 9 // 8 + q * (4 * case["D"] + 4),
            "flops": 4.0 * pairs * case["Hq"] * case["D"]}


# ----------------------------------------------------------------------------- layouts
def record_maps(d, device):
    """Byte of a 16-token cache record that holds each code pair and scale: four int64
    tensors [16][d/2], [16][d/16] (keys), [16][d/2], [16][d/16] (values).

    Key codes are token rows. A key's scales lie by (token % 8, quarter of the row,
    token / 8), d/64 bytes each. Value codes lie by 16-element group, 8 bytes a token, the
    two halves of 8 tokens swapped in odd groups. Value scales lie by group, the tokens in
    the order 0 1 8 9 2 3 10 11 ..."""
    tok = torch.arange(16, device=device)[:, None]
    byte = torch.arange(d // 2, device=device)[None]
    grp = torch.arange(d // 16, device=device)[None]
    per = d // 64
    kc = tok * (d // 2) + byte
    c = byte // 8
    vc = 8 * d + c * 128 + ((tok // 8) ^ (c % 2)) * 64 + (tok % 8) * 8 + byte % 8
    ks = 16 * d + (tok % 8) * (8 * per) + (grp // per) * (2 * per) + (tok // 8) * per + grp % per
    vs = 17 * d + grp * 16 + (tok % 8 // 2) * 4 + (tok // 8) * 2 + tok % 2
    return kc, ks, vc, vs


def quantize(a, g):
    """NVFP4 of fp32 a [..., 16 n] with tensor scale(s) g (broadcast over a[..., 0]):
    (codes [..., 8 n] bytes, scales [..., n] bytes)."""
    x = a.reshape(*a.shape[:-1], -1, 16)
    g = g.unsqueeze(-1)
    sf = (x.abs().amax(-1) / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = (sf.float() * g).unsqueeze(-1)
    q = x * torch.where(d > 0, 1.0 / d, torch.zeros_like(d))
    m = q.abs()
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0)
            + 8 * torch.signbit(q).to(torch.uint8)).reshape(*a.shape[:-1], -1, 2)
    return code[..., 0] + 16 * code[..., 1], sf.view(torch.uint8)


def values(codes, scales):
    """fp32 val * dec(sf) of packed codes [..., n/2] and scale bytes [..., n/16]."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1)
    v = v.reshape(*codes.shape[:-1], -1, 16) * scales.contiguous().view(torch.float8_e4m3fn).float().unsqueeze(-1)
    return v.reshape(*codes.shape[:-1], -1)


def tile_scales(sf):
    """[rows][groups] scale bytes -> the GEMM's tiled layout (rows in tiles of 128, 64 columns a chunk)."""
    n, q = sf.shape
    t = torch.zeros(-(-n // 128) * 128, q, dtype=torch.uint8, device=sf.device)
    t[:n] = sf
    return t.view(-1, 4, 32, q // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def untile_scales(t, n, q):
    return t.view(-1, q // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, q)[:n]


def packed(resid, g, nt, kt):
    """The packed residual blocks (nt, kt) of resid [n][k], ascending, as the GEMM reads them."""
    n, k = resid.shape
    kb, nblk = k // 64, nt.numel()
    rc, rs = quantize(resid.view(n // 64, 64, kb, 64)[nt, :, kt], g)
    sf = torch.zeros(nblk, 512, dtype=torch.uint8, device="cuda")
    t = 64 * (nt % 2)[:, None, None] + torch.arange(64, device="cuda")[None, :, None]
    sf.scatter_(1, ((t % 32) * 16 + (t // 32) * 4 + torch.arange(4, device="cuda")).reshape(nblk, 256), rs.reshape(nblk, 256))
    kw = -(-kb // 32)
    bits = torch.zeros(n // 64, kw * 32, dtype=torch.int64, device="cuda")
    bits[nt, kt] = 1
    word = (bits.view(n // 64, kw, 32) << torch.arange(32, device="cuda")).sum(-1)
    return {"N": n, "K": k, "nblk": nblk,
            "blk_codes": rc.view(nblk, 8, 8, 2, 16).permute(0, 1, 3, 2, 4).reshape(nblk, 2048).contiguous(),
            "blk_sf": sf, "blk_kt": kt.int(),
            "tile_ptr": torch.searchsorted(nt, torch.arange(n // 64 + 1, device="cuda")).int(),
            "bitmap": torch.where(word >= 2 ** 31, word - 2 ** 32, word).int()}


# ----------------------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    dt = DT[case["dtype"]]
    s = {"case": case}
    if case["op"] == "gemv":
        m, n, k = case["M"], case["N"], case["K"]
        w = (0.02 * rnd(n, k)).to(torch.bfloat16).float()
        kb, nblk = k // 64, int(case["frac"] * (n // 64) * (k // 64))
        sel = torch.randperm((n // 64) * kb, generator=gen, device="cuda")[:nblk].sort().values
        nt, kt = sel // kb, sel % kb
        blk = torch.zeros((n // 64) * kb, device="cuda")
        blk[sel[::3]] = 1.0  # outliers sit in a third of the selected blocks
        w = w * (1 + 19 * (torch.rand(n, k, generator=gen, device="cuda") < 0.1)
                 * blk.view(n // 64, kb).repeat_interleave(64, 0).repeat_interleave(64, 1))
        g = (w.abs().max() / 2688.0).reshape(1)
        codes, sf = quantize(w, g)
        s["w"] = {"rows": n, "cols": k, "codes": codes, "sf": None, "sf_swz": tile_scales(sf), "gscale": g}
        s["r"] = packed(w - values(codes, sf) * g, g, nt, kt) if nblk else None
        hot = 1 + 29 * (torch.rand(k, generator=gen, device="cuda") < 0.01)
        s["x"] = (rnd(m, k) * hot).to(dt)
        s["y"] = torch.empty(m, n, dtype=dt, device="cuda")
        return s
    if case["op"] == "rope":
        t, hq, hk, d = case["T"], case["Hq"], case["Hk"], case["D"]
        qkv = (2.0 * rnd(t, hq + 2 * hk, d)).to(dt)  # the three projections in one tensor, as a fused layer leaves them
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        s["qo"], s["ko"] = torch.empty(t, hq, d, dtype=dt, device="cuda"), torch.empty(t, hk, d, dtype=dt, device="cuda")
        s["wq"] = (1 + 0.1 * rnd(d)).to(dt) if case["norm"] else None
        s["wk"] = (1 + 0.1 * rnd(d)).to(dt) if case["norm"] else None
        s["pos"] = torch.randint(0, case["far"], (t,), generator=gen, device="cuda")
        i = torch.arange(case["rot"] // 2, dtype=torch.float64, device="cuda")
        s["freq"] = case["theta"] ** (-2 * i / case["rot"])
        return s
    h, d, p = case.get("Hk", case.get("H")), case["D"], case["P"]
    s["ks"] = 0.5 + torch.rand(h, generator=gen, device="cuda")  # calibrated tensor scales, one a head
    s["vs"] = 0.5 + torch.rand(h, generator=gen, device="cuda")
    if case["op"] == "append":
        t = case["T"]
        s["pages"] = torch.zeros(case["pages"], h, p // 16, 18 * d, dtype=torch.uint8, device="cuda")
        s["k"], s["v"] = (3 * rnd(t, h, d)).to(dt), rnd(t, h, d).to(dt)
        s["slots"] = torch.randperm(case["pages"] * p, generator=gen, device="cuda")[:t]
        s["ko"], s["vo"] = torch.empty_like(s["k"]), torch.empty_like(s["v"])
        return s
    lens = lengths(case)
    b, nq, most = case["B"], case["nq"], max(lens)
    per = -(-most // p)
    s["table"] = torch.randperm(b * per, generator=gen, device="cuda").int().view(b, per)
    s["len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["cu"] = nq * torch.arange(b + 1, dtype=torch.int32, device="cuda") if nq > 1 else None
    pages = torch.empty(b * per, h, p // 16, 18 * d, dtype=torch.uint8, device="cuda")
    kc, ks, vc, vs = (m.reshape(-1) for m in record_maps(d, "cuda"))
    hot = 1 + 7 * (torch.rand(h, 1, 1, d, generator=gen, device="cuda") < 0.03)
    step = max(1, (1 << 26) // (h * p * d))
    for at in range(0, b * per, step):
        for codes, scales, scale, mul in ((kc, ks, s["ks"], hot), (vc, vs, s["vs"], 1.0)):
            x = (rnd(min(step, b * per - at), h, p // 16, 16, d) * mul).to(dt).float()
            c, f = quantize(x, scale.view(1, h, 1, 1))
            pages[at:at + step, :, :, codes] = c.flatten(3)
            pages[at:at + step, :, :, scales] = f.flatten(3)
    s["pages"] = pages
    s["q"] = rnd(b * nq, case["Hq"], d).to(dt)
    s["o"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(b * nq, case["Hq"], device="cuda")
    return s


# ----------------------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if own:
        from bit_quantized_gemm_zipperengine_b200 import mosaic
        return {"gemv": own_gemv, "rope": own_rope, "append": own_append, "attn": own_attn}[op](mosaic, s)
    return {"gemv": plain_gemv, "rope": plain_rope, "append": plain_append, "attn": plain_attn}[op](s)


def own_gemv(mosaic, s):
    if "handle" not in s:
        s["handle"] = mosaic.Weight(s["w"], s["r"])
    mosaic.mq_gemv(s["x"], s["handle"], s["y"])
    return s["y"]


def own_rope(mosaic, s):
    mosaic.mq_qk_norm_rope(s["q"], s["k"], s["qo"], s["ko"], s["pos"], s["freq"], q_weight=s["wq"], k_weight=s["wk"],
                           eps=1e-6, interleaved=s["case"]["inter"])
    return s["qo"], s["ko"]


def own_append(mosaic, s):
    if "handle" not in s:
        s["handle"] = mosaic.KVCache(s["pages"], s["ks"], s["vs"])
    mosaic.mq_kv_append(s["k"], s["v"], s["slots"], s["handle"])
    mosaic.mq_kv_read(s["handle"], s["slots"], s["ko"], s["vo"])
    return s["ko"], s["vo"]


def own_attn(mosaic, s):
    c = s["case"]
    if "handle" not in s:
        s["handle"] = mosaic.KVCache(s["pages"], s["ks"], s["vs"])
        s["ws"] = mosaic.kv_attention_workspace(s["q"], s["handle"], c["nq"])
    mosaic.mq_kv_attention(s["q"], s["handle"], s["table"], s["len"], s["o"], scale=c["D"] ** -0.5, cu_q=s["cu"],
                           max_q=c["nq"], window=c["window"], lse=s["lse"], ws=s["ws"])
    return s["o"], s["lse"]


def plain_gemv(s):
    w, r = s["w"], s["r"]
    n, k = w["rows"], w["cols"]
    full = values(w["codes"], untile_scales(w["sf_swz"], n, k // 16))
    if r is not None:
        nt = torch.searchsorted(r["tile_ptr"], torch.arange(r["nblk"], device="cuda", dtype=torch.int32), right=True) - 1
        t = 64 * (nt % 2)[:, None, None] + torch.arange(64, device="cuda")[None, :, None]
        at = ((t % 32) * 16 + (t // 32) * 4 + torch.arange(4, device="cuda")).reshape(-1, 256)
        sf = r["blk_sf"].gather(1, at).view(-1, 64, 4)
        codes = r["blk_codes"].view(-1, 8, 2, 8, 16).permute(0, 1, 3, 2, 4).reshape(-1, 64, 32)
        full.view(n // 64, 64, k // 64, 64)[nt, :, r["blk_kt"].long()] += values(codes, sf)
    return ((s["x"].float() @ full.t()) * w["gscale"]).to(s["y"].dtype)


def plain_rope(s):
    c = s["case"]
    rot = c["rot"]
    angle = (s["pos"].double()[:, None] * s["freq"])[:, None]
    cos, sin = angle.cos().float(), angle.sin().float()

    def one(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if c["inter"] else (x[..., :rot // 2], x[..., rot // 2:rot])
        u, v = a * cos - b * sin, b * cos + a * sin
        y = torch.stack((u, v), -1).flatten(-2) if c["inter"] else torch.cat((u, v), -1)
        return torch.cat((y, x[..., rot:]), -1).to(s["qo"].dtype)

    return one(s["q"], s["wq"]), one(s["k"], s["wk"])


def plain_append(s):
    c = s["case"]
    kc, ks, vc, vs = record_maps(c["D"], "cuda")
    slots, p = s["slots"], c["P"]
    page, rec, tok = slots // p, slots % p // 16, slots % 16
    h = torch.arange(c["H"], device="cuda")

    def put_and_get(x, scale, codes, scales):
        b, f = quantize(x.float(), scale.view(1, -1))
        at = (page[:, None, None], h[None, :, None], rec[:, None, None])
        s["pages"][(*at, codes[tok][:, None])] = b
        s["pages"][(*at, scales[tok][:, None])] = f
        b, f = s["pages"][(*at, codes[tok][:, None])], s["pages"][(*at, scales[tok][:, None])]
        d = f.view(torch.float8_e4m3fn).float() * scale.view(1, -1, 1)
        v = values(b, torch.full_like(f, 0x38))  # 0x38: a scale of one
        return (v.unflatten(-1, (-1, 16)) * d.unsqueeze(-1)).flatten(-2).to(x.dtype)

    return put_and_get(s["k"], s["ks"], kc, ks), put_and_get(s["v"], s["vs"], vc, vs)


def plain_attn(s):
    c = s["case"]
    b, nq, hk, d, p = c["B"], c["nq"], c["Hk"], c["D"], c["P"]
    kc, ks, vc, vs = record_maps(d, "cuda")
    rec = s["pages"][s["table"].long()]  # [b][pages][hk][p/16][18 d]
    n = rec.shape[1] * p

    def dense(codes, scales, scale):
        v = values(rec[..., codes.reshape(-1)].unflatten(-1, (16, d // 2)), rec[..., scales.reshape(-1)].unflatten(-1, (16, d // 16)))
        return v.permute(0, 2, 1, 3, 4, 5).reshape(b, hk, n, d) * scale.view(1, hk, 1, 1)

    q = s["q"].float().view(b, nq, hk, -1, d).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, d)
    z = (q @ dense(kc, ks, s["ks"]).transpose(2, 3)).view(b, hk, -1, nq, n) * d ** -0.5
    at = s["len"][:, None].long() - nq + torch.arange(nq, device="cuda")  # positions [b][nq]
    j = torch.arange(n, device="cuda")
    see = j <= at[..., None]
    if c["window"]:
        see &= j > at[..., None] - c["window"]
    z = z.masked_fill(~see[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    e = (z - top.masked_fill(top == -math.inf, 0.0)).exp()
    total = e.sum(-1, keepdim=True)
    o = (e.view(b, hk, -1, n) @ dense(vc, vs, s["vs"])).view(b, hk, -1, nq, d) / total.masked_fill(total == 0, 1.0)
    lse = (total.log() + top.masked_fill(top == -math.inf, 0.0)).squeeze(-1)
    return (o.permute(0, 3, 1, 2, 4).reshape(b * nq, -1, d).to(s["q"].dtype),
            lse.permute(0, 3, 1, 2).reshape(b * nq, -1))


# ------------------------------------------------------------------ the definitions, in 64 bits
def e2m1(c):
    """Value of a code by its bits: sign, two exponent bits, one mantissa bit."""
    e, m = (c >> 1) & 3, (c & 1).double()
    v = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(e.double() - 1))
    return torch.where(c >= 8, -v, v)


def e4m3(c):
    e, m = (c >> 3) & 15, (c & 7).double()
    return torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2(e.double() - 7))


def exact(case, seed):
    s = prepare(case, seed)
    return {"gemv": exact_gemv, "rope": exact_rope, "append": exact_append, "attn": exact_attn}[case["op"]](s)


def exact_gemv(s):
    w, r = s["w"], s["r"]
    n, k = w["rows"], w["cols"]
    x, y = s["x"].double(), []
    for at in range(0, n, 64):  # one block row at a time
        c = w["codes"][at:at + 64].long()
        q = torch.arange(k // 16, device="cuda")[None]
        t = torch.arange(at, at + 64, device="cuda")[:, None]
        f = e4m3(w["sf_swz"][((t // 128) * (k // 64) + q // 4) * 512 + (t % 32) * 16 + (t % 128 // 32) * 4 + q % 4].long())
        row = torch.empty(64, k, dtype=torch.float64, device="cuda")
        row[:, 0::2], row[:, 1::2] = e2m1(c & 15), e2m1(c >> 4)
        row = row * f.repeat_interleave(16, 1)
        if r is not None:
            lo, hi = int(r["tile_ptr"][at // 64]), int(r["tile_ptr"][at // 64 + 1])
            i, j = torch.arange(64, device="cuda")[:, None], torch.arange(32, device="cuda")[None]
            bc = r["blk_codes"][lo:hi][:, (i // 8) * 256 + (j // 16) * 128 + (i % 8) * 16 + j % 16].long()
            t = 64 * (at // 64 % 2) + i
            bs = e4m3(r["blk_sf"][lo:hi][:, (t % 32) * 16 + (t // 32) * 4 + j[:, :4]].long())
            v = torch.stack((e2m1(bc & 15), e2m1(bc >> 4)), -1).reshape(hi - lo, 64, 64) * bs.repeat_interleave(16, 2)
            col = 64 * r["blk_kt"][lo:hi].long()[:, None] + torch.arange(64, device="cuda")
            row.index_add_(1, col.reshape(-1), v.permute(1, 0, 2).reshape(64, -1))
        y.append(x @ row.t() * w["gscale"].double())
    return torch.cat(y, 1)


def exact_rope(s):
    c, out = s["case"], []
    half = c["rot"] // 2
    lo = 2 * torch.arange(half, device="cuda") if c["inter"] else torch.arange(half, device="cuda")
    hi = lo + 1 if c["inter"] else lo + half
    z = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), torch.outer(s["pos"].double(), s["freq"]))
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        y = x.double().clone()
        if w is not None:
            y = y / ((y * y).sum(-1, keepdim=True) / c["D"] + 1e-6).sqrt() * w.double()
        turned = torch.complex(y[..., lo], y[..., hi]) * z[:, None]
        y[..., lo], y[..., hi] = turned.real, turned.imag
        out.append(y)
    return tuple(out)


def exact_append(s):
    """The values that the codes stand for; the codes by the format's own steps, each one
    fp32 operation, so that a value on a border falls on the side that the definition says."""
    grid = np.array(E2M1)

    def one(x, scale):
        a = x.float().cpu().numpy().reshape(*x.shape[:2], -1, 16)
        g = scale.cpu().numpy().reshape(1, -1, 1)
        want = np.abs(a).max(-1) / (np.float32(6) * g)
        e = np.clip(np.floor(np.log2(np.maximum(want.astype(np.float64), 2.0 ** -20))), -6, 8)
        sf = np.minimum(np.rint(want.astype(np.float64) / 2.0 ** (e - 3)) * 2.0 ** (e - 3), 448.0)
        d = (sf.astype(np.float32) * g)[..., None]
        with np.errstate(divide="ignore"):
            q = (a * np.where(d > 0, np.float32(1) / d, np.float32(0))).astype(np.float64)
        m = np.minimum(np.abs(q), 6.0)
        step = np.where(m < 2, 0.5, np.where(m < 4, 1.0, 2.0))
        near = np.rint(m / step) * step
        assert np.isin(near, grid).all()
        return (np.copysign(near, q) * sf[..., None] * g[..., None].astype(np.float64)).reshape(x.shape)

    return one(s["k"], s["ks"]), one(s["v"], s["vs"])


def exact_attn(s):
    c = s["case"]
    nq, hk, d, p, g = c["nq"], c["Hk"], c["D"], c["P"], c["Hq"] // c["Hk"]
    if c["B"] * hk > 256 or sum(lengths(c)) * hk * d > 1 << 30:
        return None
    out = torch.zeros(c["B"] * nq, c["Hq"], d, dtype=torch.float64, device="cuda")
    lse = torch.full((c["B"] * nq, c["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
    maps = record_maps(d, "cuda")
    for b, n in enumerate(lengths(c)):
        tok = torch.arange(n, device="cuda")
        page = s["table"][b].long()[tok // p]
        for h in range(hk):
            kv = []
            for at, sc, scale in ((maps[0], maps[1], s["ks"][h]), (maps[2], maps[3], s["vs"][h])):
                rec = s["pages"][page, h, tok % p // 16]
                code, f = rec.gather(1, at[tok % 16]).long(), e4m3(rec.gather(1, sc[tok % 16]).long())
                v = torch.stack((e2m1(code & 15), e2m1(code >> 4)), -1).view(n, d // 16, 16) * f[..., None]
                kv.append(v.reshape(n, d) * scale.double())
            for i in range(max(0, nq - n), nq):
                at = n - nq + i
                lo = max(0, at - c["window"] + 1) if c["window"] else 0
                if nq > 16:
                    break
                z = s["q"][b * nq + i, h * g:(h + 1) * g].double() @ kv[0][lo:at + 1].t() / math.sqrt(d)
                lse[b * nq + i, h * g:(h + 1) * g] = torch.logsumexp(z, 1)
                out[b * nq + i, h * g:(h + 1) * g] = torch.softmax(z, 1) @ kv[1][lo:at + 1]
            if nq > 16:
                z = torch.einsum("igd,nd->ign", s["q"][b * nq:(b + 1) * nq, h * g:(h + 1) * g].double(), kv[0]) / math.sqrt(d)
                at = n - nq + torch.arange(nq, device="cuda")[:, None]
                no = (tok > at) | ((tok <= at - c["window"]) if c["window"] else torch.zeros_like(tok > at))
                z = z.masked_fill(no[:, None], -math.inf)
                lse[b * nq:(b + 1) * nq, h * g:(h + 1) * g] = torch.logsumexp(z, 2)
                out[b * nq:(b + 1) * nq, h * g:(h + 1) * g] = torch.softmax(z, 2).nan_to_num(0.0) @ kv[1]
    return out, lse
