"""Plain 64-bit references for the operators of include/mosaic_ops.h, and their inputs.

The cache layout is written here from the header's text, one byte at a time."""
from __future__ import annotations

import math

import numpy as np
import torch

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def rounding(ref: torch.Tensor, dtype) -> torch.Tensor:
    """Largest error of one rounding of ref to dtype (subnormal steps included)."""
    fi = torch.finfo(dtype)
    return half_step(dtype) * ref.abs() + fi.smallest_normal * half_step(dtype)


def code_values(c: torch.Tensor) -> torch.Tensor:
    v = torch.tensor(E2M1 + [-x for x in E2M1], dtype=torch.float64, device=c.device)
    return v[c.long()]


def scale_values(c: torch.Tensor) -> torch.Tensor:
    c = c.long()
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2((e - 7).double()))
    return torch.where((c & 127) == 127, torch.full_like(v, math.nan), v)


# ------------------------------------------------------------------ weights
def dense_weight(base: dict, packed: dict | None, mode: str = "both") -> torch.Tensor:
    """fp64 [N][K] of the packed weight without its tensor scale."""
    N, K = base["rows"], base["cols"]
    dev = base["codes"].device
    W = torch.zeros(N, K, dtype=torch.float64, device=dev)
    r, q = torch.arange(N, device=dev)[:, None], torch.arange(K // 16, device=dev)[None]
    if mode != "residual":
        at = ((r // 128) * (K // 64) + q // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + q % 4
        W[:, 0::2], W[:, 1::2] = code_values(base["codes"] & 15), code_values(base["codes"] >> 4)
        W *= scale_values(base["sf_swz"][at]).repeat_interleave(16, 1)
    if packed is not None and packed["nblk"] and mode != "base":
        ptr = packed["tile_ptr"].tolist()
        i, j = torch.arange(64, device=dev)[:, None], torch.arange(32, device=dev)[None]
        for nt in range(N // 64):
            t = 64 * (nt % 2) + i
            for e in range(ptr[nt], ptr[nt + 1]):
                c = packed["blk_codes"][e][(i // 8) * 256 + (j // 16) * 128 + (i % 8) * 16 + j % 16]
                s = scale_values(packed["blk_sf"][e][(t % 32) * 16 + (t // 32) * 4 + j[:, :4]])
                v = torch.stack((code_values(c & 15), code_values(c >> 4)), -1).reshape(64, 64)
                k0 = 64 * int(packed["blk_kt"][e])
                W[64 * nt:64 * nt + 64, k0:k0 + 64] += v * s.repeat_interleave(16, 1)
    return W


def random_weight(N: int, K: int, budget: int, seed: int, dev):
    """A random packed weight (codes and scales drawn directly), its blocks at random places."""
    g = torch.Generator().manual_seed(seed)
    rb = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, dtype=torch.uint8).to(dev)  # noqa: E731
    base = {"rows": N, "cols": K, "codes": rb(0, 256, N, K // 2), "sf": None,
            "sf_swz": rb(0x20, 0x50, -(-N // 128) * 128 * (K // 16)),
            "gscale": torch.tensor([0.0173], dtype=torch.float32, device=dev)}
    if not budget:
        return base, None
    KB = K // 64
    sel = torch.randperm((N // 64) * KB, generator=g)[:budget].sort().values
    bits = torch.zeros(N // 64, -(-KB // 32) * 32, dtype=torch.int64)
    bits[sel // KB, sel % KB] = 1
    word = (bits.view(N // 64, -1, 32) << torch.arange(32)).sum(-1)
    packed = {"N": N, "K": K, "nblk": budget, "blk_codes": rb(0, 256, budget, 2048), "blk_sf": rb(0x10, 0x40, budget, 512),
              "blk_kt": (sel % KB).int().to(dev),
              "tile_ptr": torch.searchsorted(sel // KB, torch.arange(N // 64 + 1)).int().to(dev),
              "bitmap": torch.where(word >= 2 ** 31, word - 2 ** 32, word).int().to(dev)}
    return base, packed


# ------------------------------------------------------------------ heads
def norm_rope(x, w, eps, pos, freq, rot, inter):
    """(fp64 result, fp64 |a| + |b| of the pair that each element is made of)."""
    y = x.double()
    if w is not None:
        y = y / ((y * y).mean(-1, keepdim=True) + eps).sqrt() * w.double()
    mag = y.abs().clone()
    if rot:
        half = rot // 2
        i = torch.arange(half, device=x.device)
        lo, hi = (2 * i, 2 * i + 1) if inter else (i, i + half)
        ang = (pos.double()[:, None] * freq)[:, None]
        a, b = y[..., lo], y[..., hi]
        out = y.clone()
        out[..., lo], out[..., hi] = a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()
        mag[..., lo] = mag[..., hi] = a.abs() + b.abs()
        y = out
    return y, mag


# ------------------------------------------------------------------ cache
def record_bytes(i: int, d: int, D: int):
    """(key code byte, value code byte, key scale byte, value scale byte) of token i, element d."""
    q, L = d // 16, D // 64
    kc = i * (D // 2) + d // 2
    vc = 8 * D + q * 128 + (((i // 8) ^ (q % 2)) * 64) + (i % 8) * 8 + (d % 16) // 2
    ks = 16 * D + (i % 8) * 8 * L + (q // L) * 2 * L + (i // 8) * L + q % L
    vs = 17 * D + q * 16 + (i % 8) // 2 * 4 + (i // 8) * 2 + i % 2
    return kc, vc, ks, vs


def record_maps(D: int, dev):
    m = np.array([[record_bytes(i, d, D) for d in range(D)] for i in range(16)])
    return [torch.from_numpy(m[:, :, j].copy()).to(dev) for j in range(4)]


def cache_rows(pages: torch.Tensor, slots: torch.Tensor, head: int, value: bool) -> torch.Tensor:
    """fp64 [n][D] val * dec(sf) of the slots' rows (without the tensor scale)."""
    P, D = 16 * pages.shape[2], pages.shape[3] // 18
    kc, vc, ks, vs = record_maps(D, pages.device)
    rec = pages[slots // P, head, slots % P // 16]
    i = slots % 16
    c = rec.gather(1, (vc if value else kc)[i])
    d = torch.arange(D, device=pages.device)
    c = torch.where(d % 2 == 0, c & 15, c >> 4)
    return code_values(c) * scale_values(rec.gather(1, (vs if value else ks)[i]))


def random_cache(num_pages: int, P: int, H: int, D: int, seed: int, dev, scales: bool = True):
    """Random codes and scales everywhere, and the heads' tensor scales."""
    g = torch.Generator().manual_seed(seed)
    kc, vc, ks, vs = record_maps(D, "cpu")
    pages = torch.randint(0, 256, (num_pages, H, P // 16, 18 * D), generator=g, dtype=torch.uint8)
    for m in (ks, vs):
        u = m.unique()
        pages[..., u] = torch.randint(0x28, 0x3C, (num_pages, H, P // 16, u.numel()), generator=g, dtype=torch.uint8)
    s = [(0.5 + torch.rand(H, generator=g)).to(dev) if scales else None for _ in range(2)]
    return pages.to(dev), s[0], s[1]


def poison(pages: torch.Tensor, table, lens):
    """Every slot that no sequence holds gets NaN scales and arbitrary codes."""
    P, D = 16 * pages.shape[2], pages.shape[3] // 18
    used = torch.zeros(pages.shape[0] * P, dtype=torch.bool)
    for b, n in enumerate(lens):
        tok = torch.arange(n)
        used[table[b].cpu().long()[tok // P] * P + tok % P] = True
    kc, vc, ks, vs = record_maps(D, "cpu")
    page, slot = torch.nonzero(~used.view(-1, P), as_tuple=True)
    host = pages.cpu()
    for m in (ks, vs):
        host[page[:, None], :, (slot // 16)[:, None], m[slot % 16]] = 0x7F
    pages.copy_(host)


def attention(q, pages, ks, vs, table, lens, nqs, scale, window):
    """fp64 (out, lse, bound parts) of rows in sequence order. bound parts: sum_j p_j |v_j|
    and the largest score magnitude scale * sum |q||k|, for the tolerance."""
    T, Hq, D = sum(nqs), q.shape[1], q.shape[2]
    H, P = pages.shape[1], 16 * pages.shape[2]
    G, dev = Hq // H, q.device
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device=dev)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=dev)
    mass, smax, vmax = torch.zeros_like(out), torch.zeros_like(lse), torch.zeros_like(lse)
    at = 0
    for b, (n, nq) in enumerate(zip(lens, nqs)):
        if n == 0 or nq == 0:
            at += nq
            continue
        tok = torch.arange(n, device=dev)
        slots = table[b].long()[tok // P] * P + tok % P
        pos = n - nq + torch.arange(nq, device=dev)[:, None]
        no = tok > pos
        if window:
            no |= tok <= pos - window
        for h in range(H):
            K = cache_rows(pages, slots, h, False) * (1.0 if ks is None else ks[h].double())
            V = cache_rows(pages, slots, h, True) * (1.0 if vs is None else vs[h].double())
            for g in range(G):
                x = q[at:at + nq, h * G + g].double()
                z = (x @ K.t() * scale).masked_fill(no, -math.inf)
                p = torch.softmax(z, 1).nan_to_num(0.0)
                hh = h * G + g
                out[at:at + nq, hh], lse[at:at + nq, hh] = p @ V, torch.logsumexp(z, 1)
                mass[at:at + nq, hh] = p @ V.abs()
                smax[at:at + nq, hh] = (abs(scale) * (x.abs() @ K.abs().t())).masked_fill(no, 0.0).amax(1)
                vmax[at:at + nq, hh] = V.abs().max()
        at += nq
    return out, lse, mass, smax, vmax
